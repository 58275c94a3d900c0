"""The serving operators written out in float64 (numpy), and their error bounds.

Residual RMS norm, the 4-bit key-value cache's rows and layout, attention over it, and the
mixture-of-experts layer, each from its definition in include/dgemm.h.  Nothing here is shared
with the CUDA sources.  A quantised row's codes are decided in IEEE single precision, which is
part of their definition; everything else is float64.

A bound counts the roundings that the operators' definitions name, each at most half a step of
its type relative to the value (BF16 2^-8, E4M3 2^-4, FP32 2^-24), and the FP32 sums: a sum of n
products taken 16 at a time has n / 16 + 4 roundings, each at most 2^-22 of the sum of absolute
values (twice two units of 2^-24: tensor cores may truncate).
"""
from __future__ import annotations

import numpy as np

BF16, E4M3, F32 = 2.0 ** -8, 2.0 ** -4, 2.0 ** -24


def bf16(x):
    """float32 -> the nearest BF16 value (ties to even), as float32; finite inputs."""
    b = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    b = (b + 0x7FFF + ((b >> np.uint64(16)) & np.uint64(1))) & np.uint64(0xFFFF0000)
    return b.astype(np.uint32).view(np.float32)


def bf16_bits(x):
    return (bf16(x).view(np.uint32) >> 16).astype(np.uint16)


def widen(bits):
    return (np.ascontiguousarray(bits, dtype=np.uint16).astype(np.uint32) << 16).view(np.float32)


def sum_err(n):
    return (n / 16 + 4) * 2.0 ** -22


# ------------------------------------------------------------------ residual RMS norm
def rmsnorm(x, r, gain, eps):
    """(h, y) in float64; r may be None."""
    h = x.astype(np.float64) + (0 if r is None else r.astype(np.float64))
    return h, h / np.sqrt((h * h).sum(1, keepdims=True) / h.shape[1] + eps) * gain.astype(np.float64)


def rmsnorm_codes(y):
    """(y * 448 / amax unrounded, scales) of rows y."""
    amax = np.abs(y).max(1, keepdims=True)
    return y * np.divide(448.0, amax, out=np.zeros_like(amax), where=amax > 0), amax[:, 0] / 448.0


# ------------------------------------------------------------------ 4-bit rows
def kv4_quantise(x):
    """Rows x [..., d] float32 holding BF16 values -> (codes uint8, scale, zero) float32."""
    x = np.asarray(x, dtype=np.float32)
    zero = x.min(-1)
    scale = bf16((x.max(-1) - zero) / np.float32(15))
    s = scale[..., None]
    q = np.divide(x - zero[..., None], s, out=np.zeros_like(x), where=s > 0)
    return np.clip(np.rint(q), 0, 15).astype(np.uint8), scale, zero


def kv4_value(codes, scale, zero):
    """The float64 values that codes stand for."""
    return zero[..., None].astype(np.float64) + scale[..., None].astype(np.float64) * codes


class Kv4Pool:
    """A cache in plain arrays, and its bytes."""

    def __init__(self, pages, page_size, heads, d):
        self.pages, self.page_size, self.heads, self.d = pages, page_size, heads, d
        self.codes = np.zeros((2, pages * page_size, heads, d), np.uint8)
        self.scale = np.zeros((2, pages * page_size, heads), np.float32)
        self.zero = np.zeros((2, pages * page_size, heads), np.float32)

    def append(self, k, v, slots):
        """k, v [tokens, heads, d] float32."""
        for w, x in enumerate((k, v)):
            c, s, z = kv4_quantise(x)
            for i, at in enumerate(slots):
                if 0 <= at < self.pages * self.page_size:
                    self.codes[w, at], self.scale[w, at], self.zero[w, at] = c[i], s[i], z[i]

    def rows(self, which, slots):
        """[len(slots), heads, d] float64 values."""
        s = np.asarray(slots)
        return kv4_value(self.codes[which, s], self.scale[which, s], self.zero[which, s])

    def pack(self):
        """The bytes, element by element from the layout's definition."""
        d = self.d
        rec = 16 * (d + 8)
        out = np.zeros((self.pages, self.heads, self.page_size // 16, rec), np.uint8)
        prm = np.zeros((2,) + self.scale.shape[1:], np.uint32)
        for w in range(2):
            prm[w] = bf16_bits(self.scale[w]).astype(np.uint32) | (bf16_bits(self.zero[w]).astype(np.uint32) << 16)
        for at in range(self.pages * self.page_size):
            page, t = divmod(at, self.page_size)
            r, u = divmod(t, 16)
            dst = out[page, :, r]
            for c in range(d):
                dst[:, u * (d // 2) + c // 2] |= self.codes[0, at, :, c] << (4 * (c & 1))
                g, m = divmod(c, d // 8)
                at_v = ((((u // 8) * 8 + g) * 4 + (u % 8) // 2) * (d // 32) + m // 4) * 4 + (u % 2) * 2 + (m % 4) // 2
                dst[:, 8 * d + at_v] |= self.codes[1, at, :, c] << (4 * (c & 1))
            for w in range(2):
                for b in range(4):
                    dst[:, 16 * d + 64 * w + 4 * u + b] = (prm[w, at] >> (8 * b)) & 255
        return out.reshape(self.pages, self.heads, -1)

    def pack_all(self):
        """pack() with whole arrays, for large pools."""
        d, recs = self.d, self.page_size // 16
        codes = self.codes.reshape(2, self.pages, recs, 16, self.heads, d)
        bits = [bf16_bits(x).astype(np.uint32).reshape(2, self.pages, recs, 16, self.heads) for x in (self.scale, self.zero)]
        out = np.empty((self.pages, self.heads, recs, 16 * (d + 8)), np.uint8)
        two = codes[..., 0::2] | (codes[..., 1::2] << 4)                                        # [2, pages, recs, 16, heads, d/2]
        out[..., :8 * d] = two[0].transpose(0, 3, 1, 2, 4).reshape(out.shape[:3] + (8 * d,))
        v = two[1].reshape(self.pages, recs, 2, 4, 2, self.heads, 8, d // 32, 2)                # half, pair, odd; group, four columns, byte
        out[..., 8 * d:16 * d] = v.transpose(0, 5, 1, 2, 6, 3, 7, 4, 8).reshape(out.shape[:3] + (8 * d,))
        words = np.ascontiguousarray((bits[0] | (bits[1] << 16)).transpose(1, 4, 2, 0, 3)).astype("<u4")
        out[..., 16 * d:] = words.view(np.uint8).reshape(out.shape[:3] + (128,))
        return out.reshape(self.pages, self.heads, -1)


def kv4_attention(pool, q, table, lens, scale):
    """q [batch, Lq, heads_q, d] float64 -> (O, bound) float64, O of a query without keys 0."""
    batch, lq, hq, d = q.shape
    g = hq // pool.heads
    out, bound = np.zeros(q.shape), np.zeros(q.shape)
    for b in range(batch):
        n = int(lens[b])
        if n == 0:
            continue
        page = np.asarray(table[b])[np.arange(n) // pool.page_size]
        ok = (page >= 0) & (page < pool.pages)
        slots = np.where(ok, page, 0) * pool.page_size + np.arange(n) % pool.page_size
        k, v = pool.rows(0, slots), pool.rows(1, slots)
        ks, vs = pool.scale[0, slots].astype(np.float64), pool.scale[1, slots].astype(np.float64)
        vc = pool.codes[1, slots] * vs[..., None]
        for i in range(lq):
            see = ok & (np.arange(n) <= n - lq + i)
            if not see.any():
                continue
            for h in range(hq):
                a = h // g
                s = scale * (k[see, a] @ q[b, i, h])
                p = np.exp(s - s.max())
                p /= p.sum()
                out[b, i, h] = p @ v[see, a]
                # A score's error: the code product taken with codes offset by 128 (at most
                # 143 |q|), and the FP32 operations on the score itself.
                es = scale * (ks[see, a].max() * 143 * np.abs(q[b, i, h]).sum() * sum_err(d)) + \
                    4 * F32 * np.abs(s).max() + 4 * F32 * scale * np.abs(pool.zero[0, slots][see, a]).max() * np.abs(q[b, i, h]).sum()
                # Weights times V's scale rounded to BF16; codes offset by 128 again in FP32.
                off = p @ vs[see, a]
                n_sum = sum_err(see.sum()) + 8 * F32
                bound[b, i, h] = BF16 * np.abs(out[b, i, h]) + (BF16 * (p @ vc[see, a])) + \
                    (2 * es + n_sum) * (p @ np.abs(v[see, a])) + n_sum * 143 * off * 2
    return out, bound


# Rows that make every unit of keys visible in the output: with queries of zeros all weights are equal,
# and each column of the output is the share of the keys whose unit was dealt to it.
def unit_rows(n, d, turn, unit=32):
    """[n, d] float32: row j is 1 in the column of its unit of keys, 0 elsewhere; `turn` deals anew."""
    u = np.arange(n) // unit
    out = np.zeros((n, d), np.float32)
    out[np.arange(n), (u + turn * (1 + u // d)) % d] = 1
    return out


def unit_mean(rows, see, units=0, ctas=152, warps=7):
    """(O, bound) of a query of zeros over the first `see` of unit_rows, in a call of `units` units
    (0: this sequence's own).

    The value 1 has scale s = bf16(1 / 15) and code 15.  A warp adds, two MMAs a unit, codes offset by
    128 (at most 143 s a key), takes 136 s a key away and adds 8 s; its share is the even one, or of
    a CTA that has up to 64 units; then at most 40 parts follow one another.  Weights are 1 and s is BF16, so that P itself is not rounded."""
    s = float(bf16(np.float32(1) / np.float32(15))[0])
    o = rows[:see].astype(np.float64).sum(0) / max(see, 1) * 15 * s
    steps = 2 * (max(-(-64 // warps), -(-max(units, len(rows) // 32 + 1) // (ctas * warps)) + 1)) + 40
    return o, BF16 * o + steps * 2.0 ** -22 * (143 + 136 + 8) * s


# ------------------------------------------------------------------ mixture of experts
def moe_route(logits, top, renorm):
    """[(expert, weight), ...] per token; experts at -inf (or NaN) are left out."""
    out = []
    for row in np.asarray(logits, dtype=np.float64):
        row = np.where(np.isnan(row), -np.inf, row)
        order = sorted((e for e in range(len(row)) if row[e] > -np.inf), key=lambda e: (-row[e], e))[:top]
        if not order:
            out.append([])
            continue
        p = np.exp(row - row[order[0]])
        total = p[order].sum() if renorm else p.sum()
        out.append([(e, p[e] / total) for e in order])
    return out


def moe(x, logits, wg, wu, wd, top, renorm):
    """(Y, bound) float64 for x [T, K], wg and wu [E, K, I], wd [E, I, K] (float32 holding BF16)."""
    x = x.astype(np.float64)
    T, K = x.shape
    I = wg.shape[2]
    y, bound = np.zeros((T, K)), np.zeros((T, K))
    ax = np.abs(x)
    for t, chosen in enumerate(moe_route(logits, top, renorm)):
        for e, w in chosen:
            g, u = x[t] @ wg[e].astype(np.float64), x[t] @ wu[e].astype(np.float64)
            silu = g / (1 + np.exp(-g))
            z = silu * u
            dg = sum_err(K) * (ax[t] @ np.abs(wg[e]).astype(np.float64))
            du = sum_err(K) * (ax[t] @ np.abs(wu[e]).astype(np.float64))
            dz = 1.1 * dg * np.abs(u) + (np.abs(silu) + 1.1 * dg) * du + 8 * F32 * np.abs(z)
            awd = np.abs(wd[e]).astype(np.float64)
            y[t] += w * (z @ wd[e].astype(np.float64))
            # z enters as two BF16 numbers: the second's rounding is what is left.
            bound[t] += w * ((np.abs(z) * BF16 ** 2 + dz * (1 + BF16)) @ awd) + \
                w * (sum_err(I) + (len(chosen) + 32) * F32) * (np.abs(z) @ awd)
    return y, bound + BF16 * np.abs(y) + BF16 * bound
