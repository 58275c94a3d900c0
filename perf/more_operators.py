"""One step of speculative decoding in 4 bits as a program calls it: cases, inputs, plain forms,
exact values.

  rows    weights quantised to 4 bits with group scales, and read back
  gemm    tokens times 4-bit weights: the projections of a token step or of drafted tokens
  tree    attention of a tree of drafted tokens over the paged 4-bit cache
  accept  the accepted tokens' rows moved to the end of what the sequences keep
  copy    pages copied: sequences forked, a pool compacted

`own` selects the library's kernels; otherwise `run` computes the same from elementary torch
operations in 32 bits.
"""
import math

import torch

own = False

OPS = ("rows", "gemm", "tree", "accept", "copy")


# ------------------------------------------------------------------ cases
def listed():
    return [
        # One fused projection of odd sizes, small groups: a model being loaded, layer by layer.
        dict(name="rows_ragged", op="rows", n=1000, k=1500, group=32),
        # The FFN's weight.
        dict(name="rows_ffn", op="rows", n=12288, k=4096, group=128),
        # One token through a 4096-wide projection: latency alone.
        dict(name="gemm_token", op="gemm", m=1, n=4096, k=4096, group=128, out="bf16"),
        # Sixteen drafted tokens through the FFN's projection.
        dict(name="gemm_draft_ffn", op="gemm", m=16, n=12288, k=4096, group=64, out="bf16"),
        # The logits of a batch of drafted tokens over a large vocabulary of an odd size, in FP32.
        dict(name="gemm_head", op="gemm", m=61, n=100003, k=4096, group=128, out="f32"),
        # One user, a tree of 16 tokens, 8192 tokens of context.
        dict(name="tree_one_8k", op="tree", batch=1, lq=16, hq=32, hkv=8, d=128, page=64, lo=8192, hi=8192, ragged=False),
        # A batch of very different contexts (an empty one among them) and trees, narrow heads in
        # groups of an odd size, pages of an odd size.
        dict(name="tree_ragged_batch", op="tree", batch=24, lq=25, hq=28, hkv=4, d=64, page=48, lo=0, hi=6001, ragged=True),
        # Wide trees over long contexts.
        dict(name="tree_wide_long", op="tree", batch=4, lq=64, hq=32, hkv=8, d=128, page=128, lo=16000, hi=32001, ragged=False),
        # One user's accepted tokens: latency.
        dict(name="accept_one", op="accept", batch=1, lq=8, heads=8, d=128, page=64, ctx=1000),
        # A full batch's.
        dict(name="accept_batch", op="accept", batch=128, lq=64, heads=8, d=128, page=16, ctx=500),
        # The last pages of sequences that fork into four.
        dict(name="copy_fork", op="copy", pages=48, heads=8, d=128, page=64),
        # A pool being compacted.
        dict(name="copy_compact", op="copy", pages=5000, heads=8, d=128, page=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = {op: {n: max(work(c)[n] for c in listed() if c["op"] == op) for n in ("bytes", "flops")} for op in OPS}
    while True:
        op = rng.choice(["rows", "gemm", "gemm", "gemm", "tree", "tree", "tree", "accept", "copy"])
        if op in ("rows", "gemm"):
            c = dict(op=op, n=_log(rng, 16, 40000), k=_log(rng, 33, 16384), group=rng.choice([32, 64, 128]))
            if rng.random() < 0.6:  # model widths are mostly round
                c["n"], c["k"] = max(64, c["n"] // 64 * 64), max(64, c["k"] // 64 * 64)
            if op == "gemm":
                c.update(m=_log(rng, 1, 256), out=rng.choice(["bf16", "bf16", "f32"]))
        elif op == "tree":
            hkv = rng.choice([1, 2, 4, 8])
            hi = _log(rng, 1, 32000)
            c = dict(op=op, batch=_log(rng, 1, 64), lq=_log(rng, 1, 64), hq=hkv * rng.choice([1, 4, 7, 8]), hkv=hkv,
                     d=rng.choice([64, 128]), page=rng.choice([16, 32, 48, 64, 128]), lo=rng.choice([0, hi // 2, hi]), hi=hi,
                     ragged=rng.random() < 0.5)
        elif op == "accept":
            c = dict(op=op, batch=_log(rng, 1, 128), lq=_log(rng, 2, 64), heads=rng.choice([1, 2, 4, 8]), d=rng.choice([64, 128]),
                     page=rng.choice([16, 32, 48, 64, 128]), ctx=_log(rng, 1, 500))
        else:
            c = dict(op=op, pages=_log(rng, 1, 5000), heads=rng.choice([1, 2, 4, 8]), d=rng.choice([64, 128]),
                     page=rng.choice([16, 32, 48, 64, 128]))
        if all(work(c)[n] <= most[op][n] for n in most[op]):
            return c


def _spread(n, lo, hi):
    """n whole numbers spread over [lo, hi], the same set for every seed."""
    return [hi] if n == 1 else [lo + (hi - lo) * j // (n - 1) for j in range(n)]


def _nodes(c):
    """The trees' sizes."""
    return _spread(c["batch"], max(1, c["lq"] // 2), c["lq"]) if c.get("ragged") else [c["lq"]] * c["batch"]


def _counts(c):
    """The numbers of accepted tokens."""
    return _spread(c["batch"], 1, c["lq"])


def work(c):
    if c["op"] == "rows":
        n = c["n"] * c["k"]
        groups = c["n"] * -(-c["k"] // c["group"])
        return {"bytes": 2 * n + n / 2 + 4 * groups + 2 * n, "flops": 8 * n}
    if c["op"] == "gemm":
        m, n, k = c["m"], c["n"], c["k"]
        return {"bytes": n * k / 2 + 4 * n * -(-k // c["group"]) + 2 * m * k + (4 if c["out"] == "f32" else 2) * m * n, "flops": 2 * m * n * k}
    if c["op"] == "tree":
        lens, nodes = _spread(c["batch"], c["lo"], c["hi"]), _nodes(c)
        total = sum(lens) + sum(nodes)
        return {"bytes": total * c["hkv"] * (c["d"] + 8) + 4 * c["batch"] * c["lq"] * c["hq"] * c["d"] + 8 * c["batch"] * c["lq"],
                "flops": sum(4 * (n + m / 2) * m * c["hq"] * c["d"] for n, m in zip(lens, nodes))}
    if c["op"] == "accept":
        return {"bytes": 2 * sum(_counts(c)) * c["heads"] * (c["d"] + 8), "flops": 0}
    return {"bytes": 2 * c["pages"] * c["heads"] * c["page"] * (c["d"] + 8), "flops": 0}


# ------------------------------------------------------------------ layouts
# 4-bit weights: row n holds output column n's codes; 32-bit word w of it the codes of k = 8 w .. 8 w + 7,
# the even ones in its low half and the odd ones in its high half, in order from the lowest bits.
# Parameters [group][n]: BF16 scale and BF16 zero.  A code stands for zero + scale * code.
_AT = [0, 16, 4, 20, 8, 24, 12, 28]  # where in its word the code of k % 8 begins


def _weights(q, params, k, group):
    """Words q [n, w] int32 and params [groups, >= n, 2] BF16 -> [n, k] float32."""
    shift = torch.tensor(_AT, dtype=torch.int32, device=q.device)
    codes = ((q[:, :, None] >> shift) & 15).flatten(1)[:, :k].float()
    prm = params[:, :q.shape[0]].float().repeat_interleave(group, 0)[:k].transpose(0, 1)      # [n, k, 2]
    return prm[..., 1] + prm[..., 0] * codes


# The cache's pages: one byte buffer [page][head][block].  A block holds page / 16 records of 16 tokens:
#   K codes  16 x d/2 bytes: a token's row, two codes a byte, the even element in the low half
#   V codes  16 x d/2 bytes, [token / 8][column group of d/8][token % 8 / 2][4 columns][token % 2]
#            in pieces of two bytes (four columns of one token)
#   K scale and zero, 16 x 4 bytes, then V's: BF16 scale in the low half, BF16 zero in the high
def _parts(pool, d):
    """Views of a pool [pages, heads, block]: K codes [pages, heads, records, 16, d/2], V codes
    [pages, heads, records, 2, 8, 4, d/32, 2, 2], parameters [pages, heads, records, 2, 16, 2] BF16."""
    pages, heads, block = pool.shape
    r = pool.view(pages, heads, block // (16 * (d + 8)), 16 * (d + 8))
    k = r[..., :8 * d].unflatten(-1, (16, d // 2))
    v = r[..., 8 * d:16 * d].unflatten(-1, (2, 8, 4, d // 32, 2, 2))
    p = r.view(torch.bfloat16)[..., 8 * d:].unflatten(-1, (2, 16, 2))
    return k, v, p


def _values(codes, params):
    """codes [..., d/2] bytes and params [..., 2] BF16 of rows -> [..., d] float32."""
    both = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float()
    return params[..., 1:].float() + params[..., :1].float() * both


def _rows(pool, d):
    """Every token's K and V of a pool, [pages, heads, page_size, d] float32."""
    k, v, p = _parts(pool, d)
    v = v.permute(0, 1, 2, 3, 5, 7, 4, 6, 8).flatten(6).flatten(3, 5)  # [pages, heads, records, 16, d/2]
    return _values(k, p[..., 0, :, :]).flatten(2, 3), _values(v, p[..., 1, :, :]).flatten(2, 3)


# ------------------------------------------------------------------ inputs
def _codes(g, shape):
    """Bytes of two codes of normal values."""
    n = torch.randn((2,) + shape, generator=g, device="cuda", dtype=torch.bfloat16)
    n = n.mul_(2.86).add_(7.5).round_().clamp_(0, 15).to(torch.uint8)
    return n[0] | (n[1] << 4)


def _pool(g, pages, heads, d, page):
    """A pool of normal rows."""
    pool = _codes(g, (pages, heads, page * (d + 8)))
    params = _parts(pool, d)[2]
    scale = torch.exp(torch.randn(params.shape[:-1], generator=g, device="cuda") * 0.3).mul_(0.35)
    params[..., 0] = scale
    params[..., 1] = scale.mul_(-7.5).add_(torch.randn(params.shape[:-1], generator=g, device="cuda") * 0.2)
    return pool


def _table(g, tokens, page):
    """(page table [batch, width], pages of a pool) of sequences with room for `tokens` (a list)."""
    need = torch.tensor([-(-n // page) for n in tokens], device="cuda")
    width, total = max(1, -(-max(tokens) // page)), sum(-(-n // page) for n in tokens)
    table = torch.full((len(tokens), width), -1, dtype=torch.int32, device="cuda")
    table[torch.arange(width, device="cuda")[None] < need[:, None]] = torch.randperm(total + 1, generator=g, device="cuda", dtype=torch.int32)[:total]
    return table, total + 1


def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * seed + 29)

    def normal(shape, std=1.0, dtype=torch.bfloat16):
        t = torch.randn(shape, generator=g, device="cuda", dtype=dtype)
        return t.mul_(std) if std != 1.0 else t

    def order(values):
        t = torch.tensor(values, dtype=torch.int32, device="cuda")
        return t[torch.randperm(len(values), generator=g, device="cuda")].contiguous()

    s = dict(case=c)
    if c["op"] in ("rows", "gemm"):
        n, k, group = c["n"], c["k"], c["group"]
        words, groups = -(-k // 32) * 4, -(-k // group)       # rows of whole 16 bytes
        ldp = -(-n // 4) * 4
    if c["op"] == "rows":
        # Weights by output column; a few input channels are far larger than the rest.
        w = normal((n, -(-k // 8) * 8), 1.0 / math.sqrt(k))
        w[:, ::61] *= 6.0
        s["w"] = w[:, :k]
        s["q"] = torch.zeros((n, words), dtype=torch.int32, device="cuda")
        s["params"] = torch.zeros((groups, ldp, 2), dtype=torch.bfloat16, device="cuda")
        s["back"] = torch.empty((n, k), dtype=torch.bfloat16, device="cuda")
    elif c["op"] == "gemm":
        # Activations with a few large channels, rows of different size.
        x = torch.randn((c["m"], -(-k // 8) * 8), generator=g, device="cuda")
        x[:, ::97] *= 12.0
        x *= torch.exp(torch.randn((c["m"], 1), generator=g, device="cuda") * 0.5)
        s["x"] = x.to(torch.bfloat16)[:, :k]
        s["q"] = _codes(g, (n, words * 4)).view(torch.int32)
        scale = torch.exp(torch.randn((groups, ldp), generator=g, device="cuda") * 0.3).mul_(0.35 / math.sqrt(k))
        zero = scale * (torch.randn((groups, ldp), generator=g, device="cuda") * 0.5 - 7.5)
        s["params"] = torch.stack((scale, zero), -1).to(torch.bfloat16)
        s["c"] = torch.empty((c["m"], n), dtype=torch.float32 if c["out"] == "f32" else torch.bfloat16, device="cuda")
        if own:
            import dense_gemm_sm_gb300 as dg
            s["ws"] = torch.zeros(dg.dg_gemm_w4_workspace_bytes(c["m"], n, k), dtype=torch.uint8, device="cuda")
    elif c["op"] == "tree":
        b, lq, hq, hkv, d, page = (c[n] for n in ("batch", "lq", "hq", "hkv", "d", "page"))
        ctx, nodes = order(_spread(b, c["lo"], c["hi"])), order(_nodes(c))
        lens = (ctx + nodes).contiguous()
        table, pages = _table(g, lens.tolist(), page)
        pool = _pool(g, pages, hkv, d, page)
        # Slots past a sequence's end hold what an earlier user left, NaN in the scales among it.
        params = _parts(pool, d)[2]
        tail = (lens.long() % page != 0).nonzero()[:, 0]
        if tail.numel():
            last = table[tail, (lens.long()[tail] - 1) // page].long()
            stale = torch.arange(page, device="cuda")[None] >= (lens.long()[tail] % page)[:, None]
            block = params[last]  # [n, heads, records, 2, 16, 2]
            block[stale.view(-1, 1, page // 16, 1, 16, 1).expand(block.shape)] = float("nan")
            params[last] = block
        # Trees: each node's parent is an earlier one, and it sees its ancestors and itself.
        parent = (torch.rand((b, lq), generator=g, device="cuda") * torch.arange(lq, device="cuda")).long()
        mask = torch.ones(lq, dtype=torch.int64, device="cuda") << torch.arange(lq, device="cuda")
        mask = mask[None].repeat(b, 1)
        for i in range(1, lq):
            mask[:, i] |= mask.gather(1, parent[:, i:i + 1])[:, 0]
        qkv = normal((b, lq, (hq + 2 * hkv) * d), 1.5)
        s.update(pool=pool, table=table, lens=lens, nodes=nodes, mask=mask, q=qkv[..., :hq * d], scale=1.0 / math.sqrt(d))
        s["o"] = torch.empty((b, lq, hq * d), dtype=torch.bfloat16, device="cuda")
        if own:
            import dense_gemm_sm_gb300 as dg
            s["cache"] = dg.dg_kv4_cache(pool, pages, page, hkv, d)
            s["ws"] = torch.zeros(dg.dg_attention_kv4_workspace_bytes(b, lq, hq, hkv, d), dtype=torch.uint8, device="cuda")
    elif c["op"] == "accept":
        b, lq, page = c["batch"], c["lq"], c["page"]
        lens = order([c["ctx"] + lq + 3 * j for j in range(b)])
        table, pages = _table(g, lens.tolist(), page)
        s.update(pool=_pool(g, pages, c["heads"], c["d"], page), table=table, lens=lens, counts=order(_counts(c)))
        # Accepted nodes: `count` of the tree's in ascending order, the first among them.
        rank = torch.rand((b, lq), generator=g, device="cuda")
        rank[:, 0] = -1.0
        chosen = rank.argsort(1).argsort(1) < s["counts"][:, None]
        s["path"] = torch.where(chosen, torch.arange(lq, device="cuda")[None], lq).sort(1)[0].to(torch.int32)
        s["new_lens"] = torch.empty_like(lens)
        if own:
            import dense_gemm_sm_gb300 as dg
            s["cache"] = dg.dg_kv4_cache(s["pool"], pages, page, c["heads"], c["d"])
    else:
        n = c["pages"]
        s["pool"] = _pool(g, 2 * n + 1, c["heads"], c["d"], c["page"])
        at = torch.randperm(2 * n + 1, generator=g, device="cuda", dtype=torch.int32)
        s["src"], s["dst"] = at[:n].contiguous(), at[n:2 * n].contiguous()
        if own:
            import dense_gemm_sm_gb300 as dg
            s["cache"] = dg.dg_kv4_cache(s["pool"], 2 * n + 1, c["page"], c["heads"], c["d"])
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import dense_gemm_sm_gb300 as dg
    c = s["case"]
    if c["op"] == "rows":
        q, p = s["q"], s["params"]
        dg.quantize_groups_w4(c["n"], c["k"], c["group"], s["w"], s["w"].stride(0), q, 4 * q.stride(0), p, p.shape[1])
        dg.dequantize_groups_w4(c["n"], c["k"], c["group"], q, 4 * q.stride(0), p, p.shape[1], s["back"], s["back"].stride(0))
        return s["back"], p
    if c["op"] == "gemm":
        x, q, p, y = s["x"], s["q"], s["params"], s["c"]
        dg.gemm_w4_bf16(c["m"], c["n"], c["k"], c["group"], x, x.stride(0), q, 4 * q.stride(0), p, p.shape[1], y, y.stride(0),
                        dg.DG_OUT_F32 if c["out"] == "f32" else dg.DG_OUT_BF16, s["ws"], s["ws"].numel())
        return y
    if c["op"] == "tree":
        q, o = s["q"], s["o"]
        dg.attention_kv4_tree(s["cache"], c["batch"], c["lq"], c["hq"], s["scale"], q, q.stride(1), q.stride(0), s["table"],
                              s["table"].shape[1], s["lens"], s["nodes"], s["mask"], o, o.stride(1), o.stride(0), s["ws"], s["ws"].numel())
        return o
    if c["op"] == "accept":
        dg.kv4_accept(s["cache"], c["batch"], c["lq"], s["table"], s["table"].shape[1], s["lens"], None, s["path"], c["lq"],
                      s["counts"], s["new_lens"])
        return s["pool"], s["new_lens"]
    dg.kv4_copy_pages(s["cache"], c["pages"], s["src"], s["dst"])
    return s["pool"]


def _run_plain(s):
    return {"rows": _plain_rows, "gemm": _plain_gemm, "tree": _plain_tree, "accept": _plain_accept, "copy": _plain_copy}[s["case"]["op"]](s)


def _plain_rows(s):
    c = s["case"]
    n, k, group = c["n"], c["k"], c["group"]
    groups, pad = -(-k // group), -k % group
    w = s["w"].float()
    # The last group may be short: what fills it up takes no part in its range.
    lo = torch.nn.functional.pad(w, (0, pad), value=math.inf).unflatten(1, (groups, group)).amin(-1)
    hi = torch.nn.functional.pad(w, (0, pad), value=-math.inf).unflatten(1, (groups, group)).amax(-1)
    scale = ((hi - lo) / 15.0).to(torch.bfloat16)
    wide = scale.float().repeat_interleave(group, 1)[:, :k]
    code = torch.where(wide > 0, (w - lo.repeat_interleave(group, 1)[:, :k]) / wide, torch.zeros_like(w)).round().clamp(0, 15)
    words = -(-k // 8)
    code = torch.nn.functional.pad(code, (0, 8 * words - k)).to(torch.int32).unflatten(1, (words, 8))
    s["q"][:, :words] = (code << torch.tensor(_AT, dtype=torch.int32, device="cuda")).sum(-1).to(torch.int32)
    s["params"][:, :n, 0] = scale.transpose(0, 1)
    s["params"][:, :n, 1] = lo.to(torch.bfloat16).transpose(0, 1)
    return _weights(s["q"], s["params"], k, group).to(torch.bfloat16), s["params"]


def _plain_gemm(s):
    c = s["case"]
    return (s["x"].float() @ _weights(s["q"], s["params"], c["k"], c["group"]).transpose(0, 1)).to(s["c"].dtype)


def _plain_tree(s):
    c = s["case"]
    b, lq, hq, hkv, d, page = (c[n] for n in ("batch", "lq", "hq", "hkv", "d", "page"))
    n = s["table"].shape[1] * page
    q = s["q"].float().reshape(b, lq, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).flatten(2, 3)         # [b, hkv, g lq, d]
    k, v = _rows(s["pool"][s["table"].clamp(min=0).long()].flatten(0, 1), d)
    k = k.unflatten(0, (b, n // page)).transpose(1, 2).flatten(2, 3)                                  # [b, hkv, n, d]
    v = v.unflatten(0, (b, n // page)).transpose(1, 2).flatten(2, 3)
    pos = torch.arange(n, device="cuda")[None]
    lens, nodes = s["lens"].long()[:, None], s["nodes"].long()[:, None]
    live = (pos < lens)[:, None, :, None]
    k, v = torch.where(live, k, torch.zeros_like(k)), torch.where(live, v, torch.zeros_like(v))
    node = pos - (lens - nodes)                                                                       # [b, n]
    bit = (s["mask"][:, :, None] >> node.clamp(0, 63)[:, None]) & 1                                   # [b, lq, n]
    see = ((node < 0)[:, None] | (bit == 1)) & (pos < lens)[:, None] & (torch.arange(lq, device="cuda")[None] < nodes)[..., None]
    see = see[:, None, None]                                                                          # [b, 1, 1, lq, n]
    w = (q @ k.transpose(2, 3)).unflatten(2, (hq // hkv, lq)) * s["scale"]
    w = torch.where(see, w, torch.full_like(w, -math.inf))
    top = w.amax(-1, keepdim=True)
    w = torch.exp(w - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    total = w.sum(-1, keepdim=True)
    w = w / torch.where(total > 0, total, torch.ones_like(total))
    o = (w.flatten(2, 3) @ v).unflatten(2, (hq // hkv, lq))
    return o.permute(0, 3, 1, 2, 4).reshape(b, lq, hq * d).to(torch.bfloat16)


def _plain_accept(s):
    c = s["case"]
    lq, page = c["lq"], c["page"]
    pk, pv, pp = _parts(s["pool"], c["d"])
    kview = pk.permute(0, 2, 3, 1, 4)                        # [pages, records, 16, heads, d/2]
    vview = pv.permute(0, 2, 3, 5, 7, 1, 4, 6, 8)            # [pages, records, 2, 4, 2, heads, 8, d/32, 2]
    pview = pp.permute(0, 2, 4, 3, 1, 5)                     # [pages, records, 16, 2, heads, 2]
    base = (s["lens"].long() - lq)[:, None]
    at = torch.arange(lq, device="cuda")[None]
    src = base + torch.where(at < s["counts"][:, None], s["path"].long(), at)      # the others stay
    dst = base + at

    def where(pos):
        slot = (torch.gather(s["table"].long(), 1, pos // page) * page + pos % page).flatten()
        return slot // page, slot % page // 16, slot % 16

    (a, r, u), (a2, r2, u2) = where(src), where(dst)
    k, v, p = kview[a, r, u], vview[a, r, u // 8, u % 8 // 2, u % 2], pview[a, r, u]
    kview[a2, r2, u2] = k
    vview[a2, r2, u2 // 8, u2 % 8 // 2, u2 % 2] = v
    pview[a2, r2, u2] = p
    return s["pool"], s["lens"] - lq + s["counts"]


def _plain_copy(s):
    s["pool"][s["dst"].long()] = s["pool"][s["src"].long()]
    return s["pool"]


# ------------------------------------------------------------------ from the definitions, in 64 bits
def exact(c, seed):
    if c["op"] in ("accept", "copy"):
        return None  # bytes that move
    s = prepare(c, seed)
    f = torch.float64
    if c["op"] == "rows":
        # The code is the definition's decision, which is taken in IEEE single precision on the
        # BF16 group (minimum, difference, division); the value it stands for is exact.
        n, k, group = c["n"], c["k"], c["group"]
        w = s["w"].float().cpu().numpy()
        back = torch.empty((n, k), dtype=f)
        params = torch.zeros(s["params"].shape, dtype=f)
        for i, a in enumerate(range(0, k, group)):
            x = w[:, a:a + group]
            lo = x.min(1, keepdims=True)
            step = torch.from_numpy((x.max(1, keepdims=True) - lo) / x.dtype.type(15)).to(torch.bfloat16).float().numpy()
            code = ((x - lo) / step.clip(min=1e-38)).round().clip(0, 15)  # numpy rounds halves to even
            back[:, a:a + group] = torch.from_numpy(lo.astype("float64") + step.astype("float64") * code.astype("float64"))
            params[i, :n, 0], params[i, :n, 1] = torch.from_numpy(step[:, 0]).to(f), torch.from_numpy(lo[:, 0]).to(f)
        return back, params
    if c["op"] == "gemm":
        n, k, group = c["n"], c["k"], c["group"]
        x, out = s["x"].to(f), torch.zeros((c["m"], n), dtype=f, device="cuda")
        for a in range(0, k, group):
            z = min(group, k - a)
            w = torch.empty((n, z), dtype=f, device="cuda")
            for j in range(z):
                word, at = divmod(a + j, 8)
                w[:, j] = (s["q"][:, word] >> (4 * (at // 2) + 16 * (at % 2))).remainder(16).to(f)
            step, zero = s["params"][a // group, :n, 0].to(f), s["params"][a // group, :n, 1].to(f)
            out += x[:, a:a + z] @ (w * step[:, None] + zero[:, None]).T
        return out
    b, lq, hq, hkv, d, page = (c[n] for n in ("batch", "lq", "hq", "hkv", "d", "page"))
    # Byte offsets of a token's 64- or 128-wide rows inside its page's block.
    tok, col = torch.arange(page, device="cuda")[:, None], torch.arange(d, device="cuda")[None]
    base, u = tok // 16 * 16 * (d + 8), tok % 16
    k_at = base + u * (d // 2) + col // 2
    grp, l = col // (d // 8), col % (d // 8)
    v_at = base + 8 * d + ((u // 8 * 32 + grp * 4 + u % 8 // 2) * (d // 8) + l // 4 * 4 + u % 2 * 2 + l % 4 // 2)
    odd = (col % 2 * 4).to(torch.uint8)
    out = torch.zeros((b, lq, hq, d), dtype=f, device="cuda")
    for i, (n, m) in enumerate(zip(s["lens"].tolist(), s["nodes"].tolist())):
        see = torch.ones((m, n), dtype=torch.bool, device="cuda")
        for t in range(m):
            see[:, n - m + t] = (s["mask"][i, :m] >> t).remainder(2) == 1
        for h in range(hkv):
            blk = s["pool"][s["table"][i, :-(-n // page)].long(), h]
            prm = blk.view(torch.bfloat16).to(f)
            at = ((base + 16 * d) // 2 + 2 * u)[:, 0]
            kz, ks = prm[:, at + 1].flatten()[:n], prm[:, at].flatten()[:n]
            vz, vs = prm[:, at + 33].flatten()[:n], prm[:, at + 32].flatten()[:n]
            k = kz[:, None] + ks[:, None] * ((blk[:, k_at] >> odd) & 15).flatten(0, 1)[:n].to(f)
            v = vz[:, None] + vs[:, None] * ((blk[:, v_at] >> odd) & 15).flatten(0, 1)[:n].to(f)
            q = s["q"][i, :m].reshape(m, hkv, hq // hkv, d)[:, h].to(f)                               # [m, g, d]
            w = torch.softmax((q @ k.T * s["scale"]).masked_fill(~see[:, None], -math.inf), -1)
            out[i, :m].view(m, hkv, hq // hkv, d)[:, h] = w @ v
    return out.view(b, lq, hq * d)
