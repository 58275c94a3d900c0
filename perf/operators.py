"""The serving operators as a program calls them: cases, inputs, plain forms, exact values.

Three groups, the parts of one token step of a decoder layer that stand between the GEMMs:

  norm    residual addition and root-mean-square norm, output BF16 or E4M3 with row scales
  append  new keys and values into a paged 4-bit cache, and the rows read back
  attn    attention of the newest tokens over that cache
  moe     a mixture-of-experts layer for few tokens, from the router's logits on

`own` selects the library's kernels; otherwise `run` computes the same from elementary torch
operations in 32 bits.
"""
import math

import torch

own = False

EPS = 1e-5
E4M3_MAX = 448.0


# ------------------------------------------------------------------ cases
def listed():
    return [
        # One token between two projections of a 4096-wide layer: latency alone.
        dict(name="norm_token", op="norm", rows=1, cols=4096, pad=0, x="bf16", r="bf16", out="bf16"),
        # FP32 activations of a ragged width and row stride, no residual.
        dict(name="norm_ragged_f32", op="norm", rows=1000, cols=777, pad=3, x="f32", r="none", out="bf16"),
        # The FFN's 1024 tokens, codes and scales for the FP8 projection.
        dict(name="norm_ffn_e4m3", op="norm", rows=1024, cols=4096, pad=0, x="bf16", r="bf16", out="e4m3"),
        # A long prompt with the residual stream kept in FP32.
        dict(name="norm_prompt_e4m3", op="norm", rows=16384, cols=4096, pad=0, x="bf16", r="f32", out="e4m3"),
        # A prompt's keys and values written to the cache and read back.
        dict(name="append_prompt", op="append", tokens=8192, heads=8, d=128, page=64),
        # One user, one token, 8192 tokens of context.
        dict(name="attn_one_8k", op="attn", batch=1, lq=1, hq=32, hkv=8, d=128, page=64, lo=8192, hi=8192),
        # A full batch of very different lengths (an empty one among them), small pages.
        dict(name="attn_ragged_batch", op="attn", batch=64, lq=1, hq=64, hkv=8, d=128, page=16, lo=0, hi=4100),
        # A few very long contexts.
        dict(name="attn_long", op="attn", batch=8, lq=1, hq=32, hkv=8, d=128, page=128, lo=65000, hi=66001),
        # Four drafted tokens a sequence to verify, 64-wide heads, pages of an odd size.
        dict(name="attn_draft", op="attn", batch=16, lq=4, hq=32, hkv=4, d=64, page=48, lo=1001, hi=8003),
        # One token through small experts: latency.
        dict(name="moe_token_small", op="moe", tokens=1, k=1024, i=512, experts=32, top=4, off=0, renorm=True),
        # One token through two of eight experts of the FFN's size: the weights' bytes.
        dict(name="moe_token_ffn", op="moe", tokens=1, k=4096, i=12288, experts=8, top=2, off=0, renorm=True),
        # A decode batch over many small experts of an odd width, some of them switched off.
        dict(name="moe_batch", op="moe", tokens=48, k=2048, i=1000, experts=64, top=8, off=3, renorm=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = {op: {n: max(work(c)[n] for c in listed() if c["op"] == op) for n in ("bytes", "flops")}
            for op in ("norm", "append", "attn", "moe")}
    while True:
        op = rng.choice(["norm", "append", "attn", "attn", "moe", "moe"])
        if op == "norm":
            c = dict(op=op, rows=_log(rng, 1, 16384), cols=_log(rng, 33, 16384), pad=rng.choice([0, 0, 8, 5]),
                     x=rng.choice(["bf16", "f32"]), r=rng.choice(["none", "bf16", "f32"]), out=rng.choice(["bf16", "e4m3"]))
            if rng.random() < 0.7:  # model widths are mostly round
                c["cols"] = max(64, c["cols"] // 64 * 64)
        elif op == "append":
            c = dict(op=op, tokens=_log(rng, 1, 16384), heads=rng.choice([1, 2, 4, 8, 16]), d=rng.choice([64, 128]),
                     page=rng.choice([16, 32, 48, 64, 128]))
        elif op == "attn":
            hkv = rng.choice([1, 2, 4, 8])
            hi = _log(rng, 1, 66000)
            c = dict(op=op, batch=_log(rng, 1, 128), lq=rng.choice([1, 1, 1, 2, 5]), hq=hkv * rng.choice([1, 4, 7, 8, 16]), hkv=hkv,
                     d=rng.choice([64, 128]), page=rng.choice([16, 32, 48, 64, 128]), lo=rng.choice([0, hi // 2, hi]), hi=hi)
        else:
            e = rng.choice([8, 16, 33, 64, 128])
            c = dict(op=op, tokens=_log(rng, 1, 64), k=_log(rng, 128, 4096) // 8 * 8, i=_log(rng, 64, 8192), experts=e,
                     top=rng.choice([1, 2, 4, 8]), off=rng.choice([0, 0, e // 8]), renorm=rng.random() < 0.5)
        # Every drawn case costs at most its group's largest listed one; all experts' weights
        # are made, whatever the share that is chosen.
        total = 6 * c["k"] * c["i"] * c["experts"] if op == "moe" else 0
        if all(work(c)[n] <= most[op][n] for n in most[op]) and total <= 2.5e9:
            return c


def _lengths(c):
    """The batch's lengths: spread over [lo, hi], the same set for every seed."""
    if c["batch"] == 1:
        return [c["hi"]]
    n = c["batch"]
    return [c["lo"] + (c["hi"] - c["lo"]) * ((j * 61) % n) // (n - 1) for j in range(n)] if n % 61 else \
        [c["lo"] + (c["hi"] - c["lo"]) * j // (n - 1) for j in range(n)]


def _active(c):
    """The number of experts that `tokens` random choices of `top` of the usable ones reach (expected)."""
    usable = c["experts"] - c["off"]
    return usable * (1.0 - (1.0 - min(1.0, c["top"] / usable)) ** c["tokens"])


def work(c):
    if c["op"] == "norm":
        n = c["rows"] * c["cols"]
        xb, rb = {"bf16": 2, "f32": 4}[c["x"]], {"none": 0, "bf16": 2, "f32": 4}[c["r"]]
        out = 2 * n if c["out"] == "bf16" else n + 4 * c["rows"]
        return {"bytes": n * (xb + 2 * rb) + out + 2 * c["cols"], "flops": 6 * n}
    if c["op"] == "append":
        rows = c["tokens"] * c["heads"]
        return {"bytes": rows * (4 * c["d"] + c["d"] + 8 + 4 * c["d"]) + 8 * c["tokens"], "flops": 12 * rows * c["d"]}
    if c["op"] == "attn":
        total = sum(_lengths(c))
        return {"bytes": total * c["hkv"] * (c["d"] + 8) + 4 * c["batch"] * c["lq"] * c["hq"] * c["d"],
                "flops": 4 * total * c["lq"] * c["hq"] * c["d"]}
    pairs = c["tokens"] * min(c["top"], c["experts"] - c["off"])
    return {"bytes": int(_active(c) * 6 * c["k"] * c["i"]) + 4 * c["tokens"] * c["k"] + 4 * c["tokens"] * c["experts"],
            "flops": 6 * pairs * c["k"] * c["i"]}


# ------------------------------------------------------------------ the 4-bit cache's layout
# One byte buffer [page][head][block].  A block holds page / 16 records of 16 tokens:
#   K codes  16 x d/2 bytes: a token's row, two codes a byte, the even element in the low half
#   V codes  16 x d/2 bytes, [token / 8][column group of d/8][token % 8 / 2][4 columns][token % 2]
#            in pieces of two bytes (four columns of one token)
#   K scale and zero, 16 x 4 bytes, then V's: BF16 scale in the low half, BF16 zero in the high
# and a code stands for zero + scale * code.
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
def _type(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * seed + 17)

    def normal(shape, std=1.0, dtype=torch.bfloat16):
        t = torch.randn(shape, generator=g, device="cuda", dtype=dtype)
        return t.mul_(std) if std != 1.0 else t

    s = dict(case=c)
    if c["op"] == "norm":
        rows, cols, ld = c["rows"], c["cols"], c["cols"] + c["pad"]
        # Hidden states: rows of different size, a few columns far larger than the rest.
        size = torch.exp(torch.randn((rows, 1), generator=g, device="cuda") * 0.5)
        x = torch.randn((rows, ld), generator=g, device="cuda")
        x[:, ::97] *= 12.0
        s["x"] = x.mul_(size).to(_type(c["x"]))[:, :cols]
        if c["r"] != "none":
            s["r"] = normal((rows, ld), 2.0, _type(c["r"]))[:, :cols]
        s["gain"] = torch.randn(cols, generator=g, device="cuda").mul_(0.1).add_(1.0).to(torch.bfloat16)
        if own:
            if c["r"] != "none":
                s["h"] = torch.empty((rows, cols), dtype=_type(c["r"]), device="cuda")
            if c["out"] == "bf16":
                s["y"] = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
            else:
                s["q"] = torch.empty((rows, cols), dtype=torch.uint8, device="cuda")
                s["scale"] = torch.empty(rows, dtype=torch.float32, device="cuda")
    elif c["op"] == "append":
        t, h, d, page = c["tokens"], c["heads"], c["d"], c["page"]
        # K and V of a fused projection's output: [tokens][K | V]; K has a few large channels.
        kv = normal((t, 2 * h * d))
        kv.view(t, 2, h, d)[:, 0, :, ::31] *= 4.0
        s["k"], s["v"] = kv[:, :h * d], kv[:, h * d:]
        pages = -(-t // page) + 2
        where = torch.randperm(pages, generator=g, device="cuda")
        at = torch.arange(t, device="cuda") + page // 3  # the sequence starts inside a page
        s["slots"] = where[at // page] * page + at % page
        s["pool"] = torch.zeros((pages, h, page * (d + 8)), dtype=torch.uint8, device="cuda")
        if own:
            import dense_gemm_sm_gb300 as dg
            s["cache"] = dg.dg_kv4_cache(s["pool"], pages, page, h, d)
            s["ko"] = torch.empty((t, h * d), dtype=torch.bfloat16, device="cuda")
            s["vo"] = torch.empty((t, h * d), dtype=torch.bfloat16, device="cuda")
    elif c["op"] == "attn":
        b, lq, hq, hkv, d, page = (c[n] for n in ("batch", "lq", "hq", "hkv", "d", "page"))
        lens = torch.tensor(_lengths(c), dtype=torch.int32, device="cuda")
        lens = lens[torch.randperm(b, generator=g, device="cuda")].contiguous()
        width = max(1, -(-c["hi"] // page))
        need = (lens.long() + page - 1) // page
        cols = torch.arange(width, device="cuda")
        used = cols[None] < need[:, None]
        pages = int(sum(-(-n // page) for n in _lengths(c))) + 1
        table = torch.full((b, width), -1, dtype=torch.int32, device="cuda")
        table[used] = torch.randperm(pages, generator=g, device="cuda", dtype=torch.int32)[:pages - 1]
        # Codes of normal rows; slots past a sequence's end hold what an earlier user left,
        # NaN in the scales among it.
        pool = torch.empty((pages, hkv, page * (d + 8)), dtype=torch.uint8, device="cuda")
        step = max(1, (1 << 26) // pool[0].numel())
        for i in range(0, pages, step):
            part = pool[i:i + step]
            n = torch.randn((2,) + tuple(part.shape), generator=g, device="cuda", dtype=torch.bfloat16)
            n = n.mul_(2.86).add_(7.5).round_().clamp_(0, 15).to(torch.uint8)
            part.copy_(n[0] | (n[1] << 4))
        params = _parts(pool, d)[2]
        shape = params.shape[:-1]
        scale = torch.exp(torch.randn(shape, generator=g, device="cuda") * 0.3).mul_(0.35)
        params[..., 0] = scale
        params[..., 1] = scale.mul_(-7.5).add_(torch.randn(shape, generator=g, device="cuda") * 0.2)
        tail = (lens.long() % page != 0).nonzero()[:, 0]
        if tail.numel():
            last = table[tail, need[tail] - 1].long()
            stale = torch.arange(page, device="cuda")[None] >= (lens.long()[tail] % page)[:, None]
            block = params[last]  # [n, heads, records, 2, 16, 2]
            block[stale.view(-1, 1, page // 16, 1, 16, 1).expand(block.shape)] = float("nan")
            params[last] = block
        # The queries are the first columns of the fused projection's output.
        qkv = normal((b, lq, (hq + 2 * hkv) * d), 1.5)
        s.update(pool=pool, table=table, lens=lens, q=qkv[..., :hq * d], scale=1.0 / math.sqrt(d))
        if own:
            import dense_gemm_sm_gb300 as dg
            s["cache"] = dg.dg_kv4_cache(pool, pages, page, hkv, d)
            s["o"] = torch.empty((b, lq, hq * d), dtype=torch.bfloat16, device="cuda")
            s["ws"] = torch.zeros(dg.dg_attention_kv4_workspace_bytes(b, lq, hq, hkv, d), dtype=torch.uint8, device="cuda")
    else:
        t, k, i, e = c["tokens"], c["k"], c["i"], c["experts"]
        ldi = -(-i // 8) * 8
        s["x"] = normal((t, k))
        logits = torch.randn((t, e), generator=g, device="cuda").mul_(1.5)
        if c["off"]:
            logits[:, torch.randperm(e, generator=g, device="cuda")[:c["off"]]] = -math.inf
        s["logits"] = logits
        s["wg"] = normal((e, k, ldi), 1.0 / math.sqrt(k))
        s["wu"] = normal((e, k, ldi), 1.0 / math.sqrt(k))
        s["wd"] = normal((e, i, k), 1.0 / math.sqrt(i))
        if own:
            import dense_gemm_sm_gb300 as dg
            s["y"] = torch.empty((t, k), dtype=torch.bfloat16, device="cuda")
            s["ws"] = torch.zeros(dg.dg_moe_workspace_bytes(t, k, i, e, c["top"]), dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import dense_gemm_sm_gb300 as dg
    c = s["case"]
    if c["op"] == "norm":
        x, r, h = s["x"], s.get("r"), s.get("h")
        ldr, rt = (r.stride(0), _out(dg, r)) if r is not None else (0, dg.DG_OUT_BF16)
        ldh = h.stride(0) if h is not None else 0
        if c["out"] == "bf16":
            dg.rmsnorm_residual_bf16(c["rows"], c["cols"], x, x.stride(0), _out(dg, x), r, ldr, rt, h, ldh, s["gain"], EPS,
                                     s["y"], s["y"].stride(0))
            return (s["y"],) if h is None else (h, s["y"])
        dg.rmsnorm_residual_e4m3(c["rows"], c["cols"], x, x.stride(0), _out(dg, x), r, ldr, rt, h, ldh, s["gain"], EPS,
                                 s["q"], s["q"].stride(0), s["scale"])
        q = s["q"].view(torch.float8_e4m3fn)
        return (q, s["scale"]) if h is None else (h, q, s["scale"])
    if c["op"] == "append":
        dg.kv4_append(s["cache"], c["tokens"], s["k"], s["k"].stride(0), s["v"], s["v"].stride(0), s["slots"])
        dg.kv4_gather(s["cache"], c["tokens"], s["slots"], s["ko"], s["ko"].stride(0), s["vo"], s["vo"].stride(0))
        return s["ko"], s["vo"]
    if c["op"] == "attn":
        q, o = s["q"], s["o"]
        dg.attention_kv4(s["cache"], c["batch"], c["lq"], c["hq"], s["scale"], q, q.stride(1), q.stride(0), s["table"],
                         s["table"].shape[1], s["lens"], o, o.stride(1), o.stride(0), s["ws"], s["ws"].numel())
        return o
    dg.moe_bf16(c["tokens"], c["k"], c["i"], c["experts"], c["top"], c["renorm"], s["x"], s["x"].stride(0), s["logits"],
                s["logits"].stride(0), s["wg"], s["wg"].stride(1), s["wg"].stride(0), s["wu"], s["wu"].stride(1), s["wu"].stride(0),
                s["wd"], s["wd"].stride(1), s["wd"].stride(0), s["y"], s["y"].stride(0), s["ws"], s["ws"].numel())
    return s["y"]


def _out(dg, t):
    return dg.DG_OUT_F32 if t.dtype == torch.float32 else dg.DG_OUT_BF16


def _run_plain(s):
    return {"norm": _plain_norm, "append": _plain_append, "attn": _plain_attn, "moe": _plain_moe}[s["case"]["op"]](s)


def _plain_norm(s):
    c = s["case"]
    h = s["x"].float()
    if "r" in s:
        h = h + s["r"].float()
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * s["gain"].float()
    if c["out"] == "bf16":
        out = (y.to(torch.bfloat16),)
    else:
        amax = y.abs().amax(1)
        inv = torch.where(amax > 0, E4M3_MAX / amax, torch.zeros_like(amax))
        out = ((y * inv[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), amax / E4M3_MAX)
    return out if "r" not in s else (h.to(s["r"].dtype),) + out


def _quantise(x):
    """Rows x [..., d] float32 -> codes [..., d/2] bytes, params [..., 2] BF16."""
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    scale = ((hi - lo) / 15.0).to(torch.bfloat16)
    code = torch.where(scale > 0, (x - lo) / scale.float(), torch.zeros_like(x)).round().clamp(0, 15).to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), torch.cat((scale, lo.to(torch.bfloat16)), -1)


def _plain_append(s):
    c = s["case"]
    t, h, d, page = c["tokens"], c["heads"], c["d"], c["page"]
    pk, pv, pp = _parts(s["pool"], d)
    at, rec, row = s["slots"] // page, s["slots"] % page // 16, s["slots"] % 16
    kq, kp = _quantise(s["k"].float().view(t, h, d))
    vq, vp = _quantise(s["v"].float().view(t, h, d))
    kview = pk.permute(0, 2, 3, 1, 4)                        # [pages, records, 16, heads, d/2]
    vview = pv.permute(0, 2, 3, 5, 7, 1, 4, 6, 8)            # [pages, records, 2, 4, 2, heads, 8, d/32, 2]
    pview = pp.permute(0, 2, 4, 3, 1, 5)                     # [pages, records, 16, 2, heads, 2]
    kview[at, rec, row] = kq
    vview[at, rec, row // 8, row % 8 // 2, row % 2] = vq.view(t, h, 8, d // 32, 2)
    pview[at, rec, row, 0] = kp
    pview[at, rec, row, 1] = vp
    k = _values(kview[at, rec, row], pview[at, rec, row, 0])
    v = _values(vview[at, rec, row // 8, row % 8 // 2, row % 2].flatten(2), pview[at, rec, row, 1])
    return k.to(torch.bfloat16).view(t, h * d), v.to(torch.bfloat16).view(t, h * d)


def _plain_attn(s):
    c = s["case"]
    b, lq, hq, hkv, d, page = (c[n] for n in ("batch", "lq", "hq", "hkv", "d", "page"))
    n = s["table"].shape[1] * page
    q = s["q"].float().reshape(b, lq, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4)      # [b, hkv, g, lq, d]
    out = torch.empty((b, hkv, hq // hkv, lq, d), dtype=torch.float32, device="cuda")
    pos = torch.arange(n, device="cuda")
    step = max(1, (1 << 28) // (n * hkv * d))                # sequences at a time: bounds the memory
    for i in range(0, b, step):
        k, v = _rows(s["pool"][s["table"][i:i + step].clamp(min=0).long()].flatten(0, 1), d)
        k = k.unflatten(0, (-1, n // page)).transpose(1, 2).flatten(2, 3)            # [step, hkv, n, d]
        v = v.unflatten(0, (-1, n // page)).transpose(1, 2).flatten(2, 3)
        lens = s["lens"][i:i + step].long()
        v = torch.where((pos[None] < lens[:, None])[:, None, :, None], v, torch.zeros_like(v))
        last = lens[:, None] - lq + torch.arange(lq, device="cuda")[None]            # [step, lq]
        see = (pos[None, None] <= last[..., None])[:, None, None]                    # [step, 1, 1, lq, n]
        w = (q[i:i + step].flatten(2, 3) @ k.transpose(2, 3)).unflatten(2, (hq // hkv, lq)) * s["scale"]
        w = torch.where(see, w, torch.full_like(w, -math.inf))
        top = w.amax(-1, keepdim=True)
        w = torch.exp(w - torch.where(top > -math.inf, top, torch.zeros_like(top)))
        total = w.sum(-1, keepdim=True)
        w = w / torch.where(total > 0, total, torch.ones_like(total))
        out[i:i + step] = (w.flatten(2, 3) @ v).unflatten(2, (hq // hkv, lq))
    return out.permute(0, 3, 1, 2, 4).reshape(b, lq, hq * d).to(torch.bfloat16)


def _plain_moe(s):
    c = s["case"]
    x, logits, i = s["x"].float(), s["logits"], c["i"]
    top = logits.amax(1, keepdim=True)
    p = torch.exp(logits - top)
    p = p / p.sum(1, keepdim=True)
    chosen = torch.sort(logits, dim=1, descending=True, stable=True)[1][:, :c["top"]]
    w = torch.gather(p, 1, chosen)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    y = torch.zeros_like(x)
    for e in torch.unique(chosen[w > 0]).tolist():
        t, j = (chosen == e).nonzero(as_tuple=True)
        gate, up = x[t] @ s["wg"][e, :, :i].float(), x[t] @ s["wu"][e, :, :i].float()
        z = gate / (1.0 + torch.exp(-gate)) * up
        y[t] += w[t, j][:, None] * (z @ s["wd"][e].float())
    return y.to(torch.bfloat16)


# ------------------------------------------------------------------ from the definitions, in 64 bits
def exact(c, seed):
    s = prepare(c, seed)
    f = torch.float64
    if c["op"] == "norm":
        h = s["x"].to(f) + (s["r"].to(f) if "r" in s else 0.0)
        y = h / torch.sqrt(h.square().sum(1, keepdim=True) / c["cols"] + EPS) * s["gain"].to(f)
        head = (h,) if "r" in s else ()
        if c["out"] == "bf16":
            return head + (y,)
        amax = torch.linalg.vector_norm(y, ord=math.inf, dim=1)
        return head + (y * (E4M3_MAX / amax.clamp_min(1e-300))[:, None], amax / E4M3_MAX)
    if c["op"] == "append":
        # The code is the definition's decision, which is taken in IEEE single precision on the
        # BF16 row (minimum, difference, division); the value it stands for is exact.
        def value(x):
            x = x.float().reshape(c["tokens"], c["heads"], c["d"]).cpu().numpy()
            lo = x.min(2, keepdims=True)
            step = torch.from_numpy((x.max(2, keepdims=True) - lo) / x.dtype.type(15)).to(torch.bfloat16).float().numpy()
            n = ((x - lo) / step.clip(min=1e-38)).round().clip(0, 15)  # numpy rounds halves to even
            return torch.from_numpy(lo.astype("float64") + step.astype("float64") * n.astype("float64")).flatten(1)
        return value(s["k"]), value(s["v"])
    if c["op"] == "attn":
        b, lq, hq, hkv, d, page = (c[n] for n in ("batch", "lq", "hq", "hkv", "d", "page"))
        if b * hkv > 600:
            return None
        # Byte offsets of a token's 64- or 128-wide rows inside its page's block.
        tok, col = torch.arange(page, device="cuda")[:, None], torch.arange(d, device="cuda")[None]
        base, u = tok // 16 * 16 * (d + 8), tok % 16
        k_at = base + u * (d // 2) + col // 2
        g, l = col // (d // 8), col % (d // 8)
        v_at = base + 8 * d + ((u // 8 * 32 + g * 4 + u % 8 // 2) * (d // 8) + l // 4 * 4 + u % 2 * 2 + l % 4 // 2)
        odd = (col % 2 * 4).to(torch.uint8)
        out = torch.zeros((b, lq, hq, d), dtype=f, device="cuda")
        for i, n in enumerate(s["lens"].tolist()):
            for h in range(hkv if n else 0):
                blk = s["pool"][s["table"][i, :-(-n // page)].long(), h]
                prm = blk.view(torch.bfloat16).to(f)
                where = ((base + 16 * d) // 2 + 2 * u)[:, 0]
                kz, ks = prm[:, where + 1].flatten()[:n], prm[:, where].flatten()[:n]
                vz, vs = prm[:, where + 33].flatten()[:n], prm[:, where + 32].flatten()[:n]
                k = kz[:, None] + ks[:, None] * ((blk[:, k_at] >> odd) & 15).flatten(0, 1)[:n].to(f)
                v = vz[:, None] + vs[:, None] * ((blk[:, v_at] >> odd) & 15).flatten(0, 1)[:n].to(f)
                for j in range(lq):
                    m = n - lq + j + 1
                    if m > 0:
                        q = s["q"][i, j].view(hkv, hq // hkv, d)[h].to(f)
                        out[i, j].view(hkv, hq // hkv, d)[h] = torch.softmax(q @ k[:m].T * s["scale"], -1) @ v[:m]
        return out.view(b, lq, hq * d)
    x, i = s["x"].to(f), c["i"]
    y = torch.zeros_like(x)
    for t in range(c["tokens"]):
        row = s["logits"][t].to(f)
        order = sorted(range(c["experts"]), key=lambda e: (-float(row[e]), e))[:c["top"]]
        p = torch.softmax(row, 0)[order]
        if c["renorm"]:
            p = p / p.sum()
        for e, w in zip(order, p.tolist()):
            if w > 0:
                s.setdefault("of", {}).setdefault(e, []).append((t, w))
    for e, who in s["of"].items():
        t = [a for a, _ in who]
        z = torch.nn.functional.silu(x[t] @ s["wg"][e, :, :i].to(f)) * (x[t] @ s["wu"][e, :, :i].to(f))
        y[t] += (z @ s["wd"][e].to(f)) * torch.tensor([w for _, w in who], dtype=f, device="cuda")[:, None]
    return y
