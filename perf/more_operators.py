"""More operators of a serving step over a paged Cactus Quants KV cache, as they are measured.

Three operators that a layer of a served model needs beside the projections and the cache:

  norm      a block's output through its own norm and gate onto the residual stream, and the next block's norm of
            the sum, as floats or as the int8 activations of the quantised products                       cq_block_norm
  adapters  low-rank adapters of many requests at once, added to the outputs of shared projections       cq_lora_add
  window    attention of new tokens over the paged cache with a sliding window and a few first tokens
            that stay visible                                                                            cq_kv_window_attend

`own = False` computes them with elementary torch operations, `own = True` calls the library.

A cache is one CQ blob of `cap` rows: codes [cap][groups * 16 * width] as bytes, then fp16 norms [cap][groups]; a row is
a token's key (or value) heads side by side in groups of 128, zero-padded. Block b of the pool is the rows
b * block_size .. (b + 1) * block_size - 1.
"""
import math
import random

import numpy as np
import torch

own = False

GROUP = 128
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "i8": torch.int8}
SIZE = {"f32": 4, "f16": 2, "bf16": 2, "i8": 1}
DEV = "cuda"
EPS = 1e-6

# Lloyd-Max levels of the standard normal (2, 3 and 4 bits) and the ternary levels, before the division by sqrt(128).
_LEVELS = {
    2: [-1.5104176, -0.4527800, 0.4527800, 1.5104176],
    3: [-2.1519457, -1.3439093, -0.7560053, -0.2450942, 0.2450942, 0.7560053, 1.3439093, 2.1519457],
    4: [-2.7325896, -2.0690172, -1.6180464, -1.2562312, -0.9423405, -0.6567591, -0.3880483, -0.1283950,
        0.1283950, 0.3880483, 0.6567591, 0.9423405, 1.2562312, 1.6180464, 2.0690172, 2.7325896],
    5: [-1.2240064, 0.0, 1.2240064],
}


def _width(bits):
    """Bits a code takes in memory (the ternary marker 5 stores two-bit crumbs)."""
    return 2 if bits == 5 else bits


def _groups(width):
    return (width + GROUP - 1) // GROUP


def _codebook(bits):
    return (np.array(_LEVELS[bits], dtype=np.float64) / math.sqrt(GROUP)).astype(np.float32)


def _spread(lo, hi, n):
    """n lengths spread evenly over lo..hi."""
    return [lo + (hi - lo) * i // max(1, n - 1) for i in range(n)]


# ------------------------------------------------------------------------------------------------------- the cases

def listed():
    return [
        # One decode step of a small model of width 512: the output projection's fp32 result onto an fp32 residual
        # stream, and the next block's norm. Pure latency.
        dict(name="norm one step", op="norm", tokens=4, d=512, dtype="f32", res="f32", out="f32", post=False, gate="none",
             branch=1.0, residual=1.0, offset=1.0),
        # Drafted tokens of a small batch at an odd width: 16-bit rows, the block's own norm, a gate computed from the
        # block's input, a residual scale.
        dict(name="norm drafts", op="norm", tokens=777, d=1000, dtype="f16", res="f16", out="f16", post=True, gate="sigmoid",
             branch=0.5, residual=0.70710678, offset=0.0),
        # Prefill of long prompts: the quantised product's fp32 rows, bf16 residual stream, int8 activations for the
        # next quantised product (returned as the values they stand for).
        dict(name="norm prompt int8", op="norm", tokens=8190, d=4096, dtype="f32", res="bf16", out="i8", post=True, gate="none",
             branch=1.0, residual=1.0, offset=0.0),
        # The same in bf16 throughout, with a gate for every element.
        dict(name="norm prompt gated", op="norm", tokens=16383, d=2048, dtype="bf16", res="bf16", out="bf16", post=True,
             gate="silu", branch=1.0, residual=1.0, offset=1.0),
        # One token of one request through the query, key and value projections of the small model. Pure latency.
        dict(name="adapters one token", op="adapters", seqs=1, n_lo=1, n_hi=1, n_in=512, outs="512,256,256", rank=8, adapters=4,
             x="f32", w="bf16", none=0),
        # Decode of a batch in which nearly every request has an adapter of its own: the adapters' bytes are what counts.
        dict(name="adapters decode batch", op="adapters", seqs=64, n_lo=1, n_hi=1, n_in=4096, outs="4096,1024,1024", rank=16,
             adapters=60, x="i8", w="bf16", none=4),
        # Drafted tokens of a small batch, ragged: some requests have none, some no adapter; odd sizes.
        dict(name="adapters drafts", op="adapters", seqs=19, n_lo=0, n_hi=32, n_in=1000, outs="777", rank=20, adapters=7,
             x="f16", w="f16", none=3),
        # Prefill of three prompts with an adapter each, onto one wide projection.
        dict(name="adapters prompt", op="adapters", seqs=3, n_lo=1460, n_hi=4000, n_in=4096, outs="4096", rank=64, adapters=3,
             x="bf16", w="bf16", none=0),
        # A single request, one token, a short window: what a chat on a small device-sized model pays in latency.
        dict(name="window one token", op="window", seqs=1, ctx_lo=500, ctx_hi=500, n_lo=1, n_hi=1, window=128, sinks=4, tree=False,
             hq=12, hkv=2, dk=48, dv=64, kb=2, vb=2, bs=16, dtype="f16"),
        # Decode of a large batch whose contexts are several windows long.
        dict(name="window decode batch", op="window", seqs=256, ctx_lo=7900, ctx_hi=8191, n_lo=1, n_hi=1, window=2048, sinks=4,
             tree=False, hq=12, hkv=2, dk=48, dv=64, kb=2, vb=2, bs=64, dtype="f16"),
        # Ragged trees of 0 to 32 drafted tokens, contexts shorter and longer than an odd window, mixed widths.
        dict(name="window drafts", op="window", seqs=19, ctx_lo=0, ctx_hi=4001, n_lo=0, n_hi=32, window=501, sinks=5, tree=True,
             hq=8, hkv=4, dk=64, dv=64, kb=4, vb=3, bs=16, dtype="bf16"),
        # Chunks of long prompts: 256 tokens each behind contexts of up to 131071, grouped heads of 128, four bits.
        dict(name="window prompt chunks", op="window", seqs=16, ctx_lo=0, ctx_hi=131071, n_lo=200, n_hi=256, window=4096, sinks=64,
             tree=False, hq=32, hkv=8, dk=128, dv=128, kb=4, vb=4, bs=64, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "adapters", "window"])
    if op == "norm":
        d = rng.choice([512, 1000, 80, 2048, 4096, 8192, 333, _log(rng, 16, 8192)])
        dtype = rng.choice(["f32", "f16", "bf16"])
        return dict(op=op, tokens=_log(rng, 1, 8190 * 4096 // (2 * d)), d=d, dtype=dtype, res=rng.choice(["f32", dtype, dtype]),
                    out=rng.choice([dtype, "f16", "bf16", "i8"]), post=rng.random() < 0.6,
                    gate=rng.choice(["none", "none", "plain", "sigmoid", "silu"]), branch=rng.choice([1.0, 0.5]),
                    residual=rng.choice([1.0, 0.70710678]), offset=rng.choice([0.0, 1.0]))
    if op == "adapters":
        n_in = rng.choice([512, 1000, 2048, 4096, _log(rng, 32, 4096)])
        outs = rng.choice([(512, 256, 256), (777,), (4096, 1024, 1024), (2048, 2048), (4096,), (_log(rng, 32, 4096),)])
        seqs = _log(rng, 1, 100)
        n_hi = _log(rng, 1, max(2, min(4000, 8190 * 4096 // (2 * seqs * max(n_in, sum(outs))))))
        w = rng.choice(["f16", "bf16"])
        return dict(op=op, seqs=seqs, n_lo=rng.randint(0 if seqs > 1 else 1, n_hi), n_hi=n_hi, n_in=n_in,
                    outs=",".join(map(str, outs)), rank=rng.choice([4, 8, 16, 16, 20, 32, 64]), adapters=rng.randint(1, 2 * min(seqs, 32)),
                    x=rng.choice(["f32", "i8", w]), w=w, none=rng.randint(0, seqs // 4))
    hq, hkv, dk, dv = rng.choice([(8, 4, 64, 64), (12, 2, 48, 64), (32, 8, 128, 128), (16, 16, 96, 96), (8, 1, 256, 256),
                                  (10, 5, 80, 80), (16, 2, 128, 64)])
    seqs = _log(rng, 1, 64)
    n_hi = _log(rng, 1, 64)
    window = _log(rng, 1, 8192)
    sinks = rng.choice([0, 1, 4, 16, 64, 300])
    ctx_hi = _log(rng, 1, min(131071, 1400000 // seqs))
    return dict(op=op, seqs=seqs, ctx_lo=rng.randint(0, ctx_hi), ctx_hi=ctx_hi, n_lo=rng.randint(0 if seqs > 1 else 1, n_hi), n_hi=n_hi,
                window=max(1, min(window, 16 * 256 * 4400 * 32 // (seqs * n_hi * hq) // 2 - sinks)), sinks=sinks, tree=rng.random() < 0.5,
                hq=hq, hkv=hkv, dk=dk, dv=dv, kb=rng.choice([2, 3, 4, 5]), vb=rng.choice([2, 3, 4, 5]), bs=rng.choice([16, 32, 48, 64, 128]),
                dtype=rng.choice(["f16", "bf16"]))


def _outs(c):
    return [int(o) for o in c["outs"].split(",")]


def _visible(c, ctx, n):
    """Cache rows of a request that any of its tokens attends: the sinks, and from the first token's window on."""
    return min(ctx + n, c["sinks"] + c["window"] - 1 + n)


def work(case):
    c = case
    if c["op"] == "norm":
        n = c["tokens"] * c["d"]
        size = SIZE[c["dtype"]] + (SIZE[c["dtype"]] if c["gate"] != "none" else 0) + 2 * SIZE[c["res"]] + SIZE[c["out"]]
        return {"bytes": n * size + 4 * c["tokens"] * (c["out"] == "i8") + 4 * c["d"] * (1 + c["post"]), "flops": 12 * n}
    if c["op"] == "adapters":
        outs, new = _outs(c), _spread(c["n_lo"], c["n_hi"], c["seqs"])
        who = _who(c)
        live = sum(n for n, a in zip(new, who) if a >= 0)
        used = len({a for n, a in zip(new, who) if n and a >= 0})
        per = c["rank"] * sum(c["n_in"] + o for o in outs)
        return {"bytes": sum(new) * 8 * sum(outs) + live * (c["n_in"] * SIZE[c["x"]] + 4 * (c["x"] == "i8")) + used * (2 * per + 4)
                + 4 * (2 * c["seqs"] + 1), "flops": 2 * live * per}
    kg, vg = _groups(c["hkv"] * c["dk"]), _groups(c["hkv"] * c["dv"])
    row = kg * (16 * _width(c["kb"]) + 2) + vg * (16 * _width(c["vb"]) + 2)
    ctx, nodes = _spread(c["ctx_lo"], c["ctx_hi"], c["seqs"]), _spread(c["n_lo"], c["n_hi"], c["seqs"])[::-1]
    rows = [_visible(c, l, n) if n else 0 for l, n in zip(ctx, nodes)]
    total, words = sum(nodes), (max(1, max(nodes)) + 31) // 32
    # a token attends its sinks and its window, itself in it (a tree's tokens at most as many)
    pairs = sum(n * min(l + n, c["sinks"] + c["window"]) for l, n in zip(ctx, nodes))
    return {"bytes": sum(rows) * row + total * (c["hq"] * (c["dk"] + c["dv"]) * 2 + (4 * words + 4) * c["tree"])
            + 4 * (sum(r // c["bs"] + 1 for r in rows) + 2 * c["seqs"] + 1), "flops": 2 * pairs * c["hq"] * (c["dk"] + c["dv"])}


# ------------------------------------------------------------------------------------------------------- the inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _prepare_norm(c, seed):
    g, t, d = _gen(seed), c["tokens"], c["d"]
    dt = DTYPES[c["dtype"]]

    def rows(spread):
        x = torch.randn(t, d, generator=g, device=DEV)
        x *= torch.exp(spread * torch.randn(t, 1, generator=g, device=DEV))
        x[:, :: max(1, d // 7)] *= 6.0  # a few channels of larger size, as residual streams have them
        return x

    x, res = rows(0.5).to(dt), (2.0 * rows(0.3)).to(DTYPES[c["res"]])
    gate = (1.5 * torch.randn(t, d, generator=g, device=DEV)).to(dt) if c["gate"] != "none" else None
    w = 0.1 * torch.randn(d, generator=g, device=DEV) + 1.0 - c["offset"]
    wb = 0.1 * torch.randn(d, generator=g, device=DEV) + 1.0 - c["offset"] if c["post"] else None
    out = DTYPES[c["out"]]
    return dict(c=c, x=x, res=res, gate=gate, w=w, wb=wb, sum=torch.empty_like(res), y=torch.empty(t, d, dtype=out, device=DEV),
                s=torch.empty(t, device=DEV) if c["out"] == "i8" else None,
                values=torch.empty(t, d, dtype=torch.bfloat16, device=DEV) if c["out"] == "i8" else None)


def _who(c):
    """The adapter of each request: the last `none` have none."""
    return [i * 7 % c["adapters"] if i < c["seqs"] - c["none"] else -1 for i in range(c["seqs"])]


def _prepare_adapters(c, seed):
    g, rng = _gen(seed), random.Random(seed)
    outs, dt = _outs(c), DTYPES[c["w"]]
    new, who = _spread(c["n_lo"], c["n_hi"], c["seqs"]), _who(c)
    order = list(range(c["seqs"]))
    rng.shuffle(order)
    new, who = [new[i] for i in order], [who[i] for i in order]
    total, n_in, r, m = sum(new), c["n_in"], c["rank"], c["adapters"]
    x = torch.randn(total, n_in, generator=g, device=DEV)
    x *= torch.exp(0.3 * torch.randn(total, 1, generator=g, device=DEV))
    x_scale = None
    if c["x"] == "i8":  # activations quantised per token, as the shared projection reads them
        x_scale = (x.abs().amax(-1) / 127.0).clamp(min=1e-30)
        x = torch.round(x / x_scale[:, None])
    a = [(torch.randn(m, r, n_in, generator=g, device=DEV) * n_in ** -0.5).to(dt) for o in outs]
    b = [(0.5 * torch.randn(m, o, r, generator=g, device=DEV) * r ** -0.5).to(dt) for o in outs]
    scales = 0.5 + 1.5 * torch.rand(m, generator=g, device=DEV)
    ys = [torch.randn(total, o, generator=g, device=DEV) for o in outs]
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    return dict(c=c, x=x.to(DTYPES[c["x"]]), x_scale=x_scale, a=a, b=b, scales=scales, ys=ys, sums=[torch.empty_like(y) for y in ys],
                cu=_ints(cu), who=_ints(who), most=max(1, max(new)), total=total)


def _random_cache(cap, width, bits, g):
    """A blob of `cap` rows of Gaussian vectors, encoded in chunks: the rotation leaves a Gaussian a Gaussian."""
    groups, w = _groups(width), _width(bits)
    codes = torch.empty(cap, groups * 16 * w, dtype=torch.uint8, device=DEV)
    norms = torch.empty(cap, groups, dtype=torch.float16, device=DEV)
    lv = torch.from_numpy(_codebook(bits)).to(DEV)
    mids = (lv[1:] + lv[:-1]) / 2
    for a in range(0, cap, 1 << 16):
        n = min(1 << 16, cap - a)
        r = torch.randn(n, groups, GROUP, generator=g, device=DEV)
        r *= torch.exp(0.25 * torch.randn(n, groups, 1, generator=g, device=DEV))
        norm = r.norm(dim=-1, keepdim=True)
        code = torch.bucketize(r / norm, mids)
        if bits == 5:
            code = (code - 1) & 3
        codes[a:a + n] = _pack(code.reshape(n, groups * GROUP), w)
        norms[a:a + n] = norm[..., 0].half()
    return torch.cat([codes.reshape(-1), norms.view(torch.uint8).reshape(-1)])


def _prepare_window(c, seed):
    g, rng = _gen(seed), random.Random(seed)
    ctx, nodes = _spread(c["ctx_lo"], c["ctx_hi"], c["seqs"]), _spread(c["n_lo"], c["n_hi"], c["seqs"])[::-1]
    order = list(range(c["seqs"]))
    rng.shuffle(order)
    ctx, nodes = [ctx[i] for i in order], [nodes[i] for i in order]
    if not sum(nodes):
        nodes[0] = 1
    bs, total, most = c["bs"], sum(nodes), max(nodes)
    # Blocks that lie wholly before the window and behind the sinks have gone back to the pool: their table entries are -1.
    pages = [(l + n + bs - 1) // bs for l, n in zip(ctx, nodes)]
    keep = [[b * bs < c["sinks"] or (b + 1) * bs > l - c["window"] + 1 for b in range(p)] for l, p in zip(ctx, pages)]
    blocks = sum(map(sum, keep)) + 2
    perm = torch.randperm(blocks, generator=g, device=DEV).cpu().numpy()
    table, at = np.full((c["seqs"], max(1, max(pages))), -1, dtype=np.int32), 0
    for s, k in enumerate(keep):
        where = np.flatnonzero(np.array(k, dtype=bool))
        table[s, where] = perm[at:at + len(where)]
        at += len(where)
    # trees: each node's parent is one of the few nodes before it (or the context); a node sees its ancestors and itself
    words = (most + 31) // 32
    bits, pos, first = np.zeros((total, words * 32), dtype=bool), np.zeros(total, dtype=np.int32), 0
    for l, n in zip(ctx, nodes):
        for i in range(n):
            parent = max(-1, i - 1 - int(rng.expovariate(0.5))) if c["tree"] else i - 1
            pos[first + i] = pos[first + parent] + 1 if parent >= 0 else l
            if parent >= 0:
                bits[first + i] = bits[first + parent]
            bits[first + i, i] = True
        first += n
    mask = torch.from_numpy(np.packbits(bits, axis=1, bitorder="little").view(np.int32).copy()).to(DEV)
    k_cache = _random_cache(blocks * bs, c["hkv"] * c["dk"], c["kb"], g)
    v_cache = _random_cache(blocks * bs, c["hkv"] * c["dv"], c["vb"], g)
    # queries as a per-head norm leaves them, of somewhat more than unit size so that some tokens stand out
    q = torch.randn(total, c["hq"], c["dk"], generator=g, device=DEV)
    q = 1.5 * q / q.pow(2).mean(-1, keepdim=True).sqrt()
    cu = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int64)
    st = dict(c=c, q=q.to(DTYPES[c["dtype"]]), k_cache=k_cache, v_cache=v_cache, cap=blocks * bs, table=torch.from_numpy(table).to(DEV),
              ctx=_ints(ctx), cu=_ints(cu.tolist()), mask=mask if c["tree"] else None, pos=torch.from_numpy(pos).to(DEV) if c["tree"] else None,
              most=most, longest=max(_visible(c, l, n) for l, n in zip(ctx, nodes)), scale=c["dk"] ** -0.5,
              o=torch.empty(total, c["hq"], c["dv"], dtype=DTYPES[c["dtype"]], device=DEV))
    if own:
        import hadamard_rotated_codebook_gb300 as cq
        st["geom"] = cq.cq_kv_geometry(c["hq"], c["hkv"], c["dk"], c["dv"], c["kb"], c["vb"], _codebook(c["kb"]), _codebook(c["vb"]),
                                       st["scale"])
    return st


def prepare(case, seed):
    return {"norm": _prepare_norm, "adapters": _prepare_adapters, "window": _prepare_window}[case["op"]](case, seed)


# --------------------------------------------------------------------------------------------------- the plain forms

def _rms(x, weight):
    return x * torch.rsqrt(x.pow(2).mean(-1, keepdim=True) + EPS) * weight


def _norm_plain(st):
    c = st["c"]
    z = st["x"].float()
    if c["post"]:
        z = _rms(z, st["wb"] + c["offset"])
    if c["gate"] != "none":
        gate = st["gate"].float()
        z = z * (gate if c["gate"] == "plain" else torch.sigmoid(gate) * (gate if c["gate"] == "silu" else 1.0))
    r = c["residual"] * st["res"].float() + c["branch"] * z
    y = _rms(r, st["w"] + c["offset"])
    if c["out"] == "i8":
        top = y.abs().amax(-1, keepdim=True)
        s = torch.where(top > 0, top / 127.0, 1.0)
        return {"sum": r.to(st["sum"].dtype), "scale": s[:, 0], "y": (torch.round(y / s).clamp(-128, 127) * s).to(torch.bfloat16)}
    return {"sum": r.to(st["sum"].dtype), "y": y.to(st["y"].dtype)}


def _adapters_plain(st):
    cu, who = st["cu"].long(), st["who"].long()
    token = torch.arange(st["total"], device=DEV)
    seq = torch.searchsorted(cu[1:].contiguous(), token, right=True)
    # the requests side by side, padded to the longest
    at = (cu[:-1, None] + torch.arange(st["most"], device=DEV)[None]).clamp(max=max(0, st["total"] - 1))
    x = st["x"].float()
    if st["x_scale"] is not None:
        x = x * st["x_scale"][:, None]
    x = x[at]
    pick = who.clamp(min=0)
    scale = torch.where(who >= 0, st["scales"][pick], 0.0)

    def one(y, a, b):
        u = torch.bmm(x, a[pick].float().transpose(1, 2)) * scale[:, None, None]
        d = torch.bmm(u, b[pick].float().transpose(1, 2))
        return y + d[seq, token - cu[seq]]

    return [one(y, a, b) for y, a, b in zip(st["ys"], st["a"], st["b"])]


def _hadamard(dtype):
    i = torch.arange(GROUP, device=DEV)
    both = i[:, None] & i[None]
    both = both ^ (both >> 4)
    both = both ^ (both >> 2)
    odd = (both ^ (both >> 1)) & 1
    return (1 - 2 * odd).to(dtype) / math.sqrt(GROUP)


def _pack(codes, w):
    """codes [n][k] -> bytes [n][k * w / 8], least significant bit first."""
    n, k = codes.shape
    if w == 3:
        c = codes.reshape(n, k // 8, 8).to(torch.int32)
        word = (c << (3 * torch.arange(8, device=DEV, dtype=torch.int32))).sum(-1)
        return ((word[..., None] >> (8 * torch.arange(3, device=DEV))) & 255).to(torch.uint8).reshape(n, -1)
    per = 8 // w
    c = codes.reshape(n, k // per, per).to(torch.int32)
    return (c << (w * torch.arange(per, device=DEV, dtype=torch.int32))).sum(-1).to(torch.uint8)


def _unpack(data, w):
    """bytes [..., m] -> codes [..., m * 8 / w]"""
    lead = data.shape[:-1]
    if w == 3:
        b = data.reshape(*lead, -1, 3).to(torch.int32)
        word = b[..., 0] | (b[..., 1] << 8) | (b[..., 2] << 16)
        return ((word[..., None] >> (3 * torch.arange(8, device=DEV, dtype=torch.int32))) & 7).reshape(*lead, -1)
    per = 8 // w
    return ((data[..., None] >> (w * torch.arange(per, device=DEV, dtype=torch.uint8))) & ((1 << w) - 1)).to(torch.int32).reshape(*lead, -1)


def _views(cache, cap, width, bits):
    groups, w = _groups(width), _width(bits)
    n = cap * groups * 16 * w
    return cache[:n].view(cap, groups * 16 * w), cache[n:].view(torch.float16).view(cap, groups)


def _by_code(bits):
    """Level of each stored code (a ternary crumb is a signed two-bit number)."""
    lv = _codebook(bits).tolist()
    if bits == 5:
        lv = [lv[1], lv[2], 2 * lv[0], lv[0]]
    return torch.tensor(lv, dtype=torch.float32, device=DEV)


def _dense(cache, cap, width, bits, rows):
    codes, norms = _views(cache, cap, width, bits)
    c = _by_code(bits)[_unpack(codes[rows], _width(bits)).long()]
    c = c.view(*rows.shape, -1, GROUP) * norms[rows].float()[..., None]
    return (c @ _hadamard(torch.float32)).flatten(-2)[..., :width]


def _window_plain(st):
    c = st["c"]
    s_n, t_n, l_n, bs, total = c["seqs"], max(1, st["most"]), st["longest"], c["bs"], st["q"].shape[0]
    ctx, cu = st["ctx"].long(), st["cu"].long()
    n = cu[1:] - cu[:-1]
    # only the rows that some token attends: the sinks, then what follows the first token's window's beginning
    first = (ctx - c["window"] + 1).clamp(min=c["sinks"])
    i = torch.arange(l_n, device=DEV)[None]
    pos = torch.where(i < c["sinks"], i, i - c["sinks"] + first[:, None])
    real = pos < (ctx + n)[:, None]
    p = torch.where(real, pos, 0)
    rows = torch.gather(st["table"].long(), 1, p // bs) * bs + p % bs
    rows = torch.where(real, rows, 0).clamp(min=0)
    k = _dense(st["k_cache"], st["cap"], c["hkv"] * c["dk"], c["kb"], rows).view(s_n, l_n, c["hkv"], c["dk"])
    v = _dense(st["v_cache"], st["cap"], c["hkv"] * c["dv"], c["vb"], rows).view(s_n, l_n, c["hkv"], c["dv"])
    node = torch.arange(t_n, device=DEV)
    at = (cu[:-1, None] + node[None]).clamp(max=total - 1)
    q = st["q"].float()[at].view(s_n, t_n, c["hkv"], c["hq"] // c["hkv"], c["dk"])
    j = pos - ctx[:, None]  # which new token a row holds
    jj = j.clamp(0, t_n - 1)
    if st["mask"] is None:
        where, place = ctx[:, None] + node[None], pos
        seen = jj[:, None] <= node[None, :, None]
    else:
        where = st["pos"].long()[at]
        place = torch.where(j < 0, pos, torch.gather(where, 1, jj))
        word = torch.gather(st["mask"][at], 2, (jj // 32)[:, None].expand(s_n, t_n, l_n))
        seen = ((word >> (jj % 32)[:, None].to(torch.int32)) & 1).bool()
    near = (where[:, :, None] - place[:, None] < c["window"]) | (place < c["sinks"])[:, None]
    seen = ((j < 0)[:, None] | seen) & near & real[:, None]
    logit = torch.einsum("stgrd,slgd->sgrtl", q, k) * st["scale"]
    logit = logit.masked_fill(~seen[:, None, None], -math.inf)
    top = logit.amax(-1, keepdim=True)
    p = torch.exp(logit - torch.where(top > -math.inf, top, 0.0))
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-38)
    o = torch.einsum("sgrtl,slgd->stgrd", p, v).reshape(s_n, t_n, c["hq"], c["dv"])
    seq = torch.searchsorted(cu[1:].contiguous(), torch.arange(total, device=DEV), right=True)
    return o[seq, torch.arange(total, device=DEV) - cu[seq]].to(st["o"].dtype)


# ------------------------------------------------------------------------------------------------------------- a pass

def run(state):
    st, c = state, state["c"]
    if not own:
        return {"norm": _norm_plain, "adapters": _adapters_plain, "window": _window_plain}[c["op"]](st)
    import hadamard_rotated_codebook_gb300 as cq
    if c["op"] == "norm":
        gate = None if c["gate"] in ("none", "plain") else c["gate"]
        out = cq.cq_block_norm(st["x"], st["res"], st["w"], post_norm=c["post"], branch_weight=st["wb"], gate=st["gate"], gate_act=gate,
                               branch_scale=c["branch"], residual_scale=c["residual"], eps=EPS, weight_offset=c["offset"],
                               residual_out=st["sum"], out=st["y"], out_scale=st["s"])
        if c["out"] == "i8":  # what the codes stand for, in the 16 bits of such a model's activations
            return {"sum": out[0], "scale": out[2], "y": torch.mul(out[1], out[2][:, None], out=st["values"])}
        return {"sum": out[0], "y": out[1]}
    if c["op"] == "adapters":
        return cq.cq_lora_add(st["ys"], st["x"], st["a"], st["b"], st["who"], st["cu"], scales=st["scales"], x_scale=st["x_scale"],
                              outs=st["sums"])
    return cq.cq_kv_window_attend(st["geom"], st["q"], st["k_cache"], st["v_cache"], st["cap"], st["table"], c["bs"], st["ctx"], st["cu"],
                                  st["mask"], st["most"], c["window"], c["sinks"], positions=st["pos"], o=st["o"])


# ------------------------------------------------------------------------------------------------------ in 64 bits

def _exact_norm(c, st):
    def unit(x, w):
        return x / (x.square().sum(-1, keepdim=True) / c["d"] + EPS).sqrt() * (c["offset"] + w.double())

    z = st["x"].double()
    if c["post"]:
        z = unit(z, st["wb"])
    if c["gate"] != "none":
        g = st["gate"].double()
        z = z * {"plain": g, "sigmoid": 1 / (1 + torch.exp(-g)), "silu": g / (1 + torch.exp(-g))}[c["gate"]]
    r = st["res"].double() * c["residual"] + z * c["branch"]
    y = unit(r, st["w"])
    if c["out"] != "i8":
        return {"sum": r, "y": y}
    s = y.abs().max(-1).values / 127
    s = torch.where(s > 0, s, torch.ones_like(s))
    return {"sum": r, "scale": s, "y": (y / s[:, None]).round() * s[:, None]}


def _exact_adapters(c, st):
    cu, who = st["cu"].tolist(), st["who"].tolist()
    out = [y.double() for y in st["ys"]]
    for s in range(c["seqs"]):
        if who[s] < 0 or cu[s] == cu[s + 1]:
            continue
        rows = slice(cu[s], cu[s + 1])
        x = st["x"][rows].double()
        if st["x_scale"] is not None:
            x = x * st["x_scale"][rows].double()[:, None]
        for y, a, b in zip(out, st["a"], st["b"]):
            y[rows] += (x @ a[who[s]].double().T) @ b[who[s]].double().T * st["scales"][who[s]].double()
    return out


def _exact_rows(cache, cap, width, bits, rows):
    """The dequantised rows, from single bits."""
    groups, w = _groups(width), _width(bits)
    stride = groups * 16 * w
    data = cache[:cap * stride].view(cap, stride)[rows]
    bit = ((data[..., None].int() >> torch.arange(8, device=DEV, dtype=torch.int32)) & 1).view(len(rows), groups * GROUP, w)
    code = (bit * (2 ** torch.arange(w, device=DEV, dtype=torch.int32))).sum(-1)
    lv = torch.from_numpy(_codebook(bits)).to(DEV).double()
    if bits == 5:
        level = lv[2] * torch.where(code >= 2, code - 4, code).double()
    else:
        level = lv[code]
    norm = cache[cap * stride:].view(torch.float16).view(cap, groups)[rows].double()
    sign = torch.ones(1, 1, dtype=torch.float64, device=DEV)
    for _ in range(7):  # Sylvester's matrix, doubled seven times
        sign = torch.cat([torch.cat([sign, sign], 1), torch.cat([sign, -sign], 1)], 0)
    return torch.matmul(level.view(len(rows), groups, GROUP), sign / math.sqrt(GROUP)).mul(norm[..., None]).view(len(rows), -1)[:, :width]


def _exact_window(c, st):
    table, ctx, cu = st["table"].cpu().numpy().astype(np.int64), st["ctx"].tolist(), st["cu"].tolist()
    mask = None if st["mask"] is None else st["mask"].cpu().numpy()
    out = torch.zeros(st["q"].shape[0], c["hq"], c["dv"], dtype=torch.float64, device=DEV)
    per = c["hq"] // c["hkv"]
    for s in range(c["seqs"]):
        a, n, l = cu[s], cu[s + 1] - cu[s], ctx[s]
        if not n:
            continue
        at = l + np.arange(n) if st["pos"] is None else st["pos"][a:a + n].cpu().numpy().astype(np.int64)
        if mask is None:
            inner = np.tri(n, dtype=bool)
        else:
            inner = np.unpackbits(mask[a:a + n].view(np.uint8), axis=1, bitorder="little")[:, :n].astype(bool)
        p = np.arange(l + n)
        p = p[(p < c["sinks"]) | (p >= l) | (p > l - c["window"])]  # rows that the first token's window leaves to any
        place = np.where(p < l, p, at[np.maximum(p - l, 0)])
        see = np.where(p[None] < l, True, inner[:, np.maximum(p - l, 0)])
        see &= (place[None] < c["sinks"]) | (at[:, None] - place[None] < c["window"])
        shut = torch.from_numpy(~see).to(DEV)
        rows = torch.from_numpy(table[s, p // c["bs"]] * c["bs"] + p % c["bs"]).to(DEV)
        k = _exact_rows(st["k_cache"], st["cap"], c["hkv"] * c["dk"], c["kb"], rows)
        v = _exact_rows(st["v_cache"], st["cap"], c["hkv"] * c["dv"], c["vb"], rows)
        for h in range(c["hq"]):
            g = h // per
            x = st["q"][a:a + n, h].double() @ k[:, g * c["dk"]:(g + 1) * c["dk"]].T * st["scale"]
            x[shut] = -math.inf
            out[a:a + n, h] = torch.nan_to_num(torch.softmax(x, -1)) @ v[:, g * c["dv"]:(g + 1) * c["dv"]]
    return out


def exact(case, seed):
    if case["op"] == "window" and work(case)["flops"] > 4e12:  # 64-bit products at about half a TFLOP/s
        return None
    st = prepare(case, seed)
    return {"norm": _exact_norm, "adapters": _exact_adapters, "window": _exact_window}[case["op"]](case, st)
