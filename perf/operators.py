"""The operators around a paged Cactus Quants KV cache, as they are measured.

Four operators make up the attention half of a serving step that verifies drafted tokens (a plain decode step is the
case of one drafted token):

  rope    per-head norms of queries and keys and their position rotation, one pass         cq_qk_norm_rope
  plan    block tables and slot maps of the step's new tokens, from the request lengths    cq_kv_plan
  write   the new tokens' keys and values quantised into the cache at their slots          cq_kv_write_slots
  attend  attention of every drafted token over its context and its ancestors in the tree  cq_kv_tree_attend

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
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
DEV = "cuda"

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
        # One decode step of a small model: 8 query heads of 64 over 4 key heads, fp32 projections straight from the
        # matrix product; queries go to attention in fp16, keys to the cache writer in fp32. Pure latency.
        dict(name="rope one step", op="rope", tokens=4, hq=8, hkv=4, d=64, rot=64, interleaved=False, packed=False,
             dtype="f32", q_out="f16", k_out="f32", offset=1.0, far=8192),
        # A verification step of a batch: 37 requests with 21 drafted tokens each, heads cut out of one projection.
        dict(name="rope drafts", op="rope", tokens=777, hq=12, hkv=2, d=48, rot=48, interleaved=True, packed=True,
             dtype="f16", q_out="f16", k_out="f32", offset=0.0, far=8192),
        # Prefill of a long prompt, bf16, partial rotation, far positions.
        dict(name="rope prefill", op="rope", tokens=16383, hq=32, hkv=8, d=128, rot=96, interleaved=False, packed=True,
             dtype="bf16", q_out="bf16", k_out="bf16", offset=0.0, far=1000000),
        # One drafting round of a small batch.
        dict(name="plan drafts", op="plan", seqs=33, len_lo=0, len_hi=8000, new_lo=0, new_hi=32, bs=16, slack=40),
        # A full server: decode steps and chunks of prompts in one batch, ragged, blocks of 64.
        dict(name="plan mixed", op="plan", seqs=1021, len_lo=1, len_hi=32000, new_lo=1, new_hi=300, bs=64, slack=1000),
        # The drafted tokens of one small batch: 2 key heads of 48 and value heads of 64, fp32, CQ2.
        dict(name="write drafts", op="write", rows=77, hkv=2, dk=48, dv=64, kb=2, vb=2, dtype="f32", bs=16),
        # A prompt's keys and values, 8 heads of 128 in bf16, four bits for keys and three for values.
        dict(name="write prompt", op="write", rows=8190, hkv=8, dk=128, dv=128, kb=4, vb=3, dtype="bf16", bs=64),
        # A single request, one token at a time, short context: what a chat pays in latency.
        dict(name="attend one token", op="attend", seqs=1, ctx_lo=500, ctx_hi=500, n_lo=1, n_hi=1, hq=12, hkv=2, dk=48,
             dv=64, kb=2, vb=2, bs=16, dtype="f16"),
        # Decode of a large batch at the model's whole context of 8192: the cache is what counts.
        dict(name="attend decode batch", op="attend", seqs=256, ctx_lo=7900, ctx_hi=8191, n_lo=1, n_hi=1, hq=12, hkv=2,
             dk=48, dv=64, kb=2, vb=2, bs=64, dtype="f16"),
        # Ragged requests with trees of 0 to 32 drafted tokens, an empty context among them, mixed widths.
        dict(name="attend drafts", op="attend", seqs=19, ctx_lo=0, ctx_hi=4001, n_lo=0, n_hi=32, hq=8, hkv=4, dk=64,
             dv=64, kb=4, vb=3, bs=16, dtype="bf16"),
        # One request with a very long context and a tree of 64.
        dict(name="attend long context", op="attend", seqs=1, ctx_lo=131071, ctx_hi=131071, n_lo=64, n_hi=64, hq=32,
             hkv=8, dk=128, dv=128, kb=2, vb=2, bs=128, dtype="bf16"),
        # A verification step of a server: 32 requests with trees of up to 64, grouped heads of 128, four bits.
        dict(name="attend server", op="attend", seqs=32, ctx_lo=2000, ctx_hi=8001, n_lo=40, n_hi=64, hq=32, hkv=8,
             dk=128, dv=128, kb=4, vb=4, bs=64, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "plan", "write", "attend", "attend"])
    if op == "rope":
        hq, hkv, d = rng.choice([(8, 4, 64), (12, 2, 48), (32, 8, 128), (16, 16, 96), (8, 1, 256), (5, 5, 80), (3, 1, 34)])
        rot = rng.choice([d, d, d // 4 * 2, 16])
        dtype = rng.choice(["f32", "f16", "bf16"])
        return dict(op=op, tokens=_log(rng, 1, 16383 * 40 * 128 // ((hq + hkv) * d) // 2), hq=hq, hkv=hkv, d=d, rot=rot,
                    interleaved=rng.random() < 0.4, packed=rng.random() < 0.6, dtype=dtype,
                    q_out=rng.choice([dtype, "f16", "bf16"]), k_out=rng.choice([dtype, "f32"]),
                    offset=rng.choice([0.0, 1.0]), far=_log(rng, 100, 1000000))
    if op == "plan":
        seqs = _log(rng, 1, 1500)
        new_hi = _log(rng, 1, max(1, min(2000, 150000 // seqs)))
        return dict(op=op, seqs=seqs, len_lo=rng.randint(0, 50), len_hi=_log(rng, 60, 32000), new_lo=rng.randint(0, new_hi),
                    new_hi=new_hi, bs=rng.choice([16, 32, 64, 128]), slack=_log(rng, 1, 1000))
    hq, hkv, dk, dv = rng.choice([(8, 4, 64, 64), (12, 2, 48, 64), (32, 8, 128, 128), (16, 16, 96, 96), (8, 1, 256, 256),
                                  (10, 5, 80, 80), (16, 2, 128, 64)])
    kb, vb = rng.choice([2, 3, 4, 5]), rng.choice([2, 3, 4, 5])
    bs = rng.choice([16, 32, 48, 64, 128])
    if op == "write":
        return dict(op=op, rows=_log(rng, 1, 8190 * 1024 // (hkv * max(dk, dv))), hkv=hkv, dk=dk, dv=dv, kb=kb, vb=vb,
                    dtype=rng.choice(["f32", "f16", "bf16"]), bs=bs)
    seqs = _log(rng, 1, 64)
    n_hi = _log(rng, 1, 80)
    most = min(100000, 32 * 5000 * 52 * 32 // (seqs * n_hi * hq), 700000 // seqs)
    ctx_hi = _log(rng, 1, max(2, most))
    return dict(op=op, seqs=seqs, ctx_lo=rng.randint(0, ctx_hi), ctx_hi=ctx_hi, n_lo=rng.randint(0 if seqs > 1 else 1, n_hi),
                n_hi=n_hi, hq=hq, hkv=hkv, dk=dk, dv=dv, kb=kb, vb=vb, bs=bs, dtype=rng.choice(["f16", "bf16"]))


def work(case):
    c = case
    if c["op"] == "rope":
        size = {"f32": 4, "f16": 2, "bf16": 2}
        n_q, n_k = c["tokens"] * c["hq"] * c["d"], c["tokens"] * c["hkv"] * c["d"]
        n = n_q + n_k
        return {"bytes": n * size[c["dtype"]] + n_q * size[c["q_out"]] + n_k * size[c["k_out"]] + 4 * c["tokens"] + 8 * c["d"],
                "flops": 7 * n}
    if c["op"] == "plan":
        lens, new, held, total, need = _plan_sizes(c)
        pages = sum(max(0, n - h) for n, h in zip(need, held))
        return {"bytes": 4 * (4 * c["seqs"] + 3 * (total + 7) + 3 * pages + c["seqs"] + 3), "flops": 0}
    kg, vg = _groups(c["hkv"] * c["dk"]), _groups(c["hkv"] * c["dv"])
    row = kg * (16 * _width(c["kb"]) + 2) + vg * (16 * _width(c["vb"]) + 2)
    if c["op"] == "write":
        size = {"f32": 4, "f16": 2, "bf16": 2}[c["dtype"]]
        return {"bytes": c["rows"] * (c["hkv"] * (c["dk"] + c["dv"]) * size + row + 4),
                "flops": c["rows"] * (kg + vg) * 128 * 12}
    ctx, nodes = _spread(c["ctx_lo"], c["ctx_hi"], c["seqs"]), _spread(c["n_lo"], c["n_hi"], c["seqs"])[::-1]
    tokens, total = sum(a + b for a, b in zip(ctx, nodes) if b), sum(nodes)
    pages = sum((a + b + c["bs"] - 1) // c["bs"] for a, b in zip(ctx, nodes) if b)
    words = (max(1, max(nodes)) + 31) // 32
    return {"bytes": tokens * row + total * (c["hq"] * (c["dk"] + c["dv"]) * 2 + 4 * words) + 4 * (pages + 2 * c["seqs"] + 1),
            "flops": sum(2 * n * c["hq"] * (c["dk"] + c["dv"]) * (l + n) for l, n in zip(ctx, nodes))}


# ------------------------------------------------------------------------------------------------------- the inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _plan_sizes(c):
    lens = _spread(c["len_lo"], c["len_hi"], c["seqs"])
    new = _spread(c["new_lo"], c["new_hi"], c["seqs"])[::-1]
    held = [(l + c["bs"] - 1) // c["bs"] + (i % 3 == 2) for i, l in enumerate(lens)]  # some kept a page of rejected drafts
    need = [(l + n + c["bs"] - 1) // c["bs"] if n else 0 for l, n in zip(lens, new)]
    return lens, new, held, sum(new), need


def _prepare_rope(c, seed):
    g = _gen(seed)
    t, hq, hkv, d, dt = c["tokens"], c["hq"], c["hkv"], c["d"], DTYPES[c["dtype"]]
    x = torch.randn(t, hq + 2 * hkv, d, generator=g, device=DEV)
    x *= torch.exp(0.5 * torch.randn(t, hq + 2 * hkv, 1, generator=g, device=DEV))
    x[..., :: max(1, d // 5)] *= 4.0  # a few channels of larger size, as projections have them
    x = x.to(dt)
    q, k = x[:, :hq], x[:, hq:hq + hkv]
    if not c["packed"]:
        q, k = q.contiguous(), k.contiguous()
    pos = torch.randint(0, c["far"], (t,), generator=g, device=DEV, dtype=torch.int32)
    inv_freq = 10000.0 ** (-np.arange(0, c["rot"], 2, dtype=np.float64) / c["rot"])
    wq = 0.1 * torch.randn(d, generator=g, device=DEV) + 1.0 - c["offset"]
    wk = 0.1 * torch.randn(d, generator=g, device=DEV) + 1.0 - c["offset"]
    st = dict(c=c, q=q, k=k, pos=pos, inv_freq=torch.from_numpy(inv_freq).to(DEV), wq=wq, wk=wk, eps=1e-6,
              q_out=torch.empty(t, hq, d, dtype=DTYPES[c["q_out"]], device=DEV),
              k_out=torch.empty(t, hkv, d, dtype=DTYPES[c["k_out"]], device=DEV))
    if own:
        import hadamard_rotated_codebook_gb300 as cq
        st["rope"] = cq.cq_rope_init(c["rot"], inv_freq=inv_freq)
    return st


def _prepare_plan(c, seed):
    rng = random.Random(seed)
    lens, new, held, total, need = _plan_sizes(c)
    order = list(range(c["seqs"]))
    rng.shuffle(order)
    lens, new, held, need = ([x[i] for i in order] for x in (lens, new, held, need))
    wide = max(max(held), max(need)) + 1
    demand = sum(max(0, n - h) for n, h in zip(need, held))
    pool = torch.randperm(sum(held) + demand + c["slack"], generator=_gen(seed), device=DEV, dtype=torch.int64).to(torch.int32)
    used = sum(held)
    cols = torch.arange(wide, device=DEV)[None]
    h = torch.tensor(held, device=DEV)[:, None]
    start = torch.cumsum(h, 0) - h
    table = torch.where(cols < h, pool[(start + cols).clamp(max=pool.numel() - 1)], -1).to(torch.int32).contiguous()
    room = total + 7  # the slot map has room for the largest step: its tail holds no token
    st = dict(c=c, lens=_ints(lens), new=_ints(new), held=_ints(held), table=table, free=pool[used:].contiguous(),
              n_free=_ints([pool.numel() - used]), room=room)
    if own:
        st["out"] = dict(held_out=torch.empty_like(st["held"]), n_free_out=torch.empty_like(st["n_free"]),
                         slots=torch.empty(room, dtype=torch.int32, device=DEV),
                         positions=torch.empty(room, dtype=torch.int32, device=DEV),
                         token_seq=torch.empty(room, dtype=torch.int32, device=DEV),
                         cu_new=torch.empty(c["seqs"] + 1, dtype=torch.int32, device=DEV))
    return st


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


def _prepare_write(c, seed):
    g = _gen(seed)
    n, dt = c["rows"], DTYPES[c["dtype"]]
    blocks = (n + c["bs"] - 1) // c["bs"] + 3
    cap = blocks * c["bs"]
    perm = torch.randperm(blocks, generator=g, device=DEV)
    t = torch.arange(n, device=DEV) + 3
    slots = (perm[t // c["bs"]] * c["bs"] + t % c["bs"]).to(torch.int32)
    if n > 8:
        slots[n // 2] = -1  # padding of a captured step: no token there
    rows = torch.randn(n, c["hkv"], c["dk"] + c["dv"], generator=g, device=DEV)
    rows *= torch.exp(0.5 * torch.randn(n, c["hkv"], 1, generator=g, device=DEV))
    rows[..., ::17] *= 3.0
    if n > 8:
        rows[n // 3] = 0.0
    k = rows[..., :c["dk"]].reshape(n, -1).to(dt)
    v = rows[..., c["dk"]:].reshape(n, -1).to(dt)
    st = dict(c=c, k=k, v=v, slots=slots, cap=cap, k_cache=_random_cache(cap, k.shape[1], c["kb"], g),
              v_cache=_random_cache(cap, v.shape[1], c["vb"], g))
    if own:
        st["geom"] = _geometry(c, 1.0)
    return st


def _geometry(c, scale):
    import hadamard_rotated_codebook_gb300 as cq
    return cq.cq_kv_geometry(c.get("hq", c["hkv"]), c["hkv"], c["dk"], c["dv"], c["kb"], c["vb"], _codebook(c["kb"]),
                             _codebook(c["vb"]), scale)


def _prepare_attend(c, seed):
    g, rng = _gen(seed), random.Random(seed)
    ctx, nodes = _spread(c["ctx_lo"], c["ctx_hi"], c["seqs"]), _spread(c["n_lo"], c["n_hi"], c["seqs"])[::-1]
    order = list(range(c["seqs"]))
    rng.shuffle(order)
    ctx, nodes = [ctx[i] for i in order], [nodes[i] for i in order]
    if not sum(nodes):
        nodes[0] = 1
    bs, total = c["bs"], sum(nodes)
    pages = [(a + b + bs - 1) // bs for a, b in zip(ctx, nodes)]
    blocks = sum(pages) + 2
    perm = torch.randperm(blocks, generator=g, device=DEV).to(torch.int32)
    cols = torch.arange(max(1, max(pages)), device=DEV)[None]
    p = torch.tensor(pages, device=DEV)[:, None]
    start = torch.cumsum(p, 0) - p
    table = torch.where(cols < p, perm[(start + cols).clamp(max=blocks - 1)], -1).to(torch.int32).contiguous()
    # trees: each node's parent is one of the few nodes before it (or the context); a node sees its ancestors and itself
    most = max(nodes)
    words = (most + 31) // 32
    bits = np.zeros((total, words * 32), dtype=bool)
    at = 0
    for n in nodes:
        for i in range(n):
            parent = max(-1, i - 1 - int(rng.expovariate(0.5)))
            if parent >= 0:
                bits[at + i] = bits[at + parent]
            bits[at + i, i] = True
        at += n
    mask = np.packbits(bits, axis=1, bitorder="little").view(np.uint32).astype(np.int64)
    mask = torch.from_numpy(mask.astype(np.uint32).view(np.int32).copy()).to(DEV)
    k_cache = _random_cache(blocks * bs, c["hkv"] * c["dk"], c["kb"], g)
    v_cache = _random_cache(blocks * bs, c["hkv"] * c["dv"], c["vb"], g)
    # queries as a per-head norm leaves them, of somewhat more than unit size so that some tokens stand out
    q = torch.randn(total, c["hq"], c["dk"], generator=g, device=DEV)
    q = 1.5 * q / q.pow(2).mean(-1, keepdim=True).sqrt()
    cu = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int64)
    st = dict(c=c, q=q.to(DTYPES[c["dtype"]]), k_cache=k_cache, v_cache=v_cache, cap=blocks * bs, table=table, ctx=_ints(ctx),
              cu=_ints(cu.tolist()), mask=mask, most=most, longest=max(a + b for a, b in zip(ctx, nodes)), scale=c["dk"] ** -0.5,
              o=torch.empty(total, c["hq"], c["dv"], dtype=DTYPES[c["dtype"]], device=DEV))
    if own:
        st["geom"] = _geometry(c, st["scale"])
    return st


def prepare(case, seed):
    return {"rope": _prepare_rope, "plan": _prepare_plan, "write": _prepare_write, "attend": _prepare_attend}[case["op"]](case, seed)


# --------------------------------------------------------------------------------------------------- the plain forms

def _hadamard(dtype):
    h = torch.ones(1, 1, dtype=dtype, device=DEV)
    for _ in range(7):
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return h / math.sqrt(GROUP)


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


def _rope_plain(st):
    c = st["c"]
    ang = st["pos"].double()[:, None] * st["inv_freq"][None]
    cos, sin = ang.cos().float()[:, None], ang.sin().float()[:, None]

    def one(x, w, dtype):
        x = x.float()
        y = x * torch.rsqrt(x.pow(2).mean(-1, keepdim=True) + st["eps"]) * (w + c["offset"])
        r, rest = y[..., :c["rot"]], y[..., c["rot"]:]
        a, b = (r[..., 0::2], r[..., 1::2]) if c["interleaved"] else r.chunk(2, dim=-1)
        u, v = a * cos - b * sin, b * cos + a * sin
        r = torch.stack([u, v], -1).flatten(-2) if c["interleaved"] else torch.cat([u, v], -1)
        return torch.cat([r, rest], -1).to(dtype)

    return {"q": one(st["q"], st["wq"], st["q_out"].dtype), "k": one(st["k"], st["wk"], st["k_out"].dtype)}


def _plan_plain(st):
    bs = st["c"]["bs"]
    lens, new, held, table, free, n_free = st["lens"], st["new"], st["held"], st["table"], st["free"], st["n_free"]
    need = torch.where(new > 0, (lens + new + bs - 1) // bs, 0)
    extra = (need - held).clamp(min=0)
    before = torch.cumsum(extra, 0) - extra
    cu = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), torch.cumsum(new, 0)])
    cols = torch.arange(table.shape[1], device=DEV)[None]
    at = n_free.long() - 1 - (before[:, None] + cols - held[:, None])
    popped = torch.where(at >= 0, free[at.clamp(0, free.numel() - 1)], -1)
    table = torch.where((cols >= held[:, None]) & (cols < need[:, None]), popped, table)
    t = torch.arange(st["room"], device=DEV)
    seq = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    real = seq < lens.numel()
    s = seq.clamp(max=lens.numel() - 1)
    pos = lens[s] + t - cu[s]
    block = table[s, (pos // bs).clamp(max=table.shape[1] - 1)]
    slots = torch.where(real & (block >= 0), block * bs + pos % bs, -1)
    i32 = torch.int32
    return {"table": table.to(i32), "held": torch.maximum(held, need).to(i32), "n_free": (n_free - extra.sum()).to(i32),
            "slots": slots.to(i32), "positions": torch.where(real, pos, -1).to(i32), "token_seq": torch.where(real, seq, -1).to(i32),
            "cu_new": cu.to(i32)}


def _encode_plain(x, bits):
    """rows [n][width] -> (codes, fp16 norms), in 64 bits: a direction next to a border between two levels has to fall right."""
    n, width = x.shape
    groups = _groups(width)
    x = torch.nn.functional.pad(x.double(), (0, groups * GROUP - width)).view(n, groups, GROUP)
    r = x @ _hadamard(torch.float64).sign()  # sums without 1/sqrt(128): exact for narrow types, where ties happen
    norm = x.pow(2).sum(-1, keepdim=True).sqrt()
    lv = torch.from_numpy(_codebook(bits)).to(DEV).double()
    border = (lv[1:] + lv[:-1]) / 2 * (norm.clamp(min=1e-12) * math.sqrt(GROUP))[..., None]
    code = (r[..., None] > border).sum(-1)  # a tie falls to the lower level
    if bits == 5:
        code = (code - 1) & 3
    return _pack(code.view(n, groups * GROUP), _width(bits)), norm[..., 0].half()


def _write_plain(st):
    c, slots = st["c"], st["slots"].long()
    real = (slots >= 0)[:, None]
    to = torch.where(slots >= 0, slots, slots[0])  # the first row has a slot: padding repeats what it writes
    out = {}
    for name, bits in (("k", c["kb"]), ("v", c["vb"])):
        x = st[name]
        codes, norms = _views(st[name + "_cache"], st["cap"], x.shape[1], bits)
        a, b = _encode_plain(x, bits)
        codes[to] = torch.where(real, a, a[:1])
        norms[to] = torch.where(real, b, b[:1])
        out[name + "_codes"], out[name + "_norms"] = codes, norms
    return out


def _dense(cache, cap, width, bits, rows):
    codes, norms = _views(cache, cap, width, bits)
    c = _by_code(bits)[_unpack(codes[rows], _width(bits)).long()]
    c = c.view(*rows.shape, -1, GROUP) * norms[rows].float()[..., None]
    return (c @ _hadamard(torch.float32)).flatten(-2)[..., :width]


def _attend_plain(st):
    c = st["c"]
    s_n, t_n, l_n, bs, total = c["seqs"], max(1, st["most"]), st["longest"], c["bs"], st["q"].shape[0]
    ctx, cu = st["ctx"].long(), st["cu"].long()
    n = cu[1:] - cu[:-1]
    pos = torch.arange(l_n, device=DEV)
    real = pos[None] < (ctx + n)[:, None]
    rows = st["table"].long()[:, (pos // bs)] * bs + pos % bs
    rows = torch.where(real, rows, 0)
    k = _dense(st["k_cache"], st["cap"], c["hkv"] * c["dk"], c["kb"], rows).view(s_n, l_n, c["hkv"], c["dk"])
    v = _dense(st["v_cache"], st["cap"], c["hkv"] * c["dv"], c["vb"], rows).view(s_n, l_n, c["hkv"], c["dv"])
    node = torch.arange(t_n, device=DEV)
    at = (cu[:-1, None] + node[None]).clamp(max=total - 1)
    q = st["q"].float()[at].view(s_n, t_n, c["hkv"], c["hq"] // c["hkv"], c["dk"])
    logit = torch.einsum("stgrd,slgd->sgrtl", q, k) * st["scale"]
    j = pos[None] - ctx[:, None]  # which drafted token a position holds
    words = st["mask"][at]
    jj = j.clamp(0, t_n - 1)
    word = torch.gather(words, 2, (jj // 32)[:, None].expand(s_n, t_n, l_n))
    seen = ((word >> (jj % 32)[:, None].to(torch.int32)) & 1).bool()
    seen = ((j < 0)[:, None] | seen) & real[:, None]
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
        return {"rope": _rope_plain, "plan": _plan_plain, "write": _write_plain, "attend": _attend_plain}[c["op"]](st)
    import hadamard_rotated_codebook_gb300 as cq
    if c["op"] == "rope":
        q, k = cq.cq_qk_norm_rope(st["q"], st["k"], st["pos"], st["rope"], st["wq"], st["wk"], eps=st["eps"],
                                  weight_offset=c["offset"], interleaved=c["interleaved"], q_out=st["q_out"], k_out=st["k_out"])
        return {"q": q, "k": k}
    if c["op"] == "plan":
        out = st["out"]
        cq.cq_kv_plan(st["lens"], st["new"], st["held"], st["table"], st["free"], st["n_free"], c["bs"], **out)
        return {"table": st["table"], "held": out["held_out"], "n_free": out["n_free_out"], "slots": out["slots"],
                "positions": out["positions"], "token_seq": out["token_seq"], "cu_new": out["cu_new"]}
    if c["op"] == "write":
        cq.cq_kv_write_slots(st["geom"], st["k_cache"], st["v_cache"], st["cap"], st["k"], st["v"], st["slots"])
        out = {}
        for name, bits in (("k", c["kb"]), ("v", c["vb"])):
            out[name + "_codes"], out[name + "_norms"] = _views(st[name + "_cache"], st["cap"], st[name].shape[1], bits)
        return out
    return cq.cq_kv_tree_attend(st["geom"], st["q"], st["k_cache"], st["v_cache"], st["cap"], st["table"], c["bs"], st["ctx"],
                                st["cu"], st["mask"], st["most"], o=st["o"])


# ------------------------------------------------------------------------------------------------------ in 64 bits

def _sylvester():
    """The normalised matrix from its definition: the sign of entry (i, k) is the parity of i & k."""
    i = torch.arange(GROUP, device=DEV)
    both = i[:, None] & i[None]
    odd = torch.zeros_like(both)
    for b in range(7):
        odd = odd ^ ((both >> b) & 1)
    return (1.0 - 2.0 * odd.double()) / math.sqrt(GROUP)


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
    return torch.matmul(level.view(len(rows), groups, GROUP), _sylvester()).mul(norm[..., None]).view(len(rows), -1)[:, :width]


def _exact_attend(c, st):
    table, mask = st["table"].cpu().numpy().astype(np.int64), st["mask"].cpu().numpy().view(np.uint32)
    ctx, cu = st["ctx"].tolist(), st["cu"].tolist()
    out = torch.zeros(st["q"].shape[0], c["hq"], c["dv"], dtype=torch.float64, device=DEV)
    per = c["hq"] // c["hkv"]
    for s in range(c["seqs"]):
        a, b = cu[s], cu[s + 1]
        n = b - a
        if not n or not ctx[s] + n:
            continue
        p = np.arange(ctx[s] + n)
        rows = torch.from_numpy(table[s, p // c["bs"]] * c["bs"] + p % c["bs"]).to(DEV)
        k = _exact_rows(st["k_cache"], st["cap"], c["hkv"] * c["dk"], c["kb"], rows)
        v = _exact_rows(st["v_cache"], st["cap"], c["hkv"] * c["dv"], c["vb"], rows)
        bits = np.unpackbits(mask[a:b].view(np.uint8), axis=1, bitorder="little")[:, :n]
        shut = torch.from_numpy(bits == 0).to(DEV)
        for h in range(c["hq"]):
            g = h // per
            x = st["q"][a:b, h].double() @ k[:, g * c["dk"]:(g + 1) * c["dk"]].T * st["scale"]
            x[:, ctx[s]:][shut] = -math.inf
            w = torch.softmax(x, -1)
            out[a:b, h] = torch.nan_to_num(w) @ v[:, g * c["dv"]:(g + 1) * c["dv"]]
    return out


def _exact_rope(c, st):
    turn = torch.outer(st["pos"].double(), st["inv_freq"])
    turn = torch.polar(torch.ones_like(turn), turn)[:, None]

    def one(x, w):
        x = x.double()
        y = x / (x.square().sum(-1, keepdim=True) / c["d"] + st["eps"]).sqrt() * (c["offset"] + w.double())
        half = c["rot"] // 2
        i = torch.arange(half, device=DEV)
        first, second = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + half)
        z = torch.complex(y[..., first], y[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        return y

    return {"q": one(st["q"], st["wq"]), "k": one(st["k"], st["wk"])}


def _exact_write(c, st):
    out = {}
    for name, bits in (("k", c["kb"]), ("v", c["vb"])):
        x = st[name].double()
        norms = _views(st[name + "_cache"], st["cap"], x.shape[1], bits)[1].double()
        for g in range(norms.shape[1]):  # the rotation keeps a group's length
            size = x[:, g * GROUP:(g + 1) * GROUP].square().sum(-1).sqrt()
            keep = st["slots"] >= 0
            norms[st["slots"][keep].long(), g] = size[keep]
        out[name + "_codes"], out[name + "_norms"] = None, norms
    return out


def exact(case, seed):
    if case["op"] == "plan":
        return None  # whole numbers throughout
    if case["op"] == "attend":  # 64-bit products at about half a TFLOP/s
        if work(case)["flops"] > 4e12:
            return None
    st = prepare(case, seed)
    return {"rope": _exact_rope, "write": _exact_write, "attend": _exact_attend}[case["op"]](case, st)
