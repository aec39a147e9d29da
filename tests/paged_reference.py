"""Plain 64-bit definitions of the paged cache's operators, for the tests
(numpy only; nothing here comes from the CUDA path)."""
import math

import numpy as np

EPS24 = 2.0 ** -24
HALF_STEP = {"float32": 2.0 ** -24, "float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}
TINY = {"float32": 2.0 ** -149, "float16": 2.0 ** -25, "bfloat16": 2.0 ** -133}  # half a step at zero


def hadamard():
    i = np.arange(128)
    par = np.zeros((128, 128), dtype=np.int64)
    both = i[:, None] & i[None]
    for b in range(7):
        par ^= (both >> b) & 1
    return (1 - 2 * par) / math.sqrt(128)


def width_of(bits):
    return 2 if bits == 5 else bits


def rope(x, w, pos, inv_freq, eps, offset, interleaved):
    """x [t, h, d] -> (y, magnitude of each element's pair)."""
    x = x.astype(np.float64)
    t, h, d = x.shape
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (offset + (w.astype(np.float64) if w is not None else 1.0))
    half = len(inv_freq)
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    ang = np.asarray(pos, dtype=np.longdouble)[:, None] * np.asarray(inv_freq, dtype=np.longdouble)[None]
    c, s = np.cos(ang).astype(np.float64)[:, None], np.sin(ang).astype(np.float64)[:, None]
    out, mag = y.copy(), np.abs(y)
    out[..., a] = y[..., a] * c - y[..., b] * s
    out[..., b] = y[..., b] * c + y[..., a] * s
    mag[..., a] = mag[..., b] = np.abs(y[..., a]) + np.abs(y[..., b])
    return out, mag


def plan(lens, new, held, table, free, n_free, bs, room):
    """Returns table, held_out, n_free_out, slots, positions, token_seq, cu_new."""
    table = table.copy()
    held_out, cu = [], [0]
    slots, positions, seqs = [np.full(room, -1, dtype=np.int64) for _ in range(3)]
    taken, at = 0, 0
    wide = table.shape[1]
    for s in range(len(lens)):
        l, n, h = max(lens[s], 0), max(new[s], 0), min(max(held[s], 0), wide)
        need = min(-(-(l + n) // bs), wide) if n else 0
        for b in range(h, need):
            i = n_free - 1 - taken
            table[s, b] = free[i] if 0 <= i < len(free) else -1
            taken += 1
        held_out.append(max(h, need))
        for i in range(n):
            pos = l + i
            if at < room:
                blk = table[s, pos // bs] if pos // bs < wide else -1
                slots[at] = blk * bs + pos % bs if blk >= 0 else -1
                positions[at], seqs[at] = pos, s
            at += 1
        cu.append(at)
    return table, np.array(held_out, dtype=np.int64), n_free - taken, slots, positions, seqs, np.array(cu)


def encode(x, bits, codebook):
    """Rows [n, width] -> (codes [n, padded], norms fp16 [n, groups]); decisions in 64 bits."""
    n, width = x.shape
    g = -(-width // 128)
    p = np.zeros((n, g * 128))
    p[:, :width] = x.astype(np.float64)
    p = p.reshape(n, g, 128)
    # the signs alone, without 1/sqrt(128): sums of narrow types are then exact, and a tie is a tie
    r = p @ np.sign(hadamard())
    nn = np.sqrt((p * p).sum(-1, keepdims=True))
    cb = codebook.astype(np.float64)
    code = (r[..., None] > (cb[1:] + cb[:-1]) / 2 * (np.maximum(nn, 1e-12) * math.sqrt(128))[..., None]).sum(-1)
    if bits == 5:
        code = (code - 1) & 3
    with np.errstate(over="ignore"):  # a norm past 65504 is stored as infinity
        return code.reshape(n, g * 128), nn[..., 0].astype(np.float32).astype(np.float16)


def pack(codes, w):
    n, k = codes.shape
    bit = (codes[..., None] >> np.arange(w)) & 1
    return np.packbits(bit.reshape(n, k * w).astype(np.uint8), axis=1, bitorder="little")


def levels_by_code(bits, codebook):
    cb = codebook.astype(np.float64)
    return np.array([0.0, cb[2], -2 * cb[2], -cb[2]]) if bits == 5 else cb


def split_blob(blob, cap, width, bits):
    g = -(-width // 128)
    m = cap * g * 16 * width_of(bits)
    return blob[:m].reshape(cap, -1), blob[m:m + cap * g * 2].view(np.float16).reshape(cap, g)


def dequant(blob, cap, width, bits, codebook, rows):
    """(dequantised rows [n, width], rows before the rotation [n, groups, 128])."""
    codes, norms = split_blob(blob, cap, width, bits)
    w, g = width_of(bits), norms.shape[1]
    bit = np.unpackbits(codes[rows], axis=1, bitorder="little").reshape(len(rows), g * 128, w)
    code = (bit.astype(np.int64) << np.arange(w)).sum(-1)
    turned = levels_by_code(bits, codebook)[code].reshape(len(rows), g, 128) * norms[rows].astype(np.float64)[..., None]
    return (turned @ hadamard()).reshape(len(rows), -1)[:, :width], turned


def attend(q, k_blob, v_blob, cap, table, bs, ctx, cu, seen, geom, kb, vb, cbk, cbv, scale):
    """q [nodes, hq, dk] -> (o, bound on the error of the stated arithmetic before the output's rounding).

    seen(s, i, j): whether drafted token i of request s attends drafted token j.
    The bound: query and level roundings to fp16 move a logit by at most
    d = scale * (2 * 2^-11 + 2^-18) * |q| |k of its groups| (Cauchy; the last
    term for products and fp32 sums), a weight by a factor within e^(2 max d);
    p * n in fp16 and the value levels in fp16 move the sum before its
    rotation by 2 * 2^-11 |v of its groups| p per token in the 2-norm, and an
    fp16 weight below its normal range by 2^-24 of the largest weight."""
    hq, hkv, dk, dv = geom
    per = hq // hkv
    o, bound = np.zeros((len(q), hq, dv)), np.zeros((len(q), hq, dv))
    for s in range(len(ctx)):
        a, n = cu[s], cu[s + 1] - cu[s]
        if n == 0:
            continue
        p = np.arange(ctx[s] + n)
        rows = table[s, p // bs].astype(np.int64) * bs + p % bs
        vis = np.ones((n, ctx[s] + n), dtype=bool)
        for i in range(n):
            for j in range(n):
                vis[i, ctx[s] + j] = seen(s, i, j)
        use = vis.any(0)  # rows nobody attends may hold anything
        kd, kt = dequant(k_blob, cap, hkv * dk, kb, cbk, np.where(use, rows, rows[use][0] if use.any() else 0))
        vd, vt = dequant(v_blob, cap, hkv * dv, vb, cbv, np.where(use, rows, rows[use][0] if use.any() else 0))
        for h in range(hq):
            g = h // per
            k, v = kd[:, g * dk:(g + 1) * dk], vd[:, g * dv:(g + 1) * dv]
            kg = kt[:, g * dk // 128:((g + 1) * dk + 127) // 128].reshape(len(p), -1)
            vg = vt[:, g * dv // 128:((g + 1) * dv + 127) // 128].reshape(len(p), -1)
            for i in range(n):
                e = vis[i]
                if not e.any():
                    continue
                x = k[e] @ q[a + i, h].astype(np.float64) * scale
                w = np.exp(x - x.max())
                w /= w.sum()
                o[a + i, h] = w @ v[e]
                nk, nv = np.linalg.norm(kg[e], axis=1), np.linalg.norm(vg[e], axis=1)
                d = abs(scale) * (2 * 2.0 ** -11 + 2.0 ** -18) * np.linalg.norm(q[a + i, h].astype(np.float64)) * nk.max()
                bound[a + i, h] = (np.expm1(2 * d) * (w @ np.abs(v[e] - o[a + i, h])) + 2 * 2.0 ** -11 * (w @ nv)
                                   + 2.0 ** -24 * e.sum() * (w * nv).max() + 2.0 ** -18 * (w @ nv))
    return o, bound
