"""Plain 64-bit definitions of a layer's other serving steps (block norm,
low-rank adapters), with bounds on the error of their stated arithmetic
(numpy only; nothing here comes from the CUDA path)."""
import numpy as np

from tests.paged_reference import EPS24, HALF_STEP, TINY


def block_norm(x, res, w, *, post=False, wb=None, gate=None, act=None, branch=1.0, keep=1.0, eps=1e-6, offset=0.0):
    """(r, y, bound on r's error, bound on y's), before the outputs' own rounding.

    Roundings of 2^-24 (a unit): a sum of squares adds up to 32 elements one after the other and joins up to 9 + 5 partial
    sums, so it is off by 48 units at most, its root by half of that, rsqrtf by 4, the mean's product and sum by 1 each:
    32 in all. A branch has 3 more products and the sum of its weight: 36; a gate's function 2 for its reciprocal, 2
    for the sum and the product, and of its power of two 4 and the 1.44 |g| by which its exponent is rounded; r is one
    fma of two products."""
    f = np.float64
    x = x.astype(f)
    with np.errstate(over="ignore", invalid="ignore"):
        z, units = x, 2.0
        if post:
            z, units = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps), 36.0
        if wb is not None:
            z = z * (offset + wb.astype(f))
        elif post:
            z = z * (offset + 1.0)
        if gate is not None:
            g = gate.astype(f)
            s = 1 / (1 + np.exp(-g))
            z = z * {None: g, "sigmoid": s, "silu": g * s}[act]
            units = units + 1 + (0 if act is None else 10 + 2.4 * np.abs(g))
        b = branch * z
        a = keep * (res.astype(f) if res is not None else 0.0)
        r = a + b
        er = (units + 2) * EPS24 * np.abs(b) + 2 * EPS24 * np.abs(a) + EPS24 * np.abs(r)
        d = x.shape[-1]
        inv = 1 / np.sqrt((r * r).mean(-1, keepdims=True) + eps)
        weight = offset + (w.astype(f) if w is not None else 1.0)
        y = r * inv * weight
        moved = np.sqrt((er * er).sum(-1, keepdims=True)) * inv / np.sqrt(d)  # the norm's part in er, over sqrt(mean + eps)
        ey = np.abs(weight) * inv * er + np.abs(y) * (36 * EPS24 + moved)
        # the sum of the weight and its offset is rounded too, where they cancel by more than it shows
        if w is not None:
            ey = ey + EPS24 * np.abs(r * inv) * (abs(offset) + np.abs(w))
    return r, y, er, ey


def rounded(v, err, dtype):
    """The bound once v is rounded to a type."""
    return err + HALF_STEP[dtype] * (np.abs(v) + err) + TINY[dtype]


def lora(ys, x, a, b, adapters, cu, scales=None, ranks=None, x_scale=None, terms=False):
    """[(result, bound)] for each y (float64 arrays; weights [adapters, rank, in] and [adapters, out, rank]).

    A tensor core's sum of 8 or 16 products loses a step of 2^-23 of what it adds up at most, as does each addition after
    it: one sum runs over 2 or 8 (fp32: two terms, 8 inputs at a time) products for each 32 inputs that a warp has (a
    quarter of them at least), then over 4 to 8 warps and up to 8 blocks, all within sum |a x|. Two terms of 11 bits leave
    2^-21 of a value of fp32 at most (x in two of tf32; u, in the second product, in two of fp16 or three of bf16)."""
    f = np.float64
    x = x.astype(f)
    if x_scale is not None:
        x = x * x_scale.astype(f)[:, None]
    n_in, step = x.shape[1], 2.0 ** -23
    out = []
    with np.errstate(invalid="ignore"):
        for y, aj, bj in zip(ys, a, b):
            aj, bj = aj.astype(f), bj.astype(f)
            o, e = y.astype(f).copy(), np.zeros(y.shape)
            for s, k in enumerate(adapters):
                t = slice(cu[s], cu[s + 1])
                if k < 0 or cu[s] == cu[s + 1]:
                    continue
                r = aj.shape[1] if ranks is None else ranks[k]
                c = 1.0 if scales is None else float(scales[k])
                A, B = aj[k, :r], bj[k][:, :r]
                u, mag = c * (x[t] @ A.T), abs(c) * (np.abs(x[t]) @ np.abs(A).T)
                chain = (8 if terms else 2) * -(-n_in // 128) + 24
                eu = mag * (chain * step + (2.0 ** -21 if terms else 0.0))
                whole = np.abs(u) @ np.abs(B).T
                runs = -(-r // 64)  # y takes 64 ranks at a time
                e[t] = eu @ np.abs(B).T + whole * (2.0 ** -21 + (16 * -(-min(r, 64) // 16) + 2) * step)
                e[t] += runs * EPS24 * (np.abs(y[t]) + whole + e[t])
                o[t] += u @ B.T
            out.append((o, e + TINY["float32"]))
    return out


def attend_rows(q, k_blob, v_blob, cap, rows, sees, cu, geom, kb, vb, cbk, cbv, scale):
    """Attention of tokens q [nodes, hq, dk] over cache rows rows[s], of which token i of request s attends those with
    sees[s][i]: (o, bound) by the arithmetic and the reasoning of paged_reference.attend."""
    from tests.paged_reference import dequant
    hq, hkv, dk, dv = geom
    per = hq // hkv
    o, bound = np.zeros((len(q), hq, dv)), np.zeros((len(q), hq, dv))
    for s, (at, see) in enumerate(zip(rows, sees)):
        a, n = cu[s], cu[s + 1] - cu[s]
        if n == 0 or not see.any():
            continue
        use = see.any(0)
        at, see = at[use], see[:, use]
        kd, kt = dequant(k_blob, cap, hkv * dk, kb, cbk, at)
        vd, vt = dequant(v_blob, cap, hkv * dv, vb, cbv, at)
        for h in range(hq):
            g = h // per
            k, v = kd[:, g * dk:(g + 1) * dk], vd[:, g * dv:(g + 1) * dv]
            nk = np.linalg.norm(kt[:, g * dk // 128:((g + 1) * dk + 127) // 128].reshape(len(at), -1), axis=1)
            nv = np.linalg.norm(vt[:, g * dv // 128:((g + 1) * dv + 127) // 128].reshape(len(at), -1), axis=1)
            qh = q[a:a + n, h].astype(np.float64)
            x = np.where(see, qh @ k.T * scale, -np.inf)
            top = x.max(1, keepdims=True)
            w = np.exp(x - np.where(np.isfinite(top), top, 0.0))
            some = w.sum(1, keepdims=True)
            w = w / np.where(some > 0, some, 1.0)
            o[a:a + n, h] = w @ v
            d = abs(scale) * (2 * 2.0 ** -11 + 2.0 ** -18) * np.linalg.norm(qh, axis=1) * np.where(see, nk, 0.0).max(1)
            for i in range(n):
                bound[a + i, h] = (np.expm1(2 * d[i]) * (w[i] @ np.abs(v - o[a + i, h])) + 2 * 2.0 ** -11 * (w[i] @ nv)
                                   + 2.0 ** -24 * see[i].sum() * (w[i] * nv).max() + 2.0 ** -18 * (w[i] @ nv))
    return o, bound
