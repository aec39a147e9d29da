"""GPU parity of the paged cache's operators (cq_qk_norm_rope, cq_kv_plan,
cq_kv_write_slots, cq_kv_tree_attend) with their 64-bit definitions."""
import math

import numpy as np
import pytest
import torch

import oracle as O
from tests import paged_reference as R

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def C():
    import hadamard_rotated_codebook_gb300 as pkg
    return pkg


def _np(t):
    return t.detach().double().cpu().numpy()


def _name(dtype):
    return str(dtype).replace("torch.", "")


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------------------------------------------- rope

def _check_rope(C, t, hq, hkv, d, rot, il, dtype, qd, kd, packed=True, weights=True, offset=0.0, far=1 << 20, eps=1e-6, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(t, hq + 2 * hkv, d, generator=g, device="cuda") * 3).to(dtype)
    q, k = x[:, :hq], x[:, hq:hq + hkv]
    if not packed:
        q, k = q.contiguous(), k.contiguous()
    pos = torch.randint(0, far, (t,), generator=g, device="cuda", dtype=torch.int32)
    if t:
        pos[-1] = far
    inv = 10000.0 ** (-np.arange(0, rot, 2) / max(rot, 1))
    w = [torch.randn(d, generator=g, device="cuda") if weights else None for _ in range(2)]
    before = x.clone()
    qo, ko = C.cq_qk_norm_rope(q, k, pos, C.cq_rope_init(rot, inv_freq=inv), *w, eps=eps, weight_offset=offset, interleaved=il,
                               q_dtype=qd, k_dtype=kd)
    torch.cuda.synchronize()
    assert torch.equal(x, before)
    for a, b, ww, od in ((q, qo, w[0], qd), (k, ko, w[1], kd)):
        assert b.dtype == od and b.shape == a.shape
        y, mag = R.rope(_np(a), None if ww is None else _np(ww), pos.cpu().numpy(), inv, eps, offset, il)
        # roundings of 2^-24 of a pair's magnitude: 13 of the sum of squares (half of them through the
        # root), 4 of rsqrtf, 3 of the products with the weight, 4 of sine and cosine, 3 of the turn
        tol = 24 * R.EPS24 * mag + R.HALF_STEP[_name(od)] * np.abs(y) * (1 + 1e-6) + R.TINY[_name(od)]
        err = np.abs(_np(b) - y)
        assert (err <= tol).all(), f"worst {np.max(err / tol)}"


@pytest.mark.parametrize("d,rot", [(64, 64), (128, 128), (48, 48), (256, 256), (96, 32), (34, 34), (34, 6), (2, 2), (80, 0), (36, 20)])
@pytest.mark.parametrize("il", [False, True])
def test_rope_widths(C, d, rot, il):
    _check_rope(C, 7, 5, 3, d, rot, il, F32, F32, F32, seed=d + rot)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("qd,kd", [(F32, F16), (F16, F32), (BF16, BF16)])
def test_rope_types(C, dtype, qd, kd):
    _check_rope(C, 9, 12, 2, 48, 48, False, dtype, qd, kd)
    _check_rope(C, 5, 4, 4, 128, 64, True, dtype, qd, kd, packed=False, offset=1.0)


@pytest.mark.parametrize("t", [0, 1, 2, 33, 1000])
def test_rope_token_counts(C, t):
    _check_rope(C, t, 32, 8, 128, 128, False, BF16, BF16, BF16, seed=t)


def test_rope_one_side_and_no_weights(C):
    _check_rope(C, 5, 3, 0, 64, 64, False, F32, F32, F32)
    _check_rope(C, 5, 0, 3, 64, 64, False, F32, F32, F32)
    _check_rope(C, 5, 3, 1, 64, 32, False, F16, F32, F32, weights=False)
    _check_rope(C, 300, 70, 1, 32, 32, False, F32, F32, F32)


def test_rope_far_positions(C):
    """The angle at 2^31 - 1 is as exact as at 1."""
    _check_rope(C, 64, 2, 1, 64, 64, False, F32, F32, F32, far=2 ** 31 - 1)


def test_rope_misaligned_rows(C):
    """Rows one element off every vector boundary give the same values."""
    x = torch.randn(6, 3, 65, device="cuda").to(F16)
    pos, rates = _i32([0, 1, 5, 1000, 7, 3]), C.cq_rope_init(64)
    a = C.cq_qk_norm_rope(x[:, :2, 1:], x[:, 2:, 1:], pos, rates)
    b = C.cq_qk_norm_rope(x[:, :2, 1:].contiguous(), x[:, 2:, 1:].contiguous(), pos, rates)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_rope_in_place(C):
    x = torch.randn(37, 6, 64, device="cuda")
    pos, rates = _i32(np.arange(37)), C.cq_rope_init(64)
    want = C.cq_qk_norm_rope(x[:, :4], x[:, 4:], pos, rates)
    got = C.cq_qk_norm_rope(x[:, :4], x[:, 4:], pos, rates, q_out=x[:, :4], k_out=x[:, 4:])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_rope_zeros_and_non_finite_rows_stay_apart(C):
    x = torch.randn(4, 2, 64, device="cuda")
    x[0] = 0
    x[1, 0, 3] = math.nan
    x[2, 1, 5] = math.inf
    q, k = C.cq_qk_norm_rope(x, x[:, :1].contiguous(), _i32([3, 4, 5, 6]), C.cq_rope_init(64), eps=1e-6)
    assert (q[0] == 0).all() and q[1, 0].isnan().all() and torch.isfinite(q[1, 1]).all()
    assert torch.isfinite(q[2, 0]).all() and torch.isfinite(q[3]).all()


def test_rope_refuses_bad_tensors(C):
    x, pos, rates = torch.zeros(2, 2, 64, device="cuda"), _i32([0, 1]), C.cq_rope_init(64)
    with pytest.raises(TypeError):
        C.cq_qk_norm_rope(x.int(), x.int(), pos, rates)
    with pytest.raises(TypeError):
        C.cq_qk_norm_rope(x, x, pos.long(), rates)
    with pytest.raises(TypeError):
        C.cq_qk_norm_rope(x, x, pos, rates.astype(np.float64))
    with pytest.raises(ValueError):
        C.cq_qk_norm_rope(x, x[:1], pos, rates)
    with pytest.raises(ValueError):
        C.cq_qk_norm_rope(x, x, pos[:1], rates)
    with pytest.raises(ValueError):
        C.cq_qk_norm_rope(x.transpose(1, 2), x.transpose(1, 2), pos, rates)
    with pytest.raises(ValueError):
        C.cq_qk_norm_rope(x, x, pos, rates, torch.ones(63, device="cuda"))
    with pytest.raises(ValueError):
        C.cq_qk_norm_rope(x, x, pos, rates, q_out=torch.zeros(1, 1, 64, device="cuda").expand(2, 2, 64))
    with pytest.raises(C.CQError):
        C.cq_qk_norm_rope(x[..., :32], x[..., :32], pos, rates)  # 64 rotating elements of 32


# ------------------------------------------------------------------------------------------------------------- plan

def _check_plan(C, lens, new, held, bs, free_n, room, wide=None, n_free=None, seed=0, pad=0):
    rng = np.random.RandomState(seed)
    s = len(lens)
    wide = wide if wide is not None else max([1] + [max(-(-(l + n) // bs), h) for l, n, h in zip(lens, new, held)]) + 2
    ids = rng.permutation(sum(held) + free_n + 5)
    table, at = rng.randint(-9, -1, size=(s, wide + pad)), 0
    for i, h in enumerate(held):
        table[i, :h] = ids[at:at + h]
        at += h
    free = ids[at:at + free_n]
    n_free = len(free) if n_free is None else n_free
    dev = _i32(table.reshape(s, wide + pad))
    out = C.cq_kv_plan(_i32(lens), _i32(new), _i32(held), dev[:, :wide], _i32(free), _i32([n_free]), bs, room)
    torch.cuda.synchronize()
    want = R.plan(lens, new, held, table[:, :wide], free, n_free, bs, room)
    np.testing.assert_array_equal(dev.cpu().numpy()[:, :wide], want[0])
    np.testing.assert_array_equal(dev.cpu().numpy()[:, wide:], table[:, wide:])
    for name, w in zip(("held_out", "n_free_out", "slots", "positions", "token_seq", "cu_new"), want[1:]):
        np.testing.assert_array_equal(out[name].cpu().numpy(), np.atleast_1d(w), err_msg=name)


@pytest.mark.parametrize("s,bs,hi", [(1, 16, 1), (1, 16, 40), (5, 1, 7), (33, 16, 33), (300, 7, 20), (1024, 32, 3), (1025, 64, 5),
                                     (2600, 16, 9)])
def test_plan_matches_definition(C, s, bs, hi):
    rng = np.random.RandomState(s + bs)
    lens = rng.randint(0, 200, s).tolist()
    new = (rng.randint(0, hi + 1, s) * (rng.rand(s) < 0.8)).tolist()
    held = [-(-l // bs) + int(rng.rand() < 0.3) for l in lens]
    free_n = sum(max(0, -(-(l + n) // bs) - h) for l, n, h in zip(lens, new, held)) + 3
    _check_plan(C, lens, new, held, bs, free_n, sum(new) + 11, seed=s, pad=3)
    C.cq_device_status()


def test_plan_long_prompts(C):
    """One prompt of many blocks beside decode steps; a step without tokens; an empty batch."""
    _check_plan(C, [0, 77, 5, 0], [50000, 1, 0, 3000], [0, 5, 1, 0], 16, 4000, 53001)
    _check_plan(C, [3, 9], [0, 0], [1, 1], 16, 4, 5)
    _check_plan(C, [3, 9], [0, 0], [1, 1], 16, 4, 0)
    out = C.cq_kv_plan(*[_i32([])] * 3, torch.empty(0, 4, dtype=torch.int32, device="cuda"), _i32([1]), _i32([1]), 16, 3)
    assert out["cu_new"].tolist() == [0] and out["n_free_out"].tolist() == [1] and out["slots"].tolist() == [-1] * 3
    C.cq_device_status()


def test_plan_marks_what_is_missing(C):
    """Too few free blocks, a table row too short, too little room: -1 in the
    places that miss, and the device status says so; n_free above the stack's
    length or below zero reads nothing past it."""
    cases = [dict(lens=[10, 10], new=[30, 30], held=[1, 1], bs=16, free_n=3, room=60),
             dict(lens=[10, 10], new=[30, 30], held=[1, 1], bs=16, free_n=9, room=60, wide=2),
             dict(lens=[10, 10], new=[30, 30], held=[1, 1], bs=16, free_n=9, room=41),
             dict(lens=[10, 10], new=[30, 30], held=[1, 1], bs=16, free_n=3, room=60, n_free=5),
             dict(lens=[10, 10], new=[30, 30], held=[1, 1], bs=16, free_n=3, room=60, n_free=-2),
             dict(lens=[0], new=[4], held=[0], bs=16, free_n=0, room=4)]
    for c in cases:
        _check_plan(C, **c)
        with pytest.raises(C.CQError):
            C.cq_device_status()
        C.cq_device_status()


def test_plan_refuses(C):
    a, t = _i32([1, 2]), torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    ok = dict(seq_lens=a, new_lens=a, held=a, block_table=t, free_list=a, n_free=a[:1], block_size=16, n_tokens=4)
    for kw, err in ((dict(new_lens=a[:1]), ValueError), (dict(seq_lens=a.long()), TypeError), (dict(block_table=t[:1]), ValueError),
                    (dict(block_table=t.t()), ValueError), (dict(held=a.cpu()), TypeError), (dict(block_size=0), C.CQError),
                    (dict(held_out=a), C.CQError), (dict(n_tokens=None), ValueError)):
        with pytest.raises(err):
            C.cq_kv_plan(**{**ok, **kw})


# ------------------------------------------------------------------------------------------------------- slot writes

def _geom(C, hq, hkv, dk, dv, kb, vb, scale=0.125):
    return C.cq_kv_geometry(hq, hkv, dk, dv, kb, vb, O.analytic_codebook(kb), O.analytic_codebook(vb), scale)


def _check_write(C, hkv, dk, dv, kb, vb, dtype, k, v, slots, cap):
    geom = _geom(C, hkv, hkv, dk, dv, kb, vb)
    rng = np.random.RandomState(1)
    blobs = [rng.randint(0, 256, C.cq_packed_bytes(cap, hkv * d, 128, b)).astype(np.uint8) for d, b in ((dk, kb), (dv, vb))]
    dev = [torch.from_numpy(b).cuda() for b in blobs]
    C.cq_kv_write_slots(geom, dev[0], dev[1], cap, k, v, _i32(slots))
    torch.cuda.synchronize()
    for x, d, b, blob, got in ((k, dk, kb, blobs[0], dev[0]), (v, dv, vb, blobs[1], dev[1])):
        codes, norms = R.encode(_np(x).reshape(len(slots), hkv * d), b, O.analytic_codebook(b))
        wc, wn = R.split_blob(blob, cap, hkv * d, b)
        for i, s in enumerate(slots):
            if 0 <= s < cap:
                wc[s] = R.pack(codes[i:i + 1], R.width_of(b))
                wn[s] = norms[i]
        gc, gn = R.split_blob(got.cpu().numpy(), cap, hkv * d, b)
        np.testing.assert_array_equal(gc, wc)
        np.testing.assert_array_equal(gn.view(np.uint16), wn.view(np.uint16))


@pytest.mark.parametrize("kb,vb", [(2, 2), (3, 4), (4, 5), (5, 3)])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("hkv,dk,dv", [(2, 48, 64), (8, 128, 128), (3, 34, 50), (1, 1, 200)])
def test_write_slots_is_exact(C, kb, vb, dtype, hkv, dk, dv):
    n, cap = 41, 64
    g = torch.Generator(device="cuda").manual_seed(kb + 8 * vb)
    k = (torch.randn(n, hkv * dk, generator=g, device="cuda") * torch.exp(torch.randn(n, 1, generator=g, device="cuda"))).to(dtype)
    v = (torch.randn(n, hkv, dv, generator=g, device="cuda") * 0.05).to(dtype)
    slots = np.random.RandomState(3).permutation(cap)[:n]
    slots[5] = -1
    _check_write(C, hkv, dk, dv, kb, vb, dtype, k, v, slots.tolist(), cap)
    C.cq_device_status()


@pytest.mark.parametrize("bits", [2, 3, 4, 5])
def test_write_slots_borders(C, bits):
    """Zeros, constants, unit vectors and few-valued rows put coordinates on and next to borders between levels."""
    rng = np.random.RandomState(bits)
    rows = [np.zeros(128), np.ones(128), np.eye(128)[0], -np.eye(128)[77], rng.choice([-1.0, 1.0], 128)]
    H = R.hadamard()
    cb = O.analytic_codebook(bits).astype(np.float64)
    mids = (cb[1:] + cb[:-1]) / 2
    for i in range(60):  # rotated coordinate 0 a few units of 2^-24 from a border
        u = rng.randn(128)
        m = mids[i % len(mids)] * (1 + (i - 30) * 2.0 ** -24)
        u[0] = 0
        u *= math.sqrt(1 - m * m) / np.linalg.norm(u)
        u[0] = m
        rows.append(u @ H * 10.0 ** rng.randint(-6, 6))
    rows += [np.full(128, 1e-25), np.full(128, 1e-13), rng.randn(128) * 3e-20, rng.randn(128) * 1e17]
    x = torch.from_numpy(np.array(rows, dtype=np.float32)).cuda()
    _check_write(C, 1, 128, 128, bits, bits, F32, x, x.flip(0).contiguous(), list(range(len(rows))), len(rows) + 3)


def test_write_slots_other_codebooks(C):
    """Codebooks that are not symmetric, with midpoints closer than a cell of the lookup, past the largest
    coordinate, and on round numbers."""
    rng = np.random.RandomState(0)
    x = torch.randn(64, 300, device="cuda")
    books = [np.sort(rng.uniform(-0.3, 0.3, 16)), 0.001 * np.arange(16) - 0.004, np.linspace(-3, 3, 16), np.linspace(-0.25, 0.25, 16),
             np.concatenate([np.linspace(-0.2, 0.2, 15), [9.0]])]
    for cb in books:
        cb = cb.astype(np.float32)
        g = C.cq_kv_geometry(1, 1, 300, 300, 4, 4, cb, cb[::-1] * -1, 1.0)
        blobs = [torch.zeros(C.cq_packed_bytes(64, 300, 128, 4), dtype=torch.uint8, device="cuda") for _ in range(2)]
        C.cq_kv_write_slots(g, *blobs, 64, x, x, _i32(np.arange(64)))
        for blob, book in zip(blobs, (cb, cb[::-1] * -1)):
            codes, norms = R.encode(_np(x), 4, book)
            gc, gn = R.split_blob(blob.cpu().numpy(), 64, 300, 4)
            np.testing.assert_array_equal(gc, R.pack(codes, 4))
            np.testing.assert_array_equal(gn.view(np.uint16), norms.view(np.uint16))


def test_write_slots_non_finite_rows(C):
    """A row with a NaN or an infinity gets a norm that is not finite and reaches no other row."""
    x = torch.randn(9, 128, device="cuda")
    bad = x.clone()
    bad[2, 5], bad[4, 0], bad[6, 9] = math.nan, math.inf, -math.inf
    cb = O.analytic_codebook(4)
    g = C.cq_kv_geometry(1, 1, 128, 128, 4, 4, cb, cb, 1.0)
    out = []
    for rows in (x, bad):
        blobs = [torch.zeros(C.cq_packed_bytes(9, 128, 128, 4), dtype=torch.uint8, device="cuda") for _ in range(2)]
        C.cq_kv_write_slots(g, *blobs, 9, rows, rows, _i32(np.arange(9)))
        out.append(R.split_blob(blobs[0].cpu().numpy(), 9, 128, 4))
    keep = [0, 1, 3, 5, 7, 8]
    np.testing.assert_array_equal(out[0][0][keep], out[1][0][keep])
    np.testing.assert_array_equal(out[0][1][keep], out[1][1][keep])
    assert not np.isfinite(out[1][1][[2, 4, 6]].astype(np.float32)).any()


def test_write_slots_matches_kv_write(C):
    """Away from borders it is cq_kv_write: the same bytes for ordinary rows."""
    x, y = torch.randn(50, 96, device="cuda"), torch.randn(50, 128, device="cuda")
    cb = O.analytic_codebook(4)
    a, b = (torch.zeros(C.cq_packed_bytes(60, w, 128, 4), dtype=torch.uint8, device="cuda") for w in (96, 128))
    c = torch.zeros_like(a)
    C.cq_kv_write_slots(C.cq_kv_geometry(2, 2, 48, 64, 4, 4, cb, cb, 1.0), a, b, 60, x, y, _i32(np.arange(50) + 7))
    C.cq_kv_write(c, 60, 96, 4, cb, x, 7)
    assert (a != c).float().mean() < 1e-3


def test_write_slots_outside_and_strided(C):
    """Slots past the cache are skipped and reported; rows may be slices."""
    big = torch.randn(10, 300, device="cuda")
    k, v = big[:, 3:99], big[:, 100:228]
    slots = [0, 5, -1, 99, 3, -7, 8, 20, 2, 1]
    _check_write(C, 2, 48, 64, 2, 3, F32, k, v, slots, 20)
    with pytest.raises(C.CQError):
        C.cq_device_status()
    _check_write(C, 2, 48, 64, 2, 3, F32, k[:1], v[:1], [19], 20)
    _check_write(C, 2, 48, 64, 2, 3, F32, k[:0], v[:0], [], 20)
    C.cq_device_status()


def test_write_slots_refuses(C):
    g = _geom(C, 2, 2, 48, 64, 2, 2)
    kc, vc = (torch.zeros(C.cq_packed_bytes(8, w, 128, 2), dtype=torch.uint8, device="cuda") for w in (96, 128))
    k, v, s = torch.zeros(4, 96, device="cuda"), torch.zeros(4, 128, device="cuda"), _i32([0, 1, 2, 3])
    for args, err in (((kc[:-1], vc, 8, k, v, s), ValueError), ((kc, vc, 9, k, v, s), ValueError),
                      ((kc, vc, 8, k[:, :95], v, s), ValueError), ((kc, vc, 8, k, v[:3], s), ValueError),
                      ((kc, vc, 8, k, v.half(), s), ValueError), ((kc, vc, 8, k, v, s.long()), TypeError),
                      ((kc, vc, 8, k.int(), v.int(), s), TypeError), ((kc.int(), vc, 8, k, v, s), TypeError)):
        with pytest.raises(err):
            C.cq_kv_write_slots(g, *args)


# -------------------------------------------------------------------------------------------------------- attention

def _blob(cap, width, bits, rng, lo=1.0, hi=8.0):
    """Uniform codes, norms uniform in [lo, hi)."""
    g = -(-width // 128)
    if bits == 5:
        codes = R.pack(rng.choice([0, 1, 3], size=(cap, g * 128)), 2)
    else:
        codes = rng.randint(0, 256, (cap, g * 16 * R.width_of(bits))).astype(np.uint8)
    norms = rng.uniform(lo, hi, (cap, g)).astype(np.float16)
    return np.concatenate([codes.reshape(-1), norms.view(np.uint8).reshape(-1)])


def _tree_mask(nodes, rng, words, empty=False):
    bits = np.zeros((sum(nodes), words * 32), dtype=bool)
    at = 0
    for n in nodes:
        for i in range(n):
            p = rng.randint(-1, i) if i else -1
            if p >= 0:
                bits[at + i] = bits[at + p]
            bits[at + i, i] = True
        if empty and n:
            bits[at + n - 1] = False
        at += n
    return bits, np.packbits(bits, axis=1, bitorder="little").view(np.int32)


def _check_attend(C, geom, kb, vb, ctx, nodes, bs=16, dtype=F16, masked=True, empty=False, seed=0, poison=True, scale=None,
                  lo=1.0, hi=8.0, q_scale=1.0, max_nodes=None, words=None, contiguous=False, books=None, rms=None):
    hq, hkv, dk, dv = geom
    rng = np.random.RandomState(seed)
    pages = [-(-(c + n) // bs) for c, n in zip(ctx, nodes)]
    blocks = sum(pages) + 2
    perm, wide = rng.permutation(blocks), max(pages + [1]) + 1
    table, at = np.full((len(ctx), wide), -1), 0
    for s, p in enumerate(pages):
        table[s, :p] = perm[at:at + p]
        at += p
    cap = blocks * bs
    kc, vc = _blob(cap, hkv * dk, kb, rng, lo, hi), _blob(cap, hkv * dv, vb, rng, lo, hi)
    most = max(nodes) if max_nodes is None else max_nodes
    words = words or max(1, -(-most // 32))
    bits, mask = _tree_mask(nodes, rng, words, empty)
    cu = np.concatenate([[0], np.cumsum(nodes)])
    total = int(cu[-1])
    if poison:  # rows that nobody attends hold NaN norms: the rest of the pool, and drafted tokens no row's mask has
        used = np.zeros(cap, dtype=bool)
        for s in range(len(ctx)):
            vis = np.ones(ctx[s] + nodes[s], dtype=bool)
            if masked:
                vis[ctx[s]:] = bits[cu[s]:cu[s + 1], :nodes[s]].any(0)
            if not nodes[s]:
                vis[:] = False
            p = np.nonzero(vis)[0]
            used[table[s, p // bs] * bs + p % bs] = True
        for blob, w, b in ((kc, hkv * dk, kb), (vc, hkv * dv, vb)):
            R.split_blob(blob, cap, w, b)[1][~used] = np.nan
    big = torch.randn(total, hq + 1, dk + 3, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed)) * q_scale
    q = big.to(dtype)[:, 1:, 2:2 + dk]
    if contiguous:
        q = q.contiguous()
    out = torch.full((total, hq, dv + 5), 7.0, dtype=dtype, device="cuda")
    scale = 1.0 / math.sqrt(dk) if scale is None else scale
    cbk, cbv = books or (O.analytic_codebook(kb), O.analytic_codebook(vb))
    g = C.cq_kv_geometry(hq, hkv, dk, dv, kb, vb, cbk, cbv, scale)
    C.cq_kv_tree_attend(g, q, torch.from_numpy(kc).cuda(), torch.from_numpy(vc).cuda(), cap, _i32(table), bs, _i32(ctx), _i32(cu),
                        torch.from_numpy(mask).cuda() if masked else None, most, o=out[..., 2:2 + dv])
    torch.cuda.synchronize()
    C.cq_device_status()
    got = _np(out)
    assert (got[..., :2] == 7).all() and (got[..., 2 + dv:] == 7).all()
    got = got[..., 2:2 + dv]
    seen = (lambda s, i, j: bits[cu[s] + i, j]) if masked else (lambda s, i, j: j <= i)
    want, bound = R.attend(_np(q), kc, vc, cap, table, bs, ctx, cu, seen, geom, kb, vb, cbk, cbv, np.float64(np.float32(scale)))
    tol = bound + R.HALF_STEP[_name(dtype)] * (np.abs(want) + bound) + R.TINY[_name(dtype)]
    err = np.abs(got - want)
    assert np.isfinite(got).all()
    assert (err <= tol).all(), f"worst error/tolerance {np.max(err / np.maximum(tol, 1e-300)):.3g}"
    if rms is not None:
        share = math.sqrt(np.mean(err ** 2) / np.mean(want ** 2))
        assert share <= rms, f"{share:.2e} of the result's size, allowed {rms:.2e}"
    return got, float(np.max(err / np.maximum(tol, 1e-300))) if total else 0.0


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("geom", [(12, 2, 48, 64), (8, 4, 64, 64), (8, 2, 128, 128), (6, 6, 80, 80), (4, 1, 256, 256), (6, 3, 40, 24), (1, 1, 16, 16)])
@pytest.mark.parametrize("nodes", [[1], [2, 0, 5], [33, 3]])
def test_attend_contiguous_queries(C, dtype, geom, nodes):
    """Queries on vector boundaries, as they come from cq_qk_norm_rope; each request's context spans several blocks."""
    _check_attend(C, geom, 4, 2, ctx=[300 + 7 * i for i in range(len(nodes))], nodes=nodes, dtype=dtype, contiguous=True, seed=sum(geom))


GEOMS = [(12, 2, 48, 64), (8, 4, 64, 64), (8, 2, 128, 128), (4, 1, 256, 256), (6, 6, 80, 80), (6, 3, 40, 24), (16, 1, 128, 64),
         (3, 3, 1, 5), (4, 2, 96, 128), (2, 2, 256, 48)]


@pytest.mark.parametrize("geom", GEOMS)
@pytest.mark.parametrize("bits", [(2, 2), (3, 4), (4, 5), (5, 3)])
def test_attend_geometries(C, geom, bits):
    """Ragged requests: no context, one token, tiles filled to the brim and one over, no drafted tokens at all."""
    _, worst = _check_attend(C, geom, *bits, ctx=[0, 1, 127, 128, 300, 55], nodes=[5, 1, 1, 2, 13, 0], seed=sum(geom) + bits[0])
    print(f"{geom} {bits}: worst error / tolerance {worst:.2e}")


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("nodes", [[1], [2], [16], [17, 0, 3], [64, 1, 63], [100], [256, 7]])
def test_attend_tree_sizes(C, dtype, nodes):
    _check_attend(C, (4, 2, 64, 64), 4, 4, ctx=[70 + 41 * i for i in range(len(nodes))], nodes=nodes, dtype=dtype, seed=len(nodes))


@pytest.mark.parametrize("bs", [1, 7, 16, 48, 128, 200, 1024])
def test_attend_block_sizes(C, bs):
    """Blocks that end inside a tile, blocks larger than one."""
    _check_attend(C, (4, 2, 128, 128), 2, 3, ctx=[333, 129], nodes=[9, 20], bs=bs, seed=bs)


@pytest.mark.parametrize("masked", [False, True])
def test_attend_without_context(C, masked):
    """Only drafted tokens; with a mask, one of them attends nothing."""
    got, _ = _check_attend(C, (8, 4, 64, 64), 4, 4, ctx=[0, 0, 0], nodes=[33, 1, 130], masked=masked, empty=masked)
    if masked:
        assert (got[32] == 0).all() and (got[33] == 0).all() and (got[-1] == 0).all()


@pytest.mark.parametrize("kb,vb", [(4, 4), (2, 4), (4, 2), (3, 3), (2, 2)])
@pytest.mark.parametrize("nodes", [[3], [40, 2]])
def test_attend_own_codebooks(C, kb, vb, nodes):
    """Codebooks that are not symmetric, differ between keys and values, and are of another size than the
    analytic ones: two large level tables leave less room for the columns of a large tree."""
    rng = np.random.RandomState(kb + vb)
    books = tuple((np.sort(rng.uniform(-1, 1, 2 ** b)) * s + 0.01 * s).astype(np.float32) for b, s in ((kb, 0.3), (vb, 40.0)))
    _check_attend(C, (8, 2, 128, 128), kb, vb, ctx=[250, 3][:len(nodes)], nodes=nodes, dtype=BF16, books=books, seed=kb)
    _check_attend(C, (8, 4, 64, 64), kb, vb, ctx=[250, 3][:len(nodes)], nodes=nodes, dtype=F16, books=books, seed=vb, contiguous=True)


def test_attend_negative_norms(C):
    """A norm below zero turns its row round; the formula holds for it as for any other."""
    _check_attend(C, (8, 4, 64, 64), 4, 3, ctx=[150], nodes=[5], lo=-4.0, hi=4.0)
    _check_attend(C, (4, 1, 256, 256), 2, 4, ctx=[150], nodes=[5], lo=-4.0, hi=4.0)
    _check_attend(C, (4, 1, 128, 128), 3, 2, ctx=[150], nodes=[33], lo=-4.0, hi=4.0)


def test_attend_all_requests_empty(C):
    """No drafted tokens at all: nothing is written, nothing is reported."""
    cb = O.analytic_codebook(2)
    g = C.cq_kv_geometry(4, 2, 48, 64, 2, 2, cb, cb, 0.125)
    kc, vc = (torch.from_numpy(_blob(64, w, 2, np.random.RandomState(i))).cuda() for i, w in ((1, 96), (2, 128)))
    o = torch.full((3, 4, 64), 5.0, dtype=F16, device="cuda")
    C.cq_kv_tree_attend(g, torch.zeros(3, 4, 48, dtype=F16, device="cuda"), kc, vc, 64, _i32([[0, 1], [2, 3]]), 16, _i32([20, 7]),
                        _i32([0, 0, 0]), None, 3, o=o)
    torch.cuda.synchronize()
    assert (o == 5).all()
    C.cq_device_status()


def test_attend_causal_chunk(C):
    _check_attend(C, (8, 2, 128, 128), 4, 3, ctx=[200, 0, 5], nodes=[128, 200, 31], masked=False)


def test_attend_long_context_in_parts(C):
    """Contexts that many thread blocks share; a short request in the same call."""
    _check_attend(C, (8, 4, 64, 64), 2, 2, ctx=[20011, 64], nodes=[3, 2], bs=64)
    _check_attend(C, (4, 1, 128, 128), 3, 2, ctx=[9000], nodes=[40], bs=32, dtype=BF16)


def test_attend_many_requests(C):
    rng = np.random.RandomState(0)
    _check_attend(C, (4, 2, 48, 64), 2, 2, ctx=rng.randint(0, 60, 700).tolist(), nodes=rng.randint(0, 3, 700).tolist(), max_nodes=8)


def test_attend_many_uneven_requests(C):
    """Lengths from nothing to several tiles: the runs of the thread blocks begin and end anywhere, and
    the requests are more than a block's threads."""
    rng = np.random.RandomState(1)
    ctx = np.where(rng.rand(700) < 0.1, rng.randint(100, 900, 700), rng.randint(0, 40, 700))
    _check_attend(C, (4, 2, 48, 64), 2, 3, ctx=ctx.tolist(), nodes=rng.randint(0, 3, 700).tolist())
    _check_attend(C, (4, 1, 128, 128), 4, 2, ctx=ctx[:90].tolist(), nodes=rng.randint(0, 40, 90).tolist(), dtype=BF16)


@pytest.mark.parametrize("geom", [(8, 4, 64, 64), (4, 1, 128, 128), (4, 1, 256, 256), (6, 6, 80, 80)])
@pytest.mark.parametrize("bits", [(2, 2), (4, 4), (5, 3)])
@pytest.mark.parametrize("nodes", [[3], [40]])
def test_attend_fp16_precision(C, geom, bits, nodes):
    """An fp16 result carries three roundings to fp16, of the weights, of the result and, where a head has two groups, of the
    values of one: each of at most half a step, uniform, so 2^-11 / sqrt(3) of the value in the mean square, and sqrt(3)
    times that together. (Queries in one fp16 term would add as much again.)"""
    _check_attend(C, geom, *bits, ctx=[2500], nodes=nodes, contiguous=True, seed=geom[2] + bits[0], q_scale=1.5, rms=2.0 ** -11)


def test_attend_peaked_flat_and_extreme_sizes(C):
    """Nearly one-hot and uniform weights; queries and norms of extreme size; growing logits."""
    _check_attend(C, (4, 2, 64, 64), 2, 4, ctx=[400], nodes=[9], lo=20.0, hi=40.0, q_scale=4.0)
    _check_attend(C, (4, 2, 64, 64), 2, 4, ctx=[400], nodes=[9], scale=0.0)
    _check_attend(C, (4, 2, 64, 64), 4, 4, ctx=[400], nodes=[9], scale=-0.1)
    _check_attend(C, (4, 2, 64, 64), 4, 4, ctx=[300], nodes=[9], dtype=BF16, q_scale=1e8, scale=1e-9)
    _check_attend(C, (4, 2, 64, 64), 4, 4, ctx=[300], nodes=[9], dtype=BF16, q_scale=1e-12, scale=1e11)
    _check_attend(C, (4, 2, 64, 64), 4, 4, ctx=[300], nodes=[9], dtype=BF16, lo=1e-4, hi=2e-4, scale=1000.0)
    _check_attend(C, (4, 2, 64, 64), 4, 4, ctx=[300], nodes=[9], dtype=BF16, lo=3e4, hi=6e4, scale=1e-5)


def test_attend_logits_that_grow_along_the_context(C):
    """The running maximum rises in every tile; a zero norm among the values counts in the denominator."""
    hq, hkv, d, n, bs = 2, 1, 128, 1000, 64
    rng = np.random.RandomState(5)
    cap = 1024
    kc, vc = _blob(cap, d, 4, rng), _blob(cap, d, 4, rng)
    row = np.tile(R.split_blob(kc, cap, d, 4)[0][:1], (cap, 1))
    R.split_blob(kc, cap, d, 4)[0][:] = row
    R.split_blob(kc, cap, d, 4)[1][:, 0] = np.linspace(0.5, 60, cap)
    R.split_blob(vc, cap, d, 4)[1][::3] = 0
    cb = O.analytic_codebook(4)
    k0 = R.dequant(kc, cap, d, 4, cb, np.array([100]))[0][0]
    q = torch.from_numpy(np.stack([k0, -k0]) / np.linalg.norm(k0) * 12).to(F16).cuda()[None]
    g = C.cq_kv_geometry(hq, hkv, d, d, 4, 4, cb, cb, 0.5)
    table = np.arange(cap // bs)[None]
    o = C.cq_kv_tree_attend(g, q, torch.from_numpy(kc).cuda(), torch.from_numpy(vc).cuda(), cap, _i32(table), bs, _i32([n]),
                            _i32([0, 1]), None, 1)
    want, bound = R.attend(_np(q), kc, vc, cap, table, bs, [n], [0, 1], lambda s, i, j: True, (hq, hkv, d, d), 4, 4, cb, cb, 0.5)
    assert (np.abs(_np(o) - want) <= bound + 2.0 ** -11 * (np.abs(want) + bound) + 2.0 ** -25).all()


def test_attend_infinite_and_nan_norms_reach_only_who_attends_them(C):
    """Drafted token 1 has NaN and infinite norms: its own row is lost, its siblings are as without it."""
    hq, hkv, d, bs, ctx, n = 4, 2, 64, 16, 37, 4
    rng = np.random.RandomState(2)
    cap = 64
    cb = O.analytic_codebook(2)
    g = C.cq_kv_geometry(hq, hkv, d, d, 2, 2, cb, cb, 0.125)
    mask = _i32([[0b0001], [0b0010], [0b0101], [0b1001]])
    q = torch.randn(n, hq, d, device="cuda").to(F16)
    table = _i32([[2, 0, 3]])

    def run(kn, vn):
        kc, vc = _blob(cap, hkv * d, 2, np.random.RandomState(2)), _blob(cap, hkv * d, 2, np.random.RandomState(3))
        r = 3 * bs + (ctx + 1) % bs
        R.split_blob(kc, cap, hkv * d, 2)[1][r] = kn
        R.split_blob(vc, cap, hkv * d, 2)[1][r] = vn
        return C.cq_kv_tree_attend(g, q, torch.from_numpy(kc).cuda(), torch.from_numpy(vc).cuda(), cap, table, bs, _i32([ctx]),
                                   _i32([0, n]), mask, n)

    clean = run(1.0, 1.0)
    for kn, vn in ((np.nan, 1.0), (1.0, np.nan), (np.inf, np.inf), (-np.inf, 1.0), (65504.0, 65504.0), (0.0, 0.0)):
        got = run(kn, vn)
        keep = [0, 2, 3]
        assert torch.equal(got[keep], clean[keep]), (kn, vn)
        if np.isnan(kn) or np.isnan(vn):
            assert got[1].isnan().any()


def test_attend_non_finite_query_stays_in_its_row(C):
    cb = O.analytic_codebook(4)
    g = C.cq_kv_geometry(4, 2, 64, 64, 4, 4, cb, cb, 0.125)
    kc, vc = (torch.from_numpy(_blob(64, 128, 4, np.random.RandomState(i))).cuda() for i in (1, 2))
    q = torch.randn(3, 4, 64, device="cuda").to(BF16)
    bad = q.clone()
    bad[1, 2, 7] = math.inf
    bad[2, 0, 0] = math.nan
    run = lambda x: C.cq_kv_tree_attend(g, x, kc, vc, 64, _i32([[0, 1]]), 32, _i32([50]), _i32([0, 3]), None, 3)  # noqa: E731
    a, b = run(q), run(bad)
    assert b[1, 2].isnan().all() and b[2, 0].isnan().all()
    ok = torch.ones(3, 4, dtype=torch.bool)
    ok[1, 2] = ok[2, 0] = False
    assert torch.equal(a[ok.cuda()], b[ok.cuda()])


def test_attend_reports_bad_pages_and_lengths(C):
    """A block number outside the pool, a table too short, more drafted tokens
    than max_nodes or than rows of q: nothing out of range is touched and the
    status says so."""
    cb = O.analytic_codebook(2)
    g = C.cq_kv_geometry(4, 2, 48, 64, 2, 2, cb, cb, 0.125)
    kc, vc = (torch.from_numpy(_blob(64, w, 2, np.random.RandomState(i))).cuda() for i, w in ((1, 96), (2, 128)))
    q = torch.randn(3, 4, 48, device="cuda").to(F16)

    def run(table, ctx, cu, most):
        o = torch.full((3, 4, 64), 5.0, dtype=F16, device="cuda")
        C.cq_kv_tree_attend(g, q, kc, vc, 64, _i32(table), 16, _i32(ctx), _i32(cu), None, most, o=o)
        torch.cuda.synchronize()
        return o

    good = run([[0, 1, 2]], [40], [0, 3], 3)
    C.cq_device_status()
    assert torch.isfinite(good).all()
    for table, ctx, cu, most in (([[0, 4, 2]], [40], [0, 3], 3), ([[0, -1, 2]], [40], [0, 3], 3), ([[0, 2 ** 30, 2]], [40], [0, 3], 3),
                                 ([[0, 1]], [40], [0, 3], 3), ([[0, 1, 2]], [40], [0, 3], 2), ([[0, 1, 2]], [40], [0, 9], 3),
                                 ([[0, 1, 2]], [-5], [0, 3], 3), ([[0, 1, 2]], [2 ** 31 - 1], [0, 3], 3),
                                 ([[0, 1, 2]], [40], [-2, 1], 3), ([[0, 1, 2]] * 2, [40, 3], [0, 3, 1], 3)):
        o = run(table, ctx, cu, most)
        assert not o.isnan().any()
        with pytest.raises(C.CQError):
            C.cq_device_status()
        C.cq_device_status()
    assert torch.equal(run([[0, 1, 2]], [40], [0, 3], 3), good)


def test_attend_offsets_past_32_bits(C):
    """Rows at the end of caches of more than 2^32 bytes, written and attended."""
    hkv, d, bs = 64, 128, 16
    row = C.cq_packed_bytes(1, hkv * d, 128, 4)
    cap = ((1 << 32) // (row - 128) + 4096) // bs * bs
    cb = O.analytic_codebook(4)
    g = C.cq_kv_geometry(hkv, hkv, d, d, 4, 4, cb, cb, d ** -0.5)
    kc, vc = (torch.zeros(C.cq_packed_bytes(cap, hkv * d, 128, 4), dtype=torch.uint8, device="cuda") for _ in range(2))
    small = [torch.zeros(C.cq_packed_bytes(64, hkv * d, 128, 4), dtype=torch.uint8, device="cuda") for _ in range(2)]
    k, v = (torch.randn(40, hkv, d, device="cuda").to(BF16) for _ in range(2))
    q = torch.randn(2, hkv, d, device="cuda").to(BF16)
    last = cap // bs - 1
    out = []
    for (a, b), c, table in (((kc, vc), cap, [last, 1, last - 1]), (small, 64, [3, 1, 2])):
        t = np.arange(40)
        C.cq_kv_write_slots(g, a, b, c, k, v, _i32(np.array(table)[t // bs] * bs + t % bs))
        out.append(C.cq_kv_tree_attend(g, q, a, b, c, _i32([table]), bs, _i32([38]), _i32([0, 2]), None, 2))
    torch.cuda.synchronize()
    assert torch.equal(out[0], out[1]) and torch.isfinite(out[0]).all()
    C.cq_device_status()


def test_attend_refuses(C):
    cb = O.analytic_codebook(2)
    g = C.cq_kv_geometry(4, 2, 48, 64, 2, 2, cb, cb, 0.125)
    kc, vc = (torch.zeros(C.cq_packed_bytes(64, w, 128, 2), dtype=torch.uint8, device="cuda") for w in (96, 128))
    q, t, c, cu = torch.zeros(3, 4, 48, dtype=F16, device="cuda"), _i32([[0, 1]]), _i32([4]), _i32([0, 3])
    m = _i32([[1], [3], [7]])
    ok = dict(geom=g, q=q, k_cache=kc, v_cache=vc, cap=64, block_table=t, block_size=16, context_lens=c, cu_nodes=cu, mask=m,
              max_nodes=3)
    C.cq_kv_tree_attend(**ok)
    for kw, err in ((dict(q=q.float()), TypeError), (dict(q=q[:, :3]), ValueError), (dict(cap=65), ValueError),
                    (dict(cu_nodes=cu[:1]), ValueError), (dict(mask=m[:2]), ValueError), (dict(mask=m.long()), ValueError),
                    (dict(max_nodes=257), C.CQError), (dict(max_nodes=40), C.CQError), (dict(block_size=0), C.CQError),
                    (dict(block_table=t[0]), ValueError), (dict(o=torch.zeros(3, 4, 64, device="cuda")), ValueError),
                    (dict(context_lens=c.cpu()), TypeError), (dict(k_cache=kc.cpu()), TypeError)):
        with pytest.raises(err):
            C.cq_kv_tree_attend(**{**ok, **kw})


# --------------------------------------------------------------------------------------------- the step as a whole

class _Step:
    """A verification step over static buffers, as a server captures it."""

    def __init__(self, C, seed=0):
        self.C = C
        hq, hkv, dk, dv, self.bs, s, room = 12, 2, 48, 64, 16, 5, 64
        rng = np.random.RandomState(seed)
        cb = O.analytic_codebook(4)
        self.geom = C.cq_kv_geometry(hq, hkv, dk, dv, 4, 4, cb, cb, dk ** -0.5)
        self.cap = 80 * self.bs
        self.kc, self.vc = (torch.from_numpy(_blob(self.cap, hkv * d, 4, rng)).cuda() for d in (dk, dv))
        self.lens, self.new = _i32([0, 17, 100, 33, 250]), _i32([3, 8, 0, 16, 1])
        self.held = _i32([0, 2, 7, 3, 16])
        self.table = torch.full((s, 20), -1, dtype=torch.int32, device="cuda")
        at = 0
        for i, h in enumerate(self.held.tolist()):
            self.table[i, :h] = torch.arange(at, at + h)
            at += h
        self.free, self.n_free = _i32(np.arange(at, 80)), _i32([80 - at])
        self.q, self.k = torch.randn(room, hq, dk, device="cuda"), torch.randn(room, hkv, dk, device="cuda")
        self.v = torch.randn(room, hkv, dv, device="cuda")
        self.rates = C.cq_rope_init(dk)
        self.room = room

    def run(self):
        C = self.C
        p = C.cq_kv_plan(self.lens, self.new, self.held, self.table, self.free, self.n_free, self.bs, self.room)
        q, k = C.cq_qk_norm_rope(self.q, self.k, p["positions"], self.rates, q_dtype=F16)
        C.cq_kv_write_slots(self.geom, self.kc, self.vc, self.cap, k, self.v, p["slots"])
        o = torch.zeros(self.room, 12, 64, dtype=F16, device="cuda")
        return C.cq_kv_tree_attend(self.geom, q, self.kc, self.vc, self.cap, self.table, self.bs, self.lens, p["cu_new"], None, 32, o=o)


def test_step_matches_definition(C):
    st = _Step(C)
    o = st.run()
    torch.cuda.synchronize()
    C.cq_device_status()
    cu = np.concatenate([[0], np.cumsum(st.new.cpu().numpy())])
    total = int(cu[-1])
    assert (o[total:] == 0).all()
    pos = np.concatenate([l + np.arange(n) for l, n in zip(st.lens.tolist(), st.new.tolist())])
    q = R.rope(_np(st.q[:total]), None, pos, 10000.0 ** (-np.arange(0, 48, 2) / 48), 1e-6, 0.0, False)[0].astype(np.float16)
    cb = O.analytic_codebook(4)
    want, bound = R.attend(q, st.kc.cpu().numpy(), st.vc.cpu().numpy(), st.cap, st.table.cpu().numpy(), st.bs, st.lens.tolist(), cu,
                           lambda s, i, j: j <= i, (12, 2, 48, 64), 4, 4, cb, cb, np.float64(np.float32(48 ** -0.5)))
    # the query may round to the neighbouring fp16 value: one more rounding of it in each logit, as the bound's first term has two
    tol = 2 * bound + 2.0 ** -11 * np.abs(want) + 2.0 ** -24
    assert (np.abs(_np(o[:total]) - want) <= tol).all()


def test_step_on_another_stream_and_in_a_graph(C):
    """The same bits on a side stream, and replayed from a graph with other lengths in the same buffers."""
    base = _Step(C)
    want = base.run().clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    st = _Step(C)
    for x in ("q", "k", "v"):
        getattr(st, x).copy_(getattr(base, x))
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = st.run()
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        out = st.run()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    other, fresh = _i32([20, 1, 3, 40, 300]), _i32([1, 1, 20, 4, 9])
    held = _i32([2, 1, 1, 3, 19])
    for x in (st, base):
        x.lens.copy_(other), x.new.copy_(fresh), x.held.copy_(held)
        x.table.fill_(-1)
        for i, h in enumerate(held.tolist()):
            x.table[i, :h] = torch.arange(16 * i, 16 * i + h)
        x.table[4, :19] = torch.arange(40, 59)
        x.free[:4] = torch.arange(70, 74)
        x.n_free.fill_(4)
    g.replay()
    want = base.run()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    C.cq_device_status()


def test_results_do_not_depend_on_the_run(C):
    """No atomics on results: the same bits every time."""
    cb = O.analytic_codebook(2)
    g = C.cq_kv_geometry(8, 2, 128, 128, 2, 2, cb, cb, 128 ** -0.5)
    cap, bs = 6400, 64
    kc, vc = (torch.from_numpy(_blob(cap, 256, 2, np.random.RandomState(i))).cuda() for i in (1, 2))
    q = torch.randn(70, 8, 128, device="cuda").to(BF16)
    args = (g, q, kc, vc, cap, _i32(np.arange(100).reshape(2, 50)), bs, _i32([3000, 2500]), _i32([0, 60, 70]), None, 64)
    first = C.cq_kv_tree_attend(*args)
    for _ in range(20):
        assert torch.equal(C.cq_kv_tree_attend(*args), first)


def test_example_tree_gives_what_single_tokens_give():
    """The example's layer: the verified path of a tree against the same tokens one
    at a time. Both attend the same cache rows in another order: fp16 roundings of
    the attention (2^-10), and at most one step of the int8 quantisation behind it
    (1/127 of the largest element), of which few elements take one."""
    from examples import verify_drafts
    worst, accepted, _ = verify_drafts.run(requests=3, context=40, nodes=9, steps=3)
    assert accepted >= 9 and worst < 2 ** -10 + 1 / 127
