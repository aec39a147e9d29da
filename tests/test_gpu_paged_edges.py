"""GPU tests of the paged cache's operators at the ends of their ranges: sizes far apart in one call, values past what
fp32 squares hold, long contexts under one dominant row, lengths that leave 32 bits, waits that run out."""
import math

import numpy as np
import pytest
import torch

import oracle as O
from tests import paged_reference as R
from tests.test_gpu_paged import BF16, F16, _blob, _i32, _np

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def C():
    import hadamard_rotated_codebook_gb300 as pkg
    return pkg


class _Pool:
    """One request of `ctx` cached and `n` drafted tokens, causal."""

    def __init__(self, C, geom, bits, ctx, n, scale, seed=0, bs=32):
        self.C, self.dims, self.bits, self.ctx, self.n, self.bs, self.scale = C, geom, bits, ctx, n, bs, scale
        hq, hkv, dk, dv = geom
        rng = np.random.RandomState(seed)
        self.cap = (ctx + n + bs - 1) // bs * bs
        self.kc, self.vc = _blob(self.cap, hkv * dk, bits, rng), _blob(self.cap, hkv * dv, bits, rng)
        self.cb = O.analytic_codebook(bits)
        self.g = C.cq_kv_geometry(hq, hkv, dk, dv, bits, bits, self.cb, self.cb, scale)
        self.table = rng.permutation(self.cap // bs)[None]
        self.q = torch.randn(n, hq, dk, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed))

    def run(self, q):
        kc, vc = (torch.from_numpy(x).cuda() for x in (self.kc, self.vc))
        o = self.C.cq_kv_tree_attend(self.g, q, kc, vc, self.cap, _i32(self.table), self.bs, _i32([self.ctx]), _i32([0, self.n]), None, self.n)
        torch.cuda.synchronize()
        self.C.cq_device_status()
        return o

    def reference(self, q):
        return R.attend(_np(q), self.kc, self.vc, self.cap, self.table, self.bs, [self.ctx], [0, self.n], lambda s, i, j: j <= i, self.dims,
                        self.bits, self.bits, self.cb, self.cb, np.float64(np.float32(self.scale)))


# whole runs of 16 and not, one group and two
SPANS = [(4, 2, 64, 64), (6, 3, 40, 24), (8, 2, 128, 128), (6, 6, 80, 80), (4, 1, 256, 256)]


@pytest.mark.parametrize("geom", SPANS)
@pytest.mark.parametrize("n", [4, 40])
@pytest.mark.parametrize("dtype,factor", [(BF16, 2.0 ** 28), (BF16, 1e12), (BF16, 1e30), (BF16, 6e37), (BF16, 1e-30), (F16, 2.0 ** 13), (F16, 2.0 ** -12)])
def test_attend_a_query_of_another_size_leaves_its_tile_mates_alone(C, geom, n, dtype, factor):
    """One token, and one head of another, are far larger (or smaller) than the rest of their column tile: every other
    row has the bits that it has without them, and they have the bits that they have by themselves."""
    pool = _Pool(C, geom, 4, 150, n, 0.125, seed=geom[2] + n)
    q = pool.q.to(dtype)
    odd = torch.zeros(n, geom[0], dtype=torch.bool, device="cuda")
    odd[1] = odd[2, geom[0] - 1] = True
    mixed = torch.where(odd[..., None], (q.float() * factor).to(dtype), q)
    assert torch.isfinite(mixed).all()
    a, b = pool.run(q), pool.run(mixed)
    assert torch.equal(a[~odd], b[~odd])
    alone = pool.run(torch.where(odd[..., None], mixed, torch.zeros_like(q)))
    assert torch.equal(alone[odd].nan_to_num(7e4), b[odd].nan_to_num(7e4))


@pytest.mark.parametrize("geom", SPANS)
@pytest.mark.parametrize("scale", [0.125, 0.125 * 2.0 ** -40])
def test_attend_queries_of_every_size_match_the_definition(C, geom, scale):
    """Token i is 2^(5 i - 20) times as large: the logits of some or of others are of ordinary size, and the definition's
    bound holds for each row by itself."""
    n = 9
    pool = _Pool(C, geom, 4, 150, n, scale, seed=geom[2])
    size = 2.0 ** (5.0 * torch.arange(n, device="cuda") - 20) if scale > 1e-3 else 2.0 ** (5.0 * torch.arange(n, device="cuda"))
    q = (pool.q * size[:, None, None]).to(BF16)
    got = _np(pool.run(q))
    with np.errstate(over="ignore", invalid="ignore"):
        want, bound = pool.reference(q)
        tol = bound + R.HALF_STEP["bfloat16"] * (np.abs(want) + bound) + R.TINY["bfloat16"]
    tol = np.where(np.isnan(tol), np.inf, tol)  # logits past what the bound's exponential holds
    assert np.isfinite(got).all() and (np.abs(got - want) <= tol).all()
    assert np.isfinite(tol).mean() > 0.3


@pytest.mark.parametrize("where", [0, 40, 5000])
@pytest.mark.parametrize("gap", [17.5, 22.3, 25.05])
@pytest.mark.parametrize("n", [1, 40])
def test_attend_rows_far_below_a_dominant_one_still_count(C, where, gap, n):
    """131071 rows with 2^-gap times the weight of one row, which comes first, later or much later, in more requests than
    thread blocks, so that one block has nearly all of a request. Together they are 0.4% to 70% of that row, against its
    sign. Allowed in the 2-norm: one rounding of the result and one of the dominant weight, 2^-11 each, and a quarter of one
    for levels, the others' weights and sums."""
    seqs, ctx, d, bs = 160, 131071, 128, 1024
    cap = (ctx + n + bs - 1) // bs * bs
    cb = O.analytic_codebook(2)
    rng = np.random.RandomState(where + n)
    kc, vc = _blob(cap, d, 2, rng), _blob(cap, d, 2, rng)
    kn, (vcodes, vn) = R.split_blob(kc, cap, d, 2)[1], R.split_blob(vc, cap, d, 2)
    kn[:] = 0  # a logit of exactly zero
    kn[where], vn[:] = 1.0, 1.0
    vcodes[:] = vcodes[where]
    vn[where] = -1.0
    k0 = R.dequant(kc, cap, d, 2, cb, np.array([where]))[0][0]
    q = torch.from_numpy(k0 / np.dot(k0, k0) * gap * math.log(2)).to(F16).cuda().expand(seqs * n, 1, d).contiguous()
    g = C.cq_kv_geometry(1, 1, d, d, 2, 2, cb, cb, 1.0)
    table = torch.arange(cap // bs, dtype=torch.int32, device="cuda").expand(seqs, -1).contiguous()
    o = C.cq_kv_tree_attend(g, q, torch.from_numpy(kc).cuda(), torch.from_numpy(vc).cuda(), cap, table, bs, _i32([ctx] * seqs),
                            _i32(np.arange(seqs + 1) * n), None, n)
    torch.cuda.synchronize()
    C.cq_device_status()
    top = np.exp(np.dot(_np(q[0, 0]), k0))
    v = R.dequant(vc, cap, d, 2, cb, np.array([where]))[0][0]  # the others are its negative
    rows = ctx + np.tile(np.arange(n), seqs)  # others that a token attends
    want = v[None] * ((top - rows) / (top + rows))[:, None]
    err = np.linalg.norm(_np(o[:, 0]) - want, axis=1) / np.linalg.norm(v)
    print(f"worst {err.max() * 2048:.2f} of 2^-11")
    assert (err <= 2.25 * 2.0 ** -11).all()


@pytest.mark.parametrize("geom", [(4, 1, 64, 64), (2, 1, 128, 128), (1, 1, 256, 256), (3, 3, 80, 80)])
@pytest.mark.parametrize("n", [1, 12, 40])
@pytest.mark.parametrize("first,last", [(0.5, 24.0), (24.0, 0.5)])
def test_attend_long_parts_are_joined_from_chunks(C, geom, n, first, last):
    """More requests (over the same rows) than thread blocks, so that a block sums 20000 rows of one; key norms that grow or
    shrink along the context, so that the chunks' references lie far apart."""
    hq, hkv, dk, dv = geom
    pool = _Pool(C, geom, 4, 20000, n, 0.25, seed=n + dk)
    R.split_blob(pool.kc, pool.cap, hkv * dk, 4)[1][pool.table[0][np.arange(pool.cap) // pool.bs] * pool.bs + np.arange(pool.cap) % pool.bs] = \
        np.linspace(first, last, pool.cap).astype(np.float16)[:, None]
    seqs = 160
    q = pool.q.to(F16)
    o = C.cq_kv_tree_attend(pool.g, q.repeat(seqs, 1, 1), torch.from_numpy(pool.kc).cuda(), torch.from_numpy(pool.vc).cuda(), pool.cap,
                            _i32(np.repeat(pool.table, seqs, 0)), pool.bs, _i32([pool.ctx] * seqs), _i32(np.arange(seqs + 1) * n), None, n)
    torch.cuda.synchronize()
    C.cq_device_status()
    want, bound = pool.reference(q)
    tol = bound + R.HALF_STEP["float16"] * (np.abs(want) + bound) + R.TINY["float16"]
    err = np.abs(_np(o).reshape(seqs, n, hq, dv) - want)
    assert (err <= tol).all(), f"worst error/tolerance {np.max(err / tol):.3g}"

@pytest.mark.parametrize("n_seqs,most", [(2, 3), (0, 3), (2, 0)])
def test_attend_rows_that_no_request_covers_keep_what_they_hold(C, n_seqs, most):
    """Rows before the first request and behind the last one, as in a batch padded to a captured size."""
    hq, hkv, d = 4, 2, 64
    cb = O.analytic_codebook(4)
    g = C.cq_kv_geometry(hq, hkv, d, d, 4, 4, cb, cb, 0.125)
    kc, vc = (torch.from_numpy(_blob(64, hkv * d, 4, np.random.RandomState(i))).cuda() for i in (1, 2))
    q = torch.randn(9, hq, d, device="cuda").to(F16)
    q[:2], q[6:] = math.nan, math.nan  # rows that are not read either
    o = torch.full((9, hq, d), 7.0, dtype=F16, device="cuda")
    cu = _i32([2, 5, 6][:n_seqs + 1]) if most else _i32([2, 2, 2])
    C.cq_kv_tree_attend(g, q, kc, vc, 64, _i32([[0, 1], [2, 3]]), 16, _i32([20, 7][:n_seqs]), cu, None, most, o=o)
    torch.cuda.synchronize()
    C.cq_device_status()
    covered = slice(2, 6) if n_seqs and most else slice(0, 0)
    keep = torch.ones(9, dtype=torch.bool)
    keep[covered] = False
    assert (o[keep.cuda()] == 7).all()
    assert torch.isfinite(o).all() and (o[covered] != 7).any(-1).all()

# ------------------------------------------------------------------------------------------------------- slot writes

@pytest.mark.parametrize("bits", [2, 3, 4, 5])
@pytest.mark.parametrize("dtype", [torch.float32, BF16])
def test_write_slots_of_rows_whose_squares_leave_fp32(C, bits, dtype):
    """Elements of 1e15 to 3e38: the sum of squares, the norm and then the sums of elements pass fp32. Codes are those of
    exact arithmetic all the same, the norm is an infinity of fp16, and ordinary rows beside them keep their bytes."""
    rng = np.random.RandomState(bits)
    sizes = [1.0, 1e15, 3e18, 1e19, 2.0, 1e25, 1e30, 1e36, 0.5, 1e37]
    rows = [rng.randn(256) * s for s in sizes] + [rng.uniform(-3.3e38, 3.3e38, 256), np.full(256, 3e38), np.full(256, -1e20), np.eye(256)[3] * 3e38,
                                                  rng.choice([-1e30, 1e30], 256), np.concatenate([rng.randn(128), rng.randn(128) * 1e22])]
    x = torch.from_numpy(np.array(rows, dtype=np.float32)).cuda().to(dtype)
    assert torch.isfinite(x).all()
    n, cap = len(rows), len(rows) + 2
    cb = O.analytic_codebook(bits)
    g = C.cq_kv_geometry(1, 1, 256, 256, bits, bits, cb, cb, 1.0)
    blobs = [torch.zeros(C.cq_packed_bytes(cap, 256, 128, bits), dtype=torch.uint8, device="cuda") for _ in range(2)]
    C.cq_kv_write_slots(g, *blobs, cap, x, x, _i32(np.arange(n)))
    codes, norms = R.encode(_np(x), bits, cb)
    for blob in blobs:
        gc, gn = R.split_blob(blob.cpu().numpy(), cap, 256, bits)
        np.testing.assert_array_equal(gc[:n], R.pack(codes, R.width_of(bits)))
        np.testing.assert_array_equal(gn[:n].view(np.uint16), norms.view(np.uint16))


@pytest.mark.parametrize("book", [[-0.4, 0.2, 0.9, 0.98], [-1.01, -0.985, 0.95, 0.999], [-0.3, -0.1, 0.1, 0.3]])
def test_write_slots_next_to_large_midpoints(C, book):
    """Coordinates a few units of 2^-24 from midpoints of 0.04 to 0.9975, where fp32's error grows with the coordinate."""
    cb = np.array(book, dtype=np.float32)
    mids = (cb[1:].astype(np.float64) + cb[:-1].astype(np.float64)) / 2
    rng = np.random.RandomState(int(abs(book[0]) * 100))
    H, rows = R.hadamard(), []
    for i in range(600):
        m, k = mids[i % 3] * (1 + (i // 3 - 100) * 2.0 ** -25), rng.randint(128)
        u = rng.randn(128) * np.exp(rng.randn(128))
        u[k] = 0
        u *= math.sqrt(1 - m * m) / np.linalg.norm(u)
        u[k] = m
        rows.append(u @ H * 2.0 ** rng.uniform(-8, 8))
    x = torch.from_numpy(np.array(rows, dtype=np.float32)).cuda()
    g = C.cq_kv_geometry(1, 1, 128, 128, 2, 2, cb, cb, 1.0)
    blobs = [torch.zeros(C.cq_packed_bytes(600, 128, 128, 2), dtype=torch.uint8, device="cuda") for _ in range(2)]
    C.cq_kv_write_slots(g, *blobs, 600, x, x, _i32(np.arange(600)))
    codes, norms = R.encode(_np(x), 2, cb)
    gc, gn = R.split_blob(blobs[0].cpu().numpy(), 600, 128, 2)
    np.testing.assert_array_equal(gc, R.pack(codes, 2))
    np.testing.assert_array_equal(gn.view(np.uint16), norms.view(np.uint16))

# ------------------------------------------------------------------------------------------------------------- plan

TOP = 2 ** 31 - 1


def _plan(C, lens, new, held, table, free, bs, room):
    t = _i32(table)
    out = C.cq_kv_plan(_i32(lens), _i32(new), _i32(held), t, _i32(free), _i32([len(free)]), bs, room)
    torch.cuda.synchronize()
    with pytest.raises(C.CQError):
        C.cq_device_status()
    C.cq_device_status()
    return t.tolist(), {k: v.tolist() for k, v in out.items()}


def test_plan_lengths_whose_sum_leaves_32_bits(C):
    """Four requests of 2^30 new tokens: what fits into the slot map is planned, the rest is dropped and reported."""
    table, out = _plan(C, [0] * 4, [2 ** 30] * 4, [0] * 4, [[-1, -1]] * 4, [3, 2, 1, 0], 2 ** 30, 8)
    assert table == [[0, -1], [1, -1], [2, -1], [3, -1]] and out["held_out"] == [1] * 4 and out["n_free_out"] == [0]
    assert out["cu_new"] == [0, 2 ** 30, TOP, TOP, TOP]
    assert out["slots"] == out["positions"] == list(range(8)) and out["token_seq"] == [0] * 8
    # over more than one chunk of requests
    n = 1100
    table, out = _plan(C, [0] * n, [2 ** 22] * n, [0] * n, [[-1]] * n, list(range(n))[::-1], 2 ** 22, 16)
    assert table == [[i] for i in range(n)] and out["n_free_out"] == [0]
    assert out["cu_new"] == [min(i * 2 ** 22, TOP) for i in range(n + 1)]
    assert out["slots"] == out["positions"] == list(range(16)) and out["token_seq"] == [0] * 16


def test_plan_positions_that_leave_32_bits(C):
    table, out = _plan(C, [TOP - 2, 5], [5, 1], [2, 1], [[0, 1, -1], [1, -1, -1]], [7, 9], 2 ** 30, 7)
    assert table == [[0, 1, 9], [1, -1, -1]] and out["held_out"] == [3, 1] and out["n_free_out"] == [1]
    assert out["positions"] == [TOP - 2, TOP - 1, TOP, -1, -1, 5, -1]
    assert out["slots"] == [TOP - 2, TOP - 1, TOP, -1, -1, 2 ** 30 + 5, -1]
    assert out["token_seq"] == [0, 0, 0, 0, 0, 1, -1] and out["cu_new"] == [0, 5, 6]


def test_plan_missing_blocks_stay_countable(C):
    """A stack that is already below zero by all it can be: the count stays where it is."""
    t = _i32([[-1, -1]])
    out = C.cq_kv_plan(_i32([0]), _i32([20]), _i32([0]), t, _i32([4]), _i32([-(2 ** 31)]), 16, 20)
    torch.cuda.synchronize()
    assert out["n_free_out"].tolist() == [-(2 ** 31)] and t.tolist() == [[-1, -1]] and out["slots"].tolist() == [-1] * 20
    with pytest.raises(C.CQError):
        C.cq_device_status()

# ------------------------------------------------------------------------------------------------- waits that run out

@pytest.mark.parametrize("geom", [(4, 2, 64, 64), (8, 2, 128, 128), (6, 6, 80, 80), (4, 1, 256, 256)])
@pytest.mark.parametrize("n", [1, 7, 40])
def test_attend_waits_that_run_out_end_the_call_with_a_status(C, monkeypatch, geom, n):
    """A wait that nothing ends gives up: every role runs through its tiles without waiting, the kernel ends, the host
    reads CQ_ERR_TIMEOUT, and the next call gives what the one before gave."""
    from hadamard_rotated_codebook_gb300 import _capi
    lib = _capi.load()
    pool = _Pool(C, geom, 4, 700, n, 0.125, seed=n)
    q = pool.q.to(BF16)
    want = pool.run(q)
    with monkeypatch.context() as m:
        m.setattr(lib, "cq_kv_tree_attend", lib.cq_selftest_tree_timeout)
        with pytest.raises(C.CQError, match="0x4749"):
            pool.run(q)
    C.cq_device_status()
    assert torch.equal(pool.run(q), want)
