"""GPU parity of cq_kv_window_attend with its 64-bit definition."""
import numpy as np
import pytest
import torch

import oracle as O
from tests import layer_reference as L
from tests import paged_reference as R

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def C():
    import hadamard_rotated_codebook_gb300 as pkg
    return pkg


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _np(t):
    return t.detach().double().cpu().numpy()


def _poison(blob, cap, width, bits, rows):
    """The norms of rows that nobody may look at become no numbers."""
    if len(rows):
        codes = cap * -(-width // 128) * 16 * R.width_of(bits)
        blob[codes:].view(F16).view(cap, -1)[torch.as_tensor(rows, device="cuda").long()] = float("nan")


class Case:
    """Requests of ctx[s] tokens with nodes[s] new ones, a tree's or one after the other; blocks wholly between sinks and window are
    not in the table, and rows that no token attends hold no numbers."""

    def __init__(self, C, ctx, nodes, window, sinks, geom=(8, 4, 64, 64), bits=(2, 2), bs=16, tree=False, dtype=BF16, seed=0, amp=1.5):
        rng = np.random.RandomState(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        hq, hkv, dk, dv = self.dims = geom
        self.C, self.ctx, self.nodes, self.window, self.sinks, self.bs, self.bits = C, ctx, nodes, window, sinks, bs, bits
        self.cu = np.concatenate([[0], np.cumsum(nodes)])
        total, most = int(self.cu[-1]), max(nodes)
        pages = [-(-(l + n) // bs) for l, n in zip(ctx, nodes)]
        keep = [[b * bs < sinks or (b + 1) * bs > l - window + 1 for b in range(p)] for l, p in zip(ctx, pages)]
        blocks = sum(map(sum, keep)) + 1
        order, at = rng.permutation(blocks), 0
        self.table = np.full((len(ctx), max(1, max(pages))), -1, dtype=np.int64)
        for s, k in enumerate(keep):
            for b in np.flatnonzero(k):
                self.table[s, b] = order[at]
                at += 1
        self.cap = blocks * bs
        words = -(-max(most, 1) // 32)
        see = np.zeros((total, words * 32), dtype=bool)
        self.pos = np.zeros(total, dtype=np.int64)
        for s, n in enumerate(nodes):
            for i in range(n):
                parent = (rng.randint(max(-1, i - 4), i) if i else -1) if tree else i - 1
                a = self.cu[s]
                self.pos[a + i] = self.pos[a + parent] + 1 if parent >= 0 else ctx[s]
                if parent >= 0:
                    see[a + i] = see[a + parent]
                see[a + i, i] = True
        self.mask = _i32(np.packbits(see, axis=1, bitorder="little").view(np.int32)) if tree else None
        self.positions = _i32(self.pos) if tree else None
        # who attends what, from the definition
        self.rows, self.sees, used = [], [], np.zeros(self.cap, dtype=bool)
        for s, (l, n) in enumerate(zip(ctx, nodes)):
            t = np.arange(l + n)
            t = t[(t < sinks) | (t > l - window)]  # positions that any token may attend
            a = self.cu[s]
            where = np.where(t < l, t, self.pos[a + np.clip(t - l, 0, max(n - 1, 0))] if n else t)
            vis = np.ones((n, len(t)), dtype=bool)
            for i in range(n):
                vis[i] = np.where(t < l, True, see[a + i, np.clip(t - l, 0, n - 1)])
                vis[i] &= (where < sinks) | (self.pos[a + i] - where < window)
            rows = self.table[s, t // bs] * bs + t % bs if len(t) else t
            self.rows.append(rows)
            self.sees.append(vis)
            if n:
                used[rows[vis.any(0)]] = True
        kb, vb = bits
        self.cb = O.analytic_codebook(kb), O.analytic_codebook(vb)
        self.k, self.v = (C.cq_encode(torch.randn(self.cap, hkv * d, generator=g, device="cuda"), b, c) for d, b, c in
                          ((dk, kb, self.cb[0]), (dv, vb, self.cb[1])))
        self.clean = self.k.cpu().numpy(), self.v.cpu().numpy()
        for blob, d, b in ((self.k, dk, kb), (self.v, dv, vb)):
            _poison(blob, self.cap, hkv * d, b, np.flatnonzero(~used))
        q = torch.randn(total, hq, dk, generator=g, device="cuda")
        self.q = (amp * q / q.pow(2).mean(-1, keepdim=True).sqrt()).to(dtype)
        self.scale = float(np.float32(dk ** -0.5))
        self.geom = C.cq_kv_geometry(hq, hkv, dk, dv, kb, vb, *self.cb, self.scale)
        self.most = max(most, 1)

    def args(self):
        return (self.geom, self.q, self.k, self.v, self.cap, _i32(self.table), self.bs, _i32(self.ctx), _i32(self.cu), self.mask, self.most)

    def run(self, **kw):
        return self.C.cq_kv_window_attend(*self.args(), self.window, self.sinks, positions=self.positions, **kw)

    def check(self):
        got = self.run()
        torch.cuda.synchronize()
        self.C.cq_device_status()
        o, bound = L.attend_rows(_np(self.q), *self.clean, self.cap, self.rows, self.sees, self.cu, self.dims, *self.bits, *self.cb, self.scale)
        name = str(got.dtype).replace("torch.", "")
        tol = bound + R.HALF_STEP[name] * (np.abs(o) + bound) + R.TINY[name]
        err = np.abs(_np(got) - o)
        assert (err <= tol).all(), f"worst {np.nanmax(err / tol)}, {np.isnan(err).sum()} no numbers"
        return got


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 3), (5, 0), (100, 4), (127, 1), (128, 0), (129, 130), (300, 64), (10 ** 9, 0), (2 ** 31 - 1, 5),
                                          (3, 2 ** 31 - 1)])
@pytest.mark.parametrize("nodes", [[1, 1, 1, 1, 1], [5, 0, 3, 1, 7], [40, 33, 1, 0, 17]])
def test_windows(C, window, sinks, nodes):
    for tree in (False, True):
        Case(C, [500, 0, 129, 3, 700], nodes, window, sinks, tree=tree, seed=window % 97 + sinks % 89).check()


@pytest.mark.parametrize("geom", [(12, 2, 48, 64), (32, 8, 128, 128), (16, 16, 96, 96), (8, 1, 256, 256), (10, 5, 80, 80), (16, 2, 128, 64), (3, 3, 40, 24)])
@pytest.mark.parametrize("n", [1, 9, 30])
def test_window_geometries(C, geom, n):
    for dtype, bits in ((F16, (4, 3)), (BF16, (2, 5))):
        Case(C, [333, 60], [n, n], 70, 5, geom, bits, 16, n == 9, dtype, seed=n).check()


@pytest.mark.parametrize("bits", [(2, 2), (3, 4), (4, 4), (5, 3)])
@pytest.mark.parametrize("bs", [1, 16, 48, 256])
def test_window_blocks_and_bits(C, bits, bs):
    Case(C, [1000, 257, 31], [1, 12, 33], 200, 20, (8, 4, 64, 64), bits, bs, True, BF16, seed=bs).check()


@pytest.mark.parametrize("n", [200, 256])
@pytest.mark.parametrize("window,sinks", [(1, 0), (50, 0), (128, 7), (255, 300), (256, 0), (600, 3)])
def test_window_prompt_chunks(C, n, window, sinks):
    """Chunks longer than the window: their own first tokens fall out of it, too."""
    for ctx in ([0, 40], [900, 130]):
        Case(C, ctx, [n, 77], window, sinks, (4, 2, 64, 64), (2, 2), 64, dtype=BF16, seed=n + window).check()


@pytest.mark.parametrize("window,sinks", [(3, 0), (10, 2), (40, 0)])
def test_window_within_trees(C, window, sinks):
    """Trees deeper than the window, of up to 256 tokens."""
    Case(C, [20, 300], [256, 100], window, sinks, (4, 2, 64, 64), (4, 4), 16, True, F16, seed=window).check()


def test_window_long_context(C):
    """More than one chunk of 128 tiles, and a context that the window cuts to one."""
    Case(C, [20000], [3], 18000, 100, (4, 2, 64, 64), (2, 2), 64, True, BF16).check()
    Case(C, [131071, 70000], [1, 2], 300, 4, (4, 2, 64, 64), (2, 2), 64, False, F16).check()


def test_window_that_holds_everything_is_the_tree_attention(C):
    for nodes, tree in (([1, 1, 1], False), ([9, 0, 30], True), ([70, 256, 3], False), ([64, 40, 1], True)):
        for dtype in (F16, BF16):
            c = Case(C, [700, 33, 4000], nodes, 2 ** 31 - 1, 0, tree=tree, dtype=dtype)
            o = torch.zeros(c.q.shape, dtype=dtype, device="cuda")
            want = C.cq_kv_tree_attend(*c.args(), o=o)
            assert torch.equal(c.run(o=torch.zeros_like(o)), want)


def test_window_positions_beyond_the_table_of_a_short_one(C):
    """Positions far past 2^30: only the blocks of the sinks and the window are looked up."""
    bs, cap = 1 << 28, 64
    g = torch.Generator(device="cuda").manual_seed(0)
    cb = O.analytic_codebook(2)
    k, v = (C.cq_encode(torch.randn(cap, 128, generator=g, device="cuda"), 2, cb) for _ in range(2))
    table = np.full((1, 8), -1)
    table[0, 0] = table[0, 7] = 0
    geom = C.cq_kv_geometry(4, 2, 64, 64, 2, 2, cb, cb, 0.125)
    q = torch.randn(3, 4, 64, generator=g, device="cuda").to(F16)
    ctx = 7 * bs + 40
    got = C.cq_kv_window_attend(geom, q, k, v, cap, _i32(table), bs, _i32([ctx]), _i32([0, 3]), None, 3, 20, 4)
    C.cq_device_status()
    rows = np.concatenate([np.arange(4), np.arange(21, 43)])
    place = np.concatenate([np.arange(4), 7 * bs + np.arange(21, 43)])
    see = np.array([[(t < 4) | ((t <= ctx + i) & (ctx + i - t < 20)) for t in place] for i in range(3)])
    o, bound = L.attend_rows(_np(q), k.cpu().numpy(), v.cpu().numpy(), cap, [rows], [see], [0, 3], (4, 2, 64, 64), 2, 2, cb, cb, 0.125)
    assert (np.abs(_np(got) - o) <= bound + 2.0 ** -11 * (np.abs(o) + bound) + 2.0 ** -25).all()


def test_window_reports_what_does_not_fit(C):
    c = Case(C, [100, 50], [3, 2], 30, 2, tree=True)
    want = c.run()
    good = c.positions.clone()
    for at, x in ((1, 99), (2, 100 + 256), (4, -5)):  # before the context's end, past any depth
        c.positions = good.clone()
        c.positions[at] = x
        got = c.run()
        with pytest.raises(C.CQError):
            C.cq_device_status()
        C.cq_device_status()
        other = slice(3, 5) if at < 3 else slice(0, 3)
        assert torch.equal(got[other], want[other])
    c.positions = good
    for ctx in ([2 ** 31 - 1, 50], [2 ** 30, 50], [-7, 50]):  # contexts past the table, or below zero
        c.ctx = ctx
        got = c.run()
        with pytest.raises(C.CQError):
            C.cq_device_status()
        assert torch.equal(got[3:], want[3:])


def test_window_missing_block_inside_is_reported(C):
    c = Case(C, [100], [2], 30, 2, bs=16)
    c.table[0, 5] = -1
    c.run()
    with pytest.raises(C.CQError):
        C.cq_device_status()
    C.cq_device_status()


def test_window_captured(C):
    """A graph serves other lengths: the window moves on with the context."""
    c = Case(C, [300, 200], [4, 3], 64, 4, tree=False)
    ctx, o = _i32(c.ctx), torch.zeros_like(c.run())
    cu, table = _i32(c.cu), _i32(np.arange(2 * 40).reshape(2, 40) % (c.cap // c.bs))
    k = C.cq_encode(torch.randn(c.cap, 256, device="cuda"), 2, c.cb[0])

    def call(out):
        return C.cq_kv_window_attend(c.geom, c.q, k, k, c.cap, table, c.bs, ctx, cu, None, c.most, c.window, c.sinks, o=out)

    call(o)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(o)
    for l in ([300, 200], [0, 1], [500, 63], [64, 400]):
        ctx.copy_(_i32(l))
        o.zero_()
        g.replay()
        assert torch.equal(o, call(torch.zeros_like(o)))
    C.cq_device_status()


def test_window_refuses(C):
    c = Case(C, [20], [2], 8, 1)
    for kw in (dict(window=0), dict(window=-3), dict(sinks=-1)):
        with pytest.raises(C.CQError):
            C.cq_kv_window_attend(*c.args(), **{**dict(window=8, sinks=0), **kw})
    for kw in (dict(window=2 ** 31), dict(sinks=2 ** 32 + 1), dict(positions=_i32([20]))):
        with pytest.raises(ValueError):
            C.cq_kv_window_attend(*c.args(), **{**dict(window=8, sinks=0), **kw})
    with pytest.raises(TypeError):
        C.cq_kv_window_attend(*c.args(), 8, 0, positions=torch.zeros(2, device="cuda"))


@pytest.mark.parametrize("geom", [(8, 2, 64, 64), (32, 8, 128, 128), (16, 1, 128, 128), (6, 6, 48, 64), (8, 1, 256, 256), (14, 7, 40, 40)])
@pytest.mark.parametrize("window,sinks,ctx", [(20, 0, 0), (33, 100, 10), (64, 3, 500), (300, 500, 200), (40, 30, 25), (257, 1, 1000)])
def test_window_column_tiles_have_windows_of_their_own(C, geom, window, sinks, ctx):
    """Chunks over many column tiles: windows that begin before, within and behind the chunk, sinks that reach into it."""
    Case(C, [ctx, 7, 0], [150, 256, 31], window, sinks, geom, (2, 2), 32, dtype=BF16, seed=window).check()


def test_window_on_two_streams_at_once(C):
    cases = [Case(C, [700, 90, 3], [1, 30, 200], 64, 4, seed=1), Case(C, [300, 2000], [4, 1], 500, 0, bits=(4, 3), seed=2)]
    want = [c.run() for c in cases]
    args = [(c.args(), torch.cuda.Stream(), [torch.zeros_like(w) for _ in range(8)]) for c, w in zip(cases, want)]
    torch.cuda.synchronize()
    for i in range(8):
        for c, (a, s, o) in zip(cases, args):
            with torch.cuda.stream(s):
                C.cq_kv_window_attend(*a, c.window, c.sinks, o=o[i])
    torch.cuda.synchronize()
    C.cq_device_status()
    for w, (_, _, o) in zip(want, args):
        assert all(torch.equal(x, w) for x in o)
