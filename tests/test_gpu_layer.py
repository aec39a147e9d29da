"""GPU parity of a layer's other serving steps (cq_block_norm, cq_lora_add)
with their 64-bit definitions."""
import math
import sys

import numpy as np
import pytest
import torch

from tests import layer_reference as L

pytestmark = pytest.mark.gpu

F32, F16, BF16, I8 = torch.float32, torch.float16, torch.bfloat16, torch.int8


@pytest.fixture(scope="module")
def C():
    import hadamard_rotated_codebook_gb300 as pkg
    return pkg


@pytest.fixture(autouse=True)
def status(C):
    """No test leaves a mark in the device status word."""
    yield
    C.cq_device_status()


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _name(dtype):
    return str(dtype).replace("torch.", "")


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------------------------------------- block norm

def _norm_inputs(n, d, dtype, res=None, gate=None, weights=True, post=False, seed=0, wide=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(n, d + wide, generator=g, device="cuda") * torch.exp(0.5 * torch.randn(n, 1, generator=g, device="cuda"))
    kw = dict(x=x.to(dtype)[:, :d])
    if res is not None:
        kw["residual"] = (2 * torch.randn(n, d + wide, generator=g, device="cuda")).to(res)[:, :d]
    if gate is not None:
        kw["gate"] = (3 * torch.randn(n, gate + (wide if gate > 1 else 0), generator=g, device="cuda")).to(dtype)[:, :gate]
    if weights:
        kw["weight"] = torch.randn(d, generator=g, device="cuda")
        kw["branch_weight"] = torch.randn(d, generator=g, device="cuda") if post else None
    return kw


def _check_norm(C, kw, **opt):
    before = {k: v.clone() for k, v in kw.items() if v is not None}
    got = C.cq_block_norm(**kw, **opt)
    torch.cuda.synchronize()
    for k, v in before.items():
        assert torch.equal(kw[k].nan_to_num(), v.nan_to_num())
    r, y, er, ey = L.block_norm(_np(kw["x"]), _np(kw.get("residual")), _np(kw.get("weight")), post=opt.get("post_norm", False),
                                wb=_np(kw.get("branch_weight")), gate=_np(kw.get("gate")), act=opt.get("gate_act"),
                                branch=np.float64(np.float32(opt.get("branch_scale", 1.0))), keep=np.float64(np.float32(opt.get("residual_scale", 1.0))),
                                eps=np.float64(np.float32(opt.get("eps", 1e-6))), offset=opt.get("weight_offset", 0.0))
    for name, a, b, e in (("r", got[0], r, er),) + ((("y", got[1], y, ey),) if got[1].dtype != I8 else ()):
        tol = L.rounded(b, e, _name(a.dtype))
        err = np.abs(_np(a) - b)
        assert (err <= tol).all(), f"{name}: worst {np.nanmax(err / tol)}"
    if got[1].dtype == I8:  # the bits of the quantiser over the fp32 result
        opt32 = {k: v for k, v in opt.items() if k != "out_dtype"}
        z = C.cq_block_norm(**kw, **opt32, out_dtype=F32)[1]
        q, s = C.cq_act_quant_int8(z)
        assert torch.equal(got[1], q) and torch.equal(got[2], s)
    return got


@pytest.mark.parametrize("d", [1, 3, 7, 8, 64, 80, 255, 256, 257, 333, 512, 520, 1000, 1024, 1025, 1032, 2048, 4096, 5000, 8192, 8200, 16384])
@pytest.mark.parametrize("post", [False, True])
def test_norm_widths(C, d, post):
    _check_norm(C, _norm_inputs(5, d, F32, F32, None, True, post, seed=d), post_norm=post, weight_offset=1.0)
    _check_norm(C, _norm_inputs(5, d, BF16, BF16, d, True, post, seed=d), post_norm=post, gate_act="sigmoid", out_dtype=I8)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("res", [F32, F16, BF16, None])
@pytest.mark.parametrize("out", [F32, F16, BF16, I8])
def test_norm_types(C, dtype, res, out):
    for d in (96, 1536, 1537):
        _check_norm(C, _norm_inputs(7, d, dtype, res, d, post=True, seed=d), post_norm=True, gate_act="silu", out_dtype=out, branch_scale=0.5,
                    residual_scale=0.7)


@pytest.mark.parametrize("gate,act", [(None, None), (1, None), (1, "sigmoid"), (1, "silu"), (-1, None), (-1, "sigmoid"), (-1, "silu")])
@pytest.mark.parametrize("d", [1, 200, 1000, 2056])
def test_norm_gates(C, gate, act, d):
    _check_norm(C, _norm_inputs(6, d, F16, F32, d if gate == -1 else gate, seed=d), gate_act=act)


@pytest.mark.parametrize("n", [0, 1, 2, 3, 127, 1000, 5001])
def test_norm_token_counts(C, n):
    for d in (64, 1088):
        _check_norm(C, _norm_inputs(n, d, BF16, BF16, d, post=True, seed=n), post_norm=True, gate_act="silu")


def test_norm_without_weights(C):
    for post in (False, True):
        _check_norm(C, _norm_inputs(9, 640, F16, F16, weights=False), post_norm=post, weight_offset=0.25)
    kw = _norm_inputs(9, 640, F16, None, weights=False)  # the bare norm of a first block
    _check_norm(C, kw)
    kw["branch_weight"] = torch.randn(640, device="cuda")  # a scale per channel
    _check_norm(C, kw)


def test_norm_rows_that_are_not_runs(C):
    """Rows off every vector boundary, and rows of a wider tensor, give the same bits."""
    for d in (512, 1096):
        kw = _norm_inputs(6, d, F16, F16, d, post=True, seed=1, wide=3)
        opt = dict(post_norm=True, gate_act="sigmoid")
        want = C.cq_block_norm(**{k: v.contiguous() for k, v in kw.items()}, **opt)
        got = _check_norm(C, kw, **opt)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        wide = torch.zeros(6, d + 5, dtype=F16, device="cuda")
        C.cq_block_norm(**kw, **opt, out=wide[:, 1:d + 1], residual_out=torch.empty_like(want[0]))
        assert torch.equal(wide[:, 1:d + 1], want[1]) and (wide[:, 0] == 0).all() and (wide[:, d + 1:] == 0).all()


def test_norm_rows_do_not_depend_on_each_other(C):
    for d in (320, 2048):
        kw = _norm_inputs(700, d, BF16, F32, d, post=True, seed=3)
        opt = dict(post_norm=True, gate_act="silu")
        want = C.cq_block_norm(**kw, **opt)
        one = C.cq_block_norm(**{k: v[411:412] if v.dim() == 2 else v for k, v in kw.items()}, **opt)
        assert torch.equal(one[0][0], want[0][411]) and torch.equal(one[1][0], want[1][411])


def test_norm_in_place(C):
    for d in (256, 3000):
        kw = _norm_inputs(400, d, BF16, BF16, seed=4)
        want = C.cq_block_norm(**kw)
        got = C.cq_block_norm(**kw, residual_out=kw["residual"], out=kw["x"])
        assert got[0].data_ptr() == kw["residual"].data_ptr() and torch.equal(got[0], want[0]) and torch.equal(kw["x"], want[1])


def test_norm_zeros_and_non_finite_rows_stay_apart(C):
    for d in (128, 2048):
        kw = _norm_inputs(6, d, F32, F32, post=True)
        kw["x"][0], kw["residual"][0] = 0, 0
        kw["x"][1, 3] = math.nan
        kw["residual"][2, 5] = math.inf
        kw["x"][3, 7] = -math.inf
        r, y = C.cq_block_norm(**kw, post_norm=True)
        assert (r[0] == 0).all() and (y[0] == 0).all() and r[1].isnan().all() and y[1].isnan().all()
        assert y[2, 5].isnan() and (y[2, :5] == 0).all() and torch.isfinite(y[4:]).all() and torch.isfinite(r[4:]).all()
        _, q, s = C.cq_block_norm(**kw, post_norm=True, out_dtype=I8)
        want = C.cq_act_quant_int8(y)
        assert torch.equal(q, want[0]) and torch.equal(s, want[1]) and s[0] == 1 and (q[0] == 0).all()


@pytest.mark.parametrize("d", [96, 333, 2048])
def test_norm_codes_of_every_kind_of_row(C, d):
    """Codes and scales are the quantiser's where quotients lie on ties, rows are tiny, huge or zero, or weights are no numbers."""
    g = torch.Generator(device="cuda").manual_seed(d)
    x = torch.randint(-254, 255, (12, d), generator=g, device="cuda").float() / 2
    x[:, 0] = 127.0  # the scale is 1 times the norm's factor: halves lie near ties
    x[1] *= 1e-30
    x[2] *= 1e30
    x[3] *= 2.0 ** -140
    x[4] = 0
    x[5, 1] = 3e38
    for eps in (1e-6, 0.0):
        for weight in (None, torch.ones(d, device="cuda"), torch.randn(d, generator=g, device="cuda") * 1e-38,
                       torch.randn(d, generator=g, device="cuda") * 1e37, torch.full((d,), 2.0, device="cuda").index_fill_(0, _i32([2]).long(), math.nan),
                       torch.full((d,), 2.0, device="cuda").index_fill_(0, _i32([3]).long(), math.inf)):
            y = C.cq_block_norm(x, None, weight, eps=eps)[1]
            _, q, s = C.cq_block_norm(x, None, weight, eps=eps, out_dtype=I8)
            want = C.cq_act_quant_int8(y)
            assert torch.equal(q, want[0]) and torch.equal(s, want[1])


def test_norm_gates_that_are_far_out(C):
    kw = _norm_inputs(1, 8, F32, None, 8, weights=False)
    kw["gate"][0] = torch.tensor([0.0, 100.0, -100.0, 1e4, -1e4, math.inf, -math.inf, 88.5])
    kw["x"][0] = 1.0
    r, _ = C.cq_block_norm(**kw, gate_act="sigmoid")
    want = torch.sigmoid(kw["gate"][0])
    assert torch.isfinite(r).all() and (r[0] - want).abs().max() <= 4 * 2.0 ** -24


def test_norm_refuses_bad_tensors(C):
    x, w = torch.randn(4, 64, device="cuda"), torch.ones(64, device="cuda")
    for kw, kind in ((dict(x=x.t()), ValueError), (dict(x=x[0]), ValueError), (dict(x=x.int()), TypeError),
                     (dict(x=x, residual=x[:3]), ValueError), (dict(x=x, residual=x[:, :32]), ValueError), (dict(x=x, residual=x.cpu()), TypeError),
                     (dict(x=x, weight=w[:63]), ValueError), (dict(x=x, weight=w.half()), ValueError), (dict(x=x, branch_weight=w[None]), ValueError),
                     (dict(x=x, gate=x.half()), ValueError), (dict(x=x, gate=x[:, :2]), ValueError), (dict(x=x, gate_act="silu"), ValueError),
                     (dict(x=x, gate=x, gate_act="tanh"), ValueError), (dict(x=x, out=x.half(), out_dtype=BF16), TypeError),
                     (dict(x=x, out=torch.empty(1, 64, device="cuda").expand(4, 64)), ValueError),
                     (dict(x=x, residual=x.half(), residual_out=x.clone()), TypeError), (dict(x=x, out=x.view(BF16)[:, :64]), ValueError),
                     (dict(x=x, out_dtype=I8, out_scale=w[:3]), ValueError), (dict(x=x, eps=-1.0), C.CQError),
                     (dict(x=torch.randn(2, 16385, device="cuda")), C.CQError)):
        with pytest.raises(kind):
            C.cq_block_norm(**kw)


def test_norm_captured_and_on_another_stream(C):
    kw = _norm_inputs(64, 2048, BF16, BF16, 2048, post=True)
    opt = dict(post_norm=True, gate_act="silu")
    want = C.cq_block_norm(**kw, **opt)
    out, res = torch.empty_like(want[1]), torch.empty_like(want[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        C.cq_block_norm(**kw, **opt, out=out, residual_out=res)
    for _ in range(3):
        out.zero_(), res.zero_()
        g.replay()
        assert torch.equal(out, want[1]) and torch.equal(res, want[0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = C.cq_block_norm(**kw, **opt)
    s.synchronize()
    assert torch.equal(got[1], want[1])


# ---------------------------------------------------------------------------------------------------------- adapters

def _lora_inputs(new, adapters, n_in, outs, rank, w=BF16, x=F32, seed=0, extra=0, ragged=False, n_adapters=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n, m = sum(new) + extra, n_adapters or max(list(adapters) + [0]) + 1
    xv = torch.randn(n, n_in, generator=g, device="cuda")
    kw = dict(x_scale=None, ranks=None)
    if x == I8:
        kw["x_scale"] = torch.rand(n, generator=g, device="cuda") * 0.02
        xv = (xv * 40).clamp(-128, 127).round()
    kw["x"] = xv.to(x)
    kw["a"] = [(torch.randn(m, rank, n_in, generator=g, device="cuda") * n_in ** -0.5).to(w) for _ in outs]
    kw["b"] = [torch.randn(m, o, rank, generator=g, device="cuda").to(w) for o in outs]
    kw["scales"] = torch.randn(m, generator=g, device="cuda")
    if ragged:
        ranks = [(i * 5 + 1) % (rank + 1) for i in range(m)]
        kw["ranks"] = _i32(ranks)
        for a, b in zip(kw["a"], kw["b"]):  # what is not in use may hold anything
            for i, r in enumerate(ranks):
                a[i, r:], b[i, :, r:] = math.nan, math.inf
    kw["ys"] = [torch.randn(n, o, generator=g, device="cuda") for o in outs]
    kw["adapters"], kw["cu_tokens"] = _i32(adapters), _i32(np.concatenate([[0], np.cumsum(new)]))
    return kw


def _check_lora(C, kw, in_place=False):
    want = L.lora([_np(y) for y in kw["ys"]], _np(kw["x"]), [_np(a) for a in kw["a"]], [_np(b) for b in kw["b"]], kw["adapters"].tolist(),
                  kw["cu_tokens"].tolist(), None if kw["scales"] is None else _np(kw["scales"]),
                  None if kw["ranks"] is None else kw["ranks"].tolist(), _np(kw["x_scale"]), kw["x"].dtype == F32)
    last = int(kw["cu_tokens"][-1])
    args = dict(kw)
    if in_place:
        args["ys"] = [y.clone() for y in kw["ys"]]
        got = C.cq_lora_add(**args)
        assert all(a is b for a, b in zip(got, args["ys"]))
    else:
        args["outs"] = [torch.full_like(y, 7.0) for y in kw["ys"]]
        got = C.cq_lora_add(**args)
    torch.cuda.synchronize()
    C.cq_device_status()
    for j, (o, e) in enumerate(want):
        err = np.abs(_np(got[j]) - o)[:last]
        assert (err <= e[:last]).all(), f"matrix {j}: worst {np.nanmax(err / e[:last])}"
        tail = got[j][last:]
        assert torch.equal(tail, kw["ys"][j][last:]) if in_place else (tail == 7.0).all()
    return got


W_X = [(F16, F32), (F16, I8), (F16, F16), (BF16, F32), (BF16, I8), (BF16, BF16)]


@pytest.mark.parametrize("w,x", W_X)
@pytest.mark.parametrize("new", [[1], [1] * 9, [5, 0, 33, 1], [200, 3]])
def test_lora_types(C, w, x, new):
    who = [i % 3 for i in range(len(new))]
    kw = _lora_inputs(new, who, 512, (256, 128), 16, w, x, seed=len(new))
    a = _check_lora(C, kw)
    b = _check_lora(C, kw, True)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("rank", [1, 3, 4, 8, 15, 16, 17, 20, 32, 33, 48, 64, 65, 100, 128, 255, 256])
def test_lora_ranks(C, rank):
    for new in ([1, 1, 1], [70, 2]):
        who = [i % 2 for i in range(len(new))]
        for w, x, outs in ((BF16, F32, (96, 33)), (F16, I8, (96, 33)), (BF16, BF16, (300,)), (F16, F16, (300,))):
            kw = _lora_inputs(new, who, 160, outs, rank, w, x, seed=rank)
            a, b = _check_lora(C, kw), _check_lora(C, kw, True)
            assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("n_in,out", [(1, 1), (7, 5), (8, 4), (31, 33), (32, 32), (40, 64), (1000, 777), (1001, 100), (2048, 36), (520, 2052), (6000, 4100), (136, 128),
                                        (264, 129), (72, 1000)])
@pytest.mark.parametrize("x", [F32, I8, F16])
def test_lora_sizes(C, n_in, out, x):
    _check_lora(C, _lora_inputs([1, 2, 1], [0, 1, 0], n_in, (out,), 8, F16, x, seed=n_in))
    _check_lora(C, _lora_inputs([40, 0, 90], [0, 1, 2], n_in, (out,), 20, F16, x, seed=out))


def test_lora_long_prompts(C):
    for w, x, rank in ((BF16, BF16, 64), (BF16, I8, 16), (F16, F32, 32)):
        _check_lora(C, _lora_inputs([1500, 1, 700, 64], [1, 0, 2, 1], 768, (512,), rank, w, x, seed=rank))


def test_lora_many_requests(C):
    """More requests than are looked at in one go, some of them empty, some without an adapter."""
    rng = np.random.RandomState(0)
    new = rng.randint(0, 3, 500).tolist()
    who = rng.randint(-1, 40, 500).tolist()
    kw = _lora_inputs(new, who, 64, (40,), 8, F16, F32, n_adapters=40)
    _check_lora(C, kw)
    _check_lora(C, kw, True)
    new[260] = 400
    _check_lora(C, _lora_inputs(new, who, 64, (40,), 8, F16, F16, n_adapters=40), True)


@pytest.mark.parametrize("new", [[3, 1, 1, 2], [100, 30, 1, 2]])
def test_lora_ranks_in_use(C, new):
    """Rows and columns past an adapter's rank do not count, whatever they hold; a rank of zero adds nothing."""
    for rank, x in ((8, F32), (19, I8), (64, BF16), (130, F32)):
        kw = _lora_inputs(new, [0, 1, 2, 3], 100, (70,), rank, BF16, x, seed=rank, ragged=True)
        kw["ranks"][3] = 0
        _check_lora(C, kw)
        _check_lora(C, kw, True)


def test_lora_rows_behind_the_last_request_stay(C):
    kw = _lora_inputs([2, 3], [0, 1], 64, (64,), 8, extra=9)
    _check_lora(C, kw)
    _check_lora(C, kw, True)
    kw["cu_tokens"] += 4  # rows before the first request, too
    y = kw["ys"][0].clone()
    C.cq_lora_add(**kw)
    assert torch.equal(kw["ys"][0][:4], y[:4]) and torch.equal(kw["ys"][0][9:], y[9:]) and not torch.equal(kw["ys"][0][4:9], y[4:9])


def test_lora_values_of_every_size(C):
    """The terms of the second product hold large and small values side by side: tokens of any scale, ranks of any scale."""
    for w in (F16, BF16):
        for new in ([2, 3], [70, 40]):
            for rank in (16, 40, 130):
                kw = _lora_inputs(new, [0, 1], 128, (140,), rank, w, F32, seed=rank)
                kw["x"] *= torch.exp2(torch.linspace(-60, 60, sum(new), device="cuda"))[:, None]
                kw["a"][0] *= torch.exp2(-(torch.arange(rank, device="cuda") % 9).float())[None, :, None].to(w)
                _check_lora(C, kw)


def test_lora_without_anything(C):
    kw = _lora_inputs([2, 3], [-1, -1], 64, (64,), 8, n_adapters=1)
    got = _check_lora(C, kw)
    assert torch.equal(got[0], kw["ys"][0])
    empty = dict(kw, a=[kw["a"][0][:0]], b=[kw["b"][0][:0]], scales=None)  # a server that has loaded no adapter yet
    assert torch.equal(C.cq_lora_add(**empty, outs=[torch.empty_like(kw["ys"][0])])[0], kw["ys"][0])
    kw["scales"] = None
    none = dict(kw, x=kw["x"][:0], ys=[kw["ys"][0][:0]], cu_tokens=_i32([0]), adapters=_i32([]))
    C.cq_lora_add(**none)
    C.cq_device_status()


def test_lora_of_many_tokens_without_anything(C):
    """Prompts of a server that has loaded no adapter, and of requests that have none."""
    kw = _lora_inputs([200, 90], [-1, -1], 64, (160,), 8, n_adapters=1)
    none = dict(kw, a=[kw["a"][0][:0]], b=[kw["b"][0][:0]], scales=None)
    for k in (kw, none):
        outs = [torch.full_like(kw["ys"][0], 7.0)]
        assert torch.equal(C.cq_lora_add(**dict(k, outs=outs))[0], kw["ys"][0])
    C.cq_device_status()


def test_lora_rows_on_eight_bytes(C):
    """int8 rows that tensor copies do not reach, and a single token with rows of any stride."""
    for n_in in (1000, 1016, 1032):
        _check_lora(C, _lora_inputs([300, 40], [0, 1], n_in, (160,), 16, BF16, I8, seed=n_in))
    kw = _lora_inputs([1], [0], 33, (160,), 8, extra=6)
    wide = torch.randn(7, 163, device="cuda")
    kw["ys"] = [wide[:, :160][:1]]
    kw["x"] = kw["x"][:1]
    _check_lora(C, kw)


def test_lora_shared_rows(C):
    """One row of x and y for every token (strides of zero)."""
    kw = _lora_inputs([1, 90], [0, 1], 64, (160,), 8)
    kw["x"] = kw["x"][:1].expand(91, 64)
    kw["ys"] = [kw["ys"][0][:1].expand(91, 160)]
    _check_lora(C, kw)


def test_lora_strides(C):
    """Rows of wider tensors, on and off vector boundaries."""
    kw = _lora_inputs([3, 40], [0, 1], 256, (128, 64), 16)
    want = L.lora([_np(y) for y in kw["ys"]], _np(kw["x"]), [_np(a) for a in kw["a"]], [_np(b) for b in kw["b"]], [0, 1], [0, 3, 43],
                  _np(kw["scales"]), terms=True)
    for off in (4, 1):
        wide = torch.zeros(43, 256 + 8, device="cuda")
        wide[:, off:off + 256] = kw["x"]
        packed = torch.full((43, 128 + 64 + 8), 3.0, device="cuda")
        parts = [packed[:, off:off + 128], packed[:, off + 128:off + 192]]
        for p, y in zip(parts, kw["ys"]):
            p.copy_(y)
        got = C.cq_lora_add(**dict(kw, x=wide[:, off:off + 256], ys=parts))
        for p, (o, e) in zip(got, want):
            assert (np.abs(_np(p) - o) <= e).all()
        assert (packed[:, :off] == 3.0).all() and (packed[:, off + 192:] == 3.0).all()


def test_lora_non_finite_tokens_stay_apart(C):
    for x in (F32, BF16):
        for new in ([3, 2], [60, 50]):
            kw = _lora_inputs(new, [0, 1], 96, (48,), 20, BF16, x)
            want = C.cq_lora_add(**dict(kw, outs=[torch.empty_like(kw["ys"][0])]))[0]
            kw["x"][1, 5], kw["x"][2, 9] = math.nan, math.inf
            got = C.cq_lora_add(**dict(kw, outs=[torch.empty_like(kw["ys"][0])]))[0]
            keep = torch.ones(sum(new), dtype=torch.bool, device="cuda")
            keep[1:3] = False
            assert got[1].isnan().all() and not got[2].isfinite().any() and torch.equal(got[keep], want[keep])


def test_lora_reports_what_does_not_fit(C):
    kw = _lora_inputs([2, 2, 2], [0, 1, 2], 64, (64,), 8)
    want = C.cq_lora_add(**dict(kw, outs=[torch.empty_like(kw["ys"][0])]))[0]
    for adapters, cu, ranks, same in (([0, 3, 2], [0, 2, 4, 6], None, slice(2, 4)), ([0, -2, 2], [0, 2, 4, 6], None, slice(2, 4)),
                                      ([0, 1, 2], [0, 2, 4, 7], None, slice(4, 6)), ([0, 1, 2], [-1, 2, 4, 6], None, slice(0, 2)),
                                      ([0, 1, 2], [0, 2, 4, 6], [8, 9, 8], slice(2, 4)), ([0, 1, 2], [0, 2, 4, 6], [8, 8, -1], slice(4, 6))):
        ys = [kw["ys"][0].clone()]
        C.cq_lora_add(**dict(kw, ys=ys, adapters=_i32(adapters), cu_tokens=_i32(cu), ranks=None if ranks is None else _i32(ranks)))
        with pytest.raises(C.CQError):
            C.cq_device_status()
        C.cq_device_status()
        left = torch.ones(6, dtype=torch.bool, device="cuda")
        left[same] = False
        assert torch.equal(ys[0][same], kw["ys"][0][same]) and torch.equal(ys[0][left], want[left])


def test_lora_refuses_bad_tensors(C):
    kw = _lora_inputs([2, 2], [0, 1], 64, (32, 16), 8)
    a, b, ys = kw["a"], kw["b"], kw["ys"]
    for change, kind in ((dict(ys=[]), ValueError), (dict(ys=ys[:1]), ValueError), (dict(ys=ys * 5, a=a * 5, b=b * 5), ValueError),
                         (dict(a=[t.float() for t in a]), TypeError), (dict(a=[a[0][0], a[1]]), ValueError), (dict(b=[b[1], b[0]]), ValueError),
                         (dict(a=[a[0], a[1].half()]), ValueError), (dict(x=kw["x"].half()), TypeError), (dict(x=kw["x"].to(I8)), ValueError),
                         (dict(x=kw["x"][:, :63]), ValueError), (dict(ys=[y.half() for y in ys]), TypeError), (dict(ys=[y[:3] for y in ys]), ValueError),
                         (dict(adapters=kw["adapters"].long()), TypeError), (dict(cu_tokens=kw["cu_tokens"][:2]), ValueError),
                         (dict(scales=kw["scales"][:1]), ValueError), (dict(ranks=kw["scales"]), TypeError), (dict(x=kw["x"].cpu()), TypeError),
                         (dict(outs=[y.t().contiguous().t() for y in ys]), ValueError)):
        with pytest.raises(kind):
            C.cq_lora_add(**dict(kw, **change))


def test_lora_is_the_same_every_time(C):
    for new, rank in (([1] * 20, 16), ([300, 5, 1], 64)):
        kw = _lora_inputs(new, [i % 4 for i in range(len(new))], 4096, (1024,), rank, BF16, I8, n_adapters=4)
        outs = [torch.empty_like(kw["ys"][0])]
        want = C.cq_lora_add(**dict(kw, outs=outs))[0].clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            C.cq_lora_add(**dict(kw, outs=outs))
        for _ in range(5):
            outs[0].zero_()
            g.replay()
            assert torch.equal(outs[0], want)
        # a replay serves other requests: lengths and adapters are read on the device
        kw["adapters"].copy_(_i32([(i + 1) % 4 for i in range(len(new))]))
        g.replay()
        ref = C.cq_lora_add(**dict(kw, outs=[torch.empty_like(want)]))[0]
        assert torch.equal(outs[0], ref) and not torch.equal(ref, want)


# Which kernels a call takes goes by its tokens, ranks and widths. What stands above is taken once more with so many rows that no
# request covers that the kernels of many tokens run.

def _rows_for_many(new, n_in, outs, rank):
    return 13_000_000 // (-(-rank // 16) * (n_in + 3 * sum(outs))) + 33 * len(new)


@pytest.fixture
def many(monkeypatch):
    make = _lora_inputs

    def wide(new, adapters, n_in, outs, rank, *args, extra=0, **kw):
        return make(new, adapters, n_in, outs, rank, *args, extra=extra + _rows_for_many(new, n_in, outs, rank), **kw)

    monkeypatch.setattr(sys.modules[__name__], "_lora_inputs", wide)


def _both_ways(C, kw, n):
    """Into outputs of their own and in place: the same bits (of the requests' rows)."""
    a, b = _check_lora(C, kw), _check_lora(C, kw, True)
    assert all(torch.equal(p[:n], q[:n]) for p, q in zip(a, b))


@pytest.mark.parametrize("w,x", W_X)
@pytest.mark.parametrize("new", [[1], [5, 0, 33, 1], [200, 3], [64, 0, 128, 65, 63]])
def test_lora_of_many_types(C, many, w, x, new):
    kw = _lora_inputs(new, [i % 3 for i in range(len(new))], 512, (256, 128), 16, w, x, seed=len(new))
    _both_ways(C, kw, sum(new))


@pytest.mark.parametrize("rank", [1, 8, 15, 16, 17, 20, 32, 33, 48, 64, 65, 100, 128, 255, 256])
def test_lora_of_many_ranks(C, many, rank):
    for new in ([1, 1, 1], [70, 2]):
        for w, x, outs in ((BF16, F32, (96, 33)), (F16, I8, (96, 33)), (BF16, BF16, (300,)), (F16, F16, (300,))):
            _both_ways(C, _lora_inputs(new, [i % 2 for i in range(len(new))], 160, outs, rank, w, x, seed=rank), sum(new))


@pytest.mark.parametrize("n_in,out", [(1, 1), (7, 5), (8, 4), (31, 33), (32, 32), (40, 64), (1000, 777), (1001, 100), (2048, 36), (520, 2052), (6000, 4100), (136, 128),
                                        (264, 129), (72, 1000)])
@pytest.mark.parametrize("x", [F32, I8, F16])
def test_lora_of_many_sizes(C, many, n_in, out, x):
    test_lora_sizes(C, n_in, out, x)


def test_lora_of_many_long_prompts(C, many):
    test_lora_long_prompts(C)
    test_lora_many_requests(C)
    test_lora_rows_on_eight_bytes(C)


@pytest.mark.parametrize("new", [[3, 1, 1, 2], [100, 30, 1, 2]])
def test_lora_of_many_ranks_in_use(C, many, new):
    test_lora_ranks_in_use(C, new)


def test_lora_of_many_values_of_every_size(C, many):
    for w in (F16, BF16):
        for rank in (16, 40, 130):
            kw = _lora_inputs([70, 40], [0, 1], 128, (140,), rank, w, F32, seed=rank)
            kw["x"][:110] *= torch.exp2(torch.linspace(-60, 60, 110, device="cuda"))[:, None]
            kw["a"][0] *= torch.exp2(-(torch.arange(rank, device="cuda") % 9).float())[None, :, None].to(w)
            _check_lora(C, kw)


def test_lora_of_many_without_adapters(C, many):
    kw = _lora_inputs([200, 90], [-1, -1], 64, (160,), 8, n_adapters=1)
    none = dict(kw, a=[kw["a"][0][:0]], b=[kw["b"][0][:0]], scales=None)
    for k in (kw, none):
        outs = [torch.full_like(kw["ys"][0], 7.0)]
        C.cq_lora_add(**dict(k, outs=outs))
        assert torch.equal(outs[0][:290], kw["ys"][0][:290]) and (outs[0][290:] == 7.0).all()
    C.cq_device_status()


def test_lora_of_many_strides(C, many):
    """Rows of wider tensors, on and off vector boundaries; one row of x and y for every token."""
    for x in (F32, BF16):
        kw = _lora_inputs([3, 70], [0, 1], 256, (128, 64), 16, BF16, x)
        n = kw["x"].shape[0]
        cu = [0, 3, 73]
        args = [_np(a) for a in kw["a"]], [_np(b) for b in kw["b"]], [0, 1], cu, _np(kw["scales"])
        want = L.lora([_np(y) for y in kw["ys"]], _np(kw["x"]), *args, terms=x == F32)
        for off in (8, 4, 1):
            wide = torch.zeros(n, 256 + 8, device="cuda", dtype=x)
            wide[:, off:off + 256] = kw["x"]
            packed = torch.full((n, 128 + 64 + 8), 3.0, device="cuda")
            parts = [packed[:, off:off + 128], packed[:, off + 128:off + 192]]
            for p, y in zip(parts, kw["ys"]):
                p.copy_(y)
            got = C.cq_lora_add(**dict(kw, x=wide[:, off:off + 256], ys=parts))
            for p, (o, e) in zip(got, want):
                assert (np.abs(_np(p) - o) <= e).all()
            assert (packed[:, :off] == 3.0).all() and (packed[:, off + 192:] == 3.0).all()
        kw["x"] = kw["x"][:1].expand(n, 256)
        kw["ys"] = [y[:1].expand(n, y.shape[1]) for y in kw["ys"]]
        _check_lora(C, kw)


def test_lora_of_many_non_finite_tokens_stay_apart(C, many):
    for x in (F32, BF16):
        kw = _lora_inputs([60, 50], [0, 1], 96, (48,), 20, BF16, x)
        want = C.cq_lora_add(**dict(kw, outs=[torch.zeros_like(kw["ys"][0])]))[0]
        kw["x"][1, 5], kw["x"][2, 9] = math.nan, math.inf
        kw["x"][110:] = math.nan  # rows that no request covers
        got = C.cq_lora_add(**dict(kw, outs=[torch.zeros_like(kw["ys"][0])]))[0]
        keep = torch.ones(len(got), dtype=torch.bool, device="cuda")
        keep[1:3] = False
        assert got[1].isnan().all() and not got[2].isfinite().any() and torch.equal(got[keep], want[keep])


def test_lora_of_many_is_the_same_every_time(C):
    new = [600, 5, 1]
    kw = _lora_inputs(new, [0, 1, 2], 4096, (1024,), 64, BF16, I8, n_adapters=4)
    outs = [torch.empty_like(kw["ys"][0])]
    want = C.cq_lora_add(**dict(kw, outs=outs))[0].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        C.cq_lora_add(**dict(kw, outs=outs))
    for _ in range(5):
        outs[0].zero_()
        g.replay()
        assert torch.equal(outs[0], want)
    kw["adapters"].copy_(_i32([3, 0, 1]))
    kw["cu_tokens"].copy_(_i32([0, 70, 71, 606]))
    g.replay()
    ref = C.cq_lora_add(**dict(kw, outs=[torch.empty_like(want)]))[0]
    assert torch.equal(outs[0], ref) and not torch.equal(ref, want)


def test_lora_kernels_agree_over_the_whole_range(C):
    """The same requests in calls of either kind."""
    for x, rank in ((I8, 16), (F32, 40), (BF16, 200)):
        kw = _lora_inputs([90, 0, 33, 1], [0, 1, 2, -1], 512, (260, 64), rank, BF16, x, seed=rank)
        got = _check_lora(C, kw)
        more = _rows_for_many([90, 0, 33, 1], 512, (260, 64), rank)

        def pad(t):
            return torch.cat([t, torch.ones(more, *t.shape[1:], device="cuda").to(t.dtype)])

        wide = dict(kw, x=pad(kw["x"]), ys=[pad(y) for y in kw["ys"]], x_scale=None if kw["x_scale"] is None else pad(kw["x_scale"]))
        both = _check_lora(C, wide)
        assert not torch.equal(both[0][:124], got[0]) or x == I8  # other orders of the sums


@pytest.mark.parametrize("new,rank", [([1] * 20, 16), ([1200, 0, 5], 64)])
def test_lora_on_two_streams_at_once(C, new, rank):
    """Calls of different inputs side by side, each with a workspace of its own."""
    kws = [_lora_inputs(new, [i % 3 for i in range(len(new))], 1024, (1024, 256), rank, BF16, BF16, seed=s, n_adapters=3) for s in range(2)]
    want = [C.cq_lora_add(**dict(kw, outs=[torch.empty_like(y) for y in kw["ys"]])) for kw in kws]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in kws]
    outs = [[[torch.zeros_like(y) for y in kw["ys"]] for _ in range(8)] for kw in kws]
    torch.cuda.synchronize()
    for i in range(8):
        for kw, s, o in zip(kws, streams, outs):
            with torch.cuda.stream(s):
                C.cq_lora_add(**dict(kw, outs=o[i]))
    torch.cuda.synchronize()
    C.cq_device_status()
    for w, o in zip(want, outs):
        assert all(torch.equal(a, b) for got in o for a, b in zip(got, w))
