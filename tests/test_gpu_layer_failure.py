"""Waits of a layer's other serving steps that run out: the call ends with a status, and the next one works as ever."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

F32, F16, BF16, I8 = torch.float32, torch.float16, torch.bfloat16, torch.int8


@pytest.fixture(scope="module")
def C():
    import hadamard_rotated_codebook_gb300 as pkg
    return pkg


@pytest.fixture(scope="module")
def lib():
    from hadamard_rotated_codebook_gb300 import _capi
    return _capi.load()


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("w,x", [(BF16, BF16), (F16, F16), (BF16, I8), (F16, I8), (BF16, F32)])
@pytest.mark.parametrize("rank,out", [(16, 4096), (24, 4100), (64, 4096), (130, 4099)])
def test_adapters_whose_waits_run_out(C, lib, monkeypatch, w, x, rank, out):
    """Whole and partial pieces, outputs by tensor copies (rows on 16 bytes) and by the threads, ranks in one run and in several."""
    g = torch.Generator(device="cuda").manual_seed(rank)
    new, n_in = [1000, 64, 0, 130], 1024
    n = sum(new)
    xs = torch.randn(n, n_in, generator=g, device="cuda")
    scale = torch.rand(n, generator=g, device="cuda") * 0.02 if x == I8 else None
    xs = (40 * xs).clamp(-128, 127).round().to(I8) if x == I8 else xs.to(x)
    a = [(torch.randn(3, rank, n_in, generator=g, device="cuda") * n_in ** -0.5).to(w)]
    b = [torch.randn(3, out, rank, generator=g, device="cuda").to(w)]
    wide = -(-out // 4) * 4 + 8  # rows of a wider tensor: what lies beside them stays as it is
    y = torch.randn(n, wide, generator=g, device="cuda")
    cu, who = _i32(np.concatenate([[0], np.cumsum(new)])), _i32([0, 2, 1, 1])

    def call():
        o = torch.full_like(y, 7.0)
        C.cq_lora_add([y[:, 4:out + 4]], xs, a, b, who, cu, x_scale=scale, outs=[o[:, 4:out + 4]])
        C.cq_device_status()
        return o

    want = call()
    assert (want[:, :4] == 7.0).all() and (want[:, out + 4:] == 7.0).all()
    for in_place in (False, True):
        o = y.clone() if in_place else torch.full_like(y, 7.0)
        sides = o[:, :4].clone(), o[:, out + 4:].clone()
        with monkeypatch.context() as m:
            m.setattr(lib, "cq_lora_add", lib.cq_selftest_lora_timeout)
            C.cq_lora_add([o[:, 4:out + 4] if in_place else y[:, 4:out + 4]], xs, a, b, who, cu, x_scale=scale, outs=None if in_place else [o[:, 4:out + 4]])
        with pytest.raises(C.CQError, match="0x474b0001"):
            C.cq_device_status()
        C.cq_device_status()
        assert torch.equal(o[:, :4], sides[0]) and torch.equal(o[:, out + 4:], sides[1])
        assert torch.equal(call(), want)


@pytest.mark.parametrize("n,d", [(3, 64), (5000, 128), (20000, 512), (2, 4096), (3001, 1024), (5000, 2048), (2000, 8192), (700, 16384)])
@pytest.mark.parametrize("dtype,out", [(F32, I8), (BF16, BF16)])
def test_norms_whose_waits_run_out(C, lib, monkeypatch, n, d, dtype, out):
    """Rows of a warp and of a block, rings of one stage and of several, one row of a team and many."""
    g = torch.Generator(device="cuda").manual_seed(d)
    x = torch.randn(n, d, generator=g, device="cuda").to(dtype)
    res, gate = torch.randn(n, d, generator=g, device="cuda").to(dtype), torch.randn(n, d, generator=g, device="cuda").to(dtype)
    w = torch.randn(d, generator=g, device="cuda")

    def call():
        return C.cq_block_norm(x, res, w, post_norm=True, gate=gate, gate_act="silu", out_dtype=out)

    want = call()
    C.cq_device_status()
    with monkeypatch.context() as m:
        m.setattr(lib, "cq_block_norm", lib.cq_selftest_norm_timeout)
        call()
    with pytest.raises(C.CQError, match="0x474a0001"):
        C.cq_device_status()
    C.cq_device_status()
    assert all(torch.equal(a, b) for a, b in zip(call(), want))
