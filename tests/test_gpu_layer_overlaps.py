"""GPU: what tensors of a layer's other serving steps may share, and that the rest is refused before a launch."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

F32, F16, BF16, I8 = torch.float32, torch.float16, torch.bfloat16, torch.int8


@pytest.fixture(scope="module")
def C():
    import hadamard_rotated_codebook_gb300 as pkg
    return pkg


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("d", [1, 7, 320, 333, 1000, 2048, 2056])
@pytest.mark.parametrize("n", [1, 5000])
def test_norm_outputs_in_the_place_of_inputs(C, d, n):
    """Each output over each input of its type, rows of a wider tensor among them: the bits of a call into tensors of their own."""
    g = torch.Generator(device="cuda").manual_seed(d)
    w = torch.randn(d, generator=g, device="cuda")
    opt = dict(post_norm=True, gate_act="silu")
    for wide in (0, 3):
        first = [torch.randn(n, d + wide, generator=g, device="cuda").to(BF16) for _ in range(3)]
        want = C.cq_block_norm(first[0][:, wide:], first[1][:, wide:], w, gate=first[2][:, wide:], **opt)
        for a in (None, 0, 1, 2):
            for b in (None, 0, 1, 2):
                if a == b:
                    continue
                t = [f.clone() for f in first]
                x, res, gate = (f[:, wide:] for f in t)
                r, y = C.cq_block_norm(x, res, w, gate=gate, residual_out=None if a is None else (x, res, gate)[a],
                                       out=None if b is None else (x, res, gate)[b], **opt)
                assert torch.equal(r, want[0]) and torch.equal(y, want[1])
                assert all(torch.equal(f[:, :wide], s[:, :wide]) for f, s in zip(t, first))


def test_norm_of_columns_of_one_tensor(C):
    """x, its gate, the residual and the outputs side by side in one tensor's rows."""
    d = 256
    t = torch.randn(100, 5 * d, device="cuda").to(F16)
    x, gate, res, r, y = t.split(d, 1)
    want = C.cq_block_norm(x.contiguous(), res.contiguous(), gate=gate.contiguous(), gate_act="sigmoid")
    got = C.cq_block_norm(x, res, gate=gate, gate_act="sigmoid", residual_out=r, out=y)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(t[:, 3 * d:4 * d], want[0])


def test_norm_refuses_shared_memory(C):
    t = torch.randn(40, 512, device="cuda")
    before = t.clone()
    x, half = t[:16, :256], t.view(BF16)
    for kw in (dict(x=x, residual=t[16:32, :256], residual_out=t[17:33, :256]), dict(x=x, residual=t[:16, 256:], out=t[:16, 128:384]),
               dict(x=x, residual=t[16:32, :256], out=half[16:32, :256], out_dtype=BF16), dict(x=x, out=t.view(I8)[16:32, :256], residual_out=t[16:32, :256]),
               dict(x=x, residual=t[16:32, 256:], residual_out=t[16:32, 256:], gate=t[16:32, 300:301]),
               dict(x=x, weight=t[3, 256:], out=t[:16, 256:]), dict(x=x, out=t[16:32, :256], residual_out=t[16:32, 64:320])):
        with pytest.raises(C.CQError, match="share"):
            C.cq_block_norm(**kw)
    assert torch.equal(t, before)


def test_adapters_refuse_shared_memory(C):
    t = torch.randn(12, 200, device="cuda")
    before = t.clone()
    a, b = [torch.randn(1, 8, 64, device="cuda").to(F16)] * 2, [torch.randn(1, 32, 8, device="cuda").to(F16)] * 2
    cu, who, x = _i32([0, 5]), _i32([0]), t[:5, 128:192]
    for ys, xs, outs in (([t[:5, :32], t[:5, 32:64]], t[:5, 40:104], None), ([t[:5, :32], t[:5, 31:63]], x, None),
                         ([t[:5, :32], t[:5, 32:64]], x, [t[1:6, :32], t[:5, 64:96]]), ([t[:5, :32], t[:5, 32:64]], x, [t[:5, 32:64], t[:5, :32]])):
        with pytest.raises(C.CQError, match="shares memory"):
            C.cq_lora_add(ys, xs, a, b, who, cu, outs=outs)
    assert torch.equal(t, before)
    want = C.cq_lora_add([t[:5, :32].clone(), t[:5, 32:64].clone()], x.clone(), a, b, who, cu)
    got = C.cq_lora_add([t[:5, :32], t[:5, 32:64]], x, a, b, who, cu)  # side by side
    assert all(torch.equal(p, q) for p, q in zip(got, want)) and torch.equal(t[:, 64:], before[:, 64:])
