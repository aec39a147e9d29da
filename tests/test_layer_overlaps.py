"""Outputs of a layer's other serving steps that share memory with each other or with what is read (no GPU): refused, but for an output
that takes an input's place element by element."""
import ctypes

import pytest

F32, F16, BF16, I8 = 0, 1, 2, 3


@pytest.fixture(scope="module")
def A():
    from hadamard_rotated_codebook_gb300 import build
    build.build()
    from hadamard_rotated_codebook_gb300 import _capi
    return _capi


def _norm(A, **kw):
    """Rows of 64 elements: x in fp32, a residual in fp32, codes; no two of them near each other."""
    d = dict(x=1 << 20, residual=2 << 20, out=3 << 20, residual_out=4 << 20, out_scale=5 << 20, weight=6 << 20, branch_weight=7 << 20, x_stride=64,
             residual_stride=64, out_stride=64, residual_out_stride=64, n_tokens=9, width=64, out_dtype=I8, eps=1e-6, branch_scale=1.0,
             residual_scale=1.0)
    d.update(kw)
    return A.load().cq_block_norm(ctypes.byref(A.NormDesc(**d)), None)


@pytest.mark.parametrize("kw", [
    dict(out=1 << 20),                                                        # codes over x
    dict(out=(1 << 20) + 64 * 4 * 8 + 255),                                   # over its last byte
    dict(out=(1 << 20) - 8 * 64 - 63),                                        # over its first
    dict(out=2 << 20, out_dtype=BF16),                                        # a narrower type over the residual
    dict(out=(2 << 20) + 256, out_dtype=F32),                                 # the residual's next row
    dict(out=(1 << 20) + 4, out_dtype=F32),                                   # x's next element
    dict(residual_out=2 << 20, residual_out_stride=128),                      # the residual in another layout
    dict(residual_out=1 << 20, residual_dtype=BF16),                          # x in another type
    dict(residual_out=(3 << 20) + 5),                                         # the two outputs, rows of one within the other's
    dict(residual_out=(3 << 20) + 48, out_stride=256, residual_out_stride=64),  # likewise, and only some of them meet
    dict(gate=(2 << 20) + 4 * 5, gate_width=1, gate_stride=64, residual_out=2 << 20),  # a gate that is a column of the residual
    dict(gate=(4 << 20) + 4, gate_width=64, gate_stride=64),                  # a gate an element off
    dict(out=6 << 20), dict(residual_out=(7 << 20) + 252), dict(out_scale=(1 << 20) + 8), dict(out_scale=(4 << 20) + 100),
])
def test_norms_refuse_shared_memory(A, kw):
    assert _norm(A, **kw) == A.CQ_ERR_ARG and b"share" in A.load().cq_last_error()


def _lora(A, **kw):
    """Two matrices of 32 outputs that lie side by side in rows of 96, x in fp32; the call ends at its missing workspace."""
    d = dict(x=1 << 20, x_stride=64, y0=2 << 20, y1=(2 << 20) + 128, o0=2 << 20, o1=(2 << 20) + 128, ys0=96, ys1=96, os0=96, os1=96, n=9)
    d.update(kw)
    t = A.LoraDesc(x=d["x"], adapters=16, cu_tokens=16, x_stride=d["x_stride"], n_mats=2, n_tokens=d["n"], n_seqs=2, n_adapters=3, in_=64, rank=8,
                   x_dtype=F32, w_dtype=F16)
    for j in range(2):
        t.a[j] = t.b[j] = 16
        t.y[j], t.y_out[j], t.y_stride[j], t.y_out_stride[j], t.out[j] = d[f"y{j}"], d[f"o{j}"], d[f"ys{j}"], d[f"os{j}"], 32
    assert A.load().cq_lora_add(ctypes.byref(t), None) == A.CQ_ERR_ARG
    return A.load().cq_last_error()


@pytest.mark.parametrize("kw", [
    dict(o1=(2 << 20) + 124), dict(o0=(2 << 20) + 4), dict(o0=(2 << 20) + 384), dict(o0=(2 << 20) - 384),  # an element or a row off
    dict(o0=4 << 20, o1=(4 << 20) + 64),                                    # outputs over each other by half
    dict(o0=4 << 20, o1=(4 << 20) + 128, os0=32),                           # rows of one through the other's
    dict(o0=4 << 20, o1=2 << 20),                                           # one matrix's output in the other's y
    dict(x=(2 << 20) + 4 * 60, x_stride=96),                                # columns of x in the last ones of an output
    dict(x=(2 << 20) - 255, x_stride=64), dict(x=(2 << 20) + 8 * 384 + 252),  # a byte of x
    dict(n=1, o0=(2 << 20) + 124),
])
def test_adapters_refuse_shared_memory(A, kw):
    assert b"shares memory" in _lora(A, **kw)


@pytest.mark.parametrize("kw", [
    dict(), dict(o0=4 << 20, o1=5 << 20), dict(o0=4 << 20, o1=(4 << 20) + 128),
    dict(x=(2 << 20) + 256, x_stride=160, y0=2 << 20, ys0=160, os0=160, ys1=160, os1=160),  # x beside them in the same rows
    dict(y0=4 << 20, y1=4 << 20, ys0=0, ys1=0, o0=2 << 20),                 # a row that all tokens share, and both matrices
    dict(x=1 << 20, x_stride=0), dict(x=1 << 20, x_stride=-64),
    dict(n=1, ys0=7, os0=50), dict(x=(2 << 20) - 256 - 8 * 256), dict(x=(2 << 20) + 8 * 384 + 256),
])
def test_adapters_take_memory_that_is_not_shared(A, kw):
    assert b"workspace" in _lora(A, **kw)


def test_rows_that_share_a_byte(A):
    """Every small arrangement of an output's rows and x's, against the bytes themselves."""
    import random
    rng = random.Random(0)
    for _ in range(4000):
        n, ys, xs, at = rng.randint(1, 5), rng.randint(33, 90), rng.choice([0, 40, 64, 70, rng.randint(-90, 90)]), rng.randint(-3000, 3000)
        out = {(2 << 20) + 4 * (i * ys) + k for i in range(n) for k in range(128)}
        read = {(2 << 20) + at + 4 * i * xs + k for i in range(n) for k in range(256)}
        got = _lora(A, n=n, x=(2 << 20) + at, x_stride=xs, ys0=ys, os0=ys, y1=8 << 20, o1=8 << 20)
        assert (b"shares memory" in got) == bool(out & read) and (b"workspace" in got) != bool(out & read)
