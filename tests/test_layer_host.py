"""Host logic of a layer's other serving steps (no GPU): the refusal of bad
arguments before anything is launched."""
import ctypes
import math
import os
import re

import pytest


@pytest.fixture(scope="module")
def C():
    from hadamard_rotated_codebook_gb300 import build
    build.build()
    import hadamard_rotated_codebook_gb300 as pkg
    return pkg


@pytest.fixture(scope="module")
def A(C):
    from hadamard_rotated_codebook_gb300 import _capi
    return _capi


def _norm(A, **kw):
    d = dict(x=16, residual=16, out=32, residual_out=32, x_stride=64, residual_stride=64, out_stride=64, residual_out_stride=64, n_tokens=2,
             width=64, eps=1e-6, branch_scale=1.0, residual_scale=1.0)
    d.update(kw)
    return A.NormDesc(**d)


@pytest.mark.parametrize("kw,code", [
    (dict(x_dtype=3), "ARG"), (dict(residual_dtype=-1), "ARG"), (dict(out_dtype=4), "ARG"), (dict(n_tokens=-1), "SHAPE"),
    (dict(width=0), "SHAPE"), (dict(width=16385), "SHAPE"), (dict(gate=16, gate_width=2), "SHAPE"), (dict(gate_act=3), "ARG"),
    (dict(eps=-1.0), "ARG"), (dict(eps=math.nan), "ARG"), (dict(weight_offset=math.inf), "ARG"), (dict(branch_scale=math.nan), "ARG"),
    (dict(residual_scale=math.inf), "ARG"), (dict(x=None), "ARG"), (dict(out=None), "ARG"), (dict(out_dtype=3), "ARG"),
    (dict(out_stride=63), "SHAPE"), (dict(residual_out_stride=0), "SHAPE"),
])
def test_block_norm_refuses(A, kw, code):
    assert A.load().cq_block_norm(ctypes.byref(_norm(A, **kw)), None) == getattr(A, "CQ_ERR_" + code)
    assert A.load().cq_last_error()


def _lora(A, **kw):
    d = dict(x=16, adapters=16, cu_tokens=16, x_stride=64, n_mats=1, n_tokens=4, n_seqs=2, n_adapters=3, in_=64, rank=8, x_dtype=0, w_dtype=1,
             workspace=32, workspace_bytes=1 << 20)
    first = dict(a=16, b=16, y=16, y_out=32, y_stride=32, y_out_stride=32, out=32)
    first.update({k: kw[k] for k in kw if k in first})
    d.update({k: kw[k] for k in kw if k not in first})
    t = A.LoraDesc(**d)
    for k, v in first.items():
        getattr(t, k)[0] = v
    return t


@pytest.mark.parametrize("kw,code", [
    (dict(w_dtype=0), "ARG"), (dict(w_dtype=3), "ARG"), (dict(x_dtype=2), "ARG"), (dict(x_dtype=4), "ARG"), (dict(n_mats=-1), "SHAPE"),
    (dict(n_mats=9), "SHAPE"), (dict(n_tokens=-1), "SHAPE"), (dict(n_seqs=-1), "SHAPE"), (dict(n_adapters=-1), "SHAPE"), (dict(in_=0), "SHAPE"),
    (dict(in_=2 ** 30), "SHAPE"), (dict(rank=0), "SHAPE"), (dict(rank=257), "SHAPE"), (dict(out=0), "SHAPE"), (dict(out=2 ** 30), "SHAPE"),
    (dict(x=None), "ARG"), (dict(adapters=None), "ARG"), (dict(cu_tokens=None), "ARG"), (dict(x_dtype=3), "ARG"), (dict(a=None), "ARG"),
    (dict(b=None), "ARG"), (dict(y=None), "ARG"), (dict(y_out=None), "ARG"), (dict(y_out_stride=31), "SHAPE"), (dict(y=32, y_stride=40), "SHAPE"),
    (dict(workspace=None), "ARG"), (dict(workspace_bytes=16), "ARG"), (dict(workspace=40), "ARG"),
])
def test_lora_add_refuses(A, kw, code):
    assert A.load().cq_lora_add(ctypes.byref(_lora(A, **kw)), None) == getattr(A, "CQ_ERR_" + code)
    assert A.load().cq_last_error()


def test_outputs_that_share_memory_are_refused(A):
    lib = A.load()
    assert lib.cq_block_norm(ctypes.byref(_norm(A)), None) == A.CQ_ERR_ARG and b"share" in lib.cq_last_error()

    def two(**kw):
        t = _lora(A, n_mats=2)
        for f, v in dict(a=16, b=16, y=48, y_out=64, y_stride=32, y_out_stride=32, out=32).items():
            getattr(t, f)[1] = kw.get(f, v)
        return lib.cq_lora_add(ctypes.byref(t), None)

    for kw in (dict(y_out=32), dict(y=32), dict(y_out=16)):  # the other's output twice, the other's output as y, x
        assert two(**kw) == A.CQ_ERR_ARG and b"output" in lib.cq_last_error()
    t = _lora(A, x=32)
    assert lib.cq_lora_add(ctypes.byref(t), None) == A.CQ_ERR_ARG and b"output" in lib.cq_last_error()


def test_lora_workspace(A):
    """A function of sizes and types; nothing where there is nothing to do or a size is bad."""
    size = lambda **kw: A.load().cq_lora_workspace(ctypes.byref(_lora(A, **kw)))  # noqa: E731
    assert size() >= 4 * 16 * 4 and size(x=None, adapters=None) == size()
    assert size(n_tokens=400) > size() and size(rank=100) > size()
    for kw in (dict(n_tokens=0), dict(n_seqs=0), dict(n_mats=0), dict(rank=0), dict(x_dtype=2), dict(out=0)):
        assert size(**kw) == 0
    assert A.load().cq_lora_workspace(None) == 0


def test_window_attend_refuses(A):
    cb = (ctypes.c_float * 4)(-0.13, -0.04, 0.04, 0.13)
    g = A.KvGeom(n_q_heads=4, n_kv_heads=2, head_dim_k=48, head_dim_v=64, k_bits=2, v_bits=2, k_codebook=cb, v_codebook=cb, scale=0.1)
    t = A.KvTree(k_cache=16, v_cache=16, block_table=16, context_lens=16, cu_nodes=16, q=16, o=16, table_stride=4, cap=64, max_blocks=4, block_size=16,
                 n_seqs=2, n_nodes=0, max_nodes=2, dtype=1)
    call = lambda w, tree=t: A.load().cq_kv_window_attend(ctypes.byref(g), ctypes.byref(tree), w, None)  # noqa: E731
    assert call(None) == A.CQ_ERR_ARG
    assert call(ctypes.byref(A.KvWindow(None, 1, 0))) == 0  # no nodes: nothing to do
    for window, sinks in ((0, 0), (-1, 0), (1, -1)):
        assert call(ctypes.byref(A.KvWindow(None, window, sinks))) == A.CQ_ERR_SHAPE and A.load().cq_last_error()
    t.block_size = 0
    assert call(ctypes.byref(A.KvWindow(None, 1, 0))) == A.CQ_ERR_SHAPE


def test_empty_calls_do_nothing(A):
    lib = A.load()
    assert lib.cq_block_norm(ctypes.byref(_norm(A, n_tokens=0, x=None)), None) == 0
    assert lib.cq_lora_add(ctypes.byref(_lora(A, n_tokens=0, x=None)), None) == 0
    assert lib.cq_lora_add(ctypes.byref(_lora(A, n_seqs=0, adapters=None)), None) == 0
    assert lib.cq_lora_add(ctypes.byref(_lora(A, n_mats=0)), None) == 0
    assert lib.cq_block_norm(None, None) == A.CQ_ERR_ARG and lib.cq_lora_add(None, None) == A.CQ_ERR_ARG


def test_host_tensors_are_refused(C):
    """The binding takes device tensors only, and says so before it calls the library."""
    import torch
    x, i = torch.zeros(2, 8), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(TypeError):
        C.cq_block_norm(x)
    with pytest.raises(TypeError):
        C.cq_lora_add([x], x, [torch.zeros(1, 4, 8, dtype=torch.float16)], [torch.zeros(1, 8, 4, dtype=torch.float16)], i, i)


def _fields(A, struct):
    """(name, bytes) of a struct of the header, in order."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(root, "include", "cq.h")).read(), flags=re.S)
    body = re.search(r"typedef struct %s \{([^}]*)\} %s;" % (struct, struct), src).group(1)
    out = []
    for decl in filter(None, (s.strip() for s in body.split(";"))):
        kind = re.match(r"(const )?(void|float|int32_t|int64_t|size_t|int)\b", decl)
        for part in decl[kind.end():].split(","):
            size = 8 if "*" in part else {"int64_t": 8, "size_t": 8, "int": 4, "float": 4}[kind.group(2)]
            out.append((re.search(r"\w+", part).group(0), size * (A.CQ_LORA_MAX_MATS if "[" in part else 1)))
    return out


def test_packed_adapters_match_the_structure(C, A):
    """The binding packs LoraDesc in one go: every value arrives in its field."""
    from hadamard_rotated_codebook_gb300 import layer
    values = list(range(1, 74))
    data = layer._LORA_PACK(*values)
    assert len(data) == ctypes.sizeof(A.LoraDesc)
    d, got = A.LoraDesc.from_buffer_copy(data), []
    for name, _ in A.LoraDesc._fields_:
        v = getattr(d, name)
        got += list(v) if isinstance(v, ctypes.Array) else [v]
    assert got == values


def test_binding_structures_match_the_header(A):
    """Field by field: the header's structs and the binding's have the same order and sizes."""
    for name, cls in (("cq_norm_desc", A.NormDesc), ("cq_lora_desc", A.LoraDesc), ("cq_kv_window", A.KvWindow)):
        assert [(f[0].rstrip("_"), ctypes.sizeof(f[1])) for f in cls._fields_] == _fields(A, name)
