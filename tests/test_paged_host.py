"""Host logic of the paged cache's entry points (no GPU): rotation rates and
the refusal of bad arguments before anything is launched."""
import ctypes
import math

import numpy as np
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


CB2 = (ctypes.c_float * 4)(-0.13, -0.04, 0.04, 0.13)


def test_rope_rates_are_fractions_of_a_turn(C):
    rot = 64
    rates = C.cq_rope_init(rot, theta=500.0)
    assert rates.dtype == np.uint64 and rates.shape == (32,)
    want = 500.0 ** (-np.arange(0, rot, 2) / rot) / (2 * math.pi)
    np.testing.assert_allclose(rates.astype(np.float64) / 2.0 ** 64, want, rtol=1e-15)
    # whole turns drop out, and a negative rate turns the other way
    two = C.cq_rope_init(4, inv_freq=[2 * math.pi * 3.25, -2 * math.pi * 0.25]).astype(np.float64) / 2.0 ** 64
    np.testing.assert_allclose(two, [0.25, 0.75], atol=1e-14)
    assert C.cq_rope_init(0).shape == (0,)


def test_rope_rates_hold_all_their_bits(C):
    """Against 2 pi in 60 digits: within two units of 2^-64, so that the largest position moves an angle by 2^-32 of a turn."""
    from decimal import Decimal, getcontext
    getcontext().prec = 120
    two_pi = Decimal("6.28318530717958647692528676655900576839433879875021164194988918461563281257")
    rng = np.random.RandomState(0)
    freq = np.concatenate([[1.0, -1.0, 0.5, 1e-5, -1e-7, 6.283185307179586, 3.0, 1e-300, -1e-300, 0.0, 1000.0, -77.7],
                           10000.0 ** -rng.rand(40), -(500000.0 ** -rng.rand(12))])
    for at in range(0, len(freq), 32):
        part = freq[at:at + 32]
        rates = C.cq_rope_init(2 * len(part), inv_freq=part)
        for f, r in zip(part, rates):
            want = Decimal(float(f)) / two_pi * 2 ** 64
            off = (Decimal(int(r)) - want) % 2 ** 64
            assert min(off, 2 ** 64 - off) <= 2, f


def test_rope_init_refuses(C, A):
    for kw in (dict(rot_dim=7), dict(rot_dim=258), dict(rot_dim=8, theta=0.0), dict(rot_dim=8, theta=math.inf),
               dict(rot_dim=4, inv_freq=[1.0, math.nan])):
        with pytest.raises(C.CQError):
            C.cq_rope_init(**kw)
    with pytest.raises(ValueError):
        C.cq_rope_init(8, inv_freq=[1.0])
    lib = A.load()
    n = ctypes.c_size_t(0)
    assert lib.cq_rope_init(8, 10.0, None, None, 0, ctypes.byref(n)) == 0 and n.value == 4
    assert lib.cq_rope_init(8, 10.0, None, (ctypes.c_uint64 * 3)(), 3, None) == A.CQ_ERR_ARG


def _qk(A, **kw):
    d = dict(q=16, k=16, q_out=16, k_out=16, positions=16, rates=16, n_tokens=2, n_q_heads=2, n_kv_heads=1, head_dim=8,
             rot_dim=8, in_dtype=0, q_out_dtype=1, k_out_dtype=0, eps=1e-6)
    d.update(kw)
    return A.QkDesc(**d)


@pytest.mark.parametrize("kw,code", [
    (dict(in_dtype=3), "ARG"), (dict(q_out_dtype=-1), "ARG"), (dict(k_out_dtype=9), "ARG"),
    (dict(head_dim=7), "SHAPE"), (dict(head_dim=258), "SHAPE"), (dict(head_dim=0), "SHAPE"),
    (dict(rot_dim=10), "SHAPE"), (dict(rot_dim=3), "SHAPE"), (dict(rot_dim=-2), "SHAPE"),
    (dict(n_tokens=-1), "SHAPE"), (dict(n_q_heads=-1), "SHAPE"), (dict(n_q_heads=70000), "SHAPE"),
    (dict(eps=-1.0), "ARG"), (dict(eps=math.nan), "ARG"), (dict(weight_offset=math.inf), "ARG"),
    (dict(q=None), "ARG"), (dict(k_out=None), "ARG"), (dict(positions=None), "ARG"), (dict(rates=None), "ARG"),
])
def test_qk_norm_rope_refuses(A, kw, code):
    assert A.load().cq_qk_norm_rope(ctypes.byref(_qk(A, **kw)), None) == getattr(A, "CQ_ERR_" + code)
    assert A.load().cq_last_error()


def test_empty_calls_do_nothing(A):
    lib = A.load()
    assert lib.cq_qk_norm_rope(ctypes.byref(_qk(A, n_tokens=0, q=None, k=None)), None) == 0
    assert lib.cq_qk_norm_rope(ctypes.byref(_qk(A, n_q_heads=0, n_kv_heads=0)), None) == 0
    g = _geom(A)
    assert lib.cq_kv_write_slots(ctypes.byref(g), None, None, 0, None, 0, None, 0, 0, None, 0, None) == 0
    assert lib.cq_kv_tree_attend(ctypes.byref(g), ctypes.byref(_tree(A, n_seqs=0)), None) == 0
    assert lib.cq_kv_tree_attend(ctypes.byref(g), ctypes.byref(_tree(A, n_nodes=0)), None) == 0
    assert lib.cq_qk_norm_rope(None, None) == A.CQ_ERR_ARG
    assert lib.cq_kv_plan(None, None) == A.CQ_ERR_ARG
    assert lib.cq_kv_tree_attend(ctypes.byref(g), None, None) == A.CQ_ERR_ARG
    assert lib.cq_kv_tree_attend(None, ctypes.byref(_tree(A)), None) == A.CQ_ERR_ARG


def _step(A, **kw):
    d = dict(seq_lens=0x1000, new_lens=0x2000, held=0x3000, block_table=0x4000, free_list=0x5000, n_free=0x6000,
             held_out=0x7000, n_free_out=0x8000, slots=0x9000, positions=0xA000, token_seq=0xB000, cu_new=0xC000,
             table_stride=4, n_seqs=3, max_blocks=4, block_size=16, free_cap=10, n_tokens=20)
    d.update(kw)
    return A.KvStep(**d)


@pytest.mark.parametrize("kw,code", [
    (dict(n_seqs=-1), "SHAPE"), (dict(n_seqs=1 << 21), "SHAPE"), (dict(max_blocks=-1), "SHAPE"),
    (dict(free_cap=-1), "SHAPE"), (dict(n_tokens=-1), "SHAPE"), (dict(block_size=0), "SHAPE"), (dict(table_stride=3), "SHAPE"),
    (dict(cu_new=None), "ARG"), (dict(n_free=None), "ARG"), (dict(n_free_out=None), "ARG"), (dict(seq_lens=None), "ARG"),
    (dict(held_out=None), "ARG"), (dict(block_table=None), "ARG"), (dict(free_list=None), "ARG"), (dict(slots=None), "ARG"),
    (dict(held_out=0x3000), "ARG"), (dict(held_out=0x3004), "ARG"), (dict(n_free_out=0x6000), "ARG"),
])
def test_kv_plan_refuses(A, kw, code):
    assert A.load().cq_kv_plan(ctypes.byref(_step(A, **kw)), None) == getattr(A, "CQ_ERR_" + code)
    assert A.load().cq_last_error()


def _geom(A, **kw):
    d = dict(n_q_heads=4, n_kv_heads=2, head_dim_k=48, head_dim_v=64, k_bits=2, v_bits=2, k_codebook=CB2, v_codebook=CB2,
             scale=0.1)
    d.update(kw)
    return A.KvGeom(**d)


BAD_CACHE = [
    (dict(n_kv_heads=0), "SHAPE"), (dict(head_dim_k=0), "SHAPE"), (dict(head_dim_v=-1), "SHAPE"),
    (dict(n_kv_heads=4096, n_q_heads=4096), "SHAPE"), (dict(k_bits=1), "ARG"), (dict(v_bits=6), "ARG"),
    (dict(k_codebook=None), "ARG"), (dict(v_codebook=(ctypes.c_float * 4)(0, 1, 1, 2)), "ARG"),
]


@pytest.mark.parametrize("kw,code", BAD_CACHE)
def test_kv_write_slots_refuses_geometry(A, kw, code):
    g = _geom(A, **kw)
    assert A.load().cq_kv_write_slots(ctypes.byref(g), 16, 16, 8, 16, 96, 16, 128, 0, 16, 2, None) == getattr(A, "CQ_ERR_" + code)


def test_kv_write_slots_refuses(A):
    lib, g = A.load(), _geom(A)

    def call(kc=16, vc=16, cap=8, k=16, ks=96, v=16, vs=128, dtype=0, slots=16, n=2):
        return lib.cq_kv_write_slots(ctypes.byref(g), kc, vc, cap, k, ks, v, vs, dtype, slots, n, None)

    assert lib.cq_kv_write_slots(None, 16, 16, 8, 16, 96, 16, 128, 0, 16, 2, None) == A.CQ_ERR_ARG
    assert call(dtype=3) == A.CQ_ERR_ARG
    assert call(cap=-1) == A.CQ_ERR_SHAPE and call(n=-1) == A.CQ_ERR_SHAPE
    assert call(slots=None) == A.CQ_ERR_ARG and call(k=None) == A.CQ_ERR_ARG and call(vc=None) == A.CQ_ERR_ARG
    assert call(kc=24) == A.CQ_ERR_ARG  # not 16-byte aligned
    assert call(ks=95) == A.CQ_ERR_SHAPE and call(vs=0) == A.CQ_ERR_SHAPE


def _tree(A, **kw):
    d = dict(k_cache=16, v_cache=16, block_table=16, context_lens=16, cu_nodes=16, mask=16, q=16, o=16, workspace=None,
             workspace_bytes=0, table_stride=4, q_stride_t=192, q_stride_h=48, o_stride_t=256, o_stride_h=64, cap=64,
             max_blocks=4, block_size=16, n_seqs=2, n_nodes=3, max_nodes=2, mask_words=1, dtype=1)
    d.update(kw)
    return A.KvTree(**d)


@pytest.mark.parametrize("kw,code", BAD_CACHE + [
    (dict(n_q_heads=3), "SHAPE"), (dict(n_q_heads=0), "SHAPE"), (dict(scale=math.nan), "ARG"),
    (dict(head_dim_k=300), "SHAPE"),   # three groups to a head
    (dict(head_dim_v=200, n_kv_heads=4), "SHAPE"),  # the second head lies in groups 1 to 3
])
def test_kv_tree_attend_refuses_geometry(A, kw, code):
    lib, g = A.load(), _geom(A, **kw)
    assert lib.cq_kv_tree_attend(ctypes.byref(g), ctypes.byref(_tree(A)), None) == getattr(A, "CQ_ERR_" + code)
    assert lib.cq_kv_tree_workspace(ctypes.byref(g), 2, 2) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=0), "ARG"), (dict(n_seqs=-1), "SHAPE"), (dict(n_nodes=-1), "SHAPE"), (dict(cap=-1), "SHAPE"),
    (dict(max_blocks=-1), "SHAPE"), (dict(max_nodes=257, mask_words=9), "SHAPE"), (dict(max_nodes=-1), "SHAPE"),
    (dict(block_size=0), "SHAPE"), (dict(table_stride=3), "SHAPE"), (dict(max_nodes=33), "SHAPE"), (dict(q=None), "ARG"),
    (dict(o=None), "ARG"), (dict(context_lens=None), "ARG"), (dict(cu_nodes=None), "ARG"), (dict(block_table=None), "ARG"),
    (dict(v_cache=None), "ARG"), (dict(k_cache=24), "ARG"),
])
def test_kv_tree_attend_refuses(A, kw, code):
    lib, g = A.load(), _geom(A)
    assert lib.cq_kv_tree_attend(ctypes.byref(g), ctypes.byref(_tree(A, **kw)), None) == getattr(A, "CQ_ERR_" + code)
    assert lib.cq_last_error()


@pytest.mark.parametrize("reserved", [-1, 0, 1023, 1025, 2048])
def test_kv_tree_attend_refuses_another_shared_memory_layout(A, reserved):
    """The kernel's addresses count on shared memory that starts behind 1024 bytes: a device that
    keeps another number is refused on the host, so that the joining kernel never runs over parts
    that no block wrote."""
    lib = A.load()
    assert lib.cq_selftest_tree_smem(1024) == 0
    assert lib.cq_selftest_tree_smem(reserved) == A.CQ_ERR_CUDA
    assert b"shared memory" in lib.cq_last_error()


def test_host_tensors_are_refused(C):
    """The binding takes device tensors only, and says so before it calls the library."""
    import torch
    x, i = torch.zeros(2, 4, 8), torch.zeros(2, dtype=torch.int32)
    rates = C.cq_rope_init(8)
    with pytest.raises(TypeError):
        C.cq_qk_norm_rope(x, x, i, rates)
    with pytest.raises(TypeError):
        C.cq_kv_plan(i, i, i, torch.zeros(2, 2, dtype=torch.int32), i, i, 16, 4)
    cb = np.array(CB2, dtype=np.float32)
    g = C.cq_kv_geometry(4, 2, 48, 64, 2, 2, cb, cb, 0.1)
    with pytest.raises(TypeError):
        C.cq_kv_write_slots(g, x, x, 4, torch.zeros(2, 96), torch.zeros(2, 128), i)
    with pytest.raises(TypeError):
        C.cq_kv_tree_attend(g, x, x, x, 4, i, 16, i, i, None, 2)
    with pytest.raises(ValueError):
        C.cq_kv_geometry(4, 2, 48, 64, 3, 2, cb, cb, 0.1)  # four levels for three bits


def test_sizes_past_32_bits_are_refused(C):
    """They are cut to 32 bits on the way into the library: 2^32 + 16 would pass as 16."""
    import torch
    x, i = torch.zeros(2, 4, 8), torch.zeros(2, dtype=torch.int32)
    wide = 2 ** 32
    cb = np.array(CB2, dtype=np.float32)
    g = C.cq_kv_geometry(4, 2, 48, 64, 2, 2, cb, cb, 0.1)
    for call in (lambda: C.cq_rope_init(wide + 8),
                 lambda: C.cq_kv_geometry(wide + 4, 2, 48, 64, 2, 2, cb, cb, 0.1), lambda: C.cq_kv_geometry(4, 2 - wide, 48, 64, 2, 2, cb, cb, 0.1),
                 lambda: C.cq_kv_geometry(4, 2, wide + 48, 64, 2, 2, cb, cb, 0.1), lambda: C.cq_kv_geometry(4, 2, 48, wide + 64, 2, 2, cb, cb, 0.1),
                 lambda: C.cq_kv_plan(i, i, i, torch.zeros(2, 2, dtype=torch.int32), i, i, wide + 16, 4),
                 lambda: C.cq_kv_plan(i, i, i, torch.zeros(2, 2, dtype=torch.int32), i, i, 16, wide + 4),
                 lambda: C.cq_kv_write_slots(g, x, x, wide + 4, torch.zeros(2, 96), torch.zeros(2, 128), i),
                 lambda: C.cq_kv_tree_attend(g, x, x, x, wide + 4, i, 16, i, i, None, 2),
                 lambda: C.cq_kv_tree_attend(g, x, x, x, 4, i, wide + 16, i, i, None, 2),
                 lambda: C.cq_kv_tree_attend(g, x, x, x, 4, i, 16, i, i, None, wide + 2)):
        with pytest.raises(ValueError, match="32 bits"):
            call()
