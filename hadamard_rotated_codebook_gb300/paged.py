"""Serving steps over a paged CQ KV cache: per-head norms with the position
rotation, block tables and slot maps, slot writes, and attention of drafted
tokens. Thin bindings like the rest of the package: arguments are checked and
marshalled, all arithmetic runs in libcq's kernels.

A cache is one uint8 tensor of ``cq_packed_bytes(cap, width, 128, bits)`` bytes;
block b is its rows b*block_size .. (b+1)*block_size - 1. Lengths, tables and
slots are int32 device tensors, so a captured graph serves any lengths up to
the sizes of its tensors.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
from typing import Optional

import numpy as np
import torch

from . import _capi
from . import _codebook_arg, cq_packed_bytes
from ._capi import CQ_T_BF16, CQ_T_F16, CQ_T_F32, KvGeom, KvStep, KvTree, QkDesc, check

_TYPE = {torch.float32: CQ_T_F32, torch.float16: CQ_T_F16, torch.bfloat16: CQ_T_BF16}
_load = _capi.load
_stay = contextlib.nullcontext()
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (  # the handle without a Stream object around it
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _ints(**sizes) -> None:
    """The library's sizes are 32 bits wide, and ctypes cuts what is wider without a word. (Calls come here where
    the sizes or'ed together leave 31 bits; what is below zero is the library's to refuse.)"""
    for name, x in sizes.items():
        if not -0x80000000 <= x <= 0x7FFFFFFF:
            raise ValueError(f"{name} must fit 32 bits, got {x}")


def _type(t: torch.Tensor, name: str) -> int:
    try:
        return _TYPE[t.dtype]
    except KeyError:
        raise TypeError(f"{name} must be float32, float16 or bfloat16, got {t.dtype}") from None


def _dev(t: torch.Tensor, name: str, device) -> None:
    """Every tensor of a call lives on the device of its first one."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _i32(t: torch.Tensor, name: str, n: int, device) -> int:
    _dev(t, name, device)
    if t.dtype != torch.int32:
        raise TypeError(f"{name} must be torch.int32, got {t.dtype}")
    if t.numel() < n or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous with at least {n} entries, got {tuple(t.shape)}")
    return t.data_ptr()


def _heads(t: torch.Tensor, name: str, device, out: bool = False):
    """[tokens, heads, width] with a contiguous last dimension; other strides
    are free, but an output's elements must not share memory. Returns the shape
    and the first two strides."""
    _dev(t, name, device)
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or (shape[2] > 1 and stride[2] != 1):
        raise ValueError(f"{name} must be [tokens, heads, width] with a contiguous last dimension, "
                         f"got {tuple(shape)} strides {stride}")
    n, h, d = shape
    st, sh, _ = stride
    if out and n * h * d and not ((h == 1 or sh >= d) and (n == 1 or st >= (h - 1) * sh + d)
                                  or (n == 1 or st >= d) and (h == 1 or sh >= (n - 1) * st + d)):
        raise ValueError(f"{name} overlaps itself: shape {tuple(shape)}, strides {stride}")
    return n, h, d, st, sh


def _weight(w: Optional[torch.Tensor], name: str, d: int, device):
    if w is None:
        return None
    _dev(w, name, device)
    if w.dtype != torch.float32 or w.shape != (d,) or not w.is_contiguous():
        raise ValueError(f"{name} must be contiguous float32 [{d}], got {w.dtype} {tuple(w.shape)}")
    return w.data_ptr()


def _table(t: torch.Tensor, n_seqs: int, device) -> int:
    _dev(t, "block_table", device)
    if t.dtype != torch.int32:
        raise TypeError(f"block_table must be torch.int32, got {t.dtype}")
    if t.dim() != 2 or t.shape[0] < n_seqs or (t.shape[1] > 1 and t.stride(1) != 1) or \
            (n_seqs > 1 and t.stride(0) < t.shape[1]):
        raise ValueError(f"block_table must be [{n_seqs}, blocks] with contiguous rows, got {tuple(t.shape)} "
                         f"strides {t.stride()}")
    return t.data_ptr()


def _call(device, fn, *args) -> None:
    """Calls fn(*args, stream) with `device` current."""
    if device.index == torch.cuda.current_device():
        code = fn(*args, _raw_stream(device.index))
    else:
        with torch.cuda.device(device):
            code = fn(*args, _raw_stream(device.index))
    if code:
        check(code)


def cq_rope_init(rot_dim: int, theta: float = 10000.0, inv_freq=None) -> np.ndarray:
    """Rotation rates for cq_qk_norm_rope, made once per model: ``rot_dim / 2``
    64-bit fractions of a turn per position, of theta^(-2i/rot_dim) or of the
    given ``inv_freq`` (radians per position)."""
    _ints(rot_dim=rot_dim)
    n = max(0, rot_dim // 2)
    rates = np.zeros(n, dtype=np.uint64)
    f = None
    if inv_freq is not None:
        if isinstance(inv_freq, torch.Tensor):
            inv_freq = inv_freq.detach().cpu().numpy()
        f = np.ascontiguousarray(inv_freq, dtype=np.float64)
        if f.shape != (n,):
            raise ValueError(f"inv_freq must have {n} entries, got shape {f.shape}")
    check(_load().cq_rope_init(rot_dim, theta, f.ctypes.data_as(ctypes.POINTER(ctypes.c_double)) if f is not None else None,
                               rates.ctypes.data_as(ctypes.POINTER(ctypes.c_uint64)), n, None))
    return rates


def cq_qk_norm_rope(q: torch.Tensor, k: torch.Tensor, positions: torch.Tensor, rates: np.ndarray,
                    q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None, *,
                    eps: float = 1e-6, weight_offset: float = 0.0, interleaved: bool = False,
                    q_dtype: Optional[torch.dtype] = None, k_dtype: Optional[torch.dtype] = None,
                    q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None):
    """Norm of every head of q [tokens, Hq, d] and k [tokens, Hkv, d] (fp32,
    fp16 or bf16; slices of a packed projection are fine) and its rotation by
    ``positions`` (int32 [tokens]), in one launch:
    ``y = x / sqrt(mean(x^2) + eps) * (weight_offset + weight)``, then the
    pairs (i, i + rot/2), or (2i, 2i + 1) if ``interleaved``, of the first
    ``2 * len(rates)`` elements turn by position * inv_freq. Weights are fp32
    [d] (None: ones). Returns (q_out, k_out); outputs may be given, may have
    another type than the input, and may be the inputs themselves."""
    dev = q.device
    n, hq, d, qt, qh = _heads(q, "q", dev)
    if n >> 31:
        _ints(tokens=n)
    nk, hkv, dk, kt, kh = _heads(k, "k", dev)
    dtype = q.dtype
    if n != nk or d != dk or k.dtype != dtype:
        raise ValueError(f"q {tuple(q.shape)} {dtype} and k {tuple(k.shape)} {k.dtype} do not belong together")
    if not isinstance(rates, np.ndarray) or rates.dtype != np.uint64 or not rates.flags.c_contiguous:
        raise TypeError("rates must be the array cq_rope_init returned")
    if q_out is None:
        q_out = torch.empty((n, hq, d), dtype=q_dtype or dtype, device=dev)
    if k_out is None:
        k_out = torch.empty((n, hkv, d), dtype=k_dtype or dtype, device=dev)
    qn, qc, qd, qot, qoh = _heads(q_out, "q_out", dev, True)
    kn, kc, kd, kot, koh = _heads(k_out, "k_out", dev, True)
    if qn != n or kn != n or qc != hq or kc != hkv or qd != d or kd != d:
        raise ValueError(f"outputs {tuple(q_out.shape)}, {tuple(k_out.shape)} for inputs {tuple(q.shape)}, {tuple(k.shape)}")
    desc = QkDesc(q.data_ptr(), k.data_ptr(), q_out.data_ptr(), k_out.data_ptr(),
                  _weight(q_weight, "q_weight", d, dev), _weight(k_weight, "k_weight", d, dev),
                  _i32(positions, "positions", n, dev), rates.ctypes.data, qt, qh, kt, kh, qot, qoh, kot, koh,
                  _type(q, "q"), _type(q_out, "q_out"), _type(k_out, "k_out"),
                  n, hq, hkv, d, 2 * rates.size, interleaved, eps, weight_offset)
    _call(dev, _load().cq_qk_norm_rope, desc)
    return q_out, k_out


def cq_kv_plan(seq_lens: torch.Tensor, new_lens: torch.Tensor, held: torch.Tensor, block_table: torch.Tensor,
               free_list: torch.Tensor, n_free: torch.Tensor, block_size: int, n_tokens: Optional[int] = None, *,
               held_out: Optional[torch.Tensor] = None, n_free_out: Optional[torch.Tensor] = None,
               slots: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
               token_seq: Optional[torch.Tensor] = None, cu_new: Optional[torch.Tensor] = None) -> dict:
    """Block tables and slot maps of a step on the device: request s appends
    new_lens[s] tokens at positions seq_lens[s] .. ; blocks past the held[s] its
    row of block_table (updated in place) has are popped from the end of
    free_list[:n_free]. ``n_tokens`` is the room of the slot map (default: of
    the given ``slots``); entries past the step's tokens are -1. Returns a dict of held_out,
    n_free_out, slots, positions, token_seq, cu_new (any of them may be given).
    Missing blocks and dropped tokens make a following cq_device_status raise."""
    dev = seq_lens.device
    n = seq_lens.numel()
    if n_tokens is None:
        if slots is None:
            raise ValueError("give n_tokens or slots")
        n_tokens = slots.numel()
    n_free_max = free_list.numel()
    if (n | n_tokens | block_size | n_free_max) >> 31:
        _ints(requests=n, n_tokens=n_tokens, block_size=block_size, free_list=n_free_max)

    def out(t, m):
        return torch.empty(m, dtype=torch.int32, device=dev) if t is None else t

    held_out, n_free_out, cu_new = out(held_out, n), out(n_free_out, 1), out(cu_new, n + 1)
    slots, positions, token_seq = out(slots, n_tokens), out(positions, n_tokens), out(token_seq, n_tokens)
    step = KvStep(_i32(seq_lens, "seq_lens", n, dev), _i32(new_lens, "new_lens", n, dev), _i32(held, "held", n, dev),
                  _table(block_table, n, dev), _i32(free_list, "free_list", 0, dev), _i32(n_free, "n_free", 1, dev),
                  _i32(held_out, "held_out", n, dev), _i32(n_free_out, "n_free_out", 1, dev),
                  _i32(slots, "slots", n_tokens, dev), _i32(positions, "positions", n_tokens, dev),
                  _i32(token_seq, "token_seq", n_tokens, dev), _i32(cu_new, "cu_new", n + 1, dev),
                  block_table.stride(0) if n > 1 else block_table.shape[1], n, block_table.shape[1], block_size,
                  n_free_max, n_tokens)
    _call(dev, _load().cq_kv_plan, step)
    return {"held_out": held_out, "n_free_out": n_free_out, "slots": slots, "positions": positions,
            "token_seq": token_seq, "cu_new": cu_new}


class KvGeometry:
    """What the layers of a model share: heads, widths, bits, codebooks and the
    logit scale, laid out once (see cq_kv_geometry)."""

    def __init__(self, n_q_heads, n_kv_heads, head_dim_k, head_dim_v, k_bits, v_bits, k_codebook, v_codebook, scale):
        _ints(n_q_heads=n_q_heads, n_kv_heads=n_kv_heads, head_dim_k=head_dim_k, head_dim_v=head_dim_v)
        self._keep = _codebook_arg(k_codebook, k_bits), _codebook_arg(v_codebook, v_bits)
        self.n_q_heads, self.n_kv_heads = n_q_heads, n_kv_heads
        self.head_dim_k, self.head_dim_v = head_dim_k, head_dim_v
        self.k_width, self.v_width = n_kv_heads * head_dim_k, n_kv_heads * head_dim_v
        self.k_bits, self.v_bits = k_bits, v_bits
        self.c = KvGeom(n_q_heads=n_q_heads, n_kv_heads=n_kv_heads, head_dim_k=head_dim_k, head_dim_v=head_dim_v,
                        k_bits=k_bits, v_bits=v_bits, k_codebook=self._keep[0][1], v_codebook=self._keep[1][1], scale=scale)
        self._row = [cq_packed_bytes(1, w, 128, b) for w, b in ((self.k_width, k_bits), (self.v_width, v_bits))]
        self._ws: dict = {}

    def check_caches(self, k_cache: torch.Tensor, v_cache: torch.Tensor, cap: int, device) -> None:
        for t, row, name in ((k_cache, self._row[0], "k_cache"), (v_cache, self._row[1], "v_cache")):
            _dev(t, name, device)
            if t.dtype != torch.uint8 or not t.is_contiguous():
                raise TypeError(f"{name} must be a contiguous uint8 tensor")
            if t.numel() < row * cap:
                raise ValueError(f"{name} holds {t.numel()} bytes, {cap} rows need {row * cap}")

    def workspace_bytes(self, n_seqs: int, max_nodes: int, device) -> int:
        key = (n_seqs, max_nodes, device.index)
        n = self._ws.get(key)
        if n is None:
            with (_stay if device.index == torch.cuda.current_device() else torch.cuda.device(device)):
                n = self._ws[key] = _load().cq_kv_tree_workspace(self.c, n_seqs, max_nodes)
        return n


def cq_kv_geometry(n_q_heads: int, n_kv_heads: int, head_dim_k: int, head_dim_v: int, k_bits: int, v_bits: int,
                   k_codebook, v_codebook, scale: float) -> KvGeometry:
    """The geometry that cq_kv_write_slots and cq_kv_tree_attend take."""
    return KvGeometry(n_q_heads, n_kv_heads, head_dim_k, head_dim_v, k_bits, v_bits, k_codebook, v_codebook, scale)


def _rows(t: torch.Tensor, width: int, name: str, device):
    """[n, width] or [n, heads, head width] whose rows are contiguous: (n, row stride)."""
    _dev(t, name, device)
    if t.dim() == 3:
        ok = t.shape[1] * t.shape[2] == width and (t.shape[2] <= 1 or t.stride(2) == 1) and \
            (t.shape[1] <= 1 or t.stride(1) == t.shape[2])
    else:
        ok = t.dim() == 2 and t.shape[1] == width and (width <= 1 or t.stride(1) == 1)
    if not ok:
        raise ValueError(f"{name} must be [n, {width}] or [n, heads, width per head] with contiguous rows, got "
                         f"{tuple(t.shape)} strides {t.stride()}")
    return t.shape[0], t.stride(0)


def cq_kv_write_slots(geom: KvGeometry, k_cache: torch.Tensor, v_cache: torch.Tensor, cap: int, k: torch.Tensor,
                      v: torch.Tensor, slots: torch.Tensor) -> None:
    """Encodes keys and values (fp32, fp16 or bf16, [n, width] or [n, heads,
    head width]) into rows slots[i] of the two caches in one launch; -1 skips
    a row. Slots must be distinct; one outside the cache is skipped and makes a
    following cq_device_status raise."""
    if cap >> 31:
        _ints(cap=cap)
    dev = k.device
    (n, ks), (nv, vs) = _rows(k, geom.k_width, "k", dev), _rows(v, geom.v_width, "v", dev)
    if n != nv or k.dtype != v.dtype:
        raise ValueError(f"k {tuple(k.shape)} {k.dtype} and v {tuple(v.shape)} {v.dtype} do not belong together")
    geom.check_caches(k_cache, v_cache, cap, dev)
    _call(dev, _load().cq_kv_write_slots, geom.c, k_cache.data_ptr(), v_cache.data_ptr(), cap, k.data_ptr(), ks,
          v.data_ptr(), vs, _type(k, "k"), _i32(slots, "slots", n, dev), n)


def cq_kv_tree_attend(geom: KvGeometry, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, cap: int,
                      block_table: torch.Tensor, block_size: int, context_lens: torch.Tensor, cu_nodes: torch.Tensor,
                      mask: Optional[torch.Tensor], max_nodes: int, o: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Attention of drafted tokens q [nodes, Hq, head_dim_k] (fp16 or bf16) over
    a paged cache: token cu_nodes[s] + i of request s attends its context
    (positions 0 .. context_lens[s] - 1) and the drafted tokens j of its
    request (position context_lens[s] + j) whose bit j is set in row i of
    ``mask`` (int32 words, [nodes, words]); with mask None, tokens 0 .. i. No
    request has more than ``max_nodes`` (up to 256: a longer prompt takes several
    calls). Returns o [nodes, Hq, head_dim_v] of q's type; a token that attends
    nothing gets zeros. Rows that no request covers (padding behind the last one,
    say) are not written: an o made by the call is uninitialised there, so give
    one where such rows are read."""
    dev = q.device
    if (cap | block_size | max_nodes) >> 31:
        _ints(cap=cap, block_size=block_size, max_nodes=max_nodes)
    n, hq, dk, qt, qh = _heads(q, "q", dev)
    if hq != geom.n_q_heads or dk != geom.head_dim_k:
        raise ValueError(f"q has shape {tuple(q.shape)}, expected [nodes, {geom.n_q_heads}, {geom.head_dim_k}]")
    if q.dtype not in (torch.float16, torch.bfloat16):
        raise TypeError(f"q must be float16 or bfloat16, got {q.dtype}")
    if o is None:
        o = torch.empty((n, hq, geom.head_dim_v), dtype=q.dtype, device=dev)
    on, oc, od, ot, oh = _heads(o, "o", dev, True)
    if on != n or oc != hq or od != geom.head_dim_v or o.dtype != q.dtype:
        raise ValueError(f"o must be {q.dtype} [{n}, {hq}, {geom.head_dim_v}], got {o.dtype} {tuple(o.shape)}")
    n_seqs = context_lens.numel()
    geom.check_caches(k_cache, v_cache, cap, dev)
    words = 0
    if mask is not None:
        _dev(mask, "mask", dev)
        if mask.dtype != torch.int32 or mask.dim() != 2 or mask.shape[0] != n or not mask.is_contiguous():
            raise ValueError(f"mask must be contiguous int32 [{n}, words], got {mask.dtype} {tuple(mask.shape)}")
        words = mask.shape[1]
    size = geom.workspace_bytes(n_seqs, max_nodes, dev)
    ws = torch.empty(size, dtype=torch.uint8, device=dev) if size else None
    tree = KvTree(k_cache.data_ptr(), v_cache.data_ptr(), _table(block_table, n_seqs, dev),
                  _i32(context_lens, "context_lens", n_seqs, dev), _i32(cu_nodes, "cu_nodes", n_seqs + 1, dev),
                  mask.data_ptr() if mask is not None else None, q.data_ptr(), o.data_ptr(),
                  ws.data_ptr() if size else None, size,
                  block_table.stride(0) if n_seqs > 1 else block_table.shape[1],
                  qt, qh, ot, oh,
                  cap, block_table.shape[1], block_size, n_seqs, n, max_nodes, words, _TYPE[q.dtype])
    _call(dev, _load().cq_kv_tree_attend, geom.c, tree)
    return o
