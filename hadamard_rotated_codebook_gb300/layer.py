"""A layer's other serving steps, beside the quantised products and the cache:
block norms on the residual stream, and the low-rank adapters of a batch's
requests. Thin bindings like the rest of the package: arguments are checked
and marshalled, all arithmetic runs in libcq's kernels.
"""
from __future__ import annotations

import struct
from typing import Optional, Sequence

import torch

from . import _capi
from ._capi import (CQ_GATE_PLAIN, CQ_GATE_SIGMOID, CQ_GATE_SILU, CQ_LORA_MAX_MATS, CQ_T_BF16, CQ_T_F16, CQ_T_F32, CQ_T_I8,
                    LoraDesc, NormDesc)
from .paged import _call, _dev, _i32, _ints, _stay, _type, _weight

_ACT = {None: CQ_GATE_PLAIN, "sigmoid": CQ_GATE_SIGMOID, "silu": CQ_GATE_SILU}
_load = _capi.load
_lora_bytes: dict = {}
_LORA_W = {torch.float16: CQ_T_F16, torch.bfloat16: CQ_T_BF16}
_LORA_X = {torch.float32: CQ_T_F32, torch.int8: CQ_T_I8}
_LORA_PACK = struct.Struct("@6P32P16q8iqPN8i").pack  # LoraDesc, field by field: its arrays cost a Python object an access


def _matrix(t: torch.Tensor, name: str, device, shape=None, out: bool = False) -> int:
    """[n, width] with contiguous rows (of an output, rows that do not share
    memory): the row stride."""
    _dev(t, name, device)
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be two-dimensional with contiguous rows, got {tuple(t.shape)} strides {t.stride()}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if out and t.shape[0] > 1 and t.stride(0) < t.shape[1]:
        raise ValueError(f"{name} overlaps itself: shape {tuple(t.shape)}, strides {t.stride()}")
    return t.stride(0)


def cq_block_norm(x: torch.Tensor, residual: Optional[torch.Tensor] = None, weight: Optional[torch.Tensor] = None, *,
                  post_norm: bool = False, branch_weight: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
                  gate_act: Optional[str] = None, branch_scale: float = 1.0, residual_scale: float = 1.0, eps: float = 1e-6,
                  weight_offset: float = 0.0, out_dtype: Optional[torch.dtype] = None, residual_out: Optional[torch.Tensor] = None,
                  out: Optional[torch.Tensor] = None, out_scale: Optional[torch.Tensor] = None):
    """A block's output x [tokens, width] (fp32, fp16 or bf16) onto the residual
    stream, and the norm the next block begins with, in one launch:
    ``z = norm(x) * (weight_offset + branch_weight)`` (x itself without
    ``post_norm``; branch_weight None: a norm's weight counts as 1, and x
    keeps its scale), ``r = residual_scale * residual + branch_scale *
    act(gate) * z``, ``y = norm(r) * (weight_offset + weight)``, with
    ``norm(v) = v / sqrt(mean(v^2) + eps)``. The gate is [tokens, width] or
    [tokens, 1] of x's type, gate_act None, "sigmoid" or "silu" (None: the gate
    itself); weights are fp32 [width]; the residual may have another type than x
    (None: zeros). Returns (r in the residual's type, y), or with out_dtype
    torch.int8 (r, codes, scales) with the bits of cq_act_quant_int8 over the
    fp32 y. Outputs may be given; residual_out and out
    may each be x, residual or a gate of full width itself. Outputs that share
    memory with each other, or in another way with an input, are refused."""
    dev = x.device
    xs = _matrix(x, "x", dev)
    n, d = x.shape
    if (n | d) >> 31:
        _ints(tokens=n, width=d)
    xt = _type(x, "x")
    rd, rs, rt, gs, gw = x.dtype, 0, xt, 0, 0
    if residual is not None:
        rd, rs, rt = residual.dtype, _matrix(residual, "residual", dev, x.shape), _type(residual, "residual")
    if gate is not None:
        gs, gw = _matrix(gate, "gate", dev), gate.shape[1]
        if gate.dtype != x.dtype or gate.shape[0] != n or gw not in (1, d):
            raise ValueError(f"gate must be {x.dtype} [{n}, {d}] or [{n}, 1], got {gate.dtype} {tuple(gate.shape)}")
    elif gate_act is not None:
        raise ValueError("gate_act without a gate")
    if gate_act not in _ACT:
        raise ValueError(f"gate_act must be None, 'sigmoid' or 'silu', got {gate_act!r}")
    if residual_out is None:
        residual_out = torch.empty((n, d), dtype=rd, device=dev)
    elif residual_out.dtype != rd:
        raise TypeError(f"residual_out must be {rd}, got {residual_out.dtype}")
    if out is None:
        out = torch.empty((n, d), dtype=out_dtype or x.dtype, device=dev)
    elif out_dtype is not None and out.dtype != out_dtype:
        raise TypeError(f"out must be {out_dtype}, got {out.dtype}")
    os, ss = _matrix(out, "out", dev, x.shape, True), _matrix(residual_out, "residual_out", dev, x.shape, True)
    coded = out.dtype == torch.int8
    if coded:
        if out_scale is None:
            out_scale = torch.empty(n, dtype=torch.float32, device=dev)
        _dev(out_scale, "out_scale", dev)
        if out_scale.dtype != torch.float32 or out_scale.shape != (n,) or not out_scale.is_contiguous():
            raise ValueError(f"out_scale must be contiguous float32 [{n}], got {out_scale.dtype} {tuple(out_scale.shape)}")
    rp, op, xp = residual_out.data_ptr(), out.data_ptr(), x.data_ptr()
    ip = residual.data_ptr() if residual is not None else None
    if n and (rp == ip and n > 1 and ss != rs or op == xp and (out.dtype != x.dtype or n > 1 and os != xs)):
        raise ValueError("an output shares memory with its input in another layout")
    desc = NormDesc(xp, ip, gate.data_ptr() if gate is not None else None, _weight(branch_weight, "branch_weight", d, dev),
                    _weight(weight, "weight", d, dev), rp, op, out_scale.data_ptr() if coded else None, xs, rs, gs, ss, os, xt, rt,
                    CQ_T_I8 if coded else _type(out, "out"), n, d, gw, _ACT[gate_act], post_norm, branch_scale, residual_scale, eps,
                    weight_offset)
    _call(dev, _load().cq_block_norm, desc)
    return (residual_out, out, out_scale) if coded else (residual_out, out)


def cq_lora_add(ys: Sequence[torch.Tensor], x: torch.Tensor, a: Sequence[torch.Tensor], b: Sequence[torch.Tensor],
                adapters: torch.Tensor, cu_tokens: torch.Tensor, *, scales: Optional[torch.Tensor] = None,
                ranks: Optional[torch.Tensor] = None, x_scale: Optional[torch.Tensor] = None,
                outs: Optional[Sequence[torch.Tensor]] = None) -> list:
    """Low-rank adapters of many requests beside shared projections, in one
    call (two kernels): ``outs[j][t] = ys[j][t] + scales[e] * b[j][e] @ (a[j][e] @ x[t])`` with
    e = adapters[s] the adapter of token t's request (-1: none; tokens of
    request s are cu_tokens[s] .. cu_tokens[s + 1] - 1, as cq_kv_plan gives them).
    x is [tokens, in] in fp32, the weights' type, or int8 with per-token scales
    x_scale (what the quantised products read); a[j] is [adapters, rank, in] and
    b[j] [adapters, out_j, rank], both fp16 or bf16; ys[j] is fp32 [tokens,
    out_j], up to 8 of them. ``ranks`` (int32 [adapters]): how many ranks of each
    adapter are in use. Without ``outs`` the ys are added to in place. Returns the
    outs. An output that shares memory with x, another output or a y (but its own,
    in place) is refused. Rows that no request covers are not written, but count
    where kernels are chosen: give a decode step's tensors no more rows than its
    graph needs. A request outside the tokens, and an adapter or rank outside its
    size, make a following cq_device_status raise."""
    dev = x.device
    m = len(ys)
    outs = ys if outs is None else outs
    if not m or not (len(a) == len(b) == len(outs) == m) or m > CQ_LORA_MAX_MATS:
        raise ValueError(f"ys, a, b (and outs) must be 1 to {CQ_LORA_MAX_MATS} tensors each, got {m}, {len(a)}, {len(b)}, {len(outs)}")
    xs = _matrix(x, "x", dev)
    n, n_in = x.shape
    wd, xd, at, index = a[0].dtype, x.dtype, a[0].shape, dev.index
    wt = _LORA_W.get(wd)
    if wt is None:
        raise TypeError(f"a must be float16 or bfloat16, got {wd}")
    xt = wt if xd == wd else _LORA_X.get(xd)
    if xt is None:
        raise TypeError(f"x must be float32, int8 or the weights' {wd}, got {xd}")
    if len(at) != 3:
        raise ValueError(f"a must be [adapters, rank, in], got {tuple(at)}")
    n_adapters, rank, _ = at
    n_seqs = adapters.numel()
    if (n | n_in | n_seqs | n_adapters | rank) >> 31:
        _ints(tokens=n, n_in=n_in, requests=n_seqs, adapters=n_adapters, rank=rank)
    a_ptr, b_ptr, y_ptr, o_ptr, y_stride, o_stride, widths = [0] * 8, [0] * 8, [0] * 8, [0] * 8, [0] * 8, [0] * 8, [0] * 8
    for j in range(m):
        y, o, aj, bj = ys[j], outs[j], a[j], b[j]
        try:  # what a good call passes in a few looks
            rows, width = y.shape
            st = y.stride()
            good = (y.dtype is torch.float32 and rows == n and (st[1] == 1 or width <= 1) and y.get_device() == index
                    and aj.dtype is wd and bj.dtype is wd and aj.shape == (n_adapters, rank, n_in) and bj.shape == (n_adapters, width, rank)
                    and aj.is_contiguous() and bj.is_contiguous() and aj.get_device() == index and bj.get_device() == index)
            so = st[0]
            if o is y:
                good = good and (n <= 1 or so >= width)
            else:
                su = o.stride()
                so = su[0]
                good = (good and o.dtype is torch.float32 and o.shape == y.shape and (su[1] == 1 or width <= 1) and (n <= 1 or so >= width)
                        and o.get_device() == index)
        except (AttributeError, ValueError, IndexError):
            good = False
        if not good:
            _lora_complain(y, o, aj, bj, dev, wd, n, (n_adapters, rank, n_in))
        if width >> 31:
            _ints(out=width)
        a_ptr[j], b_ptr[j], y_ptr[j], widths[j], y_stride[j], o_stride[j] = aj.data_ptr(), bj.data_ptr(), y.data_ptr(), width, st[0], so
        o_ptr[j] = y_ptr[j] if o is y else o.data_ptr()
    for t, name, size in ((scales, "scales", n_adapters), (x_scale, "x_scale", n)):
        if t is None:
            continue
        _dev(t, name, dev)
        if t.dtype != torch.float32 or t.numel() < size or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous float32 with at least {size} entries, got {t.dtype} {tuple(t.shape)}")
    if xt == CQ_T_I8 and x_scale is None:
        raise ValueError("int8 activations need x_scale")
    key = (m, n, n_seqs, n_in, rank, xt, index)  # what the workspace goes by, besides the device
    size = _lora_bytes.get(key)

    def desc(ws, size):
        return LoraDesc.from_buffer_copy(_LORA_PACK(
            x.data_ptr(), 0 if x_scale is None else x_scale.data_ptr(), 0 if scales is None else scales.data_ptr(),
            0 if ranks is None else _i32(ranks, "ranks", n_adapters, dev), _i32(adapters, "adapters", n_seqs, dev),
            _i32(cu_tokens, "cu_tokens", n_seqs + 1, dev), *a_ptr, *b_ptr, *y_ptr, *o_ptr, *y_stride, *o_stride, *widths, xs, ws, size,
            m, n, n_seqs, n_adapters, n_in, rank, xt, wt))

    if size is None:
        with (_stay if index == torch.cuda.current_device() else torch.cuda.device(dev)):
            size = _load().cq_lora_workspace(desc(0, 0))
        if size:  # (none: nothing to do, or the library refuses something that the key may not hold)
            if len(_lora_bytes) >= 4096:
                _lora_bytes.clear()
            _lora_bytes[key] = size
    ws = torch.empty(size, dtype=torch.uint8, device=dev)
    _call(dev, _load().cq_lora_add, desc(ws.data_ptr(), size))
    return list(outs)


def _lora_complain(y, o, aj, bj, dev, wd, n, a_shape) -> None:
    """Says what is wrong with a matrix's tensors."""
    _matrix(y, "y", dev, None, o is y)
    _matrix(o, "out", dev, y.shape, True)
    if y.dtype != torch.float32 or o.dtype != torch.float32:
        raise TypeError(f"ys and outs must be float32, got {y.dtype}, {o.dtype}")
    if y.shape[0] != n:
        raise ValueError(f"y has {y.shape[0]} rows, x has {n}")
    for t, name, shape in ((aj, "a", a_shape), (bj, "b", (a_shape[0], y.shape[1], a_shape[1]))):
        _dev(t, name, dev)
        if t.dtype != wd or t.shape != shape or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous {wd} {list(shape)}, got {t.dtype} {list(t.shape)}")
    raise ValueError("ys, outs, a and b do not belong together")
