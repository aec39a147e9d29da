"""A layer's other serving steps, beside the quantised products and the cache:
block norms on the residual stream, and the low-rank adapters of a batch's
requests. Thin bindings like the rest of the package: arguments are checked
and marshalled, all arithmetic runs in libcq's kernels.
"""
from __future__ import annotations

from typing import Optional, Sequence

import torch

from . import _capi
from ._capi import (CQ_GATE_PLAIN, CQ_GATE_SIGMOID, CQ_GATE_SILU, CQ_LORA_MAX_MATS, CQ_T_BF16, CQ_T_F16, CQ_T_F32, CQ_T_I8,
                    LoraDesc, NormDesc)
from .paged import _call, _dev, _i32, _ints, _stay, _type, _weight

_ACT = {None: CQ_GATE_PLAIN, "sigmoid": CQ_GATE_SIGMOID, "silu": CQ_GATE_SILU}
_load = _capi.load
_lora_bytes: dict = {}


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
    fp32 y. Outputs may be given; residual_out may be residual, out may be x."""
    dev = x.device
    xs = _matrix(x, "x", dev)
    n, d = x.shape
    if n >> 31:
        _ints(tokens=n)
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
    launch: ``outs[j][t] = ys[j][t] + scales[e] * b[j][e] @ (a[j][e] @ x[t])`` with
    e = adapters[s] the adapter of token t's request (-1: none; tokens of
    request s are cu_tokens[s] .. cu_tokens[s + 1] - 1, as cq_kv_plan gives them).
    x is [tokens, in] in fp32, the weights' type, or int8 with per-token scales
    x_scale (what the quantised products read); a[j] is [adapters, rank, in] and
    b[j] [adapters, out_j, rank], both fp16 or bf16; ys[j] is fp32 [tokens,
    out_j], up to 8 of them. ``ranks`` (int32 [adapters]): how many ranks of each
    adapter are in use. Without ``outs`` the ys are added to in place. Returns the
    outs. Rows that no request covers are not written. A request outside the
    tokens, and an adapter or rank outside its size, make a following
    cq_device_status raise."""
    dev = x.device
    xs = _matrix(x, "x", dev)
    m = len(ys)
    outs = ys if outs is None else outs
    if not m or not (len(a) == len(b) == len(outs) == m) or m > CQ_LORA_MAX_MATS:
        raise ValueError(f"ys, a, b (and outs) must be 1 to {CQ_LORA_MAX_MATS} tensors each, got {m}, {len(a)}, {len(b)}, {len(outs)}")
    n, n_in = x.shape
    wd = a[0].dtype
    if wd not in (torch.float16, torch.bfloat16):
        raise TypeError(f"a must be float16 or bfloat16, got {wd}")
    if a[0].dim() != 3:
        raise ValueError(f"a must be [adapters, rank, in], got {tuple(a[0].shape)}")
    n_adapters, rank = a[0].shape[:2]
    if x.dtype not in (torch.float32, torch.int8, wd):
        raise TypeError(f"x must be float32, int8 or the weights' {wd}, got {x.dtype}")
    n_seqs = adapters.numel()
    if (n | n_in | n_seqs | n_adapters) >> 31:
        _ints(tokens=n, n_in=n_in, requests=n_seqs, adapters=n_adapters)
    d = LoraDesc()
    for j in range(m):
        y, o, aj, bj = ys[j], outs[j], a[j], b[j]
        if y.dtype != torch.float32 or o.dtype != torch.float32:
            raise TypeError(f"ys and outs must be float32, got {y.dtype}, {o.dtype}")
        d.y_stride[j] = _matrix(y, "y", dev, None, o is y)
        if y.shape[0] != n:
            raise ValueError(f"y has {y.shape[0]} rows, x has {n}")
        width = y.shape[1]
        if width >> 31:
            _ints(out=width)
        d.y_out_stride[j] = d.y_stride[j] if o is y else _matrix(o, "out", dev, y.shape, True)
        for t, name, shape in ((aj, "a", (n_adapters, rank, n_in)), (bj, "b", (n_adapters, width, rank))):
            _dev(t, name, dev)
            if t.dtype != wd or t.shape != shape or not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous {wd} {list(shape)}, got {t.dtype} {list(t.shape)}")
        d.a[j], d.b[j], d.y[j], d.y_out[j], d.out[j] = aj.data_ptr(), bj.data_ptr(), y.data_ptr(), o.data_ptr(), width
    for t, name, size in ((scales, "scales", n_adapters), (x_scale, "x_scale", n)):
        if t is None:
            continue
        _dev(t, name, dev)
        if t.dtype != torch.float32 or t.numel() < size or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous float32 with at least {size} entries, got {t.dtype} {tuple(t.shape)}")
        setattr(d, name, t.data_ptr())
    if x.dtype == torch.int8 and x_scale is None:
        raise ValueError("int8 activations need x_scale")
    d.x, d.x_stride = x.data_ptr(), xs
    d.ranks = None if ranks is None else _i32(ranks, "ranks", n_adapters, dev)
    d.adapters, d.cu_tokens = _i32(adapters, "adapters", n_seqs, dev), _i32(cu_tokens, "cu_tokens", n_seqs + 1, dev)
    d.n_mats, d.n_tokens, d.n_seqs, d.n_adapters, d.in_, d.rank = m, n, n_seqs, n_adapters, n_in, rank
    d.w_dtype = CQ_T_F16 if wd == torch.float16 else CQ_T_BF16
    d.x_dtype = CQ_T_F32 if x.dtype == torch.float32 else CQ_T_I8 if x.dtype == torch.int8 else d.w_dtype
    key = (m, n, n_seqs, n_in, rank, d.x_dtype, dev.index)  # what the workspace goes by, besides the device
    size = _lora_bytes.get(key)
    if size is None:
        with (_stay if dev.index == torch.cuda.current_device() else torch.cuda.device(dev)):
            size = _load().cq_lora_workspace(d)
        if len(_lora_bytes) >= 4096:
            _lora_bytes.clear()
        _lora_bytes[key] = size
    ws = torch.empty(size, dtype=torch.uint8, device=dev)
    d.workspace, d.workspace_bytes = ws.data_ptr(), size
    _call(dev, _load().cq_lora_add, d)
    return list(outs)
