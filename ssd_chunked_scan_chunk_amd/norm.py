"""The norm over groups of channels of every row, with an activation or a gate.

As in ``layer``, x and gate may be views of wider rows: the channels have to be
dense, the strides between rows and batches are free.
"""
from __future__ import annotations

import torch

from . import _L, _dtype_code, _lib
from .layer import _at, _bytes, _enqueue, _need, _rows, _same, _seqlens, _workspace


def _norm_check(x, groups, weight, bias, gate, eps, center, silu, gate_first):
    """The desc of a norm of x [rows, channels] or [batch, seqlen, channels]."""
    if not isinstance(x, torch.Tensor) or x.dim() not in (2, 3):
        raise ValueError("x must be a tensor [batch, channels] or [batch, seqlen, channels]")
    code, dev, shape = _dtype_code(x), x.device, x.shape
    C = shape[-1]
    sx = _rows("x", x, shape, 1, x.dtype, dev)
    sz = _rows("gate", gate, shape, 1, x.dtype, dev) if gate is not None else (0, 0, 0)
    if gate_first and gate is None:
        raise ValueError("gate_first needs a gate")
    _same("weight", weight, (C,), torch.float32, dev)
    _same("bias", bias, (C,), torch.float32, dev)
    form = (float(eps), code, 1 if center else 0, 1 if silu else 0, 1 if gate_first else 0, 0)
    if len(shape) == 3:
        return _lib.GroupNormDesc(shape[0], shape[1], C, int(groups), sx[0], sx[1], sz[0], sz[1], *form)
    return _lib.GroupNormDesc(1, shape[0], C, int(groups), 0, sx[0], 0, sz[0], *form)


def _norm_lens(seqlens, x):
    if seqlens is not None and x.dim() != 3:
        raise ValueError("seqlens needs x [batch, seqlen, channels]")
    _seqlens(seqlens, x.shape[0], x.device)


def group_norm_fwd(x, groups, weight=None, bias=None, gate=None, eps=1e-5, center=True, silu=True, gate_first=False,
                   seqlens=None, y=None):
    """Norm over each row's groups of consecutive channels: n = (x - mean) /
    sqrt(var + eps) (mean 0 and var the mean square unless center), p = weight n + bias.

    Returns act(p) without a gate, p act(gate) with one, and with gate_first p of
    x act(gate) in the place of x; act is SiLU, or nothing if not silu.  x and gate
    [Bz,L,C], or [Bz,C] for a token (bf16 or f32, rows dense), weight and bias [C] f32, up
    to 16384 channels in a group.  seqlens [Bz] int32 on the GPU: sequence b has that
    many rows; later ones are not read and y is 0 there."""
    d = _norm_check(x, groups, weight, bias, gate, eps, center, silu, gate_first)
    _norm_lens(seqlens, x)
    _same("y", y, x.shape, x.dtype, x.device)
    if y is None:
        y = x.new_empty(x.shape)
    _enqueue(x.device, _L().ssd_group_norm_fwd, d, _at(x), _at(weight), _at(bias), _at(gate), _at(seqlens), _at(y))
    return y


def _norm_bytes(d):
    return _bytes("ssd_group_norm_bwd_workspace_bytes", _lib.GroupNormDesc, d.batch, d.seqlen, d.channels, d.groups,
                  0, 0, 0, 0, 0.0, d.dtype, 0, 0, 0, 0)


def group_norm_bwd_workspace_bytes(x, groups) -> int:
    return _norm_bytes(_norm_check(x, groups, None, None, None, 0.0, True, True, False))


def group_norm_bwd(x, groups, dy, weight=None, bias=None, gate=None, eps=1e-5, center=True, silu=True, gate_first=False,
                   seqlens=None, workspace=None):
    """Gradients of group_norm_fwd for upstream dy (x's shape, contiguous).

    Returns a dict with dx and dgate (x's dtype), dweight and dbias (f32); dgate,
    dweight and dbias are None without their input, and without weight and bias no
    workspace is used."""
    d = _norm_check(x, groups, weight, bias, gate, eps, center, silu, gate_first)
    _need("dy", dy)
    _same("dy", dy, x.shape, x.dtype, x.device)
    _norm_lens(seqlens, x)
    if workspace is None and weight is None and bias is None:
        wsz = 0
    else:
        workspace, wsz = _workspace(workspace, _norm_bytes(d), x.device)
    g = {"dx": x.new_empty(x.shape), "dgate": x.new_empty(x.shape) if gate is not None else None,
         "dweight": torch.empty_like(weight) if weight is not None else None,
         "dbias": torch.empty_like(bias) if bias is not None else None}
    _enqueue(x.device, _L().ssd_group_norm_bwd, d, _at(x), _at(weight), _at(bias), _at(gate), _at(seqlens), _at(dy),
             *map(_at, g.values()), _at(workspace), wsz)
    return g
