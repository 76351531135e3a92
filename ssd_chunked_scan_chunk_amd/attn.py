"""Linear attention with a constant decay for each head: prompts, gradients and
single tokens.

As in ``layer``, q, k and v may be views of wider rows (parts of one projection):
each step's [heads, dim] has to be dense, the strides between steps and batches
are free.  States, upstream gradients and log_decay are contiguous.
"""
from __future__ import annotations

import torch

from . import _L, _dtype_code, _lib
from .layer import _at, _bytes, _enqueue, _need, _rows, _same, _seqlens, _workspace


def _attn_check(q, k, v, log_decay, scale, lead):
    """(desc, the states' shape) of attention over q [*lead, heads, key]."""
    if not isinstance(q, torch.Tensor) or q.dim() != lead + 2:
        raise ValueError("q must be a %d-D tensor [batch, %sheads, key]" % (lead + 2, "seqlen, " if lead == 2 else ""))
    for name, t in (("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor) or t.dim() != lead + 2:
            raise ValueError("%s must be a %d-D tensor [batch, %skv_heads, %s]"
                             % (name, lead + 2, "seqlen, " if lead == 2 else "", "key" if name == "k" else "value"))
    code, dt, dev, shape = _dtype_code(q), q.dtype, q.device, q.shape
    rows, (H, Dk), K, Dv = shape[:lead], shape[lead:], k.shape[lead], v.shape[-1]
    sq = _rows("q", q, shape, 2, dt, dev)
    sk = _rows("k", k, rows + (K, Dk), 2, dt, dev)
    sv = _rows("v", v, rows + (K, Dv), 2, dt, dev)
    _need("log_decay", log_decay)
    _same("log_decay", log_decay, (H,), torch.float32, dev)
    scale = Dk ** -0.5 if scale is None and Dk > 0 else 1.0 if scale is None else float(scale)
    if lead == 2:
        d = _lib.LinearAttnDesc(shape[0], shape[1], H, K, Dk, Dv, sq[0], sq[1], sk[0], sk[1], sv[0], sv[1], scale, code)
    else:
        d = _lib.LinearAttnDesc(shape[0], 1, H, K, Dk, Dv, sq[0], 0, sk[0], 0, sv[0], 0, scale, code)
    return d, (shape[0], H, Dv, Dk)


def _attn_bytes(query, d):
    return _bytes(query, _lib.LinearAttnDesc, d.batch, d.seqlen, d.nheads, d.kv_heads, d.key_dim, d.value_dim,
                  *(0,) * 6, 1.0, d.dtype)


def linear_attn_fwd_workspace_bytes(q, k, v, log_decay) -> int:
    return _attn_bytes("ssd_linear_attn_fwd_workspace_bytes", _attn_check(q, k, v, log_decay, None, 2)[0])


def linear_attn_fwd(q, k, v, log_decay, scale=None, initial_state=None, seqlens=None, return_final_state=False, y=None,
                    final_state=None, workspace=None):
    """Attention without a softmax whose past decays: S = e^log_decay S + v k^T,
    y = scale S q for every head, in chunks.

    q [Bz,L,H,Dk], k [Bz,L,K,Dk], v [Bz,L,K,Dv] (bf16 or f32; the [heads, dim] of a step
    dense; K divides H, head h reads key and value head h*K//H; dims up to 256),
    log_decay [H] f32: constants, normally below 0, that get no gradient.  scale: Dk^-0.5 if None.
    initial_state [Bz,H,Dv,Dk] f32 (None: zero).  seqlens [Bz] int32 on the GPU:
    sequence b has that many steps; later rows are not read, y is 0 there and the
    final state is the one after the last step.  Returns (y [Bz,L,H,Dv],
    final_state or None); linear_attn_step continues from the state."""
    d, state = _attn_check(q, k, v, log_decay, scale, 2)
    dev, out = q.device, (d.batch, d.seqlen, d.nheads, d.value_dim)
    _same("initial_state", initial_state, state, torch.float32, dev)
    _same("final_state", final_state, state, torch.float32, dev)
    _same("y", y, out, q.dtype, dev)
    _seqlens(seqlens, d.batch, dev)
    if y is None:
        y = q.new_empty(out)
    if final_state is None and return_final_state:
        final_state = log_decay.new_empty(state)
    workspace, wsz = _workspace(workspace, _attn_bytes("ssd_linear_attn_fwd_workspace_bytes", d), dev)
    _enqueue(dev, _L().ssd_linear_attn_fwd, d, _at(q), _at(k), _at(v), _at(log_decay), _at(initial_state), _at(seqlens),
             _at(y), _at(final_state), _at(workspace), wsz)
    return y, final_state


def linear_attn_bwd_workspace_bytes(q, k, v, log_decay) -> int:
    return _attn_bytes("ssd_linear_attn_bwd_workspace_bytes", _attn_check(q, k, v, log_decay, None, 2)[0])


def linear_attn_bwd(q, k, v, log_decay, dy, scale=None, initial_state=None, dfinal_state=None, seqlens=None,
                    return_dinitial_state=False, workspace=None):
    """Gradients of linear_attn_fwd for upstream dy [Bz,L,H,Dv] and dfinal_state
    (None: zero).

    Returns a dict with dq, dk, dv (q's dtype; dk and dv summed over the heads that
    share a key and value head) and dinitial_state (f32; None unless requested)."""
    d, state = _attn_check(q, k, v, log_decay, scale, 2)
    dev = q.device
    _need("dy", dy)
    _same("dy", dy, (d.batch, d.seqlen, d.nheads, d.value_dim), q.dtype, dev)
    _same("initial_state", initial_state, state, torch.float32, dev)
    _same("dfinal_state", dfinal_state, state, torch.float32, dev)
    _seqlens(seqlens, d.batch, dev)
    workspace, wsz = _workspace(workspace, _attn_bytes("ssd_linear_attn_bwd_workspace_bytes", d), dev)
    g = {"dq": q.new_empty(q.shape), "dk": q.new_empty(k.shape), "dv": q.new_empty(v.shape),
         "dinitial_state": log_decay.new_empty(state) if return_dinitial_state else None}
    _enqueue(dev, _L().ssd_linear_attn_bwd, d, _at(q), _at(k), _at(v), _at(log_decay), _at(initial_state), _at(seqlens),
             _at(dy), _at(dfinal_state), *map(_at, g.values()), _at(workspace), wsz)
    return g


def linear_attn_step(state, q, k, v, log_decay, scale=None, y=None):
    """One token: state [Bz,H,Dv,Dk] f32 is updated in place.  q [Bz,H,Dk], k [Bz,K,Dk]
    and v [Bz,K,Dv], each request's [heads, dim] dense.  Returns y [Bz,H,Dv]."""
    d, shape = _attn_check(q, k, v, log_decay, scale, 1)
    _need("state", state)
    _same("state", state, shape, torch.float32, q.device)
    _same("y", y, shape[:3], q.dtype, q.device)
    if y is None:
        y = q.new_empty(shape[:3])
    _enqueue(q.device, _L().ssd_linear_attn_step, d, _at(state), _at(q), _at(k), _at(v), _at(log_decay), _at(y))
    return y
