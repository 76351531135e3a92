"""The operators around the chunked scan: the short causal convolution and the
scan with one decay per channel and state.

Like the rest of the package these only check arguments, allocate outputs and
workspace and pass pointers to libssd.so.  Inputs that a layer cuts out of a
projection's rows (x; u, delta, gate, B and C) may be views: their rows have to be
dense, the strides between rows and batches are free.  Parameters, states and
upstream gradients are contiguous.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _L, _check, _check_bytes, _dtype_code, _lib

_P = ctypes.c_void_p * 3


def _same(name, t, shape, dtype, device):
    """_check, with the usual outcome decided first: these calls take tens of
    microseconds for a token, so their checks have to be quick."""
    if t is None or (t.__class__ is torch.Tensor and t.shape == shape and t.dtype is dtype and t.device == device
                     and t.is_contiguous()):
        return
    _check(name, t, shape, dtype, device)


def _rows(name, t, shape, dense, dtype, device):
    """Check a tensor of ``shape`` whose last ``dense`` dimensions are dense and
    return the strides of the leading ones."""
    if t.__class__ is torch.Tensor and t.shape == shape and t.dtype is dtype and t.device == device:
        strides = t.stride()   # the usual outcome first, as in _same
        if strides[-1] == 1 and (dense == 1 or shape[-2] == 1 or strides[-2] == shape[-1]):
            return strides
    if not isinstance(t, torch.Tensor):
        raise ValueError("%s is required" % name)
    if t.shape != shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if t.dtype is not dtype:
        raise ValueError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    strides = t.stride()
    if strides[-1] != 1 or dense > 1:   # a dimension of size 1 may have any stride
        want = 1
        for k in range(1, dense + 1):
            if strides[-k] != want and shape[-k] > 1:
                raise ValueError("the rows of %s must be contiguous" % name)
            want *= shape[-k]
    return strides


def _need(name, t):
    if t is None:
        raise ValueError("%s is required" % name)


def _at(t):
    return None if t is None else t.data_ptr()


def _seqlens(seqlens, Bz, device):
    if seqlens is not None:
        if not isinstance(seqlens, torch.Tensor):
            raise TypeError("seqlens must be a torch.Tensor on the GPU")
        _same("seqlens", seqlens, (Bz,), torch.int32, device)


@functools.lru_cache(maxsize=1024)
def _bytes(query, kind, *sizes):
    """The workspace an entry point asks for, by the sizes that decide it."""
    n = ctypes.c_size_t()
    _lib.check(getattr(_L(), query)(kind(*sizes), n))
    return n.value


def _workspace(workspace, nbytes, device):
    if workspace is None:
        return (torch.empty(nbytes, dtype=torch.uint8, device=device), nbytes) if nbytes > 0 else (None, 0)
    _check_bytes("workspace", workspace, nbytes, device)
    return workspace, workspace.numel() * workspace.element_size()


def _enqueue(device, fn, *args):
    """Call an entry point with the current stream of the tensors' device, that
    device being the current one."""
    if device.type != "cuda":
        raise ValueError("tensors must live on the GPU")
    stream = torch._C._cuda_getCurrentRawStream(device.index)
    if device.index == torch._C._cuda_getDevice():
        status = fn(*args, stream)
    else:
        with torch.cuda.device(device):
            status = fn(*args, stream)
    if status:
        _lib.check(status)


# ---- short causal convolution ------------------------------------------------------

def _conv_check(x, weight, bias, silu, pieces, lead):
    """(desc, pieces) of a convolution of x [*lead, channels]."""
    if not isinstance(x, torch.Tensor) or x.dim() != lead + 1:
        raise ValueError("x must be a %d-D tensor [batch, %schannels]" % (lead + 1, "seqlen, " if lead == 2 else ""))
    code, shape, dev = _dtype_code(x), x.shape, x.device
    C = shape[-1]
    strides = _rows("x", x, shape, 1, x.dtype, dev)
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be a 2-D tensor [channels, width]")
    W = weight.shape[1]
    _same("weight", weight, (C, W), torch.float32, dev)
    _same("bias", bias, (C,), torch.float32, dev)
    if pieces is None:
        given, three = (C,), (C, 0, 0)
    else:
        given = tuple(int(w) for w in pieces)
        if not 1 <= len(given) <= 3 or min(given) < 1 or sum(given) != C:
            raise ValueError("pieces must be one to three widths that add up to the %d channels, got %s" % (C, given))
        three = given + (0,) * (3 - len(given))
    L, xr = (shape[1], strides[1]) if lead == 2 else (1, 0)
    return _lib.ConvDesc(shape[0], L, C, W, strides[0], xr, three, len(given), code, 1 if silu else 0, 0), given


def _conv_outputs(x, given, pieces, y):
    """The y pieces to write, as a tuple, and what the caller gets back."""
    lead = tuple(x.shape[:-1])
    if y is None:
        ys = tuple([x.new_empty(lead + (w,)) for w in given])
        return ys, ys[0] if pieces is None else ys
    ys = (y,) if pieces is None else tuple(y)
    _conv_given("y", ys, lead, given, x)
    return ys, y


def _conv_given(name, ts, lead, given, x):
    if len(ts) != len(given):
        raise ValueError("%s has %d pieces, expected %d" % (name, len(ts), len(given)))
    for i, (t, w) in enumerate(zip(ts, given)):
        label = name if len(given) == 1 else "%s[%d]" % (name, i)
        _need(label, t)
        _same(label, t, lead + (w,), x.dtype, x.device)


def short_conv_fwd(x, weight, bias=None, initial_window=None, seqlens=None, silu=True, pieces=None,
                   return_final_window=False, y=None, final_window=None):
    """Causal convolution of every channel along the sequence, then SiLU.

    x [Bz,L,C] (bf16 or f32, rows dense), weight [C,W] f32 with W 2 to 4, bias
    [C] f32, initial_window [Bz,W-1,C] in x's dtype: the inputs before the first
    step (None: zeros).  seqlens [Bz] int32 on the GPU: sequence b has that many
    steps; later rows of x are not read and those of y are 0.  pieces: widths
    that add up to C; y is then a tuple of contiguous [Bz,L,width] tensors (X,
    B and C for chunk_scan_fwd, after a view).  Returns (y, final_window or None):
    the window [Bz,W-1,C] continues the sequence here or in short_conv_step."""
    d, given = _conv_check(x, weight, bias, silu, pieces, 2)
    dev, Bz, window = x.device, d.batch, (d.batch, d.width - 1, d.channels)
    _same("initial_window", initial_window, window, x.dtype, dev)
    _same("final_window", final_window, window, x.dtype, dev)
    _seqlens(seqlens, Bz, dev)
    ys, back = _conv_outputs(x, given, pieces, y)
    if final_window is None and return_final_window:
        final_window = x.new_empty(window if d.width > 0 else (Bz, 0, d.channels))
    _enqueue(dev, _L().ssd_short_conv_fwd, d, _at(x), _at(weight), _at(bias), _at(initial_window), _at(seqlens),
             _P(*map(_at, ys)), _at(final_window))
    return back, final_window


def short_conv_bwd_workspace_bytes(x, weight, pieces=None) -> int:
    return _conv_bwd_bytes(_conv_check(x, weight, None, True, pieces, 2)[0])


def _conv_bwd_bytes(d):
    return _bytes("ssd_short_conv_bwd_workspace_bytes", _lib.ConvDesc, d.batch, d.seqlen, d.channels, d.width, 0, 0,
                  tuple(d.piece), d.npieces, d.dtype, 1, 0)


def short_conv_bwd(x, weight, dy, bias=None, initial_window=None, dfinal_window=None, seqlens=None, silu=True,
                   return_dinitial_window=False, workspace=None):
    """Gradients of short_conv_fwd for upstream dy (one contiguous tensor, or a
    tuple of the forward's pieces) and dfinal_window (None: zero).

    Returns a dict with dx [Bz,L,C] and dinitial_window (x's dtype; None unless
    requested), dweight and dbias (f32; dbias None without a bias)."""
    several = isinstance(dy, (tuple, list))
    if not several:
        _need("dy", dy)
    dys = tuple(dy) if several else (dy,)
    if several and not all(isinstance(t, torch.Tensor) and t.dim() == 3 for t in dys):
        raise ValueError("the pieces of dy must be 3-D tensors")
    d, given = _conv_check(x, weight, bias, silu, [t.shape[2] for t in dys] if several else None, 2)
    Bz, L, C = x.shape
    W = weight.shape[1]
    _conv_given("dy", dys, (Bz, L), given, x)
    _same("initial_window", initial_window, (Bz, W - 1, C), x.dtype, x.device)
    _same("dfinal_window", dfinal_window, (Bz, W - 1, C), x.dtype, x.device)
    _seqlens(seqlens, Bz, x.device)
    workspace, wsz = _workspace(workspace, _conv_bwd_bytes(d), x.device)
    dx = x.new_empty((Bz, L, C))
    dweight = torch.empty_like(weight)
    dbias = torch.empty_like(bias) if bias is not None else None
    dwin = x.new_empty((Bz, W - 1, C)) if return_dinitial_window else None
    _enqueue(x.device, _L().ssd_short_conv_bwd, d, _at(x), _at(weight), _at(bias), _at(initial_window), _at(seqlens),
             _P(*map(_at, dys)), _at(dfinal_window), _at(dx), _at(dweight), _at(dbias), _at(dwin), _at(workspace), wsz)
    return {"dx": dx, "dweight": dweight, "dbias": dbias, "dinitial_window": dwin}


def short_conv_step(window, x, weight, bias=None, silu=True, pieces=None, y=None):
    """One token: x [Bz,C] (rows dense) against window [Bz,W-1,C], which is
    updated in place.  Returns y [Bz,C], or its pieces as a tuple."""
    d, given = _conv_check(x, weight, bias, silu, pieces, 1)
    _need("window", window)
    dev = x.device
    _same("window", window, (d.batch, d.width - 1, d.channels), x.dtype, dev)
    ys, back = _conv_outputs(x, given, pieces, y)
    _enqueue(dev, _L().ssd_short_conv_step, d, _at(window), _at(x), _at(weight), _at(bias), _P(*map(_at, ys)))
    return back


# ---- scan with one decay per channel and state -----------------------------------------

def _chan_check(u, delta, A, B, C, skip, gate, delta_bias, softplus, lead):
    """The desc of a scan of u [*lead, channels]; everything but the states checked."""
    if not isinstance(u, torch.Tensor) or u.dim() != lead + 1:
        raise ValueError("u must be a %d-D tensor [batch, %schannels]" % (lead + 1, "seqlen, " if lead == 2 else ""))
    code, dt, dev, D = _dtype_code(u), u.dtype, u.device, u.shape[-1]
    if not isinstance(A, torch.Tensor) or A.dim() != 2:
        raise ValueError("A must be a 2-D tensor [channels, dstate]")
    _same("A", A, (D, A.shape[1]), torch.float32, dev)
    if not isinstance(B, torch.Tensor) or B.dim() != lead + 2:
        raise ValueError("B must be a %d-D tensor [batch, %sngroups, dstate]"
                         % (lead + 2, "seqlen, " if lead == 2 else ""))
    G, N, rows = B.shape[-2], A.shape[1], tuple(u.shape[:-1])
    su = _rows("u", u, u.shape, 1, dt, dev)
    sd = _rows("delta", delta, u.shape, 1, dt, dev)
    sz = _rows("gate", gate, u.shape, 1, dt, dev) if gate is not None else (0, 0)
    sB = _rows("B", B, rows + (G, N), 2, dt, dev)
    sC = _rows("C", C, rows + (G, N), 2, dt, dev)
    _same("skip", skip, (D,), torch.float32, dev)
    _same("delta_bias", delta_bias, (D,), torch.float32, dev)
    if lead == 2:
        return _lib.ChannelDesc(rows[0], rows[1], D, N, G, su[0], su[1], sd[0], sd[1], sz[0], sz[1], sB[0], sB[1],
                                sC[0], sC[1], code, 1 if softplus else 0)
    return _lib.ChannelDesc(rows[0], 1, D, N, G, su[0], 0, sd[0], 0, sz[0], 0, sB[0], 0, sC[0], 0, code,
                            1 if softplus else 0)


def _chan_bytes(query, d):
    return _bytes(query, _lib.ChannelDesc, d.batch, d.seqlen, d.channels, d.dstate, d.ngroups, *(0,) * 10, d.dtype, 1)


def channel_scan_fwd_workspace_bytes(u, delta, A, B, C) -> int:
    return _chan_bytes("ssd_channel_scan_fwd_workspace_bytes", _chan_check(u, delta, A, B, C, None, None, None, True, 2))


def channel_scan_fwd(u, delta, A, B, C, skip=None, gate=None, delta_bias=None, softplus=False, initial_state=None,
                     seqlens=None, return_final_state=False, y=None, final_state=None, workspace=None):
    """Scan h = exp(dt A) h + dt u B, y = (h C + skip u) silu(gate), with a decay
    of its own for every channel and state; dt = delta + delta_bias, through a
    softplus if asked.

    u, delta, gate [Bz,L,D] and B, C [Bz,L,G,N] (bf16 or f32, rows dense; N up to
    64, channel c reads group c*G//D), A [D,N], skip, delta_bias [D] f32,
    initial_state [Bz,D,N] f32 (None: zero).  seqlens [Bz] int32 on the GPU:
    sequence b has that many steps; later rows are not read, y is 0 there and the
    final state is the one after the last step.  With softplus a step of delta =
    -inf leaves the state as it is.  Returns (y, final_state or None); channel_step
    continues from the state."""
    d = _chan_check(u, delta, A, B, C, skip, gate, delta_bias, softplus, 2)
    dev, state = u.device, (u.shape[0], u.shape[2], A.shape[1])
    _same("initial_state", initial_state, state, torch.float32, dev)
    _same("final_state", final_state, state, torch.float32, dev)
    _same("y", y, u.shape, u.dtype, dev)
    _seqlens(seqlens, u.shape[0], dev)
    if y is None:
        y = torch.empty_like(u, memory_format=torch.contiguous_format)
    if final_state is None and return_final_state:
        final_state = A.new_empty(state)
    workspace, wsz = _workspace(workspace, _chan_bytes("ssd_channel_scan_fwd_workspace_bytes", d), dev)
    _enqueue(dev, _L().ssd_channel_scan_fwd, d, _at(u), _at(delta), _at(A), _at(B), _at(C), _at(skip), _at(gate),
             _at(delta_bias), _at(initial_state), _at(seqlens), _at(y), _at(final_state), _at(workspace), wsz)
    return y, final_state


def channel_scan_bwd_workspace_bytes(u, delta, A, B, C) -> int:
    return _chan_bytes("ssd_channel_scan_bwd_workspace_bytes", _chan_check(u, delta, A, B, C, None, None, None, True, 2))


def channel_scan_bwd(u, delta, A, B, C, dy, skip=None, gate=None, delta_bias=None, softplus=False,
                     initial_state=None, dfinal_state=None, seqlens=None, return_dinitial_state=False,
                     workspace=None):
    """Gradients of channel_scan_fwd for upstream dy [Bz,L,D] and dfinal_state
    (None: zero).

    Returns a dict with du, ddelta, dB, dC and dgate (u's dtype), dA, dskip and
    ddelta_bias (f32; dgate, dskip, ddelta_bias None without their input) and
    dinitial_state (f32; None unless requested)."""
    d = _chan_check(u, delta, A, B, C, skip, gate, delta_bias, softplus, 2)
    dev, dt, f32, state = u.device, u.dtype, torch.float32, (u.shape[0], u.shape[2], A.shape[1])
    _need("dy", dy)
    _same("dy", dy, u.shape, dt, dev)
    _same("initial_state", initial_state, state, f32, dev)
    _same("dfinal_state", dfinal_state, state, f32, dev)
    _seqlens(seqlens, u.shape[0], dev)
    workspace, wsz = _workspace(workspace, _chan_bytes("ssd_channel_scan_bwd_workspace_bytes", d), dev)
    rows, cols = u.new_empty, A.new_empty   # in the type of the inputs and of the parameters
    g = {"du": rows(u.shape), "ddelta": rows(u.shape), "dgate": rows(u.shape) if gate is not None else None,
         "dB": rows(B.shape), "dC": rows(B.shape), "dA": cols(A.shape),
         "dskip": cols(A.shape[:1]) if skip is not None else None,
         "ddelta_bias": cols(A.shape[:1]) if delta_bias is not None else None,
         "dinitial_state": cols(state) if return_dinitial_state else None}
    _enqueue(dev, _L().ssd_channel_scan_bwd, d, _at(u), _at(delta), _at(A), _at(B), _at(C), _at(skip), _at(gate),
             _at(delta_bias), _at(initial_state), _at(seqlens), _at(dy), _at(dfinal_state),
             _lib.ChannelGrads(*map(_at, g.values())), _at(workspace), wsz)
    return g


def channel_step(state, u, delta, A, B, C, skip=None, gate=None, delta_bias=None, softplus=False, y=None):
    """One token: state [Bz,D,N] f32 is updated in place.  u, delta, gate [Bz,D] and
    B, C [Bz,G,N] with dense rows.  Returns y [Bz,D]."""
    d = _chan_check(u, delta, A, B, C, skip, gate, delta_bias, softplus, 1)
    _need("state", state)
    _same("state", state, (u.shape[0], u.shape[1], A.shape[1]), torch.float32, u.device)
    _same("y", y, u.shape, u.dtype, u.device)
    if y is None:
        y = torch.empty_like(u, memory_format=torch.contiguous_format)
    _enqueue(u.device, _L().ssd_channel_step, d, _at(state), _at(u), _at(delta), _at(A), _at(B), _at(C), _at(skip),
             _at(gate), _at(delta_bias), _at(y))
    return y
