"""Plain 64-bit numpy forms of the operators around the chunked scan, step by
step from their definitions, each with the magnitudes that bound its rounding:
the same sums over absolute values.  Tolerances of the GPU tests are counts of
fp32 roundings (2^-24 of a magnitude each) plus half a step of the output's
type.

A hardware exponential or reciprocal is off by at most 2 roundings here (1 ulp
each), its argument by one more, which moves an exponential by |argument|
roundings."""
import numpy as np

U = 2.0 ** -24                       # half a step of fp32, relative
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}   # half a step of an output


def sigmoid(v):
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0, e) / (1.0 + e)


def lengths(seqlens, Bz, L):
    return [L] * Bz if seqlens is None else [min(max(int(n), 0), L) for n in seqlens]


def conv(x, weight, bias, win, seqlens, silu, dy=None, dwin=None, walk=32):
    """Everything of the convolution: y and the final window, and with dy the
    gradients.  Every entry of the result comes with its tolerance in fp32
    roundings (times U), under the name with "~" before it.  ``walk``: the most
    steps that the backward sums in one chain."""
    Bz, L, C = x.shape
    W = weight.shape[1]
    out = {"y": np.zeros_like(x), "window": np.zeros((Bz, W - 1, C)), "dx": np.zeros_like(x),
           "dweight": np.zeros_like(weight), "dbias": np.zeros(C), "dinitial_window": np.zeros((Bz, W - 1, C))}
    out.update({"~" + k: np.zeros_like(v) for k, v in list(out.items())})
    aw = np.abs(weight)
    chain = lambda n: walk + 16 + Bz * (1 + n / 128)
    for b, n in enumerate(lengths(seqlens, Bz, L)):
        xe = np.zeros((n + W - 1, C))
        if win is not None:
            xe[:W - 1] = win[b]
        xe[W - 1:] = x[b, :n]
        pre = np.zeros((n, C)) + (0 if bias is None else bias)
        mag = np.abs(pre)
        for k in range(W):
            pre = pre + weight[:, k] * xe[k:k + n]
            mag = mag + aw[:, k] * np.abs(xe[k:k + n])
        dpre_err = W * mag              # W fused multiply-adds
        if silu:
            s = sigmoid(pre)
            out["y"][b, :n] = pre * s
            # |d(p sigma)/dp| <= 1.1; sigma to |p| + 6 roundings, the product one more
            out["~y"][b, :n] = 1.1 * dpre_err + (np.abs(pre) + 7) * np.abs(pre * s)
        else:
            s = None
            out["y"][b, :n], out["~y"][b, :n] = pre, dpre_err
        out["window"][b] = xe[n:]
        if dy is None:
            continue
        d, err = dy[b, :n].copy(), np.zeros((n, C))
        if silu:
            f = 1 + pre * (1 - s)
            # f: sigma's error and two roundings meet |p|, one more on f; f's slope
            # and sigma's are below 1.1; |d(act')/dp| <= 0.5
            ferr = np.abs(pre) * ((np.abs(pre) + 6) * s + 2) + np.abs(f)
            err = np.abs(d) * (s * ferr + (np.abs(pre) + 8) * s * np.abs(f) + 0.5 * dpre_err) + 2 * np.abs(d * s * f)
            d = d * s * f
        dxe, ex = np.zeros((n + W - 1, C)), np.zeros((n + W - 1, C))
        for k in range(W):
            dxe[k:k + n] += weight[:, k] * d
            ex[k:k + n] += aw[:, k] * (err + W * np.abs(d))
            out["dweight"][:, k] += (xe[k:k + n] * d).sum(0)
            # a chain of `walk` terms, three additions over the wavefronts; then the parts, at
            # least 16 steps each (four walks of four or more), every fourth of them in groups
            # of four (a chain of a sixteenth of them, and the group's and the last ones' five),
            # three more additions over the wavefronts
            out["~dweight"][:, k] += (np.abs(xe[k:k + n]) * (err + chain(n) * np.abs(d))).sum(0)
        if dwin is not None:
            dxe[n:] += dwin[b]
            ex[n:] += np.abs(dxe[n:]) + np.abs(dwin[b])
        out["dbias"] += d.sum(0)
        out["~dbias"] += (err + chain(n) * np.abs(d)).sum(0)
        out["dx"][b, :n], out["~dx"][b, :n] = dxe[W - 1:], ex[W - 1:]
        out["dinitial_window"][b], out["~dinitial_window"][b] = dxe[:W - 1], ex[:W - 1]
    return out


def check(name, got, out, dtype):
    """``got`` (torch, CPU or GPU) against out[name] within its tolerance; the
    rounding to the output's type ("f32" or "bf16") is added."""
    g = got.detach().double().cpu().numpy()
    ref, tol = out[name], out["~" + name]
    assert g.shape == ref.shape, (name, g.shape, ref.shape)
    lim = U * tol * 1.01 + HALF[dtype] * (np.abs(ref) + U * tol) + 2.0 ** -126
    bad = ~(np.abs(g - ref) <= lim)
    assert not bad.any(), "%s: %d of %d off; worst at %s: got %r, expected %r +- %.3g" % (
        (name, bad.sum(), bad.size) + (lambda i: (i, g[i], ref[i], lim[i]))(
            np.unravel_index(np.argmax(np.where(bad, np.abs(g - ref) / lim, 0)), bad.shape)))


def softplus(v):
    return np.maximum(v, 0) + np.log1p(np.exp(-np.abs(v)))


def scan(u, delta, A, B, C, skip=None, gate=None, bias=None, use_softplus=True, h0=None, seqlens=None, adds=0,
         dy=None, dh=None):
    """Everything of the per-channel scan (names as in the binding), with "~"
    tolerances as in ``conv``: errors are carried along the recurrences as the
    values are.  ``adds``: additions in a sum of dt, where segments are joined
    through e^{A sum dt} (each moves the exponent by a rounding)."""
    Bz, L, D = u.shape
    G, N = B.shape[2:]
    per, aA = D // G, np.abs(A)
    up = lambda v: np.repeat(v, per, axis=0)                 # [G, N] -> [D, N]
    down = lambda v: v.reshape(G, per, N).sum(1)             # [D, N] -> [G, N]
    sk = np.zeros(D) if skip is None else skip
    out = {"y": np.zeros_like(u), "final_state": np.zeros((Bz, D, N))}
    if dy is not None:
        out.update({"du": np.zeros_like(u), "ddelta": np.zeros_like(u), "dB": np.zeros_like(B), "dC": np.zeros_like(C),
                    "dgate": np.zeros_like(u), "dA": np.zeros_like(A), "dskip": np.zeros(D),
                    "ddelta_bias": np.zeros(D), "dinitial_state": np.zeros((Bz, D, N))})
    out.update({"~" + k: np.zeros_like(v) for k, v in list(out.items())})
    for b, n in enumerate(lengths(seqlens, Bz, L)):
        raw = delta[b, :n] + (0 if bias is None else bias)
        # the sum's rounding moves dt by |raw| roundings at most; the softplus is a
        # few operations and two hardware approximations
        dt, edt = (softplus(raw), 12 + np.abs(raw)) if use_softplus else (raw, np.ones_like(raw))
        du_ = dt * u[b, :n]
        arg = dt[..., None] * A                               # [n, D, N]
        e = np.exp(arg)
        rel = np.abs(arg) * (edt[..., None] + 2 + adds) + 2   # of e
        h = np.zeros((n + 1, D, N))
        eh = np.zeros_like(h)
        if h0 is not None:
            h[0] = h0[b]
        y, ey = np.zeros((n, D)), np.zeros((n, D))
        for t in range(n):
            inj = du_[t][:, None] * up(B[b, t])
            h[t + 1] = e[t] * h[t] + inj
            eh[t + 1] = e[t] * (eh[t] + np.abs(h[t]) * rel[t]) + np.abs(inj) * (edt[t][:, None] + 3) + np.abs(h[t + 1])
            c = up(C[b, t])
            y[t] = (h[t + 1] * c).sum(-1) + sk * u[b, t]
            ey[t] = (eh[t + 1] * np.abs(c) + (N + 4) * np.abs(h[t + 1] * c)).sum(-1) + np.abs(sk * u[b, t]) \
                + np.abs(y[t])
        out["final_state"][b], out["~final_state"][b] = h[n], eh[n]
        if gate is None:
            out["y"][b, :n], out["~y"][b, :n] = y, ey
        else:
            z = gate[b, :n]
            sg = sigmoid(z)
            out["y"][b, :n] = y * z * sg
            out["~y"][b, :n] = ey * np.abs(z * sg) + 10 * np.abs(y * z * sg)
        if dy is None:
            continue
        K = 64 + L + Bz                                       # longest chain of any sum over steps and batches
        d = dy[b, :n].copy()
        ed = np.zeros_like(d)
        if gate is not None:
            f = sg * (1 + z * (1 - sg))
            # 1 - sg is a sigmoid's complement: sg's error and one rounding meet |z|
            ef = sg * (np.abs(z) * (7 * sg + 2) + 1) + 9 * np.abs(f)
            out["dgate"][b, :n] = d * y * f
            out["~dgate"][b, :n] = np.abs(d) * (ey * np.abs(f) + np.abs(y) * ef) + 3 * np.abs(d * y * f)
            d = d * z * sg
            ed = 10 * np.abs(d)
        carry = np.zeros((D, N)) if dh is None else dh[b].copy()
        ecarry = np.zeros((D, N))
        for t in reversed(range(n)):
            Bt, Ct = up(B[b, t]), up(C[b, t])
            g = carry + d[t][:, None] * Ct
            eg = ecarry + ed[t][:, None] * np.abs(Ct) + np.abs(d[t][:, None] * Ct) + np.abs(g)
            fed = (g * Bt).sum(-1)
            efed = (eg * np.abs(Bt) + (N + 4) * np.abs(g * Bt)).sum(-1)
            gin = g * du_[t][:, None]
            out["dB"][b, t] = down(gin)
            out["~dB"][b, t] = down(eg * np.abs(du_[t][:, None]) + np.abs(gin) * (edt[t][:, None] + 40 + per / 16))
            hd = h[t + 1] * d[t][:, None]
            out["dC"][b, t] = down(hd)
            out["~dC"][b, t] = down(eh[t + 1] * np.abs(d[t][:, None]) + np.abs(h[t + 1]) * ed[t][:, None]
                                    + np.abs(hd) * (40 + per / 16))
            carry = g * e[t]
            ecarry = e[t] * eg + np.abs(carry) * (rel[t] + 1)
            mv = carry * h[t]
            emv = ecarry * np.abs(h[t]) + np.abs(carry) * eh[t] + np.abs(mv)
            out["dA"] += mv * dt[t][:, None]
            out["~dA"] += np.abs(dt[t][:, None]) * (emv + np.abs(mv) * (edt[t][:, None] + K))
            ddt = fed * u[b, t] + (mv * A).sum(-1)
            eddt = efed * np.abs(u[b, t]) + (emv * aA + (N + 5) * np.abs(mv * A)).sum(-1) + 2 * np.abs(fed * u[b, t]) \
                + np.abs(ddt)
            sig = sigmoid(raw[t]) if use_softplus else np.ones(D)
            out["ddelta"][b, t] = ddt * sig
            out["~ddelta"][b, t] = eddt * sig + np.abs(ddt * sig) * (9 + np.abs(raw[t]))
            out["du"][b, t] = fed * dt[t] + sk * d[t]
            out["~du"][b, t] = (efed + np.abs(fed) * (edt[t] + 1)) * np.abs(dt[t]) + np.abs(sk) * (ed[t] + np.abs(d[t])) \
                + np.abs(out["du"][b, t])
        out["dinitial_state"][b], out["~dinitial_state"][b] = carry, ecarry
        out["dskip"] += (d * u[b, :n]).sum(0)
        out["~dskip"] += (np.abs(u[b, :n]) * (ed + K * np.abs(d))).sum(0)
        out["ddelta_bias"] += out["ddelta"][b, :n].sum(0)
        out["~ddelta_bias"] += (out["~ddelta"][b, :n] + K * np.abs(out["ddelta"][b, :n])).sum(0)
    return out
