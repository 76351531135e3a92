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


def conv(x, weight, bias, win, seqlens, silu, dy=None, dwin=None):
    """Everything of the convolution: y and the final window, and with dy the
    gradients.  Every entry of the result comes with its tolerance in fp32
    roundings (times U), under the name with "~" before it."""
    Bz, L, C = x.shape
    W = weight.shape[1]
    out = {"y": np.zeros_like(x), "window": np.zeros((Bz, W - 1, C)), "dx": np.zeros_like(x),
           "dweight": np.zeros_like(weight), "dbias": np.zeros(C), "dinitial_window": np.zeros((Bz, W - 1, C))}
    out.update({"~" + k: np.zeros_like(v) for k, v in list(out.items())})
    aw = np.abs(weight)
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
            # sums of at most 32 + 3 terms in a chain, then one chain over parts
            out["~dweight"][:, k] += (np.abs(xe[k:k + n]) * (err + (48 + Bz * (1 + n / 128)) * np.abs(d))).sum(0)
        if dwin is not None:
            dxe[n:] += dwin[b]
            ex[n:] += np.abs(dxe[n:]) + np.abs(dwin[b])
        out["dbias"] += d.sum(0)
        out["~dbias"] += (err + (48 + Bz * (1 + n / 128)) * np.abs(d)).sum(0)
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
