"""Plain 64-bit numpy forms of linear attention with a decay per head, step by step,
and of the group norm, with tolerances as in layer_ref: every value's
magnitude (its sums over absolute values) times a count of fp32 roundings.

Linear attention.  Each product gamma^n a.c x passes: the decays (a chunk's
power and one per chunk boundary, each within 4 roundings: the exponential's one
ulp, its exponent's corrected parts, the product), at most an addition per step and
per contracted element (counted as an ulp, twice a rounding, as the matrix
instructions' order and intermediate rounding are theirs), and a few products.
In bf16 the decayed scores and the state are split into two bf16 parts (what is
left out is below 2^-17 of the value), decayed rows into three (2^-26).  In fp32 every
factor is three bf16 parts and six of the nine products are formed: each part is at most
2^-9 of the one before, so the three left out are below 2^-26 + 2^-26 + 2^-36 of the product,
half a rounding, within the several that are counted for it."""
import numpy as np

from layer_ref import HALF, U, check, lengths, sigmoid  # noqa: F401


def _walk(a, c, x, decay, first, n, lead, dtype, scale_w=1.0, dim=1):
    """y[t] = S[t] a[t] along S[t] = decay S[t-1] + scale_w x[t] c[t]^T over n steps, S [.., x, c],
    ``first`` entering step 0 as decay^lead first; and the last S.  With the tolerances."""
    S = np.zeros(x.shape[1:] + (c.shape[-1],)) if first is None else first * decay ** lead / (decay if decay > 0 else 1)
    M = np.abs(S)
    y, ey = np.zeros((n, x.shape[-1])), np.zeros((n, x.shape[-1]))
    chunk = 64 if dtype == "bf16" else 32
    cuts = 2.0 ** -26 / U if dtype == "bf16" else 0.0
    for t in range(n):
        inj = scale_w * x[t][:, None] * c[t][None, :]
        if t == 0 and decay == 0 and first is not None:
            S, M = (first if lead == 0 else 0 * first), (np.abs(first) if lead == 0 else 0 * M)
            S, M = S + inj, M + np.abs(inj)
        else:
            S, M = decay * S + inj, decay * M + np.abs(inj)
        steps = 2 * (t + 1) + 5 * (t // chunk + 2) + 10 + cuts
        y[t] = S @ a[t]
        ey[t] = (M @ np.abs(a[t])) * (steps + 2 * a.shape[-1] + 2 * chunk + (2.0 ** -17 / U if dtype == "bf16" else 0))
    return y, ey, S, M * (2 * n + 5 * (n // chunk + 2) + 10 + cuts)


def attention(q, k, v, log_decay, scale=None, first=None, seqlens=None, dy=None, dlast=None, dtype="f32"):
    """Everything of the attention; q [Bz,L,H,Dk], k, v [Bz,L,K,..], first [Bz,H,Dv,Dk]."""
    Bz, L, H, Dk = q.shape
    K, Dv = v.shape[2:]
    scale = Dk ** -0.5 if scale is None else scale
    out = {"y": np.zeros((Bz, L, H, Dv)), "final_state": np.zeros((Bz, H, Dv, Dk)), "dq": np.zeros_like(q),
           "dk": np.zeros_like(k), "dv": np.zeros_like(v), "dinitial_state": np.zeros((Bz, H, Dv, Dk))}
    out.update({"~" + n: np.zeros_like(t) for n, t in list(out.items())})

    def put(name, at, value, err):
        out[name][at] += value
        out["~" + name][at] += err + 2 * (H // K) * np.abs(value)   # the sum over the heads that share

    for b, n in enumerate(lengths(seqlens, Bz, L)):
        for h in range(H):
            g, decay = h * K // H, float(np.exp(log_decay[h]))
            a, c, x = q[b, :n, h], k[b, :n, g], v[b, :n, g]
            S0 = None if first is None else first[b, h]
            y, ey, S, eS = _walk(a, c, x, decay, S0, n, 1, dtype)
            if n == 0:
                S, eS = (S0 if S0 is not None else S), 0 * S
            out["y"][b, :n, h], out["~y"][b, :n, h] = scale * y, abs(scale) * ey
            out["final_state"][b, h], out["~final_state"][b, h] = S, eS
            if dy is None:
                continue
            d = dy[b, :n, h]
            y, ey, _, _ = _walk(d, x, c, decay, None if S0 is None else S0.T, n, 1, dtype)
            put("dq", (b, slice(0, n), h), scale * y, abs(scale) * ey)
            G0 = None if dlast is None else dlast[b, h]
            turn = slice(None, None, -1)
            # against time the given adjoint is the last step's own
            y, ey, G, eG = _walk(c[turn], a[turn], d[turn], decay, G0, n, 0, dtype, scale_w=scale)
            put("dv", (b, slice(0, n), g), y[turn], ey[turn])
            if n == 0:
                G, eG = (G0 if G0 is not None else G), 0 * G
            else:
                G, eG = G * decay, (eG + 4 * np.abs(G)) * decay
            out["dinitial_state"][b, h], out["~dinitial_state"][b, h] = G, eG
            y, ey, _, _ = _walk(x[turn], d[turn], a[turn], decay, None if G0 is None else G0.T, n, 0, dtype, scale_w=scale)
            put("dk", (b, slice(0, n), g), y[turn], ey[turn])
    return out


def norm(x, groups, weight=None, bias=None, gate=None, eps=1e-5, center=True, silu=True, gate_first=False, seqlens=None,
         dy=None):
    """Everything of the group norm; x [Bz,L,C].  A sum over a group passes at most ``A``
    additions on any path: 32 elements of a thread, 6 steps over a wavefront, 16
    wavefronts.  A sigmoid is within |z| + 9 roundings (its exponential's argument, two
    hardware approximations of an ulp, a sum, a product)."""
    Bz, L, C = x.shape
    m, A = C // groups, 60.0
    rows = lambda t: t.reshape(t.shape[0], groups, m)   # noqa: E731
    w = np.ones(C) if weight is None else weight
    bs = np.zeros(C) if bias is None else bias
    w, bs = w.reshape(groups, m), bs.reshape(groups, m)
    out = {"y": np.zeros_like(x), "dx": np.zeros_like(x), "dgate": np.zeros_like(x), "dweight": np.zeros(C),
           "dbias": np.zeros(C)}
    out.update({"~" + n: np.zeros_like(t) for n, t in list(out.items())})

    def slope(z, s, es):
        f = 1 + z * (1 - s)
        # 1 - s: s's error and a rounding meet |z|; then the sum's and the product's roundings
        return s * f, s * (np.abs(z) * (es * s + 1) + 2 + 2 * np.abs(f)) + es * s * np.abs(f)

    for b, n in enumerate(lengths(seqlens, Bz, L)):
        if n == 0:
            continue
        X = rows(x[b, :n])
        u, eu = X, np.zeros_like(X)
        if gate is not None:
            Z = rows(gate[b, :n])
            s, es = (sigmoid(Z), np.abs(Z) + 9) if silu else (np.ones_like(Z), np.zeros_like(Z))
            act = Z * s
            eact = (es + 1) * np.abs(act)
            if gate_first:
                u = X * act
                eu = np.abs(X) * eact + np.abs(u)
        mean = lambda t: t.mean(-1, keepdims=True)      # noqa: E731
        c, ec = u, eu
        if center:
            c = u - mean(u)
            ec = eu + mean(eu) + (A + 2) * mean(np.abs(u)) + np.abs(c)
        var = mean(c * c)
        # second order in ec matters where a group is constant: its squares are then all of var
        evar = 2 * mean(np.abs(c) * ec) + U * mean(ec * ec) + (A + 3) * var
        r = 1 / np.sqrt(var + eps)
        rel = 0.5 * evar / np.maximum(var + eps - U * evar, 1e-300) + 4
        nn = c * r
        en = ec * r + np.abs(nn) * (rel + 1)
        p = nn * w + bs
        ep = en * np.abs(w) + np.abs(nn * w) + np.abs(p)
        flat = lambda t: t.reshape(n, C)                # noqa: E731
        if gate is None and silu:
            sp, esp = sigmoid(p), np.abs(p) + 9
            y, ey = p * sp, 1.1 * ep + (esp + 1) * np.abs(p * sp)
        elif gate is not None and not gate_first:
            y, ey = p * act, ep * np.abs(act) + np.abs(p) * eact + np.abs(p * act)
        else:
            y, ey = p, ep
        out["y"][b, :n], out["~y"][b, :n] = flat(y), flat(ey)
        if dy is None:
            continue
        d, ed = rows(dy[b, :n]), np.zeros_like(X)
        if gate is None and silu:
            f, ef = slope(p, sp, esp)
            ef = ef + 0.5 * ep                         # the slope's own slope is at most a half
            d, ed = d * f, np.abs(d) * ef + np.abs(d * f)
        elif gate is not None and not gate_first:
            f, ef = slope(Z, s, es) if silu else (np.ones_like(Z), 0 * Z)
            dz = d * p * f
            out["dgate"][b, :n] = flat(dz)
            out["~dgate"][b, :n] = flat(np.abs(d) * (ep * np.abs(f) + np.abs(p) * ef) + 3 * np.abs(dz))
            d, ed = d * act, np.abs(d) * eact + np.abs(d * act)
        K = n + 40                                     # additions over rows, parts and their sums
        out["dweight"] += (d * nn).sum(0).ravel()
        out["~dweight"] += (ed * np.abs(nn) + np.abs(d) * en + (K + Bz * L) * np.abs(d * nn)).sum(0).ravel()
        out["dbias"] += d.sum(0).ravel()
        out["~dbias"] += (ed + (K + Bz * L) * np.abs(d)).sum(0).ravel()
        dn = d * w
        edn = ed * np.abs(w) + np.abs(dn)
        c1 = mean(dn) if center else 0 * mean(dn)
        ec1 = (mean(edn) + (A + 2) * mean(np.abs(dn))) if center else 0 * c1
        c2 = mean(dn * nn)
        ec2 = mean(edn * np.abs(nn) + np.abs(dn) * en) + (A + 2) * mean(np.abs(dn * nn))
        t = dn - c1 - nn * c2
        et = edn + ec1 + en * np.abs(c2) + np.abs(nn) * ec2 + 3 * (np.abs(dn) + np.abs(c1) + np.abs(nn * c2))
        du = t * r
        edu = et * r + (rel + 1) * np.abs(du)
        if gate_first:
            f, ef = slope(Z, s, es) if silu else (np.ones_like(Z), 0 * Z)
            dz = du * X * f
            out["dgate"][b, :n] = flat(dz)
            out["~dgate"][b, :n] = flat(np.abs(X) * (edu * np.abs(f) + np.abs(du) * ef) + 3 * np.abs(dz))
            du, edu = du * act, edu * np.abs(act) + np.abs(du) * eact + np.abs(du * act)
        out["dx"][b, :n], out["~dx"][b, :n] = flat(du), flat(edu)
    return out
