"""Linear attention with a decay for each head and the norms before and after a
block in 64 bits, as their definitions read (numpy, token by token): what the
GPU kernels are compared with.

Each function also gives, under `..._terms`, the same sums over the terms'
sizes: what an error relative to every term adds up to."""

import numpy as np


def _heads(x, H):
    return np.repeat(np.asarray(x, np.float64), H // x.shape[-2], axis=-2)


def _decays(g, B, T, H):
    return np.exp(np.broadcast_to(np.asarray(g, np.float64), (B, T, H)))


def linattn_forward(q, k, v, g, scale, h0=None, lens=None):
    """Returns o, h_final, and a dict of their terms and of the states."""
    B, T, H, P = v.shape
    N = q.shape[-1]
    q, k, v = _heads(q, H), _heads(k, H), np.asarray(v, np.float64)
    a = _decays(g, B, T, H)
    S = np.zeros((B, H, N, P)) if h0 is None else np.array(h0, np.float64)
    A = np.abs(S)
    lens = np.full(B, T) if lens is None else np.clip(lens, 0, T)
    o, ot = np.zeros((B, T, H, P)), np.zeros((B, T, H, P))
    states, sizes = [S.copy()], [A.copy()]
    for t in range(T):
        on = np.nonzero(t < lens)[0]
        S, A = S.copy(), A.copy()
        if len(on):
            d = a[on, t][..., None, None]
            with np.errstate(invalid="ignore"):
                S[on] = d * S[on] + k[on, t][..., :, None] * v[on, t][..., None, :]
                A[on] = d * A[on] + np.abs(k[on, t])[..., :, None] * np.abs(v[on, t])[..., None, :]
            o[on, t] = scale * np.einsum("bhn,bhnp->bhp", q[on, t], S[on])
            ot[on, t] = abs(scale) * np.einsum("bhn,bhnp->bhp", np.abs(q[on, t]), A[on])
        states.append(S)
        sizes.append(A)
    return o, S, {"o_terms": ot, "h_terms": A, "states": states, "sizes": sizes}


def linattn_backward(q, k, v, g, scale, do, h0=None, dh=None, lens=None):
    B, T, H, P = v.shape
    KH, N = q.shape[-2:]
    f = linattn_forward(q, k, v, g, scale, h0, lens)[2]
    q, k = _heads(q, H), _heads(k, H)
    v, do = np.asarray(v, np.float64), scale * np.asarray(do, np.float64)
    a = _decays(g, B, T, H)
    lens = np.full(B, T) if lens is None else np.clip(lens, 0, T)
    D = np.zeros((B, H, N, P)) if dh is None else np.array(dh, np.float64)
    A = np.abs(D)
    z = lambda *w: np.zeros((B, T, *w))  # noqa: E731
    r = {"gq": z(H, N), "gk": z(H, N), "gv": z(H, P), "gg": z(H)}
    w = {n + "_terms": np.zeros_like(x) for n, x in r.items()}
    for t in reversed(range(T)):
        on = np.nonzero(t < lens)[0]
        if not len(on):
            continue
        D, A = D.copy(), A.copy()
        qt, kt, vt, dt, at = q[on, t], k[on, t], v[on, t], do[on, t], a[on, t][..., None, None]
        S, B_ = f["states"][t + 1][on], f["sizes"][t + 1][on]
        X = D[on] + qt[..., :, None] * dt[..., None, :]  # the gradient of S_t
        Y = A[on] + np.abs(qt)[..., :, None] * np.abs(dt)[..., None, :]
        r["gq"][on, t] = np.einsum("bhnp,bhp->bhn", S, dt)
        r["gk"][on, t] = np.einsum("bhnp,bhp->bhn", X, vt)
        r["gv"][on, t] = np.einsum("bhnp,bhn->bhp", X, kt)
        r["gg"][on, t] = (at * X * f["states"][t][on]).sum((-1, -2))
        w["gq_terms"][on, t] = np.einsum("bhnp,bhp->bhn", B_, np.abs(dt))
        w["gk_terms"][on, t] = np.einsum("bhnp,bhp->bhn", Y, np.abs(vt))
        w["gv_terms"][on, t] = np.einsum("bhnp,bhn->bhp", Y, np.abs(kt))
        # (taken as <S_t, dL/dS_t> less the token's own write)
        w["gg_terms"][on, t] = (Y * B_).sum((-1, -2)) + np.einsum("bhn,bhnp,bhp->bh", np.abs(kt), Y, np.abs(vt))
        D[on], A[on] = at * X, at * Y
    for n in ("gq", "gk"):
        r[n] = r[n].reshape(B, T, KH, H // KH, N).sum(3)
        w[n + "_terms"] = w[n + "_terms"].reshape(B, T, KH, H // KH, N).sum(3)
    if np.ndim(g) == 1:
        r["gg"], w["gg_terms"] = r["gg"].sum((0, 1)), w["gg_terms"].sum((0, 1))
    return {**r, **w, "gh0": D, "gh0_terms": A}


def silu(z):
    return z / (1 + np.exp(-z))


def norm(h, layer, eps):
    m = h.mean(-1, keepdims=True) if layer else 0 * h[..., :1]
    r = 1 / np.sqrt(((h - m) ** 2).mean(-1, keepdims=True) + eps)
    return (h - m) * r, m[..., 0], r[..., 0]


def norm_back(a, hh, r, layer):
    t = a - hh * (a * hh).mean(-1, keepdims=True)
    return r[..., None] * (t - a.mean(-1, keepdims=True) if layer else t)


def add_norm(x, residual, w, b, layer, alpha, scale, eps, rounded=lambda s: s):
    s = rounded(residual + alpha * (x if scale is None else scale * x))
    hh, m, r = norm(s, layer, eps)
    y = hh * (1 if w is None else w) + (0 if b is None else b)
    return y, s, m, r


def add_norm_backward(dy, ds, x, s, w, layer, alpha, scale, eps):
    hh, _, r = norm(s, layer, eps)
    t = norm_back(dy * (1 if w is None else w), hh, r, layer) + (0 if ds is None else ds)
    return {"gresidual": t, "gx": alpha * t * (1 if scale is None else scale), "gweight": (dy * hh).sum(0), "gbias": dy.sum(0),
            "gscale": alpha * (t * x).sum(0), "gweight_terms": np.abs(dy * hh).sum(0), "gbias_terms": np.abs(dy).sum(0),
            "gscale_terms": np.abs(alpha * t * x).sum(0)}


def gated_norm(x, z, w, b, layer, group, first, eps):
    R, D = x.shape
    h = (x * silu(z) if first else x).reshape(R, D // group, group)
    hh, m, r = norm(h, layer, eps)
    u = hh.reshape(R, D) * (1 if w is None else w) + (0 if b is None else b)
    return (u if first else u * silu(z)), m, r


def gated_norm_backward(dy, x, z, w, b, layer, group, first, eps):
    R, D = x.shape
    sg = 1 / (1 + np.exp(-z))
    gate, slope = z * sg, sg * (1 + z * (1 - sg))
    h = (x * gate if first else x).reshape(R, D // group, group)
    hh, _, r = norm(h, layer, eps)
    du = dy if first else dy * gate
    dh = norm_back((du * (1 if w is None else w)).reshape(h.shape), hh, r, layer).reshape(R, D)
    hh = hh.reshape(R, D)
    if first:
        gx, gz = dh * gate, dh * x * slope
    else:
        gx, gz = dh, dy * (hh * (1 if w is None else w) + (0 if b is None else b)) * slope
    return {"gx": gx, "gz": gz, "gweight": (du * hh).sum(0), "gbias": du.sum(0), "gweight_terms": np.abs(du * hh).sum(0),
            "gbias_terms": np.abs(du).sum(0)}
