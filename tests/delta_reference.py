"""The gated delta rule and layer norm in 64 bits, as their definitions read
(numpy, token by token): what the GPU kernels are compared with.

delta_forward returns (o, h_final, states); delta_backward the gradients of
L = <o, do> + <h_final, dh> by the reversed recurrence, and for each token the
size of the terms whose difference dL/dg is."""

import numpy as np


def _heads(x, H):
    return np.repeat(np.asarray(x, np.float64), H // x.shape[-2], axis=-2)


def token(S, q, k, v, g, beta):
    """One token on a state [..., N, P]; returns (S, o without scale, v - prediction)."""
    with np.errstate(invalid="ignore"):
        S = np.exp(g)[..., None, None] * S
    e = v - np.einsum("...np,...n->...p", S, k)
    S = S + k[..., :, None] * (beta[..., None] * e)[..., None, :]
    return S, np.einsum("...np,...n->...p", S, q), e


def delta_forward(q, k, v, g, beta, scale, h0=None, lens=None):
    B, T, H, P = v.shape
    N = q.shape[-1]
    q, k = _heads(q, H), _heads(k, H)
    v, g, beta = (np.asarray(x, np.float64) for x in (v, g, beta))
    S = np.zeros((B, H, N, P)) if h0 is None else np.array(h0, np.float64)
    lens = np.full(B, T) if lens is None else np.clip(lens, 0, T)
    o = np.zeros((B, T, H, P))
    states = [S.copy()]
    for t in range(T):
        on = np.nonzero(t < lens)[0]
        if len(on):
            S = S.copy()
            S[on], ot, _ = token(S[on], q[on, t], k[on, t], v[on, t], g[on, t], beta[on, t])
            o[on, t] = scale * ot
        states.append(S)
    return o, S, states


def delta_backward(q, k, v, g, beta, scale, do, h0=None, dh=None, lens=None):
    B, T, H, P = v.shape
    KH, N = q.shape[-2:]
    _, _, states = delta_forward(q, k, v, g, beta, scale, h0, lens)
    q, k = _heads(q, H), _heads(k, H)
    v, g, beta, do = (np.asarray(x, np.float64) for x in (v, g, beta, do))
    lens = np.full(B, T) if lens is None else np.clip(lens, 0, T)
    D = np.zeros((B, H, N, P)) if dh is None else np.array(dh, np.float64)
    r = {n: np.zeros(s) for n, s in (("gq", (B, T, H, N)), ("gk", (B, T, H, N)), ("gv", (B, T, H, P)),
                                     ("gg", (B, T, H)), ("gbeta", (B, T, H)), ("gg_terms", (B, T, H)))}
    for t in reversed(range(T)):
        on = np.nonzero(t < lens)[0]
        if not len(on):
            continue
        qt, kt, bt = q[on, t], k[on, t], beta[on, t]
        a = np.exp(g[on, t])[..., None, None] * states[t][on]  # the decayed state
        e = v[on, t] - np.einsum("bhnp,bhn->bhp", a, kt)
        d = D[on] + scale * qt[..., :, None] * do[on, t][..., None, :]
        r["gq"][on, t] = scale * np.einsum("bhnp,bhp->bhn", states[t + 1][on], do[on, t])
        w = np.einsum("bhnp,bhn->bhp", d, kt)  # gradient of the write beta e
        r["gv"][on, t] = bt[..., None] * w
        r["gbeta"][on, t] = np.sum(w * e, -1)
        r["gk"][on, t] = (np.einsum("bhnp,bhp->bhn", d, bt[..., None] * e)
                          - np.einsum("bhnp,bhp->bhn", a, r["gv"][on, t]))
        d = d - kt[..., :, None] * r["gv"][on, t][..., None, :]
        r["gg"][on, t] = np.sum(d * a, (-1, -2))
        r["gg_terms"][on, t] = np.sum(np.abs(d * a), (-1, -2))
        D = D.copy()
        D[on] = np.exp(g[on, t])[..., None, None] * d
    r["gq"], r["gk"] = (r[n].reshape(B, T, KH, H // KH, N).sum(3) for n in ("gq", "gk"))
    r["gh0"] = D
    return r


def layernorm(x, w, b, eps):
    x = np.asarray(x, np.float64)
    m = x.mean(-1, keepdims=True)
    r = 1.0 / np.sqrt(((x - m) ** 2).mean(-1, keepdims=True) + eps)
    y = (x - m) * r
    if w is not None:
        y = y * np.asarray(w, np.float64)
    if b is not None:
        y = y + np.asarray(b, np.float64)
    return y, m[..., 0], r[..., 0]


def layernorm_backward(dy, x, w, eps):
    _, m, r = layernorm(x, None, None, eps)
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    xh = (x - m[..., None]) * r[..., None]
    a = dy * (1.0 if w is None else np.asarray(w, np.float64))
    gx = r[..., None] * (a - a.mean(-1, keepdims=True) - xh * (a * xh).mean(-1, keepdims=True))
    lead = tuple(range(x.ndim - 1))
    return gx, (dy * xh).sum(lead), dy.sum(lead)
