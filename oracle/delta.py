"""fp64 references of the gated delta rule and layer norm, in plain numpy.

TEST INFRASTRUCTURE ONLY, like the rest of this package.

``gdr_forward`` is the recurrence token by token,

    u_t = v_t - e^{g_t} S_{t-1} k_t,  S_t = e^{g_t} S_{t-1} + beta_t u_t k_t^T,
    y_t = scale S_t q_t                                     (S [P, N] per head)

``gdr_backward`` the chain rule applied to it in reverse, token by token, and
``gdr_step`` one token.  Inputs of any float type are upcast exactly.
"""
from __future__ import annotations

import numpy as np

from . import _f64


def _heads(x, H):
    """[.., G, N] -> [.., H, N]: head h uses group h * G // H."""
    return np.repeat(x, H // x.shape[-2], axis=-2)


def gdr_step(q, k, v, g, beta, state, scale=1.0):
    """y, state after one token: q, k [b,G,N], v [b,H,P], g, beta [b,H], state [b,H,P,N]."""
    q, k, v, g, beta, S = (_f64(x) for x in (q, k, v, g, beta, state))
    H = v.shape[1]
    q, k = _heads(q, H), _heads(k, H)
    S = S * np.exp(g)[..., None, None]
    u = v - (S * k[:, :, None]).sum(-1)
    S = S + (beta[..., None] * u)[..., None] * k[:, :, None]
    return scale * (S * q[:, :, None]).sum(-1), S


def _segments(T, seq_idx, nseq):
    """Token ranges of every segment id."""
    ids = np.asarray(seq_idx.cpu() if hasattr(seq_idx, "cpu") else seq_idx)
    return [(int(np.searchsorted(ids, i, "left")), int(np.searchsorted(ids, i, "right"))) for i in range(nseq)]


def gdr_forward(q, k, v, g, beta, scale=1.0, initial_states=None, seq_idx=None, nseq=None):
    """y [b,T,H,P] and the final states [b,H,P,N] (packed: [nseq,H,P,N])."""
    q, k, v, g, beta = (_f64(x) for x in (q, k, v, g, beta))
    b, T, H, P = v.shape
    N = q.shape[3]
    if seq_idx is not None:
        init = np.zeros((nseq, H, P, N)) if initial_states is None else _f64(initial_states)
        y, fin = np.zeros_like(v), init.copy()
        for i, (lo, hi) in enumerate(_segments(T, seq_idx, nseq)):
            if hi > lo:
                s = slice(lo, hi)
                y[:, s], fin[i:i + 1] = gdr_forward(q[:, s], k[:, s], v[:, s], g[:, s], beta[:, s], scale, init[i:i + 1])
        return y, fin
    S = np.zeros((b, H, P, N)) if initial_states is None else _f64(initial_states).copy()
    y = np.zeros_like(v)
    for t in range(T):
        y[:, t], S = gdr_step(q[:, t], k[:, t], v[:, t], g[:, t], beta[:, t], S, scale)
    return y, S


def gdr_backward(q, k, v, g, beta, dy, scale=1.0, initial_states=None, dfinal_states=None, seq_idx=None, nseq=None):
    """dict of dq, dk, dv, dg, dbeta, dinitial_states for L = sum(y dy) + sum(final dfinal)."""
    q, k, v, g, beta, dy = (_f64(x) for x in (q, k, v, g, beta, dy))
    b, T, H, P = v.shape
    G, N = q.shape[2:]
    n = nseq if seq_idx is not None else b
    init = np.zeros((n, H, P, N)) if initial_states is None else _f64(initial_states)
    dfin = np.zeros((n, H, P, N)) if dfinal_states is None else _f64(dfinal_states)
    if seq_idx is not None:
        out = {"d" + nm: np.zeros_like(x) for nm, x in zip("qkvg", (q, k, v, g))}
        out["dbeta"], out["dinitial_states"] = np.zeros_like(beta), dfin.copy()
        for i, (lo, hi) in enumerate(_segments(T, seq_idx, nseq)):
            if hi > lo:
                s = slice(lo, hi)
                r = gdr_backward(q[:, s], k[:, s], v[:, s], g[:, s], beta[:, s], dy[:, s], scale, init[i:i + 1], dfin[i:i + 1])
                out["dinitial_states"][i:i + 1] = r.pop("dinitial_states")
                for nm, x in r.items():
                    out[nm][:, s] = x
        return out
    before, S = [], init.copy()
    for t in range(T):
        before.append(S)
        _, S = gdr_step(q[:, t], k[:, t], v[:, t], g[:, t], beta[:, t], S)
    D = dfin.copy()
    out = {"d" + nm: np.zeros_like(x) for nm, x in zip("qkvg", (q, k, v, g))}
    out["dbeta"] = np.zeros_like(beta)
    group = lambda x: x.reshape(b, G, H // G, N).sum(2)
    for t in range(T - 1, -1, -1):
        S0, a, bt = before[t], np.exp(g[:, t]), beta[:, t]
        qt, kt = _heads(q[:, t], H), _heads(k[:, t], H)
        Sd = S0 * a[..., None, None]
        u = v[:, t] - (Sd * kt[:, :, None]).sum(-1)
        S1 = Sd + (bt[..., None] * u)[..., None] * kt[:, :, None]
        dyt = scale * dy[:, t]
        out["dq"][:, t] = group((dyt[..., None] * S1).sum(2))
        D = D + dyt[..., None] * qt[:, :, None]                  # dL/dS_t
        Dk = (D * kt[:, :, None]).sum(-1)
        du = bt[..., None] * Dk
        out["dv"][:, t], out["dbeta"][:, t] = du, (Dk * u).sum(-1)
        out["dk"][:, t] = group(((bt[..., None] * u)[..., None] * D).sum(2) - (du[..., None] * Sd).sum(2))
        D = D - du[..., None] * kt[:, :, None]                   # dL/d(decayed state)
        out["dg"][:, t] = (D * Sd).sum((2, 3))
        D = D * a[..., None, None]
    out["dinitial_states"] = D
    return out


def layer_norm(x, weight=None, bias=None, eps=1e-5):
    """y, mean, rstd over the last axis."""
    x = _f64(x)
    mean = x.mean(-1)
    d = x - mean[..., None]
    rstd = 1 / np.sqrt((d * d).mean(-1) + eps)
    y = d * rstd[..., None]
    return y * (1 if weight is None else _f64(weight)) + (0 if bias is None else _f64(bias)), mean, rstd


def layer_norm_backward(x, dy, mean, rstd, weight=None):
    """dx, dweight, dbias."""
    x, dy, mean, rstd = (_f64(a) for a in (x, dy, mean, rstd))
    xhat = (x - mean[..., None]) * rstd[..., None]
    w = dy * (1 if weight is None else _f64(weight))
    dx = rstd[..., None] * (w - w.mean(-1, keepdims=True) - xhat * (w * xhat).mean(-1, keepdims=True))
    lead = tuple(range(x.ndim - 1))
    return dx, (dy * xhat).sum(lead), dy.sum(lead)
