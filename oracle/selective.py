"""The selective scan, its causal convolution, RMS norm and the 8-bit product in fp64 (numpy), token by
token from their definitions; the gradients by the chain rule, with the sizes of the terms that a sum over
tokens adds (what a tolerance for it has to be measured against).

Tensors are torch tensors or arrays of any type; results are fp64 arrays.  ``lengths`` are the lengths of a
packed stream's segments (batch 1), None for batch rows.
"""
from __future__ import annotations

import numpy as np
import torch


def f64(t):
    if t is None:
        return None
    if isinstance(t, torch.Tensor):
        t = t.detach().cpu()
        return t.to(torch.float64).numpy() if t.dtype != torch.float8_e4m3fn else t.to(torch.float32).numpy().astype(np.float64)
    return np.asarray(t, dtype=np.float64)


def rows_of(b, T, lengths):
    """Slices of the flattened tokens, one a row."""
    if lengths is None:
        return [slice(i * T, (i + 1) * T) for i in range(b)]
    ends = np.cumsum([0, *lengths])
    return [slice(int(ends[i]), int(ends[i + 1])) for i in range(len(lengths))]


def sigmoid(v):
    return 0.5 * (1 + np.tanh(0.5 * v))


def _scan_inputs(x, dt, A, B, C, D, z, dt_bias, softplus):
    x, dt, A, B, C, D, z, dt_bias = (f64(t) for t in (x, dt, A, B, C, D, z, dt_bias))
    b, T, dim = x.shape
    G, N = B.shape[2:]
    raw = dt if dt_bias is None else dt + dt_bias
    delta = np.maximum(raw, 0) + np.log1p(np.exp(-np.abs(raw))) if softplus else raw
    slope = sigmoid(raw) if softplus else np.ones_like(raw)
    flat = lambda t, w: None if t is None else t.reshape(b * T, *w)
    keys = lambda t: np.repeat(t.reshape(b * T, G, N), dim // G, axis=1)
    return (flat(x, (dim,)), A, keys(B), keys(C), np.zeros(dim) if D is None else D, flat(z, (dim,)), flat(delta, (dim,)),
            flat(slope, (dim,)))


def scan_forward(x, dt, A, B, C, D=None, z=None, dt_bias=None, softplus=True, init=None, lengths=None):
    """y [b,T,dim] and the final states [rows,dim,N]."""
    shape = tuple(x.shape)
    x, A, B, C, D, z, delta, _ = _scan_inputs(x, dt, A, B, C, D, z, dt_bias, softplus)
    init = f64(init)
    y, finals = np.zeros_like(x), []
    for r, at in enumerate(rows_of(shape[0], shape[1], lengths)):
        h = np.zeros(A.shape) if init is None else init[r].copy()
        for t in range(at.start, at.stop):
            h = np.exp(delta[t][:, None] * A) * h + (delta[t] * x[t])[:, None] * B[t]
            y[t] = (h * C[t]).sum(1) + D * x[t]
        finals.append(h)
    if z is not None:
        y = y * z * sigmoid(z)
    return y.reshape(shape), np.stack(finals)


def scan_backward(x, dt, A, B, C, dy, D=None, z=None, dt_bias=None, softplus=True, init=None, dfinal=None, lengths=None):
    """Every gradient, and under "sizes" the sums of the absolute terms of dA, dB, dC, dD, ddt_bias and ddt."""
    shape, keys = tuple(x.shape), tuple(B.shape)
    x, A, B, C, D, z, delta, slope = _scan_inputs(x, dt, A, B, C, D, z, dt_bias, softplus)
    init, dfinal = f64(init), f64(dfinal)
    dim, N = A.shape
    G = keys[2]
    out = f64(dy).reshape(x.shape)
    gate = 1.0 if z is None else z * sigmoid(z)
    dy = out * gate
    g_ = {n: np.zeros_like(x) for n in ("dx", "ddt", "dz")}
    dB, dC, sB, sC = (np.zeros((x.shape[0], G, N)) for _ in range(4))
    dA, sA, s_ddt = np.zeros_like(A), np.zeros_like(A), np.zeros_like(x)
    dinit = []
    group = lambda v: v.reshape(G, dim // G, N).sum(1)
    for r, at in enumerate(rows_of(shape[0], shape[1], lengths)):
        h = np.zeros(A.shape) if init is None else init[r].copy()
        hs = [h]
        for t in range(at.start, at.stop):
            h = np.exp(delta[t][:, None] * A) * h + (delta[t] * x[t])[:, None] * B[t]
            hs.append(h)
        g = np.zeros(A.shape) if dfinal is None else dfinal[r].copy()
        for t in range(at.stop - 1, at.start - 1, -1):
            h1, h0 = hs[t - at.start + 1], hs[t - at.start]
            g_["dz"][t] = out[t] * ((h1 * C[t]).sum(1) + D * x[t])
            g = g + dy[t][:, None] * C[t]
            vC, vB = dy[t][:, None] * h1, (delta[t] * x[t])[:, None] * g
            dC[t], dB[t], sC[t], sB[t] = group(vC), group(vB), group(np.abs(vC)), group(np.abs(vB))
            along = (g * B[t]).sum(1)
            g_["dx"][t] = delta[t] * along + D * dy[t]
            a = np.exp(delta[t][:, None] * A)
            gh = a * g * h0
            g_["ddt"][t] = (x[t] * along + (gh * A).sum(1)) * slope[t]
            s_ddt[t] = (np.abs(x[t]) * np.abs(g * B[t]).sum(1) + np.abs(gh * A).sum(1)) * slope[t]
            dA += gh * delta[t][:, None]
            sA += np.abs(gh * delta[t][:, None])
            g = a * g
        dinit.append(g)
    res = {"dx": g_["dx"].reshape(shape), "ddt": g_["ddt"].reshape(shape), "dA": dA, "dB": dB.reshape(keys), "dC": dC.reshape(keys),
           "dD": (dy * x).sum(0), "ddt_bias": g_["ddt"].sum(0), "dinitial_states": np.stack(dinit), "dz": None}
    if z is not None:
        s = sigmoid(z)
        res["dz"] = (g_["dz"] * s * (1 + z * (1 - s))).reshape(shape)
    res["sizes"] = {"dA": sA, "dB": sB.reshape(keys), "dC": sC.reshape(keys), "dD": np.abs(dy * x).sum(0), "ddt": s_ddt.reshape(shape),
                    "ddt_bias": s_ddt.sum(0)}
    return res


def _conv_rows(x, weight, bias, window, lengths):
    shape = tuple(x.shape)
    x, weight, bias, window = (f64(t) for t in (x, weight, bias, window))
    dim, K = weight.shape
    x = x.reshape(-1, dim)
    for r, at in enumerate(rows_of(shape[0], shape[1], lengths)):
        past = np.zeros((K - 1, dim)) if window is None else window[r]
        sig = np.concatenate([past, x[at]])
        n = at.stop - at.start
        v = np.zeros((n, dim)) if bias is None else np.tile(bias, (n, 1))
        for k in range(K):
            v += sig[k:k + n] * weight[:, k]
        yield at, sig, v


def conv_forward(x, weight, bias=None, silu=True, window=None, lengths=None):
    """y and the final windows [rows, width-1, dim]."""
    dim, K = weight.shape
    y, ends = np.zeros(tuple(x.shape)), []
    for at, sig, v in _conv_rows(x, weight, bias, window, lengths):
        y.reshape(-1, dim)[at] = v * sigmoid(v) if silu else v
        ends.append(sig[len(sig) - (K - 1):])
    return y, np.stack(ends)


def conv_backward(x, weight, dy, bias=None, silu=True, window=None, dwindow=None, lengths=None):
    """dx, dweight, dbias, dinitial_window, and the sizes of the terms of dweight and dbias."""
    dim, K = weight.shape
    w, dy, dwindow = f64(weight), f64(dy).reshape(-1, dim), f64(dwindow)
    dx = np.zeros((int(np.prod(x.shape[:2])), dim))
    dw, db, sw, sb, firsts = np.zeros((dim, K)), np.zeros(dim), np.zeros((dim, K)), np.zeros(dim), []
    for r, (at, sig, v) in enumerate(_conv_rows(x, weight, bias, window, lengths)):
        dv = dy[at]
        if silu:
            s = sigmoid(v)
            dv = dv * s * (1 + v * (1 - s))
        ds = np.zeros_like(sig)
        if dwindow is not None and K > 1:
            ds[len(sig) - (K - 1):] = dwindow[r]
        for k in range(K):
            ds[k:k + len(dv)] += dv * w[:, k]
            dw[:, k] += (dv * sig[k:k + len(dv)]).sum(0)
            sw[:, k] += np.abs(dv * sig[k:k + len(dv)]).sum(0)
        db += dv.sum(0)
        sb += np.abs(dv).sum(0)
        dx[at] = ds[K - 1:]
        firsts.append(ds[:K - 1])
    return {"dx": dx.reshape(tuple(x.shape)), "dweight": dw, "dbias": db, "dinitial_window": np.stack(firsts),
            "sizes": {"dweight": sw, "dbias": sb}}


def rms_norm(r, weight=None, eps=1e-5):
    """y and rstd of the rows of r as they are."""
    r = f64(r)
    rstd = 1 / np.sqrt((r * r).mean(-1) + eps)
    y = r * rstd[..., None]
    return (y if weight is None else y * f64(weight)), rstd


def rms_norm_backward(r, dy, rstd, weight=None, dresidual=None):
    """dr, dweight and the size of dweight's terms."""
    r, dy, rstd = f64(r), f64(dy), f64(rstd)[..., None]
    hat = r * rstd
    w = dy if weight is None else dy * f64(weight)
    dr = rstd * (w - hat * (w * hat).mean(-1, keepdims=True))
    if dresidual is not None:
        dr = dr + f64(dresidual)
    flat = (dy * hat).reshape(-1, r.shape[-1])
    return dr, flat.sum(0), np.abs(flat).sum(0)


def to_8bit(y):
    """The scales of every 128 values of a row of y, and y in units of them."""
    y = f64(y)
    dim = y.shape[-1]
    nb = -(-dim // 128)
    pad = np.zeros((*y.shape[:-1], nb * 128))
    pad[..., :dim] = y
    b = pad.reshape(*y.shape[:-1], nb, 128)
    scales = np.maximum(np.abs(b).max(-1) / 448, 2.0 ** -126)
    return scales, (b / scales[..., None]).reshape(pad.shape)[..., :dim]


def matmul_fp8(a, a_scale, w, w_scale, bias=None):
    """The product, and the sum of its absolute terms."""
    a, sa, w, sw = f64(a), f64(a_scale), f64(w), f64(w_scale)
    k, n = a.shape[-1], w.shape[0]
    av = a * np.repeat(sa, 128, axis=-1)[..., :k]
    wv = w * np.repeat(np.repeat(sw, 128, axis=0)[:n], 128, axis=1)[:, :k]
    out = av @ wv.T
    size = np.abs(av) @ np.abs(wv).T
    return (out if bias is None else out + f64(bias)), size
