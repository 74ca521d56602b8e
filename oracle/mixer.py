"""fp64 NumPy oracle of layer norm and the gated linear recurrence.

Plain loops over tokens, no code shared with the CUDA library.  The
``*_bound`` functions run the same recurrences on absolute values and return
how far a 32-bit evaluation may end up from the exact one.
"""
from __future__ import annotations

import numpy as np

U32 = 2.0 ** -24        # half a unit in the last place, relative, of fp32
U16 = 2.0 ** -8         # the same of bf16 (8 significant bits)


def f64(t):
    """A tensor or array as fp64 NumPy (None stays None)."""
    if t is None:
        return None
    return t.detach().double().cpu().numpy() if hasattr(t, "detach") \
        else np.asarray(t, dtype=np.float64)


def ln_fwd(x, weight=None, bias=None, eps=1e-5, residual=None):
    """(y, s, mean, rstd) of s = x + residual."""
    s = f64(x) if residual is None else f64(x) + f64(residual)
    mean = s.mean(-1)
    c = s - mean[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        rstd = 1.0 / np.sqrt((c * c).mean(-1) + eps)
        y = c * rstd[..., None]
    if weight is not None:
        y = y * f64(weight)
    if bias is not None:
        y = y + f64(bias)
    return y, s, mean, rstd


def ln_bwd(y_grad, x, weight, mean, rstd, sum_grad=None):
    """(dx, dw, db) with the given statistics; rows are all axes but the
    last."""
    dy, r = f64(y_grad), f64(rstd)[..., None]
    xh = (f64(x) - f64(mean)[..., None]) * r
    g = dy if weight is None else dy * f64(weight)
    dx = r * (g - g.mean(-1, keepdims=True)
              - xh * (g * xh).mean(-1, keepdims=True))
    if sum_grad is not None:
        dx = dx + f64(sum_grad)
    rows = tuple(range(dy.ndim - 1))
    return dx, (dy * xh).sum(rows), dy.sum(rows)


def _sequences(x, cu):
    """The token ranges of each sequence: a list of index expressions."""
    if cu is None:
        return [(n, slice(None)) for n in range(x.shape[0])]
    return [slice(int(a), int(b)) for a, b in zip(cu[:-1], cu[1:])]


def glr_fwd(x, log_alpha, h0=None, cu=None):
    """(o, hT): x, log_alpha [B,T,D], or [T,D] with the offsets ``cu``."""
    x, la = f64(x), f64(log_alpha)
    seqs = _sequences(x, cu)
    D = x.shape[-1]
    hT = np.zeros((len(seqs), D)) if h0 is None else f64(h0).copy()
    o = np.empty_like(x)
    with np.errstate(invalid="ignore", over="ignore"):
        alpha = np.exp(la)
        for n, q in enumerate(seqs):
            h, xs, al = hT[n], x[q], alpha[q]
            out = np.empty_like(xs)
            for t in range(xs.shape[0]):
                h = al[t] * h + xs[t]
                out[t] = h
            o[q] = out
            hT[n] = h
    return o, hT


def glr_bwd(o, log_alpha, o_grad, hT_grad=None, h0=None, cu=None):
    """(dx, dlog_alpha, dh0) with h_{t-1} read from the given o."""
    o, la, do = f64(o), f64(log_alpha), f64(o_grad)
    seqs = _sequences(o, cu)
    D = o.shape[-1]
    zero = np.zeros((len(seqs), D))
    h0 = zero if h0 is None else f64(h0)
    dh0 = zero.copy() if hT_grad is None else f64(hT_grad).copy()
    dx, dla = np.empty_like(o), np.empty_like(o)
    alpha = np.exp(la)
    for n, q in enumerate(seqs):
        c, al, dos = dh0[n], alpha[q], do[q]
        h = np.concatenate([h0[n][None], o[q]])
        g, a = np.empty_like(dos), np.empty_like(dos)
        for t in range(dos.shape[0] - 1, -1, -1):
            g[t] = dos[t] + c
            c = al[t] * g[t]
            a[t] = c * h[t]
        dx[q], dla[q] = g, a
        dh0[n] = c
    return dx, dla, dh0


def glr_fwd_bound(x, log_alpha, h0=None, cu=None, k=8):
    """Error of a 32-bit forward: each step adds at most k units of
    max-magnitude state (one rounding of alpha h + x, and alpha's own
    relative error), decayed by the later steps.  Products of alpha over a
    block carry the sum of their factors' relative errors, which is the same
    recurrence.  Returns the bounds of (o, hT)."""
    mag, _ = glr_fwd(np.abs(f64(x)), log_alpha,
                     None if h0 is None else np.abs(f64(h0)), cu)
    return glr_fwd(k * U32 * mag + 1e-30, log_alpha, None, cu)


def glr_bwd_bound(o, log_alpha, o_grad, hT_grad=None, h0=None, cu=None, k=8):
    """The same for the backward: bounds of (dx, dlog_alpha, dh0)."""
    ab = lambda v: None if v is None else np.abs(f64(v))  # noqa: E731
    mag, da, d0 = glr_bwd(ab(o), log_alpha, ab(o_grad), ab(hT_grad), ab(h0),
                          cu)
    e, ea, e0 = glr_bwd(ab(o), log_alpha, k * U32 * mag + 1e-30, None,
                        ab(h0), cu)
    return e, ea + k * U32 * da, e0 + k * U32 * d0
