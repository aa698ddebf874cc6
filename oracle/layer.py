"""The operators around a layer's scan, the plain definitions (float64, sequential in t), with a
bound on the error of an f32 evaluation beside each value.

TEST INFRASTRUCTURE ONLY (see oracle/__init__.py): never called by the product path.

The bounds follow the arithmetic of any straightforward f32 evaluation, first order in u = 2^-24:
  exp(v)     relative error (3 + 1.2 |v|) 2 u: the product with log2(e) rounds once (0.7 |v| 2 u in
             the exponent's units), and the hardware's 2^x is good to 2 ulp.
  silu(a)    = a / (1 + exp(-a)): relative (5 + 1.2 |a|) 2 u, and |silu'| <= 1.1 times a's error.
  softplus   relative (5 + 1.2 |v|) 2 u, and the error of v itself (softplus' <= 1).
  a sum of n terms in any order: n u times the sum of their absolute values.
Outputs in bf16 add 2^-8 of the value (unit roundoff, with room for a value at a binade's end).
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24


def _lens(lens, b, L):
    return [L] * b if lens is None else [int(min(max(n, 0), L)) for n in lens]


def _exp_rel(v):
    return (3 + 1.2 * np.abs(v)) * 2 * U


def _silu(a, err):
    """silu(a) and its error for an a that is off by err."""
    v = a / (1 + np.exp(np.minimum(-a, 700.0)))
    return v, 1.1 * err + np.abs(v) * (5 + 1.2 * np.abs(a)) * 2 * U


def conv(x, w, bias=None, state=None, lens=None, silu=True):
    """x [b, L, d], w [d, W], state [b, W - 1, d] -> (y, error of y, state after the prompt)."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    b, L, d = x.shape
    W = w.shape[1]
    bias = np.zeros(d) if bias is None else np.asarray(bias, np.float64)
    state = np.zeros((b, W - 1, d)) if state is None else np.asarray(state, np.float64)
    y, err, out = np.zeros((b, L, d)), np.zeros((b, L, d)), np.zeros((b, W - 1, d))
    for i, n in enumerate(_lens(lens, b, L)):
        rows = np.concatenate([state[i], x[i, :n]])
        for t in range(n):
            terms = rows[t : t + W].T * w  # [d, W]
            a = bias + terms.sum(1)
            e = (W + 1) * U * (np.abs(bias) + np.abs(terms).sum(1))
            y[i, t], err[i, t] = _silu(a, e) if silu else (a, e)
        out[i] = rows[n : n + W - 1]
    return y, err, out


def selscan(u, dt, A, B, C, D=None, z=None, dt_bias=None, h0=None, lens=None, softplus=True, pieces=1):
    """u, dt, z [b, L, d], A [d, N], B, C [b, L, G, N], h0 [b, d, N]
    -> (y, error of y, h, error of h).

    pieces: of how many tokens the longest sum of delta is whose exponential is taken in one go
    (an evaluation that joins pieces of the time axis): it has relative error pieces * u, which
    moves exp(-s) by at most s exp(-s) pieces u <= 0.37 pieces u of the state it multiplies.
    """
    u, dt, A, B, C = (np.asarray(v, np.float64) for v in (u, dt, A, B, C))
    b, L, d = u.shape
    N, G = A.shape[1], B.shape[2]
    D = np.zeros(d) if D is None else np.asarray(D, np.float64)
    bias = np.zeros(d) if dt_bias is None else np.asarray(dt_bias, np.float64)
    grp = np.arange(d) // (d // G)
    h = np.zeros((b, d, N)) if h0 is None else np.asarray(h0, np.float64).copy()
    mag = np.abs(h)           # sum of the absolute values of h's contributions
    eh = np.zeros((b, d, N))  # error of h
    y, ey = np.zeros((b, L, d)), np.zeros((b, L, d))
    ns = np.asarray(_lens(lens, b, L))
    for t in range(L):
        on = ns > t
        if not on.any():
            break
        ut, Bt, Ct = u[on, t], B[on, t][:, grp], C[on, t][:, grp]
        v = dt[on, t] + bias
        if softplus:
            delta = np.logaddexp(v, 0)
            rel = (5 + 1.2 * np.abs(v)) * 2 * U + U * np.abs(v) / delta
        else:
            delta = v
            rel = U + 0 * v
        x = delta[..., None] * A
        a = np.exp(x)
        # relative error of a (for a piece boundary, over the whole piece: added once at the end)
        ra = _exp_rel(x) + np.abs(x) * (rel[..., None] + 2 * U)
        s = (delta * ut)[..., None] * Bt
        es = np.abs(s) * (rel[..., None] + 2 * U)
        mag[on] = a * mag[on] + np.abs(s)
        eh[on] = a * eh[on] + a * np.abs(h[on]) * ra + es
        h[on] = a * h[on] + s
        eh[on] += U * np.abs(h[on]) + U * np.abs(s)
        piece = 0.37 * pieces * U * mag[on] if pieces > 1 else 0.0
        yt = (h[on] * Ct).sum(-1) + D * ut
        e = ((eh[on] + piece) * np.abs(Ct)).sum(-1) + (N + 2) * U * ((np.abs(h[on] * Ct)).sum(-1) + np.abs(D * ut))
        if z is not None:
            g, eg = _silu(np.asarray(z, np.float64)[on, t], 0.0)
            e = e * np.abs(g) + np.abs(yt) * eg + U * np.abs(yt * g)
            yt = yt * g
        y[on, t], ey[on, t] = yt, e
    if pieces > 1:
        eh = eh + 0.37 * pieces * U * mag
    return y, ey, h, eh


def rmsnorm(x, w, residual=None, eps=1e-5):
    """x [rows, d] -> (v, error of v, r): sums of d squares by threads and trees, d / 16 + 40 deep."""
    r = np.asarray(x, np.float64) + (0 if residual is None else np.asarray(residual, np.float64))
    rs = 1 / np.sqrt((r * r).mean(-1, keepdims=True) + eps)
    v = r * rs * np.asarray(w, np.float64)
    rel = (0.5 * (r.shape[-1] / 16 + 40) + 8) * U
    er = 0 if residual is None else U * np.abs(r)
    return v, np.abs(v) * rel + er * rs * np.abs(np.asarray(w, np.float64)), r
