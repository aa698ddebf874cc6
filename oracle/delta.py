"""The gated delta rule and the norms around it, the plain definitions (float64, sequential in t), with a
bound on the error of an f32 evaluation beside each value.

TEST INFRASTRUCTURE ONLY (see oracle/__init__.py): never called by the product path.

delta's bound goes by rows of the state (2-norms over the dstate columns), u = 2^-24.  A token maps a row S to
a S (I - beta k k^T) + beta v k^T.  With |k| <= 1 and 0 <= beta <= 2 that matrix has norm at most a, so an error that a row
has is carried on with a factor of at most a, and each token adds errors of its own:
  the sum S k of N terms          sqrt(N) u a |S| |k|, its roundings taken as independent, and with them those of d
  a                               relative (3 + 1.2 |x|) 2 u for the exponential (see oracle/layer.py), and x's own
                                  rounding |x| times softplus' (5 + 1.2 |v|) 2 u, of a |S|
  a S + d k                       2 u (|a S| + |d| |k|)
The tokens' errors are added as independent ones (squares), and the result is held to SIGMAS times that.
An evaluation in chunks whose operands are split into halves adds `split` (the halves' joint unit roundoff) of
what enters the corrections: a |S| |k| for S k; the largest |v| + a |S| so far for the inverse and what it is multiplied
with, sqrt(2) each with a sum of squares of the inverse's row of 2; and |d| |k|.  Its outputs are
sums over the chunk's corrections with operands rounded to `out`: out sqrt(sum of squares) of those terms.
Outputs in bf16 add 2^-8 of the value.
"""
from __future__ import annotations

import numpy as np

from .layer import U, _exp_rel, _lens, _silu

SIGMAS = 6.0
EPS = 1e-6


def _unit(v):
    return v / np.sqrt((v * v).sum(-1, keepdims=True) + EPS)


def delta(q, k, v, dt, beta, A, dt_bias=None, h0=None, lens=None, scale=None, softplus=True, sigmoid=True, l2norm=True,
          split=0.0, out=0.0):
    """q, k [b, L, G, N], v [b, L, nh, H], dt, beta [b, L, nh], A [nh], h0 [b, nh, H, N]
    -> (y, error of y, h, error of h), the latter one of a whole row."""
    q, k, v, dt, beta, A = (np.asarray(x, np.float64) for x in (q, k, v, dt, beta, A))
    b, L, nh, H = v.shape
    G, N = q.shape[2:]
    scale = N ** -0.5 if scale is None else scale
    grp = np.arange(nh) // (nh // G)
    bias = np.zeros(nh) if dt_bias is None else np.asarray(dt_bias, np.float64)
    if l2norm:
        q, k = _unit(q), _unit(k)
    rate = 1 / (1 + np.exp(-beta)) if sigmoid else beta
    x = dt + bias
    step = np.logaddexp(x, 0) if softplus else x
    rel_step = (5 + 1.2 * np.abs(x)) * 2 * U + U * np.abs(x) / np.maximum(np.abs(step), 1e-300) if softplus else U + 0 * x
    g = step * A
    a, ra = np.exp(g), _exp_rel(g) + np.abs(g) * (rel_step + 2 * U)
    h = np.zeros((b, nh, H, N)) if h0 is None else np.asarray(h0, np.float64).copy()
    var = np.zeros((b, nh, H))   # squared error of a row
    worst = np.zeros((b, nh, H))  # largest |v| + a |S| so far
    terms = np.zeros((b, nh, H))  # sum of squared decayed corrections
    y, ey = np.zeros((b, L, nh, H)), np.zeros((b, L, nh, H))
    ns = np.asarray(_lens(lens, b, L))
    for t in range(L):
        on = ns > t
        if not on.any():
            break
        kt, qt = k[on, t][:, grp], q[on, t][:, grp]
        at, bt, rat = (z[on, t][..., None] for z in (a, rate, ra))
        lk, lq = np.linalg.norm(kt, axis=-1)[..., None], np.linalg.norm(qt, axis=-1)[..., None] * abs(scale)
        old = at[..., None] * h[on]
        size = np.linalg.norm(old, axis=-1)
        vt = v[on, t]
        d = bt * (vt - np.einsum("bhpn,bhn->bhp", old, kt))
        new = old + d[..., None] * kt[:, :, None]
        worst[on] = np.maximum(worst[on], np.abs(vt) + size)
        into = np.abs(bt) * lk * (size + np.abs(vt))
        local = U * ((N ** 0.5 + 6) * into + 4 * size + 4 * np.abs(d) * lk) + rat * size + split * (np.abs(bt) * lk * (size + 2 * worst[on]) + np.abs(d) * lk)
        if l2norm:  # the lengths' roundings: relative sqrt(N) u of k, once in d and once beside it
            local = local + 2 * U * (N ** 0.5 / 2 + 4) * (into + np.abs(d))
        var[on] = at ** 2 * var[on] + local ** 2
        terms[on] = at ** 2 * terms[on] + (d * lk) ** 2
        h[on] = new
        size = np.linalg.norm(new, axis=-1)
        y[on, t] = np.einsum("bhpn,bhn->bhp", new, qt) * scale
        ey[on, t] = lq * (np.sqrt(var[on]) + (1.5 * N ** 0.5 + 8) * U * (size + np.abs(d)) + out * np.sqrt(terms[on])
                          + 2 * split * worst[on])
    return y, SIGMAS * ey, h, SIGMAS * np.sqrt(var)


def _rms(v, eps):
    """v / sqrt(mean(v^2) + eps) over the last axis, and its relative error (sums of squares by threads and trees)."""
    n = v.shape[-1]
    return v / np.sqrt((v * v).mean(-1, keepdims=True) + eps), (0.5 * (n / 16 + 40) + 8) * U


def gatednorm(x, z, w, group=0, gate_first=False, eps=1e-5):
    """x, z [rows, d], w [d] or [group] -> (y, error of y)."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    rows, d = x.shape
    group = group or d
    gate, eg = _silu(np.asarray(z, np.float64), 0.0)
    rel_gate = eg / np.maximum(np.abs(gate), 1e-300)
    w = np.tile(w, d // w.shape[0])
    u = x * gate if gate_first else x
    v, rel = _rms(u.reshape(rows, d // group, group), eps)
    v = v.reshape(rows, d) * w
    if gate_first:  # the gates' errors in the sum of squares too: at most the largest of them
        return v, np.abs(v) * (rel + rel_gate + rel_gate.reshape(rows, -1, group).max(-1).repeat(group, -1) + 2 * U)
    return v * gate, np.abs(v * gate) * (rel + rel_gate + 2 * U)


def blocknorm(x, w, residual, next_weight, z=None, alpha=1.0, eps=1e-5):
    """x [rows, d] -> (y, error of y, r, error of r)."""
    x, res, w2 = (np.asarray(v, np.float64) for v in (x, residual, next_weight))
    v, rel = _rms(x, eps)
    v = v * np.asarray(w, np.float64)
    ev = np.abs(v) * (rel + 2 * U)
    if z is not None:
        gate, eg = _silu(np.asarray(z, np.float64), 0.0)
        ev = ev * np.abs(gate) + np.abs(v) * eg + U * np.abs(v * gate)
        v = v * gate
    r = alpha * res + v
    er = ev + 2 * U * (np.abs(alpha * res) + np.abs(v))
    y, rel = _rms(r, eps)
    rs = 1 / np.sqrt((r * r).mean(-1, keepdims=True) + eps)
    # r's errors in the mean square: at most sqrt(mean(er^2)) of its root
    both = rel + np.sqrt((er * er).mean(-1, keepdims=True)) * rs
    return y * w2, np.abs(w2) * (np.abs(y) * (both + 2 * U) + er * rs), r, er
