"""CPU oracle of the gated delta rule, and of the norm and rotation of queries
and keys -- TEST INFRASTRUCTURE.

Only ``tests/`` and the examples' checks may import this module; the CUDA
library shares no code with it.  Plain fp64 numpy, token by token, written
straight from the definitions:

* delta rule, per head with a state S (P x N):
      Sd = exp(g) S;  e = v - Sd k;  S = Sd + beta e k^T;  o = scale S q
  and its reverse sweep from stored states (every token's state is kept);
* norm and rotation of one row x: y = w x / sqrt(m + eps), m the mean or the
  sum of the squares; the first R elements turned in pairs.
"""
from __future__ import annotations

import numpy as np


def _f64(a):
    if a is None:
        return None
    if hasattr(a, "detach"):
        a = a.detach().cpu().double().numpy()
    return np.asarray(a, dtype=np.float64)


def _ranges(b, T, cu):
    """(row, first token, end) of every sequence."""
    if cu is None:
        return [(i, 0, T) for i in range(b)]
    cu = [int(x) for x in np.asarray(cu.cpu() if hasattr(cu, "cpu") else cu)]
    return [(0, cu[i], cu[i + 1]) for i in range(len(cu) - 1)]


def fwd(q, k, v, g, beta, scale, init=None, cu=None, keep=False):
    """(o, final states); with ``keep`` also the list of per-sequence trails."""
    q, k, v, g, beta, init = (_f64(x) for x in (q, k, v, g, beta, init))
    b, T, G, N = q.shape
    H, P = v.shape[2:]
    rep = H // G
    seqs = _ranges(b, T, cu)
    o = np.zeros((b, T, H, P))
    final = np.zeros((len(seqs), H, P, N))
    trails = []
    for i, (r, t0, t1) in enumerate(seqs):
        S = np.zeros((H, P, N)) if init is None else init[i].copy()
        trail = []
        for t in range(t0, t1):
            kt, qt = np.repeat(k[r, t], rep, 0), np.repeat(q[r, t], rep, 0)
            dec = np.exp(g[r, t])[:, None, None]
            Sd = np.where(dec == 0, 0.0, dec * S)
            e = v[r, t] - np.einsum("hpn,hn->hp", Sd, kt)
            S = Sd + beta[r, t][:, None, None] * e[:, :, None] * kt[:, None, :]
            o[r, t] = scale * np.einsum("hpn,hn->hp", S, qt)
            if keep:
                trail.append((Sd, e, S))
        final[i] = S
        trails.append(trail)
    return (o, final, trails) if keep else (o, final)


def bwd(q, k, v, g, beta, scale, dout, init=None, cu=None, dfinal=None):
    """Gradients of sum(o * dout) + sum(final * dfinal); ``dg_abs`` is the sum
    of the magnitudes of dg's terms, the scale of its cancellation."""
    o, final, trails = fwd(q, k, v, g, beta, scale, init, cu, keep=True)
    q, k, v, g, beta, dout, dfinal = (_f64(x) for x in (q, k, v, g, beta, dout, dfinal))
    b, T, G, N = q.shape
    H, P = v.shape[2:]
    rep = H // G
    seqs = _ranges(b, T, cu)
    dq, dk = np.zeros_like(q), np.zeros_like(k)
    dv, dg, db, dga = np.zeros_like(v), np.zeros_like(g), np.zeros_like(beta), np.zeros_like(g)
    dinit = np.zeros_like(final)
    for i, (r, t0, t1) in enumerate(seqs):
        dS = np.zeros((H, P, N)) if dfinal is None else dfinal[i].copy()
        for t in range(t1 - 1, t0 - 1, -1):
            kt, qt = np.repeat(k[r, t], rep, 0), np.repeat(q[r, t], rep, 0)
            Sd, e, S = trails[i][t - t0]
            do, be = dout[r, t], beta[r, t][:, None]
            dq[r, t] = (scale * np.einsum("hpn,hp->hn", S, do)).reshape(G, rep, N).sum(1)
            dS = dS + scale * do[:, :, None] * qt[:, None, :]
            F = np.einsum("hpn,hn->hp", dS, kt)
            db[r, t] = (F * e).sum(1)
            dv[r, t] = be * F
            dkh = np.einsum("hpn,hp->hn", dS, be * e) - np.einsum("hpn,hp->hn", Sd, dv[r, t])
            dk[r, t] = dkh.reshape(G, rep, N).sum(1)
            dS = dS - dv[r, t][:, :, None] * kt[:, None, :]
            dg[r, t] = (dS * Sd).sum((1, 2))
            dga[r, t] = np.abs(dS * Sd).sum((1, 2))
            dS = np.exp(g[r, t])[:, None, None] * dS
        dinit[i] = dS
    return dict(o=o, final=final, dq=dq, dk=dk, dv=dv, dg=dg, dbeta=db, dinit=dinit, dg_abs=dga)


def chunked_fwd(q, k, v, g, beta, scale, chunk):
    """o of one row by the chunked form: a unit lower triangular solve inside each chunk."""
    q, k, v, g, beta = (_f64(x)[0] for x in (q, k, v, g, beta))
    T, G, N = q.shape
    H, P = v.shape[1:]
    o = np.zeros((1, T, H, P))
    for h in range(H):
        S = np.zeros((P, N))
        for t0 in range(0, T, chunk):
            sl = slice(t0, min(T, t0 + chunk))
            Q, K, V, be = q[sl, h * G // H], k[sl, h * G // H], v[sl, h], beta[sl, h]
            Gs = np.cumsum(g[sl, h])
            D = np.tril(np.exp(np.minimum(Gs[:, None] - Gs[None], 0)))
            A = np.tril(D * (K @ K.T), -1) * be[None]
            E = np.linalg.solve(np.eye(len(Gs)) + A, V - np.exp(Gs)[:, None] * (K @ S.T))
            U = be[:, None] * E
            o[0, sl, h] = scale * (np.exp(Gs)[:, None] * (Q @ S.T) + (D * (Q @ K.T)) @ U)
            S = np.exp(Gs[-1]) * S + (np.exp(Gs[-1] - Gs)[:, None] * U).T @ K
    return o


# ---- norm and rotation --------------------------------------------------------

def _pairs(R, interleaved):
    return (np.arange(0, R, 2), np.arange(1, R, 2)) if interleaved else (np.arange(R // 2), np.arange(R // 2, R))


def qk_fwd(x, w, cos, sin, pos, rms, eps, interleaved):
    """z (b,T,H,D) of one of q and k."""
    x, w, cos, sin = (_f64(a) for a in (x, w, cos, sin))
    m = (x * x).mean(-1) if rms else (x * x).sum(-1)
    y = x / np.sqrt(m + eps)[..., None] * (1.0 if w is None else w)
    if cos is not None:
        a, b = _pairs(2 * cos.shape[1], interleaved)
        p = np.asarray(pos.cpu() if hasattr(pos, "cpu") else pos)
        c, s = cos[p][:, :, None], sin[p][:, :, None]
        ya, yb = y[..., a], y[..., b]
        y = y.copy()
        y[..., a], y[..., b] = ya * c - yb * s, ya * s + yb * c
    return y


def qk_bwd(x, dz, w, cos, sin, pos, rms, eps, interleaved):
    """(dx, dw) of sum(z * dz)."""
    x, dz, w, cos, sin = (_f64(a) for a in (x, dz, w, cos, sin))
    if cos is not None:
        dz = qk_fwd_turn(dz, cos, -sin, pos, interleaved)
    over = x.shape[-1] if rms else 1
    root = np.sqrt((x * x).sum(-1) / over + eps)[..., None]
    dw = (dz * x / root).sum((0, 1, 2))
    u = dz if w is None else dz * w
    dx = u / root - x * (u * x).sum(-1)[..., None] / (over * root ** 3)
    return dx, dw


def qk_fwd_turn(y, cos, sin, pos, interleaved):
    a, b = _pairs(2 * cos.shape[1], interleaved)
    p = np.asarray(pos.cpu() if hasattr(pos, "cpu") else pos)
    c, s = cos[p][:, :, None], sin[p][:, :, None]
    z = y.copy()
    z[..., a], z[..., b] = y[..., a] * c - y[..., b] * s, y[..., a] * s + y[..., b] * c
    return z
