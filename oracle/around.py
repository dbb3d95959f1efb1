"""CPU oracle of the operators around the block: the norm of query and key
heads with their rotation, and cross attention, each with its gradients.

TEST INFRASTRUCTURE, NOT PRODUCT CODE: plain numpy in float64, written from
the formulas, sharing no code with the CUDA library.  Beside each result the
functions return what a tolerance on it is made of: the sums of magnitudes
that its roundings scale with.
"""
from __future__ import annotations

import math

import numpy as np


def f64(a) -> np.ndarray:
    if hasattr(a, "detach"):
        a = a.detach().double().cpu().numpy()
    return np.asarray(a, dtype=np.float64)


def angles(positions, axes, d_h, theta=10000.0):
    """[N, d_h/2] angles of each token's pairs; positions [N, 3]."""
    out = np.zeros((len(positions), d_h // 2))
    j = 0
    for a, n in enumerate(axes):
        for i in range(n):
            out[:, j] = np.asarray(positions)[:, a] * theta ** (-i / n)
            j += 1
    return out


def grid_positions(N, grid, token0=0):
    T, Hg, Wg = grid
    n = (np.arange(N) + token0) % (T * Hg * Wg)
    return np.stack([n // (Hg * Wg), n // Wg % Hg, n % Wg], 1)


def _pairs(d, halves):
    j = np.arange(d // 2)
    return (j, j + d // 2) if halves else (2 * j, 2 * j + 1)


def rotate(z, ang, halves, sign=1.0):
    """Turns the pairs of z [N, H, d] by sign * ang [N, d/2] (ang None: not)."""
    if ang is None:
        return z.copy()
    a, b = _pairs(z.shape[-1], halves)
    c, s = np.cos(ang)[:, None], sign * np.sin(ang)[:, None]
    y = np.empty_like(z)
    y[..., a] = z[..., a] * c - z[..., b] * s
    y[..., b] = z[..., a] * s + z[..., b] * c
    return y


def pair_size(z, halves):
    """|z_a| + |z_b| of each channel's pair."""
    a, b = _pairs(z.shape[-1], halves)
    y = np.empty_like(z)
    y[..., a] = y[..., b] = np.abs(z[..., a]) + np.abs(z[..., b])
    return y


def norm_rope(x, w, eps, ang, halves):
    """(y, size): size of an element is |z_a| + |z_b| of its pair before the rotation."""
    x = f64(x)
    z = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps) * (1.0 if w is None else f64(w))
    return rotate(z, ang, halves), pair_size(z, halves)


def norm_rope_backward(dy, x, w, eps, ang, halves):
    """dict(dx, dw, dx_size, dw_size)."""
    dy, x = f64(dy), f64(x)
    w = np.ones(x.shape[-1]) if w is None else f64(w)
    dz = rotate(dy, ang, halves, -1.0)
    size = pair_size(dy, halves)
    r = 1.0 / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps)
    n, g, gs = x * r, dz * w, size * np.abs(w)
    return {"dx": r * (g - n * (g * n).mean(-1, keepdims=True)), "dw": (dz * n).sum((0, 1)),
            "dx_size": r * (gs + np.abs(n) * (gs * np.abs(n)).mean(-1, keepdims=True)),
            "dw_size": (size * np.abs(n)).sum((0, 1))}


def cross(q, k, v, segments, dout=None, out_seen=None):
    """Cross attention of q [N, H, d] to k, v [L, Hk, d]; segments: (q0, q1, k0,
    k1) each.  Rows of no segment stay NaN in out, lse and dq, and in dk, dv.

    out_size = sum_j p_ij |v_j|.  With dout also the gradients and their sizes:
      dv_size = sum_i p_ij |dO_i|,
      dq_size = scale sum_j |dS_ij| |K_j|, dk_size likewise over |Q_i|,
      dq_d = scale sum_j p_ij |K_j| sum_c |dO_ic O_ic| (what an error of D does), dk_d likewise,
      dq_p = scale sum_j p_ij |K_j| (|dP_ij| + |D_i|) (what a relative error of P does), dk_p likewise,
      dq_1 = scale sum_j p_ij |K_j| (what an error of dP does), dk_1 likewise.
    """
    q, k, v = f64(q), f64(k), f64(v)
    N, H, d = q.shape
    L, Hk, _ = k.shape
    sc = 1.0 / math.sqrt(d)
    nan = lambda *s: np.full(s, np.nan)  # noqa: E731
    r = {"out": nan(N, H, d), "out_size": nan(N, H, d), "lse": nan(H, N)}
    grads = ("dq", "dq_size", "dq_d", "dq_p", "dq_1"), ("dk", "dk_size", "dk_d", "dk_p", "dk_1", "dv", "dv_size")
    if dout is not None:
        dout = f64(dout)
        r.update({n: nan(N, H, d) for n in grads[0]})
        r.update({n: nan(L, Hk, d) for n in grads[1]})
    for q0, q1, k0, k1 in segments:
        for n in ("out", "out_size"):
            r[n][q0:q1] = 0.0
        r["lse"][:, q0:q1] = -np.inf
        if dout is not None:
            for n in grads[0]:
                r[n][q0:q1] = 0.0
            for n in grads[1]:
                r[n][k0:k1] = 0.0
        if q1 == q0 or k1 == k0:
            continue
        for h in range(H):
            g = h // (H // Hk)
            Q, K, V = q[q0:q1, h], k[k0:k1, g], v[k0:k1, g]
            S = Q @ K.T * sc
            m = S.max(1, keepdims=True)
            e = np.exp(S - m)
            P = e / e.sum(1, keepdims=True)
            r["out"][q0:q1, h], r["out_size"][q0:q1, h] = P @ V, P @ np.abs(V)
            r["lse"][h, q0:q1] = (m + np.log(e.sum(1, keepdims=True)))[:, 0]
            if dout is None:
                continue
            dO = dout[q0:q1, h]
            dP = dO @ V.T
            D = (P * dP).sum(1, keepdims=True)
            dS = P * (dP - D)
            Dm = np.abs(dO * (P @ V)).sum(1, keepdims=True)
            Pm = P * (np.abs(dP) + np.abs(D))
            aK, aQ = np.abs(K), np.abs(Q)
            r["dq"][q0:q1, h], r["dq_size"][q0:q1, h] = sc * dS @ K, sc * np.abs(dS) @ aK
            r["dq_d"][q0:q1, h], r["dq_p"][q0:q1, h] = sc * Dm * (P @ aK), sc * Pm @ aK
            r["dq_1"][q0:q1, h] = sc * P @ aK
            r["dk_1"][k0:k1, g] += sc * P.T @ aQ
            r["dk"][k0:k1, g] += sc * dS.T @ Q
            r["dk_size"][k0:k1, g] += sc * np.abs(dS).T @ aQ
            r["dk_d"][k0:k1, g] += sc * (P * Dm).T @ aQ
            r["dk_p"][k0:k1, g] += sc * Pm.T @ aQ
            r["dv"][k0:k1, g] += P.T @ dO
            r["dv_size"][k0:k1, g] += P.T @ np.abs(dO)
    return r
