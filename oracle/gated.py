"""Float64 oracle of gated linear attention and of the query/key norm with
position rotation, token by token, in numpy.  Test infrastructure only; shares
no code with the library.

Arrays are float64: q [B, T, H, d], k, v [B, T, Hk, d], g [B, T, Hk] (log gates,
-inf allowed), states [B, Hk, d, d] as [key value c][value value e].
"""
from __future__ import annotations

import numpy as np


def _groups(q, Hk):
    B, T, H, d = q.shape
    return q.reshape(B, T, Hk, H // Hk, d)


def _lens(lens, B, T):
    return np.full(B, T) if lens is None else np.clip(np.asarray(lens), 0, T)


def gated_forward(q, k, v, g, scale, state=None, lens=None, keep=False):
    """(out, final state); with keep also every state [T + 1, B, Hk, d, d] (after t tokens)."""
    B, T, H, d = q.shape
    Hk = k.shape[2]
    qg, n = _groups(q, Hk), _lens(lens, B, T)
    S = np.zeros((B, Hk, d, d)) if state is None else state.astype(np.float64).copy()
    out = np.zeros_like(qg)
    states = [S.copy()] if keep else None
    for t in range(T):
        on = t < n
        new = np.exp(g[on, t])[..., None, None] * S[on] + k[on, t][..., :, None] * v[on, t][..., None, :]
        S[on] = new
        out[on, t] = scale * np.einsum("bhgc,bhce->bhge", qg[on, t], new)
        if keep:
            states.append(S.copy())
    out = out.reshape(B, T, H, d)
    return (out, S, np.stack(states)) if keep else (out, S)


def gated_backward(q, k, v, g, dout, scale, state=None, dstate=None, lens=None):
    """(dq, dk, dv, dg, gradient of the initial state)."""
    B, T, H, d = q.shape
    Hk = k.shape[2]
    n = _lens(lens, B, T)
    _, _, S = gated_forward(q, k, v, g, scale, state, lens, keep=True)
    qg, dog = _groups(q, Hk), _groups(dout, Hk)
    D = np.zeros((B, Hk, d, d)) if dstate is None else dstate.astype(np.float64).copy()
    dq, dk, dv, dg = np.zeros_like(qg), np.zeros_like(k), np.zeros_like(v), np.zeros_like(g)
    for t in range(T - 1, -1, -1):
        on = t < n
        D[on] += scale * np.einsum("bhgc,bhge->bhce", qg[on, t], dog[on, t])
        dq[on, t] = scale * np.einsum("bhce,bhge->bhgc", S[t + 1][on], dog[on, t])
        dk[on, t] = np.einsum("bhce,bhe->bhc", D[on], v[on, t])
        dv[on, t] = np.einsum("bhce,bhc->bhe", D[on], k[on, t])
        D[on] *= np.exp(g[on, t])[..., None, None]
        dg[on, t] = np.einsum("bhce,bhce->bh", S[t][on], D[on])
    return dq.reshape(B, T, H, d), dk, dv, dg, D


def gated_pairs(q, k, v, g, scale):
    """out of one head [T, d] from the T x T matrix of weights scale exp(g_{s+1} + .. + g_t) (q_t . k_s)."""
    T = q.shape[0]
    A = np.zeros((T, T))
    for t in range(T):
        for s in range(t + 1):
            A[t, s] = scale * np.exp(np.sum(g[s + 1:t + 1])) * (q[t] @ k[s])
    return A @ v


def gated_step(q, k, v, g, pool, scale, slots=None):
    """Rows in order: (out [B, H, d], the pool afterwards)."""
    B, H, d = q.shape
    Hk = k.shape[1]
    pool = pool.astype(np.float64).copy()
    out = np.zeros((B, H, d))
    for b in range(B):
        s = b if slots is None else int(slots[b])
        if not 0 <= s < pool.shape[0]:
            continue
        for h in range(H):
            if h % (H // Hk) == 0:
                j = h // (H // Hk)
                pool[s, j] = np.exp(g[b, j]) * pool[s, j] + np.outer(k[b, j], v[b, j])
            out[b, h] = scale * (q[b, h] @ pool[s, h // (H // Hk)])
    return out, pool


# ---------------------------------------------------------------- norm and rotation

def rope_matrix(pos, freq, sections, d, interleaved):
    """The d x d matrix that turns one head of a token at positions pos."""
    R = np.eye(d)
    P = sum(sections)
    axis = np.repeat(np.arange(len(sections)), sections)
    for i in range(P):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, P + i)
        th = float(pos[axis[i]]) * float(freq[i])
        R[a, a] = R[b, b] = np.cos(th)
        R[a, b], R[b, a] = -np.sin(th), np.sin(th)
    return R


def norm_rope(x, w, pos, freq, sections, interleaved, eps):
    """x [B, T, H, d], w [d], pos [B, T, axes]."""
    B, T, H, d = x.shape
    n = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * w
    out = np.empty_like(x)
    for b in range(B):
        for t in range(T):
            out[b, t] = n[b, t] @ rope_matrix(pos[b, t], freq, sections, d, interleaved).T
    return out


def norm_rope_backward(x, w, pos, freq, sections, interleaved, eps, dy):
    """(dx, dw)."""
    B, T, H, d = x.shape
    dx, dw = np.empty_like(x), np.zeros(d)
    for b in range(B):
        for t in range(T):
            R = rope_matrix(pos[b, t], freq, sections, d, interleaved)
            for h in range(H):
                dn, y = dy[b, t, h] @ R, x[b, t, h]
                r = 1.0 / np.sqrt(np.mean(y * y) + eps)
                dw += dn * y * r
                # d(r y_j)/dy_i = r (delta_ij - r^2 y_i y_j / d)
                dx[b, t, h] = (np.eye(d) - r * r * np.outer(y, y) / d) @ (dn * w) * r
    return dx, dw
