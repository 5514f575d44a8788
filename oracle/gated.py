"""Gated lightning attention in fp64, token by token (NumPy).

    S_t = e^{g_t} S_{t-1} + k_t v_t^T,   o_t = S_t^T q_t

and its gradients by the adjoint of the same recurrence: with dS_t the gradient of S_t,

    dS_t  = q_t do_t^T + e^{g_{t+1}} dS_{t+1}        (dS_N also takes d_state)
    dq_t  = S_t do_t,   dk_t = dS_t v_t,   dv_t = dS_t^T k_t
    dg_t  = e^{g_t} <dS_t, S_{t-1}>,   d_initial = e^{g_1} dS_1

Every quantity is formed as written; there are no blocks.
"""
from __future__ import annotations

import numpy as np


def _np(x):
    if x is None:
        return None
    if hasattr(x, "detach"):
        x = x.detach().double().cpu().numpy()
    return np.asarray(x, dtype=np.float64)


def prefill(q, k, v, g, cu, initial=None):
    """o [T, H, D] and the final states [S, H, D, D]; g may be None."""
    q, k, v, g, initial = map(_np, (q, k, v, g, initial))
    T, H, D = q.shape
    o = np.zeros((T, H, D))
    last = np.zeros((len(cu) - 1, H, D, D))
    for s in range(len(cu) - 1):
        S = np.zeros((H, D, D)) if initial is None else initial[s].copy()
        for t in range(cu[s], cu[s + 1]):
            a = np.ones(H) if g is None else np.exp(g[t])
            S = a[:, None, None] * S + k[t][:, :, None] * v[t][:, None, :]
            o[t] = np.einsum("hx,hxy->hy", q[t], S)
        last[s] = S
    return o, last


def backward(q, k, v, g, do, cu, initial=None, d_state=None):
    """dq, dk, dv [T, H, D], dg [T, H] and d_initial [S, H, D, D]."""
    q, k, v, g, do, initial, d_state = map(_np, (q, k, v, g, do, initial, d_state))
    T, H, D = q.shape
    dq, dk, dv = (np.zeros((T, H, D)) for _ in range(3))
    dg = np.zeros((T, H))
    first = np.zeros((len(cu) - 1, H, D, D))
    for s in range(len(cu) - 1):
        lo, hi = cu[s], cu[s + 1]
        S = np.zeros((H, D, D)) if initial is None else initial[s].copy()
        before = []
        for t in range(lo, hi):
            a = np.ones(H) if g is None else np.exp(g[t])
            before.append(S)
            S = a[:, None, None] * S + k[t][:, :, None] * v[t][:, None, :]
            dq[t] = np.einsum("hxy,hy->hx", S, do[t])
        dS = np.zeros((H, D, D)) if d_state is None else d_state[s].copy()
        for t in range(hi - 1, lo - 1, -1):
            dS = dS + q[t][:, :, None] * do[t][:, None, :]
            dk[t] = np.einsum("hxy,hy->hx", dS, v[t])
            dv[t] = np.einsum("hxy,hx->hy", dS, k[t])
            a = np.ones(H) if g is None else np.exp(g[t])
            dg[t] = a * np.einsum("hxy,hxy->h", dS, before[t - lo])
            dS = a[:, None, None] * dS
        first[s] = dS
    return dq, dk, dv, dg, first


def decode_step(q, k, v, g, state):
    """o [B, H, D] and the new states [B, H, D, D]."""
    q, k, v, g, state = map(_np, (q, k, v, g, state))
    a = np.ones(q.shape[:2]) if g is None else np.exp(g)
    new = a[:, :, None, None] * state + k[..., :, None] * v[..., None, :]
    return np.einsum("bhx,bhxy->bhy", q, new), new
