"""fp64 references of linear attention with a decay per head and of trees of drafted tokens
(numpy, token by token; states in the library's layout [.., Dv, Dk]). They share no code with the
kernels; central differences of the forward forms pin the gradients."""
from __future__ import annotations

import numpy as np


def _share(x, H):
    """Query or key heads [T, Hk, D] as the H value heads read them."""
    return np.repeat(x, H // x.shape[-2], axis=-2)


def recurrent(q, k, v, g, S0=None, cu_seqlens=None):
    """S_t = exp(g_t) S_{t-1} + v_t k_t^T, o_t = S_t q_t over packed sequences. q, k [T, Hk, Dk], v [T, H, Dv], g [T, H],
    S0 [N, H, Dv, Dk] or None. Returns (o, final states); rows of no sequence are zero."""
    T, H, Dv = v.shape
    cu = [0, T] if cu_seqlens is None else cu_seqlens
    q, k = _share(q, H), _share(k, H)
    N = len(cu) - 1
    S = np.zeros((N, H, Dv, q.shape[-1])) if S0 is None else np.array(S0, dtype=np.float64)
    o = np.zeros((T, H, Dv))
    for n in range(N):
        for t in range(cu[n], cu[n + 1]):
            S[n] = np.exp(g[t])[:, None, None] * S[n] + v[t][:, :, None] * k[t][:, None, :]
            o[t] = np.einsum("hvk,hk->hv", S[n], q[t])
    return o, S


def backward(q, k, v, g, dout, S0=None, dS_out=None, cu_seqlens=None):
    """Gradients of sum(o * dout) + sum(S * dS_out) as a dict of dq, dk [T, Hk, Dk], dv, dg [T, H], dS0."""
    T, H, Dv = v.shape
    Hk, Dk = q.shape[-2:]
    cu = [0, T] if cu_seqlens is None else cu_seqlens
    qs, ks = _share(q, H), _share(k, H)
    N = len(cu) - 1
    dq, dk = np.zeros((T, H, Dk)), np.zeros((T, H, Dk))
    dv, dg, dS0 = np.zeros((T, H, Dv)), np.zeros((T, H)), np.zeros((N, H, Dv, Dk))
    for n in range(N):
        S = np.zeros((H, Dv, Dk)) if S0 is None else np.array(S0[n], dtype=np.float64)
        before = []
        for t in range(cu[n], cu[n + 1]):
            before.append(S)
            S = np.exp(g[t])[:, None, None] * S + v[t][:, :, None] * ks[t][:, None, :]
        dS = np.zeros_like(S) if dS_out is None else np.array(dS_out[n], dtype=np.float64)
        for t in reversed(range(cu[n], cu[n + 1])):
            last, a = before.pop(), np.exp(g[t])
            now = a[:, None, None] * last + v[t][:, :, None] * ks[t][:, None, :]
            dq[t] = np.einsum("hvk,hv->hk", now, dout[t])
            dS = dS + dout[t][:, :, None] * qs[t][:, None, :]
            dv[t] = np.einsum("hvk,hk->hv", dS, ks[t])
            dk[t] = np.einsum("hvk,hv->hk", dS, v[t])
            dg[t] = a * (dS * last).sum((1, 2))
            dS = a[:, None, None] * dS
        dS0[n] = dS
    shared = lambda x: x.reshape(T, Hk, H // Hk, Dk).sum(2)
    return dict(dq=shared(dq), dk=shared(dk), dv=dv, dg=dg, dS0=dS0)


def _next(S, k, v, a, beta):
    S = S * a
    u = v if beta is None else beta[:, None] * (v - np.einsum("hvk,hk->hv", S, k))
    return S + u[:, :, None] * k[:, None, :]


def _decay(g, t, H):
    """Decays of node t as they multiply a state [H, Dv, Dk]."""
    if g is None:
        return np.ones((H, 1, 1))
    a = np.exp(g[t] if g.ndim > 1 else g)
    return a[:, None, :] if a.ndim == 2 else a[:, None, None]


def tree_states(k, v, g, beta, S, parent):
    """One sequence's tree: {node: state behind it}, -1 the sequence's own; absent nodes are left out. k [T, Hk, Dk], v [T, H, Dv],
    g [T, H, Dk], [T, H], [H] or None, beta [T, H] or None (no delta rule), S [H, Dv, Dk], parent [T]."""
    H = v.shape[1]
    k = _share(k, H)
    states = {-1: np.array(S, dtype=np.float64)}
    for t, p in enumerate(parent):
        if p < t and p in states:
            states[t] = _next(states[p], k[t], v[t], _decay(g, t, H), None if beta is None else beta[t])
    return states


def tree(q, k, v, g, beta, S, parent):
    """The outputs [T, H, Dv] of a tree's nodes, zero for absent ones."""
    H = v.shape[1]
    out = np.zeros(v.shape)
    q = _share(q, H)
    for t, state in tree_states(k, v, g, beta, S, parent).items():
        if t >= 0:
            out[t] = np.einsum("hvk,hk->hv", state, q[t])
    return out
