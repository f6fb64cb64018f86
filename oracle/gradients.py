"""fp64 gradients of the KDA recurrence, the output gate and the row norms.

TEST INFRASTRUCTURE, as the rest of this package. Written from the definitions
in numpy, sharing no code with the HIP library; pinned by finite differences of
the forward oracles (``tests/test_oracle_gradients.py``).

``recurrent_backward`` differentiates the per-token recurrence in reverse. With
the state as M = S^T (key channels in rows), M' = Diag(alpha) M_prev, e = v - M'^T k,
u = beta e, M = M' + k u^T, o = M^T q, and dM the gradient of M from later tokens:
    dM += q do^T;  dq = M do;  du = dM^T k;  dk = dM u - M' dv with dv = beta du
    dbeta = du . e;  dM' = dM - k dv^T;  dg = alpha rowsum(dM' M_prev);  dM_prev = Diag(alpha) dM'
"""
from __future__ import annotations

import numpy as np

from . import _f64


def recurrent_backward(q, k, v, g, beta, dout, S0=None, dS_out=None, cu_seqlens=None, l2norm_eps=None):
    """Layouts as ``oracle.recurrent``: q, k, g [T, H, Dk]; v, dout [T, H, Dv]; beta [T, H];
    S0, dS_out [N, H, Dk, Dv] or None. ``l2norm_eps``: q and k are normalised first (see
    ``oracle.l2norm``) and the gradients are those of the raw ones. Returns a dict of dq, dk,
    dv, dg, dbeta and dS0."""
    q, k, v, g, beta, dout = (_f64(x) for x in (q, k, v, g, beta, dout))
    T, H, Dk = q.shape
    Dv = v.shape[-1]
    cu = np.array([0, T]) if cu_seqlens is None else np.asarray(cu_seqlens, dtype=np.int64)
    N = len(cu) - 1
    if l2norm_eps is not None:
        nq, nk = (np.sqrt((x * x).sum(-1, keepdims=True) + l2norm_eps) for x in (q, k))
        q, k = q / nq, k / nk
    alpha = np.exp(g)
    res = dict(dq=np.zeros_like(q), dk=np.zeros_like(k), dv=np.zeros_like(v), dg=np.zeros_like(g),
               dbeta=np.zeros_like(beta), dS0=np.zeros((N, H, Dk, Dv)))
    for n in range(N):
        M = np.zeros((H, Dk, Dv)) if S0 is None else _f64(S0)[n].copy()
        states = [M]
        for t in range(cu[n], cu[n + 1]):
            D = alpha[t][:, :, None] * M
            e = v[t] - np.einsum("hkv,hk->hv", D, k[t])
            M = D + k[t][:, :, None] * (beta[t][:, None] * e)[:, None, :]
            states.append(M)
        dM = np.zeros((H, Dk, Dv)) if dS_out is None else _f64(dS_out)[n].copy()
        for t in range(cu[n + 1] - 1, cu[n] - 1, -1):
            M, prev = states[t - cu[n] + 1], states[t - cu[n]]
            D = alpha[t][:, :, None] * prev
            e = v[t] - np.einsum("hkv,hk->hv", D, k[t])
            res["dq"][t] = np.einsum("hkv,hv->hk", M, dout[t])
            dM = dM + q[t][:, :, None] * dout[t][:, None, :]
            du = np.einsum("hkv,hk->hv", dM, k[t])
            dv = beta[t][:, None] * du
            res["dv"][t] = dv
            res["dbeta"][t] = (du * e).sum(-1)
            res["dk"][t] = np.einsum("hkv,hv->hk", dM, beta[t][:, None] * e) - np.einsum("hkv,hv->hk", D, dv)
            dD = dM - k[t][:, :, None] * dv[:, None, :]
            res["dg"][t] = alpha[t] * (dD * prev).sum(-1)
            dM = alpha[t][:, :, None] * dD
        res["dS0"][n] = dM
    if l2norm_eps is not None:
        res["dq"] = (res["dq"] - q * (q * res["dq"]).sum(-1, keepdims=True)) / nq
        res["dk"] = (res["dk"] - k * (k * res["dk"]).sum(-1, keepdims=True)) / nk
    return res


def output_gate_backward(o, gate, dout, weight=None, eps: float = 1e-6):
    """Gradients (do, dgate, dweight) of ``oracle.output_gate``, [..., H, Dv]."""
    o, z, d = _f64(o), _f64(gate), _f64(dout)
    w = np.ones(o.shape[-1]) if weight is None else _f64(weight)
    rho = np.sqrt(np.mean(o * o, axis=-1, keepdims=True) + eps)
    s, c = 1.0 / (1.0 + np.exp(-z)), 1.0 / (1.0 + np.exp(z))
    dn = d * w * s
    do = dn / rho - o * np.mean(dn * o, axis=-1, keepdims=True) / rho ** 3
    return do, d * w * o / rho * s * c, (d * s * o / rho).reshape(-1, o.shape[-1]).sum(0)


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, rms: bool = False):
    """(y, mean, rstd) of rows x [..., W]; mean is zero for the RMS norm."""
    x = _f64(x)
    mean = np.zeros(x.shape[:-1]) if rms else x.mean(-1)
    c = x - mean[..., None]
    rstd = 1.0 / np.sqrt((c * c).mean(-1) + eps)
    y = c * rstd[..., None]
    if weight is not None:
        y = y * _f64(weight)
    if bias is not None:
        y = y + _f64(bias)
    return y, mean, rstd


def layer_norm_backward(x, dy, weight=None, eps: float = 1e-5, rms: bool = False):
    """(dx, dweight, dbias) of ``layer_norm``."""
    x, dy = _f64(x), _f64(dy)
    W = x.shape[-1]
    _, mean, rstd = layer_norm(x, eps=eps, rms=rms)
    c, r = x - mean[..., None], rstd[..., None]
    h = dy * (1.0 if weight is None else _f64(weight))
    dx = r * h - r ** 3 * c * (h * c).sum(-1, keepdims=True) / W
    if not rms:
        dx = dx - r * h.mean(-1, keepdims=True)
    return dx, (dy * c * r).reshape(-1, W).sum(0), dy.reshape(-1, W).sum(0)
