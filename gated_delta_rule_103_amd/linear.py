"""Linear attention with a decay for each head (lin_*): the binding of its entry points.

S_t = exp(g_t) S_{t-1} + v_t k_t^T, o_t = S_t q_t. q and k may have fewer heads than v (head h
uses head h // (H // Hk)); g is one log-decay per token and head, one per head for all tokens
(a 1-D tensor), or None. As in ``kda``, every call marshals its arguments and runs the library.
"""
from __future__ import annotations

from typing import Optional

import torch

from .kda import (_FLOAT_IO, GATE_FIXED, GATE_HEAD, KDAError, _at, _dt, _expect, _expect_workspace, _running, _same_gpu,
                  _stream, _workspace, load_library)

_F32 = (torch.float32,)


def _heads(q, k, v, dims):
    """Checks q, k [..., Hk, Dk] and v [..., H, Dv] of ``dims`` axes; returns (lead, H, Hk, Dk, Dv)."""
    for name, x in (("q", q), ("v", v)):
        if not isinstance(x, torch.Tensor) or x.dim() != dims:
            raise ValueError(f"{name} must be a {dims}-D tensor [..., heads, channels]")
    lead, (Hk, Dk), (H, Dv) = q.shape[:-2], q.shape[-2:], v.shape[-2:]
    _expect(q, "q", q.shape, _FLOAT_IO)
    _expect(k, "k", q.shape, (q.dtype,))
    _expect(v, "v", (*lead, H, Dv), (q.dtype,))
    return lead, H, Hk, Dk, Dv


def _gate(g, lead, H):
    """Checks a per-head gate; returns its code."""
    fixed = isinstance(g, torch.Tensor) and g.dim() == 1
    _expect(g, "g", (H,) if fixed else (*lead, H), _F32, optional=True)
    return GATE_FIXED if fixed else GATE_HEAD


def _sequences(lead, cu_seqlens):
    if cu_seqlens is None:
        return lead[0]
    if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must be a 1-D tensor of N + 1 >= 2 offsets")
    _expect(cu_seqlens, "cu_seqlens", cu_seqlens.shape, (torch.int32,))
    if lead[0] != 1:
        raise ValueError("packed sequences (cu_seqlens) need B == 1")
    return cu_seqlens.numel() - 1


def lin_prefill_workspace_size(N: int, T_total: int, H: int, Dk: int, Dv: int) -> int:
    return int(load_library().lin_prefill_workspace_size(N, T_total, H, Dk, Dv))


def lin_prefill_backward_workspace_size(N: int, T_total: int, H: int, Hk: int, Dk: int, Dv: int) -> int:
    return int(load_library().lin_prefill_backward_workspace_size(N, T_total, H, Hk, Dk, Dv))


def lin_prefill(q, k, v, g=None, S0=None, *, out=None, S_out=None, cu_seqlens=None, out_dtype: Optional[torch.dtype] = None,
                workspace=None, stream=None, return_state: bool = True):
    """Chunked linear attention. q, k: [B, T, Hk, Dk]; v: [B, T, H, Dv]; g: [B, T, H] or [H] fp32, or None;
    S0: [N, H, Dv, Dk] fp32 or None; cu_seqlens: int32 [N+1] on the device (B == 1) or None. Returns (out
    [B, T, H, Dv], S_out [N, H, Dv, Dk] or None); rows of tokens in no sequence are zero, but left as they
    were in an ``out`` that is given."""
    lib = load_library()
    lead, H, Hk, Dk, Dv = _heads(q, k, v, 4)
    gate, (B, T), N = _gate(g, lead, H), lead, _sequences(lead, cu_seqlens)
    _expect(S0, "S0", (N, H, Dv, Dk), _F32, optional=True)
    _expect(out, "out", v.shape, _FLOAT_IO, optional=True)
    _expect(S_out, "S_out", (N, H, Dv, Dk), _F32, optional=True)
    _expect_workspace(workspace)
    dev = _same_gpu(q=q, k=k, v=v, g=g, S0=S0, out=out, S_out=S_out, cu_seqlens=cu_seqlens, workspace=workspace)
    zero_rows = int(out is None and cu_seqlens is not None)
    with _running(dev, stream):
        if out is None:
            out = torch.empty(v.shape, dtype=out_dtype or q.dtype, device=dev)
        if S_out is None and return_state:
            S_out = torch.empty(N, H, Dv, Dk, dtype=torch.float32, device=dev)
        workspace, ws_bytes = _workspace(int(lib.lin_prefill_workspace_size(N, B * T, H, Dk, Dv)), workspace, dev)
        st = lib.lin_prefill(_at(q), _at(k), _at(v), _at(g), _at(S0), _at(out), _at(S_out), _at(cu_seqlens), N, B, T, H, Hk,
                             Dk, Dv, _dt(q), _dt(out), gate, zero_rows, _at(workspace), ws_bytes, _stream(stream, dev))
    if st != 0:
        raise KDAError(st, "lin_prefill")
    return out, S_out


def lin_prefill_backward(q, k, v, g, dout, S0=None, dS_out=None, *, cu_seqlens=None, dq=None, dk=None, dv=None, dg=None,
                         dS0=None, workspace=None, stream=None):
    """The gradient of lin_prefill: q, k, v, g, S0 and cu_seqlens as given to it, dout [B, T, H, Dv] (q's dtype)
    the gradient of out and dS_out [N, H, Dv, Dk] that of S_out (None: zero). Returns (dq, dk, dv, dg, dS0),
    each of its input's dtype and shape; dg is None without a gate, dS0 when neither S0 nor a buffer for it
    is given. Rows of tokens in no sequence are zero, but left as they were in buffers that the caller gives."""
    lib = load_library()
    lead, H, Hk, Dk, Dv = _heads(q, k, v, 4)
    gate, (B, T), N = _gate(g, lead, H), lead, _sequences(lead, cu_seqlens)
    _expect(dout, "dout", v.shape, (q.dtype,))
    state = (N, H, Dv, Dk)
    for name, x in (("S0", S0), ("dS_out", dS_out), ("dS0", dS0)):
        _expect(x, name, state, _F32, optional=True)
    for name, x, like in (("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
        _expect(x, name, like.shape, (like.dtype,), optional=True)
    if g is None and dg is not None:
        raise ValueError("dg must be None when there is no gate")
    if dg is not None:
        _expect(dg, "dg", g.shape, _F32)
    _expect_workspace(workspace)
    dev = _same_gpu(q=q, k=k, v=v, g=g, dout=dout, S0=S0, dS_out=dS_out, cu_seqlens=cu_seqlens, dq=dq, dk=dk, dv=dv, dg=dg,
                    dS0=dS0, workspace=workspace)
    zero_rows = 0
    if cu_seqlens is not None:
        zero_rows = sum(bit for bit, x in zip((1, 2, 4, 8), (dq, dk, dv, dg)) if x is None)
    with _running(dev, stream):
        dq, dk, dv = (torch.empty_like(like) if x is None else x for x, like in ((dq, q), (dk, k), (dv, v)))
        if dg is None and g is not None:
            dg = torch.empty_like(g)
        if dS0 is None and S0 is not None:
            dS0 = torch.empty_like(S0)
        need = int(lib.lin_prefill_backward_workspace_size(N, B * T, H, Hk, Dk, Dv))
        workspace, ws_bytes = _workspace(need, workspace, dev)
        st = lib.lin_prefill_backward(_at(q), _at(k), _at(v), _at(g), _at(dout), _at(S0), _at(dS_out), _at(dq), _at(dk),
                                      _at(dv), _at(dg), _at(dS0), _at(cu_seqlens), N, B, T, H, Hk, Dk, Dv, _dt(q), gate,
                                      zero_rows, _at(workspace), ws_bytes, _stream(stream, dev))
    if st != 0:
        raise KDAError(st, "lin_prefill_backward")
    return dq, dk, dv, dg, dS0


def lin_decode(q, k, v, g, S, *, out=None, out_dtype: Optional[torch.dtype] = None, stream=None):
    """One token per sequence, S [N, H, Dv, Dk] fp32 updated in place. q, k: [N, Hk, Dk]; v: [N, H, Dv];
    g: [N, H] or [H] fp32, or None. Returns out [N, H, Dv]."""
    lib = load_library()
    lead, H, Hk, Dk, Dv = _heads(q, k, v, 3)
    gate, N = _gate(g, lead, H), lead[0]
    _expect(S, "S", (N, H, Dv, Dk), _F32)
    _expect(out, "out", v.shape, _FLOAT_IO, optional=True)
    dev = _same_gpu(q=q, k=k, v=v, g=g, S=S, out=out)
    with _running(dev, stream):
        if out is None:
            out = torch.empty(v.shape, dtype=out_dtype or q.dtype, device=dev)
        st = lib.lin_decode(_at(q), _at(k), _at(v), _at(g), _at(S), _at(out), N, H, Hk, Dk, Dv, _dt(q), _dt(out), gate,
                            _stream(stream, dev))
    if st != 0:
        raise KDAError(st, "lin_decode")
    return out


def lin_recurrent(q, k, v, g, S, slot_in, slot_out, cu_seqlens, *, out=None, out_dtype: Optional[torch.dtype] = None,
                  stream=None):
    """A few tokens per sequence over a pool of slots S [slots, H, Dv, Dk]: q, k [T, Hk, Dk]; v [T, H, Dv];
    g [T, H] or [H] fp32, or None; cu_seqlens, slot_in and slot_out, and the rule for slots that sequences
    share, as for kda_recurrent. Returns out [T, H, Dv]."""
    lib = load_library()
    lead, H, Hk, Dk, Dv = _heads(q, k, v, 3)
    gate, T = _gate(g, lead, H), lead[0]
    if not isinstance(S, torch.Tensor) or S.dim() != 4:
        raise ValueError("S must be a pool of states [slots, H, Dv, Dk]")
    _expect(S, "S", (S.shape[0], H, Dv, Dk), _F32)
    if cu_seqlens is None:
        raise ValueError("cu_seqlens is required")
    N = _sequences((1,), cu_seqlens)
    _expect(slot_in, "slot_in", (N,), (torch.int32,), optional=True)
    _expect(slot_out, "slot_out", (T,), (torch.int32,), optional=True)
    _expect(out, "out", v.shape, _FLOAT_IO, optional=True)
    dev = _same_gpu(q=q, k=k, v=v, g=g, S=S, cu_seqlens=cu_seqlens, slot_in=slot_in, slot_out=slot_out, out=out)
    zero_rows = int(out is None)        # rows of no sequence: left alone in the caller's out
    with _running(dev, stream):
        if out is None:
            out = torch.empty(v.shape, dtype=out_dtype or q.dtype, device=dev)
        st = lib.lin_recurrent(_at(q), _at(k), _at(v), _at(g), _at(S), _at(out), _at(cu_seqlens), _at(slot_in),
                               _at(slot_out), N, T, H, Hk, Dk, Dv, S.shape[0], _dt(q), _dt(out), gate, zero_rows,
                               _stream(stream, dev))
    if st != 0:
        raise KDAError(st, "lin_recurrent")
    return out
