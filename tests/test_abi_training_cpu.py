"""Refusals of the gradient, recurrent and norm entry points (no GPU needed): the C ABI
returns the documented status before launching anything, and the Python binding rejects
tensors that the C ABI cannot check. Every case here is one that must be refused."""
import ctypes

import pytest
import torch

import gated_delta_rule_103_amd as lib_py
from gated_delta_rule_103_amd.kda import Options

INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3
P = [ctypes.c_void_p((i + 1) << 20) for i in range(20)]      # never dereferenced: checks return first


@pytest.fixture(scope="module")
def lib():
    return lib_py.load_library()


def _backward(lib, **kw):
    a = dict(q=P[0], k=P[1], v=P[2], g=P[3], beta=P[4], dout=P[5], S0=None, dS=None, dq=P[6], dk=P[7], dv=P[8], dg=P[9],
             db=P[10], dS0=None, cu=None, N=1, B=1, T=64, H=2, Dk=64, Dv=64, io=1, bd=1, dd=1, opt=None, ws=None, wsb=0)
    a.update(kw)
    opt = None if a["opt"] is None else ctypes.byref(a["opt"])
    return lib.kda_prefill_backward(*(a[n] for n in ("q", "k", "v", "g", "beta", "dout", "S0", "dS", "dq", "dk", "dv",
                                                     "dg", "db", "dS0", "cu", "N", "B", "T", "H", "Dk", "Dv", "io",
                                                     "bd", "dd")), opt, a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INVALID), (dict(dout=None), INVALID), (dict(dq=None), INVALID), (dict(db=None), INVALID),
    (dict(g=None), INVALID), (dict(dg=None), INVALID),
    (dict(g=None, dg=P[9], opt=Options(gate=1)), INVALID),       # no gate has no gradient
    (dict(dg=None, opt=Options(gate=1)), INVALID),               # a gate has one
    (dict(N=0), INVALID), (dict(H=0), INVALID), (dict(T=-1), INVALID), (dict(N=2), INVALID), (dict(B=2, cu=P[11]), INVALID),
    (dict(io=2), INVALID), (dict(bd=-1), INVALID), (dict(dd=5), INVALID), (dict(T=2 ** 30), INVALID),
    (dict(opt=Options(gate=2)), INVALID), (dict(opt=Options(qk_l2norm=1)), INVALID),
    (dict(opt=Options(snapshots=1 << 20, snapshot_every=64, max_snapshots=1)), INVALID),
    (dict(q=ctypes.c_void_p(8)), INVALID), (dict(dout=ctypes.c_void_p(24)), INVALID), (dict(dv=ctypes.c_void_p(4)), INVALID),
    (dict(g=ctypes.c_void_p(20)), INVALID), (dict(g=ctypes.c_void_p(18), opt=Options(gate=1)), INVALID),
    (dict(dS0=ctypes.c_void_p(8)), INVALID),
    (dict(dq=P[0]), INVALID), (dict(dv=P[5]), INVALID), (dict(dq=P[7]), INVALID), (dict(dS=P[12], dS0=P[12]), INVALID),
    (dict(Dk=96, Dv=96), UNSUPPORTED), (dict(Dk=64, Dv=128), UNSUPPORTED), (dict(io=0, bd=1, dd=0), UNSUPPORTED),
    (dict(io=0, bd=0, dd=1), UNSUPPORTED), (dict(H=70000, Dk=128, Dv=128), UNSUPPORTED),
    (dict(T=2 ** 29, H=64), UNSUPPORTED),                        # more chunks than one launch has workgroups
    (dict(), WORKSPACE), (dict(ws=P[13], wsb=1024), WORKSPACE), (dict(ws=ctypes.c_void_p(64), wsb=1 << 40), WORKSPACE),
])
def test_prefill_backward(lib, kw, status):
    assert _backward(lib, **kw) == status


def test_prefill_backward_workspace(lib):
    size = lib.kda_prefill_backward_workspace_size
    assert size(1, 64, 1, 64, 64) > 0 and size(1, 0, 1, 128, 128) > 0
    assert size(3, 1000, 8, 128, 128) > size(1, 1000, 8, 128, 128) > size(1, 1000, 8, 64, 64)
    for bad in ((0, 64, 1, 64, 64), (1, -1, 1, 64, 64), (1, 64, 0, 64, 64), (1, 64, 1, 64, 128), (1, 2 ** 29, 64, 64, 64)):
        assert size(*bad) == 0


def _recurrent(lib, **kw):
    a = dict(q=P[0], k=P[1], v=P[2], g=P[3], beta=P[4], S=P[5], out=P[6], cu=P[7], si=P[8], so=P[9], N=2, T=5, H=2, Dk=64,
             Dv=64, slots=3, io=1, bd=1, od=1, opt=None)
    a.update(kw)
    opt = None if a["opt"] is None else ctypes.byref(a["opt"])
    return lib.kda_recurrent(*(a[n] for n in ("q", "k", "v", "g", "beta", "S", "out", "cu", "si", "so", "N", "T", "H",
                                              "Dk", "Dv", "slots", "io", "bd", "od")), opt, None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INVALID), (dict(S=None), INVALID), (dict(cu=None), INVALID), (dict(out=None), INVALID), (dict(g=None), INVALID),
    (dict(N=0), INVALID), (dict(T=-1), INVALID), (dict(slots=0), INVALID), (dict(H=0), INVALID), (dict(io=3), INVALID),
    (dict(T=2 ** 30), INVALID), (dict(q=ctypes.c_void_p(8)), INVALID), (dict(S=ctypes.c_void_p(8)), INVALID),
    (dict(out=P[2]), INVALID), (dict(out=P[5]), INVALID), (dict(opt=Options(qk_l2norm=1, l2norm_eps=0.0)), INVALID),
    (dict(opt=Options(snapshots=1 << 20)), INVALID), (dict(Dk=32, Dv=32), UNSUPPORTED), (dict(Dk=64, Dv=128), UNSUPPORTED),
    (dict(N=2 ** 20, H=4096), UNSUPPORTED),
])
def test_recurrent(lib, kw, status):
    assert _recurrent(lib, **kw) == status


def _gate(lib, **kw):
    a = dict(o=P[0], z=P[1], d=P[2], w=P[3], do=P[4], dz=P[5], dw=P[6], rows=400, H=2, Dv=64, eps=1e-6, od=1, zd=1, dd=1,
             ws=None, wsb=0)
    a.update(kw)
    return lib.kda_output_gate_backward(*(a[n] for n in ("o", "z", "d", "w", "do", "dz", "dw", "rows", "H", "Dv", "eps",
                                                         "od", "zd", "dd", "ws", "wsb")), None)


@pytest.mark.parametrize("kw,status", [
    (dict(o=None), INVALID), (dict(d=None), INVALID), (dict(do=None), INVALID), (dict(rows=-1), INVALID), (dict(H=0), INVALID),
    (dict(eps=0.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(od=2), INVALID), (dict(rows=2 ** 30, H=4), INVALID),
    (dict(o=ctypes.c_void_p(8)), INVALID), (dict(w=ctypes.c_void_p(4)), INVALID), (dict(dw=ctypes.c_void_p(2)), INVALID),
    (dict(do=P[0]), INVALID), (dict(dz=P[2]), INVALID), (dict(dz=P[4]), INVALID), (dict(dw=P[3]), INVALID),
    (dict(Dv=96), UNSUPPORTED), (dict(), WORKSPACE), (dict(ws=P[7], wsb=4), WORKSPACE),
    (dict(ws=ctypes.c_void_p(128), wsb=1 << 30), WORKSPACE),
])
def test_output_gate_backward(lib, kw, status):
    assert _gate(lib, **kw) == status


def _norm(lib, **kw):
    a = dict(x=P[0], w=P[1], b=P[2], y=P[3], m=P[4], r=P[5], rows=4, W=10, eps=1e-5, rms=0, xd=1, yd=1)
    a.update(kw)
    return lib.kda_layer_norm(*(a[n] for n in ("x", "w", "b", "y", "m", "r", "rows", "W", "eps", "rms", "xd", "yd")), None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), INVALID), (dict(y=None), INVALID), (dict(rows=-1), INVALID), (dict(W=0), INVALID), (dict(eps=0.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(xd=2), INVALID), (dict(yd=-1), INVALID), (dict(rms=1), INVALID),   # a mean for RMS
    (dict(x=ctypes.c_void_p(1)), INVALID), (dict(y=ctypes.c_void_p(2), yd=0), INVALID), (dict(w=ctypes.c_void_p(2)), INVALID),
    (dict(y=P[0], yd=0), INVALID), (dict(y=P[1]), INVALID), (dict(m=P[0]), INVALID), (dict(m=P[5]), INVALID),
    (dict(W=16385), UNSUPPORTED),
])
def test_layer_norm(lib, kw, status):
    assert _norm(lib, **kw) == status


def _norm_back(lib, **kw):
    a = dict(x=P[0], dy=P[1], m=P[2], r=P[3], w=P[4], dx=P[5], dw=P[6], db=P[7], rows=400, W=10, rms=0, xd=1, yd=1, ws=None, wsb=0)
    a.update(kw)
    return lib.kda_layer_norm_backward(*(a[n] for n in ("x", "dy", "m", "r", "w", "dx", "dw", "db", "rows", "W", "rms",
                                                        "xd", "yd", "ws", "wsb")), None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), INVALID), (dict(r=None), INVALID), (dict(m=None), INVALID), (dict(rms=1), INVALID), (dict(dx=None), INVALID),
    (dict(rows=-1), INVALID), (dict(W=0), INVALID), (dict(xd=2), INVALID), (dict(dx=P[0]), INVALID), (dict(dx=P[1]), INVALID),
    (dict(dw=P[7]), INVALID), (dict(db=P[4]), INVALID), (dict(dw=P[3]), INVALID), (dict(dy=ctypes.c_void_p(1)), INVALID),
    (dict(W=20000), UNSUPPORTED), (dict(), WORKSPACE), (dict(ws=P[8], wsb=16), WORKSPACE),
    (dict(ws=ctypes.c_void_p(64), wsb=1 << 30), WORKSPACE),
])
def test_layer_norm_backward(lib, kw, status):
    assert _norm_back(lib, **kw) == status


def test_small_workspaces(lib):
    assert 0 < lib.kda_output_gate_backward_workspace_size(2 ** 20, 64, 128) <= 1 << 20
    assert lib.kda_output_gate_backward_workspace_size(1, 1, 96) == 0 and lib.kda_output_gate_backward_workspace_size(-1, 1, 64) == 0
    assert 0 < lib.kda_layer_norm_backward_workspace_size(2 ** 20, 4096) <= 4096 * 4096
    assert lib.kda_layer_norm_backward_workspace_size(4, 16385) == 0
    # a few rows are one workgroup's, which needs none
    assert lib.kda_output_gate_backward_workspace_size(1, 1, 128) == 0 and lib.kda_layer_norm_backward_workspace_size(4, 100) == 0


def test_binding_refuses():
    z = lambda *s, d=torch.bfloat16: torch.zeros(*s, dtype=d)
    f = torch.float32
    q, g, b = z(1, 8, 2, 64), z(1, 8, 2, 64, d=f), z(1, 8, 2)
    back = lib_py.kda_prefill_backward
    with pytest.raises(ValueError, match="dout must have shape"):
        back(q, q, q, g, b, z(1, 8, 2, 32))
    with pytest.raises(ValueError, match="dS_out must have shape"):
        back(q, q, q, g, b, q, dS_out=z(2, 2, 64, 64, d=f))
    with pytest.raises(ValueError, match="dg must have shape"):
        back(q, q, q, g, b, q, dg=g[..., 0])
    with pytest.raises(ValueError, match="dq must be one of"):
        back(q, q, q, g, b, q, dq=g)
    with pytest.raises(ValueError, match="must be a GPU tensor"):
        back(q, q, q, g, b, q)
    t, S, cu = z(3, 2, 64), z(4, 2, 64, 64, d=f), torch.tensor([0, 3], dtype=torch.int32)
    rec = lib_py.kda_recurrent
    with pytest.raises(ValueError, match="cu_seqlens must be one of"):
        rec(t, t, t, t.float(), t[..., 0], S, None, None, cu.long())
    with pytest.raises(ValueError, match="S must be a pool"):
        rec(t, t, t, t.float(), t[..., 0], S[0], None, None, cu)
    with pytest.raises(ValueError, match="g must have shape"):
        lib_py.gdn_recurrent(t, t, t, t.float(), t[..., 0], S, None, None, cu)
    with pytest.raises(ValueError, match="must be a GPU tensor"):
        rec(t, t, t, t.float(), t[..., 0].contiguous(), S, None, None, cu)
    with pytest.raises(ValueError, match="gate must have shape"):
        lib_py.kda_output_gate_backward(t, t[:2], t)
    with pytest.raises(ValueError, match="weight must have shape"):
        lib_py.kda_layer_norm(t, torch.ones(63))
    with pytest.raises(ValueError, match="no mean"):
        lib_py.kda_layer_norm(t, rms=True, mean=torch.zeros(3, 2))
    with pytest.raises(ValueError, match="rstd must have shape"):
        lib_py.kda_layer_norm_backward(t, t, torch.zeros(3, 2), torch.zeros(3))
    with pytest.raises(ValueError, match="must be a GPU tensor"):
        lib_py.kda_layer_norm(t)


def test_binding_refuses_counts_beyond_an_int():
    """Row counts that a C int would cut short (no memory behind these tensors)."""
    for shape in ((2 ** 31, 1), (2 ** 16, 2 ** 16, 1), (1, 2 ** 32 + 8)):
        x = torch.empty(*shape, dtype=torch.bfloat16, device="meta")
        with pytest.raises(ValueError, match="more than the library counts"):
            lib_py.kda_layer_norm(x)
        with pytest.raises(ValueError, match="more than the library counts"):
            lib_py.kda_layer_norm_backward(x, x, None, None, rms=True)
