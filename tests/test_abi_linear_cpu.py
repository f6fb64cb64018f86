"""Refusals of linear attention's, the trees' and the slots' entry points (no GPU needed): the documented status before anything
is launched, and what the binding rejects because the C ABI cannot see it. Every case here is one that must be refused."""
import ctypes

import pytest
import torch

import gated_delta_rule_103_amd as lib_py
from gated_delta_rule_103_amd.kda import Options

INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3
P = [ctypes.c_void_p((i + 1) << 20) for i in range(20)]      # never dereferenced: checks return first
ODD = ctypes.c_void_p(8)


@pytest.fixture(scope="module")
def lib():
    return lib_py.load_library()


def caller(name, **defaults):
    def call(lib, kw):
        a = dict(defaults)
        assert set(kw) <= set(a), kw
        a.update(kw)
        return getattr(lib, name)(*(None if x is None else ctypes.byref(x) if isinstance(x, Options) else x for x in a.values()))
    return call


prefill = caller("lin_prefill", q=P[0], k=P[1], v=P[2], g=P[3], S0=None, out=P[4], S_out=P[5], cu=None, N=1, B=1, T=4096, H=4,
                 Hk=2, Dk=64, Dv=128, io=1, od=1, gate=1, zero=0, ws=None, wsb=0, stream=None)
SIZES = [
    (dict(N=0), INVALID), (dict(B=0), INVALID), (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(Hk=0), INVALID),
    (dict(Hk=3), INVALID), (dict(Hk=8), INVALID), (dict(N=2), INVALID), (dict(B=2, cu=P[6]), INVALID), (dict(io=2), INVALID),
    (dict(gate=0), INVALID), (dict(gate=3), INVALID), (dict(T=2 ** 30), INVALID), (dict(g=ctypes.c_void_p(2)), INVALID),
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(q=ODD), INVALID), (dict(v=ODD), INVALID),
    (dict(S0=ODD), INVALID), (dict(Dk=32), UNSUPPORTED), (dict(Dv=96), UNSUPPORTED), (dict(Dk=256), UNSUPPORTED),
    (dict(T=2 ** 28, H=4), UNSUPPORTED), (dict(), WORKSPACE), (dict(ws=P[7], wsb=1024), WORKSPACE),
    (dict(ws=ctypes.c_void_p(64), wsb=1 << 40), WORKSPACE)]


@pytest.mark.parametrize("kw,status", SIZES + [
    (dict(out=None), INVALID), (dict(out=P[0]), INVALID), (dict(out=P[3]), INVALID), (dict(out=P[5]), INVALID),
    (dict(S_out=P[2]), INVALID), (dict(S_out=ODD), INVALID), (dict(zero=2), INVALID), (dict(od=-1), INVALID),
    (dict(io=0, od=1), UNSUPPORTED)])
def test_lin_prefill(lib, kw, status):
    assert prefill(lib, kw) == status


backward = caller("lin_prefill_backward", q=P[0], k=P[1], v=P[2], g=P[3], dout=P[4], S0=None, dS=None, dq=P[8], dk=P[9], dv=P[10],
                  dg=P[11], dS0=None, cu=None, N=1, B=1, T=4096, H=4, Hk=2, Dk=64, Dv=128, io=1, gate=1, zero=0, ws=None, wsb=0,
                  stream=None)


@pytest.mark.parametrize("kw,status", SIZES + [
    (dict(dout=None), INVALID), (dict(dq=None), INVALID), (dict(dv=None), INVALID), (dict(dg=None), INVALID), (dict(g=None), INVALID),
    (dict(dq=P[0]), INVALID), (dict(dk=P[4]), INVALID), (dict(dv=P[9]), INVALID), (dict(dg=P[3]), INVALID), (dict(dS0=P[2]), INVALID),
    (dict(dS=P[12], dS0=P[12]), INVALID), (dict(zero=16), INVALID), (dict(zero=-1), INVALID), (dict(dq=ODD), INVALID),
    (dict(dS0=ODD), INVALID), (dict(dg=ctypes.c_void_p(2)), INVALID)])
def test_lin_prefill_backward(lib, kw, status):
    assert backward(lib, kw) == status


def test_workspaces(lib):
    f, b = lib.lin_prefill_workspace_size, lib.lin_prefill_backward_workspace_size
    assert f(1, 64, 4, 64, 64) == 0 and f(1, 4096, 4, 128, 128) > f(1, 4096, 4, 64, 128) > 0
    assert b(1, 4096, 4, 2, 64, 64) > b(1, 4096, 4, 4, 64, 64) > 0 and b(1, 0, 4, 4, 64, 64) == 0
    for bad in ((0, 64, 4, 64, 64), (1, -1, 4, 64, 64), (1, 64, 0, 64, 64), (1, 64, 4, 64, 96), (1, 2 ** 28, 4, 64, 64)):
        assert f(*bad) == 0 and b(*bad[:3], 1, *bad[3:]) == 0
    assert b(1, 64, 4, 3, 64, 64) == 0
    size = lib.kda_slots_compact_workspace_size
    assert size(0) == 0 and size(2 ** 30) == 0 and size(100) >= 800


decode = caller("lin_decode", q=P[0], k=P[1], v=P[2], g=P[3], S=P[4], out=P[5], N=2, H=4, Hk=2, Dk=64, Dv=128, io=1, od=1, gate=1,
                stream=None)
recurrent = caller("lin_recurrent", q=P[0], k=P[1], v=P[2], g=P[3], S=P[4], out=P[5], cu=P[6], si=P[7], so=P[8], N=2, T=5, H=4, Hk=2,
                   Dk=64, Dv=128, slots=3, io=1, od=1, gate=1, zero=0, stream=None)
STEP = [(dict(q=None), INVALID), (dict(S=None), INVALID), (dict(out=None), INVALID), (dict(N=0), INVALID), (dict(H=0), INVALID),
        (dict(Hk=3), INVALID), (dict(gate=0), INVALID), (dict(io=2), INVALID), (dict(od=2), INVALID), (dict(S=ODD), INVALID),
        (dict(out=ODD), INVALID), (dict(out=P[4]), INVALID), (dict(out=P[1]), INVALID), (dict(S=P[2]), INVALID),
        (dict(Dk=32), UNSUPPORTED), (dict(N=2 ** 20, H=4096, Hk=1), UNSUPPORTED)]


@pytest.mark.parametrize("kw,status", STEP)
def test_lin_decode(lib, kw, status):
    assert decode(lib, kw) == status


@pytest.mark.parametrize("kw,status", STEP + [(dict(cu=None), INVALID), (dict(T=-1), INVALID), (dict(slots=0), INVALID),
                                              (dict(zero=2), INVALID), (dict(T=2 ** 30), INVALID)])
def test_lin_recurrent(lib, kw, status):
    assert recurrent(lib, kw) == status


kda_tree = caller("kda_tree", q=P[0], k=P[1], v=P[2], g=P[3], beta=P[4], S=P[5], out=P[6], si=P[7], parent=P[8], N=2, T=9, H=4, Dk=64,
                  Dv=64, slots=3, io=1, bd=1, od=1, zero=0, opt=None, stream=None)
kda_accept = caller("kda_tree_accept", k=P[1], v=P[2], g=P[3], beta=P[4], S=P[5], si=P[7], so=P[9], parent=P[8], node=P[10], N=2, T=9,
                    H=4, Dk=64, Dv=64, slots=3, io=1, bd=1, opt=None, stream=None)
lin_tree = caller("lin_tree", q=P[0], k=P[1], v=P[2], g=P[3], S=P[5], out=P[6], si=P[7], parent=P[8], N=2, T=9, H=4, Hk=2, Dk=64,
                  Dv=128, slots=3, io=1, od=1, gate=1, zero=0, stream=None)
lin_accept = caller("lin_tree_accept", k=P[1], v=P[2], g=P[3], S=P[5], si=P[7], so=P[9], parent=P[8], node=P[10], N=2, T=9, H=4, Hk=2,
                    Dk=64, Dv=128, slots=3, io=1, gate=1, stream=None)
TREE = [(dict(k=None), INVALID), (dict(v=None), INVALID), (dict(S=None), INVALID), (dict(parent=None), INVALID), (dict(N=0), INVALID),
        (dict(T=0), INVALID), (dict(H=0), INVALID), (dict(slots=0), INVALID), (dict(io=2), INVALID), (dict(k=ODD), INVALID),
        (dict(S=ODD), INVALID), (dict(T=65), UNSUPPORTED), (dict(Dk=32), UNSUPPORTED), (dict(N=2 ** 12, H=2 ** 11), UNSUPPORTED),
        (dict(N=2 ** 26, T=64), INVALID)]
DELTA = [(dict(beta=None), INVALID), (dict(g=None), INVALID), (dict(bd=2), INVALID), (dict(Dv=128), UNSUPPORTED), (dict(g=ODD), INVALID),
         (dict(opt=Options(gate=2)), INVALID), (dict(opt=Options(qk_l2norm=1)), INVALID), (dict(opt=Options(snapshots=1 << 20)), INVALID)]
LIN = [(dict(gate=0), INVALID), (dict(gate=4), INVALID), (dict(Hk=3), INVALID), (dict(Dv=32), UNSUPPORTED),
       (dict(g=ctypes.c_void_p(2)), INVALID)]
OUT = [(dict(q=None), INVALID), (dict(out=None), INVALID), (dict(out=P[5]), INVALID), (dict(out=P[8]), INVALID), (dict(zero=3), INVALID),
       (dict(od=7), INVALID), (dict(out=ODD), INVALID)]
KEEP = [(dict(so=None), INVALID), (dict(node=None), INVALID)]


@pytest.mark.parametrize("call,kw,status", [(c, *x) for c, l in ((kda_tree, TREE + DELTA + OUT), (lin_tree, TREE + LIN + OUT),
                                                                (kda_accept, TREE + DELTA + KEEP), (lin_accept, TREE + LIN + KEEP))
                                            for x in l])
def test_trees(lib, call, kw, status):
    assert call(lib, kw) == status


copy = caller("kda_slots_copy", frm=P[0], to=P[1], src=P[2], dst=P[3], n=2, layers=1, fs=4, ts=4, size=64, stream=None)
compact = caller("kda_slots_compact", pool=P[0], uses=P[1], table=P[2], count=P[3], tn=4, layers=1, slots=4, size=64, ws=P[4], wsb=1024,
                 stream=None)


@pytest.mark.parametrize("call,kw,status", [(copy, *x) for x in [
    (dict(frm=None), INVALID), (dict(to=None), INVALID), (dict(src=None), INVALID), (dict(dst=None), INVALID), (dict(n=-1), INVALID),
    (dict(layers=0), INVALID), (dict(fs=0), INVALID), (dict(ts=0), INVALID), (dict(size=0), INVALID), (dict(size=24), INVALID),
    (dict(frm=ODD), INVALID), (dict(to=P[0], ts=5), INVALID), (dict(n=2 ** 24), UNSUPPORTED),
    (dict(n=2 ** 20, size=1 << 20), UNSUPPORTED)]] + [(compact, *x) for x in [
        (dict(pool=None), INVALID), (dict(uses=None), INVALID), (dict(count=None), INVALID), (dict(table=None), INVALID),
        (dict(tn=-1), INVALID), (dict(slots=0), INVALID), (dict(size=8), INVALID), (dict(count=P[1]), INVALID),
        (dict(table=P[1]), INVALID), (dict(pool=ODD), INVALID), (dict(ws=None), WORKSPACE), (dict(wsb=16), WORKSPACE),
        (dict(ws=ODD), WORKSPACE), (dict(slots=2 ** 25), UNSUPPORTED)]])
def test_slots(lib, call, kw, status):
    assert call(lib, kw) == status


@pytest.mark.parametrize("name", ["kda_slots_share", "kda_slots_release", "kda_slots_acquire"])
def test_counts(lib, name):
    f = getattr(lib, name)
    for bad in ((None, P[1], 1, 4), (P[0], None, 1, 4), (P[0], P[1], -1, 4), (P[0], P[1], 1, 0), (P[0], P[0], 1, 4)):
        assert f(*bad, None) == INVALID


def test_largest_counts(lib):
    big = 2 ** 31 - 1                                       # an index a stride further would pass 32 bits
    for name in ("kda_slots_share", "kda_slots_release", "kda_slots_acquire"):
        assert getattr(lib, name)(P[0], P[1], big, 4, None) == INVALID
    assert lib.kda_slots_acquire(P[0], P[1], 1, big, None) == INVALID
    assert compact(lib, dict(tn=big)) == INVALID
    # 9000 states of 32 MB, 302 GB: refused for the missing workspace only
    assert compact(lib, dict(slots=9000, size=32 << 20, ws=None)) == WORKSPACE
    with pytest.raises(ValueError, match="n must be a count"):
        lib_py.kda_slots_acquire(torch.zeros(4, dtype=torch.int32), 2 ** 30)
    with pytest.raises(ValueError, match="which must have fewer than"):
        lib_py.kda_slots_share(torch.zeros(4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32).expand(2 ** 30))
    with pytest.raises(ValueError, match="table must have fewer than"):
        lib_py.kda_slots_compact(torch.zeros(4, 1, 64, 64), torch.zeros(4, dtype=torch.int32),
                                 torch.zeros(1, dtype=torch.int32).expand(2, 2 ** 30))


def test_binding_refuses():
    z = lambda *s, d=torch.bfloat16: torch.zeros(*s, dtype=d)
    f, i = torch.float32, torch.int32
    q, v, g = z(1, 8, 2, 64), z(1, 8, 4, 128), z(1, 8, 4, d=f)
    pre, back = lib_py.lin_prefill, lib_py.lin_prefill_backward
    with pytest.raises(ValueError, match="q must be a 4-D"):
        pre(q[0], q, v, g)
    with pytest.raises(ValueError, match="k must have shape"):
        pre(q, v, v, g)
    with pytest.raises(ValueError, match="g must have shape"):
        pre(q, q, v, g[..., :2])
    with pytest.raises(ValueError, match="g must have shape"):
        pre(q, q, v, g[0, 0, :2])
    with pytest.raises(ValueError, match="g must be one of"):
        pre(q, q, v, g.double())
    with pytest.raises(ValueError, match="v must be one of"):
        pre(q, q, v.float(), g)
    with pytest.raises(ValueError, match="S0 must have shape"):
        pre(q, q, v, g, z(1, 4, 64, 128, d=f))
    with pytest.raises(ValueError, match="cu_seqlens must be one of"):
        pre(q, q, v, g, cu_seqlens=torch.tensor([0, 8]))
    with pytest.raises(ValueError, match="need B == 1"):
        pre(*(x.expand(2, *x.shape[1:]) for x in (q, q, v, g)), cu_seqlens=torch.tensor([0, 8], dtype=i))
    with pytest.raises(ValueError, match="workspace must be"):
        pre(q, q, v, g, workspace=z(9))
    with pytest.raises(ValueError, match="must be a GPU tensor"):
        pre(q, q, v, g)
    with pytest.raises(ValueError, match="dout must have shape"):
        back(q, q, v, g, q)
    with pytest.raises(ValueError, match="dg must be None"):
        back(q, q, v, None, v, dg=g)
    with pytest.raises(ValueError, match="dq must have shape"):
        back(q, q, v, g, v, dq=v)
    with pytest.raises(ValueError, match="S must have shape"):
        lib_py.lin_decode(q[0], q[0], v[0], g[0], z(8, 4, 64, 128, d=f))
    with pytest.raises(ValueError, match="cu_seqlens is required"):
        lib_py.lin_recurrent(q[0], q[0], v[0], g[0], z(3, 4, 128, 64, d=f), None, None, None)
    k, S, par = z(2, 5, 4, 64), z(3, 4, 64, 64, d=f), z(2, 5, d=i)
    with pytest.raises(ValueError, match="parent must have shape"):
        lib_py.kda_tree(k, k, k, z(2, 5, 4, 64, d=f), z(2, 5, 4), S, None, par[:1])
    with pytest.raises(ValueError, match="parent must be one of"):
        lib_py.kda_tree(k, k, k, z(2, 5, 4, 64, d=f), z(2, 5, 4), S, None, par.long())
    with pytest.raises(ValueError, match="g is required"):
        lib_py.kda_tree(k, k, k, None, z(2, 5, 4), S, None, par)
    with pytest.raises(ValueError, match="g must have shape"):
        lib_py.gdn_tree(k, k, k, z(2, 5, 4, 64, d=f), z(2, 5, 4), S, None, par)
    with pytest.raises(ValueError, match="k must have shape"):
        lib_py.gdn_tree(k[:, :, :2], k[:, :, :2], k, None, z(2, 5, 4), S, None, par)
    with pytest.raises(ValueError, match="node must have shape"):
        lib_py.lin_tree_accept(k, k, None, S, None, z(2, d=i), par, z(3, d=i))
    with pytest.raises(ValueError, match="slot_out is required"):
        lib_py.lin_tree_accept(k, k, None, S, None, None, par, z(2, d=i))
    with pytest.raises(ValueError, match="must be a GPU tensor"):
        lib_py.lin_tree(k, k, k, None, S, None, par)
    u = z(3, d=i)
    with pytest.raises(ValueError, match="pool must be a pool"):
        lib_py.kda_slots_copy(S[0], u, u)
    with pytest.raises(ValueError, match="src must be a 1-D"):
        lib_py.kda_slots_copy(S, None, u)
    with pytest.raises(ValueError, match="n must be a count"):
        lib_py.kda_slots_acquire(u, -1)
    with pytest.raises(ValueError, match="uses must be one of"):
        lib_py.kda_slots_release(u.long(), u)
    with pytest.raises(ValueError, match="pool is empty"):
        lib_py.kda_slots_compact(S[:0], u)
    with pytest.raises(ValueError, match="must be a GPU tensor"):
        lib_py.kda_slots_compact(S, u)
