"""Refusals of the entry points for padded batches (no GPU needed)."""
import ctypes

import pytest

import gated_delta_rule_103_amd as lib_py
from gated_delta_rule_103_amd.kda import Options

INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3
P = [ctypes.c_void_p((i + 1) << 20) for i in range(20)]      # never dereferenced: checks return first


@pytest.fixture(scope="module")
def lib():
    return lib_py.load_library()


def _backward(lib, **kw):
    a = dict(q=P[0], k=P[1], v=P[2], g=P[3], beta=P[4], dout=P[5], S0=None, dS=None, dq=P[6], dk=P[7], dv=P[8], dg=P[9],
             db=P[10], dS0=None, cu=P[11], N=3, B=1, T=64, H=2, Dk=64, Dv=64, io=1, bd=1, dd=1, zero=31, opt=None, ws=None,
             wsb=0)
    a.update(kw)
    opt = None if a["opt"] is None else ctypes.byref(a["opt"])
    return lib.kda_prefill_backward_padded(*(a[n] for n in ("q", "k", "v", "g", "beta", "dout", "S0", "dS", "dq", "dk", "dv",
                                                            "dg", "db", "dS0", "cu", "N", "B", "T", "H", "Dk", "Dv", "io",
                                                            "bd", "dd", "zero")), opt, a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(zero=32), INVALID), (dict(zero=-1), INVALID), (dict(q=None), INVALID), (dict(dq=P[0]), INVALID),
    (dict(N=0), INVALID), (dict(B=2), INVALID), (dict(dv=ctypes.c_void_p(4)), INVALID), (dict(dg=None), INVALID),
    (dict(opt=Options(gate=2)), INVALID), (dict(Dk=96, Dv=96), UNSUPPORTED), (dict(zero=0), WORKSPACE), (dict(), WORKSPACE),
])
def test_prefill_backward_padded(lib, kw, status):
    assert _backward(lib, **kw) == status


def _recurrent(lib, **kw):
    a = dict(q=P[0], k=P[1], v=P[2], g=P[3], beta=P[4], S=P[5], out=P[6], cu=P[7], si=P[8], so=P[9], N=2, T=5, H=2, Dk=64,
             Dv=64, slots=3, io=1, bd=1, od=1, zero=1, opt=None)
    a.update(kw)
    return lib.kda_recurrent_padded(*(a[n] for n in ("q", "k", "v", "g", "beta", "S", "out", "cu", "si", "so", "N", "T", "H",
                                                     "Dk", "Dv", "slots", "io", "bd", "od", "zero", "opt")), None)


@pytest.mark.parametrize("kw,status", [
    (dict(zero=2), INVALID), (dict(zero=-1), INVALID), (dict(q=None), INVALID), (dict(out=P[2]), INVALID),
    (dict(slots=0), INVALID), (dict(cu=None), INVALID), (dict(Dk=32, Dv=32), UNSUPPORTED), (dict(N=2 ** 20, H=4096), UNSUPPORTED),
])
def test_recurrent_padded(lib, kw, status):
    assert _recurrent(lib, **kw) == status
