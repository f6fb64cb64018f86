"""Packed linear attention with offsets that fall or lie outside the rows: with up to 64 sequences the call is that of the offsets
cut to the rows and to the ones before them, and writes every state; with more, nothing outside its buffers is written."""
import numpy as np
import pytest
import torch

import gated_delta_rule_103_amd as lib
from test_gpu_linear import draw, on

pytestmark = pytest.mark.gpu
T, GUARD = 500, 4096


def guarded(shape, dtype):
    """A buffer of 3s for a tensor of ``shape`` inside guards of 3s; the tensor."""
    n = int(np.prod(shape))
    buf = torch.full((n + 2 * GUARD,), 3.0, dtype=dtype, device="cuda")
    return buf, buf[GUARD:GUARD + n].view(shape)


def calls(x, dout, dS, cu):
    """The forward call and the gradient into buffers of 3s (a workspace of NaNs): {name: (buffer, tensor)}."""
    y = {n: on(x[n])[None] for n in "qkv"}
    g = on(x["g"]) if x["g"].dim() == 1 else on(x["g"])[None]
    N, H, Dv, Dk = x["S0"].shape
    Hk = x["q"].shape[1]
    c = torch.tensor(cu, dtype=torch.int64).clamp(-2 ** 31, 2 ** 31 - 1).to(torch.int32).cuda()
    out = {"out": guarded(y["v"].shape, y["v"].dtype), "S_out": guarded((N, H, Dv, Dk), torch.float32),
           **{"d" + n: guarded(y[n].shape, y[n].dtype) for n in "qkv"}, "dg": guarded(g.shape, torch.float32),
           "dS0": guarded((N, H, Dv, Dk), torch.float32)}
    b = {n: t for n, (_, t) in out.items()}
    nans = lambda n: torch.full((n // 4,), float("nan"), device="cuda").view(torch.uint8)
    lib.lin_prefill(y["q"], y["k"], y["v"], g, on(x["S0"]), out=b["out"], S_out=b["S_out"], cu_seqlens=c,
                    workspace=nans(lib.lin_prefill_workspace_size(N, T, H, Dk, Dv)))
    lib.lin_prefill_backward(y["q"], y["k"], y["v"], g, on(dout)[None], on(x["S0"]), on(dS), cu_seqlens=c, dq=b["dq"], dk=b["dk"],
                             dv=b["dv"], dg=b["dg"], dS0=b["dS0"],
                             workspace=nans(lib.lin_prefill_backward_workspace_size(N, T, H, Hk, Dk, Dv)))
    torch.cuda.synchronize()
    for name, (buf, _) in out.items():
        assert (buf[:GUARD] == 3).all() and (buf[-GUARD:] == 3).all(), name
    return b


def falling(N, seed):
    """Offsets that rise by and large and fall here and there."""
    rng = np.random.default_rng(seed)
    return (np.linspace(20, 470, N + 1).astype(int) + rng.integers(-60, 60, N + 1)).tolist()


@pytest.mark.parametrize("cu", [[0, 300, 100, 400, 50, 500], [-9, 10, 2 ** 31 - 1, 20, -2 ** 31, 30], [500, 400, 300, 200, 100, 0],
                                [7, 130, 129, 480], falling(64, 1), falling(33, 2)], ids=lambda c: f"{len(c) - 1}of{c[1]}")
@pytest.mark.parametrize("io,Hk,gate", [("f32", 2, "head"), ("bf16", 1, "head"), ("f32", 1, "fixed")])
def test_cut_to_the_ones_before(cu, io, Hk, gate):
    N = len(cu) - 1
    x, rn = draw(T, 2, Hk, 64, 64, N, io, gate, seed=3)
    dout, dS = rn(T, 2, 64).to(x["v"].dtype), rn(N, 2, 64, 64)
    cut = np.maximum.accumulate(np.clip(cu, 0, T)).tolist()
    got, want = calls(x, dout, dS, cu), calls(x, dout, dS, cut)
    for name in want:
        assert torch.isfinite(want[name]).all() and torch.equal(got[name], want[name]), name
    for name in ("out", "dq", "dk", "dv"):
        assert (got[name][0, :cut[0]] == 3).all() and (got[name][0, cut[-1]:] == 3).all(), name


@pytest.mark.parametrize("N", [65, 300])
def test_many_that_fall_stay_inside(N):
    x, rn = draw(T, 2, 1, 64, 64, N, "f32", "head", seed=4)
    calls(x, rn(T, 2, 64), rn(N, 2, 64, 64), falling(N, N))
