"""kda_prefill_backward / gdn_prefill_backward against the fp64 reverse-mode recurrence.

Bars, derived before the first run. The kernels compute in fp32: the longest chains of
roundings are sums of at most 128 + 64 terms per product and a handful of products per
chunk, while the state between chunks only contracts, so errors are a few tens of fp32
steps of the tensor's RMS, and dg's sums of up to 64 rows that partly cancel lose another
factor of about ten: 1e-4 x RMS (the fp32 bar of the forward tests) is about 1700 half
steps of 2^-24. A gradient that leaves in bf16 is off by half a bf16 step of its own value,
2^-8 relative, besides.
"""
import sys

import numpy as np
import pytest
import torch

from gated_delta_rule_103_amd import (gdn_prefill_backward, inputs, kda_prefill_backward,
                                      kda_prefill_backward_workspace_size)
from gated_delta_rule_103_amd.kda import KDAError
from kda_testlib import host64, orc_state, to_dev
from oracle import gradients

pytestmark = pytest.mark.gpu
BAR = 1e-4
EPS = 1e-6
NAMES = ("dq", "dk", "dv", "dg", "dbeta", "dS0")


def check(name, got, ref):
    got, ref = host64(got), np.asarray(ref)
    assert got.shape == ref.shape and np.isfinite(got).all(), name
    rms = np.sqrt(np.mean(ref * ref)) if ref.size else 0.0
    return np.abs(got - ref), rms


def assert_close(name, got, ref):
    err, rms = check(name, got, ref)
    half = 2.0 ** -8 * np.abs(ref) if got.dtype == torch.bfloat16 else 0.0
    worst = float((err - half).max()) if err.size else 0.0
    print(f"  {name}: max err {err.max() if err.size else 0:.2e}, rms {rms:.2e}", file=sys.stderr, flush=True)
    assert worst <= BAR * rms, (name, worst, rms)


def draw(gate="channel", s0=True, ds=True, l2=False, dout_io=None, scale=0.05, **kw):
    """A prefill problem, its gate brought to `gate`'s layout, and the gradients that come in."""
    p = inputs.prefill(qk_scale=(0.3, 2.0) if l2 else None, s0_std=0.1 if s0 else None, **kw)
    gen = torch.Generator().manual_seed(kw["seed"] + 1)
    if gate == "head":
        p.g = p.g[..., 0].contiguous()
    elif gate == "none":
        p.g = None
    dout = (torch.randn(p.v.shape, generator=gen) * scale).to(torch.float32 if dout_io == "f32" else p.q.dtype)
    N, H, D = p.num_seqs, p.q.shape[2], p.q.shape[3]
    dS = torch.randn(N, H, D, D, generator=gen) * scale if ds else None
    return p, dout, dS


def reference(p, dout, dS, l2):
    H, D = p.q.shape[2], p.q.shape[3]
    flat = lambda t: host64(t).reshape(-1, H, t.shape[-1])
    g = np.zeros((p.num_tokens, H, D)) if p.g is None else \
        np.repeat(host64(p.g).reshape(-1, H, 1), D, 2) if p.g.dim() == 3 else flat(p.g)
    cu = np.arange(p.q.shape[0] + 1) * p.q.shape[1] if p.cu_seqlens is None else p.cu_seqlens.cpu().numpy()
    r = gradients.recurrent_backward(flat(p.q), flat(p.k), flat(p.v), g, host64(p.beta).reshape(-1, H), flat(dout),
                                     orc_state(p.S0), orc_state(dS), cu, EPS if l2 else None)
    r["dg"] = None if p.g is None else r["dg"].sum(-1) if p.g.dim() == 3 else r["dg"]
    r["dS0"] = orc_state(r["dS0"])
    shaped = dict(dq=p.q, dk=p.k, dv=p.v, dg=p.g, dbeta=p.beta)
    return {n: None if r[n] is None else r[n].reshape(shaped[n].shape) if n in shaped else r[n] for n in NAMES}


def gpu(p, dout, dS, l2=False, **kw):
    d = to_dev(p)
    f = kda_prefill_backward if p.g is not None and p.g.dim() == 4 else gdn_prefill_backward
    if p.S0 is None and "dS0" not in kw:
        kw["dS0"] = torch.empty(p.num_seqs, p.q.shape[2], p.q.shape[3], p.q.shape[3], device="cuda")
    r = f(d.q, d.k, d.v, d.g, d.beta, dout.cuda(), d.S0, None if dS is None else dS.cuda(), cu_seqlens=d.cu_seqlens,
          qk_l2norm=l2, l2norm_eps=EPS, **kw)
    torch.cuda.synchronize()
    return dict(zip(NAMES, r))


def run(l2=False, **kw):
    print(f"prefill_backward {kw} l2={l2}", file=sys.stderr, flush=True)
    p, dout, dS = draw(l2=l2, **kw)
    ref, got = reference(p, dout, dS, l2), gpu(p, dout, dS, l2)
    for n in NAMES:
        if ref[n] is None:
            assert got[n] is None
        else:
            assert_close(n, got[n], ref[n])
    return p, dout, dS, got


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 15, 16, 17, 63, 64, 65, 200])
def test_lengths(D, io, T):
    run(H=2, D=D, B=2, T=T, io=io, seed=T + D)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("gate", ["channel", "head", "none"])
@pytest.mark.parametrize("l2", [False, True])
def test_gates_and_norm(D, io, gate, l2):
    run(H=3, D=D, lengths=[70, 0, 1, 129], io=io, gate=gate, l2=l2, shift=0.0, seed=11)


@pytest.mark.parametrize("s0,ds", [(False, False), (True, False), (False, True)])
def test_states_absent(s0, ds):
    run(H=2, D=64, B=1, T=100, io="f32", s0=s0, ds=ds, seed=5)


@pytest.mark.parametrize("io,beta_io,dout_io", [("bf16", "f32", None), ("bf16", None, "f32"), ("bf16", "f32", "f32")])
def test_mixed_types(io, beta_io, dout_io):
    run(H=2, D=128, B=1, T=80, io=io, beta_io=beta_io, dout_io=dout_io, seed=6)


@pytest.mark.parametrize("shift", [-8.0, -4.0, 0.0, 4.0, 30.0])
@pytest.mark.parametrize("D", [64, 128])
def test_decay_strengths(shift, D):
    """From almost no decay to e^-30 a token, which cuts a channel off from one token to the next."""
    run(H=2, D=D, B=1, T=150, io="f32", shift=shift, seed=7)


@pytest.mark.parametrize("scale", [1e-8, 1e-3, 1e4])
def test_gradient_magnitudes(scale):
    run(H=2, D=128, B=1, T=130, io="bf16", scale=scale, seed=8)


def test_one_head_many_sequences():
    run(H=1, D=64, lengths=[3, 64, 0, 0, 65, 1, 1, 17, 128, 5, 0], io="bf16", seed=9)


def test_odd_head_count_long():
    run(H=5, D=128, B=1, T=700, io="bf16", shift=-4.0, seed=10)


def test_wiped_channels():
    """g = -inf forgets a channel: its gradient is 0, everything else as the definition has it."""
    p, dout, dS = draw(H=2, D=64, B=1, T=140, io="f32", shift=-3.0, seed=12)
    p.g[:, 5, :, :7] = -float("inf")
    p.g[:, 63:66, 0, 20:40] = -float("inf")
    p.g[:, 100, 1] = -1e30
    ref, got = reference(p, dout, dS, False), gpu(p, dout, dS)
    for n in NAMES:
        assert_close(n, got[n], ref[n])
    assert (got["dg"][:, 5, :, :7] == 0).all()


@pytest.mark.parametrize("beta", [0.0, 1.0])
def test_beta_ends(beta):
    """beta = 0 leaves the state alone and dbeta is still the error's."""
    p, dout, dS = draw(H=2, D=64, B=1, T=90, io="f32", shift=0.0, seed=13)
    p.beta.fill_(beta)
    ref, got = reference(p, dout, dS, False), gpu(p, dout, dS)
    for n in NAMES:
        assert_close(n, got[n], ref[n])


def test_repeats_bit_for_bit_and_leaves_other_rows():
    """The same call twice, on another stream, and with buffers of the caller's: the same bits; rows
    behind the last sequence and elements around the buffers stay as they were."""
    p, dout, dS, first = run(H=3, D=128, lengths=[100, 37], io="bf16", seed=14)
    d = to_dev(p)
    T, H, D = p.num_tokens, 3, 128
    pad = lambda t, fill=7.0: torch.cat([t, torch.full((1, 9, *t.shape[2:]), fill, dtype=t.dtype, device=t.device)], 1).contiguous()
    q, k, v, g, beta, do = (pad(t) for t in (d.q, d.k, d.v, d.g, d.beta, dout.cuda()))
    bufs = {n: torch.full_like(t, 3.0) for n, t in dict(dq=q, dk=k, dv=v, dg=g, dbeta=beta).items()}
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    need = kda_prefill_backward_workspace_size(2, T + 9, H, D, D)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    r = kda_prefill_backward(q, k, v, g, beta, do, d.S0, dS.cuda(), cu_seqlens=d.cu_seqlens, workspace=ws, stream=st, **bufs)
    torch.cuda.synchronize()
    for n, x in zip(NAMES, r):
        if n == "dS0":
            assert torch.equal(x, first[n])
        else:
            assert x.data_ptr() == bufs[n].data_ptr()
            assert torch.equal(x[:, :T], first[n]) and (x[:, T:] == 3.0).all()


def test_captured_into_a_graph():
    """Replayed on new inputs, several times, with eager work between."""
    p, dout, dS = draw(H=2, D=128, B=1, T=200, io="bf16", seed=15)
    d = to_dev(p)
    do, ds = dout.cuda(), dS.cuda()
    need = kda_prefill_backward_workspace_size(1, 200, 2, 128, 128)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    call = lambda: kda_prefill_backward(d.q, d.k, d.v, d.g, d.beta, do, d.S0, ds, workspace=ws)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for i in range(3):
        do.copy_(torch.randn(do.shape, device="cuda") * 0.1)
        d.S0.mul_(-0.5)
        graph.replay()
        torch.cuda.synchronize()
        again = [x.clone() for x in got]
        want = kda_prefill_backward(d.q, d.k, d.v, d.g, d.beta, do, d.S0, ds)
        torch.cuda.synchronize()
        for n, a, b in zip(NAMES, again, want):
            assert torch.equal(a, b), (i, n)


def test_dS_out_may_be_absent_and_empty_batch():
    """No tokens at all: dS0 is dS_out."""
    p, dout, dS = draw(H=2, D=64, B=2, T=0, io="f32", seed=16)
    got = gpu(p, dout, dS)
    assert torch.equal(got["dS0"].cpu(), dS)
    assert got["dq"].numel() == 0


def test_refusals():
    p, dout, dS = draw(H=2, D=64, B=1, T=64, io="bf16", seed=17)
    d, do = to_dev(p), dout.cuda()
    with pytest.raises(KDAError, match="WORKSPACE"):
        kda_prefill_backward(d.q, d.k, d.v, d.g, d.beta, do, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(KDAError, match="INVALID_ARG"):
        kda_prefill_backward(d.q, d.k, d.v, d.g, d.beta, do, dq=d.q)
    with pytest.raises(KDAError, match="INVALID_ARG"):
        kda_prefill_backward(d.q, d.k, d.v, d.g, d.beta, do, qk_l2norm=True, l2norm_eps=0.0)
    with pytest.raises(ValueError, match="dg must be None"):
        gdn_prefill_backward(d.q, d.k, d.v, None, d.beta, do, dg=d.g[..., 0].contiguous())


@pytest.mark.parametrize("D,io", [(128, "bf16"), (128, "f32"), (64, "bf16")])
def test_many_chains(D, io):
    """Enough chains for the scan that takes 32 value channels a workgroup, dense and packed."""
    run(H=40 if D == 128 else 80, D=D, B=4, T=70, io=io, shift=-1.0, seed=18)
    run(H=40 if D == 128 else 80, D=D, lengths=[70, 1, 0, 33, 64, 10], io=io, shift=-1.0, seed=19)


def test_offsets_are_cut_and_rows_of_no_sequence_do_not_count():
    """Offsets that fall or leave the rows name what remains when they are cut; NaN in rows of no
    sequence reaches nothing, and their gradients stay as they were."""
    p, dout, dS, first = run(H=2, D=64, lengths=[37, 0, 50], io="bf16", seed=20)
    d, T = to_dev(p), p.num_tokens
    edge = lambda t, n: torch.full((1, n, *t.shape[2:]), float("nan"), dtype=t.dtype, device="cuda")
    for cu, behind in (([3, 40, 20, 500], 0), ([3, 40, -2 ** 31, 90], 70), ([3, 40, 40, 90], 1)):
        pad = lambda t: torch.cat([edge(t, 3), t.cuda(), edge(t, behind)], 1).contiguous()
        ins = [pad(t) for t in (d.q, d.k, d.v, d.g, d.beta, dout)]
        bufs = {n: torch.full_like(t, 3.0) for n, t in zip(("dq", "dk", "dv", "dg", "dbeta"), ins)}
        got = kda_prefill_backward(*ins, d.S0, dS.cuda(), cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"), **bufs)
        torch.cuda.synchronize()
        for n, x in zip(NAMES, got):
            if n == "dS0":
                assert torch.equal(x, first[n]), cu
            else:
                assert torch.equal(x[:, 3:3 + T], first[n]) and (x[:, :3] == 3.0).all() and (x[:, 3 + T:] == 3.0).all(), (cu, n)
    none = kda_prefill_backward(*ins, d.S0, dS.cuda(), cu_seqlens=torch.tensor([500, 7, 7, 7], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(none[5].cpu(), dS)


def test_a_gate_that_is_no_number_is_not_hidden():
    p, dout, dS = draw(H=2, D=64, B=1, T=80, io="f32", seed=21)
    p.g[0, 30, 1, 5] = float("nan")
    got = gpu(p, dout, dS)
    assert got["dg"][0, :, 1].isnan().any() and got["dq"][0, 31:, 1].isnan().any() and got["dS0"][0, 1].isnan().any()
    assert all(torch.isfinite(got[n][:, :, 0]).all() for n in ("dq", "dk", "dv", "dg", "dbeta"))


@pytest.mark.parametrize("scale", [1e-28, 1e25])
@pytest.mark.parametrize("D,io", [(64, "bf16"), (128, "f32")])
def test_gradient_magnitudes_far_from_one(D, io, scale):
    """The gradients are linear in dout and dS_out: far magnitudes lose nothing while the smallest
    part of a value cut in three (2^-16 of it) stays a normal fp32 number."""
    run(H=2, D=D, B=1, T=130, io=io, l2=D == 64, scale=scale, seed=22)
