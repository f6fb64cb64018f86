"""The operators together, as a KDA block uses them.

Training: norm, projections, chunked recurrence with normalised q and k, output gate, and
the whole way back, against torch's reverse mode through the per-token definition in fp64
on the CPU. Bar: five operators in a row, each good to 1e-4 of its RMS (1e-5 for the
pointwise ones), through linear maps whose norms are of order 1 here: 1e-3 x RMS.

Serving: a prompt's prefill, then drafts checked with every state kept, then decoding from
the accepted state, against one long prefill.
"""
import numpy as np
import pytest
import torch

from gated_delta_rule_103_amd import (inputs, kda_decode, kda_layer_norm, kda_layer_norm_backward, kda_output_gate,
                                      kda_output_gate_backward, kda_prefill, kda_prefill_backward, kda_recurrent)
from kda_testlib import host64

pytestmark = pytest.mark.gpu


def _reference(x, wn, bn, W, wo, d, H, D):
    """Gradients of sum(block(x) * d) by autograd, fp64, token by token."""
    T = x.shape[0]
    leaves = [t.double().requires_grad_() for t in (x, wn, bn, W, wo)]
    x, wn, bn, W, wo = leaves
    y = (x - x.mean(-1, keepdim=True)) / torch.sqrt(x.var(-1, unbiased=False, keepdim=True) + 1e-5) * wn + bn
    z = y @ W
    q, k, v, gz, og = (z[:, i * H * D:(i + 1) * H * D].view(T, H, D) for i in range(5))
    beta = torch.sigmoid(z[:, 5 * H * D:])
    q, k = (a / torch.sqrt((a * a).sum(-1, keepdim=True) + 1e-6) for a in (q, k))
    alpha = torch.exp(-torch.nn.functional.softplus(gz))
    S, outs = torch.zeros(H, D, D, dtype=torch.float64), []
    for t in range(T):
        Sp = S * alpha[t][:, None, :]
        u = beta[t][:, None] * (v[t] - (Sp * k[t][:, None, :]).sum(-1))
        S = Sp + u[:, :, None] * k[t][:, None, :]
        outs.append((S * q[t][:, None, :]).sum(-1))
    o = torch.stack(outs)
    r = o / torch.sqrt((o * o).mean(-1, keepdim=True) + 1e-6) * wo * torch.sigmoid(og)
    (r * d.double()).sum().backward()
    return [r.detach()] + [t.grad for t in leaves]


@pytest.mark.parametrize("T", [1, 70, 133])
def test_training_step_of_a_block(T):
    H, D, width = 2, 64, 200
    gen = torch.Generator().manual_seed(T)
    rn = lambda *s: torch.randn(*s, generator=gen)
    x, wn, bn, wo = rn(T, width) + 0.2, 1 + 0.1 * rn(width), 0.1 * rn(width), 1 + 0.1 * rn(D)
    W, d = rn(width, 5 * H * D + H) / width ** 0.5, 0.1 * rn(T, H, D)
    ref = _reference(x, wn, bn, W, wo, d, H, D)

    x, wn, bn, W, wo, d = (t.cuda() for t in (x, wn, bn, W, wo, d))
    y, mean, rstd = kda_layer_norm(x, wn, bn)
    z = y @ W
    cut = lambda a, i: a[:, i * H * D:(i + 1) * H * D].reshape(1, T, H, D).contiguous()
    q, k, v, gz, og = (cut(z, i) for i in range(5))
    beta, g = torch.sigmoid(z[:, 5 * H * D:])[None].contiguous(), -torch.nn.functional.softplus(gz)
    o, _ = kda_prefill(q, k, v, g, beta, qk_l2norm=True)
    r = kda_output_gate(o, og, wo)

    do, dog, dwo = kda_output_gate_backward(o, og, d[None].contiguous(), wo)
    dq, dk, dv, dg, dbeta, dS0 = kda_prefill_backward(q, k, v, g, beta, do, qk_l2norm=True)
    assert dS0 is None
    dgz, dbz = -dg * torch.sigmoid(gz), dbeta * beta * (1 - beta)
    dz = torch.cat([a.reshape(T, H * D) for a in (dq, dk, dv, dgz, dog)] + [dbz.reshape(T, H)], 1)
    dW, dy = y.t() @ dz, dz @ W.t()
    dx, dwn, dbn = kda_layer_norm_backward(x, dy, mean, rstd, wn, bias=True)
    torch.cuda.synchronize()
    for name, got, want in zip(("out", "dx", "dwn", "dbn", "dW", "dwo"), (r[0], dx, dwn, dbn, dW, dwo), ref):
        want = want.numpy()
        err, rms = np.abs(host64(got) - want).max(), np.sqrt(np.mean(want * want))
        assert err <= 1e-3 * rms, (name, err, rms)


def test_drafts_checked_and_continued():
    H, D, N, T, drafts, accepted = 4, 128, 3, 100, 4, 2
    p = inputs.prefill(H, D, B=N, T=T + drafts, io="bf16", shift=0.0, seed=3)
    q, k, v, g, beta = (t.cuda() for t in (p.q, p.k, p.v, p.g, p.beta))
    part = lambda a, b: [t[:, a:b].contiguous() for t in (q, k, v, g, beta)]
    flat = lambda a, b: [t.reshape(-1, *t.shape[2:]).contiguous() for t in part(a, b)]
    _, S = kda_prefill(*part(0, T))
    pool = torch.empty(N * (1 + drafts), H, D, D, device="cuda")
    pool[:N] = S
    cu = torch.arange(N + 1, dtype=torch.int32).cuda() * drafts
    slot_in = torch.arange(N, dtype=torch.int32).cuda()
    slot_out = N + torch.arange(N * drafts, dtype=torch.int32).cuda()
    out = kda_recurrent(*flat(T, T + drafts), pool, slot_in, slot_out, cu, out_dtype=torch.float32)
    taken = pool[N + torch.arange(N).cuda() * drafts + accepted - 1].contiguous()      # the state behind the accepted drafts
    nxt = kda_decode(*flat(T + accepted, T + accepted + 1), taken, out_dtype=torch.float32)
    long_out, long_S = kda_prefill(*part(0, T + accepted + 1), out_dtype=torch.float32)
    torch.cuda.synchronize()
    # the chunked path's own bar against the definition: 2e-2 x RMS for out, 5e-3 for states
    for got, want, bar in ((out.view(N, drafts, H, D)[:, :accepted], long_out[:, T:T + accepted], 2e-2),
                           (nxt, long_out[:, -1], 2e-2), (taken, long_S, 5e-3)):
        assert (got - want).abs().max() <= bar * want.square().mean().sqrt()


@pytest.mark.parametrize("raw", [False, True])
def test_buffers_belong_to_the_given_stream(raw):
    """The caller's stream still has to fill (and has already freed) memory of the sizes that the
    calls allocate: a call on another stream must not be given that memory."""
    x = torch.randn(512, 512, device="cuda")
    o, z, d = (torch.randn(512, 4, 128, device="cuda") for _ in range(3))
    w = torch.ones(128, device="cuda")
    want = kda_layer_norm(x), kda_output_gate_backward(o, z, d, w)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    for _ in range(3):
        torch.cuda._sleep(20_000_000)
        junk = [torch.full(s, float("nan"), device="cuda") for s in ((512, 512), (512,), (512,), o.shape, o.shape, (128,))]
        junk.append(torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda"))
        del junk
        stream = st.cuda_stream if raw else st
        got = kda_layer_norm(x, stream=stream), kda_output_gate_backward(o, z, d, w, stream=stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for g, t in zip(got, want) for a, b in zip(g, t))
        del got
