"""Linear attention, trees and slots where indexes, counts and buffers are largest: many sequences, tensors beyond 2^31 values,
workspaces of exactly the size asked for, calls from several threads. Bars as in test_gpu_linear.py."""
import sys
import threading

import numpy as np
import pytest
import torch

import gated_delta_rule_103_amd as lib
from kda_testlib import host64
from oracle import linear
from test_gpu_linear import close, draw, forward, gates, offsets, on, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,most", [(64, 9), (65, 5), (300, 5), (5000, 2), (9000, 1)])
def test_many_sequences(N, most):
    """Up to thousands of short sequences, empty ones among them, found by segments that span several."""
    lengths = torch.randint(0, most + 1, (N,), generator=torch.Generator().manual_seed(N)).tolist()
    lengths[N // 2] = 400                                   # and a long one in the middle
    cu = offsets(lengths, before=3)
    x, rn = draw(cu[-1] + 2, 1, 1, 64, 64, N, "f32", seed=N)
    o, S = reference(x, cu)
    out, S_out = forward(x, cu)
    close("out", out, o)
    close("S", S_out, S)
    dout, dS = rn(cu[-1] + 2, 1, 64), rn(N, 1, 64, 64)
    batch = {n: on(x[n])[None] for n in "qkvg"}
    got = lib.lin_prefill_backward(batch["q"], batch["k"], batch["v"], batch["g"], on(dout)[None], on(x["S0"]), on(dS),
                                   cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda())
    ref = linear.backward(*(host64(x[n]) for n in "qkv"), gates(x), host64(dout), host64(x["S0"]), host64(dS), cu)
    for name, y in zip(("dq", "dk", "dv", "dg", "dS0"), got):
        close(name, y, ref[name])


@pytest.mark.parametrize("B,T,H,Hk,D,io", [(1, 700, 3, 3, 64, "f32"), (40, 200, 8, 2, 64, "f32"), (3, 130, 16, 16, 128, "bf16"),
                                           (1, 3000, 4, 4, 128, "bf16"), (130, 66, 2, 1, 64, "bf16")])
def test_workspaces_suffice(B, T, H, Hk, D, io):
    """Workspaces of exactly the size asked for, with what lies behind them unchanged; results as with the binding's own."""
    x, rn = draw(B * T, H, Hk, D, D, B, io, seed=T)
    batch = {n: on(x[n]).view(B, T, *x[n].shape[1:]) for n in "qkvg"}
    S0, dS = on(x["S0"]), on(rn(B, H, D, D))
    dout = on(rn(B, T, H, D).to(batch["v"].dtype))

    def guarded(need):
        buf = torch.full((need + 4096,), 77, dtype=torch.uint8, device="cuda")
        return buf, buf[:need]

    for dS_out in (None, dS):
        for packed in (False, True):
            y, d, kw = batch, dout, {}
            if packed:
                y, d = ({n: z.view(1, B * T, *z.shape[2:]) for n, z in batch.items()}, dout.view(1, B * T, H, D))
                kw = dict(cu_seqlens=torch.arange(0, B * T + 1, T, dtype=torch.int32).cuda())
            buf, ws = guarded(lib.lin_prefill_workspace_size(B, B * T, H, D, D))
            a = lib.lin_prefill(y["q"], y["k"], y["v"], y["g"], S0, workspace=ws, **kw)
            assert (buf[ws.numel():] == 77).all()
            assert all(torch.equal(p, q) for p, q in zip(a, lib.lin_prefill(y["q"], y["k"], y["v"], y["g"], S0, **kw)))
            buf, ws = guarded(lib.lin_prefill_backward_workspace_size(B, B * T, H, Hk, D, D))
            a = lib.lin_prefill_backward(y["q"], y["k"], y["v"], y["g"], d, S0, dS_out, workspace=ws, **kw)
            assert (buf[ws.numel():] == 77).all()
            b = lib.lin_prefill_backward(y["q"], y["k"], y["v"], y["g"], d, S0, dS_out, **kw)
            assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_tokens_beyond_32_bits():
    """More than 2^31 values a tensor: the tail of one long call is that of a call that starts there."""
    T, H, D, tail = 262400, 65, 128, 300
    gen = torch.Generator(device="cuda").manual_seed(0)
    q, k, v = (torch.randn(1, T, H, D, generator=gen, device="cuda", dtype=torch.bfloat16).mul_(0.09) for _ in range(3))
    g = torch.full((H,), -0.05, device="cuda")
    print("long call", file=sys.stderr, flush=True)
    out, S = lib.lin_prefill(q, k, v, g)
    _, before = lib.lin_prefill(*(x[:, :T - tail].contiguous() for x in (q, k, v)), g)
    a, b = lib.lin_prefill(*(x[:, T - tail:].contiguous() for x in (q, k, v)), g, before)
    close("out", out[:, T - tail:], host64(a), rounded=2)
    close("S", S, host64(b))
    print("its gradient", file=sys.stderr, flush=True)
    dout = torch.randn(1, T, H, D, generator=gen, device="cuda", dtype=torch.bfloat16).mul_(0.09)
    full = lib.lin_prefill_backward(q, k, v, g, dout)
    part = lib.lin_prefill_backward(*(x[:, T - tail:].contiguous() for x in (q, k, v)), g, dout[:, T - tail:].contiguous(), before)
    for name, x, y in zip(("dq", "dk", "dv"), full, part):
        close(name, x[:, T - tail:], host64(y), rounded=2)


def test_pools_beyond_32_bits():
    """States of the last slots of a pool of more than 2^31 values."""
    slots, H, D = 4200, 32, 128
    pool = torch.zeros(slots, H, D, D, device="cuda")
    x, rn = draw(6, H, H, D, D, seed=1)
    first = (rn(2, H, D, D) * 0.2)
    pool[[4199, 4100]] = first.cuda()
    small = first.cuda()
    d = [on(x[n]) for n in "qkvg"]
    idx = lambda *a: torch.tensor(a, dtype=torch.int32).cuda()
    cu = idx(0, 3, 6)
    a = lib.lin_recurrent(*d, pool, idx(4199, 4100), idx(-1, -1, 4198, -1, -1, 4100), cu)
    b = lib.lin_recurrent(*d, small, idx(0, 1), idx(-1, -1, 0, -1, -1, 1), cu)
    assert torch.equal(a, b) and torch.equal(pool[4198], small[0]) and torch.equal(pool[4100], small[1])
    parent = idx(-1, 0, 0, -1, 0, 1).view(2, 3)
    t = [z.view(2, 3, *z.shape[1:]) for z in d]
    pool2 = pool[[4198, 4100]].clone()
    assert torch.equal(lib.lin_tree(*t, pool, idx(4198, 4100), parent), lib.lin_tree(*t, pool2, idx(0, 1), parent))
    lib.lin_tree_accept(*t[1:], pool, idx(4198, 4100), idx(4197, 4100), parent, idx(2, 1))
    lib.lin_tree_accept(*t[1:], pool2, idx(0, 1), idx(0, 1), parent, idx(2, 1))
    assert torch.equal(pool[4197], pool2[0]) and torch.equal(pool[4100], pool2[1])
    S = torch.zeros(4200, H, D, D, device="cuda")
    S[4199] = first[0].cuda()
    many = [z[:1].expand(4200, *z.shape[1:]).contiguous() for z in d]
    out = lib.lin_decode(*many, S)
    one = first[:1].cuda()
    assert torch.equal(out[4199:], lib.lin_decode(*(z[:1] for z in d), one)) and torch.equal(S[4199], one[0])


def test_threads():
    """Calls from four host threads, each on a stream of its own."""
    x, _ = draw(700, 4, 2, 128, 128, 2, "bf16", seed=2)
    y = {n: on(x[n])[None] for n in "qkvg"}
    cu, S0 = torch.tensor([0, 650, 700], dtype=torch.int32).cuda(), on(x["S0"])
    want = lib.lin_prefill(y["q"], y["k"], y["v"], y["g"], S0, cu_seqlens=cu)
    torch.cuda.synchronize()
    bad = []

    def work():
        try:
            stream = torch.cuda.Stream()
            for _ in range(10):
                got = lib.lin_prefill(y["q"], y["k"], y["v"], y["g"], S0, cu_seqlens=cu, stream=stream)
                stream.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want)):
                    bad.append("differs")
        except Exception as e:  # noqa: BLE001
            bad.append(repr(e))

    threads = [threading.Thread(target=work) for _ in range(4)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not bad


def test_falling_offsets_do_not_fault():
    """Offsets that fall or lie outside the rows: whatever comes back, the call ends and rows of no sequence stay."""
    x, _ = draw(500, 2, 2, 64, 64, 5, "f32", seed=3)
    y = {n: on(x[n])[None] for n in "qkvg"}
    for cu in ([0, 300, 100, 400, 50, 500], [-9, 10, 2 ** 31 - 1, 20, -2 ** 31, 30], [500, 400, 300, 200, 100, 0]):
        c = torch.tensor(cu, dtype=torch.int32).cuda()
        out, S = lib.lin_prefill(y["q"], y["k"], y["v"], y["g"], on(x["S0"]), cu_seqlens=c)
        lib.lin_prefill_backward(y["q"], y["k"], y["v"], y["g"], y["v"], on(x["S0"]), on(x["S0"]), cu_seqlens=c)
        torch.cuda.synchronize()
        assert out.shape == y["v"].shape and np.isfinite(host64(S)).all()
