"""The operators together, as a serving loop and a training step use them. Bars: fp32 arithmetic throughout, 1e-4 x RMS;
bf16 results are off by half a step, 2^-8 relative, besides."""
import numpy as np
import pytest
import torch

import gated_delta_rule_103_amd as lib
from kda_testlib import host64
from oracle import linear
from test_gpu_linear import close, draw, gates, on

pytestmark = pytest.mark.gpu


def test_prompts_drafts_forks_and_steps():
    """Three prompts are read, their states put into a pool, two rounds of draft trees checked and accepted in place, one sequence
    forked and one ended, the pool closed up, and a token decoded for each: the states and outputs of the plain recurrence."""
    H, Hk, D, lengths, T = 4, 2, 64, [100, 70, 131], 7
    x, rn = draw(sum(lengths), H, Hk, D, D, io="f32", shift=-1.0, seed=0)
    cu = np.cumsum([0, *lengths])
    batch = {n: on(x[n])[None] for n in "qkvg"}
    i32 = lambda a: torch.tensor(a, dtype=torch.int32).cuda()
    _, S = lib.lin_prefill(batch["q"], batch["k"], batch["v"], batch["g"], cu_seqlens=i32(cu.tolist()))
    _, ref = linear.recurrent(*(host64(x[n]) for n in "qkv"), gates(x), None, cu)
    ref = list(ref)
    pool, uses = torch.full((8, H, D, D), float("nan")).cuda(), i32([1, 0, 1, 0, 0, 1, 0, 0])    # three slots are another's
    slots = lib.kda_slots_acquire(uses, 3)
    assert slots.tolist() == [1, 3, 4]
    lib.kda_slots_copy(S, i32([0, 1, 2]), slots, to=pool)
    pool[[0, 2, 5]] = 0
    for turn in range(2):
        y, _ = draw(3 * T, H, Hk, D, D, io="f32", shift=-1.0, seed=turn + 1)
        t = {n: on(y[n]).view(3, T, *y[n].shape[1:]) for n in "qkvg"}
        parent = [[-1, 0, 0, 1, 1, 2, -1], [-1, -1, 1, 1, 3, 4, 2], [-1, 0, 1, 2, 3, 4, -2]]
        out = lib.lin_tree(t["q"], t["k"], t["v"], t["g"], pool, slots, i32(parent))
        node = [[4, 6, -1], [5, 0, 3]][turn]
        want = []
        for n in range(3):
            z = {m: host64(t[m][n]) for m in "qkvg"}
            want.append(linear.tree(z["q"], z["k"], z["v"], z["g"], None, ref[n], parent[n]))
            ref[n] = linear.tree_states(z["k"], z["v"], z["g"], None, ref[n], parent[n])[node[n]]
        close("tree", out, np.stack(want))
        lib.lin_tree_accept(t["k"], t["v"], t["g"], pool, slots, slots, i32(parent), i32(node))
    # the first sequence forks, the second ends, another's slots are given back
    lib.kda_slots_release(uses, torch.cat([slots[1:2], i32([0, 2, 5])]))
    fork = lib.kda_slots_acquire(uses, 1)
    lib.kda_slots_copy(pool, slots[:1], fork)
    table = torch.cat([slots[:1], slots[2:], fork])
    ref = [ref[0], ref[2], ref[0]]
    count = lib.kda_slots_compact(pool, uses, table)
    assert count.item() == 3 and sorted(table.tolist()) == [0, 1, 2] and uses.tolist() == [1, 1, 1, 0, 0, 0, 0, 0]
    y, _ = draw(3, H, Hk, D, D, io="f32", shift=-1.0, seed=9)
    cu1, o, new = [0, 1, 2, 3], [], []
    out = lib.lin_recurrent(*(on(y[n]) for n in "qkvg"), pool, table, table, i32(cu1))
    for n in range(3):
        one = slice(n, n + 1)
        a, b = linear.recurrent(*(host64(y[m][one]) for m in "qkvg"), ref[n][None])
        o.append(a[0])
        new.append(b[0])
    close("out", out, np.stack(o))
    close("S", pool[table.long()], np.stack(new))


def test_training_step_through_norm_attention_and_gate():
    """Row norm -> linear attention -> output norm and gate, and back through the three gradients, against automatic
    differentiation of the plain formulas in 64 bits."""
    T, H, Hk, D, W = 150, 2, 1, 64, 256
    gen = torch.Generator().manual_seed(5)
    rn = lambda *s: torch.randn(*s, generator=gen)
    leaf = dict(x=rn(T, W), w=1 + 0.1 * rn(W), g=-torch.nn.functional.softplus(rn(T, H)), z=rn(T, H, D), ow=1 + 0.1 * rn(D),
                S0=0.2 * rn(1, H, D, D))
    dy, dS = rn(T, H, D), rn(1, H, D, D)

    c = {n: y.cuda() for n, y in leaf.items()}
    n, mean, rstd = lib.kda_layer_norm(c["x"], c["w"])
    q, k = (n[:, i * D:(i + 1) * D].reshape(1, T, Hk, D).contiguous() * 0.1 for i in (0, 1))
    v = n[:, 2 * D:].reshape(1, T, H, D).contiguous()
    o, S = lib.lin_prefill(q, k, v, c["g"][None], c["S0"])
    y = lib.kda_output_gate(o, c["z"][None], c["ow"])
    do, dz, dow = lib.kda_output_gate_backward(o, c["z"][None], dy.cuda()[None], c["ow"])
    dq, dk, dv, dg, dS0 = lib.lin_prefill_backward(q, k, v, c["g"][None], do, c["S0"], dS.cuda())
    dn = torch.cat([0.1 * dq.reshape(T, D), 0.1 * dk.reshape(T, D), dv.reshape(T, H * D)], 1).contiguous()
    dx, dw, _ = lib.kda_layer_norm_backward(c["x"], dn, mean, rstd, c["w"])

    d = {m: x.double().requires_grad_() for m, x in leaf.items()}
    xc = d["x"] - d["x"].mean(-1, keepdim=True)
    rn_ = xc / torch.sqrt(xc.square().mean(-1, keepdim=True) + 1e-5) * d["w"]
    q, k, v = 0.1 * rn_[:, :D], 0.1 * rn_[:, D:2 * D], rn_[:, 2 * D:].view(T, H, D)
    state, outs = d["S0"][0], []
    for t in range(T):
        state = torch.exp(d["g"][t])[:, None, None] * state + v[t][:, :, None] * k[t][None, None, :]
        outs.append((state * q[t]).sum(-1))
    oo = torch.stack(outs)
    yy = oo / torch.sqrt(oo.square().mean(-1, keepdim=True) + 1e-6) * d["ow"] * torch.sigmoid(d["z"])
    close("y", y, host64(yy))
    close("S", S[0], host64(state))
    ((yy * dy).sum() + (state * dS[0]).sum()).backward()
    for name, got in dict(x=dx, w=dw, g=dg, z=dz, ow=dow, S0=dS0).items():
        close("d" + name, got, host64(d[name].grad))
