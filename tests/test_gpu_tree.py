"""Trees of drafted tokens (outputs and accepted states) against fp64 states kept for every node.

Bar, as max |error| / RMS over a tensor: fp32 arithmetic over paths of at most 64 nodes, each adding
sums of D terms to a state that contracts: 1e-4, the recurrent form's bar; a bf16 result is off by half
a step, 2^-8 relative, besides.
"""
import sys

import numpy as np
import pytest
import torch

import gated_delta_rule_103_amd as lib
import oracle
from kda_testlib import host64
from oracle import linear
from test_gpu_linear import close, on

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def draw(N, T, H, Hk, Dk, Dv, form, gate, io="bf16", l2=False, slots=None, shift=0.0, seed=0):
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=gen)
    qk = [rn(N, T, Hk, Dk) for _ in range(2)]
    qk = [x * y if l2 else torch.nn.functional.normalize(x, dim=-1) for x, y in zip(qk, (1.7, 0.4))]
    g = {"channel": (N, T, H, Dk), "head": (N, T, H), "fixed": (H,), "none": None}[gate]
    return dict(q=qk[0].to(DT[io]), k=qk[1].to(DT[io]), v=rn(N, T, H, Dv).to(DT[io]),
                g=None if g is None else -torch.nn.functional.softplus(rn(*g) + shift),
                beta=None if form == "lin" else torch.sigmoid(rn(N, T, H)).to(DT[io]),
                S=rn(slots or N, H, Dv, Dk) * 0.3), gen


def random_parents(N, T, gen, reach):
    back = torch.randint(1, reach + 1, (N, T), generator=gen)
    return (torch.arange(T) - back).clamp(min=-1).to(torch.int32)


def one(x, n):
    """Sequence n's tensors in fp64."""
    g = x["g"]
    return dict(k=host64(x["k"][n]), v=host64(x["v"][n]), g=None if g is None else host64(g if g.dim() == 1 else g[n]),
                beta=None if x["beta"] is None else host64(x["beta"][n]))


def start(x, slot_in, n):
    s = -1 if slot_in is None else slot_in[n]
    return host64(x["S"][s]) if 0 <= s < x["S"].shape[0] else np.zeros(x["S"].shape[1:])


def references(x, slot_in, parent, l2):
    outs, states = [], []
    for n in range(x["k"].shape[0]):
        y, q = one(x, n), host64(x["q"][n])
        if l2:
            q, y["k"] = oracle.l2norm(q, 1e-6), oracle.l2norm(y["k"], 1e-6)
        S = start(x, slot_in, n)
        outs.append(linear.tree(q, y["k"], y["v"], y["g"], y["beta"], S, parent[n].tolist()))
        states.append(linear.tree_states(y["k"], y["v"], y["g"], y["beta"], S, parent[n].tolist()))
    return np.stack(outs), states


def call(x, form, slot_in, parent, **kw):
    idx = lambda a: None if a is None else torch.tensor(a, dtype=torch.int32).cuda()
    args = [on(x[n]) for n in "qkvg"] + ([] if form == "lin" else [on(x["beta"])])
    return getattr(lib, form + "_tree")(*args, on(x["S"]), idx(slot_in), on(parent), **kw)


def accept(x, form, S, slot_in, slot_out, parent, node, **kw):
    idx = lambda a: None if a is None else torch.tensor(a, dtype=torch.int32).cuda()
    args = [on(x[n]) for n in "kvg"] + ([] if form == "lin" else [on(x["beta"])])
    getattr(lib, form + "_tree_accept")(*args, S, idx(slot_in), idx(slot_out), on(parent), idx(node), **kw)


FORMS = [("kda", "channel", 64, 64), ("kda", "channel", 128, 128), ("gdn", "head", 128, 128), ("gdn", "none", 64, 64),
         ("lin", "head", 64, 128), ("lin", "fixed", 128, 64), ("lin", "none", 128, 128), ("lin", "head", 64, 64)]


@pytest.mark.parametrize("form,gate,Dk,Dv", FORMS)
@pytest.mark.parametrize("T", [1, 5, 16, 17, 32, 33, 64])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_trees(form, gate, Dk, Dv, T, io):
    l2 = form != "lin" and T % 2 == 1
    print(f"tree {form} {gate} {Dk} {Dv} T={T} {io}", file=sys.stderr, flush=True)
    N, H, Hk = 3, 4, 2 if form == "lin" else 4
    x, gen = draw(N, T, H, Hk, Dk, Dv, form, gate, io, l2, slots=7, seed=T + Dk)
    parent = random_parents(N, T, gen, 5)
    slot_in, slot_out = [4, -1, 0], [1, 6, 0]
    ref, states = references(x, slot_in, parent, l2)
    kw = dict(qk_l2norm=True) if l2 else {}
    close("out", call(x, form, slot_in, parent, **kw), ref)
    close("fp32 out", call(x, form, slot_in, parent, out_dtype=torch.float32, **kw), ref)
    node = [T - 1, T // 2, -1 if T % 3 else 0]
    S = on(x["S"])
    before = S.clone()
    accept(x, form, S, slot_in, slot_out, parent, node, **(dict(k_l2norm=True) if l2 else {}))
    close("S", S[slot_out], np.stack([states[n][node[n]] for n in range(N)]))
    rest = [s for s in range(7) if s not in slot_out]
    assert torch.equal(S[rest], before[rest])


@pytest.mark.parametrize("form,gate", [("kda", "channel"), ("gdn", "head"), ("lin", "head")])
def test_chains_are_the_recurrent_form(form, gate):
    """A tree without branches: what the recurrent kernels give, token by token, kept state included."""
    N, T, H, D = 3, 40, 2, 128
    x, _ = draw(N, T, H, H, D, D, form, gate, "bf16", slots=3, shift=-2.0, seed=1)
    parent = (torch.arange(T) - 1).to(torch.int32).repeat(N, 1)
    out = call(x, form, [0, 1, 2], parent, out_dtype=torch.float32)
    flat = [on(x[n].flatten(0, 1)) for n in "qkvg"] + ([] if form == "lin" else [on(x["beta"].flatten(0, 1))])
    cu = torch.arange(0, N * T + 1, T, dtype=torch.int32).cuda()
    S = on(x["S"])
    slots = torch.arange(N, dtype=torch.int32).cuda()
    keep = torch.full((N, T), -1, dtype=torch.int32).cuda()
    keep[:, -1] = slots
    want = getattr(lib, form + "_recurrent")(*flat, S, slots, keep.flatten(), cu, out_dtype=torch.float32)
    close("out", out, host64(want).reshape(out.shape))
    mine = on(x["S"])
    accept(x, form, mine, [0, 1, 2], [0, 1, 2], parent, [T - 1] * N)
    close("S", mine, host64(S))


@pytest.mark.parametrize("N,H", [(1, 1), (1, 33), (70, 4), (300, 1)])
def test_batch_sizes(N, H):
    """Both splits of a state over workgroups."""
    x, gen = draw(N, 7, H, H, 128, 128, "kda", "channel", seed=N)
    parent = random_parents(N, 7, gen, 3)
    ref, _ = references(x, list(range(N)), parent, False)
    close("out", call(x, "kda", list(range(N)), parent), ref)


@pytest.mark.parametrize("form,gate", [("kda", "channel"), ("lin", "head")])
def test_absent_nodes(form, gate):
    """Parents that are no earlier node: the node is absent, and all that descends from it; NaN in its inputs stays there."""
    N, T, H, D = 4, 20, 2, 64
    x, _ = draw(N, T, H, H, D, D, form, gate, "f32", slots=9, seed=2)
    parent = torch.zeros(N, T, dtype=torch.int32)
    parent[0] = torch.tensor([-1, 0, 2, 1, 2, 50, 5, 3, -2, 8, 7, -1, 11, 2 ** 31 - 1, -2 ** 31, 13, 12, 16, 16, 3])
    parent[1] = -2
    parent[2] = torch.arange(T) - 1
    parent[2, 10:] = -2
    parent[3] = torch.arange(T)                             # every node its own parent
    gone = [set(range(T)) - set(s) for s in
            ([0, 1, 3, 7, 10, 11, 12, 16, 17, 18, 19], [], range(10), [])]
    ref, states = references(x, [0, 1, 2, 3], parent, False)
    for n in range(N):
        assert set(states[n]) - {-1} == set(range(T)) - gone[n]
        for t in gone[n]:
            for m in ("q", "k", "v", "g", "beta"):
                if x[m] is not None:
                    x[m][n, t] = float("nan")
    out = call(x, form, [0, 1, 2, 3], parent)
    close("out", out, ref)
    kept = torch.full((N, T, H, D), 3.0).cuda()
    call(x, form, [0, 1, 2, 3], parent, out=kept)
    for n in range(N):
        for t in range(T):
            if t in gone[n]:
                assert (out[n, t] == 0).all() and (kept[n, t] == 3).all()
            else:
                assert torch.equal(out[n, t], kept[n, t])
    S = on(x["S"])
    before = S.clone()
    accept(x, form, S, [0, 1, 2, 3], [5, 6, 7, 8], parent, [6, -1, T, -2])      # absent, the state itself, out of range twice
    assert torch.equal(S[6], before[1]) and torch.equal(S[[0, 1, 2, 3, 4, 5, 7, 8]], before[[0, 1, 2, 3, 4, 5, 7, 8]])
    accept(x, form, S, [0, -1, 99, 3], [-1, 9, 4, 2 ** 31 - 1], parent, [0, -1, -1, -1])  # nowhere to put them; the zero state
    assert (S[4] == 0).all() and torch.equal(S[[0, 1, 2, 3, 5, 7, 8]], before[[0, 1, 2, 3, 5, 7, 8]])
    accept(x, form, S, None, [4, -1, -1, -1], parent, [0, 0, 0, 0])             # no slots to start from
    y = one(x, 0)
    first = linear.tree_states(y["k"][:1], y["v"][:1], y["g"][:1], None if y["beta"] is None else y["beta"][:1],
                               np.zeros((H, D, D)), [-1])[0]
    close("S", S[4], first)


def test_types():
    x, gen = draw(2, 9, 2, 2, 64, 64, "kda", "channel", "f32", seed=3)
    x["beta"] = x["beta"].to(torch.bfloat16)
    parent = random_parents(2, 9, gen, 4)
    ref, states = references(x, [0, 1], parent, False)
    close("bf16 beta and out", call(x, "kda", [0, 1], parent, out_dtype=torch.bfloat16), ref)
    S = on(x["S"])
    accept(x, "kda", S, [0, 1], [0, 1], parent, [8, 4])
    close("S", S, np.stack([states[0][8], states[1][4]]))


def test_wiped_decays():
    x, gen = draw(2, 24, 2, 2, 128, 128, "kda", "channel", "f32", seed=4)
    x["g"][0, 3] = -np.inf
    x["g"][1, ::5] = -1000.0
    parent = random_parents(2, 24, gen, 3)
    ref, _ = references(x, [0, 1], parent, False)
    close("out", call(x, "kda", [0, 1], parent), ref)


def test_graph_replays_and_another_stream():
    x, gen = draw(5, 18, 2, 2, 128, 128, "kda", "channel", slots=10, seed=5)
    parent = on(random_parents(5, 18, gen, 4))
    d = {n: on(y) for n, y in x.items()}
    ins, outs, node = (torch.tensor(a, dtype=torch.int32).cuda() for a in
                       ([0, 1, 2, 3, 4], [5, 6, 7, 8, 9], [17, 3, -1, 9, 11]))

    def step(S, stream=None):
        out = lib.kda_tree(d["q"], d["k"], d["v"], d["g"], d["beta"], S, ins, parent, stream=stream)
        lib.kda_tree_accept(d["k"], d["v"], d["g"], d["beta"], S, ins, outs, parent, node, stream=stream)
        return out

    step(d["S"])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(d["S"])
    for i in range(3):
        d["v"].mul_(-0.7)
        d["S"][:5].add_(0.01)
        other = d["S"].clone()
        graph.replay()
        torch.cuda.synchronize()
        st = torch.cuda.Stream()
        want = step(other, st)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(d["S"], other), i
