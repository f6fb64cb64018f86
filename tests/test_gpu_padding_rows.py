"""Packed batches whose offsets leave rows out, with results that the binding allocates: a row
that belongs to no sequence has gradient zero, and output zero of the recurrent form, whatever
the memory held before.

Every call runs on memory that held NaN: buffers of the results' sizes are filled and freed
just before it, so the allocator hands the same blocks out again. Values of rows that belong
to a sequence are those of the same sequences packed without any rows around them, bit for bit.
"""
import pytest
import torch

from gated_delta_rule_103_amd import gdn_prefill_backward, gdn_recurrent, inputs, kda_prefill_backward, kda_recurrent

pytestmark = pytest.mark.gpu
NAMES = ("dq", "dk", "dv", "dg", "dbeta")


def spoil(tensors):
    """Leave NaN in the free blocks that results like these will be given."""
    junk = [torch.full_like(t, float("nan")) for t in tensors if t is not None for _ in range(2)]
    torch.cuda.synchronize()
    del junk


def problem(lengths, H, D, io, gate, seed):
    p = inputs.prefill(H, D, lengths=lengths, io=io, shift=0.0, seed=seed)
    g = p.g if gate == "channel" else p.g[..., 0].contiguous() if gate == "head" else None
    dout = (torch.randn(p.v.shape, generator=torch.Generator().manual_seed(seed + 1)) * 0.1).to(p.q.dtype)
    return [None if t is None else t.cuda() for t in (p.q, p.k, p.v, g, p.beta, dout)], p.cu_seqlens


def surround(t, before, behind):
    if t is None:
        return None
    edge = lambda n: torch.full((1, n, *t.shape[2:]), float("nan"), dtype=t.dtype, device=t.device)
    return torch.cat([edge(before), t, edge(behind)], 1).contiguous()


def backward(gate):
    return kda_prefill_backward if gate == "channel" else gdn_prefill_backward


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("gate", ["channel", "head", "none"])
@pytest.mark.parametrize("l2", [False, True])
def test_gradients_of_rows_in_no_sequence_are_zero(D, io, gate, l2):
    """Rows before the first sequence and behind the last one: none, one, part of a chunk, several chunks."""
    x, cu = problem([37, 0, 64, 1], 3, D, io, gate, D)
    first = backward(gate)(*x, cu_seqlens=cu.cuda(), qk_l2norm=l2)
    for before, behind in ((0, 1), (1, 0), (5, 63), (64, 65), (200, 130), (0, 300)):
        ins = [surround(t, before, behind) for t in x]
        at = (cu + before).cuda()
        spoil(ins[:5])
        got = backward(gate)(*ins, cu_seqlens=at, qk_l2norm=l2)
        torch.cuda.synchronize()
        T = x[0].shape[1]
        for n, a, b in zip(NAMES, got, first):
            if a is None:
                assert b is None
                continue
            assert torch.equal(a[:, before:before + T], b), (n, before, behind)
            assert (a[:, :before] == 0).all() and (a[:, before + T:] == 0).all(), (n, before, behind)


def test_all_rows_in_no_sequence():
    """Every sequence empty, and offsets that are cut to nothing."""
    x, _ = problem([130], 2, 128, "bf16", "channel", 1)
    for cu in ([0, 0, 0], [130, 130], [7, 7, 7, 7], [500, 3, 3]):
        spoil(x[:5])
        got = kda_prefill_backward(*x, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"))
        torch.cuda.synchronize()
        assert all((t == 0).all() for t in got[:5]), cu


def test_many_empty_sequences_before_the_rows():
    """More sequences than chunks: the workgroups without a chunk are far more than the rows left out need."""
    x, _ = problem([150], 1, 64, "f32", "head", 2)
    cu = torch.tensor([3] * 300 + [70] * 200 + [100] * 50, dtype=torch.int32, device="cuda")
    spoil(x[:5])
    got = gdn_prefill_backward(*x, cu_seqlens=cu)
    part = [t[:, 3:100].contiguous() for t in x]
    want = gdn_prefill_backward(*part, cu_seqlens=torch.tensor([0, 67, 97], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    for n, a, b in zip(NAMES, got, want):
        assert torch.equal(a[:, 3:100], b) and (a[:, :3] == 0).all() and (a[:, 100:] == 0).all(), n


def test_buffers_of_the_caller_keep_their_rows():
    """One buffer given, the others allocated: only the rows of the allocated ones are cleared."""
    x, cu = problem([37, 20], 2, 64, "bf16", "channel", 3)
    ins = [surround(t, 4, 9) for t in x]
    like = dict(zip(NAMES, ins[:5]))
    for name in NAMES:
        spoil(ins[:5])
        own = torch.full_like(like[name], 3.0)
        got = dict(zip(NAMES, kda_prefill_backward(*ins, cu_seqlens=(cu + 4).cuda(), **{name: own})))
        torch.cuda.synchronize()
        assert got[name].data_ptr() == own.data_ptr()
        for n, t in got.items():
            rest = torch.cat([t[:, :4], t[:, 4 + 57:]], 1)
            assert (rest == (3.0 if n == name else 0.0)).all(), (name, n)


def test_captured_with_offsets_that_change():
    """A captured call follows the offsets that a replay finds: rows that leave the batch become zero."""
    x, _ = problem([100, 60], 2, 128, "bf16", "channel", 4)
    cu = torch.tensor([0, 100, 160], dtype=torch.int32, device="cuda")
    kda_prefill_backward(*x, cu_seqlens=cu)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = kda_prefill_backward(*x, cu_seqlens=cu)
    for new in ([0, 100, 160], [10, 90, 120], [0, 0, 31], [0, 100, 160]):
        cu.copy_(torch.tensor(new, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        spoil(x[:5])
        want = kda_prefill_backward(*x, cu_seqlens=cu)
        torch.cuda.synchronize()
        for n, a, b in zip(NAMES, got, want):
            assert torch.equal(a, b), (new, n)
            assert (a[:, :new[0]] == 0).all() and (a[:, new[-1]:] == 0).all(), (new, n)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("gate", ["channel", "head", "none"])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_recurrent_rows_in_no_sequence_are_zero(D, gate, out_dtype):
    x, cu = problem([3, 0, 1, 5], 3, D, "bf16", gate, D)
    x = [None if t is None else t[0] for t in x[:5]]
    f = kda_recurrent if gate == "channel" else gdn_recurrent
    pool = torch.randn(13, 3, D, D, generator=torch.Generator().manual_seed(1)).cuda() * 0.1
    idx = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    start = idx([0, 1, 2, 3])
    first, kept = pool.clone(), idx(range(4, 13))
    want = f(*x, first, start, kept, cu.cuda(), out_dtype=out_dtype)
    for before, behind in ((0, 1), (1, 0), (7, 9), (70, 33)):
        ins = [None if t is None else surround(t[None], before, behind)[0] for t in x]
        none = lambda n: torch.full((n,), -1, dtype=torch.int32, device="cuda")
        S, T = pool.clone(), before + 9 + behind
        spoil([torch.empty(T, 3, D, dtype=out_dtype, device="cuda")])
        got = f(*ins, S, start, torch.cat([none(before), kept, none(behind)]), (cu + before).cuda(), out_dtype=out_dtype)
        torch.cuda.synchronize()
        assert torch.equal(got[before:before + 9], want) and torch.equal(S, first), (before, behind)
        assert (got[:before] == 0).all() and (got[before + 9:] == 0).all(), (before, behind)
        mine = torch.full_like(got, 3.0)
        f(*ins, pool.clone(), start, None, (cu + before).cuda(), out=mine)
        torch.cuda.synchronize()
        assert (mine[:before] == 3).all() and (mine[before + 9:] == 3).all() and torch.equal(mine[before:before + 9], want)


def test_recurrent_without_any_sequence():
    x, _ = problem([20], 2, 64, "f32", "channel", 5)
    x = [t[0] for t in x[:5]]
    pool = torch.ones(2, 2, 64, 64, device="cuda")
    for cu in ([0, 0], [20, 20, 20], [6, 6, 6], [50, 50]):
        spoil([x[2]])
        got = kda_recurrent(*x, pool, None, None, torch.tensor(cu, dtype=torch.int32, device="cuda"))
        torch.cuda.synchronize()
        assert (got == 0).all() and (pool == 1).all(), cu
