"""The state pool's slots: copies, counts, acquisition and compaction, all exact."""
import pytest
import torch

import gated_delta_rule_103_amd as lib

pytestmark = pytest.mark.gpu
i32 = lambda *a: torch.tensor(a, dtype=torch.int32).cuda()


def pool_of(*shape, seed=0, dtype=torch.float32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


@pytest.mark.parametrize("shape", [(9, 2, 64, 64), (3, 9, 1, 64, 128), (2, 9, 5, 3, 4), (9, 32, 128, 128), (9, 1, 1, 4)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_copy(shape, dtype):
    p = pool_of(*shape, dtype=dtype)
    if shape[-3] * shape[-2] * shape[-1] * p.element_size() % 16:      # states of 8 and 120 bytes
        with pytest.raises(lib.KDAError, match="INVALID_ARG"):
            lib.kda_slots_copy(p, i32(8), i32(0))
        return
    want = p.clone()
    w = want if want.dim() == 5 else want[None]
    for s, d in ((8, 0), (3, 5), (3, 6)):
        w[:, d] = w[:, s]
    w[:, 7] = 0
    lib.kda_slots_copy(p, i32(8, 3, 3, -1, 4, 2, 99), i32(0, 5, 6, 7, -1, 9, -5))
    assert torch.equal(p, want)
    other = torch.full([y * 2 if i == len(shape) - 4 else y for i, y in enumerate(shape)], 7.0, dtype=dtype).cuda()
    lib.kda_slots_copy(p, i32(2, 9, 0), i32(17, 3, 18), to=other)
    o = other if other.dim() == 5 else other[None]
    w = p if p.dim() == 5 else p[None]
    assert torch.equal(o[:, 17], w[:, 2]) and (o[:, 3] == 0).all() and (o[:, [0, 1, 2] + list(range(4, 17))] == 7).all()
    lib.kda_slots_copy(p, i32()[:0], i32()[:0])
    assert torch.equal(p, want)


def test_copy_beyond_32_bits():
    """A pool of more than 4 GiB: its last slots."""
    p = torch.zeros(2300, 32, 128, 128, device="cuda")
    p[2] = 1.5
    lib.kda_slots_copy(p, i32(2, 2299), i32(2298, 1))
    assert (p[2298] == 1.5).all() and (p[2297] == 0).all() and (p[2299] == 0).all() and (p[1] == 0).all()


def test_counts():
    u = i32(0, 1, 2, 3, 0)
    lib.kda_slots_share(u, i32(1, 1, 4, -1, 5, 2 ** 31 - 1))
    assert u.tolist() == [0, 3, 2, 3, 1]
    lib.kda_slots_release(u, i32(0, 1, 2, 2, 2, 3, -7, 5))
    assert u.tolist() == [0, 2, 0, 2, 1]
    many = torch.zeros(700, dtype=torch.int32).cuda()
    which = torch.randint(0, 700, (5000,), generator=torch.Generator().manual_seed(1)).to(torch.int32)
    lib.kda_slots_share(many, which.cuda())
    assert torch.equal(many.cpu(), torch.bincount(which.long(), minlength=700).to(torch.int32))
    lib.kda_slots_release(many, torch.cat([which, which[:100]]).cuda())
    assert (many == 0).all()


@pytest.mark.parametrize("slots,n,fill", [(1, 1, 0.0), (1, 3, 1.0), (37, 5, 0.5), (1024, 300, 0.7), (1025, 1025, 0.0),
                                          (5000, 1500, 0.4), (5000, 0, 0.5)])
def test_acquire(slots, n, fill):
    u = (torch.rand(slots, generator=torch.Generator().manual_seed(slots)) < fill).to(torch.int32) * 2
    free = (u == 0).nonzero()[:, 0].tolist()[:n]
    d = u.cuda()
    taken = lib.kda_slots_acquire(d, n)
    assert taken.tolist() == free + [-1] * (n - len(free))
    u[free] = 1
    assert torch.equal(d.cpu(), u)


@pytest.mark.parametrize("shape", [(1, 1, 4, 4), (37, 2, 64, 64), (3, 50, 1, 64, 128), (2, 2500, 1, 2, 4), (300, 8, 128, 128)])
@pytest.mark.parametrize("fill", [0.0, 0.3, 0.8, 1.0])
def test_compact(shape, fill):
    p = pool_of(*shape, seed=3)
    slots = shape[-4]
    u = (torch.rand(slots, generator=torch.Generator().manual_seed(slots)) < fill).to(torch.int32) * torch.arange(1, slots + 1)
    u = u.to(torch.int32)
    table = torch.cat([torch.arange(slots), torch.tensor([-1, slots, 0])]).to(torch.int32)
    live = (u > 0).nonzero()[:, 0].tolist()
    c = len(live)
    movers, holes = [s for s in live if s >= c], [s for s in range(c) if u[s] == 0]
    place = {s: s for s in live} | dict(zip(movers, holes))
    want = p.clone()
    w = want if want.dim() == 5 else want[None]
    for s, d in zip(movers, holes):
        w[:, d] = w[:, s]
    uses = torch.zeros_like(u)
    for s, d in place.items():
        uses[d] = u[s]
    d, t = u.cuda(), table.cuda()
    count = lib.kda_slots_compact(p, d, t)
    assert count.tolist() == [c] and torch.equal(p, want) and torch.equal(d.cpu(), uses)
    assert t.tolist() == [place.get(s, -1) for s in range(slots)] + [-1, slots, place.get(0, -1)]
    again = lib.kda_slots_compact(p, d)                    # nothing left to move
    assert again.tolist() == [c] and torch.equal(p, want) and torch.equal(d.cpu(), uses)


def test_graph_replays_of_a_serving_step():
    """Finished sequences give their slots back, new ones fork a prefix, the pool closes up: captured once, replayed, equal to the
    eager calls each time."""
    p = pool_of(2, 40, 2, 64, 64, seed=4)
    uses = (torch.arange(40) % 3 != 0).to(torch.int32).cuda()
    done, source, table = i32(4, 7, 39), i32(38, 38, 2, 5, -1), torch.arange(40, dtype=torch.int32).cuda()

    def step(p, uses, table):
        lib.kda_slots_release(uses, done)
        taken = lib.kda_slots_acquire(uses, 5)
        lib.kda_slots_copy(p, source, taken)
        lib.kda_slots_share(uses, taken[:2])
        return taken, lib.kda_slots_compact(p, uses, table)

    step(p.clone(), uses.clone(), table.clone())
    torch.cuda.synchronize()
    start = [x.clone() for x in (p, uses, table)]
    work = [x.clone() for x in start]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(*work)
    for i in range(3):
        start[0].mul_(-0.7)
        for x, y in zip(work, start):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        eager = [x.clone() for x in start]
        want = step(*eager)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((*work, *got), (*eager, *want))), i


def test_refusals():
    p, u = pool_of(4, 1, 4, 4), i32(0, 1, 0, 1)
    with pytest.raises(ValueError, match="src must be one of"):
        lib.kda_slots_copy(p, i32(0).long(), i32(1))
    with pytest.raises(ValueError, match="dst must have shape"):
        lib.kda_slots_copy(p, i32(0), i32(1, 2))
    with pytest.raises(ValueError, match="layers and states"):
        lib.kda_slots_copy(p, i32(0), i32(1), to=pool_of(4, 1, 4, 8))
    with pytest.raises(lib.KDAError, match="INVALID_ARG"):
        lib.kda_slots_copy(pool_of(4, 1, 1, 3), i32(0), i32(1))
    with pytest.raises(lib.KDAError, match="INVALID_ARG"):
        lib.kda_slots_share(u, u)
    with pytest.raises(ValueError, match="uses must have shape"):
        lib.kda_slots_compact(p, i32(0, 1))
    with pytest.raises(lib.KDAError, match="WORKSPACE"):
        lib.kda_slots_compact(p, u, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
