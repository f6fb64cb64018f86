"""Row norms of fp32 rows that start on a 16-byte boundary which is not a 32-byte one, the least
alignment that the vector path takes. The kernels add in the same order whatever the
address, so results are those of an aligned copy, bit for bit."""
import pytest
import torch

from gated_delta_rule_103_amd import kda_layer_norm, kda_layer_norm_backward

pytestmark = pytest.mark.gpu


def shifted(t, n):
    """A copy of t that starts n elements behind an allocation's start (which is 512-byte aligned)."""
    return torch.empty(t.numel() + n, dtype=t.dtype, device=t.device)[n:].view(t.shape).copy_(t)


@pytest.mark.parametrize("W", [8, 24, 256, 1000, 2048, 4104])
@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("d_io", [torch.float32, torch.bfloat16])
def test_rows_on_a_16_byte_boundary(W, rms, d_io):
    gen = torch.Generator(device="cuda").manual_seed(W)
    rn = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    x, dy, w, b = rn(21, W) + 0.3, rn(21, W).to(d_io), 1 + 0.1 * rn(W), 0.1 * rn(W)
    off = lambda t: shifted(t, 16 // t.element_size())
    xs, dys, ws, bs = off(x), off(dy), off(w), off(b)
    assert xs.data_ptr() % 32 == 16 and dys.data_ptr() % 32 == 16 and ws.data_ptr() % 32 == 16
    want = kda_layer_norm(x, w, b, rms=rms)
    got = kda_layer_norm(xs, ws, bs, rms=rms, out=off(x))
    gw = kda_layer_norm_backward(x, dy, want[1], want[2], w, rms=rms, bias=True)
    gg = kda_layer_norm_backward(xs, dys, want[1], want[2], ws, rms=rms, dx=off(x), dweight=off(w), dbias=off(b))
    torch.cuda.synchronize()
    assert got[0].data_ptr() % 32 == 16
    for a, c in zip([*want, *gw], [*got, *gg]):
        assert a is c is None or torch.equal(a, c)
