"""What the gradient's matrix products leave out, and its workspace, on the CPU.

Emulates the cut of a value into three bf16 parts (rounded on one side of a product, truncated on
the other) in torch and checks the bound that the kernels rely on: the parts are the whole, and
the three products left out are at most 3 x 2^-24 (1 + 2^-9) of the product, 0 on average.
"""
import pytest
import torch

from gated_delta_rule_103_amd import kda_prefill_backward_workspace_size

STEP = 2.0 ** -24


def parts(x, near):
    """Three parts of the fp32 values x, as fp64; x - h and what follows it are exact in fp32."""
    res = []
    for _ in range(3):
        h = x.bfloat16().float() if near else (x.view(torch.int32) & -65536).view(torch.float32)
        res.append(h.double())
        x = x - h
    assert (x == 0).all()
    return res


def left_out(a, b, near_b):
    (_, m, l), (_, n, k) = parts(a, True), parts(b, near_b)
    return (m * k + l * n + l * k) / (a.double() * b.double())


def operands(seed):
    gen = torch.Generator().manual_seed(seed)
    a, b = (torch.randn(1 << 20, generator=gen) for _ in range(2))
    far = torch.tensor([1 + 2.0 ** -7 - 2.0 ** -23, 1 + 2.0 ** -8 + 2.0 ** -16 - 2.0 ** -23, 1 + 2.0 ** -8 - 2.0 ** -17,
                        2 - 2.0 ** -23, 1 - 2.0 ** -24, 1 + 2.0 ** -8])
    a[:36], b[:36] = far.repeat_interleave(6), far.repeat(6)
    return a, b


@pytest.mark.parametrize("near_b,steps", [(False, 3.0), (True, 1.0)])
def test_products_left_out(near_b, steps):
    err = left_out(*operands(1), near_b)
    assert err.abs().max() <= steps * (1 + 2.0 ** -8) * STEP
    assert err.mean().abs() <= 4 * err.std() / err.numel() ** 0.5


def test_truncation_of_both_sides_would_lose_one_way():
    a, b = operands(2)
    (_, m, l), (_, n, k) = parts(a, False), parts(b, False)
    err = (m * k + l * n + l * k) / (a.double() * b.double())
    assert (err >= 0).all() and err.max() > 6 * STEP and err.mean() > 0.5 * STEP


@pytest.mark.parametrize("D,kb", [(128, 381), (64, 169)])
@pytest.mark.parametrize("N,T,H", [(1, 64, 1), (1, 8192, 32), (9, 5000, 8), (4096, 4096, 2), (700, 0, 3)])
def test_workspace_is_what_the_header_says(D, kb, N, T, H):
    """(ceil(T / 64) + N) * H times 381 KB (D = 128) or 169 KB, within 2% and the offsets' few KB."""
    said = ((T + 63) // 64 + N) * H * kb * 1000
    assert abs(kda_prefill_backward_workspace_size(N, T, H, D, D) - said) <= 0.02 * said + 8 * (N + 1) + 2048
