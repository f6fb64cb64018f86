"""The decays' gradient of linear attention between an initial state and a gradient of the final one, from weak to strong
decays: the two ends' sums differ by e^g for every token between them, and so would their roundings."""
import sys

import numpy as np
import pytest
import torch

import gated_delta_rule_103_amd as lib
from kda_testlib import host64
from oracle import linear

pytestmark = pytest.mark.gpu

# Relative, in the 2-norm. A term (a row's sum over channels, a border's inner product) is off by some 40 independent
# roundings of 2^-24: 9 for operands cut in three, decays and state updates, 14 for a sum over channels, 17 for a border's. A
# token's value has up to 2 x 64 terms, none larger than the value where they start from the nearer end, and both ends' sums
# weighted by the squares of their magnitudes are off by 1.21 times the better one at most:
# sqrt(40 x 128) x 1.21 x 2^-24 = 5.2e-6, and twice that for inputs whose sums are smaller than their terms.
BAR = 1e-5


@pytest.mark.parametrize("scale", [1.0, 30.0])
@pytest.mark.parametrize("T", [2, 8, 32, 64])
@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("Hk", [1, 2])
def test_between_two_states(io, T, scale, Hk):
    gen = torch.Generator().manual_seed(T + Hk)
    N, H, D = 3, 2, 64
    rn = lambda *s: torch.randn(*s, generator=gen)
    unit = lambda *s: torch.nn.functional.normalize(rn(*s), dim=-1)
    q, k, v, dout = (x.to(io) for x in (unit(N, T, Hk, D), unit(N, T, Hk, D), rn(N, T, H, D), rn(N, T, H, D)))
    S0, dS = rn(N, H, D, D) * scale, rn(N, H, D, D) * scale
    for decay in (-1., -4., -8., -12., -16.):
        g = torch.full((N, T, H), decay)
        dg = lib.lin_prefill_backward(*(x.cuda() for x in (q, k, v, g, dout, S0, dS)))[3]
        flat = lambda x: host64(x.reshape(N * T, *x.shape[2:]))
        ref = linear.backward(*(flat(x) for x in (q, k, v, g, dout)), host64(S0), host64(dS), list(range(0, N * T + 1, T)))["dg"]
        off = np.linalg.norm(flat(dg) - ref) / np.linalg.norm(ref)
        print(f"  g {decay}: {off:.1e}", file=sys.stderr, flush=True)
        assert off <= BAR, decay
