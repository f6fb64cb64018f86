"""The fp64 gradient oracles against central differences of the forward oracles.

With f summed against fixed random cotangents, (f(x + h d) - f(x - h d)) / 2h is the
directional derivative up to h^2 f'''/6 and rounding eps |f| / h. At h = 1e-5, values
of order 1 and third derivatives of order up to 1e2 both are below 1e-8; the bar is
1e-7 of the derivative's scale (the product of the norms of gradient and direction).
"""
import numpy as np
import pytest

import oracle
from oracle import gradients

H_STEP = 1e-5
BAR = 1e-7


def _check(f, inputs, grads, rng):
    for name, x in inputs.items():
        d = rng.standard_normal(x.shape)
        plus, minus = ({**inputs, name: x + s * H_STEP * d} for s in (1.0, -1.0))
        got = (f(**plus) - f(**minus)) / (2 * H_STEP)
        want = float((grads[name] * d).sum())
        scale = np.linalg.norm(grads[name]) * np.linalg.norm(d)
        assert abs(got - want) <= BAR * max(scale, 1.0), (name, got, want)


@pytest.mark.parametrize("l2", [None, 1e-3])
@pytest.mark.parametrize("cu", [None, [0, 5, 5, 6, 13]])
def test_recurrent_backward_against_differences(cu, l2):
    rng = np.random.default_rng(3)
    T, H, D = 13, 2, 5
    N = 1 if cu is None else len(cu) - 1
    x = dict(q=rng.standard_normal((T, H, D)), k=0.5 * rng.standard_normal((T, H, D)), v=rng.standard_normal((T, H, D)),
             g=-np.abs(rng.standard_normal((T, H, D))), beta=rng.uniform(0, 1, (T, H)),
             S0=rng.standard_normal((N, H, D, D)))
    dout, dS = rng.standard_normal((T, H, D)), rng.standard_normal((N, H, D, D))

    def f(q, k, v, g, beta, S0):
        if l2 is not None:
            q, k = oracle.l2norm(q, l2), oracle.l2norm(k, l2)
        o, S = oracle.recurrent(q, k, v, g, beta, S0=S0, cu_seqlens=[0, T] if cu is None else cu)
        return float((o * dout).sum() + (S * dS).sum())

    r = gradients.recurrent_backward(**{n: x[n] for n in ("q", "k", "v", "g", "beta")}, dout=dout, S0=x["S0"], dS_out=dS,
                                     cu_seqlens=cu, l2norm_eps=l2)
    _check(f, x, {n: r["d" + n] for n in x}, rng)


def test_output_gate_backward_against_differences():
    rng = np.random.default_rng(4)
    x = dict(o=rng.standard_normal((3, 2, 8)), z=2 * rng.standard_normal((3, 2, 8)), w=1 + 0.1 * rng.standard_normal(8))
    d = rng.standard_normal((3, 2, 8))
    do, dz, dw = gradients.output_gate_backward(x["o"], x["z"], d, x["w"], eps=1e-2)
    _check(lambda o, z, w: float((oracle.output_gate(o, z, w, 1e-2) * d).sum()), x, dict(o=do, z=dz, w=dw), rng)


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("W", [1, 2, 9])
def test_layer_norm_backward_against_differences(W, rms):
    rng = np.random.default_rng(5)
    x = dict(x=rng.standard_normal((4, W)) + 0.5, weight=1 + 0.1 * rng.standard_normal(W), bias=rng.standard_normal(W))
    d = rng.standard_normal((4, W))
    dx, dw, db = gradients.layer_norm_backward(x["x"], d, x["weight"], eps=1e-2, rms=rms)
    _check(lambda x, weight, bias: float((gradients.layer_norm(x, weight, bias, 1e-2, rms)[0] * d).sum()), x,
           dict(x=dx, weight=dw, bias=db), rng)
