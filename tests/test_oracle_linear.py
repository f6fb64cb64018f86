"""The fp64 references of linear attention and of draft trees, pinned: closed forms, the KDA oracle where they meet,
and central differences for the gradients."""
import numpy as np
import pytest

import oracle
from oracle import linear


def draw(T, H, Hk, Dk, Dv, N=1, seed=0):
    r = np.random.default_rng(seed)
    return dict(q=r.normal(size=(T, Hk, Dk)), k=r.normal(size=(T, Hk, Dk)), v=r.normal(size=(T, H, Dv)),
                g=-np.abs(r.normal(size=(T, H))), S0=r.normal(size=(N, H, Dv, Dk)))


def test_one_token():
    x = draw(1, 2, 1, 3, 4)
    o, S = linear.recurrent(**x)
    for h in range(2):
        want = np.exp(x["g"][0, h]) * x["S0"][0, h] + np.outer(x["v"][0, h], x["k"][0, 0])
        assert np.allclose(S[0, h], want, rtol=1e-14) and np.allclose(o[0, h], want @ x["q"][0, 0], rtol=1e-14)


def test_sums_over_all_earlier_tokens():
    x = draw(9, 3, 3, 4, 5, seed=1)
    o, S = linear.recurrent(**x)
    a = np.cumsum(x["g"], 0)
    for t in range(9):
        for h in range(3):
            want = np.exp(a[t, h]) * x["S0"][0, h] @ x["q"][t, h]
            for s in range(t + 1):
                want = want + np.exp(a[t, h] - a[s, h]) * (x["q"][t, h] @ x["k"][s, h]) * x["v"][s, h]
            assert np.allclose(o[t, h], want, rtol=1e-12)


def test_no_delta_is_the_kda_oracle_with_orthogonal_keys():
    """With orthonormal keys and no decay the delta rule has nothing to correct (beta 1, zero state)."""
    k = np.eye(6)[:, None, :]
    r = np.random.default_rng(2)
    q, v = r.normal(size=(6, 1, 6)), r.normal(size=(6, 1, 6))
    o, S = linear.recurrent(q, k, v, np.zeros((6, 1)))
    ko, kS = oracle.recurrent(q, k, v, np.zeros((6, 1, 6)), np.ones((6, 1)))
    assert np.allclose(o, ko, atol=1e-13) and np.allclose(S, np.swapaxes(kS, -1, -2), atol=1e-13)


def test_packed_is_separate():
    x, cu = draw(10, 2, 2, 3, 4, N=3, seed=3), [1, 4, 4, 9]
    o, S = linear.recurrent(**x, cu_seqlens=cu)
    assert (o[0] == 0).all() and (o[9] == 0).all() and (S[1] == x["S0"][1]).all()
    for n in (0, 2):
        one = {m: x[m][cu[n]:cu[n + 1]] for m in "qkvg"}
        oo, SS = linear.recurrent(**one, S0=x["S0"][n:n + 1])
        assert np.array_equal(oo, o[cu[n]:cu[n + 1]]) and np.array_equal(SS[0], S[n])


@pytest.mark.parametrize("Hk", [1, 2])
def test_gradients_by_differences(Hk):
    x, cu = draw(7, 2, Hk, 3, 2, N=2, seed=4), [0, 4, 6]
    r = np.random.default_rng(5)
    dout, dS = r.normal(size=(7, 2, 2)), r.normal(size=(2, 2, 2, 3))
    dout[6] = 0                                            # a row of no sequence

    def loss():
        o, S = linear.recurrent(**x, cu_seqlens=cu)
        return (o * dout).sum() + (S * dS).sum()

    got = linear.backward(x["q"], x["k"], x["v"], x["g"], dout, x["S0"], dS, cu)
    for name in ("q", "k", "v", "g", "S0"):
        want = np.zeros_like(x[name])
        for i in np.ndindex(*want.shape):
            keep = x[name][i]
            x[name][i] = keep + 1e-5
            up = loss()
            x[name][i] = keep - 1e-5
            want[i] = (up - loss()) / 2e-5
            x[name][i] = keep
        assert np.abs(got["d" + name] - want).max() < 1e-7, name


def test_a_chain_is_the_recurrence():
    """A tree without branches: the KDA oracle's outputs and states, the linear one's without the delta rule."""
    r = np.random.default_rng(6)
    q, k, v = (r.normal(size=(5, 2, 4)) for _ in range(3))
    g, beta, S = -np.abs(r.normal(size=(5, 2, 4))), r.uniform(size=(5, 2)), r.normal(size=(2, 4, 4))
    chain = [-1, 0, 1, 2, 3]
    ko, kS = oracle.recurrent(q, k, v, g, beta, S0=np.swapaxes(S, -1, -2)[None].copy())
    assert np.allclose(linear.tree(q, k, v, g, beta, S, chain), ko, atol=1e-13)
    assert np.allclose(linear.tree_states(k, v, g, beta, S, chain)[4], np.swapaxes(kS[0], -1, -2), atol=1e-13)
    o, S1 = linear.recurrent(q, k, v, g[..., 0], S[None])
    assert np.allclose(linear.tree(q, k, v, g[..., 0], None, S, chain), o, atol=1e-13)
    assert np.allclose(linear.tree_states(k, v, g[..., 0], None, S, chain)[4], S1[0], atol=1e-13)


def test_branches_do_not_meet():
    """Every node's output is that of the chain of its ancestors; absent nodes and what descends from them are left out."""
    r = np.random.default_rng(7)
    T, parent = 8, [-1, 0, 0, -1, 2, 4, 9, 6]
    q, k, v = (r.normal(size=(T, 2, 4)) for _ in range(3))
    g, beta, S = -np.abs(r.normal(size=(T, 2))), r.uniform(size=(T, 2)), r.normal(size=(2, 4, 4))
    out = linear.tree(q, k, v, g, beta, S, parent)
    for path in ([0], [0, 1], [0, 2], [3], [0, 2, 4], [0, 2, 4, 5]):
        chain = linear.tree(q[path], k[path], v[path], g[path], beta[path], S, [-1, 0, 1, 2][:len(path)])
        assert np.allclose(out[path[-1]], chain[-1], atol=1e-13)
    assert (out[6:] == 0).all() and 7 not in linear.tree_states(k, v, g, beta, S, parent)
