"""An accepted state's pool is none of the call's other buffers (no GPU needed: every call here is refused)."""
import pytest

from test_abi_linear_cpu import INVALID, P, kda_accept, lib, lin_accept  # noqa: F401


@pytest.mark.parametrize("call,name", [(c, n) for c in (kda_accept, lin_accept) for n in ("k", "v", "g", "si", "so", "parent", "node")] +
                         [(kda_accept, "beta")])
def test_pool_apart(lib, call, name):  # noqa: F811
    assert call(lib, {name: P[5]}) == INVALID
