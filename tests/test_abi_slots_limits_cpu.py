"""The limits of the slots' counts, each at its value and one past it (no GPU needed: every call here is refused; where the size is
allowed, for another argument that is checked behind it)."""
import ctypes

import pytest

import gated_delta_rule_103_amd as lib_py

INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3
P = [ctypes.c_void_p((i + 1) << 20) for i in range(5)]       # never dereferenced


@pytest.fixture(scope="module")
def lib():
    return lib_py.load_library()


@pytest.mark.parametrize("name", ["kda_slots_share", "kda_slots_release", "kda_slots_acquire"])
@pytest.mark.parametrize("n,slots", [(1, 2 ** 30), (1, 2 ** 31 - 1), (2 ** 30, 4), (0, 2 ** 30)])
def test_counts_and_slots(lib, name, n, slots):
    f = getattr(lib, name)
    assert f(P[0], P[1], n, slots, None) == INVALID
    assert f(P[0], None, 0, 2 ** 30 - 1, None) == 0          # nothing to do: allowed, and nothing is launched


@pytest.mark.parametrize("slots,status", [(2 ** 25 - 1, WORKSPACE), (2 ** 25, UNSUPPORTED), (2 ** 28, UNSUPPORTED),
                                          (2 ** 31 - 1, UNSUPPORTED)])
def test_slots_of_a_compaction(lib, slots, status):
    assert lib.kda_slots_compact(P[0], P[1], P[2], P[3], 4, 1, slots, 64, None, 0, None) == status
