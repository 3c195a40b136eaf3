"""Largest sizes of the gated delta rule's C ABI (no device needed)."""
import ctypes

import pytest

INT_MAX = 2 ** 31 - 1


@pytest.fixture(scope="module")
def lib():
    from gated_linear_recurrence_b200 import build
    build.build()
    from gated_linear_recurrence_b200 import esa
    return esa.load_library()


@pytest.mark.parametrize("dtype", [0, 1, 2])
@pytest.mark.parametrize("keep", [0, 1])
@pytest.mark.parametrize("D", [32, 64, 128])
def test_longest_sequences(lib, D, keep, dtype):
    """A chunk's end passes 32 bits for the last lengths: refused.  Up to there a longer sequence needs more."""
    sizes = [lib.esa_delta_workspace_size(1, T, 1, D, dtype, keep) for T in (1 << 20, 1 << 26, 1 << 30, INT_MAX - 64)]
    if dtype == 0 and not keep:   # a sweep from end to end needs nothing, states between chunks do
        assert sizes == sorted(sizes)
    else:
        assert all(a < b for a, b in zip(sizes, sizes[1:]))
    chunks = (INT_MAX - 64 + 63) // 64
    if keep:
        assert sizes[-1] > chunks * D * D * 2
    for T in range(INT_MAX - 63, INT_MAX + 1):
        assert lib.esa_delta_workspace_size(1, T, 1, D, dtype, keep) == 0


def test_too_long_a_sequence_is_refused(lib):
    from gated_linear_recurrence_b200 import esa
    P = ctypes.c_void_p
    for T in (INT_MAX - 63, INT_MAX):
        assert lib.esa_delta_fwd(P(0x1000), P(0x2000), 32, P(0x3000), 32, P(0x4000), P(0x5000), 1, P(0x6000), None, 1, T, 1, 32,
                                 0.1, None, 1, 0, P(0x10000), 1 << 60, None) == esa.ESA_ERR_ARG
        assert lib.esa_delta_bwd(P(0x1000), P(0x2000), 32, P(0x3000), 32, P(0x4000), P(0x5000), 1, P(0x6000), None, P(0x7000),
                                 P(0x8000), P(0x9000), P(0xa000), P(0xb000), None, 1, T, 1, 32, 0.1, None, 1, P(0x10000),
                                 1 << 60, None) == esa.ESA_ERR_ARG
