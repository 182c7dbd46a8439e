"""What the paged cache's C checks refuse beside test_paged_cpu's list, without a GPU."""
import pytest

from test_paged_cpu import FAKE, cache, calls, sa, strides  # noqa: F401 (sa: fixture)


@pytest.mark.parametrize("value", [-1, 2])
def test_other_values_of_keep_tail_are_refused(sa, value):
    import ctypes as C
    L, lib = sa._abi, sa.lib()
    d = L.sa_paged_decode_desc(dtype=0, num_q_heads=8, keep_tail=value)
    n = C.c_size_t()
    assert lib.sa_paged_decode_workspace_size(C.byref(cache(sa)), C.byref(d), C.byref(n)) == 1
    d.keep_tail = 1
    assert lib.sa_paged_decode_workspace_size(C.byref(cache(sa)), C.byref(d), C.byref(n)) == 0
