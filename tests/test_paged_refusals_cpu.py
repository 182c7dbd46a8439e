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


# pools [64 pages, 8 heads, 16 positions, 128]
@pytest.mark.parametrize("s", [
    (0, 2048, 128), (8 * 2048, 0, 128), (8 * 2048, 2048, 0),  # expanded axes
    (8 * 2048, 2048, 64), (8 * 2048, 1024, 128), (4 * 2048, 2048, 128),
    (128, 128, 128),
])
def test_pools_whose_rows_overlap_are_refused_where_they_are_written(sa, s):
    c = cache(sa, strides=strides(*s))
    for op in ("append", "evict"):
        assert calls(sa, c)[op]() == 1, op
    assert calls(sa, c, ws_bytes=100)["decode"]() == 3  # read only: refused for its workspace alone


@pytest.mark.parametrize("s", [
    (8 * 2048, 2048, 128), (8 * 2048, 128, 8 * 128), (2048, 64 * 2048, 128), (128, 64 * 128, 64 * 8 * 128),
    (2 * 8 * 2048, 2048, 128), (8 * 2048 + 8, 2048, 128), (1 << 33, 2048, 128),
])
def test_pools_in_any_order_of_their_axes_are_taken(sa, s):
    for op, call in calls(sa, cache(sa, strides=strides(*s)), ws_bytes=100).items():
        assert call() == 3, op  # refused for its workspace alone


def test_axes_of_one_entry_need_no_stride(sa):
    c = cache(sa, n_pages=1, num_kv_heads=1, page_size=1, max_pages=160, table_stride=160, n_seq=1, strides=strides(0, 0, 0))
    kw = dict(num_q_heads=1, score_strides=strides(0, 0), out_strides=strides(0, 0), o_strides=strides(0, 0),
              dst_max_pages=64, dst_table_stride=64, ws_bytes=100)
    for op, call in calls(sa, c, **kw).items():
        assert call() == 3, op


# 4 sequences, 8 heads, capacity 160, 64 kept
@pytest.mark.parametrize("s", [(160, 160), (0, 160), (1279, 160), (160, 639), (1 << 62, 100)])
def test_scores_whose_rows_overlap_are_refused(sa, s):
    for op in ("append", "decode", "evict"):
        assert calls(sa, cache(sa), score_strides=strides(*s))[op]() == 1, op


@pytest.mark.parametrize("s", [(1280, 160), (160, 640), (8 * 163, 163), (1 << 60, 160)])
def test_scores_in_either_order_of_their_axes_are_taken(sa, s):
    for op, call in calls(sa, cache(sa), score_strides=strides(*s), ws_bytes=100).items():
        assert call() == 3, op


@pytest.mark.parametrize("s", [(64, 64), (511, 64), (64, 255)])
def test_moved_scores_whose_rows_overlap_are_refused(sa, s):
    assert calls(sa, cache(sa), out_strides=strides(*s))["evict"]() == 1


# 32 query heads of 128
@pytest.mark.parametrize("s", [(0, 128), (4096, 0), (4096, 64), (128, 128), (2048, 128)])
def test_outputs_whose_rows_overlap_are_refused(sa, s):
    assert calls(sa, cache(sa), o_strides=strides(*s))["decode"]() == 1


def test_queries_may_be_shared_and_outputs_strided(sa):
    for kw in (dict(q_strides=strides(0, 128)), dict(q_strides=strides(0, 0)), dict(o_strides=strides(128, 512)),
               dict(o_strides=strides(4096 + 8, 128))):
        assert calls(sa, cache(sa), ws_bytes=100, **kw)["decode"]() == 3
