"""Paged cache operators at the edges of their contracts; bounds as in test_gpu_paged."""
import numpy as np
import pytest
import torch

from test_gpu_paged import LOCAL, TYPES, U, Case, check_decode, half_step, new_rows, status, to_np

from oracle import paged as Pg

pytestmark = pytest.mark.gpu


# ------------------------------------------------ scores to another array
@pytest.mark.parametrize("lens,hq,hkv,d,page,cache,window,sinks", [
    ([0, 5, 300, 16, 513], 8, 2, 128, 16, "bf16", 0, 0),
    ([1, 700, 0, 40], 12, 4, 64, 24, "fp16", 50, 3),
    ([90, 2, 257], 5, 1, 128, 7, "e4m3", 0, 0),
    ([3000, 1], 32, 2, 64, 32, "bf16", 64, 4),
])
def test_scores_to_another_array_are_whole(sa, lens, hq, hkv, d, page, cache, window, sinks):
    """scores_out = scores_in plus the weights, positions behind the lengths among
    them, whatever it held; with keep_tail those stay as they were."""
    c = Case(sa, 300 + len(lens), lens, hkv, d, page, cache, extra_pages=70)
    q = c.query(hq)
    before = c.scores()
    work = before.clone()
    o, lse = sa.paged_decode(c.cache, q, window, sinks, scores=work)
    check_decode(c, q, o, lse, window, sinks, None, before, work)
    held = before.clone()
    o2, lse2, out = torch.empty_like(o), torch.empty_like(lse), torch.full_like(before, float("nan"))
    for keep_tail in (False, True):
        dd = sa.paged_decode_desc(q, o2, window, sinks, scores=before, keep_tail=keep_tail)
        sa.sa_paged_decode(c.cache, dd, q, o2, lse2, before, out, sa.paged_decode_workspace(c.cache, dd))
        assert torch.equal(o2, o) and torch.equal(lse2, lse)
        if keep_tail:
            for s, n in enumerate(lens):
                assert torch.equal(out[s, :, :n], work[s, :, :n]) and (out[s, :, n:] == 9).all()
        else:  # work was added to in place: behind the lengths it holds the scores so far
            assert torch.equal(out, work)
        out.fill_(9.0)
    sa.paged_decode(c.cache, q, window, sinks, scores=before, scores_out=out, keep_tail=False)
    assert torch.equal(out, work) and torch.equal(before, held)


def test_scores_are_carried_up_to_a_bound_on_the_lengths(sa):
    c = Case(sa, 310, [200, 31, 0], 2, 128, 16, extra_pages=40)
    q = c.query(8)
    before = c.scores()
    cache = sa.PagedCache(c.k, c.v, c.table, c.seq_lens, max_len=215)
    work, out = before.clone(), torch.full_like(before, 9.0)
    sa.paged_decode(cache, q, scores=work)
    sa.paged_decode(cache, q, scores=before, scores_out=out, keep_tail=False)
    assert torch.equal(out[:, :, :215], work[:, :, :215]) and (out[:, :, 215:] == 9).all()


def test_a_captured_decode_carries_scores_behind_the_lengths_of_the_replay(sa):
    c = Case(sa, 311, [300, 17, 128], 2, 64, 16)
    q = c.query(8)
    before = c.scores()
    out = torch.zeros_like(before)
    sa.paged_decode(c.cache, q, scores=before, scores_out=out, keep_tail=False)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sa.paged_decode(c.cache, q, scores=before, scores_out=out, keep_tail=False)
    for lens in ([300, 17, 128], [2, 0, 64]):
        c.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        before.copy_(torch.rand_like(before))
        work = before.clone()
        out.fill_(float("nan"))
        g.replay()
        sa.paged_decode(c.cache, q, scores=work)
        assert torch.equal(out, work)
