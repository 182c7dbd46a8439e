"""Paged cache operators at the edges of their contracts; bounds as in test_gpu_paged."""
import numpy as np
import pytest
import torch

from test_gpu_paged import LOCAL, TYPES, Case, check_decode, expect_append, new_rows, status

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


# ------------------------------------------- weights far below the largest
def put_rows(c, i, s, x):
    """Rows x [Hkv, n, d] of sequence s into the keys (0) or values (1)."""
    x = x.to(c.k.dtype)
    c.rows[i][s] = x
    j = torch.arange(x.shape[1], device="cuda")
    bits = torch.uint8 if x.dtype == TYPES["e4m3"] else torch.int16
    pool = (c.k, c.v)[i].view(bits)
    pool[c.table[s].long()[j // c.page], :, j % c.page] = x.cuda().view(bits).transpose(0, 1)


@pytest.mark.parametrize("tail", ["equal", "spread"])
@pytest.mark.parametrize("at", [0, 700])
@pytest.mark.parametrize("cache,hq,hkv,d,n", [
    ("fp16", 300, 300, 64, 1024), ("e4m3", 300, 300, 64, 1100), ("bf16", 300, 300, 64, 1024),
    ("fp16", 320, 40, 128, 1500), ("e4m3", 320, 40, 128, 1500),
    ("fp16", 480, 40, 128, 1111), ("e4m3", 480, 40, 64, 1111),
])
def test_one_key_far_above_the_rest_with_a_value_of_zero(sa, cache, hq, hkv, d, n, at, tail):
    """A first key that takes almost all of the weight and gives nothing, as trained
    models leave it: O is the sum over the rest, each of whose weights is 10 to 45
    nats smaller (another gap for every query head), and has to be as exact
    relative to that sum as any other."""
    c = Case(sa, 320, [n], hkv, d, 16, cache, scales=False)
    r = np.random.default_rng(321)
    k = torch.zeros(hkv, n, d) if tail == "equal" else torch.tensor(r.standard_normal((hkv, n, d)) * 0.2).float()
    k[:, at] = 4.0
    v = torch.full((hkv, n, d), 96.0) if tail == "equal" else torch.tensor(1 + r.standard_normal((hkv, n, d))).float()
    v[:, at] = 0.0
    put_rows(c, 0, 0, k)
    put_rows(c, 1, 0, v)
    gap = torch.linspace(10, 45, hq)[torch.tensor(r.permutation(hq))]
    q = (gap / (4 * d ** 0.5))[None, :, None].expand(1, hq, d).to(c.query(hq).dtype).contiguous().cuda()
    before = c.scores()
    work = before.clone()
    o, lse = sa.paged_decode(c.cache, q, scores=work)
    assert status(sa.paged_decode) == (0, 0)
    check_decode(c, q, o, lse, before=before, after=work)


@pytest.mark.parametrize("cache", ["fp16", "e4m3"])
def test_logits_that_fall_and_rise_over_a_long_row(sa, cache):
    """Tiles of keys whose logits step down and up by tens of nats: the running
    maximum is raised many times, and most tiles lie far below it."""
    n, hkv, d = 4096, 2, 64
    c = Case(sa, 330, [n, n], hkv, d, 64, cache, scales=False)
    r = np.random.default_rng(331)
    level = torch.tensor(r.permutation(n // 64) / (n // 64) * 4.0).repeat_interleave(64).float()
    for s in range(2):
        k = torch.tensor(r.standard_normal((hkv, n, d)) * 0.05).float() + (level if s else level.sort().values)[None, :, None]
        put_rows(c, 0, s, k)
    q = torch.full((2, 16, d), 1.0, dtype=c.query(16).dtype, device="cuda")  # logits 0 .. 32
    o, lse = sa.paged_decode(c.cache, q)
    check_decode(c, q, o, lse)


# ------------------------------------------------ ranges that do not ascend
@pytest.mark.parametrize("cache,t", [("bf16", "bf16"), ("e4m3", "bf16"), ("e4m3", "fp16")])
@pytest.mark.parametrize("cu,lens,bad", [
    ([0, 99, 8, 12], [20, 30, 40], [0, 1]),                 # a valid range behind a start past the rows
    ([0, 4, 2, 12], [20, 30, 40], [1]),                     # rows 2 and 3 belong to two ranges
    ([0, 12, 3, 9, 1, 5], [20, 12, 6, 9, 7], [1, 3]),       # ranges inside another
    ([5, 9, 2, 2, 12], [9, 9, 0, 30], [1]),                 # does not begin at row 0
    ([0, -5, 3, 7], [3, 8, 60], [0, 1]),                    # a negative start
    ([0, 12, 0, 12, 0, 12] * 8 + [2 ** 31 - 1, -2 ** 31, 0, 4], [33] * 51, None),
])
def test_append_writes_every_valid_range_whatever_their_order(sa, cu, lens, bad, cache, t):
    c = Case(sa, 340, lens, 2, 64, 16, cache)
    total = 12
    valid = [0 <= a <= b <= total and b - a <= n for a, b, n in zip(cu, cu[1:], lens)]
    assert bad is None or [s for s, ok in enumerate(valid) if not ok] == bad
    kn, vn = new_rows(c, total, t)
    bits = torch.uint8 if cache == "e4m3" else torch.int16
    want = [p.view(bits).cpu().numpy().copy() for p in (c.k, c.v)]
    scores = c.scores()
    old = scores.clone()
    sa.paged_append(c.cache, kn, vn, torch.tensor(cu, dtype=torch.int32).cuda(), scores)
    assert status(sa.paged_append) == (sa.SA_ERR_DEVICE, LOCAL["where_range"])
    for i, (x, scale) in enumerate(((kn, c.ks), (vn, c.vs))):
        rows = expect_append(c, x, scale)
        for s, ok in enumerate(valid):
            for r in range(cu[s], cu[s + 1]) if ok else ():
                j = lens[s] - (cu[s + 1] - r)
                want[i][c.table_np[s, j // 16], :, j % 16] = rows[r]
                old[s, :, j] = 0
        np.testing.assert_array_equal((c.k, c.v)[i].view(bits).cpu().numpy(), want[i])
    assert torch.equal(scores, old)


# --------------------------------------------------- offsets past 32 bits
def test_eviction_moves_rows_past_32_bits(sa):
    """Pages 0 and 1 are 2^32 + 4096 elements apart: rows move in place, and from
    either page to the other, and every byte of both pools is compared."""
    d, page, far = 128, 16, 2 ** 32 + 4096
    flat = [torch.zeros(far + 2 * page * d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    pools = [torch.as_strided(x, (2, 2, page, d), (far, page * d, d, 1)) for x in flat]
    g = torch.Generator(device="cuda").manual_seed(5)
    lens = torch.empty(1, dtype=torch.int32, device="cuda")
    for src, dst, n, budget in (([1, 0], None, 29, 20), ([0, 1], None, 32, 7), ([1], [0], 16, 9), ([0], [1], 13, 5)):
        for x in pools:
            x.copy_(torch.randn(2, 2, page, d, device="cuda", generator=g))
        was = [x.clone() for x in pools]
        scores = torch.rand(1, 2, len(src) * page, device="cuda", generator=g)
        host = scores.cpu().numpy()
        cache = sa.PagedCache(*pools, torch.tensor([src], dtype=torch.int32, device="cuda"), lens.fill_(n))
        to = None if dst is None else torch.tensor([dst], dtype=torch.int32, device="cuda")
        keep = sa.cache_evict(cache, scores, budget, 1, 2, to)
        assert status(sa.cache_evict) == (0, 0) and lens.item() == budget
        want = [x.clone() for x in was]
        for h in range(2):
            kept = Pg.keep_one(host[0, h], n, budget, 1, 2)
            assert keep[0, h].tolist() == kept.tolist()
            for x, y in zip(want, was):
                for i, j in enumerate(kept.tolist()):
                    x[(dst or src)[i // page], h, i % page] = y[src[j // page], h, j % page]
        for x, y in zip(pools, want):
            assert torch.equal(x, y)
    for x in flat:  # nothing between the pages was touched
        assert not x[2 * page * d:far].any()


# ------------------------------------------------------------ two streams
def test_weights_of_calls_on_two_streams_do_not_meet(sa):
    cs = [Case(sa, 350 + i, [700, 33, 90 + 40 * i], 2, 128, 16) for i in range(2)]
    qs = [c.query(8) for c in cs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    calls = []
    for k in range(12):
        c, q, s = cs[k % 2], qs[k % 2], streams[k % 2]
        before = c.scores()
        calls.append((c, q, s, before, before.clone(), torch.full_like(before, -1.0), (0, 0) if k % 4 < 2 else (60, 4)))
    torch.cuda.synchronize()
    got = [sa.paged_decode(c.cache, q, *see, scores=work, stream=s) if k % 3 else
           sa.paged_decode(c.cache, q, *see, scores=work, scores_out=out, stream=s, keep_tail=False)
           for k, (c, q, s, _, work, out, see) in enumerate(calls)]
    torch.cuda.synchronize()
    for k, ((c, q, _, before, work, out, see), (o, lse)) in enumerate(zip(calls, got)):
        after = work if k % 3 else out
        check_decode(c, q, o, lse, *see, None, before, after)
        for s, n in enumerate(c.lens):
            assert torch.equal(after[s, :, n:], before[s, :, n:])


def test_evictions_and_appends_on_two_streams_do_not_meet(sa):
    cs = [Case(sa, 360 + i, [300, 80 + i], 2, 64, 16) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    scores = [c.scores() for c in cs]
    host = [s.cpu().numpy() for s in scores]
    rows = [[c.read(c.table_np, s, n) for s, n in enumerate(c.lens)] for c in cs]
    new = [new_rows(c, 2, "bf16", i) for i, c in enumerate(cs)]
    torch.cuda.synchronize()
    keeps = []
    for budget in (70, 40):
        for c, w, s in zip(cs, scores, streams):
            keeps.append(sa.cache_evict(c.cache, w, budget, 2, 5, stream=s))
    for c, (kn, vn), w, s in zip(cs, new, scores, streams):
        sa.paged_append(c.cache, kn, vn, scores=w, stream=s)  # over the last position
    torch.cuda.synchronize()
    for i, c in enumerate(cs):
        for s, n in enumerate(c.lens):
            got = c.read(c.table_np, s, 40)
            for h in range(2):
                a = Pg.keep_one(host[i][s, h], n, 70, 2, 5)
                b = Pg.keep_one(host[i][s, h][a], 70, 40, 2, 5)
                assert keeps[i][s, h].tolist() == a.tolist() and keeps[2 + i][s, h].tolist() == b.tolist()
                for x in range(2):
                    want = rows[i][s][x][h][a[b]]
                    want[39] = new[i][x][s, h].view(torch.int16).cpu().numpy()
                    np.testing.assert_array_equal(got[x][h], want)
                left = host[i][s, h][a[b]].copy()
                left[39] = 0
                np.testing.assert_array_equal(scores[i][s, h, :40].cpu().numpy(), left)
