"""Cases of the paged key/value cache operators: append, decode attention and
eviction, each in a plain form of elementary torch operations and through the
library's entry points.

A paged cache holds keys and values in pools of pages [n_pages, Hkv,
page_size, d]; page_table[s, i] names the page of positions
i * page_size .. of sequence s, seq_lens[s] how many positions it holds.

* append: the new tokens' keys and values go to the last positions of their
  sequences (a cache in 8 bits stores e4m3(x / scale)), and their accumulated
  weights start at zero.
* decode: attention of one query token per sequence over its cache, all of it
  or the first `sinks` and the last `window` positions, with the log-sum-exp;
  on request each key's softmax weight, summed over the query heads that share
  it, is added to its accumulated weight.
* evict: the first `sinks`, the last `recent` and the positions of the highest
  accumulated weight, `budget` in all, chosen for each key/value head (ties to
  the lowest position), are moved, in order, to the pages of another table.
"""
import math
import random

import torch

own = False

F8 = torch.float8_e4m3fn
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": F8}
F8_MAX = 448.0


# ------------------------------------------------------------------- cases
def _append(name, q_type, cache, n_seq, new_lo, new_hi, old_hi, kv_heads, d, page):
    return {"name": name, "op": "append", "type": q_type, "cache": cache, "n_seq": n_seq,
            "new_lo": new_lo, "new_hi": new_hi, "old_hi": old_hi, "kv_heads": kv_heads, "d": d,
            "page": page}


def _decode(name, q_type, cache, n_seq, lo, hi, heads, kv_heads, d, page, window=0, sinks=0,
            scores=False):
    return {"name": name, "op": "decode", "type": q_type, "cache": cache, "n_seq": n_seq, "lo": lo,
            "hi": hi, "heads": heads, "kv_heads": kv_heads, "d": d, "page": page,
            "window": window, "sinks": sinks, "scores": scores}


def _evict(name, cache, n_seq, lo, hi, kv_heads, d, page, budget, sinks, recent):
    return {"name": name, "op": "evict", "type": "bf16", "cache": cache, "n_seq": n_seq, "lo": lo,
            "hi": hi, "kv_heads": kv_heads, "d": d, "page": page, "budget": budget,
            "sinks": sinks, "recent": recent}


def listed():
    return [
        # one decode step of a batch: a token per sequence, latency counts
        _append("append_step_16", "bf16", "bf16", 16, 1, 1, 32768, 8, 128, 16),
        # a batch of ragged prompts enters a cache in 8 bits
        _append("append_prompts_e4m3", "bf16", "e4m3", 8, 513, 16384, 4096, 8, 128, 64),
        # a single user's short chat: the smallest call
        _decode("decode_1x1777", "bf16", "bf16", 1, 1777, 1777, 32, 8, 128, 16),
        # a single user's long document: one row, the whole card
        _decode("decode_1x128k", "bf16", "bf16", 1, 131072, 131072, 32, 8, 128, 64),
        # the library's own decode workload as a paged cache: 16 long sequences
        _decode("decode_16x128k", "bf16", "bf16", 16, 65537, 131072, 32, 8, 128, 128),
        # many short chats, a key/value head per query head, pages of an odd size
        _decode("decode_96_short_mha", "fp16", "fp16", 96, 3, 2048, 12, 12, 64, 24),
        # a cache in 8 bits with per-head scales, 8 query heads per key/value head
        _decode("decode_24_e4m3", "bf16", "e4m3", 24, 1000, 32768, 64, 8, 128, 32),
        # streaming: a window and the first tokens of long sequences
        _decode("decode_32_window", "bf16", "bf16", 32, 100, 65536, 32, 8, 128, 16, 4096, 128),
        # a step that also accumulates the weights that the eviction reads
        _decode("decode_8x32k_scores", "bf16", "bf16", 8, 16384, 32768, 32, 8, 128, 16,
                scores=True),
        # one sequence reaches its budget
        _evict("evict_1x8k", "bf16", 1, 8192, 8192, 8, 128, 16, 2048, 4, 256),
        # a batch of long prompts is cut to a quarter
        _evict("evict_16x32k", "bf16", 16, 20000, 32768, 8, 128, 64, 8192, 128, 1024),
        # a ragged batch in 8 bits, some of it below its budget
        _evict("evict_48_e4m3", "e4m3", 48, 700, 16000, 4, 64, 24, 1000, 4, 333),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "decode", "evict"])
    cache = rng.choice(["bf16", "bf16", "fp16", "e4m3"])
    q_type = rng.choice(["bf16", "fp16"]) if cache == "e4m3" else cache
    d = rng.choice([64, 128, 128])
    kv_heads = rng.choice([1, 2, 3, 4, 8, 8, 12])
    page = rng.choice([1, 7, 16, 16, 24, 32, 64, 100, 128, 256])
    n_seq = _log(rng, 1, 128)
    # positions over the whole batch and all heads, at most a quarter of the largest listed case
    room = 16 * 131072 * 8 // 4 // (n_seq * kv_heads)
    hi = _log(rng, 16, min(131072, room))
    lo = rng.randint(1, hi)
    if op == "append":
        new_hi = rng.choice([1, min(hi, 5), hi])
        c = _append("", q_type, cache, n_seq, rng.randint(1, new_hi), new_hi, _log(rng, 1, 20000),
                    kv_heads, d, page)
    elif op == "decode":
        heads = kv_heads * rng.choice([1, 2, 4, 4, 5, 8, 16])
        window = rng.choice([0, 0, 1, _log(rng, 1, hi)])
        sinks = rng.choice([0, 1, 4, 128]) if window else 0
        c = _decode("", q_type, cache, n_seq, lo, hi, heads, kv_heads, d, page, window, sinks,
                    rng.random() < 0.4)
    else:
        budget = _log(rng, 1, hi)
        sinks = min(rng.choice([0, 1, 4, 100]), budget)
        recent = rng.randint(0, budget - sinks)
        c = _evict("", cache, n_seq, lo, hi, kv_heads, d, page, budget, sinks, recent)
    del c["name"]
    return c


def _spread(tag, n, lo, hi):
    """n lengths in [lo, hi], the same for every seed; the first is hi."""
    r = random.Random("%s %d %d %d" % (tag, n, lo, hi))
    return [hi] + [r.randint(lo, hi) for _ in range(n - 1)]


def _lens(case):
    """(positions of each sequence, of them new)."""
    if case["op"] != "append":
        return _spread("len", case["n_seq"], case["lo"], case["hi"]), None
    new = _spread("new", case["n_seq"], case["new_lo"], case["new_hi"])
    old = _spread("old", case["n_seq"], 0, case["old_hi"])
    return [a + b for a, b in zip(old, new)], new


def _visible(case, n):
    """(first positions, start of the last ones) that a query at length n sees."""
    lo = max(0, n - case["window"]) if case["window"] else 0
    return min(case["sinks"], lo), lo


# ------------------------------------------------------------------ inputs
def _randn(g, shape, dtype, scale=1.0):
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 28):
        part = flat[i:i + (1 << 28)]
        x = torch.randn(part.numel(), device="cuda", dtype=torch.bfloat16, generator=g)
        part.copy_((x.float() * scale).clamp_(-F8_MAX, F8_MAX) if dtype == F8 else x)
    return out


def _pages(n, page):
    return (n + page - 1) // page


def _table(g, rows, max_pages, first, n_pages):
    """Page table with the given pages per row, in random order of the pool."""
    order = torch.randperm(n_pages, device="cuda", generator=g).to(torch.int32) + first
    t = torch.zeros(len(rows), max_pages, dtype=torch.int32, device="cuda")
    at = 0
    for s, n in enumerate(rows):
        t[s, :n] = order[at:at + n]
        at += n
    return t


class State:
    pass


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 17)
    st = State()
    st.case = case
    lens, new = _lens(case)
    op, page, d, H, n = case["op"], case["page"], case["d"], case["kv_heads"], case["n_seq"]
    cdt, qdt = DTYPES[case["cache"]], DTYPES[case["type"]]
    st.lens_host, st.new_host = lens, new
    rows = [_pages(x, page) for x in lens]
    st.max_pages = max(rows)
    if op == "decode":
        st.most_visible = max(a + x - b for x in lens for a, b in [_visible(case, x)])
    n_src = n_pages = sum(rows)
    if op == "evict":
        st.kept = [min(x, case["budget"]) for x in lens]
        dst = [_pages(x, page) for x in st.kept]
        n_pages += sum(dst)
    scale = None
    if cdt == F8:  # per-head scales as a calibration leaves them: the largest values near 448
        scale = [0.01 * (0.5 + torch.rand(H, device="cuda", generator=g)) for _ in range(2)]
    st.k_scale, st.v_scale = scale if scale else (None, None)
    fill = 60.0 if cdt == F8 else 1.0
    st.k = _randn(g, (n_pages, H, page, d), cdt, fill)
    st.v = _randn(g, (n_pages, H, page, d), cdt, fill)
    st.table = _table(g, rows, st.max_pages, 0, n_src)
    st.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    cap = st.max_pages * page
    st.scores = None
    if op != "decode" or case["scores"]:
        # accumulated weights: many small, a few large
        st.scores = torch.exp(1.5 * torch.randn(n, H, cap, device="cuda", generator=g) - 3)
    if op == "append":
        total = sum(new)
        st.k_new = _randn(g, (total, H, d), qdt)
        st.v_new = _randn(g, (total, H, d), qdt)
        cu = [0]
        for x in new:
            cu.append(cu[-1] + x)
        st.cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    elif op == "decode":
        st.q = _randn(g, (n, case["heads"], d), qdt)
        st.o = torch.empty_like(st.q)
        st.lse = torch.empty(n, case["heads"], dtype=torch.float32, device="cuda")
        st.scores_out = torch.zeros_like(st.scores) if case["scores"] else None
    else:
        st.dst_table = _table(g, dst, max(dst), n_src, n_pages - n_src)
        for i in range(n_src, n_pages, 1 << 16):  # pages that the cache hands out anew
            st.k[i:i + (1 << 16)].view(torch.uint8).zero_()
            st.v[i:i + (1 << 16)].view(torch.uint8).zero_()
        st.keep = torch.empty(n, H, case["budget"], dtype=torch.int32, device="cuda")
        st.scores_out = torch.zeros(n, H, max(dst) * page, device="cuda")
        st.lens_out = torch.empty_like(st.lens)
    if own:
        import content_adaptive_block_sa_b200 as sa
        st.sa = sa
        st.cache = sa.PagedCache(st.k, st.v, st.table, st.lens, st.k_scale, st.v_scale)
        if op == "append":
            st.desc = sa.paged_append_desc(st.k_new, st.v_new, st.scores)
            st.ws = sa.paged_append_workspace(st.cache, st.desc)
        elif op == "decode":
            st.desc = sa.paged_decode_desc(st.q, st.o, case["window"], case["sinks"],
                                           scores=st.scores)
            st.ws = sa.paged_decode_workspace(st.cache, st.desc)
        else:
            st.desc = sa.cache_evict_desc(st.scores, case["budget"], case["sinks"],
                                          case["recent"], dst_table=st.dst_table,
                                          scores_out=st.scores_out)
            st.ws = sa.cache_evict_workspace(st.cache, st.desc)
    return st


# ------------------------------------------------------------- plain forms
def _rows(pool, table, pos):
    """The pool's rows at positions [n_seq, m]: [n_seq, Hkv, m, d] in 32 bits."""
    page = pool.shape[2]
    at = table.gather(1, pos // page).long()
    x = _bits(pool)[at, :, pos % page]
    return (x.view(F8) if pool.dtype == F8 else x).float().transpose(1, 2)


def _plain_append(st):
    page, H = st.case["page"], st.case["kv_heads"]
    total = st.k_new.shape[0]
    count = st.cu.diff()
    t = torch.arange(total, device="cuda")
    seq = torch.repeat_interleave(torch.arange(st.case["n_seq"], device="cuda"), count.long(),
                                  output_size=total)
    pos = (st.lens[seq] - count[seq] + t - st.cu[seq]).long()
    at = st.table[seq, pos // page].long()
    for pool, x, scale in ((st.k, st.k_new, st.k_scale), (st.v, st.v_new, st.v_scale)):
        if pool.dtype == F8:
            y = (x.float() / scale[:, None]).clamp(-F8_MAX, F8_MAX).to(F8)
            pool.view(torch.uint8)[at, :, pos % page] = y.view(torch.uint8)
        else:
            pool[at, :, pos % page] = x
    st.scores[seq[:, None], torch.arange(H, device="cuda")[None], pos[:, None]] = 0.0
    return {"k": st.k, "v": st.v, "scores": st.scores}


def _plain_decode(st):
    c = st.case
    n_seq, H, d = c["n_seq"], c["kv_heads"], c["d"]
    rep = c["heads"] // H
    # the visible positions of each sequence side by side: the first ones, then the last ones
    n = st.lens.long()[:, None]
    lo = (n - c["window"]).clamp(min=0) if c["window"] else torch.zeros_like(n)
    first = lo.clamp(max=c["sinks"])
    i = torch.arange(st.most_visible, device="cuda")[None]
    pos = torch.where(i < first, i, i - first + lo)
    seen = pos < n
    pos = torch.where(seen, pos, 0)
    k = _rows(st.k, st.table, pos)
    if st.k_scale is not None:
        k = k * st.k_scale[:, None, None]
    x = torch.matmul(st.q.float().view(n_seq, H, rep, d), k.transpose(2, 3)) / math.sqrt(d)
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    del k
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - top)
    z = e.sum(-1, keepdim=True)
    p = e / z
    v = _rows(st.v, st.table, pos)
    if st.v_scale is not None:
        v = v * st.v_scale[:, None, None]
    out = {"o": torch.matmul(p, v).view(st.q.shape).to(st.q.dtype),
           "lse": (top + torch.log(z)).view(st.lse.shape)}
    if c["scores"]:
        out["scores"] = st.scores.scatter_add(2, pos[:, None].expand(n_seq, H, -1), p.sum(2))
    return out


def _bits(pool):
    return pool.view(torch.uint8) if pool.dtype == F8 else pool


def _plain_evict(st):
    c = st.case
    n_seq, H, page, budget = c["n_seq"], c["kv_heads"], c["page"], c["budget"]
    m = min(budget, st.scores.shape[2])
    pos = torch.arange(st.scores.shape[2], device="cuda")
    n = st.lens[:, None]
    always = (pos < c["sinks"]) | (pos >= n - c["recent"]) | (n <= budget)
    rank = st.scores.masked_fill(always[:, None], math.inf)
    rank = rank.masked_fill((pos >= n)[:, None], -math.inf)
    order = torch.sort(rank, dim=2, descending=True, stable=True).indices[:, :, :m]
    order = torch.where(order < n[:, None], order, pos.numel()).sort(2).values
    kept = order < pos.numel()
    st.keep.fill_(-1)
    st.keep[:, :, :m] = torch.where(kept, order, -1).to(torch.int32)
    # what is not kept repeats the first row's move
    src = torch.where(kept, order, order[:, :, :1])
    to = torch.where(kept, torch.arange(m, device="cuda"), 0)
    seqs = torch.arange(n_seq, device="cuda")[:, None, None]
    heads = torch.arange(H, device="cuda")[None, :, None]
    a, b = st.table[seqs, src // page].long(), st.dst_table[seqs, to // page].long()
    for pool in (_bits(st.k), _bits(st.v)):
        pool[b, heads, to % page] = pool[a, heads, src % page]
    st.scores_out[seqs, heads, to] = st.scores.gather(2, src)
    st.lens_out.copy_(st.lens.clamp(max=budget))
    return {"keep": st.keep, "lens": st.lens_out, "scores": st.scores_out, "k": st.k, "v": st.v}


def run(st):
    op = st.case["op"]
    if not own:
        return {"append": _plain_append, "decode": _plain_decode, "evict": _plain_evict}[op](st)
    if op == "append":
        st.sa.sa_paged_append(st.cache, st.desc, st.k_new, st.v_new, st.cu, st.scores, st.ws)
        return {"k": st.k, "v": st.v, "scores": st.scores}
    if op == "decode":
        st.sa.sa_paged_decode(st.cache, st.desc, st.q, st.o, st.lse, st.scores, st.scores_out,
                              st.ws)
        out = {"o": st.o, "lse": st.lse}
        if st.scores is not None:
            out["scores"] = st.scores_out
        return out
    st.sa.sa_cache_evict(st.cache, st.desc, st.scores, st.dst_table, st.keep, st.scores_out,
                         st.lens_out, st.ws)
    return {"keep": st.keep, "lens": st.lens_out, "scores": st.scores_out, "k": st.k, "v": st.v}


# -------------------------------------------------------------------- work
def work(case):
    lens, new = _lens(case)
    H, d = case["kv_heads"], case["d"]
    size = 1 if case["cache"] == "e4m3" else 2
    if case["op"] == "append":
        t = sum(new)
        return {"bytes": t * H * (d * 2 * (2 + size) + 4), "flops": 0}
    if case["op"] == "decode":
        seen = 0
        for n in lens:
            first, lo = _visible(case, n)
            seen += first + n - lo
        b = seen * H * d * size * 2 + case["n_seq"] * case["heads"] * (d * 4 + 4)
        if case["scores"]:
            b += sum(lens) * H * 8
        return {"bytes": b, "flops": 4 * seen * case["heads"] * d}
    kept = sum(min(n, case["budget"]) for n in lens)
    read = sum(n for n in lens if n > case["budget"])
    return {"bytes": H * (read * 4 + kept * (d * size * 4 + 12)), "flops": 0}


# ------------------------------------------------------------------- exact
def exact(case, seed):
    st = prepare(case, seed)
    return {"append": _exact_append, "decode": _exact_decode, "evict": _exact_evict}[case["op"]](st)


def _round_e4m3(x):
    """e4m3 values of 64-bit numbers: nearest, ties to even, at most 448."""
    a = x.abs().clamp(max=F8_MAX)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    return torch.copysign((torch.round(a / step) * step).clamp(max=F8_MAX), x)


def _exact_append(st):
    page = st.case["page"]
    out = [st.k.float(), st.v.float()]
    table, cu = st.table.cpu().tolist(), st.cu.cpu().tolist()
    for s, n in enumerate(st.lens_host):
        start = n - st.new_host[s]
        for i in range(start // page, _pages(n, page)):
            a, b = max(start, i * page), min(n, (i + 1) * page)
            at = slice(cu[s] + a - start, cu[s] + b - start)
            for pool, x, scale in ((out[0], st.k_new, st.k_scale), (out[1], st.v_new, st.v_scale)):
                y = x[at].double().transpose(0, 1)
                if scale is not None:
                    y = _round_e4m3(y / scale.double()[:, None, None])
                pool[table[s][i], :, a - i * page:b - i * page] = y.float()
        st.scores[s, :, start:n] = 0
    return {"k": out[0], "v": out[1], "scores": st.scores}


def _exact_decode(st):
    c = st.case
    H, page, rep = c["kv_heads"], c["page"], c["heads"] // c["kv_heads"]
    o = torch.zeros(c["n_seq"], c["heads"], c["d"], dtype=torch.float64, device="cuda")
    lse = torch.zeros(c["n_seq"], c["heads"], dtype=torch.float64, device="cuda")
    total = st.scores.double() if c["scores"] else None
    every = torch.arange(st.max_pages * page, device="cuda")
    for s, n in enumerate(st.lens_host):
        pos = every[:n]
        if c["window"]:
            pos = pos[(pos >= n - c["window"]) | (pos < c["sinks"])]
        where = st.table[s].long()[pos // page] * page + pos % page
        for h in range(H):
            ks, vs = [], []
            for pool, scale, to in ((st.k, st.k_scale, ks), (st.v, st.v_scale, vs)):
                flat = _bits(pool)[where // page, h, where % page]
                x = (flat.view(F8) if pool.dtype == F8 else flat).double()
                to.append(x if scale is None else x * scale[h].double())
            x = st.q[s, h * rep:(h + 1) * rep].double() @ ks[0].t() * c["d"] ** -0.5
            z = torch.logsumexp(x, 1)
            p = torch.exp(x - z[:, None])
            o[s, h * rep:(h + 1) * rep] = p @ vs[0]
            lse[s, h * rep:(h + 1) * rep] = z
            if total is not None:
                total[s, h].index_add_(0, pos, p.sum(0))
    out = {"o": o, "lse": lse}
    if total is not None:
        out["scores"] = total
    return out


def _exact_evict(st):
    c = st.case
    page, budget = c["page"], c["budget"]
    k, v = _bits(st.k).clone(), _bits(st.v).clone()
    keep = torch.full_like(st.keep, -1)
    scores = torch.zeros_like(st.scores_out)
    for s, n in enumerate(st.lens_host):
        pos = torch.arange(n, device="cuda")
        for h in range(c["kv_heads"]):
            # rank by (kept anyway, weight, lower position)
            w = st.scores[s, h, :n].double()
            if n > budget:
                w = torch.where((pos < c["sinks"]) | (pos >= n - c["recent"]), torch.inf, w)
            kept = torch.argsort(-w, stable=True)[:budget].sort().values
            m = kept.numel()
            keep[s, h, :m] = kept.to(torch.int32)
            scores[s, h, :m] = st.scores[s, h][kept]
            a, b = st.table[s].long()[kept // page], st.dst_table[s].long()[pos[:m] // page]
            k[b, h, pos[:m] % page] = k[a, h, kept % page]
            v[b, h, pos[:m] % page] = v[a, h, kept % page]
    view = (lambda x: x.view(F8)) if st.k.dtype == F8 else (lambda x: x)
    return {"keep": keep, "lens": torch.tensor(st.kept, dtype=torch.int32), "scores": scores,
            "k": view(k), "v": view(v)}
