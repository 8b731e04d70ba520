"""Bounds of the 4-bit cache's pages, the pages chosen by them, and the attention
over the chosen pages on the B200.  Bounds, pages and lengths have to be equal to
the definition's; the attention is compared in binary64 within the bound that its
roundings allow."""
import math

import numpy as np
import pytest
import torch

from tests import kv4_ref as ref
from tests.gpu_util import wq
from tests.test_kv4_gpu import COUNTERS, fill, ints, new_cache, starts_of

pytestmark = pytest.mark.gpu


def random_cache(seed, pages, heads, d, page, group, spread=1.0):
    """Any codes, scales of a few sizes, any zeros: a cache as if written."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = wq().kv4_cache(pages, heads, d, page_size=page, group=group)
    for codes in (c.k_codes, c.v_codes):
        codes.copy_(torch.randint(0, 256, codes.shape, generator=g, device="cuda",
                                  dtype=torch.uint8))
    for meta in (c.k_meta, c.v_meta):
        meta[..., 0] = torch.exp2(spread * torch.randn(meta.shape[:-1], generator=g,
                                                       device="cuda") - 3)
        meta[..., 1] = torch.randint(0, 16, meta.shape[:-1], generator=g, device="cuda").half()
    return c


def key_values(cache):
    """All keys as float64 [pages, heads, page, D]."""
    codes, meta = cache.k_codes.cpu().numpy(), cache.k_meta.cpu().numpy().astype(np.float64)
    u = ref.unpack(codes, "k").reshape(*codes.shape[:3], -1, cache.group)
    return ((u - meta[..., 1:]) * meta[..., :1]).reshape(*codes.shape[:3], -1)


def grid_of(top):
    """The smallest power of two with 127 times it at least top; 1 for 0."""
    if top == 0:
        return 1.0
    e = math.floor(math.log2(top)) - 8
    while 127 * 2.0 ** e < top:
        e += 1
    return 2.0 ** e


def expected_bounds(keys, lens, rows, table, page, codes, grid):
    for b, (n, t) in enumerate(zip(lens, rows)):
        if t == 0:
            continue
        for j in range(max(0, n - t) // page, (n + page - 1) // page):
            p = int(table[b][j])
            for h in range(keys.shape[1]):
                k = keys[p, h, :n - j * page]
                g = grid_of(np.abs(k).max())
                codes[p, h, 0], codes[p, h, 1] = np.floor(k.min(0) / g), np.ceil(k.max(0) / g)
                grid[p, h] = g


def expected_pages(q, codes, grid, lens, rows, table, page, max_pages, first, last, n_rows):
    """lists [n_rows, H, max_pages], lens [n_rows]; q [rows, Hq, D] float64."""
    heads = codes.shape[1]
    r = q.shape[1] // heads
    lists = np.full((n_rows, heads, max_pages), -1, dtype=np.int64)
    held = np.full(n_rows, -1, dtype=np.int64)
    at = 0
    for b, (n, t) in enumerate(zip(lens, rows)):
        for i in range(t):
            limit = max(0, n - t + i + 1)
            pages = (limit + page - 1) // page
            count = min(pages, max_pages)
            held[at] = limit - (pages - count) * page
            ids = np.asarray(table[b][:pages], dtype=np.int64)
            for h in range(heads):
                x = q[at, h * r:(h + 1) * r]
                c = np.rint(x / grid_of(np.abs(x).max()))
                up, down = np.maximum(c, 0).sum(0), np.minimum(c, 0).sum(0)
                lo, hi = codes[ids, h, 0].astype(np.float64), codes[ids, h, 1].astype(np.float64)
                score = (hi @ up + lo @ down).astype(np.float32) * grid[ids, h].astype(np.float32)
                must = [j for j in range(pages) if j < first or j >= pages - last]
                if pages > max_pages:
                    free = sorted((j for j in range(first, pages - last)),
                                  key=lambda j: (-score[j], j))[:max_pages - first - last]
                    chosen = sorted(must + free)
                else:
                    chosen = range(pages)
                lists[at, h, :count] = ids[list(chosen)]
            at += 1
    return lists, held


def attention_over(q, cache, lists, held, scale):
    """Each row and kv head over its own list, float64, with the bound."""
    kc, vc = cache.k_codes.cpu().numpy(), cache.v_codes.cpu().numpy()
    km, vm = cache.k_meta.cpu().numpy(), cache.v_meta.cpu().numpy()
    x = q.double().cpu().numpy()
    r = x.shape[1] // cache.kv_heads
    out, bound = np.zeros_like(x), np.zeros_like(x)
    for i, n in enumerate(held):
        if n <= 0:
            continue
        for h in range(cache.kv_heads):
            one = slice(h, h + 1)
            k = ref.sequence_values(kc[:, one], km[:, one], lists[i, h], n, cache.page_size, "k")
            v = ref.sequence_values(vc[:, one], vm[:, one], lists[i, h], n, cache.page_size, "v")
            o, e = ref.attention(x[i:i + 1, h * r:(h + 1) * r], k, v, n, scale, True)
            out[i, h * r:(h + 1) * r], bound[i, h * r:(h + 1) * r] = o[0], e[0]
    return out, bound


FORMATS = [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128)]


@pytest.mark.parametrize("d,group", FORMATS)
@pytest.mark.parametrize("heads,page,lens,rows", [
    (1, 16, [1], [1]),
    (8, 64, [777], [1]),
    (3, 32, [5, 64, 33, 320], [5, 7, 33, 320]),
    (2, 128, [300, 129, 128], [2, 1, 1]),
    (4, 256, [700], [500]),
    (5, 16, [100, 0, 17, 3], [50, 0, 17, 6]),
    (2, 16, [40] * 45, [3] * 45),
])
def test_bounds(d, group, heads, page, lens, rows):
    table, pages = ref.random_batch(d + group, lens, page)
    cache = random_cache(d + page, pages, heads, d, page, group)
    bounds = wq().kv4_bounds(cache)
    bounds.codes.fill_(99)
    bounds.grid.fill_(-5.0)
    codes, grid = bounds.codes.cpu().numpy().astype(np.int64), bounds.grid.cpu().numpy()
    expected_bounds(key_values(cache), lens, rows, table, page, codes, grid)
    wq().kv4_update_bounds(cache, bounds, ints(lens), ints(table), ints(starts_of(rows)),
                           rows=sum(rows) + 3)
    assert np.array_equal(bounds.codes.cpu().numpy(), codes)
    assert np.array_equal(bounds.grid.cpu().numpy(), grid)
    assert wq().get_device_error() == 0


def test_bounds_of_uniform_rows_and_of_zeros():
    """rows/seqs rows each without row_starts; pages of zeros have the grid 1; NaN metadata
    behind a sequence's end is not looked at."""
    lens, page, heads, d = [50, 70, 33], 16, 2, 64
    table, pages = ref.random_batch(1, lens, page)
    cache = random_cache(2, pages, heads, d, page, 32, spread=4.0)
    cache.k_codes[int(table[1, 4])] = 0
    cache.k_meta[int(table[1, 4]), ..., 1] = 0
    cache.k_meta[int(table[0, 3]), :, 2:] = float("nan")
    bounds = wq().kv4_bounds(cache)
    codes, grid = bounds.codes.cpu().numpy().astype(np.int64), bounds.grid.cpu().numpy()
    expected_bounds(key_values(cache), lens, [20] * 3, table, page, codes, grid)
    wq().kv4_update_bounds(cache, bounds, ints(lens), ints(table), rows=60)
    assert np.array_equal(bounds.codes.cpu().numpy(), codes)
    assert np.array_equal(bounds.grid.cpu().numpy(), grid)
    assert grid[int(table[1, 4])].tolist() == [1.0, 1.0]


def random_bounds(seed, cache, levels=127):
    g = torch.Generator(device="cuda").manual_seed(seed)
    b = wq().kv4_bounds(cache)
    a = torch.randint(-levels, levels + 1, b.codes.shape, generator=g, device="cuda")
    b.codes.copy_(torch.stack((a.amin(2), a.amax(2)), 2).to(torch.int8))
    b.grid.copy_(torch.exp2(torch.randint(-6, -2, b.grid.shape, generator=g, device="cuda").float()))
    return b


def choose(q, cache, bounds, lens, rows, table, max_pages, first=1, last=2, behind=0, ragged=True):
    n = sum(rows)
    lists = torch.full((n + behind, cache.kv_heads, max_pages), 88, dtype=torch.int32, device="cuda")
    held = torch.full((n + behind,), 88, dtype=torch.int32, device="cuda")
    wq().kv4_select(q, cache, bounds, ints(lens), ints(table),
                    ints(starts_of(rows)) if ragged else None, max_pages=max_pages, first=first,
                    last=last, lists=lists, lens=held)
    assert wq().get_device_error() == 0
    x = q.double().cpu().numpy()
    want = expected_pages(x, bounds.codes.cpu().numpy(), bounds.grid.cpu().numpy(), lens, rows,
                          table, cache.page_size, max_pages, first, last, n + behind)
    assert np.array_equal(held.cpu().numpy(), want[1])
    assert np.array_equal(lists.cpu().numpy(), want[0])
    return lists, held


def queries(seed, n, heads, d):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(n, heads, d, generator=g).to(torch.bfloat16).cuda()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads,gqa,page,lens,rows,max_pages,first,last", [
    (1, 1, 16, [1], [1], 3, 1, 2),
    (8, 4, 64, [7777], [1], 16, 1, 2),
    (2, 7, 32, [500, 1000, 64, 3000], [1, 4, 2, 3], 8, 0, 1),
    (4, 1, 16, [100, 0, 2000, 3], [50, 0, 3, 6], 5, 2, 3),     # no room for a choice
    (2, 8, 16, [160, 176, 161, 159], [1, 1, 1, 1], 10, 1, 1),  # just as many pages, one more
    (1, 16, 128, [100_000], [2], 33, 1, 2),
    (1, 256, 16, [3000], [1], 20, 0, 2),
    (3, 5, 16, [90_000], [1], 64, 1, 2),                       # a cluster of CTAs
    (8, 2, 32, [70_000, 40_000], [1, 1], 1000, 4, 4),
    (2, 2, 16, [40] * 45, [3] * 45, 2, 0, 1),
    (1, 2, 16, [90_000, 70_000], [1, 1], 5000, 3, 2),          # more than the gathered places
    (1, 1, 16, [20_000] * 80, [8] * 80, 70, 1, 1),             # hundreds of rows
])
def test_chosen_pages(d, heads, gqa, page, lens, rows, max_pages, first, last):
    table, pages = ref.random_batch(d + page, lens, page)
    cache = wq().kv4_cache(pages, heads, d, page_size=page, group=32)
    bounds = random_bounds(d + gqa, cache)
    q = queries(heads + gqa, sum(rows) + 2, heads * gqa, d)
    choose(q, cache, bounds, lens, rows, table, max_pages, first, last, behind=2)


@pytest.mark.parametrize("what", ["zeros", "few levels", "same pages", "tiny", "huge", "one large"])
@pytest.mark.parametrize("length", [2000, 60_000])
def test_ties_and_queries_of_every_size(what, length):
    """Equal scores go to the lowest page, within a CTA and between those of a cluster."""
    heads, gqa, d, page, lens, rows = 2, 4, 128, 16, [length], [2]
    table, pages = ref.random_batch(3, lens, page)
    cache = wq().kv4_cache(pages, heads, d, page_size=page, group=32)
    bounds = random_bounds(5, cache)
    q = queries(6, 2, heads * gqa, d)
    if what == "zeros":
        q.zero_()
    elif what == "few levels":
        bounds.codes.copy_(bounds.codes.sign())
        q = q.sign()
    elif what == "same pages":
        table[0] = table[0][np.arange(table.shape[1]) % 7]
    elif what == "tiny":
        q = (q.double() * 2.0 ** -128).to(torch.bfloat16)
    elif what == "huge":
        q = (q.double() * 2.0 ** 125).to(torch.bfloat16)
        assert torch.isfinite(q).all()
    else:
        q[:, 3, 5] = 1e30
    for max_pages in (9, 64):
        choose(q, cache, bounds, lens, rows, table, max_pages)


@pytest.mark.parametrize("rows", [1, 200])
def test_the_most_pages(rows):
    """850,000 tokens in pages of 16, by a cluster and, for many rows, by one CTA."""
    page, n = 16, 53_248 * 16 - 5
    cache = wq().kv4_cache(500, 1, 64, page_size=page, group=32)
    bounds = random_bounds(7, cache)
    table = np.random.default_rng(1).integers(0, 500, (rows, 53_248)).astype(np.int32)
    lens = [n] + [4000] * (rows - 1)
    choose(queries(8, rows, 2, 64), cache, bounds, lens, [1] * rows, table, 100)


def test_uniform_rows_and_queries_as_a_slice():
    heads, d, page, lens, rows = 2, 64, 16, [900, 400, 1200], [2, 2, 2]
    table, pages = ref.random_batch(4, lens, page)
    cache = wq().kv4_cache(pages, heads, d, page_size=page, group=64)
    bounds = random_bounds(9, cache)
    wide = queries(10, 6, 3 * heads + 4, d)
    choose(wide[:, 2:2 + 3 * heads], cache, bounds, lens, rows, table, 12, ragged=False)


@pytest.mark.parametrize("d,group", FORMATS)
@pytest.mark.parametrize("heads,gqa,page,lens,rows,max_pages", [
    (1, 1, 16, [1], [1], 3),
    (8, 4, 64, [5000], [1], 12),
    (2, 7, 32, [500, 100, 1100], [1, 5, 2], 6),
    (3, 8, 16, [300, 0, 17, 3], [2, 0, 1, 6], 5),
    (2, 12, 128, [2000, 700], [2, 1], 4),
    (1, 40, 16, [600], [2], 9),
    (4, 2, 256, [3000] * 33, [1] * 33, 5),
])
def test_sparse_attention(d, group, heads, gqa, page, lens, rows, max_pages):
    table, pages = ref.random_batch(d + page, lens, page)
    cache = random_cache(d + group, pages, heads, d, page, group)
    n, behind = sum(rows), 3
    q = queries(d + heads, n + behind, heads * gqa, d)
    bounds = wq().kv4_bounds(cache)
    wq().kv4_update_bounds(cache, bounds, ints(lens), ints(table), ints(starts_of(lens)),
                           rows=sum(lens))
    codes, grid = bounds.codes.cpu().numpy().astype(np.int64), bounds.grid.cpu().numpy()
    # the rows' pages are not up to date: the call brings them
    keys = key_values(cache)
    for b, (m, t) in enumerate(zip(lens, rows)):
        for j in range(max(0, m - t) // page, (m + page - 1) // page):
            if t:
                bounds.codes[int(table[b, j])] = 1
                bounds.grid[int(table[b, j])] = 100.0
    out = torch.full((n + behind, heads * gqa, d), 7.0, dtype=torch.bfloat16, device="cuda")
    workspace = wq().kv4_workspace()
    got, lists, held = wq().kv4_sparse_attention(
        q, cache, bounds, ints(lens), ints(table), ints(starts_of(rows)), max_pages=max_pages,
        first=1, last=2, out=out, workspace=workspace)
    expected_bounds(keys, lens, rows, table, page, codes, grid)
    assert np.array_equal(bounds.codes.cpu().numpy(), codes)
    want = expected_pages(q.double().cpu().numpy(), codes, grid, lens, rows, table, page, max_pages,
                          1, 2, n + behind)
    assert np.array_equal(lists.cpu().numpy(), want[0])
    assert np.array_equal(held.cpu().numpy(), want[1])
    o, e = attention_over(q, cache, *want, d ** -0.5)
    ref.check(got[:n], o[:n], e[:n])
    assert (got[n:] == 7).all()
    assert not workspace[:COUNTERS].any()
    assert wq().get_device_error() == 0
    # its parts one by one give the same
    parts = torch.full_like(out, 7.0)
    again = wq().kv4_select(q, cache, bounds, ints(lens), ints(table), ints(starts_of(rows)),
                            max_pages=max_pages)
    assert torch.equal(again[0], lists) and torch.equal(again[1], held)
    wq().kv4_attention_pages(q, cache, lists, held, out=parts, workspace=workspace)
    assert torch.equal(parts, got)


def test_all_pages_give_the_dense_attention():
    """Lists that hold every page: the attention of wq_kv4_attention, bit for bit."""
    heads, gqa, d, page, lens = 4, 4, 128, 32, [900, 33, 640, 1]
    table, pages = ref.random_batch(8, lens, page)
    cache = new_cache(pages, heads, d, page, 64)
    fill(cache, lens, table)
    q = queries(2, len(lens), heads * gqa, d)
    bounds = wq().kv4_bounds(cache)
    wq().kv4_update_bounds(cache, bounds, ints(lens), ints(table), ints(starts_of(lens)),
                           rows=sum(lens))
    out, _, held = wq().kv4_sparse_attention(q, cache, bounds, ints(lens), ints(table),
                                             max_pages=table.shape[1])
    assert held.tolist() == lens
    assert torch.equal(out, wq().kv4_attention(q, cache, ints(lens), ints(table)))


def test_lists_of_the_callers_own():
    """Any pages in any order, the same page twice, lengths of zero and below."""
    heads, gqa, d, page = 2, 2, 64, 16
    cache = random_cache(3, 9, heads, d, page, 32)
    lists = ints(np.random.default_rng(2).integers(0, 9, (5, heads, 6)))
    lists[2, :, 1:] = -1
    held = ints([96, 50, 16, 0, -1])
    q = queries(4, 5, heads * gqa, d)
    out = torch.full_like(q, 7.0)
    wq().kv4_attention_pages(q, cache, lists, held, scale=0.3, out=out)
    o, e = attention_over(q, cache, lists.cpu().numpy(), held.tolist(), 0.3)
    ref.check(out[:4], o[:4], e[:4])
    assert (out[3] == 0).all() and (out[4] == 7).all()
    assert wq().get_device_error() == 0


def test_what_is_out_of_bounds_is_recorded():
    heads, d, page, lens = 2, 64, 16, [300, 400, 200]
    table, pages = ref.random_batch(6, lens, page)
    cache = random_cache(5, pages, heads, d, page, 32)
    bounds = random_bounds(6, cache)
    q = queries(5, 3, 4, d)
    good = wq().kv4_sparse_attention(q, cache, bounds, ints(lens), ints(table), max_pages=5)
    for change in ("page", "last page", "length", "rows"):
        t, n, starts = table.copy(), list(lens), None
        if change == "page":
            t[1, 3] = pages
        elif change == "last page":
            t[1, 24] = -5
        elif change == "length":
            n[1] = page * table.shape[1] + 1
        else:
            starts = ints([0, 1, 2, 4])
        mine = wq().KV4Bounds(bounds.codes.clone(), bounds.grid.clone())
        out, lists, held = wq().kv4_sparse_attention(q, cache, mine, ints(n), ints(t), starts,
                                                     max_pages=5)
        assert wq().get_device_error() == 1, change
        assert torch.equal(out[0], good[0][0]) and torch.equal(lists[0], good[1][0]), change
    # lists with a page outside the cache, a length above the list
    for lists, held in (([[[0, pages]] * 2], [20]), ([[[0, 1]] * 2], [33])):
        wq().kv4_attention_pages(q[:1], cache, ints(lists), ints(held))
        assert wq().get_device_error() == 1
    # a sequence without rows is checked too
    wq().kv4_select(q[:2], cache, bounds, ints([300, 10_000, 200]), ints(table), ints([0, 1, 1, 2]),
                    max_pages=5)
    assert wq().get_device_error() == 1
    wq().kv4_update_bounds(cache, bounds, ints([300, 10_000, 200]), ints(table), ints([0, 1, 1, 2]),
                           rows=2)
    assert wq().get_device_error() == 1


def test_two_streams_with_a_workspace_each():
    heads, gqa, d, page, lens = 2, 4, 128, 64, [20_000, 9000]
    table, pages = ref.random_batch(8, lens, page)
    cache = random_cache(9, pages, heads, d, page, 64)
    bounds = random_bounds(6, cache)
    q = [queries(i, 2, heads * gqa, d) for i in range(2)]
    args = (ints(lens), ints(table))
    want = [wq().kv4_sparse_attention(x, cache, bounds, *args, max_pages=40)[0] for x in q]
    streams, ws = [torch.cuda.Stream() for _ in q], [wq().kv4_workspace() for _ in q]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                lists, held = wq().kv4_select(q[i], cache, bounds, *args, max_pages=40)
                got[i].append(wq().kv4_attention_pages(q[i], cache, lists, held, workspace=ws[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, want[i]) for x in got[i])


def test_refusals_of_the_binding():
    heads, d, page, lens = 2, 64, 16, [40, 50]
    table, pages = ref.random_batch(6, lens, page)
    cache = random_cache(5, pages, heads, d, page, 32)
    bounds = random_bounds(6, cache)
    q, args = queries(5, 2, 4, d), (ints(lens), ints(table))
    lists, held = wq().kv4_select(q, cache, bounds, *args, max_pages=3)
    other = wq().kv4_bounds(wq().kv4_cache(pages + 1, heads, d, page_size=page, group=32))
    for call in (lambda: wq().KV4Bounds(bounds.codes.float(), bounds.grid),
                 lambda: wq().KV4Bounds(bounds.codes, bounds.grid[:1]),
                 lambda: wq().kv4_update_bounds(cache, other, *args),
                 lambda: wq().kv4_update_bounds(cache, bounds, *args, row_starts=ints([0, 1, 2])),
                 lambda: wq().kv4_select(q, cache, bounds, *args),
                 lambda: wq().kv4_select(q[:, :3], cache, bounds, *args, max_pages=3),
                 lambda: wq().kv4_select(q, cache, bounds, *args, max_pages=3, lists=lists[:1]),
                 lambda: wq().kv4_select(q, cache, bounds, *args, max_pages=4, lists=lists),
                 lambda: wq().kv4_select(q, cache, bounds, *args, max_pages=3, lens=held.long()),
                 lambda: wq().kv4_attention_pages(q, cache, lists.cpu(), held),
                 lambda: wq().kv4_attention_pages(q, cache, lists, held, out=q[:1]),
                 lambda: wq().kv4_attention_pages(q, cache, lists, held,
                                                  workspace=torch.zeros(4, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            call()
    for kw in (dict(max_pages=2), dict(max_pages=3, last=0), dict(max_pages=3, first=-1)):
        with pytest.raises(wq().WQError):
            wq().kv4_select(q, cache, bounds, *args, **kw)
