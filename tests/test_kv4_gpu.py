"""The 4-bit key/value cache on the B200: rows written bit-exact against the
CPU oracle's quantizer, rows read back bit-exact, and attention over the cache
against binary64 within the bound that its roundings allow."""
import numpy as np
import pytest
import torch

from tests import kv4_ref as ref
from tests.gpu_util import host_bits, wq

pytestmark = pytest.mark.gpu

FORMATS = [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128)]
SENTINEL = 0xA5
COUNTERS = 160 * 16 * 4        # bytes of the attention workspace's counters


def new_cache(pages, heads, d, page, group):
    c = wq().kv4_cache(pages, heads, d, page_size=page, group=group)
    for t in (c.k_codes, c.v_codes):
        t.fill_(SENTINEL)
    for t in (c.k_meta, c.v_meta):
        t.fill_(float("nan"))
    return c


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


def starts_of(rows):
    return np.concatenate(([0], np.cumsum(rows))).astype(np.int32)


def expect_written(cache, x, held, kind, codes, meta):
    """Apply the rows to the images codes / meta (numpy), by the oracle."""
    heads, d = cache.kv_heads, cache.head_dim
    u, s, z = ref.quantize(x.reshape(-1, d), cache.group)
    packed = ref.pack(u, kind).reshape(-1, heads, d // 2)
    sz = np.stack((s, z), -1).reshape(-1, heads, d // cache.group, 2)
    for row, _, _, page, slot in held:
        codes[page, :, slot] = packed[row]
        meta[page, :, slot] = sz[row]


def images(cache):
    return {"k": (host_bits(cache.k_codes).copy(), host_bits(cache.k_meta).copy()),
            "v": (host_bits(cache.v_codes).copy(), host_bits(cache.v_meta).copy())}


def assert_cache(cache, want):
    got = images(cache)
    for kind in "kv":
        assert np.array_equal(got[kind][0], want[kind][0]), f"{kind} codes"
        assert np.array_equal(got[kind][1], want[kind][1]), f"{kind} metadata"


def fill(cache, lens, table, seed=1, strong=8.0):
    """Write every token of every sequence; returns nothing."""
    n = sum(lens)
    k = ref.keys(seed, n, cache.kv_heads, cache.head_dim, strong).cuda()
    v = ref.keys(seed + 1, n, cache.kv_heads, cache.head_dim, 1.0).cuda()
    wq().kv4_write(k, v, cache, ints(lens), ints(table), ints(starts_of(lens)))


def reference(q, cache, lens, rows, table, scale):
    """(output, bound) of all rows in binary64, from the cache's own bits."""
    kc, vc = cache.k_codes.cpu().numpy(), cache.v_codes.cpu().numpy()
    km, vm = cache.k_meta.cpu().numpy(), cache.v_meta.cpu().numpy()
    out, bound, at = [], [], 0
    for b, (n, t) in enumerate(zip(lens, rows)):
        k = ref.sequence_values(kc, km, table[b], n, cache.page_size, "k")
        v = ref.sequence_values(vc, vm, table[b], n, cache.page_size, "v")
        x = q[at:at + t].float().cpu().numpy().astype(np.float64)
        # more than 16 rows times heads of a group: either kernel may be chosen
        o, e = ref.attention(x, k, v, n, scale, True)
        if t * (x.shape[1] // cache.kv_heads) > 16:
            e = np.maximum(e, ref.attention(x, k, v, n, scale, False)[1])
        out.append(o)
        bound.append(e)
        at += t
    return np.concatenate(out), np.concatenate(bound)


# ------------------------------------------------------------------ write, read

@pytest.mark.parametrize("d,group", FORMATS)
@pytest.mark.parametrize("heads,page,lens,rows", [
    (1, 16, [1], [1]),
    (8, 64, [777], [1]),
    (3, 32, [5, 40, 33], [5, 7, 33]),
    (5, 16, [100, 0, 17, 3], [50, 0, 17, 6]),        # no rows; more rows than tokens
    (2, 128, [300] * 40, [2] * 40),                  # more than 33 sequences
])
def test_write_bit_exact_and_read_back(d, group, heads, page, lens, rows):
    table, pages = ref.random_batch(d + group, lens, page)
    cache = new_cache(pages, heads, d, page, group)
    n, behind = sum(rows), 3
    # keys and values as slices of a wider projection, and rows that belong to no sequence
    qkv = torch.cat((ref.keys(2, n + behind, 2, d), ref.keys(3, n + behind, 2 * heads, d)), 1).cuda()
    qkv[n:] = float("nan")
    k, v = qkv[:, 2:2 + heads], qkv[:, 2 + heads:]
    want = images(cache)
    held, empty = ref.places(lens, rows, table, page)
    for kind, x in (("k", k), ("v", v)):
        expect_written(cache, x[:n], held, kind, *want[kind])
    batch = (ints(lens), ints(table), ints(starts_of(rows)))
    wq().kv4_write(k, v, cache, *batch)
    assert_cache(cache, want)

    out = [torch.full((n + behind, heads, d), 7.0, dtype=torch.bfloat16, device="cuda")
           for _ in "kv"]
    wq().kv4_read(cache, *batch, out=out)
    for kind, got in zip("kv", out):
        expected = np.full((n + behind, heads, d), 7.0, dtype=np.float32)
        expected[empty] = 0
        u = ref.unpack(want[kind][0], kind).astype(np.float32)
        m = want[kind][1].view(np.float16).astype(np.float32)
        for row, _, _, p, slot in held:
            val = (u[p, :, slot].reshape(heads, -1, group) - m[p, :, slot, :, 1:]) * \
                m[p, :, slot, :, :1]
            expected[row] = val.reshape(heads, d)
        assert torch.equal(got.cpu(), torch.tensor(expected).to(torch.bfloat16)), kind
    assert wq().get_device_error() == 0


@pytest.mark.parametrize("d,group", FORMATS)
def test_write_edge_values(d, group):
    """Zeros, constants, saturation, values below binary16, ties, signed zeros."""
    n, heads = 12, 2
    x = ref.keys(4, n, heads, d)
    x[0] = 0
    x[1] = 0.25
    x[2] = -3.0
    x[3, :, ::2], x[3, :, 1::2] = 3e38, -3e38
    x[4] = torch.arange(d) * 2.0 ** -25
    x[5] = x[5].abs()
    x[6] = -x[6].abs()
    x[7, :, ::3] = -0.0
    x[8, :, 5] = 65280.0
    x[9] = 2.0 ** -133
    x[10, :, :32] = 0
    x[11] = (torch.arange(d) % 31 - 15) * 0.5
    table, pages = ref.random_batch(1, [n], 16)
    cache = new_cache(pages, heads, d, 16, group)
    want = images(cache)
    held, _ = ref.places([n], [n], table, 16)
    expect_written(cache, x, held, "k", *want["k"])
    expect_written(cache, -x, held, "v", *want["v"])
    wq().kv4_write(x.cuda(), -x.cuda(), cache, ints([n]), ints(table))
    assert_cache(cache, want)


@pytest.mark.parametrize("d,group", FORMATS)
@pytest.mark.parametrize("kind", ["spread", "steps", "large", "nan"])
def test_write_ranges(d, group, kind):
    """Rows of every magnitude, with elements far below their row's largest;
    rows of a few distinct values, full of ties; values that saturate; a NaN,
    which counts as zero for the others and has any code."""
    n, heads = 96, 2
    g = torch.Generator().manual_seed(d + group)
    x = ref.keys(4, n, heads, d).float()
    if kind == "spread":
        x *= torch.exp2(-torch.randint(0, 18, (n, heads, d), generator=g).float())
        x *= torch.exp2(8 - torch.arange(n) / 4).view(n, 1, 1)
    elif kind == "steps":
        x = torch.randint(-15, 16, (n, heads, d), generator=g).float()
        x *= torch.exp2(-(torch.arange(n) // 4).float()).view(n, 1, 1)
    elif kind == "large":
        x *= torch.exp2(torch.randint(-4, 18, (n, heads, d), generator=g).float())
    x = x.to(torch.bfloat16)
    nan = torch.zeros(x.shape, dtype=torch.bool)
    if kind == "nan":
        nan = torch.rand(x.shape, generator=g) < 0.02
    table, pages = ref.random_batch(1, [n], 16)
    cache = new_cache(pages, heads, d, 16, group)
    want = images(cache)
    held, _ = ref.places([n], [n], table, 16)
    expect_written(cache, x.masked_fill(nan, 0), held, "k", *want["k"])
    expect_written(cache, -x.masked_fill(nan, 0), held, "v", *want["v"])
    x = x.masked_fill(nan, float("nan"))
    wq().kv4_write(x.cuda(), -x.cuda(), cache, ints([n]), ints(table))
    got = images(cache)
    for kind in "kv":
        assert np.array_equal(got[kind][1], want[kind][1])
        u, w = (ref.unpack(i[kind][0], kind) for i in (got, want))
        for row, _, _, page, slot in held:
            same = (u[page, :, slot] == w[page, :, slot]) | nan[row].numpy()
            assert same.all(), (kind, row)


def test_write_matches_the_weight_quantizer():
    """The cache's codes are those of wq_quantize for the same values."""
    n, heads, d, group = 64, 4, 128, 32
    x = ref.keys(6, n, heads, d).cuda()
    cache = new_cache(4, heads, d, 16, group)
    table = np.arange(4, dtype=np.int32)[None]
    wq().kv4_write(x, x, cache, ints([n]), ints(table))
    qw = wq().quantize(ref.to_half(x).reshape(n * heads, d), bits=4, group=group)
    codes = host_bits(qw.codes)
    u = np.stack((codes & 15, codes >> 4), -1).reshape(n, heads, d)
    got = ref.unpack(host_bits(cache.k_codes), "k").transpose(0, 2, 1, 3).reshape(n, heads, d)
    assert np.array_equal(got, u)
    meta = host_bits(cache.k_meta).transpose(0, 2, 1, 3, 4).reshape(n * heads, -1, 2)
    assert np.array_equal(meta[..., 0], host_bits(qw.scales))
    assert np.array_equal(meta[..., 1], host_bits(qw.zeros))


def test_append_token_by_token_equals_one_write():
    d, group, heads, page, n = 64, 32, 2, 16, 37
    table, pages = ref.random_batch(3, [n, n], page)
    k, v = (ref.keys(s, 2 * n, heads, d).cuda().view(2, n, heads, d) for s in (1, 2))
    a, b = new_cache(pages, heads, d, page, group), new_cache(pages, heads, d, page, group)
    wq().kv4_write(k.reshape(2 * n, heads, d), v.reshape(2 * n, heads, d), a, ints([n, n]),
                   ints(table))
    for i in range(n):
        wq().kv4_write(k[:, i], v[:, i], b, ints([i + 1, i + 1]), ints(table))
    assert_cache(b, images(a))


# ------------------------------------------------------------------- attention

def run_attention(d, group, page, heads, gqa, lens, rows, seed=0, strong=8.0, scale=None, q=None):
    table, pages = ref.random_batch(seed + 10, lens, page)
    cache = new_cache(pages, heads, d, page, group)
    fill(cache, lens, table, seed=seed + 1, strong=strong)
    n = sum(rows)
    if q is None:
        q = ref.keys(seed + 5, n, heads * gqa, d, 1.0)
    q = q.cuda()
    uniform = len(set(rows)) == 1
    out = torch.full_like(q, 3.0)
    ws = wq().kv4_workspace()
    got = wq().kv4_attention(q, cache, ints(lens), ints(table),
                             None if uniform else ints(starts_of(rows)),
                             max_rows=None if uniform else max(rows), scale=scale, out=out,
                             workspace=ws)
    torch.cuda.synchronize()
    assert wq().get_device_error() == 0
    assert not ws[:COUNTERS].any(), "the workspace's counters are not zero again"
    s = d ** -0.5 if scale is None else scale
    o, bound = reference(q, cache, lens, rows, table, s)
    ref.check(got, o, bound)
    return got, cache, table, q


@pytest.mark.parametrize("d,group", FORMATS)
@pytest.mark.parametrize("lens", [[1], [2, 31], [32, 33, 16, 15, 17], [100, 0, 64, 257]])
@pytest.mark.parametrize("gqa", [1, 4])
def test_single_tokens(d, group, lens, gqa):
    run_attention(d, group, 16, 2, gqa, lens, [1] * len(lens), seed=d + group + len(lens))


@pytest.mark.parametrize("d,group", FORMATS)
@pytest.mark.parametrize("gqa", [3, 7, 8, 12, 16])
def test_head_layouts(d, group, gqa):
    run_attention(d, group, 64, 3, gqa, [70, 129, 5], [1, 1, 1], seed=gqa)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_page_sizes(page):
    run_attention(128, 64, page, 2, 4, [page, page + 1, page - 1, 3 * page + 7], [1] * 4, seed=page)


@pytest.mark.parametrize("d,group", FORMATS)
@pytest.mark.parametrize("rows,lens", [
    ([2, 2, 2], [2, 100, 35]), ([4], [4]), ([3, 1, 5], [50, 1, 64]),
    ([6, 0, 2], [3, 20, 2]),              # rows without a token, a sequence without rows
    ([20, 7], [20, 90]), ([70], [131])])
def test_several_rows(d, group, rows, lens):
    run_attention(d, group, 32, 2, 2, lens, rows, seed=sum(rows))


@pytest.mark.parametrize("d,group", FORMATS)
@pytest.mark.parametrize("gqa,rows,lens", [
    (1, [17], [17]), (4, [5], [300]), (4, [33], [40]), (1, [128], [128]), (1, [129], [131]),
    (2, [128], [1000]), (4, [100, 1, 64], [100, 1, 260]), (7, [40, 0, 3, 90], [700, 5, 3, 20]),
    (16, [2, 2], [130, 128])])
def test_many_rows(d, group, gqa, rows, lens):
    run_attention(d, group, 16, 2, gqa, lens, rows, seed=sum(rows) + gqa)


@pytest.mark.parametrize("d,group,heads,gqa,lens,rows", [
    (128, 64, 1, 4, [5000], [40]),                 # one block over many CTAs
    (64, 32, 2, 8, [1200, 129, 70], [20, 30, 70]), # blocks with one step, two and more
    (128, 128, 1, 1, [3000], [300]),               # the last rows see most
    (128, 32, 1, 32, [2000], [1])])
def test_many_rows_split_over_ctas(d, group, heads, gqa, lens, rows):
    run_attention(d, group, 64, heads, gqa, lens, rows, seed=len(lens) + gqa)


def test_many_rows_repeated_and_captured_calls():
    """The last split to arrive adds the parts: same bits every time, in a
    graph and over other lengths too."""
    lens, rows = [2600], [50]
    got, cache, table, q = run_attention(128, 64, 64, 1, 4, lens, rows, seed=21)
    ws, n, tb = wq().kv4_workspace(), ints(lens), ints(table)
    out = torch.zeros_like(q)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        for _ in range(3):
            wq().kv4_attention(q, cache, n, tb, out=out, workspace=ws)
        stream.synchronize()
        assert torch.equal(out, got)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            wq().kv4_attention(q, cache, n, tb, out=out, workspace=ws)
    for length in (2600, 2600, 700, 30, 2600):
        n.copy_(ints([length]))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        o, e = reference(q, cache, [length], rows, table, 128 ** -0.5)
        ref.check(out, o, e)
    assert torch.equal(out, got) and not ws[:COUNTERS].any()


def test_many_rows_bad_device_arrays():
    d, group, heads, page = 64, 32, 2, 16
    lens, rows = [300, 200], [40, 30]
    table, pages = ref.random_batch(3, lens, page)
    cache = new_cache(pages, heads, d, page, group)
    fill(cache, lens, table)
    before = images(cache)
    q = ref.keys(1, 70, heads, d).cuda()
    args = (q, cache, ints(lens), ints(table), ints(starts_of(rows)))
    good = wq().kv4_attention(*args, max_rows=40)
    assert wq().get_device_error() == 0
    bad = table.copy()
    bad[1, 0], bad[1, 5] = pages, -1
    out = wq().kv4_attention(q, cache, ints(lens), ints(bad), ints(starts_of(rows)), max_rows=40)
    assert wq().get_device_error() == 1
    assert torch.equal(out[:40], good[:40])
    wq().kv4_attention(q, cache, ints([300, 10 ** 6]), ints(table), ints(starts_of(rows)))
    assert wq().get_device_error() == 1
    wq().kv4_attention(q, cache, ints(lens), ints(table), ints([0, 40, 90]))
    assert wq().get_device_error() == 1
    assert torch.equal(wq().kv4_attention(*args, max_rows=40), good)
    assert wq().get_device_error() == 0
    assert_cache(cache, before)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_many_rows_page_sizes(page):
    run_attention(128, 64, page, 1, 4, [page + 200, 600], [60, 100], seed=page)


@pytest.mark.parametrize("kind", ["large", "tiny", "zero", "mixed", "negative", "no scale"])
def test_many_rows_query_ranges(kind):
    q = ref.keys(3, 40, 8, 128, 1.0).float()
    if kind == "large":
        q *= 40
    elif kind == "tiny":
        q *= 2.0 ** -120
    elif kind == "zero":
        q *= 0
    elif kind == "mixed":
        q *= torch.exp2(torch.arange(128) % 20 - 12.0)
    run_attention(128, 32, 32, 2, 4, [350], [40], seed=4, q=q.to(torch.bfloat16),
                  scale={"negative": -0.3, "no scale": 0.0}.get(kind))


@pytest.mark.parametrize("what,strength", [("v", 2.0 ** -13), ("v", 2.0 ** -20), ("v", 2.0 ** 10),
                                           ("v", 60000.0), ("k", 60000.0), ("both", 60000.0)])
def test_many_rows_value_ranges(what, strength):
    """Scales that differ from token to token, and values at the end of
    binary16's range, whose codes can stand for more than its largest."""
    d, group, heads, n, page, t = 128, 32, 2, 400, 32, 30
    table, pages = ref.random_batch(5, [n], page)
    cache = new_cache(pages, heads, d, page, group)
    spread = torch.exp2(torch.randint(-8, 1, (n, 1, 1),
                                      generator=torch.Generator().manual_seed(3)).float())
    k, v = ref.keys(1, n, heads, d), ref.keys(2, n, heads, d, 1.0)
    if what != "k":
        v = v.float().clamp(-1, 1) * spread * strength
    if what != "v":
        k = k.float().clamp(-1, 1) * spread * strength
    wq().kv4_write(k.to(torch.bfloat16).cuda(), v.to(torch.bfloat16).cuda(), cache, ints([n]),
                   ints(table))
    q = ref.keys(9, t, 8, d, 1.0).float()
    q = (q / strength if what != "v" else q).to(torch.bfloat16).cuda()
    got = wq().kv4_attention(q, cache, ints([n]), ints(table))
    o, bound = reference(q, cache, [n], [t], table, d ** -0.5)
    ref.check(got, o, bound)


@pytest.mark.parametrize("d,group,heads,gqa,lens", [
    (128, 64, 1, 4, [9000]),                       # one head over every CTA
    (128, 32, 2, 8, [5000, 3, 2500]),
    (64, 64, 2, 16, [7000]),
    (64, 32, 8, 1, [1500] * 3 + [1] * 5),
    (128, 128, 4, 4, [37] * 150),                  # more sequences than CTAs
])
def test_split_over_ctas(d, group, heads, gqa, lens):
    run_attention(d, group, 64, heads, gqa, lens, [1] * len(lens), seed=len(lens))


@pytest.mark.parametrize("rows", [1, 17, 40])
def test_tokens_that_are_not_copied(rows):
    """Several blocks of rows over a few tokens, after a call that left NaN
    metadata in every SM's shared memory."""
    d, group, heads, page, n = 128, 32, 2, 16, max(rows, 17)
    noise = new_cache(4, heads, d, page, group)
    ones = ints([64] * 200)
    q = ref.keys(1, 200, heads, d).cuda()
    wq().kv4_attention(q, noise, ones, ints(np.tile(np.arange(4), (200, 1))))
    assert wq().get_device_error() == 0
    run_attention(d, group, page, heads, 1, [n], [rows], seed=rows)


def test_more_sequences_than_threads():
    lens = [1 + (7 * i) % 40 for i in range(700)]
    rows = [i % 3 for i in range(700)]
    run_attention(64, 64, 16, 1, 2, lens, rows, seed=2)


@pytest.mark.parametrize("kind", ["large", "tiny", "zero", "mixed", "scale"])
def test_query_ranges(kind):
    q = ref.keys(3, 2, 8, 128, 1.0).float()
    if kind == "large":
        q *= 40
    elif kind == "tiny":
        q *= 2.0 ** -120
    elif kind == "zero":
        q *= 0
    elif kind == "mixed":
        q *= torch.exp2(torch.arange(128) % 20 - 12.0)
    run_attention(128, 32, 32, 2, 4, [150, 33], [1, 1], seed=4, q=q.to(torch.bfloat16),
                  scale=-0.3 if kind == "scale" else None)


@pytest.mark.parametrize("strength", [2.0 ** -13, 1.0, 2.0 ** 10])
def test_value_ranges(strength):
    """Values whose scales differ by powers of two from token to token."""
    d, group, heads, n, page = 128, 32, 2, 200, 32
    table, pages = ref.random_batch(5, [n], page)
    cache = new_cache(pages, heads, d, page, group)
    k = ref.keys(1, n, heads, d)
    v = ref.keys(2, n, heads, d, 1.0).float() * strength
    v *= torch.exp2(torch.randint(-4, 5, (n, 1, 1), generator=torch.Generator().manual_seed(3)).float())
    v[17] = 0
    wq().kv4_write(k.cuda(), v.to(torch.bfloat16).cuda(), cache, ints([n]), ints(table))
    q = ref.keys(9, 1, 8, d, 1.0).cuda()
    got = wq().kv4_attention(q, cache, ints([n]), ints(table))
    o, bound = reference(q, cache, [n], [1], table, d ** -0.5)
    ref.check(got, o, bound)


@pytest.mark.parametrize("what,strength", [("v", 60000.0), ("k", 60000.0), ("both", 60000.0),
                                           ("v", 2.0 ** -20)])
@pytest.mark.parametrize("rows", [1, 3])
def test_values_at_the_ends_of_binary16(what, strength, rows):
    """Few rows over codes that can stand for more than binary16's largest
    value, and over scales close to its smallest."""
    d, group, heads, n, page = 128, 32, 2, 330, 32
    table, pages = ref.random_batch(5, [n], page)
    cache = new_cache(pages, heads, d, page, group)
    spread = torch.exp2(torch.randint(-8, 1, (n, 1, 1),
                                      generator=torch.Generator().manual_seed(7)).float())
    k, v = ref.keys(1, n, heads, d), ref.keys(2, n, heads, d, 1.0)
    if what != "k":
        v = v.float().clamp(-1, 1) * spread * strength
    if what != "v":
        k = k.float().clamp(-1, 1) * spread * strength
    wq().kv4_write(k.to(torch.bfloat16).cuda(), v.to(torch.bfloat16).cuda(), cache, ints([n]),
                   ints(table))
    q = ref.keys(9, rows, 8, d, 1.0).float()
    q = (q / strength if what != "v" else q).to(torch.bfloat16).cuda()
    got = wq().kv4_attention(q, cache, ints([n]), ints(table))
    o, bound = reference(q, cache, [n], [rows], table, d ** -0.5)
    ref.check(got, o, bound)


@pytest.mark.parametrize("d,group", FORMATS)
def test_nan_and_infinite_rows_are_cached_as_finite_values(d, group):
    """A NaN spoils its own row's codes at most: the metadata stays finite, so
    rows that do not see the token and tokens beside it keep their values."""
    heads, page, n = 2, 16, 40
    table, pages = ref.random_batch(2, [n], page)
    x = ref.keys(4, n, heads, d)
    clean, cache = new_cache(pages, heads, d, page, group), new_cache(pages, heads, d, page, group)
    wq().kv4_write(x.cuda(), x.cuda(), clean, ints([n]), ints(table))
    bad = x.clone()
    bad[-1, 0, 3], bad[-2, 1] = float("nan"), float("nan")
    bad[-3, 0, 7], bad[-4, 1, 9] = float("inf"), float("-inf")
    wq().kv4_write(bad.cuda(), bad.cuda(), cache, ints([n]), ints(table))
    for got, want in zip(wq().kv4_read(cache, ints([n]), ints(table), rows=n),
                         wq().kv4_read(clean, ints([n]), ints(table), rows=n)):
        assert torch.isfinite(got).all()
        assert torch.equal(got[:-4], want[:-4])
    for rows in (8, 40):          # each kernel
        q = ref.keys(6, rows, 8, d, 1.0).cuda()
        got = wq().kv4_attention(q, cache, ints([n]), ints(table))
        assert torch.isfinite(got).all()
        # The exact values of rows before the four are those of the clean cache.
        # Their bits need not be: rows that share a warp or a tile with one that
        # sees a large scale form their weights again from another reference, and
        # each way is within the bound.
        o, bound = reference(q, clean, [n], [rows], table, d ** -0.5)
        ref.check(got[:-4], o[:-4], bound[:-4])
    assert wq().get_device_error() == 0


def test_a_nan_query_among_many_rows_stays_in_its_row():
    d, heads, gqa = 128, 2, 4
    _, cache, table, q = run_attention(d, 64, 16, heads, gqa, [400], [70], seed=8)
    o, bound = reference(q, cache, [400], [70], table, d ** -0.5)
    for value in (float("nan"), float("inf")):
        bad = q.clone()
        bad[33, 5, 17] = value
        again = wq().kv4_attention(bad, cache, ints([400]), ints(table))
        keep = torch.ones(70, heads * gqa, dtype=torch.bool)
        keep[33, 5] = False
        ref.check(again[keep.cuda()], o[keep.numpy()], bound[keep.numpy()])
        assert not torch.isfinite(again[33, 5]).any()


def test_a_nan_query_stays_in_its_row():
    d, heads, gqa = 128, 2, 4
    got, cache, table, q = run_attention(d, 64, 16, heads, gqa, [90, 40], [2, 2], seed=8)
    bad = q.clone()
    bad[1, 3] = float("nan")
    again = wq().kv4_attention(bad, cache, ints([90, 40]), ints(table))
    assert torch.isnan(again[1, 3]).all()
    keep = torch.ones(4, heads * gqa, dtype=torch.bool)
    keep[1, 3] = False
    assert torch.equal(again[keep.cuda()], got[keep.cuda()])


def test_strided_rows_and_rows_behind_the_last_sequence():
    d, group, heads, gqa, lens, rows = 64, 32, 2, 3, [40, 21], [2, 3]
    got, cache, table, q = run_attention(d, group, 16, heads, gqa, lens, rows, seed=6)
    wide = torch.randn(9, heads * gqa + 4, d, device="cuda").to(torch.bfloat16)
    wide[:5, :heads * gqa] = q
    wide[5:] = float("nan")
    out = torch.full((9, heads * gqa + 1, d), 5.0, dtype=torch.bfloat16, device="cuda")
    wq().kv4_attention(wide[:, :heads * gqa], cache, ints(lens), ints(table),
                       ints(starts_of(rows)), out=out[:, :heads * gqa])
    assert torch.equal(out[:5, :heads * gqa], got)
    assert (out[5:] == 5).all() and (out[:, heads * gqa:] == 5).all()
    fresh = wq().kv4_attention(wide[:, :heads * gqa], cache, ints(lens), ints(table),
                               ints(starts_of(rows)))
    assert torch.equal(fresh[:5], got) and not fresh[5:].any()


def test_the_bound_on_rows_does_not_change_results():
    got, cache, table, q = run_attention(128, 64, 32, 2, 4, [300, 70], [1, 3], seed=7)
    for bound in (None, 1, 3, 4, 50):
        again = wq().kv4_attention(q, cache, ints([300, 70]), ints(table), ints([0, 1, 4]),
                                   max_rows=bound)
        o, e = reference(q, cache, [300, 70], [1, 3], table, 128 ** -0.5)
        ref.check(again, o, e)


def test_repeated_and_captured_calls_give_the_same_bits():
    lens = [3000, 40, 1]
    got, cache, table, q = run_attention(128, 64, 64, 2, 4, lens, [1, 1, 1], seed=3)
    ws, n, tb = wq().kv4_workspace(), ints(lens), ints(table)
    for _ in range(3):
        assert torch.equal(wq().kv4_attention(q, cache, n, tb, workspace=ws), got)
    out = torch.zeros_like(q)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        wq().kv4_attention(q, cache, n, tb, out=out, workspace=ws)
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            wq().kv4_attention(q, cache, n, tb, out=out, workspace=ws)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, got)
    # the same graph over other lengths
    n.copy_(ints([1500, 39, 1]))
    graph.replay()
    torch.cuda.synchronize()
    o, e = reference(q, cache, [1500, 39, 1], [1, 1, 1], table, 128 ** -0.5)
    ref.check(out, o, e)
    assert not ws[:COUNTERS].any()


def test_two_streams_with_a_workspace_each():
    lens = [6000]
    got, cache, table, q = run_attention(128, 64, 64, 2, 4, lens, [1], seed=11)
    n, tb = ints(lens), ints(table)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for s in streams:
        with torch.cuda.stream(s):
            ws = wq().kv4_workspace()
            outs.append([wq().kv4_attention(q, cache, n, tb, workspace=ws) for _ in range(20)])
    torch.cuda.synchronize()
    assert all(torch.equal(o, got) for out in outs for o in out)


def test_two_streams_with_many_rows_and_few():
    """Both attention kernels at once, each stream with its own workspace."""
    many = run_attention(64, 32, 32, 2, 4, [900], [60], seed=12)
    few = run_attention(128, 64, 64, 2, 4, [3000], [1], seed=13)
    torch.cuda.synchronize()
    outs = []
    for (got, cache, table, q), lens in ((many, [900]), (few, [3000])):
        with torch.cuda.stream(torch.cuda.Stream()):
            ws, n, tb = wq().kv4_workspace(), ints(lens), ints(table)
            outs.append((got, [wq().kv4_attention(q, cache, n, tb, workspace=ws)
                               for _ in range(20)]))
    torch.cuda.synchronize()
    assert all(torch.equal(o, got) for got, each in outs for o in each)


def test_page_table_that_is_part_of_a_wider_one():
    lens, rows = [70, 33, 90], [2, 1, 3]
    got, cache, table, q = run_attention(64, 64, 16, 2, 2, lens, rows, seed=14)
    wide = torch.full((3, table.shape[1] + 5), -1, dtype=torch.int32, device="cuda")
    wide[:, 2:2 + table.shape[1]] = ints(table)
    part = wide[:, 2:2 + table.shape[1]]
    starts = ints(starts_of(rows))
    assert torch.equal(wq().kv4_attention(q, cache, ints(lens), part, starts, max_rows=3), got)
    a = wq().kv4_read(cache, ints(lens), part, ints(starts_of(lens)), rows=sum(lens))
    b = wq().kv4_read(cache, ints(lens), ints(table), ints(starts_of(lens)), rows=sum(lens))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert wq().get_device_error() == 0


def test_five_thousand_sequences():
    lens = [1 + (11 * i) % 50 for i in range(5000)]
    got, cache, table, q = run_attention(64, 32, 16, 1, 1, lens, [1] * 5000, seed=15)


@pytest.mark.parametrize("gqa", [33, 70, 300])
def test_very_wide_groups(gqa):
    run_attention(128, 64, 16, 1, gqa, [40, 200], [1, 2], seed=gqa)


def test_bad_device_arrays_are_recorded_and_stay_in_bounds():
    d, group, heads, page = 64, 32, 2, 16
    lens = [40, 40]
    table, pages = ref.random_batch(3, lens, page)
    cache = new_cache(pages, heads, d, page, group)
    fill(cache, lens, table)
    before = images(cache)
    q = ref.keys(1, 2, heads, d).cuda()
    good = wq().kv4_attention(q, cache, ints(lens), ints(table))
    assert wq().get_device_error() == 0
    bad = table.copy()
    bad[1, 0], bad[1, 2] = pages, -1
    out = wq().kv4_attention(q, cache, ints(lens), ints(bad))
    assert wq().get_device_error() == 1
    assert torch.equal(out[0], good[0])             # the other sequence is right
    wq().kv4_attention(q, cache, ints([40, 10 ** 6]), ints(table))
    assert wq().get_device_error() == 1
    k = ref.keys(2, 2, heads, d).cuda()
    wq().kv4_write(k, k, cache, ints([0, 40]), ints(bad))
    assert wq().get_device_error() == 1
    wq().kv4_read(cache, ints([-5, 40]), ints(bad), rows=2)
    assert wq().get_device_error() == 1
    wq().kv4_attention(q, cache, ints(lens), ints(table), ints([0, 1, 3]))
    assert wq().get_device_error() == 1
    assert_cache(cache, before)


def test_offsets_past_32_bits():
    """A pool whose buffers are longer than 4 GB, used at its far end."""
    d, group, heads, page = 128, 128, 8, 256
    pages = (1 << 32) // (heads * page * d // 2) + 40
    cache = wq().kv4_cache(pages, heads, d, page_size=page, group=group)
    lens = [700]
    table = np.array([[pages - 1, pages - 30, pages - 7]], dtype=np.int32)
    small = new_cache(3, heads, d, page, group)
    few = np.array([[0, 1, 2]], dtype=np.int32)
    fill(cache, lens, table)
    fill(small, lens, few)
    for a, b in zip((cache.k_codes, cache.v_codes), (small.k_codes, small.v_codes)):
        at = torch.tensor(table[0].astype(np.int64)).cuda()
        assert torch.equal(a[at][:2], b[:2]) and torch.equal(a[at][2, :, :188], b[2, :, :188])
    q = ref.keys(1, 1, 32, d, 1.0).cuda()
    assert torch.equal(wq().kv4_attention(q, cache, ints(lens), ints(table)),
                       wq().kv4_attention(q, small, ints(lens), ints(few)))
    for a, b in zip(wq().kv4_read(cache, ints(lens), ints(table), rows=700),
                    wq().kv4_read(small, ints(lens), ints(few), rows=700)):
        assert torch.equal(a, b)


def test_refusals():
    mod = wq()
    cache = new_cache(4, 2, 64, 16, 32)
    n, tb = ints([4, 4]), ints([[0, 1], [2, 3]])
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device="cuda")
    for bad in (x.float(), x[:, :1], x[..., :32], x.cpu(), x.transpose(0, 1)[:, :, :]):
        if bad.shape == x.shape and bad.dtype == x.dtype and bad.is_cuda:
            bad = torch.zeros(2, 64, 2, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
        with pytest.raises(ValueError):
            mod.kv4_write(bad, x, cache, n, tb)
    for lens, table, starts in ((n.long(), tb, None), (n, tb.long(), None), (n, tb[:1], None),
                                (n, tb.t(), None), (n, tb, ints([0, 1])), (n.cpu(), tb, None),
                                (n, tb.cpu(), None)):
        with pytest.raises(ValueError):
            mod.kv4_write(x, x, cache, lens, table, starts)
    with pytest.raises(mod.WQError) as e:
        mod.kv4_write(x[:1], x[:1], cache, n, tb)       # one row of two sequences
    assert e.value.status == 1
    with pytest.raises(ValueError):
        mod.kv4_read(cache, n, tb)
    q = torch.zeros(2, 3, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        mod.kv4_attention(q, cache, n, tb)              # 3 query heads on 2
    with pytest.raises(mod.WQError) as e:
        mod.kv4_attention(x, cache, n, tb, workspace=mod.kv4_workspace()[:1024])
    assert e.value.status == 1
    with pytest.raises(ValueError):
        mod.KV4Cache(cache.k_codes, cache.k_meta, cache.v_codes, cache.v_meta, 64)
    empty = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    assert mod.kv4_attention(empty, cache, none, tb[:0]).shape == empty.shape
    mod.kv4_write(empty, empty, cache, none, tb[:0])
