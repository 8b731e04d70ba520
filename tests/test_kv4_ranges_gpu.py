"""Attention over the 4-bit cache where binary32 scores are coarse and where
tokens tie.  The keys are powers of two times one pattern, so that scores fall
on a few levels far apart and are equal, bit for bit, on each: the softmax is
known without forming a score, however large it is, and the tolerance holds
the roundings of weights, values and sums only."""
import numpy as np
import pytest
import torch

from tests import kv4_ref as ref
from tests.gpu_util import wq
from tests.test_kv4_gpu import ints, new_cache, reference

pytestmark = pytest.mark.gpu

PAGE = 32


def cached(d, group, k, v, seed=0):
    """A cache that holds the rows k and v [n, heads, d] of one sequence."""
    n, heads = k.shape[:2]
    table, pages = ref.random_batch(seed, [n], PAGE)
    cache = new_cache(pages, heads, d, PAGE, group)
    wq().kv4_write(k.to(torch.bfloat16).cuda(), v.to(torch.bfloat16).cuda(), cache, ints([n]),
                   ints(table))
    return cache, table


def known(cache, table, n, p):
    """Output and bound of rows whose softmax p [rows, n] (the same for every
    head) is known, [rows, kv_heads, d]."""
    c, s, z = ref.sequence_values(cache.v_codes.cpu().numpy(), cache.v_meta.cpu().numpy(),
                                  table[0], n, PAGE, "v")
    heads, groups = s.shape[1:]
    g = cache.head_dim // groups
    values = ((c.reshape(n, heads, groups, g) - z[..., None]) * s[..., None]).reshape(n, heads, -1)
    out = np.einsum("tn,nhd->thd", p, values)
    # few rows: half a step of binary16 of each weight times |u - 8| <= 8
    w8 = np.repeat(np.einsum("tn,nhg->thg", p, s) * 8, g, -1)
    # many rows: half a step of each weight and of each value
    wabs = np.einsum("tn,nhd->thd", p, np.abs(values))
    # weights below binary16's normal range (see ref.attention); scores below
    # 2^12, of which the few-row kernel rounds those in steps with masked tokens by
    # 2^-13 (ln 2 of that in the weight, in the numerator and the sum); and binary32
    # sums over the tokens, the zeros' correction being as large as the codes'
    tiny = n * 8 * 2.0 ** -25 * s.max(0).max(-1)[None, :, None]
    sums = n * 2.0 ** -23 * (2 * w8 + wabs) + 2.0 ** -12 * wabs
    return out, np.maximum(2.0 ** -11 * w8, 2.0 ** -10 * 1.01 * wabs) + tiny + sums


def levels_softmax(level, top, rows):
    """Softmax [rows, n] of scores that fall with `level` (rises, where top is
    negative): equal over the visible tokens of the best level."""
    n = len(level)
    p = np.zeros((rows, n))
    for i in range(rows):
        seen = level[:n - rows + i + 1]
        best = seen == (seen.min() if top[i] > 0 else seen.max())
        p[i, :len(seen)][best] = 1 / best.sum()
    return p


def far_rows(rows, exponent, heads, gqa, d, pattern):
    """Queries whose base-2 scores with the pattern are about +-2^exponent."""
    sign = torch.tensor([1.0, -1.0, -1.0, 1.0, 1.0]).roll(exponent).repeat(rows)[:rows]
    size = torch.exp2(exponent - 4 - torch.arange(rows) % 3)     # d/sqrt(d) log2(e) is about 2^4
    q = (sign * size * (128 / d) ** 0.5).view(-1, 1, 1) * pattern.sign().expand(rows, heads * gqa, d)
    return q, sign.numpy()


MANY = [(64, 32, 2, 4, 40, 300), (128, 64, 2, 4, 70, 300), (128, 128, 1, 2, 150, 700),
        (64, 64, 90, 3, 20, 200)]        # the last without splits
FEW = [(64, 32, 2, 4, 1, 300), (128, 64, 2, 4, 3, 300), (128, 32, 2, 8, 2, 1200),
       (128, 128, 1, 1, 1, 5000), (64, 64, 100, 20, 1, 200)]    # the last in blocks of rows


@pytest.mark.parametrize("d,group,heads,gqa,rows,n", MANY + FEW)
@pytest.mark.parametrize("exponent", [13, 18, 23, 24, 25, 28, 29, 31, 34, 40, 100])
def test_scores_of_any_size(d, group, heads, gqa, rows, n, exponent):
    g = torch.Generator().manual_seed(exponent)
    pattern = torch.where(torch.rand(d, generator=g) < 0.5, -1.0, 1.0)
    level = (np.arange(n) * 7 + 3) % 5
    k = torch.exp2(-torch.tensor(level).float()).view(n, 1, 1) * pattern.expand(n, heads, d)
    cache, table = cached(d, group, k, ref.keys(2, n, heads, d, 1.0))
    q, sign = far_rows(rows, exponent, heads, gqa, d, pattern)
    # a few rows of ordinary queries among them
    plain = [r for r in range(rows) if r % 7 == 3]
    q[plain] = ref.keys(3, len(plain), heads * gqa, d, 1.0).float()
    q = q.to(torch.bfloat16).cuda()
    got = wq().kv4_attention(q, cache, ints([n]), ints(table))
    assert wq().get_device_error() == 0
    out, bound = (np.repeat(x, gqa, 1) for x in known(cache, table, n,
                                                      levels_softmax(level, sign, rows)))
    if plain:
        o, e = reference(q, cache, [n], [rows], table, d ** -0.5)
        out[plain], bound[plain] = o[plain], e[plain]
    ref.check(got, out, bound)


@pytest.mark.parametrize("d,group,heads,gqa,rows,n", MANY + FEW)
@pytest.mark.parametrize("exponent", [27, 29, 33])
def test_any_large_scores_give_a_mean_of_values(d, group, heads, gqa, rows, n, exponent):
    """Scores without structure: whatever they round to, an output is a mean
    of the visible values."""
    v = ref.keys(4, n, heads, d, 1.0)
    cache, table = cached(d, group, ref.keys(1, n, heads, d), v)
    q = ref.keys(5, rows, heads * gqa, d, 1.0).float() * 2.0 ** exponent
    got = wq().kv4_attention(q.to(torch.bfloat16).cuda(), cache, ints([n]), ints(table))
    held = wq().kv4_read(cache, ints([n]), ints(table), rows=n)[1].float().abs()
    # each rounding of a value, a weight and the output is below 2^-8
    most = held.amax(0).repeat_interleave(gqa, 0) * (1 + 2.0 ** -6)
    assert (got.float().abs() <= most).all()
    assert got.float().abs().amax((1, 2)).min() > 0
    assert wq().get_device_error() == 0


@pytest.mark.parametrize("d,group,heads,gqa,rows,n", MANY + FEW)
@pytest.mark.parametrize("score", [0.0, 5.3, 33.3, 61.7, -1000.1, 70000.7, 2.0 ** 26])
@pytest.mark.parametrize("large", ["k", "v", "kv"])
def test_equal_scores_beside_the_largest_values(d, group, heads, gqa, rows, n, score, large):
    """Every key the same, and codes that can stand for more than binary16's
    largest value: as many weights as a step has are as large as one can be."""
    g = torch.Generator().manual_seed(d)
    pattern = torch.where(torch.rand(d, generator=g) < 0.5, -1.0, 1.0)
    k = pattern.expand(n, heads, d) * (60000.0 if "k" in large else 1.0)
    v = ref.keys(2, n, heads, d, 1.0).float().clamp(-1, 1)
    if "v" in large:
        v = torch.where(v.abs() > 0.5, v.sign(), v) * 60000.0
    cache, table = cached(d, group, k, v)
    size = score / (d ** 0.5 * 1.4427) / (60000.0 if "k" in large else 1.0)
    q = (pattern * size).expand(rows, heads * gqa, d).to(torch.bfloat16).cuda()
    got = wq().kv4_attention(q, cache, ints([n]), ints(table))
    assert wq().get_device_error() == 0
    p = np.zeros((rows, n))
    for i in range(rows):
        p[i, :n - rows + i + 1] = 1 / (n - rows + i + 1)
    out, bound = known(cache, table, n, p)
    ref.check(got, np.repeat(out, gqa, 1), np.repeat(bound, gqa, 1))


def test_references_that_rise_row_by_row():
    """Keys that grow with the token, over many steps of one CTA: the rows of a
    warp raise their references in different steps."""
    d, group, heads, gqa, rows, n = 64, 32, 90, 1, 64, 1500
    grow = 1 + 3 * (torch.arange(n) // 100).view(n, 1, 1)
    cache, table = cached(d, group, ref.keys(1, n, heads, d, 1.0).float() * grow,
                          ref.keys(2, n, heads, d, 1.0))
    q = ref.keys(3, rows, heads * gqa, d, 1.0).float()
    q *= torch.exp2(torch.arange(rows) % 5 - 3.0).view(-1, 1, 1)
    q = q.to(torch.bfloat16).cuda()
    got = wq().kv4_attention(q, cache, ints([n]), ints(table))
    out, bound = reference(q, cache, [n], [rows], table, d ** -0.5)
    ref.check(got, out, bound)
    assert wq().get_device_error() == 0


@pytest.mark.parametrize("d,group", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128)])
@pytest.mark.parametrize("what", ["key beside values", "value beside keys", "value of a later token",
                                  "key of a later token", "every seventh"])
def test_values_near_binary16s_smallest_beside_its_largest(d, group, what):
    """A key or a value that can stand for more than binary16's largest does
    not change what the tokens around it hold, nor the other one of its token."""
    heads, gqa, rows, n, at = 2, 4, 200, 400, 300
    k, v = ref.keys(1, n, heads, d, 1.0).float(), ref.keys(2, n, heads, d, 1.0).float()
    q = ref.keys(3, rows, heads * gqa, d, 1.0).float()
    large = torch.where(ref.keys(4, n, heads, d, 1.0).float() < 0, -60000.0, 60000.0)
    if what == "key beside values":
        k[at], v = large[at], v * 2.0 ** -20
        q *= 2.0 ** -8             # its score does not take every weight
    elif what == "value beside keys":
        k, v[at], q = k * 2.0 ** -20, large[at], q * 2.0 ** 20
    elif what == "value of a later token":
        v = v * 2.0 ** -20
        v[at] = large[at]
    elif what == "key of a later token":
        k, q = k * 2.0 ** -20, q * 2.0 ** 20
        k[at] = large[at]
    else:
        v[::7], k[3::7] = large[::7], large[3::7]
        q *= 2.0 ** -14
    cache, table = cached(d, group, k, v)
    q = q.to(torch.bfloat16).cuda()
    got = wq().kv4_attention(q, cache, ints([n]), ints(table))
    assert wq().get_device_error() == 0
    out, bound = reference(q, cache, [n], [rows], table, d ** -0.5)
    ref.check(got, out, bound)


@pytest.mark.parametrize("rows", [1, 3, 40])
@pytest.mark.parametrize("scale", [3.4e38, -3.4e38, 2.4e38, 1e-45, 0.0])
def test_queries_of_zero_give_the_mean_at_every_scale(rows, scale):
    d, group, heads, gqa, n = 64, 32, 2, 4, 300
    cache, table = cached(d, group, ref.keys(1, n, heads, d), ref.keys(2, n, heads, d, 1.0))
    q = torch.zeros(rows, heads * gqa, d, dtype=torch.bfloat16, device="cuda")
    got = wq().kv4_attention(q, cache, ints([n]), ints(table), scale=scale)
    p = np.zeros((rows, n))
    for i in range(rows):
        p[i, :n - rows + i + 1] = 1 / (n - rows + i + 1)
    out, bound = known(cache, table, n, p)
    ref.check(got, np.repeat(out, gqa, 1), np.repeat(bound, gqa, 1))
