"""Rotary positions on the way into the cache, batches that hold something out of bounds:
what a call may not touch is compared as a whole -- codes and metadata of keys and values,
pages around the cache, the other sequences' queries."""
import numpy as np
import pytest
import torch

from tests import kv4_ref as ref
from tests.gpu_util import host_bits, wq
from tests.test_kv4_gpu import SENTINEL, assert_cache, images, ints, starts_of
from tests.test_rotary_gpu import check, expect

pytestmark = pytest.mark.gpu

GUARD = 2  # pages in front of the cache and behind it


def guarded(pages, heads, d, page, group):
    def within(shape, dtype, value):
        return torch.full((pages + 2 * GUARD, heads, page, *shape), value, dtype=dtype,
                          device="cuda")
    whole = [within(s, t, v) for _ in "kv" for s, t, v in
             (((d // 2,), torch.uint8, SENTINEL), ((d // group, 2), torch.float16, float("nan")))]
    return wq().KV4Cache(*(x[GUARD:-GUARD] for x in whole), group), whole


@pytest.mark.parametrize("d,group", [(64, 32), (128, 128)])
@pytest.mark.parametrize("many", [0, 40])       # sequences behind, so that there are 32 or more
@pytest.mark.parametrize("change", ["page", "page below", "length", "rows", "rows below"])
def test_only_the_bad_sequence_is_unspecified(change, many, d, group):
    heads, q_heads, page = 2, 4, 16
    lens, rows = [20, 30, 10] + [12] * many, [2, 2, 2] + [1] * many
    n, bad = sum(rows), 1
    table, pages = ref.random_batch(3, lens, page)
    starts = starts_of(rows)
    # the bad sequence's rows come last where its end is what is wrong
    if change == "rows":
        bad = len(lens) - 1
    args = [np.asarray(lens), table.copy(), np.asarray(starts)]
    if change == "page":
        args[1][bad, 29 // page] = pages
    elif change == "page below":
        args[1][bad, 29 // page] = -1
    elif change == "length":
        args[0][bad] = page * table.shape[1] + 1
    elif change == "rows":
        args[2][-1] = n + 3
    else:
        args[2][0] = -1                        # the first sequence's rows begin before the batch
        bad = 0
    qkv = torch.cat((ref.keys(1, n, q_heads + heads, d), ref.keys(2, n, heads, d)), 1).cuda()
    q, k, v = qkv[:, :q_heads], qkv[:, q_heads:-heads], qkv[:, -heads:]
    rot = wq().Rotary(wq().rotary_frequencies(d).cuda())
    cache, whole = guarded(pages, heads, d, page, group)
    around = [host_bits(torch.cat((x[:GUARD], x[-GUARD:]))).copy() for x in whole]
    want = images(cache)
    held, _ = ref.places(lens, rows, table, page)
    positions = [m - t + i for m, t in zip(lens, rows) for i in range(t)]
    others = [h for h in held if h[1] != bad]
    expect(k, positions, rot, others, v, want, cache)
    out = wq().kv4_write_rotary(q, k, v, cache, rot, *(ints(a) for a in args))
    assert wq().get_device_error() == 1
    # the bad sequence's own pages may hold anything; all else is as expected
    own = sorted({int(p) for p in table[bad] if 0 <= p < pages})
    for t in (cache.k_codes, cache.k_meta, cache.v_codes, cache.v_meta):
        t[own] = 0
    for image in want.values():
        for x in image:
            x[own] = 0
    assert_cache(cache, want)
    for x, y in zip(whole, around):
        assert np.array_equal(host_bits(torch.cat((x[:GUARD], x[-GUARD:]))), y)
    mine = torch.tensor([r for r in range(n) if r not in range(starts[bad], starts[bad + 1])])
    check(out[mine.cuda()], q[mine.cuda()], [positions[r] for r in mine.tolist()],
          rot.freqs.cpu(), False)
