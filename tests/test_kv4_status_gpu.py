"""What the 4-bit cache's calls record in the device status word, and that it
is theirs: nothing of one call is reported for another."""
import os
import subprocess
import sys

import numpy as np
import pytest

from tests import kv4_ref as ref
from tests.gpu_util import wq
from tests.test_kv4_gpu import fill, ints, new_cache, starts_of

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_an_error_is_reported_once():
    """A padded batch of short sequences: the kernel for many rows is launched
    and finds no work in any CTA, one length is too large.  The error belongs to
    that call alone."""
    d, group, heads, gqa, page = 64, 32, 2, 4, 16
    lens, rows = [40, 33, 20, 64], [2, 2, 2, 2]
    table, pages = ref.random_batch(3, lens, page)
    cache = new_cache(pages, heads, d, page, group)
    fill(cache, lens, table)
    q = ref.keys(1, 300, heads * gqa, d).cuda()          # rows behind the last sequence
    many = [64, 33, 20, 64]
    wide = ints(np.array([[7, 1, 2, 3]] * 4) % pages)
    fill(cache, [64], np.array([[7, 1, 2, 3]]) % pages)
    for _ in range(50):
        wq().kv4_attention(q, cache, ints([40, 33, 20, 10 ** 6]), ints(table), ints(starts_of(rows)))
        assert wq().get_device_error() == 1
        wq().kv4_attention(q[:80], cache, ints([64]), wide[:1], ints([0, 60]))
        wq().kv4_attention(q[:40], cache, ints(many[:1]), wide[:1])
        assert wq().get_device_error() == 0


CAPTURE_FIRST = """
import sys
sys.path.insert(0, {root!r})
import torch
import w4a16_decode_matmul_b200 as wq
from tests import kv4_ref as ref
heads, d = 2, 64
cache = wq.kv4_cache(40, heads, d, page_size=16, group=32)
for t in (cache.k_codes, cache.v_codes, cache.k_meta, cache.v_meta):
    t.zero_()
n = torch.tensor([600], dtype=torch.int32, device="cuda")
tb = torch.randperm(40)[None].to(torch.int32).cuda()
x = ref.keys(1, 600, heads, d).cuda()
q = ref.keys(2, {rows}, 4 * heads, d, 1.0).cuda()
ws = wq.kv4_workspace()
out = torch.zeros_like(q)
back = [torch.zeros_like(x), torch.zeros_like(x)]
torch.cuda.synchronize()
stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
with torch.cuda.graph(graph, stream=stream):
    if {rows} == 1:
        wq.kv4_write(x, x, cache, n, tb)
        wq.kv4_attention(q, cache, n, tb, out=out, workspace=ws)
    else:
        wq.kv4_attention(q, cache, n, tb, out=out, workspace=ws)
        wq.kv4_write(x, x, cache, n, tb)
    wq.kv4_read(cache, n, tb, out=back)
graph.replay()
graph.replay()
torch.cuda.synchronize()
assert torch.equal(wq.kv4_attention(q, cache, n, tb), out)
for a, b in zip(wq.kv4_read(cache, n, tb, rows=600), back):
    assert torch.equal(a, b)
assert wq.get_device_error() == 0 and out.any()
print("captured")
"""


@pytest.mark.parametrize("rows", [1, 60])
def test_a_process_may_capture_its_first_calls(rows):
    run = subprocess.run([sys.executable, "-c", CAPTURE_FIRST.format(root=ROOT, rows=rows)],
                         capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert run.returncode == 0 and "captured" in run.stdout, run.stderr[-2000:]


@pytest.mark.parametrize("lens,starts", [
    ([40, 40], [0, 4, 10]),              # a range behind the last row
    ([40, 40], [-2, 0, 4]),              # one before the first
    ([40, 40, 40], [0, 4, 2, 4]),        # one that ends before it begins
    ([40, 10 ** 6, 40], [0, 2, 2, 4]),   # a sequence without rows, too long
    ([40] * 4999 + [10 ** 6], [0, 4] + [4] * 4999)])
def test_sequences_without_a_row_of_the_call_are_checked(lens, starts):
    """In every call: rows 0 .. 3 belong to other sequences than the bad one."""
    d, group, heads, page, rows = 64, 32, 2, 16, 4
    table = np.tile(np.arange(3, dtype=np.int32), (len(lens), 1))
    cache = new_cache(3, heads, d, page, group)
    fill(cache, [40], table[:1])
    x = ref.keys(1, rows, heads, d).cuda()
    good = ints([40] * len(lens)), ints(table), ints([0] + [rows] * len(lens))
    bad = ints(lens), ints(table), ints(starts)
    calls = [lambda b: wq().kv4_write(x, x, cache, *b), lambda b: wq().kv4_read(cache, *b, rows=rows),
             lambda b: wq().kv4_attention(x, cache, *b)]
    for call in calls:
        call(bad)
        assert wq().get_device_error() == 1
        call(good)
        assert wq().get_device_error() == 0
