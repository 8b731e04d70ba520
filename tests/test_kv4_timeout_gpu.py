"""The timeout paths of the attention kernels over the 4-bit cache, made to run
without faulting the GPU: through an internal test hook the copies of one CTA
(the keys of one, in the kernel for many rows) never count as complete, and
its waits give up after 20 ms instead of 2 s.  The copies themselves are made,
and end long before that, so nothing is left in flight.  The call must record
WQ_ERR_TIMEOUT, the context must stay usable, and once the workspace is
zero-filled again the next call must give the same bits as a clean one."""
import ctypes

import pytest
import torch

from tests import kv4_ref as ref
from tests.gpu_util import wq
from tests.test_kv4_gpu import COUNTERS, fill, ints, new_cache

pytestmark = pytest.mark.gpu


@pytest.fixture
def hook():
    lib = wq().lib
    lib.wq_internal_kv4_timeout_test.argtypes = [ctypes.c_int, ctypes.c_uint]
    lib.wq_internal_kv4_timeout_test.restype = None
    yield lib.wq_internal_kv4_timeout_test
    lib.wq_internal_kv4_timeout_test(-1, 0)


@pytest.mark.parametrize("d,group,heads,gqa,lens,rows", [
    (128, 64, 2, 4, [9000], 1),          # few rows: one sequence over many CTAs
    (64, 32, 4, 2, [300, 20, 700], 2),
    (128, 64, 1, 4, [5000], 40),         # many rows: a block over many CTAs
    (64, 32, 90, 3, [200], 20)])         # without splits
@pytest.mark.parametrize("cta", [0, 1, 5])
def test_timed_out_wait_is_reported_and_the_next_call_is_clean(hook, d, group, heads, gqa, lens,
                                                               rows, cta):
    mod = wq()
    table, pages = ref.random_batch(3, lens, 32)
    cache = new_cache(pages, heads, d, 32, group)
    fill(cache, lens, table)
    q = ref.keys(1, rows * len(lens), heads * gqa, d, 1.0).cuda()
    n, tb, ws = ints(lens), ints(table), mod.kv4_workspace()
    clean = mod.kv4_attention(q, cache, n, tb, workspace=ws).clone()
    assert mod.get_device_error() == 0 and not ws[:COUNTERS].any()

    hook(cta, 20_000_000)                                       # 20 ms
    mod.kv4_attention(q, cache, n, tb, workspace=ws)
    assert mod.get_device_error() == 5                          # WQ_ERR_TIMEOUT
    assert mod.get_device_error() == 0                          # read and cleared

    hook(-1, 0)
    ws.zero_()                                                  # as wq.h asks
    again = mod.kv4_attention(q, cache, n, tb, workspace=ws)
    torch.cuda.synchronize()
    assert mod.get_device_error() == 0 and not ws[:COUNTERS].any()
    assert torch.equal(again, clean)
