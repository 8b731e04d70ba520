"""Rotary positions with frequencies above one: angles of up to 2^50 radians, against the
host's sine and cosine of the binary64 product."""
import numpy as np
import pytest
import torch

from tests.gpu_util import wq
from tests.test_kv4_gpu import ints

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
def test_angles_of_up_to_2_to_the_50(interleaved, inverse):
    n, dim = 500, 64
    rng = np.random.default_rng(2)
    freqs = np.exp2(rng.uniform(-3, 19, dim // 2)).astype(np.float32)
    positions = np.exp2(rng.uniform(0, 31, n)).astype(np.int64).clip(max=2 ** 31 - 1)
    positions = (positions * rng.choice([-1, 1], n)).astype(np.int32)
    positions[:2] = 2 ** 31 - 1, -(2 ** 31)
    angle = positions.astype(np.float64)[:, None] * freqs.astype(np.float64)
    assert 2.0 ** 49 < np.abs(angle).max() < 2.0 ** 50
    c, s = np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32)
    if inverse:
        s = -s
    x = torch.randn(n, 1, dim, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    a, b = (x[:, 0, 0::2], x[:, 0, 1::2]) if interleaved else (x[:, 0, :32], x[:, 0, 32:])
    a, b, c, s = a.double().numpy(), b.double().numpy(), c.astype(np.float64), s.astype(np.float64)
    want, mag = (a * c - b * s, b * c + a * s), np.abs(a) + np.abs(b)
    got = wq().rotary(x.cuda(), ints(positions), wq().Rotary(torch.tensor(freqs).cuda(), interleaved),
                      inverse=inverse)[:, 0].double().cpu().numpy()
    got = (got[:, 0::2], got[:, 1::2]) if interleaved else (got[:, :32], got[:, 32:])
    # bfloat16's half step; c and s of either side's binary32 (2^-24 each), a product and a sum
    for g, w in zip(got, want):
        assert (np.abs(g - w) <= 2.0 ** -8 * np.abs(w) + 4 * 2.0 ** -24 * mag).all()
