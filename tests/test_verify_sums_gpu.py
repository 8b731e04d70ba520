"""Verification of drafts where every error of a row's sum of exponentials has the same
sign: rows of two levels, whose many low logits all round alike."""
import math

import numpy as np
import pytest
import torch

from tests.gpu_util import wq
from tests.test_kv4_gpu import ints
from tests.test_verify_gpu import run

pytestmark = pytest.mark.gpu

HIGH = 8.660868644714355
LOW = (0.31713345646858215, 0.3171333372592926)  # four steps of 32 bits apart


def levels(n, vocab, low, stride=4096):
    x = torch.full((n, vocab), low, device="cuda")
    x[:, ::stride] = HIGH
    return x


@pytest.mark.parametrize("seqs,vocab", [(2, 32_768), (40, 32_768), (2, 131_072), (40, 131_072)])
@pytest.mark.parametrize("swapped", [False, True])
@pytest.mark.parametrize("stride", [512, 4096])
def test_what_is_left_of_two_levels_that_differ_by_a_rounding(seqs, vocab, swapped, stride):
    """A refused draft (outside the vocabulary) leaves max(p - q, 0), which lies on the low
    tokens or on the high ones, by the true sums: p and q of the low ones differ by about
    6 10^-8 of themselves."""
    low = LOW[::-1] if swapped else LOW
    rows = [2] * seqs
    target, draft = levels(2 * seqs, vocab, low[0], stride), levels(2 * seqs, vocab, low[1], stride)
    tokens = ints([vocab] * (2 * seqs))
    # (numbers that end inside a token's mass)
    uniform = torch.tensor([(i + 0.5) / (2 * seqs) for i in range(2 * seqs)], device="cuda")
    uniform[0] = 0.2
    got, want = run(target, tokens, uniform, draft, rows)
    assert got[1:] == want[1:] and got[1] == [0] * seqs
    high = [x % stride == 0 for x in got[0][::2]]
    assert high == [x % stride == 0 for x in want[0][::2]]
    # what is left is the same for each token of a level, so a number that falls inside a
    # token's share gives that token.  The high ones are 2^k: numbers (i + 1/2) / n can fall on
    # a border between two of them, where either is right.  The low ones: one further for the
    # roundings of their running sum, one for a token without a share between.
    for g, w, u, h in zip(got[0][::2], want[0][::2], uniform[::2].tolist(), high):
        on_border = (u * (vocab // stride)).is_integer()
        assert abs(g - w) <= (stride * on_border if h else 2)


@pytest.mark.parametrize("seqs", [1, 40])
@pytest.mark.parametrize("swapped", [False, True])
def test_drafts_near_the_border_of_acceptance(seqs, swapped):
    """u q = p but for 7 10^-7, on either side.  Threads whose logits are all alike sum ones,
    exactly; what is left is one exponential between a thread's largest logit and the row's, off by
    2^-22 and a rounding, 2^-24: 3 10^-7 for p, the same for q."""
    vocab, x = 131_072, 1234
    low = LOW[::-1] if swapped else LOW
    rows = [2] * seqs
    target, draft = levels(2 * seqs, vocab, low[0]), levels(2 * seqs, vocab, low[1])
    draft[:, x] = low[1] + 0.5
    p, q = (r.double().cpu() for r in (target[0], draft[1]))
    ratio = math.exp(float(p[x] - torch.logsumexp(p, 0) - q[x] + torch.logsumexp(q, 0)))
    for side in (-1, 1):
        u = np.float32(ratio * (1 + side * 6.5e-7))
        while abs(float(u) / ratio - 1) < 6e-7:
            u = np.nextafter(u, np.float32(2 if side > 0 else 0))
        uniform = torch.full((2 * seqs,), float(u), device="cuda")
        tokens = ints([x] * (2 * seqs))
        _, accepted, _ = wq().verify_drafts(target, tokens, uniform, draft, seqs=seqs, logits=True)
        assert accepted.tolist() == [1 if side < 0 else 0] * seqs, side


@pytest.mark.parametrize("seqs,vocab", [(2, 8192), (2, 32_768), (40, 8192), (40, 65_536)])
@pytest.mark.parametrize("swapped", [False, True])
@pytest.mark.parametrize("rows", ["far apart", "neighbours"])
def test_sums_whose_errors_are_farthest_apart(seqs, vocab, swapped, rows):
    """One large logit among the 32 of every thread: of many levels these gave the sums with the
    largest errors measured, 4.3 10^-7 up and 4.4 10^-7 down (and 8.4 10^-7 between two
    neighbours), so that all of a refused draft's rows are summed again."""
    pair = {"far apart": ((1.0161354541778564, -5.315082550048828),
                          (4.238065242767334, 0.17843985557556152)),
            "neighbours": ((3.1992855072021484, -2.8756802082061768),
                           (3.1992855072021484, -2.8756825923919678))}[rows]
    at = torch.arange(vocab, device="cuda")
    first = (at % 4 == 0) & (at % 4096 < 512)          # of a thread
    p, q = (torch.where(first, hi, lo) for hi, lo in (pair[::-1] if swapped else pair))
    n = 2 * seqs
    tokens = ints([vocab] * n)
    uniform = (torch.arange(n, device="cuda") + 0.37) / n
    got, want = run(p.expand(n, vocab).contiguous(), tokens, uniform, q.expand(n, vocab).contiguous(),
                    [2] * seqs)
    assert got[1:] == want[1:] and got[1] == [0] * seqs
    # the tokens of a level all have the same mass: a number next to a border (of 8,192 to
    # 65,536 of them, within some 10^-11 of a mass) is the only one that could give a neighbour
    assert got[0] == want[0]
