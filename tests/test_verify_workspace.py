"""The workspace of the verification of drafts: its size (no GPU), and calls of so many
sequences that each has fewer shares of it than its row could fill."""
import pytest
import torch

from tests.gpu_util import wq
from tests.test_kv4_gpu import ints, starts_of
from tests.test_verify_gpu import make


def test_bytes():
    size = wq().lib.wq_verify_workspace_bytes
    rows = [1, 2, 5, 1000, 1024, 1025, 2000, 16_383, 16_384, 16_385, 1 << 20, 1 << 23]
    got = [size(r) for r in rows]
    assert got == sorted(got) and all(n % 16 == 0 for n in got)
    assert [n / r for n, r in zip(got, rows)][:5] == [12_336] * 5
    assert [n / r for n, r in zip(got, rows)][-4:] == [2_736] * 4
    # the most rows that a call may have: a seventh of the memory of one GPU
    assert got[-1] < 180e9 / 7


@pytest.mark.gpu
@pytest.mark.parametrize("pattern", [[2, 1], [2, 0, 0, 1, 0]])   # more rows, more sequences
@pytest.mark.parametrize("dense", [True, False])
def test_thousands_of_sequences(pattern, dense):
    """Sequences that are copies of a few give those sequences' tokens."""
    few, copies, vocab = 17, 153, 65_000
    rows = pattern * few
    target, draft, tokens, uniform = make(3, rows, vocab, torch.bfloat16)
    uniform[::2] = 0.99                      # (drafts are refused more often)
    if not dense:
        draft = None

    def run(k):
        out = (torch.full((k * sum(rows),), 77, dtype=torch.int32, device="cuda"),
               torch.full((k * len(rows),), 77, dtype=torch.int32, device="cuda"), None)
        wq().verify_drafts(target.repeat(k, 1), tokens.repeat(k), uniform.repeat(k),
                           draft if draft is None else draft.repeat(k, 1),
                           row_starts=ints(starts_of(rows * k)), logits=True, out=out)
        assert wq().get_device_error() == 0
        return out[0].view(k, -1), out[1].view(k, -1)
    once, many = run(1), run(copies)
    for a, b in zip(once, many):
        assert torch.equal(b, a.expand_as(b))
    assert (once[1] == 0).any() and (once[0] >= 0).sum() >= few * sum(t > 0 for t in pattern)
