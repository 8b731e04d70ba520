"""Verification of drafted tokens on the B200 against the definition in
binary64: accepted drafts, the token behind them and the lengths have to be
equal.  Numbers at the borders come from distributions whose sums are exact."""
import numpy as np
import pytest
import torch

from tests.gpu_util import wq
from tests.test_kv4_gpu import ints, starts_of

pytestmark = pytest.mark.gpu


def masses(x, logits, hot):
    x = x.astype(np.float64)
    if not logits:
        return np.where(x > 0, x, 0.0)
    x = np.where(np.isnan(x), -np.inf, x)
    top = x.max()
    if top == -np.inf:
        return np.zeros_like(x)
    if not hot > 0:
        one = np.zeros_like(x)
        one[np.argmax(x)] = 1
        return one
    with np.errstate(invalid="ignore"):
        e = np.where(x == top, 1.0, np.exp((x - top) / hot))
    e = np.where(x == -np.inf, 0.0, e)
    return e / e.sum()


def clamp(u):
    return 0.0 if np.isnan(u) else float(min(max(u, 0.0), 1 - 2.0 ** -24))


def expected(target, tokens, uniform, draft, rows, logits, temperature, lens):
    out, accepted, left, at = [], [], [], 0
    for b, t in enumerate(rows):
        hot = 1.0 if temperature is None else float(temperature[b])
        a = 0
        while a < t - 1:
            x = int(tokens[at + a + 1])
            if not 0 <= x < target.shape[1]:
                break
            p = masses(target[at + a], logits, hot)
            drawn = 1.0
            if draft is not None and not (logits and not hot > 0):
                drawn = masses(draft[at + a + 1], logits, hot)[x]
            if not clamp(uniform[at + a + 1]) * drawn < p[x]:
                break
            a += 1
        if t:
            p = masses(target[at + a], logits, hot)
            if a < t - 1:
                x = int(tokens[at + a + 1])
                if draft is None or (logits and not hot > 0):
                    q = np.zeros_like(p)
                    if 0 <= x < len(q):
                        q[x] = 1
                else:
                    q = masses(draft[at + a + 1], logits, hot)
                rest = np.maximum(p - q, 0)
                if rest.sum() > 0:
                    p = rest
            total = np.cumsum(p)
            hit = np.flatnonzero((total > clamp(uniform[at]) * total[-1]) & (p > 0))
            some = np.flatnonzero(p > 0)
            x = int(hit[0]) if len(hit) else int(some[-1]) if len(some) else -1
            out += [int(v) for v in tokens[at + 1:at + 1 + a]] + [x] + [-1] * (t - 1 - a)
        accepted.append(a if t else 0)
        left.append(int(lens[b]) - (t - 1 - a if t else 0))
        at += t
    return out, accepted, left


def host(x):
    return None if x is None else x.float().cpu().numpy()


def run(target, tokens, uniform, draft, rows, logits=True, temperature=None, behind=0, ragged=True,
        **kw):
    lens = [100 + 7 * i for i in range(len(rows))]
    n = sum(rows)
    out = (torch.full((n + behind,), 77, dtype=torch.int32, device="cuda"),
           torch.full((len(rows),), 77, dtype=torch.int32, device="cuda"),
           torch.full((len(rows),), 77, dtype=torch.int32, device="cuda"))
    got = wq().verify_drafts(
        target, tokens, uniform, draft=draft, seqs=len(rows),
        row_starts=ints(starts_of(rows)) if ragged else None, logits=logits,
        temperature=temperature, seq_lens=ints(lens), out=out, **kw)
    assert wq().get_device_error() == 0
    want = expected(host(target), tokens.cpu().numpy(), host(uniform), host(draft), rows, logits,
                    host(temperature), lens)
    assert (got[0][n:] == 77).all()
    return [x.tolist() for x in (got[0][:n], got[1], got[2])], [list(w) for w in want]


def make(seed, rows, vocab, dtype, hot=None, noise=0.5, behind=0, pad=0):
    """Target and draft logits that agree for the most part, and tokens of the draft."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = sum(rows) + behind
    base = 3 * torch.randn(n + 1, vocab + pad, generator=g, device="cuda")
    target = (base[1:] + noise * torch.randn(n, vocab + pad, generator=g, device="cuda")).to(dtype)
    draft = base[:-1].contiguous().to(dtype)
    t = torch.ones(len(rows), device="cuda") if hot is None else hot
    seq = torch.repeat_interleave(torch.arange(len(rows), device="cuda"),
                                  torch.tensor(rows, device="cuda"))
    seq = torch.cat((seq, seq.new_zeros(behind)))
    e = -torch.log(torch.rand(n, vocab, generator=g, device="cuda").clamp(1e-9, 1 - 1e-7))
    tokens = (draft[:, :vocab].float() / t.clamp(min=0.05)[seq, None] - torch.log(e)).argmax(-1)
    return target[:, :vocab], draft[:, :vocab], tokens.to(torch.int32), \
        torch.rand(n, generator=g, device="cuda")


SHAPES = [  # rows of the sequences, vocabulary, padding of a row
    ([1], 1, 0), ([2], 2, 0), ([5], 32000, 0), ([1, 4, 0, 7, 2, 1], 1003, 0), ([6] * 9, 8191, 0),
    ([3, 5], 8193, 5), ([4, 1, 6], 50021, 0), ([2, 3], 131072, 16), ([20], 300, 0),
    ([3] * 70, 777, 2), ([2], 600_001, 0), ([4] * 30, 50021, 0), ([3, 1, 0, 5, 2] * 8, 8193, 3),
    ([2] * 24, 131072, 0), ([35, 70, 33, 34], 200, 0), ([3] * 30, 40_960, 0), ([2, 2], 40_961, 0),
    ([40], 60_000, 0),
]


@pytest.mark.parametrize("rows,vocab,pad", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["logits", "probabilities"])
@pytest.mark.parametrize("dense", [True, False])
def test_verify(rows, vocab, pad, dtype, kind, dense):
    seen = set()
    for seed in range(3):
        g = torch.Generator(device="cuda").manual_seed(seed)
        hot = 0.5 + torch.rand(len(rows), generator=g, device="cuda")
        target, draft, tokens, uniform = make(seed + vocab, rows, vocab, dtype, hot, behind=2,
                                              pad=pad)
        if kind == "probabilities":
            hot = None
            target, draft = (torch.softmax(x.float(), -1).to(dtype) for x in (target, draft))
        got, want = run(target, tokens, uniform, draft if dense else None, rows, kind == "logits",
                        hot, behind=2)
        assert got == want
        seen |= set(got[1])
    if dense and len(rows) > 5:      # the inputs hold accepted and refused drafts
        assert len(seen) > 1


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dense", [True, False])
def test_greedy_beside_sampled(dtype, dense):
    rows = [4, 5, 1, 3, 6, 2]
    hot = torch.tensor([0.0, 1.0, 0.0, float("nan"), -1.0, 0.7], device="cuda")
    target, draft, tokens, uniform = make(3, rows, 5000, dtype, noise=0.0, behind=0)
    # the first sequence's drafts are the target's choices, and two tokens share the largest logit
    target[:, 4000] = target[:, 41] = target.amax(-1)
    tokens[1:4] = target[:3].float().argmax(-1).to(torch.int32).clamp(max=41)
    tokens[2] = 41
    got, want = run(target, tokens, uniform, draft if dense else None, rows, True, hot)
    assert got == want
    assert (np.asarray(got[0])[[9]] < 4000).all()          # the lowest of the largest


def test_rows_the_same_number_each_without_row_starts():
    rows = [4] * 6
    target, draft, tokens, uniform = make(5, rows, 999, torch.float32)
    got, want = run(target, tokens, uniform, draft, rows, ragged=False)
    assert got == want
    assert run(target, tokens, uniform, draft, rows)[0] == got


@pytest.mark.parametrize("vocab", [16, 4096, 40960])
def test_borders_are_strict(vocab):
    """Uniform masses of powers of two: u_0 at a border belongs to the token behind it; a draft
    whose u q equals p is refused."""
    rows, n = [2], 2
    p = torch.zeros(n, vocab, device="cuda")
    k = 16                                             # tokens with a mass of 1/16
    at = (torch.arange(k, device="cuda") * (vocab // k))
    p[:, at] = 1 / 16
    for i in (0, 3, 15):
        uniform = torch.tensor([i / 16, 0.5], device="cuda")
        draft = torch.zeros(n, vocab, device="cuda")
        draft[1, at[2]] = 1 / 8                        # u q = 1/16 = p: refused
        tokens = ints([0, int(at[2])])
        got, want = run(p, tokens, uniform, draft, rows, logits=False)
        assert got == want and got[1] == [0]
        # what is left: p - q = 0 at the refused token
        left = [int(x) for x in at if x != at[2]]
        assert got[0][0] == left[min(14, int(i * 15 / 16))]
        uniform[1] = 0.5 - 2.0 ** -25                  # a hair below: accepted
        got, want = run(p, tokens, uniform, draft, rows, logits=False)
        assert got == want and got[1] == [1] and got[0] == [int(at[2]), int(at[i])]


def test_evenly_spaced_numbers_give_the_distribution():
    """n numbers (i + 1/2)/n: token v comes up n p_v times, give or take one."""
    n, vocab = 4096, 300
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(1, vocab, generator=g, device="cuda") * 2
    uniform = (torch.arange(n, device="cuda") + 0.5) / n
    tokens, accepted, _ = wq().verify_drafts(x.expand(n, vocab).contiguous(), ints([0] * n), uniform,
                                             seqs=n, logits=True)
    count = torch.bincount(tokens.long(), minlength=vocab).double()
    p = torch.softmax(x[0].double(), -1)
    assert (accepted == 0).all() and ((count - n * p).abs() <= 1).all()
    assert (tokens[1:] >= tokens[:-1]).all()


def test_numbers_outside_the_unit_interval_and_tokens_outside_the_vocabulary():
    rows = [1, 1, 1, 1, 3, 3, 2]
    target, draft, tokens, uniform = make(8, rows, 500, torch.float32)
    uniform[0], uniform[1], uniform[2], uniform[3] = float("nan"), -3.0, 1.0, float("inf")
    tokens[5], tokens[8], tokens[11] = -1, 500, 2 ** 31 - 1
    uniform[5] = uniform[8] = uniform[11] = 0.0
    for d in (draft, None):
        got, want = run(target, tokens, uniform, d, rows)
        assert got == want
        assert got[1][4:] == [0, 0, 0]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("hot", [1.0, 0.0])
def test_masked_and_infinite_logits(dtype, hot):
    inf, vocab, rows = float("inf"), 9001, [1] * 8
    target, _, tokens, uniform = make(9, rows, vocab, dtype)
    target[0] = -inf                                 # no mass at all
    target[1] = float("nan")
    target[2, ::2] = -inf
    target[3, 1:] = -inf
    target[4, [17, 8500]] = inf                      # they share the mass
    target[5, [17, 8500]] = inf
    target[6] = torch.finfo(dtype).min               # the type's lowest value is no mask
    target[7, :vocab - 1] = torch.finfo(dtype).min
    uniform[4], uniform[5] = 0.4, 0.6
    got, want = run(target, tokens, uniform, None, rows, True, torch.full((8,), hot, device="cuda"))
    assert got == want
    # the same among many sequences, which take other kernels
    many, _ = run(target.repeat(4, 1), tokens.repeat(4), uniform.repeat(4), None, rows * 4, True,
                  torch.full((32,), hot, device="cuda"))
    assert many[0] == got[0] * 4
    assert got[0][:2] == [-1, -1] and got[0][3] == 0 and got[0][7] == vocab - 1
    assert got[0][4:6] == ([17, 8500] if hot else [17, 17])


def test_rows_without_mass_and_equal_distributions():
    """A refused draft with p = q everywhere: what is left is nothing, so p itself is sampled;
    probabilities that are negative or NaN count as zero."""
    vocab, rows = 1000, [2, 2, 1]
    p = torch.zeros(5, vocab, device="cuda")
    p[0, 10:20] = 0.1
    p[2, :] = -1.0
    p[2, 700], p[2, 5] = 0.5, float("nan")
    q = p[[0, 0, 0, 2, 0]].clone()
    tokens = ints([0, 3, 0, 5, 0])                   # p(3) = 0: refused; p(NaN) = 0: refused
    uniform = torch.tensor([0.35, 0.0, 0.9, 0.1, 0.5], device="cuda")
    got, want = run(p, tokens, uniform, q, rows, logits=False)
    assert got == want
    assert got[0] == [13, -1, 700, -1, -1] and got[1] == [0, 0, 0]
    many, _ = run(p.repeat(9, 1), tokens.repeat(9), uniform.repeat(9), q.repeat(9, 1), rows * 9,
                  logits=False)
    assert many[0] == got[0] * 9


@pytest.mark.parametrize("seqs", [3, 40])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("changed", [0, 1, 500])
def test_drafts_close_to_the_target(seqs, dtype, changed):
    """Draft logits that are the target's but for a few tokens: p and q differ by a constant
    factor close to 1 almost everywhere, on either side of it."""
    rows, vocab = [2] * seqs, 4001
    target, _, tokens, uniform = make(21, rows, vocab, dtype)
    draft = target.roll(1, 0).clone()
    for i in range(changed):
        draft[1::2, (37 * i) % vocab] -= 0.001 * (i + 1) if i % 2 else -2.0
    tokens[1::2] = 0 if changed == 1 else 37
    uniform[1::2] = 1 - 2.0 ** -24                    # refused unless p >= q
    got, want = run(target, tokens, uniform, draft, rows)
    assert got == want


@pytest.mark.parametrize("seqs", [2, 40])
@pytest.mark.parametrize("vocab", [1000, 8193, 50_001])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_refused_drafts_of_equal_logits(seqs, vocab, dtype):
    """p = q in every bit: nothing is left of the difference, so p itself is sampled.  The
    drafts are refused since they are outside the vocabulary, or have no mass."""
    rows = [2] * seqs
    target, _, tokens, uniform = make(23, rows, vocab, dtype)
    target[0::4, 5] = float("-inf")
    draft = target.roll(1, 0)
    tokens[1::4], tokens[3::4] = 5, vocab
    got, want = run(target, tokens, uniform, draft, rows)
    assert got == want and got[1] == [0] * seqs


@pytest.mark.parametrize("seqs", [2, 40])
@pytest.mark.parametrize("vocab", [1000, 50_001])
@pytest.mark.parametrize("low", [-590.0, -598.0, -601.0, -646.0, -660.0, -689.0, -700.0])
def test_what_is_left_is_next_to_nothing(seqs, vocab, low):
    """p and q are alike but for logits far below the largest: those have the rest of the mass
    where they are at most 600 below, else nothing is left, and p itself is sampled."""
    rows = [2] * seqs
    target = torch.full((2 * seqs, vocab), low, device="cuda")
    target[:, 3] = 0.0
    draft = torch.full_like(target, low - 5)
    draft[:, 3], draft[:, 7] = 0.0, -580.0
    tokens = ints([7] * (2 * seqs))                   # refused: p(7) is below q(7)
    uniform = torch.rand(2 * seqs, generator=torch.Generator().manual_seed(3)).cuda()
    uniform[1::2] = 0.99
    got, want = run(target, tokens, uniform, draft, rows)
    if low < -600:
        want[0] = [3, -1] * seqs
    assert got == want


@pytest.mark.parametrize("hot", [1e-3, 30.0, float("inf")])
def test_temperatures_far_from_one(hot):
    rows = [3, 1, 4]
    target, draft, tokens, uniform = make(11, rows, 3000, torch.float32)
    got, want = run(target * 100, tokens, uniform, draft * 100, rows, True,
                    torch.full((3,), hot, device="cuda"))
    assert got == want


def test_extreme_logits():
    rows = [2] * 4
    target, draft, tokens, uniform = make(12, rows, 2000, torch.float32)
    target[0], draft[1] = target[0] + 1e6, draft[1] - 1e6
    target[2] *= 1e30
    target[4, 7] = 3e38
    got, want = run(target, tokens, uniform, draft, rows)
    assert got == want


def test_lengths_in_place_and_own_workspace():
    rows = [4, 4, 4]
    target, draft, tokens, uniform = make(13, rows, 4000, torch.bfloat16)
    lens = ints([50, 60, 70])
    ws = wq().verify_workspace(12)
    ws.fill_(0xFF)
    out = (torch.empty(12, dtype=torch.int32, device="cuda"),
           torch.empty(3, dtype=torch.int32, device="cuda"), lens)
    _, accepted, _ = wq().verify_drafts(target, tokens, uniform, draft=draft, seqs=3, logits=True,
                                        seq_lens=lens, out=out, workspace=ws)
    assert lens.tolist() == [50 + 10 * b - 3 + a for b, a in enumerate(accepted.tolist())]


@pytest.mark.parametrize("seqs", [3, 40])
@pytest.mark.parametrize("logits", [True, False])
def test_sequences_without_rows_alone(seqs, logits):
    """A padded batch of which no sequence has rows: what follows on the stream finds the call
    finished."""
    target, draft, tokens, uniform = make(15, [1] * 8, 3000, torch.float32)
    ws, starts = wq().verify_workspace(8), ints([0] * (seqs + 1))
    for i in range(20):
        lens = torch.arange(i, i + seqs, dtype=torch.int32, device="cuda")
        out = tuple(torch.full((n,), 77, dtype=torch.int32, device="cuda")
                    for n in (8, seqs, seqs))
        wq().verify_drafts(target, tokens, uniform, draft, row_starts=starts, logits=logits,
                           seq_lens=lens, out=out, workspace=ws)
        copies = [x.clone() for x in out]
        for x in out:
            x.fill_(5)
        assert copies[0].eq(77).all() and copies[1].eq(0).all() and copies[2].equal(lens)
        assert all(x.eq(5).all() for x in out)
    assert wq().get_device_error() == 0


def test_bad_row_starts_are_recorded():
    rows = [2, 2, 2]
    target, draft, tokens, uniform = make(14, rows, 600, torch.float32)
    good = wq().verify_drafts(target, tokens, uniform, draft=draft, row_starts=ints([0, 2, 4, 6]),
                              logits=True)
    for starts in ([0, 2, 4, 9], [0, 2, 4, 1]):
        got = wq().verify_drafts(target, tokens, uniform, draft=draft, row_starts=ints(starts),
                                 logits=True)
        assert wq().get_device_error() == 1
        assert torch.equal(got[0][:4], good[0][:4])


def test_streams_and_a_captured_call():
    rows = [5] * 8
    cases = [make(20 + i, rows, 20_000, torch.float32) for i in range(3)]
    static = [x.clone() for x in cases[0]]
    ws = wq().verify_workspace(40)
    out = (torch.empty(40, dtype=torch.int32, device="cuda"),
           torch.empty(8, dtype=torch.int32, device="cuda"), None)

    def call():
        wq().verify_drafts(static[0], static[2], static[3], draft=static[1], seqs=8, logits=True,
                           out=out, workspace=ws)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        call()
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for c in cases:
        for s, x in zip(static, c):
            s.copy_(x)
        graph.replay()
        want = wq().verify_drafts(c[0], c[2], c[3], draft=c[1], seqs=8, logits=True)
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_refusals_of_the_binding():
    target, draft, tokens, uniform = make(1, [2, 2], 100, torch.float32)
    ok = dict(target=target, tokens=tokens, uniform=uniform, draft=draft, seqs=2, logits=True)
    wq().verify_drafts(**ok)
    for bad in (dict(target=target.half()), dict(target=target[0]), dict(target=target.cpu()),
                dict(draft=draft.to(torch.bfloat16)), dict(draft=draft[:3]),
                dict(draft=draft.T.contiguous().T), dict(tokens=tokens.long()),
                dict(tokens=tokens[:3]), dict(uniform=uniform.double()), dict(seqs=None),
                dict(temperature=uniform), dict(seq_lens=tokens),
                dict(seq_lens=tokens[:2], out=(tokens, tokens[:2], None)),
                dict(workspace=torch.empty(4096, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            wq().verify_drafts(**{**ok, **bad})
    with pytest.raises(wq().WQError):
        wq().verify_drafts(**{**ok, "seqs": 3})
    with pytest.raises(wq().WQError):
        wq().verify_drafts(**{**ok, "workspace": torch.empty(16, dtype=torch.uint8, device="cuda")})
