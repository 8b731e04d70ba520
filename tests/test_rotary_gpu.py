"""Rotary positions on the B200, against rotations in binary64 (angles in
extended precision); on the way into the 4-bit cache the codes are bit for bit
those of the oracle's quantizer for the turned keys."""
import numpy as np
import pytest
import torch

from tests import kv4_ref as ref
from tests.gpu_util import wq
from tests.test_kv4_gpu import assert_cache, expect_written, images, ints, new_cache, starts_of

pytestmark = pytest.mark.gpu


def turns(positions, freqs, amplitude):
    """Cosines and sines [n, dim/2] as the library defines them: of the exact
    product, rounded to binary32."""
    a = np.asarray(positions, dtype=np.longdouble)[:, None] * freqs.numpy().astype(np.longdouble)
    amp = np.float32(amplitude).astype(np.float64)
    return [(amp * f(a).astype(np.float64)).astype(np.float32).astype(np.float64)
            for f in (np.cos, np.sin)]


def turned(x, c, s, interleaved):
    """x [n, H, D] float64 -> turned, float64 (products of bfloat16 and binary32 are exact,
    their sum is rounded once), and the sum of the products' magnitudes."""
    n = c.shape[1]
    y, mag = x.copy(), np.abs(x)
    one, two = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else \
        (slice(0, n), slice(n, 2 * n))
    a, b, c, s = x[..., one], x[..., two], c[:, None], s[:, None]
    y[..., one], y[..., two] = a * c - b * s, b * c + a * s
    mag[..., one] = np.abs(a * c) + np.abs(b * s)
    mag[..., two] = np.abs(b * c) + np.abs(a * s)
    return y, mag


def check(got, x, positions, freqs, interleaved, amplitude=1.0, inverse=False):
    c, s = turns(positions, freqs, amplitude)
    y, mag = turned(x.double().cpu().numpy(), c, -s if inverse else s, interleaved)
    # binary64 of the angle: half a step of the product, which the sine and cosine of its
    # argument pass on, and a few of their own; then binary32's rounding of c and s (the
    # reference's may fall to the other side: 2^-23 together), a product and a sum (2^-24
    # each), bfloat16's half step
    angle = np.abs(np.asarray(positions, dtype=np.float64))[:, None] * freqs.double().numpy()
    slack = np.zeros_like(x[:, :1].double().cpu().numpy())
    each = 2.0 ** -53 * angle * amplitude
    n = c.shape[1]
    if interleaved:
        slack[:, 0, 0:2 * n:2] = slack[:, 0, 1:2 * n:2] = each
    else:
        slack[:, 0, :n] = slack[:, 0, n:2 * n] = each
    top = np.abs(x.double().cpu().numpy()).max(-1, keepdims=True)
    tol = 2.0 ** -8 * np.abs(y) + 1.01 * (2.0 ** -22 * mag + 2 * slack * top) + 2.0 ** -133
    err = np.abs(got.double().cpu().numpy() - y)
    assert np.isfinite(err).all() and (err <= tol).all(), float((err / tol).max())


CASES = [  # rows, heads, head_dim, dim, interleaved
    (1, 1, 8, 2, False), (1, 40, 128, 128, False), (1, 40, 128, 128, True), (3, 5, 64, 64, False),
    (7, 3, 80, 34, False), (7, 3, 80, 34, True), (2, 9, 96, 20, True), (2, 9, 96, 20, False),
    (301, 8, 128, 64, False), (301, 8, 128, 66, False), (150, 1, 256, 256, True),
    (40, 2, 512, 512, False), (3000, 3, 80, 34, False), (2500, 5, 64, 50, True), (1, 300, 512, 510, False), (40, 2, 512, 16, True), (1000, 40, 64, 64, True), (5, 200, 64, 48, False),
]


@pytest.mark.parametrize("rows,heads,d,dim,interleaved", CASES)
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("form", ["new", "in place", "strided"])
def test_rotary(rows, heads, d, dim, interleaved, inverse, form):
    g = torch.Generator().manual_seed(rows + d + dim)
    wide = torch.randn(rows, heads + 3, d, generator=g).to(torch.bfloat16).cuda()
    x = wide[:, 1:1 + heads] if form != "new" else wide[:, :heads].contiguous()
    positions = torch.randint(0, 100_000, (rows,), generator=g).to(torch.int32)
    freqs = wq().rotary_frequencies(dim)
    rot = wq().Rotary(freqs.cuda(), interleaved, 1.25)
    before, was = wide.clone(), x.clone()
    out = None
    if form == "in place":
        out = x
    elif form == "strided":
        frame = torch.full((rows, heads + 2, d), 7.0, dtype=torch.bfloat16, device="cuda")
        out = frame[:, 2:]
    got = wq().rotary(x, positions.cuda(), rot, inverse=inverse, out=out)
    check(got, was, positions, freqs, interleaved, 1.25, inverse)
    if form == "in place":     # the columns beside it are as they were
        assert torch.equal(wide[:, 0], before[:, 0])
        assert torch.equal(wide[:, 1 + heads:], before[:, 1 + heads:])
    else:
        assert torch.equal(wide, before)
    if form == "strided":
        assert (frame[:, :2] == 7).all()
    # what is not turned is copied bit for bit
    assert torch.equal(got[..., dim:], was[..., dim:])


@pytest.mark.parametrize("interleaved", [False, True])
def test_positions_of_every_size(interleaved):
    positions = [0, 1, -1, 2 ** 20, 1_000_003, -(2 ** 24) - 1, 2 ** 29, 2 ** 31 - 1, -(2 ** 31)]
    g = torch.Generator().manual_seed(1)
    x = torch.randn(len(positions), 2, 64, generator=g).to(torch.bfloat16)
    freqs = wq().rotary_frequencies(64)
    freqs[3] = 0.0
    got = wq().rotary(x.cuda(), ints(positions), wq().Rotary(freqs.cuda(), interleaved))
    check(got, x, positions, freqs, interleaved)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim", [64, 32, 22])
def test_gradient_is_the_transpose(interleaved, dim):
    """Column j of the rotation's matrix is the rotation of unit vector j, row j the
    inverse's: differences of a linear map are exact."""
    d, position = 64, 12_345
    rot = wq().Rotary(wq().rotary_frequencies(dim).cuda(), interleaved, 0.75)
    unit = torch.eye(d).to(torch.bfloat16).view(d, 1, d).cuda()
    at = torch.full((d,), position, dtype=torch.int32, device="cuda")
    forward = wq().rotary(unit, at, rot)[:, 0]
    back = wq().rotary(unit, at, rot, inverse=True)[:, 0]
    assert torch.equal(forward, back.T)
    # and the gradient of <w, R x> against autograd over the formula
    g = torch.Generator().manual_seed(3)
    w = torch.randn(d, 1, d, generator=g).to(torch.bfloat16)
    x = torch.randn(d, 1, d, generator=g, dtype=torch.float64, requires_grad=True)
    c, s = (torch.tensor(t) for t in turns([position] * d, rot.freqs.cpu(), 0.75))
    n = dim // 2
    a, b = (x[..., 0:dim:2], x[..., 1:dim:2]) if interleaved else (x[..., :n], x[..., n:dim])
    ya, yb = a * c[:, None] - b * s[:, None], b * c[:, None] + a * s[:, None]
    wa, wb = (w[..., 0:dim:2], w[..., 1:dim:2]) if interleaved else (w[..., :n], w[..., n:dim])
    ((ya * wa.double()).sum() + (yb * wb.double()).sum()
     + (x[..., dim:] * w[..., dim:].double()).sum()).backward()
    got = wq().rotary(w.cuda(), at, rot, inverse=True).double().cpu()
    tol = 2.0 ** -8 * x.grad.abs() + 2.0 ** -20 * w.abs().max().double()
    assert ((got - x.grad).abs() <= tol).all()


def test_infinities_and_nan_stay_in_their_pair():
    x = torch.ones(2, 1, 16, dtype=torch.bfloat16)
    x[0, 0, 3], x[1, 0, 12] = float("inf"), float("nan")
    rot = wq().Rotary(wq().rotary_frequencies(16).cuda())
    got = wq().rotary(x.cuda(), ints([5, 7]), rot).float().cpu()
    bad = ~torch.isfinite(got)
    assert bad[0, 0].nonzero().flatten().tolist() == [3, 11]
    assert bad[1, 0].nonzero().flatten().tolist() == [4, 12]


def test_refusals_of_the_binding():
    rot = wq().Rotary(wq().rotary_frequencies(64).cuda())
    x, at = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda"), ints([0, 1, 2])
    for bad in (x.float(), x[0], x.transpose(0, 1).transpose(1, 2), x.cpu()):
        with pytest.raises(ValueError):
            wq().rotary(bad, at, rot)
    for p in (at[:2], at.long(), at.cpu(), None):
        with pytest.raises(ValueError):
            wq().rotary(x, p, rot)
    with pytest.raises(ValueError):
        wq().rotary(x, at, rot, out=x[:2])
    with pytest.raises(ValueError):
        wq().Rotary(rot.freqs.double())
    with pytest.raises(wq().WQError):
        wq().rotary(x[..., :32].contiguous(), at, rot)          # dim above head_dim
    assert wq().rotary(x[:0], at[:0], rot).shape == (0, 2, 64)


# ------------------------------------------------------------ into the cache

def expect(k, positions, rot, held, x, want, cache):
    c, s = turns(positions, rot.freqs.cpu(), rot.amplitude)
    y, _ = turned(k.double().cpu().numpy(), c, s, rot.interleaved)
    with np.errstate(over="ignore"):
        y = torch.tensor(y).to(torch.float32).to(torch.bfloat16)
    expect_written(cache, y, held, "k", *want["k"])
    expect_written(cache, x.cpu(), held, "v", *want["v"])
    return y


@pytest.mark.parametrize("d,group", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,q_heads,heads,page,lens,rows", [
    (64, 1, 1, 16, [1], [1]),
    (64, 32, 8, 64, [777], [1]),
    (16, 6, 3, 32, [5, 40, 33], [5, 7, 33]),
    (48, 10, 5, 16, [100, 0, 17, 3], [50, 0, 17, 6]),     # no rows; more rows than tokens
    (32, 38, 19, 64, [70, 300], [3, 2]),                  # three warps' keys and values
    (64, 4, 2, 128, [300] * 40, [2] * 40),
])
def test_write_rotary(d, group, interleaved, dim, q_heads, heads, page, lens, rows):
    if d == 128:
        dim *= 2
    table, pages = ref.random_batch(d + group, lens, page)
    cache = new_cache(pages, heads, d, page, group)
    n, behind = sum(rows), 3
    qkv = torch.cat((ref.keys(2, n + behind, q_heads + heads, d),
                     ref.keys(3, n + behind, heads, d)), 1).cuda()
    qkv[n:] = float("nan")
    q, k, v = qkv[:, :q_heads], qkv[:, q_heads:q_heads + heads], qkv[:, q_heads + heads:]
    rot = wq().Rotary(wq().rotary_frequencies(dim, 500.0).cuda(), interleaved, 1.1)
    want = images(cache)
    held, _ = ref.places(lens, rows, table, page)
    positions = [m - t + i for m, t in zip(lens, rows) for i in range(t)]
    expect(k[:n], positions, rot, held, v[:n], want, cache)
    out = torch.full((n + behind, q_heads, d), 7.0, dtype=torch.bfloat16, device="cuda")
    before = qkv.clone()
    got = wq().kv4_write_rotary(q, k, v, cache, rot, ints(lens), ints(table), ints(starts_of(rows)),
                                out=out)
    assert got is out
    assert_cache(cache, want)
    check(out[:n], q[:n], positions, rot.freqs.cpu(), interleaved, 1.1)
    assert (out[n:] == 7).all() and torch.equal(qkv[:n], before[:n])
    assert wq().get_device_error() == 0


@pytest.mark.parametrize("interleaved", [False, True])
def test_write_rotary_in_place_and_by_given_positions(interleaved):
    d, heads, page, lens = 128, 2, 16, [40, 9]
    rows, given = [8, 8], [3, 100_000, 7, -5, 0, 1, 2, 9, 50, 51, 2 ** 30, 4, 5, 6, 8, 10]
    table, pages = ref.random_batch(5, lens, page)
    qkv = ref.keys(6, 16, 8, d).cuda()
    rot = wq().Rotary(wq().rotary_frequencies(d).cuda(), interleaved)
    cache = new_cache(pages, heads, d, page, 64)
    want = images(cache)
    held, _ = ref.places(lens, rows, table, page)
    expect(qkv[:, 4:6], given, rot, held, qkv[:, 6:], want, cache)
    was = qkv.clone()
    got = wq().kv4_write_rotary(qkv[:, :4], qkv[:, 4:6], qkv[:, 6:], cache, rot, ints(lens),
                                ints(table), positions=ints(given), out=qkv[:, :4])
    assert_cache(cache, want)
    check(got, was[:, :4], given, rot.freqs.cpu(), interleaved)
    assert torch.equal(qkv[:, 4:], was[:, 4:])
    # keys and values alone
    again = new_cache(pages, heads, d, page, 64)
    assert wq().kv4_write_rotary(None, was[:, 4:6], was[:, 6:], again, rot, ints(lens),
                                 ints(table), positions=ints(given)) is None
    assert_cache(again, want)


def test_write_rotary_keys_of_every_size():
    """Saturating, infinite and tiny keys; positions far out."""
    n, heads, d, page = 64, 2, 128, 64
    g = torch.Generator().manual_seed(9)
    k = ref.keys(4, n, heads, d).float()
    k *= torch.exp2(torch.randint(-30, 18, (n, 1, 1), generator=g).float())
    k[0] = 0
    k[1, :, 5], k[2, 0, 7] = 3e38, -3e38
    k[3] = 2.0 ** -120
    k = k.to(torch.bfloat16)
    table, pages = ref.random_batch(1, [n], page)
    positions = [10_000 * i + 7 for i in range(n)]
    rot = wq().Rotary(wq().rotary_frequencies(d).cuda())
    cache = new_cache(pages, heads, d, page, 64)
    want = images(cache)
    held, _ = ref.places([n], [n], table, page)
    expect(k, positions, rot, held, k, want, cache)
    wq().kv4_write_rotary(None, k.cuda(), k.cuda(), cache, rot, ints([n]), ints(table),
                          positions=ints(positions))
    assert_cache(cache, want)


@pytest.mark.parametrize("rows", [1184, 1185, 2370, 2371, 4801])
@pytest.mark.parametrize("q_heads", [0, 1])
@pytest.mark.parametrize("d", [64, 128])
def test_write_rotary_of_many_rows_with_few_heads(rows, q_heads, d):
    """Several rows a CTA, the last CTA with fewer: fewer shares of work than warps."""
    page = 64
    lens, t = [rows - 300, 400], [rows - 300, 300]
    table, pages = ref.random_batch(7, lens, page)
    qkv = ref.keys(5, rows, q_heads + 2, d).cuda()
    rot = wq().Rotary(wq().rotary_frequencies(d).cuda())
    cache = new_cache(pages, 1, d, page, 64)
    want = images(cache)
    held, _ = ref.places(lens, t, table, page)
    positions = [m - n + i for m, n in zip(lens, t) for i in range(n)]
    expect(qkv[:, q_heads:-1], positions, rot, held, qkv[:, -1:], want, cache)
    got = wq().kv4_write_rotary(qkv[:, :q_heads] if q_heads else None, qkv[:, q_heads:-1],
                                qkv[:, -1:], cache, rot, ints(lens), ints(table),
                                ints(starts_of(t)))
    assert_cache(cache, want)
    if q_heads:
        check(got, qkv[:, :q_heads], positions, rot.freqs.cpu(), False)


def test_write_rotary_matches_a_write_of_unturned_keys_at_position_zero():
    n, heads, d = 5, 4, 64
    k, v = ref.keys(1, n, heads, d).cuda(), ref.keys(2, n, heads, d).cuda()
    table, pages = ref.random_batch(2, [1] * n, 16)
    rot = wq().Rotary(wq().rotary_frequencies(d).cuda())
    a, b = (new_cache(pages, heads, d, 16, 32) for _ in "ab")
    wq().kv4_write(k, v, a, ints([1] * n), ints(table))
    wq().kv4_write_rotary(None, k, v, b, rot, ints([1] * n), ints(table))
    for x, y in ((a.k_codes, b.k_codes), (a.v_codes, b.v_codes)):
        assert torch.equal(x, y)


def test_write_rotary_records_what_is_out_of_bounds():
    """A page outside the cache, a length above the table, row ranges outside the rows: recorded,
    nothing outside the buffers written, the other sequences' rows as ever."""
    heads, d, page, lens, rows = 2, 64, 16, [20, 30, 10], [2, 2, 2]
    table, pages = ref.random_batch(3, lens, page)
    k, v = ref.keys(1, 6, heads, d).cuda(), ref.keys(2, 6, heads, d).cuda()
    rot = wq().Rotary(wq().rotary_frequencies(d).cuda())
    args = (ints(lens), ints(table), ints(starts_of(rows)))
    for change in ("page", "length", "rows"):
        bad = [t.clone() for t in args]
        if change == "page":
            bad[1][1, 29 // page] = pages
        elif change == "length":
            bad[0][1] = page * table.shape[1] + 1
        else:
            bad[2][2] = 7
        cache = new_cache(pages, heads, d, page, 32)
        wq().kv4_write_rotary(k, k, v, cache, rot, *bad)
        assert wq().get_device_error() == 1, change
        good = new_cache(pages, heads, d, page, 32)
        wq().kv4_write_rotary(k, k, v, good, rot, *args)
        assert wq().get_device_error() == 0
        for i in (18, 19):      # the first sequence's rows
            p, slot = int(table[0, i // page]), i % page
            assert torch.equal(cache.k_codes[p, :, slot], good.k_codes[p, :, slot])
