"""The 4-bit key/value cache restated for tests: the quantizer is the CPU
oracle's (the cache quantizes as the asymmetric weights are), the code order
and the attention are written here from their definitions, in binary64."""
from __future__ import annotations

import numpy as np
import torch

import oracle


def to_half(x: torch.Tensor) -> torch.Tensor:
    """What the format quantizes: bfloat16 values taken to binary16."""
    return x.float().clamp(-65504, 65504).to(torch.float16)


def quantize(x: torch.Tensor, group: int):
    """x [n, D] -> codes [n, D] (0..15), scales, zeros [n, D/group] (uint16
    bit patterns), by the oracle."""
    bits = to_half(x).cpu().contiguous().view(torch.int16).numpy().view(np.uint16)
    n, d = bits.shape
    _, packed, scales, zeros = oracle.get().quantize(bits, 4, group, False)
    packed = packed.reshape(n, d // 2)
    return (np.stack((packed & 15, packed >> 4), -1).reshape(n, d),
            scales.reshape(n, -1), zeros.reshape(n, -1))


def pack(codes: np.ndarray, kind: str) -> np.ndarray:
    """codes [n, D] -> the bytes of a key ("k") or value ("v") row."""
    n, d = codes.shape
    b = (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)
    unit = 4 if kind == "k" else 2
    return np.ascontiguousarray(
        b.reshape(n, d // 32, 16 // unit, unit).transpose(0, 2, 1, 3)).reshape(n, d // 2)


def unpack(b: np.ndarray, kind: str) -> np.ndarray:
    """The inverse of ``pack``, over any leading dimensions."""
    lead, half = b.shape[:-1], b.shape[-1]
    unit = 4 if kind == "k" else 2
    r = np.swapaxes(b.reshape(*lead, 16 // unit, half // 16, unit), -3, -2).reshape(*lead, half)
    return np.stack((r & 15, r >> 4), -1).reshape(*lead, 2 * half)


def places(lens, rows, table, page, starts=None):
    """(row, sequence, position, page, slot) of every row that holds a token,
    and the rows of a sequence that hold none."""
    held, empty, at = [], [], 0
    for b, (n, t) in enumerate(zip(lens, rows)):
        first = at if starts is None else starts[b]
        for i in range(t):
            pos = n - t + i
            if pos < 0:
                empty.append(first + i)
            else:
                held.append((first + i, b, pos, int(table[b][pos // page]), pos % page))
        at += t
    return held, empty


def sequence_values(codes, meta, table_row, n, page, kind):
    """(codes [n, H, D], scale, zero [n, H, D/G]) of the first n tokens, float64."""
    ids = np.asarray(table_row[:(n + page - 1) // page], dtype=np.int64)
    c = unpack(codes[ids], kind)                    # [P, H, page, D]
    m = meta[ids].astype(np.float64)                # [P, H, page, D/G, 2]
    c = c.transpose(0, 2, 1, 3).reshape(-1, *c.shape[1:2], c.shape[3])[:n]
    m = m.transpose(0, 2, 1, 3, 4).reshape(-1, *m.shape[1:2], *m.shape[3:])[:n]
    return c.astype(np.float64), m[..., 0], m[..., 1]


def attention(q: np.ndarray, k, v, n: int, scale: float, few: bool = True):
    """One sequence: q [T, Hq, D] float64, k and v as ``sequence_values``
    gives them.  Returns the output [T, Hq, D] and the bound on the error of a
    computation that rounds its weights (``few``), or its weights, keys and
    values (not ``few``), to binary16."""
    (kc, ks, kz), (vc, vs, vz) = k, v
    t, hq, d = q.shape
    h, ng = ks.shape[1], ks.shape[2]
    r, g = hq // h, d // ng
    kh = ((kc.reshape(n, h, ng, g) - kz[..., None]) * ks[..., None]).reshape(n, h, d)
    vh = ((vc.reshape(n, h, ng, g) - vz[..., None]) * vs[..., None]).reshape(n, h, d)
    out, bound = np.zeros((t, hq, d)), np.zeros((t, hq, d))
    for j in range(hq):
        a = j // r
        for i in range(t):
            seen = n - t + i + 1
            if seen <= 0:
                continue
            s = scale * (kh[:seen, a] @ q[i, j])
            p = np.exp(s - s.max())
            p /= p.sum()
            out[i, j] = p @ vh[:seen, a]
            # error of a score: the codes are exact, each of the at most 16
            # binary32 additions and products of a score is off by 2^-23 of
            # the magnitudes added up (tensor cores truncate)
            mags = (ks[:seen, a] * 16 * np.abs(q[i, j]).reshape(ng, g).sum(-1)).sum(-1).max()
            e = 16 * 2.0 ** -23 * abs(scale) * mags + 2.0 ** -21
            if few:
                # weights: half a step of binary16 (2^-11) each, times |u - 8|
                # <= 8; those below binary16's normal range are off by 2^-25
                # where the largest is at least 1; score errors move every
                # weight (twice: numerator and sum)
                w8 = np.repeat((p[:, None] * vs[:seen, a]).sum(0) * 8, g)
                tiny = seen * 8 * 2.0 ** -25 * vs[:seen, a].max()
                wabs = p @ (np.repeat(vs[:seen, a], g, -1) * 16)
                bound[i, j] = 2.0 ** -11 * w8 + tiny + 2 * e * wabs
            else:
                # half a step of each key moves the scores, of each weight and
                # value the sum
                e += abs(scale) * 2.0 ** -11 * (np.abs(kh[:seen, a]) @ np.abs(q[i, j])).max()
                wabs = p @ np.abs(vh[:seen, a])
                tiny = seen * 2.0 ** -25 * np.abs(vh[:seen, a]).max()
                bound[i, j] = 2.0 ** -10 * 1.01 * wabs + tiny + 2 * np.expm1(e) * wabs
    return out, bound


def check(got: torch.Tensor, ref: np.ndarray, bound: np.ndarray):
    """got bfloat16 against the reference: its half step on top of the bound."""
    y = got.detach().float().cpu().numpy().astype(np.float64)
    assert np.isfinite(y).all(), "non-finite outputs"
    tol = 2.0 ** -8 * (np.abs(ref) + bound) + bound
    err = np.abs(y - ref)
    bad = err > tol
    assert not bad.any(), (f"{int(bad.sum())} of {y.size} outputs out of tolerance, worst err/tol "
                           f"{float(np.max(err / np.maximum(tol, 1e-300)))}, first at "
                           f"{np.argwhere(bad)[0].tolist()}")


def random_batch(seed, lens, page, extra=3):
    """A page table in random page order; (table [B, width] int32, pages)."""
    rng = np.random.default_rng(seed)
    need = [(n + page - 1) // page for n in lens]
    pages = sum(need) + extra
    order = rng.permutation(pages)
    table = np.full((len(lens), max(max(need), 1) + 1), -7, dtype=np.int32)   # never used
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, pages


def keys(seed, n, heads, d, strong=8.0):
    """bfloat16 rows [n, heads, d] with a few strong channels."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, heads, d, generator=g)
    x[..., torch.randperm(d, generator=g)[:max(1, d // 32)]] *= strong
    return x.to(torch.bfloat16)


