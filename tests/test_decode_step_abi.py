"""The entry points around the cached attention on the host (no GPU): rotary
positions, chosen pages, verification of drafts.  The structs match the header,
frequencies follow their formulas, and bad arguments are refused before any
device work."""
import ctypes
import math
import os
import subprocess

import pytest

import w4a16_decode_matmul_b200 as wq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED, ALIGNMENT = 1, 2, 3
STRUCTS = {"wq_kv4_bounds": wq._KV4BoundsStruct, "wq_kv4_selection": wq._KV4SelectionStruct,
           "wq_rotary_spec": wq._RotarySpecStruct, "wq_verification": wq._VerificationStruct}


def test_structs_match_the_header(tmp_path):
    body = "".join(f'printf("%zu\\n", sizeof({n}));\n' + "".join(
        f'printf("%zu\\n", offsetof({n}, {f}));\n' for f, _ in s._fields_)
        for n, s in STRUCTS.items())
    src = tmp_path / "s.c"
    src.write_text(f'#include <stdio.h>\n#include "wq.h"\nint main(void) {{\n{body}return 0; }}\n')
    exe = tmp_path / "s"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                   check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True,
                                          check=True).stdout.split()]
    want = []
    for s in STRUCTS.values():
        want += [ctypes.sizeof(s)] + [getattr(s, f).offset for f, _ in s._fields_]
    assert got == want


def test_packed_structs_match_the_declared_ones():
    for pack, struct, values in (
            (wq._pack_kv4_bounds, wq._KV4BoundsStruct, (0x10, 0x20)),
            (wq._pack_kv4_selection, wq._KV4SelectionStruct, (64, 1, 2, 0x10, 0x20)),
            (wq._pack_rotary_spec, wq._RotarySpecStruct, (0x10, 128, 1, 1.25)),
            (wq._pack_verification, wq._VerificationStruct,
             (5, 2, 1000, 1, 1, 0x10, 0x20, 1 << 33, 0x30, 1 << 34, *range(0x40, 0x47)))):
        assert pack(*values) == bytes(struct(*values))


# ------------------------------------------------------------------ frequencies

def test_frequencies():
    dim, base = 96, 5e5
    plain = [base ** (-2 * i / dim) for i in range(dim // 2)]

    def close(got, want):
        assert got.dtype.itemsize == 4 and len(got) == len(want)
        for g, w in zip(got.tolist(), want):
            assert abs(g - w) <= 2.0 ** -24 * 1.0001 * w

    close(wq.rotary_frequencies(dim, base), plain)
    close(wq.rotary_frequencies(dim, base, "linear", factor=4), [f / 4 for f in plain])
    close(wq.rotary_frequencies(dim, base, "base", factor=8),
          [(base * 8 ** (dim / (dim - 2))) ** (-2 * i / dim) for i in range(dim // 2)])
    got = wq.rotary_frequencies(dim, base, "base", factor=8).tolist()
    assert got[0] == 1 and abs(got[-1] * 8 / plain[-1] - 1) < 1e-6
    context, low, high = 8192, 1, 4
    keep = [min(1, max(0, (context * f / (2 * math.pi) - low) / (high - low))) for f in plain]
    assert 0 in keep and 1 in keep and any(0 < k < 1 for k in keep)
    close(wq.rotary_frequencies(dim, base, "parts", 16, context, low, high),
          [f * (k + (1 - k) / 16) for f, k in zip(plain, keep)])
    close(wq.rotary_frequencies(2), [1.0])


@pytest.mark.parametrize("kw", [
    dict(dim=0), dict(dim=7), dict(dim=-2), dict(base=0.0), dict(base=float("nan")),
    dict(base=float("inf")), dict(scaling="linear", factor=0.5),
    dict(scaling="linear", factor=float("nan")), dict(scaling="base", factor=2.0, dim=2),
    dict(scaling="parts", factor=2.0), dict(scaling="parts", factor=2.0, context=10, low=2, high=2),
    dict(scaling="parts", factor=2.0, context=10, low=1, high=float("inf"))])
def test_frequency_refusals(kw):
    with pytest.raises(wq.WQError) as e:
        wq.rotary_frequencies(**{"dim": 64, **kw})
    assert e.value.status == INVALID
    with pytest.raises(ValueError):
        wq.rotary_frequencies(64, scaling="other")


def test_frequencies_need_a_buffer_and_a_known_scaling():
    f = (ctypes.c_float * 4)()
    assert wq.lib.wq_rotary_frequencies(8, 1e4, 0, 1.0, 0.0, 0.0, 0.0, None) == INVALID
    assert wq.lib.wq_rotary_frequencies(8, 1e4, 4, 1.0, 0.0, 0.0, 0.0, f) == INVALID
    assert wq.lib.wq_rotary_frequencies(8, 1e4, -1, 1.0, 0.0, 0.0, 0.0, f) == INVALID


# --------------------------------------------------------------------- refusals

@pytest.fixture(scope="module")
def base():
    buf = ctypes.create_string_buffer(4096)
    yield (ctypes.addressof(buf) + 15) // 16 * 16


def make(struct, defaults, **kw):
    v = {**defaults, **kw}
    return struct(*(v[f] for f, _ in struct._fields_))


def cache(p, **kw):
    return make(wq._KV4CacheStruct, dict(k_codes=p, k_meta=p, v_codes=p, v_meta=p, pages=4,
                                         page_size=16, kv_heads=2, head_dim=64, group=32), **kw)


def batch(p, **kw):
    return make(wq._KV4BatchStruct, dict(seqs=2, rows=4, row_starts=None, seq_lens=p,
                                         page_table=p, table_width=2, table_stride=2,
                                         max_rows=0), **kw)


def bounds(p, **kw):
    return make(wq._KV4BoundsStruct, dict(codes=p, grid=p), **kw)


def selection(p, **kw):
    return make(wq._KV4SelectionStruct, dict(max_pages=4, first=1, last=2, lists=p, lens=p), **kw)


def spec(p, **kw):
    return make(wq._RotarySpecStruct, dict(freqs=p, dim=32, interleaved=0, amplitude=1.0), **kw)


def verification(p, **kw):
    return make(wq._VerificationStruct, dict(
        rows=4, seqs=2, vocab=100, dtype=0, flags=1, row_starts=None, target=p, target_stride=100,
        draft=p, draft_stride=100, tokens=p, uniform=p, temperature=p, seq_lens=p, out_tokens=p,
        accepted=p, out_lens=p), **kw)


def rotary(p, s=None, **kw):
    a = {**dict(x=p, xs=256, rows=3, heads=4, d=64, pos=p, spec=ctypes.byref(s or spec(p)),
                flags=0, y=p, ys=256, stream=None), **kw}
    return wq.lib.wq_rotary(*a.values())


def write(p, s=None, c=None, b=None, **kw):
    a = {**dict(q=p, qs=256, heads=4, o=p, os=256, k=p, ks=128, v=p, vs=128,
                spec=ctypes.byref(s or spec(p)), pos=None, c=ctypes.byref(c or cache(p)),
                b=ctypes.byref(b or batch(p)), stream=None), **kw}
    return wq.lib.wq_kv4_write_rotary(*a.values())


def paged(p, c=None, b=None, n=None, s=None, **kw):
    """(update_bounds, select, attention_pages, sparse_attention)."""
    c, b, n, s = c or cache(p), b or batch(p), n or bounds(p), s or selection(p)
    a = {**dict(q=p, qs=256, heads=4, scale=0.1, o=p, os=256, w=p,
                wn=wq.lib.wq_kv4_attention_workspace_bytes(), rows=4), **kw}
    cr, br, nr, sr = (ctypes.byref(x) for x in (c, b, n, s))
    q, tail = (a["q"], a["qs"], a["heads"]), (a["scale"], a["o"], a["os"], a["w"], a["wn"], None)
    return (wq.lib.wq_kv4_update_bounds(cr, nr, br, None),
            wq.lib.wq_kv4_select(*q, cr, nr, br, sr, None),
            wq.lib.wq_kv4_attention_pages(*q, cr, a["rows"], sr, *tail),
            wq.lib.wq_kv4_sparse_attention(*q, cr, nr, br, sr, *tail))


def verify(p, ws=None, n=None, **kw):
    v = verification(p, **kw)
    return wq.lib.wq_verify_drafts(ctypes.byref(v), p if ws is None else ws,
                                   wq.lib.wq_verify_workspace_bytes(4) if n is None else n, None)


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), INVALID), (dict(heads=0), INVALID), (dict(heads=(1 << 20) + 1), INVALID),
    (dict(d=0), INVALID), (dict(d=60), UNSUPPORTED), (dict(d=520), UNSUPPORTED),
    (dict(flags=2), INVALID), (dict(pos=None), INVALID), (dict(x=None), INVALID),
    (dict(y=None), INVALID), (dict(xs=248), INVALID), (dict(ys=260), ALIGNMENT),
    (dict(ys=264), INVALID), (dict(spec=None), INVALID)])
def test_rotary_refusals(base, change, status):
    assert rotary(base, **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(freqs=None), INVALID), (dict(dim=0), INVALID), (dict(dim=31), INVALID),
    (dict(dim=66), INVALID), (dict(interleaved=2), INVALID),
    (dict(amplitude=float("inf")), INVALID), (dict(amplitude=float("nan")), INVALID)])
def test_rotary_spec_refusals(base, change, status):
    assert rotary(base, spec(base, **change)) == status
    assert write(base, spec(base, **change)) == status


def test_rotary_alignment_and_no_rows(base):
    assert rotary(base, x=base + 8) == ALIGNMENT and rotary(base, y=base + 2) == ALIGNMENT
    assert rotary(base, pos=base + 2) == ALIGNMENT
    assert rotary(base, spec(base, freqs=base + 4)) == ALIGNMENT
    assert rotary(base, rows=0, x=None, y=None, pos=None) == 0
    assert write(base, q=base + 8) == ALIGNMENT and write(base, pos=base + 1) == ALIGNMENT
    assert write(base, spec(base, freqs=base + 8)) == ALIGNMENT
    assert write(base, b=batch(base, rows=0, seqs=0), q=None, k=None) == 0


@pytest.mark.parametrize("change,status", [
    (dict(heads=-1), INVALID), (dict(q=None), INVALID), (dict(o=None), INVALID),
    (dict(os=264), INVALID), (dict(qs=128), INVALID), (dict(k=None), INVALID),
    (dict(v=None), INVALID), (dict(ks=64), INVALID), (dict(vs=132), ALIGNMENT)])
def test_write_rotary_refusals(base, change, status):
    assert write(base, **change) == status


def test_write_rotary_refuses_what_its_parts_refuse(base):
    for dim in (8, 24, 40):
        assert write(base, spec(base, dim=dim)) == UNSUPPORTED
    assert write(base, c=cache(base, page_size=48)) == UNSUPPORTED
    assert write(base, c=cache(base, v_meta=None)) == INVALID
    for kw in (dict(rows=-1), dict(seqs=0), dict(seqs=3), dict(seq_lens=None),
               dict(table_stride=1), dict(rows=1 << 30)):
        assert write(base, b=batch(base, **kw)) == INVALID


def test_bounds_refusals(base):
    for kw in (dict(codes=None), dict(grid=None)):
        assert [paged(base, n=bounds(base, **kw))[i] for i in (0, 1, 3)] == [INVALID] * 3
    for kw in (dict(codes=base + 8), dict(grid=base + 4)):
        assert [paged(base, n=bounds(base, **kw))[i] for i in (0, 1, 3)] == [ALIGNMENT] * 3


def test_selection_refusals(base):
    for kw in (dict(lists=None), dict(lens=None), dict(max_pages=0)):
        assert paged(base, s=selection(base, **kw))[1:] == (INVALID,) * 3
    for kw in (dict(lists=base + 8), dict(lens=base + 4)):
        assert paged(base, s=selection(base, **kw))[1:] == (ALIGNMENT,) * 3
    for kw in (dict(first=-1), dict(last=0), dict(first=3), dict(first=2 ** 31 - 1, last=2 ** 31 - 1)):
        got = paged(base, s=selection(base, **kw))
        assert got[1] == INVALID and got[3] == INVALID
    got = paged(base, b=batch(base, table_width=53249, table_stride=53249))
    assert got[1] == UNSUPPORTED and got[3] == UNSUPPORTED
    got = paged(base, heads=514, qs=514 * 64, os=514 * 64)
    assert got[1] == UNSUPPORTED and got[3] == UNSUPPORTED


@pytest.mark.parametrize("change", [
    dict(heads=0), dict(heads=3), dict(q=None), dict(qs=128)])
def test_query_refusals(base, change):
    assert paged(base, **change)[1:] == (INVALID,) * 3


@pytest.mark.parametrize("change,status", [
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(o=None), INVALID), (dict(os=260), ALIGNMENT), (dict(w=None), INVALID),
    (dict(wn=16), INVALID)])
def test_paged_attention_refusals(base, change, status):
    got = paged(base, **change)
    assert got[2] == status and got[3] == status


def test_paged_batch_refusals(base):
    for kw in (dict(rows=-1), dict(seqs=0), dict(seqs=3), dict(seq_lens=None),
               dict(page_table=None), dict(table_width=0), dict(max_rows=-1)):
        got = paged(base, b=batch(base, **kw))
        assert [got[i] for i in (0, 1, 3)] == [INVALID] * 3
    assert paged(base, rows=-1)[2] == INVALID
    assert set(paged(base, c=cache(base, head_dim=96))) == {UNSUPPORTED}
    none = batch(base, rows=0, seqs=0, seq_lens=None, page_table=None)
    assert set(paged(base, b=none, rows=0, n=bounds(base, codes=None))) == {0}


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), INVALID), (dict(seqs=0), INVALID), (dict(seqs=3), INVALID),
    (dict(vocab=0), INVALID), (dict(dtype=2), INVALID), (dict(flags=2), INVALID),
    (dict(target=None), INVALID), (dict(tokens=None), INVALID), (dict(uniform=None), INVALID),
    (dict(out_tokens=None), INVALID), (dict(accepted=None), INVALID),
    (dict(seq_lens=None), INVALID), (dict(flags=0), INVALID), (dict(target_stride=99), INVALID),
    (dict(draft_stride=99), INVALID)])
def test_verify_refusals(base, change, status):
    assert verify(base, **change) == status


def test_verify_alignment_and_workspace(base):
    for f in ("target", "draft"):
        assert verify(base, **{f: base + 8}) == ALIGNMENT
    for f in ("tokens", "uniform", "temperature", "seq_lens", "out_tokens", "accepted",
              "out_lens", "row_starts"):
        assert verify(base, **{f: base + 2}) == ALIGNMENT
    assert verify(base, ws=base + 8) == ALIGNMENT
    assert verify(base, ws=0) == INVALID
    n = wq.lib.wq_verify_workspace_bytes(4)
    assert n > 0 and verify(base, n=n - 1) == INVALID
    assert wq.lib.wq_verify_workspace_bytes(0) == wq.lib.wq_verify_workspace_bytes(1 << 31) == 0
    assert verify(base, rows=0, seqs=0, target=None) == 0
