"""The 4-bit cache's entry points on the host (no GPU): the structs match the
header, the tests' own packing is its inverse, and bad arguments are refused
before any device work."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

import w4a16_decode_matmul_b200 as wq
from tests import kv4_ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED, ALIGNMENT = 1, 2, 3


def test_structs_match_the_header(tmp_path):
    fields = {"wq_kv4_cache": wq._KV4CacheStruct, "wq_kv4_batch": wq._KV4BatchStruct}
    body = "".join(f'printf("%zu\\n", sizeof({n}));\n' + "".join(
        f'printf("%zu\\n", offsetof({n}, {f}));\n' for f, _ in s._fields_)
        for n, s in fields.items())
    src = tmp_path / "s.c"
    src.write_text(f'#include <stdio.h>\n#include "wq.h"\nint main(void) {{\n{body}return 0; }}\n')
    exe = tmp_path / "s"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                   check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True,
                                          check=True).stdout.split()]
    want = []
    for s in fields.values():
        want += [ctypes.sizeof(s)] + [getattr(s, f).offset for f, _ in s._fields_]
    assert got == want


def test_packed_structs_match_the_declared_ones():
    """What the binding passes is the bytes of the declared structs."""
    values = (0x10, 0x20, 0x30, 0x40, 1 << 33, 64, 8, 128, 32)
    assert wq._pack_kv4_cache(*values) == bytes(wq._KV4CacheStruct(*values))
    values = (3, 7, 0x50, 0x60, 0x70, 9, 1 << 34, 5)
    assert wq._pack_kv4_batch(*values) == bytes(wq._KV4BatchStruct(*values))


@pytest.mark.parametrize("d", [64, 128])
def test_code_order(d):
    """Two codes a byte, even element low; key words and value halfwords of
    one index together."""
    codes = np.random.default_rng(d).integers(0, 16, (5, d)).astype(np.uint8)
    k, v = kv4_ref.pack(codes, "k"), kv4_ref.pack(codes, "v")
    for e in range(d):
        chunk, inside = e // 32, e % 32
        word = (inside // 8) * (d // 32) + chunk          # 4-byte words, [4][d/32]
        assert ((k[:, word * 4 + inside % 8 // 2] >> (4 * (e % 2))) & 15 == codes[:, e]).all()
        half = (inside // 4) * (d // 32) + chunk          # 2-byte units, [8][d/32]
        assert ((v[:, half * 2 + inside % 4 // 2] >> (4 * (e % 2))) & 15 == codes[:, e]).all()
    assert (kv4_ref.unpack(k, "k") == codes).all() and (kv4_ref.unpack(v, "v") == codes).all()


@pytest.fixture(scope="module")
def base():
    buf = ctypes.create_string_buffer(4096)
    return buf, (ctypes.addressof(buf) + 15) // 16 * 16


def cache(base, **kw):
    c = dict(k_codes=base, k_meta=base, v_codes=base, v_meta=base, pages=4, page_size=16,
             kv_heads=2, head_dim=64, group=32)
    c.update(kw)
    return wq._KV4CacheStruct(*(c[f] for f, _ in wq._KV4CacheStruct._fields_))


def batch(base, **kw):
    b = dict(seqs=2, rows=4, row_starts=None, seq_lens=base, page_table=base, table_width=2,
             table_stride=2, max_rows=0)
    b.update(kw)
    return wq._KV4BatchStruct(*(b[f] for f, _ in wq._KV4BatchStruct._fields_))


def calls(base, c, b, stride=None, ptr=None):
    p = base if ptr is None else ptr
    s = 128 if stride is None else stride
    ws = wq.lib.wq_kv4_attention_workspace_bytes()
    cr, br = ctypes.byref(c), ctypes.byref(b)
    return (wq.lib.wq_kv4_write(p, s, p, s, cr, br, None),
            wq.lib.wq_kv4_attention(p, 2 * s, 4, cr, br, 0.125, p, 2 * s, base, ws, None),
            wq.lib.wq_kv4_read(cr, br, p, p, None))


@pytest.mark.parametrize("change,status", [
    (dict(k_codes=None), INVALID), (dict(v_meta=None), INVALID), (dict(pages=0), INVALID),
    (dict(pages=1 << 31), INVALID), (dict(kv_heads=0), INVALID), (dict(head_dim=96), UNSUPPORTED),
    (dict(head_dim=256), UNSUPPORTED), (dict(group=16), UNSUPPORTED), (dict(group=128), INVALID),
    (dict(page_size=8), UNSUPPORTED), (dict(page_size=48), UNSUPPORTED),
    (dict(page_size=512), UNSUPPORTED), (dict(page_size=0), INVALID)])
def test_cache_refusals(base, change, status):
    _, p = base
    assert set(calls(p, cache(p, **change), batch(p))) == {status}


def test_misaligned_buffers(base):
    _, p = base
    for f in ("k_codes", "k_meta", "v_codes", "v_meta"):
        assert set(calls(p, cache(p, **{f: p + 8}), batch(p))) == {ALIGNMENT}
    assert set(calls(p, cache(p), batch(p), ptr=p + 2)) == {ALIGNMENT}
    assert calls(p, cache(p), batch(p), stride=132)[:1] == (ALIGNMENT,)


@pytest.mark.parametrize("change", [
    dict(rows=-1), dict(seqs=0), dict(seqs=3), dict(seq_lens=None), dict(page_table=None),
    dict(table_width=0), dict(table_stride=1), dict(max_rows=-1)])
def test_batch_refusals(base, change):
    _, p = base
    assert set(calls(p, cache(p), batch(p, **change))) == {INVALID}


def test_row_and_workspace_refusals(base):
    _, p = base
    c, b = cache(p), batch(p)
    ws = wq.lib.wq_kv4_attention_workspace_bytes()
    attn = lambda **kw: wq.lib.wq_kv4_attention(*{**dict(  # noqa: E731
        q=p, qs=256, heads=4, c=ctypes.byref(c), b=ctypes.byref(b), scale=0.1, o=p, os=256, w=p,
        n=ws, s=None), **kw}.values())
    assert calls(p, c, b, stride=120)[0] == INVALID            # rows overlap
    assert attn(heads=3) == INVALID and attn(heads=0) == INVALID
    assert attn(scale=float("nan")) == INVALID and attn(scale=float("inf")) == INVALID
    assert attn(w=None) == INVALID and attn(n=ws - 1) == INVALID and attn(w=p + 4) == ALIGNMENT
    assert attn(q=None) == INVALID and attn(o=None) == INVALID
    assert attn(qs=248) == INVALID and attn(os=260) == ALIGNMENT
    assert attn(b=ctypes.byref(batch(p, rows=1 << 29, seqs=1, row_starts=p))) == INVALID


def test_calls_without_rows(base):
    """No rows: no work, nothing launched, and no pointer of the batch looked at."""
    _, p = base
    empty = batch(p, rows=0, seqs=0, seq_lens=None, page_table=None, table_width=0)
    assert set(calls(p, cache(p), empty)) == {0}
    assert wq.lib.wq_kv4_attention_workspace_bytes() > 0
