"""The 4-bit key/value cache operators as measured workloads: writing rows
into the cache (and reading them back), reading cached sequences, and
attention over the cache, each in a plain form of elementary torch operations
and through the package.

A case names sizes only; lengths of ragged batches follow from the case's
``spread`` number, so that the work of a case does not depend on a seed.
"""
from __future__ import annotations

import math
import random

import torch

own = False

# Where a cache slot has never been written its metadata is whatever memory
# held: the prepared caches put NaN there.


# ------------------------------------------------------------------ the cases

def _case(name, op, seqs, rows, length, q_heads=32, kv_heads=8, head_dim=128, group=64, page=64,
          ragged=False, ragged_rows=False, spread=1):
    return {"name": name, "op": op, "seqs": seqs, "rows": rows, "length": length,
            "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim, "group": group,
            "page": page, "ragged": ragged, "ragged_rows": ragged_rows, "spread": spread}


def listed():
    return [
        # one new token of one sequence: the append of every layer of every decode step
        _case("write-token", "write", 1, 1, 777),
        # a mixed batch of chunks with odd lengths, small heads, groups of 32
        _case("write-ragged", "write", 13, 611, 2500, q_heads=16, kv_heads=4, head_dim=64, group=32,
              page=16, ragged=True, ragged_rows=True, spread=5),
        # prompts of 8192 tokens entering the cache
        _case("write-prompts", "write", 4, 8192, 8192, group=128),
        # a shared prefix handed to code that takes 16-bit keys and values
        _case("read-short", "read", 1, 333, 333, page=32),
        # the caches of a ragged batch, whole
        _case("read-ragged", "read", 24, 6000, 6000, group=32, ragged=True, ragged_rows=True, spread=9),
        # one user's decode step at a short context: latency
        _case("decode-one-short", "attention", 1, 1, 1000),
        # one user's decode step at a long context
        _case("decode-one-long", "attention", 1, 1, 131072),
        # a serving batch, ragged, groups of 32, small pages
        _case("decode-batch", "attention", 32, 1, 4096, group=32, page=16, ragged=True, spread=3),
        # the largest decode batch
        _case("decode-large", "attention", 128, 1, 8192, group=64, ragged=True, spread=7),
        # verification of a few drafted tokens in every sequence
        _case("few-tokens", "attention", 16, 4, 5000, head_dim=64, group=64, ragged=True, spread=2),
        # chunks of prompts on top of cached prefixes, ragged in both
        _case("chunk", "attention", 6, 700, 4500, q_heads=28, kv_heads=4, group=32, page=32,
              ragged=True, ragged_rows=True, spread=11),
        # a whole prompt over its own cache
        _case("prompt", "attention", 1, 8192, 8192, group=128, page=128),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    head_dim = rng.choice([64, 128, 128])
    kv_heads = rng.choice([1, 2, 4, 5, 8])
    case = _case("", rng.choice(["write", "read", "attention", "attention", "attention"]), 1, 1, 1,
                 q_heads=kv_heads * rng.choice([1, 2, 3, 4, 4, 7, 8]), kv_heads=kv_heads,
                 head_dim=head_dim, group=rng.choice([g for g in (32, 64, 128) if g <= head_dim]),
                 page=rng.choice([16, 32, 64, 128]), ragged=rng.random() < 0.7,
                 spread=rng.randrange(1, 1 << 20))
    del case["name"]
    tokens = 600_000 if case["op"] == "attention" else 32_768
    seqs = log(1, 128)
    length = min(log(1, 131_072), max(1, tokens // seqs))
    if case["op"] == "attention":
        kind = rng.choice(["one", "one", "few", "chunk"])
        rows = {"one": 1, "few": rng.randrange(2, 9), "chunk": log(9, 4096)}[kind]
        # the products and the largest listed prompt's bound the rows
        rows = max(1, min(rows, length, (1 << 30) // (case["q_heads"] * seqs * length) or 1))
        case["ragged_rows"] = rows > 1 and rng.random() < 0.5
    else:
        rows = length if case["op"] == "read" else min(length, log(1, 8192))
        case["ragged_rows"] = rng.random() < 0.5
    return dict(case, seqs=seqs, rows=rows, length=length)


def _lengths(case):
    """(tokens, new rows) of every sequence."""
    rng = random.Random(case["spread"])
    lens = [rng.randint((case["length"] + 3) // 4, case["length"]) if case["ragged"] else case["length"]
            for _ in range(case["seqs"])]
    if case["op"] == "read" and case["ragged_rows"]:
        return lens, list(lens)
    rows = [rng.randint((case["rows"] + 9) // 10, case["rows"]) if case["ragged_rows"] else case["rows"]
            for _ in range(case["seqs"])]
    return lens, rows


def work(case):
    lens, rows = _lengths(case)
    h, hq, d = case["kv_heads"], case["q_heads"], case["head_dim"]
    token = 2 * h * (d // 2 + 4 * (d // case["group"]))      # codes and metadata of one token
    values = 2 * h * d * 2                                   # its keys and values in 16 bits
    if case["op"] == "attention":
        seen = sum(max(0, length - t + i + 1) for length, t in zip(lens, rows) for i in range(t))
        return {"bytes": sum(lens) * token + 2 * sum(rows) * hq * d * 2, "flops": 4 * d * hq * seen}
    n = sum(min(length, t) for length, t in zip(lens, rows))
    per_row = values + token + (values if case["op"] == "write" else 0)
    return {"bytes": n * per_row, "flops": n * 2 * h * d * 4}


# ------------------------------------------------- the format, in plain torch

def _quantize(x, group):
    """x [..., D] -> codes (0..15) [..., D/G, G], scale, zero [..., D/G], all
    in 64 bits: the exact map of values taken to binary16."""
    x = x.to(torch.float32).clamp(-65504, 65504).to(torch.float16).to(torch.float64)
    x = x.unflatten(-1, (-1, group))
    lo, hi = x.amin(-1).clamp(max=0), x.amax(-1).clamp(min=0)
    exact = (hi - lo) / 15
    near = exact.to(torch.float16)
    up = (near.view(torch.int16) + 1).view(torch.float16)
    scale = torch.where(near.to(torch.float64) < exact, up, near).to(torch.float64)
    scale = torch.where(hi == lo, torch.ones_like(scale), scale)
    zero = torch.round(-lo / scale).clamp(0, 15)
    codes = (torch.round(x / scale[..., None]) + zero[..., None]).clamp(0, 15)
    return codes, scale, zero


def _pack_k(codes):
    """[..., D] codes -> bytes: two codes a byte, low nibble first; 4-byte
    words in the order [4][D/32] of the row's [D/32][4] words."""
    b = codes.to(torch.uint8)
    b = b[..., 0::2] | (b[..., 1::2] << 4)
    return b.unflatten(-1, (-1, 4, 4)).transpose(-3, -2).flatten(-3)


def _pack_v(codes):
    """As _pack_k with 2-byte units in the order [8][D/32] of [D/32][8]."""
    b = codes.to(torch.uint8)
    b = b[..., 0::2] | (b[..., 1::2] << 4)
    return b.unflatten(-1, (-1, 8, 2)).transpose(-3, -2).flatten(-3)


def _unpack_k(b):
    b = b.unflatten(-1, (4, -1, 4)).transpose(-3, -2).flatten(-3)
    return torch.stack((b & 15, b >> 4), -1).flatten(-2)


def _unpack_v(b):
    b = b.unflatten(-1, (8, -1, 2)).transpose(-3, -2).flatten(-3)
    return torch.stack((b & 15, b >> 4), -1).flatten(-2)


def _values(codes, meta):
    """s (u - z) in 32 bits (exact): codes [..., D], meta [..., D/G, 2]."""
    m = meta.to(torch.float32)
    u = codes.to(torch.float32).unflatten(-1, (m.shape[-2], -1))
    return ((u - m[..., 1:]) * m[..., :1]).flatten(-2)


# ------------------------------------------------------------------ the state

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    lens, rows = _lengths(case)
    h, hq, d, page, group = (case[k] for k in ("kv_heads", "q_heads", "head_dim", "page", "group"))
    # pages in random order, a few to spare
    need = [(n + page - 1) // page for n in lens]
    pages, width = sum(need) + 3, max(need) + 1
    order = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
    table = torch.zeros(len(lens), width, dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    state = {"op": case["op"], "group": group, "max_rows": max(rows), "width": max(need),
             "scale": 1 / math.sqrt(d), "n_rows": sum(rows), "uniform": not case["ragged_rows"],
             "seq_lens": torch.tensor(lens, dtype=torch.int32, device=dev), "page_table": table,
             "row_starts": None if not case["ragged_rows"] else torch.tensor(
                 [sum(rows[:b]) for b in range(len(rows) + 1)], dtype=torch.int32, device=dev)}
    # keys with a few strong channels, as trained models have them; slots never
    # written hold any codes and NaN metadata
    strong = 1 + 7 * (torch.rand(h, d, generator=gen, device=dev) < 0.03).to(torch.float32)
    caches = []
    for channel in (strong, torch.ones_like(strong)):
        codes = torch.empty(pages, h, page, d // 2, dtype=torch.uint8, device=dev)
        meta = torch.empty(pages, h, page, d // group, 2, dtype=torch.float16, device=dev)
        for p in range(0, pages, 1024):
            n = min(1024, pages - p)
            x = torch.randn(n, h, page, d, generator=gen, device=dev) * channel[:, None]
            q, s, z = _quantize(x.to(torch.bfloat16), group)
            codes[p:p + n] = (_pack_k if not caches else _pack_v)(q.flatten(-2))
            meta[p:p + n] = torch.stack((s, z), -1).to(torch.float16)
        for b, n in enumerate(lens):
            if n % page:
                meta[order[sum(need[:b + 1]) - 1].long(), :, n % page:] = float("nan")
        caches.append((codes, meta))
    (state["k_codes"], state["k_meta"]), (state["v_codes"], state["v_meta"]) = caches
    n = state["n_rows"]
    # the fused projection's output: queries, keys and values of a row side by side
    if case["op"] == "write":
        qkv = torch.randn(n, hq + 2 * h, d, generator=gen, device=dev)
        qkv[:, hq:hq + h] *= strong
        qkv = qkv.to(torch.bfloat16)
        state["k"], state["v"] = qkv[:, hq:hq + h], qkv[:, hq + h:]
    if case["op"] == "attention":
        state["q"] = torch.randn(n, hq, d, generator=gen, device=dev).to(torch.bfloat16)
        state["out"] = torch.zeros(n, hq, d, dtype=torch.bfloat16, device=dev)
    else:
        state["out"] = [torch.zeros(n, h, d, dtype=torch.bfloat16, device=dev) for _ in "kv"]
    if own:  # the cache handle and the workspace that a serving loop keeps
        import w4a16_decode_matmul_b200 as wq
        state["cache"] = wq.KV4Cache(state["k_codes"], state["k_meta"], state["v_codes"],
                                     state["v_meta"], group)
        state["workspace"] = wq.kv4_workspace(dev)
    return state


# -------------------------------------------------------------------- one pass

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(st):
    import w4a16_decode_matmul_b200 as wq
    batch = (st["seq_lens"], st["page_table"], st["row_starts"])
    if st["op"] == "attention":
        return wq.kv4_attention(st["q"], st["cache"], *batch, max_rows=st["max_rows"],
                                scale=st["scale"], out=st["out"], workspace=st["workspace"])
    if st["op"] == "write":
        wq.kv4_write(st["k"], st["v"], st["cache"], *batch)
    wq.kv4_read(st["cache"], *batch, out=st["out"])
    return st["out"]


def _run_plain(st):
    if st["op"] == "attention":
        return _attention(st)
    page_of, slot, live = _slots(st)
    at = (page_of, slice(None), slot)
    if st["op"] == "write":
        _store(st["k"][live], st["k_codes"], st["k_meta"], at, st["group"], _pack_k)
        _store(st["v"][live], st["v_codes"], st["v_meta"], at, st["group"], _pack_v)
    k_out, v_out = st["out"]
    k_out[live] = _values(_unpack_k(st["k_codes"][at]), st["k_meta"][at]).to(torch.bfloat16)
    v_out[live] = _values(_unpack_v(st["v_codes"][at]), st["v_meta"][at]).to(torch.bfloat16)
    return st["out"]


def _store(x, codes, meta, at, group, pack):
    q, s, z = _quantize(x, group)
    codes[at] = pack(q.flatten(-2))
    meta[at] = torch.stack((s, z), -1).to(torch.float16)


def _starts(st):
    if not st["uniform"]:
        return st["row_starts"].long()
    b = st["seq_lens"].numel()
    return torch.arange(b + 1, device=st["seq_lens"].device) * (st["n_rows"] // b)


def _slots(st):
    """Page and slot of every row that holds a token, and which rows those are."""
    starts = _starts(st)
    row = torch.arange(st["n_rows"], device=starts.device)
    b = torch.searchsorted(starts, row, right=True) - 1
    pos = st["seq_lens"].long()[b] - starts[b + 1] + row
    live = pos >= 0
    b, pos = b[live], pos[live]
    page = st["k_codes"].shape[2]
    return st["page_table"][b, pos // page].long(), pos % page, live


def _gather(codes, meta, table, unpack):
    """The values of every sequence's pages: [B, H, width * page, D]."""
    return _values(unpack(codes[table]), meta[table]).transpose(1, 2).flatten(2, 3)


def _attention(st):
    """All sequences at once, padded to the longest."""
    starts, lens = _starts(st), st["seq_lens"].long()
    table = st["page_table"][:, :st["width"]].long()
    k = _gather(st["k_codes"], st["k_meta"], table, _unpack_k)
    v = _gather(st["v_codes"], st["v_meta"], table, _unpack_v)
    b, h, n, d = k.shape
    token = torch.arange(n, device=k.device)
    v = torch.where((token < lens[:, None])[:, None, :, None], v, 0)
    i = torch.arange(st["max_rows"], device=k.device)
    rows = starts[1:] - starts[:-1]
    live = i < rows[:, None]                                              # [B, T]
    at = torch.where(live, starts[:-1, None] + i, 0)
    q = st["q"][at].to(torch.float32).unflatten(2, (h, -1))               # [B, T, H, R, D]
    q = q.permute(0, 2, 3, 1, 4).flatten(2, 3)                            # [B, H, R T, D]
    s = torch.matmul(q, k.transpose(-1, -2)) * st["scale"]
    pos = (lens - rows)[:, None] + i
    seen = (token <= pos[:, :, None])[:, None, None]                      # [B, 1, 1, T, n]
    s = torch.where(seen, s.unflatten(2, (-1, i.numel())), -math.inf).flatten(2, 3)
    top = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(top == -math.inf, 0, top))
    o = torch.matmul(e, v) / e.sum(-1, keepdim=True).clamp(min=1e-30)
    o = o.unflatten(2, (-1, i.numel())).permute(0, 3, 1, 2, 4).flatten(2, 3)
    st["out"][at[live]] = o[live].to(torch.bfloat16)
    return st["out"]


# --------------------------------------------------------- the same in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    lens, rows = _lengths(case)
    h, hq, d, page = (case[k] for k in ("kv_heads", "q_heads", "head_dim", "page"))
    group, table = case["group"], st["page_table"].tolist()

    def nibbles(b):
        return torch.stack((b % 16, torch.div(b, 16, rounding_mode="floor")), -1)

    def cached(b, first, last):
        """Keys and values of positions first..last-1 of sequence b, 64 bits: [H, n, D]."""
        found = []
        pos = torch.arange(first, last, device="cuda")
        ids = torch.tensor(table[b], device="cuda")[pos // page]
        for codes, meta, units, size in ((st["k_codes"], st["k_meta"], 4, 4),
                                         (st["v_codes"], st["v_meta"], 8, 2)):
            c = codes[ids, :, pos % page].reshape(len(pos), h, units, d // 32, size)
            u = nibbles(c.permute(0, 1, 3, 2, 4).reshape(len(pos), h, d // 2)).reshape(
                len(pos), h, d // group, group).double()
            m = meta[ids, :, pos % page].double()
            found.append(((u - m[..., 1:2]) * m[..., 0:1]).reshape(len(pos), h, d).transpose(0, 1))
        return found

    def rounded(x):
        """Quantized and back, from the definition: x [n, H, D]."""
        x = x.double().clamp(-65504, 65504)
        tiny = x.abs() < 2.0 ** -17          # below this binary16 drops bits of a bfloat16
        x = torch.where(tiny, torch.round(x * 2.0 ** 24) / 2.0 ** 24, x)
        x = x.reshape(x.shape[0], h, d // group, group)
        lo = torch.minimum(x.min(-1, keepdim=True).values, torch.zeros((), device="cuda").double())
        hi = torch.maximum(x.max(-1, keepdim=True).values, torch.zeros((), device="cuda").double())
        step = (hi - lo) / 15
        unit = torch.exp2(torch.floor(torch.log2(step.clamp(min=2.0 ** -14))) - 10)
        s = torch.ceil(step / unit) * unit
        s = torch.where(hi > lo, s, torch.ones_like(s))
        z = torch.round(-lo / s)
        u = torch.minimum(torch.maximum(torch.round(x / s) + z, torch.zeros_like(x)),
                          torch.full_like(x, 15))
        return ((u - z) * s).reshape(x.shape[0], h, d)

    if case["op"] == "write":
        live = torch.cat([torch.arange(t) >= t - n for n, t in zip(lens, rows)]).cuda()[:, None, None]
        return [torch.where(live, rounded(st[x]), 0) for x in "kv"]
    if case["op"] == "read":
        whole = [torch.zeros(sum(rows), h, d, dtype=torch.float64, device="cuda") for _ in "kv"]
        at = 0
        for b, (n, t) in enumerate(zip(lens, rows)):
            at += t
            held = min(n, t)                 # rows before the sequence's first token hold none
            for x, found in zip(whole, cached(b, n - held, n)):
                x[at - held:at] = found.transpose(0, 1)
        return whole
    out, at = [], 0
    for b, (n, t) in enumerate(zip(lens, rows)):
        k, v = cached(b, 0, n)
        q = st["q"][at:at + t].double().reshape(t, h, hq // h, d)
        at += t
        o = torch.zeros(t, h, hq // h, d, dtype=torch.float64, device="cuda")
        for i in range(0, t, 512):
            s = torch.einsum("thrd,hnd->thrn", q[i:i + 512], k) / math.sqrt(d)
            pos = n - t + i + torch.arange(s.shape[0], device="cuda")
            hidden = torch.arange(n, device="cuda")[None] > pos[:, None]
            s = s.masked_fill(hidden[:, None, None], -math.inf)
            w = torch.softmax(s, -1).nan_to_num(0.0)
            o[i:i + 512] = torch.einsum("thrn,hnd->thrd", w, v)
        out.append(o.reshape(t, hq, d))
    return torch.cat(out)
