"""What a step of speculative decoding does around the products and the
attention over the 4-bit key/value cache, as measured workloads: rotary
positions (alone, and fused with the rows' way into the cache), attention over
the pages that a score selects, and the verification of drafted tokens; each
in a plain form of elementary torch operations and through the package.

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

def _rotary(name, rows, heads, head_dim=128, dim=128, interleaved=False, inverse=False, far=8192):
    return {"name": name, "op": "rotary", "rows": rows, "heads": heads, "head_dim": head_dim, "dim": dim,
            "interleaved": interleaved, "inverse": inverse, "far": far}


def _write(name, seqs, rows, length, q_heads=32, kv_heads=8, head_dim=128, dim=128, group=64, page=64,
           interleaved=False, ragged=False, ragged_rows=False, spread=1):
    return {"name": name, "op": "write", "seqs": seqs, "rows": rows, "length": length, "q_heads": q_heads,
            "kv_heads": kv_heads, "head_dim": head_dim, "dim": dim, "group": group, "page": page,
            "interleaved": interleaved, "ragged": ragged, "ragged_rows": ragged_rows, "spread": spread}


def _sparse(name, seqs, rows, length, pages, q_heads=32, kv_heads=8, head_dim=128, group=64, page=64,
            first=1, last=2, ragged=False, spread=1):
    return {"name": name, "op": "sparse", "seqs": seqs, "rows": rows, "length": length, "pages": pages,
            "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim, "group": group, "page": page,
            "first": first, "last": last, "ragged": ragged, "ragged_rows": False, "spread": spread}


def _verify(name, seqs, rows, vocab, kind="logits", dtype="float32", drafts="dense", greedy=False,
            ragged_rows=False, spread=1):
    return {"name": name, "op": "verify", "seqs": seqs, "rows": rows, "vocab": vocab, "kind": kind,
            "dtype": dtype, "drafts": drafts, "greedy": greedy, "ragged_rows": ragged_rows, "spread": spread}


def listed():
    return [
        # queries and keys of one new token, side by side in the fused projection's row
        _rotary("rotary-token", 1, 40),
        # a prompt's queries and keys at positions of a long context
        _rotary("rotary-prompt", 8192, 40, far=1_000_000),
        # the gradient of a rotation: half of each head, interleaved, an odd number of rows
        _rotary("rotary-gradient", 3001, 24, head_dim=64, dim=32, interleaved=True, inverse=True),
        # the append of every layer of every decode step
        _write("write-token", 1, 1, 777),
        # five fed tokens (one sampled, four drafted) in every sequence of a batch
        _write("write-drafts", 64, 5, 6000, page=32, group=32, ragged=True, spread=5),
        # prompts of odd lengths entering the cache, part of each head rotated
        _write("write-prompts", 4, 8192, 8192, dim=64, group=128, ragged_rows=True, spread=3),
        # one user's decode step on a long context
        _sparse("sparse-one", 1, 1, 131072, 64),
        # a serving batch, ragged, small pages
        _sparse("sparse-batch", 16, 1, 32768, 64, page=32, group=32, ragged=True, spread=3),
        # a sampled and four drafted tokens in every sequence, small heads
        _sparse("sparse-drafts", 8, 5, 65536, 48, q_heads=28, kv_heads=4, head_dim=64, ragged=True, spread=9),
        # one user's four drafts against probabilities that the sampler made
        _verify("verify-one", 1, 5, 32000, kind="probabilities"),
        # the logits of a batch, drafts of odd lengths, an odd vocabulary
        _verify("verify-batch", 32, 6, 50021, dtype="bfloat16", ragged_rows=True, spread=7),
        # the largest batch and vocabulary, logits in 32 bits
        _verify("verify-large", 64, 6, 131072),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    op = rng.choice(["rotary", "write", "sparse", "sparse", "verify", "verify"])
    head_dim = rng.choice([64, 128, 128])
    kv_heads = rng.choice([1, 2, 4, 5, 8])
    spread = rng.randrange(1, 1 << 20)
    if op == "rotary":
        heads, head_dim = rng.choice([1, 5, 8, 20, 40]), rng.choice([64, 80, 96, 128, 256])
        rows = log(1, min(8192, (8192 * 40 * 128) // (heads * head_dim)))
        case = _rotary("", rows, heads, head_dim, 2 * rng.randrange(8, head_dim // 2 + 1),
                       rng.random() < 0.5, rng.random() < 0.4, log(1000, 1_000_000))
    elif op == "write":
        seqs = log(1, 128)
        length = log(1, 16384)
        rows = max(1, min(length, log(1, 8192), 32768 // seqs))
        case = _write("", seqs, rows, min(length, max(1, 400_000 // seqs)), kv_heads * rng.choice([1, 2, 4, 7]), kv_heads,
                      head_dim, 16 * rng.randrange(1, head_dim // 16 + 1),
                      rng.choice([g for g in (32, 64, 128) if g <= head_dim]), rng.choice([16, 32, 64, 128]),
                      rng.random() < 0.4, rng.random() < 0.7, rng.random() < 0.5, spread)
        case["rows"] = min(case["rows"], case["length"])
    elif op == "sparse":
        seqs = log(1, 32)
        length = log(200, min(131_072, 500_000 // seqs))
        first, last = rng.randrange(0, 3), rng.randrange(1, 4)
        page = rng.choice([16, 32, 64, 128])
        case = _sparse("", seqs, rng.choice([1, 1, 1, rng.randrange(2, 9)]), length,
                       rng.randrange(first + last, max(first + last + 1, min(256, 8192 // page))),
                       kv_heads * rng.choice([1, 2, 4, 7, 8]), kv_heads, head_dim,
                       rng.choice([g for g in (32, 64, 128) if g <= head_dim]), page, first, last,
                       rng.random() < 0.7, spread)
        # what the rows' lists hold bounds the rows and the pages
        page_work = seqs * page * kv_heads * head_dim
        if case["rows"] * (first + last) * page_work > 1 << 26:
            case["rows"] = 1
        case["pages"] = min(case["pages"], max(first + last, (1 << 26) // (case["rows"] * page_work)))
    else:
        vocab = rng.choice([log(100, 131_072), rng.choice([32000, 50021, 64000, 128000])])
        seqs = log(1, 64)
        case = _verify("", seqs, rng.randrange(1, 7), vocab, rng.choice(["logits", "logits", "probabilities"]),
                       rng.choice(["float32", "bfloat16"]), rng.choice(["dense", "dense", "none"]),
                       False, rng.random() < 0.5, spread)
        case["greedy"] = case["kind"] == "logits" and rng.random() < 0.3
    del case["name"]
    return case


def _lengths(case):
    """(tokens, rows) of every sequence."""
    rng = random.Random(case["spread"])
    length = case.get("length", 0)
    lens = [rng.randint((length + 3) // 4, length) if case.get("ragged") else length
            for _ in range(case["seqs"])]
    rows = [rng.randint((case["rows"] + 9) // 10, case["rows"]) if case["ragged_rows"] else case["rows"]
            for _ in range(case["seqs"])]
    return lens, rows


def work(case):
    if case["op"] == "rotary":
        n = case["rows"] * case["heads"]
        return {"bytes": n * case["head_dim"] * 4 + case["rows"] * 4 + case["dim"] * 2,
                "flops": n * case["dim"] * 3}
    lens, rows = _lengths(case)
    if case["op"] == "verify":
        size = 4 if case["dtype"] == "float32" else 2
        drafts = sum(t - 1 for t in rows)
        if case["kind"] == "logits":
            read = sum(rows) + (drafts if case["drafts"] == "dense" else 0)
            return {"bytes": read * case["vocab"] * size + sum(rows) * 12 + case["seqs"] * 12,
                    "flops": read * case["vocab"] * 3}
        read = case["seqs"] * (2 if case["drafts"] == "dense" else 1)
        return {"bytes": read * case["vocab"] * size + drafts * 2 * size + sum(rows) * 12 + case["seqs"] * 12,
                "flops": read * case["vocab"] * 2}
    h, hq, d = case["kv_heads"], case["q_heads"], case["head_dim"]
    token = 2 * h * (d // 2 + 4 * (d // case["group"]))      # codes and metadata of one token
    if case["op"] == "write":
        n = sum(min(length, t) for length, t in zip(lens, rows))
        # queries in and out; keys and values in, into the cache, and out of it again
        return {"bytes": n * (4 * hq * d + 4 * h * d + 2 * token + 4 * h * d),
                "flops": n * (3 * (hq + h) * case["dim"] + 2 * h * d * 4)}
    total, flops = 0, 0
    for n, t in zip(lens, rows):
        pages = -(-n // case["page"])
        kept = min(pages, case["pages"])
        total += pages * h * (2 * d + 4) + min(pages, t * kept) * case["page"] * token
        total += t * (4 * hq * d + h * case["pages"] * 4 + 4)
        flops += t * (4 * d * hq * kept * case["page"] + 4 * d * h * pages)
    return {"bytes": total, "flops": flops}


# ------------------------------------------- the cache's format, in plain torch

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


def _pack(codes, unit):
    """[..., D] codes -> bytes: two codes a byte, low nibble first; units of
    `unit` bytes in the order [16/unit][D/32] of the row's [D/32][16/unit]
    (keys 4, values 2)."""
    b = codes.to(torch.uint8)
    b = b[..., 0::2] | (b[..., 1::2] << 4)
    return b.unflatten(-1, (-1, 16 // unit, unit)).transpose(-3, -2).flatten(-3)


def _unpack(b, unit):
    b = b.unflatten(-1, (16 // unit, -1, unit)).transpose(-3, -2).flatten(-3)
    return torch.stack((b & 15, b >> 4), -1).flatten(-2)


def _values(codes, meta):
    """s (u - z) in 32 bits (exact): codes [..., D], meta [..., D/G, 2]."""
    m = meta.to(torch.float32)
    u = codes.to(torch.float32).unflatten(-1, (m.shape[-2], -1))
    return ((u - m[..., 1:]) * m[..., :1]).flatten(-2)


def _power(top):
    """The smallest power of two p with 127 p >= top (32 bits; 1 where top is 0)."""
    m, e = torch.frexp(top)
    e = torch.where(m <= 127 / 128, e - 7, e - 6)
    return torch.where(top > 0, torch.ldexp(torch.ones_like(top), e), torch.ones_like(top))


def _bounds(values, live):
    """values [..., P, D] of pages' keys, live [..., P] -> smallest and largest
    of every dimension on a grid of a power of two, int8 [..., 2, D], and the grid."""
    lo = torch.where(live[..., None], values, math.inf).amin(-2)
    hi = torch.where(live[..., None], values, -math.inf).amax(-2)
    grid = _power(torch.maximum(lo.abs(), hi.abs()).amax(-1))
    return torch.stack((torch.floor(lo / grid[..., None]), torch.ceil(hi / grid[..., None])),
                       -2).to(torch.int8), grid


# ------------------------------------------------------------------ the state

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    state = {"rotary": _prepare_rotary, "write": _prepare_cache, "sparse": _prepare_cache,
             "verify": _prepare_verify}[case["op"]](case, gen, dev)
    state["op"] = case["op"]
    if own:  # the handles and the workspace that a serving loop keeps
        import w4a16_decode_matmul_b200 as wq
        if "freqs" in state:
            state["rot"] = wq.Rotary(state["freqs"], state["interleaved"], state["amplitude"])
        if "k_codes" in state:
            state["cache"] = wq.KV4Cache(state["k_codes"], state["k_meta"], state["v_codes"],
                                         state["v_meta"], state["group"])
        if case["op"] == "sparse":
            state["handle"] = wq.KV4Bounds(state["bounds"], state["grid"])
            state["workspace"] = wq.kv4_workspace(dev)
        if case["op"] == "verify":
            state["workspace"] = wq.verify_workspace(state["n_rows"], dev)
    return state


def _frequencies(dim, far, dev):
    """Base 10,000, the slow ones stretched for contexts of `far` positions."""
    f = 10_000.0 ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim)
    stretch = max(1.0, far / 32768)
    f = torch.where(f * 32768 / (2 * math.pi) < 1, f / stretch, f)
    return f.to(torch.float32).to(dev), 0.1 * math.log(stretch) + 1


def _prepare_rotary(case, gen, dev):
    n, h, d = case["rows"], case["heads"], case["head_dim"]
    freqs, amplitude = _frequencies(case["dim"], case["far"], dev)
    start = int(torch.randint(0, max(1, case["far"] - n + 1), (1,), generator=gen, device=dev))
    # queries, keys and values of a row side by side; the values are not rotated
    qkv = torch.randn(n, h + max(1, h // 5), d, generator=gen, device=dev).to(torch.bfloat16)
    return {"x": qkv[:, :h], "positions": torch.arange(start, start + n, device=dev, dtype=torch.int32),
            "freqs": freqs, "amplitude": amplitude, "interleaved": case["interleaved"],
            "inverse": case["inverse"], "out": torch.zeros(n, h, d, dtype=torch.bfloat16, device=dev)}


def _prepare_cache(case, gen, dev):
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
    n = sum(rows)
    state = {"group": group, "max_rows": max(rows), "width": max(need), "scale": 1 / math.sqrt(d),
             "n_rows": n, "uniform": not case["ragged_rows"], "page": page,
             "seq_lens": torch.tensor(lens, dtype=torch.int32, device=dev), "page_table": table,
             "row_starts": None if not case["ragged_rows"] else torch.tensor(
                 [sum(rows[:b]) for b in range(len(rows) + 1)], dtype=torch.int32, device=dev)}
    strong = 1 + 7 * (torch.rand(h, d, generator=gen, device=dev) < 0.03).to(torch.float32)
    if case["op"] == "write":
        # what the cache held before does not matter to a write: any codes, NaN metadata
        for kind in "kv":
            state[kind + "_codes"] = torch.zeros(pages, h, page, d // 2, dtype=torch.uint8, device=dev)
            state[kind + "_meta"] = torch.full((pages, h, page, d // group, 2), float("nan"),
                                               dtype=torch.float16, device=dev)
        # the fused projection's output: queries, keys and values of a row side by side
        qkv = torch.randn(n, hq + 2 * h, d, generator=gen, device=dev)
        qkv[:, hq:hq + h] *= strong
        qkv = qkv.to(torch.bfloat16)
        state["q"], state["k"], state["v"] = qkv[:, :hq], qkv[:, hq:hq + h], qkv[:, hq + h:]
        state["freqs"], state["amplitude"] = _frequencies(case["dim"], case["length"], dev)
        state["interleaved"] = case["interleaved"]
        state["q_out"] = torch.zeros(n, hq, d, dtype=torch.bfloat16, device=dev)
        state["out"] = [torch.zeros(n, h, d, dtype=torch.bfloat16, device=dev) for _ in "kv"]
        return state
    # keys with a few strong channels and a part that neighbouring tokens share, as trained
    # models have them; slots never written hold any codes and NaN metadata
    live = torch.zeros(pages, page, dtype=torch.bool, device=dev)
    for b, m in enumerate(lens):
        ids = order[sum(need[:b]):sum(need[:b + 1])].long()
        live[ids] = (torch.arange(len(ids) * page, device=dev) < m).view(-1, page)
    bounds = torch.zeros(pages, h, 2, d, dtype=torch.int8, device=dev)
    grid = torch.ones(pages, h, dtype=torch.float32, device=dev)
    for kind, channel, unit in (("k", strong, 4), ("v", torch.ones_like(strong), 2)):
        codes = torch.empty(pages, h, page, d // 2, dtype=torch.uint8, device=dev)
        meta = torch.empty(pages, h, page, d // group, 2, dtype=torch.float16, device=dev)
        for p in range(0, pages, 1024):
            m = min(1024, pages - p)
            x = torch.randn(m, h, page, d, generator=gen, device=dev)
            x = (x + torch.randn(m, h, 1, d, generator=gen, device=dev)) * channel[:, None]
            q, s, z = _quantize(x.to(torch.bfloat16), group)
            q = q.flatten(-2)
            codes[p:p + m] = _pack(q, unit)
            meta[p:p + m] = torch.stack((s, z), -1).to(torch.float16)
            if kind == "k":
                bounds[p:p + m], grid[p:p + m] = _bounds(_values(q, meta[p:p + m]),
                                                         live[p:p + m, None].expand(m, h, page))
        meta.masked_fill_(~live[:, None, :, None, None], float("nan"))
        state[kind + "_codes"], state[kind + "_meta"] = codes, meta
    # the pages of the new rows are not up to date yet
    for b, (m, t) in enumerate(zip(lens, rows)):
        ids = order[sum(need[:b]) + max(0, m - t) // page:sum(need[:b + 1])].long()
        bounds[ids] = 0
        grid[ids] = 1
    state["bounds"], state["grid"] = bounds, grid
    state["q"] = torch.randn(n, hq, d, generator=gen, device=dev).to(torch.bfloat16)
    state["pages"], state["first"], state["last"] = case["pages"], case["first"], case["last"]
    state["out"] = torch.zeros(n, hq, d, dtype=torch.bfloat16, device=dev)
    state["lists"] = torch.zeros(n, h, case["pages"], dtype=torch.int32, device=dev)
    state["lens"] = torch.zeros(n, dtype=torch.int32, device=dev)
    return state


def _prepare_verify(case, gen, dev):
    lens, rows = _lengths(case)
    n, v = sum(rows), case["vocab"]
    dtype = getattr(torch, case["dtype"])
    first = torch.tensor([sum(rows[:b]) for b in range(len(rows) + 1)], dtype=torch.int32, device=dev)
    seq = torch.repeat_interleave(torch.arange(len(rows), device=dev), torch.tensor(rows, device=dev))
    # a draft model's logits and a target's that agrees with it for the most part: row r of the
    # draft made row r's token, and row r - 1 of the target judges it
    base = 3 * torch.randn(n + 1, v, generator=gen, device=dev)
    target = (base[1:] + 0.5 * torch.randn(n, v, generator=gen, device=dev)).to(dtype)
    draft = base[:-1].to(dtype)
    del base
    temperature = 0.6 + 0.6 * torch.rand(len(rows), generator=gen, device=dev)
    if case["greedy"]:
        temperature = temperature * (torch.arange(len(rows), device=dev) % 2)
    hot = temperature.clamp(min=1e-3)[seq]
    noise = -torch.log(-torch.log(torch.rand(n, v, generator=gen, device=dev).clamp(1e-9, 1 - 1e-7)))
    tokens = (draft.float() + noise * hot[:, None]).argmax(-1).to(torch.int32)
    del noise
    if case["kind"] == "probabilities":
        target = torch.softmax(target.float() / hot[:, None], -1).to(dtype)
        draft = torch.softmax(draft.float() / hot[:, None], -1).to(dtype)
    return {"target": target, "draft": draft if case["drafts"] == "dense" else None, "tokens": tokens,
            "logits": case["kind"] == "logits", "temperature": temperature if case["kind"] == "logits" else None,
            "uniform": torch.rand(n, generator=gen, device=dev), "n_rows": n, "uniform_rows": not case["ragged_rows"],
            "row_starts": first if case["ragged_rows"] else None, "seqs": len(rows),
            "seq_lens": torch.full((len(rows),), 5000, dtype=torch.int32, device=dev),
            "out": (torch.zeros(n, dtype=torch.int32, device=dev),
                    torch.zeros(len(rows), dtype=torch.int32, device=dev),
                    torch.zeros(len(rows), dtype=torch.int32, device=dev))}


# -------------------------------------------------------------------- one pass

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(st):
    import w4a16_decode_matmul_b200 as wq
    if st["op"] == "rotary":
        return wq.rotary(st["x"], st["positions"], st["rot"], inverse=st["inverse"], out=st["out"])
    if st["op"] == "verify":
        return wq.verify_drafts(st["target"], st["tokens"], st["uniform"], draft=st["draft"],
                                seqs=st["seqs"], row_starts=st["row_starts"], logits=st["logits"],
                                temperature=st["temperature"], seq_lens=st["seq_lens"], out=st["out"],
                                workspace=st["workspace"])
    batch = (st["seq_lens"], st["page_table"], st["row_starts"])
    if st["op"] == "write":
        wq.kv4_write_rotary(st["q"], st["k"], st["v"], st["cache"], st["rot"], *batch, out=st["q_out"])
        wq.kv4_read(st["cache"], *batch, out=st["out"])
        return [st["q_out"], *st["out"]]
    wq.kv4_sparse_attention(st["q"], st["cache"], st["handle"], *batch, max_pages=st["pages"],
                            first=st["first"], last=st["last"], scale=st["scale"], out=st["out"],
                            lists=st["lists"], lens=st["lens"], workspace=st["workspace"])
    # whole numbers all but the first: the pages, tokens of the lists, and the pages' bounds with
    # their grids, exact by definition
    return [st["out"], st["lists"], st["lens"], st["bounds"], st["grid"]]


def _run_plain(st):
    return {"rotary": _plain_rotary, "write": _plain_write, "sparse": _plain_sparse,
            "verify": _plain_verify}[st["op"]](st)


def _turns(st, positions):
    """Cosines and sines [rows, 1, dim/2] in 32 bits of the positions' angles, which are products in 64."""
    angle = positions.to(torch.float64)[:, None, None] * st["freqs"].to(torch.float64)
    # the amplitude is a number of 32 bits, as the package takes it
    amplitude = torch.tensor(st["amplitude"], dtype=torch.float32).item()
    return (amplitude * torch.cos(angle)).to(torch.float32), (amplitude * torch.sin(angle)).to(torch.float32)


def _rotate(x, c, s, interleaved):
    """x [rows, heads, D] in the type it is to be computed in."""
    half = c.shape[-1]
    turned, rest = x[..., :2 * half], x[..., 2 * half:]
    a, b = (turned[..., 0::2], turned[..., 1::2]) if interleaved else (turned[..., :half], turned[..., half:])
    a, b = a * c - b * s, b * c + a * s
    return torch.cat(((torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)), rest), -1)


def _plain_rotary(st):
    c, s = _turns(st, st["positions"])
    st["out"].copy_(_rotate(st["x"].to(torch.float32), c, -s if st["inverse"] else s, st["interleaved"]))
    return st["out"]


def _starts(st):
    if st["row_starts"] is not None:
        return st["row_starts"].long()
    b = st["seq_lens"].numel()
    return torch.arange(b + 1, device=st["seq_lens"].device) * (st["n_rows"] // b)


def _slots(st):
    """Sequence, token of every row that holds one, and which rows those are."""
    starts = _starts(st)
    row = torch.arange(st["n_rows"], device=starts.device)
    b = torch.searchsorted(starts, row, right=True) - 1
    pos = st["seq_lens"].long()[b] - starts[b + 1] + row
    return b, pos, pos >= 0


def _plain_write(st):
    b, pos, live = _slots(st)
    c, s = _turns(st, pos)
    st["q_out"].copy_(_rotate(st["q"].to(torch.float32), c, s, st["interleaved"]))
    # keys in 64 bits, rounded to 32 and to 16: next to a border of the codes a bit of a key is a step of its value
    k = _rotate(st["k"].to(torch.float64), c.to(torch.float64), s.to(torch.float64), st["interleaved"])
    k = k.to(torch.float32).to(torch.bfloat16)
    b, pos = b[live], pos[live]
    at = (st["page_table"][b, pos // st["page"]].long(), slice(None), pos % st["page"])
    for x, kind, unit, out in ((k, "k", 4, st["out"][0]), (st["v"], "v", 2, st["out"][1])):
        q, scale, zero = _quantize(x[live], st["group"])
        st[kind + "_codes"][at] = _pack(q.flatten(-2), unit)
        st[kind + "_meta"][at] = torch.stack((scale, zero), -1).to(torch.float16)
        out[live] = _values(_unpack(st[kind + "_codes"][at], unit), st[kind + "_meta"][at]).to(torch.bfloat16)
    return [st["q_out"], *st["out"]]


def _plain_sparse(st):
    page, dev = st["page"], st["q"].device
    b, pos, live = _slots(st)
    lens, table = st["seq_lens"].long(), st["page_table"].long()
    # ---- bounds of the pages that the rows are in
    bl, pl = b[live], pos[live]
    ids = table[bl, pl // page]
    there = (pl // page * page)[:, None] + torch.arange(page, device=dev) < lens[bl][:, None]
    keys = _values(_unpack(st["k_codes"][ids], 4), st["k_meta"][ids])            # [rows, H, P, D]
    st["bounds"][ids], st["grid"][ids] = _bounds(keys, there[:, None].expand(keys.shape[:3]))
    # ---- scores of all pages of a sequence, for its rows at once; in 64 bits, where they are exact
    seqs, h = lens.numel(), st["bounds"].shape[1]
    t = st["n_rows"] // seqs
    q = st["q"].to(torch.float32).unflatten(1, (h, -1))                          # [rows, H, R, D]
    q8 = torch.round(q / _power(q.abs().amax((-2, -1)))[..., None, None]).to(torch.float64)
    up_down = torch.cat((q8.clamp(max=0).sum(2), q8.clamp(min=0).sum(2)), -1)    # [rows, H, 2 D]
    table = table[:, :st["width"]]
    box = st["bounds"][table].flatten(-2).to(torch.float64)                      # [B, n, H, 2 D]
    score = torch.matmul(up_down.unflatten(0, (seqs, t)).transpose(1, 2), box.permute(0, 2, 3, 1))
    score = score.to(torch.float32) * st["grid"][table].transpose(1, 2)[:, :, None]
    score = score.transpose(1, 2).flatten(0, 1)                                  # [rows, H, n]
    # ---- the first, the last and the best
    limit = (pos + 1).clamp(min=0)
    n = (limit + page - 1) // page
    j = torch.arange(st["width"], device=dev)
    keep = (j < st["first"]) | (j >= (n - st["last"])[:, None])
    score = torch.where(keep[:, None], math.inf, score)
    score = torch.where((j < n[:, None])[:, None], score, -math.inf)
    best = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :st["pages"]]
    count = n.clamp(max=st["pages"])
    k = best.shape[-1]
    used = torch.arange(k, device=dev) < count[:, None]
    best = torch.sort(torch.where(used[:, None], best, st["width"]), -1).values
    chosen = table[b[:, None, None], best.clamp(max=st["width"] - 1)]
    st["lists"].fill_(-1)
    st["lists"][..., :k] = torch.where(used[:, None], chosen, -1)
    st["lens"].copy_(torch.where(count > 0, (count - 1) * page + limit - (n - 1) * page, 0))
    # ---- attention over them
    heads = torch.arange(h, device=dev)[:, None]
    k_ = _values(_unpack(st["k_codes"][chosen, heads], 4), st["k_meta"][chosen, heads]).flatten(2, 3)
    v_ = _values(_unpack(st["v_codes"][chosen, heads], 2), st["v_meta"][chosen, heads]).flatten(2, 3)
    seen = torch.arange(k_.shape[2], device=dev) < st["lens"][:, None]           # [rows, tokens]
    v_ = torch.where(seen[:, None, :, None], v_, 0)
    s = torch.matmul(q, k_.transpose(-1, -2)) * st["scale"]
    s = torch.where(seen[:, None, None], s, -math.inf)
    top = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(top == -math.inf, 0, top))
    o = torch.matmul(e, v_) / e.sum(-1, keepdim=True).clamp(min=1e-30)
    st["out"].copy_(o.flatten(1, 2))
    return [st["out"], st["lists"], st["lens"], st["bounds"], st["grid"]]


def _plain_verify(st):
    """In 64 bits: a token is chosen by where a number falls between sums over the vocabulary."""
    dev, n, seqs = st["target"].device, st["n_rows"], st["seqs"]
    starts = torch.arange(seqs + 1, device=dev) * (n // seqs) if st["row_starts"] is None else st["row_starts"].long()
    row = torch.arange(n, device=dev)
    b = torch.searchsorted(starts, row, right=True) - 1
    p, q = st["target"].to(torch.float64), None if st["draft"] is None else st["draft"].to(torch.float64)
    if st["logits"]:
        t = st["temperature"].to(torch.float64)[b, None]
        p, q = _distribution(p, t), None if q is None else _distribution(q, t)
    u, x = st["uniform"].to(torch.float64), st["tokens"].long()
    drafted = row > starts[b]
    judged = p[(row - 1).clamp(min=0), x]
    drawn = torch.ones_like(judged) if q is None else q[row, x]
    fails = drafted & ~(u * drawn < judged)
    # accepted: the drafts before a sequence's first that fails
    count = starts[1:] - starts[:-1]
    accepted = (count - 1).scatter_reduce(0, b, torch.where(fails, row - starts[b] - 1, 1 << 30), "amin")
    at = starts[:-1] + accepted
    mass, whole = p[at], p[at]
    refused = accepted < count - 1
    after = (at + 1).clamp(max=n - 1)
    if q is None:
        less = mass.scatter(1, x[after, None], 0.0)
    else:
        less = (mass - q[after]).clamp(min=0)
    mass = torch.where(refused[:, None] & (less.sum(-1, keepdim=True) > 0), less, whole)
    total = torch.cumsum(mass, -1)
    found = torch.searchsorted(total, u[starts[:-1], None] * total[:, -1:], right=True)[:, 0]
    last = torch.where(mass > 0, torch.arange(mass.shape[1], device=dev), -1).amax(-1)
    found = torch.minimum(found, last)
    i = row - starts[b]
    fed = x[(row + 1).clamp(max=n - 1)]
    tokens, accept_out, lens_out = st["out"]
    tokens.copy_(torch.where(i < accepted[b], fed, torch.where(i == accepted[b], found[b], -1)))
    accept_out.copy_(accepted)
    lens_out.copy_(st["seq_lens"] - (count - 1 - accepted))
    return list(st["out"])


def _distribution(x, t):
    top = x.amax(-1, keepdim=True)
    e = torch.exp((x - top) / torch.where(t > 0, t, 1))
    e = e / e.sum(-1, keepdim=True)
    # temperature 0: the first of the largest
    at = torch.arange(x.shape[-1], device=x.device)
    first = torch.where(x == top, at, x.shape[-1]).amin(-1, keepdim=True)
    return torch.where(t > 0, e, (at == first).to(torch.float64))


# --------------------------------------------------------- the same in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    return {"rotary": _exact_rotary, "write": _exact_write, "sparse": _exact_sparse,
            "verify": _exact_verify}[case["op"]](case, st)


def _turned(x, pos, st, sign=1.0):
    """The rotation as a product of complex numbers; x [n, H, D], pos [n], 64 bits."""
    f = st["freqs"].double()
    a = pos.double()[:, None] * f[None]
    amplitude = torch.tensor(st["amplitude"], dtype=torch.float32).double().item()
    turn = torch.complex((amplitude * torch.cos(a)).float().double(),
                         (sign * amplitude * torch.sin(a)).float().double())[:, None]
    n = f.numel()
    y = x.double().clone()
    if st["interleaved"]:
        z = torch.view_as_complex(y[..., :2 * n].reshape(*y.shape[:-1], n, 2).contiguous()) * turn
        y[..., :2 * n] = torch.view_as_real(z).reshape(*y.shape[:-1], 2 * n)
    else:
        z = torch.complex(y[..., :n].contiguous(), y[..., n:2 * n].contiguous()) * turn
        y[..., :n], y[..., n:2 * n] = z.real, z.imag
    return y


def _exact_rotary(case, st):
    return _turned(st["x"], st["positions"], st, -1.0 if case["inverse"] else 1.0)


def _exact_write(case, st):
    lens, rows = _lengths(case)
    h, d, group = case["kv_heads"], case["head_dim"], case["group"]

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

    pos = torch.cat([torch.arange(n - t, n) for n, t in zip(lens, rows)]).cuda()
    live = (pos >= 0)[:, None, None]
    # keys are rounded to 32 bits and to 16 before they are quantized, by definition
    k = _turned(st["k"], pos, st).float().bfloat16()
    return [_turned(st["q"], pos, st), torch.where(live, rounded(k), 0), torch.where(live, rounded(st["v"]), 0)]


def _grid_of(top):
    e = math.floor(math.log2(top)) - 8 if top > 0 else 0
    while top > 127 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def _exact_sparse(case, st):
    lens, rows = _lengths(case)
    h, hq, d, page = (case[k] for k in ("kv_heads", "q_heads", "head_dim", "page"))
    r, table = hq // h, st["page_table"].tolist()
    bounds, grid = st["bounds"].clone(), st["grid"].clone()

    def rows_of(kind, ids, head):
        """Values of whole pages of one head, 64 bits: [pages * page, D]."""
        units, size = (4, 4) if kind == "k" else (8, 2)
        c = st[kind + "_codes"][ids, head].reshape(-1, units, d // 32, size)
        c = c.permute(0, 2, 1, 3).reshape(-1, d // 2).long()
        u = torch.stack((c % 16, c // 16), -1).reshape(-1, d // case["group"], case["group"]).double()
        m = st[kind + "_meta"][ids, head].reshape(-1, d // case["group"], 2).double()
        return ((u - m[..., 1:2]) * m[..., 0:1]).reshape(-1, d)

    for b, (n, t) in enumerate(zip(lens, rows)):
        for j in range(max(0, n - t) // page, (n + page - 1) // page):
            for head in range(h):
                k = rows_of("k", torch.tensor([table[b][j]], device="cuda"), head)[:n - j * page]
                g = _grid_of(float(k.abs().max()))
                bounds[table[b][j], head, 0] = torch.floor(k.min(0).values / g).to(torch.int8)
                bounds[table[b][j], head, 1] = torch.ceil(k.max(0).values / g).to(torch.int8)
                grid[table[b][j], head] = g
    out = torch.zeros(sum(rows), hq, d, dtype=torch.float64, device="cuda")
    lists = torch.full((sum(rows), h, case["pages"]), -1, dtype=torch.int32, device="cuda")
    counts, at = [], 0
    for b, (n, t) in enumerate(zip(lens, rows)):
        for i in range(t):
            seen = n - t + i + 1
            pages = (seen + page - 1) // page if seen > 0 else 0
            kept = min(pages, case["pages"])
            counts.append(0 if seen <= 0 else seen - (pages - kept) * page)
            ids = torch.tensor(table[b][:pages], device="cuda", dtype=torch.long)
            for head in range(h if pages else 0):
                q = st["q"][at, head * r:(head + 1) * r].double()
                q8 = torch.round(q / _grid_of(float(q.abs().max())))
                lo, hi = bounds[ids, head, 0].double(), bounds[ids, head, 1].double()
                pos = torch.where(q8 > 0, q8, torch.zeros_like(q8)).sum(0)
                neg = torch.where(q8 < 0, q8, torch.zeros_like(q8)).sum(0)
                score = ((hi * pos + lo * neg).sum(-1).float() * grid[ids, head]).tolist()
                must = [j for j in range(pages) if j < case["first"] or j >= pages - case["last"]]
                free = [j for j in range(pages) if j not in set(must)]
                if pages > kept:
                    free = sorted(free, key=lambda j: (-score[j], j))[:kept - len(must)]
                mine = ids[torch.tensor(sorted(must + free), device="cuda")]
                lists[at, head, :kept] = mine.int()
                k, v = rows_of("k", mine, head)[:counts[-1]], rows_of("v", mine, head)[:counts[-1]]
                w = torch.softmax(q @ k.T / math.sqrt(d), -1)
                out[at, head * r:(head + 1) * r] = w @ v
            at += 1
    return [out, lists, torch.tensor(counts, dtype=torch.int32), bounds, grid]


def _exact_verify(case, st):
    _, rows = _lengths(case)
    tokens, accepted, lens, at = [], [], [], 0
    for b, t in enumerate(rows):
        def mass(x):
            x = x.double()
            if case["kind"] != "logits":
                return x
            hot = float(st["temperature"][b])
            if hot == 0:
                one = torch.zeros_like(x)
                one[int((x == x.max()).nonzero()[0])] = 1
                return one
            return torch.softmax(x / hot, -1)

        fed, u = st["tokens"][at:at + t].tolist(), st["uniform"][at:at + t].tolist()
        a = 0
        while a < t - 1:
            drawn = 1.0 if st["draft"] is None else float(mass(st["draft"][at + a + 1])[fed[a + 1]])
            if not u[a + 1] * drawn < float(mass(st["target"][at + a])[fed[a + 1]]):
                break
            a += 1
        p = mass(st["target"][at + a])
        if a < t - 1:
            if st["draft"] is None:
                left = p.clone()
                left[fed[a + 1]] = 0
            else:
                left = (p - mass(st["draft"][at + a + 1])).clamp(min=0)
            p = left if float(left.sum()) > 0 else p
        total = p.cumsum(0)
        hit = (total > u[0] * total[-1]).nonzero()
        chosen = int(hit[0]) if len(hit) else int((p > 0).nonzero()[-1])
        tokens += fed[1:a + 1] + [chosen] + [-1] * (t - 1 - a)
        accepted.append(a)
        lens.append(5000 - (t - 1 - a))
        at += t
    return [torch.tensor(x, dtype=torch.int32) for x in (tokens, accepted, lens)]
