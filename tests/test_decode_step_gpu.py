"""A step of speculative decoding as a decoder runs it, from a captured graph: the fused
projection in 4-bit weights, queries and keys at their positions, keys and values into
the 4-bit cache, attention over chosen pages, the logits in 4-bit weights, and the
verification of the drafts, which says where the next step goes on."""
import numpy as np
import pytest
import torch

import synth
from tests import kv4_ref as ref
from tests.gpu_util import wq
from tests.test_kv4_gpu import COUNTERS, assert_cache, images, ints, new_cache, starts_of
from tests.test_kv4_select_gpu import attention_over, expected_bounds, expected_pages, key_values
from tests.test_rotary_gpu import check as check_turned
from tests.test_rotary_gpu import expect as expect_keys
from tests.test_verify_gpu import expected as expected_tokens

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,group,kv_heads,gqa,page,drafted", [(64, 32, 2, 4, 16, 3),
                                                               (128, 64, 1, 2, 32, 1)])
def test_steps_of_speculative_decoding(d, group, kv_heads, gqa, page, drafted):
    mod = wq()
    hidden, vocab, q_heads, t = 256, 1024, kv_heads * gqa, drafted + 1
    lens, max_pages, steps = [150, 333, 40], 5, 5
    seqs = len(lens)
    wide = (q_heads + 2 * kv_heads) * d
    w_qkv = mod.quantize(synth.weight(wide, hidden, seed=1).cuda(), bits=4, group=64)
    w_out = mod.quantize(synth.weight(hidden, q_heads * d, seed=2).cuda(), bits=4, group=64)
    w_head = mod.quantize(synth.weight(vocab, hidden, seed=3).cuda(), bits=4, group=64)
    embed = synth.activation(vocab, hidden, seed=4).cuda()
    table, pages = ref.random_batch(4, [n + steps * t for n in lens], page)
    cache = new_cache(pages, kv_heads, d, page, group)
    bounds = mod.kv4_bounds(cache)
    rot = mod.Rotary(mod.rotary_frequencies(d, 500.0).cuda())
    n, tb, ws = ints(lens), ints(table), mod.kv4_workspace()
    vws = mod.verify_workspace(seqs * t)

    # ---- prompts
    starts = ints(starts_of(lens))
    x = synth.activation(sum(lens), hidden, seed=7).cuda()
    qkv = mod.matmul(x, w_qkv, out_dtype=torch.bfloat16).view(-1, q_heads + 2 * kv_heads, d)
    q, k, v = qkv[:, :q_heads], qkv[:, q_heads:q_heads + kv_heads], qkv[:, q_heads + kv_heads:]
    mod.kv4_write_rotary(q, k, v, cache, rot, n, tb, starts)
    mod.kv4_update_bounds(cache, bounds, n, tb, starts, rows=sum(lens))
    codes, grid = bounds.codes.cpu().numpy().astype(np.int64), bounds.grid.cpu().numpy()
    expected_bounds(key_values(cache), lens, lens, table, page, codes, grid)
    assert np.array_equal(bounds.codes.cpu().numpy(), codes)

    # ---- a step: tokens [seqs, t], the first of which stands
    tokens = ints(np.random.default_rng(1).integers(0, vocab, (seqs, t)))
    drafts = torch.zeros(seqs, drafted, dtype=torch.int32, device="cuda")
    draft_logits = torch.zeros(seqs * t, vocab, device="cuda")
    uniform = torch.zeros(seqs * t, device="cuda")
    hot = torch.tensor([0.8, 1.3, 0.0], device="cuda")
    out = (torch.zeros(seqs * t, dtype=torch.int32, device="cuda"), ints([0] * seqs), n)
    kept = {}

    def step():
        tokens[:, 1:] = drafts
        n.add_(t)
        kept["n"] = n.clone()
        kept["fed"] = tokens.clone()
        qkv = mod.matmul(embed[tokens.view(-1).long()], w_qkv, out_dtype=torch.bfloat16)
        qkv = qkv.view(-1, q_heads + 2 * kv_heads, d)
        kept["qkv"] = qkv.clone()
        q = qkv[:, :q_heads]
        mod.kv4_write_rotary(q, qkv[:, q_heads:q_heads + kv_heads], qkv[:, q_heads + kv_heads:],
                             cache, rot, n, tb, out=q)
        o, lists, held = mod.kv4_sparse_attention(q, cache, bounds, n, tb, max_pages=max_pages,
                                                  workspace=ws)
        y = mod.matmul(o.view(seqs * t, -1), w_out, out_dtype=torch.bfloat16)
        logits = mod.matmul(y, w_head)
        mod.verify_drafts(logits, tokens.view(-1), uniform, draft=draft_logits, seqs=seqs,
                          logits=True, temperature=hot, seq_lens=n, out=out, workspace=vws)
        tokens[:, :1] = out[0].view(seqs, t).gather(1, out[1].long()[:, None])
        kept.update(q=q, o=o, lists=lists, held=held, logits=logits)

    def fill(seed):
        """What the draft model would give: logits near enough to be accepted now and then."""
        g = torch.Generator(device="cuda").manual_seed(seed)
        draft_logits.copy_(torch.randn(seqs * t, vocab, generator=g, device="cuda") * 0.3)
        uniform.copy_(torch.rand(seqs * t, generator=g, device="cuda"))
        drafts.copy_(torch.randint(0, vocab, drafts.shape, generator=g, device="cuda",
                                   dtype=torch.int32))

    def check(want, codes, grid, before):
        torch.cuda.synchronize()
        assert mod.get_device_error() == 0
        now = [m + t for m in before]
        assert kept["n"].tolist() == now
        rows = [t] * seqs
        qkv = kept["qkv"]
        positions = [m - t + i for m in now for i in range(t)]
        held, _ = ref.places(now, rows, table, page)
        expect_keys(qkv[:, q_heads:q_heads + kv_heads], positions, rot, held,
                    qkv[:, q_heads + kv_heads:], want, cache)
        assert_cache(cache, want)
        check_turned(kept["q"], qkv[:, :q_heads], positions, rot.freqs.cpu(), False)
        expected_bounds(key_values(cache), now, rows, table, page, codes, grid)
        assert np.array_equal(bounds.codes.cpu().numpy(), codes)
        assert np.array_equal(bounds.grid.cpu().numpy(), grid)
        lists, count = expected_pages(kept["q"].double().cpu().numpy(), codes, grid, now, rows, table,
                                      page, max_pages, 1, 2, seqs * t)
        assert np.array_equal(kept["lists"].cpu().numpy(), lists)
        assert np.array_equal(kept["held"].cpu().numpy(), count)
        o, e = attention_over(kept["q"], cache, lists, count, d ** -0.5)
        ref.check(kept["o"], o, e)
        tok, acc, left = expected_tokens(kept["logits"].float().cpu().numpy(),
                                         kept["fed"].view(-1).cpu().numpy(), uniform.cpu().numpy(),
                                         draft_logits.cpu().numpy(), rows, True,
                                         hot.cpu().numpy(), now)
        assert out[0].tolist() == tok and out[1].tolist() == acc and n.tolist() == left
        assert not ws[:COUNTERS].any()
        return left

    lengths, want = lens, images(cache)
    fill(100)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()                        # the first outside the graph
    stream.synchronize()
    lengths = check(want, codes, grid, lengths)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step()
    for i in range(1, steps):
        fill(100 + i)
        graph.replay()
        torch.cuda.synchronize()
        lengths = check(want, codes, grid, lengths)
