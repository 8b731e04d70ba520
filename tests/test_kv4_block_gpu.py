"""An attention block as a decoder runs it: the fused projection and the
output projection in 4-bit weights, keys and values into the 4-bit cache,
attention over it -- a prompt, then tokens one by one from a captured graph."""
import numpy as np
import pytest
import torch

import synth
from tests import kv4_ref as ref
from tests.gpu_util import wq
from tests.test_kv4_gpu import COUNTERS, ints, new_cache, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,group,kv_heads,gqa", [(64, 32, 2, 4), (128, 64, 1, 4)])
def test_prompt_then_tokens(d, group, kv_heads, gqa):
    mod = wq()
    hidden, q_heads, page = 512, kv_heads * gqa, 16
    wide = (q_heads + 2 * kv_heads) * d
    w_qkv = mod.quantize(synth.weight(wide, hidden, seed=1).cuda(), bits=4, group=128)
    w_out = mod.quantize(synth.weight(hidden, q_heads * d, seed=2).cuda(), bits=4, group=64)
    lens, steps = [45, 70], 6
    table, pages = ref.random_batch(4, [n + steps for n in lens], page)
    cache = new_cache(pages, kv_heads, d, page, group)
    n, tb, ws = ints(lens), ints(table), mod.kv4_workspace()
    scale = d ** -0.5

    def block(x, starts=None, max_rows=None):
        qkv = mod.matmul(x, w_qkv, out_dtype=torch.bfloat16).view(-1, q_heads + 2 * kv_heads, d)
        q, k = qkv[:, :q_heads], qkv[:, q_heads:q_heads + kv_heads]
        mod.kv4_write(k, qkv[:, q_heads + kv_heads:], cache, n, tb, starts)
        o = mod.kv4_attention(q, cache, n, tb, starts, max_rows=max_rows, workspace=ws)
        return qkv, o, mod.matmul(o.view(o.shape[0], -1), w_out)

    def check(qkv, o, y, now, rows):
        torch.cuda.synchronize()
        assert mod.get_device_error() == 0
        out, bound = reference(qkv[:, :q_heads], cache, now, rows, table, scale)
        ref.check(o, out, bound)
        # the cache holds this step's keys and values to half a quantization step
        k, v = mod.kv4_read(cache, n, tb, ints(np.cumsum([0, *rows])), rows=sum(rows))
        for got, x in ((k, qkv[:, q_heads:-kv_heads]), (v, qkv[:, -kv_heads:])):
            g = ref.to_half(x).float().unflatten(-1, (-1, group))
            span = g.amax(-1).clamp(min=0) - g.amin(-1).clamp(max=0)
            # s/2 with s at most a binary16 step above span/15 (2^-10, or 2^-24
            # where it is subnormal), and the read's bfloat16 rounding
            bound = (span / 30 * (1 + 2 ** -10) + 2 ** -24)[..., None]
            err = (got.float().unflatten(-1, (-1, group)) - g).abs()
            assert (err <= bound + 2 ** -8 * (g.abs() + bound)).all()
        dense = mod.dequantize(w_out).double()
        # dequantized weights are bfloat16 (2^-8), the product's own bound 1e-4
        flat = o.reshape(o.shape[0], -1).double()
        tol = (2 ** -8 + 1e-4) * (flat.abs() @ dense.abs().T) * (1 + 2 ** -8)
        assert ((y.double() - flat @ dense.T).abs() <= tol).all()

    rows = list(lens)
    x = synth.activation(sum(rows), hidden, seed=7).cuda()
    check(*block(x, ints(np.cumsum([0, *rows])), max(rows)), lens, rows)

    token = synth.activation(2, hidden, seed=8).cuda()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        n.add_(1)                     # the first token outside the graph
        got = block(token)
    stream.synchronize()
    check(*got, [m + 1 for m in lens], [1, 1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        n.add_(1)
        got = block(token)
    for step in range(2, steps + 1):
        token.copy_(synth.activation(2, hidden, seed=20 + step))
        graph.replay()
        check(*got, [m + step for m in lens], [1, 1])
    assert not ws[:COUNTERS].any()
