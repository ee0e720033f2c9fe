"""GPU: the example that quantizes, packs and runs a block, against float32 on the dequantized weights."""
import importlib.util
import os

import pytest
import torch

from parity import say

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "packed_block.py")


def _module():
    spec = importlib.util.spec_from_file_location("packed_block", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("lengths,tokens,chunk", [((70, 1, 33), 4, 32), ((130,), 2, 200)])
def test_prompts_in_chunks_then_tokens(lengths, tokens, chunk):
    say("block:", lengths, tokens, chunk)
    m = _module()
    torch.manual_seed(1)
    block = m.Block(dim=512, heads=8, kv_heads=2, head_dim=64, ffn=640, requests=len(lengths), pages=64)
    prompts = [torch.randn(n + tokens, 512, device="cuda").bfloat16() for n in lengths]
    for x, y in zip(prompts, m.generate(block, prompts, tokens, chunk)):
        want = block.whole(x)
        # ten roundings to bfloat16 (relative error 2^-8 at most, 2^-9 in the root mean square of each) on the way
        assert float((y.float() - want).norm() / want.norm()) < 10 * 2.0 ** -9
    assert block.ctx.tolist() == [n + tokens for n in lengths]
    assert int(block.n_free) == 64 - sum(-(-(n + tokens) // 16) for n in lengths)


def test_replayed_token_steps():
    """Token steps replayed as a graph, with eager work between, equal the same steps called one by one."""
    m = _module()
    kw = dict(dim=512, heads=8, kv_heads=2, head_dim=64, ffn=640, requests=2, pages=64, seed=3)
    a, b = m.Block(**kw), m.Block(**kw)
    torch.manual_seed(2)
    prompt = torch.randn(60, 512, device="cuda").bfloat16()
    new = torch.tensor([40, 20], dtype=torch.int32, device="cuda")
    one = torch.ones(2, dtype=torch.int32, device="cuda")
    x = torch.randn(2, 512, device="cuda").bfloat16()
    for block in (a, b):
        block.step(prompt, new, 40)
        block.step(x, one, 1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = a.step(x, one, 1)
    for _ in range(20):
        x.copy_(torch.randn_like(x))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, b.step(x, one, 1))
        assert torch.equal(a.ctx, b.ctx) and torch.equal(a.n_free, b.n_free)
