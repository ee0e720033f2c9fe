"""A transformer block quantized, packed and run: prompts in chunks, then tokens, over a paged cache.

    python examples/packed_block.py

The weights (random) are quantized with the minimax scales of this library and packed as GPTQ-v1 tensors, layer by
layer: each on the activations that the calibration windows have behind the layers packed before it, which the serving
operators run.  The block is then run by them: one block map per step, the q-k-v projection, the cache write,
attention over the pages, the output projection with its residual, the gated feed-forward layer.  The result is
compared with the same block in float32 on the dequantized weights and the whole sequences at once, and a step of
one token per request is timed, call by call and replayed as a graph.
"""
import math
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import post_weight_quantization_group_amd as cq  # noqa: E402


class PackedLinear:
    """W [out, in] as qweight and scales, quantized for the activations x [E, T, in]."""

    def __init__(self, weight, x):
        out, inp = weight.shape
        d = cq.environment_diagonals(x)
        r = cq.quantize_groups(weight.reshape(-1, 128), d, inp // 128, method="bounded")
        codes, scales = r["codes"].reshape(out, inp), r["scales"].reshape(out, inp // 128)
        self.qweight, self.scales = cq.pack_gptq_v1(codes, scales, out, inp)
        self.dense = codes.float() * scales.view(torch.float16).float().repeat_interleave(128, dim=1)

    def __call__(self, x, **kw):
        return cq.w4a16_linear(x, self.qweight, self.scales, **kw)


def rotate(x, positions):
    """Rotary embedding of x [T, heads, D] at int positions [T], in float32."""
    half = x.shape[-1] // 2
    angle = positions.float()[:, None] * 10000.0 ** (-torch.arange(half, device=x.device).float() / half)
    cos, sin = angle.cos()[:, None], angle.sin()[:, None]
    a, b = x[..., :half].float(), x[..., half:].float()
    return torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1).to(x.dtype)


class Block:
    """Pre-norm attention and a gated feed-forward layer, with its paged cache."""

    def __init__(self, dim=1024, heads=8, kv_heads=2, head_dim=128, ffn=3584, pages=256, page=16, requests=3,
                 max_kv=1024, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def rand(*shape):
            return torch.randn(shape, generator=g, device=device)

        self.H, self.Hkv, self.D, self.page, self.max_kv = heads, kv_heads, head_dim, page, max_kv
        self.k, self.v = (torch.zeros((pages, kv_heads, page, head_dim), dtype=torch.bfloat16, device=device)
                          for _ in range(2))
        self.free = torch.randperm(pages, generator=g, device=device).int()
        # four environments of a window each, through every layer as soon as it is packed
        E, n = 4, 64
        self._requests(E)
        x = rand(E * n, dim).bfloat16()
        m = cq.kv_block_map(self.ctx, torch.full_like(self.ctx, n), self.free, self.n_free, self.table, page, E * n)
        h = F.rms_norm(x, x.shape[-1:])
        self.qkv = PackedLinear(rand((heads + 2 * kv_heads) * head_dim, dim) * dim ** -0.5, h.view(E, n, -1))
        a = self._attend(self.qkv(h), m, n)
        self.out = PackedLinear(rand(dim, heads * head_dim) * dim ** -0.5, a.view(E, n, -1))
        x = self.out(a, residual=x)
        h = F.rms_norm(x, x.shape[-1:])
        self.gate_up = PackedLinear(rand(2 * ffn, dim) * dim ** -0.5, h.view(E, n, -1))
        h = self.gate_up(h, activation="silu", gated=True)
        self.down = PackedLinear(rand(dim, ffn) * ffn ** -0.5, h.view(E, n, -1))
        self._requests(requests)

    def _requests(self, n):
        """n empty requests, all pages free."""
        device = self.k.device
        self.table = torch.full((n, self.max_kv // self.page), -1, dtype=torch.int32, device=device)
        self.n_free = torch.tensor([self.k.shape[0]], dtype=torch.int32, device=device)
        self.ctx = torch.zeros(n, dtype=torch.int32, device=device)

    def _attend(self, qkv, m, max_q):
        """Attention's output [T, heads * D] of the packed rows qkv, whose keys and values go into the cache."""
        T = qkv.shape[0]
        qkv = qkv.view(T, self.H + 2 * self.Hkv, self.D)
        q = rotate(qkv[:, : self.H], m["positions"])
        k = rotate(qkv[:, self.H: self.H + self.Hkv], m["positions"])
        cq.kv_cache_write(k, qkv[:, self.H + self.Hkv:], self.k, self.v, m["slots"])
        return cq.paged_attention(q, self.k, self.v, self.table, m["cu_q"], m["kv_len"], max_q, self.max_kv).view(T, -1)

    def step(self, x, new, max_q):
        """x [T, dim] of the requests' new tokens (int32 [R] of them, at most max_q each), packed."""
        T = x.shape[0]
        m = cq.kv_block_map(self.ctx, new, self.free, self.n_free, self.table, self.page, T)
        a = self._attend(self.qkv(F.rms_norm(x, x.shape[-1:])), m, max_q)
        x = self.out(a, residual=x)
        h = self.gate_up(F.rms_norm(x, x.shape[-1:]), activation="silu", gated=True)
        x = self.down(h, residual=x)
        self.ctx.copy_(m["kv_len"])
        self.n_free.copy_(m["n_left"])
        return x

    def whole(self, x):
        """The same block in float32 on the dequantized weights, x [n, dim] one whole sequence."""
        x = x.float()
        n = x.shape[0]
        at = torch.arange(n, device=x.device)
        qkv = (F.rms_norm(x, x.shape[-1:]) @ self.qkv.dense.T).view(n, -1, self.D)
        q, k = rotate(qkv[:, : self.H], at), rotate(qkv[:, self.H: self.H + self.Hkv], at)
        v = qkv[:, self.H + self.Hkv:]
        G = self.H // self.Hkv
        s = torch.stack([q[:, h] @ k[:, h // G].T for h in range(self.H)]) / math.sqrt(self.D)
        p = torch.softmax(s.masked_fill(torch.ones_like(s).triu(1).bool(), -math.inf), dim=-1)
        a = torch.stack([p[h] @ v[:, h // G] for h in range(self.H)], dim=1).reshape(n, -1)
        x = x + a @ self.out.dense.T
        gate, up = (F.rms_norm(x, x.shape[-1:]) @ self.gate_up.dense.T).chunk(2, dim=-1)
        return x + (F.silu(gate) * up) @ self.down.dense.T


def generate(block, prompts, tokens, chunk=64):
    """Runs the prompts' rows in chunks, then `tokens` further rows of each one at a time; x of request r is
    prompts[r] [n_r + tokens, dim].  Returns the outputs, a tensor per request."""
    done = [0] * len(prompts)
    outs = [[] for _ in prompts]
    while any(d < p.shape[0] for d, p in zip(done, prompts)):
        new = [min(chunk, p.shape[0] - tokens - d) if d < p.shape[0] - tokens else min(1, p.shape[0] - d)
               for d, p in zip(done, prompts)]
        x = torch.cat([p[d:d + n] for d, n, p in zip(done, new, prompts)])
        y = block.step(x, torch.tensor(new, dtype=torch.int32, device=x.device), max(new))
        for r, part in enumerate(y.split(new)):
            outs[r].append(part)
            done[r] += new[r]
    return [torch.cat(o) for o in outs]


def main():
    torch.manual_seed(0)
    block = Block()
    lengths, tokens = (200, 77, 130), 20
    prompts = [torch.randn(n + tokens, 1024, device="cuda").bfloat16() for n in lengths]
    outs = generate(block, prompts, tokens)
    for r, (x, y) in enumerate(zip(prompts, outs)):
        want = block.whole(x)
        print(f"request {r}: {x.shape[0]} tokens, relative error {float((y.float() - want).norm() / want.norm()):.2e}")

    # a token per request: call by call, and replayed as one graph
    x = torch.randn(3, 1024, device="cuda").bfloat16()
    one = torch.ones(3, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block.step(x, one, 1)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block.step(x, one, 1)
    for name, run in (("calls", lambda: block.step(x, one, 1)), ("graph", graph.replay)):
        begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        run()
        begin.record()
        for _ in range(100):
            run()
        end.record()
        torch.cuda.synchronize()
        print(f"a token per request, {name}: {begin.elapsed_time(end) * 10:.1f} us")


if __name__ == "__main__":
    main()
