"""One decode step of a small mixture-of-experts layer on 4-bit weights and a
4-bit cache, with every product, the cache and the attention in this library:

  q, k, v   = three products of the normalised token with MXFP4 weights
  cache     <- k, v quantized into the sequence's next slot
  attention over the paged cache, its output product added to the token
  router    -> the top experts and their weights; mxfp4_moe_route sorts the routes
  experts   = gate/up products, SiLU gate, down products, their weighted sum

Run it on a GPU:  python examples/decode_step.py
It prints how far the step is from the same step in plain float32 torch on the
dequantized weights and cache (BF16 activations leave about 2^-8).
"""
import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import mxfp4_block_quantization_gb300 as mx  # noqa: E402


@dataclass
class Layer:
    """Sizes and quantized weights of one layer."""
    hidden: int = 512
    q_heads: int = 16
    kv_heads: int = 2
    head_dim: int = 64
    experts: int = 12
    width: int = 256
    top_k: int = 3
    page_size: int = 16


def dequantize_experts(codes, scales, rows, cols):
    per = scales.numel() // codes.shape[0]
    return torch.stack([mx.dequantize(codes[e], scales[e * per:(e + 1) * per], rows, cols)
                        for e in range(codes.shape[0])]).float()


class DecodeStep:
    """Weights quantized once; `step` runs one token for each sequence."""

    def __init__(self, layer: Layer, sequences: int, max_len: int, seed: int = 0, device="cuda"):
        self.layer = c = layer
        gen = torch.Generator(device=device).manual_seed(seed)

        def weight(*shape):
            return (torch.randn(shape, device=device, generator=gen) * shape[-1] ** -0.5).bfloat16()

        kv = c.kv_heads * c.head_dim
        self.wq = mx.quantize(weight(c.q_heads * c.head_dim, c.hidden))
        self.wkv = mx.quantize(weight(2 * kv, c.hidden))
        self.wo = mx.quantize(weight(c.hidden, c.q_heads * c.head_dim))
        self.router = weight(c.experts, c.hidden)
        # experts' weights: one tiled scale buffer per expert, one after another
        w13 = weight(c.experts, 2 * c.width, c.hidden)
        w2 = weight(c.experts, c.hidden, c.width)
        self.w13, self.w2 = (
            tuple(torch.cat(t) if t[0].dim() == 1 else torch.stack(t) for t in zip(*map(mx.quantize, w)))
            for w in (w13, w2))
        pages = -(-max_len // c.page_size)
        self.cache = mx.cache_alloc(sequences * pages, c.page_size, c.kv_heads, c.head_dim,
                                    device=device)
        order = torch.randperm(sequences * pages, device=device, generator=gen)
        self.table = order.view(sequences, pages).to(torch.int32)
        self.lens = torch.zeros(sequences, dtype=torch.int32, device=device)

    def slots(self):
        """The cache slot of each sequence's next position."""
        at = self.lens.long()
        page = self.table.gather(1, (at // self.layer.page_size).unsqueeze(1)).squeeze(1)
        return (page * self.layer.page_size + at % self.layer.page_size).to(torch.int32)

    def step(self, x):
        """x [sequences, hidden] BF16 -> the layer's output; the cache grows by one."""
        c, B = self.layer, x.shape[0]
        h = torch.nn.functional.rms_norm(x, (c.hidden,))
        q = mx.matvec(h, *self.wq).view(B, c.q_heads, c.head_dim)
        kv = mx.matvec(h, *self.wkv).view(B, 2, c.kv_heads, c.head_dim)
        mx.cache_write(kv[:, 0], kv[:, 1], self.slots(), self.cache)
        self.lens += 1
        o, _, _ = mx.cache_attention(q, self.cache, self.table, self.lens, c.head_dim ** -0.5)
        x = x + mx.matvec(o.view(B, -1), *self.wo)

        h = torch.nn.functional.rms_norm(x, (c.hidden,))
        ids, weights = mx.moe_topk(h.float() @ self.router.float().T, c.top_k, renormalize=False)
        self.chosen = ids.long()
        offsets, dest, rows, _ = mx.moe_route(ids, c.experts)
        gate_up, _ = mx.moe_matvec(h, rows, offsets, *self.w13)
        gate, up = gate_up.chunk(2, -1)
        y, _ = mx.moe_matvec((torch.nn.functional.silu(gate) * up).contiguous(), None, offsets,
                             *self.w2, out_dtype=torch.float32)
        return mx.moe_combine(y, dest, weights, residual=x)[0]

    def plain(self, x, k_cache, v_cache):
        """The last step in float32 on the dequantized weights, with the experts
        that it chose; k_cache and v_cache [sequences, positions, kv_heads,
        head_dim] are what the 4-bit cache holds, the step's positions among
        them."""
        c, B = self.layer, x.shape[0]

        def w(q, rows, cols):
            return mx.dequantize(*q, rows, cols).float()

        x = x.float()
        h = torch.nn.functional.rms_norm(x, (c.hidden,))
        q = (h @ w(self.wq, c.q_heads * c.head_dim, c.hidden).T).view(B, c.kv_heads, -1, c.head_dim)
        a = torch.softmax(torch.einsum("bhgd,bthd->bhgt", q, k_cache) * c.head_dim ** -0.5, -1)
        o = torch.einsum("bhgt,bthd->bhgd", a, v_cache).reshape(B, -1)
        x = x + o @ w(self.wo, c.hidden, c.q_heads * c.head_dim).T
        h = torch.nn.functional.rms_norm(x, (c.hidden,))
        ids = self.chosen                    # a near tie may fall either way
        weights = torch.softmax(h @ self.router.float().T, -1).gather(1, ids)
        w13 = dequantize_experts(*self.w13, 2 * c.width, c.hidden)[ids]
        w2 = dequantize_experts(*self.w2, c.hidden, c.width)[ids]
        gate, up = torch.einsum("bknh,bh->bkn", w13, h).chunk(2, -1)
        y = torch.einsum("bkhn,bkn->bkh", w2, torch.nn.functional.silu(gate) * up)
        return x + (y * weights.unsqueeze(-1)).sum(1)

    def cached(self, positions):
        """What the cache holds of the first positions, [sequences, positions, kv_heads, head_dim]."""
        c = self.layer
        at = torch.arange(positions, device=self.table.device)
        slots = self.table[:, at // c.page_size] * c.page_size + at % c.page_size
        k, v, _ = mx.cache_read(self.cache, slots.to(torch.int32).flatten())
        shape = (self.table.shape[0], positions, c.kv_heads, c.head_dim)
        return k.float().view(shape), v.float().view(shape)


def main(sequences=5, steps=40):
    model = DecodeStep(Layer(), sequences, max_len=steps)
    gen = torch.Generator(device="cuda").manual_seed(1)
    worst = 0.0
    for _ in range(steps):
        x = torch.randn(sequences, model.layer.hidden, device="cuda", generator=gen).bfloat16()
        y = model.step(x)
        want = model.plain(x, *model.cached(int(model.lens[0])))
        worst = max(worst, float((y.float() - want).norm() / want.norm()))
    print(f"{steps} steps of {sequences} sequences: largest relative difference from float32 {worst:.2e}")
    return worst


if __name__ == "__main__":
    main()
