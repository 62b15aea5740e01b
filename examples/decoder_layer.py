"""A decoder layer on the GPU: attention over a paged cache, then the routed-expert MoE layer, both on FP4 weights.

    python examples/decoder_layer.py

A prefix is read once, eight requests are answered behind it token by token.  Synthetic weights and activations of a
small shape; prints the time of a step.
"""
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_fp4_group_amd as moe  # noqa: E402


def fp4(g, E, n, k, exponent):
    """Random MXFP4 weights with block scales around 2^exponent."""
    codes = torch.randint(0, 256, (E, n, k // 2), generator=g, dtype=torch.uint8)
    scales = torch.randint(126 + exponent, 129 + exponent, (E, n, k // 32), generator=g, dtype=torch.uint8)
    return moe.Weights(codes.cuda(), scales.cuda())


def rotation(positions, dims, theta=10000.0):
    angle = torch.arange(positions, dtype=torch.float64)[:, None] * theta ** (-torch.arange(0, dims, 2, dtype=torch.float64) / dims)
    return torch.cat([angle.cos(), angle.sin()], 1).float().cuda()


def norm(x):
    """The norm before each half, as the surrounding program applies it."""
    return torch.nn.functional.rms_norm(x, x.shape[-1:], eps=1e-6)


class DecoderLayer:
    def __init__(self, hidden=512, inter=256, experts=32, q_heads=8, kv_heads=2, k_dim=128, v_dim=128, requests=8,
                 context=256, max_tokens=1024, seed=0):
        g = torch.Generator().manual_seed(seed)
        n = (q_heads + kv_heads) * k_dim + kv_heads * v_dim
        aw = moe.AttentionWeights(fp4(g, 1, n, hidden, -6), fp4(g, 1, hidden, q_heads * v_dim, -6),
                                  torch.ones(k_dim, device="cuda"), torch.ones(k_dim, device="cuda"))
        page = 16
        pages = (requests + 1) * -(-max(context, max_tokens) // page)
        self.attention = moe.AttentionLayer(aw, q_heads, kv_heads, k_dim, v_dim, rotation(4096, k_dim), pages, page, requests,
                                            max(context, max_tokens), max_tokens)
        mw = moe.LayerWeights(fp4(g, experts, inter, hidden, -6), fp4(g, experts, inter, hidden, -6),
                              fp4(g, experts, hidden, inter, -6))
        router = torch.randn((experts, hidden), generator=g).cuda() / hidden ** 0.5
        self.experts = moe.MoELayer(mw, experts, 8, 4, 8, 2.827, max_tokens, router_weight=router)

    def prompt(self, x, lens, prefix=False):
        return self._experts(self.attention.prompt(norm(x), lens, residual=x, prefix=prefix))

    def decode(self, x):
        return self._experts(self.attention.decode(norm(x), residual=x))

    def _experts(self, h):
        return self.experts.forward(norm(h), None, residual=h)


def main():
    layer, g = DecoderLayer(), torch.Generator(device="cuda").manual_seed(1)

    def tokens(n):
        return torch.randn((n, 512), generator=g, device="cuda").to(torch.bfloat16)

    layer.prompt(tokens(777), [777], prefix=True)
    for _ in range(8):
        y = layer.decode(tokens(8))
    torch.cuda.synchronize()
    start = time.perf_counter()
    for _ in range(50):
        y = layer.decode(y)
    torch.cuda.synchronize()
    step = (time.perf_counter() - start) / 50
    print(f"decode step of 8 requests behind {layer.attention.prefix_len} shared tokens: {step * 1e6:.0f} us")
    return y


if __name__ == "__main__":
    main()
