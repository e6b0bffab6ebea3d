#!/usr/bin/env python3
"""A feed-forward layer whose work is split over experts, on libbitlinear's 8-bit floating point
operators: the router's logits (block-scaled linear layer), the choice of experts, and their
gated products. Weights are quantised once from fp32; the prompt runs in one pass, then tokens
are decoded one at a time from a HIP graph.

    python examples/experts_decode.py [--hidden 4096] [--inner 1024] [--experts 64] [--top 8]
                                      [--prompt 512] [--tokens 64]
"""
from __future__ import annotations

import argparse
import os
import sys
import time

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import ternary_weight_linear_amd as tw  # noqa: E402


class ExpertsLayer:
    """Random weights of the given sizes, quantised by blocks of 128 x 128."""

    def __init__(self, hidden: int, inner: int, experts: int, top: int, groups: int, kept: int, seed: int, device):
        gen = torch.Generator(device=device).manual_seed(seed)

        def quantised(rows, cols):
            return tw.bl_fp8_quant_weight(torch.randn(rows, cols, generator=gen, device=device) * cols ** -0.5)

        def stacked(matrices, *shape):
            codes, scales = zip(*matrices)
            return (torch.stack([c.view(torch.uint8) for c in codes]).view(torch.float8_e4m3fn).view(*shape, *codes[0].shape),
                    torch.stack(scales).view(*shape, *scales[0].shape))

        self.top, self.groups, self.kept = top, groups, kept
        self.router, self.router_scales = quantised(experts, hidden)
        # steps of 0.001, as training for an even load leaves them
        self.bias = torch.round(torch.randn(experts, generator=gen, device=device) * 20) * 0.001
        self.gate_up, self.gate_up_scales = stacked([quantised(inner, hidden) for _ in range(2 * experts)], experts, 2)
        self.down, self.down_scales = stacked([quantised(hidden, inner) for _ in range(experts)], experts)

    def choose(self, x):
        """Weights fp32 [M, top] and indices int32 [M, top] of each token's experts."""
        logits = tw.bl_fp8_forward(x, self.router, self.router_scales)
        return tw.bl_route_experts(logits, self.top, bias=self.bias, score="sigmoid", groups=self.groups,
                                   kept_groups=self.kept)

    def __call__(self, x):
        weight, index = self.choose(x)
        return tw.bl_fp8_experts(x, index, weight, self.gate_up, self.gate_up_scales, self.down, self.down_scales)

    def plain(self, x):
        """The same layer on dequantised weights in fp32, without quantising activations."""
        def values(codes, scales):
            rows, cols = codes.shape
            return codes.float() * scales.repeat_interleave(128, 0)[:rows].repeat_interleave(128, 1)[:, :cols]

        weight, index = self.choose(x)
        y = torch.zeros_like(x, dtype=torch.float32)
        for m in range(x.shape[0]):
            for w, e in zip(weight[m].tolist(), index[m].tolist()):
                g, u = (values(self.gate_up[e, i], self.gate_up_scales[e, i]) @ x[m].float() for i in (0, 1))
                y[m] += w * (values(self.down[e], self.down_scales[e]) @ (torch.nn.functional.silu(g) * u))
        return y


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--hidden", type=int, default=4096)
    p.add_argument("--inner", type=int, default=1024)
    p.add_argument("--experts", type=int, default=64)
    p.add_argument("--top", type=int, default=8)
    p.add_argument("--groups", type=int, default=8)
    p.add_argument("--kept-groups", type=int, default=4)
    p.add_argument("--prompt", type=int, default=512)
    p.add_argument("--tokens", type=int, default=64)
    p.add_argument("--seed", type=int, default=0)
    a = p.parse_args(argv)
    device = torch.device("cuda:0")
    layer = ExpertsLayer(a.hidden, a.inner, a.experts, a.top, a.groups, a.kept_groups, a.seed, device)
    gen = torch.Generator(device=device).manual_seed(a.seed + 1)
    prompt = torch.randn(a.prompt, a.hidden, generator=gen, device=device, dtype=torch.bfloat16)

    layer(prompt)                                   # first use of the kernels
    torch.cuda.synchronize()
    start = time.perf_counter()
    y = layer(prompt)
    torch.cuda.synchronize()
    print(f"prompt of {a.prompt} tokens: {(time.perf_counter() - start) * 1e6:.0f} us")
    few = min(4, a.prompt)
    ref = layer.plain(prompt[:few])
    error = ((y[:few].float() - ref).norm() / ref.norm()).item()
    print(f"relative difference from fp32 activations over {few} tokens: {error:.3f}")

    token = prompt[:1].clone()
    layer(token)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(token)
    torch.cuda.synchronize()
    start = time.perf_counter()
    for _ in range(a.tokens):
        graph.replay()
        token.add_(out).mul_(0.7)                   # a stand-in for the rest of the model
    torch.cuda.synchronize()
    print(f"decode: {(time.perf_counter() - start) / a.tokens * 1e6:.1f} us per token")
    return error


if __name__ == "__main__":
    main()
