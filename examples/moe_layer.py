"""A stack of mixture-of-experts layers with random ternary weights: a block of prompt tokens,
then single tokens from one captured CUDA graph.

    python examples/moe_layer.py [--layers 4] [--hidden 2048] [--inter 1024] [--experts 64]
                                 [--topk 8] [--fmt 2|1] [--prompt 512] [--tokens 64]

Each layer is  residual += delta; q, s = quantised RMS norm; router logits -> ids, weights;
delta = sum over the token's experts of w * down(SiLU(gate) * up).  (Attention, which a model has
between these layers, is left out; the router's projection is a plain matrix product.)
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from ternary_weight_dp4a_gb300 import synth, tq  # noqa: E402


class Layer:
    def __init__(self, a, seed: int):
        self.gamma = torch.ones(a.hidden, dtype=torch.bfloat16, device="cuda")
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.router = torch.randn((a.experts, a.hidden), device="cuda", generator=gen).bfloat16() * a.hidden ** -0.5
        self.gate, self.up = (self.experts(a, a.inter, a.hidden, seed + i) for i in (1, 2))
        self.down = self.experts(a, a.hidden, a.inter, seed + 3)

    @staticmethod
    def experts(a, n: int, k: int, seed: int) -> tq.PackedExperts:
        fmt = tq.FMT_TERNARY2 if a.fmt == 2 else tq.FMT_BINARY1
        codes, scales = synth.weight(a.experts * n, k, fmt, seed, device="cuda")
        return tq.pack_experts(codes.view(a.experts, n, k), fmt, scales.view(a.experts, n, -1))

    def __call__(self, residual, delta, x, topk: int, workspace):
        """residual is updated in place; returns the layer's output."""
        _, q, s = tq.add_rmsnorm_rotq(residual, delta, self.gamma, residual_out=residual, x_out=x)
        ids, weights = tq.moe_route(torch.mm(x, self.router.t()), topk)
        return tq.moe_ffn(self.gate, self.up, self.down, q, s, ids, weights, dtype=torch.bfloat16, workspace=workspace)


def forward(layers, residual, topk: int, workspace):
    """residual [m][hidden] bf16 (overwritten) -> the sum after the last layer."""
    x, delta = torch.empty_like(residual), None
    for layer in layers:
        delta = layer(residual, delta, x, topk, workspace)
    return residual.add_(delta)


def main(argv=None) -> int:
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, default in (("layers", 4), ("hidden", 2048), ("inter", 1024), ("experts", 64), ("topk", 8), ("fmt", 2),
                          ("prompt", 512), ("tokens", 64)):
        p.add_argument("--" + name, type=int, default=default)
    a = p.parse_args(argv)
    layers = [Layer(a, 1000 * i) for i in range(a.layers)]
    workspace = tq.moe_workspace(max(a.prompt, 1), a.topk, a.experts, a.hidden, a.inter)
    tokens = torch.randn((a.prompt, a.hidden), device="cuda").bfloat16()

    out = forward(layers, tokens.clone(), a.topk, workspace)                 # warm-up
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    out = forward(layers, tokens.clone(), a.topk, workspace)
    torch.cuda.synchronize()
    print(f"prompt of {a.prompt} tokens: {(time.perf_counter() - t0) * 1e3:.2f} ms")

    # one token, captured once; every replay routes its own token
    token = tokens[:1].clone()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        forward(layers, token.clone(), a.topk, workspace)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        one = forward(layers, token.clone(), a.topk, workspace)
    count = min(a.tokens, a.prompt)
    got = torch.empty_like(out[:count])
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for i in range(count):
        token.copy_(tokens[i:i + 1])
        graph.replay()
        got[i] = one[0]
    torch.cuda.synchronize()
    ms = (time.perf_counter() - t0) * 1e3
    tq.read_error_word(workspace[:4])                                        # raises if a bounded wait ran out
    # (the layers give a row the same bits in any batch; the router's matrix product may not)
    far = (got.float() - out[:count].float()).norm() / out[:count].float().norm()
    print(f"{count} tokens one by one: {ms / count * 1e3:.1f} us each; {float(far):.1e} from the prompt's rows")
    return 0


if __name__ == "__main__":
    sys.exit(main())
