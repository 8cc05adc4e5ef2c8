"""A mixture-of-experts block in Block_FP8 at any token count, from the
residual stream back to it, on the library's operators:

  residual_norm    the last block's output into the residual stream, its norm
                   and the norm's codes and scales, in one pass
  block_gemm       the shared expert's projections
  block_quantize   silu(gate) * up straight to codes and scales
  moe_route        each token's experts and weights, and the experts' lists
  grouped_gemm     the routed experts' projections over ragged lists of rows
  moe_combine      each token's weighted sum of its experts' outputs
  moe_layer        the last three steps in one call, for up to 32 tokens

    python examples/block_fp8_layer.py [--tokens 1,48,1024] [--hidden 2048] ...

builds random weights, runs the block at each token count and prints the time
per call of the whole block (the router's product, in plain torch, included).
"""
import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import bit_quantized_gemm_token_amd as w8  # noqa: E402

FMT = "Block_FP8"


class MoeBlock:
    """Weights of the block: every projection as Block_FP8 codes and scales."""

    def __init__(self, hidden=2048, width=768, experts=128, topk=8, seed=0, device="cuda:0"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def randn(*shape):
            return torch.randn(*shape, generator=g, device=device)

        def quantized(n, k):
            return w8.quantize_weight(FMT, randn(n, k) / k ** 0.5)

        self.hidden, self.width, self.experts, self.topk = hidden, width, experts, topk
        # (moe_layer takes Block_FP8 widths of whole groups)
        self.whole = hidden % w8.GROUP == 0 and width % w8.GROUP == 0
        self.post_norm = (1 + 0.1 * randn(hidden)).to(torch.bfloat16)
        self.norm = (1 + 0.1 * randn(hidden)).to(torch.bfloat16)
        self.router = randn(experts, hidden) / hidden ** 0.5
        self.shared_up = quantized(2 * width, hidden)     # gate rows, then up rows
        self.shared_down = quantized(hidden, width)
        ups = [quantized(2 * width, hidden) for _ in range(experts)]
        downs = [quantized(hidden, width) for _ in range(experts)]
        self.up = self._stack(ups)
        self.down = self._stack(downs)

    @staticmethod
    def _stack(pairs):
        q = torch.stack([p[0].view(torch.uint8) for p in pairs]).view(torch.float8_e4m3fn)
        return q, torch.stack([p[1] for p in pairs])

    def route(self, z):
        """Top-k routing: entries grouped by expert.  Returns the offsets [E + 1],
        the token row of each entry, each token's weights [T, topk] and where
        its entries went [T, topk]."""
        _, weight, offsets, rows, place = w8.moe_route(z.float() @ self.router.t(), self.topk,
                                                       renormalize=False)
        return offsets, rows, weight, place

    def expert_mlp(self, xq, sx, offsets, rows):
        both = w8.grouped_gemm(xq, sx, offsets, *self.up, rows=rows)
        aq, sa = w8.block_quantize(both[:, self.width:], gate=both[:, :self.width])
        return w8.grouped_gemm(aq, sa, offsets, *self.down)

    def shared_mlp(self, xq, sx):
        both = w8.block_gemm(xq, sx, *self.shared_up)
        aq, sa = w8.block_quantize(both[:, self.width:], gate=both[:, :self.width])
        return w8.block_gemm(aq, sa, *self.shared_down)

    def forward(self, branch, residual):
        """branch: bf16 [T, hidden], the last block's output; residual: bf16 or
        fp32 [T, hidden].  Returns this block's output and the residual after
        the last block's (its own output joins it in the next residual_norm)."""
        residual, xq, sx, z = w8.residual_norm(branch, residual, self.norm,
                                               post_weight=self.post_norm, quantize=True,
                                               with_z=True)
        shared = self.shared_mlp(xq, sx)
        if self.whole and len(z) <= w8.MAX_M:
            expert, weight = w8.moe_route(z.float() @ self.router.t(), self.topk,
                                          renormalize=False, lists=False)
            return w8.moe_layer(FMT, xq, sx, expert, weight, *self.up, *self.down,
                                base=shared), residual
        offsets, rows, weight, place = self.route(z)
        routed = self.expert_mlp(xq, sx, offsets, rows)
        return w8.moe_combine(routed, weight, place, base=shared), residual


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--tokens", default="1,48,1024")
    p.add_argument("--hidden", type=int, default=2048)
    p.add_argument("--width", type=int, default=768)
    p.add_argument("--experts", type=int, default=128)
    p.add_argument("--topk", type=int, default=8)
    p.add_argument("--reps", type=int, default=20)
    a = p.parse_args()
    block = MoeBlock(a.hidden, a.width, a.experts, a.topk)
    for T in (int(t) for t in a.tokens.split(",")):
        branch = torch.randn(T, a.hidden, device="cuda:0").to(torch.bfloat16)
        residual = 4 * torch.randn(T, a.hidden, device="cuda:0")
        for _ in range(3):
            out, after = block.forward(branch, residual)
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        for _ in range(a.reps):
            out, after = block.forward(branch, residual)
        end.record()
        end.synchronize()
        us = start.elapsed_time(end) / a.reps * 1e3
        print(f"T={T}: {us:.1f} us a block, output rms {out.float().square().mean().sqrt():.3g}",
              flush=True)


if __name__ == "__main__":
    main()
