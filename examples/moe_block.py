"""A mixture-of-experts block on 4-bit weights, for prompts and single tokens.

    python examples/moe_block.py [--tokens 512] [--steps 8]

Float weights are quantized to microscaled 4-bit (MX4) and packed once. Then a
prompt and a few single tokens run through the block: the router chooses
experts, their gate and up products meet in SiLU, the down products are summed
per token; a shared projection follows, with the activations in 16 bits or
quantized to 4 on the way in. Every output is compared with fp32 matrix
products on the same quantized weights.
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import weight_only_lut_amd as lutq  # noqa: E402


class MoeBlock:
    """Router, experts and an output projection, quantized from float weights."""

    def __init__(self, D, F, E, k, dtype=torch.bfloat16, device="cuda"):
        self.k, self.dtype = k, dtype
        self.router = (torch.randn(E, D, device=device) / D ** 0.5).to(dtype)
        self.balance = 0.02 * torch.randn(E, device=device)

        def pack(*shape):
            w = torch.randn(shape, device=device) / shape[-1] ** 0.5
            codes, scales = lutq.mx_quantize(w.view(-1, shape[-1]))
            if len(shape) == 3:
                codes, scales = codes.view(*shape[:2], -1), scales.view(*shape[:2], -1)
            return lutq.mx_pack(codes, scales), lutq.mx_dequantize(codes, scales, torch.float32)
        (self.gate_up, self._gate_up), (self.down, self._down) = pack(E, 2 * F, D), pack(E, D, F)
        self.out, self._out = pack(D, D)

    def route(self, x):
        return lutq.moe_route(x @ self.router.T, self.k, score="sigmoid", bias=self.balance, scale=1.5)

    def __call__(self, x, four_bit=False):
        y = lutq.moe_mlp(x, self.gate_up, self.down, self.route(x))
        return lutq.mx_matmul(lutq.mx_quantize(y) if four_bit else y, self.out, dtype=self.dtype)

    def reference(self, x):
        """The experts' part in fp32, one token at a time."""
        r, rows = self.route(x), []
        for t in range(x.shape[0]):
            y = torch.zeros(x.shape[1], device=x.device)
            for e, w in zip(r.ids[t].tolist(), r.weights[t]):
                g, u = (self._gate_up[e] @ x[t].float()).chunk(2)
                y += w * (self._down[e] @ (torch.nn.functional.silu(g) * u))
            rows.append(y)
        return torch.stack(rows)


def relative(a, b):
    return float((a.float() - b.float()).norm() / b.float().norm())


def main(tokens=512, steps=8, D=1024, F=512, E=16, k=4):
    """Returns the largest relative errors: (experts' block, projection, 4-bit projection)."""
    torch.manual_seed(0)
    block = MoeBlock(D, F, E, k)
    worst = [0.0, 0.0, 0.0]
    for n in [tokens] + [1] * steps:
        x = torch.randn(n, D, device="cuda").to(torch.bfloat16)
        y = lutq.moe_mlp(x, block.gate_up, block.down, block.route(x))
        q = lutq.mx_dequantize(*lutq.mx_quantize(y), torch.float32)
        got = (y, block(x), block(x, four_bit=True))
        want = (block.reference(x), y.float() @ block._out.T, q @ block._out.T)
        worst = [max(w, relative(a, b)) for w, a, b in zip(worst, got, want)]
    load = torch.diff(block.route(torch.randn(tokens, D, device="cuda").to(torch.bfloat16)).offsets)
    print(f"{tokens} tokens and {steps} single ones over {E} experts, {k} each: pairs per expert "
          f"{int(load.min())} to {int(load.max())}")
    print("largest relative error: experts %.2g, projection %.2g, 4-bit projection %.2g" % tuple(worst))
    return worst


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--steps", type=int, default=8)
    main(**vars(ap.parse_args()))
