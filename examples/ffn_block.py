"""The norm and the gated feed-forward operators together, as a model's feed-forward block
has them.

A block with random weights (hidden 2048 and a dense layer by default): the residual's
addition and the root-mean-square norm, the gate/up product with SwiGLU, the down
product, every product on MX operands.

    train    forward and backward, with all gradients: the norm makes the gate/up product's
             two operand copies, that product makes the down product's, and on the way
             back the down product's data gradient makes the gate/up gradients' copies
    decode   the same for a few tokens

    python examples/ffn_block.py          # on a GPU, after building
"""

import argparse
import os
import sys
import time

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from block_quant_gemm_amd import mxq

EPS = 1e-6


class FeedForwardBlock:
    def __init__(self, hidden=2048, ffn=2816, seed=0, device="cuda"):
        gen = torch.Generator(device=device)
        gen.manual_seed(seed)

        def draw(n, k):
            return (torch.randn((n, k), device=device, generator=gen) * k ** -0.5).to(torch.bfloat16)

        self.hidden, self.ffn = hidden, ffn
        self.weights = {"norm": (1 + 0.1 * torch.randn(hidden, device=device, generator=gen)).to(torch.bfloat16),
                        "gate_up": draw(2 * ffn, hidden), "down": draw(hidden, ffn)}
        # each weight's two copies, made once
        rows = lambda n: torch.tensor([0, n], dtype=torch.int64, device=device)
        self.gate_up = mxq.mx_quantize_dual(self.weights["gate_up"], rows(2 * ffn))[:4]
        self.down = mxq.mx_quantize_dual(self.weights["down"], rows(hidden))[:4]

    def _stacked(self, q, s):
        """One group's codes and scales as the grouped calls take them."""
        return q.unsqueeze(0), s.unsqueeze(0)

    def forward(self, x, residual):
        """(the stream x + residual, the block's output, what backward() needs)"""
        one = torch.tensor([0, x.shape[0]], dtype=torch.int64, device=x.device)
        total, rstd, _, q, s, xT, xTs = mxq.mx_rms_norm(x, self.weights["norm"], residual=residual, eps=EPS,
                                                        columns=True)
        gu, hq, hs, hT, hTs, poff = mxq.mx_grouped_gemm_swiglu(q, s, *self._stacked(*self.gate_up[:2]), one)
        return total, mxq.mx_gemm(hq, hs, *self.down[:2]), (total, rstd, xT, xTs, gu, hT, hTs, one, poff)

    def backward(self, dy, dtotal, kept):
        """(gradient of x and of residual, {weight name: gradient}) from those of the output
        and of the stream past this block."""
        total, rstd, xT, xTs, gu, hT, hTs, one, poff = kept
        dq, ds, dT, dTs, _ = mxq.mx_quantize_dual(dy, one)
        dw = {"down": mxq.mx_grouped_gemm_wgrad(dT, dTs, hT, hTs, poff)[0]}
        wT = mxq.expert_view(self.down[2], self.down[3], 1, self.hidden)
        _, gq, gs, gT, gTs, _ = mxq.mx_grouped_gemm_swiglu_backward(dq, ds, *wT, gu, one)
        dw["gate_up"] = mxq.mx_grouped_gemm_wgrad(gT, gTs, xT, xTs, poff)[0]
        n = 2 * self.ffn
        dn = mxq.mx_gemm(gq, gs, self.gate_up[2][:, :n], self.gate_up[3][:, :n // 32])
        dx, dw["norm"] = mxq.mx_rms_norm_backward(dn, total, rstd, self.weights["norm"], dtotal=dtotal)
        return dx, dw

    def decode(self, x, residual):
        """(the stream, the block's output) of a few tokens"""
        total, _, _, q, s, _, _ = mxq.mx_rms_norm(x, self.weights["norm"], residual=residual, eps=EPS)
        return total, mxq.mx_gated_ffn_decode(q, s, *self._stacked(*self.gate_up[:2]),
                                              *self._stacked(*self.down[:2]))


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--ffn", type=int, default=10944)
    a = ap.parse_args()
    block = FeedForwardBlock(ffn=a.ffn)
    draw = lambda n, sigma=1.0: (torch.randn((n, block.hidden), device="cuda") * sigma).to(torch.bfloat16)
    x, r, dy, dt = draw(a.tokens), draw(a.tokens), draw(a.tokens, 1e-3), draw(a.tokens, 1e-3)

    def step():
        _, y, kept = block.forward(x, r)
        return y, block.backward(dy, dt, kept)
    step()
    torch.cuda.synchronize()
    t = time.perf_counter()
    y, (dx, dw) = step()
    torch.cuda.synchronize()
    print(f"train: {a.tokens} tokens, {1e3 * (time.perf_counter() - t):.2f} ms; gradients "
          f"{', '.join(f'{n} {g.float().norm():.3g}' for n, g in dw.items())}", flush=True)
    for n in (1, 8, 48):
        block.decode(x[:n], r[:n])
        torch.cuda.synchronize()
        t = time.perf_counter()
        _, z = block.decode(x[:n], r[:n])
        torch.cuda.synchronize()
        e = (z.float() - y[:n].float()).norm() / y[:n].float().norm()
        print(f"decode: {n} tokens, {1e6 * (time.perf_counter() - t):.0f} us, relative difference from the "
              f"training form {e:.4f}", flush=True)


if __name__ == "__main__":
    main()
