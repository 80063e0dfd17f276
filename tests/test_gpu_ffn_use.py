"""The norm and feed-forward operators as they are used: the example block against float32
PyTorch, one chain of them in a HIP graph, on two streams at once, and from tensors made
on another stream.

Tolerance of the block: an E4M3 value has 3 mantissa bits, so rounding moves it by at most
1/16, about 3.6 % rms at worst, values that saturate at 448 up to 12.5 %, one in 32 of every
fifth block: 1 % rms.  A product of two such operands is off by at most 1.41 * 3.8 = 5.3 % rms,
and errors of chained products add as squares: the longest chain (dW of gate_up and dx: gate_up,
whose error reaches the gradient twice, through g and u; down; dW) has four products, 10.6 %,
tested at 20 %.  Decoding rounds the same operands: it differs from the training form by the FP8 unit's
truncation (2^-13 of a product) where that moves h across a code's border, and BF16's half
step: 2 %."""

import numpy as np
import pytest
import torch

from block_quant_gemm_amd import mxq
from examples import ffn_block
from tests.gpu_helpers import say

pytestmark = pytest.mark.gpu


def _rel(a, b):
    a, b = a.detach().float(), b.detach().float()
    return float((a - b).norm() / b.norm())


def _draw(n, k, seed, sigma=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn((n, k), generator=gen, device="cuda") * sigma).to(torch.bfloat16)


def _reference(block, x, r, dy, dt):
    w = {n: t.float().requires_grad_() for n, t in block.weights.items()}
    x, r = x.float().requires_grad_(), r.float().requires_grad_()
    s = x + r
    n = s * torch.rsqrt((s * s).mean(1, keepdim=True) + ffn_block.EPS) * w["norm"]
    gu = n @ w["gate_up"].t()
    g, u = gu[:, :block.ffn], gu[:, block.ffn:]
    y = (g * torch.sigmoid(g) * u) @ w["down"].t()
    ((y * dy.float()).sum() + (s * dt.float()).sum()).backward()
    assert torch.equal(x.grad, r.grad)
    return s, y, x.grad, {n: t.grad for n, t in w.items()}


@pytest.mark.parametrize("tokens,ffn", [(333, 352), (1, 96), (1300, 1408)])
def test_training_step(tokens, ffn):
    say(f"ffn block: training step of {tokens} tokens, {ffn} columns")
    block = ffn_block.FeedForwardBlock(hidden=512, ffn=ffn, seed=tokens)
    x, r = _draw(tokens, 512, 1), _draw(tokens, 512, 2)
    dy, dt = _draw(tokens, 512, 3, 1e-3), _draw(tokens, 512, 4, 1e-3)
    total, y, kept = block.forward(x, r)
    dx, dw = block.backward(dy, dt, kept)
    s, ry, rdx, rdw = _reference(block, x, r, dy, dt)
    assert torch.equal(total, s.to(torch.bfloat16))
    assert _rel(y, ry) < 0.2
    assert _rel(dx, rdx) < 0.2
    for n in rdw:
        assert _rel(dw[n], rdw[n]) < 0.2, n


@pytest.mark.parametrize("tokens", [1, 8, 48])
def test_decoding_is_the_training_forms_output(tokens):
    block = ffn_block.FeedForwardBlock(seed=5)
    x, r = _draw(tokens, 2048, 6), _draw(tokens, 2048, 7)
    total, y, _ = block.forward(x, r)
    t2, z = block.decode(x, r)
    assert torch.equal(total, t2)
    assert _rel(z, y) < 0.02


class _Chain:
    """One step of everything, into buffers of its own."""

    def __init__(self, seed, tokens=200, few=5):
        self.block = ffn_block.FeedForwardBlock(hidden=512, ffn=288, seed=seed)
        self.x, self.r = _draw(tokens, 512, seed), _draw(tokens, 512, seed + 1)
        self.dy, self.dt = _draw(tokens, 512, seed + 2, 1e-3), _draw(tokens, 512, seed + 3, 1e-3)
        self.few, self.one = few, torch.tensor([0, tokens], device="cuda")
        b = self.block
        self.wT = mxq.expert_view(b.down[2], b.down[3], 1, 512)

    def run(self):
        b = self.block
        total, rstd, y, q, s, xT, xTs = mxq.mx_rms_norm(self.x, b.weights["norm"], residual=self.r, y=True,
                                                        columns=True)
        gu, hq, hs, hT, hTs, poff = mxq.mx_grouped_gemm_swiglu(q, s, *b._stacked(*b.gate_up[:2]), self.one)
        dq, ds, _, _, _ = mxq.mx_quantize_dual(self.dy, self.one)
        dgu, gq, gs, gT, gTs, p2 = mxq.mx_grouped_gemm_swiglu_backward(dq, ds, *self.wT, gu, self.one, dgu=True)
        n = 2 * b.ffn
        dn = mxq.mx_gemm(gq, gs, b.gate_up[2][:, :n], b.gate_up[3][:, :n // 32])
        dx, dw = mxq.mx_rms_norm_backward(dn, total, rstd, b.weights["norm"], dtotal=self.dt)
        t2, z = b.decode(self.x[:self.few], self.r[:self.few])
        return [total, rstd, y, q, s, xT, xTs, gq, gs, gT, gTs, dgu, poff, p2, dx, dw, t2, z]


def _same(a, b):
    return all(torch.equal(u.view(torch.uint8) if u.dtype == torch.uint8 else u,
                           v.view(torch.uint8) if v.dtype == torch.uint8 else v) for u, v in zip(a, b))


def test_in_a_graph():
    say("norm and feed-forward chain in a HIP graph")
    chain = _Chain(20)
    want = [t.clone() for t in chain.run()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        chain.run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = chain.run()
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert _same(got, want)
        assert _same(chain.run(), want)              # eager work between the replays
    # new values in the same buffers
    chain.x.copy_(_draw(200, 512, 99))
    graph.replay()
    torch.cuda.synchronize()
    assert _same(got, chain.run())


def test_on_two_streams_at_once():
    say("norm and feed-forward chains on two streams")
    chains = [_Chain(30), _Chain(40)]
    want = [[t.clone() for t in c.run()] for c in chains]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    out = [[], []]
    for _ in range(5):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                out[i].append(chains[i].run())
    torch.cuda.synchronize()
    for i in (0, 1):
        for got in out[i]:
            assert _same(got, want[i])


def test_offsets_past_32_bits():
    """Rows whose byte offset passes 2^32: the last rows of a large strided matrix."""
    say("rms norm past 2^32 bytes")
    K, ld, M = 64, 1 << 20, 2200                                  # 2200 rows of 2 MiB
    big = torch.empty(M * ld, dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((M, K), (ld, 1))
    vals = _draw(M, K, 50)
    x.copy_(vals)
    w = _draw(1, K, 51)[0]
    a, b = mxq.mx_rms_norm(x, w, y=True, columns=True), mxq.mx_rms_norm(vals, w, y=True, columns=True)
    assert _same(a[1:], b[1:])
    dy = _draw(M, K, 52)
    c = mxq.mx_rms_norm_backward(dy, x, a[1], w)
    d = mxq.mx_rms_norm_backward(dy, vals, a[1], w)
    assert _same(c, d)
