"""The example that runs the latent attention operators together: its training
step against float32 PyTorch, and its prefill in chunks and decoding over the
cache against one pass without a cache.

Tolerances: an E4M3 value has 3 mantissa bits, so rounding moves it by at most
1/16, about 1/16/sqrt(3) = 3.6 % rms at worst.  A product of two such operands
is off by at most 1.41 * 3.6 % = 5.1 % rms, and errors of chained products add as
squares: the longest chain of the training step (dW of q: kv_down, kv_up, q, o's
gradient, the product itself) has five products, 11.4 %; attention's own rounding
adds less than 1 %.  Serving differs from one pass by the cache's rounding (3.6 %,
in the keys and the values: 5.1 %) and by the absorbed products' (three more
roundings each way, 2 * 5.1 %): 1.41 * 10.2 = 15 % at worst in root of squares.
Both are tested at 20 %."""

import torch
import pytest

from examples import latent_block
from tests.gpu_helpers import say

pytestmark = pytest.mark.gpu


def _reference(block, x, dy, lens, positions):
    """float32 PyTorch: the same block, no quantization."""
    H, N, V, L = block.H, latent_block.NOPE, latent_block.VALUE, latent_block.LATENT
    w = {n: t.float().requires_grad_() for n, t in block.weights.items()}
    x = x.float().requires_grad_()
    q = (x @ w["q"].t()).view(-1, H, N + latent_block.ROPE)
    d = x @ w["kv_down"].t()
    kr = latent_block.rotate(d[:, L:], positions)
    q = torch.cat([q[..., :N], latent_block.rotate(q[..., N:], positions)], -1)
    kv = (d[:, :L] @ w["kv_up"].t()).view(-1, H, N + V)
    outs, t = [], 0
    for n in lens:
        k = torch.cat([kv[t:t + n, :, :N], kr[t:t + n, None].expand(-1, H, -1)], -1)
        z = torch.stack([q[t:t + n, h] @ k[:, h].t() for h in range(H)]) * block.scale
        p = z.masked_fill(torch.ones(n, n, device="cuda").triu(1).bool(), -torch.inf).softmax(-1)
        outs.append(torch.stack([p[h] @ kv[t:t + n, h, N:] for h in range(H)], 1))
        t += n
    y = torch.cat(outs).reshape(x.shape[0], -1) @ w["o"].t()
    y.backward(dy.float())
    return y, x.grad, {n: t.grad for n, t in w.items()}


def _rel(a, b):
    a, b = a.detach().float(), b.detach().float()
    return float((a - b).norm() / b.norm())


def _positions(lens):
    return torch.cat([torch.arange(n, device="cuda") for n in lens])


def test_training_step():
    say("latent block: training step")
    block = latent_block.LatentBlock(heads=4)
    lens = [200, 1, 77]
    torch.manual_seed(3)
    x = torch.randn((sum(lens), block.hidden), device="cuda").to(torch.bfloat16)
    dy = (torch.randn_like(x) * 1e-3)
    y, dx, dw = block.train(x, dy, latent_block.offsets_of(lens), _positions(lens))
    ry, rdx, rdw = _reference(block, x, dy, lens, _positions(lens))
    assert _rel(y, ry) < 0.2
    assert _rel(dx, rdx) < 0.2
    for n in rdw:
        assert _rel(dw[n], rdw[n]) < 0.2, n


def test_prefill_in_chunks_and_decoding():
    say("latent block: prefill in chunks, decoding")
    block = latent_block.LatentBlock(heads=4, seed=2)
    prompts, new = [130, 1, 64, 300], 3
    xs, out = latent_block.serve(block, prompts, new, chunk=96, page_size=24)
    lens = [len(v) for v in xs]
    x = torch.cat(xs)
    y = block.train(x, torch.zeros_like(x), latent_block.offsets_of(lens), _positions(lens))[0]
    for o, r, n in zip(out, y.split(lens), prompts):
        assert _rel(o[:n], r[:n]) < 0.2
        assert _rel(o[n:], r[n:]) < 0.2
