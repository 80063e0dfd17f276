"""The gradient product and the few-token block on operands and outputs whose byte offsets
pass 2^32: rows and experts far apart in one large buffer, against the same call on compact
tensors, bit for bit."""

import pytest
import torch

from block_quant_gemm_amd import mxq
from tests.gpu_helpers import say

pytestmark = pytest.mark.gpu


class _Far:
    """Rows `stride` bytes apart; every tensor takes the next columns of the same buffer."""

    def __init__(self, rows, stride):
        self.buf = torch.empty(rows * stride, dtype=torch.uint8, device="cuda")
        self.stride, self.at = stride, 0

    def empty(self, rows, cols, dtype=torch.uint8):
        size = torch.empty(0, dtype=dtype).element_size()
        assert self.at + cols * size <= self.stride and rows * self.stride <= self.buf.numel()
        t = self.buf.view(dtype).as_strided((rows, cols), (self.stride // size, 1), self.at // size)
        self.at += (cols * size + 255) // 256 * 256
        return t

    def put(self, t):
        f = self.empty(t.shape[0], t.shape[1], t.dtype)
        f.copy_(t)
        return f


def _draw(gen, rows, cols, sigma=1.0):
    return (torch.randn((rows, cols), generator=gen, device="cuda") * sigma).to(torch.bfloat16)


def _same(a, b):
    return all((u is None and v is None) or torch.equal(u, v) for u, v in zip(a, b, strict=True))


@pytest.mark.parametrize("accum", [mxq.ACC_MFMA_FP8, mxq.ACC_FP32])
@pytest.mark.parametrize("wide", [2, 16])                    # the weights' scale rows: windows from 16 on
def test_gate_up_gradient(accum, wide):
    say(f"SwiGLU gradient past 2^32 bytes, accum={accum} scale rows of {wide}")
    M, E, F, K = 700, 4, 96, 64
    gen = torch.Generator(device="cuda").manual_seed(accum)
    dy = mxq.mx_quantize_rowwise(_draw(gen, M, K))
    wq, ws = mxq.mx_quantize_rowwise(_draw(gen, E * F, K, 0.02))
    padded = torch.zeros((E * F, wide), dtype=torch.uint8, device="cuda")
    padded[:, :K // 32] = ws
    gu, offs = _draw(gen, M, 2 * F), torch.tensor([0, 300, 301, 301, M], device="cuda")
    want = mxq.mx_grouped_gemm_swiglu_backward(*dy, wq.view(E, F, K), padded.view(E, F, wide)[:, :, :K // 32], gu, offs,
                                               dgu=True, accum=accum)
    cap = want[3].shape[1]
    far = _Far(M, 8_000_000)                                 # 257 rows stay within 2^31, 700 pass 2^32
    out = dict(dgu=far.empty(M, 2 * F, torch.bfloat16), q=far.empty(M, 2 * F), scale=far.empty(M, F // 16))
    dyf, guf = [far.put(t) for t in dy], far.put(gu)
    cols = _Far(2 * F, 48_000_000)                           # the column copy's 192 rows
    out.update(qT=cols.empty(2 * F, cap), scaleT=cols.empty(2 * F, cap // 32))
    experts = _Far(E, 1_600_000_000)                         # the last expert starts past 2^32
    w = [experts.put(t.reshape(E, -1)).unflatten(1, (F, n)) for t, n in ((wq, K), (padded, wide))]
    got = mxq.mx_grouped_gemm_swiglu_backward(*dyf, w[0], w[1][:, :, :K // 32], guf, offs, accum=accum, **out)
    assert _same(got, want)


def test_few_tokens_rows():
    say("gated ffn, rows past 2^32 bytes")
    M, K, F, N = 40, 96, 64, 50
    gen = torch.Generator(device="cuda").manual_seed(9)
    x, wg = mxq.mx_quantize_rowwise(_draw(gen, M, K)), mxq.mx_quantize_rowwise(_draw(gen, 2 * F, K, 0.1))
    wd = mxq.mx_quantize_rowwise(_draw(gen, N, F, 0.1))
    one = lambda ts: [t.unsqueeze(0) for t in ts]
    want = mxq.mx_gated_ffn_decode(*x, *one(wg), *one(wd))
    far = _Far(2 * F, 120_000_000)
    put = lambda ts: [far.put(t) for t in ts]
    got = mxq.mx_gated_ffn_decode(*put(x), *one(put(wg)), *one(put(wd)), y=far.empty(M, N, torch.bfloat16))
    assert torch.equal(got, want)


def test_few_tokens_experts():
    say("gated ffn, experts past 2^32 bytes")
    E, K, F, N = 4, 96, 64, 50
    offs = torch.tensor([0, 3, 3, 20, 37], device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(10)
    x = mxq.mx_quantize_rowwise(_draw(gen, 37, K))
    wg, wd = mxq.mx_quantize_rowwise(_draw(gen, E * 2 * F, K, 0.1)), mxq.mx_quantize_rowwise(_draw(gen, E * N, F, 0.1))
    stacks = [(t.contiguous().view(E, -1, t.shape[1])) for t in (*wg, *wd)]
    want = mxq.mx_gated_ffn_decode(*x, *stacks, offsets=offs)
    far = _Far(E, 1_600_000_000)                             # the last expert starts past 2^32
    got = mxq.mx_gated_ffn_decode(*x, *[far.put(t.reshape(E, -1)).unflatten(1, t.shape[1:]) for t in stacks],
                                  offsets=offs)
    assert torch.equal(got, want)
