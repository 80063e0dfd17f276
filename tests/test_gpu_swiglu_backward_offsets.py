"""mx_grouped_gemm_swiglu_backward with offsets that decrease, are negative or leave the matrix:
which rows are written is unspecified, nothing outside the outputs is."""

import pytest
import torch

from block_quant_gemm_amd import mxq
from tests.gpu_helpers import say

pytestmark = pytest.mark.gpu

MARK = 0xAB


def _inside(rows, cols, dtype, around=2):
    """(buffer, view): `rows` rows and `cols` columns with marked rows and 16 marked columns on all sides."""
    one = torch.full((rows + 2 * around, cols + 32), 3.0 if dtype == torch.bfloat16 else MARK, dtype=dtype, device="cuda")
    return one, one[around:around + rows, 16:16 + cols]


def _outside_is_marked(buf, view, around=2):
    mark = torch.full_like(buf, 3.0 if buf.dtype == torch.bfloat16 else MARK)
    keep = torch.ones_like(buf, dtype=torch.bool)
    keep[around:around + view.shape[0], 16:16 + view.shape[1]] = False
    return torch.equal(buf[keep], mark[keep])


@pytest.mark.parametrize("accum", [mxq.ACC_MFMA_FP8, mxq.ACC_FP32])
@pytest.mark.parametrize("offs", [[0, 350, 20, 200], [-9, 150, 10, 1 << 40], [301, 302, 303, 304], [300, 0, 300, 0],
                                  [0, 300, 0, 300], [0, 300, 300, 300]])
def test_nothing_outside(offs, accum):
    say(f"SwiGLU gradient offsets={offs} accum={accum}")
    M, E, F, K = 300, 3, 288, 64
    gen = torch.Generator(device="cuda").manual_seed(1)
    draw = lambda *s, sigma=1.0: (torch.randn(*s, generator=gen, device="cuda") * sigma).to(torch.bfloat16)
    dy, w = mxq.mx_quantize_rowwise(draw(M, K)), mxq.mx_quantize_rowwise(draw(E * F, K, sigma=0.02))
    w = w[0].view(E, F, K), w[1].contiguous().view(E, F, K // 32)
    cap = mxq.colwise_capacity(M, E)
    outs = {"dgu": _inside(M, 2 * F, torch.bfloat16), "q": _inside(M, 2 * F, torch.uint8),
            "scale": _inside(M, F // 16, torch.uint8), "qT": _inside(2 * F, cap, torch.uint8),
            "scaleT": _inside(2 * F, cap // 32, torch.uint8)}
    mxq.mx_grouped_gemm_swiglu_backward(*dy, *w, draw(M, 2 * F), torch.tensor(offs, device="cuda"), accum=accum,
                                        **{n: v for n, (_, v) in outs.items()})
    torch.cuda.synchronize()
    for n, (buf, view) in outs.items():
        assert _outside_is_marked(buf, view), n
