"""mx_rms_norm of more rows than one launch takes (2^21): each row is as in a call of its own."""

import pytest
import torch

from block_quant_gemm_amd import mxq
from tests.gpu_helpers import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K,residual", [(64, True), (64, False), (2080, False)])
def test_rows_past_a_launch(K, residual):
    say(f"rms norm of 2^21 + 101 rows, K={K} residual={residual}")
    edge, M = 1 << 21, (1 << 21) + 101
    gen = torch.Generator(device="cuda").manual_seed(K)
    some = torch.randn((1 << 12, K + 8), device="cuda", generator=gen).to(torch.bfloat16)
    wide = some.repeat((M + 4095) // 4096, 1)[:M]
    wide[edge - 60:] = torch.randn((M - edge + 60, K + 8), device="cuda", generator=gen).to(torch.bfloat16)
    x = wide[:, 8:]                                          # a column range: the stride is not the width
    r = x.flip(1).contiguous() if residual else None
    w = (1 + 0.1 * torch.randn(K, device="cuda", generator=gen)).to(torch.bfloat16)
    every = mxq.mx_rms_norm(x, w, residual=r, y=True)
    for a, b in ((0, 50), (edge - 50, edge), (edge, edge + 50), (edge - 20, M)):
        part = mxq.mx_rms_norm(x[a:b], w, residual=None if r is None else r[a:b], y=True)
        for u, v in zip(every[:5], part[:5]):
            assert torch.equal(u[a:b], v)
