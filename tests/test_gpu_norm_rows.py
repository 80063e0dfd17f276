"""mx_rms_norm's row copy alone, whose kernels for few columns no call with both copies takes, against
the oracle; and of more rows than one launch takes (2^21): each row is as in a call of its own."""

import pytest
import torch

from block_quant_gemm_amd import mxq
from oracle import norm
from oracle.codec import bf16_bits_to_f64
from tests.gpu_helpers import say, to_dev_bf16
from tests.test_gpu_norm import EPS, _bits, _check_norm, _weight

pytestmark = pytest.mark.gpu


ROWS = [(1, 32), (3, 64), (33, 96), (5, 512), (130, 480), (2051, 288), (40, 1024), (2050, 992), (6, 2080)]


@pytest.mark.parametrize("M,K", ROWS)
@pytest.mark.parametrize("residual", [False, True])
def test_row_copy_alone(M, K, residual):
    say(f"rms norm, row copy, M={M} K={K} residual={residual}")
    x, r, w = _bits((M, K), M + K, "nx"), _bits((M, K), M + K, "nr"), _weight(K, K)
    out = mxq.mx_rms_norm(to_dev_bf16(x), to_dev_bf16(w), eps=EPS, y=True,
                          residual=to_dev_bf16(r) if residual else None)
    assert out[5] is None and out[6] is None
    s = norm.residual_sum(x, r) if residual else bf16_bits_to_f64(x)
    _check_norm(s, bf16_bits_to_f64(w), out)


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
