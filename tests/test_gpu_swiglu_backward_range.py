"""mx_grouped_gemm_swiglu_backward where dh times the gate leaves FP32: the up value's gradient
is infinite (its MX blocks NaN), the gate's has no such factor and keeps its value.

dh = 4, exact in either mode of sums.  For g = 2^127 and 1.5 * 2^126 the sigmoid is 1 in FP32, so
d gate = dh u exactly; for g = -2^127 it is 0, and so are both gradients."""

import numpy as np
import pytest

from block_quant_gemm_amd import mxq
from oracle.codec import bf16_bits_to_f64
from tests.gpu_helpers import say
from tests.test_gpu_swiglu_backward import _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("accum", [mxq.ACC_MFMA_FP8, mxq.ACC_FP32])
def test_gate_gradient_where_the_other_overflows(accum):
    say(f"SwiGLU gradient past FP32, accum={accum}")
    M, F, K = 70, 64, 32
    dq, ds = np.zeros((M, K), np.uint8), np.full((M, 1), 127, np.uint8)
    wq, ws = np.zeros((F, K), np.uint8), np.full((F, 1), 127, np.uint8)
    dq[:, 0] = wq[:, 0] = 0x40                              # 2
    gu = np.full((M, 2 * F), 0x3F80, np.uint16)             # 1
    gu[:, :F] = 0                                           # g = 0: d gate = dh u / 2, d up = 0
    gu[3, 5], gu[40, 33], gu[69, 0] = 0x7F00, 0x7EC0, 0xFF00
    dgu, q, sc, qT, sT, _ = _run(np.array([0, M]), dq, ds, wq, ws, gu, accum=accum)
    v = bf16_bits_to_f64(dgu)
    want = np.zeros((M, 2 * F))
    want[:, :F] = 2
    want[3, 5] = want[40, 33] = 4
    want[69, 0] = 0
    want[3, F + 5] = want[40, F + 33] = np.inf
    np.testing.assert_array_equal(v, want)
    bad = np.isinf(want)
    np.testing.assert_array_equal(sc == 0xFF, bad.reshape(M, -1, 32).any(2))
    cols = np.zeros((2 * F, sT.shape[1] * 32), bool)
    cols[:, :M] = bad.T
    np.testing.assert_array_equal(sT == 0xFF, cols.reshape(2 * F, -1, 32).any(2))
