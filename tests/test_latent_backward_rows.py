"""Which workgroups the gradient of latent attention takes (the rule that the launches
follow, through the library).  CPU only."""

import pytest

from block_quant_gemm_amd import mxq


@pytest.mark.parametrize("T,H,B,causal,rows", [
    (360, 16, 1, True, 64), (2048, 16, 1, True, 64), (2048, 16, 1, False, 128),   # one causal sequence: two turns
    (4 * 4096, 16, 4, True, 128), (1200, 16, 4, True, 128), (2000, 8, 2, True, 64),
    (512, 32, 4, True, 64), (480, 32, 4, False, 64), (512, 64, 2, True, 128),     # small calls
    (512, 16, 64, True, 64), (0, 1, 1, True, 64),
    (1, 1, 601, True, 128), (317, 5, 602, True, 128), (813, 1, 602, True, 128),   # with many empty sequences
    (1 << 27, 65536, 65536, True, 128), (-1, 1, 1, True, 0), (5, 0, 1, True, 0), (5, 1, 0, True, 0)])
def test_rows(T, H, B, causal, rows):
    assert mxq.latent_backward_rows(T, H, B, causal) == rows
