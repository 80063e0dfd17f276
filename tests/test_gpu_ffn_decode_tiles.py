"""mx_gated_ffn_decode's workgroups of two and four token tiles, dense and per expert, with
contractions of several iterations a wavefront, against the float64 oracle (the allowance is
test_gpu_ffn_decode.py's).  test_ffn_variants.py keeps the list of kernels that these reach."""

import numpy as np
import pytest
import torch

from block_quant_gemm_amd import workloads
from tests.gpu_helpers import host, say
from tests.test_gpu_ffn_decode import _call, _check, _operands

pytestmark = pytest.mark.gpu

# M, K, F, N
TILES = [(41, 2336, 2816, 2000), (70, 2336, 2816, 1999), (48, 1024, 2816, 2048), (33, 512, 1408, 4100),
         # sixteen wavefronts for y: shares of two iterations, the second partial, full and of one block
         (48, 32, 8224, 2048), (200, 32, 8224, 2048), (64, 96, 10944, 2047), (130, 64, 9216, 2048)]

# rows of each expert (their average picks the tiles), K, F, N: groups that end inside a
# workgroup's tiles, after whole ones, and with one row more
EXPERTS = [([50, 0, 3, 17, 33, 1, 64, 20], 1056, 544, 300), ([120, 0, 3, 47, 33, 1, 90, 70], 1056, 544, 300),
           ([30, 11], 64, 8224, 1100), ([75, 41], 64, 8224, 1100), ([0, 129, 64, 1, 0, 32, 65, 2], 544, 1408, 270)]


@pytest.mark.parametrize("M,K,F,N", TILES)
def test_dense(M, K, F, N):
    say(f"gated ffn tiles M={M} K={K} F={F} N={N}")
    ops = _operands(M, 1, K, F, N, seed=M + K + F)
    _check(host(_call(*ops)), *ops, [0, M])


@pytest.mark.parametrize("counts,K,F,N", EXPERTS)
def test_experts(counts, K, F, N):
    say(f"gated ffn tiles experts {counts} K={K} F={F} N={N}")
    offs = workloads.offsets_from_counts(np.array(counts, np.int64))
    ops = _operands(int(offs[-1]), len(counts), K, F, N, seed=K + F + len(counts))
    y = torch.full((int(offs[-1]) + 3, N), 3.0, dtype=torch.bfloat16, device="cuda")
    _call(*ops, offs, y=y[:-3])
    assert (y[-3:] == 3).all()
    _check(host(y[:-3]), *ops, offs)
