"""Absorbed attention over cache blocks of every scale code, those that the writer gives only
to tiny blocks (0 to 2) or to none (from 247) among them: a request of one token
returns that token's latent, so what decoding makes of a block is what reading it gives."""

import numpy as np
import pytest
import torch

from block_quant_gemm_amd import mxq
from oracle import codec, latent, mx
from tests.gpu_helpers import host, say, to_dev, to_dev_bf16

pytestmark = pytest.mark.gpu


def _codes():
    """[256, 512] codes, row e for scale code e: all but the NaN codes, and those alone that
    stay finite in BF16 under 2^(e - 127)."""
    out = np.zeros((256, 512), np.uint8)
    every = np.array([c for c in range(256) if c & 0x7F != 0x7F], np.uint8)
    for e in range(256):
        with np.errstate(over="ignore", invalid="ignore"):
            v = mx.mx_dequantize(np.resize(every, (1, 512)), np.full((1, 16), min(e, 254), np.uint8))[0, :len(every)]
        ok = every[np.isfinite(codec.bf16_bits_to_f64(codec.bf16_round_to_bits(v)))]
        out[e] = np.resize(ok, 512)
    return out


@pytest.mark.parametrize("S,H", [(1, 1), (1, 20), (2, 40)])
def test_one_token_returns_its_latent(S, H):
    say(f"latent decode, one token under each scale code, S={S} H={H}")
    codes = _codes()
    scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 16, 1)
    cache = (to_dev(codes), to_dev(scales), torch.zeros((256, 64), dtype=torch.bfloat16, device="cuda"))
    q = torch.zeros((256, S, H, 576), dtype=torch.bfloat16, device="cuda")
    o, lse = mxq.mx_latent_decode(q, cache, to_dev(np.arange(256, dtype=np.int32)[:, None]),
                                  torch.ones(256, dtype=torch.int64, device="cuda"), 1, 1, 0.1)
    want = host(mxq.mx_latent_cache_read(cache, torch.arange(256, device="cuda"))[0])
    ref = latent.cache_read((codes, scales, np.zeros((256, 64), np.uint16)), np.arange(256))[0]
    got = host(o)[:, -1]                             # the last query token sees the token
    assert np.array_equal(want[:255], ref[:255])
    got, want = codec.bf16_bits_to_f64(got), codec.bf16_bits_to_f64(want)   # a sum has no minus 0
    off = [e for e in range(255) if not (got[e] == want[e][None]).all()]
    assert not off, f"scale codes {off}"
    assert np.isnan(got[255]).all() and np.isnan(want[255]).all()
    assert (lse[:255, -1] == 0).all()
