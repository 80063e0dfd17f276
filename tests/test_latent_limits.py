"""The sizes that the header says the gradient of latent attention takes, up to their limits:
such a call passes every host check and reaches the launch.  Runs where no GPU is visible
(the addresses are made up and the launch fails for want of a device).  CPU only."""

import pytest

from block_quant_gemm_amd import mxq
from tests.test_library import host_only_lib, lib  # noqa: F401

SHAPE, HIP = 2, 6
P, BIG = 4096, 1 << 62


def _backward(lib, Tq, Tk, B, H):
    row = 1 << 20                                         # strides: rows and heads may lie as they like
    attn = mxq._ATTN_STRUCT.pack(P, row, 192, P, row, 128, P, 64, P, row, 128, P, P, Tq, Tk, B, H, 0.07, 1)
    return lib.latent_attention_backward(attn, P, row, 128, P, max(Tq, 1), P, row, 128, P, row, 192, P, row, 128, P, 64,
                                         P, row, 128, P, BIG, None)


@pytest.mark.parametrize("Tq,Tk,B,H", [
    (100, 1 << 27, 1, 7), (512, 1 << 26, 3, 15), (1, 1 << 24, 1, 63), (1 << 26, 100, 2, 15), (513, 1 << 27, 1, 7),
    (0, 1 << 27, 1, 7), (100, 100, 8191, 1023), (64, 64, 63, 65536)])
def test_documented_sizes_are_taken(host_only_lib, Tq, Tk, B, H):  # noqa: F811
    assert (Tq // 128 + B) * H < 1 << 23 and (Tk // 128 + B) * H < 1 << 23
    assert _backward(host_only_lib, Tq, Tk, B, H) == HIP


@pytest.mark.parametrize("Tq,Tk,B,H", [(100, 1 << 27, 1, 8), (1 << 27, 100, 1, 8), (100, 100, 8192, 1024)])
def test_larger_ones_are_refused(host_only_lib, Tq, Tk, B, H):  # noqa: F811
    assert _backward(host_only_lib, Tq, Tk, B, H) == SHAPE


@pytest.mark.parametrize("scale,want", [(2e38, HIP), (2.4e38, 4), (3.4e38, 4), (1e-44, HIP)])
def test_scales_whose_power_of_two_form_overflows_are_refused(host_only_lib, scale, want):  # noqa: F811
    """The exponentials are taken of scale * log2(e) times the products."""
    attn = mxq._ATTN_STRUCT.pack(P, 384, 192, P, 256, 128, P, 64, P, 256, 128, P, P, 10, 10, 1, 2, scale, 1)
    assert host_only_lib.latent_attention(attn, P, 256, 128, P, 10, P, BIG, None) == want
    assert host_only_lib.latent_attention_backward(attn, P, 256, 128, P, 10, P, 256, 128, P, 384, 192, P, 256, 128, P, 64,
                                                   P, 256, 128, P, BIG, None) == want
    cache = mxq._CACHE_STRUCT.pack(P, 512, P, 16, P, 64, 64)
    assert host_only_lib.mx_latent_decode(P, 1152, 1152, 576, cache, P, 4, 4, 8, P, 2, 1, 2, 32, scale, P, 1024, 1024, 512,
                                          P, P, BIG, None) == want
