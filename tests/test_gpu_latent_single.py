"""Tensors with a dimension of one, whose stride means nothing and may be anything: the calls
take them, and give what they give for the same values in an ordinary layout."""

import pytest
import torch

from block_quant_gemm_amd import mxq
from tests.gpu_helpers import say

pytestmark = pytest.mark.gpu


def _odd(t):
    """The same values and memory, every stride of a dimension of one (but the last) set to 1."""
    return t.as_strided(t.shape, [1 if n == 1 and i + 1 < t.dim() else s
                                  for i, (n, s) in enumerate(zip(t.shape, t.stride()))], t.storage_offset())


def _rnd(*s):
    return torch.randn(*s, device="cuda").to(torch.bfloat16)


def _same(a, b):
    for x, y in zip(a, b):
        assert torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))


@pytest.mark.parametrize("slots", [1, 5])
def test_cache_of_one_token(slots):
    say(f"latent cache, one token of {slots} slots")
    torch.manual_seed(0)
    c, kr = _rnd(1, 512), _rnd(1, 64)
    at = torch.tensor([slots - 1], device="cuda")
    plain, odd = mxq.latent_cache(slots), tuple(_odd(t) for t in mxq.latent_cache(slots))
    _same(mxq.mx_latent_cache_write(_odd(c), _odd(kr), at, odd), mxq.mx_latent_cache_write(c, kr, at, plain))
    out = _odd(torch.empty_like(c)), _odd(torch.empty_like(kr))
    _same(mxq.mx_latent_cache_read(odd, at, *out), mxq.mx_latent_cache_read(plain, at))
    _same(out, mxq.mx_latent_cache_read(plain, at))


@pytest.mark.parametrize("B,S,H", [(1, 1, 1), (1, 1, 16), (3, 1, 16), (1, 2, 1), (2, 2, 1)])
def test_decode(B, S, H):
    say(f"latent decode, B={B} S={S} H={H}")
    torch.manual_seed(1)
    cache = mxq.latent_cache(256)
    mxq.mx_latent_cache_write(_rnd(256, 512), _rnd(256, 64), torch.arange(256, device="cuda"), cache)
    q, lens = _rnd(B, S, H, 576), torch.full((B,), 70, device="cuda")
    pages = torch.arange(B, device="cuda", dtype=torch.int32).view(B, 1)
    want = mxq.mx_latent_decode(q, cache, pages, lens, 80, 70, 0.07)
    o = _odd(torch.empty_like(want[0]))
    _same(mxq.mx_latent_decode(_odd(q), cache, _odd(pages), lens, 80, 70, 0.07, o=o), want)


@pytest.mark.parametrize("Tq,Tk,H", [(1, 1, 1), (1, 90, 1), (1, 90, 4), (70, 1, 2), (70, 90, 1), (1, 1, 5)])
def test_attention(Tq, Tk, H):
    say(f"latent attention, Tq={Tq} Tk={Tk} H={H}")
    torch.manual_seed(2)
    t = [_rnd(Tq, H, 192), _rnd(Tk, H, 128), _rnd(Tk, 64), _rnd(Tk, H, 128)]
    do = _rnd(Tq, H, 128)
    want = mxq.latent_attention(*t)
    grads = mxq.latent_attention_backward(do, *t, *want)
    odd = [_odd(x) for x in t]
    got = mxq.latent_attention(*odd, o=_odd(torch.empty_like(want[0])), lse=_odd(torch.empty_like(want[1])))
    _same(got, want)
    out = dict(zip(("dq", "dk_nope", "dk_rope", "dv"), (_odd(torch.empty_like(x, memory_format=torch.contiguous_format))
                                                       for x in grads)))
    _same(mxq.latent_attention_backward(_odd(do), *odd, *got, **out), grads)
