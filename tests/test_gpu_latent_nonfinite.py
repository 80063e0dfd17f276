"""Expanded and absorbed latent attention where operands hold NaN or infinities: what a
row sees reaches it, what the mask hides does not, and a call with such values takes a
small multiple of a sound call's time, whatever they are and wherever they stand.

Times: rows that a hidden value may have reached are walked a second time, in which only
the tiles that the mask cuts are added key by key; so twice the sound call and those
tiles.  The bound is eight times the sound call, and 100 us for the shortest."""

import numpy as np
import pytest
import torch

from block_quant_gemm_amd import mxq
from tests.gpu_helpers import say

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


def _rnd(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *s, sigma=1.0: (torch.randn(*s, generator=g, device="cuda") * sigma).to(torch.bfloat16)


def _inputs(lq, lk, H, seed):
    r = _rnd(seed)
    kv = r(lk, H, 256)
    return {"q": r(lq, H, 192), "k_nope": kv[..., :128].contiguous(), "k_rope": r(lk, 64),
            "v": kv[..., 128:].contiguous(), "dout": r(lq, H, 128, sigma=0.02),
            "off_q": torch.tensor([0, lq], device="cuda"), "off_k": torch.tensor([0, lk], device="cuda")}


def _forward(d):
    return mxq.latent_attention(d["q"], d["k_nope"], d["k_rope"], d["v"], d["off_q"], d["off_k"])


def _us(f, n=5):
    """Median time of a call on the GPU, in microseconds."""
    f()
    t = []
    for _ in range(n):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        f()
        b.record()
        b.synchronize()
        t.append(1e3 * a.elapsed_time(b))
    return float(np.median(t))


def _in_time(broken, sound, what):
    tb, ts = _us(broken), _us(sound)
    say(f"{what}: {tb:.0f} us, the sound call {ts:.0f}")
    assert tb < 8 * ts + 100, f"{what}: {tb:.0f} us, the sound call {ts:.0f}"


def _near(got, want, size):
    """Equal but for the rounding of P and of the result, at most 2^-8 each on either side,
    relative to the largest operand `size` of the average."""
    d = (got.double() - want.double()).abs().max().item()
    assert d <= 4 * 2.0 ** -8 * size, f"off by {d:.3g}"


@pytest.mark.parametrize("what", [NAN, INF, -INF])
@pytest.mark.parametrize("lq,lk,H", [(2048, 2048, 8), (700, 700, 40), (64, 3000, 4)])
def test_forward_with_a_broken_value(lq, lk, H, what):
    """One value of one row: the rows before do not see it, the others have it in its column."""
    say(f"latent attention, {lq} queries {lk} keys {H} heads, one {what} among the values")
    d = _inputs(lq, lk, H, 1)
    j, col = lk - 29 if lk > lq else 500, 77
    d["v"][j, :, col] = 0
    sound = dict(d)
    d = dict(d, v=d["v"].clone())
    d["v"][j, :, col] = what
    o, lse = _forward(d)
    ro, rlse = _forward(sound)
    i = j - (lk - lq)                                     # the first query that sees key j
    apart = max(0, i - 63)                                # rows of no tile that holds key j
    assert torch.equal(lse[:, :apart], rlse[:, :apart]) and (lse - rlse).abs().max() < 1e-4
    got = o[i:, :, col].double()
    assert (torch.isnan(got) if np.isnan(what) else got == what).all()
    rest = torch.arange(128, device="cuda") != col
    size = d["v"][..., rest].abs().max().item()
    _near(o[:, :, rest], ro[:, :, rest], size)
    _near(o[:i, :, col], ro[:i, :, col], sound["v"][..., col].abs().max().item())
    _in_time(lambda: _forward(d), lambda: _forward(sound), f"forward with one {what}")


@pytest.mark.parametrize("what", [NAN, INF])
def test_forward_with_broken_values_everywhere(what):
    say(f"latent attention, all values {what}")
    d = _inputs(1500, 1500, 8, 2)
    sound = dict(d)
    d = dict(d, v=torch.full_like(d["v"], what))
    o, _ = _forward(d)
    assert (torch.isnan(o) if np.isnan(what) else o == what).all()
    _in_time(lambda: _forward(d), lambda: _forward(sound), f"forward with all values {what}")
