"""The gradient of expanded latent attention, what its exactness rests on: a sequence's
gradient does not depend on what shares the call, and where a query sees few keys it is
as exact as the rounding of the result allows."""

import numpy as np
import pytest
import torch

from block_quant_gemm_amd import mxq
from tests.gpu_helpers import say

pytestmark = pytest.mark.gpu

SCALE = 192 ** -0.5
GRADS = ("dq", "dk_nope", "dk_rope", "dv")


def _inputs(lq, lk, H, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s, sigma=1.0: (torch.randn(*s, generator=g, device="cuda") * sigma).to(torch.bfloat16)
    Tq, Tk = sum(lq), sum(lk)
    off = lambda n: torch.from_numpy(np.concatenate([[0], np.cumsum(n)]).astype(np.int64)).cuda()
    return {"q": rnd(Tq, H, 192), "k_nope": rnd(Tk, H, 128), "k_rope": rnd(Tk, 64), "v": rnd(Tk, H, 128),
            "do": rnd(Tq, H, 128, sigma=0.02), "oq": off(lq), "ok": off(lk), "lq": lq, "lk": lk}


def _run(d, causal):
    how = dict(offsets_q=d["oq"], offsets_k=d["ok"], scale=SCALE, causal=causal)
    t = (d["q"], d["k_nope"], d["k_rope"], d["v"])
    o, lse = mxq.latent_attention(*t, **how)
    return o, lse, dict(zip(GRADS, mxq.latent_attention_backward(d["do"], *t, o, lse, **how)))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens", [[60, 700, 1, 2, 17, 100, 400, 300], [20] * 40, [300, 129, 1000]])
def test_a_gradient_does_not_depend_on_what_shares_the_call(lens, causal):
    """Each sequence of a packed call against a call with that sequence alone, bit for bit."""
    H = 5
    say(f"latent attention backward, {lens} packed and alone, causal={causal}")
    d = _inputs(lens, lens, H, len(lens))
    o, lse, got = _run(d, causal)
    for b in sorted({0, 1, len(lens) // 2, len(lens) - 1}):
        r = slice(int(d["oq"][b]), int(d["oq"][b + 1]))
        t = [d[n][r] for n in ("q", "k_nope", "k_rope", "v")]
        one = mxq.latent_attention_backward(d["do"][r], *t, o[r], lse[:, r].contiguous(), scale=SCALE, causal=causal)
        for n, x in zip(GRADS, one):
            assert torch.equal(x.contiguous().view(torch.int16), got[n][r].contiguous().view(torch.int16)), (b, n)


def _exact(d, causal):
    """The gradients in 64 bits."""
    x = [d[n].double().requires_grad_() for n in ("q", "k_nope", "k_rope", "v")]
    outs = []
    for b, (lq, lk) in enumerate(zip(d["lq"], d["lk"])):
        rq, rk = (slice(int(d[n][b]), int(d[n][b + 1])) for n in ("oq", "ok"))
        k = torch.cat([x[1][rk], x[2][rk, None].expand(-1, x[1].shape[1], -1)], -1)
        z = torch.einsum("ihd,jhd->hij", x[0][rq], k) * SCALE
        if causal:
            z = z.masked_fill(torch.ones(lq, lk, dtype=torch.bool, device="cuda").triu(lk - lq + 1), -np.inf)
        outs.append(torch.einsum("hij,jhd->ihd", torch.softmax(z, -1), x[3][rk]))
    return dict(zip(GRADS, torch.autograd.grad(torch.cat(outs), x, d["do"].double())))


def _times_least(got, want):
    """The error of `got` against that of the exact result rounded once."""
    least = (want.to(torch.bfloat16).double() - want).norm()
    return ((got.double() - want).norm() / least).item()


@pytest.mark.parametrize("lq,lk,H,causal", [
    ([18], [18], 2, False), ([2], [2], 1, True), ([20] * 40, [20] * 40, 2, True), ([30] * 30, [30] * 30, 3, False),
    ([1, 5, 60, 33, 64] * 6, [1, 5, 60, 33, 64] * 6, 2, True), ([1] * 700, [40] * 700, 1, False),
    ([5] * 200, [9] * 200, 2, True)])
def test_where_queries_see_few_keys(lq, lk, H, causal):
    """At most 64 keys a query, in calls of few and of many rows: dS is handed on to 16 bits,
    so what is left is the rounding of the result and FP32 sums; 1.2 times the least."""
    say(f"latent attention backward, {len(lq)} sequences of {max(lq)} and fewer, {H} heads, causal={causal}")
    d = _inputs(lq, lk, H, 50 + len(lq))
    got, want = _run(d, causal)[2], _exact(d, causal)
    for n in ("dq", "dk_nope", "dk_rope"):
        r = _times_least(got[n], want[n])
        assert r < 1.2, f"{n}: {r:.3f} times the least error"


def test_the_first_rows_of_a_long_sequence():
    say("latent attention backward, the first rows of 1500")
    d = _inputs([1500, 700], [1500, 700], 3, 90)
    got, want = _run(d, True)[2], _exact(d, True)
    for r in (slice(0, 64), slice(1500, 1564)):
        assert _times_least(got["dq"][r], want["dq"][r]) < 1.2
    # evenly 2^0.5 from there on: two roundings of about the same size
    for n in GRADS:
        assert _times_least(got[n], want[n]) < 1.5, n
