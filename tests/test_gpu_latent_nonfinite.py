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
from oracle import codec, latent
from tests.gpu_helpers import host, say
from tests.test_gpu_latent_attention import SCALE, _f64, _run, _with_empty
from tests.test_gpu_latent_attention import _inputs as oracle_inputs

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


GRADS = ("dq", "dk_nope", "dk_rope", "dv")


def _backward(d, o, lse):
    return dict(zip(GRADS, mxq.latent_attention_backward(d["dout"], d["q"], d["k_nope"], d["k_rope"], d["v"], o, lse,
                                                         d["off_q"], d["off_k"])))


def _same(a, b):
    return torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


def _close(got, want):
    """Either side is off by at most (2 / 3)^0.5 * 2^-8 of its norm: two roundings to BF16, each
    spread evenly over half a unit in the last place."""
    e = ((got.double() - want.double()).norm() / want.double().norm()).item()
    assert e <= 2 * (2 / 3) ** 0.5 * 2.0 ** -8, f"off by {e:.3g}"


@pytest.mark.parametrize("what", [NAN, INF, -INF])
@pytest.mark.parametrize("lq,lk,H", [(2048, 2048, 8), (700, 700, 40), (300, 1500, 4)])
def test_backward_with_a_broken_gradient(lq, lk, H, what):
    """One value of one query's dO: that query's gradient and those of the keys that it sees are
    broken, dv in its column alone; nothing else is."""
    say(f"latent attention backward, {lq} queries {lk} keys {H} heads, one {what} in dO")
    d = _inputs(lq, lk, H, 3)
    o, lse = _forward(d)
    i, col = 220, 41
    d["dout"][i, :, col] = 0
    sound = dict(d)
    d = dict(d, dout=d["dout"].clone())
    d["dout"][i, :, col] = what
    got, ref = _backward(d, o, lse), _backward(sound, o, lse)
    j = i + lk - lq                                       # the last key that query i sees
    others = torch.arange(lq, device="cuda") != i
    assert not torch.isfinite(got["dq"][i]).any() and _same(got["dq"][others], ref["dq"][others])
    for n in ("dk_nope", "dk_rope"):
        assert not torch.isfinite(got[n][:j + 1]).any(), n
    hit = got["dv"][:j + 1, :, col].double()
    assert (torch.isnan(hit) if np.isnan(what) else hit == what).all()
    rest = torch.arange(128, device="cuda") != col
    _close(got["dv"][..., rest], ref["dv"][..., rest])
    apart = (j // 64 + 1) * 64 + 128                      # keys of no tile that query i is in
    for n in ("dk_nope", "dk_rope", "dv"):
        _close(got[n][j + 1:], ref[n][j + 1:])
        assert _same(got[n][apart:], ref[n][apart:]), n
    _in_time(lambda: _backward(d, o, lse), lambda: _backward(sound, o, lse), f"backward with one {what}")


@pytest.mark.parametrize("what", [NAN, INF])
def test_backward_with_broken_gradients_everywhere(what):
    say(f"latent attention backward, dO all {what}")
    d = _inputs(1500, 1500, 8, 4)
    o, lse = _forward(d)
    sound = dict(d)
    d = dict(d, dout=torch.full_like(d["dout"], what))
    got = _backward(d, o, lse)
    assert not any(torch.isfinite(got[n]).any() for n in ("dq", "dk_nope", "dk_rope"))
    assert (torch.isnan(got["dv"]) if np.isnan(what) else got["dv"] == what).all()
    _in_time(lambda: _backward(d, o, lse), lambda: _backward(sound, o, lse), f"backward with dO all {what}")


@pytest.mark.parametrize("where", ["k_nope", "k_rope", "v", "q"])
def test_backward_with_a_broken_operand(where):
    """One row's key, rotary key, value or query is NaN: queries before it have sound
    gradients, and, of a query, keys after it."""
    say(f"latent attention, forward and backward, a NaN in {where}")
    n, H, at = 1600, 8, 1000
    d = _inputs(n, n, H, 5)
    sound = dict(d)
    d = dict(d, **{where: d[where].clone()})
    d[where][at, ..., 9] = NAN
    (o, lse), (ro, rlse) = _forward(d), _forward(sound)
    got, ref = _backward(d, o, lse), _backward(sound, ro, rlse)
    assert (lse[:, :at] - rlse[:, :at]).abs().max() < 1e-4
    _close(o[:at], ro[:at])
    _close(got["dq"][:at], ref["dq"][:at])
    if where == "q":
        _close(got["dq"][at + 1:], ref["dq"][at + 1:])
        for g in ("dk_nope", "dk_rope", "dv"):
            _close(got[g][at + 1:], ref[g][at + 1:])
            assert not torch.isfinite(got[g][:at + 1]).any(), g
    else:
        # every query from there on sees it, and every key is seen by the last query
        assert not torch.isfinite(got["dq"][at:]).any()
        assert not torch.isfinite(got["dk_nope"]).any() and not torch.isfinite(got["dk_rope"]).any()
    _in_time(lambda: _backward(d, o, lse), lambda: _backward(sound, ro, rlse), f"backward with a NaN in {where}")


@pytest.mark.parametrize("n,H", [(64, 1), (200, 3), (700, 40)])
def test_hidden_nan_does_not_reach_a_key_of_minus_infinity(n, H):
    """A key whose logits are all minus infinity has probability 0 and gradient 0, whatever
    the queries hold that do not see it."""
    say(f"latent attention backward, a key of minus infinity, {n} rows {H} heads")
    d = _inputs(n, n, H, 6)
    j, i = 45, 40
    d["q"][..., 3] = d["q"][..., 3].abs() + 0.1
    d["k_nope"][j, :, 3] = -INF
    d["q"][i, :, 7] = NAN
    d["dout"][i, :, 7] = NAN
    o, lse = _forward(d)
    g = _backward(d, o, lse)
    for name in ("dk_nope", "dk_rope", "dv"):
        assert (g[name][j] == 0).all(), name
        assert not torch.isfinite(g[name][:i + 1]).any() or name == "dv"
        assert torch.isfinite(g[name][i + 1:]).all(), name


@pytest.mark.parametrize("lq,lk,H", [(100, 37, 2), (900, 300, 20)])
def test_a_row_that_sees_nothing_has_no_gradient(lq, lk, H):
    """More queries than keys: the first see none, and neither their own dO nor the keys after
    them make a gradient."""
    say(f"latent attention backward, rows that see nothing, {lq} queries {lk} keys {H} heads")
    d = _inputs(lq, lk, H, 7)
    first = lq - lk                                       # the first query that sees a key
    d["dout"][first - 9:first - 3, :, 5] = NAN
    d["dout"][first - 3:first, :, 5] = INF
    d["k_nope"][3, :, 11] = NAN
    d["k_rope"][5, 2] = -INF
    o, lse = _forward(d)
    g = _backward(d, o, lse)
    assert (o[:first] == 0).all() and torch.isneginf(lse[:, :first]).all()
    assert (g["dq"][:first] == 0).all()


def _decode_inputs(lens, S, H, seed):
    r, page = _rnd(seed), 32
    need = -(-max(lens) // page)
    cache = mxq.latent_cache(len(lens) * need * page)
    pages = torch.randperm(len(lens) * need, device="cuda", generator=torch.Generator("cuda").manual_seed(seed))
    pages = pages.view(len(lens), need).to(torch.int32)
    n = cache[0].shape[0]
    mxq.mx_latent_cache_write(r(n, 512), r(n, 64), torch.arange(n, device="cuda"), cache)
    return {"q": r(len(lens), S, H, 576, sigma=0.7), "cache": cache, "pages": pages, "page_size": page,
            "lens": torch.tensor(lens, device="cuda"), "max_len": max(lens), "scale": 192 ** -0.5}


def _slot(d, b, t):
    return int(d["pages"][b, t // d["page_size"]]) * d["page_size"] + t % d["page_size"]


@pytest.mark.parametrize("S,H,lens", [(2, 64, [5000, 700, 64]), (3, 5, [4000, 90]), (2, 16, [3000] * 8), (2, 8, [1200, 1])])
@pytest.mark.parametrize("where", ["seen", "last", "both"])
def test_decode_with_a_broken_token(S, H, lens, where):
    """A NaN block in a token that all query tokens of the first request see makes its rows NaN; in
    its last token, the last query token's rows alone.  Other requests do not notice."""
    say(f"latent decode, {len(lens)} requests, {S} tokens, {H} heads, a NaN token ({where})")
    d = _decode_inputs(lens, S, H, 8)
    ro, rlse = mxq.mx_latent_decode(**d)
    sound = dict(d, cache=tuple(t.clone() for t in d["cache"]))
    for t in {"seen": [lens[0] - 70], "last": [lens[0] - 1], "both": [lens[0] - 70, lens[0] - 1]}[where]:
        s = _slot(d, 0, t)
        d["cache"][0][s, 64:96] = 0x7F
        d["cache"][1][s, 2] = 0xFF
    o, lse = mxq.mx_latent_decode(**d)
    assert _same(o[1:], ro[1:]) and torch.equal(lse[1:], rlse[1:])
    assert torch.isnan(o[0, -1]).all() and torch.isnan(lse[0, -1]).all()
    if where == "last":
        assert (lse[0, :-1] - rlse[0, :-1]).abs().max() < 1e-4
        _near(o[0, :-1], ro[0, :-1], 6.0)                 # 6: the largest of the normal latents, nearly
    else:
        assert torch.isnan(o[0]).all() and torch.isnan(lse[0]).all()
    _in_time(lambda: mxq.mx_latent_decode(**d), lambda: mxq.mx_latent_decode(**sound), "decode with a NaN token")


def test_decode_with_nan_everywhere():
    say("latent decode, all tokens NaN")
    d = _decode_inputs([4000] * 6, 2, 64, 9)
    sound = dict(d, cache=tuple(t.clone() for t in d["cache"]))
    d["cache"][1].fill_(0xFF)
    o, lse = mxq.mx_latent_decode(**d)
    assert torch.isnan(o).all() and torch.isnan(lse).all()
    _in_time(lambda: mxq.mx_latent_decode(**d), lambda: mxq.mx_latent_decode(**sound), "decode with NaN everywhere")


@pytest.mark.parametrize("rows", [64, 128])
@pytest.mark.parametrize("seed", range(16))
def test_scattered_broken_values_against_the_oracle(seed, rows):
    """NaN and infinities at a few places of all operands, odd lengths: exactly the outputs that the
    definition makes not finite are not, of o and dv in kind, and the others are within the bounds."""
    rng = np.random.default_rng(seed)
    lq, lk, H = [int(n) for n in rng.integers(2, 230, 3)], [int(n) for n in rng.integers(2, 230, 3)], 2
    say(f"latent attention, scattered broken values, lq={lq} lk={lk}, {rows}-row workgroups")
    d = oracle_inputs(lq, lk, H, 300 + seed)
    for b in range(3):
        for name, n in (("q", lq[b]), ("do", lq[b]), ("kv", lk[b]), ("kr", lk[b])):
            first = int(d["oq" if name in ("q", "do") else "ok"][b])
            for _ in range(rng.integers(0, 3)):
                what = (0x7FC0, 0x7F80, 0xFF80)[rng.integers(0, 3)]
                # a sequence's first key stays sound, so that no row's logits are all minus infinity
                r = first + int(rng.integers(n // 2 if n > 1 else 0, n)) if name in ("q", "do") else \
                    first + int(rng.integers(max(1, n // 2), n))
                if name == "kr":
                    d[name][r, rng.integers(0, 64)] = what
                else:
                    d[name][r, rng.integers(0, H), rng.integers(0, d[name].shape[2])] = what
    with np.errstate(all="ignore"):
        ref = latent.attention_backward(codec.bf16_bits_to_f64(d["do"]), *_f64(d), d["oq"], d["ok"], SCALE, True)
    run = d if rows == 64 else _with_empty(d)
    for n in ("q", "kr"):
        assert mxq.latent_backward_rows(d[n].shape[0], H, len(run["oq"]) - 1) == rows
    got = _run(run, True)
    for name, (val, err) in ref.items():
        g = host(got[name].contiguous())
        g = g.astype(np.float64) if name == "lse" else codec.bf16_bits_to_f64(g)
        ok = np.isfinite(val)
        if name in ("o", "dv", "lse"):
            assert np.array_equal(g[~ok], val[~ok], equal_nan=True), name
        assert np.array_equal(np.isfinite(g), ok), (name, int((np.isfinite(g) != ok).sum()))
        tol = np.where(np.isnan(err), np.inf, err)[ok]
        assert (np.abs(g[ok] - val[ok]) <= tol).all(), name
