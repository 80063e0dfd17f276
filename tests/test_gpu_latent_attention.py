"""Expanded latent attention and its gradient on the GPU against the float64
oracle, within bounds derived from the formats (oracle.latent); rows without
keys, hidden NaN and infinities, strides, shared rotary key, repeatability."""

import numpy as np
import pytest
import torch

from block_quant_gemm_amd import mxq, workloads
from oracle import codec, latent
from tests.gpu_helpers import host, say, to_dev, to_dev_bf16

pytestmark = pytest.mark.gpu

SCALE = 192 ** -0.5


def _bits(shape, seed, name, sigma=1.0):
    return workloads.bf16_normal(shape, sigma, seed=seed, name=name)


def _inputs(lq, lk, H, seed, sigma=1.0):
    Tq, Tk = sum(lq), sum(lk)
    d = {"q": _bits((Tq, H, 192), seed, "aq", sigma), "kv": _bits((Tk, H, 256), seed, "akv"),
         "kr": _bits((Tk, 64), seed, "akr"), "do": _bits((Tq, H, 128), seed, "ado", 0.02)}
    d["oq"] = np.concatenate([[0], np.cumsum(lq)]).astype(np.int64)
    d["ok"] = np.concatenate([[0], np.cumsum(lk)]).astype(np.int64)
    return d


def _device(d):
    kv = to_dev_bf16(d["kv"])
    return (to_dev_bf16(d["q"]), kv[..., :128], to_dev_bf16(d["kr"]), kv[..., 128:])


def _f64(d):
    kv = codec.bf16_bits_to_f64(d["kv"])
    return (codec.bf16_bits_to_f64(d["q"]), kv[..., :128], codec.bf16_bits_to_f64(d["kr"]), kv[..., 128:])


def _run(d, causal, scale=SCALE, **kw):
    t = _device(d)
    how = dict(offsets_q=to_dev(d["oq"]), offsets_k=to_dev(d["ok"]), scale=scale, causal=causal)
    o, lse = mxq.latent_attention(*t, **how, **kw)
    dq, dkn, dkr, dv = mxq.latent_attention_backward(to_dev_bf16(d["do"]), *t, o, lse, **how)
    return {"o": o, "lse": lse, "dq": dq, "dk_nope": dkn, "dk_rope": dkr, "dv": dv}


def _compare(got, ref):
    for name, (val, err) in ref.items():
        g = host(got[name])
        g = g.astype(np.float64) if name == "lse" else codec.bf16_bits_to_f64(g)
        inf = np.isneginf(val)
        assert np.array_equal(np.isneginf(g), inf), name
        d = np.abs(g[~inf] - val[~inf])
        assert np.isfinite(d).all(), f"{name}: not finite"
        tol = err[~inf]
        assert (d <= tol).all(), f"{name} off by {np.max(d / np.maximum(tol, 1e-300)):.3g} of its bound"


CASES = [
    # query lengths, key lengths, heads, causal
    ([1], [1], 1, True),
    ([5], [5], 2, False),
    ([77], [77], 3, True),
    ([64, 128], [64, 128], 1, True),
    ([129, 1, 0, 63], [129, 1, 0, 63], 2, True),
    ([130], [200], 2, True),                     # keys before the queries
    ([1, 1, 3], [65, 300, 64], 2, True),
    ([100, 40], [37, 0], 2, True),               # more queries than keys: rows that see nothing
    ([50, 70], [0, 90], 1, False),               # a sequence without keys
    ([0, 33], [40, 33], 1, True),                # keys that no query sees
    ([140], [70], 2, False),
    ([257], [257], 1, True),
    ([300, 17], [300, 17], 5, True),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_forward_and_backward(case):
    lq, lk, H, causal = CASES[case]
    say(f"latent attention lq={lq} lk={lk} H={H} causal={causal}")
    d = _inputs(lq, lk, H, case)
    ref = latent.attention_backward(codec.bf16_bits_to_f64(d["do"]), *_f64(d), d["oq"], d["ok"],
                                    SCALE, causal)
    _compare(_run(d, causal), ref)


@pytest.mark.parametrize("sigma,scale", [(12.0, 1.0), (1.0, 1e-4), (0.0, 1.0)])
def test_extreme_logits(sigma, scale):
    say(f"latent attention sigma={sigma} scale={scale}")
    d = _inputs([150], [150], 2, 40, sigma)
    ref = latent.attention_backward(codec.bf16_bits_to_f64(d["do"]), *_f64(d), d["oq"], d["ok"],
                                    scale, True)
    _compare(_run(d, True, scale), ref)


def test_rising_logits_move_the_reference():
    """Logits that rise by hundreds along the keys: every tile moves the running maximum."""
    say("latent attention, rising logits")
    d = _inputs([320], [320], 1, 41)
    d["q"][:] = _bits((1, 1, 192), 3, "one")
    kv = d["kv"]
    one = codec.bf16_bits_to_f64(d["q"][0, 0, :128])
    ramp = np.arange(320)[:, None] * one[None] * 0.02
    kv[:, 0, :128] = codec.bf16_round_to_bits(ramp)
    for causal in (True, False):
        ref = latent.attention_backward(codec.bf16_bits_to_f64(d["do"]), *_f64(d), d["oq"],
                                        d["ok"], SCALE, causal)
        _compare(_run(d, causal), ref)


def test_one_sequence_without_offsets():
    say("latent attention without offsets")
    d = _inputs([90], [100], 2, 50)
    t = _device(d)
    o, lse = mxq.latent_attention(*t)
    g = mxq.latent_attention_backward(to_dev_bf16(d["do"]), *t, o, lse)
    ref = latent.attention_backward(codec.bf16_bits_to_f64(d["do"]), *_f64(d), None, None, SCALE, True)
    _compare(dict(zip(("o", "lse", "dq", "dk_nope", "dk_rope", "dv"), (o, lse, *g))), ref)


def test_strided_operands_and_results():
    """Row and head strides of their own for every operand and result; bytes between rows stay."""
    say("latent attention, strided")
    lq, H = [100, 61], 3
    d = _inputs(lq, lq, H, 60)
    T = sum(lq)

    def wide(bits, cols, fill=9.0):
        big = torch.full((T + 2, H + 1, cols + 24), fill, dtype=torch.bfloat16, device="cuda")
        v = big[1:T + 1, :H, 8:8 + cols]
        if bits is not None:
            v.copy_(to_dev_bf16(bits))
        return big, v

    _, q = wide(d["q"], 192)
    _, kn = wide(np.ascontiguousarray(d["kv"][..., :128]), 128)
    _, v = wide(np.ascontiguousarray(d["kv"][..., 128:]), 128)
    _, do = wide(d["do"], 128)
    kr = torch.full((T, 576), float("nan"), dtype=torch.bfloat16, device="cuda")[:, 512:]
    kr.copy_(to_dev_bf16(d["kr"]))
    bo, o = wide(None, 128)
    lse = torch.full((H, T + 5), 4.0, device="cuda")
    off = to_dev(d["oq"])
    mxq.latent_attention(q, kn, kr, v, off, o=o, lse=lse[:, :T])
    bdq, dq = wide(None, 192)
    bdk, dkn = wide(None, 128)
    bdv, dv = wide(None, 128)
    bdr = torch.full((T, 72), 9.0, dtype=torch.bfloat16, device="cuda")
    mxq.latent_attention_backward(do, q, kn, kr, v, o, lse[:, :T], off, dq=dq, dk_nope=dkn,
                                  dk_rope=bdr[:, :64], dv=dv)
    ref = latent.attention_backward(codec.bf16_bits_to_f64(d["do"]), *_f64(d), d["oq"], d["ok"],
                                    SCALE, True)
    got = {"o": o, "lse": lse[:, :T], "dq": dq, "dk_nope": dkn, "dk_rope": bdr[:, :64], "dv": dv}
    _compare({n: x.contiguous() for n, x in got.items()}, ref)
    for big, cols in ((bo, 128), (bdq, 192), (bdk, 128), (bdv, 128)):
        big[1:T + 1, :H, 8:8 + cols] = 9.0
        assert (big == 9.0).all()
    assert (lse[:, T:] == 4.0).all() and (bdr[:, 64:] == 9.0).all()


def _bad_rows(d, rows, what):
    """NaN or infinity in all operands of these rows (same numbering for queries and keys)."""
    for r in rows:
        d["q"][r, 0, 3] = what
        d["kv"][r, 0, 5] = what
        d["kv"][r, 0, 140] = what
        d["kr"][r, 7] = what
        d["do"][r, 0, 9] = what


@pytest.mark.parametrize("what", [0x7FC0, 0x7F80])
def test_hidden_nan_and_infinity_stay_hidden(what):
    """Rows from 70 on are broken.  Under the causal mask the queries before see
    only sound keys: their outputs and gradients are those of the sound prefix.
    Keys are seen by broken queries, so their gradients are broken; and a key
    after every broken query is not."""
    say(f"latent attention, rows of {what:#x}")
    n, cut = 150, 70
    d = _inputs([n], [n], 1, 70)
    sound = {k: (v[:cut].copy() if k not in ("oq", "ok") else np.array([0, cut])) for k, v in d.items()}
    _bad_rows(d, range(cut, n, 7), what)
    got = _run(d, True)
    ref = latent.attention_backward(codec.bf16_bits_to_f64(sound["do"]), *_f64(sound), sound["oq"],
                                    sound["ok"], SCALE, True)
    for name in ("o", "dq"):
        _compare({name: got[name][:cut]}, {name: ref[name]})
    _compare({"lse": got["lse"][:, :cut].contiguous()}, {"lse": ref["lse"]})

    # broken queries and gradients in the first rows: keys after them are not touched
    d = _inputs([n], [n], 1, 71)
    for r in range(0, 20, 3):
        d["q"][r, 0, 3] = what
        d["do"][r, 0, 9] = what
    got = _run(d, True)
    full = latent.attention_backward(
        np.where(np.isfinite(x := codec.bf16_bits_to_f64(d["do"])), x, 0.0),
        *[np.where(np.isfinite(y), y, 0.0) for y in _f64(d)], d["oq"], d["ok"], SCALE, True)
    for name in ("dk_nope", "dk_rope", "dv"):
        val, err = full[name]
        _compare({name: got[name][19:]}, {name: (val[19:], err[19:])})


def test_other_sequences_nan_does_not_reach():
    say("latent attention, NaN in a neighbouring sequence")
    d = _inputs([40, 50, 30], [40, 50, 30], 2, 72)
    for k in ("q", "kv", "kr", "do"):
        d[k][40:90] = 0x7FC0
    got = _run(d, False)
    d2 = {k: np.concatenate([d[k][:40], d[k][90:]]) for k in ("q", "kv", "kr", "do")}
    o2 = np.array([0, 40, 70], np.int64)
    kv = codec.bf16_bits_to_f64(d2["kv"])
    ref = latent.attention_backward(codec.bf16_bits_to_f64(d2["do"]), codec.bf16_bits_to_f64(d2["q"]),
                                    kv[..., :128], codec.bf16_bits_to_f64(d2["kr"]), kv[..., 128:],
                                    o2, o2, SCALE, False)
    keep = torch.tensor(list(range(40)) + list(range(90, 120)), device="cuda")
    _compare({n: (x[:, keep] if n == "lse" else x[keep]).contiguous() for n, x in got.items()}, ref)


def test_malformed_offsets_stay_inside():
    """Offsets out of range, decreasing or overlapping: unspecified values in those
    sequences' rows, nothing else; a sound sequence beside them is right."""
    say("latent attention, malformed offsets")
    d = _inputs([60, 80], [60, 80], 1, 73)
    t = _device(d)
    for bad in ([0, 60, 10 ** 12], [-50, 60, 140], [100, 60, 140], [0, 140, 60]):
        off = to_dev(np.array(bad, np.int64))
        o, lse = mxq.latent_attention(*t, off)
        mxq.latent_attention_backward(to_dev_bf16(d["do"]), *t, o, lse, off)
    torch.cuda.synchronize()
    got = _run(d, True)
    ref = latent.attention_backward(codec.bf16_bits_to_f64(d["do"]), *_f64(d), d["oq"], d["ok"],
                                    SCALE, True)
    _compare(got, ref)


def test_empty_inputs():
    say("latent attention, empty")
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")
    o, lse = mxq.latent_attention(z(0, 2, 192), z(0, 2, 128), z(0, 64), z(0, 2, 128))
    assert o.shape == (0, 2, 128)
    k = (z(9, 2, 128), z(9, 64), z(9, 2, 128))
    o, lse = mxq.latent_attention(z(0, 2, 192), *k)
    g = mxq.latent_attention_backward(z(0, 2, 128), z(0, 2, 192), *k, o, lse)
    assert all((x == 0).all() for x in g[1:])             # keys that no query sees
    q = z(9, 2, 192)
    o, lse = mxq.latent_attention(q, z(0, 2, 128), z(0, 64), z(0, 2, 128))
    assert (o == 0).all() and torch.isneginf(lse).all()
    dq = mxq.latent_attention_backward(z(9, 2, 128), q, z(0, 2, 128), z(0, 64), z(0, 2, 128), o, lse)[0]
    assert (dq == 0).all()


def test_repeats_give_the_same_bits():
    say("latent attention, repeated")
    lens = [700, 1, 333]
    d = _inputs(lens, lens, 4, 80)
    first = {n: x.clone() for n, x in _run(d, True).items()}
    for _ in range(3):
        for n, x in _run(d, True).items():
            assert torch.equal(x.view(torch.int16), first[n].view(torch.int16)), n


@pytest.mark.parametrize("H,lens", [(16, [2048, 1111]), (32, [1500])])
def test_long_rows_against_64_bit_products(H, lens):
    """Sizes of real layers, against float64 products on the GPU."""
    say(f"latent attention H={H} lens={lens}")
    g = torch.Generator(device="cuda").manual_seed(H)
    T = sum(lens)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
    q, kv, kr, do = rnd(T, H, 192), rnd(T, H, 256), rnd(T, 64), rnd(T, H, 128)
    off = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), device="cuda")
    kn, v = kv[..., :128], kv[..., 128:]
    o, lse = mxq.latent_attention(q, kn, kr, v, off)
    got = dict(zip(("dq", "dk_nope", "dk_rope", "dv"),
                   mxq.latent_attention_backward(do, q, kn, kr, v, o, lse, off)), o=o)
    x = [t.double().requires_grad_() for t in (q, kn, kr, v)]
    outs, at = [], 0
    for n in lens:
        r = slice(at, at + n)
        k = torch.cat([x[1][r], x[2][r, None].expand(-1, H, -1)], -1)
        z = torch.einsum("ihd,jhd->hij", x[0][r], k) * SCALE
        z = z.masked_fill(torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1), -np.inf)
        outs.append(torch.einsum("hij,jhd->ihd", torch.softmax(z, -1), x[3][r]))
        assert (lse[:, r] - torch.logsumexp(z.detach(), -1)).abs().max() < 2e-5
        at += n
    ref = torch.cat(outs)
    grads = torch.autograd.grad(ref, x, do.double())
    # independent roundings of P (or dS) and of the result: each is spread evenly over half a
    # unit in the last place, at most 2^-8, so 2^-8 / sqrt(3) in the root mean square
    for name, r in zip(("o", "dq", "dk_nope", "dk_rope", "dv"), (ref.detach(), *grads)):
        e = ((got[name].double() - r).norm() / r.norm()).item()
        assert e < (2 / 3) ** 0.5 * 2 ** -8, f"{name}: {e:.3g}"


def _with_empty(d, n=600):
    """The same sequences and n empty ones after them: more workgroups than a small
    call has, which decides how many rows one of them takes."""
    return {k: np.concatenate([v, np.full(n, v[-1])]) if k in ("oq", "ok") else v for k, v in d.items()}


@pytest.mark.parametrize("case", range(len(CASES)))
def test_with_many_empty_sequences(case):
    """Both workgroup sizes of the backward kernels, against the oracle and bit for bit."""
    lq, lk, H, causal = CASES[case]
    say(f"latent attention and 600 empty sequences, lq={lq} lk={lk} H={H} causal={causal}")
    d = _inputs(lq, lk, H, case)
    few, many = _run(d, causal), _run(_with_empty(d), causal)
    ref = latent.attention_backward(codec.bf16_bits_to_f64(d["do"]), *_f64(d), d["oq"], d["ok"],
                                    SCALE, causal)
    _compare(many, ref)
    for n, x in few.items():
        assert torch.equal(x.contiguous().view(torch.int16), many[n].contiguous().view(torch.int16)), n


@pytest.mark.parametrize("what", [0x7FC0, 0x7F80])
def test_hidden_nan_with_many_empty_sequences(what):
    say(f"latent attention and 600 empty sequences, rows of {what:#x}")
    n, cut = 150, 70
    d = _inputs([n], [n], 1, 70)
    sound = {k: (v[:cut].copy() if k not in ("oq", "ok") else np.array([0, cut])) for k, v in d.items()}
    _bad_rows(d, range(cut, n, 7), what)
    got = _run(_with_empty(d), True)
    ref = latent.attention_backward(codec.bf16_bits_to_f64(sound["do"]), *_f64(sound), sound["oq"],
                                    sound["ok"], SCALE, True)
    for name in ("o", "dq"):
        _compare({name: got[name][:cut]}, {name: ref[name]})
    few = _run(d, True)
    for name in ("dk_nope", "dk_rope", "dv"):
        a, b = host(few[name].contiguous()), host(got[name].contiguous())
        nan = lambda x: ~np.isfinite(codec.bf16_bits_to_f64(x))
        assert np.array_equal(nan(a), nan(b)) and np.array_equal(a[~nan(a)], b[~nan(b)]), name


@pytest.mark.parametrize("H,lens", [(64, [300, 0, 513, 129]), (64, [700, 90, 400]), (128, [140, 1, 128, 600]),
                                    (256, [129, 300]), (300, [130, 65]), (51, [900])])
def test_many_workgroups(H, lens):
    """More than 256 workgroups, which start two to a CU: every tile is taken once, and each
    head's rows are what a call with that head alone gives, bit for bit."""
    say(f"latent attention H={H} lens={lens}")
    d = _inputs(lens, lens, H, H)
    for causal in (True, False):
        got = _run(d, causal)
        for h in (0, H // 2, H - 1):
            one = {k: v if k in ("oq", "ok", "kr") else np.ascontiguousarray(v[:, h:h + 1]) for k, v in d.items()}
            ref = _run(one, causal)
            for n in ("o", "dq", "dk_nope", "dv"):
                assert torch.equal(got[n][:, h:h + 1].contiguous().view(torch.int16),
                                   ref[n].contiguous().view(torch.int16)), (n, h)
            assert torch.equal(got["lse"][h], ref["lse"][0]), h


SPLIT = [
    # few queries, many keys: query lengths, key lengths, heads, causal
    ([16], [4100], 2, True),
    ([1], [2600], 3, False),
    ([130], [1500], 2, True),
    ([1300], [1090], 1, True),                   # more queries than keys: rows that see nothing
    ([40, 0, 3, 200], [2100, 1500, 2, 1700], 2, True),
    ([64, 129], [3000, 700], 1, False),
]


@pytest.mark.parametrize("case", range(len(SPLIT)))
def test_few_queries_many_keys(case):
    """Calls whose tiles' keys several workgroups take between them."""
    lq, lk, H, causal = SPLIT[case]
    say(f"latent attention lq={lq} lk={lk} H={H} causal={causal}")
    assert mxq.workspace_size(mxq.WS_LATENT_FORWARD, sum(lq), sum(lk), H, len(lq)) > 0
    d = _inputs(lq, lk, H, 100 + case)
    ref = latent.attention_backward(codec.bf16_bits_to_f64(d["do"]), *_f64(d), d["oq"], d["ok"],
                                    SCALE, causal)
    got = _run(d, causal)
    _compare(got, ref)
    again = _run(d, causal)
    for n in got:
        assert torch.equal(got[n].contiguous().view(torch.int16), again[n].contiguous().view(torch.int16)), n


@pytest.mark.parametrize("what", [0x7FC0, 0x7F80])
def test_hidden_nan_with_few_queries_many_keys(what):
    """The last queries and their keys are broken: those before see sound keys only."""
    say(f"latent attention 60 queries after 1940 keys, rows of {what:#x}")
    lq, lk, cut = 60, 2000, 45
    d = _inputs([lq], [lk], 2, 120)
    sound = {k: v.copy() for k, v in d.items()}
    sound["q"], sound["do"] = d["q"][:cut].copy(), d["do"][:cut].copy()
    sound["kv"], sound["kr"] = d["kv"][:lk - lq + cut].copy(), d["kr"][:lk - lq + cut].copy()
    sound["oq"], sound["ok"] = np.array([0, cut]), np.array([0, lk - lq + cut])
    for r in range(cut, lq, 4):
        d["q"][r, 0, 3] = what
        d["kv"][lk - lq + r, :, 5] = what
        d["kv"][lk - lq + r, :, 140] = what
        d["kr"][lk - lq + r, 7] = what
    t = _device(d)
    o, lse = mxq.latent_attention(*t, to_dev(d["oq"]), to_dev(d["ok"]))
    ref = latent.attention_backward(codec.bf16_bits_to_f64(sound["do"]), *_f64(sound), sound["oq"],
                                    sound["ok"], SCALE, True)
    _compare({"o": o[:cut].contiguous(), "lse": lse[:, :cut].contiguous()},
             {n: ref[n] for n in ("o", "lse")})


@pytest.mark.parametrize("what", [0x7FC0, 0x7F80])
def test_hidden_nan_in_large_calls(what):
    """The forms that large calls take, with broken rows: each head's finite values are those
    of a call with that head alone, and the same ones are not finite."""
    say(f"latent attention 40 heads, rows of {what:#x}")
    n, H = 1100, 40
    d = _inputs([n], [n], H, 130)
    for h in (0, 17, H - 1):
        for r in (700, 955, n - 1):
            d["q"][r, h, 3] = what
            d["kv"][r, h, 5] = what
            d["kv"][r, h, 140] = what
            d["do"][r, h, 9] = what
    got = _run(d, True)
    for h in (0, 5, 17, H - 1):
        one = {k: v if k in ("oq", "ok", "kr") else np.ascontiguousarray(v[:, h:h + 1]) for k, v in d.items()}
        ref = _run(one, True)
        for name in ("o", "dq", "dk_nope", "dv"):
            a, b = host(got[name][:, h:h + 1].contiguous()), host(ref[name].contiguous())
            va, vb = codec.bf16_bits_to_f64(a), codec.bf16_bits_to_f64(b)
            assert np.array_equal(np.isfinite(va), np.isfinite(vb)), (name, h)
            assert h == 5 or not np.isfinite(va).all(), (name, h)
            ok = np.isfinite(va)
            if ok.any():                                  # every key is seen by a broken query
                assert np.abs(va[ok] - vb[ok]).max() <= 2 ** -6 * np.abs(vb[ok]).max(), (name, h)
        clean = slice(0, 700)                             # rows before the first broken one
        assert np.isfinite(codec.bf16_bits_to_f64(host(got["o"][clean, h].contiguous()))).all()
        assert np.isfinite(codec.bf16_bits_to_f64(host(got["dq"][clean, h].contiguous()))).all()
