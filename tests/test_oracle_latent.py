"""The latent-attention oracle against what pins it: hand-made softmaxes, the
absorbed form against the expanded one (they are the same function when the
heads' projections are multiplied into queries and outputs), gradients
against central differences, and hidden values that must not matter.  CPU only."""

import numpy as np
import pytest

from oracle import codec, latent, mx


def _case(seed, Tq=7, Tk=9, H=2):
    r = np.random.default_rng(seed)
    return (r.standard_normal((Tq, H, 192)), r.standard_normal((Tk, H, 128)),
            r.standard_normal((Tk, 64)), r.standard_normal((Tk, H, 128)))


def test_one_key_gives_its_value():
    q, kn, kr, v = _case(0, 3, 1, 1)
    o, lse = latent.attention(q, kn, kr, v, None, None, 0.1, False)
    assert np.allclose(o, v[[0, 0, 0]])
    z = 0.1 * (q[:, 0, :128] @ kn[0, 0] + q[:, 0, 128:] @ kr[0])
    assert np.allclose(lse[0], z)


def test_equal_logits_average():
    q, kn, kr, v = _case(1)
    o, lse = latent.attention(q * 0, kn, kr, v, None, None, 1.0, False)
    assert np.allclose(o, v.mean(0)[None]) and np.allclose(lse, np.log(9))


@pytest.mark.parametrize("lq,lk,want", [(3, 3, [1, 2, 3]), (2, 5, [4, 5]), (4, 2, [0, 0, 1, 2]),
                                        (3, 0, [0, 0, 0])])
def test_causal_visibility(lq, lk, want):
    assert [latent.visible(i, lq, lk, True) for i in range(lq)] == want
    assert all(latent.visible(i, lq, lk, False) == lk for i in range(lq))


def test_rows_without_keys_are_zero():
    q, kn, kr, v = _case(2, 5, 2)
    o, lse = latent.attention(q, kn, kr, v, None, None, 0.1, True)
    assert (o[:3] == 0).all() and np.isneginf(lse[:, :3]).all() and np.isfinite(lse[:, 3:]).all()


def test_hidden_values_do_not_matter():
    q, kn, kr, v = _case(3, 6, 6)
    want = latent.attention(q, kn, kr, v, None, None, 0.1, True)
    kn[4:], kr[4:], v[4:], q[4:] = np.nan, np.inf, np.nan, np.nan
    got = latent.attention(q, kn, kr, v, None, None, 0.1, True)
    assert np.array_equal(got[0][:4], want[0][:4]) and np.array_equal(got[1][:, :4], want[1][:, :4])


def test_sequences_are_independent():
    q, kn, kr, v = _case(4, 9, 9)
    off = np.array([0, 4, 4, 9])
    o, lse = latent.attention(q, kn, kr, v, off, off, 0.1, True)
    for a, b in ((0, 4), (4, 9)):
        o1, l1 = latent.attention(q[a:b], kn[a:b], kr[a:b], v[a:b], None, None, 0.1, True)
        assert np.array_equal(o[a:b], o1) and np.array_equal(lse[:, a:b], l1)


def test_absorbed_form_equals_expanded_form():
    """k_nope = c Wk and v = c Wv: multiplying Wk into the queries and Wv into the
    result turns one form into the other."""
    r = np.random.default_rng(5)
    L, H = 11, 3
    c, kr = r.standard_normal((L, 512)), r.standard_normal((L, 64))
    wk, wv = r.standard_normal((H, 512, 128)) * 0.05, r.standard_normal((H, 512, 128)) * 0.05
    q = r.standard_normal((1, H, 192))
    kn = np.einsum("lc,hcd->lhd", c, wk)
    v = np.einsum("lc,hcd->lhd", c, wv)
    o, lse = latent.attention(q, kn, kr, v, None, None, 0.07, True)
    qa = np.concatenate([np.einsum("ihd,hcd->ihc", q[..., :128], wk), q[..., 128:]], -1)
    oa, la, _, _ = latent.decode(qa[None], c, kr, [np.arange(L)], [L], 0.07)
    assert np.allclose(la[0, 0], lse[:, 0])
    assert np.allclose(np.einsum("hc,hcd->hd", oa[0, 0], wv), o[0])


def test_decode_sees_the_tokens_before_each_query():
    r = np.random.default_rng(6)
    c, kr, q = r.standard_normal((9, 512)), r.standard_normal((9, 64)), r.standard_normal((1, 3, 2, 576))
    o, lse, _, _ = latent.decode(q, c, kr, [np.arange(9)], [2], 0.05)
    assert (o[0, 0] == 0).all() and np.isneginf(lse[0, 0]).all()
    assert np.allclose(o[0, 1], c[0]) and np.isfinite(lse[0, 2]).all()


@pytest.mark.parametrize("causal", [False, True])
def test_gradient_against_differences(causal):
    x = _case(7, 5, 6)
    g = np.random.default_rng(8).standard_normal((5, 2, 128))
    off_q, off_k = np.array([0, 2, 5]), np.array([0, 3, 6])
    ref = latent.attention_backward(g, *x, off_q, off_k, 0.07, causal)

    def f(y):
        return (latent.attention(*y, off_q, off_k, 0.07, causal)[0] * g).sum()

    r = np.random.default_rng(9)
    for i, name in enumerate(("dq", "dk_nope", "dk_rope", "dv")):
        for _ in range(4):
            u = r.standard_normal(x[i].shape)
            hi = [a + 1e-5 * u if j == i else a for j, a in enumerate(x)]
            lo = [a - 1e-5 * u if j == i else a for j, a in enumerate(x)]
            slope = (f(hi) - f(lo)) / 2e-5
            # differences of a smooth function: second-order error, and rounding / step
            assert abs((ref[name][0] * u).sum() - slope) < 1e-6 * (1 + abs(slope))


def test_bounds_cover_a_bf16_model():
    """Rounding P, dS and the results to BF16 stays inside the bounds that the GPU
    tests use (which also allow for FP32 sums)."""
    r = np.random.default_rng(10)
    bf = lambda *s: codec.bf16_round(r.standard_normal(s))
    q, kn, kr, v, g = bf(8, 1, 192), bf(8, 1, 128), bf(8, 64), bf(8, 1, 128), bf(8, 1, 128)
    ref = latent.attention_backward(g, q, kn, kr, v, None, None, 0.07, True)
    k = np.concatenate([kn[:, 0], kr], 1)
    z = np.where(np.tril(np.ones((8, 8))) > 0, q[:, 0] @ k.T * 0.07, -np.inf)
    p = np.exp(z - z.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    pr = codec.bf16_round(p)
    o = codec.bf16_round(pr @ v[:, 0])
    ds = codec.bf16_round(p * (g[:, 0] @ v[:, 0].T - (g[:, 0] * o).sum(1, keepdims=True)))
    got = {"o": o, "dq": codec.bf16_round(0.07 * ds @ k), "dv": codec.bf16_round(pr.T @ g[:, 0])}
    dk = codec.bf16_round(0.07 * ds.T @ q[:, 0])
    got["dk_nope"], got["dk_rope"] = dk[:, :128], dk[:, 128:]
    for n, x in got.items():
        val, err = ref[n]
        assert (np.abs(x.reshape(val.shape) - val) <= err).all(), n


def test_cache_round_trip():
    r = np.random.default_rng(11)
    x = codec.bf16_round_to_bits(r.standard_normal((5, 576)))
    empty = (np.zeros((8, 512), np.uint8), np.zeros((8, 16), np.uint8), np.zeros((8, 64), np.uint16))
    cache = latent.cache_write(empty, x[:, :512], x[:, 512:], [7, -1, 3, 8, 0])
    c, kr = latent.cache_read(cache, [7, 3, 0, 1, -1, 8])
    q, s = mx.mx_quantize_rowwise(x[:, :512])
    want = codec.bf16_round_to_bits(mx.mx_dequantize(q, s))
    assert np.array_equal(c[:3], want[[0, 2, 4]]) and np.array_equal(kr[:3], x[[0, 2, 4], 512:])
    assert (c[3:] == 0).all() and (kr[3:] == 0).all()
