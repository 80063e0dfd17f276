"""mx_gated_ffn_decode (the gated feed-forward block of few tokens) against the float64
oracle, through the C ABI.

Both products are exact with FP32 sums: within 1e-5 S.  h is then known to lie in an
interval (tests/test_gpu_swiglu.py's h_bounds), and its MX value in the range of the
codes of the interval's ends under the scales that its block's largest value allows.
y is within sum |w| times how far h's value may be from the oracle's, 1e-5 S of its own
sum, and half a step of BF16."""

import numpy as np
import pytest
import torch

from block_quant_gemm_amd import mxq, workloads
from oracle import gemm, mx
from oracle import swiglu as sw
from oracle.codec import bf16_bits_to_f64, e4m3_decode, e4m3_encode
from oracle.mx import block_shared_exponent
from tests.gpu_helpers import host, say, to_dev
from tests.test_gpu_swiglu import h_bounds

pytestmark = pytest.mark.gpu


def _weights(E, rows, cols, seed, name, sigma=0.02):
    w = workloads.bf16_normal((E * rows, cols), sigma, seed=seed, name=name)
    q, s = mx.mx_quantize_rowwise(w)
    return q.reshape(E, rows, cols), s.reshape(E, rows, cols // 32)


def _operands(M, E, K, F, N, seed):
    x = workloads.bf16_normal((M, K), 1.0, seed=seed, name="fx", outlier_frac=0.005, outlier_scale=20.0)
    return mx.mx_quantize_rowwise(x), _weights(E, 2 * F, K, seed, "fgu"), _weights(E, N, F, seed, "fdn")


def _mx_range(lo, hi):
    """Least and largest MX value of values in [lo, hi], and the middle's."""
    M, F = lo.shape
    blocks = lambda a: a.reshape(M, F // 32, 32)
    big = np.maximum(np.abs(lo), np.abs(hi))
    small = np.where((lo <= 0) & (hi >= 0), 0.0, np.minimum(np.abs(lo), np.abs(hi)))
    ends = [block_shared_exponent(blocks(a).max(2))[0] for a in (small, big)]
    vmin, vmax = np.full(lo.shape, np.inf), np.full(lo.shape, -np.inf)
    for e in ends:
        e = np.repeat(e, 32, axis=1)
        q = lambda v: np.ldexp(e4m3_decode(e4m3_encode(np.ldexp(v, -e))), e)
        vmin, vmax = np.minimum(vmin, q(lo)), np.maximum(vmax, q(hi))
    return vmin, vmax


def _check(y, x, w_gu, w_down, offs):
    E, N = w_down[0].shape[0], w_down[0].shape[1]
    A = mx.mx_dequantize(*x)
    F = w_gu[0].shape[1] // 2
    got = bf16_bits_to_f64(y)
    for e in range(E):
        rows = slice(int(offs[e]), int(offs[e + 1]))
        if rows.start == rows.stop:
            continue
        Y, S = gemm.gemm_ref(A[rows], mx.mx_dequantize(w_gu[0][e], w_gu[1][e]))
        g, u = sw.split_gate_up(Y)
        lo, hi = h_bounds(g, u, 1e-5 * S[:, :F], 1e-5 * S[:, F:])
        vmin, vmax = _mx_range(lo, hi)
        h = mx.mx_dequantize(*[a.reshape(len(g), -1) for a in mx.quantize_blocks(
            sw.swiglu(g, u).reshape(len(g), F // 32, 32))])
        W = mx.mx_dequantize(w_down[0][e], w_down[1][e])
        Y, S = gemm.gemm_ref(h, W)
        off = np.maximum(vmax - h, h - vmin) @ np.abs(W).T
        ok = np.abs(got[rows] - Y) <= (off + 1e-5 * S) * 1.01 + 2.0 ** -8 * np.abs(Y) + 2.0 ** -133
        fixed = (vmin == vmax).mean()
        assert ok.all(), (e, (~ok).sum(), fixed)
        # The bounds have to fix most codes to test anything.  S is about 0.64 sqrt(K) of
        # Y's size, 41 at K = 4128: h is known to 1e-5 * 41 * 2 = 8e-4 of its size, which is
        # less than a tenth of E4M3's step down to 2^-4 of the block's largest value (step 2^-8 of
        # it and more); smaller values are one in ten, and their steps are as small as that.
        assert fixed > 0.8 or lo.size < 2000


def _call(x, w_gu, w_down, offs=None, **kw):
    return mxq.mx_gated_ffn_decode(*map(to_dev, x), *map(to_dev, w_gu), *map(to_dev, w_down),
                                   offsets=None if offs is None else to_dev(offs), **kw)


# M, K, F, N: one token, partial token tiles, one and many blocks, odd N, both splits of F
DENSE = [(1, 32, 32, 1), (1, 2048, 352, 256), (2, 96, 64, 17), (7, 288, 2080, 40), (16, 512, 96, 64),
         (17, 640, 128, 33), (31, 2080, 32, 16), (33, 544, 160, 100), (64, 256, 2112, 48),
         (65, 256, 64, 31), (130, 128, 96, 8), (3, 4128, 64, 5),
         # a wavefront's whole share of the contraction in one iteration
         (9, 64, 1408, 20), (1, 64, 10944, 24), (8, 32, 9216, 16), (2, 64, 1408, 9), (12, 64, 1536, 16),
         # two and four token tiles a workgroup; more token tiles than workgroups along them
         (20, 64, 8256, 24), (64, 64, 10944, 16), (50, 96, 64, 4112), (1100, 32, 32, 16)]


@pytest.mark.parametrize("M,K,F,N", DENSE)
def test_dense(M, K, F, N):
    say(f"gated ffn M={M} K={K} F={F} N={N}")
    ops = _operands(M, 1, K, F, N, seed=M + K + F)
    _check(host(_call(*ops)), *ops, [0, M])


@pytest.mark.parametrize("counts,K,F,N", [
    ([1, 0, 3, 2], 256, 96, 48), ([0, 0, 9], 160, 64, 33), ([17, 1, 0, 40, 70], 288, 128, 64),
    ([2] * 40, 512, 32, 16), ([0, 300, 1, 0], 64, 64, 40), ([3, 0, 2, 1, 7, 9], 64, 1408, 24)])
def test_experts(counts, K, F, N):
    say(f"gated ffn experts {counts} K={K} F={F} N={N}")
    offs = workloads.offsets_from_counts(np.array(counts, np.int64))
    ops = _operands(int(offs[-1]), len(counts), K, F, N, seed=K + F)
    _check(host(_call(*ops, offs)), *ops, offs)


def test_a_token_alone_and_in_a_batch():
    """The rows that share a call do not change a row's result."""
    x, w_gu, w_down = _operands(70, 1, 512, 2144, 48, seed=3)
    every = _call(x, w_gu, w_down)
    for a, b in ((0, 1), (5, 12), (20, 45), (69, 70)):
        assert torch.equal(_call((x[0][a:b], x[1][a:b]), w_gu, w_down), every[a:b])


def test_strides_and_rows_outside_the_groups():
    M, E, K, F, N = 30, 3, 96, 64, 40
    x, w_gu, w_down = _operands(M, E, K, F, N, seed=4)
    offs = np.array([4, 4, 20, 27], np.int64)

    def wide(a, extra, step):
        a = to_dev(a)
        b = torch.full((*a.shape[:-1], a.shape[-1] + extra), 0x7F, dtype=torch.uint8, device="cuda")
        b[..., step:step + a.shape[-1]] = a
        return b[..., step:step + a.shape[-1]]
    y = torch.full((M, N + 7), 3.0, dtype=torch.bfloat16, device="cuda")
    mxq.mx_gated_ffn_decode(wide(x[0], 32, 16), wide(x[1], 2, 1), wide(w_gu[0], 48, 32), wide(w_gu[1], 3, 1),
                            wide(w_down[0], 16, 16), wide(w_down[1], 5, 2), offsets=to_dev(offs), y=y[:, 3:3 + N])
    assert (y[:, :3] == 3).all() and (y[:, 3 + N:] == 3).all()
    assert (y[:4] == 3).all() and (y[27:] == 3).all()
    inner = [a[4:27] for a in x]
    _check(host(y[4:27, 3:3 + N].contiguous()), inner, w_gu, w_down, offs - 4)


def test_values_that_are_not_finite():
    """A NaN block of a token makes its own row NaN; one of a weight row its h column, then
    every token's h block and so the rows of its group; others keep their bits."""
    x, w_gu, w_down = _operands(9, 2, 256, 96, 40, seed=5)
    offs = np.array([0, 5, 9], np.int64)
    clean = _call(x, w_gu, w_down, offs)
    x[1][2, 3] = 0xFF
    y = _call(x, w_gu, w_down, offs)
    assert y[2].isnan().all() and torch.equal(y[[0, 1, *range(3, 9)]], clean[[0, 1, *range(3, 9)]])
    w_down[1][1, 7, 1] = 0xFF
    y = _call(x, w_gu, w_down, offs)
    assert y[5:, 7].isnan().all() and not y[:, :7][[0, 1, 3, 4, 5, 6, 7, 8]].isnan().any()
    w_gu[1][1, 10, 2] = 0xFF
    y = _call(x, w_gu, w_down, offs)
    assert y[5:].isnan().all() and torch.equal(y[[0, 1, 3, 4]], clean[[0, 1, 3, 4]])


def test_empty_dimensions():
    z = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")
    y = mxq.mx_gated_ffn_decode(z(0, 64), z(0, 2), z(1, 64, 64), z(1, 64, 2), z(1, 8, 32), z(1, 8, 1))
    assert y.shape == (0, 8)
    y = mxq.mx_gated_ffn_decode(z(3, 0), z(3, 0), z(1, 64, 0), z(1, 64, 0), z(1, 8, 32), z(1, 8, 1))
    assert (y == 0).all() and y.shape == (3, 8)
    y = mxq.mx_gated_ffn_decode(z(3, 64), z(3, 2), z(1, 0, 64), z(1, 0, 2), z(1, 8, 0), z(1, 8, 0))
    assert (y == 0).all() and y.shape == (3, 8)


def test_offsets_that_break_the_rules_stay_inside():
    """Decreasing, negative and too large offsets: unspecified rows, nothing outside y."""
    x, w_gu, w_down = _operands(20, 3, 64, 32, 16, seed=6)
    base = torch.full((24, 16), 3.0, dtype=torch.bfloat16, device="cuda")
    for offs in ([0, 50, 10, 20], [-9, 5, 2, 1 << 40], [30, 31, 32, 33]):
        mxq.mx_gated_ffn_decode(*map(to_dev, x), *map(to_dev, w_gu), *map(to_dev, w_down),
                                offsets=to_dev(np.array(offs, np.int64)), y=base[2:22])
        assert (base[:2] == 3).all() and (base[22:] == 3).all()
