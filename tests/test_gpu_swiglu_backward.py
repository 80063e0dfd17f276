"""mx_grouped_gemm_swiglu_backward (the down product's data gradient with SwiGLU's
gradient and the MX copies in its epilogue) against the float64 oracle, through the C ABI.

dh comes from the matrix unit: within 1e-5 S of the exact product (S the sum of
the products' magnitudes), plus the FP8 unit's truncation allowance in that mode
(tests/fp8_mode.py).  Of the epilogue, with u24 = 2^-24 and the hardware's 2^x and 1/x
good to a unit in the last place (2 u24):
  e^-g     argument -g log2 e rounded twice, 2 |g| log2(e) u24 absolute, so 2.9 |g| u24
           of the value, and 2 u24 of 2^x: (3 |g| + 2) u24
  sg       that times 1 - sg <= 1, 1 + e rounded, 1/x: dl = (3 |g| + 5) u24 of sg
  1 - sg   sg dl + u24 absolute
  s = dh sg, d up = s g    two products: |dh g| sg dl + 3 u24 |d up|
  d gate = u (d up (1 - sg) + s) = u s P, P = 1 + g (1 - sg)    the FMA's product is off by
    |s| |g| (sg dl + u24 + u24 (1 - sg)) and it rounds once: with eP = |g| (sg dl + 2 u24) +
    u24 |P|, |dh u| (sg eP + |P| sg dl) + 4 u24 |d gate|
and both with dh's own error times |u sg P| and |g sg|; underflow to 2^-126 (1 + |g|)|u dh|
where a factor is subnormal, and for g < -87, where e^-g is infinite in FP32, sg is 0:
the whole term, |dh u g| e^g.  Codes are checked against these intervals
(tests/mx_interval.py)."""

import numpy as np
import pytest
import torch

from block_quant_gemm_amd import mxq, workloads
from oracle import gemm, mx, norm
from oracle.codec import bf16_bits_to_f64
from tests import fp8_mode as f8
from tests.gpu_helpers import host, say, to_dev, to_dev_bf16
from tests.mx_interval import mx_valid
from tests.test_gpu_gemm import _relayout_scales

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
SENTINEL = 0xAB


def grad_bounds(dh, ddh, g, u):
    """(dgu, its allowance) [M, 2F] from the exact dh and its allowance."""
    dg, du = norm.swiglu_backward(dh, g, u)
    with np.errstate(over="ignore"):
        sg = 1.0 / (1.0 + np.exp(-g))
    ag, au, ah = np.abs(g), np.abs(u), np.abs(dh) + ddh
    dl = (3 * ag + 5) * U
    P = 1 + g * (1 - sg)
    eP = ag * (sg * dl + 2 * U) + U * np.abs(P)
    tiny = 2.0 ** -126 * (1 + ag) * (1 + au * ah)
    lost = np.where(g < -87, ag * np.exp(np.minimum(g, 0.0)) * 1.01, 0.0)
    eg = ddh * np.abs(u * sg * P) + ah * au * (sg * eP + np.abs(P) * sg * dl + lost) + 4 * U * np.abs(dg) + tiny
    eu = ddh * np.abs(g * sg) + ah * ag * sg * dl + ah * lost + 3 * U * np.abs(du) + tiny
    return np.concatenate([dg, du], 1), 1.01 * np.concatenate([eg, eu], 1)


def _operands(counts, F, K, seed, g_sigma=1.5):
    counts = np.array(counts, np.int64)
    offs = workloads.offsets_from_counts(counts)
    E, M = len(counts), int(counts.sum())
    dy = workloads.bf16_normal((M, K), 1.0, seed=seed, name="bdy")
    w = workloads.bf16_normal((F, E * K), 0.02, seed=seed, name="bw")   # down weights' column copies
    gu = workloads.bf16_normal((M, 2 * F), g_sigma, seed=seed, name="bgu")
    return offs, *mx.mx_quantize_rowwise(dy), *mx.mx_quantize_rowwise(w), gu


def _layout(s, layout):
    if layout == "pad16":
        buf = mxq._scale_buffer(s.shape[0], s.shape[1], "cuda")
        buf.copy_(to_dev(s))
        return buf
    return _relayout_scales(to_dev(s), layout)


def _run(offs, dq, ds, wq, ws, gu, layout="pad16", dgu=True, accum=mxq.ACC_MFMA_FP8, rows=None, cap=None):
    E, M, K = len(offs) - 1, dq.shape[0], dq.shape[1]
    F = wq.shape[0]
    w, wsc = to_dev(wq).view(F, E, K).transpose(0, 1), _layout(ws, layout)
    wsc = wsc.as_strided((E, F, K // 32), (K // 32, wsc.stride(0), 1), wsc.storage_offset())
    cap = mxq.colwise_capacity(M, E) if cap is None else cap
    full = lambda *s: torch.full(s, SENTINEL, dtype=torch.uint8, device="cuda")
    sT = mxq._scale_buffer(2 * F, cap // 32, "cuda")
    sT.fill_(SENTINEL)
    out = mxq.mx_grouped_gemm_swiglu_backward(
        to_dev(dq), _layout(ds, layout), w, wsc, to_dev_bf16(gu), to_dev(offs), dgu=dgu, accum=accum,
        M_cap=cap, q=full(M, 2 * F), scale=full(M, F // 16), qT=full(2 * F, cap), scaleT=sT)
    return [None if t is None else host(t) for t in out]


def _reference(offs, dq, ds, wq, ws, accum):
    """Exact dh and its allowance."""
    E, M, K = len(offs) - 1, dq.shape[0], dq.shape[1]
    F = wq.shape[0]
    A = mx.mx_dequantize(dq, ds)
    B = mx.mx_dequantize(wq, ws).reshape(F, E, K).transpose(1, 0, 2)
    Y, S = gemm.grouped_gemm_ref(A, B, offs)
    if accum == mxq.ACC_FP32:
        return Y, 1e-5 * S
    e = np.searchsorted(offs, np.arange(M), side="right") - 1
    T = np.zeros((M, F))
    for x in range(E):
        at = np.flatnonzero(e == x)
        rows, cols = np.repeat(at, F), np.tile(np.arange(F), len(at))
        T[at] = f8.fp8_mfma_truncation_bound(dq, ds, np.ascontiguousarray(wq.reshape(F, E, K)[:, x]),
                                             np.ascontiguousarray(ws.reshape(F, E, K // 32)[:, x]),
                                             rows, cols).reshape(len(at), F)
    return Y, 1e-5 * S + T


def _check(offs, dh, ddh, gu, out):
    dgu, q, sc, qT, sT, poff = out
    F = dh.shape[1]
    v = bf16_bits_to_f64(gu)
    ref, d = grad_bounds(dh, ddh, v[:, :F], v[:, F:])
    if dgu is not None:
        got = bf16_bits_to_f64(dgu)
        assert (np.abs(got - ref) <= d + 2.0 ** -8 * (np.abs(ref) + d) + 2.0 ** -133).all()
    ok_c, ok_s, uniq = mx_valid(q, sc, ref - d, ref + d)
    say(f"  codes fixed by the bounds {uniq.mean():.5f}; bad codes {(~ok_c).sum()}, scales {(~ok_s).sum()}")
    assert ok_c.all() and ok_s.all()
    np.testing.assert_array_equal(poff, mx.padded_offsets(offs))
    lo, hi = np.zeros((2 * F, qT.shape[1])), np.zeros((2 * F, qT.shape[1]))
    for e in range(len(offs) - 1):
        a, b, p = int(offs[e]), int(offs[e + 1]), int(poff[e])
        lo[:, p:p + b - a], hi[:, p:p + b - a] = (ref - d)[a:b].T, (ref + d)[a:b].T
    ok_c, ok_s, _ = mx_valid(qT, sT, lo, hi)                 # padding and what is past it: zeros
    assert ok_c.all() and ok_s.all()
    return uniq


CASES = [
    ([300, 0, 1, 257, 31, 600], 320, 256),      # partial column tile, 1-row and 257-row groups
    ([5], 32, 64),
    ([1], 288, 32),
    ([128, 128, 0, 1, 127, 129], 128, 1408),
    ([40, 0, 2, 700], 96, 96),                  # odd k-step count
    ([0, 0, 513], 1408, 128),                   # the expert FFN width
]


@pytest.mark.parametrize("counts,F,K", CASES)
@pytest.mark.parametrize("layout", ["pad16", "odd", "shift5"])
@pytest.mark.parametrize("accum", [mxq.ACC_MFMA_FP8, mxq.ACC_FP32])
def test_gradient(counts, F, K, layout, accum):
    say(f"SwiGLU gradient counts={counts} F={F} K={K} scales={layout} accum={accum}")
    ops = _operands(counts, F, K, seed=len(counts) * 31 + F + K)
    out = _run(*ops, layout=layout, accum=accum)
    uniq = _check(ops[0], *_reference(*ops[:5], accum), ops[5], out)
    if accum == mxq.ACC_FP32 and uniq.size > 2000:
        # 1e-5 S is 1e-5 * 0.64 sqrt(K) of dh, at most 2.4e-4: a fiftieth of E4M3's step at
        # the block's largest value; only values below 2^-5 of it, one in ten, have steps as small
        assert uniq.mean() > 0.8


def test_gradient_without_its_bf16_copy():
    ops = _operands([77, 0, 300], 160, 192, seed=3)
    a, b = _run(*ops), _run(*ops, dgu=False)
    assert b[0] is None
    for u, v in zip(a[1:], b[1:]):
        np.testing.assert_array_equal(u, v)


def test_gradient_at_large_gate_values():
    """|g| past 100: e^-g overflows in FP32, sg is 0 or 1."""
    ops = _operands([200, 61], 96, 256, seed=4, g_sigma=60.0)
    v = bf16_bits_to_f64(ops[5])[:, :96]
    assert v.min() < -88 and v.max() > 88
    _check(ops[0], *_reference(*ops[:5], mxq.ACC_FP32), ops[5], _run(*ops, accum=mxq.ACC_FP32))


def test_gradient_against_differences():
    """The sum of dy-weighted outputs moves by dgu along random directions of the gate/up
    product, as the oracle's float64 SwiGLU and down product do."""
    F, K, h = 64, 64, 1e-5
    ops = _operands([9, 30], F, K, seed=5)
    offs, dq, ds, wq, ws, gu = ops
    dgu = bf16_bits_to_f64(_run(*ops, accum=mxq.ACC_FP32)[0])
    A = mx.mx_dequantize(dq, ds)
    B = mx.mx_dequantize(wq, ws).reshape(F, 2, K)
    v = bf16_bits_to_f64(gu)

    def loss(v):
        g, u = v[:, :F], v[:, F:]
        act = g / (1 + np.exp(-g)) * u
        return sum((act[a:b] @ B[:, e] * A[a:b]).sum() for e, (a, b) in enumerate(zip(offs, offs[1:])))
    rng = np.random.default_rng(0)
    for _ in range(4):
        d = rng.normal(size=v.shape)
        num = (loss(v + h * d) - loss(v - h * d)) / (2 * h)
        # half a BF16 step on every value and dh's 1e-5, and the quotient's own error
        assert abs((dgu * d).sum() - num) <= (2.0 ** -8 + 1e-4) * np.abs(dgu * d).sum() + 1e-6


@pytest.mark.parametrize("rows,split", [(256 * 14 + 40, 2), (256 * 30, 1), (256 * 45 + 7, 4)])
def test_tiles_in_parts(rows, split):
    """Whole tiles, and the last ones in halves or quarters: how a call's tiles are dealt does
    not change a row's or a block's result.  Columns 1408: 6 tiles across, so 90, 180 and 276
    tiles; against calls of one group's 640 rows, whose 18 tiles go in quarters."""
    say(f"SwiGLU gradient {rows} rows, the last tiles in {split}")
    F, K, step = 1408, 64, 640
    gen = torch.Generator(device="cuda").manual_seed(rows)
    draw = lambda *s, sigma=1.0: (torch.randn(*s, generator=gen, device="cuda") * sigma).to(torch.bfloat16)
    dq, ds = mxq.mx_quantize_rowwise(draw(rows, K))
    wq, ws = mxq.mx_quantize_rowwise(draw(F, K, sigma=0.02))
    w = wq.view(1, F, K), ws.view(1, F, K // 32)
    gu = draw(rows, 2 * F)
    off = lambda n: torch.tensor([0, n], device="cuda")
    for accum in (mxq.ACC_MFMA_FP8, mxq.ACC_FP32):
        every = mxq.mx_grouped_gemm_swiglu_backward(dq, ds, *w, gu, off(rows), dgu=True, accum=accum)
        for a in range(0, rows, step):
            n = min(step, rows - a)
            part = mxq.mx_grouped_gemm_swiglu_backward(dq[a:a + n], ds[a:a + n], *w, gu[a:a + n], off(n),
                                                       dgu=True, accum=accum)
            for u, v in zip(every[:3], part[:3]):
                assert torch.equal(u[a:a + n], v)
            p = -(-n // 32) * 32
            assert torch.equal(every[3][:, a:a + p], part[3][:, :p])
            assert torch.equal(every[4][:, a // 32:(a + p) // 32], part[4][:, :p // 32])
        assert (every[3][:, -(-rows // 32) * 32:] == 0).all()


def test_rows_outside_the_groups_are_left():
    """Offsets that start after row 0 and end before row M."""
    ops = _operands([40, 90, 50], 96, 64, seed=6)
    offs = np.array([40, 40, 130], np.int64)
    dq, ds, wq, ws, gu = ops[1:]
    wq, ws = wq[:, :2 * 64].copy(), ws[:, :2 * 2].copy()
    M, F = 180, 96
    out = mxq.mx_grouped_gemm_swiglu_backward(
        to_dev(dq), to_dev(ds), to_dev(wq).view(F, 2, 64).transpose(0, 1), to_dev(ws).view(F, 2, 2).transpose(0, 1),
        to_dev_bf16(gu), to_dev(offs), accum=mxq.ACC_FP32,
        dgu=torch.full((M, 2 * F), 7.0, dtype=torch.bfloat16, device="cuda"),
        q=torch.full((M, 2 * F), SENTINEL, dtype=torch.uint8, device="cuda"),
        scale=torch.full((M, F // 16), SENTINEL, dtype=torch.uint8, device="cuda"))
    dgu, q, sc = [host(t) for t in out[:3]]
    for a, b in ((0, 40), (130, 180)):
        assert (q[a:b] == SENTINEL).all() and (sc[a:b] == SENTINEL).all()
        assert (bf16_bits_to_f64(dgu[a:b]) == 7).all()
    inner = _run(np.array([0, 0, 90]), dq[40:130], ds[40:130], wq, ws, gu[40:130], accum=mxq.ACC_FP32,
                 cap=host(out[3]).shape[1])
    np.testing.assert_array_equal(q[40:130], inner[1])
    np.testing.assert_array_equal(sc[40:130], inner[2])
    np.testing.assert_array_equal(host(out[3]), inner[3])


def test_values_that_are_not_finite():
    """NaN in dY's row, in the gate and in the up value reach their own blocks only."""
    F, K = 96, 64
    offs, dq, ds, wq, ws, gu = _operands([70], F, K, seed=7)
    clean = _run(offs, dq, ds, wq, ws, gu)
    ds[5, 1], gu[20, 40], gu[33, F + 70], gu[50, 3] = 0xFF, 0x7FC0, 0x7F80, 0xFF80
    _, q, sc, qT, sT, _ = _run(offs, dq, ds, wq, ws, gu)
    bad = np.zeros((70, 2 * F), bool)
    bad[5] = True
    bad[20, [40, F + 40]] = bad[50, [3, F + 3]] = True
    bad[33, 70] = True                                       # u = inf: d gate; d up does not have it
    rows = bad.reshape(70, -1, 32).any(2)
    np.testing.assert_array_equal(sc == 0xFF, rows)
    assert (q.reshape(70, -1, 32)[rows] == 0x7F).all()
    np.testing.assert_array_equal(np.where(rows[..., None], 0, q.reshape(70, -1, 32)),
                                  np.where(rows[..., None], 0, clean[1].reshape(70, -1, 32)))
    pad = np.zeros((2 * F, sT.shape[1] * 32), bool)
    pad[:, :70] = bad.T
    cols = pad.reshape(2 * F, -1, 32).any(2)
    np.testing.assert_array_equal(sT == 0xFF, cols)
    assert (qT.reshape(2 * F, -1, 32)[cols] == 0x7F).all()
    np.testing.assert_array_equal(np.where(cols[..., None], 0, qT.reshape(2 * F, -1, 32)),
                                  np.where(cols[..., None], 0, clean[3].reshape(2 * F, -1, 32)))


def test_no_rows():
    F, K = 64, 64
    z = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")
    qT = torch.full((2 * F, 128), SENTINEL, dtype=torch.uint8, device="cuda")
    sT = torch.full((2 * F, 4), SENTINEL, dtype=torch.uint8, device="cuda")
    out = mxq.mx_grouped_gemm_swiglu_backward(
        z(0, K), z(0, K // 32), z(3, F, K), z(3, F, K // 32), torch.empty((0, 2 * F), dtype=torch.bfloat16, device="cuda"),
        to_dev(np.zeros(4, np.int64)), qT=qT, scaleT=sT)
    assert (host(out[5]) == 0).all() and (qT == 0).all() and (sT == 0).all()


def test_equals_the_unfused_chain():
    """The epilogue's codes against quantizing the BF16 gradient: the same but where BF16's
    rounding moves a value across a code's border; at most a step of E4M3 there."""
    offs, dq, ds, wq, ws, gu = _operands([500, 12], 256, 512, seed=8)
    dgu, q, sc, _, _, _ = _run(offs, dq, ds, wq, ws, gu)
    q2, sc2 = mx.mx_quantize_rowwise(dgu)
    a, b = mx.mx_dequantize(q, sc), mx.mx_dequantize(q2, sc2)
    top = np.repeat(np.abs(b).reshape(512, -1, 32).max(2), 32, axis=1)
    assert (np.abs(a - b) <= 2.0 ** -3 * np.abs(b) + 2.0 ** -3 * top).all()
    assert (a == b).mean() > 0.9


@pytest.mark.parametrize("accum", [mxq.ACC_MFMA_FP8, mxq.ACC_FP32])
def test_values_past_the_range_of_bfloat16(accum):
    """A gradient that FP32 holds and BF16 does not is infinite in dgu; its codes come from
    the FP32 value.  dh = 1.75 + 0.25 - 2^-9 and g = u = 2^127, so sg = 1 and both
    gradients are (2 - 2^-9) 2^127, which rounds to 2^128; every sum is exact."""
    M, F, K = 70, 64, 32
    dq, ds = np.zeros((M, K), np.uint8), np.full((M, 1), 127, np.uint8)
    wq, ws = np.zeros((F, K), np.uint8), np.full((F, 1), 127, np.uint8)
    dq[:, :3] = 0x38                                        # 1
    wq[:, 0], wq[:, 1], wq[:, 2] = 0x3E, 0x28, 0x81         # 1.75, 0.25, -2^-9
    gu = np.full((M, 2 * F), 0x3F80, np.uint16)
    gu[[0, 33, 69]] = 0x7F00                                # 2^127
    dgu, q, sc, qT, sT, _ = _run(np.array([0, M]), dq, ds, wq, ws, gu, accum=accum)
    v = bf16_bits_to_f64(dgu)
    assert np.isposinf(v[[0, 33, 69]]).all() and np.isfinite(np.delete(v, [0, 33, 69], 0)).all()
    # 1.998 2^127 = 448 * 2^119 * 1.14, saturated
    assert (sc[[0, 33, 69]] == 127 + 119).all() and (q[[0, 33, 69]] == 0x7E).all()
    assert (sT[:, :3] == 127 + 119).all() and (qT[:, [0, 33, 69]] == 0x7E).all()
