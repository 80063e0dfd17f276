"""mx_rms_norm and its gradient against the float64 oracle, through the C ABI.

Allowances, with u = 2^-24 (half a step of FP32) and BF16's half step 2^-8:
  total   none: one FP32 addition and one rounding, as the oracle's.
  rstd    the FP64 value rounded once: u (1 + 2^-20), the excess for FP64's own roundings.
  y       rstd's rounding and two products: 3 u, (1 + u)^3 - 1 < 3.01 u; BF16's
          half step on top; the codes' intervals (tests/mx_interval.py) are 3.01 u wide
          each way.
  dx      with g = dy w (one rounding), xh = s rstd (one): c is a sum of K products
          of depth d = 8 chunks a lane + 6 + wavefronts, its error at most
          (d + 3) u mean|g xh| =: ec, its own division u more; xh c: |xh| (ec + 3 u |c|);
          g - xh c and rstd ( ) + ds are one FMA each: 2 u of their results; the
          rounding to BF16 half a step of the result.
  dw      sums of M products, each with two roundings (xh, the FMA), over a depth of at
          most rows a lane + 4 + parts / 16 + 16: depth u sum|dy xh|.
The gradient is also compared with differences of the float64 oracle."""

import numpy as np
import pytest
import torch

from block_quant_gemm_amd import mxq, workloads
from oracle import mx, norm
from oracle.codec import bf16_bits_to_f64, bf16_round
from tests.gpu_helpers import host, say, to_dev, to_dev_bf16
from tests.mx_interval import mx_valid

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 1e-6
SENTINEL = 0xAB


def _bits(shape, seed, name, sigma=1.0):
    return workloads.bf16_normal(shape, sigma, seed=seed, name=name, outlier_frac=0.005,
                                 outlier_scale=20.0)


def _weight(K, seed):
    return _bits((1, K), seed, "nw", 0.3)[0]


def _wide(t, extra, rows=3):
    """t's values as a column range of a wider matrix."""
    w = torch.full((t.shape[0] + rows, t.shape[1] + extra), float("nan"), dtype=t.dtype, device=t.device)
    w[:t.shape[0], 8:8 + t.shape[1]] = t
    return w[:t.shape[0], 8:8 + t.shape[1]]


def _check_bf16(got, ref, slack):
    got = bf16_bits_to_f64(got)
    assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 1.01 * slack + 2.0 ** -133).all()


def _check_norm(s, w, out, cap=None):
    total, rstd, y, q, scale, qT, scaleT = [None if t is None else host(t) for t in out]
    M, K = s.shape
    r_rstd, r_y = norm.rms_norm(s, w, EPS)
    if total is not None:
        np.testing.assert_array_equal(bf16_bits_to_f64(total), s)
    assert (np.abs(rstd.astype(np.float64) - r_rstd) <= U * (1 + 2.0 ** -20) * r_rstd).all()
    d = 3.01 * U * np.abs(r_y) + 2.0 ** -148
    if y is not None:
        _check_bf16(y, r_y, d)
    ok_c, ok_s, uniq = mx_valid(q, scale, r_y - d, r_y + d)
    assert ok_c.all() and ok_s.all()
    assert uniq.mean() > 0.999 or uniq.size < 4096
    if qT is not None:
        lo, hi = np.zeros((K, qT.shape[1])), np.zeros((K, qT.shape[1]))
        lo[:, :M], hi[:, :M] = (r_y - d).T, (r_y + d).T
        ok_c, ok_s, _ = mx_valid(qT, scaleT, lo, hi)        # zeros past M: codes and scales 0
        assert ok_c.all() and ok_s.all()


ROWS = [(1, 32), (3, 64), (33, 96), (5, 512), (129, 544), (40, 2048), (1030, 2048), (1025, 1056),
        (37, 2080), (7, 4096), (9, 4128), (4, 8192), (3, 8224), (2, 16384), (2, 12000),
        (300, 1024), (4100, 2048)]


@pytest.mark.parametrize("M,K", ROWS)
@pytest.mark.parametrize("residual", [False, True])
def test_norm(M, K, residual):
    say(f"rms norm M={M} K={K} residual={residual}")
    x, r, w = _bits((M, K), M + K, "nx"), _bits((M, K), M + K, "nr"), _weight(K, K)
    out = mxq.mx_rms_norm(to_dev_bf16(x), to_dev_bf16(w), eps=EPS, y=True, columns=True,
                          residual=to_dev_bf16(r) if residual else None)
    s = norm.residual_sum(x, r) if residual else bf16_bits_to_f64(x)
    _check_norm(s, bf16_bits_to_f64(w), out)


@pytest.mark.parametrize("M,K", [(1, 512), (70, 512), (259, 2048), (1500, 2048)])
def test_norm_of_column_ranges_into_column_ranges(M, K):
    """Strided operands and outputs; what lies beside them stays as it was."""
    say(f"rms norm strided M={M} K={K}")
    x, r, w = _bits((M, K), 5, "nx"), _bits((M, K), 5, "nr"), _weight(K, 5)
    dx, dr = _wide(to_dev_bf16(x), 64), _wide(to_dev_bf16(r), 24)
    cap = (M + 31) // 32 * 32
    wide = lambda rows, cols, dt: torch.full((rows, cols + 32), 5 if dt == torch.uint8 else 5.0, dtype=dt,
                                             device="cuda")
    bt, by, bq, bs = (wide(M, n, dt) for n, dt in ((K, torch.bfloat16), (K, torch.bfloat16),
                                                   (K, torch.uint8), (K // 32, torch.uint8)))
    bqT, bsT = wide(K, cap, torch.uint8), wide(K, cap // 32, torch.uint8)
    out = mxq.mx_rms_norm(dx, to_dev_bf16(w), residual=dr, eps=EPS, total=bt[:, 8:8 + K],
                          y=by[:, 16:16 + K], q=bq[:, 16:16 + K], scale=bs[:, 3:3 + K // 32],
                          qT=bqT[:, 16:16 + cap], scaleT=bsT[:, 1:1 + cap // 32])
    _check_norm(norm.residual_sum(x, r), bf16_bits_to_f64(w), out)
    for b, at, n in ((bt, 8, K), (by, 16, K), (bq, 16, K), (bs, 3, K // 32), (bqT, 16, cap), (bsT, 1, cap // 32)):
        assert (b[:, :at] == 5).all() and (b[:, at + n:] == 5).all()


@pytest.mark.parametrize("which", ["x", "residual"])
def test_norm_in_place(which):
    M, K = 300, 2048
    x, r, w = _bits((M, K), 6, "nx"), _bits((M, K), 6, "nr"), _weight(K, 6)
    dx, dr = to_dev_bf16(x), to_dev_bf16(r)
    out = mxq.mx_rms_norm(dx, to_dev_bf16(w), residual=dr, eps=EPS, columns=True,
                          total=dx if which == "x" else dr)
    _check_norm(norm.residual_sum(x, r), bf16_bits_to_f64(w), out)


def test_forms_agree():
    """Few and many rows take different workgroups and give the same values."""
    M, K = 1200, 2048
    x, w = to_dev_bf16(_bits((M, K), 7, "nx")), to_dev_bf16(_weight(K, 7))
    a = mxq.mx_rms_norm(x, w, y=True, columns=True)
    for i in range(0, M, 400):
        b = mxq.mx_rms_norm(x[i:i + 400], w, y=True)
        for u, v in zip(a[1:5], b[1:5]):
            assert torch.equal(u[i:i + 400], v)


def test_rows_that_hold_nothing_finite():
    """A row of zeros gives zeros; NaN makes its row NaN; an infinity makes rstd 0, so that
    the row's other values are zeros and its own block NaN.  Other rows are untouched."""
    M, K = 70, 96
    x = _bits((M, K), 8, "nx")
    x[3] = 0
    x[10, 40] = 0x7FC1                                       # NaN
    x[20, 70] = 0xFF80                                       # -inf
    w = np.full(K, 0x3F80, np.uint16)
    total, rstd, y, q, sc, qT, sT = [None if t is None else host(t) for t in mxq.mx_rms_norm(
        to_dev_bf16(x), to_dev_bf16(w), eps=EPS, y=True, columns=True)]
    assert (q[3] == 0).all() and (sc[3] == 0).all() and rstd[3] == np.float32(1 / np.sqrt(np.float64(np.float32(EPS))))
    assert (q[10] == 0x7F).all() and (sc[10] == 0xFF).all() and np.isnan(rstd[10])
    assert rstd[20] == 0 and (q[20, 64:] == 0x7F).all() and (sc[20] == [0, 0, 0xFF]).all()
    assert ((q[20, :64] & 0x7F) == 0).all()
    # columns: the blocks of rows 0-31 hold a NaN in every column, those after hold none
    assert (sT[:, 0] == 0xFF).all() and (qT[:, :32] == 0x7F).all() and (sT[:, 1:3] != 0xFF).all()
    keep = [i for i in range(M) if i not in (10, 20)]
    ref = mxq.mx_rms_norm(to_dev_bf16(x[keep]), to_dev_bf16(w), eps=EPS)
    np.testing.assert_array_equal(q[keep], host(ref[3]))
    np.testing.assert_array_equal(sc[keep], host(ref[4]))


def test_extreme_magnitudes():
    """Squares that leave FP32 on either side: BF16 values near 2^120 and 2^-120."""
    K = 256
    for e in (120, -120):
        x = _bits((9, K), 9, "nx")
        v = np.ldexp(bf16_bits_to_f64(x), e)
        xb = (v.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
        v = bf16_bits_to_f64(xb)
        out = mxq.mx_rms_norm(to_dev_bf16(xb), to_dev_bf16(np.full(K, 0x3F80, np.uint16)), eps=1e-38, y=True)
        r, ry = norm.rms_norm(v, np.ones(K), 1e-38)
        rstd, y = host(out[1]).astype(np.float64), host(out[2])
        # the quotient may be subnormal in FP32: half a step of 2^-149
        assert (np.abs(rstd - r) <= U * 1.01 * r + 2.0 ** -150).all()
        if e < 0:
            _check_bf16(y, ry, 3.01 * U * np.abs(ry))


def test_empty():
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    qT = torch.full((64, 64), SENTINEL, dtype=torch.uint8, device="cuda")
    sT = torch.full((64, 2), SENTINEL, dtype=torch.uint8, device="cuda")
    out = mxq.mx_rms_norm(x, w, qT=qT, scaleT=sT)
    assert out[3].shape == (0, 64) and (qT == 0).all() and (sT == 0).all()
    dx, dw = mxq.mx_rms_norm_backward(x, x, torch.empty(0, device="cuda"), w)
    assert dx.shape == (0, 64) and (dw == 0).all()


# ---------------------------------------------------------------------------
# gradient
# ---------------------------------------------------------------------------

def _grad_case(M, K, seed, stream):
    dy, s, w = _bits((M, K), seed, "ndy", 1e-3), _bits((M, K), seed, "ns"), _weight(K, seed)
    ds = _bits((M, K), seed, "nds", 1e-3) if stream else None
    rstd = norm.rms_norm(bf16_bits_to_f64(s), 1.0, EPS)[0].astype(np.float32)
    return dy, s, w, ds, rstd


def _check_grad(dy, s, w, ds, rstd, dx, dw):
    f = bf16_bits_to_f64
    vdy, vs, vw, r = f(dy), f(s), f(w), rstd.astype(np.float64)
    M, K = vdy.shape
    rdx, rdw = norm.rms_norm_backward(vdy, vs, r, vw, None if ds is None else f(ds))
    g, xh = vdy * vw, vs * r[:, None]
    c = (g * xh).mean(axis=1, keepdims=True)
    ec = (8 * 4 + 6 + 16 + 3) * U * np.abs(g * xh).mean(axis=1, keepdims=True)
    inner = U * np.abs(g) + np.abs(xh) * (ec + 3 * U * np.abs(c)) + U * (np.abs(g) + np.abs(xh * c))
    d = r[:, None] * inner + U * (np.abs(rdx) + (0 if ds is None else np.abs(f(ds))))
    _check_bf16(host(dx), rdx, d)
    if dw is not None:
        depth = -(-M // 512) + 4 + 32 + 16
        assert (np.abs(host(dw).astype(np.float64) - rdw) <= 1.01 * depth * U * np.abs(vdy * xh).sum(axis=0)).all()


@pytest.mark.parametrize("M,K", ROWS + [(2500, 512), (2100, 64)])
@pytest.mark.parametrize("stream", [False, True])
def test_gradient(M, K, stream):
    say(f"rms norm gradient M={M} K={K} stream={stream}")
    dy, s, w, ds, rstd = _grad_case(M, K, M + 2 * K, stream)
    got = mxq.mx_rms_norm_backward(to_dev_bf16(dy), to_dev_bf16(s), to_dev(rstd), to_dev_bf16(w),
                                   dtotal=None if ds is None else to_dev_bf16(ds))
    _check_grad(dy, s, w, ds, rstd, *got)


def test_gradient_strided_in_place_and_without_dw():
    M, K = 700, 2048
    dy, s, w, ds, rstd = _grad_case(M, K, 11, True)
    args = to_dev(rstd), to_dev_bf16(w)
    a = mxq.mx_rms_norm_backward(to_dev_bf16(dy), to_dev_bf16(s), *args, dtotal=to_dev_bf16(ds))
    _check_grad(dy, s, w, ds, rstd, *a)
    wide = [_wide(to_dev_bf16(t), n) for t, n in ((dy, 64), (s, 24), (ds, 16))]
    b = mxq.mx_rms_norm_backward(wide[0], wide[1], *args, dtotal=wide[2], dx=wide[2], dw=False)
    assert b[1] is None and torch.equal(a[0], b[0]) and b[0].data_ptr() == wide[2].data_ptr()
    c = mxq.mx_rms_norm_backward(wide[0], wide[1], *args, dtotal=to_dev_bf16(ds), dx=wide[0])
    assert torch.equal(a[0], c[0]) and torch.equal(a[1], c[1])


def test_gradient_against_differences():
    """dx and dw along random directions, against differences of the oracle's float64 norm."""
    M, K, h = 6, 96, 1e-5
    rng = np.random.default_rng(3)
    dy, s, w, ds, _ = _grad_case(M, K, 12, True)
    f = bf16_bits_to_f64
    rstd = norm.rms_norm(f(s), f(w), EPS)[0].astype(np.float32)
    dx, dw = mxq.mx_rms_norm_backward(to_dev_bf16(dy), to_dev_bf16(s), to_dev(rstd), to_dev_bf16(w),
                                      dtotal=to_dev_bf16(ds))
    dx, dw = f(host(dx)), host(dw).astype(np.float64)
    loss = lambda s, w: (norm.rms_norm(s, w, EPS)[1] * f(dy)).sum() + (s * f(ds)).sum()
    for _ in range(6):
        a, b = rng.normal(size=(M, K)), rng.normal(size=K)
        num = (loss(f(s) + h * a, f(w)) - loss(f(s) - h * a, f(w))) / (2 * h)
        # BF16's half step on each of dx's values, and the difference quotient's own 1e-6
        assert abs((dx * a).sum() - num) <= 2.0 ** -8 * np.abs(dx * a).sum() + 1e-6
        num = (loss(f(s), f(w) + h * b) - loss(f(s), f(w) - h * b)) / (2 * h)
        assert abs((dw * b).sum() - num) <= 100 * U * np.abs(dw * b).sum() + 1e-6


def test_repeated_calls_give_the_same_bits():
    M, K = 5000, 2048
    x, dy, w = (to_dev_bf16(_bits((M, K), 13, n)) for n in ("nx", "ny", "nz"))
    w = w[0].contiguous()
    out = mxq.mx_rms_norm(x, w, columns=True)
    a = mxq.mx_rms_norm_backward(dy, x, out[1], w)
    for _ in range(3):
        b = mxq.mx_rms_norm_backward(dy, x, out[1], w)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("K,columns", [(96, False), (96, True), (544, True), (1056, True), (4128, False)])
def test_values_past_the_range_of_bfloat16(K, columns):
    """total and y that FP32 holds and BF16 does not are infinite, with the column copy too;
    their codes come from the FP32 value."""
    M = 33
    top = 0x7F7F                                            # (2 - 2^-7) 2^127
    x = np.zeros((M, K), np.uint16)
    r = np.zeros((M, K), np.uint16)
    x[5, 40], r[5, 40] = top, 0x7B00                        # + 2^119: a tie, to the even 2^128
    x[6, 40], r[6, 40] = top | 0x8000, 0xFB00
    x[7, 40], r[7, 40] = top, 0x7A80                        # + 2^118: back to the largest value
    w = np.full(K, 0x3F80, np.uint16)
    total, rstd, y, *_ = [None if t is None else host(t) for t in mxq.mx_rms_norm(
        to_dev_bf16(x), to_dev_bf16(w[None])[0].contiguous(), residual=to_dev_bf16(r), eps=EPS, y=True,
        columns=columns)]
    assert (total[5, 40], total[6, 40], total[7, 40]) == (0x7F80, 0xFF80, top)
    assert np.isnan(bf16_bits_to_f64(y[5:7])).any(axis=1).all()
    # y = s w / rms.  Rows of ones: rms just above 1, y just below w's largest value
    s = np.full((M, K), 0x3F80, np.uint16)
    s[3, 64], w[64] = 0x3FC0, top                           # 1.5: past FP32's range too
    s[4, 64] = 0x3F81                                       # (1 + 2^-7) (2 - 2^-7) > 2: as well
    # 181^2 / 2^14 = 1.99957 is between BF16's largest (2 - 2^-7, up to 2 - 2^-8 rounding to it) and
    # FP32's; the row's squares are K - 2 + 0 + 1.99945, so rms is 1 to 3 / K 10^-4
    s[8, 65], s[8, 66], w[65] = 0x3FB5, 0, 0x7F35
    v = bf16_bits_to_f64(s)
    ref = norm.rms_norm(v, bf16_bits_to_f64(w), EPS)[1]
    assert (2 - 2.0 ** -8) * 2.0 ** 127 < ref[8, 65] < (2 - 2.0 ** -13) * 2.0 ** 127
    assert (ref[[3, 4], 64] > 2.0 ** 128).all()
    out = mxq.mx_rms_norm(to_dev_bf16(s), to_dev_bf16(w[None])[0].contiguous(), eps=EPS, y=True, columns=columns)
    got = bf16_bits_to_f64(host(out[2]))
    big = np.zeros((M, K), bool)
    big[[3, 4], 64] = big[8, 65] = True
    assert np.isinf(got[big]).all() and np.isfinite(got[~big]).all()
    scale = host(out[4])
    assert (scale[[3, 4], 2] == 0xFF).all() and scale[8, 2] == 127 + 119 and host(out[3])[8, 65] == 0x7E
    if columns:
        assert host(out[6])[64, 0] == 0xFF and host(out[6])[65, 0] == 127 + 119 and host(out[5])[65, 8] == 0x7E
