"""The MX latent cache and the absorbed attention over it, on the GPU, against
the float64 oracle: written codes and scales bit for bit (they are the row-wise
quantizer's), values read back bit for bit, attention within bounds derived
from the formats (one BF16 rounding of the probabilities and of the result,
FP32 sums)."""

import numpy as np
import pytest
import torch

from block_quant_gemm_amd import mxq, workloads
from oracle import codec, latent, mx
from tests.gpu_helpers import host, say, to_dev, to_dev_bf16

pytestmark = pytest.mark.gpu

U16, U32 = 2.0 ** -8, 2.0 ** -24              # half units in the last place, relative


def _tokens(T, seed, special=True):
    """BF16 bits [T, 576] as the kv-down projection gives them (latent, rotary key),
    with blocks of zeros, subnormals, NaN, infinities and the largest value."""
    x = workloads.bf16_normal((T, 576), 1.0, seed=seed, name="latent", outlier_frac=0.01,
                              outlier_scale=40.0)
    if special and T >= 8:
        x[0, 0:32] = 0
        x[1, 32:64] = 0x0001                    # smallest subnormal
        x[2, 64] = 0x7FC0                       # NaN
        x[3, 96] = 0xFF80                       # -inf
        x[4, 128:160] = 0x7F7F                  # largest finite
        x[5, 160:192] = 0x8000                  # -0
        x[6, 511] = 0x7F80
        x[7, 192:224] = 0x0080                  # smallest normal
    return x


def _random_cache(slots, seed):
    rng = np.random.default_rng(seed)
    return (rng.integers(0, 256, (slots, 512), dtype=np.uint8),
            rng.integers(0, 256, (slots, 16), dtype=np.uint8),
            rng.integers(0, 65536, (slots, 64)).astype(np.uint16))


def _to_gpu(cache):
    return to_dev(cache[0]), to_dev(cache[1]), to_dev_bf16(cache[2])


@pytest.mark.parametrize("T", [0, 1, 3, 8, 67, 1025, 5000])
def test_write_equals_rowwise_quantization(T):
    say(f"latent cache write T={T}")
    slots_n = T + 37
    x = _tokens(T, T + 1)
    rng = np.random.default_rng(T)
    slots = rng.permutation(slots_n)[:T].astype(np.int64)
    if T >= 8:
        slots[1], slots[5], slots[6] = -1, slots_n, 1 << 40      # not in the cache: skipped
    before = _random_cache(slots_n, T)
    cache = _to_gpu(before)
    xd = to_dev_bf16(x)
    mxq.mx_latent_cache_write(xd[:, :512], xd[:, 512:], to_dev(slots), cache)
    ref = latent.cache_write(before, np.ascontiguousarray(x[:, :512]) if T else x[:, :512],
                             x[:, 512:], slots)
    for got, want, name in zip(cache, ref, ("codes", "scales", "k_rope")):
        assert np.array_equal(host(got), want), name


def test_write_into_strided_arrays_leaves_the_gaps():
    say("latent cache write, strided cache arrays")
    T, n = 130, 200
    x = _tokens(T, 5)
    codes = torch.full((n, 640), 0xEE, dtype=torch.uint8, device="cuda")
    scales = torch.full((n, 23), 0xEE, dtype=torch.uint8, device="cuda")
    rope = torch.full((n, 72), 7.0, dtype=torch.bfloat16, device="cuda")
    cache = (codes[:, 64:576], scales[:, 3:19], rope[:, :64])
    c = to_dev_bf16(x[:, :512])
    r = to_dev_bf16(x[:, 512:])
    slots = np.arange(T, dtype=np.int64)[::-1].copy()
    mxq.mx_latent_cache_write(c, r, to_dev(slots), cache)
    q, s = mx.mx_quantize_rowwise(np.ascontiguousarray(x[:, :512]))
    assert np.array_equal(host(cache[0])[slots], q) and np.array_equal(host(cache[1])[slots], s)
    assert np.array_equal(host(cache[2])[slots], x[:, 512:])
    assert (codes[:, :64] == 0xEE).all() and (codes[:, 576:] == 0xEE).all()
    assert (scales[:, :3] == 0xEE).all() and (scales[:, 19:] == 0xEE).all()
    assert (rope[:, 64:] == 7.0).all() and (codes[T:] == 0xEE).all()
    c2, r2 = mxq.mx_latent_cache_read(cache, to_dev(slots))
    rc, rr = latent.cache_read((q, s, x[:, 512:]), np.arange(T))
    assert np.array_equal(host(r2), rr)
    _equal_bf16(host(c2), rc)


def _equal_bf16(got, want):
    """Bit equality, any NaN for NaN."""
    nan = ((want & 0x7F80) == 0x7F80) & ((want & 0x7F) != 0)
    gnan = ((got & 0x7F80) == 0x7F80) & ((got & 0x7F) != 0)
    assert np.array_equal(nan, gnan)
    assert np.array_equal(got[~nan], want[~nan])


def test_read_every_code_under_every_scale():
    say("latent cache read, 256 codes x 256 scales")
    codes = np.tile(np.arange(256, dtype=np.uint8), (256, 2))
    scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 16, 1)
    rope = _random_cache(256, 9)[2]
    cache = (codes, scales, rope)
    slots = np.concatenate([np.arange(256), [-1, 256, 1 << 50, 3, 3]]).astype(np.int64)
    c, r = mxq.mx_latent_cache_read(_to_gpu(cache), to_dev(slots))
    rc, rr = latent.cache_read(cache, slots)
    assert np.array_equal(host(r), rr)
    _equal_bf16(host(c), rc)


@pytest.mark.parametrize("T", [0, 1, 5, 700, 4099])
def test_read_into_strided_rows(T):
    say(f"latent cache read T={T}")
    cache = _random_cache(900, 3)
    cache[1][:] = np.clip(cache[1], 90, 160)
    slots = np.random.default_rng(T).integers(0, 900, T).astype(np.int64)
    out = torch.full((T, 592), 5.0, dtype=torch.bfloat16, device="cuda")
    mxq.mx_latent_cache_read(_to_gpu(cache), to_dev(slots), c=out[:, 8:520], k_rope=out[:, 520:584])
    rc, rr = latent.cache_read(cache, slots)
    _equal_bf16(host(out[:, 8:520]), rc)
    assert np.array_equal(host(out[:, 520:584]), rr)
    assert (out[:, :8] == 5.0).all() and (out[:, 584:] == 5.0).all()


# ---------------------------------------------------------------------------

def _pool(lens, page, spare, seed, fill_nan=False, gpu_slots=None):
    """A written cache, its page table and the slots of each request's tokens.
    Slots that no token owns hold NaN codes with fill_nan."""
    rng = np.random.default_rng(seed)
    need = [-(-int(n) // page) for n in lens]
    npages = sum(need) + spare
    order = rng.permutation(npages)
    width = max(1, max(need) if need else 1)
    pages = np.full((len(lens), width), -7, np.int32)            # entries past the end: not read
    slots, at = [], 0
    for b, n in enumerate(lens):
        own = order[at:at + need[b]]
        at += need[b]
        pages[b, :need[b]] = own
        t = np.arange(int(n))
        slots.append(own[t // page] * page + t % page if n else np.zeros(0, np.int64))
    total = npages * page
    x = _tokens(total, seed, special=False)
    codes, scales = mx.mx_quantize_rowwise(np.ascontiguousarray(x[:, :512]))
    rope = np.ascontiguousarray(x[:, 512:])
    if fill_nan:
        free = np.ones(total, bool)
        for s in slots:
            free[s] = False
        codes[free], scales[free], rope[free] = 0x7F, 0xFF, 0x7FC0
    return (codes, scales, rope), pages, slots


def _check_decode(q_bits, cache, slots, lens, scale, o, lse):
    q = codec.bf16_bits_to_f64(q_bits)
    c = mx.mx_dequantize(cache[0], cache[1])
    kr = codec.bf16_bits_to_f64(cache[2])
    ro, rl, mag, zmag = latent.decode(q, c, kr, slots, lens, scale)
    nmax = max([1] + [int(n) for n in lens])
    # logits: 576 products summed in FP32, then the exponential's argument and result
    dz = 580 * U32 * scale * zmag + 8 * U32 * np.abs(np.where(np.isfinite(rl), rl, 0))
    rp = 2 * dz + 16 * U32 + nmax * U32
    tol = U16 * np.abs(ro) + (U16 + rp)[..., None] * mag * (1 + U16) + 2.0 ** -126
    go = codec.bf16_bits_to_f64(host(o))
    gl = host(lse).astype(np.float64)
    bad = np.isnan(ro)
    assert np.array_equal(np.isnan(go), bad)
    assert np.array_equal(np.isneginf(gl), np.isneginf(rl)) and np.array_equal(np.isnan(gl), np.isnan(rl))
    d = np.abs(go[~bad] - ro[~bad])
    assert (d <= tol[~bad]).all(), f"o off by {np.max(d / tol[~bad]):.3g} of its bound"
    fine = np.isfinite(rl)
    dl = np.abs(gl[fine] - rl[fine])
    tl = (dz + 4 * U32 * (np.abs(np.where(fine, rl, 0)) + 16) + nmax * U32)[fine]
    assert (dl <= tl).all(), f"lse off by {np.max(dl / tl):.3g} of its bound"


CASES = [
    # lens, page, S, H
    ([1], 16, 1, 16),
    ([0, 1, 2, 63, 64, 65, 127, 128, 129], 16, 1, 16),
    ([200, 3, 77], 7, 1, 5),
    ([64, 640, 1], 1, 1, 1),
    ([300, 0, 1, 2, 3], 100, 3, 16),
    ([333, 65], 48, 2, 12),
    ([129, 1000], 64, 1, 33),
    ([500, 64], 32, 2, 64),
    ([70, 5], 64, 1, 128),
    ([5000], 64, 1, 16),
    ([4500, 1, 900], 128, 2, 8),
    ([10] * 130, 16, 1, 4),
    ([200] * 300, 16, 1, 2),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_decode(case):
    lens, page, S, H = CASES[case]
    say(f"latent decode B={len(lens)} S={S} H={H} page={page} longest={max(lens)}")
    cache, pages, slots = _pool(lens, page, 2, case, fill_nan=True)
    q = workloads.bf16_normal((len(lens), S, H, 576), 0.7, seed=case, name="dq")
    scale = 192 ** -0.5
    o, lse = mxq.mx_latent_decode(to_dev_bf16(q), _to_gpu(cache), to_dev(pages),
                                  to_dev(np.array(lens, np.int64)), page, max(lens), scale)
    _check_decode(q, cache, slots, lens, scale, o, lse)


def test_decode_strided_loose_bound_and_repeatable():
    """Strided queries and results, a bound far above the lengths (another split
    of the work), lengths past the bound, and the same bits from run to run."""
    say("latent decode, strided, loose bound")
    lens, page, S, H = [700, 64, 0, 1300], 16, 2, 16
    cache, pages, slots = _pool(lens, page, 40, 77)
    wide = np.concatenate([pages, np.zeros((4, 400), np.int32)], 1)
    q = workloads.bf16_normal((4, S, H, 576), 0.7, seed=9, name="sq")
    buf = torch.zeros((4, S, H + 2, 640), dtype=torch.bfloat16, device="cuda")
    buf[:, :, 1:H + 1, 16:592] = to_dev_bf16(q)
    ob = torch.full((4, H, S, 520), 3.0, dtype=torch.bfloat16, device="cuda")
    qv, ov = buf[:, :, 1:H + 1, 16:592], ob.transpose(1, 2)[..., :512]
    dev = _to_gpu(cache)
    args = (qv, dev, to_dev(wide), to_dev(np.array(lens, np.int64)), page)
    o, lse = mxq.mx_latent_decode(*args, 6000, 0.1, o=ov)
    _check_decode(q, cache, slots, lens, 0.1, o.contiguous(), lse)
    assert (ob[..., 512:] == 3.0).all()
    first = (o.clone(), lse.clone())
    for _ in range(3):
        o2, lse2 = mxq.mx_latent_decode(*args, 6000, 0.1)
        assert torch.equal(o2.view(torch.int16), first[0].view(torch.int16)) and torch.equal(lse2, first[1])
    cut = [600, 64, 0, 600]
    o, lse = mxq.mx_latent_decode(*args, 600, 0.1)
    _check_decode(q, cache, slots, cut, 0.1, o, lse)


@pytest.mark.parametrize("lens,S", [([66, 300], 3), ([65], 2), ([2, 200, 129], 2)])
def test_decode_nan_in_hidden_tokens_stays_hidden(lens, S):
    """The last tokens hold NaN and infinity: query tokens before them do not see
    them, later ones do."""
    say(f"latent decode, NaN in the last tokens, lens={lens} S={S}")
    cache, pages, slots = _pool(lens, 16, 1, 31)
    for b, n in enumerate(lens):
        s = int(slots[b][n - 1])
        if b % 2 == 0:
            cache[0][s, 32:64], cache[1][s, 1] = 0x7F, 0xFF      # as a NaN block is written
        else:
            cache[0][s, 40] = 0x7F                               # one NaN code
    q = workloads.bf16_normal((len(lens), S, 20, 576), 0.7, seed=4, name="nq")
    o, lse = mxq.mx_latent_decode(to_dev_bf16(q), _to_gpu(cache), to_dev(pages),
                                  to_dev(np.array(lens, np.int64)), 16, max(lens), 0.05)
    go, gl = codec.bf16_bits_to_f64(host(o)), host(lse)
    assert np.isnan(go[:, -1]).all() and np.isnan(gl[:, -1]).all()
    sub = [n - 1 for n in lens]
    _check_decode(q[:, :-1], cache, slots, sub, 0.05, o[:, :-1].contiguous(), lse[:, :-1].contiguous())


def test_decode_extreme_logits():
    """One key far ahead of the others, logits of hundreds, equal logits."""
    say("latent decode, extreme logits")
    lens = [130, 257]
    cache, pages, slots = _pool(lens, 16, 1, 5)
    q = workloads.bf16_normal((2, 1, 16, 576), 30.0, seed=6, name="xq")
    q[0, 0, 3] = 0                                               # all logits equal
    for scale in (1.0, 1e-3):
        o, lse = mxq.mx_latent_decode(to_dev_bf16(q), _to_gpu(cache), to_dev(pages),
                                      to_dev(np.array(lens, np.int64)), 16, 257, scale)
        _check_decode(q, cache, slots, lens, scale, o, lse)


def test_slots_past_32_bit_byte_offsets():
    """A pool whose code bytes pass 2^32: writing, reading and attending at its end."""
    n = (1 << 23) + 4096                                         # 512 n > 2^32
    say(f"latent cache of {n} slots")
    cache = mxq.latent_cache(n)
    T, page = 300, 64
    x = _tokens(T, 2, special=False)
    base = n // page - 5
    pages = np.array([[base + 4, base, base + 2, base + 1, base + 3]], np.int32)
    t = np.arange(T)
    slots = (pages[0][t // page].astype(np.int64) * page + t % page)
    xd = to_dev_bf16(x)
    mxq.mx_latent_cache_write(xd[:, :512], xd[:, 512:], to_dev(slots), cache)
    codes, scales = mx.mx_quantize_rowwise(np.ascontiguousarray(x[:, :512]))
    small = (codes, scales, np.ascontiguousarray(x[:, 512:]))
    c, r = mxq.mx_latent_cache_read(cache, to_dev(slots))
    rc, rr = latent.cache_read(small, t)
    assert np.array_equal(host(c), rc) and np.array_equal(host(r), rr)
    assert int(cache[0][:n - 5 * page].count_nonzero()) == 0     # nothing wrapped around
    q = workloads.bf16_normal((1, 1, 16, 576), 0.7, seed=1, name="bq")
    o, lse = mxq.mx_latent_decode(to_dev_bf16(q), cache, to_dev(pages),
                                  to_dev(np.array([T], np.int64)), page, T, 0.07)
    _check_decode(q, small, [t], [T], 0.07, o, lse)


def test_pages_outside_the_pool_are_not_read():
    """Bad page numbers give that request unspecified values; the others' are unharmed."""
    say("latent decode, bad page numbers")
    lens = [200, 150]
    cache, pages, slots = _pool(lens, 16, 1, 8)
    pages[0, :3] = [-5, 1 << 30, cache[0].shape[0] // 16]
    q = workloads.bf16_normal((2, 1, 16, 576), 0.7, seed=8, name="pq")
    o, lse = mxq.mx_latent_decode(to_dev_bf16(q), _to_gpu(cache), to_dev(pages),
                                  to_dev(np.array(lens, np.int64)), 16, 200, 0.07)
    _check_decode(q[1:], cache, slots[1:], lens[1:], 0.07, o[1:], lse[1:])


def test_empty_batch_and_all_empty_requests():
    say("latent decode, empty")
    cache = _to_gpu(_pool([5], 16, 1, 1)[0])
    q = torch.zeros((0, 1, 16, 576), dtype=torch.bfloat16, device="cuda")
    o, lse = mxq.mx_latent_decode(q, cache, torch.zeros((0, 3), dtype=torch.int32, device="cuda"),
                                  torch.zeros(0, dtype=torch.int64, device="cuda"), 16, 40, 0.1)
    assert o.shape == (0, 1, 16, 512) and lse.shape == (0, 1, 16)
    q = torch.ones((3, 2, 16, 576), dtype=torch.bfloat16, device="cuda")
    lens = torch.tensor([0, -4, 0], dtype=torch.int64, device="cuda")
    for max_len in (0, 40):
        o, lse = mxq.mx_latent_decode(q, cache, torch.zeros((3, 3), dtype=torch.int32, device="cuda"),
                                      lens, 16, max_len, 0.1)
        assert (o == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("T", [32767, 32768, 40001])
def test_read_many_tokens(T):
    """Around the size from which a wavefront reads several tokens; the last of them
    ends inside a workgroup, and some slots are absent."""
    say(f"latent cache read T={T}")
    cache = _random_cache(900, 13)
    slots = np.random.default_rng(T).integers(-20, 920, T).astype(np.int64)
    out = torch.full((T + 1, 576), 5.0, dtype=torch.bfloat16, device="cuda")
    mxq.mx_latent_cache_read(_to_gpu(cache), to_dev(slots), c=out[:T, :512], k_rope=out[:T, 512:])
    rc, rr = latent.cache_read(cache, slots)
    _equal_bf16(host(out[:T, :512]), rc)
    assert np.array_equal(host(out[:T, 512:]), rr)
    assert (out[T:] == 5.0).all()


@pytest.mark.parametrize("T", [3, 33000])
def test_read_from_an_empty_cache(T):
    say(f"latent cache read T={T}, no slots")
    c, r = mxq.mx_latent_cache_read(mxq.latent_cache(0), torch.zeros(T, dtype=torch.int64, device="cuda"))
    assert not c.any() and not r.any()
