"""Latent attention oracle: the MX latent cache, absorbed attention over it, and
expanded attention with its gradient.  Test infrastructure.

Float64 NumPy, row by row over each row's visible keys alone, so that nothing a
mask hides can reach a result.  The cache's codes and scales are those of
:mod:`oracle.mx` (1x32 blocks).
"""

import numpy as np

from . import codec, mx

LATENT, ROPE, NOPE, VALUE = 512, 64, 128, 128


def cache_write(cache, c_bits, rope_bits, slots):
    """Copies of (codes, scales, k_rope bits) with the tokens in their slots;
    slots outside the cache are skipped."""
    codes, scales, rope = (a.copy() for a in cache)
    q, s = mx.mx_quantize_rowwise(c_bits)
    for t, slot in enumerate(np.asarray(slots)):
        if 0 <= slot < codes.shape[0]:
            codes[slot], scales[slot], rope[slot] = q[t], s[t], rope_bits[t]
    return codes, scales, rope


def cache_read(cache, slots):
    """BF16 bit patterns (c, k_rope) of the slots; zeros outside the cache."""
    codes, scales, rope = cache
    slots = np.asarray(slots)
    ok = (slots >= 0) & (slots < codes.shape[0])
    at = np.where(ok, slots, 0)
    c = codec.bf16_round_to_bits(mx.mx_dequantize(codes[at], scales[at]))
    return (np.where(ok[:, None], c, 0).astype(np.uint16),
            np.where(ok[:, None], rope[at], 0).astype(np.uint16))


def softmax_row(z):
    """(probabilities, log-sum-exp) of one row's visible logits."""
    if z.size == 0:
        return z, -np.inf
    m = z.max()
    if not np.isfinite(m):
        with np.errstate(invalid="ignore"):
            return np.full_like(z, np.nan), np.nan
    e = np.exp(z - m)
    return e / e.sum(), m + np.log(e.sum())


def decode(q, cache_values, k_rope, slots_of, lens, scale):
    """Absorbed attention: q [B, S, H, 576], cache_values [slots, 512] and
    k_rope [slots, 64] in float64, slots_of[b][t] the slot of token t.  Returns
    o [B, S, H, 512], lse [B, S, H] and the error scales of o:
    sum p |c| and the rows' largest sum |q| |k|."""
    B, S, H, _ = q.shape
    o = np.zeros((B, S, H, LATENT))
    lse = np.full((B, S, H), -np.inf)
    mag = np.zeros((B, S, H, LATENT))
    zmag = np.zeros((B, S, H))
    for b in range(B):
        for s in range(S):
            n = max(0, int(lens[b]) - (S - 1 - s))
            at = np.asarray(slots_of[b])[:n].astype(np.int64)
            c = cache_values[at]
            k = np.concatenate([c, k_rope[at]], 1)
            with np.errstate(invalid="ignore"):
                z = q[b, s] @ k.T * scale
            for h in range(H):
                p, lse[b, s, h] = softmax_row(z[h])
                with np.errstate(invalid="ignore"):
                    o[b, s, h] = p @ c
                    mag[b, s, h] = p @ np.abs(c)
                if n:
                    zmag[b, s, h] = (np.abs(q[b, s, h]) @ np.abs(k).T).max()
    return o, lse, mag, zmag


def visible(i, lq, lk, causal):
    """Keys that query i of a sequence sees: the first of them."""
    return max(0, min(lk, i + lk - lq + 1)) if causal else lk


def _sequences(q, k_nope, offsets_q, offsets_k):
    if offsets_q is None:
        return [(0, q.shape[0], 0, k_nope.shape[0])]
    oq, ok = np.asarray(offsets_q), np.asarray(offsets_k)
    return [(oq[b], oq[b + 1], ok[b], ok[b + 1]) for b in range(len(oq) - 1)]


def attention(q, k_nope, k_rope, v, offsets_q, offsets_k, scale, causal):
    """Expanded attention, forward: o [Tq, H, 128], lse [H, Tq]."""
    Tq, H, _ = q.shape
    o = np.zeros((Tq, H, VALUE))
    lse = np.full((H, Tq), -np.inf)
    for q0, q1, k0, k1 in _sequences(q, k_nope, offsets_q, offsets_k):
        for h in range(H):
            k = np.concatenate([k_nope[k0:k1, h], k_rope[k0:k1]], 1)
            for i in range(q1 - q0):
                n = visible(i, q1 - q0, k1 - k0, causal)
                with np.errstate(invalid="ignore"):
                    p, lse[h, q0 + i] = softmax_row(k[:n] @ q[q0 + i, h] * scale)
                    o[q0 + i, h] = p @ v[k0:k0 + n, h]
    return o, lse


def attention_backward(dout, q, k_nope, k_rope, v, offsets_q, offsets_k, scale, causal):
    """Gradients of attention() and, for each, a bound of what BF16 operands,
    FP32 sums and one BF16 rounding of P, dS and the result can add:
    {name: (value, bound)} for o, lse, dq, dk_nope, dk_rope and dv."""
    u16, u32 = 2.0 ** -8, 2.0 ** -24            # half a unit in the last place, relative
    Tq, H, _ = q.shape
    val = {"o": np.zeros((Tq, H, VALUE)), "lse": np.full((H, Tq), -np.inf),
           "dq": np.zeros_like(q), "dk_nope": np.zeros_like(k_nope),
           "dk_rope": np.zeros_like(k_rope), "dv": np.zeros_like(v)}
    err = {n: np.zeros_like(a) for n, a in val.items()}
    err["lse"] = np.zeros((H, Tq))
    for q0, q1, k0, k1 in _sequences(q, k_nope, offsets_q, offsets_k):
        for h in range(H):
            k = np.concatenate([k_nope[k0:k1, h], k_rope[k0:k1]], 1)
            vh = v[k0:k1, h]
            dk, dke = np.zeros_like(k), np.zeros_like(k)
            dv, dve = np.zeros_like(vh), np.zeros_like(vh)
            for i in range(q1 - q0):
                n = visible(i, q1 - q0, k1 - k0, causal)
                if n == 0:
                    continue
                qi, g = q[q0 + i, h], dout[q0 + i, h]
                kn, vn = k[:n], vh[:n]
                z = kn @ qi * scale
                p, lse = softmax_row(z)
                o = p @ vn
                # logits: sums of 192 products in FP32 and the exponential's argument and
                # result; a probability's relative error is then at most 2 dz + a few units
                dz = 200 * u32 * scale * (np.abs(kn) @ np.abs(qi)).max() + 8 * u32 * np.abs(z).max()
                rp = 2 * dz + 16 * u32 + n * u32
                oe = u16 * np.abs(o) + (u16 + rp) * (p @ np.abs(vn)) * (1 + u16)
                val["o"][q0 + i, h], err["o"][q0 + i, h] = o, oe
                val["lse"][h, q0 + i] = lse
                err["lse"][h, q0 + i] = dz + 4 * u32 * (np.abs(lse) + 16) + n * u32
                dp = vn @ g
                d = g @ o
                ds = p * (dp - d)
                dpe = 136 * u32 * (np.abs(vn) @ np.abs(g))
                de = np.abs(g) @ oe + 136 * u32 * (np.abs(g) @ np.abs(o))
                dse = p * (rp * np.abs(dp - d) + (dpe + de) * (1 + rp))
                dse = dse + u16 * (np.abs(ds) + dse)
                val["dq"][q0 + i, h] = scale * (ds @ kn)
                err["dq"][q0 + i, h] = scale * ((dse + n * u32 * np.abs(ds)) @ np.abs(kn))
                dk[:n] += scale * np.outer(ds, qi)
                dke[:n] += scale * np.outer(dse + 1e-3 * u16 * np.abs(ds), np.abs(qi))
                dv[:n] += np.outer(p, g)
                dve[:n] += np.outer(p * (u16 + rp) * (1 + u16), np.abs(g))
            val["dk_nope"][k0:k1, h], err["dk_nope"][k0:k1, h] = dk[:, :NOPE], dke[:, :NOPE]
            val["dk_rope"][k0:k1] += dk[:, NOPE:]
            err["dk_rope"][k0:k1] += dke[:, NOPE:]
            val["dv"][k0:k1, h], err["dv"][k0:k1, h] = dv, dve
    for n in ("dq", "dk_nope", "dk_rope", "dv"):    # the result's own rounding
        err[n] += u16 * (np.abs(val[n]) + err[n]) + 2.0 ** -126
    return {n: (val[n], err[n]) for n in val}
