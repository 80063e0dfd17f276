"""Measured cases of the latent-attention operators: the MX latent cache
(written, read back, attended to by decoding tokens) and the expanded
attention with its gradient.

One token's latent vector c (512 values) and its rotary key (64 values, shared
by all heads) are what a cache keeps: c as E4M3 codes with one E8M0 scale per
32 values, the rotary key in BF16.  In the expanded form each head has its own
128 key and 128 value columns beside the shared rotary key.

``own = False`` computes every operator in its plain form (elementary torch
operations in 32 bits, rounded once at the end); ``own = True`` makes the
calls of ``block_quant_gemm_amd.mxq``.
"""

import math
import random

import torch

own = False

LATENT, ROPE, NOPE, VALUE = 512, 64, 128, 128
BLOCK = 32
QK = NOPE + ROPE


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decoding step's new tokens of 48 requests enter the cache: latency
        {"name": "write step", "kind": "write", "tokens": 48, "slots": 20000},
        # the block step's 16384 tokens (4096 x 4) enter the cache after a prefill
        {"name": "write prefill", "kind": "write", "tokens": 16384, "slots": 50000},
        # a short cached prefix comes back for a chunk's expanded attention
        {"name": "read short prefix", "kind": "read", "tokens": 419, "slots": 20000, "page": 64},
        # long cached prefixes of a batch, scattered over the pool in small pages
        {"name": "read long prefixes", "kind": "read", "tokens": 65521, "slots": 131072,
         "page": 16},
        # one request decodes by itself: latency
        {"name": "decode one", "kind": "decode", "seqs": 1, "tokens": 1, "heads": 16,
         "low": 1500, "high": 1500, "page": 64, "pick": 1},
        # a serving batch of very different lengths
        {"name": "decode ragged", "kind": "decode", "seqs": 96, "tokens": 1, "heads": 16,
         "low": 1, "high": 6000, "page": 16, "pick": 2},
        # few requests over long documents
        {"name": "decode long", "kind": "decode", "seqs": 6, "tokens": 1, "heads": 16,
         "low": 60000, "high": 120000, "page": 64, "pick": 3},
        # two tokens a request (one drafted) and more heads: 128 query rows a request
        {"name": "decode drafted", "kind": "decode", "seqs": 24, "tokens": 2, "heads": 64,
         "low": 300, "high": 4200, "page": 32, "pick": 4},
        # a short prompt's prefill: latency
        {"name": "prefill short", "kind": "attention", "seqs": 1, "heads": 16, "low": 77,
         "high": 77, "prefix": 0, "causal": True, "train": False, "pick": 5},
        # a ragged batch of prompt chunks that follow cached prefixes
        {"name": "prefill chunks", "kind": "attention", "seqs": 5, "heads": 16, "low": 300,
         "high": 2900, "prefix": 1700, "causal": True, "train": False, "pick": 6},
        # packed short documents in training
        {"name": "train packed", "kind": "attention", "seqs": 7, "heads": 16, "low": 90,
         "high": 700, "prefix": 0, "causal": True, "train": True, "pick": 7},
        # the block step: sequence 4096 x batch 4
        {"name": "train block", "kind": "attention", "seqs": 4, "heads": 16, "low": 4096,
         "high": 4096, "prefix": 0, "causal": True, "train": True, "pick": 8},
    ]


def _log_int(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


#: What the largest listed cases ask of the plain form: logits held, and cached values gathered.
MOST_LOGITS = 4 * 16 * 4096 * 4096
MOST_GATHER = 6 * 120000


def draw(rng):
    kind = rng.choice(["write", "read", "decode", "decode", "attention", "attention"])
    if kind == "write":
        tokens = _log_int(rng, 1, 16384)
        return {"kind": "write", "tokens": tokens, "slots": tokens + _log_int(rng, 1, 30000)}
    if kind == "read":
        tokens = _log_int(rng, 1, 65536)
        return {"kind": "read", "tokens": tokens, "slots": tokens + _log_int(rng, 300, 60000),
                "page": rng.choice([1, 16, 32, 48, 64, 128])}
    if kind == "decode":
        while True:
            c = {"kind": "decode", "seqs": _log_int(rng, 1, 128), "tokens": rng.choice([1, 1, 1, 2, 3]),
                 "heads": rng.choice([4, 8, 16, 16, 32, 64]), "high": _log_int(rng, 40, 120000),
                 "page": rng.choice([16, 32, 48, 64, 128]), "pick": rng.randrange(1 << 20)}
            c["low"] = _log_int(rng, 1, c["high"])
            rows = c["tokens"] * c["heads"]
            if c["seqs"] * c["high"] <= MOST_GATHER and c["seqs"] * c["high"] * rows <= 128 * 24 * 4200:
                return c
    while True:
        c = {"kind": "attention", "seqs": _log_int(rng, 1, 16), "heads": rng.choice([2, 5, 8, 16, 16, 32]),
             "high": _log_int(rng, 16, 8192), "prefix": 0, "causal": rng.random() < 0.8,
             "train": rng.random() < 0.6, "pick": rng.randrange(1 << 20)}
        c["low"] = _log_int(rng, 1, c["high"])
        if not c["train"] or rng.random() < 0.2:
            c["prefix"] = rng.choice([0, _log_int(rng, 1, 4096)])
        lk = c["high"] + c["prefix"]
        # at most half the largest's logits without the causal mask, which halves its work
        most = MOST_LOGITS if c["causal"] and not c["prefix"] else MOST_LOGITS // 2
        if c["seqs"] * c["heads"] * c["high"] * lk <= most:
            return c


def _lengths(case):
    """The sequences' lengths: from the case alone, the first two the extremes, the rest
    spread over the logarithm between them."""
    r = random.Random("%d %d" % (case["pick"], case["seqs"]))
    got = [_log_int(r, case["low"], case["high"]) for _ in range(case["seqs"])]
    got[0] = case["high"]
    if len(got) > 1:
        got[1] = case["low"]
    return got


def _prefixes(case):
    """Cached tokens before each sequence's own (keys and values only)."""
    r = random.Random("prefix %d" % case["pick"])
    got = [r.randint(0, case["prefix"]) for _ in range(case["seqs"])]
    got[0] = case["prefix"]
    return got


def _pairs(case):
    """Query-key pairs that the mask leaves, over all sequences."""
    n = 0
    for lq, pre in zip(_lengths(case), _prefixes(case)):
        n += lq * pre + (lq * (lq + 1) // 2 if case["causal"] else lq * lq)
    return n


def work(case):
    record = LATENT + LATENT // BLOCK + 2 * ROPE             # a token's bytes in the cache
    if case["kind"] in ("write", "read"):
        return {"bytes": case["tokens"] * (2 * (LATENT + ROPE) + record + 8), "flops": 0}
    h = case["heads"]
    lens = _lengths(case)
    if case["kind"] == "decode":
        s = case["tokens"]
        pairs = sum(max(0, n - i) for n in lens for i in range(s))
        rows = case["seqs"] * s * h
        return {"bytes": sum(lens) * record + rows * (2 * (2 * LATENT + ROPE) + 4),
                "flops": 2 * pairs * h * (2 * LATENT + ROPE)}
    tq = sum(lens)
    tk = tq + sum(_prefixes(case))
    # forward: q, keys, values, rotary keys in; output and log-sum-exp out
    reads = 2 * (tq * h * QK + tk * h * (NOPE + VALUE) + tk * ROPE)
    outs = tq * h * (2 * VALUE + 4)
    flops = 2 * _pairs(case) * h * (QK + VALUE)
    if case["train"]:
        # backward: the output's gradient in, the four gradients out; five products
        outs += 2 * tq * h * VALUE + reads
        flops += 2 * _pairs(case) * h * (3 * QK + 2 * VALUE)
    return {"bytes": reads + outs, "flops": flops}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _normal(g, *shape, sigma=1.0):
    return (torch.randn(*shape, generator=g, device=g.device) * sigma).to(torch.bfloat16)


def _latents(g, rows):
    """The kv-down projection's output [rows, 576]: latent and rotary key side by side, 0.5%
    of the values outliers."""
    x = torch.randn(rows, LATENT + ROPE, generator=g, device=g.device)
    big = torch.rand(rows, LATENT + ROPE, generator=g, device=g.device) < 0.005
    return torch.where(big, x * 20, x).to(torch.bfloat16)


def _empty_cache(g, slots):
    """A pool whose slots hold earlier tokens' values."""
    codes = torch.randint(0, 0x78, (slots, LATENT), generator=g, device=g.device, dtype=torch.uint8)
    codes += 0x80 * torch.randint(0, 2, (slots, LATENT), generator=g, device=g.device, dtype=torch.uint8)
    scales = torch.randint(112, 122, (slots, LATENT // BLOCK), generator=g, device=g.device,
                           dtype=torch.uint8)
    return codes, scales, _normal(g, slots, ROPE)


def _paged(g, tokens, slots, page):
    """Slots of `tokens` consecutive tokens whose pages are scattered over the pool."""
    pages = torch.randperm(slots // page, generator=g, device=g.device)
    need = -(-tokens // page)
    at = pages[:need, None] * page + torch.arange(page, device=g.device)
    return at.reshape(-1)[:tokens].contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    if case["kind"] == "write":
        x = _latents(g, case["tokens"])
        s["c"], s["k_rope"] = x[:, :LATENT], x[:, LATENT:]
        s["slots"] = torch.randperm(case["slots"], generator=g, device="cuda")[:case["tokens"]].contiguous()
        s["cache"] = _empty_cache(g, case["slots"])
    elif case["kind"] == "read":
        slots = -(-case["slots"] // case["page"]) * case["page"]
        s["cache"] = _empty_cache(g, slots)
        s["slots"] = _paged(g, case["tokens"], slots, case["page"])
    elif case["kind"] == "decode":
        lens, page = _lengths(case), case["page"]
        need = [-(-n // page) for n in lens]
        pool = sum(need) + 3
        x = _latents(g, pool * page)
        codes, scales = _quantise(x[:, :LATENT])
        s["cache"] = (codes, scales, x[:, LATENT:].contiguous())
        del x
        order = torch.randperm(pool, generator=g, device="cuda")
        starts = torch.tensor([sum(need[:i]) for i in range(len(need))], device="cuda")
        widths = torch.tensor(need, device="cuda")
        col = torch.arange(max(need), device="cuda")
        at = torch.where(col < widths[:, None], starts[:, None] + col, 0)
        s["pages"] = order[at].to(torch.int32).contiguous()
        s["lens"] = torch.tensor(lens, dtype=torch.int64, device="cuda")
        s["max_len"] = case["high"]
        s["q"] = _normal(g, case["seqs"], case["tokens"], case["heads"], LATENT + ROPE, sigma=0.7)
        s["scale"] = QK ** -0.5
    else:
        lq = _lengths(case)
        lk = [a + b for a, b in zip(lq, _prefixes(case))]
        tq, tk, h = sum(lq), sum(lk), case["heads"]
        s["q"] = _normal(g, tq, h, QK)
        kv = _normal(g, tk, h, NOPE + VALUE)           # the kv-up projection's output
        s["k_nope"], s["v"] = kv[..., :NOPE], kv[..., NOPE:]
        s["k_rope"] = _latents(g, tk)[:, LATENT:]      # beside the latent, as projected
        s["do"] = _normal(g, tq, h, VALUE, sigma=1e-2)
        s["offsets_q"], s["offsets_k"] = _offsets(lq), _offsets(lk)
        s["scale"] = QK ** -0.5
        # the padded layout's plan, as a program with the plain form would keep it
        s["pad_q"], s["row_q"] = _padding(lq)
        s["pad_k"], s["row_k"] = _padding(lk)
        i = torch.arange(max(lq), device="cuda")[:, None]
        j = torch.arange(max(lk), device="cuda")[None, :]
        nq = torch.tensor(lq, device="cuda")[:, None, None]
        nk = torch.tensor(lk, device="cuda")[:, None, None]
        seen = (i < nq) & (j < nk)
        if case["causal"]:
            seen = seen & (j <= i + (nk - nq))
        s["seen"] = seen[:, None]
    return s


def _offsets(lens):
    return torch.tensor([0] + lens, dtype=torch.int64, device="cuda").cumsum(0)


def _padding(lens):
    """Row of each (sequence, position), clamped inside the sequence; and the place of each
    row in the padded layout."""
    n = torch.tensor(lens, device="cuda")
    first = n.cumsum(0) - n
    col = torch.arange(max(lens), device="cuda")
    pad = first[:, None] + torch.minimum(col[None, :], n[:, None] - 1)
    seq = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), n)
    row = seq * max(lens) + torch.arange(int(n.sum()), device="cuda") - first[seq]
    return pad, row


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _quantise(x):
    """E4M3 codes and E8M0 scales of BF16 rows, one scale per 32 values."""
    v = x.float().reshape(x.shape[0], -1, BLOCK)
    amax = v.abs().amax(-1)
    bad = ~torch.isfinite(amax)
    e = (torch.frexp(torch.where(bad | (amax == 0), torch.ones_like(amax), amax))[1] - 1 - 8).clamp_min(-127)
    e = torch.where(amax == 0, torch.full_like(e, -127), e)
    codes = (v * torch.exp2(-e.float())[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    codes = torch.where(bad[..., None], 0x7F, codes.view(torch.uint8))
    scales = torch.where(bad, 0xFF, e + 127).to(torch.uint8)
    return codes.to(torch.uint8).reshape(x.shape), scales


def _values(codes, scales):
    """The 32-bit values that codes [..., 512] and scales [..., 16] stand for."""
    v = codes.view(torch.float8_e4m3fn).float()
    return (v.unflatten(-1, (-1, BLOCK)) * torch.exp2(scales.float() - 127)[..., None]).flatten(-2)


def _softmax(logits, seen):
    """Probabilities and log-sum-exp of the logits that `seen` leaves; rows that see nothing
    get zeros and minus infinity."""
    logits = torch.where(seen, logits, -math.inf)
    m = logits.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = torch.exp(logits - m)
    total = p.sum(-1, keepdim=True)
    lse = (m + torch.log(total)).squeeze(-1)
    return p / torch.where(total == 0, torch.ones_like(total), total), lse


def _write_plain(s):
    codes, scales, k_rope = s["cache"]
    q, e = _quantise(s["c"])
    codes[s["slots"]] = q
    scales[s["slots"]] = e
    k_rope[s["slots"]] = s["k_rope"]


def _read_plain(s):
    codes, scales, k_rope = s["cache"]
    at = s["slots"]
    return _values(codes[at], scales[at]).to(torch.bfloat16), k_rope[at]


def _decode_plain(s):
    codes, scales, k_rope = s["cache"]
    q, lens, page = s["q"], s["lens"], s["case"]["page"]
    b, t, h, _ = q.shape
    col = torch.arange(s["max_len"], device=q.device)
    slot = s["pages"][:, col // page].long() * page + col % page                  # [B, L]
    c = _values(codes[slot], scales[slot])                                        # [B, L, 512]
    k = torch.cat([c, k_rope[slot].float()], -1)
    logits = torch.matmul(q.float().reshape(b, t * h, -1), k.transpose(1, 2)) * s["scale"]
    last = lens[:, None] - (t - torch.arange(t, device=q.device))                 # [B, t]
    seen = col <= last[..., None]                                                 # [B, t, L]
    p, lse = _softmax(logits.reshape(b, t, h, -1), seen[:, :, None])
    o = torch.matmul(p.reshape(b, t * h, -1), c).reshape(b, t, h, LATENT)
    return {"o": o.to(torch.bfloat16), "lse": lse}


def _attention_plain(s):
    pad_q, pad_k, h = s["pad_q"], s["pad_k"], s["case"]["heads"]
    q = s["q"][pad_q].float().transpose(1, 2)                                     # [B, H, Lq, 192]
    rope = s["k_rope"][pad_k].float()[:, None].expand(-1, h, -1, -1)
    k = torch.cat([s["k_nope"][pad_k].float().transpose(1, 2), rope], -1)         # [B, H, Lk, 192]
    v = s["v"][pad_k].float().transpose(1, 2)
    p, lse = _softmax(torch.matmul(q, k.transpose(2, 3)) * s["scale"], s["seen"])
    o = torch.matmul(p, v)
    out = {"o": _packed(o, s["row_q"]),
           "lse": lse.transpose(1, 2).reshape(-1, h)[s["row_q"]].t().contiguous()}
    if not s["case"]["train"]:
        return out
    do = s["do"][pad_q].float().transpose(1, 2)
    dp = torch.matmul(do, v.transpose(2, 3))
    ds = p * (dp - (do * o).sum(-1, keepdim=True)) * s["scale"]
    dq = torch.matmul(ds, k)
    dk = torch.matmul(ds.transpose(2, 3), q)
    dv = torch.matmul(p.transpose(2, 3), do)
    out["dq"] = _packed(dq, s["row_q"])
    out["dk_nope"] = _packed(dk[..., :NOPE], s["row_k"])
    out["dk_rope"] = dk[..., NOPE:].sum(1).reshape(-1, ROPE)[s["row_k"]].to(torch.bfloat16)
    out["dv"] = _packed(dv, s["row_k"])
    return out


def _packed(x, row):
    """[B, H, L, d] without its padding, as BF16 [T, H, d]."""
    return x.transpose(1, 2).flatten(0, 1)[row].to(torch.bfloat16)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _cache_values(cache):
    """The cache's buffers as the values that they stand for."""
    codes, scales, k_rope = cache
    return {"codes": codes.view(torch.float8_e4m3fn), "scales": scales.view(torch.float8_e8m0fnu),
            "k_rope": k_rope}


def run(s):
    kind = s["case"]["kind"]
    if kind == "write":
        if own:
            from block_quant_gemm_amd import mxq
            mxq.mx_latent_cache_write(s["c"], s["k_rope"], s["slots"], s["cache"])
        else:
            _write_plain(s)
        return _cache_values(s["cache"])
    if kind == "read":
        if own:
            from block_quant_gemm_amd import mxq
            c, k_rope = mxq.mx_latent_cache_read(s["cache"], s["slots"])
        else:
            c, k_rope = _read_plain(s)
        return {"c": c, "k_rope": k_rope}
    if kind == "decode":
        if own:
            from block_quant_gemm_amd import mxq
            o, lse = mxq.mx_latent_decode(s["q"], s["cache"], s["pages"], s["lens"], s["case"]["page"],
                                          s["max_len"], s["scale"])
            return {"o": o, "lse": lse}
        return _decode_plain(s)
    if not own:
        return _attention_plain(s)
    from block_quant_gemm_amd import mxq
    args = (s["q"], s["k_nope"], s["k_rope"], s["v"])
    how = dict(offsets_q=s["offsets_q"], offsets_k=s["offsets_k"], scale=s["scale"],
               causal=s["case"]["causal"])
    o, lse = mxq.latent_attention(*args, **how)
    out = {"o": o, "lse": lse}
    if s["case"]["train"]:
        dq, dk_nope, dk_rope, dv = mxq.latent_attention_backward(s["do"], *args, o, lse, **how)
        out.update(dq=dq, dk_nope=dk_nope, dk_rope=dk_rope, dv=dv)
    return out


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_e4m3(x):
    """The E4M3 value nearest to each 64-bit value, ties to the even mantissa, at most 448."""
    a = x.abs()
    step = torch.exp2(torch.floor(torch.log2(a.clamp_min(2.0 ** -6))) - 3)
    return torch.sign(x) * (torch.round(a / step) * step).clamp_max(448.0)


def _exact_cache(codes, scales):
    """64-bit values of E4M3 codes under E8M0 scales, from their bit fields."""
    c = codes.long()
    field, mant = (c >> 3) & 15, (c & 7).double()
    v = torch.where(field == 0, mant * 2.0 ** -9, (8 + mant) * torch.exp2(field.double() - 10))
    v = torch.where(c > 127, -v, v)
    return v * torch.exp2(scales.double() - 127).repeat_interleave(BLOCK, -1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "write":
        codes, scales, k_rope = s["cache"]
        out = {"codes": codes.view(torch.float8_e4m3fn).double(),
               "scales": torch.exp2(scales.double() - 127), "k_rope": k_rope.double()}
        blocks = s["c"].double().reshape(case["tokens"], -1, BLOCK)
        e = torch.floor(torch.log2(blocks.abs().amax(-1))) - 8
        out["codes"][s["slots"]] = _exact_e4m3(blocks * torch.exp2(-e)[..., None]).flatten(1)
        out["scales"][s["slots"]] = torch.exp2(e)
        out["k_rope"][s["slots"]] = s["k_rope"].double()
        return out
    if case["kind"] == "read":
        codes, scales, k_rope = s["cache"]
        return {"c": _exact_cache(codes[s["slots"]], scales[s["slots"]]),
                "k_rope": k_rope[s["slots"]].double()}
    if case["kind"] == "decode":
        return _exact_decode(s)
    return _exact_attention(s)


def _exact_decode(s):
    codes, scales, k_rope = s["cache"]
    b, t, h, _ = s["q"].shape
    page = s["case"]["page"]
    o = torch.zeros(b, t, h, LATENT, dtype=torch.float64, device="cuda")
    lse = torch.full((b, t, h), -math.inf, dtype=torch.float64, device="cuda")
    for i, n in enumerate(_lengths(s["case"])):
        col = torch.arange(n, device="cuda")
        slot = s["pages"][i, col // page].long() * page + col % page
        c = _exact_cache(codes[slot], scales[slot])
        k = torch.cat([c, k_rope[slot].double()], 1)
        for j in range(t):
            m = n - (t - 1 - j)
            if m > 0:
                z = (s["q"][i, j].double() @ k[:m].t()) * s["scale"]
                lse[i, j] = torch.logsumexp(z, -1)
                o[i, j] = torch.exp(z - lse[i, j][:, None]) @ c[:m]
    return {"o": o, "lse": lse}


def _exact_attention(s):
    case = s["case"]
    h, train = case["heads"], case["train"]
    names = ["q", "k_nope", "k_rope", "v"]
    x = {n: s[n].double() for n in names}
    o = torch.zeros(*s["q"].shape[:2], VALUE, dtype=torch.float64, device="cuda")
    lse = torch.full((h, s["q"].shape[0]), -math.inf, dtype=torch.float64, device="cuda")
    grads = {n: torch.zeros_like(x[n]) for n in names}
    oq, ok = s["offsets_q"].tolist(), s["offsets_k"].tolist()
    for i in range(case["seqs"]):
        rq, rk = slice(oq[i], oq[i + 1]), slice(ok[i], ok[i + 1])
        lq, lk = oq[i + 1] - oq[i], ok[i + 1] - ok[i]
        hidden = torch.zeros(lq, lk, dtype=torch.bool, device="cuda")
        if case["causal"]:
            hidden = torch.ones_like(hidden).triu(lk - lq + 1)
        for head in range(h):
            leaf = [x["q"][rq, head], x["k_nope"][rk, head], x["k_rope"][rk], x["v"][rk, head]]
            leaf = [u.detach().clone().requires_grad_(train) for u in leaf]
            qh, kn, kr, vh = leaf
            z = (qh[:, :NOPE] @ kn.t() + qh[:, NOPE:] @ kr.t()) * s["scale"]
            z = z.masked_fill(hidden, -math.inf)
            y = torch.softmax(z, -1) @ vh
            o[rq, head] = y.detach()
            lse[head, rq] = torch.logsumexp(z.detach(), -1)
            if train:
                got = torch.autograd.grad(y, leaf, s["do"][rq, head].double())
                grads["q"][rq, head] = got[0]
                grads["k_nope"][rk, head] = got[1]
                grads["k_rope"][rk] += got[2]
                grads["v"][rk, head] = got[3]
    out = {"o": o, "lse": lse}
    if train:
        out.update(dq=grads["q"], dk_nope=grads["k_nope"], dk_rope=grads["k_rope"], dv=grads["v"])
    return out
