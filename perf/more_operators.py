"""Measured cases of the feed-forward half of a block around the MX products: the
root-mean-square norm that makes a product's MX operand (with the residual's addition),
its gradient, the gradient of the routed experts' gate/up product with SwiGLU, and the
feed-forward block of few tokens.

``own = False`` computes every operator in its plain form (elementary torch operations in
32 bits, rounded once at the end); ``own = True`` makes the calls of
``block_quant_gemm_amd.mxq``.  E4M3 codes and E8M0 scales are returned as the values they
stand for (codes in units of their block's scale).
"""

import math
import random

import torch

own = False

BLOCK = 32
EPS = 1e-6
HIDDEN, DENSE, EXPERT = 2048, 10944, 1408


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # decoding: the tokens of a few requests before the feed-forward block: latency
        {"name": "norm step", "kind": "norm", "rows": 7, "cols": HIDDEN, "residual": True,
         "columns": False, "y": False, "part": False},
        # a ragged batch of prompt chunks; the router reads y in BF16
        {"name": "norm prompts", "kind": "norm", "rows": 1777, "cols": HIDDEN, "residual": True,
         "columns": False, "y": True, "part": False},
        # training, the block step's tokens (4096 x 4): both MX copies
        {"name": "norm train", "kind": "norm", "rows": 16384, "cols": HIDDEN, "residual": True,
         "columns": True, "y": False, "part": False},
        # the latent vectors' norm, without residual, on columns of the [T, 576] projection
        {"name": "norm latent", "kind": "norm", "rows": 8190, "cols": 512, "residual": False,
         "columns": True, "y": False, "part": True},
        # the gradients of the last two
        {"name": "norm grad train", "kind": "norm grad", "rows": 16384, "cols": HIDDEN, "stream": True},
        {"name": "norm grad latent", "kind": "norm grad", "rows": 333, "cols": 512, "stream": False},
        # training, the routed experts' step: 8192 tokens x top-6 over 64 experts
        {"name": "experts grad", "kind": "ffn grad", "rows": 49152, "groups": 64, "ffn": EXPERT,
         "hidden": HIDDEN, "keep": False, "sums": False, "pick": 1},
        # one rank's share of the experts in a small step, products exact
        {"name": "experts grad few", "kind": "ffn grad", "rows": 1501, "groups": 8, "ffn": EXPERT,
         "hidden": HIDDEN, "keep": True, "sums": True, "pick": 2},
        # the dense feed-forward layer, one group
        {"name": "dense grad", "kind": "ffn grad", "rows": 2048, "groups": 1, "ffn": DENSE,
         "hidden": HIDDEN, "keep": False, "sums": False, "pick": 3},
        # decoding, the dense layer for one token: latency
        {"name": "ffn token", "kind": "ffn", "rows": 1, "groups": 1, "ffn": DENSE, "hidden": HIDDEN,
         "pick": 4},
        # decoding, the shared experts for a serving batch
        {"name": "ffn batch", "kind": "ffn", "rows": 48, "groups": 1, "ffn": 2 * EXPERT,
         "hidden": HIDDEN, "pick": 5},
        # decoding, 16 tokens x top-6 over 64 routed experts
        {"name": "ffn experts", "kind": "ffn", "rows": 96, "groups": 64, "ffn": EXPERT,
         "hidden": HIDDEN, "pick": 6},
    ]


def _log_int(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


#: What the largest listed cases hold: norm elements, gradient products, weights.
MOST_NORM = 16384 * HIDDEN
MOST_MACS = 49152 * EXPERT * HIDDEN
MOST_PADDED = 4 * 49152
MOST_WEIGHTS = 64 * EXPERT * HIDDEN


def draw(rng):
    kind = rng.choice(["norm", "norm", "norm grad", "ffn grad", "ffn", "ffn"])
    if kind in ("norm", "norm grad"):
        while True:
            rows, cols = _log_int(rng, 1, 32768), BLOCK * _log_int(rng, 2, 256)
            if rows * cols <= MOST_NORM:
                break
        if kind == "norm grad":
            return {"kind": kind, "rows": rows, "cols": cols, "stream": rng.random() < 0.6}
        return {"kind": kind, "rows": rows, "cols": cols, "residual": rng.random() < 0.6,
                "columns": rng.random() < 0.5, "y": rng.random() < 0.4, "part": rng.random() < 0.3}
    while True:
        c = {"kind": kind, "rows": _log_int(rng, 1, 49152 if kind == "ffn grad" else 256),
             "groups": rng.choice([1, 1, _log_int(rng, 2, 64)]), "ffn": BLOCK * _log_int(rng, 4, 342),
             "hidden": BLOCK * _log_int(rng, 8, 128)}
        if kind == "ffn grad":
            c["keep"], c["sums"] = rng.random() < 0.3, rng.random() < 0.3
        c["pick"] = rng.randrange(1 << 20)
        if c["groups"] * c["ffn"] * c["hidden"] > MOST_WEIGHTS:
            continue
        if c["rows"] * c["ffn"] * c["hidden"] * (2 if c.get("sums") else 1) > MOST_MACS:
            continue
        if c["rows"] * c["ffn"] <= 49152 * EXPERT and c["groups"] * max(_counts(c)) <= MOST_PADDED:
            return c


def _counts(case):
    """Rows of each group, from the case alone: uneven, some groups without a row."""
    r = random.Random("%d %d" % (case["pick"], case["groups"]))
    if case["groups"] == 1:
        return [case["rows"]]
    share = [0.0 if r.random() < 0.05 else math.exp(r.gauss(0, 0.5)) for _ in range(case["groups"])]
    share[r.randrange(len(share))] = 1.0
    got = [int(case["rows"] * s / sum(share)) for s in share]
    live = [i for i, s in enumerate(share) if s]
    while sum(got) < case["rows"]:
        got[r.choice(live)] += 1
    return got


def _capacity(rows, groups=None):
    """Columns of a column copy, as the library's callers allocate them."""
    need = rows + 31 * groups if groups else -(-rows // 32) * 32
    return -(-need // 128) * 128


def work(case):
    if case["kind"] == "norm":
        n = case["rows"] * case["cols"]
        mx = 1 + 1 / BLOCK
        b = 2 * n + 2 * case["cols"] + 4 * case["rows"] + mx * n
        b += 4 * n if case["residual"] else 0
        b += mx * n if case["columns"] else 0
        b += 2 * n if case["y"] else 0
        return {"bytes": b, "flops": 0}
    if case["kind"] == "norm grad":
        n = case["rows"] * case["cols"]
        return {"bytes": (8 if case["stream"] else 6) * n + 6 * case["cols"] + 4 * case["rows"], "flops": 0}
    m, f, h = case["rows"], case["ffn"], case["hidden"]
    mx = 1 + 1 / BLOCK
    live = sum(n > 0 for n in _counts(case))
    if case["kind"] == "ffn":
        return {"bytes": mx * (3 * live * f * h + m * h) + 2 * m * h, "flops": 6 * m * f * h}
    b = mx * (m * h + live * f * h) + 4 * m * f + 4 * mx * m * f + (4 * m * f if case["keep"] else 0)
    return {"bytes": b, "flops": 2 * m * f * h}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _normal(g, *shape, sigma=1.0):
    return (torch.randn(*shape, generator=g, device=g.device) * sigma).to(torch.bfloat16)


def _stream(g, rows, cols):
    """Rows of a residual stream: channels of different size, 0.5% of the values outliers."""
    x = torch.randn(rows, cols, generator=g, device=g.device)
    x *= torch.exp(0.5 * torch.randn(cols, generator=g, device=g.device))
    big = torch.rand(rows, cols, generator=g, device=g.device) < 0.005
    return torch.where(big, x * 20, x).to(torch.bfloat16)


def _offsets(lens):
    return torch.tensor([0] + lens, dtype=torch.int64, device="cuda").cumsum(0)


def _groups(s, case):
    """The groups' offsets, and the plans of the plain form: each group's rows padded to the
    longest (for products), and to whole blocks of 32 (for column copies)."""
    lens = _counts(case)
    n = torch.tensor(lens, device="cuda")
    s["offsets"] = _offsets(lens)
    first = s["offsets"][:-1]
    col = torch.arange(max(lens), device="cuda")
    s["pad"] = (first[:, None] + torch.minimum(col[None, :], (n[:, None] - 1).clamp_min(0))).clamp_max(
        case["rows"] - 1)
    group = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), n)
    at = torch.arange(case["rows"], device="cuda") - first[group]
    s["row"] = group * max(lens) + at
    blocks = _offsets([-(-x // BLOCK) * BLOCK for x in lens])
    s["padded_offsets"] = blocks
    s["column"] = blocks[group] + at                              # a row's column in the column copy


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    if case["kind"] in ("norm", "norm grad"):
        rows, cols = case["rows"], case["cols"]
        s["weight"] = (1 + 0.2 * torch.randn(cols, generator=g, device="cuda")).to(torch.bfloat16)
        if case["kind"] == "norm":
            wide = _stream(g, rows, cols + (64 if case["part"] else 0))
            s["x"] = wide[:, :cols]
            s["residual"] = _stream(g, rows, cols) if case["residual"] else None
            s["column"] = torch.arange(rows, device="cuda")
            return s
        s["total"] = _stream(g, rows, cols)
        s["rstd"] = _rstd(s["total"].float())
        s["dy"] = _normal(g, rows, cols, sigma=1e-3)
        s["dtotal"] = _normal(g, rows, cols, sigma=1e-3) if case["stream"] else None
        return s
    m, e, f, h = case["rows"], case["groups"], case["ffn"], case["hidden"]
    _groups(s, case)
    if case["kind"] == "ffn":
        s["x"] = _quantise(_normal(g, m, h))
        s["w_gu"] = _weight(g, e, 2 * f, h)
        s["w_down"] = _weight(g, e, h, f)
        return s
    s["dy"] = _quantise(_normal(g, m, h, sigma=1e-3))
    # the down weights' column copies [F, E H]: an expert's transposed weight is a column range
    codes, scales = _quantise(_normal(g, f, e * h, sigma=0.02))
    s["w_down"] = codes.view(f, e, h).transpose(0, 1), scales.view(f, e, h // BLOCK).transpose(0, 1)
    s["gu"] = _normal(g, m, 2 * f, sigma=0.9)                     # the forward's gate/up product
    return s


def _weight(g, groups, rows, cols):
    codes, scales = _quantise(_normal(g, groups * rows, cols, sigma=0.02))
    return codes.view(groups, rows, cols), scales.view(groups, rows, cols // BLOCK)


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _quantise(x):
    """E4M3 codes and E8M0 scales of rows, one scale per 32 values."""
    v = x.float().reshape(x.shape[0], -1, BLOCK)
    amax = v.abs().amax(-1)
    bad = ~torch.isfinite(amax)
    e = (torch.frexp(torch.where(bad | (amax == 0), torch.ones_like(amax), amax))[1] - 1 - 8).clamp_min(-127)
    e = torch.where(amax == 0, torch.full_like(e, -127), e)
    codes = (v * torch.exp2(-e.float())[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    codes = torch.where(bad[..., None], 0x7F, codes.view(torch.uint8))
    scales = torch.where(bad, 0xFF, e + 127).to(torch.uint8)
    return codes.to(torch.uint8).reshape(x.shape), scales


def _quantise_columns(x, column, capacity):
    """The column copy: rows of x at their columns of the transpose, zeros elsewhere."""
    t = x.new_zeros(capacity, x.shape[1])
    t[column] = x
    return _quantise(t.t())


def _values(codes, scales):
    """The 32-bit values that codes and scales stand for."""
    v = codes.view(torch.float8_e4m3fn).float()
    return (v.unflatten(-1, (-1, BLOCK)) * torch.exp2(scales.float() - 127)[..., None]).flatten(-2)


def _rstd(x):
    return 1 / torch.sqrt((x * x).mean(-1) + EPS)


def _norm_plain(s):
    case = s["case"]
    total = s["x"]
    if case["residual"]:
        total = (s["x"].float() + s["residual"].float()).to(torch.bfloat16)
    x = total.float()
    rstd = _rstd(x)
    y = x * rstd[:, None] * s["weight"].float()
    out = {"rstd": rstd, "row": _quantise(y)}
    if case["residual"]:
        out["total"] = total
    if case["y"]:
        out["y"] = y.to(torch.bfloat16)
    if case["columns"]:
        out["columns"] = _quantise_columns(y, s["column"], _capacity(case["rows"]))
    return out


def _norm_grad_plain(s):
    dy, xh = s["dy"].float(), s["total"].float() * s["rstd"][:, None]
    g = dy * s["weight"].float()
    dx = s["rstd"][:, None] * (g - xh * (g * xh).mean(-1, keepdim=True))
    if s["dtotal"] is not None:
        dx = dx + s["dtotal"].float()
    return {"dx": dx.to(torch.bfloat16), "dw": (dy * xh).sum(0)}


def _product(s, a, w):
    """Rows of a times the transposed weights w [E, N, K] of their group."""
    return torch.matmul(a[s["pad"]], w.transpose(1, 2)).flatten(0, 1)[s["row"]]


def _ffn_plain(s):
    f = s["case"]["ffn"]
    gu = _product(s, _values(*s["x"]), _values(*s["w_gu"]))
    h = gu[:, :f] / (1 + torch.exp(-gu[:, :f])) * gu[:, f:]
    return {"y": _product(s, _values(*_quantise(h)), _values(*s["w_down"])).to(torch.bfloat16)}


def _ffn_grad_plain(s):
    case = s["case"]
    f = case["ffn"]
    dh = _product(s, _values(*s["dy"]), _values(*s["w_down"]))
    g, u = s["gu"][:, :f].float(), s["gu"][:, f:].float()
    sig = 1 / (1 + torch.exp(-g))
    dgu = torch.cat([dh * u * sig * (1 + g * (1 - sig)), dh * g * sig], 1)
    out = {"row": _quantise(dgu), "offsets": s["padded_offsets"],
           "columns": _quantise_columns(dgu, s["column"], _capacity(case["rows"], case["groups"]))}
    if case["keep"]:
        out["dgu"] = dgu.to(torch.bfloat16)
    return out


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _read(pair):
    """Codes and scales as the values they stand for."""
    return {"codes": pair[0].view(torch.float8_e4m3fn), "scales": pair[1].view(torch.float8_e8m0fnu)}


def run(s):
    kind = s["case"]["kind"]
    if kind == "norm":
        out = _norm_own(s) if own else _norm_plain(s)
    elif kind == "norm grad":
        out = _norm_grad_own(s) if own else _norm_grad_plain(s)
    elif kind == "ffn":
        out = _ffn_own(s) if own else _ffn_plain(s)
    else:
        out = _ffn_grad_own(s) if own else _ffn_grad_plain(s)
    return {n: _read(v) if isinstance(v, tuple) else v for n, v in out.items()}


def _norm_own(s):
    from block_quant_gemm_amd import mxq
    case = s["case"]
    total, rstd, y, q, scale, qT, scaleT = mxq.mx_rms_norm(
        s["x"], s["weight"], residual=s["residual"], eps=EPS, y=case["y"], columns=case["columns"])
    out = {"rstd": rstd, "row": (q, scale)}
    if case["residual"]:
        out["total"] = total
    if case["y"]:
        out["y"] = y
    if case["columns"]:
        out["columns"] = qT, scaleT
    return out


def _norm_grad_own(s):
    from block_quant_gemm_amd import mxq
    dx, dw = mxq.mx_rms_norm_backward(s["dy"], s["total"], s["rstd"], s["weight"], dtotal=s["dtotal"])
    return {"dx": dx, "dw": dw}


def _ffn_own(s):
    from block_quant_gemm_amd import mxq
    return {"y": mxq.mx_gated_ffn_decode(*s["x"], *s["w_gu"], *s["w_down"], offsets=s["offsets"])}


def _ffn_grad_own(s):
    from block_quant_gemm_amd import mxq
    case = s["case"]
    dgu, q, scale, qT, scaleT, padded = mxq.mx_grouped_gemm_swiglu_backward(
        *s["dy"], *s["w_down"], s["gu"], s["offsets"], dgu=case["keep"],
        accum=mxq.ACC_FP32 if case["sums"] else mxq.ACC_MFMA_FP8)
    out = {"row": (q, scale), "offsets": padded, "columns": (qT, scaleT)}
    if case["keep"]:
        out["dgu"] = dgu
    return out


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

# Codes are given before their rounding, in units of the exact block's scale: that is what
# they stand for, and both sides' error is then the rounding to E4M3.  The scales themselves
# are powers of two that jump where a block's largest value crosses one, so that a value a
# rounding error away from there has the double or the half of another's: they have no value
# to be near to, and are judged through the codes.

def _exact_e4m3(x):
    """The E4M3 value nearest to each 64-bit value, ties to the even mantissa, at most 448."""
    a = x.abs()
    step = torch.exp2(torch.floor(torch.log2(a.clamp_min(2.0 ** -6))) - 3)
    return torch.sign(x) * (torch.round(a / step) * step).clamp_max(448.0)


def _exact_blocks(v):
    """(values in units of their block's scale, the scales) of 64-bit rows."""
    b = v.unflatten(-1, (-1, BLOCK))
    top = b.abs().amax(-1)
    e = torch.where(top > 0, torch.floor(torch.log2(top.clamp_min(1e-300))) - 8, -127.0).clamp_min(-127)
    scale = torch.exp2(e)
    return (b / scale[..., None]).flatten(-2), scale


def _exact_codes(v):
    return {"codes": _exact_blocks(v)[0], "scales": None}


def _exact_values(pair):
    """64-bit values of E4M3 codes under E8M0 scales, from their bit fields."""
    c = pair[0].long()
    field, mant = (c >> 3) & 15, (c & 7).double()
    v = torch.where(field == 0, mant * 2.0 ** -9, (8 + mant) * torch.exp2(field.double() - 10))
    v = torch.where(c > 127, -v, v)
    return v * torch.exp2(pair[1].double() - 127).repeat_interleave(BLOCK, -1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "norm":
        return _exact_norm(s)
    if case["kind"] == "norm grad":
        leaf, w = s["total"].double(), s["weight"].double()
        r = s["rstd"].double()[:, None]                # what the forward pass left
        dy = s["dy"].double()
        along = (dy * w * leaf).sum(1, keepdim=True)
        dx = r * dy * w - r ** 3 * leaf * along / leaf.shape[1]
        if s["dtotal"] is not None:
            dx = dx + s["dtotal"].double()
        return {"dx": dx, "dw": torch.matmul(torch.ones(1, dy.shape[0], dtype=dy.dtype, device="cuda"),
                                             dy * leaf * r)[0]}
    return _exact_ffn(s) if case["kind"] == "ffn" else _exact_ffn_grad(s)


def _exact_norm(s):
    case = s["case"]
    total = s["x"].double()
    if case["residual"]:
        total = total + s["residual"].double()
    out = {"total": total} if case["residual"] else {}
    x = total.to(torch.bfloat16).double()              # the norm is of the stream as it is stored
    out["rstd"] = (x.square().sum(1) / x.shape[1] + EPS).rsqrt()
    y = x * out["rstd"][:, None] * s["weight"].double()
    out["row"] = _exact_codes(y)
    if case["y"]:
        out["y"] = y
    if case["columns"]:
        t = torch.zeros(y.shape[1], _capacity(case["rows"]), dtype=y.dtype, device="cuda")
        t[:, :case["rows"]] = y.t()
        out["columns"] = _exact_codes(t)
    return out


def _exact_ffn(s):
    f = s["case"]["ffn"]
    x, at = _exact_values(s["x"]), s["offsets"].tolist()
    y = torch.zeros_like(x)
    for e in range(s["case"]["groups"]):
        if at[e] == at[e + 1]:
            continue
        gu = x[at[e]:at[e + 1]] @ _exact_values([t[e] for t in s["w_gu"]]).t()
        v, scale = _exact_blocks(gu[:, :f] * torch.sigmoid(gu[:, :f]) * gu[:, f:])
        h = _exact_e4m3(v) * scale.repeat_interleave(BLOCK, -1)
        y[at[e]:at[e + 1]] = h @ _exact_values([t[e] for t in s["w_down"]]).t()
    return {"y": y}


def _exact_ffn_grad(s):
    case = s["case"]
    f, at, to = case["ffn"], s["offsets"].tolist(), s["padded_offsets"].tolist()
    dgu = torch.zeros(case["rows"], 2 * f, dtype=torch.float64, device="cuda")
    t = torch.zeros(2 * f, _capacity(case["rows"], case["groups"]), dtype=torch.float64, device="cuda")
    for e in range(case["groups"]):
        n = at[e + 1] - at[e]
        if n == 0:
            continue
        rows = slice(at[e], at[e + 1])
        dh = _exact_values([v[rows] for v in s["dy"]]) @ _exact_values([v[e] for v in s["w_down"]]).t()
        g = s["gu"][rows, :f].double().requires_grad_()
        u = s["gu"][rows, f:].double().requires_grad_()
        dg, du = torch.autograd.grad(torch.nn.functional.silu(g) * u, [g, u], dh)
        dgu[rows, :f], dgu[rows, f:] = dg, du
        t[:, to[e]:to[e] + n] = dgu[rows].t()
    out = {"row": _exact_codes(dgu), "offsets": None, "columns": _exact_codes(t)}
    if case["keep"]:
        out["dgu"] = dgu
    return out
