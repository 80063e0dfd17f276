"""The latent attention calls as a program uses them: on two streams at once,
recorded into a HIP graph and replayed, and refused where a tensor has the wrong
type, shape, layout or device (an exception, nothing launched).  Also the
gradient against differences of the forward pass on the GPU."""

import numpy as np
import pytest
import torch

from block_quant_gemm_amd import mxq, workloads
from tests.gpu_helpers import say, to_dev_bf16

pytestmark = pytest.mark.gpu

SCALE = 192 ** -0.5


def _bf(shape, seed, name, sigma=1.0):
    return to_dev_bf16(workloads.bf16_normal(shape, sigma, seed=seed, name=name))


def _offsets(lens):
    return torch.from_numpy(workloads.offsets_from_counts(np.array(lens))).to("cuda")


def _inputs(seed, lens, H):
    T, B = sum(lens), len(lens)
    d = dict(tok=_bf((T, 576), seed, "utok"), q=_bf((T, H, 192), seed, "uq"),
             kv=_bf((T, H, 256), seed, "ukv"), do=_bf((T, H, 128), seed, "udo", 0.02),
             qa=_bf((B, 1, H, 576), seed, "uqa"), off=_offsets(lens), H=H, max_len=max(lens))
    page = 16
    per = -(-max(lens) // page)
    g = torch.Generator()
    g.manual_seed(seed)
    d["pages"] = torch.randperm(B * per, generator=g).view(B, per).to(torch.int32).cuda()
    at = [torch.arange(n) for n in lens]
    d["slots"] = torch.cat([d["pages"].cpu()[b, t // page].long() * page + t % page
                            for b, t in enumerate(at)]).cuda()
    d["lens"] = torch.tensor(lens, dtype=torch.int64, device="cuda")
    d["cache"] = mxq.latent_cache(B * per * page)
    d["page"] = page
    return d


def _chain(d):
    mxq.mx_latent_cache_write(d["tok"][:, :512], d["tok"][:, 512:], d["slots"], d["cache"])
    c, kr = mxq.mx_latent_cache_read(d["cache"], d["slots"])
    o, lse = mxq.mx_latent_decode(d["qa"], d["cache"], d["pages"], d["lens"], d["page"], d["max_len"], SCALE)
    args = (d["q"], d["kv"][..., :128], kr, d["kv"][..., 128:])
    eo, elsee = mxq.latent_attention(*args, offsets_q=d["off"])
    grads = mxq.latent_attention_backward(d["do"], *args, eo, elsee, offsets_q=d["off"])
    return [c, kr, o, lse, eo, elsee, *grads]


def _bits(ts):
    return [t.contiguous().clone().view(torch.uint8) for t in ts]


def test_two_streams_equal_each_alone():
    say("latent attention: two chains on two streams")
    d1, d2 = _inputs(1, [300, 1, 700, 65], 3), _inputs(2, [40, 1200], 8)
    ref1, ref2 = _bits(_chain(d1)), _bits(_chain(d2))
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for rep in range(3):
        with torch.cuda.stream(s1):
            out1 = _chain(d1)
        with torch.cuda.stream(s2):
            out2 = _chain(d2)
        torch.cuda.synchronize()
        for ref, out in ((ref1, out1), (ref2, out2)):
            for i, (a, b) in enumerate(zip(_bits(out), ref)):
                assert torch.equal(a, b), f"rep {rep}: output {i} differs"


def test_graph_replays_equal_eager():
    say("latent attention: graph capture and replays")
    d = _inputs(3, [200, 33, 1000], 4)
    eager = _bits(_chain(d))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        _chain(d)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = _chain(d)
    for r in range(4):
        for t in outs:
            t.fill_(7.0)
        for t in d["cache"]:
            t.fill_(1)
        junk = torch.randn(1 << 20, device="cuda").sum()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(_bits(outs), eager)):
            assert torch.equal(a, b), f"replay {r}: output {i} differs"
        del junk
    # lengths are read on the device: a replay follows them
    d["lens"].copy_(torch.tensor([7, 0, 999], device="cuda"))
    want = _bits(_chain(d)[2:4])
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    for a, b in zip(_bits(outs[2:4]), want):
        assert torch.equal(a, b)


def test_gradient_against_differences():
    """The loss sum(g * o) along each operand's own gradient, both sides.  The step
    moves no logit by more than about 0.16 (and v enters linearly), so what central
    differences leave out is of the order 0.16^2 / 6 of the slope; o's rounding to
    BF16 adds noise of at most sqrt(sum (g o)^2) * 2^-8 / sqrt(3) in each loss, of
    which six standard deviations are allowed, beside 5 %."""
    say("latent attention: gradient against differences")
    lens, H = [150, 90], 2
    T = sum(lens)
    q, kv = _bf((T, H, 192), 5, "gq"), _bf((T, H, 256), 5, "gkv")
    kr, g = _bf((T, 64), 5, "gkr"), _bf((T, H, 128), 5, "gg")
    how = dict(offsets_q=_offsets(lens), scale=SCALE)
    ops = [q, kv[..., :128].contiguous(), kr, kv[..., 128:].contiguous()]
    o, lse = mxq.latent_attention(*ops, **how)
    grads = mxq.latent_attention_backward(g, *ops, o, lse, **how)
    noise = float((g.double() * o.double()).norm()) * 2.0 ** -8 / 3 ** 0.5

    def loss(ts):
        return float((g.double() * mxq.latent_attention(*ts, **how)[0].double()).sum())

    for i, name in enumerate(("q", "k_nope", "k_rope", "v")):
        d = grads[i].double()
        # along the gradient, every entry of one size.  A row of two keys has a gradient
        # along their difference: its logits part by at most scale * 0.01 * sum |k1 - k2|,
        # about 192 * 1.13 * 0.01 / sqrt(192) = 0.16
        size = 0.5 if name == "v" else 0.01
        step = torch.sign(d) * size
        plus, minus = list(ops), list(ops)
        plus[i] = (ops[i].double() + step).to(torch.bfloat16)
        minus[i] = (ops[i].double() - step).to(torch.bfloat16)
        moved = plus[i].double() - minus[i].double()          # as rounded
        slope = float((d * moved).sum())
        diff = loss(plus) - loss(minus)
        assert slope > 40 * noise, f"{name}: the step is too small to tell"
        assert abs(diff - slope) < 0.05 * slope + 6 * 2 ** 0.5 * noise, (name, diff, slope)


def _args(name):
    T, H, B = 5, 2, 2
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")
    i64 = lambda *s: torch.zeros(s, dtype=torch.int64, device="cuda")
    cache = mxq.latent_cache(64)
    return {
        "write": (mxq.mx_latent_cache_write, dict(c=bf(T, 512), k_rope=bf(T, 64), slots=i64(T), cache=cache)),
        "read": (mxq.mx_latent_cache_read, dict(cache=cache, slots=i64(T), c=bf(T, 512), k_rope=bf(T, 64))),
        "decode": (mxq.mx_latent_decode,
                   dict(q=bf(B, 1, H, 576), cache=cache, pages=torch.zeros((B, 4), dtype=torch.int32, device="cuda"),
                        lens=i64(B), page_size=8, max_len=32, scale=0.1, o=bf(B, 1, H, 512),
                        lse=torch.zeros((B, 1, H), device="cuda"))),
        "forward": (mxq.latent_attention,
                    dict(q=bf(T, H, 192), k_nope=bf(T, H, 128), k_rope=bf(T, 64), v=bf(T, H, 128),
                         offsets_q=i64(3), offsets_k=i64(3), o=bf(T, H, 128), lse=torch.zeros((H, T), device="cuda"))),
        "backward": (mxq.latent_attention_backward,
                     dict(dout=bf(T, H, 128), q=bf(T, H, 192), k_nope=bf(T, H, 128), k_rope=bf(T, 64),
                          v=bf(T, H, 128), o=bf(T, H, 128), lse=torch.zeros((H, T), device="cuda"),
                          offsets_q=i64(3), offsets_k=i64(3), dq=bf(T, H, 192), dk_nope=bf(T, H, 128),
                          dk_rope=bf(T, 64), dv=bf(T, H, 128))),
    }[name]


@pytest.mark.parametrize("name", ["write", "read", "decode", "forward", "backward"])
def test_wrong_tensors_are_refused(name):
    say(f"latent attention refusals: {name}")
    fn, good = _args(name)
    fn(**good)
    torch.cuda.synchronize()
    for arg, t in good.items():
        parts = [t] if isinstance(t, torch.Tensor) else list(t) if isinstance(t, tuple) else []
        for i, x in enumerate(parts):
            def with_(y):
                v = y if isinstance(t, torch.Tensor) else tuple(y if j == i else z for j, z in enumerate(parts))
                return {**good, arg: v}
            with pytest.raises(TypeError):
                fn(**with_(x.to(torch.float64)))
            with pytest.raises(ValueError):
                fn(**with_(x.cpu()))                          # a host address
            with pytest.raises(ValueError):
                fn(**with_(x[:0] if name == "backward" or arg in ("lse", "pages") else x[..., :0]))
            if x.dim() > 1 and arg != "lse":
                with pytest.raises(ValueError):               # last dimension not contiguous
                    fn(**with_(x.transpose(-1, -2).contiguous().transpose(-1, -2)))
    for arg in ("scale", "max_len", "page_size"):
        if arg in good:
            with pytest.raises(mxq.MxqError):
                fn(**{**good, arg: 0 if arg != "max_len" else 33})
    if name in ("forward", "backward"):
        for bad in (0.0, -1.0, float("inf"), float("nan")):
            with pytest.raises(mxq.MxqError):
                fn(**good, scale=bad)
        with pytest.raises(mxq.MxqError):
            fn(**good, causal=2)
    if name in ("decode", "backward"):
        with pytest.raises(mxq.MxqError):
            fn(**good, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))
        with pytest.raises(ValueError):
            fn(**good, workspace=torch.zeros(1 << 24, dtype=torch.uint8))
