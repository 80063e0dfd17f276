"""Both workgroup sizes of the gradient kernels on the cases where they can go wrong: every
case runs in a call that takes 64-row workgroups and in one that takes 128-row ones (asked
from the library), beside an ordinary sequence, and every output is compared with the
float64 oracle."""

import numpy as np
import pytest
import torch

from block_quant_gemm_amd import mxq
from oracle import codec, latent
from tests.gpu_helpers import say, to_dev, to_dev_bf16
from tests.test_gpu_latent_attention import CASES, SCALE, _bits, _compare, _device, _f64, _inputs, _run, _with_empty

pytestmark = pytest.mark.gpu

ROWS = [64, 128]
BESIDE = 150                                     # an ordinary sequence's rows


def _shape(d, rows):
    """The call's sequences, with empty ones after them where 128-row workgroups are wanted;
    fails if the library would take another size."""
    d = d if rows == 64 else _with_empty(d)
    for n in ("q", "kr"):
        assert mxq.latent_backward_rows(d[n].shape[0], d["q"].shape[1], len(d["oq"]) - 1) == rows, n
    return d


def _oracle(d, scale, causal):
    return latent.attention_backward(codec.bf16_bits_to_f64(d["do"]), *_f64(d), d["oq"], d["ok"], scale, causal)


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("case", range(len(CASES)))
def test_cases(case, rows):
    """lq and lk that differ, rows that see nothing, sequences without keys or queries."""
    lq, lk, H, causal = CASES[case]
    say(f"latent attention lq={lq} lk={lk} H={H} causal={causal}, {rows}-row workgroups")
    d = _shape(_inputs(lq + [BESIDE], lk + [BESIDE], H, 200 + case), rows)
    _compare(_run(d, causal), _oracle(d, SCALE, causal))


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("lq,lk", [([190, 33], [260, 33]), ([260], [190])])
@pytest.mark.parametrize("sigma,scale", [(12.0, 1.0), (1.0, 1e-4), (0.0, 1.0)])
def test_extreme_logits(sigma, scale, lq, lk, rows):
    say(f"latent attention sigma={sigma} scale={scale} lq={lq} lk={lk}, {rows}-row workgroups")
    d = _shape(_inputs(lq, lk, 2, 240, sigma), rows)
    _compare(_run(d, True, scale), _oracle(d, scale, True))


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("causal", [True, False])
def test_rising_logits(causal, rows):
    say(f"latent attention, rising logits, causal={causal}, {rows}-row workgroups")
    d = _inputs([320], [320], 1, 241)
    d["q"][:] = _bits((1, 1, 192), 3, "one")
    one = codec.bf16_bits_to_f64(d["q"][0, 0, :128])
    d["kv"][:, 0, :128] = codec.bf16_round_to_bits(np.arange(320)[:, None] * one[None] * 0.02)
    d = _shape(d, rows)
    _compare(_run(d, causal), _oracle(d, SCALE, causal))


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("causal", [True, False])
def test_strides(causal, rows):
    """Row and head strides of their own for every operand and result, lq and lk that differ;
    what lies between the rows stays."""
    say(f"latent attention, strided, causal={causal}, {rows}-row workgroups")
    lq, lk, H = [100, 61, 7], [161, 30, 0], 3
    d = _shape(_inputs(lq, lk, H, 242), rows)

    def wide(T, cols, bits=None):
        big = torch.full((T + 2, H + 1, cols + 24), 9.0, dtype=torch.bfloat16, device="cuda")
        v = big[1:T + 1, :H, 8:8 + cols]
        if bits is not None:
            v.copy_(to_dev_bf16(np.ascontiguousarray(bits)))
        return big, v

    Tq, Tk = sum(lq), sum(lk)
    q, do = wide(Tq, 192, d["q"])[1], wide(Tq, 128, d["do"])[1]
    kn, v = wide(Tk, 128, d["kv"][..., :128])[1], wide(Tk, 128, d["kv"][..., 128:])[1]
    kr = torch.full((Tk, 576), float("nan"), dtype=torch.bfloat16, device="cuda")[:, 512:]
    kr.copy_(to_dev_bf16(d["kr"]))
    lse = torch.full((H, Tq + 5), 4.0, device="cuda")
    how = dict(offsets_q=to_dev(d["oq"]), offsets_k=to_dev(d["ok"]), scale=SCALE, causal=causal)
    bo, o = wide(Tq, 128)
    mxq.latent_attention(q, kn, kr, v, **how, o=o, lse=lse[:, :Tq])
    bdq, dq = wide(Tq, 192)
    bdk, dkn = wide(Tk, 128)
    bdv, dv = wide(Tk, 128)
    bdr = torch.full((Tk, 72), 9.0, dtype=torch.bfloat16, device="cuda")
    mxq.latent_attention_backward(do, q, kn, kr, v, o, lse[:, :Tq], **how, dq=dq, dk_nope=dkn, dk_rope=bdr[:, :64], dv=dv)
    got = {"o": o, "lse": lse[:, :Tq], "dq": dq, "dk_nope": dkn, "dk_rope": bdr[:, :64], "dv": dv}
    _compare({n: x.contiguous() for n, x in got.items()}, _oracle(d, SCALE, causal))
    for big, view in ((bo, o), (bdq, dq), (bdk, dkn), (bdv, dv)):
        view.fill_(9.0)
        assert (big == 9.0).all()
    assert (lse[:, Tq:] == 4.0).all() and (bdr[:, 64:] == 9.0).all()


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("causal", [True, False])
def test_a_neighbours_nan_does_not_reach(causal, rows):
    say(f"latent attention, NaN in a neighbouring sequence, causal={causal}, {rows}-row workgroups")
    d = _inputs([40, 50, 130], [60, 50, 70], 2, 243)
    keep_q = np.r_[0:40, 90:220]
    keep_k = np.r_[0:60, 110:180]
    d["q"][40:90], d["do"][40:90], d["kv"][60:110], d["kr"][60:110] = 0x7FC0, 0x7FC0, 0x7FC0, 0x7FC0
    sound = {"q": d["q"][keep_q], "do": d["do"][keep_q], "kv": d["kv"][keep_k], "kr": d["kr"][keep_k],
             "oq": np.array([0, 40, 170]), "ok": np.array([0, 60, 130])}
    got = _run(_shape(d, rows), causal)
    kq, kk = torch.from_numpy(keep_q).cuda(), torch.from_numpy(keep_k).cuda()
    got = {n: (x[:, kq] if n == "lse" else x[kq] if n in ("o", "dq") else x[kk]).contiguous() for n, x in got.items()}
    _compare(got, _oracle(sound, SCALE, causal))


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("lq,lk", [([150], [260]), ([260], [150])])
@pytest.mark.parametrize("what", [0x7FC0, 0x7F80])
def test_hidden_nan_where_lengths_differ(what, lq, lk, rows):
    """The last rows are broken; the queries before them see only sound keys."""
    say(f"latent attention, last rows {what:#x}, lq={lq} lk={lk}, {rows}-row workgroups")
    d = _inputs(lq, lk, 2, 244)
    cut_q, cut_k = lq[0] - 57, lk[0] - 57
    sound = {"q": d["q"][:cut_q].copy(), "do": d["do"][:cut_q].copy(), "kv": d["kv"][:cut_k].copy(),
             "kr": d["kr"][:cut_k].copy(), "oq": np.array([0, cut_q]), "ok": np.array([0, cut_k])}
    for r in range(0, 57, 7):
        d["q"][cut_q + r, :, 3] = d["do"][cut_q + r, :, 9] = what
        d["kv"][cut_k + r, :, 5] = d["kv"][cut_k + r, :, 140] = d["kr"][cut_k + r, 7] = what
    got = _run(_shape(d, rows), True)
    ref = _oracle(sound, SCALE, True)
    _compare({n: got[n][:cut_q].contiguous() for n in ("o", "dq")}, {n: ref[n] for n in ("o", "dq")})
    _compare({"lse": got["lse"][:, :cut_q].contiguous()}, {"lse": ref["lse"]})
