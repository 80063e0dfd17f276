"""Refusals of the norm and feed-forward calls: the library's host-side checks, on fake
addresses that are never dereferenced, and the binding's.  CPU only."""

import pytest
import torch

from block_quant_gemm_amd import mxq
from tests.test_library import host_only_lib, lib  # noqa: F401  (fixtures)

P = 4096


def _call(lib, name, good, **change):
    args = dict(good)
    assert set(change) <= set(args)
    args.update(change)
    values = [v or 0 for v in args.values()]
    pack = STRUCTS.get(name)
    return getattr(lib, name)(*((pack.pack(*values), None) if pack else args.values()))


STRUCTS = {"mx_rms_norm": mxq._NORM_STRUCT, "mx_rms_norm_backward": mxq._NORM_GRAD_STRUCT,
           "mx_gated_ffn_decode": mxq._FFN_STRUCT}
NORM = dict(x=P, ldx=64, r=P, ldr=64, w=P, total=P, ldt=64, rstd=P, y=P, ldy=64, q=P, ldq=64, scale=P, lds=2,
            qT=P, ldqT=32, scaleT=P, ldsT=1, M=4, K=64, M_cap=32, eps=1e-6)
GRAD = dict(dy=P, lddy=64, total=P, ldt=64, rstd=P, w=P, dtotal=P, lddt=64, dx=P, lddx=64, dw=P, ws=P,
            ws_bytes=1 << 20, M=4, K=64)
SWIGLU = dict(dy=P, dys=P, ldd=64, ldsd=2, wT=P, wTs=P, ldw=64, ldsw=2, we=64 * 32, wse=64, offsets=P, E=2, M=40,
              F=32, K=64, gu=P, ldgu=64, dgu=P, lddgu=64, q=P, ldq=64, scale=P, lds=2, qT=P, ldqT=128, scaleT=P,
              ldsT=4, M_cap=128, poff=P, accum=0, stream=None)
FFN = dict(x=P, xs=P, ldx=64, ldsx=2, gu=P, gus=P, ldgu=64, ldsgu=2, gue=64 * 64, guse=128, d=P, dsc=P, ldd=32,
           ldsd=1, de=32 * 40, dse=40, offsets=P, y=P, ldy=40, ws=P, ws_bytes=1 << 20, M=4, K=64, F=32, N=40, E=2)


@pytest.mark.parametrize("change,status", [
    ({"M": -1}, 2), ({"K": 48}, 2), ({"K": 32768, "ldx": 32768}, 2), ({"M": 1 << 26}, 2), ({"eps": 0.0}, 4),
    ({"eps": -1.0}, 4), ({"eps": float("nan")}, 4), ({"eps": float("inf")}, 4), ({"x": None}, 1), ({"w": None}, 1),
    ({"rstd": None}, 1), ({"q": None}, 1), ({"scale": None}, 1), ({"total": None}, 1), ({"scaleT": None}, 1),
    ({"ldx": 60}, 2), ({"ldx": 68}, 3), ({"ldr": 68}, 3), ({"ldt": 32}, 2), ({"ldy": 68}, 3), ({"ldq": 72}, 3),
    ({"lds": 1}, 2), ({"M_cap": 0}, 2), ({"M_cap": 48}, 2), ({"M": 33}, 2), ({"ldqT": 40}, 3), ({"ldqT": 16}, 2),
    ({"ldsT": 0}, 2), ({"x": P + 8}, 3), ({"r": P + 2}, 3), ({"w": P + 2}, 3), ({"y": P + 8}, 3), ({"q": P + 8}, 3),
    ({"qT": P + 8}, 3), ({"rstd": P + 2}, 3), ({"K": 0}, 0), ({"M": 0, "qT": None}, 0)])
def test_norm(host_only_lib, change, status):  # noqa: F811
    assert _call(host_only_lib, "mx_rms_norm", NORM, **change) == status


@pytest.mark.parametrize("change,status", [
    ({"M": -1}, 2), ({"K": 40}, 2), ({"K": 16416}, 2), ({"dy": None}, 1), ({"total": None}, 1), ({"rstd": None}, 1),
    ({"w": None}, 1), ({"dx": None}, 1), ({"ws": None}, 1), ({"ws_bytes": 4 * 64 - 1}, 5), ({"ws": P + 8}, 3),
    ({"dw": P + 2}, 3), ({"lddy": 32}, 2), ({"ldt": 68}, 3), ({"lddt": 68}, 3), ({"lddx": 60}, 2), ({"dx": P + 8}, 3),
    ({"K": 0}, 0), ({"M": 0, "dw": None}, 0)])
def test_norm_gradient(host_only_lib, change, status):  # noqa: F811
    assert _call(host_only_lib, "mx_rms_norm_backward", GRAD, **change) == status


@pytest.mark.parametrize("change,status", [
    ({"M": -1}, 2), ({"F": 40}, 2), ({"K": 40}, 2), ({"M_cap": 96}, 2), ({"M_cap": 100}, 2), ({"E": 0}, 2),
    ({"E": 257}, 2), ({"accum": 2}, 4), ({"offsets": None}, 1), ({"dy": None}, 1), ({"wTs": None}, 1), ({"gu": None}, 1),
    ({"q": None}, 1), ({"scale": None}, 1), ({"qT": None}, 1), ({"scaleT": None}, 1), ({"ldd": 32}, 2),
    ({"ldd": 72}, 3), ({"ldw": 72}, 3), ({"we": 8}, 3), ({"we": -16}, 2), ({"ldgu": 32}, 2), ({"ldgu": 68}, 3),
    ({"lddgu": 60}, 2), ({"dgu": P + 2}, 3), ({"gu": P + 8}, 3), ({"ldq": 72}, 3), ({"lds": 1}, 2), ({"ldqT": 136}, 3),
    ({"ldqT": 64}, 2), ({"ldsT": 3}, 2), ({"q": P + 8}, 3), ({"qT": P + 8}, 3), ({"F": 0}, 0),
    ({"ldgu": 1 << 23}, 2), ({"ldq": 1 << 24}, 2), ({"ldqT": 1 << 32}, 2),
    ({"M": 1 << 39, "M_cap": 1 << 39, "ldqT": 1 << 39, "ldsT": 1 << 39, "E": 1}, 2)])
def test_swiglu_gradient(host_only_lib, change, status):  # noqa: F811
    assert _call(host_only_lib, "mx_grouped_gemm_swiglu_backward", SWIGLU, **change) == status


@pytest.mark.parametrize("change,status", [
    ({"M": -1}, 2), ({"K": 40}, 2), ({"F": 40}, 2), ({"E": 0}, 2), ({"E": 257}, 2), ({"offsets": None}, 2),
    ({"M": 1 << 21}, 2), ({"N": 1 << 21}, 2), ({"x": None}, 1), ({"gus": None}, 1), ({"d": None}, 1), ({"y": None}, 1),
    ({"ws": None}, 1), ({"ws_bytes": 4 * 33 - 1}, 5), ({"ws": P + 8}, 3), ({"ldx": 32}, 2), ({"ldx": 72}, 3),
    ({"ldsgu": 1}, 2), ({"ldd": 40}, 3), ({"gue": 8}, 3), ({"de": -16}, 2), ({"ldy": 39}, 2), ({"y": P + 1}, 3),
    ({"x": P + 8}, 3), ({"d": P + 8}, 3), ({"M": 0}, 0), ({"N": 0}, 0)])
def test_ffn_decode(host_only_lib, change, status):  # noqa: F811
    assert _call(host_only_lib, "mx_gated_ffn_decode", FFN, **change) == status


def test_no_struct(host_only_lib):  # noqa: F811
    for name in STRUCTS:
        assert getattr(host_only_lib, name)(None, None) == 1


def test_workspaces():
    assert mxq.workspace_size(mxq.WS_FFN_DECODE, 4, 32) == 4 * 33
    assert mxq.workspace_size(mxq.WS_FFN_DECODE, 0, 32) == 0
    assert mxq.workspace_size(mxq.WS_NORM_BACKWARD, 3, 2048) == 3 * 2048 * 4
    assert mxq.workspace_size(mxq.WS_NORM_BACKWARD, 0, 64) == 0
    big = mxq.workspace_size(mxq.WS_NORM_BACKWARD, 1 << 25, 16384)
    assert 0 < big <= 512 * 16384 * 4


def test_binding_refuses_what_the_library_cannot_see(monkeypatch):
    """Shapes, types and devices, before any address is passed on."""
    monkeypatch.setattr(mxq, "_current_gpu", lambda: -1)          # where CPU tensors say they are
    bf, u8 = torch.bfloat16, torch.uint8
    x, w = torch.zeros(4, 64, dtype=bf), torch.zeros(64, dtype=bf)
    with pytest.raises(TypeError):
        mxq.mx_rms_norm(x.float(), w)
    with pytest.raises(ValueError):
        mxq.mx_rms_norm(x, torch.zeros(32, dtype=bf))
    with pytest.raises(ValueError):
        mxq.mx_rms_norm(x, w, residual=torch.zeros(3, 64, dtype=bf))
    with pytest.raises(ValueError):
        mxq.mx_rms_norm(x, w, total=torch.zeros(4, 64, dtype=bf))
    with pytest.raises(ValueError):
        mxq.mx_rms_norm(x.t().contiguous().t(), w)
    with pytest.raises(ValueError):
        mxq.mx_rms_norm_backward(x, x, torch.zeros(5), w)
    with pytest.raises(ValueError):
        mxq.mx_rms_norm_backward(x, x, torch.zeros(4), w, dx=torch.zeros(4, 32, dtype=bf))
    q, s = torch.zeros(4, 64, dtype=u8), torch.zeros(4, 2, dtype=u8)
    wq, ws = torch.zeros(1, 32, 64, dtype=u8), torch.zeros(1, 32, 2, dtype=u8)
    gu, offs = torch.zeros(4, 64, dtype=bf), torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError):
        mxq.mx_grouped_gemm_swiglu_backward(q, s, wq, ws, gu[:3], offs)
    with pytest.raises(ValueError):
        mxq.mx_grouped_gemm_swiglu_backward(q, s, wq, ws[:, :, :1], gu, offs)
    with pytest.raises(TypeError):
        mxq.mx_grouped_gemm_swiglu_backward(q, s, wq, ws, gu, offs.int())
    wd, wds = torch.zeros(1, 8, 32, dtype=u8), torch.zeros(1, 8, 1, dtype=u8)
    with pytest.raises(ValueError):
        mxq.mx_gated_ffn_decode(q, s, torch.zeros(1, 62, 64, dtype=u8), ws, wd, wds)
    with pytest.raises(ValueError):
        mxq.mx_gated_ffn_decode(q, s, torch.zeros(1, 64, 64, dtype=u8), torch.zeros(1, 64, 2, dtype=u8),
                                torch.zeros(2, 8, 32, dtype=u8), torch.zeros(2, 8, 1, dtype=u8))
    monkeypatch.setattr(mxq, "_current_gpu", lambda: 1)
    with pytest.raises(ValueError, match="current GPU"):
        mxq.mx_rms_norm(x, w)
