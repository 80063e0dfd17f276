"""The latent attention calls refuse a call one of whose tensors is on another GPU than the
current one, whichever tensor it is, before the library is called.  CPU only: tensors that
say where they are, and a library that must not be reached."""

import pytest
import torch

from block_quant_gemm_amd import mxq


class Tensor:
    """What the binding asks of a tensor."""

    def __init__(self, dtype, *shape, device=0):
        self.dtype, self.shape, self.index = dtype, torch.Size(shape), device
        self.is_cuda, self.device = True, torch.device("cuda", device)

    def get_device(self):
        return self.index

    def on(self, device):
        return Tensor(self.dtype, *self.shape, device=device)

    def stride(self, dim=None):
        s, n = [], 1
        for x in reversed(self.shape):
            s.append(n)
            n *= x
        return tuple(reversed(s)) if dim is None else s[::-1][dim]

    def numel(self):
        return self.shape.numel()

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096


class Reached(Exception):
    pass


BF, U8, I64, F32 = torch.bfloat16, torch.uint8, torch.int64, torch.float32
T, H, B = 5, 2, 3
WS = Tensor(U8, 1 << 30)
CACHE = (Tensor(U8, 64, 512), Tensor(U8, 64, 16), Tensor(BF, 64, 64))
ATTN = dict(q=Tensor(BF, T, H, 192), k_nope=Tensor(BF, T, H, 128), k_rope=Tensor(BF, T, 64), v=Tensor(BF, T, H, 128),
            offsets_q=Tensor(I64, 3), offsets_k=Tensor(I64, 3), o=Tensor(BF, T, H, 128), lse=Tensor(F32, H, T), workspace=WS)
CALLS = {
    "mx_latent_cache_write": dict(c=Tensor(BF, T, 512), k_rope=Tensor(BF, T, 64), slots=Tensor(I64, T), cache=CACHE),
    "mx_latent_cache_read": dict(cache=CACHE, slots=Tensor(I64, T), c=Tensor(BF, T, 512), k_rope=Tensor(BF, T, 64)),
    "mx_latent_decode": dict(q=Tensor(BF, B, 1, H, 576), cache=CACHE, pages=Tensor(torch.int32, B, 4), lens=Tensor(I64, B),
                             page_size=8, max_len=32, scale=0.1, o=Tensor(BF, B, 1, H, 512), lse=Tensor(F32, B, 1, H),
                             workspace=WS),
    "latent_attention": ATTN,
    "latent_attention_backward": dict(dout=Tensor(BF, T, H, 128), dq=Tensor(BF, T, H, 192), dk_nope=Tensor(BF, T, H, 128),
                                      dk_rope=Tensor(BF, T, 64), dv=Tensor(BF, T, H, 128), **ATTN),
}


@pytest.fixture
def library(monkeypatch):
    def load():
        raise Reached

    monkeypatch.setattr(mxq, "load", load)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0, raising=False)


@pytest.mark.parametrize("name", CALLS)
def test_a_tensor_on_another_gpu_is_refused(library, name):
    fn, good = getattr(mxq, name), CALLS[name]
    with pytest.raises(Reached):
        fn(**good)
    for arg, x in good.items():
        parts = x if isinstance(x, tuple) else (x,)
        for i, t in enumerate(parts):
            if isinstance(t, Tensor):
                moved = tuple(p.on(1) if j == i else p for j, p in enumerate(parts))
                with pytest.raises(ValueError, match="cuda:1"):
                    fn(**{**good, arg: moved if isinstance(x, tuple) else moved[0]})
