"""The latent attention operators together, as a model's attention block has them.

A block with random weights (hidden 2048, latent 512, rotary key 64, heads of
128 + 64 query columns and 128 value columns), every Linear an MX product:

    train    forward and backward over packed sequences, with all gradients
    prefill  prompts of different lengths into the MX latent cache, page by page,
             in chunks: a chunk attends to what its sequence has cached before
    decode   new tokens, their latents written to the cache, absorbed attention

Absorbed and expanded attention are the same function: with W_uk, W_uv the
halves of the up projection, q . (W_uk c) = (W_uk^T q) . c and
sum p (W_uv c) = W_uv (sum p c).  So decode() multiplies W_uk into the queries
and W_uv into the result, both as grouped products with a group a head.

    python examples/latent_block.py          # on a GPU, after building
"""

import argparse
import os
import sys
import time

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from block_quant_gemm_amd import mxq

LATENT, ROPE, NOPE, VALUE = 512, 64, 128, 128


def rotate(x, positions):
    """Rotary embedding of the last dimension's halves, at each token's position."""
    half = x.shape[-1] // 2
    f = 10000.0 ** (-torch.arange(half, device=x.device, dtype=torch.float32) / half)
    a = positions.to(torch.float32)[:, None] * f
    a = a.view(a.shape[:1] + (1,) * (x.dim() - 2) + a.shape[1:])
    c, s, u, v = a.cos(), a.sin(), x[..., :half].float(), x[..., half:].float()
    return torch.cat([u * c - v * s, u * s + v * c], -1).to(x.dtype)


class Linear:
    """y = x W^T with both operands as MX blocks along the summed dimension.  The
    weight's two copies are made once."""

    def __init__(self, w):
        self.out, self.inp = w.shape
        rows = torch.tensor([0, self.out], dtype=torch.int64, device=w.device)
        self.w = mxq.mx_quantize_dual(w, rows)[:4]

    def forward(self, x):
        """(y, what backward() needs)"""
        one = torch.tensor([0, x.shape[0]], dtype=torch.int64, device=x.device)
        q, s, qT, sT, poff = mxq.mx_quantize_dual(x, one)
        return mxq.mx_gemm(q, s, self.w[0], self.w[1]), (qT, sT, poff, one)

    def __call__(self, x):
        return mxq.mx_gemm(*mxq.mx_quantize_rowwise(x), self.w[0], self.w[1])

    def backward(self, dy, kept):
        """(dx, dW)"""
        xT, xTs, poff, one = kept
        q, s, qT, sT, _ = mxq.mx_quantize_dual(dy, one)
        dx = mxq.mx_gemm(q, s, self.w[2][:, :self.out], self.w[3][:, :self.out // 32])
        return dx, mxq.mx_grouped_gemm_wgrad(qT, sT, xT, xTs, poff)[0]


class LatentBlock:
    def __init__(self, hidden=2048, heads=8, seed=0, device="cuda"):
        gen = torch.Generator(device=device)
        gen.manual_seed(seed)

        def draw(n, k):
            return (torch.randn((n, k), device=device, generator=gen) * k ** -0.5).to(torch.bfloat16)

        self.H, self.hidden = heads, hidden
        self.scale = (NOPE + ROPE) ** -0.5
        self.weights = {"q": draw(heads * (NOPE + ROPE), hidden), "kv_down": draw(LATENT + ROPE, hidden),
                        "kv_up": draw(heads * (NOPE + VALUE), LATENT), "o": draw(hidden, heads * VALUE)}
        self.lin = {n: Linear(w) for n, w in self.weights.items()}
        up = self.weights["kv_up"].view(heads, NOPE + VALUE, LATENT)
        # absorbed decoding: W_uk transposed [H, 512, 128] and W_uv [H, 128, 512]
        self.uk = self._stack(up[:, :NOPE].transpose(1, 2).contiguous())
        self.uv = self._stack(up[:, NOPE:].contiguous())

    @staticmethod
    def _stack(w):
        q, s = mxq.mx_quantize_rowwise(w.view(-1, w.shape[-1]))
        return q.view(w.shape), s.view(w.shape[0], w.shape[1], -1)

    def _per_head(self, x, w):
        """[T, H, K] times each head's [N, K]: [T, H, N]."""
        T, H, K = x.shape
        off = torch.arange(H + 1, dtype=torch.int64, device=x.device) * T
        q, s = mxq.mx_quantize_rowwise(x.transpose(0, 1).reshape(H * T, K))
        return mxq.mx_grouped_gemm(q, s, *w, off).view(H, T, -1).transpose(0, 1)

    def _queries(self, y, positions):
        q = y.view(-1, self.H, NOPE + ROPE).clone()
        q[..., NOPE:] = rotate(q[..., NOPE:], positions)
        return q

    def train(self, x, dy, offsets, positions):
        """Output and gradients of one step over packed sequences:
        (y, dx, {weight name: gradient})."""
        T = x.shape[0]
        yq, kq = self.lin["q"].forward(x)
        yd, kd = self.lin["kv_down"].forward(x)
        q = self._queries(yq, positions)
        kr = rotate(yd[:, LATENT:], positions)
        yu, ku = self.lin["kv_up"].forward(yd[:, :LATENT])
        kv = yu.view(T, self.H, NOPE + VALUE)
        how = dict(offsets_q=offsets, scale=self.scale)
        args = (q, kv[..., :NOPE], kr, kv[..., NOPE:])
        o, lse = mxq.latent_attention(*args, **how)
        y, ko = self.lin["o"].forward(o.view(T, -1))

        dw = {}
        do, dw["o"] = self.lin["o"].backward(dy, ko)
        dkv = torch.empty_like(kv)
        dq, _, dkr, _ = mxq.latent_attention_backward(do.view(T, self.H, VALUE), *args, o, lse, **how,
                                                      dk_nope=dkv[..., :NOPE], dv=dkv[..., NOPE:])
        dq[..., NOPE:] = rotate(dq[..., NOPE:], -positions)         # the rotation's transpose
        dc, dw["kv_up"] = self.lin["kv_up"].backward(dkv.view(T, -1), ku)
        dd = torch.cat([dc, rotate(dkr, -positions)], 1)
        dx, dw["kv_down"] = self.lin["kv_down"].backward(dd, kd)
        dxq, dw["q"] = self.lin["q"].backward(dq.view(T, -1), kq)
        return y, dx + dxq, dw

    def _cache_tokens(self, x, positions, slots, cache):
        d = self.lin["kv_down"](x)
        mxq.mx_latent_cache_write(d[:, :LATENT], rotate(d[:, LATENT:], positions), slots, cache)

    def prefill(self, x, positions, slots, offsets_q, all_slots, offsets_k, cache):
        """A chunk of each sequence: its tokens x (in slots `slots`) attend to all
        their sequence's tokens, which are in `all_slots`, the chunk's the last."""
        self._cache_tokens(x, positions, slots, cache)
        q = self._queries(self.lin["q"](x), positions)
        c, kr = mxq.mx_latent_cache_read(cache, all_slots)
        kv = self.lin["kv_up"](c).view(-1, self.H, NOPE + VALUE)
        o, _ = mxq.latent_attention(q, kv[..., :NOPE], kr, kv[..., NOPE:], offsets_q=offsets_q,
                                    offsets_k=offsets_k, scale=self.scale)
        return self.lin["o"](o.view(x.shape[0], -1))

    def decode(self, x, positions, slots, pages, lens, page_size, max_len, cache):
        """S new tokens of each of B requests, x [B * S, hidden]: cached, then
        attending to the lens[b] tokens the request has with them."""
        B = lens.shape[0]
        self._cache_tokens(x, positions, slots, cache)
        q = self._queries(self.lin["q"](x), positions)
        qa = torch.cat([self._per_head(q[..., :NOPE], self.uk), q[..., NOPE:]], -1)
        o, _ = mxq.mx_latent_decode(qa.view(B, -1, self.H, LATENT + ROPE), cache, pages, lens, page_size,
                                    max_len, self.scale)
        o = self._per_head(o.view(-1, self.H, LATENT), self.uv)
        return self.lin["o"](o.reshape(x.shape[0], -1))


class Pages:
    """Pages of a pool for B requests, drawn in a shuffled order."""

    def __init__(self, B, max_len, page_size, device="cuda", seed=0):
        self.size, per = page_size, -(-max_len // page_size)
        gen = torch.Generator()
        gen.manual_seed(seed)
        self.table = torch.randperm(B * per, generator=gen).view(B, per).to(torch.int32).to(device)
        self.slots_total = B * per * page_size

    def slots(self, b, t0, t1):
        t = torch.arange(t0, t1, device=self.table.device)
        return self.table[b, t // self.size].to(torch.int64) * self.size + t % self.size


def offsets_of(lens, device="cuda"):
    return torch.tensor([0, *torch.tensor(lens).cumsum(0).tolist()], dtype=torch.int64, device=device)


def serve(block, prompts, new, chunk=512, page_size=64, seed=1, device="cuda"):
    """Prefill of the prompts in chunks, then `new` decoding steps, on random token
    vectors.  Returns (x, outputs): each sequence's [length, hidden]."""
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    B, total = len(prompts), [n + new for n in prompts]
    x = [torch.randn((n, block.hidden), device=device, generator=gen).to(torch.bfloat16) for n in total]
    out = [torch.empty_like(t) for t in x]
    pages = Pages(B, max(total), page_size, device)
    cache = mxq.latent_cache(pages.slots_total, device)
    for t0 in range(0, max(prompts), chunk):
        part = [(b, t0, min(t0 + chunk, n)) for b, n in enumerate(prompts) if n > t0]
        slots = torch.cat([pages.slots(b, s, e) for b, s, e in part])
        every = torch.cat([pages.slots(b, 0, e) for b, _, e in part])
        pos = torch.cat([torch.arange(s, e, device=device) for _, s, e in part])
        y = block.prefill(torch.cat([x[b][s:e] for b, s, e in part]), pos, slots,
                          offsets_of([e - s for _, s, e in part], device), every,
                          offsets_of([e for _, _, e in part], device), cache)
        for (b, s, e), v in zip(part, y.split([e - s for _, s, e in part])):
            out[b][s:e] = v
    for i in range(new):
        at = [n + i for n in prompts]
        y = block.decode(torch.stack([x[b][t] for b, t in enumerate(at)]),
                         torch.tensor(at, device=device),
                         torch.cat([pages.slots(b, t, t + 1) for b, t in enumerate(at)]), pages.table,
                         torch.tensor([t + 1 for t in at], dtype=torch.int64, device=device), page_size,
                         max(at) + 1, cache)
        for b, t in enumerate(at):
            out[b][t] = y[b]
    return x, out


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--heads", type=int, default=8)
    ap.add_argument("--prompts", type=int, nargs="+", default=[700, 1, 77, 1500])
    ap.add_argument("--new", type=int, default=8)
    a = ap.parse_args()
    block = LatentBlock(heads=a.heads)

    lens = [1024, 300, 2048, 1]
    T = sum(lens)
    pos = torch.cat([torch.arange(n, device="cuda") for n in lens])
    x = torch.randn((T, block.hidden), device="cuda").to(torch.bfloat16)
    dy = torch.randn_like(x) * 1e-3
    block.train(x, dy, offsets_of(lens), pos)
    torch.cuda.synchronize()
    t = time.perf_counter()
    y, dx, dw = block.train(x, dy, offsets_of(lens), pos)
    torch.cuda.synchronize()
    print(f"train: {T} tokens in {len(lens)} sequences, {1e3 * (time.perf_counter() - t):.2f} ms; "
          f"gradients {', '.join(f'{n} {g.float().norm():.3g}' for n, g in dw.items())}", flush=True)

    xs, out = serve(block, a.prompts, a.new)
    lens = [len(v) for v in xs]
    pos = torch.cat([torch.arange(n, device="cuda") for n in lens])
    y = block.train(torch.cat(xs), torch.zeros_like(torch.cat(xs)), offsets_of(lens), pos)[0]
    for b, (o, r) in enumerate(zip(out, y.split(lens))):
        n = a.prompts[b]
        e = [(u.float() - v.float()).norm() / v.float().norm() for u, v in ((o[:n], r[:n]), (o[n:], r[n:]))]
        print(f"request {b}: {n} prompt tokens and {a.new} decoded, relative difference from one pass "
              f"without a cache {e[0]:.3f} and {e[1]:.3f}", flush=True)


if __name__ == "__main__":
    main()
