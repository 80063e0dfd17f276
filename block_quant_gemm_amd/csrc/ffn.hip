// The gated feed-forward block of few tokens, and its C-ABI launcher.
//
//   h = MX(silu(x Wg^T) (x Wu^T)),   y = h Wd^T      (per expert: its rows, its weights)
//
// Every weight byte meets at most a few dozen rows, so reading the weights is
// what it costs.  A workgroup takes 32 h columns (their 32 gate and 32 up rows:
// one MX block of h) or 16 output columns; its wavefronts split the contraction,
// each holding its weights in registers as they come from memory, and add their
// sums in LDS in a fixed order.
//
// Products are exact: codes are widened to BF16 with the block's scale folded in
// and multiplied on v_mfma_f32_16x16x32_bf16, which takes, per lane l, 8 values of row
// (token) l % 16.  Which k each lane's values are is free as long as both
// operands agree: here lane l holds block l / 16 of every four 32-blocks, so
// that it needs one scale byte a row and step.  The weights are the first operand: a
// lane's 4 sums are 4 consecutive weight rows of token l % 16.

#include "common.h"

namespace mxq {

struct FfnArgs {
  const uint8_t* x; const uint8_t* xs; int64_t ldx, ldxs;
  const uint8_t* w; const uint8_t* ws; int64_t ldw, ldws, w_estride, ws_estride;
  const int64_t* offsets;                           // or null: one group of all rows
  int64_t M;
  uint32_t nblk;                                    // blocks of 32 along the contraction
  int64_t F;                                        // gate/up: h columns
  uint8_t* hq; uint8_t* hs; int64_t ldhq, ldhs;
  uint16_t* y; int64_t ldy, N;                      // down: output [M, N]
};

__device__ __forceinline__ bf16x8 widen_half(uint4 v, int hi, float s) {
  return hi ? widen8_bf16(v.z, v.w, s) : widen8_bf16(v.x, v.y, s);
}

// acc[i][t] += (16 weight rows of tile i) x (16 tokens of tile t) over this
// wavefront's blocks: STEPS x 4 blocks at a time, every nw-th such run.
template <int R, int T, int STEPS>
__device__ __forceinline__ void rows_product(f32x4 (&acc)[R][T], const uint8_t* const (&w)[R],
                                             const uint8_t* const (&ws)[R],
                                             const uint8_t* const (&x)[T],
                                             const uint8_t* const (&xs)[T], uint32_t nblk,
                                             uint32_t wave, uint32_t nw) {
  const uint32_t quarter = (threadIdx.x & 63u) >> 4;
#pragma unroll 1
  for (uint32_t b0 = wave * 4 * STEPS; b0 < nblk; b0 += nw * 4 * STEPS) {
    uint4 wv[STEPS][R][2];
    uint32_t wsc[STEPS][R];
    uint32_t blk[STEPS];
    bool ok[STEPS];
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      blk[s] = b0 + 4 * s + quarter;
      ok[s] = blk[s] < nblk;
      if (!ok[s]) blk[s] = 0;                       // read anything valid; x's values become 0
#pragma unroll
      for (int i = 0; i < R; ++i) {
        wv[s][i][0] = *reinterpret_cast<const uint4*>(w[i] + blk[s] * 32u);
        wv[s][i][1] = *reinterpret_cast<const uint4*>(w[i] + blk[s] * 32u + 16);
        wsc[s][i] = ws[i][blk[s]];
      }
    }
#pragma unroll
    for (int t = 0; t < T; ++t) {
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        uint4 xv[2];
        xv[0] = *reinterpret_cast<const uint4*>(x[t] + blk[s] * 32u);
        xv[1] = *reinterpret_cast<const uint4*>(x[t] + blk[s] * 32u + 16);
        uint32_t xc = xs[t][blk[s]];
        if (!ok[s]) xv[0] = xv[1] = make_uint4(0, 0, 0, 0), xc = 0;
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const bf16x8 b = widen_half(xv[p >> 1], p & 1, e8m0_f32(xc));
#pragma unroll
          for (int i = 0; i < R; ++i)
            acc[i][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                widen_half(wv[s][i][p >> 1], p & 1, e8m0_f32(wsc[s][i])), b, acc[i][t], 0, 0, 0);
        }
      }
    }
  }
}

// The rows of this workgroup's group, clamped to the matrix.
__device__ __forceinline__ void group_rows(const int64_t* offsets, int64_t M, int64_t& lo, int64_t& hi) {
  lo = 0;
  hi = M;
  if (!offsets) return;
  lo = offsets[blockIdx.y];
  hi = offsets[blockIdx.y + 1];
  lo = lo < 0 ? 0 : lo;
  hi = hi > M ? M : hi;
}

constexpr int kGateWaves = 8;

template <int T>
__global__ __launch_bounds__(kGateWaves * 64, T == 1 ? 4 : 2) void k_ffn_gate(FfnArgs g) {
  constexpr int LD = 68;                            // 64 rows and padding
  __shared__ float red[kGateWaves][16 * T][LD];
  int64_t lo, hi;
  group_rows(g.offsets, g.M, lo, hi);
  if (lo >= hi) return;
  const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6, r = lane & 15u;
  const int64_t f0 = (int64_t)blockIdx.x * 32;
  const uint8_t *w[4], *ws[4], *x[T], *xs[T];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t row = (i >> 1) * g.F + f0 + (i & 1) * 16 + r;
    w[i] = g.w + blockIdx.y * g.w_estride + row * g.ldw;
    ws[i] = g.ws + blockIdx.y * g.ws_estride + row * g.ldws;
  }
  for (int64_t m0 = lo; m0 < hi; m0 += 16 * T) {
#pragma unroll
    for (int t = 0; t < T; ++t) {
      int64_t m = m0 + t * 16 + r;
      m = m < hi ? m : hi - 1;
      x[t] = g.x + m * g.ldx;
      xs[t] = g.xs + m * g.ldxs;
    }
    f32x4 acc[4][T];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int t = 0; t < T; ++t) acc[i][t] = f32x4{0, 0, 0, 0};
    rows_product<4, T, 2>(acc, w, ws, x, xs, g.nblk, wave, kGateWaves);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int t = 0; t < T; ++t)
        *reinterpret_cast<f32x4*>(&red[wave][t * 16 + r][i * 16 + (lane >> 4) * 4]) = acc[i][t];
    __syncthreads();
    // (token, h column) items: the 32 lanes of half a wavefront hold one MX block
#pragma unroll
    for (int k = 0; k < T; ++k) {
      const int tok = k * 16 + (threadIdx.x >> 5), c = threadIdx.x & 31;
      float a = 0.0f, u = 0.0f;
#pragma unroll
      for (int v = 0; v < kGateWaves; ++v) {
        a += red[v][tok][c];
        u += red[v][tok][32 + c];
      }
      const float h = a * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-a * 1.4426950408889634f)) * u;
      uint32_t am = __builtin_bit_cast(uint32_t, h) & 0x7FFFFFFFu;
#pragma unroll
      for (int sh = 16; sh >= 1; sh >>= 1) {
        const uint32_t o = (uint32_t)__shfl_xor((int)am, sh, 64);
        am = am > o ? am : o;
      }
      const uint32_t E = am >> 23;
      const uint32_t code = am >= 0x7F800000u ? 0xFFu : (E > 8u ? E - 8u : 0u);
      const float hv = h * mx_inv_scale(code == 0xFFu ? 127u : code);
      const uint32_t q = code == 0xFFu ? 0x7Fu : cvt2_e4m3_sat<false>(hv, 0.0f, 0u) & 0xFFu;
      const int64_t m = m0 + tok;
      if (m < hi) {
        g.hq[m * g.ldhq + f0 + c] = (uint8_t)q;
        if (c == 0) g.hs[m * g.ldhs + (f0 >> 5)] = (uint8_t)code;
      }
    }
    __syncthreads();
  }
}

template <int T, int NW>
__global__ __launch_bounds__(NW * 64, NW == 16 ? 4 : 2) void k_ffn_down(FfnArgs g) {
  constexpr int LD = 20;                            // 16 rows and padding
  __shared__ float red[NW][16 * T][LD];
  int64_t lo, hi;
  group_rows(g.offsets, g.M, lo, hi);
  if (lo >= hi) return;
  const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6, r = lane & 15u;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const uint8_t *w[1], *ws[1], *x[T], *xs[T];
  const int64_t row = n0 + r < g.N ? n0 + r : g.N - 1;
  w[0] = g.w + blockIdx.y * g.w_estride + row * g.ldw;
  ws[0] = g.ws + blockIdx.y * g.ws_estride + row * g.ldws;
  for (int64_t m0 = lo; m0 < hi; m0 += 16 * T) {
#pragma unroll
    for (int t = 0; t < T; ++t) {
      int64_t m = m0 + t * 16 + r;
      m = m < hi ? m : hi - 1;
      x[t] = g.hq + m * g.ldhq;
      xs[t] = g.hs + m * g.ldhs;
    }
    f32x4 acc[1][T];
#pragma unroll
    for (int t = 0; t < T; ++t) acc[0][t] = f32x4{0, 0, 0, 0};
    rows_product<1, T, 4>(acc, w, ws, x, xs, g.nblk, wave, NW);
#pragma unroll
    for (int t = 0; t < T; ++t)
      *reinterpret_cast<f32x4*>(&red[wave][t * 16 + r][(lane >> 4) * 4]) = acc[0][t];
    __syncthreads();
    for (int it = threadIdx.x; it < 256 * T; it += NW * 64) {
      const int tok = it >> 4, c = it & 15;
      float a = 0.0f;
#pragma unroll
      for (int v = 0; v < NW; ++v) a += red[v][tok][c];
      if (m0 + tok < hi && n0 + c < g.N)
        g.y[(m0 + tok) * g.ldy + n0 + c] = (uint16_t)bf16x2_bits(a, 0.0f);
    }
    __syncthreads();
  }
}

}  // namespace mxq

using namespace mxq;

static inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

constexpr int64_t kMaxStride = int64_t(1) << 39;

// Codes [rows, K] and their scales.
static int check_codes(const uint8_t* q, const uint8_t* s, int64_t ld, int64_t lds, int64_t K) {
  if (!q || !s) return MXQ_ERR_NULL;
  if (ld < K || lds < K / 32 || ld > kMaxStride || lds > kMaxStride) return MXQ_ERR_SHAPE;
  return ld % 16 == 0 && aligned(q, 16) ? MXQ_OK : MXQ_ERR_ALIGN;
}

extern "C" int mx_gated_ffn_decode(const mxq_ffn_decode* ffn, hipStream_t stream) {
  if (!ffn) return MXQ_ERR_NULL;
  const mxq_ffn_decode& f = *ffn;
  const int64_t M = f.M, K = f.K, F = f.F, N = f.N;
  const int32_t E = f.E;
  if (M < 0 || K < 0 || F < 0 || N < 0 || M > MXQ_FFN_DECODE_MAX_ROWS ||
      K > MXQ_FFN_DECODE_MAX_DIM || F > MXQ_FFN_DECODE_MAX_DIM || N > MXQ_FFN_DECODE_MAX_DIM)
    return MXQ_ERR_SHAPE;
  if (f.offsets ? E < 1 || E > 256 : E != 1) return MXQ_ERR_SHAPE;
  if (K % 32 != 0 || F % 32 != 0) return MXQ_ERR_SHAPE;
  if (M == 0 || N == 0) return MXQ_OK;
  int st;
  if (K > 0 && F > 0) {
    if ((st = check_codes(f.x, f.x_scale, f.ldx, f.ldsx, K))) return st;
    if ((st = check_codes(f.w_gu, f.w_gu_scale, f.ldgu, f.ldsgu, K))) return st;
  }
  if (F > 0 && (st = check_codes(f.w_down, f.w_down_scale, f.ldd, f.ldsd, F))) return st;
  if (!f.y) return MXQ_ERR_NULL;
  if (f.ldy < N || f.ldy > kMaxStride) return MXQ_ERR_SHAPE;
  if (!aligned(f.y, 2)) return MXQ_ERR_ALIGN;
  for (const int64_t s : {f.gu_estride, f.gus_estride, f.d_estride, f.ds_estride})
    if (s < 0 || s > kMaxStride) return MXQ_ERR_SHAPE;
  if (f.gu_estride % 16 != 0 || f.d_estride % 16 != 0) return MXQ_ERR_ALIGN;
  if (F > 0 && !f.workspace) return MXQ_ERR_NULL;
  if (!aligned(f.workspace, 16)) return MXQ_ERR_ALIGN;
  if (f.workspace_bytes < ffn_decode_workspace(M, F)) return MXQ_ERR_WORKSPACE;
  uint8_t* hq = static_cast<uint8_t*>(f.workspace);
  FfnArgs a{f.x, f.x_scale, f.ldx, f.ldsx, f.w_gu, f.w_gu_scale, f.ldgu, f.ldsgu, f.gu_estride,
            f.gus_estride, f.offsets, M, (uint32_t)(K / 32), F, hq, hq + M * F, F, F / 32, f.y,
            f.ldy, N};
  const int64_t per = M / E;
  const int T = E == 1 ? (M <= 16 ? 1 : M <= 32 ? 2 : 4) : (per <= 8 ? 1 : per <= 16 ? 2 : 4);
  if (F > 0) {
    const dim3 grid((uint32_t)(F / 32), (uint32_t)E), block(kGateWaves * 64);
    if (T == 1) hipLaunchKernelGGL(k_ffn_gate<1>, grid, block, 0, stream, a);
    else if (T == 2) hipLaunchKernelGGL(k_ffn_gate<2>, grid, block, 0, stream, a);
    else hipLaunchKernelGGL(k_ffn_gate<4>, grid, block, 0, stream, a);
    if (hipGetLastError() != hipSuccess) return MXQ_ERR_HIP;
  }
  a.w = f.w_down; a.ws = f.w_down_scale; a.ldw = f.ldd; a.ldws = f.ldsd;
  a.w_estride = f.d_estride; a.ws_estride = f.ds_estride;
  a.nblk = (uint32_t)(F / 32);
  const dim3 grid((uint32_t)((N + 15) / 16), (uint32_t)E);
#define MXQ_DOWN(T, NW) hipLaunchKernelGGL((k_ffn_down<T, NW>), grid, dim3(NW * 64), 0, stream, a)
  if (F > 2048) {
    if (T == 1) MXQ_DOWN(1, 16); else if (T == 2) MXQ_DOWN(2, 16); else MXQ_DOWN(4, 16);
  } else {
    if (T == 1) MXQ_DOWN(1, 4); else if (T == 2) MXQ_DOWN(2, 4); else MXQ_DOWN(4, 4);
  }
#undef MXQ_DOWN
  return hipGetLastError() == hipSuccess ? MXQ_OK : MXQ_ERR_HIP;
}
