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
// Bound: the bytes where there are many (64 experts of 2048 x 1408, 96 rows over 56 of them: gate/up 79 us
// for 333 MB of weights, 4.2 TB/s, but L2 fetches 428 MB, 5.4 TB/s: two loads touch each 128-byte line, and
// some have left L2 by the second; down 35 us for 167 MB, 4.8 TB/s, fetched once), else the chain
// of offsets, weights and sums (one token, 2048 x 10944: gate/up 16 us for 46 MB, 61 fetched, down 6 us
// for 23 MB; a workgroup alone takes 7.6 us) and the rate at which a CU takes load instructions, some 50
// cycles each.  Weights through LDS, their scales through LDS or as dwords, 16 wavefronts for gate/up,
// and loads past the caches were all slower.
//
// Products are exact: codes are widened to BF16 with the block's scale folded in
// and multiplied on v_mfma_f32_16x16x32_bf16, which takes, per lane l, 8 values of row
// (token) l % 16.  Which k each lane's values are is free as long as both
// operands agree: here lane l holds block l / 16 of every four 32-blocks, so
// that it needs one scale a row and run of four.  The weights are the first operand: a
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

// Eight of a lane's 32 codes.
__device__ __forceinline__ bf16x8 widen_part(const uint4 (&v)[2], int p, float s) {
  const uint4 x = v[p >> 1];
  return p & 1 ? widen8_bf16(x.z, x.w, s) : widen8_bf16(x.x, x.y, s);
}

// Wavefront `wave` of nw takes blocks [first, last) of n: equal shares, whole runs.
__device__ __forceinline__ void share(uint32_t n, uint32_t wave, uint32_t nw, uint32_t run, uint32_t& first,
                                      uint32_t& last) {
  const uint32_t per = ((n + nw - 1) / nw + run - 1) / run * run;
  first = wave * per;
  last = first + per < n ? first + per : n;
}

// acc[i][t] += (weight rows of tile i) x (tokens of tile t) over blocks [first, last), which
// are this wavefront's, STEPS runs at a time.  SPAN = 1: lane l holds row l % 16 and block l / 16 of a run
// of four.  SPAN = 2, for at most 8 tokens: rows and tokens are l % 8, runs 8 blocks, of
// which lanes with bit 3 set hold the second four: of the instruction's 16 x 16 sums
// the two 8 x 8 on the diagonal count.
template <int R, int T, int STEPS, int SPAN>
__device__ __forceinline__ void rows_product(f32x4 (&acc)[R][T], const uint8_t* const (&w)[R],
                                             const uint8_t* const (&ws)[R],
                                             const uint8_t* const (&x)[T],
                                             const uint8_t* const (&xs)[T], uint32_t first,
                                             uint32_t last) {
  const uint32_t lane = threadIdx.x & 63u;
  const uint32_t mine = (lane >> 4) + (SPAN == 2 ? (lane >> 3 & 1) * 4 : 0);
#pragma unroll 1
  for (uint32_t b0 = first; b0 < last; b0 += 4 * SPAN * STEPS) {
    uint4 wv[STEPS][R][2];
    uint32_t wsc[STEPS][R], blk[STEPS];
    bool ok[STEPS];
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      blk[s] = b0 + 4 * SPAN * s + mine;
      ok[s] = blk[s] < last;
      if (!ok[s]) blk[s] = b0;                      // read anything valid; x's values become 0
#pragma unroll
      for (int i = 0; i < R; ++i) {
        wv[s][i][0] = *reinterpret_cast<const uint4*>(w[i] + blk[s] * 32u);
        wv[s][i][1] = *reinterpret_cast<const uint4*>(w[i] + blk[s] * 32u + 16);
        wsc[s][i] = ws[i][blk[s]];
      }
    }
#pragma unroll
    for (int t = 0; t < T; ++t) {
      uint4 xv[STEPS][2];
      uint32_t xc[STEPS];
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        xv[s][0] = *reinterpret_cast<const uint4*>(x[t] + blk[s] * 32u);
        xv[s][1] = *reinterpret_cast<const uint4*>(x[t] + blk[s] * 32u + 16);
        xc[s] = xs[t][blk[s]];
      }
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        if (!ok[s]) xv[s][0] = xv[s][1] = make_uint4(0, 0, 0, 0), xc[s] = 0;
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const bf16x8 b = widen_part(xv[s], p, e8m0_f32(xc[s]));
#pragma unroll
          for (int i = 0; i < R; ++i)
            acc[i][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                widen_part(wv[s][i], p, e8m0_f32(wsc[s][i])), b, acc[i][t], 0, 0, 0);
        }
      }
    }
  }
}

// Waits out the last product before its sums are read: the compiler leaves too few wait states between a
// matrix instruction at a loop's end and an LDS write of its result behind the loop, and the write
// took the sums without that product (rows of 36 to 48 blocks over 4 wavefronts: off by 27 %).
__device__ __forceinline__ void settle(f32x4& acc) { asm volatile("s_nop 15" : "+v"(acc)); }

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

// h = silu(a) u of row m, column f0 + c; the 32 lanes of half a wavefront hold one MX block.
__device__ __forceinline__ void gate_store(const FfnArgs& g, float a, float u, int64_t m, int64_t hi,
                                           int64_t f0, int c) {
  const float h = a * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(a * -1.4426950408889634f)) * u;
  float top = __builtin_fabsf(h);
#pragma unroll
  for (int sh = 16; sh >= 1; sh >>= 1)
    top = __builtin_elementwise_maximum(top, __shfl_xor(top, sh, 64));
  const uint32_t code = mx_code_of(top);
  // clamped by hand: with saturating conversions a NaN block's weights and tokens would be finite
  const uint32_t q = cvt2_e4m3_sat<false>(h * mx_inv_scale(code == 0xFFu ? 127u : code), 0.0f, 0u);
  if (m < hi) {
    g.hq[m * g.ldhq + f0 + c] = code == 0xFFu ? 0x7F : (uint8_t)q;
    if (c == 0) g.hs[m * g.ldhs + (f0 >> 5)] = (uint8_t)code;
  }
}

// Workgroups along z take a group's token tiles in turn.  T tiles of 16 tokens share a weight read;
// two runs of loads ahead (STEPS) as far as the registers go.
template <int T, int NW, int STEPS>
__global__ __launch_bounds__(NW * 64, T == 1 ? 4 : 2) void k_ffn_gate(FfnArgs g) {
  constexpr int LD = 68;                            // 64 rows and padding
  __shared__ float red[NW][16 * T][LD];
  int64_t lo, hi;
  group_rows(g.offsets, g.M, lo, hi);
  const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6, r = lane & 15u;
  const int64_t f0 = (int64_t)blockIdx.x * 32;
  const uint8_t *w[4], *ws[4], *x[T], *xs[T];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t row = (i >> 1) * g.F + f0 + (i & 1) * 16 + r;
    w[i] = g.w + blockIdx.y * g.w_estride + row * g.ldw;
    ws[i] = g.ws + blockIdx.y * g.ws_estride + row * g.ldws;
  }
  uint32_t first, last;
  share(g.nblk, __builtin_amdgcn_readfirstlane(wave), NW, 4, first, last);
  for (int64_t m0 = lo + (int64_t)blockIdx.z * 16 * T; m0 < hi; m0 += (int64_t)gridDim.z * 16 * T) {
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
    rows_product<4, T, STEPS, 1>(acc, w, ws, x, xs, first, last);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int t = 0; t < T; ++t) settle(acc[i][t]);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int t = 0; t < T; ++t)
        *reinterpret_cast<f32x4*>(&red[wave][t * 16 + r][i * 16 + (lane >> 4) * 4]) = acc[i][t];
    __syncthreads();
    for (int it = threadIdx.x; it < 512 * T; it += NW * 64) {
      const int tok = it >> 5, c = it & 31;
      float a = 0.0f, u = 0.0f;
#pragma unroll
      for (int v = 0; v < NW; ++v) {
        a += red[v][tok][c];
        u += red[v][tok][32 + c];
      }
      gate_store(g, a, u, m0 + tok, hi, f0, c);
    }
    __syncthreads();
  }
}

// Workgroups of 16 output columns, or 8 (SPAN = 2).
template <int T, int SPAN, int NW>
__global__ __launch_bounds__(NW * 64, NW == 16 ? 4 : 2) void k_ffn_down(FfnArgs g) {
  static_assert(SPAN == 1 || T == 1, "8 tokens at most");
  constexpr int ROWS = 16 / SPAN, LD = 20;          // 16 rows and padding
  __shared__ float red[NW][16 * T][LD];
  int64_t lo, hi;
  group_rows(g.offsets, g.M, lo, hi);
  const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6, r = lane & (ROWS - 1);
  const int64_t n0 = (int64_t)blockIdx.x * ROWS, row = n0 + r < g.N ? n0 + r : g.N - 1;
  const uint8_t* w[1] = {g.w + blockIdx.y * g.w_estride + row * g.ldw};
  const uint8_t* ws[1] = {g.ws + blockIdx.y * g.ws_estride + row * g.ldws};
  const uint8_t *x[T], *xs[T];
  uint32_t first, last;
  share(g.nblk, __builtin_amdgcn_readfirstlane(wave), NW, 4 * SPAN, first, last);
  for (int64_t m0 = lo + (int64_t)blockIdx.z * ROWS * T; m0 < hi; m0 += (int64_t)gridDim.z * ROWS * T) {
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
    rows_product<1, T, 3, SPAN>(acc, w, ws, x, xs, first, last);
#pragma unroll
    for (int t = 0; t < T; ++t) settle(acc[0][t]);
#pragma unroll
    for (int t = 0; t < T; ++t)
      *reinterpret_cast<f32x4*>(&red[wave][t * 16 + (lane & 15)][(lane >> 4) * 4]) = acc[0][t];
    __syncthreads();
    for (int it = threadIdx.x; it < ROWS * ROWS * T; it += NW * 64) {
      const int tok = it / ROWS, c = it % ROWS;
      float a = 0.0f;
#pragma unroll
      for (int v = 0; v < NW; ++v) {
        a += red[v][tok][c];
        if (SPAN == 2) a += red[v][8 + tok][8 + c];
      }
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
  // Tokens a workgroup: the fewest tiles of 16 with which the workgroups still run at once, one a
  // CU; where there are more anyway, as many as a group has on average, so that an average group's
  // weights are read once.  A larger group's tiles go one after another in the same workgroups (64 experts
  // of 2048 x 1408: all 96 rows on one 61 us, 64 rows on one and 32 experts with one 79).
  const int64_t per = E == 1 ? M : M / E;
  auto tiles = [&](int64_t units) {
    for (const int T : {1, 2})
      if (units * ((per + 16 * T - 1) / (16 * T)) <= 256 || per <= 16 * T) return T;
    return 4;
  };
  auto along_z = [&](int T) { return (uint32_t)(per <= 16 * T ? 1 : per >= 64 * 16 * T ? 64 : (per + 16 * T - 1) / (16 * T)); };
  if (F > 0) {
    const int T = tiles(F / 32 * E);
    const dim3 grid((uint32_t)(F / 32), (uint32_t)E, along_z(T));
#define MXQ_GATE(T, NW, STEPS)                                                                 \
  hipLaunchKernelGGL((k_ffn_gate<T, NW, STEPS>), grid, dim3(NW * 64), 0, stream, a)
    if (T == 1) MXQ_GATE(1, 8, 2);
    else if (T == 2) MXQ_GATE(2, 8, 2);
    else MXQ_GATE(4, 8, 1);
#undef MXQ_GATE
    if (hipGetLastError() != hipSuccess) return MXQ_ERR_HIP;
  }
  a.w = f.w_down; a.ws = f.w_down_scale; a.ldw = f.ldd; a.ldws = f.ldsd;
  a.w_estride = f.d_estride; a.ws_estride = f.ds_estride;
  a.nblk = (uint32_t)(F / 32);
  const int64_t units = (N + 15) / 16 * E;
  const int T = tiles(units);
  // eight columns a workgroup where sixteen would leave CUs without one (one token, 2048 x 10944:
  // 6.0 us and 9.4)
  const bool narrow = M <= 8 && units <= 256;
  const dim3 grid((uint32_t)(narrow ? (N + 7) / 8 : (N + 15) / 16), (uint32_t)E, along_z(T));
#define MXQ_DOWN(T, SPAN, NW)                                                                  \
  hipLaunchKernelGGL((k_ffn_down<T, SPAN, NW>), grid, dim3(NW * 64), 0, stream, a)
  // sixteen wavefronts for long rows only, where four would take many turns each (one token, F =
  // 10944: 6.1 us and 7.3, F = 8192: 7.0 and 6.7, F = 4096: 6.9 and 5.1; 48 tokens, F = 10944: 19.5 and
  // 21.6; 64 experts, F = 1408: 107 and 41)
  if (F > 8192) {
    if (narrow) MXQ_DOWN(1, 2, 16);
    else if (T == 1) MXQ_DOWN(1, 1, 16);
    else if (T == 2) MXQ_DOWN(2, 1, 16);
    else MXQ_DOWN(4, 1, 16);
  } else {
    if (narrow) MXQ_DOWN(1, 2, 4);
    else if (T == 1) MXQ_DOWN(1, 1, 4);
    else if (T == 2) MXQ_DOWN(2, 1, 4);
    else MXQ_DOWN(4, 1, 4);
  }
#undef MXQ_DOWN
  return hipGetLastError() == hipSuccess ? MXQ_OK : MXQ_ERR_HIP;
}
