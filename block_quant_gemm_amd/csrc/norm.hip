// Root-mean-square norm with the residual's addition and MX output, its
// gradient, and their C-ABI launchers.
//
//   s = BF16(x + r),  rstd = 1 / sqrt(mean_k s^2 + eps),  y = s rstd w
//   dx = rstd (dy w - s rstd c) + ds,  c = mean_k(dy w s rstd),  dw = sum_m dy s rstd
//
// Both are streams: every element is read and written once (the column copy
// of wide rows reads s again), so bytes bound them; under a few thousand rows the latency of one
// row's chain does (7 rows of 2048: 3.4 us), and below that the host's time of the call.

#include "common.h"

namespace mxq {

__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8]) {
  f[0] = bf16_lo(v.x); f[1] = bf16_hi(v.x); f[2] = bf16_lo(v.y); f[3] = bf16_hi(v.y);
  f[4] = bf16_lo(v.z); f[5] = bf16_hi(v.z); f[6] = bf16_lo(v.w); f[7] = bf16_hi(v.w);
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(bf16x2_bits(f[0], f[1]), bf16x2_bits(f[2], f[3]), bf16x2_bits(f[4], f[5]),
                    bf16x2_bits(f[6], f[7]));
}

// One MX block of 32 FP32 values held by a DPP quad, 8 a lane.
__device__ __forceinline__ uint2 quant8_f32(const float (&v)[8], uint32_t& code) {
  uint32_t am = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t m = __builtin_bit_cast(uint32_t, v[i]) & 0x7FFFFFFFu;
    am = am > m ? am : m;
  }
  uint32_t o = dpp_u32(am, kQuadXor1);
  am = am > o ? am : o;
  o = dpp_u32(am, kQuadXor2);
  am = am > o ? am : o;
  code = mx_code_of_bits(am);
  if (code == 0xFFu) return make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
  const float inv = mx_inv_scale(code);
  uint32_t lo = cvt2_e4m3_sat<false>(v[0] * inv, v[1] * inv, 0u);
  lo = cvt2_e4m3_sat<true>(v[2] * inv, v[3] * inv, lo);
  uint32_t hi = cvt2_e4m3_sat<false>(v[4] * inv, v[5] * inv, 0u);
  hi = cvt2_e4m3_sat<true>(v[6] * inv, v[7] * inv, hi);
  return make_uint2(lo, hi);
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int sh = 32; sh >= 1; sh >>= 1) v += __shfl_xor(v, sh, 64);
  return v;
}

// rstd of a row from its sum of squares.  The squares are summed in FP64, in
// which those of BF16 values are exact and neither overflow nor vanish.
__device__ __forceinline__ float rstd_of(double ss, uint32_t K, float eps) {
  return (float)(1.0 / __builtin_sqrt(ss / (double)K + (double)eps));
}

// y of 8 elements: two FP32 roundings, the same wherever it is formed.
__device__ __forceinline__ void normed8(uint4 s, float rstd, uint4 w, float (&y)[8]) {
  float a[8], b[8];
  unpack8(s, a);
  unpack8(w, b);
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = a[i] * rstd * b[i];
}

// A row is held by W wavefronts, CH chunks of 8 elements a lane, so it is read
// once.  Lane l of wavefront v holds elements 8 (64 (W c + v) + l) .. + 8 of
// chunk c.  Measured, 16384 x 2048 with a residual: 42 us for 235 MB (5.6 TB/s).
template <int W, int CH>
__global__ __launch_bounds__(W == 16 ? 1024 : 256) void k_norm_rows(mxq_norm g) {
  constexpr int ROWS = W >= 4 ? 1 : 4 / W;          // rows a workgroup
  __shared__ double s_part[W > 1 ? W : 1];
  const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
  const uint32_t v = W > 1 ? wave : 0u;
  const int64_t row = (int64_t)blockIdx.x * ROWS + (W > 1 ? 0 : wave);
  if (W == 1 && row >= g.M) return;
  uint32_t col[CH];
  uint4 s[CH];
  double ss = 0;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    col[c] = 8u * (64u * (W * c + v) + lane);
    s[c] = col[c] < g.K ? *reinterpret_cast<const uint4*>(g.x + row * g.ldx + col[c])
                        : make_uint4(0, 0, 0, 0);
  }
  if (g.residual) {
    uint4 r[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c)
      r[c] = col[c] < g.K ? *reinterpret_cast<const uint4*>(g.residual + row * g.ldr + col[c])
                          : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float a[8], b[8];
      unpack8(s[c], a);
      unpack8(r[c], b);
#pragma unroll
      for (int i = 0; i < 8; ++i) a[i] += b[i];
      s[c] = pack8(a);
      if (col[c] < g.K) *reinterpret_cast<uint4*>(g.total + row * g.ldt + col[c]) = s[c];
    }
  }
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    float a[8];
    unpack8(s[c], a);
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = __builtin_fma((double)a[i], (double)a[i], ss);
  }
  ss = wave_sum(ss);
  if (W > 1) {
    if (lane == 0) s_part[wave] = ss;
    __syncthreads();
    ss = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) ss += s_part[i];
  }
  const float rstd = rstd_of(ss, (uint32_t)g.K, g.eps);
  if (lane == 0 && v == 0) g.rstd[row] = rstd;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const bool ok = col[c] < g.K;
    const uint4 w = ok ? *reinterpret_cast<const uint4*>(g.weight + col[c]) : make_uint4(0, 0, 0, 0);
    float y[8];
    normed8(s[c], rstd, w, y);
    uint32_t code;
    const uint2 q = quant8_f32(y, code);            // all four lanes of a quad take part
    if (ok) {
      *reinterpret_cast<uint2*>(g.q + row * g.ldq + col[c]) = q;
      if ((lane & 3u) == 0u) g.scale[row * g.lds + (col[c] >> 5)] = (uint8_t)code;
      if (g.y) *reinterpret_cast<uint4*>(g.y + row * g.ldy + col[c]) = pack8(y);
    }
  }
}

// Both copies from one read, for rows of at most 512 CH columns (CH = 1, 2): a workgroup takes 32 rows,
// a block of the column copy, 4 a wavefront, in registers.  y goes through LDS 512
// columns at a time, from which a lane makes a column's block.  A block is 32 bytes of
// a column copy's row; the four that share a 128-byte line go to workgroups of one XCD, whose L2
// then has the line whole (workgroup 32 q + 8 r + x takes block 32 q + 4 x + r).
// Measured, 8190 x 512: 9.8 us; with a residual 12.9, and 17.8 as two kernels.
template <int CH>
__global__ __launch_bounds__(512, 4) void k_norm_dual(mxq_norm g) {
  constexpr int RW = 4, LD = 512 + 4;               // rows a wavefront; LDS row of floats
  __shared__ __attribute__((aligned(16))) float tile[32 * LD];
  const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
  uint32_t rb = blockIdx.x;
  if ((rb | 31u) < gridDim.x) rb = (rb & ~31u) | ((rb & 7u) << 2) | ((rb >> 3) & 3u);
  const int64_t m0 = (int64_t)rb * 32 + wave * RW;
  const uint32_t K = (uint32_t)g.K;
  uint4 s[RW][CH];
  float rstd[RW];
#pragma unroll
  for (int k = 0; k < RW; ++k)
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const uint32_t col = 512 * c + 8 * lane;
      s[k][c] = m0 + k < g.M && col < K ? *reinterpret_cast<const uint4*>(g.x + (m0 + k) * g.ldx + col)
                                        : make_uint4(0, 0, 0, 0);
    }
  if (g.residual) {
#pragma unroll
    for (int k = 0; k < RW; ++k) {
      uint4 r[CH];
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const uint32_t col = 512 * c + 8 * lane;
        r[c] = m0 + k < g.M && col < K
                   ? *reinterpret_cast<const uint4*>(g.residual + (m0 + k) * g.ldr + col)
                   : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const uint32_t col = 512 * c + 8 * lane;
        float a[8], b[8];
        unpack8(s[k][c], a);
        unpack8(r[c], b);
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] += b[i];
        s[k][c] = pack8(a);
        if (m0 + k < g.M && col < K)
          *reinterpret_cast<uint4*>(g.total + (m0 + k) * g.ldt + col) = s[k][c];
      }
    }
  }
#pragma unroll
  for (int k = 0; k < RW; ++k) {
    double ss = 0;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float a[8];
      unpack8(s[k][c], a);
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = __builtin_fma((double)a[i], (double)a[i], ss);
    }
    rstd[k] = rstd_of(wave_sum(ss), K, g.eps);
    if (lane == 0 && m0 + k < g.M) g.rstd[m0 + k] = rstd[k];
  }
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    if (512u * c >= K) break;                       // uniform
    const uint32_t col = 512 * c + 8 * lane;
    const bool in = col < K;
    uint4 w = in ? *reinterpret_cast<const uint4*>(g.weight + col) : make_uint4(0, 0, 0, 0);
    if (c) {
      plain_conversions();
      pin(w.x), pin(w.y), pin(w.z), pin(w.w);       // y is formed after it
      __syncthreads();                              // the columns before have been read
    }
#pragma unroll
    for (int k = 0; k < RW; ++k) {
      float y[8];
      normed8(s[k][c], rstd[k], w, y);
      const bool ok = m0 + k < g.M;
      uint32_t code;
      const uint2 q = quant8_f32(y, code);
      if (ok && in) {
        *reinterpret_cast<uint2*>(g.q + (m0 + k) * g.ldq + col) = q;
        if ((lane & 3u) == 0u) g.scale[(m0 + k) * g.lds + (col >> 5)] = (uint8_t)code;
        if (g.y) *reinterpret_cast<uint4*>(g.y + (m0 + k) * g.ldy + col) = pack8(y);
      }
      float* t = &tile[(wave * RW + k) * LD + 8 * lane];
      *reinterpret_cast<f32x4*>(t) = ok ? f32x4{y[0], y[1], y[2], y[3]} : f32x4{0, 0, 0, 0};
      *reinterpret_cast<f32x4*>(t + 4) = ok ? f32x4{y[4], y[5], y[6], y[7]} : f32x4{0, 0, 0, 0};
    }
    __syncthreads();
    saturate_conversions();                         // not over total and y
    const uint32_t kc = 512 * c + threadIdx.x;
    if (kc < K) {
      float v[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = tile[i * LD + threadIdx.x];
      uint32_t o[8];
      const uint32_t code = mx_block(v, o);
#pragma unroll
      for (int i = 0; i < 8; ++i) pin(o[i]);
      uint8_t* d = g.qT + kc * g.ldqT + (int64_t)rb * 32;
      *reinterpret_cast<uint4*>(d) = make_uint4(o[0], o[1], o[2], o[3]);
      *reinterpret_cast<uint4*>(d + 16) = make_uint4(o[4], o[5], o[6], o[7]);
      g.scaleT[kc * g.ldsT + rb] = (uint8_t)code;
    }
  }
}

// The column copy of wider rows: `width` columns of 128 rows a workgroup, 64 at a time: y, formed again from
// s and rstd, in LDS, each wavefront a block of 32 rows, a column a lane; the codes leave as
// 128-byte lines of the transpose.  The next columns' loads are under way meanwhile.
// Measured, 16384 x 2048: 20 us for 101 MB (5.0 TB/s; 3 us more without the loads ahead), after 42 us of
// k_norm_rows for 235 MB more (5.6).  One kernel for both with 32 whole rows a workgroup in registers took
// 73: it reads s once, but 8 wavefronts a CU are too few to load and store at once.
constexpr int kNcRows = 128, kNcCols = 64, kNcLd = kNcCols + 1;

__global__ __launch_bounds__(256) void k_norm_columns(mxq_norm g, uint32_t width) {
  __shared__ float tile[kNcRows * kNcLd];
  __shared__ __attribute__((aligned(16))) uint8_t outq[kNcCols * (kNcRows + 16)];
  __shared__ uint8_t outs[kNcCols * 4];
  saturate_conversions();
  const uint32_t K = (uint32_t)g.K, nk = (K + width - 1) / width;
  const int64_t p0 = (int64_t)(blockIdx.x / nk) * kNcRows;
  const uint32_t kw = blockIdx.x % nk * width;
  const uint16_t* s = g.residual ? g.total : g.x;
  const int64_t ld = g.residual ? g.ldt : g.ldx;
  const int tid = threadIdx.x, chunk = tid & 7;
  const uint16_t* src[4];
  float rstd[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int64_t row = p0 + u * 32 + (tid >> 3);
    src[u] = row < g.M ? s + row * ld : nullptr;
    rstd[u] = row < g.M ? g.rstd[row] : 0.0f;
  }
  uint4 v[4], w;
  auto load = [&](uint32_t k) {
    w = k < K ? *reinterpret_cast<const uint4*>(g.weight + k) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int u = 0; u < 4; ++u)
      v[u] = src[u] && k < K ? *reinterpret_cast<const uint4*>(src[u] + k) : make_uint4(0, 0, 0, 0);
  };
  load(kw + chunk * 8);
#pragma unroll 1
  for (uint32_t k0 = kw; k0 < kw + width && k0 < K; k0 += kNcCols) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      float y[8];
      normed8(v[u], rstd[u], w, y);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        tile[(u * 32 + (tid >> 3)) * kNcLd + chunk * 8 + e] = src[u] ? y[e] : 0.0f;
    }
    load(k0 + kNcCols + chunk * 8);                 // the next columns, while these are made
    __syncthreads();
    {
      const int c = tid & 63, b = tid >> 6;
      float f[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) f[i] = tile[(b * 32 + i) * kNcLd + c];
      uint32_t o[8];
      const uint32_t code = mx_block(f, o);
      uint4* oq = reinterpret_cast<uint4*>(&outq[c * (kNcRows + 16) + b * 32]);
      oq[0] = make_uint4(o[0], o[1], o[2], o[3]);
      oq[1] = make_uint4(o[4], o[5], o[6], o[7]);
      outs[c * 4 + b] = (uint8_t)code;
    }
    __syncthreads();
#pragma unroll
    for (int it = 0; it < 2; ++it) {
      const int cc = it * 32 + (tid >> 3), c16 = tid & 7;
      const int64_t p = p0 + c16 * 16;
      if (k0 + cc < K && p < g.M_cap)
        *reinterpret_cast<uint4*>(g.qT + (int64_t)(k0 + cc) * g.ldqT + p) =
            *reinterpret_cast<const uint4*>(&outq[cc * (kNcRows + 16) + c16 * 16]);
    }
    const int cc = tid >> 2, bb = tid & 3;
    if (k0 + cc < K && p0 + bb * 32 < g.M_cap)
      g.scaleT[(int64_t)(k0 + cc) * g.ldsT + (p0 >> 5) + bb] = outs[cc * 4 + bb];
  }
}

// Workgroup b takes rows b, b + grid, ...; a row is held as in k_norm_rows.
// dw's sums stay in registers over a wavefront's rows; the workgroup's wavefronts
// add theirs in order, and k_norm_join the workgroups', so the result
// does not depend on timing.  Measured, 16384 x 2048 with ds: 51 us for 268 MB
// (5.3 TB/s), then 4.8 us for the join of 512 sums.
template <int W, int CH>
__global__ __launch_bounds__(W == 16 ? 1024 : 256) void k_norm_grad(mxq_norm_grad g) {
  constexpr int ROWS = W >= 4 ? 1 : 4 / W;
  __shared__ float s_part[2][W > 1 ? W : 1];
  __shared__ float s_dw[W > 1 ? 1 : 512 * CH];
  const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
  const uint32_t v = W > 1 ? wave : 0u;
  uint32_t col[CH];
  uint4 w[CH];
  float acc[CH][8];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    col[c] = 8u * (64u * (W * c + v) + lane);
    w[c] = col[c] < g.K ? *reinterpret_cast<const uint4*>(g.weight + col[c]) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[c][i] = 0.0f;
  }
  // the widest rows have no registers for ds until dy's sums are made
  constexpr bool LATE = W == 16 && CH == 2;
  auto load_ds = [&](int64_t row, int c) {
    return col[c] < g.K && g.dtotal ? *reinterpret_cast<const uint4*>(g.dtotal + row * g.lddt + col[c])
                                    : make_uint4(0, 0, 0, 0);
  };
  int flip = 0;
  for (int64_t row = (int64_t)blockIdx.x * ROWS + (W > 1 ? 0 : wave); row < g.M;
       row += (int64_t)gridDim.x * ROWS) {
    uint4 dy[CH], s[CH], ds[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const bool ok = col[c] < g.K;
      dy[c] = ok ? *reinterpret_cast<const uint4*>(g.dy + row * g.lddy + col[c]) : make_uint4(0, 0, 0, 0);
      s[c] = ok ? *reinterpret_cast<const uint4*>(g.total + row * g.ldt + col[c]) : make_uint4(0, 0, 0, 0);
      if (!LATE) ds[c] = load_ds(row, c);
    }
    const float rstd = g.rstd[row];
    float along = 0.0f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float a[8], b[8], h[8];
      unpack8(dy[c], a);
      unpack8(s[c], b);
      unpack8(w[c], h);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float xh = b[i] * rstd;
        acc[c][i] = __builtin_fmaf(a[i], xh, acc[c][i]);
        along = __builtin_fmaf(a[i] * h[i], xh, along);
      }
    }
#pragma unroll
    for (int sh = 32; sh >= 1; sh >>= 1) along += __shfl_xor(along, sh, 64);
    if (W > 1) {
      // two buffers in turn: a wavefront writes a row's only after all have read the one before
      if (lane == 0) s_part[flip][wave] = along;
      __syncthreads();
      along = 0.0f;
#pragma unroll
      for (int i = 0; i < W; ++i) along += s_part[flip][i];
      flip ^= 1;
    }
    const float m = along / (float)g.K;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if (LATE) ds[c] = load_ds(row, c);
      float a[8], b[8], h[8], e[8];
      unpack8(dy[c], a);
      unpack8(s[c], b);
      unpack8(w[c], h);
      unpack8(ds[c], e);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        a[i] = __builtin_fmaf(rstd, __builtin_fmaf(-(b[i] * rstd), m, a[i] * h[i]), e[i]);
      if (col[c] < g.K) *reinterpret_cast<uint4*>(g.dx + row * g.lddx + col[c]) = pack8(a);
    }
  }
  if (!g.dw) return;
  float* out = static_cast<float*>(g.workspace) + (int64_t)blockIdx.x * g.K;
  if (W > 1) {
#pragma unroll
    for (int c = 0; c < CH; ++c)
      if (col[c] < g.K) {
        *reinterpret_cast<float4*>(out + col[c]) = make_float4(acc[c][0], acc[c][1], acc[c][2], acc[c][3]);
        *reinterpret_cast<float4*>(out + col[c] + 4) = make_float4(acc[c][4], acc[c][5], acc[c][6], acc[c][7]);
      }
  } else {
    for (uint32_t k = 0; k < 4; ++k) {
      if (wave == k) {
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float* p = &s_dw[col[c] + i];
            *p = k ? *p + acc[c][i] : acc[c][i];
          }
      }
      __syncthreads();
    }
    for (uint32_t k = threadIdx.x; k < g.K; k += blockDim.x) out[k] = s_dw[k];
  }
}

// dw from the workgroups' sums: 16 columns a workgroup, 16 threads a column,
// eight loads in flight each.
__global__ __launch_bounds__(256) void k_norm_join(const float* part, uint32_t parts, uint32_t K,
                                                   float* dw) {
  __shared__ float s[16][17];
  const uint32_t c = threadIdx.x & 15, t = threadIdx.x >> 4, k = blockIdx.x * 16 + c;
  float a = 0.0f;
  if (k < K)
    for (uint32_t p0 = t; p0 < parts; p0 += 128) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t p = p0 + 16 * i;
        v[i] = p < parts ? part[(int64_t)p * K + k] : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) a += v[i];
    }
  s[t][c] = a;
  __syncthreads();
  if (t == 0 && k < K) {
#pragma unroll
    for (int i = 1; i < 16; ++i) a += s[i][c];
    dw[k] = a;
  }
}

}  // namespace mxq

using namespace mxq;

static inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

constexpr int64_t kMaxStride = INT64_C(1) << 39;
// Rows a launch of k_norm_rows: a grid holds less than 2^32 threads, a row takes up to 1024 of them.
constexpr int64_t kRowsALaunch = INT64_C(1) << 21;

// A row operand of K BF16 values: NULL, stride and alignment.
static int check_rows(const void* p, int64_t ld, int64_t K) {
  if (!p) return MXQ_ERR_NULL;
  if (ld < K || ld > kMaxStride) return MXQ_ERR_SHAPE;
  return ld % 8 == 0 && aligned(p, 16) ? MXQ_OK : MXQ_ERR_ALIGN;
}

static int check_norm_size(int64_t M, int64_t K) {
  if (M < 0 || K < 0 || M > MXQ_NORM_MAX_ROWS || K > MXQ_NORM_MAX_COLS || K % 32 != 0)
    return MXQ_ERR_SHAPE;
  return MXQ_OK;
}

extern "C" int mx_rms_norm(const mxq_norm* norm, hipStream_t stream) {
  if (!norm) return MXQ_ERR_NULL;
  const mxq_norm& g = *norm;
  const int64_t M = g.M, K = g.K;
  int st = check_norm_size(M, K);
  if (st) return st;
  if (!(g.eps > 0.0f) || !(g.eps <= 3.4028235e38f)) return MXQ_ERR_ARG;
  if (g.qT) {
    if (g.M_cap < 0 || g.M_cap % 32 != 0 || g.M_cap < M || g.M_cap > 2 * (int64_t)MXQ_NORM_MAX_ROWS ||
        g.ldqT < g.M_cap || g.ldsT < g.M_cap / 32 || g.ldqT > kMaxStride || g.ldsT > kMaxStride)
      return MXQ_ERR_SHAPE;
    if (!g.scaleT) return MXQ_ERR_NULL;
    if (g.ldqT % 16 != 0 || !aligned(g.qT, 16)) return MXQ_ERR_ALIGN;
  }
  if (K == 0 || (M == 0 && (!g.qT || g.M_cap == 0))) return MXQ_OK;
  if (!g.weight) return MXQ_ERR_NULL;               // the column copy's kernels read it without rows too
  if (!aligned(g.weight, 16)) return MXQ_ERR_ALIGN;
  if (M > 0) {
    if ((st = check_rows(g.x, g.ldx, K))) return st;
    if (g.residual && (st = check_rows(g.residual, g.ldr, K))) return st;
    if (g.residual && (st = check_rows(g.total, g.ldt, K))) return st;
    if (g.y && (st = check_rows(g.y, g.ldy, K))) return st;
    if (!g.rstd || !g.q || !g.scale) return MXQ_ERR_NULL;
    if (g.ldq < K || g.lds < K / 32 || g.ldq > kMaxStride || g.lds > kMaxStride) return MXQ_ERR_SHAPE;
    if (!aligned(g.rstd, 4) || g.ldq % 16 != 0 || !aligned(g.q, 16)) return MXQ_ERR_ALIGN;
  }
  // one kernel for both copies, with a residual: 16384 x 512 19.5 us and 21.8 as two, 16384 x 1024 34.9
  // and 37.2, 3000 rows 9.5 and 9.5, 15.1 and 15.5; fewer rows take longer than as two (1024 rows 8.3 and
  // 7.8, 12.3 and 8.9; 256 rows 8.1 and 7.5, 11.5 and 7.2), for a launch less of the host's time
  if (g.qT && K <= 1024) {
    const dim3 grid((uint32_t)(g.M_cap / 32)), block(512);
    if (K <= 512) hipLaunchKernelGGL(k_norm_dual<1>, grid, block, 0, stream, g);
    else hipLaunchKernelGGL(k_norm_dual<2>, grid, block, 0, stream, g);
    return hipGetLastError() == hipSuccess ? MXQ_OK : MXQ_ERR_HIP;
  }
#define MXQ_ROWS(W, CH)                                                                        \
  hipLaunchKernelGGL((k_norm_rows<W, CH>), dim3((uint32_t)(W >= 4 ? r.M : (r.M + 3) / 4)),     \
                     dim3(W == 16 ? 1024 : 256), 0, stream, r)
  for (int64_t m = 0; m < M; m += kRowsALaunch) {
    mxq_norm r = g;
    r.M = M - m < kRowsALaunch ? M - m : kRowsALaunch;
    r.x += m * g.ldx;
    if (g.residual) r.residual += m * g.ldr, r.total += m * g.ldt;
    r.rstd += m;
    if (g.y) r.y += m * g.ldy;
    r.q += m * g.ldq;
    r.scale += m * g.lds;
    if (K <= 512) MXQ_ROWS(1, 1);
    // a wavefront a row once there are rows enough to fill the chip, a workgroup a row before (K = 2048:
    // 512 rows 6.0 us and 4.5, 1024 6.6 and 5.2, 2048 9.5 and 9.4, 4096 13.7 and 13.2, 16384 41.4 and
    // 44.0; K = 1056: 2048 rows 7.2 and 6.6, 4096 11.0 and 10.8, 16384 27.4 and 30.3; K = 544, where
    // one of the four chunks a lane is nearly full: 6.2 and 6.1, 8.8 and 9.8, 21.5 and 27.0)
    else if (K <= 2048 && M >= 2048) MXQ_ROWS(1, 4);
    else if (K <= 2048) MXQ_ROWS(4, 1);
    else if (K <= 4096) MXQ_ROWS(4, 2);
    else if (K <= 8192) MXQ_ROWS(4, 4);
    else MXQ_ROWS(16, 2);
    if (hipGetLastError() != hipSuccess) return MXQ_ERR_HIP;
  }
#undef MXQ_ROWS
  if (g.qT && g.M_cap > 0) {
    // up to 8 passes a workgroup, its loads a pass ahead, as long as two workgroups a CU remain
    const int64_t high = (g.M_cap + kNcRows - 1) / kNcRows, passes = high * (K / kNcCols + 1) / 512;
    const uint32_t width = kNcCols * (uint32_t)(passes < 1 ? 1 : passes > 8 ? 8 : passes);
    hipLaunchKernelGGL(k_norm_columns, dim3((uint32_t)(high * ((K + width - 1) / width))), dim3(256), 0,
                       stream, g, width);
    if (hipGetLastError() != hipSuccess) return MXQ_ERR_HIP;
  }
  return MXQ_OK;
}

extern "C" int mx_rms_norm_backward(const mxq_norm_grad* grad, hipStream_t stream) {
  if (!grad) return MXQ_ERR_NULL;
  const mxq_norm_grad& g = *grad;
  const int64_t M = g.M, K = g.K;
  int st = check_norm_size(M, K);
  if (st) return st;
  if (K == 0 || (M == 0 && !g.dw)) return MXQ_OK;
  if (M > 0) {
    if ((st = check_rows(g.dy, g.lddy, K))) return st;
    if ((st = check_rows(g.total, g.ldt, K))) return st;
    if (g.dtotal && (st = check_rows(g.dtotal, g.lddt, K))) return st;
    if ((st = check_rows(g.dx, g.lddx, K))) return st;
    if (!g.rstd || !g.weight) return MXQ_ERR_NULL;
    if (!aligned(g.rstd, 4) || !aligned(g.weight, 16)) return MXQ_ERR_ALIGN;
  }
  const uint32_t parts = norm_backward_parts(M, K);
  if (g.dw) {
    if (M > 0 && !g.workspace) return MXQ_ERR_NULL;
    if (!aligned(g.dw, 4) || !aligned(g.workspace, 16)) return MXQ_ERR_ALIGN;
    if (g.workspace_bytes < norm_backward_workspace(M, K)) return MXQ_ERR_WORKSPACE;
  }
#define MXQ_GRAD(W, CH)                                                                        \
  hipLaunchKernelGGL((k_norm_grad<W, CH>), dim3(parts), dim3(W == 16 ? 1024 : 256), 0, stream, g)
  if (M > 0) {
    if (K <= 512) MXQ_GRAD(1, 1);
    else if (K <= 2048) MXQ_GRAD(4, 1);
    else if (K <= 4096) MXQ_GRAD(4, 2);
    else if (K <= 8192) MXQ_GRAD(16, 1);
    else MXQ_GRAD(16, 2);
    if (hipGetLastError() != hipSuccess) return MXQ_ERR_HIP;
  }
#undef MXQ_GRAD
  if (g.dw) {
    hipLaunchKernelGGL(k_norm_join, dim3((uint32_t)((K + 15) / 16)), dim3(256), 0, stream,
                       static_cast<const float*>(g.workspace), M > 0 ? parts : 0u, (uint32_t)K, g.dw);
    if (hipGetLastError() != hipSuccess) return MXQ_ERR_HIP;
  }
  return MXQ_OK;
}
