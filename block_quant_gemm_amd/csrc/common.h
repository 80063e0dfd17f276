// Shared device helpers for the gfx950 kernels of libmxq.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mxq.h"

namespace mxq {

// Size arithmetic of the host-side checks on caller-supplied (non-negative)
// sizes: the product or sum, or INT64_MAX when it does not fit, so that a
// limit check on the result rejects it instead of overflowing.
inline int64_t sat_mul(int64_t a, int64_t b) {
  int64_t r;
  return __builtin_mul_overflow(a, b, &r) ? INT64_MAX : r;
}
inline int64_t sat_add(int64_t a, int64_t b) {
  int64_t r;
  return __builtin_add_overflow(a, b, &r) ? INT64_MAX : r;
}

// Largest scale of the logits: with it, scale * log2(e), the exponents' factor, is finite.
constexpr float kMaxScale = 2e38f;

// Tokens of a tile of the latent cache's absorbed attention.
#define MXQ_LATENT_TILE 64

// How mx_latent_decode splits its work: `rows` query rows a workgroup (the
// smallest of 16, 32 and 64 that holds a request's S * H rows, else 64 and as many
// row tiles), and along the batch's 64-token tiles runs of one length that stay
// inside a request.  With `runs` runs' worth of tiles there are at most
// runs + B runs: `grid` workgroups, and a workspace of one part each (512
// sums, a maximum and a total a row) and 8 bytes a request.  grid = 0: too large.
struct LatentDecodePlan {
  int rows;
  uint32_t row_tiles, runs, grid;
  int64_t part_rows;
  size_t bytes;
};
inline LatentDecodePlan latent_decode_plan(int64_t B, int64_t S, int64_t H, int64_t max_len) {
  LatentDecodePlan p{};
  if (B < 1 || S < 1 || H < 1 || max_len < 0 || sat_mul(S, H) > 65536) return p;
  p.rows = S * H <= 16 ? 16 : S * H <= 32 ? 32 : 64;
  p.row_tiles = (uint32_t)((S * H + p.rows - 1) / p.rows);
  const int64_t tiles = sat_mul(B, max_len > 0 ? sat_add(max_len, MXQ_LATENT_TILE - 1) / MXQ_LATENT_TILE : 1);
  if (tiles > 0x3FFFFFFFLL) return p;
  // workgroups of 16 rows have four wavefronts, two to a CU; the others have eight
  int64_t want = (p.rows == 16 ? 512 : 256) / (int64_t)p.row_tiles;
  if (want < 2) want = 2;
  const int64_t runs = want - B > want / 2 ? want - B : want / 2;
  p.runs = (uint32_t)runs;
  p.grid = (uint32_t)(runs + B < tiles ? runs + B : tiles);
  p.part_rows = (int64_t)p.grid * p.row_tiles * p.rows;
  if (p.part_rows > (INT64_C(1) << 40)) return LatentDecodePlan{};
  p.bytes = (size_t)p.part_rows * (MXQ_LATENT_DIM + 2) * sizeof(float) + (size_t)B * 8;
  return p;
}

// Parts along the keys that latent_attention gives a tile of 128 query rows: as
// many as fill two workgroups on each of 256 CUs, of 384 keys at least for a
// sequence of average length, and none below 1024 keys (a part's 6 tiles take about
// 8 us, joining the parts 5).  With parts and without: 16 queries after 4080 keys, 16 heads, 29 us and
// 103; 512 after 2488, 41 and 77; one sequence of 2000, 4 heads, 29 and 46.
constexpr int kPartKeys = 384;
inline int latent_forward_parts(int64_t Tq, int64_t Tk, int64_t H, int64_t B) {
  if (Tq < 1 || Tk < 1 || H < 1 || B < 1) return 1;
  // tiles: half of one more than full ones a sequence, one at least
  const int64_t half = Tq / 128 + B / 2 + B % 2, tiles = half > B ? half : B;
  const int64_t fill = 512 / sat_mul(tiles, H), keys = Tk / B < 1024 ? 1 : Tk / B / kPartKeys;
  const int64_t n = fill < keys ? fill : keys;
  return n < 1 ? 1 : n > 16 ? 16 : (int)n;
}
// One part's sums a row and head (128, with their reference and total), FP32.
inline size_t latent_forward_workspace(int64_t Tq, int64_t Tk, int64_t H, int64_t B) {
  const int n = latent_forward_parts(Tq, Tk, H, B);
  if (n == 1) return 0;
  const int64_t bytes = sat_mul(sat_mul(sat_mul(H, Tq), n), (MXQ_VALUE_DIM + 2) * (int64_t)sizeof(float));
  return bytes == INT64_MAX ? SIZE_MAX : (size_t)bytes;
}

// Rows that a workgroup of latent_attention_backward takes, of T query rows or of T key rows
// in B sequences: 64 where about that many workgroups, T / 64 and half a tile a
// sequence, still run at once, one a CU (one sequence of 360, 16 heads: 41 us for the three
// kernels against 59; 2 of 1000, 8 heads: 74 against 100), or, in one causal
// sequence, whose longest start first, in two turns (5000, 4 heads: 264 against 338;
// 2048, 16 heads: 149 against 164; 5400, 8 heads, more than that: 446 against 392).
// Else 128 (4 of 300, 16 heads: 56 against 60; 8 of 512: 138 against 152).  In calls of at
// most 512 rows and 64 sequences the half tiles are not counted: a second turn of short ones
// costs less than wavefronts past a sequence's end (forward and backward, 4 of 128, 32
// heads: 41 against 54; 64 of 8, 16 heads: 74 against 82).
inline int latent_backward_rows(int64_t T, int64_t H, int64_t B, bool causal) {
  const int64_t turn = causal && B == 1 ? 512 : 256;
  return sat_mul(T / 64 + (T > 512 || B > 64 ? B / 2 : 0), H) <= turn ? 64 : 128;
}

// Workspace of latent_attention_backward: the rotary key's gradient of each
// head, and D of each row, both FP32.  SIZE_MAX when it does not fit.
inline size_t latent_backward_workspace(int64_t Tq, int64_t Tk, int64_t H) {
  if (Tq < 0 || Tk < 0 || H < 1) return 0;
  const int64_t words = sat_add(sat_mul(sat_mul(H, Tk), MXQ_ROPE_DIM), sat_mul(H, Tq));
  return words > INT64_MAX / (int64_t)sizeof(float) ? SIZE_MAX : (size_t)words * sizeof(float);
}

typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef short i16x2 __attribute__((ext_vector_type(2)));

// a and b rounded to BF16 (nearest even) by one packed conversion, a in the
// low half.  Converting each value on its own costs a conversion per value
// plus a shift and an OR per pair.
__device__ __forceinline__ uint32_t bf16x2_bits(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){a, b}, bf16x2));
}

constexpr int kWave = 64;

// DPP quad permutations: exchange with lane^1 and lane^2 inside groups of 4.
constexpr int kQuadXor1 = 0xB1;  // quad_perm [1,0,3,2]
constexpr int kQuadXor2 = 0x4E;  // quad_perm [2,3,0,1]

__device__ __forceinline__ uint32_t dpp_u32(uint32_t v, int ctrl_xor1_or_2) {
  if (ctrl_xor1_or_2 == kQuadXor1)
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, kQuadXor1, 0xF, 0xF, false);
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, kQuadXor2, 0xF, 0xF, false);
}

// Inclusive sum over the lanes up to this one, all 64 lanes active: within rows
// of 16 by shifts, then rows 0 and 2 into 1 and 3, then the lower half into the
// upper.  Register moves only.
__device__ __forceinline__ uint32_t wave_scan(uint32_t x) {
  x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x111, 0xF, 0xF, true);   // row_shr 1
  x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x112, 0xF, 0xF, true);
  x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x114, 0xF, 0xF, true);
  x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x118, 0xF, 0xF, true);
  x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x142, 0xA, 0xF, false);  // row_bcast 15
  x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x143, 0xC, 0xF, false);  // row_bcast 31
  return x;
}
__device__ __forceinline__ uint32_t lane_u32(uint32_t x, int lane) {
  return (uint32_t)__builtin_amdgcn_readlane((int)x, lane);
}

// A run of products with their tile operands read DEPTH ahead: read(i) gives
// operand i, use(i, operand) multiplies it.  The scheduling barriers keep that
// order: left alone, the compiler reads each operand right before its use, and
// every product waits out the LDS latency.
template <int N, int DEPTH, class Read, class Use>
__device__ __forceinline__ void pipelined(Read read, Use use) {
  decltype(read(0)) f[N];
#pragma unroll
  for (int i = 0; i < DEPTH && i < N; ++i) f[i] = read(i);
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (i + DEPTH < N) f[i + DEPTH] = read(i + DEPTH);
    use(i, f[i]);
    __builtin_amdgcn_sched_barrier(0);
  }
}

// Packed max of the magnitudes of two BF16 values held in one dword.  The
// sign bits are cleared, so integer order equals magnitude order, and every
// NaN pattern (0x7F81..0x7FFF) compares above Inf (0x7F80) above all finite
// values: the maximum propagates NaN, then Inf.
__device__ __forceinline__ u16x2 absmax2(uint32_t a, uint32_t b) {
  u16x2 x = __builtin_bit_cast(u16x2, a & 0x7FFF7FFFu);
  u16x2 y = __builtin_bit_cast(u16x2, b & 0x7FFF7FFFu);
  return __builtin_elementwise_max(x, y);
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __builtin_bit_cast(float, w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __builtin_bit_cast(float, w & 0xFFFF0000u); }

// E8M0 scale code of an MX block from the largest BF16 magnitude pattern
// (sign cleared).  floor(log2(amax)) is the unbiased exponent field E - 127,
// so e = E - 127 - 8, clamped at -127: code = e + 127 = max(E - 8, 0).  BF16
// subnormals and zero (E == 0) give code 0; NaN/Inf give 0xFF.
__device__ __forceinline__ uint32_t mx_scale_code(uint32_t amax_bits) {
  uint32_t E = amax_bits >> 7;
  if (amax_bits >= 0x7F80u) return 0xFFu;
  return E > 8u ? E - 8u : 0u;
}

// 2^-e as FP32 for scale code c = e + 127 (c <= 253): exponent field 254 - c.
__device__ __forceinline__ float mx_inv_scale(uint32_t code) {
  return __builtin_bit_cast(float, (254u - code) << 23);
}

// Saturating round-to-nearest-even of two FP32 values to E4M3, packed into
// byte pair HI (false: bytes 0-1, true: bytes 2-3) of `old`.  The hardware
// conversion rounds to nearest even, including subnormals, but returns NaN
// instead of saturating at >= 464, so values are clamped to +-448 first.
template <bool HI>
__device__ __forceinline__ uint32_t cvt2_e4m3_sat(float a, float b, uint32_t old) {
  a = __builtin_amdgcn_fmed3f(a, -448.0f, 448.0f);
  b = __builtin_amdgcn_fmed3f(b, -448.0f, 448.0f);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(a, b, (int)old, HI);
}

// One MX block of 32 BF16 values held by a DPP quad, 8 per lane: the E8M0
// scale code from the block's largest magnitude (every lane of the quad gets
// it) and the lane's 8 E4M3 codes.
__device__ __forceinline__ void quant8(uint4 v, uint32_t& lo, uint32_t& hi, uint32_t& code) {
  u16x2 m = __builtin_elementwise_max(absmax2(v.x, v.y), absmax2(v.z, v.w));
  uint32_t am = m.x > m.y ? m.x : m.y;
  uint32_t o = dpp_u32(am, kQuadXor1);
  am = am > o ? am : o;
  o = dpp_u32(am, kQuadXor2);
  am = am > o ? am : o;
  code = mx_scale_code(am);
  if (code == 0xFFu) {                 // NaN or Inf in the block
    lo = hi = 0x7F7F7F7Fu;
    return;
  }
  float inv = mx_inv_scale(code);      // x * 2^-e is exact in FP32
  lo = cvt2_e4m3_sat<false>(bf16_lo(v.x) * inv, bf16_hi(v.x) * inv, 0u);
  lo = cvt2_e4m3_sat<true>(bf16_lo(v.y) * inv, bf16_hi(v.y) * inv, lo);
  hi = cvt2_e4m3_sat<false>(bf16_lo(v.z) * inv, bf16_hi(v.z) * inv, 0u);
  hi = cvt2_e4m3_sat<true>(bf16_lo(v.w) * inv, bf16_hi(v.w) * inv, hi);
}

// E8M0 code c as the FP32 scale operand of the scaled conversions, which
// take its exponent field: 2^(c - 127); 0xFF (a NaN block) turns every
// converted value into NaN.
__device__ __forceinline__ float e8m0_f32(uint32_t c) { return __builtin_bit_cast(float, c << 23); }

// Eight E4M3 codes (bytes of w0, then w1) times 2^(c - 127) as BF16, element
// i from byte i.  Exact while the product is a normal or subnormal BF16
// value with its bits intact: scale codes 3..246.  Under the others the product is
// rounded to nearest even, as the same product formed in FP32 is (all codes under all scales compared).
__device__ __forceinline__ bf16x8 widen8_bf16(uint32_t w0, uint32_t w1, float s) {
  typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
  const bf16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, s, false);
  const bf16x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, s, true);
  const bf16x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, s, false);
  const bf16x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, s, true);
  const bf16x4 lo = __builtin_shufflevector(p0, p1, 0, 1, 2, 3);
  const bf16x4 hi = __builtin_shufflevector(p2, p3, 0, 1, 2, 3);
  return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

// Which of 4 BF16 values are NaN or infinite: a bit each.
__device__ __forceinline__ uint32_t nonfinite4(uint2 x) {
  return ((x.x & 0x7F80u) == 0x7F80u ? 1u : 0u) | ((x.x & 0x7F800000u) == 0x7F800000u ? 2u : 0u) |
         ((x.y & 0x7F80u) == 0x7F80u ? 4u : 0u) | ((x.y & 0x7F800000u) == 0x7F800000u ? 8u : 0u);
}

// Sets the NaN and infinities among `bytes` bytes of BF16 values in LDS to 0, by `threads` threads.
__device__ __forceinline__ void clear_nonfinite(uint8_t* t, uint32_t bytes, uint32_t threads) {
#pragma unroll 1
  for (uint32_t i = threadIdx.x * 8; i < bytes; i += threads * 8) {
    uint2 x = *reinterpret_cast<const uint2*>(t + i);
    const uint32_t bits = nonfinite4(x);
    if (bits & 1) x.x &= 0xFFFF0000u;
    if (bits & 2) x.x &= 0xFFFFu;
    if (bits & 4) x.y &= 0xFFFF0000u;
    if (bits & 8) x.y &= 0xFFFFu;
    *reinterpret_cast<uint2*>(t + i) = x;
  }
}

// Buffer descriptor for gfx9: 48-bit base, stride 0, num_records bytes (range
// checked: loads at or past it read 0), data format word 0x00020000.
__device__ __forceinline__ i32x4 make_rsrc(const void* p, uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(p);
  i32x4 r;
  r[0] = (int)(uint32_t)a;
  r[1] = (int)((a >> 32) & 0xFFFFu);
  r[2] = (int)bytes;
  r[3] = 0x00020000;
  return r;
}

}  // namespace mxq
