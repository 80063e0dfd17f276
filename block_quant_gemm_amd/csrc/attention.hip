// Expanded latent attention for gfx950: softmax attention over sequences packed
// row by row, forward and backward, whose keys are a per-head part (128 columns)
// beside a rotary part (64 columns) that all heads share.  BF16 operands on the
// BF16 matrix instruction, FP32 sums and softmax statistics.
//
// With z = scale * (q . k) over the visible keys of a row:
//   m = max z,  l = sum exp(z - m),  o = sum exp(z - m) v / l,  lse = m + ln l
//   P = exp(z - lse),  dP = dO V^T,  D = rowsum(dO * o) = rowsum(P * dP)
//   dS = P * (dP - D),  dQ = scale * dS K,  dK = scale * dS^T Q,  dV = P^T dO
//
// One shape serves the three kernels.  Each wavefront keeps the rows of its
// own side in registers (queries in the forward and dQ kernels, keys in the
// dK/dV kernel) and walks the other side in tiles of 64 rows that the whole
// workgroup stages in LDS.  The logits are formed transposed, with the
// wavefront's own row along the lanes, so a row's maximum and sum are a
// reduction over registers and one exchange between the two lane halves, and
// the probabilities are already in the operand layout of the second product:
// the matrix instruction leaves lane (n, h) the rows 8a + 4h + b (a, b = 0..3)
// of its column, and the second product's slab of 16 takes its elements in that
// same order, with the staged tile read transposed (ds_read_b64_tr_b16) to match.
// Probabilities and dS never pass through memory.

#include <type_traits>

#include "common.h"

namespace mxq {

namespace {

constexpr int kNope = MXQ_NOPE_DIM, kRope = MXQ_ROPE_DIM, kVal = MXQ_VALUE_DIM;
constexpr int kQk = kNope + kRope;              // 192
constexpr int kSteps = kQk / 16, kVSteps = kVal / 16;   // 16-deep steps of the two products
constexpr int kBN = 64;                         // rows of a staged tile
constexpr int kThr = 256;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// The reference that a row's exponentials are taken against follows the
// running maximum only when that is more than this many powers of two ahead:
// any reference gives the same quotients, 2^8 times the largest loses no bits,
// and the sums are then hardly ever rescaled.
constexpr float kSlack = 8.0f;
// The backward kernels form P and dS 2^24 times too large (a shift of the
// exponent's argument) and scale the finished sums back, so that probabilities
// far below a row's largest do not underflow FP32.
constexpr float kShift = 24.0f, kUnshift = 1.0f / 16777216.0f;

// One operand: rows of `ld` elements, heads `ldh` elements apart.
struct Op {
  const uint16_t* p;
  int64_t ld, ldh;
};
struct OpOut {
  uint16_t* p;
  int64_t ld, ldh;
};

struct AttnArgs {
  Op q, kn, v, o, dout;
  const uint16_t* kr;
  int64_t ldr;
  const int64_t* offq;
  const int64_t* offk;
  int32_t B, H, causal;
  int64_t Tq, Tk;
  float scale;
  OpOut out, dq, dkn, dv;
  uint16_t* dkr;
  int64_t lddr;
  float* lse;
  int64_t ldl;
  float* delta;                                  // [H, Tq]
  float* rope_part;                              // [H, Tk, 64]
  int32_t parts;                                 // at most, of a forward tile's keys
  float* part_o;                                 // [parts, H, Tq, 128]
  float* part_ml;                                // [parts, H, Tq, 2]
};

// ---------------------------------------------------------------------------
// Packed sequences.  Offsets are clamped into the rows that exist, so a
// malformed table never leads outside the buffers.
// ---------------------------------------------------------------------------

struct SeqTile {
  int64_t q0, k0;                                // the sequence's first rows
  int lq, lk;                                    // and lengths
  int row0;                                      // first row of this tile in the sequence
  bool ok;
};

__device__ __forceinline__ int64_t clamp_off(int64_t o, int64_t n) { return o < 0 ? 0 : o > n ? n : o; }

__device__ __forceinline__ int64_t bcast64(int64_t v, int lane) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)((uint64_t)v >> 32), lane);
  return (int64_t)(((uint64_t)hi << 32) | lo);
}

// Sequence b's rows, clamped; nothing past the batch.
__device__ __forceinline__ void seq_rows(const AttnArgs& a, int32_t b, int64_t& q0, int64_t& k0, int64_t& lq,
                                         int64_t& lk) {
  q0 = k0 = lq = lk = 0;
  if (b >= a.B) return;
  q0 = a.offq ? clamp_off(a.offq[b], a.Tq) : 0;
  lq = (a.offq ? clamp_off(a.offq[b + 1], a.Tq) : a.Tq) - q0;
  k0 = a.offk ? clamp_off(a.offk[b], a.Tk) : 0;
  lk = (a.offk ? clamp_off(a.offk[b + 1], a.Tk) : a.Tk) - k0;
  lq = lq < 0 ? 0 : lq;
  lk = lk < 0 ? 0 : lk;
}

// Tile t of the list of all sequences' tiles of `rows` rows (of the keys with
// KEYS, of the queries without); a causal sequence's query tiles come last
// first, the ones with the most keys.  Every wavefront works it out for itself.
// With TWO, where two workgroups share a CU: those that start in pairs on the 256
// CUs (the first 256 and the next) take tiles from both ends of that part of the
// list, so that no CU has two of the longest (2 sequences of 2048, 16 heads: 64 us
// against 74; 8 of 512: 26.5 against 30).  Lists of more than two turns balance by themselves.
template <bool KEYS, bool TWO = false>
__device__ __forceinline__ SeqTile find_tile(const AttnArgs& a, uint32_t t, int rows) {
  SeqTile s{};
  const int lane = threadIdx.x & 63;
  int64_t q0, k0, lq, lk;
  const uint32_t lo = 256 / (uint32_t)a.H, two = 2 * lo;
  if (TWO && t >= lo && t < two) {
    uint32_t total = 0;
    for (int32_t base = 0; base < a.B && total <= 2 * two; base += 64) {
      seq_rows(a, base + lane, q0, k0, lq, lk);
      total += lane_u32(wave_scan((uint32_t)(((KEYS ? lk : lq) + rows - 1) / rows)), 63);
    }
    const uint32_t hi = total < two ? total : two;
    if (t >= hi) return s;
    if (total <= 2 * two) t = lo + hi - 1 - t;
  }
  uint32_t before = 0;
  for (int32_t base = 0; base < a.B; base += 64) {
    seq_rows(a, base + lane, q0, k0, lq, lk);
    const uint32_t n = (uint32_t)(((KEYS ? lk : lq) + rows - 1) / rows);
    const uint32_t incl = wave_scan(n);
    const uint64_t past = __ballot(t < before + incl);
    if (past) {
      const int at = __builtin_ctzll(past);
      s.q0 = bcast64(q0, at);
      s.k0 = bcast64(k0, at);
      s.lq = (int)bcast64(lq, at);
      s.lk = (int)bcast64(lk, at);
      const uint32_t nn = lane_u32(n, at);
      const uint32_t first = before + lane_u32(incl, at) - nn;
      const uint32_t i = t - first;
      s.row0 = (int)((!KEYS && a.causal ? nn - 1 - i : i) * (uint32_t)rows);
      s.ok = true;
      return s;
    }
    before += lane_u32(incl, 63);
  }
  return s;
}

// ---------------------------------------------------------------------------
// Staged tiles: 64 rows of the other side as three sub-tiles, N (128 columns),
// R (the 64 rotary columns) and Y (128 columns), copied from memory straight
// into LDS.  The 16-byte units of a row are permuted by an XOR with a function
// of the row, chosen for both ways the tiles are read: 16 rows at one unit (the
// first products' operand) and 4 consecutive rows at 4 consecutive units (the
// transposed reads) each cover the 16 units of a 256-byte bank line once.  Rows
// past the end read as zeros through the descriptors' range check.
// ---------------------------------------------------------------------------

constexpr int kNB = kBN * 256, kRB = kBN * 128;  // bytes of N (and Y) and of R
constexpr int kTile = 2 * kNB + kRB;             // 40 KB
constexpr int kOffR = kNB, kOffY = kNB + kRB;

__device__ __forceinline__ uint32_t f_wide(uint32_t r) { return ((r & 3) << 2) | ((r >> 2) & 3); }
__device__ __forceinline__ uint32_t f_rope(uint32_t r) {   // bits 1..3 of r, reversed
  return ((r & 2) << 1) | ((r & 4) >> 1) | ((r & 8) >> 3);
}

__device__ __forceinline__ i32x4 uniform(i32x4 r) {
  i32x4 u;
#pragma unroll
  for (int i = 0; i < 4; ++i) u[i] = __builtin_amdgcn_readfirstlane(r[i]);
  return u;
}

// 16 bytes a lane from descriptor offset `off + step` to LDS byte m0 + 16 lane.
// Not tracked by the compiler: tile_wait() orders it.
__device__ __forceinline__ void dma16(i32x4 r, uint32_t lds, uint32_t off, uint32_t step) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :: "s"(lds), "v"(off), "s"(r), "s"(step) : "memory");
}

// This lane's part of the copies.  Of NW wavefronts, w copies the 1 KB pieces w,
// w + NW, .. of each sub-tile (4 rows of N or Y, 8 rows of R), so a lane's unit
// is the same in every piece and only the row advances.
struct Copy {
  uint32_t n, r, y;                              // offset in the first piece
  uint32_t dn, dr, dy;                           // from piece to piece (uniform)
  uint32_t ldn, ldr, ldy;                        // row strides in bytes
  uint32_t lds;                                  // wavefront's LDS byte in a tile
};

template <int NW>
__device__ __forceinline__ Copy copy_plan(const void* lds, int64_t ldn, int64_t ldr, int64_t ldy) {
  Copy c;
  const uint32_t l = threadIdx.x & 63;
  const uint32_t w = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  c.ldn = (uint32_t)ldn * 2; c.ldr = (uint32_t)ldr * 2; c.ldy = (uint32_t)ldy * 2;
  const uint32_t r4 = 4 * w + (l >> 4), r8 = 8 * w + (l >> 3);
  const uint32_t uw = ((l & 15) ^ f_wide(r4)) * 16, ur = ((l & 7) ^ f_rope(r8)) * 16;
  c.n = r4 * c.ldn + uw;
  c.r = r8 * c.ldr + ur;
  c.y = r4 * c.ldy + uw;
  c.dn = 4 * NW * c.ldn; c.dr = 8 * NW * c.ldr; c.dy = 4 * NW * c.ldy;
  c.lds = (uint32_t)reinterpret_cast<uintptr_t>(lds) + w * 1024;
  return c;
}

// Bytes of `rows` rows (0 at least, 64 at most) of `ld` bytes, the last one `width`.
__device__ __forceinline__ uint32_t span(int rows, uint32_t ld, uint32_t width) {
  const int r = rows > kBN ? kBN : rows;
  return r > 0 ? (uint32_t)(r - 1) * ld + width : 0u;
}

// Starts the copy of rows row0 .. row0 + 63 of `rows` to tile buffer `buf`.
template <int NW>
__device__ __forceinline__ void tile_copy(const Copy& c, const uint16_t* n, const uint16_t* r,
                                          const uint16_t* y, int row0, int rows, int buf) {
  const uint8_t* pn = reinterpret_cast<const uint8_t*>(n) + (int64_t)row0 * c.ldn;
  const uint8_t* pr = reinterpret_cast<const uint8_t*>(r) + (int64_t)row0 * c.ldr;
  const uint8_t* py = reinterpret_cast<const uint8_t*>(y) + (int64_t)row0 * c.ldy;
  const i32x4 dn = uniform(make_rsrc(pn, span(rows - row0, c.ldn, 256)));
  const i32x4 dr = uniform(make_rsrc(pr, span(rows - row0, c.ldr, 128)));
  const i32x4 dy = uniform(make_rsrc(py, span(rows - row0, c.ldy, 256)));
  const uint32_t lds = (uint32_t)__builtin_amdgcn_readfirstlane((int)(c.lds + buf * kTile));
#pragma unroll
  for (int i = 0; i < 16 / NW; ++i) dma16(dn, lds + i * (NW * 1024), c.n, i * c.dn);
#pragma unroll
  for (int i = 0; i < 8 / NW; ++i) dma16(dr, lds + kOffR + i * (NW * 1024), c.r, i * c.dr);
#pragma unroll
  for (int i = 0; i < 16 / NW; ++i) dma16(dy, lds + kOffY + i * (NW * 1024), c.y, i * c.dy);
}

// Every copy this wavefront started has landed, and so, past the barrier, has
// every other wavefront's; and all reads before it are done.
__device__ __forceinline__ void tile_wait() {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
}

// Rows of the wavefront's own side as operands: lane (n, h) holds columns
// 16 s + 8 h .. + 7 of row n for each step s, from step 8 on of `pr`; rows past
// the end are zeros.
template <int STEPS>
__device__ __forceinline__ void own_rows(bf16x8 (&f)[STEPS], const uint16_t* p, int64_t ld,
                                         const uint16_t* pr, int64_t ldr, int row, int rows) {
  const int h = (threadIdx.x & 63) >> 5;
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (row < rows)
      v = *reinterpret_cast<const uint4*>(s < 8 ? p + (int64_t)row * ld + s * 16 + h * 8
                                                : pr + (int64_t)row * ldr + (s - 8) * 16 + h * 8);
    f[s] = __builtin_bit_cast(bf16x8, v);
  }
}

typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) i16x4 lds_i16x4;

// Where a lane reads in a tile.  Each step or column block only flips bits of
// the unit, so one base a kind of read serves them all.
struct Reads {
  uint32_t n, r;                                 // first products: N or Y, and R
  uint32_t tn, tr;                               // transposed: N or Y, and R
};

__device__ __forceinline__ Reads read_plan() {
  const uint32_t l = threadIdx.x & 63, n = l & 31, h = l >> 5, g = l >> 4, i = l & 15;
  Reads p;
  p.n = n * 256 + ((h ^ f_wide(n)) << 4);
  p.r = n * 128 + ((h ^ f_rope(n)) << 4);
  // each 16 lanes read 4 rows of 16 columns and receive one column of 4 rows each
  const uint32_t row = 4 * (g >> 1) + (i >> 2), u = 2 * (g & 1) + ((i & 3) >> 1);
  p.tn = row * 256 + ((u ^ f_wide(row)) << 4) + (i & 1) * 8;
  p.tr = row * 128 + ((u ^ f_rope(row)) << 4) + (i & 1) * 8;
  return p;
}

// First products: rows 32 sub .. + 31 of a tile, columns 16 s .. + 15.
__device__ __forceinline__ bf16x8 x_frag(const uint8_t* t, const Reads& p, int sub, int s) {
  return s < 8 ? *reinterpret_cast<const bf16x8*>(t + (p.n ^ (s << 5)) + sub * 8192)
               : *reinterpret_cast<const bf16x8*>(t + kOffR + (p.r ^ ((s - 8) << 5)) + sub * 4096);
}
__device__ __forceinline__ bf16x8 y_frag(const uint8_t* t, const Reads& p, int sub, int s) {
  return *reinterpret_cast<const bf16x8*>(t + kOffY + (p.n ^ (s << 5)) + sub * 8192);
}

// Second products: columns 32 d .. + 31 of the tile's rows 16 j .. + 15,
// transposed: lane (c, h) gets rows 16 j + 4 h + 0..3 and 16 j + 8 + 4 h + 0..3
// of column 32 d + c.
__device__ __forceinline__ bf16x8 tr_pair(const uint8_t* a, const uint8_t* b) {
  const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)a);
  const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)b);
  return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}
// From a sub-tile of 128 columns (N or Y) or of 64 (R) at t.
__device__ __forceinline__ bf16x8 wide_tr(const uint8_t* t, const Reads& p, int j, int d) {
  const uint32_t o = p.tn ^ (d << 6);
  return tr_pair(t + o + j * 4096, t + (o ^ 32) + 2048 + j * 4096);
}
__device__ __forceinline__ bf16x8 rope_tr(const uint8_t* t, const Reads& p, int j, int d) {
  const uint32_t o = p.tr ^ (d << 6);
  return tr_pair(t + o + j * 2048, t + (o ^ 16) + 1024 + j * 2048);
}

__device__ __forceinline__ f32x16 mfma(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// The tile row that register i of a 32-row block holds in lane half h.
__device__ __forceinline__ int reg_row(int i, int h) { return 8 * (i >> 2) + 4 * h + (i & 3); }

// 8 FP32 values rounded to BF16 (registers 8 j .. 8 j + 7 of a block: slab j).
__device__ __forceinline__ bf16x8 slab(const f32x16& p, int j) {
  uint4 w;
  w.x = bf16x2_bits(p[8 * j], p[8 * j + 1]);
  w.y = bf16x2_bits(p[8 * j + 2], p[8 * j + 3]);
  w.z = bf16x2_bits(p[8 * j + 4], p[8 * j + 5]);
  w.w = bf16x2_bits(p[8 * j + 6], p[8 * j + 7]);
  return __builtin_bit_cast(bf16x8, w);
}

__device__ __forceinline__ float half_max(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __builtin_fmaxf(__builtin_bit_cast(float, (uint32_t)r[0]),
                         __builtin_bit_cast(float, (uint32_t)r[1]));
}
__device__ __forceinline__ float half_sum(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __builtin_bit_cast(float, (uint32_t)r[0]) + __builtin_bit_cast(float, (uint32_t)r[1]);
}

// Transposed result blocks to memory: lane (n, h) holds columns reg_row(i, h)
// of each 32-column block of its row, 4 consecutive ones a store.
__device__ __forceinline__ void store_block(const f32x16& b, float mul, uint16_t* p) {
  const int h = (threadIdx.x & 63) >> 5;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint2 w;
    w.x = bf16x2_bits(b[4 * i] * mul, b[4 * i + 1] * mul);
    w.y = bf16x2_bits(b[4 * i + 2] * mul, b[4 * i + 3] * mul);
    *reinterpret_cast<uint2*>(p + 8 * i + 4 * h) = w;
  }
}

template <int NT>
__device__ __forceinline__ bool any_nonfinite(const f32x16 (&acc)[NT]) {
  bool bad = false;
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < 16; ++i) bad |= !(__builtin_fabsf(acc[t][i]) < __builtin_inff());
  return bad;
}

// ---------------------------------------------------------------------------
// Hidden values that are not finite.  A hidden key's probability is an exact 0, but
// the matrix unit still multiplies it, and 0 * NaN or 0 * infinity would reach
// rows that the mask keeps apart.  Such a product always leaves a NaN, so a
// workgroup some of whose results are not finite walks the other side a second
// time: tiles that all its rows see whole go through the matrix unit as before,
// since whatever they hold belongs in the result.  Of the tiles that the mask
// cuts, the forward kernel adds the keys one by one to the rows that see
// them; the backward kernels, whose sums leave no registers for that, set what is not
// finite in the staged tile to 0 for the second products, and note for each sum
// which of it the row sees.  Only rows that were not finite are written again, without the
// slack and the shift above.  Costs a sound call one check of the results; with
// a NaN the kernels take 2.5 to 4 times as long, 6 where few rows are cut often
// (one sequence of 2048, 8 heads: forward 145 us against 50, backward 370 against 140).
// ---------------------------------------------------------------------------

// o[i .. i + 3] += w times the 4 BF16 values at t, where they are seen.
__device__ __forceinline__ void add4(f32x16& o, int i, bool seen, float w, const uint8_t* t) {
  uint2 x = *reinterpret_cast<const uint2*>(t);
  x.x = seen ? x.x : 0u;
  x.y = seen ? x.y : 0u;
  o[i] = __builtin_fmaf(w, bf16_lo(x.x), o[i]);
  o[i + 1] = __builtin_fmaf(w, bf16_hi(x.x), o[i + 1]);
  o[i + 2] = __builtin_fmaf(w, bf16_lo(x.y), o[i + 2]);
  o[i + 3] = __builtin_fmaf(w, bf16_hi(x.y), o[i + 3]);
}

// Which of 4 BF16 values are NaN: a bit each.
__device__ __forceinline__ uint32_t nan4(uint2 x) {
  return ((x.x & 0x7FFFu) > 0x7F80u ? 1u : 0u) | ((x.x & 0x7FFFFFFFu) > 0x7F80FFFFu ? 2u : 0u) |
         ((x.y & 0x7FFFu) > 0x7F80u ? 4u : 0u) | ((x.y & 0x7FFFFFFFu) > 0x7F80FFFFu ? 8u : 0u);
}

// Whether any of the workgroup's `waves` wavefronts has bits set, through the first words
// of `lds`, which no wavefront needs any more once all are here.
__device__ __forceinline__ bool any_wave(uint8_t* lds, uint32_t bits, int waves) {
  uint32_t* w = reinterpret_cast<uint32_t*>(lds);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) w[threadIdx.x >> 6] = bits;
  __syncthreads();
  uint32_t all = 0;
  for (int i = 0; i < waves; ++i) all |= w[i];
  __syncthreads();
  return all != 0;
}

__device__ __forceinline__ float bf(const uint16_t* p) {
  return __builtin_bit_cast(float, (uint32_t)*p << 16);
}

__device__ __forceinline__ int lane_id() { return __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u)); }

// A head's operands of one sequence.
struct Head {
  const uint16_t *q, *kn, *kr, *v, *o, *g;       // g: the output's gradient
  const float *lse, *delta;
};
__device__ __forceinline__ Head head_of(const AttnArgs& a, const SeqTile& s, int head) {
  Head x;
  x.q = a.q.p + s.q0 * a.q.ld + head * a.q.ldh;
  x.kn = a.kn.p + s.k0 * a.kn.ld + head * a.kn.ldh;
  x.kr = a.kr + s.k0 * a.ldr;
  x.v = a.v.p + s.k0 * a.v.ld + head * a.v.ldh;
  x.o = a.o.p + s.q0 * a.o.ld + head * a.o.ldh;
  x.g = a.dout.p + s.q0 * a.dout.ld + head * a.dout.ldh;
  x.lse = a.lse + head * a.ldl + s.q0;
  x.delta = a.delta + head * a.Tq + s.q0;
  return x;
}

// Keys that query row i sees.
__device__ __forceinline__ int keys_seen(const AttnArgs& a, const SeqTile& s, int i) {
  if (!a.causal) return s.lk;
  const int64_t e = (int64_t)i + s.lk - s.lq + 1;
  return e < 0 ? 0 : e < s.lk ? (int)e : s.lk;
}

// ---------------------------------------------------------------------------
// Forward.  A workgroup of four wavefronts takes 128 query rows of one head, 32 a
// wavefront; two workgroups share a CU, so that one's exponentials run beside
// the other's products.
//
// Bound by the matrix unit and what has to run between its products.  4 sequences
// of 4096, 16 heads, causal: 357 to 378 us by machine, at best 0.96 PFLOP/s (a
// large matrix product reaches 1.16 to 1.25 on the same card, and its rate on such
// data is set by power).  Of 363 us in an early form the products alone took 297, and 326 were left without
// LDS reads, 329 without maxima and exponentials.  64 rows a wavefront halve the
// LDS reads but leave one wavefront a SIMD: 600 us.  Eight wavefronts that split
// each tile's keys shorten the chain of a single long sequence (one of 2000, 4
// heads: 46 us to 42) and cost every other case (this one: 470 us).
// ---------------------------------------------------------------------------

// With SPLIT, a call of few workgroups, several take a tile's keys between them,
// and k_attn_join joins their sums.

// Parts of a tile whose rows see `keys` keys.
__device__ __forceinline__ int parts_of(const AttnArgs& a, int keys) {
  const int n = keys / kPartKeys;
  return n < 1 ? 1 : n < a.parts ? n : a.parts;
}

// Adds the keys of the tile at k0 that a lane's row sees (those below `lim`) to its sums
// one by one.  s: the probabilities, as the matrix unit left the logits.
__device__ __forceinline__ void add_seen_keys(f32x16 (&o)[4], f32x16 (&s)[2], const uint8_t* tile, int k0, int lim) {
  const uint32_t h = (threadIdx.x & 63) >> 5;
#pragma unroll 1
  for (uint32_t g = 0; g < 8; ++g) {               // keys 8 g .. 8 g + 7: registers 0..3 of both halves
#pragma unroll
    for (uint32_t e = 0; e < 4; ++e) {
      const float own = s[0][e], other = __shfl_xor(own, 32, 64);
#pragma unroll
      for (uint32_t hh = 0; hh < 2; ++hh) {
        const uint32_t key = 8 * g + 4 * hh + e;
        const bool seen = k0 + (int)key < lim;
        const float p = h == hh ? own : other;
#pragma unroll
        for (uint32_t x = 0; x < 16; ++x)          // columns 8 x + 4 h .. + 3
          add4(o[x >> 2], 4 * (x & 3), seen, p, tile + kOffY + key * 256 + ((x ^ f_wide(key)) << 4) + 8 * h);
      }
    }
#pragma unroll
    for (int i = 0; i < 12; ++i) s[0][i] = s[0][i + 4];
#pragma unroll
    for (int i = 0; i < 4; ++i) s[0][12 + i] = s[1][i];
#pragma unroll
    for (int i = 0; i < 12; ++i) s[1][i] = s[1][i + 4];
  }
}

template <bool SPLIT>
__global__ __launch_bounds__(kThr, 2) void k_attn_fwd(AttnArgs a) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * kTile];
  constexpr int BM = 128;
  const int head = blockIdx.x % a.H;
  const uint32_t unit = blockIdx.x / a.H;
  const SeqTile st = find_tile<false, !SPLIT>(a, SPLIT ? unit / a.parts : unit, BM);
  if (!st.ok) return;                              // uniform over the workgroup
  const int l = threadIdx.x & 63, n = l & 31, h = l >> 5;
  const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int wrow0 = st.row0 + w * 32, row = wrow0 + n;   // the wavefront's first row, this lane's
  const uint16_t* kn = a.kn.p + st.k0 * a.kn.ld + head * a.kn.ldh;
  const uint16_t* kr = a.kr + st.k0 * a.ldr;
  const uint16_t* v = a.v.p + st.k0 * a.v.ld + head * a.v.ldh;
  const Copy cp = copy_plan<4>(lds, a.kn.ld, a.ldr, a.v.ld);
  const Reads rp = read_plan();

  // keys that any row of the workgroup sees, and the wavefront's first and last row
  const int last = (st.row0 + BM < st.lq ? st.row0 + BM : st.lq) - 1;
  const int kend = keys_seen(a, st, last);
  const int wfirst = keys_seen(a, st, wrow0), wlast = keys_seen(a, st, wrow0 + 31);
  const int lim = keys_seen(a, st, row);
  int part = 0, parts = 1, kfirst = 0, kstop = kend;
  if (SPLIT) {
    part = (int)(unit % a.parts);
    parts = parts_of(a, kend);
    if (part >= parts) return;
    const int tiles = (kend + kBN - 1) / kBN;
    kfirst = tiles * part / parts * kBN;
    if (part + 1 < parts) kstop = tiles * (part + 1) / parts * kBN;
  }
  if (kstop > kfirst) tile_copy<4>(cp, kn, kr, v, kfirst, st.lk, 0);

  bf16x8 q[kSteps];
  const uint16_t* qp = a.q.p + st.q0 * a.q.ld + head * a.q.ldh;
  own_rows(q, qp, a.q.ld, qp + kNope, a.q.ld, row, st.lq);
  f32x16 o[4];
  float m, sum, total;                             // reference (powers of two), total
  const float c = a.scale * kLog2e;
  // The sums over this workgroup's keys.  CAREFUL: of a tile that not all rows of the
  // wavefront see, keys are added one by one to the rows that see them, and the
  // reference is the running maximum itself.
  auto walk = [&](auto careful) __attribute__((always_inline)) {
    constexpr bool CAREFUL = decltype(careful)::value;
#pragma unroll
    for (int d = 0; d < 4; ++d) o[d] = f32x16{};
    m = -__builtin_inff();
    sum = 0.0f;
    int buf = 0;
    for (int k0 = kfirst; k0 < kstop; k0 += kBN, buf ^= 1) {
      tile_wait();
      if (k0 + kBN < kstop) tile_copy<4>(cp, kn, kr, v, k0 + kBN, st.lk, buf ^ 1);
      if (k0 >= wlast) continue;                   // nothing seen by this wavefront
      const uint8_t* tile = lds + buf * kTile;
      f32x16 s[2] = {};
      pipelined<2 * kSteps, 6>([&](int i) { return x_frag(tile, rp, i & 1, i >> 1); },
                               [&](int i, bf16x8 f) { s[i & 1] = mfma(f, q[i >> 1], s[i & 1]); });
      if (k0 + kBN > wfirst) {                     // some row does not see all of the tile
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (k0 + 32 * b + reg_row(i, h) >= lim) s[b][i] = -__builtin_inff();
      }
      float mx = s[0][0];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        mx = __builtin_fmaxf(mx, s[0][i]);
        mx = __builtin_fmaxf(mx, s[1][i]);
      }
      mx = half_max(mx) * c;
      if (__builtin_expect(__ballot(mx > m + (CAREFUL ? 0.0f : kSlack)) != 0, 0)) {
        const float mn = __builtin_fmaxf(m, mx);
        const float alpha = mn == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f(m - mn);
        m = mn;
        sum *= alpha;
#pragma unroll
        for (int d = 0; d < 4; ++d) o[d] *= alpha;
      }
      const float mc = m == -__builtin_inff() ? 0.0f : m;   // nothing seen yet: all zeros
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(s[b][i], c, -mc));
          s[b][i] = e;
          sum += e;
        }
      if (CAREFUL && k0 + kBN > wfirst) {
        add_seen_keys(o, s, tile, k0, lim);
        continue;
      }
      bf16x8 p[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) p[j] = slab(s[j >> 1], j & 1);
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int d = 0; d < 4; ++d) o[d] = mfma(wide_tr(tile + kOffY, rp, j, d), p[j], o[d]);
    }
    total = half_sum(sum);
  };
  // this lane's row, if `write`: the result, or its part
  auto store = [&](bool write, bool with_lse) {
    if (!write) return;
    if (SPLIT && parts > 1) {
      const int64_t pr = ((int64_t)part * a.H + head) * a.Tq + st.q0 + row;
#pragma unroll
      for (int d = 0; d < 4; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<f32x4*>(a.part_o + pr * kVal + 32 * d + 8 * i + 4 * h) =
              f32x4{o[d][4 * i], o[d][4 * i + 1], o[d][4 * i + 2], o[d][4 * i + 3]};
      if (h == 0) a.part_ml[2 * pr] = m, a.part_ml[2 * pr + 1] = total;
      return;
    }
    // a row that sees nothing: zeros, and minus infinity
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;
    uint16_t* p = a.out.p + (st.q0 + row) * a.out.ld + head * a.out.ldh;
#pragma unroll
    for (int d = 0; d < 4; ++d) store_block(o[d], inv, p + 32 * d);
    if (with_lse && h == 0)
      a.lse[head * a.ldl + st.q0 + row] =
          total == 0.0f ? -__builtin_inff() : kLn2 * (m + __builtin_amdgcn_logf(total));
  };
  walk(std::false_type{});
  store(row < st.lq, true);
  if (!a.causal) return;
  // rows that a hidden value may have reached, of a wavefront whose last tile hides some keys from some rows
  const int walked = kstop < wlast ? kstop : (wlast + kBN - 1) / kBN * kBN;
  const uint64_t bad = __ballot(any_nonfinite(o) && row < st.lq && total == total && walked > wfirst);
  const uint32_t redo = (uint32_t)bad | (uint32_t)(bad >> 32);
  if (!any_wave(lds, redo, 4)) return;             // uniform over the workgroup
  tile_copy<4>(cp, kn, kr, v, kfirst, st.lk, 0);
  walk(std::true_type{});
  store(row < st.lq && ((redo >> n) & 1), false);
}

// Joins the parts of the tiles that have several, in their order: with M = max m,
// o = sum 2^(m - M) O / sum 2^(m - M) l.  A workgroup takes 32 rows of a tile, 8
// lanes a row.
__global__ __launch_bounds__(kThr) void k_attn_join(AttnArgs a) {
  const int head = blockIdx.x % a.H;
  const uint32_t unit = blockIdx.x / a.H;
  const SeqTile st = find_tile<false>(a, unit / 4, 128);
  if (!st.ok) return;
  const int last = (st.row0 + 128 < st.lq ? st.row0 + 128 : st.lq) - 1;
  const int parts = parts_of(a, keys_seen(a, st, last));
  const int l = threadIdx.x & 63, w = threadIdx.x >> 6, c = l & 7;
  const int row0 = st.row0 + (int)(unit % 4) * 32 + w * 8, row = row0 + (l >> 3);
  if (parts == 1 || row0 >= st.lq) return;         // uniform over the wavefront
  const bool ok = row < st.lq;
  const int64_t pr = (int64_t)head * a.Tq + st.q0 + (ok ? row : row0), step = (int64_t)a.H * a.Tq;
  float m = -__builtin_inff();
  for (int p = 0; p < parts; ++p) m = __builtin_fmaxf(m, a.part_ml[2 * (pr + p * step)]);
  const float ref = m == -__builtin_inff() ? 0.0f : m;
  f32x4 o[4] = {};
  float total = 0.0f;
#pragma unroll 2
  for (int p = 0; p < parts; ++p) {
    const int64_t at = pr + p * step;
    const float f = __builtin_amdgcn_exp2f(a.part_ml[2 * at] - ref);
    total = __builtin_fmaf(f, a.part_ml[2 * at + 1], total);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const f32x4 v = *reinterpret_cast<const f32x4*>(a.part_o + at * kVal + 32 * j + 4 * c);
#pragma unroll
      for (int e = 0; e < 4; ++e) o[j][e] = __builtin_fmaf(f, v[e], o[j][e]);
    }
  }
  if (!ok) return;
  const float inv = total == 0.0f ? 0.0f : 1.0f / total;
  uint16_t* p = a.out.p + (st.q0 + row) * a.out.ld + head * a.out.ldh + 4 * c;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint2 x;
    x.x = bf16x2_bits(o[j][0] * inv, o[j][1] * inv);
    x.y = bf16x2_bits(o[j][2] * inv, o[j][3] * inv);
    *reinterpret_cast<uint2*>(p + 32 * j) = x;
  }
  if (c == 0)
    a.lse[head * a.ldl + st.q0 + row] =
        total == 0.0f ? -__builtin_inff() : kLn2 * (ref + __builtin_amdgcn_logf(total));
}

// ---------------------------------------------------------------------------
// Backward.  With PAIRS = 4, eight wavefronts, two a SIMD: a pair shares 32 rows
// of the workgroup's 128.  Of each tile of 64, one of the pair forms P and dS against
// the first 32 rows, the other against the last, and they hand each other the
// operands through LDS (as they are, in lane order).  Then each takes half of
// the result's columns over all 64.  That halves the sums a wavefront holds,
// which is what lets two of them share a SIMD: one's exponentials run beside
// the other's products.  The sums over a tile are taken beside the next tile's P
// and dS, between one pair of barriers, which takes three tile buffers (1540 us for
// the three kernels on the case below with two buffers, 1480 with three).  With
// PAIRS = 2, 64 rows and a wavefront a SIMD: shorter steps, for calls that leave
// CUs idle otherwise.
//
// 4 sequences of 4096, 16 heads, causal: dQ 720 to 759 us and dK and dV 709 to 750
// by machine, at best 1.05 and 0.97 PFLOP/s of the 11 and 10 products of 64 columns
// that they form a pair (13 in all are the least; S and dP are formed by both, and
// P K makes D exact).  Bound by
// the matrix unit and the chain before P and dS: without the sums over the tiles
// 1080 us of 1470 are left, though they are half of the products; without the
// copies 6 % less, without the second barrier nothing.  The two of a pair taking
// the two parts in opposite orders are slower (1556 us), and 64 rows a wavefront do
// not fit.
// ---------------------------------------------------------------------------

// Slabs that a wavefront hands over: 2 of P and 2 of dS.
template <int PAIRS>
struct Exchange {
  uint4 f[PAIRS][2][4][64];                      // pair, half, slab, lane
};

// Rounding dS once costs dQ and dK as much as rounding the result does; the two
// together are 1.41 times the least error, evenly where many entries of dS make a
// result.  Where few do it varies, up to 1.7 times (one sequence of 18, 2 heads).  So where
// queries see at most kFew keys, what the rounding left of dS is handed on as a second
// BF16 term and multiplied in a run of its own: 1.0 times the least.  It lies in the tile
// buffer that is free until the next tile but one is copied, whose copy then starts
// after it is read.  Whether a group of 32 query rows (dQ) or a tile of 64 (dK) has it goes by
// what its first row sees, so a sequence's gradient does not depend on what shares the
// call, and it costs a sequence's first tiles alone.  The second walk does without.
constexpr int kFew = 64;
struct Rests {
  uint4 f[2][2][64];                             // half, slab, lane, of one pair
};
__device__ __forceinline__ Rests& rests_of(uint8_t* lds, int buf, int pair) {
  return reinterpret_cast<Rests*>(lds + buf * kTile)[pair];
}

// Tile row r's entry for this lane's own row, of the slabs `slab` and `slab + 1` that were
// handed over.
template <int PAIRS>
__device__ __forceinline__ float handed(const Exchange<PAIRS>& ex, int pair, uint32_t r, int slab) {
  const uint32_t n = threadIdx.x & 31, lane = n + 32 * ((r >> 2) & 1), at = (r & 3) + 4 * ((r >> 3) & 1);
  return bf(reinterpret_cast<const uint16_t*>(&ex.f[pair][r >> 5][slab + ((r >> 4) & 1)][lane]) + at);
}

// What rounding to BF16 left of 8 values (slab j of p, rounded to w), rounded.
__device__ __forceinline__ uint4 slab_rest(const f32x16& p, uint4 w, int j) {
  f32x16 r;
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r[8 * j + 2 * i] = p[8 * j + 2 * i] - __builtin_bit_cast(float, x[i] << 16);
    r[8 * j + 2 * i + 1] = p[8 * j + 2 * i + 1] - __builtin_bit_cast(float, x[i] & 0xFFFF0000u);
  }
  return __builtin_bit_cast(uint4, slab(r, j));
}

// Backward, queries: dQ and D, which the keys' kernel reads.
//
// D is wanted before the loop that could sum it.  The BF16 output gives it but
// for the output's rounding, d = rowsum(dO * o), and that is not good enough where
// few keys hold a row's weight (dS is then a difference of nearly equal
// numbers).  With dS' = P * (dP - d), the row sum r of dS' is D - d, and
//   dQ = scale * (dS' K - r (P K)):
// the products P K and dS' K share the reads of K.
template <int PAIRS>
__global__ __launch_bounds__(128 * PAIRS, PAIRS / 2) void k_attn_dq(AttnArgs a) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[3 * kTile];
  __shared__ __attribute__((aligned(16))) Exchange<PAIRS> ex;
  __shared__ float s_rest[PAIRS][2][32];
  __shared__ uint32_t s_bad[PAIRS][2];
  constexpr int BM = 32 * PAIRS;
  const int head = blockIdx.x % a.H;
  const SeqTile st = find_tile<false>(a, blockIdx.x / a.H, BM);
  if (!st.ok) return;
  const int l = threadIdx.x & 63, n = l & 31, h = l >> 5;
  const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int pair = w % PAIRS, half = w / PAIRS;
  const int wrow0 = st.row0 + pair * 32, row = wrow0 + n;
  const Head x = head_of(a, st, head);
  const Copy cp = copy_plan<2 * PAIRS>(lds, a.kn.ld, a.ldr, a.v.ld);
  Reads rp = read_plan();
  const int last = (st.row0 + BM < st.lq ? st.row0 + BM : st.lq) - 1;
  const int kend = keys_seen(a, st, last);
  const int wfirst = keys_seen(a, st, wrow0), wlast = keys_seen(a, st, wrow0 + 31);
  const int lim = keys_seen(a, st, row);
  if (kend > 0) tile_copy<2 * PAIRS>(cp, x.kn, x.kr, x.v, 0, st.lk, 0);

  bf16x8 q[kSteps], g[kVSteps];
  own_rows(q, x.q, a.q.ld, x.q + kNope, a.q.ld, row, st.lq);
  own_rows(g, x.g, a.dout.ld, nullptr, 0, row, st.lq);
  float delta = 0.0f;                              // d
  {
    bf16x8 of[kVSteps];
    own_rows(of, x.o, a.o.ld, nullptr, 0, row, st.lq);
#pragma unroll
    for (int s = 0; s < kVSteps; ++s)
#pragma unroll
      for (int e = 0; e < 8; ++e) delta = __builtin_fmaf((float)of[s][e], (float)g[s][e], delta);
    delta = half_sum(delta);
  }
  float lse2 = row < st.lq ? x.lse[row] : -__builtin_inff();   // in powers of two
  lse2 = lse2 == -__builtin_inff() ? __builtin_inff() : lse2 * kLog2e - kShift;   // no keys: P = 0

  // this wavefront's columns: N blocks 2 half, 2 half + 1 and R block half
  f32x16 dq[3] = {}, pk[3] = {};
  float rest = 0.0f, unshift = kUnshift;           // row sum of this half's dS'
  const float c = a.scale * kLog2e;
  const int cut = keys_seen(a, st, st.row0);       // tiles before it are seen whole by all
  // tiles before these have a second term of dS: for the pair's rows, and for any of the workgroup's
  const int few = wfirst <= kFew ? wlast : 0, few_any = cut <= kFew ? kFew + 32 : 0;
  // P and dS against the tile at k0 (in buffer `buf`), this wavefront's 32 keys of it
  auto first = [&](auto again, uint4 (&mine)[4], int k0, int buf, int spare) __attribute__((always_inline)) {
    if (k0 >= wlast) return;                       // the same for both of a pair
    const uint8_t* tile = lds + buf * kTile;
    // the units' addresses are formed again in every tile: kept, they cost too many registers
    asm volatile("" : "+v"(rp.n), "+v"(rp.r), "+v"(rp.tn), "+v"(rp.tr));
    f32x16 s = {}, dp = {};
    // the two chains alternate while both last
    pipelined<kSteps + kVSteps, 4>(
        [&](int i) {
          return i < 2 * kVSteps && (i & 1) ? y_frag(tile, rp, half, i >> 1)
                                            : x_frag(tile, rp, half, i < 2 * kVSteps ? i >> 1 : i - kVSteps);
        },
        [&](int i, bf16x8 f) {
          if (i < 2 * kVSteps && (i & 1))
            dp = mfma(f, g[i >> 1], dp);
          else
            s = mfma(f, q[i < 2 * kVSteps ? i >> 1 : i - kVSteps], s);
        });
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      s[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], c, -lse2));
      dp[i] = s[i] * (dp[i] - delta);
    }
    if (k0 + kBN > wfirst) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (k0 + 32 * half + reg_row(i, h) >= lim) s[i] = 0.0f, dp[i] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) rest += dp[i];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      mine[j] = __builtin_bit_cast(uint4, slab(s, j));
      mine[2 + j] = __builtin_bit_cast(uint4, slab(dp, j));
      if (!decltype(again)::value && k0 < few) rests_of(lds, spare, pair).f[half][j][l] = slab_rest(dp, mine[2 + j], j);
    }
  };
  // the sums over the tile at k0, with the pair's P and dS
  auto second = [&](auto again, int k0, int buf, int spare) __attribute__((always_inline)) {
    if (k0 < 0 || k0 >= wlast) return;
    const uint8_t* tile = lds + buf * kTile;
    asm volatile("" : "+v"(rp.n), "+v"(rp.r), "+v"(rp.tn), "+v"(rp.tr));
    bf16x8 p[4], ds[4];
    pipelined<12, 3>(
        [&](int i) {
          const int j = i / 3, d = i % 3;
          if (d == 0) {
            p[j] = __builtin_bit_cast(bf16x8, ex.f[pair][j >> 1][j & 1][l]);
            ds[j] = __builtin_bit_cast(bf16x8, ex.f[pair][j >> 1][2 + (j & 1)][l]);
          }
          return d < 2 ? wide_tr(tile, rp, j, 2 * half + d) : rope_tr(tile + kOffR, rp, j, half);
        },
        [&](int i, bf16x8 f) {
          dq[i % 3] = mfma(f, ds[i / 3], dq[i % 3]);
          pk[i % 3] = mfma(f, p[i / 3], pk[i % 3]);
        });
    if (!decltype(again)::value && k0 < few) {
#pragma unroll 1
      for (int j = 0; j < 4; ++j) {
        const bf16x8 rs = __builtin_bit_cast(bf16x8, rests_of(lds, spare, pair).f[j >> 1][j & 1][l]);
        dq[0] = mfma(wide_tr(tile, rp, j, 2 * half), rs, dq[0]);
        dq[1] = mfma(wide_tr(tile, rp, j, 2 * half + 1), rs, dq[1]);
        dq[2] = mfma(rope_tr(tile + kOffR, rp, j, half), rs, dq[2]);
      }
    }
  };
  // The second walk: where this lane's row sees a key that is not finite, its gradient is not
  // (such a key's logit makes the whole row NaN, or, at minus infinity, its P an exact 0).
  uint64_t nan = 0;                                // a bit for each of this lane's 48 sums
  auto cover = [&](int k0, int buf) __attribute__((always_inline)) {
    uint8_t* tile = lds + buf * kTile;
#pragma unroll 1
    for (uint32_t key = 0; key < kBN; ++key) {
      uint64_t bits = 0;
#pragma unroll
      for (uint32_t u = 0; u < 12; ++u) {          // columns 8 u + 4 h .. + 3 of this half's 96
        const uint8_t* t = u < 8 ? tile + key * 256 + (((8 * half + u) ^ f_wide(key)) << 4)
                                 : tile + kOffR + key * 128 + (((4 * half + u - 8) ^ f_rope(key)) << 4);
        bits |= (uint64_t)nonfinite4(*reinterpret_cast<const uint2*>(t + 8 * h)) << (4 * u);
      }
      nan |= k0 + (int)key < lim ? bits : 0;
    }
    __syncthreads();
    clear_nonfinite(tile, kOffY, 128 * PAIRS);     // N and R
    __syncthreads();
  };
  // The sums over the keys that the workgroup sees.
  auto walk = [&](auto again) __attribute__((always_inline)) {
    constexpr bool FIRST = !decltype(again)::value;
    int buf = 0, prev = 2;                         // of this tile and of the one before
    for (int k0 = 0; k0 < kend + kBN; k0 += kBN) {
      tile_wait();
      const int next = buf == 2 ? 0 : buf + 1;
      // whether the last tile's rests lie where the next copy goes
      const bool late = FIRST && k0 > 0 && k0 - kBN < few_any;
      if (!late && k0 + kBN < kend) tile_copy<2 * PAIRS>(cp, x.kn, x.kr, x.v, k0 + kBN, st.lk, next);
      uint4 mine[4];                               // this wavefront's P and dS slabs
      if (!FIRST && k0 > cut) cover(k0 - kBN, prev);
      second(again, k0 - kBN, prev, next);
      if (late || (FIRST && k0 < few_any)) __syncthreads();   // the last tile and its rests are consumed
      if (late && k0 + kBN < kend) tile_copy<2 * PAIRS>(cp, x.kn, x.kr, x.v, k0 + kBN, st.lk, next);
      if (k0 < kend) first(again, mine, k0, buf, prev);
      __syncthreads();                             // the last tile's operands are consumed
      if (k0 < kend && k0 < wlast) {
#pragma unroll
        for (int j = 0; j < 4; ++j) ex.f[pair][half][j][l] = mine[j];
      }
      prev = buf;
      buf = next;
    }
    rest = half_sum(rest);
    const int lane = lane_id();                    // formed again: kept through the loop, it costs a register
    if (lane < 32) s_rest[pair][half][lane] = rest;
    __syncthreads();
    const float r = (s_rest[pair][0][lane & 31] + s_rest[pair][1][lane & 31]) * unshift;
#pragma unroll
    for (int d = 0; d < 3; ++d) dq[d] -= pk[d] * r;
    return r;
  };
  auto store = [&](bool write) {
    const int row = wrow0 + (lane_id() & 31);
    if (row >= st.lq || !write) return;
    uint16_t* p = a.dq.p + (st.q0 + row) * a.dq.ld + head * a.dq.ldh;
#pragma unroll
    for (int d = 0; d < 2; ++d) store_block(dq[d], a.scale * unshift, p + 64 * half + 32 * d);
    store_block(dq[2], a.scale * unshift, p + kNope + 32 * half);
  };
  const float r = walk(std::false_type{});
  store(true);
  const int after = wrow0 + (lane_id() & 31);      // this lane's row
  if (after < st.lq && lane_id() < 32 && half == 0) a.delta[head * a.Tq + st.q0 + after] = delta + r;
  if (!a.causal) return;
  // rows that a hidden key may have reached
  const uint64_t bad = __ballot(any_nonfinite(dq) && after < st.lq && (lim == 0 || (lse2 == lse2 && delta == delta)));
  if (lane_id() == 0) s_bad[pair][half] = (uint32_t)bad | (uint32_t)(bad >> 32);
  __syncthreads();
  uint32_t any = 0;
#pragma unroll
  for (int i = 0; i < PAIRS; ++i) any |= s_bad[i][0] | s_bad[i][1];
  if (!any) return;                                // uniform over the workgroup
  if (kend > 0) tile_copy<2 * PAIRS>(cp, x.kn, x.kr, x.v, 0, st.lk, 0);
#pragma unroll
  for (int d = 0; d < 3; ++d) dq[d] = f32x16{}, pk[d] = f32x16{};
  rest = 0.0f;
  lse2 += kShift;
  unshift = 1.0f;
  walk(std::true_type{});
#pragma unroll
  for (int i = 0; i < 48; ++i)
    if ((nan >> i) & 1) dq[i / 16][i % 16] = __builtin_nanf("");
  store(((s_bad[pair][0] | s_bad[pair][1]) >> (lane_id() & 31)) & 1);
}

// Backward, keys: dK, dV, walking the queries that see the workgroup's keys.  The
// rotary part of dK is summed over the heads by k_attn_drope, from one FP32 part
// a head, in head order.
template <int PAIRS>
__global__ __launch_bounds__(128 * PAIRS, PAIRS / 2) void k_attn_dkv(AttnArgs a) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[3 * kTile];
  __shared__ __attribute__((aligned(16))) Exchange<PAIRS> ex;
  __shared__ __attribute__((aligned(16))) float stat[2][2][kBN];   // lse (powers of two), D
  __shared__ uint32_t s_bad[PAIRS][2];
  constexpr int BM = 32 * PAIRS;
  const int head = blockIdx.x % a.H;
  const SeqTile st = find_tile<true>(a, blockIdx.x / a.H, BM);
  if (!st.ok) return;
  const int l = threadIdx.x & 63, n = l & 31, h = l >> 5;
  const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int pair = w % PAIRS, half = w / PAIRS;
  const int wkey = st.row0 + pair * 32, row = wkey + n;   // the pair's keys, this lane's
  const int diff = st.lk - st.lq;                  // query i sees keys j <= i + diff
  const Head x = head_of(a, st, head);
  const Copy cp = copy_plan<2 * PAIRS>(lds, a.q.ld, a.q.ld, a.dout.ld);
  Reads rp = read_plan();

  // queries from lim on see this lane's key; the tile starts at the first that sees any
  const int lim = !a.causal || row - diff < 0 ? 0 : row - diff;
  int q0 = 0;
  if (a.causal) {
    const int f = st.row0 - diff;
    q0 = f <= 0 ? 0 : f >= st.lq ? st.lq : f;
    q0 = q0 / kBN * kBN;
  }
  const int wlim = !a.causal ? 0 : wkey - diff;    // first query that sees the pair's first key
  // lse and D of a tile's queries, one value a lane of the first two wavefronts
  auto stat_of = [&](int r0) {
    const int i = r0 + l;
    float z = 0.0f;
    if (w < 2 && i < st.lq) z = w == 0 ? x.lse[i] : x.delta[i];
    return z;
  };
  float z = 0.0f;
  if (q0 < st.lq) {
    z = stat_of(q0);
    tile_copy<2 * PAIRS>(cp, x.q, x.q + kNope, x.g, q0, st.lq, 0);
  }
  bf16x8 k[kSteps], v[kVSteps];
  own_rows(k, x.kn, a.kn.ld, x.kr, a.ldr, row, st.lk);
  own_rows(v, x.v, a.v.ld, nullptr, 0, row, st.lk);

  // this wavefront's columns: all of dV (half 0) or of dK's own part (half 1), and
  // block `half` of the rotary part
  f32x16 wide[4] = {}, rope = {};
  const uint32_t side = half ? 0 : kOffY, op = half ? 2 : 0;   // queries and dS, or dO and P
  const float c = a.scale * kLog2e;
  // Tiles before it have a second term of dS: their first query sees at most kFew keys.
  // Without a mask all queries see as many, and the first two tiles are taken.
  const int few = a.causal ? kFew - diff : st.lk <= kFew ? 2 * kBN : 0;
  // P and dS against the tile at r0 (in buffer `buf`), this wavefront's 32 queries of it
  auto first = [&](auto fine, uint4 (&mine)[4], int r0, int buf, int spare, int sb) __attribute__((always_inline)) {
    if (r0 + kBN <= wlim) return;                  // no query here sees the pair's keys
    const uint8_t* tile = lds + buf * kTile;
    // the units' addresses are formed again in every tile: kept, they cost too many registers
    asm volatile("" : "+v"(rp.n), "+v"(rp.r), "+v"(rp.tn), "+v"(rp.tr));
    f32x16 s = {}, dp = {};
    // the two chains alternate while both last
    pipelined<kSteps + kVSteps, 4>(
        [&](int i) {
          return i < 2 * kVSteps && (i & 1) ? y_frag(tile, rp, half, i >> 1)
                                            : x_frag(tile, rp, half, i < 2 * kVSteps ? i >> 1 : i - kVSteps);
        },
        [&](int i, bf16x8 f) {
          if (i < 2 * kVSteps && (i & 1))
            dp = mfma(f, v[i >> 1], dp);
          else
            s = mfma(f, k[i < 2 * kVSteps ? i >> 1 : i - kVSteps], s);
        });
#pragma unroll
    for (int q4 = 0; q4 < 4; ++q4) {
      const int r4 = 32 * half + 8 * q4 + 4 * h;
      const f32x4 ls = *reinterpret_cast<const f32x4*>(&stat[sb][0][r4]);
      const f32x4 dl = *reinterpret_cast<const f32x4*>(&stat[sb][1][r4]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = 4 * q4 + e;
        s[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], c, -ls[e]));
        dp[i] = s[i] * (dp[i] - dl[e]);
      }
    }
    if (r0 + kBN > st.lq || r0 < wlim + 31) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int qi = r0 + 32 * half + reg_row(i, h);
        if (qi < lim || qi >= st.lq) s[i] = 0.0f, dp[i] = 0.0f;
      }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      mine[j] = __builtin_bit_cast(uint4, slab(s, j));
      mine[2 + j] = __builtin_bit_cast(uint4, slab(dp, j));
      if (decltype(fine)::value && r0 < few) rests_of(lds, spare, pair).f[half][j][l] = slab_rest(dp, mine[2 + j], j);
    }
  };
  // the sums over the tile at r0, with the pair's P and dS
  const int begin = q0;
  auto second = [&](auto fine, int r0, int buf, int spare) __attribute__((always_inline)) {
    if (r0 < begin || r0 + kBN <= wlim) return;
    const uint8_t* tile = lds + buf * kTile;
    asm volatile("" : "+v"(rp.n), "+v"(rp.r), "+v"(rp.tn), "+v"(rp.tr));
    bf16x8 f0[4], ds[4];
    pipelined<20, 3>(
        [&](int i) {
          const int j = i / 5, d = i % 5;
          if (d == 0) f0[j] = __builtin_bit_cast(bf16x8, ex.f[pair][j >> 1][op + (j & 1)][l]);
          if (d == 4) ds[j] = __builtin_bit_cast(bf16x8, ex.f[pair][j >> 1][2 + (j & 1)][l]);
          return d < 4 ? wide_tr(tile + side, rp, j, d) : rope_tr(tile + kOffR, rp, j, half);
        },
        [&](int i, bf16x8 f) {
          if (i % 5 < 4) {
            wide[i % 5] = mfma(f, f0[i / 5], wide[i % 5]);
          } else {
            rope = mfma(f, ds[i / 5], rope);
          }
        });
    if (decltype(fine)::value && r0 < few) {
#pragma unroll 1
      for (int j = 0; j < 4; ++j) {
        const bf16x8 rs = __builtin_bit_cast(bf16x8, rests_of(lds, spare, pair).f[j >> 1][j & 1][l]);
        if (half) {
#pragma unroll
          for (int d = 0; d < 4; ++d) wide[d] = mfma(wide_tr(tile, rp, j, d), rs, wide[d]);
        }
        rope = mfma(rope_tr(tile + kOffR, rp, j, half), rs, rope);
      }
    }
  };
  // The second walk: what queries and gradients that are not finite add to this lane's sums: a
  // bit each where it is plus infinity, and minus infinity, both where it is NaN.
  uint64_t pos = 0, neg = 0;                       // wide
  uint32_t nan = 0;                                // rope, always NaN: a query that is not finite
  const int cut = (st.row0 + BM < st.lk ? st.row0 + BM : st.lk) - 1 - diff;   // queries from here on see all keys
  auto cover = [&](int r0, int buf) __attribute__((always_inline)) {
    uint8_t* tile = lds + buf * kTile;
#pragma unroll 1
    for (uint32_t i = 0; i < kBN; ++i) {
      const bool seen = r0 + (int)i >= lim && r0 + (int)i < st.lq;
      const bool zero = handed(ex, pair, i, 0) == 0.0f;   // 0 * infinity
      uint64_t up = 0, down = 0;
#pragma unroll 4
      for (uint32_t u = 0; u < 16; ++u) {          // columns 8 u + 4 h .. + 3
        const uint2 v = *reinterpret_cast<const uint2*>(tile + side + i * 256 + ((u ^ f_wide(i)) << 4) + 8 * h);
        const uint32_t bits = nonfinite4(v), nans = half || zero ? bits : nan4(v);
        const uint32_t minus = (v.x >> 15 & 1) | (v.x >> 30 & 2) | (v.y >> 13 & 4) | (v.y >> 28 & 8);
        up |= (uint64_t)((bits & ~minus) | nans) << (4 * u);
        down |= (uint64_t)((bits & minus) | nans) << (4 * u);
      }
      uint32_t r = 0;
#pragma unroll
      for (uint32_t u = 0; u < 4; ++u)
        r |= nonfinite4(*reinterpret_cast<const uint2*>(tile + kOffR + i * 128 + (((4 * half + u) ^ f_rope(i)) << 4) +
                                                         8 * h)) << (4 * u);
      pos |= seen ? up : 0;
      neg |= seen ? down : 0;
      nan |= seen ? r : 0;
    }
    __syncthreads();
    clear_nonfinite(tile, kTile, 128 * PAIRS);
    __syncthreads();
  };
  // The sums over the queries that see the workgroup's keys.
  float shift = kShift, unshift = kUnshift;
  auto walk = [&](auto again) __attribute__((always_inline)) {
    int q0 = begin, buf = 0, prev = 2, sb = 0;     // this tile, its buffer and the last tile's
    // FINE: there may be second terms, of this tile or of the last, which are in the next copy's way
    auto step = [&](auto fine) __attribute__((always_inline)) {
      constexpr bool FINE = decltype(fine)::value;
      if (w == 0)
        stat[sb][0][l] = z == -__builtin_inff() ? __builtin_inff() : z * kLog2e - shift;   // no keys: P = 0
      else if (w == 1)
        stat[sb][1][l] = z;
      tile_wait();
      const int next = buf == 2 ? 0 : buf + 1;
      const bool late = FINE && q0 > begin;
      if (q0 + kBN < st.lq) {
        z = stat_of(q0 + kBN);
        if (!late) tile_copy<2 * PAIRS>(cp, x.q, x.q + kNope, x.g, q0 + kBN, st.lq, next);
      }
      uint4 mine[4];                               // this wavefront's P and dS slabs
      if (decltype(again)::value && q0 > begin && q0 - kBN < cut) cover(q0 - kBN, prev);
      second(fine, q0 - kBN, prev, next);
      if (FINE) __syncthreads();                   // the last tile and its rests are consumed
      if (late && q0 + kBN < st.lq) tile_copy<2 * PAIRS>(cp, x.q, x.q + kNope, x.g, q0 + kBN, st.lq, next);
      if (q0 < st.lq) first(fine, mine, q0, buf, prev, sb);
      __syncthreads();                             // the last tile's operands are consumed
      if (q0 < st.lq && q0 + kBN > wlim) {
#pragma unroll
        for (int j = 0; j < 4; ++j) ex.f[pair][half][j][l] = mine[j];
      }
      prev = buf;
      buf = next;
      q0 += kBN;
      sb ^= 1;
    };
    if (!decltype(again)::value && begin < few)
      while (q0 < st.lq + kBN && q0 < few + kBN) step(std::true_type{});
    while (q0 < st.lq + kBN) step(std::false_type{});
  };
  auto store = [&](bool write) {
    if (!write) return;
    const int64_t kr = st.k0 + row;
    uint16_t* p = half ? a.dkn.p + kr * a.dkn.ld + head * a.dkn.ldh : a.dv.p + kr * a.dv.ld + head * a.dv.ldh;
    const float mul = half ? a.scale * unshift : unshift;
#pragma unroll
    for (int d = 0; d < 4; ++d) store_block(wide[d], mul, p + 32 * d);
    float* pr = a.rope_part + (head * a.Tk + kr) * kRope + 32 * half + 4 * h;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<f32x4*>(pr + 8 * i) =
          f32x4{rope[4 * i], rope[4 * i + 1], rope[4 * i + 2], rope[4 * i + 3]} * unshift;
  };
  walk(std::false_type{});
  store(row < st.lk);
  if (!a.causal) return;
  // rows that a hidden query or gradient may have reached
  bool nf = any_nonfinite(wide);
#pragma unroll
  for (int i = 0; i < 16; ++i) nf |= !(__builtin_fabsf(rope[i]) < __builtin_inff());
  const uint64_t bad = __ballot(nf && row < st.lk);
  if (l == 0) s_bad[pair][half] = (uint32_t)bad | (uint32_t)(bad >> 32);
  __syncthreads();
  uint32_t any = 0;
#pragma unroll
  for (int i = 0; i < PAIRS; ++i) any |= s_bad[i][0] | s_bad[i][1];
  if (!any || begin >= cut) return;                // uniform over the workgroup
  const uint32_t redo = s_bad[pair][0] | s_bad[pair][1];
  if (begin < st.lq) {
    z = stat_of(begin);
    tile_copy<2 * PAIRS>(cp, x.q, x.q + kNope, x.g, begin, st.lq, 0);
  }
#pragma unroll
  for (int d = 0; d < 4; ++d) wide[d] = f32x16{};
  rope = f32x16{};
  shift = 0.0f;
  unshift = 1.0f;
  walk(std::true_type{});
#pragma unroll
  for (int i = 0; i < 64; ++i) {
    const bool p = (pos >> i) & 1, m = (neg >> i) & 1;
    wide[i / 16][i % 16] += p && m ? __builtin_nanf("") : p ? __builtin_inff() : m ? -__builtin_inff() : 0.0f;
  }
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if ((nan >> i) & 1) rope[i] = __builtin_nanf("");
  store(row < st.lk && ((redo >> n) & 1));
}

// dk_rope[t] = scale * sum over heads, in head order, rounded once.  Four
// columns a lane.  Rows outside every sequence get unspecified values.  Reads its
// parts once: 16384 keys, 16 heads, 67 MB in 12.9 us, 5.2 TB/s.
__global__ __launch_bounds__(kThr) void k_attn_drope(AttnArgs a) {
  const int64_t i = (int64_t)blockIdx.x * kThr + threadIdx.x;
  const int64_t t = i / (kRope / 4);
  const int c = (int)(i % (kRope / 4)) * 4;
  if (t >= a.Tk) return;
  const float* p = a.rope_part + t * kRope + c;
  f32x4 s = {};
#pragma unroll 8
  for (int h = 0; h < a.H; ++h) s += *reinterpret_cast<const f32x4*>(p + h * a.Tk * kRope);
  uint2 w;
  w.x = bf16x2_bits(s[0] * a.scale, s[1] * a.scale);
  w.y = bf16x2_bits(s[2] * a.scale, s[3] * a.scale);
  *reinterpret_cast<uint2*>(a.dkr + t * a.lddr + c) = w;
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

constexpr int64_t kMaxRows = INT64_C(1) << 27, kMaxStride = INT64_C(1) << 23;

inline bool aligned16(const void* p) { return ((uintptr_t)p % 16) == 0; }
inline int launch_status() { return hipGetLastError() == hipSuccess ? MXQ_OK : MXQ_ERR_HIP; }

// Strides of a [rows, heads, cols] operand: 16-byte rows that do not overlap
// in the last dimension.
int check_op(const void* p, int64_t rows, int64_t ld, int64_t ldh, int cols) {
  if (rows == 0) return MXQ_OK;                    // nothing is read or written
  if (!p) return MXQ_ERR_NULL;
  // a staged tile's 64 rows are addressed with 32-bit byte offsets
  if (ld < cols || ldh < cols || ld > kMaxStride) return MXQ_ERR_SHAPE;
  if (ld % 8 != 0 || ldh % 8 != 0 || !aligned16(p)) return MXQ_ERR_ALIGN;
  return MXQ_OK;
}

#define MXQ_TRY(expr)                  \
  do {                                 \
    const int st_ = (expr);            \
    if (st_ != MXQ_OK) return st_;     \
  } while (0)

int check_attn(const mxq_latent_attn* d, AttnArgs* a) {
  if (!d) return MXQ_ERR_NULL;
  if (d->H < 1 || d->H > 65536 || d->Tq < 0 || d->Tk < 0 || d->Tq > kMaxRows || d->Tk > kMaxRows)
    return MXQ_ERR_SHAPE;
  if (d->causal != 0 && d->causal != 1) return MXQ_ERR_ARG;
  if (!(d->scale > 0.0f && d->scale <= kMaxScale)) return MXQ_ERR_ARG;
  if ((d->offsets_q == nullptr) != (d->offsets_k == nullptr)) return MXQ_ERR_NULL;
  if (d->offsets_q && (d->B < 1 || d->B > 65536)) return MXQ_ERR_SHAPE;
  MXQ_TRY(check_op(d->q, d->Tq, d->ldq, d->ldq_head, kQk));
  MXQ_TRY(check_op(d->k_nope, d->Tk, d->ldk, d->ldk_head, kNope));
  MXQ_TRY(check_op(d->k_rope, d->Tk, d->ldr, kRope, kRope));
  MXQ_TRY(check_op(d->v, d->Tk, d->ldv, d->ldv_head, kVal));
  *a = AttnArgs{};
  a->q = {d->q, d->ldq, d->ldq_head};
  a->kn = {d->k_nope, d->ldk, d->ldk_head};
  a->v = {d->v, d->ldv, d->ldv_head};
  a->kr = d->k_rope;
  a->ldr = d->ldr;
  a->offq = d->offsets_q;
  a->offk = d->offsets_k;
  a->B = d->offsets_q ? d->B : 1;
  a->H = d->H;
  a->causal = d->causal;
  a->Tq = d->Tq;
  a->Tk = d->Tk;
  a->scale = d->scale;
  return MXQ_OK;
}

// Workgroups that hold every sequence's tiles of `rows` rows, for all heads.  A
// launch has fewer than 2^32 work items, of which a workgroup has up to 512.
int grid_of(int64_t T, int64_t rows, const AttnArgs& a, uint32_t* n) {
  const int64_t g = sat_mul(T / rows + a.B, a.H);
  if (g >= (INT64_C(1) << 23)) return MXQ_ERR_SHAPE;
  *n = (uint32_t)g;
  return MXQ_OK;
}

}  // namespace

}  // namespace mxq

using namespace mxq;

extern "C" int latent_attention(const mxq_latent_attn* d, uint16_t* o, int64_t ldo,
                                int64_t ldo_head, float* lse, int64_t ldl, void* workspace,
                                size_t workspace_bytes, hipStream_t stream) {
  AttnArgs a;
  MXQ_TRY(check_attn(d, &a));
  MXQ_TRY(check_op(o, a.Tq, ldo, ldo_head, kVal));
  if (a.Tq > 0 && !lse) return MXQ_ERR_NULL;
  if (ldl < a.Tq) return MXQ_ERR_SHAPE;
  if ((uintptr_t)lse % 4 != 0) return MXQ_ERR_ALIGN;
  a.parts = latent_forward_parts(a.Tq, a.Tk, a.H, a.B);
  const size_t need = latent_forward_workspace(a.Tq, a.Tk, a.H, a.B);
  if (workspace_bytes < need) return MXQ_ERR_WORKSPACE;
  if (need > 0 && !workspace) return MXQ_ERR_NULL;
  if (need > 0 && !aligned16(workspace)) return MXQ_ERR_ALIGN;
  if (a.Tq == 0) return MXQ_OK;
  a.out = {o, ldo, ldo_head};
  a.lse = lse;
  a.ldl = ldl;
  uint32_t n;
  MXQ_TRY(grid_of(a.Tq, 128, a, &n));
  if (a.parts == 1) {
    hipLaunchKernelGGL(k_attn_fwd<false>, dim3(n), dim3(kThr), 0, stream, a);
    return launch_status();
  }
  a.part_o = static_cast<float*>(workspace);
  a.part_ml = a.part_o + (int64_t)a.parts * a.H * a.Tq * kVal;
  // few rows, so n times 16 is far from a launch's limit
  hipLaunchKernelGGL(k_attn_fwd<true>, dim3(n * (uint32_t)a.parts), dim3(kThr), 0, stream, a);
  MXQ_TRY(launch_status());
  hipLaunchKernelGGL(k_attn_join, dim3(n * 4), dim3(kThr), 0, stream, a);
  return launch_status();
}

extern "C" int latent_attention_backward(
    const mxq_latent_attn* d, const uint16_t* o, int64_t ldo, int64_t ldo_head, const float* lse,
    int64_t ldl, const uint16_t* dout, int64_t lddo, int64_t lddo_head, uint16_t* dq, int64_t lddq,
    int64_t lddq_head, uint16_t* dk_nope, int64_t lddk, int64_t lddk_head, uint16_t* dk_rope,
    int64_t lddr, uint16_t* dv, int64_t lddv, int64_t lddv_head, void* workspace,
    size_t workspace_bytes, hipStream_t stream) {
  AttnArgs a;
  MXQ_TRY(check_attn(d, &a));
  MXQ_TRY(check_op(o, a.Tq, ldo, ldo_head, kVal));
  MXQ_TRY(check_op(dout, a.Tq, lddo, lddo_head, kVal));
  MXQ_TRY(check_op(dq, a.Tq, lddq, lddq_head, kQk));
  MXQ_TRY(check_op(dk_nope, a.Tk, lddk, lddk_head, kNope));
  MXQ_TRY(check_op(dk_rope, a.Tk, lddr, kRope, kRope));
  MXQ_TRY(check_op(dv, a.Tk, lddv, lddv_head, kVal));
  if (a.Tq > 0 && !lse) return MXQ_ERR_NULL;
  if (ldl < a.Tq) return MXQ_ERR_SHAPE;
  if ((uintptr_t)lse % 4 != 0) return MXQ_ERR_ALIGN;
  const size_t need = latent_backward_workspace(a.Tq, a.Tk, a.H);
  if (workspace_bytes < need) return MXQ_ERR_WORKSPACE;
  if (need > 0 && !workspace) return MXQ_ERR_NULL;
  if (!aligned16(workspace)) return MXQ_ERR_ALIGN;
  const auto few = [&](int64_t T) { return latent_backward_rows(T, a.H, a.B, a.causal) == 64; };
  const bool fewq = few(a.Tq), fewk = few(a.Tk);
  uint32_t nq, nk, nr;
  MXQ_TRY(grid_of(a.Tq, fewq ? 64 : 128, a, &nq));
  MXQ_TRY(grid_of(a.Tk, fewk ? 64 : 128, a, &nk));
  nr = (uint32_t)((a.Tk * (kRope / 4) + kThr - 1) / kThr);     // at most 2^23
  a.o = {o, ldo, ldo_head};
  a.dout = {dout, lddo, lddo_head};
  a.lse = const_cast<float*>(lse);
  a.ldl = ldl;
  a.dq = {dq, lddq, lddq_head};
  a.dkn = {dk_nope, lddk, lddk_head};
  a.dv = {dv, lddv, lddv_head};
  a.dkr = dk_rope;
  a.lddr = lddr;
  a.rope_part = static_cast<float*>(workspace);
  a.delta = a.rope_part + a.H * a.Tk * kRope;
  if (a.Tq > 0) {
    if (fewq)
      hipLaunchKernelGGL(k_attn_dq<2>, dim3(nq), dim3(256), 0, stream, a);
    else
      hipLaunchKernelGGL(k_attn_dq<4>, dim3(nq), dim3(512), 0, stream, a);
    MXQ_TRY(launch_status());
  }
  if (a.Tk > 0) {
    if (fewk)
      hipLaunchKernelGGL(k_attn_dkv<2>, dim3(nk), dim3(256), 0, stream, a);
    else
      hipLaunchKernelGGL(k_attn_dkv<4>, dim3(nk), dim3(512), 0, stream, a);
    MXQ_TRY(launch_status());
    hipLaunchKernelGGL(k_attn_drope, dim3(nr), dim3(kThr), 0, stream, a);
    MXQ_TRY(launch_status());
  }
  return MXQ_OK;
}

extern "C" int mxq_latent_backward_rows(int64_t T, int32_t H, int32_t B, int causal) {
  return T < 0 || H < 1 || B < 1 ? 0 : latent_backward_rows(T, H, B, causal);
}
