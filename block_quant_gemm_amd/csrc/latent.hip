// The MX latent cache for gfx950: writing tokens into it, reading them back,
// and the absorbed attention of decoding tokens that reads it.
//
// A slot keeps a token's latent vector c (512 values) as E4M3 codes with one
// E8M0 scale per 32 values, and its rotary key (64 values) in BF16: 656 bytes
// instead of 1152.  Absorbed attention multiplies the queries by the latent
// vector itself, which is both key (with the rotary key beside it) and value:
//   z[r, t] = scale * (q[r, :512] . c[t] + q[r, 512:] . k_rope[t])
//   o[r]    = sum_t softmax(z[r])_t c[t]
// so one read of a slot serves every head and every query token of a request.

#include <type_traits>

#include "common.h"

namespace mxq {

namespace {

constexpr int kLat = MXQ_LATENT_DIM, kRope = MXQ_ROPE_DIM, kBlocks = kLat / 32;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kThr = 256;

struct Cache {
  uint8_t* codes;
  uint8_t* scales;
  uint16_t* rope;
  int64_t ldc, lds, ldr, slots;
};

// ---------------------------------------------------------------------------
// Write and read.  Both move bytes: 1816 a token (1152 of BF16, 656 of cache, 8
// of slot number), no arithmetic that shows.  One wavefront a token: lane l
// holds latent values 8 l .. 8 l + 7 (a DPP quad one block of 32), so a token's
// codes are one 512-byte store and its row of BF16 one 1 KB load; lanes 0-7
// carry the rotary key's 16 bytes 16 l.  16384 tokens are written in 6.4 us
// (4.6 TB/s); 65521 are read in 28.2 us (4.2 TB/s), 19.6 us (6.1 TB/s) when the
// last-level cache holds them from the call before.  A large copy reaches 5.0 TB/s.
// ---------------------------------------------------------------------------

__global__ __launch_bounds__(kThr) void k_latent_write(const uint16_t* __restrict__ c, int64_t ldc,
                                                       const uint16_t* __restrict__ k_rope,
                                                       int64_t ldr,
                                                       const int64_t* __restrict__ slots, int64_t T,
                                                       Cache k) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * (kThr / 64) + (threadIdx.x >> 6);
  if (t >= T) return;                              // uniform over the wavefront
  const int64_t s = slots[t];
  const uint4 v = *reinterpret_cast<const uint4*>(c + t * ldc + lane * 8);
  uint4 r = make_uint4(0, 0, 0, 0);
  if (lane < 8) r = *reinterpret_cast<const uint4*>(k_rope + t * ldr + lane * 8);
  uint32_t lo, hi, code;
  quant8(v, lo, hi, code);
  if (s < 0 || s >= k.slots) return;
  *reinterpret_cast<uint2*>(k.codes + s * k.ldc + lane * 8) = make_uint2(lo, hi);
  if ((lane & 3) == 0) k.scales[s * k.lds + (lane >> 2)] = (uint8_t)code;
  if (lane < 8) *reinterpret_cast<uint4*>(k.rope + s * k.ldr + lane * 8) = r;
}

// Two codes of a dword (HI: bytes 2-3) times the scale 2^(e - 127), rounded to
// BF16 once.  Formed in FP32, so that the smallest scales' values round instead
// of losing bits in the conversion.
template <bool HI>
__device__ __forceinline__ uint32_t decode2(uint32_t w, float s) {
  const f32x2 f = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, HI);
  return bf16x2_bits(f[0] * s, f[1] * s);
}

// 2^(e - 127) as FP32: e = 0 is the subnormal 2^-127, e = 0xFF NaN.
__device__ __forceinline__ float scale_f32(uint32_t e) {
  return __builtin_bit_cast(float, e == 0u ? 0x00400000u : e == 0xFFu ? 0x7FC00000u : e << 23);
}

// U tokens a wavefront, kThr / 64 apart.  Loads are unconditional (an absent
// slot's from slot 0) so that all U tokens' leave together.
template <int U>
__global__ __launch_bounds__(kThr) void k_latent_read(Cache k, const int64_t* __restrict__ slots,
                                                      int64_t T, uint16_t* __restrict__ c,
                                                      int64_t ldc, uint16_t* __restrict__ k_rope,
                                                      int64_t ldr) {
  const int lane = threadIdx.x & 63;
  const int64_t t0 = (int64_t)blockIdx.x * (kThr / 64 * U) + (threadIdx.x >> 6);
  int64_t s[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t t = t0 + u * (kThr / 64);
    s[u] = slots[t < T ? t : T - 1];
  }
  uint2 v[U];
  uint4 r[U];
  uint32_t e[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const bool in = s[u] >= 0 && s[u] < k.slots;
    const int64_t x = in ? s[u] : 0;
    v[u] = make_uint2(0, 0);
    r[u] = make_uint4(0, 0, 0, 0);
    e[u] = 127;
    if (k.slots > 0) {
      v[u] = *reinterpret_cast<const uint2*>(k.codes + x * k.ldc + lane * 8);
      e[u] = k.scales[x * k.lds + (lane >> 2)];
      r[u] = *reinterpret_cast<const uint4*>(k.rope + x * k.ldr + (lane & 7) * 8);
    }
    if (!in) {
      v[u] = make_uint2(0, 0);
      r[u] = make_uint4(0, 0, 0, 0);
      e[u] = 127;
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t t = t0 + u * (kThr / 64);
    if (t >= T) break;
    const float f = scale_f32(e[u]);
    uint4 w;
    w.x = decode2<false>(v[u].x, f);
    w.y = decode2<true>(v[u].x, f);
    w.z = decode2<false>(v[u].y, f);
    w.w = decode2<true>(v[u].y, f);
    *reinterpret_cast<uint4*>(c + t * ldc + lane * 8) = w;
    if (lane < 8) *reinterpret_cast<uint4*>(k_rope + t * ldr + lane * 8) = r[u];
  }
}

// ---------------------------------------------------------------------------
// Absorbed attention of decoding tokens.
//
// The rows of one request are its query tokens' heads (row s * H + h).  A
// workgroup takes 16 R G of them (G groups of four wavefronts with 16 R each) and
// a run of one request's 64-token tiles; all runs are about equally long, so
// ragged lengths balance, and a request with more than one leaves parts (FP32
// sums, maximum and total) for k_decode_merge.  A run stays inside a request, so
// a workgroup loads its queries once.  A tile's codes are widened to BF16 once,
// into LDS, exactly (the scale folded in), and serve all rows as keys and
// again, read transposed, as values:
//   logits  wavefront w takes tokens 16 w .. 16 w + 15 against all rows,
//           queries in registers (with 64 rows, 4 of 18 steps; the rest in LDS);
//   values  wavefront w takes 128 latent columns for all rows and 64 tokens.
// So each group reads the tile once per product whatever R is.  Both
// products leave the query row along the lanes, and a lane's probabilities go
// to the same lane of the other wavefronts of its group, rounded to BF16 as the
// matrix unit wants them; maxima, totals and sums stay FP32.
//
// 16 rows (77 KB of LDS, two workgroups a CU: one's loads run beside the other's
// products) are bound by the cache's bytes when requests are long: 6 of 60 to 120
// thousand tokens, 16 heads, 73 to 76 us by machine (71 at best), 4.7 to 4.9 TB/s; a large copy
// reaches 5.0.  96
// requests of 1 to 6000 tokens take 20 us in three tiles a run, 8 of them the chain
// of lengths, page, slot and first tile.  32 and 64 rows take eight wavefronts,
// one workgroup a CU.  24 requests of 300 to 4200 tokens with 128 rows: 32 us, 14
// of them the setup and the parts' stores (25 MB), then 2.9 us a tile, of which
// LDS is busy for 1.9 (the keys once a wavefront, and the queries that registers
// do not hold; at R = 4 they do not fit in any split tried).
// ---------------------------------------------------------------------------

constexpr int kTok = MXQ_LATENT_TILE;            // tokens of a tile
constexpr int kUnits = (kLat + kRope) / 8;       // 16-byte units of a widened row: 72
constexpr int kRowB = kUnits * 16;               // 1152 bytes
constexpr int kSteps = (kLat + kRope) / 32;      // 18 steps of 32 columns
constexpr int kWaves = kThr / 64;

struct DecodeArgs {
  const uint16_t* q;
  int64_t ldq_seq, ldq_tok, ldq_head;
  Cache k;
  const int32_t* pages;
  int64_t ldp;
  int64_t npages;                                // pages in the pool
  uint32_t page, page_mul, page_shift;           // t / page == t * page_mul >> page_shift
  int32_t max_pages;                             // entries in a row of `pages`
  const int64_t* lens;
  int32_t B, S, H, rows;
  int64_t max_len;
  float scale;
  uint32_t runs;                                 // runs to aim at
  uint16_t* o;
  int64_t ldo_seq, ldo_tok, ldo_head;
  float* lse;                                    // [B, S, H]
  float* part_o;                                 // [grid.x][row tiles][rows][512]
  float* part_ml;                                // [grid.x][row tiles][rows][2]
  uint2* runs_of;                                // [B]: a request's first run, and runs
};

// Units of a widened row go to slots so that a lane that widens 16 codes
// (units 2 i, 2 i + 1) stores each half beside its neighbours' halves: unit
// 2 i is slot i, unit 2 i + 1 slot 32 + i, the rotary key's units 64..71 stay.
// The sum over columns takes any order, so queries are loaded in slot order;
// results are stored back in unit order.
__device__ __forceinline__ int slot_unit(int s) {
  return s < 32 ? 2 * s : s < 64 ? 2 * (s - 32) + 1 : s;
}
// Slots of row r are permuted by an XOR: 16 rows at one slot, and 8 consecutive
// rows at 2 consecutive slots (transposed reads), cover a 256-byte bank line once.
__device__ __forceinline__ uint32_t fd(uint32_t r) { return (((r >> 1) & 3) << 1) | ((r >> 3) & 1); }

typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) i16x4 lds_i16x4;

__device__ __forceinline__ f32x4 mfma16(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Maximum / sum over the four 16-lane groups.
__device__ __forceinline__ float groups_max(float x) {
  uint32_t u = __builtin_bit_cast(uint32_t, x);
  auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  x = __builtin_fmaxf(__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1]));
  u = __builtin_bit_cast(uint32_t, x);
  r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __builtin_fmaxf(__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1]));
}
__device__ __forceinline__ float groups_sum(float x) {
  uint32_t u = __builtin_bit_cast(uint32_t, x);
  auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  x = __builtin_bit_cast(float, (uint32_t)r[0]) + __builtin_bit_cast(float, (uint32_t)r[1]);
  u = __builtin_bit_cast(uint32_t, x);
  r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __builtin_bit_cast(float, (uint32_t)r[0]) + __builtin_bit_cast(float, (uint32_t)r[1]);
}

// Tokens of sequence b, cut to max_len, and its tiles: at least one, so that
// an empty sequence's rows are written too.
__device__ __forceinline__ int seq_len(const DecodeArgs& a, int32_t b) {
  const int64_t n = a.lens[b];
  return (int)(n < 0 ? 0 : n > a.max_len ? a.max_len : n);
}
__device__ __forceinline__ uint32_t seq_tiles(int len) {
  return len > 0 ? (uint32_t)((len + kTok - 1) / kTok) : 1u;
}

// This lane's sequence base + lane: its tiles, 0 past the batch.
__device__ __forceinline__ uint32_t lane_tiles(const DecodeArgs& a, int32_t base) {
  const int32_t b = base + (int32_t)(threadIdx.x & 63);
  return b < a.B ? seq_tiles(seq_len(a, b)) : 0u;
}

// The slot of token t of a request with this page table, or -1: past the end,
// or a page outside the pool.
__device__ __forceinline__ int32_t slot_of(const DecodeArgs& a, const int32_t* pages, uint32_t t, int len) {
  if (t >= (uint32_t)len) return -1;
  const uint32_t p = (uint32_t)(((uint64_t)t * a.page_mul) >> a.page_shift);
  if (p >= (uint32_t)a.max_pages) return -1;
  const int32_t pg = pages[p];
  if (pg < 0 || pg >= a.npages) return -1;
  return (int32_t)((int64_t)pg * a.page + (t - p * a.page));
}

// Four latent columns of a finished row.
__device__ __forceinline__ uint2 bf16x4_bits(f32x4 v, float mul) {
  return make_uint2(bf16x2_bits(v[0] * mul, v[1] * mul), bf16x2_bits(v[2] * mul, v[3] * mul));
}

template <int R, int G>
__global__ __launch_bounds__(kThr * G, R * G == 1 ? 2 : G) void k_decode(DecodeArgs a) {
  constexpr int kRows = 16 * R * G;                // query rows of the workgroup
  constexpr int kCl = kTok * 32 / (kThr * G), kRl = kTok * 8 / (kThr * G);   // loads a lane
  __shared__ __attribute__((aligned(256))) uint8_t tile[kTok * kRowB];
  __shared__ __attribute__((aligned(16))) uint2 s_p[kWaves][R * G][64];
  __shared__ float s_max[kWaves][kRows];
  __shared__ int32_t s_slot[2][kTok];
  __shared__ uint32_t s_redo[kRows];
  // steps of the queries held in registers; the others are read from LDS, in lane order
  constexpr int KQ = R == 1 ? kSteps : 4;
  __shared__ __attribute__((aligned(16))) uint4 s_q[R * G][KQ < kSteps ? kSteps - KQ : 1][KQ < kSteps ? 64 : 1];
  const int tid = threadIdx.x, l = tid & 63, n = l & 15, g = l >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int w = wave & 3, rg = (wave >> 2) * R;    // part of the tile; first of its 16-row groups
  const int rt = blockIdx.y;

  // the request and the run of its tiles that this workgroup takes
  // (`runs` runs hold the whole batch's tiles; each sequence adds at most one
  // run that is shorter)
  int32_t b = -1;
  uint32_t k = 0, nrun = 0;                        // run k of nrun
  {
    const uint32_t first = lane_tiles(a, 0);       // of the first 64 sequences, kept
    uint32_t total = 0;
    for (int32_t base = 0; base < a.B; base += 64)
      total += lane_u32(wave_scan(base == 0 ? first : lane_tiles(a, base)), 63);
    const uint32_t per = (total + a.runs - 1) / a.runs;
    uint32_t before = 0;
    for (int32_t base = 0; base < a.B; base += 64) {
      const uint32_t own = ((base == 0 ? first : lane_tiles(a, base)) + per - 1) / per;
      const uint32_t incl = wave_scan(own);
      const uint64_t past = __ballot(blockIdx.x < before + incl);
      if (past) {
        const int at = __builtin_ctzll(past);
        b = base + at;
        nrun = lane_u32(own, at);
        k = blockIdx.x - before - lane_u32(incl - own, at);
        break;
      }
      before += lane_u32(incl, 63);
    }
  }
  if (b < 0) return;                               // uniform over the workgroup
  if (k == 0 && rt == 0 && tid == 0) a.runs_of[b] = make_uint2(blockIdx.x, nrun);   // for the merge
  const int len = seq_len(a, b);
  const uint32_t ntile = seq_tiles(len);
  const uint32_t i0 = (uint32_t)((uint64_t)k * ntile / nrun);
  const uint32_t i1 = (uint32_t)((uint64_t)(k + 1) * ntile / nrun);   // > i0: nrun <= ntile
  const int32_t* pages = a.pages + (int64_t)b * a.ldp;

  // where this lane writes and reads in the tile (bytes); what varies from
  // step to step are constants and single bits
  const uint32_t r0 = tid >> 5, ch = tid & 31;
  const uint32_t wr = r0 * kRowB + ((ch ^ fd(r0)) << 4);
  const uint32_t wrr = (tid >> 3) * kRowB + ((64 + ((tid & 7) ^ fd(tid >> 3))) << 4);
  const uint32_t rk = (16 * w + n) * kRowB + ((g ^ fd(n)) << 4);
  const uint32_t trow = 4 * g + (n >> 2);
  const uint32_t rv = trow * kRowB + w * 256 + ((((n & 3) >> 1) ^ fd(trow)) << 4) + (n & 1) * 8;

  auto put_slot = [&](uint32_t i) {                // slots of tile i, by the first wavefront
    if (wave == 0) s_slot[i & 1][l] = i < i1 ? slot_of(a, pages, i * kTok + l, len) : -1;
  };
  // Loads are unconditional (an absent token's from slot 0) so that they leave
  // together; `gone` marks what has to be zeroed when the tile is widened.
  uint4 sc[kCl], sr[kRl];
  uint32_t se[kCl], gone = ~0u;
  auto load = [&](uint32_t i) {
    int32_t s[kCl], t[kRl];
#pragma unroll
    for (int j = 0; j < kCl; ++j) s[j] = s_slot[i & 1][j * (8 * G) + r0];
#pragma unroll
    for (int j = 0; j < kRl; ++j) t[j] = s_slot[i & 1][j * (32 * G) + (tid >> 3)];
    gone = 0;
#pragma unroll
    for (int j = 0; j < kCl; ++j) {
      gone |= s[j] < 0 ? 1u << j : 0u;
      const int32_t x = s[j] < 0 ? 0 : s[j];
      sc[j] = *reinterpret_cast<const uint4*>(a.k.codes + x * a.k.ldc + ch * 16);
      se[j] = a.k.scales[x * a.k.lds + (ch >> 1)];
    }
#pragma unroll
    for (int j = 0; j < kRl; ++j) {
      gone |= t[j] < 0 ? 256u << j : 0u;
      const int32_t x = t[j] < 0 ? 0 : t[j];
      sr[j] = *reinterpret_cast<const uint4*>(a.k.rope + x * a.k.ldr + (tid & 7) * 8);
    }
  };
  put_slot(i0);
  put_slot(i0 + 1);
  if (tid < kRows) s_redo[tid] = 0;

  // queries: lane (n, g) holds slot 4 kk + g of row n for each step kk
  bf16x8 q[R][KQ];
  int lim[R];                                      // tokens below lim are seen by this lane's row
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int row = rt * kRows + (rg + r) * 16 + n;
    const int s = row / a.H, h = row - s * a.H;
    const bool ok = row < a.rows;
    lim[r] = ok ? len - (a.S - 1 - s) : 0;
    const uint16_t* qp = a.q + (int64_t)b * a.ldq_seq + (int64_t)s * a.ldq_tok + (int64_t)h * a.ldq_head;
    auto step = [&](int kk) {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (ok) v = *reinterpret_cast<const uint4*>(qp + slot_unit(4 * kk + g) * 8);
      return v;
    };
#pragma unroll
    for (int kk = 0; kk < KQ; ++kk) q[r][kk] = __builtin_bit_cast(bf16x8, step(kk));
    if (KQ < kSteps)
      for (int kk = KQ + w; kk < kSteps; kk += 4) s_q[rg + r][kk - KQ][l] = step(kk);
  }
  f32x4 o[R][8];
  float m[R], sum[R];
  const float c = a.scale * kLog2e;
  // The second walk, a tile that not all query tokens see: takes what is not finite out of it,
  // and notes which of this lane's sums would have had it from tokens that their row sees.
  uint32_t nan[R];
  auto cover = [&](uint32_t i) __attribute__((always_inline)) {
#pragma unroll 1
    for (uint32_t t = 0; t < kTok; ++t) {
      uint32_t bits = 0;
#pragma unroll
      for (int d = 0; d < 8; ++d) {
        const uint32_t slot = 16 * w + 2 * d + (g >> 1);
        bits |= nonfinite4(*reinterpret_cast<const uint2*>(tile + t * kRowB + ((slot ^ fd(t)) << 4) + 8 * (g & 1)))
                << (4 * d);
      }
#pragma unroll
      for (int r = 0; r < R; ++r) nan[r] |= (int)(i * kTok + t) < lim[r] ? bits : 0u;
    }
    __syncthreads();
    clear_nonfinite(tile, kTok * kRowB, kThr * G);
    __syncthreads();
  };
  // The sums over the run's tokens.
  auto walk = [&](auto again) __attribute__((always_inline)) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      m[r] = -__builtin_inff();
      sum[r] = 0.0f;
#pragma unroll
      for (int d = 0; d < 8; ++d) o[r][d] = f32x4{};
    }
    __syncthreads();
    if (a.k.slots > 0) load(i0);
    for (uint32_t i = i0; i < i1; ++i) {
      __syncthreads();                               // the last tile is consumed
      if (__ballot(gone != 0)) {
#pragma unroll
        for (int j = 0; j < kCl; ++j)
          if ((gone >> j) & 1) sc[j] = make_uint4(0, 0, 0, 0), se[j] = 127;
#pragma unroll
        for (int j = 0; j < kRl; ++j)
          if ((gone >> (8 + j)) & 1) sr[j] = make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int j = 0; j < kCl; ++j) {
        const float f = e8m0_f32(se[j]);
        uint8_t* p = tile + (G == 1 ? wr ^ ((j & 1) << 4) : wr) + j * (8 * G * kRowB);
        *reinterpret_cast<bf16x8*>(p) = widen8_bf16(sc[j].x, sc[j].y, f);
        *reinterpret_cast<bf16x8*>(p + 512) = widen8_bf16(sc[j].z, sc[j].w, f);
      }
#pragma unroll
      for (int j = 0; j < kRl; ++j)
        *reinterpret_cast<uint4*>(tile + wrr + j * (32 * G * kRowB)) = sr[j];
      __syncthreads();
      if (i + 1 < i1 && a.k.slots > 0) load(i + 1);

      f32x4 s[R] = {}, s2[R] = {};                   // two chains a row group
      struct Step {
        bf16x8 k, q[R];
      };
      pipelined<kSteps, (R == 1 ? 4 : 3)>(
          [&](int kk) {
            Step x;
            x.k = *reinterpret_cast<const bf16x8*>(tile + (rk ^ ((kk & 1) << 6)) + (kk >> 1) * 128);
            if (kk >= KQ) {
#pragma unroll
              for (int r = 0; r < R; ++r)
                x.q[r] = __builtin_bit_cast(bf16x8, s_q[rg + r][kk < KQ ? 0 : kk - KQ][l]);
            }
            return x;
          },
          [&](int kk, const Step& x) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
              const bf16x8 qf = kk < KQ ? q[r][kk < KQ ? kk : 0] : x.q[r];
              if (kk & 1)
                s2[r] = mfma16(x.k, qf, s2[r]);
              else
                s[r] = mfma16(x.k, qf, s[r]);
            }
          });
#pragma unroll
      for (int r = 0; r < R; ++r) s[r] += s2[r];
      const int tok0 = (int)(i * kTok) + 16 * w + 4 * g;   // this lane's 4 tokens
#pragma unroll
      for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (tok0 + e >= lim[r]) s[r][e] = -__builtin_inff();
        const float mx = groups_max(__builtin_fmaxf(__builtin_fmaxf(s[r][0], s[r][1]),
                                                    __builtin_fmaxf(s[r][2], s[r][3])));
        if (g == 0) s_max[w][(rg + r) * 16 + n] = mx;
      }
      __syncthreads();
      put_slot(i + 2);                               // its loads are a whole tile away
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float mn = m[r];
#pragma unroll
        for (int x = 0; x < kWaves; ++x) mn = __builtin_fmaxf(mn, s_max[x][(rg + r) * 16 + n] * c);
        if (__ballot(mn != m[r])) {
          const float alpha = mn == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f(m[r] - mn);
          m[r] = mn;
          sum[r] *= alpha;
#pragma unroll
          for (int d = 0; d < 8; ++d) o[r][d] *= alpha;
        }
        const float mc = mn == -__builtin_inff() ? 0.0f : mn;
        float p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          p[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[r][e], c, -mc));
          sum[r] += p[e];
        }
        s_p[w][rg + r][l] = make_uint2(bf16x2_bits(p[0], p[1]), bf16x2_bits(p[2], p[3]));
      }
      __syncthreads();
      if (decltype(again)::value && (int)(i + 1) * kTok > len - (a.S - 1)) cover(i);
      // values: tokens 4 g + 0..3 of two wavefronts' 16 a step of 32
      bf16x8 pf[2][R];
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const uint2 x = s_p[2 * j][rg + r][l], y = s_p[2 * j + 1][rg + r][l];
          pf[j][r] = __builtin_bit_cast(bf16x8, make_uint4(x.x, x.y, y.x, y.y));
        }
      pipelined<16, (R == 1 ? 4 : 3)>(
          [&](int i2) {
            const int j = i2 >> 3, d = i2 & 7;
            const uint8_t* p = tile + (rv ^ ((d & 3) << 5)) + (d >> 2) * 128 + j * (32 * kRowB);
            const i16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)p);
            const i16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(p + 16 * kRowB));
            return __builtin_bit_cast(bf16x8, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
          },
          [&](int i2, bf16x8 vf) {
#pragma unroll
            for (int r = 0; r < R; ++r) o[r][i2 & 7] = mfma16(vf, pf[i2 >> 3][r], o[r][i2 & 7]);
          });
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r) {                  // totals of all wavefronts' tokens
      const float x = groups_sum(sum[r]);
      if (g == 0) s_max[w][(rg + r) * 16 + n] = x;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r) {
      sum[r] = 0.0f;
#pragma unroll
      for (int x = 0; x < kWaves; ++x) sum[r] += s_max[x][(rg + r) * 16 + n];
    }
  };
  const int64_t part = ((int64_t)blockIdx.x * gridDim.y + rt) * kRows;
  // this lane's rows, `all` or those marked: the results, or their parts
  auto store = [&](bool all) __attribute__((always_inline)) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int row = rt * kRows + (rg + r) * 16 + n;
      const float total = sum[r];
      const bool mine = row < a.rows && (all || s_redo[(rg + r) * 16 + n] != 0);
      if (nrun == 1) {
        const int sq = row / a.H, h = row - sq * a.H;
        uint16_t* op = a.o + (int64_t)b * a.ldo_seq + (int64_t)sq * a.ldo_tok + (int64_t)h * a.ldo_head;
        const float inv = total == 0.0f ? 0.0f : 1.0f / total;
        if (mine) {
#pragma unroll
          for (int d = 0; d < 8; ++d)
            *reinterpret_cast<uint2*>(op + slot_unit(16 * w + 2 * d + (g >> 1)) * 8 + 4 * (g & 1)) =
                bf16x4_bits(o[r][d], inv);
        }
        if (mine && w == 0 && g == 0)
          a.lse[(int64_t)b * a.rows + row] =
              total == 0.0f ? -__builtin_inff() : kLn2 * (m[r] + __builtin_amdgcn_logf(total));
      } else {
        const int64_t pr = part + (rg + r) * 16 + n;
        if (mine) {
#pragma unroll
          for (int d = 0; d < 8; ++d)
            *reinterpret_cast<f32x4*>(a.part_o + pr * kLat + slot_unit(16 * w + 2 * d + (g >> 1)) * 8 +
                                      4 * (g & 1)) = o[r][d];
        }
        if (mine && w == 0 && g == 0) {
          a.part_ml[2 * pr] = m[r];
          a.part_ml[2 * pr + 1] = total;
        }
      }
    }
  };
  walk(std::false_type{});
  store(true);
  // Query tokens that do not see a tile's last tokens still multiply them, by 0, and a NaN
  // there leaves a NaN.  A workgroup with such rows walks its run again.
  if (a.S == 1 || (int)i1 * kTok <= len - (a.S - 1)) return;   // all of the run is seen by all
#pragma unroll
  for (int r = 0; r < R; ++r) {
    bool bad = false;
#pragma unroll
    for (int d = 0; d < 8; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e) bad |= !(__builtin_fabsf(o[r][d][e]) < __builtin_inff());
    if (bad && sum[r] == sum[r]) s_redo[(rg + r) * 16 + n] = 1;   // a row that sees a NaN has a NaN total
  }
  __syncthreads();
  if (!__ballot(s_redo[l % kRows] != 0)) return;   // uniform over the workgroup
  put_slot(i0);
  put_slot(i0 + 1);
#pragma unroll
  for (int r = 0; r < R; ++r) nan[r] = 0;
  walk(std::true_type{});
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int e = 0; e < 32; ++e)
      if ((nan[r] >> e) & 1) o[r][e / 4][e % 4] = __builtin_nanf("");
  store(false);
}

// Joins the parts of the requests that more than one workgroup worked on, in
// their order: with M = max m, o = sum 2^(m - M) O / sum 2^(m - M) l.  One
// workgroup a row, 128 lanes of 4 columns, GROUPS such groups taking every
// GROUPS-th part.  Reads what k_decode wrote last (5 us for 96 requests of 16 rows
// and 418 parts, 7.5 us for 6 of 84 parts each), little more than a launch takes.
template <int GROUPS>
__global__ __launch_bounds__(128 * GROUPS) void k_decode_merge(DecodeArgs a, uint32_t nrt, int rows_per_tile) {
  __shared__ __attribute__((aligned(16))) float s_o[GROUPS > 1 ? GROUPS - 1 : 1][kLat];
  __shared__ float s_l[GROUPS];
  const int32_t b = (int32_t)(blockIdx.x / (uint32_t)a.rows);
  const int row = (int)(blockIdx.x % (uint32_t)a.rows);
  const uint2 runs = a.runs_of[b];
  const uint32_t g0 = runs.x, n = runs.y;
  if (n == 1) return;                              // written whole; uniform
  const int rt = row / rows_per_tile, rr = row % rows_per_tile;
  auto part_row = [&](uint32_t x) { return ((int64_t)(g0 + x) * nrt + rt) * rows_per_tile + rr; };
  float mx = -__builtin_inff();
  for (uint32_t x = threadIdx.x & 63; x < n; x += 64)
    mx = __builtin_fmaxf(mx, a.part_ml[2 * part_row(x)]);
#pragma unroll
  for (int sh = 32; sh > 0; sh >>= 1) mx = __builtin_fmaxf(mx, __shfl_xor(mx, sh, 64));
  const float ref = mx == -__builtin_inff() ? 0.0f : mx;
  const int grp = threadIdx.x >> 7, d = (threadIdx.x & 127) * 4;
  f32x4 acc = {};
  float lsum = 0.0f;
#pragma unroll 4
  for (uint32_t x = grp; x < n; x += GROUPS) {
    const int64_t pr = part_row(x);
    const float f = __builtin_amdgcn_exp2f(a.part_ml[2 * pr] - ref);
    lsum = __builtin_fmaf(f, a.part_ml[2 * pr + 1], lsum);
    const f32x4 v = *reinterpret_cast<const f32x4*>(a.part_o + pr * kLat + d);
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] = __builtin_fmaf(f, v[e], acc[e]);
  }
  if (grp > 0) *reinterpret_cast<f32x4*>(&s_o[grp - 1][d]) = acc;
  if ((threadIdx.x & 127) == 0) s_l[grp] = lsum;
  __syncthreads();
  if (grp > 0) return;
#pragma unroll
  for (int y = 0; y < GROUPS - 1; ++y) acc += *reinterpret_cast<const f32x4*>(&s_o[y][d]);
  float total = 0.0f;
#pragma unroll
  for (int y = 0; y < GROUPS; ++y) total += s_l[y];
  const int sq = row / a.H, h = row - sq * a.H;
  uint16_t* op = a.o + (int64_t)b * a.ldo_seq + (int64_t)sq * a.ldo_tok + (int64_t)h * a.ldo_head;
  *reinterpret_cast<uint2*>(op + d) = bf16x4_bits(acc, total == 0.0f ? 0.0f : 1.0f / total);
  if (threadIdx.x == 0)
    a.lse[(int64_t)b * a.rows + row] =
        total == 0.0f ? -__builtin_inff() : kLn2 * (ref + __builtin_amdgcn_logf(total));
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

inline bool aligned16(const void* p) { return ((uintptr_t)p % 16) == 0; }
inline int launch_status() { return hipGetLastError() == hipSuccess ? MXQ_OK : MXQ_ERR_HIP; }

#define MXQ_TRY(expr)              \
  do {                             \
    const int st_ = (expr);        \
    if (st_ != MXQ_OK) return st_; \
  } while (0)

int check_cache(const mxq_latent_cache* d, Cache* k) {
  if (!d) return MXQ_ERR_NULL;
  // slots are held in 32 bits; addresses in 64
  if (d->slots < 0 || d->slots > 0x7FFFFFFFLL) return MXQ_ERR_SHAPE;
  if (d->slots > 0 && (!d->codes || !d->scales || !d->k_rope)) return MXQ_ERR_NULL;
  if (d->ld_codes < kLat || d->ld_scales < kBlocks || d->ld_rope < kRope) return MXQ_ERR_SHAPE;
  if (d->ld_codes % 16 != 0 || d->ld_rope % 8 != 0 || !aligned16(d->codes) || !aligned16(d->k_rope))
    return MXQ_ERR_ALIGN;
  *k = {d->codes, d->scales, d->k_rope, d->ld_codes, d->ld_scales, d->ld_rope, d->slots};
  return MXQ_OK;
}

int check_rows(const uint16_t* c, int64_t ldc, const uint16_t* r, int64_t ldr, const int64_t* slots,
               int64_t T) {
  if (T < 0 || T > MXQ_LATENT_MAX_TOKENS) return MXQ_ERR_SHAPE;   // 64 T work items a launch
  if (T == 0) return MXQ_OK;
  if (!c || !r || !slots) return MXQ_ERR_NULL;
  if (ldc < kLat || ldr < kRope) return MXQ_ERR_SHAPE;
  if (ldc % 8 != 0 || ldr % 8 != 0 || !aligned16(c) || !aligned16(r) || (uintptr_t)slots % 8 != 0)
    return MXQ_ERR_ALIGN;
  return MXQ_OK;
}

}  // namespace

}  // namespace mxq

using namespace mxq;

extern "C" int mx_latent_cache_write(const uint16_t* c, int64_t ldc, const uint16_t* k_rope,
                                     int64_t ldr, const int64_t* slots, int64_t T,
                                     const mxq_latent_cache* cache, hipStream_t stream) {
  Cache k;
  MXQ_TRY(check_cache(cache, &k));
  MXQ_TRY(check_rows(c, ldc, k_rope, ldr, slots, T));
  if (T == 0) return MXQ_OK;
  hipLaunchKernelGGL(k_latent_write, dim3((uint32_t)((T + 3) / 4)), dim3(kThr), 0, stream, c,
                     ldc, k_rope, ldr, slots, T, k);
  return launch_status();
}

extern "C" int mx_latent_cache_read(const mxq_latent_cache* cache, const int64_t* slots, int64_t T,
                                    uint16_t* c, int64_t ldc, uint16_t* k_rope, int64_t ldr,
                                    hipStream_t stream) {
  Cache k;
  MXQ_TRY(check_cache(cache, &k));
  MXQ_TRY(check_rows(c, ldc, k_rope, ldr, slots, T));
  if (T == 0) return MXQ_OK;
  // Four tokens a wavefront where that still leaves eight workgroups to every CU
  // (65521 tokens whose cache and outputs are in no cache: 28.2 us against 30.3 with
  // one), else one (419 tokens: 2.2 us against 2.8).
  if (T >= 256 * 8 * 16)
    hipLaunchKernelGGL(k_latent_read<4>, dim3((uint32_t)((T + 15) / 16)), dim3(kThr), 0, stream, k,
                       slots, T, c, ldc, k_rope, ldr);
  else
    hipLaunchKernelGGL(k_latent_read<1>, dim3((uint32_t)((T + 3) / 4)), dim3(kThr), 0, stream, k,
                       slots, T, c, ldc, k_rope, ldr);
  return launch_status();
}

extern "C" int mx_latent_decode(const uint16_t* q, int64_t ldq_seq, int64_t ldq_tok,
                                int64_t ldq_head, const mxq_latent_cache* cache,
                                const int32_t* pages, int64_t ld_pages, int32_t max_pages,
                                int32_t page_size, const int64_t* lens, int32_t B, int32_t S,
                                int32_t H, int64_t max_len, float scale, uint16_t* o,
                                int64_t ldo_seq, int64_t ldo_tok, int64_t ldo_head, float* lse,
                                void* workspace, size_t workspace_bytes, hipStream_t stream) {
  DecodeArgs a{};
  MXQ_TRY(check_cache(cache, &a.k));
  if (B < 0 || S < 1 || H < 1 || max_pages < 0 || page_size < 1 || max_len < 0) return MXQ_ERR_SHAPE;
  // the merge launches a workgroup of 256 a row (of 1024 only where B <= 32)
  if (sat_mul(S, H) > 65536 || sat_mul(B, sat_mul(S, H)) >= (INT64_C(1) << 24)) return MXQ_ERR_SHAPE;
  // tokens are counted in 32 bits, and every sequence's pages must be in the table
  if (max_len > (INT64_C(1) << 30) || max_len > sat_mul(max_pages, page_size)) return MXQ_ERR_SHAPE;
  if (!(scale > 0.0f && scale <= kMaxScale)) return MXQ_ERR_ARG;
  if (B == 0) return MXQ_OK;
  if (ldq_head < kLat + kRope || ldq_tok < kLat + kRope || ldq_seq < kLat + kRope ||
      ldo_head < kLat || ldo_tok < kLat || ldo_seq < kLat || ld_pages < max_pages)
    return MXQ_ERR_SHAPE;
  if (!q || !lens || !o || !lse || (max_len > 0 && !pages)) return MXQ_ERR_NULL;
  if (ldq_seq % 8 != 0 || ldq_tok % 8 != 0 || ldq_head % 8 != 0 || ldo_seq % 4 != 0 ||
      ldo_tok % 4 != 0 || ldo_head % 4 != 0 || !aligned16(q) || (uintptr_t)o % 8 != 0 ||
      (uintptr_t)lens % 8 != 0 || (uintptr_t)lse % 4 != 0 || (uintptr_t)pages % 4 != 0)
    return MXQ_ERR_ALIGN;
  const LatentDecodePlan p = latent_decode_plan(B, S, H, max_len);
  if (p.grid == 0) return MXQ_ERR_SHAPE;
  if (workspace_bytes < p.bytes) return MXQ_ERR_WORKSPACE;
  if (!workspace) return MXQ_ERR_NULL;
  if (!aligned16(workspace)) return MXQ_ERR_ALIGN;
  a.q = q;
  a.ldq_seq = ldq_seq; a.ldq_tok = ldq_tok; a.ldq_head = ldq_head;
  a.pages = pages; a.ldp = ld_pages; a.npages = a.k.slots / page_size; a.max_pages = max_pages;
  a.page = (uint32_t)page_size;
  // t / page for t < 2^31: with 2^e >= page, ceil(2^(31 + e) / page) times t
  // exceeds the exact quotient by less than 1 / page
  uint32_t e = 0;
  while ((UINT64_C(1) << e) < (uint64_t)page_size) ++e;
  a.page_shift = 31 + e;
  a.page_mul = (uint32_t)(((UINT64_C(1) << (31 + e)) + page_size - 1) / page_size);
  a.lens = lens;
  a.B = B; a.S = S; a.H = H; a.rows = S * H;
  a.max_len = max_len;
  a.scale = scale;
  a.o = o;
  a.ldo_seq = ldo_seq; a.ldo_tok = ldo_tok; a.ldo_head = ldo_head;
  a.lse = lse;
  a.part_o = static_cast<float*>(workspace);
  a.part_ml = a.part_o + p.part_rows * kLat;
  a.runs_of = reinterpret_cast<uint2*>(a.part_ml + p.part_rows * 2);
  a.runs = p.runs;
  const dim3 grid(p.grid, p.row_tiles);
  if (p.rows == 16)
    hipLaunchKernelGGL((k_decode<1, 1>), grid, dim3(kThr), 0, stream, a);
  else if (p.rows == 32)
    hipLaunchKernelGGL((k_decode<1, 2>), grid, dim3(2 * kThr), 0, stream, a);
  else
    hipLaunchKernelGGL((k_decode<2, 2>), grid, dim3(2 * kThr), 0, stream, a);
  MXQ_TRY(launch_status());
  if (p.grid > 1) {
    // parts a request: about runs / B; few rows with many parts take more groups
    const dim3 rows((uint32_t)((int64_t)B * a.rows));
    if (p.runs / (uint32_t)B >= 16)
      hipLaunchKernelGGL(k_decode_merge<8>, rows, dim3(1024), 0, stream, a, p.row_tiles, p.rows);
    else
      hipLaunchKernelGGL(k_decode_merge<2>, rows, dim3(256), 0, stream, a, p.row_tiles, p.rows);
  }
  return launch_status();
}
