// Host-side argument validation of mx_grouped_gemm_swiglu_backward, as ffn.cpp has it for the
// other feed-forward calls: fake device addresses, every case fails a check (its expected
// status) or reaches the launch, which fails without a device (MXQ_ERR_HIP).  Sizes near the
// limits probe the size arithmetic (M + 31 E, 2 F strides, tiles and parts of tiles).
#include <cstdint>
#include <cstdio>

#include "mxq.h"

static int g_fail = 0, g_n = 0;

constexpr int64_t HUGE_ = INT64_MAX, EVEN_ = INT64_MAX / 32 * 32, DIM_ = INT64_C(1) << 39;

struct Args {
  const uint8_t *dy, *dys, *w, *ws;
  int64_t ldd = 64, ldsd = 2, ldw = 64, ldsw = 2, we = 64 * 32, wse = 64;
  const int64_t* offsets;
  int32_t E = 2;
  int64_t M = 40, F = 32, K = 64;
  const uint16_t* gu;
  int64_t ldgu = 64;
  void* dgu;
  int64_t lddgu = 64;
  uint8_t *q, *s, *qT, *sT;
  int64_t ldq = 64, lds = 2, ldqT = 128, ldsT = 4, cap = 128;
  int64_t* poff;
  int accum = 0;
  Args() {
    auto* p = reinterpret_cast<uint8_t*>(uintptr_t(4096));
    dy = dys = w = ws = q = s = qT = sT = p;
    offsets = poff = reinterpret_cast<int64_t*>(p);
    gu = reinterpret_cast<uint16_t*>(p);
    dgu = p;
  }
};

#define CASE(change, want)                                                                       \
  do {                                                                                           \
    Args t;                                                                                      \
    change;                                                                                      \
    ++g_n;                                                                                       \
    const int got_ = mx_grouped_gemm_swiglu_backward(                                            \
        t.dy, t.dys, t.ldd, t.ldsd, t.w, t.ws, t.ldw, t.ldsw, t.we, t.wse, t.offsets, t.E, t.M, t.F, t.K, t.gu, \
        t.ldgu, t.dgu, t.lddgu, t.q, t.ldq, t.s, t.lds, t.qT, t.ldqT, t.sT, t.ldsT, t.cap, t.poff, t.accum, nullptr); \
    if (got_ != (want)) {                                                                        \
      ++g_fail;                                                                                  \
      std::printf("FAIL line %d: %s -> %d, expected %d\n", __LINE__, #change, got_, (int)(want)); \
    }                                                                                            \
  } while (0)

int main() {
  CASE(, MXQ_ERR_HIP);
  CASE(t.accum = 1, MXQ_ERR_HIP);
  CASE(t.M = HUGE_, MXQ_ERR_SHAPE);
  CASE(t.M = INT64_MIN, MXQ_ERR_SHAPE);
  CASE(t.F = EVEN_, MXQ_ERR_SHAPE);
  CASE(t.K = EVEN_, MXQ_ERR_SHAPE);
  CASE(t.cap = EVEN_, MXQ_ERR_SHAPE);
  CASE((t.M = t.cap = t.ldqT = t.ldsT = DIM_, t.E = 256), MXQ_ERR_SHAPE);      // no room for the groups' padding
  CASE((t.M = DIM_ - (1 << 14), t.cap = t.ldqT = DIM_, t.ldsT = DIM_ / 32, t.E = 256), MXQ_ERR_SHAPE);
  CASE((t.M = (INT64_C(1) << 31) - (1 << 14), t.cap = t.ldqT = INT64_C(1) << 31, t.ldsT = t.cap / 32, t.E = 256), MXQ_ERR_HIP);
  CASE((t.F = DIM_ / 2, t.ldgu = t.lddgu = t.ldq = t.lds = DIM_), MXQ_ERR_SHAPE);   // a tile's offsets
  // the widest rows with 257 of them below 2^31 bytes
  CASE((t.F = 2000000 / 32 * 32, t.ldgu = t.lddgu = t.ldq = 2 * t.F, t.lds = t.F / 16, t.E = 256, t.M = 1 << 20,
        t.cap = t.ldqT = 1 << 21, t.ldsT = 1 << 16, t.we = t.F * 64, t.wse = t.F * 2), MXQ_ERR_HIP);
  CASE((t.F = 2100000 / 32 * 32, t.ldgu = t.lddgu = t.ldq = 2 * t.F, t.lds = t.F / 16), MXQ_ERR_SHAPE);
  for (int64_t Args::* ld : {&Args::ldd, &Args::ldsd, &Args::ldw, &Args::ldsw, &Args::we, &Args::wse, &Args::ldgu, &Args::lddgu,
                             &Args::ldq, &Args::lds, &Args::ldqT, &Args::ldsT}) {
    CASE(t.*ld = HUGE_, MXQ_ERR_SHAPE);
    CASE(t.*ld = EVEN_, MXQ_ERR_SHAPE);
    CASE(t.*ld = INT64_MIN, MXQ_ERR_SHAPE);
  }
  CASE(t.E = INT32_MAX, MXQ_ERR_SHAPE);
  CASE(t.E = INT32_MIN, MXQ_ERR_SHAPE);
  CASE((t.M = 0, t.dy = t.dys = t.w = t.ws = nullptr, t.gu = nullptr, t.q = t.s = nullptr), MXQ_ERR_HIP);   // the copy's zeros
  CASE((t.K = 0, t.dy = t.dys = t.w = t.ws = nullptr), MXQ_ERR_HIP);
  CASE((t.dgu = nullptr, t.lddgu = 0, t.poff = nullptr), MXQ_ERR_HIP);

  std::printf("%d checks, %d failed\n", g_n, g_fail);
  return g_fail != 0;
}
