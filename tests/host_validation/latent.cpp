// Host-side argument validation of the latent attention entry points, built with
// AddressSanitizer and UndefinedBehaviorSanitizer on the host code only and run
// where no GPU is visible.  Device pointers are fake addresses that no call
// may dereference: every case either fails a host-side check (its expected
// status) or reaches the launch, which fails without a device (MXQ_ERR_HIP).
// Extreme sizes probe the 64-bit size arithmetic, where an overflow is undefined
// behaviour and stops the run.
#include <cmath>
#include <cstdint>
#include <cstdio>

#include "mxq.h"

static int g_fail = 0, g_n = 0;

#define EXPECT(call, want)                                                               \
  do {                                                                                   \
    ++g_n;                                                                               \
    const long long got_ = (long long)(call);                                            \
    if (got_ != (long long)(want)) {                                                     \
      ++g_fail;                                                                          \
      std::printf("FAIL line %d: %s -> %lld, expected %lld\n", __LINE__, #call, got_,    \
                  (long long)(want));                                                    \
    }                                                                                    \
  } while (0)

// One call's arguments, so that a case changes one of them.
struct Decode {
  const uint16_t* q = reinterpret_cast<const uint16_t*>(uintptr_t(4096));
  int64_t lq_seq = 2 * 576, lq_tok = 2 * 576, lq_head = 576;
  mxq_latent_cache cache{reinterpret_cast<uint8_t*>(uintptr_t(4096)), 512,
                         reinterpret_cast<uint8_t*>(uintptr_t(4096)), 16,
                         reinterpret_cast<uint16_t*>(uintptr_t(4096)), 64, 1024};
  const int32_t* pages = reinterpret_cast<const int32_t*>(uintptr_t(4096));
  int64_t ld_pages = 4;
  int32_t max_pages = 4, page = 64;
  const int64_t* lens = reinterpret_cast<const int64_t*>(uintptr_t(4096));
  int32_t B = 3, S = 1, H = 2;
  int64_t max_len = 200;
  float scale = 0.1f;
  uint16_t* o = reinterpret_cast<uint16_t*>(uintptr_t(4096));
  int64_t lo_seq = 1024, lo_tok = 1024, lo_head = 512;
  float* lse = reinterpret_cast<float*>(uintptr_t(4096));
  void* ws = reinterpret_cast<void*>(uintptr_t(4096));
  size_t ws_bytes = size_t(1) << 40;
  int run() const {
    return mx_latent_decode(q, lq_seq, lq_tok, lq_head, &cache, pages, ld_pages, max_pages, page,
                            lens, B, S, H, max_len, scale, o, lo_seq, lo_tok, lo_head, lse, ws,
                            ws_bytes, nullptr);
  }
};

struct Attn {
  uint16_t* x = reinterpret_cast<uint16_t*>(uintptr_t(4096));
  mxq_latent_attn d{};
  uint16_t* o = x;
  int64_t lo = 256, loh = 128;
  float* lse = reinterpret_cast<float*>(uintptr_t(4096));
  int64_t ll = 100;
  const uint16_t* go = x;
  int64_t lg = 256, lgh = 128;
  uint16_t *dq = x, *dk = x, *dr = x, *dv = x;
  int64_t ldq = 384, ldqh = 192, ldk = 512, ldkh = 256, ldr = 64, ldv = 512, ldvh = 256;
  void* ws = x;
  size_t ws_bytes = size_t(1) << 50;
  Attn() {
    const int64_t* off = reinterpret_cast<const int64_t*>(uintptr_t(4096));
    d.q = x; d.ldq = 384; d.ldq_head = 192;
    d.k_nope = x; d.ldk = 512; d.ldk_head = 256;
    d.k_rope = x; d.ldr = 64;
    d.v = x; d.ldv = 512; d.ldv_head = 256;
    d.offsets_q = d.offsets_k = off;
    d.Tq = 100; d.Tk = 120;
    d.B = 3; d.H = 2;
    d.scale = 0.07f;
    d.causal = 1;
  }
  void* fws = x;
  size_t fws_bytes = size_t(1) << 50;
  int fwd() const { return latent_attention(&d, o, lo, loh, lse, ll, fws, fws_bytes, nullptr); }
  int bwd() const {
    return latent_attention_backward(&d, o, lo, loh, lse, ll, go, lg, lgh, dq, ldq, ldqh, dk, ldk,
                                     ldkh, dr, ldr, dv, ldv, ldvh, ws, ws_bytes, nullptr);
  }
};

// `both` changes an argument of the forward and backward calls
#define ATTN(change, want)            \
  do {                                \
    Attn t;                           \
    change;                           \
    EXPECT(t.fwd(), want);            \
    EXPECT(t.bwd(), want);            \
  } while (0)
#define BACK(change, want) \
  do {                     \
    Attn t;                \
    change;                \
    EXPECT(t.bwd(), want); \
  } while (0)
#define DECODE(change, want) \
  do {                       \
    Decode t;                \
    change;                  \
    EXPECT(t.run(), want);   \
  } while (0)

int main() {
  int ndev = 0;
  if (hipGetDeviceCount(&ndev) == hipSuccess && ndev > 0) {
    std::printf("skipped: a GPU is visible (these calls pass fake device addresses)\n");
    return 0;
  }
  const int64_t BIG = INT64_C(1) << 62, HUGE_ = INT64_MAX;
  uint8_t* P = reinterpret_cast<uint8_t*>(uintptr_t(4096));   // never dereferenced
  uint16_t* X = reinterpret_cast<uint16_t*>(P);
  int64_t* S = reinterpret_cast<int64_t*>(P);
  const int HIP = MXQ_ERR_HIP;
  const float inf = INFINITY;

  // ---- cache write and read ----
  const mxq_latent_cache good{P, 512, P, 16, X, 64, 1024};
  EXPECT(mx_latent_cache_write(X, 576, X, 576, S, 7, &good, nullptr), HIP);
  EXPECT(mx_latent_cache_read(&good, S, 7, X, 512, X, 64, nullptr), HIP);
  EXPECT(mx_latent_cache_write(nullptr, 0, nullptr, 0, nullptr, 0, &good, nullptr), MXQ_OK);
  EXPECT(mx_latent_cache_read(&good, nullptr, 0, nullptr, 0, nullptr, 0, nullptr), MXQ_OK);
  struct Row {
    uint16_t* c; int64_t ldc; uint16_t* r; int64_t ldr; int64_t* s; int64_t T; int want;
  };
  const Row rows[] = {
      {nullptr, 512, X, 64, S, 7, MXQ_ERR_NULL}, {X, 512, nullptr, 64, S, 7, MXQ_ERR_NULL},
      {X, 512, X, 64, nullptr, 7, MXQ_ERR_NULL}, {X, 504, X, 64, S, 7, MXQ_ERR_SHAPE},
      {X, 512, X, 56, S, 7, MXQ_ERR_SHAPE},      {X, 516, X, 64, S, 7, MXQ_ERR_ALIGN},
      {X, 512, X, 66, S, 7, MXQ_ERR_ALIGN},      {X + 4, 512, X, 64, S, 7, MXQ_ERR_ALIGN},
      {X, 512, X + 1, 64, S, 7, MXQ_ERR_ALIGN},  {X, 512, X, 64, S, -1, MXQ_ERR_SHAPE},
      {X, 512, X, 64, S, MXQ_LATENT_MAX_TOKENS, HIP},
      {X, 512, X, 64, S, MXQ_LATENT_MAX_TOKENS + 1, MXQ_ERR_SHAPE},
      {X, 512, X, 64, S, HUGE_, MXQ_ERR_SHAPE},  {X, BIG, X, BIG, S, 7, HIP},
      {X, 512, X, 64, reinterpret_cast<int64_t*>(P + 4), 7, MXQ_ERR_ALIGN},
  };
  for (const Row& r : rows) {
    EXPECT(mx_latent_cache_write(r.c, r.ldc, r.r, r.ldr, r.s, r.T, &good, nullptr), r.want);
    EXPECT(mx_latent_cache_read(&good, r.s, r.T, r.c, r.ldc, r.r, r.ldr, nullptr), r.want);
  }
  EXPECT(mx_latent_cache_write(X, 512, X, 64, S, 7, nullptr, nullptr), MXQ_ERR_NULL);
  EXPECT(mx_latent_cache_read(nullptr, S, 7, X, 512, X, 64, nullptr), MXQ_ERR_NULL);
  struct Bad {
    mxq_latent_cache k; int want;
  };
  const Bad bad[] = {
      {{nullptr, 512, P, 16, X, 64, 8}, MXQ_ERR_NULL}, {{P, 512, nullptr, 16, X, 64, 8}, MXQ_ERR_NULL},
      {{P, 512, P, 16, nullptr, 64, 8}, MXQ_ERR_NULL}, {{P, 496, P, 16, X, 64, 8}, MXQ_ERR_SHAPE},
      {{P, 512, P, 15, X, 64, 8}, MXQ_ERR_SHAPE},      {{P, 512, P, 16, X, 56, 8}, MXQ_ERR_SHAPE},
      {{P, 520, P, 16, X, 64, 8}, MXQ_ERR_ALIGN},      {{P, 512, P, 16, X, 68, 8}, MXQ_ERR_ALIGN},
      {{P + 8, 512, P, 16, X, 64, 8}, MXQ_ERR_ALIGN},  {{P, 512, P, 16, X + 4, 64, 8}, MXQ_ERR_ALIGN},
      {{P, 512, P, 16, X, 64, -1}, MXQ_ERR_SHAPE},     {{P, 512, P, 16, X, 64, BIG}, MXQ_ERR_SHAPE},
      {{P, 656, P + 512, 656, X, 328, 8}, HIP},        // one 656-byte record a slot
      {{nullptr, 512, nullptr, 16, nullptr, 64, 0}, HIP},
  };
  for (const Bad& b : bad) {
    EXPECT(mx_latent_cache_write(X, 512, X, 64, S, 7, &b.k, nullptr), b.want);
    EXPECT(mx_latent_cache_read(&b.k, S, 7, X, 512, X, 64, nullptr), b.want);
    DECODE(t.cache = b.k, b.want);
  }

  // ---- decode ----
  DECODE((void)0, HIP);
  DECODE(t.B = 0; t.q = nullptr, MXQ_OK);
  DECODE(t.B = -1, MXQ_ERR_SHAPE);
  DECODE(t.S = 0, MXQ_ERR_SHAPE);
  DECODE(t.H = 0, MXQ_ERR_SHAPE);
  DECODE(t.S = 65536; t.H = 2, MXQ_ERR_SHAPE);
  DECODE(t.S = INT32_MAX; t.H = INT32_MAX, MXQ_ERR_SHAPE);
  DECODE(t.S = INT32_MAX; t.H = INT32_MAX; t.B = INT32_MAX, MXQ_ERR_SHAPE);
  DECODE(t.B = 1 << 20; t.H = 16, MXQ_ERR_SHAPE);
  DECODE(t.B = 1 << 20; t.H = 8, HIP);
  DECODE(t.page = 0, MXQ_ERR_SHAPE);
  DECODE(t.page = -64, MXQ_ERR_SHAPE);
  DECODE(t.max_pages = -1, MXQ_ERR_SHAPE);
  DECODE(t.max_len = -1, MXQ_ERR_SHAPE);
  DECODE(t.max_len = 257, MXQ_ERR_SHAPE);                     // past the page table
  DECODE(t.max_len = HUGE_, MXQ_ERR_SHAPE);
  DECODE(t.max_len = 0; t.max_pages = 0; t.ld_pages = 0; t.pages = nullptr, HIP);
  DECODE(t.page = INT32_MAX; t.max_len = INT64_C(1) << 30, HIP);
  DECODE(t.page = INT32_MAX; t.max_pages = INT32_MAX; t.ld_pages = HUGE_;
         t.max_len = (INT64_C(1) << 30) + 1, MXQ_ERR_SHAPE);
  DECODE(t.ld_pages = 3, MXQ_ERR_SHAPE);
  DECODE(t.scale = 0.0f, MXQ_ERR_ARG);
  DECODE(t.scale = -1.0f, MXQ_ERR_ARG);
  DECODE(t.scale = inf, MXQ_ERR_ARG);
  DECODE(t.scale = NAN, MXQ_ERR_ARG);
  DECODE(t.q = nullptr, MXQ_ERR_NULL);
  DECODE(t.pages = nullptr, MXQ_ERR_NULL);
  DECODE(t.lens = nullptr, MXQ_ERR_NULL);
  DECODE(t.o = nullptr, MXQ_ERR_NULL);
  DECODE(t.lse = nullptr, MXQ_ERR_NULL);
  DECODE(t.ws = nullptr, MXQ_ERR_NULL);
  DECODE(t.ws = P + 8, MXQ_ERR_ALIGN);
  DECODE(t.ws_bytes = 0, MXQ_ERR_WORKSPACE);
  {
    const size_t need = mxq_workspace_size(MXQ_WS_LATENT_DECODE, 3, 1, 2, 200);
    DECODE(t.ws_bytes = need, HIP);
    DECODE(t.ws_bytes = need - 1, MXQ_ERR_WORKSPACE);
  }
  DECODE(t.lq_head = 568, MXQ_ERR_SHAPE);
  DECODE(t.lq_tok = 0, MXQ_ERR_SHAPE);
  DECODE(t.lq_seq = 64, MXQ_ERR_SHAPE);
  DECODE(t.lo_head = 508, MXQ_ERR_SHAPE);
  DECODE(t.lo_tok = 0, MXQ_ERR_SHAPE);
  DECODE(t.lo_seq = 0, MXQ_ERR_SHAPE);
  DECODE(t.lq_head = 580, MXQ_ERR_ALIGN);
  DECODE(t.lq_seq = 1156, MXQ_ERR_ALIGN);
  DECODE(t.lo_head = 514, MXQ_ERR_ALIGN);
  DECODE(t.q = X + 4, MXQ_ERR_ALIGN);
  DECODE(t.o = X + 2, MXQ_ERR_ALIGN);
  DECODE(t.o = X + 4, HIP);                                   // 8 bytes are enough
  DECODE(t.lens = reinterpret_cast<int64_t*>(P + 4), MXQ_ERR_ALIGN);
  DECODE(t.lse = reinterpret_cast<float*>(P + 2), MXQ_ERR_ALIGN);
  DECODE(t.pages = reinterpret_cast<int32_t*>(P + 2), MXQ_ERR_ALIGN);
  DECODE(t.lq_seq = BIG; t.lo_seq = BIG; t.ld_pages = BIG, HIP);
  for (int64_t x : {INT64_C(0), INT64_C(1), BIG, HUGE_, -HUGE_})
    for (int64_t y : {INT64_C(1), INT64_C(65536), HUGE_})
      (void)mxq_workspace_size(MXQ_WS_LATENT_DECODE, x, y, y, x),
          (void)mxq_workspace_size(MXQ_WS_LATENT_BACKWARD, x, x, y, 0),
          (void)mxq_workspace_size(MXQ_WS_LATENT_FORWARD, x, x, y, y);

  // ---- expanded attention and its gradient ----
  ATTN((void)0, HIP);
  ATTN(t.d.offsets_q = t.d.offsets_k = nullptr; t.d.B = 0, HIP);
  ATTN(t.d.offsets_q = nullptr, MXQ_ERR_NULL);
  ATTN(t.d.offsets_k = nullptr, MXQ_ERR_NULL);
  ATTN(t.d.B = 0, MXQ_ERR_SHAPE);
  ATTN(t.d.B = 65537, MXQ_ERR_SHAPE);
  ATTN(t.d.H = 0, MXQ_ERR_SHAPE);
  ATTN(t.d.H = 65537, MXQ_ERR_SHAPE);
  ATTN(t.d.Tq = -1, MXQ_ERR_SHAPE);
  ATTN(t.d.Tk = -1, MXQ_ERR_SHAPE);
  ATTN(t.d.Tq = (INT64_C(1) << 27) + 1; t.ll = t.d.Tq, MXQ_ERR_SHAPE);
  ATTN(t.d.Tq = HUGE_; t.ll = HUGE_, MXQ_ERR_SHAPE);
  ATTN(t.d.Tq = INT64_C(1) << 27; t.ll = t.d.Tq; t.d.H = 16, MXQ_ERR_SHAPE);   // 2^24 workgroups
  ATTN(t.d.Tq = INT64_C(1) << 27; t.ll = t.d.Tq, HIP);
  ATTN(t.d.B = 65536; t.d.H = 65536, MXQ_ERR_SHAPE);
  BACK(t.d.Tk = INT64_C(1) << 27; t.d.H = 16, MXQ_ERR_SHAPE);
  ATTN(t.d.causal = 2, MXQ_ERR_ARG);
  ATTN(t.d.causal = -1, MXQ_ERR_ARG);
  ATTN(t.d.scale = 0.0f, MXQ_ERR_ARG);
  ATTN(t.d.scale = -0.1f, MXQ_ERR_ARG);
  ATTN(t.d.scale = inf, MXQ_ERR_ARG);
  ATTN(t.d.scale = NAN, MXQ_ERR_ARG);
  ATTN(t.d.q = nullptr, MXQ_ERR_NULL);
  ATTN(t.d.k_nope = nullptr, MXQ_ERR_NULL);
  ATTN(t.d.k_rope = nullptr, MXQ_ERR_NULL);
  ATTN(t.d.v = nullptr, MXQ_ERR_NULL);
  ATTN(t.o = nullptr, MXQ_ERR_NULL);
  ATTN(t.lse = nullptr, MXQ_ERR_NULL);
  ATTN(t.d.ldq = 184, MXQ_ERR_SHAPE);
  ATTN(t.d.ldq_head = 128, MXQ_ERR_SHAPE);
  ATTN(t.d.ldk = 120, MXQ_ERR_SHAPE);
  ATTN(t.d.ldk_head = 0, MXQ_ERR_SHAPE);
  ATTN(t.d.ldr = 56, MXQ_ERR_SHAPE);
  ATTN(t.d.ldv = 0, MXQ_ERR_SHAPE);
  ATTN(t.d.ldv_head = 120, MXQ_ERR_SHAPE);
  ATTN(t.lo = 120, MXQ_ERR_SHAPE);
  ATTN(t.loh = 120, MXQ_ERR_SHAPE);
  ATTN(t.ll = 99, MXQ_ERR_SHAPE);
  ATTN(t.d.ldk = BIG, MXQ_ERR_SHAPE);
  ATTN(t.d.ldk_head = BIG, HIP);
  ATTN(t.d.ldq = 388, MXQ_ERR_ALIGN);
  ATTN(t.d.ldk_head = 132, MXQ_ERR_ALIGN);
  ATTN(t.d.ldr = 68, MXQ_ERR_ALIGN);
  ATTN(t.lo = 260, MXQ_ERR_ALIGN);
  ATTN(t.d.q = t.x + 1, MXQ_ERR_ALIGN);
  ATTN(t.d.v = t.x + 4, MXQ_ERR_ALIGN);
  ATTN(t.o = t.x + 4, MXQ_ERR_ALIGN);
  ATTN(t.lse = reinterpret_cast<float*>(P + 2), MXQ_ERR_ALIGN);
  EXPECT(latent_attention(nullptr, X, 256, 128, nullptr, 100, nullptr, 0, nullptr), MXQ_ERR_NULL);
  {
    Attn t;
    t.d.Tq = 0; t.d.q = nullptr; t.o = nullptr; t.lse = nullptr;
    EXPECT(t.fwd(), MXQ_OK);                                  // nothing to write
    t.go = nullptr; t.dq = nullptr;
    EXPECT(t.bwd(), HIP);                                     // zeros for dk and dv
    t.d.Tk = 0;
    EXPECT(t.bwd(), MXQ_OK);
  }
  {
    Attn t;                                                   // few queries, many keys
    t.d.B = 1;
    t.d.Tk = 8000;
    const size_t need = mxq_workspace_size(MXQ_WS_LATENT_FORWARD, 100, 8000, 2, 1);
    EXPECT(need > 0 && need % (4 * 2 * 100 * 130) == 0, true);
    t.fws_bytes = need;
    EXPECT(t.fwd(), HIP);
    t.fws_bytes = need - 1;
    EXPECT(t.fwd(), MXQ_ERR_WORKSPACE);
    t.fws_bytes = need;
    t.fws = nullptr;
    EXPECT(t.fwd(), MXQ_ERR_NULL);
    t.fws = P + 4;
    EXPECT(t.fwd(), MXQ_ERR_ALIGN);
    EXPECT(mxq_workspace_size(MXQ_WS_LATENT_FORWARD, 16384, 16384, 16, 4), 0);
    Attn u;
    u.fws = nullptr;
    u.fws_bytes = 0;
    EXPECT(u.fwd(), HIP);                                     // none is needed
  }
  BACK(t.go = nullptr, MXQ_ERR_NULL);
  BACK(t.dq = nullptr, MXQ_ERR_NULL);
  BACK(t.dk = nullptr, MXQ_ERR_NULL);
  BACK(t.dr = nullptr, MXQ_ERR_NULL);
  BACK(t.dv = nullptr, MXQ_ERR_NULL);
  BACK(t.lg = 64, MXQ_ERR_SHAPE);
  BACK(t.ldq = 128, MXQ_ERR_SHAPE);
  BACK(t.ldkh = 64, MXQ_ERR_SHAPE);
  BACK(t.ldr = 32, MXQ_ERR_SHAPE);
  BACK(t.ldv = 0, MXQ_ERR_SHAPE);
  BACK(t.lgh = 132, MXQ_ERR_ALIGN);
  BACK(t.ldr = 68, MXQ_ERR_ALIGN);
  BACK(t.dq = t.x + 4, MXQ_ERR_ALIGN);
  BACK(t.go = t.x + 4, MXQ_ERR_ALIGN);
  BACK(t.ws = nullptr, MXQ_ERR_NULL);
  BACK(t.ws = P + 4, MXQ_ERR_ALIGN);
  {
    const size_t need = mxq_workspace_size(MXQ_WS_LATENT_BACKWARD, 100, 120, 2, 0);
    EXPECT(need, 4 * (2 * 120 * 64 + 2 * 100));
    BACK(t.ws_bytes = need, HIP);
    BACK(t.ws_bytes = need - 1, MXQ_ERR_WORKSPACE);
  }
  EXPECT(mxq_workspace_size(MXQ_WS_LATENT_BACKWARD, HUGE_, HUGE_, HUGE_, 0), SIZE_MAX);
  EXPECT(mxq_workspace_size(MXQ_WS_LATENT_DECODE, 0, 1, 1, 1), 0);

  std::printf("%d checks, %d failed\n", g_n, g_fail);
  return g_fail != 0;
}
