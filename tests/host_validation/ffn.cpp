// Host-side argument validation of the norm and few-token block entry points, built
// with AddressSanitizer and UndefinedBehaviorSanitizer on the host code only and run
// where no GPU is visible.  Device pointers are fake addresses that no call may
// dereference: every case either fails a host-side check (its expected status) or
// reaches the launch, which fails without a device (MXQ_ERR_HIP).  Extreme sizes probe
// the 64-bit size arithmetic, where an overflow is undefined behaviour and stops the run.
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

constexpr int64_t HUGE_ = INT64_MAX, FAR_ = INT64_C(1) << 39;

template <class T>
static T* at() { return reinterpret_cast<T*>(uintptr_t(4096)); }

static mxq_norm norm() {
  mxq_norm n{};
  n.x = at<uint16_t>(); n.residual = at<uint16_t>(); n.weight = at<uint16_t>();
  n.total = at<uint16_t>(); n.rstd = at<float>(); n.y = at<uint16_t>();
  n.q = n.scale = n.qT = n.scaleT = at<uint8_t>();
  n.ldx = n.ldr = n.ldt = n.ldy = n.ldq = 64;
  n.lds = 2; n.ldqT = 64; n.ldsT = 2;
  n.M = 40; n.K = 64; n.M_cap = 64; n.eps = 1e-6f;
  return n;
}

static mxq_norm_grad grad() {
  mxq_norm_grad g{};
  g.dy = g.total = g.weight = g.dtotal = at<uint16_t>(); g.rstd = at<float>();
  g.dx = at<uint16_t>(); g.dw = at<float>(); g.workspace = at<void>();
  g.lddy = g.ldt = g.lddt = g.lddx = 64;
  g.workspace_bytes = SIZE_MAX; g.M = 40; g.K = 64;
  return g;
}

static mxq_ffn_decode ffn() {
  mxq_ffn_decode f{};
  f.x = f.x_scale = f.w_gu = f.w_gu_scale = f.w_down = f.w_down_scale = at<uint8_t>();
  f.offsets = at<int64_t>(); f.y = at<uint16_t>(); f.workspace = at<void>();
  f.workspace_bytes = SIZE_MAX;
  f.ldx = f.ldgu = 64; f.ldsx = f.ldsgu = 2; f.gu_estride = 64 * 64; f.gus_estride = 128;
  f.ldd = 32; f.ldsd = 1; f.d_estride = 32 * 40; f.ds_estride = 40;
  f.ldy = 40; f.M = 4; f.K = 64; f.F = 32; f.N = 40; f.E = 2;
  return f;
}

#define CASE(make, call, change, want)                                                   \
  do {                                                                                   \
    auto t = make();                                                                     \
    change;                                                                              \
    EXPECT(call(&t, nullptr), want);                                                     \
  } while (0)
#define NORM(change, want) CASE(norm, mx_rms_norm, change, want)
#define GRAD(change, want) CASE(grad, mx_rms_norm_backward, change, want)
#define FFN(change, want) CASE(ffn, mx_gated_ffn_decode, change, want)

int main() {
  EXPECT(mx_rms_norm(nullptr, nullptr), MXQ_ERR_NULL);
  EXPECT(mx_rms_norm_backward(nullptr, nullptr), MXQ_ERR_NULL);
  EXPECT(mx_gated_ffn_decode(nullptr, nullptr), MXQ_ERR_NULL);

  NORM(, MXQ_ERR_HIP);
  NORM(t.M = HUGE_, MXQ_ERR_SHAPE);
  NORM(t.K = HUGE_ / 32 * 32, MXQ_ERR_SHAPE);
  NORM(t.M_cap = HUGE_ / 32 * 32, MXQ_ERR_SHAPE);
  NORM(t.ldx = HUGE_, MXQ_ERR_SHAPE);
  NORM(t.ldqT = HUGE_, MXQ_ERR_SHAPE);
  NORM(t.M = INT64_MIN, MXQ_ERR_SHAPE);
  NORM(t.ldy = INT64_MIN, MXQ_ERR_SHAPE);
  NORM(t.ldx = t.ldr = t.ldt = t.ldy = t.ldq = t.lds = FAR_, MXQ_ERR_HIP);
  NORM((t.M = MXQ_NORM_MAX_ROWS, t.M_cap = t.ldqT = 2 * (int64_t)MXQ_NORM_MAX_ROWS, t.ldsT = t.M_cap / 32), MXQ_ERR_HIP);
  NORM((t.M = MXQ_NORM_MAX_ROWS, t.M_cap = t.ldqT = 2 * (int64_t)MXQ_NORM_MAX_ROWS, t.ldsT = t.M_cap / 32,
        t.K = MXQ_NORM_MAX_COLS, t.ldx = t.ldr = t.ldt = t.ldy = t.ldq = t.lds = FAR_), MXQ_ERR_HIP);
  NORM((t.M = 0, t.x = nullptr), MXQ_ERR_HIP);           // the column copy's zeros

  GRAD(, MXQ_ERR_HIP);
  GRAD(t.M = HUGE_, MXQ_ERR_SHAPE);
  GRAD(t.K = HUGE_ / 32 * 32, MXQ_ERR_SHAPE);
  GRAD(t.lddx = HUGE_, MXQ_ERR_SHAPE);
  GRAD((t.M = MXQ_NORM_MAX_ROWS, t.K = MXQ_NORM_MAX_COLS, t.lddy = t.ldt = t.lddt = t.lddx = FAR_), MXQ_ERR_HIP);
  GRAD(t.M = 0, MXQ_ERR_HIP);                            // dw's zeros

  FFN(, MXQ_ERR_HIP);
  FFN(t.M = HUGE_, MXQ_ERR_SHAPE);
  FFN(t.N = HUGE_, MXQ_ERR_SHAPE);
  FFN(t.F = HUGE_ / 32 * 32, MXQ_ERR_SHAPE);
  FFN(t.gu_estride = HUGE_ / 16 * 16, MXQ_ERR_SHAPE);
  FFN(t.ldgu = HUGE_ / 16 * 16, MXQ_ERR_SHAPE);
  FFN(t.ldy = HUGE_, MXQ_ERR_SHAPE);
  FFN((t.M = MXQ_FFN_DECODE_MAX_ROWS, t.K = t.F = t.N = MXQ_FFN_DECODE_MAX_DIM, t.E = 256, t.ldx = t.ldgu = t.ldd = FAR_,
       t.ldsx = t.ldsgu = t.ldsd = t.ldy = FAR_, t.gu_estride = t.gus_estride = t.d_estride = t.ds_estride = FAR_),
      MXQ_ERR_HIP);

  EXPECT(mxq_workspace_size(MXQ_WS_NORM_BACKWARD, HUGE_, HUGE_, 0, 0), 0);
  EXPECT(mxq_workspace_size(MXQ_WS_FFN_DECODE, HUGE_, HUGE_, 0, 0), 0);
  EXPECT(mxq_workspace_size(MXQ_WS_FFN_DECODE, 4, 32, 0, 0), 4 * 33);
  EXPECT(mxq_workspace_size(MXQ_WS_FFN_DECODE, MXQ_FFN_DECODE_MAX_ROWS, MXQ_FFN_DECODE_MAX_DIM, 0, 0),
         (INT64_C(1) << 40) + (INT64_C(1) << 35));

  std::printf("%d checks, %d failed\n", g_n, g_fail);
  return g_fail != 0;
}
