// What the norm and feed-forward entry points would launch, without a GPU: this program
// defines the HIP runtime's launch functions, which the library then uses in place of the
// runtime's own, and logs kernel, grid and block of every launch.  Device pointers are
// fake addresses, nothing runs.
//   launches <libmxq.so>      reads calls from stdin, one a line:
//     norm M K columns residual | grad M K | swiglu E M F K accum windows | ffn M K F N E
//   and prints a line for each: the status, then "kernel gx,gy,gz bx,by,bz" per launch,
//   separated by semicolons; before them a line "kernels" with all kernels of the library.
#include <dlfcn.h>

#include <cstdio>
#include <cstring>
#include <string>

#include "mxq.h"

namespace {
constexpr int kMost = 4096;
const void* g_host[kMost];
const char* g_name[kMost];
int g_count = 0;
struct Config { dim3 grid, block; size_t shared; hipStream_t stream; } g_config;
std::string& log() { static std::string s; return s; }
}  // namespace

extern "C" {
void** __hipRegisterFatBinary(const void*) { static void* module; return &module; }
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterVar(void**, void*, char*, char*, int, size_t, int, int) {}
void __hipRegisterFunction(void**, const void* host, char*, const char* name, unsigned, void*, void*,
                           void*, void*, int*) {
  if (g_count == kMost) __builtin_trap();
  g_host[g_count] = host;
  g_name[g_count++] = name;
}
hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t shared, hipStream_t stream) {
  g_config = {grid, block, shared, stream};
  return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* shared, hipStream_t* stream) {
  *grid = g_config.grid; *block = g_config.block; *shared = g_config.shared; *stream = g_config.stream;
  return hipSuccess;
}
hipError_t hipLaunchKernel(const void* f, dim3 g, dim3 b, void**, size_t, hipStream_t) {
  const char* name = "?";
  for (int i = 0; i < g_count; ++i)
    if (g_host[i] == f) name = g_name[i];
  char text[512];
  std::snprintf(text, sizeof text, ";%s %u,%u,%u %u,%u,%u", name, g.x, g.y, g.z, b.x, b.y, b.z);
  log() += text;
  return hipSuccess;
}
hipError_t hipGetLastError() { return hipSuccess; }
}

template <class T>
static T* at() { return reinterpret_cast<T*>(uintptr_t(4096)); }
static int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

int main(int argc, char** argv) {
  void* lib = argc == 2 ? dlopen(argv[1], RTLD_NOW | RTLD_GLOBAL) : nullptr;
  if (!lib) {
    std::fprintf(stderr, "%s\n", argc == 2 ? dlerror() : "usage: launches <libmxq.so>");
    return 1;
  }
#define ENTRY(name) const auto name##_ = reinterpret_cast<decltype(&name)>(dlsym(lib, #name))
  ENTRY(mx_rms_norm);
  ENTRY(mx_rms_norm_backward);
  ENTRY(mx_grouped_gemm_swiglu_backward);
  ENTRY(mx_gated_ffn_decode);
  std::printf("kernels");
  for (int i = 0; i < g_count; ++i) std::printf(";%s", g_name[i]);
  std::printf("\n");
  char what[32];
  while (std::scanf("%31s", what) == 1) {
    long long v[6];
    const int n = !std::strcmp(what, "grad") ? 2 : !std::strcmp(what, "norm") ? 4 : !std::strcmp(what, "ffn") ? 5 : 6;
    for (int i = 0; i < n; ++i)
      if (std::scanf("%lld", &v[i]) != 1) return 1;
    log().clear();
    int status = -1;
    if (n == 4) {
      mxq_norm t{};
      t.M = v[0]; t.K = v[1]; t.eps = 1e-6f;
      t.x = t.weight = at<uint16_t>(); t.y = at<uint16_t>(); t.rstd = at<float>(); t.q = t.scale = at<uint8_t>();
      t.ldx = t.ldr = t.ldt = t.ldy = t.ldq = t.K; t.lds = t.K / 32;
      if (v[3]) t.residual = at<uint16_t>(), t.total = at<uint16_t>();
      if (v[2]) {
        t.M_cap = t.ldqT = up(t.M, 128); t.ldsT = t.M_cap / 32;
        t.qT = t.scaleT = at<uint8_t>();
      }
      status = mx_rms_norm_(&t, nullptr);
    } else if (n == 2) {
      mxq_norm_grad t{};
      t.M = v[0]; t.K = v[1];
      t.dy = t.total = t.weight = t.dtotal = at<uint16_t>(); t.rstd = at<float>();
      t.dx = at<uint16_t>(); t.dw = at<float>(); t.workspace = at<void>(); t.workspace_bytes = SIZE_MAX;
      t.lddy = t.ldt = t.lddt = t.lddx = t.K;
      status = mx_rms_norm_backward_(&t, nullptr);
    } else if (n == 5) {
      mxq_ffn_decode t{};
      t.M = v[0]; t.K = v[1]; t.F = v[2]; t.N = v[3]; t.E = (int32_t)v[4];
      t.x = t.x_scale = t.w_gu = t.w_gu_scale = t.w_down = t.w_down_scale = at<uint8_t>();
      t.offsets = at<int64_t>(); t.y = at<uint16_t>(); t.workspace = at<void>(); t.workspace_bytes = SIZE_MAX;
      t.ldx = t.ldgu = t.K; t.ldsx = t.ldsgu = t.K / 32; t.gu_estride = 2 * t.F * t.K; t.gus_estride = t.gu_estride / 32;
      t.ldd = t.F; t.ldsd = t.F / 32; t.d_estride = t.N * t.F; t.ds_estride = t.d_estride / 32; t.ldy = t.N;
      status = mx_gated_ffn_decode_(&t, nullptr);
    } else {
      const int64_t E = v[0], M = v[1], F = v[2], K = v[3], cap = up(M + 31 * E, 128);
      const int64_t lds = v[5] ? up(K / 32, 16) : K / 32 + (K / 32 % 16 == 0);
      auto* p = at<uint8_t>();
      status = mx_grouped_gemm_swiglu_backward_(
          p, p, K, lds, p, p, K, lds, F * K, F * lds, at<int64_t>(), (int32_t)E, M, F, K, at<uint16_t>(), 2 * F,
          p, 2 * F, p, 2 * F, p, F / 16, p, cap, p, cap / 32, cap, at<int64_t>(), (int)v[4], nullptr);
    }
    std::printf("%d%s\n", status, log().c_str());
  }
  return 0;
}
