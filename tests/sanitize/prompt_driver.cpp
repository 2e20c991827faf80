// Host-side driver of the prompt-side C ABI for sanitizer builds: api_prompt.cpp linked against
// stand-ins for its kernel launchers that only count calls; pointers are aligned addresses
// that nothing dereferences.
#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstring>

#include "prompt.hpp"
#include "replayssm.h"

namespace rs {
static int g_launches = 0;
static hipError_t count() {
  ++g_launches;
  return hipSuccess;
}
int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return code;
}
hipError_t launch_ragged(const RaggedArgs&, hipStream_t) { return count(); }
hipError_t launch_qk_norm(const QkNormArgs&, hipStream_t) { return count(); }
hipError_t launch_qk_norm_backward(const QkNormArgs&, hipStream_t) { return count(); }
int qk_norm_partials(int n, int, int, int) { return n < 1024 ? n : 1024; }
hipError_t launch_delta_step(const DeltaArgs&, hipStream_t) { return count(); }
int64_t delta_forward_bytes(const replayssm_delta_config& c, int blocks) { return (int64_t)blocks * c.H * 1000; }
int64_t delta_backward_bytes(const replayssm_delta_config& c, int blocks) { return (int64_t)blocks * c.H * 1000; }
hipError_t launch_delta_prompt(const DeltaArgs&, hipStream_t) { return count(); }
hipError_t launch_delta_prompt_backward(const DeltaArgs&, hipStream_t) { return count(); }
}  // namespace rs

static int g_fail = 0;
static void expect(int got, int want, int line) {
  if (got != want) {
    std::printf("line %d: %d, expected %d\n", line, got, want);
    ++g_fail;
  }
}
#define EXPECT(expr, want) expect((expr), (want), __LINE__)

static void* p(uintptr_t i) { return reinterpret_cast<void*>((i + 1) << 20); }
static float* F(uintptr_t i) { return static_cast<float*>(p(i)); }
static int32_t* I(uintptr_t i) { return static_cast<int32_t*>(p(i)); }

int main() {
  replayssm_ragged m{I(1), I(2), I(3), I(4), I(5), I(6)};
  int64_t n = 0, w = 0;
  for (int64_t tokens : {(int64_t)1, (int64_t)1000, (int64_t)1 << 30, ((int64_t)1 << 30) + 1, INT64_MAX, INT64_MIN})
    for (int seqs : {0, 1, 16384, 16385, INT32_MAX, INT32_MIN})
      for (int block : {0, 1, 64, 65536, INT32_MAX, INT32_MIN}) {
        replayssm_ragged_config c{seqs, block, tokens};
        const bool ok = tokens >= 1 && tokens <= (int64_t)1 << 30 && seqs >= 1 && seqs <= 16384 && block >= 1 &&
                        block <= 65536 && tokens / block + seqs < (int64_t)1 << 30;
        EXPECT(replayssm_ragged_sizes(&c, &n), ok ? REPLAYSSM_OK : REPLAYSSM_EINVAL);
        EXPECT(replayssm_ragged_maps(&c, &m, I(7), nullptr, nullptr), ok ? REPLAYSSM_OK : REPLAYSSM_EINVAL);
      }
  for (int heads : {INT32_MIN, -1, 0, 1, 4096, INT32_MAX})
    for (int D : {INT32_MIN, 0, 16, 100, 256, INT32_MAX})
      for (int rot : {INT32_MIN, 0, 2, 16, 256, INT32_MAX}) {
        replayssm_qk_norm_config c{};
        c.n_tokens = 100;
        c.Hq = heads;
        c.Hk = 1;
        c.D = D;
        c.rot = rot;
        c.rep = 2;
        c.q_stride = c.k_stride = 1 << 21;
        const int r = replayssm_qk_norm_sizes(&c, &w);
        EXPECT(replayssm_qk_norm(&c, p(1), p(2), F(3), F(4), I(5), F(6), p(7), p(8), nullptr), r);
        EXPECT(replayssm_qk_norm_backward(&c, p(1), p(2), F(3), F(4), I(5), F(6), p(7), p(8), p(9), p(10), F(11), F(12), p(13),
                                          nullptr),
               r);
        if (r == REPLAYSSM_OK) EXPECT(replayssm_qk_norm(&c, p(1), p(2), F(3), F(4), nullptr, F(6), p(7), p(8), nullptr),
                                      rot > 0 ? REPLAYSSM_EINVAL : REPLAYSSM_OK);
      }
  for (int H : {INT32_MIN, 0, 4, 65536, INT32_MAX})
    for (int64_t tokens : {INT64_MIN, (int64_t)0, (int64_t)100, (int64_t)1 << 30, INT64_MAX})
      for (int64_t stride : {INT64_MIN, (int64_t)0, (int64_t)1 << 23, INT64_MAX}) {
        replayssm_delta_config c{};
        c.n_seqs = 3;
        c.H = H;
        c.Hk = H > 0 ? H / 2 + H % 2 : H;
        c.dk = 64;
        c.dv = 32;
        c.n_tokens = tokens;
        c.q_stride = c.k_stride = c.v_stride = stride;
        c.scale = 1.f;
        const int r = replayssm_delta_sizes(&c, &n, &w);
        EXPECT(replayssm_delta_step(&c, I(1), I(2), 4, p(3), p(4), p(5), F(6), F(7), F(8), F(9), p(10), I(11), nullptr), r);
        EXPECT(replayssm_delta_prompt(&c, &m, p(3), p(4), p(5), F(6), F(7), F(8), p(9), F(10), p(11), I(12), nullptr), r);
        EXPECT(replayssm_delta_prompt_backward(&c, &m, p(3), p(4), p(5), F(6), F(7), F(8), p(9), F(10), p(11), p(12), p(13),
                                               F(14), F(15), F(16), p(17), I(18), nullptr),
               r);
      }
  EXPECT(replayssm_delta_sizes(nullptr, &n, &w), REPLAYSSM_EINVAL);
  EXPECT(replayssm_ragged_sizes(nullptr, &n), REPLAYSSM_EINVAL);
  EXPECT(replayssm_qk_norm_sizes(nullptr, &n), REPLAYSSM_EINVAL);
  std::printf("launches=%d failures=%d\n", rs::g_launches, g_fail);
  return g_fail != 0;
}
