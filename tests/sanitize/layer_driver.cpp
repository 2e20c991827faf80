// Host-side driver of the C ABI of a Mamba-2 layer on whole sequences for sanitizer builds: api_layer.cpp linked
// against stand-ins for its kernel launchers that only count calls; pointers are aligned addresses that nothing
// dereferences.
#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdint>
#include <cstdio>

#include "layer.hpp"
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
hipError_t launch_conv_prompt(const ConvPromptArgs&, hipStream_t) { return count(); }
hipError_t launch_conv_prompt_backward(const ConvPromptArgs&, hipStream_t) { return count(); }
int64_t conv_prompt_backward_bytes(const replayssm_conv_prompt_config& c) { return (int64_t)c.D * c.W * 1000; }
hipError_t launch_conv_restore(const ConvRestoreArgs&, hipStream_t) { return count(); }
hipError_t launch_gated_norm(const GatedNormArgs&, hipStream_t) { return count(); }
hipError_t launch_gated_norm_backward(const GatedNormArgs&, hipStream_t) { return count(); }
int64_t gated_norm_backward_bytes(const replayssm_gated_norm_config& c) { return (int64_t)c.D * c.groups * 1000; }
hipError_t launch_linear_step(const DeltaArgs&, hipStream_t) { return count(); }
int linear_segment_for(const replayssm_linear_config&) { return 256; }
int64_t linear_forward_bytes(const replayssm_linear_config& c, int segments) { return (int64_t)segments * c.H * 1000; }
int64_t linear_backward_bytes(const replayssm_linear_config& c, int segments) { return (int64_t)segments * c.H * 1000; }
hipError_t launch_linear_prompt(const LinearArgs&, hipStream_t) { return count(); }
hipError_t launch_linear_prompt_backward(const LinearArgs&, hipStream_t) { return count(); }
}  // namespace rs

extern "C" int replayssm_conv_sizes(const replayssm_conv_config* c, int64_t* ring, int64_t* ptr) {
  if (c == nullptr || c->B < 1) return REPLAYSSM_EINVAL;
  *ring = *ptr = 16;
  return REPLAYSSM_OK;
}

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
  const replayssm_ragged m{I(1), I(2), I(3), I(4), I(5), I(6)};
  int64_t a = 0, b = 0;
  int32_t seg = 0;
  const int64_t tokens[] = {INT64_MIN, 0, 1, 1000, (int64_t)1 << 30, ((int64_t)1 << 30) + 1, INT64_MAX};
  const int sizes[] = {INT32_MIN, -1, 0, 1, 4, 16, 64, 128, 256, 65536, 1 << 17, INT32_MAX};
  const int64_t strides[] = {INT64_MIN, 0, 64, 1 << 20, (int64_t)1 << 31, INT64_MAX};
  for (int64_t t : tokens)
    for (int D : sizes)
      for (int W : sizes)
        for (int64_t s : strides) {
          replayssm_conv_prompt_config c{3, D, W, 1, REPLAYSSM_BF16, t, s};
          const int r = replayssm_conv_prompt_sizes(&c, &a);
          EXPECT(r, t >= 1 && t <= (int64_t)1 << 30 && D >= 8 && D <= 1 << 17 && D % 8 == 0 && W >= 1 && W <= 4 && s >= D && s <= (int64_t)1 << 31 ? 0 : -1);
          EXPECT(replayssm_conv_prompt(&c, &m, p(7), F(8), nullptr, nullptr, p(9), F(10), I(11), nullptr), r);
          EXPECT(replayssm_conv_prompt_backward(&c, &m, p(7), F(8), F(9), F(10), p(11), F(12), p(13), F(14), F(15), F(16), p(17), I(18), nullptr), r);
          if (r == 0)
            EXPECT(replayssm_conv_prompt_backward(&c, &m, p(7), F(8), F(9), F(10), p(11), F(12), p(13), F(14), F(15), F(16), nullptr, I(18), nullptr), -1);
        }
  for (int n : sizes) {
    const replayssm_conv_config c{4, 64, 4, 2};
    const replayssm_conv_state st{F(1), I(2), I(3), I(4), I(5)};
    EXPECT(replayssm_conv_restore(&c, &st, n, I(6), F(7), nullptr), n >= 0 && n <= 65535 ? 0 : -1);
  }
  for (int64_t t : tokens)
    for (int D : sizes)
      for (int groups : sizes)
        for (int64_t s : strides) {
          replayssm_gated_norm_config c{(int32_t)(t > INT32_MAX ? INT32_MAX : t < INT32_MIN ? INT32_MIN : t), groups, D, REPLAYSSM_GATE_AFTER, 0, REPLAYSSM_F16, 1e-5f, s, s};
          const int r = replayssm_gated_norm_sizes(&c, &a);
          EXPECT(replayssm_gated_norm(&c, p(7), p(8), F(9), p(10), nullptr), r);
          EXPECT(replayssm_gated_norm_backward(&c, p(7), p(8), F(9), p(10), p(11), p(12), F(13), p(14), nullptr), r);
          if (r == 0) EXPECT(replayssm_gated_norm(&c, p(7), nullptr, F(9), p(10), nullptr), -1);
        }
  for (int64_t t : tokens)
    for (int H : sizes)
      for (int Hk : sizes)
        for (int d : sizes)
          for (int segment : sizes) {
            replayssm_linear_config c{2, H, Hk, d, d, REPLAYSSM_F32, t, (int64_t)1 << 24, (int64_t)1 << 24, (int64_t)1 << 24, 1.f, segment};
            const int r = replayssm_linear_sizes(&c, &a, &b);
            const int any = replayssm_linear_segment(&c, &seg);
            if (r == 0) EXPECT(any, 0);
            EXPECT(replayssm_linear_step(&c, I(1), I(2), 5, p(3), p(4), p(5), F(6), nullptr, nullptr, F(7), F(8), p(9), I(10), nullptr), any);
            EXPECT(replayssm_linear_prompt(&c, &m, p(7), p(8), p(9), F(10), F(11), F(12), F(13), p(14), F(15), p(16), I(17), nullptr), r);
            EXPECT(replayssm_linear_prompt_backward(&c, &m, p(7), p(8), p(9), F(10), F(11), F(12), F(13), p(14), F(15), p(16), p(17), p(18), F(19), F(20), F(21),
                                                    F(22), p(23), I(24), nullptr),
                   r);
          }
  std::printf("launches=%d failures=%d\n", rs::g_launches, g_fail);
  return g_fail != 0;
}
