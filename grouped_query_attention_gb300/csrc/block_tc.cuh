// Device pieces shared by the tensor-core kernels over the block-scaled cache.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "common.cuh"

namespace gqa {

// Sixteen codes as fp16: byte x ^ 0x80 under the exponent of 1024, less 1152.
__device__ __forceinline__ void codes16(uint4 w, uint32_t* h) {
  const __half2 bias = __floats2half2_rn(1152.f, 1152.f);
  const uint32_t wv[4] = {w.x ^ 0x80808080u, w.y ^ 0x80808080u, w.z ^ 0x80808080u, w.w ^ 0x80808080u};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t p01 = __byte_perm(wv[k], 0x64646464u, 0x4140u);
    const uint32_t p23 = __byte_perm(wv[k], 0x64646464u, 0x4342u);
    const __half2 a = __hsub2(*reinterpret_cast<const __half2*>(&p01), bias);
    const __half2 c = __hsub2(*reinterpret_cast<const __half2*>(&p23), bias);
    h[2 * k] = *reinterpret_cast<const uint32_t*>(&a);
    h[2 * k + 1] = *reinterpret_cast<const uint32_t*>(&c);
  }
}

// Softcap in the log2 domain, c2 tanh(u), c2 = softcap log2(e), as u Q(u^2)
// with Q the least-squares fit of tanh(u) / u in u^2: degree 3 on |u| <= 0.35,
// degree 7 on |u| <= 1 (relative error 9e-8 each in fp32 Horner). Beyond,
// c2 (1 - 2 / (e^2u + 1)), whose cancellation the value's own size keeps
// harmless. A pair of scores costs 6 or 10 packed instructions on the FMA pipe.
constexpr float kCapLow = 0.35f, kCapHigh = 1.0f;
__device__ constexpr float kFit3[4] = {0.9999999403953552f, -0.3333241641521454f, 0.13295666873455048f, -0.04895104840397835f};
__device__ constexpr float kFit7[8] = {1.0f, -0.33333274722099304f, 0.13332107663154602f, -0.05386783555150032f,
                                       0.021456174552440643f, -0.00790493842214346f, 0.0022732384968549013f,
                                       -0.0003508012741804123f};
// c2 Q(z): the coefficients times c2 are loop constants of the caller.
template <int DEG>
__device__ __forceinline__ float2 cap_fit(float2 z, float c2) {
  constexpr const float* q = DEG == 3 ? kFit3 : kFit7;
  float2 y = make_float2(q[DEG] * c2, q[DEG] * c2);
#pragma unroll
  for (int i = DEG - 1; i >= 0; --i) y = ffma2(y, z, make_float2(q[i] * c2, q[i] * c2));
  return y;
}
__device__ __forceinline__ float cap_far(float u, float c2) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(ex2(u * (2.f * kLog2e)) + 1.f));
  return fmaf(r, -2.f * c2, c2);
}
// Both forms computed, one selected (no branch).
__device__ __forceinline__ float2 cap_any(float2 u, float c2) {
  const float2 z = ffma2(u, u, make_float2(0.f, 0.f));
  const float2 y = ffma2(u, cap_fit<7>(z, c2), make_float2(0.f, 0.f));
  const float fx = cap_far(u.x, c2), fy = cap_far(u.y, c2);
  float2 r;
  asm("{ .reg .pred p; setp.le.f32 p, %1, %2; selp.f32 %0, %3, %4, p; }" : "=f"(r.x) : "f"(z.x), "f"(kCapHigh), "f"(y.x), "f"(fx));
  asm("{ .reg .pred p; setp.le.f32 p, %1, %2; selp.f32 %0, %3, %4, p; }" : "=f"(r.y) : "f"(z.y), "f"(kCapHigh), "f"(y.y), "f"(fy));
  return r;
}

}  // namespace gqa
