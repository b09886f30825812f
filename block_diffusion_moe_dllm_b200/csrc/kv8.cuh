// Device helpers of the 8-bit KV cache: E4M3 codes with one fp32 scale per run of scale_len tokens and kv head.
#pragma once
#include "common.cuh"
#include <cuda_fp16.h>

namespace dllm {
namespace kv8 {

// Two E4M3 codes (low half of u) as f16 pairs: every E4M3 value is an f16 value, so this is exact.
DLLM_DEV uint32_t e4m3x2_to_f16x2(uint32_t u) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(u));
  return r;
}
// Four codes as two f16 pairs.
DLLM_DEV void e4m3x4_to_f16x4(uint32_t u, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(u));
}
// lo, hi rounded to E4M3 (nearest, ties to even; beyond +-448 saturates, NaN stays NaN), lo in the low byte.
DLLM_DEV uint32_t f32x2_to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// 16 codes of one vector as fp32.
DLLM_DEV void codes16_to_f32(const uint4& u, float* f) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t a, b;
    e4m3x4_to_f16x4(w[i], a, b);
    const float2 x = __half22float2(*reinterpret_cast<__half2*>(&a));
    const float2 y = __half22float2(*reinterpret_cast<__half2*>(&b));
    f[4 * i] = x.x;
    f[4 * i + 1] = x.y;
    f[4 * i + 2] = y.x;
    f[4 * i + 3] = y.y;
  }
}

// Scale exponents of the cache: a run whose largest magnitude is below 448 * 2^-64 keeps the scale 2^-64.
constexpr int kMinExp = -64, kMaxExp = 120;

// The least k with amax <= 448 * 2^k (448 = 1.75 * 2^8, so the comparison is one of mantissas), within the limits.
// amax is finite and not negative.
DLLM_DEV int scale_exp(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int k = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return min(max(k, kMinExp), kMaxExp);
}
DLLM_DEV float exp2i(int k) { return __uint_as_float((uint32_t)(k + 127) << 23); }   // 2^k, -126 <= k <= 127

// Length of batch row b's prefix: the device lengths clamped to [0, P], or P without them.
DLLM_DEV int prefix_len(const int32_t* lens, int b, int P) { return lens ? min(max(lens[b], 0), P) : P; }

// Thread-block clusters: a barrier over all CTAs, and the same shared variable of another CTA.
DLLM_DEV void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
DLLM_DEV uint32_t peer_u32(const void* mine, uint32_t rank) {
  uint32_t v, at;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(mine)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}
DLLM_DEV void peer_store_u32(void* mine, uint32_t rank, uint32_t v) {
  uint32_t at;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(mine)), "r"(rank));
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}

}  // namespace kv8
}  // namespace dllm
