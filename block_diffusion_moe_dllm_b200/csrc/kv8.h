// Internal launchers of the 8-bit KV cache operators (not part of the public ABI).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>
#include <stddef.h>
#include <atomic>
#include "common.cuh"

namespace dllm {

// Raises a kernel's dynamic shared memory limit on the current device (once per device and kernel).
template <auto kernel>
inline int set_max_smem(int bytes) {
  static std::atomic<uint64_t> done{0};      // one bit per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && dev < 64 && (done.load(std::memory_order_acquire) >> dev & 1)) return DLLM_OK;
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return dllm_host::cuda_status(e, "cudaFuncSetAttribute");
  if (dev < 64) done.fetch_or(1ull << dev, std::memory_order_release);
  return DLLM_OK;
}

struct Kv8StoreArgs {
  int B, Hkv, d, n, cap_src, src_row, cap, dst_row, S, dtype, pos_stride;
  const void* k;
  const void* v;
  const int32_t* src_pos;   // nullable: [B, pos_stride] source rows
  const int32_t* dst_rows;  // nullable: [B] first destination row of each batch row
  uint8_t* k_codes;
  uint8_t* v_codes;
  float* k_scale;
  float* v_scale;
};
int launch_kv8_store(const Kv8StoreArgs& a, cudaStream_t s);

struct Kv8AttnArgs {
  int B, Lq, Hq, Hkv, d, blk_len, P, cap, cap_own, S, dtype;
  float scale;
  const void* q;
  const uint8_t* k_codes;
  const uint8_t* v_codes;   // attention only
  const float* k_scale;
  const float* v_scale;
  const int32_t* lens;      // nullable: [B]
  const void* k_own;        // nullable with v_own: no own keys
  const void* v_own;
  void* out;
  float* lse_out;           // nullable
  // attention weights
  const float* lse_in;
  const float* mass_in;     // nullable: zeros
  float* mass_out;
  float decay;
  void* ws;                 // scratch past the status block
  int32_t* status;
};
size_t attn_kv8_workspace_bytes(int B, int Lq, int Hq, int Hkv, int d, int P, int own, int dtype);
int launch_attn_kv8(const Kv8AttnArgs& a, cudaStream_t s);
int launch_attn_mass_kv8(const Kv8AttnArgs& a, cudaStream_t s);
// tensor-core variants (bf16)
size_t attn_kv8_tc_workspace_bytes(int B, int Lq, int Hq, int Hkv);
int launch_attn_kv8_tc(const Kv8AttnArgs& a, cudaStream_t s);
int launch_attn_mass_kv8_tc(const Kv8AttnArgs& a, cudaStream_t s);
// SIMT variants (fp32)
size_t attn_kv8_simt_workspace_bytes(int B, int Lq, int Hq, int Hkv, int d, int P, int own);
int launch_attn_kv8_simt(const Kv8AttnArgs& a, cudaStream_t s);
int launch_attn_mass_kv8_simt(const Kv8AttnArgs& a, cudaStream_t s);

struct Kv8EvictArgs {
  int B, Hkv, d, P, cap, n_keep, cap_out, S, n_first, n_last, per_head;
  const uint8_t* k_codes;
  const uint8_t* v_codes;
  const float* k_scale;
  const float* v_scale;
  const float* mass;
  const int32_t* lens;   // nullable: [B]
  const int32_t* pos;    // nullable: [B, Hs, cap]
  uint8_t* k_out;
  uint8_t* v_out;
  float* k_scale_out;
  float* v_scale_out;
  float* mass_out;
  int32_t* keep_pos;     // [B, Hs, cap_out]
  int32_t* len_out;
  void* ws;
};
size_t kv8_evict_workspace_bytes(int B, int Hkv, int P, int n_keep, int per_head);
int launch_kv8_evict(const Kv8EvictArgs& a, cudaStream_t s);

}  // namespace dllm
