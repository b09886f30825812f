// Attention over an 8-bit prefix cache and the block's own K/V, and the weight each cached position receives: SIMT
// variants for fp32 storage (the tensor-core variants are in attn_kv8_tc.cu).
//
// For batch row b, kv head h and G = Hq / Hkv query heads, the rows of the problem are the (query, head of the group)
// pairs in memory order (row R = query R / G, head R % G), so any G fills the row tiles:
//   s[R, j] = scale * q[R] . K[j],  K[j] = k_scale[j / S] * k_codes[j] over the prefix, the storage type over the
//             block's own keys; visible prefix keys are j < len[b], own key j is visible iff
//             j / blk_len <= query(R) / blk_len
//   o[R] = sum_j exp(s - lse[R]) V[j],  lse[R] = log sum_j exp(s)
//   mass[j] = decay * mass_in[j] + sum_R exp(s[R, j] - lse[R])   (prefix keys)
#include "kv8.cuh"
#include "kv8.h"
#include "misc.h"
#include <algorithm>
#include <type_traits>

namespace dllm {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int ROWS = 64, KB = 32, PD = 36;   // rows and keys of a tile; row pitch of the weights (floats)

struct SimtPlan {
  int n_rt, n_splits, tps;   // row tiles per (b, h), key splits, key tiles per split
};

SimtPlan simt_plan(int B, int Lq, int Hq, int Hkv, int P, int own) {
  SimtPlan p;
  p.n_rt = (Lq * (Hq / Hkv) + ROWS - 1) / ROWS;
  const int64_t base = (int64_t)B * Hkv * p.n_rt;
  const int tiles = (P + KB - 1) / KB + (own ? (Lq + KB - 1) / KB : 0);
  // two CTAs per SM as far as there are key tiles
  const int want = (int)((2 * num_sms() + base - 1) / base);
  p.n_splits = std::max(1, std::min(std::min(want, 32), tiles));
  p.tps = std::max(1, (tiles + p.n_splits - 1) / p.n_splits);
  p.n_splits = std::max(1, (tiles + p.tps - 1) / p.tps);
  return p;
}

// ROWS rows of the queries, scaled, into shared memory (pitch d + 4); rows past the last are zero.
DLLM_DEV void load_rows(const Kv8AttnArgs& a, int b, int h, int R0, float mul, float* qs) {
  const int G = a.Hq / a.Hkv, vpr = a.d / 4, pitch = a.d + 4;
  for (int i = threadIdx.x; i < ROWS * vpr; i += 256) {
    const int r = i / vpr, c = (i - r * vpr) * 4, R = R0 + r;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (R < a.Lq * G)
      x = *reinterpret_cast<const float4*>(static_cast<const float*>(a.q) +
                                           (((int64_t)b * a.Lq + R / G) * a.Hq + h * G + R % G) * a.d + c);
    *reinterpret_cast<float4*>(qs + r * pitch + c) = make_float4(x.x * mul, x.y * mul, x.z * mul, x.w * mul);
  }
}

// nk rows of the cache from row j0 as values in shared memory; the tile's other rows are zero.
DLLM_DEV void load_codes(const uint8_t* codes, const float* scale, int64_t bh, int cap, int S, int d, int j0, int nk,
                         float* dst) {
  const int vpr = d / 16, pitch = d + 4;
  const int64_t runs = (cap + S - 1) / S;
  for (int i = threadIdx.x; i < KB * vpr; i += 256) {
    const int r = i / vpr, c = (i - r * vpr) * 16;
    uint4 u = make_uint4(0, 0, 0, 0);
    float sc = 0.f;
    if (r < nk) {
      sc = scale[bh * runs + (j0 + r) / S];
      u = *reinterpret_cast<const uint4*>(codes + (bh * cap + j0 + r) * (int64_t)d + c);
    }
    float f[16];
    kv8::codes16_to_f32(u, f);
#pragma unroll
    for (int k = 0; k < 16; k += 4)
      *reinterpret_cast<float4*>(dst + r * pitch + c + k) = make_float4(f[k] * sc, f[k + 1] * sc, f[k + 2] * sc, f[k + 3] * sc);
  }
}

DLLM_DEV void load_own(const float* src, int64_t bh, int cap_own, int d, int j0, int nk, float* dst) {
  const int vpr = d / 4, pitch = d + 4;
  for (int i = threadIdx.x; i < KB * vpr; i += 256) {
    const int r = i / vpr, c = (i - r * vpr) * 4;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < nk) x = *reinterpret_cast<const float4*>(src + (bh * cap_own + j0 + r) * (int64_t)d + c);
    *reinterpret_cast<float4*>(dst + r * pitch + c) = x;
  }
}

// Thread (rg, cg) of the 16 x 16: dot products of rows 4 rg .. 4 rg + 3 with keys cg and cg + 16.
DLLM_DEV void scores(const float* qs, const float* ks, int d, int rg, int cg, float (&s)[4][2]) {
  const int pitch = d + 4;
#pragma unroll
  for (int r = 0; r < 4; ++r) s[r][0] = s[r][1] = 0.f;
  for (int c = 0; c < d; c += 4) {
    const float4 k0 = *reinterpret_cast<const float4*>(ks + cg * pitch + c);
    const float4 k1 = *reinterpret_cast<const float4*>(ks + (cg + 16) * pitch + c);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float4 q = *reinterpret_cast<const float4*>(qs + (4 * rg + r) * pitch + c);
      s[r][0] = fmaf(q.x, k0.x, fmaf(q.y, k0.y, fmaf(q.z, k0.z, fmaf(q.w, k0.w, s[r][0]))));
      s[r][1] = fmaf(q.x, k1.x, fmaf(q.y, k1.y, fmaf(q.z, k1.z, fmaf(q.w, k1.w, s[r][1]))));
    }
  }
}

// One CTA per (b, h, row tile) and key split. Partial results (unnormalised o, m, l per row) go to the workspace when
// there are several splits.
__global__ void __launch_bounds__(256, 1) attn_kv8_simt_kernel(const Kv8AttnArgs a, SimtPlan p, float* part) {
  pdl_enter();
  extern __shared__ float sm[];
  const int d = a.d, pitch = d + 4, G = a.Hq / a.Hkv;
  float* qs = sm;
  float* ks = qs + ROWS * pitch;
  float* vs = ks + KB * pitch;
  float* ps = vs + KB * pitch;     // [ROWS][PD]
  const int tid = threadIdx.x, rg = tid >> 4, cg = tid & 15;
  int u = blockIdx.x;
  const int rt = u % p.n_rt;
  u /= p.n_rt;
  const int h = u % a.Hkv, b = u / a.Hkv;
  const int64_t bh = (int64_t)b * a.Hkv + h;
  const int len = kv8::prefix_len(a.lens, b, a.P);
  const int R0 = rt * ROWS, n_rows = a.Lq * G;
  load_rows(a, b, h, R0, a.scale * kLog2e, qs);

  // own keys visible to this thread's rows, and to any row of the tile
  int lim[4];
  const int last_q = (min(R0 + ROWS, n_rows) - 1) / G;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int64_t q = min(R0 + 4 * rg + r, n_rows - 1) / G;
    lim[r] = a.k_own ? (int)min((int64_t)a.Lq, (q / a.blk_len + 1) * a.blk_len) : 0;
  }
  const int own = a.k_own ? (int)min((int64_t)a.Lq, ((int64_t)(last_q / a.blk_len) + 1) * a.blk_len) : 0;
  const int tp = (len + KB - 1) / KB, tiles = tp + (own + KB - 1) / KB;
  const int t_begin = blockIdx.y * p.tps, t_end = min(tiles, t_begin + p.tps);

  float m[4], l[4], o[4][8];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.f;
#pragma unroll
    for (int c = 0; c < 8; ++c) o[r][c] = 0.f;
  }
  const int c0 = cg * 4, c1 = 64 + cg * 4;      // this thread's output columns
  for (int t = t_begin; t < t_end; ++t) {
    __syncthreads();
    const bool pre = t < tp;
    const int j0 = (pre ? t : t - tp) * KB, nk = min(KB, (pre ? len : own) - j0);
    if (pre) {
      load_codes(a.k_codes, a.k_scale, bh, a.cap, a.S, d, j0, nk, ks);
      load_codes(a.v_codes, a.v_scale, bh, a.cap, a.S, d, j0, nk, vs);
    } else {
      load_own(static_cast<const float*>(a.k_own), bh, a.cap_own, d, j0, nk, ks);
      load_own(static_cast<const float*>(a.v_own), bh, a.cap_own, d, j0, nk, vs);
    }
    __syncthreads();
    float s[4][2];
    scores(qs, ks, d, rg, cg, s);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int seen = pre ? nk : min(nk, lim[r] - j0);
      if (cg >= seen) s[r][0] = -INFINITY;
      if (cg + 16 >= seen) s[r][1] = -INFINITY;
      float mt = fmaxf(s[r][0], s[r][1]);
#pragma unroll
      for (int x = 8; x > 0; x >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, x));
      const float mn = fmaxf(m[r], mt);
      const bool any = mn != -INFINITY;
      // a NaN score is above no maximum but reaches its own weight, as in the formula
      const float p0 = cg < seen ? exp2f(s[r][0] - (any ? mn : 0.f)) : 0.f;
      const float p1 = cg + 16 < seen ? exp2f(s[r][1] - (any ? mn : 0.f)) : 0.f;
      const float alpha = m[r] == -INFINITY ? 0.f : exp2f(m[r] - mn);
      float sum = p0 + p1;
#pragma unroll
      for (int x = 8; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
      l[r] = l[r] * alpha + sum;
      m[r] = mn;
#pragma unroll
      for (int c = 0; c < 8; ++c) o[r][c] *= alpha;
      ps[(4 * rg + r) * PD + cg] = p0;
      ps[(4 * rg + r) * PD + cg + 16] = p1;
    }
    __syncwarp();                 // a row's weights are written and read by the same half-warp
    // own keys that a row does not see are left out: their V may be infinite or NaN. Keys that all four rows see come
    // first, without the question (asked for every key it took 3 x 300 keys from 17 to 20 us)
    int seen[4], all = nk;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      seen[r] = pre ? nk : lim[r] - j0;
      all = min(all, seen[r]);
    }
    auto add = [&](int j, auto ask) {
      float4 v0 = make_float4(0.f, 0.f, 0.f, 0.f), v1 = v0;
      if (c0 < d) v0 = *reinterpret_cast<const float4*>(vs + j * pitch + c0);
      if (c1 < d) v1 = *reinterpret_cast<const float4*>(vs + j * pitch + c1);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if (decltype(ask)::value && j >= seen[r]) continue;
        const float w = ps[(4 * rg + r) * PD + j];
        o[r][0] = fmaf(w, v0.x, o[r][0]);
        o[r][1] = fmaf(w, v0.y, o[r][1]);
        o[r][2] = fmaf(w, v0.z, o[r][2]);
        o[r][3] = fmaf(w, v0.w, o[r][3]);
        o[r][4] = fmaf(w, v1.x, o[r][4]);
        o[r][5] = fmaf(w, v1.y, o[r][5]);
        o[r][6] = fmaf(w, v1.z, o[r][6]);
        o[r][7] = fmaf(w, v1.w, o[r][7]);
      }
    };
    for (int j = 0; j < all; ++j) add(j, std::false_type{});
    for (int j = max(all, 0); j < nk; ++j) add(j, std::true_type{});
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int R = R0 + 4 * rg + r;
    if (R >= n_rows) continue;
    if (p.n_splits > 1) {
      float* dst = part + (((int64_t)blockIdx.x * p.n_splits + blockIdx.y) * ROWS + 4 * rg + r) * (d + 4);
      if (c0 < d) *reinterpret_cast<float4*>(dst + c0) = make_float4(o[r][0], o[r][1], o[r][2], o[r][3]);
      if (c1 < d) *reinterpret_cast<float4*>(dst + c1) = make_float4(o[r][4], o[r][5], o[r][6], o[r][7]);
      if (cg == 0) {
        dst[d] = m[r];
        dst[d + 1] = l[r];
      }
    } else {
      const float inv = l[r] == 0.f ? 0.f : 1.0f / l[r];      // no visible key: zeros; NaN stays
      const int64_t qh = ((int64_t)b * a.Lq + R / G) * a.Hq + h * G + R % G;
      float* dst = static_cast<float*>(a.out) + qh * d;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (c0 < d) dst[c0 + c] = o[r][c] * inv;
        if (c1 < d) dst[c1 + c] = o[r][4 + c] * inv;
      }
      if (cg == 0 && a.lse_out) a.lse_out[qh] = l[r] == 0.f ? -INFINITY : (m[r] + log2f(l[r])) * kLn2;
    }
  }
}

// One warp per row: the splits' partial results joined by their log-sum-exp, in split order.
__global__ void __launch_bounds__(256) attn_kv8_simt_merge_kernel(const Kv8AttnArgs a, SimtPlan p, const float* part) {
  pdl_enter();
  const int d = a.d, G = a.Hq / a.Hkv, n_rows = a.Lq * G, lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= (int64_t)a.B * a.Hkv * n_rows) return;
  const int64_t bh = row / n_rows;
  const int R = (int)(row - bh * n_rows), h = (int)(bh % a.Hkv), b = (int)(bh / a.Hkv);
  const float* src = part + ((bh * p.n_rt + R / ROWS) * p.n_splits * ROWS + R % ROWS) * (d + 4);
  const int64_t step = (int64_t)ROWS * (d + 4);
  float M = -INFINITY;
  for (int s = 0; s < p.n_splits; ++s) M = fmaxf(M, src[s * step + d]);
  float L = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < p.n_splits; ++s) {
    const float* q = src + s * step;
    const float l = q[d + 1];
    if (l == 0.f) continue;        // this split had no visible key
    const float w = exp2f(q[d] - M);
    L += w * l;
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (lane + 32 * c < d) o[c] = fmaf(w, q[lane + 32 * c], o[c]);
  }
  const float inv = L == 0.f ? 0.f : 1.0f / L;
  const int64_t qh = ((int64_t)b * a.Lq + R / G) * a.Hq + h * G + R % G;
#pragma unroll
  for (int c = 0; c < 4; ++c)
    if (lane + 32 * c < d) static_cast<float*>(a.out)[qh * d + lane + 32 * c] = o[c] * inv;
  if (lane == 0 && a.lse_out) a.lse_out[qh] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
}

// One cluster of C CTAs per (b, h, tile of KB keys): the weights of all rows on its keys, each CTA on every C-th row tile;
// the first CTA adds the others' sums to its own, in their order. Bound by shared-memory reads (6 vectors for 32 products) and
// by the latency of a row tile where there are few CTAs: 512 rows on 1000 keys, one head of 128, 15.6 us with clusters of 8,
// 53 us with one CTA per key tile; 2000 keys of 16 (row, head)s with one row tile 32 us.
__global__ void __launch_bounds__(256) attn_mass_kv8_simt_kernel(const Kv8AttnArgs a, int n_kt, int n_rt, int C) {
  pdl_enter();
  extern __shared__ float sm[];
  const int d = a.d, pitch = d + 4, G = a.Hq / a.Hkv;
  float* qs = sm;
  float* ks = qs + ROWS * pitch;
  float* red = ks + KB * pitch;     // [16][KB]
  const int tid = threadIdx.x, rg = tid >> 4, cg = tid & 15;
  __shared__ float sums[KB];
  const int rank = blockIdx.x % C, tile = blockIdx.x / C, kt = tile % n_kt;
  const int64_t bh = tile / n_kt;
  const int h = (int)(bh % a.Hkv), b = (int)(bh / a.Hkv);
  const int len = kv8::prefix_len(a.lens, b, a.P), j0 = kt * KB, nk = min(KB, len - j0);
  if (nk <= 0) return;      // the whole cluster
  load_codes(a.k_codes, a.k_scale, bh, a.cap, a.S, d, j0, nk, ks);
  float sum0 = 0.f, sum1 = 0.f;
  const int n_rows = a.Lq * G;
  for (int rt = rank; rt < n_rt; rt += C) {
    __syncthreads();
    load_rows(a, b, h, rt * ROWS, a.scale * kLog2e, qs);
    __syncthreads();
    float s[4][2];
    scores(qs, ks, d, rg, cg, s);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int R = rt * ROWS + 4 * rg + r;
      if (R < n_rows) {
        const float lse = a.lse_in[((int64_t)b * a.Lq + R / G) * a.Hq + h * G + R % G];
        if (lse != -INFINITY) {     // a row that saw no key gives no weight
          sum0 += exp2f(s[r][0] - lse * kLog2e);
          sum1 += exp2f(s[r][1] - lse * kLog2e);
        }
      }
    }
  }
  red[rg * KB + cg] = sum0;
  red[rg * KB + cg + 16] = sum1;
  __syncthreads();
  if (tid < nk) {
    float t = 0.f;
    for (int g = 0; g < 16; ++g) t += red[g * KB + tid];
    sums[tid] = t;
  }
  if (C > 1) kv8::cluster_sync();
  if (rank == 0 && tid < nk) {
    float t = sums[tid];
    for (int r = 1; r < C; ++r) t += __uint_as_float(kv8::peer_u32(&sums[tid], r));
    const int64_t at = bh * a.cap + j0 + tid;
    a.mass_out[at] = a.mass_in ? fmaf(a.decay, a.mass_in[at], t) : t;
  }
  if (C > 1) kv8::cluster_sync();      // no CTA leaves while its sums are read
}

}  // namespace

size_t attn_kv8_simt_workspace_bytes(int B, int Lq, int Hq, int Hkv, int d, int P, int own) {
  const SimtPlan p = simt_plan(B, Lq, Hq, Hkv, P, own);
  if (p.n_splits <= 1) return 0;
  return (size_t)B * Hkv * p.n_rt * p.n_splits * ROWS * (d + 4) * 4;
}

int launch_attn_kv8_simt(const Kv8AttnArgs& a, cudaStream_t s) {
  const SimtPlan p = simt_plan(a.B, a.Lq, a.Hq, a.Hkv, a.P, a.k_own != nullptr);
  const size_t smem = ((size_t)(ROWS + 2 * KB) * (a.d + 4) + ROWS * PD) * 4;
  const int st = set_max_smem<attn_kv8_simt_kernel>(((ROWS + 2 * KB) * 132 + ROWS * PD) * 4);
  if (st) return st;
  float* part = static_cast<float*>(a.ws);
  launch_pdl(attn_kv8_simt_kernel, dim3((unsigned)(a.B * a.Hkv * p.n_rt), p.n_splits), 256, smem, s, a, p, part);
  DLLM_CHECK_LAUNCH("attn_kv8_simt_kernel");
  if (p.n_splits > 1) {
    const int64_t rows = (int64_t)a.B * a.Lq * a.Hq;
    launch_pdl(attn_kv8_simt_merge_kernel, (unsigned)((rows + 7) / 8), 256, 0, s, a, p, (const float*)part);
    DLLM_CHECK_LAUNCH("attn_kv8_simt_merge_kernel");
  }
  return DLLM_OK;
}

int launch_attn_mass_kv8_simt(const Kv8AttnArgs& a, cudaStream_t s) {
  const int n_kt = (a.P + KB - 1) / KB, n_rt = (a.Lq * (a.Hq / a.Hkv) + ROWS - 1) / ROWS;
  const size_t smem = ((size_t)(ROWS + KB) * (a.d + 4) + 16 * KB) * 4;
  // with few key tiles, CTAs share the row tiles: up to two CTAs per SM, each with a row tile at least
  const int64_t tiles = (int64_t)a.B * a.Hkv * n_kt;
  int C = 1;
  while (C < 8 && 2 * C <= n_rt && 2 * C * tiles <= 2 * num_sms()) C *= 2;
  const int st = set_max_smem<attn_mass_kv8_simt_kernel>(((ROWS + KB) * 132 + 16 * KB) * 4);
  if (st) return st;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * C), 1, 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, attn_mass_kv8_simt_kernel, a, n_kt, n_rt, C);
  if (e != cudaSuccess) return dllm_host::cuda_status(e, "cudaLaunchKernelEx(attn_mass_kv8_simt_kernel)");
  DLLM_CHECK_LAUNCH("attn_mass_kv8_simt_kernel");
  return DLLM_OK;
}

size_t attn_kv8_workspace_bytes(int B, int Lq, int Hq, int Hkv, int d, int P, int own, int dtype) {
  if (dtype == DLLM_BF16) return attn_kv8_tc_workspace_bytes(B, Lq, Hq, Hkv);
  return attn_kv8_simt_workspace_bytes(B, Lq, Hq, Hkv, d, P, own);
}
int launch_attn_kv8(const Kv8AttnArgs& a, cudaStream_t s) {
  return a.dtype == DLLM_BF16 ? launch_attn_kv8_tc(a, s) : launch_attn_kv8_simt(a, s);
}
int launch_attn_mass_kv8(const Kv8AttnArgs& a, cudaStream_t s) {
  return a.dtype == DLLM_BF16 ? launch_attn_mass_kv8_tc(a, s) : launch_attn_mass_kv8_simt(a, s);
}

}  // namespace dllm
