// The 8-bit KV cache's data movement: quantising K/V rows into it, and evicting its least attended positions.
//
// Format: E4M3 codes [B, Hkv, cap, d] and one fp32 scale per run of S tokens and kv head. The scale is the least
// power of two that brings the run's largest magnitude to at most 448, so x / scale is exact and each value is rounded
// once, to four significant bits (E4M3, nearest even): half a step is 2^-4 of the value, whatever the scale, so a
// power of two costs no precision against amax / 448, and it lets eviction move rows between runs without rounding
// them again.
#include "kv8.cuh"
#include "kv8.h"
#include "misc.h"
#include <algorithm>

namespace dllm {
namespace {

constexpr int kThreads = 256;

// ------------------------------------------------------------------------------------------------ store
// A group of TG threads quantises one run (up to S rows of d elements): its vectors are read once, kept in registers
// while the group's largest magnitude is found, then written as codes. TG = 2 S gives a thread at most VPT = 8
// 16-byte vectors of bf16 (16 of fp32) at d = 128. Bound by HBM: 8 rows x 4 kv heads x 4091 tokens 19.9 us, 5.1 TB/s (32.7 us
// with magnitudes compared as floats and a division per vector: 7 instructions a value were the limit then).
template <typename T, int TG, int VPT>
__global__ void __launch_bounds__(kThreads) kv8_store_kernel(const Kv8StoreArgs a, int runs) {
  pdl_enter();
  constexpr int VE = 16 / (int)sizeof(T);
  __shared__ float red[kThreads / 32];
  const int tid = threadIdx.x, gt = tid % TG;
  const int64_t unit = (int64_t)blockIdx.x * (kThreads / TG) + tid / TG;
  const bool is_v = blockIdx.y != 0;
  const bool live = unit < (int64_t)a.B * a.Hkv * runs;
  const int run = live ? (int)(unit % runs) : 0;
  const int64_t bh = live ? unit / runs : 0;
  const int b = (int)(bh / a.Hkv);
  const int row0 = a.dst_rows ? a.dst_rows[b] : a.dst_row;
  // a destination outside the cache or inside a run: nothing is written for this batch row
  const bool ok = live && row0 >= 0 && row0 % a.S == 0 && row0 <= a.cap - a.n;
  const int t0 = run * a.S, rows = min(a.S, a.n - t0);
  const int vpr = a.d / VE;                       // vectors per row
  const int nvec = ok ? rows * vpr : 0;
  const T* src = static_cast<const T*>(is_v ? a.v : a.k) + bh * (int64_t)a.cap_src * a.d;
  uint4 vec[VPT];
  // without a position list the run's source rows are contiguous, and so are its vectors
  const T* run_src = src + ((int64_t)a.src_row + t0) * a.d;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int id = gt + i * TG;
    vec[i] = make_uint4(0, 0, 0, 0);
    if (id < nvec) {
      if (!a.src_pos) {
        vec[i] = ld_nc_v4(run_src + id * VE);
      } else {
        const int r = id / vpr, row = a.src_pos[(int64_t)b * a.pos_stride + t0 + r];
        if (row >= 0 && row < a.cap_src) vec[i] = ld_nc_v4(src + (int64_t)row * a.d + (id - r * vpr) * VE);
      }
    }
  }
  // Magnitudes compare as their bits. Infinities and NaN, which do not count (infinities saturate, NaN stays NaN), show as
  // the largest patterns; the values are then looked at one by one.
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const uint4& u = vec[i];
    if constexpr (sizeof(T) == 2) {
      top = __vmaxu2(top, __vmaxu2(__vmaxu2(u.x & 0x7fff7fffu, u.y & 0x7fff7fffu),
                                   __vmaxu2(u.z & 0x7fff7fffu, u.w & 0x7fff7fffu)));
    } else {
      top = max(top, max(max(u.x & 0x7fffffffu, u.y & 0x7fffffffu), max(u.z & 0x7fffffffu, u.w & 0x7fffffffu)));
    }
  }
  if constexpr (sizeof(T) == 2) top = max(top & 0xffffu, top >> 16) << 16;
  float amax = __uint_as_float(top);
  if (top >= 0x7f800000u) {
    amax = 0.f;
#pragma unroll 1
    for (int id = gt; id < nvec; id += TG) {
      const int r = id / vpr, c = id - r * vpr;
      int row = a.src_row + t0 + r;
      if (a.src_pos) row = a.src_pos[(int64_t)b * a.pos_stride + t0 + r];
      if (row < 0 || row >= a.cap_src) continue;
      for (int j = 0; j < VE; ++j) {
        const float m = fabsf(to_f32(src[(int64_t)row * a.d + c * VE + j]));
        if (m < INFINITY) amax = fmaxf(amax, m);
      }
    }
  }
  amax = warp_max(amax);
  if constexpr (TG > 32) {
    if ((tid & 31) == 0) red[tid >> 5] = amax;
    __syncthreads();
    const int w0 = tid / TG * (TG / 32);
#pragma unroll
    for (int w = 0; w < TG / 32; ++w) amax = fmaxf(amax, red[w0 + w]);
  }
  if (!ok) return;
  const int k = kv8::scale_exp(amax);
  const float inv = kv8::exp2i(-k);
  uint8_t* dst = (is_v ? a.v_codes : a.k_codes) + (bh * (int64_t)a.cap + row0 + t0) * a.d;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int id = gt + i * TG;
    if (id < nvec) {
      const uint32_t u[4] = {vec[i].x, vec[i].y, vec[i].z, vec[i].w};
      uint32_t w[VE / 4];
#pragma unroll
      for (int j = 0; j < VE / 4; ++j) {
        float f[4];
        if constexpr (sizeof(T) == 2) {
          f[0] = __uint_as_float(u[2 * j] << 16);
          f[1] = __uint_as_float(u[2 * j] & 0xffff0000u);
          f[2] = __uint_as_float(u[2 * j + 1] << 16);
          f[3] = __uint_as_float(u[2 * j + 1] & 0xffff0000u);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) f[k] = __uint_as_float(u[k]);
        }
        w[j] = kv8::f32x2_to_e4m3x2(f[0] * inv, f[1] * inv) | (kv8::f32x2_to_e4m3x2(f[2] * inv, f[3] * inv) << 16);
      }
      // the run's rows are contiguous, so vector id of the source lands at id * VE codes
      if constexpr (VE == 8)
        *reinterpret_cast<uint2*>(dst + (int64_t)id * 8) = make_uint2(w[0], w[1]);
      else
        *reinterpret_cast<uint32_t*>(dst + (int64_t)id * 4) = w[0];
    }
  }
  if (gt == 0) {
    const int n_runs = (a.cap + a.S - 1) / a.S;
    (is_v ? a.v_scale : a.k_scale)[bh * n_runs + row0 / a.S + run] = kv8::exp2i(k);
  }
}

// ------------------------------------------------------------------------------------------------ evict
// Ordered key of a position: the bits of its accumulated weight (non-negative, so bit order is value order; NaN and
// negative values count as 0), above every weight for the positions that are always kept.
constexpr uint32_t kForced = 0x7f800001u;

// One cluster per selection (batch row, or batch row and kv head), each of its C CTAs on a contiguous part of the
// positions: the n_keep-th largest key by a radix search over digits of 11, 11 and 10 bits (histograms added up through
// distributed shared memory; 11 bits spread the exponents of a heavy-tailed accumulator over enough counters that the
// shared-memory atomics hardly collide), then the kept positions in increasing order (equal keys at the threshold: the
// lower position first). Keys stay in shared memory where the part fits, else in the workspace.
// Bound by its dependent passes: with the gather 16.8 us for 8 x 4096 positions of 4 heads (45 us with one CTA, byte digits
// and keys in the workspace), 28.9 us for 4 heads of 131072 (390 us). A CTA per 4096 positions, at most 8: 1024 or 2048 took
// 27.3 and 24.4 us where 4096 took 23.7.
constexpr int kSelThreads = 1024, kBins = 2048;
constexpr int kSelPart = 4096;              // positions for which a selection gets another CTA
constexpr int kSelSmemKeys = 32768;         // keys of a part that fit shared memory

__global__ void __launch_bounds__(kSelThreads, 1) kv8_select_kernel(const Kv8EvictArgs a, int C, uint32_t* __restrict__ keys,
                                                                    int32_t* __restrict__ index) {
  pdl_enter();
  extern __shared__ uint32_t dyn[];
  __shared__ uint32_t hist[2][kBins], sums[kBins];
  __shared__ uint32_t wsum[32], wsum2[32];
  __shared__ uint32_t s_bin, s_need;
  __shared__ uint32_t counts[2];             // of this part: keys above the threshold, keys equal to it
  const int rank = blockIdx.x % C, sel = blockIdx.x / C;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int Hs = a.per_head ? a.Hkv : 1;
  const int b = sel / Hs, h = sel - b * Hs;
  const int len = kv8::prefix_len(a.lens, b, a.P);
  const int keep = min(len, a.n_keep);
  const int part = (len + C - 1) / C, lo = min(len, rank * part), n = min(len, lo + part) - lo;
  uint32_t* key = (a.P + C - 1) / C <= kSelSmemKeys ? dyn : keys + (int64_t)sel * a.P + lo;
  if (h == 0 && rank == 0 && tid == 0) a.len_out[b] = keep;
  const float* m = a.mass + (int64_t)b * a.Hkv * a.cap;
  // kFlight positions of a thread are loaded before the first is used
  constexpr int kFlight = 8;
  const int heads = a.per_head ? 1 : a.Hkv;
  if (a.per_head) m += (int64_t)h * a.cap;
  for (int i0 = tid; i0 < n; i0 += kFlight * kSelThreads) {
    double t[kFlight];
#pragma unroll
    for (int k = 0; k < kFlight; ++k) t[k] = 0.0;
    for (int g = 0; g < heads; ++g) {        // summed in 64 bits, in head order
      float f[kFlight];
#pragma unroll
      for (int k = 0; k < kFlight; ++k)
        f[k] = i0 + k * kSelThreads < n ? m[(int64_t)g * a.cap + lo + i0 + k * kSelThreads] : 0.f;
#pragma unroll
      for (int k = 0; k < kFlight; ++k) t[k] += (double)f[k];
    }
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      const int i = i0 + k * kSelThreads, j = lo + i;
      const float f = (float)t[k];
      if (i < n) key[i] = (j < a.n_first || j >= len - a.n_last) ? kForced : __float_as_uint(f > 0.f ? f : 0.f);
    }
  }
  uint32_t prefix = 0, mask = 0;
  uint32_t need = (uint32_t)keep;      // how many of the keys that match the prefix are still to be taken
  const bool all = keep == len;        // the whole cluster agrees
  for (int pass = 0; pass < 3 && !all; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
    uint32_t* hs = hist[pass & 1];
    hs[tid] = hs[tid + kSelThreads] = 0;
    __syncthreads();
#pragma unroll 4
    for (int i = tid; i < n; i += kSelThreads) {
      const uint32_t u = key[i];
      if ((u & mask) == prefix) atomicAdd(&hs[(u >> shift) & ((1u << bits) - 1u)], 1u);
    }
    kv8::cluster_sync();
    if (C > 1) {      // each CTA adds up its share of the bins over the cluster and gives every CTA the sums
      const int per = kBins / C;
      for (int i = tid; i < per; i += kSelThreads) {
        const int bin = rank * per + i;
        uint32_t t = 0;
        for (int r = 0; r < C; ++r) t += kv8::peer_u32(&hs[bin], r);
        for (int r = 0; r < C; ++r) kv8::peer_store_u32(&sums[bin], r, t);
      }
      kv8::cluster_sync();
    }
    // thread t holds bins 2047 - 2 t and 2046 - 2 t: a prefix sum over the threads counts from the largest key down
    const uint32_t* tot = C > 1 ? sums : hs;
    const uint32_t c0 = tot[kBins - 1 - 2 * tid], c1 = tot[kBins - 2 - 2 * tid];
    uint32_t run = c0 + c1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += y;
    }
    if (lane == 31) wsum[w] = run;
    __syncthreads();
    const uint32_t above = run - (c0 + c1) + __reduce_add_sync(0xffffffffu, lane < w ? wsum[lane] : 0u);
    if (above < need && need <= above + c0 + c1) {      // exactly one thread of the CTA
      const bool first = need <= above + c0;
      s_bin = (uint32_t)(kBins - 1 - 2 * tid) - (first ? 0u : 1u);
      s_need = need - above - (first ? 0u : c0);
    }
    __syncthreads();
    prefix |= s_bin << shift;
    need = s_need;
    mask |= ((1u << bits) - 1u) << shift;
  }
  // prefix is now the threshold: larger keys are kept, and the first `need` equal ones. Each warp takes a contiguous
  // stretch of the part: it counts, the counts are summed over warps and CTAs, and it writes.
  const int per_warp = (n + 31) / 32, w0 = min(n, w * per_warp), w1 = min(n, w0 + per_warp);
  uint32_t gt = 0, eq = 0;
  __syncthreads();
  for (int i0 = w0; i0 < w1; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t u = i < w1 ? key[i] : 0u;
    gt += __popc(__ballot_sync(0xffffffffu, i < w1 && (all || u > prefix)));
    eq += __popc(__ballot_sync(0xffffffffu, i < w1 && !all && u == prefix));
  }
  if (lane == 0) {
    wsum[w] = gt;
    wsum2[w] = eq;
  }
  __syncthreads();
  uint32_t gt_before = __reduce_add_sync(0xffffffffu, lane < w ? wsum[lane] : 0u);
  uint32_t eq_before = __reduce_add_sync(0xffffffffu, lane < w ? wsum2[lane] : 0u);
  const uint32_t gt_all = __reduce_add_sync(0xffffffffu, wsum[lane]), eq_all = __reduce_add_sync(0xffffffffu, wsum2[lane]);
  if (tid == 0) {
    counts[0] = gt_all;
    counts[1] = eq_all;
  }
  kv8::cluster_sync();
  for (int r = 0; r < rank; ++r) {
    gt_before += kv8::peer_u32(&counts[0], r);
    eq_before += kv8::peer_u32(&counts[1], r);
  }
  kv8::cluster_sync();        // no CTA leaves while another reads its counts
  const int32_t* pos = a.pos ? a.pos + (int64_t)sel * a.cap + lo : nullptr;
  int32_t* out = a.keep_pos + (int64_t)sel * a.cap_out;
  int32_t* idx = index + (int64_t)sel * a.n_keep;
  const unsigned below = (1u << lane) - 1u;
  for (int i0 = w0; i0 < w1; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t u = i < w1 ? key[i] : 0u;
    const unsigned g = __ballot_sync(0xffffffffu, i < w1 && (all || u > prefix));
    const unsigned e = __ballot_sync(0xffffffffu, i < w1 && !all && u == prefix);
    const uint32_t eq_rank = eq_before + __popc(e & below);
    const bool take = (g >> lane & 1u) || ((e >> lane & 1u) && eq_rank < need);
    if (take) {
      const uint32_t at = gt_before + __popc(g & below) + min(eq_rank, need);
      idx[at] = lo + i;
      out[at] = pos ? pos[i] : lo + i;
    }
    gt_before += __popc(g);
    eq_before += __popc(e);
  }
}

// A group of TG = 2 S threads moves one run of S kept rows of a (batch row, kv head): K and V codes and the
// accumulated weights. The run's scale is the largest of its rows' scales; a row whose scale is smaller has its codes
// multiplied by the ratio and rounded again, which for power-of-two scales changes only values below 2^-6 of the new
// scale (E4M3's subnormals). Bound by the latency of position list -> row: all of a thread's vectors are in flight at once.
template <int TG>
__global__ void __launch_bounds__(kThreads) kv8_gather_kernel(const Kv8EvictArgs a, const int32_t* __restrict__ index,
                                                              int runs) {
  pdl_enter();
  constexpr int S = TG / 2, GROUPS = kThreads / TG;
  __shared__ int src_s[GROUPS][S];
  __shared__ float sc_s[GROUPS][2][S];
  __shared__ float top_s[2][kThreads / 32];
  const int tid = threadIdx.x, gt = tid % TG, grp = tid / TG;
  const int64_t unit = (int64_t)blockIdx.x * GROUPS + grp;
  const bool live = unit < (int64_t)a.B * a.Hkv * runs;
  const int run = live ? (int)(unit % runs) : 0;
  const int64_t bh = live ? unit / runs : 0;
  const int b = (int)(bh / a.Hkv);
  const int keep = min(kv8::prefix_len(a.lens, b, a.P), a.n_keep);
  const int t0 = run * S, rows = live ? min(S, keep - t0) : 0;
  const int64_t sel = a.per_head ? bh : b;
  const int64_t runs_in = (a.cap + S - 1) / S, runs_out = (a.cap_out + S - 1) / S;
  float sk = 0.f, sv = 0.f;
  if (gt < rows) {
    const int j = index[sel * a.n_keep + t0 + gt];
    src_s[grp][gt] = j;
    sc_s[grp][0][gt] = sk = a.k_scale[bh * runs_in + j / S];
    sc_s[grp][1][gt] = sv = a.v_scale[bh * runs_in + j / S];
    a.mass_out[bh * (int64_t)a.cap_out + t0 + gt] = a.mass[bh * (int64_t)a.cap + j];
  }
  sk = warp_max(sk);
  sv = warp_max(sv);
  if ((tid & 31) == 0) {
    top_s[0][tid >> 5] = sk;
    top_s[1][tid >> 5] = sv;
  }
  __syncthreads();
  if (rows <= 0) return;
  // S d / 16 vectors of K and as many of V, at most 4 of each per thread (d <= 128), all loaded before the first is used
  const int vpr = a.d / 16, nvec = rows * vpr;
  const int per = (65536 + vpr - 1) / vpr;        // id / vpr = id * per >> 16 for id < 1024 and vpr <= 8
  uint4 vec[2][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int id = gt + i * TG;
    if (id < nvec) {
      const int r = id * per >> 16;
      const int64_t at = bh * (int64_t)a.cap * a.d + (int64_t)src_s[grp][r] * a.d + (id - r * vpr) * 16;
      vec[0][i] = ld_nc_v4(a.k_codes + at);
      vec[1][i] = ld_nc_v4(a.v_codes + at);
    }
  }
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < (S + 31) / 32; ++i) top = fmaxf(top, top_s[kv][grp * (TG / 32) + i]);
    uint8_t* dst = (kv ? a.v_out : a.k_out) + (bh * (int64_t)a.cap_out + t0) * a.d;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int id = gt + i * TG;
      if (id >= nvec) break;
      uint4 u = vec[kv][i];
      const float old = sc_s[grp][kv][id * per >> 16];
      if (old != top) {
        const float ratio = top > 0.f ? old / top : 0.f;
        float f[16];
        kv8::codes16_to_f32(u, f);
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          o[j] = kv8::f32x2_to_e4m3x2(f[4 * j] * ratio, f[4 * j + 1] * ratio) |
                 (kv8::f32x2_to_e4m3x2(f[4 * j + 2] * ratio, f[4 * j + 3] * ratio) << 16);
        u = make_uint4(o[0], o[1], o[2], o[3]);
      }
      *reinterpret_cast<uint4*>(dst + (int64_t)id * 16) = u;
    }
    if (gt == 0) (kv ? a.v_scale_out : a.k_scale_out)[bh * runs_out + run] = top;
  }
}

}  // namespace

int launch_kv8_store(const Kv8StoreArgs& a, cudaStream_t s) {
  const int runs = (a.n + a.S - 1) / a.S;
  const int64_t units = (int64_t)a.B * a.Hkv * runs;
  const int per = kThreads / (2 * a.S);
  const dim3 grid((unsigned)((units + per - 1) / per), 2);
#define DLLM_STORE(T, V)                                                                        \
  switch (a.S) {                                                                                \
    case 16: launch_pdl(kv8_store_kernel<T, 32, V>, grid, kThreads, 0, s, a, runs); break;      \
    case 32: launch_pdl(kv8_store_kernel<T, 64, V>, grid, kThreads, 0, s, a, runs); break;      \
    case 64: launch_pdl(kv8_store_kernel<T, 128, V>, grid, kThreads, 0, s, a, runs); break;     \
    default: launch_pdl(kv8_store_kernel<T, 256, V>, grid, kThreads, 0, s, a, runs); break;     \
  }
  if (a.dtype == DLLM_BF16) {
    DLLM_STORE(__nv_bfloat16, 8)
  } else {
    DLLM_STORE(float, 16)
  }
#undef DLLM_STORE
  DLLM_CHECK_LAUNCH("kv8_store_kernel");
  return DLLM_OK;
}

size_t kv8_evict_workspace_bytes(int B, int Hkv, int P, int n_keep, int per_head) {
  const size_t sel = (size_t)B * (per_head ? Hkv : 1);
  return (sel * P * 4 + 255) / 256 * 256 + sel * n_keep * 4;
}

int launch_kv8_evict(const Kv8EvictArgs& a, cudaStream_t s) {
  const int64_t sel = (int64_t)a.B * (a.per_head ? a.Hkv : 1);
  uint32_t* keys = static_cast<uint32_t*>(a.ws);
  int32_t* index = reinterpret_cast<int32_t*>(static_cast<char*>(a.ws) + ((size_t)sel * a.P * 4 + 255) / 256 * 256);
  {
    // CTAs of a selection: enough that a thread handles few positions, at most a portable cluster
    int C = 1;
    while (C < 8 && C * kSelPart < a.P) C *= 2;
    const int part = (a.P + C - 1) / C;
    const size_t smem = part <= kSelSmemKeys ? (size_t)part * 4 : 0;
    const int st = set_max_smem<kv8_select_kernel>(kSelSmemKeys * 4);
    if (st) return st;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(sel * C), 1, 1);
    cfg.blockDim = dim3(kSelThreads, 1, 1);
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
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kv8_select_kernel, a, C, keys, index);
    if (e != cudaSuccess) return dllm_host::cuda_status(e, "cudaLaunchKernelEx(kv8_select_kernel)");
  }
  DLLM_CHECK_LAUNCH("kv8_select_kernel");
  const int most = min(a.n_keep, a.P);
  if (most == 0) return DLLM_OK;
  const int runs = (most + a.S - 1) / a.S;
  const int64_t units = (int64_t)a.B * a.Hkv * runs;
  const int per = kThreads / (2 * a.S);
  const unsigned grid = (unsigned)((units + per - 1) / per);
  switch (a.S) {
    case 16: launch_pdl(kv8_gather_kernel<32>, grid, kThreads, 0, s, a, (const int32_t*)index, runs); break;
    case 32: launch_pdl(kv8_gather_kernel<64>, grid, kThreads, 0, s, a, (const int32_t*)index, runs); break;
    case 64: launch_pdl(kv8_gather_kernel<128>, grid, kThreads, 0, s, a, (const int32_t*)index, runs); break;
    default: launch_pdl(kv8_gather_kernel<256>, grid, kThreads, 0, s, a, (const int32_t*)index, runs); break;
  }
  DLLM_CHECK_LAUNCH("kv8_gather_kernel");
  return DLLM_OK;
}

}  // namespace dllm
