// Attention over an 8-bit prefix cache and the block's own K/V on the 5th-generation tensor cores (tcgen05 + TMEM),
// bf16 queries, head dim 128. The formulas are in attn_kv8.cu.
//
// Work: the (query, head of the group) rows of a (batch row, kv head) are cut into tiles of 128 rows, each a unit of
// ceil(len[b] / 128) prefix key tiles and the own key tiles its last query sees. All units' key tiles in a row are
// dealt to one CTA per SM in equal contiguous shares, a unit's end counting for some tiles too, so rows of different
// lengths, few rows and many rows all keep every SM busy equally long; a unit that spans several CTAs leaves its partial
// results (unnormalised o, m, l per row) in the workspace and a second kernel joins them.
//
// Per key tile of 128:
//   S = Q K^T   kind::f8f6f4, K's codes straight from the cache by TMA (never converted). The queries are exact
//               to 2^-17.8 of their row's largest magnitude as two E4M3 parts: q * 2^-k brought to at most 448, hi =
//               E4M3(q), lo = E4M3(q - hi) (bf16 has 8 significant bits, two parts of 4); both parts accumulate into the
//               same fp32 S. fp8 MMAs run at twice the bf16 rate, so the two cost what one bf16 product would.
//               Own keys are split the same way by the converter warps (two parts: four products), each with a
//               power-of-two scale of its own, and own V rows too: no row's precision depends on another row, least of all
//               on one that the query does not see (a scale for 128 own keys was 5 % faster in the smallest calls, and let
//               hidden rows change the results of earlier queries).
//   softmax     one thread per row; x = S * (2^k scale log2(e) k_scale) + log2(v_scale) - m: the V scale of each run rides
//               in the exponent, so that P V needs no scaled copy of V; the row sum divides it out again run by run.
//               P = 2^(x + 2) as f16. The reference m is not a running maximum: it is the largest of the first 32 scores
//               that a row sees, and moves (rescaling O and the P of the tile so far) only when 32 weights add up to more
//               than 30000, that is before one could leave f16's range. So the scores are read once, and no maximum is
//               taken on the way. What is rounded is weight times V scale: it keeps 11 bits down to 2^-16 of the
//               reference and is dropped below 2^-27 (n keys lose at most n 2^-26 of the largest such product times their
//               codes, where the reference has moved and rounded them twice).
//   O += P V    kind::f16 with A = P from TMEM and B = V as f16 (every E4M3 value is one), written from the codes by four
//               converter warps into the MN-major layout.
// Tensor time of a tile: 8 + 8 MMAs of 64 clocks, and about 250 clocks for each of the two changes of the instruction
// descriptor (measured on bare loops: 512 clocks per 8 MMAs of one kind, 756 when S and P V alternate, whatever their
// operand sources), so about 1510 clocks, against 1420 for the tile's bytes at one SM's share of the HBM rate and 1024
// for its exponentials. Two softmax groups of four warps take alternate tiles, one thread per row, each with an S and an O
// of its own in TMEM and references of its own; their results are joined at the end of a unit. Measured on the way, 8 x 32
// queries of 16 heads over 32768 keys: two threads per row on the same tile 134 us; one O with a reference that the groups
// pass on to each other and a pass for the maximum 105 us.
// Measured (with the joining kernel, 1965 MHz but for the long case's power limit): those 8 rows 103-108 us (2.5-2.6 TB/s of
// codes, 0.4 of the bf16 tensor rate), 16 x 32 queries over up to 2688 keys 31.6 us, one row over 1024 keys 15.8 us. Bound
// by a group's chain (its S waits for the P V before it: about 2100 clocks a tile with two groups in flight), in small
// calls by set-up (2 us to the first load, 5 to the first score) and the joining kernel.
//
// Roles: warp 0 TMA, warp 1 MMA, warps 2 and 3 the runs' scales (alternate prefix tiles), warps 4-7 and 8-11 softmax (even
// and odd tiles), warps 12-15 convert Q, V and the own rows. Warps whose rows are all past the last only
// keep count. Every wait is bounded; a wait that gives up sets the abort flag and the status word, after which every
// role runs through its loops without waiting, issuing or storing anything.
#include "attn_tc.cuh"
#include "kv8.cuh"
#include "kv8.h"
#include "misc.h"
#include <algorithm>
#include <type_traits>

namespace dllm {
namespace {

constexpr int NT = 512;
constexpr int KT = 128;                    // keys per tile = rows per unit
constexpr int KSTAGE = 128 * 128;          // K or V codes of a tile: 16 KB
constexpr int VTILE = 2 * 128 * 64 * 2;    // V of a tile as f16: two 64-wide chunks of 16 KB
constexpr int VCHUNK = VTILE / 2;
constexpr int NK = 3, NV = 2, NB = 2;      // stages of the K and V code rings; f16 V buffers
// Key tiles that a unit's end (products, merge of the halves, output, the next unit's start) counts for in the CTAs' shares.
// Measured with 0 / 3 / 4 / 5 / 8 (us, the middle of three runs in turn; runs of one differ by 0.5 at most): 16 x 2688 34.6 /
// 31.7 / 31.6 / 32.6 / 33.9, 8 x 32768 110.1 / 108.2 / 107.3 / 107.3 / 107.2, 64 x 4001 single tokens 86.3 / 76.5 / 73.1 / 72.9 /
// 76.1, 2 x 500 rows on 4000 keys 78.2 / 77.4 / 77.7 / 76.7 / 80.7: 4 and 5 are alike, 3 and 8 lose somewhere.
constexpr int kUnitEnd = 4;
constexpr float kMost = 30000.f;           // 32 weights that add up to more move the reference
constexpr float kOff = 2.f;                // P is 2^2 times the weight relative to the reference
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// named barriers: the 128 converter threads; 2 + i: the two warps of rows 32 i ..
constexpr int kBarConv = 1, kBarPair = 2;
constexpr int kPart = 33 * 128 * 4;        // floats of one partial result: 32 float4 columns and (m, l, -, -), by row

// Code size is speed here: four kinds of warps run different loops on every scheduler, and what does not fit the
// instruction caches is fetched again for every tile. Waits are therefore written compactly (the reason for giving up is
// left in the abort flag and reported once, at the end), divisions are multiplications, and every loop body appears once.
DLLM_DEV bool wait_for(uint64_t* bar, uint32_t parity, int* abort_flag, int code) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .u32 n, f;\n\t"
      "mov.u32 n, 0;\n\t"
      "WAIT_%=:\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "mov.u32 %0, 1;\n\t"
      "@p bra DONE_%=;\n\t"
      "ld.volatile.shared.u32 f, [%3];\n\t"
      "mov.u32 %0, 0;\n\t"
      "setp.ne.u32 p, f, 0;\n\t"
      "@p bra DONE_%=;\n\t"
      "add.u32 n, n, 1;\n\t"
      "setp.lt.u32 p, n, 4194304;\n\t"
      "@p bra WAIT_%=;\n\t"
      "st.volatile.shared.u32 [%3], %4;\n\t"
      "DONE_%=:\n\t}"
      : "=&r"(ok)
      : "r"(tc::smem_u32(bar)), "r"(parity), "r"(tc::smem_u32(abort_flag)), "r"(code)
      : "memory");
  return ok != 0;
}

// Whether the phase of the given parity is complete, without waiting.
DLLM_DEV bool ready(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(tc::smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// Per key of an own tile: K scale, log2(V scale), 1 / V scale (read as pairs).
struct OwnScales {
  alignas(16) float k[KT], lv[KT], iv[KT];
};

struct Bars {
  uint64_t q_full[2], q_empty[2];          // Q of a unit, staged while the unit before is worked on
  uint64_t k_full[NK], k_empty[NK];
  uint64_t k_grant[NK];                    // a free K stage handed to the converters, for own rows
  uint64_t v_full[NV], v_empty[NV];
  uint64_t w_full[NB], w_empty[NB];        // f16 V of a tile; empty = the tile's P V is complete
  uint64_t s_full[2], p_ready[2];          // per softmax group
  uint64_t r_full[4], r_empty[4];          // scales of a prefix tile
  uint64_t o_free;                         // O of the finished unit has been read
  uint64_t done;
  uint32_t tmem_base;
  int abort_flag;
  int walk[7];                             // b, h, rt, first tile, number of tiles of this CTA, prefix length of b; all tiles
  float qscale[2][KT];                     // per row: 2^k * scale * log2(e)
  float4 run[4][8];                        // per prefix tile and 16 keys: k scale, log2(v scale), 1 / v scale
  float4 run_one;                          // a run whose scores are exponents already: 1, 0, 1
  OwnScales own[NB];                       // of an own tile
  float2 ml[2][2][KT];                     // [unit parity][group][row]: reference and sum
};
constexpr int SMEM = 1024 + 4 * KSTAGE /*Q*/ + NK * KSTAGE + NV * KSTAGE + NB * VTILE + (int)sizeof(Bars);
static_assert(SMEM <= 232448, "shared memory budget");
static_assert(SMEM > 233472 / 2, "tensor-memory kernels must not share an SM");

struct Params {
  Kv8AttnArgs a;
  int G, n_rows, n_rt;        // rows Lq * G of a (b, kv head), row tiles
  FastDiv by_G, by_blk;
  int s_shift;                // log2 of scale_len
  int64_t own_sum;            // own key tiles of all row tiles of a (b, kv head)
  int extra;                  // key tiles that a unit's end counts for in the shares (see Walk)
  int n_cta;
  int merge_shift;            // log2 of the rows that a block of the joining kernel takes, 3 to 7
  float* part;                // [n_cta][2][kPart]
  int2* span;                 // [units]: first and last CTA that work on the unit (one alone has written its rows)
  int reuse;                  // several row tiles read the same keys: keep them in L2
};

// Own keys that query q sees: up to the end of its block. (blk_len is at most Lq here, see the launch.)
DLLM_DEV int visible_own(const Params& p, int q) { return min(p.a.Lq, (p.by_blk(q) + 1) * p.a.blk_len); }
// Own keys that rows of tile rt see (their last query's block).
DLLM_DEV int own_keys(const Params& p, int rt) {
  if (!p.a.k_own) return 0;
  return visible_own(p, p.by_G(min((rt + 1) * KT, p.n_rows) - 1));
}
DLLM_DEV int cdiv128(int x) { return (int)(((unsigned)x + 127u) >> 7); }
// Key tiles of all units of batch row b, at least one per unit, so that rows without keys are written too, and each unit's
// extra ones. The host checks that all of them stay below 2^31.
DLLM_DEV uint32_t row_tiles(const Params& p, int b) {
  const int tp = cdiv128(kv8::prefix_len(p.a.lens, b, p.a.P));
  return (uint32_t)p.a.Hkv *
         ((uint32_t)p.n_rt * (uint32_t)((p.a.k_own ? tp : max(tp, 1)) + p.extra) + (uint32_t)p.own_sum);
}

// CTA c's share of T tiles: the first T mod n CTAs take one more than the others.
struct Share {
  uint32_t q, r;
  DLLM_DEV Share(uint32_t T, uint32_t n) : q(T / n), r(T - T / n * n) {}
  DLLM_DEV uint32_t first(uint32_t c) const { return c * q + min(c, r); }
  DLLM_DEV uint32_t cta_of(uint32_t x) const {
    const uint32_t big = r * (q + 1);
    return x < big ? x / (q + 1) : r + (x - big) / max(q, 1u);
  }
};

// Position in the sequence of key tiles, advanced unit by unit; every role walks it by itself. Behind its key tiles a unit
// has p.extra that stand for the cost of its end and are no work themselves: a share that begins in them begins with the
// next unit, so that CTAs which finish a unit get fewer tiles.
struct Walk {
  int b, h, rt, ta, n;      // unit, first tile in it, tiles left to this CTA (extra ones included)
  int len, tp, own, tiles;  // of the unit: prefix length, prefix tiles, own keys, key tiles
  DLLM_DEV void unit(const Params& p) {
    own = own_keys(p, rt);
    tiles = max(1, tp + cdiv128(own));
  }
  DLLM_DEV void start(const Params& p, const int* w) {
    b = w[0]; h = w[1]; rt = w[2]; ta = w[3]; n = w[4]; len = w[5];
    tp = cdiv128(len);
    if (n > 0) {
      unit(p);
      if (ta >= tiles) next(p);
    }
  }
  DLLM_DEV int end() const { return min(tiles, ta + n); }    // the CTA's key tiles of this unit: [ta, end()), never empty
  DLLM_DEV void next(const Params& p) {
    n -= min(tiles + p.extra - ta, n);
    ta = 0;
    if (++rt == p.n_rt) {
      rt = 0;
      if (++h == p.a.Hkv) {
        h = 0;
        ++b;
        if (n > 0) {
          len = kv8::prefix_len(p.a.lens, b, p.a.P);
          tp = cdiv128(len);
        }
      }
    }
    if (n > 0) unit(p);
  }
};

// This CTA's walk[] (see Bars), by one warp.
DLLM_DEV void make_walk(const Params& p, int* walk) {
  const Kv8AttnArgs& a = p.a;
  const int lane = threadIdx.x & 31;
  const uint32_t mine = lane < a.B ? row_tiles(p, lane) : 0;      // the first 32 batch rows' tiles, read once
  uint32_t T = mine;
  for (int b = lane + 32; b < a.B; b += 32) T += row_tiles(p, b);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) T += __shfl_xor_sync(0xffffffffu, T, o);
  const Share share(T, p.n_cta);
  const uint32_t x = share.first(blockIdx.x), n = share.first(blockIdx.x + 1) - x;
  uint32_t before = 0, rem = 0, in_row = (uint32_t)a.Hkv;      // of a CTA without a share: any but 0 tiles a head
  int b = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const uint32_t own = b0 == 0 ? mine : (b0 + lane < a.B ? row_tiles(p, b0 + lane) : 0);
    uint32_t v = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += y;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, before + v > x);
    if (hit) {
      const int l = __ffs(hit) - 1;
      in_row = __shfl_sync(0xffffffffu, own, l);
      rem = x - before - (__shfl_sync(0xffffffffu, v, l) - in_row);
      b = b0 + l;
      break;
    }
    before += __shfl_sync(0xffffffffu, v, 31);
  }
  if (lane == 0) {
    const uint32_t per_h = in_row / (uint32_t)a.Hkv;
    const int h = (int)(rem / per_h);
    rem -= (uint32_t)h * per_h;
    const int len = kv8::prefix_len(a.lens, b, a.P), tp = cdiv128(len);
    int rt = 0;
    for (; rt + 1 < p.n_rt; ++rt) {
      const uint32_t t = (uint32_t)(max(1, tp + cdiv128(own_keys(p, rt))) + p.extra);
      if (rem < t) break;
      rem -= t;
    }
    walk[0] = b; walk[1] = h; walk[2] = rt; walk[3] = (int)rem; walk[4] = (int)n; walk[5] = len; walk[6] = (int)T;
  }
}

__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
  uint32_t z = 0;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, {%5, %5, %5, %5}, p;\n\t}" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc), "r"(z)
      : "memory");
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Four threads quantise a row of 128 bf16 values into two E4M3 parts: this thread's quarter (32 values, src NULL: zeros).
// The code is kept short: it runs once per unit, and fetching cold instructions is what it costs (a version with a test
// of every value for infinities took 5 us at the start of the kernel).
struct Quarter {
  uint4 raw[4];
  DLLM_DEV void load(const __nv_bfloat16* src) {
#pragma unroll
    for (int i = 0; i < 4; ++i) raw[i] = src ? reinterpret_cast<const uint4*>(src)[i] : make_uint4(0, 0, 0, 0);
  }
  // largest magnitude of the row, as bf16 bits (0x7f80 and above: a value is infinite or NaN), over its four threads
  DLLM_DEV uint32_t amax() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m = __vmaxu2(m, __vmaxu2(raw[i].x & 0x7fff7fffu, raw[i].y & 0x7fff7fffu));
      m = __vmaxu2(m, __vmaxu2(raw[i].z & 0x7fff7fffu, raw[i].w & 0x7fff7fffu));
    }
    m = max(m & 0xffffu, m >> 16);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    return max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  }
  // the two parts of each value times inv (a power of two, or NaN), at the swizzled places of row r of two K-major tiles
  DLLM_DEV void split(float inv, int r, int quarter, uint8_t* hi_tile, uint8_t* lo_tile) const {
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4& q = raw[2 * g + (i >> 1)];
        const uint32_t w[2] = {i & 1 ? q.z : q.x, i & 1 ? q.w : q.y};
        uint32_t h2[2], l2[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float a = __uint_as_float(w[j] << 16) * inv, b = __uint_as_float(w[j] & 0xffff0000u) * inv;
          h2[j] = kv8::f32x2_to_e4m3x2(a, b);
          const uint32_t back = kv8::e4m3x2_to_f16x2(h2[j]);
          const float2 hf = __half22float2(*reinterpret_cast<const __half2*>(&back));
          l2[j] = kv8::f32x2_to_e4m3x2(a - hf.x, b - hf.y);
        }
        hi[i] = h2[0] | (h2[1] << 16);
        lo[i] = l2[0] | (l2[1] << 16);
      }
      const int at = r * 128 + (((2 * quarter + g) ^ (r & 7)) << 4);
      *reinterpret_cast<uint4*>(hi_tile + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      *reinterpret_cast<uint4*>(lo_tile + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
  }
};
constexpr uint32_t kInfBits = 0x7f80u;
DLLM_DEV float qnan() { return __int_as_float(0x7fffffff); }
DLLM_DEV int bits_exp(uint32_t bf16_bits) { return kv8::scale_exp(__uint_as_float(bf16_bits << 16)); }
// Address of a unit's query row (NULL past the last).
DLLM_DEV const __nv_bfloat16* query_row(const Params& p, int b, int h, int rt, int r) {
  const int R = rt * KT + r, qi = p.by_G(R);
  return R < p.n_rows ? static_cast<const __nv_bfloat16*>(p.a.q) +
                            (((int64_t)b * p.a.Lq + qi) * p.a.Hq + h * p.G + R - qi * p.G) * 128
                      : nullptr;
}
// Q of a unit into shared memory by n threads (t = 0 .. n - 1, n a multiple of 128): parts and row scales. q holds the
// first pass's values. A row with an infinity or NaN gets the scale NaN, which reaches all its weights.
DLLM_DEV void stage_q(const Params& p, int b, int h, int rt, int t, int n, uint8_t* sQ, float* qscale, Quarter& q) {
#pragma unroll 1
  for (int r = t >> 2;;) {
    const uint32_t m = q.amax();
    const int k = m >= kInfBits ? 0 : bits_exp(m);
    if ((t & 3) == 0) qscale[r] = m >= kInfBits ? qnan() : kv8::exp2i(k) * (p.a.scale * kLog2e);
    q.split(kv8::exp2i(-k), r, t & 3, sQ, sQ + KSTAGE);
    r += n >> 2;
    if (r >= KT) break;
    const __nv_bfloat16* src = query_row(p, b, h, rt, r);
    q.load(src ? src + 32 * (t & 3) : nullptr);
  }
}
// 32 values of a unit's query row (t >> 2), by the thread's quarter.
DLLM_DEV void load_q(const Params& p, int b, int h, int rt, int t, Quarter& q) {
  const __nv_bfloat16* src = query_row(p, b, h, rt, t >> 2);
  q.load(src ? src + 32 * (t & 3) : nullptr);
}

// Factor and offset of a run's exponents: x = S c + d. c is kept above 0 (a zero K scale), so that a masked score of -inf
// stays -inf; NaN stays NaN.
DLLM_DEV float run_factor(float rowc, const float4& rs) {
  const float c = rowc * rs.x;
  return c < 1e-30f ? 1e-30f : c;
}
// The first lim of 32 columns are visible, if not all are.
DLLM_DEV void mask_scores(bool partly, int lim, float* v) {
  if (partly) {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = i < lim ? v[i] : -INFINITY;
  }
}
// The largest x = S c + lv of 32 columns.
DLLM_DEV float scores_max(const float* v, float rowc, const float4* run, int rstep) {
  float mt = -INFINITY;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const float4 rs = run[u * rstep];
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = fmaxf(m, v[16 * u + i]);
    mt = fmaxf(mt, fmaf(m, run_factor(rowc, rs), rs.y));
  }
  return mt;
}
// 32 own keys' scores as exponents, x = S c + log2(V scale) with a factor c of each key. Before the mask, so c may be 0.
DLLM_DEV void own_exponents(float* v, float rowc, const float* k, const float* lv) {
#pragma unroll
  for (int i = 0; i < 32; i += 4) {
    const float4 ks = *reinterpret_cast<const float4*>(k + i), ls = *reinterpret_cast<const float4*>(lv + i);
    v[i] = fmaf(v[i], rowc * ks.x, ls.x);
    v[i + 1] = fmaf(v[i + 1], rowc * ks.y, ls.y);
    v[i + 2] = fmaf(v[i + 2], rowc * ks.z, ls.z);
    v[i + 3] = fmaf(v[i + 3], rowc * ks.w, ls.w);
  }
}
// The weights of 32 own keys' exponents as f16 pairs, their sum, and their sum with the keys' V scales divided out (l).
DLLM_DEV float own_exp(const float* v, const float* iv, float shift, uint32_t* pk, float& l) {
  const uint64_t d2 = pk2(shift, shift);
  uint64_t s2 = pk2(0.f, 0.f), l2 = s2;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float x0, x1;
    upk2(add2(pk2(v[2 * i], v[2 * i + 1]), d2), x0, x1);
    const float e0 = ex2(x0), e1 = ex2(x1);
    const uint64_t e2 = pk2(e0, e1);
    pk[i] = f16x2(e0, e1);
    s2 = add2(s2, e2);
    l2 = fma2(e2, *reinterpret_cast<const uint64_t*>(iv + 2 * i), l2);
  }
  float s0, s1, l0, l1;
  upk2(s2, s0, s1);
  upk2(l2, l0, l1);
  l = l0 + l1;
  return s0 + s1;
}
// The weights of 32 columns as f16 pairs, their sum, and their sum with the V scales divided out (l).
DLLM_DEV float scores_exp(const float* v, float rowc, const float4* run, int rstep, float shift, uint32_t* pk, float& l) {
  float all = 0.f;
  l = 0.f;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const float4 rs = run[u * rstep];
    const float c = run_factor(rowc, rs), d = rs.y + shift;
    const uint64_t c2 = pk2(c, c), d2 = pk2(d, d);
    uint64_t s2 = pk2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float x0, x1;
      upk2(fma2(pk2(v[16 * u + 2 * i], v[16 * u + 2 * i + 1]), c2, d2), x0, x1);
      const float e0 = ex2(x0), e1 = ex2(x1);
      pk[8 * u + i] = f16x2(e0, e1);
      s2 = add2(s2, pk2(e0, e1));
    }
    float s0, s1;
    upk2(s2, s0, s1);
    all += s0 + s1;
    l = fmaf(s0 + s1, rs.z, l);
  }
  return all;
}
// n groups of 8 TMEM columns of a row times alpha, as fp32 or as pairs of f16.
template <bool F16>
DLLM_DEV void scale_columns(uint32_t at, int n, float alpha) {
#pragma unroll 1
  for (int c = 0; c < n; ++c, at += 8) {
    uint32_t x[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t"
                 "tcgen05.wait::ld.sync.aligned;"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]), "=r"(x[6]), "=r"(x[7])
                 : "r"(at)
                 : "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (F16) {
        // in fp32: alpha is mostly below f16's normal range
        const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&x[i]));
        x[i] = f16x2(y.x * alpha, y.y * alpha);
      } else {
        x[i] = __float_as_uint(__uint_as_float(x[i]) * alpha);
      }
    }
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(at), "r"(x[0]), "r"(x[1]),
                 "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                 : "memory");
  }
  tc::tmem_st_wait();
}
DLLM_DEV void arrive_n(uint64_t* bar, uint32_t n) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(tc::smem_u32(bar)), "r"(n) : "memory");
}

__global__ void __launch_bounds__(NT, 1)
attn_kv8_tc_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                   const __grid_constant__ Params p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = base;                          // [2][hi, lo]
  uint8_t* sK = sQ + 4 * KSTAGE;               // [NK]
  uint8_t* sW = sK + NK * KSTAGE;              // [NB] f16 V
  uint8_t* sV = sW + NB * VTILE;               // [NV]
  Bars& bar = *reinterpret_cast<Bars*>(sV + NV * KSTAGE);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Kv8AttnArgs& a = p.a;

  if (tid == 0) {
    bar.abort_flag = 0;
    bar.run_one = make_float4(1.f, 0.f, 1.f, 0.f);
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&bar.q_full[i], 8);
      tc::mbar_init(&bar.q_empty[i], 1 + 8);
    }
    for (int i = 0; i < NK; ++i) {
      tc::mbar_init(&bar.k_full[i], 1);
      tc::mbar_init(&bar.k_empty[i], 1);
      tc::mbar_init(&bar.k_grant[i], 1);
    }
    for (int i = 0; i < NV; ++i) {
      tc::mbar_init(&bar.v_full[i], 1);
      tc::mbar_init(&bar.v_empty[i], 4);
    }
    for (int i = 0; i < NB; ++i) {
      tc::mbar_init(&bar.w_full[i], 4);
      tc::mbar_init(&bar.w_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&bar.s_full[i], 1);
      tc::mbar_init(&bar.p_ready[i], 4);
    }
    for (int i = 0; i < 4; ++i) {
      tc::mbar_init(&bar.r_full[i], 1);
      tc::mbar_init(&bar.r_empty[i], 4);
    }
    tc::mbar_init(&bar.o_free, 8);
    tc::mbar_init(&bar.done, 1);
    tc::fence_mbar_init();
    tc::prefetch_tmap(&tm_k);
    tc::prefetch_tmap(&tm_v);
  }
  if (warp == 1) tc::tmem_alloc(&bar.tmem_base, 512);
  pdl_trigger();
  if (warp == 0) {
    pdl_wait();        // the lengths may come from the kernel before
    make_walk(p, bar.walk);
  }
  __syncthreads();
  pdl_wait();
  volatile int* abort_flag = &bar.abort_flag;
  const uint32_t tS = bar.tmem_base, tO = bar.tmem_base + 256;      // S_0, S_1; O_0, O_1
  auto arrive = [&](uint64_t* b) {       // once for the warp, after all its lanes
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(b);
  };

  // The four warpgroups launch with 128 registers a thread each and go to 120, 136, 136, 120 (the same sum), which is where
  // nothing spills. Shared memory leaves the L1 next to nothing, so a spill goes to L2: builds with a few hundred bytes of
  // them took up to 3 times as long.
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 120;");
  if (warp == 0) {
    // ------------------------------------------------------------------ TMA: codes of the prefix tiles
    if (tc::elect_one()) {
      Walk w;
      w.start(p, bar.walk);
      const uint64_t pol = p.reuse ? tc::policy_evict_last() : tc::policy_evict_first();
      uint32_t ks = 0, vs = 0;      // slots of the K and V rings so far
      uint32_t kq = 0, vq = 0;      // one past the last slot that this thread filled (for the drain)
      bool ok = true;
      // 128 rows of codes: rows past P read as zeros, rows past the prefix are masked (K) or cleared (V)
      auto load = [&](const CUtensorMap* map, uint8_t* dst, uint64_t* full, int row, int bh) {
        tc::mbar_arrive_expect_tx(full, KSTAGE);
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
            " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(tc::smem_u32(dst)),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(bh), "r"(tc::smem_u32(full)), "l"(pol)
            : "memory");
      };
      for (; w.n > 0 && ok; w.next(p)) {
        const int bh = w.b * a.Hkv + w.h;
        for (int t = w.ta; t < w.end() && ok; ++t) {
          if (t >= w.tp) {
            // own rows: the converters write two K stages (V goes past the code ring). This thread alone waits for
            // free stages, in order, and hands them over: waiting for one's own slots only would miss whole phases
            for (int i = t < w.tp + cdiv128(w.own) ? 2 : 1; i > 0 && ok; --i, ++ks) {
              ok = wait_for(&bar.k_empty[ks % NK], ((ks / NK) & 1) ^ 1, &bar.abort_flag, ST_TIMEOUT_PRODUCER);
              if (ok) tc::mbar_arrive(&bar.k_grant[ks % NK]);
            }
            continue;
          }
          const uint32_t k = ks % NK, v = vs % NV;
          if (!wait_for(&bar.k_empty[k], ((ks / NK) & 1) ^ 1, &bar.abort_flag, ST_TIMEOUT_PRODUCER)) { ok = false; break; }
          load(&tm_k, sK + k * KSTAGE, &bar.k_full[k], t * KT, bh);
          kq = ++ks;
          if (!wait_for(&bar.v_empty[v], ((vs / NV) & 1) ^ 1, &bar.abort_flag, ST_TIMEOUT_PRODUCER)) { ok = false; break; }
          load(&tm_v, sV + v * KSTAGE, &bar.v_full[v], t * KT, bh);
          vq = ++vs;
        }
      }
      if (!ok) {    // let this thread's own copies land before the CTA leaves
        for (uint32_t i = kq > NK ? kq - NK : 0; i < kq; ++i) tc::mbar_wait(&bar.k_full[i % NK], (i / NK) & 1, 1u << 12);
        for (uint32_t i = vq > NV ? vq - NV : 0; i < vq; ++i) tc::mbar_wait(&bar.v_full[i % NV], (i / NV) & 1, 1u << 12);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA
    if (tc::elect_one()) {
      Walk w;
      w.start(p, bar.walk);
      const uint32_t id_s = (1u << 4) | ((KT >> 3) << 17) | ((KT >> 4) << 24);                // E4M3 x E4M3 -> f32
      const uint32_t id_o = (1u << 4) | (1u << 16) | ((128u >> 3) << 17) | ((KT >> 4) << 24);  // f16 x f16, B MN-major
      const uint64_t dQ = tc::sdesc_k128(tc::smem_u32(sQ)), dK = tc::sdesc_k128(tc::smem_u32(sK));
      const uint64_t dW = sdesc_mn128(tc::smem_u32(sW), VCHUNK);      // addresses step by bytes >> 4
      // The S products have a walk of their own, up to two tiles ahead of P V, but no further than the unit after the one
      // P V works on: the Q of the unit after that is staged only when the softmax warps have left this one. S of tile
      // i + 2 goes into the buffer of P of tile i, behind its P V in the issue order.
      Walk ws = w;
      int ts = w.ta, te = w.n > 0 ? w.end() : 0;      // next tile of ws, end of its tiles
      int j = 0, n = te - ts;                         // next tile and number of tiles of w's unit
      uint32_t k = 0, kph = 0, it_s = 0, seg_s = 0, it = 0, g = 0, ph = 0, seg = 0;
      int ahead = 0;
      uint32_t idle = 0;
      bool q_ready = false;
      while (w.n > 0) {
        const bool can_s = ahead < 2 && ws.n > 0 && seg_s <= seg + 1;
        // an S whose operands are not there yet (a unit's own rows, the next unit's queries) does not hold up a P V
        bool go = can_s;
        if (can_s) {
          const bool two = ts >= ws.tp && ws.own > 0;
          if (ahead == 0) {
            if (!q_ready && !wait_for(&bar.q_full[seg_s & 1], (seg_s >> 1) & 1, &bar.abort_flag, ST_TIMEOUT_MMA)) break;
          } else {
            go = (q_ready || ready(&bar.q_full[seg_s & 1], (seg_s >> 1) & 1)) && ready(&bar.k_full[k], kph) &&
                 (!two || ready(&bar.k_full[k + 1 == NK ? 0 : k + 1], k + 1 == NK ? kph ^ 1 : kph));
          }
        }
        if (go) {
          idle = 0;
          q_ready = true;
          const bool own = ts >= ws.tp && ws.own > 0;
          const uint32_t d = tS + (it_s & 1) * 128;
          bool ok = true;
#pragma unroll 1
          for (int part = 0; part < (own ? 2 : 1); ++part) {
            ok = ok && wait_for(&bar.k_full[k], kph, &bar.abort_flag, ST_TIMEOUT_MMA);
            if (!ok) break;
            tc::fence_after_sync();
            const uint64_t dk = dK + k * (KSTAGE >> 4), dq = dQ + (seg_s & 1) * (2 * KSTAGE >> 4);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)      // hi, then lo
              mma_f8(d, dq + (kk >> 2) * (KSTAGE >> 4) + (kk & 3) * 2, dk + (kk & 3) * 2, id_s, part != 0 || kk != 0);
            tc::mma_commit(&bar.k_empty[k]);
            if (++k == NK) {
              k = 0;
              kph ^= 1;
            }
          }
          if (!ok) break;
          tc::mma_commit(&bar.s_full[it_s & 1]);
          ++it_s;
          ++ahead;
          if (++ts == te) {
            tc::mma_commit(&bar.q_empty[seg_s & 1]);
            ws.next(p);
            ts = 0;
            te = ws.n > 0 ? ws.end() : 0;
            ++seg_s;
            q_ready = false;
          }
          continue;
        }
        if (can_s) {      // neither may block the other: look again
          if ((j == 0 && seg > 0 && !ready(&bar.o_free, (seg - 1) & 1)) || !ready(&bar.w_full[g], ph) ||
              !ready(&bar.p_ready[it & 1], (it >> 1) & 1)) {
            if (*abort_flag) break;
            if (++idle > (1u << 24)) {
              *abort_flag = ST_TIMEOUT_MMA;
              break;
            }
            continue;
          }
          idle = 0;
        }
        if (j == 0 && seg > 0 && !wait_for(&bar.o_free, (seg - 1) & 1, &bar.abort_flag, ST_TIMEOUT_MMA)) break;
        if (!wait_for(&bar.w_full[g], ph, &bar.abort_flag, ST_TIMEOUT_MMA) ||
            !wait_for(&bar.p_ready[it & 1], (it >> 1) & 1, &bar.abort_flag, ST_TIMEOUT_MMA))
          break;
        tc::fence_after_sync();
        const uint64_t dw = dW + g * (VTILE >> 4);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          tc::mma_bf16_tmem_a(tO + (it & 1) * 128, tS + (it & 1) * 128 + kk * 8, dw + kk * (2048 >> 4), id_o,
                              (j >= 2 || kk != 0) ? 1u : 0u);
        tc::mma_commit(&bar.w_empty[g]);
        --ahead;
        ++it;
        if (++g == NB) {
          g = 0;
          ph ^= 1;
        }
        if (++j == n) {
          w.next(p);
          j = 0;
          n = w.n > 0 ? w.end() : 0;
          ++seg;
        }
      }
      tc::mma_commit(&bar.done);
      tc::mbar_wait(&bar.done, 0, 1u << 20);
    }
  } else {
    // ------------------------------------------------------------------ scales of the prefix tiles
    // lanes 0-7 K, 8-15 V, one per 16 keys; the next of this warp's tiles is loaded while the last waits for its slot
    Walk w;
    w.start(p, bar.walk);
    const int64_t runs = (a.cap + a.S - 1) >> p.s_shift;
    uint32_t pt = 0;
    float held = 0.f;
    bool have = false;
    uint32_t held_pt = 0;
    auto put = [&]() {
      const uint32_t s = held_pt & 3;
      wait_for(&bar.r_empty[s], ((held_pt >> 2) & 1) ^ 1, &bar.abort_flag, ST_TIMEOUT_PRODUCER);
      const float v = fmaxf(__shfl_down_sync(0xffffffffu, held, 8), 5.421010862427522e-20f);   // 2^-64
      if (lane < 8) bar.run[s][lane] = make_float4(held, log2f(v), 1.0f / v, 0.f);
      arrive(&bar.r_full[s]);
    };
    for (; w.n > 0; w.next(p)) {
      const int64_t bh = (int64_t)w.b * a.Hkv + w.h;
      const int t1 = min(w.end(), w.tp);
      for (int t = w.ta; t < t1; ++t, ++pt) {
        if ((int)(pt & 1) != warp - 2) continue;
        float x = 0.f;      // 16 keys past the prefix: masked, any finite scale will do
        const int key = t * KT + 16 * (lane & 7);
        if (lane < 16 && key < w.len) x = (lane < 8 ? a.k_scale : a.v_scale)[bh * runs + (key >> p.s_shift)];
        if (have) put();
        held = x;
        held_pt = pt;
        have = true;
      }
    }
    if (have) put();
  }
  } else if (warp >= 12) {
    // ------------------------------------------------------------------ converters
    asm volatile("setmaxnreg.dec.sync.aligned.u32 120;");
    Walk w;
    w.start(p, bar.walk);
    const int ct = tid - 384;
    const uint32_t cw = warp - 12;
    uint32_t k = 0, v = 0, vph = 0, g = 0, wph = 1, seg = 0, granted = 0;
    for (; w.n > 0; w.next(p), ++seg) {
      const int64_t bh = (int64_t)w.b * a.Hkv + w.h;
      // the next unit's queries, staged when this unit's first tiles are on their way (the first unit's by the softmax
      // warps, which have nothing to do yet)
      const int t_end = w.end(), t_stage = min(w.ta + 2, t_end) - 1;
      auto stage_next = [&]() {
        Walk nx = w;
        nx.next(p);
        if (nx.n <= 0) return;
        const uint32_t qb = (seg + 1) & 1;
        Quarter q;
        load_q(p, nx.b, nx.h, nx.rt, ct, q);
        if (seg >= 1)
          wait_for(&bar.q_empty[qb], (((seg + 1) >> 1) - 1) & 1, &bar.abort_flag, ST_TIMEOUT_PRODUCER);
        stage_q(p, nx.b, nx.h, nx.rt, ct, 128, sQ + qb * 2 * KSTAGE, bar.qscale[qb], q);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) arrive_n(&bar.q_full[qb], 2);
      };
      for (int t = w.ta; t < t_end; ++t) {
        uint8_t* dst = sW + g * VTILE;
        if (t < w.tp) {
          const int n = min(KT, w.len - t * KT);
          wait_for(&bar.w_empty[g], wph, &bar.abort_flag, ST_TIMEOUT_PRODUCER);
          wait_for(&bar.v_full[v], vph, &bar.abort_flag, ST_TIMEOUT_PRODUCER);
          // Eight neighbouring lanes take the same 16 columns of eight neighbouring keys: with the 128-byte swizzle on both
          // sides their 16-byte pieces fall on different banks, and every address is a lane's own plus a constant.
          const int x = lane & 7, e = lane >> 3, key0 = x + 8 * (int)cw;
          const uint8_t* src = sV + v * KSTAGE + key0 * 128 + ((e ^ x) << 4);
          uint8_t* out = dst + key0 * 128;
          const int o0 = ((2 * e) ^ x) << 4, o1 = ((2 * e + 1) ^ x) << 4;
#pragma unroll 2
          for (int i = 0; i < 4; ++i) {          // keys key0 + 32 i
#pragma unroll
            for (int c = 0; c < 2; ++c) {        // columns 16 (e + 4 c) .. of the key: half of chunk c
              uint4 u = *reinterpret_cast<const uint4*>(src + i * 4096 + (c ? ((e ^ x) & 4 ? -64 : 64) : 0));
              if (n < KT && key0 + 32 * i >= n) u = make_uint4(0, 0, 0, 0);    // past the prefix: 0 times anything but NaN
              uint32_t h[8];
              kv8::e4m3x4_to_f16x4(u.x, h[0], h[1]);
              kv8::e4m3x4_to_f16x4(u.y, h[2], h[3]);
              kv8::e4m3x4_to_f16x4(u.z, h[4], h[5]);
              kv8::e4m3x4_to_f16x4(u.w, h[6], h[7]);
              *reinterpret_cast<uint4*>(out + c * VCHUNK + i * 4096 + o0) = make_uint4(h[0], h[1], h[2], h[3]);
              *reinterpret_cast<uint4*>(out + c * VCHUNK + i * 4096 + o1) = make_uint4(h[4], h[5], h[6], h[7]);
            }
          }
          arrive(&bar.v_empty[v]);
          if (++v == NV) {
            v = 0;
            vph ^= 1;
          }
          k = k == NK - 1 ? 0 : k + 1;
        } else {
          // own rows (none at all in a unit without keys): four threads per key, 32 keys at a time, the next 32 on their
          // way (the first ones ahead of the waits)
          const int j0 = (t - w.tp) * KT, n = min(KT, w.own - j0), parts = n > 0 ? 2 : 1;
          const int64_t at = (bh * a.cap_own + j0) * 128 + 32 * (ct & 3);
          Quarter k8, v8;
          auto load_own = [&](int r) {
            k8.load(r < n ? static_cast<const __nv_bfloat16*>(a.k_own) + at + r * 128 : nullptr);
            v8.load(r < n ? static_cast<const __nv_bfloat16*>(a.v_own) + at + r * 128 : nullptr);
          };
          load_own(ct >> 2);
          wait_for(&bar.w_empty[g], wph, &bar.abort_flag, ST_TIMEOUT_PRODUCER);
          const uint32_t k0 = k, k1 = parts == 2 ? (k + 1) % NK : k;
          for (int i = 0; i < parts; ++i) {
            const uint32_t kk = i ? k1 : k0;
            wait_for(&bar.k_grant[kk], (granted >> kk) & 1, &bar.abort_flag, ST_TIMEOUT_PRODUCER);
            granted ^= 1u << kk;
          }
#pragma unroll 1
          for (int r = ct >> 2; r < KT; r += 32) {
            // rows past the last: V has to be zeros (their weight is 0), K may be anything (their scores are masked)
            const bool zero = r - (ct >> 2) >= n;
            const Quarter kr = k8, vr = v8;
            load_own(r + 32);
            // A row with an infinity or NaN: K makes all its codes NaN; V is zeros (0 times anything else is not 0 for the
            // queries that do not see it) and its exponent NaN, which reaches the queries that do
            int ek = 0, ev = 0;
            bool bad = false;
            if (!zero) {
              const uint32_t x = kr.amax(), y = vr.amax();
              if (x < kInfBits) ek = bits_exp(x);
              bad = y >= kInfBits;
              if (!bad) ev = bits_exp(y);
              kr.split(x < kInfBits ? kv8::exp2i(-ek) : qnan(), r, ct & 3, sK + k0 * KSTAGE, sK + k1 * KSTAGE);
            }
            const float iv = kv8::exp2i(-ev);
            if ((ct & 3) == 0) {
              bar.own[g].k[r] = kv8::exp2i(ek);
              bar.own[g].lv[r] = bad ? qnan() : (float)ev;
              bar.own[g].iv[r] = iv;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int gr = 4 * (ct & 3) + i;      // granule of 8 values: chunk gr >> 3
              uint4 x = make_uint4(0, 0, 0, 0);
              if (!zero && !bad) {
                float f[8];
                bf16x8_to_f32(vr.raw[i], f);
                x = make_uint4(f16x2(f[0] * iv, f[1] * iv), f16x2(f[2] * iv, f[3] * iv), f16x2(f[4] * iv, f[5] * iv),
                               f16x2(f[6] * iv, f[7] * iv));
              }
              *reinterpret_cast<uint4*>(dst + (gr >> 3) * VCHUNK + r * 128 + (((gr & 7) ^ (r & 7)) << 4)) = x;
            }
          }
          fence_async_smem();
          tc::named_bar_sync(kBarConv, 128);
          if (ct < parts) tc::mbar_arrive(&bar.k_full[ct ? k1 : k0]);
          k = (k + parts) % NK;
        }
        fence_async_smem();
        arrive(&bar.w_full[g]);
        if (++g == NB) {
          g = 0;
          wph ^= 1;
        }
        if (t == t_stage) stage_next();
      }
    }
  } else {
    // ------------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 136;");
    Walk w;
    w.start(p, bar.walk);
    const int grp = (warp - 4) >> 2, row = (warp & 3) * 32 + lane, pair = kBarPair + (warp & 3);
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tSg = tS + grp * 128 + lane_off, tOg = tO + grp * 128 + lane_off;
    uint32_t it = 0, g = 0, ph = 0, pt = 0, seg = 0;
    if (w.n > 0) {
      Quarter q;
      load_q(p, w.b, w.h, w.rt, tid - 128, q);
      stage_q(p, w.b, w.h, w.rt, tid - 128, 256, sQ, bar.qscale[0], q);
      fence_async_smem();
      arrive(&bar.q_full[0]);
    }
    for (; w.n > 0; w.next(p), ++seg) {
      const int R = w.rt * KT + row;
      const bool live = R < p.n_rows, warp_live = w.rt * KT + (warp & 3) * 32 < p.n_rows;
      const int qi = p.by_G(live ? R : p.n_rows - 1);
      const int own_lim = a.k_own ? visible_own(p, qi) : 0;
      wait_for(&bar.q_full[seg & 1], (seg >> 1) & 1, &bar.abort_flag, ST_TIMEOUT_EPILOGUE);
      const float rowc = bar.qscale[seg & 1][row];
      arrive(&bar.q_empty[seg & 1]);
      float mg = -INFINITY, l = 0.f;      // reference and sum of this group's tiles
      uint32_t lastg = 0, lastph = 0;     // V buffer and phase of the group's last tile
      bool any = false;                   // the group has had a tile of this unit
      const int t_end = w.end();
      for (int t = w.ta; t < t_end; ++t, ++it) {
        const bool pre = t < w.tp;
        if ((int)(it & 1) == grp) {
          const uint32_t rs = pt & 3;
          const int lim = pre ? w.len - t * KT : own_lim - (t - w.tp) * KT;
          // S of this tile was issued behind P V of tile it - 2, the last one of this group, so its O is complete and no
          // barrier waited for here is more than one phase behind
          wait_for(&bar.s_full[grp], (it >> 1) & 1, &bar.abort_flag, ST_TIMEOUT_EPILOGUE);
          if (pre)
            wait_for(&bar.r_full[rs], (pt >> 2) & 1, &bar.abort_flag, ST_TIMEOUT_EPILOGUE);
          else
            wait_for(&bar.w_full[g], ph, &bar.abort_flag, ST_TIMEOUT_EPILOGUE);
          if (warp_live) {
            const bool partly = !__all_sync(0xffffffffu, lim >= KT);
            tc::fence_after_sync();
            // 32 columns at a time, P into half the columns of the scores that it replaces. Own tiles, the rarer ones, have
            // a copy of the loop of their own: with both forms in one the prefix tiles took 8 to 17 % longer
            float lt = 0.f;
            auto weigh = [&](auto of_prefix) {
              constexpr bool PRE = decltype(of_prefix)::value;
              const float4* run = PRE ? bar.run[rs] : &bar.run_one;
              const int rstep = PRE ? 1 : 0;
              const float c1 = PRE ? rowc : 1.f;      // factor of the row's scores
#pragma unroll 1
              for (int c = 0; c < 4; ++c) {
                float v[32];
                tmem_ld32(tSg + 32 * c, v);
                if (!PRE) own_exponents(v, rowc, bar.own[g].k + 32 * c, bar.own[g].lv + 32 * c);
                mask_scores(partly, lim - 32 * c, v);
                uint32_t pk[16];
                float lc;
#pragma unroll 1
                for (int tries = 0;; ++tries) {
                  const float shift = kOff - (mg == -INFINITY ? 0.f : mg);
                  const float sum = PRE ? scores_exp(v, c1, run + 2 * c * rstep, rstep, shift, pk, lc)
                                        : own_exp(v, bar.own[g].iv + 32 * c, shift, pk, lc);
                  const bool move = sum > kMost || mg == -INFINITY;
                  if (tries || !__any_sync(0xffffffffu, move)) break;
                  // the reference of the rows concerned moves to the largest score here, and what they have so far with it
                  const float m = scores_max(v, c1, run + 2 * c * rstep, rstep);
                  float alpha = 1.f;
                  if (move && m > mg) {
                    alpha = mg == -INFINITY ? 1.f : ex2(mg - m);
                    mg = m;
                  }
                  l *= alpha;
                  lt *= alpha;
                  if (__any_sync(0xffffffffu, alpha != 1.f)) {
                    tc::tmem_st_wait();
                    scale_columns<true>(tSg, 2 * c, alpha);
                    if (any) scale_columns<false>(tOg, 16, alpha);
                  }
                }
                lt += lc;
                asm volatile(
                    "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::
                        "r"(tSg + 16 * c),
                    "r"(pk[0]), "r"(pk[1]), "r"(pk[2]), "r"(pk[3]), "r"(pk[4]), "r"(pk[5]), "r"(pk[6]), "r"(pk[7]), "r"(pk[8]),
                    "r"(pk[9]), "r"(pk[10]), "r"(pk[11]), "r"(pk[12]), "r"(pk[13]), "r"(pk[14]), "r"(pk[15])
                    : "memory");
              }
            };
            if (pre)
              weigh(std::true_type{});
            else
              weigh(std::false_type{});
            l += lt;
            tc::tmem_st_wait();
            tc::fence_before_sync();
          }
          arrive(&bar.p_ready[grp]);
          if (pre && lane == 0) tc::mbar_arrive(&bar.r_empty[rs]);
          any = true;
          lastg = g;
          lastph = ph;
        }
        pt += pre;
        if (++g == NB) {
          g = 0;
          ph ^= 1;
        }
      }
      // this group's last P V, then the other's too
      if (any) wait_for(&bar.w_empty[lastg], lastph, &bar.abort_flag, ST_TIMEOUT_EPILOGUE);
      bar.ml[seg & 1][grp][row] = make_float2(mg, l);
      tc::fence_before_sync();
      tc::named_bar_sync(pair, 64);
      const bool whole = w.ta == 0 && w.end() == w.tiles;
      if (warp_live) {
        const float2 x0 = bar.ml[seg & 1][0][row], x1 = bar.ml[seg & 1][1][row];
        mg = fmaxf(x0.x, x1.x);
        const float wa = x0.x == -INFINITY ? 0.f : ex2(x0.x - mg), wb = x1.x == -INFINITY ? 0.f : ex2(x1.x - mg);
        const float L = fmaf(wa, x0.y, wb * x1.y);
        const float inv = L == 0.f ? 0.f : 1.0f / L;
        const bool put = !*abort_flag && live;
        const int64_t qh = ((int64_t)w.b * a.Lq + qi) * a.Hq + w.h * p.G + (live ? R - qi * p.G : 0);
        float4* part = reinterpret_cast<float4*>(p.part + ((int64_t)blockIdx.x * 2 + (w.ta == 0 ? 1 : 0)) * kPart);
        __syncwarp();
        tc::fence_after_sync();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int col = 64 * grp + 32 * c;
          float o[32], x[32];
          // a group without a tile here has left nothing (or another unit's rows) in its O: weight 0 does not read it
          tmem_ld32(tO + col + lane_off, o);
          tmem_ld32(tO + 128 + col + lane_off, x);
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = (wa != 0.f ? wa * o[i] : 0.f) + (wb != 0.f ? wb * x[i] : 0.f);
          if (put && whole) {
            uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + qh * 128 + col);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t u[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                __nv_bfloat162 r = __floats2bfloat162_rn(o[8 * i + 2 * j] * inv, o[8 * i + 2 * j + 1] * inv);
                u[j] = *reinterpret_cast<uint32_t*>(&r);
              }
              dst[i] = make_uint4(u[0], u[1], u[2], u[3]);
            }
          } else if (put) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              part[(col / 4 + i) * KT + row] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
          }
          __syncwarp();
        }
        tc::fence_before_sync();
        if (put && grp == 0) {
          if (!whole) part[32 * KT + row] = make_float4(mg, L, 0.f, 0.f);
          else if (a.lse_out) a.lse_out[qh] = L == 0.f ? -INFINITY : (mg - kOff + log2f(L)) * kLn2;
        }
      }
      if (tid == 128 && w.ta == 0) {
        const Share share((uint32_t)bar.walk[6], p.n_cta);
        const uint32_t first = share.first(blockIdx.x + 1) - (uint32_t)w.n;
        const int last = (int)share.cta_of(first + (uint32_t)w.tiles - 1);      // its last key tile's
        p.span[((int64_t)w.b * a.Hkv + w.h) * p.n_rt + w.rt] = make_int2((int)blockIdx.x, last);
      }
      arrive(&bar.o_free);
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(bar.tmem_base, 512);
    if (lane == 0 && *abort_flag && a.status) atomicExch(a.status, *abort_flag);
  }
}

// Joins the partial results of the units that span several CTAs, the CTAs in order: a thread takes 8 output columns of a
// row. A block is as many rows as a unit has, rounded up to a power of two, and the column groups that fill it up to 128
// threads: a full row tile takes 16 blocks, a single token's few heads one (see the launch). Bound by the latency of its
// loads.
constexpr int kMergeCols = 8;
static_assert(KT * kMergeCols == 128 << 3, "16 column groups of 8: blocks per unit are rows / 8");
__global__ void __launch_bounds__(KT) attn_kv8_merge_kernel(const __grid_constant__ Params p) {
  pdl_enter();
  const Kv8AttnArgs& a = p.a;
  const int sh = p.merge_shift, row = threadIdx.x & ((1 << sh) - 1);
  const int part_col = (int)((blockIdx.x & ((1u << (sh - 3)) - 1u)) << (7 - sh)) + (int)(threadIdx.x >> sh);
  const int64_t unit = blockIdx.x >> (sh - 3);
  const int2 sp = p.span[unit];
  const int rt = (int)(unit % p.n_rt), R = rt * KT + row, n = sp.y - sp.x + 1;
  if (n == 1 || R >= p.n_rows) return;
  auto slot = [&](int k) {
    return reinterpret_cast<const float4*>(p.part) + ((int64_t)(sp.x + k) * 2 + (k == 0 ? 1 : 0)) * (kPart / 4);
  };
  // one pass, kBatch partial results in flight, against the largest reference so far
  constexpr int kBatch = 8;
  float M = -INFINITY, L = 0.f, o[kMergeCols];
#pragma unroll
  for (int i = 0; i < kMergeCols; ++i) o[i] = 0.f;
#pragma unroll 1
  for (int k0 = 0; k0 < n; k0 += kBatch) {
    float2 ml[kBatch];
    float4 x[kBatch][kMergeCols / 4];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const bool in = k0 + k < n;
      const float4* s = slot(in ? k0 + k : k0);
      ml[k] = *reinterpret_cast<const float2*>(s + 32 * KT + row);
      if (!in) ml[k] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int i = 0; i < kMergeCols / 4; ++i) x[k][i] = s[(part_col * (kMergeCols / 4) + i) * KT + row];
    }
    float now = M;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) now = fmaxf(now, ml[k].x);
    const float old = M == -INFINITY ? 0.f : ex2(M - now);
    M = now;
    L *= old;
#pragma unroll
    for (int i = 0; i < kMergeCols; ++i) o[i] *= old;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const float wt = ml[k].x == -INFINITY ? 0.f : ex2(ml[k].x - M);
      L = fmaf(wt, ml[k].y, L);
#pragma unroll
      for (int i = 0; i < kMergeCols / 4; ++i) {
        o[4 * i] = fmaf(wt, x[k][i].x, o[4 * i]);
        o[4 * i + 1] = fmaf(wt, x[k][i].y, o[4 * i + 1]);
        o[4 * i + 2] = fmaf(wt, x[k][i].z, o[4 * i + 2]);
        o[4 * i + 3] = fmaf(wt, x[k][i].w, o[4 * i + 3]);
      }
    }
  }
  const float inv = L == 0.f ? 0.f : 1.0f / L;
  const int64_t bh = unit / p.n_rt;
  const int b = (int)(bh / a.Hkv), h = (int)(bh - (int64_t)b * a.Hkv), qi = p.by_G(R);
  const int64_t qh = ((int64_t)b * a.Lq + qi) * a.Hq + h * p.G + R - qi * p.G;
  uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + qh * 128 + part_col * kMergeCols);
#pragma unroll
  for (int i = 0; i < kMergeCols / 8; ++i) {
    uint32_t u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      __nv_bfloat162 r = __floats2bfloat162_rn(o[8 * i + 2 * j] * inv, o[8 * i + 2 * j + 1] * inv);
      u[j] = *reinterpret_cast<uint32_t*>(&r);
    }
    dst[i] = make_uint4(u[0], u[1], u[2], u[3]);
  }
  if (part_col == 0 && a.lse_out) a.lse_out[qh] = L == 0.f ? -INFINITY : (M - kOff + log2f(L)) * kLn2;
}

// ------------------------------------------------------------------------------------------------ attention weight
// mass[j] (+)= sum over the query rows R of 2^(S[R, j] c - lse2[R]). The product is transposed, S^T = K Q^T: keys are the
// rows of the accumulator, so a thread owns a key and adds its row up in registers, with no sum across threads and no
// atomics. A query row's factor 2^k scale log2(e) (a power-of-two scale of its own, as in the attention that wrote its
// lse) and its lse2 come from shared memory, the key's scale is the thread's own. A row that gives no weight (lse -inf) is
// staged as zeros, whatever it holds. Key tiles are dealt to the CTAs like the attention's; a CTA goes over
// its tiles of a (b, kv head) once per row tile of the queries (more than one: K comes from L2 after the first time).
// Bound by the exponentials: 128 x 128 per key tile and row tile, 1024 clocks, against 512 of MMAs and 710 of HBM; 16 x 32
// queries over up to 2688 keys 16.6 us, 4 x 32 over 32768 34 us (31.9 with one query scale for a row tile, a packed product
// less per two weights, which cost small rows beside large ones their precision).
// Roles: warp 0 TMA, warp 1 MMA, warps 4-15 three groups that take the key tiles in turn, each with an S buffer (a thread's
// loads, exponentials and sums follow one another, so two groups leave the special-function units half idle: 4 rows of
// 32768 keys, 128 rows a kv head, 36.6 us with two, 34.3 with three, 35.5 with four, which spill; 16 x 2688 17.2, 16.6 and
// 19.0), warps 16-19 stage the queries.
constexpr int MK = 5, MS = 3;              // stages of the K ring, S buffers = groups
constexpr int MASS_NT = 128 * (2 + MS);
struct MassBars {
  uint64_t q_full[2], q_empty[2];
  uint64_t k_full[MK], k_empty[MK];
  uint64_t s_full[MS], s_empty[MS];
  uint64_t done;
  uint32_t tmem_base;
  int abort_flag;
  int walk[7];
  alignas(16) float factor[2][KT];   // per staged query row: 2^k scale log2(e)
  alignas(16) float nlse[2][KT];     // -lse log2(e); -inf for rows that give no weight
};
constexpr int MASS_SMEM = 1024 + 2 * 2 * KSTAGE /*Q*/ + MK * KSTAGE + (int)sizeof(MassBars);
static_assert(MASS_SMEM <= 232448, "shared memory budget");
static_assert(MASS_SMEM > 233472 / 2, "tensor-memory kernels must not share an SM");

__global__ void __launch_bounds__(MASS_NT, 1)
attn_mass_kv8_tc_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ Params p, int q_rt) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = base;                          // [2][hi, lo]
  uint8_t* sK = sQ + 4 * KSTAGE;               // [MK]
  MassBars& bar = *reinterpret_cast<MassBars*>(sK + MK * KSTAGE);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Kv8AttnArgs& a = p.a;

  if (tid == 0) {
    bar.abort_flag = 0;
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&bar.q_full[i], 4);
      tc::mbar_init(&bar.q_empty[i], 1 + 4 * MS);
    }
    for (int i = 0; i < MK; ++i) {
      tc::mbar_init(&bar.k_full[i], 1);
      tc::mbar_init(&bar.k_empty[i], 1);
    }
    for (int i = 0; i < MS; ++i) {
      tc::mbar_init(&bar.s_full[i], 1);
      tc::mbar_init(&bar.s_empty[i], 4);
    }
    tc::mbar_init(&bar.done, 1);
    tc::fence_mbar_init();
    tc::prefetch_tmap(&tm_k);
  }
  if (warp == 1) tc::tmem_alloc(&bar.tmem_base, 512);
  pdl_trigger();
  if (warp == 0) {
    pdl_wait();
    make_walk(p, bar.walk);
  }
  __syncthreads();
  pdl_wait();
  volatile int* abort_flag = &bar.abort_flag;
  const uint32_t tS = bar.tmem_base;
  Walk w;
  w.start(p, bar.walk);
  auto arrive = [&](uint64_t* b) {       // once for the warp, after all its lanes
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(b);
  };

  if (warp == 0) {
    if (tc::elect_one()) {
      const uint64_t pol = q_rt > 1 ? tc::policy_evict_last() : tc::policy_evict_first();
      uint32_t k = 0, ph = 1, filled = 0;
      bool ok = true;
      for (; w.n > 0 && ok; w.next(p)) {
        const int bh = w.b * a.Hkv + w.h;
        for (int rt = 0; rt < q_rt && ok; ++rt)
          for (int t = w.ta; t < w.end(); ++t) {
            if (!wait_for(&bar.k_empty[k], ph, &bar.abort_flag, ST_TIMEOUT_PRODUCER)) { ok = false; break; }
            tc::mbar_arrive_expect_tx(&bar.k_full[k], KSTAGE);
            asm volatile(
                "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
                " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(tc::smem_u32(sK + k * KSTAGE)),
                "l"(reinterpret_cast<uint64_t>(&tm_k)), "r"(0), "r"(t * KT), "r"(bh),
                "r"(tc::smem_u32(&bar.k_full[k])), "l"(pol)
                : "memory");
            ++filled;
            if (++k == MK) {
              k = 0;
              ph ^= 1;
            }
          }
      }
      if (!ok)      // let the copies land before the CTA leaves
        for (uint32_t i = filled > MK ? filled - MK : 0; i < filled; ++i)
          tc::mbar_wait(&bar.k_full[i % MK], (i / MK) & 1, 1u << 12);
    }
  } else if (warp == 1) {
    if (tc::elect_one()) {
      const uint32_t id_s = (1u << 4) | ((KT >> 3) << 17) | ((KT >> 4) << 24);
      const uint64_t dQ = tc::sdesc_k128(tc::smem_u32(sQ)), dK = tc::sdesc_k128(tc::smem_u32(sK));
      uint32_t k = 0, kph = 0, sb = 0, sph = 1, seg = 0;
      bool ok = true;
      for (; w.n > 0 && ok; w.next(p))
        for (int rt = 0; rt < q_rt && ok; ++rt, ++seg) {
          const uint32_t qb = seg & 1;
          const uint64_t dq = dQ + qb * (2 * KSTAGE >> 4);
          if (!wait_for(&bar.q_full[qb], (seg >> 1) & 1, &bar.abort_flag, ST_TIMEOUT_MMA)) { ok = false; break; }
          for (int n = w.end() - w.ta; n > 0; --n) {
            if (!wait_for(&bar.s_empty[sb], sph, &bar.abort_flag, ST_TIMEOUT_MMA) ||
                !wait_for(&bar.k_full[k], kph, &bar.abort_flag, ST_TIMEOUT_MMA)) {
              ok = false;
              break;
            }
            tc::fence_after_sync();
            const uint64_t dk = dK + k * (KSTAGE >> 4);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)      // hi, then lo
              mma_f8(tS + sb * 128, dk + (kk & 3) * 2, dq + (kk >> 2) * (KSTAGE >> 4) + (kk & 3) * 2, id_s, kk != 0);
            tc::mma_commit(&bar.s_full[sb]);
            tc::mma_commit(&bar.k_empty[k]);
            if (++k == MK) {
              k = 0;
              kph ^= 1;
            }
            if (++sb == MS) {
              sb = 0;
              sph ^= 1;
            }
          }
          tc::mma_commit(&bar.q_empty[qb]);
        }
      tc::mma_commit(&bar.done);
      tc::mbar_wait(&bar.done, 0, 1u << 20);
    }
  } else if (warp >= 4 + 4 * MS) {
    // ------------------------------------------------------------------ queries: four threads per row, 32 rows at a time
    const int ct = tid - 128 * (1 + MS);
    uint32_t seg = 0;
    for (; w.n > 0; w.next(p))
      for (int rt = 0; rt < q_rt; ++rt, ++seg) {
        const uint32_t qb = seg & 1;
        Quarter q;
        float nl;
        // the next 32 rows are on their way while these are converted (the first ones ahead of the wait)
        auto load = [&](int r) {
          const __nv_bfloat16* src = r < KT ? query_row(p, w.b, w.h, rt, r) : nullptr;
          nl = -INFINITY;
          if (src) {
            const int R = rt * KT + r, qi = p.by_G(R);
            const float lse = a.lse_in[((int64_t)w.b * a.Lq + qi) * a.Hq + w.h * p.G + R - qi * p.G];
            if (lse == -INFINITY)
              src = nullptr;
            else
              nl = -lse * kLog2e;
          }
          q.load(src ? src + 32 * (ct & 3) : nullptr);
        };
        load(ct >> 2);
        if (seg >= 2) wait_for(&bar.q_empty[qb], ((seg >> 1) & 1) ^ 1, &bar.abort_flag, ST_TIMEOUT_PRODUCER);
#pragma unroll 1
        for (int r = ct >> 2; r < KT; r += 32) {
          const Quarter x = q;
          const float n = nl;
          load(r + 32);
          const uint32_t m = x.amax();
          const int k = m >= kInfBits ? 0 : bits_exp(m);
          if ((ct & 3) == 0) {
            // an infinity or NaN reaches the row's weight on every key
            bar.factor[qb][r] = m >= kInfBits ? qnan() : kv8::exp2i(k) * (a.scale * kLog2e);
            bar.nlse[qb][r] = n;
          }
          x.split(kv8::exp2i(-k), r, ct & 3, sQ + qb * 2 * KSTAGE, sQ + (qb * 2 + 1) * KSTAGE);
        }
        fence_async_smem();
        arrive(&bar.q_full[qb]);
      }
  } else if (warp >= 4) {
    // ------------------------------------------------------------------ weights
    const int grp = (warp - 4) >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const int64_t runs = (a.cap + a.S - 1) >> p.s_shift;
    uint32_t it = 0, sb = 0, ph = 0, seg = 0;
    for (; w.n > 0; w.next(p)) {
      const int64_t bh = (int64_t)w.b * a.Hkv + w.h;
      const int t_end = w.end();
      for (int rt = 0; rt < q_rt; ++rt, ++seg) {
        const uint32_t qb = seg & 1;
        const int cols = min(KT, p.n_rows - rt * KT);
        wait_for(&bar.q_full[qb], (seg >> 1) & 1, &bar.abort_flag, ST_TIMEOUT_EPILOGUE);
        // another group may have added the last row tile to this group's tiles
        if (rt > 0) tc::named_bar_sync(kBarPair, 128 * MS);
        for (int t = w.ta; t < t_end; ++t, ++it) {
          if ((int)(it % MS) == grp) {
            const int key = t * KT + row;
            const bool live = key < w.len;
            float ks = 0.f, old = 0.f;
            const int64_t at = bh * a.cap + key;
            if (live) {
              ks = a.k_scale[bh * runs + (key >> p.s_shift)];
              if (rt > 0) old = a.mass_out[at];
              else if (a.mass_in) old = a.decay * a.mass_in[at];
            }
            wait_for(&bar.s_full[sb], ph, &bar.abort_flag, ST_TIMEOUT_EPILOGUE);
            __syncwarp();
            tc::fence_after_sync();
            const uint64_t ks2 = pk2(ks, ks);
            uint64_t s2 = pk2(0.f, 0.f);
#pragma unroll 1
            for (int j = 0; j < cols; j += 32) {
              float v[32];
              tmem_ld32(tS + sb * 128 + j + lane_off, v);
              const float4* nl = reinterpret_cast<const float4*>(bar.nlse[qb] + j);
              const float4* fs = reinterpret_cast<const float4*>(bar.factor[qb] + j);
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float4 n4 = nl[i], f4 = fs[i];
                float x0, x1, x2, x3;
                upk2(fma2(pk2(v[4 * i], v[4 * i + 1]), mul2(ks2, pk2(f4.x, f4.y)), pk2(n4.x, n4.y)), x0, x1);
                upk2(fma2(pk2(v[4 * i + 2], v[4 * i + 3]), mul2(ks2, pk2(f4.z, f4.w)), pk2(n4.z, n4.w)), x2, x3);
                s2 = add2(s2, pk2(ex2(x0), ex2(x1)));
                s2 = add2(s2, pk2(ex2(x2), ex2(x3)));
              }
            }
            tc::fence_before_sync();
            arrive(&bar.s_empty[sb]);
            float s0, s1;
            upk2(s2, s0, s1);
            if (live && !*abort_flag) a.mass_out[at] = old + (s0 + s1);
          }
          if (++sb == MS) {
            sb = 0;
            ph ^= 1;
          }
        }
        arrive(&bar.q_empty[qb]);
      }
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(bar.tmem_base, 512);
    if (lane == 0 && *abort_flag && a.status) atomicExch(a.status, *abort_flag);
  }
}

// Map of bh heads of `rows` rows of codes, cap rows apart. Its extent is the rows that the call may read, not cap: a tile's
// rows past them read as zeros and are never fetched (a cache may be a part of a longer one that ends with its last head's
// rows).
int encode_codes(CUtensorMap* m, const void* codes, int64_t rows, int64_t cap, int64_t bh) {
  EncodeTiledFn enc = encoder();
  if (!enc) {
    dllm_host::set_error("cuTensorMapEncodeTiled unavailable");
    return DLLM_ERR_CUDA;
  }
  const cuuint64_t dims[3] = {128, (cuuint64_t)rows, (cuuint64_t)bh};
  const cuuint64_t str[2] = {128, (cuuint64_t)cap * 128};
  const cuuint32_t box[3] = {128, KT, 1}, es[3] = {1, 1, 1};
  const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(codes), dims, str, box, es,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    dllm_host::set_error("attention over 8-bit codes: cuTensorMapEncodeTiled failed (%d)", (int)r);
    return DLLM_ERR_CUDA;
  }
  return DLLM_OK;
}

void set_shape(Params& p) {
  p.G = p.a.Hq / p.a.Hkv;
  p.n_rows = p.a.Lq * p.G;
  p.a.blk_len = std::min(p.a.blk_len, p.a.Lq);     // a longer block is the whole of the queries all the same
  p.by_G = fast_div(p.G);
  p.by_blk = fast_div(p.a.blk_len);
  p.s_shift = p.a.S == 16 ? 4 : p.a.S == 32 ? 5 : p.a.S == 64 ? 6 : 7;
}

// Own key tiles of all row tiles (own_keys on the host).
int64_t own_tiles_sum(const Kv8AttnArgs& a, int n_rt, int G) {
  if (!a.k_own) return 0;
  int64_t t = 0;
  for (int rt = 0; rt < n_rt; ++rt) {
    const int last_q = (std::min((int64_t)(rt + 1) * KT, (int64_t)a.Lq * G) - 1) / G;
    t += (std::min<int64_t>(a.Lq, ((int64_t)(last_q / a.blk_len) + 1) * a.blk_len) + KT - 1) / KT;
  }
  return t;
}

}  // namespace

// Partial results of every CTA, then the units' spans.
size_t attn_kv8_tc_workspace_bytes(int B, int Lq, int Hq, int Hkv) {
  const size_t units = (size_t)B * Hkv * (((size_t)Lq * (Hq / Hkv) + KT - 1) / KT);
  return (size_t)num_sms() * 2 * kPart * sizeof(float) + units * sizeof(int2);
}

int launch_attn_kv8_tc(const Kv8AttnArgs& a, cudaStream_t s) {
  Params p;
  p.a = a;
  set_shape(p);
  p.n_rt = (p.n_rows + KT - 1) / KT;
  p.own_sum = own_tiles_sum(a, p.n_rt, p.G);
  p.part = static_cast<float*>(a.ws);
  p.span = reinterpret_cast<int2*>(p.part + (size_t)num_sms() * 2 * kPart);
  p.reuse = p.n_rt > 1;
  p.merge_shift = 3;
  while (p.merge_shift < 7 && (1 << p.merge_shift) < p.n_rows) ++p.merge_shift;
  // most tiles there can be (lengths may be shorter): no more CTAs than those. With a CTA for every tile the ends are not
  // counted: the extra tiles would only bring CTAs without work (block of 1 x 1024: 15.8 us either way)
  const int64_t tp = (a.P + KT - 1) / KT;
  int64_t most = (int64_t)a.B * a.Hkv * (p.n_rt * (a.k_own ? tp : std::max<int64_t>(tp, 1)) + p.own_sum);
  p.extra = most > num_sms() ? kUnitEnd : 0;
  most += (int64_t)a.B * a.Hkv * p.n_rt * p.extra;
  DLLM_REQUIRE(most < (1ll << 31), DLLM_ERR_UNSUPPORTED, "block_attn_kv8: too many rows and keys for one call");
  p.n_cta = (int)std::min<int64_t>(num_sms(), most);
  CUtensorMap mk, mv;
  // without prefix rows no tile is loaded; the maps then describe the queries' memory, which exists
  int st = a.P > 0 ? encode_codes(&mk, a.k_codes, a.P, a.cap, (int64_t)a.B * a.Hkv) : encode_codes(&mk, a.q, 1, 1, 1);
  if (st) return st;
  st = a.P > 0 ? encode_codes(&mv, a.v_codes, a.P, a.cap, (int64_t)a.B * a.Hkv) : encode_codes(&mv, a.q, 1, 1, 1);
  if (st) return st;
  st = set_max_smem<attn_kv8_tc_kernel>(SMEM);
  if (st) return st;
  launch_pdl(attn_kv8_tc_kernel, p.n_cta, NT, SMEM, s, mk, mv, p);
  DLLM_CHECK_LAUNCH("attn_kv8_tc_kernel");
  if (p.n_cta > 1) {
    launch_pdl(attn_kv8_merge_kernel, (unsigned)(((int64_t)a.B * a.Hkv * p.n_rt) << (p.merge_shift - 3)), KT, 0, s, p);
    DLLM_CHECK_LAUNCH("attn_kv8_merge_kernel");
  }
  return DLLM_OK;
}

int launch_attn_mass_kv8_tc(const Kv8AttnArgs& a, cudaStream_t s) {
  Params p = {};
  p.a = a;
  p.a.k_own = nullptr;
  set_shape(p);
  p.n_rt = 1;                  // units of the walk are whole (b, kv head)s
  const int64_t most = (int64_t)a.B * a.Hkv * ((a.P + KT - 1) / KT);
  p.n_cta = (int)std::min<int64_t>(num_sms(), most);
  CUtensorMap mk;
  int st = encode_codes(&mk, a.k_codes, a.P, a.cap, (int64_t)a.B * a.Hkv);
  if (st) return st;
  st = set_max_smem<attn_mass_kv8_tc_kernel>(MASS_SMEM);
  if (st) return st;
  launch_pdl(attn_mass_kv8_tc_kernel, p.n_cta, MASS_NT, MASS_SMEM, s, mk, p, (p.n_rows + KT - 1) / KT);
  DLLM_CHECK_LAUNCH("attn_mass_kv8_tc_kernel");
  return DLLM_OK;
}

}  // namespace dllm
