// Attention over the rotated int8 cache for many rows: trees of drafted tokens and
// chunks, on the 5th-generation tensor cores. The mathematics, the line of work
// and the join are those of cache_attention.cu; a tile is 128 query rows by 128 keys.
//
// Here a key is read for 128 rows, so the softmax bounds it, as in the dense INT8
// attention: one exponential per row and key and five or six instructions beside it.
// One CTA per SM, two pipelines in it that take turns over the key tiles, so that
// one's softmax runs while the other's products do; each has its own sums (O in
// TMEM, maximum and row sum in registers), joined at the end of a run:
//   warps 0-3, 4-7 : softmax of pipeline 0 and 1, a query row per thread: S from
//                    TMEM, logits, weights p s_v in fp16 into swizzled shared memory;
//   warps 8-11     : the tile's values, widened exactly from int8 to fp16 into the
//                    (MN-major) operand of P V, and its scales;
//   warp 12        : key codes by TMA (boxes of 16 keys: pages are no smaller);
//   warp 13        : issues S = Q K^T (kind::i8, 128 x 128 x 128) and O += P V
//                    (kind::f16, fp16 operands);
//   warps 14, 15   : idle (they complete a register group).
// The softmax holds 128 logits a thread: its warps take 192 registers and leave
// 64 to the others.
// The reference of a row's exponentials is chosen so that the weights, not the
// exponentials, fit fp16: the largest weight so far lies between 1 and 2^15, whatever
// the range of the value scales. It moves only where a tile's largest logit and
// largest value scale together could pass that, and then by the weights themselves.
// Every wait is bounded.

#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <cstdint>

#include "cache_attention.cuh"
#include "convrot.h"
#include "fwht128.cuh"
#include "fwht_dev.cuh"
#include "ptx_sm100.cuh"

namespace convrot {

namespace {

constexpr int CW_KT = 128;           // keys of a tile
constexpr int CW_THREADS = 512;
constexpr int CW_HALF = 128 * 128;   // 128 rows of 128 bytes
constexpr uint64_t CW_TIMEOUT_NS = 2000000000ull;
// a run costs about as much as three tiles beside its tiles
using CwGrain = CaGrain<CA_WIDE_ROWS, CW_KT, 3, 2>;
constexpr uint32_t CW_IDESC_S = idesc_i8(128, CW_KT);
// fp16 operands, float32 sums, 128 x 128, B MN-major
constexpr uint32_t CW_IDESC_O = (1u << 4) | (1u << 16) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
constexpr float CW_FIT = 15.0f;      // weights stay below 2^15
constexpr float CW_SPAN = 100.0f;    // exponentials below 2^100

struct CwSmem {
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kOffQ + CW_HALF;            // two pipelines
  static constexpr int kOffP = kOffK + 2 * CW_HALF;
  static constexpr int kOffV = kOffP + 2 * 2 * CW_HALF;
  static constexpr int kOffScale = kOffV + 2 * 2 * CW_HALF;  // [pipeline][buffer] 128 key, 128 value scales
  static constexpr int kOffTile = kOffScale + 2 * 2 * 256 * 4;  // [pipeline][buffer] 4 words of keys there, 4 largest value scales
  static constexpr int kOffRow = kOffTile + 2 * 2 * 8 * 4;   // query factors
  static constexpr int kOffStat = kOffRow + 128 * 4;         // [pipeline][row] maximum, sum
  static constexpr int kOffScan = kOffStat + 2 * 128 * 8;
  // per pipeline: k_full, k_empty, s_full, s_empty, p_full, o_done, v_full, sc_full; then drain
  static constexpr int kOffBar = kOffScan + 18 * 8;
  static constexpr int kOffMisc = kOffBar + 17 * 8;
  static constexpr int kBytes = kOffMisc + 16;
  static constexpr int kAlloc = kBytes + 1024;
};

enum CwBar { kKFull, kKEmpty, kSFull, kSEmpty, kPFull, kODone, kVFull, kScFull, kBars };

__device__ __forceinline__ void cw_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

template <int N>
__device__ __forceinline__ void regs_more() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_fewer() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// A word of the keys below `n` among keys 32 w .. 32 w + 31 of a tile.
__device__ __forceinline__ uint32_t below(int n, int w) {
  const int m = n - 32 * w;
  return m <= 0 ? 0u : m >= 32 ? 0xFFFFFFFFu : (1u << m) - 1u;
}

// Word w of 64 bits placed at bit `at` (which may be negative) of a tile's keys.
__device__ __forceinline__ uint32_t placed(unsigned long long bits, int at, int w) {
  const int shift = 32 * w - at;  // the word's first key is this bit
  if (shift >= 64 || shift <= -32) return 0u;
  return static_cast<uint32_t>(shift >= 0 ? bits >> shift : bits << -shift);
}

// Weights of 64 keys (half h) of a row, in fp16 in its line of the operand; the sum of their exponentials.
template <bool MASKED>
__device__ __forceinline__ float2 cw_weights(const float (&u)[128], int h, float c, float ref, const uint32_t (&vis)[4],
                                             const float* sv, uint8_t* line, int sw) {
  const float2 c2 = make_float2(c, c), nref = make_float2(-ref, -ref);
  float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const float4 f = *reinterpret_cast<const float4*>(sv + h * 64 + i * 8 + 4 * q);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int k = h * 64 + i * 8 + 4 * q + 2 * e;
        const float2 t = __ffma2_rn(c2, make_float2(u[k], u[k + 1]), nref);
        float2 pr = make_float2(ex2_approx(t.x), ex2_approx(t.y));
        float2 x = __fmul2_rn(pr, e == 0 ? make_float2(f.x, f.y) : make_float2(f.z, f.w));
        if (MASKED) {
          const bool a = vis[k >> 5] >> (k & 31) & 1u, b = vis[k >> 5] >> ((k & 31) + 1) & 1u;
          pr = make_float2(a ? pr.x : 0.0f, b ? pr.y : 0.0f);
          x = make_float2(a ? x.x : 0.0f, b ? x.y : 0.0f);
        }
        sum[e] = __fadd2_rn(sum[e], pr);
        const __half2 hx = __floats2half2_rn(x.x, x.y);
        w[2 * q + e] = *reinterpret_cast<const uint32_t*>(&hx);
      }
    }
    *reinterpret_cast<uint4*>(line + ((i ^ sw) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  return __fadd2_rn(sum[0], sum[1]);
}

template <bool F16>
__global__ void __launch_bounds__(CW_THREADS, 1)
    cache_attention_wide_kernel(const __grid_constant__ CUtensorMap tmK, const CaParams p) {
  using L = CwSmem;
  extern __shared__ uint8_t smem_raw[];
  // aligned by an offset, not through an integer, so that the compiler still knows it is shared memory
  uint8_t* smem = smem_raw + ((0u - smem_addr(smem_raw)) & 1023u);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
  uint64_t* drain = bars + 16;
  volatile int* abort = reinterpret_cast<volatile int*>(smem + L::kOffMisc);
  uint32_t* tmem_ptr = reinterpret_cast<uint32_t*>(smem + L::kOffMisc + 8);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto bar = [&](int pipe, int which) { return bars + pipe * kBars + which; };

  griddep_launch_dependents();
  if (tid == 0) {
    prefetch_tensormap(&tmK);
    for (int pipe = 0; pipe < 2; ++pipe) {
      mbar_init(bar(pipe, kKFull), 1);
      mbar_init(bar(pipe, kKEmpty), 1);
      mbar_init(bar(pipe, kSFull), 1);
      mbar_init(bar(pipe, kSEmpty), 4);
      mbar_init(bar(pipe, kPFull), 4);
      mbar_init(bar(pipe, kODone), 1);
      mbar_init(bar(pipe, kVFull), 4);
      mbar_init(bar(pipe, kScFull), 4);
    }
    mbar_init(drain, 1);
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == 13) {
    tmem_alloc(tmem_ptr, 512);
    tmem_relinquish();
  }
  int bad = 0;
  CaWalk<CwGrain> walk{};
  const int64_t per = ca_piece<CwGrain, CW_THREADS>(p, reinterpret_cast<int64_t*>(smem + L::kOffScan), &walk, bad);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_ptr;  // S of the two pipelines, then O

  // A wait of the role; false once one has run out anywhere in the CTA.
  auto wait = [&](uint64_t* b, int use) {
    const bool ok = mbar_wait_bounded(b, static_cast<uint32_t>(use & 1), abort, CW_TIMEOUT_NS);
    if (!ok) {
      *abort = 1;
      bad |= CA_LATE;
    }
    return ok;
  };
  // Tiles that a pipeline has taken in earlier runs: the parity of its barriers. Every role counts alike, and
  // meets the others twice a run (barrier 0): the queries are in place; the sums have been read.
  int used[2] = {0, 0};
  CaRun r;
  CaCut cut{};

  if (warp < 8) {
    // ---------------------------------------------------------------- softmax
    regs_more<192>();
    const int pipe = warp >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t tS = tmem + lanes + pipe * 128, tO = tmem + lanes + 256 + pipe * 128;
    uint8_t* line = smem + L::kOffP + pipe * 2 * CW_HALF + row * 128;
    const int sw = row & 7;
    float* row_c = reinterpret_cast<float*>(smem + L::kOffRow);
    float2* stat = reinterpret_cast<float2*>(smem + L::kOffStat);
    while (walk.next(p, &r, bad)) {
      const int keys = walk.s.keys, context = keys - walk.s.news;
      if (keys == 0) {  // nothing to see: zeros
        for (int i = tid; i < r.rows * (CA_D / 8); i += 256) {
          const int of = r.row0 + i / (CA_D / 8), token = of / p.G;
          *reinterpret_cast<uint4*>(p.o + (walk.s.first + token) * p.ot + (r.head * p.G + (of - token * p.G)) * p.oh +
                                    8 * (i % (CA_D / 8))) = make_uint4(0u, 0u, 0u, 0u);
        }
        continue;
      }
      if (p.tree != nullptr && walk.s.news > 64) bad |= CA_BAD;
      // the tile's queries, rotated and quantised: 16 rows a warp, four at a time
#pragma unroll 1
      for (int k0 = 0; k0 < 16; k0 += 4) {
        float v[4][4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int at = warp + 8 * (k0 + k);
          v[k][0] = v[k][1] = v[k][2] = v[k][3] = 0.0f;
          if (at < r.rows) {
            const int of = r.row0 + at, i = of / p.G;
            const uint16_t* src = p.q + (walk.s.first + i) * p.qt + (r.head * p.G + (of - i * p.G)) * p.qh;
            const uint2 w = __ldg(reinterpret_cast<const uint2*>(src + 4 * lane));
            const float2 a = fwht::widen_pair<F16>(w.x), b = fwht::widen_pair<F16>(w.y);
            v[k][0] = a.x, v[k][1] = a.y, v[k][2] = b.x, v[k][3] = b.y;
          }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int at = warp + 8 * (k0 + k);
          fwht::fwht128_warp(v[k], lane);
          float amax = fmaxf(fmaxf(fabsf(v[k][0]), fabsf(v[k][1])), fmaxf(fabsf(v[k][2]), fabsf(v[k][3])));
#pragma unroll
          for (int m = 16; m > 0; m >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, m));
          const fwht::CodeFactor f = fwht::code_factor(amax);
          float c[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) c[e] = fmaf(v[k][e] * f.pre, f.ci, fwht::kRoundMagic);
          *reinterpret_cast<uint32_t*>(smem + L::kOffQ + at * 128 + (((lane >> 2) ^ (at & 7)) << 4) + (lane & 3) * 4) =
              fwht::pack4(c[0], c[1], c[2], c[3]);
          if (lane == 0) row_c[at] = fwht::scale_of<128>(amax) * p.c_scale;
        }
      }
      fence_proxy_async_smem();
      cw_sync(0, CW_THREADS);

      const float c = row_c[row];  // >= 0
      int lim = 0;                 // keys below it are seen, and with a tree the drafted keys whose bit is set
      unsigned long long bits = 0;
      {
        const int i = row < r.rows ? (r.row0 + row) / p.G : 0;
        lim = p.tree != nullptr ? context : context + i + 1;
        if (p.tree != nullptr && row < r.rows) bits = __ldg(p.tree + walk.s.first + i);
      }
      const int clear = p.tree != nullptr ? context : context + 1;  // keys below it are seen by every row
      float ref = CA_NONE, l = 0.0f;
      bool weighed = false;  // the row has had a weight
      bool ok = true;
      int use = used[pipe];
      for (int t = r.t0 + pipe; t < r.t1; t += 2, ++use) {
        const int key0 = t * CW_KT;
        const int buffer = pipe * 2 + (use & 1);
        const float* sk = reinterpret_cast<const float*>(smem + L::kOffScale) + buffer * 256;
        const float* sv = sk + 128;
        const uint32_t* there = reinterpret_cast<const uint32_t*>(smem + L::kOffTile) + buffer * 8;
        const float* most = reinterpret_cast<const float*>(there + 4);
        ok = __all_sync(0xFFFFFFFFu, wait(bar(pipe, kScFull), use) && wait(bar(pipe, kSFull), use));
        if (!ok) break;
        tc_fence_after();
        float u[128];  // s_k[key] S[row, key]: the logit without the row's factor
        {
          uint32_t a0[32], a1[32];
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            tmem_ld_32x32b_x32(tS + half * 64, a0);
            tmem_ld_32x32b_x32(tS + half * 64 + 32, a1);
            tmem_ld_wait_regs(a0);
            tmem_ld_wait_regs(a1);
            if (half == 1) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(bar(pipe, kSEmpty));
            }
            const float2 mg = make_float2(-12582912.0f, -12582912.0f);
#pragma unroll
            for (int k4 = 0; k4 < 16; ++k4) {
              const float4 s4 = *reinterpret_cast<const float4*>(sk + half * 64 + 4 * k4);
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int k = 4 * k4 + 2 * e;
                const uint32_t x0 = (k < 32) ? a0[k] : a1[k - 32], x1 = (k + 1 < 32) ? a0[k + 1] : a1[k - 31];
                // float(acc) for |acc| < 2^22: the integer added to the bits of 1.5 * 2^23, minus 1.5 * 2^23
                const float2 x = make_float2(__uint_as_float(x0 + 0x4B400000u), __uint_as_float(x1 + 0x4B400000u));
                const float2 v =
                    __fmul2_rn(__fadd2_rn(x, mg), e == 0 ? make_float2(s4.x, s4.y) : make_float2(s4.z, s4.w));
                u[half * 64 + k] = v.x;
                u[half * 64 + k + 1] = v.y;
              }
            }
          }
        }
        uint32_t vis[4] = {there[0], there[1], there[2], there[3]};
        const bool masked = key0 + CW_KT > clear || (vis[0] & vis[1] & vis[2] & vis[3]) != 0xFFFFFFFFu;
        float top;
        if (!masked) {
          float a[43], b[15], c5[5];
#pragma unroll
          for (int i = 0; i < 42; ++i) a[i] = fwht::fmax3f(u[3 * i], u[3 * i + 1], u[3 * i + 2]);
          a[42] = fmaxf(u[126], u[127]);
#pragma unroll
          for (int i = 0; i < 14; ++i) b[i] = fwht::fmax3f(a[3 * i], a[3 * i + 1], a[3 * i + 2]);
          b[14] = a[42];
#pragma unroll
          for (int i = 0; i < 5; ++i) c5[i] = fwht::fmax3f(b[3 * i], b[3 * i + 1], b[3 * i + 2]);
          top = fmaxf(fwht::fmax3f(c5[0], c5[1], c5[2]), fmaxf(c5[3], c5[4]));
        } else {
          top = -INFINITY;
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            vis[w] &= below(lim - key0, w) | placed(bits, context - key0, w);
#pragma unroll
            for (int k = 0; k < 32; ++k) top = (vis[w] >> k & 1u) ? fmaxf(top, u[32 * w + k]) : top;
          }
        }
        const bool some = (vis[0] | vis[1] | vis[2] | vis[3]) != 0;
        const float tm = some ? c * top : CA_NONE;
        // log2 of the tile's largest value scale, rounded up
        const float high = fmaxf(fmaxf(most[0], most[1]), fmaxf(most[2], most[3]));
        const float e_high = static_cast<float>(static_cast<int>(__float_as_uint(high) >> 23) - 126);
        float alpha = 1.0f;
        if (__any_sync(0xFFFFFFFFu, some && (!weighed || tm + e_high > ref + CW_FIT || tm > ref + CW_SPAN))) {
          // the row's largest weight, as a power of two over its largest logit
          float big = 0.0f;
#pragma unroll
          for (int k = 0; k < 128; ++k) {
            const float x = ex2_approx(fmaf(c, u[k], -tm)) * sv[k];
            big = (vis[k >> 5] >> (k & 31) & 1u) ? fmaxf(big, x) : big;
          }
          const float at = tm + static_cast<float>(static_cast<int>(__float_as_uint(big) >> 23) - 127);
          float now = ref;
          if (some) {
            if (!weighed) now = big > 0.0f ? at : tm;
            else if (big > 0.0f && at > ref + (CW_FIT - 1.0f)) now = at;
            if (tm > now + CW_SPAN) now = tm - CW_SPAN;
            weighed |= big > 0.0f;
          }
          alpha = ref == CA_NONE ? 0.0f : ex2_approx(ref - now);
          if (now == ref) alpha = 1.0f;
          ref = now;
        }
        // the pipeline's last P V has finished: O is stable and the operand's memory free
        if (use > 0) {
          ok = __all_sync(0xFFFFFFFFu, wait(bar(pipe, kODone), use - 1));
          if (!ok) break;
        }
        tc_fence_after();
        float2 sum;
        if (!masked) {
          sum = __fadd2_rn(cw_weights<false>(u, 0, c, ref, vis, sv, line, sw),
                           cw_weights<false>(u, 1, c, ref, vis, sv, line + CW_HALF, sw));
        } else {
          sum = __fadd2_rn(cw_weights<true>(u, 0, c, ref, vis, sv, line, sw),
                           cw_weights<true>(u, 1, c, ref, vis, sv, line + CW_HALF, sw));
        }
        l = l * alpha + (sum.x + sum.y);
        if (t >= r.t0 + 2 && __any_sync(0xFFFFFFFFu, alpha != 1.0f)) {
#pragma unroll
          for (int ch = 0; ch < 4; ++ch) {
            uint32_t o[32];
            tmem_ld_32x32b_x32(tO + ch * 32, o);
            tmem_ld_wait_regs(o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            tmem_st_32x32b_x32(tO + ch * 32, o);
          }
          tmem_st_wait();
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(pipe, kPFull));
      }
      const int mine = r.t1 - r.t0 > pipe ? (r.t1 - r.t0 - pipe + 1) / 2 : 0;
      if (ok && mine > 0) ok = __all_sync(0xFFFFFFFFu, wait(bar(pipe, kODone), used[pipe] + mine - 1));
      stat[pipe * 128 + row] = make_float2(ref, l);
      tc_fence_before();
      cw_sync(1, 256);
      tc_fence_after();
      // ---- the pipelines joined; channels 0 .. 63 here, 64 .. 127 in the other pipeline's warps
      const bool second = r.t1 - r.t0 > 1;
      const float2 s0 = stat[row], s1 = second ? stat[128 + row] : make_float2(CA_NONE, 0.0f);
      const float top = fmaxf(s0.x, s1.x);
      const float f0 = ex2_approx(s0.x - top), f1 = ex2_approx(s1.x - top);
      const float total = s0.y * f0 + s1.y * f1;
      const bool whole = r.t0 == 0 && r.t1 == walk.s.tiles;
      const uint32_t tO0 = tmem + lanes + 256, tO1 = tO0 + 128;
      const bool alive = *abort == 0;  // else there may be no sums
      float v[64];
#pragma unroll
      for (int ch = 0; ch < 2; ++ch) {
        uint32_t a[32], b[32];
        // whole: the last butterfly stage, between channels 64 apart, comes first; part: this half's channels
        const int from = whole ? ch * 32 : pipe * 64 + ch * 32;
        tmem_ld_32x32b_x32(tO0 + from, a);
        tmem_ld_wait_regs(a);
#pragma unroll
        for (int i = 0; i < 32; ++i) v[ch * 32 + i] = __uint_as_float(a[i]) * f0;
        if (second) {
          tmem_ld_32x32b_x32(tO1 + from, b);
          tmem_ld_wait_regs(b);
#pragma unroll
          for (int i = 0; i < 32; ++i) v[ch * 32 + i] = fmaf(__uint_as_float(b[i]), f1, v[ch * 32 + i]);
        }
        if (whole) {
          const float sign = pipe == 0 ? 1.0f : -1.0f;
          tmem_ld_32x32b_x32(tO0 + 64 + from, a);
          tmem_ld_wait_regs(a);
#pragma unroll
          for (int i = 0; i < 32; ++i) v[ch * 32 + i] = fmaf(__uint_as_float(a[i]), sign * f0, v[ch * 32 + i]);
          if (second) {
            tmem_ld_32x32b_x32(tO1 + 64 + from, b);
            tmem_ld_wait_regs(b);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[ch * 32 + i] = fmaf(__uint_as_float(b[i]), sign * f1, v[ch * 32 + i]);
          }
        }
      }
      if (whole) {
        const float norm = total == 0.0f ? 0.0f : fwht::kInvSqrt128 / total;
#pragma unroll
        for (int i = 0; i < 64; ++i) v[i] = total == 0.0f ? 0.0f : v[i] * norm;
        fwht::reg_stage<64, 1>(v);
        fwht::reg_stage<64, 2>(v);
        fwht::reg_stage<64, 4>(v);
        fwht::reg_stage<64, 8>(v);
        fwht::reg_stage<64, 16>(v);
        fwht::reg_stage<64, 32>(v);
        if (row < r.rows && alive) {
          const int of = r.row0 + row, i = of / p.G;
          uint16_t* dst = p.o + (walk.s.first + i) * p.ot + (r.head * p.G + (of - i * p.G)) * p.oh + 64 * pipe;
#pragma unroll
          for (int k = 0; k < 8; ++k)
            *reinterpret_cast<uint4*>(dst + 8 * k) = make_uint4(
                fwht::narrow_pair<F16>(v[8 * k], v[8 * k + 1]), fwht::narrow_pair<F16>(v[8 * k + 2], v[8 * k + 3]),
                fwht::narrow_pair<F16>(v[8 * k + 4], v[8 * k + 5]), fwht::narrow_pair<F16>(v[8 * k + 6], v[8 * k + 7]));
        }
      } else if (row < r.rows && alive) {
        const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (r.t0 == 0 ? 1 : 0);
        float4* dst = reinterpret_cast<float4*>(p.part + (slot * CA_WIDE_ROWS + row) * CA_D + 64 * pipe);
#pragma unroll
        for (int k = 0; k < 16; ++k) dst[k] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
        if (pipe == 0) p.part_ml[slot * CA_WIDE_ROWS + row] = make_float2(top, total);
      }
      if (r.t0 == 0 && !whole) {
        // the piece ends inside an item that begins in it: it describes the item to the join
        cut.pieces = static_cast<int>((walk.end + r.left - 1) / per) - static_cast<int>(blockIdx.x) + 1;
        cut.rows = r.rows;
        cut.row0 = r.row0;
        cut.head = r.head;
        cut.token0 = walk.s.first;
      }
      used[0] += (r.t1 - r.t0 + 1) / 2;
      used[1] += (r.t1 - r.t0) / 2;
      tc_fence_before();
      cw_sync(0, CW_THREADS);
    }
    if (tid == 0) p.cuts[blockIdx.x] = cut;
  } else if (warp < 12) {
    // ----------------------------------------------------------------- values
    regs_fewer<64>();
    const int me = tid - 256;  // the thread's key of a tile, for the scales
    const int w4 = warp - 8;
    while (walk.next(p, &r, bad)) {
      if (walk.s.keys == 0) continue;
      const int keys = walk.s.keys;
      const int32_t* table = p.pages + walk.b * p.table_stride;
      auto cell_of = [&](int key) {  // the cell of a key, or -1
        if (key >= keys) return -1;
        const int page = __ldg(table + (key >> p.page_shift));
        if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(p.num_pages)) {
          bad |= CA_BAD;  // its keys are not seen
          return -1;
        }
        return ((page * p.Hkv + r.head) << p.page_shift) + (key & ((1 << p.page_shift) - 1));
      };
      cw_sync(0, CW_THREADS);
      bool ok = true;
      for (int t = r.t0; t < r.t1 && ok; ++t) {
        const int pipe = (t - r.t0) & 1, use = used[pipe] + ((t - r.t0) >> 1);
        const int key0 = t * CW_KT;
        // eight lanes a key, 16 codes each: keys w4 * 32 + 4 i + lane / 8
        uint4 code[8];
        const int my_cell = cell_of(key0 + me);
        const float mk = my_cell >= 0 ? __ldg(p.k_scale + my_cell) : 0.0f;
        const float mv = my_cell >= 0 ? __ldg(p.v_scale + my_cell) : 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int cell = __shfl_sync(0xFFFFFFFFu, my_cell, 4 * i + (lane >> 3));
          code[i] = cell >= 0 ? __ldg(reinterpret_cast<const uint4*>(p.v_codes + static_cast<int64_t>(cell) * CA_D) +
                                      (lane & 7))
                              : make_uint4(0u, 0u, 0u, 0u);
        }
        // the scale buffer was last used two tiles of this pipeline ago, whose softmax is done once the next began
        if (use > 0) ok = __all_sync(0xFFFFFFFFu, wait(bar(pipe, kSEmpty), use - 1));
        if (!ok) break;
        const int buffer = pipe * 2 + (use & 1);
        float* sk = reinterpret_cast<float*>(smem + L::kOffScale) + buffer * 256;
        uint32_t* there = reinterpret_cast<uint32_t*>(smem + L::kOffTile) + buffer * 8;
        sk[me] = mk;
        sk[128 + me] = mv;
        const uint32_t on = __ballot_sync(0xFFFFFFFFu, my_cell >= 0);
        float most = fabsf(mv);
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, m));
        if (lane == 0) {
          there[w4] = on;
          reinterpret_cast<float*>(there + 4)[w4] = most;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(pipe, kScFull));
        if (use > 0) ok = __all_sync(0xFFFFFFFFu, wait(bar(pipe, kODone), use - 1));
        if (!ok) break;
        uint8_t* to = smem + L::kOffV + pipe * 2 * CW_HALF + ((lane >> 2) & 1) * CW_HALF;  // channels from 64 on: second half
        const __half2 offset = __floats2half2_rn(1152.0f, 1152.0f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int key = w4 * 32 + 4 * i + (lane >> 3);
          const uint32_t word[4] = {code[i].x ^ 0x80808080u, code[i].y ^ 0x80808080u, code[i].z ^ 0x80808080u,
                                    code[i].w ^ 0x80808080u};
          uint32_t h[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            // fp16 of a code: the byte plus 128 in the low bits of 1024, minus 1152, exactly
            const uint32_t x = __byte_perm(word[e >> 1], 0x64646464u, e & 1 ? 0x4342 : 0x4140);
            const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&x), offset);
            h[e] = *reinterpret_cast<const uint32_t*>(&y);
          }
          const int chunk = 2 * (lane & 3);
          *reinterpret_cast<uint4*>(to + key * 128 + ((chunk ^ (key & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
          *reinterpret_cast<uint4*>(to + key * 128 + (((chunk + 1) ^ (key & 7)) << 4)) =
              make_uint4(h[4], h[5], h[6], h[7]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(pipe, kVFull));
      }
      used[0] += (r.t1 - r.t0 + 1) / 2;
      used[1] += (r.t1 - r.t0) / 2;
      cw_sync(0, CW_THREADS);
    }
  } else {
    regs_fewer<64>();
    if (warp == 12) {
      // ------------------------------------------------------------------ keys
      int issued[2] = {0, 0};
      while (walk.next(p, &r, bad)) {
        if (walk.s.keys == 0) continue;
        cw_sync(0, CW_THREADS);
        if (lane == 0) {
          const int32_t* table = p.pages + walk.b * p.table_stride;
          bool ok = true;
          for (int t = r.t0; t < r.t1; ++t) {
            const int pipe = (t - r.t0) & 1, use = used[pipe] + ((t - r.t0) >> 1);
            if (use > 0) ok = wait(bar(pipe, kKEmpty), use - 1);
            if (!ok) break;
            int cell[8], boxes = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int key = t * CW_KT + 16 * i;
              cell[i] = -1;
              if (key < walk.s.keys) {
                const int page = __ldg(table + (key >> p.page_shift));
                if (static_cast<uint32_t>(page) < static_cast<uint32_t>(p.num_pages)) {
                  cell[i] = ((page * p.Hkv + r.head) << p.page_shift) + (key & ((1 << p.page_shift) - 1));
                  ++boxes;
                }
              }
            }
            mbar_arrive_expect_tx(bar(pipe, kKFull), boxes * 16 * CA_D);
            uint8_t* to = smem + L::kOffK + pipe * CW_HALF;
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (cell[i] >= 0) tma_load_2d(to + i * 16 * CA_D, &tmK, bar(pipe, kKFull), 0, cell[i]);
            issued[pipe] = use + 1;
          }
        }
        used[0] += (r.t1 - r.t0 + 1) / 2;
        used[1] += (r.t1 - r.t0) / 2;
        __syncwarp();
        cw_sync(0, CW_THREADS);
      }
      // every copy has landed before the shared memory goes away
      if (lane == 0)
        for (int pipe = 0; pipe < 2; ++pipe)
          if (issued[pipe] > 0)
            mbar_wait_bounded(bar(pipe, kKFull), static_cast<uint32_t>((issued[pipe] - 1) & 1), nullptr, CW_TIMEOUT_NS);
    } else if (warp == 13) {
      // -------------------------------------------------------------- products
      const uint32_t qa = smem_addr(smem + L::kOffQ);
      while (walk.next(p, &r, bad)) {
        if (walk.s.keys == 0) continue;
        cw_sync(0, CW_THREADS);
        tc_fence_after();
        if (lane == 0) {
          const int tiles = r.t1 - r.t0;
          auto logits = [&](int n) {  // S of tile n of the run
            const int pipe = n & 1, use = used[pipe] + (n >> 1);
            if (!wait(bar(pipe, kKFull), use)) return false;
            tc_fence_after();
            const uint32_t kb = smem_addr(smem + L::kOffK + pipe * CW_HALF);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_i8(tmem + pipe * 128, smem_desc_k_sw128(qa + k * 32), smem_desc_k_sw128(kb + k * 32), CW_IDESC_S,
                     k > 0 ? 1u : 0u);
            mma_commit(bar(pipe, kSFull));
            mma_commit(bar(pipe, kKEmpty));
            return true;
          };
          bool ok = logits(0);
          if (ok && tiles > 1) ok = logits(1);
          for (int n = 0; n < tiles && ok; ++n) {
            const int pipe = n & 1, use = used[pipe] + (n >> 1);
            // the pipeline's next S once its softmax has read this one
            if (n + 2 < tiles) ok = wait(bar(pipe, kSEmpty), use) && logits(n + 2);
            if (!ok || !wait(bar(pipe, kPFull), use) || !wait(bar(pipe, kVFull), use)) break;
            tc_fence_after();
            const uint32_t pa = smem_addr(smem + L::kOffP + pipe * 2 * CW_HALF);
            const uint32_t va = smem_addr(smem + L::kOffV + pipe * 2 * CW_HALF);
            // 16 keys an instruction: P's K-major rows advance 32 bytes inside a 64-key half; the values' atoms are
            // 8 keys x 64 channels (1 KB apart along the keys, the second 64 channels 16 KB on)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma_bf16(tmem + 256 + pipe * 128, smem_desc_k_sw128(pa + h * CW_HALF + k * 32),
                         smem_desc_mn_sw128(va + (4 * h + k) * 2048, CW_HALF, 1024), CW_IDESC_O,
                         (n >= 2 || h > 0 || k > 0) ? 1u : 0u);
            mma_commit(bar(pipe, kODone));
          }
        }
        used[0] += (r.t1 - r.t0 + 1) / 2;
        used[1] += (r.t1 - r.t0) / 2;
        __syncwarp();
        cw_sync(0, CW_THREADS);
      }
      if (lane == 0) {
        // every product issued has finished before TMEM is released
        mma_commit(drain);
        mbar_wait_bounded(drain, 0u, nullptr, CW_TIMEOUT_NS);
      }
      __syncwarp();
    } else {
      while (walk.next(p, &r, bad)) {
        if (walk.s.keys == 0) continue;
        cw_sync(0, CW_THREADS);
        cw_sync(0, CW_THREADS);
      }
    }
  }
  tc_fence_before();
  const int any_bad = __syncthreads_or(bad & CA_BAD), late = __syncthreads_or(bad & 4);  // a timeout is 5
  if (tid == 0) p.piece_status[blockIdx.x] = late ? CA_LATE : any_bad ? CA_BAD : 0;
  if (warp == 13) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

PFN_cuTensorMapEncodeTiled_v12000 cw_encoder() {
  static std::atomic<void*> fn{nullptr};
  void* f = fn.load(std::memory_order_acquire);
  if (f == nullptr) {
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    fn.store(f, std::memory_order_release);
  }
  return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
}

template <bool F16>
cudaError_t cw_launch(const CUtensorMap& tk, const CaParams& p, cudaStream_t s) {
  static std::atomic<int> ready[64];  // devices whose attribute is set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool known = dev >= 0 && dev < 64;
  if (!known || ready[dev].load(std::memory_order_acquire) == 0) {
    e = cudaFuncSetAttribute(cache_attention_wide_kernel<F16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             CwSmem::kAlloc);
    if (e != cudaSuccess) return e;
    if (known) ready[dev].store(1, std::memory_order_release);
  }
  cache_attention_wide_kernel<F16><<<p.workers, CW_THREADS, CwSmem::kAlloc, s>>>(tk, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_attention_wide(const CaParams& p, bool f16, int64_t cells, cudaStream_t stream) {
  const auto enc = cw_encoder();
  if (enc == nullptr) return cudaErrorNotSupported;
  // key codes as rows of 128 bytes, boxes of 16 keys, 128-byte swizzle
  const cuuint64_t dims[2] = {CA_D, static_cast<cuuint64_t>(cells)};
  const cuuint64_t strides[1] = {CA_D};
  const cuuint32_t box[2] = {CA_D, 16};
  const cuuint32_t step[2] = {1, 1};
  CUtensorMap tk;
  if (enc(&tk, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t*>(p.k_codes), dims, strides, box, step,
          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  return f16 ? cw_launch<true>(tk, p, stream) : cw_launch<false>(tk, p, stream);
}

}  // namespace convrot
