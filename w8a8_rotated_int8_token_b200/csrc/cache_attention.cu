// Attention of a few new tokens per sequence over the rotated int8 key/value
// cache: single tokens, causal chunks and trees of drafted tokens.
//
//   S[r, j] = (cq[r] . ck[j]) s_q[r] s_k[j] softmax_scale,  O = (softmax(S) (cv s_v)) R,
//
// with cq, s_q the int8 codes of the rotated query (the rule of the INT8
// attention), the integer products exact, softmax in float32 in one pass over
// the keys with a running maximum and sum, and one rotation of the output row
// (R = H_128 / sqrt(128) is its own inverse and linear, so it commutes with the
// sum over keys).
//
// Bound by memory: every key costs 264 bytes and is read once per tile of
// query rows. The rows of a tile are the query heads that share a key head
// times the sequence's new tokens. The work (sequence, row tile, key head,
// tiles of 64 keys) is one long line cut into equal pieces, one per CTA, so that
// ragged lengths and small batches fill the GPU alike; a CTA finds its piece
// from the lengths on the device. Where an item is cut, each CTA leaves its
// unnormalised sum, maximum and row sum in the workspace, and a second kernel
// joins them in a fixed order, so the result does not depend on timing.
//
// One CTA is four warps; warp w takes keys 16 w .. 16 w + 15 of every 64-key tile
// for all 8 NT rows. Each warp feeds itself: its lanes copy its keys' codes and
// scales (16 bytes a lane, asynchronously, swizzled against bank conflicts) into
// the warp's own ring of stages, so no warp waits for another before the end of a
// run, and 16 keys never cross a page. TMA boxes and bulk copies of the same 16
// keys under mbarriers took three times the instructions a stage and 268 us where
// these took 251 (64 sequences of up to 16384 keys).
// The keys and channels are the long side of the matrix instructions, the rows
// the short one (8), so a tile of 8 rows, the usual one of single tokens, wastes
// no more than it must:
//   S^T = K Q^T      int8 m16n8k32, the key codes through ldmatrix;
//   O^T = V^T P^T    fp16 m16n8k16: the value codes widened exactly to fp16 in
//         registers, the weights transposed by movmatrix. The weights p s_v are
//         brought to fp16's range by a factor per row, kept so that the largest
//         weight so far lies between 1 and 2^15: rounding one to fp16 costs at
//         most 2^-11 of it or 2^-25 of the largest, whatever the range of the
//         value scales. That is far below bf16's own rounding of the output; for
//         an fp16 output, whose rounding is no larger, a second product adds what
//         the first rounding left.
// The reference maximum and that factor move only when a key passes them by far;
// a vote of the warp is all it costs otherwise.
// Times here and below are of the device, for captured calls with bf16 outputs.

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <initializer_list>

#include "cache_attention.cuh"
#include "convrot.h"
#include "fwht128.cuh"
#include "fwht_dev.cuh"
#include "ptx_sm100.cuh"

namespace convrot {

namespace {

constexpr int CA_WARPS = 4;
constexpr int CA_THREADS = 32 * CA_WARPS;
constexpr int CA_SUB = 16;                 // keys of a warp's stage
constexpr int CA_KT = CA_SUB * CA_WARPS;   // keys of a tile
constexpr int CA_CODES = CA_SUB * CA_D;    // key (or value) codes of a stage
constexpr int CA_STAGE = 2 * CA_CODES;
constexpr int CA_QPITCH = CA_D + 16;       // bytes between query rows in shared memory
// What a run costs beside its tiles, and the least a piece takes, in tiles: with a cost of 6 the trees of 8 sequences
// took 74 us against 83 with 4 and 102 with none (64 long sequences 218 us, 226 with 4, 223 with 8), and one sequence of
// 4224 keys takes 10.9 us with a least of 3, 12.4 with 2, 11.4 with 4, 11.7 with 6.
constexpr int CA_SETUP = 6;
constexpr int CA_LEAST = 3;

// A shape of CTA: 8 NT rows, stages of a warp's ring, CTAs per SM.
template <int NT, int ST, int OCC>
struct CaShape {
  static constexpr int kNt = NT, kStages = ST, kOcc = OCC;
  static constexpr int kRows = 8 * NT;
  static constexpr int kOffScale = CA_WARPS * ST * CA_STAGE;  // per stage: 16 key, 16 value scales
  static constexpr int kOffQ = kOffScale + CA_WARPS * ST * 2 * CA_SUB * 4;
  static constexpr int kOffRow = kOffQ + kRows * CA_QPITCH;   // per row: tree bits, factor, first key not seen
  static constexpr int kOffScan = kOffRow + kRows * 16;
  static constexpr int kBytes = kOffScan + 64;
  // the end of a run exchanges sums through the (then idle) ring: per warp 4 KB and statistics per 8 rows
  static constexpr int kJoinWarp = NT * 8 * 32 * 16 + NT * 32 * 16;
  static_assert(2 * kJoinWarp <= kOffScale, "exchange fits the ring");
};

// Two stages of 16 keys a warp at four CTAs per SM keep 130 KB of copies in flight; three stages took 3 % longer (64
// long sequences), five CTAs with 96 registers 9 %. A tile of 32 rows with 255 registers and two CTAs took 1.1 times
// as long as two of 16 rows on a tree of 64 drafts.
using Shape8 = CaShape<1, 2, 4>;
using Shape16 = CaShape<2, 3, 3>;

__device__ __forceinline__ void mma_s8(int (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The same with a zero accumulator.
__device__ __forceinline__ void mma_s8_first(int (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "r"(0));
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Four 8 x 16-byte matrices; each lane names a row of one.
__device__ __forceinline__ void load_matrices(uint32_t (&a)[4], uint32_t from) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3])
               : "r"(from)
               : "memory");
}

// The transpose of an 8 x 8 matrix of 16-bit values.
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// Two sums of 128 products of codes up to 127 (|acc| < 2^22) as floats times `by`, without a conversion
// instruction: the integer added to the bits of 1.5 * 2^23 is exact, and so is subtracting 1.5 * 2^23.
__device__ __forceinline__ float2 code_sums(int a, int b, float2 by) {
  const float2 x = make_float2(__uint_as_float(static_cast<uint32_t>(a) + 0x4B400000u),
                               __uint_as_float(static_cast<uint32_t>(b) + 0x4B400000u));
  return __fmul2_rn(__fadd2_rn(x, make_float2(-12582912.0f, -12582912.0f)), by);
}

// Sixteen bytes global -> shared, past L1, at constant offsets.
template <int TO, int FROM>
__device__ __forceinline__ void copy_async(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0 + %2], [%1 + %3], 16;" ::"r"(to), "l"(from), "n"(TO), "n"(FROM)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {  // all but the last N groups have landed
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// The reference of a row moves when a logit passes it by 24 (exponentials of up to 2^24 cost float32 no
// precision), and the factor when a weight passes 2^15 of fp16's 65504: with 8 and 2^12 a tile of 32 rows moved one of
// them at every other step of a short run.
constexpr float CA_RISE = 24.0f;
constexpr float CA_MOST = 32768.0f;
// The weights' factor of a row without a weight, and the largest there is: the first weight brings it down.
constexpr float CA_UNSET = 0x1p100f;

// The maximum of each row over the lanes that hold its keys.
__device__ __forceinline__ float2 row_max(float2 v) {
#pragma unroll
  for (int m = 4; m < 32; m <<= 1) {
    v.x = fmaxf(v.x, __shfl_xor_sync(0xFFFFFFFFu, v.x, m));
    v.y = fmaxf(v.y, __shfl_xor_sync(0xFFFFFFFFu, v.y, m));
  }
  return v;
}

// 2^-e for the exponent e of a row's largest weight, within float32's normal range: it brings that weight to [1, 2).
__device__ __forceinline__ float weight_factor(float weight) {
  const uint32_t e = min(max(__float_as_uint(weight) >> 23, 27u), 253u);
  return __uint_as_float((254u - e) << 23);
}

// The exponent of a sum of exponentials; 0 below 2, and at most 100, which no number of keys reaches.
__device__ __forceinline__ float sum_exponent(float sum) {
  return static_cast<float>(min(max(__float_as_uint(sum) >> 23, 127u), 227u) - 127u);
}

template <class Shape, bool F16>
__global__ void __launch_bounds__(CA_THREADS, Shape::kOcc)
    cache_attention_kernel(const CaParams p) {
  using Grain = CaGrain<Shape::kRows, CA_KT, CA_SETUP, CA_LEAST>;
  constexpr int NT = Shape::kNt, ST = Shape::kStages, ROWS = Shape::kRows;
  extern __shared__ __align__(128) uint8_t smem[];
  int64_t* scan = reinterpret_cast<int64_t*>(smem + Shape::kOffScan);  // a sum per warp; then found
  uint8_t* qs = smem + Shape::kOffQ;
  unsigned long long* row_bits = reinterpret_cast<unsigned long long*>(smem + Shape::kOffRow);
  float* row_c = reinterpret_cast<float*>(row_bits + ROWS);
  int* row_lim = reinterpret_cast<int*>(row_c + ROWS);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t4 = lane & 3;
  uint8_t* ring = smem + warp * ST * CA_STAGE;
  const float* ring_scale = reinterpret_cast<const float*>(smem + Shape::kOffScale) + warp * ST * 2 * CA_SUB;
  // a lane copies 16-byte chunk lane % 8 of keys lane / 8 + 4 i; chunk c of key j lies at c ^ (j % 8)
  const uint32_t ring_to = smem_addr(ring) + (lane >> 3) * CA_D + (((lane & 7) ^ (lane >> 3)) << 4);
  const uint32_t scale_to = smem_addr(ring_scale) + lane * 16;
  const int8_t* k_from = p.k_codes + lane * 16;
  const int8_t* v_from = p.v_codes + lane * 16;
  const float* scale_from = (lane < 4 ? p.k_scale : p.v_scale) + (lane & 3) * 4;
  // the row this lane names to ldmatrix: key lane % 16, chunk lane / 16 of each pair
  const uint32_t key_at = smem_addr(ring) + (lane & 15) * CA_D + (((lane >> 4) ^ (lane & 7)) << 4);
  // the value chunks of a lane: channels 16 g .. 16 g + 15 of keys 2 t, 2 t + 1 (and 8 more)
  const uint8_t* value_at = ring + CA_CODES + 2 * t4 * CA_D + ((g ^ (2 * t4)) << 4);
  const uint8_t* value_at1 = ring + CA_CODES + (2 * t4 + 1) * CA_D + ((g ^ (2 * t4 + 1)) << 4);

  griddep_launch_dependents();  // the join's CTAs may take their places; they wait for this grid

  int bad = 0;
  CaWalk<Grain> walk{};
  const int64_t per = ca_piece<Grain, CA_THREADS>(p, scan, &walk, bad);

  CaRun r;
  CaCut cut{};
  while (walk.next(p, &r, bad)) {
    const int keys = walk.s.keys;
    const int context = keys - walk.s.news;  // key of the first new token; may be negative
    const int32_t* table = p.pages + walk.b * p.table_stride;
    if (keys == 0) {  // nothing to see: zeros
      for (int i = tid; i < r.rows * (CA_D / 8); i += CA_THREADS) {
        const int of = r.row0 + i / (CA_D / 8), token = of / p.G;
        *reinterpret_cast<uint4*>(p.o + (walk.s.first + token) * p.ot + (r.head * p.G + (of - token * p.G)) * p.oh +
                                  8 * (i % (CA_D / 8))) = make_uint4(0u, 0u, 0u, 0u);
      }
      continue;
    }
    uint32_t live = 0;  // stages that hold keys
    // tiles of the run in which this warp has keys end before `last`
    const int with_keys = (keys - warp * CA_SUB + CA_KT - 1) / CA_KT;
    const int last = r.t1 < with_keys ? r.t1 : with_keys;
    auto lookup = [&](int t) {
      return t < last ? __ldg(table + ((t * CA_KT + warp * CA_SUB) >> p.page_shift)) : 0;
    };
    auto issue = [&](int t, int st, int page) {
      live &= ~(1u << st);
      if (t < last) {
        if (static_cast<uint32_t>(page) < static_cast<uint32_t>(p.num_pages)) {
          live |= 1u << st;
          // cells of a cache are fewer than 2^31
          const int cell = ((page * p.Hkv + r.head) << p.page_shift) +
                           ((t * CA_KT + warp * CA_SUB) & ((1 << p.page_shift) - 1));
          const int8_t* kf = k_from + static_cast<int64_t>(cell) * CA_D;
          const int8_t* vf = v_from + static_cast<int64_t>(cell) * CA_D;
          const uint32_t to = ring_to + st * CA_STAGE, to4 = to ^ 64u;  // four keys on, key % 8 differs in its top bit
          copy_async<0, 0>(to, kf);
          copy_async<512, 512>(to4, kf);
          copy_async<1024, 1024>(to, kf);
          copy_async<1536, 1536>(to4, kf);
          copy_async<CA_CODES, 0>(to, vf);
          copy_async<CA_CODES + 512, 512>(to4, vf);
          copy_async<CA_CODES + 1024, 1024>(to, vf);
          copy_async<CA_CODES + 1536, 1536>(to4, vf);
          if (lane < 8) copy_async<0, 0>(scale_to + st * (2 * CA_SUB * 4), scale_from + cell);
        } else {
          bad |= CA_BAD;  // its keys are not seen
        }
      }
      copy_commit();
    };
    int ahead;  // page of the next tile to issue
    {
      int page[ST];
#pragma unroll
      for (int i = 0; i < ST; ++i) page[i] = lookup(r.t0 + i);
      ahead = lookup(r.t0 + ST);
#pragma unroll
      for (int i = 0; i < ST; ++i) issue(r.t0 + i, i, page[i]);
    }

    // ---- the tile's queries: rotated, quantised, into shared memory
    if (p.tree != nullptr && walk.s.news > 64) bad |= CA_BAD;
#pragma unroll
    for (int k = 0; k < ROWS / CA_WARPS; ++k) {
      const int row = warp + k * CA_WARPS;
      float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      int i = 0;
      if (row < r.rows) {
        const int of = r.row0 + row;
        i = of / p.G;
        const uint16_t* src = p.q + (walk.s.first + i) * p.qt + (r.head * p.G + (of - i * p.G)) * p.qh;
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(src + 4 * lane));
        const float2 a = fwht::widen_pair<F16>(w.x), b = fwht::widen_pair<F16>(w.y);
        v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
      }
      fwht::fwht128_warp(v, lane);
      float amax = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
#pragma unroll
      for (int m = 16; m > 0; m >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, m));
      const fwht::CodeFactor f = fwht::code_factor(amax);
      float c[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) c[e] = fmaf(v[e] * f.pre, f.ci, fwht::kRoundMagic);
      *reinterpret_cast<uint32_t*>(qs + row * CA_QPITCH + 4 * lane) = fwht::pack4(c[0], c[1], c[2], c[3]);
      if (lane == 0) {
        row_c[row] = ca_query_factor(p, amax);
        // keys below the limit are seen, and with a tree the drafted keys whose bit is set
        const bool tree = p.tree != nullptr;
        row_lim[row] = tree ? context : context + i + 1;
        row_bits[row] = tree && row < r.rows ? __ldg(p.tree + walk.s.first + i) : 0ull;
      }
    }
    __syncthreads();
    uint32_t qb[NT][8];  // row g of each 8: bytes 4 t .. of every 16
    float2 cr[NT];       // factors of rows 2 t, 2 t + 1
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        qb[n][i] = *reinterpret_cast<const uint32_t*>(qs + (8 * n + g) * CA_QPITCH + 16 * i + 4 * t4);
      cr[n] = *reinterpret_cast<const float2*>(row_c + 8 * n + 2 * t4);
    }
    // acc[n][i]: channels 16 g + 2 i (rows 2 t, 2 t + 1 of the 8), then 16 g + 2 i + 1
    float acc[NT][8][4];
    float2 mx[NT], l[NT], inv[NT];  // maximum, sum and weights' factor of rows 2 t, 2 t + 1
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[n][i][0] = acc[n][i][1] = acc[n][i][2] = acc[n][i][3] = 0.0f;
      mx[n] = both(CA_NONE);
      inv[n] = both(CA_UNSET);
      l[n] = make_float2(0.0f, 0.0f);
    }

    // ---- the keys
    const int clear = p.tree != nullptr ? context : context + 1;  // keys below it are seen by every row
    int st = 0;
#pragma unroll 1
    for (int t = r.t0; t < r.t1; ++t) {
      copy_wait<ST - 1>();
      __syncwarp();  // every lane's copies
      if (live >> st & 1) {
        const int key0 = t * CA_KT + warp * CA_SUB;
        int d[NT][4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t a[4];  // channels 32 k .. 32 k + 31 of the 16 keys
          load_matrices(a, (key_at + st * CA_STAGE) ^ (k << 5));
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            if (k == 0) mma_s8_first(d[n], a, qb[n][0], qb[n][1]);
            else mma_s8(d[n], a, qb[n][2 * k], qb[n][2 * k + 1]);
          }
        }
        // keys g and g + 8
        const float* sk = ring_scale + st * 2 * CA_SUB + g;
        const float fk[2] = {sk[0], sk[8]};
        float fv[2] = {sk[CA_SUB], sk[CA_SUB + 8]};
        float2 s[NT][2];  // logits in base 2 of rows 2 t, 2 t + 1
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          s[n][0] = code_sums(d[n][0], d[n][1], __fmul2_rn(cr[n], both(fk[0])));
          s[n][1] = code_sums(d[n][2], d[n][3], __fmul2_rn(cr[n], both(fk[1])));
        }
        if (key0 + CA_SUB > clear || key0 + CA_SUB > keys) {
          // keys a row does not see; their scales may be anything, so nothing computed from them is kept
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int key = key0 + g + 8 * e;
            const int drafted = key - context;
            // a value scale that is no number stays with the rows that see it, through their logit
            const bool wild = !(fabsf(fv[e]) < INFINITY);
            if (wild || key >= keys) fv[e] = 0.0f;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const int row = 8 * n + 2 * t4 + y;
                const bool seen = key < keys && (key < row_lim[row] || (drafted >= 0 && drafted < 64 &&
                                                                        (row_bits[row] >> drafted & 1ull) != 0));
                float& logit = y ? s[n][e].y : s[n][e].x;
                if (!seen) logit = -INFINITY;
                else if (wild) logit = __uint_as_float(0x7FFFFFFFu);
              }
            }
          }
        }
        uint32_t pw[NT][2], rest[NT][2];  // weights in fp16, and for fp16 outputs what that rounding left
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float2 top = make_float2(fmaxf(s[n][0].x, s[n][1].x), fmaxf(s[n][0].y, s[n][1].y));
          // takes the references up to the largest logits
          auto rise = [&]() {
            const float2 most = row_max(top);
            // the sums stay as they are: their unit shrinks with the weights'
            const float2 now = make_float2(fmaxf(mx[n].x, most.x), fmaxf(mx[n].y, most.y));
            const float2 by = make_float2(ex2_approx(mx[n].x - now.x), ex2_approx(mx[n].y - now.y));
            l[n] = __fmul2_rn(l[n], by);
            inv[n].x *= ex2_approx(now.x - mx[n].x);
            inv[n].y *= ex2_approx(now.y - mx[n].y);
            mx[n] = now;
            // nothing that came before is left beside such a key
            const bool fresh_x = !(inv[n].x <= CA_UNSET), fresh_y = !(inv[n].y <= CA_UNSET);
            if (fresh_x) inv[n].x = CA_UNSET;
            if (fresh_y) inv[n].y = CA_UNSET;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              if (fresh_x) acc[n][i][0] = acc[n][i][2] = 0.0f;
              if (fresh_y) acc[n][i][1] = acc[n][i][3] = 0.0f;
            }
          };
          if (__any_sync(0xFFFFFFFFu, top.x > mx[n].x + CA_RISE || top.y > mx[n].y + CA_RISE)) rise();
          float2 pr[2], x[2], big;  // exponentials, weights p s_v and the largest of them
          auto weigh = [&]() {
            const float2 away = make_float2(-mx[n].x, -mx[n].y);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float2 y = __fadd2_rn(s[n][e], away);
              pr[e] = make_float2(ex2_approx(y.x), ex2_approx(y.y));
              x[e] = __fmul2_rn(pr[e], both(fv[e]));
            }
            big = make_float2(fmaxf(x[0].x, x[1].x), fmaxf(x[0].y, x[1].y));
          };
          weigh();
          if (__any_sync(0xFFFFFFFFu, big.x * inv[n].x > CA_MOST || big.y * inv[n].y > CA_MOST)) {
            // an exponential above 1 may take a weight out of float32, which is left by none up to 1
            if (__any_sync(0xFFFFFFFFu, big.x == INFINITY || big.y == INFINITY)) {
              rise();
              weigh();
            }
            big = row_max(big);
            const float2 to = make_float2(fminf(inv[n].x, weight_factor(big.x)), fminf(inv[n].y, weight_factor(big.y)));
            const float2 by = make_float2(to.x / inv[n].x, to.y / inv[n].y);
            inv[n] = to;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              acc[n][i][0] *= by.x;
              acc[n][i][1] *= by.y;
              acc[n][i][2] *= by.x;
              acc[n][i][3] *= by.y;
            }
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            l[n] = __fadd2_rn(l[n], pr[e]);
            const float2 w = __fmul2_rn(x[e], inv[n]);
            const __half2 h = __floats2half2_rn(w.x, w.y);
            pw[n][e] = transpose8(*reinterpret_cast<const uint32_t*>(&h));
            if (F16) {
              const float2 f = __half22float2(h);
              const __half2 h2 = __floats2half2_rn(w.x - f.x, w.y - f.y);
              rest[n][e] = transpose8(*reinterpret_cast<const uint32_t*>(&h2));
            }
          }
        }
        // values: channels 16 g .. 16 g + 15 of keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9
        uint4 w[4];
        w[0] = *reinterpret_cast<const uint4*>(value_at + st * CA_STAGE);
        w[1] = *reinterpret_cast<const uint4*>(value_at1 + st * CA_STAGE);
        w[2] = *reinterpret_cast<const uint4*>(value_at + st * CA_STAGE + 8 * CA_D);
        w[3] = *reinterpret_cast<const uint4*>(value_at1 + st * CA_STAGE + 8 * CA_D);
        const __half2 offset = __floats2half2_rn(1152.0f, 1152.0f);
#pragma unroll
        for (int q4 = 0; q4 < 4; ++q4) {
          uint32_t u[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            u[k] = (q4 == 0 ? w[k].x : q4 == 1 ? w[k].y : q4 == 2 ? w[k].z : w[k].w) ^ 0x80808080u;
#pragma unroll
          for (int pair = 0; pair < 2; ++pair) {
            // bytes of channels 4 q4 + 2 pair and + 1 of two keys, interleaved
            const uint32_t z[2] = {__byte_perm(u[0], u[1], pair ? 0x7362 : 0x5140),
                                   __byte_perm(u[2], u[3], pair ? 0x7362 : 0x5140)};
            uint32_t a[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              // fp16 of a code: the byte plus 128 in the low bits of 1024, minus 1152, exactly
              const uint32_t h = __byte_perm(z[e >> 1], 0x64646464u, e & 1 ? 0x4342 : 0x4140);
              const __half2 c = __hsub2(*reinterpret_cast<const __half2*>(&h), offset);
              a[e] = *reinterpret_cast<const uint32_t*>(&c);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              mma_f16(acc[n][2 * q4 + pair], a, pw[n][0], pw[n][1]);
              if (F16) mma_f16(acc[n][2 * q4 + pair], a, rest[n][0], rest[n][1]);
            }
          }
        }
      }
      __syncwarp();  // the stage has been read by every lane
      issue(t + ST, st, ahead);
      ahead = lookup(t + ST + 1);
      if (++st == ST) st = 0;
    }
    copy_wait<0>();

    // ---- the four warps joined through the idle ring: 2, 3 into 0, 1, then 1 into 0
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int m = 4; m < 32; m <<= 1) {
        l[n].x += __shfl_xor_sync(0xFFFFFFFFu, l[n].x, m);
        l[n].y += __shfl_xor_sync(0xFFFFFFFFu, l[n].y, m);
      }
      // the references taken up by the sums' exponents: the sums of values stay within twice the largest value
      const float2 now = make_float2(mx[n].x + sum_exponent(l[n].x), mx[n].y + sum_exponent(l[n].y));
      const float2 down = make_float2(ex2_approx(mx[n].x - now.x), ex2_approx(mx[n].y - now.y));
      mx[n] = now;
      l[n] = __fmul2_rn(l[n], down);
      const float2 by = make_float2(down.x / inv[n].x, down.y / inv[n].y);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        acc[n][i][0] *= by.x;
        acc[n][i][1] *= by.y;
        acc[n][i][2] *= by.x;
        acc[n][i][3] *= by.y;
      }
    }
    __syncthreads();
#pragma unroll
    for (int step = 2; step > 0; step >>= 1) {
      // warps 2 and 3 use areas 0 and 1; warp 1, which has then read area 1, uses it again
      if (warp >= step && warp < 2 * step) {
        float4* to = reinterpret_cast<float4*>(smem + (warp == 2 ? 0 : Shape::kJoinWarp));
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            to[(n * 8 + i) * 32 + lane] = make_float4(acc[n][i][0], acc[n][i][1], acc[n][i][2], acc[n][i][3]);
          to[NT * 256 + n * 32 + lane] = make_float4(mx[n].x, mx[n].y, l[n].x, l[n].y);
        }
      }
      __syncthreads();
      if (warp < step) {
        const float4* from =
            reinterpret_cast<const float4*>(smem + (step == 2 && warp == 0 ? 0 : Shape::kJoinWarp));
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float4 other = from[NT * 256 + n * 32 + lane];
          const float2 now = make_float2(fmaxf(mx[n].x, other.x), fmaxf(mx[n].y, other.y));
          const float2 fa = make_float2(ex2_approx(mx[n].x - now.x), ex2_approx(mx[n].y - now.y));
          const float2 fb = make_float2(ex2_approx(other.x - now.x), ex2_approx(other.y - now.y));
          mx[n] = now;
          l[n] = make_float2(l[n].x * fa.x + other.z * fb.x, l[n].y * fa.y + other.w * fb.y);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float4 o = from[(n * 8 + i) * 32 + lane];
            acc[n][i][0] = acc[n][i][0] * fa.x + o.x * fb.x;
            acc[n][i][1] = acc[n][i][1] * fa.y + o.y * fb.y;
            acc[n][i][2] = acc[n][i][2] * fa.x + o.z * fb.x;
            acc[n][i][3] = acc[n][i][3] * fa.y + o.w * fb.y;
          }
        }
      }
    }
    __syncthreads();  // the next run's copies write where these exchanges were
    const bool whole = r.t0 == 0 && r.t1 == walk.s.tiles;
    if (r.t0 == 0 && !whole) {
      // the piece ends inside an item that begins in it: it describes the item to the join
      cut.pieces = static_cast<int>((walk.end + r.left - 1) / per) - static_cast<int>(blockIdx.x) + 1;
      cut.rows = r.rows;
      cut.row0 = r.row0;
      cut.head = r.head;
      cut.token0 = walk.s.first;
    }
    if (warp == 0) {
      const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (r.t0 == 0 ? 1 : 0);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int row = 8 * n + 2 * t4 + y;
          const float sum = y ? l[n].y : l[n].x;
          float v[16];  // channels 16 g .. 16 g + 15
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            v[2 * i] = acc[n][i][y];
            v[2 * i + 1] = acc[n][i][2 + y];
          }
          if (whole) {
            const float norm = sum == 0.0f ? 0.0f : fwht::kInvSqrt128 / sum;
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] *= norm;
            fwht::reg_stage<16, 1>(v);
            fwht::reg_stage<16, 2>(v);
            fwht::reg_stage<16, 4>(v);
            fwht::reg_stage<16, 8>(v);
            fwht::lane_stage(v, 4, (g & 1) != 0);
            fwht::lane_stage(v, 8, (g & 2) != 0);
            fwht::lane_stage(v, 16, (g & 4) != 0);
            if (row < r.rows) {
              const int of = r.row0 + row, i = of / p.G;
              uint16_t* dst = p.o + (walk.s.first + i) * p.ot + (r.head * p.G + (of - i * p.G)) * p.oh + 16 * g;
#pragma unroll
              for (int c = 0; c < 2; ++c)
                *reinterpret_cast<uint4*>(dst + 8 * c) = make_uint4(
                    fwht::narrow_pair<F16>(v[8 * c], v[8 * c + 1]), fwht::narrow_pair<F16>(v[8 * c + 2], v[8 * c + 3]),
                    fwht::narrow_pair<F16>(v[8 * c + 4], v[8 * c + 5]),
                    fwht::narrow_pair<F16>(v[8 * c + 6], v[8 * c + 7]));
            }
          } else if (row < r.rows) {
            float4* dst = reinterpret_cast<float4*>(p.part + (slot * ROWS + row) * CA_D + 16 * g);
#pragma unroll
            for (int c = 0; c < 4; ++c) dst[c] = make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
            if (g == 0) p.part_ml[slot * ROWS + row] = make_float2(y ? mx[n].y : mx[n].x, sum);
          }
        }
      }
    }
  }
  if (tid == 0) p.cuts[blockIdx.x] = cut;
  bad = __syncthreads_or(bad);
  if (tid == 0) p.piece_status[blockIdx.x] = bad ? CA_BAD : 0;
}

// Joins the parts of the items that were cut: one CTA per piece, a warp per row of
// the item that begins in the piece (and goes on in the next ones), four channels
// per lane.
constexpr int kJoinWarps = 8;
constexpr int kJoinAhead = 8;  // parts whose loads a lane has in flight
constexpr int kWideAhead = 4;
// The weight of a part at the row's maximum: the sum of all pieces' parts stays within one part's range.
constexpr float kJoinUnit = 0x1p-12f;

// The call's status from the pieces' (by the first CTA).
__device__ __forceinline__ void join_status(const CaParams& p) {
  if (blockIdx.x == 0 && blockIdx.y == 0) {
    int st = 0;
    for (int i = threadIdx.x; i < p.workers; i += 32 * kJoinWarps) st |= p.piece_status[i];
    const int any_bad = __syncthreads_or(st & CA_BAD), late = __syncthreads_or(st & 4);  // a timeout is 5
    if (threadIdx.x == 0) {
      const int all = late ? CA_LATE : any_bad ? CA_BAD : 0;
      *p.status = all;
      if (all != 0 && p.told != nullptr) atomicOr(p.told, all);
    }
  }
}

// The rotation of a row's mean and its rounding, four channels a lane.
template <bool F16>
__device__ __forceinline__ void join_out(const CaParams& p, const CaCut& cut, int row, float (&v)[4], int lane) {
  fwht::fwht128_warp(v, lane);
  const int of = cut.row0 + row, i = of / p.G;
  uint16_t* dst = p.o + (cut.token0 + i) * p.ot + (cut.head * p.G + (of - i * p.G)) * p.oh + 4 * lane;
  *reinterpret_cast<uint2*>(dst) = make_uint2(fwht::narrow_pair<F16>(v[0], v[1]), fwht::narrow_pair<F16>(v[2], v[3]));
}

template <bool F16>
__global__ void __launch_bounds__(32 * kJoinWarps) cache_attention_join_kernel(const CaParams p, int rows) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  griddep_wait();
  join_status(p);
  const CaCut cut = p.cuts[blockIdx.x];
  if (cut.pieces < 1) return;
  // part 0 of the item is slot 2 c + 1, the k-th after it slot 2 (c + k)
  auto slot = [&](int k) { return 2 * (static_cast<int>(blockIdx.x) + k) + (k == 0 ? 1 : 0); };
  for (int row = blockIdx.y * kJoinWarps + warp; row < cut.rows; row += kJoinWarps * gridDim.y) {
    auto load = [&](int k) {
      return k < cut.pieces ? *reinterpret_cast<const float4*>(
                                  p.part + (static_cast<int64_t>(slot(k)) * rows + row) * CA_D + 4 * lane)
                            : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    };
    auto statistic = [&](int k) {
      return k < cut.pieces ? p.part_ml[slot(k) * rows + row] : make_float2(CA_NONE, 0.0f);
    };
    // the first parts are under way before their weights are known
    const float2 first = statistic(lane);
    float4 o[kJoinAhead];
#pragma unroll
    for (int j = 0; j < kJoinAhead; ++j) o[j] = load(j);
    float top = first.x;
    for (int k = lane + 32; k < cut.pieces; k += 32) top = fmaxf(top, statistic(k).x);
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, m));
    float sum = 0.0f;
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int k0 = 0; k0 < cut.pieces; k0 += 32) {
      const int here = cut.pieces - k0 < 32 ? cut.pieces - k0 : 32;
      const float2 ml = k0 == 0 ? first : statistic(k0 + lane);
      const float weight = ex2_approx(ml.x - top) * kJoinUnit;
      sum += weight * ml.y;  // a statistic of no part: 0
      for (int j0 = 0; j0 < here; j0 += kJoinAhead) {
#pragma unroll
        for (int j = 0; j < kJoinAhead; ++j) {
          const float w = __shfl_sync(0xFFFFFFFFu, weight, (j0 + j) & 31);
          v[0] = fmaf(w, o[j].x, v[0]), v[1] = fmaf(w, o[j].y, v[1]);
          v[2] = fmaf(w, o[j].z, v[2]), v[3] = fmaf(w, o[j].w, v[3]);
        }
#pragma unroll
        for (int j = 0; j < kJoinAhead; ++j) o[j] = load(k0 + j0 + kJoinAhead + j);
      }
    }
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, m);
    const float norm = sum == 0.0f ? 0.0f : fwht::kInvSqrt128 / sum;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] *= norm;
    join_out<F16>(p, cut, row, v, lane);
  }
}

// The same for tiles of 128 rows, whose parts lie four channels of all rows after one
// another: eight rows a CTA, a row and four channels a thread, so that eight lanes
// read a line; then a warp per row as above.
template <bool F16>
__global__ void __launch_bounds__(32 * kJoinWarps) cache_attention_join_wide_kernel(const CaParams p) {
  __shared__ float sums[kJoinWarps][CA_D + 4];
  __shared__ float norms[kJoinWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  griddep_wait();
  join_status(p);
  const CaCut cut = p.cuts[blockIdx.x];
  const int row0 = blockIdx.y * kJoinWarps;
  if (row0 >= (cut.pieces < 1 ? 0 : cut.rows)) return;
  {
    const int r = tid & (kJoinWarps - 1), c = tid / kJoinWarps;  // c of 32
    const int row = row0 + r < cut.rows ? row0 + r : cut.rows - 1;
    auto slot = [&](int k) { return 2 * (static_cast<int>(blockIdx.x) + k) + (k == 0 ? 1 : 0); };
    // parts in fours, the next four under way while these are added
    float4 o[kWideAhead];
    float2 ml[kWideAhead];
    auto load = [&](int k0) {
#pragma unroll
      for (int i = 0; i < kWideAhead; ++i) {
        const int k = k0 + i;
        o[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        ml[i] = make_float2(CA_NONE, 0.0f);
        if (k < cut.pieces) {
          o[i] = reinterpret_cast<const float4*>(p.part)[(static_cast<int64_t>(slot(k)) * (CA_D / 4) + c) * CA_WIDE_ROWS + row];
          ml[i] = p.part_ml[slot(k) * CA_WIDE_ROWS + row];
        }
      }
    };
    load(0);
    float top = CA_NONE, sum = 0.0f;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int k0 = 0; k0 < cut.pieces; k0 += kWideAhead) {
      float4 x[kWideAhead];
      float2 st[kWideAhead];
#pragma unroll
      for (int i = 0; i < kWideAhead; ++i) x[i] = o[i], st[i] = ml[i];
      load(k0 + kWideAhead);
      float most = top;
#pragma unroll
      for (int i = 0; i < kWideAhead; ++i) most = fmaxf(most, st[i].x);
      // a part's sum of exponentials reaches 2^110: its factor in two halves, where one is lost below 2^-126
      const float h = ex2_approx(0.5f * (top - most)), f = h * h;
      top = most;
      sum = sum * h * h;
      v.x *= f, v.y *= f, v.z *= f, v.w *= f;
#pragma unroll
      for (int i = 0; i < kWideAhead; ++i) {
        const float half = ex2_approx(0.5f * (st[i].x - top)), w = half * half;  // of no part: no sum, no values
        sum = fmaf(half * st[i].y, half, sum);
        v.x = fmaf(w, x[i].x, v.x), v.y = fmaf(w, x[i].y, v.y), v.z = fmaf(w, x[i].z, v.z), v.w = fmaf(w, x[i].w, v.w);
      }
    }
    *reinterpret_cast<float4*>(&sums[r][4 * c]) = v;
    if (c == 0) norms[r] = sum == 0.0f ? 0.0f : fwht::kInvSqrt128 / sum;
  }
  __syncthreads();
  const int row = row0 + warp;
  if (row >= cut.rows) return;
  const float4 s = *reinterpret_cast<const float4*>(&sums[warp][4 * lane]);
  const float norm = norms[warp];
  float v[4] = {s.x * norm, s.y * norm, s.z * norm, s.w * norm};
  join_out<F16>(p, cut, row, v, lane);
}

// ------------------------------------------------------------------------ host

struct CaLayout {
  size_t status, cuts, ml, part, total;
};

CaLayout ca_layout(int rows) {
  const size_t workers = rows == CA_WIDE_ROWS ? CA_WIDE_WORKERS : CA_MAX_WORKERS;
  CaLayout w;
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  w.status = 256;
  w.cuts = up(w.status + workers * sizeof(int));
  w.ml = up(w.cuts + workers * sizeof(CaCut));
  w.part = up(w.ml + 2 * workers * rows * sizeof(float2));
  w.total = up(w.part + 2 * workers * rows * CA_D * sizeof(float));
  return w;
}

// The tile of rows by the mean number of rows a sequence has for a key head. A taller tile reads the keys for
// fewer tiles, a lower one wastes fewer of its rows. Tiles of 16 rows against 128, 8 sequences and 8 key heads, bf16
// outputs: behind 4096 keys 36 rows each 50 against 49 us, 48 rows 50 against 51, 64 rows 63 against 51, 96 rows 86
// against 56; behind 512 keys 36 rows 22 against 25, 64 rows 26 against 27, 96 rows 32 against 28; behind 16384 36 rows
// 149 against 141, 64 rows 202 against 144. fp16 outputs: behind 4096 36 rows 55 against 60, 64 rows 69 against 62; behind
// 16384 36 rows 176 against 169, 64 rows 240 against 173.
int ca_rows(int64_t T, int64_t B, int64_t G) { return T * G <= 8 * B ? 8 : T * G <= 32 * B ? 16 : CA_WIDE_ROWS; }

bool ca_sizes_ok(int64_t T, int64_t B, int64_t Hq, int64_t Hkv, int64_t D) {
  return D == CA_D && T >= 0 && B >= 0 && Hkv >= 1 && Hq >= Hkv && Hq % Hkv == 0 && Hkv <= CONVROT_MAX_CACHE_HEADS &&
         Hq / Hkv <= CONVROT_MAX_CACHE_HEADS && B <= (int64_t{1} << 24) && T <= (int64_t{1} << 20);
}

template <class Shape, bool F16>
cudaError_t ca_launch(const CaParams& p, int dev, cudaStream_t s) {
  static std::atomic<int> ready[64];  // devices whose attribute is set
  const bool known = dev >= 0 && dev < 64;
  if (!known || ready[dev].load(std::memory_order_acquire) == 0) {
    const cudaError_t e = cudaFuncSetAttribute(cache_attention_kernel<Shape, F16>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, Shape::kBytes);
    if (e != cudaSuccess) return e;
    if (known) ready[dev].store(1, std::memory_order_release);
  }
  cache_attention_kernel<Shape, F16><<<p.workers, CA_THREADS, Shape::kBytes, s>>>(p);
  return cudaGetLastError();
}

cudaError_t ca_run(CaParams p, int rows, bool f16, int64_t cells, uint8_t* ws, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int most = rows == CA_WIDE_ROWS ? CA_WIDE_WORKERS : CA_MAX_WORKERS;
  const int want = sms * (rows == 8 ? Shape8::kOcc : rows == 16 ? Shape16::kOcc : 1);
  const CaLayout lay = ca_layout(rows);
  p.workers = want < most ? want : most;
  p.status = reinterpret_cast<int*>(ws);
  p.piece_status = reinterpret_cast<int*>(ws + lay.status);
  p.cuts = reinterpret_cast<CaCut*>(ws + lay.cuts);
  p.part_ml = reinterpret_cast<float2*>(ws + lay.ml);
  p.part = reinterpret_cast<float*>(ws + lay.part);
  if (rows == 8) e = f16 ? ca_launch<Shape8, true>(p, dev, s) : ca_launch<Shape8, false>(p, dev, s);
  else if (rows == 16) e = f16 ? ca_launch<Shape16, true>(p, dev, s) : ca_launch<Shape16, false>(p, dev, s);
  else e = launch_cache_attention_wide(p, f16, cells, s);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(p.workers, (rows + kJoinWarps - 1) / kJoinWarps);
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (rows == CA_WIDE_ROWS)
    return f16 ? cudaLaunchKernelEx(&cfg, cache_attention_join_wide_kernel<true>, p)
               : cudaLaunchKernelEx(&cfg, cache_attention_join_wide_kernel<false>, p);
  return f16 ? cudaLaunchKernelEx(&cfg, cache_attention_join_kernel<true>, p, rows)
             : cudaLaunchKernelEx(&cfg, cache_attention_join_kernel<false>, p, rows);
}

}  // namespace

}  // namespace convrot

extern "C" {

size_t convrot_cache_attention_workspace_bytes(int64_t T, int64_t B, int64_t Hq, int64_t Hkv, int64_t D) {
  using namespace convrot;
  if (!ca_sizes_ok(T, B, Hq, Hkv, D)) return 0;
  if (T == 0 || B == 0) return 256;
  return ca_layout(ca_rows(T, B, Hq / Hkv)).total;
}

convrot_status convrot_cache_attention(const convrot_cache_attention_args* args, convrot_stream_t stream) {
  return convrot_cache_attention_ex(args, nullptr, 0, stream);
}

convrot_status convrot_cache_attention_ex(const convrot_cache_attention_args* args, int* status, int64_t wait_ns,
                                          convrot_stream_t stream) {
  using namespace convrot;
  if (args == nullptr || wait_ns < 0 || reinterpret_cast<uintptr_t>(status) % alignof(int) != 0)
    return CONVROT_ERR_INVALID_ARG;
  const convrot_cache_attention_args& a = *args;
  const convrot_cells& c = a.cells;
  if (a.dtype != CONVROT_DTYPE_BF16 && a.dtype != CONVROT_DTYPE_F16) return CONVROT_ERR_UNSUPPORTED;
  if (c.D != CA_D) return CONVROT_ERR_UNSUPPORTED;
  if (a.T < 0 || a.B < 0 || c.H < 1 || a.Hq < 1 || a.Hq % c.H != 0 || c.num_pages < 1 || c.page_size < 1 ||
      a.table_pages < 0)
    return CONVROT_ERR_INVALID_ARG;
  if (c.page_size < CONVROT_MIN_PAGE || c.page_size > CONVROT_MAX_PAGE || (c.page_size & (c.page_size - 1)) != 0)
    return CONVROT_ERR_UNSUPPORTED;
  if (!ca_sizes_ok(a.T, a.B, a.Hq, c.H, c.D) || c.num_pages > 0x7FFFFFFF / c.page_size / c.H ||
      a.table_pages > 0x7FFFF000 / c.page_size)
    return CONVROT_ERR_UNSUPPORTED;
  if (a.starts == nullptr && a.T != a.B) return CONVROT_ERR_INVALID_ARG;
  const float c_scale = a.softmax_scale * 1.4426950408889634f;
  if (!(a.softmax_scale > 0.0f) || !(c_scale < INFINITY)) return CONVROT_ERR_INVALID_ARG;
  auto stride = [](int64_t n, int64_t st) { return n > 1 ? st : 0; };
  CaParams p{};
  p.qt = stride(a.T, a.q_token), p.qh = stride(a.Hq, a.q_head);
  p.ot = stride(a.T, a.o_token), p.oh = stride(a.Hq, a.o_head);
  p.table_stride = stride(a.B, a.table_stride);
  if ((p.qt | p.qh | p.ot | p.oh) % 8 != 0 || p.table_stride < 0) return CONVROT_ERR_INVALID_ARG;
  if (a.T == 0) return CONVROT_OK;  // no queries
  auto aligned = [](const void* ptr, uintptr_t to) { return (reinterpret_cast<uintptr_t>(ptr) % to) == 0; };
  const bool room = a.ws != nullptr && aligned(a.ws, 256) &&
                    a.ws_bytes >= convrot_cache_attention_workspace_bytes(a.T, a.B, a.Hq, c.H, c.D);
  if (a.B == 0) {  // queries of no sequence: a clean status word is all there is to do
    if (!room) return CONVROT_ERR_WORKSPACE;
    return cudaMemsetAsync(a.ws, 0, sizeof(int), reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? CONVROT_OK
                                                                                                         : CONVROT_ERR_CUDA;
  }
  for (const void* ptr : {a.Q, static_cast<const void*>(a.O), static_cast<const void*>(c.k_codes),
                          static_cast<const void*>(c.v_codes), static_cast<const void*>(c.k_scale),
                          static_cast<const void*>(c.v_scale)})
    if (ptr == nullptr || !aligned(ptr, 16)) return CONVROT_ERR_INVALID_ARG;
  if (a.lengths == nullptr || (a.pages == nullptr && a.table_pages > 0) || !aligned(a.pages, 4) ||
      !aligned(a.lengths, 4) || !aligned(a.starts, 4) || !aligned(a.tree, 8))
    return CONVROT_ERR_INVALID_ARG;
  if (!room) return CONVROT_ERR_WORKSPACE;
  p.q = static_cast<const uint16_t*>(a.Q);
  p.o = static_cast<uint16_t*>(a.O);
  p.k_codes = c.k_codes;
  p.v_codes = c.v_codes;
  p.k_scale = c.k_scale;
  p.v_scale = c.v_scale;
  p.pages = a.pages;
  p.lengths = a.lengths;
  p.starts = a.starts;
  p.tree = reinterpret_cast<const unsigned long long*>(a.tree);
  p.T = static_cast<int>(a.T);
  p.B = static_cast<int>(a.B);
  p.Hkv = static_cast<int>(c.H);
  p.G = static_cast<int>(a.Hq / c.H);
  p.table_pages = static_cast<int>(a.table_pages);
  p.num_pages = static_cast<int>(c.num_pages);
  while ((int64_t{1} << p.page_shift) < c.page_size) ++p.page_shift;
  p.c_scale = c_scale;
  p.told = status;
  p.wait_ns = wait_ns > 0 ? static_cast<uint64_t>(wait_ns) : CA_WAIT_NS;
  p.wait_step = p.wait_ns < 2000 ? static_cast<uint32_t>(p.wait_ns) : 2000;
  const cudaError_t e = ca_run(p, ca_rows(a.T, a.B, p.G), a.dtype == CONVROT_DTYPE_F16, c.num_pages * c.H * c.page_size,
                               static_cast<uint8_t*>(a.ws), reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? CONVROT_OK : CONVROT_ERR_CUDA;
}

}  // extern "C"
