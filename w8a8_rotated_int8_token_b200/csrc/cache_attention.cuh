// What the two kernels of the attention over the rotated int8 cache share: the
// arguments, the line of work that is cut into one piece per CTA, and what a cut
// item leaves for the join.
#pragma once

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "convrot.h"
#include "fwht_dev.cuh"

namespace convrot {

constexpr int CA_D = 128;
constexpr int CA_BAD = CONVROT_ERR_INVALID_ARG;
constexpr int CA_LATE = CONVROT_ERR_DEVICE_TIMEOUT;
constexpr uint64_t CA_WAIT_NS = 2000000000ull;  // limit of a wait, unless the caller sets one
constexpr int CA_MAX_WORKERS = 640;  // pieces the workspace has room for
// The maximum of a row that has seen no key: below every other logit, and finite, so that exponents of
// differences need no special case.
constexpr float CA_NONE = -3.402823466e38f;

// What a piece leaves for the join: its last item, if that goes on in the next pieces.
struct CaCut {
  int pieces;       // pieces that hold a part of the item (0: nothing to join)
  int rows;         // rows of the tile
  int row0;         // first row of the tile in the sequence's rows
  int head;         // key head
  int token0;       // first query token of the sequence
  int pad[3];
};

struct CaParams {
  const uint16_t* q;
  uint16_t* o;
  int64_t qt, qh, ot, oh;
  const int8_t* k_codes;
  const int8_t* v_codes;
  const float* k_scale;
  const float* v_scale;
  const int32_t* pages;
  const int32_t* lengths;
  const int32_t* starts;      // null: token b belongs to sequence b
  const unsigned long long* tree;  // null: causal
  int64_t table_stride;
  int T, B, Hkv, G, table_pages, num_pages, page_shift;
  float c_scale;              // softmax_scale log2(e)
  int* piece_status;          // [workers]
  CaCut* cuts;                // [workers]
  float* part;                // [2 workers][rows][128]
  float2* part_ml;            // [2 workers][rows] maximum, sum
  int* status;                // the call's status word, written by the join
  int* told;                  // null, or a word that it is ORed into as well
  uint64_t wait_ns;           // limit of a wait
  uint32_t wait_step;         // nanoseconds between two looks at it
  int workers;
};

// What turns a row's integer products into logits in base 2, from the largest magnitude of the rotated query. A channel
// that is NaN or infinite leaves no other in its vector finite, and no code stands for such a vector: NaN, and so
// are the logits of the keys that the row sees.
__device__ __forceinline__ float ca_query_factor(const CaParams& p, float amax) {
  return amax < INFINITY ? fwht::scale_of<128>(amax) * p.c_scale : __uint_as_float(0x7FFFFFFFu);
}

// How a kernel cuts the work: rows and keys of a tile, and in units of one tile what a run costs beside its
// tiles (queries, first loads, the join) and the least that a piece takes.
template <int ROWS, int KEYS, int SETUP, int LEAST>
struct CaGrain {
  static constexpr int kRows = ROWS, kKeys = KEYS, kSetup = SETUP, kLeast = LEAST;
};

// A sequence: its keys, its query tokens, and its share of the line of work. An item is kSetup units and one for each
// key tile; without keys one unit, in which its rows are zeroed.
struct CaSeq {
  int keys, first, news;
  int tiles, span;  // key tiles and units of an item
  int64_t count;    // units of all its items
};

template <class Grain>
__device__ __forceinline__ CaSeq ca_seq(const CaParams& p, int b, int& bad) {
  CaSeq s;
  const int64_t room = static_cast<int64_t>(p.table_pages) << p.page_shift;
  int keys = __ldg(p.lengths + b), lo = b, hi = b + 1;
  if (p.starts != nullptr) lo = __ldg(p.starts + b), hi = __ldg(p.starts + b + 1);
  if (keys < 0 || keys > room || lo < 0 || hi < lo || hi > p.T) bad |= CA_BAD;
  keys = keys < 0 ? 0 : keys > room ? static_cast<int>(room) : keys;
  lo = lo < 0 ? 0 : lo > p.T ? p.T : lo;
  hi = hi < lo ? lo : hi > p.T ? p.T : hi;
  s.keys = keys;
  s.first = lo;
  s.news = hi - lo;
  s.tiles = static_cast<int>((static_cast<uint32_t>(keys) + Grain::kKeys - 1) / Grain::kKeys);
  s.span = s.tiles > 0 ? s.tiles + Grain::kSetup : 1;
  const uint32_t tall = (static_cast<uint32_t>(s.news) * static_cast<uint32_t>(p.G) + Grain::kRows - 1) / Grain::kRows;
  // rows of all heads are fewer than 2^32: the output would not fit otherwise
  s.count = static_cast<int64_t>(tall * static_cast<uint32_t>(p.Hkv)) * s.span;
  return s;
}

// A run of one item's tiles within a piece.
struct CaRun {
  int head, row0, rows, t0, t1;
  int left;  // units of the item behind the run
};

// Walks a piece: the runs from `pos` to `end`, the same for every warp.
template <class Grain>
struct CaWalk {
  int64_t pos, end, base;
  int b;
  CaSeq s;
  __device__ __forceinline__ bool next(const CaParams& p, CaRun* r, int& bad) {
    while (pos < end) {
      while (pos >= base + s.count) {
        base += s.count;
        ++b;
        s = ca_seq<Grain>(p, b, bad);  // pos < total, so a sequence with work follows
      }
      const int64_t rel = pos - base;
      int64_t item;
      if (rel < (int64_t{1} << 32)) item = static_cast<uint32_t>(rel) / static_cast<uint32_t>(s.span);
      else item = rel / s.span;
      const int u0 = static_cast<int>(rel - item * s.span);
      const int take = end - pos < s.span - u0 ? static_cast<int>(end - pos) : s.span - u0;
      pos += take;
      const int setup = s.tiles > 0 ? Grain::kSetup : 0;
      r->t0 = u0 > setup ? u0 - setup : 0;
      r->t1 = u0 + take > setup ? u0 + take - setup : 0;
      if (r->t1 <= r->t0) continue;  // the piece ends before the item's first tile
      r->left = s.span - u0 - take;
      const uint32_t tall = static_cast<uint32_t>(item) / static_cast<uint32_t>(p.Hkv);  // items of a sequence < 2^32
      r->head = static_cast<int>(static_cast<uint32_t>(item) - tall * p.Hkv);
      r->row0 = static_cast<int>(tall * Grain::kRows);
      const int rows = s.news * p.G - r->row0;
      r->rows = rows < Grain::kRows ? rows : Grain::kRows;
      return true;
    }
    return false;
  }
};

// The piece of this CTA: all units summed over the sequences, then the sequence the piece starts in. Every
// thread of the CTA calls it; `scan` is shared memory for a sum per warp and two values more. Returns the units
// of a piece.
template <class Grain, int THREADS>
__device__ __forceinline__ int64_t ca_piece(const CaParams& p, int64_t* scan, CaWalk<Grain>* walk, int& bad) {
  constexpr int WARPS = THREADS / 32;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (p.B <= 32) {  // every warp finds it by itself
    const CaSeq s = ca_seq<Grain>(p, lane < p.B ? lane : p.B - 1, bad);
    const int64_t count = lane < p.B ? s.count : 0;
    int64_t incl = count;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const int64_t other = __shfl_up_sync(0xFFFFFFFFu, incl, m);
      if (lane >= m) incl += other;
    }
    const int64_t total = __shfl_sync(0xFFFFFFFFu, incl, 31);
    int64_t per = (total + gridDim.x - 1) / gridDim.x;
    if (per < Grain::kLeast) per = Grain::kLeast;
    walk->pos = blockIdx.x * per;
    walk->end = walk->pos + per < total ? walk->pos + per : total;
    if (walk->pos < total) {
      const uint32_t past = __ballot_sync(0xFFFFFFFFu, incl > walk->pos);
      walk->b = __ffs(past) - 1;
      walk->base = __shfl_sync(0xFFFFFFFFu, incl - count, walk->b);
      walk->s.keys = __shfl_sync(0xFFFFFFFFu, s.keys, walk->b);
      walk->s.first = __shfl_sync(0xFFFFFFFFu, s.first, walk->b);
      walk->s.news = __shfl_sync(0xFFFFFFFFu, s.news, walk->b);
      walk->s.tiles = __shfl_sync(0xFFFFFFFFu, s.tiles, walk->b);
      walk->s.span = __shfl_sync(0xFFFFFFFFu, s.span, walk->b);
      walk->s.count = __shfl_sync(0xFFFFFFFFu, s.count, walk->b);
    }
    return per;
  }
  int64_t mine = 0, sum = 0;
  for (int b = tid; b < p.B; b += THREADS) {
    const int64_t count = ca_seq<Grain>(p, b, bad).count;
    if (b == tid) mine = count;
    sum += count;
  }
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, m);
  if (lane == 0) scan[warp] = sum;
  __syncthreads();
  int64_t total = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) total += scan[w];
  int64_t per = (total + gridDim.x - 1) / gridDim.x;
  if (per < Grain::kLeast) per = Grain::kLeast;
  walk->pos = blockIdx.x * per;
  walk->end = walk->pos + per < total ? walk->pos + per : total;
  if (walk->pos < total) {
    int64_t before = 0;
    for (int b0 = 0; b0 < p.B; b0 += THREADS) {
      const int b = b0 + tid;
      int64_t count = mine;
      if (b0 > 0) count = b < p.B ? ca_seq<Grain>(p, b, bad).count : 0;
      int64_t incl = count;
#pragma unroll
      for (int m = 1; m < 32; m <<= 1) {
        const int64_t other = __shfl_up_sync(0xFFFFFFFFu, incl, m);
        if (lane >= m) incl += other;
      }
      __syncthreads();  // the sums before have been read
      if (lane == 31) scan[warp] = incl;
      __syncthreads();
      int64_t lo = before + incl - count;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        if (w < warp) lo += scan[w];
        before += scan[w];
      }
      if (lo <= walk->pos && walk->pos < lo + count) {
        scan[WARPS] = b;
        scan[WARPS + 1] = lo;
      }
      if (walk->pos < before) break;  // the same for every thread
    }
    __syncthreads();
    walk->b = static_cast<int>(scan[WARPS]);
    walk->base = scan[WARPS + 1];
    walk->s = ca_seq<Grain>(p, walk->b, bad);
  }
  return per;
}

// The kernel for many rows (cache_attention_wide.cu), its rows of a tile and its pieces on a device of `sms` SMs.
constexpr int CA_WIDE_ROWS = 128;
constexpr int CA_WIDE_WORKERS = 160;
cudaError_t launch_cache_attention_wide(const CaParams& p, bool f16, int64_t cells, cudaStream_t stream);

}  // namespace convrot
