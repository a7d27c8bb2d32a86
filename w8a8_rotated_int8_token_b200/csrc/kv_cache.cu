// The rotated int8 key/value cache: written (convrot_cache_append) and read
// back (convrot_cache_read).
//
// A cell is one token of one head: 128 int8 codes c = rne(x R / s) and one
// float32 scale s = absmax(x R) / 127, R = H_128 / sqrt(128): the linear layer's
// per-token rule over a head vector, to the same bits as convrot_quant_act with
// g = 128. Reading gives (c s) R, since R is its own inverse.
//
// Bound by memory: 256 bytes on the dense side and 132 in the cell per vector.
// Four lanes share a vector, 32 channels each: five of the seven butterfly
// stages stay in registers and two cross lanes (64 shuffles a lane; with 16
// lanes a vector it would be twice the shuffles per vector), and every access
// is 16 bytes a lane on the dense side with 64-byte runs per vector.

#include <cuda_runtime.h>

#include <cstdint>
#include <initializer_list>

#include "convrot.h"
#include "fwht128.cuh"
#include "fwht_dev.cuh"

namespace convrot {

namespace {

constexpr int kCellThreads = 128;
constexpr int kCellDim = 128;
constexpr int kBadSlot = CONVROT_ERR_INVALID_ARG;

struct CellParams {
  uint16_t* k;               // dense keys and values, [T, H, 128] with strides
  uint16_t* v;
  int64_t kt, kh, vt, vh;
  const int32_t* slots;
  int8_t* k_codes;           // [P, H, page, 128]
  int8_t* v_codes;
  float* k_scale;            // [P, H, page]
  float* v_scale;
  int64_t vectors;           // 2 T H
  int H, page_shift;
  int capacity;              // P * page
  int* status;
};

// The vector of a thread: token t, head h, keys or values; its cell, or -1.
struct CellPlace {
  int64_t t;
  int h;
  bool value;
  int64_t cell;
};

__device__ __forceinline__ CellPlace cell_place(const CellParams& p, int64_t vec) {
  CellPlace c;
  const uint32_t two_h = 2u * static_cast<uint32_t>(p.H);
  const uint32_t t = static_cast<uint32_t>(vec) / two_h;  // vectors < 2^31
  const uint32_t rest = static_cast<uint32_t>(vec) - t * two_h;
  c.t = t;
  c.value = rest >= static_cast<uint32_t>(p.H);
  c.h = static_cast<int>(c.value ? rest - p.H : rest);
  const int slot = __ldg(p.slots + t);
  c.cell = -1;
  if (slot >= 0 && slot < p.capacity) {
    const int page = slot >> p.page_shift, off = slot & ((1 << p.page_shift) - 1);
    c.cell = ((static_cast<int64_t>(page) * p.H + c.h) << p.page_shift) + off;
  } else if (slot >= p.capacity && p.status != nullptr) {
    atomicOr(p.status, kBadSlot);
  }
  return c;
}

template <bool F16>
__global__ void __launch_bounds__(kCellThreads) cache_append_kernel(const CellParams p) {
  const int64_t vec = (static_cast<int64_t>(blockIdx.x) * kCellThreads + threadIdx.x) >> 2;
  const int l = threadIdx.x & 3;
  const bool there = vec < p.vectors;
  CellPlace c{};
  c.cell = -1;
  float v[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = 0.0f;
  if (there) {
    c = cell_place(p, vec);
    const uint16_t* src = c.value ? p.v + c.t * p.vt + c.h * p.vh : p.k + c.t * p.kt + c.h * p.kh;
    uint4 w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = __ldg(reinterpret_cast<const uint4*>(src + 32 * j + 8 * l));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t* u = reinterpret_cast<const uint32_t*>(&w[j]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = fwht::widen_pair<F16>(u[e]);
        v[8 * j + 2 * e] = f.x;
        v[8 * j + 2 * e + 1] = f.y;
      }
    }
  }
  fwht::fwht128_quad(v, l);
  float m[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    m[i] = fwht::fmax3f(fabsf(v[4 * i]), fabsf(v[4 * i + 1]), fmaxf(fabsf(v[4 * i + 2]), fabsf(v[4 * i + 3])));
  float amax = fwht::fmax3f(fwht::fmax3f(m[0], m[1], m[2]), fwht::fmax3f(m[3], m[4], m[5]), fmaxf(m[6], m[7]));
  amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
  if (c.cell < 0) return;
  const fwht::CodeFactor f = fwht::code_factor(amax);
  int8_t* dst = (c.value ? p.v_codes : p.k_codes) + c.cell * kCellDim;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float r[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = fmaf(v[8 * j + e] * f.pre, f.ci, fwht::kRoundMagic);
    *reinterpret_cast<uint2*>(dst + 32 * j + 8 * l) =
        make_uint2(fwht::pack4(r[0], r[1], r[2], r[3]), fwht::pack4(r[4], r[5], r[6], r[7]));
  }
  if (l == 0) (c.value ? p.v_scale : p.k_scale)[c.cell] = fwht::scale_of<128>(amax);
}

template <bool F16>
__global__ void __launch_bounds__(kCellThreads) cache_read_kernel(const CellParams p) {
  const int64_t vec = (static_cast<int64_t>(blockIdx.x) * kCellThreads + threadIdx.x) >> 2;
  const int l = threadIdx.x & 3;
  const bool there = vec < p.vectors;
  CellPlace c{};
  c.cell = -1;
  if (there) c = cell_place(p, vec);
  float v[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = 0.0f;
  float scale = 0.0f;
  if (c.cell >= 0) {
    const int8_t* src = (c.value ? p.v_codes : p.k_codes) + c.cell * kCellDim;
    scale = __ldg((c.value ? p.v_scale : p.k_scale) + c.cell) * fwht::kInvSqrt128;
    uint2 w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = __ldg(reinterpret_cast<const uint2*>(src + 32 * j + 8 * l));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        // float of a signed byte: the byte plus 128 in the low bits of 2^23, exactly
        const uint32_t u = (e < 4 ? w[j].x : w[j].y) ^ 0x80808080u;
        v[8 * j + e] = __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440 + (e & 3))) - 8388736.0f;
      }
    }
  }
  fwht::fwht128_quad(v, l);  // sums of 128 codes: exact in float32
  if (!there) return;
  uint16_t* dst = c.value ? p.v + c.t * p.vt + c.h * p.vh : p.k + c.t * p.kt + c.h * p.kh;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint4 o;
    uint32_t* u = reinterpret_cast<uint32_t*>(&o);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      u[e] = c.cell < 0 ? 0u : fwht::narrow_pair<F16>(v[8 * j + 2 * e] * scale, v[8 * j + 2 * e + 1] * scale);
    *reinterpret_cast<uint4*>(dst + 32 * j + 8 * l) = o;
  }
}

bool aligned_to(const void* ptr, uintptr_t a) { return (reinterpret_cast<uintptr_t>(ptr) % a) == 0; }

// The checks both directions share; CONVROT_OK with p filled in, or an error.
convrot_status cell_params(const convrot_cache_args* args, CellParams* p) {
  if (args == nullptr) return CONVROT_ERR_INVALID_ARG;
  const convrot_cache_args& a = *args;
  const convrot_cells& c = a.cells;
  if (a.dtype != CONVROT_DTYPE_BF16 && a.dtype != CONVROT_DTYPE_F16) return CONVROT_ERR_UNSUPPORTED;
  if (c.D != kCellDim) return CONVROT_ERR_UNSUPPORTED;
  if (a.T < 0 || c.H < 1 || c.num_pages < 1 || c.page_size < 1) return CONVROT_ERR_INVALID_ARG;
  if (c.page_size < CONVROT_MIN_PAGE || c.page_size > CONVROT_MAX_PAGE || (c.page_size & (c.page_size - 1)) != 0)
    return CONVROT_ERR_UNSUPPORTED;
  if (c.H > CONVROT_MAX_CACHE_HEADS || c.num_pages > 0x7FFFFFFF / c.page_size || a.T > 0x3FFFFFFF / c.H)
    return CONVROT_ERR_UNSUPPORTED;
  auto stride = [](int64_t n, int64_t st) { return n > 1 ? st : 0; };
  p->kt = stride(a.T, a.k_token), p->kh = stride(c.H, a.k_head);
  p->vt = stride(a.T, a.v_token), p->vh = stride(c.H, a.v_head);
  if ((p->kt | p->kh | p->vt | p->vh) % 8 != 0) return CONVROT_ERR_INVALID_ARG;
  if (a.T == 0) return CONVROT_OK;
  for (const void* ptr : {static_cast<const void*>(a.K), static_cast<const void*>(a.V),
                          static_cast<const void*>(c.k_codes), static_cast<const void*>(c.v_codes),
                          static_cast<const void*>(c.k_scale), static_cast<const void*>(c.v_scale)})
    if (ptr == nullptr || !aligned_to(ptr, 16)) return CONVROT_ERR_INVALID_ARG;
  if (a.slots == nullptr || !aligned_to(a.slots, 4) || !aligned_to(a.status, 4)) return CONVROT_ERR_INVALID_ARG;
  p->k = static_cast<uint16_t*>(a.K);
  p->v = static_cast<uint16_t*>(a.V);
  p->slots = a.slots;
  p->k_codes = c.k_codes;
  p->v_codes = c.v_codes;
  p->k_scale = c.k_scale;
  p->v_scale = c.v_scale;
  p->vectors = 2 * a.T * c.H;
  p->H = static_cast<int>(c.H);
  p->page_shift = 0;
  while ((int64_t{1} << p->page_shift) < c.page_size) ++p->page_shift;
  p->capacity = static_cast<int>(c.num_pages * c.page_size);
  p->status = a.status;
  return CONVROT_OK;
}

unsigned cell_grid(const CellParams& p) {
  return static_cast<unsigned>((p.vectors * 4 + kCellThreads - 1) / kCellThreads);
}

}  // namespace

}  // namespace convrot

extern "C" {

convrot_status convrot_cache_append(const convrot_cache_args* args, convrot_stream_t stream) {
  using namespace convrot;
  CellParams p{};
  const convrot_status st = cell_params(args, &p);
  if (st != CONVROT_OK || args->T == 0) return st;
  (args->dtype == CONVROT_DTYPE_F16 ? cache_append_kernel<true> : cache_append_kernel<false>)<<<
      cell_grid(p), kCellThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? CONVROT_OK : CONVROT_ERR_CUDA;
}

convrot_status convrot_cache_read(const convrot_cache_args* args, convrot_stream_t stream) {
  using namespace convrot;
  CellParams p{};
  const convrot_status st = cell_params(args, &p);
  if (st != CONVROT_OK || args->T == 0) return st;
  (args->dtype == CONVROT_DTYPE_F16 ? cache_read_kernel<true> : cache_read_kernel<false>)<<<
      cell_grid(p), kCellThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? CONVROT_OK : CONVROT_ERR_CUDA;
}

}  // extern "C"
