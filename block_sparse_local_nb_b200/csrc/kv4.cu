// The 4-bit key/value cache: quantising rows as they are written, and reading
// them back (layout in kv4.cuh).
//
// Per token, head and group of 32 channels, with lo and hi the extremes of x:
//   m = the largest bf16 <= (lo + hi) / 2
//   s = the smallest bf16 >= max(hi - m, m - lo) / 7.5
//   c = floor((x - m) / s) + 8,  which stands for m + s (c - 7.5)
// so |x - value| <= s / 2 and no code leaves 0..15.  Every border is decided
// exactly, whatever the inputs: m and s are rounded in one direction (a
// directed rounding to fp32 followed by one to bf16 in the same direction is
// the directed rounding of the exact value), 7.5 s and k s have at most 12
// significant bits and are exact in fp32, and x - m rounded down is below k s
// exactly when x - m is.  An estimate of the quotient therefore needs only one
// exact comparison: r = rint(estimate), k = r if r s <= x - m, else r - 1.
// A group with a non-finite value (or a span beyond fp32) has s = m = NaN.
//
// A thread handles eight channels of the key row and of the value row of one
// token; four neighbouring threads share a group.  The value codes are
// transposed among eight lanes by three exchange steps.  Both kernels are
// bound by memory: 2 d e + d + d / 4 bytes per token and head for both rows
// (e = element size).
#include <cuda_bf16.h>

#include "kv4.cuh"
#include "nb_internal.h"
#include "sm100.cuh"

namespace nb {
namespace {

using namespace kv4;

constexpr int kThreads = 256;

__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// The largest bf16 <= x (x finite or NaN; NaN stays NaN), as a float.
__device__ __forceinline__ float bf16_below(float x) {
  const uint32_t u = __float_as_uint(x);
  const uint32_t up = (x < 0.f && (u & 0xffffu)) ? 0x10000u : 0u;
  return __uint_as_float((u & 0xffff0000u) + up);
}

struct Row8 {
  float x[8];
};

template <bool kF32>
__device__ __forceinline__ Row8 load8(const void* p, int64_t at) {
  Row8 r;
  if constexpr (kF32) {
    const float4* src = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
    const float4 a = __ldcs(src), b = __ldcs(src + 1);
    r.x[0] = a.x; r.x[1] = a.y; r.x[2] = a.z; r.x[3] = a.w;
    r.x[4] = b.x; r.x[5] = b.y; r.x[6] = b.z; r.x[7] = b.w;
  } else {
    const uint4 a =
        __ldcs(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + at));
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r.x[2 * i] = __uint_as_float(w[i] << 16);
      r.x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  return r;
}

// Eight codes of this thread (nibble i = channel i) and the group's param word.
__device__ __forceinline__ uint32_t quantise8(const Row8& v, uint32_t& param) {
  float lo = v.x[0], hi = v.x[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    lo = min_nan(lo, v.x[i]);
    hi = max_nan(hi, v.x[i]);
  }
#pragma unroll
  for (int off = 1; off < 4; off <<= 1) {
    lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, off));
    hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, off));
  }
  const float mid = bf16_below(__fadd_rd(0.5f * lo, 0.5f * hi));
  const float half = max_nan(__fsub_ru(hi, mid), __fsub_ru(mid, lo));
  if (!(half < __uint_as_float(0x7f800000u))) {  // NaN, infinity or overflow in the group
    param = 0x7fc07fc0u;
    return 0x88888888u;
  }
  // the estimate half / 7.5 is off by a few 2^-24, so the smallest bf16 whose
  // 7.5-fold (exact) reaches half is its floor or one of the next two
  const uint32_t c0 = __float_as_uint(half * (1.f / 7.5f)) & 0xffff0000u;
  uint32_t su = c0;
  if (7.5f * __uint_as_float(su) < half) su += 0x10000u;
  if (7.5f * __uint_as_float(su) < half) su += 0x10000u;
  param = (su >> 16) | (__float_as_uint(mid) & 0xffff0000u);
  // steps near the bottom of the range are scaled up (exactly) for the reciprocal
  const float f = __uint_as_float(su) < 0x1p-100f ? 0x1p+100f : 1.f;
  const float s = __uint_as_float(su) * f;
  const float inv = s > 0.f ? __frcp_rn(s) : 0.f;  // s = 0: every x is m
  constexpr float kRint = 12582912.f;              // 1.5 * 2^23: adding it rounds to an integer
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float y = __fsub_rd(v.x[i], mid) * f;
    const float m = __fadd_rn(__fmul_rn(y, inv), kRint);
    const float r = __fadd_rn(m, -kRint);
    const bool over = __fmaf_rn(r, s, -y) > 0.f;  // r s > y, exactly
    const uint32_t code = (__float_as_uint(m) + (over ? 7u : 8u)) & 15u;
    w |= code << (4 * i);
  }
  return w;
}

// Transposes the 8 x 8 nibbles held by eight neighbouring lanes (lane j nibble
// i <-> lane i nibble j).
__device__ __forceinline__ uint32_t transpose8(uint32_t w, int lane) {
  uint32_t o = __shfl_xor_sync(0xffffffffu, w, 4);
  w = (lane & 4) ? (w & 0xffff0000u) | (o >> 16) : (w & 0x0000ffffu) | (o << 16);
  o = __shfl_xor_sync(0xffffffffu, w, 2);
  w = (lane & 2) ? (w & 0xff00ff00u) | ((o >> 8) & 0x00ff00ffu)
                 : (w & 0x00ff00ffu) | ((o & 0x00ff00ffu) << 8);
  o = __shfl_xor_sync(0xffffffffu, w, 1);
  return (lane & 1) ? (w & 0xf0f0f0f0u) | ((o >> 4) & 0x0f0f0f0fu)
                    : (w & 0x0f0f0f0fu) | ((o & 0x0f0f0f0fu) << 4);
}

// Row `row` of a [batch][kv_heads][n] tensor, and where its token lives.
struct Slot {
  uint8_t* page;  // null: not one of the listed tokens, or not mapped
  int token;      // within the page
  bool listed;    // row is one of the sequence's `count` tokens
};

__device__ __forceinline__ Slot find_slot(const Pool& pool, const int32_t* starts,
                                          const int32_t* counts, int n, int row, int page_bytes) {
  Slot s = {nullptr, 0, false};
  const int bh = row / n, t = row - bh * n;
  const int b = bh / pool.kv_heads, h = bh - b * pool.kv_heads;
  s.listed = counts == nullptr || t < counts[b];
  if (!s.listed) return s;
  const int64_t pos = static_cast<int64_t>(starts ? starts[b] : 0) + t;
  if (pos < 0 || pos >= static_cast<int64_t>(pool.max_pages) * kPage) return s;
  const int id = pool.table[static_cast<int64_t>(b) * pool.max_pages + (pos >> 5)];
  if (id < 0 || id >= pool.num_pages) return s;
  s.page = pool.base + (static_cast<int64_t>(id) * pool.kv_heads + h) * page_bytes;
  s.token = static_cast<int>(pos) & (kPage - 1);
  return s;
}

template <int D, bool kF32>
__global__ void __launch_bounds__(kThreads)
    kv4_write_kernel(const void* k, const void* v, Pool pool, const int32_t* starts,
                     const int32_t* counts, int n, int rows, int* err) {
  using P = Page<D>;
  constexpr int kLanes = D / 8;  // threads per row
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, j = threadIdx.x % kLanes;
  const int row = static_cast<int>(
      (blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x) / kLanes);
  Slot s = {nullptr, 0, false};
  Row8 kr = {}, vr = {};
  if (row < rows) {
    s = find_slot(pool, starts, counts, n, row, P::kBytes);
    if (s.page) {
      const int64_t at = static_cast<int64_t>(row) * D + 8 * j;
      kr = load8<kF32>(k, at);
      vr = load8<kF32>(v, at);
    } else if (s.listed && j == 0) {
      sm100::record_error(err, kErrWriteSlot);
    }
  }
  uint32_t kpar, vpar;  // every lane takes part in the exchanges
  const uint32_t kw = quantise8(kr, kpar);
  const uint32_t vw = transpose8(quantise8(vr, vpar), lane);
  if (!s.page) return;
  const int g = j >> 2, t = j & 3;
  *reinterpret_cast<uint32_t*>(s.page + P::oK + s.token * P::kRow + (t * P::kGroups + g) * 4) = kw;
  *reinterpret_cast<uint32_t*>(s.page + P::oV + s.token * P::kRow + P::v_chunk(s.token, j & 7) +
                               (j >> 3) * 4) = vw;
  if (t == 0) {
    *reinterpret_cast<uint32_t*>(s.page + P::oKPar + s.token * P::kParRow + g * 4) = kpar;
    *reinterpret_cast<uint32_t*>(s.page + P::oVPar + s.token * P::kParRow + g * 4) = vpar;
  }
}

// m + s (c - 7.5) for eight codes: s (c - 7.5) is exact inside the fused
// multiply-add, so an fp32 output is rounded once.
template <bool kF32>
__device__ __forceinline__ void store8(void* p, int64_t at, uint32_t w, uint32_t param,
                                       bool zero) {
  const float s = __uint_as_float(param << 16), m = __uint_as_float(param & 0xffff0000u);
  float x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // 2^23 + code - (2^23 + 7.5) would round; code - 7.5 through a shifted mantissa is exact:
    // bits 0x4b000000 | 2 code is 2^23 + 2 code, minus 2^23 + 15 gives 2 (code - 7.5)
    const uint32_t twice = i == 0 ? (w << 1) & 30u : (w >> (4 * i - 1)) & 30u;
    const float c2 = __uint_as_float(0x4b000000u | twice) - 8388623.f;
    x[i] = zero ? 0.f : fmaf(0.5f * s, c2, m);
  }
  if constexpr (kF32) {
    float4* out = reinterpret_cast<float4*>(static_cast<float*>(p) + at);
    __stcs(out, make_float4(x[0], x[1], x[2], x[3]));
    __stcs(out + 1, make_float4(x[4], x[5], x[6], x[7]));
  } else {
    __stcs(reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p) + at),
           make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                      pack_bf16(x[6], x[7])));
  }
}

template <int D, bool kF32>
__global__ void __launch_bounds__(kThreads)
    kv4_read_kernel(void* k, void* v, Pool pool, const int32_t* starts, const int32_t* counts,
                    int n, int rows, int* err) {
  using P = Page<D>;
  constexpr int kLanes = D / 8;
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, j = threadIdx.x % kLanes;
  const int row = static_cast<int>(
      (blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x) / kLanes);
  const int g = j >> 2, t = j & 3;
  Slot s = {nullptr, 0, false};
  uint32_t kw = 0, vw = 0, kpar = 0, vpar = 0;
  if (row < rows) {
    s = find_slot(pool, starts, counts, n, row, P::kBytes);
    if (s.page) {
      kw = *reinterpret_cast<const uint32_t*>(s.page + P::oK + s.token * P::kRow +
                                              (t * P::kGroups + g) * 4);
      vw = *reinterpret_cast<const uint32_t*>(s.page + P::oV + s.token * P::kRow +
                                              P::v_chunk(s.token, j & 7) + (j >> 3) * 4);
      kpar = *reinterpret_cast<const uint32_t*>(s.page + P::oKPar + s.token * P::kParRow + g * 4);
      vpar = *reinterpret_cast<const uint32_t*>(s.page + P::oVPar + s.token * P::kParRow + g * 4);
    } else if (s.listed && j == 0) {
      sm100::record_error(err, kErrReadSlot);
    }
  }
  vw = transpose8(vw, lane);
  if (row >= rows) return;
  const int64_t at = static_cast<int64_t>(row) * D + 8 * j;
  store8<kF32>(k, at, kw, kpar, !s.page);
  store8<kF32>(v, at, vw, vpar, !s.page);
}

Pool make_pool(const Kv4Args& a) {
  return Pool{static_cast<uint8_t*>(a.cache), a.table, a.max_pages, a.num_pages, a.kv_heads};
}

unsigned blocks_for(const Kv4Args& a, int64_t rows) {
  return static_cast<unsigned>((rows * (a.d / 8) + kThreads - 1) / kThreads);
}

template <int D, bool kF32>
cudaError_t run(const Kv4Args& a, bool write, cudaStream_t stream) {
  const int rows = a.batch * a.kv_heads * a.n;  // checked to fit by the caller
  const dim3 grid(blocks_for(a, rows)), block(kThreads);
  if (write)
    return launch_pdl(kv4_write_kernel<D, kF32>, grid, block, 0, stream,
                      static_cast<const void*>(a.k), static_cast<const void*>(a.v), make_pool(a),
                      a.starts, a.counts, a.n, rows, a.err);
  return launch_pdl(kv4_read_kernel<D, kF32>, grid, block, 0, stream, a.k, a.v, make_pool(a),
                    a.starts, a.counts, a.n, rows, a.err);
}

}  // namespace

int kv4_page_bytes(int d) { return d == 64 ? Page<64>::kBytes : Page<128>::kBytes; }

cudaError_t launch_kv4(const Kv4Args& a, bool write, cudaStream_t stream) {
  if (a.d == 64)
    return a.f32 ? run<64, true>(a, write, stream) : run<64, false>(a, write, stream);
  return a.f32 ? run<128, true>(a, write, stream) : run<128, false>(a, write, stream);
}

}  // namespace nb
