// Rows that a tile computed beside values which they do not see.
//
// The tensor cores multiply every row of a tile with every row of a chunk, and the mask
// enters as a weight of 0.  Where the hidden row of the chunk holds a NaN or an infinity,
// 0 times it is NaN.  Finite inputs never meet this, so nothing of it stands in the path of
// a chunk: the epilogue notes rows that came out non-finite (a multiply-add for two
// values), and when a block has finished its tiles, its warps look at such rows again: a
// row that only visible values made non-finite stays, and one with a non-finite hidden row
// among its chunks' is summed once more over the rows that it sees, in fp32 and in a fixed
// order; the other rows keep their bits.  (Each lane reads a row of its own 16 bytes at a
// time, which binds it: one bad token makes a forward of 32768 x 64 with window 1024 1.2 ms
// longer, of 32768 x 128 2.2 ms.  Clean inputs pay 0.3 to 0.8 % for the notes,
// forward and backward of 2 x 4 heads x 333 x 64 1.4 %, 0.5 us.)
// The sinks' blocks, which every later tile reads, would make this the common case for one
// bad token near a sequence's begin: there the tensor map itself ends with the sinks.
#pragma once

#include <cuda_bf16.h>

#include "sm100.cuh"

namespace nb {
namespace hidden {

using bf16 = __nv_bfloat16;

// Sums two bf16 a word times 0: NaN in a half once it met a NaN or an infinity there.
__device__ __forceinline__ uint32_t add_zeros(uint32_t w, uint32_t acc) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(w), "r"(0u), "r"(acc));
  return r;
}
__device__ __forceinline__ bool word_bad(uint32_t w) {
  return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

// Whether some of the rows [lo, hi) of x holds a NaN or an infinity.  Whole warp.
template <int D>
__device__ __forceinline__ bool any_bad(const bf16* x, int lo, int hi, int lane) {
  bool bad = false;
  for (int r = lo + lane; r < hi; r += 32) {
    const uint4* row = reinterpret_cast<const uint4*>(x + static_cast<int64_t>(r) * D);
#pragma unroll 1
    for (int i = 0; i < D / 8; ++i) {
      const uint4 w = row[i];
      bad |= word_bad(w.x) || word_bad(w.y) || word_bad(w.z) || word_bad(w.w);
    }
  }
  return __any_sync(0xffffffffu, bad);
}

// One thread's product of two rows.
template <int D>
__device__ __forceinline__ float dot(const bf16* a, const bf16* b) {
  const uint4* pa = reinterpret_cast<const uint4*>(a);
  const uint4* pb = reinterpret_cast<const uint4*>(b);
  float s = 0.f;
#pragma unroll 4
  for (int i = 0; i < D / 8; ++i) {
    const uint4 x = pa[i], y = pb[i];
    const uint32_t u[4] = {x.x, x.y, x.z, x.w}, v[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      s = fmaf(__uint_as_float(u[e] << 16), __uint_as_float(v[e] << 16), s);
      s = fmaf(__uint_as_float(u[e] & 0xffff0000u), __uint_as_float(v[e] & 0xffff0000u), s);
    }
  }
  return s;
}

// A row spread over a warp: lane l has its channels D / 32 l and on.
template <int D>
struct Row {
  static constexpr int N = D / 32;
  float v[N];

  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = 0.f;
  }
  __device__ __forceinline__ void scale(float f) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] *= f;
  }
  __device__ __forceinline__ void add(const bf16* row, float w, int lane) {
    const uint32_t* p = reinterpret_cast<const uint32_t*>(row + N * lane);
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const uint32_t x = p[i];
      v[2 * i] = fmaf(w, __uint_as_float(x << 16), v[2 * i]);
      v[2 * i + 1] = fmaf(w, __uint_as_float(x & 0xffff0000u), v[2 * i + 1]);
    }
  }
  // sum_j weight_j row_j over the rows base + jj, lo <= jj < hi; lane jj holds weight_jj
  __device__ __forceinline__ void add_rows(const bf16* x, int64_t base, int lo, int hi, float weight,
                                           int lane) {
#pragma unroll 8
    for (int jj = lo; jj < hi; ++jj)
      add(x + (base + jj) * D, __shfl_sync(0xffffffffu, weight, jj), lane);
  }
};

// The channels of a stored row that are not finite (bit i: the lane's i-th), through L2:
// a tensor store may have written them.
template <int D>
__device__ __forceinline__ uint32_t bad_channels(const bf16* row, int lane) {
  const uint32_t* p = reinterpret_cast<const uint32_t*>(row + Row<D>::N * lane);
  uint32_t bad = 0;
#pragma unroll
  for (int i = 0; i < Row<D>::N / 2; ++i) {
    const uint32_t w = __ldcg(p + i);
    if ((w & 0x7f80u) == 0x7f80u) bad |= 1u << (2 * i);
    if ((w & 0x7f800000u) == 0x7f800000u) bad |= 2u << (2 * i);
  }
  return bad;
}
// The same of a row of fp32 written by other threads of this block.
template <int D>
__device__ __forceinline__ uint32_t bad_channels(const float* row, int lane) {
  uint32_t bad = 0;
#pragma unroll
  for (int i = 0; i < Row<D>::N; ++i) {
    const uint32_t w = __float_as_uint(__ldcg(row + Row<D>::N * lane + i));
    if ((w & 0x7f800000u) == 0x7f800000u) bad |= 1u << i;
  }
  return bad;
}
// Writes the channels of `which`.
template <int D>
__device__ __forceinline__ void store_channels(bf16* row, const Row<D>& r, uint32_t which, int lane) {
#pragma unroll
  for (int i = 0; i < Row<D>::N; ++i)
    if (which >> i & 1u) row[Row<D>::N * lane + i] = __float2bfloat16_rn(r.v[i]);
}
template <int D>
__device__ __forceinline__ void store_channels(float* row, const Row<D>& r, uint32_t which, int lane) {
#pragma unroll
  for (int i = 0; i < Row<D>::N; ++i)
    if (which >> i & 1u) row[Row<D>::N * lane + i] = r.v[i];
}
// Every channel of `which`, in all lanes, is NaN: no further term changes the row.
template <int D>
__device__ __forceinline__ bool settled(const Row<D>& r, uint32_t which) {
  bool all = true;
#pragma unroll
  for (int i = 0; i < Row<D>::N; ++i) all = all && (!(which >> i & 1u) || r.v[i] != r.v[i]);
  return __all_sync(0xffffffffu, all);
}

}  // namespace hidden
}  // namespace nb
