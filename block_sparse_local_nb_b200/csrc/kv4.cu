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
// A writing thread handles sixteen channels of the key row and of the value row of
// one token; two threads share a group, four transpose the value codes of 64 channels
// among them.  (With eight channels a thread it was bound by issued instructions:
// 523 a warp of 512 values, 78 us for 4 x 8 heads x 8192 x 128 bf16, where the
// bytes take 27 us.)  Bytes per token and head for
// both rows: 2 d e + d + d / 4 (e = element size).
#include <cuda_bf16.h>

#include "kv4.cuh"
#include "serving.cuh"

namespace nb {
namespace {

using namespace kv4;

constexpr int kThreads = 256;

// The largest bf16 <= x (x finite or NaN; NaN stays NaN), as a float.
__device__ __forceinline__ float bf16_below(float x) {
  const uint32_t u = __float_as_uint(x);
  const uint32_t up = (x < 0.f && (u & 0xffffu)) ? 0x10000u : 0u;
  return __uint_as_float((u & 0xffff0000u) + up);
}

struct Row16 {
  float x[16];
};

template <bool kF32>
__device__ __forceinline__ Row16 load16(const void* p, int64_t at) {
  Row16 r;
  if constexpr (kF32) {
    const float4* src = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 a = __ldcs(src + i);
      r.x[4 * i] = a.x;
      r.x[4 * i + 1] = a.y;
      r.x[4 * i + 2] = a.z;
      r.x[4 * i + 3] = a.w;
    }
  } else {
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + at);
    const uint4 a = __ldcs(src), b = __ldcs(src + 1);
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      r.x[2 * i] = __uint_as_float(w[i] << 16);
      r.x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  return r;
}

// Eight codes, nibble i = channel i.  The estimate z (-1 / s) of (x - m) / s is
// rounded to an integer by adding 1.5 * 2^23 + 8, whose low bits then hold r + 8;
// r s - (x - m) > 0 lowers it by one.  The constant's high bits go at the end.
template <bool kTiny>
__device__ __forceinline__ uint32_t codes8(const float* x, float mid, float s, float ninv) {
  constexpr float kRint = 12582920.f;
  constexpr uint32_t kBase = 0x4b400000u;
  uint32_t w = 0u - (kBase + (kBase << 4) + (kBase << 8));  // further shifts leave nothing
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float z = __fsub_ru(mid, x[i]);  // -(x - m rounded down)
    if (kTiny) z *= 0x1p+100f;
    const float m = __fmaf_rn(z, ninv, kRint);
    float over;  // 1 or 0: taking it off in fp32 spares the integer pipe, which is the busy one
    asm("set.gt.f32.f32 %0, %1, 0f00000000;"
        : "=f"(over)
        : "f"(__fmaf_rn(__fadd_rn(m, -kRint), s, z)));
    w += __float_as_uint(__fadd_rn(m, -over)) << (4 * i);
  }
  return w;
}

// The codes of this thread's sixteen channels and the group's param word.
__device__ __forceinline__ void quantise16(const Row16& v, uint32_t (&w)[2], uint32_t& param) {
  float lo = v.x[0], hi = v.x[0];
#pragma unroll
  for (int i = 1; i < 16; ++i) {
    lo = min_nan(lo, v.x[i]);
    hi = max_nan(hi, v.x[i]);
  }
  lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, 1));
  hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, 1));
  // halved before the sum only where that could overflow: half of a subnormal is not
  // exact, and two roundings down of the whole sum are one
  const float mid = bf16_below(fmaxf(fabsf(lo), fabsf(hi)) < 0x1p126f
                                   ? __fmul_rd(0.5f, __fadd_rd(lo, hi))
                                   : __fadd_rd(__fmul_rd(0.5f, lo), __fmul_rd(0.5f, hi)));
  const float half = max_nan(__fsub_ru(hi, mid), __fsub_ru(mid, lo));
  if (!(half < __uint_as_float(0x7f800000u))) {  // NaN, infinity or overflow in the group
    param = 0x7fc07fc0u;
    w[0] = w[1] = 0x88888888u;
    return;
  }
  // the estimate half / 7.5 is off by a few 2^-24, so the smallest bf16 whose
  // 7.5-fold (exact) reaches half is its floor or one of the next two
  uint32_t su = __float_as_uint(half * (1.f / 7.5f)) & 0xffff0000u;
  if (7.5f * __uint_as_float(su) < half) su += 0x10000u;
  if (7.5f * __uint_as_float(su) < half) su += 0x10000u;
  param = (su >> 16) | (__float_as_uint(mid) & 0xffff0000u);
  float s = __uint_as_float(su);
  if (s >= 0x1p-100f || s == 0.f) {
    const float ninv = s > 0.f ? __frcp_rn(-s) : 0.f;  // s = 0: every x is m
    w[0] = codes8<false>(v.x, mid, s, ninv);
    w[1] = codes8<false>(v.x + 8, mid, s, ninv);
  } else {  // near the bottom of the range: scaled up (exactly) for the reciprocal
    s *= 0x1p+100f;
    const float ninv = __frcp_rn(-s);
    w[0] = codes8<true>(v.x, mid, s, ninv);
    w[1] = codes8<true>(v.x + 8, mid, s, ninv);
  }
}

// Transposes the 8 x 8 nibbles held by four neighbouring threads, words 2 j and
// 2 j + 1 by thread j (word a nibble b <-> word b nibble a).
__device__ __forceinline__ void transpose8(uint32_t (&w)[2], int lane) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t o = __shfl_xor_sync(0xffffffffu, w[i], 2);
    w[i] = __byte_perm(w[i], o, (lane & 2) ? 0x3276u : 0x5410u);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t o = __shfl_xor_sync(0xffffffffu, w[i], 1);
    w[i] = __byte_perm(w[i], o, (lane & 1) ? 0x3715u : 0x6240u);
  }
  const uint32_t a = w[0], b = w[1];
  w[0] = (a & 0x0f0f0f0fu) | ((b & 0x0f0f0f0fu) << 4);
  w[1] = (b & 0xf0f0f0f0u) | ((a >> 4) & 0x0f0f0f0fu);
}

// Where token t of a sequence's `count` lives.
struct Slot {
  uint8_t* page;  // null: not one of the listed tokens, or not mapped
  int token;      // within the page
};

__device__ __forceinline__ Slot find_slot(const Pool& pool, const int32_t* starts, int b, int h,
                                          int t, int count, int page_bytes) {
  Slot s = {nullptr, 0};
  if (t >= count) return s;
  const int64_t pos = static_cast<int64_t>(starts ? starts[b] : 0) + t;
  if (pos < 0 || pos >= static_cast<int64_t>(pool.max_pages) * kPage) return s;
  const int id = pool.table[static_cast<int64_t>(b) * pool.max_pages + (pos >> 5)];
  if (id < 0 || id >= pool.num_pages) return s;
  s.page = pool.base + (static_cast<int64_t>(id) * pool.kv_heads + h) * page_bytes;
  s.token = static_cast<int>(pos) & (kPage - 1);
  return s;
}

// Places of thread j's words in a row: K words j and j + kGroups of the row's
// first (its group g = j / 2, lane words t = 2 (j mod 2) and the next), V word
// j / 4 of chunks r and r + 1, r = 2 (j mod 4).
template <int D>
struct Places {
  using P = Page<D>;
  uint8_t *k0, *k1, *v0, *v1;
  uint32_t *kp, *vp;
  __device__ __forceinline__ Places(uint8_t* page, int token, int j) {
    const int g = j >> 1, t = 2 * (j & 1), r = 2 * (j & 3);
    k0 = page + P::oK + token * P::kRow + (t * P::kGroups + g) * 4;
    k1 = k0 + P::kGroups * 4;
    uint8_t* v = page + P::oV + token * P::kRow + (j >> 2) * 4;
    v0 = v + P::v_chunk(token, r);
    v1 = v + P::v_chunk(token, r + 1);
    kp = reinterpret_cast<uint32_t*>(page + P::oKPar + token * P::kParRow) + g;
    vp = reinterpret_cast<uint32_t*>(page + P::oVPar + token * P::kParRow) + g;
  }
};

template <int D>
constexpr int kRows = kThreads / (D / 16);  // tokens of a block

// Grid: blocks of tokens, heads, sequences.
template <int D, bool kF32>
__global__ void __launch_bounds__(kThreads)
    kv4_write_kernel(const void* k, const void* v, Pool pool, const int32_t* starts,
                     const int32_t* counts, int n, int* skip) {
  constexpr int kLanes = D / 16;  // threads per row
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, j = threadIdx.x % kLanes;
  const int t = blockIdx.x * kRows<D> + threadIdx.x / kLanes, h = blockIdx.y, b = blockIdx.z;
  const int count = counts ? min(counts[b], n) : n;
  if (!__any_sync(0xffffffffu, t < count)) return;
  const Slot s = find_slot(pool, starts, b, h, t, count, Page<D>::kBytes);
  // threads past the last token take its row along, for the exchanges
  const int64_t at =
      ((static_cast<int64_t>(b) * pool.kv_heads + h) * n + min(t, count - 1)) * D + 16 * j;
  const Row16 kr = load16<kF32>(k, at), vr = load16<kF32>(v, at);
  if (!s.page && t < count && j == 0) sm100::record_error(skip, kErrWriteSlot);
  uint32_t kw[2], vw[2], kpar, vpar;
  quantise16(kr, kw, kpar);
  quantise16(vr, vw, vpar);
  transpose8(vw, lane);
  if (!s.page) return;
  const Places<D> to(s.page, s.token, j);
  *reinterpret_cast<uint32_t*>(to.k0) = kw[0];
  *reinterpret_cast<uint32_t*>(to.k1) = kw[1];
  if constexpr (D == 64) {  // the two chunks are neighbours
    *reinterpret_cast<uint2*>(to.v0) = make_uint2(vw[0], vw[1]);
  } else {
    *reinterpret_cast<uint32_t*>(to.v0) = vw[0];
    *reinterpret_cast<uint32_t*>(to.v1) = vw[1];
  }
  if ((j & 1) == 0) {
    *to.kp = kpar;
    *to.vp = vpar;
  }
}

// m + s (c - 7.5) of eight codes, rounded once: in bf16 by one fused multiply-add
// of exact bf16 operands, in fp32 likewise.  Channel i is nibble i, or (kMixed)
// nibble 4 (i mod 2) + i / 2, which puts neighbours four nibbles apart.
template <bool kF32, bool kMixed>
__device__ __forceinline__ void store8(void* p, int64_t at, uint32_t w, uint32_t param) {
  if constexpr (kF32) {
    const float s = __uint_as_float(param << 16), m = __uint_as_float(param & 0xffff0000u);
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // the code doubled in the low bits of 2^23, minus 2^23 + 15: 2 (c - 7.5), exact
      const int nib = kMixed ? 4 * (i & 1) + (i >> 1) : i;
      const uint32_t twice = nib == 0 ? (w << 1) & 30u : (w >> (4 * nib - 1)) & 30u;
      x[i] = fmaf(0.5f * s, __uint_as_float(0x4b000000u | twice) - 8388623.f, m);
    }
    float4* out = reinterpret_cast<float4*>(static_cast<float*>(p) + at);
    __stcs(out, make_float4(x[0], x[1], x[2], x[3]));
    __stcs(out + 1, make_float4(x[4], x[5], x[6], x[7]));
  } else {
    const uint32_t s2 = __byte_perm(param, 0, 0x1010), m2 = __byte_perm(param, 0, 0x3232);
    const uint32_t c = 0x421e421eu;  // 39.5, 39.5
    auto h2 = [](const uint32_t& x) { return *reinterpret_cast<const __nv_bfloat162*>(&x); };
    uint32_t y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // nibbles i and i + 4: 32 + c minus 39.5, exact
      const uint32_t x = ((i == 0 ? w << 2 : w >> (4 * i - 2)) & 0x003c003cu) | 0x42004200u;
      const __nv_bfloat162 r = __hfma2(__hsub2(h2(x), h2(c)), h2(s2), h2(m2));
      y[i] = *reinterpret_cast<const uint32_t*>(&r);
    }
    uint4* out = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p) + at);
    __stcs(out, kMixed ? make_uint4(y[0], y[1], y[2], y[3])
                       : make_uint4(__byte_perm(y[0], y[1], 0x5410), __byte_perm(y[2], y[3], 0x5410),
                                    __byte_perm(y[0], y[1], 0x7632),
                                    __byte_perm(y[2], y[3], 0x7632)));
  }
}

// Four threads read a token's rows back, one wide load each for codes and params:
// thread j has K word [j][g], channels 32 g + 8 j .., of every group g, and V
// chunks 2 j, 2 j + 1, whose words of 64 channels the four transpose among them
// so that it ends with the same channels.  (A word a load was bound by the load
// unit: 42 us for 4 x 8 x 8192 x 128.)
template <int D, bool kF32>
__global__ void __launch_bounds__(kThreads)
    kv4_read_kernel(void* k, void* v, Pool pool, const int32_t* starts, const int32_t* counts,
                    int n, int* skip) {
  using P = Page<D>;
  constexpr int NG = P::kGroups;
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, j = threadIdx.x & 3;
  const int t = blockIdx.x * (kThreads / 4) + threadIdx.x / 4, h = blockIdx.y, b = blockIdx.z;
  // codes 0 with s = m = 0 stand for 0: rows that are not listed or not mapped
  uint32_t kw[NG] = {}, vw[NG] = {}, kpar[NG] = {}, vpar[NG] = {};
  if (t < n) {
    const int count = counts ? min(counts[b], n) : n;
    const Slot s = find_slot(pool, starts, b, h, t, count, P::kBytes);
    if (s.page) {
      auto load = [](uint32_t (&w)[NG], const uint8_t* p) {
        if constexpr (NG == 4) {
          const uint4 x = *reinterpret_cast<const uint4*>(p);
          w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
        } else {
          const uint2 x = *reinterpret_cast<const uint2*>(p);
          w[0] = x.x; w[1] = x.y;
        }
      };
      load(kw, s.page + P::oK + s.token * P::kRow + j * (4 * NG));
      load(vw, s.page + P::oV + s.token * P::kRow + P::v_chunk(s.token, 2 * j));
      load(kpar, s.page + P::oKPar + s.token * P::kParRow);
      load(vpar, s.page + P::oVPar + s.token * P::kParRow);
    } else if (t < count && j == 0) {
      sm100::record_error(skip, kErrReadSlot);
    }
  }
  // The words of chunks 2 j, 2 j + 1 (chunk bits j1 j0 e, word bit e its own), nibble
  // bits n2 n1 n0: three exchanges bring n1 n0 to the thread and n2 to e, and leave
  // nibble bits e j1 j0.
  uint32_t vo[NG];
#pragma unroll
  for (int w = 0; w < NG / 2; ++w) {  // 64 channels each: vw = [chunk][word]
    uint32_t x[2] = {vw[w], vw[NG / 2 + w]};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t o = __shfl_xor_sync(0xffffffffu, x[i], 2);
      x[i] = __byte_perm(x[i], o, (lane & 2) ? 0x3715u : 0x6240u);
      o = __shfl_xor_sync(0xffffffffu, x[i], 1);
      x[i] = (lane & 1) ? (x[i] & 0xf0f0f0f0u) | ((o >> 4) & 0x0f0f0f0fu)
                        : (x[i] & 0x0f0f0f0fu) | ((o & 0x0f0f0f0fu) << 4);
    }
    vo[2 * w] = __byte_perm(x[0], x[1], 0x5410);
    vo[2 * w + 1] = __byte_perm(x[0], x[1], 0x7632);
  }
  if (t >= n) return;
  const int64_t at = ((static_cast<int64_t>(b) * pool.kv_heads + h) * n + t) * D + 8 * j;
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    store8<kF32, false>(k, at + 32 * g, kw[g], kpar[g]);
    store8<kF32, true>(v, at + 32 * g, vo[g], vpar[g]);
  }
}

Pool make_pool(const Kv4Args& a) {
  return Pool{static_cast<uint8_t*>(a.cache), a.table, a.max_pages, a.num_pages, a.kv_heads};
}

template <int D, bool kF32>
cudaError_t run(const Kv4Args& a, bool write, cudaStream_t stream) {
  const int rows = write ? kRows<D> : kThreads / 4;  // tokens of a block
  const dim3 grid((a.n + rows - 1) / rows, a.kv_heads, a.batch), block(kThreads);
  if (write)
    return launch_pdl(kv4_write_kernel<D, kF32>, grid, block, 0, stream,
                      static_cast<const void*>(a.k), static_cast<const void*>(a.v), make_pool(a),
                      a.starts, a.counts, a.n, a.skip);
  return launch_pdl(kv4_read_kernel<D, kF32>, grid, block, 0, stream, a.k, a.v, make_pool(a),
                    a.starts, a.counts, a.n, a.skip);
}

}  // namespace

int kv4_page_bytes(int d) { return d == 64 ? Page<64>::kBytes : Page<128>::kBytes; }

cudaError_t launch_kv4(const Kv4Args& a, bool write, cudaStream_t stream) {
  if (a.d == 64)
    return a.f32 ? run<64, true>(a, write, stream) : run<64, false>(a, write, stream);
  return a.f32 ? run<128, true>(a, write, stream) : run<128, false>(a, write, stream);
}

}  // namespace nb
