// Attention of one query token per sequence over the 4-bit cache, with a
// sliding window and visible first tokens (layout of the cache in kv4.cuh).
//
// With key value k_j = m_jg + s_jg (c - 7.5) on channel group g,
//   q . k_j = sum_g s_jg (q_g . c_jg) + (m_jg - 7.5 s_jg) sum(q_g)
//   O = sum_j p_j v_j = sum_j (p_j s_jg)(c - 7.5) + sum_j p_j m_jg
// so the codes themselves are the operands of a warp matrix product (m16n8k16,
// rows = the query heads that share the key/value head): no row is ever
// dequantised in memory, and s and m enter in fp32 outside the products.  A
// nibble becomes bf16 by or-ing it into the mantissa of 32 (32 + c, exact); the
// 39.5 = 32 + 7.5 is taken off through sum(q_g) for the keys and by an exact
// bf16 subtraction for the values.  Softmax statistics, sums and outputs are
// fp32; p s is rounded to bf16 as the operand of the value product (the output
// is bf16, and each p carries an error of its own).
//
// A block of four warps takes one key/value head of one sequence and a share of
// its visible pages (the pages of the sinks, then those of the window); warp w
// takes every fourth page, brought by one bulk copy each into the warp's own
// ring, and keeps its own maximum, sum and output.  The warps, and then the
// shares, are joined by their maxima.  Bound by memory: the page bytes, once.
#include <math.h>

#include "kv4.cuh"
#include "nb_internal.h"
#include "sm100.cuh"

namespace nb {
namespace {

using namespace kv4;
using namespace sm100;

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kHeads = 16;  // query heads of one block (the rows of a product)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <int D>
struct Cfg {
  using P = Page<D>;
  static constexpr int kStages = 3;
  static constexpr int kRing = kWarps * kStages * P::kBytes;
  // the warps' results take the place of the ring when the pages are done
  static constexpr int kJoin = kWarps * kHeads * (D + 2) * 4;
  static constexpr int oBar = kRing > kJoin ? kRing : kJoin;
  static constexpr int oOk = oBar + kWarps * kStages * 8;  // 1: the stage holds a page
  static constexpr int kSmem = oOk + kWarps * kStages * 4;
  static_assert(P::kBytes % 16 == 0, "bulk copy size");
};

struct Params {
  Pool pool;
  const __nv_bfloat16* q;  // [batch][heads][d]
  __nv_bfloat16* o;
  float* lse;              // [batch][heads] or null
  const int32_t* lengths;  // null: every sequence is max_pages pages long
  float* part;             // splits > 1: [batch][heads][splits][d], then (m, l) pairs
  float2* part_ml;
  int* err;
  int heads, group, head_blocks, splits, window, sinks;
  float sl2;  // log2(e) / sqrt(d)
};

// The visible pages of a sequence of `len` tokens, in order: the pages that hold
// sinks and lie before the window's first page, then the window's pages.
struct Visible {
  int len, first;         // tokens below `first` are visible only as sinks
  int sink_pages, page0;  // page0: the window's first page
  int count;
};

__device__ __forceinline__ Visible visible_pages(const Params& p, int b) {
  Visible v;
  const int64_t cap = static_cast<int64_t>(p.pool.max_pages) * kPage;
  int64_t len = p.lengths ? p.lengths[b] : cap;
  len = len < 0 ? 0 : (len > cap ? cap : len);
  v.len = static_cast<int>(len);
  v.first = v.len > p.window ? v.len - p.window : 0;
  v.page0 = v.first / kPage;
  const int sp = (min(p.sinks, v.len) + kPage - 1) / kPage;
  v.sink_pages = min(sp, v.page0);
  v.count = v.sink_pages + (v.len + kPage - 1) / kPage - v.page0;
  return v;
}

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Nibbles i and i + 4 of w as the bf16 pair (32 + c_i, 32 + c_{i+4}).
template <int I>
__device__ __forceinline__ uint32_t codes_bf16(uint32_t w) {
  const uint32_t x = I == 0 ? w << 2 : w >> (4 * I - 2);
  return (x & 0x003c003cu) | 0x42004200u;
}
// the same minus 39.5: c - 7.5, exact
template <int I>
__device__ __forceinline__ uint32_t centred_bf16(uint32_t w) {
  const uint32_t x = codes_bf16<I>(w);
  const uint32_t c = 0x421e421eu;  // 39.5, 39.5
  __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&x),
                             *reinterpret_cast<const __nv_bfloat162*>(&c));
  return *reinterpret_cast<uint32_t*>(&r);
}

__device__ __forceinline__ float step_of(uint32_t par) { return __uint_as_float(par << 16); }
__device__ __forceinline__ float mid_of(uint32_t par) {
  return __uint_as_float(par & 0xffff0000u);
}

template <int N>
__device__ __forceinline__ void lds_words(uint32_t (&w)[N], const uint8_t* p) {
  if constexpr (N == 4) {
    const uint4 x = *reinterpret_cast<const uint4*>(p);
    w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
  } else if constexpr (N == 2) {
    const uint2 x = *reinterpret_cast<const uint2*>(p);
    w[0] = x.x; w[1] = x.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

// kRows: 1 when at most eight heads share the cache (rows 8..15 of the products
// are zero), 2 otherwise.
template <int D, int kRows>
__global__ void __launch_bounds__(kThreads) kv4_decode_kernel(const Params p) {
  using C = Cfg<D>;
  using P = Page<D>;
  constexpr int NG = P::kGroups, NV = D / 64;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, t = lane & 3;
  const uint32_t base = smem_u32(smem);
  const uint32_t bar = base + C::oBar + warp * C::kStages * 8;
  volatile int* ok = reinterpret_cast<volatile int*>(smem + C::oOk) + warp * C::kStages;
  uint8_t* ring = smem + warp * C::kStages * P::kBytes;
  const uint32_t ring_s = base + warp * C::kStages * P::kBytes;

  if (lane == 0) {
    for (int i = 0; i < C::kStages; ++i) mbar_init(bar + 8 * i, 1);
    fence_barrier_init();
  }
  __syncwarp();
  pdl_trigger();
  pdl_wait();

  const int split = blockIdx.x % p.splits;
  const int hb = (blockIdx.x / p.splits) % p.head_blocks;
  const int bk = blockIdx.x / (p.splits * p.head_blocks);
  const int b = bk / p.pool.kv_heads, kvh = bk - b * p.pool.kv_heads;
  const int head0 = kvh * p.group + hb * kHeads;  // first query head of the block
  const int nh = min(kHeads, p.group - hb * kHeads);

  const Visible vis = visible_pages(p, b);
  const int i0 = static_cast<int>(static_cast<int64_t>(vis.count) * split / p.splits);
  const int i1 = static_cast<int>(static_cast<int64_t>(vis.count) * (split + 1) / p.splits);
  const int mine = i1 - i0 > warp ? (i1 - i0 - warp + kWarps - 1) / kWarps : 0;  // this warp's pages
  auto page_of = [&](int i) {  // logical page of this warp's i-th page
    const int x = i0 + warp + i * kWarps;
    return x < vis.sink_pages ? x : vis.page0 + (x - vis.sink_pages);
  };
  const int32_t* table = p.pool.table + static_cast<int64_t>(b) * p.pool.max_pages;
  int ids = lane < mine ? table[page_of(lane)] : -1;  // 32 table entries, one per lane
  int ids_from = 0;
  auto issue = [&](int i) {  // all lanes; brings this warp's i-th page
    if (i - ids_from == 32) {
      ids_from = i;
      ids = i + lane < mine ? table[page_of(i + lane)] : -1;
    }
    const int id = __shfl_sync(0xffffffffu, ids, i - ids_from);
    if (lane == 0) {
      const int st = i % C::kStages;
      const bool good = id >= 0 && id < p.pool.num_pages;
      ok[st] = good;
      if (good) {
        mbar_arrive_expect_tx(bar + 8 * st, P::kBytes);
        bulk_load(ring_s + st * P::kBytes,
                  p.pool.base + (static_cast<int64_t>(id) * p.pool.kv_heads + kvh) * P::kBytes,
                  P::kBytes, bar + 8 * st);
      } else {  // a page outside the pool is reported and not seen
        record_error(p.err, kErrDecodePage);
        mbar_arrive(bar + 8 * st);
      }
    }
  };
  for (int i = 0; i < min(C::kStages, mine); ++i) issue(i);

  // query operand: k-step 2 g + s of the products holds channels 32 g + 8 t + 2 s
  // + {0, 4} (first half) and {1, 5} (second half) of lane t, matching the nibble
  // pairs of a code word; qs_g = sum of q over the group
  uint32_t qa[2 * NG][4];
  float qs[kRows][NG];
#pragma unroll
  for (int hr = 0; hr < 2; ++hr) {
    const int head = r + 8 * hr;
    const bool in = hr < kRows && head < nh;
    const uint4* src = reinterpret_cast<const uint4*>(
        p.q + (static_cast<int64_t>(b) * p.heads + head0 + (in ? head : 0)) * D);
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const uint4 x = in ? src[4 * g + t] : make_uint4(0, 0, 0, 0);  // channels 32 g + 8 t ..+ 7
      qa[2 * g][hr] = __byte_perm(x.x, x.z, 0x5410);          // 0, 4
      qa[2 * g][2 + hr] = __byte_perm(x.x, x.z, 0x7632);      // 1, 5
      qa[2 * g + 1][hr] = __byte_perm(x.y, x.w, 0x5410);      // 2, 6
      qa[2 * g + 1][2 + hr] = __byte_perm(x.y, x.w, 0x7632);  // 3, 7
      if (hr < kRows) {
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          sum += __uint_as_float(w[i] << 16) + __uint_as_float(w[i] & 0xffff0000u);
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        qs[hr < kRows ? hr : 0][g] = sum;
      }
    }
  }

  float m[kRows], l[kRows], om[kRows][NG];  // running max, this lane's sum and sum of p m_g
  float o[D / 8][2 * kRows];                // output: channels 8 i + 2 t, + 1 of heads r (, r + 8)
#pragma unroll
  for (int hr = 0; hr < kRows; ++hr) {
    m[hr] = -INFINITY;
    l[hr] = 0.f;
#pragma unroll
    for (int g = 0; g < NG; ++g) om[hr][g] = 0.f;
  }
#pragma unroll
  for (int i = 0; i < D / 8; ++i)
#pragma unroll
    for (int e = 0; e < 2 * kRows; ++e) o[i][e] = 0.f;

  bool timed_out = false;
  for (int i = 0; i < mine; ++i) {
    const int st = i % C::kStages;
    if (!__all_sync(0xffffffffu, mbar_wait(bar + 8 * st, (i / C::kStages) & 1))) {
      if (lane == 0) record_error(p.err, kErrDecodeWait);
      timed_out = true;
      break;
    }
    if (ok[st]) {
      const uint8_t* pg = ring + st * P::kBytes;
      const int tok0 = page_of(i) * kPage;
      // every token of the page is visible (the rule for all but the edge pages)
      const bool whole = tok0 + kPage <= vis.len && (tok0 >= vis.first || tok0 + kPage <= p.sinks);
      auto seen = [&](int tok) { return tok < vis.len && (tok >= vis.first || tok < p.sinks); };

      // scores of tokens 8 nt + 2 t, + 1
      float s[kRows][4][2];
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) {
        uint32_t w[NG];
        lds_words(w, pg + P::oK + (8 * nt + r) * P::kRow + t * (4 * NG));
        uint32_t par[2][NG];
#pragma unroll
        for (int e = 0; e < 2; ++e)
          lds_words(par[e], pg + P::oKPar + (8 * nt + 2 * t + e) * P::kParRow);
#pragma unroll
        for (int hr = 0; hr < kRows; ++hr) s[hr][nt][0] = s[hr][nt][1] = 0.f;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          float acc[4] = {0.f, 0.f, 0.f, 0.f};
          mma16816(acc, qa[2 * g], codes_bf16<0>(w[g]), codes_bf16<1>(w[g]));
          mma16816(acc, qa[2 * g + 1], codes_bf16<2>(w[g]), codes_bf16<3>(w[g]));
#pragma unroll
          for (int hr = 0; hr < kRows; ++hr)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              // s (acc - 39.5 qs) + m qs
              const float x = fmaf(-39.5f, qs[hr][g], acc[2 * hr + e]);
              s[hr][nt][e] = fmaf(step_of(par[e][g]), x, s[hr][nt][e]);
              s[hr][nt][e] = fmaf(mid_of(par[e][g]), qs[hr][g], s[hr][nt][e]);
            }
        }
        if (!whole) {
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (!seen(tok0 + 8 * nt + 2 * t + e)) {
#pragma unroll
              for (int hr = 0; hr < kRows; ++hr) s[hr][nt][e] = -INFINITY;
            }
        }
      }
#pragma unroll
      for (int hr = 0; hr < kRows; ++hr) {
        float mx = fmaxf(fmaxf(fmaxf(s[hr][0][0], s[hr][0][1]), fmaxf(s[hr][1][0], s[hr][1][1])),
                         fmaxf(fmaxf(s[hr][2][0], s[hr][2][1]), fmaxf(s[hr][3][0], s[hr][3][1])));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        mx *= p.sl2;
        if (__any_sync(0xffffffffu, mx > m[hr])) {
          const float mn = fmaxf(m[hr], mx);
          const float a = m[hr] == -INFINITY ? 0.f : ex2_approx(m[hr] - mn);
          m[hr] = mn;
          l[hr] *= a;
#pragma unroll
          for (int g = 0; g < NG; ++g) om[hr][g] *= a;
#pragma unroll
          for (int c = 0; c < D / 8; ++c) {
            o[c][2 * hr] *= a;
            o[c][2 * hr + 1] *= a;
          }
        }
        const float nm = m[hr] == -INFINITY ? 0.f : -m[hr];
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            s[hr][nt][e] = ex2_approx(fmaf(s[hr][nt][e], p.sl2, nm));
            l[hr] += s[hr][nt][e];
          }
      }
      // values: 16 tokens 16 kk + {2 t, 2 t + 1, 2 t + 8, 2 t + 9} at a time
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        uint32_t a[NG][4], vw[4][NV];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int tok = 16 * kk + 2 * t + (e & 1) + 8 * (e >> 1);
          lds_words(vw[e], pg + P::oV + tok * P::kRow + P::v_chunk(tok, r));
        }
#pragma unroll
        for (int h2 = 0; h2 < 2; ++h2) {  // the two tokens of each operand half
          uint32_t par[2][NG];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int tok = 16 * kk + 2 * t + e + 8 * h2;
            lds_words(par[e], pg + P::oVPar + tok * P::kParRow);
            if (!whole && !seen(tok0 + tok)) {  // unseen tokens may hold anything, NaN too
#pragma unroll
              for (int g = 0; g < NG; ++g) par[e][g] = 0u;
            }
          }
#pragma unroll
          for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int hr = 0; hr < 2; ++hr) {
              if (hr < kRows) {
                const float p0 = s[hr < kRows ? hr : 0][2 * kk + h2][0];
                const float p1 = s[hr < kRows ? hr : 0][2 * kk + h2][1];
                a[g][2 * h2 + hr] = pack_bf16(p0 * step_of(par[0][g]), p1 * step_of(par[1][g]));
                float& acc = om[hr < kRows ? hr : 0][g];
                acc = fmaf(p0, mid_of(par[0][g]), acc);
                acc = fmaf(p1, mid_of(par[1][g]), acc);
              } else {
                a[g][2 * h2 + hr] = 0u;
              }
            }
        }
#pragma unroll
        for (int w = 0; w < NV; ++w) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {  // nibbles 0-3, 4-7: channel groups 2 w, 2 w + 1
            const uint32_t sel = half ? 0x7632u : 0x5410u;
            const uint32_t x = __byte_perm(vw[0][w], vw[1][w], sel);
            const uint32_t y = __byte_perm(vw[2][w], vw[3][w], sel);
            const uint32_t b0[4] = {centred_bf16<0>(x), centred_bf16<1>(x), centred_bf16<2>(x),
                                    centred_bf16<3>(x)};
            const uint32_t b1[4] = {centred_bf16<0>(y), centred_bf16<1>(y), centred_bf16<2>(y),
                                    centred_bf16<3>(y)};
#pragma unroll
            for (int n = 0; n < 4; ++n) {
              const int c = 8 * w + 4 * half + n;
              float d[4] = {o[c][0], o[c][1], kRows == 2 ? o[c][kRows == 2 ? 2 : 0] : 0.f,
                            kRows == 2 ? o[c][kRows == 2 ? 3 : 0] : 0.f};
              mma16816(d, a[2 * w + half], b0[n], b1[n]);
#pragma unroll
              for (int e = 0; e < 2 * kRows; ++e) o[c][e] = d[e];
            }
          }
        }
      }
    }
    __syncwarp();  // every lane has read the stage: it may be refilled
    if (i + C::kStages < mine) issue(i + C::kStages);
  }
  if (timed_out) {  // copies still in flight must land before the block may exit
    for (int i = 0; i < C::kStages; ++i) mbar_wait(bar + 8 * i, 0);
  }

  // the lanes t of a head hold different tokens' sums
#pragma unroll
  for (int hr = 0; hr < kRows; ++hr) {
    l[hr] += __shfl_xor_sync(0xffffffffu, l[hr], 1);
    l[hr] += __shfl_xor_sync(0xffffffffu, l[hr], 2);
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      om[hr][g] += __shfl_xor_sync(0xffffffffu, om[hr][g], 1);
      om[hr][g] += __shfl_xor_sync(0xffffffffu, om[hr][g], 2);
    }
  }
  __syncthreads();  // every warp is done with its ring
  float* join = reinterpret_cast<float*>(smem);  // [warp][head][d], then [warp][head] (m, l)
  float2* join_ml = reinterpret_cast<float2*>(join + kWarps * kHeads * D);
#pragma unroll
  for (int hr = 0; hr < kRows; ++hr) {
    const int head = r + 8 * hr;
    float* dst = join + (warp * kHeads + head) * D;
#pragma unroll
    for (int c = 0; c < D / 8; ++c)
      *reinterpret_cast<float2*>(dst + 8 * c + 2 * t) =
          make_float2(o[c][2 * hr] + om[hr][c / 4], o[c][2 * hr + 1] + om[hr][c / 4]);
    if (t == 0) join_ml[warp * kHeads + head] = make_float2(m[hr], l[hr]);
  }
  __syncthreads();
  for (int idx = threadIdx.x; idx < nh * (D / 2); idx += kThreads) {
    const int head = idx / (D / 2), c = idx % (D / 2);
    float mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, join_ml[w * kHeads + head].x);
    float sum = 0.f;
    float2 acc = make_float2(0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 ml = join_ml[w * kHeads + head];
      if (ml.x == -INFINITY) continue;  // this warp saw no token
      const float f = ex2_approx(ml.x - mx);
      const float2 x = *reinterpret_cast<const float2*>(join + (w * kHeads + head) * D + 2 * c);
      sum = fmaf(ml.y, f, sum);
      acc.x = fmaf(x.x, f, acc.x);
      acc.y = fmaf(x.y, f, acc.y);
    }
    const int64_t row = static_cast<int64_t>(b) * p.heads + head0 + head;
    if (p.splits > 1) {
      *reinterpret_cast<float2*>(p.part + (row * p.splits + split) * D + 2 * c) = acc;
      if (c == 0) p.part_ml[row * p.splits + split] = make_float2(mx, sum);
    } else {
      const bool has = mx != -INFINITY;  // an empty sequence: 0 and -inf
      const float inv = has ? 1.f / sum : 0.f;
      *reinterpret_cast<uint32_t*>(p.o + row * D + 2 * c) =
          has ? pack_bf16(acc.x * inv, acc.y * inv) : 0u;
      if (c == 0 && p.lse) p.lse[row] = has ? (mx + log2f(sum)) * kLn2 : -INFINITY;
    }
  }
}

// Joins the shares of a row: one warp per (sequence, head).
template <int D>
__global__ void __launch_bounds__(128) kv4_join_kernel(const Params p, int rows) {
  pdl_trigger();
  pdl_wait();
  const int row = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (row >= rows) return;
  const float2* ml = p.part_ml + static_cast<int64_t>(row) * p.splits;
  const float* part = p.part + static_cast<int64_t>(row) * p.splits * D;
  float mx = -INFINITY;
  for (int s = lane; s < p.splits; s += 32) mx = fmaxf(mx, ml[s].x);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
  float sum = 0.f, acc[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) acc[i] = 0.f;
  for (int s = 0; s < p.splits; ++s) {
    const float2 x = ml[s];
    if (x.x == -INFINITY) continue;
    const float f = ex2_approx(x.x - mx);
    sum = fmaf(x.y, f, sum);
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      const float2 v = *reinterpret_cast<const float2*>(part + static_cast<int64_t>(s) * D +
                                                        64 * i + 2 * lane);
      acc[2 * i] = fmaf(v.x, f, acc[2 * i]);
      acc[2 * i + 1] = fmaf(v.y, f, acc[2 * i + 1]);
    }
  }
  const bool has = mx != -INFINITY;
  const float inv = has ? 1.f / sum : 0.f;
#pragma unroll
  for (int i = 0; i < D / 64; ++i)
    *reinterpret_cast<uint32_t*>(p.o + static_cast<int64_t>(row) * D + 64 * i + 2 * lane) =
        has ? pack_bf16(acc[2 * i] * inv, acc[2 * i + 1] * inv) : 0u;
  if (lane == 0 && p.lse) p.lse[row] = has ? (mx + log2f(sum)) * kLn2 : -INFINITY;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Pages that a sequence can have visible at most.
int64_t most_pages(const Kv4DecodeArgs& a) {
  const int64_t w = ceil_div(a.window, kPage) + 1, s = ceil_div(a.sinks, kPage);
  return w + s < a.max_pages ? w + s : a.max_pages;
}

// Shares per sequence and head: enough blocks to fill the GPU, each with a few
// pages for every warp.
int splits_for(const Kv4DecodeArgs& a) {
  const int64_t blocks =
      static_cast<int64_t>(a.batch) * a.kv_heads * ceil_div(a.heads / a.kv_heads, kHeads);
  const int64_t want = ceil_div(148 * 6, blocks);
  const int64_t most = ceil_div(most_pages(a), 4 * kWarps);
  const int64_t s = want < most ? want : most;
  return static_cast<int>(s < 1 ? 1 : (s > 256 ? 256 : s));
}

template <int D, int kRows>
cudaError_t launch_main(const Params& p, dim3 grid, cudaStream_t stream) {
  cudaError_t e = cudaFuncSetAttribute(kv4_decode_kernel<D, kRows>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kv4_decode_kernel<D, kRows>, grid, dim3(kThreads), Cfg<D>::kSmem, stream, p);
}

template <int D>
cudaError_t run(const Kv4DecodeArgs& a, cudaStream_t stream) {
  Params p;
  p.pool = Pool{static_cast<uint8_t*>(const_cast<void*>(a.cache)), a.table, a.max_pages,
                a.num_pages, a.kv_heads};
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.o = static_cast<__nv_bfloat16*>(a.o);
  p.lse = a.lse;
  p.lengths = a.lengths;
  p.err = a.err;
  p.heads = a.heads;
  p.group = a.heads / a.kv_heads;
  p.head_blocks = (p.group + kHeads - 1) / kHeads;
  p.splits = splits_for(a);
  p.window = a.window;
  p.sinks = a.sinks;
  p.sl2 = kLog2e / sqrtf(static_cast<float>(D));
  const int64_t rows = static_cast<int64_t>(a.batch) * a.heads;
  p.part = static_cast<float*>(a.workspace);
  p.part_ml = reinterpret_cast<float2*>(p.part + rows * p.splits * D);
  const int64_t blocks = static_cast<int64_t>(a.batch) * a.kv_heads * p.head_blocks * p.splits;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(blocks));
  cudaError_t e = p.group <= 8 ? launch_main<D, 1>(p, grid, stream)
                               : launch_main<D, 2>(p, grid, stream);
  if (e != cudaSuccess || p.splits == 1) return e;
  return launch_pdl(kv4_join_kernel<D>, dim3(static_cast<unsigned>((rows + 3) / 4)), dim3(128), 0,
                    stream, p, static_cast<int>(rows));
}

}  // namespace

size_t kv4_decode_workspace_bytes(const Kv4DecodeArgs& a) {
  const int splits = splits_for(a);
  if (splits == 1) return 0;
  return static_cast<size_t>(a.batch) * a.heads * splits * (a.d + 2) * 4;
}

cudaError_t launch_kv4_decode(const Kv4DecodeArgs& a, cudaStream_t stream) {
  return a.d == 64 ? run<64>(a, stream) : run<128>(a, stream);
}

}  // namespace nb
