// Attention of one query token per sequence over the 4-bit cache, with a
// sliding window and visible first tokens (layout of the cache in kv4.cuh).
//
// With key value k_j = m_jg + s_jg (c - 7.5) on channel group g,
//   q . k_j = sum_g s_jg (q_g . c_jg - 7.5 sum(q_g)) + sum_g m_jg sum(q_g)
//   O = sum_j p_j v_j = sum_j (p_j s_jg)(c - 7.5) + sum_j p_j m_jg
// so the codes themselves are the operands of warp matrix products (m16n8k16): no
// row is ever dequantised in memory, and s and m enter in fp32 outside them.  A
// nibble alone in a bf16 is a subnormal number, exactly (even_codes, below).
//   Scores: rows = 16 tokens, columns = 8 query heads that share the key/value
//   head; the products start from -7.5 sum(q_g).  sum_g m_jg sum(q_g) is one
//   product more, over the bf16 midpoints and sum(q_g) cut into three bf16 parts
//   (24 bits).
//   Values: rows = 16 channels, columns = 8 heads; here the offset is subtracted
//   from the codes before the product (exact in bf16), because the output sums
//   over many tokens and would cancel.  p s is rounded to bf16 and transposed
//   within the warp to become the operand (the output is bf16 and every token's
//   error is its own); softmax statistics, sum p m and the outputs are fp32.
//
// A block of four warps takes one key/value head of one sequence and a share of
// its visible pages (the pages of the sinks, then those of the window); warp w
// takes every fourth page, brought by one bulk copy each into the warp's own
// ring, and keeps its own maximum, sum and output.  The warps, and then the
// shares, are joined by their maxima.  It cannot do without the page bytes, once; what
// sets its time is arithmetic, 690 instructions a page and warp (DRAM is at 24 to 32 %
// of its rate), and 6 to 8 us that every block takes to start and to join.
#include <math.h>

#include <type_traits>

#include "kv4.cuh"
#include "serving.cuh"

namespace nb {
namespace {

using namespace kv4;
using namespace sm100;

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kHeads = 16;  // query heads of one block (two sets of a product's eight columns)
constexpr int kMinShare = kWarps;  // pages of a share, at least: one for each warp
constexpr float kTau = 8.0f;           // lazy-rescale threshold, log2 units
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <int D>
struct Cfg {
  using P = Page<D>;
  static constexpr int kStages = D == 64 ? 3 : 4;
  static constexpr int kRing = kWarps * kStages * P::kBytes;
  // the warps' results take the place of the ring when the pages are done
  // (rows of D + 4 floats: the lanes of a store fall into different banks)
  static constexpr int kJoinRow = D + 4;
  static constexpr int kJoin = kHeads * (kWarps * (kJoinRow + 2 + P::kGroups) + 2) * 4;
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
  int* err;   // a wait that ran out
  int* skip;  // a page that is not mapped
  int heads, group, head_blocks, splits, window, sinks;
  bool cluster;  // the shares of a row are one cluster
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

// A nibble alone in a bf16 is a number: the least significant bit of the exponent
// goes on where the mantissa of the subnormals ends, so c in bits 0-3 is c 2^-133 and
// c in bits 4-7 is c 2^-129, exactly.  One `and` yields a pair of codes of two halves.
__device__ __forceinline__ uint32_t even_codes(uint32_t w) { return w & 0x000f000fu; }
__device__ __forceinline__ uint32_t odd_codes(uint32_t w) { return w & 0x00f000f0u; }

__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {  // two bf16 products
  const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                   *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// The codes times 2^127 less their centre: (c - 7.5) / 64 of the even ones, (c - 7.5) / 4
// of the odd ones, exact.
constexpr float kEvenUnit = 64.f, kOddUnit = 4.f;
__device__ __forceinline__ uint32_t centred(uint32_t codes, uint32_t centre) {
  const uint32_t up = 0x7f007f00u;
  const __nv_bfloat162 r = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&codes),
                                   *reinterpret_cast<const __nv_bfloat162*>(&up),
                                   *reinterpret_cast<const __nv_bfloat162*>(&centre));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t centred_even(uint32_t w) {
  return centred(even_codes(w), 0xbdf0bdf0u);  // -7.5 / 64
}
__device__ __forceinline__ uint32_t centred_odd(uint32_t w) {
  return centred(odd_codes(w), 0xbff0bff0u);  // -7.5 / 4
}

constexpr int kBigQuery = 112, kBigUnit = 16;  // (see the query operand)

__device__ __forceinline__ float pow2(int e) {  // -126 <= e <= 127
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
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

// The 8 x 8 matrix of 16-bit values held two a lane (row r, columns 2 t, 2 t + 1),
// transposed.
__device__ __forceinline__ uint32_t transpose_b16(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

constexpr int kMaxCluster = 8;  // blocks of a cluster on every device

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
// Two floats at this block's shared-memory address `at`, in block `rank` of the cluster.
__device__ __forceinline__ float2 load_cluster(uint32_t at, int rank) {
  float2 v;
  asm volatile(
      "{\n\t.reg .b32 a;\n\t"
      "mapa.shared::cluster.u32 a, %2, %3;\n\t"
      "ld.shared::cluster.v2.f32 {%0, %1}, [a];\n\t}"
      : "=f"(v.x), "=f"(v.y)
      : "r"(at), "r"(rank)
      : "memory");
  return v;
}

// Channels 2 c, 2 c + 1 of a finished row; an empty sequence gives 0 and -inf.
__device__ __forceinline__ void store_row(const Params& p, int d, int64_t row, int c, float2 acc,
                                          float mx, float sum) {
  const bool has = mx != -INFINITY;
  const float inv = has ? 1.f / sum : 0.f;
  *reinterpret_cast<uint32_t*>(p.o + row * d + 2 * c) =
      has ? pack_bf16(acc.x * inv, acc.y * inv) : 0u;
  if (c == 0 && p.lse) p.lse[row] = has ? (mx + log2f(sum)) * kLn2 : -INFINITY;
}

// Blocks that should fit an SM at once (registers; the shared memory follows).  At
// d = 128 two blocks of 200 registers schedule better than three of 168: 57 us against
// 62 at 32 ragged contexts of up to 8192 tokens, 45 either way at one of 2^20; four of
// 128 take 79 and 58.  At d = 64 five blocks of 96 take 22.3 us where four take 18.5
// (64 streams x 4100 visible tokens), and three 18.5.  Two sets of heads (16 share the
// cache): at d = 64 three blocks take 57.4 us at 32 ragged contexts and 46.1 at one of
// 2^20, two 62 and 60.4, four 63.5 and 49; at d = 128 one or two (the kernel wants 255
// registers either way) 93.0 and 68.6, three 111 and 89.
constexpr int blocks_per_sm(int d, int sets) { return d == 64 ? (sets == 1 ? 4 : 3) : 2; }

// kSets: sets of eight heads (the columns of a product): 1 when at most eight
// share the cache, 2 otherwise.
template <int D, int kSets>
__global__ void __launch_bounds__(kThreads, blocks_per_sm(D, kSets)) kv4_decode_kernel(const Params p) {
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
  const int share = max(kMinShare, (vis.count + p.splits - 1) / p.splits);
  const int i0 = min(split * share, vis.count), i1 = min(i0 + share, vis.count);
  const int mine = i1 - i0 > warp ? (i1 - i0 - warp + kWarps - 1) / kWarps : 0;  // this warp's pages
  auto page_of = [&](int i) {  // logical page of this warp's i-th page
    const int x = i0 + warp + i * kWarps;
    return x < vis.sink_pages ? x : vis.page0 + (x - vis.sink_pages);
  };
  const int32_t* table = p.pool.table + static_cast<int64_t>(b) * p.pool.max_pages;
  int ids = lane < mine ? table[page_of(lane)] : -1;  // 32 table entries, one per lane
  int ids_from = 0;
  auto issue = [&](int i, int st) {  // all lanes; brings this warp's i-th page into stage st
    if (i - ids_from == 32) {
      ids_from = i;
      ids = i + lane < mine ? table[page_of(i + lane)] : -1;
    }
    const int id = __shfl_sync(0xffffffffu, ids, i - ids_from);
    if (lane == 0) {
      const bool good = id >= 0 && id < p.pool.num_pages;
      ok[st] = good;
      if (good) {
        mbar_arrive_expect_tx(bar + 8 * st, P::kBytes);
        bulk_load(ring_s + st * P::kBytes,
                  p.pool.base + (static_cast<int64_t>(id) * p.pool.kv_heads + kvh) * P::kBytes,
                  P::kBytes, bar + 8 * st);
      } else {  // a page outside the pool is reported and not seen
        record_error(p.skip, kErrDecodePage);
        mbar_arrive(bar + 8 * st);
      }
    }
  };
  for (int i = 0; i < min(C::kStages, mine); ++i) issue(i, i);

  // query operand: k-step 2 g + i of the products holds channels 32 g + 8 t + 2 i
  // + {0, 4} (first half) and {1, 5} (second half) of lane t, matching the nibble
  // pairs of a code word.  With 2^e the largest power of two in the head's row, the
  // operands are q 2^(126 - e) for the even codes (c 2^-133) and a sixteenth of it for
  // the odd ones (c 2^-129): the products are q c 2^(-7 - e), and the scores carry that
  // factor until sl2 takes it out.  That takes up to 2^134, which is no float: heads with
  // e > kBigQuery have kBigUnit of it multiplied into their scores first.
  // off_g = -7.5 sum(q_g) of heads 2 t, 2 t + 1.
  constexpr int NP = NG / 2;
  uint32_t qb[kSets][2 * NG][2], qm[kSets][2];
  float off[kSets][NG][2], sl2[kSets][2];
  uint32_t big = 0;  // bit 2 hs + j: such a head
#pragma unroll
  for (int hs = 0; hs < kSets; ++hs) {
    const int head = r + 8 * hs;
    const bool in = head < nh;
    const uint4* src = reinterpret_cast<const uint4*>(
        p.q + (static_cast<int64_t>(b) * p.heads + head0 + (in ? head : 0)) * D);
    uint4 x[NG];
    uint32_t top = 0;  // the largest magnitude: bf16 bits order like integers
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      x[g] = in ? src[4 * g + t] : make_uint4(0, 0, 0, 0);  // channels 32 g + 8 t ..+ 7
      const uint32_t w[4] = {x[g].x, x[g].y, x[g].z, x[g].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) top = __vmaxu2(top, w[i] & 0x7fff7fffu);
    }
    top = max(top & 0xffffu, top >> 16);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    // subnormal rows count as 2^-126, infinite ones as 2^127 (their scores are no numbers)
    const int e = min(max(static_cast<int>(top >> 7), 1), 254) - 127;
    const uint32_t down1 = e == 127 ? 0x0040u : static_cast<uint32_t>(127 - e) << 7;  // 2^-e
    const uint32_t down = down1 | down1 << 16;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int ej = __shfl_sync(0xffffffffu, e, 8 * t + 4 * j);
      if (ej > kBigQuery) big |= 1u << (2 * hs + j);
      const int n = 7 + ej - (ej > kBigQuery ? kBigUnit : 0);
      sl2[hs][j] = p.sl2 * pow2(n / 2) * pow2(n - n / 2);
    }
    float qs[NG];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const uint32_t w[4] = {mul2(x[g].x, down), mul2(x[g].y, down), mul2(x[g].z, down),
                             mul2(x[g].w, down)};  // below 2
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        sum += __uint_as_float(w[i] << 16) + __uint_as_float(w[i] & 0xffff0000u);
#pragma unroll
      for (int i = 0; i < 2; ++i) {  // 0, 4 and 1, 5; then 2, 6 and 3, 7
        qb[hs][2 * g + i][0] = mul2(__byte_perm(w[i], w[i + 2], 0x5410), 0x7e807e80u);  // 2^126
        qb[hs][2 * g + i][1] = mul2(__byte_perm(w[i], w[i + 2], 0x7632), 0x7c807c80u);  // 2^122
      }
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      sum *= 0.0078125f;
      qs[g] = sum;
      off[hs][g][0] = -7.5f * __shfl_sync(0xffffffffu, sum, 8 * t);
      off[hs][g][1] = -7.5f * __shfl_sync(0xffffffffu, sum, 8 * t + 4);
    }
    // lane t of the midpoint product multiplies the pair (m_2u, m_2u+1), u = t mod
    // NP, by part t / NP of the sums (and by one part more in its second half)
    const int u = t % NP, part = t / NP;
    float x0 = u == 0 ? qs[0] : qs[NG - 2], x1 = u == 0 ? qs[1] : qs[NG - 1];
    uint32_t parts[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      parts[i] = pack_bf16(x0, x1);
      x0 -= __uint_as_float(parts[i] << 16);
      x1 -= __uint_as_float(parts[i] & 0xffff0000u);
    }
    qm[hs][0] = part == 0 ? parts[0] : part == 1 ? parts[1] : part == 2 ? parts[2] : 0u;
    qm[hs][1] = NP == 2 && part == 0 ? parts[2] : 0u;
  }

  const bool any_big = __any_sync(0xffffffffu, big != 0);

  // of heads 2 t + j (+ 8 hs): the maximum in use, this lane's sums of p and of p m_g
  // (its tokens are 16 i + r, + 8), and the output at channels 16 i + r, + 8
  float m[kSets][2], l[kSets][2], om[kSets][2][NG], o[kSets][D / 16][4];
#pragma unroll
  for (int hs = 0; hs < kSets; ++hs) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      m[hs][j] = -INFINITY;
      l[hs][j] = 0.f;
#pragma unroll
      for (int g = 0; g < NG; ++g) om[hs][j][g] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[hs][i][e] = 0.f;
  }

  // One page; kWhole: every token of it is visible (all but the edge pages), which
  // keeps the common path free of branches.
  auto page = [&](const uint8_t* pg, int tok0, auto whole_tag) {
    constexpr bool kWhole = decltype(whole_tag)::value;
    auto seen = [&](int tok) {
      return tok0 + tok < vis.len && (tok0 + tok >= vis.first || tok0 + tok < p.sinks);
    };
    float s[kSets][2][4];  // scores of tokens 16 mt + r (heads 2 t, 2 t + 1) and + 8
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      uint32_t w[2][NG], par[2][NG], mw[2][2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int tok = 16 * mt + 8 * e + r;
        lds_words(w[e], pg + P::oK + tok * P::kRow + t * (4 * NG));
        lds_words(par[e], pg + P::oKPar + tok * P::kParRow);
        lds_words(mw[e], pg + P::oKPar + tok * P::kParRow + (t % NP) * 8);
      }
      const uint32_t m0 = __byte_perm(mw[0][0], mw[0][1], 0x7632);
      const uint32_t m1 = __byte_perm(mw[1][0], mw[1][1], 0x7632);
      const uint32_t ma[4] = {m0, m1, m0, m1};
      const float zero[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int hs = 0; hs < kSets; ++hs)
        mma16816(s[hs][mt], ma, qm[hs][0], qm[hs][1], zero);  // sum_g m_g sum(q_g)
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const uint32_t h0 = w[0][g] >> 8, h1 = w[1][g] >> 8;
        const uint32_t a0[4] = {even_codes(w[0][g]), even_codes(w[1][g]), odd_codes(w[0][g]),
                                odd_codes(w[1][g])};
        const uint32_t a1[4] = {even_codes(h0), even_codes(h1), odd_codes(h0), odd_codes(h1)};
        const float st0 = step_of(par[0][g]), st1 = step_of(par[1][g]);
#pragma unroll
        for (int hs = 0; hs < kSets; ++hs) {
          float acc[4] = {off[hs][g][0], off[hs][g][1], off[hs][g][0], off[hs][g][1]};
          mma16816(acc, a0, qb[hs][2 * g][0], qb[hs][2 * g][1], acc);
          mma16816(acc, a1, qb[hs][2 * g + 1][0], qb[hs][2 * g + 1][1], acc);
          s[hs][mt][0] = fmaf(st0, acc[0], s[hs][mt][0]);
          s[hs][mt][1] = fmaf(st0, acc[1], s[hs][mt][1]);
          s[hs][mt][2] = fmaf(st1, acc[2], s[hs][mt][2]);
          s[hs][mt][3] = fmaf(st1, acc[3], s[hs][mt][3]);
        }
      }
      if (any_big) {
#pragma unroll
        for (int hs = 0; hs < kSets; ++hs)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            s[hs][mt][e] *= big >> (2 * hs + (e & 1)) & 1 ? pow2(kBigUnit) : 1.f;
      }
      if (!kWhole) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const bool v = seen(16 * mt + 8 * e + r);
#pragma unroll
          for (int hs = 0; hs < kSets; ++hs)
#pragma unroll
            for (int j = 0; j < 2; ++j)
              s[hs][mt][2 * e + j] = v ? s[hs][mt][2 * e + j] : -INFINITY;
        }
      }
    }
#pragma unroll
    for (int hs = 0; hs < kSets; ++hs) {
      float mx[2];
#pragma unroll
      for (int j = 0; j < 2; ++j)
        mx[j] = sl2[hs][j] * max_nan(max_nan(s[hs][0][j], s[hs][0][2 + j]),
                                     max_nan(s[hs][1][j], s[hs][1][2 + j]));
      // the maximum in use may lag by 2^8: exact after the final division.  A score that
      // is no number becomes the maximum, and the output then is none either.
      if (__any_sync(0xffffffffu, !(mx[0] <= m[hs][0] + kTau && mx[1] <= m[hs][1] + kTau))) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1)  // over the lanes that hold the page's other tokens
#pragma unroll
          for (int j = 0; j < 2; ++j)
            mx[j] = max_nan(mx[j], __shfl_xor_sync(0xffffffffu, mx[j], x));
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float mn = max_nan(m[hs][j], mx[j]);
          const float a = m[hs][j] == -INFINITY ? 0.f : ex2_approx(m[hs][j] - mn);
          m[hs][j] = mn;
          l[hs][j] *= a;
#pragma unroll
          for (int g = 0; g < NG; ++g) om[hs][j][g] *= a;
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            o[hs][c][j] *= a;
            o[hs][c][2 + j] *= a;
          }
        }
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float nm = m[hs][j] == -INFINITY ? 0.f : -m[hs][j];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float& x = s[hs][i >> 1][2 * (i & 1) + j];
          x = ex2_approx(fmaf(x, sl2[hs][j], nm));
          l[hs][j] += x;
        }
      }
    }
    // values: 16 tokens at a time
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      uint32_t ps[kSets][NG][2], vw[4][NV];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int tok = 16 * kk + 8 * e + r;
        uint32_t par[NG];
        lds_words(par, pg + P::oVPar + tok * P::kParRow);
        if (!kWhole && !seen(tok)) {  // unseen tokens may hold anything, NaN too
#pragma unroll
          for (int g = 0; g < NG; ++g) par[g] = 0u;
        }
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const float step = step_of(par[g]), mid = mid_of(par[g]);
#pragma unroll
          for (int hs = 0; hs < kSets; ++hs) {
            const float p0 = s[hs][kk][2 * e], p1 = s[hs][kk][2 * e + 1];
            ps[hs][g][e] = transpose_b16(pack_bf16(p0 * step, p1 * step));
            om[hs][0][g] = fmaf(p0, mid, om[hs][0][g]);
            om[hs][1][g] = fmaf(p1, mid, om[hs][1][g]);
          }
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {  // the operand's tokens 2 t, 2 t + 1, 2 t + 8, 2 t + 9
        const int tok = 16 * kk + 2 * t + (e & 1) + 8 * (e >> 1);
        lds_words(vw[e], pg + P::oV + tok * P::kRow + P::v_chunk(tok, r));
      }
#pragma unroll
      for (int w = 0; w < NV; ++w) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {  // nibbles 0-3, 4-7: channel groups 2 w, 2 w + 1
          const uint32_t sel = half ? 0x7632u : 0x5410u;
          const uint32_t x = __byte_perm(vw[0][w], vw[1][w], sel);
          const uint32_t y = __byte_perm(vw[2][w], vw[3][w], sel);
          const uint32_t x8 = x >> 8, y8 = y >> 8;
          const uint32_t a0[4] = {centred_even(x), centred_odd(x), centred_even(y), centred_odd(y)};
          const uint32_t a1[4] = {centred_even(x8), centred_odd(x8), centred_even(y8),
                                  centred_odd(y8)};
          const int g = 2 * w + half;
#pragma unroll
          for (int hs = 0; hs < kSets; ++hs) {
            mma16816(o[hs][2 * g], a0, ps[hs][g][0], ps[hs][g][1], o[hs][2 * g]);
            mma16816(o[hs][2 * g + 1], a1, ps[hs][g][0], ps[hs][g][1], o[hs][2 * g + 1]);
          }
        }
      }
    }
  };

  int st = 0, phase = 0;
  for (int i = 0; i < mine; ++i) {
    if (!__all_sync(0xffffffffu, mbar_wait(bar + 8 * st, phase))) {
      if (lane == 0) record_error(p.err, kErrDecodeWait);
      // copies still in flight must land before the ring is reused and the block exits
      drain_pages<C::kStages>(i, mine, [&](int s, uint32_t ph) { mbar_wait(bar + 8 * s, ph); });
      break;
    }
    if (ok[st]) {
      const int tok0 = page_of(i) * kPage;
      const uint8_t* pg = ring + st * P::kBytes;
      if (tok0 + kPage <= vis.len && (tok0 >= vis.first || tok0 + kPage <= p.sinks))
        page(pg, tok0, std::true_type{});
      else
        page(pg, tok0, std::false_type{});
    }
    __syncwarp();  // every lane has read the stage: it may be refilled
    if (i + C::kStages < mine) issue(i + C::kStages, st);
    if (++st == C::kStages) {
      st = 0;
      phase ^= 1;
    }
  }

  __syncthreads();  // every warp is done with its ring
  float* join = reinterpret_cast<float*>(smem);  // [warp][head][d], then (m, l), then sum p m_g
  float2* join_ml = reinterpret_cast<float2*>(join + kWarps * kHeads * C::kJoinRow);
  float2* share_ml = join_ml + kWarps * kHeads;  // [head] (m, l) of the whole block
  float* join_om = reinterpret_cast<float*>(share_ml + kHeads);
#pragma unroll
  for (int hs = 0; hs < kSets; ++hs) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int at = warp * kHeads + 8 * hs + 2 * t + j;
      // the lanes r of a head hold different tokens' sums
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) {
        l[hs][j] += __shfl_xor_sync(0xffffffffu, l[hs][j], x);
#pragma unroll
        for (int g = 0; g < NG; ++g)
          om[hs][j][g] += __shfl_xor_sync(0xffffffffu, om[hs][j][g], x);
      }
      if (r == 0) {
        join_ml[at] = make_float2(m[hs][j], l[hs][j]);
#pragma unroll
        for (int g = 0; g < NG; ++g) join_om[at * NG + g] = om[hs][j][g];
      }
      float* dst = join + at * C::kJoinRow + r;
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
        dst[16 * c] = kEvenUnit * o[hs][c][j];
        dst[16 * c + 8] = kOddUnit * o[hs][c][2 + j];
      }
    }
  }
  __syncthreads();
  for (int idx = threadIdx.x; idx < nh * (D / 2); idx += kThreads) {
    const int head = idx / (D / 2), c = idx % (D / 2);
    float mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mx = max_nan(mx, join_ml[w * kHeads + head].x);
    float sum = 0.f;
    float2 acc = make_float2(0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const int at = w * kHeads + head;
      const float2 ml = join_ml[at];
      if (ml.x == -INFINITY) continue;  // this warp saw no token
      const float f = ex2_approx(ml.x - mx);
      const float2 x = *reinterpret_cast<const float2*>(join + at * C::kJoinRow + 2 * c);
      const float mid = join_om[at * NG + c / 16];
      sum = fmaf(ml.y, f, sum);
      acc.x = fmaf(x.x + mid, f, acc.x);
      acc.y = fmaf(x.y + mid, f, acc.y);
    }
    if (p.splits == 1) {
      store_row(p, D, static_cast<int64_t>(b) * p.heads + head0 + head, c, acc, mx, sum);
    } else if (p.cluster) {  // this thread alone read the place it writes
      *reinterpret_cast<float2*>(join + head * C::kJoinRow + 2 * c) = acc;
      if (c == 0) share_ml[head] = make_float2(mx, sum);
    } else {
      const int64_t at = (static_cast<int64_t>(b) * p.heads + head0 + head) * p.splits + split;
      *reinterpret_cast<float2*>(p.part + at * D + 2 * c) = acc;
      if (c == 0) p.part_ml[at] = make_float2(mx, sum);
    }
  }
  if (!p.cluster) return;
  // the blocks of the cluster hold the shares of the same rows: each joins a part of
  // the output from all blocks' shared memory
  cluster_sync();
  for (int idx = split * kThreads + threadIdx.x; idx < nh * (D / 2);
       idx += p.splits * kThreads) {
    const int head = idx / (D / 2), c = idx % (D / 2);
    const uint32_t at_ml = smem_u32(share_ml + head);
    const uint32_t at = smem_u32(join + head * C::kJoinRow + 2 * c);
    float2 ml[kMaxCluster], x[kMaxCluster];
    float mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < kMaxCluster; ++i)
      if (i < p.splits) {
        ml[i] = load_cluster(at_ml, i);
        x[i] = load_cluster(at, i);
        mx = max_nan(mx, ml[i].x);
      }
    float sum = 0.f;
    float2 acc = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kMaxCluster; ++i)
      if (i < p.splits && ml[i].x != -INFINITY) {
        const float f = ex2_approx(ml[i].x - mx);
        sum = fmaf(ml[i].y, f, sum);
        acc.x = fmaf(x[i].x, f, acc.x);
        acc.y = fmaf(x[i].y, f, acc.y);
      }
    store_row(p, D, static_cast<int64_t>(b) * p.heads + head0 + head, c, acc, mx, sum);
  }
  cluster_sync();  // no block leaves while another reads its shared memory
}

// Joins the shares of a row: one block per (sequence, head), a share to each
// D / 4 threads at a time, then the threads' sums in order.
template <int D, int kJoinWarps>
__global__ void __launch_bounds__(32 * kJoinWarps) kv4_join_kernel(const Params p) {
  constexpr int kPer = 32 / (D / 4);  // shares that a warp reads at once, 16 bytes a lane
  constexpr int kAll = kJoinWarps * kPer;
  __shared__ float4 acc_s[kAll][D / 4];
  __shared__ float sum_s[kAll], max_s[kJoinWarps];
  pdl_trigger();
  pdl_wait();
  const int row = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = threadIdx.x / (D / 4), c = threadIdx.x % (D / 4);
  const float2* ml = p.part_ml + static_cast<int64_t>(row) * p.splits;
  const float4* part =
      reinterpret_cast<const float4*>(p.part + static_cast<int64_t>(row) * p.splits * D) + c;
  float mx = -INFINITY;
  for (int s = threadIdx.x; s < p.splits; s += 32 * kJoinWarps) mx = max_nan(mx, ml[s].x);
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, x));
  if (lane == 0) max_s[warp] = mx;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) mx = max_nan(mx, max_s[w]);
  const bool has = mx != -INFINITY;  // some share saw a token
  float sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int s = sub; s < p.splits; s += kAll) {
    const float2 x = ml[s];
    const float4 v = part[static_cast<int64_t>(s) * (D / 4)];
    const float f = x.x == -INFINITY ? 0.f : ex2_approx(x.x - mx);  // 0: a share without a token
    sum = fmaf(x.y, f, sum);
    acc.x = fmaf(v.x, f, acc.x);
    acc.y = fmaf(v.y, f, acc.y);
    acc.z = fmaf(v.z, f, acc.z);
    acc.w = fmaf(v.w, f, acc.w);
  }
  acc_s[sub][c] = acc;
  if (c == 0) sum_s[sub] = sum;
  __syncthreads();
  if (sub > 0) return;
#pragma unroll
  for (int w = 1; w < kAll; ++w) {
    const float4 v = acc_s[w][c];
    acc.x += v.x;
    acc.y += v.y;
    acc.z += v.z;
    acc.w += v.w;
    sum += sum_s[w];
  }
  const float inv = has ? 1.f / sum : 0.f;
  *reinterpret_cast<uint2*>(p.o + static_cast<int64_t>(row) * D + 4 * c) =
      has ? make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv))
          : make_uint2(0u, 0u);
  if (c == 0 && p.lse) p.lse[row] = has ? (mx + log2f(sum)) * kLn2 : -INFINITY;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Pages that a sequence can have visible at most.
int64_t most_pages(const Kv4DecodeArgs& a) {
  const int64_t w = ceil_div(a.window, kPage) + 1, s = ceil_div(a.sinks, kPage);
  return w + s < a.max_pages ? w + s : a.max_pages;
}

// Shares per sequence and head: enough blocks to fill the GPU once (with twice as many
// the next wave costs 32 ragged contexts of up to 8192 tokens 67 us instead of 57, one of
// 2^20 53 instead of 45), and no share below a page a warp (one sequence of 600 tokens of
// 128 channels takes 5.2 us with shares of 4 pages, 6.4 with 8 and 7.9 with 16; one of
// 16000 8.4, 10.0, 10.0).  Up to eight shares are one cluster and join through its shared
// memory; more (a few long sequences) go through the workspace and a second launch, which
// pays from sixteen on (4000 tokens of one sequence: 32 shares 7.0 us, eight 7.9).
struct Plan {
  int splits;
  bool cluster;
};
Plan plan_for(const Kv4DecodeArgs& a) {
  const int64_t blocks =
      static_cast<int64_t>(a.batch) * a.kv_heads * ceil_div(a.heads / a.kv_heads, kHeads);
  const int64_t want = ceil_div(148 * (a.d == 64 ? 3 : 2), blocks);
  const int64_t most = ceil_div(most_pages(a), kMinShare);
  int64_t s = want < most ? want : most;
  if (s < 1) s = 1;
  if (s > kMaxCluster && s < 2 * kMaxCluster) s = kMaxCluster;
  return Plan{static_cast<int>(s), s > 1 && s <= kMaxCluster};
}

template <int D, int kSets>
cudaError_t launch_main(const Params& p, dim3 grid, cudaStream_t stream) {
  auto kernel = kv4_decode_kernel<D, kSets>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       Cfg<D>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl_cluster(kernel, grid, dim3(kThreads), Cfg<D>::kSmem, stream,
                            p.cluster ? p.splits : 1, p);
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
  p.skip = a.skip;
  p.heads = a.heads;
  p.group = a.heads / a.kv_heads;
  p.head_blocks = (p.group + kHeads - 1) / kHeads;
  const Plan plan = plan_for(a);
  p.splits = plan.splits;
  p.cluster = plan.cluster;
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
  if (e != cudaSuccess || p.splits == 1 || p.cluster) return e;
  // few rows with many shares: the larger block reads more of them at once
  const dim3 jgrid(static_cast<unsigned>(rows));
  if (p.splits > 64)
    return launch_pdl(kv4_join_kernel<D, 16>, jgrid, dim3(512), 0, stream, p);
  return launch_pdl(kv4_join_kernel<D, 4>, jgrid, dim3(128), 0, stream, p);
}

}  // namespace

size_t kv4_decode_workspace_bytes(const Kv4DecodeArgs& a) {
  const Plan plan = plan_for(a);
  if (plan.splits == 1 || plan.cluster) return 0;
  return static_cast<size_t>(a.batch) * a.heads * plan.splits * (a.d + 2) * 4;
}

cudaError_t launch_kv4_decode(const Kv4DecodeArgs& a, cudaStream_t stream) {
  return a.d == 64 ? run<64>(a, stream) : run<128>(a, stream);
}

}  // namespace nb
