// Causal attention with a sliding window and visible first tokens (sinks),
// backward, on the 5th-generation tensor cores (tcgen05 + TMEM), bf16 in / fp32
// accumulate.  With P recomputed from the stored log-sum-exp and
// D_i = sum_k dO_ik O_ik:
//   dS = P (dO V^T - D),  dV = P^T dO,  dK = dS^T Q / sqrt(d),  dQ = dS K / sqrt(d),
// dK and dV summed over the query heads that share a key/value head.
//
// Four launches on the caller's stream:
//   rows   per query row -D (from its keys where they are few, see kFew) and
//          -lse log2(e) into the workspace (-inf past the length, so P is 0
//          there), and zeros for gradient tiles past it;
//   main   <kDQ = false>: a 128-key tile of K and V stays, 64-query chunks of Q
//          and dO stream past: S^T = K Q^T, dP^T = V dO^T (keys on the lanes),
//          dV += P^T dO, dK += dS^T Q;
//   main   <kDQ = true>: a 128-query tile of Q and dO stays, 64-key chunks of K
//          and V stream past: S = Q K^T, dP = dO V^T, dQ += dS K;
//   join   adds the parts of key tiles that were split (below).
// S and dP are computed twice (7 products instead of 5), but every gradient is
// accumulated in tensor memory in a fixed order: no fp32 accumulator of dQ in
// global memory (cleared, added to with atomics and read back), and results
// that repeat bit for bit.  P and dS go back into tensor memory and are the A
// operands of the gradient products from there; neither passes through shared
// memory.  Both are rounded to bf16 as operands.
//
// The first key tile holds the sinks, which every later query of every head of
// the group sees: up to group * n / 64 chunks against group * (window + 128) / 64
// for another tile.  A tile's chunks are therefore cut into parts when they are
// a large piece of an SM's even share; parts are fp32 tiles in the workspace that
// the last launch adds in order.  The work items differ in cost, so a persistent
// grid of one CTA per SM takes them from a counter in the workspace, the largest
// first; which CTA takes an item does not change its result.
//
// Warp roles (512 threads, four warpgroups with reallocated registers): warp 0
// takes the items, decodes them for the others into a ring in shared memory, and
// is the TMA producer (a chunk that reaches past the length lands on a barrier of its
// own, and the warp zeroes the rows past it: P is 0 there, but 0 x NaN is not; what other
// hidden rows may do is mended at the end, sink_hidden.cuh);
// warp 1 TMEM owner and S/dP issuer; warp 2 issuer of the gradient products;
// warpgroups 1 and 2 take the chunks in turn (thread = lane, 64 columns): a group
// moves S and dP into registers and hands their columns back at once, so the next
// chunk's products run under its arithmetic; P and dS have columns of their own
// for each group;
// warpgroup 3 epilogue (thread = lane), staging through swizzled shared memory
// and TMA tensor stores.  Every wait is bounded (sm100.cuh).
#include <math.h>

#include "serving.cuh"
#include "sink_hidden.cuh"

namespace nb {
namespace {

using namespace sm100;

constexpr int kThreads = 512;
constexpr int kLaunchRegs = 65536 / kThreads / 8 * 8;
constexpr int kRows = 128;                // rows of the tile that stays
constexpr int kSlab = kRows * 128;        // swizzled box of the tile: 128 rows x 64 bf16
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMaxBatch = 1024;           // sequences in the shared-memory work table
constexpr int kItems = 4;                 // items decoded ahead
constexpr int kTakers = 14;               // arrivals that free one: 2 issuers, 8 + 4 warps

struct Params {
  const void* q;
  const void* k;
  const void* v;
  const void* o;
  const void* dout;
  const float* lse;
  const int32_t* lengths;
  void* dq;
  void* dk;
  void* dv;
  float* nd;     // [batch * heads][npad]: -D
  float* nlse2;  // [batch * heads][npad]: -lse log2(e)
  float* part0;  // parts of the first key tiles, [batch * kv_heads][s0][dV, dK][128][d]
  float* part1;  // parts of the others, [batch * kv_heads][ntiles - 1][s1][dV, dK][128][d]
  int* err;
  int batch, heads, kv_heads, group, n, npad, ntiles, window, sinks;
  int s0, s1;    // parts of the first key tile, of another
  int items;     // of the main kernel
  int term_blocks;  // of the row kernel: those of rows that see few keys
  int* taken;    // items taken so far by the CTAs of <kDQ = false>, <kDQ = true>
  int* noted;    // [items][4]: quarter tiles with rows that are not finite, linked (epi_warps)
  float scale;
};

__device__ __forceinline__ int length_of(const Params& p, int b) {
  const int L = p.lengths ? __ldcg(p.lengths + b) : p.n;
  return min(max(L, 0), p.n);
}

// Rows of a streamed chunk.  A product of 64 columns reads its 128-row operand from
// shared memory for half the work (16 of them take 773 cycles, 16 of 128 columns
// 1030), but 128 need room in tensor memory for S and dP of that width, and waste
// more at the window's edges: they pay for dQ at d = 128 (252 -> 227 us at 8 heads x
// 16384, window 2048; at d = 64 and window 160 dK and dV take 66 us with them, 54
// without).
constexpr int chunk_rows(int d, bool dq) { return dq && d == 128 ? 128 : 64; }

// Chunks of queries that see key tile `tile` (per head), in a sequence of length L > 128 tile.
__host__ __device__ __forceinline__ int query_chunks(int tile, int L, int window, int sinks,
                                                     int chunk) {
  const int k0 = tile * kRows;
  // the last key of the tile is seen up to its window's end, the sinks by every query
  const int64_t far = static_cast<int64_t>(k0) + kRows - 1 + window;
  const int end = (tile == 0 && sinks > 0) || far > L ? L : static_cast<int>(far);
  return (end - k0 + chunk - 1) / chunk;
}

template <int D, bool kDQ>
struct Cfg {
  static constexpr int kChunk = chunk_rows(D, kDQ);
  static constexpr bool kWide = kChunk == 128;  // both groups share every chunk, 64 columns each
  static constexpr int kChunkSlab = kChunk * 128;  // swizzled box of a chunk
  // tiles that stay: two buffers at d = 64 (the next item's loads overlap), one at d = 128
  static constexpr int NT = D == 64 ? 2 : 1;
  // stages of the chunk's two operands X (Q, or K) and Y (dO, or V).  Wide: dQ needs V for
  // dP only, so V's one stage is free long before K's and a third of K fits; V then has
  // barriers and a producer of its own (two shared stages: 222 us where this takes 170, at
  // 16 heads x 8192 x 128; at the other widths sharing barriers is 10-15 % faster).
  static constexpr bool kSplit = kWide;
  static constexpr int NX = D == 64 ? 6 : kWide ? 3 : 4;
  static constexpr int NY = kSplit ? 1 : NX;
  // buffers in tensor memory: S and dP, P and dS, accumulators
  static constexpr int NSB = D == 64 && kDQ ? 2 : 1;
  static constexpr int NPB = 2;
  static constexpr int NOUT = kDQ ? 1 : 2;      // gradients of an item
  static constexpr int NACC = D == 64 ? 2 : 1;
  static constexpr int kTile = kRows * D * 2;
  static constexpr int kHalf = kChunk * D * 2;         // one operand of a chunk
  static constexpr int oTile = 0;                      // buffer i: X at oTile + 2 i kTile, Y after it
  static constexpr int oX = oTile + NT * 2 * kTile;
  static constexpr int oY = oX + NX * kHalf;
  static constexpr int oStg = oY + NY * kHalf;         // output staging, 64 columns of a tile
  static constexpr int oCol = oStg + kSlab;            // X stage s: -lse log2 e and -D of its columns
  // kDQ: -lse log2 e and -D of the tile's rows, one set per tile buffer
  static constexpr int oRow = oCol + (kDQ ? 0 : NX * 2 * kChunk * 4);
  static constexpr int oItem = oRow + (kDQ ? NT * 2 * kRows * 4 : 0);  // ring of items
  static constexpr int oBar = oItem + kItems * 64;
  static constexpr int bTFull = 0, bTFree = bTFull + NT, bXFull = bTFree + NT, bXFree = bXFull + NX,
                       bYFull = bXFree + NX, bYFree = bYFull + NY, bSFull = bYFree + NY,
                       bSFree = bSFull + 2, bPFull = bSFree + NSB, bPFree = bPFull + NPB,
                       bAFull = bPFree + NPB, bAFree = bAFull + NACC, bIFull = bAFree + NACC,
                       bIFree = bIFull + kItems, bFix = bIFree + kItems, bDone = bFix + 2,
                       nBar = bDone + 1;
  static constexpr int oSlot = oBar + nBar * 8;
  static constexpr int oNoted = oSlot + 16;  // of each epilogue warp: its last noted quarter, or -1
  static constexpr int oFound = oNoted + 16;  // of every fourth tile: some value is not finite
  static constexpr int oPre = oFound + 16;  // work table: pre[0..batch], len[0..batch)
  static constexpr int kSmem = oPre + (2 * kMaxBatch + 1) * 4 + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory per CTA");
  static constexpr uint32_t kTmemCols = 512;
  // accumulators first, then S, dP, then dS and P (two bf16 per column)
  __device__ static constexpr uint32_t tAcc(int acc, int out) { return (acc * NOUT + out) * D; }
  __device__ static constexpr uint32_t tS(int sb) { return NACC * NOUT * D + sb * 2 * kChunk; }  // dP: + kChunk
  __device__ static constexpr uint32_t tDS(int pb) { return tS(NSB) + pb * NOUT * (kChunk / 2); }
  __device__ static constexpr uint32_t tP(int pb) { return tDS(pb) + kChunk / 2; }
  static_assert(NACC * NOUT * D + NSB * 2 * kChunk + NPB * NOUT * (kChunk / 2) <= kTmemCols,
                "tensor memory columns");
  static constexpr int kRegsCtl = 72;
  static constexpr int kRegsGrad = 176;
  static constexpr int kRegsEpi = 88;
  static_assert(128 * (kRegsCtl + 2 * kRegsGrad + kRegsEpi) <= kThreads * kLaunchRegs,
                "register budget");
};

struct Item {
  int b, h, tile, L;  // h: query head (kDQ) or key/value head
  int c0, nch;        // first chunk and number of chunks
  int nq;             // chunks per head (key tiles)
  int k0, far;        // kDQ: first key of the window's chunks, chunks of sinks before them
  int part, parts;    // key tiles: this item's part
  int id;             // its place in the list
};

// Items of a sequence of length L (kDQ: query tiles of all heads; else the key
// tiles but the first, whose parts make a list of their own).
template <bool kDQ>
__device__ __forceinline__ int items_of(const Params& p, int L) {
  const int t = (L + kRows - 1) / kRows;
  return kDQ ? p.heads * t : p.kv_heads * max(t - 1, 0) * p.s1;
}

// Warp-cooperative: prefix sums of the items per sequence, and the lengths.
template <bool kDQ>
__device__ void build_table(int* pre, const Params& p, int lane) {
  if (p.batch > kMaxBatch) return;
  int carry = 0;
  for (int b0 = 0; b0 < p.batch; b0 += 32) {
    const int b = b0 + lane;
    int v = 0;
    if (b < p.batch) {
      const int L = length_of(p, b);
      pre[kMaxBatch + 1 + b] = L;
      v = items_of<kDQ>(p, L);
    }
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, v, off);
      if (lane >= off) v += t;
    }
    if (b < p.batch) pre[b + 1] = carry + v;
    carry += __shfl_sync(0xffffffffu, v, 31);
  }
  if (lane == 0) pre[0] = 0;
}

// Parts of the first key tiles, at the head of the list.
template <bool kDQ>
__device__ __forceinline__ int first_items(const Params& p) {
  return kDQ ? 0 : p.batch * p.kv_heads * p.s0;
}
template <bool kDQ>
__device__ __forceinline__ int item_count(const Params& p, const int* pre) {
  return p.batch <= kMaxBatch ? first_items<kDQ>(p) + pre[p.batch] : p.items;
}

// Item k.  Heads are innermost; query tiles run from the last (most keys) to the
// first; key tiles begin with the parts of the first ones (the sinks').
template <int D, bool kDQ>
__device__ Item item(const Params& p, const int* pre, int k) {
  constexpr int kChunk = chunk_rows(D, kDQ);
  Item x;
  x.id = k;
  x.c0 = x.nch = x.nq = x.k0 = x.far = x.part = 0;
  x.parts = 1;
  const int lead = first_items<kDQ>(p);
  if (k < lead) {
    const int bkv = p.batch * p.kv_heads;
    x.part = k / bkv;
    x.parts = p.s0;
    const int bh = k - x.part * bkv;
    x.b = bh / p.kv_heads;
    x.h = bh - x.b * p.kv_heads;
    x.L = length_of(p, x.b);
    x.tile = 0;
  } else {
    int rem = k - lead;
    if (p.batch <= kMaxBatch) {
      int lo = 0, hi = p.batch - 1;  // largest b with pre[b] <= rem
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (pre[mid] <= rem) lo = mid; else hi = mid - 1;
      }
      x.b = lo;
      rem -= pre[lo];
      x.L = pre[kMaxBatch + 1 + lo];
    } else {
      const int per = (p.items - lead) / p.batch;
      x.b = rem / per;
      rem -= x.b * per;
      x.L = length_of(p, x.b);
    }
    const int heads = kDQ ? p.heads : p.kv_heads;
    const int slot = rem / heads;
    x.h = rem - slot * heads;
    if (kDQ) {
      x.tile = (p.batch <= kMaxBatch ? (x.L + kRows - 1) / kRows : p.ntiles) - 1 - slot;
    } else {
      x.tile = 1 + slot / p.s1;
      x.part = slot % p.s1;
      x.parts = p.s1;
    }
  }
  const int r0 = x.tile * kRows;
  if (r0 >= x.L) return x;
  if (kDQ) {
    x.k0 = r0 >= p.window ? r0 - p.window + 1 : 0;
    if (p.sinks > 0 && x.k0 > 0) {
      const int f = (p.sinks + kChunk - 1) / kChunk;
      if (x.k0 <= f * kChunk) x.k0 = 0;  // as many chunks either way
      else x.far = f;
    }
    x.nch = x.far + (min(r0 + kRows, x.L) - x.k0 + kChunk - 1) / kChunk;
  } else {
    x.nq = query_chunks(x.tile, x.L, p.window, p.sinks, kChunk);
    const int64_t all = static_cast<int64_t>(x.nq) * p.group;
    x.c0 = static_cast<int>(all * x.part / x.parts);
    x.nch = static_cast<int>(all * (x.part + 1) / x.parts) - x.c0;
  }
  return x;
}

// The rd-th item of this CTA from the ring, for the warps that work on it;
// x.nch < 0 after the last.  Called by whole warps.
template <int D, bool kDQ>
__device__ __forceinline__ bool next_item(Item& x, int rd, uint32_t bar, const uint8_t* gbase,
                                          int lane) {
  using C = Cfg<D, kDQ>;
  const int q = rd % kItems;
  if (!__all_sync(0xffffffffu, mbar_wait(bar + 8 * (C::bIFull + q), (rd / kItems) & 1)))
    return false;
  x = *reinterpret_cast<const Item*>(gbase + C::oItem + q * 64);
  __syncwarp();  // every lane has read it
  if (lane == 0) mbar_arrive(bar + 8 * (C::bIFree + q));
  return true;
}

// Chunk c of an item: its first row and the head it belongs to.
struct Chunk {
  int row, bh;
};
template <int D, bool kDQ>
__device__ __forceinline__ Chunk chunk(const Params& p, const Item& x, int c) {
  constexpr int kChunk = chunk_rows(D, kDQ);
  Chunk k;
  if (kDQ) {
    k.row = c < x.far ? c * kChunk : x.k0 + (c - x.far) * kChunk;
    k.bh = x.b * p.kv_heads + x.h / p.group;
  } else {
    const int j = x.c0 + c, g = j / x.nq;
    k.row = x.tile * kRows + (j - g * x.nq) * kChunk;
    k.bh = x.b * p.heads + x.h * p.group + g;
  }
  return k;
}

enum : int { kErrTFree = 0x81, kErrXFree, kErrFix, kErrTFull, kErrXFull, kErrSFree, kErrPFull, kErrAFree,
             kErrSFull, kErrYFree, kErrYFull, kErrDone, kErrIFree, kErrIFull, kErrGTFull, kErrAFull };

// A chunk's operands into their stages (whole warp; lane 0 issues): one, or where
// map1 is not null two.  Where the chunk reaches past the length (other data lies
// there: P is 0, but 0 x NaN is not) they land on `fixbar`, and the warp zeroes the
// rows past the length before it hands the stage on.  `stats`: rows of statistics
// that come along, or 0.
template <int D, bool kDQ, bool kTwo>
__device__ __forceinline__ int load_chunk(const Params& p, int L, Chunk k, uint32_t base,
                                          uint8_t* gbase, const CUtensorMap* map0, int off0,
                                          const CUtensorMap* map1, int off1, uint32_t full,
                                          uint32_t fixbar, int& fixes, uint32_t stats, int lane) {
  using C = Cfg<D, kDQ>;
  const bool fix = k.row + C::kChunk > L && L < p.n;
  const uint32_t land = fix ? fixbar : full;
  if (lane == 0) {
    mbar_arrive_expect_tx(land, (kTwo ? 2 : 1) * C::kHalf + (stats ? 2 * C::kChunk * 4 : 0));
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      tma_load_3d(base + off0 + i * C::kChunkSlab, map0, land, i * 64, k.row, k.bh);
      if (kTwo) tma_load_3d(base + off1 + i * C::kChunkSlab, map1, land, i * 64, k.row, k.bh);
    }
    if (stats) {  // the columns' statistics, padded to whole tiles of 128
      const int64_t at = static_cast<int64_t>(k.bh) * p.npad + k.row;
      bulk_load(stats, p.nlse2 + at, C::kChunk * 4, land);
      bulk_load(stats + C::kChunk * 4, p.nd + at, C::kChunk * 4, land);
    }
  }
  if (!fix) return 0;
  if (!__all_sync(0xffffffffu, mbar_wait(fixbar, fixes & 1))) return kErrFix;
  ++fixes;
#pragma unroll
  for (int o = 0; o < (kTwo ? 2 : 1); ++o) {
    uint4* v = reinterpret_cast<uint4*>(gbase + (o ? off1 : off0));
    // whole 128-byte rows of every box, so the swizzle does not matter
    for (int i = 0; i < D / 64; ++i)
      for (int j = (L - k.row) * 8 + lane; j < C::kChunk * 8; j += 32)
        v[i * (C::kChunkSlab / 16) + j] = make_uint4(0, 0, 0, 0);
  }
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) mbar_arrive(full);
  return 0;
}

// Items, tiles and the chunks' operands, kSplit: X alone (warp 0, the whole warp).
// cf: X's map for the chunks of sinks (kDQ).
template <int D, bool kDQ>
__device__ int producer(const Params& p, const int* pre, uint32_t base, uint8_t* gbase, int lane,
                        const CUtensorMap* tx, const CUtensorMap* ty, const CUtensorMap* cx,
                        const CUtensorMap* cf, const CUtensorMap* cy) {
  using C = Cfg<D, kDQ>;
  const uint32_t bar = base + C::oBar;
  const int count = item_count<kDQ>(p, pre);
  int fixes = 0;
  Ring<C::NX> ring;
  Ring<C::NT> tile;
  auto run = [&]() -> int {
    int* taken = p.taken + (kDQ ? 1 : 0);
    int fetched = lane == 0 ? atomicAdd(taken, 1) : 0;
    for (int rd = 0;;) {
      const int it = __shfl_sync(0xffffffffu, fetched, 0);
      Item x;
      if (it < count) {
        if (lane == 0) fetched = atomicAdd(taken, 1);  // the next one, needed only after this
        x = item<D, kDQ>(p, pre, it);
        if (x.nch == 0) continue;
      } else {
        x.nch = -1;
      }
      const int q = rd % kItems;
      if (!__all_sync(0xffffffffu,
                      lane != 0 || mbar_wait(bar + 8 * (C::bIFree + q), ((rd / kItems) & 1) ^ 1)))
        return kErrIFree;
      if (lane == 0) {
        *reinterpret_cast<Item*>(gbase + C::oItem + q * 64) = x;
        mbar_arrive(bar + 8 * (C::bIFull + q));
      }
      ++rd;
      if (x.nch < 0) break;
      const int tb = tile.i;
      bool ok = true;
      if (lane == 0) {
        ok = mbar_wait(bar + 8 * (C::bTFree + tb), tile.ph ^ 1);
        if (ok) {
          const uint32_t full = bar + 8 * (C::bTFull + tb);
          mbar_arrive_expect_tx(full, 2 * C::kTile + (kDQ ? 2 * kRows * 4 : 0));
          const uint32_t s = base + C::oTile + tb * 2 * C::kTile;
          const int bh = x.b * (kDQ ? p.heads : p.kv_heads) + x.h;
          if (kDQ) {  // the rows' statistics, padded to whole tiles
            const int64_t at = static_cast<int64_t>(bh) * p.npad + x.tile * kRows;
            const uint32_t sr = base + C::oRow + tb * 2 * kRows * 4;
            bulk_load(sr, p.nlse2 + at, kRows * 4, full);
            bulk_load(sr + kRows * 4, p.nd + at, kRows * 4, full);
          }
#pragma unroll
          for (int i = 0; i < D / 64; ++i) {
            tma_load_3d(s + i * kSlab, tx, full, i * 64, x.tile * kRows, bh);
            tma_load_3d(s + C::kTile + i * kSlab, ty, full, i * 64, x.tile * kRows, bh);
          }
        }
      }
      if (!__all_sync(0xffffffffu, ok)) return kErrTFree;
      tile.next();
      for (int c = 0; c < x.nch; ++c) {
        if (!__all_sync(0xffffffffu,
                        lane != 0 || mbar_wait(bar + 8 * (C::bXFree + ring.i), ring.ph ^ 1)))
          return kErrXFree;
        const int err = load_chunk<D, kDQ, !C::kSplit>(
            p, x.L, chunk<D, kDQ>(p, x, c), base, gbase, kDQ && c < x.far ? cf : cx,
            C::oX + ring.i * C::kHalf, cy, C::oY + ring.i * C::kHalf,
            bar + 8 * (C::bXFull + ring.i), bar + 8 * C::bFix, fixes,
            kDQ ? 0 : base + C::oCol + ring.i * 2 * C::kChunk * 4, lane);
        if (err) return err;
        ring.next();
      }
    }
    return 0;
  };
  const int err = run();
  // copies that nobody took have landed before the block exits
  if (err == kErrFix) mbar_wait(bar + 8 * C::bFix, fixes & 1);
  drain_ring<C::NT>(tile.i, tile.ph, [&](int i, uint32_t ph) { mbar_wait(bar + 8 * (C::bTFull + i), ph); });
  drain_ring<C::NX>(ring.i, ring.ph, [&](int i, uint32_t ph) { mbar_wait(bar + 8 * (C::bXFull + i), ph); });
  return err;
}

// kSplit: the Y operand of the chunks (warp 3, the whole warp).
template <int D, bool kDQ>
__device__ int y_producer(const Params& p, uint32_t base, uint8_t* gbase, int lane,
                          const CUtensorMap* cy) {
  using C = Cfg<D, kDQ>;
  const uint32_t bar = base + C::oBar;
  int fixes = 0;
  Ring<C::NY> ring;
  auto run = [&]() -> int {
    for (int rd = 0;; ++rd) {
      Item x;
      if (!next_item<D, kDQ>(x, rd, bar, gbase, lane)) return kErrIFull;
      if (x.nch < 0) break;
      for (int c = 0; c < x.nch; ++c) {
        if (!__all_sync(0xffffffffu,
                        lane != 0 || mbar_wait(bar + 8 * (C::bYFree + ring.i), ring.ph ^ 1)))
          return kErrYFree;
        const int err = load_chunk<D, kDQ, false>(
            p, x.L, chunk<D, kDQ>(p, x, c), base, gbase, cy, C::oY + ring.i * C::kHalf, nullptr, 0,
            bar + 8 * (C::bYFull + ring.i), bar + 8 * (C::bFix + 1), fixes, 0, lane);
        if (err) return err;
        ring.next();
      }
    }
    return 0;
  };
  const int err = run();
  if (err == kErrFix) mbar_wait(bar + 8 * (C::bFix + 1), fixes & 1);
  drain_ring<C::NY>(ring.i, ring.ph, [&](int i, uint32_t ph) { mbar_wait(bar + 8 * (C::bYFull + i), ph); });
  return err;
}

// Number of chunks of the rd-th item, for the single-thread roles (the rest of the
// item does not concern them); < 0 after the last, kNoItem on a timeout.
constexpr int kNoItem = -2;
template <int D, bool kDQ>
__device__ __forceinline__ int next_chunks(int rd, uint32_t bar, const uint8_t* gbase) {
  using C = Cfg<D, kDQ>;
  const int q = rd % kItems;
  if (!mbar_wait(bar + 8 * (C::bIFull + q), (rd / kItems) & 1)) return kNoItem;
  const int nch = reinterpret_cast<const Item*>(gbase + C::oItem + q * 64)->nch;
  mbar_arrive(bar + 8 * (C::bIFree + q));
  return nch;
}

// S and dP of every chunk (warp 1, one thread).  A lone thread takes four cycles
// and more an instruction, and what it does between two chunks is time the tensor
// cores may stand still: positions advance by steps, descriptors by adds.
template <int D, bool kDQ>
__device__ int s_issuer(const Params& p, uint32_t base, const uint8_t* gbase, uint32_t tmem) {
  using C = Cfg<D, kDQ>;
  const uint32_t bar = base + C::oBar;
  constexpr uint32_t kId = idesc_bf16_f32(128, C::kChunk, false, false);
  const uint64_t tX = smem_desc_sw128(base + C::oTile, 0, 1024);
  const uint64_t tY = smem_desc_sw128(base + C::oTile + C::kTile, 0, 1024);
  const uint64_t cX = smem_desc_sw128(base + C::oX, 0, 1024);
  const uint64_t cY = smem_desc_sw128(base + C::oY, 0, 1024);
  Ring<C::NT> tile;
  Ring<C::NX> xr;
  Ring<C::NY> yr;
  Ring<C::NSB> sb;
  int G = 0;
  for (int rd = 0;; ++rd) {
    const int nch = next_chunks<D, kDQ>(rd, bar, gbase);
    if (nch == kNoItem) return kErrIFull;
    if (nch < 0) break;
    const uint32_t ot = tile.i * (2 * C::kTile >> 4);
    const uint64_t dX = desc_add(tX, ot), dY = desc_add(tY, ot);
    if (!mbar_wait(bar + 8 * (C::bTFull + tile.i), tile.ph)) return kErrTFull;
    for (int c = 0; c < nch; ++c, ++G) {
      // the chunk is there, and the scores that used the buffers before have moved to
      // registers; all are asked for before the first answer is looked at
      const uint32_t xbar = bar + 8 * (C::bXFull + xr.i), ybar = bar + 8 * (C::bYFull + yr.i);
      const uint32_t sfree = bar + 8 * (C::bSFree + sb.i);
      const bool okx = mbar_try_wait(xbar, xr.ph), oks = mbar_try_wait(sfree, sb.ph ^ 1);
      const bool oky = !C::kSplit || mbar_try_wait(ybar, yr.ph);
      if (!okx && !mbar_wait(xbar, xr.ph)) return kErrXFull;
      if (!oks && !mbar_wait(sfree, sb.ph ^ 1)) return kErrSFree;
      tc_fence_after();
      const uint64_t eX = desc_add(cX, xr.i * (C::kHalf >> 4));
      const uint32_t tS = tmem + C::tS(sb.i), tDP = tS + C::kChunk;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint32_t kt = ((k >> 2) * kSlab + (k & 3) * 32) >> 4;
        const uint32_t kc = ((k >> 2) * C::kChunkSlab + (k & 3) * 32) >> 4;
        mma_bf16_ss(tS, desc_add(dX, kt), desc_add(eX, kc), kId, k > 0);
      }
      if (C::kSplit) {
        if (!oky && !mbar_wait(ybar, yr.ph)) return kErrYFull;
        tc_fence_after();
      }
      const uint64_t eY = desc_add(cY, yr.i * (C::kHalf >> 4));
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint32_t kt = ((k >> 2) * kSlab + (k & 3) * 32) >> 4;
        const uint32_t kc = ((k >> 2) * C::kChunkSlab + (k & 3) * 32) >> 4;
        mma_bf16_ss(tDP, desc_add(dY, kt), desc_add(eY, kc), kId, k > 0);
      }
      // groups that take turns have a barrier each, so that each sees all its phases
      mma_commit(bar + 8 * (C::bSFull + (C::kWide ? 0 : G & 1)));
      if (C::kSplit) mma_commit(bar + 8 * (C::bYFree + yr.i));  // V's only reader
      if (c == nch - 1) mma_commit(bar + 8 * (C::bTFree + tile.i));  // the tile's only readers
      xr.next();
      yr.next();
      sb.next();
    }
    tile.next();
  }
  return 0;
}

// The gradient products of every chunk (warp 2, one thread): A = P or dS from
// tensor memory, B = the chunk's rows (MN-major: 64-column atoms C::kChunkSlab
// apart, 16 rows = 2048 bytes per step).
template <int D, bool kDQ>
__device__ int grad_issuer(const Params& p, uint32_t base, const uint8_t* gbase, uint32_t tmem) {
  using C = Cfg<D, kDQ>;
  const uint32_t bar = base + C::oBar;
  constexpr uint32_t kId = idesc_bf16_f32(128, D, false, true);
  const uint64_t cX = smem_desc_sw128(base + C::oX, C::kChunkSlab, 1024);
  const uint64_t cY = smem_desc_sw128(base + C::oY, C::kChunkSlab, 1024);
  Ring<C::NACC> acc;
  Ring<C::NX> xr;
  Ring<C::NY> yr;
  Ring<C::NPB> pb;
  for (int rd = 0;; ++rd) {
    const int nch = next_chunks<D, kDQ>(rd, bar, gbase);
    if (nch == kNoItem) return kErrIFull;
    if (nch < 0) break;
    const uint32_t out0 = tmem + C::tAcc(acc.i, 0);
    if (!mbar_wait(bar + 8 * (C::bAFree + acc.i), acc.ph ^ 1)) return kErrAFree;
    for (int c = 0; c < nch; ++c) {
      const uint64_t eX = desc_add(cX, xr.i * (C::kHalf >> 4));
      const uint32_t tP = tmem + C::tP(pb.i), tDS = tmem + C::tDS(pb.i);
      if (!mbar_wait(bar + 8 * (C::bPFull + pb.i), pb.ph)) return kErrPFull;
      tc_fence_after();
      if (kDQ) {  // dQ += dS K
#pragma unroll
        for (int k = 0; k < C::kChunk / 16; ++k)
          mma_bf16_ts(out0, tDS + 8 * k, desc_add(eX, (k * 2048) >> 4), kId, c > 0 || k > 0);
      } else {    // dV += P^T dO, dK += dS^T Q
        const uint32_t out1 = tmem + C::tAcc(acc.i, C::NOUT - 1);
        const uint64_t eY = desc_add(cY, yr.i * (C::kHalf >> 4));
#pragma unroll
        for (int k = 0; k < C::kChunk / 16; ++k)
          mma_bf16_ts(out0, tP + 8 * k, desc_add(eY, (k * 2048) >> 4), kId, c > 0 || k > 0);
#pragma unroll
        for (int k = 0; k < C::kChunk / 16; ++k)
          mma_bf16_ts(out1, tDS + 8 * k, desc_add(eX, (k * 2048) >> 4), kId, c > 0 || k > 0);
      }
      mma_commit(bar + 8 * (C::bPFree + pb.i));
      mma_commit(bar + 8 * (C::bXFree + xr.i));
      if (c == nch - 1) mma_commit(bar + 8 * (C::bAFull + acc.i));
      xr.next();
      yr.next();
      pb.next();
    }
    acc.next();
  }
  return 0;
}

// Bits [lo, hi) of a 64-bit word (clipped to it).
__device__ __forceinline__ uint64_t bit_range(int64_t lo, int64_t hi) {
  const int a = static_cast<int>(lo < 0 ? 0 : (lo > 64 ? 64 : lo));
  const int b = static_cast<int>(hi < 0 ? 0 : (hi > 64 ? 64 : hi));
  return b > a ? (~0ull >> (64 - (b - a))) << a : 0ull;
}

// The sign of byte b of x in every bit of the low half, of y in the high half.
__device__ __forceinline__ uint32_t sign_halves(uint32_t x, uint32_t y, int b) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;"
      : "=r"(r)
      : "r"(x), "r"(y), "r"(0x8888u + 0x11u * b + 0x1100u * (4 + b)));
  return r;
}

// P and dS of 64 columns of a chunk a warpgroup: half of every chunk (wide chunks),
// or every second chunk.  Thread = lane r.
template <int D, bool kDQ>
__device__ int grad_warps(const Params& p, uint32_t base, uint8_t* gbase,
                          uint32_t tmem, int wg, int wq, int lane) {
  using C = Cfg<D, kDQ>;
  const uint32_t bar = base + C::oBar;
  const int r = wq * 32 + lane;
  const uint32_t trow = tmem + (static_cast<uint32_t>(wq * 32) << 16);
  const float sl2 = p.scale * kLog2e;
  auto all_ok = [](bool ok) { return __all_sync(0xffffffffu, ok); };
  // this group's chunks: all (wide), or those of its parity, counted over all items
  constexpr int kStep = C::kWide ? 1 : 2;
  int G = C::kWide ? 0 : wg, g = 0;  // its next chunk, and the item's first
  Ring<C::NX> xr;                    // chunk G's X stage, S/dP buffer, P/dS buffer; the
  Ring<C::NSB> sb;                   // parity of its own S barrier is full.ph
  Ring<C::NPB> pb;
  Ring<1> full;
  if (!C::kWide && wg) {
    xr.next();
    sb.next();
    pb.next();
  }
  const int half = C::kWide ? 64 * wg : 0;  // this group's 64 columns of a chunk
  const uint32_t sfull = bar + 8 * (C::bSFull + (C::kWide ? 0 : wg));
  Ring<C::NT> tile;
  for (int rd = 0;; ++rd) {
    Item x;
    if (!next_item<D, kDQ>(x, rd, bar, gbase, lane)) return kErrIFull;
    if (x.nch < 0) break;
    const int t0 = x.tile * kRows, row = t0 + r;  // row: key (or query, kDQ) of this lane
    float nl_row = 0.f, nd_row = 0.f;
    if (kDQ) {
      if (!all_ok(mbar_wait(bar + 8 * (C::bTFull + tile.i), tile.ph))) return kErrGTFull;
      const float* st = reinterpret_cast<const float*>(gbase + C::oRow + tile.i * 2 * kRows * 4);
      nl_row = st[r];
      nd_row = st[kRows + r];
      __syncwarp();
      if (lane == 0) mbar_arrive(bar + 8 * (C::bTFree + tile.i));  // read; see the barrier's count
      tile.next();
    }
    // rows of the chunks run through the window once (kDQ), or once per head
    int at = kDQ ? 0 : (x.c0 + (G - g)) % x.nq;
    for (; G < g + x.nch; G += kStep) {
      int col = half;  // first column's query (or key, kDQ)
      if (kDQ) {
        const int c = G - g;
        col += c < x.far ? c * C::kChunk : x.k0 + (c - x.far) * C::kChunk;
      } else {
        col += t0 + at * C::kChunk;
        at += kStep;
        while (at >= x.nq) at -= x.nq;
      }
      bool whole;
      uint64_t mask = ~0ull;
      if (kDQ) {
        whole = G - g >= x.far && col + 63 <= t0 && col > t0 + kRows - 1 - p.window &&
                t0 + kRows <= x.L;
        if (!whole) {
          const int first = row >= p.window ? row - p.window + 1 : 0;
          if (G - g < x.far) mask = bit_range(0, p.sinks - col);
          else mask = bit_range(first - col, row + 1 - col) |
                      (x.far ? 0ull : bit_range(0, min(p.sinks, row + 1) - col));
          if (row >= x.L) mask = 0ull;
        }
      } else {
        whole = col >= t0 + kRows - 1 && col - t0 < p.window - 63 &&
                col + 64 <= x.L;  // then the keys, which come before col, are below L too
        if (!whole) {
          const int64_t end = row < p.sinks ? x.L : static_cast<int64_t>(row) + p.window;
          mask = row < x.L ? bit_range(row - col, (end < x.L ? end : x.L) - col) : 0ull;
        }
      }
      // the products of an earlier chunk have read these P and dS (long since: waiting
      // here keeps the wait's own cost out of the chain from S to P), and (kDQ not) the
      // columns' statistics are there
      bool ok = mbar_wait(bar + 8 * (C::bPFree + pb.i), pb.ph ^ 1);
      if (!kDQ) ok = ok && mbar_wait(bar + 8 * (C::bXFull + xr.i), xr.ph);
      if (!all_ok(ok && mbar_wait(sfull, full.ph))) return kErrSFull;
      tc_fence_after();
      const float* nl = reinterpret_cast<const float*>(gbase + C::oCol + xr.i * 2 * C::kChunk * 4) + half;
      const float* nd = nl + C::kChunk;
      const float2 sl = make_float2(sl2, sl2);
      float s[2][32], dp[2][32];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        tmem_ld32(trow + C::tS(sb.i) + half + 32 * j, s[j]);
        tmem_ld32(trow + C::tS(sb.i) + C::kChunk + half + 32 * j, dp[j]);
      }
      tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        reg_fence(s[j]);
        reg_fence(dp[j]);
      }
      tc_fence_before();
      mbar_arrive(bar + 8 * (C::bSFree + sb.i));
#pragma unroll
      for (int j = 0; j < 2; ++j) {  // 32 columns at a time
        uint32_t wp[16], ws[16];  // P and dS of columns 2 i, 2 i + 1
        const uint32_t mw = static_cast<uint32_t>(mask >> (32 * j));
        if (whole || __any_sync(0xffffffffu, mw != 0u)) {
#pragma unroll
          for (int i = 0; i < 16; i += 2) {  // pairs of columns, packed fp32x2 arithmetic
            float4 n4, d4;
            if (kDQ) {
              n4 = make_float4(nl_row, nl_row, nl_row, nl_row);
              d4 = make_float4(nd_row, nd_row, nd_row, nd_row);
            } else {
              n4 = *reinterpret_cast<const float4*>(nl + 32 * j + 2 * i);
              d4 = *reinterpret_cast<const float4*>(nd + 32 * j + 2 * i);
            }
            const float2 n2[2] = {make_float2(n4.x, n4.y), make_float2(n4.z, n4.w)};
            const float2 d2[2] = {make_float2(d4.x, d4.y), make_float2(d4.z, d4.w)};
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int k = 2 * (i + e);
              const float2 ex = __ffma2_rn(make_float2(s[j][k], s[j][k + 1]), sl, n2[e]);
              const float2 pe = make_float2(ex2_approx(ex.x), ex2_approx(ex.y));
              const float2 de =
                  __fmul2_rn(pe, __fadd2_rn(make_float2(dp[j][k], dp[j][k + 1]), d2[e]));
              wp[i + e] = pack_bf16(pe.x, pe.y);
              ws[i + e] = pack_bf16(de.x, de.y);
            }
          }
          if (!whole && !__all_sync(0xffffffffu, mw == ~0u)) {
            // masked places are cleared in the packed words: they may hold anything, NaN too
            if (__all_sync(0xffffffffu, mw == ~0u || mw == 0u)) {  // whole rows (the sinks')
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                wp[i] &= mw;
                ws[i] &= mw;
              }
            } else {
              uint32_t top[8];  // bit 8 b + k of the word as the sign of byte b
#pragma unroll
              for (int k = 0; k < 8; ++k) top[k] = mw << (7 - k);
#pragma unroll
              for (int i = 0; i < 16; ++i) {  // two bits to two half words of ones or zeros
                const uint32_t keep = sign_halves(top[2 * i % 8], top[2 * i % 8 + 1], i / 4);
                wp[i] &= keep;
                ws[i] &= keep;
              }
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) wp[i] = ws[i] = 0u;
        }
        if (!kDQ) tmem_st16u(trow + C::tP(pb.i) + half / 2 + 16 * j, wp);
        tmem_st16u(trow + C::tDS(pb.i) + half / 2 + 16 * j, ws);
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(bar + 8 * (C::bPFull + pb.i));
      xr.next(kStep);
      if (C::NSB > 1) sb.next(kStep);
      if (C::kWide) pb.next(); else pb.ph ^= 1;
      full.next();
    }
    g += x.nch;
  }
  return 0;
}

// Where the part of a split key tile goes ([dV, dK][128][D]), or null.
template <int D>
__device__ __forceinline__ float* part_of(const Params& p, const Item& x, int bh) {
  if (x.parts <= 1) return nullptr;
  const int64_t slot =
      x.tile == 0 ? static_cast<int64_t>(bh) * p.s0 + x.part
                  : (static_cast<int64_t>(bh) * (p.ntiles - 1) + x.tile - 1) * p.s1 + x.part;
  return (x.tile == 0 ? p.part0 : p.part1) + slot * 2 * kRows * D;
}

// Gradients of finished items (warpgroup 3, thread = lane r): bf16 tiles through
// the staging buffer and a TMA store, or fp32 parts straight to the workspace.
template <int D, bool kDQ>
__device__ int epi_warps(const Params& p, uint32_t base, uint8_t* gbase,
                         uint32_t tmem, int wq, int lane, const CUtensorMap* to0,
                         const CUtensorMap* to1) {
  using C = Cfg<D, kDQ>;
  const uint32_t bar = base + C::oBar;
  const int r = wq * 32 + lane;
  const uint32_t trow = tmem + (static_cast<uint32_t>(wq * 32) << 16);
  const bool leader = r == 0;
  auto all_ok = [](bool ok) { return __all_sync(0xffffffffu, ok); };
  int tc = 0, noted = -1;
  volatile int* found = reinterpret_cast<volatile int*>(gbase + C::oFound);
  for (int rd = 0;; ++rd) {
    Item x;
    if (!next_item<D, kDQ>(x, rd, bar, gbase, lane)) return kErrIFull;
    if (x.nch < 0) break;
    // a hidden row that is not finite makes a column of the whole tile so, in rows past the
    // length too: each warp looks at a quarter of the columns, for all four
    float2 zeros[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    const int acc = tc % C::NACC;
    if (!all_ok(mbar_wait(bar + 8 * (C::bAFull + acc), (tc / C::NACC) & 1))) return kErrAFull;
    tc_fence_after();
    const bool valid = x.tile * kRows + r < x.L;
    const int bh = x.b * (kDQ ? p.heads : p.kv_heads) + x.h;
    float* part = kDQ ? nullptr : part_of<D>(p, x, bh);
    if (part != nullptr) part += r * D;
#pragma unroll
    for (int out = 0; out < C::NOUT; ++out) {
      const float mul = kDQ || out == 1 ? p.scale : 1.f;  // dQ, dK; dV
#pragma unroll
      for (int sl = 0; sl < D / 64; ++sl) {  // 64 columns at a time
        if (part == nullptr) {
          if (leader) bulk_wait_read0();  // the previous store is done with the staging
          named_barrier(2, 128);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int col = 64 * sl + 32 * j;
          float v[32];
          tmem_ld32(trow + C::tAcc(acc, out) + col, v);
          tmem_wait_ld();
          reg_fence(v);
          float2 x[16];
#pragma unroll
          for (int i = 0; i < 16; ++i)
            x[i] = __fmul2_rn(make_float2(v[2 * i], v[2 * i + 1]), make_float2(mul, mul));
#pragma unroll
          for (int e = 0; e < 2; ++e)  // 16 columns of 64
            if (wq == 2 * j + e) {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                zeros[i & 1] = __ffma2_rn(x[8 * e + i], make_float2(0.f, 0.f), zeros[i & 1]);
            }
          if (part != nullptr) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<float4*>(part + out * kRows * D + col + 4 * i) =
                  valid ? make_float4(x[2 * i].x, x[2 * i].y, x[2 * i + 1].x, x[2 * i + 1].y)
                        : make_float4(0.f, 0.f, 0.f, 0.f);
          } else {
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = valid ? pack_bf16(x[i].x, x[i].y) : 0u;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const int gc = 4 * j + u;  // 16-byte chunk of the slab's row
              *reinterpret_cast<uint4*>(gbase + C::oStg + r * 128 + ((gc ^ (r & 7)) << 4)) =
                  make_uint4(w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]);
            }
          }
        }
        const bool last = out == C::NOUT - 1 && sl == D / 64 - 1;
        if (last) {
          tc_fence_before();
          mbar_arrive(bar + 8 * (C::bAFree + acc));
          const float z = (zeros[0].x + zeros[0].y) + (zeros[1].x + zeros[1].y);
          if (z != z) found[tc & 3] = 1;
          // read by all before the last tile's barrier, set by none before this one's
          if (leader) found[(tc + 2) & 3] = 0;
        }
        if (part == nullptr) fence_proxy_async_smem();
        if (part == nullptr || last) named_barrier(1, 128);
        if (part == nullptr) {
          if (leader) {
            tma_store_3d(out == 0 ? to0 : to1, base + C::oStg, sl * 64, x.tile * kRows, bh);
            bulk_commit();
          }
        }
      }
    }
    if (found[tc & 3]) {
      if (lane == 0) p.noted[4 * x.id + wq] = noted;
      noted = 4 * x.id + wq;
    }
    ++tc;
  }
  if (leader) bulk_wait_all0();
  if (lane == 0) *reinterpret_cast<volatile int*>(gbase + C::oNoted + 4 * wq) = noted;
  return 0;
}

// The rows of dQ that the epilogue noted and that have a hidden row of K that is not
// finite among their chunks' (sink_hidden.cuh): eight warps, two to a quarter tile.
template <int D>
__device__ __forceinline__ void sum_queries_again(const Params& p, const int* pre, int at, int second,
                                                  int lane) {
  using hidden::bf16;
  const float sl2 = p.scale * kLog2e;
  for (; at >= 0; at = __ldcg(p.noted + at)) {
    const Item x = item<D, true>(p, pre, at >> 2);
    const int64_t bh = static_cast<int64_t>(x.b) * p.heads + x.h;
    const int64_t bkv = static_cast<int64_t>(x.b) * p.kv_heads + x.h / p.group;
    const bf16* k = static_cast<const bf16*>(p.k) + bkv * p.n * D;
    const bf16* v = static_cast<const bf16*>(p.v) + bkv * p.n * D;
    // end of the chunks' keys
    const int brought = min(x.k0 + (x.nch - x.far) * chunk_rows(D, true), x.L);
    for (int r = 0; r < 16; ++r) {
      const int q = x.tile * kRows + 32 * (at & 3) + 16 * second + r;
      if (q >= x.L) break;
      bf16* out = static_cast<bf16*>(p.dq) + (bh * p.n + q) * D;
      const uint32_t bad = hidden::bad_channels<D>(out, lane);
      if (!__any_sync(0xffffffffu, bad != 0)) continue;
      const int first = q >= p.window ? q - p.window + 1 : 0, sinks = min(p.sinks, first);
      if (!hidden::any_bad<D>(k, x.far ? x.k0 : max(x.k0, sinks), first, lane) &&
          !hidden::any_bad<D>(k, q + 1, brought, lane))
        continue;
      const bf16* qrow = static_cast<const bf16*>(p.q) + (bh * p.n + q) * D;
      const bf16* grow = static_cast<const bf16*>(p.dout) + (bh * p.n + q) * D;
      const float nl = p.nlse2[bh * p.npad + q], nd = p.nd[bh * p.npad + q];
      hidden::Row<D> acc;
      acc.zero();
      bool more = true;
      auto keys = [&](int from, int end) {
        for (int base = from; base < end && more; base += 32) {
          const int64_t j = min(base + lane, end - 1);
          const float s = hidden::dot<D>(qrow, k + j * D), dp = hidden::dot<D>(grow, v + j * D);
          acc.add_rows(k, base, 0, min(32, end - base), ex2_approx(fmaf(s, sl2, nl)) * (dp + nd), lane);
          more = !hidden::settled<D>(acc, bad);
        }
      };
      keys(0, sinks);
      keys(first, q + 1);
      acc.scale(p.scale);
      hidden::store_channels<D>(out, acc, bad, lane);
    }
  }
}

// The same of dV (hidden rows of dO) and dK (of Q), in bf16 or in the item's part.
template <int D>
__device__ __forceinline__ void sum_keys_again(const Params& p, const int* pre, int at, int second,
                                               int lane) {
  using hidden::bf16;
  constexpr int kChunk = chunk_rows(D, false);
  const float sl2 = p.scale * kLog2e;
  for (; at >= 0; at = __ldcg(p.noted + at)) {
    const Item x = item<D, false>(p, pre, at >> 2);
    const int bh = x.b * p.kv_heads + x.h;
    float* part = part_of<D>(p, x, bh);
    for (int r = 0; r < 16; ++r) {
      const int row = 32 * (at & 3) + 16 * second + r, key = x.tile * kRows + row;
      if (key >= x.L) break;
      const int64_t place = (static_cast<int64_t>(bh) * p.n + key) * D;
      bf16* dv = static_cast<bf16*>(p.dv) + place;
      bf16* dk = static_cast<bf16*>(p.dk) + place;
      float* pv = part + row * D;  // unused without a part
      float* pk = pv + kRows * D;
      const uint32_t badv = part ? hidden::bad_channels<D>(pv, lane) : hidden::bad_channels<D>(dv, lane);
      const uint32_t badk = part ? hidden::bad_channels<D>(pk, lane) : hidden::bad_channels<D>(dk, lane);
      if (!__any_sync(0xffffffffu, (badv | badk) != 0)) continue;
      const int end = key < p.sinks ? x.L  // of the queries that see the key
                                    : static_cast<int>(min(static_cast<int64_t>(key) + p.window,
                                                           static_cast<int64_t>(x.L)));
      const bf16* krow = static_cast<const bf16*>(p.k) + place;
      const bf16* vrow = static_cast<const bf16*>(p.v) + place;
      // every chunk's queries of the item: visible ones are [lo, hi)
      auto chunks = [&](auto&& f) {
        for (int c = 0; c < x.nch; ++c) {
          const Chunk ch = chunk<D, false>(p, x, c);
          const int lo = max(ch.row, key), hi = min(ch.row + kChunk, end);
          if (!f(ch, lo, hi)) return false;
        }
        return true;
      };
      // (beside the sinks nearly all queries are hidden, and few are seen: these rows are
      // summed without the look)
      if (!(x.tile == 0 && p.sinks > 0 && key >= p.sinks) &&
          chunks([&](const Chunk& ch, int lo, int hi) {
            const bf16* q = static_cast<const bf16*>(p.q) + static_cast<int64_t>(ch.bh) * p.n * D;
            const bf16* g = static_cast<const bf16*>(p.dout) + static_cast<int64_t>(ch.bh) * p.n * D;
            const int last = min(ch.row + kChunk, x.L), a = min(lo, last), b = max(hi, ch.row);
            return !(hidden::any_bad<D>(q, ch.row, a, lane) || hidden::any_bad<D>(g, ch.row, a, lane) ||
                     hidden::any_bad<D>(q, max(a, b), last, lane) ||
                     hidden::any_bad<D>(g, max(a, b), last, lane));
          }))
        continue;
      hidden::Row<D> av, ak;
      av.zero();
      ak.zero();
      chunks([&](const Chunk& ch, int lo, int hi) {
        const bf16* q = static_cast<const bf16*>(p.q) + static_cast<int64_t>(ch.bh) * p.n * D;
        const bf16* g = static_cast<const bf16*>(p.dout) + static_cast<int64_t>(ch.bh) * p.n * D;
        const int64_t stats = static_cast<int64_t>(ch.bh) * p.npad;
        for (int from = lo; from < hi; from += 32) {
          const int j = min(from + lane, hi - 1);
          const float s = hidden::dot<D>(krow, q + static_cast<int64_t>(j) * D);
          const float dp = hidden::dot<D>(vrow, g + static_cast<int64_t>(j) * D);
          const float w = ex2_approx(fmaf(s, sl2, p.nlse2[stats + j]));
          av.add_rows(g, from, 0, min(32, hi - from), w, lane);
          ak.add_rows(q, from, 0, min(32, hi - from), w * (dp + p.nd[stats + j]), lane);
        }
        return !(hidden::settled<D>(av, badv) && hidden::settled<D>(ak, badk));
      });
      ak.scale(p.scale);
      if (part) {
        hidden::store_channels<D>(pv, av, badv, lane);
        hidden::store_channels<D>(pk, ak, badk, lane);
      } else {
        hidden::store_channels<D>(dv, av, badv, lane);
        hidden::store_channels<D>(dk, ak, badk, lane);
      }
    }
  }
}

// tx, ty: the tile that stays (K, V or Q, dO); cx, cy: the chunks (Q, dO or K, V); cf: the
// chunks of sinks (K); to0, to1: dV, dK or dQ twice.
template <int D, bool kDQ>
__global__ void __launch_bounds__(kThreads, 1)
    attn_sink_bwd_kernel(const __grid_constant__ CUtensorMap tx, const __grid_constant__ CUtensorMap ty,
                         const __grid_constant__ CUtensorMap cx, const __grid_constant__ CUtensorMap cf,
                         const __grid_constant__ CUtensorMap cy, const __grid_constant__ CUtensorMap to0,
                         const __grid_constant__ CUtensorMap to1, const Params p) {
  using C = Cfg<D, kDQ>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t bar = base + C::oBar;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NT; ++i) {
      mbar_init(bar + 8 * (C::bTFull + i), 1);
      // the issuer's commit, and (kDQ) the eight warps that have read the row statistics
      mbar_init(bar + 8 * (C::bTFree + i), kDQ ? 9 : 1);
    }
    for (int i = 0; i < C::NX; ++i) {
      mbar_init(bar + 8 * (C::bXFull + i), 1);
      mbar_init(bar + 8 * (C::bXFree + i), 1);
    }
    for (int i = 0; i < C::NY; ++i) {
      mbar_init(bar + 8 * (C::bYFull + i), 1);
      mbar_init(bar + 8 * (C::bYFree + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar + 8 * (C::bSFull + i), 1);
      mbar_init(bar + 8 * (C::bFix + i), 1);
    }
    for (int i = 0; i < C::NSB; ++i) mbar_init(bar + 8 * (C::bSFree + i), C::kWide ? 256 : 128);
    for (int i = 0; i < C::NPB; ++i) {
      mbar_init(bar + 8 * (C::bPFull + i), C::kWide ? 256 : 128);
      mbar_init(bar + 8 * (C::bPFree + i), 1);
    }
    for (int i = 0; i < C::NACC; ++i) {
      mbar_init(bar + 8 * (C::bAFull + i), 1);
      mbar_init(bar + 8 * (C::bAFree + i), 128);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(bar + 8 * (C::bIFull + i), 1);
      mbar_init(bar + 8 * (C::bIFree + i), kTakers + (C::kSplit ? 1 : 0));
    }
    mbar_init(bar + 8 * C::bDone, 2);  // one commit per MMA-issuing thread
    fence_barrier_init();
    for (int i = 0; i < 4; ++i) {
      *reinterpret_cast<volatile int*>(gbase + C::oNoted + 4 * i) = -1;
      *reinterpret_cast<volatile int*>(gbase + C::oFound + 4 * i) = 0;
    }
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tx);
    prefetch_tmap(&ty);
    prefetch_tmap(&cx);
    if (kDQ) prefetch_tmap(&cf);
    prefetch_tmap(&cy);
    prefetch_tmap(&to0);
    prefetch_tmap(&to1);
  }
  if (warp == 1) {
    tmem_alloc(base + C::oSlot, C::kTmemCols);
    tmem_relinquish();
  }
  // Everything above overlaps the previous kernel's tail.  The dQ kernel reads nothing of
  // the dK/dV kernel before it, but what the row kernel wrote is promised to be visible
  // only behind this wait (starting dQ blocks without it took 2 to 4 us off the backward:
  // 25.1 us against 27.7 at 2 x 4 heads x 333 x 64).
  pdl_wait();
  int* pre = reinterpret_cast<int*>(gbase + C::oPre);
  if (warp == 0) build_table<kDQ>(pre, p, lane);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(gbase + C::oSlot);

  int err = 0;
  if (warp < 4) {
    regs_dec<C::kRegsCtl, kLaunchRegs>();
    if (warp == 0) err = producer<D, kDQ>(p, pre, base, gbase, lane, &tx, &ty, &cx, &cf, &cy);
    if (warp == 1 && lane == 0) err = s_issuer<D, kDQ>(p, base, gbase, tmem);
    if (warp == 2 && lane == 0) err = grad_issuer<D, kDQ>(p, base, gbase, tmem);
    if (C::kSplit && warp == 3) err = y_producer<D, kDQ>(p, base, gbase, lane, &cy);
  } else if (warp < 12) {
    regs_inc<C::kRegsGrad, kLaunchRegs>();
    err = grad_warps<D, kDQ>(p, base, gbase, tmem, (warp - 4) >> 2, warp & 3, lane);
  } else {
    regs_dec<C::kRegsEpi, kLaunchRegs>();
    err = epi_warps<D, kDQ>(p, base, gbase, tmem, warp & 3, lane, &to0, &to1);
    if (err) bulk_wait_all0();  // a store that is still reading the staging
  }
  if (err) record_error(p.err, err);

  pdl_trigger();
  __syncthreads();
  if (warp == 2 && lane == 0) mma_commit(bar + 8 * C::bDone);
  if (warp == 1) {
    if (lane == 0) {  // every tensor-core operation of this CTA has completed
      mma_commit(bar + 8 * C::bDone);
      if (!mbar_wait(bar + 8 * C::bDone, 0)) record_error(p.err, kErrDone);
    }
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
  // The epilogue has stored every tile.  (Last, so that the code above stays together: in
  // the warps' own branch this cost 0.6 us a launch without being run.)
  if (warp >= 4 && warp < 12) {
    const int noted = *reinterpret_cast<volatile int*>(gbase + C::oNoted + 4 * (warp & 3));
    if (kDQ) sum_queries_again<D>(p, pre, noted, (warp - 4) >> 2, lane);
    else sum_keys_again<D>(p, pre, noted, (warp - 4) >> 2, lane);
  }
}

// D of a row is rowsum(dO O), but O comes rounded to bf16, and the error that this
// leaves in D is the same for all keys of the row: it falls with the root of their
// number, and a row of a few keys has large gradients.  (Relative error of dQ and dK
// at window 2: 0.0037, at lengths of 3: 0.010, where the rounding of dS and of the
// result make 0.0024.)  Rows that see at most kFew keys, the first of a sequence or
// all under a small window, therefore take D = sum_j P_j dP_j from their keys.
constexpr int kFew = 32;
// The rows of a sequence, from its first, that see few (npad: whole tiles of them).
__host__ __device__ __forceinline__ int few_rows(int window, int sinks, int npad) {
  return window <= kFew - sinks ? npad : kFew;
}

// -D of rows q0 .. q0 + 15 from their keys: a block of eight warps, each with eight keys
// (there are hardly more than 64), so that the block takes little longer than those that
// stream: the backward of 2 x 4 heads x 333 x 64 grows by 2 us, 4 with one warp for
// all keys.  Warp products of 16 rows by 8 keys; a
// lane's 16 bytes of a row are its operands of two products (which channels share a
// step does not matter to the sum).
template <int D>
__device__ __forceinline__ void row_terms(const Params& p, int b, int h, int L, int q0) {
  __shared__ float part[8][16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, t = lane & 3;
  const int bh = b * p.heads + h, bkv = b * p.kv_heads + h / p.group;
  auto piece = [&](const void* x, int head, int row) {  // the lane's first 16 bytes of a row
    return reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(x) +
                                          (static_cast<int64_t>(head) * p.n + min(row, L - 1)) * D) + t;
  };
  const uint4* q[2];
  const uint4* g[2];
  float nl[2], sum[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = min(q0 + r + 8 * i, L - 1);
    q[i] = piece(p.q, bh, row);
    g[i] = piece(p.dout, bh, row);
    nl[i] = -p.lse[static_cast<int64_t>(bh) * p.n + row] * kLog2e;
  }
  const float sl2 = p.scale * kLog2e;
  const int k0 = q0 >= p.window ? q0 - p.window + 1 : 0;  // the first row's window
  const int far = min(p.sinks, k0), far_steps = (far + 7) / 8;
  const int steps = far_steps + (min(q0 + 16, L) - k0 + 7) / 8;
#pragma unroll 1
  for (int i = warp; i < steps; i += 8) {
    const int first = i < far_steps ? 8 * i : k0 + 8 * (i - far_steps);
    const uint4* k = piece(p.k, bkv, first + r);
    const uint4* v = piece(p.v, bkv, first + r);
    float s[4] = {0.f, 0.f, 0.f, 0.f}, dp[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
    for (int c = 0; c < D / 32; ++c) {  // 32 channels
      auto step = [&](float (&acc)[4], const uint4* const (&a)[2], const uint4* b) {
        const uint4 x = a[0][4 * c], y = a[1][4 * c], z = b[4 * c];
        const uint32_t lo[4] = {x.x, y.x, x.y, y.y}, hi[4] = {x.z, y.z, x.w, y.w};
        mma16816(acc, lo, z.x, z.y, acc);
        mma16816(acc, hi, z.z, z.w, acc);
      };
      step(s, q, k);
      step(dp, g, v);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int row = q0 + r + 8 * (e >> 1), key = first + 2 * t + (e & 1);
      const bool seen = i < far_steps ? key < far
                                      : key <= row && (row - key < p.window || key < p.sinks);
      if (seen)
        sum[e >> 1] = fmaf(ex2_approx(fmaf(s[e], sl2, nl[e >> 1])), dp[e], sum[e >> 1]);
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 1);
    sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 2);
    if (t == 0) part[warp][r + 8 * i] = sum[i];
  }
  __syncthreads();
  if (threadIdx.x < 16 && q0 + static_cast<int>(threadIdx.x) < L) {
    float all = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) all += part[w][threadIdx.x];
    p.nd[static_cast<int64_t>(bh) * p.npad + q0 + threadIdx.x] = -all;
  }
}

// Row statistics (padded to whole tiles), zeros for the gradient rows of tiles
// that lie past their sequence's length, and the counters of the main kernels.
// The first blocks take the rows that see few keys, beside the others.
// Block = kRowsPer rows of one (sequence, head); a thread has eight elements
// (16 bytes) of kPer rows, all loaded before the first is used.
constexpr int kPer = 4;
template <int D>
constexpr int kRowsPer = kPer * 256 / (D / 8);  // 64 or 128: divides a tile
template <int D>
__global__ void __launch_bounds__(256, 3) sink_rows_kernel(const Params p) {
  constexpr int TPR = D / 8, kStep = 256 / TPR;  // threads per row, rows at once
  pdl_trigger();
  pdl_wait();
  if (blockIdx.x == 0 && threadIdx.x < 2) p.taken[threadIdx.x] = 0;
  if (static_cast<int>(blockIdx.x) < p.term_blocks) {  // sixteen rows
    const int per = few_rows(p.window, p.sinks, p.npad) / 16;
    const int bh = static_cast<int>(blockIdx.x) / per;
    const int f0 = (static_cast<int>(blockIdx.x) - bh * per) * 16;
    const int b = bh / p.heads, L = length_of(p, b);
    if (f0 < L) row_terms<D>(p, b, bh - b * p.heads, L, f0);
    return;
  }
  const int per = p.npad / kRowsPer<D>;  // blocks per (sequence, head)
  const int block = static_cast<int>(blockIdx.x) - p.term_blocks;
  const int bh = block / per;
  const int q0 = (block - bh * per) * kRowsPer<D> + threadIdx.x / TPR;
  const int part = threadIdx.x % TPR;
  const int b = bh / p.heads, h = bh - b * p.heads;
  const int L = length_of(p, b);
  uint4 ov[kPer], dv[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int q = q0 + i * kStep;
    const int64_t at = (static_cast<int64_t>(bh) * p.n + q) * D + part * 8;
    ov[i] = dv[i] = make_uint4(0, 0, 0, 0);
    if (q < L) {
      ov[i] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.o) + at);
      dv[i] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.dout) + at);
    }
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int q = q0 + i * kStep;
    const __nv_bfloat162* o2 = reinterpret_cast<const __nv_bfloat162*>(&ov[i]);
    const __nv_bfloat162* d2 = reinterpret_cast<const __nv_bfloat162*>(&dv[i]);
    float acc = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 of = __bfloat1622float2(o2[e]);
      const float2 df = __bfloat1622float2(d2[e]);
      acc = fmaf(of.x, df.x, acc);
      acc = fmaf(of.y, df.y, acc);
    }
#pragma unroll
    for (int off = TPR / 2; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
    if (part == 0) {
      const int64_t row = static_cast<int64_t>(bh) * p.npad + q;
      // stored negated: the main kernels form dP + (-D)
      if (q >= L || q >= few_rows(p.window, p.sinks, p.npad)) p.nd[row] = -acc;
      p.nlse2[row] = q < L ? -p.lse[static_cast<int64_t>(bh) * p.n + q] * kLog2e : -INFINITY;
    }
    if (q < p.n && q / kRows * kRows >= L) {
      const uint4 z = make_uint4(0, 0, 0, 0);
      const int64_t at = (static_cast<int64_t>(bh) * p.n + q) * D;
      reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.dq) + at)[part] = z;
      if (h % p.group == 0) {
        const int64_t kv = ((static_cast<int64_t>(b) * p.kv_heads + h / p.group) * p.n + q) * D;
        reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.dk) + kv)[part] = z;
        reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.dv) + kv)[part] = z;
      }
    }
  }
}

// dV and dK of split key tiles: the parts added in order, rounded once.  Block =
// 1024 / D rows of 128 (grid x: rows of the listed tiles; y: dV, dK).
template <int D>
__global__ void __launch_bounds__(256) sink_join_kernel(const Params p, int tiles) {
  constexpr int TPR = D / 4, kPer = 256 / TPR;  // threads per row, rows per block
  pdl_trigger();
  pdl_wait();
  const int blocks = kRows / kPer;
  const int64_t tl = blockIdx.x / blocks;  // (sequence and head, listed tile)
  const int r = static_cast<int>(blockIdx.x % blocks) * kPer + threadIdx.x / TPR;
  const int c = 4 * (threadIdx.x % TPR), out = blockIdx.y;
  const int64_t bh = tl / tiles;
  // the list has tile 0 when it is split, and the others when they are
  const int tile = static_cast<int>(tl - bh * tiles) + (p.s0 > 1 ? 0 : 1);
  const int L = length_of(p, static_cast<int>(bh / p.kv_heads));
  const int k = tile * kRows + r;
  if (tile * kRows >= L || k >= p.n) return;  // zeroed with the row statistics
  const int parts = tile == 0 ? p.s0 : p.s1;
  const float* src = tile == 0
                         ? p.part0 + bh * parts * 2 * kRows * D
                         : p.part1 + (bh * (p.ntiles - 1) + tile - 1) * parts * 2 * kRows * D;
  src += (static_cast<int64_t>(out) * kRows + r) * D + c;
  const int64_t all = static_cast<int64_t>(query_chunks(tile, L, p.window, p.sinks, chunk_rows(D, false))) * p.group;
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = 0; i < parts; ++i) {
    if (all * i / parts == all * (i + 1) / parts) continue;  // an empty part was not written
    const float4 v = *reinterpret_cast<const float4*>(src + static_cast<int64_t>(i) * 2 * kRows * D);
    sum.x += v.x;
    sum.y += v.y;
    sum.z += v.z;
    sum.w += v.w;
  }
  __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(out == 0 ? p.dv : p.dk) + (bh * p.n + k) * D + c;
  *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(sum.x, sum.y), pack_bf16(sum.z, sum.w));
}

struct Plan {
  int npad, ntiles, s0, s1;
  int64_t taken, nd, nlse2, noted, part0, part1, bytes;  // workspace offsets and size
};

// Cuts key tiles into parts: the first ones when they are more than a third of an
// SM's even share of all chunks (and larger than the others), the others when they
// exceed that share; never below 1024 queries a part, which costs a tile of fp32
// written and read.
Plan make_plan(const SinkArgs& a) {
  Plan w;
  w.ntiles = (a.n + kRows - 1) / kRows;
  w.npad = w.ntiles * kRows;
  const int64_t group = a.heads / a.kv_heads, bkv = static_cast<int64_t>(a.batch) * a.kv_heads;
  const int chunk = chunk_rows(a.d, false), f = kRows / chunk;  // f chunks span a tile
  const int64_t c0 = group * query_chunks(0, a.n, a.window, a.sinks, chunk);
  const int64_t c1 =
      w.ntiles > 1 ? group * query_chunks(1, a.n, a.window, a.sinks, chunk) : 0;
  // tile t >= 1 has min(per, rest - f t) chunks a head: its window's, or to the sequence's end
  const int64_t per = (static_cast<int64_t>(a.window) + kRows - 1 + chunk - 1) / chunk;
  const int64_t rest = (static_cast<int64_t>(a.n) + chunk - 1) / chunk, last = w.ntiles - 1;
  int64_t m = rest > per ? (rest - per) / f : 0;  // tiles 1..m have `per`
  if (m > last) m = last;
  const int64_t all = c0 + group * (m * per + (last - m) * rest -
                                    f * (last * (last + 1) - m * (m + 1)) / 2);
  auto at_least = [](int64_t x, int64_t lo) { return x < lo ? lo : x; };
  const int64_t share = (all * bkv + 147) / 148;
  const int64_t least = 1024 / chunk;  // chunks of a part, at least
  const int64_t cap1 = at_least(share, least);
  const int64_t s1 = (c1 + cap1 - 1) / cap1;
  const int64_t cap0 = at_least(share / 3, at_least(s1 > 1 ? cap1 : c1, least));
  const int64_t s0 = (c0 + cap0 - 1) / cap0;
  w.s0 = static_cast<int>(s0 < 1 ? 1 : s0);
  w.s1 = static_cast<int>(s1 < 1 ? 1 : s1);
  const int64_t rows = static_cast<int64_t>(a.batch) * a.heads * w.npad;
  const int64_t tile = 2ll * kRows * a.d * 4;
  w.taken = 0;
  w.nd = 256;
  w.nlse2 = w.nd + align_up(rows * 4, 256);
  w.noted = w.nlse2 + align_up(rows * 4, 256);
  // four words an item, of the kernel that has more of them
  const int64_t tiles_q = static_cast<int64_t>(a.batch) * a.heads * w.ntiles;
  const int64_t tiles_k = bkv * (w.s0 + static_cast<int64_t>(w.ntiles - 1) * w.s1);
  w.part0 = w.noted + align_up((tiles_q > tiles_k ? tiles_q : tiles_k) * 16, 256);
  w.part1 = w.part0 + (w.s0 > 1 ? bkv * w.s0 * tile : 0);
  w.bytes = w.part1 + (w.s1 > 1 ? bkv * (w.ntiles - 1) * w.s1 * tile : 0);
  return w;
}

template <int D, bool kDQ>
cudaError_t launch_main(const SinkArgs& a, Params p, cudaStream_t stream) {
  using C = Cfg<D, kDQ>;
  const int64_t hq = static_cast<int64_t>(a.batch) * a.heads;
  const int64_t hk = static_cast<int64_t>(a.batch) * a.kv_heads;
  CUtensorMap tx, ty, cx, cf, cy, to0, to1;
  const bool maps =
      kDQ ? make_tmap_bf16_rows(&tx, a.q, D, a.n, hq, kRows) &&
                make_tmap_bf16_rows(&ty, a.dout, D, a.n, hq, kRows) &&
                make_tmap_bf16_rows(&cx, a.k, D, a.n, hk, C::kChunk) &&
                make_tmap_bf16_rows(&cy, a.v, D, a.n, hk, C::kChunk) &&
                make_tmap_bf16_rows(&to0, a.dq, D, a.n, hq, kRows) &&
                make_tmap_bf16_rows(&to1, a.dq, D, a.n, hq, kRows)
          : make_tmap_bf16_rows(&tx, a.k, D, a.n, hk, kRows) &&
                make_tmap_bf16_rows(&ty, a.v, D, a.n, hk, kRows) &&
                make_tmap_bf16_rows(&cx, a.q, D, a.n, hq, C::kChunk) &&
                make_tmap_bf16_rows(&cy, a.dout, D, a.n, hq, C::kChunk) &&
                make_tmap_bf16_rows(&to0, a.dv, D, a.n, hk, kRows) &&
                make_tmap_bf16_rows(&to1, a.dk, D, a.n, hk, kRows);
  if (!maps) return cudaErrorInvalidValue;
  cf = cx;  // without sinks, or with every key in every window, no tile has chunks of sinks
  if (kDQ && a.sinks > 0 && a.n > a.window &&
      !make_tmap_first_rows(&cf, a.k, D, a.n, hk, a.sinks, C::kChunk))
    return cudaErrorInvalidValue;
  const int64_t items = kDQ ? hq * p.ntiles
                            : hk * (p.s0 + static_cast<int64_t>(p.ntiles - 1) * p.s1);
  if (items > (1ll << 28)) return cudaErrorInvalidValue;  // four words each are numbered in 31 bits
  p.items = static_cast<int>(items);
  cudaError_t e = cudaFuncSetAttribute(attn_sink_bwd_kernel<D, kDQ>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  const int grid = static_cast<int>(items < num_sms() ? items : num_sms());
  return launch_pdl(attn_sink_bwd_kernel<D, kDQ>, dim3(grid), dim3(kThreads), C::kSmem, stream, tx,
                    ty, cx, cf, cy, to0, to1, p);
}

template <int D>
cudaError_t run(const SinkArgs& a, cudaStream_t stream) {
  const Plan w = make_plan(a);
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  Params p = {};
  p.q = a.q;
  p.k = a.k;
  p.v = a.v;
  p.o = a.o;
  p.dout = a.dout;
  p.lse = a.lse;
  p.lengths = a.lengths;
  p.dq = a.dq;
  p.dk = a.dk;
  p.dv = a.dv;
  p.taken = reinterpret_cast<int*>(ws + w.taken);
  p.nd = reinterpret_cast<float*>(ws + w.nd);
  p.nlse2 = reinterpret_cast<float*>(ws + w.nlse2);
  p.noted = reinterpret_cast<int*>(ws + w.noted);
  p.part0 = reinterpret_cast<float*>(ws + w.part0);
  p.part1 = reinterpret_cast<float*>(ws + w.part1);
  p.err = a.err;
  p.batch = a.batch;
  p.heads = a.heads;
  p.kv_heads = a.kv_heads;
  p.group = a.heads / a.kv_heads;
  p.n = a.n;
  p.npad = w.npad;
  p.ntiles = w.ntiles;
  p.window = a.window;
  p.sinks = a.sinks;
  p.s0 = w.s0;
  p.s1 = w.s1;
  p.scale = a.scale;
  const int64_t hq = static_cast<int64_t>(a.batch) * a.heads;
  const int64_t terms = hq * (few_rows(a.window, a.sinks, w.npad) / 16);
  const int64_t blocks = terms + hq * (w.npad / kRowsPer<D>);
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  p.term_blocks = static_cast<int>(terms);
  cudaError_t e = launch_pdl(sink_rows_kernel<D>, dim3(static_cast<unsigned>(blocks)), dim3(256), 0,
                             stream, p);
  if (e == cudaSuccess) e = launch_main<D, false>(a, p, stream);
  if (e == cudaSuccess) e = launch_main<D, true>(a, p, stream);
  if (e != cudaSuccess) return e;
  const int tiles = (w.s0 > 1 ? 1 : 0) + (w.s1 > 1 ? w.ntiles - 1 : 0);
  if (tiles == 0) return cudaSuccess;
  const int64_t joins = static_cast<int64_t>(a.batch) * a.kv_heads * tiles * (kRows / (1024 / D));
  if (joins > INT32_MAX) return cudaErrorInvalidValue;
  return launch_pdl(sink_join_kernel<D>, dim3(static_cast<unsigned>(joins), 2), dim3(256), 0, stream,
                    p, tiles);
}

}  // namespace

size_t sink_bwd_workspace_bytes(const SinkArgs& a) { return static_cast<size_t>(make_plan(a).bytes); }

cudaError_t launch_attn_sink_bwd(const SinkArgs& a, cudaStream_t stream) {
  return a.d == 64 ? run<64>(a, stream) : run<128>(a, stream);
}

}  // namespace nb
