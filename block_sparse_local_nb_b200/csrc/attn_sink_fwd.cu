// Causal attention with a sliding window and visible first tokens (sinks),
// forward, on the 5th-generation tensor cores (tcgen05 + TMEM), bf16 in / fp32
// accumulate: query q sees key k when k <= q, k < L and (q - k < window or
// k < sinks); S = Q K^T / sqrt(d), online softmax, O = P V, lse.
//
// Work item = one query tile of 128 rows of one (sequence, query head).  Its keys
// are the tokens [q0 - window + 1, q0 + 127] clipped to the sequence, in blocks of
// 64 from exactly that first token (a TMA box may start at any row), and before
// them, when they begin past the sinks' blocks, one or two blocks of sinks.  A
// chunk is two blocks, wherever they lie.  A block between the window's edge and
// the diagonal is visible to all rows and takes no mask; in the others a row's
// visible columns are one 64-bit word.
// A persistent grid of one CTA per SM walks the items, the longest (last) tiles
// of a sequence first and every second round of items in reverse, so that the
// SMs' totals differ by little; the heads that share a key/value head follow one
// another, so its chunks come from L2.
//
// Warp roles (512 threads, four warpgroups with reallocated registers):
//   warp 0     TMA producer: Q tile and K chunks (128-byte swizzled boxes; rows
//              past the tensor are zero-filled by TMA).
//   warp 3     TMA producer of the V chunks, which go separately because a K
//              stage is free after its S product and a V stage only after P V.
//              Rows past the sequence's length are set to zero in shared memory
//              before the chunk is handed on: P is 0 there, but 0 x NaN is not.
//              (Of the sinks' blocks the tensor map reads the sinks alone; what other
//              hidden rows may do is mended at the end, sink_hidden.cuh.)
//   warp 1     TMEM owner and S issuer (one thread): S_c = Q K_c^T (M 128, N 128)
//              into three TMEM buffers at d = 64, two at d = 128.
//   warp 2     P V issuer (one thread): O_h += P_c,h V_c,h (M 128, N d, K 64; P
//              read from TMEM).
//   warps 4-11 softmax, two groups of four warps; thread (r, half) owns row r
//              (TMEM lane r) and 64 of the chunk's 128 columns, with a running
//              max, sum and output of its own; P = 2^(s - m) goes back into TMEM
//              as bf16 over the scores it came from.  P is rounded to bf16 as the
//              operand of P V; the sum takes it unrounded.  The output is rescaled
//              only when the half's max grows by more than 2^8.
//   warps 12-15 epilogue: O = (O_0 2^(m_0 - M) + O_1 2^(m_1 - M)) / l, lse = M +
//              log l, one TMA tensor store per tile.
// Every mbarrier wait is bounded; on a timeout the kernel records an error code
// and tears down (frees TMEM) instead of hanging.
#include <math.h>

#include <cudaTypedefs.h>

#include <mutex>

#include "schedule.cuh"
#include "serving.cuh"
#include "sink_hidden.cuh"

namespace nb {
namespace {

using namespace sm100;

constexpr int kThreads = 512;
constexpr int kLaunchRegs = 65536 / kThreads / 8 * 8;  // per thread at launch
constexpr int kRows = 128;   // query rows per tile
constexpr int kHalf = 64;    // keys of a block
constexpr int kChunk = 128;  // keys of a chunk: two blocks
constexpr int kSlab = 128 * 128;  // one swizzled box: 128 rows x 64 bf16
constexpr int kItems = 4;          // items decoded ahead
constexpr int kTakers = 15;         // arrivals that free one: V producer, 2 issuers, 8 + 4 warps
constexpr float kTau = 8.0f;      // lazy-rescale threshold, log2 units
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <int D>
struct Cfg {
  static constexpr int NQ = 2;                 // Q tile buffers
  static constexpr int NKV = D == 64 ? 3 : 2;  // K chunk stages, and as many V chunk stages
  static constexpr int NSB = NKV;              // S buffers
  static constexpr int kQBytes = kRows * D * 2;
  static constexpr int kKBytes = kChunk * D * 2;
  static constexpr int oQ = 0;
  static constexpr int oK = oQ + NQ * kQBytes;
  static constexpr int oV = oK + NKV * kKBytes;
  static constexpr int oStg = oV + NKV * kKBytes;  // output staging, 64 columns of a tile
  static constexpr int oItem = oStg + kSlab;  // ring of items
  static constexpr int oBar = oItem + kItems * 32;
  static_assert(oItem % 16 == 0, "items are read 16 bytes at once");
  // barrier indices ([S buffer][half] for P, [half][buffer] for O)
  static constexpr int bQFull = 0, bQFree = bQFull + NQ, bKFull = bQFree + NQ,
                       bVFull = bKFull + NKV, bSFull = bVFull + NKV, bSFree = bSFull + NSB,
                       bPFull = bSFree + NSB, bOFull = bPFull + NSB, bOFree = bOFull + 1,
                       bXFull = bOFree + 1, bXFree = bXFull + 2,
                       bIFull = bXFree + 2, bIFree = bIFull + kItems, bVFix = bIFree + kItems,
                       bDone = bVFix + 1, nBar = bDone + 1;
  static constexpr int oSlot = oBar + nBar * 8;
  // per-tile hand-off of the halves' running max and sum to the epilogue warps:
  // [parity][half][m, l][row] fp32
  static constexpr int oBad = oSlot + 8;  // some row of this CTA's tiles is not finite
  static constexpr int oXSum = oSlot + 16;
  static constexpr int oSched = oXSum + 2 * 2 * 2 * 128 * 4;  // work-order prefix table
  static constexpr int kSmem = oSched + kSchedBytes + 1024;  // + slack for 1024-byte alignment
  static_assert(oXSum % 4 == 0 && oSched % 4 == 0, "words");
  static_assert(kSmem <= 227 * 1024, "shared memory per CTA");
  static constexpr uint32_t kTmemCols = 512;
  // S buffer i: columns [128 i, 128 i + 128).  Half h's P (64 keys, two bf16
  // per column) overwrites the first 32 columns of that half's 64 S columns.
  // The O accumulators follow (d = 64: 384 + 2 x 64 columns; d = 128: 256 +
  // 2 x 128).
  static constexpr uint32_t tS = 0;
  __device__ static constexpr uint32_t tP(int sb, int h) { return tS + sb * kChunk + 64 * h; }
  __device__ static constexpr uint32_t tO(int h) { return NSB * kChunk + h * D; }
  static_assert(NSB * kChunk + 2 * D <= kTmemCols, "tensor memory columns");
  // registers per thread after reallocation: TMA/MMA warpgroup, each softmax
  // warpgroup, epilogue warpgroup (the 16 warps share the 64K-register file;
  // the d = 128 softmax spills less with 176, the d = 64 one runs faster at 168)
  static constexpr int kRegsCtl = 56;
  static constexpr int kRegsSoft = D == 64 ? 168 : 176;
  static constexpr int kRegsEpi = D == 64 ? 120 : 104;
  static_assert(128 * (kRegsCtl + 2 * kRegsSoft + kRegsEpi) <= 65536, "register budget");
};

struct Params {
  AttnArgs a;
  int group;   // query heads per key/value head
  int window, sinks;
  int ntiles;  // query tiles per (batch, head)
  int items;   // batch * heads * ntiles
};

struct alignas(16) Item {
  int b, h, tile, L;
  int k0;    // first key of the window's blocks
  int far;   // blocks of sinks (keys 0.. and 64..) before them
  int nch;   // chunks of two blocks, 0 for a tile past the sequence's length
  // first of the 64 keys of block i; the last chunk's second may lie past the tile's keys
  __device__ __forceinline__ int key(int i) const {
    return i < far ? i * kHalf : k0 + (i - far) * kHalf;
  }
};

__device__ __forceinline__ Item decode_bht(const Params& p, int b, int h, int tile, int L) {
  Item x;
  x.b = b;
  x.h = h;
  x.tile = tile;
  x.L = L;  // clamped to [0, n]
  x.k0 = x.far = x.nch = 0;
  const int q0 = tile * kRows;
  if (q0 < L) {
    // tokens below k0 are outside every row's window
    x.k0 = q0 >= p.window ? q0 - p.window + 1 : 0;
    if (p.sinks > 0 && x.k0 > 0) {
      const int f = (p.sinks + kHalf - 1) / kHalf;
      if (x.k0 <= f * kHalf) x.k0 = 0;  // no more blocks than with separate ones
      else x.far = f;
    }
    const int end = min(q0 + kRows, L);
    x.nch = (x.far + (end - x.k0 + kHalf - 1) / kHalf + 1) / 2;
  }
  return x;
}

// This CTA's item of round r: every second round runs backwards over the CTAs,
// so that costs falling along the list even out.
__device__ __forceinline__ int item_at(int r) {
  const int c = static_cast<int>(blockIdx.x), g = static_cast<int>(gridDim.x);
  return r * g + ((r & 1) ? g - 1 - c : c);
}

// Item k of the list: non-empty tiles when balanced (tiles from the last to the
// first, heads innermost), else every tile.
__device__ __forceinline__ Item sched_item(const Params& p, const Sched& s, int k) {
  const int heads = p.a.heads;
  if (!s.balanced) {
    const int per = heads * p.ntiles;
    const int b = k / per, rem = k - b * per;
    const int t = rem / heads;
    return decode_bht(p, b, rem - t * heads, p.ntiles - 1 - t, sched_length(s, p.a, b));
  }
  int lo = 0, hi = p.a.batch - 1;  // largest b with pre[b] <= k
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s.pre[mid] <= k) lo = mid; else hi = mid - 1;
  }
  const int L = sched_length(s, p.a, lo), rem = k - s.pre[lo];
  const int t = rem / heads;
  return decode_bht(p, lo, rem - t * heads, (L + kRows - 1) / kRows - 1 - t, L);
}

// error codes: 0x60 + site
enum : int { kErrQFree = 0x61, kErrKFree, kErrQFull, kErrKFull, kErrSFree, kErrOFree, kErrPFull,
             kErrSFull, kErrPPrev, kErrOFull, kErrDone, kErrXFull, kErrXFree, kErrVFree, kErrVFull,
             kErrVFix, kErrIFree, kErrIFull };

static_assert(sizeof(Item) <= 32, "slot of the ring");

// The rd-th item of this CTA from the ring, for the warps that work on it; x.nch < 0
// after the last.  Called by whole warps.
template <int D>
__device__ __forceinline__ bool next_item(Item& x, int rd, uint32_t bar, const uint8_t* gbase,
                                          int lane) {
  using C = Cfg<D>;
  const int i = rd % kItems;
  if (!__all_sync(0xffffffffu, mbar_wait(bar + 8 * (C::bIFull + i), (rd / kItems) & 1)))
    return false;
  x = *reinterpret_cast<const Item*>(gbase + C::oItem + i * 32);
  __syncwarp();  // every lane has read it
  if (lane == 0) mbar_arrive(bar + 8 * (C::bIFree + i));
  return true;
}

// Number of chunks of the rd-th item, for the single-thread roles; < 0 after the last,
// kNoItem on a timeout.
constexpr int kNoItem = -2;
template <int D>
__device__ __forceinline__ int next_chunks(int rd, uint32_t bar, const uint8_t* gbase) {
  using C = Cfg<D>;
  const int i = rd % kItems;
  if (!mbar_wait(bar + 8 * (C::bIFull + i), (rd / kItems) & 1)) return kNoItem;
  const int nch = reinterpret_cast<const Item*>(gbase + C::oItem + i * 32)->nch;
  mbar_arrive(bar + 8 * (C::bIFree + i));
  return nch;
}

// Items, Q tiles and K chunks (warp 0, one thread).  An item is decoded once, here,
// and handed to the other roles through a ring: its search and divisions take a
// thousand cycles, which each role spent between two tiles before.
template <int D>
__device__ int producer(const Params& p, const Sched& sch, uint32_t base, uint8_t* gbase,
                        const CUtensorMap* tq, const CUtensorMap* tk) {
  using C = Cfg<D>;
  const uint32_t bar = base + C::oBar;
  Ring<C::NQ> qr;
  Ring<C::NKV> kr;
  auto run = [&]() -> int {
    for (int rd = 0;; ++rd) {
      const int it = item_at(rd), i = rd % kItems;
      Item x;
      if (it < sch.count) x = sched_item(p, sch, it);
      else x.nch = -1;
      if (!mbar_wait(bar + 8 * (C::bIFree + i), ((rd / kItems) & 1) ^ 1)) return kErrIFree;
      *reinterpret_cast<Item*>(gbase + C::oItem + i * 32) = x;
      mbar_arrive(bar + 8 * (C::bIFull + i));
      if (x.nch < 0) break;
      if (x.nch == 0) continue;
      const int bh = x.b * p.a.heads + x.h, bkv = bh / p.group;
      if (!mbar_wait(bar + 8 * (C::bQFree + qr.i), qr.ph ^ 1)) return kErrQFree;
      mbar_arrive_expect_tx(bar + 8 * (C::bQFull + qr.i), C::kQBytes);
#pragma unroll
      for (int s = 0; s < D / 64; ++s)
        tma_load_3d(base + C::oQ + qr.i * C::kQBytes + s * kSlab, tq, bar + 8 * (C::bQFull + qr.i),
                    s * 64, x.tile * kRows, bh);
      qr.next();
      for (int c = 0; c < x.nch; ++c) {
        if (!mbar_wait(bar + 8 * (C::bSFull + kr.i), kr.ph ^ 1)) return kErrKFree;
        const uint32_t full = bar + 8 * (C::bKFull + kr.i);
        mbar_arrive_expect_tx(full, C::kKBytes);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int s = 0; s < D / 64; ++s)
            tma_load_3d(base + C::oK + kr.i * C::kKBytes + s * kSlab + h * kHalf * 128, tk, full,
                        s * 64, x.key(2 * c + h), bkv);
        kr.next();
      }
    }
    return 0;
  };
  const int err = run();
  // copies that nobody took have landed before the block exits
  drain_ring<C::NQ>(qr.i, qr.ph, [&](int i, uint32_t ph) { mbar_wait(bar + 8 * (C::bQFull + i), ph); });
  drain_ring<C::NKV>(kr.i, kr.ph, [&](int i, uint32_t ph) { mbar_wait(bar + 8 * (C::bKFull + i), ph); });
  return err;
}

// V chunks (warp 3, the whole warp; lane 0 issues).  A chunk that reaches past
// the sequence's length lands on a barrier of its own; the warp zeroes the rows
// past the length and then hands the chunk on.  tf: V's map for the sinks' blocks.
template <int D>
__device__ int v_producer(const Params& p, uint32_t base, uint8_t* gbase, int lane,
                          const CUtensorMap* tv, const CUtensorMap* tf) {
  using C = Cfg<D>;
  const uint32_t bar = base + C::oBar;
  int fixes = 0;
  Ring<C::NKV> vr;
  auto run = [&]() -> int {
    for (int rd = 0;; ++rd) {
      Item x;
      if (!next_item<D>(x, rd, bar, gbase, lane)) return kErrIFull;
      if (x.nch < 0) break;
      const int bkv = (x.b * p.a.heads + x.h) / p.group;
      for (int c = 0; c < x.nch; ++c) {
        const int st = vr.i;
        const int y[2] = {x.key(2 * c), x.key(2 * c + 1)};
        // rows of a block from L - y on hold other data
        const bool fix = max(y[0], y[1]) + kHalf > x.L && x.L < p.a.n;
        const uint32_t full = bar + 8 * (C::bVFull + st);
        const uint32_t land = fix ? bar + 8 * C::bVFix : full;
        bool ok = true;
        if (lane == 0) {
          ok = mbar_wait(bar + 8 * (C::bSFree + st), vr.ph ^ 1);
          if (ok) {
            mbar_arrive_expect_tx(land, C::kKBytes);
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int s = 0; s < D / 64; ++s)
                tma_load_3d(base + C::oV + st * C::kKBytes + s * kSlab + h * kHalf * 128,
                            2 * c + h < x.far ? tf : tv, land, s * 64, y[h], bkv);
          }
        }
        if (!__all_sync(0xffffffffu, ok)) return kErrVFree;
        if (fix) {
          if (!__all_sync(0xffffffffu, mbar_wait(land, fixes & 1))) return kErrVFix;
          ++fixes;
          uint4* v = reinterpret_cast<uint4*>(gbase + C::oV + st * C::kKBytes);
          for (int h = 0; h < 2; ++h)  // whole 128-byte rows, so the swizzle does not matter
            for (int s = 0; s < D / 64; ++s)
              for (int i = max(x.L - y[h], 0) * 8 + lane; i < kHalf * 8; i += 32)
                v[s * (kSlab / 16) + h * kHalf * 8 + i] = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(full);
        }
        vr.next();
      }
    }
    return 0;
  };
  const int err = run();
  if (err == kErrVFix) mbar_wait(bar + 8 * C::bVFix, fixes & 1);
  drain_ring<C::NKV>(vr.i, vr.ph, [&](int i, uint32_t ph) { mbar_wait(bar + 8 * (C::bVFull + i), ph); });
  return err;
}

// S = Q K^T for every chunk into S buffer G % NSB (warp 1, one thread).  P of
// chunk G replaces S in that buffer, so S of chunk G + NSB waits for P V of
// chunk G, which the other issuer signals on bSFree.
// A lone thread takes four cycles and more an instruction, on the chain from P to the
// next S: positions advance by steps, descriptors by adds.
template <int D>
__device__ int s_issuer(uint32_t base, const uint8_t* gbase, uint32_t tmem) {
  using C = Cfg<D>;
  const uint32_t bar = base + C::oBar;
  constexpr uint32_t kIdS = idesc_bf16_f32(128, kChunk, false, false);  // Q K^T: both K-major
  const uint64_t dQ0 = smem_desc_sw128(base + C::oQ, 0, 1024);
  const uint64_t dK0 = smem_desc_sw128(base + C::oK, 0, 1024);
  Ring<C::NQ> qr;
  Ring<C::NKV> kr;  // K stage and S buffer
  for (int rd = 0;; ++rd) {
    const int nch = next_chunks<D>(rd, bar, gbase);
    if (nch == kNoItem) return kErrIFull;
    if (nch < 0) break;
    if (nch == 0) continue;
    if (!mbar_wait(bar + 8 * (C::bQFull + qr.i), qr.ph)) return kErrQFull;
    const uint64_t dQ = desc_add(dQ0, qr.i * (C::kQBytes >> 4));
    for (int c = 0; c < nch; ++c) {
      const uint64_t dK = desc_add(dK0, kr.i * (C::kKBytes >> 4));
      const uint32_t tD = tmem + C::tS + kr.i * kChunk;
      const uint32_t kfull = bar + 8 * (C::bKFull + kr.i), sfree = bar + 8 * (C::bSFree + kr.i);
      // both are asked before the first answer is looked at
      const bool okk = mbar_try_wait(kfull, kr.ph), oks = mbar_try_wait(sfree, kr.ph ^ 1);
      if (!okk && !mbar_wait(kfull, kr.ph)) return kErrKFull;
      if (!oks && !mbar_wait(sfree, kr.ph ^ 1)) return kErrSFree;
      tc_fence_after();
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint32_t off = ((k >> 2) * kSlab + (k & 3) * 32) >> 4;  // descriptor address units
        mma_bf16_ss(tD, desc_add(dQ, off), desc_add(dK, off), kIdS, k > 0);
      }
      mma_commit(bar + 8 * (C::bSFull + kr.i));  // also frees the K stage: its only reader
      if (c == nch - 1) mma_commit(bar + 8 * (C::bQFree + qr.i));  // the tile's S products issued
      kr.next();
    }
    qr.next();
  }
  return 0;
}

// O_h += P_h V_h for every chunk and half (warp 2, one thread): P from TMEM,
// V from shared memory.  Completion of a chunk's products frees its S buffer
// and its V stage (its S completed before its softmax began).
template <int D>
__device__ int pv_issuer(uint32_t base, const uint8_t* gbase, uint32_t tmem) {
  using C = Cfg<D>;
  const uint32_t bar = base + C::oBar;
  constexpr uint32_t kIdPV = idesc_bf16_f32(128, D, false, true);  // V is MN-major (K = 64 per half)
  // V is MN-major: 64-column swizzle atoms kSlab apart, 8-key groups 1024 bytes apart
  const uint64_t dV0 = smem_desc_sw128(base + C::oV, kSlab, 1024);
  Ring<C::NKV> vr;  // V stage and S buffer
  Ring<1> o;
  for (int rd = 0;; ++rd) {
    const int nch = next_chunks<D>(rd, bar, gbase);
    if (nch == kNoItem) return kErrIFull;
    if (nch < 0) break;
    if (nch == 0) continue;
    if (!mbar_wait(bar + 8 * C::bOFree, o.ph ^ 1)) return kErrOFree;
    for (int c = 0; c < nch; ++c) {
      const uint64_t dV = desc_add(dV0, vr.i * (C::kKBytes >> 4));
      const uint32_t tP0 = tmem + C::tS + vr.i * kChunk;
      if (!mbar_wait(bar + 8 * (C::bVFull + vr.i), vr.ph)) return kErrVFull;
      if (!mbar_wait(bar + 8 * (C::bPFull + vr.i), vr.ph)) return kErrPFull;
      tc_fence_after();
#pragma unroll
      for (int h = 0; h < 2; ++h)  // each half's 64 keys into its own O accumulator
#pragma unroll
        for (int k = 0; k < 4; ++k)  // 16 keys = 8 P columns = 2048 bytes of V per step
          mma_bf16_ts(tmem + C::tO(h), tP0 + 64 * h + 8 * k, desc_add(dV, (h * 8192 + k * 2048) >> 4),
                      kIdPV, c > 0 || k > 0);
      // frees the S buffer and the V stage, and tells the softmax warps that O may be rescaled
      mma_commit(bar + 8 * (C::bSFree + vr.i));
      if (c == nch - 1) mma_commit(bar + 8 * C::bOFull);
      vr.next();
    }
    o.next();
  }
  return 0;
}

// Bits [lo, hi) of a 64-bit word (clipped to it).
__device__ __forceinline__ uint64_t bit_range(int lo, int hi) {
  lo = max(lo, 0);
  hi = min(hi, 64);
  return hi > lo ? (~0ull >> (64 - (hi - lo))) << lo : 0ull;
}

template <int D>
__device__ int softmax_warps(const Params& p, const Sched& sch, uint32_t base, uint8_t* gbase,
                             uint32_t tmem, int wq, int hf, int lane) {
  using C = Cfg<D>;
  const AttnArgs& a = p.a;
  const uint32_t bar = base + C::oBar;
  const int r = wq * 32 + lane;  // tile row == TMEM lane
  const uint32_t trow = tmem + (static_cast<uint32_t>(wq * 32) << 16);
  const float sl2 = a.scale * kLog2e;
  float* xs = reinterpret_cast<float*>(gbase + C::oXSum);
  auto all_ok = [](bool ok) { return __all_sync(0xffffffffu, ok); };
  // a tile entirely past its sequence's length: O = 0, lse = -inf
  // (the tile's rows are contiguous: the 256 threads store it as one coalesced run)
  auto zero_tile = [&](const Item& x) {
    const int64_t row0 = (static_cast<int64_t>(x.b) * a.heads + x.h) * a.n + x.tile * kRows;
    const int rows = min(kRows, a.n - x.tile * kRows);
    uint4* out = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(const_cast<void*>(a.o)) +
                                          row0 * D);
    for (int i = hf * 128 + r; i < rows * (D / 8); i += 256) out[i] = make_uint4(0, 0, 0, 0);
    if (a.lse && hf == 0 && r < rows) a.lse[row0 + r] = -INFINITY;
  };
  Ring<C::NSB> sr;
  int tc = 0;
  for (int rd = 0;; ++rd) {
    Item x;
    if (!next_item<D>(x, rd, bar, gbase, lane)) return kErrIFull;
    if (x.nch < 0) break;
    const int q0 = x.tile * kRows, q = q0 + r, qw = q0 + wq * 32;  // qw: the warp's first row
    if (x.nch == 0) {  // the whole tile is padding
      zero_tile(x);
      continue;
    }
    float m_used = -INFINITY, l = 0.f;
    for (int c = 0; c < x.nch; ++c) {
      const int sb = sr.i;
      const int blk = 2 * c + hf, kc = x.key(blk);  // this half's block and its first key
      // 32 keys visible to every row of the warp: none after its first row, none at or
      // before its last row's window edge, and all its rows below the length.  (The
      // bits of a mask cost two instructions a key, a quarter of the warp's time.)
      bool whole[2];
#pragma unroll
      for (int j = 0; j < 2; ++j)
        whole[j] = blk >= x.far && kc + 32 * j + 31 <= qw && kc + 32 * j > qw + 31 - p.window &&
                   qw + 32 <= x.L;
      uint64_t mask = ~0ull;
      if (!(whole[0] && whole[1])) {
        const int first = q >= p.window ? q - p.window + 1 : 0;
        if (blk < x.far) mask = bit_range(-kc, p.sinks - kc);
        else mask = bit_range(first - kc, q + 1 - kc) |
                    (x.far ? 0ull : bit_range(-kc, min(p.sinks, q + 1) - kc));
        if (q >= x.L) mask = 0ull;
      }
      if (!all_ok(mbar_wait(bar + 8 * (C::bSFull + sb), sr.ph))) return kErrSFull;
      tc_fence_after();
      float s[2][32];
#pragma unroll
      for (int j = 0; j < 2; ++j) tmem_ld32(trow + C::tS + sb * kChunk + 64 * hf + 32 * j, s[j]);
      tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < 2; ++j) reg_fence(s[j]);

      bool vis[2];  // some row of the warp sees some of these 32 keys
      float pm[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) pm[i] = -INFINITY;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t mw = static_cast<uint32_t>(mask >> (32 * j));
        vis[j] = whole[j] || __any_sync(0xffffffffu, mw != 0u);
        if (vis[j]) {
          if (!whole[j]) {
#pragma unroll
            for (int i = 0; i < 32; ++i) s[j][i] = (mw >> i) & 1u ? s[j][i] : -INFINITY;
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) pm[i & 7] = fmaxf(pm[i & 7], s[j][i]);
        }
      }
      // this half's running max (raw scores times the positive scale, base 2)
      const float cmax = fmaxf(fmaxf(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3])),
                               fmaxf(fmaxf(pm[4], pm[5]), fmaxf(pm[6], pm[7]))) * sl2;
      bool need = false;
      float alpha = 1.f;
      if (cmax > m_used + kTau) {
        if (m_used != -INFINITY) {
          need = true;
          alpha = ex2_approx(m_used - cmax);
        }
        m_used = cmax;
      }
      // P = 2^(s scale log2e - m) in bf16 for this half's 64 keys
      const float m_sub = m_used == -INFINITY ? 0.f : m_used;  // no visible key yet: P = 0
      const float2 nm = make_float2(-m_sub, -m_sub);
      const float2 sl = make_float2(sl2, sl2);
      uint32_t w[32];  // P of keys 2i, 2i + 1 of this half in w[i]
      float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (vis[j]) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {  // pairs of keys, packed fp32x2 arithmetic
            const float2 xv = __ffma2_rn(make_float2(s[j][2 * i], s[j][2 * i + 1]), sl, nm);
            const float2 pv = make_float2(ex2_approx(xv.x), ex2_approx(xv.y));
            ls[i & 1] = __fadd2_rn(ls[i & 1], pv);
            w[16 * j + i] = pack_bf16(pv.x, pv.y);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) w[16 * j + i] = 0u;
        }
      }
      if (__any_sync(0xffffffffu, need)) {
        // this half's previous P V product must have landed before its O is rescaled
        // (need implies c > 0, so the chunk before belongs to this tile)
        const bool wrap = sr.i == 0;
        if (!all_ok(mbar_wait(bar + 8 * (C::bSFree + (wrap ? C::NSB : sr.i) - 1),
                              wrap ? sr.ph ^ 1 : sr.ph)))
          return kErrPPrev;
        tc_fence_after();
        const uint32_t to = trow + C::tO(hf);
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
          float ov[32];
          tmem_ld32(to + 32 * j, ov);
          tmem_wait_ld();
          reg_fence(ov);
#pragma unroll
          for (int i = 0; i < 32; ++i) ov[i] *= alpha;
          tmem_st32(to + 32 * j, ov);
        }
        tmem_wait_st();
        l *= alpha;
      }
      l += (ls[0].x + ls[0].y) + (ls[1].x + ls[1].y);
      // P over this half's S columns (already read into registers)
      tmem_st32u(trow + C::tP(sb, hf), w);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(bar + 8 * (C::bPFull + sb));
      sr.next();
    }
    // hand this half's (m, l) of the row to the epilogue warps
    const int par = tc & 1;
    if (!all_ok(mbar_wait(bar + 8 * (C::bXFree + par), ((tc >> 1) & 1) ^ 1))) return kErrXFree;
    xs[((par * 2 + hf) * 2 + 0) * 128 + r] = m_used;
    xs[((par * 2 + hf) * 2 + 1) * 128 + r] = l;
    mbar_arrive(bar + 8 * (C::bXFull + par));
    ++tc;
  }
  if (sch.balanced) {  // second pass: the empty tiles, listed directly
    for (int e = blockIdx.x; e < p.items - sch.count; e += gridDim.x) {
      int b, h, tile;
      sched_empty(sch, a.batch, a.heads, p.ntiles, e, b, h, tile);
      zero_tile(decode_bht(p, b, h, tile, sched_length(sch, a, b)));
    }
  }
  return 0;
}

// Epilogue warps (one warpgroup, thread = tile row r): per tile, combine the
// halves O = (O_0 2^(m_0 - M) + O_1 2^(m_1 - M)) / l, l = l_0 2^(m_0 - M) +
// l_1 2^(m_1 - M), lse = M + log l; stage the bf16 tile in swizzled shared
// memory and write it with one TMA tensor store.  Off the softmax warps' path:
// they hand over (m, l) and move on to the next tile.
template <int D>
__device__ int epi_warps(const Params& p, uint32_t base, uint8_t* gbase, uint32_t tmem, int wq,
                         int lane, const CUtensorMap* to) {
  using C = Cfg<D>;
  const AttnArgs& a = p.a;
  const uint32_t bar = base + C::oBar;
  const int r = wq * 32 + lane;
  const uint32_t trow = tmem + (static_cast<uint32_t>(wq * 32) << 16);
  const float* xs = reinterpret_cast<const float*>(gbase + C::oXSum);
  uint8_t* stg = gbase + C::oStg;
  const bool leader = r == 0;
  auto all_ok = [](bool ok) { return __all_sync(0xffffffffu, ok); };
  int tc = 0;
  uint32_t zeros[4] = {0u, 0u, 0u, 0u};  // no longer 0: some output was not finite
  for (int rd = 0;; ++rd) {
    Item x;
    if (!next_item<D>(x, rd, bar, gbase, lane)) return kErrIFull;
    if (x.nch < 0) break;
    if (x.nch == 0) continue;
    const int64_t bh = static_cast<int64_t>(x.b) * a.heads + x.h;
    const int par = tc & 1;
    if (!all_ok(mbar_wait(bar + 8 * (C::bXFull + par), (tc >> 1) & 1))) return kErrXFull;
    const float m0 = xs[((par * 2 + 0) * 2 + 0) * 128 + r], l0 = xs[((par * 2 + 0) * 2 + 1) * 128 + r];
    const float m1 = xs[((par * 2 + 1) * 2 + 0) * 128 + r], l1 = xs[((par * 2 + 1) * 2 + 1) * 128 + r];
    mbar_arrive(bar + 8 * (C::bXFree + par));
    const float M = fmaxf(m0, m1);
    const float f0 = m0 == -INFINITY ? 0.f : ex2_approx(m0 - M);
    const float f1 = m1 == -INFINITY ? 0.f : ex2_approx(m1 - M);
    const float L = l0 * f0 + l1 * f1;
    const bool has = L != 0.f;  // padding rows: 0; a sum that is no number goes on
    const float inv = has ? 1.f / L : 0.f;
    const float g0 = f0 * inv, g1 = f1 * inv;
    if (!all_ok(mbar_wait(bar + 8 * C::bOFull, tc & 1))) return kErrOFull;
    tc_fence_after();
    const int q = x.tile * kRows + r;
    if (q < a.n && a.lse) a.lse[bh * a.n + q] = has ? (M + log2f(L)) * kLn2 : -INFINITY;
#pragma unroll
    for (int s = 0; s < D / 64; ++s) {  // 64 output columns at a time
      uint32_t w[32];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float o0[32], o1[32];
        tmem_ld32(trow + C::tO(0) + 64 * s + 32 * j, o0);
        tmem_ld32(trow + C::tO(1) + 64 * s + 32 * j, o1);
        tmem_wait_ld();
        reg_fence(o0);
        reg_fence(o1);
#pragma unroll
        for (int i = 0; i < 16; ++i)
          w[16 * j + i] = has ? pack_bf16(fmaf(o0[2 * i], g0, o1[2 * i] * g1),
                                          fmaf(o0[2 * i + 1], g0, o1[2 * i + 1] * g1))
                              : 0u;
      }
#pragma unroll
      for (int i = 0; i < 32; ++i) zeros[i & 3] = hidden::add_zeros(w[i], zeros[i & 3]);
      if (s == D / 64 - 1) {  // the next tile's products may begin
        tc_fence_before();
        mbar_arrive(bar + 8 * C::bOFree);
      }
      if (leader) bulk_wait_read0();  // the store before is done with the staging
      named_barrier(2, 128);
#pragma unroll
      for (int v = 0; v < 8; ++v)  // 16-byte pieces of the row, swizzled
        *reinterpret_cast<uint4*>(stg + r * 128 + ((v ^ (r & 7)) << 4)) =
            make_uint4(w[4 * v], w[4 * v + 1], w[4 * v + 2], w[4 * v + 3]);
      fence_proxy_async_smem();
      named_barrier(1, 128);  // they are staged
      if (leader) {
        tma_store_3d(to, base + C::oStg, s * 64, x.tile * kRows, static_cast<int>(bh));
        bulk_commit();
      }
    }
    ++tc;
  }
  if (leader) bulk_wait_all0();  // the last tile's store has landed before the CTA exits
  if (hidden::word_bad(zeros[0]) || hidden::word_bad(zeros[1]) || hidden::word_bad(zeros[2]) ||
      hidden::word_bad(zeros[3]))
    *reinterpret_cast<volatile int*>(gbase + C::oBad) = 1;
  return 0;
}

// Rows of this CTA's tiles that are not finite and have a hidden row of V that is not
// among their chunks' (sink_hidden.cuh), by the eight softmax warps, sixteen rows of a
// tile each.
template <int D>
__device__ __forceinline__ void sum_again(const Params& p, const Sched& sch, int warp, int lane) {
  using hidden::bf16;
  const float sl2 = p.a.scale * kLog2e;
  for (int rd = 0;; ++rd) {
    const int it = item_at(rd);
    if (it >= sch.count) break;
    const Item x = sched_item(p, sch, it);
    const int64_t bh = static_cast<int64_t>(x.b) * p.a.heads + x.h, bkv = bh / p.group;
    const bf16* k = static_cast<const bf16*>(p.a.k) + bkv * p.a.n * D;
    const bf16* v = static_cast<const bf16*>(p.a.v) + bkv * p.a.n * D;
    const int brought = min(x.key(2 * x.nch - 1) + kHalf, x.L);  // end of the chunks' keys
    for (int r = 0; r < kRows / 8 && x.nch > 0; ++r) {
      const int q = x.tile * kRows + warp * (kRows / 8) + r;
      if (q >= x.L) break;
      bf16* out = static_cast<bf16*>(const_cast<void*>(p.a.o)) + (bh * p.a.n + q) * D;
      const uint32_t bad = hidden::bad_channels<D>(out, lane);
      if (!__any_sync(0xffffffffu, bad != 0)) continue;
      const int first = q >= p.window ? q - p.window + 1 : 0, sinks = min(p.sinks, first);
      if (!hidden::any_bad<D>(v, x.far ? x.k0 : max(x.k0, sinks), first, lane) &&
          !hidden::any_bad<D>(v, q + 1, brought, lane))
        continue;
      const bf16* qrow = static_cast<const bf16*>(p.a.q) + (bh * p.a.n + q) * D;
      hidden::Row<D> acc;
      acc.zero();
      float m = -INFINITY, l = 0.f;
      bool more = true;
      auto keys = [&](int from, int end) {
        for (int base = from; base < end && more; base += 32) {
          const int j = base + lane;
          const float s = j < end ? sl2 * hidden::dot<D>(qrow, k + static_cast<int64_t>(j) * D)
                                  : -INFINITY;
          float mx = s;
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
          mx = fmaxf(mx, m);
          const float sub = mx == -INFINITY ? 0.f : mx;
          const float a = m == -INFINITY ? 0.f : ex2_approx(m - sub);
          const float w = ex2_approx(s - sub);
          m = mx;
          l = l * a + w;
          if (a != 1.f) acc.scale(a);
          acc.add_rows(v, base, 0, min(32, end - base), w, lane);
          more = !hidden::settled<D>(acc, bad);
        }
      };
      keys(0, sinks);
      keys(first, q + 1);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
      acc.scale(1.f / l);
      hidden::store_channels<D>(out, acc, bad, lane);
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_sink_fwd_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                       const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap tf,
                       const __grid_constant__ CUtensorMap to, const Params p) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t bar = base + C::oBar;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NQ; ++i) {
      mbar_init(bar + 8 * (C::bQFull + i), 1);
      mbar_init(bar + 8 * (C::bQFree + i), 1);
    }
    for (int i = 0; i < C::NKV; ++i) {
      mbar_init(bar + 8 * (C::bKFull + i), 1);
      mbar_init(bar + 8 * (C::bVFull + i), 1);
    }
    for (int i = 0; i < C::NSB; ++i) {
      mbar_init(bar + 8 * (C::bSFull + i), 1);
      mbar_init(bar + 8 * (C::bSFree + i), 1);
      mbar_init(bar + 8 * (C::bPFull + i), 256);
    }
    mbar_init(bar + 8 * C::bOFull, 1);
    mbar_init(bar + 8 * C::bOFree, 128);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar + 8 * (C::bXFull + i), 256);
      mbar_init(bar + 8 * (C::bXFree + i), 128);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(bar + 8 * (C::bIFull + i), 1);
      mbar_init(bar + 8 * (C::bIFree + i), kTakers);
    }
    mbar_init(bar + 8 * C::bVFix, 1);
    mbar_init(bar + 8 * C::bDone, 2);  // one commit per MMA-issuing thread
    fence_barrier_init();
    *reinterpret_cast<volatile int*>(gbase + C::oBad) = 0;
  }
  if (warp == 0) {
    if (lane == 0) {
      prefetch_tmap(&tq);
      prefetch_tmap(&tk);
      prefetch_tmap(&tv);
      prefetch_tmap(&tf);
      prefetch_tmap(&to);
    }
  }
  if (warp == 1) {
    tmem_alloc(base + C::oSlot, C::kTmemCols);
    tmem_relinquish();
  }
  pdl_wait();  // everything above overlaps the previous kernel's tail
  if (warp == 0) sched_build(reinterpret_cast<int*>(gbase + C::oSched), p.a, kRows, lane);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(gbase + C::oSlot);
  const Sched sch = sched_view(reinterpret_cast<const int*>(gbase + C::oSched), p.a, p.items);

  int err = 0;
  if (warp < 4) {
    regs_dec<C::kRegsCtl, kLaunchRegs>();
    if (warp == 0 && lane == 0) err = producer<D>(p, sch, base, gbase, &tq, &tk);
    if (warp == 1 && lane == 0) err = s_issuer<D>(base, gbase, tmem);
    if (warp == 2 && lane == 0) err = pv_issuer<D>(base, gbase, tmem);
    if (warp == 3) err = v_producer<D>(p, base, gbase, lane, &tv, &tf);
  } else if (warp < 12) {
    regs_inc<C::kRegsSoft, kLaunchRegs>();
    err = softmax_warps<D>(p, sch, base, gbase, tmem, warp & 3, (warp - 4) >> 2, lane);
    named_barrier(3, 384);  // the epilogue has stored every tile
    if (*reinterpret_cast<volatile int*>(gbase + C::oBad)) sum_again<D>(p, sch, warp - 4, lane);
  } else {
    regs_dec<C::kRegsEpi, kLaunchRegs>();
    err = epi_warps<D>(p, base, gbase, tmem, warp & 3, lane, &to);
    if (err) bulk_wait_all0();  // a store that is still reading the staging
    named_barrier(3, 384);
  }
  if (err) record_error(p.a.err, err);

  pdl_trigger();  // this CTA's work is issued: the next kernel may start launching
  __syncthreads();
  if (warp == 2 && lane == 0) mma_commit(bar + 8 * C::bDone);
  if (warp == 1) {
    if (lane == 0) {  // every tensor-core operation of this CTA has completed
      mma_commit(bar + 8 * C::bDone);
      if (!mbar_wait(bar + 8 * C::bDone, 0)) record_error(p.a.err, kErrDone);
    }
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;

template <int D>
cudaError_t launch(const SinkArgs& g, cudaStream_t stream) {
  using C = Cfg<D>;
  const int64_t heads_total = static_cast<int64_t>(g.batch) * g.heads;
  const int64_t kv_total = static_cast<int64_t>(g.batch) * g.kv_heads;
  CUtensorMap tq, tk, tv, tf, to;
  if (!make_tmap_bf16_rows(&tq, g.q, D, g.n, heads_total, kRows) ||
      !make_tmap_bf16_rows(&tk, g.k, D, g.n, kv_total, kHalf) ||
      !make_tmap_bf16_rows(&tv, g.v, D, g.n, kv_total, kHalf) ||
      !make_tmap_bf16_rows(&to, g.o, D, g.n, heads_total, kRows))
    return cudaErrorInvalidValue;
  tf = tv;  // without sinks, or with every key in every window, no tile has blocks of sinks
  if (g.sinks > 0 && g.n > g.window &&
      !make_tmap_first_rows(&tf, g.v, D, g.n, kv_total, g.sinks, kHalf))
    return cudaErrorInvalidValue;
  Params p;
  p.a = AttnArgs{};
  p.a.q = g.q;
  p.a.k = g.k;
  p.a.v = g.v;
  p.a.o = g.o;
  p.a.lse = g.lse;
  p.a.lengths = g.lengths;
  p.a.err = g.err;
  p.a.batch = g.batch;
  p.a.heads = g.heads;
  p.a.n = g.n;
  p.a.d = D;
  p.a.scale = g.scale;
  p.group = g.heads / g.kv_heads;
  p.window = g.window;
  p.sinks = g.sinks;
  p.ntiles = (g.n + kRows - 1) / kRows;
  const int64_t items = heads_total * p.ntiles;
  if (items > (1ll << 30)) return cudaErrorInvalidValue;
  p.items = static_cast<int>(items);
  cudaError_t e = cudaFuncSetAttribute(attn_sink_fwd_kernel<D>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  const int grid = static_cast<int>(items < num_sms() ? items : num_sms());
  return launch_pdl(attn_sink_fwd_kernel<D>, dim3(grid), dim3(kThreads), C::kSmem, stream, tq, tk,
                    tv, tf, to, p);
}

}  // namespace

bool make_tmap_first_rows(CUtensorMap* m, const void* base, int d, int64_t n, int64_t heads_total,
                          int first, int box_rows) {
  std::call_once(g_encode_once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  if (!g_encode) return false;
  const int64_t rows = first < 1 ? 1 : (first < n ? first : n);
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(heads_total)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 2, static_cast<cuuint64_t>(n) * d * 2};
  const cuuint32_t box[3] = {64u, static_cast<cuuint32_t>(box_rows), 1u}, steps[3] = {1u, 1u, 1u};
  return g_encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides,
                  box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_attn_sink_fwd(const SinkArgs& a, cudaStream_t stream) {
  return a.d == 64 ? launch<64>(a, stream) : launch<128>(a, stream);
}

}  // namespace nb
