// Layout of the 4-bit key/value cache, shared by the kernels that write it,
// read it back and attend over it.
//
// A page holds NB_KV4_PAGE = 32 tokens of one key/value head, contiguous, so
// that one bulk copy brings everything attention needs of it:
//   K codes   32 rows of d/2 bytes      V codes   32 rows of d/2 bytes
//   K params  32 rows of d/32 words     V params  32 rows of d/32 words
// A param word belongs to one token and group of 32 channels: the step s (bf16)
// in its low half and the midpoint m (bf16) in its high half.  A code c stands
// for m + s (c - 7.5).
//
// Both code layouts follow the operand fragments of the warp-level matrix
// product that attention uses, so a lane reads its operands with one wide load
// and no shuffles (lane = 4 r + t, r = 0..7, t = 0..3):
//   K row  word [t][g] = channels 32 g + 8 t + 0..7, channel i in nibble i (the
//          product runs over channels: lane t takes eight of each group).
//   V row  chunk r (d/64 words): word w nibble i = channel 64 w + 8 i + r (the
//          output columns of lane row r).  At d = 128 the chunk index is xored
//          with 4 in every second pair of tokens, which spreads the eight-byte
//          reads of a half warp over all banks.
#pragma once

#include <stdint.h>

#include "../../include/nb.h"

namespace nb {
namespace kv4 {

constexpr int kPage = NB_KV4_PAGE;  // tokens per page
constexpr int kGroup = 32;          // channels that share a step and a midpoint

template <int D>
struct Page {
  static constexpr int kGroups = D / kGroup;
  static constexpr int kRow = D / 2;           // bytes of a row of codes
  static constexpr int kParRow = kGroups * 4;  // bytes of a row of params
  static constexpr int oK = 0, oV = kPage * kRow;
  static constexpr int oKPar = 2 * kPage * kRow, oVPar = oKPar + kPage * kParRow;
  static constexpr int kBytes = oVPar + kPage * kParRow;

  // byte offset of the V chunk of lane row r in the row of `token`
  __host__ __device__ static constexpr int v_chunk(int token, int r) {
    return (D == 128 ? r ^ (((token >> 1) & 1) << 2) : r) * (D / 16);
  }
};

// Extremes that are no number when an operand is none.
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

// Where the tokens of a sequence lie: pages of the pool through a block table.
struct Pool {
  uint8_t* base;         // [num_pages][kv_heads][page bytes]
  const int32_t* table;  // [batch][max_pages]
  int max_pages, num_pages, kv_heads;
};

// A warp brings the `count` pages of its share through N stages, page i into stage i mod N:
// N pages at the start, and page i + N once page i has been used.  When the wait for page i
// gives up, pages i .. i + N - 1 are on their way: calls wait(stage, parity) for each, with
// the parity of the pass that the stage's barrier is in (i / N passes are complete).
template <int N, class Wait>
__host__ __device__ __forceinline__ void drain_pages(int i, int count, Wait&& wait) {
  const int end = count - i < N ? count : i + N;
  for (; i < end; ++i) wait(i % N, static_cast<uint32_t>(i / N) & 1u);
}

// codes of slots that the table does not map into the pool, and the site of a wait
enum : int { kErrWriteSlot = NB_KERR_KV4_WRITE, kErrReadSlot = NB_KERR_KV4_READ,
             kErrDecodePage = NB_KERR_KV4_DECODE, kErrDecodeWait = 0xa1 };

}  // namespace kv4
}  // namespace nb
