// decode_units.cuh -- how the per-sequence decodes over packed pools (decode_int4.cu,
// decode_fp8_block.cu) share out a batch: units, cut into equal pieces or into ranges (UnitPlan,
// kernels.h). The figures here are of int4 pools.
//
// Equal pieces: a unit is cut into pieces of the same length, one CTA each: as many as let all
// units fill the resident CTAs once, of at least 32 blocks by the sequence's own length
// (a block table is as wide as a captured step may need; CTAs that its sequence leaves without
// a piece end at once). Units of one piece are written out, without parts and a join.
//
// Ranges: where a piece would be longer than kMaxPiece, the length of the longest sequence
// says too little about the others. The units' blocks are laid end to end and cut into equal
// ranges, one per resident CTA: batches of any lengths give every CTA the same work. A CTA
// goes through its range unit by unit; a unit that lies in one range is written out. Where the
// table's width does not rule ranges out every CTA looks for the longest sequence, in batches of
// up to kMaxLook; larger ones are cut into ranges (tables of 4096 blocks, 32 heads on 8, us with the
// look and with ranges at once: 512 sequences of 64 tokens 56 61, of 1024 134 150; 1024 of 64
// 123 110, of 256 158 154, of 1024 272 290; 2048 of 64 303 213, of 1024 582 563).
//
// Measured from HBM (pieces, ranges; us), 32 heads on 8: 64 sequences of 256 blocks 63 68, of 512
// 118 113, of 600 139 130, of 1000 225 210, of 2000 439 397; of up to 512 106 96, of up to 1024
// 189 138; 4 of 8192 (pieces of 432) 105 109. 32 heads on one: 16 of 2000 (pieces of 106) 63 69,
// 48 of up to 3750 (pieces of 1250) 215 145.
//
// The other parts go to the workspace (at most two per CTA: slot 2 c + 1 for a unit that
// begins in CTA c's places, 2 c for one that began before) and are merged by
// combine_units_kernel (decode_units.cu).
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace lazy {

constexpr int kMinPieceLog2 = 5;  // 32 blocks of a piece at least: one of 16384 tokens 17 us, with 16 or 64 19
constexpr int kMaxPiece = 512;
constexpr int kMinChunk = 16;   // blocks of a range at least
constexpr int kMaxLook = 1024;  // sequences that every CTA looks through

// Blocks and slots of sequence s.
__device__ __forceinline__ int blocks_of(const UnitDecodeArgs& a, int s, int& seq_len) {
  seq_len = a.seq_lens[s];
  if (seq_len < 0 || seq_len > kBlock * a.max_blocks) {
    raise_status(a.status, LAZY_DEV_BAD_LEN);
    seq_len = seq_len < 0 ? 0 : kBlock * a.max_blocks;
  }
  return (seq_len + kBlock - 1) / kBlock;
}

// Blocks of a piece of a sequence of nb blocks.
__host__ __device__ __forceinline__ int piece_of(const UnitPlan& p, int nb) {
  if (p.splits == 1) return nb;
  const int n = max(1, min(p.splits, nb >> p.least_log2));
  return (int)((unsigned)(nb + n - 1) / (unsigned)n);
}

// Blocks of a range, of `total` in all.
__device__ __forceinline__ int64_t chunk_of(const UnitDecodeArgs& a, int64_t total) {
  const int64_t c = (total + a.plan.range_ctas - 1) / a.plan.range_ctas;
  return c > kMinChunk ? c : kMinChunk;
}

// Whether the batch is cut into ranges: some sequence's pieces would be too long (every warp
// looks by itself).
__device__ __forceinline__ bool takes_ranges(const UnitDecodeArgs& a, int lane) {
  if (a.plan.range_ctas == 0) return false;
  if (a.B > kMaxLook) return true;
  int longest = 0;
  for (int b = lane; b < a.B; b += 32) {
    int len;
    longest = max(longest, blocks_of(a, b, len));
  }
  return __reduce_max_sync(0xffffffffu, longest) > kMaxPiece * a.plan.splits;
}

// A CTA's parts, one after the other: blocks lo .. hi - 1 of unit u of sequence s, which has seq_len
// slots in nb blocks. Every warp walks by itself, and all take the same way.
struct UnitWalk {
  int s, seq_len, nb, u, lo, hi;
  int64_t at, left;  // ranges: place within sequence s (its units end to end), places left of the range

  // false: the CTA has nothing to do. The first CTA leaves `prefix` for the join.
  __device__ __forceinline__ bool begin(const UnitDecodeArgs& a, int warp, int lane) {
    const int U = a.plan.units;
    s = seq_len = nb = u = lo = hi = 0;
    at = left = 0;
    const bool ranges = takes_ranges(a, lane);
    if (a.plan.range_ctas > 0 && blockIdx.x == 0 && threadIdx.x == 0) a.prefix[a.B + 1] = ranges;
    if (!ranges) {  // first pieces first: CTAs without one are the last, not between those of one SM
      const unsigned units = (unsigned)a.B * U, piece = blockIdx.x / units, unit = blockIdx.x - piece * units;
      s = unit / U;
      u = unit - s * U;
      nb = blocks_of(a, s, seq_len);
      const int len = piece_of(a.plan, nb);
      lo = piece * len;
      hi = min(nb, lo + len);
      return piece == 0 || lo < nb;
    }
    // every warp for itself: the total, then the sequence of the range's first place
    int64_t total = 0;
    int own = 0, inc = 0;  // of the last 32 sequences: the lane's blocks, and up to them
    auto scan = [&](int b) {
      int len;
      inc = own = b + lane < a.B ? blocks_of(a, b + lane, len) : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += x;
      }
    };
    for (int b = 0; b < a.B; b += 32) {
      scan(b);
      if (blockIdx.x == 0 && warp == 0 && b + lane < a.B) a.prefix[b + lane] = total + inc - own;
      total += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) a.prefix[a.B] = total;
    total *= U;
    const int64_t chunk = chunk_of(a, total), first = blockIdx.x * chunk;
    left = min(chunk, total - first);
    if (left <= 0) return false;
    int64_t before = 0;
    for (s = 0; s < a.B; s += 32) {
      if (a.B > 32) scan(s);
      const uint32_t past = __ballot_sync(0xffffffffu, (before + inc) * U > first);  // sequences that end behind it
      if (past) {
        const int l = __ffs(past) - 1;
        s += l;
        at = first - (before + __shfl_sync(0xffffffffu, inc, l) - __shfl_sync(0xffffffffu, own, l)) * U;
        break;
      }
      before += __shfl_sync(0xffffffffu, inc, 31);
    }
    return true;
  }

  // The next part; false: a range behind the last sequence.
  __device__ __forceinline__ bool next(const UnitDecodeArgs& a) {
    if (left <= 0) return true;  // a piece
    const int U = a.plan.units;
    for (; s < a.B; ++s) {
      nb = blocks_of(a, s, seq_len);
      if (nb > 0 && at < (int64_t)U * nb) break;
      at -= (int64_t)U * nb;
    }
    if (s >= a.B) return false;
    u = (int)(at / nb), lo = (int)(at - (int64_t)u * nb);
    hi = (int)min((int64_t)nb, lo + left);
    at += hi - lo;
    left -= hi - lo;
    return true;
  }

  __device__ __forceinline__ bool last() const { return left <= 0; }
};

}  // namespace lazy
