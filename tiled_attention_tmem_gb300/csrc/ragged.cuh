// Work items of packed sequences: tokens cu[b] .. cu[b + 1] - 1 of one array are
// sequence b, lengths known on the device only.
//
// Grouped heads: the G = H / Hkv query heads of a kv head are G rows of a token, so a
// tile of M rows holds M / G tokens (rounded down) with all of their heads, row r being
// token r / G and head r % G.  K and V tiles are then read once for the G heads, and the
// kernels are those of equal heads over G rows a token.  The rows past (M / G) * G of a
// tile belong to nobody.
//
// Ends: a tile that reaches past its sequence's end must read zeros there, and not what the next
// sequence or the rows behind the last one hold: a NaN there times a probability of 0 would be NaN.  Such tiles are
// loaded by a map of the sequence's own (made by ragged_plan_kernel), whose token dimension ends
// there; other tiles go by the launch's maps, since a new map costs a fence and a fetch.  The forward without a plan
// has no such maps: its softmax warps clear those rows of V in shared memory.
#pragma once
#include "common.cuh"

namespace fa {

struct RaggedSched {
  const int* base;   // [B + 1] first work item of each sequence, longest sequence first; [B]: their number
  const int4* seqs;  // [B] in the same order: first token, tokens, sequence, heads per launch-order group
  int* counter;      // items claimed beyond the first of each CTA (zero at launch)
  int B;
  // Without a plan the scheduling warps put the sequences, kRaggedDirect at most, in order themselves, and take their
  // items in turn, without a counter; only B and these are set.
  const int* cu;
  int T;
};
constexpr int kRaggedDirect = 32;  // sequences that need no plan: a lane each

struct RaggedItem {
  int start, len, seq;  // first token and tokens of the sequence, its index
  int tile, head;       // rank of the tile (the heaviest first), kv head
};

constexpr int kRaggedRing = 4;        // items between the scheduling warp and its slowest reader
constexpr int kRaggedRingBytes = 32;  // a slot of the ring

// The scheduling warp waits for as long as an item takes, and longer for a longer sequence: a step (a query or
// key tile of one token or more; 2200 to 2500 cycles measured) for each of its tokens at most.  Under the limit of all other waits,
// 4 x 10^9 cycles, a correct dK/dV item of 10^8 rows would be reported as one that hangs.
__host__ __device__ constexpr long long ragged_wait_limit(int longest) { return kWaitLimitCycles + 8192LL * longest; }

// The scheduling warp of a persistent CTA: claims work items (the first is the CTA's own
// index, the rest come from the counter, so that idle SMs take the next ones, longest sequences first),
// looks up their sequences and passes them to the other roles through a ring in shared memory.  Each item
// after the first is claimed when the producer asks for it (`ask`, one arrival an item), while it
// loads the one before: earlier, a CTA that is still busy would hold items that others could start.
// Claimed indices only grow, so the search goes on from the last sequence, 32 at a time.
// DIRECT: without a plan; CTA c takes items c, 2G - 1 - c, 2G + c, ... of G CTAs.
template <bool DIRECT>
__device__ __forceinline__ void ragged_schedule(const RaggedSched& s, int tile_tokens, int parts, int heads,
                                                volatile int* ring, uint32_t full0, uint32_t empty0, uint32_t ask,
                                                const CtaAbort& ab, int where) {
  const int lane = lane_id();
  int total, rank = 0, w = blockIdx.x, longest = 0;  // longest: tokens of the longest sequence it has passed on
  // DIRECT: lane r holds the sequence of rank r and its first item.
  int my_start = 0, my_len = 0, my_seq = lane, my_base = 0, my_end = 0;
  if constexpr (DIRECT) {
    if (lane < s.B) {
      my_start = s.cu[lane];
      const int end = s.cu[lane + 1];
      if (my_start >= 0 && my_start <= end && end <= s.T) my_len = end - my_start;
    }
    int my_rank = 0, from = lane;
#pragma unroll
    for (int k = 0; k < 32; ++k) {
      const int other = __shfl_sync(0xffffffffu, my_len, k);
      my_rank += other > my_len || (other == my_len && k < lane);
    }
#pragma unroll
    for (int k = 0; k < 32; ++k)
      if (__shfl_sync(0xffffffffu, my_rank, k) == lane) from = k;
    my_start = __shfl_sync(0xffffffffu, my_start, from);
    my_len = __shfl_sync(0xffffffffu, my_len, from);
    my_seq = from;
    const int items = ((my_len + tile_tokens - 1) / tile_tokens) * parts * heads;
    my_end = items;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, my_end, d);
      if (lane >= d) my_end += y;
    }
    my_base = my_end - items;
    total = __shfl_sync(0xffffffffu, my_end, 31);
    // (No work where they hold more than the tokens, as in plan_schedule; few items, so the sum stays below 2^31.)
    if (__reduce_add_sync(0xffffffffu, (unsigned)my_len) > (unsigned)s.T) total = 0;
  } else {
    total = s.base[s.B];
  }
  for (int t = 0;; ++t) {
    const int k = t % kRaggedRing;
    const long long limit = DIRECT ? kWaitLimitCycles : ragged_wait_limit(longest);  // (few items are short ones)
    if (!wait_warp(empty0 + 8 * k, ((t / kRaggedRing) & 1) ^ 1, ab, where, limit)) return;
    if (DIRECT && t > 0) {
      w = t * (int)gridDim.x + ((t & 1) ? (int)(gridDim.x - 1 - blockIdx.x) : (int)blockIdx.x);
    } else if (t > 0) {
      if (!wait_warp(ask, (t - 1) & 1, ab, where, limit)) return;
      if (lane == 0) w = (int)gridDim.x + atomicAdd(s.counter, 1);
      w = __shfl_sync(0xffffffffu, w, 0);
    }
    int start = -1, len = 0, seq = 0, tile = 0, head = 0;
    if (DIRECT && w < total) {
      rank = __ffs(__ballot_sync(0xffffffffu, my_end > w)) - 1;
      start = __shfl_sync(0xffffffffu, my_start, rank);
      len = __shfl_sync(0xffffffffu, my_len, rank);
      seq = __shfl_sync(0xffffffffu, my_seq, rank);
      grouped_order(w - __shfl_sync(0xffffffffu, my_base, rank), ((len + tile_tokens - 1) / tile_tokens) * parts, heads,
                    heads, tile, head);
    } else if (w < total) {
      for (; rank < s.B; rank += 32) {
        const int i = rank + lane;
        const unsigned past = __ballot_sync(0xffffffffu, i < s.B && s.base[min(i + 1, s.B)] > w);
        if (past) {
          rank += __ffs(past) - 1;
          break;
        }
      }
      const int4 q = s.seqs[rank];
      start = q.x, len = q.y, seq = q.z;
      grouped_order(w - s.base[rank], ((len + tile_tokens - 1) / tile_tokens) * parts, heads, q.w, tile, head);
    }
    if (lane == 0) {
      volatile int* slot = ring + k * (kRaggedRingBytes / 4);
      slot[0] = start, slot[1] = len, slot[2] = seq, slot[3] = tile, slot[4] = head;
      mbar_arrive(full0 + 8 * k);
    }
    __syncwarp();
    if (start < 0) return;
    longest = max(longest, len);
  }
}

// Who reads an item: a whole warp, or a single thread.
struct ByWarp {
  static constexpr bool value = false;
};
struct ByThread {
  static constexpr bool value = true;
};

// The t-th item of this CTA, for a whole warp or (ONE) a single thread; false after the
// last, or if the wait gave up.
template <bool ONE>
__device__ __forceinline__ bool ragged_item(int t, RaggedItem& I, const volatile int* ring, uint32_t full0,
                                            uint32_t empty0, const CtaAbort& ab, int where) {
  const int k = t % kRaggedRing;
  const uint32_t parity = (t / kRaggedRing) & 1;
  if constexpr (ONE) {
    if (!wait_one(full0 + 8 * k, parity, ab, where)) return false;
  } else {
    if (!wait_warp(full0 + 8 * k, parity, ab, where)) return false;
  }
  const volatile int* slot = ring + k * (kRaggedRingBytes / 4);
  I.start = slot[0], I.len = slot[1], I.seq = slot[2], I.tile = slot[3], I.head = slot[4];
  if constexpr (ONE) {
    mbar_arrive(empty0 + 8 * k);
  } else {
    __syncwarp();
    if (lane_id() == 0) mbar_arrive(empty0 + 8 * k);
  }
  return I.start >= 0;
}

}  // namespace fa
