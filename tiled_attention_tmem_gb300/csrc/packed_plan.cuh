// The plan of a call over packed sequences, made on the GPU from their lengths: the order
// of work, and tensor maps that end where the sequences do.
#pragma once
#include "packed_host.h"

namespace fa {

constexpr int kPlanSorted = 2048;  // sequences that are put in order of their lengths
constexpr int kPlanCounted = 256;  // up to these by counting the longer ones: a pass instead of a sort's 36
constexpr int kPlanItems = 1 << 30;

struct RaggedPlanParams {
  CUtensorMap map[kPackedMaxMaps];
  const int* cu;
  CUtensorMap* maps;
  RaggedSched sched[2];
  PackedCut cut[2];
  int ncuts, nmaps;
  int query_maps;  // these first ones have the heads of a group in front of their tokens
  int B, T, heads, sms;
};

// First token and tokens of sequence b; none where its tokens do not lie in [0, T).
__device__ __forceinline__ int plan_seq(const RaggedPlanParams& p, int b, int& start) {
  start = p.cu[b];
  const int end = p.cu[b + 1];
  return start >= 0 && start <= end && end <= p.T ? end - start : 0;
}

// A warp a tensor map, copied from its template and cut at the sequence's end.  `block` of `blocks`.
template <int THREADS>
__device__ __forceinline__ void plan_maps(const RaggedPlanParams& p, int block, int blocks) {
  constexpr int WARPS = THREADS / 32;
  __shared__ alignas(128) uint32_t slot[WARPS][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long tasks = (long long)p.B * p.nmaps, step = (long long)blocks * WARPS;
  for (long long i = (long long)block * WARPS + warp; i < tasks; i += step) {
    const int b = (int)(i / p.nmaps), m = (int)(i - (long long)b * p.nmaps);
    int start;
    const int len = plan_seq(p, b, start);
    const uint32_t end = len > 0 ? (uint32_t)(start + len) : 1u;
    slot[warp][lane] = reinterpret_cast<const uint32_t*>(&p.map[m])[lane];
    __syncwarp();
    const uint32_t at = smem_u32(slot[warp]);
    if (lane == 0) {
      if (m < p.query_maps)
        asm volatile("tensormap.replace.tile.global_dim.shared::cta.b1024.b32 [%0], 2, %1;" ::"r"(at), "r"(end)
                     : "memory");
      else
        asm volatile("tensormap.replace.tile.global_dim.shared::cta.b1024.b32 [%0], 1, %1;" ::"r"(at), "r"(end)
                     : "memory");
    }
    __syncwarp();
    asm volatile(
        "tensormap.cp_fenceproxy.global.shared::cta.tensormap::generic.release.gpu.sync.aligned [%0], [%1], 128;" ::"l"(
            reinterpret_cast<uint64_t>(p.maps + i)),
        "r"(at)
        : "memory");
    __syncwarp();
  }
}

// One block, for one sequence or more: sequences by length, longest first (so that what is claimed last is short; by index where there
// are over 2048: the longest is a small part of the work then, or the launch is long anyway), and the
// running sum of their work items.  There are none where the sequences hold more than T tokens together: they overlap (cu
// decreases), and could be B times the work of T tokens.  Latency bounds it (a count or a sort, a scan): a
// forward of 16 sequences takes 2.5 us more with a plan than without (6 with a sort in a block of 1024 threads, before
// the forward's blocks started beside it).
template <int THREADS>
__device__ __forceinline__ void plan_schedule(const RaggedPlanParams& p) {
  __shared__ unsigned long long keys[kPlanSorted];
  __shared__ long long sums[THREADS / 32], tokens[THREADS / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool sorted = p.B <= kPlanSorted, counted = p.B <= kPlanCounted;
  auto key_of = [&](int i) {
    int start;
    return (unsigned long long)(0x7fffffff - plan_seq(p, i, start)) << 32 | (unsigned)i;
  };
  if (counted) {
    for (int i = tid; i < p.B; i += THREADS) keys[kPlanCounted + i] = key_of(i);
    __syncthreads();
    for (int i = tid; i < p.B; i += THREADS) {
      const unsigned long long mine = keys[kPlanCounted + i];
      int rank = 0;
#pragma unroll 4
      for (int j = 0; j < p.B; ++j) rank += keys[kPlanCounted + j] < mine;
      keys[rank] = mine;
    }
    __syncthreads();
  } else if (sorted) {
    int n = 1;
    while (n < p.B) n *= 2;
    for (int i = tid; i < n; i += THREADS) keys[i] = i < p.B ? key_of(i) : ~0ull;
    __syncthreads();
    for (int size = 2; size <= n; size *= 2)
      for (int gap = size / 2; gap > 0; gap /= 2) {
        for (int i = tid; i < n / 2; i += THREADS) {
          const int a = 2 * i - (i & (gap - 1)), b = a + gap;
          const unsigned long long x = keys[a], y = keys[b];
          if ((x > y) == ((a & size) == 0)) keys[a] = y, keys[b] = x;
        }
        __syncthreads();
      }
  }
  const int run = (p.B + THREADS - 1) / THREADS;
  const int r0 = min(tid * run, p.B), r1 = min(r0 + run, p.B);
  for (int c = 0; c < p.ncuts; ++c) {
    const PackedCut cut = p.cut[c];
    const RaggedSched s = p.sched[c];
    auto tiles_of = [&](int len) -> long long { return (long long)((len + cut.tokens - 1) / cut.tokens) * cut.parts; };
    auto seq_of = [&](int r) { return sorted ? (int)(uint32_t)keys[r] : r; };
    long long sum = 0;
    int start;
    long long held = 0;
    for (int r = r0; r < r1; ++r) {
      const int len = plan_seq(p, seq_of(r), start);
      held += len;
      sum += tiles_of(len) * p.heads;
    }
    long long before = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, before, d);
      if (lane >= d) before += y;
      held += __shfl_xor_sync(0xffffffffu, held, d);
    }
    if (lane == 31) sums[warp] = before, tokens[warp] = held;
    __syncthreads();
    before -= sum;
    for (int w = 0; w < warp; ++w) before += sums[w];
    held = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) held += tokens[w];
    __syncthreads();
    const bool valid = held <= p.T;
    if (!valid) before = 0;
    for (int r = r0; r < r1; ++r) {
      const int b = seq_of(r), len = plan_seq(p, b, start);
      const long long tiles = tiles_of(len);
      // Heads whose re-read operands stay in L2 together (96 MB), with three rounds of items a group
      // at least; groups of the same size.
      long long g = (long long)(96.0 * 1024 * 1024 / (cut.token_bytes * max(len, 1)));
      g = max(g, (3 * p.sms + tiles - 1) / max(tiles, 1LL));
      g = min(max(g, 1LL), (long long)p.heads);
      const int groups = p.heads / (int)g;
      const_cast<int*>(s.base)[r] = (int)min(before, (long long)kPlanItems);
      const_cast<int4*>(s.seqs)[r] = make_int4(start, len, b, (p.heads + groups - 1) / groups);
      if (valid) before += tiles * p.heads;
      if (r == p.B - 1) const_cast<int*>(s.base)[p.B] = (int)min(before, (long long)kPlanItems);
    }
    if (tid == 0) *s.counter = 0;
  }
}


}  // namespace fa
