// Host-side helpers of attention over packed sequences (not part of the ABI).
#pragma once
#include <cstdint>

#include "fa_packed.h"
#include "host.h"
#include "ragged.cuh"

namespace fa {

// One [T, heads, d] bf16 array with dense channels: strides in elements.
struct PackedRows {
  void* data;
  long long token, head;
};

struct PackedShape {
  int B, T, H, Hkv, d;
  int G() const { return H / Hkv; }
};

constexpr int kPackedMaxGroup = 32;  // query heads of a kv head: 32 rows are the smallest query tile (d = 384)

// How work items are cut for one kernel: `tokens` tokens a tile, `parts` items a tile and kv
// head; `token_bytes` per token and kv head are read again by the other tiles of a sequence.
struct PackedCut {
  int tokens, parts;
  double token_bytes;
};

// What ragged_plan_kernel makes of the lengths, in the caller's workspace: for each cut the order of
// the sequences, their first work items and a counter; for each sequence its tensor maps.
constexpr int kPackedMaxMaps = 6;
struct PackedPlan {
  RaggedSched sched[2];
  CUtensorMap* maps;  // [B][nmaps]
};
size_t packed_plan_bytes(int B, int cuts, int nmaps);
// Lays the plan out at `at` (256-byte aligned) without launching anything.
PackedPlan packed_plan_at(void* at, int B, int cuts);
fa_status run_packed_plan(const PackedPlan& plan, const int* cu, const PackedShape& s, const PackedCut* cuts, int ncuts,
                          const CUtensorMap* maps, int nmaps, int query_maps, cudaStream_t st);

// Tensor maps, of which the plan makes one for each sequence that ends with it (the first query_maps of
// them are of queries): query rows
// {d, G, T, Hkv} with a box of `tokens` tokens of all G heads, key rows {d, T, Hkv}.
fa_status packed_query_map(CUtensorMap* map, const PackedRows& r, const PackedShape& s, int tokens);
fa_status packed_key_map(CUtensorMap* map, const PackedRows& r, const PackedShape& s, int box_rows);

// Checks shared by the entry points.
fa_status packed_shape_checks(const PackedShape& s, float scale, int causal);
fa_status packed_rows_checks(const PackedRows& r, int T, int heads);

fa_status run_packed_fwd(const PackedRows& q, const PackedRows& k, const PackedRows& v, const PackedRows& o, float* lse,
                         const int* cu, const PackedShape& s, float scale, int causal, void* workspace, cudaStream_t st);
size_t packed_fwd_bytes(const PackedShape& s);
fa_status run_packed_bwd(const PackedRows& q, const PackedRows& k, const PackedRows& v, const PackedRows& o,
                         const PackedRows& dO, const float* lse, const PackedRows& dq, const PackedRows& dk,
                         const PackedRows& dv, const int* cu, const PackedShape& s, float scale, int causal,
                         int variant, void* workspace, cudaStream_t st);
size_t packed_bwd_bytes(const PackedShape& s, int variant);

}  // namespace fa
