// Host-side helpers of attention over packed sequences (not part of the ABI).
#pragma once
#include <cstdint>

#include "fa_packed.h"
#include "host.h"
#include "ragged.cuh"

namespace fa {

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
// The plan's parameters (packed_plan.cuh), the blocks that its maps keep busy, and its launch.
struct RaggedPlanParams;
RaggedPlanParams packed_plan_params(const PackedPlan& plan, const int* cu, const PackedShape& s, const PackedCut* cuts,
                                    int ncuts, const CUtensorMap* maps, int nmaps, int query_maps);
int packed_map_blocks(int B, int nmaps, int threads);
fa_status run_packed_plan(const RaggedPlanParams& p, cudaStream_t st);

// Tensor maps, of which the plan makes one for each sequence that ends with it (the first query_maps of
// them are of queries): query rows
// {d, G, T, Hkv} with a box of `tokens` tokens of all G heads, key rows {d, T, Hkv}.
fa_status packed_query_map(CUtensorMap* map, const fa_rows& r, const PackedShape& s, int tokens);
fa_status packed_key_map(CUtensorMap* map, const fa_rows& r, const PackedShape& s, int box_rows);

// Checks shared by the entry points.
fa_status packed_shape_checks(const PackedShape& s, float scale, int causal);
fa_status packed_rows_checks(const fa_rows& r, int T, int heads);

// Arguments checked, and not without work.  form: FA_BWD_5GEMM or FA_BWD_7GEMM.
fa_status run_packed_fwd(const fa_packed_fwd_args& a, const PackedShape& s);
size_t packed_fwd_bytes(const PackedShape& s);
fa_status run_packed_bwd(const fa_packed_bwd_args& a, const PackedShape& s, int form);
size_t packed_bwd_bytes(const PackedShape& s, int form);

}  // namespace fa
