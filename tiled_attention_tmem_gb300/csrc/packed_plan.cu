// The plan of a call over packed sequences, its checks, and the entry points.
#include <algorithm>
#include <cmath>

#include "kv4_host.h"
#include "packed_host.h"
#include "packed_plan.cuh"

namespace fa {
namespace {

template <int THREADS>
__global__ void __launch_bounds__(THREADS) ragged_plan_kernel(const __grid_constant__ RaggedPlanParams p) {
  grid_dep_wait();
  grid_dep_launch();  // (the forward's blocks set up beside the plan)
  if (blockIdx.x == 0) plan_schedule<THREADS>(p);
  else plan_maps<THREADS>(p, blockIdx.x - 1, gridDim.x - 1);
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

size_t packed_plan_bytes(int B, int cuts, int nmaps) {
  return cuts * (align256(4 * ((size_t)B + 1)) + align256(16 * (size_t)B) + 256) + align256(128 * (size_t)B * nmaps);
}

PackedPlan packed_plan_at(void* at, int B, int cuts) {
  uint8_t* b = static_cast<uint8_t*>(at);
  PackedPlan plan = {};
  for (int c = 0; c < cuts; ++c) {
    RaggedSched& s = plan.sched[c];
    s.B = B;
    s.base = reinterpret_cast<int*>(b);
    b += align256(4 * ((size_t)B + 1));
    s.seqs = reinterpret_cast<int4*>(b);
    b += align256(16 * (size_t)B);
    s.counter = reinterpret_cast<int*>(b);
    b += 256;
  }
  plan.maps = reinterpret_cast<CUtensorMap*>(b);
  return plan;
}

RaggedPlanParams packed_plan_params(const PackedPlan& plan, const int* cu, const PackedShape& s, const PackedCut* cuts,
                                    int ncuts, const CUtensorMap* maps, int nmaps, int query_maps) {
  RaggedPlanParams p = {};
  p.cu = cu;
  p.maps = plan.maps;
  for (int c = 0; c < ncuts; ++c) p.sched[c] = plan.sched[c], p.cut[c] = cuts[c];
  for (int m = 0; m < nmaps; ++m) p.map[m] = maps[m];
  p.ncuts = ncuts;
  p.nmaps = nmaps;
  p.query_maps = query_maps;
  p.B = s.B;
  p.T = s.T;
  p.heads = s.Hkv;
  p.sms = sm_count_cached();
  return p;
}

int packed_map_blocks(int B, int nmaps, int threads) {
  const long long blocks = ((long long)B * nmaps + threads / 32 - 1) / (threads / 32);
  return (int)std::min<long long>(blocks, 4LL * sm_count_cached());
}

fa_status run_packed_plan(const RaggedPlanParams& p, cudaStream_t st) {
  // Few sequences: a small block, whose barriers are cheaper.
  const bool few = p.B <= kPlanCounted;
  const int threads = few ? 256 : 1024;
  return launch(FA_KERNEL_PACKED_PLAN, few ? ragged_plan_kernel<256> : ragged_plan_kernel<1024>,
                dim3(1 + packed_map_blocks(p.B, p.nmaps, threads)), dim3(threads), 0, st, p);
}

// A dimension of one element may have any stride; it gets a dense one, which the encoder takes.
fa_status packed_query_map(CUtensorMap* map, const fa_rows& r, const PackedShape& s, int tokens) {
  const long long head = s.H > 1 ? r.head : s.d, token = s.T > 1 ? r.token : s.d;
  const cuuint64_t dims[4] = {(cuuint64_t)s.d, (cuuint64_t)s.G(), (cuuint64_t)s.T, (cuuint64_t)s.Hkv};
  const cuuint64_t strides[3] = {2 * (cuuint64_t)head, 2 * (cuuint64_t)token, 2 * (cuuint64_t)head * s.G()};
  const cuuint32_t box[4] = {64, (cuuint32_t)s.G(), (cuuint32_t)tokens, 1};
  return encode_tile_map(map, r.data, 4, dims, strides, box);
}

fa_status packed_key_map(CUtensorMap* map, const fa_rows& r, const PackedShape& s, int box_rows) {
  const long long head = s.Hkv > 1 ? r.head : s.d, token = s.T > 1 ? r.token : s.d;
  const cuuint64_t dims[3] = {(cuuint64_t)s.d, (cuuint64_t)s.T, (cuuint64_t)s.Hkv};
  const cuuint64_t strides[2] = {2 * (cuuint64_t)token, 2 * (cuuint64_t)head};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1};
  return encode_tile_map(map, r.data, 3, dims, strides, box);
}

fa_status packed_shape_checks(const PackedShape& s, float scale, int causal) {
  if (s.B < 0 || s.T < 0 || s.H < 0 || s.Hkv < 0) return FA_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !(scale > 0.f)) return FA_ERR_INVALID_ARG;
  if (causal != 0 && causal != 1) return FA_ERR_INVALID_ARG;
  if (padded_head_dim(s.d) == 0) return FA_ERR_UNSUPPORTED;
  if (s.H == 0 && s.Hkv == 0) return FA_OK;
  if (s.Hkv == 0 || s.H % s.Hkv != 0) return FA_ERR_INVALID_ARG;
  if (s.G() > kPackedMaxGroup) return FA_ERR_UNSUPPORTED;
  // Work items, at most (tokens + sequences) * heads of a part each, are counted in 30 bits.
  if (s.T > (1 << 30) || s.B > (1 << 30) || ((long long)s.T + s.B) * s.Hkv > (long long)kPlanItems / 4)
    return FA_ERR_INVALID_ARG;
  return FA_OK;
}

fa_status packed_rows_checks(const fa_rows& r, int T, int heads) {
  if (!r.data) return FA_ERR_INVALID_ARG;
  if (!all_aligned(16, static_cast<const char*>(r.data))) return FA_ERR_MISALIGNED;
  const long long most = 1LL << 34;  // elements: strides of 2^40 bytes and more are not encoded, over 32 heads
  if ((T > 1 && (r.token <= 0 || r.token >= most)) || (heads > 1 && (r.head <= 0 || r.head >= most)))
    return FA_ERR_INVALID_ARG;
  if ((T > 1 && (r.token & 7)) || (heads > 1 && (r.head & 7))) return FA_ERR_MISALIGNED;
  return FA_OK;
}

// The form that a call of this variant runs (0: none).
static int packed_variant(int d, int variant) {
  if (variant == FA_BWD_AUTO) return fa_bwd_choose(1, 1, 1, d, 1);
  return bwd_supported(d, variant) ? variant : 0;
}

}  // namespace fa

using namespace fa;

extern "C" {

size_t fa_packed_fwd_workspace_size(int B, int T, int H, int Hkv, int d) {
  const PackedShape s = {B, T, H, Hkv, d};
  if (packed_shape_checks(s, 1.f, 0) != FA_OK || T == 0 || B == 0 || H == 0) return 0;
  return packed_fwd_bytes(s);
}

fa_status fa_packed_fwd(const fa_packed_fwd_args* a) {
  if (!a) return FA_ERR_INVALID_ARG;
  const PackedShape s = {a->B, a->T, a->H, a->Hkv, a->d};
  fa_status st = packed_shape_checks(s, a->scale, a->causal);
  if (st != FA_OK) return st;
  if (s.B == 0 || s.T == 0 || s.H == 0) return FA_OK;
  if (!a->lse || !a->cu) return FA_ERR_INVALID_ARG;
  for (const fa_rows* r : {&a->q, &a->o})
    if ((st = packed_rows_checks(*r, s.T, s.H)) != FA_OK) return st;
  for (const fa_rows* r : {&a->k, &a->v})
    if ((st = packed_rows_checks(*r, s.T, s.Hkv)) != FA_OK) return st;
  if (!all_aligned(4, a->lse, a->cu)) return FA_ERR_MISALIGNED;
  const size_t need = packed_fwd_bytes(s);
  if (need > 0 && (!a->workspace || !all_aligned(256, static_cast<char*>(a->workspace)) || a->workspace_bytes < need))
    return FA_ERR_WORKSPACE;
  return run_packed_fwd(*a, s);
}

size_t fa_packed_bwd_workspace_size(int B, int T, int H, int Hkv, int d, int variant) {
  const PackedShape s = {B, T, H, Hkv, d};
  if (packed_shape_checks(s, 1.f, 0) != FA_OK || T == 0 || H == 0) return 0;
  const int form = packed_variant(d, variant);
  return form ? packed_bwd_bytes(s, form) : 0;
}

fa_status fa_packed_bwd(const fa_packed_bwd_args* a) {
  if (!a) return FA_ERR_INVALID_ARG;
  const PackedShape s = {a->B, a->T, a->H, a->Hkv, a->d};
  fa_status st = packed_shape_checks(s, a->scale, a->causal);
  if (st != FA_OK) return st;
  if (a->variant != FA_BWD_AUTO && a->variant != FA_BWD_5GEMM && a->variant != FA_BWD_7GEMM) return FA_ERR_INVALID_ARG;
  const int form = packed_variant(s.d, a->variant);
  if (!form) return FA_ERR_UNSUPPORTED;
  if (s.T == 0 || s.H == 0) return FA_OK;
  if (!a->lse || (s.B > 0 && !a->cu)) return FA_ERR_INVALID_ARG;
  for (const fa_rows* r : {&a->q, &a->o, &a->dO, &a->dq})
    if ((st = packed_rows_checks(*r, s.T, s.H)) != FA_OK) return st;
  for (const fa_rows* r : {&a->k, &a->v, &a->dk, &a->dv})
    if ((st = packed_rows_checks(*r, s.T, s.Hkv)) != FA_OK) return st;
  if (!all_aligned(4, a->lse, a->cu)) return FA_ERR_MISALIGNED;
  if (!a->workspace || !all_aligned(256, static_cast<char*>(a->workspace)) ||
      a->workspace_bytes < packed_bwd_bytes(s, form))
    return FA_ERR_WORKSPACE;
  return run_packed_bwd(*a, s, form);
}

}  // extern "C"
