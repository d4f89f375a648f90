// The plan of a call over packed sequences (order of work, tensor maps), its
// checks, and the entry points.
#include <algorithm>
#include <cmath>

#include "packed_host.h"

namespace fa {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kPlanSorted = 4096;  // sequences that are put in order of their lengths
constexpr int kPlanItems = 1 << 30;

struct PlanParams {
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
__device__ __forceinline__ int plan_seq(const PlanParams& p, int b, int& start) {
  start = p.cu[b];
  const int end = p.cu[b + 1];
  return start >= 0 && start <= end && end <= p.T ? end - start : 0;
}

// Block 0: sequences by length, longest first (so that what is claimed last is short; by index where there are
// over 4096, where the longest is a small part of the work or the launch is long anyway), and the
// running sum of their work items.  The other blocks: a warp a tensor map, copied from its
// template and cut at the sequence's end.  Latency bounds it (a sort of 16 keys, a scan).
__global__ void __launch_bounds__(kPlanThreads) ragged_plan_kernel(const __grid_constant__ PlanParams p) {
  __shared__ unsigned long long keys[kPlanSorted];
  __shared__ long long sums[kPlanWarps];
  __shared__ alignas(128) uint32_t slot[kPlanWarps][32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_dep_wait();
  if (blockIdx.x > 0) {
    const long long tasks = (long long)p.B * p.nmaps, step = (long long)(gridDim.x - 1) * kPlanWarps;
    for (long long i = (long long)(blockIdx.x - 1) * kPlanWarps + warp; i < tasks; i += step) {
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
    return;
  }

  const bool sorted = p.B <= kPlanSorted;
  if (sorted) {
    int n = 1;
    while (n < p.B) n *= 2;
    for (int i = tid; i < n; i += kPlanThreads) {
      int start;
      keys[i] = i < p.B ? (unsigned long long)(0x7fffffff - plan_seq(p, i, start)) << 32 | (unsigned)i : ~0ull;
    }
    __syncthreads();
    for (int size = 2; size <= n; size *= 2)
      for (int gap = size / 2; gap > 0; gap /= 2) {
        for (int i = tid; i < n / 2; i += kPlanThreads) {
          const int a = 2 * i - (i & (gap - 1)), b = a + gap;
          const unsigned long long x = keys[a], y = keys[b];
          if ((x > y) == ((a & size) == 0)) keys[a] = y, keys[b] = x;
        }
        __syncthreads();
      }
  }
  const int run = (p.B + kPlanThreads - 1) / kPlanThreads;
  const int r0 = min(tid * run, p.B), r1 = min(r0 + run, p.B);
  for (int c = 0; c < p.ncuts; ++c) {
    const PackedCut cut = p.cut[c];
    const RaggedSched s = p.sched[c];
    auto tiles_of = [&](int len) -> long long { return (long long)((len + cut.tokens - 1) / cut.tokens) * cut.parts; };
    auto seq_of = [&](int r) { return sorted ? (int)(uint32_t)keys[r] : r; };
    long long sum = 0;
    int start;
    for (int r = r0; r < r1; ++r) sum += tiles_of(plan_seq(p, seq_of(r), start)) * p.heads;
    long long before = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, before, d);
      if (lane >= d) before += y;
    }
    if (lane == 31) sums[warp] = before;
    __syncthreads();
    before -= sum;
    for (int w = 0; w < warp; ++w) before += sums[w];
    __syncthreads();
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
      before += tiles * p.heads;
      if (r == p.B - 1) const_cast<int*>(s.base)[p.B] = (int)min(before, (long long)kPlanItems);
    }
    if (tid == 0) {
      *s.counter = 0;
      if (p.B == 0) const_cast<int*>(s.base)[0] = 0;
    }
  }
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

bool aligned(const void* p, size_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

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

fa_status run_packed_plan(const PackedPlan& plan, const int* cu, const PackedShape& s, const PackedCut* cuts, int ncuts,
                          const CUtensorMap* maps, int nmaps, int query_maps, cudaStream_t st) {
  PlanParams p = {};
  p.cu = cu;
  p.maps = plan.maps;
  for (int c = 0; c < ncuts; ++c) p.sched[c] = plan.sched[c], p.cut[c] = cuts[c];
  for (int m = 0; m < nmaps; ++m) p.map[m] = maps[m];
  p.ncuts = ncuts;
  p.nmaps = nmaps;
  p.B = s.B;
  p.T = s.T;
  p.heads = s.Hkv;
  p.sms = sm_count_cached();
  p.query_maps = query_maps;
  const long long tasks = ((long long)s.B * nmaps + kPlanWarps - 1) / kPlanWarps;
  const unsigned grid = 1 + (unsigned)std::min<long long>(tasks, 4LL * p.sms);
  return launch(FA_KERNEL_PACKED_PLAN, ragged_plan_kernel, dim3(grid), dim3(kPlanThreads), 0, st, p);
}

// A dimension of one element may have any stride; it gets a dense one, which the encoder takes.
fa_status packed_query_map(CUtensorMap* map, const PackedRows& r, const PackedShape& s, int tokens) {
  const long long head = s.H > 1 ? r.head : s.d, token = s.T > 1 ? r.token : s.d;
  const cuuint64_t dims[4] = {(cuuint64_t)s.d, (cuuint64_t)s.G(), (cuuint64_t)s.T, (cuuint64_t)s.Hkv};
  const cuuint64_t strides[3] = {2 * (cuuint64_t)head, 2 * (cuuint64_t)token, 2 * (cuuint64_t)head * s.G()};
  const cuuint32_t box[4] = {64, (cuuint32_t)s.G(), (cuuint32_t)tokens, 1};
  return encode_tile_map(map, r.data, 4, dims, strides, box);
}

fa_status packed_key_map(CUtensorMap* map, const PackedRows& r, const PackedShape& s, int box_rows) {
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

fa_status packed_rows_checks(const PackedRows& r, int T, int heads) {
  if (!r.data) return FA_ERR_INVALID_ARG;
  if (!aligned(r.data, 16)) return FA_ERR_MISALIGNED;
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

fa_status fa_packed_fwd(const void* q, long long q_token, long long q_head, const void* k, long long k_token,
                        long long k_head, const void* v, long long v_token, long long v_head, void* o,
                        long long o_token, long long o_head, float* lse, const int* cu, int B, int T, int H, int Hkv,
                        int d, float scale, int causal, void* workspace, size_t workspace_bytes, void* stream) {
  const PackedShape s = {B, T, H, Hkv, d};
  fa_status st = packed_shape_checks(s, scale, causal);
  if (st != FA_OK) return st;
  if (B == 0 || T == 0 || H == 0) return FA_OK;
  const PackedRows rq = {const_cast<void*>(q), q_token, q_head}, rk = {const_cast<void*>(k), k_token, k_head},
                   rv = {const_cast<void*>(v), v_token, v_head}, ro = {o, o_token, o_head};
  if (!lse || !cu) return FA_ERR_INVALID_ARG;
  for (const PackedRows* r : {&rq, &ro})
    if ((st = packed_rows_checks(*r, T, H)) != FA_OK) return st;
  for (const PackedRows* r : {&rk, &rv})
    if ((st = packed_rows_checks(*r, T, Hkv)) != FA_OK) return st;
  if (!aligned(lse, 4) || !aligned(cu, 4)) return FA_ERR_MISALIGNED;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < packed_fwd_bytes(s)) return FA_ERR_WORKSPACE;
  return run_packed_fwd(rq, rk, rv, ro, lse, cu, s, scale, causal, workspace, (cudaStream_t)stream);
}

size_t fa_packed_bwd_workspace_size(int B, int T, int H, int Hkv, int d, int variant) {
  const PackedShape s = {B, T, H, Hkv, d};
  if (packed_shape_checks(s, 1.f, 0) != FA_OK || T == 0 || H == 0) return 0;
  const int form = packed_variant(d, variant);
  return form ? packed_bwd_bytes(s, form) : 0;
}

fa_status fa_packed_bwd(const void* q, long long q_token, long long q_head, const void* k, long long k_token,
                        long long k_head, const void* v, long long v_token, long long v_head, const void* o,
                        long long o_token, long long o_head, const void* dO, long long do_token, long long do_head,
                        const float* lse, void* dq, long long dq_token, long long dq_head, void* dk, long long dk_token,
                        long long dk_head, void* dv, long long dv_token, long long dv_head, const int* cu, int B, int T,
                        int H, int Hkv, int d, float scale, int causal, int variant, void* workspace,
                        size_t workspace_bytes, void* stream) {
  const PackedShape s = {B, T, H, Hkv, d};
  fa_status st = packed_shape_checks(s, scale, causal);
  if (st != FA_OK) return st;
  if (variant != FA_BWD_AUTO && variant != FA_BWD_5GEMM && variant != FA_BWD_7GEMM) return FA_ERR_INVALID_ARG;
  const int form = packed_variant(d, variant);
  if (!form) return FA_ERR_UNSUPPORTED;
  if (T == 0 || H == 0) return FA_OK;
  const PackedRows rq = {const_cast<void*>(q), q_token, q_head}, rk = {const_cast<void*>(k), k_token, k_head},
                   rv = {const_cast<void*>(v), v_token, v_head}, ro = {const_cast<void*>(o), o_token, o_head},
                   rg = {const_cast<void*>(dO), do_token, do_head}, rdq = {dq, dq_token, dq_head},
                   rdk = {dk, dk_token, dk_head}, rdv = {dv, dv_token, dv_head};
  if (!lse || (B > 0 && !cu)) return FA_ERR_INVALID_ARG;
  for (const PackedRows* r : {&rq, &ro, &rg, &rdq})
    if ((st = packed_rows_checks(*r, T, H)) != FA_OK) return st;
  for (const PackedRows* r : {&rk, &rv, &rdk, &rdv})
    if ((st = packed_rows_checks(*r, T, Hkv)) != FA_OK) return st;
  if (!aligned(lse, 4) || !aligned(cu, 4)) return FA_ERR_MISALIGNED;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < packed_bwd_bytes(s, form)) return FA_ERR_WORKSPACE;
  return run_packed_bwd(rq, rk, rv, ro, rg, lse, rdq, rdk, rdv, cu, s, scale, causal, form, workspace,
                        (cudaStream_t)stream);
}

}  // extern "C"
