// Forward launcher of attention over packed sequences: the dense forward's tile
// configurations (fwd.cu) over items that ragged_plan_kernel lays out.
#include <algorithm>

#include "fwd.cuh"
#include "packed_host.h"

namespace fa {
namespace {

template <class C>
fa_status run(const PackedRows& q, const PackedRows& k, const PackedRows& v, const PackedRows& o, float* lse,
              const int* cu, const PackedShape& s, float scale, int causal, void* workspace, cudaStream_t st) {
  const int tokens = 128 / s.G();
  RaggedFwdParams p;
  fa_status e;
  if ((e = packed_query_map(&p.q_map, q, s, tokens)) != FA_OK) return e;
  if ((e = packed_key_map(&p.k_map, k, s, C::BN)) != FA_OK) return e;
  if ((e = packed_key_map(&p.v_map, v, s, C::BN)) != FA_OK) return e;
  const PackedPlan plan = packed_plan_at(workspace, s.B, 1);
  const PackedCut cut = {C::NQ * tokens, 1, 4.0 * s.d};  // K and V
  if ((e = run_packed_plan(plan, cu, s, &cut, 1, &p.v_map, 1, 0, st)) != FA_OK) return e;
  p.v_ends = plan.maps;
  p.sched = plan.sched[0];
  p.o = static_cast<uint16_t*>(o.data);
  p.o_token = o.token, p.o_head = o.head;
  p.lse = lse;
  p.err = device_error_word();
  if (!p.err) return record_cuda_error(cudaErrorMemoryAllocation);
  p.H = s.H, p.Hkv = s.Hkv, p.G = s.G(), p.by_G = (65536 + s.G() - 1) / s.G(), p.tokens = tokens, p.dv = s.d;
  p.scale_log2 = scale * kLog2e;
  p.causal = causal;
  // One CTA an SM, and no more than there can be items.
  const long long most = ((long long)s.T / cut.tokens + s.B) * s.Hkv;
  const unsigned grid = (unsigned)std::min<long long>(most, sm_count_cached());
  return launch(FA_KERNEL_FWD, fwd_kernel<C, false, RaggedFwdParams>, dim3(grid), dim3(C::THREADS), C::SMEM_BYTES, st, p);
}

}  // namespace

size_t packed_fwd_bytes(const PackedShape& s) { return packed_plan_bytes(s.B, 1, 1); }

fa_status run_packed_fwd(const PackedRows& q, const PackedRows& k, const PackedRows& v, const PackedRows& o, float* lse,
                         const int* cu, const PackedShape& s, float scale, int causal, void* workspace, cudaStream_t st) {
  switch (s.d) {
    case 64: return run<RaggedFwd64>(q, k, v, o, lse, cu, s, scale, causal, workspace, st);
    case 96:
    case 128: return run<Fwd128>(q, k, v, o, lse, cu, s, scale, causal, workspace, st);
    case 192: return run<Fwd192>(q, k, v, o, lse, cu, s, scale, causal, workspace, st);
    case 256: return run<Fwd256>(q, k, v, o, lse, cu, s, scale, causal, workspace, st);
    case 384: return run<Fwd384>(q, k, v, o, lse, cu, s, scale, causal, workspace, st);
  }
  return FA_ERR_UNSUPPORTED;
}

}  // namespace fa
