// Forward launcher of attention over packed sequences: the dense forward's tile
// configurations (fwd.cu) over items that ragged_plan_kernel lays out.
#include <algorithm>

#include "fwd.cuh"
#include "kv4_host.h"
#include "packed_host.h"
#include "packed_plan.cuh"

namespace fa {
namespace {

template <class C>
fa_status run(const fa_packed_fwd_args& a, const PackedShape& s) {
  static std::atomic<unsigned long long> raised{0};
  const cudaStream_t st = (cudaStream_t)a.stream;
  const int tokens = 128 / s.G();
  RaggedFwdParams p;
  fa_status e;
  if ((e = packed_query_map(&p.q_map, a.q, s, tokens)) != FA_OK) return e;
  if ((e = packed_key_map(&p.k_map, a.k, s, C::BN)) != FA_OK) return e;
  if ((e = packed_key_map(&p.v_map, a.v, s, C::BN)) != FA_OK) return e;
  const PackedPlan plan = packed_plan_at(a.workspace, s.B, 1);
  // Items of one tile where those of two would not fill the SMs: shorter by half, if slower a tile.  Measured in us
  // (items of two / of one): two sequences up to 1500, four heads on two of 64: 21 / 17; one of 2048, eight on one of
  // 128: 26 / 25; two up to 2048, eight on two of 128: 26 / 24; above an item an SM, four up to 1500: 24 / 29.
  const double items = (s.T / (2.0 * tokens) + s.B / 2.0) * s.Hkv;
  p.tiles = C::NQ > 1 && items < sm_count_cached() ? 1 : C::NQ;
  const PackedCut cut = {p.tiles * tokens, 1, 4.0 * s.d};  // K and V
  if ((e = run_packed_plan(packed_plan_params(plan, a.cu, s, &cut, 1, &p.v_map, 1, 0), st)) != FA_OK) return e;
  p.v_ends = plan.maps;
  p.sched = plan.sched[0];
  p.o = static_cast<uint16_t*>(const_cast<void*>(a.o.data));
  p.o_token = a.o.token, p.o_head = a.o.head;
  p.lse = a.lse;
  p.err = device_error_word();
  if (!p.err) return record_cuda_error(cudaErrorMemoryAllocation);
  p.H = s.H, p.Hkv = s.Hkv, p.G = s.G(), p.by_G = (65536 + s.G() - 1) / s.G(), p.tokens = tokens, p.dv = s.d;
  p.scale_log2 = a.scale * kLog2e;
  p.causal = a.causal;
  // One CTA an SM, and no more than there can be items.
  const long long most = ((long long)s.T / cut.tokens + s.B) * s.Hkv;
  const unsigned grid = (unsigned)std::min<long long>(most, sm_count_cached());
  return launch_raised(FA_KERNEL_FWD, fwd_kernel<C, false, RaggedFwdParams>, dim3(grid), dim3(C::THREADS), C::SMEM_BYTES,
                       st, p, raised);
}

}  // namespace

size_t packed_fwd_bytes(const PackedShape& s) { return packed_plan_bytes(s.B, 1, 1); }

fa_status run_packed_fwd(const fa_packed_fwd_args& a, const PackedShape& s) {
  switch (s.d) {
    case 64: return run<RaggedFwd64>(a, s);
    case 96:
    case 128: return run<Fwd128>(a, s);
    case 192: return run<Fwd192>(a, s);
    case 256: return run<Fwd256>(a, s);
    case 384: return run<Fwd384>(a, s);
  }
  return FA_ERR_UNSUPPORTED;
}

}  // namespace fa
