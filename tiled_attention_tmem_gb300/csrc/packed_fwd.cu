// Forward launcher of attention over packed sequences: the dense forward's tile
// configurations (fwd.cuh) over items that ragged_plan_kernel lays out, or, where there are few, the kernel itself.
#include <algorithm>

#include "fwd.cuh"
#include "kv4_host.h"
#include "packed_host.h"
#include "packed_plan.cuh"

namespace fa {
namespace {

// P: DirectFwdParams or RaggedFwdParams, without or with a plan.
template <class C, class P>
fa_status run(const fa_packed_fwd_args& a, const PackedShape& s) {
  static std::atomic<unsigned long long> raised{0};
  const cudaStream_t st = (cudaStream_t)a.stream;
  const int tokens = 128 / s.G();
  P p;
  fa_status e;
  if ((e = packed_query_map(&p.q_map, a.q, s, tokens)) != FA_OK) return e;
  if ((e = packed_key_map(&p.k_map, a.k, s, C::BN)) != FA_OK) return e;
  if ((e = packed_key_map(&p.v_map, a.v, s, C::BN)) != FA_OK) return e;
  if constexpr (P::kDirect) {
    p.v_ends = nullptr;
    p.sched = RaggedSched{};
    p.sched.B = s.B, p.sched.cu = a.cu, p.sched.T = s.T;
  } else {
    const PackedPlan plan = packed_plan_at(a.workspace, s.B, 1);
    const PackedCut cut = {C::NQ * tokens, 1, 4.0 * s.d};  // K and V
    if ((e = run_packed_plan(packed_plan_params(plan, a.cu, s, &cut, 1, &p.v_map, 1, 0), st)) != FA_OK) return e;
    p.v_ends = plan.maps;
    p.sched = plan.sched[0];
  }
  p.o = static_cast<uint16_t*>(const_cast<void*>(a.o.data));
  p.o_token = a.o.token, p.o_head = a.o.head;
  p.lse = a.lse;
  p.err = device_error_word();
  if (!p.err) return record_cuda_error(cudaErrorMemoryAllocation);
  p.H = s.H, p.Hkv = s.Hkv, p.G = s.G(), p.by_G = (65536 + s.G() - 1) / s.G(), p.tokens = tokens, p.dv = s.d;
  p.scale_log2 = a.scale * kLog2e;
  p.causal = a.causal;
  // As many CTAs as the SMs hold, and no more than there can be items.
  const long long most = ((long long)s.T / (C::NQ * tokens) + s.B) * s.Hkv;
  const unsigned grid = (unsigned)std::min<long long>(most, C::CTAS * sm_count_cached());
  return launch_raised(FA_KERNEL_FWD, fwd_kernel<C, false, P>, dim3(grid), dim3(C::THREADS), C::SMEM_BYTES,
                       st, p, raised);
}

// Items of one tile that there can be, and whether the SMs take two of them each or fewer.
bool few_items(const PackedShape& s) {
  return ((long long)s.T / (128 / s.G()) + s.B) * s.Hkv <= 2LL * sm_count_cached();
}

// Whether d = 96 or 128 runs two CTAs an SM: where items are few, since a lone tile's MMAs do not overlap its
// softmax in the tiles of two, and by the tokens of a mean sequence, since short items are mostly item changes.
// Measured, tiles of two (with one of them used where items are few) / two CTAs in us, d = 128.  Few items, causal: one
// sequence of 2048, eight heads on one, 24.9 / 20.1; one of 16384, one head, 156 / 123; two of 2048, eight on eight, 41 /
// 27; at d = 96 41 / 33, at the worst one of 8192, four on two, 81 / 93.  Above that, one of 6000, 32 on one: 176 /
// 203.  Many, 32 heads on 8, lengths at random, means in a loop at the power limit: causal, 42 of 431: 115 / 100, 21 of 758:
// 139 / 135, 16 of 1160: 191 / 195, 4 of 5001: 669 / 745; without the mask, where an item has twice the keys and both of
// its tiles the same ones, 128 of 129: 100 / 89, 64 of 257: 118 / 113, 32 of 475: 153 / 161.  d = 96, whose tiles' last
// quarter is loaded as zeros: causal, 32 of 475: 101 / 100, 21 of 758: 132 / 150; without the mask 85 of 206: 109 / 103, 32
// of 475: 144 / 168.  (d = 64 always runs two: causal, 32 of 475: 90 / 74, 8 of 2182: 198 / 186, 4 of 5001: 497 / 505; without the
// mask 930 / 971: long sequences lose 2 to 4 % by it.)
bool two_ctas(const PackedShape& s, int causal) {
  const long long mean = s.T / s.B;
  return few_items(s) || (causal ? mean : 3 * mean) <= (s.d == 96 ? 576 : 960);
}

template <class P>
fa_status run_with(const fa_packed_fwd_args& a, const PackedShape& s) {
  switch (s.d) {
    case 64: return run<RaggedFwd64, P>(a, s);
    case 96:
    case 128:
      if constexpr (!P::kDirect)
        if (!two_ctas(s, a.causal)) return run<Fwd128, P>(a, s);
      return run<RaggedFwd128, P>(a, s);
    case 192: return run<Fwd192, P>(a, s);
    case 256: return run<Fwd256, P>(a, s);
    case 384: return run<Fwd384, P>(a, s);
  }
  return FA_ERR_UNSUPPORTED;
}

}  // namespace

// Without a plan (and a workspace) where items are few and a lane each suffices for the sequences.  A plan is a launch
// before the kernel's, and lets more items than that be claimed by whoever is free.  Measured in us on the GPU, and of
// a call's time on the host (without / with a plan): four sequences of 71 tokens in all, eight heads on two of
// 64: 5.2 / 8.1, 14 / 20; four of 512, eight on eight of 64: 9.0 / 11.5; eight of 900, four on two of 128, 240 items: 17.3
// / 19.9; 1500 and 700, eight on four of 384: 35.3 / 36.9.
size_t packed_fwd_bytes(const PackedShape& s) {
  return s.B <= kRaggedDirect && few_items(s) ? 0 : packed_plan_bytes(s.B, 1, 1);
}

fa_status run_packed_fwd(const fa_packed_fwd_args& a, const PackedShape& s) {
  return packed_fwd_bytes(s) > 0 ? run_with<RaggedFwdParams>(a, s) : run_with<DirectFwdParams>(a, s);
}

}  // namespace fa
