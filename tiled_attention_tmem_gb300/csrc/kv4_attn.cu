// Launcher of attention over the paged 4-bit cache: tile choice, workspace, checks.
#include "kv4_attn.cuh"
#include "kv4_wide.cuh"

#include <algorithm>
#include <cmath>

#include "kv4_host.h"

namespace fa {
namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
size_t round256(size_t x) { return (x + 255) / 256 * 256; }

// Tiles of 8 query rows that a warp keeps: as many as the rows need, up to what
// its registers hold (d*NT/4 of O, d*NT/8 of Q and half a unit of scores).
constexpr int most_nt(int d) { return d <= 64 ? 4 : d <= 192 ? 2 : 1; }
int choose_nt(int d, long long rows) {
  int nt = 1;
  while (nt < most_nt(d) && 8 * nt < rows) nt *= 2;
  return nt;
}

// The tcgen05 kernel takes a call whose requests have this many rows a kv head on average: the
// narrow tiles read and convert the cache again for each, its own time hardly depends on the
// rows.  Measured in us (narrow / wide), 8 / 32 requests of 8192 tokens and 4 kv heads:
//   d = 64   64 rows 32 / 32, 89 / 89     96 rows 43 / 33, 127 / 92
//   d = 96   32 rows 29 / 34, 81 / 97     40 rows 38 / 35, 114 / 97
//   d = 128  32 rows 34 / 36, 88 / 98     40 rows 44 / 37, 125 / 98
//   d = 192  16 rows 35 / 41, 85 / 113    17 rows 48 / 41, 141 / 113
//   d = 256  8 rows 34 / 42, 77 / 118     9 rows 44 / 42, 127 / 118
//   d = 384  16 rows 63 / 67, 186 / 195   20 rows 86 / 69, 269 / 197
// With fewer tokens it starts a few us later (8 of 2048, first case above the bound: 24 / 21,
// 20 / 20, 22 / 21, 21 / 22, 21 / 23, 36 / 35).  All with as many queries a request: where one
// request has many and the others one, the mean gives the narrow form, which reads that
// request's tokens for each of its tiles.
bool use_wide(int d, long long rows) { return rows > 8 * most_nt(d) * (d == 192 || d == 256 ? 1 : 2); }

// Three tiles, on units of 32 tokens, where they save the second pass of two row tiles of 16.
// Measured in us (one of 24 / two of 16): d = 128, 20 rows, 8 requests of 16384 tokens and 8
// kv heads 74 / 89, 64 of 4096 133 / 166; d = 96, 24 rows, 8 of 8192 41 / 47.  Two of 24 lose
// to three of 16: 40 rows, d = 128, 16 up to 4096 28 / 25, d = 96, 8 of 8192 67 / 63; and so
// does one in the form of a block per triple: d = 96, 20 rows, 8 of 300 11.8 / 10.4.
constexpr bool has_three(int d) { return d == 96 || d == 128; }

// The form a call takes, tiles and triples of its kernel, and its workspace.
struct Plan {
  int nt;
  bool solo, wide;
  int row_tiles, triples;            // of 8 * nt rows
  int wide_row_tiles, wide_triples;  // of 128 rows
  size_t off_ml, off_cuts, bytes;
};

// mean: rows of a request and kv head on average.
bool make_plan(int B, int H, int Hkv, int d, int max_q, int page, int width, long long mean, Plan& plan) {
  const long long rows = (long long)max_q * (H / Hkv);
  if (rows > 0x7fffffffLL || (long long)B * Hkv > 0x7fffffffLL) return false;
  plan.nt = choose_nt(d, rows);
  plan.wide = use_wide(d, std::min(mean, rows));
  const long long tiles = (rows + 8 * plan.nt - 1) / (8 * plan.nt), wide_tiles = (rows + 127) / 128;
  if (tiles * B * Hkv > 0x7fffffffLL / (8 * plan.nt)) return false;
  plan.row_tiles = (int)tiles;
  plan.triples = (int)(tiles * B * Hkv);
  plan.wide_row_tiles = (int)wide_tiles;
  plan.wide_triples = (int)(wide_tiles * B * Hkv);
  // A (request, kv head)'s units over all its row tiles are counted in 32 bits.
  if (((long long)width * page / 32 + 1) * tiles > 0x7fffffffLL) return false;
  // A block per triple while all fit the SMs at once and none has many units: measured in
  // us (solo / split) at d = 128, page 64: 64 triples of 4, 8, 16, 32 units 6.0 / 9.0,
  // 7.4 / 9.3, 10.5 / 10.0, 16.9 / 12.5; 256 triples 6.6 / 11.4, 8.7 / 13.9, 15.0 / 20.8,
  // 24.4 / 27.8; 4 triples of 16 units 11.0 / 8.6; 2048 triples (several waves) of 4 units
  // 35.8 / 30.2.  (Measured with tiles of 8 rows; other d and tiles follow the same rule.)
  const long long units = ((long long)width * page + kv4_unit(d, plan.nt) - 1) / kv4_unit(d, plan.nt);
  const int sms = sm_count_cached();
  plan.solo = plan.triples <= kv4_solo_blocks(d, plan.nt) * sms && units <= 10 + plan.triples / 10;
  plan.bytes = plan.off_ml = plan.off_cuts = 0;
  if (plan.solo) return true;
  if (has_three(d) && rows > 16 && rows <= 24) {
    plan.nt = 3;
    plan.row_tiles = 1;
    plan.triples = B * Hkv;
  }
  // Two slots of a tile's rows for every warp, or of 128 rows for every block.
  const size_t held = plan.wide ? (size_t)sms * 2 * 128 : (size_t)sms * kv4_warps(d, plan.nt) * 2 * 8 * plan.nt;
  plan.off_ml = round256(held * d * sizeof(float));
  plan.off_cuts = plan.off_ml + round256(held * 2 * sizeof(float));
  plan.bytes = plan.off_cuts + round256((plan.wide ? plan.wide_triples : plan.triples) * sizeof(int2));
  return true;
}

fa_status shape_checks(int B, int H, int Hkv, int d, int max_q) {
  if (B < 0 || H < 0 || Hkv < 0 || max_q < 0) return FA_ERR_INVALID_ARG;
  if (Hkv > 0 && H % Hkv != 0) return FA_ERR_INVALID_ARG;
  if (Hkv == 0 && H != 0) return FA_ERR_INVALID_ARG;
  if (padded_head_dim(d) == 0) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

// The merge of a kernel's parts: about eight blocks an SM, and no more than one warp for
// 16 channels of a row.
template <class C>
fa_status run_merge(const Kv4AttnParams& p, int triples, int most_rows, cudaStream_t st) {
  const int split = std::max(1, std::min(8 * sm_count_cached() / triples, std::min(C::ROWS, most_rows) * C::D / 16 / 8));
  return launch(FA_KERNEL_KV4_MERGE, kv4_merge_kernel<C>, dim3((unsigned)triples, (unsigned)split), dim3(256), 0, st, p);
}

template <int D, int NT>
fa_status run(Kv4AttnParams p, const Plan& plan, cudaStream_t st) {
  const int sms = sm_count_cached(), triples = plan.triples;
  const int most_rows = (int)std::min<long long>((long long)p.max_q * p.G, 1 << 20);
  p.row_tiles = plan.row_tiles;
  if constexpr (NT != 3) if (plan.solo) {
    using Solo = Kv4Cfg<D, NT, true>;
    static std::atomic<unsigned long long> raised{0};
    return launch_raised(FA_KERNEL_KV4_ATTN, kv4_attn_kernel<Solo>, dim3((unsigned)triples), dim3(Solo::THREADS),
                         Solo::SMEM, st, p, raised);
  }
  if (NT == most_nt(D) && plan.wide) {
    static std::atomic<unsigned long long> raised{0};
    using W = Kv4WideCfg<D>;
    p.row_tiles = plan.wide_row_tiles;
    fa_status s = launch_raised(FA_KERNEL_KV4_ATTN, kv4_wide_kernel<W>, dim3((unsigned)sms), dim3(W::THREADS), W::SMEM, st,
                                p, raised);
    return s != FA_OK ? s : run_merge<W>(p, plan.wide_triples, most_rows, st);
  }
  using C = Kv4Cfg<D, NT, false>;
  static std::atomic<unsigned long long> raised{0};
  fa_status s = launch_raised(FA_KERNEL_KV4_ATTN, kv4_attn_kernel<C>, dim3((unsigned)sms), dim3(C::THREADS), C::SMEM, st,
                              p, raised);
  return s != FA_OK ? s : run_merge<C>(p, triples, most_rows, st);
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

size_t fa_kv4_attn_workspace_size(int B, int H, int Hkv, int d, int max_q, int page, int width) {
  if (shape_checks(B, H, Hkv, d, max_q) != FA_OK || page_log2_of(page) < 0 || width < 0) return 0;
  if ((long long)width * page > 0x7fffffffLL) return 0;
  if (B == 0 || H == 0 || max_q == 0) return 0;
  // (The queries' mean, which the call knows, decides between two forms: enough for either.)
  Plan few, many;
  return make_plan(B, H, Hkv, d, max_q, page, width, 0, few) && make_plan(B, H, Hkv, d, max_q, page, width, 0x7fffffff, many)
             ? std::max(few.bytes, many.bytes)
             : 0;
}

fa_status fa_kv4_attn(const fa_kv4_cache* cache, const void* q, long long q_token, long long q_head, int T,
                      const int* cu, int max_q, const int* table, int width, const int* lengths, int B, int H,
                      float scale, void* o, long long o_token, long long o_head, float* lse, void* workspace,
                      size_t workspace_bytes, void* stream) {
  fa_status s = kv4_cache_checks(cache);
  if (s != FA_OK) return s;
  const int Hkv = cache->Hkv, d = cache->d;
  if ((s = shape_checks(B, H, Hkv, d, max_q)) != FA_OK) return s;
  if (T < 0 || width < 0 || !std::isfinite(scale) || !(scale > 0.f)) return FA_ERR_INVALID_ARG;
  if (!cu && (T < B || max_q < 1)) return FA_ERR_INVALID_ARG;
  if ((long long)width * cache->page > 0x7fffffffLL) return FA_ERR_INVALID_ARG;
  if (B == 0 || H == 0 || T == 0 || max_q == 0) return FA_OK;
  if (!q || !o || !lse || !lengths || (width > 0 && !table)) return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(o) || (q_token & 7) || (q_head & 7) || (o_token & 7) || (o_head & 7) ||
      !all_aligned(4, cu, table, lengths, lse))
    return FA_ERR_MISALIGNED;
  if (!cu) max_q = 1;
  Plan plan;
  const long long mean = ((long long)(cu ? T : B) * (H / Hkv) + B - 1) / B;
  if (!make_plan(B, H, Hkv, d, max_q, cache->page, width, mean, plan)) return FA_ERR_INVALID_ARG;
  if (plan.bytes &&
      (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 || workspace_bytes < plan.bytes))
    return FA_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  Kv4AttnParams p = {};
  p.q = static_cast<const uint16_t*>(q);
  p.o = static_cast<uint16_t*>(o);
  p.lse = lse;
  p.codes[0] = static_cast<const uint8_t*>(cache->k_codes);
  p.codes[1] = static_cast<const uint8_t*>(cache->v_codes);
  p.scales[0] = static_cast<const uint8_t*>(cache->k_scales);
  p.scales[1] = static_cast<const uint8_t*>(cache->v_scales);
  p.table = table;
  p.lengths = lengths;
  p.cu = cu;
  p.part_o = reinterpret_cast<float*>(ws);
  p.part_ml = reinterpret_cast<float*>(ws + plan.off_ml);
  p.cuts = reinterpret_cast<int2*>(ws + plan.off_cuts);
  p.err = device_error_word();
  if (!p.err) return record_cuda_error(cudaErrorMemoryAllocation);
  p.q_token = q_token;
  p.q_head = q_head;
  p.o_token = o_token;
  p.o_head = o_head;
  p.B = B;
  p.H = H;
  p.Hkv = Hkv;
  p.G = H / Hkv;
  p.T = T;
  p.width = width;
  p.pages = cache->pages;
  p.page_log2 = page_log2_of(cache->page);
  p.max_q = max_q;
  // (in fp64, which holds the product of any scale and gain)
  p.score = (float)(2.0 * std::frexp((double)scale * 1.4426950408889634 * cache->k_gain * kKv4ScaleBias, &p.score_exp));
  p.score_exp -= 1;
  p.v_gain = cache->v_gain * kKv4ScaleBias;
  cudaStream_t st = (cudaStream_t)stream;
  switch (d * 8 + plan.nt) {
    case 64 * 8 + 1: return run<64, 1>(p, plan, st);
    case 64 * 8 + 2: return run<64, 2>(p, plan, st);
    case 64 * 8 + 4: return run<64, 4>(p, plan, st);
    case 96 * 8 + 1: return run<96, 1>(p, plan, st);
    case 96 * 8 + 3: return run<96, 3>(p, plan, st);
    case 128 * 8 + 3: return run<128, 3>(p, plan, st);
    case 96 * 8 + 2: return run<96, 2>(p, plan, st);
    case 128 * 8 + 1: return run<128, 1>(p, plan, st);
    case 128 * 8 + 2: return run<128, 2>(p, plan, st);
    case 192 * 8 + 1: return run<192, 1>(p, plan, st);
    case 192 * 8 + 2: return run<192, 2>(p, plan, st);
    case 256 * 8 + 1: return run<256, 1>(p, plan, st);
    case 384 * 8 + 1: return run<384, 1>(p, plan, st);
  }
  return FA_ERR_UNSUPPORTED;
}

}  // extern "C"
