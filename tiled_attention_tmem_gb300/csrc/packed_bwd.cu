// Backward of attention over packed sequences: the dense backward's kernels (bwd.cuh)
// over items in the plan's order, with a preprocess (which makes the plan) and a dQ conversion that
// go by query tiles.  12 sequences up to 4096, 32 heads on 8 of 128, causal: 145 + 1590 + 104 us.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "bwd.cuh"
#include "kv4_host.h"
#include "packed_host.h"
#include "packed_plan.cuh"

namespace fa {
namespace {

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

struct RowsIn {
  const uint16_t* data;
  long long token, head;
};
struct RowsOut {
  uint16_t* data;
  long long token, head;
};

// Tiles of `tokens` tokens with the G heads of a kv head: `rows` rows of the row
// arrays, of which the last rows - tokens * G are nobody's.
struct RowTiles {
  const int* cu;
  int B, T, H, Hkv, G;
  int tokens, rows, slots;
  int hd;
  int by_G;  // 65536 / G rounded up: r / G = r * by_G >> 16 for r < 128, G <= 32
};

// The rows [lo, hi) of the sequences: cu does not decrease, so those that do not lie in [0, T) are the
// first ones and the last.  (Whatever cu holds, 0 <= lo <= hi <= T.)
__device__ __forceinline__ void rows_of_sequences(const int* cu, int B, int T, int& lo, int& hi) {
  auto first_at_least = [&](long long bound) {  // the first entry that is, or B + 1
    int a = 0, b = B + 1;
    while (a < b) {
      const int mid = a + (b - a) / 2;
      if (cu[mid] >= bound) b = mid;
      else a = mid + 1;
    }
    return a;
  };
  lo = hi = 0;
  if (B == 0) return;
  lo = cu[0];
  if (lo < 0) {
    const int b = first_at_least(0);
    lo = b <= B ? cu[b] : T;
  }
  hi = cu[B];
  if (hi > T) {
    const int b = first_at_least(T + 1LL) - 1;
    hi = b >= 0 ? cu[b] : 0;
  }
  lo = min(max(lo, 0), T), hi = min(max(hi, lo), T);
}

// The sequence that holds tile slot ts, and the slot's first token in it; false where none does.
// Sequence b has the slots from cu[b] / tokens + b on, which grow with b: a warp looks at 32 of
// them at a time.
__device__ __forceinline__ bool tile_of_slot(const RowTiles& t, int ts, int& start, int& len, int& tok0) {
  if (t.B == 0) return false;
  const int lane = threadIdx.x & 31;
  int lo = 0, end = t.B;  // the last b in [lo, end) whose first slot is not past ts (or lo)
  while (end - lo > 1) {
    const int step = (end - lo + 31) / 32, b = lo + lane * step;
    const bool past = b >= end || (long long)min(max(t.cu[b], 0), t.T) / t.tokens + b > ts;
    const unsigned mask = __ballot_sync(0xffffffffu, past);
    const int first = mask ? __ffs(mask) - 1 : 32;
    if (first == 0) {
      end = lo + 1;
    } else {
      lo += (first - 1) * step;
      end = min(end, lo + step);
    }
  }
  start = t.cu[lo];
  const int stop = t.cu[lo + 1];
  if (start < 0 || start > stop || stop > t.T) return false;
  len = stop - start;
  const long long first = (long long)ts - start / t.tokens - lo;
  if (first < 0 || first * t.tokens >= len) return false;
  tok0 = (int)first * t.tokens;
  return true;
}

struct RaggedPreParams {
  RaggedPlanParams plan;
  int plan_blocks;  // the first block makes the schedule, the next plan_blocks - 1 the tensor maps (0: no sequences)
  RowTiles tiles;
  RowsIn o, dO;
  const float* lse;
  float* lse2;
  float* dd;
  float* dqacc;  // NULL for the 7-GEMM form
  RowsOut out[3];  // dq, dk, dv: their rows of no sequence are zeroed
};

// The plan, and beside it the rows: a block a tile slot at a time, GT threads a row: D_i = sum_c dO_ic O_ic (fp32) and the log2-domain
// LSE, both negated, and (5-GEMM) zeros for the fp32 dQ rows.  Memory bounds it: 12 sequences up to 4096, 32 heads of
// 128, 145 us; 64 up to 512, 16 of 64, 24 us.
template <int D>
__global__ void __launch_bounds__(256, D <= 256 ? 4 : 2) ragged_pre_kernel(const __grid_constant__ RaggedPreParams p) {
  grid_dep_wait();
  if ((int)blockIdx.x < p.plan_blocks) {
    if (blockIdx.x == 0) plan_schedule<256>(p.plan);
    else plan_maps<256>(p.plan, blockIdx.x - 1, p.plan_blocks - 1);
    return;
  }
  const int block = blockIdx.x - p.plan_blocks, blocks = gridDim.x - p.plan_blocks;
  constexpr int GT = D / 8 <= 32 ? D / 8 : 16;
  constexpr int CH = D / 8 / GT;
  const RowTiles& t = p.tiles;
  const int sub = threadIdx.x % GT;
  const long long work = (long long)t.slots * t.Hkv;
  for (long long w = block; w < work; w += blocks) {
    const int ts = (int)(w / t.Hkv), kvh = (int)(w - (long long)ts * t.Hkv);
    int start, len, tok0;
    if (!tile_of_slot(t, ts, start, len, tok0)) continue;
    // UN rows of a thread's at a time, all of their loads first.
    constexpr int STEP = 256 / GT, UN = 4;
#pragma unroll 1
    for (int r0 = threadIdx.x / GT; r0 < t.rows; r0 += UN * STEP) {
      uint4 a[UN][CH], b[UN][CH];
      float lse[UN];
#pragma unroll
      for (int i = 0; i < UN; ++i) {
        const int r = r0 + i * STEP, of = (r * t.by_G) >> 16, tok = tok0 + of, head = kvh * t.G + r - of * t.G;
        const bool have = of < t.tokens && r < t.rows && tok < len;
        const uint16_t* o = p.o.data + (have ? (start + tok) * p.o.token + head * p.o.head : 0);
        const uint16_t* g = p.dO.data + (have ? (start + tok) * p.dO.token + head * p.dO.head : 0);
        lse[i] = have && sub == 0 ? p.lse[(long long)(start + tok) * t.H + head] : -INFINITY;
#pragma unroll
        for (int ch = 0; ch < CH; ++ch) {
          const int c = (ch * GT + sub) * 8;
          a[i][ch] = b[i][ch] = make_uint4(0u, 0u, 0u, 0u);
          if (have && c < t.hd) {
            a[i][ch] = *reinterpret_cast<const uint4*>(o + c);
            b[i][ch] = *reinterpret_cast<const uint4*>(g + c);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < UN; ++i) {
        const int r = r0 + i * STEP;
        float acc = 0.f;
#pragma unroll
        for (int ch = 0; ch < CH; ++ch) {
          const uint32_t av[4] = {a[i][ch].x, a[i][ch].y, a[i][ch].z, a[i][ch].w};
          const uint32_t bv[4] = {b[i][ch].x, b[i][ch].y, b[i][ch].z, b[i][ch].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            acc = fmaf(__uint_as_float(av[e] << 16), __uint_as_float(bv[e] << 16), acc);
            acc = fmaf(__uint_as_float(av[e] & 0xffff0000u), __uint_as_float(bv[e] & 0xffff0000u), acc);
          }
        }
#pragma unroll
        for (int d = GT / 2; d > 0; d >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, d, GT);
        if (r >= t.rows) continue;
        const size_t row = ((size_t)kvh * t.slots + ts) * t.rows + r;
        if (sub == 0) {
          p.dd[row] = -acc;
          // (a row whose scores are all -inf has no probabilities: -inf - -inf would be NaN)
          p.lse2[row] = lse[i] == -INFINITY ? -INFINITY : -(lse[i] * kLog2e);
        }
        if (p.dqacc) {
#pragma unroll
          for (int ch = 0; ch < CH; ++ch) {
            float4* z = reinterpret_cast<float4*>(p.dqacc + row * D + (ch * GT + sub) * 8);
            z[0] = z[1] = make_float4(0.f, 0.f, 0.f, 0.f);
          }
        }
      }
    }
  }
  // Gradients of the rows of no sequence: before the first one and behind the last.
  int lo, hi;
  rows_of_sequences(t.cu, t.B, t.T, lo, hi);
  const long long spare = (long long)lo + (t.T - hi), chunks = t.hd / 8;
#pragma unroll
  for (int x = 0; x < 3; ++x) {
    const int heads = x == 0 ? t.H : t.Hkv;
    const long long n = spare * heads * chunks;
    for (long long i = (long long)block * 256 + threadIdx.x; i < n; i += (long long)blocks * 256) {
      const long long row = i / (heads * chunks), rest = i - row * heads * chunks;
      const long long tok = row < lo ? row : hi + (row - lo);
      *reinterpret_cast<uint4*>(p.out[x].data + tok * p.out[x].token + rest / chunks * p.out[x].head +
                                rest % chunks * 8) = make_uint4(0u, 0u, 0u, 0u);
    }
  }
}

struct RaggedConvParams {
  RowTiles tiles;
  const float* dqacc;
  RowsOut dq;
  int* err;
  float scale;
};

// dq = scale * the fp32 sums (5-GEMM), bf16.  A block a tile slot, eight columns a thread, four rows at a
// time.  Memory bounds it: 104 us and 14 at the sizes above.
template <int D>
__global__ void __launch_bounds__(256) ragged_conv_kernel(const __grid_constant__ RaggedConvParams p) {
  grid_dep_wait();
  if (*reinterpret_cast<volatile const int*>(p.err) != 0) return;
  const RowTiles& t = p.tiles;
  const long long work = (long long)t.slots * t.Hkv;
  for (long long w = blockIdx.x; w < work; w += gridDim.x) {
    const int ts = (int)(w / t.Hkv), kvh = (int)(w - (long long)ts * t.Hkv);
    int start, len, tok0;
    if (!tile_of_slot(t, ts, start, len, tok0)) continue;
    const int rows = min(t.tokens, len - tok0) * t.G;
    const float* slot = p.dqacc + ((size_t)kvh * t.slots + ts) * t.rows * D;
    constexpr int GT = D / 8, STEP = 256 / GT, UN = 4;
    const int c = threadIdx.x % GT * 8;
    if (c >= t.hd) continue;
#pragma unroll 1
    for (int r0 = threadIdx.x / GT; r0 < rows; r0 += UN * STEP) {
      float4 a[UN], b[UN];
#pragma unroll
      for (int u = 0; u < UN; ++u) {
        const int r = min(r0 + u * STEP, rows - 1);
        a[u] = *reinterpret_cast<const float4*>(slot + r * D + dq_swz(r, c));
        b[u] = *reinterpret_cast<const float4*>(slot + r * D + dq_swz(r, c + 4));
      }
#pragma unroll
      for (int u = 0; u < UN; ++u) {
        const int r = r0 + u * STEP, of = (r * t.by_G) >> 16;
        if (r >= rows) break;
        *reinterpret_cast<uint4*>(p.dq.data + (start + tok0 + of) * p.dq.token + (kvh * t.G + r - of * t.G) * p.dq.head + c) =
            make_uint4(pack_bf16(a[u].x * p.scale, a[u].y * p.scale), pack_bf16(a[u].z * p.scale, a[u].w * p.scale),
                       pack_bf16(b[u].x * p.scale, b[u].y * p.scale), pack_bf16(b[u].z * p.scale, b[u].w * p.scale));
      }
    }
  }
}

// Sum of the query-range parts: dv = sum_s dvpart[s], dk = scale sum_s dkpart[s], in a fixed order, bf16.
struct RaggedKVSumParams {
  const float* dkpart;
  const float* dvpart;
  RowsOut dk, dv;
  const int* cu;
  int* err;
  int B, T, Hkv, hd, D, parts;
  float scale;
};

__global__ void __launch_bounds__(256) ragged_kvsum_kernel(const __grid_constant__ RaggedKVSumParams p) {
  grid_dep_wait();
  if (*reinterpret_cast<volatile const int*>(p.err) != 0) return;
  const int chunks = p.hd / 8;
  int lo, hi;  // (the other rows are zeros already)
  rows_of_sequences(p.cu, p.B, p.T, lo, hi);
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x, work = (long long)(hi - lo) * p.Hkv * chunks;
  if (i >= work) return;
  const long long row = i / chunks;
  const int c = (int)(i - row * chunks) * 8, tok = lo + (int)(row / p.Hkv), head = (int)(row % p.Hkv);
  const size_t off = ((size_t)head * p.T + tok) * p.D + c, stride = (size_t)p.Hkv * p.T * p.D;
  float a[8] = {}, b[8] = {};
  for (int s = 0; s < p.parts; ++s) {
    const float4* v4 = reinterpret_cast<const float4*>(p.dvpart + s * stride + off);
    const float4* k4 = reinterpret_cast<const float4*>(p.dkpart + s * stride + off);
    const float4 v0 = v4[0], v1 = v4[1], k0 = k4[0], k1 = k4[1];
    a[0] += v0.x, a[1] += v0.y, a[2] += v0.z, a[3] += v0.w, a[4] += v1.x, a[5] += v1.y, a[6] += v1.z, a[7] += v1.w;
    b[0] += k0.x, b[1] += k0.y, b[2] += k0.z, b[3] += k0.w, b[4] += k1.x, b[5] += k1.y, b[6] += k1.z, b[7] += k1.w;
  }
  const float sc = p.scale;
  *reinterpret_cast<uint4*>(p.dv.data + tok * p.dv.token + head * p.dv.head + c) =
      make_uint4(pack_bf16(a[0], a[1]), pack_bf16(a[2], a[3]), pack_bf16(a[4], a[5]), pack_bf16(a[6], a[7]));
  *reinterpret_cast<uint4*>(p.dk.data + tok * p.dk.token + head * p.dk.head + c) =
      make_uint4(pack_bf16(b[0] * sc, b[1] * sc), pack_bf16(b[2] * sc, b[3] * sc), pack_bf16(b[4] * sc, b[5] * sc),
                 pack_bf16(b[6] * sc, b[7] * sc));
}

// Query parts per key tile, by the rule of the dense backward (bwd.cu, choose_qsplit) over what is known of the
// sequences without reading them: key tiles from the tokens and half a tile a sequence, and the rows of a mean
// sequence's group of heads, of which a part gets 512 at least.  Measured, dK/dV kernel without / with parts: one
// sequence of 2048, eight heads on one of 128: 320 / 57 us; four up to 1574, three on one of 192: 142 / 65.  From two
// items an SM on the SMs are full, and the parts' sums would be extra traffic.
int packed_qsplit(const PackedShape& s, int dsplit, int causal) {
  if (s.B == 0) return 1;
  const double items = (s.T / 128.0 + s.B / 2.0) * s.Hkv * dsplit, sms = sm_count_cached();
  if (items >= 2.0 * sms) return 1;
  const long cap = std::max(1LL, std::min(8LL, (long long)s.T / s.B * s.G() / 512));
  long parts = 1;
  if (causal) parts = std::lround(3.0 * sms / items);
  else if (items <= 0.85 * sms) parts = std::max(2L, std::lround(0.85 * sms / items));
  return (int)std::max(1L, std::min(cap, parts));
}

// The workspace: the plan, then lse2, dd, (5-GEMM) dqacc by query tiles, and the parts of a split (as many as
// either mask has).
struct BwdLayout {
  int cuts, nmaps, slots;
  size_t rows, plan, total, parts;  // parts: where they begin
  BwdLayout(const PackedShape& s, int variant, int tile_rows, int D, int dsplit) {
    const bool five = variant == FA_BWD_5GEMM;
    cuts = five ? 1 : 2, nmaps = five ? 4 : 6;
    slots = s.T / (tile_rows / s.G()) + s.B;
    rows = (size_t)s.Hkv * slots * tile_rows;
    plan = packed_plan_bytes(s.B, cuts, nmaps);
    parts = plan + 2 * align256(4 * rows) + (five ? align256(4 * rows * D) : 0);
    const int most = std::max(packed_qsplit(s, dsplit, 0), packed_qsplit(s, dsplit, 1));
    total = parts + (most > 1 ? 2 * (size_t)most * s.Hkv * s.T * D * sizeof(float) : 0);
  }
};

RowsIn in(const fa_rows& r) { return {static_cast<const uint16_t*>(r.data), r.token, r.head}; }
RowsOut out(const fa_rows& r) { return {static_cast<uint16_t*>(const_cast<void*>(r.data)), r.token, r.head}; }

// KV: the dK/dV kernel; Q: the dQ kernel (void: 5-GEMM).  DP: the preprocess's head dimension.
template <int DP, class KV, class Q>
fa_status run(const fa_packed_bwd_args& c, const PackedShape& s) {
  static std::atomic<unsigned long long> kv_raised{0}, few_raised{0}, q_raised{0};
  constexpr bool five = KV::DQ;
  const cudaStream_t st = (cudaStream_t)c.stream;
  const BwdLayout lay(s, five ? FA_BWD_5GEMM : FA_BWD_7GEMM, KV::BM, KV::D, KV::DSPLIT);
  const int qsplit = packed_qsplit(s, KV::DSPLIT, c.causal);
  const PackedPlan plan = packed_plan_at(c.workspace, s.B, lay.cuts);
  uint8_t* at = static_cast<uint8_t*>(c.workspace) + lay.plan;
  float* const lse2 = reinterpret_cast<float*>(at);
  float* const dd = reinterpret_cast<float*>(at + align256(4 * lay.rows));
  float* const dqacc = five ? reinterpret_cast<float*>(at + 2 * align256(4 * lay.rows)) : nullptr;
  int* const err = device_error_word();
  if (!err) return record_cuda_error(cudaErrorMemoryAllocation);

  // Operands that other tiles of a head read again: Q and dO of its G heads, K, V, (5-GEMM) the fp32 dQ.
  const double token_bytes = 2.0 * s.d * (2 * s.G() + 2) + (five ? 4.0 * KV::D * s.G() : 0.0);
  const int tokens = KV::BM / s.G();
  CUtensorMap maps[kPackedMaxMaps];
  PackedCut cuts[2] = {{KV::BN, KV::DSPLIT * qsplit, token_bytes}, {}};
  fa_status e;
  if ((e = packed_query_map(&maps[0], c.q, s, tokens)) != FA_OK) return e;
  if ((e = packed_query_map(&maps[1], c.dO, s, tokens)) != FA_OK) return e;
  if ((e = packed_key_map(&maps[2], c.k, s, KV::BN)) != FA_OK) return e;
  if ((e = packed_key_map(&maps[3], c.v, s, KV::BN)) != FA_OK) return e;
  if constexpr (!five) {
    if ((e = packed_key_map(&maps[4], c.k, s, Q::BN)) != FA_OK) return e;
    if ((e = packed_key_map(&maps[5], c.v, s, Q::BN)) != FA_OK) return e;
    cuts[1] = {128 / s.G(), Q::DQS, 4.0 * s.d};
  }
  const long long sms = sm_count_cached();
  RaggedPreParams pre = {packed_plan_params(plan, c.cu, s, cuts, lay.cuts, maps, lay.nmaps, 2)};
  pre.plan_blocks = s.B > 0 ? 1 + packed_map_blocks(s.B, lay.nmaps, 256) : 0;
  pre.tiles = {c.cu, s.B, s.T, s.H, s.Hkv, s.G(), tokens, KV::BM, lay.slots, s.d,
               (65536 + s.G() - 1) / s.G()};
  pre.o = in(c.o), pre.dO = in(c.dO);
  pre.lse = c.lse, pre.lse2 = lse2, pre.dd = dd, pre.dqacc = dqacc;
  pre.out[0] = out(c.dq), pre.out[1] = out(c.dk), pre.out[2] = out(c.dv);
  const unsigned blocks = (unsigned)std::min<long long>((long long)(lay.slots + 1) * s.Hkv, 4 * sms);
  if ((e = launch(FA_KERNEL_BWD_PRE, ragged_pre_kernel<DP>, dim3(pre.plan_blocks + blocks), dim3(256), 0, st, pre)) != FA_OK)
    return e;
  if (s.B == 0) return FA_OK;  // (every row is of no sequence)

  RaggedKVParams p;
  p.q_map = maps[0], p.do_map = maps[1], p.k_map = maps[2], p.v_map = maps[3];
  p.ends = plan.maps, p.nmaps = lay.nmaps, p.sched = plan.sched[0];
  p.v = in(c.v).data, p.v_token = c.v.token, p.v_head = c.v.head;
  p.lse2 = lse2, p.dd = dd, p.dqacc = dqacc;
  p.dk = out(c.dk).data, p.dk_token = c.dk.token, p.dk_head = c.dk.head;
  p.dv = out(c.dv).data, p.dv_token = c.dv.token, p.dv_head = c.dv.head;
  p.err = err, p.slots = lay.slots, p.Hkv = s.Hkv, p.G = s.G(), p.tokens = tokens, p.hd = s.d;
  p.scale_log2 = c.scale * kLog2e, p.scale = c.scale, p.causal = c.causal;
  p.qsplit = qsplit, p.T = s.T;
  p.dkpart = reinterpret_cast<float*>(static_cast<uint8_t*>(c.workspace) + lay.parts);
  p.dvpart = p.dkpart + (size_t)qsplit * s.Hkv * s.T * KV::D;
  const unsigned kv_grid =
      (unsigned)std::min<long long>(((long long)s.T / KV::BN + s.B) * s.Hkv * KV::DSPLIT * qsplit, sms);
  const int kind = five ? FA_KERNEL_BWD_KV5 : FA_KERNEL_BWD_KV7;
  if (qsplit == 1) {
    if ((e = launch_raised(kind, bwd_kv_kernel<KV, false, RaggedKVParams>, dim3(kv_grid), dim3(KV::THREADS), KV::SMEM_BYTES,
                           st, p, kv_raised)) != FA_OK)
      return e;
  } else {
    if ((e = launch_raised(kind, bwd_kv_kernel<KV, true, RaggedKVParams>, dim3(kv_grid), dim3(KV::THREADS), KV::SMEM_BYTES,
                           st, p, few_raised)) != FA_OK)
      return e;
    const RaggedKVSumParams sum = {p.dkpart, p.dvpart, out(c.dk), out(c.dv), c.cu, err, s.B, s.T, s.Hkv, s.d, KV::D, qsplit,
                                   c.scale};
    const long long threads = (long long)s.T * s.Hkv * (s.d / 8);
    if ((e = launch(FA_KERNEL_BWD_KVSUM, ragged_kvsum_kernel, dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, st,
                    sum)) != FA_OK)
      return e;
  }
  if constexpr (five) {
    RaggedConvParams conv = {pre.tiles, dqacc, out(c.dq), err, c.scale};
    return launch(FA_KERNEL_BWD_CONV, ragged_conv_kernel<KV::D>, dim3(blocks), dim3(256), 0, st, conv);
  } else {
    RaggedQParams r;
    if ((e = packed_query_map(&r.q_map, c.q, s, 128 / s.G())) != FA_OK) return e;
    if ((e = packed_query_map(&r.do_map, c.dO, s, 128 / s.G())) != FA_OK) return e;
    r.k_map = maps[4], r.v_map = maps[5];
    r.ends = plan.maps + 4, r.nmaps = lay.nmaps, r.sched = plan.sched[1];
    r.dO = in(c.dO).data, r.do_token = c.dO.token, r.do_head = c.dO.head;
    r.lse2 = lse2, r.dd = dd;
    r.dq = out(c.dq).data, r.dq_token = c.dq.token, r.dq_head = c.dq.head;
    r.err = err, r.slots = lay.slots, r.pre_tokens = tokens, r.pre_rows = KV::BM;
    r.Hkv = s.Hkv, r.G = s.G(), r.tokens = 128 / s.G(), r.hd = s.d;
    r.scale_log2 = c.scale * kLog2e, r.scale = c.scale, r.causal = c.causal;
    const unsigned q_grid = (unsigned)std::min<long long>(((long long)s.T / r.tokens + s.B) * s.Hkv * Q::DQS, sms);
    return launch_raised(FA_KERNEL_BWD_Q7, bwd_q_kernel<Q, false, RaggedQParams>, dim3(q_grid), dim3(Q::THREADS),
                         Q::SMEM_BYTES, st, r, q_raised);
  }
}

// Query rows of a tile of the dK/dV kernels.
int tile_rows(int d) { return d == 64 ? 128 : d == 384 ? 32 : 64; }
static_assert(KV5_64::BM == 128 && KV7_64::BM == 128 && KV5_128::BM == 64 && KV7_128::BM == 64 && KV7_192::BM == 64 &&
                  KV7_256::BM == 64 && KV7_384::BM == 32,
              "tile_rows");

}  // namespace

size_t packed_bwd_bytes(const PackedShape& s, int variant) {
  // (the kernels' D and DSPLIT: run below)
  const int D = s.d == 192 ? 192 : padded_head_dim(s.d);
  return BwdLayout(s, variant, tile_rows(s.d), D, D == 384 ? KV7_384::DSPLIT : D == 256 ? KV7_256::DSPLIT : 1).total;
}

fa_status run_packed_bwd(const fa_packed_bwd_args& a, const PackedShape& s, int form) {
  const bool five = form == FA_BWD_5GEMM;
  switch (s.d) {
    case 64: return five ? run<64, KV5_64, void>(a, s) : run<64, KV7_64, Q7_64>(a, s);
    case 96:
    case 128: return five ? run<128, KV5_128, void>(a, s) : run<128, KV7_128, Q7_128>(a, s);
    case 192: return run<256, KV7_192, Q7_192>(a, s);
    case 256: return run<256, KV7_256, Q7_256>(a, s);
    case 384: return run<384, KV7_384, Q7_384>(a, s);
  }
  return FA_ERR_UNSUPPORTED;
}

}  // namespace fa
