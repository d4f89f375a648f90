// Attention over the paged 4-bit cache for many query rows a kv head (several query
// tokens, large groups): the same mathematics and the same division of the units as
// kv4_attn.cuh, on tcgen05.
//
// With few rows the work per cached byte is its conversion, and mma.m16n8k16 keeps up.
// With many, tiles of 8 or 16 rows would convert every byte again for each tile, so here
// a block converts a unit once, into f16 operand tiles in shared memory, and 128 rows
// use it: S = Q K^T (A = Q from TMEM, or from shared memory at d = 384, where it does not
// fit next to O) and O += P V (A = P from TMEM, written over S), accumulators in TMEM.
//
//   warps 0-3    softmax: thread r owns row r (TMEM lane r) of the tile
//   warps 4-11   conversion: packed K and V of a unit to 128-byte-swizzled panels
//   warp 12      TMEM allocation and MMA issue, in the order S(0) S(1) PV(0) S(2) PV(1) ..
//   warps 13, 14 bulk copies of packed K and of V into a ring of staging slots
//
// A block takes an even share of the units of all (request, kv head, row tile) triples and
// leaves a part per cut triple, as a warp does there; kv4_merge_kernel joins them.
// What bounds it now, in cycles per 64 tokens at d = 128 (floors: reading 410, MMAs 510,
// exponentials 4 a row): the softmax warps, 1070 of work and 490 of hand-over between
// units; conversion takes 800 a tile beside it, and the MMA warp sees a probability tile
// 450 after it is written (clock64 stamps of an instrumented copy, which is not kept).
// 15 warps at 128 registers fill the register file, so d = 128, 192 and 256 spill 56, 4 and
// 24 bytes a thread.
#pragma once
#include "kv4_attn.cuh"

namespace fa {

// Instruction descriptor of kind::f16 with f16 A and B and fp32 D (make_idesc has bf16).
__host__ __device__ constexpr uint32_t make_idesc_f16(int M, int N, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// wait_warp for a warp that runs ahead of the others and mostly waits: it sleeps between
// its looks, so that its polling takes no issue slots from the softmax warp on its
// scheduler.
template <int NS>
__device__ __forceinline__ bool wait_asleep(uint32_t bar, uint32_t parity, const CtaAbort& ab, int where) {
  const long long t0 = clock64();
  while (true) {
    const bool ok = mbar_test(bar, parity);
    if (__all_sync(0xffffffffu, ok)) return true;
    // (Lanes agree on the end: one that left alone would leave the others in the vote.)
    const bool late = clock64() - t0 > kWaitLimitCycles;
    if (late) raise_timeout(ab, where);
    if (__any_sync(0xffffffffu, late || *ab.flag)) return false;
    __nanosleep(NS);
  }
}

template <int D_>
struct Kv4WideCfg {
  // Units of 32 tokens at d = 384, so that two operand slots each for K and V fit beside Q.
  static constexpr int D = D_, ROWS = 128, UNIT = D <= 256 ? 64 : 32;
  static constexpr int CONVERT = 8;  // warps
  static constexpr int MMA_WARP = 4 + CONVERT, COPY_WARP = MMA_WARP + 1, THREADS = 32 * (COPY_WARP + 2);
  static constexpr int CODE_ROW = D / 2, SCALE_ROW = D / 16;
  static constexpr int OFF_SCALE = UNIT * CODE_ROW, PART = UNIT * (CODE_ROW + SCALE_ROW);
  static constexpr int PANELS = (D + 63) / 64, PANEL = UNIT * 128;  // operand panels of 64 channels
  static constexpr int TILE = PANELS * PANEL;
  static constexpr bool QT = D <= 256;  // Q in TMEM
  static constexpr int Q_PANEL = ROWS * 128, Q_BYTES = QT ? 0 : PANELS * Q_PANEL;
  // Operand slots few, staging slots many: what is on its way has to cover memory's latency.
  static constexpr int TILES = D <= 128 ? 6 : 4;
  static constexpr int STAGED = D <= 128 ? 22 : D == 192 ? 16 : D == 256 ? 8 : 4;
  static constexpr int OFF_Q = TILES * TILE, OFF_STAGE = OFF_Q + Q_BYTES;
  static constexpr int OFF_BAR = OFF_STAGE + STAGED * PART;
  // Barriers: staging full and empty, operand full and empty, then S, P, O (two each), Q, done.
  static constexpr int B_SFULL = 0, B_SEMPTY = STAGED, B_TFULL = 2 * STAGED, B_TEMPTY = B_TFULL + TILES,
                       B_S = B_TEMPTY + TILES, B_P = B_S + 2, B_O = B_P + 2, B_Q = B_O + 2, B_DONE = B_Q + 1,
                       BARS = B_DONE + 1;
  static constexpr int OFF_PREFIX = OFF_BAR + BARS * 8;
  static constexpr int OFF_REQ = OFF_PREFIX + (THREADS + 1) * 8;
  static constexpr bool KEEP = D < 384;  // room for the requests
  static constexpr int OFF_BITS = OFF_REQ + (KEEP ? THREADS * 16 : 0);  // a byte for each of the last 32 units
  static constexpr int OFF_MISC = OFF_BITS + 32;
  static constexpr int SMEM = OFF_MISC + 16 + THREADS / 32 * 8 + 1024;  // and the tiles' alignment
  // O has a column for every channel of the panels: at d = 96 the last 32 are never read.
  static constexpr int OD = PANELS * 64;
  static constexpr int TMEM_S = 0, TMEM_O = 2 * UNIT, TMEM_Q = TMEM_O + OD;
  static constexpr int NPV = (OD + 255) / 256, PVN = OD / NPV;  // O += P V as NPV MMAs
  static_assert(TMEM_Q + (QT ? D / 2 : 0) <= 512 && SMEM <= 232448 && OFF_REQ % 8 == 0 && OFF_MISC % 8 == 0, "budgets");
  static_assert((STAGED + TILES) / 2 + 4 < 32, "units in flight");
  // Slots belong to K or to V: a slot that alternated between the warps that convert them
  // would let each miss every other phase of its barrier, which a parity cannot tell.
  static_assert(TILES % 2 == 0 && STAGED % 2 == 0, "even rings");
};

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1) kv4_wide_kernel(const __grid_constant__ Kv4AttnParams p) {
  constexpr int D = C::D, UNIT = C::UNIT;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  const int warp = warp_id(), lane = lane_id();
  long long* prefix = reinterpret_cast<long long*>(smem + C::OFF_PREFIX);
  int* kept = C::KEEP ? reinterpret_cast<int*>(smem + C::OFF_REQ) : nullptr;
  volatile uint8_t* unit_bits = smem + C::OFF_BITS;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC + 4);
  long long* sums = reinterpret_cast<long long*>(smem + C::OFF_MISC + 16);
  auto BAR = [&](int i) -> uint32_t { return base + C::OFF_BAR + 8u * (uint32_t)i; };

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int s = 0; s < C::STAGED; ++s) mbar_init(BAR(C::B_SFULL + s), 1), mbar_init(BAR(C::B_SEMPTY + s), C::CONVERT / 2);
    for (int s = 0; s < C::TILES; ++s) mbar_init(BAR(C::B_TFULL + s), C::CONVERT / 2), mbar_init(BAR(C::B_TEMPTY + s), 1);
    for (int b = 0; b < 2; ++b) mbar_init(BAR(C::B_S + b), 1), mbar_init(BAR(C::B_P + b), 4), mbar_init(BAR(C::B_O + b), 1);
    mbar_init(BAR(C::B_Q), 4);
    mbar_init(BAR(C::B_DONE), 1);
    fence_mbar_init();
  }
  if (warp == C::MMA_WARP) {
    tmem_alloc(smem_u32(tmem_holder), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const CtaAbort ab{abort_flag, p.err};
  grid_dep_wait();
  const bool skip = *reinterpret_cast<volatile int*>(p.err) != 0;
  const long long total = kv4_scan<C>(p, prefix, kept, sums);
  const int* req = p.B <= C::THREADS ? kept : nullptr;
  const int me = blockIdx.x;
  const Kv4Share share(total, gridDim.x, me);
  Kv4Cursor cur;
  const int units = !skip && share.units > 0 && kv4_locate<C>(p, prefix, req, share.x0, cur) ? share.units : 0;
  // The units of the cursor's triple that lie in this block's share, and the next triple.
  auto run_of = [&](int left) -> int { return min(cur.units - cur.u, left); };
  auto skip_run = [&](int n) {
    cur.u += n - 1;
    kv4_advance<C>(p, req, cur);
  };
  const int fr_log2 = min(p.page_log2, UNIT == 64 ? 6 : 5);

  if (warp >= C::COPY_WARP) {
    // ------------------------------------------------------------------ copies
    // One warp copies K, the other V.  The page ids are read AHEAD units before their
    // copies; `cur` runs that far ahead.
    const int kv = warp - C::COPY_WARP;
    const int frag = lane >> 1;
    const int row_bytes = (lane & 1) ? C::SCALE_ROW : C::CODE_ROW;
    const uint32_t copy_bytes = (uint32_t)row_bytes << fr_log2;
    const uint32_t copy_dst = base + C::OFF_STAGE + ((lane & 1) ? C::OFF_SCALE : 0) + frag * copy_bytes;
    const uint8_t* const array = (lane & 1) ? p.scales[kv] : p.codes[kv];
    constexpr int AHEAD = 4;
    int ids[AHEAD], heads[AHEAD], firsts[AHEAD], left = units;
    auto look_up = [&](int k) {
      ids[k] = -1;
      heads[k] = cur.kvh;
      firsts[k] = cur.u * UNIT + (frag << fr_log2);
      if (left <= 0) return;
      const int col = firsts[k] >> p.page_log2;
      if (frag < (UNIT >> fr_log2) && firsts[k] < cur.n && col < p.width) ids[k] = p.table[(size_t)cur.b * p.width + col];
      if (--left > 0) kv4_advance<C>(p, req, cur);
    };
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) look_up(k);
    int issued = 0, slot = kv;
    uint32_t parity = 1;
    bool ok = true;
    for (int u0 = 0; u0 < units && ok; u0 += AHEAD) {
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        const int u = u0 + k;
        if (u >= units || !ok) break;
        const int id = (unsigned)ids[k] < (unsigned)p.pages ? ids[k] : -1;
        const uint32_t have = __ballot_sync(0xffffffffu, id >= 0 && !(lane & 1));
        const uint32_t bits = (have & 1u) | ((have >> 1) & 2u) | ((have >> 2) & 4u) | ((have >> 3) & 8u);
        const uint8_t* src =
            array + ((((long long)id * p.Hkv + heads[k]) << p.page_log2) + (firsts[k] & ((1 << p.page_log2) - 1))) * row_bytes;
        look_up(k);
        if (!wait_asleep<200>(BAR(C::B_SEMPTY + slot), parity, ab, (kKKv4 << 8) | 8)) {
          ok = false;
          break;
        }
        const uint32_t bar = BAR(C::B_SFULL + slot);
        if (lane == 0) {
          if (kv == 0) unit_bits[u & 31] = (uint8_t)bits;
          mbar_expect_tx(bar, (uint32_t)(__popc(bits) << fr_log2) * (C::CODE_ROW + C::SCALE_ROW));
        }
        __syncwarp();
        if (id >= 0) bulk_load(copy_dst + slot * C::PART, src, copy_bytes, bar);
        ++issued;
        if ((slot += 2) >= C::STAGED) {
          slot = kv;
          parity ^= 1;
        }
      }
    }
    // Every copy lands before the block can exit.
    constexpr int OWN = C::STAGED / 2;
    for (int i = max(issued - OWN, 0); i < issued; ++i)
      wait_done(BAR(C::B_SFULL + 2 * (i % OWN) + kv), (uint32_t)((i / OWN) & 1));
  } else if (warp == C::MMA_WARP) {
    // --------------------------------------------------------------------- MMAs
    constexpr uint32_t idS = make_idesc_f16(128, UNIT, false);
    constexpr uint32_t idO = make_idesc_f16(128, C::PVN, true);
    // One warp's instructions pace the block here, so the loops run on uniform registers:
    // their bounds come out of a warp reduction (which the compiler knows to be uniform), the
    // slots are counted instead of divided out, and the descriptors differ by additions.
    auto uniform = [](int x) -> int { return (int)__reduce_max_sync(0xffffffffu, (unsigned)x); };
    const uint64_t k_desc = desc_kmajor(base, C::PANEL, 0), v_desc = desc_mnmajor(base, C::PANEL, 0);
    const uint64_t q_desc = desc_kmajor(base + C::OFF_Q, C::Q_PANEL, 0);
    bool ok = true;
    int g = 0;  // the unit of the next PV; S runs one ahead
    int k_slot = 0, v_slot = 1;
    uint32_t k_phase = 0, v_phase = 0;
    auto issue_s = [&](int buffer) -> bool {
      if (!wait_warp(BAR(C::B_TFULL + k_slot), k_phase, ab, (kKKv4 << 8) | 9)) return false;
      tc_fence_after();
      const uint64_t kd = sdesc_advance(k_desc, (uint32_t)k_slot * (C::TILE >> 4));
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        // 16 channels on: 32 bytes in a panel row, or the next panel.
        const uint64_t b = sdesc_advance(kd, (uint32_t)((k >> 2) * C::PANEL + (k & 3) * 32) >> 4);
        if constexpr (C::QT)
          mma_ts(tmem + C::TMEM_S + buffer * UNIT, tmem + C::TMEM_Q + 8 * k, b, idS, k > 0 ? 1u : 0u);
        else
          mma_ss(tmem + C::TMEM_S + buffer * UNIT,
                 sdesc_advance(q_desc, (uint32_t)((k >> 2) * C::Q_PANEL + (k & 3) * 32) >> 4), b, idS, k > 0 ? 1u : 0u);
      }
      mma_commit(BAR(C::B_S + buffer));  // (the softmax warps hand K's slot back)
      if ((k_slot += 2) >= C::TILES) {
        k_slot = 0;
        k_phase ^= 1;
      }
      return true;
    };
    int triple = 0;
    for (int left = uniform(units); left > 0 && ok; ++triple) {
      const int n = uniform(run_of(left));
      left -= n;
      if (left > 0) skip_run(n);
      ok = wait_warp(BAR(C::B_Q), triple & 1, ab, (kKKv4 << 8) | 10);
      if (ok) tc_fence_after();
      ok = ok && issue_s(g & 1);
      for (int j = 0; j < n && ok; ++j, ++g) {
        const int buffer = g & 1;
        if (j + 1 < n && !(ok = issue_s(buffer ^ 1))) break;
        ok = wait_warp(BAR(C::B_P + buffer), (g >> 1) & 1, ab, (kKKv4 << 8) | 11) &&
             wait_warp(BAR(C::B_TFULL + v_slot), v_phase, ab, (kKKv4 << 8) | 12);
        if (!ok) break;
        tc_fence_after();
        const uint64_t vd = sdesc_advance(v_desc, (uint32_t)v_slot * (C::TILE >> 4));
#pragma unroll
        for (int k = 0; k < UNIT / 16; ++k)
#pragma unroll
          for (int c = 0; c < C::NPV; ++c)
            mma_ts(tmem + C::TMEM_O + c * C::PVN, tmem + C::TMEM_S + buffer * UNIT + 8 * k,
                   sdesc_advance(vd, (uint32_t)(c * (C::PVN / 64) * C::PANEL + k * 2048) >> 4), idO,
                   (j > 0 || k > 0) ? 1u : 0u);
        mma_commit(BAR(C::B_O + buffer));
        mma_commit(BAR(C::B_TEMPTY + v_slot));
        if ((v_slot += 2) >= C::TILES) {
          v_slot = 1;
          v_phase ^= 1;
        }
      }
    }
    // Every MMA issued above finishes before TMEM is released.
    mma_commit(BAR(C::B_DONE));
    wait_done(BAR(C::B_DONE), 0);
    __syncwarp();
  } else if (warp >= 4) {
    // --------------------------------------------------------------- conversion
    // An item is 16 packed bytes of a token, 32 channels: four 16-byte chunks of half a
    // panel row.  Lanes take neighbouring bytes, and the order in which a lane writes its
    // chunks depends on its panel, so that eight lanes write eight chunk positions.
    // Half of the warps convert K, the others V, so that the latencies of the two overlap.
    constexpr int NQ = D / 32, ITEMS = UNIT * NQ, T = 16 * C::CONVERT;
    const int tid = (threadIdx.x - 128) % T;
    int stage = (threadIdx.x - 128) / T, tile = stage;
    uint32_t stage_phase = 0, tile_parity = 1;
    for (int u = 0; u < units; ++u) {
      if (!wait_asleep<20>(BAR(C::B_SFULL + stage), stage_phase, ab, (kKKv4 << 8) | 13)) break;
      if (!wait_asleep<20>(BAR(C::B_TEMPTY + tile), tile_parity, ab, (kKKv4 << 8) | 14)) break;
      const uint8_t* src = smem + C::OFF_STAGE + stage * C::PART;
      uint8_t* dst = smem + tile * C::TILE;
      // (All of a thread's reads first: the compiler cannot move them over the writes.)
      constexpr int MINE = (ITEMS + T - 1) / T;
      uint4 packed[MINE];
      uint32_t scale[MINE];
#pragma unroll
      for (int k = 0; k < MINE; ++k) {
        const int it = min(tid + k * T, ITEMS - 1);
        const int tok = it / NQ, q = it - tok * NQ;
        packed[k] = *reinterpret_cast<const uint4*>(src + tok * C::CODE_ROW + q * 16);
        scale[k] = *reinterpret_cast<const uint16_t*>(src + C::OFF_SCALE + tok * C::SCALE_ROW + 2 * q);
      }
#pragma unroll
      for (int k0 = 0; k0 < MINE; ++k0) {
        const int it = tid + k0 * T;
        if (it >= ITEMS) break;
        const int tok = it / NQ, q = it - tok * NQ;
        const uint4 c = packed[k0];
        uint32_t s0 = kv4_scale_both(scale[k0]), s1 = kv4_scale_both(scale[k0] >> 8);
        const int turn = NQ == 4 ? 2 * (q >> 1) : (q >> 1) & 3;
        uint32_t w[4] = {c.x, c.y, c.z, c.w};
        if (turn & 2) {
          uint32_t x = w[0];
          w[0] = w[2], w[2] = x;
          x = w[1], w[1] = w[3], w[3] = x;
          x = s0, s0 = s1, s1 = x;
        }
        if (NQ != 4 && (turn & 1)) {
          uint32_t x = w[0];
          w[0] = w[1], w[1] = x;
          x = w[2], w[2] = w[3], w[3] = x;
        }
        uint8_t* row = dst + (q >> 1) * C::PANEL + tok * 128;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t r[4];
          kv4_codes(w[k], r);
          const uint32_t s = k < 2 ? s0 : s1;
          const int chunk = (4 * (q & 1) + (k ^ turn)) ^ (tok & 7);
          *reinterpret_cast<uint4*>(row + chunk * 16) =
              make_uint4(h2mul(r[0], s), h2mul(r[1], s), h2mul(r[2], s), h2mul(r[3], s));
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(BAR(C::B_TFULL + tile));
        mbar_arrive(BAR(C::B_SEMPTY + stage));
      }
      if ((stage += 2) >= C::STAGED) {
        stage -= C::STAGED;
        stage_phase ^= 1;
      }
      if ((tile += 2) >= C::TILES) {
        tile -= C::TILES;
        tile_parity ^= 1;
      }
    }
  } else {
    // ------------------------------------------------------------------ softmax
    const int r = threadIdx.x;
    const uint32_t trow = tmem + ((uint32_t)(warp * 32) << 16);
    const uint32_t all_bits = (1u << (UNIT >> fr_log2)) - 1u;
    // Query row r of the cursor's triple as f16, scaled by a power of two into f16's range
    // (zeros past the last row); returns the factor that takes scores to the log2 domain.
    auto exponent = [](uint32_t top) -> int { return min(max((int)(top >> 7) - 127, -120), 120); };
    auto write_q = [&]() -> float {
      const int row = cur.rt * C::ROWS + r;
      const int i = row / p.G, h = row - i * p.G;
      const bool have = i < cur.nq;
      const uint4* src = reinterpret_cast<const uint4*>(p.q + (long long)(cur.tok0 + (have ? i : 0)) * p.q_token +
                                                        (long long)(cur.kvh * p.G + h) * p.q_head);
      // CH channels at a time with all their loads in flight: the whole row where the registers
      // hold it, else twice, first for the largest magnitude (as bf16 bits), which gives the
      // power of two.
      constexpr int CH = D <= 128 ? D : D == 192 ? 96 : 128, N = CH / 8, ONCE = CH == D;
      uint32_t top = 0;
#pragma unroll 1
      for (int c0 = 0; c0 < (ONCE ? D : 2 * D); c0 += CH) {
        const int c = c0 < D ? c0 : c0 - D;
        uint4 x[N];
#pragma unroll
        for (int u = 0; u < N; ++u) x[u] = have ? src[c / 8 + u] : make_uint4(0u, 0u, 0u, 0u);
        if (c0 < D) {
#pragma unroll
          for (int u = 0; u < N; ++u) {
            const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) top = max(top, max(w[k] & 0x7fffu, (w[k] >> 16) & 0x7fffu));
          }
          if (!ONCE) continue;
        }
        const float down = __uint_as_float((uint32_t)(127 - exponent(top)) << 23);
        uint32_t qw[4 * N];
#pragma unroll
        for (int u = 0; u < N; ++u) {
          const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
          for (int k = 0; k < 4; ++k)
            qw[4 * u + k] = pack_f16(__uint_as_float(w[k] << 16) * down, __uint_as_float(w[k] & 0xffff0000u) * down);
        }
        if constexpr (C::QT) {
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 4 * N; k += 32) {
            if (4 * N - k >= 32)
              tmem_st_32x32b_x32(trow + C::TMEM_Q + (c >> 1) + k, qw + k);
            else
              tmem_st_32x32b_x16(trow + C::TMEM_Q + (c >> 1) + k, qw + k);
          }
        } else {
#pragma unroll
          for (int u = 0; u < N; ++u) {
            const int chunk = c / 8 + u;
            *reinterpret_cast<uint4*>(smem + C::OFF_Q + (chunk >> 3) * C::Q_PANEL + r * 128 + ((chunk & 7) ^ (r & 7)) * 16) =
                make_uint4(qw[4 * u], qw[4 * u + 1], qw[4 * u + 2], qw[4 * u + 3]);
          }
        }
      }
      if constexpr (C::QT) {
        tmem_wait_st();
        tc_fence_before();
      } else {
        fence_proxy_async_smem();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(C::B_Q));
      return kv4_score_factor(p, exponent(top));
    };
    // O with unit u added.  S runs one unit ahead, so a barrier for every other unit cannot
    // be two phases ahead of its waiter.
    auto wait_o = [&](int u) -> bool {
      return wait_warp(BAR(C::B_O + (u & 1)), (u >> 1) & 1, ab, (kKKv4 << 8) | 16);
    };
    float fac = units > 0 ? write_q() : 0.f;
    int g = 0;
    long long began = share.x0 - cur.u;
    bool ok = true;
    for (int left = units; left > 0 && ok;) {
      const int n = run_of(left);
      left -= n;
      // This row, and the triple, which the cursor leaves before the row is written.
      const int rt = cur.rt, kvh = cur.kvh, tok0 = cur.tok0, nq = cur.nq, u0 = cur.u, triple_units = cur.units;
      const long long triple = ((long long)cur.b * p.Hkv + kvh) * p.row_tiles + rt;
      const int row = rt * C::ROWS + r;
      const int i = row / p.G, h = kvh * p.G + row - i * p.G;
      const bool have = i < nq;
      const bool busy = __any_sync(0xffffffffu, have);  // a warp past the last row only keeps pace
      // (A row past the last sees everything: its zeros cost no masking, and are not stored.)
      const int lim = have ? cur.first + i : 0x7fffffff;
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < n; ++j, ++g) {
        const uint32_t tS = trow + C::TMEM_S + (g & 1) * UNIT;
        if (!wait_warp(BAR(C::B_S + (g & 1)), (g >> 1) & 1, ab, (kKKv4 << 8) | 15)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (threadIdx.x == 0) mbar_arrive(BAR(C::B_TEMPTY + (2 * g) % C::TILES));
        if (busy) {
          uint32_t sr[UNIT];
          tmem_ld_32x32b_x32(tS, sr);
          if constexpr (UNIT == 64) tmem_ld_32x32b_x32(tS + 32, sr + 32);
          tmem_wait_ld();
          reg_fence<UNIT>(sr);
          const uint32_t bits = unit_bits[g & 31];
          const int key0 = (u0 + j) * UNIT;
          if (key0 + UNIT - 1 > lim || bits != all_bits) {
#pragma unroll
            for (int c = 0; c < UNIT; ++c)
              if (key0 + c > lim || !((bits >> (c >> fr_log2)) & 1u)) sr[c] = __float_as_uint(-INFINITY);
          }
          __syncwarp();
          float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
          for (int c = 0; c < UNIT; c += 4) {
            mx0 = max3(mx0, __uint_as_float(sr[c]), __uint_as_float(sr[c + 1]));
            mx1 = max3(mx1, __uint_as_float(sr[c + 2]), __uint_as_float(sr[c + 3]));
          }
          const float high = fmaxf(mx0, mx1) * fac - kKv4Lift;
          const bool grow = high > m + kKv4Grow;
          const float alpha = grow ? ex2(m - high) : 1.f;
          if (grow) m = high;
          l *= alpha;
          const float msub = m == -INFINITY ? 0.f : m;
          float la = 0.f, lb = 0.f;
          uint32_t pk[UNIT / 2];
#pragma unroll
          for (int c = 0; c < UNIT; c += 2) {
            const float a = ex2(fmaf(__uint_as_float(sr[c]), fac, -msub));
            const float b = ex2(fmaf(__uint_as_float(sr[c + 1]), fac, -msub));
            la += a;
            lb += b;
            pk[c >> 1] = pack_f16(a, b);
          }
          l += la + lb;
          if constexpr (UNIT == 64)
            tmem_st_32x32b_x32(tS, pk);
          else
            tmem_st_32x32b_x16(tS, pk);
          tmem_wait_st();
          if (j > 0 && __any_sync(0xffffffffu, grow)) {
            // The running O, once the MMA that added to it last is done.
            if (!wait_o(g - 1)) {
              ok = false;
              break;
            }
            tc_fence_after();
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 32) {
              uint32_t o[32];
              tmem_ld_32x32b_x32(trow + C::TMEM_O + c0, o);
              tmem_wait_ld();
              reg_fence<32>(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tmem_st_32x32b_x32(trow + C::TMEM_O + c0, o);
            }
            tmem_wait_st();
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(C::B_P + (g & 1)));
      }
      if (!ok) break;
      // The triple's last S is done with Q: the next triple's, while its last PV runs.
      if (left > 0) {
        skip_run(n);
        fac = write_q();
      }
      if (!wait_o(g - 1)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const bool first_here = began >= share.x0;
      const bool direct = first_here && u0 + n == triple_units;
      if (first_here && threadIdx.x == 0)
        p.cuts[triple] =
            make_int2(me, direct ? 0 : share.parts(me, (int)(began + triple_units - (share.x0 + units))));
      // Slot 1: the triple begins in this share and goes on; slot 0: it began before.
      const size_t part = ((size_t)me * 2 + (first_here ? 1 : 0)) * C::ROWS + r;
      const float inv = direct ? (l == 0.f ? 0.f : p.v_gain / l) : 1.f;
      if (busy) {
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 32) {
          uint32_t o[32];
          tmem_ld_32x32b_x32(trow + C::TMEM_O + c0, o);
          tmem_wait_ld();
          reg_fence<32>(o);
          if (have && direct) {
            uint4* dst =
                reinterpret_cast<uint4*>(p.o + (long long)(tok0 + i) * p.o_token + (long long)h * p.o_head + c0);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t x[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                x[e] = pack_bf16(__uint_as_float(o[8 * k + 2 * e]) * inv, __uint_as_float(o[8 * k + 2 * e + 1]) * inv);
              dst[k] = make_uint4(x[0], x[1], x[2], x[3]);
            }
          } else if (have) {
            uint4* dst = reinterpret_cast<uint4*>(p.part_o + part * D + c0);
#pragma unroll
            for (int k = 0; k < 8; ++k) dst[k] = make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
          }
          __syncwarp();
        }
        if (have) {
          if (direct)
            p.lse[(long long)(tok0 + i) * p.H + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
          else
            *reinterpret_cast<float2*>(p.part_ml + part * 2) = make_float2(m, l);
        }
      }
      began += triple_units;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == C::MMA_WARP) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace fa
