// Attention of a few query tokens per request over the paged 4-bit cache.
//
// Per request b and kv head, the R = n_q * (H/Hkv) query rows that share the
// cached head are cut into tiles of 8*NT rows, and the tokens into units of UNIT.
// All units of all (request, kv head, row tile) triples, laid end to end, are
// shared out evenly over the warps of the grid: warp w takes units
// [w*T/W, (w+1)*T/W), whatever requests they belong to, so ragged batches and one
// long request load the SMs alike, and no warp waits for another.  A triple that
// lies in one warp's range is finished there; one that is cut leaves a part
// (unnormalised fp32 O, running maximum m, sum l) per warp for kv4_merge_kernel.
//
// One unit: its K and V codes and scales (UNIT*d*1.125 bytes) come by bulk copies
// into the warp's own ring of STAGES slots; both products run on mma.m16n8k16 with
// f16 operands and fp32 accumulators, from registers:
//   S^T = K Q^T : A = 16 tokens x 16 channels, dequantised in registers (exact in
//                 f16), B = Q rows (f16; each row scaled by a power of two into
//                 f16's range, which its score factor takes back)
//   O^T += V^T P^T : A = 16 channels x 16 tokens; the codes of two tokens are
//                 interleaved before conversion, so each f16 pair is one channel at
//                 two tokens; B = P, transposed by movmatrix from S^T's layout
// K's channels and V's channels are dealt to lanes so that every lane reads
// contiguous bytes: the order of a contraction's terms is free, and O's channel
// order is undone at the store.
//
// Reading the cache bounds it in principle; the work per byte is what needs care:
// converting a code costs half a conversion (64 a cycle and SM) and half an f16
// multiplication.  The legacy tensor path (1024 f16 MACs a cycle and SM, measured)
// is enough for 8 rows a tile at full bandwidth (about 335 needed), and takes its
// operands from the registers where the codes are converted; tcgen05 would need
// them written to shared memory or TMEM first, in tiles of 128 rows of which a
// decoding step fills 1 to 16.
#pragma once
#include "kv4.cuh"

namespace fa {

struct Kv4AttnParams {
  const uint16_t* q;
  uint16_t* o;
  float* lse;
  const uint8_t* codes[2];   // K, V
  const uint8_t* scales[2];
  const int* table;
  const int* lengths;
  const int* cu;  // NULL: one query a request
  float* part_o;   // [W][2][8*NT][D]
  float* part_ml;  // [W][2][8*NT][2]
  int2* meta;      // [B*Hkv*row_tiles]: first warp of a cut triple and its number of parts (0: not cut)
  int* err;
  long long q_token, q_head, o_token, o_head;
  int B, H, Hkv, G, T, width, pages, page_log2, max_q;
  int row_tiles;  // most row tiles of a request
  int unit, rows;  // tokens of a unit and rows of a tile
  float score;    // scale * log2(e) * k_gain * 2^8
  float v_gain;   // v_gain * 2^8
};

// P is kept times 2^7 (m is the maximum less 7), and the maximum is only renewed
// when it grew by more than 8: p <= 2^15 fits f16, and what f16 flushes lies
// 2^-32 below the largest.
constexpr float kKv4Lift = 7.f;
constexpr float kKv4Grow = 8.f;

template <int D_, int NT_>
struct Kv4Cfg {
  static constexpr int D = D_, NT = NT_;
  static constexpr int ROWS = 8 * NT;
  static constexpr int UNIT = D <= 128 ? 64 : 32;
  static constexpr int MT = UNIT / 16;
  static constexpr int WARPS = 8;
  static constexpr int CODE_ROW = D / 2, SCALE_ROW = D / 16;  // bytes a token
  static constexpr int STAGE = 2 * UNIT * (CODE_ROW + SCALE_ROW);
  static constexpr int FIT = (224 * 1024 - 4096) / (WARPS * STAGE);
  static constexpr int STAGES = FIT < 4 ? FIT : 4;
  static constexpr int OFF_KS = UNIT * CODE_ROW, OFF_V = OFF_KS + UNIT * SCALE_ROW, OFF_VS = OFF_V + UNIT * CODE_ROW;
  static constexpr int OFF_BAR = WARPS * STAGES * STAGE;
  static constexpr int OFF_PREFIX = OFF_BAR + WARPS * STAGES * 8;
  static constexpr int THREADS = 32 * WARPS;
  static constexpr int OFF_MISC = OFF_PREFIX + (THREADS + 1) * 8;
  static constexpr int SMEM = OFF_MISC + 16 + WARPS * 8;
  static constexpr int WK = D / 32;         // words of 8 codes a lane reads of a K row
  static constexpr int WV = (D + 63) / 64;  // words a lane reads of a V row (d = 96: one and a half)
  static constexpr bool HALF = D % 64 != 0;
  static constexpr int CT = D / 16;  // O^T tiles of 16 channels
  static_assert(STAGES >= 2, "shared memory");
};

// A position in the sequence of units.
struct Kv4Cursor {
  int b, kvh, rt, u;      // request, kv head, row tile, unit
  int units, tiles;       // units and row tiles of request b
  int n, tok0, nq;        // tokens of b, its first query token, its queries
};

__device__ __forceinline__ void kv4_request(const Kv4AttnParams& p, int b, int unit, int rows, Kv4Cursor& c) {
  c.n = max(p.lengths[b], 0);
  if (p.cu) {
    c.tok0 = p.cu[b];
    const long long nq = (long long)p.cu[b + 1] - c.tok0;
    c.nq = (int)min(max(nq, 0LL), (long long)p.max_q);
    if (c.tok0 < 0 || c.tok0 > p.T - c.nq) c.nq = 0;  // queries outside q: not computed
  } else {
    c.tok0 = b;
    c.nq = 1;
  }
  c.tiles = (int)(((long long)c.nq * p.G + rows - 1) / rows);
  // Tokens past the table's width are no keys.
  const long long held = min((long long)c.n, (long long)p.width << p.page_log2);
  c.units = c.tiles ? max((int)((held + unit - 1) / unit), 1) : 0;
}

__device__ __forceinline__ void kv4_advance(const Kv4AttnParams& p, int unit, int rows, Kv4Cursor& c) {
  if (++c.u < c.units) return;
  c.u = 0;
  if (++c.rt < c.tiles) return;
  c.rt = 0;
  if (++c.kvh < p.Hkv) return;
  c.kvh = 0;
  do {
    if (++c.b >= p.B) {  // past the last unit (only if the lengths changed meanwhile): nothing to do there
      c.b = p.B - 1;
      c.n = c.nq = 0;
      c.units = c.tiles = 1;
      return;
    }
    kv4_request(p, c.b, unit, rows, c);
  } while (c.units == 0);
}

// Bounded wait for a copy in flight that does not give up early on an abort.
__device__ __forceinline__ void wait_done(uint32_t bar, uint32_t parity) {
  const long long t0 = clock64();
  while (!mbar_test(bar, parity))
    if (clock64() - t0 > kWaitLimitCycles) return;
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

__device__ __forceinline__ void mma_f16(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// N consecutive words of shared memory by the widest loads their alignment allows.
template <int N>
__device__ __forceinline__ void lds_words(const uint8_t* s, uint32_t* w) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const uint4 x = *reinterpret_cast<const uint4*>(s + 4 * i);
      w[i] = x.x, w[i + 1] = x.y, w[i + 2] = x.z, w[i + 3] = x.w;
    }
  } else if constexpr (N % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const uint2 x = *reinterpret_cast<const uint2*>(s + 4 * i);
      w[i] = x.x, w[i + 1] = x.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = *reinterpret_cast<const uint32_t*>(s + 4 * i);
  }
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1) kv4_attn_kernel(const __grid_constant__ Kv4AttnParams p) {
  constexpr int D = C::D, NT = C::NT, UNIT = C::UNIT, MT = C::MT, S = C::STAGES, WK = C::WK, WV = C::WV;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = warp_id(), lane = lane_id();
  const int g = lane >> 2, t = lane & 3;
  long long* prefix = reinterpret_cast<long long*>(smem + C::OFF_PREFIX);  // units before thread i's requests
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC);
  long long* sums = reinterpret_cast<long long*>(smem + C::OFF_MISC + 16);
  const uint32_t bar0 = smem_u32(smem + C::OFF_BAR) + warp * S * 8;
  uint8_t* ring = smem + warp * S * C::STAGE;
  const uint32_t ring_addr = smem_u32(ring);

  if (threadIdx.x == 0) *abort_flag = 0;
  if (lane == 0) {
    for (int s = 0; s < S; ++s) mbar_init(bar0 + 8 * s, 1);
    fence_mbar_init();
  }
  grid_dep_wait();
  const bool skip = *reinterpret_cast<volatile int*>(p.err) != 0;

  // Units before each thread's run of ceil(B / THREADS) requests, and in all.
  const int run = (p.B + C::THREADS - 1) / C::THREADS;
  {
    const int b0 = min((int)threadIdx.x * run, p.B), b1 = min(b0 + run, p.B);
    long long sum = 0;
    for (int b = b0; b < b1; ++b) {
      Kv4Cursor c;
      kv4_request(p, b, UNIT, C::ROWS, c);
      sum += (long long)c.units * c.tiles * p.Hkv;
    }
    long long x = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x += y;
    }
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    long long before = 0, total = 0;
    for (int w = 0; w < C::WARPS; ++w) {
      if (w < warp) before += sums[w];
      total += sums[w];
    }
    prefix[threadIdx.x] = before + x - sum;
    if (threadIdx.x == 0) prefix[C::THREADS] = total;
  }
  __syncthreads();
  if (skip) return;
  const CtaAbort ab{abort_flag, p.err};
  const long long total = prefix[C::THREADS];
  // Neighbouring ranges go to different SMs, so that few units spread over all.
  const int workers = (int)min((long long)gridDim.x * C::WARPS, total);
  const int me = warp * gridDim.x + blockIdx.x;
  if (me >= workers) return;
  const long long x0 = total * me / workers, x1 = total * (me + 1) / workers;
  auto worker_of = [&](long long x) -> int { return (int)(((x + 1) * workers - 1) / total); };

  // Where unit x0 lies.
  Kv4Cursor cur;
  {
    int lo = 0, hi = C::THREADS;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (prefix[mid] <= x0) lo = mid;
      else hi = mid;
    }
    long long rest = x0 - prefix[lo];
    cur.b = lo * run;
    for (;; ++cur.b) {
      if (cur.b >= p.B) return;
      kv4_request(p, cur.b, UNIT, C::ROWS, cur);
      const long long mine = (long long)cur.units * cur.tiles * p.Hkv;
      if (rest < mine) break;
      rest -= mine;
    }
    const long long seg = rest / cur.units;
    cur.u = (int)(rest - seg * cur.units);
    cur.kvh = (int)(seg / cur.tiles);
    cur.rt = (int)(seg - (long long)cur.kvh * cur.tiles);
  }

  // ------------------------------------------------------------- producer side
  // A unit is UNIT / FR fragments of FR = min(page, UNIT) tokens, each inside one
  // page: lane 4*f + a copies array a (K codes, K scales, V codes, V scales) of
  // fragment f, so all of a unit's copies are issued at once.
  const int fr_log2 = min(p.page_log2, UNIT == 64 ? 6 : 5);
  const int frags = UNIT >> fr_log2;
  Kv4Cursor pre = cur;  // the next unit to copy; its page id is read one unit ahead
  long long pre_x = x0;
  const int frag = lane >> 2, array = lane & 3;
  auto page_of = [&](const Kv4Cursor& c) -> int {
    const long long tok = (long long)c.u * UNIT + ((long long)frag << fr_log2);
    if (frag >= frags || tok >= c.n) return -1;
    const long long col = tok >> p.page_log2;
    if (col >= p.width) return -1;
    const int id = p.table[(size_t)c.b * p.width + col];
    return (unsigned)id < (unsigned)p.pages ? id : -1;
  };
  int next_page = page_of(pre);
  uint32_t valid_bits = 0;  // four bits a stage: which fragments have a page
  auto produce = [&](int s) {
    if (pre_x >= x1) return;
    const int id = next_page;
    const uint32_t have = __ballot_sync(0xffffffffu, id >= 0 && array == 0);
    uint32_t bits = 0;
#pragma unroll
    for (int f = 0; f < 4; ++f) bits |= ((have >> (4 * f)) & 1u) << f;
    valid_bits = (valid_bits & ~(0xfu << (4 * s))) | (bits << (4 * s));
    const uint32_t bar = bar0 + 8 * s;
    if (lane == 0) mbar_expect_tx(bar, (uint32_t)(__popc(bits) << fr_log2) * 2 * (C::CODE_ROW + C::SCALE_ROW));
    __syncwarp();
    if (id >= 0) {
      const long long tok = (long long)pre.u * UNIT + ((long long)frag << fr_log2);
      const long long row =
          (((long long)id * p.Hkv + pre.kvh) << p.page_log2) + (tok & ((1 << p.page_log2) - 1));
      const bool is_scale = array & 1;
      const int row_bytes = is_scale ? C::SCALE_ROW : C::CODE_ROW;
      const uint8_t* base = is_scale ? p.scales[array >> 1] : p.codes[array >> 1];
      const int off = array == 0 ? 0 : array == 1 ? C::OFF_KS : array == 2 ? C::OFF_V : C::OFF_VS;
      bulk_load(ring_addr + s * C::STAGE + off + (frag << fr_log2) * row_bytes, base + row * row_bytes,
                (uint32_t)row_bytes << fr_log2, bar);
    }
    ++pre_x;
    if (pre_x < x1) {
      kv4_advance(p, UNIT, C::ROWS, pre);
      next_page = page_of(pre);
    }
  };
#pragma unroll 1
  for (int s = 0; s < S; ++s) produce(s);

  // ------------------------------------------------------------- consumer side
  uint32_t qf[NT][WK][4];  // Q rows as B operands: per word of 8 channels, two k-steps of two registers
  float acc[NT][C::CT][4];
  float m[NT][2], l[NT][2], fac[NT][2];
  int lim[NT][2];  // last key that the lane's two columns (rows of Q) see
  int lim_min = 0;

  bool ok = true;
  int stage = 0;
  uint32_t phase = 0;
  bool fresh = true;
#pragma unroll 1
  for (long long x = x0; x < x1; ++x) {
    if (fresh) {
      fresh = false;
      lim_min = 0x7fffffff;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int row = cur.rt * C::ROWS + 8 * n + g;
        const int i = row / p.G, h = row - i * p.G;
        const bool have = i < cur.nq;
        const uint16_t* src =
            p.q + (long long)(cur.tok0 + (have ? i : 0)) * p.q_token + (long long)(cur.kvh * p.G + h) * p.q_head + t * (D / 4);
        uint32_t w[D / 8];
#pragma unroll
        for (int c = 0; c < D / 8; c += 4) {
          uint4 v = make_uint4(0u, 0u, 0u, 0u);
          if (have) v = *reinterpret_cast<const uint4*>(src + 2 * c);
          w[c] = v.x, w[c + 1] = v.y, w[c + 2] = v.z, w[c + 3] = v.w;
        }
        // The row's largest magnitude, as bf16 bits, gives the power of two.
        uint32_t top = 0;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) top = max(top, max(w[c] & 0x7fffu, (w[c] >> 16) & 0x7fffu));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // 2^-e with e the exponent of the largest, both factors normal fp32.
        const int e = min(max((int)(top >> 7) - 127, -120), 120);
        const float down = __uint_as_float((uint32_t)(127 - e) << 23);
        const float up = __uint_as_float((uint32_t)(127 + e) << 23) * p.score;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          const float lo = __uint_as_float(w[c] << 16) * down, hi = __uint_as_float(w[c] & 0xffff0000u) * down;
          qf[n][c >> 2][c & 3] = pack_f16(lo, hi);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          fac[n][j] = __shfl_sync(0xffffffffu, up, (2 * t + j) * 4);
          const int r = cur.rt * C::ROWS + 8 * n + 2 * t + j;
          const int qi = r / p.G;
          lim[n][j] = qi < cur.nq ? cur.n - cur.nq + qi : -1;
          m[n][j] = -INFINITY;
          l[n][j] = 0.f;
          if (qi < cur.nq) lim_min = min(lim_min, lim[n][j]);
        }
#pragma unroll
        for (int c = 0; c < C::CT; ++c) acc[n][c][0] = acc[n][c][1] = acc[n][c][2] = acc[n][c][3] = 0.f;
      }
      lim_min = __reduce_min_sync(0xffffffffu, lim_min);
    }

    if (!wait_warp(bar0 + 8 * stage, phase, ab, (kKKv4 << 8) | 1)) {
      ok = false;
      break;
    }
    const uint8_t* sk = ring + stage * C::STAGE;
    const uint8_t* sv = sk + C::OFF_V;
    const uint32_t bits = (valid_bits >> (4 * stage)) & 0xfu;

    // S^T = K Q^T.
    float sc[MT][NT][4];
#pragma unroll
    for (int a = 0; a < MT; ++a) {
#pragma unroll
      for (int n = 0; n < NT; ++n) sc[a][n][0] = sc[a][n][1] = sc[a][n][2] = sc[a][n][3] = 0.f;
      uint32_t w[2][WK], s2[2][(WK + 1) / 2 + 1];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int tok = 16 * a + 8 * h + g;
        lds_words<WK>(sk + tok * C::CODE_ROW + t * (4 * WK), w[h]);
        const uint8_t* ss = sk + C::OFF_KS + tok * C::SCALE_ROW + ((t * WK) >> 1);
        if constexpr (WK % 2 == 0) {
#pragma unroll
          for (int i = 0; i < WK / 2; ++i) s2[h][i] = kv4_scale_both(ss[i]);
        } else {
          // Three words: odd lanes start in the middle of a scale's group.
          const uint32_t s0 = kv4_scale_both(ss[0]), s1 = kv4_scale_both(ss[1]);
          s2[h][0] = s0;
          s2[h][1] = (t & 1) ? s1 : s0;
          s2[h][2] = s1;
        }
      }
#pragma unroll
      for (int i = 0; i < WK; ++i) {
        uint32_t r0[4], r1[4];
        kv4_codes(w[0][i], r0);
        kv4_codes(w[1][i], r1);
        const int si = WK % 2 == 0 ? i >> 1 : i;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          r0[j] = h2mul(r0[j], s2[0][si]);
          r1[j] = h2mul(r1[j], s2[1][si]);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mma_f16(sc[a][n], r0[0], r1[0], r0[1], r1[1], qf[n][i][0], qf[n][i][1]);
          mma_f16(sc[a][n], r0[2], r1[2], r0[3], r1[3], qf[n][i][2], qf[n][i][3]);
        }
      }
    }

    // Softmax over the unit's tokens: column 2t + j of every tile belongs to this lane's (n, j).
    const long long key0 = (long long)cur.u * UNIT;
    const bool whole = key0 + UNIT - 1 <= lim_min && bits == (1u << frags) - 1u;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float mx = -INFINITY;
        if (whole) {
#pragma unroll
          for (int a = 0; a < MT; ++a) mx = max3(mx, sc[a][n][j] *= fac[n][j], sc[a][n][2 + j] *= fac[n][j]);
        } else {
#pragma unroll
          for (int a = 0; a < MT; ++a)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int tok = 16 * a + 8 * h + g;
              const bool seen = key0 + tok <= lim[n][j] && ((bits >> (tok >> fr_log2)) & 1u);
              const float v = seen ? sc[a][n][2 * h + j] * fac[n][j] : -INFINITY;
              sc[a][n][2 * h + j] = v;
              mx = fmaxf(mx, v);
            }
        }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
        mx -= kKv4Lift;
        const bool grow = mx > m[n][j] + kKv4Grow;
        const float alpha = grow ? ex2(m[n][j] - mx) : 1.f;
        if (grow) m[n][j] = mx;
        l[n][j] *= alpha;
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int c = 0; c < C::CT; ++c) {
            acc[n][c][j] *= alpha;
            acc[n][c][2 + j] *= alpha;
          }
        }
        const float msub = m[n][j] == -INFINITY ? 0.f : m[n][j];
        float sum = 0.f;
#pragma unroll
        for (int a = 0; a < MT; ++a) {
          sc[a][n][j] = ex2(sc[a][n][j] - msub);
          sc[a][n][2 + j] = ex2(sc[a][n][2 + j] - msub);
          sum += sc[a][n][j] + sc[a][n][2 + j];
        }
        l[n][j] += sum;
      }
    }

    // O^T += V^T P^T.
#pragma unroll
    for (int a = 0; a < MT; ++a) {
      uint32_t pb[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        pb[n][0] = transpose8(pack_f16(sc[a][n][0], sc[a][n][1]));
        pb[n][1] = transpose8(pack_f16(sc[a][n][2], sc[a][n][3]));
      }
      const int tok = 16 * a + 2 * t;  // with tok + 1, tok + 8, tok + 9
      uint32_t w[4][WV];
      const uint8_t* row[4] = {sv + tok * C::CODE_ROW, sv + (tok + 1) * C::CODE_ROW, sv + (tok + 8) * C::CODE_ROW,
                               sv + (tok + 9) * C::CODE_ROW};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if constexpr (C::HALF) {
          const uint16_t* h = reinterpret_cast<const uint16_t*>(row[k] + g * (D / 16));
          w[k][0] = h[0] | ((uint32_t)h[1] << 16);
          w[k][1] = h[2];
        } else {
          lds_words<WV>(row[k] + g * (D / 16), w[k]);
        }
      }
      const uint8_t* ss = sk + C::OFF_VS + tok * C::SCALE_ROW;
#pragma unroll
      for (int i = 0; i < WV; ++i) {
        // The scales of channels 8i.. of the lane's D/8, at tokens (tok, tok+1) and (tok+8, tok+9).
        uint32_t s2[2][2];  // [half of the word][token pair]
#pragma unroll
        for (int hw = 0; hw < 2; ++hw) {
          if (hw == 1 && !C::HALF) {
            s2[1][0] = s2[0][0];
            s2[1][1] = s2[0][1];
          } else {
            const int grp = (g * (D / 8) + 8 * i + 4 * hw) >> 4;
            if (C::HALF && 8 * i + 4 * hw >= D / 8) {
              s2[1][0] = s2[1][1] = 0;
            } else {
              s2[hw][0] = kv4_scale_pair(ss[grp], ss[C::SCALE_ROW + grp]);
              s2[hw][1] = kv4_scale_pair(ss[8 * C::SCALE_ROW + grp], ss[9 * C::SCALE_ROW + grp]);
            }
          }
        }
        constexpr uint32_t M = 0x0f0f0f0fu;
        uint32_t e0[4], e1[4], o0[4], o1[4];  // even and odd channels at the two token pairs
        kv4_codes((w[0][i] & M) | ((w[1][i] << 4) & ~M), e0);
        kv4_codes(((w[0][i] >> 4) & M) | (w[1][i] & ~M), o0);
        kv4_codes((w[2][i] & M) | ((w[3][i] << 4) & ~M), e1);
        kv4_codes(((w[2][i] >> 4) & M) | (w[3][i] & ~M), o1);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          if (4 * i + b >= C::CT) continue;
          const uint32_t a0 = h2mul(e0[b], s2[b >> 1][0]), a1 = h2mul(o0[b], s2[b >> 1][0]);
          const uint32_t a2 = h2mul(e1[b], s2[b >> 1][1]), a3 = h2mul(o1[b], s2[b >> 1][1]);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma_f16(acc[n][4 * i + b], a0, a1, a2, a3, pb[n][0], pb[n][1]);
        }
      }
    }

    // Every lane is done with the slot: refill it.
    __syncwarp();
    produce(stage);
    if (++stage == S) {
      stage = 0;
      phase ^= 1;
    }

    const bool last_unit = cur.u == cur.units - 1;
    if (last_unit || x == x1 - 1) {
      const bool first_here = x - cur.u >= x0;  // the triple began in this warp's range
      const bool direct = last_unit && first_here;
      float* po = nullptr;
      if (!direct) {
        // Slot 1: the triple begins here and goes on; slot 0: it began before.
        const size_t slot = (size_t)me * 2 + (first_here ? 1 : 0);
        po = p.part_o + slot * C::ROWS * D;
        float* pml = p.part_ml + slot * C::ROWS * 2;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float s = l[n][j];
            s += __shfl_xor_sync(0xffffffffu, s, 4);
            s += __shfl_xor_sync(0xffffffffu, s, 8);
            s += __shfl_xor_sync(0xffffffffu, s, 16);
            if (g == 0) *reinterpret_cast<float2*>(pml + (8 * n + 2 * t + j) * 2) = make_float2(m[n][j], s);
          }
      }
      if (first_here && lane == 0) {
        const int seg = (cur.b * p.Hkv + cur.kvh) * p.row_tiles + cur.rt;
        const long long start = x - cur.u;
        p.meta[seg] = make_int2(me, direct ? 0 : worker_of(start + cur.units - 1) - me + 1);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int rr = 8 * n + 2 * t + j;
          if (!direct) {
            float* dst = po + (size_t)rr * D + g * (D / 8);
#pragma unroll
            for (int c = 0; c < C::CT; c += 2)
              *reinterpret_cast<float4*>(dst + 2 * c) =
                  make_float4(acc[n][c][j], acc[n][c][2 + j], acc[n][c + 1][j], acc[n][c + 1][2 + j]);
          } else {
            float s = l[n][j];
            s += __shfl_xor_sync(0xffffffffu, s, 4);
            s += __shfl_xor_sync(0xffffffffu, s, 8);
            s += __shfl_xor_sync(0xffffffffu, s, 16);
            const int r = cur.rt * C::ROWS + rr;
            const int i = r / p.G, h = cur.kvh * p.G + r - i * p.G;
            if (i < cur.nq) {
              const float inv = s == 0.f ? 0.f : p.v_gain / s;
              uint16_t* dst = p.o + (long long)(cur.tok0 + i) * p.o_token + (long long)h * p.o_head + g * (D / 8);
#pragma unroll
              for (int c = 0; c < C::CT; c += 2)
                *reinterpret_cast<uint2*>(dst + 2 * c) =
                    make_uint2(pack_bf16(acc[n][c][j] * inv, acc[n][c][2 + j] * inv),
                               pack_bf16(acc[n][c + 1][j] * inv, acc[n][c + 1][2 + j] * inv));
              if (g == 0)
                p.lse[(long long)(cur.tok0 + i) * p.H + h] = s == 0.f ? -INFINITY : (m[n][j] + log2f(s)) * kLn2;
            }
          }
        }
      fresh = true;
    }
    if (x + 1 < x1) kv4_advance(p, UNIT, C::ROWS, cur);
  }
  // A warp that gave up lets its copies land before the block can exit.
  if (!ok)
    for (long long x = max(pre_x - S, x0); x < pre_x; ++x) {
      const long long i = x - x0;
      wait_done(bar0 + 8 * (uint32_t)(i % S), (uint32_t)((i / S) & 1));
    }
}

// Joins the parts of cut triples: with M the largest m of a row's parts,
// O = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s.  One block per row of a
// triple; its warps take the parts in turn, each lane one to three runs of four
// channels, and the sums are joined in shared memory in a fixed order.
template <int D>
__global__ void __launch_bounds__(128) kv4_merge_kernel(const __grid_constant__ Kv4AttnParams p) {
  __shared__ float acc[4][D];
  __shared__ float ml[4][2];
  const int unit = p.unit, rows = p.rows;
  grid_dep_wait();
  if (*reinterpret_cast<volatile const int*>(p.err) != 0) return;
  const int seg = blockIdx.x / rows, rr = blockIdx.x - seg * rows;
  const int bk = seg / p.row_tiles, rt = seg - bk * p.row_tiles;
  const int b = bk / p.Hkv, kvh = bk - b * p.Hkv;
  Kv4Cursor c;
  kv4_request(p, b, unit, rows, c);
  const int r = rt * rows + rr;
  const int i = r / p.G, h = kvh * p.G + r - i * p.G;
  if (rt >= c.tiles || i >= c.nq) return;
  const int2 meta = p.meta[seg];
  if (meta.y == 0) return;
  const int warp = warp_id(), lane = lane_id();
  // Part s of the triple: slot 1 of its first warp, slot 0 of the later ones.
  auto slot = [&](int s) -> size_t { return (size_t)(meta.x + s) * 2 + (s == 0 ? 1 : 0); };
  float top = -INFINITY;
  for (int s = lane; s < meta.y; s += 32) top = fmaxf(top, p.part_ml[(slot(s) * rows + rr) * 2]);
#pragma unroll
  for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  const float sub = top == -INFINITY ? 0.f : top;
  constexpr int V = (D + 127) / 128;
  float4 o[V];
#pragma unroll
  for (int v = 0; v < V; ++v) o[v] = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f;
#pragma unroll 4
  for (int s = warp; s < meta.y; s += 4) {
    const float2 x = *reinterpret_cast<const float2*>(p.part_ml + (slot(s) * rows + rr) * 2);
    const float wt = ex2(x.x - sub);
    sum += wt * x.y;
    const float* src = p.part_o + (slot(s) * rows + rr) * D;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int col = 128 * v + 4 * lane;
      if (col < D) {
        const float4 y = *reinterpret_cast<const float4*>(src + col);
        o[v].x += wt * y.x;
        o[v].y += wt * y.y;
        o[v].z += wt * y.z;
        o[v].w += wt * y.w;
      }
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (128 * v + 4 * lane < D) *reinterpret_cast<float4*>(&acc[warp][128 * v + 4 * lane]) = o[v];
  if (lane == 0) ml[warp][0] = sum;
  __syncthreads();
  const float s = (ml[0][0] + ml[1][0]) + (ml[2][0] + ml[3][0]);
  const float inv = s == 0.f ? 0.f : p.v_gain / s;
  uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + (long long)(c.tok0 + i) * p.o_token + (long long)h * p.o_head);
  for (int k = threadIdx.x; k < D / 2; k += 128) {
    const float lo = (acc[0][2 * k] + acc[1][2 * k]) + (acc[2][2 * k] + acc[3][2 * k]);
    const float hi = (acc[0][2 * k + 1] + acc[1][2 * k + 1]) + (acc[2][2 * k + 1] + acc[3][2 * k + 1]);
    dst[k] = pack_bf16(lo * inv, hi * inv);
  }
  if (threadIdx.x == 0) p.lse[(long long)(c.tok0 + i) * p.H + h] = s == 0.f ? -INFINITY : (top + log2f(s)) * kLn2;
}

}  // namespace fa
