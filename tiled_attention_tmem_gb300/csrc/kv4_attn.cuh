// Attention of a few query tokens per request over the paged 4-bit cache.
//
// Per request b and kv head, the R = n_q * (H/Hkv) query rows that share the
// cached head are cut into tiles of 8*NT rows, and the tokens into units of UNIT.
// All units of all (request, kv head, row tile) triples, laid end to end, are
// shared out evenly over the warps of the grid: warp w takes units
// [w*T/W, (w+1)*T/W), whatever requests they belong to, so ragged batches and one
// long request load the SMs alike, and no warp waits for another.  A triple that
// lies in one warp's range is finished there; one that is cut leaves a part
// (unnormalised fp32 O, running maximum m, sum l) a warp for kv4_merge_kernel.
//
// One unit: its K and its V (codes and scales, UNIT*d*0.5625 bytes each) come by bulk
// copies into the warp's own ring of STAGES units, refilled by the warp itself as
// soon as it is done with a K or a V; both products run on mma.m16n8k16 with f16
// operands and fp32 accumulators, from registers:
//   S^T = K Q^T : A = 16 tokens x 16 channels, dequantised in registers (exact in
//                 f16), B = Q rows (f16, the type that K's products are exact in and so
//                 the MMA's; each row scaled by a power of two so that its largest channel
//                 is in [1, 2), which its score factor takes back: bf16's eight bits are
//                 exact down to 2^-17, and what is below is off by 2^-25 at most)
//   O^T += V^T P^T : A = 16 channels x 16 tokens; the codes of two tokens are
//                 interleaved before conversion, so each f16 pair is one channel at
//                 two tokens; B = P, transposed by movmatrix from S^T's layout
// K's channels and V's channels are dealt to lanes so that every lane reads
// contiguous bytes: the order of a contraction's terms is free, and O's channel
// order is undone at the store.
//
// Reading the cache bounds it in principle: 64 requests up to 16384 tokens, 8 kv heads, d = 128,
// group 4 (686 MB) take 126 us, 5450 GB/s; 163 us for each GB and, where all SMs are in
// use, about 14 us beside that: two launches, four loads that wait for one another, and the
// first and last units, which are not overlapped.  The issue slots are 63 % used, the ALU
// pipe 54 %, so the work per byte is what needs care:
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
  int2* cuts;      // [B*Hkv*row_tiles]: a triple's first warp and its parts (0: not cut)
  int* err;
  long long q_token, q_head, o_token, o_head;
  int B, H, Hkv, G, T, width, pages, page_log2, max_q;
  int row_tiles;  // most row tiles of a request
  float score;    // scale * log2(e) * k_gain * 2^8 = score * 2^score_exp, score in [1, 2]
  int score_exp;
  float v_gain;   // v_gain * 2^8
};

// P is rounded to f16 for the product with V (both operands of an MMA have one type), and
// its sum taken before that, in fp32: the rounding errors of a row are independent, 2^-11 of
// a probability at most each, and shared between numerator and sum they would be no smaller.
// P is kept times 2^7 (m is the maximum less 7), and the maximum is only renewed
// when it grew by more than 8: p <= 2^15 fits f16, and what f16 flushes lies
// 2^-32 below the largest.  (ex2.approx is good to 2^-22 of its value; a score
// of a few units is no finer in fp32.)
constexpr float kKv4Lift = 7.f;
constexpr float kKv4Grow = 8.f;

// What takes scores of a row that was scaled by 2^-e to the log2 domain.  The exponents are
// added before they meet fp32: a scale at one end of its range and a gain or a query at the
// other give ordinary scores.  Not 0, so that a masked score stays -inf, and finite, so that a
// score of 0 stays 0.
__device__ __forceinline__ float kv4_score_factor(const Kv4AttnParams& p, int e) {
  const int x = min(max(e + p.score_exp, -126), 127);
  return fminf(fmaxf(__uint_as_float((uint32_t)(127 + x) << 23) * p.score, 1e-37f), 3e38f);
}

// Warps per SM and tokens per unit for head dim d and nt tiles of 8 rows (what the registers
// hold: with three tiles and 64 tokens the scores would not fit).
constexpr int kv4_warps(int d, int nt) {
  return d * nt <= 128 || (nt == 1 && d <= 256) ? 12 : 8;
}
constexpr int kv4_unit(int d, int nt) { return d <= 128 && nt != 3 ? 64 : 32; }

// SOLO: a block per triple, whose warps take its units in turn and join their parts in
// shared memory: one launch, and no search for where a range begins.  For short
// contexts; several of its smaller blocks share an SM.
constexpr int kKv4SoloWarps = 4;
constexpr int kv4_solo_blocks(int d, int nt) { return nt == 1 && d <= 256 ? 3 : 2; }  // an SM
template <int D_, int NT_, bool SOLO_>
struct Kv4Cfg {
  static constexpr int D = D_, NT = NT_;
  static constexpr bool SOLO = SOLO_;
  static constexpr int ROWS = 8 * NT;
  static constexpr int UNIT = kv4_unit(D, NT);
  static constexpr int MT = UNIT / 16;
  static constexpr int WARPS = SOLO ? kKv4SoloWarps : kv4_warps(D, NT);
  static constexpr int THREADS = 32 * WARPS;
  static constexpr int CODE_ROW = D / 2, SCALE_ROW = D / 16;  // bytes a token
  static constexpr int OFF_SCALE = UNIT * CODE_ROW;
  static constexpr int PART = UNIT * (CODE_ROW + SCALE_ROW);  // K or V of a unit
  static constexpr int OTHER = SOLO ? 512 : THREADS * 24 + 1024;  // what follows the ring
  static constexpr int BLOCKS = SOLO ? kv4_solo_blocks(D, NT) : 1;  // an SM
  static constexpr int FIT = (233472 / BLOCKS - 1024 - OTHER) / (WARPS * 2 * PART);
  static constexpr int STAGES = FIT < 4 ? FIT : 4;
  static constexpr int OFF_BAR = WARPS * STAGES * 2 * PART;       // per stage: K full, V full
  static constexpr int OFF_PREFIX = OFF_BAR + WARPS * STAGES * 16;
  static constexpr int OFF_REQ = OFF_PREFIX + (SOLO ? 0 : (THREADS + 1) * 8);  // the requests
  static constexpr int OFF_MISC = OFF_REQ + (SOLO ? 0 : THREADS * 16);
  static constexpr int SMEM = OFF_MISC + 16 + WARPS * 8;
  static constexpr int WK = D / 32;         // words of 8 codes a lane reads of a K row
  static constexpr int WV = (D + 63) / 64;  // words a lane reads of a V row (d = 96: one and a half)
  static constexpr bool HALF = D % 64 != 0;
  static constexpr int CT = D / 16;  // O^T tiles of 16 channels
  static_assert(STAGES >= 2 && BLOCKS * (SMEM + 1024) <= 233472, "shared memory");
  // A SOLO warp's part, O and then (m, l), lies where its ring was.
  static constexpr int RING = STAGES * 2 * PART;
  static_assert(ROWS * (D + 2) * 4 <= RING, "a part fits a ring");
};

// A position in the sequence of units.
struct Kv4Cursor {
  int b, kvh, rt, u;      // request, kv head, row tile, unit
  int units, tiles;       // units and row tiles of request b
  int n, tok0, nq;        // tokens of b, its first query token, its queries (max_q at most)
  int first;              // position of its first query (negative: that one sees nothing)
};

// Tokens, first query and queries of request b from the caller's arrays.
__device__ __forceinline__ void kv4_lookup(const Kv4AttnParams& p, int b, Kv4Cursor& c) {
  c.n = max(p.lengths[b], 0);
  if (p.cu) {
    c.tok0 = p.cu[b];
    const long long nq = (long long)p.cu[b + 1] - c.tok0;
    c.nq = (int)min(max(nq, 0LL), (long long)p.max_q);
    c.first = (int)max(c.n - max(nq, 0LL), -0x7fffffffLL);
    if (c.tok0 < 0 || c.tok0 + nq > p.T) c.nq = 0;  // queries outside q, past max_q or not: none is computed
  } else {
    c.tok0 = b;
    c.nq = 1;
    c.first = c.n - 1;
  }
}

// Request b, from shared memory where the block keeps all requests (req not NULL).
template <class C>
__device__ __forceinline__ void kv4_request(const Kv4AttnParams& p, const int* req, int b, Kv4Cursor& c) {
  if (req) {
    c.n = req[4 * b], c.tok0 = req[4 * b + 1], c.nq = req[4 * b + 2], c.first = req[4 * b + 3];
  } else {
    kv4_lookup(p, b, c);
  }
  c.tiles = (int)(((long long)c.nq * p.G + C::ROWS - 1) / C::ROWS);
  // Tokens past the table's width are no keys.
  const long long held = min((long long)c.n, (long long)p.width << p.page_log2);
  c.units = c.tiles ? max((int)((held + C::UNIT - 1) / C::UNIT), 1) : 0;
}

template <class C>
__device__ __forceinline__ void kv4_advance(const Kv4AttnParams& p, const int* req, Kv4Cursor& c) {
  if (++c.u < c.units) return;
  c.u = 0;
  if (++c.rt < c.tiles) return;
  c.rt = 0;
  if (++c.kvh < p.Hkv) return;
  c.kvh = 0;
  do {
    if (++c.b >= p.B) {  // past the last unit (only if the lengths changed meanwhile): nothing to do there
      c.b = p.B - 1;
      c.n = c.nq = c.first = 0;
      c.units = c.tiles = 1;
      return;
    }
    kv4_request<C>(p, req, c.b, c);
  } while (c.units == 0);
}

// Where each thread's run of requests begins in the sequence of units: prefix[i] units
// lie before thread i's ceil(B / THREADS) requests, prefix[THREADS] in all.  `kept` takes
// the requests themselves (tokens, first query token, queries, position) if every thread has one at most.
// `sums` has a word for each warp.  Ends with a barrier.
template <class C>
__device__ __forceinline__ long long kv4_scan(const Kv4AttnParams& p, long long* prefix, int* kept, long long* sums) {
  const int warp = warp_id(), lane = lane_id();
  const int run = (p.B + C::THREADS - 1) / C::THREADS;
  const int b0 = min((int)threadIdx.x * run, p.B), b1 = min(b0 + run, p.B);
  long long sum = 0;
  for (int b = b0; b < b1; ++b) {
    Kv4Cursor c;
    kv4_request<C>(p, nullptr, b, c);
    if (run == 1 && kept) kept[4 * b] = c.n, kept[4 * b + 1] = c.tok0, kept[4 * b + 2] = c.nq, kept[4 * b + 3] = c.first;
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
  for (int w = 0; w < C::THREADS / 32; ++w) {
    if (w < warp) before += sums[w];
    total += sums[w];
  }
  prefix[threadIdx.x] = before + x - sum;
  if (threadIdx.x == 0) prefix[C::THREADS] = total;
  __syncthreads();
  return total;
}

// Sets c to unit x of the sequence.  False only if the lengths changed meanwhile.
template <class C>
__device__ __forceinline__ bool kv4_locate(const Kv4AttnParams& p, const long long* prefix, const int* req, long long x,
                                           Kv4Cursor& c) {
  const int run = (p.B + C::THREADS - 1) / C::THREADS;
  int lo = 0, hi = C::THREADS;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid] <= x) lo = mid;
    else hi = mid;
  }
  long long rest = x - prefix[lo];
  for (c.b = lo * run; c.b < p.B; ++c.b) {
    kv4_request<C>(p, req, c.b, c);
    const long long mine = (long long)c.units * c.tiles * p.Hkv;
    if (rest < mine) {
      const int per_kvh = c.units * c.tiles;  // below 2^31: see the launcher
      c.kvh = 0;
      if (rest >= per_kvh) {
        c.kvh = (int)(rest / per_kvh);
        rest -= (long long)c.kvh * per_kvh;
      }
      c.rt = (int)rest / c.units;
      c.u = (int)rest - c.rt * c.units;
      return true;
    }
    rest -= mine;
  }
  return false;
}

// An even share of `total` units for each of `workers`: the first `more` take per + 1,
// the others per.  worker_parts: over how many workers from `me` on a triple runs whose
// last unit but `rest` more lies in me's share.
struct Kv4Share {
  long long x0;
  int units, per, more;
  __device__ __forceinline__ Kv4Share(long long total, int workers, int me) {
    per = (int)min(total / workers, 0x7ffffffell);
    more = (int)(total - (long long)per * workers);
    x0 = (long long)per * me + min(me, more);
    units = per + (me < more ? 1 : 0);
  }
  __device__ __forceinline__ int parts(int me, int rest) const {
    const int wide = max(more - (me + 1), 0);  // of the workers after me, those that take per + 1
    return 1 + (rest <= (long long)wide * (per + 1) ? (rest + per) / (per + 1)
                                                    : wide + (rest - wide * (per + 1) + per - 1) / per);
  }
};

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
  asm(
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
__global__ void __launch_bounds__(C::THREADS, C::BLOCKS) kv4_attn_kernel(const __grid_constant__ Kv4AttnParams p) {
  constexpr int D = C::D, NT = C::NT, UNIT = C::UNIT, MT = C::MT, S = C::STAGES, WK = C::WK, WV = C::WV;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = warp_id(), lane = lane_id();
  const int g = lane >> 2, t = lane & 3;
  long long* prefix = reinterpret_cast<long long*>(smem + C::OFF_PREFIX);  // units before thread i's requests
  int* kept = reinterpret_cast<int*>(smem + C::OFF_REQ);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC);
  long long* sums = reinterpret_cast<long long*>(smem + C::OFF_MISC + 16);
  const uint32_t bars = smem_u32(smem + C::OFF_BAR) + warp * S * 16;
  uint8_t* ring = smem + warp * S * 2 * C::PART;
  const uint32_t ring_addr = smem_u32(ring);

  if (threadIdx.x == 0) *abort_flag = 0;
  if (lane < 2 * S) {
    mbar_init(bars + 8 * lane, 1);
    fence_mbar_init();
  }
  grid_dep_wait();
  const bool skip = *reinterpret_cast<volatile int*>(p.err) != 0;

  const CtaAbort ab{abort_flag, p.err};
  const int* req = nullptr;  // the requests in shared memory, if they fit there
  Kv4Cursor cur;
  Kv4Share share(0, 1, 0);      // of this warp
  int units = 0, me = 0;
  if constexpr (C::SOLO) {
    __syncthreads();  // (the barriers and the abort flag)
    if (skip) return;
    const int bk = blockIdx.x / p.row_tiles;
    cur.b = bk / p.Hkv;
    kv4_request<C>(p, nullptr, cur.b, cur);
    cur.kvh = bk - cur.b * p.Hkv;
    cur.rt = blockIdx.x - bk * p.row_tiles;
    cur.u = warp;
    if (cur.rt >= cur.tiles) return;
    units = max(cur.units - warp + C::WARPS - 1, 0) / C::WARPS;
    if (cur.units == 1 && warp > 0) return;  // one unit: its warp finishes the triple
  } else {
  const long long total = kv4_scan<C>(p, prefix, kept, sums);
  if (skip) return;
  req = p.B <= C::THREADS ? kept : nullptr;
  // Neighbouring ranges go to different SMs, so that few units spread over all.
  me = warp * gridDim.x + blockIdx.x;
  share = Kv4Share(total, gridDim.x * C::WARPS, me);
  units = share.units;
  if (units == 0 || !kv4_locate<C>(p, prefix, req, share.x0, cur)) return;
  }
  int left = units, ahead = units;  // still to compute and to copy (a SOLO warp may have none)

  // ------------------------------------------------------------------- copies
  // A K or V is UNIT / FR fragments of FR = min(page, UNIT) tokens, each inside one
  // page: lane 2f copies fragment f's codes, lane 2f + 1 its scales.  V's source lies
  // where K's does in its own arrays.  A unit's page ids are read a unit ahead.
  const int fr_log2 = min(p.page_log2, UNIT == 64 ? 6 : 5);
  const uint32_t all_bits = (1u << (UNIT >> fr_log2)) - 1u;
  const int frag = lane >> 1;
  const int row_bytes = (lane & 1) ? C::SCALE_ROW : C::CODE_ROW;
  const uint32_t copy_bytes = (uint32_t)row_bytes << fr_log2;
  const uint32_t copy_dst = ring_addr + ((lane & 1) ? C::OFF_SCALE : 0) + frag * copy_bytes;
  Kv4Cursor pre = cur;
  auto page_of = [&]() -> int {
    const long long tok = (long long)pre.u * UNIT + ((long long)frag << fr_log2);
    const int col = (int)(tok >> p.page_log2);
    if (frag >= (UNIT >> fr_log2) || tok >= pre.n || col >= p.width) return -1;
    const int id = p.table[(size_t)pre.b * p.width + col];
    return (unsigned)id < (unsigned)p.pages ? id : -1;
  };
  int next_id = page_of();
  uint32_t valid_bits = 0;   // four bits a stage: which fragments have a page
  const uint8_t* v_src = nullptr;  // of the unit whose K was copied last
  bool v_have = false, k_alone = false;  // k_alone: its V is not copied yet
  uint32_t v_bytes = 0;
  auto copy_k = [&](int s) {
    if (ahead <= 0) return;
    const int id = next_id;
    const uint32_t have = __ballot_sync(0xffffffffu, id >= 0 && !(lane & 1));
    const uint32_t bits = (have & 1u) | ((have >> 1) & 2u) | ((have >> 2) & 4u) | ((have >> 3) & 8u);
    valid_bits = (valid_bits & ~(0xfu << (4 * s))) | (bits << (4 * s));
    v_bytes = (uint32_t)(__popc(bits) << fr_log2) * (C::CODE_ROW + C::SCALE_ROW);
    v_have = id >= 0;
    k_alone = true;
    if (lane == 0) mbar_expect_tx(bars + 16 * s, v_bytes);
    __syncwarp();
    if (v_have) {
      const uint32_t in_page = (uint32_t)((pre.u * UNIT + (frag << fr_log2)) & ((1 << p.page_log2) - 1));
      const long long row = (((long long)id * p.Hkv + pre.kvh) << p.page_log2) + in_page;
      const long long off = row * row_bytes;
      bulk_load(copy_dst + s * 2 * C::PART, ((lane & 1) ? p.scales[0] : p.codes[0]) + off, copy_bytes, bars + 16 * s);
      v_src = ((lane & 1) ? p.scales[1] : p.codes[1]) + off;
    }
    if (ahead > 1) {
      if constexpr (C::SOLO) pre.u += C::WARPS;
      else kv4_advance<C>(p, req, pre);
      next_id = page_of();
    }
  };
  auto copy_v = [&](int s) {
    if (ahead <= 0) return;
    --ahead;
    k_alone = false;
    if (lane == 0) mbar_expect_tx(bars + 16 * s + 8, v_bytes);
    __syncwarp();
    if (v_have) bulk_load(copy_dst + (2 * s + 1) * C::PART, v_src, copy_bytes, bars + 16 * s + 8);
  };
#pragma unroll 1
  for (int s = 0; s < S; ++s) {
    copy_k(s);
    copy_v(s);
  }

  // -------------------------------------------------------------- computation
  uint32_t qf[NT][WK][4];  // Q rows as B operands: per word of 8 channels, two k-steps of two registers
  float acc[NT][C::CT][4];
  float m[NT][2], l[NT][2], fac[NT][2];
  int lim[NT][2];  // last key that the lane's two columns (rows of Q) see
  int lim_min = 0;
  int stage = 0;
  uint32_t phase = 0;
  bool fresh = true;
  long long began = share.x0 - cur.u;  // first unit of the current triple
#pragma unroll 1
  for (; left > 0; --left) {
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
        // 2^-e with e the exponent of the largest, kept where 2^-e is normal fp32.
        const int e = min(max((int)(top >> 7) - 127, -120), 120);
        const float down = __uint_as_float((uint32_t)(127 - e) << 23);
        const float up = kv4_score_factor(p, e);
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
          lim[n][j] = qi < cur.nq ? cur.first + qi : -1;
          m[n][j] = -INFINITY;
          l[n][j] = 0.f;
          if (qi < cur.nq) lim_min = min(lim_min, lim[n][j]);
        }
#pragma unroll
        for (int c = 0; c < C::CT; ++c) acc[n][c][0] = acc[n][c][1] = acc[n][c][2] = acc[n][c][3] = 0.f;
      }
      lim_min = __reduce_min_sync(0xffffffffu, lim_min);
    }

    if (!wait_warp(bars + 16 * stage, phase, ab, (kKKv4 << 8) | 1)) break;
    const uint8_t* sk = ring + stage * 2 * C::PART;
    const uint8_t* sv = sk + C::PART;
    const uint32_t bits = (valid_bits >> (4 * stage)) & 0xfu;

    // S^T = K Q^T, PAIR tiles of 16 tokens at a time: the products of one tile are a chain
    // through its accumulators, so two run between one another.  Row r of a tile's half is
    // token r ^ ((r >> 1) & 1): of the rows that a lane's V loads take together, two are
    // then even tokens and two odd, which halves their bank conflicts (64-byte rows).
    constexpr int PAIR = NT == 1 ? 2 : 1;
    const int gt = g ^ ((g >> 1) & 1);
    float sc[MT][NT][4];
#pragma unroll
    for (int a0 = 0; a0 < MT; a0 += PAIR) {
      uint32_t w[PAIR][2][WK], s2[PAIR][2][(WK + 1) / 2 + 1];
#pragma unroll
      for (int q = 0; q < PAIR; ++q)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int tok = 16 * (a0 + q) + 8 * h + gt;
          lds_words<WK>(sk + tok * C::CODE_ROW + t * (4 * WK), w[q][h]);
          const uint8_t* ss = sk + C::OFF_SCALE + tok * C::SCALE_ROW + ((t * WK) >> 1);
          if constexpr (WK % 2 == 0) {
#pragma unroll
            for (int i = 0; i < WK / 2; ++i) s2[q][h][i] = kv4_scale_both(ss[i]);
          } else {
            // Three words: odd lanes start in the middle of a scale's group.
            const uint32_t s0 = kv4_scale_both(ss[0]), s1 = kv4_scale_both(ss[1]);
            s2[q][h][0] = s0;
            s2[q][h][1] = (t & 1) ? s1 : s0;
            s2[q][h][2] = s1;
          }
        }
#pragma unroll
      for (int i = 0; i < WK; ++i) {
        const int si = WK % 2 == 0 ? i >> 1 : i;
        uint32_t r[PAIR][2][4];
#pragma unroll
        for (int q = 0; q < PAIR; ++q)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            kv4_codes(w[q][h][i], r[q][h]);
#pragma unroll
            for (int j = 0; j < 4; ++j) r[q][h][j] = h2mul(r[q][h][j], s2[q][h][si]);
          }
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int q = 0; q < PAIR; ++q)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              float* c = sc[a0 + q][n];
              if (i == 0 && k == 0) c[0] = c[1] = c[2] = c[3] = 0.f;
              mma_f16(c, r[q][0][2 * k], r[q][1][2 * k], r[q][0][2 * k + 1], r[q][1][2 * k + 1], qf[n][i][2 * k],
                      qf[n][i][2 * k + 1]);
            }
      }
    }

    __syncwarp();
    copy_k(stage);  // every lane is done with this K

    // Softmax over the unit's tokens: column 2t + j of every tile belongs to this lane's (n, j).
    const int key0 = cur.u * UNIT;
    if (!(key0 + UNIT - 1 <= lim_min && bits == all_bits)) {
#pragma unroll
      for (int a = 0; a < MT; ++a)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int tok = 16 * a + 8 * h + gt;
          const bool held = (bits >> (tok >> fr_log2)) & 1u;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j)
              if (key0 + tok > lim[n][j] || !held) sc[a][n][2 * h + j] = -INFINITY;
        }
    }
    float mx[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        mx[n][j] = fmaxf(sc[0][n][j], sc[0][n][2 + j]);
#pragma unroll
        for (int a = 1; a < MT; ++a) mx[n][j] = max3(mx[n][j], sc[a][n][j], sc[a][n][2 + j]);
      }
#pragma unroll
    for (int d = 4; d < 32; d <<= 1)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) mx[n][j] = fmaxf(mx[n][j], __shfl_xor_sync(0xffffffffu, mx[n][j], d));
    float alpha[NT][2];
    bool grows = false;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float high = mx[n][j] * fac[n][j] - kKv4Lift;
        const bool grow = high > m[n][j] + kKv4Grow;
        alpha[n][j] = grow ? ex2(m[n][j] - high) : 1.f;
        if (grow) m[n][j] = high;
        grows |= grow;
      }
    if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          l[n][j] *= alpha[n][j];
#pragma unroll
          for (int c = 0; c < C::CT; ++c) {
            acc[n][c][j] *= alpha[n][j];
            acc[n][c][2 + j] *= alpha[n][j];
          }
        }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float msub = m[n][j] == -INFINITY ? 0.f : m[n][j];
        float sum = 0.f;
#pragma unroll
        for (int a = 0; a < MT; ++a) {
          sc[a][n][j] = ex2(fmaf(sc[a][n][j], fac[n][j], -msub));
          sc[a][n][2 + j] = ex2(fmaf(sc[a][n][2 + j], fac[n][j], -msub));
          sum += sc[a][n][j] + sc[a][n][2 + j];
        }
        l[n][j] += sum;
      }

    if (!wait_warp(bars + 16 * stage + 8, phase, ab, (kKKv4 << 8) | 2)) break;

    // O^T += V^T P^T.
#pragma unroll
    for (int a = 0; a < MT; ++a) {
      uint32_t pb[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        pb[n][0] = transpose8(pack_f16(sc[a][n][0], sc[a][n][1]));
        pb[n][1] = transpose8(pack_f16(sc[a][n][2], sc[a][n][3]));
      }
      const int t0 = 16 * a + (2 * t ^ (t & 1)), t1 = t0 ^ 1;  // rows 2t and 2t + 1; with 8 more each
      uint32_t w[4][WV];
      const uint8_t* row[4] = {sv + t0 * C::CODE_ROW, sv + t1 * C::CODE_ROW, sv + (t0 + 8) * C::CODE_ROW,
                               sv + (t1 + 8) * C::CODE_ROW};
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
      const uint8_t* ss0 = sv + C::OFF_SCALE + t0 * C::SCALE_ROW;
      const uint8_t* ss1 = sv + C::OFF_SCALE + t1 * C::SCALE_ROW;
#pragma unroll
      for (int i = 0; i < WV; ++i) {
        // The scales of channels 8i.. of the lane's D/8, at tokens (t0, t1) and (t0 + 8, t1 + 8).
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
              s2[hw][0] = kv4_scale_pair(ss0[grp], ss1[grp]);
              s2[hw][1] = kv4_scale_pair(ss0[8 * C::SCALE_ROW + grp], ss1[8 * C::SCALE_ROW + grp]);
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

    __syncwarp();
    copy_v(stage);
    if (++stage == S) {
      stage = 0;
      phase ^= 1;
    }

    const bool last_unit = !C::SOLO && cur.u == cur.units - 1;
    if (last_unit || left == 1) {
      const bool first_here = began >= share.x0;  // the triple began in this warp's range
      const bool direct = C::SOLO ? cur.units == 1 : last_unit && first_here;
      // Slot 1: the triple begins in this range and goes on; slot 0: it began before.
      const size_t part = (size_t)me * 2 + (first_here ? 1 : 0);
      if (!C::SOLO && first_here && lane == 0) {
        // (and the warps after this one that the rest of the triple goes to)
        const int count = direct ? 0 : share.parts(me, (int)(began + cur.units - (share.x0 + units)));
        p.cuts[((size_t)cur.b * p.Hkv + cur.kvh) * p.row_tiles + cur.rt] = make_int2(me, count);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float s = l[n][j];
          s += __shfl_xor_sync(0xffffffffu, s, 4);
          s += __shfl_xor_sync(0xffffffffu, s, 8);
          s += __shfl_xor_sync(0xffffffffu, s, 16);
          const int rr = 8 * n + 2 * t + j;
          const int r = cur.rt * C::ROWS + rr;
          const int i = r / p.G, h = cur.kvh * p.G + r - i * p.G;
          if (i >= cur.nq) continue;
          if (!direct) {
            float* const po = C::SOLO ? reinterpret_cast<float*>(ring) : p.part_o + part * C::ROWS * D;
            float* const pml = C::SOLO ? reinterpret_cast<float*>(ring) + C::ROWS * D : p.part_ml + part * C::ROWS * 2;
            float* dst = po + rr * D + g * (D / 8);
#pragma unroll
            for (int c = 0; c < C::CT; c += 2)
              *reinterpret_cast<float4*>(dst + 2 * c) =
                  make_float4(acc[n][c][j], acc[n][c][2 + j], acc[n][c + 1][j], acc[n][c + 1][2 + j]);
            if (g == 0) *reinterpret_cast<float2*>(pml + 2 * rr) = make_float2(m[n][j], s);
          } else {
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
      fresh = true;
      began += cur.units;
    }
    if (left > 1) {
      if constexpr (C::SOLO) cur.u += C::WARPS;
      else kv4_advance<C>(p, req, cur);
    }
  }
  // A warp that gave up lets its copies land before the block can exit.
  if (left > 0) {
    const int v_units = units - ahead, k_units = v_units + (k_alone ? 1 : 0);
    for (int i = max(k_units - S, 0); i < k_units; ++i) wait_done(bars + 16 * (i % S), (uint32_t)((i / S) & 1));
    for (int i = max(v_units - S, 0); i < v_units; ++i) wait_done(bars + 16 * (i % S) + 8, (uint32_t)((i / S) & 1));
  }
  if constexpr (C::SOLO) {
    // The warps' parts of the triple, a row a warp at a time.
    if (cur.units == 1) return;
    __syncthreads();
    if (*abort_flag) return;
    const int parts = min(C::WARPS, cur.units), rows = min(C::ROWS, cur.nq * p.G - cur.rt * C::ROWS);
    for (int rr = warp; rr < rows; rr += C::WARPS) {
      auto part = [&](int w) -> const float* { return reinterpret_cast<const float*>(smem + w * C::RING); };
      float top = -INFINITY, sum = 0.f;
      for (int w = 0; w < parts; ++w) top = fmaxf(top, part(w)[C::ROWS * D + 2 * rr]);
      const float under = top == -INFINITY ? 0.f : top;
      for (int w = 0; w < parts; ++w)
        sum += ex2(part(w)[C::ROWS * D + 2 * rr] - under) * part(w)[C::ROWS * D + 2 * rr + 1];
      const float inv = sum == 0.f ? 0.f : p.v_gain / sum;
      const int r = cur.rt * C::ROWS + rr;
      const int i = r / p.G, h = cur.kvh * p.G + r - i * p.G;
      uint16_t* dst = p.o + (long long)(cur.tok0 + i) * p.o_token + (long long)h * p.o_head;
      for (int col = 2 * lane; col < D; col += 64) {
        float a = 0.f, b = 0.f;
        for (int w = 0; w < parts; ++w) {
          const float wt = ex2(part(w)[C::ROWS * D + 2 * rr] - under);
          const float2 y = *reinterpret_cast<const float2*>(part(w) + rr * D + col);
          a += wt * y.x;
          b += wt * y.y;
        }
        *reinterpret_cast<uint32_t*>(dst + col) = pack_bf16(a * inv, b * inv);
      }
      if (lane == 0)
        p.lse[(long long)(cur.tok0 + i) * p.H + h] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
    }
  }
}

// Joins the parts of cut triples: with M the largest m of a row's parts,
// O = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s.  blockIdx.x is the triple, and
// blockIdx.y cuts its work further where there are few.  A warp takes 4*L channels of a
// row at a time: L lanes of four channels for each of 32/L sets of parts, eight parts in
// flight a lane, which are joined against the lane's own maximum; then the sets are, in a
// fixed order.  L = 32, 8 or 4, so that a lane rarely has more than eight parts.
// Latency bounds it: two dependent loads, the cut and the parts.
template <class C>
__global__ void __launch_bounds__(256, 2) kv4_merge_kernel(const __grid_constant__ Kv4AttnParams p) {
  constexpr int D = C::D;
  grid_dep_wait();
  const int2 cut = p.cuts[blockIdx.x];
  const int bk = blockIdx.x / p.row_tiles, rt = blockIdx.x - bk * p.row_tiles;
  const int b = bk / p.Hkv, kvh = bk - b * p.Hkv;
  Kv4Cursor c;
  kv4_lookup(p, b, c);
  const int rows = min(C::ROWS, c.nq * p.G - rt * C::ROWS);  // none: the triple does not exist
  const int parts = cut.y;
  if (rows <= 0 || parts == 0 || *reinterpret_cast<volatile const int*>(p.err) != 0) return;
  const int warp = warp_id(), lane = lane_id();
  const int log_lanes = parts <= 8 ? 5 : parts <= 32 ? 3 : 2;
  const int set = lane >> log_lanes, sets = 32 >> log_lanes;
  const int chunks = (D + (4 << log_lanes) - 1) / (4 << log_lanes);
#pragma unroll 1
  for (int item = blockIdx.y * 8 + warp; item < rows * chunks; item += 8 * gridDim.y) {
    const int rr = item / chunks;
    const int col = (((item - rr * chunks) << log_lanes) + (lane & ((1 << log_lanes) - 1))) * 4;
    const int load_col = min(col, D - 4);
    // Part s: slot 1 of its first warp, slot 0 of the later ones.
    auto slot = [&](int s) -> size_t { return (size_t)(2 * (cut.x + s) + (s == 0 ? 1 : 0)) * C::ROWS + rr; };
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float top = -INFINITY, sum = 0.f;
#pragma unroll 1
    for (int s0 = set; s0 < parts; s0 += 8 * sets) {
      float2 x[8];
      float4 y[8];
      float high = top;
#pragma unroll
      for (int k = 0; k < 8; ++k) {  // (loads without branches stay together)
        const size_t at = slot(min(s0 + k * sets, parts - 1));
        x[k] = *reinterpret_cast<const float2*>(p.part_ml + at * 2);
        y[k] = *reinterpret_cast<const float4*>(p.part_o + at * D + load_col);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (s0 + k * sets >= parts) x[k].x = -INFINITY;
        high = fmaxf(high, x[k].x);
      }
      const float under = high == -INFINITY ? 0.f : high;
      const float scale = ex2(top - under);
      top = high;
      sum *= scale;
      o.x *= scale, o.y *= scale, o.z *= scale, o.w *= scale;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float w = ex2(x[k].x - under);
        if (s0 + k * sets < parts) {  // (the weight of a row of NaN is NaN)
          sum += w * x[k].y;
          o.x += w * y[k].x;
          o.y += w * y[k].y;
          o.z += w * y[k].z;
          o.w += w * y[k].w;
        }
      }
    }
#pragma unroll 1
    for (int d = 16; d >> log_lanes; d >>= 1) {
      const float other = __shfl_xor_sync(0xffffffffu, top, d);
      const float high = fmaxf(top, other);
      const float under = high == -INFINITY ? 0.f : high;
      const float wa = ex2(top - under), wb = ex2(other - under);
      top = high;
      sum = wa * sum + wb * __shfl_xor_sync(0xffffffffu, sum, d);
      o.x = wa * o.x + wb * __shfl_xor_sync(0xffffffffu, o.x, d);
      o.y = wa * o.y + wb * __shfl_xor_sync(0xffffffffu, o.y, d);
      o.z = wa * o.z + wb * __shfl_xor_sync(0xffffffffu, o.z, d);
      o.w = wa * o.w + wb * __shfl_xor_sync(0xffffffffu, o.w, d);
    }
    if (set == 0 && col < D) {
      const int r = rt * C::ROWS + rr;
      const int i = r / p.G, h = kvh * p.G + r - i * p.G;
      const float inv = sum == 0.f ? 0.f : p.v_gain / sum;
      *reinterpret_cast<uint2*>(p.o + (long long)(c.tok0 + i) * p.o_token + (long long)h * p.o_head + col) =
          make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
      if (col == 0)
        p.lse[(long long)(c.tok0 + i) * p.H + h] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
    }
  }
}

}  // namespace fa
