// Norms and rotation of queries and keys, per head and in one pass: for training with
// their gradients, for serving on the way into the paged 4-bit cache.
//
//   r = (mean_c x_c^2 + eps)^-1/2,  n_c = x_c r w_c
//   pair (a, b) of channels:  y_a = n_a cos - n_b sin,  y_b = n_b cos + n_a sin
// with pairs (i, i + rot/2) or (2i, 2i + 1) of the first rot channels; the others are n.
//
// Lanes: a head's d channels are d/8 chunks of 16 bytes.  Lane u of the d/16 of a head
// holds chunks u and u + rot/16 (of the channels behind rot: chunk j and the one half of them on), so both
// members of every pair are its own, in either pairing, and the rotation needs no
// shuffle; chunk ^ 1, the other half of a 4-bit scale's group, is lane ^ 1's (rot is a multiple of
// 32).  A head's lanes are padded to a power of two for the sums of its squares.
// A warp takes one token and U times 32 lanes of its heads, all loads first, with the
// token's cosines and sines in registers: what bounds the passes is memory.  Measured at 16384 tokens, 32 heads and 8
// of 128, all channels turned: the pass 56 us (335 MB: 6.0 TB/s, of 6.8 that a copy reaches), the gradients 90 us (503 MB:
// 5.6 TB/s) and their sum 3, the append to the cache 66 us (354 MB: 5.4 TB/s); at 64 tokens the pass 1.9 us.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "fa_packed.h"
#include "kv4.cuh"
#include "kv4_host.h"

namespace fa {
namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct HeadRows {
  const uint16_t* in;
  uint16_t* out;  // (NULL: not wanted)
  long long in_token, in_head, out_token, out_head;
  const uint16_t* weight;  // bf16 [d], or NULL: no norm
  int heads;
};

struct RotateParams {
  HeadRows x[3];  // q, k, and (append) v, which is neither normed nor turned
  const float* rotary;  // [positions, rot]: cosines, then sines
  const int* position;
  int positions, rot, T;
  float eps;
  // Append to the 4-bit cache: of k and v.
  uint8_t* codes[2];
  uint8_t* scales[2];
  const long long* slots;
  float inv_gain[2];
  int page_log2;
  long long slot_end;
};

template <int D>
struct HeadLanes {
  static constexpr int LANES = D / 16;
  static constexpr int GROUP = LANES <= 4 ? 4 : LANES <= 8 ? 8 : LANES <= 16 ? 16 : 32;
  static constexpr int ROWS = 32 / GROUP;  // heads a warp takes at a time
  int u, chunk[2];
  bool active, turned;
  __device__ __forceinline__ explicit HeadLanes(int rot) {
    u = lane_id() % GROUP;
    active = u < LANES;
    const int rc = rot / 16;
    turned = u < rc;
    chunk[0] = turned ? u : u + rc;
    chunk[1] = turned ? u + rc : u + LANES;
    if (!active) chunk[0] = chunk[1] = 0;
  }
};

// Eight channels as four pairs of neighbours: the arithmetic goes two channels an instruction.
__device__ __forceinline__ void unpack8(const uint4& v, float2* x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
__device__ __forceinline__ uint4 pack8(const float2* x) {
  return make_uint4(pack_bf16(x[0].x, x[0].y), pack_bf16(x[1].x, x[1].y), pack_bf16(x[2].x, x[2].y),
                    pack_bf16(x[3].x, x[3].y));
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 neg2(float2 v) { return make_float2(-v.x, -v.y); }

// Cosines and sines of a lane's eight pairs (BACK: of the angles' negatives), from where load(i) gives the
// i-th four of the cosines, then of the sines.
struct Angles {
  float2 c[4], s[4];
};
template <bool BACK, class Load>
__device__ __forceinline__ void load_angles(Angles& a, Load load) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float4 c = load(h), s = load(2 + h);
    a.c[2 * h] = make_float2(c.x, c.y), a.c[2 * h + 1] = make_float2(c.z, c.w);
    a.s[2 * h] = make_float2(s.x, s.y), a.s[2 * h + 1] = make_float2(s.z, s.w);
    if (BACK) a.s[2 * h] = neg2(a.s[2 * h]), a.s[2 * h + 1] = neg2(a.s[2 * h + 1]);
  }
}
// Where in its row of the table the h-th four of a lane's angles begin.
template <int D, bool NEXT>
__device__ __forceinline__ int angle_at(const HeadLanes<D>& at, int h) {
  return NEXT ? 4 * at.chunk[h] : 8 * at.u + 4 * h;
}

// The sum of two products that are rounded on their own.  (An add.rn of single values is never taken together with a product;
// of pairs it is, even where both are written with their rounding: that gave other bits in two of 10^5 results.)
__device__ __forceinline__ float2 add_alone(float2 a, float2 b) {
  return make_float2(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y));
}

// Turns a lane's 16 channels (two chunks of 8).  Each product and sum is rounded on its own, in this order, so
// that the result is that of the formula's operations one after the other.
template <bool NEXT>
__device__ __forceinline__ void turn(float2* x, const Angles& a) {
  if constexpr (NEXT) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float c = i & 1 ? a.c[i / 2].y : a.c[i / 2].x, s = i & 1 ? a.s[i / 2].y : a.s[i / 2].x;
      x[i] = add_alone(fmul2(x[i], both(c)), fmul2(make_float2(x[i].y, x[i].x), make_float2(-s, s)));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 u = x[i], v = x[4 + i];
      x[i] = add_alone(fmul2(u, a.c[i]), fmul2(v, neg2(a.s[i])));
      x[4 + i] = add_alone(fmul2(v, a.c[i]), fmul2(u, a.s[i]));
    }
  }
}

template <int D>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int d = HeadLanes<D>::GROUP / 2; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

// blockIdx.x: eight tokens, one a warp; blockIdx.y: U steps of ROWS heads, those of q, then k, then v
// (a step is of one kind, so what differs between the kinds is the same for a warp).
template <int D, bool NEXT, bool APPEND, int U>
__global__ void __launch_bounds__(256, 4) rotate_kernel(const __grid_constant__ RotateParams p) {
  using L = HeadLanes<D>;
  grid_dep_wait();
  const int tok = blockIdx.x * 8 + warp_id();
  if (tok >= p.T) return;
  const int pos = p.position[tok];  // (the rows do not wait for it)
  long long slot = -1;
  if constexpr (APPEND) slot = p.slots[tok];
  const L at(p.rot);
  const int sub = lane_id() / L::GROUP;
  const int steps[2] = {(p.x[0].heads + L::ROWS - 1) / L::ROWS, (p.x[1].heads + L::ROWS - 1) / L::ROWS};
  auto kind_of = [&](int step) { return step < steps[0] ? 0 : !APPEND || step < steps[0] + steps[1] ? 1 : 2; };
  auto head_of = [&](int step, int kind) {
    return (step - (kind > 0 ? steps[0] : 0) - (kind > 1 ? steps[1] : 0)) * L::ROWS + sub;
  };
  uint4 raw[U][2];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int step = blockIdx.y * U + i, kind = kind_of(step), head = head_of(step, kind);
    const HeadRows& x = p.x[kind];
    const uint16_t* src = x.in + tok * x.in_token + head * x.in_head;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      raw[i][h] = make_uint4(0u, 0u, 0u, 0u);
      if (at.active && head < x.heads) raw[i][h] = *reinterpret_cast<const uint4*>(src + 8 * at.chunk[h]);
    }
  }
  if (pos < 0 || pos >= p.positions) return;  // a token without a position is left out
  Angles angles;
  if (at.turned) {
    const float* row = p.rotary + (long long)pos * p.rot;
    load_angles<false>(angles, [&](int i) {
      return *reinterpret_cast<const float4*>(row + (i >> 1) * (p.rot / 2) + angle_at<D, NEXT>(at, i & 1));
    });
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int step = blockIdx.y * U + i, kind = kind_of(step), head = head_of(step, kind);
    const HeadRows& row = p.x[kind];
    const bool have = at.active && head < row.heads;
    if (kind < 2) {
      float2 x[8];
      unpack8(raw[i][0], x);
      unpack8(raw[i][1], x + 4);
      if (row.weight != nullptr) {
        float2 sum = make_float2(0.f, 0.f), w[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) unpack8(*reinterpret_cast<const uint4*>(row.weight + 8 * at.chunk[h]), w + 4 * h);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum = ffma2(x[e], x[e], sum);
        const float r = rsqrtf(head_sum<D>(sum.x + sum.y) * (1.f / D) + p.eps);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = fmul2(fmul2(x[e], both(r)), w[e]);
      }
      if (at.turned) turn<NEXT>(x, angles);
      raw[i][0] = pack8(x), raw[i][1] = pack8(x + 4);
      if (have && row.out != nullptr) {
        uint16_t* dst = row.out + tok * row.out_token + head * row.out_head;
#pragma unroll
        for (int h = 0; h < 2; ++h) *reinterpret_cast<uint4*>(dst + 8 * at.chunk[h]) = raw[i][h];
      }
    }
    if constexpr (APPEND) {
      if (kind > 0) {
        const int kv = kind - 1;
        const bool store = have && slot >= 0 && slot < p.slot_end;
        const long long cell = (((slot >> p.page_log2) * row.heads + head) << p.page_log2) +
                               (slot & ((1 << p.page_log2) - 1));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t w[4] = {raw[i][h].x, raw[i][h].y, raw[i][h].z, raw[i][h].w};
          uint32_t scale;
          const uint32_t codes = kv4_quantise(w, p.inv_gain[kv], scale);
          if (store) {
            *reinterpret_cast<uint32_t*>(p.codes[kv] + cell * (D / 2) + at.chunk[h] * 4) = codes;
            if (!(at.u & 1)) p.scales[kv][cell * (D / 16) + (at.chunk[h] >> 1)] = (uint8_t)scale;
          }
        }
      }
    }
  }
}

// Gradients.  With g = R^T dy, z = w g and xhat = x r:
//   dx = r (z - xhat mean_c(xhat z)),  dw = sum over tokens and heads of g xhat
struct RotateBwdParams {
  HeadRows dy[2], x[2];  // dy: in the gradient of the result, out the gradient of x; x: in the pass's input
  const float* rotary;
  const int* position;
  int positions, rot, T;
  float eps;
  int q_blocks;  // blocks of the grid that take q; the others take k
  float* part;   // [blocks][d]: each block's sum of g xhat (NULL: no weights)
};

constexpr int kRotateBack = 2;  // steps of heads a warp takes at a time

// A block takes q or k; its warps walk tokens (and runs of U steps of heads), keeping the weight's
// gradient of their channels in registers, all loads of a run first.  Tokens without a position have a
// gradient of zero.
template <int D, bool NEXT>
__global__ void __launch_bounds__(256, 2) rotate_bwd_kernel(const __grid_constant__ RotateBwdParams p) {
  using L = HeadLanes<D>;
  constexpr int U = kRotateBack;
  __shared__ float sums[8][D];
  grid_dep_wait();
  const L at(p.rot);
  const int warp = warp_id(), lane = lane_id();  // (a shuffle of the whole warp: never inside a branch)
  const int kind = (int)blockIdx.x < p.q_blocks ? 0 : 1;
  const int block = kind ? blockIdx.x - p.q_blocks : blockIdx.x, blocks = kind ? gridDim.x - p.q_blocks : p.q_blocks;
  const HeadRows &gy = p.dy[kind], &xx = p.x[kind];
  const bool normed = xx.weight != nullptr;
  const int runs = (gy.heads + U * L::ROWS - 1) / (U * L::ROWS), sub = lane / L::GROUP;
  float2 dw[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) dw[e] = make_float2(0.f, 0.f);
  uint4 rw[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
  if (normed) {
#pragma unroll
    for (int h = 0; h < 2; ++h) rw[h] = *reinterpret_cast<const uint4*>(xx.weight + 8 * at.chunk[h]);
  }
  // A run: its token and place in the token; the next of this warp is 8 * blocks runs on (without a division each).
  struct Run {
    int tok, at;
  };
  const int tok_step = runs > 0 ? 8 * blocks / runs : 0, at_step = 8 * blocks - tok_step * runs;
  auto after = [&](Run j) {
    j.tok += tok_step, j.at += at_step;
    if (j.at >= runs) j.at -= runs, ++j.tok;
    return j;
  };
  auto position = [&](Run j) { return j.tok < p.T ? p.position[j.tok] : -1; };
  auto is_live = [&](int pos) { return pos >= 0 && pos < p.positions; };
  const int begin = block * 8 + warp;
  Run job = {runs > 0 ? begin / runs : p.T, runs > 0 ? begin % runs : 0}, next = after(job);
  int pos = position(job);
  while (job.tok < p.T) {
    const int tok = job.tok, first = job.at * U * L::ROWS + sub;
    if (!is_live(pos)) {  // (not as zeros through what follows: 0 times a weight that is not finite is a NaN)
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int head = first + i * L::ROWS;
        if (!at.active || head >= gy.heads) continue;
        uint16_t* dst = gy.out + tok * gy.out_token + head * gy.out_head;
#pragma unroll
        for (int h = 0; h < 2; ++h) *reinterpret_cast<uint4*>(dst + 8 * at.chunk[h]) = make_uint4(0u, 0u, 0u, 0u);
      }
      pos = position(next);
      job = next, next = after(next);
      continue;
    }
    uint4 rg[U][2], rx[U][2];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int head = first + i * L::ROWS;
      const bool have = at.active && head < gy.heads;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        rg[i][h] = rx[i][h] = make_uint4(0u, 0u, 0u, 0u);
        if (have) {
          rg[i][h] = *reinterpret_cast<const uint4*>(gy.in + tok * gy.in_token + head * gy.in_head + 8 * at.chunk[h]);
          if (normed)
            rx[i][h] = *reinterpret_cast<const uint4*>(xx.in + tok * xx.in_token + head * xx.in_head + 8 * at.chunk[h]);
        }
      }
    }
    Angles angles;
    if (at.turned) {
      const float* row = p.rotary + (long long)pos * p.rot;
      load_angles<true>(angles, [&](int i) {
        return *reinterpret_cast<const float4*>(row + (i >> 1) * (p.rot / 2) + angle_at<D, NEXT>(at, i & 1));
      });
    }
    pos = position(next);  // (a run ahead: the next one's loads do not wait for it)
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int head = first + i * L::ROWS;
      float2 g[8];
#pragma unroll
      for (int h = 0; h < 2; ++h) unpack8(rg[i][h], g + 4 * h);
      if (at.turned) turn<NEXT>(g, angles);
      if (normed) {
        float2 x[8], z[8], sum = make_float2(0.f, 0.f), dot = make_float2(0.f, 0.f);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          unpack8(rx[i][h], x + 4 * h);
          unpack8(rw[h], z + 4 * h);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          z[e] = fmul2(g[e], z[e]);
          sum = ffma2(x[e], x[e], sum);
          dot = ffma2(x[e], z[e], dot);
        }
        const float total = head_sum<D>(sum.x + sum.y), inner = head_sum<D>(dot.x + dot.y);
        // (a head that is not there must not turn eps = 0 into 0 * inf)
        const float r = head < gy.heads ? rsqrtf(total * (1.f / D) + p.eps) : 0.f;
        const float2 m = both(-inner * r * (1.f / D)), r2 = both(r);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 unit = fmul2(x[e], r2);
          dw[e] = ffma2(g[e], unit, dw[e]);
          g[e] = fmul2(r2, ffma2(unit, m, z[e]));
        }
      }
      if (at.active && head < gy.heads) {
        uint16_t* dst = gy.out + tok * gy.out_token + head * gy.out_head;
#pragma unroll
        for (int h = 0; h < 2; ++h) *reinterpret_cast<uint4*>(dst + 8 * at.chunk[h]) = pack8(g + 4 * h);
      }
    }
    job = next, next = after(next);
  }
  if (p.part == nullptr) return;
  // The lanes that hold the same channels, then the warps, in a fixed order.
#pragma unroll
  for (int d = L::GROUP; d < 32; d <<= 1)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      dw[e].x += __shfl_xor_sync(0xffffffffu, dw[e].x, d);
      dw[e].y += __shfl_xor_sync(0xffffffffu, dw[e].y, d);
    }
  if (lane < L::GROUP && at.active)
#pragma unroll
    for (int e = 0; e < 8; ++e)
      *reinterpret_cast<float2*>(&sums[warp][8 * at.chunk[e >> 2] + 2 * (e & 3)]) = dw[e];
  __syncthreads();
  for (int e = threadIdx.x; e < D; e += 256) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v += sums[i][e];
    p.part[(long long)blockIdx.x * D + e] = v;
  }
}

struct RotateSumParams {
  const float* part;
  float* out[2];
  int q_blocks, blocks, d;
};

// A weight's gradient: the blocks' sums, 32 columns a block (blockIdx.x) of q or k (blockIdx.y), each of 32 rows
// of threads adding every 32nd, in a fixed order.  Latency bounds it.
__global__ void __launch_bounds__(1024) rotate_sum_kernel(const __grid_constant__ RotateSumParams p) {
  __shared__ float sums[32][33];
  grid_dep_wait();
  const int kind = blockIdx.y, col = blockIdx.x * 32 + threadIdx.x % 32, row = threadIdx.x / 32;
  if (p.out[kind] == nullptr) return;
  const int b0 = kind ? p.q_blocks : 0, b1 = kind ? p.blocks : p.q_blocks;
  float v = 0.f;
  for (int b = b0 + row; b < b1; b += 32) v += p.part[(long long)b * p.d + col];
  sums[row][threadIdx.x % 32] = v;
  __syncthreads();
  if (row == 0) {
    float total = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) total += sums[i][threadIdx.x];
    p.out[kind][col] = total;
  }
}

fa_status rows_checks(const fa_rows& r, int heads) {
  if (heads == 0) return FA_OK;
  if (!r.data) return FA_ERR_INVALID_ARG;
  return aligned16(r.data) && !(r.token & 7) && !(r.head & 7) ? FA_OK : FA_ERR_MISALIGNED;
}

// A: any of the argument structures.
template <class A>
fa_status rotary_checks(const A& a, int Hkv, int d) {
  const int T = a.T, H = a.H, positions = a.positions, rot = a.rot, interleaved = a.interleaved;
  const float eps = a.eps;
  const float* rotary = a.rotary;
  const int* position = a.position;
  if (T < 0 || H < 0 || Hkv < 0 || positions < 0 || rot < 0 || (interleaved != 0 && interleaved != 1))
    return FA_ERR_INVALID_ARG;
  if (!std::isfinite(eps) || eps < 0.f) return FA_ERR_INVALID_ARG;
  if (padded_head_dim(d) == 0) return FA_ERR_UNSUPPORTED;
  if (rot > d || rot % 32 != 0) return FA_ERR_UNSUPPORTED;
  if (T > (1 << 30) || (long long)H + 2LL * Hkv > 65535) return FA_ERR_INVALID_ARG;
  if (T == 0 || H + Hkv == 0) return FA_OK;
  if (!position || (rot > 0 && positions > 0 && !rotary)) return FA_ERR_INVALID_ARG;
  if (!aligned16(rotary) || !aligned16(a.q_weight) || !aligned16(a.k_weight) || !all_aligned(4, position))
    return FA_ERR_MISALIGNED;
  return FA_OK;
}

HeadRows head_rows(const fa_rows& in, const fa_rows& out, const void* weight, int heads) {
  return {static_cast<const uint16_t*>(in.data), static_cast<uint16_t*>(const_cast<void*>(out.data)), in.token, in.head,
          out.token, out.head, static_cast<const uint16_t*>(weight), heads};
}

template <class A>
void rotate_fill(RotateParams& p, const A& a, int Hkv) {
  p.x[0] = head_rows(a.q, a.q_out, a.q_weight, a.H);
  p.x[1] = head_rows(a.k, a.k_out, a.k_weight, Hkv);
  p.rotary = a.rotary, p.position = a.position, p.positions = a.positions, p.rot = a.rot, p.T = a.T, p.eps = a.eps;
}

// Steps of heads a warp: kRotateSteps where that leaves 32 warps an SM, else one.  Measured at the sizes above with
// 1 / 2 / 4 steps: the pass 71 / 62 / 66 us, the append 80 / 68 / 75 (before the arithmetic went two channels an
// instruction); two keep 2 KB of loads in flight a warp, four cost occupancy in registers.
constexpr int kRotateSteps = 2;
template <int D, bool NEXT, bool APPEND>
fa_status run_rotate(const RotateParams& p, cudaStream_t st) {
  constexpr int ROWS = HeadLanes<D>::ROWS;
  int steps = 0;
  for (int i = 0; i < (APPEND ? 3 : 2); ++i) steps += (p.x[i].heads + ROWS - 1) / ROWS;
  const int kind = APPEND ? FA_KERNEL_KV4_APPEND : FA_KERNEL_ROTATE;
  const unsigned gx = (unsigned)((p.T + 7) / 8);
  const int runs = (steps + kRotateSteps - 1) / kRotateSteps;
  if ((long long)p.T * runs >= 32LL * sm_count_cached())
    return launch(kind, rotate_kernel<D, NEXT, APPEND, kRotateSteps>, dim3(gx, runs), dim3(256), 0, st, p);
  return launch(kind, rotate_kernel<D, NEXT, APPEND, 1>, dim3(gx, steps), dim3(256), 0, st, p);
}

template <bool APPEND>
fa_status rotate_by_dim(const RotateParams& p, int d, int interleaved, cudaStream_t st) {
  switch (d) {
    case 64: return interleaved ? run_rotate<64, true, APPEND>(p, st) : run_rotate<64, false, APPEND>(p, st);
    case 96: return interleaved ? run_rotate<96, true, APPEND>(p, st) : run_rotate<96, false, APPEND>(p, st);
    case 128: return interleaved ? run_rotate<128, true, APPEND>(p, st) : run_rotate<128, false, APPEND>(p, st);
    case 192: return interleaved ? run_rotate<192, true, APPEND>(p, st) : run_rotate<192, false, APPEND>(p, st);
    case 256: return interleaved ? run_rotate<256, true, APPEND>(p, st) : run_rotate<256, false, APPEND>(p, st);
    case 384: return interleaved ? run_rotate<384, true, APPEND>(p, st) : run_rotate<384, false, APPEND>(p, st);
  }
  return FA_ERR_UNSUPPORTED;
}

// Blocks an SM of the gradients' kernel: those that fit with two steps' loads in registers.  Measured at the sizes above:
// two steps and two blocks 90 us, two and three (spilling) 139, one and three 123, one and four 165.
constexpr int kRotateBlocks = 2;

int rotate_bwd_blocks(int T, int H, int Hkv) {
  const long long most = ((long long)T * (H + Hkv) + 7) / 8;  // no more than rows
  return (int)std::max(2LL, std::min<long long>(most, (long long)kRotateBlocks * sm_count_cached()));
}

template <int D, bool NEXT>
fa_status run_rotate_bwd(RotateBwdParams p, int blocks, float* dwq, float* dwk, cudaStream_t st) {
  fa_status s = launch(FA_KERNEL_ROTATE_BWD, rotate_bwd_kernel<D, NEXT>, dim3(blocks), dim3(256), 0, st, p);
  if (s != FA_OK || p.part == nullptr) return s;
  const RotateSumParams q = {p.part, {dwq, dwk}, p.q_blocks, blocks, D};
  return launch(FA_KERNEL_ROTATE_SUM, rotate_sum_kernel, dim3(D / 32, 2), dim3(1024), 0, st, q);
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

fa_status fa_qk_norm_rope(const fa_qk_norm_rope_args* a) {
  if (!a) return FA_ERR_INVALID_ARG;
  fa_status s = rotary_checks(*a, a->Hkv, a->d);
  if (s != FA_OK) return s;
  if (a->T == 0 || a->H + a->Hkv == 0) return FA_OK;
  for (const fa_rows* r : {&a->q, &a->q_out})
    if ((s = rows_checks(*r, a->H)) != FA_OK) return s;
  for (const fa_rows* r : {&a->k, &a->k_out})
    if ((s = rows_checks(*r, a->Hkv)) != FA_OK) return s;
  RotateParams p = {};
  rotate_fill(p, *a, a->Hkv);
  return rotate_by_dim<false>(p, a->d, a->interleaved, (cudaStream_t)a->stream);
}

fa_status fa_kv4_append(const fa_kv4_append_args* a) {
  if (!a) return FA_ERR_INVALID_ARG;
  const fa_kv4_cache* cache = a->cache;
  fa_status s = kv4_cache_checks(cache);
  if (s != FA_OK) return s;
  const int Hkv = cache->Hkv;
  if ((s = rotary_checks(*a, Hkv, cache->d)) != FA_OK) return s;
  if (a->T == 0 || a->H + Hkv == 0) return FA_OK;
  for (const fa_rows* r : {&a->q, &a->q_out})
    if ((s = rows_checks(*r, a->H)) != FA_OK) return s;
  for (const fa_rows* r : {&a->k, &a->v})
    if ((s = rows_checks(*r, Hkv)) != FA_OK) return s;
  if (a->k_out.data && (s = rows_checks(a->k_out, Hkv)) != FA_OK) return s;
  if (!a->slots) return FA_ERR_INVALID_ARG;
  if (!all_aligned(8, a->slots)) return FA_ERR_MISALIGNED;
  RotateParams p = {};
  rotate_fill(p, *a, Hkv);
  p.x[2] = head_rows(a->v, {}, nullptr, Hkv);
  p.codes[0] = static_cast<uint8_t*>(cache->k_codes), p.codes[1] = static_cast<uint8_t*>(cache->v_codes);
  p.scales[0] = static_cast<uint8_t*>(cache->k_scales), p.scales[1] = static_cast<uint8_t*>(cache->v_scales);
  p.slots = a->slots;
  p.inv_gain[0] = 1.f / cache->k_gain, p.inv_gain[1] = 1.f / cache->v_gain;
  p.page_log2 = page_log2_of(cache->page);
  p.slot_end = (long long)cache->pages * cache->page;
  return rotate_by_dim<true>(p, cache->d, a->interleaved, (cudaStream_t)a->stream);
}

size_t fa_qk_norm_rope_bwd_workspace_size(int T, int H, int Hkv, int d) {
  if (T <= 0 || H < 0 || Hkv < 0 || H + (long long)Hkv == 0 || padded_head_dim(d) == 0) return 0;
  return (size_t)rotate_bwd_blocks(T, H, Hkv) * d * sizeof(float);
}

fa_status fa_qk_norm_rope_bwd(const fa_qk_norm_rope_bwd_args* a) {
  if (!a) return FA_ERR_INVALID_ARG;
  const int T = a->T, H = a->H, Hkv = a->Hkv, d = a->d;
  fa_status s = rotary_checks(*a, Hkv, d);
  if (s != FA_OK) return s;
  // A weight's gradient is written where there is the weight.
  if ((a->q_weight && !a->dq_weight) || (a->k_weight && !a->dk_weight)) return FA_ERR_INVALID_ARG;
  if (!all_aligned(4, a->dq_weight, a->dk_weight)) return FA_ERR_MISALIGNED;
  const cudaStream_t st = (cudaStream_t)a->stream;
  float *const wq_out = a->q_weight ? a->dq_weight : nullptr, *const wk_out = a->k_weight ? a->dk_weight : nullptr;
  if (T == 0 || H + Hkv == 0) {
    for (float* w : {wq_out, wk_out})
      if (w) {
        const cudaError_t e = cudaMemsetAsync(w, 0, d * sizeof(float), st);
        if (e != cudaSuccess) return record_cuda_error(e);
      }
    return FA_OK;
  }
  for (const fa_rows* r : {&a->dq_out, &a->dq})
    if ((s = rows_checks(*r, H)) != FA_OK) return s;
  for (const fa_rows* r : {&a->dk_out, &a->dk})
    if ((s = rows_checks(*r, Hkv)) != FA_OK) return s;
  if ((a->q_weight && (s = rows_checks(a->q, H)) != FA_OK) || (a->k_weight && (s = rows_checks(a->k, Hkv)) != FA_OK))
    return s;
  const int blocks = rotate_bwd_blocks(T, H, Hkv);
  const bool weights = wq_out || wk_out;
  if (weights && (!a->workspace || !all_aligned(256, static_cast<char*>(a->workspace)) ||
                  a->workspace_bytes < (size_t)blocks * d * sizeof(float)))
    return FA_ERR_WORKSPACE;
  RotateBwdParams p = {};
  p.dy[0] = head_rows(a->dq_out, a->dq, nullptr, H);
  p.dy[1] = head_rows(a->dk_out, a->dk, nullptr, Hkv);
  p.x[0] = head_rows(a->q, {}, a->q_weight, H);
  p.x[1] = head_rows(a->k, {}, a->k_weight, Hkv);
  p.rotary = a->rotary, p.position = a->position, p.positions = a->positions, p.rot = a->rot, p.T = T, p.eps = a->eps;
  // Blocks by the bytes of each: a head costs more where it has a norm, whose input is read.
  const double wq = H * (wq_out ? 3.0 : 2.0), wk = Hkv * (wk_out ? 3.0 : 2.0);
  p.q_blocks = std::min(blocks - 1, std::max(1, (int)std::lround(blocks * wq / (wq + wk))));
  p.part = weights ? static_cast<float*>(a->workspace) : nullptr;
  const auto run = [&](auto next) -> fa_status {
    constexpr bool NEXT = decltype(next)::value;
    switch (d) {
      case 64: return run_rotate_bwd<64, NEXT>(p, blocks, wq_out, wk_out, st);
      case 96: return run_rotate_bwd<96, NEXT>(p, blocks, wq_out, wk_out, st);
      case 128: return run_rotate_bwd<128, NEXT>(p, blocks, wq_out, wk_out, st);
      case 192: return run_rotate_bwd<192, NEXT>(p, blocks, wq_out, wk_out, st);
      case 256: return run_rotate_bwd<256, NEXT>(p, blocks, wq_out, wk_out, st);
      case 384: return run_rotate_bwd<384, NEXT>(p, blocks, wq_out, wk_out, st);
    }
    return FA_ERR_UNSUPPORTED;
  };
  return a->interleaved ? run(std::true_type{}) : run(std::false_type{});
}

}  // extern "C"
