// Page tables and slots from request lengths, and the 4-bit cache's store and load.
#include <algorithm>
#include <cmath>
#include <cuda_bf16.h>

#include "fa_paged.h"
#include "kv4.cuh"
#include "kv4_host.h"

namespace fa {
namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// ------------------------------------------------------------------ page tables

struct PageParams {
  const int* held;   // tokens held (grow) or first position (slots only)
  const int* add;    // tokens to place
  int* table;
  const int* free_pages;  // (NULL: an empty stack)
  const int* free_count;
  long long* slots;
  int* cu;
  int* held_out;
  int* count_out;
  int B, width, page_log2, T, free_size;
  int per_block;  // requests per block (grid.x)
  bool grow;      // else slots only
};

constexpr int kPageThreads = 256;

struct PageRow {
  long long off;  // pages that the requests before need
  int held, add, cu, owned, need;
};

// Exclusive scan of one value a thread over the block; total through `total`.
__device__ __forceinline__ long long block_scan(long long x, long long* warp_sums, long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long s = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, s, d);
    if (lane >= d) s += y;
  }
  if (lane == 31) warp_sums[warp] = s;
  __syncthreads();
  long long before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kPageThreads / 32; ++w) {
    if (w < warp) before += warp_sums[w];
    total += warp_sums[w];
  }
  __syncthreads();
  return before + s - x;
}

// Everything follows from two prefix sums over the requests: of the new tokens
// (cut at T) and of the pages they need.  The latency of the sums bounds it (3.1 us for 512
// requests of a token, 4.0 for 256 prompts of 512 on average), and is less than a second launch
// would take, so every block computes both over all requests (each thread a run of ceil(B / 256) of them) and then fills in
// its own `per_block` requests; blockIdx.y cuts the tokens of long prompts.  The page of a
// new token comes from the old table or from the stack, never from an entry that
// this launch writes, so blocks do not wait for one another.
__global__ void __launch_bounds__(kPageThreads) page_kernel(const __grid_constant__ PageParams p) {
  extern __shared__ long long warp_sums[];  // a word a warp, then per_block rows
  PageRow* rows = reinterpret_cast<PageRow*>(warp_sums + kPageThreads / 32);
  grid_dep_wait();
  const int page = 1 << p.page_log2;
  const int run = (p.B + kPageThreads - 1) / kPageThreads;
  const int b0 = min((int)threadIdx.x * run, p.B), b1 = min(b0 + run, p.B);
  long long sum = 0, total_new, total_need = 0;
  for (int b = b0; b < b1; ++b) sum += max(p.add[b], 0);
  const long long new0 = block_scan(sum, warp_sums, total_new);
  const int my0 = blockIdx.x * p.per_block, my1 = min(my0 + p.per_block, p.B);

  // One request: its tokens after the cut at T, and the pages they need.
  auto place = [&](int b, long long raw, int& held, int& cu, int& add, int& owned) -> int {
    held = max(p.held[b], 0);
    cu = (int)min(raw, (long long)p.T);
    add = (int)(min(raw + max(p.add[b], 0), (long long)p.T) - cu);
    owned = (held >> p.page_log2) + ((held & (page - 1)) ? 1 : 0);
    const long long wanted = min(((long long)held + add + page - 1) >> p.page_log2, (long long)p.width);
    return p.grow ? (int)max(wanted - owned, 0LL) : 0;
  };
  long long need_sum = 0, raw = new0;
  for (int b = b0; b < b1; ++b) {
    int held, cu, add, owned;
    need_sum += place(b, raw, held, cu, add, owned);
    raw += max(p.add[b], 0);
  }
  long long off = 0;
  if (p.grow) off = block_scan(need_sum, warp_sums, total_need);
  raw = new0;
  for (int b = b0; b < b1; ++b) {
    int held, cu, add, owned;
    const int need = place(b, raw, held, cu, add, owned);
    raw += max(p.add[b], 0);
    if (b >= my0 && b < my1) rows[b - my0] = PageRow{off, held, add, cu, owned, need};
    off += need;
  }
  const int count = p.grow ? min(max(*p.free_count, 0), p.free_size) : 0;
  const int total = (int)min(total_new, (long long)p.T);
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) {
    p.cu[p.B] = total;
    if (p.count_out) *p.count_out = (int)max((long long)count - total_need, 0LL);
  }
  __syncthreads();

  // A warp takes a request; blockIdx.y takes every gridDim.y-th run of 32 tokens.
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int b = my0 + warp; b < my1; b += kPageThreads / 32) {
    const PageRow r = rows[b - my0];
    int* entry = p.table + (size_t)b * p.width;
    if (blockIdx.y == 0) {
      if (lane == 0) {
        p.cu[b] = r.cu;
        if (p.held_out) {
          const int given = (int)min(max(count - r.off, 0LL), (long long)r.need);
          const long long room = min((long long)r.owned + given, (long long)p.width) * page - r.held;
          p.held_out[b] = r.held + (int)max(min(room, (long long)r.add), 0LL);
        }
      }
      for (int i = lane; i < r.need; i += 32) {
        const long long src = count - 1 - r.off - i;
        entry[r.owned + i] = src >= 0 ? p.free_pages[src] : -1;
      }
    }
    for (long long i = blockIdx.y * 32 + lane; i < r.add; i += 32 * gridDim.y) {
      const long long pos = r.held + i;
      const long long col = pos >> p.page_log2;
      int id = -1;
      if (col < p.width) {
        if (!p.grow || col < r.owned) {
          id = entry[col];
        } else {
          const long long src = count - 1 - r.off - (col - r.owned);
          id = src >= 0 ? p.free_pages[src] : -1;
        }
      }
      p.slots[r.cu + i] = id >= 0 ? ((long long)id << p.page_log2) + (pos & (page - 1)) : -1;
    }
  }
  // The rest of `slots`.
  const long long step = (long long)gridDim.x * gridDim.y * kPageThreads;
  for (long long t = total + ((long long)blockIdx.y * gridDim.x + blockIdx.x) * kPageThreads + threadIdx.x; t < p.T;
       t += step)
    p.slots[t] = -1;
}

fa_status run_pages(PageParams p, cudaStream_t st) {
  // Requests per block: eight (one a warp) until the grid covers the SMs twice.
  // Tokens: another block for every 64 of the mean request, within the same bound.
  const int cap = 2 * sm_count_cached();
  p.per_block = std::max(8, (p.B + cap - 1) / cap);
  const int gx = (p.B + p.per_block - 1) / p.per_block;
  const int gy = std::max(1, std::min(cap / gx, (int)((long long)p.T / std::max(1, p.B) / 64)));
  return launch(FA_KERNEL_PAGE, page_kernel, dim3(gx, gy), dim3(kPageThreads),
                kPageThreads / 32 * sizeof(long long) + p.per_block * sizeof(PageRow), st, p);
}

// At most 2^21 requests (a block keeps a row for each of its own in shared memory),
// and positions of 31 bits.
bool pages_ok(int B, int width, int page, int T) {
  return B >= 0 && B <= (1 << 21) && width >= 0 && T >= 0 && page_log2_of(page) >= 0 && (long long)width * page <= 0x7fffffffLL;
}


// ------------------------------------------------------------------ store and load

struct Kv4IoParams {
  const uint16_t* in[2];  // store: k, v
  long long token[2], head[2];
  uint16_t* out[2];  // load: k, v
  uint8_t* codes[2];
  uint8_t* scales[2];
  const long long* slots;
  float inv_gain[2], gain[2];
  int T, heads, page_log2;
  int pieces;    // runs of eight channels a token: heads * d / 8
  int per_warp;  // tokens a warp (above 1 only where a token has fewer than 32 pieces)
  long long slot_end;
};

// A lane's eight channels of token `tok`: head and run in the head, and the row of the
// cache (the token's slot, the head) that holds them.  blockIdx.y takes 32 pieces of a
// token, so a warp's accesses to the dense side are 512 contiguous bytes and there is no
// division by a length that is only known at run time.
template <int D>
struct Kv4Piece {
  int head, run, sub;
  bool have;
  __device__ __forceinline__ explicit Kv4Piece(const Kv4IoParams& p) {
    const int lane = lane_id();
    int piece = blockIdx.y * 32 + lane;
    sub = 0;
    have = piece < p.pieces;
    if (p.per_warp > 1) {
      sub = lane / p.pieces;
      piece = lane - sub * p.pieces;
      have = sub < p.per_warp;
    }
    head = piece / (D / 8);
    run = piece - head * (D / 8);
  }
  // -1: the token has no slot.
  __device__ __forceinline__ long long row(const Kv4IoParams& p, long long slot) const {
    if (slot < 0 || slot >= p.slot_end) return -1;
    const long long pg = slot >> p.page_log2;
    return ((pg * p.heads + head) << p.page_log2) + (slot & ((1 << p.page_log2) - 1));
  }
};

// A quotient is taken by a reciprocal and then cut to 12 bits after a push of 2^-13:
// where x has bf16's eight bits and the gain is a power of two, a quotient on the border
// of two results lands on it exactly, and any other is at least 2^-8 of itself away, so
// both scale and code are those of the exact quotient.
constexpr float kKv4Push = 1.f + 1.f / 8192.f;
__device__ __forceinline__ float cut12(float x) { return __uint_as_float(__float_as_uint(x) & 0xfffff000u); }

// Two lanes per group of 16 channels, which share its scale; keys and values, and U
// tokens a warp, together: what bounds it is the latency of a slot and then the rows,
// and then reading (2 bytes in for 0.5625 out) and the ALU pipe (68 % used): 16384 tokens of 8
// heads of 128, written and then read back, 32 us (172 MB, 5400 GB/s); 64 tokens, 2.9 us.
template <int D, int U>
__global__ void __launch_bounds__(256) kv4_store_kernel(const __grid_constant__ Kv4IoParams p) {
  grid_dep_wait();
  const Kv4Piece<D> at(p);
  const long long tok0 = ((long long)blockIdx.x * 8 + warp_id()) * U * p.per_warp + at.sub;
  long long slot[U];
  uint4 x[U][2];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const long long tok = tok0 + (long long)u * p.per_warp;
    const bool have = at.have && tok < p.T;
    slot[u] = have ? p.slots[tok] : -1;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      x[u][i] = make_uint4(0u, 0u, 0u, 0u);
      if (have)
        x[u][i] = *reinterpret_cast<const uint4*>(p.in[i] + tok * p.token[i] + at.head * p.head[i] + at.run * 8);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const long long row = at.row(p, slot[u]);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t w[4] = {x[u][i].x, x[u][i].y, x[u][i].z, x[u][i].w};
      uint32_t pair = 0;  // (a NaN is passed over)
#pragma unroll
      for (int k = 0; k < 4; ++k) asm("max.bf16x2 %0, %0, %1;" : "+r"(pair) : "r"(w[k] & 0x7fff7fffu));
      float top = fmaxf(__uint_as_float(pair << 16), __uint_as_float(pair & 0xffff0000u));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      uint16_t sb;
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
          : "=h"(sb)
          : "f"(0.f), "f"(cut12(top * p.inv_gain[i] * (kKv4Push / 6.f))));
      const uint32_t s = sb & 0xffu;
      // e4m3 to fp32 by way of f16 (2^-8 of the scale; exact).
      const float sf = __half2float(__ushort_as_half((unsigned short)((s & 0x7f) << 7))) * kKv4ScaleBias;
      float inv;
      asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(sf));
      const float mul = sf > 0.f ? inv * p.inv_gain[i] * kKv4Push : 0.f;
      uint32_t q[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float lo = cut12(__uint_as_float(w[k] << 16) * mul);
        const float hi = cut12(__uint_as_float(w[k] & 0xffff0000u) * mul);
        asm("{\n\t.reg .b8 x;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 x, %1, %2;\n\t"
            "cvt.u32.u8 %0, x;\n\t}"
            : "=r"(q[k])
            : "f"(hi), "f"(lo));
      }
      if (row >= 0) {
        *reinterpret_cast<uint32_t*>(p.codes[i] + row * (D / 2) + at.run * 4) =
            q[0] | (q[1] << 8) | (q[2] << 16) | (q[3] << 24);
        if (!(at.run & 1)) p.scales[i][row * (D / 16) + (at.run >> 1)] = (uint8_t)s;
      }
    }
  }
}

// The inverse, with the same split.  f16 products are exact, so the one rounding is the
// last, to bf16.  Writing bounds it: 65536 tokens of 4 heads of 128, 31.5 us (172 MB, 5470 GB/s);
// 1021 of 4 of 96, 1.7 us.
template <int D, int U>
__global__ void __launch_bounds__(256) kv4_load_kernel(const __grid_constant__ Kv4IoParams p) {
  grid_dep_wait();
  const Kv4Piece<D> at(p);
  const long long tok0 = ((long long)blockIdx.x * 8 + warp_id()) * U * p.per_warp + at.sub;
  if (!at.have) return;
  long long slot[U];
  uint32_t c[U][2], s[U][2];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const long long tok = tok0 + (long long)u * p.per_warp;
    slot[u] = tok < p.T ? p.slots[tok] : -1;
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const long long row = at.row(p, slot[u]);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      c[u][i] = s[u][i] = 0;
      if (row >= 0) {
        c[u][i] = *reinterpret_cast<const uint32_t*>(p.codes[i] + row * (D / 2) + at.run * 4);
        s[u][i] = p.scales[i][row * (D / 16) + (at.run >> 1)];
      }
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const long long tok = tok0 + (long long)u * p.per_warp;
    if (tok >= p.T) return;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t r[4], o[4];
      kv4_codes(c[u][i], r);
      const uint32_t s2 = kv4_scale_both(s[u][i]);
      const float gain = p.gain[i] * kKv4ScaleBias;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t v = h2mul(r[k], s2);
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v));
        o[k] = pack_bf16(f.x * gain, f.y * gain);
      }
      *reinterpret_cast<uint4*>(p.out[i] + (tok * p.heads + at.head) * D + at.run * 8) =
          make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

// Tokens a warp (per row of tokens): four where that still leaves 32 warps an SM, else one.
constexpr int kKv4Batch = 4;

fa_status kv4_io_fill(const fa_kv4_cache& c, const long long* slots, int T, Kv4IoParams& p, dim3& grid, bool& batch) {
  p.codes[0] = static_cast<uint8_t*>(c.k_codes);
  p.codes[1] = static_cast<uint8_t*>(c.v_codes);
  p.scales[0] = static_cast<uint8_t*>(c.k_scales);
  p.scales[1] = static_cast<uint8_t*>(c.v_scales);
  p.slots = slots;
  p.gain[0] = c.k_gain;
  p.gain[1] = c.v_gain;
  p.inv_gain[0] = 1.f / c.k_gain;
  p.inv_gain[1] = 1.f / c.v_gain;
  p.T = T;
  p.heads = c.Hkv;
  p.page_log2 = page_log2_of(c.page);
  p.slot_end = (long long)c.pages * c.page;
  const long long pieces = (long long)c.Hkv * (c.d / 8), chunks = (pieces + 31) / 32;
  p.pieces = (int)pieces;
  p.per_warp = std::max(1, 32 / p.pieces);
  batch = (long long)T / p.per_warp * chunks >= 32LL * kKv4Batch * sm_count_cached();
  const long long per_block = 8LL * p.per_warp * (batch ? kKv4Batch : 1);
  grid = dim3((unsigned)((T + per_block - 1) / per_block), (unsigned)chunks);
  return FA_OK;
}

}  // namespace

fa_status kv4_cache_checks(const fa_kv4_cache* c) {
  if (!c || c->pages < 0 || c->Hkv < 0 || page_log2_of(c->page) < 0) return FA_ERR_INVALID_ARG;
  // Gains whose products with 2^8 and whose reciprocals' with 2^9 (of the smallest scale) stay
  // finite: what the kernels multiply by, so that a code of 0 never meets an infinity.
  for (float g : {c->k_gain, c->v_gain})
    if (!(g >= 0x1p-100f && g <= 0x1p100f)) return FA_ERR_INVALID_ARG;
  if (padded_head_dim(c->d) == 0) return FA_ERR_UNSUPPORTED;
  // A token's runs of eight channels, 32 at a time, have to fit a grid's second dimension.
  if ((long long)c->Hkv * c->d > 65535LL * 256) return FA_ERR_INVALID_ARG;
  if (c->pages > 0 && c->Hkv > 0 && (!c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales))
    return FA_ERR_INVALID_ARG;
  if (!aligned16(c->k_codes) || !aligned16(c->k_scales) || !aligned16(c->v_codes) || !aligned16(c->v_scales))
    return FA_ERR_MISALIGNED;
  return FA_OK;
}

}  // namespace fa

using namespace fa;

extern "C" {

fa_status fa_page_grow(const int* lengths, const int* new_tokens, int* table, int B, int width, int page,
                       const int* free_pages, int free_size, const int* free_count, int T, long long* slots, int* cu,
                       int* lengths_out, int* count_out, void* stream) {
  if (!pages_ok(B, width, page, T) || free_size < 0) return FA_ERR_INVALID_ARG;
  if (B == 0) return FA_OK;
  if (!lengths || !new_tokens || !free_count || !cu || !lengths_out || !count_out) return FA_ERR_INVALID_ARG;
  if (free_size > 0 && !free_pages) return FA_ERR_INVALID_ARG;
  if ((width > 0 && !table) || (T > 0 && !slots)) return FA_ERR_INVALID_ARG;
  if (!all_aligned(4, lengths, new_tokens, table, free_pages, free_count, cu, lengths_out, count_out) ||
      !all_aligned(8, slots))
    return FA_ERR_MISALIGNED;
  PageParams p = {lengths, new_tokens, table, free_pages, free_count, slots, cu, lengths_out, count_out,
                  B, width, page_log2_of(page), T, free_size, 0, true};
  return run_pages(p, (cudaStream_t)stream);
}

fa_status fa_page_slots(const int* first, const int* count, const int* table, int B, int width, int page, int T,
                        long long* slots, int* cu, void* stream) {
  if (!pages_ok(B, width, page, T)) return FA_ERR_INVALID_ARG;
  if (B == 0) return FA_OK;
  if (!first || !count || !cu || (width > 0 && !table) || (T > 0 && !slots)) return FA_ERR_INVALID_ARG;
  if (!all_aligned(4, first, count, table, cu) || !all_aligned(8, slots)) return FA_ERR_MISALIGNED;
  PageParams p = {first, count, const_cast<int*>(table), nullptr, nullptr, slots, cu, nullptr, nullptr,
                  B, width, page_log2_of(page), T, 0, 0, false};
  return run_pages(p, (cudaStream_t)stream);
}

fa_status fa_kv4_store(const fa_kv4_cache* cache, const void* k, const void* v, long long k_token,
                       long long k_head, long long v_token, long long v_head, const long long* slots, int T,
                       void* stream) {
  fa_status s = kv4_cache_checks(cache);
  if (s != FA_OK) return s;
  if (T < 0) return FA_ERR_INVALID_ARG;
  if (T == 0 || cache->Hkv == 0 || cache->pages == 0) return FA_OK;
  if (!k || !v || !slots) return FA_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v) || (k_token & 7) || (k_head & 7) || (v_token & 7) || (v_head & 7) ||
      !all_aligned(8, slots))
    return FA_ERR_MISALIGNED;
  Kv4IoParams p = {};
  dim3 grid;
  bool batch;
  if ((s = kv4_io_fill(*cache, slots, T, p, grid, batch)) != FA_OK) return s;
  p.in[0] = static_cast<const uint16_t*>(k);
  p.in[1] = static_cast<const uint16_t*>(v);
  p.token[0] = k_token;
  p.token[1] = v_token;
  p.head[0] = k_head;
  p.head[1] = v_head;
  const auto run = [&](auto kernel) { return launch(FA_KERNEL_KV4_STORE, kernel, grid, dim3(256), 0, (cudaStream_t)stream, p); };
  switch (cache->d) {
    case 64: return batch ? run(kv4_store_kernel<64, kKv4Batch>) : run(kv4_store_kernel<64, 1>);
    case 96: return batch ? run(kv4_store_kernel<96, kKv4Batch>) : run(kv4_store_kernel<96, 1>);
    case 128: return batch ? run(kv4_store_kernel<128, kKv4Batch>) : run(kv4_store_kernel<128, 1>);
    case 192: return batch ? run(kv4_store_kernel<192, kKv4Batch>) : run(kv4_store_kernel<192, 1>);
    case 256: return batch ? run(kv4_store_kernel<256, kKv4Batch>) : run(kv4_store_kernel<256, 1>);
    case 384: return batch ? run(kv4_store_kernel<384, kKv4Batch>) : run(kv4_store_kernel<384, 1>);
  }
  return FA_ERR_UNSUPPORTED;
}

fa_status fa_kv4_load(const fa_kv4_cache* cache, const long long* slots, int T, void* k, void* v, void* stream) {
  fa_status s = kv4_cache_checks(cache);
  if (s != FA_OK) return s;
  if (T < 0) return FA_ERR_INVALID_ARG;
  if (T == 0 || cache->Hkv == 0) return FA_OK;
  if (!k || !v || !slots) return FA_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v) || !all_aligned(8, slots)) return FA_ERR_MISALIGNED;
  Kv4IoParams p = {};
  dim3 grid;
  bool batch;
  if ((s = kv4_io_fill(*cache, slots, T, p, grid, batch)) != FA_OK) return s;
  p.out[0] = static_cast<uint16_t*>(k);
  p.out[1] = static_cast<uint16_t*>(v);
  const auto run = [&](auto kernel) { return launch(FA_KERNEL_KV4_LOAD, kernel, grid, dim3(256), 0, (cudaStream_t)stream, p); };
  switch (cache->d) {
    case 64: return batch ? run(kv4_load_kernel<64, kKv4Batch>) : run(kv4_load_kernel<64, 1>);
    case 96: return batch ? run(kv4_load_kernel<96, kKv4Batch>) : run(kv4_load_kernel<96, 1>);
    case 128: return batch ? run(kv4_load_kernel<128, kKv4Batch>) : run(kv4_load_kernel<128, 1>);
    case 192: return batch ? run(kv4_load_kernel<192, kKv4Batch>) : run(kv4_load_kernel<192, 1>);
    case 256: return batch ? run(kv4_load_kernel<256, kKv4Batch>) : run(kv4_load_kernel<256, 1>);
    case 384: return batch ? run(kv4_load_kernel<384, kKv4Batch>) : run(kv4_load_kernel<384, 1>);
  }
  return FA_ERR_UNSUPPORTED;
}

}  // extern "C"
