// Pieces shared by the attention kernels over the paged 4-bit K/V cache:
// a request's numbers, the split of the launch's work over its CTAs, query
// rows, and the merge and store of results.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "ptx_sm100.cuh"
#include "ra_internal.h"
#include "ra_kv4.cuh"

namespace ra {

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Request r: its query tokens [first, first + n) and cached tokens.  Numbers
// outside the tensors are cut down to them; `bad` says so.
struct Kv4Req {
  int first, n, len;
  bool bad;
};
__device__ __forceinline__ Kv4Req kv4_request(const Kv4AttnParams& p, int r) {
  Kv4Req q;
  q.bad = false;
  int len = p.lens[r];
  const long long room = static_cast<long long>(p.W) * p.page;
  if (len < 0 || len > room) {
    q.bad = true;
    len = len < 0 ? 0 : static_cast<int>(room);
  }
  int a = r, b = r + 1;
  if (p.cu != nullptr) {
    a = p.cu[r];
    b = p.cu[r + 1];
    if (a < 0 || b < a || b > p.T) {
      q.bad = true;
      a = min(max(a, 0), p.T);
      b = min(max(b, a), p.T);
    }
  }
  q.first = a;
  q.n = b - a;
  q.len = len;
  return q;
}

// Tokens that packed row `row` (token row / group of the request) sees.  A row
// behind the last one is not stored; it is given every token, so that it
// does not make a block look partly hidden.
__device__ __forceinline__ int kv4_limit(const Kv4AttnParams& p, const Kv4Req& q, int row,
                                         int rows) {
  if (row >= rows) return q.len;
  return p.causal ? min(q.len, q.len - q.n + row / p.group + 1) : q.len;
}

// Index of 16-token block `blk` of request r and head h in the cache, -1 if
// the page the table names is out of range.
__device__ __forceinline__ int kv4_block_index(const Kv4AttnParams& p, int r, int h, int blk,
                                               unsigned long long* status) {
  const int bpp = p.page >> 4;
  const int col = blk / bpp;
  const int id = p.table[static_cast<long long>(r) * p.W + col];
  if (id < 0 || id >= p.num_pages) {
    kv4_record(status, RA_ERR_INVALID_ARG, KV4_SITE_PAGE);
    return -1;
  }
  return (id * p.Hkv + h) * bpp + (blk - col * bpp);
}

// N consecutive elements of packed row `row` of head group h, zeros behind
// the last row.
template <int N>
__device__ __forceinline__ void kv4_load_q(const Kv4AttnParams& p, const Kv4Req& q, int h, int row,
                                           int rows, int d0, int d, float (&x)[N]) {
  static_assert(N % 8 == 0, "16-byte loads");
  if (row >= rows) {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = 0.f;
    return;
  }
  const int tok = row / p.group, head = h * p.group + (row - tok * p.group);
  const uint4* src = reinterpret_cast<const uint4*>(
      static_cast<const uint16_t*>(p.q) + (static_cast<long long>(q.first) + tok) * p.q_stride +
      static_cast<long long>(head) * d + d0);
#pragma unroll
  for (int i = 0; i < N / 8; ++i) {
    const uint4 v = src[i];
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float2 f;
      if (p.q_f16)
        f = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
      else
        f = make_float2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u));
      x[8 * i + 2 * k] = f.x;
      x[8 * i + 2 * k + 1] = f.y;
    }
  }
}

// The power of two `up` that brings a row's largest magnitude into [2^14,
// 2^15), and its inverse.  1 for a row of zeros or one that is not finite
// (whose result is NaN with or without it).  Both stay normal: an exponent
// outside [-100, 100] is scaled as that one (such a row's scores are zero, or
// infinite, to fp32 either way).
__device__ __forceinline__ void kv4_row_scale(float am, float& up, float& down) {
  const int e = static_cast<int>((__float_as_uint(am) >> 23) & 0xff) - 127;
  int s = 14 - e;
  if (am == 0.f || e == 128) s = 0;
  s = min(max(s, -100), 100);
  up = __uint_as_float(static_cast<uint32_t>(127 + s) << 23);
  down = __uint_as_float(static_cast<uint32_t>(127 - s) << 23);
}

// (m, l, a) <- merged with another partial of the same row (log2 units).  A
// partial with m = -inf is empty.
__device__ __forceinline__ void kv4_merge(float& m, float& l, float4& a, float m2, float l2,
                                          float4 b) {
  if (m2 == -INFINITY) return;
  const float mn = fmaxf(m, m2);
  const float f = m == -INFINITY ? 0.f : m == mn ? 1.f : ex2_approx(m - mn);
  const float f2 = m2 == mn ? 1.f : ex2_approx(m2 - mn);
  m = mn;
  l = l * f + l2 * f2;
  a.x = a.x * f + b.x * f2;
  a.y = a.y * f + b.y * f2;
  a.z = a.z * f + b.z * f2;
  a.w = a.w * f + b.w * f2;
}

// Store four elements of a finished row: a / l, or zeros if the row saw no
// token, and by the row's first lane lse = (m + log2 l) ln 2, or -inf.
__device__ __forceinline__ void kv4_store(const Kv4AttnParams& p, const Kv4Req& q, int h, int row,
                                          int d0, int d, float4 a, float m, float l) {
  const int tok = row / p.group, head = h * p.group + (row - tok * p.group);
  const long long at = (static_cast<long long>(q.first) + tok) * p.Hq + head;
  const bool none = l == 0.f;
  const float inv = 1.f / l;
  const float4 y = none ? make_float4(0.f, 0.f, 0.f, 0.f)
                        : make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
  const long long o = at * d + d0;
  if (p.out_f32) {
    *reinterpret_cast<float4*>(static_cast<float*>(p.out) + o) = y;
  } else if (p.q_f16) {
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + o) =
        make_uint2(pack_f16x2(y.x, y.y), pack_f16x2(y.z, y.w));
  } else {
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + o) =
        make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
  }
  if (d0 == 0) p.lse[at] = none ? -INFINITY : (m + log2f(l)) * 0.69314718055994530942f;
}

// Requests without a cached token: their rows are empty, out = 0, lse = -inf.
// Dealt over the CTAs by request.  Also the one place that reports numbers
// outside the tensors.
template <int D, int THREADS>
__device__ __forceinline__ void kv4_fill_empty(const Kv4AttnParams& p, unsigned long long* status) {
  for (int r = blockIdx.x; r < p.R; r += gridDim.x) {
    const Kv4Req q = kv4_request(p, r);
    if (q.bad && threadIdx.x == 0)
      kv4_record(status, RA_ERR_INVALID_ARG, KV4_SITE_LENGTH);
    if (q.len != 0) continue;
    const long long n = static_cast<long long>(q.n) * p.Hq;
    const long long first = static_cast<long long>(q.first) * p.Hq;
    for (long long i = threadIdx.x; i < n * (D / 8); i += THREADS) {
      const uint4 zero = make_uint4(0, 0, 0, 0);
      if (p.out_f32) {
        uint4* dst = reinterpret_cast<uint4*>(static_cast<float*>(p.out) + first * D) + 2 * i;
        dst[0] = zero;
        dst[1] = zero;
      } else {
        reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + first * D)[i] = zero;
      }
    }
    for (long long i = threadIdx.x; i < n; i += THREADS) p.lse[first + i] = -INFINITY;
  }
}

// Cells that request r takes on the line of work: for each of its units
// (head, row tile) the blocks of its tokens, and UNIT_COST before them.
template <int ROWS, int UNIT_COST>
__device__ __forceinline__ long long kv4_work(const Kv4AttnParams& p, int r) {
  const Kv4Req q = kv4_request(p, r);
  const int tiles = (q.n * p.group + ROWS - 1) / ROWS;
  const int nb = (q.len + KV4_BLOCK - 1) / KV4_BLOCK;
  return nb == 0 ? 0 : static_cast<long long>(tiles) * p.Hkv * (nb + UNIT_COST);
}

// Where a warp's stretch of the line begins: cell in_r of request r.
struct Kv4Start {
  long long in_r;
  int r;
};

// The whole CTA: the line's length, the stretch of one warp (`per` cells, at
// least MIN_CELLS, the same for every warp of the launch) and the request in
// which each of this CTA's warps begins.  Requests are taken WARPS * 32 at a
// time; the second pass ends once the last warp's is found.  Ends with the
// CTA's threads synchronised.
template <int ROWS, int MIN_CELLS, int UNIT_COST, int WARPS>
__device__ __forceinline__ void kv4_find_start(const Kv4AttnParams& p, long long* s_scan,
                                               Kv4Start* out, long long& per, long long& total) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int THREADS = WARPS * 32;
  const long long first = tid < p.R ? kv4_work<ROWS, UNIT_COST>(p, tid) : 0;
  long long mine = first;
  for (int r = tid + THREADS; r < p.R; r += THREADS) mine += kv4_work<ROWS, UNIT_COST>(p, r);
  // one scan gives the total, and the places of the first THREADS requests
  auto scan = [&](long long x, long long& sum) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s_scan[warp] = x;
    __syncthreads();
    long long before = 0;
    sum = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      if (w < warp) before += s_scan[w];
      sum += s_scan[w];
    }
    __syncthreads();
    return before + x;
  };
  long long hi = scan(mine, total);
  const long long warps = static_cast<long long>(gridDim.x) * WARPS;
  per = (total + warps - 1) / warps;
  if (per < MIN_CELLS) per = MIN_CELLS;
  const long long cta0 = per * (static_cast<long long>(blockIdx.x) * WARPS);
  long long base = 0;
  for (int r0 = 0; r0 < p.R && base <= cta0 + (WARPS - 1) * per; r0 += THREADS) {
    const int r = r0 + tid;
    long long w = first, all = total;
    if (p.R > THREADS) {
      w = r0 == 0 ? first : r < p.R ? kv4_work<ROWS, UNIT_COST>(p, r) : 0;
      hi = base + scan(w, all);
      all += base;
    }
    const long long lo = hi - w;
#pragma unroll
    for (int x = 0; x < WARPS; ++x) {
      const long long at = cta0 + x * per;
      if (lo <= at && at < hi) out[x] = {at - lo, r};
    }
    base = all;
  }
  __syncthreads();
}

}  // namespace ra
