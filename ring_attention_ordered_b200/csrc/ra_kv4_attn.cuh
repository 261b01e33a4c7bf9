// Pieces shared by the attention kernels over the paged 4-bit K/V cache:
// a request's numbers, the split of the launch's work over its CTAs, query
// rows, and the merge and store of results.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>
#include <type_traits>

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
  bool falls;   // cu falls here: then the requests' rows may overlap (see kv4_load)
};
__device__ __forceinline__ Kv4Req kv4_request(const Kv4AttnParams& p, int r) {
  Kv4Req q;
  q.bad = q.falls = false;
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
      q.falls = b < a;
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

// N consecutive elements of packed row `row` of head group h as they are in
// memory, zeros behind the last row.
template <int N>
__device__ __forceinline__ void kv4_load_q(const Kv4AttnParams& p, const Kv4Req& q, int h, int row,
                                           int rows, int d0, int d, uint4 (&x)[N / 8]) {
  static_assert(N % 8 == 0, "16-byte loads");
#pragma unroll
  for (int i = 0; i < N / 8; ++i) x[i] = make_uint4(0, 0, 0, 0);
  if (row >= rows) return;
  const int tok = row / p.group, head = h * p.group + (row - tok * p.group);
  const uint4* src = reinterpret_cast<const uint4*>(
      static_cast<const uint16_t*>(p.q) + (static_cast<long long>(q.first) + tok) * p.q_stride +
      static_cast<long long>(head) * d + d0);
#pragma unroll
  for (int i = 0; i < N / 8; ++i) x[i] = src[i];
}
__device__ __forceinline__ float2 kv4_q_pair(const Kv4AttnParams& p, uint32_t w) {
  return p.q_f16 ? __half22float2(*reinterpret_cast<const __half2*>(&w))
                 : make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
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

// Store four elements of a finished row: a / l, or zeros if the row saw no
// token, and by the row's first lane lse = (m + log2 l) ln 2, or -inf.
__device__ __forceinline__ void kv4_store(const Kv4AttnParams& p, int first, int h, int row, int d0,
                                          int d, float4 a, float m, float l) {
  const int tok = row / p.group, head = h * p.group + (row - tok * p.group);
  const long long at = (static_cast<long long>(first) + tok) * p.Hq + head;
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
__device__ __noinline__ void kv4_fill_empty(const Kv4AttnParams& p, unsigned long long* status) {
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

// The line of work.  Each unit (request, head, row tile) takes cells on it:
// `lead` cells for what a unit costs beside its blocks, one for each 2^shift
// blocks, and as many as bring it to a multiple of `align`.  The warps of the
// launch take equal stretches of `per` cells.
//
// Packed (lead > 0, align 1): every warp the same share of the work, whatever
// the lengths; but units then cross warps and CTAs where it happens.  Aligned
// (lead 0): every unit starts at a multiple of `align` cells, the stretches of
// 1, 2, 4 or 8 warps, so that it stays in those, or, being longer, in whole CTAs.
// Chosen where the longest stretch grows by 3 cells and a 32nd at most: that is
// about what pieces that cross CTAs cost (measured: 64 units of 512 blocks 27.7 us
// packed, 25.5 us aligned; 128 units of 300 blocks 31.0 us packed, 33.5 us aligned
// with stretches 12 cells longer).
//
// Cell numbers are 32 bits wide: the host chooses `shift` so that the longest
// line the arguments allow stays below 2^31.
struct Kv4Line {
  int shift, lead, align, per, total;
  bool odd;        // some request has no cached token, or numbers that do not fit
  __device__ __forceinline__ int cells(int nb) const {
    const int c = ((nb + (1 << shift) - 1) >> shift) + lead;
    return align == 1 ? c : (c + align - 1) / align * align;
  }
};

// Where a warp's stretch of the line begins: cell `off` of unit `unit` of
// request r.
struct Kv4Start {
  int r, unit, off;
};

// Where cu falls anywhere the launch does nothing: only as long as it does not,
// the requests together have no more rows than q, which is what keeps the cells of
// the line in 32 bits.
struct Kv4Load {
  int units, nb;
  bool odd, falls;
};
template <int ROWS>
__device__ __forceinline__ Kv4Load kv4_load(const Kv4AttnParams& p, int r) {
  if (r >= p.R) return {0, 0, false, false};
  const Kv4Req q = kv4_request(p, r);
  const int nb = (q.len + KV4_BLOCK - 1) / KV4_BLOCK, rows = q.n * p.group;
  return {nb == 0 || rows > p.rows_max ? 0 : (rows + ROWS - 1) / ROWS * p.Hkv, nb,
          q.bad || nb == 0, q.falls};
}

__device__ __forceinline__ int kv4_warp_scan(int x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// Cells of a warp's stretch, packed; and the alignment (0: none) and cells of
// one in which `units` units, the longest of `most` cells and `total` in all,
// start in warps of their own.
struct Kv4Layout {
  int per, align;
};
template <int WARPS>
__device__ __forceinline__ Kv4Layout kv4_layout(int units, int most, int total, int packed,
                                                int warps, int min_cells) {
  const int per = max((packed + warps - 1) / warps, min_cells);
  if (units == 0 || units > warps) return {per, 0};
  int per2, align;
  const int each = warps / units;           // warps a unit
  if (each < WARPS) {
    const int a = each >= 8 ? 8 : each >= 4 ? 4 : each >= 2 ? 2 : 1;
    per2 = (most + a - 1) / a;
    align = a;
  } else {
    // the same number of CTAs for each, or one stretch each left partly empty
    const int ctas = warps / WARPS, same = ctas / units * WARPS;
    per2 = (most + same - 1) / same;
    if (units < ctas) {
      const int rest = (ctas - units) * WARPS;
      per2 = min(per2, (total + rest - 1) / rest);
    }
    align = WARPS;
  }
  per2 = max(per2, min_cells);
  if (per2 > per + per / 32 + 3) return {per, 0};
  return {per2, align * per2};
}

// Lays the line out and finds where warp `me` of the launch's `warps` begins.
// Up to 64 requests each warp does so by itself, one or two a lane (64 requests of 0
// to 8191 tokens: 28.4 us, 29.3 us by the CTA; one form of this for all numbers: one
// request of 509 tokens 9.5 us instead of 8.8; 128 requests with four a lane are no
// faster than by the CTA).  More are taken a thread at a time by the CTA (s_scan: 3
// WARPS ints, s_start: one a warp).
template <int ROWS, int WARPS>
__device__ __forceinline__ Kv4Start kv4_find_start(const Kv4AttnParams& p, int lead, int min_cells,
                                                   int me, int warps, int* s_scan,
                                                   Kv4Start* s_start, Kv4Line& line) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  line.shift = p.cell_shift;
  line.lead = lead;
  line.align = 1;
  auto lay_out = [&](int units, int most, int packed) {
    const Kv4Layout x = kv4_layout<WARPS>(units, most, packed - units * lead, packed, warps,
                                          min_cells);
    line.per = x.per;
    if (x.align) {
      line.lead = 0;
      line.align = x.align;
    }
    return x.align != 0;
  };
  // by the warp alone: lane i has requests i E .. i E + E - 1
  auto by_warp = [&](auto each_c) -> Kv4Start {
    constexpr int E = decltype(each_c)::value;
    Kv4Load x[E];
    bool odd = false, falls = false;
    int units = 0, most = 0, all[E], mine = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      x[e] = kv4_load<ROWS>(p, lane * E + e);
      all[e] = line.cells(x[e].nb);
      odd |= x[e].odd;
      falls |= x[e].falls;
      units += x[e].units;
      most = max(most, x[e].units ? all[e] - lead : 0);
      mine += x[e].units * all[e];
    }
    line.odd = __any_sync(0xffffffffu, odd);
    if (line.odd && __any_sync(0xffffffffu, falls)) {
      line.total = 0;
      line.per = min_cells;
      return {0, 0, 0};
    }
    int hi = kv4_warp_scan(mine);
    line.total = __shfl_sync(0xffffffffu, hi, 31);
    if (lay_out(__reduce_add_sync(0xffffffffu, units), __reduce_max_sync(0xffffffffu, most),
                line.total)) {
      mine = 0;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        all[e] = line.cells(x[e].nb);
        mine += x[e].units * all[e];
      }
      hi = kv4_warp_scan(mine);
      line.total = __shfl_sync(0xffffffffu, hi, 31);
    }
    const int at = me * line.per;
    const unsigned found = __ballot_sync(0xffffffffu, hi > at);
    if (found == 0) return {0, 0, 0};
    const int from = __ffs(found) - 1;
    int in = at - __shfl_sync(0xffffffffu, hi - mine, from), r = from * E, cells = 0;
    bool there = false;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int c = __shfl_sync(0xffffffffu, x[e].units * all[e], from);
      const int one = __shfl_sync(0xffffffffu, all[e], from);
      if (!there) {
        there = in < c;
        cells = one;
        if (!there) {
          in -= c;
          ++r;
        }
      }
    }
    const int u = in / cells;
    return {r, u, in - u * cells};
  };
  if (p.R <= 32) return by_warp(std::integral_constant<int, 1>{});
  if (p.R <= 64) return by_warp(std::integral_constant<int, 2>{});
  // thread tid: requests [tid * each, tid * each + each)
  const int each = (p.R + WARPS * 32 - 1) / (WARPS * 32);
  int mine = 0, units = 0, most = 0;
  bool odd = false, falls = false;
  Kv4Load only = {0, 0, false, false};   // the thread's request if it has but one
  auto load = [&](int i) { return each == 1 ? only : kv4_load<ROWS>(p, tid * each + i); };
  for (int i = 0; i < each; ++i) {
    const Kv4Load x = kv4_load<ROWS>(p, tid * each + i);
    only = x;
    mine += x.units * line.cells(x.nb);
    units += x.units;
    if (x.units) most = max(most, line.cells(x.nb) - lead);
    odd |= x.odd;
    falls |= x.falls;
  }
  int inc = kv4_warp_scan(mine);
  units = __reduce_add_sync(0xffffffffu, units);
  most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 31) {
    s_scan[warp] = inc;
    s_scan[WARPS + warp] = units;
    s_scan[2 * WARPS + warp] = most;
  }
  line.odd = __syncthreads_or(odd);
  if (line.odd && __syncthreads_or(falls)) {
    line.total = 0;
    line.per = min_cells;
    return {0, 0, 0};
  }
  int lo = inc - mine;
  line.total = units = most = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) lo += s_scan[w];
    line.total += s_scan[w];
    units += s_scan[WARPS + w];
    most = max(most, s_scan[2 * WARPS + w]);
  }
  if (lay_out(units, most, line.total)) {
    __syncthreads();
    mine = 0;
    for (int i = 0; i < each; ++i) {
      const Kv4Load x = load(i);
      mine += x.units * line.cells(x.nb);
    }
    inc = kv4_warp_scan(mine);
    if (lane == 31) s_scan[warp] = inc;
    __syncthreads();
    lo = inc - mine;
    line.total = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      if (w < warp) lo += s_scan[w];
      line.total += s_scan[w];
    }
  }
  // the first of this CTA's warps that begins behind `lo`
  const int me0 = me - warp;
  int x = max((lo + line.per - 1) / line.per - me0, 0);
  if (x < WARPS && (me0 + x) * line.per < lo + mine) {
    for (int i = 0; i < each; ++i) {
      const Kv4Load l = load(i);
      const int all = line.cells(l.nb), hi = lo + l.units * all;
      for (; x < WARPS && (me0 + x) * line.per < hi; ++x) {
        const int in = (me0 + x) * line.per - lo, u = in / all;
        s_start[x] = {tid * each + i, u, in - u * all};
      }
      lo = hi;
    }
  }
  __syncthreads();
  return s_start[warp];
}

}  // namespace ra
