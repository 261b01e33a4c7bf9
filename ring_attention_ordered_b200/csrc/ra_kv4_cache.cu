// The paged 4-bit K/V cache (sm_100a): the page plan, the append and the
// read.  Layout and format: ra_kv4.cuh.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "ra_internal.h"
#include "ptx_sm100.cuh"
#include "ra_kv4.cuh"

namespace ra {
namespace {

namespace cg = cooperative_groups;

__device__ unsigned long long g_kv4_cache_status = 0ull;

// ------------------------------------------------------------------ plan
// Block tables and slot maps from request lengths.  Every CTA of the
// launch's one cluster computes the same prefix sums over the requests (new
// tokens, pages that come back, pages that are needed) in shared memory;
// the lists they number -- released pages, new pages, tokens -- are then
// dealt out over the cluster's threads.  Three cluster barriers order the
// phases: everything old has been read before anything is overwritten (the
// outputs may be the inputs), released pages are on the stack before they
// are taken again, the table is complete before the slots read it.  The
// stack positions follow from the prefix sums alone, so the result does not
// depend on which thread does what.  A page index outside the cache (of a table or
// a stack that something else spoiled) keeps its place in them, is reported, and
// gives no slots: page * p.page of such an index may be any slot of another
// request, or pass for the -1 of no slot.
//
// Bound by latency: 6.4 us for 8 requests (one CTA), 15.6 us for 1000 requests
// with a table of 1000 x 256 that is copied and 18.5K slots (eight CTAs), of which
// the bytes are 0.4 us.
constexpr int PLAN_THREADS = 1024;

constexpr size_t plan_smem_bytes(int R) { return (4 * static_cast<size_t>(R) + 3) * sizeof(int); }

struct PlanSums {
  long long tok;   // new tokens
  int rel;         // released pages
  int take;        // new pages
};

__device__ __forceinline__ PlanSums operator+(const PlanSums& a, const PlanSums& b) {
  return {a.tok + b.tok, a.rel + b.rel, a.take + b.take};
}
__device__ __forceinline__ PlanSums shfl_up(const PlanSums& a, int n) {
  return {__shfl_up_sync(0xffffffffu, a.tok, n), __shfl_up_sync(0xffffffffu, a.rel, n),
          __shfl_up_sync(0xffffffffu, a.take, n)};
}

// The last index r in [0, n) with pre[r] <= i (pre ascending, pre[0] = 0).
__device__ __forceinline__ int find_request(const int* pre, int n, int i) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pre[mid] <= i) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// n ints by threads tid, tid + size, ...: 16 bytes at a time where both
// pointers allow, four loads under way.
__device__ __forceinline__ void copy_ints(int32_t* dst, const int32_t* src, long long n, int tid,
                                          int size) {
  constexpr int U = 4;
  long long done = 0;
  if (((reinterpret_cast<uintptr_t>(dst) | reinterpret_cast<uintptr_t>(src)) & 15u) == 0) {
    const long long n4 = n >> 2;
    for (long long i = tid; i < n4; i += U * static_cast<long long>(size)) {
      int4 x[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i + u * static_cast<long long>(size) < n4)
          x[u] = reinterpret_cast<const int4*>(src)[i + u * static_cast<long long>(size)];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i + u * static_cast<long long>(size) < n4)
          reinterpret_cast<int4*>(dst)[i + u * static_cast<long long>(size)] = x[u];
    }
    done = n4 << 2;
  }
#pragma unroll 4
  for (long long i = done + tid; i < n; i += size) dst[i] = src[i];
}

__global__ void __launch_bounds__(PLAN_THREADS) ra_kv4_plan_kernel(const Kv4PlanParams p) {
  cg::cluster_group cluster = cg::this_cluster();
  extern __shared__ int plan_smem[];
  const int R = p.R;
  int* s_cu = plan_smem;             // [R + 1] new tokens before request r
  int* s_rel = s_cu + R + 1;         // [R + 1] released pages before request r
  int* s_take = s_rel + R + 1;       // [R + 1] new pages before request r
  int* s_len = s_take + R + 1;       // [R]     tokens held before the call (plan_smem_bytes)
  __shared__ PlanSums s_warp[PLAN_THREADS / 32];
  __shared__ PlanSums s_carry;
  __shared__ int s_bad;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gtid = blockIdx.x * PLAN_THREADS + tid;
  const int gsize = gridDim.x * PLAN_THREADS;
  const int n_free = p.pool[0];
  if (tid == 0) {
    s_carry = {0, 0, 0};
    s_bad = n_free < 0 || n_free > p.num_pages;
  }
  __syncthreads();

  const long long room = static_cast<long long>(p.W) * p.page;
  for (int r0 = 0; r0 < R; r0 += PLAN_THREADS) {
    const int r = r0 + tid;
    PlanSums x{0, 0, 0};
    int len = 0;
    if (r < R) {
      len = p.lens[r];
      const int add = p.add[r];
      const bool bad = len < 0 || add < -1 || len > room || (add > 0 && add > room - len);
      if (bad) {
        s_bad = 1;
        len = 0;
      } else {
        const int old = static_cast<int>((static_cast<long long>(len) + p.page - 1) / p.page);
        if (add < 0) {
          x.rel = old;
        } else {
          x.tok = add;
          x.take =
              static_cast<int>((static_cast<long long>(len) + add + p.page - 1) / p.page) - old;
        }
      }
      s_len[r] = len;
    }
    PlanSums inc = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const PlanSums y = shfl_up(inc, o);
      if (lane >= o) inc = inc + y;
    }
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    PlanSums base = s_carry;
    for (int w = 0; w < warp; ++w) base = base + s_warp[w];
    const PlanSums end = base + inc;
    if (r < R) {
      // totals above the limits are refused below; the stored value is then unused
      s_cu[r + 1] = static_cast<int>(end.tok);
      s_rel[r + 1] = end.rel;
      s_take[r + 1] = end.take;
    }
    __syncthreads();
    if (tid == PLAN_THREADS - 1) s_carry = end;
    __syncthreads();
  }
  if (tid == 0) s_cu[0] = s_rel[0] = s_take[0] = 0;
  __syncthreads();
  const PlanSums all = s_carry;
  const bool bad = s_bad != 0 || all.tok > p.max_tokens ||
                   static_cast<long long>(n_free) + all.rel > p.num_pages;
  const long long top = bad ? 0 : static_cast<long long>(n_free) + all.rel;
  const long long missing = bad ? -1 : (all.take > top ? all.take - top : 0);
  const bool keep = missing != 0;   // nothing changes
  const int n_rel = keep ? 0 : all.rel, n_take = keep ? 0 : all.take;
  const int n_tok = keep ? 0 : static_cast<int>(all.tok);
  const int itop = keep ? n_free : static_cast<int>(top);
  const int left = itop - n_take;   // free pages after the call

  cluster.sync();   // every CTA has read lens, add and pool[0]

  if (p.table_out != p.table)
    copy_ints(p.table_out, p.table, static_cast<long long>(R) * p.W, gtid, gsize);
  if (p.pool_out != p.pool)
    copy_ints(p.pool_out + 1, p.pool + 1, keep ? p.num_pages : min(left, n_free), gtid, gsize);
  if (!keep) {
    // above the stack's new top nothing is left
    for (int i = itop + 1 + gtid; i <= p.num_pages; i += gsize) p.pool_out[i] = -1;
  }
  bool outside = false;   // a page index outside the cache
  for (int i = gtid; i < n_rel; i += gsize) {
    const int r = find_request(s_rel, R + 1, i);
    const int page = p.table[static_cast<long long>(r) * p.W + (i - s_rel[r])];
    outside |= page < 0 || page >= p.num_pages;
    p.pool_out[n_free + 1 + i] = page;
  }
  for (int r = gtid; r < R; r += gsize) {
    p.cu[r] = keep ? 0 : s_cu[r];
    const bool done = s_rel[r + 1] != s_rel[r] || p.add[r] < 0;
    p.lens_out[r] = keep ? p.lens[r] : done ? 0 : s_len[r] + (s_cu[r + 1] - s_cu[r]);
  }
  if (gtid == 0) {
    p.cu[R] = n_tok;
    p.shortage[0] = static_cast<int>(missing);
  }

  cluster.sync();   // the released pages are on the stack, the table is copied

  if (gtid == 0) p.pool_out[0] = keep ? n_free : left;
  for (int i = gtid; i < n_rel; i += gsize) {
    const int r = find_request(s_rel, R + 1, i);
    p.table_out[static_cast<long long>(r) * p.W + (i - s_rel[r])] = -1;
  }
  for (int i = gtid; i < n_take; i += gsize) {
    const int r = find_request(s_take, R + 1, i);
    const int at = itop - i;        // from the top of the stack
    const int page = at <= n_free ? __ldcg(p.pool + at) : __ldcg(p.pool_out + at);
    const int old = (s_len[r] + p.page - 1) / p.page;
    outside |= page < 0 || page >= p.num_pages;
    p.table_out[static_cast<long long>(r) * p.W + old + (i - s_take[r])] = page;
    p.pool_out[at] = -1;
  }

  cluster.sync();   // the table is complete

  for (long long i = gtid; i < p.max_tokens; i += gsize) {
    int slot = -1;
    if (i < n_tok) {
      const int r = find_request(s_cu, R + 1, static_cast<int>(i));
      const int pos = s_len[r] + (static_cast<int>(i) - s_cu[r]);
      const int page = __ldcg(p.table_out + static_cast<long long>(r) * p.W + pos / p.page);
      if (page < 0 || page >= p.num_pages)
        outside = true;
      else
        slot = page * p.page + pos % p.page;
    }
    p.slots[i] = slot;
  }
  if (outside) kv4_record(&g_kv4_cache_status, RA_ERR_INVALID_ARG, KV4_SITE_PAGE);
}

// ------------------------------------------------------------------ append
template <class T>
struct Pair;
template <>
struct Pair<__nv_bfloat16> {
  using T2 = __nv_bfloat162;
  static __device__ __forceinline__ float2 to_float(T2 x) { return __bfloat1622float2(x); }
};
template <>
struct Pair<__half> {
  using T2 = __half2;
  static __device__ __forceinline__ float2 to_float(T2 x) { return __half22float2(x); }
};

template <class T2>
__device__ __forceinline__ T2 as_pair(uint32_t x) {
  return *reinterpret_cast<T2*>(&x);
}
template <class T2>
__device__ __forceinline__ uint32_t as_word(T2 x) {
  return *reinterpret_cast<uint32_t*>(&x);
}

// The code of one value: the nearest level of 0..15 to (x - zero) / step,
// ties to the even code.  n is a level within one of it; the residual
// r = a - n step with a = x - zero rounded is exact (n step has 15 bits, and r
// is a multiple of a's last place no larger than step), and e is what the
// rounding of a left out, which decides where r lies on a border.
__device__ __forceinline__ uint32_t kv4_code(float x, float zero, float step, float inv) {
  const float a = x - zero, b = a - x;
  const float e = (x - (a - b)) - (zero + b);
  const float n = rintf(fminf(fmaxf(a * inv, 0.f), 15.f));
  const float r = fmaf(-n, step, a), half = 0.5f * step;
  const bool odd = (static_cast<int>(n) & 1) != 0;
  const bool up = r > half || (r == half && (e > 0.f || (e == 0.f && odd)));
  const bool down = r < -half || (r == -half && (e < 0.f || (e == 0.f && odd)));
  return static_cast<uint32_t>(min(max(static_cast<int>(n) + up - down, 0), 15));
}

// Sixteen values of one lane; the LANES lanes of the vector agree on its
// range.  `use`: whether anything is made of the result.  Returns the codes (element
// i in nibble i) and the parameter word.
//
// The codes come from t = (x - zero) / step rounded to an integer by adding 1.5
// * 2^23, four codes joined as one float below 2^24.  The quotient by the
// approximate reciprocal (one ulp) is within 15 * 2^-22 of the exact one, so
// only a value within 2^-17 of a border can be wrong; a lane that has one (one
// in 90 does: values and steps of few bits often lie exactly half way) takes
// kv4_code for its own, and so does a vector in which t may leave [0, 15]: a
// step so small that rounding it or the zero to fp16's subnormals counts, or
// values that were clamped.
//
// The quotient (max - min) / 15 is formed by Markstein's method, a product by
// the rounded reciprocal and one correction, which gives the correctly rounded
// one (the tests check every significand).
struct Kv4Codes {
  uint32_t lo, hi, params;
};
template <class T, int LANES>
__device__ __forceinline__ Kv4Codes kv4_encode16(uint4 x, uint4 y, bool use) {
  using T2 = typename Pair<T>::T2;
  const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
  T2 mn = as_pair<T2>(w[0]), mx = mn;
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    mn = __hmin2_nan(mn, as_pair<T2>(w[i]));
    mx = __hmax2_nan(mx, as_pair<T2>(w[i]));
  }
  // (min, -max) in one word: both are minima, exact in the input's type
  const uint32_t mnw = as_word<T2>(mn), mxw = as_word<T2>(mx) ^ 0x80008000u;
  T2 m = __hmin2_nan(as_pair<T2>(__byte_perm(mnw, mxw, 0x5410)),
                     as_pair<T2>(__byte_perm(mnw, mxw, 0x7632)));
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1)
    m = __hmin2_nan(m, as_pair<T2>(__shfl_xor_sync(0xffffffffu, as_word<T2>(m), o)));
  const float2 r = Pair<T>::to_float(m);
  const bool nan = r.x != r.x;   // a NaN reaches both halves
  const float lo = fminf(fmaxf(r.x, -65504.f), 65504.f);
  const float hi = fminf(fmaxf(-r.y, -65504.f), 65504.f);
  const float span = hi - lo;
  constexpr float FIFTEENTH = 1.f / 15.f;
  const float q0 = span * FIFTEENTH;
  const __half zh = __float2half_rn(lo);
  __half sh = __float2half_rz(fmaf(fmaf(-15.f, q0, span), FIFTEENTH, q0));
  if (__half_as_ushort(sh) == 0) sh = __ushort_as_half(1);
  const float zero = __half2float(zh), step = __half2float(sh);
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(step));
  const uint64_t mz2 = f2_pack(-zero, -zero), inv2 = f2_pack(inv, inv);
  const uint64_t big = f2_pack(12582912.f, 12582912.f), mbig = f2_pack(-12582912.f, -12582912.f);
  // all sixteen again where t may leave [0, 15], else those near a border
  uint32_t again = step >= 1.220703125e-4f && lo == r.x && hi == -r.y ? 0u : 0xffffu;
  float q[4], d[16], off = 0.f;
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    float n[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 v = Pair<T>::to_float(as_pair<T2>(w[2 * h + i]));
      const uint64_t t = f2_mul(f2_add(f2_pack(v.x, v.y), mz2), inv2);
      const uint64_t k = f2_add(f2_add(t, big), mbig);
      float* e = d + 4 * h + 2 * i;
      f2_unpack(f2_sub(t, k), e[0], e[1]);
      f2_unpack(k, n[2 * i], n[2 * i + 1]);
      off = fmax3(off, fabsf(e[0]), fabsf(e[1]));
    }
    q[h] = fmaf(n[3], 4096.f, fmaf(n[2], 256.f, fmaf(n[1], 16.f, n[0] + 8388608.f)));
  }
  Kv4Codes c;
  c.lo = __byte_perm(__float_as_uint(q[0]), __float_as_uint(q[1]), 0x5410);
  c.hi = __byte_perm(__float_as_uint(q[2]), __float_as_uint(q[3]), 0x5410);
  c.params = nan ? 0x7FFF7FFFu
                 : static_cast<uint32_t>(__half_as_ushort(sh)) |
                       (static_cast<uint32_t>(__half_as_ushort(zh)) << 16);
  constexpr float NEAR = 0.5f - 7.62939453125e-6f;
  if (off >= NEAR) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (fabsf(d[i]) >= NEAR) again |= 1u << i;
  }
  if (nan || !use) c.lo = c.hi = again = 0u;
#pragma unroll 1
  while (again) {
    const int i = __ffs(again) - 1;
    again &= again - 1;
    // selected, not indexed: the words stay in registers
    const uint32_t p0 = (i & 2) ? w[1] : w[0], p1 = (i & 2) ? w[3] : w[2];
    const uint32_t p2 = (i & 2) ? w[5] : w[4], p3 = (i & 2) ? w[7] : w[6];
    const uint32_t p4 = (i & 4) ? p1 : p0, p5 = (i & 4) ? p3 : p2;
    const float2 v = Pair<T>::to_float(as_pair<T2>((i & 8) ? p5 : p4));
    const uint32_t code = kv4_code((i & 1) ? v.y : v.x, zero, step, inv);
    const int at = 4 * (i & 7);
    const uint32_t keep = ~(15u << at), put = code << at;
    if (i < 8) c.lo = (c.lo & keep) | put; else c.hi = (c.hi & keep) | put;
  }
  return c;
}

// Bound: the append by instruction issue (71% of the slots) and, between, by the loads
// that each vector waits for at 42% occupancy (32749 tokens, 8 heads, d = 128: 48 us,
// 3600 GB/s), the read by memory latency (128K tokens: 126 us,
// 5400 GB/s, 0.82 of the copy rate).
//
// Work of append and read: d / EACH lanes take the d values of a token and
// head (EACH = 16 in the append, which divides what a vector costs by fewer
// lanes; 8 in the read, whose lanes then store side by side); a CTA takes 16
// tokens (so that the tokens whose V codes share a sector are handled together)
// of HEADS heads, HEADS_AT_ONCE of them in each thread with their loads under
// way together: two in the read (126 us for 128K tokens, 141 us with one), one in
// the append, whose code then fits the instruction cache (32749 tokens, read back
// included: 98 us with two).
constexpr int CACHE_THREADS = 256;
template <int D, int EACH, int HEADS_AT_ONCE>
struct CacheCta {
  static constexpr int LANES = D / EACH;
  static constexpr int ACROSS = CACHE_THREADS / (16 * LANES);   // heads side by side
  static constexpr int HEADS = ACROSS * HEADS_AT_ONCE;
};
struct Place {
  long long token;
  int head0, lane;      // head u of the thread: head0 + u * ACROSS
};
template <class C>
__device__ __forceinline__ Place place_of(int Hkv) {
  const unsigned per = (Hkv + C::HEADS - 1) / C::HEADS;
  const unsigned group = blockIdx.x / per;
  const int t = threadIdx.x;
  return {static_cast<long long>(group) * 16 + (t / C::LANES) % 16,
          static_cast<int>(blockIdx.x - group * per) * C::HEADS + t / (16 * C::LANES),
          t % C::LANES};
}
// The slot of a token, -1 if it has none (one out of range is reported).
__device__ __forceinline__ int slot_of(const Kv4CopyParams& p, long long token) {
  const int slot = token < p.T ? p.slots[token] : -1;
  if (slot < -1 || slot >= p.num_slots) {
    kv4_record(&g_kv4_cache_status, RA_ERR_INVALID_ARG, KV4_SITE_SLOT);
    return -1;
  }
  return slot;
}

template <int D, class T>
__global__ void __launch_bounds__(CACHE_THREADS) ra_kv4_append_kernel(const Kv4CopyParams p) {
  using L = Kv4<D>;
  constexpr int HEADS_AT_ONCE = 1;
  using C = CacheCta<D, 16, HEADS_AT_ONCE>;
  constexpr int LANES = C::LANES;
  const Place at = place_of<C>(p.Hkv);
  const int j = at.lane;
  uint4 k[HEADS_AT_ONCE][2], v[HEADS_AT_ONCE][2];
#pragma unroll
  for (int u = 0; u < HEADS_AT_ONCE; ++u) {
    const int head = at.head0 + u * C::ACROSS;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      k[u][e] = v[u][e] = make_uint4(0, 0, 0, 0);
      if (at.token < p.T && head < p.Hkv) {
        const int o = head * D + j * 16 + e * 8;
        k[u][e] = *reinterpret_cast<const uint4*>(static_cast<const T*>(p.k) +
                                                  at.token * p.k_stride + o);
        v[u][e] = *reinterpret_cast<const uint4*>(static_cast<const T*>(p.v) +
                                                  at.token * p.v_stride + o);
      }
    }
  }
  const int slot = slot_of(p, at.token);
  // neighbouring vectors of the warp are neighbouring tokens of a head; if
  // their slots are an even one and the next, their V codes share words
  const int side = static_cast<int>(at.token) & 1;
  const int slot2 = __shfl_xor_sync(0xffffffffu, slot, LANES);
  const bool paired = slot >= 0 && (slot & 1) == side && slot2 == (slot ^ 1);
  const unsigned page = max(slot, 0) / static_cast<unsigned>(p.page);
  const int o = max(slot, 0) - page * p.page, i = o & 15;
#pragma unroll
  for (int u = 0; u < HEADS_AT_ONCE; ++u) {
    const int head = at.head0 + u * C::ACROSS;
    const bool use = slot >= 0 && head < p.Hkv;
    const Kv4Codes kc = kv4_encode16<T, LANES>(k[u][0], k[u][1], use);
    const Kv4Codes vc = kv4_encode16<T, LANES>(v[u][0], v[u][1], use);
    const uint32_t send = side == 0 ? vc.hi : vc.lo;
    const uint32_t got = __shfl_xor_sync(0xffffffffu, send, LANES);
    if (!use) continue;
    uint8_t* blk = p.cache + ((static_cast<long long>(page) * p.Hkv + head) * (p.page >> 4) +
                              (o >> 4)) * L::BLOCK_BYTES;
    *reinterpret_cast<uint2*>(blk + i * L::ROW + j * 8) = make_uint2(kc.lo, kc.hi);
    uint8_t* vb = blk + L::OFF_V;
    if (paired) {
      // both tokens of a word in this warp: the even one's lane stores the
      // words of its first eight elements, the odd one's those of the others
      const uint32_t even = side == 0 ? vc.lo : got, odd = side == 0 ? got : vc.hi;
      *reinterpret_cast<uint2*>(vb + L::v_code_offset(i & ~1, 4 * j + 2 * side)) =
          make_uint2(__byte_perm(even, odd, 0x5410), __byte_perm(even, odd, 0x7632));
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *reinterpret_cast<uint16_t*>(vb + L::v_code_offset(i, 4 * j + e)) =
            static_cast<uint16_t>((e < 2 ? vc.lo : vc.hi) >> (16 * (e & 1)));
    }
    if (j == 0) {
      *reinterpret_cast<uint32_t*>(blk + L::OFF_KP + 4 * i) = kc.params;
      *reinterpret_cast<uint32_t*>(blk + L::OFF_VP + 4 * i) = vc.params;
    }
  }
}

// ------------------------------------------------------------------ read
__device__ __forceinline__ void store8(float* dst, const float (&x)[8]) {
  reinterpret_cast<float4*>(dst)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(dst)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* dst, const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = as_word<__nv_bfloat162>(__floats2bfloat162_rn(x[2 * i], x[2 * i + 1]));
  *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(__half* dst, const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = as_word<__half2>(__floats2half2_rn(x[2 * i], x[2 * i + 1]));
  *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
}

// step * code + zero of eight codes.  The nibbles under 0x000f000f are, as
// fp16 numbers, code 2^-24, under 0x00f000f0 code 2^-20; converted to fp32
// exactly, the powers of two go into the step, so the one rounding is the
// sum's, as for the code itself.
template <class T>
__device__ __forceinline__ void decode8(T* dst, uint32_t codes, uint32_t params) {
  const float2 sz = kv4_params(params);
  const float s24 = sz.x * 16777216.f, s20 = sz.x * 1048576.f;
  float x[8];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t w = codes >> (8 * i);
    const float2 lo = __half22float2(as_pair<__half2>(w & 0x000f000fu));
    const float2 hi = __half22float2(as_pair<__half2>(w & 0x00f000f0u));
    x[2 * i] = fmaf(s24, lo.x, sz.y);
    x[2 * i + 4] = fmaf(s24, lo.y, sz.y);
    x[2 * i + 1] = fmaf(s20, hi.x, sz.y);
    x[2 * i + 5] = fmaf(s20, hi.y, sz.y);
  }
  store8(dst, x);
}

template <int D, class T>
__global__ void __launch_bounds__(CACHE_THREADS) ra_kv4_read_kernel(const Kv4CopyParams p) {
  using L = Kv4<D>;
  constexpr int HEADS_AT_ONCE = 2;
  using C = CacheCta<D, 8, HEADS_AT_ONCE>;
  const Place at = place_of<C>(p.Hkv);
  const int j = at.lane;
  if (at.token >= p.T) return;
  const int slot = slot_of(p, at.token);
  const unsigned page = max(slot, 0) / static_cast<unsigned>(p.page);
  const int o = max(slot, 0) - page * p.page, i = o & 15;
  uint32_t kc[HEADS_AT_ONCE], vc[HEADS_AT_ONCE], kp[HEADS_AT_ONCE], vp[HEADS_AT_ONCE];
#pragma unroll
  for (int u = 0; u < HEADS_AT_ONCE; ++u) {
    const int head = at.head0 + u * C::ACROSS;
    kc[u] = vc[u] = kp[u] = vp[u] = 0;
    if (slot >= 0 && head < p.Hkv) {
      const uint8_t* blk = p.cache + ((static_cast<long long>(page) * p.Hkv + head) *
                                          (p.page >> 4) + (o >> 4)) * L::BLOCK_BYTES;
      kc[u] = *reinterpret_cast<const uint32_t*>(blk + i * L::ROW + j * 4);
      // the words with the token's halves of its elements, side by side with
      // those of its neighbour's
      const uint2 w = *reinterpret_cast<const uint2*>(blk + L::OFF_V +
                                                      L::v_code_offset(i & ~1, 2 * j));
      vc[u] = __byte_perm(w.x, w.y, (i & 1) ? 0x7632 : 0x5410);
      kp[u] = *reinterpret_cast<const uint32_t*>(blk + L::OFF_KP + 4 * i);
      vp[u] = *reinterpret_cast<const uint32_t*>(blk + L::OFF_VP + 4 * i);
    }
  }
#pragma unroll
  for (int u = 0; u < HEADS_AT_ONCE; ++u) {
    const int head = at.head0 + u * C::ACROSS;
    if (head >= p.Hkv) continue;
    const long long dst = (at.token * p.Hkv + head) * D + j * 8;
    decode8(static_cast<T*>(p.k_out) + dst, kc[u], kp[u]);
    decode8(static_cast<T*>(p.v_out) + dst, vc[u], vp[u]);
  }
}

template <class C>
cudaError_t launch_copy(void (*kernel)(const Kv4CopyParams), const Kv4CopyParams& p,
                        cudaStream_t stream) {
  const long long groups = (p.T + 15) / 16;
  const long long grid = groups * ((p.Hkv + C::HEADS - 1) / C::HEADS);
  if (grid > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  kernel<<<static_cast<unsigned>(grid), CACHE_THREADS, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv4_plan(const Kv4PlanParams& p, cudaStream_t stream) {
  const size_t smem = plan_smem_bytes(p.R);
  // The limit is the kernel's, not the launch's: set once a device, to what the
  // largest call needs.  Set to each call's own size, one thread's call lowered it
  // between another's and its launch, which then failed (25 of 8000 launches of two
  // threads with 8192 and 2600 requests).
  static int configured_dev[64] = {0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!configured_dev[dev]) {
    e = cudaFuncSetAttribute(ra_kv4_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(plan_smem_bytes(KV4_PLAN_MAX_R)));
    if (e != cudaSuccess) return e;
    configured_dev[dev] = 1;
  }
  // One CTA for what one CTA's threads do in a few rounds, else a cluster.
  long long work = p.max_tokens;
  if (p.table_out != p.table) work += static_cast<long long>(p.R) * p.W;
  if (p.pool_out != p.pool) work += p.num_pages;
  const unsigned ctas = work <= 8 * PLAN_THREADS ? 1 : 8;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(PLAN_THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = ctas;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, ra_kv4_plan_kernel, p);
}

namespace {

template <class T>
cudaError_t append(const Kv4CopyParams& p, int d, cudaStream_t stream) {
  return d == 128 ? launch_copy<CacheCta<128, 16, 1>>(ra_kv4_append_kernel<128, T>, p, stream)
                  : launch_copy<CacheCta<64, 16, 1>>(ra_kv4_append_kernel<64, T>, p, stream);
}

template <class T>
cudaError_t read(const Kv4CopyParams& p, int d, cudaStream_t stream) {
  return d == 128 ? launch_copy<CacheCta<128, 8, 2>>(ra_kv4_read_kernel<128, T>, p, stream)
                  : launch_copy<CacheCta<64, 8, 2>>(ra_kv4_read_kernel<64, T>, p, stream);
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4CopyParams& p, int d, int dtype, cudaStream_t stream) {
  return dtype == RA_BF16 ? append<__nv_bfloat16>(p, d, stream) : append<__half>(p, d, stream);
}

cudaError_t launch_kv4_read(const Kv4CopyParams& p, int d, int dtype, cudaStream_t stream) {
  return dtype == RA_BF16   ? read<__nv_bfloat16>(p, d, stream)
         : dtype == RA_FP16 ? read<__half>(p, d, stream)
                            : read<float>(p, d, stream);
}

cudaError_t read_and_clear_kv4_cache_status(unsigned long long* out) {
  unsigned long long v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_kv4_cache_status, sizeof(v));
  if (e == cudaSuccess && v != 0) e = cudaMemcpyToSymbol(g_kv4_cache_status, &zero, sizeof(zero));
  *out = v;
  return e;
}

}  // namespace ra
