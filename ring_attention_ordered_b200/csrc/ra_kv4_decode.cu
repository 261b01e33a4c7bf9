// Attention of a few query rows over the paged 4-bit K/V cache (sm_100a).
//
// For every request r, K/V head h and query row (query token t of the
// request, query head of h's group)
//     out = sum_c softmax_c(scale q . k_c) v_c,   lse = ln sum_c exp(scale q . k_c)
// over the cached tokens c the row sees, with k = ks codeK + kz and
// v = vs codeV + vz (step and zero of each token and head).
//
// The codes go to the matrix instructions as they are, and the steps and
// zeros are applied in fp32 around them, so nothing of K or V is rounded:
//     q . k   = ks (q . codeK) + kz sum(q)
//     sum p v = sum (p vs) codeV + sum p vz
// * A nibble under the mask 0x000f is a subnormal fp16 number, code 2^-24,
//   and under 0x00f0 it is code 2^-20: two codes become an operand register
//   with one AND (and one shift for every second pair), no conversion.  The
//   factor 16 between them is taken back in q (K: both lie in the sum over d,
//   q there is divided by 16) and in the result (V: they are different rows
//   of it).
// * q is scaled by a power of two per row so that its largest value lies in
//   [2^14, 2^15): exact in fp16 for bf16 and fp16 inputs down to 2^-24 of the
//   row's maximum.
// * p vs = 2^(s - m + 8) vs is rounded to fp16 (2^-12 relative, finer than the
//   output type) for the product with the codes; the row sum and the sum of
//   p vz use the fp32 values.  m is any reference that keeps p vs below
//   2^15: it is moved, and the accumulators rescaled, only when a value of the
//   block in hand would pass that, which one vote per block finds out.  The
//   step is part of what is bounded, so m follows max(s + log2 vs).
//
// Work: S^T = K q^T and O^T = V^T P^T with mma m16n8k16: a block of 16 tokens
// is the M side, 8 query rows (NT tiles of them) the N side, so the padding of
// a small group costs idle columns, not tensor time.  The transposition of P
// between the products is one movmatrix per 8 tokens.  Each warp streams
// pairs of blocks through a private ring of shared-memory stages (one bulk
// copy a block; a stage is refilled as soon as its words are in registers);
// the warps of a CTA take every 8th pair of the CTA's piece and are merged
// at its end.
//
// Split: the blocks of all (request, head, row tile) units form one line,
// request-major, and the CTAs take equal stretches of it, so a long request is spread
// over the GPU and short ones are packed, whatever the lengths, which only
// the device knows.  A unit that crosses stretches is merged by the CTA that
// finishes last (a counter that it sets back to zero), over the pieces in
// their order, so the result does not depend on the order of arrival.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "ptx_sm100.cuh"
#include "ra_internal.h"
#include "ra_kv4.cuh"
#include "ra_kv4_attn.cuh"
#include "ra_sync.cuh"

namespace ra {
namespace kv4d {

#ifndef KV4_WARPS
#define KV4_WARPS 8
#endif
constexpr int WARPS = KV4_WARPS;
constexpr int THREADS = WARPS * 32;
constexpr int STAGES = 2;          // of two blocks each
constexpr int MIN_CELLS = 48;     // cells below which a stretch is not cut further
// What a unit costs beside its blocks (start, merge, store), in blocks: it
// takes so many cells of the line before its first block.
constexpr int UNIT_COST = 16;
constexpr float P_SHIFT = 8.f;     // p vs = 2^P_SHIFT at the reference
constexpr float P_LIMIT = 32768.f;

__device__ unsigned long long g_status = 0ull;

template <int D, int NT>
struct Smem {
  static constexpr int RING = WARPS * STAGES * 2 * Kv4<D>::BLOCK_BYTES;
  static constexpr int ROWS = 8 * NT;
  static constexpr int RS = D + 4;                       // row stride of the merge buffer
  static constexpr int MERGE = WARPS * ROWS * RS * 4;
  static constexpr int OFF_ML = RING > MERGE ? RING : MERGE;
  static constexpr int OFF_BAR = OFF_ML + 2 * WARPS * ROWS * 4;
  static constexpr int BYTES = OFF_BAR + WARPS * STAGES * 8;
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
template <int N>
__device__ __forceinline__ void lds_words(uint32_t (&r)[N], uint32_t addr) {
  static_assert(N == 2 || N == 4, "8 or 16 bytes");
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
  else
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(addr));
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t r;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(addr));
  return r;
}
// Nibbles (0, 4), (1, 5), (2, 6), (3, 7) of a word as fp16 pairs: codes times
// 2^-24, 2^-20, 2^-24, 2^-20.
__device__ __forceinline__ void code_pairs(uint32_t x, uint32_t (&p)[4]) {
  const uint32_t y = x >> 8;
  p[0] = x & 0x000f000fu;
  p[1] = x & 0x00f000f0u;
  p[2] = y & 0x000f000fu;
  p[3] = y & 0x00f000f0u;
}

// Row `row`, elements 4 d4 .. 4 d4 + 3 of the warps' partials, merged in the
// warps' order.
template <int D, int NT>
__device__ __forceinline__ float4 merge_warps(const float* s_merge, const float* s_m,
                                              const float* s_l, int row, int d4, float& m,
                                              float& ls) {
  constexpr int ROWS = 8 * NT;
  m = -INFINITY;
  ls = 0.f;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int w = 0; w < WARPS; ++w) m = fmaxf(m, s_m[w * ROWS + row]);
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    const float mw = s_m[w * ROWS + row];
    if (mw == -INFINITY) continue;
    const float f = mw == m ? 1.f : ex2_approx(mw - m);
    const float4 x =
        *reinterpret_cast<const float4*>(s_merge + (w * ROWS + row) * Smem<D, NT>::RS + 4 * d4);
    a.x = fmaf(f, x.x, a.x);
    a.y = fmaf(f, x.y, a.y);
    a.z = fmaf(f, x.z, a.z);
    a.w = fmaf(f, x.w, a.w);
    ls = fmaf(f, s_l[w * ROWS + row], ls);
  }
  return a;
}

template <int D, int NT>
__global__ void __launch_bounds__(THREADS, (NT == 1 ? 16 : 8) / WARPS)
    ra_kv4_decode_kernel(const Kv4AttnParams p) {
  using L = Kv4<D>;
  using S = Smem<D, NT>;
  constexpr int WPL = D / 32;        // code words of a row per lane (16 or 8 bytes)
  constexpr int ROWS = 8 * NT;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint32_t s_abort;
  __shared__ int s_last;
  __shared__ Kv4Start s_start;
  __shared__ long long s_scan[WARPS + 1];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const uint32_t ring = smem_u32(smem) + warp * STAGES * 2 * L::BLOCK_BYTES;
  const uint32_t bars = smem_u32(smem) + S::OFF_BAR + warp * STAGES * 8;
  float* s_merge = reinterpret_cast<float*>(smem);
  float* s_m = reinterpret_cast<float*>(smem + S::OFF_ML);
  float* s_l = s_m + WARPS * ROWS;
  const Ctl cx{&s_abort, p.wait_limit_ns, &g_status};

  if (tid == 0) s_abort = 0u;
  if (lane == 0) {
    for (int i = 0; i < STAGES; ++i) mbar_init(bars + 8 * i, 1);
    fence_mbarrier_init();
  }
  kv4_fill_empty<D, THREADS>(p, &g_status);
  // the stretch of this CTA: [start.at, start.end) of the line of blocks
  kv4_find_start<ROWS, MIN_CELLS, UNIT_COST, WARPS>(p, KV4_BLOCK, s_scan, s_start);
  __syncthreads();
  long long at = s_start.at;
  const long long end = s_start.end;
  const long long per_cta = s_start.per_cta;
  int r = s_start.r;
  long long in_r = s_start.in_r;     // blocks of request r before `at`
  uint32_t it = 0;                   // pairs of blocks this warp has taken from its ring

  while (at < end) {
    Kv4Req q = kv4_request(p, r);
    const int nb = (q.len + KV4_BLOCK - 1) / KV4_BLOCK;
    const int rows = q.n * p.group;
    const int tiles = (rows + ROWS - 1) / ROWS;
    if (nb == 0 || in_r >= static_cast<long long>(tiles) * p.Hkv * (nb + UNIT_COST)) {
      ++r;
      in_r = 0;
      continue;
    }
    const int unit = static_cast<int>(in_r / (nb + UNIT_COST));
    const int off = static_cast<int>(in_r - static_cast<long long>(unit) * (nb + UNIT_COST));
    const int cells = static_cast<int>(min(end - at, static_cast<long long>(nb + UNIT_COST - off)));
    const long long u0 = at - off;
    const int b0 = max(off - UNIT_COST, 0), b1 = off + cells - UNIT_COST;
    at += cells;
    in_r += cells;
    if (b1 <= b0) continue;
    const int take = b1 - b0;
    const int h = unit / tiles, row0 = (unit - h * tiles) * ROWS;

    // ---- copies: pair i of this warp is blocks b0 + 2 (warp + WARPS i) and the
    // next; lane 2 j + x looks up block x of pair j (mod 16)
    const int pairs = (take + 1) >> 1;
    const int n_mine = pairs > warp ? (pairs - warp + WARPS - 1) / WARPS : 0;
    const uint32_t it0 = it;
    int ent = -1;
    uint32_t have = 0;   // bits 2 s, 2 s + 1: the blocks that stage s holds
    int issued = 0;
    auto issue_next = [&] {
      if (issued >= n_mine) return;
      if ((issued & 15) == 0) {
        const int blk = b0 + 2 * (warp + WARPS * (issued + (lane >> 1))) + (lane & 1);
        ent = blk < b1 ? kv4_block_index(p, r, h, blk, &g_status) : -1;
      }
      const int e0 = __shfl_sync(0xffffffffu, ent, 2 * (issued & 15));
      const int e1 = __shfl_sync(0xffffffffu, ent, 2 * (issued & 15) + 1);
      const uint32_t s = (it0 + issued) % STAGES;
      have = (have & ~(3u << (2 * s))) | ((e0 >= 0 ? 1u : 0u) << (2 * s)) |
             ((e1 >= 0 ? 2u : 0u) << (2 * s));
      if (lane == 0) {
        const uint32_t bar = bars + 8 * s, dst = ring + s * (2 * L::BLOCK_BYTES);
        mbar_arrive_expect_tx(bar, L::BLOCK_BYTES * ((e0 >= 0) + (e1 >= 0)));
        if (e0 >= 0)
          bulk_load(dst, p.cache + static_cast<long long>(e0) * L::BLOCK_BYTES, L::BLOCK_BYTES, bar);
        if (e1 >= 0)
          bulk_load(dst + L::BLOCK_BYTES, p.cache + static_cast<long long>(e1) * L::BLOCK_BYTES,
                    L::BLOCK_BYTES, bar);
      }
      ++issued;
    };
#pragma unroll
    for (int i = 0; i < STAGES; ++i) issue_next();

    // ---- q: operand registers, scale and sum of each row
    uint32_t qf[NT][2 * WPL][2];
    float rho[NT][2], sigma[NT][2];
    int lim[NT][2];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int row = row0 + 8 * j + g;
      float x[8 * WPL];
      kv4_load_q<8 * WPL>(p, q, h, row, rows, t * 8 * WPL, D, x);
      float am = 0.f, sum = 0.f;
#pragma unroll
      for (int i = 0; i < 8 * WPL; ++i) {
        am = fmaxf(am, fabsf(x[i]));
        sum += x[i];
      }
      am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 1));
      am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 2));
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      float up, down;
      kv4_row_scale(am, up, down);
      float y[8 * WPL];
#pragma unroll
      for (int i = 0; i < 8 * WPL; ++i) y[i] = x[i] * up;
#pragma unroll
      for (int w = 0; w < WPL; ++w) {
        const float* e = y + 8 * w;
        const float k = 0.0625f;
        qf[j][2 * w][0] = pack_f16x2(e[0], e[4]);
        qf[j][2 * w][1] = pack_f16x2(e[1] * k, e[5] * k);
        qf[j][2 * w + 1][0] = pack_f16x2(e[2], e[6]);
        qf[j][2 * w + 1][1] = pack_f16x2(e[3] * k, e[7] * k);
      }
      // columns 2t, 2t + 1 of the product are the rows of lanes 8t, 8t + 4
      const float ro = down * p.scale_log2, so = sum * p.scale_log2;
      const int lo = kv4_limit(p, q, row, rows);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int src = (2 * t + c) * 4;
        rho[j][c] = __shfl_sync(0xffffffffu, ro, src) * 16777216.f;
        sigma[j][c] = __shfl_sync(0xffffffffu, so, src);
        lim[j][c] = __shfl_sync(0xffffffffu, lo, src);
      }
    }
    int lim_min = lim[0][0];
#pragma unroll
    for (int j = 0; j < NT; ++j) lim_min = min(lim_min, min(lim[j][0], lim[j][1]));
    lim_min = __reduce_min_sync(0xffffffffu, lim_min);

    float o[NT][2 * WPL][4];
    float mo[NT][2], l[NT][2], z[NT][2];   // mo = P_SHIFT - m
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int i = 0; i < 2 * WPL; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[j][i][c] = 0.f;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        mo[j][c] = INFINITY;
        l[j][c] = z[j][c] = 0.f;
      }
    }

    // One pair of blocks.  TAIL: some of its tokens are hidden from some row.
      auto step = [&](auto tail_c, int i) {
      constexpr bool TAIL = decltype(tail_c)::value;
      const uint32_t s = (it0 + i) % STAGES;
      const uint32_t held = (have >> (2 * s)) & 3u;
      const uint32_t blk = ring + s * (2 * L::BLOCK_BYTES);
      float c[NT][2][4];
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int x = 0; x < 2; ++x) c[j][x][0] = c[j][x][1] = c[j][x][2] = c[j][x][3] = 0.f;
      uint32_t kp[2][2], vp[2][2], v0[2][WPL], v1[2][WPL];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const uint32_t at = blk + x * L::BLOCK_BYTES;
        uint32_t k0[WPL], k1[WPL];
        lds_words(k0, at + g * L::ROW + t * (4 * WPL));
        lds_words(k1, at + (g + 8) * L::ROW + t * (4 * WPL));
        kp[x][0] = lds32(at + L::OFF_KP + 4 * g);
        kp[x][1] = lds32(at + L::OFF_KP + 4 * g + 32);
        vp[x][0] = lds32(at + L::OFF_VP + 4 * g);
        vp[x][1] = lds32(at + L::OFF_VP + 4 * g + 32);
#pragma unroll
        for (int w = 0; w < WPL; ++w) {
          uint32_t a[4], b[4];
          code_pairs(k0[w], a);
          code_pairs(k1[w], b);
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            mma_f16(c[j][x], a[0], b[0], a[1], b[1], qf[j][2 * w][0], qf[j][2 * w][1]);
            mma_f16(c[j][x], a[2], b[2], a[3], b[3], qf[j][2 * w + 1][0], qf[j][2 * w + 1][1]);
          }
        }
        lds_words(v0[x], at + L::OFF_V + lane * (4 * WPL));
        lds_words(v1[x], at + L::OFF_V + 4 * D + lane * (4 * WPL));
      }
      __syncwarp();
      issue_next();   // everything of the stage is in registers

      const int key = (b0 + 2 * (warp + WARPS * i)) * KV4_BLOCK + g;
      uint32_t pb[NT][2][2];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        // element [x][q]: token key + 16 x + 8 (q / 2), query column 2 t + q % 2
        float e[2][4], pv[2][4];
        auto hidden = [&](int x, int q4) {
          return key + 16 * x + 8 * (q4 >> 1) >= lim[j][q4 & 1] || !((held >> x) & 1u);
        };
        auto weights = [&] {
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int q4 = 0; q4 < 4; ++q4) {
              const float2 ks = kv4_params(kp[x][q4 >> 1]);
              const float2 vs = kv4_params(vp[x][q4 >> 1]);
              const int cc = q4 & 1;
              // the score exactly as the reference below is formed from it:
              // scores may be so large that another rounding is a big factor
              const float sc = fmaf(c[j][x][q4] * rho[j][cc], ks.x, ks.y * sigma[j][cc]);
              e[x][q4] = ex2_approx(sc + mo[j][cc]);
              pv[x][q4] = e[x][q4] * vs.x;
            }
          if constexpr (TAIL) {
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
              for (int q4 = 0; q4 < 4; ++q4)
                if (hidden(x, q4)) e[x][q4] = pv[x][q4] = 0.f;
          }
        };
        weights();
        // the sum bounds each of them, and is NaN if one is
        const float top = ((pv[0][0] + pv[0][1]) + (pv[0][2] + pv[0][3])) +
                          ((pv[1][0] + pv[1][1]) + (pv[1][2] + pv[1][3]));
        if (__any_sync(0xffffffffu, !(top <= P_LIMIT))) {
          // move the reference to the largest s + log2(vs) so far
#pragma unroll
          for (int cc = 0; cc < 2; ++cc) {
            float w = -INFINITY;
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const float2 ks = kv4_params(kp[x][y]);
                const float lv = __log2f(fmaxf(kv4_params(vp[x][y]).x, 5.9604645e-8f));
                const float sc = fmaf(c[j][x][2 * y + cc] * rho[j][cc], ks.x, ks.y * sigma[j][cc]);
                if (!TAIL || !hidden(x, 2 * y + cc)) w = fmaxf(w, sc + lv);
              }
            w = fmaxf(w, __shfl_xor_sync(0xffffffffu, w, 4));
            w = fmaxf(w, __shfl_xor_sync(0xffffffffu, w, 8));
            w = fmaxf(w, __shfl_xor_sync(0xffffffffu, w, 16));
            const float mo_new = fminf(mo[j][cc], P_SHIFT - w);
            const float alpha = mo_new == mo[j][cc] ? 1.f : ex2_approx(mo_new - mo[j][cc]);
            mo[j][cc] = mo_new;
            l[j][cc] *= alpha;
            z[j][cc] *= alpha;
#pragma unroll
            for (int i2 = 0; i2 < 2 * WPL; ++i2) {
              o[j][i2][cc] *= alpha;
              o[j][i2][2 + cc] *= alpha;
            }
          }
          weights();
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4) {
            const float vz = kv4_params(vp[x][q4 >> 1]).y;
            const int cc = q4 & 1;
            l[j][cc] += e[x][q4];
            // a hidden token's zero may be NaN: 0 times it is not 0
            if (!TAIL || !hidden(x, q4)) z[j][cc] = fmaf(e[x][q4], vz, z[j][cc]);
          }
          pb[j][x][0] = transpose8(pack_f16x2(pv[x][0], pv[x][1]));
          pb[j][x][1] = transpose8(pack_f16x2(pv[x][2], pv[x][3]));
        }
      }
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int w = 0; w < WPL; ++w) {
          uint32_t a[4], b[4];
          code_pairs(v0[x][w], a);
          code_pairs(v1[x][w], b);
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            mma_f16(o[j][2 * w], a[0], a[1], b[0], b[1], pb[j][x][0], pb[j][x][1]);
            mma_f16(o[j][2 * w + 1], a[2], a[3], b[2], b[3], pb[j][x][0], pb[j][x][1]);
          }
        }
    };
    // pairs whose tokens every row sees, as long as their pages are there;
    // then the others
    const int n_seen = max(min(lim_min, b1 * KV4_BLOCK) / KV4_BLOCK - b0, 0) >> 1;
    const int n_full = n_seen > warp ? min((n_seen - warp + WARPS - 1) / WARPS, n_mine) : 0;
    bool alive = true;
    int done = 0;
    for (; done < n_full; ++done) {
      const uint32_t s = (it0 + done) % STAGES;
      alive = wait_warp(bars + 8 * s, ((it0 + done) / STAGES) & 1u, cx, KV4_SITE_COPY);
      if (!alive || ((have >> (2 * s)) & 3u) != 3u) break;
      step(std::false_type{}, done);
    }
    for (; alive && done < n_mine; ++done) {
      const uint32_t s = (it0 + done) % STAGES;
      alive = wait_warp(bars + 8 * s, ((it0 + done) / STAGES) & 1u, cx, KV4_SITE_COPY);
      if (alive) step(std::true_type{}, done);
    }
    if (!alive) {
      // let the copies in flight land before the shared memory goes
      for (int i = 0; i < issued; ++i)
        if (i + STAGES >= issued && lane == 0)
          drain_wait(bars + 8 * ((it0 + i) % STAGES), ((it0 + i) / STAGES) & 1u, 200000000ull);
      __syncwarp();
    }
    it = it0 + n_mine;

    // ---- merge the warps: A = sum p v (relative to m), m, l per row
    __syncthreads();   // every warp has left its ring, which the buffer overlaps
    if (s_abort) return;
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int cc = 0; cc < 2; ++cc) {
        float ls = l[j][cc], zs = z[j][cc];
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) {
          ls += __shfl_xor_sync(0xffffffffu, ls, x);
          zs += __shfl_xor_sync(0xffffffffu, zs, x);
        }
        const int row = 8 * j + 2 * t + cc;
        float* dst = s_merge + (warp * ROWS + row) * S::RS + g * (D / 8);
#pragma unroll
        for (int w = 0; w < WPL; ++w)
          *reinterpret_cast<float4*>(dst + 4 * w) =
              make_float4(fmaf(o[j][2 * w][cc], 16777216.f, zs),
                          fmaf(o[j][2 * w][2 + cc], 1048576.f, zs),
                          fmaf(o[j][2 * w + 1][cc], 16777216.f, zs),
                          fmaf(o[j][2 * w + 1][2 + cc], 1048576.f, zs));
        if (g == 0) {
          s_m[warp * ROWS + row] = P_SHIFT - mo[j][cc];
          s_l[warp * ROWS + row] = ls;
        }
      }
    __syncthreads();

    const bool whole = b0 == 0 && b1 == nb;
    // the CTAs whose stretches hold the unit's blocks
    const int c0 = static_cast<int>((u0 + UNIT_COST) / per_cta);
    const int c1 = static_cast<int>((u0 + UNIT_COST + nb - 1) / per_cta);
    float* slot = p.partials + (2ll * blockIdx.x + (static_cast<int>(blockIdx.x) == c0)) * KV4_PIECE_FLOATS;
    const int n_rows = min(ROWS, rows - row0);
    for (int i = tid; i < n_rows * (D / 4); i += THREADS) {
      const int row = i / (D / 4), d4 = i - row * (D / 4);
      float m, ls;
      const float4 a = merge_warps<D, NT>(s_merge, s_m, s_l, row, d4, m, ls);
      if (whole) {
        kv4_store(p, q, h, row0 + row, 4 * d4, D, a, m - P_SHIFT, ls);
      } else {
        *reinterpret_cast<float4*>(slot + row * D + 4 * d4) = a;
        if (d4 == 0) {
          slot[ROWS * D + row] = m;
          slot[ROWS * D + ROWS + row] = ls;
        }
      }
    }
    if (!whole) {
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        const unsigned old = atomicAdd(p.counters + c0, 1u);
        s_last = old == static_cast<unsigned>(c1 - c0);
        if (s_last) p.counters[c0] = 0u;
        __threadfence();
      }
      __syncthreads();
      if (s_last) {
        // warp w folds the pieces c0 + w, c0 + w + WARPS, ..., then the warps
        // are merged as before
        constexpr int LPR = D / 4;             // lanes of a row
        constexpr int RPW = 32 / LPR;          // rows a warp folds at once
        const int d4 = lane % LPR;
        for (int rb = 0; rb < n_rows; rb += RPW) {
          const int row = min(rb + lane / LPR, n_rows - 1);
          float m = -INFINITY, ls = 0.f;
          float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
          constexpr int U = 4;
          for (int c = c0 + warp; c <= c1; c += U * WARPS) {
            float mm[U], ll[U];
            float4 aa[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
              const int cu = c + u * WARPS;
              const float* src = p.partials + (2ll * cu + (cu == c0)) * KV4_PIECE_FLOATS;
              mm[u] = -INFINITY;
              if (cu <= c1) {
                mm[u] = __ldcg(src + ROWS * D + row);
                ll[u] = __ldcg(src + ROWS * D + ROWS + row);
                aa[u] = __ldcg(reinterpret_cast<const float4*>(src + row * D + 4 * d4));
              }
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
              if (mm[u] != -INFINITY) kv4_merge(m, ls, a, mm[u], ll[u], aa[u]);
          }
          *reinterpret_cast<float4*>(s_merge + (warp * ROWS + row) * S::RS + 4 * d4) = a;
          if (d4 == 0) {
            s_m[warp * ROWS + row] = m;
            s_l[warp * ROWS + row] = ls;
          }
        }
        __syncthreads();
        for (int i = tid; i < n_rows * (D / 4); i += THREADS) {
          const int row = i / (D / 4), d4 = i - row * (D / 4);
          float m, ls;
          const float4 a = merge_warps<D, NT>(s_merge, s_m, s_l, row, d4, m, ls);
          kv4_store(p, q, h, row0 + row, 4 * d4, D, a, m - P_SHIFT, ls);
        }
      }
    }
    fence_proxy_async();
    __syncthreads();     // the merge buffer is free for copies again
  }
}

template <int D, int NT>
cudaError_t launch(const Kv4AttnParams& p, int num_sms, int max_ctas, cudaStream_t stream) {
  using S = Smem<D, NT>;
  cudaError_t e = cudaFuncSetAttribute(ra_kv4_decode_kernel<D, NT>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, S::BYTES);
  if (e != cudaSuccess) return e;
  int grid = num_sms * ((NT == 1 ? 16 : 8) / WARPS);
  if (max_ctas > 0 && max_ctas < grid) grid = max_ctas;
  if (grid > KV4_MAX_CTAS) grid = KV4_MAX_CTAS;
  ra_kv4_decode_kernel<D, NT><<<grid, THREADS, S::BYTES, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace kv4d

cudaError_t launch_kv4_decode(const Kv4AttnParams& p, int d, int rows, int num_sms, int max_ctas,
                              cudaStream_t stream) {
  if (rows <= 8)
    return d == 128 ? kv4d::launch<128, 1>(p, num_sms, max_ctas, stream)
                    : kv4d::launch<64, 1>(p, num_sms, max_ctas, stream);
  return d == 128 ? kv4d::launch<128, 2>(p, num_sms, max_ctas, stream)
                  : kv4d::launch<64, 2>(p, num_sms, max_ctas, stream);
}

cudaError_t read_and_clear_kv4_decode_status(unsigned long long* out) {
  unsigned long long v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, kv4d::g_status, sizeof(v));
  if (e == cudaSuccess && v != 0) e = cudaMemcpyToSymbol(kv4d::g_status, &zero, sizeof(zero));
  *out = v;
  return e;
}

}  // namespace ra
