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
//     sum p v = sum (p vs) (codeV - 8) + sum p (vz + 8 vs)
// * A nibble under a mask is a subnormal fp16 number, code 2^-24 under 0x000f, or a
//   power of two times that after a shift: two codes become an operand register with
//   one AND and a shift, no conversion.  An instruction aligns its products before
//   it adds them, and numbers far below fp16's normal range lose places there.
//   So K's codes enter as code 2^-22 and code 2^-18 (one shift for two pairs; q is
//   divided by 16 where it meets the larger ones): with 2^-24 and 2^-20, half a shift
//   less, lse was up to 1.1e-5 off for fp16 q and short requests, 3e-6 so (193 us and
//   196 us below; all at 2^-20, a shift more, 202 us).  V takes all codes at 2^-20,
//   which over a million tokens shows (0.0016 off, below, and 0.0019 with 2^-24).
// * The 8 is taken off V's codes after the product, so that nothing is done to
//   a single code: one more matrix instruction per block forms the sum of
//   the rounded p vs.  Two blocks go through together, and the second enters
//   as (15 - code) (-p vs), its complement, which costs nothing: what the two
//   add to the accumulators is centred, so neither they nor their rounding,
//   which is towards zero, grow with sum p vs.  (One request of 1M tokens, bf16,
//   relative to the exact result: 0.0026 off with the codes as they are,
//   0.0016 so, which is the rounding of the output.  Taking 8 off each code
//   instead costs an operation a pair: 234 us against 200 us for 8 x 32K tokens
//   of 32 heads.)
// * q is scaled by a power of two per row so that its largest value lies in
//   [2^14, 2^15): exact in fp16 for bf16 and fp16 inputs down to 2^-24 of the
//   row's maximum.
// * p vs = 2^(s - m + 8) vs is rounded to fp16 (half a step, 2^-11 relative: no
//   coarser than the output) for the product with the codes; the row sum and
//   the sum of p vz use the fp32 values.  m is any reference that keeps p vs below
//   2^15: it is moved, and the accumulators rescaled, only when a value of the
//   two blocks in hand would pass that, which one vote finds out.  The step is
//   part of what is bounded, so m follows max(s + log2 vs).
//
// Work: S^T = K q^T and O^T = V^T P^T with mma m16n8k16: a block of 16 tokens
// is the M side, 8 query rows (NT tiles of them) the N side, so the padding of
// a small group costs idle columns, not tensor time.  The transposition of P
// between the products is one movmatrix per 8 tokens.  Each warp streams
// pairs of blocks through a private ring of shared-memory stages (one bulk
// copy for two that lie side by side, 3% less than one for each; a stage is
// refilled as soon as its words are in registers).
//
// Split: the blocks of all (request, head, row tile) units form one line,
// request-major, and the warps of the launch take equal stretches of it, so a
// long request is spread over the GPU and short ones are packed, whatever the
// lengths, which only the device knows.  A unit inside one warp's stretch is
// finished by that warp alone, without the CTA; one that crosses warps is merged
// by their CTA at its end, and one that crosses CTAs by the CTA that finishes last of
// each 16, then by the last of these (counters that they set back to zero),
// always over the pieces in their order, so the result does not depend on the
// order of arrival.
//
// What bounds it, measured: with much work the instruction issue of unpacking
// (271 instructions a block and head, 55% of the issue slots, the ALU pipe 52%
// busy): 8 requests of 32K tokens, 32 K/V heads, d = 128 take 196 us at 1.95 GHz,
// 5570 GB/s of cache, 0.85 of the copy rate; it follows the clock, and under a load
// that lasts, where the power limit holds that at 1.71 GHz, it takes 223 us (0.75).
// With little work the chain lens, table, block,
// products, merge: 8.8 us for one request of 509 tokens.
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

// Cells below which a stretch is not cut further (one request of 509 tokens: 9.3 us
// with 2, 8.9 us with 4, 9.8 us with 8).
constexpr int MIN_CELLS = 4;
// What a unit costs a warp beside its blocks (start, store), in blocks: it
// takes so many cells of the line before its first block (64 requests of 0 to 8191
// tokens: 36.8 us with 4, 30.9 us with 8, 31.4 us with 12; 8 of 32K tokens and 32
// heads: 193 us with 4, 191 us with 8, 195 us with 16).
constexpr int UNIT_COST = 8;
constexpr int FOLD = KV4_FOLD;     // pieces that one CTA folds at a time
constexpr float P_SHIFT = 8.f;     // p vs = 2^P_SHIFT at the reference
constexpr float P_LIMIT = 32768.f;

__device__ unsigned long long g_status = 0ull;

// Shared memory: the warps' rings, a warp's ring taking its tail piece once
// the warp has read its last block; the head pieces; their m and l; barriers.
template <int D, int NT>
struct Smem {
  static constexpr int STAGES = 2;   // of two blocks each
  // One CTA an SM: two of 8 warps make twice as many units cross CTAs (one request of
  // 1M tokens: 71 us against 67 us).  Of 16 warps, with 128 registers a thread, where
  // what that spills costs less than half the warps: 16 rows at d = 64, which spill
  // 508 bytes, 37.9 us against 42.2 us with 8 warps (8 x 8 drafts over 4000 tokens, 64
  // query and 8 K/V heads), 31.1 against 32.1 us (16 x 1 to 8 drafts over 900 to 16000),
  // 19.2 against 18.8 us (16 x 4 drafts over 8000).  16 rows at d = 128 need 249 registers.
  static constexpr int WARPS = D * NT <= 128 ? 16 : 8;
  static constexpr int THREADS = WARPS * 32;
  static constexpr int WRING = STAGES * 2 * Kv4<D>::BLOCK_BYTES;
  static constexpr int ROWS = 8 * NT;
  static constexpr int RS = D + 4;                       // row stride of a piece
  static constexpr int PIECE = ROWS * RS * 4;
  static_assert(PIECE <= WRING, "a piece fits the ring");
  static constexpr int OFF_HEAD = WARPS * WRING;
  static constexpr int OFF_ML = OFF_HEAD + WARPS * PIECE;
  static constexpr int OFF_BAR = OFF_ML + 2 * 2 * WARPS * ROWS * 4;
  static constexpr int BYTES = OFF_BAR + WARPS * STAGES * 8;
  // of a piece in the workspace: m and l of its rows, then the rows
  static constexpr int SLOT = 2 * ROWS + ROWS * D;       // floats
  static_assert(SLOT <= KV4_PIECE_FLOATS && SLOT % 4 == 0, "a piece fits its place");
  static_assert(FOLD * SLOT * 4 <= OFF_ML, "the pieces of a fold fit the shared memory");
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same onto zeros.
__device__ __forceinline__ void mma_f16_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
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
// 2^-22, 2^-18, 2^-22, 2^-18.
__device__ __forceinline__ void code_pairs(uint32_t x, uint32_t (&p)[4]) {
  const uint32_t y = x << 2, z = x >> 6;
  p[0] = y & 0x003c003cu;
  p[1] = y & 0x03c003c0u;
  p[2] = z & 0x003c003cu;
  p[3] = z & 0x03c003c0u;
}
// All four as codes (or 15 less the codes) times 2^-20.
template <bool COMPLEMENT>
__device__ __forceinline__ void code_pairs_v(uint32_t x, uint32_t (&p)[4]) {
  const uint32_t m = 0x00f000f0u;
  const uint32_t a = x << 4, b = x >> 4, c = x >> 8;
  p[0] = COMPLEMENT ? ~a & m : a & m;
  p[1] = COMPLEMENT ? ~x & m : x & m;
  p[2] = COMPLEMENT ? ~b & m : b & m;
  p[3] = COMPLEMENT ? ~c & m : c & m;
}

// A unit of which this CTA holds pieces: where its rows are, and the warps w0
// .. w1 of the launch.
struct Group {
  int n_rows, first, h, row0, w0, w1;
};

template <int D, int NT>
__device__ __forceinline__ float* kv4_slot(const Kv4AttnParams& p, int cta, bool starts) {
  return p.partials + (2ll * cta + starts) * KV4_PIECE_FLOATS;
}

// Pieces of a unit in shared memory (float offsets): the i-th has its rows at
// rows + i step, row_step apart, and m, l of row x at ml + i ml_step + 2 x; the
// first one is at rows0 and ml0.
struct Pieces {
  int n, rows0, rows, step, row_step, ml0, ml, ml_step;
};

// Merges elements d .. d + 3 of their row `row`, in their order: stored as the
// unit's result, or, if `slot` is given, as a piece there.  First the largest m,
// then the sums: the loads of a few pieces are in flight together (one piece
// after the other, running maximum: 64 requests of 0 to 8191 tokens 31.6 us, so
// 30.8 us).
template <int D, int NT>
__device__ __forceinline__ void kv4_merge_row(const Kv4AttnParams& p, const Group& u,
                                              const Pieces& x, int row, int d, const float* smem,
                                              float* slot) {
  auto ml = [&](int c) {
    return *reinterpret_cast<const float2*>(smem + (c == 0 ? x.ml0 : x.ml + c * x.ml_step) +
                                            2 * row);
  };
  float m = -INFINITY, ls = 0.f;
#pragma unroll 4
  for (int c = 0; c < x.n; ++c) m = fmaxf(m, ml(c).x);
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int c = 0; c < x.n; ++c) {
    const float2 t = ml(c);
    const float4 b = *reinterpret_cast<const float4*>(
        smem + (c == 0 ? x.rows0 : x.rows + c * x.step) + row * x.row_step + d);
    // a piece whose row saw nothing has m = -inf and zeros
    const float f = t.x == m ? 1.f : ex2_approx(t.x - m);
    ls = fmaf(t.y, f, ls);
    a.x = fmaf(b.x, f, a.x);
    a.y = fmaf(b.y, f, a.y);
    a.z = fmaf(b.z, f, a.z);
    a.w = fmaf(b.w, f, a.w);
  }
  if (slot == nullptr) {
    kv4_store(p, u.first, u.h, u.row0 + row, d, D, a, m - P_SHIFT, ls);
  } else {
    *reinterpret_cast<float4*>(slot + 2 * Smem<D, NT>::ROWS + row * D + d) = a;
    if (d == 0) *reinterpret_cast<float2*>(slot + 2 * row) = make_float2(m, ls);
  }
}

// Pieces of unit u in the workspace, of the CTAs c0 + i step, i < n, folded in
// that order: stored as the result, or as the piece of the first of them.
// smem: room for the pieces.
template <int D, int NT>
__device__ __forceinline__ void kv4_fold(const Kv4AttnParams& p, const Group u, int c0, int step,
                                         int n, bool starts, bool finish, float* smem) {
  using S = Smem<D, NT>;
  const int chunks = (2 * S::ROWS + u.n_rows * D) / 4;
#pragma unroll 1
  for (int c = 0; c < n; ++c) {
    const float* src = kv4_slot<D, NT>(p, c0 + c * step, starts && c == 0);
    const uint32_t dst = smem_u32(smem + c * S::SLOT);
#pragma unroll 1
    for (int i = threadIdx.x; i < chunks; i += S::THREADS)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + 16 * i), "l"(src + 4 * i)
                   : "memory");
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  const Pieces x = {n, 2 * S::ROWS, 2 * S::ROWS, S::SLOT, D, 0, 0, S::SLOT};
  float* slot = finish ? nullptr : kv4_slot<D, NT>(p, c0, starts);
  constexpr int LPR = D / 4;             // lanes of a row
#pragma unroll 1
  for (int i = threadIdx.x; i < u.n_rows * LPR; i += S::THREADS)
    kv4_merge_row<D, NT>(p, u, x, i / LPR, 4 * (i % LPR), smem, slot);
  __syncthreads();
}

// Counts this CTA, all of whose threads have passed a barrier since they wrote,
// in at `counter`; true if it is the last of `n`, which sets the counter back
// to zero.  By one thread.
__device__ __forceinline__ bool kv4_last(unsigned* counter, int n) {
  __threadfence();
  const bool last = atomicAdd(counter, 1u) == static_cast<unsigned>(n - 1);
  if (last) {
    __threadfence();
    *counter = 0u;
  }
  return last;
}

template <int D, int NT>
__global__ void __launch_bounds__((Smem<D, NT>::THREADS), 1)
    ra_kv4_decode_kernel(const __grid_constant__ Kv4AttnParams p) {
  using L = Kv4<D>;
  using S = Smem<D, NT>;
  constexpr int WPL = D / 32;        // code words of a row per lane (16 or 8 bytes)
  constexpr int ROWS = 8 * NT, STAGES = S::STAGES, WARPS = S::WARPS, THREADS = S::THREADS;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint32_t s_abort;
  __shared__ bool s_last[2];
  __shared__ Kv4Start s_start[WARPS];
  __shared__ int s_scan[3 * WARPS];
  __shared__ Group s_group[WARPS + 1];   // 0: the CTA's first piece, 1 + w: warp w's tail
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const uint32_t ring = smem_u32(smem) + warp * S::WRING;
  const uint32_t bars = smem_u32(smem) + S::OFF_BAR + warp * STAGES * 8;
  auto piece_at = [&](int w, bool head) {
    return reinterpret_cast<float*>(smem + (head ? S::OFF_HEAD + w * S::PIECE : w * S::WRING));
  };
  float* s_ml = reinterpret_cast<float*>(smem + S::OFF_ML);   // [warp][head][row][m, l]
  const Ctl cx{&s_abort, p.wait_limit_ns, &g_status};

  if (tid == 0) s_abort = 0u;
  if (tid <= WARPS) s_group[tid].n_rows = 0;
  if (lane == 0) {
    for (int i = 0; i < STAGES; ++i) mbar_init(bars + 8 * i, 1);
    fence_mbarrier_init();
  }
  __syncthreads();
  // the stretch of this warp: [at, end) of the line of cells
  const int me = blockIdx.x * WARPS + warp;
  Kv4Line line;
  const Kv4Start start = kv4_find_start<ROWS, WARPS>(p, UNIT_COST, MIN_CELLS, me, gridDim.x * WARPS,
                                                     s_scan, s_start, line);
  const int per = line.per;
  int at = me < (line.total + per - 1) / per ? me * per : line.total;
  const int end = line.total - at < per ? line.total : at + per;
  int r = start.r, unit = start.unit, off = start.off;
  uint32_t it = 0;                   // pairs of blocks this warp has taken from its ring
  bool alive = true;

  while (at < end && r < p.R) {
    const Kv4Req q = kv4_request(p, r);
    const int nb = (q.len + KV4_BLOCK - 1) / KV4_BLOCK;
    const int rows = q.n * p.group;
    const int tiles = (rows + ROWS - 1) / ROWS;
    if (nb == 0 || rows > p.rows_max || unit >= tiles * p.Hkv) {
      ++r;
      unit = off = 0;
      continue;
    }
    const int all = line.cells(nb);
    const int cells = min(end - at, all - off);
    // the unit's blocks are in the cells [first, last]
    const int first = at - off + line.lead, last = first + ((nb - 1) >> line.shift);
    const int b0 = max(off - line.lead, 0) << line.shift;
    const int b1 = min(max(off + cells - line.lead, 0) << line.shift, nb);
    const int here = unit;
    at += cells;
    off += cells;
    if (off == all) {
      ++unit;
      off = 0;
    }
    if (b1 <= b0) continue;
    const int take = b1 - b0;
    const int h = here / tiles, row0 = (here - h * tiles) * ROWS;

    // ---- q: on its way while the pages are looked up
    uint4 qw[NT][WPL];
#pragma unroll
    for (int j = 0; j < NT; ++j)
      kv4_load_q<8 * WPL>(p, q, h, row0 + 8 * j + g, rows, t * 8 * WPL, D, qw[j]);

    // ---- copies: pair i is blocks b0 + 2 i and the next; lane j looks up
    // block j (mod 32) from b0
    const int n_mine = (take + 1) >> 1;
    const uint32_t it0 = it;
    int ent = -1;
    uint32_t have = 0;   // bits 2 s, 2 s + 1: the blocks that stage s holds
    int issued = 0;
    auto issue_next = [&] {
      if (issued >= n_mine) return;
      if ((issued & 15) == 0) {
        const int blk = b0 + 2 * issued + lane;
        ent = blk < b1 ? kv4_block_index(p, r, h, blk, &g_status) : -1;
      }
      const int e0 = __shfl_sync(0xffffffffu, ent, 2 * (issued & 15));
      const int e1 = __shfl_sync(0xffffffffu, ent, 2 * (issued & 15) + 1);
      const uint32_t s = (it0 + issued) % STAGES;
      const uint32_t bar = bars + 8 * s, dst = ring + s * (2 * L::BLOCK_BYTES);
      const uint8_t* src = p.cache + static_cast<long long>(e0) * L::BLOCK_BYTES;
      if (e0 >= 0 && e1 == e0 + 1) {
        // side by side in one page: one copy
        have |= 3u << (2 * s);
        if (elect_one()) {
          mbar_arrive_expect_tx(bar, 2 * L::BLOCK_BYTES);
          bulk_load(dst, src, 2 * L::BLOCK_BYTES, bar);
        }
      } else {
        have = (have & ~(3u << (2 * s))) | ((e0 >= 0 ? 1u : 0u) << (2 * s)) |
               ((e1 >= 0 ? 2u : 0u) << (2 * s));
        if (lane == 0) {
          mbar_arrive_expect_tx(bar, L::BLOCK_BYTES * ((e0 >= 0) + (e1 >= 0)));
          if (e0 >= 0) bulk_load(dst, src, L::BLOCK_BYTES, bar);
          if (e1 >= 0)
            bulk_load(dst + L::BLOCK_BYTES,
                      p.cache + static_cast<long long>(e1) * L::BLOCK_BYTES, L::BLOCK_BYTES, bar);
        }
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
#pragma unroll
      for (int i = 0; i < WPL; ++i) {
        const uint32_t w[4] = {qw[j][i].x, qw[j][i].y, qw[j][i].z, qw[j][i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 f = kv4_q_pair(p, w[k]);
          x[8 * i + 2 * k] = f.x;
          x[8 * i + 2 * k + 1] = f.y;
        }
      }
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
        rho[j][c] = __shfl_sync(0xffffffffu, ro, src) * 4194304.f;
        sigma[j][c] = __shfl_sync(0xffffffffu, so, src);
        lim[j][c] = __shfl_sync(0xffffffffu, lo, src);
      }
    }
    int lim_min = lim[0][0];
#pragma unroll
    for (int j = 0; j < NT; ++j) lim_min = min(lim_min, min(lim[j][0], lim[j][1]));
    lim_min = __reduce_min_sync(0xffffffffu, lim_min);

    float o[NT][2 * WPL][4], c8[NT][4];    // c8: what makes it codes less 8
    float mo[NT][2], l[NT][2], z[NT][2];   // mo = P_SHIFT - m
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int i = 0; i < 2 * WPL; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[j][i][c] = 0.f;
      c8[j][0] = c8[j][1] = c8[j][2] = c8[j][3] = 0.f;
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
      uint32_t kp[2][2], vp[2][2];
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
            if (w == 0)
              mma_f16_first(c[j][x], a[0], b[0], a[1], b[1], qf[j][0][0], qf[j][0][1]);
            else
              mma_f16(c[j][x], a[0], b[0], a[1], b[1], qf[j][2 * w][0], qf[j][2 * w][1]);
            mma_f16(c[j][x], a[2], b[2], a[3], b[3], qf[j][2 * w + 1][0], qf[j][2 * w + 1][1]);
          }
        }
      }

      const int key = (b0 + 2 * i) * KV4_BLOCK + g;
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
            c8[j][cc] *= alpha;
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
            const float2 vs = kv4_params(vp[x][q4 >> 1]);
            const float vz = fmaf(8.f, vs.x, vs.y);   // the value of code 8
            const int cc = q4 & 1;
            l[j][cc] += e[x][q4];
            // a hidden token's zero may be NaN: 0 times it is not 0
            if (!TAIL || !hidden(x, q4)) z[j][cc] = fmaf(e[x][q4], vz, z[j][cc]);
          }
          pb[j][x][0] = transpose8(pack_f16x2(pv[x][0], pv[x][1]));
          pb[j][x][1] = transpose8(pack_f16x2(pv[x][2], pv[x][3]));
        }
      }
      uint32_t v0[2][WPL], v1[2][WPL];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const uint32_t at = blk + x * L::BLOCK_BYTES + L::OFF_V + lane * (4 * WPL);
        lds_words(v0[x], at);
        lds_words(v1[x], at + 4 * D);
      }
      __syncwarp();
      issue_next();   // everything of the stage is in registers
      // block 0 adds p vs code, and p vs times -8; block 1 adds -p vs (15 - code),
      // and -p vs times -7
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          if (x == 1) {
            pb[j][x][0] ^= 0x80008000u;
            pb[j][x][1] ^= 0x80008000u;
          }
          const uint32_t k = x == 0 ? 0x80808080u : 0x80708070u;   // -8 2^-20, -7 2^-20
          mma_f16(c8[j], k, k, k, k, pb[j][x][0], pb[j][x][1]);
        }
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int w = 0; w < WPL; ++w) {
          uint32_t a[4], b[4];
          if (x == 0) {
            code_pairs_v<false>(v0[x][w], a);
            code_pairs_v<false>(v1[x][w], b);
          } else {
            code_pairs_v<true>(v0[x][w], a);
            code_pairs_v<true>(v1[x][w], b);
          }
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            mma_f16(o[j][2 * w], a[0], a[1], b[0], b[1], pb[j][x][0], pb[j][x][1]);
            mma_f16(o[j][2 * w + 1], a[2], a[3], b[2], b[3], pb[j][x][0], pb[j][x][1]);
          }
        }
    };
    // pairs whose tokens every row sees, as long as their pages are there;
    // then the others
    const int n_full = max(min(lim_min / KV4_BLOCK, b1) - b0, 0) >> 1;
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
    it = it0 + n_mine;
    if (!alive) {
      // let the copies in flight land before the shared memory goes
      for (int i = max(issued - STAGES, 0); i < issued; ++i)
        if (lane == 0)
          drain_wait(bars + 8 * ((it0 + i) % STAGES), ((it0 + i) / STAGES) & 1u, 200000000ull);
      __syncwarp();
      break;
    }

    // ---- the piece's result: A = sum p v relative to m, and l
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i2 = 0; i2 < 2 * WPL; ++i2)
#pragma unroll
        for (int cc = 0; cc < 2; ++cc) {
          o[j][i2][cc] += c8[j][cc];
          o[j][i2][2 + cc] += c8[j][cc];
        }
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int cc = 0; cc < 2; ++cc)
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) {
          l[j][cc] += __shfl_xor_sync(0xffffffffu, l[j][cc], x);
          z[j][cc] += __shfl_xor_sync(0xffffffffu, z[j][cc], x);
        }
    auto values = [&](int j, int cc, int w) {   // elements g d/8 + 4 w .. + 3 of column 2 t + cc
      return make_float4(fmaf(o[j][2 * w][cc], 1048576.f, z[j][cc]),
                         fmaf(o[j][2 * w][2 + cc], 1048576.f, z[j][cc]),
                         fmaf(o[j][2 * w + 1][cc], 1048576.f, z[j][cc]),
                         fmaf(o[j][2 * w + 1][2 + cc], 1048576.f, z[j][cc]));
    };
    const bool head = first < me * per;              // its blocks begin before this warp's
    const bool open = last >= me * per + per;        // and go on behind them
    if (!head && !open) {
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int cc = 0; cc < 2; ++cc) {
          const int row = row0 + 8 * j + 2 * t + cc;
          if (row < rows)
#pragma unroll
            for (int w = 0; w < WPL; ++w)
              kv4_store(p, q.first, h, row, g * (D / 8) + 4 * w, D, values(j, cc, w), -mo[j][cc],
                        l[j][cc]);
        }
      continue;
    }
    if (!head) __syncwarp();   // every lane has read its last block: the ring is free
    float* dst = piece_at(warp, head);
    float* ml = s_ml + ((warp * 2 + head) * ROWS) * 2;
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int cc = 0; cc < 2; ++cc) {
        const int row = 8 * j + 2 * t + cc;
#pragma unroll
        for (int w = 0; w < WPL; ++w)
          *reinterpret_cast<float4*>(dst + row * S::RS + g * (D / 8) + 4 * w) = values(j, cc, w);
        if (g == 0) {
          ml[2 * row] = P_SHIFT - mo[j][cc];
          ml[2 * row + 1] = l[j][cc];
        }
      }
    if (lane == 0 && (!head || warp == 0))
      s_group[head ? 0 : 1 + warp] = {min(ROWS, rows - row0), q.first, h, row0, first / per,
                                      last / per};
  }

  // ---- units that cross warps: merged by the CTA, their rows dealt over its
  // threads
  __syncthreads();
  if (s_abort) return;
  const int cta0 = blockIdx.x * WARPS;
  const bool any = lane <= WARPS && s_group[min(lane, WARPS)].n_rows > 0;
  const unsigned groups = __ballot_sync(0xffffffffu, any);
  // those of which other CTAs hold pieces
  const unsigned crossing = __ballot_sync(
      0xffffffffu, any && s_group[lane].w0 / WARPS != s_group[lane].w1 / WARPS);
  float* const pieces = reinterpret_cast<float*>(smem);
  constexpr int LPR = D / 4;             // lanes of a row
  int base = 0;                          // rows of the groups before
#pragma unroll 1
  for (unsigned rest = groups; rest != 0; rest &= rest - 1) {
    const int k = __ffs(rest) - 1;
    const Group u = s_group[k];
    // this thread's first row of the group
    int row = (tid / LPR - base) % (THREADS / LPR);
    if (row < 0) row += THREADS / LPR;
    base += u.n_rows;
    if (row >= u.n_rows) continue;
    const int lo = max(u.w0 - cta0, 0), hi = min(u.w1 - cta0, WARPS - 1);
    const bool head = cta0 + lo != u.w0;     // the first piece is no tail
    const Pieces x = {hi - lo + 1,
                      head ? S::OFF_HEAD / 4 + lo * (S::PIECE / 4) : lo * (S::WRING / 4),
                      S::OFF_HEAD / 4 + lo * (S::PIECE / 4), S::PIECE / 4, S::RS,
                      S::OFF_ML / 4 + (2 * lo + head) * 2 * ROWS,
                      S::OFF_ML / 4 + (2 * lo + 1) * 2 * ROWS, 4 * ROWS};
    float* slot = (crossing >> k) & 1u
                      ? kv4_slot<D, NT>(p, blockIdx.x,
                                        static_cast<int>(blockIdx.x) == u.w0 / WARPS)
                      : nullptr;
#pragma unroll 1
    for (; row < u.n_rows; row += THREADS / LPR)
      kv4_merge_row<D, NT>(p, u, x, row, 4 * (tid % LPR), pieces, slot);
  }

  // ---- units that cross CTAs, one from before this CTA and one to behind it: the
  // last of every FOLD of them folds their pieces, the last to do so folds these
  if (crossing == 0) {
    if (line.odd) kv4_fill_empty<D, THREADS>(p, &g_status);
    return;
  }
  __syncthreads();   // all is written, and the pieces in shared memory have been read
  const int k0 = __ffs(crossing) - 1, k1 = 31 - __clz(crossing);
  if (tid < 2) {
    const Group u = s_group[tid == 0 ? k0 : k1];
    const int c0 = u.w0 / WARPS, c1 = u.w1 / WARPS;
    const int sub = (static_cast<int>(blockIdx.x) - c0) / FOLD, first = c0 + sub * FOLD;
    s_last[tid] = (tid == 0 || k0 != k1) &&
                  kv4_last(p.counters + 2 * first + (sub == 0), min(FOLD, c1 - first + 1));
  }
  __syncthreads();
#pragma unroll 1
  for (int i = 0; i < 2; ++i) {
    if (!s_last[i]) continue;
    const Group u = s_group[i == 0 ? k0 : k1];
    const int c0 = u.w0 / WARPS, c1 = u.w1 / WARPS;
    const int sub = (static_cast<int>(blockIdx.x) - c0) / FOLD, first = c0 + sub * FOLD;
    const bool one = c1 - c0 < FOLD;
    const int subs = (c1 - c0) / FOLD + 1;
#pragma unroll 1
    for (bool top = false;; top = true) {
      kv4_fold<D, NT>(p, u, top ? c0 : first, top ? FOLD : 1,
                      top ? subs : min(FOLD, c1 - first + 1), top || sub == 0, top || one, pieces);
      if (one || top) break;
      // s_last[i] has been read by all: the fold has barriers
      if (tid == 0) s_last[i] = kv4_last(p.counters + 2 * KV4_MAX_CTAS + c0, subs);
      __syncthreads();
      if (!s_last[i]) break;
    }
  }
  if (line.odd) kv4_fill_empty<D, THREADS>(p, &g_status);
}

template <int D, int NT>
cudaError_t launch(Kv4AttnParams p, int num_sms, int max_ctas, cudaStream_t stream) {
  using S = Smem<D, NT>;
  static int configured_dev[64] = {0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!configured_dev[dev]) {
    e = cudaFuncSetAttribute(ra_kv4_decode_kernel<D, NT>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, S::BYTES);
    if (e != cudaSuccess) return e;
    configured_dev[dev] = 1;
  }
  int grid = num_sms;
  if (max_ctas > 0 && max_ctas < grid) grid = max_ctas;
  if (grid > KV4_MAX_CTAS) grid = KV4_MAX_CTAS;
  // no more units, and with the longest requests the table can name cells,
  // than these (aligned units are padded to four times their cells at most)
  const double units = kv4_decode_units(p.T, p.group, p.R, p.Hkv, p.rows_max);
  const double blocks = 4.0 * p.W * p.page / KV4_BLOCK;
  p.cell_shift = 0;
  auto cells = [&] {
    return units * (blocks / (1ll << p.cell_shift) + UNIT_COST + MIN_CELLS * S::WARPS);
  };
  while (cells() >= 2e9) ++p.cell_shift;
  ra_kv4_decode_kernel<D, NT><<<grid, S::THREADS, S::BYTES, stream>>>(p);
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
