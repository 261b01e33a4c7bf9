// Attention of many query rows over the paged 4-bit K/V cache (sm_100a): a
// prompt's next chunk, or drafted tokens of several heads.  The arithmetic of
// ra_kv4_decode.cu on the tcgen05 tensor cores.
//
// * The rows of a request and K/V head are its query tokens times the group's
//   query heads, packed token-major; a unit is 256 of them (two tiles of 128)
//   over the tokens they see.  One CTA per SM; the roles and the order of the
//   MMAs are the bf16 forward's (ra_fwd_roles.cuh).
// * Warps 0-3 and 4-7 own a row tile each: they bring their rows' q into
//   shared memory (fp16, scaled by a power of two: see Rows), read S from tensor
//   memory, form s = ks C + kz sum(q) in fp32 (C = q . codes; the steps
//   and zeros lie in shared memory), keep the reference and the running sum, and
//   write P in fp16 over S.
// * Warp 8 copies the blocks' K and V parts into a ring of raw stages; warps
//   12-15 turn them into fp16 operand tiles (128-byte swizzle): the codes of K
//   as subnormal fp16 numbers, code 2^-22 and code 2^-18 (one AND a pair and a shift
//   for two), the values of V, step * code + zero rounded to fp16
//   (half a step, 2^-11 of the value at most, next to an output of that
//   precision at most).  One unpacking serves 256 rows.
//   The products of subnormal numbers lose places where an instruction aligns them,
//   which shows in lse of rows that see few tokens, the first of a prompt: relative
//   error for fp16 q 1.1e-6 with the nibbles where they lie (2^-24 and 2^-20, half a
//   shift less, 552 us below), 2.2e-7 so (560 us), 1.8e-7 as normal numbers by a fused
//   multiply-add a pair (577 us); 1.1e-7 in plain 32-bit arithmetic.
// * P = 2^(s - m + 5) in fp16.  m is a maximum of the row that is moved, and O
//   rescaled, only when P would pass 2^15: so a tile takes one pass over S, no
//   separate search for its maximum, and what lies up to 2^29 below the
//   reference still counts, as it has to in a long cache with a few dominant
//   tokens.
// * A token whose V is NaN would reach, through 0 * NaN, the rows of the tile
//   that do not see it: its V is taken as 0 and its position kept, and the
//   rows that see it become NaN at the end.
//
// Split: the tiles of all units form one line that the CTAs share equally, as in
// ra_kv4_decode.cu.  Under the causal mask a request's row tiles see from few
// to many tokens; they are laid out in pairs, the one with most tokens beside
// the one with fewest, so that every pair takes the same room and a place on
// the line is found by one division.  Units that cross CTAs: the last of their
// CTAs folds the pieces, in their order.
//
// What bounds it, measured: two chunks of 1024 tokens over 16K, 32 query and 8
// K/V heads, d = 128: 556 us, 914 TFLOP/s, 0.56 of cuBLAS's burst rate (at 1.95 GHz;
// 581 us where the power limit holds the clock at 1.88).  A tile's
// softmax (2480 clocks) and the P V and Q K^T that wait for it (1430) alternate for
// each of the two row tiles; neither the tensor pipe nor the MUFU is half busy.
// P V started on the first half of P, with S read half a tile at a time, lost more
// in the softmax than it took off the wait (582 us, and 242 us against 270 us for
// a prompt of 4096 tokens, whose units are short); the same with both halves unrolled
// outgrew the instruction cache (828 us).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "ptx_sm100.cuh"
#include "ra_fwd_roles.cuh"
#include "ra_internal.h"
#include "ra_kv4.cuh"
#include "ra_kv4_attn.cuh"
#include "ra_mma16.cuh"
#include "ra_sync.cuh"

namespace ra {
namespace kv4c {

constexpr int THREADS = 512;
constexpr int TILE_ROWS = 128, UNIT_ROWS = 256, TILE_KEYS = 128;
constexpr int WARP_LOAD = 8, WARP_MMA = 9, WARP_UNPACK = 12;
// Register split (setmaxnreg) of the launch's 512 x 128.
constexpr int LAUNCH_REGS = 128;
constexpr int SOFTMAX_REGS = 200, CONTROL_REGS = 48, UNPACK_REGS = 64;
static_assert(256 * SOFTMAX_REGS + 128 * CONTROL_REGS + 128 * UNPACK_REGS <= THREADS * LAUNCH_REGS,
              "register split exceeds the launch allocation");
constexpr int NS = 4;         // operand stages (K or V tile)
constexpr int NRAW = 3;       // raw stages (the K or V part of 8 blocks)
constexpr int NPAR = 4;       // slots of a tile's steps and zeros
// Pieces that the loader has under way, the one in hand among them (prompts as one
// call, 32 query and 8 K/V heads, d = 128: 64 of 200 tokens 289 us with 1, 274 with 2,
// 286 with 3, 298 with 4; 128 of 60 tokens 146, 134, 134, 134 us; longer ones alike).
constexpr int AHEAD = 2;
static_assert(AHEAD < UQ, "a place of the queue is free when the piece AHEAD before is done");
constexpr int UNIT_COST = 2;  // what a unit costs beside its tiles, in tiles
constexpr int MIN_TILES = 8;  // tiles below which a stretch is not cut further
constexpr int FOLD = KV4_FOLD;   // pieces that one CTA folds at a time
constexpr float P_SHIFT = 5.f;         // p = 2^P_SHIFT at the reference
constexpr float P_LIMIT = 32768.f;     // beyond which the reference moves
constexpr float Q_SCALE = 256.f;       // of q in fp16, see Rows

__device__ unsigned long long g_status = 0ull;

enum Site : uint32_t { SITE_RAW_FULL = 32, SITE_RAW_EMPTY, SITE_PAR, SITE_DONE, SITE_ROWS };

// One piece of work of the CTA: tiles [t0, t1) of a unit.
struct Piece {
  int n_kv, valid1;            // t1 - t0; whether the second row tile has rows
  int r, h, row0, t0;
  int first, n, len, rows;     // of the request
  int c0, c1, whole;           // CTAs that hold the unit; whether this is all of it
  int nan_at;                  // first visible token whose V is NaN
};

// What the shared MMA role asks of a piece.
struct PieceView {
  const volatile Piece* pieces;
};
__device__ __forceinline__ Unit decode_unit(const PieceView& p, int u) {
  Unit x;
  x.n_kv = p.pieces[u].n_kv;
  x.valid1 = p.pieces[u].valid1;
  return x;
}

template <int D>
struct Cfg {
  static constexpr int Q_BYTES = TILE_ROWS * D * 2;
  static constexpr int KV_BYTES = TILE_KEYS * D * 2;
  static constexpr int PART = KV4_BLOCK * (D / 2) + KV4_BLOCK * 4;   // K or V part of a block
  static constexpr int RAW_BYTES = 8 * PART;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_KV = 2 * Q_BYTES;
  static constexpr int OFF_RAW = OFF_KV + NS * KV_BYTES;
  static constexpr int OFF_PAR = OFF_RAW + NRAW * RAW_BYTES;
  static constexpr int OFF_BAR = OFF_PAR + NPAR * TILE_KEYS * 8;
  static constexpr int NUM_BARS = fwd_num_bars(NS) + 2 * NRAW + NPAR + UQ + 1;
  static constexpr int OFF_MISC = OFF_BAR + NUM_BARS * 8;
  static constexpr int OFF_UNITS = OFF_MISC + 16;
  static constexpr int SMEM_BYTES = OFF_UNITS + UQ * 4 + 1024;   // + alignment slack
  static_assert(SMEM_BYTES <= 232448 - 1024, "shared memory budget");
  static_assert(UNIT_ROWS * (D + 2) <= KV4C_PIECE_FLOATS, "workspace piece");
  static_assert(FOLD * UNIT_ROWS * 4 <= 2 * Q_BYTES, "the factors of a fold fit q's place");
};

template <int D>
struct Geom {
  using C = Cfg<D>;
  static constexpr int Q_BYTES = C::Q_BYTES;
  static constexpr int KV_BYTES = C::KV_BYTES;
  static constexpr int NS = kv4c::NS;
  static constexpr uint32_t IDESC_QK = idesc_f16_f32(TILE_ROWS, TILE_KEYS, false);
  static constexpr uint32_t IDESC_PV = idesc_f16_f32(TILE_ROWS, D, true);
  uint32_t q_lo, k_lo, v_lo, k_hi, v_hi;
  __device__ explicit Geom(uint32_t smem_base) {
    const uint64_t dq = smem_desc_sw128(smem_base + C::OFF_Q, 16, 1024);
    const uint64_t dk = smem_desc_sw128(smem_base + C::OFF_KV, 16, 1024);
    const uint64_t dv = smem_desc_sw128(smem_base + C::OFF_KV, BOX_BYTES, 1024);
    q_lo = static_cast<uint32_t>(dq);
    k_lo = static_cast<uint32_t>(dk);
    v_lo = static_cast<uint32_t>(dv);
    k_hi = static_cast<uint32_t>(dk >> 32);
    v_hi = static_cast<uint32_t>(dv >> 32);
  }
  __device__ __forceinline__ void issue_qk(uint32_t d, int w, int stage) const {
    mma_qk_steps<D>(d, q_lo + ((w * Q_BYTES) >> 4), k_lo + ((stage * KV_BYTES) >> 4), k_hi,
                    IDESC_QK);
  }
  template <int HALF>
  __device__ __forceinline__ void issue_pv_half(uint32_t d, uint32_t p_tmem, int stage,
                                                uint32_t acc) const {
    mma_pv_half<HALF>(d, p_tmem, v_lo + ((stage * KV_BYTES) >> 4), v_hi, IDESC_PV, acc);
  }
};

struct Bars : FwdBars {
  uint32_t raw_full0, raw_empty0, par_full0, unit_done0, rows;
  __device__ __forceinline__ uint32_t raw_full(int s) const { return raw_full0 + 8u * s; }
  __device__ __forceinline__ uint32_t raw_empty(int s) const { return raw_empty0 + 8u * s; }
  __device__ __forceinline__ uint32_t par_full(int s) const { return par_full0 + 8u * s; }
  // Piece k is done: one barrier a place of the queue, so that the phase waited for is
  // the place's latest or the one before.  With one for all, a wait for a piece two
  // back blocked until the one in hand was done, and the softmax group that skips a
  // second row tile without rows arrived in the other's phase.
  __device__ __forceinline__ uint32_t unit_done(int k) const { return unit_done0 + 8u * (k % UQ); }
  __device__ __forceinline__ void place(uint32_t bar0, uint32_t units_addr) {
    layout(bar0, NS, units_addr);
    raw_full0 = bar0 + 8u * fwd_num_bars(NS);
    raw_empty0 = raw_full0 + 8u * NRAW;
    par_full0 = raw_empty0 + 8u * NRAW;
    unit_done0 = par_full0 + 8u * NPAR;
    rows = unit_done0 + 8u * UQ;
  }
  __device__ __forceinline__ void start() const {
    mbar_init(q_full, 256);
    mbar_init(q_empty, 1);
    for (int s = 0; s < NS; ++s) {
      mbar_init(kv_full(s), 128);
      mbar_init(kv_empty(s), 1);
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(s_full(w), 1);
      mbar_init(p_full(w), 128);
      mbar_init(o_done(w), 1);
      mbar_init(o_free(w), 128);
      mbar_init(p_half(w), 128);
    }
    mbar_init(drain, 1);
    for (int i = 0; i < UQ; ++i) mbar_init(unit_full0 + 8u * i, 1);
    for (int s = 0; s < NRAW; ++s) {
      mbar_init(raw_full(s), 1);
      mbar_init(raw_empty(s), 128);
    }
    for (int s = 0; s < NPAR; ++s) mbar_init(par_full(s), 128);
    for (int i = 0; i < UQ; ++i) mbar_init(unit_done0 + 8u * i, 256);
    mbar_init(rows, 256);
  }
};

// ------------------------------------------------------------------ the line
// Row tiles (of 256 rows) of request r and head h come in pairs: pair i is
// tile T - 1 - i and tile i, T tiles in all (the middle one alone if T is
// odd).  `room` cells hold any pair: its tiles of 128 tokens (one at least, also
// for rows that see no token) and UNIT_COST for each of the two.
struct Req : Kv4Req {
  int rows, tiles, pairs, room;
};
// Tokens that some row of row tile i sees.
__device__ __forceinline__ int tile_limit(const Kv4AttnParams& p, const Kv4Req& q, int rows,
                                          int i) {
  const int last = min((i + 1) * UNIT_ROWS, rows) - 1;
  return max(kv4_limit(p, q, last, rows), 0);
}
__device__ __forceinline__ int key_tiles(int tokens) {
  return max((tokens + TILE_KEYS - 1) / TILE_KEYS, 1);
}

__device__ __forceinline__ Req request(const Kv4AttnParams& p, int r) {
  Req q;
  static_cast<Kv4Req&>(q) = kv4_request(p, r);
  q.rows = q.n * p.group;
  if (q.len == 0 || q.rows <= p.rows_min) q.rows = 0;   // not this kernel's
  q.tiles = (q.rows + UNIT_ROWS - 1) / UNIT_ROWS;
  q.pairs = (q.tiles + 1) / 2;
  // Up to the rounding of rows to tokens and a short last tile (256 tokens at
  // most) no pair sees more tokens than the outermost; either count of key
  // tiles exceeds its tokens by less than a tile.
  q.room = 0;
  if (q.tiles > 0)
    q.room = key_tiles(tile_limit(p, q, q.rows, 0)) +
             key_tiles(tile_limit(p, q, q.rows, q.tiles - 1)) + 4 + 2 * UNIT_COST;
  return q;
}

struct Start {
  long long total, per;
  int r;
  long long in;      // cells of request r before the CTA's stretch
};

// Every thread of the CTA takes part.
__device__ __forceinline__ void find_start(const Kv4AttnParams& p, long long* s_scan,
                                           Start* s_start, int* s_odd) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int each = (p.R + THREADS - 1) / THREADS;
  auto cells = [&](const Req& q) { return static_cast<long long>(q.pairs) * p.Hkv * q.room; };
  long long mine = 0;
  bool odd = false, falls = false;
  for (int i = 0; i < each; ++i) {
    const int r = tid * each + i;
    if (r >= p.R) break;
    const Req q = request(p, r);
    mine += cells(q);
    falls |= q.falls;
    odd |= q.bad || q.len == 0;
  }
  long long inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) s_scan[warp] = inc;
  const int any = __syncthreads_or(odd);
  long long lo = inc - mine, total = 0;
#pragma unroll 1
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) lo += s_scan[w];
    total += s_scan[w];
  }
  // cu that falls: nothing is done
  if (any && __syncthreads_or(falls)) total = 0;
  const long long per =
      max((total + gridDim.x - 1) / gridDim.x, static_cast<long long>(MIN_TILES));
  const long long at = per * blockIdx.x;
  if (tid == 0) {
    *s_odd = any;
    s_start->total = total;
    s_start->per = per;
  }
  if (at < total && at >= lo && at < lo + mine)
    for (int i = 0; i < each; ++i) {
      const long long c = cells(request(p, tid * each + i));
      if (at < lo + c) {
        s_start->r = tid * each + i;
        s_start->in = at - lo;
        break;
      }
      lo += c;
    }
  __syncthreads();
}

// ------------------------------------------------------------------ loader
// Finds the CTA's pieces, publishes them and copies their blocks.
template <int D>
__device__ void loader_role(const Kv4AttnParams& p, const Bars& br, uint32_t base, const Start& st,
                            Piece* pieces, volatile uint32_t* held, const Ctl& cx) {
  using C = Cfg<D>;
  const int lane = threadIdx.x & 31;
  uint32_t it = 0;         // raw stages filled
  uint32_t tiles_done = 0; // tiles of tokens handed out
  int k = 0;
  auto place_for = [&](int k) {
    return k < AHEAD ||
           wait_warp(br.unit_done(k - AHEAD), ((k - AHEAD) / UQ) & 1u, cx, SITE_DONE);
  };
  long long at = st.per * blockIdx.x;
  const long long end = min(at + st.per, st.total);
  int r = 0;
  long long in = 0;
  if (at < end) {
    r = st.r;
    in = st.in;
  }
  while (at < end && r < p.R) {
    const Req q = request(p, r);
    const long long all = static_cast<long long>(q.pairs) * p.Hkv * q.room;
    if (in >= all) {
      ++r;
      in = 0;
      continue;
    }
    const int pair_no = static_cast<int>(in / q.room);
    const int off = static_cast<int>(in - static_cast<long long>(pair_no) * q.room);
    const long long pair0 = at - off;
    const int cells = static_cast<int>(min(end - at, static_cast<long long>(q.room - off)));
    at += cells;
    in += cells;
    const int h = pair_no / q.pairs, pi = pair_no - h * q.pairs;
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
      // the unit's tiles are the cells [first, first + nt) of the pair
      const int big = q.tiles - 1 - pi;
      if (half == 1 && big == pi) break;
      const int rt = half == 0 ? big : pi;
      const int nt = key_tiles(tile_limit(p, q, q.rows, rt));
      const int first = half == 0 ? UNIT_COST
                                  : 2 * UNIT_COST + key_tiles(tile_limit(p, q, q.rows, big));
      const int row0 = rt * UNIT_ROWS;
      const int t0 = max(off - first, 0), t1 = min(off + cells - first, nt);
      if (t1 <= t0) continue;
      if (!place_for(k)) goto drain;
      if (lane == 0) {
        Piece x;
        x.n_kv = t1 - t0;
        x.valid1 = row0 + TILE_ROWS < q.rows;
        x.r = r;
        x.h = h;
        x.row0 = row0;
        x.t0 = t0;
        x.first = q.first;
        x.n = q.n;
        x.len = q.len;
        x.rows = q.rows;
        x.c0 = static_cast<int>((pair0 + first) / st.per);
        x.c1 = static_cast<int>((pair0 + first + nt - 1) / st.per);
        x.whole = t1 - t0 == nt;
        x.nan_at = 0x7fffffff;
        pieces[k % UQ] = x;
        asm volatile("st.shared.s32 [%0], %1;" ::"r"(br.units + 4u * (k % UQ)), "r"(k % UQ)
                     : "memory");
        mbar_arrive(br.unit_full(k));
      }
      __syncwarp();
      ++k;
      // lane i < 8: block i of a tile, looked up one tile ahead
      const int nb = (q.len + KV4_BLOCK - 1) / KV4_BLOCK;
      auto lookup = [&](int t) {
        const int blk = t * 8 + lane;
        return lane < 8 && t < t1 && blk < nb ? kv4_block_index(p, r, h, blk, &g_status) : -1;
      };
      int next = lookup(t0);
      for (int t = t0; t < t1; ++t, ++tiles_done) {
        const int e = next;
        const uint32_t have = __ballot_sync(0xffffffffu, e >= 0);
        next = lookup(t + 1);
#pragma unroll 1
        for (int v = 0; v < 2; ++v, ++it) {
          const int s = it % NRAW;
          if (it >= NRAW &&
              !wait_warp(br.raw_empty(s), (it / NRAW - 1) & 1u, cx, SITE_RAW_EMPTY)) goto drain;
          if (lane == 0) {
            held[s] = have;
            mbar_arrive_expect_tx(br.raw_full(s), __popc(have) * C::PART);
          }
          __syncwarp();
          if (e >= 0)
            bulk_load(base + C::OFF_RAW + s * C::RAW_BYTES + lane * C::PART,
                      p.cache + static_cast<long long>(e) * Kv4<D>::BLOCK_BYTES + v * C::PART,
                      C::PART, br.raw_full(s));
          __syncwarp();
        }
      }
    }
  }
  if (!place_for(k)) goto drain;
  if (lane == 0) {
    asm volatile("st.shared.s32 [%0], %1;" ::"r"(br.units + 4u * (k % UQ)), "r"(-1) : "memory");
    mbar_arrive(br.unit_full(k));
  }
  __syncwarp();
  return;
drain:
  // let the copies already issued land before the CTA's shared memory goes
  if (lane == 0)
    for (uint32_t i = it > NRAW ? it - NRAW : 0; i < it; ++i)
      drain_wait(br.raw_full(i % NRAW), (i / NRAW) & 1u, 200000000ull);
  __syncwarp();
}

// ------------------------------------------------------------------ unpack
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                       uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}
__device__ __forceinline__ void lds128(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t r;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(addr));
  return r;
}
// fma.rn.f16x2
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

template <int D>
__device__ void unpack_role(const Kv4AttnParams& p, const Bars& br, uint32_t base, Piece* pieces,
                            volatile uint32_t* held, const Ctl& cx) {
  using C = Cfg<D>;
  const int i = threadIdx.x - WARP_UNPACK * 32;   // 0..127
  uint32_t it = 0, tile = 0;
  for (int k = 0;; ++k) {
    int u;
    const bool got = next_unit(br, k, cx, u);
    if (!__all_sync(0xffffffffu, got)) return;
    if (u < 0) break;
    const int n = pieces[u].n_kv, t0 = pieces[u].t0, len = pieces[u].len;
    for (int t = 0; t < n; ++t, ++tile) {
#pragma unroll 1
      for (int v = 0; v < 2; ++v, ++it) {
        const int rs = it % NRAW, s = it % NS;
        bool ok = wait_bar(br.raw_full(rs), (it / NRAW) & 1u, cx, SITE_RAW_FULL);
        if (!__all_sync(0xffffffffu, ok)) return;
        ok = it < NS || wait_bar(br.kv_empty(s), (it / NS - 1) & 1u, cx, SITE_KV_EMPTY);
        if (!__all_sync(0xffffffffu, ok)) return;
        const uint32_t raw = base + C::OFF_RAW + rs * C::RAW_BYTES;
        const uint32_t dst = base + C::OFF_KV + s * C::KV_BYTES;
        const uint32_t have = held[rs];
        const int room = len - (t0 + t) * TILE_KEYS;   // tokens of the tile
        if (v == 0) {
          // K: 16 bytes are 32 codes of one token, four swizzle chunks; the
          // eight lanes of a phase take eight tokens, whose chunks then lie in
          // eight places.  Nibbles (0, 4), (1, 5), (2, 6), (3, 7) of a word are pairs
          // of code 2^-22, 2^-18, 2^-22, 2^-18
          constexpr int CPR = D / 32;                    // 16-byte parts of a row
#pragma unroll 1
          for (int q = 0; q < CPR; ++q) {
            uint32_t x[4];
            lds128(x, raw + (i >> 4) * C::PART + (i & 15) * (D / 2) + q * 16);
            const uint32_t row = dst + (q >> 1) * BOX_BYTES + i * 128;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const uint32_t y = x[w] << 2, z = x[w] >> 6;
              sts128(row + (((q & 1) * 4 + w) ^ (i & 7)) * 16, y & 0x003c003cu,
                     y & 0x03c003c0u, z & 0x003c003cu, z & 0x03c003c0u);
            }
          }
          // step and zero of token i: pairs of tokens as (step, step, zero, zero)
          const uint32_t w =
              lds32(raw + (i >> 4) * C::PART + KV4_BLOCK * (D / 2) + (i & 15) * 4);
          const float2 sz = ((have >> (i >> 4)) & 1u) ? kv4_params(w) : make_float2(0.f, 0.f);
          const uint32_t par =
              base + C::OFF_PAR + (tile % NPAR) * TILE_KEYS * 8 + (i >> 1) * 16 + (i & 1) * 4;
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(par),
                       "f"(sz.x * (p.scale_log2 * (4194304.f / Q_SCALE))) : "memory");
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(par + 8), "f"(sz.y * p.scale_log2)
                       : "memory");
          if (i == 0) held[NRAW + tile % NPAR] = have;
          mbar_arrive(br.par_full(tile % NPAR));
        } else {
          // V: thread i has two tokens, ka and ka + 1, and every second group
          // of D / 8 elements; their codes lie side by side in the block
          constexpr int WPL = D / 32;                    // words of a group
          const int kp = i & 63, blk = kp >> 3;
          const int ka = 2 * kp;
          const uint32_t part = raw + blk * C::PART;
          uint32_t wa = lds32(part + KV4_BLOCK * (D / 2) + (ka & 15) * 4);
          uint32_t wb = lds32(part + KV4_BLOCK * (D / 2) + (ka & 15) * 4 + 4);
          const bool in = (have >> blk) & 1u;
          // tokens that are not there: zeros, whatever the stage holds
          if (!in || ka >= room) wa = 0u;
          if (!in || ka + 1 >= room) wb = 0u;
          if ((wa & 0x7fffu) > 0x7c00u) {
            atomicMin(&pieces[u].nan_at, (t0 + t) * TILE_KEYS + ka);
            wa = 0u;
          }
          if ((wb & 0x7fffu) > 0x7c00u) {
            atomicMin(&pieces[u].nan_at, (t0 + t) * TILE_KEYS + ka + 1);
            wb = 0u;
          }
          const uint32_t step = __byte_perm(wa, wb, 0x5410), zero = __byte_perm(wa, wb, 0x7632);
#pragma unroll 1
          for (int g = i >> 6; g < 8; g += 2) {
            uint32_t x[WPL];
            const uint32_t src = part + ((kp >> 2) & 1) * (4 * D) + (g * 4 + (kp & 3)) * (4 * WPL);
            if constexpr (WPL == 4) {
              lds128(x, src);
            } else {
              asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(x[0]), "=r"(x[1]) : "r"(src));
            }
            uint32_t ra[2 * WPL], rb[2 * WPL];   // pairs of elements of either token
#pragma unroll
            for (int w = 0; w < WPL; ++w) {
              const uint32_t y = x[w] >> 8;
              // 1024 + code and 1024 + 16 code, exact
              const uint32_t h0 = (x[w] & 0x000f000fu) | 0x64006400u;
              const uint32_t h1 = (x[w] & 0x00f000f0u) | 0x64006400u;
              const uint32_t h2 = (y & 0x000f000fu) | 0x64006400u;
              const uint32_t h3 = (y & 0x00f000f0u) | 0x64006400u;
              const uint32_t one = 0x3c003c00u, m1024 = 0xe400e400u;
              const uint32_t sixteenth = 0x2c002c00u, m64 = 0xd400d400u;
              const uint32_t e0 = hfma2(hfma2(h0, one, m1024), step, zero);
              const uint32_t e1 = hfma2(hfma2(h1, sixteenth, m64), step, zero);
              const uint32_t e2 = hfma2(hfma2(h2, one, m1024), step, zero);
              const uint32_t e3 = hfma2(hfma2(h3, sixteenth, m64), step, zero);
              ra[2 * w] = __byte_perm(e0, e1, 0x5410);
              ra[2 * w + 1] = __byte_perm(e2, e3, 0x5410);
              rb[2 * w] = __byte_perm(e0, e1, 0x7632);
              rb[2 * w + 1] = __byte_perm(e2, e3, 0x7632);
            }
            // D / 8 values: one or two 16-byte chunks of each token's row
            const int e = g * (D / 8);
            const uint32_t row = dst + (e >> 6) * BOX_BYTES + ka * 128;
#pragma unroll
            for (int c = 0; c < WPL / 2; ++c) {
              const int chunk = ((e & 63) >> 3) + c;
              sts128(row + ((chunk ^ (ka & 7)) * 16), ra[4 * c], ra[4 * c + 1], ra[4 * c + 2],
                     ra[4 * c + 3]);
              sts128(row + 128 + ((chunk ^ ((ka + 1) & 7)) * 16), rb[4 * c], rb[4 * c + 1],
                     rb[4 * c + 2], rb[4 * c + 3]);
            }
          }
        }
        fence_proxy_async();
        mbar_arrive(br.kv_full(s));
        mbar_arrive(br.raw_empty(rs));
      }
    }
  }
}

// ------------------------------------------------------------------ softmax
// A softmax warp holds its 32 rows as the fragments of four m16n8 products
// (tmem_ld_16x256_x8): thread (g, t) has the rows g, g + 8, g + 16, g + 24 and of
// every 8 columns 2t and 2t + 1.  So the steps and zeros of two tokens, which
// every row needs, are one 16-byte read for four rows instead of one for
// each (LDS was the kernel's busiest pipe with a row to a thread), and the row
// sums are joined over the four lanes of a row once, at the end of a piece.
//
// Scores in log2 units are s = C ks' + kz' sigma with ks' = ks scale log2(e)
// 2^22 / Q_SCALE and kz' = kz scale log2(e), which the unpacking warps
// prepare; q is scaled by Q_SCALE for every row (and divided by 16 where it meets
// the larger codes), so the exponent s - m + 5 is two fused multiply-adds.  A row
// whose magnitudes that scale would take out of fp16's range has a scale of its own,
// and its C a factor `f`.  Scaled so, q is exact in fp16 but for elements that are
// small in a row of small ones: with the largest at 2^-14, the least the common scale
// is used for, they are off by 2^-15 of it, and scores by 2^-29 |k|.
struct Rows {
  uint64_t sigma2[4];   // sum of q, twice
  float f[4];
  int sees[4];          // tokens that the row sees
};

// P = 2^(s - m + P_SHIFT) of 64 of the rows' columns as fp16 pairs in pk, added to acc.
// SLOW: with the rows' factors; the columns behind a row's last token and the
// blocks that are not in `on` are 0; and s is rounded before the sum, as the
// reference was formed, which very large scores need.
template <bool SLOW>
__device__ __forceinline__ void weights64(uint32_t (&pk)[2][16], uint64_t (&acc)[4], uint32_t tS,
                                          uint32_t par, const Rows& r, const uint64_t (&nm2)[4],
                                          int key0, uint32_t on) {
  const int t = threadIdx.x & 3;
  uint32_t x[2][32];
  tmem_ld_16x256_x8(tS, x[0]);
  tmem_ld_16x256_x8(tS + (16u << 16), x[1]);
  tmem_wait_ld();
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    uint32_t k[4];
    lds128(k, par + 64 * j + 16 * t);
    const uint64_t ks = f2_pack(__uint_as_float(k[0]), __uint_as_float(k[1]));
    const uint64_t kz = f2_pack(__uint_as_float(k[2]), __uint_as_float(k[3]));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t* c = x[i >> 1] + 4 * j + 2 * (i & 1);
      uint64_t c2 = f2_pack(__uint_as_float(c[0]), __uint_as_float(c[1]));
      float p0, p1;
      if (SLOW) {
        c2 = f2_mul(c2, f2_pack(r.f[i], r.f[i]));
        f2_unpack(f2_add(f2_fma(c2, ks, f2_mul(kz, r.sigma2[i])), nm2[i]), p0, p1);
        const int left = r.sees[i] - key0 - 2 * t;   // columns 8j, 8j + 1 below it
        const bool in = (on >> (j >> 1)) & 1u;
        if (8 * j >= left || !in) p0 = -INFINITY;
        if (8 * j + 1 >= left || !in) p1 = -INFINITY;
      } else {
        f2_unpack(f2_fma(c2, ks, f2_fma(kz, r.sigma2[i], nm2[i])), p0, p1);
      }
      p0 = ex2_approx(p0);
      p1 = ex2_approx(p1);
      acc[i] = f2_add(acc[i], f2_pack(p0, p1));
      pk[i >> 1][2 * j + (i & 1)] = pack_f16x2(p0, p1);
    }
  }
}

// The two halves of a tile; the rows' sums in `sum`.  The reference has to move
// if a sum passes P_LIMIT, which bounds its terms.
template <bool SLOW>
__device__ __forceinline__ void weights(uint32_t (&pk)[2][2][16], uint32_t tS, uint32_t par,
                                        const Rows& r, const float (&m)[4], int key0,
                                        uint32_t have, float (&sum)[4]) {
  uint64_t acc[4], nm2[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    acc[i] = f2_pack(0.f, 0.f);
    nm2[i] = f2_pack(P_SHIFT - m[i], P_SHIFT - m[i]);
  }
  if (SLOW) {
    // one copy of the code, which is seldom run
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        pk[0][0][j] = pk[1][0][j];
        pk[0][1][j] = pk[1][1][j];
      }
      weights64<true>(pk[1], acc, tS + 64 * half, par + 512 * half, r, nm2, key0 + 64 * half,
                      have >> (4 * half));
    }
  } else {
    weights64<false>(pk[0], acc, tS, par, r, nm2, key0, have);
    weights64<false>(pk[1], acc, tS + 64, par + 512, r, nm2, key0 + 64, have >> 4);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    f2_unpack(acc[i], a, b);
    sum[i] = a + b;
  }
}

// The largest scores of the rows, -inf for a row that sees no token.
__device__ __forceinline__ void row_max(float (&m)[4], uint32_t tS, uint32_t par, const Rows& r,
                                        int key0, uint32_t have) {
  const int t = threadIdx.x & 3;
#pragma unroll
  for (int i = 0; i < 4; ++i) m[i] = -INFINITY;
#pragma unroll 1
  for (int half = 0; half < 2; ++half) {
    uint32_t x[2][32];
    tmem_ld_16x256_x8(tS + 64 * half, x[0]);
    tmem_ld_16x256_x8(tS + (16u << 16) + 64 * half, x[1]);
    tmem_wait_ld();
    const uint32_t on = have >> (4 * half);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      uint32_t k[4];
      lds128(k, par + 512 * half + 64 * j + 16 * t);
      const uint64_t ks = f2_pack(__uint_as_float(k[0]), __uint_as_float(k[1]));
      const uint64_t kz = f2_pack(__uint_as_float(k[2]), __uint_as_float(k[3]));
      const bool in = (on >> (j >> 1)) & 1u;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t* c = x[i >> 1] + 4 * j + 2 * (i & 1);
        const uint64_t c2 = f2_mul(f2_pack(__uint_as_float(c[0]), __uint_as_float(c[1])),
                                   f2_pack(r.f[i], r.f[i]));
        float s0, s1;
        f2_unpack(f2_fma(c2, ks, f2_mul(kz, r.sigma2[i])), s0, s1);
        const int left = r.sees[i] - key0 - 64 * half - 2 * t;
        if (in && 8 * j < left) m[i] = fmaxf(m[i], s0);
        if (in && 8 * j + 1 < left) m[i] = fmaxf(m[i], s1);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = fmaxf(m[i], __shfl_xor_sync(0xffffffffu, m[i], 1));
    m[i] = fmaxf(m[i], __shfl_xor_sync(0xffffffffu, m[i], 2));
  }
}

// Barrier of the 256 softmax threads, bounded as every wait; false if the
// kernel is aborting.
struct RowSync {
  uint32_t bar, phase;
  __device__ __forceinline__ bool operator()(const Ctl& cx) {
    mbar_arrive(bar);
    const bool ok = wait_bar(bar, phase, cx, SITE_ROWS);
    phase ^= 1u;
    return __all_sync(0xffffffffu, ok);
  }
};

// Pieces of a unit in the workspace, of the CTAs c0 + i step, i < n, folded in
// that order: stored as the result, or as the piece of the first of them.  By
// the softmax threads: first a thread for each row, which finds the factors of
// the row's pieces, in `tab` (shared memory, [piece][row]); then a row to D / 4
// lanes, each thread with 8 rows in flight.  False if the kernel is aborting.
template <int D>
__device__ __forceinline__ bool fold(const Kv4AttnParams& p, const Piece& x, int c0, int step,
                                     int n, bool starts, bool finish, float* tab, RowSync& sync,
                                     const Ctl& cx) {
  constexpr int LPR = D / 4, RPR = 256 / LPR, V = 8;   // rows a round, rows a thread
  // pieces in flight (d = 128, before K's codes: 549 us with 1, 553 with 2, two chunks
  // of 1024 over 16K;
  // d = 64: 93 us and 88 us, 8 chunks of 200 over 3K)
  constexpr int E = D == 128 ? 1 : 2;
  const int rows = min(UNIT_ROWS, x.rows - x.row0);
  const float* first = p.partials + (2ll * c0 + starts) * KV4C_PIECE_FLOATS;
  auto piece_at = [&](int c) {
    return c == 0 ? first : p.partials + 2ll * (c0 + c * step) * KV4C_PIECE_FLOATS;
  };
  auto row_at = [&](int row) {     // of the row's first element in out
    const int tok = (x.row0 + row) / p.group;
    return (static_cast<long long>(x.first) + tok) * p.Hq + x.h * p.group +
           (x.row0 + row - tok * p.group);
  };
  const int mine = threadIdx.x;
  if (mine < rows) {
    float m = -INFINITY, l = 0.f;
#pragma unroll 4
    for (int c = 0; c < n; ++c) {
      const float mc = __ldcg(piece_at(c) + UNIT_ROWS * D + mine);
      tab[c * UNIT_ROWS + mine] = mc;
      m = fmaxf(m, mc);
    }
#pragma unroll 4
    for (int c = 0; c < n; ++c) {
      // a piece whose row saw nothing has m = -inf and zeros
      const float mc = tab[c * UNIT_ROWS + mine], f = mc == m ? 1.f : ex2_approx(mc - m);
      tab[c * UNIT_ROWS + mine] = f;
      l = fmaf(__ldcg(piece_at(c) + UNIT_ROWS * D + UNIT_ROWS + mine), f, l);
    }
    if (finish) {
      const float inv = l == 0.f ? 0.f : 1.f / l;
      for (int c = 0; c < n; ++c) tab[c * UNIT_ROWS + mine] *= inv;
      p.lse[row_at(mine)] =
          l == 0.f ? -INFINITY : (m - P_SHIFT + log2f(l)) * 0.69314718055994530942f;
    } else {
      float* dst = p.partials + (2ll * c0 + starts) * KV4C_PIECE_FLOATS + UNIT_ROWS * D + mine;
      dst[0] = m;
      dst[UNIT_ROWS] = l;
    }
  }
  if (!sync(cx)) return false;
  const int d = 4 * (threadIdx.x % LPR);
#pragma unroll 1
  for (int rb = 0; rb < rows; rb += RPR * V) {
    const int r0 = rb + threadIdx.x / LPR;
    float4 a[V];
#pragma unroll
    for (int v = 0; v < V; ++v) a[v] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int c = 0; c < n; c += E) {
      float4 b[E][V];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float* src = piece_at(min(c + e, n - 1)) + r0 * D + d;
#pragma unroll
        for (int v = 0; v < V; ++v)
          if (r0 + v * RPR < rows)
            b[e][v] = __ldcg(reinterpret_cast<const float4*>(src + v * RPR * D));
      }
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if (c + e >= n) break;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          if (r0 + v * RPR >= rows) continue;
          const float f = tab[(c + e) * UNIT_ROWS + r0 + v * RPR];
          a[v].x = fmaf(b[e][v].x, f, a[v].x);
          a[v].y = fmaf(b[e][v].y, f, a[v].y);
          a[v].z = fmaf(b[e][v].z, f, a[v].z);
          a[v].w = fmaf(b[e][v].w, f, a[v].w);
        }
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int row = r0 + v * RPR;
      if (row >= rows) continue;
      if (!finish) {
        // this thread alone reads and writes these elements
        *reinterpret_cast<float4*>(const_cast<float*>(first) + row * D + d) = a[v];
        continue;
      }
      const long long o = row_at(row) * D + d;
      if (p.out_f32)
        *reinterpret_cast<float4*>(static_cast<float*>(p.out) + o) = a[v];
      else if (p.q_f16)
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + o) =
            make_uint2(pack_f16x2(a[v].x, a[v].y), pack_f16x2(a[v].z, a[v].w));
      else
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + o) =
            make_uint2(pack_bf16x2(a[v].x, a[v].y), pack_bf16x2(a[v].z, a[v].w));
    }
  }
  return sync(cx);   // the table has been read
}

// Counts the CTA, all of whose softmax threads have passed a barrier since they
// wrote, in at `counter`; true if it is the last of `n`, which sets the counter
// back to zero.  By one thread.
__device__ __forceinline__ bool count_in(unsigned* counter, int n) {
  __threadfence();
  const bool last = atomicAdd(counter, 1u) == static_cast<unsigned>(n - 1);
  if (last) {
    __threadfence();
    *counter = 0u;
  }
  return last;
}

template <int D>
__device__ void softmax_role(const Kv4AttnParams& p, const Bars& br, uint32_t base, uint32_t tmem,
                             int w, Piece* pieces, volatile uint32_t* held, Piece* cut,
                             volatile int* s_last, const Ctl& cx) {
  using C = Cfg<D>;
  const int t = threadIdx.x - w * 128;            // row inside the tile
  const int quarter = (threadIdx.x >> 5) & 3;
  const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
  const uint32_t tS = tmem + lane_off + w * 128;
  const uint32_t tO = tmem + lane_off + 256 + w * 128;
  uint32_t s_phase = 0u, units_w = 0u, q_uses = 0u, tile = 0u;
  RowSync sync{br.rows, 0u};
  int n_cut = 0;      // pieces that are not whole units

  for (int k = 0;; ++k) {
    int u;
    bool ok = next_unit(br, k, cx, u);
    if (!__all_sync(0xffffffffu, ok)) return;
    if (u < 0) break;
    const int n_kv = pieces[u].n_kv, t0 = pieces[u].t0;
    const bool mine = w == 0 || pieces[u].valid1;
    Kv4Req q;
    q.first = pieces[u].first;
    q.n = pieces[u].n;
    q.len = pieces[u].len;
    const int rows = pieces[u].rows, row = pieces[u].row0 + w * TILE_ROWS + t;
    Rows r;
    bool odd;               // some row of the warp has a factor
    // ---- q of this row: fp16 in shared memory, in the order of the codes
    {
      uint4 qw[D / 8];
      kv4_load_q<D>(p, q, pieces[u].h, row, rows, 0, D, qw);
      float am = 0.f, sum = 0.f;
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        const uint32_t ww[4] = {qw[c].x, qw[c].y, qw[c].z, qw[c].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = kv4_q_pair(p, ww[e]);
          am = fmaxf(am, fmaxf(fabsf(f.x), fabsf(f.y)));
          sum += f.x + f.y;
        }
      }
      float up = Q_SCALE, f = 1.f;
      if (!(am == 0.f || (am < 255.f && am >= 6.1035156e-5f))) {
        float down;
        kv4_row_scale(am, up, down);
        f = down * Q_SCALE;
      }
      odd = __any_sync(0xffffffffu, f != 1.f);
      const int sees = kv4_limit(p, q, row, rows);
      // to the threads that hold the row's fragments
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int from = 8 * i + ((threadIdx.x & 31) >> 2);
        const float sg = __shfl_sync(0xffffffffu, sum, from);
        r.sigma2[i] = f2_pack(sg, sg);
        r.f[i] = __shfl_sync(0xffffffffu, f, from);
        r.sees[i] = __shfl_sync(0xffffffffu, sees, from);
      }
      if (q_uses > 0) {
        ok = wait_bar(br.q_empty, (q_uses - 1) & 1u, cx, SITE_Q_EMPTY);
        if (!__all_sync(0xffffffffu, ok)) return;
      }
      ++q_uses;
      const uint32_t dst = base + C::OFF_Q + w * C::Q_BYTES + t * 128;
      const float up16 = up * 0.0625f;
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        const float2 f0 = kv4_q_pair(p, qw[c].x), f1 = kv4_q_pair(p, qw[c].y);
        const float2 f2 = kv4_q_pair(p, qw[c].z), f3 = kv4_q_pair(p, qw[c].w);
        // elements (0, 4), (1, 5), (2, 6), (3, 7)
        sts128(dst + (c >> 3) * BOX_BYTES + (((c & 7) ^ (t & 7)) * 16),
               pack_f16x2(f0.x * up, f2.x * up), pack_f16x2(f0.y * up16, f2.y * up16),
               pack_f16x2(f1.x * up, f3.x * up), pack_f16x2(f1.y * up16, f3.y * up16));
      }
      fence_proxy_async();
      mbar_arrive(br.q_full);
    }

    const int sees_min = __reduce_min_sync(
        0xffffffffu, min(min(r.sees[0], r.sees[1]), min(r.sees[2], r.sees[3])));
    float m[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
    }
    bool far = false;       // some row's reference is so large that roundings count
    for (int idx = 0; idx < n_kv; ++idx, ++tile) {
      if (!mine) continue;
      const int slot = tile % NPAR;
      ok = wait_bar(br.par_full(slot), (tile / NPAR) & 1u, cx, SITE_PAR);
      if (!__all_sync(0xffffffffu, ok)) return;
      ok = wait_bar(br.s_full(w), s_phase, cx, SITE_S_FULL);
      if (!__all_sync(0xffffffffu, ok)) return;
      s_phase ^= 1u;
      tc_fence_after();
      const uint32_t have = held[NRAW + slot];
      const int key0 = (t0 + idx) * TILE_KEYS;
      const bool masked = sees_min < key0 + TILE_KEYS || have != 0xffu;
      const uint32_t par = base + C::OFF_PAR + slot * TILE_KEYS * 8;

      // P with the reference in hand; where that would pass fp16's range (or is
      // none yet), the reference first moves to the row's maximum
      uint32_t pk[2][2][16];
      float sum[4];
#pragma unroll 1
      for (int round = 0; round < 2; ++round) {
        if (masked || far || odd)
          weights<true>(pk, tS, par, r, m, key0, have, sum);
        else
          weights<false>(pk, tS, par, r, m, key0, have, sum);
        const float top = fmaxf(fmaxf(sum[0], sum[1]), fmaxf(sum[2], sum[3]));
        if (round == 1 || !__any_sync(0xffffffffu, top > P_LIMIT)) break;
        float rmax[4], alpha[4];
        row_max(rmax, tS, par, r, key0, have);
        bool big = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float m_new = fmaxf(m[i], rmax[i]);
          alpha[i] = m_new == m[i] ? 1.f : ex2_approx(m[i] - m_new);
          l[i] *= alpha[i];
          m[i] = m_new;
          big |= fabsf(m_new) > 4096.f && m_new != -INFINITY;
        }
        far = __any_sync(0xffffffffu, big);
        if (idx > 0) {
          // O already holds every earlier P V of this tile: the commit that
          // signalled S for this step fires only after them
#pragma unroll 1
          for (int cc = 0; cc < D / 64; ++cc) {
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              uint32_t o[32];
              const uint32_t at = tO + (static_cast<uint32_t>(16 * hh) << 16) + cc * 64;
              tmem_ld_16x256_x8(at, o);
              tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 32; ++j)
                o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha[2 * hh + ((j >> 1) & 1)]);
              tmem_st_16x256_x8(at, o);
            }
          }
          tmem_wait_st();
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) l[i] += sum[i];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        tmem_st_16x128_x8(tS + 32 * half, pk[half][0]);
        tmem_st_16x128_x8(tS + (16u << 16) + 32 * half, pk[half][1]);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(half == 0 ? br.p_half(w) : br.p_full(w));
      }
    }

    // ---- the piece's rows: finished, or a partial in the workspace
    if (mine) {
      ok = wait_bar(br.o_done(w), units_w & 1u, cx, SITE_O_DONE);
      if (!__all_sync(0xffffffffu, ok)) return;
      tc_fence_after();
      const int lane = threadIdx.x & 31, g = lane >> 2, tt = lane & 3;
      const int nan_at = *reinterpret_cast<volatile int*>(&pieces[u].nan_at);
      const bool whole = pieces[u].whole;
      const int n_rows = pieces[u].rows, h = pieces[u].h, row0 = pieces[u].row0;
      const bool starts = static_cast<int>(blockIdx.x) == pieces[u].c0;
      float* part = p.partials + (2ll * blockIdx.x + starts) * KV4C_PIECE_FLOATS;
      long long at[4];                 // of the row's first element in out
      float inv[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
        const int lrow = w * TILE_ROWS + quarter * 32 + 8 * i + g;
        const int tok = (row0 + lrow) / p.group;
        at[i] = row0 + lrow >= n_rows ? -1
                : whole ? (static_cast<long long>(pieces[u].first) + tok) * p.Hq + h * p.group +
                              (row0 + lrow - tok * p.group)
                        : lrow;
        // a row that saw no token has l = 0 and O = 0
        inv[i] = !whole ? 1.f : l[i] == 0.f ? 0.f : 1.f / l[i];
        if (nan_at < r.sees[i]) inv[i] = __uint_as_float(0x7fffffffu);
        if (at[i] >= 0 && tt == 0) {
          if (whole) {
            p.lse[at[i]] = l[i] == 0.f ? -INFINITY
                                       : (m[i] - P_SHIFT + log2f(l[i])) * 0.69314718055994530942f;
          } else {
            part[UNIT_ROWS * D + lrow] = m[i];
            part[UNIT_ROWS * D + UNIT_ROWS + lrow] = l[i];
          }
        }
      }
#pragma unroll 1
      for (int cc = 0; cc < D / 64; ++cc) {
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          uint32_t o[32];
          tmem_ld_16x256_x8(tO + (static_cast<uint32_t>(16 * hh) << 16) + cc * 64, o);
          tmem_wait_ld();
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const int i = 2 * hh + b;
            if (at[i] < 0) continue;
            const long long e = at[i] * D + cc * 64 + 2 * tt;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float y0 = __uint_as_float(o[4 * j + 2 * b]) * inv[i];
              const float y1 = __uint_as_float(o[4 * j + 2 * b + 1]) * inv[i];
              if (!whole)
                *reinterpret_cast<float2*>(part + e + 8 * j) = make_float2(y0, y1);
              else if (p.out_f32)
                *reinterpret_cast<float2*>(static_cast<float*>(p.out) + e + 8 * j) =
                    make_float2(y0, y1);
              else
                *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + e + 8 * j) =
                    p.q_f16 ? pack_f16x2(y0, y1) : pack_bf16x2(y0, y1);
            }
          }
        }
      }
      tc_fence_before();
      mbar_arrive(br.o_free(w));
      ++units_w;
    }
    if (!pieces[u].whole) {
      if (!sync(cx)) return;
      if (threadIdx.x == 0) {
        const int c0 = pieces[u].c0, sub = (static_cast<int>(blockIdx.x) - c0) / FOLD;
        const int first = c0 + sub * FOLD;
        cut[n_cut] = pieces[u];
        s_last[n_cut] = count_in(p.counters + 2 * first + (sub == 0),
                                 min(FOLD, pieces[u].c1 - first + 1));
      }
      ++n_cut;
    }
    mbar_arrive(br.unit_done(k));
  }

  // ---- units that cross CTAs, one from before this CTA and one to behind it: the
  // last of every FOLD of them folds their pieces, the last to do so folds these.
  // They are counted as they are done, so that it is mostly the second that this
  // CTA is the last for, and folded at the end: amid the tiles the fold's registers
  // are theirs (two chunks of 1024 tokens over 16K, before K's codes: 573 us, so 549 us).
  if (n_cut == 0 || !sync(cx)) return;
  extern __shared__ __align__(1024) uint8_t smem_raw[];   // q is no longer needed
  float* tab = reinterpret_cast<float*>(smem_raw + (base + C::OFF_Q - smem_u32(smem_raw)));
#pragma unroll 1
  for (int i = 0; i < n_cut; ++i) {
    if (!s_last[i]) continue;
    const Piece x = cut[i];
    const int sub = (static_cast<int>(blockIdx.x) - x.c0) / FOLD, first = x.c0 + sub * FOLD;
    const int n = min(FOLD, x.c1 - first + 1), subs = (x.c1 - x.c0) / FOLD + 1;
    const bool one = subs == 1;
#pragma unroll 1
    for (bool top = false;; top = true) {
      if (!fold<D>(p, x, top ? x.c0 : first, top ? FOLD : 1, top ? subs : n, top || sub == 0,
                   top || one, tab, sync, cx))
        return;
      if (top || one) break;
      if (threadIdx.x == 0)
        s_last[i] = count_in(p.counters + 2 * KV4C_MAX_CTAS + x.c0, subs);
      if (!sync(cx)) return;
      if (!s_last[i]) break;
    }
  }
}

// ------------------------------------------------------------------ kernel
template <int D>
__global__ void __launch_bounds__(THREADS, 1)
    ra_kv4_chunk_kernel(const __grid_constant__ Kv4AttnParams p) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ Piece pieces[UQ];
  __shared__ uint32_t held_[NRAW + NPAR];   // blocks that a raw stage, a tile's slot holds
  __shared__ Start s_start;
  __shared__ long long s_scan[THREADS / 32];
  __shared__ Piece s_cut[2];
  __shared__ int s_odd, s_last[2];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* base_ptr = smem_raw + (base - raw);
  volatile uint32_t* held = held_;

  Bars br;
  br.place(base + C::OFF_BAR, base + C::OFF_UNITS);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(base_ptr + C::OFF_MISC);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(base_ptr + C::OFF_MISC + 4);
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    br.start();
    *abort_flag = 0u;
    fence_mbarrier_init();
  }
  if (warp == WARP_MMA) {
    tmem_alloc(smem_u32(tmem_holder), 512);
    tmem_relinquish();
  }
  find_start(p, s_scan, &s_start, &s_odd);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const Ctl cx{abort_flag, p.wait_limit_ns, &g_status};

  // A call of its own, so before the roles take their registers: here every
  // thread has the launch's, which cover it; behind, warps hold as few as
  // CONTROL_REGS.
  if (s_odd && p.rows_min == 0) kv4_fill_empty<D, THREADS>(p, &g_status);

  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(SOFTMAX_REGS));
    softmax_role<D>(p, br, base, tmem, warp >> 2, pieces, held, s_cut, s_last, cx);
  } else if (warp < WARP_UNPACK) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(CONTROL_REGS));
    if (warp == WARP_LOAD)
      loader_role<D>(p, br, base, s_start, pieces, held, cx);
    else if (warp == WARP_MMA)
      fwd_mma_role<Geom<D>>(PieceView{pieces}, static_cast<const FwdBars&>(br), base, tmem, cx);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(UNPACK_REGS));
    unpack_role<D>(p, br, base, pieces, held, cx);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == WARP_MMA) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D>
cudaError_t launch(const Kv4AttnParams& p, int num_sms, int max_ctas, cudaStream_t stream) {
  using C = Cfg<D>;
  static int configured_dev[64] = {0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!configured_dev[dev]) {
    // the setmaxnreg split is only safe if the kernel launches with LAUNCH_REGS
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, ra_kv4_chunk_kernel<D>);
    if (e != cudaSuccess) return e;
    if (fa.numRegs != LAUNCH_REGS) return cudaErrorInvalidKernelImage;
    e = cudaFuncSetAttribute(ra_kv4_chunk_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             C::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    configured_dev[dev] = 1;
  }
  int grid = num_sms;
  if (max_ctas > 0 && max_ctas < grid) grid = max_ctas;
  if (grid > KV4C_MAX_CTAS) grid = KV4C_MAX_CTAS;
  ra_kv4_chunk_kernel<D><<<grid, THREADS, C::SMEM_BYTES, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace kv4c

cudaError_t launch_kv4_chunk(const Kv4AttnParams& p, int d, int num_sms, int max_ctas,
                             cudaStream_t stream) {
  return d == 128 ? kv4c::launch<128>(p, num_sms, max_ctas, stream)
                  : kv4c::launch<64>(p, num_sms, max_ctas, stream);
}

cudaError_t read_and_clear_kv4_chunk_status(unsigned long long* out) {
  unsigned long long v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, kv4c::g_status, sizeof(v));
  if (e == cudaSuccess && v != 0) e = cudaMemcpyToSymbol(kv4c::g_status, &zero, sizeof(zero));
  *out = v;
  return e;
}

}  // namespace ra
