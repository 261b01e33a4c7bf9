// Attention of many query rows over the paged 4-bit K/V cache (sm_100a): a
// prompt's next chunk, or drafted tokens of several heads.  The arithmetic of
// ra_kv4_decode.cu on the tcgen05 tensor cores.
//
// * The rows of a request and K/V head are its query tokens times the group's
//   query heads, packed token-major; a unit is 256 of them (two tiles of 128)
//   over the tokens they see.  One CTA per SM; the roles and the order of the
//   MMAs are the bf16 forward's (ra_fwd_roles.cuh).
// * Warps 0-3 and 4-7 own a row tile each, one row a thread: they bring the
//   row's q into shared memory (fp16, scaled by a power of two, exact), read S
//   from tensor memory, form s = ks C + kz sum(q) in fp32 (C = q . codes; the steps
//   and zeros lie in shared memory), keep the running maximum and sum, and
//   write P in fp16 over S.
// * Warp 8 copies the blocks' K and V parts into a ring of raw stages; warps
//   12-15 turn them into fp16 operand tiles (128-byte swizzle): the codes of K
//   as they are, as subnormal fp16 numbers (one AND a pair), so S has no
//   rounding beyond fp32; the values of V, step * code + zero rounded to fp16
//   (half a step 2^-12 of the value, next to an output of at most that
//   precision).  Unpacking costs each tile of 128 tokens about 230 operations
//   a thread of the four warps, once for 256 rows.
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
// the line is found by one division.
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
constexpr int UNIT_COST = 2;  // what a unit costs beside its tiles, in tiles
constexpr int MIN_TILES = 8;  // tiles below which a stretch is not cut further
constexpr int FOLD = 16;      // pieces that one CTA folds at a time
constexpr float P_SHIFT = 5.f;         // p = 2^P_SHIFT at the reference
constexpr float P_LIMIT_LOG2 = 15.f;   // beyond which the reference moves

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
  static constexpr int NUM_BARS = fwd_num_bars(NS) + 2 * NRAW + NPAR + 2;
  static constexpr int OFF_MISC = OFF_BAR + NUM_BARS * 8;
  static constexpr int OFF_UNITS = OFF_MISC + 16;
  static constexpr int SMEM_BYTES = OFF_UNITS + UQ * 4 + 1024;   // + alignment slack
  static_assert(SMEM_BYTES <= 232448 - 1024, "shared memory budget");
  static_assert(UNIT_ROWS * (D + 2) <= KV4C_PIECE_FLOATS, "workspace piece");
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
  uint32_t raw_full0, raw_empty0, par_full0, unit_done, rows;
  __device__ __forceinline__ uint32_t raw_full(int s) const { return raw_full0 + 8u * s; }
  __device__ __forceinline__ uint32_t raw_empty(int s) const { return raw_empty0 + 8u * s; }
  __device__ __forceinline__ uint32_t par_full(int s) const { return par_full0 + 8u * s; }
  __device__ __forceinline__ void place(uint32_t bar0, uint32_t units_addr) {
    layout(bar0, NS, units_addr);
    raw_full0 = bar0 + 8u * fwd_num_bars(NS);
    raw_empty0 = raw_full0 + 8u * NRAW;
    par_full0 = raw_empty0 + 8u * NRAW;
    unit_done = par_full0 + 8u * NPAR;
    rows = unit_done + 8u;
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
    mbar_init(unit_done, 256);
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
__device__ __forceinline__ int tile_limit(const Kv4AttnParams& p, const Kv4Req& q, int rows, int i) {
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
__device__ __forceinline__ void find_start(const Kv4AttnParams& p, long long* s_scan, Start* s_start,
                                           int* s_odd) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int each = (p.R + THREADS - 1) / THREADS;
  auto cells = [&](const Req& q) { return static_cast<long long>(q.pairs) * p.Hkv * q.room; };
  long long mine = 0;
  bool odd = false;
  for (int i = 0; i < each; ++i) {
    const int r = tid * each + i;
    if (r >= p.R) break;
    const Req q = request(p, r);
    mine += cells(q);
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
  const long long per =
      max((total + gridDim.x - 1) / gridDim.x, static_cast<long long>(MIN_TILES));
  const long long at = per * blockIdx.x;
  if (tid == 0) {
    *s_odd = any;
    s_start->total = total;
    s_start->per = per;
  }
  if (at >= lo && at < lo + mine)
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
      if (k >= UQ - 1 &&
          !wait_warp(br.unit_done, (k - (UQ - 1)) & 1u, cx, SITE_DONE)) goto drain;
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
        asm volatile("st.shared.s32 [%0], %1;" ::"r"(br.units + 4u * (k % UQ)), "r"(k % UQ) : "memory");
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
  if (k >= UQ - 1 && !wait_warp(br.unit_done, (k - (UQ - 1)) & 1u, cx, SITE_DONE)) goto drain;
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
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
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
          // K: 16 bytes are 32 codes of one token, four swizzle chunks
          constexpr int CPR = D / 32;                    // 16-byte chunks of a row
#pragma unroll 1
          for (int c = 0; c < CPR; ++c) {
            const int id = i + 128 * c, key = id / CPR, q = id % CPR;
            uint32_t x[4];
            lds128(x, raw + (key >> 4) * C::PART + (key & 15) * (D / 2) + q * 16);
            const uint32_t row = dst + (q >> 1) * BOX_BYTES + key * 128;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              // odd boxes in another order: the eight lanes of a phase then
              // store to eight different chunks
              const int ww = w ^ ((q >> 1) << 1);
              const uint32_t a = ww == 0 ? x[0] : ww == 1 ? x[1] : ww == 2 ? x[2] : x[3];
              const uint32_t b = a >> 8;
              const int chunk = ((q & 1) * 4 + ww) ^ (key & 7);
              sts128(row + chunk * 16, a & 0x000f000fu, a & 0x00f000f0u, b & 0x000f000fu,
                     b & 0x00f000f0u);
            }
          }
          // steps and zeros of the tile's tokens
          const uint32_t w =
              lds32(raw + (i >> 4) * C::PART + KV4_BLOCK * (D / 2) + (i & 15) * 4);
          const float2 sz = ((have >> (i >> 4)) & 1u) ? kv4_params(w) : make_float2(0.f, 0.f);
          const uint32_t par = base + C::OFF_PAR + (tile % NPAR) * TILE_KEYS * 8 + i * 4;
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(par), "f"(sz.x) : "memory");
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(par + TILE_KEYS * 4), "f"(sz.y) : "memory");
          if (i == 0) held[NRAW + tile % NPAR] = have;
          mbar_arrive(br.par_full(tile % NPAR));
        } else {
          // V: D / 8 bytes of a lane are D / 8 values of two tokens
          constexpr int WPL = D / 32;                    // words of a lane
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            const int id = i + 128 * c;                  // [block][half][lane]
            const int blk = id >> 6, half = (id >> 5) & 1, ln = id & 31;
            const int g = ln >> 2, tt = ln & 3;
            const int ka = blk * 16 + half * 8 + 2 * tt;   // tokens ka, ka + 1
            const uint32_t part = raw + blk * C::PART;
            uint32_t x[WPL];
            const uint32_t src = part + half * (4 * D) + ln * (4 * WPL);
            if constexpr (WPL == 4) {
              lds128(x, src);
            } else {
              asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(x[0]), "=r"(x[1]) : "r"(src));
            }
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
            for (int cc = 0; cc < WPL / 2; ++cc) {
              const int c2 = WPL == 4 ? (cc ^ (g & 1)) : cc;
              const int chunk = ((e & 63) >> 3) + c2;
              const uint32_t* pa = ra;
              const uint32_t* pb = rb;
              uint32_t a4[4], b4[4];
#pragma unroll
              for (int z = 0; z < 4; ++z) {
                a4[z] = (WPL == 4 && c2 == 1) ? pa[(4 + z) % (2 * WPL)] : pa[z];
                b4[z] = (WPL == 4 && c2 == 1) ? pb[(4 + z) % (2 * WPL)] : pb[z];
              }
              sts128(row + ((chunk ^ (ka & 7)) * 16), a4[0], a4[1], a4[2], a4[3]);
              sts128(row + 128 + ((chunk ^ ((ka + 1) & 7)) * 16), b4[0], b4[1], b4[2], b4[3]);
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
// Scores of 32 columns before the factor rho: C in sr becomes ks C + kz sigma,
// the steps and zeros from shared memory at `par`.
__device__ __forceinline__ void scores32(uint32_t (&sr)[32], uint32_t par, uint64_t sigma2) {
#pragma unroll
  for (int j = 0; j < 32; j += 4) {
    uint32_t ks[4], kz[4];
    lds128(ks, par + 4 * j);
    lds128(kz, par + TILE_KEYS * 4 + 4 * j);
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
      const uint64_t b =
          f2_mul(f2_pack(__uint_as_float(kz[e]), __uint_as_float(kz[e + 1])), sigma2);
      float a0, a1;
      f2_unpack(f2_fma(f2_pack(__uint_as_float(sr[j + e]), __uint_as_float(sr[j + e + 1])),
                       f2_pack(__uint_as_float(ks[e]), __uint_as_float(ks[e + 1])), b),
                a0, a1);
      sr[j + e] = __float_as_uint(a0);
      sr[j + e + 1] = __float_as_uint(a1);
    }
  }
}

// P = 2^(u rho + nm) of one row as fp16 pairs in pk, its row sum, and the
// largest exponent in `top` (NaN if one is).  MASKED: the columns behind `lim`
// and the blocks that are not in `have` are 0; and the product is rounded
// before the sum, as the reference was formed, which very large scores need.
template <bool MASKED>
__device__ __forceinline__ float weights(uint32_t (&pk)[64], uint32_t tS, uint32_t par,
                                         uint64_t sigma2, float rho, float nm, int lim,
                                         uint32_t have, float& top) {
  const uint64_t rho2 = f2_pack(rho, rho), nm2 = f2_pack(nm, nm);
  uint64_t acc[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
  float mx[2] = {-INFINITY, -INFINITY};
  // two halves of 64 columns in one copy of the code: the tile's loop has to
  // fit the instruction cache beside the unpacking and MMA loops
#pragma unroll 1
  for (int half = 0; half < 2; ++half) {
    uint32_t sr[2][32];
    tmem_ld32(tS + 64 * half, sr[0]);
    if (half == 1) {
#pragma unroll
      for (int j = 0; j < 32; ++j) pk[j] = pk[32 + j];
    }
    const int left = lim - 64 * half;
    const uint32_t on = have >> (4 * half);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      tmem_wait_ld();
      if (c < 1) tmem_ld32(tS + 64 * half + 32, sr[1]);
      uint32_t(&x)[32] = sr[c];
      scores32(x, par + 256 * half + 128 * c, sigma2);
#pragma unroll
      for (int j = 0; j < 32; j += 2) {
        const int col = 32 * c + j;
        const uint64_t s2 = f2_pack(__uint_as_float(x[j]), __uint_as_float(x[j + 1]));
        float p0, p1;
        f2_unpack(MASKED ? f2_add(f2_mul(s2, rho2), nm2) : f2_fma(s2, rho2, nm2), p0, p1);
        if (MASKED) {
          const bool in = (on >> (col >> 4)) & 1u;
          if (col > left || !in) p0 = -INFINITY;
          if (col + 1 > left || !in) p1 = -INFINITY;
        }
        mx[(j >> 1) & 1] = fmax3(mx[(j >> 1) & 1], p0, p1);
        p0 = ex2_approx(p0);
        p1 = ex2_approx(p1);
        acc[(j >> 1) & 1] = f2_add(acc[(j >> 1) & 1], f2_pack(p0, p1));
        pk[32 + 16 * c + (j >> 1)] = pack_f16x2(p0, p1);
      }
    }
  }
  float a, b;
  f2_unpack(f2_add(acc[0], acc[1]), a, b);
  top = fmaxf(mx[0], mx[1]);
  return a + b;
}

// The largest score of a row before the factor rho, -inf if it sees none.
__device__ __forceinline__ float row_max(uint32_t tS, uint32_t par, uint64_t sigma2, int lim,
                                         uint32_t have) {
  float m = -INFINITY;
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    uint32_t x[32];
    tmem_ld32(tS + 32 * c, x);
    tmem_wait_ld();
    scores32(x, par + 128 * c, sigma2);
    const int n = lim - 32 * c;
    const uint32_t on = have >> (2 * c);
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (j <= n && ((on >> (j >> 4)) & 1u)) m = fmaxf(m, __uint_as_float(x[j]));
  }
  return m;
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
// the softmax threads, a row to D / 4 lanes; each thread has 8 rows of two
// pieces in flight.  Returns the barrier's phase, or -1 if the kernel is
// aborting.  A function of its own, with the piece in shared memory, so that
// the loop over the tiles keeps its registers.
template <int D>
__device__ __noinline__ int fold(const Kv4AttnParams& p, const Piece* piece, int c0, int step,
                                 int n, bool starts, bool finish, RowSync sync, Ctl cx) {
  constexpr int LPR = D / 4, RPR = 256 / LPR, V = 8;   // rows a round, rows a thread
  const Piece x = *piece;
  const int rows = min(UNIT_ROWS, x.rows - x.row0);
  const int d = 4 * (threadIdx.x % LPR);
#pragma unroll 1
  for (int rb = 0; rb < rows; rb += RPR * V) {
    const int r0 = rb + threadIdx.x / LPR;
    float m[V], ls[V];
    float4 a[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      m[v] = -INFINITY;
      ls[v] = 0.f;
      a[v] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll 1
    for (int c = 0; c < n; ++c) {
      const float* src =
          p.partials + (2ll * (c0 + c * step) + (starts && c == 0)) * KV4C_PIECE_FLOATS;
      float mm[V], ll[V];
      float4 aa[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int row = r0 + v * RPR;
        mm[v] = -INFINITY;
        if (row < rows) {
          mm[v] = __ldcg(src + UNIT_ROWS * D + row);
          ll[v] = __ldcg(src + UNIT_ROWS * D + UNIT_ROWS + row);
          aa[v] = __ldcg(reinterpret_cast<const float4*>(src + row * D + d));
        }
      }
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (mm[v] != -INFINITY) kv4_merge(m[v], ls[v], a[v], mm[v], ll[v], aa[v]);
    }
    if (!finish && !sync(cx)) return -1;   // the round's rows have been read
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int row = r0 + v * RPR;
      if (row >= rows) continue;
      if (finish) {
        kv4_store(p, x.first, x.h, x.row0 + row, d, D, a[v], m[v] - P_SHIFT, ls[v]);
      } else {
        float* dst = p.partials + (2ll * c0 + starts) * KV4C_PIECE_FLOATS;
        *reinterpret_cast<float4*>(dst + row * D + d) = a[v];
        if (d == 0) {
          dst[UNIT_ROWS * D + row] = m[v];
          dst[UNIT_ROWS * D + UNIT_ROWS + row] = ls[v];
        }
      }
    }
  }
  return static_cast<int>(sync.phase);
}

// Counts the CTA in at `counter`: 1 if it is the last of `n` (the counter is
// then zero again), 0 if not, -1 if the kernel is aborting.
__device__ __forceinline__ int count_in(unsigned* counter, int n, volatile int* s_last,
                                        RowSync& sync, const Ctl& cx) {
  __threadfence();
  if (!sync(cx)) return -1;
  if (threadIdx.x == 0) {
    const unsigned old = atomicAdd(counter, 1u);
    *s_last = old == static_cast<unsigned>(n - 1);
    if (*s_last) *counter = 0u;
    __threadfence();
  }
  if (!sync(cx)) return -1;
  return *s_last;
}

template <int D>
__device__ void softmax_role(const Kv4AttnParams& p, const Bars& br, uint32_t base, uint32_t tmem,
                             int w, Piece* pieces, volatile uint32_t* held, volatile int* s_last,
                             const Ctl& cx) {
  using C = Cfg<D>;
  const int t = threadIdx.x - w * 128;            // row inside the tile
  const int quarter = (threadIdx.x >> 5) & 3;
  const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
  const uint32_t tS = tmem + lane_off + w * 128;
  const uint32_t tO = tmem + lane_off + 256 + w * 128;
  uint32_t s_phase = 0u, units_w = 0u, q_uses = 0u, tile = 0u;
  RowSync sync{br.rows, 0u};

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
    const int sees = kv4_limit(p, q, row, rows);       // tokens that the row sees
    float rho = 0.f;
    uint64_t sigma2 = 0;
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
      float up, down;
      kv4_row_scale(am, up, down);
      rho = p.scale_log2 * down * 16777216.f;
      const float sg = sum * up * 5.9604644775390625e-8f;
      sigma2 = f2_pack(sg, sg);
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

    float m = -INFINITY, l = 0.f;
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
      const int lim = min(sees - (t0 + idx) * TILE_KEYS, TILE_KEYS) - 1;
      const bool masked = __any_sync(0xffffffffu, lim < TILE_KEYS - 1) || have != 0xffu;
      const uint32_t par = base + C::OFF_PAR + slot * TILE_KEYS * 8;

      // P with the reference in hand; where that would pass fp16's range (or is
      // none yet), the reference first moves to the row's maximum
      uint32_t pk[64];
      float rsum = 0.f;
      bool slow = masked || far;
#pragma unroll 1
      for (int round = 0; round < 2; ++round) {
        float top;
        rsum = slow ? weights<true>(pk, tS, par, sigma2, rho, P_SHIFT - m, lim, have, top)
                    : weights<false>(pk, tS, par, sigma2, rho, P_SHIFT - m, lim, have, top);
        if (round == 1 || !__any_sync(0xffffffffu, top > P_LIMIT_LOG2)) break;
        const float rmax = row_max(tS, par, sigma2, lim, have);
        const float m_new = rmax == -INFINITY ? m : fmaxf(m, __fmul_rn(rmax, rho));
        const float alpha = m_new == m ? 1.f : ex2_approx(m - m_new);
        if (idx > 0) {
          // O already holds every earlier P V of this tile: the commit that
          // signalled S for this step fires only after them
#pragma unroll 1
          for (int cc = 0; cc < D / 32; ++cc) {
            uint32_t o[32];
            tmem_ld32(tO + cc * 32, o);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
            tmem_st32(tO + cc * 32, o);
          }
          tmem_wait_st();
        }
        l *= alpha;
        m = m_new;
        far = __any_sync(0xffffffffu, fabsf(m) > 4096.f && m != -INFINITY);
        slow = masked || far;
      }
      l += rsum;
      tmem_st32(tS, *reinterpret_cast<uint32_t(*)[32]>(&pk[0]));
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(br.p_half(w));
      tmem_st32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&pk[32]));
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(br.p_full(w));
    }

    // ---- the piece's rows: finished, or a partial in the workspace
    if (mine) {
      ok = wait_bar(br.o_done(w), units_w & 1u, cx, SITE_O_DONE);
      if (!__all_sync(0xffffffffu, ok)) return;
      tc_fence_after();
      const bool bad = *reinterpret_cast<volatile int*>(&pieces[u].nan_at) < sees;
      const bool whole = pieces[u].whole, row_ok = row < pieces[u].rows;
      const int h = pieces[u].h, lrow = w * TILE_ROWS + t;
      q.first = pieces[u].first;
      float* slot = p.partials + (2ll * blockIdx.x + (static_cast<int>(blockIdx.x) == pieces[u].c0)) *
                                     KV4C_PIECE_FLOATS;
#pragma unroll 1
      for (int cc = 0; cc < D / 32; ++cc) {
        uint32_t o[32];
        tmem_ld32(tO + cc * 32, o);
        tmem_wait_ld();
        if (row_ok) {
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            float4 a = make_float4(__uint_as_float(o[j]), __uint_as_float(o[j + 1]),
                                   __uint_as_float(o[j + 2]), __uint_as_float(o[j + 3]));
            if (bad) a.x = a.y = a.z = a.w = __uint_as_float(0x7fffffffu);
            if (whole)
              kv4_store(p, q.first, h, row, cc * 32 + j, D, a, m - P_SHIFT, l);
            else
              *reinterpret_cast<float4*>(slot + lrow * D + cc * 32 + j) = a;
          }
        }
      }
      if (row_ok && !whole) {
        slot[UNIT_ROWS * D + lrow] = m;
        slot[UNIT_ROWS * D + UNIT_ROWS + lrow] = l;
      }
      tc_fence_before();
      mbar_arrive(br.o_free(w));
      ++units_w;
    }
    if (!pieces[u].whole) {
      const int c0 = pieces[u].c0, c1 = pieces[u].c1;
      const int sub = (static_cast<int>(blockIdx.x) - c0) / FOLD, first = c0 + sub * FOLD;
      const int n = min(FOLD, c1 - first + 1);
      const bool starts = sub == 0, one = c1 - c0 < FOLD;
      int last = count_in(p.counters + 2 * first + starts, n, s_last, sync, cx);
      if (last > 0) {
        int ph = fold<D>(p, pieces + u, first, 1, n, starts, one, sync, cx);
        if (ph < 0) return;
        sync.phase = ph;
        if (!one) {
          const int subs = (c1 - c0) / FOLD + 1;
          last = count_in(p.counters + 2 * KV4C_MAX_CTAS + c0, subs, s_last, sync, cx);
          if (last > 0) ph = fold<D>(p, pieces + u, c0, FOLD, subs, true, true, sync, cx);
          if (ph < 0) return;
          sync.phase = last > 0 ? ph : sync.phase;
        }
      }
      if (last < 0) return;
    }
    mbar_arrive(br.unit_done);
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
  __shared__ int s_odd, s_last;
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

  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(SOFTMAX_REGS));
    softmax_role<D>(p, br, base, tmem, warp >> 2, pieces, held, &s_last, cx);
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
  if (s_odd && p.rows_min == 0) kv4_fill_empty<D, THREADS>(p, &g_status);
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
