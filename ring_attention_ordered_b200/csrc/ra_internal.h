// Internal declarations shared by the kernels and the C ABI layer.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "ring_attn.h"

namespace ra {

// Parameters of one forward launch.  The tensor maps describe q, k and v as
// 3-D arrays {d, H, B*L} of bf16 (d fastest) with a box of {64, 1, 128}:
// 64 head-dim columns (one 128-byte swizzle row) of 128 consecutive rows of
// one head.
struct FwdParams {
  CUtensorMap tm_q;
  CUtensorMap tm_k;
  CUtensorMap tm_v;
  __nv_bfloat16* out;  // bf16 output; may be NULL in a per-visit launch
  float* lse;
  // Per-visit launch (o_acc != NULL): the whole launch is one ring visit of a
  // query block against one K/V block (n_ring == 1, causal == diagonal
  // visit); its fp32 result goes to o_acc [B, L, Hq, d] and lse, folded into
  // what they hold when visit_fold == 1, and out (if not NULL) receives the
  // bf16 rounding of the folded result.
  float* o_acc;
  int visit_fold;
  int diag_shift;      // 1: the diagonal visit excludes the key at the query's own row
  int B, Hq, Hkv, group;
  int L, blk_len, n_ring, causal;
  int tiles_per_blk;   // ceil(blk_len / 128)
  int pair_heads;      // 1: a unit is two heads of one GQA group on the same rows
  int head_slots;      // ceil(group / 2), when pair_heads
  int pairs_per_blk;   // ceil(tiles_per_blk / 2), when !pair_heads
  int total_units;     // < 2^31, checked by the host
  int head_major;      // unit order: 1 = K/V-head major (L2 reuse), 0 = global longest first
  float scale_log2;    // scale * log2(e)
  unsigned long long wait_limit_ns;
  unsigned debug_flags;
  // Work queue of this launch: a counter (zero at launch) from which each
  // CTA's loader takes the next unit, in the unit order above.
  unsigned int* tickets;
};

// Parameters of one FP8 forward launch (d = 128).  The tensor maps describe
// the E4M3 codes of q, k and v as 3-D byte arrays {128, H, B*L} with a box of
// {128, 1, 128}: one 128-byte swizzle row per head row, 128 consecutive rows
// of one head.  sq [B, Hq, T], sk and sv [B, Hkv, T] hold the float32 scale
// of each 128-row tile (T = L / 128).  The scheduling fields mean what they
// mean in FwdParams.
struct Fp8FwdParams {
  CUtensorMap tm_q;
  CUtensorMap tm_k;
  CUtensorMap tm_v;
  const float* sq;
  const float* sk;
  const float* sv;
  __nv_bfloat16* out;
  float* lse;
  int B, Hq, Hkv, group;
  int L, blk_len, n_ring, causal;
  int tiles_per_blk;
  int pair_heads;
  int head_slots;
  int pairs_per_blk;
  int total_units;
  int head_major;
  int n_tiles;         // T = L / 128
  float scale_log2;    // scale * log2(e), before the per-tile scales
  unsigned long long wait_limit_ns;
  unsigned debug_flags;
  unsigned int* tickets;   // the launch's work queue (see FwdParams)
};

// Parameters of the two backward launches (dQ kernel, then dK/dV kernel).
// tm_q/tm_do view q and dout as {d, Hq, B*L}, tm_k/tm_v view k and v as
// {d, Hkv, B*L}, with the forward's box and swizzle.
struct BwdParams {
  CUtensorMap tm_q;
  CUtensorMap tm_k;
  CUtensorMap tm_v;
  CUtensorMap tm_do;
  const __nv_bfloat16* out;    // forward output O [B, L, Hq, d]
  const __nv_bfloat16* dout;   // upstream gradient dO [B, L, Hq, d]
  const float* lse;            // forward lse [B, Hq, L] (natural log)
  float* dvec;                 // workspace: D = rowsum(dO * O) [B, Hq, L]
  __nv_bfloat16* dq;
  __nv_bfloat16* dk;
  __nv_bfloat16* dv;
  int B, Hq, Hkv, group;
  int L, blk_len, n_ring, causal;
  int tiles_per_blk;
  int units_dq;                // B * Hq * n_ring * tiles_per_blk
  int units_kv;                // B * Hkv * n_ring * tiles_per_blk
  // work-queue counters of the two launches (set by the launcher, see
  // next_ticket_counter)
  unsigned int* tickets_dq;
  unsigned int* tickets_kv;
  float scale;
  float scale_log2;
  unsigned long long wait_limit_ns;
  unsigned debug_flags;
  // Which kernels run: bit 0 the dQ kernel (also writes D), bit 1 the dK/dV
  // kernel (reads D).  ring_attn_bwd runs both.
  int parts;
  // Per-visit launches (ring_attn_bwd_visit): when dq_acc / dk_acc are set,
  // the dQ (dK, dV) rows are written to, or with fold_q (fold_kv) added to,
  // these fp32 accumulators [B, L, H, d]; dq, if set, then receives the bf16
  // rounding of the new dq_acc.  diag_shift = 1 makes the diagonal block
  // exclude the key at the query's own row.
  float* dq_acc;
  float* dk_acc;
  float* dv_acc;
  int fold_q, fold_kv;
  int diag_shift;
};

cudaError_t launch_fwd(const FwdParams& prm, int d, int grid, cudaStream_t stream);
cudaError_t launch_bwd(const BwdParams& prm, int d, int num_sms, int max_ctas,
                       cudaStream_t stream);
cudaError_t read_and_clear_bwd_status(unsigned long long* out);

// Static scratch of ring_attn_bwd_noalloc (fp32 entries, 4 MiB).
constexpr long long kNoAllocScratchRows = 1ll << 20;
// Device address of that scratch in the current context.  Looked up on every
// call made while `stream` is not capturing (the module, and so the address,
// belongs to a context, which cudaDeviceReset or a caller's own context can
// change); during a capture the address cached for the current context is
// used, so a context's first call must come before any capture.
cudaError_t noalloc_scratch(void** ptr, cudaStream_t stream);
// The calling thread's current driver context (nullptr if none).
cudaError_t current_context(CUcontext* ctx);
// Device address of a static __device__ variable of this library in the
// current context.  Looked up on every call made while `stream` is not
// capturing (the module, and so the address, belongs to a context, which
// cudaDeviceReset or a caller's own context can change); during a capture
// the address last found for the current context is used.
cudaError_t symbol_address(const void* symbol, void** ptr, cudaStream_t stream);
cudaError_t read_and_clear_status(unsigned long long* out);
// A zeroed work-queue counter for the next launch on `stream` (forward, FP8
// forward, each backward kernel): one of kTicketSlots static device
// counters, taken in rotation and reset by a memset ordered on the stream
// (so launches on different streams use different counters, up to
// kTicketSlots at a time).
constexpr int kTicketSlots = 64;
cudaError_t next_ticket_counter(cudaStream_t stream, unsigned int** counter);

cudaError_t launch_fwd_fp8(const Fp8FwdParams& prm, int grid, cudaStream_t stream);
cudaError_t read_and_clear_fp8_status(unsigned long long* out);
// Block quantisation of x bf16 [B, L, H, d] to E4M3 codes and per-tile scales.
cudaError_t launch_quantize_fp8(const __nv_bfloat16* x, uint8_t* codes, float* scales, int B,
                                long long L, int H, int d, cudaStream_t stream);

// ---- the paged 4-bit K/V cache (layout and format: ra_kv4.cuh)
constexpr int KV4_PLAN_MAX_R = 8192;   // requests of a plan: its sums lie in shared memory
struct Kv4PlanParams {
  const int32_t* lens;    // [R] tokens held by each request
  const int32_t* add;     // [R] tokens to add, -1: the request is done
  const int32_t* table;   // [R, W]
  const int32_t* pool;    // [num_pages + 1] stack of free pages, its size first
  int32_t* lens_out;
  int32_t* table_out;
  int32_t* pool_out;
  int32_t* cu;            // [R + 1]
  int32_t* slots;         // [max_tokens]
  int32_t* shortage;      // [1]
  int R, W, num_pages, page;
  long long max_tokens;
};
// Append (k, v -> cache) and read (cache -> k_out, v_out) of the tokens at `slots`.
struct Kv4CopyParams {
  const void* k;          // [T, Hkv, d], tokens k_stride elements apart
  const void* v;
  long long k_stride, v_stride;
  void* k_out;            // [T, Hkv, d]
  void* v_out;
  const int32_t* slots;   // [T], -1: none
  uint8_t* cache;
  long long T, num_slots; // num_slots = num_pages * page
  int Hkv, page;
};
// Attention of the query tokens of R requests over their cached tokens.
struct Kv4AttnParams {
  const void* q;          // [T, Hq, d], tokens q_stride elements apart
  long long q_stride;
  void* out;              // [T, Hq, d] of q's type, or fp32
  float* lse;             // [T, Hq]
  const uint8_t* cache;
  const int32_t* table;   // [R, W]
  const int32_t* lens;    // [R]
  const int32_t* cu;      // [R + 1], or NULL: one query token a request
  int T, R, Hq, Hkv, group, W, page, num_pages, causal;
  int q_f16, out_f32;
  float scale_log2;       // scale * log2(e)
  // requests with more rows (query tokens * group) than rows_max are not
  // the decoding kernel's, those with rows_min or fewer not the chunk kernel's;
  // rows_min 0: every request is the chunk kernel's
  int rows_min, rows_max;
  int cell_shift;         // decoding: see Kv4Line
  unsigned* counters;     // workspace: zero before and after the launch
  float* partials;        // workspace
  unsigned long long wait_limit_ns;
};
// No more units (a K/V head and a tile of 8 rows of a request) than this come
// to the decoding kernel, which counts their cells in 32 bits: KV4_MAX_UNITS.
inline double kv4_decode_units(int T, int group, int R, int Hkv, int rows_max) {
  const double tiles = static_cast<double>(T) * group / 8 + R;
  const double most = static_cast<double>(R) * (rows_max / 8 + 1);
  return (tiles < most ? tiles : most) * Hkv;
}
constexpr double KV4_MAX_UNITS = 16777216.0;
cudaError_t launch_kv4_plan(const Kv4PlanParams& p, cudaStream_t stream);
cudaError_t launch_kv4_append(const Kv4CopyParams& p, int d, int dtype, cudaStream_t stream);
cudaError_t launch_kv4_read(const Kv4CopyParams& p, int d, int dtype, cudaStream_t stream);
cudaError_t read_and_clear_kv4_cache_status(unsigned long long* out);
cudaError_t launch_kv4_decode(const Kv4AttnParams& p, int d, int rows, int num_sms, int max_ctas,
                              cudaStream_t stream);
cudaError_t read_and_clear_kv4_decode_status(unsigned long long* out);
cudaError_t launch_kv4_chunk(const Kv4AttnParams& p, int d, int num_sms, int max_ctas,
                             cudaStream_t stream);
cudaError_t read_and_clear_kv4_chunk_status(unsigned long long* out);
// Workspace of kv4 attention: the counters of the decoding kernel, those of
// the chunk kernel (three a CTA each), then partial results of the pieces into
// which a launch cuts the work (two a CTA; the two kernels, one after the
// other on the stream, use the same room).  A unit's pieces are folded at two
// levels of KV4_FOLD at most, in room for KV4_FOLD pieces, so a launch has no
// more CTAs than KV4_FOLD squared.
constexpr int KV4_FOLD = 16;
constexpr int KV4_MAX_CTAS = 256, KV4C_MAX_CTAS = 160;
static_assert(KV4_MAX_CTAS <= KV4_FOLD * KV4_FOLD && KV4C_MAX_CTAS <= KV4_FOLD * KV4_FOLD,
              "two levels of folds");
constexpr int KV4_PIECE_FLOATS = 16 * (128 + 2), KV4C_PIECE_FLOATS = 256 * (128 + 2);
constexpr size_t KV4_COUNTER_BYTES = 3 * KV4_MAX_CTAS * 4;
constexpr size_t KV4C_COUNTER_BYTES = 3 * KV4C_MAX_CTAS * 4;
constexpr size_t KV4_PARTIAL_BYTES = 2ull * KV4C_MAX_CTAS * KV4C_PIECE_FLOATS * 4;
static_assert(KV4_PARTIAL_BYTES >= 2ull * KV4_MAX_CTAS * KV4_PIECE_FLOATS * 4, "partials");
// The partials lie behind all that the caller is told to find zero.
static_assert(KV4_COUNTER_BYTES + KV4C_COUNTER_BYTES <= RA_KV4_COUNTER_BYTES, "counters");
static_assert(RA_KV4_COUNTER_BYTES % 16 == 0, "partials are 16-byte aligned");
constexpr size_t KV4_WORKSPACE_BYTES = RA_KV4_COUNTER_BYTES + KV4_PARTIAL_BYTES;

cudaError_t launch_round_bf16(const float* src, __nv_bfloat16* dst, long long n, int num_sms,
                              cudaStream_t stream);

cudaError_t launch_merge(const float* o_a, const float* lse_a, const float* o_b,
                         const float* lse_b, float* o_out, float* lse_out, long long rows, int d,
                         int num_sms, cudaStream_t stream);

}  // namespace ra
