// The paged 4-bit K/V cache: layout, element format and device-side checks
// shared by its kernels (plan, append, read, attention).
//
// Layout: uint8 [num_pages, Hkv, page / 16, 16 (d + 8)].  The last axis is
// one block: 16 tokens of one page and head, in four parts,
//     K codes   16 rows of d / 2 bytes (element 2i in the low nibble of
//               byte i, element 2i + 1 in the high one),
//     K params  16 pairs (step, zero) in fp16,
//     V codes   8 d bytes, see v_code_offset,
//     V params  16 pairs (step, zero) in fp16.
// A block is one contiguous copy of 16 (d + 8) bytes whatever the page size,
// so the attention kernels stream blocks and look a page up only to find
// them.  The code orders are those in which a warp's matrix instructions
// take the operands: lane (g, t) (g = lane / 4, t = lane % 4) of the
// decoding kernel finds its part of 8 key rows as 16 consecutive bytes (8
// for d = 64), and so its part of the values of 8 keys, lanes side by side.
// In V the four nibbles of a 16-bit half belong to one token, so that two
// tokens never share a byte and a single token can be written alone.
//
// Format: a vector x of d values of one token and head is held as
//     zero = fp16(min x), step = fp16 of (max x - min x) / 15 rounded
//     towards zero, at least 2^-24, code = the nearest of 0..15 to
//     (x - zero) / step, ties to the even code;
//     value = step * code + zero, in fp32.
// x is clamped to +-65504 first.  Rounding the step down keeps every value
// inside the range of the data (so it stays finite in fp16), and the floor
// keeps a constant vector from dividing by zero.  A vector that holds a NaN
// has NaN parameters and reads as NaN.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "ring_attn.h"

namespace ra {

constexpr int KV4_BLOCK = 16;   // tokens per block

template <int D>
struct Kv4 {
  static constexpr int ROW = D / 2;             // bytes of one token's codes
  static constexpr int CODES = KV4_BLOCK * ROW;
  static constexpr int OFF_KP = CODES;
  static constexpr int OFF_V = CODES + KV4_BLOCK * 4;
  static constexpr int OFF_VP = OFF_V + CODES;
  static constexpr int BLOCK_BYTES = OFF_VP + KV4_BLOCK * 4;
  static_assert(BLOCK_BYTES == KV4_BLOCK * (D + 8), "block size");
  // V codes of token i of the block, elements 4 quad .. 4 quad + 3: 2 bytes.
  // [h = i / 8][g = quad / (D / 32)][t = (i % 8) / 2][w = quad % (D / 32)]
  // [s = i % 2][2 bytes].
  static __host__ __device__ __forceinline__ int v_code_offset(int i, int quad) {
    constexpr int W = D / 32;
    return (i >> 3) * (4 * D) + ((quad / W) * 4 + ((i & 7) >> 1)) * (D / 8) + (quad % W) * 4 +
           (i & 1) * 2;
  }
};

// Device status word of the kv4 kernels: 0 = ok, else (code << 32) | site << 16 | CTA.
enum Kv4Site : uint32_t {
  KV4_SITE_COPY = 1, KV4_SITE_SLOT, KV4_SITE_PAGE, KV4_SITE_LENGTH
};
__device__ __forceinline__ void kv4_record(unsigned long long* status, int code, uint32_t site) {
  atomicCAS(status, 0ull, (static_cast<unsigned long long>(code) << 32) |
                              (static_cast<unsigned long long>(site) << 16) |
                              (blockIdx.x & 0xFFFFu));
}

// (step, zero) halves of a parameter word as floats.
__device__ __forceinline__ float2 kv4_params(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

}  // namespace ra
