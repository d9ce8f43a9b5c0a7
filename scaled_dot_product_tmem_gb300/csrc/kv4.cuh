// kv4.cuh -- the 4-bit paged key/value cache: its layout and its number format, shared by
// the kernels that fill, read and attend over it.
//
// A pool is [n_pages][H_kv][block] bytes; the block of one page and kv head holds
// page_size tokens of head dim d (64 or 128) in four consecutive parts:
//   K codes   [page_size][d/2]            two codes a byte, the even dim in the low nibble
//   V codes   [page_size/2][8][2][d/16]   token pair u: eighth g of the head dim at slot
//                                         g ^ x(u), the pair's two tokens side by side
//   K scales  [page_size][d/16]           one byte for 16 dims
//   V scales  [page_size/2][d/16][2]
// so a page's block is one contiguous piece of page_size * 9d/8 bytes (4.5 bits a value).
// V is stored by token pairs because P.V contracts over tokens: a lane then reads both
// tokens of an operand register in one access.  The slot permutation x(u) spreads the 4
// token pairs that a quarter-warp reads at once over all shared-memory banks.
//
// A code c (0..15) stands for (c - 8) s.  The scale byte holds bits 14..7 of a
// half-precision number: 5 exponent bits, 3 mantissa bits, no sign, up to 61440.  A
// 4-bit integer times a 4-bit significand has at most 8 significant bits, so every held
// value is exactly a bf16 number and the tensor core multiplies it without a rounding.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace sdpa {

struct Kv4Pool {
  const int* page_table;  // [B, max_pages]
  int n_pages, page_size, max_pages;
  int H_kv, d;
  int page_shift;  // log2(page_size)
};

// Byte offsets of the four parts inside a block.
__host__ __device__ __forceinline__ int kv4_block_bytes(int P, int d) { return P * d * 9 / 8; }
__host__ __device__ __forceinline__ int kv4_off_v(int P, int d) { return P * d / 2; }
__host__ __device__ __forceinline__ int kv4_off_sk(int P, int d) { return P * d; }
__host__ __device__ __forceinline__ int kv4_off_sv(int P, int d) { return P * d + P * d / 16; }

// Slot permutation of token pair u.
__host__ __device__ __forceinline__ int kv4_slot_xor(int u, int d) {
  return d == 128 ? 2 * (u & 3) : 4 * ((u >> 1) & 1);
}

// Byte offset of token w's codes of eighth g (d/16 bytes) inside the V part.
__host__ __device__ __forceinline__ int kv4_v_at(int w, int g, int d) {
  const int u = w >> 1;
  return u * d + (g ^ kv4_slot_xor(u, d)) * (d / 8) + (w & 1) * (d / 16);
}

// Scale byte of 16 values whose largest magnitude is amax: amax / 7 rounded to 3 mantissa
// bits, ties to even, at most 0xF7.  Below 2^-14 the format's step is 2^-17.
__device__ __forceinline__ int kv4_scale_byte(float amax) {
  const float r = __fdiv_rn(amax, 7.f);
  if (r < 6.103515625e-05f) return __float2int_rn(r * 131072.f);
  const uint32_t u = __float_as_uint(r);
  const int b = (int)((u + 0x7FFFFu + ((u >> 20) & 1u)) >> 20) - (112 << 3);
  return b < 0xF7 ? b : 0xF7;
}

__device__ __forceinline__ float kv4_scale_value(int byte) {
  return __half2float(__ushort_as_half((unsigned short)(byte << 7)));
}

constexpr int kKv4BadScale = 0xFF;  // 16 values with an infinity or NaN among them: a NaN scale

// The page that holds token `pos` of sequence b, or -1 (outside the table or the pool).
__device__ __forceinline__ int kv4_page(const Kv4Pool& c, int b, int pos) {
  if (pos < 0 || (pos >> c.page_shift) >= c.max_pages) return -1;
  const int pg = __ldg(c.page_table + (size_t)b * c.max_pages + (pos >> c.page_shift));
  return (pg < 0 || pg >= c.n_pages) ? -1 : pg;
}

// Which sequence holds row t of a packed tensor: the last b with cu[b] <= t, checked
// against its end; -1 when no sequence does.  Offsets that are not ascending may give any
// sequence, never a row outside the one returned.
__device__ __forceinline__ int packed_row_entry(const int* cu, int B, int t) {
  int lo = 0, hi = B;  // cu[lo] <= t is looked for in [0, B)
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(cu + mid) <= t) lo = mid + 1;
    else hi = mid;
  }
  const int b = lo - 1;
  return (b >= 0 && __ldg(cu + b) <= t && t < __ldg(cu + b + 1)) ? b : -1;
}

}  // namespace sdpa
