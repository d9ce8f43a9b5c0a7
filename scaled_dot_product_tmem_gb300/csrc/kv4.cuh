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

#include "ptx.cuh"

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

// Paired bf16 arithmetic.
__device__ __forceinline__ uint32_t bf2_fma(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t bf2_mul(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// Codes c in bits 0-3 and 16-19 of w as the bf16 pair (c - 8) s, with s and -136 s paired.
// The mask and the exponent bits are one three-input operation, (w & mask) | bits.
__device__ __forceinline__ uint32_t decode_pair(uint32_t w, uint32_t s, uint32_t m136s) {
  uint32_t x;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(x) : "r"(w), "r"(0x000F000Fu), "r"(0x43004300u));
  return bf2_fma(x, s, m136s);
}
// Two scale bytes (low, next) as a bf16 pair: bits 14..7 of two half-precision numbers.
__device__ __forceinline__ uint32_t scale_pair(uint32_t two) {
  const uint32_t h = __byte_perm(two, 0u, 0x4140) << 7;
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return pack_bf16x2(f.x, f.y);
}
constexpr uint32_t kM136 = 0xC308C308u;  // -136 as a bf16 pair

// The same pair times 2^-23, with fewer operations.  bf16 bits below 256 are linear across the
// subnormal numbers and the first normal binade: bits v stand for v 2^-133.  So a code masked
// out of bits 0-3 or 4-7 of a half is already a number, c 2^-133 or 16 c 2^-133, and one fma
// with s 2^110 or s 2^106 and -8 s 2^-23 gives (c - 8) s 2^-23, exact as before (s < 2^16): two
// nibbles of every half need no shift, and no code needs exponent bits.
struct Kv4Small {
  uint32_t lo, hi, m8;  // s 2^110, s 2^106, -8 s 2^-23
};
__device__ __forceinline__ Kv4Small small_scales(uint32_t s) {
  Kv4Small r;
  r.lo = bf2_mul(s, 0x76807680u);  // 2^110
  r.hi = bf2_mul(s, 0x74807480u);  // 2^106
  r.m8 = bf2_mul(s, 0xB580B580u);  // -2^-20
  return r;
}
__device__ __forceinline__ uint32_t decode_small_lo(uint32_t w, const Kv4Small& k) {
  return bf2_fma(w & 0x000F000Fu, k.lo, k.m8);
}
__device__ __forceinline__ uint32_t decode_small_hi(uint32_t w, const Kv4Small& k) {
  return bf2_fma(w & 0x00F000F0u, k.hi, k.m8);
}
constexpr float kKv4SmallUndo = 8388608.f;  // 2^23

constexpr int kKv4BadScale = 0xFF;  // 16 values with an infinity or NaN among them: a NaN scale

// A load of what no kernel writes while this one lives; with EARLY, in a kernel that is launched while the one before it
// runs, an ordinary load, since that one may write it (a read-only load is then undefined).
template <bool EARLY, class T>
__device__ __forceinline__ T load_input(const T* p) {
  if constexpr (EARLY) return *p;
  else return __ldg(p);
}

// The page that holds token `pos` of sequence b, or -1 (outside the table or the pool).
template <bool EARLY = false>
__device__ __forceinline__ int kv4_page(const Kv4Pool& c, int b, int pos) {
  if (pos < 0 || (pos >> c.page_shift) >= c.max_pages) return -1;
  const int pg = load_input<EARLY>(c.page_table + (size_t)b * c.max_pages + (pos >> c.page_shift));
  return (pg < 0 || pg >= c.n_pages) ? -1 : pg;
}

}  // namespace sdpa
