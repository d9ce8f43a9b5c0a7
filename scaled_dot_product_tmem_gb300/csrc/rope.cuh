// rope.cuh -- rotation of query and key heads by their rows' positions, shared by the kernels
// that rotate (rope.cu) and the one that rotates keys on their way into the cache (kv4_store.cu).
//
// A pair (x1, x2) of a head becomes (x1 c - x2 s, x2 c + x1 s) with c and s from a table
// [rows][2][n] of fp32 (cosines, then sines, of a row's n pairs).  Dims first .. first + 2n of a
// head hold the pairs: (f, f + n), or (2f, 2f + 1) when interleaved; the other dims stay.  The
// two products of a value are rounded to fp32 before their sum, the same everywhere, so that a
// key rotated on its way into the cache is bit for bit the one rotated by itself.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "ptx.cuh"

namespace sdpa {

struct RopeHeads {  // one tensor's rows: x read, y written (may be the same)
  const __nv_bfloat16* x = nullptr;
  __nv_bfloat16* y = nullptr;
  long long xs = 0, ys = 0;  // elements from row to row
  int H = 0;
};
struct RopeParams {
  RopeHeads a, b;      // queries and keys
  const float* table;  // [table_rows][2][n]; row t takes table row t % table_rows
  int T, table_rows, d, n, first;
  int inverse;  // turn back: the transposed rotation
  int copies;   // some tensor is turned out of place: the dims that stay are copied
};

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// x1 c - x2 s of 8 values, or x1 c + x2 s.  (Single operations: paired ones, mul.rn.f32x2 and add.rn.f32x2, are
// fused into one rounding by the assembler in spite of their .rn.)
template <bool ADD = false>
__device__ __forceinline__ uint4 rope_turn8(const uint4& x1, const uint4& x2, const float (&c)[8], const float (&s)[8]) {
  const uint32_t u[4] = {x1.x, x1.y, x1.z, x1.w}, w[4] = {x2.x, x2.y, x2.z, x2.w};
  uint32_t y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a0 = __fmul_rn(bf16_lo(u[i]), c[2 * i]), a1 = __fmul_rn(bf16_hi(u[i]), c[2 * i + 1]);
    const float b0 = __fmul_rn(bf16_lo(w[i]), s[2 * i]), b1 = __fmul_rn(bf16_hi(w[i]), s[2 * i + 1]);
    y[i] = ADD ? pack_bf16x2(__fadd_rn(a0, b0), __fadd_rn(a1, b1)) : pack_bf16x2(__fsub_rn(a0, b0), __fsub_rn(a1, b1));
  }
  return make_uint4(y[0], y[1], y[2], y[3]);
}
// 4 pairs side by side
__device__ __forceinline__ uint4 rope_turn_pairs(const uint4& x, const float* c, const float* s) {
  const uint32_t u[4] = {x.x, x.y, x.z, x.w};
  uint32_t y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = bf16_lo(u[i]), b = bf16_hi(u[i]);
    y[i] = pack_bf16x2(__fsub_rn(__fmul_rn(a, c[i]), __fmul_rn(b, s[i])), __fadd_rn(__fmul_rn(b, c[i]), __fmul_rn(a, s[i])));
  }
  return make_uint4(y[0], y[1], y[2], y[3]);
}
// (Ordinary loads: the table is written while the kernel that reads it is already set up, and a read-only load
// (__ldg) is defined only for data that nobody writes in the kernel's lifetime.)
__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = load4(p), b = load4(p + 4);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

// A head's work: n / 8 pieces of 8 pairs, and, out of place, the dims that stay in pieces of 16.
__host__ __device__ __forceinline__ int rope_pieces(const RopeParams& p) {
  return p.n / 8 + (p.copies ? (p.d - 2 * p.n + 15) / 16 : 0);
}
constexpr int kRopeHeads = 4;  // heads of a thread: h, h + groups, ...; all loaded before the first is stored
__host__ __device__ __forceinline__ int rope_groups(const RopeParams& p) { return (p.a.H + p.b.H + kRopeHeads - 1) / kRopeHeads; }
__host__ __device__ __forceinline__ long long rope_blocks(const RopeParams& p) {
  const long long items = (long long)p.T * rope_groups(p) * rope_pieces(p);
  return (items + 255) / 256;
}

// Block `block` of rope_blocks(): 256 threads, consecutive ones take consecutive pieces of a head, then
// heads, then rows.  Bound by memory: a piece is 32 bytes read and written; its place and its 64 bytes
// of the table serve all heads of a thread.
template <bool IL>
__device__ __forceinline__ void rope_block(const RopeParams& p, long long block) {
  const unsigned pieces = rope_pieces(p), turn = p.n / 8, heads = p.a.H + p.b.H, groups = rope_groups(p);
  const long long e = block * 256 + threadIdx.x;
  unsigned piece, g;
  long long t;
  if (e <= 0xffffffffLL) {  // 32-bit division
    const unsigned r = (unsigned)e / pieces, tt = r / groups;
    piece = (unsigned)e - r * pieces;
    t = tt;
    g = r - tt * groups;
  } else {
    const long long r = e / pieces;
    piece = (unsigned)(e - r * pieces);
    t = r / groups;
    g = (unsigned)(r - t * groups);
  }
  if (t >= p.T) return;
  const bool turns = piece < turn;
  int at, second;  // a piece's first vector, and from it to the second (0: there is none)
  if (turns) {
    at = p.first + piece * (IL ? 16 : 8);
    second = IL ? 8 : p.n;
  } else {
    // the dims that stay, 16 from the piece's start on: those before `first`, then those behind the pairs
    const int k = (piece - turn) * 16;
    at = k < p.first ? k : k + 2 * p.n;
    second = k + 8 >= p.d - 2 * p.n ? 0 : k + 8 < p.first ? 8 : k + 8 + 2 * p.n - at;
  }
  const long long xa = t * p.a.xs + at, xb = t * p.b.xs + at;
  uint4 v0[kRopeHeads], v1[kRopeHeads];
#pragma unroll
  for (int i = 0; i < kRopeHeads; ++i) {
    const unsigned h = g + i * groups;
    if (h >= heads) continue;
    const __nv_bfloat16* x = h < (unsigned)p.a.H ? p.a.x + xa + (size_t)h * p.d : p.b.x + xb + (size_t)(h - p.a.H) * p.d;
    v0[i] = __ldcs(reinterpret_cast<const uint4*>(x));
    if (second) v1[i] = __ldcs(reinterpret_cast<const uint4*>(x + second));
  }
  float c[8], s[8];
  if (turns) {
    const float* cs = p.table + (size_t)(p.table_rows == p.T ? t : t % p.table_rows) * 2 * p.n + piece * 8;
    load8(cs, c);
    load8(cs + p.n, s);
    if (p.inverse) {
#pragma unroll
      for (int j = 0; j < 8; ++j) s[j] = -s[j];
    }
  }
  const long long ya = t * p.a.ys + at, yb = t * p.b.ys + at;
#pragma unroll
  for (int i = 0; i < kRopeHeads; ++i) {
    const unsigned h = g + i * groups;
    if (h >= heads) continue;
    __nv_bfloat16* y = h < (unsigned)p.a.H ? p.a.y + ya + (size_t)h * p.d : p.b.y + yb + (size_t)(h - p.a.H) * p.d;
    uint4 y0 = v0[i], y1 = v1[i];
    if (turns) {
      if constexpr (IL) {
        y0 = rope_turn_pairs(v0[i], c, s);
        y1 = rope_turn_pairs(v1[i], c + 4, s + 4);
      } else {
        y0 = rope_turn8(v0[i], v1[i], c, s);
        y1 = rope_turn8<true>(v1[i], v0[i], c, s);
      }
    }
    *reinterpret_cast<uint4*>(y) = y0;
    if (second) *reinterpret_cast<uint4*>(y + second) = y1;
  }
}

}  // namespace sdpa
