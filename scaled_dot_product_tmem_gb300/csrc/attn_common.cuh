// attn_common.cuh -- index arithmetic shared by the forward and backward kernels:
// which keys a query row sees, which kv tiles a block of query rows touches, and
// which query tiles a block of keys is seen by.
//
// Masking rule (causal with an optional left window, top-left diagonal):
//   key j is visible to query i  iff  i < S_q and j < S_kv and (!causal or j <= i)
//                                     and (window < 0 or j >= i - window).
// In a padded batch S_q and S_kv are the entry's own lengths, so its padded query
// rows see no key and its padded keys are seen by no query.
// ("JAX: Single-GPU Attention with TransformerEngine", sections 1-2: causal
// mask plus sliding window; codelab "Speed up attention on GPU with cuDNN and
// TransformerEngine", step 7: query i sees keys j <= i.)
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace sdpa {

struct MaskSpec {
  int S_q, S_kv, causal, window;
};

// VL: the batch is padded (S_q is the entry's own length and rows past it exist);
// without it every row the kernels look at is below S_q and the row test is dropped.
template <bool VL>
__host__ __device__ __forceinline__ bool key_visible(const MaskSpec& m, int i, int j) {
  return (!VL || i < m.S_q) && j < m.S_kv && (!m.causal || j <= i) && (m.window < 0 || j >= i - m.window);
}

// The keys query row i sees form one interval [*lo, *hi] (empty when lo > hi):
// the same set key_visible<VL> describes, as two bounds a mask loop can compare with.
template <bool VL>
__host__ __device__ __forceinline__ void visible_keys(const MaskSpec& m, int i, int* lo, int* hi) {
  int a = m.window >= 0 ? i - m.window : 0;
  int z = m.causal ? i : m.S_kv - 1;
  if (z > m.S_kv - 1) z = m.S_kv - 1;
  *lo = a < 0 ? 0 : a;
  *hi = (VL && i >= m.S_q) ? -1 : z;
}

// The query rows that see key j form one interval [*lo, *hi] (empty when lo > hi).
template <bool VL>
__host__ __device__ __forceinline__ void visible_rows(const MaskSpec& m, int j, int* lo, int* hi) {
  int a = m.causal ? j : 0;
  int z = m.window >= 0 ? j + m.window : 0x7fffffff - 1;
  if (VL && z > m.S_q - 1) z = m.S_q - 1;
  *lo = a;
  *hi = j < m.S_kv ? z : -1;
}

// Length of batch entry b: lens[b] clamped to [0, S], or S without a length array.
__host__ __device__ __forceinline__ int entry_len(const int* lens, int b, int S) {
  if (!lens) return S;
  const int l = lens[b];
  return l < 0 ? 0 : (l > S ? S : l);
}

// Inclusive range of kv tiles (size bn) touched by query rows [r0, r1]; returns
// false when those rows see no key at all.
__host__ __device__ __forceinline__ bool kv_tile_range(const MaskSpec& m, int r0, int r1, int bn, int* jlo,
                                                       int* jhi) {
  if (r1 > m.S_q - 1) r1 = m.S_q - 1;
  if (r1 < r0) return false;
  int lo = m.window >= 0 ? (r0 - m.window > 0 ? r0 - m.window : 0) : 0;
  int hi = m.causal ? (r1 < m.S_kv - 1 ? r1 : m.S_kv - 1) : m.S_kv - 1;
  if (hi < lo || m.S_kv <= 0) return false;
  *jlo = lo / bn;
  *jhi = hi / bn;
  return true;
}

// Inclusive range of query tiles (size bm) that see at least one key of
// [k0, k1]; returns false when none does.
__host__ __device__ __forceinline__ bool q_tile_range(const MaskSpec& m, int k0, int k1, int bm, int* ilo,
                                                      int* ihi) {
  if (k1 > m.S_kv - 1) k1 = m.S_kv - 1;
  if (k1 < k0) return false;
  int lo = m.causal ? k0 : 0;
  int hi = m.window >= 0 ? k1 + m.window : m.S_q - 1;
  if (hi > m.S_q - 1) hi = m.S_q - 1;
  if (hi < lo || m.S_q <= 0) return false;
  *ilo = lo / bm;
  *ihi = hi / bm;
  return true;
}

// Is the whole (rows [r0, r0+bm), keys [k0, k0+bn)) tile visible?  Then the
// per-element mask can be skipped.  (Without VL, rows past S_q are never stored.)
template <bool VL>
__host__ __device__ __forceinline__ bool tile_fully_visible(const MaskSpec& m, int r0, int bm, int k0, int bn) {
  int r1 = r0 + bm - 1;
  int k1 = k0 + bn - 1;
  if (k1 >= m.S_kv || (VL && r1 >= m.S_q)) return false;
  if (m.causal && k1 > r0) return false;
  if (m.window >= 0 && k0 < r1 - m.window) return false;
  return true;
}

// A packed batch (sequences one after another in [T, H, d] tensors): one work tile of a
// kernel, as the plan kernel lists it.  q0 / k0: the sequence's first query / key row in the
// packed tensors; Lq / Lk its lengths; m0 the tile's first row within the sequence; ws0 the
// sequence's first row in workspace rows padded to multiples of 128.
struct PackedTile {
  int q0, Lq, k0, Lk, b, m0, ws0, unused;
};
static_assert(sizeof(PackedTile) == 32, "read as two 16-byte words");

// Ordinary loads: the list is written while the kernel that reads it is already set up, and a
// read-only load (__ldg) is defined only for data that nobody writes in the kernel's lifetime.
__device__ __forceinline__ PackedTile load_packed_tile(const PackedTile* t, int i) {
  const int4* w = reinterpret_cast<const int4*>(t + i);
  const int4 a = w[0], b = w[1];
  return PackedTile{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
}

// What the plan of a packed batch counts.
struct PackedCounts {
  int fwd_tiles, kv_tiles, q_tiles;  // entries of the tile lists
  // the sequences' rows: [q_begin, q_end) and [kv_begin, kv_end) (they follow one another, so the
  // rows before and behind these belong to no sequence)
  int q_begin, q_end, kv_begin, kv_end;
  int next;  // forward: work tiles taken beyond each CTA's first
};

// A small packed batch needs no plan kernel: every CTA finds its one tile itself.
constexpr int kOwnSeqs = 31;  // one lane an offset
struct PackedOffsets {
  const int* cu_q = nullptr;
  const int* cu_kv = nullptr;
  int B = 0, T_q = 0, T_kv = 0;
};
struct OwnTile {
  PackedTile e;
  int n, q_begin, q_end, unused;  // tiles of the batch; the sequences' rows
};
// Tile i of ROWS query rows, in the order of the sequences (a warp).
template <int ROWS>
__device__ __forceinline__ void find_own_tile(const PackedOffsets& c, int i, OwnTile* out) {
  const int lane = threadIdx.x % 32;
  const bool same = c.cu_kv == c.cu_q && c.T_kv == c.T_q;
  int q = lane <= c.B ? min(max(__ldg(c.cu_q + lane), 0), c.T_q) : 0;
  int k = lane <= c.B && !same ? min(max(__ldg(c.cu_kv + lane), 0), c.T_kv) : 0;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {  // running maxima (below `off` a lane gets its own value)
    q = max(q, __shfl_up_sync(0xffffffffu, q, off));
    k = max(k, __shfl_up_sync(0xffffffffu, k, off));
  }
  if (same) k = q;
  const int Lq = __shfl_down_sync(0xffffffffu, q, 1) - q, Lk = __shfl_down_sync(0xffffffffu, k, 1) - k;
  const int n = lane < c.B ? (Lq + ROWS - 1) / ROWS : 0;
  int upto = n;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, upto, off);
    if (lane >= off) upto += o;
  }
  const int j = i - (upto - n);
  if (j >= 0 && j < n) out->e = PackedTile{q, Lq, k, Lk, lane, j * ROWS, 0, 0};
  if (lane == 31) out->n = upto;
  if (lane == 0) out->q_begin = q;
  if (lane == c.B) out->q_end = q;
}

// Zero rows [from, rows) of `chunks` shared-memory chunks of rows x 128 bytes (a warp).  Whole
// 128-byte rows: the swizzle permutes bytes inside a row only.
__device__ __forceinline__ void zero_tile_rows(uint8_t* base, int chunks, int chunk_bytes, int rows, int from,
                                               int lane) {
  for (int c = 0; c < chunks; ++c)
    for (int o = from * 128 + lane * 16; o < rows * 128; o += 32 * 16)
      *reinterpret_cast<uint4*>(base + c * chunk_bytes + o) = make_uint4(0u, 0u, 0u, 0u);
}

__device__ __forceinline__ uint8_t* align1024(uint8_t* p) {
  return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(p) + 1023) & ~static_cast<uintptr_t>(1023));
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Additive bias ("JAX: Single-GPU Attention with TransformerEngine", section "Other
// attention knobs": `bias` with an `attn_bias_type`): a bf16 [Bb, Hb, S_q, S_kv] tensor
// added to the scaled scores; Bb in {1, B} and Hb in {1, H_q} broadcast, expressed as
// element strides that are 0 along a broadcast dim.
__device__ __forceinline__ float bf16_bits_to_float(unsigned short u) { return __uint_as_float((uint32_t)u << 16); }

// 8 consecutive bias values of one row, starting at key k (0 for keys >= S_kv).  vec:
// S_kv is a multiple of 8 and k of 8, so one 16-byte load covers them (all or none
// below S_kv).
__device__ __forceinline__ void load_bias8(const __nv_bfloat16* row, int k, int S_kv, bool vec, float (&out)[8]) {
  if (vec) {
    uint4 w = make_uint4(0u, 0u, 0u, 0u);
    if (k < S_kv) w = __ldg(reinterpret_cast<const uint4*>(row + k));
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      out[2 * q] = __uint_as_float(ws[q] << 16);
      out[2 * q + 1] = __uint_as_float(ws[q] & 0xFFFF0000u);
    }
  } else {
    const unsigned short* r = reinterpret_cast<const unsigned short*>(row);
#pragma unroll
    for (int e = 0; e < 8; ++e) out[e] = (k + e < S_kv) ? bf16_bits_to_float(__ldg(r + k + e)) : 0.f;
  }
}

}  // namespace sdpa
