// attn_packed.cu -- attention over packed sequences: the plan kernel that lists the work tiles,
// the packed instantiations of the forward and of the deterministic backward kernels, and
// the backward's small kernels in their packed form.
//
// Sequence b holds rows cu_q[b] .. cu_q[b + 1] - 1 of q and o and rows cu_kv[b] .. of k and v,
// and computes as a batch entry of its own (masks, lengths and sinks as in
// attn_common.cuh).  Nothing is padded: a kernel's tiles start at a sequence's first row, the
// TMA maps see one long sequence [1, T, H, d], and what a tile holds past its sequence's end
// is masked, never stored, and zeroed where it would be a product's operand.
#include <cuda_runtime.h>

#include "attn_bwd_kernels.cuh"
#include "attn_fwd_kernel.cuh"
#include "attn_packed.h"
#include "launch.h"

namespace sdpa {

// =============================================================================
// Plan: the work tiles of every kernel, from the sequence offsets.
//
// One block.  The offsets are device data and may be anything: they are clamped to [0, T] and
// replaced by their running maximum, so sequences never overlap and the lists never pass the
// host's bounds (T / rows + B entries).  A counting sort by bucket puts the most work first:
//   forward   each 256-row query tile by the kv tiles it sees: the persistent CTAs take
//             tiles in turn, and with falling costs no CTA ends up more than one tile behind;
//   kv and q  whole sequences by length, a sequence's heaviest tiles first: the tiles in
//             flight belong to few sequences, whose other operand they share in L2.
// The order inside a bucket varies from run to run; no result depends on it.
// =============================================================================
constexpr int kPlanThreads = 1024;

namespace {

// The running maximum of clamped offsets, by the whole block.
__device__ void clean_offsets(const int* cu, int B, int T, int* out, int* part) {
  int carry = 0;
  for (int base = 0; base <= B; base += kPlanThreads) {
    const int i = base + threadIdx.x, lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    int v = i <= B ? min(max(__ldg(cu + i), 0), T) : 0;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) v = max(v, __shfl_up_sync(0xffffffffu, v, off));  // (own value below `off`)
    if (lane == 31) part[warp] = v;
    __syncthreads();
    int before = carry;
    for (int w = 0; w < warp; ++w) before = max(before, part[w]);
    v = max(v, before);
    if (i <= B) out[i] = v;
    __syncthreads();
    if (threadIdx.x == kPlanThreads - 1) part[0] = v;
    __syncthreads();
    carry = part[0];
    __syncthreads();
  }
}

enum PlanKind { kPlanFwd, kPlanKv, kPlanQ };

template <int KIND>
struct PlanRows {
  static constexpr int value = KIND == kPlanFwd ? 256 : 128;
};

// Lists one kernel's tiles; returns their number.
template <int KIND>
__device__ int list_tiles(const PackedPlanParams& p, const int* cq, const int* ck, PackedTile* out, int* hist,
                          int* part) {
  constexpr int ROWS = PlanRows<KIND>::value;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  auto bucket = [&](int Lq, int Lk, int n, int j) {
    int w = n;
    if constexpr (KIND == kPlanFwd) {
      int lo = 1, hi = 0;
      w = kv_tile_range(MaskSpec{Lq, Lk, p.causal, p.window}, j * ROWS, j * ROWS + ROWS - 1, 128, &lo, &hi)
              ? hi - lo + 1 : 0;
    }
    return min(w, kPlanThreads - 1);
  };
  // f(sequence b, its four numbers, its tiles n, first tile, step between tiles): sequences of up
  // to 8 tiles by one thread each, longer ones by the warp
  auto walk = [&](auto f) {
    for (int b0 = warp * 32; b0 < p.B; b0 += kPlanThreads) {
      const int b = b0 + lane;
      int q0 = 0, Lq = 0, k0 = 0, Lk = 0;
      if (b < p.B) {
        q0 = cq[b];
        Lq = cq[b + 1] - q0;
        k0 = ck[b];
        Lk = ck[b + 1] - k0;
      }
      const int n = ((KIND == kPlanKv ? Lk : Lq) + ROWS - 1) / ROWS;
      if (n > 0 && n <= 8) f(b, q0, Lq, k0, Lk, n, 0, 1);
      for (unsigned m = __ballot_sync(0xffffffffu, n > 8); m; m &= m - 1) {
        const int s = __ffs(m) - 1;
        f(b0 + s, __shfl_sync(0xffffffffu, q0, s), __shfl_sync(0xffffffffu, Lq, s), __shfl_sync(0xffffffffu, k0, s),
          __shfl_sync(0xffffffffu, Lk, s), __shfl_sync(0xffffffffu, n, s), lane, 32);
      }
    }
  };
  hist[threadIdx.x] = 0;
  __syncthreads();
  walk([&](int, int, int Lq, int, int Lk, int n, int j0, int step) {
    if constexpr (KIND == kPlanFwd) {
      for (int j = j0; j < n; j += step) atomicAdd(&hist[bucket(Lq, Lk, n, j)], 1);
    } else if (j0 == 0) {
      atomicAdd(&hist[bucket(Lq, Lk, n, 0)], n);
    }
  });
  __syncthreads();
  // first entry of each bucket, the highest bucket first
  const int mine = hist[kPlanThreads - 1 - threadIdx.x];
  int sum = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, sum, off);
    if (lane >= off) sum += o;
  }
  if (lane == 31) part[warp] = sum;
  __syncthreads();
  int total = 0;
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    if (w < warp) sum += part[w];
    total += part[w];
  }
  hist[kPlanThreads - 1 - threadIdx.x] = sum - mine;
  __syncthreads();
  walk([&](int b, int q0, int Lq, int k0, int Lk, int n, int j0, int step) {
    int base = 0;
    if constexpr (KIND != kPlanFwd) {
      if (j0 == 0) base = atomicAdd(&hist[bucket(Lq, Lk, n, 0)], n);
      if (step == 32) base = __shfl_sync(0xffffffffu, base, 0);
    }
    for (int j = j0; j < n; j += step) {
      int at, tile = j;
      if constexpr (KIND == kPlanFwd) {
        at = atomicAdd(&hist[bucket(Lq, Lk, n, j)], 1);
      } else {
        at = base + j;
        if (KIND == kPlanQ && p.causal) tile = n - 1 - j;  // under a causal mask the last query tile sees most
      }
      int4* e = reinterpret_cast<int4*>(out + at);
      e[0] = make_int4(q0, Lq, k0, Lk);
      e[1] = make_int4(b, tile * ROWS, (int)(((long long)q0 + 128LL * b) / 128 * 128), 0);
    }
  });
  __syncthreads();
  return total;
}

__global__ void __launch_bounds__(kPlanThreads) packed_plan_kernel(const PackedPlanParams p) {
  __shared__ int hist[kPlanThreads], part[32];
  grid_launch_dependents();
  clean_offsets(p.cu_q, p.B, p.T_q, p.clean_q, part);
  const int* ck = p.clean_q;
  if (p.cu_kv != p.cu_q || p.T_kv != p.T_q) {
    clean_offsets(p.cu_kv, p.B, p.T_kv, p.clean_kv, part);
    ck = p.clean_kv;
  }
  __syncthreads();
  PackedCounts c{};
  if (p.tiles_fwd) c.fwd_tiles = list_tiles<kPlanFwd>(p, p.clean_q, ck, p.tiles_fwd, hist, part);
  if (p.tiles_kv) c.kv_tiles = list_tiles<kPlanKv>(p, p.clean_q, ck, p.tiles_kv, hist, part);
  if (p.tiles_q) c.q_tiles = list_tiles<kPlanQ>(p, p.clean_q, ck, p.tiles_q, hist, part);
  if (threadIdx.x == 0) {
    c.q_end = p.clean_q[p.B];
    c.kv_end = ck[p.B];
    *p.counts = c;
  }
}

}  // namespace

int launch_packed_plan(const PackedPlanParams& p, cudaStream_t stream) {
  packed_plan_kernel<<<1, kPlanThreads, 0, stream>>>(p);
  return cudaPeekAtLastError() == cudaSuccess ? 0 : -1;
}

// =============================================================================
// Forward
// =============================================================================
int launch_attn_fwd_packed(int d_qk, int d_v, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                           const FwdParams& p, cudaStream_t stream) {
  if (d_qk == 128 && d_v == 128)
    return launch_fwd_t<128, 128, 2, 2, true, false, false, false, true>(tq, tk, tv, p, stream);
  if (d_qk == 64 && d_v == 64) return launch_fwd_t<64, 64, 4, 4, true, false, false, false, true>(tq, tk, tv, p, stream);
  if (d_qk == 192 && d_v == 128)
    return launch_fwd_t<192, 128, 2, 1, true, false, false, false, true>(tq, tk, tv, p, stream);
  return -2;
}

// =============================================================================
// Backward preprocess: D = rowsum(dO * O) and -LSE log2(e) in the workspace's padded rows (the
// padding: D = 0, -inf), one block per 64 rows of a query tile and head; on request also
// zeros in the gradient rows of no sequence.
// =============================================================================
template <int D_V>
__global__ void __launch_bounds__(256) packed_preprocess_kernel(const BwdParams p, int d_qk) {
  constexpr int TPR = D_V / 8, RPP = 256 / TPR, TILE = 64, NR = TILE / RPP;
  __shared__ float dsum[TILE];
  const int h = blockIdx.y;
  grid_launch_dependents();
  grid_wait();  // the plan
  if ((int)(blockIdx.x / 2) < p.counts->q_tiles) {
    const PackedTile e = load_packed_tile(p.tiles_q, blockIdx.x / 2);
    const int i0 = e.m0 + (blockIdx.x % 2) * TILE, sub = threadIdx.x % TPR;
    uint4 a[NR], g[NR];
#pragma unroll
    for (int k = 0; k < NR; ++k) {
      const int i = i0 + threadIdx.x / TPR + k * RPP;
      a[k] = g[k] = make_uint4(0u, 0u, 0u, 0u);
      if (i < e.Lq) {
        const size_t off = ((size_t)(e.q0 + i) * p.H_q + h) * D_V + sub * 8;
        a[k] = __ldcs(reinterpret_cast<const uint4*>(p.o + off));
        g[k] = __ldcs(reinterpret_cast<const uint4*>(p.dout + off));
      }
    }
#pragma unroll
    for (int k = 0; k < NR; ++k) {
      float acc = 0.f;
      const __nv_bfloat162* a2 = reinterpret_cast<const __nv_bfloat162*>(&a[k]);
      const __nv_bfloat162* g2 = reinterpret_cast<const __nv_bfloat162*>(&g[k]);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float2 fa = __bfloat1622float2(a2[q]), fg = __bfloat1622float2(g2[q]);
        acc = fmaf(fa.x, fg.x, acc);
        acc = fmaf(fa.y, fg.y, acc);
      }
#pragma unroll
      for (int off = TPR / 2; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
      if (sub == 0) dsum[threadIdx.x / TPR + k * RPP] = acc;
    }
    __syncthreads();
    if (threadIdx.x < TILE) {
      const int i = i0 + threadIdx.x;
      const bool real = i < e.Lq;
      const size_t w = (size_t)h * p.S_pad + e.ws0 + i;
      p.Dsum[w] = real ? dsum[threadIdx.x] : 0.f;
      const float l = real ? p.lse[(size_t)h * p.S_q + e.q0 + i] : -INFINITY;
      p.nlse2[w] = l == -INFINITY ? -INFINITY : -l * kLog2e;
    }
  }
  if (p.zero_rest) {
    const size_t at = ((size_t)blockIdx.y * gridDim.x + blockIdx.x) * 256 + threadIdx.x;
    const size_t step = (size_t)gridDim.x * gridDim.y * 256;
    const uint4 z = make_uint4(0u, 0u, 0u, 0u);
    auto clear = [&](__nv_bfloat16* x, int from, int rows, int H, int d) {
      uint4* x16 = reinterpret_cast<uint4*>(x + (size_t)from * H * d);
      const size_t n = (size_t)(rows - from) * H * (d / 8);
      for (size_t i = at; i < n; i += step) x16[i] = z;
    };
    clear(p.dq, p.counts->q_end, p.S_q, p.H_q, d_qk);
    clear(p.dk, p.counts->kv_end, p.S_kv, p.H_kv, d_qk);
    clear(p.dv, p.counts->kv_end, p.S_kv, p.H_kv, D_V);
  }
}

int launch_packed_preprocess(int d_qk, int d_v, const BwdParams& p, cudaStream_t stream) {
  if (2 * p.tile_bound_q > 0x7fffffffLL) return -2;
  const dim3 grid((unsigned)(2 * p.tile_bound_q), p.H_q);
  if (d_v == 64) return launch_kernel(packed_preprocess_kernel<64>, grid, 256, 0, stream, true, p, d_qk);
  if (d_v == 128) return launch_kernel(packed_preprocess_kernel<128>, grid, 256, 0, stream, true, p, d_qk);
  return -2;
}

// d offset_h = -sum_i ps_i D*_i with ps_i = exp(offset_h - LSE_i) and D*_i = dO_i . O_i of the
// unrounded O.  The kernels hold D_i from the stored bf16 O; but sum_j P_ij = 1 - ps_i, so the
// dQ kernel's fp32 row sums r_i = sum_j P_ij (dP_ij - D_i) give D*_i = r_i + D_i (1 - ps_i): the
// sum then carries fp32 rounding only.  One block per head, fixed order: bitwise reproducible.
// Padding rows hold zeros in D and r.
__global__ void __launch_bounds__(1024) packed_doffset_kernel(const BwdParams p) {
  const int h = blockIdx.x;
  const float c2 = p.offset[h] * kLog2e;
  const float4* nl = reinterpret_cast<const float4*>(p.nlse2 + (size_t)h * p.S_pad);
  const float4* dd = reinterpret_cast<const float4*>(p.Dsum + (size_t)h * p.S_pad);
  const float4* ra = reinterpret_cast<const float4*>(p.ds_rowsum + (size_t)h * p.S_pad);
  const float4* rb = reinterpret_cast<const float4*>(p.ds_rowsum + ((size_t)p.H_q + h) * p.S_pad);
  float acc = 0.f;
  auto add = [&](float n, float d, float r0, float r1) {
    if (d == 0.f && r0 == 0.f && r1 == 0.f) return;  // padding (its exponential may overflow)
    const float ps = ex2(c2 + n);
    acc = fmaf(ps, r0 + r1 + d * (1.f - ps), acc);
  };
  for (int i = threadIdx.x; i < p.S_pad / 4; i += 1024) {
    const float4 n = nl[i], d = dd[i], a = ra[i], b = rb[i];
    add(n.x, d.x, a.x, b.x);
    add(n.y, d.y, a.y, b.y);
    add(n.z, d.z, a.z, b.z);
    add(n.w, d.w, a.w, b.w);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
  __shared__ float part[32];
  if ((threadIdx.x & 31) == 0) part[threadIdx.x / 32] = acc;
  __syncthreads();
  if (threadIdx.x == 0) {
    float s = 0.f;
    for (int w = 0; w < 32; ++w) s += part[w];
    p.d_offset[h] = -s;
  }
}

int launch_packed_doffset(const BwdParams& p, cudaStream_t stream) {
  packed_doffset_kernel<<<p.H_q, 1024, 0, stream>>>(p);
  return cudaPeekAtLastError() == cudaSuccess ? 0 : -1;
}

// dK, dV = bf16(sum over the head splits of the fp32 partial slices), slice 0 first, for the
// rows of the sequences.
__global__ void __launch_bounds__(256) packed_kv_combine_kernel(const float4* __restrict__ part,
                                                                uint2* __restrict__ out, size_t slice4,
                                                                const PackedCounts* counts, int row4, int ns) {
  const size_t n4 = (size_t)counts->kv_end * row4;
  for (size_t t = (size_t)blockIdx.x * 256 + threadIdx.x; t < n4; t += (size_t)gridDim.x * 256) {
    float4 a = part[t];
    for (int s = 1; s < ns; ++s) {
      const float4 b = part[(size_t)s * slice4 + t];
      a.x += b.x; a.y += b.y; a.z += b.z; a.w += b.w;
    }
    out[t] = make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
  }
}

int launch_packed_kv_combine(int d_qk, int d_v, const BwdParams& p, cudaStream_t stream) {
  for (int w = 0; w < 2; ++w) {
    const int row4 = p.H_kv * (w == 0 ? d_qk : d_v) / 4;
    const size_t n4 = (size_t)p.S_kv * row4;
    const unsigned blocks = (unsigned)((n4 + 255) / 256 < 152 * 16 ? (n4 + 255) / 256 : 152 * 16);
    packed_kv_combine_kernel<<<blocks, 256, 0, stream>>>(
        reinterpret_cast<const float4*>(w == 0 ? p.dk_part : p.dv_part),
        reinterpret_cast<uint2*>(w == 0 ? p.dk : p.dv), n4, p.counts, row4, p.ns);
  }
  return cudaPeekAtLastError() == cudaSuccess ? 0 : -1;
}

// =============================================================================
// Backward kernels.  d_qk = d_v: the 128-row kv kernel (attn_bwd_wide.cu); (192, 128): the 64-row one.
// =============================================================================
int launch_bwd_kv_packed_mla(const CUtensorMap& tq64, const CUtensorMap& tk, const CUtensorMap& tv,
                             const CUtensorMap& tdo64, const BwdParams& p, cudaStream_t stream) {
  using C = KvCfg<192, 128, false>;
  const long long grid = p.tile_bound_kv * p.H_kv * p.ns;
  if (grid <= 0 || grid > 0x7fffffffLL) return -2;
  auto kern = attn_bwd_kv_kernel<192, 128, false, true, false, false, false, true>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess) return -1;
  return launch_kernel(kern, dim3((unsigned)grid), C::THREADS, C::SMEM, stream, true, tq64, tk, tv, tdo64, tq64, tq64, p);
}

template <int D_QK, int D_V>
static int launch_q_packed_t(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                             const CUtensorMap& tdo, const BwdParams& p, bool early, cudaStream_t stream) {
  using C = QCfg<D_QK, D_V>;
  const long long grid = p.tile_bound_q * p.H_q;
  if (grid <= 0 || grid > 0x7fffffffLL) return -2;
  auto kern = p.ds_rowsum ? attn_bwd_q_kernel<D_QK, D_V, true, false, false, false, true, true>
                          : attn_bwd_q_kernel<D_QK, D_V, true, false, false, false, true, false>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess) return -1;
  return launch_kernel(kern, dim3((unsigned)grid), C::THREADS, C::SMEM, stream, early, tq, tk, tv, tdo, p);
}

// early: right behind the kv kernel on the stream, whose tail it may overlap (it needs nothing of it).
int launch_bwd_q_packed(int d_qk, int d_v, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                        const CUtensorMap& tdo, const BwdParams& p, bool early, cudaStream_t stream) {
  if (d_qk == 128 && d_v == 128) return launch_q_packed_t<128, 128>(tq, tk, tv, tdo, p, early, stream);
  if (d_qk == 64 && d_v == 64) return launch_q_packed_t<64, 64>(tq, tk, tv, tdo, p, early, stream);
  if (d_qk == 192 && d_v == 128) return launch_q_packed_t<192, 128>(tq, tk, tv, tdo, p, early, stream);
  return -2;
}

}  // namespace sdpa
