// attn_packed.cu -- attention over packed sequences: the plan kernel that lists the work tiles
// (a small forward does without: find_own_tile in attn_common.cuh),
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
//             tiles from a counter, and with falling costs they end together;
//   kv and q  whole sequences by length, a sequence's heaviest tiles first: the tiles in
//             flight belong to few sequences, whose other operand they share in L2.
// The order inside a bucket varies from run to run; no result depends on it.
// Measured: about 4 us for 4 to 16 sequences (6.5 with 1024 threads and offsets in global memory),
// most of it hidden behind the set-up of the kernel that follows.
// =============================================================================
// Latency is all that counts here (a few thousand numbers), so the block has 256 threads where
// the sequences allow it (cheaper barriers), the offsets stay in shared memory, and the two lists
// of a backward share their barriers.
constexpr int kPlanSeqs = 1024;  // sequences whose offsets fit in shared memory

namespace {

enum PlanKind { kPlanFwd, kPlanKv, kPlanQ };

template <int KIND>
constexpr int plan_rows() { return KIND == kPlanFwd ? 256 : 128; }

// f(sequence b, its four numbers, its tiles n, first tile, step between tiles) for every sequence
// with tiles: those of up to 8 tiles by one thread each, longer ones by the warp.
template <int KIND, int NT, class F>
__device__ __forceinline__ void plan_walk(int B, const int* cq, const int* ck, F f) {
  constexpr int ROWS = plan_rows<KIND>();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  for (int b0 = warp * 32; b0 < B; b0 += NT) {
    const int b = b0 + lane;
    int q0 = 0, Lq = 0, k0 = 0, Lk = 0;
    if (b < B) {
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
}

// The bucket of tile j of a sequence of n tiles: the kv tiles it sees (forward), or n.
template <int KIND, int NT>
__device__ __forceinline__ int plan_bucket(const PackedPlanParams& p, int Lq, int Lk, int n, int j) {
  int w = n;
  if constexpr (KIND == kPlanFwd) {
    int lo = 1, hi = 0;
    w = kv_tile_range(MaskSpec{Lq, Lk, p.causal, p.window}, j * 256, j * 256 + 255, 128, &lo, &hi) ? hi - lo + 1 : 0;
  }
  return min(w, NT - 1);
}

template <int KIND, int NT>
__device__ __forceinline__ void plan_count(const PackedPlanParams& p, const int* cq, const int* ck, int* hist) {
  plan_walk<KIND, NT>(p.B, cq, ck, [&](int, int, int Lq, int, int Lk, int n, int j0, int step) {
    if constexpr (KIND == kPlanFwd) {
      for (int j = j0; j < n; j += step) atomicAdd(&hist[plan_bucket<KIND, NT>(p, Lq, Lk, n, j)], 1);
    } else if (j0 == 0) {
      atomicAdd(&hist[plan_bucket<KIND, NT>(p, Lq, Lk, n, 0)], n);
    }
  });
}

template <int KIND, int NT>
__device__ __forceinline__ void plan_place(const PackedPlanParams& p, const int* cq, const int* ck, int* next,
                                           PackedTile* out) {
  plan_walk<KIND, NT>(p.B, cq, ck, [&](int b, int q0, int Lq, int k0, int Lk, int n, int j0, int step) {
    int base = 0;
    if constexpr (KIND != kPlanFwd) {
      if (j0 == 0) base = atomicAdd(&next[plan_bucket<KIND, NT>(p, Lq, Lk, n, 0)], n);
      if (step == 32) base = __shfl_sync(0xffffffffu, base, 0);
    }
    for (int j = j0; j < n; j += step) {
      int at, tile = j;
      if constexpr (KIND == kPlanFwd) {
        at = atomicAdd(&next[plan_bucket<KIND, NT>(p, Lq, Lk, n, j)], 1);
      } else {
        at = base + j;
        if (KIND == kPlanQ && p.causal) tile = n - 1 - j;  // under a causal mask the last query tile sees most
      }
      int4* e = reinterpret_cast<int4*>(out + at);
      e[0] = make_int4(q0, Lq, k0, Lk);
      e[1] = make_int4(b, tile * plan_rows<KIND>(), (int)(((long long)q0 + 128LL * b) / 128 * 128), 0);
    }
  });
}

template <int NT, bool BWD>
__global__ void __launch_bounds__(NT) packed_plan_kernel(const PackedPlanParams p) {
  __shared__ int hist[2][NT], part[2][NT / 32], sq[kPlanSeqs + 1], sk[kPlanSeqs + 1];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  grid_launch_dependents();
  const bool same = p.cu_kv == p.cu_q && p.T_kv == p.T_q, small = p.B <= kPlanSeqs;
  int* cq = small ? sq : p.clean_q;
  int* ck = same ? cq : (small ? sk : p.clean_kv);
  hist[0][threadIdx.x] = hist[1][threadIdx.x] = 0;
  // the running maxima of the clamped offsets
  int carry_q = 0, carry_k = 0;
  for (int base = 0; base <= p.B; base += NT) {
    const int i = base + threadIdx.x;
    int q = i <= p.B ? min(max(__ldg(p.cu_q + i), 0), p.T_q) : 0;
    int k = i <= p.B && !same ? min(max(__ldg(p.cu_kv + i), 0), p.T_kv) : 0;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {  // (below `off` a lane gets its own value)
      q = max(q, __shfl_up_sync(0xffffffffu, q, off));
      k = max(k, __shfl_up_sync(0xffffffffu, k, off));
    }
    if (lane == 31) {
      part[0][warp] = q;
      part[1][warp] = k;
    }
    __syncthreads();
    int top_q = carry_q, top_k = carry_k;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
      if (w == warp) {
        q = max(q, top_q);
        k = max(k, top_k);
      }
      top_q = max(top_q, part[0][w]);
      top_k = max(top_k, part[1][w]);
    }
    carry_q = top_q;
    carry_k = top_k;
    if (i <= p.B) {
      cq[i] = q;
      if (!same) ck[i] = k;
    }
    __syncthreads();
  }
  constexpr int A = BWD ? kPlanKv : kPlanFwd;
  PackedTile* list_a = BWD ? p.tiles_kv : p.tiles_fwd;
  plan_count<A, NT>(p, cq, ck, hist[0]);
  if constexpr (BWD) plan_count<kPlanQ, NT>(p, cq, ck, hist[1]);
  __syncthreads();
  // first entry of each bucket, the highest bucket first
  int sum[2], mine[2], total[2] = {0, 0};
#pragma unroll
  for (int l = 0; l < 2; ++l) {
    mine[l] = sum[l] = hist[l][NT - 1 - threadIdx.x];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, sum[l], off);
      if (lane >= off) sum[l] += o;
    }
    if (lane == 31) part[l][warp] = sum[l];
  }
  __syncthreads();
#pragma unroll
  for (int l = 0; l < 2; ++l) {
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
      if (w < warp) sum[l] += part[l][w];
      total[l] += part[l][w];
    }
    hist[l][NT - 1 - threadIdx.x] = sum[l] - mine[l];
  }
  __syncthreads();
  plan_place<A, NT>(p, cq, ck, hist[0], list_a);
  if constexpr (BWD) plan_place<kPlanQ, NT>(p, cq, ck, hist[1], p.tiles_q);
  if (threadIdx.x == 0) {
    PackedCounts c{};
    if (BWD) {
      c.kv_tiles = total[0];
      c.q_tiles = total[1];
    } else {
      c.fwd_tiles = total[0];
    }
    c.q_begin = cq[0];
    c.q_end = cq[p.B];
    c.kv_begin = ck[0];
    c.kv_end = ck[p.B];
    *p.counts = c;
  }
}

}  // namespace

int launch_packed_plan(const PackedPlanParams& p, cudaStream_t stream) {
  const bool bwd = p.tiles_fwd == nullptr;
  if (p.B < 256) {
    if (bwd) packed_plan_kernel<256, true><<<1, 256, 0, stream>>>(p);
    else packed_plan_kernel<256, false><<<1, 256, 0, stream>>>(p);
  } else {
    if (bwd) packed_plan_kernel<1024, true><<<1, 1024, 0, stream>>>(p);
    else packed_plan_kernel<1024, false><<<1, 1024, 0, stream>>>(p);
  }
  return cudaPeekAtLastError() == cudaSuccess ? 0 : -1;
}

// =============================================================================
// Forward
// =============================================================================
template <bool OWN>
static int launch_fwd_packed_t(int d_qk, int d_v, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                               const FwdParams& p, cudaStream_t stream) {
  if (d_qk == 128 && d_v == 128)
    return launch_fwd_t<128, 128, 2, 2, true, false, false, false, true, OWN>(tq, tk, tv, p, stream);
  if (d_qk == 64 && d_v == 64)
    return launch_fwd_t<64, 64, 4, 4, true, false, false, false, true, OWN>(tq, tk, tv, p, stream);
  if (d_qk == 192 && d_v == 128)
    return launch_fwd_t<192, 128, 2, 1, true, false, false, false, true, OWN>(tq, tk, tv, p, stream);
  return -2;
}

int launch_attn_fwd_packed(int d_qk, int d_v, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                           const FwdParams& p, cudaStream_t stream) {
  return p.tiles ? launch_fwd_packed_t<false>(d_qk, d_v, tq, tk, tv, p, stream)
                 : launch_fwd_packed_t<true>(d_qk, d_v, tq, tk, tv, p, stream);
}

// =============================================================================
// Backward preprocess: D = rowsum(dO * O) and -LSE log2(e) in the workspace's padded rows (the
// padding: D = 0, -inf), one block per 64 rows of a query tile and head; on request also
// zeros in the gradient rows of no sequence.
//
// D enters dS = P (dP - D) with the rounding of the stored bf16 O, 2^-8 |O|.  Against |dP| that
// falls with the number n of keys a row sees (O is a mean of n values), while the row's dS
// (P is about 1 / n) grows: rows that see few keys carry most of the error, and they are many in a
// batch of short sequences and all there are under a short window.  Rows that see at most
// kFewKeys keys therefore get D = sum_j P_ij (dO_i . v_j) from fp32 scores.  (Eight sequences of 1
// to 512 rows: dQ and dK off by 0.0026 of their norm from the stored O; the two roundings that
// stay, of dS and of the result, are 0.0024.  Under a window of 1 it would be 0.0035.  It costs 95
// us for 16,384 rows of 32 heads that are all such rows, under a window of 8, of 660 for forward
// and backward; 135 with a lane's pieces of a row side by side instead of the four lanes'.)
// =============================================================================
constexpr int kFewKeys = 32;

// d (16 x 8 fp32) += a (16 x 16 bf16, rows) b (16 x 8 bf16, columns)
__device__ __forceinline__ void mma_16816_acc(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Products of 16 rows of a (lane / 4 and lane / 4 + 8, null: zeros) with 16 rows of b: out[c][e + 2 f] is row
// lane / 4 + 8 f of a times row 8 c + 2 (lane % 4) + e of b.  Lane t of a row's
// four has every fourth 16-byte piece of it, so that the four read 64 bytes side by side; which dims
// share a step is free as long as both operands agree.
template <int N>
__device__ __forceinline__ void rows_product(const uint4* a0, const uint4* a1, const uint4* b0, const uint4* b1,
                                             float (&out)[2][4]) {
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int e = 0; e < 4; ++e) out[c][e] = 0.f;
#pragma unroll 1
  for (int x = 0; x < N / 32; ++x) {
    const uint4 p = a0 ? __ldg(a0 + 4 * x) : zero, q = a1 ? __ldg(a1 + 4 * x) : zero;
    const uint4 r[2] = {b0 ? __ldg(b0 + 4 * x) : zero, b1 ? __ldg(b1 + 4 * x) : zero};
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      mma_16816_acc(out[c], p.x, q.x, p.y, q.y, r[c].x, r[c].y);
      mma_16816_acc(out[c], p.z, q.z, p.w, q.w, r[c].z, r[c].w);
    }
  }
}

// The part of D that every second 16 keys from 16 `part` on give the 16 rows from r0 on, counted from the
// first key that one of them with few keys sees (they see keys among the 47 from there on, since
// first keys rise by at most one a row).  A warp; rows with more keys get nothing that is used.
template <int D_QK, int D_V>
__device__ __forceinline__ void few_keys_part(const BwdParams& p, const PackedTile& e, int h, int r0, int part,
                                              float* out) {
  const int lane = threadIdx.x % 32, t = lane % 4, hk = h / p.G;
  const MaskSpec m{e.Lq, e.Lk, p.causal, p.window};
  int lo[2], hi[2], first = 0x7fffff00, last = -1;
#pragma unroll
  for (int f = 0; f < 2; ++f) {
    visible_keys<true>(m, r0 + lane / 4 + 8 * f, &lo[f], &hi[f]);
    if (hi[f] - lo[f] >= kFewKeys) hi[f] = lo[f] - 1;  // not a row of few keys
    if (hi[f] >= lo[f]) {
      first = min(first, lo[f]);
      last = max(last, hi[f]);
    }
  }
  first = __reduce_min_sync(0xffffffffu, first);
  last = __reduce_max_sync(0xffffffffu, last);
  float d[2] = {0.f, 0.f};
#pragma unroll 1
  for (int k0 = first + 16 * part; k0 <= last; k0 += 32) {  // (no such row: first is past last)
    const int key = k0 + lane / 4;
    const uint4 *q[2], *g[2], *k[2], *v[2];
    float nl[2];
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      const int i = r0 + lane / 4 + 8 * f;
      const bool row = i < e.Lq, has = key + 8 * f < e.Lk;
      const size_t qr = (size_t)(e.q0 + (row ? i : 0)) * p.H_q + h;
      const size_t kr = (size_t)(e.k0 + (has ? key + 8 * f : 0)) * p.H_kv + hk;
      q[f] = row ? reinterpret_cast<const uint4*>(p.q + qr * D_QK) + t : nullptr;
      g[f] = row ? reinterpret_cast<const uint4*>(p.dout + qr * D_V) + t : nullptr;
      k[f] = has ? reinterpret_cast<const uint4*>(p.k + kr * D_QK) + t : nullptr;
      v[f] = has ? reinterpret_cast<const uint4*>(p.v + kr * D_V) + t : nullptr;
      const float l = row ? p.lse[(size_t)h * p.S_q + e.q0 + i] : 0.f;
      nl[f] = l == -INFINITY ? -INFINITY : -l * kLog2e;
    }
    float s[2][4], dp[2][4];
    rows_product<D_QK>(q[0], q[1], k[0], k[1], s);
    rows_product<D_V>(g[0], g[1], v[0], v[1], dp);
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int f = x / 2, j = k0 + 8 * c + 2 * t + x % 2;
        if (j >= lo[f] && j <= hi[f]) d[f] = fmaf(ex2(fmaf(s[c][x], p.scale_log2, nl[f])), dp[c][x], d[f]);
      }
  }
#pragma unroll
  for (int f = 0; f < 2; ++f)
#pragma unroll
    for (int off = 1; off < 4; off <<= 1) d[f] += __shfl_xor_sync(0xffffffffu, d[f], off);
  if (t == 0) {
    out[lane / 4] = d[0];
    out[lane / 4 + 8] = d[1];
  }
}

template <int D_QK, int D_V>
__global__ void __launch_bounds__(256, 5) packed_preprocess_kernel(const BwdParams p) {
  constexpr int TPR = D_V / 8, RPP = 256 / TPR, TILE = 64, NR = TILE / RPP;
  __shared__ float dsum[TILE], few_sum[2][TILE];
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
    // rows of few keys: the first of a sequence, all under a short window, and where keys are few or
    // end early
    const bool few = i0 < kFewKeys || (p.window >= 0 && (p.window < kFewKeys || i0 + TILE > e.Lk)) || e.Lk <= kFewKeys;
    if (few) {
      const int warp = threadIdx.x / 32;
      few_keys_part<D_QK, D_V>(p, e, h, i0 + warp / 2 * 16, warp % 2, &few_sum[warp % 2][warp / 2 * 16]);
    }
    __syncthreads();
    if (threadIdx.x < TILE) {
      const int i = i0 + threadIdx.x;
      const bool real = i < e.Lq;
      const size_t w = (size_t)h * p.S_pad + e.ws0 + i;
      int lo = 0, hi = -1;
      visible_keys<true>(MaskSpec{e.Lq, e.Lk, p.causal, p.window}, i, &lo, &hi);
      const bool exact = few && hi >= lo && hi - lo < kFewKeys;
      const float d = exact ? few_sum[0][threadIdx.x] + few_sum[1][threadIdx.x] : dsum[threadIdx.x];
      p.Dsum[w] = real ? d : 0.f;
      const float l = real ? p.lse[(size_t)h * p.S_q + e.q0 + i] : -INFINITY;
      p.nlse2[w] = l == -INFINITY ? -INFINITY : -l * kLog2e;
    }
  }
  if (p.zero_rest) {
    const size_t at = ((size_t)blockIdx.y * gridDim.x + blockIdx.x) * 256 + threadIdx.x;
    const size_t step = (size_t)gridDim.x * gridDim.y * 256;
    const uint4 z = make_uint4(0u, 0u, 0u, 0u);
    auto clear = [&](__nv_bfloat16* x, int from, int to, int H, int d) {
      uint4* x16 = reinterpret_cast<uint4*>(x + (size_t)from * H * d);
      const size_t n = (size_t)(to - from) * H * (d / 8);
      for (size_t i = at; i < n; i += step) x16[i] = z;
    };
    const PackedCounts c = *p.counts;
    clear(p.dq, 0, c.q_begin, p.H_q, D_QK);
    clear(p.dq, c.q_end, p.S_q, p.H_q, D_QK);
    clear(p.dk, 0, c.kv_begin, p.H_kv, D_QK);
    clear(p.dk, c.kv_end, p.S_kv, p.H_kv, D_QK);
    clear(p.dv, 0, c.kv_begin, p.H_kv, D_V);
    clear(p.dv, c.kv_end, p.S_kv, p.H_kv, D_V);
  }
}

int launch_packed_preprocess(int d_qk, int d_v, const BwdParams& p, cudaStream_t stream) {
  if (2 * p.tile_bound_q > 0x7fffffffLL) return -2;
  const dim3 grid((unsigned)(2 * p.tile_bound_q), p.H_q);
  if (d_qk == 64 && d_v == 64) return launch_kernel(packed_preprocess_kernel<64, 64>, grid, 256, 0, stream, true, p);
  if (d_qk == 128 && d_v == 128) return launch_kernel(packed_preprocess_kernel<128, 128>, grid, 256, 0, stream, true, p);
  if (d_qk == 192 && d_v == 128) return launch_kernel(packed_preprocess_kernel<192, 128>, grid, 256, 0, stream, true, p);
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
  const size_t n4 = (size_t)counts->kv_end * row4, t0 = (size_t)counts->kv_begin * row4;
  for (size_t t = t0 + (size_t)blockIdx.x * 256 + threadIdx.x; t < n4; t += (size_t)gridDim.x * 256) {
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
  constexpr auto kern = attn_bwd_kv_kernel<192, 128, false, true, false, false, false, true>;
  if (!allow_smem<kern>(C::SMEM)) return -1;
  return launch_kernel(kern, dim3((unsigned)grid), C::THREADS, C::SMEM, stream, true, tq64, tk, tv, tdo64, tq64, tq64, p);
}

template <int D_QK, int D_V>
static int launch_q_packed_t(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                             const CUtensorMap& tdo, const BwdParams& p, bool early, cudaStream_t stream) {
  using C = QCfg<D_QK, D_V>;
  const long long grid = p.tile_bound_q * p.H_q;
  if (grid <= 0 || grid > 0x7fffffffLL) return -2;
  constexpr auto plain = attn_bwd_q_kernel<D_QK, D_V, true, false, false, false, true, false>;
  constexpr auto sums = attn_bwd_q_kernel<D_QK, D_V, true, false, false, false, true, true>;
  const auto kern = p.ds_rowsum ? sums : plain;
  if (!(p.ds_rowsum ? allow_smem<sums>(C::SMEM) : allow_smem<plain>(C::SMEM))) return -1;
  return launch_kernel(kern, dim3((unsigned)grid), C::THREADS, C::SMEM, stream, early, tq, tk, tv, tdo, p);
}

// early: right behind the kv kernel on the stream, in whose tail it is set up.
int launch_bwd_q_packed(int d_qk, int d_v, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                        const CUtensorMap& tdo, const BwdParams& p, bool early, cudaStream_t stream) {
  if (d_qk == 128 && d_v == 128) return launch_q_packed_t<128, 128>(tq, tk, tv, tdo, p, early, stream);
  if (d_qk == 64 && d_v == 64) return launch_q_packed_t<64, 64>(tq, tk, tv, tdo, p, early, stream);
  if (d_qk == 192 && d_v == 128) return launch_q_packed_t<192, 128>(tq, tk, tv, tdo, p, early, stream);
  return -2;
}

}  // namespace sdpa
