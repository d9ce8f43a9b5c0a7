// kv4_tree.cu -- attention of the nodes of drafted trees over a sequence's 4-bit paged cache.
#include "attn_kernels.h"
#include "kv4.cuh"
#include "ptx.cuh"

namespace sdpa {

namespace {

__device__ __forceinline__ float kv4_code_value(const uint8_t* code, int odd, const uint8_t* scale) {
  return (float)((int)((*code >> (4 * odd)) & 15) - 8) * kv4_scale_value(*scale);
}

}  // namespace

// One warp a node and head, one token a step.
template <int D>
__global__ void __launch_bounds__(128) kv4_tree_kernel(const Kv4TreeParams p) {
  const int lane = threadIdx.x % 32;
  const long long row = (long long)blockIdx.x * 4 + threadIdx.x / 32;
  if (row >= (long long)p.T * p.H_q) return;
  const int t = (int)(row / p.H_q), h = (int)(row % p.H_q), hk = h / (p.H_q / p.c.H_kv);
  int b = -1;
  for (int i = 0; i < p.B; ++i)
    if (p.cu[i] <= t && t < p.cu[i + 1]) b = i;
  __nv_bfloat16* o = p.o + ((size_t)t * p.H_q + h) * D;
  if (b < 0) {
    if (p.zero_rest) {
      for (int x = lane; x < D; x += 32) o[x] = __float2bfloat16(0.f);
      if (lane == 0 && p.lse) p.lse[(size_t)h * p.T + t] = -INFINITY;
    }
    return;
  }
  const int P = p.c.page_size, blk = kv4_block_bytes(P, D), first = p.cu[b], node = t - first;
  const long long cap = (long long)p.c.max_pages * P;
  const int L = entry_len(p.start, b, (int)cap);
  auto parent_of = [&](int i) {
    if (!p.parents) return i - 1;
    const int a = p.parents[first + i];
    return a < i && a >= 0 ? a : -1;
  };
  int depth = 0;
  for (int a = parent_of(node); a >= 0; a = parent_of(a)) ++depth;
  constexpr int E = D / 32;
  float q[E], acc[E], m = -INFINITY, l = 0.f;
  for (int e = 0; e < E; ++e) {
    q[e] = __bfloat162float(p.q[((size_t)t * p.H_q + h) * D + lane * E + e]);
    acc[e] = 0.f;
  }
  auto token = [&](long long j) {
    if (j >= cap) return;
    const int pg = kv4_page(p.c, b, (int)j);
    float k[E], v[E], s = 0.f;
    for (int e = 0; e < E; ++e) k[e] = v[e] = 0.f;
    if (pg < 0) {
      atomicCAS(p.page_err, 0, p.site);
    } else {
      const uint8_t* base = p.pool + ((size_t)pg * p.c.H_kv + hk) * blk;
      const int w = (int)j & (P - 1);
      for (int e = 0; e < E; ++e) {
        const int x = lane * E + e, g = x / (D / 8);
        k[e] = kv4_code_value(base + w * (D / 2) + x / 2, x & 1, base + kv4_off_sk(P, D) + w * (D / 16) + x / 16);
        v[e] = kv4_code_value(base + kv4_off_v(P, D) + kv4_v_at(w, g, D) + x % (D / 8) / 2, x & 1,
                              base + kv4_off_sv(P, D) + (w >> 1) * (D / 8) + x / 16 * 2 + (w & 1));
      }
    }
    for (int e = 0; e < E; ++e) s = fmaf(q[e], k[e], s);
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    s *= p.scale_log2;
    const float mn = fmaxf(m, s), f = m == -INFINITY ? 0.f : exp2f(m - mn), w = exp2f(s - mn);
    l = l * f + w;
    for (int e = 0; e < E; ++e) acc[e] = acc[e] * f + w * v[e];
    m = mn;
  };
  const long long lo = p.window >= 0 ? max(0LL, (long long)L + depth - p.window) : 0;
  for (long long j = lo; j < L; ++j) token(j);
  int step = 0;
  for (int a = node; a >= 0 && (p.window < 0 || step <= p.window); a = parent_of(a), ++step) token((long long)L + a);
  const float sink = p.softmax_type == 0 ? -INFINITY : p.softmax_type == 1 ? 0.f : p.offset[h] * kLog2e;
  const float mm = fmaxf(m, sink), f = m == -INFINITY ? 0.f : exp2f(m - mm);
  const float den = mm == -INFINITY ? 0.f : l * f + (sink == -INFINITY ? 0.f : exp2f(sink - mm));
  for (int e = 0; e < E; ++e) o[lane * E + e] = __float2bfloat16(mm == -INFINITY ? acc[e] : acc[e] * (f / den));
  if (lane == 0 && p.lse) p.lse[(size_t)h * p.T + t] = mm == -INFINITY ? (l == l ? -INFINITY : l) : (mm + log2f(den)) * kLn2;
}

size_t kv4_tree_workspace(int, int, int, int, int) { return 256; }

int launch_kv4_tree(const Kv4TreeParams& p, void*, cudaStream_t stream) {
  const long long blocks = ((long long)p.T * p.H_q + 3) / 4;
  if (blocks > 0x7fffffffLL) return -2;
  if (p.c.d == 128) kv4_tree_kernel<128><<<(unsigned)blocks, 128, 0, stream>>>(p);
  else kv4_tree_kernel<64><<<(unsigned)blocks, 128, 0, stream>>>(p);
  return cudaPeekAtLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace sdpa
