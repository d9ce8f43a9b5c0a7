// kv4_decode.cu -- attention of a sequence's newest tokens over its 4-bit paged cache
// (layout and number format in kv4.cuh).
//
//   S_j = scale q.k_j over the keys j in [pos - window, pos], pos the query's own place in
//   the sequence (the S_q queries are its last S_q tokens); softmax with an optional sink
//   logit; o = P V; lse = log of the denominator.
//
// One warp takes one (sequence, query, head): lane l holds d/32 dims, a score is a
// warp-wide sum, and the running maximum and denominator are kept in fp32.
#include "attn_common.cuh"
#include "attn_kernels.h"
#include "kv4.cuh"
#include "ptx.cuh"

namespace sdpa {

template <int D>
__global__ void __launch_bounds__(128) kv4_decode_kernel(const Kv4DecodeParams p) {
  constexpr int E = D / 32;  // dims of a lane
  const int lane = threadIdx.x % 32;
  const long long row = (long long)blockIdx.x * 4 + threadIdx.x / 32;
  if (row >= (long long)p.B * p.S_q * p.H_q) return;
  const int h = (int)(row % p.H_q), s = (int)(row / p.H_q % p.S_q), b = (int)(row / p.H_q / p.S_q);
  const int hk = h / (p.H_q / p.c.H_kv), P = p.c.page_size, x0 = lane * E;
  const int len = entry_len(p.seq_lens, b, p.c.max_pages * P);
  const int pos = len - p.S_q + s;
  const int lo = p.window >= 0 && pos > p.window ? pos - p.window : 0;
  float q[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = __bfloat162float(p.q[(size_t)row * D + x0 + e]) * p.scale_log2;
    o[e] = 0.f;
  }
  if (p.softmax_type == 1) { m = 0.f; l = 1.f; }
  if (p.softmax_type == 2) { m = p.offset[h] * kLog2e; l = 1.f; }
  for (int j = lo; j <= pos; ++j) {
    const int pg = kv4_page(p.c, b, j), w = j % P;
    float k[E], v[E];
    if (pg < 0 && lane == 0) atomicCAS(p.page_err, 0, p.site);
    const uint8_t* base = p.pool + ((size_t)max(pg, 0) * p.c.H_kv + hk) * kv4_block_bytes(P, D);
    const float sk = pg < 0 ? 0.f : kv4_scale_value(base[kv4_off_sk(P, D) + w * (D / 16) + x0 / 16]);
    const float sv =
        pg < 0 ? 0.f : kv4_scale_value(base[kv4_off_sv(P, D) + (w >> 1) * (D / 8) + (x0 / 16) * 2 + (w & 1)]);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int x = x0 + e;
      const int ck = pg < 0 ? 8 : (base[w * (D / 2) + x / 2] >> (4 * (x & 1))) & 15;
      const int cv = pg < 0 ? 8
                            : (base[kv4_off_v(P, D) + kv4_v_at(w, x / (D / 8), D) + (x % (D / 8)) / 2] >>
                               (4 * (x & 1))) & 15;
      k[e] = (float)(ck - 8) * sk;
      v[e] = (float)(cv - 8) * sv;
    }
    float t = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) t = fmaf(q[e], k[e], t);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
    const float mn = fmaxf(m, t);
    const float ms = mn == -INFINITY ? 0.f : mn;
    const float a = ex2(m - ms), pr = ex2(t - ms);
    l = l * a + pr;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * a + pr * v[e];
    m = mn;
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) p.o[(size_t)row * D + x0 + e] = __float2bfloat16(o[e] * inv);
  if (lane == 0 && p.lse)
    p.lse[((size_t)b * p.H_q + h) * p.S_q + s] = l > 0.f ? ((m == -INFINITY ? 0.f : m) + lg2(l)) * kLn2 : -INFINITY;
}

size_t kv4_decode_workspace(int B, int S_q, int H_q, int H_kv, int d) { return 256; }

int launch_kv4_decode(const Kv4DecodeParams& p, void* workspace, cudaStream_t stream) {
  const long long rows = (long long)p.B * p.S_q * p.H_q;
  const unsigned blocks = (unsigned)((rows + 3) / 4);
  if (p.c.d == 128) kv4_decode_kernel<128><<<blocks, 128, 0, stream>>>(p);
  else kv4_decode_kernel<64><<<blocks, 128, 0, stream>>>(p);
  return cudaPeekAtLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace sdpa
