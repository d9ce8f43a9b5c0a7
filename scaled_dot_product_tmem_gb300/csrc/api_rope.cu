// api_rope.cu -- the C ABI of the rotation by positions: argument checks and launches.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/sdpa_tmem.h"
#include "attn_kernels.h"

namespace {

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

template <class F>
int launch(const char* what, cudaStream_t s, F f) {
  const int rc = sdpa::timed_launch(
      ATTN_KERNEL_ROPE, 1, s, [](void* ctx) { return (*static_cast<F*>(ctx))(); }, &f);
  if (rc == 0) return ATTN_OK;
  if (rc == -2) return ATTN_ERR_UNSUPPORTED;
  sdpa::set_last_error(what, cudaGetLastError());
  return ATTN_ERR_CUDA;
}

}  // namespace

extern "C" {

int attn_rope_table(const double* inv_freq, const int* positions, float* table, int T, int n, float gain, void* stream) {
  if (T < 0 || n < 0 || !std::isfinite(gain)) return ATTN_ERR_INVALID_ARG;
  if (n == 0 || n % 8 != 0 || n > 128) return ATTN_ERR_UNSUPPORTED;
  if (T == 0) return ATTN_OK;
  if (!inv_freq || !positions || !table) return ATTN_ERR_INVALID_ARG;
  if (!aligned(inv_freq, 8) || !aligned(positions, 4) || !aligned(table, 16)) return ATTN_ERR_MISALIGNED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return launch("rope table launch", s, [&] { return sdpa::launch_rope_table(inv_freq, positions, table, T, n, gain, s); });
}

int attn_rope(const void* q, const void* k, const float* table, void* q_out, void* k_out, int T, int H_q, int H_k, int d,
              int n, int first_dim, int table_rows, long long q_stride, long long k_stride, long long q_out_stride,
              long long k_out_stride, int interleaved, int inverse, void* stream) {
  sdpa::RopeParams p;
  const int st = sdpa::rope_params(&p, q, k, table, q_out, k_out, T, H_q, H_k, d, n, first_dim, table_rows, q_stride,
                                   k_stride, q_out_stride, k_out_stride, inverse);
  if (st != ATTN_OK) return st;
  if (T == 0 || H_q + H_k == 0) return ATTN_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return launch("rope launch", s, [&] { return sdpa::launch_rope(p, interleaved != 0, s); });
}

}  // extern "C"

namespace sdpa {

int rope_params(RopeParams* p, const void* q, const void* k, const float* table, void* q_out, void* k_out, int T, int H_q,
                int H_k, int d, int n, int first_dim, int table_rows, long long q_stride, long long k_stride,
                long long q_out_stride, long long k_out_stride, int inverse) {
  if (T < 0 || H_q < 0 || H_k < 0 || d <= 0 || n < 0 || first_dim < 0 || table_rows < 0) return ATTN_ERR_INVALID_ARG;
  if (n == 0 || n % 8 != 0 || d % 8 != 0 || first_dim % 8 != 0 || d > 256) return ATTN_ERR_UNSUPPORTED;
  if (first_dim + 2LL * n > d) return ATTN_ERR_INVALID_ARG;
  if ((long long)H_q + H_k > 0x7ffffff0LL) return ATTN_ERR_UNSUPPORTED;
  const struct {
    const void* x;
    void* y;
    long long xs, ys;
    int H;
  } m[2] = {{q, q_out, q_stride, q_out_stride, H_q}, {k, k_out, k_stride, k_out_stride, H_k}};
  for (const auto& t : m) {
    if (t.H == 0 || T == 0) continue;
    if (!t.x || !t.y || t.xs < (long long)t.H * d || t.ys < (long long)t.H * d) return ATTN_ERR_INVALID_ARG;
    if (t.x == t.y && t.xs != t.ys) return ATTN_ERR_INVALID_ARG;  // in place: the same rows
    if (!aligned(t.x, 16) || !aligned(t.y, 16) || t.xs % 8 || t.ys % 8) return ATTN_ERR_MISALIGNED;
  }
  if (T > 0 && H_q + H_k > 0) {
    if (!table || table_rows == 0 || T % table_rows != 0) return ATTN_ERR_INVALID_ARG;
    if (!aligned(table, 16)) return ATTN_ERR_MISALIGNED;
  }
  auto heads = [](const void* x, void* y, long long xs, long long ys, int H) {
    RopeHeads h;
    h.x = static_cast<const __nv_bfloat16*>(x);
    h.y = static_cast<__nv_bfloat16*>(y);
    h.xs = xs;
    h.ys = ys;
    h.H = H;
    return h;
  };
  p->a = heads(q, q_out, q_stride, q_out_stride, H_q);
  p->b = heads(k, k_out, k_stride, k_out_stride, H_k);
  p->table = table;
  p->T = T;
  p->table_rows = table_rows;
  p->d = d;
  p->n = n;
  p->first = first_dim;
  p->inverse = inverse != 0;
  p->copies = 2 * n < d && ((H_q > 0 && q != q_out) || (H_k > 0 && k != k_out));
  return ATTN_OK;
}

}  // namespace sdpa
