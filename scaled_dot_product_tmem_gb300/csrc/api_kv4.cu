// api_kv4.cu -- the C ABI of the 4-bit paged key/value cache: argument checks and launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <new>
#include <vector>

#include "../../include/sdpa_tmem.h"
#include "attn_kernels.h"

namespace {

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

bool supported(int page_size, int d) {
  return (page_size == 16 || page_size == 32 || page_size == 64 || page_size == 128) && (d == 64 || d == 128);
}

int log2_of(int page_size) {
  int n = 0;
  while ((1 << n) < page_size) ++n;
  return n;
}

// Sizes shared by the calls that walk a page table.
int check_sizes(int B, int H_kv, int d, int n_pages, int page_size, int max_pages) {
  if (B < 0 || H_kv <= 0 || n_pages < 0 || max_pages < 0) return ATTN_ERR_INVALID_ARG;
  if (!supported(page_size, d) || H_kv > 65535) return ATTN_ERR_UNSUPPORTED;
  if ((long long)max_pages * page_size > 0x7fffffffLL) return ATTN_ERR_UNSUPPORTED;  // token numbers are int32
  return ATTN_OK;
}

template <class F>
int launch(const char* what, int n, cudaStream_t s, F f) {
  const int rc = sdpa::timed_launch(
      ATTN_KERNEL_KV4, n, s, [](void* ctx) { return (*static_cast<F*>(ctx))(); }, &f);
  if (rc == 0) return ATTN_OK;
  if (rc == -2) return ATTN_ERR_UNSUPPORTED;
  sdpa::set_last_error(what, cudaGetLastError());
  return ATTN_ERR_CUDA;
}

}  // namespace

extern "C" {

int attn_kv4_block_bytes(int page_size, int d) {
  return supported(page_size, d) ? sdpa::kv4_block_bytes(page_size, d) : 0;
}

int attn_kv4_append(const void* k, const void* v, const int* cu_seqlens, void* pool, const int* page_table,
                    const int* seq_lens, int B, int T, int H_kv, int d, int n_pages, int page_size, int max_pages,
                    long long k_row_stride, long long v_row_stride, void* stream) {
  const int st = check_sizes(B, H_kv, d, n_pages, page_size, max_pages);
  if (st != ATTN_OK) return st;
  if (T < 0 || k_row_stride < (long long)H_kv * d || v_row_stride < (long long)H_kv * d) return ATTN_ERR_INVALID_ARG;
  if (B == 0 || T == 0) return ATTN_OK;
  if (!k || !v || !cu_seqlens || !pool || !page_table || !seq_lens) return ATTN_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(pool, 16) || k_row_stride % 8 || v_row_stride % 8 ||
      !aligned(cu_seqlens, 4) || !aligned(page_table, 4) || !aligned(seq_lens, 4))
    return ATTN_ERR_MISALIGNED;
  sdpa::Kv4StoreParams p;
  p.c = {page_table, n_pages, page_size, max_pages, H_kv, d, log2_of(page_size)};
  p.B = B;
  p.T = T;
  p.cu = cu_seqlens;
  p.start = seq_lens;
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.k_stride = k_row_stride;
  p.v_stride = v_row_stride;
  p.pool = static_cast<uint8_t*>(pool);
  p.page_err = sdpa::device_page_error_word();
  p.site = ATTN_KV4_SITE_APPEND;
  if (!p.page_err) return ATTN_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return launch("kv4 append launch", 1, s, [&] { return sdpa::launch_kv4_append(p, s); });
}

int attn_kv4_append_rope(const void* q, const void* k, const void* v, const float* table, void* q_out, const int* cu_seqlens,
                         void* pool, const int* page_table, const int* seq_lens, int B, int T, int H_q, int H_kv, int d,
                         int n_pages, int page_size, int max_pages, int n, int first_dim, long long q_row_stride,
                         long long k_row_stride, long long v_row_stride, long long q_out_row_stride, int interleaved,
                         void* stream) {
  int st = check_sizes(B, H_kv, d, n_pages, page_size, max_pages);
  if (st != ATTN_OK) return st;
  sdpa::RopeParams rp;
  st = sdpa::rope_params(&rp, q, nullptr, table, q_out, nullptr, T, H_q, 0, d, n, first_dim, T, q_row_stride, 0,
                         q_out_row_stride, 0, 0);
  if (st != ATTN_OK) return st;
  if (k_row_stride < (long long)H_kv * d || v_row_stride < (long long)H_kv * d) return ATTN_ERR_INVALID_ARG;
  if (T == 0 || (B == 0 && H_q == 0)) return ATTN_OK;
  if (!table || (B > 0 && (!k || !v || !cu_seqlens || !pool || !page_table || !seq_lens))) return ATTN_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(pool, 16) || k_row_stride % 8 || v_row_stride % 8 ||
      !aligned(cu_seqlens, 4) || !aligned(page_table, 4) || !aligned(seq_lens, 4) || !aligned(table, 16))
    return ATTN_ERR_MISALIGNED;
  sdpa::Kv4StoreParams p;
  p.c = {page_table, n_pages, page_size, max_pages, H_kv, d, log2_of(page_size)};
  p.B = B;
  p.T = T;
  p.cu = cu_seqlens;
  p.start = seq_lens;
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.k_stride = k_row_stride;
  p.v_stride = v_row_stride;
  p.pool = static_cast<uint8_t*>(pool);
  p.page_err = sdpa::device_page_error_word();
  p.site = ATTN_KV4_SITE_APPEND;
  if (!p.page_err) return ATTN_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return launch("kv4 append with rotation launch", 1, s,
                [&] { return sdpa::launch_kv4_append_rope(p, rp, interleaved != 0, s); });
}

int attn_kv4_gather(const void* pool, const int* page_table, const int* cu_seqlens, const int* seq_lens, void* k,
                    void* v, int B, int T, int H_kv, int d, int n_pages, int page_size, int max_pages, int zero_rest,
                    void* stream) {
  const int st = check_sizes(B, H_kv, d, n_pages, page_size, max_pages);
  if (st != ATTN_OK) return st;
  if (T < 0) return ATTN_ERR_INVALID_ARG;
  if (T == 0 || (B == 0 && !zero_rest)) return ATTN_OK;
  if (!k || !v || !cu_seqlens || (B > 0 && (!pool || !page_table || !seq_lens))) return ATTN_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(pool, 16) || !aligned(cu_seqlens, 4) ||
      !aligned(page_table, 4) || !aligned(seq_lens, 4))
    return ATTN_ERR_MISALIGNED;
  sdpa::Kv4StoreParams p;
  p.c = {page_table, n_pages, page_size, max_pages, H_kv, d, log2_of(page_size)};
  p.B = B;
  p.T = T;
  p.cu = cu_seqlens;
  p.start = seq_lens;
  p.k_out = static_cast<__nv_bfloat16*>(k);
  p.v_out = static_cast<__nv_bfloat16*>(v);
  p.zero_rest = zero_rest != 0;
  p.pool = static_cast<uint8_t*>(const_cast<void*>(pool));
  p.page_err = sdpa::device_page_error_word();
  p.site = ATTN_KV4_SITE_GATHER;
  if (!p.page_err) return ATTN_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return launch("kv4 gather launch", 1, s, [&] { return sdpa::launch_kv4_gather(p, s); });
}

size_t attn_kv4_decode_workspace_size(int B, int S_q, int H_q, int H_kv, int d) {
  if (B < 0 || S_q < 0 || H_q <= 0 || H_kv <= 0 || H_q % H_kv != 0 || (d != 64 && d != 128)) return 0;
  return sdpa::kv4_decode_workspace(B, S_q, H_q, H_kv, d);
}

int attn_kv4_decode(const void* q, const void* pool, const int* page_table, const int* seq_lens, void* o, float* lse,
                    int B, int S_q, int H_q, int H_kv, int d, int n_pages, int page_size, int max_pages, float scale,
                    int window, int softmax_type, const float* softmax_offset, void* workspace,
                    size_t workspace_bytes, void* stream) {
  int st = check_sizes(B, H_kv, d, n_pages, page_size, max_pages);
  if (st != ATTN_OK) return st;
  // (the causal flag: a window is always allowed here)
  st = sdpa::check_common(B, S_q, 0, H_q, H_kv, d, d, 1, window, softmax_type, softmax_offset);
  if (st != ATTN_OK) return st;
  if ((long long)B * S_q * H_q > 0x7fffffffLL) return ATTN_ERR_UNSUPPORTED;
  // (the kernel multiplies scores held as 2^-23 of their value by scale 2^23 log2(e))
  if (sdpa::resolve_scale(scale, d) > 1e30f) return ATTN_ERR_UNSUPPORTED;
  if (B == 0 || S_q == 0) return ATTN_OK;
  if (!q || !o || !seq_lens || (max_pages > 0 && (!pool || !page_table))) return ATTN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(pool, 16) || !aligned(lse, 4) || !aligned(page_table, 4) ||
      !aligned(seq_lens, 4) || !aligned(softmax_offset, 4))
    return ATTN_ERR_MISALIGNED;
  if (!workspace || !aligned(workspace, 256) ||
      workspace_bytes < sdpa::kv4_decode_workspace(B, S_q, H_q, H_kv, d))
    return ATTN_ERR_WORKSPACE;
  sdpa::Kv4DecodeParams p;
  p.c = {page_table, n_pages, page_size, max_pages, H_kv, d, log2_of(page_size)};
  p.B = B;
  p.S_q = S_q;
  p.H_q = H_q;
  p.scale_log2 = sdpa::resolve_scale(scale, d) * 1.4426950408889634f;
  // a window of the whole table and more is none (and its arithmetic could pass 32 bits)
  p.window = window < 0 || window >= (long long)max_pages * page_size ? -1 : window;
  p.softmax_type = softmax_type;
  p.offset = softmax_offset;
  p.seq_lens = seq_lens;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.pool = static_cast<const uint8_t*>(pool);
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.err = sdpa::device_error_word();
  p.page_err = sdpa::device_page_error_word();
  p.site = ATTN_KV4_SITE_DECODE;
  if (!p.err || !p.page_err) return ATTN_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return launch("kv4 decode launch", 2, s, [&] { return sdpa::launch_kv4_decode(p, workspace, s); });
}

size_t attn_kv4_tree_workspace_size(int B, int T, int H_q, int H_kv, int d) {
  if (B < 0 || T < 0 || H_q <= 0 || H_kv <= 0 || H_q % H_kv != 0 || (d != 64 && d != 128)) return 0;
  return sdpa::kv4_tree_workspace(B, T, H_q, H_kv, d);
}

int attn_kv4_tree(const void* q, const int* cu_seqlens, const int* parents, const void* pool, const int* page_table,
                  const int* seq_lens, void* o, float* lse, int B, int T, int H_q, int H_kv, int d, int n_pages,
                  int page_size, int max_pages, float scale, int window, int softmax_type, const float* softmax_offset,
                  int zero_rest, void* workspace, size_t workspace_bytes, void* stream) {
  int st = check_sizes(B, H_kv, d, n_pages, page_size, max_pages);
  if (st != ATTN_OK) return st;
  st = sdpa::check_common(1, T, 0, H_q, H_kv, d, d, 1, window, softmax_type, softmax_offset);
  if (st != ATTN_OK) return st;
  if ((long long)T * H_q > 0x7fffffffLL || H_q / H_kv > 65535) return ATTN_ERR_UNSUPPORTED;
  // (the kernel multiplies scores held as 2^-23 of their value by scale 2^23 log2(e))
  if (sdpa::resolve_scale(scale, d) > 1e30f) return ATTN_ERR_UNSUPPORTED;
  if (T == 0 || (B == 0 && !zero_rest)) return ATTN_OK;
  if (!q || !o || !cu_seqlens || (B > 0 && !seq_lens) || (B > 0 && max_pages > 0 && (!pool || !page_table)))
    return ATTN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(pool, 16) || !aligned(lse, 4) || !aligned(page_table, 4) ||
      !aligned(seq_lens, 4) || !aligned(cu_seqlens, 4) || !aligned(parents, 4) || !aligned(softmax_offset, 4))
    return ATTN_ERR_MISALIGNED;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < sdpa::kv4_tree_workspace(B, T, H_q, H_kv, d))
    return ATTN_ERR_WORKSPACE;
  sdpa::Kv4TreeParams p;
  p.c = {page_table, n_pages, page_size, max_pages, H_kv, d, log2_of(page_size)};
  p.B = B;
  p.T = T;
  p.H_q = H_q;
  p.scale_log2 = sdpa::resolve_scale(scale, d) * 1.4426950408889634f;
  p.window = window < 0 ? -1 : window;
  p.softmax_type = softmax_type;
  p.offset = softmax_offset;
  p.cu = cu_seqlens;
  p.start = seq_lens;
  p.parents = parents;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.pool = static_cast<const uint8_t*>(pool);
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.zero_rest = zero_rest != 0;
  p.err = sdpa::device_error_word();
  p.page_err = sdpa::device_page_error_word();
  p.site = ATTN_KV4_SITE_TREE;
  if (!p.err || !p.page_err) return ATTN_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return launch("kv4 tree launch", 2, s, [&] { return sdpa::launch_kv4_tree(p, workspace, s); });
}

int attn_kv4_keep(void* pool, const int* page_table, const int* seq_lens, const int* kept, int B, int most, int n_layers,
                  int H_kv, int d, int n_pages, int page_size, int max_pages, void* stream) {
  const int st = check_sizes(B, H_kv, d, n_pages, page_size, max_pages);
  if (st != ATTN_OK) return st;
  if (most < 0 || n_layers < 0) return ATTN_ERR_INVALID_ARG;
  if (B == 0 || most == 0 || n_layers == 0) return ATTN_OK;
  if (B > 65535 || n_layers > 65535) return ATTN_ERR_UNSUPPORTED;
  if (!pool || !page_table || !seq_lens || !kept) return ATTN_ERR_INVALID_ARG;
  if (!aligned(pool, 16)) return ATTN_ERR_MISALIGNED;
  if (!aligned(page_table, 4) || !aligned(seq_lens, 4) || !aligned(kept, 4)) return ATTN_ERR_MISALIGNED;
  sdpa::Kv4KeepParams p;
  p.c = {page_table, n_pages, page_size, max_pages, H_kv, d, log2_of(page_size)};
  p.B = B;
  p.most = most;
  p.start = seq_lens;
  p.kept = kept;
  p.pool = static_cast<uint8_t*>(pool);
  p.n_layers = n_layers;
  p.layer_bytes = (long long)n_pages * H_kv * sdpa::kv4_block_bytes(page_size, d);
  p.page_err = sdpa::device_page_error_word();
  p.site = ATTN_KV4_SITE_KEEP;
  if (!p.page_err) return ATTN_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return launch("kv4 keep launch", 1, s, [&] { return sdpa::launch_kv4_keep(p, s); });
}

int attn_kv4_copy_pages(void* pool, int n_layers, int n_pages, size_t page_bytes, const int* src, const int* dst,
                        int n, void* stream) {
  if (n_layers < 0 || n_pages < 0 || n < 0 || page_bytes % 16 != 0) return ATTN_ERR_INVALID_ARG;
  if (n == 0 || n_layers == 0 || page_bytes == 0) return ATTN_OK;
  if (!pool || !src || !dst) return ATTN_ERR_INVALID_ARG;
  if (!aligned(pool, 16)) return ATTN_ERR_MISALIGNED;
  if (n_layers > 65535) return ATTN_ERR_UNSUPPORTED;
  for (int i = 0; i < n; ++i)
    if (src[i] < 0 || src[i] >= n_pages || dst[i] < 0 || dst[i] >= n_pages) return ATTN_ERR_INVALID_ARG;
  try {
    if (n_pages <= (1 << 20)) {  // what every page is used as
      std::vector<unsigned char> use(n_pages, 0);
      for (int i = 0; i < n; ++i) use[src[i]] = 1;
      for (int i = 0; i < n; ++i) {
        if (use[dst[i]]) return ATTN_ERR_INVALID_ARG;  // a source, or a destination already
        use[dst[i]] = 1;
      }
    } else {
      std::vector<int> from(src, src + n), to(dst, dst + n);
      std::sort(from.begin(), from.end());
      std::sort(to.begin(), to.end());
      if (std::adjacent_find(to.begin(), to.end()) != to.end()) return ATTN_ERR_INVALID_ARG;
      for (int page : to)
        if (std::binary_search(from.begin(), from.end(), page)) return ATTN_ERR_INVALID_ARG;
    }
  } catch (const std::bad_alloc&) {
    sdpa::set_last_error("kv4 page copy: host memory for the check", cudaErrorMemoryAllocation);
    return ATTN_ERR_CUDA;
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return launch("kv4 page copy launch", (n + sdpa::kKv4PairsMax - 1) / sdpa::kKv4PairsMax, s, [&] {
    return sdpa::launch_kv4_copy(static_cast<uint8_t*>(pool), n_layers, (long long)n_pages * (long long)page_bytes,
                                 (long long)page_bytes, src, dst, n, s);
  });
}

}  // extern "C"
