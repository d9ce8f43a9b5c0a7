// api_packed.cu -- the C ABI of attention over packed sequences: argument checks, workspace
// carving, tensor maps and launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/sdpa_tmem.h"
#include "attn_packed.h"
#include "tmap.h"

namespace {

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

bool supported(int d_qk, int d_v) {
  return (d_qk == d_v && (d_qk == 64 || d_qk == 128)) || (d_qk == 192 && d_v == 128);
}

// At most this many tiles of `rows` rows in B sequences of T rows together.
long long tile_bound(int B, int T, int rows) { return (long long)T / rows + B; }

// A forward of at most this many work tiles (one wave of CTAs, so that their order does not matter)
// and kOwnSeqs sequences runs without a plan kernel: 8.5 us instead of 10.5 for 32 work tiles of
// 4 sequences.  With more tiles than CTAs the plan's order is worth its kernel: 8 documents of 208
// tiles took 26 us instead of 24 when every CTA listed and sorted them itself.
constexpr int kOwnCtas = 152;

struct Layout {
  size_t counts, clean_q, clean_kv, tiles_fwd, tiles_kv, tiles_q, nlse2, dsum, rowsum, dk_part, dv_part, total;
  int ns, S_pad;
};

Layout layout(int B, int T_q, int T_kv, int H_q, int H_kv, int d_qk, int d_v, bool bwd) {
  Layout w{};
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += round256(bytes);
    return o;
  };
  w.counts = take(sizeof(sdpa::PackedCounts));
  w.clean_q = take(sizeof(int) * ((size_t)B + 1));
  w.clean_kv = take(sizeof(int) * ((size_t)B + 1));
  if (!bwd) {
    w.tiles_fwd = take(sizeof(sdpa::PackedTile) * tile_bound(B, T_q, 256));
  } else {
    w.tiles_kv = take(sizeof(sdpa::PackedTile) * tile_bound(B, T_kv, 128));
    w.tiles_q = take(sizeof(sdpa::PackedTile) * tile_bound(B, T_q, 128));
    // sequence b starts at row (cu_q[b] + 128 b) rounded down to 128: its rows rounded up to 128
    // end at or before the next one's start
    w.S_pad = (int)(((long long)T_q / 128 + B + 1) * 128);
    const size_t rows = sizeof(float) * (size_t)H_q * w.S_pad;
    w.nlse2 = take(rows);
    w.dsum = take(rows);
    w.rowsum = take(2 * rows);
    w.ns = T_q > 0 && T_kv > 0 ? sdpa::bwd_kv_head_splits(1, T_kv, H_kv, H_q / H_kv) : 1;
    const size_t kv_rows = (size_t)(w.ns > 1 ? w.ns : 0) * T_kv * H_kv;
    w.dk_part = take(sizeof(float) * kv_rows * d_qk);
    w.dv_part = take(sizeof(float) * kv_rows * d_v);
  }
  w.total = at;
  return w;
}

int check_packed(int B, int T_q, int T_kv, int H_q, int H_kv, int d_qk, int d_v, int causal, int window,
                 int softmax_type, const float* softmax_offset) {
  const int st = sdpa::check_common(B, T_q, T_kv, H_q, H_kv, d_qk, d_v, causal, window, softmax_type, softmax_offset);
  if (st != ATTN_OK) return st;
  if (!supported(d_qk, d_v)) return ATTN_ERR_UNSUPPORTED;
  // row numbers of the padded workspace and block counts stay 32-bit
  if ((long long)T_q + 128LL * B > 0x7fff0000LL || tile_bound(B, T_kv, 128) * H_q > 0x7fffffffLL ||
      tile_bound(B, T_q, 128) * H_q > 0x7fffffffLL)
    return ATTN_ERR_UNSUPPORTED;
  return ATTN_OK;
}

template <class F>
int launch(int kind, int n, const char* what, cudaStream_t s, F f) {
  const int rc = sdpa::timed_launch(kind, n, s, [](void* ctx) { return (*static_cast<F*>(ctx))(); }, &f);
  if (rc == 0) return ATTN_OK;
  if (rc == -2) return ATTN_ERR_UNSUPPORTED;
  sdpa::set_last_error(what, cudaGetLastError());
  return ATTN_ERR_CUDA;
}

int clear(void* p, size_t bytes, cudaStream_t s) {
  return bytes == 0 || cudaMemsetAsync(p, 0, bytes, s) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace

extern "C" {

size_t attn_packed_workspace_size(int B, int T_q, int T_kv, int H_q, int H_kv, int d_qk, int d_v, int backward) {
  if (check_packed(B, T_q, T_kv, H_q, H_kv, d_qk, d_v, 1, -1, 0, nullptr) != ATTN_OK) return 0;
  return layout(B, T_q, T_kv, H_q, H_kv, d_qk, d_v, backward != 0).total;
}

int attn_fwd_packed(const void* q, const void* k, const void* v, void* o, float* lse, const int* cu_seqlens_q,
                    const int* cu_seqlens_kv, int B, int T_q, int T_kv, int H_q, int H_kv, int d_qk, int d_v,
                    float scale, int causal, int window, int softmax_type, const float* softmax_offset, int zero_rest,
                    void* workspace, size_t workspace_bytes, void* stream) {
  const int st = check_packed(B, T_q, T_kv, H_q, H_kv, d_qk, d_v, causal, window, softmax_type, softmax_offset);
  if (st != ATTN_OK) return st;
  if (!cu_seqlens_kv) cu_seqlens_kv = cu_seqlens_q;
  if (T_q == 0 || (B == 0 && !zero_rest)) return ATTN_OK;
  if (!q || !o || !lse || !cu_seqlens_q || (T_kv > 0 && (!k || !v))) return ATTN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) || !aligned(lse, 4) ||
      !aligned(cu_seqlens_q, 4) || !aligned(cu_seqlens_kv, 4) || !aligned(softmax_offset, 4))
    return ATTN_ERR_MISALIGNED;
  const Layout w = layout(B, T_q, T_kv, H_q, H_kv, d_qk, d_v, false);
  if (!workspace || workspace_bytes < w.total || !aligned(workspace, 256)) return ATTN_ERR_WORKSPACE;
  int* err = sdpa::device_error_word();
  if (!err) return ATTN_ERR_CUDA;
  // TMA maps need a non-empty tensor; without keys no kv tile is ever loaded
  const bool any = T_kv > 0;
  CUtensorMap tq, tk, tv;
  if (!sdpa::make_bshd_map(&tq, q, 1, T_q, H_q, d_qk, 128) ||
      !sdpa::make_bshd_map(&tk, any ? k : q, 1, any ? T_kv : 1, any ? H_kv : H_q, d_qk, 128) ||
      !sdpa::make_bshd_map(&tv, any ? v : q, 1, any ? T_kv : 1, any ? H_kv : H_q, any ? d_v : d_qk, 128)) {
    sdpa::set_last_error("cuTensorMapEncodeTiled (packed forward operands)", cudaErrorInvalidValue);
    return ATTN_ERR_CUDA;
  }
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  sdpa::PackedPlanParams plan{};
  plan.cu_q = cu_seqlens_q;
  plan.cu_kv = cu_seqlens_kv;
  plan.B = B; plan.T_q = T_q; plan.T_kv = T_kv;
  plan.causal = causal ? 1 : 0;
  plan.window = window < 0 || window >= T_q ? -1 : window;  // (no row looks further back than T_q - 1)
  plan.clean_q = reinterpret_cast<int*>(ws + w.clean_q);
  plan.clean_kv = reinterpret_cast<int*>(ws + w.clean_kv);
  plan.counts = reinterpret_cast<sdpa::PackedCounts*>(ws + w.counts);
  plan.tiles_fwd = reinterpret_cast<sdpa::PackedTile*>(ws + w.tiles_fwd);
  sdpa::FwdParams p;
  p.B = 1; p.S_q = T_q; p.S_kv = T_kv; p.H_q = H_q; p.H_kv = H_kv; p.G = H_q / H_kv;
  p.scale_log2 = sdpa::resolve_scale(scale, d_qk) * 1.4426950408889634f;
  p.causal = plan.causal;
  p.window = plan.window;
  p.softmax_type = softmax_type;
  p.offset = softmax_offset;
  p.seq_q = nullptr;
  p.seq_kv = nullptr;
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.err = err;
  p.tiles = plan.tiles_fwd;
  p.counts = plan.counts;
  p.tile_bound = tile_bound(B, T_q, 256) > 0 ? tile_bound(B, T_q, 256) : 1;  // (one CTA at least zeroes the rest)
  p.zero_rest = zero_rest != 0;
  if (B <= sdpa::kOwnSeqs && p.tile_bound * H_q <= kOwnCtas) {
    p.tiles = nullptr;
    p.own.cu_q = cu_seqlens_q; p.own.cu_kv = cu_seqlens_kv;
    p.own.B = B; p.own.T_q = T_q; p.own.T_kv = T_kv;
    return launch(ATTN_KERNEL_FWD, 1, "packed forward launch", s,
                  [&] { return sdpa::launch_attn_fwd_packed(d_qk, d_v, tq, tk, tv, p, s); });
  }
  return launch(ATTN_KERNEL_FWD, 2, "packed forward launch", s, [&] {
    const int rc = sdpa::launch_packed_plan(plan, s);
    return rc ? rc : sdpa::launch_attn_fwd_packed(d_qk, d_v, tq, tk, tv, p, s);
  });
}

int attn_bwd_packed(const void* q, const void* k, const void* v, const void* o, const void* dout, const float* lse,
                    void* dq, void* dk, void* dv, float* d_offset, const int* cu_seqlens_q, const int* cu_seqlens_kv,
                    int B, int T_q, int T_kv, int H_q, int H_kv, int d_qk, int d_v, float scale, int causal,
                    int window, int softmax_type, const float* softmax_offset, int zero_rest, void* workspace,
                    size_t workspace_bytes, void* stream) {
  int st = check_packed(B, T_q, T_kv, H_q, H_kv, d_qk, d_v, causal, window, softmax_type, softmax_offset);
  if (st != ATTN_OK) return st;
  const bool learnable = softmax_type == ATTN_SOFTMAX_LEARNABLE;
  if (learnable && !d_offset) return ATTN_ERR_INVALID_ARG;
  if (!cu_seqlens_kv) cu_seqlens_kv = cu_seqlens_q;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if ((T_q > 0 && (!q || !o || !dout || !lse || !dq)) || (T_kv > 0 && (!k || !v || !dk || !dv)) ||
      (B > 0 && !cu_seqlens_q))
    return ATTN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) || !aligned(dout, 16) ||
      !aligned(dq, 16) || !aligned(dk, 16) || !aligned(dv, 16) || !aligned(lse, 4) || !aligned(d_offset, 4) ||
      !aligned(cu_seqlens_q, 4) || !aligned(cu_seqlens_kv, 4) || !aligned(softmax_offset, 4))
    return ATTN_ERR_MISALIGNED;
  const Layout w = layout(B, T_q, T_kv, H_q, H_kv, d_qk, d_v, true);
  if (!workspace || workspace_bytes < w.total || !aligned(workspace, 256)) return ATTN_ERR_WORKSPACE;
  if (d_offset && (!learnable || B == 0 || T_q == 0 || T_kv == 0)) {
    // other sinks have no offset; without a visible key every D is 0
    st = clear(d_offset, sizeof(float) * H_q, s);
    if (st != ATTN_OK) return st;
  }
  if (B == 0) {  // no sequence: every row is one of none
    if (!zero_rest) return ATTN_OK;
    st = clear(dq, (size_t)T_q * H_q * d_qk * 2, s);
    if (st == ATTN_OK) st = clear(dk, (size_t)T_kv * H_kv * d_qk * 2, s);
    return st == ATTN_OK ? clear(dv, (size_t)T_kv * H_kv * d_v * 2, s) : st;
  }
  if (T_q == 0 && T_kv == 0) return ATTN_OK;
  int* err = sdpa::device_error_word();
  if (!err) return ATTN_ERR_CUDA;

  uint8_t* ws = static_cast<uint8_t*>(workspace);
  sdpa::PackedPlanParams plan{};
  plan.cu_q = cu_seqlens_q;
  plan.cu_kv = cu_seqlens_kv;
  plan.B = B; plan.T_q = T_q; plan.T_kv = T_kv;
  plan.causal = causal ? 1 : 0;
  plan.window = window < 0 || window >= T_q ? -1 : window;  // (no row looks further back than T_q - 1)
  plan.clean_q = reinterpret_cast<int*>(ws + w.clean_q);
  plan.clean_kv = reinterpret_cast<int*>(ws + w.clean_kv);
  plan.counts = reinterpret_cast<sdpa::PackedCounts*>(ws + w.counts);
  plan.tiles_kv = reinterpret_cast<sdpa::PackedTile*>(ws + w.tiles_kv);
  plan.tiles_q = reinterpret_cast<sdpa::PackedTile*>(ws + w.tiles_q);
  sdpa::BwdParams p;
  p.B = 1; p.S_q = T_q; p.S_kv = T_kv; p.H_q = H_q; p.H_kv = H_kv; p.G = H_q / H_kv;
  p.scale = sdpa::resolve_scale(scale, d_qk);
  p.scale_log2 = p.scale * 1.4426950408889634f;
  p.causal = plan.causal;
  p.window = plan.window;
  p.softmax_type = softmax_type;
  p.S_pad = w.S_pad;
  p.offset = softmax_offset;
  p.seq_q = nullptr;
  p.seq_kv = nullptr;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.o = static_cast<const __nv_bfloat16*>(o);
  p.dout = static_cast<const __nv_bfloat16*>(dout);
  p.lse = lse;
  p.nlse2 = reinterpret_cast<float*>(ws + w.nlse2);
  p.Dsum = reinterpret_cast<float*>(ws + w.dsum);
  p.d_offset = d_offset;
  p.dq = static_cast<__nv_bfloat16*>(dq);
  p.dk = static_cast<__nv_bfloat16*>(dk);
  p.dv = static_cast<__nv_bfloat16*>(dv);
  p.ns = w.ns;
  p.dk_part = w.ns > 1 ? reinterpret_cast<float*>(ws + w.dk_part) : nullptr;
  p.dv_part = w.ns > 1 ? reinterpret_cast<float*>(ws + w.dv_part) : nullptr;
  p.dq_acc = nullptr;
  p.err = err;
  p.tiles_kv = plan.tiles_kv;
  p.tiles_q = plan.tiles_q;
  p.counts = plan.counts;
  p.ds_rowsum = learnable && T_q > 0 && T_kv > 0 ? reinterpret_cast<float*>(ws + w.rowsum) : nullptr;
  p.tile_bound_kv = tile_bound(B, T_kv, 128);
  p.tile_bound_q = tile_bound(B, T_q, 128);
  p.zero_rest = zero_rest != 0;
  // the offset's gradient sums over all padded rows: those of no query count as zeros
  if (p.ds_rowsum) {
    st = clear(p.nlse2, w.rowsum - w.nlse2 + 2 * sizeof(float) * (size_t)H_q * w.S_pad, s);
    if (st != ATTN_OK) return st;
  }
  st = launch(ATTN_KERNEL_BWD_PREPROCESS, 2, "packed backward preprocess launch", s, [&] {
    const int rc = sdpa::launch_packed_plan(plan, s);
    return rc ? rc : sdpa::launch_packed_preprocess(d_qk, d_v, p, s);
  });
  if (st != ATTN_OK) return st;
  // TMA maps need a non-empty tensor; without keys (or queries) no tile of them is ever loaded
  const bool wide = d_qk == d_v, aq = T_q > 0, ak = T_kv > 0;
  const void* mq = aq ? q : k;
  const void* mk = ak ? k : q;
  CUtensorMap tq128, tdo128, tk, tv, tq64, tdo64;
  bool ok = sdpa::make_bshd_map(&tq128, mq, 1, aq ? T_q : 1, aq ? H_q : 1, d_qk, 128) &&
            sdpa::make_bshd_map(&tdo128, aq ? dout : k, 1, aq ? T_q : 1, aq ? H_q : 1, d_v, 128) &&
            sdpa::make_bshd_map(&tk, mk, 1, ak ? T_kv : 1, ak ? H_kv : 1, d_qk, 128) &&
            sdpa::make_bshd_map(&tv, ak ? v : q, 1, ak ? T_kv : 1, ak ? H_kv : 1, d_v, 128);
  if (!wide)
    ok = ok && sdpa::make_bshd_map(&tq64, mq, 1, aq ? T_q : 1, aq ? H_q : 1, d_qk, 64) &&
         sdpa::make_bshd_map(&tdo64, aq ? dout : k, 1, aq ? T_q : 1, aq ? H_q : 1, d_v, 64);
  if (!ok) {
    sdpa::set_last_error("cuTensorMapEncodeTiled (packed backward operands)", cudaErrorInvalidValue);
    return ATTN_ERR_CUDA;
  }
  if (ak)
    st = launch(ATTN_KERNEL_BWD_KV, 1, "packed backward kv kernel launch", s, [&] {
      return wide ? sdpa::launch_bwd_kv_wide_packed(d_qk, tq128, tk, tv, tdo128, p, s)
                  : sdpa::launch_bwd_kv_packed_mla(tq64, tk, tv, tdo64, p, s);
    });
  // (right behind the kv kernel, in whose tail it is set up)
  if (st == ATTN_OK && aq)
    st = launch(ATTN_KERNEL_BWD_Q, 1, "packed backward dQ kernel launch", s,
                [&] { return sdpa::launch_bwd_q_packed(d_qk, d_v, tq128, tk, tv, tdo128, p, ak, s); });
  if (st == ATTN_OK && p.ns > 1)
    st = launch(ATTN_KERNEL_BWD_DQ_CONVERT, 2, "packed dK/dV combine launch", s,
                [&] { return sdpa::launch_packed_kv_combine(d_qk, d_v, p, s); });
  if (st == ATTN_OK && p.ds_rowsum)
    st = launch(ATTN_KERNEL_BWD_PREPROCESS, 1, "packed d_offset launch", s,
                [&] { return sdpa::launch_packed_doffset(p, s); });
  return st;
}

}  // extern "C"
