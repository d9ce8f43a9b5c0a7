// kv4_store.cu -- filling, reading and copying the 4-bit paged key/value cache (layout and
// number format in kv4.cuh).  All three kernels are bound by memory: they move each byte
// once.
#include "attn_kernels.h"
#include "kv4.cuh"
#include "ptx.cuh"

namespace sdpa {

namespace {

constexpr int kTok = 16;  // tokens of one block of threads

struct TokenAt {
  long long block;  // byte offset of the token's page in the pool (head 0), -1: nowhere, -2: no sequence
  int w;            // the token's place in its page
};

// Where rows t0 .. t0 + kTok - 1 of the packed tensors live in the pool.
__device__ __forceinline__ void find_tokens(const Kv4StoreParams& p, int t0, TokenAt* at) {
  if (threadIdx.x < kTok) {
    const int t = t0 + threadIdx.x;
    TokenAt a{-2, 0};
    if (t < p.T) {
      const int b = packed_row_entry(p.cu, p.B, t);
      if (b >= 0) {
        const long long pos = (long long)__ldg(p.start + b) + (t - __ldg(p.cu + b));
        const int pg = pos > 0x7fffffffLL ? -1 : kv4_page(p.c, b, (int)pos);  // (pos may be negative)
        a.block = -1;
        if (pg >= 0) {
          a.block = (long long)pg * p.c.H_kv * kv4_block_bytes(p.c.page_size, p.c.d);
          a.w = (int)pos & (p.c.page_size - 1);
        } else {
          atomicCAS(p.page_err, 0, p.site);
        }
      }
    }
    at[threadIdx.x] = a;
  }
  __syncthreads();
}

}  // namespace

// One thread quantises 16 values.  Consecutive threads take the groups of one token and
// head, then the block's tokens, then heads: a warp reads whole rows of K or V and writes
// one contiguous run of codes (K) or whole token pairs (V).
template <int D>
__global__ void __launch_bounds__(256) kv4_append_kernel(const Kv4StoreParams p) {
  constexpr int NG = D / 16;
  __shared__ TokenAt at[kTok];
  const int t0 = blockIdx.x * kTok;
  find_tokens(p, t0, at);
  const int P = p.c.page_size, blk = kv4_block_bytes(P, D);
  const int n = kTok * NG * p.c.H_kv;
  for (int it = threadIdx.x; it < 2 * n; it += 256) {
    const int is_v = it >= n;
    const int e = is_v ? it - n : it;
    const int g = e % NG, tk = (e / NG) % kTok, h = e / (NG * kTok);
    const TokenAt a = at[tk];
    if (a.block < 0) continue;
    const __nv_bfloat16* src =
        (is_v ? p.v + (t0 + tk) * p.v_stride : p.k + (t0 + tk) * p.k_stride) + (size_t)h * D + g * 16;
    const uint4 x0 = __ldg(reinterpret_cast<const uint4*>(src)), x1 = __ldg(reinterpret_cast<const uint4*>(src) + 1);
    const uint32_t ws[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
    float f[16], amax = 0.f;
    bool bad = false;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      f[2 * q] = __uint_as_float(ws[q] << 16);
      f[2 * q + 1] = __uint_as_float(ws[q] & 0xFFFF0000u);
    }
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      bad |= !(fabsf(f[q]) <= 3.4028234e38f);
      amax = fmaxf(amax, fabsf(f[q]));
    }
    const int sb = bad ? kKv4BadScale : kv4_scale_byte(amax);
    const float s = kv4_scale_value(sb);
    uint32_t c[2] = {0x88888888u, 0x88888888u};  // all zeros
    if (!bad && sb > 0) {
      c[0] = c[1] = 0u;
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        const int v = max(-8, min(7, __float2int_rn(__fdiv_rn(f[q], s)))) + 8;
        c[q / 8] |= (uint32_t)v << (4 * (q % 8));
      }
    }
    uint8_t* base = p.pool + a.block + (size_t)h * blk;
    if (!is_v) {
      *reinterpret_cast<uint2*>(base + a.w * (D / 2) + g * 8) = make_uint2(c[0], c[1]);
      base[kv4_off_sk(P, D) + a.w * NG + g] = (uint8_t)sb;
    } else {
      uint8_t* vb = base + kv4_off_v(P, D);
      if constexpr (D == 128) {
        *reinterpret_cast<uint2*>(vb + kv4_v_at(a.w, g, D)) = make_uint2(c[0], c[1]);
      } else {  // 16 values are two eighths of the head dim
        *reinterpret_cast<uint32_t*>(vb + kv4_v_at(a.w, 2 * g, D)) = c[0];
        *reinterpret_cast<uint32_t*>(vb + kv4_v_at(a.w, 2 * g + 1, D)) = c[1];
      }
      base[kv4_off_sv(P, D) + (a.w >> 1) * 2 * NG + 2 * g + (a.w & 1)] = (uint8_t)sb;
    }
  }
}

// The reverse: one thread turns 16 codes into 16 bf16 values (exact).  Tokens whose page is
// not in the pool read as zeros; rows of no sequence are left alone, or zeroed on request.
template <int D>
__global__ void __launch_bounds__(256) kv4_gather_kernel(const Kv4StoreParams p) {
  constexpr int NG = D / 16;
  __shared__ TokenAt at[kTok];
  const int t0 = blockIdx.x * kTok;
  find_tokens(p, t0, at);
  const int P = p.c.page_size, blk = kv4_block_bytes(P, D);
  const int n = kTok * NG * p.c.H_kv;
  for (int it = threadIdx.x; it < 2 * n; it += 256) {
    const int is_v = it >= n;
    const int e = is_v ? it - n : it;
    const int g = e % NG, tk = (e / NG) % kTok, h = e / (NG * kTok);
    const TokenAt a = at[tk];
    if (t0 + tk >= p.T || (a.block == -2 && !p.zero_rest)) continue;
    uint2 c = make_uint2(0u, 0u);
    float s = 0.f;
    if (a.block >= 0) {
      const uint8_t* base = p.pool + a.block + (size_t)h * blk;
      if (!is_v) {
        c = __ldg(reinterpret_cast<const uint2*>(base + a.w * (D / 2) + g * 8));
        s = kv4_scale_value(__ldg(base + kv4_off_sk(P, D) + a.w * NG + g));
      } else {
        const uint8_t* vb = base + kv4_off_v(P, D);
        if constexpr (D == 128) {
          c = __ldg(reinterpret_cast<const uint2*>(vb + kv4_v_at(a.w, g, D)));
        } else {
          c.x = __ldg(reinterpret_cast<const uint32_t*>(vb + kv4_v_at(a.w, 2 * g, D)));
          c.y = __ldg(reinterpret_cast<const uint32_t*>(vb + kv4_v_at(a.w, 2 * g + 1, D)));
        }
        s = kv4_scale_value(__ldg(base + kv4_off_sv(P, D) + (a.w >> 1) * 2 * NG + 2 * g + (a.w & 1)));
      }
    }
    uint32_t o[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const uint32_t w = q < 4 ? c.x : c.y;
      const int lo = (int)((w >> (8 * (q % 4))) & 15u) - 8, hi = (int)((w >> (8 * (q % 4) + 4)) & 15u) - 8;
      o[q] = pack_bf16x2((float)lo * s, (float)hi * s);
    }
    __nv_bfloat16* dst = (is_v ? p.v_out : p.k_out) + ((size_t)(t0 + tk) * p.c.H_kv + h) * D + g * 16;
    reinterpret_cast<uint4*>(dst)[0] = make_uint4(o[0], o[1], o[2], o[3]);
    reinterpret_cast<uint4*>(dst)[1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

int launch_kv4_append(const Kv4StoreParams& p, cudaStream_t stream) {
  const unsigned blocks = (unsigned)((p.T + kTok - 1) / kTok);
  if (p.c.d == 128) kv4_append_kernel<128><<<blocks, 256, 0, stream>>>(p);
  else kv4_append_kernel<64><<<blocks, 256, 0, stream>>>(p);
  return cudaPeekAtLastError() == cudaSuccess ? 0 : -1;
}

int launch_kv4_gather(const Kv4StoreParams& p, cudaStream_t stream) {
  const unsigned blocks = (unsigned)((p.T + kTok - 1) / kTok);
  if (p.c.d == 128) kv4_gather_kernel<128><<<blocks, 256, 0, stream>>>(p);
  else kv4_gather_kernel<64><<<blocks, 256, 0, stream>>>(p);
  return cudaPeekAtLastError() == cudaSuccess ? 0 : -1;
}

// Pages are copied 16 bytes a thread.  The pairs are kernel arguments: the call needs no
// host-to-device copy, keeps nothing after it returns, and can be captured.
__global__ void __launch_bounds__(256) kv4_copy_kernel(uint8_t* pool, long long layer_bytes, long long page_bytes,
                                                       const __grid_constant__ Kv4Pairs pairs) {
  const int2 pr = pairs.at[blockIdx.y];
  uint8_t* layer = pool + (size_t)blockIdx.z * layer_bytes;
  const uint4* src = reinterpret_cast<const uint4*>(layer + (size_t)pr.x * page_bytes);
  uint4* dst = reinterpret_cast<uint4*>(layer + (size_t)pr.y * page_bytes);
  const long long n = page_bytes / 16;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * 256)
    dst[i] = __ldg(src + i);
}

int launch_kv4_copy(uint8_t* pool, int n_layers, long long layer_bytes, long long page_bytes, const int* src,
                    const int* dst, int n, cudaStream_t stream) {
  Kv4Pairs pairs;
  const long long units = page_bytes / 16;
  const unsigned gx = (unsigned)((units + 1023) / 1024 < 64 ? (units + 1023) / 1024 : 64);
  for (int a = 0; a < n; a += kKv4PairsMax) {
    const int m = n - a < kKv4PairsMax ? n - a : kKv4PairsMax;
    for (int i = 0; i < m; ++i) pairs.at[i] = make_int2(src[a + i], dst[a + i]);
    kv4_copy_kernel<<<dim3(gx, m, n_layers), 256, 0, stream>>>(pool, layer_bytes, page_bytes, pairs);
    if (cudaPeekAtLastError() != cudaSuccess) return -1;
  }
  return 0;
}

}  // namespace sdpa
