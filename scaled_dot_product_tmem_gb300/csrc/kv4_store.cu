// kv4_store.cu -- filling, reading and copying the 4-bit paged key/value cache (layout and
// number format in kv4.cuh).  Each kernel moves each byte once.  Measured with 8 heads of 128:
// 15,677 tokens appended in 16 us (83 MB; 18 us without the loads ahead of the lookup) and
// read back in 14 us; 1500 pages of 64 tokens copied in 4 layers in 134 us (885 MB moved,
// 6.6 TB/s); one token of each of 64 sequences appended or read back in about 3 us (lookups).  With the keys
// rotated on the way and 32 query heads beside them, 15,677 tokens in 61 us (347 MB).  Up to 9 kept tokens of
// each of 64 sequences moved in 32 layers in 14 us (23 with their places worked out anew for every head).
#include "attn_kernels.h"
#include "kv4.cuh"
#include "launch.h"
#include "ptx.cuh"
#include "rope.cuh"

namespace sdpa {

namespace {

constexpr int kTok = 16;  // tokens of one block of 256 threads: 16 threads look each one up

struct TokenAt {
  long long block;  // byte offset of the token's page in the pool (head 0), -1: nowhere, -2: no sequence
  int w;            // the token's place in its page
};

// Where rows t0 .. t0 + kTok - 1 of the packed tensors live in the pool.  A row's sequence is the
// last b with cu[b] <= t (checked against its end): 16 lanes search the offsets 16 ways at a
// time, so that a few dependent loads find it.  Offsets that are not ascending may give any
// sequence, never a row outside the one returned.
template <bool EARLY = false>
__device__ __forceinline__ void find_tokens(const Kv4StoreParams& p, int t0, TokenAt* at) {
  const int lane16 = threadIdx.x % 16, half = threadIdx.x & 16, i = threadIdx.x / 16;
  const int t = t0 + i;
  int lo = 0, n = p.B;  // the count of cu[0 .. B) that are <= t lies in [lo, lo + n]
  while (__any_sync(0xffffffffu, n > 0)) {
    const int step = (n + 15) / 16, at_ = lo + lane16 * step;
    const bool le = lane16 * step < n && load_input<EARLY>(p.cu + at_) <= t;
    const int c = __popc((__ballot_sync(0xffffffffu, le) >> half) & 0xFFFFu);
    if (c == 0) {
      n = 0;
    } else {
      const int rest = n - ((c - 1) * step + 1);
      lo += (c - 1) * step + 1;
      n = min(step - 1, rest);
    }
  }
  if (lane16 == 0) {
    TokenAt a{-2, 0};
    const int b = lo - 1;
    if (t < p.T && b >= 0) {
      const int first = load_input<EARLY>(p.cu + b), end = load_input<EARLY>(p.cu + b + 1), start = load_input<EARLY>(p.start + b);
      if (first <= t && t < end) {
        const long long pos = (long long)start + (t - first);
        const int pg = pos > 0x7fffffffLL ? -1 : kv4_page<EARLY>(p.c, b, (int)pos);  // (pos may be negative)
        a.block = -1;
        if (pg >= 0) {
          a.block = (long long)pg * p.c.H_kv * kv4_block_bytes(p.c.page_size, p.c.d);
          a.w = (int)pos & (p.c.page_size - 1);
        } else {
          atomicCAS(p.page_err, 0, p.site);
        }
      }
    }
    at[i] = a;
  }
  __syncthreads();
}

// 16 values to codes and a scale byte.  c = round(x / s) without a division: x (1/s) is off by
// 2^-22 or so, ties x / s = k + 1/2 are exact numbers, and any other x / s is at least 2^-9
// away from a tie (x has 8 significant bits, s has 4), so one fma that rounds x (1/s) to multiples
// of 2^-12 (by adding 3 * 2^10) falls on the same side as x / s, and ties on themselves; the
// second rounding, to whole numbers (by going on to 3 * 2^22), is then the definition's.  The
// bits of those sums are whole numbers with an offset, so a word of 8 codes is their sum with
// weights 16^i and one constant for all offsets.
__device__ __forceinline__ int quantise16(const uint4& x0, const uint4& x1, uint32_t (&c)[2]) {
  const uint32_t ws[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
  uint32_t mx = 0u;  // largest magnitudes of both halves: bf16 bits order as the numbers do
#pragma unroll
  for (int q = 0; q < 8; ++q) mx = __vmaxu2(mx, ws[q] & 0x7FFF7FFFu);
  const uint32_t top = max(mx >> 16, mx & 0xFFFFu);
  c[0] = c[1] = 0x88888888u;  // zeros
  if (top >= 0x7F80u) return kKv4BadScale;
  const int sb = kv4_scale_byte(__uint_as_float(top << 16));
  if (sb == 0) return 0;
  // s is within 2^-4 of max|x| / 7, so |x / s| < 7.5 and needs no clamping, unless s is below 2^-14
  // (fewer bits) or the largest scale
  const bool far = sb < 8 || sb == 0xF7;
  const float inv = __frcp_rn(kv4_scale_value(sb));
  const uint64_t inv2 = f2_pack(inv, inv);
  constexpr float kGrid = 1.5f * 2048.f, kInt = 1.5f * 8388608.f;
  const uint64_t grid = f2_pack(kGrid, kGrid), whole = f2_pack(kInt - kGrid, kInt - kGrid);
  uint64_t y[8];
#pragma unroll
  for (int q = 0; q < 8; ++q)
    y[q] = f2_fma(f2_pack(__uint_as_float(ws[q] << 16), __uint_as_float(ws[q] & 0xFFFF0000u)), inv2, grid);
  if (far) {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      float a, b;
      f2_unpack(y[q], a, b);
      y[q] = f2_pack(fminf(fmaxf(a, kGrid - 8.f), kGrid + 7.f), fminf(fmaxf(b, kGrid - 8.f), kGrid + 7.f));
    }
  }
  constexpr uint32_t kOffset = 0x4B400000u - 8u;  // bits of kInt, and code 8 for 0
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t w = 0u;
#pragma unroll
    for (int q = 3; q >= 0; --q) {
      float a, b;
      f2_unpack(f2_add(y[4 * h + q], whole), a, b);
      w = (w * 16u + __float_as_uint(b)) * 16u + __float_as_uint(a);
    }
    c[h] = w - kOffset * 0x11111111u;
  }
  return sb;
}

}  // namespace

// One thread quantises 16 dims of a token's K and of its V for one head after another.
// Consecutive threads take the groups of one token and head, then the block's tokens, then
// heads: a warp reads whole rows of K or V and writes one contiguous run of codes (K) or
// whole token pairs (V).
// ROT: 1 (half layout) or 2 (interleaved) turns K by the row's position first (rope.cuh): a thread
// reads the partners of its 16 dims too (the lines are in L1 for the partner's own thread) and keeps its cosines
// and sines for all heads.  The turned values are rounded to bf16, as a rotation of its own would
// leave them, and then quantised.
// Block bx takes tokens 16 bx on, and of the heads groups by, by + gy, ... of HS.
template <int D, int ROT>
__device__ __forceinline__ void append_block(const Kv4StoreParams& p, const RopeParams& rp, int bx, int by, unsigned gy) {
  constexpr int NG = D / 16, HS = 256 / (NG * kTok);  // heads a block takes at a time
  constexpr bool EARLY = ROT != 0;                    // launched while the kernel before it runs
  const unsigned step = HS * gy;  // (signed, it costs the loop ten registers)
  __shared__ TokenAt at[kTok];
  const int t0 = bx * kTok;
  const int P = p.c.page_size, blk = kv4_block_bytes(P, D);
  const int g = threadIdx.x % NG, tk = threadIdx.x / NG % kTok;
  const __nv_bfloat16* kr = p.k + (size_t)(t0 + tk) * p.k_stride + g * 16;
  const __nv_bfloat16* vr = p.v + (size_t)(t0 + tk) * p.v_stride + g * 16;
  [[maybe_unused]] int part[2] = {0, 0};  // where the partners of dims 16 g + 8 i lie (0: these dims stay)
  [[maybe_unused]] float c[ROT ? 2 : 1][8], sn[ROT ? 2 : 1][8];
  if constexpr (ROT != 0) {
    if (t0 + tk < p.T) {
      const float* row = rp.table + (size_t)(t0 + tk) * 2 * rp.n;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int x = 16 * g + 8 * i - rp.first;
        if (x < 0 || x >= 2 * rp.n) continue;
        if constexpr (ROT == 1) {
          part[i] = x < rp.n ? rp.n : -rp.n;
          const float* f = row + (x < rp.n ? x : x - rp.n);
          load8(f, c[i]);
          load8(f + rp.n, sn[i]);
          if (x >= rp.n) {
#pragma unroll
            for (int j = 0; j < 8; ++j) sn[i][j] = -sn[i][j];
          }
        } else {
          part[i] = 1;
          const float4 a = load4(row + x / 2), b = load4(row + rp.n + x / 2);
          c[i][0] = a.x, c[i][1] = a.y, c[i][2] = a.z, c[i][3] = a.w;
          sn[i][0] = b.x, sn[i][1] = b.y, sn[i][2] = b.z, sn[i][3] = b.w;
        }
      }
    }
  }
  // a head's values are loaded ahead: the first while the tokens are looked up, then each while
  // the one before it is rounded
  uint4 k0, k1, v0, v1;
  [[maybe_unused]] uint4 q0, q1;  // the partners
  auto load = [&](int h) {
    const uint4* ks = reinterpret_cast<const uint4*>(kr + (size_t)h * D);
    const uint4* vs = reinterpret_cast<const uint4*>(vr + (size_t)h * D);
    k0 = load_input<EARLY>(ks);
    k1 = load_input<EARLY>(ks + 1);
    if constexpr (ROT == 1) {
      q0 = load_input<EARLY>(reinterpret_cast<const uint4*>(kr + (size_t)h * D + part[0]));
      q1 = load_input<EARLY>(reinterpret_cast<const uint4*>(kr + (size_t)h * D + 8 + part[1]));
    }
    v0 = load_input<EARLY>(vs);
    v1 = load_input<EARLY>(vs + 1);
  };
  int h = threadIdx.x / (NG * kTok) + HS * by;
  if (t0 + tk < p.T && h < p.c.H_kv) load(h);
  find_tokens<EARLY>(p, t0, at);
  const TokenAt a = at[tk];
  if (a.block < 0) return;
  uint8_t* page = p.pool + a.block;
  const int at_k = a.w * (D / 2) + g * 8, at_sk = kv4_off_sk(P, D) + a.w * NG + g;
  const int at_sv = kv4_off_sv(P, D) + (a.w >> 1) * 2 * NG + 2 * g + (a.w & 1);
  const int at_v0 = kv4_off_v(P, D) + kv4_v_at(a.w, D == 128 ? g : 2 * g, D);
  const int at_v1 = kv4_off_v(P, D) + kv4_v_at(a.w, 2 * g + 1, D);  // D = 64: 16 dims are two eighths
#pragma unroll 2
  for (; h < p.c.H_kv; h += step) {
    uint4 ka = k0, kb = k1;
    const uint4 va = v0, vb = v1;
    if constexpr (ROT == 1) {
      if (part[0]) ka = rope_turn8(k0, q0, c[0], sn[0]);
      if (part[1]) kb = rope_turn8(k1, q1, c[1], sn[1]);
    } else if constexpr (ROT == 2) {
      if (part[0]) ka = rope_turn_pairs(k0, c[0], sn[0]);
      if (part[1]) kb = rope_turn_pairs(k1, c[1], sn[1]);
    }
    if (h + step < p.c.H_kv) load(h + step);
    uint8_t* base = page + (size_t)h * blk;
    uint32_t cd[2];
    int sb = quantise16(ka, kb, cd);
    *reinterpret_cast<uint2*>(base + at_k) = make_uint2(cd[0], cd[1]);
    base[at_sk] = (uint8_t)sb;
    sb = quantise16(va, vb, cd);
    if constexpr (D == 128) {
      *reinterpret_cast<uint2*>(base + at_v0) = make_uint2(cd[0], cd[1]);
    } else {
      *reinterpret_cast<uint32_t*>(base + at_v0) = cd[0];
      *reinterpret_cast<uint32_t*>(base + at_v1) = cd[1];
    }
    base[at_sv] = (uint8_t)sb;
  }
}

template <int D>
__global__ void __launch_bounds__(256) kv4_append_kernel(const Kv4StoreParams p) {
  append_block<D, 0>(p, RopeParams{}, blockIdx.x, blockIdx.y, gridDim.y);
}

// gx x gy blocks append, those behind them turn the queries.  (A kernel of its own: as one with the plain append, that
// took 13.5 us instead of 12.9 for 15,677 tokens.)
template <int D, int ROT>
__global__ void __launch_bounds__(256, ROT == 1 ? 2 : 3)
    kv4_append_rope_kernel(const Kv4StoreParams p, const RopeParams rp, int gx, int gy) {
  grid_wait();  // the table, or whatever was before
  if ((int)blockIdx.x >= gx * gy) return rope_block<ROT == 2>(rp, blockIdx.x - gx * gy);
  const int by = blockIdx.x / gx;
  append_block<D, ROT>(p, rp, blockIdx.x - by * gx, by, gy);
}

// 8 codes as 8 bf16 values (exact).
__device__ __forceinline__ uint4 held8(uint32_t w, int sb) {
  const uint32_t s = scale_pair((uint32_t)sb * 0x0101u), m = bf2_mul(s, kM136);
  // pairs (0, 4), (1, 5), (2, 6), (3, 7), then neighbours
  const uint32_t a = decode_pair(w, s, m), b = decode_pair(w >> 4, s, m), d = decode_pair(w >> 8, s, m),
                 e = decode_pair(w >> 12, s, m);
  return make_uint4(__byte_perm(a, b, 0x5410), __byte_perm(d, e, 0x5410), __byte_perm(a, b, 0x7632),
                    __byte_perm(d, e, 0x7632));
}

// The reverse: one thread turns a word of 8 codes into 16 bytes, so that a warp writes whole rows.
// Tokens whose page is not in the pool read as zeros; rows of no sequence are left alone, or
// zeroed on request.
template <int D>
__global__ void __launch_bounds__(256) kv4_gather_kernel(const Kv4StoreParams p) {
  constexpr int NW = D / 8, TS = 256 / NW;  // words of a row; tokens a block takes at a time
  __shared__ TokenAt at[kTok];
  const int t0 = blockIdx.x * kTok;
  find_tokens(p, t0, at);
  const int P = p.c.page_size, blk = kv4_block_bytes(P, D);
  const int x = threadIdx.x % NW, g = x / 2;
#pragma unroll
  for (int tk = threadIdx.x / NW; tk < kTok; tk += TS) {
    const TokenAt a = at[tk];
    if (t0 + tk >= p.T || (a.block == -2 && !p.zero_rest)) continue;
    const bool have = a.block >= 0;
    const uint8_t* page = p.pool + (have ? a.block : 0);
    const int at_k = a.w * (D / 2) + x * 4, at_sk = kv4_off_sk(P, D) + a.w * (D / 16) + g;
    const int at_v = kv4_off_v(P, D) + (D == 128 ? kv4_v_at(a.w, g, D) + (x % 2) * 4 : kv4_v_at(a.w, x, D));
    const int at_sv = kv4_off_sv(P, D) + (a.w >> 1) * (D / 8) + 2 * g + (a.w & 1);
    const size_t row = (size_t)(t0 + tk) * p.c.H_kv;
#pragma unroll 4
    for (int h = blockIdx.y; h < p.c.H_kv; h += gridDim.y) {
      const uint8_t* base = page + (size_t)h * blk;
      uint32_t ck = 0u, cv = 0u;
      int sk = 0, sv = 0;
      if (have) {
        ck = __ldg(reinterpret_cast<const uint32_t*>(base + at_k));
        cv = __ldg(reinterpret_cast<const uint32_t*>(base + at_v));
        sk = __ldg(base + at_sk);
        sv = __ldg(base + at_sv);
      }
      *reinterpret_cast<uint4*>(p.k_out + (row + h) * D + x * 8) = held8(ck, sk);
      *reinterpret_cast<uint4*>(p.v_out + (row + h) * D + x * 8) = held8(cv, sv);
    }
  }
}

// Blocks: kTok tokens each, `heads` of them at a time; with few tokens the heads are spread over
// more blocks.
static dim3 store_grid(const Kv4StoreParams& p, int heads) {
  const int x = (p.T + kTok - 1) / kTok, y_max = (p.c.H_kv + heads - 1) / heads;
  const int y = x >= 152 * 4 ? 1 : (152 * 4 + x - 1) / x;
  return dim3((unsigned)x, (unsigned)(y < y_max ? y : y_max));
}

int launch_kv4_append(const Kv4StoreParams& p, cudaStream_t stream) {
  const dim3 blocks = store_grid(p, 256 / (p.c.d / 16 * kTok));
  if (p.c.d == 128) kv4_append_kernel<128><<<blocks, 256, 0, stream>>>(p);
  else kv4_append_kernel<64><<<blocks, 256, 0, stream>>>(p);
  return cudaPeekAtLastError() == cudaSuccess ? 0 : -1;
}

int launch_kv4_append_rope(const Kv4StoreParams& p, const RopeParams& rp, bool interleaved, cudaStream_t stream) {
  dim3 g = store_grid(p, 256 / (p.c.d / 16 * kTok));
  if (p.B == 0) g = dim3(0, 1);  // only queries to turn
  const long long blocks = (long long)g.x * g.y + rope_blocks(rp);
  if (blocks > 0x7fffffffLL) return -2;
  auto kern = p.c.d == 128 ? (interleaved ? kv4_append_rope_kernel<128, 2> : kv4_append_rope_kernel<128, 1>)
                           : (interleaved ? kv4_append_rope_kernel<64, 2> : kv4_append_rope_kernel<64, 1>);
  return launch_kernel(kern, dim3((unsigned)blocks), 256, 0, stream, true, p, rp, (int)g.x, (int)g.y);
}

// Kept tokens: node kept[b][i] of sequence b's tree (its token start[b] + kept[b][i]) becomes token
// start[b] + i, in the order of i, until the first negative entry.  A block takes one sequence: a warp
// looks 32 entries' pages up at once, for all heads and layers that the block then walks.  A thread owns
// the same few bytes of every token of a head and layer, so its moves follow one another without a
// barrier, whatever the entries are.  Entries that only move down (kept >= i, as ascending ones do)
// cannot read what an earlier one of the same eight wrote, so eight are loaded at once (sixteen: 15.0 instead of 14.2 us
// for up to 9 tokens of each of 64 sequences in 32 layers).
template <int D>
__global__ void __launch_bounds__(256) kv4_keep_kernel(const Kv4KeepParams p) {
  // words (4 bytes) of K codes, of V codes, of K scales; then V's scale bytes
  constexpr int KW = D / 8, VW = D / 8, SW = D / 64, NV = D / 16, BATCH = 8;
  static_assert(KW + VW + SW + NV <= 64, "64 threads a head and layer");
  struct Move {
    long long src, dst;  // a page's offset in a layer, or -1: this entry moves nothing
    int ws, wd;          // the tokens' places in their pages
  };
  __shared__ Move moves[32];
  __shared__ longlong2 at[32][64];  // where each thread's bytes of a move lie in a layer's head 0 (x < 0: it moves nothing)
  __shared__ int n_moves, n_down;  // entries until the end; how many of the first keep to kept >= i
  const int x = threadIdx.x % 64, b = blockIdx.y;
  const int P = p.c.page_size, blk = kv4_block_bytes(P, D), units = p.c.H_kv * p.n_layers;
  const long long page_bytes = (long long)p.c.H_kv * blk;
  const int start = __ldg(p.start + b);
  // this thread's bytes of the token at place w of a page
  auto place = [&](int w) {
    if (x < KW) return w * (D / 2) + 4 * x;
    if (x < KW + VW) return kv4_off_v(P, D) + kv4_v_at(w, (x - KW) * 4 / (D / 16), D) + (x - KW) * 4 % (D / 16);
    if (x < KW + VW + SW) return kv4_off_sk(P, D) + w * (D / 16) + 4 * (x - KW - VW);
    return kv4_off_sv(P, D) + (w >> 1) * (D / 8) + 2 * (x - KW - VW - SW) + (w & 1);
  };
  const bool byte = x >= KW + VW + SW;
  for (int i0 = 0; i0 < p.most; i0 += 32) {
    if (threadIdx.x < 32) {
      const int i = i0 + threadIdx.x, from = i < p.most ? __ldg(p.kept + (size_t)b * p.most + i) : -1;
      const unsigned end = __ballot_sync(0xffffffffu, from < 0), up = __ballot_sync(0xffffffffu, from < i);
      const int n = end ? __ffs(end) - 1 : 32;
      Move m{-1, -1, 0, 0};
      if ((int)threadIdx.x < n && from != i) {
        const long long ts = (long long)start + from, td = (long long)start + i;
        const int ps = ts > 0x7fffffffLL ? -1 : kv4_page(p.c, b, (int)ts), pd = td > 0x7fffffffLL ? -1 : kv4_page(p.c, b, (int)td);
        if (ps >= 0 && pd >= 0) m = Move{ps * page_bytes, pd * page_bytes, (int)ts & (P - 1), (int)td & (P - 1)};
        else atomicCAS(p.page_err, 0, p.site);
      }
      moves[threadIdx.x] = m;
      if (threadIdx.x == 0) {
        n_moves = n;
        n_down = up ? __ffs(up) - 1 : 32;
      }
    }
    __syncthreads();
    const int n = n_moves, down = min(n_down, n);
    if (x < KW + VW + SW + NV)
      for (int j = threadIdx.x / 64; j < n; j += 4) {
        const Move m = moves[j];
        at[j][x] = m.src < 0 ? make_longlong2(-1, -1) : make_longlong2(m.src + place(m.ws), m.dst + place(m.wd));
      }
    __syncthreads();
    if (x < KW + VW + SW + NV) {
      for (int u = blockIdx.x * 4 + threadIdx.x / 64; u < units; u += gridDim.x * 4) {
        uint8_t* base = p.pool + (size_t)(u / p.c.H_kv) * p.layer_bytes + (size_t)(u % p.c.H_kv) * blk;
        auto get = [&](long long o) { return byte ? (uint32_t)base[o] : *reinterpret_cast<const uint32_t*>(base + o); };
        auto put = [&](long long o, uint32_t v) {
          if (byte) base[o] = (uint8_t)v;
          else *reinterpret_cast<uint32_t*>(base + o) = v;
        };
        int j = 0;
        for (; j < down; j += BATCH) {
          uint32_t v[BATCH];
          const int last = min(BATCH, down - j);
#pragma unroll
          for (int q = 0; q < BATCH; ++q)
            if (q < last && at[j + q][x].x >= 0) v[q] = get(at[j + q][x].x);
#pragma unroll
          for (int q = 0; q < BATCH; ++q)
            if (q < last && at[j + q][x].x >= 0) put(at[j + q][x].y, v[q]);
        }
        for (j = down; j < n; ++j)
          if (at[j][x].x >= 0) put(at[j][x].y, get(at[j][x].x));
      }
    }
    if (n < 32) break;
    __syncthreads();
  }
}

int launch_kv4_gather(const Kv4StoreParams& p, cudaStream_t stream) {
  const dim3 blocks = store_grid(p, 1);
  if (p.c.d == 128) kv4_gather_kernel<128><<<blocks, 256, 0, stream>>>(p);
  else kv4_gather_kernel<64><<<blocks, 256, 0, stream>>>(p);
  return cudaPeekAtLastError() == cudaSuccess ? 0 : -1;
}

int launch_kv4_keep(const Kv4KeepParams& p, cudaStream_t stream) {
  // four (head, layer) units a block at a time; enough blocks a sequence to fill the device
  const int units = (p.c.H_kv * p.n_layers + 3) / 4, fill = (152 * 8 + p.B - 1) / p.B;
  const dim3 grid((unsigned)(units < fill ? units : fill), (unsigned)p.B);
  if (p.c.d == 128) kv4_keep_kernel<128><<<grid, 256, 0, stream>>>(p);
  else kv4_keep_kernel<64><<<grid, 256, 0, stream>>>(p);
  return cudaPeekAtLastError() == cudaSuccess ? 0 : -1;
}

// Pages are copied 16 bytes a thread, four loads ahead of their stores.  The pairs are kernel
// arguments: the call needs no host-to-device copy, keeps nothing after it returns, and can be
// captured.
template <int N>
__global__ void __launch_bounds__(256) kv4_copy_kernel(uint8_t* pool, long long layer_bytes, long long page_bytes,
                                                       const __grid_constant__ Kv4Pairs<N> pairs) {
  const int2 pr = pairs.at[blockIdx.y];
  uint8_t* layer = pool + (size_t)blockIdx.z * layer_bytes;
  const uint4* src = reinterpret_cast<const uint4*>(layer + (size_t)pr.x * page_bytes);
  uint4* dst = reinterpret_cast<uint4*>(layer + (size_t)pr.y * page_bytes);
  const long long n = page_bytes / 16, step = (long long)gridDim.x * 256;
  long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  for (; i + 3 * step < n; i += 4 * step) {
    const uint4 a = __ldg(src + i), b = __ldg(src + i + step), c = __ldg(src + i + 2 * step),
                d = __ldg(src + i + 3 * step);
    dst[i] = a;
    dst[i + step] = b;
    dst[i + 2 * step] = c;
    dst[i + 3 * step] = d;
  }
  for (; i < n; i += step) dst[i] = __ldg(src + i);
}

template <int N>
static int copy_some(uint8_t* pool, int n_layers, long long layer_bytes, long long page_bytes, const int* src,
                     const int* dst, int n, cudaStream_t stream) {
  Kv4Pairs<N> pairs;
  for (int i = 0; i < n; ++i) pairs.at[i] = make_int2(src[i], dst[i]);
  const long long units = page_bytes / 16;
  const unsigned gx = (unsigned)((units + 1023) / 1024 < 64 ? (units + 1023) / 1024 : 64);
  kv4_copy_kernel<N><<<dim3(gx, n, n_layers), 256, 0, stream>>>(pool, layer_bytes, page_bytes, pairs);
  return cudaPeekAtLastError() == cudaSuccess ? 0 : -1;
}

int launch_kv4_copy(uint8_t* pool, int n_layers, long long layer_bytes, long long page_bytes, const int* src,
                    const int* dst, int n, cudaStream_t stream) {
  int rc = 0;
  for (int a = 0; a < n && rc == 0; a += kKv4PairsMax) {
    const int m = n - a < kKv4PairsMax ? n - a : kKv4PairsMax;
    rc = m <= kKv4PairsFew
             ? copy_some<kKv4PairsFew>(pool, n_layers, layer_bytes, page_bytes, src + a, dst + a, m, stream)
             : copy_some<kKv4PairsMax>(pool, n_layers, layer_bytes, page_bytes, src + a, dst + a, m, stream);
  }
  return rc;
}

}  // namespace sdpa
