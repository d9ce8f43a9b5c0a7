// kv4_tree.cu -- attention of the nodes of drafted trees over a sequence's 4-bit paged cache
// (layout and number format in kv4.cuh).
//
//   Node i of a sequence with L tokens before its tree is its token L + i, at position L + depth(i).
//   S_j = scale q.k_j over the tokens j < L, the node's ancestors and itself, under a window only
//   those of the last window + 1 positions; softmax with an optional sink logit; o = P V.
//
// All nodes and all query heads of a kv head share every byte of the cache: n G rows.  Up to about 64 rows
// the call is bound by reading the cache, from 128 on by the tensor cores, so the products run there:
//   - A unit is 128 tokens of one sequence and kv head.  A producer warp streams its pages' blocks into
//     shared memory; eight warps decode K and V into bf16 operand tiles (128-byte swizzle, a lane's
//     16-byte stores of a quarter warp on different banks); one warp issues S = Q K^T and O += P V
//     (tcgen05, 128 rows a tile); two warpgroups take the softmax, a thread a row, with P back into
//     TMEM where S was.
//   - Codes are decoded as (c - 8) s 2^-23 (kv4.cuh), exact; the power of two is undone in the scores'
//     scale and in the outputs.  Eight dims of a word come out in the order 0 4 1 5 2 6 3 7: Q is
//     laid out alike, and the outputs are put back when they are stored.
//   - Up to 128 rows: one row tile, whose even units one warpgroup takes and whose odd units the
//     other, each with its own sums, joined at the end.  More rows: two row tiles that share the
//     decoded operands (a tile of its own would decode the cache again).
//   - Work is cut evenly over a persistent grid, whatever the lengths (units of one sequence, kv head
//     and row block in order, and kSegCost units more for each such segment); a segment that spans
//     several CTAs leaves fp32 partial sums in the workspace, joined in CTA order by a second kernel:
//     bitwise reproducible.
//   - The probabilities are rounded to bf16 (2^-9 relative) for P V; their sum is fp32.
#include <algorithm>
#include <atomic>

#include "attn_common.cuh"
#include "attn_kernels.h"
#include "kv4.cuh"
#include "launch.h"
#include "ptx.cuh"

namespace sdpa {

namespace {

constexpr int kUnit = 128;    // tokens of a unit
constexpr int kMaxGrid = 152;  // CTAs, and pairs of partial sums in the workspace
constexpr int kSegCost = 2;   // a segment's fixed costs, in units
constexpr int kDecWarps = 8;
constexpr int kThreads = 32 * (8 + kDecWarps + 4);  // (the last two warps have nothing to do: registers are split by fours)
// Registers a thread of the launch, and after the split: softmax, decoding, the rest.
constexpr int kRegs = 96, kRegsSoft = 136, kRegsDec = 72, kRegsRest = 64;
static_assert(256 * kRegsSoft + 256 * kRegsDec + 128 * kRegsRest <= kThreads * kRegs, "the launch's registers");

enum TreeSite { kTreeRawFull = 0xB0, kTreeRawEmpty, kTreeKFull, kTreeKEmpty, kTreeVFull, kTreeVEmpty, kTreeQFull, kTreeQEmpty,
                kTreeS, kTreeP, kTreeO, kTreeDrain };

template <int D, bool TWO>
struct TreeCfg {
  static constexpr int ROWS = TWO ? 256 : 128;  // rows of a block
  static constexpr int BLK = 128 * 128;         // one operand block: 128 rows of 64 bf16
  static constexpr int TILE = BLK * (D / 64);
  static constexpr int NK = 2, NV = TWO ? 1 : 2;
  static constexpr int STAGES = D == 128 ? 3 : 6;
  static constexpr int STAGE = kUnit * D * 9 / 8;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = OFF_Q + (TWO ? 2 : 1) * TILE;
  static constexpr int OFF_V = OFF_K + NK * TILE;
  static constexpr int OFF_RAW = OFF_V + NV * TILE;
  static constexpr int OFF_NAN = OFF_RAW + STAGES * STAGE;  // [NV][D / 16][64] bits of the two tokens of a pair
  static constexpr int OFF_ML = OFF_NAN + NV * D / 16 * 64;  // [2][128] maxima, sums, NaN groups
  static constexpr int OFF_BAR = OFF_ML + 3 * 2 * 128 * 4;
  static constexpr int N_BAR = 2 * STAGES + 2 * NK + 2 * NV + 2 + 6 + 1;
  static constexpr int OFF_SLOT = OFF_BAR + N_BAR * 8;
  static constexpr int SMEM = OFF_SLOT + 16 + 1024;  // (aligned by the kernel)
  static constexpr int PART = ROWS * (D + 2);        // floats of one partial: sums, maxima, denominators
  static_assert(SMEM <= 232448, "shared memory budget");
  static_assert(SMEM > 116 * 1024, "one CTA per SM keeps the 512-column TMEM allocation uncontended");
};

// A sequence's sizes.
struct TreeSeq {
  int row0, n;   // its rows of q
  int L, len;    // tokens before the tree, and all (as far as the table goes)
  int lo, first;  // first token some node sees, its unit
  int units, blocks;
  __device__ __forceinline__ int seg() const { return units > 0 ? units + kSegCost : 0; }
};
template <int ROWS>
__device__ __forceinline__ TreeSeq tree_seq(const Kv4TreeParams& p, int b) {
  TreeSeq s;
  const int cap = p.c.max_pages * p.c.page_size, a = max(__ldg(p.cu + b), 0), z = min(__ldg(p.cu + b + 1), p.T);
  s.row0 = a;
  s.n = max(z - a, 0);
  s.L = entry_len(p.start, b, cap);
  s.len = (int)min((long long)s.L + s.n, (long long)cap);
  s.lo = p.window >= 0 && s.L > p.window ? s.L - p.window : 0;
  s.first = s.lo / kUnit;
  s.units = s.n > 0 && s.len > 0 ? max((s.len - 1) / kUnit - s.first + 1, 0) : 0;
  s.blocks = (int)(((long long)s.n * (p.H_q / p.c.H_kv) + ROWS - 1) / ROWS);
  return s;
}
// Units that row block rb of the sequence needs: up to its last node's own token.
template <int ROWS>
__device__ __forceinline__ int block_units(const Kv4TreeParams& p, const TreeSeq& s, int rb) {
  const int G = p.H_q / p.c.H_kv;
  const int last = (int)min((long long)s.n - 1, (((long long)rb + 1) * ROWS - 1) / G);
  const int len = (int)min((long long)s.L + last + 1, (long long)s.len);
  return max((len - 1) / kUnit - s.first + 1, 0);
}

// How the units of a call are numbered: sequence by sequence, in it kv head by kv head, in it row
// block by row block; each such segment has units + kSegCost numbers, the first kSegCost for its
// fixed costs.  Every warp works this out for itself.
template <int ROWS>
struct TreeScan {
  __device__ __forceinline__ static long long numbers(const Kv4TreeParams& p, int b) {
    if (b >= p.B) return 0;
    const TreeSeq s = tree_seq<ROWS>(p, b);
    return (long long)s.seg() * s.blocks * p.c.H_kv;
  }
  __device__ static long long sum(const Kv4TreeParams& p, int end) {
    long long t = 0;
    for (int b = threadIdx.x % 32; b < end; b += 32) t += numbers(p, b);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
    return t;
  }
  // The sequence that holds number u (below the total); the numbers before it are returned.
  __device__ static long long find(const Kv4TreeParams& p, long long u, int* b) {
    const int lane = threadIdx.x % 32;
    long long carry = 0;
    for (int base = 0;; base += 32) {
      const long long m = numbers(p, base + lane);
      long long s = m;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, s, off);
        if (lane >= off) s += o;
      }
      s += carry;
      const unsigned holds = __ballot_sync(0xffffffffu, u < s);
      if (holds || base + 32 >= p.B) {
        const int w = holds ? __ffs(holds) - 1 : 0;
        *b = base + w;
        return __shfl_sync(0xffffffffu, s - m, w);
      }
      carry = __shfl_sync(0xffffffffu, s, 31);
    }
  }
};

// CTA c of n takes numbers [tree_cut(c), tree_cut(c + 1)).
__device__ __forceinline__ long long tree_cut(long long total, int n, int c) { return total * c / n; }
__device__ __forceinline__ int tree_cta_of(long long total, int n, long long u) {
  int c = (int)min((long long)n - 1, u * n / total);
  while (c > 0 && tree_cut(total, n, c) > u) --c;
  while (c + 1 < n && tree_cut(total, n, c + 1) <= u) ++c;
  return c;
}
__device__ __forceinline__ int tree_ctas(long long total, int grid) {
  const long long want = (total + kSegCost) / (kSegCost + 1);
  return want < grid ? (int)want : grid;
}

// A CTA's run of segments.
template <int ROWS>
struct TreeWalk {
  int b, vh;           // sequence; kv head and row block in it
  int from, to;        // this CTA's units of the segment
  long long left;      // numbers of this CTA after it
  TreeSeq s;
  __device__ __forceinline__ int segments(const Kv4TreeParams& p) const { return p.c.H_kv * s.blocks; }
  __device__ __forceinline__ int hk() const { return vh / s.blocks; }
  __device__ __forceinline__ int rb() const { return vh % s.blocks; }
  __device__ __forceinline__ void enter(int number) {
    const int take = (int)min((long long)(s.seg() - number), left);
    from = max(number - kSegCost, 0);
    to = max(number + take - kSegCost, 0);
    left -= take;
  }
  __device__ __forceinline__ void begin(const Kv4TreeParams& p, long long u_begin, long long u_end) {
    const long long r = u_begin - TreeScan<ROWS>::find(p, u_begin, &b);
    s = tree_seq<ROWS>(p, b);
    vh = (int)(r / s.seg());
    left = u_end - u_begin;
    enter((int)(r % s.seg()));
  }
  // To the next segment of which this CTA has units; false: none.
  __device__ __forceinline__ bool settle(const Kv4TreeParams& p) {
    while (from == to) {
      if (left == 0) return false;
      next(p);
    }
    return true;
  }
  __device__ __forceinline__ void next(const Kv4TreeParams& p) {
    if (++vh == segments(p)) {
      vh = 0;
      do {
        ++b;
        s = tree_seq<ROWS>(p, b);
      } while (s.units == 0);
    }
    enter(0);
  }
  __device__ __forceinline__ bool advance(const Kv4TreeParams& p) {
    if (left == 0) return false;
    next(p);
    return settle(p);
  }
  // This CTA's units that the segment's row block needs.
  __device__ __forceinline__ int count(const Kv4TreeParams& p) const {
    return max(min(to, block_units<ROWS>(p, s, rb())) - from, 0);
  }
};

__device__ __forceinline__ int tree_parent(const Kv4TreeParams& p, const TreeSeq& s, int i) {
  if (!p.parents) return i - 1;
  const int a = __ldg(p.parents + s.row0 + i);
  return a < i && a >= 0 ? a : -1;
}

template <int N>
__device__ __forceinline__ void regs_less() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_more() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// bits [from, to) of the 128 tokens of a unit
__device__ __forceinline__ void set_range(uint32_t (&vis)[4], int from, int to) {
  from = max(from, 0);
  to = min(to, kUnit);
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const int a = max(from - 32 * w, 0), z = min(to - 32 * w, 32);
    if (a < z) vis[w] |= (0xffffffffu << a) & (0xffffffffu >> (32 - z));
  }
}

// A row's end: its sums relative to maximum m (log2 units), the sink joins the denominator.
struct TreeSums {
  float mul, lse;  // what the sums are multiplied by; log of the denominator
};
__device__ __forceinline__ TreeSums tree_finish(const Kv4TreeParams& p, int h, float m, float l) {
  const float sink = p.softmax_type == 0 ? -INFINITY : p.softmax_type == 1 ? 0.f : p.offset[h] * kLog2e;
  const float mm = fmaxf(m, sink);
  if (mm == -INFINITY) return l == l ? TreeSums{0.f, -INFINITY} : TreeSums{l, l};  // no key (l is 0) or a NaN
  const float f = m == -INFINITY ? (l == l ? 0.f : l) : ex2(m - mm);
  const float den = (m == -INFINITY ? f : l * f) + (sink == -INFINITY ? 0.f : ex2(sink - mm));
  return TreeSums{f / den * kKv4SmallUndo, (mm + lg2(den)) * kLn2};
}

// 8 dims of a code word as bf16, in the order 0 4 1 5 2 6 3 7
__device__ __forceinline__ uint4 decode8(uint32_t w, const Kv4Small& k) {
  const uint32_t w8 = w >> 8;
  return make_uint4(decode_small_lo(w, k), decode_small_hi(w, k), decode_small_lo(w8, k), decode_small_hi(w8, k));
}
__device__ __forceinline__ Kv4Small scales_low(uint32_t pair) { return small_scales(__byte_perm(pair, 0u, 0x1010)); }
__device__ __forceinline__ Kv4Small scales_high(uint32_t pair) { return small_scales(__byte_perm(pair, 0u, 0x3232)); }

// columns of 8 output dims back in order, as bf16
__device__ __forceinline__ uint4 ordered8(const float* v) {
  return make_uint4(pack_bf16x2(v[0], v[2]), pack_bf16x2(v[4], v[6]), pack_bf16x2(v[1], v[3]), pack_bf16x2(v[5], v[7]));
}

}  // namespace

template <int D, bool TWO>
__global__ void __launch_bounds__(kThreads, 1) kv4_tree_kernel(const Kv4TreeParams p, float* partial) {
  using C = TreeCfg<D, TWO>;
  using Walk = TreeWalk<C::ROWS>;
  constexpr int NST = C::STAGES, NK = C::NK, NV = C::NV;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint64_t* raw_full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* raw_empty = raw_full + NST;
  uint64_t* k_full = raw_empty + NST;
  uint64_t* k_empty = k_full + NK;
  uint64_t* v_full = k_empty + NK;
  uint64_t* v_empty = v_full + NV;
  uint64_t* q_full = v_empty + NV;
  uint64_t* q_empty = q_full + 1;
  uint64_t* s_ready = q_empty + 1;  // [2]
  uint64_t* p_ready = s_ready + 2;
  uint64_t* o_done = p_ready + 2;
  uint64_t* mma_done = o_done + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_SLOT);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  int* err = p.err;

  grid_launch_dependents();  // the join may be set up meanwhile
  const long long total = TreeScan<C::ROWS>::sum(p, p.B);
  if (total == 0) return;
  const int n_cta = tree_ctas(total, gridDim.x);
  if ((int)blockIdx.x >= n_cta) return;
  if (threadIdx.x == 0) {
    for (int s = 0; s < NST; ++s) {
      mbar_init(&raw_full[s], 1);
      mbar_init(&raw_empty[s], kDecWarps);
    }
    for (int s = 0; s < NK; ++s) {
      mbar_init(&k_full[s], kDecWarps);
      mbar_init(&k_empty[s], 1);
    }
    for (int s = 0; s < NV; ++s) {
      mbar_init(&v_full[s], kDecWarps);
      mbar_init(&v_empty[s], 1);
    }
    mbar_init(q_full, kDecWarps);
    mbar_init(q_empty, 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(&s_ready[t], 1);
      mbar_init(&p_ready[t], 128);
      mbar_init(&o_done[t], 1);
    }
    mbar_init(mma_done, 1);
    fence_barrier_init();
  }
  if (warp == 16) {
    tmem_alloc<512>(tmem_slot);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int G = p.H_q / p.c.H_kv;
  Walk at;
  at.begin(p, tree_cut(total, n_cta, blockIdx.x), tree_cut(total, n_cta, blockIdx.x + 1));
  bool ok = true;

  if (warp >= 16) regs_less<kRegsRest>();
  if (warp == 17) {
    // ---------------------------------------------------------------- producer
    // Lane i copies the block of page i of a unit (whole, also past the sequence's end), if some node
    // sees a token of it: the pages before a window may be gone from the table.  Its page is looked up one
    // unit ahead.
    const int P = p.c.page_size, pieces = kUnit / P, t0 = lane * P;
    const int block = kv4_block_bytes(P, D);
    const size_t page_bytes = (size_t)block * p.c.H_kv;
    bool more = at.settle(p);
    int k = 0, cnt = more ? at.count(p) : 0;
    auto skip = [&]() {  // to the next unit there is
      while (more && k >= cnt) {
        more = at.advance(p);
        k = 0;
        cnt = more ? at.count(p) : 0;
      }
    };
    auto page_of = [&]() {
      const long long tok = (long long)(at.s.first + at.from + k) * kUnit + t0;
      return lane < pieces && tok < at.s.len && tok + P > at.s.lo ? kv4_page(p.c, at.b, (int)tok) : -2;
    };
    skip();
    int page = more ? page_of() : -2, n = 0;
    for (; more && ok; ++n) {
      const int stage = n % NST;
      uint8_t* st = smem + C::OFF_RAW + stage * C::STAGE;
      const uint8_t* src = p.pool + (size_t)max(page, 0) * page_bytes + (size_t)at.hk() * block;
      const int have = page;
      ++k;
      skip();
      if (more) page = page_of();
      if (n >= NST) ok = mbar_wait_warp(&raw_empty[stage], (n / NST - 1) & 1, err, kTreeRawEmpty);
      if (!ok) break;
      if (__any_sync(0xffffffffu, have == -1)) {  // not a page: its tokens read as zeros (scale 0)
        if (have == -1) {
          for (int o = kv4_off_sk(P, D); o < block; o += 16)
            *reinterpret_cast<uint4*>(st + lane * block + o) = make_uint4(0u, 0u, 0u, 0u);
          atomicCAS(p.page_err, 0, p.site);
          fence_proxy_async_smem();
        }
        __syncwarp();
      }
      const uint32_t all = __popc(__ballot_sync(0xffffffffu, have >= 0)) * block;
      if (lane == 0) mbar_arrive_expect_tx(&raw_full[stage], all);
      __syncwarp();
      if (have >= 0) bulk_load(st + lane * block, src, block, &raw_full[stage]);
    }
    // every copy this warp started must land before the CTA may exit: wait for the last ones
    for (int s = 0; s < NST && s < n; ++s) {
      const int last = s + (n - 1 - s) / NST * NST;
      mbar_wait_warp(&raw_full[s], (last / NST) & 1, err, kTreeDrain);
    }
  } else if (warp == 16) {
    // ---------------------------------------------------------------- MMA issuer
    constexpr uint32_t idS = idesc_bf16_f32(128, 128, false, false), idO = idesc_bf16_f32(128, D, false, true);
    const uint32_t sQ = smem_u32(smem + C::OFF_Q), sK = smem_u32(smem + C::OFF_K), sV = smem_u32(smem + C::OFF_V);
    auto issue_S = [&](int t, int stage) {
      const uint64_t dq = smem_desc_sw128(sQ + (TWO ? t * C::TILE : 0), 16, 1024);
      const uint64_t dk = smem_desc_sw128(sK + stage * C::TILE, 16, 1024);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = (kk / 4) * C::BLK + (kk % 4) * 32;
        mma_ss_warp(tmem + t * 256, desc_add(dq, off), desc_add(dk, off), idS, kk > 0);
      }
      mma_commit_warp(&s_ready[t]);
    };
    auto issue_PV = [&](int t, int stage, bool acc) {
      const uint64_t dv = smem_desc_sw128(sV + stage * C::TILE, C::BLK, 1024);
#pragma unroll
      for (int kk = 0; kk < kUnit / 16; ++kk)
        mma_ts_warp(tmem + t * 256 + 128, tmem + t * 256 + kk * 8, desc_add(dv, kk * 2048), idO, (acc || kk > 0) ? 1u : 0u);
    };
    int nq = 0, nk = 0, nv = 0, np[2] = {0, 0};  // phases consumed
    bool issued = false;
    auto wait_K = [&]() {
      ok = ok && mbar_wait_warp(&k_full[nk % NK], (nk / NK) & 1, err, kTreeKFull);
      if (ok) tc_fence_after();
      return ok;
    };
    for (bool more = at.settle(p); more && ok; more = at.advance(p)) {
      const int cnt = at.count(p);
      if (cnt == 0) continue;
      ok = mbar_wait_warp(q_full, nq++ & 1, err, kTreeQFull);
      if (!ok) break;
      issued = true;
      if constexpr (TWO) {
        if (!wait_K()) break;
        issue_S(0, nk % NK);
        issue_S(1, nk % NK);
        mma_commit_warp(&k_empty[nk++ % NK]);
        if (cnt == 1) mma_commit_warp(q_empty);
        for (int k = 0; k < cnt && ok; ++k) {
          const bool need_k = k + 1 < cnt;
          ok = mbar_wait_warp(&v_full[nv % NV], (nv / NV) & 1, err, kTreeVFull);
          if (ok && need_k) wait_K();
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            ok = ok && mbar_wait_warp(&p_ready[t], np[t] & 1, err, kTreeP);
            if (!ok) break;
            ++np[t];
            tc_fence_after();
            issue_PV(t, nv % NV, k > 0);
            if (!need_k) mma_commit_warp(&o_done[t]);
            else issue_S(t, nk % NK);
          }
          if (!ok) break;
          mma_commit_warp(&v_empty[nv++ % NV]);
          if (need_k) mma_commit_warp(&k_empty[nk++ % NK]);
          if (k + 2 == cnt) mma_commit_warp(q_empty);  // every S of the segment is issued
        }
      } else {
        for (int k = 0; k < min(cnt, 2); ++k) {
          if (!wait_K()) break;
          issue_S(k, nk % NK);
          mma_commit_warp(&k_empty[nk++ % NK]);
        }
        if (!ok) break;
        if (cnt <= 2) mma_commit_warp(q_empty);
        for (int k = 0; k < cnt; ++k) {
          const int t = k & 1;
          ok = mbar_wait_warp(&v_full[nv % NV], (nv / NV) & 1, err, kTreeVFull);
          ok = ok && mbar_wait_warp(&p_ready[t], (t ? np[1] : np[0]) & 1, err, kTreeP);
          if (!ok) break;
          if (t) ++np[1];
          else ++np[0];
          tc_fence_after();
          issue_PV(t, nv % NV, k > 1);
          mma_commit_warp(&v_empty[nv++ % NV]);
          if (k + 2 >= cnt) {
            mma_commit_warp(&o_done[t]);
            continue;
          }
          if (!wait_K()) break;
          issue_S(t, nk % NK);
          mma_commit_warp(&k_empty[nk++ % NK]);
          if (k + 3 == cnt) mma_commit_warp(q_empty);
        }
      }
    }
    // every MMA must be complete before TMEM is released
    if (issued) {
      mma_commit_warp(mma_done);
      mbar_wait_warp(mma_done, 0, err, kTreeDrain);
    }
  } else if (warp >= 8 && warp < 16) {
    // ---------------------------------------------------------------- decoding warps
    regs_less<kRegsDec>();
    const int tid = threadIdx.x - 256, P = p.c.page_size, block = kv4_block_bytes(P, D);
    constexpr int KI = D / 64, VI = D / 64;  // 16-byte pieces of K, of V a thread takes of a unit
    int k_code[KI], k_scale[KI], k_dst[KI], v_code[VI], v_scale[VI], v_dst[VI], v_tok[VI], v_flip[VI];
    bool k_swap[KI];
#pragma unroll
    for (int i = 0; i < KI; ++i) {
      // 32 dims q of a token.  Lanes of dims 64.. store their pieces two further on: the quarter warp's
      // eight stores then fall on eight different banks groups
      const int e = i * 256 + tid, tok = e / (D / 32), q = e % (D / 32), w = tok & (P - 1), base = tok / P * block;
      k_code[i] = base + w * (D / 2) + q * 16;
      k_scale[i] = base + kv4_off_sk(P, D) + w * (D / 16) + q * 2;
      k_dst[i] = (q / 2) * C::BLK + tok * 128 + ((((q & 1) * 4) ^ (tok & 7)) << 4);
      k_swap[i] = q >= 2;
    }
#pragma unroll
    for (int i = 0; i < VI; ++i) {
      // 16 dims (group g) of a pair of tokens
      const int e = i * 256 + tid, u = e / (D / 16), s = e % (D / 16), w = 2 * u & (P - 1), base = 2 * u / P * block;
      const int x = kv4_slot_xor(w / 2, D), g = D == 128 ? s ^ x : s ^ (x >> 1);
      v_code[i] = base + kv4_off_v(P, D) + (w / 2) * D + s * 16;
      v_scale[i] = base + kv4_off_sv(P, D) + (w / 2) * (D / 8) + 2 * g;
      v_tok[i] = 2 * u;
      v_dst[i] = g;
      v_flip[i] = D == 128 ? g / 4 : u & 1;  // which of the two pieces is stored first: different banks again
    }
    int nq = 0, n = 0;
    for (bool more = at.settle(p); more && ok; more = at.advance(p)) {
      const int cnt = at.count(p);
      if (cnt == 0) continue;
      // ---- Q: loaded while the segment before is still computed, stored when its last scores are done
      {
        constexpr int QI = C::ROWS * (D / 8) / 256, QB = QI < 8 ? QI : 8;
        const int R = (int)min((long long)at.s.n * G - (long long)at.rb() * C::ROWS, (long long)C::ROWS);
        const long long r0 = (long long)at.rb() * C::ROWS;
        const int hk = at.hk();
#pragma unroll 1
        for (int i0 = 0; i0 < QI; i0 += QB) {
          uint4 w[QB];
#pragma unroll
          for (int i = 0; i < QB; ++i) {
            const int e = (i0 + i) * 256 + tid, r = e / (D / 8), c = e % (D / 8);
            w[i] = make_uint4(0u, 0u, 0u, 0u);
            if (r < R) {
              const long long rr = r0 + r, node = rr / G;
              w[i] = __ldg(reinterpret_cast<const uint4*>(
                  p.q + ((size_t)(at.s.row0 + node) * p.H_q + (size_t)hk * G + (rr - node * G)) * D + c * 8));
            }
          }
          if (i0 == 0 && nq > 0) {
            ok = mbar_wait_warp(q_empty, (nq - 1) & 1, err, kTreeQEmpty);
            if (!ok) break;
          }
#pragma unroll
          for (int i = 0; i < QB; ++i) {
            const int e = (i0 + i) * 256 + tid, r = e / (D / 8), c = e % (D / 8), rt = r % 128;
            uint8_t* dst = smem + C::OFF_Q + (r / 128) * C::TILE + (c / 8) * C::BLK + rt * 128 + (((c % 8) ^ (rt & 7)) << 4);
            *reinterpret_cast<uint4*>(dst) =
                make_uint4(__byte_perm(w[i].x, w[i].z, 0x5410), __byte_perm(w[i].x, w[i].z, 0x7632),
                           __byte_perm(w[i].y, w[i].w, 0x5410), __byte_perm(w[i].y, w[i].w, 0x7632));
          }
        }
        if (!ok) break;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full);
        ++nq;
      }
      // units whose tokens are not all seen by all rows, as the softmax warps decide it
      long long k0 = (long long)(at.s.first + at.from) * kUnit;
      for (int k = 0; k < cnt; ++k, ++n, k0 += kUnit) {
        const int stage = n % NST, sk = n % NK, sv = n % NV;
        const uint8_t* st = smem + C::OFF_RAW + stage * C::STAGE;
        ok = mbar_wait_warp(&raw_full[stage], (n / NST) & 1, err, kTreeRawFull);
        if (ok && n >= NK) ok = mbar_wait_warp(&k_empty[sk], (n / NK - 1) & 1, err, kTreeKEmpty);
        if (!ok) break;
        uint8_t* kd = smem + C::OFF_K + sk * C::TILE;
#pragma unroll
        for (int i = 0; i < KI; ++i) {
          uint4 w = *reinterpret_cast<const uint4*>(st + k_code[i]);
          const uint32_t sp = scale_pair(*reinterpret_cast<const unsigned short*>(st + k_scale[i]));
          Kv4Small a = scales_low(sp), b = scales_high(sp);
          // words 0, 1 share the first scale, 2, 3 the second; word c goes to piece c
          if (k_swap[i]) {
            w = make_uint4(w.z, w.w, w.x, w.y);
            const Kv4Small t = a;
            a = b;
            b = t;
          }
          uint8_t* d = kd + k_dst[i];
          const int x = k_swap[i] ? 32 : 0;  // piece c ^ 2 first
          // (the destination's piece number is k_dst's exclusive-or c: c lies in its low two bits)
          uint8_t* base = reinterpret_cast<uint8_t*>(reinterpret_cast<uintptr_t>(d) & ~(uintptr_t)127);
          const int at16 = (int)(reinterpret_cast<uintptr_t>(d) & 127);
          *reinterpret_cast<uint4*>(base + (at16 ^ x)) = decode8(w.x, a);
          *reinterpret_cast<uint4*>(base + (at16 ^ x ^ 16)) = decode8(w.y, a);
          *reinterpret_cast<uint4*>(base + (at16 ^ x ^ 32)) = decode8(w.z, b);
          *reinterpret_cast<uint4*>(base + (at16 ^ x ^ 48)) = decode8(w.w, b);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&k_full[sk]);
        if (n >= NV) ok = mbar_wait_warp(&v_empty[sv], (n / NV - 1) & 1, err, kTreeVEmpty);
        if (!ok) break;
        const bool edge = k0 + kUnit > at.s.L || (p.window >= 0 && k0 < (long long)at.s.L + at.s.n - 1 - p.window);
        uint8_t* vd = smem + C::OFF_V + sv * C::TILE;
        uint4 w[VI];
        uint32_t two[VI];
#pragma unroll
        for (int i = 0; i < VI; ++i) {
          w[i] = *reinterpret_cast<const uint4*>(st + v_code[i]);
          two[i] = *reinterpret_cast<const unsigned short*>(st + v_scale[i]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&raw_empty[stage]);  // the stage is read
#pragma unroll
        for (int i = 0; i < VI; ++i) {
          const int g = v_dst[i], tok = v_tok[i];
          if (edge) {
            // A token that no row sees adds nothing, whatever its bytes are.  One held as NaN adds nothing
            // either: rows that do not see it have P = 0, but 0 times NaN is NaN.  The rows that see it
            // learn of it from these bits.
            uint32_t bits = 0u;
            if (k0 + tok >= at.s.len || k0 + tok < at.s.lo) two[i] &= 0xFF00u;
            if (k0 + tok + 1 >= at.s.len || k0 + tok + 1 < at.s.lo) two[i] &= 0x00FFu;
            if ((two[i] & 0x00F8u) == 0x00F8u) {
              bits |= 1u;
              two[i] &= 0xFF00u;
            }
            if ((two[i] & 0xF800u) == 0xF800u) {
              bits |= 2u;
              two[i] &= 0x00FFu;
            }
            smem[C::OFF_NAN + (sv * (D / 16) + g) * 64 + tok / 2] = (uint8_t)bits;
          }
          const uint32_t sp = scale_pair(two[i]);
          const Kv4Small a = scales_low(sp), b = scales_high(sp);
          uint8_t* d = vd + (g / 4) * C::BLK + tok * 128;
          const int c0 = 2 * (g % 4), fl = v_flip[i];
          // (D = 128: 8 bytes a token; D = 64: the two eighths' 4 bytes a token)
          const uint32_t t0w0 = w[i].x, t0w1 = D == 128 ? w[i].y : w[i].z, t1w0 = D == 128 ? w[i].z : w[i].y, t1w1 = w[i].w;
          const int r0 = tok & 7, r1 = (tok + 1) & 7;
          *reinterpret_cast<uint4*>(d + (((c0 + fl) ^ r0) << 4)) = decode8(fl ? t0w1 : t0w0, a);
          *reinterpret_cast<uint4*>(d + (((c0 + 1 - fl) ^ r0) << 4)) = decode8(fl ? t0w0 : t0w1, a);
          *reinterpret_cast<uint4*>(d + 128 + (((c0 + fl) ^ r1) << 4)) = decode8(fl ? t1w1 : t1w0, b);
          *reinterpret_cast<uint4*>(d + 128 + (((c0 + 1 - fl) ^ r1) << 4)) = decode8(fl ? t1w0 : t1w1, b);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&v_full[sv]);
      }
    }
  } else if (warp < 8) {
    // ---------------------------------------------------------------- softmax and output
    regs_more<kRegsSoft>();
    const int t = warp / 4, r = (warp % 4) * 32 + lane;
    const uint32_t lane_addr = tmem + ((uint32_t)((warp % 4) * 32) << 16);
    const uint32_t colS = t * 256, colO = t * 256 + 128;
    const float sl2 = p.scale_log2 * kKv4SmallUndo;
    float* xm = reinterpret_cast<float*>(smem + C::OFF_ML);  // [2][128] maxima, sums, NaN groups of the two halves
    float* xl = xm + 256;
    uint32_t* xn = reinterpret_cast<uint32_t*>(xl + 256);
    int ns = 0, no[2] = {0, 0}, n_seg0 = 0;  // s_ready and o_done phases consumed; units of the segments before
    bool at_begin = true;
    for (bool more = at.settle(p); more && ok; more = at.advance(p), at_begin = false) {
      const int cnt = at.count(p);
      const bool whole = at.from == 0 && at.to == at.s.units;
      const int hk = at.hk();
      const long long r_all = (long long)at.rb() * C::ROWS + (TWO ? t * 128 : 0) + r;  // this thread's row of the kv head
      const bool row_ok = r_all < (long long)at.s.n * G;
      const bool warp_ok = r_all - lane < (long long)at.s.n * G;
      const int node = row_ok ? (int)(r_all / G) : at.s.n - 1, h = hk * G + (row_ok ? (int)(r_all % G) : 0);
      const int L = at.s.L;
      int lo_row = 0;  // first token before the tree that this row sees
      if (p.window >= 0) {
        int depth = 0;
        if (p.parents) {
          for (int a = tree_parent(p, at.s, node); a >= 0; a = tree_parent(p, at.s, a)) ++depth;
        } else {
          depth = node;
        }
        lo_row = (int)min(max((long long)L + depth - p.window, 0LL), 0x7fffffffLL);
      }
      float m_run = -INFINITY, l = 0.f;
      uint32_t nans = 0u;  // groups of 16 dims in which this row sees a NaN
      long long k0 = (long long)(at.s.first + at.from + (TWO ? 0 : t)) * kUnit;
      bool first = true;
      for (int k = TWO ? 0 : t; k < cnt; k += TWO ? 1 : 2, k0 += TWO ? kUnit : 2 * kUnit) {
        const bool edge = k0 + kUnit > L || (p.window >= 0 && k0 < (long long)L + at.s.n - 1 - p.window);
        uint32_t vis[4] = {0u, 0u, 0u, 0u};
        if (edge && warp_ok) {
          set_range(vis, (int)max((long long)lo_row - k0, 0LL), (int)min((long long)L - k0, (long long)kUnit));
          const long long a0 = k0 - L;  // the node at the unit's first token
          if (!p.parents) {
            const long long from = p.window >= 0 ? max((long long)node - p.window, 0LL) : 0;
            set_range(vis, (int)min(max(max(from, 0LL) - a0, 0LL), (long long)kUnit),
                      (int)min(min((long long)node + 1, (long long)at.s.len - L) - a0, (long long)kUnit));
          } else {
            int step = 0;
            for (int a = node; a >= 0 && a >= a0 && (p.window < 0 || step <= p.window); a = tree_parent(p, at.s, a), ++step) {
              const long long j = a - a0;
              if (j < kUnit && L + a < at.s.len) {
#pragma unroll
                for (int w = 0; w < 4; ++w)
                  if ((int)j / 32 == w) vis[w] |= 1u << ((int)j & 31);
              }
            }
          }
        }
        ok = mbar_wait_warp(&s_ready[t], ns & 1, err, kTreeS);
        ++ns;
        if (!ok) break;
        if (!warp_ok) {  // no row of this warp exists: its P may be anything
          mbar_arrive(&p_ready[t]);
          first = false;
          continue;
        }
        tc_fence_after();
        float mx = -INFINITY;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t s[32];
          float cm;
          tmem_ld32_max(lane_addr + colS + 32 * c, s, cm);
          tmem_ld_wait();
          if (edge) {
            cm = -INFINITY;
#pragma unroll
            for (int e = 0; e < 32; ++e) cm = fmaxf(cm, vis[c] >> e & 1u ? __uint_as_float(s[e]) : -INFINITY);
          }
          mx = fmaxf(mx, cm);
        }
        const float m_tile = mx * sl2;
        // The running maximum (log2 units) moves only when some row of the warp passes it by 2^8; the
        // sums stay exact, they are relative to the maximum that was used.
        if (__any_sync(0xffffffffu, m_tile > m_run + 8.f)) {
          const float m_new = fmaxf(m_run, m_tile);
          const float alpha = m_new == m_run ? 1.f : ex2(m_run - m_new);
          l *= alpha;
          if (!first) {
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 16) {
              uint32_t o[16];
              tmem_ld16(lane_addr + colO + c0, o);
              tmem_ld_wait();
#pragma unroll
              for (int c = 0; c < 16; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
              tmem_st16(lane_addr + colO + c0, o);
            }
          }
          m_run = m_new;
        }
        first = false;
        const float neg = m_run == -INFINITY ? 0.f : -m_run;
        const uint64_t sl2x2 = f2_pack(sl2, sl2), neg2 = f2_pack(neg, neg);
        uint64_t ls[2] = {0ull, 0ull};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t s[32], pk[16];
          tmem_ld32(lane_addr + colS + 32 * c, s);
          tmem_ld_wait();
          if (edge) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!(vis[c] >> e & 1u)) s[e] = 0xff800000u;
          }
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float xa, xb;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), sl2x2, neg2), xa, xb);
            const float a = ex2(xa), b = ex2(xb);
            ls[e % 2] = f2_add(ls[e % 2], f2_pack(a, b));
            pk[e] = pack_bf16x2(a, b);
          }
          tmem_st16(lane_addr + colS + 16 * c, pk);
        }
        {
          float a, b, c, d;
          f2_unpack(ls[0], a, b);
          f2_unpack(ls[1], c, d);
          l += (a + b) + (c + d);
        }
        if (edge) {  // NaN values that this row sees
          const int nu = n_seg0 + k;  // the CTA's unit
          ok = mbar_wait_warp(&v_full[nu % NV], (nu / NV) & 1, err, kTreeVFull);
          if (!ok) break;
          const uint4* bits = reinterpret_cast<const uint4*>(smem + C::OFF_NAN + (nu % NV) * (D / 16) * 64);
          uint32_t any = 0u;
#pragma unroll 4
          for (int i = 0; i < D / 16 * 4; ++i) any |= bits[i].x | bits[i].y | bits[i].z | bits[i].w;
          if (any) {
            const uint8_t* by = reinterpret_cast<const uint8_t*>(bits);
            for (int u = 0; u < 64; ++u) {
              uint32_t word = 0u;
#pragma unroll
              for (int w = 0; w < 4; ++w)
                if (u / 16 == w) word = vis[w];
              const uint32_t seen = word >> (2 * u & 31) & 3u;
              for (int g = 0; g < D / 16; ++g)
                if (by[g * 64 + u] & seen) nans |= 1u << g;
            }
          }
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&p_ready[t]);
      }
      n_seg0 += cnt;
      // ---- the segment's end: whole, its outputs; a piece of it, its sums
      const bool have0 = TWO ? (t == 0 && cnt > 0) : cnt > 0, have1 = TWO ? (t == 1 && cnt > 0) : cnt > 1;
      if (ok && have0) {
        ok = mbar_wait_warp(&o_done[0], no[0] & 1, err, kTreeO);
        ++no[0];
      }
      if (ok && have1) {
        ok = mbar_wait_warp(&o_done[1], no[1] & 1, err, kTreeO);
        ++no[1];
      }
      float m = m_run, f0 = 1.f, f1 = 1.f;
      if constexpr (!TWO) {
        xm[t * 128 + r] = m_run;
        xl[t * 128 + r] = l;
        xn[t * 128 + r] = nans;
      }
      if constexpr (!TWO) {
        // (a warp whose wait gave up comes here too, so that nobody waits for it, and all stop)
        ok = bar_red_and(1, 256, ok);
        const float m0 = xm[r], m1 = xm[128 + r], l0 = xl[r], l1 = xl[128 + r];
        nans = xn[r] | xn[128 + r];
        m = fmaxf(m0, m1);
        f0 = m0 == -INFINITY ? 0.f : ex2(m0 - m);
        f1 = m1 == -INFINITY ? 0.f : ex2(m1 - m);
        // (no key: the sum is 0, or a NaN that has to stay)
        l = (m0 == -INFINITY ? l0 : l0 * f0) + (m1 == -INFINITY ? l1 : l1 * f1);
      }
      if (!ok) break;
      tc_fence_after();
      if (warp_ok) {
        TreeSums z{0.f, 0.f};
        if (whole && row_ok) z = tree_finish(p, h, m, l);
        float* slot = partial + ((size_t)2 * blockIdx.x + (at_begin ? 0 : 1)) * C::PART;
        const int rr = (TWO ? t * 128 : 0) + r;
        __nv_bfloat16* o = p.o + ((size_t)(at.s.row0 + node) * p.H_q + h) * D;
        constexpr int COLS = TWO ? D : D / 2;  // one tile: each half of the warps stores half of the dims
        const int c_first = TWO ? 0 : t * COLS;
#pragma unroll 1
        for (int c0 = c_first; c0 < c_first + COLS; c0 += 16) {
          uint32_t a[16], b[16];
          float v[16];
          if (have0) tmem_ld16(lane_addr + 128 + c0, a);
          if (have1) tmem_ld16(lane_addr + 256 + 128 + c0, b);
          tmem_ld_wait();
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            v[c] = 0.f;
            if (have0) v[c] = __uint_as_float(a[c]) * f0;
            if (have1) v[c] = fmaf(__uint_as_float(b[c]), f1, v[c]);
          }
          if (nans >> (c0 / 16) & 1u) {
#pragma unroll
            for (int c = 0; c < 16; ++c) v[c] = NAN;
          }
          if (row_ok && whole) {
#pragma unroll
            for (int c = 0; c < 16; ++c) v[c] *= z.mul;
            *reinterpret_cast<uint4*>(o + c0) = ordered8(v);
            *reinterpret_cast<uint4*>(o + c0 + 8) = ordered8(v + 8);
          } else if (row_ok) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              *reinterpret_cast<float4*>(slot + rr * D + c0 + 4 * q) = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
          }
        }
        if (row_ok && (TWO || t == 0)) {
          if (whole) {
            if (p.lse) p.lse[(size_t)h * p.T + at.s.row0 + node] = z.lse;
          } else {
            slot[C::ROWS * D + rr] = m;
            slot[C::ROWS * D + C::ROWS + rr] = l;
          }
        }
      }
      tc_fence_before();
      if constexpr (!TWO) named_bar_sync(1, 256);  // both halves have read the sums: they may be overwritten
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 16) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc<512>(tmem);
  }
}

// Joins the pieces of every segment that spans several CTAs, in CTA order, and writes the rows without a
// token and, on request, those of no sequence.  WPR warps a row: warp w takes pieces w, w + WPR, ...,
// then their sums are added in order.
// Launched while the kernel before it runs: it waits for that kernel's end before it reads a piece.
// Every block waits, also one with nothing to do: this grid must not end before that kernel, or what
// follows on the stream could start beside it.
template <int D, int ROWS, int WPR>
__global__ void __launch_bounds__(256) kv4_tree_join_kernel(const Kv4TreeParams p, int grid, const float* partial) {
  constexpr int PART = ROWS * (D + 2), E = D / 32;
  __shared__ float red[2][8], sums[8][D];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, wr = warp % WPR;
  const long long row = (long long)blockIdx.x * (8 / WPR) + warp / WPR;
  const int G = p.H_q / p.c.H_kv;
  const bool have = row < (long long)p.T * p.H_q;
  const int t = have ? (int)(row / p.H_q) : 0, h = have ? (int)(row % p.H_q) : 0, hk = h / G;
  int b = -1;  // the row's sequence
  for (int base = 0; base < p.B && b < 0; base += 32) {
    const int i = base + lane;
    const unsigned in = __ballot_sync(0xffffffffu, i < p.B && __ldg(p.cu + i) <= t && t < __ldg(p.cu + min(i, p.B - 1) + 1));
    if (in) b = base + __ffs(in) - 1;
  }
  TreeSeq s{};
  long long total = 0, u0 = 0;
  int n_cta = 1, c0 = 0, c1 = 0, r = 0;
  if (b >= 0) {
    s = tree_seq<ROWS>(p, b);
    total = TreeScan<ROWS>::sum(p, p.B);
    if (s.units > 0) {
      const long long r_all = (long long)(t - s.row0) * G + h % G;
      r = (int)(r_all % ROWS);
      u0 = TreeScan<ROWS>::sum(p, b) + ((long long)hk * s.blocks + r_all / ROWS) * s.seg();
      n_cta = tree_ctas(total, grid);
      c0 = tree_cta_of(total, n_cta, u0 + kSegCost);
      c1 = tree_cta_of(total, n_cta, u0 + kSegCost + s.units - 1);
    }
  }
  grid_wait();
  if (!have || (b < 0 && !p.zero_rest) || (s.units > 0 && c0 == c1)) return;  // one CTA had all of it
  float a[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) a[e] = 0.f;
  if (s.units > 0) {
#pragma unroll 4
    for (int c = c0 + wr; c <= c1; c += WPR) {
      // the piece is the CTA's first where the CTA starts inside the segment
      const float* sl = partial + ((size_t)2 * c + (tree_cut(total, n_cta, c) >= u0 ? 0 : 1)) * PART;
      const float mi = sl[ROWS * D + r], li = sl[ROWS * D + ROWS + r];
      float v[E];
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const float2 x = *reinterpret_cast<const float2*>(sl + r * D + lane * E + e);
        v[e] = x.x;
        v[e + 1] = x.y;
      }
      const float mn = fmaxf(m, mi);
      const float f = m == -INFINITY ? 0.f : ex2(m - mn), w = mi == -INFINITY ? 0.f : ex2(mi - mn);
      l = (m == -INFINITY ? l : l * f) + (mi == -INFINITY ? li : li * w);  // (no key: 0, or a NaN that has to stay)
#pragma unroll
      for (int e = 0; e < E; ++e) a[e] = a[e] * f + v[e] * w;  // (a NaN stays, also of a piece without weight)
      m = mn;
    }
  }
  if constexpr (WPR > 1) {
    if (lane == 0) {
      red[0][warp] = m;
      red[1][warp] = l;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) sums[warp][lane * E + e] = a[e];
    __syncthreads();
    if (warp > 0) return;
    m = red[0][0];
    for (int w = 1; w < WPR; ++w) m = fmaxf(m, red[0][w]);
    l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) a[e] = 0.f;
#pragma unroll
    for (int w = 0; w < WPR; ++w) {
      const float f = red[0][w] == -INFINITY ? 0.f : ex2(red[0][w] - m);
      l += red[0][w] == -INFINITY ? red[1][w] : red[1][w] * f;
#pragma unroll
      for (int e = 0; e < E; ++e) a[e] = fmaf(sums[w][lane * E + e], f, a[e]);
    }
  }
  const TreeSums z = b < 0 ? TreeSums{0.f, -INFINITY} : tree_finish(p, h, m, l);
  // lane's columns back to their dims: of 8 columns 0 .. 7 the dims 0 4 1 5 2 6 3 7
  __nv_bfloat16* o = p.o + ((size_t)t * p.H_q + h) * D;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int col = lane * E + e, c = col & 7;
    o[(col & ~7) + (c >> 1) + (c & 1) * 4] = __float2bfloat16(a[e] * z.mul);
  }
  if (lane == 0 && p.lse) p.lse[(size_t)h * p.T + t] = z.lse;
}

namespace {

template <int D, bool TWO>
int launch_t(const Kv4TreeParams& p, float* partial, cudaStream_t stream) {
  using C = TreeCfg<D, TWO>;
  if (!allow_smem<kv4_tree_kernel<D, TWO>>(C::SMEM)) return -1;
  static std::atomic<int> sms[64];  // SMs of each device
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return -1;
  int n = sms[dev].load(std::memory_order_acquire);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return -1;
    sms[dev].store(n, std::memory_order_release);
  }
  const int grid = std::min(n, kMaxGrid);
  if (launch_kernel(kv4_tree_kernel<D, TWO>, dim3((unsigned)grid), kThreads, C::SMEM, stream, false, p, partial) != 0) return -1;
  const long long rows = (long long)p.T * p.H_q;
  if (rows <= 1216)  // few rows: eight warps take a row's pieces
    return launch_kernel(kv4_tree_join_kernel<D, C::ROWS, 8>, dim3((unsigned)rows), 256, 0, stream, true, p, grid,
                         (const float*)partial);
  return launch_kernel(kv4_tree_join_kernel<D, C::ROWS, 1>, dim3((unsigned)((rows + 7) / 8)), 256, 0, stream, true, p, grid,
                       (const float*)partial);
}

// Two row tiles a block where the sequences have more than 128 rows a kv head on average.
bool two_tiles(int B, int T, int H_q, int H_kv) { return B > 0 && (long long)T * (H_q / H_kv) > 128LL * B; }

}  // namespace

size_t kv4_tree_workspace(int B, int T, int H_q, int H_kv, int d) {
  return (size_t)kMaxGrid * 2 * (two_tiles(B, T, H_q, H_kv) ? 256 : 128) * (d + 2) * sizeof(float);
}

int launch_kv4_tree(const Kv4TreeParams& p, void* workspace, cudaStream_t stream) {
  float* partial = static_cast<float*>(workspace);
  const bool two = two_tiles(p.B, p.T, p.H_q, p.c.H_kv);
  if (p.c.d == 128) return two ? launch_t<128, true>(p, partial, stream) : launch_t<128, false>(p, partial, stream);
  return two ? launch_t<64, true>(p, partial, stream) : launch_t<64, false>(p, partial, stream);
}

}  // namespace sdpa
