// kv4_tree.cu -- attention of the nodes of drafted trees over a sequence's 4-bit paged cache
// (layout and number format in kv4.cuh).
//
//   Node i of a sequence with L tokens before its tree is its token L + i, at position L + depth(i).
//   S_j = scale q.k_j over the tokens j < L, the node's ancestors and itself, under a window only
//   those of the last window + 1 positions; softmax with an optional sink logit; o = P V.
//
// All n nodes and all G query heads of a kv head share every byte of the cache: n G rows.  Reading the cache
// bounds a call of few rows, the tensor cores one of many (256 rows: 178 us of products, 56 us of
// bytes for 329,377 tokens of 8 kv heads of 128).  So there are four forms, by the sequences' rows a kv head
// on average (block_rows); a call has one form for all of its sequences, and a sequence of more rows than its blocks have
// is read and decoded again for each of them (what that costs an uneven batch stands at block_rows):
//   - Up to 8 and 16 rows (kv4_tree_few_kernel): rows are the 8-wide columns of mma.sync products whose
//     16 rows are tokens (scores) or head dims (outputs); operands are decoded in registers.
//   - Up to 128 rows, and more (kv4_tree_kernel): tcgen05 products of 128-row tiles.  Four warps decode
//     K and V into bf16 operand tiles in shared memory (128-byte swizzle; the eight lanes of a quarter
//     warp store to different banks), S = Q K^T and O += P V accumulate in TMEM, two warpgroups take the
//     softmax, a thread a row, with P where S was.  Up to 128 rows they take the units in turn, each with its
//     own sums, joined at a part's end; above, they hold a row tile each and share the operands.
// All forms:
//   - A unit is 128 tokens of one sequence and kv head.  A loading warp works out the CTA's work, looks pages up
//     and streams their blocks into shared memory, a page and head in one bulk copy.
//   - Codes are decoded as (c - 8) s 2^-23 (kv4.cuh), exact; the power of two is undone in the scores'
//     scale and in the outputs.  Eight dims of a word come out in the order 0 4 1 5 2 6 3 7: Q is
//     laid out alike, and the outputs are put back when they are stored.
//   - Work is cut evenly over a persistent grid, whatever the lengths (units of one sequence, kv head
//     and row block in order, and kSegCost units more for each such segment); a segment that spans
//     several CTAs leaves fp32 partial sums in the workspace, joined in CTA order by a second kernel:
//     bitwise reproducible.
//   - The probabilities are rounded to bf16 (2^-8 of each at most) for P V, the operand type of the products; their sum
//     is of the unrounded ones, fp32.  Against 64 bits an output's error, of which its own rounding to bf16 is 0.00166
//     (root mean square, relative), becomes 0.00186 for 16 sequences of 16 nodes, 0.0023 for tokens of much the same weight.
//   - Units with tokens that some row does not see (the tree's own, the ends of a window) take each row's 128 bits
//     of what it sees, found by walking up from its node: the walk is a dependent load a level.
//
// Measured on the device (329,377 tokens of 4 sequences, 8 kv heads of 128, 4 query heads each): 2 nodes 79 us,
// 4 nodes 104, 8 and 16 nodes 167 and 172, 32 nodes 179, 64 nodes 255 (1.33 PFLOP/s, 70 % of the measured bf16
// rate), 128 nodes 480.  16 sequences of 1 to 8191 tokens with 16 nodes: 41 us.  What the steps brought, for
// 131,072 tokens and 64 / 16 nodes: sizes worked out by every warp 200 / 127 us; by the loading warp, rare
// paths without the scores' registers 165 / 114; shorter loops of products 151 / 98; join's pieces
// found at once and longer output steps 136 / 92; K and V of a unit loaded together 136 / 89; waits without
// reports and other code out of the roles' loops 133 / 86; places of pieces by two offsets 130 / 81; more blocks of
// the join 121 / 81.
// What bounds it: one tile, decoding (some 2500 cycles a unit in four warps, their waits included; with eight warps the
// chain S - softmax - P V of a warpgroup's units, 4900 cycles for two, gives the same).  That chain is as long as it is
// because rows are the tile's lanes: a thread takes 128 exponentials and the products 128 rows whether 32 or 128 of them
// exist.  Tokens on the lanes and rows as columns, as in the few-row form, have not been tried with tcgen05.  Two tiles, that chain with both
// tiles' products (2048 cycles a unit at full rate) and the decoded operands' way through shared memory.  Few rows:
// the copies and the decoding arithmetic, as in kv4_decode.cu.
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
// a segment's fixed costs, in units
template <int ROWS>
constexpr int kSegCost = ROWS == 8 ? 1 : ROWS == 16 ? 2 : ROWS == 256 ? 5 : 4;
// What an expired wait is reported as: the role that gave up.
enum TreeSite { kTreeLoad = 0xB0, kTreeIssue, kTreeDecode, kTreeSoftmax, kTreeFew };

__device__ __forceinline__ uint32_t globaltimer_lo() {
  uint32_t t;
  asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
  return t;
}

// A bounded wait of a whole warp for a barrier's phase, true if it completed.  Some thirty of these are in line, and all
// roles' code comes from the same instruction cache, so a warp reports an expired wait once, where its role ends
// (tree_report): 16 sequences of 16 nodes took 45 us, 47 with the report in line, 49 with a look at the other roles'
// reports in the loop.
__device__ __forceinline__ bool tree_wait(uint64_t* bar, uint32_t parity) {
  static_assert(SDPA_WAIT_LIMIT_NS < 0xffffffffull, "32 bits of the timer");
  const uint32_t a = smem_u32(bar);
  bool ok = mbar_try_wait(a, parity);
  if (!ok) {
    const uint32_t t0 = globaltimer_lo();
#pragma unroll 1
    do {
      ok = mbar_try_wait(a, parity) || mbar_try_wait(a, parity);
    } while (!ok && globaltimer_lo() - t0 <= (uint32_t)SDPA_WAIT_LIMIT_NS);
  }
  return __all_sync(0xffffffffu, ok) != 0;
}
__device__ __forceinline__ void tree_report(const Kv4TreeParams& p, bool ok, int site) {
  if (!ok && threadIdx.x % 32 == 0) atomicCAS(p.err, 0, kErrTimeoutBase + site);
}

// A sequence's sizes.
struct TreeSeq {
  int row0, n;   // its rows of q
  int L, len;    // tokens before the tree, and all (as far as the table goes)
  int lo, first;  // first token some node sees, its unit
  int units, blocks;
  int seg;       // numbers of a segment (below)
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
  s.seg = s.units > 0 ? s.units + kSegCost<ROWS> : 0;
  s.blocks = (int)(((long long)s.n * (p.H_q / p.c.H_kv) + ROWS - 1) / ROWS);
  return s;
}
// How the units of a call are numbered: sequence by sequence, in it kv head by kv head, in it row
// block by row block; each such segment has units + kSegCost numbers, the first kSegCost for its
// fixed costs.  CTA c takes an even share of the numbers, in order.

// A CTA's part of a segment, as the loading warp works it out for the others.
struct TreePart {
  int row0, n, L, len, lo;  // the sequence (TreeSeq)
  int unit0, cnt;           // first unit (of 128 tokens) and how many; -1: there are no more parts
  int hk, node0, rem0, R;   // kv head; the row block's first node, its first head in the group, its rows
  int slot;                 // the whole of a segment: -1; a piece: which of the CTA's two places it takes
  // Units below u_win and from u_tree on have tokens that not every row sees: at a window's lower end,
  // and from the unit on that holds the tree's first node or ends past the tokens before it.
  int u_win, u_tree;
  int G;       // query heads a kv head
  float inv_G;
};
constexpr int kParts = 4;  // parts the loading warp may be ahead

// What the join has to know of a piece.
struct TreePiece {
  int row0, node0, rem0, R, hk;
  int valid, starts, ends;  // the segment's first piece, its last
};
static_assert(sizeof(TreePiece) == 32, "read as two 16-byte words");

__device__ __forceinline__ int tree_parent(const Kv4TreeParams& p, int row0, int i) {
  if (!p.parents) return i - 1;
  const int a = __ldg(p.parents + row0 + i);
  return a < i && a >= 0 ? a : -1;
}

// x / g for 0 <= x < 2^20, inv = 1 / g: the fp32 product is off by less than half of 1 / g.
__device__ __forceinline__ int small_div(int x, float inv) { return (int)(((float)x + 0.5f) * inv); }

// x / n for 0 <= x, in one place: 64-bit division is long.
__device__ __noinline__ long long divide(long long x, unsigned n) {
  if (x <= 0xffffffffLL) return (unsigned)x / n;
  return (unsigned long long)x / n;
}

// This CTA's numbers (a whole warp): the sequence b they begin in, `skip` of its numbers before them, and how
// many.
template <int ROWS>
__device__ __forceinline__ void tree_share(const Kv4TreeParams& p, int& b, long long& skip, long long& left) {
  const int lane = threadIdx.x % 32;
  long long total = 0, mine = 0, upto = 0, first = 0;
  bool found = false;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    long long carry = 0;
#pragma unroll 1
    for (int base = 0; base < p.B && !found; base += 32) {
      if (pass == 0 || p.B > 32) {
        mine = 0;
        if (base + lane < p.B) {
          const TreeSeq s = tree_seq<ROWS>(p, base + lane);
          mine = (long long)s.seg * s.blocks * p.c.H_kv;
        }
        upto = mine;
#pragma unroll 1
        for (int off = 1; off < 32; off <<= 1) {
          const long long o = __shfl_up_sync(0xffffffffu, upto, off);
          if (lane >= off) upto += o;
        }
      }
      if (pass == 1) {
        const unsigned holds = __ballot_sync(0xffffffffu, first < carry + upto);
        if (holds) {
          const int w = __ffs(holds) - 1;
          b = base + w;
          skip = first - carry - __shfl_sync(0xffffffffu, upto - mine, w);
          found = true;
        }
      }
      carry += __shfl_sync(0xffffffffu, upto, 31);
    }
    if (pass == 0) {
      total = carry;
      const long long want = total / 2 + 1;
      const int n = (int)min((long long)gridDim.x, want);
      if (total == 0 || (int)blockIdx.x >= n) break;
      const long long q = divide(total, (unsigned)n);
      const int rest = (int)(total - q * n);
      first = q * blockIdx.x + min((int)blockIdx.x, rest);
      left = q + ((int)blockIdx.x < rest ? 1 : 0);
    }
  }
}

// The loading warp: walks the CTA's segments, passes their parts on, and streams their units.
template <class C>
__device__ __forceinline__ void tree_load(const Kv4TreeParams& p, TreePiece* pieces, uint8_t* smem, uint64_t* raw_full,
                                          uint64_t* raw_empty, TreePart* parts, uint64_t* part_full, uint64_t* part_empty, int b,
                                          long long skip, long long left) {
  constexpr int D = C::DIM;
  const int lane = threadIdx.x % 32;
  int n_part = 0;
  bool ok = true;
  // Lane i copies the block of page i of a unit (whole, also past the sequence's end), if some node sees a token of it: the pages
  // before a window may be gone from the table.  Its page is looked up one unit ahead.
  const int P = p.c.page_size, n_pages = kUnit >> p.c.page_shift, t0 = lane * P;
  const int block = kv4_block_bytes(P, D), G = p.H_q / p.c.H_kv;
  const size_t page_bytes = (size_t)block * p.c.H_kv;
  const float inv_G = __fdividef(1.f, (float)G);
  TreeSeq s{};
  int hk = 0, rb = 0, n = 0;
  bool enter = true;          // the sequence's sizes are still to be read
  int used = 0;               // this CTA's places for pieces that are taken, a bit each
  bool first = true;
#pragma unroll 1
  while (ok) {
    TreePart t{};
    bool starts = false, ends = false;
    if (left > 0) {
      if (enter) {
        if (b >= p.B) {  // (the offsets were changed meanwhile)
          left = 0;
          continue;
        }
        s = tree_seq<C::ROWS>(p, b);
        if (s.seg == 0) {
          ++b;
          continue;
        }
        const long long vh = divide(skip, (unsigned)s.seg);
        skip -= vh * s.seg;
        hk = (int)((unsigned)vh / (unsigned)s.blocks);
        rb = (int)vh - hk * s.blocks;
        hk = min(hk, p.c.H_kv - 1);  // (the offsets were changed meanwhile)
        enter = false;
      }
      // the CTA's units [from, to) of the segment
      const int take = (int)min((long long)s.seg - skip, left);
      const int from = max((int)skip - kSegCost<C::ROWS>, 0), to = max((int)skip + take - kSegCost<C::ROWS>, 0);
      left -= take;
      skip = 0;
      const int r0 = rb * C::ROWS;  // (rows of a kv head are below 2^31)
      t.row0 = s.row0, t.n = s.n, t.L = s.L, t.len = s.len, t.lo = s.lo;
      t.G = G;
      t.inv_G = inv_G;
      t.hk = hk;
      t.node0 = r0 / G;
      t.rem0 = r0 - t.node0 * G;
      t.R = min(s.n * G - r0, C::ROWS);
      // of them those that the row block needs: up to its last node's own token
      const int last = t.node0 + (t.rem0 + t.R - 1) / G;
      const int len = (int)min((long long)s.L + last + 1, (long long)s.len);
      t.unit0 = s.first + from;
      t.cnt = max(min(to, (len - 1) / kUnit - s.first + 1) - from, 0);
      t.u_tree = s.L / kUnit;
      const long long all_see = (long long)s.L + s.n - 1 - p.window;  // from this token on every row sees the prefix
      t.u_win = p.window >= 0 && all_see > 0 ? (int)((unsigned)all_see / kUnit) + 1 : 0;
      starts = from == 0;
      ends = to == s.units;
      t.slot = starts && ends ? -1 : first ? 0 : 1;
      if (++rb == s.blocks) {
        rb = 0;
        if (++hk == p.c.H_kv) {
          ++b;
          enter = true;
        }
      }
      if (from == to) continue;  // only fixed costs
      first = false;
      if (t.slot >= 0) {
        used |= 1 << t.slot;
        if (lane == 0) pieces[2 * blockIdx.x + t.slot] = TreePiece{t.row0, t.node0, t.rem0, t.R, t.hk, 1, starts, ends};
      }
    } else {
      t.cnt = -1;
    }
    const int slot = n_part % kParts;
    if (n_part >= kParts) ok = tree_wait(&part_empty[slot], (n_part / kParts - 1) & 1);
    if (!ok) break;
    if (lane == 0) {
      parts[slot] = t;
      mbar_arrive(&part_full[slot]);
    }
    ++n_part;
    __syncwarp();
    if (t.cnt < 0) break;
    auto page_of = [&](int k) {
      const long long tok = (long long)(t.unit0 + k) * kUnit + t0;
      return k < t.cnt && lane < n_pages && tok < t.len && tok + P > t.lo ? kv4_page(p.c, b - (enter ? 1 : 0), (int)tok) : -2;
    };
    int page = page_of(0);
#pragma unroll 1
    for (int k = 0; k < t.cnt; ++k, ++n) {
      const int stage = n % C::STAGES;
      uint8_t* st = smem + C::OFF_RAW + stage * C::STAGE;
      const uint8_t* src = p.pool + (size_t)max(page, 0) * page_bytes + (size_t)t.hk * block;
      const int have = page;
      page = page_of(k + 1);
      if (n >= C::STAGES) ok = tree_wait(&raw_empty[stage], (n / C::STAGES - 1) & 1);
      if (!ok) break;
      if (__any_sync(0xffffffffu, have == -1)) {  // not a page: its tokens read as zeros (scale 0)
        if (have == -1) {
#pragma unroll 1
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
  }
  if (lane < 2 && !(used >> lane & 1)) pieces[2 * blockIdx.x + lane].valid = 0;
  // every copy this warp started must land before the CTA may exit: wait for the last ones
#pragma unroll 1
  for (int s = 0; s < C::STAGES && s < n; ++s) {
    const int last = s + (n - 1 - s) / C::STAGES * C::STAGES;
    ok = tree_wait(&raw_full[s], (last / C::STAGES) & 1) && ok;
  }
  tree_report(p, ok, kTreeLoad);
}

template <int D, bool TWO>
struct TreeCfg {
  static constexpr int DIM = D;
  static constexpr int ROWS = TWO ? 256 : 128;  // rows of a block
  static constexpr int BLK = 128 * 128;         // one operand block: 128 rows of 64 bf16
  static constexpr int TILE = BLK * (D / 64);
  static constexpr int NK = TWO ? 1 : 2, NV = 2;  // (two row tiles: S of a unit is done long before its P V)
  static constexpr int STAGES = D == 128 ? 3 : 6;
  static constexpr int STAGE = kUnit * D * 9 / 8;
  // Warps: 8 softmax, 4 decode, one or two issue the products, one loads (the last shares their registers).
  // One row tile has an issuer for each warpgroup's units: with one for both, its waits and instructions
  // bound the call (110 instead of 98 us for 131,072 tokens, 8 kv heads, 64 rows).  Two row tiles have one
  // issuer, which takes them in turn: with two 180 instead of 156 us for 256 rows.
  static constexpr int DEC_WARP = 8, MMA_WARP = 12, ISSUERS = TWO ? 1 : 2, LOAD_WARP = 14, THREADS = 512;
  // registers a thread of the launch, and after the split: softmax, decoding, the rest
  static constexpr int REGS = 128, REGS_SOFT = 184, REGS_DEC = 88, REGS_REST = 56;
  static_assert(256 * REGS_SOFT + 128 * REGS_DEC + 128 * REGS_REST <= THREADS * REGS, "the launch's registers");
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = OFF_Q + (TWO ? 2 : 1) * TILE;
  static constexpr int OFF_V = OFF_K + NK * TILE;
  static constexpr int OFF_RAW = OFF_V + NV * TILE;
  static constexpr int OFF_NAN = OFF_RAW + STAGES * STAGE;  // [NV][D / 16][64] bits of the two tokens of a pair
  static constexpr int OFF_ML = OFF_NAN + NV * D / 16 * 64;  // [2][128] maxima, sums, NaN groups
  static constexpr int OFF_PART = OFF_ML + 3 * 2 * 128 * 4;
  static constexpr int OFF_BAR = OFF_PART + kParts * (int)sizeof(TreePart);
  static constexpr int N_BAR = 2 * STAGES + 2 * NK + 2 * NV + 2 + 6 + 2 + 2 * kParts + 4;
  static constexpr int OFF_SLOT = OFF_BAR + N_BAR * 8;
  static constexpr int SMEM = OFF_SLOT + 16 + 1024;  // (aligned by the kernel)
  static constexpr int PART = ROWS * (D + 2);  // floats of one partial: sums, maxima, denominators
  static_assert(SMEM <= 232448, "shared memory budget");
  static_assert(SMEM > 116 * 1024, "one CTA per SM keeps the 512-column TMEM allocation uncontended");
};

template <int N>
__device__ __forceinline__ void regs_less() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_more() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// sets bits [from, to) of the 128 tokens of a unit
__device__ __forceinline__ void set_range(uint32_t (&vis)[4], int from, int to) {
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const int a = min(max(from - 32 * w, 0), 32), z = min(max(to - 32 * w, 0), 32);
    // (funnel shifts: a shift by 32 leaves nothing)
    const uint32_t below_a = __funnelshift_lc(0xffffffffu, 0u, a), below_z = __funnelshift_lc(0xffffffffu, 0u, z);
    vis[w] |= below_z & ~below_a;
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
__global__ void __launch_bounds__(TreeCfg<D, TWO>::THREADS, 1) kv4_tree_kernel(const Kv4TreeParams p, TreePiece* pieces, float* partial) {
  using C = TreeCfg<D, TWO>;
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
  uint64_t* part_full = mma_done + 2;
  uint64_t* part_empty = part_full + kParts;
  uint64_t* x_ready = part_empty + kParts;  // [2] a warpgroup's sums of a shared part are there
  uint64_t* x_read = x_ready + 2;           // [2] it has read the other's
  TreePart* parts = reinterpret_cast<TreePart*>(smem + C::OFF_PART);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_SLOT);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

  grid_launch_dependents();  // the join may be set up meanwhile
  if (threadIdx.x == 0) {
    for (int s = 0; s < NST; ++s) {
      mbar_init(&raw_full[s], 1);
      mbar_init(&raw_empty[s], 4);
    }
    for (int s = 0; s < NK; ++s) {
      mbar_init(&k_full[s], 4);
      mbar_init(&k_empty[s], 1);
    }
    for (int s = 0; s < NV; ++s) {
      mbar_init(&v_full[s], 4);
      mbar_init(&v_empty[s], 1);
    }
    mbar_init(q_full, 4);
    mbar_init(q_empty, C::ISSUERS);
    for (int t = 0; t < 2; ++t) {
      mbar_init(&s_ready[t], 1);
      mbar_init(&p_ready[t], 4);
      mbar_init(&o_done[t], 1);
      mbar_init(&x_ready[t], 4);
      mbar_init(&x_read[t], 4);
      mbar_init(&mma_done[t], 1);
    }
    for (int s = 0; s < kParts; ++s) {
      mbar_init(&part_full[s], 1);
      mbar_init(&part_empty[s], 8 + 4 + C::ISSUERS);
    }
    fence_barrier_init();
  }
  if (warp == C::MMA_WARP) {
    tmem_alloc<512>(tmem_slot);
    tmem_relinquish();
  }
  int b = 0;
  long long skip = 0, left = 0;
  if (warp == C::LOAD_WARP) tree_share<C::ROWS>(p, b, skip, left);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  bool ok = true;
  // The next part of this CTA's work; cnt < 0: there is none.  It stays in shared memory (few registers hold
  // what a role needs of it all the time) until part_done().
  int n_part = 0;
  auto next_part = [&]() {
    ok = ok && tree_wait(&part_full[n_part % kParts], (n_part / kParts) & 1);
    return ok && parts[n_part % kParts].cnt >= 0;
  };
  auto part_done = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(&part_empty[n_part % kParts]);
    ++n_part;
  };

  if (warp >= C::MMA_WARP) regs_less<C::REGS_REST>();
  if (warp == C::LOAD_WARP) {
    tree_load<C>(p, pieces, smem, raw_full, raw_empty, parts, part_full, part_empty, b, skip, left);
  } else if (warp >= C::MMA_WARP && warp < C::MMA_WARP + C::ISSUERS) {
    // ---------------------------------------------------------------- issuers of the products
    constexpr uint32_t idS = idesc_bf16_f32(128, 128, false, false), idO = idesc_bf16_f32(128, D, false, true);
    bool issued = false;
    if constexpr (TWO) {
      const uint32_t sQ = smem_u32(smem + C::OFF_Q), sK = smem_u32(smem + C::OFF_K), sV = smem_u32(smem + C::OFF_V);
      auto issue_S = [&](int t, int stage) {
        const uint64_t dq = smem_desc_sw128(sQ + (TWO ? t * C::TILE : 0), 16, 1024);
        const uint64_t dk = smem_desc_sw128(sK + stage * C::TILE, 16, 1024);
#pragma unroll 4
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk / 4) * C::BLK + (kk % 4) * 32;
          mma_ss_warp(tmem + t * 256, desc_add(dq, off), desc_add(dk, off), idS, kk > 0);
        }
        mma_commit_warp(&s_ready[t]);
      };
      auto issue_PV = [&](int t, int stage, bool acc) {
        const uint64_t dv = smem_desc_sw128(sV + stage * C::TILE, C::BLK, 1024);
#pragma unroll 4
        for (int kk = 0; kk < kUnit / 16; ++kk)
          mma_ts_warp(tmem + t * 256 + 128, tmem + t * 256 + kk * 8, desc_add(dv, kk * 2048), idO, (acc || kk > 0) ? 1u : 0u);
      };
      int nq = 0, nk = 0, nv = 0;  // phases consumed
      uint32_t np = 0u;            // parities of p_ready, a bit a tile
      auto wait_K = [&]() {
        ok = ok && tree_wait(&k_full[nk % NK], (nk / NK) & 1);
        if (ok) tc_fence_after();
        return ok;
      };
#pragma unroll 1
      while (next_part()) {
        const int cnt = parts[n_part % kParts].cnt;
        part_done();
        if (cnt == 0) continue;
        ok = tree_wait(q_full, nq++ & 1);
        if (!ok) break;
        issued = true;
        if (!wait_K()) break;
        issue_S(0, nk % NK);
        issue_S(1, nk % NK);
        mma_commit_warp(&k_empty[nk++ % NK]);
        if (cnt == 1) mma_commit_warp(q_empty);
        for (int k = 0; k < cnt && ok; ++k) {
          const bool need_k = k + 1 < cnt;
          ok = tree_wait(&v_full[nv % NV], (nv / NV) & 1);
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            ok = ok && tree_wait(&p_ready[t], np >> t & 1u);
            if (!ok) break;
            np ^= 1u << t;
            tc_fence_after();
            issue_PV(t, nv % NV, k > 0);
            if (!need_k) {
              mma_commit_warp(&o_done[t]);
            } else {
              if (t == 0 && !wait_K()) break;
              issue_S(t, nk % NK);
            }
          }
          if (!ok) break;
          mma_commit_warp(&v_empty[nv++ % NV]);
          if (need_k) mma_commit_warp(&k_empty[nk++ % NK]);
          if (k + 2 == cnt) mma_commit_warp(q_empty);  // every S of the part is issued
        }
      }
    } else {
      // A tile's S, P V and next S follow one another (P lies where S was); the two warpgroups' tiles are
      // independent.
      const int t = warp - C::MMA_WARP;
      const uint32_t tS = tmem + t * 256, tO = tS + 128;
      const uint64_t dQ = smem_desc_sw128(smem_u32(smem + C::OFF_Q), 16, 1024);
      const uint64_t dK = smem_desc_sw128(smem_u32(smem + C::OFF_K), 16, 1024);
      const uint64_t dV = smem_desc_sw128(smem_u32(smem + C::OFF_V), C::BLK, 1024);
      int n = 0, nq = 0, np = 0;  // units of the CTA's stream; parts with units; phases of p_ready
#pragma unroll 1
      while (ok && next_part()) {
        const int cnt = parts[n_part % kParts].cnt;
        part_done();
        if (cnt == 0) continue;
        ok = tree_wait(q_full, nq++ & 1);
        if (!ok) break;
        const int k_first = (n ^ t) & 1;
        if (k_first >= cnt) {  // the other tile has the part's only unit
          if (lane == 0) mbar_arrive(q_empty);
          n += cnt;
          continue;
        }
        issued = true;
#pragma unroll 1
        for (int k = k_first; k < cnt; k += 2) {
          const int u = n + k, sk = u % NK, sv = u % NV;
          const bool last = k + 2 >= cnt;
          ok = tree_wait(&k_full[sk], (u / NK) & 1);
          if (!ok) break;
          tc_fence_after();
#pragma unroll 2
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (kk / 4) * C::BLK + (kk % 4) * 32;
            mma_ss_warp(tS, desc_add(dQ, off), desc_add(dK, sk * C::TILE + off), idS, kk > 0);
          }
          mma_commit_warp(&s_ready[t]);
          mma_commit_warp(&k_empty[sk]);
          if (last) mma_commit_warp(q_empty);  // every S of the part is issued
          ok = tree_wait(&v_full[sv], (u / NV) & 1);
          ok = ok && tree_wait(&p_ready[t], np++ & 1);
          if (!ok) break;
          tc_fence_after();
#pragma unroll 2
          for (int kk = 0; kk < kUnit / 16; ++kk)
            mma_ts_warp(tO, tS + kk * 8, desc_add(dV, sv * C::TILE + kk * 2048), idO, (k > k_first || kk > 0) ? 1u : 0u);
          mma_commit_warp(&v_empty[sv]);
          if (last) mma_commit_warp(&o_done[t]);
        }
        n += cnt;
      }
    }
    // every product must be complete before TMEM is released
    if (issued) {
      uint64_t* bar = &mma_done[warp - C::MMA_WARP];
      mma_commit_warp(bar);
      ok = tree_wait(bar, 0) && ok;
    }
  } else if (warp >= C::DEC_WARP && warp < C::MMA_WARP) {
    // ---------------------------------------------------------------- decoding warps
    regs_less<C::REGS_DEC>();
    const int tid = threadIdx.x % 128, P = p.c.page_size, block = kv4_block_bytes(P, D);
    constexpr int N = D / 32, STEP = 128 / N, NG = D / 16;  // 16-byte pieces a thread takes of K, of V; tokens between them
    auto page_at = [&](int tok) { return (tok >> p.c.page_shift) * block; };
    // what 32 and 64 tokens on adds to the place of a code, of a scale (of K and of V alike): pages are whole powers of two
    const int c64 = P <= 64 ? page_at(64) : 64 * (D / 2), s64 = P <= 64 ? c64 : 64 * (D / 16);
    const int c32 = P <= 32 ? page_at(32) : 32 * (D / 2), s32 = P <= 32 ? c32 : 32 * (D / 16);
    auto code_at = [&](int tok) { return (tok & 32 ? c32 : 0) + (tok & 64 ? c64 : 0); };
    auto scale_at = [&](int tok) { return (tok & 32 ? s32 : 0) + (tok & 64 ? s64 : 0); };
    // K: 32 dims (quarter q) of a token a piece.  Lanes of dims 64.. store their four chunks two further on:
    // the eight lanes of a quarter warp then hit all banks.
    const int tok_k = tid / N, q = tid % N, w_k = tok_k & (P - 1);
    const int code_k = page_at(tok_k) + w_k * (D / 2) + q * 16;
    const int scale_k = page_at(tok_k) + kv4_off_sk(P, D) + w_k * (D / 16) + q * 2;
    const int dst_k = (q / 2) * C::BLK + tok_k * 128 + (((((q & 1) * 4) ^ (tok_k & 7)) << 4) ^ (q >= 2 ? 32 : 0));
    const bool swap = q >= 2;
    // V: 16 dims (group g) of a pair of tokens a piece; which of a token's two chunks is stored first differs
    // between the lanes of a quarter warp that would meet in a bank.
    const int u = tid / NG, w_v = 2 * u & (P - 1), x_v = kv4_slot_xor(w_v / 2, D);
    const int g = D == 128 ? (tid % NG) ^ x_v : (tid % NG) ^ (x_v >> 1), flip = D == 128 ? g / 4 : u & 1;
    const int code_v = page_at(2 * u) + kv4_off_v(P, D) + w_v / 2 * D + tid % NG * 16;
    const int scale_v = page_at(2 * u) + kv4_off_sv(P, D) + w_v / 2 * (D / 8) + 2 * g;
    const int dst_v = (g / 4) * C::BLK + 2 * u * 128 + (((2 * (g % 4) + flip) ^ (2 * u & 7)) << 4);
    int n = 0, nq = 0;
#pragma unroll 1
    for (; next_part(); part_done()) {
      const TreePart& part = parts[n_part % kParts];
      const int cnt = part.cnt;
      if (cnt == 0) continue;
      // ---- Q: loaded early, stored when the last scores of the part before are done
      {
        constexpr int QI = C::ROWS * (D / 8) / 128, QB = 8;
        const int R = part.R, rem0 = part.rem0, G = part.G;
        const float inv_G = part.inv_G;
        const __nv_bfloat16* q0 = p.q + ((size_t)(part.row0 + part.node0) * p.H_q + part.hk * G) * D;
#pragma unroll 1
        for (int i0 = 0; i0 < QI; i0 += QB) {
          uint4 w[QB];
#pragma unroll
          for (int i = 0; i < QB; ++i) {
            const int e = (i0 + i) * 128 + tid, r = e / (D / 8), c = e % (D / 8);
            w[i] = make_uint4(0u, 0u, 0u, 0u);
            if (r < R) {
              const int node = small_div(rem0 + r, inv_G);
              w[i] = __ldg(reinterpret_cast<const uint4*>(q0 + ((size_t)node * p.H_q + (rem0 + r - node * G)) * D + c * 8));
            }
          }
          if (i0 == 0 && nq > 0) {
            ok = tree_wait(q_empty, (nq - 1) & 1);
            if (!ok) break;
          }
#pragma unroll
          for (int i = 0; i < QB; ++i) {
            const int e = (i0 + i) * 128 + tid, r = e / (D / 8), c = e % (D / 8), rt = r % 128;
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
      int unit = part.unit0;
      const int u_win = part.u_win, u_tree = part.u_tree;
#pragma unroll 1
      for (int k = 0; k < cnt; ++k, ++n, ++unit) {
        const int stage = n % NST, sk = n % NK, sv = n % NV;
        const uint8_t* st = smem + C::OFF_RAW + stage * C::STAGE;
        // The unit's bytes, and K's place free.  One row tile, whose pace the decoding sets: half of the lanes looks
        // at each barrier, so that two waits cost one (200 of some 2700 cycles a unit).  Two: K's place is
        // what the call waits for, so the bytes are in registers by then.
        if constexpr (TWO) {
          ok = tree_wait(&raw_full[stage], (n / NST) & 1);
        } else {
          const bool other = lane % 2 == 1 && n >= NK;
          ok = tree_wait(other ? &k_empty[sk] : &raw_full[stage], other ? (n / NK - 1) & 1 : (n / NST) & 1);
        }
        if (!ok) break;
        uint4 w[N], wv[N];
        uint32_t sc[N], sv2[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
          w[i] = *reinterpret_cast<const uint4*>(st + code_k + code_at(STEP * i));
          sc[i] = *reinterpret_cast<const unsigned short*>(st + scale_k + scale_at(STEP * i));
        }
        auto load_V = [&]() {
#pragma unroll
          for (int i = 0; i < N; ++i) {
            wv[i] = *reinterpret_cast<const uint4*>(st + code_v + code_at(STEP * i));
            sv2[i] = *reinterpret_cast<const unsigned short*>(st + scale_v + scale_at(STEP * i));
          }
          __syncwarp();  // every lane has read its pieces
          if (lane == 0) mbar_arrive(&raw_empty[stage]);
        };
        if constexpr (TWO) {
          if (n >= NK) ok = tree_wait(&k_empty[sk], (n / NK - 1) & 1);
          if (!ok) break;
        } else {
          load_V();
        }
        {
          uint8_t* d = smem + C::OFF_K + sk * C::TILE;
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const uint32_t sp = scale_pair(swap ? __byte_perm(sc[i], 0u, 0x4401) : sc[i]);
            const Kv4Small a = scales_low(sp), b2 = scales_high(sp);
            const uint4 x = swap ? make_uint4(w[i].z, w[i].w, w[i].x, w[i].y) : w[i];
            *reinterpret_cast<uint4*>(d + i * STEP * 128 + dst_k) = decode8(x.x, a);
            *reinterpret_cast<uint4*>(d + i * STEP * 128 + (dst_k ^ 16)) = decode8(x.y, a);
            *reinterpret_cast<uint4*>(d + i * STEP * 128 + (dst_k ^ 32)) = decode8(x.z, b2);
            *reinterpret_cast<uint4*>(d + i * STEP * 128 + (dst_k ^ 48)) = decode8(x.w, b2);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&k_full[sk]);
        if constexpr (TWO) load_V();
        if (n >= NV) ok = tree_wait(&v_empty[sv], (n / NV - 1) & 1);
        if (!ok) break;
        // units whose tokens are not all seen by all rows, as the softmax warps decide it
        if (unit < u_win || unit >= u_tree) {
          const int len = part.len - unit * kUnit, lo = part.lo - unit * kUnit;  // (a token's number is below 2^31)
          // A token that no row sees adds nothing, whatever its bytes are.  One held as NaN adds nothing
          // either: rows that do not see it have P = 0, but 0 times NaN is NaN.  The rows that see it
          // learn of it from these bits.
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const int tok = 2 * u + STEP * i;
            uint32_t bits = 0u;
            if (tok >= len || tok < lo) sv2[i] &= 0xFF00u;
            if (tok + 1 >= len || tok + 1 < lo) sv2[i] &= 0x00FFu;
            if ((sv2[i] & 0x00F8u) == 0x00F8u) {
              bits |= 1u;
              sv2[i] &= 0xFF00u;
            }
            if ((sv2[i] & 0xF800u) == 0xF800u) {
              bits |= 2u;
              sv2[i] &= 0x00FFu;
            }
            smem[C::OFF_NAN + (sv * NG + g) * 64 + tok / 2] = (uint8_t)bits;
          }
        }
        {
          uint8_t* d = smem + C::OFF_V + sv * C::TILE;
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const uint32_t sp = scale_pair(sv2[i]);
            const Kv4Small a = scales_low(sp), b2 = scales_high(sp);
            // (D = 128: 8 bytes a token; D = 64: the two eighths' 4 bytes a token)
            const uint32_t t0w0 = wv[i].x, t0w1 = D == 128 ? wv[i].y : wv[i].z, t1w0 = D == 128 ? wv[i].z : wv[i].y,
                           t1w1 = wv[i].w;
            uint8_t* di = d + i * STEP * 128;  // (the chunk's exclusive-or with 1: the row's next token)
            *reinterpret_cast<uint4*>(di + dst_v) = decode8(flip ? t0w1 : t0w0, a);
            *reinterpret_cast<uint4*>(di + (dst_v ^ 16)) = decode8(flip ? t0w0 : t0w1, a);
            *reinterpret_cast<uint4*>(di + 128 + (dst_v ^ 16)) = decode8(flip ? t1w1 : t1w0, b2);
            *reinterpret_cast<uint4*>(di + 128 + dst_v) = decode8(flip ? t1w0 : t1w1, b2);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&v_full[sv]);
      }
      if (!ok) break;
    }
  } else if (warp < 8) {
    // ---------------------------------------------------------------- softmax and output
    regs_more<C::REGS_SOFT>();
    const int t = warp / 4, r = (warp % 4) * 32 + lane;
    const uint32_t lane_addr = tmem + ((uint32_t)((warp % 4) * 32) << 16);
    const uint32_t aS = lane_addr + t * 256, aO = aS + 128;
    const float sl2 = p.scale_log2 * kKv4SmallUndo;
    float* xm = reinterpret_cast<float*>(smem + C::OFF_ML);  // [2][128] maxima, sums, NaN groups of the two halves
    float* xl = xm + 256;
    uint32_t* xn = reinterpret_cast<uint32_t*>(xl + 256);
    int ns = 0, nx = 0, n_before = 0;  // s_ready phases consumed; parts shared with the other warpgroup; units of the parts before
    uint32_t no = 0u;          // parity of o_done
#pragma unroll 1
    for (; next_part(); part_done()) {
      const TreePart& part = parts[n_part % kParts];
      const int cnt = part.cnt, rr = (TWO ? t * 128 : 0) + r;
      const bool row_ok = rr < part.R, warp_ok = rr - lane < part.R;
      // this row's node, and its head
      int node = small_div(part.rem0 + (row_ok ? rr : 0), part.inv_G);
      const int h = part.hk * part.G + part.rem0 + (row_ok ? rr : 0) - node * part.G;
      node += part.node0;
      float m_run = -INFINITY, l = 0.f;
      uint32_t nans = 0u;  // groups of 16 dims in which this row sees a NaN
      bool first = true;
      // one tile: unit n of the CTA's stream is warpgroup n % 2's
      const int k_first = TWO ? 0 : (n_before ^ t) & 1;
      if (!TWO && cnt <= 1 && k_first != 0) {  // the other warpgroup has all of it
        n_before += cnt;
        continue;
      }
      int unit = part.unit0 + k_first;
      const int u_win = part.u_win, u_tree = part.u_tree;
#pragma unroll 1
      for (int k = k_first; k < cnt; k += TWO ? 1 : 2, unit += TWO ? 1 : 2) {
        const bool edge = unit < u_win || unit >= u_tree;
        uint32_t vis[4] = {0u, 0u, 0u, 0u};  // the unit's tokens that this row sees
        if (edge && warp_ok) {
          const int L = part.L, row0 = part.row0, k0 = unit * kUnit, a0 = k0 - L;  // the unit's first token; the node there
          const int end = part.len - L;  // nodes that have a token
          int lo = 0;                    // first token before the tree that this row sees
          if (p.window >= 0) {
            int depth = node;
            if (p.parents) {
              depth = 0;
              for (int a = tree_parent(p, row0, node); a >= 0; a = tree_parent(p, row0, a)) ++depth;
            }
            lo = depth >= p.window ? L : max(L - (p.window - depth), 0);
          }
          set_range(vis, lo - k0, L - k0);
          if (!p.parents) {
            set_range(vis, (p.window >= 0 && node > p.window ? min(node - p.window, end) : 0) - a0, min(node + 1, end) - a0);
          } else {
            int step = 0;
            for (int a = node; a >= max(a0, 0) && (p.window < 0 || step <= p.window); a = tree_parent(p, row0, a), ++step) {
              const int j = a - a0;
              if (j < kUnit && a < end) {
                const uint32_t bit = 1u << (j & 31);
#pragma unroll
                for (int w = 0; w < 4; ++w)
                  if (j / 32 == w) vis[w] |= bit;
              }
            }
          }
        }
        ok = tree_wait(&s_ready[t], ns & 1);
        ++ns;
        if (!ok) break;
        if (!warp_ok) {  // no row of this warp exists: its P may be anything
          if (lane == 0) mbar_arrive(&p_ready[t]);
          continue;
        }
        tc_fence_after();
        if (edge) {  // hidden tokens' scores become -inf where they are
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            uint32_t s[16];
            tmem_ld16(aS + 16 * c, s);
            const uint32_t word = (c & 4 ? (c & 2 ? vis[3] : vis[2]) : (c & 2 ? vis[1] : vis[0])) >> ((c & 1) * 16);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (!(word >> e & 1u)) s[e] = 0xff800000u;
            tmem_st16(aS + 16 * c, s);
          }
          tmem_st_wait();
        }
        // the row's 128 scores in one batch of loads, each with the maximum of its 32
        uint32_t s[4][32];
        float cm[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32_max(aS + 32 * c, s[c], cm[c]);
        tmem_ld_wait();
        const float mx = fmax3(cm[0], cm[1], fmaxf(cm[2], cm[3]));
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
              tmem_ld16(aO + c0, o);
              tmem_ld_wait();
#pragma unroll
              for (int c = 0; c < 16; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
              tmem_st16(aO + c0, o);
            }
          }
          m_run = m_new;
          // (read anew, so that this rare path does not need the scores' registers beside its own)
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(aS + 32 * c, s[c]);
          tmem_ld_wait();
        }
        first = false;
        const float neg = m_run == -INFINITY ? 0.f : -m_run;
        const uint64_t sl2x2 = f2_pack(sl2, sl2), neg2 = f2_pack(neg, neg);
        uint64_t ls[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float xa, xb;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(s[c][2 * e]), __uint_as_float(s[c][2 * e + 1])), sl2x2, neg2), xa, xb);
            const float a = ex2(xa), b2 = ex2(xb);
            ls[e % 4] = f2_add(ls[e % 4], f2_pack(a, b2));
            pk[e] = pack_bf16x2(a, b2);
          }
          tmem_st16(aS + 16 * c, pk);
        }
        {
          float a, b2;
          f2_unpack(f2_add(f2_add(ls[0], ls[1]), f2_add(ls[2], ls[3])), a, b2);
          l += a + b2;
        }
        if (edge) {  // NaN values that this row sees
          const int nu = n_before + k;  // the CTA's unit
          ok = tree_wait(&v_full[nu % NV], (nu / NV) & 1);
          if (!ok) break;
          const uint8_t* by = smem + C::OFF_NAN + (nu % NV) * (D / 16) * 64;
          uint32_t any = 0u;
          for (int i = lane; i < D / 16 * 16; i += 32) any |= reinterpret_cast<const uint32_t*>(by)[i];
          if (__any_sync(0xffffffffu, any != 0u)) {
#pragma unroll 1
            for (int u = 0; u < 64; ++u) {
              const uint32_t word = u & 32 ? (u & 16 ? vis[3] : vis[2]) : (u & 16 ? vis[1] : vis[0]);
              const uint32_t seen = word >> (2 * u & 31) & 3u;
#pragma unroll 1
              for (int g = 0; g < D / 16; ++g)
                if (by[g * 64 + u] & seen) nans |= 1u << g;
            }
          }
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_ready[t]);
      }
      n_before += cnt;
      // ---- the part's end: of a whole segment the outputs, of a piece its sums
      const bool both = !TWO && cnt > 1;  // the other warpgroup has sums of these rows too
      if (ok && cnt > 0) {
        ok = tree_wait(&o_done[t], no & 1u);
        no ^= 1u;
      }
      float m = m_run, f_own = 1.f, f_other = 0.f;
      if (both) {
        xm[t * 128 + r] = m_run;
        xl[t * 128 + r] = l;
        xn[t * 128 + r] = nans;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&x_ready[t]);
        ok = ok && tree_wait(&x_ready[1 - t], nx & 1);
        const float m2 = xm[(1 - t) * 128 + r], l2 = xl[(1 - t) * 128 + r];
        nans |= xn[(1 - t) * 128 + r];
        m = fmaxf(m_run, m2);
        f_own = m_run == -INFINITY ? 0.f : ex2(m_run - m);
        f_other = m2 == -INFINITY ? 0.f : ex2(m2 - m);
        // (no key: the sum is 0, or a NaN that has to stay)
        const float a = m_run == -INFINITY ? l : l * f_own, b2 = m2 == -INFINITY ? l2 : l2 * f_other;
        l = t == 0 ? a + b2 : b2 + a;
      }
      if (!ok) break;
      tc_fence_after();
      if (warp_ok) {
        const bool whole = part.slot < 0;
        TreeSums z{0.f, 0.f};
        if (whole && row_ok) z = tree_finish(p, h, m, l);
        float* slot = partial + ((size_t)2 * blockIdx.x + max(part.slot, 0)) * C::PART;
        __nv_bfloat16* o = p.o + ((size_t)(part.row0 + node) * p.H_q + h) * D;
        // where both warpgroups have sums, each stores half of the dims
        const int c_first = both ? t * (D / 2) : 0, c_end = both ? c_first + D / 2 : D;
        constexpr int EC = TWO ? 32 : 16;  // columns at a time (two tiles' sums of 32 would not fit the registers)
#pragma unroll 1
        for (int c0 = c_first; c0 < c_end; c0 += EC) {
          uint32_t a[EC], b2[TWO ? 1 : EC];
          if constexpr (TWO) {
            if (cnt > 0) tmem_ld32(aO + c0, a);
          } else {
            if (cnt > 0) tmem_ld16(aO + c0, a);
            if (both) tmem_ld16(lane_addr + (1 - t) * 256 + 128 + c0, b2);
          }
          tmem_ld_wait();
          float v[EC];
#pragma unroll
          for (int c = 0; c < EC; ++c) {
            v[c] = cnt > 0 ? __uint_as_float(a[c]) * f_own : 0.f;
            if constexpr (!TWO) {
              if (both) v[c] = fmaf(__uint_as_float(b2[c]), f_other, v[c]);
            }
          }
#pragma unroll
          for (int q = 0; q < EC / 16; ++q)
            if (nans >> (c0 / 16 + q) & 1u) {
#pragma unroll
              for (int c = 0; c < 16; ++c) v[16 * q + c] = NAN;
            }
          if (row_ok && whole) {
#pragma unroll
            for (int c = 0; c < EC; ++c) v[c] *= z.mul;
#pragma unroll
            for (int q = 0; q < EC / 8; ++q) *reinterpret_cast<uint4*>(o + c0 + 8 * q) = ordered8(v + 8 * q);
          } else if (row_ok) {
#pragma unroll
            for (int q = 0; q < EC / 4; ++q)
              *reinterpret_cast<float4*>(slot + rr * D + c0 + 4 * q) = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
          }
        }
        if (row_ok && (!both || t == 0)) {
          if (whole) {
            if (p.lse) p.lse[(size_t)h * p.T + part.row0 + node] = z.lse;
          } else {
            slot[C::ROWS * D + rr] = m;
            slot[C::ROWS * D + C::ROWS + rr] = l;
          }
        }
      }
      tc_fence_before();
      if (both) {  // the other warpgroup has read this one's sums: they may be overwritten
        __syncwarp();
        if (lane == 0) mbar_arrive(&x_read[t]);
        ok = tree_wait(&x_read[1 - t], nx & 1);
        ++nx;
      }
    }
  }

  tree_report(p, ok, warp < C::DEC_WARP ? kTreeSoftmax : warp < C::MMA_WARP ? kTreeDecode : kTreeIssue);
  tc_fence_before();
  __syncthreads();
  if (warp == C::MMA_WARP) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc<512>(tmem);
  }
}

// ------------------------------------------------------------------------------------------ few rows
// Up to 16 rows a kv head fill little of a 128-row tile, and its chain S - softmax - P V bounds a unit
// whatever its rows are.  So few rows are the columns of mma.sync products instead, whose 16 rows are tokens
// (scores) or head dims (outputs): four computing warps take 32 tokens of every unit each, decode their
// operands in registers, and keep their own sums.
// d (16 x 8 fp32) += a (16 x 16 bf16, rows) b (16 x 8 bf16, columns)
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// transpose of an 8 x 8 matrix of 16-bit values spread over a warp
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

template <int D, int NT>
struct FewCfg {
  static constexpr int DIM = D, ROWS = 8 * NT, WARPS = 4, THREADS = 32 * (WARPS + 1), LOAD_WARP = WARPS;
  static constexpr int CTAS = NT == 1 ? 3 : 2;  // CTAs an SM
  static constexpr int STAGES = 3, STAGE = kUnit * D * 9 / 8;
  static constexpr bool Q_SMEM = NT > 1;  // query fragments that do not fit the registers
  static constexpr int OFF_RAW = 0;
  static constexpr int OFF_Q = OFF_RAW + STAGES * STAGE;
  static constexpr int XS = D + 4;  // row stride of the exchange (bank spread)
  static constexpr int OFF_X = OFF_Q + (Q_SMEM ? (D / 16) * NT * 32 * 8 : 0);  // [WARPS][ROWS][XS] sums of the four warps
  static constexpr int OFF_ML = OFF_X + WARPS * ROWS * XS * 4;                 // [WARPS][ROWS] maxima, then denominators
  static constexpr int OFF_PART = OFF_ML + 2 * WARPS * ROWS * 4;
  static constexpr int OFF_BAR = OFF_PART + kParts * (int)sizeof(TreePart);
  static constexpr int SMEM = OFF_BAR + (2 * STAGES + 2 * kParts + 3) * 8 + 128;  // (aligned by the kernel)
  static constexpr int PART = ROWS * (D + 2);
  static_assert(CTAS * (SMEM + 1024) <= 228 * 1024, "shared memory of an SM");
};

template <int D, int NT>
__global__ void __launch_bounds__(FewCfg<D, NT>::THREADS, FewCfg<D, NT>::CTAS)
    kv4_tree_few_kernel(const Kv4TreeParams p, TreePiece* pieces, float* partial) {
  using C = FewCfg<D, NT>;
  constexpr int MT = D / 16;  // 16-row tiles of the head dim = k steps of a score
  constexpr int NST = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~(uintptr_t)127);
  uint64_t* raw_full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* raw_empty = raw_full + NST;
  uint64_t* part_full = raw_empty + NST;
  uint64_t* part_empty = part_full + kParts;
  uint64_t* x_ready = part_empty + kParts;  // every warp's sums of the part are there
  uint64_t* x_read = x_ready + 1;           // and every warp has read them
  uint64_t* q_ready = x_read + 1;
  TreePart* parts = reinterpret_cast<TreePart*>(smem + C::OFF_PART);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  grid_launch_dependents();  // the join may be set up meanwhile
  if (threadIdx.x == 0) {
    for (int s = 0; s < NST; ++s) {
      mbar_init(&raw_full[s], 1);
      mbar_init(&raw_empty[s], C::WARPS);
    }
    for (int s = 0; s < kParts; ++s) {
      mbar_init(&part_full[s], 1);
      mbar_init(&part_empty[s], C::WARPS);
    }
    mbar_init(x_ready, C::WARPS);
    mbar_init(x_read, C::WARPS);
    mbar_init(q_ready, C::WARPS);
    fence_barrier_init();
  }
  int b = 0;
  long long skip = 0, left = 0;
  if (warp == C::LOAD_WARP) tree_share<C::ROWS>(p, b, skip, left);
  __syncthreads();
  if (warp == C::LOAD_WARP) {
    tree_load<C>(p, pieces, smem, raw_full, raw_empty, parts, part_full, part_empty, b, skip, left);
    return;
  }
  // ------------------------------------------------------------------ computing warps
  float* xch = reinterpret_cast<float*>(smem + C::OFF_X);
  float* xm = reinterpret_cast<float*>(smem + C::OFF_ML);
  float* xl = xm + C::WARPS * C::ROWS;
  [[maybe_unused]] uint2* qs = reinterpret_cast<uint2*>(smem + C::OFF_Q);
  const int g = lane / 4, t = lane % 4;
  const float sl2 = p.scale_log2 * kKv4SmallUndo;
  // where this warp's tokens lie in a stage: tokens warp * 32 + 16 sub on start at token `in` of a
  // page, and sub 1 follows in the same page or is the next one
  const int P = p.c.page_size, in = warp * 32 & (P - 1);
  const int at_page = (warp * 32 >> p.c.page_shift) * kv4_block_bytes(P, D);
  const bool next_page = P == 16;
  const int d_k = next_page ? kv4_block_bytes(16, D) : 16 * (D / 2), d_sk = next_page ? d_k : 16 * (D / 16);
  const int off_k = at_page + (in + g) * (D / 2) + t * (D / 8);
  const int off_sk = at_page + kv4_off_sk(P, D) + (in + g) * (D / 16) + t * (D / 64);
  // token pairs u = 4 n + t of this warp's tokens: the slot permutation depends on t alone
  const int off_v = at_page + kv4_off_v(P, D) + (in / 2 + t) * D + (g ^ kv4_slot_xor(t, D)) * (D / 8);
  const int off_sv = at_page + kv4_off_sv(P, D) + (in / 2 + t) * (D / 8) + 2 * (D == 128 ? g : g / 2);
  int i = 0, n_part = 0;  // units, parts consumed
  bool ok = true;
  for (;; ++n_part) {
    ok = tree_wait(&part_full[n_part % kParts], (n_part / kParts) & 1);
    const TreePart& part = parts[n_part % kParts];
    if (!ok || part.cnt < 0) break;
    const int cnt = part.cnt;
    // (the rest of the part is read from shared memory where it is needed: few registers are left)
    // query fragments: lane (g, t) holds row 8 nt + g; dims [t D/4, (t + 1) D/4), in pairs (x, x + 4) of each
    // 8, the pairing of a code word's nibbles
    uint32_t qf[C::Q_SMEM ? 1 : MT][NT][2];
    {
      const int rem0 = part.rem0, node0 = part.node0, R = part.R, hk = part.hk, row0 = part.row0, G = part.G;
      const float inv_G = part.inv_G;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (C::Q_SMEM && nt != warp) continue;  // (warp nt stores tile nt; all have left the part before, see x_ready)
        const int r = 8 * nt + g, node = small_div(rem0 + r, inv_G);
        const uint4* src = reinterpret_cast<const uint4*>(
            p.q + ((size_t)(row0 + node0 + node) * p.H_q + hk * G + (rem0 + r - node * G)) * D + t * (D / 4));
#pragma unroll
        for (int j = 0; j < MT / 2; ++j) {
          uint4 w = make_uint4(0u, 0u, 0u, 0u);
          if (r < R) w = __ldg(src + j);
          const uint32_t p0 = __byte_perm(w.x, w.z, 0x5410), p1 = __byte_perm(w.x, w.z, 0x7632);
          const uint32_t p2 = __byte_perm(w.y, w.w, 0x5410), p3 = __byte_perm(w.y, w.w, 0x7632);
          if constexpr (C::Q_SMEM) {
            qs[((2 * j) * NT + nt) * 32 + lane] = make_uint2(p0, p1);
            qs[((2 * j + 1) * NT + nt) * 32 + lane] = make_uint2(p2, p3);
          } else {
            qf[2 * j][nt][0] = p0;
            qf[2 * j][nt][1] = p1;
            qf[2 * j + 1][nt][0] = p2;
            qf[2 * j + 1][nt][1] = p3;
          }
        }
      }
    }
    if constexpr (C::Q_SMEM) {
      __syncwarp();
      if (lane == 0) mbar_arrive(q_ready);
      ok = tree_wait(q_ready, n_part & 1);
      if (!ok) break;
    }
    float acc[MT][NT][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[mt][nt][e] = 0.f;
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
    }

    int unit = part.unit0;
    for (int k = 0; k < cnt; ++k, ++i, ++unit) {
      const int stage = i % NST, k0 = unit * kUnit + warp * 32;  // this warp's first token of the unit
      ok = tree_wait(&raw_full[stage], (i / NST) & 1);
      if (!ok) break;
      const bool edge = unit < part.u_win || unit >= part.u_tree;  // some token is hidden from some row
      if (!edge || (k0 < part.len && k0 + 32 > part.lo)) {
        const uint8_t* st = smem + C::OFF_RAW + stage * C::STAGE;
        float s[2][NT][4];
        // ---- scores of 2 x 16 tokens: lane (g, t) decodes tokens g, g + 8, its quarter of the dims
        uint32_t wk[2][2][MT / 2], sk[2][2];  // [half of 16][token g or g + 8]
#pragma unroll
        for (int sub = 0; sub < 2; ++sub)
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            const uint8_t* kc = st + off_k + sub * d_k + 8 * f * (D / 2);
            const uint8_t* ks = st + off_sk + sub * d_sk + 8 * f * (D / 16);
            if constexpr (D == 128) {
              *reinterpret_cast<uint4*>(wk[sub][f]) = *reinterpret_cast<const uint4*>(kc);
              sk[sub][f] = scale_pair(*reinterpret_cast<const unsigned short*>(ks));
            } else {
              *reinterpret_cast<uint2*>(wk[sub][f]) = *reinterpret_cast<const uint2*>(kc);
              sk[sub][f] = scale_pair(ks[0]);
            }
          }
#pragma unroll
        for (int sub = 0; sub < 2; ++sub)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[sub][nt][e] = 0.f;
#pragma unroll
        for (int j = 0; j < MT / 2; ++j)  // a word: 8 dims, two k steps; 16 dims share a scale
#pragma unroll
          for (int sub = 0; sub < 2; ++sub) {
            uint32_t a[2][4];
#pragma unroll
            for (int f = 0; f < 2; ++f) {
              const Kv4Small k2 = j < 2 ? scales_low(sk[sub][f]) : scales_high(sk[sub][f]);
              const uint4 v = decode8(wk[sub][f][j], k2);
              a[f][0] = v.x, a[f][1] = v.y, a[f][2] = v.z, a[f][3] = v.w;
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              uint2 q0, q1;
              if constexpr (C::Q_SMEM) {
                q0 = qs[((2 * j) * NT + nt) * 32 + lane];
                q1 = qs[((2 * j + 1) * NT + nt) * 32 + lane];
              } else {
                q0 = make_uint2(qf[2 * j][nt][0], qf[2 * j][nt][1]);
                q1 = make_uint2(qf[2 * j + 1][nt][0], qf[2 * j + 1][nt][1]);
              }
              mma_16816(s[sub][nt], a[0][0], a[1][0], a[0][1], a[1][1], q0.x, q0.y);
              mma_16816(s[sub][nt], a[0][2], a[1][2], a[0][3], a[1][3], q1.x, q1.y);
            }
          }
        // ---- softmax: s[sub][nt][e + 2 f] is token 16 sub + g + 8 f, row 8 nt + 2 t + e.  The running
        // maximum (in log2 units) moves only when some score passes it by 2^8
        uint32_t keep[2][2] = {{0xFFFFu, 0xFFFFu}, {0xFFFFu, 0xFFFFu}};  // the V scales that count, as read below
        if (edge) {
          const int len = part.len;
          uint32_t sees = 0u;  // lane r: the warp's 32 tokens that row r sees
          if (lane < C::ROWS) {
            const int row0 = part.row0, node = part.node0 + small_div(part.rem0 + min(lane, part.R - 1), part.inv_G), L = part.L, a0 = k0 - L, end = len - L;
            int lo = 0;
            if (p.window >= 0) {
              int depth = node;
              if (p.parents) {
                depth = 0;
                for (int a = tree_parent(p, row0, node); a >= 0; a = tree_parent(p, row0, a)) ++depth;
              }
              lo = depth >= p.window ? L : max(L - (p.window - depth), 0);
            }
            auto range = [&](int from, int to) {
              from = max(from, 0);
              to = min(to, 32);
              if (from < to) sees |= (0xffffffffu << from) & (0xffffffffu >> (32 - to));
            };
            range(lo - k0, L - k0);
            if (!p.parents) {
              range((p.window >= 0 && node > p.window ? min(node - p.window, end) : 0) - a0, min(node + 1, end) - a0);
            } else {
              int step = 0;
              for (int a = node; a >= max(a0, 0) && (p.window < 0 || step <= p.window); a = tree_parent(p, row0, a), ++step)
                if (a - a0 < 32 && a < end) sees |= 1u << (a - a0);
            }
          }
          __syncwarp();
          // A token that no row sees adds nothing, whatever its bytes are.  One with a NaN scale adds
          // nothing either: rows that do not see it have P = 0, but 0 times NaN is NaN.  The rows that see it
          // get their NaN here, and keep it.
          uint32_t nans = 0u;  // eighth g of the warp's 32 tokens, a bit each
#pragma unroll
          for (int sub = 0; sub < 2; ++sub)
#pragma unroll
            for (int f = 0; f < 2; ++f) {
              const int u = 8 * sub + 4 * f + t, j = k0 + 2 * u;
              uint32_t k2 = 0xFFFFu;
              if (j >= len || j < part.lo) k2 &= 0xFF00u;
              if (j + 1 >= len || j + 1 < part.lo) k2 &= 0x00FFu;
              const uint32_t two = k2 & *reinterpret_cast<const unsigned short*>(st + off_sv + sub * d_sk + 4 * f * (D / 8));
              if ((two & 0x00F8u) == 0x00F8u) {
                nans |= 1u << (2 * u);
                k2 &= 0xFF00u;
              }
              if ((two & 0xF800u) == 0xF800u) {
                nans |= 2u << (2 * u);
                k2 &= 0x00FFu;
              }
              keep[sub][f] = k2;
            }
          nans |= __shfl_xor_sync(0xffffffffu, nans, 1);
          nans |= __shfl_xor_sync(0xffffffffu, nans, 2);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint32_t row = __shfl_sync(0xffffffffu, sees, 8 * nt + 2 * t + e);
              if (nans & row) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) acc[mt][nt][e] = acc[mt][nt][e + 2] = NAN;
              }
#pragma unroll
              for (int sub = 0; sub < 2; ++sub)
#pragma unroll
                for (int f = 0; f < 2; ++f)
                  if (!(row >> (16 * sub + g + 8 * f) & 1u)) s[sub][nt][e + 2 * f] = -INFINITY;
            }
        }
        float mx[NT][2];
        bool grow = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            mx[nt][e] = sl2 * fmaxf(fmax3(s[0][nt][e], s[0][nt][e + 2], s[1][nt][e]), s[1][nt][e + 2]);
            grow |= mx[nt][e] > m[nt][e] + 8.f;
          }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
              for (int off = 4; off < 32; off <<= 1)
                mx[nt][e] = fmaxf(mx[nt][e], __shfl_xor_sync(0xffffffffu, mx[nt][e], off));
              const float mn = fmaxf(m[nt][e], mx[nt][e]);
              const float alpha = mn == m[nt][e] ? 1.f : ex2(m[nt][e] - mn);
              m[nt][e] = mn;
              l[nt][e] *= alpha;
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                acc[mt][nt][e] *= alpha;
                acc[mt][nt][e + 2] *= alpha;
              }
            }
        }
        uint32_t pb[2][NT][2];  // P as the column operand: rows of the product = tokens
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float m0 = m[nt][0] == -INFINITY ? 0.f : -m[nt][0], m1 = m[nt][1] == -INFINITY ? 0.f : -m[nt][1];
#pragma unroll
          for (int sub = 0; sub < 2; ++sub)
#pragma unroll
            for (int f = 0; f < 2; ++f) {
              const float x0 = ex2(fmaf(s[sub][nt][2 * f], sl2, m0));
              const float x1 = ex2(fmaf(s[sub][nt][2 * f + 1], sl2, m1));
              l[nt][0] += x0;
              l[nt][1] += x1;
              pb[sub][nt][f] = transpose_8x8(pack_bf16x2(x0, x1));
            }
        }
        // ---- outputs: lane (g, t) decodes eighth g of the head dim of token pairs t and t + 4
#pragma unroll
        for (int sub = 0; sub < 2; ++sub) {
          uint32_t lo[2][MT / 4], hi[2][MT / 4];  // [pair][word]: both tokens' nibbles 0-3, 4-7
          Kv4Small kv[2];
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            const uint8_t* va = st + off_v + sub * d_k + 4 * f * D;
            const uint32_t two = *reinterpret_cast<const unsigned short*>(st + off_sv + sub * d_sk + 4 * f * (D / 8));
            if constexpr (D == 128) {
              const uint4 w = *reinterpret_cast<const uint4*>(va);  // token 2u: x, y; token 2u + 1: z, w
              lo[f][0] = __byte_perm(w.x, w.z, 0x5410);
              hi[f][0] = __byte_perm(w.x, w.z, 0x7632);
              lo[f][1] = __byte_perm(w.y, w.w, 0x5410);
              hi[f][1] = __byte_perm(w.y, w.w, 0x7632);
            } else {
              const uint2 w = *reinterpret_cast<const uint2*>(va);
              lo[f][0] = __byte_perm(w.x, w.y, 0x5410);
              hi[f][0] = __byte_perm(w.x, w.y, 0x7632);
            }
            kv[f] = small_scales(scale_pair(two & keep[sub][f]));
          }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            // rows g and g + 8 of the tile: dims x and x + D/16 of the eighth
            uint32_t a[4];
#pragma unroll
            for (int f = 0; f < 2; ++f) {
              const int e = mt % 4;  // nibble of the half
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                const uint32_t* half = D == 128 ? (mt < 4 ? lo[f] : hi[f]) + (r * MT / 8) : r == 0 ? lo[f] : hi[f];
                const uint32_t w = *half >> (e < 2 ? 0 : 8);
                a[2 * f + r] = e % 2 == 0 ? decode_small_lo(w, kv[f]) : decode_small_hi(w, kv[f]);
              }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_16816(acc[mt][nt], a[0], a[1], a[2], a[3], pb[sub][nt][0], pb[sub][nt][1]);
          }
        }
      }
      __syncwarp();  // every lane has read the stage: it may be filled again
      if (lane == 0) mbar_arrive(&raw_empty[stage]);
    }
    if (!ok) break;

    // ---- the warps' sums become one: each leaves its own, with its maxima and denominators
    if (n_part > 0) ok = tree_wait(x_read, (n_part - 1) & 1);
    if (!ok) break;
    {
      float* mine = xch + warp * C::ROWS * C::XS;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = 8 * nt + 2 * t + e;
          float ll = l[nt][e];
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) ll += __shfl_xor_sync(0xffffffffu, ll, off);
          if (g == 0) {
            xm[warp * C::ROWS + r] = m[nt][e];
            xl[warp * C::ROWS + r] = ll;
          }
#pragma unroll
          for (int q = 0; q < MT / 2; ++q) {
            // D/8 consecutive dims of row r: tiles 0.. give the first half, their + 8 rows the second
            constexpr int QH = MT / 4;
            const int mt = 4 * (q % QH), hf = q / QH;
            *reinterpret_cast<float4*>(mine + r * C::XS + g * (D / 8) + 4 * q) =
                make_float4(acc[mt][nt][e + 2 * hf], acc[mt + 1][nt][e + 2 * hf], acc[mt + 2][nt][e + 2 * hf],
                            acc[mt + 3][nt][e + 2 * hf]);
          }
        }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(x_ready);
    ok = tree_wait(x_ready, n_part & 1);
    if (!ok) break;
    // ---- the whole of a segment: outputs; a piece of it: partial sums
    const bool whole = part.slot < 0;
    float* slot = partial + ((size_t)2 * blockIdx.x + max(part.slot, 0)) * C::PART;
    const int rem0 = part.rem0, node0 = part.node0, R = part.R, hk = part.hk, row0 = part.row0, G = part.G;
    const float inv_G = part.inv_G;
    for (int r = warp; r < R; r += C::WARPS) {
      float mm = xm[r], ll = 0.f, f[C::WARPS];
#pragma unroll
      for (int w = 1; w < C::WARPS; ++w) mm = fmaxf(mm, xm[w * C::ROWS + r]);
#pragma unroll
      for (int w = 0; w < C::WARPS; ++w) {
        const float mw = xm[w * C::ROWS + r], lw = xl[w * C::ROWS + r];
        f[w] = mw == -INFINITY ? 0.f : ex2(mw - mm);
        ll += mw == -INFINITY ? lw : lw * f[w];  // (no key: lw is 0, or a NaN that has to stay)
      }
      const int node = small_div(rem0 + r, inv_G), h = hk * G + rem0 + r - node * G, row = row0 + node0 + node;
      TreeSums z{1.f, 0.f};
      if (whole) z = tree_finish(p, h, mm, ll);
#pragma unroll
      for (int x = 2 * lane; x < D; x += 64) {
        float2 v = make_float2(0.f, 0.f);
#pragma unroll
        for (int w = 0; w < C::WARPS; ++w) {
          const float2 o = *reinterpret_cast<const float2*>(xch + (w * C::ROWS + r) * C::XS + x);
          v.x = fmaf(o.x, f[w], v.x);
          v.y = fmaf(o.y, f[w], v.y);
        }
        if (whole) *reinterpret_cast<uint32_t*>(p.o + ((size_t)row * p.H_q + h) * D + x) = pack_bf16x2(v.x * z.mul, v.y * z.mul);
        else *reinterpret_cast<float2*>(slot + r * D + x) = v;
      }
      if (lane == 0) {
        if (!whole) {
          slot[C::ROWS * D + r] = mm;
          slot[C::ROWS * D + C::ROWS + r] = ll;
        } else if (p.lse) {
          p.lse[(size_t)h * p.T + row] = z.lse;
        }
      }
    }
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(x_read);
      mbar_arrive(&part_empty[n_part % kParts]);
    }
  }
  tree_report(p, ok, kTreeFew);
}

// Joins the pieces of every segment that spans several CTAs, in CTA order: block (c, y) the segment whose
// first piece is CTA c's, if there is one.  WPR warps a row (few rows, whose segments span more CTAs): warp w
// takes pieces w, w + WPR, ..., then their sums are added in order.  Then the rows without a token, and on
// request those of no sequence.
// Launched while the kernel before it runs: it waits for that kernel's end before it reads a piece.
template <int D, int ROWS>
__global__ void __launch_bounds__(256) kv4_tree_join_kernel(const Kv4TreeParams p, const TreePiece* pieces, const float* partial) {
  constexpr int PART = ROWS * (D + 2), E = D / 32, WPR = ROWS <= 32 ? 64 / ROWS : 1, RPB = 8 / WPR;  // warps a row, rows a block
  __shared__ float red[2][8], sums[WPR > 1 ? 8 : 1][D];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, G = p.H_q / p.c.H_kv;
  grid_wait();
  // (ordinary loads: the pieces were written while this kernel was already set up)
  auto piece = [&](int i) {
    const int4* w = reinterpret_cast<const int4*>(pieces + i);
    const int4 a = w[0], b = w[1];
    return TreePiece{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  };
  auto store = [&](int t, int h, const float (&a)[E], const TreeSums& z) {
    // of 8 columns 0 .. 7 the tiles' forms hold the dims 0 4 1 5 2 6 3 7
    __nv_bfloat16* o = p.o + ((size_t)t * p.H_q + h) * D;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int col = lane * E + e, c = col & 7;
      o[ROWS >= 128 ? (col & ~7) + (c >> 1) + (c & 1) * 4 : col] = __float2bfloat16(a[e] * z.mul);
    }
    if (lane == 0 && p.lse) p.lse[(size_t)h * p.T + t] = z.lse;
  };
  const int c = blockIdx.x;
  const TreePiece p0 = piece(2 * c), p1 = piece(2 * c + 1);
  const bool second = p1.valid != 0;
  const TreePiece f = second ? p1 : p0;
  if (f.valid && f.starts) {
    int last = c;  // the CTA of the last piece: the next whose first piece is its segment's end
    if (!f.ends) {
      for (int base = c + 1; base < (int)gridDim.x; base += 32) {
        const int i = min(base + lane, (int)gridDim.x - 1);
        const unsigned end = __ballot_sync(0xffffffffu, pieces[2 * i].ends != 0 || i == (int)gridDim.x - 1);
        last = min(base + (end ? __ffs(end) - 1 : 31), (int)gridDim.x - 1);
        if (end) break;
      }
    }
    for (int r0 = blockIdx.y * RPB; r0 < f.R; r0 += gridDim.y * RPB) {
      const int r = r0 + warp / WPR;
      float a[E], m = -INFINITY, l = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) a[e] = 0.f;
      if (r < f.R) {
#pragma unroll 4
        for (int i = c + warp % WPR; i <= last; i += WPR) {
          const float* sl = partial + ((size_t)2 * i + (i == c && second ? 1 : 0)) * PART;
          const float mi = sl[ROWS * D + r], li = sl[ROWS * D + ROWS + r];
          float v[E];
#pragma unroll
          for (int e = 0; e < E; e += 2) {
            const float2 x = *reinterpret_cast<const float2*>(sl + r * D + lane * E + e);
            v[e] = x.x;
            v[e + 1] = x.y;
          }
          const float mn = fmaxf(m, mi);
          const float fo = m == -INFINITY ? 0.f : ex2(m - mn), w = mi == -INFINITY ? 0.f : ex2(mi - mn);
          l = (m == -INFINITY ? l : l * fo) + (mi == -INFINITY ? li : li * w);  // (no key: 0, or a NaN that has to stay)
#pragma unroll
          for (int e = 0; e < E; ++e) a[e] = a[e] * fo + v[e] * w;  // (a NaN stays, also of a piece without weight)
          m = mn;
        }
      }
      if constexpr (WPR > 1) {
        __syncthreads();  // (the sums of the row before are read)
        if (lane == 0) {
          red[0][warp] = m;
          red[1][warp] = l;
        }
#pragma unroll
        for (int e = 0; e < E; ++e) sums[warp][lane * E + e] = a[e];
        __syncthreads();
        if (warp % WPR != 0) continue;
        m = red[0][warp];
        for (int w = 1; w < WPR; ++w) m = fmaxf(m, red[0][warp + w]);
        l = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) a[e] = 0.f;
#pragma unroll
        for (int w = 0; w < WPR; ++w) {
          const float mw = red[0][warp + w], lw = red[1][warp + w], fo = mw == -INFINITY ? 0.f : ex2(mw - m);
          l += mw == -INFINITY ? lw : lw * fo;
#pragma unroll
          for (int e = 0; e < E; ++e) a[e] = fmaf(sums[warp + w][lane * E + e], fo, a[e]);
        }
      }
      if (r < f.R) {
        const int node = (f.rem0 + r) / G, h = f.hk * G + f.rem0 + r - node * G;
        store(f.row0 + f.node0 + node, h, a, tree_finish(p, h, m, l));
      }
    }
  }
  const float none[E] = {};
  const int w_all = ((int)blockIdx.x * gridDim.y + blockIdx.y) * 8 + warp, n_all = gridDim.x * gridDim.y * 8;
  for (int b = w_all; b < p.B; b += n_all) {
    const TreeSeq s = tree_seq<ROWS>(p, b);
    if (s.units > 0) continue;
    for (int t = s.row0; t < s.row0 + s.n; ++t)
      for (int h = 0; h < p.H_q; ++h) store(t, h, none, tree_finish(p, h, -INFINITY, 0.f));
  }
  if (p.zero_rest) {
    const int first = max(p.cu[0], 0), end = max(min(p.cu[p.B], p.T), 0);
    for (int t = w_all; t < p.T; t += n_all) {
      if (t >= first && t < end) continue;
      for (int h = 0; h < p.H_q; ++h) store(t, h, none, TreeSums{0.f, -INFINITY});
    }
  }
}

namespace {

constexpr int kMaxGrid = 152 * 3;  // CTAs, each with two places for partial sums
constexpr size_t kPieceBytes = (kMaxGrid * 2 * sizeof(TreePiece) + 255) / 256 * 256;

// SMs of the current device (0: CUDA cannot tell), looked up once.
int device_sms() {
  static std::atomic<int> sms[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  int n = sms[dev].load(std::memory_order_acquire);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 0;
    sms[dev].store(n, std::memory_order_release);
  }
  return n;
}

template <auto KERN, class C>
int launch_t(const Kv4TreeParams& p, int ctas, void* workspace, cudaStream_t stream) {
  const int n = device_sms();
  if (n == 0 || !allow_smem<KERN>(C::SMEM)) return -1;
  const int grid = std::min(n, 152) * ctas;
  TreePiece* pieces = static_cast<TreePiece*>(workspace);
  float* partial = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kPieceBytes);
  if (launch_kernel(KERN, dim3((unsigned)grid), C::THREADS, C::SMEM, stream, false, p, pieces, partial) != 0) return -1;
  // (256 rows: 16 blocks a segment, two rows a warp; with 8 one sequence of 131,072 tokens takes 127 us instead of 121.
  // Fewer rows: more blocks take longer to start than they save.)
  return launch_kernel(kv4_tree_join_kernel<C::DIM, C::ROWS>, dim3((unsigned)grid, C::ROWS == 256 ? 16 : 8), 256, 0, stream, true, p,
                       (const TreePiece*)pieces, (const float*)partial);
}
template <int D, int NT>
int launch_few(const Kv4TreeParams& p, void* workspace, cudaStream_t stream) {
  using C = FewCfg<D, NT>;
  return launch_t<kv4_tree_few_kernel<D, NT>, C>(p, C::CTAS, workspace, stream);
}
template <int D, bool TWO>
int launch_tiles(const Kv4TreeParams& p, void* workspace, cudaStream_t stream) {
  return launch_t<kv4_tree_kernel<D, TWO>, TreeCfg<D, TWO>>(p, 1, workspace, stream);
}

// Rows of a block, by the sequences' rows a kv head on average: a block of more than a sequence has works on
// rows that do not exist, a smaller one decodes the cache again for the rest.  Measured on both sides of a bound (heads
// of 128 / 64): 131,072 tokens with 16 rows 52 / 37 us as columns, 78 / 59 as a tile; with 32 rows 87 / 57 as columns, 78 /
// 59 as a tile, and 76 sequences of 100 tokens 39 / 31 and 29 / 23.  One tile 178 us and two 260 for 329,377 tokens of 8
// heads, so that 256 rows as two blocks of one tile would take 356.
// These are even batches.  The average counts sequences without nodes and rows of no sequence too, so a large sequence among
// small ones gets blocks too small for it: 131,072 tokens with 64 nodes (4 heads a kv head) take 124 us alone, 822 beside 31
// sequences without nodes and 596 beside 31 of 2000 tokens with one node (29 alone); a chain of 512 nodes over 4096 tokens 60
// alone, 348 beside 255 of 2000 tokens with one node (133 alone).
int block_rows(int B, int T, int H_q, int H_kv) {
  const long long rows = (long long)T * (H_q / H_kv), n = B > 0 ? B : 1;
  return rows <= 8 * n ? 8 : rows <= 16 * n ? 16 : rows <= 128 * n ? 128 : 256;
}

}  // namespace

size_t kv4_tree_workspace(int B, int T, int H_q, int H_kv, int d) {
  const int rows = block_rows(B, T, H_q, H_kv), ctas = rows == 8 ? 3 : rows == 16 ? 2 : 1;
  return kPieceBytes + (size_t)152 * ctas * 2 * rows * (d + 2) * sizeof(float);
}

int launch_kv4_tree(const Kv4TreeParams& p, void* workspace, cudaStream_t stream) {
  switch (block_rows(p.B, p.T, p.H_q, p.c.H_kv)) {
    case 8: return p.c.d == 128 ? launch_few<128, 1>(p, workspace, stream) : launch_few<64, 1>(p, workspace, stream);
    case 16: return p.c.d == 128 ? launch_few<128, 2>(p, workspace, stream) : launch_few<64, 2>(p, workspace, stream);
    case 128: return p.c.d == 128 ? launch_tiles<128, false>(p, workspace, stream) : launch_tiles<64, false>(p, workspace, stream);
    default: return p.c.d == 128 ? launch_tiles<128, true>(p, workspace, stream) : launch_tiles<64, true>(p, workspace, stream);
  }
}

}  // namespace sdpa
