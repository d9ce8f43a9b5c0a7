// kv4_decode.cu -- attention of a sequence's newest tokens over its 4-bit paged cache
// (layout and number format in kv4.cuh).
//
//   S_j = scale q.k_j over the keys j in [pos - window, pos], pos the query's own place in
//   the sequence (the S_q queries are its last S_q tokens); softmax with an optional sink
//   logit; o = P V; lse = log of the denominator.
//
// Bound by reading the cache (9d/8 bytes for each token and kv head), so each byte is read
// once for all query rows that share a kv head (rows = G S_q, in blocks of 8 NT <= 32), and
// the arithmetic must keep up with the memory: 23 bytes a cycle and SM are 41 values to
// decode, for which the CUDA cores have 3 instructions each and no time left for products.
//   - Products run on the tensor core as mma.sync m16n8k16 with tokens (scores) or head dims
//     (outputs) as the 16 rows and the query rows as the 8 columns, so that a group of 4 to 8
//     query heads wastes little of it, and a decoded operand serves every column block.
//     (A tcgen05 product wants 128 rows of decoded operand in shared memory or TMEM: writing
//     them back costs more than the whole decode.)
//   - A code pair is decoded by a mask and one paired fma with the scale, as (c - 8) s 2^-23
//     (kv4.cuh; the power of two is undone in the scores' scale and in the outputs): exact, and
//     half of the codes need no shift.  Which pairs of dims or tokens share a register is free
//     as long as both operands of a product agree, so a lane's 16-byte load feeds its own
//     fragments.
//   - The probabilities are rounded to bf16 (2^-8 relative) for P V; their sum is fp32.
//   - Work is cut evenly over the CTAs of a persistent grid (units of 128 tokens of one
//     sequence and kv head, in order, and one unit more for each such segment: its queries,
//     the sum over its warps and its output cost about as much), whatever the lengths; a
//     (sequence, head) that spans several CTAs leaves fp32 partial sums in the workspace, which a
//     second kernel joins in CTA order: bitwise reproducible.
//   - A fifth warp walks the page table and streams units into a ring, a page and head in one
//     bulk copy; each of the other four takes 32 tokens of every unit.
//
// Measured (d = 128, 8 kv heads): 329,377 tokens of 4 sequences with 8 query rows a kv head, 380 MB
// of cache, 76 us (5.0 TB/s; the copies alone 66.  Steps before: 88 with an exponent set in every code
// and a shift for three of four, 80 with four copies a page, 78 with hidden tokens masked in the output
// loop); 42,031 tokens of 16 sequences, 48 MB, 21 us, of which about 10 are the chain lengths - page -
// copy - products - join.  More query rows a kv head are bound by the computing warps, of which fewer fit an
// SM: the same tokens take 106 us with 9 to 16 rows and 176 with 17 to 32.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "attn_common.cuh"
#include "attn_kernels.h"
#include "kv4.cuh"
#include "launch.h"
#include "ptx.cuh"

namespace sdpa {

namespace {

constexpr int kWarps = 4;                  // computing warps
constexpr int kSub = 32;                   // tokens of a unit that one warp takes
constexpr int kUnit = kWarps * kSub;       // tokens of one unit (one ring stage)
constexpr int kStages = 3;
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kMaxCtas = 152 * 4;  // partial-sum slots in the workspace
constexpr int kSegCost = 1;        // a segment's fixed costs, in units

enum Kv4Site { kKv4Full = 0xA0, kKv4Empty };

// d (16 x 8 fp32) += a (16 x 16 bf16, rows) b (16 x 8 bf16, columns)
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// d = a b
__device__ __forceinline__ void mma_16816_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// transpose of an 8 x 8 matrix of 16-bit values spread over a warp
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// A row's end: sums relative to maximum m (log2 units), the sink joins the denominator.
struct Kv4Sums {
  float mul, lse;  // what the sums are multiplied by; log of the denominator
};
__device__ __forceinline__ Kv4Sums kv4_finish(const Kv4DecodeParams& p, int h, float m, float l) {
  const float sink = p.softmax_type == 0 ? -INFINITY : p.softmax_type == 1 ? 0.f : p.offset[h] * kLog2e;
  const float mm = fmaxf(m, sink);
  if (mm == -INFINITY) return l == l ? Kv4Sums{0.f, -INFINITY} : Kv4Sums{l, l};  // no key (l is 0) or a NaN
  const float f = m == -INFINITY ? 0.f : ex2(m - mm);
  const float den = l * f + (sink == -INFINITY ? 0.f : ex2(sink - mm));
  return Kv4Sums{f / den * kKv4SmallUndo, (mm + lg2(den)) * kLn2};
}

// The keys of one unit row and the sizes of one sequence.
struct Seq {
  int len;    // tokens in the cache
  int lo;     // first token any query sees
  int first;  // its unit
  int n;      // units
  __device__ __forceinline__ int numbers() const { return n > 0 ? n + kSegCost : 0; }
};
__device__ __forceinline__ Seq seq_of(const Kv4DecodeParams& p, int b) {
  Seq s;
  s.len = entry_len(p.seq_lens, b, p.c.max_pages * p.c.page_size);
  s.lo = p.window >= 0 && s.len - p.S_q > p.window ? s.len - p.S_q - p.window : 0;  // the first query's
  s.first = s.lo / kUnit;
  s.n = s.len > 0 ? (s.len - 1) / kUnit - s.first + 1 : 0;
  return s;
}

// How the units of a call are numbered: sequence by sequence, each sequence's H_eff heads (kv
// head and row block) one after another; a segment (sequence, head) of n units has n + kSegCost
// numbers, the first of them for its fixed costs.  Every warp works this out for itself: a few loads
// and shuffles, and no barrier.
struct UnitScan {
  long long total;  // numbers of all sequences and heads
  int n, upto;      // up to 32 sequences: this lane's sequence, and all up to and with it (one head's)
  __device__ __forceinline__ static int numbers_of(const Kv4DecodeParams& p, int b) {
    return b < p.B ? seq_of(p, b).numbers() : 0;
  }
  __device__ void run(const Kv4DecodeParams& p, int H_eff) {
    const int lane = threadIdx.x % 32;
    if (p.B <= 32) {  // (a sequence has less than 2^24 units)
      n = upto = numbers_of(p, lane);
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, upto, off);
        if (lane >= off) upto += o;
      }
      total = (long long)__shfl_sync(0xffffffffu, upto, 31) * H_eff;
      return;
    }
    long long t = 0;
    for (int b = lane; b < p.B; b += 32) t += numbers_of(p, b);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
    total = t * H_eff;
  }
  // The numbers before sequence b.
  __device__ long long before(const Kv4DecodeParams& p, int H_eff, int b) const {
    if (p.B <= 32) return (long long)__shfl_sync(0xffffffffu, upto - n, b) * H_eff;
    long long t = 0;
    for (int i = threadIdx.x % 32; i < b; i += 32) t += numbers_of(p, i);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
    return t * H_eff;
  }
  // The sequence that holds number u, and the numbers before it.
  __device__ long long find(const Kv4DecodeParams& p, int H_eff, long long u, int* b) const {
    const int lane = threadIdx.x % 32;
    if (p.B <= 32) {
      const int w = __ffs(__ballot_sync(0xffffffffu, u < (long long)upto * H_eff)) - 1;
      *b = w;
      return (long long)__shfl_sync(0xffffffffu, upto - n, w) * H_eff;
    }
    long long carry = 0;
    for (int base = 0;; base += 32) {  // (u < total: some sequence holds it)
      const long long m = (long long)numbers_of(p, base + lane) * H_eff;
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

// CTA c of n takes units [cta_first(c), cta_first(c + 1)).
// (32-bit division where the product fits, as it nearly always does)
__device__ __forceinline__ long long muldiv(long long a, int b, long long d) {
  return a < (1 << 22) && d < (1LL << 32) ? (long long)((unsigned)a * (unsigned)b / (unsigned)d) : a * b / d;
}
static_assert(((1LL << 22) - 1) * kMaxCtas < (1LL << 32), "the 32-bit product");
__device__ __forceinline__ long long cta_first(long long total, int n, int c) { return muldiv(total, c, n); }
__device__ __forceinline__ int cta_of(long long total, int n, long long u) {
  int c = (int)muldiv(u, n, total);  // near the last c with cta_first(c) <= u
  while (c > 0 && cta_first(total, n, c) > u) --c;
  while (c + 1 < n && cta_first(total, n, c + 1) <= u) ++c;
  return c;
}
__device__ __forceinline__ int ctas_used(long long total, int grid) {
  const long long want = (total + kSegCost) / (kSegCost + 1);
  return want < grid ? (int)want : grid;
}

template <int D, int NT>
struct DecCfg {
  static constexpr int ROWS = 8 * NT;
  static constexpr int STAGE = kUnit * D * 9 / 8;
  static constexpr int OFF_Q = kStages * STAGE;  // query fragments where they do not stay in registers
  static constexpr bool Q_SMEM = NT > 2;
  static constexpr int Q_BYTES = Q_SMEM ? (D / 16) * NT * 32 * 8 : 0;
  static constexpr int XS = D + 4;  // row stride of the exchange (bank spread)
  static constexpr int OFF_X = OFF_Q + Q_BYTES;                  // [kWarps][ROWS][XS] sums of the four warps
  static constexpr int OFF_ML = OFF_X + kWarps * ROWS * XS * 4;  // [kWarps][ROWS] maxima, then denominators
  static constexpr int OFF_BAR = OFF_ML + 2 * kWarps * ROWS * 4;  // full[kStages], empty[kStages]
  static constexpr int SMEM = OFF_BAR + 2 * kStages * 8;
  static constexpr int SLOT = ROWS * (D + 2);  // floats of one partial: rows of sums, maxima, denominators
};

}  // namespace

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 3 : NT == 2 ? 2 : 1)
    kv4_decode_kernel(const Kv4DecodeParams p, int row_blocks, float* partial) {
  using C = DecCfg<D, NT>;
  constexpr int MT = D / 16;  // 16-row tiles of the head dim = k steps of a score
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* empty = full + kStages;
  const int G = p.H_q / p.c.H_kv, R = G * p.S_q, H_eff = p.c.H_kv * row_blocks;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kWarps);
    }
    fence_barrier_init();
  }
  grid_launch_dependents();  // the join may be set up meanwhile
  UnitScan scan;
  scan.run(p, H_eff);
  __syncthreads();  // the barriers are set up
  if (scan.total == 0) return;
  const int n_cta = ctas_used(scan.total, gridDim.x);
  if ((int)blockIdx.x >= n_cta) return;
  const long long u_begin = cta_first(scan.total, n_cta, blockIdx.x);
  const long long u_end = cta_first(scan.total, n_cta, blockIdx.x + 1);
  // The CTA's units are a run of segments: units of one (sequence, kv head, row block) in order.
  struct Cursor {
    int b, vh;      // sequence, kv head and row block
    int from, to;   // this CTA's units of it (from == to: only its fixed costs)
    int left;       // numbers of this CTA after this segment
    Seq s;
  } at;
  auto enter = [&](Cursor& c, int number) {  // the segment from its `number` on
    const int take = min(c.s.numbers() - number, c.left);
    c.from = max(number - kSegCost, 0);
    c.to = max(number + take - kSegCost, 0);
    c.left -= take;
  };
  auto next_segment = [&](Cursor& c) {
    if (++c.vh == H_eff) {
      c.vh = 0;
      do {
        ++c.b;
        c.s = seq_of(p, c.b);
      } while (c.s.n == 0);
    }
    enter(c, 0);
  };
  {
    const long long r = u_begin - scan.find(p, H_eff, u_begin, &at.b);
    at.s = seq_of(p, at.b);
    at.vh = (int)(r / at.s.numbers());
    at.left = (int)(u_end - u_begin);
    enter(at, (int)(r % at.s.numbers()));
  }

  if (warp == kWarps) {
    // ---------------------------------------------------------------- producer
    // Lane i copies the block of page i of a unit (whole, also past the sequence's end), if some query
    // sees a token of it: the pages before a window may be gone from the table.  Its page is looked up
    // one unit ahead.
    const int P = p.c.page_size, pieces = kUnit / P, t0 = lane * P;
    const int block = kv4_block_bytes(P, D);
    const size_t page_bytes = (size_t)block * p.c.H_kv;
    int unit = at.from;
    auto settle = [&]() {  // to the next unit there is; false: none
      while (unit >= at.to) {
        if (at.left == 0) return false;
        next_segment(at);
        unit = at.from;
      }
      return true;
    };
    auto page_of = [&]() {
      const int tok = (at.s.first + unit) * kUnit + t0;
      return lane < pieces && tok < at.s.len && tok + P > at.s.lo ? kv4_page(p.c, at.b, tok) : -2;
    };
    bool more = settle();
    int page = more ? page_of() : -2, n = 0;
    bool ok = true;
    for (; more && ok; ++n) {
      const int stage = n % kStages;
      uint8_t* st = smem + stage * C::STAGE;
      const uint8_t* src = p.pool + (size_t)max(page, 0) * page_bytes + (size_t)(at.vh / row_blocks) * block;
      const int have = page;
      ++unit;
      more = settle();
      if (more) page = page_of();
      if (n >= kStages) ok = mbar_wait_warp(&empty[stage], (n / kStages - 1) & 1, p.err, kKv4Empty);
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
      if (lane == 0) mbar_arrive_expect_tx(&full[stage], all);
      __syncwarp();
      if (have >= 0) bulk_load(st + lane * block, src, block, &full[stage]);
    }
    // every copy this warp started must land before the CTA may exit: wait for the last ones
    for (int s = 0; s < kStages && s < n; ++s) {
      const int last = s + (n - 1 - s) / kStages * kStages;
      mbar_wait_warp(&full[s], (last / kStages) & 1, p.err, kKv4Full);
    }
    return;
  }

  // ------------------------------------------------------------------ computing warps
  float* xch = reinterpret_cast<float*>(smem + C::OFF_X);
  float* xm = reinterpret_cast<float*>(smem + C::OFF_ML);
  float* xl = xm + kWarps * C::ROWS;
  const int g = lane / 4, t = lane % 4;
  // where this warp's tokens lie in a stage: tokens warp * 32 + 16 sub on start at token `in` of a
  // page, and sub 1 follows in the same page or is the next one
  const int P = p.c.page_size, in = warp * kSub & (P - 1);
  const int at_page = warp * kSub / P * kv4_block_bytes(P, D);
  const bool next_page = P == 16;
  const int d_k = next_page ? kv4_block_bytes(16, D) : 16 * (D / 2), d_sk = next_page ? d_k : 16 * (D / 16);
  const int off_k = at_page + (in + g) * (D / 2) + t * (D / 8);
  const int off_sk = at_page + kv4_off_sk(P, D) + (in + g) * (D / 16) + t * (D / 64);
  // token pairs u = 4 n + t of this warp's tokens: the slot permutation depends on t alone
  const int off_v = at_page + kv4_off_v(P, D) + (in / 2 + t) * D + (g ^ kv4_slot_xor(t, D)) * (D / 8);
  const int off_sv = at_page + kv4_off_sv(P, D) + (in / 2 + t) * (D / 8) + 2 * (D == 128 ? g : g / 2);
  const float sl2 = p.scale_log2 * kKv4SmallUndo;
  int i = 0;  // units consumed
  bool ok = true;
  for (bool at_begin = true;; at_begin = false) {
    if (at.from == at.to) {
      if (at.left == 0) break;
      next_segment(at);
      continue;
    }
    const int seg_n = at.to - at.from;
    const bool whole = seg_n == at.s.n;
    const int hk = at.vh / row_blocks, r0 = (at.vh % row_blocks) * C::ROWS;
    const int len = at.s.len;
    // query fragments: lane (g, t) holds row r0 + 8 nt + g; dims [t D/4, (t + 1) D/4), in pairs
    // (x, x + 4) of each 8, the pairing of a code word's nibbles
    uint32_t qf[C::Q_SMEM ? 1 : MT][NT][2];
    [[maybe_unused]] uint2* qs = reinterpret_cast<uint2*>(smem + C::OFF_Q);
    if (!C::Q_SMEM || warp == 0) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int r = r0 + 8 * nt + g;
        const uint4* src = reinterpret_cast<const uint4*>(
            p.q + (((size_t)at.b * p.S_q + r / G) * p.H_q + hk * G + r % G) * D + t * (D / 4));
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
    if constexpr (C::Q_SMEM) named_bar_sync(1, 32 * kWarps);
    // keys that every row sees: [lo_max, hi_min]; that some row sees: [lo_min, len - 1]
    const int hi_min = len - p.S_q + r0 / G;
    const int lo_max = p.window >= 0 ? len - 1 - p.window : 0;
    const int lo_min = at.s.lo;
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

    int k0 = (at.s.first + at.from) * kUnit + warp * kSub;  // this warp's first token of the unit
    for (int k = 0; k < seg_n; ++k, ++i, k0 += kUnit) {
      const int stage = i % kStages;
      ok = ok && mbar_wait_warp(&full[stage], (i / kStages) & 1, p.err, kKv4Full);
      if (ok && k0 < len && k0 + kSub > lo_min) {
        const uint8_t* st = smem + stage * C::STAGE;
        const bool edge = k0 + kSub - 1 > hi_min || k0 < lo_max;  // some key is hidden from some row
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
        for (int j = 0; j < MT / 2; ++j)  // a word: 8 dims, two k steps; 16 dims share a scale
#pragma unroll
          for (int sub = 0; sub < 2; ++sub) {
            uint32_t a[2][4];
#pragma unroll
            for (int f = 0; f < 2; ++f) {
              const Kv4Small k2 = small_scales(__byte_perm(sk[sub][f], 0u, j < 2 ? 0x1010 : 0x3232));
              const uint32_t w = wk[sub][f][j], w8 = w >> 8;
              a[f][0] = decode_small_lo(w, k2);
              a[f][1] = decode_small_hi(w, k2);
              a[f][2] = decode_small_lo(w8, k2);
              a[f][3] = decode_small_hi(w8, k2);
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
              if (j == 0) mma_16816_zero(s[sub][nt], a[0][0], a[1][0], a[0][1], a[1][1], q0.x, q0.y);
              else mma_16816(s[sub][nt], a[0][0], a[1][0], a[0][1], a[1][1], q0.x, q0.y);
              mma_16816(s[sub][nt], a[0][2], a[1][2], a[0][3], a[1][3], q1.x, q1.y);
            }
          }
        // ---- softmax: s[sub][nt][e + 2 f] is token 16 sub + g + 8 f, row r0 + 8 nt + 2 t + e.  The
        // running maximum (in log2 units) moves only when some score passes it by 2^8 (the sums
        // stay exact: they are relative to the maximum that was used)
        uint32_t keep[2][2] = {{0xFFFFu, 0xFFFFu}, {0xFFFFu, 0xFFFFu}};  // the V scales that count, as read below
        if (edge) {
          // A token that no row sees adds nothing, whatever its bytes are.  One with a NaN scale adds
          // nothing either: rows that do not see it have P = 0, but 0 times NaN is NaN.  The rows that
          // see it get their NaN here, and keep it.
          uint32_t nans = 0u;  // eighth g of the warp's 32 tokens, a bit each
#pragma unroll
          for (int sub = 0; sub < 2; ++sub)
#pragma unroll
            for (int f = 0; f < 2; ++f) {
              const int u = 8 * sub + 4 * f + t, j = k0 + 2 * u;
              uint32_t k2 = 0xFFFFu;
              if (j > len - 1 || j < lo_min) k2 &= 0xFF00u;
              if (j + 1 > len - 1 || j + 1 < lo_min) k2 &= 0x00FFu;
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
          if (__any_sync(0xffffffffu, nans != 0u)) {  // (rare)
            nans |= __shfl_xor_sync(0xffffffffu, nans, 1);
            nans |= __shfl_xor_sync(0xffffffffu, nans, 2);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int pos = len - p.S_q + min(r0 + 8 * nt + 2 * t + e, R - 1) / G;
                const int lo = p.window >= 0 && pos > p.window ? pos - p.window : 0;
                if (pos < k0 || lo - k0 > 31) continue;  // the row sees none of the 32
                const int from = max(lo - k0, 0), to = min(pos - k0, 31);
                if (nans & (0xffffffffu << from) & (0xffffffffu >> (31 - to))) {
#pragma unroll
                  for (int mt = 0; mt < MT; ++mt) acc[mt][nt][e] = acc[mt][nt][e + 2] = NAN;
                }
              }
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int pos = len - p.S_q + min(r0 + 8 * nt + 2 * t + e, R - 1) / G;
              const int lo = p.window >= 0 && pos > p.window ? pos - p.window : 0;
#pragma unroll
              for (int sub = 0; sub < 2; ++sub)
#pragma unroll
                for (int f = 0; f < 2; ++f) {
                  const int j = k0 + 16 * sub + g + 8 * f;
                  if (j > pos || j < lo) s[sub][nt][e + 2 * f] = -INFINITY;
                }
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
      if (lane == 0) mbar_arrive(&empty[stage]);
    }

    // ---- the warps' sums become one: each leaves its own, with its maxima and denominators
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
    named_bar_sync(1, 32 * kWarps);
    // ---- the whole of a (sequence, head): outputs; a piece of it: partial sums
    float* slot = partial + ((size_t)2 * blockIdx.x + (at_begin ? 0 : 1)) * C::SLOT;
    for (int r = warp; r < C::ROWS && r0 + r < R; r += kWarps) {
      float mm = xm[r], ll = 0.f, f[kWarps];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) mm = fmaxf(mm, xm[w * C::ROWS + r]);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float mw = xm[w * C::ROWS + r], lw = xl[w * C::ROWS + r];
        f[w] = mw == -INFINITY ? 0.f : ex2(mw - mm);
        ll += mw == -INFINITY ? lw : lw * f[w];  // (no key: lw is 0, or a NaN that has to stay)
      }
      auto sum2 = [&](int x) {  // dims x, x + 1
        float2 v = make_float2(0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float2 o = *reinterpret_cast<const float2*>(xch + (w * C::ROWS + r) * C::XS + x);
          v.x = fmaf(o.x, f[w], v.x);
          v.y = fmaf(o.y, f[w], v.y);
        }
        return v;
      };
      if (whole) {
        const int qs_ = (r0 + r) / G, h = hk * G + (r0 + r) % G;
        const Kv4Sums z = kv4_finish(p, h, mm, ll);
        __nv_bfloat16* o = p.o + (((size_t)at.b * p.S_q + qs_) * p.H_q + h) * D;
#pragma unroll
        for (int x = 2 * lane; x < D; x += 64) {
          const float2 v = sum2(x);
          *reinterpret_cast<uint32_t*>(o + x) = pack_bf16x2(v.x * z.mul, v.y * z.mul);
        }
        if (lane == 0 && p.lse) p.lse[((size_t)at.b * p.H_q + h) * p.S_q + qs_] = z.lse;
      } else {
#pragma unroll
        for (int x = 2 * lane; x < D; x += 64) *reinterpret_cast<float2*>(slot + r * D + x) = sum2(x);
        if (lane == 0) {
          slot[C::ROWS * D + r] = mm;
          slot[C::ROWS * D + C::ROWS + r] = ll;
        }
      }
    }
    if (at.left == 0) break;
    named_bar_sync(1, 32 * kWarps);  // the exchange is free for the next segment
    next_segment(at);
  }
}

// Joins the pieces of every (sequence, head) that spans several CTAs, in CTA order, and writes the
// rows of sequences without a token.  One block per (sequence, kv head, row block, row): warp w
// takes pieces w, w + 8, ..., then the eight are added in order.  (A warp per row, taking its
// pieces one after another, took 12.3 us instead of 8.9 for 128 segments of 1 to 11 pieces.)  Every
// block works out the numbering for itself, so that above 32 sequences the join's work grows with the square of
// their number: 256 sequences of 500 to 4000 tokens, 8 kv heads of 4 rows, take 183 us with a floor of
// 94, 1024 of them 967 with a floor of 396.
// Launched while the decode kernel runs: it waits for that kernel's end before it reads a piece.  (The
// lengths it reads before are older than the decode kernel, which began when all before it on the
// stream had ended.)
template <int D>
__global__ void __launch_bounds__(256) kv4_join_kernel(const Kv4DecodeParams p, int row_blocks, int rows, int grid,
                                                       const float* partial) {
  const int G = p.H_q / p.c.H_kv, R = G * p.S_q, H_eff = p.c.H_kv * row_blocks;
  const int b = blockIdx.x / H_eff, vh = blockIdx.x % H_eff;
  const int hk = vh / row_blocks, row0 = (vh % row_blocks) * rows;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const Seq s = seq_of(p, b);
  UnitScan scan;
  scan.run(p, H_eff);
  long long u0 = 0;
  int n_cta = 1, c0 = 0, c1 = 0;
  if (s.n > 0) {
    u0 = scan.before(p, H_eff, b) + (long long)vh * s.numbers();
    n_cta = ctas_used(scan.total, grid);
    c0 = cta_of(scan.total, n_cta, u0 + kSegCost);
    c1 = cta_of(scan.total, n_cta, u0 + kSegCost + s.n - 1);
  }
  // every block waits, also one with nothing to do: this grid must not end before the decode
  // kernel, or what follows on the stream could start beside it
  grid_wait();
  if (s.n > 0 && c0 == c1) return;  // one CTA had all of it
  const int slot_floats = rows * (D + 2);
  constexpr int E = D / 32;  // dims of a lane
  float a[E], m, l;
  // pieces first, first + step, ... of row r into a (relative to maximum m) and l
  auto gather = [&](int r, int first, int step) {
    m = -INFINITY;
    l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) a[e] = 0.f;
    if (s.n == 0) return;
#pragma unroll 4
    for (int c = c0 + first; c <= c1; c += step) {
      // the piece is the CTA's first where the CTA starts inside it
      const float* sl = partial + ((size_t)2 * c + (cta_first(scan.total, n_cta, c) >= u0 ? 0 : 1)) * slot_floats;
      const float mi = sl[rows * D + r], li = sl[rows * D + rows + r];
      float v[E];
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const float2 t = *reinterpret_cast<const float2*>(sl + r * D + lane * E + e);
        v[e] = t.x;
        v[e + 1] = t.y;
      }
      const float mn = fmaxf(m, mi);
      const float f = m == -INFINITY ? 0.f : ex2(m - mn), w = mi == -INFINITY ? 0.f : ex2(mi - mn);
      l = (m == -INFINITY ? l : l * f) + (mi == -INFINITY ? li : li * w);  // (no key: 0, or a NaN that has to stay)
#pragma unroll
      for (int e = 0; e < E; ++e) a[e] = a[e] * f + v[e] * w;  // (a NaN stays, also of a piece without weight)
      m = mn;
    }
  };
  auto out = [&](int row, const Kv4Sums& z, int h) {
    __nv_bfloat16* o = p.o + (((size_t)b * p.S_q + row / G) * p.H_q + h) * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; e += 2)
      *reinterpret_cast<uint32_t*>(o + e) = pack_bf16x2(a[e] * z.mul, a[e + 1] * z.mul);
    if (lane == 0 && p.lse) p.lse[((size_t)b * p.H_q + h) * p.S_q + row / G] = z.lse;
  };
  __shared__ float red[2][8], sums[8][D];
  const int r = blockIdx.y;
  if (row0 + r >= R) return;
  gather(r, warp, 8);
  if (lane == 0) {
    red[0][warp] = m;
    red[1][warp] = l;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) sums[warp][lane * E + e] = a[e];
  __syncthreads();
  if (warp > 0) return;
  float mx = red[0][0], ll = 0.f;
  for (int w = 1; w < 8; ++w) mx = fmaxf(mx, red[0][w]);
#pragma unroll
  for (int e = 0; e < E; ++e) a[e] = 0.f;
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    const float f = red[0][w] == -INFINITY ? 0.f : ex2(red[0][w] - mx);
    ll += red[0][w] == -INFINITY ? red[1][w] : red[1][w] * f;
#pragma unroll
    for (int e = 0; e < E; ++e) a[e] = fmaf(sums[w][lane * E + e], f, a[e]);
  }
  const int h = hk * G + (row0 + r) % G;
  out(row0 + r, kv4_finish(p, h, mx, ll), h);
}

namespace {

// Column blocks of 8 query rows a CTA takes at a time.  Fewer leave room for more CTAs an SM (3, 2, 1),
// more decode each token less often.  329,377 tokens, 8 kv heads, d = 128, us with 1, 2 and 4 blocks:
// 8 rows 77, 105, 170; 16 rows 139, 106, 172; 24 rows 203, 201, 175; 32 rows 267, 201, 176; and 160
// rows of one kv head 167, 127, 112.  (Small caches prefer fewer at 32 rows: 42,031 tokens of one
// kv head in 16 sequences 17, 19, 21.)
int n_tiles(int rows) { return rows <= 8 ? 1 : rows <= 16 ? 2 : 4; }

template <int D, int NT>
int launch_t(const Kv4DecodeParams& p, float* partial, cudaStream_t stream) {
  using C = DecCfg<D, NT>;
  auto kern = kv4_decode_kernel<D, NT>;
  // the grid that fills the device, found (and the kernel's shared memory allowed) once a device
  static std::atomic<int> grids[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return -1;
  int grid = grids[dev].load(std::memory_order_acquire);
  if (grid == 0) {
    int per_sm = 0, sms = 0;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, kThreads, C::SMEM) != cudaSuccess)
      return -1;
    grid = std::max(1, std::min(kMaxCtas, per_sm * sms));
    grids[dev].store(grid, std::memory_order_release);
  }
  const int rows = p.H_q / p.c.H_kv * p.S_q, blocks = (rows + C::ROWS - 1) / C::ROWS;
  const long long join = (long long)p.B * p.c.H_kv * blocks;
  if (join > 0x7fffffffLL) return -2;
  if (launch_kernel(kern, dim3((unsigned)grid), kThreads, C::SMEM, stream, false, p, blocks, partial) != 0) return -1;
  return launch_kernel(kv4_join_kernel<D>, dim3((unsigned)join, std::min(rows, C::ROWS)), 256, 0, stream, true, p, blocks,
                       (int)C::ROWS, grid, (const float*)partial);
}

}  // namespace

size_t kv4_decode_workspace(int B, int S_q, int H_q, int H_kv, int d) {
  const long long rows = (long long)(H_q / H_kv) * S_q;
  const int nt = rows > 16 ? 4 : n_tiles((int)rows);
  return (size_t)kMaxCtas * 2 * 8 * nt * (d + 2) * sizeof(float);
}

int launch_kv4_decode(const Kv4DecodeParams& p, void* workspace, cudaStream_t stream) {
  float* partial = static_cast<float*>(workspace);
  const int nt = n_tiles(p.H_q / p.c.H_kv * p.S_q);
  if (p.c.d == 128)
    return nt == 1   ? launch_t<128, 1>(p, partial, stream)
           : nt == 2 ? launch_t<128, 2>(p, partial, stream)
                     : launch_t<128, 4>(p, partial, stream);
  return nt == 1   ? launch_t<64, 1>(p, partial, stream)
         : nt == 2 ? launch_t<64, 2>(p, partial, stream)
                   : launch_t<64, 4>(p, partial, stream);
}

}  // namespace sdpa
