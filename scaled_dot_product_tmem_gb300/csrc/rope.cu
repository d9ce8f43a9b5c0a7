// rope.cu -- cosines and sines of positions, and heads rotated by them (rope.cuh).
#include "attn_kernels.h"
#include "launch.h"
#include "ptx.cuh"
#include "rope.cuh"

namespace sdpa {

// table[t][0][f] = gain cos(p_t w_f), table[t][1][f] = gain sin(p_t w_f).
//
// An angle p w of a far position has lost its fraction of a turn long before 32 bits can hold it.
// So a frequency becomes f turns per position, w / 2 pi, as a 64-bit fraction of a turn (whole turns
// dropped), and p times that in 64-bit whole numbers, wrapping, is the angle's fraction of a turn.  The product
// is exact for every position; the frequency has two roundings (of 1 / 2 pi and of f, 2^-52 of it together) and is
// cut to a multiple of 2^-64, so an angle is off by at most |p| (2^-64 + 2^-52 f) turns.  A negative frequency
// is its magnitude negated: 1 less a small fraction would lose all but 2^-53 of a turn.  The
// frequencies are converted once a block: 64-bit floating point has 2 operations a cycle and SM.
// Sine and cosine of what is left after whole quarter turns are their power series: on |x| <= pi / 4 the
// first left-out terms are x^11 / 11! < 2^-29 and x^10 / 10! < 2^-25.  (The library's sine and cosine of half
// turns took 9 us instead of 7.8 for 16,000 rows of 64 pairs, cold.)
__global__ void __launch_bounds__(256) rope_table_kernel(const double* inv_freq, const int* positions, float* table, int T,
                                                         int n, float gain) {
  __shared__ unsigned long long turns[128];
  grid_launch_dependents();  // the rotation may be set up meanwhile
  if (threadIdx.x < n) {
    const double a = inv_freq[threadIdx.x] * 0.15915494309189533577, f = fabs(a);  // 1 / (2 pi)
    const unsigned long long u = __double2ull_rz((f - floor(f)) * 18446744073709551616.0);
    turns[threadIdx.x] = a < 0.0 ? 0ull - u : u;
  }
  __syncthreads();
  const int rows = 256 / n, f = threadIdx.x % n, r = threadIdx.x / n;
  if (r >= rows) return;
  const unsigned long long w = turns[f];
  for (long long t = (long long)blockIdx.x * rows + r; t < T; t += (long long)gridDim.x * rows) {
    const unsigned long long turn = (unsigned long long)(long long)__ldg(positions + t) * w;
    // the nearest quarter turn, and what is left, in [-2^61, 2^61) of 2^64, as two words
    const unsigned quarter = (unsigned)(turn >> 61) + 1u >> 1;
    const long long left = (long long)(turn - ((unsigned long long)quarter << 62));
    const float x = fmaf((float)(int)(left >> 32), 1.46291807926715970e-9f, (float)(unsigned)left * 3.40611980845280650e-19f);
    const float q = x * x;  // x in radians: the factors are 2 pi / 2^32 and 2 pi / 2^64
    const float sx = x + x * q * fmaf(q, fmaf(q, fmaf(q, 2.75573192e-6f, -1.98412698e-4f), 8.33333333e-3f), -1.66666667e-1f);
    const float cx = fmaf(q, fmaf(q, fmaf(q, fmaf(q, 2.48015873e-5f, -1.38888889e-3f), 4.16666667e-2f), -0.5f), 1.f);
    const float c = quarter & 1 ? sx : cx, s = quarter & 1 ? cx : sx;
    table[(size_t)t * 2 * n + f] = (quarter + 1) & 2 ? -gain * c : gain * c;
    table[(size_t)t * 2 * n + n + f] = quarter & 2 ? -gain * s : gain * s;
  }
}

// Measured: 32,511 rows of 40 heads of 128 (666 MB) about 103 us, 6.5 TB/s, 95 % of the measured copy rate; with a
// lookup of cosines and sines for every head 130, and with the dims that stay stored before the next head was loaded
// another third more where half of a head stays.
template <bool IL>
__global__ void __launch_bounds__(256) rope_kernel(const RopeParams p) {
  grid_wait();  // the table, or whatever was before
  rope_block<IL>(p, blockIdx.x);
}

int launch_rope_table(const double* inv_freq, const int* positions, float* table, int T, int n, float gain,
                      cudaStream_t stream) {
  const int rows = 256 / n;
  const int blocks = T / rows + (T % rows != 0);
  rope_table_kernel<<<blocks < 152 * 4 ? blocks : 152 * 4, 256, 0, stream>>>(inv_freq, positions, table, T, n, gain);
  return cudaPeekAtLastError() == cudaSuccess ? 0 : -1;
}

int launch_rope(const RopeParams& p, bool interleaved, cudaStream_t stream) {
  const long long blocks = rope_blocks(p);
  if (blocks > 0x7fffffffLL) return -2;
  return launch_kernel(interleaved ? rope_kernel<true> : rope_kernel<false>, dim3((unsigned)blocks), 256, 0, stream, true, p);
}

}  // namespace sdpa
