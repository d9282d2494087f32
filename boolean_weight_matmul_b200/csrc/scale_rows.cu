// Activations for the fp16 tensor-core products: each token's bf16 values
// times a power of two that puts its largest finite magnitude in [2^14, 2^15).
//
// fp16 holds 11 bits where bf16 holds 8, so the scaled values are exact down
// to 2^-29 of the token's largest and off by at most 2^-39 of it below that (half
// a step of fp16's subnormals, 2^-25, where the largest is 2^14), far under the fp32 accumulation; and weight levels, which need more than
// bf16's 8 bits, keep 11 in the same tensor-core instruction.  (An instruction
// takes two operands of one type; bf16 levels would add an error as large as
// the output's own rounding, and two bf16 terms per level twice the work.)
// A memory-bound pass of 4 bytes per element, small beside the product.
#include "scale_rows.h"

namespace mbok {

constexpr int kScaleThreads = 256;

// Eight values of a row as bf16 bits; zeros beyond the row.  Rows whose length
// is no multiple of 8 are read in 4-byte words: a row that starts on an odd
// element by five words, shifted by one value (the first word begins in the row
// before; the row's last value, which may be the tensor's, is read alone).  1700
// tokens of two dY, 287 and 9553 rows: 28 us by single values, 22 by words.
__device__ __forceinline__ uint4 row_vec(const uint16_t* row, int cols, int v, bool vectors) {
  if (vectors) return *(reinterpret_cast<const uint4*>(row) + v);
  const int odd = int(reinterpret_cast<uintptr_t>(row) >> 1) & 1;
  uint32_t w[5];
#pragma unroll
  for (int i = 0; i < 5; ++i) {
    const int c = 8 * v + 2 * i - odd;   // the word's first value
    w[i] = 0u;
    if (i < 4 || odd) {
      if (c + 1 < cols) w[i] = *reinterpret_cast<const uint32_t*>(row + c);
      else if (c < cols) w[i] = row[c];
    }
  }
  if (odd)
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The larger of m and the finite magnitudes (bf16 bits) in a pair.
__device__ __forceinline__ uint32_t max_finite(uint32_t m, uint32_t pair) {
  const uint32_t lo = pair & 0x7FFFu, hi = (pair >> 16) & 0x7FFFu;
  if (lo < 0x7F80u) m = max(m, lo);
  if (hi < 0x7F80u) m = max(m, hi);
  return m;
}

__device__ __forceinline__ uint32_t scaled_pair(uint32_t pair, float f) {
  const __half2 h = __floats2half2_rn(__uint_as_float(pair << 16) * f, __uint_as_float(pair & 0xFFFF0000u) * f);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__global__ void __launch_bounds__(kScaleThreads) scale_rows_kernel(const __grid_constant__ ScaleRows p) {
  __shared__ uint32_t warp_max[kScaleThreads / 32];
  const size_t t = blockIdx.x;
  pdl_wait();   // the sources, and the workspace of an earlier call
  pdl_launch();   // after the wait: the product that follows reads weights beside this grid
  uint32_t m = 0;
  for (int s = 0; s < p.nseg; ++s) {
    const ScaleSeg& g = p.seg[s];
    const uint16_t* row = g.src + t * g.cols;
    const bool vectors = g.cols % 8 == 0;
    for (int v = threadIdx.x; v < g.ld / 8; v += kScaleThreads) {
      const uint4 x = row_vec(row, g.cols, v, vectors);
      m = max_finite(max_finite(max_finite(max_finite(m, x.x), x.y), x.z), x.w);
    }
  }
  m = __reduce_max_sync(0xffffffffu, m);
  if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kScaleThreads / 32; ++i) m = max(m, warp_max[i]);
  // biased exponent E of the maximum (0 for zeros and subnormals): scale by
  // 2^(141 - E), at most 2^126 (both it and its reciprocal stay normal)
  const int e = m == 0 ? 0 : min(141 - int(m >> 7), 126);
  const float f = __uint_as_float(uint32_t(127 + e) << 23);
  if (threadIdx.x == 0) p.inverse[t] = __uint_as_float(uint32_t(127 - e) << 23) * p.factor;
  for (int s = 0; s < p.nseg; ++s) {
    const ScaleSeg& g = p.seg[s];
    const uint16_t* row = g.src + t * g.cols;
    const bool vectors = g.cols % 8 == 0;
    for (int v = threadIdx.x; v < g.ld / 8; v += kScaleThreads) {
      const uint4 x = row_vec(row, g.cols, v, vectors);
      const uint4 y = make_uint4(scaled_pair(x.x, f), scaled_pair(x.y, f), scaled_pair(x.z, f), scaled_pair(x.w, f));
      if (g.dst != nullptr) *(reinterpret_cast<uint4*>(g.dst + t * g.ld) + v) = y;
      if (g.copy != nullptr) *(reinterpret_cast<uint4*>(g.copy + t * g.ld) + v) = x;
    }
  }
}

cudaError_t launch_scale_rows(const ScaleRows& p, int T, cudaStream_t stream) {
  return launch_dependent(scale_rows_kernel, dim3(unsigned(T)), dim3(kScaleThreads), 0, stream, p);
}

}  // namespace mbok
