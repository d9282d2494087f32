// The gate's gradient: from h = silu(g) u and dh, with s = 1 / (1 + exp(-g)),
//     dg = dh u s (1 + g (1 - s)),   du = dh g s,   and h = g s u again if asked.
//
// Bound by memory: 3 bf16 arrays read, 2 (3 with h) written, 10 (12) bytes per
// element.  Every thread takes vectors of 8 elements (16 bytes), two in flight
// per array; the arithmetic is fp32 and each output is rounded once.  An output
// may be one of the inputs: an element's inputs are read before its outputs are
// written, by the same thread.  11008 x 2048 with h, calls in a stream:
// 42.2 us = 6.4 TB/s (44.8 without the early launch).
#include "mbok_common.cuh"

namespace mbok {

constexpr int kGateThreads = 256;
constexpr int kGateVecs = 2;   // vectors per thread and array in flight

__device__ __forceinline__ void gate_grad(float dh, float g, float u, float& dg, float& du, float& h) {
  // for g below about -88 exp(-g) is infinite and s is the 0 it tends to
  const float s = __fdividef(1.f, 1.f + __expf(-g));
  const float gs = g * s;
  du = dh * gs;
  h = gs * u;
  dg = dh * u * fmaf(gs, 1.f - s, s);
}

template <bool REMAKE>
__device__ __forceinline__ void gate_grad8(const uint4& dh, const uint4& g, const uint4& u, uint4& dg, uint4& du,
                                           uint4& h) {
  const uint32_t a[4] = {dh.x, dh.y, dh.z, dh.w}, b[4] = {g.x, g.y, g.z, g.w}, c[4] = {u.x, u.y, u.z, u.w};
  uint32_t x[4], y[4], z[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float dg0, du0, h0, dg1, du1, h1;
    gate_grad(__uint_as_float(a[i] << 16), __uint_as_float(b[i] << 16), __uint_as_float(c[i] << 16), dg0, du0, h0);
    gate_grad(__uint_as_float(a[i] & 0xFFFF0000u), __uint_as_float(b[i] & 0xFFFF0000u),
              __uint_as_float(c[i] & 0xFFFF0000u), dg1, du1, h1);
    const __nv_bfloat162 p = __floats2bfloat162_rn(dg0, dg1), q = __floats2bfloat162_rn(du0, du1);
    x[i] = *reinterpret_cast<const uint32_t*>(&p);
    y[i] = *reinterpret_cast<const uint32_t*>(&q);
    if (REMAKE) {
      const __nv_bfloat162 r = __floats2bfloat162_rn(h0, h1);
      z[i] = *reinterpret_cast<const uint32_t*>(&r);
    }
  }
  dg = make_uint4(x[0], x[1], x[2], x[3]);
  du = make_uint4(y[0], y[1], y[2], y[3]);
  if (REMAKE) h = make_uint4(z[0], z[1], z[2], z[3]);
}

template <bool REMAKE>
__global__ void __launch_bounds__(kGateThreads) gated_backward_kernel(const uint16_t* dh, const uint16_t* gate,
                                                                      const uint16_t* up, uint16_t* dgate,
                                                                      uint16_t* dup, uint16_t* h, size_t n) {
  const size_t nvec = n / 8;
  const size_t v0 = size_t(blockIdx.x) * (kGateThreads * kGateVecs) + threadIdx.x;
  uint4 a[kGateVecs], b[kGateVecs], c[kGateVecs];
  pdl_launch();
  pdl_wait();   // nothing is read or written before the preceding grid is complete
#pragma unroll
  for (int i = 0; i < kGateVecs; ++i) {
    const size_t v = v0 + size_t(i) * kGateThreads;
    if (v < nvec) {
      a[i] = __ldcs(reinterpret_cast<const uint4*>(dh) + v);
      b[i] = __ldcs(reinterpret_cast<const uint4*>(gate) + v);
      c[i] = __ldcs(reinterpret_cast<const uint4*>(up) + v);
    }
  }
#pragma unroll
  for (int i = 0; i < kGateVecs; ++i) {
    const size_t v = v0 + size_t(i) * kGateThreads;
    if (v < nvec) {
      uint4 x, y, z;
      gate_grad8<REMAKE>(a[i], b[i], c[i], x, y, z);
      reinterpret_cast<uint4*>(dgate)[v] = x;
      reinterpret_cast<uint4*>(dup)[v] = y;
      if (REMAKE) reinterpret_cast<uint4*>(h)[v] = z;
    }
  }
  // the last n % 8 elements
  if (blockIdx.x == gridDim.x - 1 && threadIdx.x < n % 8) {
    const size_t e = nvec * 8 + threadIdx.x;
    float x, y, z;
    gate_grad(bf16_bits_to_float(dh[e]), bf16_bits_to_float(gate[e]), bf16_bits_to_float(up[e]), x, y, z);
    dgate[e] = __bfloat16_as_ushort(__float2bfloat16_rn(x));
    dup[e] = __bfloat16_as_ushort(__float2bfloat16_rn(y));
    if (REMAKE) h[e] = __bfloat16_as_ushort(__float2bfloat16_rn(z));
  }
}

cudaError_t launch_gated_backward(const uint16_t* dh, const uint16_t* gate, const uint16_t* up, size_t n,
                                  uint16_t* dgate, uint16_t* dup, uint16_t* h, cudaStream_t stream) {
  const size_t per = size_t(kGateThreads) * kGateVecs * 8;
  const unsigned grid = unsigned((n + per - 1) / per);
  return launch_dependent(h != nullptr ? gated_backward_kernel<true> : gated_backward_kernel<false>, dim3(grid),
                          dim3(kGateThreads), 0, stream, dh, gate, up, dgate, dup, h, n);
}

}  // namespace mbok
