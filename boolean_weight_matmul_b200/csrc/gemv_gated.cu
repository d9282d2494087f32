// Gated decode  h[b] = silu(W_gate x[b]) * (W_up x[b])  for 1..16 vectors:
// the tensor-core form (two vectors or more, kernel in gemv_mma.cuh) and the
// choice between it and the lookup form (one vector, gemv_lut.cu).
//
// A gated feed-forward block reads x once for two projections and uses them
// only as this product, so neither is stored: each form gates the two sums of
// a row where it would otherwise store them.
#include "gemv_mma.cuh"

namespace mbok {

cudaError_t launch_gemv_lut_gated(const uint8_t*, const uint16_t*, const Shape&, const uint8_t*, const uint16_t*,
                                  const Shape&, const void*, bool, void*, bool, void*, cudaStream_t, bool);

template <int K, int NT, bool XF32, int MINB, bool DEEP>
static cudaError_t launch_gated_k(const GemvMmaParams& p, cudaStream_t stream) {
  auto fn = gemv_mma_kernel<K, NT, XF32, MINB, DEEP, true>;
  using G = MmaGeom<K, NT, XF32, DEEP>;
  static PerDeviceOnce attr_once;   // the attribute is per device context
  const cudaError_t ae = set_smem_attr_once(attr_once, reinterpret_cast<const void*>(fn), G::kSmem);
  if (ae != cudaSuccess) return ae;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.s.O);
  cfg.blockDim = dim3(kMmaThreads);
  cfg.dynamicSmemBytes = G::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, fn, p);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

// The variant rules are those of the plain form (gemv_mma.cu), measured there.
template <int K, bool DEEP>
static cudaError_t launch_gated_nt_d(const GemvMmaParams& p, bool x_f32, cudaStream_t stream) {
  const int cols = x_f32 ? 3 * p.nb : p.nb;
  if (cols <= 8) {
    if (p.s.O >= 3 * device_sm_count())
      return x_f32 ? launch_gated_k<K, 1, true, 3, DEEP>(p, stream) : launch_gated_k<K, 1, false, 3, DEEP>(p, stream);
    return x_f32 ? launch_gated_k<K, 1, true, 2, DEEP>(p, stream) : launch_gated_k<K, 1, false, 2, DEEP>(p, stream);
  }
  constexpr int kMinB2 = K >= 3 ? 1 : 2;
  return x_f32 ? launch_gated_k<K, 2, true, kMinB2, DEEP>(p, stream)
               : launch_gated_k<K, 2, false, kMinB2, DEEP>(p, stream);
}

template <int K>
static cudaError_t launch_gated_nt(const GemvMmaParams& p, bool x_f32, cudaStream_t stream) {
  const int slices = (p.s.N + MmaGeom<K, 1, false>::kCols - 1) / MmaGeom<K, 1, false>::kCols;
  return slices >= kMmaDeepMinSlices ? launch_gated_nt_d<K, true>(p, x_f32, stream)
                                     : launch_gated_nt_d<K, false>(p, x_f32, stream);
}

// h[b] for b < batch (x: [batch][N], h: [batch][M]).
cudaError_t launch_gemv_gated(const uint8_t* packed_gate, const uint16_t* alpha_gate, const Shape& gate,
                              const uint8_t* packed_up, const uint16_t* alpha_up, const Shape& up, const void* x,
                              bool x_f32, int batch, void* h, bool h_bf16, void* workspace, cudaStream_t stream,
                              bool weights_static) {
  if (batch == 1)
    return launch_gemv_lut_gated(packed_gate, alpha_gate, gate, packed_up, alpha_up, up, x, x_f32, h, h_bf16,
                                 workspace, stream, weights_static);
  const int per_launch = x_f32 ? (8 * kMaxNT) / 3 : 8 * kMaxNT;
  const size_t x_elem = x_f32 ? 4 : 2, h_elem = h_bf16 ? 2 : 4;
  for (int b0 = 0; b0 < batch; b0 += per_launch) {
    GemvMmaParams p = {};
    p.packed = packed_gate;
    p.alpha = alpha_gate;
    p.s = gate;
    p.packed_up = packed_up;
    p.alpha_up = alpha_up;
    p.s_up = up;
    p.x = static_cast<const char*>(x) + size_t(b0) * gate.N * x_elem;
    p.h = static_cast<char*>(h) + size_t(b0) * gate.M * h_elem;
    p.h_bf16 = h_bf16 ? 1 : 0;
    p.nb = batch - b0 < per_launch ? batch - b0 : per_launch;
    p.weights_static = weights_static ? 1 : 0;
    for (int i = 0; i < 8; ++i) p.mul[i] = 1u << (15 - 2 * i);
    cudaError_t e;
    switch (gate.K > up.K ? gate.K : up.K) {
      case 1: e = launch_gated_nt<1>(p, x_f32, stream); break;
      case 2: e = launch_gated_nt<2>(p, x_f32, stream); break;
      case 3: e = launch_gated_nt<3>(p, x_f32, stream); break;
      default: e = launch_gated_nt<4>(p, x_f32, stream); break;
    }
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

// Reads and clears the gated kernels' error flag; ~0u if the read itself failed.
unsigned gemv_gated_error_flags() {
  unsigned v = 0;
  if (cudaMemcpyFromSymbol(&v, g_gemv_mma_error, sizeof(v)) != cudaSuccess) return ~0u;
  const unsigned z = 0;
  if (v != 0 && cudaMemcpyToSymbol(g_gemv_mma_error, &z, sizeof(z)) != cudaSuccess) return ~0u;
  return v;
}

}  // namespace mbok
