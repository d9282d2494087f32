// Backward pass of Boolean linear layers that share X: the input gradient
// (gemm_pair.cu, on dY scaled to fp16) and the scales' gradients
// (gemm_dalpha.cu, on dY as it is), and their shared workspace.
#include "scale_rows.h"

namespace mbok {

cudaError_t launch_gemm_grad_x(int, const uint8_t* const*, const uint16_t* const*, const Shape*,
                               const uint16_t* const*, const int*, const float*, int, uint16_t*, void*, cudaStream_t);
size_t gemm_grad_x_workspace_bytes(int, const Shape*, int);
cudaError_t launch_gemm_dalpha(int, const uint8_t* const*, const Shape*, const uint16_t*, int, const uint16_t* const*,
                               const int*, float* const*, int, bool, void*, cudaStream_t);
int dalpha_splits(int, const Shape*, int);
size_t dalpha_workspace_bytes(int, const Shape*, int);

namespace {

// Offsets into the workspace; each region 256-byte aligned.
struct Plan {
  int ld[kMaxMats];              // row length of the scaled and copied dY
  size_t scaled[kMaxMats];       // fp16 [T][ld]
  size_t copy[kMaxMats];         // bf16 [T][ld] where M is not a multiple of 8 (TMA rows are 16-byte aligned)
  size_t inverse;                // fp32 [T rounded up to 16]
  size_t splits, splits_x;       // the scale gradients' and dX's partial sums
  size_t total;
};

Plan make_plan(int nmat, const Shape* shapes, int T) {
  Plan pl = {};
  size_t at = 0;
  auto take = [&at](size_t bytes) {
    const size_t o = at;
    at += (bytes + 255) / 256 * 256;
    return o;
  };
  for (int i = 0; i < nmat; ++i) {
    pl.ld[i] = (shapes[i].M + 7) / 8 * 8;
    pl.scaled[i] = take(size_t(T) * pl.ld[i] * 2);
    if (shapes[i].M % 8 != 0) pl.copy[i] = take(size_t(T) * pl.ld[i] * 2);
  }
  pl.inverse = take((size_t(T) + 15) / 16 * 16 * sizeof(float));
  pl.splits = take(dalpha_workspace_bytes(nmat, shapes, T));
  pl.splits_x = take(gemm_grad_x_workspace_bytes(nmat, shapes, T));
  pl.total = at;
  return pl;
}

}  // namespace

size_t gemm_backward_workspace_bytes(int nmat, const Shape* shapes, int T) { return make_plan(nmat, shapes, T).total; }

// dX may be nullptr, and dalpha or any of its entries.
cudaError_t launch_gemm_backward(int nmat, const uint8_t* const* packed, const uint16_t* const* alpha,
                                 const Shape* shapes, const uint16_t* X, int T, const uint16_t* const* dY,
                                 uint16_t* dX, float* const* dalpha, void* workspace, cudaStream_t stream) {
  const Plan pl = make_plan(nmat, shapes, T);
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  float* inverse = reinterpret_cast<float*>(ws + pl.inverse);
  const uint16_t* scaled[kMaxMats];
  const uint8_t* d_packed[kMaxMats];
  Shape d_shapes[kMaxMats];
  const uint16_t* d_dy[kMaxMats];
  int d_ld[kMaxMats];
  float* d_out[kMaxMats];
  int nd = 0;
  bool pass = dX != nullptr;
  ScaleRows sc = {};
  sc.nseg = nmat;
  sc.inverse = inverse;
  sc.factor = 4.f;   // the levels are quarters (tc_unpack.cuh)
  for (int i = 0; i < nmat; ++i) {
    const bool wanted = dalpha != nullptr && dalpha[i] != nullptr;
    const bool ragged = shapes[i].M % 8 != 0;
    ScaleSeg& g = sc.seg[i];
    g.src = dY[i];
    g.cols = shapes[i].M;
    g.ld = pl.ld[i];
    g.dst = dX != nullptr ? reinterpret_cast<uint16_t*>(ws + pl.scaled[i]) : nullptr;
    g.copy = wanted && ragged ? reinterpret_cast<uint16_t*>(ws + pl.copy[i]) : nullptr;
    scaled[i] = g.dst;
    if (wanted) {
      d_packed[nd] = packed[i];
      d_shapes[nd] = shapes[i];
      d_dy[nd] = ragged ? g.copy : dY[i];
      d_ld[nd] = pl.ld[i];
      d_out[nd] = dalpha[i];
      ++nd;
      pass = pass || ragged;
    }
  }
  cudaError_t e = pass ? launch_scale_rows(sc, T, stream) : cudaSuccess;
  if (e == cudaSuccess && dX != nullptr)
    e = launch_gemm_grad_x(nmat, packed, alpha, shapes, scaled, pl.ld, inverse, T, dX, ws + pl.splits_x, stream);
  if (e == cudaSuccess && nd > 0)
    e = launch_gemm_dalpha(nd, d_packed, d_shapes, X, T, d_dy, d_ld, d_out, dalpha_splits(nmat, shapes, T),
                           dX != nullptr, ws + pl.splits, stream);
  return e;
}

}  // namespace mbok
