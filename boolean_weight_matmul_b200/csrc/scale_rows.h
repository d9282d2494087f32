// Scaling of activations to fp16 for the tensor-core products (scale_rows.cu).
#pragma once

#include "mbok_common.cuh"

namespace mbok {

constexpr int kMaxMats = 8;   // matrices per call, as mbok_gemv_multi

struct ScaleSeg {
  const uint16_t* src;   // bf16 [T][cols]
  uint16_t* dst;         // fp16 [T][ld] or nullptr, zeros beyond cols
  uint16_t* copy;        // bf16 [T][ld] or nullptr: the source with aligned rows, zeros beyond cols
  int cols, ld;          // ld: cols rounded up to a multiple of 8
};

struct ScaleRows {
  ScaleSeg seg[kMaxMats];   // one scale per token over all of them
  int nseg;
  float* inverse;           // [T]: factor / scale
  float factor;
};

cudaError_t launch_scale_rows(const ScaleRows& p, int T, cudaStream_t stream);

}  // namespace mbok
