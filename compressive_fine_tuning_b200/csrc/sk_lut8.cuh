// LUT gradient from an 8-bit activation checkpoint: launchers.
#pragma once

#include "sk_ckpt8.cuh"

namespace sk {

// tensor-core path: X as bf16, partial bins and, with task ids (`routed`), their routing
size_t lut8_tc_workspace(int64_t n, int64_t d, int bits, int gpr, int64_t T, int ntask, bool routed);
cudaError_t launch_lut8_tc(const Problem& p, const int8_t* q, const uint8_t* scale, const uint16_t* dY, float* dlut,
                           int accumulate, bool routed, void* workspace, cudaStream_t s);
// CUDA-core path (few tokens, no workspace)
cudaError_t launch_lut8_simt(const Problem& p, const int8_t* q, const uint8_t* scale, const uint16_t* dY, float* dlut,
                             int accumulate, cudaStream_t s);

}  // namespace sk
