// Linear cross entropy: arguments and launcher.
#pragma once

#include "sk_tc.cuh"

namespace sk {

struct CrossEntropy {
  const uint16_t* H;        // bf16 [T][d]
  const uint16_t* W;        // bf16 [V][d]
  const void* target;       // int32 or int64 [T]
  int target64;
  int64_t T, V, d, ignore_index;
  int reduction;            // SK_CE_NONE, SK_CE_MEAN, SK_CE_SUM
  const float* dloss;       // [T] (NONE) or [1], or nullptr (ones)
  float* loss;              // [T] or [1], or nullptr
  uint16_t* dH;             // bf16 [T][d] or nullptr
  uint16_t* dW;             // bf16 [V][d] or nullptr
  void* workspace;
  unsigned int* check;
};

size_t cross_entropy_workspace(int64_t T, int64_t V, int64_t d, bool dh, bool dw);
cudaError_t launch_cross_entropy(const CrossEntropy& a, cudaStream_t s);
cudaError_t launch_scale_bf16(uint16_t* x, int64_t nx, uint16_t* y, int64_t ny, const float* factor, cudaStream_t s);

}  // namespace sk
