// Layer norm and RMS norm: arguments and launchers.
#pragma once

#include <type_traits>

#include "sk_tc.cuh"

namespace sk {

constexpr int64_t kNormMaxD = 32768;   // 1024 threads x 4 chunks of 8 columns

struct NormFwd {
  const void* x;         // [T][d], xtype
  const void* w;         // [d], wtype
  const void* b;         // [d], wtype, or nullptr
  void* y;               // [T][d], xtype
  float* mean;           // [T] or nullptr
  float* rstd;           // [T] or nullptr
  int8_t* q;             // [T][d] checkpoint of y, or nullptr
  uint8_t* qscale;       // [T][d / 32]
  int64_t T, d;
  float eps;
  int rms, xtype, wtype;
  unsigned int* check;
};

struct NormBwd {
  const void* dy;        // [T][d], xtype
  const void* x;         // [T][d], xtype
  const void* w;         // [d], wtype
  const float* mean;     // [T] (nullptr for RMS norm)
  const float* rstd;     // [T]
  void* dx;              // [T][d], xtype, or nullptr
  void* dw;              // [d], wtype, or nullptr
  void* db;              // [d], wtype, or nullptr
  float* part;           // [norm_bwd_parts][2][d]
  int64_t T, d;
  int rms, xtype, wtype;
  unsigned int* check;
};

int norm_bwd_parts(int64_t T, int64_t d);
cudaError_t launch_norm_fwd(const NormFwd& a, cudaStream_t s);
cudaError_t launch_norm_bwd(const NormBwd& a, cudaStream_t s);

}  // namespace sk
