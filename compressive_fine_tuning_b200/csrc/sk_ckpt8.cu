// 8-bit activation checkpoints: quantise bf16 rows and read them back (the
// format is in sk_ckpt8.cuh).  Elementwise and bound by memory: 2 + 33/32 bytes
// per value either way.  A thread owns eight values (one 16-byte word of bf16,
// eight bytes of q), so four neighbouring lanes hold one block and two shuffles
// find its largest value.
#include "sk_ckpt8.cuh"

namespace sk {
namespace {

constexpr int kThreads = 256;
constexpr int kUnits = 4;      // 16-byte loads in flight per thread

__global__ void __launch_bounds__(kThreads) ckpt8_quantize_kernel(const uint4* __restrict__ X, int64_t units,
                                                                  uint2* __restrict__ q, uint8_t* __restrict__ scale) {
  // whole warps run through the shuffles: units beyond the end are zeros
  const int64_t first = (int64_t)blockIdx.x * (kThreads * kUnits) + threadIdx.x;
  uint4 v[kUnits];
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int64_t u = first + i * kThreads;
    v[i] = u < units ? X[u] : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int64_t u = first + i * kThreads;
    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
    uint32_t byte;
    const uint2 o = ckpt8_quantize8(w, byte);
    if (u < units) {
      q[u] = o;
      if ((u & 3) == 0) scale[u >> 2] = (uint8_t)byte;
    }
  }
}

__global__ void __launch_bounds__(kThreads) ckpt8_dequantize_kernel(const uint2* __restrict__ q,
                                                                    const uint8_t* __restrict__ scale, int64_t units,
                                                                    uint4* __restrict__ X) {
  const int64_t first = (int64_t)blockIdx.x * (kThreads * kUnits) + threadIdx.x;
  uint2 v[kUnits];
  uint32_t byte[kUnits];
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int64_t u = first + i * kThreads;
    if (u < units) {
      v[i] = q[u];
      byte[i] = scale[u >> 2];
    }
  }
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int64_t u = first + i * kThreads;
    if (u >= units) break;
    uint4 o;
    const uint32_t s2 = ckpt8_scale2(byte[i]);
    ckpt8_dequant4(v[i].x, s2, o.x, o.y);
    ckpt8_dequant4(v[i].y, s2, o.z, o.w);
    X[u] = o;
  }
}

// T * d < 2^62 / 8 units, 1024 per block: the grid's x extent reaches 2^31 blocks
unsigned grid_for(int64_t units) { return (unsigned)((units + kThreads * kUnits - 1) / (kThreads * kUnits)); }

}  // namespace

cudaError_t launch_ckpt8_quantize(const uint16_t* X, int64_t T, int64_t d, int8_t* q, uint8_t* scale, cudaStream_t s) {
  const int64_t units = T * d / 8;
  ckpt8_quantize_kernel<<<grid_for(units), kThreads, 0, s>>>(reinterpret_cast<const uint4*>(X), units,
                                                             reinterpret_cast<uint2*>(q), scale);
  return cudaGetLastError();
}

cudaError_t launch_ckpt8_dequantize(const int8_t* q, const uint8_t* scale, int64_t T, int64_t d, uint16_t* X,
                                    cudaStream_t s) {
  const int64_t units = T * d / 8;
  ckpt8_dequantize_kernel<<<grid_for(units), kThreads, 0, s>>>(reinterpret_cast<const uint2*>(q), scale, units,
                                                               reinterpret_cast<uint4*>(X));
  return cudaGetLastError();
}

}  // namespace sk
