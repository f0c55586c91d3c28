// 8-bit activation checkpoints: quantise bf16 rows and read them back (the
// format is in sk_ckpt8.cuh).  Elementwise and bound by memory: 2 + 33/32 bytes
// per value either way.  A thread owns eight values (one 16-byte word of bf16,
// eight bytes of q), so four neighbouring lanes hold one block and two shuffles
// find its largest value.
#include "sk_ckpt8.cuh"

namespace sk {
namespace {

constexpr int kThreads = 256;

__global__ void __launch_bounds__(kThreads) ckpt8_quantize_kernel(const uint4* __restrict__ X, int64_t units,
                                                                  uint2* __restrict__ q, uint8_t* __restrict__ scale) {
  const int64_t step = (int64_t)gridDim.x * kThreads;
  // whole warps stay in the loop together: the shuffles name every lane
  for (int64_t u = (int64_t)blockIdx.x * kThreads + threadIdx.x; u - (threadIdx.x & 31) < units; u += step) {
    const uint4 v = u < units ? X[u] : make_uint4(0u, 0u, 0u, 0u);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
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
  const int64_t step = (int64_t)gridDim.x * kThreads;
  for (int64_t u = (int64_t)blockIdx.x * kThreads + threadIdx.x; u < units; u += step) {
    const uint2 v = q[u];
    const float s = __uint_as_float((uint32_t)scale[u >> 2] << 23);
    uint4 o;
    ckpt8_dequant4(v.x, s, o.x, o.y);
    ckpt8_dequant4(v.y, s, o.z, o.w);
    X[u] = o;
  }
}

unsigned grid_for(int64_t units) {
  const int64_t blocks = (units + kThreads - 1) / kThreads;
  const int64_t cap = (int64_t)1 << 30;
  return (unsigned)(blocks < cap ? blocks : cap);
}

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
