// Linear cross entropy: the head product, softmax cross entropy over the
// vocabulary and its gradients, without a [T][V] tensor of logits.
//
//   l = H W^T,  lse_t = log sum_v exp(l_tv),  loss_t = lse_t - l_t,target
//   P = c_t (softmax(l_t) - onehot(target)),  dH = P W,  dW = P^T H
//
// The loss alone is one product whose epilogue reduces every 256-column tile of
// a row to its largest logit and its sum of exponentials; a second kernel joins
// a row's tiles.  Nothing else is written.
//
// With gradients the epilogue also writes exp(l - tile maximum) in 16 bits, for
// a chunk of tokens whose rows fit in kExpBytes; once the row's lse is known a
// pass over that buffer turns it into P in place (bf16, the tensor cores'
// operand), and two more products give dH and dW.  Computing the logits twice
// instead would cost another 2 T V d flops, the buffer's write, read, write cost
// 6 T V bytes: at d = 4096 the second is a tenth of the first.
// Chunks are as large as the buffer allows, so dW needs an fp32 accumulator in
// memory only beyond one chunk.
//
// Precision: logits, maxima, sums and lse in fp32.  exp(l - max) lies in [0, 1]
// and is held in fp16 (2^-11 of the value; below 2^-24 of the tile's maximum it
// is lost, where P itself is below 2^-24 of the row's largest).  P is rounded to
// bf16 for the products (2^-9 of each value).  The target's entry does not come
// from the buffer: p - 1 is formed from the fp32 loss as expm1(-loss), so a
// token that is already predicted surely keeps its small gradient's precision.
//
// The bound is the tensor pipe: 2 T V d flops per product.
#include <type_traits>

#include "sk_gemm.cuh"
#include "sk_loss.cuh"

namespace sk {
namespace {

constexpr int64_t kExpBytes = int64_t(512) << 20;   // buffer of one chunk's exponentials
constexpr int64_t kLossChunk = 32768;               // tokens per launch when only the loss is wanted
constexpr float kLog2e = 1.4426950408889634f;

__host__ __device__ constexpr int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b * b; }

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The token's class, or -1 when it takes no part (ignored, or out of range,
// which is flagged).
__device__ __forceinline__ int64_t class_of(const void* target, int target64, int64_t t, int64_t V, int64_t ignore,
                                            unsigned int* check) {
  const int64_t y = target64 ? __ldg(static_cast<const long long*>(target) + t)
                             : (int64_t)__ldg(static_cast<const int*>(target) + t);
  if (y == ignore) return -1;
  if (y < 0 || y >= V) {
    atomicOr(check, SK_CHECK_TARGET_RANGE);
    return -1;
  }
  return y;
}

// ----------------------------------------------------------------------------
// logits: tile statistics, the target's logit, and the exponentials
// ----------------------------------------------------------------------------

struct LogitEpi {
  const CUtensorMap* tm_e;
  float2* stats;            // [tiles of V][T]: (maximum, sum of exp(l - maximum))
  float* target_logit;      // [T]
  const void* target;
  int target64;
  int64_t ignore_index;
  int T, V;                 // tokens of the chunk
  bool store;
  unsigned int* check;

  __device__ __forceinline__ void tile(uint32_t tmem, int m0, int n0, int warp, int lane, gemm::SlabWriter& out) {
    const int t = m0 + 32 * warp + lane;
    const int cols = min(gemm::TN, V - n0);
    int64_t y = -1;
    if (t < T) y = class_of(target, target64, t, V, ignore_index, check);
    const int rel = y >= n0 && y < n0 + cols ? (int)(y - n0) : -1;
    // the row's largest logit of the tile
    float m = -INFINITY;
#pragma unroll 1
    for (int q = 0; q < gemm::TN / 32; ++q) {
      if (32 * q >= cols) break;
      uint32_t v[32];
      tc::tmem_ld32(tmem + 32 * q, v);
      tc::tmem_ld_wait();
      if (32 * q + 32 <= cols) {
#pragma unroll
        for (int j = 0; j < 32; ++j) m = fmaxf(m, __uint_as_float(v[j]));
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (32 * q + j < cols) m = fmaxf(m, __uint_as_float(v[j]));
      }
    }
    // a tile of nothing but -inf: subtract zero, every exponential is zero then
    const float base = m == -INFINITY ? 0.f : m;
    float sum = 0.f;
#pragma unroll 1
    for (int h = 0; h < gemm::TN / 64; ++h) {
      if (64 * h >= cols) break;
      uint32_t e[32];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int c0 = 64 * h + 32 * q;
        uint32_t v[32];
        tc::tmem_ld32(tmem + c0, v);
        tc::tmem_ld_wait();
        if (__any_sync(0xffffffffu, rel >= c0 && rel < c0 + 32)) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (rel == c0 + j) target_logit[t] = __uint_as_float(v[j]);
        }
        float part = 0.f;
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
          float a = fast_exp2((__uint_as_float(v[j]) - base) * kLog2e);
          float b = fast_exp2((__uint_as_float(v[j + 1]) - base) * kLog2e);
          if (c0 + j >= cols) a = 0.f;
          if (c0 + j + 1 >= cols) b = 0.f;
          part += a;
          part += b;
          const __half2 hh = __floats2half2_rn(a, b);
          e[16 * q + (j >> 1)] = *reinterpret_cast<const uint32_t*>(&hh);
        }
        sum += part;
      }
      if (store && m0 + 32 * warp < T) out.put(tm_e, e, n0 + 64 * h, m0 + 32 * warp, lane);
    }
    if (t < T) stats[(int64_t)(n0 / gemm::TN) * T + t] = make_float2(m, sum);
  }
};

struct LogitArgs {
  gemm::Shape shape;
  float2* stats;
  float* target_logit;
  const void* target;
  int target64;
  int64_t ignore_index;
  int T, V, store;
  unsigned int* check;
};

__global__ void __launch_bounds__(gemm::THREADS, 1)
logit_kernel(const __grid_constant__ CUtensorMap tm_h, const __grid_constant__ CUtensorMap tm_w,
             const __grid_constant__ CUtensorMap tm_e, LogitArgs a) {
  LogitEpi epi{&tm_e, a.stats, a.target_logit, a.target, a.target64, a.ignore_index, a.T, a.V, a.store != 0, a.check};
  gemm::run<0, 0>(&tm_h, &tm_w, a.shape, epi, a.check);
}

// ----------------------------------------------------------------------------
// dH and dW
// ----------------------------------------------------------------------------

// bf16 output through the slab writer; or, for a dW that several chunks add up
// to, fp32 sums in memory (`acc`): read when `add`, written back as fp32 unless
// this is the last chunk, which writes bf16.
struct GradEpi {
  const CUtensorMap* tm_out;
  float* acc;
  int add, last;
  int64_t M, N;

  __device__ __forceinline__ void tile(uint32_t tmem, int m0, int n0, int warp, int lane, gemm::SlabWriter& out) {
    const int64_t row = m0 + 32 * warp + lane;
#pragma unroll 1
    for (int h = 0; h < gemm::TN / 64; ++h) {
      const int c0 = n0 + 64 * h;
      if (c0 >= N) break;
      uint32_t o[32];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t v[32];
        tc::tmem_ld32(tmem + 64 * h + 32 * q, v);
        tc::tmem_ld_wait();
        if (acc != nullptr && row < M) {
          // d % 8 == 0: groups of eight columns are inside or outside as a whole
          float4* p = reinterpret_cast<float4*>(acc + row * N + c0 + 32 * q);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (c0 + 32 * q + 4 * j >= N) break;
            float4 f = make_float4(__uint_as_float(v[4 * j]), __uint_as_float(v[4 * j + 1]),
                                   __uint_as_float(v[4 * j + 2]), __uint_as_float(v[4 * j + 3]));
            if (add) {
              const float4 g = p[j];
              f = make_float4(f.x + g.x, f.y + g.y, f.z + g.z, f.w + g.w);
            }
            if (!last) p[j] = f;
            v[4 * j] = __float_as_uint(f.x);
            v[4 * j + 1] = __float_as_uint(f.y);
            v[4 * j + 2] = __float_as_uint(f.z);
            v[4 * j + 3] = __float_as_uint(f.w);
          }
        }
#pragma unroll
        for (int j = 0; j < 16; ++j)
          o[16 * q + j] = f32x2_to_bf16x2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
      }
      if ((acc == nullptr || last) && m0 + 32 * warp < M) out.put(tm_out, o, c0, m0 + 32 * warp, lane);
    }
  }
};

struct GradArgs {
  gemm::Shape shape;
  float* acc;
  int add, last;
  int64_t M, N;
  unsigned int* check;
};

// A_MN 0: dH [tokens][d] = P W (P K-major, W MN-major); 1: dW [V][d] = P^T H (both MN-major)
template <int A_MN>
__global__ void __launch_bounds__(gemm::THREADS, 1)
grad_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
            const __grid_constant__ CUtensorMap tm_out, GradArgs a) {
  GradEpi epi{&tm_out, a.acc, a.add, a.last, a.M, a.N};
  gemm::run<A_MN, 1>(&tm_a, &tm_b, a.shape, epi, a.check);
}

// ----------------------------------------------------------------------------
// rows
// ----------------------------------------------------------------------------

// Number of tokens that take part (one CTA).
__global__ void __launch_bounds__(1024) count_kernel(const void* target, int target64, int64_t T, int64_t V,
                                                     int64_t ignore, unsigned int* check, int64_t* count) {
  __shared__ int sums[32];
  int c = 0;
  for (int64_t t = threadIdx.x; t < T; t += 1024) c += class_of(target, target64, t, V, ignore, check) >= 0;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) c += __shfl_xor_sync(0xffffffffu, c, off);
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = c;
  __syncthreads();
  if (threadIdx.x == 0) {
    int64_t total = 0;
    for (int w = 0; w < 32; ++w) total += sums[w];
    *count = total;
  }
}

// lse and loss of 32 tokens per block: eight thread rows walk the vocabulary's
// tiles and join (maximum, sum) pairs, then the eight pairs are joined in order.
// The loss is (maximum - l_target) + log(sum): next to lse - l_target it keeps the
// digits of a surely predicted token, whose maximum is the target's own logit.
// nll: the target's logits in, the losses out.
__global__ void __launch_bounds__(256) lse_kernel(const float2* __restrict__ stats, float* __restrict__ nll,
                                                  const void* target, int target64, int64_t ignore, int T, int64_t V,
                                                  int tiles, float* __restrict__ lse, float* __restrict__ losses,
                                                  unsigned int* check) {
  __shared__ float2 joined[8][32];
  const int t = blockIdx.x * 32 + threadIdx.x;
  float m = -INFINITY, s = 0.f;
  auto join = [](float& m, float& s, float m2, float s2) {
    // a NaN maximum (fmaxf drops it) still arrives through the sum
    const float top = fmaxf(m, m2);
    const float base = top == -INFINITY ? 0.f : top;
    s = s * expf(m - base) + s2 * expf(m2 - base);
    m = top;
  };
  if (t < T) {
#pragma unroll 4
    for (int i = threadIdx.y; i < tiles; i += 8) {
      const float2 p = stats[(int64_t)i * T + t];
      join(m, s, p.x, p.y);
    }
  }
  joined[threadIdx.y][threadIdx.x] = make_float2(m, s);
  __syncthreads();
  if (threadIdx.y == 0 && t < T) {
    for (int q = 1; q < 8; ++q) join(m, s, joined[q][threadIdx.x].x, joined[q][threadIdx.x].y);
    const float ls = logf(s);
    lse[t] = m + ls;
    const float loss = class_of(target, target64, t, V, ignore, check) >= 0 ? (m - nll[t]) + ls : 0.f;
    nll[t] = loss;
    if (losses != nullptr) losses[t] = loss;
  }
}

// Sum of the tokens' losses (one CTA, fixed order), divided by the count for the mean.
__global__ void __launch_bounds__(1024) loss_sum_kernel(const float* __restrict__ losses, int64_t T,
                                                        const int64_t* count, float* out) {
  __shared__ double sums[32];
  double s = 0.0;
  for (int64_t t = threadIdx.x; t < T; t += 1024) s += (double)losses[t];
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    double total = 0.0;
    for (int w = 0; w < 32; ++w) total += sums[w];
    if (count != nullptr) total /= (double)(*count > 0 ? *count : 1);
    *out = (float)total;
  }
}

// P in place of the exponentials: one CTA per token.
//   P_v = c exp(m_tile - lse) e_v,  P_target = c expm1(-loss)
struct ProbArgs {
  uint16_t* E;              // [T][pitch] fp16 in, bf16 out
  int64_t pitch;
  const float2* stats;
  const float* lse;
  const float* nll;
  const void* target;
  int target64;
  int64_t ignore_index;
  int T, V;
  const float* dloss;
  int dloss_each;           // dloss has one value per token
  const int64_t* count;     // divide by it (mean), or nullptr
  unsigned int* check;
};

constexpr int kProbThreads = 256;

__global__ void __launch_bounds__(kProbThreads) prob_kernel(ProbArgs a) {
  const int t = blockIdx.x;
  uint4* row = reinterpret_cast<uint4*>(a.E + (int64_t)t * a.pitch);
  const int units = (int)(a.pitch / 8);
  const int64_t y = class_of(a.target, a.target64, t, a.V, a.ignore_index, a.check);
  if (y < 0) {
    for (int u = threadIdx.x; u < units; u += kProbThreads) row[u] = make_uint4(0u, 0u, 0u, 0u);
    return;
  }
  float c = 1.f;
  if (a.dloss != nullptr) c = a.dloss[a.dloss_each ? t : 0];
  if (a.count != nullptr) c /= (float)(*a.count > 0 ? *a.count : 1);
  const float z = a.lse[t];
  const float at_target = c * expm1f(-a.nll[t]);
  // a warp's 32 units of eight columns are one 256-column tile: one factor per warp and step
  for (int u = threadIdx.x; u < units; u += kProbThreads) {
    const float f = c * __expf(a.stats[(int64_t)(u >> 5) * a.T + t].x - z);
    const uint4 v = row[u];
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const __half2 h = *reinterpret_cast<const __half2*>(&w[q]);
      float lo = __low2float(h) * f, hi = __high2float(h) * f;
      if ((int)y == 8 * u + 2 * q) lo = at_target;
      if ((int)y == 8 * u + 2 * q + 1) hi = at_target;
      w[q] = f32x2_to_bf16x2(lo, hi);
    }
    row[u] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// x *= factor in place, unless the factor is one
__global__ void __launch_bounds__(256) scale_kernel(uint4* __restrict__ x, int64_t units, const float* factor) {
  const float f = *factor;
  if (f == 1.f) return;
  for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < units; u += (int64_t)gridDim.x * 256) {
    const uint4 v = x[u];
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int q = 0; q < 4; ++q)
      w[q] = f32x2_to_bf16x2(__uint_as_float(w[q] << 16) * f, __uint_as_float(w[q] & 0xffff0000u) * f);
    x[u] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// ----------------------------------------------------------------------------
// workspace and launches
// ----------------------------------------------------------------------------

int64_t tiles_of(int64_t v) { return (v + 255) / 256; }

// Tokens per chunk.  With gradients: the largest multiple of 256 whose rows of
// exponentials fit the buffer (256 at least).
int64_t chunk_tokens(int64_t T, int64_t V, bool grads) {
  if (!grads) return T < kLossChunk ? T : kLossChunk;
  int64_t c = kExpBytes / (2 * up(V, 8)) / 256 * 256;
  if (c < 256) c = 256;
  return T < c ? T : c;
}

struct Layout {
  int64_t chunk, pitch;
  size_t e, acc, stats, lse, nll, losses, count, total;
};

Layout layout(int64_t T, int64_t V, int64_t d, bool dh, bool dw) {
  Layout l;
  const bool grads = dh || dw;
  l.chunk = chunk_tokens(T, V, grads);
  l.pitch = up(V, 8);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  };
  l.e = take(grads ? (size_t)l.chunk * l.pitch * 2 : 0);
  l.acc = take(dw && l.chunk < T ? (size_t)V * d * 4 : 0);
  l.stats = take((size_t)tiles_of(V) * l.chunk * 8);
  l.lse = take((size_t)l.chunk * 4);
  l.nll = take((size_t)l.chunk * 4);
  l.losses = take((size_t)T * 4);
  l.count = take(8);
  l.total = at;
  return l;
}

cudaError_t map_rows(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, int64_t pitch, int box_cols,
                     int box_rows) {
  return make_tmap_2d(m, base, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, (uint64_t)cols, (uint64_t)rows, (uint64_t)pitch * 2,
                      (uint32_t)box_cols, (uint32_t)box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <class Kern, class Args>
cudaError_t launch_pairs(Kern kern, const CUtensorMap& ma, const CUtensorMap& mb, const CUtensorMap& mc, const Args& args,
                         cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, gemm::SMEM);
  if (e != cudaSuccess) return e;
  const int tiles = args.shape.mt * args.shape.nt, pairs = num_sms() / 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2u * (unsigned)(tiles < pairs ? tiles : pairs), 1, 1);
  cfg.blockDim = dim3(gemm::THREADS, 1, 1);
  cfg.dynamicSmemBytes = gemm::SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, ma, mb, mc, args);
  return e != cudaSuccess ? e : cudaGetLastError();
}

gemm::Shape shape_of(int64_t M, int64_t N, int64_t K) {
  gemm::Shape s;
  s.mt = (int)tiles_of(M);
  s.nt = (int)tiles_of(N);
  s.ksteps = (int)((K + gemm::KS - 1) / gemm::KS);
  s.group = s.mt < 16 ? s.mt : 16;
  return s;
}

#define SK_TRY(x)                       \
  do {                                  \
    cudaError_t e_ = (x);               \
    if (e_ != cudaSuccess) return e_;   \
  } while (0)

}  // namespace

size_t cross_entropy_workspace(int64_t T, int64_t V, int64_t d, bool dh, bool dw) {
  return layout(T, V, d, dh, dw).total;
}

cudaError_t launch_cross_entropy(const CrossEntropy& a, cudaStream_t s) {
  const bool dh = a.dH != nullptr, dw = a.dW != nullptr, grads = dh || dw;
  const Layout l = layout(a.T, a.V, a.d, dh, dw);
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  uint16_t* E = reinterpret_cast<uint16_t*>(ws + l.e);
  float* acc = dw && l.chunk < a.T ? reinterpret_cast<float*>(ws + l.acc) : nullptr;
  float2* stats = reinterpret_cast<float2*>(ws + l.stats);
  float* lse = reinterpret_cast<float*>(ws + l.lse);
  float* nll = reinterpret_cast<float*>(ws + l.nll);
  float* losses = a.reduction == SK_CE_NONE ? a.loss : reinterpret_cast<float*>(ws + l.losses);
  int64_t* count = reinterpret_cast<int64_t*>(ws + l.count);
  const bool mean = a.reduction == SK_CE_MEAN;
  if (mean) {
    count_kernel<<<1, 1024, 0, s>>>(a.target, a.target64, a.T, a.V, a.ignore_index, a.check, count);
    SK_TRY(cudaGetLastError());
  }
  CUtensorMap tm_w, tm_w_mn, tm_dw;
  SK_TRY(map_rows(&tm_w, a.W, a.V, a.d, a.d, 64, 128));
  if (dh) SK_TRY(map_rows(&tm_w_mn, a.W, a.V, a.d, a.d, 64, 64));
  if (dw) SK_TRY(map_rows(&tm_dw, a.dW, a.V, a.d, a.d, 64, 32));
  const int vt = (int)tiles_of(a.V);
  for (int64_t t0 = 0; t0 < a.T; t0 += l.chunk) {
    const int64_t T = a.T - t0 < l.chunk ? a.T - t0 : l.chunk;
    const uint16_t* H = a.H + t0 * a.d;
    const void* target = static_cast<const uint8_t*>(a.target) + t0 * (a.target64 ? 8 : 4);
    CUtensorMap tm_h, tm_e;
    SK_TRY(map_rows(&tm_h, H, T, a.d, a.d, 64, 128));
    tm_e = tm_h;                                   // not used without gradients
    if (grads) SK_TRY(map_rows(&tm_e, E, T, a.V, l.pitch, 64, 32));
    LogitArgs la{shape_of(T, a.V, a.d), stats, nll, target, a.target64, a.ignore_index, (int)T, (int)a.V,
                 grads ? 1 : 0, a.check};
    SK_TRY(launch_pairs(logit_kernel, tm_h, tm_w, tm_e, la, s));
    lse_kernel<<<(unsigned)((T + 31) / 32), dim3(32, 8), 0, s>>>(stats, nll, target, a.target64, a.ignore_index,
                                                                 (int)T, a.V, vt, lse, losses ? losses + t0 : nullptr,
                                                                 a.check);
    SK_TRY(cudaGetLastError());
    if (!grads) continue;
    const bool each = a.reduction == SK_CE_NONE;
    ProbArgs pa{E, l.pitch, stats, lse, nll, target, a.target64, a.ignore_index, (int)T, (int)a.V,
                each && a.dloss ? a.dloss + t0 : a.dloss, each ? 1 : 0, mean ? count : nullptr, a.check};
    prob_kernel<<<(unsigned)T, kProbThreads, 0, s>>>(pa);
    SK_TRY(cudaGetLastError());
    if (dh) {
      CUtensorMap tm_p, tm_dh;
      SK_TRY(map_rows(&tm_p, E, T, a.V, l.pitch, 64, 128));
      SK_TRY(map_rows(&tm_dh, a.dH + t0 * a.d, T, a.d, a.d, 64, 32));
      GradArgs ga{shape_of(T, a.d, a.V), nullptr, 0, 1, T, a.d, a.check};
      SK_TRY(launch_pairs(grad_kernel<0>, tm_p, tm_w_mn, tm_dh, ga, s));
    }
    if (dw) {
      CUtensorMap tm_p, tm_hm;
      SK_TRY(map_rows(&tm_p, E, T, a.V, l.pitch, 64, 64));
      SK_TRY(map_rows(&tm_hm, H, T, a.d, a.d, 64, 64));
      GradArgs ga{shape_of(a.V, a.d, T), acc, t0 > 0 ? 1 : 0, t0 + T >= a.T ? 1 : 0, a.V, a.d, a.check};
      SK_TRY(launch_pairs(grad_kernel<1>, tm_p, tm_hm, tm_dw, ga, s));
    }
  }
  if (a.reduction != SK_CE_NONE && a.loss != nullptr) {
    loss_sum_kernel<<<1, 1024, 0, s>>>(losses, a.T, mean ? count : nullptr, a.loss);
    SK_TRY(cudaGetLastError());
  }
  return cudaSuccess;
}

cudaError_t launch_scale_bf16(uint16_t* x, int64_t count, const float* factor, cudaStream_t s) {
  const int64_t units = count / 8;
  const int64_t blocks = (units + 255) / 256, cap = (int64_t)num_sms() * 8;
  scale_kernel<<<(unsigned)(blocks < cap ? blocks : cap), 256, 0, s>>>(reinterpret_cast<uint4*>(x), units, factor);
  return cudaGetLastError();
}

}  // namespace sk
