// Layer norm and RMS norm of [T][d] rows: forward (with the 8-bit checkpoint of
// its output when asked for) and backward with the reduction of the weight's
// and the bias's gradient.
//
//   xh = (x - mu) r,  r = 1 / sqrt(mean((x - mu)^2) + eps)     (RMS norm: mu = 0)
//   y  = xh w + b
//   u  = dy w,  dx = r (u - mean(u) - xh mean(u xh))           (RMS norm: without mean(u))
//   dw = sum over rows of dy xh,  db = sum over rows of dy
//
// Every value is computed in fp32 and rounded once.  The variance is the mean
// square of the centred values (two passes over registers), so a row whose mean
// is far larger than its spread loses no more than the rounding of that mean (a few
// 2^-24 of it), which 16-bit rows do not notice.  rstd is 1 / sqrtf in the kernels of one row
// and rsqrtf (2 steps of 2^-23 at most) in those of two, and the sums' orders differ between them.
//
// Both directions are bound by memory: 2 values of traffic per element forward,
// 4 over both directions.  A team of threads (one warp for short rows, one CTA
// otherwise) holds a row in registers and owns the same columns for every row
// it takes, so w and b are read once per team and the sums for dw and db never
// leave registers until the team has no rows left; the next row's loads are
// issued before this row's reductions.  The teams' sums go to [teams][2][d]
// partials that a second kernel adds in a fixed order: deterministic, no
// atomics.
#include "sk_ckpt8.cuh"
#include "sk_norm.cuh"

namespace sk {
namespace {

// ----------------------------------------------------------------------------
// rows in registers
// ----------------------------------------------------------------------------

// eight elements of type T as 32-bit words
template <typename T>
struct Raw {
  static constexpr int NW = (int)sizeof(T) * 2;
  uint32_t w[NW];
};

template <typename T>
__device__ __forceinline__ float elem(const Raw<T>& r, int i);
template <>
__device__ __forceinline__ float elem<float>(const Raw<float>& r, int i) { return __uint_as_float(r.w[i]); }
template <>
__device__ __forceinline__ float elem<__nv_bfloat16>(const Raw<__nv_bfloat16>& r, int i) {
  return __uint_as_float((i & 1) ? (r.w[i >> 1] & 0xffff0000u) : (r.w[i >> 1] << 16));
}
template <>
__device__ __forceinline__ float elem<__half>(const Raw<__half>& r, int i) {
  const __half2 h = *reinterpret_cast<const __half2*>(&r.w[i >> 1]);
  return (i & 1) ? __high2float(h) : __low2float(h);
}

__device__ __forceinline__ uint32_t bits_of(float v) { return __float_as_uint(v); }
__device__ __forceinline__ uint32_t bits_of(__nv_bfloat16 v) { return *reinterpret_cast<uint16_t*>(&v); }
__device__ __forceinline__ uint32_t bits_of(__half v) { return *reinterpret_cast<uint16_t*>(&v); }

template <typename T>
__device__ __forceinline__ T round_to(float v);
template <>
__device__ __forceinline__ float round_to<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 round_to<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half round_to<__half>(float v) { return __float2half_rn(v); }

template <typename T>
__device__ __forceinline__ void pack8(const float (&v)[8], Raw<T>& r) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.w[i] = __float_as_uint(v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) r.w[i] = bits_of(round_to<T>(v[2 * i])) | (bits_of(round_to<T>(v[2 * i + 1])) << 16);
  }
}

// A team's view of a row: chunk c of member `me` of `team` holds eight columns, in
// groups of V consecutive ones (V = 8, 4, 2 or 1, a divisor of d, so that a group is
// aligned in every row and inside or outside it as a whole); the chunk's groups are
// team * V columns apart.
// SAFE: the first so many chunks lie inside the row, nothing to check.
template <int V, int SAFE = 0>
struct Cols {
  int me, team, d;
  __device__ __forceinline__ int col(int c, int k) const {
    return ((c * (8 / V) + k / V) * team + me) * V + k % V;
  }
  __device__ __forceinline__ bool in(int c, int k) const { return c < SAFE || col(c, k / V * V) < d; }
};

// N 32-bit words (2 or a multiple of 4, 1 for a store), aligned to their size up to 16 bytes
template <int N>
__device__ __forceinline__ void load_words(uint32_t* w, const void* p) {
  if constexpr (N == 2) {
    const uint2 v = __ldg(static_cast<const uint2*>(p));
    w[0] = v.x; w[1] = v.y;
  } else {
#pragma unroll
    for (int q = 0; q < N / 4; ++q) {
      const uint4 v = __ldg(static_cast<const uint4*>(p) + q);
      w[4 * q] = v.x; w[4 * q + 1] = v.y; w[4 * q + 2] = v.z; w[4 * q + 3] = v.w;
    }
  }
}
template <int N>
__device__ __forceinline__ void store_words(void* p, const uint32_t* w) {
  if constexpr (N == 1) {
    *static_cast<uint32_t*>(p) = w[0];
  } else if constexpr (N == 2) {
    *static_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int q = 0; q < N / 4; ++q) static_cast<uint4*>(p)[q] = make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
  }
}

template <typename T, int V, int SAFE>
__device__ __forceinline__ void load8(Raw<T>& r, const T* __restrict__ row, const Cols<V, SAFE>& C, int c) {
  if constexpr (V > 1 && V * sizeof(T) == 4) {
#pragma unroll
    for (int g = 0; g < 8 / V; ++g)
      r.w[g] = C.in(c, g * V) ? __ldg(reinterpret_cast<const uint32_t*>(row + C.col(c, g * V))) : 0u;
  } else if constexpr (V > 1) {
    constexpr int N = V * (int)sizeof(T) / 4;
#pragma unroll
    for (int g = 0; g < 8 / V; ++g) {
      if (C.in(c, g * V)) {
        load_words<N>(r.w + g * N, row + C.col(c, g * V));
      } else {
#pragma unroll
        for (int q = 0; q < N; ++q) r.w[g * N + q] = 0u;
      }
    }
  } else {
    uint32_t b[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) b[k] = C.in(c, k) ? bits_of(__ldg(row + C.col(c, k))) : 0u;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int k = 0; k < 8; ++k) r.w[k] = b[k];
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) r.w[k] = b[2 * k] | (b[2 * k + 1] << 16);
    }
  }
}

template <typename T, int V, int SAFE>
__device__ __forceinline__ void store8(T* __restrict__ row, const Raw<T>& r, const Cols<V, SAFE>& C, int c) {
  if constexpr (V > 1) {
    constexpr int N = V * (int)sizeof(T) / 4;
#pragma unroll
    for (int g = 0; g < 8 / V; ++g)
      if (C.in(c, g * V)) store_words<N>(row + C.col(c, g * V), r.w + g * N);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (!C.in(c, k)) continue;
      if constexpr (sizeof(T) == 4) reinterpret_cast<uint32_t*>(row)[C.col(c, k)] = r.w[k];
      else reinterpret_cast<uint16_t*>(row)[C.col(c, k)] = (uint16_t)(r.w[k >> 1] >> (16 * (k & 1)));
    }
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// Sum over the team, in every member.  WARP: the team is a warp; else it is the
// CTA and `buf` holds one float per warp.  A CTA's caller alternates between
// buffers so that a buffer is written again only after a later sum's barrier.
template <bool WARP>
__device__ __forceinline__ float team_sum(float v, float* buf) {
  v = warp_sum(v);
  if constexpr (WARP) return v;
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  if (lane == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_sum(lane < warps ? buf[lane] : 0.f);
}

template <bool WARP>
__device__ __forceinline__ float2 team_sum2(float2 v, float2* buf) {
  v.x = warp_sum(v.x);
  v.y = warp_sum(v.y);
  if constexpr (WARP) return v;
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  if (lane == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < warps ? buf[lane] : make_float2(0.f, 0.f);
  return make_float2(warp_sum(v.x), warp_sum(v.y));
}

// CTAs per SM to leave registers for.  Single 16-bit values take many registers for
// their addresses when left alone: one or two CTAs fit, and [4096, 4095] bf16 takes 52
// + 70 us forward and backward, against 40 + 43 at `threads` per SM.  (Single fp32
// values spill then, 4.9 against 10.2 us backward at [1111, 1001].)
template <typename T, int V>
constexpr int few_ctas(int maxt, int threads) {
  return V == 1 && sizeof(T) == 2 && maxt <= 256 ? threads / maxt : 0;     // 0: left to the compiler
}

// ----------------------------------------------------------------------------
// forward
// ----------------------------------------------------------------------------

template <typename T, typename WT, int NC, int MAXT, int V, bool WARP, bool CK>
__global__ void __launch_bounds__(MAXT, few_ctas<T, V>(MAXT, 768)) norm_fwd_kernel(NormFwd a) {
  __shared__ float buf[2][32];
  const int lane = threadIdx.x & 31;
  const Cols<V> C{WARP ? lane : (int)threadIdx.x, WARP ? 32 : (int)blockDim.x, (int)a.d};
  const int64_t teams = WARP ? (int64_t)gridDim.x * (blockDim.x >> 5) : gridDim.x;
  int64_t t = WARP ? (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
  const T* x = static_cast<const T*>(a.x);
  Raw<WT> w[NC], b[NC];
  Raw<T> cur[NC], nxt[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    if (t < a.T) load8<T>(cur[c], x + t * a.d, C, c);
    load8<WT>(w[c], static_cast<const WT*>(a.w), C, c);
    if (a.b != nullptr) load8<WT>(b[c], static_cast<const WT*>(a.b), C, c);
  }
  const float inv_d = 1.f / (float)a.d;
  // Buffers of the sums: a layer norm's two sums take turns; an RMS norm's only
  // sum changes buffers from row to row.
  int second = 1;
  for (; t < a.T; t += teams) {
    const bool more = t + teams < a.T;
#pragma unroll
    for (int c = 0; c < NC; ++c)
      if (more) load8<T>(nxt[c], x + (t + teams) * a.d, C, c);
    float mu = 0.f;
    if (!a.rms) {
      float s = 0.f;
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int k = 0; k < 8; ++k) s += elem(cur[c], k);    // columns beyond the row hold zeros
      mu = team_sum<WARP>(s, buf[0]) * inv_d;
    }
    float s2 = 0.f;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float v = C.in(c, k) ? elem(cur[c], k) - mu : 0.f;
        s2 = fmaf(v, v, s2);
      }
    const float var = team_sum<WARP>(s2, buf[second]) * inv_d;
    if (a.rms) second ^= 1;
    const float r = 1.f / sqrtf(var + a.eps);
    if (C.me == 0) {
      if (a.mean != nullptr) a.mean[t] = mu;
      if (a.rstd != nullptr) a.rstd[t] = r;
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        v[k] = (elem(cur[c], k) - mu) * r * elem(w[c], k);
        if (a.b != nullptr) v[k] += elem(b[c], k);
      }
      Raw<T> o;
      pack8<T>(v, o);
      store8<T>(static_cast<T*>(a.y) + t * a.d, o, C, c);
      if constexpr (CK) {
        // four neighbouring lanes hold one 32-column block (d % 32 == 0)
        uint32_t byte;
        const uint2 q8 = ckpt8_quantize8(o.w, byte);
        if (C.in(c, 0)) {
          const int64_t at = t * a.d + C.col(c, 0);
          *reinterpret_cast<uint2*>(a.q + at) = q8;
          if ((lane & 3) == 0) a.qscale[at >> 5] = (uint8_t)byte;
        }
      }
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) cur[c] = nxt[c];
  }
}

// ----------------------------------------------------------------------------
// backward
// ----------------------------------------------------------------------------

// DW: also accumulate dw and db over the team's rows and write them as partial
// row blockIdx.x of a.part ([parts][2][d]); else dx alone.
template <typename T, typename WT, int NC, int MAXT, int V, bool WARP, bool DW>
__global__ void __launch_bounds__(MAXT, few_ctas<T, V>(MAXT, 512)) norm_bwd_kernel(NormBwd a) {
  extern __shared__ float wpart[];                 // WARP with DW: [warps][2][NC * 256]
  __shared__ float2 buf[2][32];
  const int lane = threadIdx.x & 31;
  const Cols<V> C{WARP ? lane : (int)threadIdx.x, WARP ? 32 : (int)blockDim.x, (int)a.d};
  const int64_t teams = WARP ? (int64_t)gridDim.x * (blockDim.x >> 5) : gridDim.x;
  int64_t t = WARP ? (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
  const T* x = static_cast<const T*>(a.x);
  const T* dy = static_cast<const T*>(a.dy);
  Raw<WT> w[NC];
  Raw<T> cx[NC], cd[NC], nx[NC], nd[NC];
  float dw[DW ? NC : 1][8], db[DW ? NC : 1][8];
  float mu = 0.f, r = 0.f;
  auto fetch = [&](int64_t row, Raw<T>(&rx)[NC], Raw<T>(&rd)[NC], float& m, float& rs) {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      load8<T>(rx[c], x + row * a.d, C, c);
      load8<T>(rd[c], dy + row * a.d, C, c);
    }
    m = a.rms ? 0.f : __ldg(a.mean + row);
    rs = __ldg(a.rstd + row);
  };
  if (t < a.T) fetch(t, cx, cd, mu, r);
#pragma unroll
  for (int c = 0; c < NC; ++c) load8<WT>(w[c], static_cast<const WT*>(a.w), C, c);
  if constexpr (DW) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int k = 0; k < 8; ++k) dw[c][k] = db[c][k] = 0.f;
  }
  const float inv_d = 1.f / (float)a.d;
  int parity = 0;
  for (; t < a.T; t += teams, parity ^= 1) {
    const bool more = t + teams < a.T;
    float nmu = 0.f, nr = 0.f;
    if (more) fetch(t + teams, nx, nd, nmu, nr);
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        // beyond the row dy is zero, so these terms are too
        const float g = elem(cd[c], k), xh = (elem(cx[c], k) - mu) * r;
        const float u = g * elem(w[c], k);
        s.x += u;
        s.y = fmaf(u, xh, s.y);
        if constexpr (DW) {
          dw[c][k] = fmaf(g, xh, dw[c][k]);
          db[c][k] += g;
        }
      }
    s = team_sum2<WARP>(s, buf[parity]);
    const float m1 = a.rms ? 0.f : s.x * inv_d, m2 = s.y * inv_d;
    if (a.dx != nullptr) {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float xh = (elem(cx[c], k) - mu) * r;
          v[k] = r * (elem(cd[c], k) * elem(w[c], k) - m1 - xh * m2);
        }
        Raw<T> o;
        pack8<T>(v, o);
        store8<T>(static_cast<T*>(a.dx) + t * a.d, o, C, c);
      }
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      cx[c] = nx[c];
      cd[c] = nd[c];
    }
    mu = nmu;
    r = nr;
  }
  if constexpr (DW) {
    float* part = a.part + (int64_t)blockIdx.x * 2 * a.d;
    if constexpr (WARP) {
      // the CTA's warps own the same columns: add their sums in warp order
      const int warps = blockDim.x >> 5, span = NC * 256;
      float* mine = wpart + (size_t)(threadIdx.x >> 5) * 2 * span;
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          mine[C.col(c, k)] = dw[c][k];
          mine[span + C.col(c, k)] = db[c][k];
        }
      __syncthreads();
      for (int e = threadIdx.x; e < 2 * (int)a.d; e += blockDim.x) {
        const int which = e >= (int)a.d, col = e - which * (int)a.d;
        float sum = 0.f;
        for (int v = 0; v < warps; ++v) sum += wpart[(size_t)v * 2 * span + which * span + col];
        part[e] = sum;
      }
    } else {
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (C.in(c, k)) {
            part[C.col(c, k)] = dw[c][k];
            part[a.d + C.col(c, k)] = db[c][k];
          }
    }
  }
}

// ----------------------------------------------------------------------------
// many rows: two at a time
// ----------------------------------------------------------------------------
//
// With thousands of rows what costs is not latency but work per value: a forward
// CTA that loads w and b (8 bytes per column in fp32, from L1) for one bf16 row of
// 2 + 2 bytes per column spends more on them than on the row, and shuffles and
// barriers come once per thread and row whatever the thread holds.  So these
// kernels give a thread more columns (32 in 16 bits) and a CTA two neighbouring
// rows, whose sums cross the warps together (four sums in six shuffles, one
// barrier), and use packed fp32 pairs for the arithmetic.  At [8192, 4096] bf16
// with fp32 weights, where copying the rows takes 23 us: one row per CTA and 16
// columns per thread 33-35 us, two rows and 32 columns 27 us; more rows or more
// columns per thread lose it again to occupancy.

using f2 = uint64_t;                               // two fp32 values

__device__ __forceinline__ f2 f2_of(float lo, float hi) {
  f2 v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  return v;
}
__device__ __forceinline__ float2 f2_get(f2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f2 f2_add(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 f2_mul(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 f2_fma(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float f2_sum(f2 v) {
  const float2 r = f2_get(v);
  return r.x + r.y;
}

// values 2 i and 2 i + 1 of eight
template <typename T>
__device__ __forceinline__ f2 pair_of(const Raw<T>& r, int i) {
  return f2_of(elem(r, 2 * i), elem(r, 2 * i + 1));
}
template <typename T>
__device__ __forceinline__ void pack_pairs(const f2 (&v)[4], Raw<T>& r) {
  float e[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = f2_get(v[i]);
    e[2 * i] = x.x;
    e[2 * i + 1] = x.y;
  }
  pack8<T>(e, r);
}

// Chunks of eight columns per thread in the kernels of two rows: 32 columns in 16
// bits, 16 in fp32 (the same registers).
template <typename T>
__host__ __device__ constexpr int pair_chunks() { return sizeof(T) == 2 ? 4 : 2; }

// FULL kernels take rows that their threads cover exactly.  In the others half of a
// thread's chunks are inside the row all the same, since team_threads takes no more
// threads than d > 512 columns need.

// Sums of N = 2 or 4 values over the CTA, in every thread.  Within a warp the lanes
// share the values out as they halve: N - 1 + (5 - log2 N) shuffles.  buf: [N][32]
// floats, written again only after a later sum's barrier.
template <int N>
__device__ __forceinline__ void cta_sums(float (&v)[N], float* buf) {
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  float a;
  int which;
  if constexpr (N == 4) {
    const bool up = lane & 16;
    const float s0 = up ? v[0] : v[2], s1 = up ? v[1] : v[3];
    const float k0 = (up ? v[2] : v[0]) + __shfl_xor_sync(0xffffffffu, s0, 16);
    const float k1 = (up ? v[3] : v[1]) + __shfl_xor_sync(0xffffffffu, s1, 16);
    const bool up2 = lane & 8;
    a = (up2 ? k1 : k0) + __shfl_xor_sync(0xffffffffu, up2 ? k0 : k1, 8);
    which = (lane >> 4) * 2 + ((lane >> 3) & 1);
  } else {
    const bool up = lane & 16;
    a = (up ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, up ? v[0] : v[1], 16);
    a += __shfl_xor_sync(0xffffffffu, a, 8);
    which = lane >> 4;
  }
  a += __shfl_xor_sync(0xffffffffu, a, 4);
  a += __shfl_xor_sync(0xffffffffu, a, 2);
  a += __shfl_xor_sync(0xffffffffu, a, 1);
  if ((lane & (N == 4 ? 7 : 15)) == 0) buf[which * 32 + (threadIdx.x >> 5)] = a;
  __syncthreads();
#pragma unroll
  for (int n = 0; n < N; ++n) {
    float sum = 0.f;
    for (int w = 0; w < warps; w += 4) {           // entries beyond the warps are zero
      const float4 p = *reinterpret_cast<const float4*>(buf + n * 32 + w);
      sum += (p.x + p.y) + (p.z + p.w);
    }
    v[n] = sum;
  }
}

// The sums' entries beyond the last warp, up to the next four.
__device__ __forceinline__ void clear_sums(float* buf, int n) {
  const int warps = blockDim.x >> 5;
  if ((warps & 3) == 0) return;
  for (int i = threadIdx.x; i < n * 32; i += blockDim.x)
    if ((i & 31) >= warps) buf[i] = 0.f;              // no thread writes these entries later
}

// Forward: CTA = rows 2 blockIdx.x and the next.
template <typename T, typename WT, int MAXT, int MINB, bool RMS, bool BIAS, bool CK, bool FULL>
__global__ void __launch_bounds__(MAXT, MINB) norm_fwd_pair_kernel(NormFwd a) {
  constexpr int NC = pair_chunks<T>(), R = 2;
  __shared__ __align__(16) float buf[2][R * 32];
  const int lane = threadIdx.x & 31;
  const Cols<8, FULL ? NC : NC / 2> C{(int)threadIdx.x, (int)blockDim.x, (int)a.d};
  const int64_t t = (int64_t)blockIdx.x * R;
  const bool two = a.T - t >= R;
  const T* x = static_cast<const T*>(a.x) + t * a.d;
  Raw<T> cur[R][NC];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      if (r == 0 || two) load8<T>(cur[r][c], x + r * a.d, C, c);
      else cur[r][c] = Raw<T>{};
    }
  clear_sums(&buf[0][0], 2 * R);
  const float inv_d = 1.f / (float)a.d;
  float mu[R] = {0.f, 0.f}, var[R];
  if constexpr (!RMS) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      f2 sum = f2_of(0.f, 0.f);
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) sum = f2_add(sum, pair_of(cur[r][c], i));
      mu[r] = f2_sum(sum);
    }
    cta_sums<R>(mu, buf[0]);
#pragma unroll
    for (int r = 0; r < R; ++r) mu[r] *= inv_d;
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    f2 sum = f2_of(0.f, 0.f);
    const f2 off = f2_of(-mu[r], -mu[r]);
#pragma unroll
    for (int c = 0; c < NC; ++c)
      if (C.in(c, 0)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f2 v = RMS ? pair_of(cur[r][c], i) : f2_add(pair_of(cur[r][c], i), off);
          sum = f2_fma(v, v, sum);
        }
      }
    var[r] = f2_sum(sum);
  }
  cta_sums<R>(var, buf[1]);
  float rs[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    rs[r] = rsqrtf(var[r] * inv_d + a.eps);
    if (threadIdx.x == 0 && (r == 0 || two)) {
      if (a.mean != nullptr) a.mean[t + r] = mu[r];
      if (a.rstd != nullptr) a.rstd[t + r] = rs[r];
    }
  }
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    Raw<WT> w, b;
    load8<WT>(w, static_cast<const WT*>(a.w), C, c);
    if constexpr (BIAS) load8<WT>(b, static_cast<const WT*>(a.b), C, c);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (r > 0 && !two) break;
      const f2 off = f2_of(-mu[r], -mu[r]), scale = f2_of(rs[r], rs[r]);
      f2 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f2 xh = f2_mul(RMS ? pair_of(cur[r][c], i) : f2_add(pair_of(cur[r][c], i), off), scale);
        if constexpr (BIAS) v[i] = f2_fma(xh, pair_of(w, i), pair_of(b, i));
        else v[i] = f2_mul(xh, pair_of(w, i));
      }
      Raw<T> o;
      pack_pairs<T>(v, o);
      store8<T>(static_cast<T*>(a.y) + (t + r) * a.d, o, C, c);
      if constexpr (CK) {
        uint32_t byte;
        const uint2 q8 = ckpt8_quantize8(o.w, byte);
        if (C.in(c, 0)) {
          const int64_t at = (t + r) * a.d + C.col(c, 0);
          *reinterpret_cast<uint2*>(a.q + at) = q8;
          if ((lane & 3) == 0) a.qscale[at >> 5] = (uint8_t)byte;
        }
      }
    }
  }
}

// dx alone (a norm whose weights are not trained): CTA = rows 2 blockIdx.x and the next.
template <typename T, typename WT, int MAXT, int MINB, bool RMS, bool FULL>
__global__ void __launch_bounds__(MAXT, MINB) norm_dx_pair_kernel(NormBwd a) {
  constexpr int NC = pair_chunks<T>(), R = 2;
  __shared__ __align__(16) float buf[2 * R * 32];
  const Cols<8, FULL ? NC : NC / 2> C{(int)threadIdx.x, (int)blockDim.x, (int)a.d};
  const int64_t t = (int64_t)blockIdx.x * R;
  const bool two = a.T - t >= R;
  const T* x = static_cast<const T*>(a.x) + t * a.d;
  const T* dy = static_cast<const T*>(a.dy) + t * a.d;
  Raw<T> cx[R][NC], cd[R][NC];
  f2 off[R], scale[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const bool there = r == 0 || two;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      if (there) {
        load8<T>(cx[r][c], x + r * a.d, C, c);
        load8<T>(cd[r][c], dy + r * a.d, C, c);
      } else {
        cx[r][c] = cd[r][c] = Raw<T>{};
      }
    }
    const float m = RMS || !there ? 0.f : __ldg(a.mean + t + r), rs = there ? __ldg(a.rstd + t + r) : 0.f;
    off[r] = f2_of(-m, -m);
    scale[r] = f2_of(rs, rs);
  }
  clear_sums(buf, 2 * R);
  const float inv_d = 1.f / (float)a.d;
  float sums[2 * R];
  {
    f2 su[R], sux[R];
#pragma unroll
    for (int r = 0; r < R; ++r) su[r] = sux[r] = f2_of(0.f, 0.f);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      Raw<WT> w;
      load8<WT>(w, static_cast<const WT*>(a.w), C, c);
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f2 px = pair_of(cx[r][c], i);
          const f2 xh = f2_mul(RMS ? px : f2_add(px, off[r]), scale[r]);
          const f2 u = f2_mul(pair_of(cd[r][c], i), pair_of(w, i));      // zero beyond the row
          if constexpr (!RMS) su[r] = f2_add(su[r], u);
          sux[r] = f2_fma(u, xh, sux[r]);
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      sums[r] = f2_sum(sux[r]);
      sums[R + r] = f2_sum(su[r]);
    }
  }
  cta_sums<2 * R>(sums, buf);
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    Raw<WT> w;
    load8<WT>(w, static_cast<const WT*>(a.w), C, c);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (r > 0 && !two) break;
      const float m1 = sums[R + r] * inv_d, m2 = sums[r] * inv_d;
      const f2 n1 = f2_of(-m1, -m1), n2 = f2_of(-m2, -m2);
      f2 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f2 px = pair_of(cx[r][c], i);
        const f2 xh = f2_mul(RMS ? px : f2_add(px, off[r]), scale[r]);
        f2 u = f2_mul(pair_of(cd[r][c], i), pair_of(w, i));
        if constexpr (!RMS) u = f2_add(u, n1);
        v[i] = f2_mul(f2_fma(xh, n2, u), scale[r]);
      }
      Raw<T> o;
      pack_pairs<T>(v, o);
      store8<T>(static_cast<T*>(a.dx) + (t + r) * a.d, o, C, c);
    }
  }
}

// Backward with dw and db.  The sums over rows want few CTAs that keep their
// columns in registers (48 of them with w), so rows come through a ring in shared
// memory: thread 0 asks for pairs of rows ahead by bulk copies, and the values are
// read from there for the sums and again for dx, which leaves the registers to the
// accumulators.  A slot is asked for again after the next pair's barrier, by which
// every thread is done with it.  At [8192, 4096] bf16 (31 us for its traffic at
// the copy rate): one row at a time in registers 47-52 us, pairs from the ring 43 us,
// and 38 with the rows' statistics asked for a pair ahead too.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               ::"r"(tc::smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(tc::smem_u32(bar))
               : "memory");
}

constexpr int kMaxStages = 4;

struct Ring {
  int stages;
  uint32_t row_bytes;      // a slot holds two rows of x and two of dy
};

template <typename T, int SAFE>
__device__ __forceinline__ void take8(Raw<T>& r, const uint8_t* row, const Cols<8, SAFE>& C, int c, bool there) {
  if (there && C.in(c, 0)) {
    const uint4* p = reinterpret_cast<const uint4*>(row + (size_t)C.col(c, 0) * sizeof(T));
#pragma unroll
    for (int q = 0; q < Raw<T>::NW / 4; ++q) {
      const uint4 v = p[q];
      r.w[4 * q] = v.x; r.w[4 * q + 1] = v.y; r.w[4 * q + 2] = v.z; r.w[4 * q + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int q = 0; q < Raw<T>::NW; ++q) r.w[q] = 0u;
  }
}

template <typename T, typename WT, int MAXT, int MINB, bool RMS, bool FULL>
__global__ void __launch_bounds__(MAXT, MINB) norm_bwd_ring_kernel(NormBwd a, Ring ring) {
  constexpr int NC = 2, R = 2;
  extern __shared__ __align__(128) uint8_t rows[];           // [stages][R rows of x, R rows of dy]
  __shared__ uint64_t full[kMaxStages];
  __shared__ __align__(16) float buf[2][2 * R * 32];
  const Cols<8, FULL ? NC : NC / 2> C{(int)threadIdx.x, (int)blockDim.x, (int)a.d};
  const T* x = static_cast<const T*>(a.x);
  const T* dy = static_cast<const T*>(a.dy);
  const int64_t step = (int64_t)gridDim.x * R;
  int64_t t = (int64_t)blockIdx.x * R;
  const uint32_t half_slot = R * ring.row_bytes;
  auto ask = [&](int64_t row, int s) {
    if (row >= a.T) return;
    const uint32_t bytes = (a.T - row >= R ? R : 1) * ring.row_bytes;
    uint8_t* slot = rows + (size_t)s * 2 * half_slot;
    tc::mbar_arrive_expect_tx(&full[s], 2 * bytes);
    bulk_load(slot, x + row * a.d, bytes, &full[s]);
    bulk_load(slot + half_slot, dy + row * a.d, bytes, &full[s]);
  };
  clear_sums(&buf[0][0], 2 * 2 * R);
  if (threadIdx.x == 0) {
    for (int s = 0; s < ring.stages; ++s) tc::mbar_init(&full[s], 1);
    tc::fence_mbar_init();
    for (int s = 0; s + 1 < ring.stages; ++s) ask(t + s * step, s);
  }
  Raw<WT> w[NC];
  f2 dw[NC][4], db[NC][4];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    load8<WT>(w[c], static_cast<const WT*>(a.w), C, c);
#pragma unroll
    for (int i = 0; i < 4; ++i) dw[c][i] = db[c][i] = f2_of(0.f, 0.f);
  }
  __syncthreads();
  const float inv_d = 1.f / (float)a.d;
  int s = 0, before = ring.stages - 1, parity = 0;
  uint32_t phase = 0;
  // the next pair's statistics, asked for a pair ahead as well
  float mean[R], rstd[R];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const bool there = row + r < a.T;
      mean[r] = RMS || !there ? 0.f : __ldg(a.mean + row + r);
      rstd[r] = there ? __ldg(a.rstd + row + r) : 0.f;
    }
  };
  fetch(t);
  for (; t < a.T; t += step, parity ^= 1) {
    const bool two = a.T - t >= R;
    f2 off[R], scale[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      off[r] = f2_of(-mean[r], -mean[r]);
      scale[r] = f2_of(rstd[r], rstd[r]);
    }
    fetch(t + step);
    if (!tc::mbar_wait(&full[s], phase, a.check)) {
      // never leave with a copy still landing: the slots asked for ahead, each with its limit
      for (int k = 1; k + 1 < ring.stages && t + k * step < a.T; ++k) {
        if (++s == ring.stages) {
          s = 0;
          phase ^= 1u;
        }
        tc::mbar_wait(&full[s], phase, a.check);
      }
      return;
    }
    const uint8_t* slot = rows + (size_t)s * 2 * half_slot;
    float sums[2 * R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      f2 su = f2_of(0.f, 0.f), sux = f2_of(0.f, 0.f);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        Raw<T> vx, vd;                // beyond the row, and in a second row that is not there, zeros
        take8<T>(vx, slot + r * ring.row_bytes, C, c, r == 0 || two);
        take8<T>(vd, slot + half_slot + r * ring.row_bytes, C, c, r == 0 || two);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f2 g = pair_of(vd, i), px = pair_of(vx, i);
          const f2 xh = f2_mul(RMS ? px : f2_add(px, off[r]), scale[r]);
          const f2 u = f2_mul(g, pair_of(w[c], i));
          if constexpr (!RMS) su = f2_add(su, u);
          sux = f2_fma(u, xh, sux);
          dw[c][i] = f2_fma(g, xh, dw[c][i]);
          db[c][i] = f2_add(db[c][i], g);
        }
      }
      sums[r] = f2_sum(sux);
      sums[R + r] = f2_sum(su);
    }
    cta_sums<2 * R>(sums, buf[parity]);
    if (threadIdx.x == 0) ask(t + (ring.stages - 1) * step, before);
    before = s;
    if (++s == ring.stages) {
      s = 0;
      phase ^= 1u;
    }
    if (a.dx == nullptr) continue;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (r > 0 && !two) break;
      const float m1 = sums[R + r] * inv_d, m2 = sums[r] * inv_d;
      const f2 n1 = f2_of(-m1, -m1), n2 = f2_of(-m2, -m2);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        Raw<T> vx, vd;
        take8<T>(vx, slot + r * ring.row_bytes, C, c, true);
        take8<T>(vd, slot + half_slot + r * ring.row_bytes, C, c, true);
        f2 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f2 px = pair_of(vx, i);
          const f2 xh = f2_mul(RMS ? px : f2_add(px, off[r]), scale[r]);
          f2 u = f2_mul(pair_of(vd, i), pair_of(w[c], i));
          if constexpr (!RMS) u = f2_add(u, n1);
          v[i] = f2_mul(f2_fma(xh, n2, u), scale[r]);
        }
        Raw<T> o;
        pack_pairs<T>(v, o);
        store8<T>(static_cast<T*>(a.dx) + (t + r) * a.d, o, C, c);
      }
    }
  }
  float* part = a.part + (int64_t)blockIdx.x * 2 * a.d;
#pragma unroll
  for (int c = 0; c < NC; ++c)
    if (C.in(c, 0)) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        *reinterpret_cast<f2*>(part + C.col(c, 2 * i)) = dw[c][i];
        *reinterpret_cast<f2*>(part + a.d + C.col(c, 2 * i)) = db[c][i];
      }
    }
}

// dw and db partials by columns, for rows too long to keep their sums in
// registers: block (x, y) adds a range of rows for 256 columns.
template <typename T>
__global__ void __launch_bounds__(256) norm_dwdb_kernel(NormBwd a) {
  const int64_t col = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (col >= a.d) return;
  const int64_t per = (a.T + gridDim.y - 1) / gridDim.y;
  const int64_t t0 = blockIdx.y * per, t1 = t0 + per < a.T ? t0 + per : a.T;
  const T* x = static_cast<const T*>(a.x);
  const T* dy = static_cast<const T*>(a.dy);
  float dw = 0.f, db = 0.f;
#pragma unroll 4
  for (int64_t t = t0; t < t1; ++t) {
    const float g = (float)dy[t * a.d + col];
    const float m = a.rms ? 0.f : __ldg(a.mean + t);
    dw = fmaf(g, ((float)x[t * a.d + col] - m) * __ldg(a.rstd + t), dw);
    db += g;
  }
  float* part = a.part + (int64_t)blockIdx.y * 2 * a.d;
  part[col] = dw;
  part[a.d + col] = db;
}

// dw (blockIdx.y == 0) and db (1): X columns per block, partial rows y, y + 512 / X,
// ... per thread row, joined in a fixed order.  It is bound by the latency of a
// thread's loads, and by the number of blocks: 32 columns (a line) take 4.1 us after
// [8192, 4096] and 7.0 after [16384, 1024], where 64 blocks add 1184 rows; eight (a
// sector) 6.7 and 3.9.
template <typename WT, int X>
__global__ void __launch_bounds__(512) norm_reduce_kernel(const float* __restrict__ part, int parts, int64_t d, WT* dw,
                                                          WT* db) {
  __shared__ float sums[16][X + 1];
  WT* out = blockIdx.y ? db : dw;
  if (out == nullptr) return;
  const int x = threadIdx.x % X, y = threadIdx.x / X, lane = threadIdx.x & 31;
  const int64_t col = (int64_t)blockIdx.x * X + x;
  float s = 0.f;
  if (col < d) {
#pragma unroll 8
    for (int p = y; p < parts; p += 512 / X) s += part[(int64_t)p * 2 * d + blockIdx.y * d + col];
  }
#pragma unroll
  for (int off = X; off < 32; off *= 2) s += __shfl_xor_sync(0xffffffffu, s, off);
  if (lane < X) sums[threadIdx.x >> 5][x] = s;
  __syncthreads();
  if (threadIdx.x < X && col < d) {
    float total = 0.f;
#pragma unroll
    for (int q = 0; q < 16; ++q) total += sums[q][x];
    out[col] = round_to<WT>(total);
  }
}

// ----------------------------------------------------------------------------
// launch shapes
// ----------------------------------------------------------------------------

constexpr int kWarpTeams = 4;          // warps per CTA when a row belongs to a warp

int team_threads(int64_t d, int nc) { return (int)((d + 8 * nc * 32 - 1) / (8 * nc * 32) * 32); }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <class F>
cudaError_t by_types(int xt, int wt, F f) {
  if (xt == SK_F32) return f(float(), float());
  if (xt == SK_BF16) return wt == SK_F32 ? f(__nv_bfloat16(), float()) : f(__nv_bfloat16(), __nv_bfloat16());
  return wt == SK_F32 ? f(__half(), float()) : f(__half(), __half());
}

// Columns per access: the base pointers are 16-byte aligned, a row starts at a
// multiple of d values.  Single 16-bit values against pairs: 38.8 against 19.7 us
// forward at [2037, 4782].
template <class F>
cudaError_t by_width(int64_t d, F f) {
  if (d % 8 == 0) return f(std::integral_constant<int, 8>());
  if (d % 4 == 0) return f(std::integral_constant<int, 4>());
  if (d % 2 == 0) return f(std::integral_constant<int, 2>());
  return f(std::integral_constant<int, 1>());
}

// Shared memory of the ring: four stages where `ctas` CTAs of an SM have room for
// them, two at least (0: no room, the register kernels take such rows).
int ring_stages(size_t stage_bytes, int ctas) {
  const size_t room = (size_t)(220 << 10) / ctas;
  const size_t n = room / stage_bytes;
  return n < 2 ? 0 : n > kMaxStages ? kMaxStages : (int)n;
}

template <class Kern, class Args>
cudaError_t launch_ring(Kern kern, unsigned grid, int threads, size_t stage_bytes, const Ring& ring, const Args& a,
                        cudaStream_t s) {
  const size_t smem = stage_bytes * ring.stages;
  if (smem > (32 << 10)) {               // with the kernel's own arrays it may pass the default 48 KB
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  kern<<<grid, threads, smem, s>>>(a, ring);
  return cudaGetLastError();
}

// Two rows per CTA from eight rows per SM on: below that the rows are too few to
// fill the SMs, and one row per CTA with fewer columns per thread is sooner done
// (one row of 8192: 2.4 against 3.6 us).
bool pairs_of_rows(int64_t T, int64_t d) { return d > 512 && T >= 8 * (int64_t)num_sms(); }

template <typename T, typename WT, int V, bool CK>
cudaError_t fwd_shape(const NormFwd& a, cudaStream_t s) {
  const int64_t sms = num_sms();
  if constexpr (V == 8) {
    const int th = team_threads(a.d, pair_chunks<T>());
    if (th <= 1024 && pairs_of_rows(a.T, a.d)) {
      auto run = [&](auto kern) {
        kern<<<(unsigned)((a.T + 1) / 2), th, 0, s>>>(a);
        return cudaGetLastError();
      };
      // Rows that the threads cover exactly, nothing to check: 26.7 against 29.7 us at
      // [8192, 4096], and 30.2 against 34.3 at [4096, 5120] of a layer norm with a checkpoint.
      // An RMS norm with a checkpoint keeps the checks: without them the compiler moves more
      // ahead (121 registers against 94: three CTAs of 160 threads per SM instead of four, 26.1
      // against 24.0 us at [4096, 5120]) and gains a little elsewhere (18.5 against 18.9 at [4096, 4096], 21.5
      // against 22.4 at [2048, 8192], 36.0 against 38.1 at [4096, 7168]).
      const bool full = a.d == (int64_t)th * 8 * pair_chunks<T>();
      auto shape = [&](auto rms, auto bias) {
        constexpr bool RMS = decltype(rms)::value, BIAS = decltype(bias)::value;
        if constexpr (!(CK && RMS)) {
          if (th <= 128 && full) return run(norm_fwd_pair_kernel<T, WT, 128, 5, RMS, BIAS, CK, true>);
          if (th <= 256 && full) return run(norm_fwd_pair_kernel<T, WT, 256, 2, RMS, BIAS, CK, true>);
        }
        if (th <= 128) return run(norm_fwd_pair_kernel<T, WT, 128, 5, RMS, BIAS, CK, false>);
        if (th <= 256) return run(norm_fwd_pair_kernel<T, WT, 256, 2, RMS, BIAS, CK, false>);
        return run(norm_fwd_pair_kernel<T, WT, 1024, 1, RMS, BIAS, CK, false>);
      };
      const std::true_type yes;
      const std::false_type no;
      return a.rms ? (a.b ? shape(yes, yes) : shape(yes, no)) : (a.b ? shape(no, yes) : shape(no, no));
    }
  }
  auto go = [&](auto kern, int threads, int64_t rows_per_cta, int64_t ctas_per_sm) {
    int64_t grid = (a.T + rows_per_cta - 1) / rows_per_cta;
    if (grid > sms * ctas_per_sm) grid = sms * ctas_per_sm;
    kern<<<(unsigned)grid, threads, 0, s>>>(a);
    return cudaGetLastError();
  };
  if (a.d <= 256) return go(norm_fwd_kernel<T, WT, 1, 128, V, true, CK>, 128, kWarpTeams, 16);
  if (a.d <= 512) return go(norm_fwd_kernel<T, WT, 2, 128, V, true, CK>, 128, kWarpTeams, 8);
  if (a.d <= 16384) {
    const int th = team_threads(a.d, 2);
    if (th <= 256) return go(norm_fwd_kernel<T, WT, 2, 256, V, false, CK>, th, 1, 768 / th);
    if (th <= 512) return go(norm_fwd_kernel<T, WT, 2, 512, V, false, CK>, th, 1, 1024 / th);
    return go(norm_fwd_kernel<T, WT, 2, 1024, V, false, CK>, th, 1, 1);
  }
  return go(norm_fwd_kernel<T, WT, 4, 1024, V, false, CK>, team_threads(a.d, 4), 1, 1);
}

}  // namespace

cudaError_t launch_norm_fwd(const NormFwd& a, cudaStream_t s) {
  return by_types(a.xtype, a.wtype, [&](auto xt, auto wt) {
    using T = decltype(xt);
    using WT = decltype(wt);
    if constexpr (std::is_same<T, __nv_bfloat16>::value)
      if (a.q != nullptr) return fwd_shape<T, WT, 8, true>(a, s);
    return by_width(a.d, [&](auto v) { return fwd_shape<T, WT, decltype(v)::value, false>(a, s); });
  });
}

// Longest row whose dw and db sums stay in registers (32 threads x 8 columns x
// 2 chunks x 16 warps); longer rows take a second kernel that reads x and dy again.
constexpr int64_t kFusedDw = 8192;

// Partial rows of dw and db.  At least four rows per team, so that the partials
// (8 bytes per column and team) stay below the rows' own traffic.
int norm_bwd_parts(int64_t T, int64_t d) {
  const int64_t sms = num_sms();
  int64_t cap, rows;
  if (d <= 512) {
    cap = sms * 4;
    rows = 4 * kWarpTeams;
  } else if (d <= kFusedDw) {
    const int th = team_threads(d, 2);
    cap = sms * (th <= 512 ? 512 / th : 1);
    rows = 4;
  } else {
    cap = 64;
    rows = 32;
  }
  const int64_t want = (T + rows - 1) / rows;
  return (int)(want < 1 ? 1 : want < cap ? want : cap);
}

namespace {

template <typename T, typename WT, int V>
cudaError_t bwd_shape(const NormBwd& a, cudaStream_t s) {
  const bool dw = a.dw != nullptr || a.db != nullptr;
  const int parts = norm_bwd_parts(a.T, a.d);
  const int64_t sms = num_sms();
  cudaError_t e;
  auto check = [&] { return cudaGetLastError(); };
  bool done = false;                   // dx and, up to kFusedDw, the partials of dw and db
  if constexpr (V == 8) {
    const int th = team_threads(a.d, 2);
    const int ctas = th <= 512 ? 512 / th : 1;
    const size_t row = (size_t)a.d * sizeof(T);
    const int stages = a.d <= kFusedDw ? ring_stages(4 * row, ctas) : 0;
    const int dx_th = team_threads(a.d, pair_chunks<T>());
    if (dw && stages >= 2 && pairs_of_rows(a.T, a.d) && parts == sms * ctas) {
      const Ring ring{stages, (uint32_t)row};
      auto run = [&](auto rms) {
        constexpr bool RMS = decltype(rms)::value;
        const bool full = a.d == (int64_t)th * 16;
        auto go = [&](auto kern) { return launch_ring(kern, (unsigned)parts, th, 4 * row, ring, a, s); };
        if (th <= 256 && full) return go(norm_bwd_ring_kernel<T, WT, 256, 2, RMS, true>);
        if (th <= 256) return go(norm_bwd_ring_kernel<T, WT, 256, 2, RMS, false>);
        if (full) return go(norm_bwd_ring_kernel<T, WT, 512, 1, RMS, true>);
        return go(norm_bwd_ring_kernel<T, WT, 512, 1, RMS, false>);
      };
      e = a.rms ? run(std::true_type()) : run(std::false_type());
      if (e != cudaSuccess) return e;
      done = true;
    } else if (!dw && dx_th <= 1024 && pairs_of_rows(a.T, a.d)) {
      auto run = [&](auto kern) {
        kern<<<(unsigned)((a.T + 1) / 2), dx_th, 0, s>>>(a);
        return cudaGetLastError();
      };
      auto shape = [&](auto rms) {
        constexpr bool RMS = decltype(rms)::value;
        const bool full = a.d == (int64_t)dx_th * 8 * pair_chunks<T>();
        if (dx_th <= 128 && full) return run(norm_dx_pair_kernel<T, WT, 128, 4, RMS, true>);
        if (dx_th <= 128) return run(norm_dx_pair_kernel<T, WT, 128, 4, RMS, false>);
        if (dx_th <= 256 && full) return run(norm_dx_pair_kernel<T, WT, 256, 2, RMS, true>);
        if (dx_th <= 256) return run(norm_dx_pair_kernel<T, WT, 256, 2, RMS, false>);
        // 128 registers: at 64 dx spills (79 against 44 us at [2048, 16384] bf16), while the
        // forward pass gains more from a second CTA (26 against 34 us)
        if (dx_th <= 512) return run(norm_dx_pair_kernel<T, WT, 512, 1, RMS, false>);
        return run(norm_dx_pair_kernel<T, WT, 1024, 1, RMS, false>);
      };
      return a.rms ? shape(std::true_type()) : shape(std::false_type());
    }
  }
  if (done) {
  } else if (dw && a.d <= kFusedDw) {
    if (a.d <= 256)
      norm_bwd_kernel<T, WT, 1, 128, V, true, true><<<parts, 128, kWarpTeams * 2 * 256 * 4, s>>>(a);
    else if (a.d <= 512)
      norm_bwd_kernel<T, WT, 2, 128, V, true, true><<<parts, 128, kWarpTeams * 2 * 512 * 4, s>>>(a);
    else if (team_threads(a.d, 2) <= 256)
      norm_bwd_kernel<T, WT, 2, 256, V, false, true><<<parts, team_threads(a.d, 2), 0, s>>>(a);
    else
      norm_bwd_kernel<T, WT, 2, 512, V, false, true><<<parts, team_threads(a.d, 2), 0, s>>>(a);
    e = check();
    if (e != cudaSuccess) return e;
  } else {
    if (a.dx != nullptr) {
      if (a.d <= 512) {
        int64_t grid = (a.T + kWarpTeams - 1) / kWarpTeams;
        if (grid > sms * 8) grid = sms * 8;
        norm_bwd_kernel<T, WT, 2, 128, V, true, false><<<(unsigned)grid, 128, 0, s>>>(a);
      } else if (a.d <= 16384) {
        const int th = team_threads(a.d, 2);
        const int64_t per_sm = th < 768 ? 768 / th : 1;
        const unsigned grid = (unsigned)(a.T < sms * per_sm ? a.T : sms * per_sm);
        if (th <= 256) norm_bwd_kernel<T, WT, 2, 256, V, false, false><<<grid, th, 0, s>>>(a);
        else if (th <= 512) norm_bwd_kernel<T, WT, 2, 512, V, false, false><<<grid, th, 0, s>>>(a);
        else norm_bwd_kernel<T, WT, 2, 1024, V, false, false><<<grid, th, 0, s>>>(a);
      } else {
        const unsigned grid = (unsigned)(a.T < sms ? a.T : sms);
        norm_bwd_kernel<T, WT, 4, 1024, V, false, false><<<grid, team_threads(a.d, 4), 0, s>>>(a);
      }
      e = check();
      if (e != cudaSuccess) return e;
    }
    if (!dw) return cudaSuccess;
    norm_dwdb_kernel<T><<<dim3((unsigned)((a.d + 255) / 256), parts), 256, 0, s>>>(a);
    e = check();
    if (e != cudaSuccess) return e;
  }
  WT *out_w = static_cast<WT*>(a.dw), *out_b = static_cast<WT*>(a.db);
  if (a.d < 16 * sms && parts >= 320)          // lines would make fewer blocks than SMs, with many rows each
    norm_reduce_kernel<WT, 8><<<dim3((unsigned)((a.d + 7) / 8), 2), 512, 0, s>>>(a.part, parts, a.d, out_w, out_b);
  else
    norm_reduce_kernel<WT, 32><<<dim3((unsigned)((a.d + 31) / 32), 2), 512, 0, s>>>(a.part, parts, a.d, out_w, out_b);
  return check();
}

}  // namespace

cudaError_t launch_norm_bwd(const NormBwd& a, cudaStream_t s) {
  return by_types(a.xtype, a.wtype, [&](auto xt, auto wt) {
    using T = decltype(xt);
    using WT = decltype(wt);
    return by_width(a.d, [&](auto v) { return bwd_shape<T, WT, decltype(v)::value>(a, s); });
  });
}

}  // namespace sk
