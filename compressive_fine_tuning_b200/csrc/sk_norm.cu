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
// is far larger than its spread loses nothing.
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

// A team's view of a row: chunk c of member `me` of `team` holds eight columns.
// VEC: eight consecutive ones (16-byte accesses; d % 8 == 0 and aligned rows),
// else columns `team` apart (any d).
template <bool VEC>
struct Cols {
  int me, team, d;
  __device__ __forceinline__ int col(int c, int k) const {
    return VEC ? (c * team + me) * 8 + k : (c * 8 + k) * team + me;
  }
  __device__ __forceinline__ bool in(int c, int k) const { return col(c, VEC ? 0 : k) < d; }
};

template <typename T, bool VEC>
__device__ __forceinline__ void load8(Raw<T>& r, const T* __restrict__ row, const Cols<VEC>& C, int c) {
  if constexpr (VEC) {
    if (C.in(c, 0)) {
      const uint4* p = reinterpret_cast<const uint4*>(row + C.col(c, 0));
#pragma unroll
      for (int q = 0; q < Raw<T>::NW / 4; ++q) {
        const uint4 v = __ldg(p + q);
        r.w[4 * q] = v.x; r.w[4 * q + 1] = v.y; r.w[4 * q + 2] = v.z; r.w[4 * q + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int q = 0; q < Raw<T>::NW; ++q) r.w[q] = 0u;
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

template <typename T, bool VEC>
__device__ __forceinline__ void store8(T* __restrict__ row, const Raw<T>& r, const Cols<VEC>& C, int c) {
  if constexpr (VEC) {
    if (C.in(c, 0)) {
      uint4* p = reinterpret_cast<uint4*>(row + C.col(c, 0));
#pragma unroll
      for (int q = 0; q < Raw<T>::NW / 4; ++q)
        p[q] = make_uint4(r.w[4 * q], r.w[4 * q + 1], r.w[4 * q + 2], r.w[4 * q + 3]);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (!C.in(c, k)) continue;
      if constexpr (sizeof(T) == 4) {
        reinterpret_cast<uint32_t*>(row)[C.col(c, k)] = r.w[k];
      } else {
        reinterpret_cast<uint16_t*>(row)[C.col(c, k)] = (uint16_t)(r.w[k >> 1] >> (16 * (k & 1)));
      }
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

// ----------------------------------------------------------------------------
// forward
// ----------------------------------------------------------------------------

template <typename T, typename WT, int NC, int MAXT, bool VEC, bool WARP, bool CK>
__global__ void __launch_bounds__(MAXT) norm_fwd_kernel(NormFwd a) {
  __shared__ float buf[2][32];
  const int lane = threadIdx.x & 31;
  const Cols<VEC> C{WARP ? lane : (int)threadIdx.x, WARP ? 32 : (int)blockDim.x, (int)a.d};
  const int64_t teams = WARP ? (int64_t)gridDim.x * (blockDim.x >> 5) : gridDim.x;
  int64_t t = WARP ? (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
  const T* x = static_cast<const T*>(a.x);
  Raw<WT> w[NC], b[NC];
  Raw<T> cur[NC], nxt[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    if (t < a.T) load8<T, VEC>(cur[c], x + t * a.d, C, c);
    load8<WT, VEC>(w[c], static_cast<const WT*>(a.w), C, c);
    if (a.b != nullptr) load8<WT, VEC>(b[c], static_cast<const WT*>(a.b), C, c);
  }
  const float inv_d = 1.f / (float)a.d;
  // Buffers of the sums: a layer norm's two sums take turns; an RMS norm's only
  // sum changes buffers from row to row.
  int second = 1;
  for (; t < a.T; t += teams) {
    const bool more = t + teams < a.T;
#pragma unroll
    for (int c = 0; c < NC; ++c)
      if (more) load8<T, VEC>(nxt[c], x + (t + teams) * a.d, C, c);
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
      store8<T, VEC>(static_cast<T*>(a.y) + t * a.d, o, C, c);
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
template <typename T, typename WT, int NC, int MAXT, bool VEC, bool WARP, bool DW>
__global__ void __launch_bounds__(MAXT) norm_bwd_kernel(NormBwd a) {
  extern __shared__ float wpart[];                 // WARP with DW: [warps][2][NC * 256]
  __shared__ float2 buf[2][32];
  const int lane = threadIdx.x & 31;
  const Cols<VEC> C{WARP ? lane : (int)threadIdx.x, WARP ? 32 : (int)blockDim.x, (int)a.d};
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
      load8<T, VEC>(rx[c], x + row * a.d, C, c);
      load8<T, VEC>(rd[c], dy + row * a.d, C, c);
    }
    m = a.rms ? 0.f : __ldg(a.mean + row);
    rs = __ldg(a.rstd + row);
  };
  if (t < a.T) fetch(t, cx, cd, mu, r);
#pragma unroll
  for (int c = 0; c < NC; ++c) load8<WT, VEC>(w[c], static_cast<const WT*>(a.w), C, c);
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
        store8<T, VEC>(static_cast<T*>(a.dx) + t * a.d, o, C, c);
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

// dw (blockIdx.y == 0) and db (1): 32 columns per block, partial rows y, y + 16,
// ... per thread row, then the sixteen sums in order.
template <typename WT>
__global__ void __launch_bounds__(512) norm_reduce_kernel(const float* __restrict__ part, int parts, int64_t d, WT* dw,
                                                          WT* db) {
  __shared__ float sums[16][33];
  WT* out = blockIdx.y ? db : dw;
  if (out == nullptr) return;
  const int64_t col = (int64_t)blockIdx.x * 32 + threadIdx.x;
  float s = 0.f;
  if (col < d) {
#pragma unroll 8
    for (int p = threadIdx.y; p < parts; p += 16) s += part[(int64_t)p * 2 * d + blockIdx.y * d + col];
  }
  sums[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0 && col < d) {
    float total = 0.f;
#pragma unroll
    for (int q = 0; q < 16; ++q) total += sums[q][threadIdx.x];
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

template <typename T, typename WT, bool VEC, bool CK>
cudaError_t fwd_shape(const NormFwd& a, cudaStream_t s) {
  const int64_t sms = num_sms();
  auto go = [&](auto kern, int threads, int64_t rows_per_cta, int64_t ctas_per_sm) {
    int64_t grid = (a.T + rows_per_cta - 1) / rows_per_cta;
    if (grid > sms * ctas_per_sm) grid = sms * ctas_per_sm;
    kern<<<(unsigned)grid, threads, 0, s>>>(a);
    return cudaGetLastError();
  };
  if (a.d <= 256) return go(norm_fwd_kernel<T, WT, 1, 128, VEC, true, CK>, 128, kWarpTeams, 16);
  if (a.d <= 512) return go(norm_fwd_kernel<T, WT, 2, 128, VEC, true, CK>, 128, kWarpTeams, 8);
  if (a.d <= 16384) {
    const int th = team_threads(a.d, 2);
    if (th <= 256) return go(norm_fwd_kernel<T, WT, 2, 256, VEC, false, CK>, th, 1, 768 / th);
    if (th <= 512) return go(norm_fwd_kernel<T, WT, 2, 512, VEC, false, CK>, th, 1, 1024 / th);
    return go(norm_fwd_kernel<T, WT, 2, 1024, VEC, false, CK>, th, 1, 1);
  }
  return go(norm_fwd_kernel<T, WT, 4, 1024, VEC, false, CK>, team_threads(a.d, 4), 1, 1);
}

}  // namespace

cudaError_t launch_norm_fwd(const NormFwd& a, cudaStream_t s) {
  const bool vec = a.d % 8 == 0;       // the rows are 16-byte aligned then (the base pointers are)
  return by_types(a.xtype, a.wtype, [&](auto xt, auto wt) {
    using T = decltype(xt);
    using WT = decltype(wt);
    if constexpr (sizeof(T) == 2 && std::is_same<T, __nv_bfloat16>::value)
      if (a.q != nullptr) return fwd_shape<T, WT, true, true>(a, s);
    return vec ? fwd_shape<T, WT, true, false>(a, s) : fwd_shape<T, WT, false, false>(a, s);
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

template <typename T, typename WT, bool VEC>
cudaError_t bwd_shape(const NormBwd& a, cudaStream_t s) {
  const bool dw = a.dw != nullptr || a.db != nullptr;
  const int parts = norm_bwd_parts(a.T, a.d);
  const int64_t sms = num_sms();
  cudaError_t e;
  auto check = [&] { return cudaGetLastError(); };
  if (dw && a.d <= kFusedDw) {
    if (a.d <= 256)
      norm_bwd_kernel<T, WT, 1, 128, VEC, true, true><<<parts, 128, kWarpTeams * 2 * 256 * 4, s>>>(a);
    else if (a.d <= 512)
      norm_bwd_kernel<T, WT, 2, 128, VEC, true, true><<<parts, 128, kWarpTeams * 2 * 512 * 4, s>>>(a);
    else if (team_threads(a.d, 2) <= 256)
      norm_bwd_kernel<T, WT, 2, 256, VEC, false, true><<<parts, team_threads(a.d, 2), 0, s>>>(a);
    else
      norm_bwd_kernel<T, WT, 2, 512, VEC, false, true><<<parts, team_threads(a.d, 2), 0, s>>>(a);
    e = check();
    if (e != cudaSuccess) return e;
  } else {
    if (a.dx != nullptr) {
      if (a.d <= 512) {
        int64_t grid = (a.T + kWarpTeams - 1) / kWarpTeams;
        if (grid > sms * 8) grid = sms * 8;
        norm_bwd_kernel<T, WT, 2, 128, VEC, true, false><<<(unsigned)grid, 128, 0, s>>>(a);
      } else if (a.d <= 16384) {
        const int th = team_threads(a.d, 2);
        const int64_t per_sm = th < 768 ? 768 / th : 1;
        const unsigned grid = (unsigned)(a.T < sms * per_sm ? a.T : sms * per_sm);
        if (th <= 256) norm_bwd_kernel<T, WT, 2, 256, VEC, false, false><<<grid, th, 0, s>>>(a);
        else if (th <= 512) norm_bwd_kernel<T, WT, 2, 512, VEC, false, false><<<grid, th, 0, s>>>(a);
        else norm_bwd_kernel<T, WT, 2, 1024, VEC, false, false><<<grid, th, 0, s>>>(a);
      } else {
        const unsigned grid = (unsigned)(a.T < sms ? a.T : sms);
        norm_bwd_kernel<T, WT, 4, 1024, VEC, false, false><<<grid, team_threads(a.d, 4), 0, s>>>(a);
      }
      e = check();
      if (e != cudaSuccess) return e;
    }
    if (!dw) return cudaSuccess;
    norm_dwdb_kernel<T><<<dim3((unsigned)((a.d + 255) / 256), parts), 256, 0, s>>>(a);
    e = check();
    if (e != cudaSuccess) return e;
  }
  norm_reduce_kernel<WT><<<dim3((unsigned)((a.d + 31) / 32), 2), dim3(32, 16), 0, s>>>(
      a.part, parts, a.d, static_cast<WT*>(a.dw), static_cast<WT*>(a.db));
  return check();
}

}  // namespace

cudaError_t launch_norm_bwd(const NormBwd& a, cudaStream_t s) {
  const bool vec = a.d % 8 == 0;
  return by_types(a.xtype, a.wtype, [&](auto xt, auto wt) {
    using T = decltype(xt);
    using WT = decltype(wt);
    return vec ? bwd_shape<T, WT, true>(a, s) : bwd_shape<T, WT, false>(a, s);
  });
}

}  // namespace sk
