// Linear cross entropy: the head product, softmax cross entropy over the
// vocabulary and its gradients, without a [T][V] tensor of logits.
//
//   l = H W^T,  lse_t = log sum_v exp(l_tv),  loss_t = lse_t - l_t,target
//   P = c_t (softmax(l_t) - onehot(target)),  dH = P W,  dW = P^T H
//
// (c is taken apart into one number per chunk of tokens, which multiplies the
// products' fp32 sums, and P's own part: 1 of a reduced loss, the weight over the
// chunk's largest of per-token losses).
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
// and is held in fp16 times 2^15: off by 2^-11 of the value down to 2^-29 of the
// tile's maximum, by 2^-40 of that maximum below.  (Without the factor fp16's full
// precision ends at 2^-14: next to a surely predicted target a class 16 below it in
// the same tile was 6 % off, one 18 below it lost.)  P is rounded to bf16 for the
// products (2^-8 of each value at most).  The target's entry does not come
// from the buffer: p - 1 is formed from the fp32 loss as expm1(-loss), so a
// token that is already predicted surely keeps its small gradient's precision, down
// to the 2^-24 that a sum of exponentials next to 1 is rounded to.  What its bf16 rounding takes off is given back in dH, whose rows have one target
// each; in dW, where any number of tokens share a row, it stays (1e-3 of dW at 8192
// tokens and 32000 classes, where rounding dW to bf16 takes 1.7e-3).  A factor that
// tokens share is kept out of that rounding: 1 / 8160 in P, halfway between two bf16
// values, moved all of dW by 2^-8.
//
// The bound is the tensor pipe: 2 T V d flops per product.
#include <type_traits>

#include "sk_gemm.cuh"
#include "sk_loss.cuh"

namespace sk {
namespace {

constexpr int64_t kExpBytes = int64_t(512) << 20;   // buffer of one chunk's exponentials
constexpr int64_t kLossChunk = 32768;               // tokens per launch when only the loss is wanted
constexpr int kScoreTokens = 64;                    // tokens up to which a loss alone exchanges the product's sides
constexpr int kMinRows = 64;                        // fewest classes per CTA there
constexpr int kMinTile = 128;                       // fewest classes per tile of a loss without gradients
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kExpScale = 32768.f;                // of the exponentials in fp16

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

// Join (maximum, sum of exponentials) pairs.  fmaxf drops a NaN maximum, but a
// tile with a NaN logit has a NaN sum, which stays.
__device__ __forceinline__ void join_stats(float& m, float& s, float m2, float s2) {
  const float top = fmaxf(m, m2);
  const float base = top == -INFINITY ? 0.f : top;
  s = s * expf(m - base) + s2 * expf(m2 - base);
  m = top;
}

// ----------------------------------------------------------------------------
// logits: tile statistics, the target's logit, and the exponentials
// ----------------------------------------------------------------------------

struct LogitEpi {
  static constexpr int kTeam = 1;
  const CUtensorMap* tm_e;
  float2* stats;            // [tiles of V][T]: (maximum, sum of exp(l - maximum))
  float* target_logit;      // [T]
  const void* target;
  int target64;
  int64_t ignore_index;
  int T, V, tn;             // tokens of the chunk, classes, classes per tile
  bool store;
  unsigned int* check;
  gemm::SlabWriter out;

  __device__ __forceinline__ void start(int, int, uint8_t*) {}
  __device__ __forceinline__ void ready(const gemm::Item&, int, int, int, int) {}
  __device__ __forceinline__ void take() {}
  __device__ __forceinline__ void done(int lane) { out.drain(lane); }
  __device__ __forceinline__ void tile(uint32_t tmem, int m0, int n0, const gemm::Item&, int warp, int lane,
                                       uint8_t* scratch) {
    const int t = m0 + 32 * warp + lane;
    if (m0 + 32 * warp >= T) return;
    const int cols = min(tn, V - n0);
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
          const __half2 hh = __floats2half2_rn(a * kExpScale, b * kExpScale);
          e[16 * q + (j >> 1)] = *reinterpret_cast<const uint32_t*>(&hh);
        }
        sum += part;
      }
      if (store) out.put(scratch, tm_e, e, n0 + 64 * h, m0 + 32 * warp, warp, lane);
    }
    if (t < T) stats[(int64_t)(n0 / tn) * T + t] = make_float2(m, sum);
  }
};

// What a chunk's kernels share besides arrays: zeroed by the logit kernel, which
// runs before the others.
struct Shared {
  unsigned long long count;   // tokens that take part
  unsigned int blocks;        // blocks of lse_kernel that are done
  unsigned int dirty;         // a token that takes no part has a NaN or an infinity in its row of H
  unsigned int top;           // fp32 bits of the largest weight of a token that takes part (per-token losses)
};

// The shared part of per-token weights.
__device__ __forceinline__ float top_weight(const Shared* s) { return s->top != 0 ? __uint_as_float(s->top) : 1.f; }

__device__ __forceinline__ void start_chunk(Shared* s, int keep_count) {
  if (blockIdx.x != 0 || threadIdx.x != 0) return;
  s->blocks = 0;
  s->dirty = 0;
  s->top = 0;
  if (!keep_count) s->count = 0;
}

struct LogitArgs {
  gemm::Shape shape;
  float2* stats;
  float* target_logit;
  const void* target;
  int target64;
  int64_t ignore_index;
  int T, V, store;
  Shared* shared;
  int keep_count;             // an earlier kernel has counted all chunks' tokens
  unsigned int* check;
};

__global__ void __launch_bounds__(gemm::threads(4), 1)
logit_kernel(const __grid_constant__ CUtensorMap tm_h, const __grid_constant__ CUtensorMap tm_w,
             const __grid_constant__ CUtensorMap tm_e, LogitArgs a) {
  start_chunk(a.shared, a.keep_count);
  LogitEpi epi{&tm_e, a.stats, a.target_logit, a.target, a.target64, a.ignore_index, a.T, a.V, a.shape.tn,
               a.store != 0, a.check, {}};
  gemm::run<0, 0, 4, 6>(&tm_h, &tm_w, gemm::Plan{a.shape}, epi, a.check);
}

// The loss alone of a few tokens: the product with its sides exchanged (M = classes,
// N = the tokens, 32 or 64 of them), since a 256-row tile of tokens would spend
// the tensor pipe on rows that do not exist and no longer keep up with reading W.
// An accumulator row is then a class, so a warp turns its 32 x 32 blocks over in
// shared memory, a lane takes one token's 32 classes, and the CTA's four warps join
// their pairs: one (maximum, sum) per token and CTA tile of `rows` classes.
struct ScoreEpi {
  static constexpr int kTeam = 4;
  float2* stats;            // [CTA tiles][T]
  float* target_logit;      // [T]
  const void* target;
  int target64;
  int64_t ignore_index;
  int T, V, rows;
  unsigned int* check;

  __device__ __forceinline__ void start(int, int, uint8_t*) {}
  __device__ __forceinline__ void ready(const gemm::Item&, int, int, int, int) {}
  __device__ __forceinline__ void take() {}
  __device__ __forceinline__ void done(int) {}
  __device__ __forceinline__ void tile(uint32_t tmem, int m0, int, const gemm::Item&, int warp, int lane,
                                       uint8_t* scratch) {
    float* block = reinterpret_cast<float*>(scratch) + warp * 32 * 33;             // [class][token], padded
    float2* pairs = reinterpret_cast<float2*>(scratch + 4 * 32 * 33 * sizeof(float));   // [warp][kScoreTokens]
    const int c0 = m0 + 32 * warp, classes = min(32, min(rows - 32 * warp, V - c0));
    for (int q = 0; 32 * q < T; ++q) {
      uint32_t v[32];
      tc::tmem_ld32(tmem + 32 * q, v);
      tc::tmem_ld_wait();
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 32; ++j) block[lane * 33 + j] = __uint_as_float(v[j]);
      __syncwarp();
      const int t = 32 * q + lane;
      float m = -INFINITY, s = 0.f;
      for (int c = 0; c < classes; ++c) m = fmaxf(m, block[c * 33 + lane]);
      const float base = m == -INFINITY ? 0.f : m;
      for (int c = 0; c < classes; ++c) s += fast_exp2((block[c * 33 + lane] - base) * kLog2e);
      pairs[warp * kScoreTokens + t] = make_float2(m, s);
      if (t < T) {
        const int64_t y = class_of(target, target64, t, V, ignore_index, check);
        if (y >= c0 && y < c0 + classes) target_logit[t] = block[(int)(y - c0) * 33 + lane];
      }
    }
    tc::named_bar_sync(1, 128);
    const int t = 32 * warp + lane;
    if (t < T) {                                       // a CTA beyond the last class: (-inf, 0)
      float2 p = pairs[t];
#pragma unroll
      for (int w = 1; w < 4; ++w) {
        const float2 o = pairs[w * kScoreTokens + t];
        join_stats(p.x, p.y, o.x, o.y);
      }
      stats[(int64_t)(m0 / rows) * T + t] = p;
    }
    tc::named_bar_sync(1, 128);
  }
};

// The exchanged product with its exponentials, for a number of tokens that 256-row
// tiles of tokens would pad by much: here a tile takes as many tokens as is best (a
// multiple of 32).  Blocks of 32 x 32 turn over in shared memory as above, once for
// the tile's maxima (over the CTA's 128 classes), which the warps then share, and
// once for the exponentials: a lane writes its token's 32 classes, 64 bytes.
struct LogitTEpi {
  static constexpr int kTeam = 4;
  uint16_t* E;              // [T][pitch] fp16
  int64_t pitch;
  float2* stats;            // [CTA tiles of 128 classes][T]
  float* target_logit;      // [T]
  const void* target;
  int target64;
  int64_t ignore_index;
  int T, V, tn;
  unsigned int* check;

  __device__ __forceinline__ void start(int, int, uint8_t*) {}
  __device__ __forceinline__ void ready(const gemm::Item&, int, int, int, int) {}
  __device__ __forceinline__ void take() {}
  __device__ __forceinline__ void done(int) {}
  __device__ __forceinline__ void tile(uint32_t tmem, int m0, int n0, const gemm::Item&, int warp, int lane,
                                       uint8_t* scratch) {
    float* block = reinterpret_cast<float*>(scratch) + warp * 32 * 33;                     // [class][token], padded
    float* maxima = reinterpret_cast<float*>(scratch + 4 * 32 * 33 * sizeof(float));       // [warp][256 tokens]
    float* sums = maxima + 4 * 256;
    const int c0 = m0 + 32 * warp, classes = min(32, V - c0), tokens = min(tn, T - n0);
    auto turn = [&](int q) {
      uint32_t v[32];
      tc::tmem_ld32(tmem + 32 * q, v);
      tc::tmem_ld_wait();
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 32; ++j) block[lane * 33 + j] = __uint_as_float(v[j]);
      __syncwarp();
    };
#pragma unroll 1
    for (int q = 0; 32 * q < tokens; ++q) {
      turn(q);
      float m = -INFINITY;
      for (int c = 0; c < classes; ++c) m = fmaxf(m, block[c * 33 + lane]);
      maxima[warp * 256 + 32 * q + lane] = m;
    }
    tc::named_bar_sync(1, 128);
#pragma unroll 1
    for (int q = 0; 32 * q < tokens; ++q) {
      turn(q);
      const int k = 32 * q + lane, t = n0 + k;
      const float m = fmaxf(fmaxf(maxima[k], maxima[256 + k]), fmaxf(maxima[512 + k], maxima[768 + k]));
      const float base = m == -INFINITY ? 0.f : m;
      float s = 0.f;
      uint4* out = reinterpret_cast<uint4*>(E + (int64_t)t * pitch + c0);
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        if (8 * g >= classes) break;                  // the pitch covers whole groups of eight
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = 8 * g + 2 * i;
          const float a = c < classes ? fast_exp2((block[c * 33 + lane] - base) * kLog2e) : 0.f;
          const float b = c + 1 < classes ? fast_exp2((block[(c + 1) * 33 + lane] - base) * kLog2e) : 0.f;
          s += a;
          s += b;
          const __half2 hh = __floats2half2_rn(a * kExpScale, b * kExpScale);
          w[i] = *reinterpret_cast<const uint32_t*>(&hh);
        }
        if (k < tokens) out[g] = make_uint4(w[0], w[1], w[2], w[3]);
      }
      sums[warp * 256 + k] = s;
      if (k < tokens) {
        const int64_t y = class_of(target, target64, t, V, ignore_index, check);
        if (y >= c0 && y < c0 + classes) target_logit[t] = block[(int)(y - c0) * 33 + lane];
      }
    }
    tc::named_bar_sync(1, 128);
    for (int k = 32 * warp + lane; k < tokens && m0 < V; k += 128) {
      const float m = fmaxf(fmaxf(maxima[k], maxima[256 + k]), fmaxf(maxima[512 + k], maxima[768 + k]));
      stats[(int64_t)(m0 / 128) * T + n0 + k] = make_float2(m, (sums[k] + sums[256 + k]) + (sums[512 + k] + sums[768 + k]));
    }
    tc::named_bar_sync(1, 128);
  }
};

__global__ void __launch_bounds__(gemm::threads(4), 1)
logit_t_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_h, LogitArgs a, uint16_t* E,
               int64_t pitch) {
  start_chunk(a.shared, a.keep_count);
  LogitTEpi epi{E, pitch, a.stats, a.target_logit, a.target, a.target64, a.ignore_index, a.T, a.V, a.shape.tn, a.check};
  gemm::run<0, 0, 4, 6>(&tm_w, &tm_h, gemm::Plan{a.shape}, epi, a.check);
}

__global__ void __launch_bounds__(gemm::threads(4), 1)
score_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_h, LogitArgs a) {
  start_chunk(a.shared, a.keep_count);
  ScoreEpi epi{a.stats, a.target_logit, a.target, a.target64, a.ignore_index, a.T, a.V, a.shape.a_rows, a.check};
  gemm::run<0, 0, 4, 6>(&tm_w, &tm_h, gemm::Plan{a.shape}, epi, a.check);
}

// ----------------------------------------------------------------------------
// dH and dW
// ----------------------------------------------------------------------------

// What dH's rows still need: P's entry at the target, the largest of the row for
// most tokens, enters the product as bf16; what that rounding took off comes
// back here, times the target's row of W, in fp32.
struct TargetRest {
  const float* rest;        // [T] fp32 minus bf16 of P's target entry, or nullptr
  const uint16_t* W;
  const void* target;
  int target64;
  int64_t V, d, ignore_index;

  __device__ __forceinline__ const uint16_t* row(int64_t t, float& r, unsigned int* check) const {
    r = 0.f;
    if (rest == nullptr) return nullptr;
    const int64_t y = class_of(target, target64, t, V, ignore_index, check);
    if (y < 0) return nullptr;
    r = rest[t];
    return W + y * d;
  }
};

__device__ __forceinline__ void add_scaled8(float (&f)[8], const uint16_t* w, float r) {
  const uint4 v = __ldg(reinterpret_cast<const uint4*>(w));
  const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    f[2 * q] = fmaf(r, __uint_as_float(x[q] << 16), f[2 * q]);
    f[2 * q + 1] = fmaf(r, __uint_as_float(x[q] & 0xffff0000u), f[2 * q + 1]);
  }
}

// Where a gradient product's values go: bf16, or, for a dW that several chunks of
// tokens add up to, fp32 sums in memory (`acc`): read when `add`, written back as
// fp32 unless this is the last chunk, which writes bf16.
struct GradOut {
  float* acc;
  int add, last;
  int64_t M, N;
  TargetRest rest;
  const float* dloss;       // the factor of a reduced loss, or nullptr (one)
  const Shared* count;      // divide by its count (mean), or nullptr
  const Shared* top;        // the factor of per-token losses with weights, or nullptr

  // What the products' sums are multiplied by: 0 for dH's rows of tokens that take no
  // part, whatever the factor is.
  __device__ __forceinline__ float scale(const uint16_t* wrow) const {
    if (rest.rest != nullptr && wrow == nullptr) return 0.f;
    if (top != nullptr) return top_weight(top);
    const float c = dloss != nullptr ? __ldg(dloss) : 1.f;
    return count != nullptr ? c / (float)(count->count > 0 ? count->count : 1) : c;
  }

  // eight columns of a row (N % 8 == 0: inside or outside as a whole)
  __device__ __forceinline__ void finish(float (&f)[8], int64_t row, int64_t col, const uint16_t* wrow, float r,
                                         float c) const {
    if (wrow != nullptr) add_scaled8(f, wrow + col, r);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] *= c;
    if (acc != nullptr) {
      float4* p = reinterpret_cast<float4*>(acc + row * N + col);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (add) {
          const float4 g = p[h];
          f[4 * h] += g.x;
          f[4 * h + 1] += g.y;
          f[4 * h + 2] += g.z;
          f[4 * h + 3] += g.w;
        }
        if (!last) p[h] = make_float4(f[4 * h], f[4 * h + 1], f[4 * h + 2], f[4 * h + 3]);
      }
    }
  }
};

struct GradEpi {
  static constexpr int kTeam = 1;
  const CUtensorMap* tm_out;
  const GradOut& o;
  float4* parts;            // [parts][2 CTAs][64 groups of 4 columns][128 rows]
  unsigned int* check;
  gemm::SlabWriter out;

  __device__ __forceinline__ void start(int, int, uint8_t*) {}
  __device__ __forceinline__ void ready(const gemm::Item&, int, int, int, int) {}
  __device__ __forceinline__ void take() {}
  __device__ __forceinline__ void done(int lane) { out.drain(lane); }
  __device__ __forceinline__ void tile(uint32_t tmem, int m0, int n0, const gemm::Item& item, int warp, int lane,
                                       uint8_t* scratch) {
    const int part = item.part;
    const int64_t row = m0 + 32 * warp + lane;
    float r = 0.f;
    const uint16_t* wrow = part < 0 && row < o.M ? o.rest.row(row, r, check) : nullptr;
    const float c = o.scale(wrow);
#pragma unroll 1
    for (int h = 0; h < gemm::TN / 64; ++h) {
      const int c0 = n0 + 64 * h;
      if (c0 >= o.N) break;
      uint32_t w[32];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t v[32];
        tc::tmem_ld32(tmem + 64 * h + 32 * q, v);
        tc::tmem_ld_wait();
        if (part >= 0) {
          float4* p = parts + ((int64_t)part * 2 + (m0 >> 7 & 1)) * 64 * 128 + (16 * h + 8 * q) * 128 + 32 * warp + lane;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            p[j * 128] = make_float4(__uint_as_float(v[4 * j]), __uint_as_float(v[4 * j + 1]),
                                     __uint_as_float(v[4 * j + 2]), __uint_as_float(v[4 * j + 3]));
          continue;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float f[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(v[8 * j + e]);
          const int64_t col = c0 + 32 * q + 8 * j;
          if (row < o.M && col < o.N) o.finish(f, row, col, wrow, r, c);
#pragma unroll
          for (int e = 0; e < 4; ++e) w[16 * q + 4 * j + e] = f32x2_to_bf16x2(f[2 * e], f[2 * e + 1]);
        }
      }
      if (part < 0 && (o.acc == nullptr || o.last) && m0 + 32 * warp < o.M) out.put(scratch, tm_out, w, c0, m0 + 32 * warp, warp, lane);
    }
  }
};

struct GradArgs {
  gemm::Shape shape;
  GradOut out;
  float4* parts;
  const Shared* shared;       // dW: which H to read, see clean_kernel
  unsigned int* check;
};

// A_MN 0: dH [tokens][d] = P W (P K-major, W MN-major); 1: dW [V][d] = P^T H (both MN-major)
template <int A_MN>
__global__ void __launch_bounds__(gemm::threads(4), 1)
grad_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
            const __grid_constant__ CUtensorMap tm_clean, const __grid_constant__ CUtensorMap tm_out,
            const __grid_constant__ GradArgs a) {
  GradEpi epi{&tm_out, a.out, a.parts, a.check, {}};
  const CUtensorMap* b = A_MN && a.shared->dirty ? &tm_clean : &tm_b;
  gemm::run<A_MN, 1, 4, 6>(&tm_a, b, gemm::Plan{a.shape}, epi, a.check);
}

// dH with its sides exchanged, for the same numbers of tokens: D = W^T P^T, a
// lane of the accumulator is a column of dH.  Blocks turn over in shared memory; a
// lane writes 32 columns of its token.
struct GradTEpi {
  static constexpr int kTeam = 1;
  uint16_t* out;            // bf16 [T][d]
  const GradOut& o;         // M tokens, N columns
  float* parts;             // [parts][256 tokens][256 columns]
  int tn;
  unsigned int* check;

  __device__ __forceinline__ void start(int, int, uint8_t*) {}
  __device__ __forceinline__ void ready(const gemm::Item&, int, int, int, int) {}
  __device__ __forceinline__ void take() {}
  __device__ __forceinline__ void done(int) {}
  __device__ __forceinline__ void tile(uint32_t tmem, int m0, int n0, const gemm::Item& item, int warp, int lane,
                                       uint8_t* scratch) {
    float* block = reinterpret_cast<float*>(scratch) + warp * 32 * 33;                     // [column][token], padded
    const int64_t c0 = m0 + 32 * warp;
    if (c0 >= o.N) return;
    const int tokens = (int)(o.M - n0 < tn ? o.M - n0 : tn);
#pragma unroll 1
    for (int q = 0; 32 * q < tokens; ++q) {
      uint32_t v[32];
      tc::tmem_ld32(tmem + 32 * q, v);
      tc::tmem_ld_wait();
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 32; ++j) block[lane * 33 + j] = __uint_as_float(v[j]);
      __syncwarp();
      const int k = 32 * q + lane;
      if (k >= tokens) continue;
      const int64_t t = n0 + k;
      float r = 0.f;
      const uint16_t* wrow = item.part < 0 ? o.rest.row(t, r, check) : nullptr;
      const float c = o.scale(wrow);
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        if (c0 + 8 * g >= o.N) break;
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = block[(8 * g + e) * 33 + lane];
        if (item.part >= 0) {
          float4* p = reinterpret_cast<float4*>(parts + ((int64_t)item.part * 256 + k) * 256 + (m0 & 255) + 32 * warp + 8 * g);
          p[0] = make_float4(f[0], f[1], f[2], f[3]);
          p[1] = make_float4(f[4], f[5], f[6], f[7]);
        } else {
          o.finish(f, t, c0 + 8 * g, wrow, r, c);
          *reinterpret_cast<uint4*>(out + t * o.N + c0 + 8 * g) =
              make_uint4(f32x2_to_bf16x2(f[0], f[1]), f32x2_to_bf16x2(f[2], f[3]), f32x2_to_bf16x2(f[4], f[5]),
                         f32x2_to_bf16x2(f[6], f[7]));
        }
      }
    }
  }
};

__global__ void __launch_bounds__(gemm::threads(4), 1)
grad_t_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_p,
              const __grid_constant__ GradArgs a, uint16_t* out) {
  GradTEpi epi{out, a.out, reinterpret_cast<float*>(a.parts), a.shape.tn, a.check};
  gemm::run<1, 0, 4, 6>(&tm_w, &tm_p, gemm::Plan{a.shape}, epi, a.check);
}

// Joins its cut tiles: block (tile, eight tokens), thread = (token, eight columns).
__global__ void __launch_bounds__(256) join_t_kernel(const __grid_constant__ GradArgs a, uint16_t* __restrict__ out) {
  const gemm::Shape& s = a.shape;
  int m, n;
  gemm::tile_at(s, s.split_from + blockIdx.x, m, n);
  const int k = 8 * blockIdx.y + (threadIdx.x >> 5), c = 8 * (threadIdx.x & 31);
  const int64_t t = (int64_t)n * s.tn + k, col = (int64_t)m * 256 + c;
  if (k >= s.tn || t >= a.out.M || col >= a.out.N) return;
  float r;
  const uint16_t* wrow = a.out.rest.row(t, r, a.check);
  float f[8] = {};
  for (int q = 0; q < s.split; ++q) {
    const float4* p = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(a.parts) +
                                                      (((int64_t)blockIdx.x * s.split + q) * 256 + k) * 256 + c);
    const float4 x = p[0], y = p[1];
    f[0] += x.x; f[1] += x.y; f[2] += x.z; f[3] += x.w;
    f[4] += y.x; f[5] += y.y; f[6] += y.z; f[7] += y.w;
  }
  a.out.finish(f, t, col, wrow, r, a.out.scale(wrow));
  *reinterpret_cast<uint4*>(out + t * a.out.N + col) =
      make_uint4(f32x2_to_bf16x2(f[0], f[1]), f32x2_to_bf16x2(f[2], f[3]), f32x2_to_bf16x2(f[4], f[5]),
                 f32x2_to_bf16x2(f[6], f[7]));
}

// Joins the parts of the tiles that were cut along K, in part order: block
// (tile, CTA half, group of 64 columns), thread = (row, 32 columns).
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ GradArgs a, uint16_t* __restrict__ out) {
  const gemm::Shape& s = a.shape;
  int m, n;
  gemm::tile_at(s, s.split_from + blockIdx.x, m, n);
  const int r128 = threadIdx.x & 127, half = threadIdx.x >> 7;
  const int64_t row = (int64_t)m * gemm::TM + 128 * blockIdx.y + r128;
  const int64_t col0 = (int64_t)n * gemm::TN + 64 * blockIdx.z + 32 * half;
  if (row >= a.out.M) return;
  float r;
  const uint16_t* wrow = a.out.rest.row(row, r, a.check);
  const float c = a.out.scale(wrow);
  const float4* p = a.parts + ((int64_t)blockIdx.x * s.split * 2 + blockIdx.y) * 64 * 128 +
                    (16 * blockIdx.z + 8 * half) * 128 + r128;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int64_t col = col0 + 8 * j;
    if (col >= a.out.N) break;
    float f[8] = {};
    for (int q = 0; q < s.split; ++q) {
      const float4 x = p[(int64_t)q * 2 * 64 * 128 + (2 * j) * 128], y = p[(int64_t)q * 2 * 64 * 128 + (2 * j + 1) * 128];
      f[0] += x.x; f[1] += x.y; f[2] += x.z; f[3] += x.w;
      f[4] += y.x; f[5] += y.y; f[6] += y.z; f[7] += y.w;
    }
    a.out.finish(f, row, col, wrow, r, c);
    if (a.out.acc == nullptr || a.out.last)
      *reinterpret_cast<uint4*>(out + row * a.out.N + col) =
          make_uint4(f32x2_to_bf16x2(f[0], f[1]), f32x2_to_bf16x2(f[2], f[3]), f32x2_to_bf16x2(f[4], f[5]),
                     f32x2_to_bf16x2(f[6], f[7]));
  }
}

// ----------------------------------------------------------------------------
// rows
// ----------------------------------------------------------------------------

// Number of tokens that take part (one CTA), for a mean over several chunks: the
// first chunk's gradients need all chunks' number.
__global__ void __launch_bounds__(1024) count_kernel(const void* target, int target64, int64_t T, int64_t V,
                                                     int64_t ignore, unsigned int* check, Shared* shared) {
  __shared__ int sums[32];
  int c = 0;
  for (int64_t t = threadIdx.x; t < T; t += 1024) c += class_of(target, target64, t, V, ignore, check) >= 0;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) c += __shfl_xor_sync(0xffffffffu, c, off);
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = c;
  __syncthreads();
  if (threadIdx.x == 0) {
    unsigned long long total = 0;
    for (int w = 0; w < 32; ++w) total += (unsigned long long)sums[w];
    shared->count = total;
  }
}

struct LseArgs {
  const float2* stats;
  float* nll;               // the target's logits in, the losses out
  const void* target;
  int target64;
  int64_t ignore_index;
  int T, tiles;
  int64_t V;
  float* lse;
  float* losses;            // [T] of this chunk, or nullptr
  const float* weights;     // per-token losses: [T] of this chunk, or nullptr
  Shared* shared;
  int count;                // add this chunk's tokens to the count
  // the reduced loss, written by the last block of the last chunk (else nullptr):
  // the sum of all_losses[0 .. all), divided by the count for a mean
  float* reduced;
  const float* all_losses;
  int64_t all;
  int mean;
  unsigned int* check;
};

// lse and loss of eight tokens per block: Y thread rows walk the vocabulary's
// tiles, then their pairs are joined by halves.
// The loss is (maximum - l_target) + log(sum): next to lse - l_target it keeps the
// digits of a surely predicted token, whose maximum is the target's own logit.
// The block that finishes last sums the losses, in an order of its own, so the
// sum does not depend on which block that is.
template <int Y>
__global__ void __launch_bounds__(8 * Y) lse_kernel(LseArgs a) {
  __shared__ float2 joined[Y][8];
  __shared__ double sums[Y / 4];
  __shared__ bool last;
  const int t = blockIdx.x * 8 + threadIdx.x, y = threadIdx.y, tid = y * 8 + threadIdx.x;
  float m = -INFINITY, s = 0.f;
  if (t < a.T) {
#pragma unroll 4
    for (int i = y; i < a.tiles; i += Y) {
      const float2 p = a.stats[(int64_t)i * a.T + t];
      join_stats(m, s, p.x, p.y);
    }
  }
  joined[y][threadIdx.x] = make_float2(m, s);
#pragma unroll
  for (int half = Y / 2; half > 0; half >>= 1) {
    __syncthreads();
    if (y < half) {
      const float2 o = joined[y + half][threadIdx.x];
      join_stats(m, s, o.x, o.y);
      joined[y][threadIdx.x] = make_float2(m, s);
    }
  }
  if (y == 0) {
    bool keep = false;
    if (t < a.T) {
      const float ls = logf(s);
      a.lse[t] = m + ls;
      keep = class_of(a.target, a.target64, t, a.V, a.ignore_index, a.check) >= 0;
      const float loss = keep ? (m - a.nll[t]) + ls : 0.f;
      a.nll[t] = loss;
      if (a.losses != nullptr) a.losses[t] = loss;
    }
    if (a.weights != nullptr) {                        // the largest is the same in any order
      float w = keep ? fabsf(a.weights[t]) : 0.f;
      if (!(w < INFINITY)) w = 0.f;
#pragma unroll
      for (int off = 4; off > 0; off >>= 1) w = fmaxf(w, __shfl_xor_sync(0xffu, w, off));
      if (threadIdx.x == 0 && w > 0.f) atomicMax(&a.shared->top, __float_as_uint(w));
    }
    if (a.count) {
      const int n = __popc(__ballot_sync(0xffu, keep));
      if (threadIdx.x == 0 && n) atomicAdd(&a.shared->count, (unsigned long long)n);
    }
  }
  if (a.reduced == nullptr) return;
  __threadfence();
  __syncthreads();
  if (tid == 0) last = atomicAdd(&a.shared->blocks, 1u) == gridDim.x - 1;
  __syncthreads();
  if (!last) return;
  __threadfence();
  double sum = 0.0;
#pragma unroll 4
  for (int64_t k = tid; k < a.all; k += 8 * Y) sum += (double)__ldcg(a.all_losses + k);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  if ((tid & 31) == 0) sums[tid >> 5] = sum;
  __syncthreads();
  if (tid == 0) {
    double total = 0.0;
    for (int w = 0; w < Y / 4; ++w) total += sums[w];
    if (a.mean) {
      const unsigned long long n = *reinterpret_cast<volatile unsigned long long*>(&a.shared->count);
      total /= (double)(n > 0 ? n : 1);
    }
    *a.reduced = (float)total;
  }
}

// P in place of the exponentials: one CTA per token.
//   P_v = c exp(m_tile - lse) e_v,  P_target = c expm1(-loss),  e_v = fp16 / kExpScale
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
  const float* dloss;       // one value per token, or nullptr
  const Shared* shared;     // with dloss: its largest, which the products' sums are multiplied by
  int unit_shift;           // log2 of a stats tile's width in units of eight classes (5 or 4)
  float* rest;              // [T]: P's target entry minus its bf16
  const uint16_t* H;        // with dW: the tokens' rows, and whether one that takes no part is not finite
  int64_t d;
  unsigned int* dirty;
  unsigned int* check;
};

constexpr int kProbThreads = 256;

// one of the two bf16 values has the largest exponent
__device__ __forceinline__ bool not_finite2(uint32_t w) {
  return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

__global__ void __launch_bounds__(kProbThreads) prob_kernel(ProbArgs a) {
  const int t = blockIdx.x;
  uint4* row = reinterpret_cast<uint4*>(a.E + (int64_t)t * a.pitch);
  const int units = (int)(a.pitch / 8);
  const int64_t y = class_of(a.target, a.target64, t, a.V, a.ignore_index, a.check);
  if (y < 0) {
    for (int u = threadIdx.x; u < units; u += kProbThreads) row[u] = make_uint4(0u, 0u, 0u, 0u);
    if (a.H != nullptr) {
      const uint4* h = reinterpret_cast<const uint4*>(a.H + (int64_t)t * a.d);
      bool bad = false;
      for (int u = threadIdx.x; u < (int)(a.d / 8); u += kProbThreads) {
        const uint4 v = __ldg(h + u);
        bad = bad || not_finite2(v.x) || not_finite2(v.y) || not_finite2(v.z) || not_finite2(v.w);
      }
      if (bad) *a.dirty = 1;
    }
    return;
  }
  const float c = a.dloss != nullptr ? a.dloss[t] / top_weight(a.shared) : 1.f;
  const float z = a.lse[t];
  const float at_target = c * expm1f(-a.nll[t]);
  if (threadIdx.x == 0) a.rest[t] = at_target - __bfloat162float(__float2bfloat16_rn(at_target));
  // a warp's 32 units of eight columns are one tile or two: one factor or two per warp and step
  for (int u = threadIdx.x; u < units; u += kProbThreads) {
    const float f = c / kExpScale * __expf(a.stats[(int64_t)(u >> a.unit_shift) * a.T + t].x - z);
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

// A token that takes no part has a row of zeros in P, but zero times a NaN or an
// infinity in its row of H (padding may hold anything) would spoil all of dW.  Where
// prob_kernel has met such a row, dW reads a copy of H with zeros in these rows.
__global__ void __launch_bounds__(256) clean_kernel(const uint4* __restrict__ H, const void* target, int target64, int T,
                                                    int64_t V, int64_t ignore, int64_t units, uint4* __restrict__ out,
                                                    const Shared* shared, unsigned int* check) {
  if (!shared->dirty) return;
  for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
    const bool part = class_of(target, target64, t, V, ignore, check) >= 0;
    for (int64_t u = threadIdx.x; u < units; u += 256)
      out[t * units + u] = part ? __ldg(H + t * units + u) : make_uint4(0u, 0u, 0u, 0u);
  }
}

// x and y (each may be empty) *= factor in place, unless the factor is one
__global__ void __launch_bounds__(256) scale_kernel(uint4* __restrict__ x, int64_t x_units, uint4* __restrict__ y,
                                                    int64_t y_units, const float* factor) {
  const float f = *factor;
  if (f == 1.f) return;
  for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < x_units + y_units; u += (int64_t)gridDim.x * 256) {
    uint4* at = u < x_units ? x + u : y + (u - x_units);
    const uint4 v = *at;
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int q = 0; q < 4; ++q)
      w[q] = f32x2_to_bf16x2(__uint_as_float(w[q] << 16) * f, __uint_as_float(w[q] & 0xffff0000u) * f);
    *at = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// ----------------------------------------------------------------------------
// workspace and launches
// ----------------------------------------------------------------------------

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
  size_t e, acc, parts, stats, lse, nll, rest, losses, clean, shared, total;
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
  l.parts = take(grads ? (size_t)(num_sms() / 2) * gemm::TM * gemm::TN * 4 : 0);
  // one pair per token and tile, the narrowest tiles that balance_tiles and balance_rows choose
  const int64_t few = T < kScoreTokens ? T : kScoreTokens;
  const size_t wide = (size_t)((V + kMinTile - 1) / kMinTile) * l.chunk, narrow = (size_t)(2 * ((V + 2 * kMinRows - 1) / (2 * kMinRows))) * few;
  l.stats = take((wide > narrow ? wide : narrow) * 8);
  l.lse = take((size_t)l.chunk * 4);
  l.nll = take((size_t)l.chunk * 4);
  l.rest = take((size_t)l.chunk * 4);
  l.losses = take((size_t)T * 4);
  l.clean = take(dw ? (size_t)l.chunk * d * 2 : 0);
  l.shared = take(sizeof(Shared));
  l.total = at;
  return l;
}

cudaError_t map_rows(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, int64_t pitch, int box_cols,
                     int box_rows) {
  return make_tmap_2d(m, base, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, (uint64_t)cols, (uint64_t)rows, (uint64_t)pitch * 2,
                      (uint32_t)box_cols, (uint32_t)box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
}

// The loss alone: classes per tile.  The pairs take the tiles in rounds, and few
// tokens make few tiles, so a tile is narrowed until the last round is as full as
// the others (the time goes with rounds * width).
void balance_tiles(gemm::Shape& s, int64_t V) {
  const int64_t pairs = num_sms() / 2;
  int64_t best = 0;
  for (int tn = gemm::TN; tn >= kMinTile; tn -= 32) {
    const int64_t nt = (V + tn - 1) / tn, rounds = (s.mt * nt + pairs - 1) / pairs;
    if (best == 0 || rounds * tn < best) {
      best = rounds * tn;
      s.tn = tn;
      s.nt = (int)nt;
    }
  }
  s.split_from = s.mt * s.nt;
}

// The same for the exchanged product, whose tiles are rows of W: classes per CTA.
void balance_rows(gemm::Shape& s, int64_t V, int64_t T) {
  const int64_t pairs = num_sms() / 2;
  int64_t best = 0;
  s.tn = (int)up(T, 32);
  for (int rows = 128; rows >= kMinRows; rows -= 8) {
    const int64_t mt = (V + 2 * rows - 1) / (2 * rows), rounds = (mt + pairs - 1) / pairs;
    if (best == 0 || rounds * rows < best) {
      best = rounds * rows;
      s.a_rows = rows;
      s.mt = (int)mt;
    }
  }
  s.split_from = s.mt * s.nt;
}

// Tiles of `tn` tokens on the N side.
void token_tiles(gemm::Shape& s, int64_t T, int tn) {
  s.tn = tn;
  s.nt = (int)((T + tn - 1) / tn);
  s.split_from = s.mt * s.nt;
}

// Tokens per tile of the exchanged products, or 0 when tiles of 256 tokens are as
// good.  The pairs take the tiles (`other` times as many as there are tiles of
// tokens) in rounds; a K step of w tokens takes 0.16 + 0.00087 w us, 0.25 at least
// (measured from 32 to 256), one of the straight product what 256 take.  Both
// sides at 32000 x 4096, logits and dH, us: 50 tokens 59 + 56 straight, 51 + 48
// exchanged; 300 tokens 96 + 96 and 88 + 82; 1029 tokens at 50021 x 5120 429 + 447
// and 415 + 395; 700 and 2100 tokens of logits within 2 %.
int exchanged_tokens(int64_t T, int64_t other, bool cut) {
  const int64_t pairs = num_sms() / 2;
  auto step = [](int w) { return w < 104 ? 0.25 : 0.16 + 0.00087 * w; };
  // a last round that is cut along K costs its share of a round
  auto rounds = [&](int64_t tiles) {
    const int64_t rem = tiles % pairs, split = rem ? pairs / rem : 1;
    return (double)(tiles / pairs) + (rem == 0 ? 0.0 : cut && split >= 2 ? 1.0 / (double)(split < 8 ? split : 8) : 1.0);
  };
  double best = 0.95 * rounds(gemm::tiles_of(T) * other) * step(256);
  int tn = 0;
  for (int w = 224; w >= 32; w -= 32) {
    const int64_t tiles = (T + w - 1) / w;
    const double cost = rounds(tiles * other) * step(w);
    if (cost < best && tiles * w < up(T, 256)) {
      best = cost;
      tn = w;
    }
  }
  return tn;
}

cudaError_t launch_join(const GradArgs& a, uint16_t* out, cudaStream_t s) {
  const int cut = a.shape.mt * a.shape.nt - a.shape.split_from;
  if (cut == 0) return cudaSuccess;
  join_kernel<<<dim3((unsigned)cut, 2, 4), 256, 0, s>>>(a, out);
  return cudaGetLastError();
}

#define SK_TRY(...)                     \
  do {                                  \
    cudaError_t e_ = (__VA_ARGS__);     \
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
  float* rest = reinterpret_cast<float*>(ws + l.rest);
  float4* parts = reinterpret_cast<float4*>(ws + l.parts);
  float* losses = a.reduction == SK_CE_NONE ? a.loss : reinterpret_cast<float*>(ws + l.losses);
  Shared* shared = reinterpret_cast<Shared*>(ws + l.shared);
  const bool mean = a.reduction == SK_CE_MEAN;
  const bool count_first = mean && l.chunk < a.T;
  if (count_first) {
    count_kernel<<<1, 1024, 0, s>>>(a.target, a.target64, a.T, a.V, a.ignore_index, a.check, shared);
    SK_TRY(cudaGetLastError());
  }
  CUtensorMap tm_w_mn, tm_dw;
  if (dh) SK_TRY(map_rows(&tm_w_mn, a.W, a.V, a.d, a.d, 64, 64));
  if (dw) SK_TRY(map_rows(&tm_dw, a.dW, a.V, a.d, a.d, 64, 32));
  for (int64_t t0 = 0; t0 < a.T; t0 += l.chunk) {
    const int64_t T = a.T - t0 < l.chunk ? a.T - t0 : l.chunk;
    const uint16_t* H = a.H + t0 * a.d;
    const void* target = static_cast<const uint8_t*>(a.target) + t0 * (a.target64 ? 8 : 4);
    const bool score = !grads && T <= kScoreTokens;
    const int logit_tn = grads ? exchanged_tokens(T, gemm::tiles_of(a.V), false) : 0;
    const bool exchanged = score || logit_tn > 0;      // M = classes, N = tokens
    gemm::Shape shape = exchanged ? gemm::shape_of(a.V, T, a.d) : gemm::shape_of(T, a.V, a.d);
    if (score) balance_rows(shape, a.V, T);
    else if (exchanged) token_tiles(shape, T, logit_tn);
    else if (!grads) balance_tiles(shape, a.V);
    CUtensorMap tm_h, tm_w;
    SK_TRY(map_rows(&tm_h, H, T, a.d, a.d, 64, exchanged ? shape.tn / 2 : 128));
    SK_TRY(map_rows(&tm_w, a.W, a.V, a.d, a.d, 64, exchanged ? shape.a_rows : shape.tn / 2));
    LogitArgs la{shape, stats, nll, target, a.target64, a.ignore_index, (int)T, (int)a.V,
                 grads ? 1 : 0, shared, count_first ? 1 : 0, a.check};
    if (score) {
      SK_TRY(gemm::launch_pairs<4, 6>(score_kernel, gemm::items(shape), s, tm_w, tm_h, la));
    } else if (exchanged) {
      SK_TRY(gemm::launch_pairs<4, 6>(logit_t_kernel, gemm::items(shape), s, tm_w, tm_h, la, E, l.pitch));
    } else {
      CUtensorMap tm_e = tm_h;                       // used with gradients only
      if (grads) SK_TRY(map_rows(&tm_e, E, T, a.V, l.pitch, 64, 32));
      SK_TRY(gemm::launch_pairs<4, 6>(logit_kernel, gemm::items(shape), s, tm_h, tm_w, tm_e, la));
    }
    const int stat_tiles = score ? 2 * shape.mt : exchanged ? (int)((a.V + 127) / 128) : shape.nt;
    const bool reduce = a.reduction != SK_CE_NONE && a.loss != nullptr && t0 + T >= a.T;
    const bool each = a.reduction == SK_CE_NONE;
    const float* weights = grads && each && a.dloss != nullptr ? a.dloss + t0 : nullptr;
    LseArgs le{stats, nll, target, a.target64, a.ignore_index, (int)T, stat_tiles, a.V, lse, losses ? losses + t0 : nullptr,
               weights, shared, mean && !count_first ? 1 : 0, reduce ? a.loss : nullptr, losses, a.T, mean ? 1 : 0, a.check};
    // few tokens make few blocks: more threads in each
    if (T <= kScoreTokens) lse_kernel<128><<<(unsigned)((T + 7) / 8), dim3(8, 128), 0, s>>>(le);
    else lse_kernel<32><<<(unsigned)((T + 7) / 8), dim3(8, 32), 0, s>>>(le);
    SK_TRY(cudaGetLastError());
    if (!grads) continue;
    const float* factor = each ? nullptr : a.dloss;
    const Shared *count = mean ? shared : nullptr, *top = weights ? shared : nullptr;
    ProbArgs pa{E, l.pitch, stats, lse, nll, target, a.target64, a.ignore_index, (int)T, (int)a.V,
                weights, shared, exchanged ? 4 : 5, rest,
                dw ? H : nullptr, a.d, &shared->dirty, a.check};
    prob_kernel<<<(unsigned)T, kProbThreads, 0, s>>>(pa);
    SK_TRY(cudaGetLastError());
    if (dh) {
      CUtensorMap tm_p, tm_dh;
      uint16_t* out = a.dH + t0 * a.d;
      GradArgs ga{gemm::shape_of(T, a.d, a.V),
                  {nullptr, 0, 1, T, a.d, {rest, a.W, target, a.target64, a.V, a.d, a.ignore_index},
                   factor, count, top}, parts, shared, a.check};
      const int tn = exchanged_tokens(T, gemm::tiles_of(a.d), true);
      if (tn > 0) {
        ga.shape = gemm::shape_of(a.d, T, a.V);
        token_tiles(ga.shape, T, tn);
        gemm::split_last_round(ga.shape);
        SK_TRY(map_rows(&tm_p, E, T, a.V, l.pitch, 64, tn / 2));
        SK_TRY(gemm::launch_pairs<4, 6>(grad_t_kernel, gemm::items(ga.shape), s, tm_w_mn, tm_p, ga, out));
        const int cut = ga.shape.mt * ga.shape.nt - ga.shape.split_from;
        if (cut > 0) {
          join_t_kernel<<<dim3((unsigned)cut, (unsigned)((tn + 7) / 8)), 256, 0, s>>>(ga, out);
          SK_TRY(cudaGetLastError());
        }
      } else {
        gemm::split_last_round(ga.shape);
        SK_TRY(map_rows(&tm_p, E, T, a.V, l.pitch, 64, 128));
        SK_TRY(map_rows(&tm_dh, out, T, a.d, a.d, 64, 32));
        SK_TRY(gemm::launch_pairs<4, 6>(grad_kernel<0>, gemm::items(ga.shape), s, tm_p, tm_w_mn, tm_w_mn, tm_dh, ga));
        SK_TRY(launch_join(ga, out, s));
      }
    }
    if (dw) {
      CUtensorMap tm_p, tm_hm, tm_clean;
      uint16_t* clean = reinterpret_cast<uint16_t*>(ws + l.clean);
      SK_TRY(map_rows(&tm_p, E, T, a.V, l.pitch, 64, 64));
      SK_TRY(map_rows(&tm_hm, H, T, a.d, a.d, 64, 64));
      SK_TRY(map_rows(&tm_clean, clean, T, a.d, a.d, 64, 64));
      const int64_t blocks = 2 * (int64_t)num_sms();
      clean_kernel<<<(unsigned)(T < blocks ? T : blocks), 256, 0, s>>>(
          reinterpret_cast<const uint4*>(H), target, a.target64, (int)T, a.V, a.ignore_index, a.d / 8,
          reinterpret_cast<uint4*>(clean), shared, a.check);
      SK_TRY(cudaGetLastError());
      GradArgs ga{gemm::shape_of(a.V, a.d, T), {acc, t0 > 0 ? 1 : 0, t0 + T >= a.T ? 1 : 0, a.V, a.d, {}, factor, count, top}, parts,
                  shared, a.check};
      gemm::split_last_round(ga.shape);
      SK_TRY(gemm::launch_pairs<4, 6>(grad_kernel<1>, gemm::items(ga.shape), s, tm_p, tm_hm, tm_clean, tm_dw, ga));
      SK_TRY(launch_join(ga, a.dW, s));
    }
  }
  return cudaSuccess;
}

cudaError_t launch_scale_bf16(uint16_t* x, int64_t nx, uint16_t* y, int64_t ny, const float* factor, cudaStream_t s) {
  const int64_t units = (nx + ny) / 8;
  const int64_t blocks = (units + 255) / 256, cap = (int64_t)num_sms() * 8;
  scale_kernel<<<(unsigned)(blocks < cap ? blocks : cap), 256, 0, s>>>(reinterpret_cast<uint4*>(x), nx / 8,
                                                                       reinterpret_cast<uint4*>(y), ny / 8, factor);
  return cudaGetLastError();
}

}  // namespace sk
