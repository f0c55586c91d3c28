// LUT gradient of the sketched linear layer from an 8-bit activation checkpoint:
//
//   dlut[s][i][g][c] = sum over the tokens t of set s and the columns j of group g
//                      with idx[i][j] = c of dY[t][i] * q[t][j] * 2^e[t][j / 32]
//
// i.e. the corrected Eq. 6 of the "Sketch to Adapt" OpenReview discussion (reply
// Q1) with X as the checkpoint holds it (format in sk_ckpt8.cuh).
//
// Tensor cores: a pass over the checkpoint writes the layer's X as bf16 (exact) to
// the workspace, in task order when there are several LUT sets, and the
// persistent product of sk_gemm.cuh forms the G tiles [256 rows i x 256 columns j]
// = dY^T X over K = the set's tokens, both operands MN-major.  G is never written:
// while the next tile's MMAs run, the epilogue adds a finished tile's columns into
// the (group, centroid) bins of its rows and writes the bins.  The bound is the
// tensor pipe (2 T n d flops) from about 500 tokens per set on, the binning of
// n d accumulators per set below.
//
// The pass costs 33/32 + 2 bytes per value, 18 us next to a product of about 500
// at [8192, 4096] x [8192, 11008].  Dequantising in the product instead (warps
// that write the operand tiles in place of the copy engine) was built first and
// ran at 726 us: every step of every pair then waits for sixteen warps of two SMs,
// and each of the 43 row blocks dequantises X again.
#include <type_traits>

#include "sk_gemm.cuh"
#include "sk_lut8.cuh"

namespace sk {
namespace {

using gemm::KS;
using gemm::TN;

constexpr int COPIES = 4;              // copies of the bins per epilogue thread
// operand stages: 16 bins of 256 threads in four copies take the sixth stage's place
constexpr int stages(int bits) { return bits == 4 ? 5 : 6; }
static_assert(COPIES * 16 * 256 * 4 <= gemm::Smem<stages(4)>::SCRATCH && COPIES * 8 * 256 * 4 <= gemm::Smem<stages(3)>::SCRATCH,
              "the bins fit the epilogue's shared memory");

// Group slots of one 256-column tile.
__host__ __device__ inline int group_slots(int64_t gs, int gpr) {
  const int64_t s = (TN - 1) / gs + 2;
  return (int)(s < gpr ? s : gpr);
}

struct Lut8Args {
  gemm::Shape shape;         // of one LUT set
  const uint8_t* packed;
  int64_t row_bytes;
  int64_t n, d, gs;
  int gpr, slots, sets;
  float* part;               // [sets][jtiles][n][slots][k] partial bins
  int64_t part_set_stride;
  float* extra;              // [cut parts beyond a tile's first][256][slots][k]
  // several LUT sets: rows in task order, set z's tokens at positions
  // [segs[2z], segs[2z] + segs[2z + 1]) (multiples of 64 apart, zero rows between);
  // nullptr for one LUT set
  const int* segs;
  // several LUT sets whose groups are whole column tiles (`per_group` of them; else
  // 0): a pair takes a row block through all tiles of a group, its bins stay, and
  // dlut is written at once, without partial bins and their reduction
  int per_group;
  float* dlut;
  int accumulate;
  unsigned int* check;
};

// items: set after set, each set's tiles in the product's order; or, with
// per_group, units of (set, group, row block) whose tiles follow one another in a
// pair's sequence
struct Lut8Plan {
  const Lut8Args& a;
  __device__ __forceinline__ int units() const { return a.sets * a.gpr * a.shape.mt; }
  __device__ __forceinline__ int count() const {
    if (a.segs == nullptr) return gemm::items(a.shape);
    const int pairs = gridDim.x >> 1;
    if (a.per_group) return (units() + pairs - 1) / pairs * a.per_group * pairs;
    return a.sets * a.shape.mt * a.shape.nt;
  }
  __device__ __forceinline__ const gemm::Shape& shape() const { return a.shape; }
  __device__ __forceinline__ gemm::Item item(int i) const {
    if (a.segs == nullptr) return gemm::item_at(a.shape, i);
    gemm::Item it;
    int set;
    if (a.per_group) {
      const int pairs = gridDim.x >> 1, k = i / pairs;
      const int unit = i - k * pairs + k / a.per_group * pairs;
      if (unit >= units()) return gemm::Item{0, 0, 0, 0, -1};      // nothing left for this pair
      const int sg = unit / a.shape.mt;
      set = sg / a.gpr;
      it.m = unit - sg * a.shape.mt;
      it.n = (sg - set * a.gpr) * a.per_group + k % a.per_group;
    } else {
      set = i / (a.shape.mt * a.shape.nt);
      gemm::tile_at(a.shape, i - set * a.shape.mt * a.shape.nt, it.m, it.n);
    }
    it.part = set;                                     // a whole tile of this set
    it.k0 = __ldg(a.segs + 2 * set) / KS;
    it.k1 = it.k0 + (__ldg(a.segs + 2 * set + 1) + KS - 1) / KS;
    return it;
  }
};

// shared memory by its 32-bit address plus a constant (through a pointer that has
// lost its address space every access would be a generic one)
template <int OFF>
__device__ __forceinline__ float lds(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1 + %2];" : "=f"(v) : "r"(a), "n"(OFF));
  return v;
}
template <int OFF>
__device__ __forceinline__ void sts(uint32_t a, float v) {
  asm volatile("st.shared.f32 [%0 + %1], %2;" ::"r"(a), "n"(OFF), "f"(v));
}

// index e of a chunk times 1024
template <int BITS>
__device__ __forceinline__ uint32_t index_1024(const Chunk<BITS>& ch, int e) {
  if constexpr (BITS == 3) return chunk_index<3>(ch, e) << 10;
  const int bit = e * BITS, s = bit & 31;
  const uint32_t w = ch.w[bit >> 5], mask = ((1u << BITS) - 1u) << 10;
  return (s >= 10 ? w >> (s - 10) : w << (10 - s)) & mask;
}

template <int N, class F>
__device__ __forceinline__ void unroll(F f) {
  if constexpr (N > 0) {
    unroll<N - 1>(f);
    f(std::integral_constant<int, N - 1>());
  }
}

// Bins the accumulator's columns.  Eight warps: thread = (row, half of the tile's
// columns), so that two warps of a scheduler fill each other's waits.  A thread's
// bins are its own column of shared memory, [COPIES][K][256 threads], and
// consecutive columns add into different copies.  The group that spans the
// halves' border is written by the lower half with both halves' sums.
template <int BITS>
struct BinEpi {
  static constexpr int kTeam = 2;                    // the two warps of a row meet at a group's flush
  static constexpr int K = 1 << BITS, HB = TN / 64;
  static constexpr int COPY = K * 1024;              // bytes between a thread's copies
  const Lut8Args& a;
  Chunk<BITS> chunks[HB], coming[HB];   // the row's indices of this half tile and of the next

  // the bins start at zero and every flush leaves them there
  __device__ __forceinline__ void start(int warp, int lane, uint8_t* scratch) {
    clear(tc::smem_u32(scratch) + 4 * (32 * warp + lane));
  }
  __device__ __forceinline__ void take() {
#pragma unroll
    for (int b = 0; b < HB; ++b) chunks[b] = coming[b];
  }
  __device__ __forceinline__ void ready(const gemm::Item&, int m0, int n0, int warp, int lane) {
    const int64_t row = m0 + 32 * (warp & 3) + lane;
    const int64_t c0 = n0 + 128 * (warp >> 2);
    if (row >= a.n) return;
    const uint8_t* src = a.packed + row * a.row_bytes;
#pragma unroll
    for (int b = 0; b < HB; ++b)
      if (c0 + 32 * b < a.d) coming[b] = load_chunk<BITS>(src, (c0 >> 5) + b);
  }
  __device__ __forceinline__ void done(int) {}

  // The sums of a group: out, and the bins to zero.
  __device__ __forceinline__ void flush(uint32_t bins, float4* out, bool write) {
#pragma unroll 1
    for (int c4 = 0; c4 < K / 4; ++c4, bins += 4096) {
      float v[4];
      unroll<4>([&](auto e) {
        v[e] = (lds<e * 1024>(bins) + lds<e * 1024 + COPY>(bins)) + (lds<e * 1024 + 2 * COPY>(bins) + lds<e * 1024 + 3 * COPY>(bins));
      });
      unroll<4>([&](auto e) { unroll<COPIES>([&](auto k) { sts<e * 1024 + k * COPY>(bins, 0.f); }); });
      if (write) out[c4] = make_float4(v[0], v[1], v[2], v[3]);
    }
  }
  // The same for a group of both halves (`low`: the lower half's bins, the upper's
  // are 512 bytes further on): each half takes every other four bins.
  __device__ __forceinline__ void flush_both(uint32_t low, int half, float4* out, bool write, bool add) {
    low += 4096 * half;
#pragma unroll 1
    for (int c4 = half; c4 < K / 4; c4 += 2, low += 8192) {
      float v[4];
      unroll<4>([&](auto e) {
        v[e] = (lds<e * 1024>(low) + lds<e * 1024 + COPY>(low)) + (lds<e * 1024 + 2 * COPY>(low) + lds<e * 1024 + 3 * COPY>(low));
        v[e] += (lds<e * 1024 + 512>(low) + lds<e * 1024 + 512 + COPY>(low)) +
                (lds<e * 1024 + 512 + 2 * COPY>(low) + lds<e * 1024 + 512 + 3 * COPY>(low));
      });
      unroll<4>([&](auto e) {
        unroll<COPIES>([&](auto k) {
          sts<e * 1024 + k * COPY>(low, 0.f);
          sts<e * 1024 + 512 + k * COPY>(low, 0.f);
        });
      });
      if (write && add) {
        const float4 o = out[c4];
        out[c4] = make_float4(o.x + v[0], o.y + v[1], o.z + v[2], o.w + v[3]);
      } else if (write) {
        out[c4] = make_float4(v[0], v[1], v[2], v[3]);
      }
    }
  }
  __device__ __forceinline__ void clear(uint32_t bins) {
    unroll<COPIES * K>([&](auto c) { sts<c * 1024>(bins, 0.f); });
  }

  // the next chunk's 32 columns into the bins
  __device__ __forceinline__ void add_chunk(uint32_t tmem, bool have, uint32_t bins) {
    const Chunk<BITS> ch = chunks[0];
#pragma unroll
    for (int q = 0; q + 1 < HB; ++q) chunks[q] = chunks[q + 1];
    uint32_t v[32];
    if (have) {
      tc::tmem_ld32(tmem, v);
      tc::tmem_ld_wait();
    } else {
#pragma unroll
      for (int e = 0; e < 32; ++e) v[e] = 0u;
    }
    unroll<8>([&](auto e4) {
      uint32_t at[COPIES];
      float sum[COPIES];
      unroll<COPIES>([&](auto k) { at[k] = bins + index_1024<BITS>(ch, 4 * e4 + k); });
      unroll<COPIES>([&](auto k) { sum[k] = lds<k * COPY>(at[k]); });
      unroll<COPIES>([&](auto k) { sts<k * COPY>(at[k], sum[k] + __uint_as_float(v[4 * e4 + k])); });
    });
  }

  __device__ __forceinline__ void tile(uint32_t tmem, int m0, int n0, const gemm::Item& it, int warp, int lane,
                                       uint8_t* scratch) {
    if (a.per_group && it.part < 0) return;            // a pair without a unit
    const int quad = warp & 3, half = warp >> 2;
    const int64_t row = m0 + 32 * quad + lane;
    const bool have = it.k1 > it.k0;                   // a set without tokens: zeros
    const uint32_t bins = tc::smem_u32(scratch) + 4 * (32 * warp + lane);
    if (a.per_group) {
#pragma unroll 1
      for (int b = 0; b < HB; ++b) add_chunk(tmem + 128 * half + 32 * b, have, bins);
      const int g = it.n / a.per_group;
      if (it.n - g * a.per_group == a.per_group - 1) {
        float* out = a.dlut + (((int64_t)it.part * a.n + row) * a.gpr + g) * K;
        tc::named_bar_sync(1 + quad, 64);
        flush_both(bins - 512 * half, half, reinterpret_cast<float4*>(out), row < a.n, a.accumulate != 0);
        tc::named_bar_sync(1 + quad, 64);
      }
      return;
    }
    // where this tile's partial bins go
    float* dst;
    if (a.segs == nullptr && it.part >= 0 && it.part % a.shape.split != 0) {
      const int q = it.part % a.shape.split, cut = it.part / a.shape.split;
      dst = a.extra + (((int64_t)cut * (a.shape.split - 1) + q - 1) * gemm::TM + (row - (int64_t)it.m * gemm::TM)) * a.slots * K;
    } else {
      const int64_t set = a.segs == nullptr ? 0 : it.part;
      dst = a.part + set * a.part_set_stride + ((int64_t)it.n * a.n + row) * a.slots * K;
    }
    const int gs = (int)a.gs, first_g = n0 / gs;
    const int c0 = n0 + 128 * half;
    const int nb = a.d <= c0 ? 0 : a.d - c0 < 128 ? (int)(a.d - c0) / 32 : HB;     // chunks of this half
    // a group on both sides of the border: the two warps of these rows meet when
    // each has all of its share, and again when the bins are zero
    const int border = n0 + 128;
    const bool shared_g = border < a.d && border % gs != 0;
    int g = c0 / gs, g_end = (g + 1) * gs;
    bool first = true;
    auto finish = [&](bool last) {
      float4* out = reinterpret_cast<float4*>(dst + (g - first_g) * K);
      if (shared_g && (half ? first : last)) {
        tc::named_bar_sync(1 + quad, 64);
        flush_both(bins - 512 * half, half, out, row < a.n, false);
        tc::named_bar_sync(1 + quad, 64);
      } else {
        flush(bins, out, row < a.n);
      }
      first = false;
    };
    // one copy of the code for all chunks: instruction fetches count here
    // (unrolled over the chunks: 8 % slower)
#pragma unroll 1
    for (int b = 0; b <= nb; ++b) {
      const int jc = c0 + 32 * b;
      if (b == nb) {
        if (nb > 0) finish(true);
        break;
      }
      if (jc >= g_end) {               // a later group (d / gpr is a multiple of 32): hand the finished one on
        finish(false);
        do { ++g; g_end += gs; } while (jc >= g_end);
      }
      add_chunk(tmem + 128 * half + 32 * b, have, bins);
    }
  }
};

template <int BITS>
__global__ void __launch_bounds__(gemm::threads(8), 1)
lut8_tc_kernel(const __grid_constant__ CUtensorMap tm_dy, const __grid_constant__ CUtensorMap tm_x,
               const __grid_constant__ Lut8Args a) {
  BinEpi<BITS> epi{a, {}, {}};
  gemm::run<1, 1, 8, stages(BITS)>(&tm_dy, &tm_x, Lut8Plan{a}, epi, a.check);
}

// Sum the partial bins of every (set, row, group) over the column tiles that
// touch the group, in tile order (a tile's cut parts in part order), and write (or
// add to) dlut: four bins a thread.
template <int BITS, bool CUT>
__global__ void __launch_bounds__(256) lut8_reduce_kernel(const __grid_constant__ Lut8Args a, float4* __restrict__ dlut,
                                                          int accumulate, int64_t total) {
  constexpr int Q = (1 << BITS) / 4;
  const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (e >= total) return;
  const int c = (int)(e % Q);
  const int64_t ig = e / Q;
  const int g = (int)(ig % a.gpr);
  const int64_t si = ig / a.gpr, set = si / a.n, i = si - set * a.n;
  const float4* part = reinterpret_cast<const float4*>(a.part + set * a.part_set_stride);
  const float4* extra = reinterpret_cast<const float4*>(a.extra);
  const int t_first = (int)(((int64_t)g * a.gs) / TN);
  const int t_last = (int)(((int64_t)(g + 1) * a.gs - 1) / TN);
  const int m = (int)(i / gemm::TM);
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](const float4& v) { sum = make_float4(sum.x + v.x, sum.y + v.y, sum.z + v.z, sum.w + v.w); };
#pragma unroll 4
  for (int t = t_first; t <= t_last; ++t) {
    // only a group's first tile can start in an earlier group
    const int slot = t == t_first ? g - (int)(((int64_t)t * TN) / a.gs) : 0;
    add(__ldg(part + (((int64_t)t * a.n + i) * a.slots + slot) * Q + c));
    if constexpr (CUT) {
      const int cut = gemm::tile_index(a.shape, m, t) - a.shape.split_from;
      for (int q = 0; cut >= 0 && q < a.shape.split - 1; ++q)
        add(__ldg(extra + ((((int64_t)cut * (a.shape.split - 1) + q) * gemm::TM + (i - (int64_t)m * gemm::TM)) * a.slots + slot) * Q + c));
    }
  }
  if (accumulate) add(dlut[e]);
  dlut[e] = sum;
}

// ----------------------------------------------------------------------------
// tokens by LUT set, in token order
// ----------------------------------------------------------------------------

constexpr int kRouteThreads = 1024;

// One CTA.  A warp owns a contiguous range of tokens: it counts its tokens of
// every set, the counts are laid out set after set (segments at multiples of KS)
// and warp after warp within a set, and the warp places its tokens in order.  The
// order within a set is the token order, so sums over it never depend on timing.
__global__ void __launch_bounds__(kRouteThreads) lut8_route_kernel(const int32_t* __restrict__ task, int T, int ntask,
                                                                   int positions, int* __restrict__ perm,
                                                                   int* __restrict__ segs, unsigned int* check) {
  __shared__ int at[32][kMaxRouteTasks];        // the warp's count, then its next position, of a set
  __shared__ int total[kMaxRouteTasks];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per = ((T + 31) / 32 + 31) / 32 * 32;
  const int t0 = (int)min((int64_t)warp * per, (int64_t)T), t1 = (int)min((int64_t)t0 + per, (int64_t)T);
  for (int i = lane; i < ntask; i += 32) at[warp][i] = 0;
  for (int p = tid; p < positions; p += kRouteThreads) perm[p] = -1;
  __syncwarp();
  bool bad = false;
  // each token once per pass; the lanes of one set agree through their lowest
  auto each = [&](auto f) {
#pragma unroll 4
    for (int b = t0; b < t1; b += 32) {
      const int t = b + lane;
      int tau = t < t1 ? __ldg(task + t) : -1;
      if (tau < 0 || tau >= ntask) {
        bad = bad || t < t1;
        tau = -1;
      }
      const uint32_t same = __match_any_sync(0xffffffffu, tau);
      f(t, tau, same);
      __syncwarp();
    }
  };
  each([&](int, int tau, uint32_t same) {
    if (tau >= 0 && lane == __ffs(same) - 1) at[warp][tau] += __popc(same);
  });
  if (bad) atomicOr(check, SK_CHECK_TASK_RANGE);   // left out of every LUT set's gradient
  __syncthreads();
  for (int i = tid; i < ntask; i += kRouteThreads) {
    int c = 0;
    for (int w = 0; w < 32; ++w) {
      const int mine = at[w][i];
      at[w][i] = c;
      c += mine;
    }
    total[i] = c;
  }
  __syncthreads();
  if (tid == 0) {
    int pos = 0;
    for (int tau = 0; tau < ntask; ++tau) {
      const int c = total[tau];
      segs[2 * tau] = pos;
      segs[2 * tau + 1] = c;
      total[tau] = pos;
      pos += (c + KS - 1) / KS * KS;
    }
  }
  __syncthreads();
  each([&](int t, int tau, uint32_t same) {
    int p = 0;
    if (tau >= 0) {
      p = total[tau] + at[warp][tau] + __popc(same & ((1u << lane) - 1u));
      perm[p] = t;
    }
    __syncwarp();
    if (tau >= 0 && lane == __ffs(same) - 1) at[warp][tau] += __popc(same);
  });
}

// Both operands in task order, one position per grid row, zero rows between the
// segments: dY's rows copied, the checkpoint's rows as bf16.
__global__ void __launch_bounds__(256) lut8_gather_kernel(const uint4* __restrict__ dY, const uint2* __restrict__ q,
                                                          const uint8_t* __restrict__ scale, const int* __restrict__ perm,
                                                          int64_t dy_units, int64_t x_units, uint4* __restrict__ dYp,
                                                          uint4* __restrict__ X) {
  const int64_t p = blockIdx.y;
  const int t = perm[p];
  for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < dy_units + x_units; u += (int64_t)gridDim.x * 256) {
    uint4 o = make_uint4(0u, 0u, 0u, 0u);
    if (u < dy_units) {
      if (t >= 0) o = __ldg(dY + (int64_t)t * dy_units + u);
      dYp[p * dy_units + u] = o;
    } else {
      const int64_t v = u - dy_units;
      if (t >= 0) {
        const int64_t at = (int64_t)t * x_units + v;
        const uint2 b = __ldg(q + at);
        const uint32_t s2 = ckpt8_scale2(__ldg(scale + (at >> 2)));
        ckpt8_dequant4(b.x, s2, o.x, o.y);
        ckpt8_dequant4(b.y, s2, o.z, o.w);
      }
      X[p * x_units + v] = o;
    }
  }
}

int64_t route_positions(int64_t T, int ntask) { return T + (int64_t)ntask * (KS - 1); }

size_t pad256(size_t b) { return (b + 255) / 256 * 256; }

// Several LUT sets: whole groups per pair, whose bins go to dlut without partial bins,
// while that leaves at most a tenth of the last round idle.
bool whole_groups(int64_t n, int64_t d, int gpr, int ntask) {
  if (d / gpr % TN != 0) return false;
  const int64_t units = (int64_t)ntask * gpr * gemm::tiles_of(n), pairs = num_sms() / 2;
  return 10 * units >= 9 * ((units + pairs - 1) / pairs * pairs);
}

// Otherwise the sets go in blocks whose partial bins take kPartBytes at most (one
// set's if that is more): they grow with n d and the sets, whatever the tokens are
// (256 sets of 4-bit indices at 11008 x 4096 would take 6 GB).
constexpr size_t kPartBytes = size_t(512) << 20;

struct Layout {
  size_t perm, segs, dy, x, part, extra, total;
  int64_t rows;
  int sets;                // LUT sets per launch
};

size_t part_floats(int64_t n, int64_t d, int bits, int gpr) {
  return (size_t)gemm::tiles_of(d) * n * group_slots(d / gpr, gpr) * (1 << bits);
}

Layout layout(int64_t n, int64_t d, int bits, int gpr, int64_t T, int ntask, bool routed) {
  Layout l;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += pad256(bytes);
    return here;
  };
  l.rows = routed ? route_positions(T, ntask) : T;
  l.perm = take(routed ? (size_t)l.rows * 4 : 0);
  l.segs = take(routed ? (size_t)ntask * 8 : 0);
  l.dy = take(routed ? (size_t)l.rows * n * 2 : 0);
  l.x = take((size_t)l.rows * d * 2);
  const size_t one = part_floats(n, d, bits, gpr) * 4;
  l.sets = routed ? ntask : 1;
  if (routed && whole_groups(n, d, gpr, ntask)) {
    l.part = at;
  } else {
    const size_t fit = kPartBytes / one;
    if ((size_t)l.sets > fit) l.sets = fit < 1 ? 1 : (int)fit;
    l.part = take(l.sets * one);
  }
  // the parts of the cut round beyond each tile's first
  gemm::Shape shape = gemm::shape_of(n, d, T);
  gemm::split_last_round(shape);
  const int64_t parts = (int64_t)(shape.mt * shape.nt - shape.split_from) * (shape.split - 1);
  l.extra = take(routed ? 0 : (size_t)parts * gemm::TM * group_slots(d / gpr, gpr) * (1 << bits) * 4);
  l.total = at;
  return l;
}

// ----------------------------------------------------------------------------
// few tokens: CUDA cores, one warp per (row, group)
// ----------------------------------------------------------------------------

constexpr int kBlock = 128;

template <int BITS>
__global__ void __launch_bounds__(kBlock) lut8_simt_kernel(Problem p, const int8_t* __restrict__ q,
                                                           const uint8_t* __restrict__ scale,
                                                           const uint16_t* __restrict__ dY, float* __restrict__ dlut,
                                                           int accumulate) {
  constexpr int K = 1 << BITS;
  __shared__ float bins[K][kBlock];
  const int tid = threadIdx.x, lane = tid & 31;
  const int64_t wid = (int64_t)blockIdx.x * (kBlock / 32) + (tid >> 5);
  if (wid >= p.n * p.gpr) return;
  const int64_t i = wid / p.gpr, g = wid % p.gpr;
  const int64_t cpg = p.gs / 32, chunks = p.d / 32;
  // Of several sets a warp visits the tokens of each by ballots over 32 ids at a time,
  // so that what a set costs beside its own tokens is an id per lane and 32 tokens.
  // (A look at every token's id for every set: 9.7 ms for 64 tokens of 256 sets at
  // 4096 x 4096, 1.1 this way.)  Sets that no token names get zeros; without task ids every token
  // belongs to LUT set 0.
  const int own = p.task != nullptr && lane < p.T ? token_task(p.task, lane, p.ntask, p.check) : -1;
  auto named = [&](int64_t b, int tau) {               // tokens b .. b + 31 of the set
    const int id = b == 0 ? own : b + lane < p.T ? token_task(p.task, b + lane, p.ntask, p.check) : -1;
    return __ballot_sync(0xffffffffu, id == tau);
  };
  for (int tau = 0; tau < p.ntask; ++tau) {
    bool any = p.task == nullptr && tau == 0;
    if (p.task != nullptr)
      for (int64_t b = 0; b < p.T && !any; b += 32) any = named(b, tau) != 0u;
    if (!any) {
      if (lane < K && !accumulate) dlut[(((int64_t)tau * p.n + i) * p.gpr + g) * K + lane] = 0.f;
      continue;
    }
#pragma unroll
    for (int c = 0; c < K; ++c) bins[c][tid] = 0.f;
    for (int64_t c0 = 0; c0 < cpg; c0 += 32) {         // the whole warp: the ballots are its own
      const bool mine = c0 + lane < cpg;
      const int64_t chunk = g * cpg + (mine ? c0 + lane : 0);
      const Chunk<BITS> ch = load_chunk<BITS>(p.packed + i * p.row_bytes, chunk);
      float G[32];
#pragma unroll
      for (int e = 0; e < 32; ++e) G[e] = 0.f;
      auto add = [&](int64_t t) {
        const uint32_t s2 = __ldg(dY + t * p.n + i);
        const uint32_t sc = ckpt8_scale2(__ldg(scale + t * chunks + chunk));
        const uint4* xp = reinterpret_cast<const uint4*>(q + t * p.d + chunk * 32);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4 v = __ldg(xp + h);
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            uint32_t w0, w1;
            ckpt8_dequant4(w[b], sc, w0, w1);
            fma_bf16x2_scalar(w0, s2, G[16 * h + 4 * b + 0], G[16 * h + 4 * b + 1]);
            fma_bf16x2_scalar(w1, s2, G[16 * h + 4 * b + 2], G[16 * h + 4 * b + 3]);
          }
        }
      };
      if (p.task == nullptr) {
        if (mine)
          for (int64_t t = 0; t < p.T; ++t) add(t);
      } else {
        for (int64_t b = 0; b < p.T; b += 32)
          for (uint32_t left = named(b, tau); left != 0u && mine; left &= left - 1u) add(b + __ffs(left) - 1);
      }
      if (!mine) continue;
#pragma unroll
      for (int e = 0; e < 32; ++e) bins[chunk_index<BITS>(ch, e)][tid] += G[e];
    }
    // lane partial bins -> the warp's sums (fixed shuffle tree: deterministic)
    float mine = 0.f;
#pragma unroll
    for (int c = 0; c < K; ++c) {
      float v = bins[c][tid];
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
      if (lane == c) mine = v;
    }
    if (lane < K) {
      float* out = dlut + (((int64_t)tau * p.n + i) * p.gpr + g) * K + lane;
      *out = accumulate ? *out + mine : mine;
    }
  }
}

}  // namespace

size_t lut8_tc_workspace(int64_t n, int64_t d, int bits, int gpr, int64_t T, int ntask, bool routed) {
  return layout(n, d, bits, gpr, T, ntask, routed).total;
}

cudaError_t launch_lut8_tc(const Problem& p, const int8_t* q, const uint8_t* scale, const uint16_t* dY, float* dlut,
                           int accumulate, bool routed, void* workspace, cudaStream_t s) {
  cudaError_t e;
  const Layout l = layout(p.n, p.d, p.bits, p.gpr, p.T, p.ntask, routed);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  int* segs = nullptr;
  uint16_t* X = reinterpret_cast<uint16_t*>(ws + l.x);
  const uint16_t* a_rows = dY;
  if (routed) {
    int* perm = reinterpret_cast<int*>(ws + l.perm);
    segs = reinterpret_cast<int*>(ws + l.segs);
    uint16_t* g = reinterpret_cast<uint16_t*>(ws + l.dy);
    a_rows = g;
    lut8_route_kernel<<<1, kRouteThreads, 0, s>>>(p.task, (int)p.T, p.ntask, (int)l.rows, perm, segs, p.check);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    // one grid row per position, as many as a grid has
    const int64_t units = (p.n + p.d) / 8;
    for (int64_t r = 0; r < l.rows; r += 65535) {
      const int64_t rows = l.rows - r < 65535 ? l.rows - r : 65535;
      lut8_gather_kernel<<<dim3((unsigned)((units + 1023) / 1024), (unsigned)rows), 256, 0, s>>>(
          reinterpret_cast<const uint4*>(dY), reinterpret_cast<const uint2*>(q), scale, perm + r, p.n / 8, p.d / 8,
          reinterpret_cast<uint4*>(g + r * p.n), reinterpret_cast<uint4*>(X + r * p.d));
      if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
  } else {
    if ((e = launch_ckpt8_dequantize(q, scale, p.T, p.d, X, s)) != cudaSuccess) return e;
  }
  CUtensorMap tm_dy, tm_x;
  e = make_tmap_2d(&tm_dy, a_rows, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, (uint64_t)p.n, (uint64_t)l.rows,
                   (uint64_t)p.n * 2, 64, KS, CU_TENSOR_MAP_SWIZZLE_128B);
  if (e != cudaSuccess) return e;
  e = make_tmap_2d(&tm_x, X, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, (uint64_t)p.d, (uint64_t)l.rows, (uint64_t)p.d * 2, 64,
                   KS, CU_TENSOR_MAP_SWIZZLE_128B);
  if (e != cudaSuccess) return e;
  Lut8Args args{};
  args.shape = gemm::shape_of(p.n, p.d, p.T);
  if (!routed) gemm::split_last_round(args.shape);
  args.packed = p.packed;
  args.row_bytes = p.row_bytes;
  args.n = p.n;
  args.d = p.d;
  args.gs = p.gs;
  args.gpr = p.gpr;
  args.slots = group_slots(p.gs, p.gpr);
  args.part = reinterpret_cast<float*>(ws + l.part);
  args.part_set_stride = (int64_t)part_floats(p.n, p.d, p.bits, p.gpr);
  args.extra = reinterpret_cast<float*>(ws + l.extra);
  args.check = p.check;
  const int64_t per_set = p.n * p.gpr * (1 << p.bits);
  // without task ids the sets beyond the first have no tokens
  if (!routed && p.ntask > 1 && !accumulate) {
    e = cudaMemsetAsync(dlut + per_set, 0, (size_t)per_set * (p.ntask - 1) * 4, s);
    if (e != cudaSuccess) return e;
  }
  const bool grouped = routed && whole_groups(p.n, p.d, p.gpr, p.ntask);
  if (grouped) {
    args.per_group = (int)(p.gs / TN);
    args.accumulate = accumulate;
  }
  const bool cut = args.shape.split > 1;
  // a block of LUT sets; the next one's partial bins take the same room after it
  auto go = [&](auto bits, int first, int sets) {
    constexpr int B = decltype(bits)::value;
    args.sets = sets;
    args.segs = routed ? segs + 2 * first : nullptr;
    args.dlut = dlut + first * per_set;
    const int64_t count = grouped  ? (int64_t)sets * p.gpr * args.shape.mt
                          : routed ? (int64_t)sets * args.shape.mt * args.shape.nt
                                   : gemm::items(args.shape);
    cudaError_t err = gemm::launch_pairs<8, stages(B)>(lut8_tc_kernel<B>, count, s, tm_dy, tm_x, args);
    if (err != cudaSuccess || grouped) return err;
    const int64_t quads = per_set * sets / 4;
    const unsigned grid = (unsigned)((quads + 255) / 256);
    float4* out = reinterpret_cast<float4*>(args.dlut);
    if (cut) lut8_reduce_kernel<B, true><<<grid, 256, 0, s>>>(args, out, accumulate, quads);
    else lut8_reduce_kernel<B, false><<<grid, 256, 0, s>>>(args, out, accumulate, quads);
    return cudaGetLastError();
  };
  const int all = routed ? p.ntask : 1;
  for (int first = 0; first < all; first += l.sets) {
    const int sets = all - first < l.sets ? all - first : l.sets;
    switch (p.bits) {
      case 2: e = go(std::integral_constant<int, 2>(), first, sets); break;
      case 3: e = go(std::integral_constant<int, 3>(), first, sets); break;
      default: e = go(std::integral_constant<int, 4>(), first, sets); break;
    }
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_lut8_simt(const Problem& p, const int8_t* q, const uint8_t* scale, const uint16_t* dY, float* dlut,
                             int accumulate, cudaStream_t s) {
  const unsigned grid = (unsigned)((p.n * p.gpr + kBlock / 32 - 1) / (kBlock / 32));
  switch (p.bits) {
    case 2: lut8_simt_kernel<2><<<grid, kBlock, 0, s>>>(p, q, scale, dY, dlut, accumulate); break;
    case 3: lut8_simt_kernel<3><<<grid, kBlock, 0, s>>>(p, q, scale, dY, dlut, accumulate); break;
    default: lut8_simt_kernel<4><<<grid, kBlock, 0, s>>>(p, q, scale, dY, dlut, accumulate); break;
  }
  return cudaGetLastError();
}

}  // namespace sk
