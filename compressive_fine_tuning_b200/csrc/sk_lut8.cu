// LUT gradient of the sketched linear layer from an 8-bit activation checkpoint:
//
//   dlut[s][i][g][c] = sum over the tokens t of set s and the columns j of group g
//                      with idx[i][j] = c of dY[t][i] * q[t][j] * 2^e[t][j / 32]
//
// i.e. the corrected Eq. 6 of the "Sketch to Adapt" OpenReview discussion (reply
// Q1) with X as the checkpoint holds it (format in sk_ckpt8.cuh).
//
// Tensor cores: the G tile [256 rows i x 256 columns j] = dY^T X over K = tokens
// on a CTA pair, binned by the epilogue into (group, centroid) sums that never
// leave the SM as a dense gradient.  dY comes by TMA.  X is dequantised on its
// way into shared memory: a warp owns eight tokens of every 64-token step, a
// lane one token's 32-column block, i.e. 32 bytes and one scale byte, loaded a
// step ahead, so the checkpoint is read at 33/64 of the bytes of a bf16 X and no
// bf16 copy of it ever exists in memory.  q * 2^e is exact in bf16, so the
// products are those of the stored values, accumulated in fp32.
// The bound is the tensor pipe (2 T n d flops).
#include "sk_lut8.cuh"
#include "sk_tc.cuh"

namespace sk {
namespace {

constexpr int KS = 64;                 // tokens per pipeline step
constexpr int N = 256;                 // columns per tile
constexpr int A_BYTES = 2 * 8192;      // this CTA's 128 rows of dY^T: two 64-row MN atoms
constexpr int B_BYTES = 2 * 8192;      // this CTA's 128 columns of X: two 64-column MN atoms
constexpr int STAGE = A_BYTES + B_BYTES;
constexpr int S = 3;                   // two CTAs per SM: one bins while the other multiplies
constexpr int BAR_OFF = S * STAGE;
constexpr int SMEM = 1024 + BAR_OFF + 256;
constexpr int PRODUCERS = 8, TMA_WARP = 8, MMA_WARP = 9, THREADS = 320;
constexpr uint32_t IDESC = tc::idesc_bf16(256, N, 1, 1);
constexpr int TMEM_COLS = 256;
constexpr int COPIES = 4;             // copies of the bins in the epilogue
static_assert(PRODUCERS * 8 == KS, "a producer warp fills one K-group of eight tokens");

__host__ __device__ constexpr int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

// Group slots of one 256-column tile.
__host__ __device__ inline int group_slots(int64_t gs, int gpr) {
  const int64_t s = 255 / gs + 2;
  return (int)(s < gpr ? s : gpr);
}

struct Lut8Args {
  const uint8_t* packed;
  int64_t row_bytes;
  const int8_t* q;
  const uint8_t* scale;
  int64_t n, d, gs, T;
  int gpr, slots;
  float* part;               // [sets][jtiles][n][slots][k] partial bins
  int64_t part_set_stride;
  unsigned int* check;
  // several LUT sets: dY rows in task order, set z's tokens at positions
  // [segs[2z], segs[2z] + segs[2z + 1]) (64-aligned, zero rows between), perm
  // maps a position to its token; nullptr for one LUT set
  const int* segs;
  const int* perm;
  int row_pairs;
};

template <int BITS, bool ROUTED>
__global__ void __launch_bounds__(THREADS, 2) lut8_tc_kernel(const __grid_constant__ CUtensorMap tm_dy, Lut8Args a) {
  constexpr int K = 1 << BITS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full_a = reinterpret_cast<uint64_t*>(smem + BAR_OFF);  // even CTA: both CTAs' dY landed
  uint64_t* full_b = full_a + S;                                    // even CTA: both CTAs' X tiles written
  uint64_t* empty = full_b + S;                                     // both CTAs: the pair MMAs read the stage
  uint64_t* d_full = empty + S;                                     // both CTAs: accumulator final
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(d_full + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = tc::warp_id(), lane = tc::lane_id();
  const uint32_t rank = tc::cluster_ctarank();                      // 0: issues the MMAs
  // grid: (pair, column tile, row block + row_pairs * LUT set), column tiles fastest after the pair
  const int jt = blockIdx.y;
  const int64_t j0 = (int64_t)jt * N;
  const int set = (int)blockIdx.z / a.row_pairs;
  const int64_t i0 = (int64_t)((int)blockIdx.z - set * a.row_pairs) * 256 + 128 * rank;
  int k_first = 0;
  int tokens = (int)a.T;
  if constexpr (ROUTED) {
    k_first = a.segs[2 * set];
    tokens = a.segs[2 * set + 1];
  }
  const int nsteps = ceil_div(tokens, KS);      // a set with no tokens writes zero partials
  float* part = a.part + (int64_t)set * a.part_set_stride;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      tc::mbar_init(&full_a[s], 1);
      tc::mbar_init(&full_b[s], 2 * PRODUCERS);
      tc::mbar_init(&empty[s], 1);
    }
    tc::mbar_init(d_full, 1);
    *abort_flag = 0;
    tc::fence_mbar_init();
  }
  if (warp == MMA_WARP) tc::tmem_alloc_pair(tmem_slot, TMEM_COLS);
  if (warp == TMA_WARP && lane == 0) tc::tma_prefetch(&tm_dy);
  tc::tc_fence_before();
  // both CTAs' barriers are initialised before either CTA signals the other
  tc::cluster_sync_all();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == TMA_WARP) {
    if (lane == 0) {
      int issued = 0;
      for (int i = 0; i < nsteps && !*abort_flag; ++i) {
        const int s = i % S;
        if (!tc::mbar_wait(&empty[s], ((i / S) & 1) ^ 1, a.check)) { *abort_flag = 1; break; }
        uint8_t* st = smem + s * STAGE;
        if (rank == 0) tc::mbar_arrive_expect_tx(&full_a[s], 2 * A_BYTES);   // the bytes of both CTAs
        const uint32_t bar = tc::mapa(&full_a[s], 0);
        const int tk = k_first + i * KS;
        tc::tma_load_2d_pair(st, &tm_dy, bar, (int)i0, tk);
        tc::tma_load_2d_pair(st + 8192, &tm_dy, bar, (int)i0 + 64, tk);
        ++issued;
      }
      // never leave with a copy still landing in shared memory: the pair MMAs
      // read every landed stage before they free it
      bool ok = true;
      for (int k = issued > S ? issued - S : 0; k < issued && ok; ++k)
        ok = tc::mbar_wait(&empty[k % S], (k / S) & 1, a.check);
    }
  } else if (warp == MMA_WARP) {
    if (rank == 0 && lane == 0) {
      bool ok = true;
      for (int i = 0; i < nsteps; ++i) {
        const int s = i % S;
        if (*abort_flag || !tc::mbar_wait(&full_a[s], (i / S) & 1, a.check) ||
            !tc::mbar_wait(&full_b[s], (i / S) & 1, a.check)) {
          *abort_flag = 1; ok = false; break;
        }
        tc::tc_fence_after();
        const uint32_t ab = tc::smem_u32(smem + s * STAGE), bb = ab + A_BYTES;
#pragma unroll
        for (int kk = 0; kk < KS / 16; ++kk) {
          const uint64_t ad = tc::sdesc(ab + kk * 2048, 8192, 1024, tc::kSwizzle128);
          const uint64_t bd = tc::sdesc(bb + kk * 2048, 8192, 1024, tc::kSwizzle128);
          tc::mma_ss_pair(tmem, ad, bd, IDESC, (i > 0 || kk > 0) ? 1u : 0u);
        }
        tc::mma_commit_pair(&empty[s]);
      }
      if (ok) tc::mma_commit_pair(d_full);
    }
  } else {
    // producers: lane (r8, h) of warp w dequantises token 8 w + r8 of the step,
    // columns 32 h .. 32 h + 31 of this CTA's 128
    const int r8 = lane & 7, h = lane >> 3;
    const int lr = 8 * warp + r8;
    // the epilogue warps' row indices of this column tile, loaded while the MMAs
    // run so that their memory latency is off the binning loop
    const int64_t row_i = i0 + threadIdx.x;
    Chunk<BITS> chunks[N / 32] = {};
    if (warp < 4 && row_i < a.n) {
#pragma unroll
      for (int b = 0; b < N / 32; ++b)
        if (j0 + 32 * b < a.d) chunks[b] = load_chunk<BITS>(a.packed + row_i * a.row_bytes, (j0 >> 5) + b);
    }
    const int64_t j = j0 + 128 * rank + 32 * h;
    const bool col_ok = j < a.d;
    const int64_t sblocks = a.d >> 5;
    uint32_t slot_off[4];              // 16-byte swizzled slots of the block's four bf16 quarters
#pragma unroll
    for (int e = 0; e < 4; ++e)
      slot_off[e] = (h >> 1) * 8192 + warp * 1024 + r8 * 128 + (((4 * (h & 1) + e) ^ r8) << 4);
    // 32 bytes and a scale byte per step, loaded two steps ahead; a position's
    // token (one LUT set: the position itself) is known one step before that
    const int8_t* q_col = a.q + j;
    const uint8_t* s_col = a.scale + (j >> 5);
    auto token_of = [&](int i) -> int {
      const int t = i * KS + lr;
      if (t >= tokens || !col_ok) return -1;
      return ROUTED ? __ldg(a.perm + k_first + t) : t;
    };
    struct Block {
      uint4 q0, q1;
      uint32_t byte;
    };
    auto fetch = [&](int t) -> Block {
      Block b{make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u), 0u};   // zero scale: the tile's padding is zero
      if (t >= 0) {
        const uint4* src = reinterpret_cast<const uint4*>(q_col + (int64_t)t * a.d);
        b.q0 = __ldg(src);
        b.q1 = __ldg(src + 1);
        b.byte = __ldg(s_col + (int64_t)t * sblocks);
      }
      return b;
    };
    Block ahead[2] = {fetch(token_of(0)), fetch(token_of(1))};
    int tok = token_of(2);
    const uint32_t full_b_even = tc::mapa(&full_b[0], 0);
    bool ok = true;
#pragma unroll 1
    for (int i0s = 0; i0s < nsteps && ok; i0s += 2) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int i = i0s + half;
        if (i >= nsteps || !ok) break;
        const Block cur = ahead[half];
        ahead[half] = fetch(tok);
        tok = token_of(i + 3);
        const uint32_t s2 = ckpt8_scale2(cur.byte);
        uint4 o[4];
        ckpt8_dequant4(cur.q0.x, s2, o[0].x, o[0].y);
        ckpt8_dequant4(cur.q0.y, s2, o[0].z, o[0].w);
        ckpt8_dequant4(cur.q0.z, s2, o[1].x, o[1].y);
        ckpt8_dequant4(cur.q0.w, s2, o[1].z, o[1].w);
        ckpt8_dequant4(cur.q1.x, s2, o[2].x, o[2].y);
        ckpt8_dequant4(cur.q1.y, s2, o[2].z, o[2].w);
        ckpt8_dequant4(cur.q1.z, s2, o[3].x, o[3].y);
        ckpt8_dequant4(cur.q1.w, s2, o[3].z, o[3].w);
        const int s = i % S;
        if (*abort_flag || !tc::mbar_wait(&empty[s], ((i / S) & 1) ^ 1, a.check)) { *abort_flag = 1; ok = false; break; }
        uint8_t* bt = smem + s * STAGE + A_BYTES;
#pragma unroll
        for (int e = 0; e < 4; ++e) *reinterpret_cast<uint4*>(bt + slot_off[e]) = o[e];
        tc::fence_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive_cluster(full_b_even + 8 * s);
      }
    }
    if (warp < 4) {
      // epilogue: thread = row i (TMEM lane); bin the row's 256 columns
      __syncwarp();
      // [COPIES][K][128], tail of stage memory: consecutive columns add into different
      // copies, so their loads do not wait for one another's stores
      float* bins = reinterpret_cast<float*>(smem + BAR_OFF - COPIES * K * 128 * 4) + threadIdx.x;
      bool have = !*abort_flag && tc::mbar_wait(d_full, 0, a.check) && nsteps > 0;   // no steps: nothing accumulated
      have = __all_sync(0xffffffffu, have);  // tcgen05.ld is warp-collective
      if (have) tc::tc_fence_after();
      // the bins reuse the last stages' memory: every MMA has read it (d_full)
#pragma unroll
      for (int c = 0; c < COPIES * K; ++c) bins[c * 128] = 0.f;
      const int first_g = (int)(j0 / a.gs);
      const int gs32 = (int)a.gs;
      int g = first_g, g_end = (first_g + 1) * gs32;
      bool dirty = false;
      auto flush = [&](int gg) {
        float4* dst = reinterpret_cast<float4*>(part + (((int64_t)jt * a.n + row_i) * a.slots + (gg - first_g)) * K);
#pragma unroll
        for (int c4 = 0; c4 < K / 4; ++c4) {
          float v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int c = 4 * c4 + e;
            v[e] = bins[c * 128];
            bins[c * 128] = 0.f;
#pragma unroll
            for (int k = 1; k < COPIES; ++k) {
              v[e] += bins[(k * K + c) * 128];
              bins[(k * K + c) * 128] = 0.f;
            }
          }
          if (row_i < a.n) dst[c4] = make_float4(v[0], v[1], v[2], v[3]);
        }
      };
#pragma unroll
      for (int b = 0; b < N / 32; ++b) {
        const int64_t jc = j0 + 32 * b;
        if (jc >= a.d) break;
        uint32_t v[32];
        if (have) {
          tc::tmem_ld32(tc::tmem_addr(tmem, warp * 32, 32 * b), v);
          tc::tmem_ld_wait();
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = 0u;
        }
        if ((int)jc >= g_end) {       // chunk in a later group: hand the finished group's sums on
          if (dirty) flush(g);
          do { ++g; g_end += gs32; } while ((int)jc >= g_end);
          dirty = false;
        }
#pragma unroll
        for (int e = 0; e < 32; e += COPIES) {
          float* at[COPIES];
          float sum[COPIES];
#pragma unroll
          for (int k = 0; k < COPIES; ++k) {
            at[k] = bins + (k * K + chunk_index<BITS>(chunks[b], e + k)) * 128;
            sum[k] = *at[k];
          }
#pragma unroll
          for (int k = 0; k < COPIES; ++k) *at[k] = sum[k] + __uint_as_float(v[e + k]);
        }
        dirty = true;
      }
      if (dirty) flush(g);
    }
  }

  tc::tc_fence_before();
  __syncthreads();
  // neither CTA leaves (or frees tensor memory) while the other may still
  // signal its barriers or the pair MMAs may still use its memory
  tc::cluster_sync_all();
  if (warp == MMA_WARP) {
    tc::tc_fence_after();
    tc::tmem_dealloc_pair(tmem, TMEM_COLS);
  }
}

// Sum the partial bins of every (set, row, group) over the column tiles that
// touch the group, in tile order, and write (or add to) dlut: four bins a thread.
template <int BITS>
__global__ void __launch_bounds__(256) lut8_reduce_kernel(const float4* __restrict__ part, int64_t n, int gpr, int64_t gs,
                                                          int jtiles, int slots, float4* __restrict__ dlut,
                                                          int accumulate, int64_t total, int64_t part_set_stride) {
  constexpr int Q = (1 << BITS) / 4;
  const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (e >= total) return;
  const int c = (int)(e % Q);
  const int64_t ig = e / Q;
  const int g = (int)(ig % gpr);
  const int64_t si = ig / gpr, set = si / n, i = si - set * n;
  part += set * part_set_stride;
  const int t_first = (int)(((int64_t)g * gs) / N);
  int t_last = (int)(((int64_t)(g + 1) * gs - 1) / N);
  if (t_last > jtiles - 1) t_last = jtiles - 1;
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int t = t_first; t <= t_last; ++t) {
    // only a group's first tile can start in an earlier group
    const int slot = t == t_first ? g - (int)(((int64_t)t * N) / gs) : 0;
    const float4 v = __ldg(part + (((int64_t)t * n + i) * slots + slot) * Q + c);
    sum = make_float4(sum.x + v.x, sum.y + v.y, sum.z + v.z, sum.w + v.w);
  }
  if (accumulate) {
    const float4 o = dlut[e];
    sum = make_float4(o.x + sum.x, o.y + sum.y, o.z + sum.z, o.w + sum.w);
  }
  dlut[e] = sum;
}

// ----------------------------------------------------------------------------
// tokens by LUT set, in token order
// ----------------------------------------------------------------------------

constexpr int kRouteThreads = 1024;

// One CTA: count every set's tokens, lay the segments out at multiples of KS,
// then place the tokens tile by tile (one per thread): a token's position is
// its set's running offset plus its rank among the set's tokens of the tile
// (earlier warps' counts, then the lanes before it), so the order within a set
// is the token order and sums over it never depend on timing.
__global__ void __launch_bounds__(kRouteThreads) lut8_route_kernel(const int32_t* __restrict__ task, int T, int ntask,
                                                                   int positions, int* __restrict__ perm,
                                                                   int* __restrict__ segs, unsigned int* check) {
  __shared__ int cur[kMaxRouteTasks];
  __shared__ uint16_t per_warp[32][kMaxRouteTasks];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (int i = tid; i < ntask; i += kRouteThreads) cur[i] = 0;
  for (int p = tid; p < positions; p += kRouteThreads) perm[p] = -1;
  __syncthreads();
  for (int t = tid; t < T; t += kRouteThreads) {
    const int tau = task[t];
    if (tau >= 0 && tau < ntask) atomicAdd(&cur[tau], 1);
    else atomicOr(check, SK_CHECK_TASK_RANGE);   // left out of every LUT set's gradient
  }
  __syncthreads();
  if (tid == 0) {
    int at = 0;
    for (int tau = 0; tau < ntask; ++tau) {
      const int c = cur[tau];
      segs[2 * tau] = at;
      segs[2 * tau + 1] = c;
      cur[tau] = at;
      at += (c + KS - 1) / KS * KS;
    }
  }
  for (int base = 0; base < T; base += kRouteThreads) {
    for (int i = tid; i < 32 * kMaxRouteTasks; i += kRouteThreads) (&per_warp[0][0])[i] = 0;
    __syncthreads();
    const int t = base + tid;
    int tau = t < T ? task[t] : -1;
    if (tau < 0 || tau >= ntask) tau = -1;
    const uint32_t same = __match_any_sync(0xffffffffu, tau);
    const int before = __popc(same & ((1u << lane) - 1u));
    if (tau >= 0 && before == 0) per_warp[warp][tau] = (uint16_t)__popc(same);
    __syncthreads();
    if (tau >= 0) {
      int p = cur[tau] + before;
      for (int w = 0; w < warp; ++w) p += per_warp[w][tau];
      perm[p] = t;
    }
    __syncthreads();
    for (int i = tid; i < ntask; i += kRouteThreads) {
      int c = 0;
      for (int w = 0; w < 32; ++w) c += per_warp[w][i];
      cur[i] += c;
    }
    __syncthreads();
  }
}

__global__ void lut8_gather_kernel(const uint4* __restrict__ src, const int* __restrict__ perm, int positions,
                                   int64_t units, uint4* __restrict__ dst) {
  const int64_t e = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (e >= (int64_t)positions * units) return;
  const int64_t p = e / units, u = e - p * units;
  const int t = perm[p];
  dst[e] = t >= 0 ? __ldg(src + (int64_t)t * units + u) : make_uint4(0u, 0u, 0u, 0u);
}

int route_positions(int64_t T, int ntask) { return (int)(T + (int64_t)ntask * (KS - 1)); }

size_t route_bytes(int64_t n, int64_t T, int ntask) {
  const int64_t pos = route_positions(T, ntask);
  return ((size_t)(pos + 2 * ntask) * 4 + 255) / 256 * 256 + ((size_t)pos * n * 2 + 255) / 256 * 256;
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
  for (int tau = 0; tau < p.ntask; ++tau) {
#pragma unroll
    for (int c = 0; c < K; ++c) bins[c][tid] = 0.f;
    // without task ids every token belongs to LUT set 0; the other sets get zeros
    if (p.task != nullptr || tau == 0) {
      for (int64_t cc = lane; cc < cpg; cc += 32) {
        const int64_t chunk = g * cpg + cc;
        const Chunk<BITS> ch = load_chunk<BITS>(p.packed + i * p.row_bytes, chunk);
        float G[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) G[e] = 0.f;
        for (int64_t t = 0; t < p.T; ++t) {
          if (p.task != nullptr && token_task(p.task, t, p.ntask, p.check) != tau) continue;
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
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) bins[chunk_index<BITS>(ch, e)][tid] += G[e];
      }
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

size_t part_floats(int64_t n, int64_t d, int bits, int gpr) {
  return (size_t)ceil_div(d, N) * n * group_slots(d / gpr, gpr) * (1 << bits);
}

}  // namespace

size_t lut8_tc_workspace(int64_t n, int64_t d, int bits, int gpr, int64_t T, int ntask, bool routed) {
  const size_t part = part_floats(n, d, bits, gpr) * sizeof(float);
  return routed ? route_bytes(n, T, ntask) + (size_t)ntask * part : part;
}

cudaError_t launch_lut8_tc(const Problem& p, const int8_t* q, const uint8_t* scale, const uint16_t* dY, float* dlut,
                           int accumulate, bool routed, void* workspace, cudaStream_t s) {
  cudaError_t e;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const int sets = routed ? p.ntask : 1;
  const int *segs = nullptr, *perm = nullptr;
  const uint16_t* a_rows = dY;
  uint64_t rows = (uint64_t)p.T;
  if (routed) {
    const int pos = route_positions(p.T, p.ntask);
    int* pm = reinterpret_cast<int*>(ws);
    int* sg = pm + pos;
    uint16_t* g = reinterpret_cast<uint16_t*>(ws + ((size_t)(pos + 2 * p.ntask) * 4 + 255) / 256 * 256);
    lut8_route_kernel<<<1, kRouteThreads, 0, s>>>(p.task, (int)p.T, p.ntask, pos, pm, sg, p.check);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int64_t units = p.n / 8, total = (int64_t)pos * units;
    lut8_gather_kernel<<<(unsigned)((total + 255) / 256), 256, 0, s>>>(reinterpret_cast<const uint4*>(dY), pm, pos, units,
                                                                       reinterpret_cast<uint4*>(g));
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    segs = sg;
    perm = pm;
    a_rows = g;
    rows = (uint64_t)pos;
    ws += route_bytes(p.n, p.T, p.ntask);
  }
  CUtensorMap tm;
  e = make_tmap_2d(&tm, a_rows, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, (uint64_t)p.n, rows, (uint64_t)p.n * 2, 64, KS,
                   CU_TENSOR_MAP_SWIZZLE_128B);
  if (e != cudaSuccess) return e;
  const int slots = group_slots(p.gs, p.gpr), jtiles = ceil_div(p.d, N), pairs = ceil_div(p.n, 256);
  const int64_t stride = (int64_t)part_floats(p.n, p.d, p.bits, p.gpr);
  float* part = reinterpret_cast<float*>(ws);
  Lut8Args args{p.packed, p.row_bytes, q, scale, p.n, p.d, p.gs, p.T, p.gpr, slots, part, stride, p.check,
                segs, perm, pairs};
  const int64_t per_set = p.n * p.gpr * (1 << p.bits);
  // without task ids the sets beyond the first have no tokens
  const int64_t total = per_set * sets;
  if (!routed && p.ntask > 1 && !accumulate) {
    e = cudaMemsetAsync(dlut + per_set, 0, (size_t)per_set * (p.ntask - 1) * 4, s);
    if (e != cudaSuccess) return e;
  }
  auto run = [&](auto kern, auto red) {
    cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2u, (unsigned)jtiles, (unsigned)(pairs * sets));
    cfg.blockDim = dim3(THREADS, 1, 1);
    cfg.dynamicSmemBytes = SMEM;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    err = cudaLaunchKernelEx(&cfg, kern, tm, args);
    if (err != cudaSuccess) return err;
    const int64_t quads = total / 4;
    red<<<(unsigned)((quads + 255) / 256), 256, 0, s>>>(reinterpret_cast<const float4*>(part), p.n, p.gpr, p.gs, jtiles,
                                                        slots, reinterpret_cast<float4*>(dlut), accumulate, quads,
                                                        stride / 4);
    return cudaGetLastError();
  };
  switch (p.bits) {
    case 2: return routed ? run(lut8_tc_kernel<2, true>, lut8_reduce_kernel<2>) : run(lut8_tc_kernel<2, false>, lut8_reduce_kernel<2>);
    case 3: return routed ? run(lut8_tc_kernel<3, true>, lut8_reduce_kernel<3>) : run(lut8_tc_kernel<3, false>, lut8_reduce_kernel<3>);
    default: return routed ? run(lut8_tc_kernel<4, true>, lut8_reduce_kernel<4>) : run(lut8_tc_kernel<4, false>, lut8_reduce_kernel<4>);
  }
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
