// Persistent bf16 matrix product on CTA pairs, C[M][N] = A B^T over K, with the
// epilogue left to the caller.
//
// A pair of CTAs (cta_group::2) owns a 256 x 256 tile: each CTA loads its own
// 128 rows of A and half of B's 256 rows per 64-deep K step (32 KB, TMA, 128-byte
// swizzle), the even CTA issues M = 256, N = 256 MMAs, and each CTA holds 128 rows
// of the accumulator.  Two accumulators of 256 TMEM columns take turns, so the
// four epilogue warps drain one tile while the next one's MMAs run: the tensor
// pipe only ever waits for operands.  One CTA per SM, the pairs walk the tiles
// in a fixed order.  Either operand may be K-major (row = M or N index, K
// contiguous) or MN-major (row = K index, M or N contiguous).
#pragma once

#include "sk_tc.cuh"

namespace sk {
namespace gemm {

constexpr int TM = 256, TN = 256, KS = 64;
constexpr int A_BYTES = 128 * KS * 2, B_BYTES = 128 * KS * 2, STAGE = A_BYTES + B_BYTES;
constexpr int SLAB = 32 * 128;                    // one warp's output slab: 32 rows x 128 bytes
constexpr int TMEM_COLS = 512;
constexpr int kVoteBar = 8;                       // named barriers of a team's common decision

// S full stages of operands; the rest of the CTA's shared memory is the epilogue's.
// Narrower tiles have smaller stages, and more of them in the same memory.  (An MMA
// reads 128 rows of A whatever a_rows is: what follows the rows in shared memory,
// the last stage's scratch among it, lands in accumulator rows nobody looks at.)
constexpr int MAX_STAGES = 14;
template <int S>
struct Smem {
  static constexpr int SCRATCH_OFF = S * STAGE, SCRATCH = (7 - S) * STAGE;
  static constexpr int BAR_OFF = SCRATCH_OFF + SCRATCH, BYTES = 1024 + BAR_OFF + 512;
  static_assert(BYTES <= 232448, "one CTA's shared memory");
};

// EW epilogue warps (4 or 8: warps w and w + 4 see the same accumulator rows),
// then one warp for the copies and one for the MMAs.
__host__ __device__ constexpr int threads(int ew) { return 32 * (ew + 2); }

struct Item {
  int m, n, k0, k1;      // tile, and the K steps [k0, k1) that it sums (none: see Epi)
  int part;              // -1: a whole tile
};

struct Shape {
  int mt, nt, ksteps;    // tiles and K steps
  int M;                 // rows of A: a CTA whose rows all lie beyond them loads none
  int a_rows;            // rows of A per CTA and tile: 128, or fewer (a multiple of 8) for a K-major A
  int tn;                // columns per tile: 256, or less for a K-major B (a multiple of 32)
  int group;             // M tiles walked together (see tile_at)
  // The last wave: the `split_from`-th and later tiles are cut along K into `split`
  // parts, one per pair, so that a few left-over tiles do not keep one pair each
  // busy for a whole tile while the others idle.  A part's accumulator goes to the
  // epilogue with its index; the caller joins the parts.
  int split_from, split;
};

__host__ __device__ inline int items(const Shape& s) {
  return s.split_from + (s.mt * s.nt - s.split_from) * s.split;
}

// Tiles in bands of `group` M tiles, N outside and M inside a band: the pairs in
// flight share a few B tiles and one band of A.
__host__ __device__ inline void tile_at(const Shape& s, int i, int& m, int& n) {
  const int per = s.group * s.nt;
  const int band = i / per, r = i - band * per;
  const int left = s.mt - band * s.group;
  const int rows = left < s.group ? left : s.group;
  n = r / rows;
  m = band * s.group + (r - n * rows);
}

// the inverse of tile_at
__host__ __device__ inline int tile_index(const Shape& s, int m, int n) {
  const int band = m / s.group, left = s.mt - band * s.group;
  const int rows = left < s.group ? left : s.group;
  return band * s.group * s.nt + n * rows + (m - band * s.group);
}

__device__ __forceinline__ Item item_at(const Shape& s, int i) {
  Item it;
  it.k0 = 0;
  it.k1 = s.ksteps;
  it.part = -1;
  int tile = i;
  if (i >= s.split_from && s.split > 1) {
    it.part = i - s.split_from;
    const int q = it.part % s.split;
    tile = s.split_from + it.part / s.split;
    it.k0 = (int)((int64_t)s.ksteps * q / s.split);
    it.k1 = (int)((int64_t)s.ksteps * (q + 1) / s.split);
  }
  tile_at(s, tile, it.m, it.n);
  return it;
}

// Output rows staged by one warp: 32 rows x 64 16-bit values in the 128-byte
// swizzle, written out by one TMA store per slab (which clips what lies outside
// the matrix).  Slabs alternate; a slab is written again only after the store
// before the last one has read it.
struct SlabWriter {
  int at = 0;
  __device__ __forceinline__ void put(uint8_t* scratch, const CUtensorMap* map, const uint32_t (&w)[32], int x, int y,
                                      int warp, int lane) {
    uint8_t* slab = scratch + (2 * warp + (at & 1)) * SLAB;
    ++at;
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
    __syncwarp();
#pragma unroll
    for (int q = 0; q < 8; ++q)
      *reinterpret_cast<uint4*>(slab + lane * 128 + ((q ^ (lane & 7)) << 4)) =
          make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
    tc::fence_async_smem();
    __syncwarp();
    if (lane == 0) {
      asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];"
                   ::"l"(reinterpret_cast<uint64_t>(map)), "r"(tc::smem_u32(slab)), "r"(x), "r"(y) : "memory");
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
  }
  // before the CTA leaves: every store has read its slab
  __device__ __forceinline__ void drain(int lane) {
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
};

// The items of one product.  Another plan has the same members.
struct Plan {
  const Shape& s;
  __device__ __forceinline__ const Shape& shape() const { return s; }
  __device__ __forceinline__ int count() const { return items(s); }
  __device__ __forceinline__ Item item(int i) const { return item_at(s, i); }
};

// Epi: struct with
//   static constexpr int kTeam
// the number of warps that meet at barriers in tile() (named ones below kVoteBar): 1 if
// none do, 2 for the warps w and w + 4, or all; and, for every epilogue warp,
//   void start(int warp, int lane, uint8_t* scratch)
// once, and for every item
//   void ready(const Item&, int m0, int n0, int warp, int lane)
// while the item before it is still to be done (loads that the tile will need),
//   void tile(uint32_t tmem, int m0, int n0, const Item&, int warp, int lane, uint8_t* scratch)
// when it is final: the warp's accumulator rows are m0 + 32 (warp % 4) + lane (TMEM
// lanes), columns n0 .. n0 + tn - 1; an item without K steps has no accumulator.
//   void take()
// between an item's ready() and its tile(): what ready() loaded is now the tile's,
// and the next ready() follows;
//   void done(int lane)
// once, before the CTA leaves.  `scratch` is the shared memory that the epilogue has
// to itself (32 KB with six stages, 64 KB with five).
template <int A_MN, int B_MN, int EW, int S, class P, class Epi>
__device__ __forceinline__ void run(const CUtensorMap* tm_a, const CUtensorMap* tm_b, const P& plan, Epi& epi,
                                    unsigned int* check) {
  constexpr int TMA_WARP = EW, MMA_WARP = EW + 1;
  const int tn = B_MN ? TN : plan.shape().tn, half_n = tn / 2;
  const int a_rows = A_MN ? 128 : plan.shape().a_rows;
  const int a_bytes = a_rows * KS * 2, b_bytes = half_n * KS * 2, stage = a_bytes + b_bytes;
  const int stages = min(MAX_STAGES, S * STAGE / stage);
  const uint32_t idesc = tc::idesc_bf16(TM, tn, A_MN, B_MN);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Smem<S>::BAR_OFF);   // even CTA: both CTAs' operands landed
  uint64_t* empty = full + MAX_STAGES;                             // both CTAs: the pair MMAs read the stage
  uint64_t* acc_full = empty + MAX_STAGES;                                  // both CTAs: accumulator b final
  uint64_t* acc_empty = acc_full + 2;                              // even CTA: both CTAs drained accumulator b
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = tc::warp_id(), lane = tc::lane_id();
  const int rank = (int)tc::cluster_ctarank();                     // 0: issues the MMAs
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int count = plan.count();

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      tc::mbar_init(&full[s], 1);
      tc::mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(&acc_full[b], 1);
      tc::mbar_init(&acc_empty[b], 2 * EW);
    }
    *abort_flag = 0;
    tc::fence_mbar_init();
  }
  if (warp == MMA_WARP) tc::tmem_alloc_pair(tmem_slot, TMEM_COLS);
  if (warp == TMA_WARP && lane == 0) {
    tc::tma_prefetch(tm_a);
    tc::tma_prefetch(tm_b);
  }
  tc::tc_fence_before();
  // both CTAs' barriers are initialised before either CTA signals the other
  tc::cluster_sync_all();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == TMA_WARP) {
    if (lane == 0) {
      int s = 0, filled = 0;            // the slot, and how many have been filled so far (at most `stages`)
      uint32_t phase = 1;               // of the wait for an empty slot: the first round's pass at once
      Item next = pair < count ? plan.item(pair) : Item{};
      for (int i = pair; i < count && !*abort_flag; i += pairs) {
        const Item w = next;
        if (i + pairs < count) next = plan.item(i + pairs);   // its arithmetic under this item's waits
        const int m0 = (2 * w.m + rank) * a_rows, n0 = w.n * tn + half_n * rank;
        // rows beyond A are not loaded: what they multiply is never looked at
        const bool odd_a = (2 * w.m + 1) * a_rows < plan.shape().M, load_a = rank == 0 || odd_a;
        const uint32_t bytes = (odd_a ? 2 : 1) * a_bytes + 2 * b_bytes;        // both CTAs' operands of a step
        for (int k = w.k0; k < w.k1; ++k) {
          if (!tc::mbar_wait(&empty[s], phase, check)) { *abort_flag = 1; break; }
          uint8_t* a = smem + s * stage;
          uint8_t* b = a + a_bytes;
          if (rank == 0) tc::mbar_arrive_expect_tx(&full[s], bytes);
          const uint32_t bar = tc::mapa(&full[s], 0);
          if (load_a) {
            if (A_MN) {
              tc::tma_load_2d_pair(a, tm_a, bar, m0, k * KS);
              tc::tma_load_2d_pair(a + 8192, tm_a, bar, m0 + 64, k * KS);
            } else {
              tc::tma_load_2d_pair(a, tm_a, bar, k * KS, m0);
            }
          }
          if (B_MN) {
            tc::tma_load_2d_pair(b, tm_b, bar, n0, k * KS);
            tc::tma_load_2d_pair(b + 8192, tm_b, bar, n0 + 64, k * KS);
          } else {
            tc::tma_load_2d_pair(b, tm_b, bar, k * KS, n0);
          }
          if (filled < stages) ++filled;
          if (++s == stages) {
            s = 0;
            phase ^= 1u;
          }
        }
      }
      // never leave with a copy still landing in shared memory: the pair MMAs
      // read every landed stage before they free it
      bool ok = true;
      for (int k = 0; k < filled && ok; ++k) {
        if (filled == stages) {         // oldest first: the slots from s on
          ok = tc::mbar_wait(&empty[s], phase, check);
          if (++s == stages) {
            s = 0;
            phase ^= 1u;
          }
        } else {
          ok = tc::mbar_wait(&empty[k], 0, check);
        }
      }
    }
  } else if (warp == MMA_WARP) {
    if (rank == 0 && lane == 0) {
      int s = 0, j = 0;
      uint32_t phase = 0;
      bool ok = true;
      // operand descriptors of stage 0; the address field (16-byte units) of later
      // stages and K steps stays within its 14 bits
      const uint32_t base = tc::smem_u32(smem);
      const uint64_t first_a = A_MN ? tc::sdesc(base, 8192, 1024, tc::kSwizzle128) : tc::sdesc(base, 16, 1024, tc::kSwizzle128);
      const uint64_t first_b = B_MN ? tc::sdesc(base + a_bytes, 8192, 1024, tc::kSwizzle128)
                                    : tc::sdesc(base + a_bytes, 16, 1024, tc::kSwizzle128);
      uint64_t desc_a = first_a, desc_b = first_b;
      Item next = pair < count ? plan.item(pair) : Item{};
      for (int i = pair; i < count && ok; i += pairs, ++j) {
        const Item w = next;
        if (i + pairs < count) next = plan.item(i + pairs);
        const int b = j & 1;
        if (*abort_flag || !tc::mbar_wait(&acc_empty[b], ((j >> 1) & 1) ^ 1, check)) { *abort_flag = 1; break; }
        tc::tc_fence_after();
        const uint32_t acc = tc::tmem_addr(tmem, 0, b * TN);
        // One thread issues everything, so what it does per step is on the critical
        // path of narrow tiles (0.32 us a step with an abort check and descriptors
        // built anew, whatever the tile's size): a failed wait is the only way out,
        // and descriptors move by constants.
        for (int k = w.k0; k < w.k1; ++k) {
          if (!tc::mbar_wait(&full[s], phase, check)) { *abort_flag = 1; ok = false; break; }
          tc::tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < KS / 16; ++kk)
            tc::mma_ss_pair(acc, desc_a + kk * ((A_MN ? 2048 : 32) >> 4), desc_b + kk * ((B_MN ? 2048 : 32) >> 4), idesc,
                            (k > w.k0 || kk > 0) ? 1u : 0u);
          tc::mma_commit_pair(&empty[s]);
          desc_a += stage >> 4;
          desc_b += stage >> 4;
          if (++s == stages) {
            s = 0;
            phase ^= 1u;
            desc_a = first_a;
            desc_b = first_b;
          }
        }
        if (ok) tc::mma_commit_pair(&acc_full[b]);
      }
    }
  } else {
    const uint32_t acc_empty_even = tc::mapa(&acc_empty[0], 0);
    uint8_t* scratch = smem + Smem<S>::SCRATCH_OFF;
    epi.start(warp, lane, scratch);
    Item next{};
    if (pair < count) {
      next = plan.item(pair);
      epi.ready(next, (2 * next.m + rank) * a_rows, next.n * tn, warp, lane);
    }
    int j = 0;
    for (int i = pair; i < count; i += pairs, ++j) {
      const int b = j & 1;
      const Item w = next;
      epi.take();
      if (i + pairs < count) {
        next = plan.item(i + pairs);
        epi.ready(next, (2 * next.m + rank) * a_rows, next.n * tn, warp, lane);
      }
      bool have = !*abort_flag && tc::mbar_wait(&acc_full[b], (j >> 1) & 1, check);
      // tcgen05.ld is warp-collective, and a warp that went on alone would wait at the
      // tile's barriers forever: the warps that meet there give up together.  (All eight
      // where pairs meet: up to 2 us of 81 with 1000 tokens of three LUT sets at 4096 x 4096.)
      if constexpr (Epi::kTeam == 1) have = __all_sync(0xffffffffu, have);
      else have = tc::named_bar_and(kVoteBar + (Epi::kTeam == 2 ? warp & 3 : 0), 32 * Epi::kTeam, have);
      if (!have) { *abort_flag = 1; break; }
      tc::tc_fence_after();
      epi.tile(tc::tmem_addr(tmem, 32 * (warp & 3), b * TN), (2 * w.m + rank) * a_rows, w.n * tn, w, warp, lane, scratch);
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive_cluster(acc_empty_even + 8 * b);
    }
    epi.done(lane);
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

// ----------------------------------------------------------------------------
// host
// ----------------------------------------------------------------------------

inline int tiles_of(int64_t v) { return (int)((v + 255) / 256); }

inline Shape shape_of(int64_t M, int64_t N, int64_t K) {
  Shape s;
  s.mt = (int)tiles_of(M);
  s.nt = (int)tiles_of(N);
  s.ksteps = (int)((K + KS - 1) / KS);
  s.M = (int)M;
  s.a_rows = 128;
  s.tn = TN;
  // about as many M as N tiles among the pairs in flight: the fewest operand bytes
  // per step (4 to 32 measured alike within the noise of the power cap)
  s.group = s.mt < 8 ? s.mt : 8;
  s.split_from = s.mt * s.nt;
  s.split = 1;
  return s;
}

// Cut the tiles of the last, partly filled round along K so that every pair has a
// part.  Worth joining the parts only when it shortens the round by more than a
// launch takes (about 32 K steps of a quarter of a microsecond).
inline void split_last_round(Shape& s) {
  const int pairs = num_sms() / 2, tiles = s.mt * s.nt, rem = tiles % pairs;
  if (rem == 0) return;
  int split = pairs / rem;
  if (split > 8) split = 8;
  if (split < 2 || s.ksteps - s.ksteps / split < 32) return;
  s.split_from = tiles - rem;
  s.split = split;
}

// One CTA pair per two SMs, or fewer when there are fewer items.
template <int EW, int S, class Kern, class... Args>
cudaError_t launch_pairs(Kern kern, int64_t count, cudaStream_t s, const Args&... args) {
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<S>::BYTES);
  if (e != cudaSuccess) return e;
  const int64_t pairs = num_sms() / 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2u * (unsigned)(count < pairs ? count : pairs), 1, 1);
  cfg.blockDim = dim3(threads(EW), 1, 1);
  cfg.dynamicSmemBytes = Smem<S>::BYTES;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, args...);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace gemm
}  // namespace sk
