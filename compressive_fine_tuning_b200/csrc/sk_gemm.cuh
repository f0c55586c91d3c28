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
constexpr int S = 6;
constexpr int EPI_WARPS = 4, TMA_WARP = 4, MMA_WARP = 5, THREADS = 192;
constexpr int SLAB = 32 * 128;                    // one warp's output slab: 32 rows x 128 bytes
constexpr int SLAB_OFF = S * STAGE;               // two slabs per epilogue warp
constexpr int BAR_OFF = SLAB_OFF + EPI_WARPS * 2 * SLAB;
constexpr int SMEM = 1024 + BAR_OFF + 256;
constexpr int TMEM_COLS = 512;
static_assert(SMEM <= 232448, "one CTA's shared memory");

struct Shape {
  int mt, nt, ksteps;    // tiles and K steps
  int tn;                // columns per tile: 256, or less for a K-major B (a multiple of 32)
  int group;             // M tiles walked together (see tile_at)
  // The last wave: the `split_from`-th and later tiles are cut along K into `split`
  // parts, one per pair, so that a few left-over tiles do not keep one pair each
  // busy for a whole tile while the others idle.  A part's accumulator goes to the
  // epilogue with its index; the caller joins the parts.
  int split_from, split;
};

struct Item {
  int m, n, k0, k1;
  int part;              // -1: a whole tile
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
  uint8_t* base;      // this warp's two slabs
  int at;
  __device__ __forceinline__ void put(const CUtensorMap* map, const uint32_t (&w)[32], int x, int y, int lane) {
    uint8_t* slab = base + (at & 1) * SLAB;
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

// Epi: struct with
//   void tile(uint32_t tmem, int m0, int n0, int part, int warp, int lane, SlabWriter&)
// called by every epilogue warp for every item: the warp's accumulator rows are
// m0 + 32 warp + lane (TMEM lanes), columns n0 .. n0 + tn - 1.
template <int A_MN, int B_MN, class Epi>
__device__ __forceinline__ void run(const CUtensorMap* tm_a, const CUtensorMap* tm_b, const Shape& sh, Epi& epi,
                                    unsigned int* check) {
  const uint32_t idesc = tc::idesc_bf16(TM, B_MN ? TN : sh.tn, A_MN, B_MN);
  const int tn = B_MN ? TN : sh.tn, half_n = tn / 2;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + BAR_OFF);   // even CTA: both CTAs' operands landed
  uint64_t* empty = full + S;                                      // both CTAs: the pair MMAs read the stage
  uint64_t* acc_full = empty + S;                                  // both CTAs: accumulator b final
  uint64_t* acc_empty = acc_full + 2;                              // even CTA: both CTAs drained accumulator b
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = tc::warp_id(), lane = tc::lane_id();
  const int rank = (int)tc::cluster_ctarank();                     // 0: issues the MMAs
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int count = items(sh);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      tc::mbar_init(&full[s], 1);
      tc::mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(&acc_full[b], 1);
      tc::mbar_init(&acc_empty[b], 2 * EPI_WARPS);
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
      int it = 0;
      const uint32_t bytes = 2u * (A_BYTES + half_n * KS * 2);             // both CTAs' operands of a step
      for (int i = pair; i < count && !*abort_flag; i += pairs) {
        const Item w = item_at(sh, i);
        const int m0 = w.m * TM + 128 * rank, n0 = w.n * tn + half_n * rank;
        for (int k = w.k0; k < w.k1; ++k, ++it) {
          const int s = it % S;
          if (*abort_flag || !tc::mbar_wait(&empty[s], ((it / S) & 1) ^ 1, check)) { *abort_flag = 1; break; }
          uint8_t* a = smem + s * STAGE;
          uint8_t* b = a + A_BYTES;
          if (rank == 0) tc::mbar_arrive_expect_tx(&full[s], bytes);
          const uint32_t bar = tc::mapa(&full[s], 0);
          if (A_MN) {
            tc::tma_load_2d_pair(a, tm_a, bar, m0, k * KS);
            tc::tma_load_2d_pair(a + 8192, tm_a, bar, m0 + 64, k * KS);
          } else {
            tc::tma_load_2d_pair(a, tm_a, bar, k * KS, m0);
          }
          if (B_MN) {
            tc::tma_load_2d_pair(b, tm_b, bar, n0, k * KS);
            tc::tma_load_2d_pair(b + 8192, tm_b, bar, n0 + 64, k * KS);
          } else {
            tc::tma_load_2d_pair(b, tm_b, bar, k * KS, n0);
          }
        }
      }
      // never leave with a copy still landing in shared memory: the pair MMAs
      // read every landed stage before they free it
      bool ok = true;
      for (int k = it > S ? it - S : 0; k < it && ok; ++k) ok = tc::mbar_wait(&empty[k % S], (k / S) & 1, check);
    }
  } else if (warp == MMA_WARP) {
    if (rank == 0 && lane == 0) {
      int it = 0, j = 0;
      bool ok = true;
      for (int i = pair; i < count && ok; i += pairs, ++j) {
        const Item w = item_at(sh, i);
        const int b = j & 1;
        if (*abort_flag || !tc::mbar_wait(&acc_empty[b], ((j >> 1) & 1) ^ 1, check)) { *abort_flag = 1; break; }
        tc::tc_fence_after();
        const uint32_t acc = tc::tmem_addr(tmem, 0, b * TN);
        for (int k = w.k0; k < w.k1; ++k, ++it) {
          const int s = it % S;
          if (*abort_flag || !tc::mbar_wait(&full[s], (it / S) & 1, check)) { *abort_flag = 1; ok = false; break; }
          tc::tc_fence_after();
          const uint32_t ab = tc::smem_u32(smem + s * STAGE), bb = ab + A_BYTES;
#pragma unroll
          for (int kk = 0; kk < KS / 16; ++kk) {
            const uint64_t ad = A_MN ? tc::sdesc(ab + kk * 2048, 8192, 1024, tc::kSwizzle128)
                                     : tc::sdesc(ab + kk * 32, 16, 1024, tc::kSwizzle128);
            const uint64_t bd = B_MN ? tc::sdesc(bb + kk * 2048, 8192, 1024, tc::kSwizzle128)
                                     : tc::sdesc(bb + kk * 32, 16, 1024, tc::kSwizzle128);
            tc::mma_ss_pair(acc, ad, bd, idesc, (k > w.k0 || kk > 0) ? 1u : 0u);
          }
          tc::mma_commit_pair(&empty[s]);
        }
        if (ok) tc::mma_commit_pair(&acc_full[b]);
      }
    }
  } else {
    SlabWriter out{smem + SLAB_OFF + warp * 2 * SLAB, 0};
    const uint32_t acc_empty_even = tc::mapa(&acc_empty[0], 0);
    int j = 0;
    for (int i = pair; i < count; i += pairs, ++j) {
      const int b = j & 1;
      bool have = !*abort_flag && tc::mbar_wait(&acc_full[b], (j >> 1) & 1, check);
      have = __all_sync(0xffffffffu, have);   // tcgen05.ld is warp-collective
      if (!have) { *abort_flag = 1; break; }
      tc::tc_fence_after();
      const Item w = item_at(sh, i);
      epi.tile(tc::tmem_addr(tmem, 32 * warp, b * TN), w.m * TM + 128 * rank, w.n * tn, w.part, warp, lane, out);
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive_cluster(acc_empty_even + 8 * b);
    }
    out.drain(lane);
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

}  // namespace gemm
}  // namespace sk
