// Operand tiles and the CTA-pair kernel of the tcgen05 products on 16- and
// 8-bit operands (gemm_f16.cu: fp32 C; linear.cu: the fused linear layer).
// Every operand tile is rows of 128 bytes of K (or, MN-major, 64-value boxes)
// in the 128-byte-swizzled layout TMA writes and the MMA reads.
#pragma once

#include <cstdint>

#include <cuda.h>

#include "device_util.cuh"
#include "kernels.h"
#include "tcgen05.cuh"

namespace mt {
namespace f16tc {

using namespace tc;

constexpr int BM = 128;
constexpr int BK = 64;            // 16-bit values of K per stage: one 128-byte row
constexpr int ROW_BYTES = 128;
constexpr int ATOM_BYTES = 8 * ROW_BYTES;
constexpr int MN_BOX = 64;        // M/N values per box of an MN-major operand
constexpr int MN_BOX_BYTES = BK * MN_BOX * 2;
constexpr uint64_t SWIZZLE_128B = 2;  // descriptor layout code
constexpr int THREADS = 192;
constexpr int EPILOGUE_THREADS = 128;
constexpr int SMEM_STAGE_BUDGET = 200 * 1024;

// Per translation unit: each reads and clears its own.
static __device__ unsigned int g_status;  // bit 0: a bounded wait expired
static inline cudaError_t read_and_clear_status(unsigned int* status) {
  cudaError_t e = cudaMemcpyFromSymbol(status, g_status, sizeof(unsigned int));
  if (e != cudaSuccess) return e;
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_status, &zero, sizeof(unsigned int));
}

// Element types of the operands: 16-bit (fp16 or bf16, by the instruction
// descriptor) and e4m3; both MMAs take 32 bytes of K per step.
struct Half {
  static constexpr int BYTES = 2;
  static __device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                             uint32_t acc) {
    mma_f16(d, a, b, idesc, acc);
  }
  static __device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b,
                                                  uint32_t idesc, uint32_t acc) {
    mma_f16_pair(d, a, b, idesc, acc);
  }
};
struct E4m3 {
  static constexpr int BYTES = 1;
  static __device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                             uint32_t acc) {
    mma_f8(d, a, b, idesc, acc);
  }
  static __device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b,
                                                  uint32_t idesc, uint32_t acc) {
    mma_f8_pair(d, a, b, idesc, acc);
  }
};

// Loads the `rows`-row tile of one operand for K tile k0 into `dst`.
template <int ROWS, bool MN>
__device__ __forceinline__ void load_operand(uint32_t dst, const CUtensorMap* map, int r0,
                                             int k0, uint32_t bar) {
  if constexpr (!MN) {
    tma_load_2d(dst, map, k0, r0, bar);  // box: 64 k x ROWS rows
  } else {
#pragma unroll
    for (int c = 0; c < ROWS / MN_BOX; ++c)  // boxes: 64 m/n x 64 k
      tma_load_2d(dst + c * MN_BOX_BYTES, map, r0 + c * MN_BOX, k0, bar);
  }
}

// Prefetches the same tile to L2.
template <int ROWS, bool MN>
__device__ __forceinline__ void prefetch_operand(const CUtensorMap* map, int r0, int k0) {
  if constexpr (!MN) {
    tma_prefetch_2d(map, k0, r0);
  } else {
#pragma unroll
    for (int c = 0; c < ROWS / MN_BOX; ++c) tma_prefetch_2d(map, r0 + c * MN_BOX, k0);
  }
}

// Descriptor of k-step j (32 bytes of K: 16 16-bit or 32 8-bit values) of an
// operand tile at `base`.
template <bool MN>
__device__ __forceinline__ uint64_t operand_desc(uint32_t base, int j) {
  if constexpr (!MN)
    return smem_desc(base + j * 32, 16, ATOM_BYTES, SWIZZLE_128B);
  else
    return smem_desc(base + j * 16 * ROW_BYTES, MN_BOX_BYTES, ATOM_BYTES, SWIZZLE_128B);
}

// ---------------------------------------------------------------------------
// CTA-pair kernel: a cluster of two CTAs on two SMs computes 256 x 256 tiles
// with tcgen05.mma.cta_group::2.  CTA r (0 or 1) of the pair holds rows
// m0 + 128 r .. +127 of A's tile and columns n0 + 128 r .. +127 of B's, so
// each SM stages 32 KB per 64-deep K tile for a 128 x 256 share of the
// product (a single-CTA 128 x 256 tile stages 48 KB for the same share).
//   both CTAs, warp 0: TMA loads of the CTA's halves into its own ring; the
//     bytes of both complete on the even CTA's full[s] (cta_group::2 copies),
//     and only the even CTA arms it (expect_tx of both halves);
//   even CTA, warp 1: per K tile 4 pair MMAs 256 x 256 x 16, then a commit
//     multicast to empty[s] of both CTAs, and after a unit's last K tile to
//     acc_full[b] of both;
//   both CTAs, warps 2 on: drain their own TMEM half (128 rows x 256) to
//     memory, then one arrival per warp on the even CTA's acc_empty[b].
// E: the element type (Half or E4m3); drain(t_row, unit, q, half, lane, sched,
// square, rank) takes the 32 x 256 accumulator of warp q's lanes at TMEM
// address t_row (rows q * 32 .. of CTA `rank`'s half) to memory; with
// Drain::WARPS = 8 two warps share it (half 0 and 1).
// Drain::STORE_BYTES: shared memory that the drain stages its stores in, each
// warp's last bulk group waited for before the CTA leaves (0: none).
// Drain::DEPENDENT_LAUNCH: the kernel is launched as a programmatic dependent
// and lets its own dependents launch early.
// ACC_BUFS accumulators of 256 columns each (1 or 2) sit in TMEM.
constexpr int PAIR_TILE = 256;
constexpr int PAIR_HALF = 128;

template <int ACC_BUFS_>
struct PairGeometry {
  static constexpr int ACC_BUFS = ACC_BUFS_;
  static constexpr int A_BYTES = PAIR_HALF * ROW_BYTES;  // this CTA's half of A
  static constexpr int B_BYTES = PAIR_HALF * ROW_BYTES;  // this CTA's half of B
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int STAGES_FIT = SMEM_STAGE_BUDGET / STAGE_BYTES;
  static constexpr int STAGES = STAGES_FIT > 8 ? 8 : STAGES_FIT;
  static constexpr uint32_t TMEM_COLS = ACC_BUFS * PAIR_TILE;
  static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + 1024 /*alignment*/ + 256 +
                                   EPI_STAGE_BYTES;
};

// A drain warp's part of the staging that Drain::STORE_BYTES asks for: past the
// barriers, from a 1024-byte boundary on, as swizzled boxes want it.  `square`:
// the warp's pointer that the pair kernel gives the drain.
template <class Drain>
__device__ __forceinline__ uint8_t* store_staging(float* square, int q, int half) {
  const uintptr_t base = reinterpret_cast<uintptr_t>(square - q * EPI_WARP_FLOATS);
  return reinterpret_cast<uint8_t*>((base + 1023) & ~static_cast<uintptr_t>(1023)) +
         (half * 4 + q) * (Drain::STORE_BYTES / Drain::WARPS);
}
// Dynamic shared memory of the pair kernel.
template <class Drain, int ACC_BUFS>
constexpr int pair_smem() {
  return PairGeometry<ACC_BUFS>::SMEM_BYTES - EPI_STAGE_BYTES +
         (Drain::STORE_BYTES > 0 ? 1024 - 256 + Drain::STORE_BYTES : 0);
}

// Threads of the pair kernel: the copy warp, the MMA warp, the drain's warps.
template <class Drain>
constexpr int pair_threads() {
  return 64 + 32 * Drain::WARPS;
}

template <class E, bool A_MN, bool B_MN, int ACC_BUFS, class Drain>
__global__ void __launch_bounds__(pair_threads<Drain>(), 1)
    pair_kernel(const __grid_constant__ CUtensorMap tmap_a,
                const __grid_constant__ CUtensorMap tmap_b, uint32_t idesc,
                const __grid_constant__ Drain drain, int Kt,
                int tiles_m, int tiles_n, int group_m, Sched sched, int fault_inject) {
  static_assert(E::BYTES == 2 || (!A_MN && !B_MN), "8-bit operands are K-major");
  using G = PairGeometry<ACC_BUFS>;
  constexpr int STAGES = G::STAGES;
  constexpr int STAGE_BYTES = G::STAGE_BYTES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + STAGES * STAGE_BYTES);
  // bars: [0, S) full (used on the even CTA), [S, 2S) empty, then
  // acc_full[ACC_BUFS], acc_empty[ACC_BUFS] (used on the even CTA), drain.
  constexpr int FULL = 0, EMPTY = STAGES, ACC_FULL = 2 * STAGES,
                ACC_EMPTY = 2 * STAGES + ACC_BUFS, DRAIN = 2 * STAGES + 2 * ACC_BUFS,
                NBARS = DRAIN + 1;
  static_assert(NBARS * 8 + 8 <= 256, "barriers, TMEM slot and abort flag fit 256 bytes");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + NBARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const WaitCtx wc{abort_flag, &g_status};
  auto bar = [&](int i) { return smem_u32(bars + i); };

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = cluster_ctarank();  // 0: even (MMA issuer), 1: odd
  const bool leader = rank == 0;
  const int cluster = static_cast<int>(cluster_id_x());
  const int clusters = static_cast<int>(cluster_count_x());
  const int num_tiles = tiles_m * tiles_n;
  const int num_units = units_of(cluster, clusters, sched, num_tiles, Kt);  // this cluster's units

  if (threadIdx.x == 0) {
    prefetch_tmap(&tmap_a);
    prefetch_tmap(&tmap_b);
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(bar(FULL + s), 1);   // the even CTA's arrival + both CTAs' bytes
      mbar_init(bar(EMPTY + s), 1);  // pair MMA commit
    }
    for (int b = 0; b < ACC_BUFS; ++b) {
      mbar_init(bar(ACC_FULL + b), 1);   // pair MMA commit
      mbar_init(bar(ACC_EMPTY + b), 2 * Drain::WARPS);  // every epilogue warp of both CTAs
    }
    mbar_init(bar(DRAIN), 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tmem_alloc_pair(smem_u32(tmem_slot), G::TMEM_COLS);
  tc_fence_before();
  cluster_sync();  // barriers initialised and TMEM allocated in both CTAs
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if constexpr (Drain::DEPENDENT_LAUNCH) {
    grid_launch_dependents();
    grid_wait();
  }

  if (warp == 0) {
    if (lane == 0) {
      // Producer (both CTAs): this CTA's halves into its own stages.
      bool stop = fault_inject != 0;
      uint32_t g = 0;
      for (int u = 0; u < num_units && !stop; ++u) {
        const Unit w = unit_at(u, cluster, clusters, sched, tiles_m, tiles_n, group_m, Kt);
        const int r0a = w.tm * PAIR_TILE + static_cast<int>(rank) * PAIR_HALF;
        const int r0b = w.tn * PAIR_TILE + static_cast<int>(rank) * PAIR_HALF;
        for (int kt = w.kt0; kt < w.kt1; ++kt, ++g) {
          const uint32_t s = g % STAGES, round = g / STAGES;
          if (g >= STAGES && !wait_phase(bar(EMPTY + s), (round + 1) & 1u, wc)) {
            stop = true;
            break;
          }
          const uint32_t full_even = map_to_cta(bar(FULL + s), 0);
          if (leader) mbar_arrive_expect_tx(bar(FULL + s), 2 * STAGE_BYTES);
          const uint32_t st = smem_u32(smem + s * STAGE_BYTES);
          const int k0 = kt * (ROW_BYTES / E::BYTES);
          if constexpr (!A_MN) {
            tma_load_2d_pair(st, &tmap_a, k0, r0a, full_even);
          } else {
            tma_load_2d_pair(st, &tmap_a, r0a, k0, full_even);
            tma_load_2d_pair(st + MN_BOX_BYTES, &tmap_a, r0a + MN_BOX, k0, full_even);
          }
          const uint32_t sb = st + G::A_BYTES;
          if constexpr (!B_MN) {
            tma_load_2d_pair(sb, &tmap_b, k0, r0b, full_even);
          } else {
            tma_load_2d_pair(sb, &tmap_b, r0b, k0, full_even);
            tma_load_2d_pair(sb + MN_BOX_BYTES, &tmap_b, r0b + MN_BOX, k0, full_even);
          }
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      // Pair MMA issuer (even CTA).
      uint32_t g = 0;
      bool stop = false;
      int it = 0;
      for (int u = 0; u < num_units && !stop; ++u, ++it) {
        const Unit w = unit_at(u, cluster, clusters, sched, tiles_m, tiles_n, group_m, Kt);
        const int b = it % ACC_BUFS, use = it / ACC_BUFS;
        // Both CTAs' epilogues must have drained this accumulator.
        if (use >= 1 && !wait_phase(bar(ACC_EMPTY + b), (use + 1) & 1u, wc)) break;
        tc_fence_after();
        const uint32_t acc_tmem = tmem + static_cast<uint32_t>(b * PAIR_TILE);
        uint32_t acc = 0;
        for (int kt = w.kt0; kt < w.kt1; ++kt, ++g) {
          const uint32_t s = g % STAGES, round = g / STAGES;
          if (!wait_phase(bar(FULL + s), round & 1u, wc)) {
            stop = true;
            break;
          }
          tc_fence_after();
          const uint32_t a_base = smem_u32(smem + s * STAGE_BYTES);
          const uint32_t b_base = a_base + G::A_BYTES;
#pragma unroll
          for (int j = 0; j < ROW_BYTES / 32; ++j) {
            E::mma_pair(acc_tmem, operand_desc<A_MN>(a_base, j), operand_desc<B_MN>(b_base, j),
                        idesc, acc);
            acc = 1;
          }
          mma_commit_pair(bar(EMPTY + s), 0x3);
        }
        if (!stop) mma_commit_pair(bar(ACC_FULL + b), 0x3);
      }
      // Every pair MMA issued has retired once DRAIN completes.
      mma_commit_pair(bar(DRAIN), 0x1);
      wait_phase(bar(DRAIN), 0, wc, false);
    }
  } else {
    // Epilogue warps of both CTAs: warp w may access TMEM lanes 32*(w%4)..+31.
    const int q = warp & 3;
    // This warp's staging square, past the barriers.
    float* const epi_square =
        reinterpret_cast<float*>(smem + STAGES * STAGE_BYTES + 256) + q * EPI_WARP_FLOATS;
    const uint32_t lane_base = static_cast<uint32_t>(q * 32) << 16;
    const uint32_t acc_empty_even = map_to_cta(bar(ACC_EMPTY), 0);
    int it = 0;
    for (int u = 0; u < num_units; ++u, ++it) {
      const int b = it % ACC_BUFS, use = it / ACC_BUFS;
      const bool ready = wait_phase(bar(ACC_FULL + b), use & 1u, wc, true,
                                    TIMEOUT_NS + 20000ull * static_cast<uint64_t>(Kt));
      if (!__all_sync(0xffffffffu, ready)) break;
      tc_fence_after();
      __syncwarp();
      const Unit w = unit_at(u, cluster, clusters, sched, tiles_m, tiles_n, group_m, Kt);
      drain(tmem + lane_base + static_cast<uint32_t>(b * PAIR_TILE), w, q, (warp - 2) / 4, lane,
            sched, epi_square, static_cast<int>(rank));
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(acc_empty_even + 8u * static_cast<uint32_t>(b));
    }
    if (Drain::STORE_BYTES > 0 && lane == 0) bulk_wait();
  }

  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    // Copies this CTA issued complete on the even CTA's barriers, which it
    // cannot wait on: give any still in flight time to land (bounded).
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 200000ull) {
    }
  }
  // The even CTA's MMAs (which read the odd CTA's shared memory) have
  // retired and every cross-CTA arrival is done before either CTA leaves.
  cluster_sync();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem, G::TMEM_COLS);
  }
}

}  // namespace f16tc
}  // namespace mt
