// The vocabulary loss's logits on CTA pairs: 256 tokens x 256 columns of the
// vocabulary a tile (the pair kernel of gemm_f16.cuh with the tokens as its A
// operand), drained to softmax statistics or to D while the next tile's MMAs
// run.  A warp has 32 tokens, one a lane, and half of the tile's columns.
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "gemm_f16.cuh"
#include "head.cuh"
#include "model.h"
#include "store_box.cuh"

namespace mt {
namespace head {

using namespace f16tc;

constexpr int CHUNK = 32;  // columns read from tensor memory at a time
constexpr int CHUNKS = PAIR_SLOT / CHUNK;

// The target's bit among a chunk's columns, `at` columns past its first; 0:
// elsewhere.  (A bit mask, so that the chunk stays in registers.)
__device__ __forceinline__ uint32_t hot_of(int at) {
  return at >= 0 && at < CHUNK ? 1u << at : 0u;
}

struct StatsDrain {
  static constexpr bool DEPENDENT_LAUNCH = true;
  static constexpr int WARPS = 8, STORE_BYTES = 0;
  HeadStats ep;

  __device__ __forceinline__ void operator()(uint32_t t_row, const Unit& w, int q, int half,
                                             int lane, const Sched&, float*, int rank) const {
    const int t = w.tm * PAIR_TILE + rank * PAIR_HALF + q * 32 + lane;
    const int c0 = w.tn * PAIR_TILE + half * PAIR_SLOT;
    const int target = ep.target_of(t) - c0;
    Softmax s{-INFINITY, 0.0f};
    float sum = 0.0f;
#pragma unroll 1
    for (int ch = 0; ch < CHUNKS; ++ch) {
      const int c = ch * CHUNK;
      float v[CHUNK];
      __syncwarp();
      tmem_ld32(t_row + half * PAIR_SLOT + c, v);
      const int left = ep.C - c0 - c;  // columns of the vocabulary from here on
      if (left < CHUNK) {
#pragma unroll
        for (int i = 0; i < CHUNK; ++i)
          if (i >= left) v[i] = -INFINITY;
      }
      if (ep.sums) {
#pragma unroll
        for (int i = 0; i < CHUNK; ++i) sum += i < left ? v[i] : 0.0f;
      }
      if (const uint32_t hot = hot_of(target - c)) {
        float z = 0.0f;
#pragma unroll
        for (int i = 0; i < CHUNK; ++i) z = hot >> i & 1u ? v[i] : z;
        ep.store_target(t, z);
      }
      float top[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
      for (int i = 4; i < CHUNK; ++i) top[i % 4] = fmaxf(top[i % 4], v[i]);
      const float most = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * LOG2E;
      const float now = fmaxf(most, s.top), base = Softmax::base(now);
      float add[4] = {s.sum * exp2_approx(s.top - base), 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < CHUNK; ++i) add[i % 4] += exp2_approx(fmaf(v[i], LOG2E, -base));
      s = Softmax{now, (add[0] + add[1]) + (add[2] + add[3])};
    }
    if (t < ep.T) ep.store(w.tn * (PAIR_TILE / PAIR_SLOT) + half, t, s, sum);
  }
};

struct GradDrain {
  static constexpr bool DEPENDENT_LAUNCH = true;
  static constexpr int WARPS = 8, STORE_BYTES = WARPS * STORE_BOX_BYTES;
  HeadGrad ep;

  template <class T>
  __device__ __forceinline__ void typed(uint32_t t_row, const Unit& w, int q, int half, int lane,
                                        uint8_t* box, int rank) const {
    const int t0 = w.tm * PAIR_TILE + rank * PAIR_HALF + q * 32, t = t0 + lane;
    const int c0 = w.tn * PAIR_TILE + half * PAIR_SLOT;
    const HeadRow r = ep.row(t, ep.T);
    const int hit = r.target;
    const int target = hit - ep.first - c0;  // negative without one
    constexpr int PER = 64 / CHUNK;          // chunks of a box
#pragma unroll 1
    for (int c = 0; c < PAIR_SLOT; c += 64) {
      store_begin(lane);
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        float v[CHUNK];
        __syncwarp();
        tmem_ld32(t_row + half * PAIR_SLOT + c + i * CHUNK, v);
#pragma unroll
        for (int k = 0; k < CHUNK; ++k)
          v[k] = hit == HeadRow::DEAD
                     ? 0.0f
                     : fmaf(exp2_approx(fmaf(v[k], LOG2E, -r.x)), r.p, -r.all);
        if (const uint32_t hot = hot_of(target - c - i * CHUNK)) {
#pragma unroll
          for (int k = 0; k < CHUNK; ++k) v[k] -= hot >> k & 1u ? r.hit : 0.0f;
        }
        store_fill<T>(box, lane, i * CHUNK, v);
      }
      store_end(&ep.map, box, lane, c0 + c, t0, c0 + c < ep.C && t0 < ep.T, false);
    }
  }

  __device__ __forceinline__ void operator()(uint32_t t_row, const Unit& w, int q, int half,
                                             int lane, const Sched&, float* square,
                                             int rank) const {
    uint8_t* const box = store_staging<GradDrain>(square, q, half);
    if (ep.dtype == DT_F16) typed<__half>(t_row, w, q, half, lane, box, rank);
    else typed<__nv_bfloat16>(t_row, w, q, half, lane, box, rank);
  }
};

template <class Ep>
using DrainOf = typename std::conditional<std::is_same<Ep, HeadStats>::value, StatsDrain,
                                          GradDrain>::type;

constexpr int ACC_BUFS = 2;

template <class Drain>
const void* kernel_for(bool w_mn) {
  return w_mn ? reinterpret_cast<const void*>(pair_kernel<Half, false, true, ACC_BUFS, Drain>)
              : reinterpret_cast<const void*>(pair_kernel<Half, false, false, ACC_BUFS, Drain>);
}

}  // namespace head

using namespace head;

template <class Ep>
cudaError_t launch_head_pair(const CUtensorMap& map_x, const CUtensorMap& map_w, uint32_t idesc,
                             const Ep& ep, bool w_mn, int kt, int clusters,
                             int fault_inject, cudaStream_t stream) {
  using Drain = DrainOf<Ep>;
  Drain drain{ep};
  int tiles_t = (ep.T + PAIR_TILE - 1) / PAIR_TILE, tiles_c = (ep.C + PAIR_TILE - 1) / PAIR_TILE;
  int group = 8;
  Sched sched{tiles_t * tiles_c, 1, kt, nullptr, 0, 0};
  CUtensorMap x = map_x, w = map_w;
  void* args[] = {&x,       &w,       &idesc, &drain, &kt,
                  &tiles_t, &tiles_c, &group, &sched, &fault_inject};
  return launch_dependent(kernel_for<Drain>(w_mn), dim3(2 * static_cast<unsigned>(clusters)),
                          pair_threads<Drain>(), pair_smem<Drain, ACC_BUFS>(), 2, stream, args);
}
template cudaError_t launch_head_pair(const CUtensorMap&, const CUtensorMap&, uint32_t,
                                      const HeadStats&, bool, int, int, int, cudaStream_t);
template cudaError_t launch_head_pair(const CUtensorMap&, const CUtensorMap&, uint32_t,
                                      const HeadGrad&, bool, int, int, int, cudaStream_t);

cudaError_t head_prepare() {
  cudaError_t r = cudaSuccess;
  auto prepare = [&](const void* k, int smem) {
    if (r == cudaSuccess)
      r = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (r == cudaSuccess)
      r = cudaFuncSetAttribute(k, cudaFuncAttributePreferredSharedMemoryCarveout,
                               cudaSharedmemCarveoutMaxShared);
  };
  for (bool w_mn : {false, true}) {
    prepare(kernel_for<StatsDrain>(w_mn), pair_smem<StatsDrain, ACC_BUFS>());
    prepare(kernel_for<GradDrain>(w_mn), pair_smem<GradDrain, ACC_BUFS>());
  }
  for (int bt : {16, 32, 64, 128}) {
    const linear::LinearKernel s = head_split_kernel_for<HeadStats>(bt);
    const linear::LinearKernel g = head_split_kernel_for<HeadGrad>(bt);
    prepare(s.kernel, s.smem);
    prepare(g.kernel, g.smem);
  }
  return r == cudaSuccess ? linear_rows_prepare() : r;
}

cudaError_t head_pair_read_and_clear_status(unsigned int* status) {
  return f16tc::read_and_clear_status(status);
}

}  // namespace mt
