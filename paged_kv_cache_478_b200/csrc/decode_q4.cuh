// Decode attention over 4-bit pools (quant4.cuh has the format).
//
// Work items, plan, split-K partials and merge are those of the other decode
// kernels (plan.cuh, decode.cuh).  One warp owns one KV head of the item and
// all of its G query heads.
#pragma once

#include <math.h>
#include <stdint.h>

#include "decode.cuh"
#include "device_utils.cuh"
#include "quant4.cuh"

namespace pa {

template <typename T, int D>
struct Q4Config {
  static constexpr int WARPS = 4;
  static constexpr int KVPI = 4;  // KV heads per work item, one warp each
  static constexpr int THREADS = WARPS * 32;
  static size_t smem_bytes(int partition_size) { return (size_t)(partition_size / kBlock) * 4; }
};

template <typename T, int D, int G, bool MASS>
__global__ void __launch_bounds__(128) paged_decode_q4_kernel(DecodeArgs a) {
  using Cfg = Q4Config<T, D>;
  constexpr int DPL = D / 32;  // dimensions per lane
  constexpr int TILE = q4_tile_bytes(D);
  extern __shared__ int32_t q4_tbl[];
  __shared__ int32_t s_item, s_merge, s_plan_ok;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int HK = a.heads, HQ = HK * G, PS = a.partition_size;

  if (a.after_plan) grid_dependency_wait();
  if (threadIdx.x == 0) {
    s_plan_ok = plan_header_ok(a);
    if (!s_plan_ok) atomicOr(a.err, PA_DEVERR_PLAN);
  }
  __syncthreads();
  if (!s_plan_ok) return;
  const int32_t num_items = a.plan->num_items;

  for (;;) {
    if (threadIdx.x == 0) s_item = atomicAdd(&a.plan->work_counter, 1);
    __syncthreads();
    const int item = s_item;
    if (item >= num_items) break;
    PlanItem it;
    if (!plan_item(a, item, &it)) {
      if (threadIdx.x == 0) atomicOr(a.err, PA_DEVERR_PLAN);
      __syncthreads();
      continue;
    }
    const int g = item % a.head_groups;
    const int s = it.s, p = it.p, L = it.L, np = it.np, ni = it.ni;
    const bool split = np > 1;
    const int tok0 = it.base + p * PS;
    const int ntok = max(0, min(L, tok0 + PS) - tok0);
    const int nblk = (ntok + kBlock - 1) / kBlock;
    for (int i = threadIdx.x; i < nblk; i += blockDim.x) {
      int32_t b = a.block_tables[(int64_t)s * a.max_blocks_per_seq + tok0 / kBlock + i];
      if (b < 0 || b >= a.num_blocks) {
        atomicOr(a.err, PA_DEVERR_BLOCK_ID);
        b = 0;
      }
      q4_tbl[i] = b;
    }
    __syncthreads();

    const int kvh = g * Cfg::KVPI + warp;
    if (kvh < HK) {
      const int64_t sh0 = (int64_t)s * HQ + kvh * G;
      const int d0 = lane * DPL;
      float q[G][DPL], acc[G][DPL], m_run[G], l_run[G];
#pragma unroll
      for (int h = 0; h < G; ++h) {
        m_run[h] = -INFINITY;
        l_run[h] = 0.f;
#pragma unroll
        for (int e = 0; e < DPL; ++e) {
          q[h][e] = (float)static_cast<const T*>(a.q)[(sh0 + h) * D + d0 + e] * a.scale_log2;
          acc[h][e] = 0.f;
        }
      }
      const int off = (d0 / 32) * 256 + (d0 % 32) / 2, word = q4_words_off(D) + (d0 / 64) * 64;
      auto row = [&](const uint8_t* tile, int t, float* x) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(tile + word + t * 4);
        const float sc = q4_scale(w), z = q4_zero(w);
#pragma unroll
        for (int e = 0; e < DPL; e += 2) {
          const uint32_t b = tile[off + t * 16 + e / 2];
          x[e] = sc * ((float)(b & 15u) - z);
          x[e + 1] = sc * ((float)(b >> 4) - z);
        }
      };
      for (int i = 0; i < nblk; ++i) {
        const int64_t at = ((int64_t)q4_tbl[i] * HK + kvh) * TILE;
        const uint8_t* kt = static_cast<const uint8_t*>(a.k_pool) + at;
        const uint8_t* vt = static_cast<const uint8_t*>(a.v_pool) + at;
        const int valid = min(kBlock, ntok - i * kBlock);
        for (int t = 0; t < valid; ++t) {
          float k[DPL], v[DPL];
          row(kt, t, k);
          row(vt, t, v);
#pragma unroll
          for (int h = 0; h < G; ++h) {
            float x = 0.f;
#pragma unroll
            for (int e = 0; e < DPL; ++e) x = fmaf(q[h][e], k[e], x);
#pragma unroll
            for (int m = 16; m >= 1; m >>= 1) x += __shfl_xor_sync(kFullMask, x, m);
            if (MASS && lane == 0) a.scores[(sh0 + h) * a.score_stride + tok0 + i * kBlock + t] = x;
            const float m_new = fmaxf(m_run[h], x);
            const float alpha = exp2f(m_run[h] - m_new), w = exp2f(x - m_new);
            m_run[h] = m_new;
            l_run[h] = fmaf(l_run[h], alpha, w);
#pragma unroll
            for (int e = 0; e < DPL; ++e) acc[h][e] = fmaf(acc[h][e], alpha, w * v[e]);
          }
        }
      }
#pragma unroll
      for (int h = 0; h < G; ++h) {
        if (!split) {
          const float inv = nblk > 0 ? 1.f / l_run[h] : 0.f;
#pragma unroll
          for (int e = 0; e < DPL; ++e) static_cast<T*>(a.out)[(sh0 + h) * D + d0 + e] = (T)(acc[h][e] * inv);
          if (MASS && lane == 0) a.lse[sh0 + h] = m_run[h] + log2f(l_run[h]);
        } else {
#pragma unroll
          for (int e = 0; e < DPL; ++e) a.part_acc[((sh0 + h) * a.max_parts + p) * D + d0 + e] = acc[h][e];
          if (lane == 0) a.part_ml[(sh0 + h) * a.max_parts + p] = make_float2(m_run[h], l_run[h]);
        }
      }
    }
    if (split) {
      __syncthreads();
      if (threadIdx.x == 0) {
        int32_t* cnt = a.merge_cnt + (int64_t)s * a.head_groups + g;
        __threadfence();
        const int arrived = atomicAdd(cnt, 1) + 1;
        __threadfence();
        s_merge = arrived == ni && *(volatile int32_t*)&a.plan->poisoned == 0;
        if (arrived == ni) *cnt = 0;
      }
      __syncthreads();
      if (s_merge && kvh < HK) {
        __threadfence();
        for (int h = 0; h < G; ++h)
          merge_partitions<T, D, MASS>(a, (int64_t)s * HQ + kvh * G + h, np, lane);
      }
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    __threadfence();
    const int done = atomicAdd(&a.plan->done_counter, 1);
    if (done == (int)gridDim.x - 1) {
      a.plan->work_counter = 0;
      a.plan->done_counter = 0;
      __threadfence();
    }
  }
}

}  // namespace pa
