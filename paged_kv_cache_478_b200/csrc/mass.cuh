// Attention weight gathered per cached token, for eviction by weight.
//
//   mass_out[s][t] = decay * mass_in[s][t] + sum_h w(s, h, t),   t < L_s,
//   w(s, h, t) = softmax over t of scale * q[s][h] . K_t
// The decode kernels compute every score once; in their MASS instantiations
// they also store it (4 bytes a token and query head, against 4 D bytes of
// 16-bit K and V) and, per query head, the logarithm of its softmax sum, which
// is known only when the sequence's last partition is merged.  This kernel
// then turns the scores into weights and adds the heads in a fixed order: for
// the same sizes and partition the result is the same from run to run.  (The
// logarithms are rounded as the work was split, into partitions and, in 4-bit
// pools, over a head's warps, so another partition may change the last bits.)
#pragma once

#include <math.h>
#include <stdint.h>

#include "device_utils.cuh"
#include "plan.cuh"

// Bound by the latency of one pass over the scores, which mostly are in L2: 9 us
// beside a decode of 98 us (200 requests x 32 heads, 4-bit), and about 3 us more
// for storing the scores there.
namespace pa {

struct MassArgs {
  const float* mass_in;  // null: zero
  float* mass_out;
  int64_t stride;  // tokens between sequences of mass_in and mass_out
  float decay;
};

// 128 tokens of one sequence a CTA: the eight warps take the heads in eight
// contiguous shares, 4 tokens a lane, and their sums are added in order.  So all
// score loads of a CTA are in flight together.
constexpr int kMassTokens = 128;
constexpr int kMassWarps = 8;

__global__ void __launch_bounds__(kMassWarps * 32) mass_kernel(DecodeArgs a, MassArgs m) {
  __shared__ float4 part[kMassWarps][32];
  grid_dependency_wait();  // the decode kernel
  if (a.plan->stamp != a.stamp || a.plan->poisoned != 0) return;  // the decode launch reported it
  const int s = blockIdx.y;
  const int64_t cap = min((int64_t)a.max_context_len, (int64_t)a.max_blocks_per_seq * kBlock);
  const int L = a.lens[s];
  if (L < 0 || L > cap) return;  // a damaged plan entry: the decode launch reported it
  const int t0 = blockIdx.x * kMassTokens;
  if (t0 >= L) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int HQ = a.heads * a.q_per_kv;
  const int h0 = HQ * warp / kMassWarps, h1 = HQ * (warp + 1) / kMassWarps;
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
  if (t0 + 4 * lane < L) {  // rows are padded to 4 tokens
    const float* lse = a.lse + (int64_t)s * HQ;
    const float* x = a.scores + ((int64_t)s * HQ + h0) * a.score_stride + t0 + 4 * lane;
#pragma unroll 8
    for (int h = h0; h < h1; ++h, x += a.score_stride) {
      const float4 v = *reinterpret_cast<const float4*>(x);
      const float z = lse[h];
      sum.x += exp2f(v.x - z);
      sum.y += exp2f(v.y - z);
      sum.z += exp2f(v.z - z);
      sum.w += exp2f(v.w - z);
    }
  }
  part[warp][lane] = sum;
  __syncthreads();
  const int t = t0 + threadIdx.x;
  if (threadIdx.x >= kMassTokens || t >= L) return;
  float w = 0.f;
#pragma unroll
  for (int i = 0; i < kMassWarps; ++i) w += reinterpret_cast<const float*>(part[i])[threadIdx.x];
  const int64_t at = s * m.stride + t;
  m.mass_out[at] = m.mass_in ? fmaf(m.decay, m.mass_in[at], w) : w;
}

}  // namespace pa
