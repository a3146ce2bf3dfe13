// Attention weight gathered per cached token, for eviction by weight.
//
//   mass_out[s][t] = decay * mass_in[s][t] + sum_h w(s, h, t),   t < L_s,
//   w(s, h, t) = softmax over t of scale * q[s][h] . K_t
// The decode kernels compute every score once; in their MASS instantiations
// they also store it (4 bytes a token and query head, against 4 D bytes of
// 16-bit K and V) and, per query head, the logarithm of its softmax sum, which
// is known only when the sequence's last partition is merged.  This kernel
// then turns the scores into weights and adds the heads in order, so that
// the result does not depend on how the work was split.
#pragma once

#include <math.h>
#include <stdint.h>

#include "device_utils.cuh"
#include "plan.cuh"

namespace pa {

struct MassArgs {
  const float* mass_in;  // null: zero
  float* mass_out;
  int64_t stride;  // tokens between sequences of mass_in and mass_out
  float decay;
};

// One thread per token: a block of 256 tokens of one sequence.
__global__ void __launch_bounds__(256) mass_kernel(DecodeArgs a, MassArgs m) {
  if (a.plan->stamp != a.stamp || a.plan->poisoned != 0) return;  // the decode launch reported it
  const int s = blockIdx.y;
  const int64_t cap = min((int64_t)a.max_context_len, (int64_t)a.max_blocks_per_seq * kBlock);
  const int L = a.lens[s];
  if (L < 0 || L > cap) return;  // a damaged plan entry: the decode launch reported it
  const int t = blockIdx.x * 256 + threadIdx.x;
  if (t >= L) return;
  const int HQ = a.heads * a.q_per_kv;
  const float* lse = a.lse + (int64_t)s * HQ;
  const float* x = a.scores + (int64_t)s * HQ * a.score_stride + t;
  float sum = 0.f;
#pragma unroll 8
  for (int h = 0; h < HQ; ++h) sum += exp2f(x[h * a.score_stride] - lse[h]);
  const int64_t at = s * m.stride + t;
  m.mass_out[at] = m.mass_in ? fmaf(m.decay, m.mass_in[at], sum) : sum;
}

}  // namespace pa
