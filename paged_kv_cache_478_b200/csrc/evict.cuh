// Eviction from the cache by accumulated attention weight.
//
// Of a sequence's L cached tokens, keep = keep_lens[s] stay: first the
// protected ones (original position below `sinks`, or among the last
// `recent` seen), then those of largest mass; ties go to the lowest slot.
// Attention does not depend on the order of the cached tokens, so nothing is
// shifted: a token that stays in a slot below `keep` stays where it is, and
// the i-th token that stays in a slot at or past `keep` moves into the i-th
// slot below `keep` that falls free (both in ascending order).  Sources and
// destinations are disjoint, so all moves run at once, in place, and their
// number is at most the number of tokens evicted.
//
// The track of a sequence: mass[t], positions[t] (the original position of
// the token in slot t, for t < held) and history = (held, next): slots at or
// past `held` arrived since, in order, from position `next` on.
#pragma once

#include <math.h>
#include <stdint.h>

#include "device_utils.cuh"
#include "pagedattn.h"
#include "plan.cuh"
#include "quant4.cuh"

namespace pa {

struct EvictArgs {
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* keep_lens;
  const float* mass_in;
  const int32_t* positions_in;
  const int32_t* history_in;
  float* mass_out;
  int32_t* positions_out;
  int32_t* history_out;
  int64_t in_stride, out_stride;
  int32_t* counts;  // [S] moves of each sequence
  int2* moves;      // [S][move_cap] (source, destination), physical slots
  uint32_t* err;
  int64_t num_blocks;
  int32_t max_blocks_per_seq;
  int32_t num_seqs;
  int32_t max_context_len;
  int32_t move_cap;
  int32_t sinks, recent;
};

// Order of eviction as an unsigned number: mass ascending, NaN above
// infinity, protected tokens above all.
__device__ __forceinline__ uint32_t evict_key(float mass) {
  if (mass != mass) return 0xfffffffeu;
  const uint32_t u = __float_as_uint(mass + 0.f);  // -0 counts as 0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive sum of v over the 1024 threads of the block; *total is the sum.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int y = __shfl_up_sync(kFullMask, x, m);
    if (lane >= m) x += y;
  }
  __syncthreads();  // warp_sums is free again
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int w = warp_sums[lane];
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const int y = __shfl_up_sync(kFullMask, w, m);
      if (lane >= m) w += y;
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  *total = warp_sums[31];
  return x - v + (warp > 0 ? warp_sums[warp - 1] : 0);
}

// One CTA per sequence: a radix selection of the keep-th key, 8 bits a pass,
// then the moves and the new track.
__global__ void __launch_bounds__(1024) evict_select_kernel(EvictArgs a) {
  __shared__ int hist[256];
  __shared__ int warp_sums[32];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  const int s = blockIdx.x, tid = threadIdx.x;
  const int64_t cap = min((int64_t)a.max_context_len, (int64_t)a.max_blocks_per_seq * kBlock);
  int L = a.context_lens[s];
  if (L < 0 || L > cap) {
    if (tid == 0) atomicOr(a.err, PA_DEVERR_CONTEXT_LEN);
    L = L < 0 ? 0 : (int)cap;
  }
  int keep = a.keep_lens[s];
  if (keep < 0) {
    if (tid == 0) atomicOr(a.err, PA_DEVERR_CONTEXT_LEN);
    keep = L;
  }
  const float* mass = a.mass_in + s * a.in_stride;
  const int32_t* pos = a.positions_in + s * a.in_stride;
  float* mass_out = a.mass_out + s * a.out_stride;
  int32_t* pos_out = a.positions_out + s * a.out_stride;
  const int held = a.history_in[2 * s], next = a.history_in[2 * s + 1];
  if (keep >= L) {  // nothing to evict
    if (tid == 0) {
      a.counts[s] = 0;
      a.history_out[2 * s] = held;
      a.history_out[2 * s + 1] = next;
    }
    if (mass_out != mass)
      for (int t = tid; t < L; t += 1024) mass_out[t] = mass[t];
    if (pos_out != pos)
      for (int t = tid; t < L; t += 1024) pos_out[t] = pos[t];
    return;
  }
  const int seen = next + L - held;
  auto position = [&](int t) { return t < held ? pos[t] : next + t - held; };
  auto key = [&](int t) {
    const int at = position(t);
    return at < a.sinks || at >= seen - a.recent ? 0xffffffffu : evict_key(mass[t]);
  };
  // the keep-th largest key, and how many tokens of that key stay
  if (tid == 0) {
    s_prefix = 0;
    s_need = keep;
  }
  for (int shift = 24; shift >= 0 && keep > 0; shift -= 8) {
    for (int i = tid; i < 256; i += 1024) hist[i] = 0;
    __syncthreads();
    const uint32_t prefix = s_prefix;
    for (int t = tid; t < L; t += 1024) {
      const uint32_t k = key(t);
      if (shift == 24 || (k >> (shift + 8)) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1);
    }
    __syncthreads();
    if (tid == 0) {
      int need = s_need, b = 255;
      while (b > 0 && hist[b] < need) need -= hist[b--];
      s_prefix = (prefix << 8) | (uint32_t)b;
      s_need = need;
    }
    __syncthreads();
  }
  __syncthreads();
  const uint32_t edge = s_prefix;
  const int ties = s_need;  // of the tokens at the edge, the first this many stay
  int2* moves = a.moves + (int64_t)s * a.move_cap;
  int done_ties = 0, holes = 0, movers = 0;
  for (int t0 = 0; t0 < L; t0 += 1024) {
    const int t = t0 + tid;
    const uint32_t k = t < L ? key(t) : 0u;
    const bool tie = t < L && keep > 0 && k == edge;
    int n;
    const int rank = done_ties + block_scan(tie, warp_sums, &n);
    done_ties += n;
    const bool stays = t < L && keep > 0 && (k > edge || (tie && rank < ties));
    const bool hole = t < keep && !stays, mover = t >= keep && stays;
    const int hi = holes + block_scan(hole, warp_sums, &n);
    holes += n;
    const int mi = movers + block_scan(mover, warp_sums, &n);
    movers += n;
    if (hole) moves[hi].y = t;
    if (mover) moves[mi].x = t;
    if (t < keep && stays) {
      const int at = position(t);
      if (mass_out != mass) mass_out[t] = mass[t];
      pos_out[t] = at;
    }
  }
  __syncthreads();
  const int32_t* table = a.block_tables + (int64_t)s * a.max_blocks_per_seq;
  auto physical = [&](int t) {
    int32_t b = table[t / kBlock];
    if (b < 0 || b >= a.num_blocks) {
      atomicOr(a.err, PA_DEVERR_BLOCK_ID);
      return -1;
    }
    return b * kBlock + t % kBlock;
  };
  for (int i = tid; i < movers; i += 1024) {
    const int2 mv = moves[i];
    mass_out[mv.y] = mass[mv.x];
    pos_out[mv.y] = position(mv.x);
    moves[i] = make_int2(physical(mv.x), physical(mv.y));
  }
  __syncthreads();
  for (int t = keep + tid; t < L; t += 1024) mass_out[t] = 0.f;
  if (tid == 0) {
    a.counts[s] = movers;
    a.history_out[2 * s] = keep;
    a.history_out[2 * s + 1] = seen;
  }
}

// Move the K and V rows of every listed token: one thread per 16-byte chunk
// (4-byte word of a 4-bit pool), heads innermost but one.
// row_chunks: 16-byte chunks per row of a head.
__global__ void __launch_bounds__(256)
    evict_move_kernel(EvictArgs a, uint4* __restrict__ k_pool, uint4* __restrict__ v_pool, int heads,
                      int row_chunks) {
  const int s = blockIdx.y;
  const int n = a.counts[s];
  const int64_t per = (int64_t)heads * row_chunks, total = n * per;
  const int2* moves = a.moves + (int64_t)s * a.move_cap;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t m = i / per;
    const int rest = (int)(i - m * per);
    const int h = rest / row_chunks, c = rest - h * row_chunks;
    const int2 mv = moves[m];
    if (mv.x < 0 || mv.y < 0) continue;  // a bad block id, reported
    const int64_t src = (((int64_t)(mv.x >> 4) * heads + h) * 16 + (mv.x & 15)) * row_chunks + c;
    const int64_t dst = (((int64_t)(mv.y >> 4) * heads + h) * 16 + (mv.y & 15)) * row_chunks + c;
    k_pool[dst] = k_pool[src];
    v_pool[dst] = v_pool[src];
  }
}

// The same for 4-bit pools: D / 8 data words and D / 64 group words a row.
__global__ void __launch_bounds__(256)
    evict_move_q4_kernel(EvictArgs a, uint8_t* __restrict__ k_pool, uint8_t* __restrict__ v_pool,
                         int heads, int D) {
  const int s = blockIdx.y;
  const int n = a.counts[s];
  const int data = D / 8, words = data + D / 64;
  const int64_t per = (int64_t)heads * words, total = n * per;
  const int2* moves = a.moves + (int64_t)s * a.move_cap;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t m = i / per;
    const int rest = (int)(i - m * per);
    const int h = rest / words, c = rest - h * words;
    const int2 mv = moves[m];
    if (mv.x < 0 || mv.y < 0) continue;
    auto at = [&](int slot) {
      const int64_t tile = ((int64_t)(slot >> 4) * heads + h) * q4_tile_bytes(D);
      return tile + (c < data ? (c / 4) * 256 + (slot & 15) * 16 + (c % 4) * 4
                              : q4_words_off(D) + ((c - data) * 16 + (slot & 15)) * 4);
    };
    const int64_t src = at(mv.x), dst = at(mv.y);
    *reinterpret_cast<uint32_t*>(k_pool + dst) = *reinterpret_cast<const uint32_t*>(k_pool + src);
    *reinterpret_cast<uint32_t*>(v_pool + dst) = *reinterpret_cast<const uint32_t*>(v_pool + src);
  }
}

}  // namespace pa
