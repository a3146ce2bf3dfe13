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
// Selecting is a radix selection of the keep-th key, 11 bits a pass.  A cluster
// of up to 8 CTAs takes a sequence, each a contiguous share of its slots, with the
// keys in shared memory: the track is read once, the passes add their
// histograms over distributed shared memory.  Moving is bound by memory: rows of
// one token and head (256 bytes at head_dim 128 in 16 bits) read and written once.
// Measured (8 heads x 128 fp16): 200 x up to 2048 to 1024, 34071 tokens moved, 14
// us selecting and 51 us moving 279 MB (5.5 TB/s); 8 x 32768 to 8192, 22 and 66
// us for 404 MB (6.1 TB/s).
#pragma once

#include <cooperative_groups.h>
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
  int4* heads;   // [S] number of moves, then the sequence's history before
  int2* moves;   // [S][move_cap] (source, destination) slots of the sequence
  uint32_t* err;
  int64_t num_blocks;
  int32_t max_blocks_per_seq;
  int32_t max_context_len;
  int32_t move_cap;
  int32_t sinks, recent;
};

constexpr int kEvictThreads = 1024;
constexpr int kEvictBins = 2048;
constexpr int kEvictMaxCluster = 8;
constexpr int kEvictCachedKeys = 40 * 1024;  // of one CTA, 160 KB; longer shares are read anew each pass

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

struct EvictShared {
  alignas(8) int hist[kEvictBins];
  int warp_sums[32];
  int counts[2][32];  // of each warp's slots
  uint32_t prefix;
  int need;
  int done;      // the pass that settled the selection, or -1
  int total[2];  // of this CTA's share
};

// One cluster per sequence.  CACHED: the CTA's keys are held in the dynamic
// shared memory.
template <bool CACHED>
__global__ void __launch_bounds__(kEvictThreads, 2) evict_select_kernel(EvictArgs a) {
  namespace cg = cooperative_groups;
  extern __shared__ uint32_t evict_keys[];
  __shared__ EvictShared sh;
  grid_dependents_launch();  // the moving kernel may start its CTAs; they wait for this grid
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int s = blockIdx.x / C, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t cap = min((int64_t)a.max_context_len, (int64_t)a.max_blocks_per_seq * kBlock);
  int L = a.context_lens[s];
  int keep = a.keep_lens[s];
  if (rank == 0 && tid == 0 && (L < 0 || L > cap || keep < 0)) atomicOr(a.err, PA_DEVERR_CONTEXT_LEN);
  L = L < 0 ? 0 : L > cap ? (int)cap : L;
  if (keep < 0) keep = L;
  const float* mass = a.mass_in + s * a.in_stride;
  const int32_t* pos = a.positions_in + s * a.in_stride;
  float* mass_out = a.mass_out + s * a.out_stride;
  int32_t* pos_out = a.positions_out + s * a.out_stride;
  const int held = a.history_in[2 * s], next = a.history_in[2 * s + 1];
  // a history that is not this sequence's (it shrank below `held`, or positions pass 32 bits): nothing is evicted
  if (keep < L && ((uint32_t)held > (uint32_t)L || (uint32_t)next > (uint32_t)(INT32_MAX - (L - held)))) {
    if (rank == 0 && tid == 0) atomicOr(a.err, PA_DEVERR_CONTEXT_LEN);
    keep = L;
  }
  // this CTA's slots, each warp's of them contiguous and a multiple of 32
  const int per = (L + C * kEvictThreads - 1) / (C * kEvictThreads) * kEvictThreads;
  const int lo = min(L, rank * per), hi = min(L, lo + per);
  if (keep >= L) {  // nothing to evict
    if (rank == 0 && tid == 0) {
      a.heads[s] = make_int4(0, held, next, 0);
      a.history_out[2 * s] = held;  // as it is: other CTAs may still read it in place
      a.history_out[2 * s + 1] = next;
    }
    if (mass_out != mass)
      for (int t = lo + tid; t < hi; t += kEvictThreads) mass_out[t] = mass[t];
    if (pos_out != pos)
      for (int t = lo + tid; t < hi; t += kEvictThreads) pos_out[t] = pos[t];
    return;  // the same in every CTA of the cluster
  }
  const int seen = next + L - held;
  auto position = [&](int t) { return t < held ? pos[t] : next + t - held; };
  auto make_key = [&](int t) {
    const int at = position(t);
    return at < a.sinks || at >= seen - a.recent ? 0xffffffffu : evict_key(mass[t]);
  };
  auto key = [&](int t) { return CACHED ? evict_keys[t - lo] : make_key(t); };
  if (CACHED)
    for (int t = lo + tid; t < hi; t += kEvictThreads) evict_keys[t - lo] = make_key(t);
  if (tid == 0) {
    sh.prefix = 0;
    sh.need = keep;
    sh.done = -1;
  }
  __syncthreads();  // keep == 0 goes past the loop's barriers
  // the keep-th largest key, from its first digit on; a pass whose whole bin stays is the last
  int pass = 0, shift = 0;
  for (; pass < 3 && keep > 0; ++pass) {
    shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t digit = pass == 2 ? 1023u : 2047u;
    for (int i = tid; i < kEvictBins; i += kEvictThreads) sh.hist[i] = 0;
    __syncthreads();
    const uint32_t prefix = sh.prefix;
    const int need = sh.need;
    for (int t = lo + tid; t < hi; t += kEvictThreads) {
      const uint32_t k = key(t);
      if (pass == 0 || (k >> (pass == 1 ? 21 : 10)) == prefix) atomicAdd(&sh.hist[(k >> shift) & digit], 1);
    }
    cluster.sync();
    // two bins a thread, the largest first, summed over the cluster
    int2 n = make_int2(0, 0);
#pragma unroll
    for (int c = 0; c < kEvictMaxCluster; ++c)
      if (c < C) {
        const int2 h = reinterpret_cast<const int2*>(cluster.map_shared_rank(sh.hist, c))[kEvictThreads - 1 - tid];
        n.x += h.y;
        n.y += h.x;
      }
    int total;
    const int above = block_scan(n.x + n.y, sh.warp_sums, &total);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int before = above + (e ? n.x : 0), in = e ? n.y : n.x;
      if (before < need && need <= before + in) {  // one thread of the block
        sh.prefix = (prefix << (pass == 2 ? 10 : 11)) | (uint32_t)(kEvictBins - 1 - 2 * tid - e);
        sh.need = need - before;
        if (need == before + in) sh.done = pass;
      }
    }
    cluster.sync();  // the histograms are free again
    if (sh.done == pass) break;
  }
  // Keys above `edge` stay, and of those equal to it the first `ties`.  A bin
  // that stays whole: its lowest key is the edge, without a limit.
  const uint32_t edge = sh.prefix << shift;
  const bool whole = sh.done >= 0;
  const int ties = sh.need;

  const int wlo = lo + warp * (per / 32), whi = min(hi, wlo + per / 32);
  // Sums of two counts over the warps before this one, in this CTA and in the
  // cluster's CTAs before it; *all: over the whole cluster.
  auto sums_before = [&](int2 mine, int2* all) {
    if (lane == 0) sh.counts[0][warp] = mine.x, sh.counts[1][warp] = mine.y;
    __syncthreads();
    const int x = sh.counts[0][lane], y = sh.counts[1][lane];
    int2 sum = make_int2(__reduce_add_sync(kFullMask, lane < warp ? x : 0), __reduce_add_sync(kFullMask, lane < warp ? y : 0));
    if (warp == 0) {
      const int tx = __reduce_add_sync(kFullMask, x), ty = __reduce_add_sync(kFullMask, y);
      if (lane == 0) sh.total[0] = tx, sh.total[1] = ty;
    }
    cluster.sync();
    int2 v = make_int2(0, 0);
    if (lane < C) {
      const int* t = cluster.map_shared_rank(sh.total, lane);
      v = make_int2(t[0], t[1]);
    }
    sum.x += __reduce_add_sync(kFullMask, lane < rank ? v.x : 0);
    sum.y += __reduce_add_sync(kFullMask, lane < rank ? v.y : 0);
    *all = make_int2(__reduce_add_sync(kFullMask, v.x), __reduce_add_sync(kFullMask, v.y));
    return sum;
  };
  // sweep 1, where not all tokens at the edge stay: their ranks
  int tie0 = 0;
  int2 all;
  if (!whole) {  // the same in every CTA of the cluster
    int count = 0;
    for (int t0 = wlo; t0 < whi; t0 += 32) {
      const int t = t0 + lane;
      count += __popc(__ballot_sync(kFullMask, t < whi && keep > 0 && key(t) == edge));
    }
    tie0 = sums_before(make_int2(count, 0), &all).x;
    cluster.sync();  // the totals are free again
  }
  // Who stays in the 32 slots from t0 on; tie: rank of the first token at the edge.
  auto stays_of = [&](int t0, int& tie) {
    const int t = t0 + lane;
    const bool real = t < whi && keep > 0;
    const uint32_t k = real ? key(t) : 0u;
    if (whole) return real && k >= edge;
    const uint32_t edges = __ballot_sync(kFullMask, real && k == edge);
    const bool stays = real && (k > edge || (k == edge && tie + __popc(edges & ((1u << lane) - 1u)) < ties));
    tie += __popc(edges);
    return stays;
  };
  // sweep 2: holes and movers of every warp
  int holes = 0, movers = 0, tie = tie0;
  for (int t0 = wlo; t0 < whi; t0 += 32) {
    const int t = t0 + lane;
    const bool stays = stays_of(t0, tie);
    holes += __popc(__ballot_sync(kFullMask, t < whi && t < keep && !stays));
    movers += __popc(__ballot_sync(kFullMask, t >= keep && stays));
  }
  const int2 first = sums_before(make_int2(holes, movers), &all);
  int hole = first.x, mover = first.y;
  const int all_movers = all.y;
  // sweep 3: the moves, and the track of what is not moved
  int2* moves = a.moves + (int64_t)s * a.move_cap;
  tie = tie0;
  for (int t0 = wlo; t0 < whi; t0 += 32) {
    const int t = t0 + lane;
    const bool stays = stays_of(t0, tie);
    const bool is_hole = t < whi && t < keep && !stays, is_mover = t >= keep && stays;
    const uint32_t hb = __ballot_sync(kFullMask, is_hole), mb = __ballot_sync(kFullMask, is_mover);
    const uint32_t below = (1u << lane) - 1u;
    if (is_hole) moves[hole + __popc(hb & below)].y = t;
    if (is_mover) moves[mover + __popc(mb & below)].x = t;
    hole += __popc(hb);
    mover += __popc(mb);
    if (t < keep && stays) {
      const int at = position(t);
      if (mass_out != mass) mass_out[t] = mass[t];
      pos_out[t] = at;
    } else if (t < whi && t >= keep && !stays) {
      mass_out[t] = 0.f;
    }
  }
  if (rank == 0 && tid == 0) {
    a.heads[s] = make_int4(all_movers, held, next, 0);
    a.history_out[2 * s] = keep;
    a.history_out[2 * s + 1] = seen;
  }
  cluster.sync();  // no CTA leaves while another may read its shared memory
}

constexpr int kEvictMovesPerCta = 16;

// Move the K and V rows of the listed tokens and their tracks.  `units` 16-byte
// copies make a head's row; 4-bit rows have their group words beside them.
template <bool Q4>
__global__ void __launch_bounds__(256)
    evict_move_kernel(EvictArgs a, uint8_t* __restrict__ k_pool, uint8_t* __restrict__ v_pool, int heads,
                      int D, int units) {
  __shared__ int2 slots[kEvictMovesPerCta];  // physical, -1: a bad block id
  grid_dependency_wait();  // the selecting kernel
  const int s = blockIdx.y;
  const int4 head = a.heads[s];
  const int32_t* table = a.block_tables + (int64_t)s * a.max_blocks_per_seq;
  for (int m0 = blockIdx.x * kEvictMovesPerCta; m0 < head.x; m0 += gridDim.x * kEvictMovesPerCta) {
    const int n = min(kEvictMovesPerCta, head.x - m0);
    __syncthreads();  // slots are free again
    if (threadIdx.x < 32) {  // two lanes a move: its source and its destination
      const bool live = threadIdx.x < 2 * n;
      const int2 mv = live ? a.moves[(int64_t)s * a.move_cap + m0 + threadIdx.x / 2] : make_int2(0, 0);
      const int t = (threadIdx.x & 1) ? mv.y : mv.x;
      int slot = -1;
      if (live) {
        const int32_t b = table[t / kBlock];
        if (b < 0 || b >= a.num_blocks) atomicOr(a.err, PA_DEVERR_BLOCK_ID);
        else slot = b * kBlock + t % kBlock;
      }
      const int other = __shfl_xor_sync(kFullMask, slot, 1);  // by all lanes, before any condition
      const bool whole = slot >= 0 && other >= 0;
      if (live) reinterpret_cast<int*>(slots)[threadIdx.x] = whole ? slot : -1;
      if (live && (threadIdx.x & 1) == 0) {
        // the token's track; its old slot starts from 0 again.  A move from or to a bad block is dropped: the
        // destination keeps its own token, and that one's track
        const int from = whole ? mv.x : mv.y;
        const int64_t in = s * a.in_stride + from, out = s * a.out_stride;
        const float mass = a.mass_in[in];
        const int at = from < head.y ? a.positions_in[in] : head.z + from - head.y;
        a.mass_out[out + mv.y] = mass;
        a.positions_out[out + mv.y] = at;
        a.mass_out[out + mv.x] = 0.f;
      }
    }
    __syncthreads();
    const int per = heads * units, total = n * per;
    // (in-block row, 16-byte units) of a slot's row of a head
    auto at = [&](int slot, int h, int c) {
      if constexpr (Q4)
        return ((int64_t)(slot >> 4) * heads + h) * q4_tile_bytes(D) + c * 256 + (slot & 15) * 16;
      else
        return ((((int64_t)(slot >> 4) * heads + h) * 16 + (slot & 15)) * units + c) * 16;
    };
    constexpr int U = 4;  // copies of K and of V in flight in a thread
    for (int i0 = threadIdx.x; i0 < total; i0 += U * 256) {
      uint4 kv[U][2];
      int64_t to[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * 256;
        to[u] = -1;
        if (i < total) {
          const int m = i / per, rest = i - m * per, h = rest / units, c = rest - h * units;
          const int2 mv = slots[m];
          if (mv.x >= 0 && mv.y >= 0) {
            const int64_t from = at(mv.x, h, c);
            to[u] = at(mv.y, h, c);
            kv[u][0] = *reinterpret_cast<const uint4*>(k_pool + from);
            kv[u][1] = *reinterpret_cast<const uint4*>(v_pool + from);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (to[u] >= 0) {
          *reinterpret_cast<uint4*>(k_pool + to[u]) = kv[u][0];
          *reinterpret_cast<uint4*>(v_pool + to[u]) = kv[u][1];
        }
    }
    if constexpr (Q4) {  // the group words
      const int groups = D / 64, words = heads * groups;
      for (int i = threadIdx.x; i < n * words; i += 256) {
        const int m = i / words, rest = i - m * words, h = rest / groups, g = rest - h * groups;
        const int2 mv = slots[m];
        if (mv.x < 0 || mv.y < 0) continue;
        auto word = [&](int slot) {
          return ((int64_t)(slot >> 4) * heads + h) * q4_tile_bytes(D) + q4_words_off(D) +
                 (g * 16 + (slot & 15)) * 4;
        };
        const int64_t from = word(mv.x), dst = word(mv.y);
        const uint32_t kw = *reinterpret_cast<const uint32_t*>(k_pool + from);
        const uint32_t vw = *reinterpret_cast<const uint32_t*>(v_pool + from);
        *reinterpret_cast<uint32_t*>(k_pool + dst) = kw;
        *reinterpret_cast<uint32_t*>(v_pool + dst) = vw;
      }
    }
  }
}

}  // namespace pa
