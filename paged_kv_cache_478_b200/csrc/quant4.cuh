// The 4-bit pool: its format, and the kernels that write and convert it.
//
// Each (block, head) tile of a 4-bit K or V pool is 9 * D bytes:
//   [0, 8 D)    data [D / 32 pieces][16 tokens][16 bytes]: byte b of piece c
//               holds dimension 32 c + 2 b in its low half, 32 c + 2 b + 1 in
//               its high half;
//   [8 D, 9 D)  one 32-bit word per group of 64 dimensions, [D / 64][16
//               tokens]: the group's scale s (bf16) in the upper half, its
//               zero point z (a whole number, fp16) in the lower.
// A held number n stands for s * (n - z): 4.5 bits a value.  The 16-byte
// pieces of 8 consecutive tokens are 128 contiguous bytes, so that the matrix
// loads (ldmatrix) of the attention kernel are free of bank conflicts.
//
// Quantisation of a group of 64 values x, in fp32:
//   s = bf16(max((max x - min x) / 15, max |x| / 2000)),  z = round(-min x / s),
//   n = clamp(round(x / s) + z, 0, 15)       (n = z = 0 where s = 0).
// z may lie outside 0..15, so a group far from zero keeps the full
// resolution of its range; the second term of s keeps |z| below 2048, where
// fp16 holds every whole number.  The error is at most s / 2, and a few
// hundredths of s more at the upper end where s was rounded down.  n and z are
// those of exact quotients (q4_quotient).  Measured (32 heads x 128 fp16):
// append of 16384 tokens 86 us, 1024 blocks to 4 bits 69 us and back 65 us, for
// 344 MB each (4.0, 5.0 and 5.3 TB/s): bound by instructions one way, and by the
// latency of its loads the other, where n - z two at a time in fp16 was no faster.
// A group that holds an infinity or NaN, or whose range passes fp32, gets s = NaN
// and reads back as NaN.
#pragma once

#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "device_utils.cuh"
#include "pagedattn.h"
#include "plan.cuh"

namespace pa {

// Bytes of one (block, head) tile, and the offset of its words.
__host__ __device__ constexpr int q4_tile_bytes(int D) { return 9 * D; }
__host__ __device__ constexpr int q4_words_off(int D) { return 8 * D; }

__device__ __forceinline__ float q4_scale(uint32_t word) { return __uint_as_float(word & 0xffff0000u); }
__device__ __forceinline__ float q4_zero(uint32_t word) {
  return __half2float(__ushort_as_half((unsigned short)(word & 0xffffu)));
}

template <typename T>
struct Pair;
template <>
struct Pair<__half> {
  using V = __half2;
  __device__ __forceinline__ static V max_nan(V a, V b) { return __hmax2_nan(a, b); }
  __device__ __forceinline__ static V min_nan(V a, V b) { return __hmin2_nan(a, b); }
  __device__ __forceinline__ static float2 floats(V a) { return __half22float2(a); }
};
template <>
struct Pair<__nv_bfloat16> {
  using V = __nv_bfloat162;
  __device__ __forceinline__ static V max_nan(V a, V b) { return __hmax2_nan(a, b); }
  __device__ __forceinline__ static V min_nan(V a, V b) { return __hmin2_nan(a, b); }
  __device__ __forceinline__ static float2 floats(V a) { return __bfloat1622float2(a); }
};

constexpr float kRoundMagic = 12582912.f;  // 1.5 * 2^23: x + kRoundMagic holds round(x) in its low bits

// round(x / s) + kRoundMagic, given inv = 1 / s rounded, halves to even as
// the exact quotient has them; |x / s| < 2048.  The product with 1.5 2^12 added is
// rounded to a multiple of 2^-11.  x inv is off by less than 2^-24 of 2048 = 2^-13,
// so a half comes back to its place.  A quotient of 11 by 8 significant bits that is
// no half is X / (S 2^t) with X < 2^11 and S < 2^8: where t <= 0 it differs from one by
// 2^-9, else by 1 / (S 2^t), which is above 2^-12 (half a step) beside 1/2 except
// for 2047 / 4096, where a step's tie goes to 1/2 and, like itself, to 0.
__device__ __forceinline__ float q4_quotient(float x, float inv) {
  constexpr float kSteps = 6144.f;
  return __fadd_rn(__fmaf_rn(x, inv, kSteps), kRoundMagic - kSteps);
}

// The largest value of a group and the smallest, negated, as a pair in the
// 16-bit type, NaN winning: the same in all of the group's 8 lanes.
template <typename T>
__device__ __forceinline__ uint32_t q4_extent(const uint4& u) {
  using P = Pair<T>;
  using V = typename P::V;
  auto as_v = [](uint32_t x) { return *reinterpret_cast<const V*>(&x); };
  auto as_u = [](V x) { return *reinterpret_cast<uint32_t*>(&x); };
  const V m = P::max_nan(P::max_nan(as_v(u.x), as_v(u.y)), P::max_nan(as_v(u.z), as_v(u.w)));
  const V l = P::min_nan(P::min_nan(as_v(u.x), as_v(u.y)), P::min_nan(as_v(u.z), as_v(u.w)));
  const uint32_t mu = as_u(m), lu = as_u(l) ^ 0x80008000u;
  V top = P::max_nan(as_v(__byte_perm(mu, lu, 0x5410)), as_v(__byte_perm(mu, lu, 0x7632)));
#pragma unroll
  for (int k = 1; k < 8; k <<= 1) top = P::max_nan(top, as_v(__shfl_xor_sync(kFullMask, as_u(top), k)));
  return as_u(top);
}

// A lane's 8 numbers, the first in the lowest 4 bits, given the group's
// scale, its reciprocal and zero point.
template <typename T>
__device__ __forceinline__ uint32_t q4_numbers(const uint4& u, float s, float inv, int z) {
  uint32_t n = 0;
  float x[8];
  Chunk<T>::to_float(u, x);
  if (s >= 1e-36f) {
    const int off = z - __float_as_int(kRoundMagic);
#pragma unroll
    for (int e = 0; e < 8; ++e)  // clamp(round(x / s) + z, 0, 15)
      n += (uint32_t)__viaddmin_s32_relu(__float_as_int(q4_quotient(x[e], inv)), off, 15) << (4 * e);
  } else if (s > 0.f) {  // 1 / s or a product may leave the normal numbers: divide
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float v = fminf(fmaxf(rintf(__fdiv_rn(x[e], s)) + (float)z, 0.f), 15.f);
      n |= (uint32_t)v << (4 * e);
    }
  }
  return n;  // 0 in a group of zeros and where s is NaN
}

// Quantise two K and two V groups of 64 values (k[u], v[u]), each held by 8
// neighbouring lanes, 8 each (all 32 lanes of the warp call).  kn[u] and vn[u] are the
// lane's numbers.  Of the 8 lanes, 2 u and 2 u + 1 work out the scale of K's group u,
// 4 + 2 u and 5 + 2 u of V's, and *word is its word.
template <typename T>
__device__ __forceinline__ void q4_quantise(const uint4* k, const uint4* v, int lane, uint32_t* kn,
                                            uint32_t* vn, uint32_t* word) {
  using V = typename Pair<T>::V;
  const uint32_t e0 = q4_extent<T>(k[0]), e1 = q4_extent<T>(k[1]);
  const uint32_t e2 = q4_extent<T>(v[0]), e3 = q4_extent<T>(v[1]);
  const uint32_t mine = (lane & 4) ? ((lane & 2) ? e3 : e2) : ((lane & 2) ? e1 : e0);
  const float2 ends = Pair<T>::floats(*reinterpret_cast<const V*>(&mine));
  const float hi = ends.x, lo = -ends.y;
  float raw = __fdiv_rn(__fsub_rn(hi, lo), 15.f);
  const float big = fmaxf(fabsf(hi), fabsf(lo));
  if (big > 1990.f * raw) raw = fmaxf(raw, __fdiv_rn(big, 2000.f));  // the other quotient may be the larger
  float s = __bfloat162float(__float2bfloat16_rn(raw));
  if (!(s < INFINITY)) s = __uint_as_float(0x7fc00000u);
  float inv = 0.f;
  int z = 0;
  if (s >= 1e-36f) {
    inv = __frcp_rn(s);
    z = __float_as_int(q4_quotient(-lo, inv)) - __float_as_int(kRoundMagic);
  } else if (s > 0.f) {
    z = (int)rintf(__fdiv_rn(-lo, s));
  }
  *word = __float_as_uint(s) | (uint32_t)__half_as_ushort(__int2half_rn(z));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int from = (lane & 24) + 2 * i;
    const float si = __shfl_sync(kFullMask, s, from), ii = __shfl_sync(kFullMask, inv, from);
    const int zi = __shfl_sync(kFullMask, z, from);
    (i < 2 ? kn[i & 1] : vn[i & 1]) = q4_numbers<T>(i < 2 ? k[i & 1] : v[i & 1], si, ii, zi);
  }
}

// Where the lane's 8 numbers of (row t, group g) go in a tile: lane j of the
// 8 holds dimensions 64 g + 8 j .. + 7.
__device__ __forceinline__ int q4_data_off(int g, int j, int t) {
  return (2 * g + (j >> 2)) * 256 + t * 16 + (j & 3) * 4;
}

// a / b, by 32-bit division where both fit (a 64-bit one costs as much as
// quantising four values).
__device__ __forceinline__ int64_t q4_div(int64_t a, int b) {
  return a <= 0xffffffffll ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// Append: each new token's K and V rows are quantised into the slot that
// slot_mapping names.  Eight lanes take one (token, head, group of 64), a warp
// U x 4 neighbouring ones a round, their loads in flight together: one 16-byte
// load of K and of V per lane, one 4-byte store each.
template <typename T>
__global__ void __launch_bounds__(256)
    q4_append_kernel(const T* __restrict__ k_new, const T* __restrict__ v_new,
                     const int32_t* __restrict__ slot_mapping, uint8_t* __restrict__ k_pool,
                     uint8_t* __restrict__ v_pool, int heads, int D, int64_t num_tokens,
                     int64_t num_slots, uint32_t* err) {
  constexpr int U = 2;
  const int lane = threadIdx.x & 31, j = lane & 7;
  const int groups = D / 64;
  const int64_t total = num_tokens * heads * groups;
  // every lane of a warp runs the same number of rounds (the shuffles need all of them)
  for (int64_t w = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5; w * 4 * U < total;
       w += ((int64_t)gridDim.x * blockDim.x) >> 5) {
    uint4 ku[U], vu[U];
    int32_t slot[U];
    int h[U], g[U];
    const int64_t u0 = w * U * 4 + (lane >> 3);
    int64_t row = u0 >> (groups - 1);  // token * heads + head; groups is 1 or 2
    int64_t t = q4_div(row, heads);
    int head = (int)(row - t * heads);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const bool live = u0 + 4 * i < total;
      if (i > 0) {  // four units on
        row += 4 >> (groups - 1);
        head += 4 >> (groups - 1);
        while (head >= heads) head -= heads, ++t;
      }
      g[i] = (int)u0 & (groups - 1);
      h[i] = head;
      slot[i] = live ? slot_mapping[t] : -1;
      const int64_t src = live ? row * D + g[i] * 64 + j * 8 : 0;
      ku[i] = *reinterpret_cast<const uint4*>(k_new + src);
      vu[i] = *reinterpret_cast<const uint4*>(v_new + src);
    }
    uint32_t kn[U], vn[U], word;
    q4_quantise<T>(ku, vu, lane, kn, vn, &word);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (slot[i] >= num_slots && h[i] == 0 && g[i] == 0 && j == 0) atomicOr(err, PA_DEVERR_SLOT);
      if (slot[i] >= 0 && slot[i] < num_slots) {  // a negative slot is padding
        const int64_t tile = ((int64_t)(slot[i] >> 4) * heads + h[i]) * q4_tile_bytes(D);
        const int r = slot[i] & 15;
        *reinterpret_cast<uint32_t*>(k_pool + tile + q4_data_off(g[i], j, r)) = kn[i];
        *reinterpret_cast<uint32_t*>(v_pool + tile + q4_data_off(g[i], j, r)) = vn[i];
        if ((j & 3) == 2 * i)
          *reinterpret_cast<uint32_t*>((j < 4 ? k_pool : v_pool) + tile + q4_words_off(D) + (g[i] * 16 + r) * 4) = word;
      }
    }
  }
}

// The same for each sequence's new token, k_new and v_new [S][heads][D], at the
// last position of its planned length (the fused append's contract).
template <typename T>
__global__ void __launch_bounds__(256)
    q4_append_last_kernel(DecodeArgs a, const T* __restrict__ k_new, const T* __restrict__ v_new, int D) {
  if (!plan_header_ok(a)) return;  // the decode launch that follows reports it
  const int lane = threadIdx.x & 31, j = lane & 7;
  const int groups = D / 64;
  const int64_t total = (int64_t)a.num_seqs * a.heads * groups;
  const int64_t cap = min((int64_t)a.max_context_len, (int64_t)a.max_blocks_per_seq * kBlock);
  constexpr int U = 2;
  for (int64_t w = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5; w * 4 * U < total;
       w += ((int64_t)gridDim.x * blockDim.x) >> 5) {
    uint4 ku[U], vu[U];
    bool write[U];
    int64_t tile[U];
    int g[U], r[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t u = (w * U + i) * 4 + (lane >> 3);
      const bool live = u < total;
      const int64_t row = live ? u >> (groups - 1) : 0;  // sequence * heads + head
      g[i] = live ? (int)(u - row * groups) : 0;
      const int s = (int)q4_div(row, a.heads);
      const int h = (int)(row - (int64_t)s * a.heads);
      const int L = live ? a.lens[s] : 0;
      write[i] = L > 0 && L <= cap;
      int32_t b = 0;
      if (write[i]) {
        b = a.block_tables[(int64_t)s * a.max_blocks_per_seq + (L - 1) / kBlock];
        write[i] = b >= 0 && b < a.num_blocks;  // the decode launch reports a bad one
      }
      ku[i] = vu[i] = make_uint4(0, 0, 0, 0);
      if (write[i]) {
        const int64_t src = row * D + g[i] * 64 + j * 8;
        ku[i] = *reinterpret_cast<const uint4*>(k_new + src);
        vu[i] = *reinterpret_cast<const uint4*>(v_new + src);
      }
      tile[i] = ((int64_t)b * a.heads + h) * q4_tile_bytes(D);
      r[i] = (L - 1) & (kBlock - 1);
    }
    uint32_t kn[U], vn[U], word;
    q4_quantise<T>(ku, vu, lane, kn, vn, &word);
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (write[i]) {
        uint8_t* kt = static_cast<uint8_t*>(const_cast<void*>(a.k_pool)) + tile[i];
        uint8_t* vt = static_cast<uint8_t*>(const_cast<void*>(a.v_pool)) + tile[i];
        *reinterpret_cast<uint32_t*>(kt + q4_data_off(g[i], j, r[i])) = kn[i];
        *reinterpret_cast<uint32_t*>(vt + q4_data_off(g[i], j, r[i])) = vn[i];
        if ((j & 3) == 2 * i)
          *reinterpret_cast<uint32_t*>((j < 4 ? kt : vt) + q4_words_off(D) + (g[i] * 16 + r[i]) * 4) = word;
      }
  }
}

// Whole blocks from a 16-bit pool into a 4-bit one (PACK) or back, for every
// (src, dst) pair.  A warp takes a (pair, head) tile, 4 tokens of one group of 64
// dimensions a step, 8 lanes a token: 16-byte loads or stores of the wide rows,
// 4-byte ones of the pieces, of which a step's four tokens are contiguous.  The
// loads of U steps are in flight together.
template <typename T, bool PACK>
__global__ void __launch_bounds__(256)
    q4_convert_kernel(const uint8_t* __restrict__ k_src, const uint8_t* __restrict__ v_src,
                      uint8_t* __restrict__ k_dst, uint8_t* __restrict__ v_dst,
                      const int32_t* __restrict__ pairs, int64_t num_pairs, int64_t src_blocks,
                      int64_t dst_blocks, int heads, int D, uint32_t* err) {
  constexpr int U = PACK ? 2 : 4;
  const int lane = threadIdx.x & 31, j = lane & 7;
  const int groups = D / 64, steps = 4 * groups;
  const int64_t wide = (int64_t)kBlock * D * sizeof(T);
  const int narrow = q4_tile_bytes(D);
  const int64_t tiles = num_pairs * heads, warps = ((int64_t)gridDim.x * blockDim.x) >> 5;
  for (int64_t tile = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5; tile < tiles; tile += warps) {
    const int64_t p = q4_div(tile, heads);
    const int h = (int)(tile - p * heads);
    const int32_t src = pairs[2 * p], dst = pairs[2 * p + 1];
    if (src < 0 || src >= src_blocks || dst < 0 || dst >= dst_blocks) {
      if (h == 0 && lane == 0) atomicOr(err, PA_DEVERR_PAIR);
      continue;
    }
    const int64_t from = ((int64_t)src * heads + h) * (PACK ? wide : narrow);
    const int64_t to = ((int64_t)dst * heads + h) * (PACK ? narrow : wide);
    const uint8_t *k_in = k_src + from, *v_in = v_src + from;
    uint8_t *k_out = k_dst + to, *v_out = v_dst + to;
    for (int i0 = 0; i0 < steps; i0 += U) {
      int g[U], t[U], row16[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        g[u] = (i0 + u) >> 2;
        t[u] = ((i0 + u) & 3) * 4 + (lane >> 3);
        row16[u] = (t[u] * D + g[u] * 64 + j * 8) * (int)sizeof(T);
      }
      if constexpr (PACK) {
        uint4 ku[U], vu[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          ku[u] = *reinterpret_cast<const uint4*>(k_in + row16[u]);
          vu[u] = *reinterpret_cast<const uint4*>(v_in + row16[u]);
        }
        uint32_t kn[U], vn[U], word;
        q4_quantise<T>(ku, vu, lane, kn, vn, &word);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          *reinterpret_cast<uint32_t*>(k_out + q4_data_off(g[u], j, t[u])) = kn[u];
          *reinterpret_cast<uint32_t*>(v_out + q4_data_off(g[u], j, t[u])) = vn[u];
          if ((j & 3) == 2 * u)
            *reinterpret_cast<uint32_t*>((j < 4 ? k_out : v_out) + q4_words_off(D) + (g[u] * 16 + t[u]) * 4) = word;
        }
      } else {
        // the largest finite value of T: the last step of a group may pass it
        constexpr float kTop = std::is_same<T, __half>::value ? 65504.f : 3.38953139e38f;
        uint32_t n[U][2], word[U][2];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int data = q4_data_off(g[u], j, t[u]), w = q4_words_off(D) + (g[u] * 16 + t[u]) * 4;
          n[u][0] = *reinterpret_cast<const uint32_t*>(k_in + data);
          n[u][1] = *reinterpret_cast<const uint32_t*>(v_in + data);
          word[u][0] = *reinterpret_cast<const uint32_t*>(k_in + w);
          word[u][1] = *reinterpret_cast<const uint32_t*>(v_in + w);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            const float s = q4_scale(word[u][kv]), z = q4_zero(word[u][kv]);
            const float base = 8388608.f + z;  // 2^23 + z: exact for the whole numbers that z may be
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)  // exact in fp32 (8 by 12 bits), rounded once to T below
              f[e] = s * (__uint_as_float(0x4b000000u | ((n[u][kv] >> (4 * e)) & 15u)) - base);
            if (!(fabsf(s) * fmaxf(15.f + z, 15.f - z) <= kTop)) {  // a value may pass the range, or s is NaN
#pragma unroll
              for (int e = 0; e < 8; ++e) f[e] = f[e] > kTop ? kTop : f[e] < -kTop ? -kTop : f[e];  // NaN stays
            }
            *reinterpret_cast<uint4*>((kv ? v_out : k_out) + row16[u]) = Chunk<T>::from_float(f);
          }
      }
    }
  }
}

}  // namespace pa
