// Decode attention over 4-bit pools (quant4.cuh has the format).
//
// Work items, plan, split-K partials and merge are those of the other decode
// kernels (plan.cuh, decode.cuh).  A warp streams the K and V tiles of one KV
// head through its own ring of bulk copies, 64 tokens (4 blocks) a stage, and
// serves all G query heads of it.
//
// The products run on the tensor cores, the held numbers n in one of two forms.
//   fp16: 4 bits n in the low bits of an fp16 word ARE the number n 2^-24 (a
//     subnormal), and bits 4-7 are n 2^-20, so one AND and one fp16 FMA make
//     (n - z) 2^-10 of two numbers, exactly (|n - z| is below 2048).  Feeding the
//     subnormals themselves to the matrix instructions would save the FMA, but
//     those line up a sum by the exponents its operands are written with:
//     subnormals cost it 6 to 10 bits (measured: sums off by 2^-18 of their terms).
//   bytes: one AND, and for the odd numbers a shift, make four numbers.
//
//   scores:  x_t = sum_g s_t,g (sum_d q_d n_t,d - z_t,g sum_d q_d), g a group of 64
//     dimensions.  K is the A operand (16 tokens), Q the B operand (8 columns).
//     One or two query heads: byte products with 32-bit integer sums.  Q becomes
//     whole numbers, the row's largest in [2^21, 2^22) (off by at most 2^-22 of it;
//     exact for what is not below 2^-11 of the largest, bf16 2^-14), of three signed
//     base-256 digits, each in a column of its own; the sums are exact, and the quad's
//     lanes, which hold a digit each, add their shares in fp32.
//     Four or eight heads need the columns: fp16, Q scaled by a power of two into
//     its range, fp32 sums.  A lane gets the scores of tokens lane / 4 and lane / 4 + 8
//     of each block and of heads 2 (lane % 4) and the next (of four heads, lane % 2).
//     In both, one word a token and group gives its zero point and its scale.
//   values:  o_d = sum_t P_t,g (n_t,d - z_t,g),  P_t,g = w_t s_t,g.
//     V^T is the A operand in fp16, exact; P, transposed 8 x 8 by movmatrix, the B
//     operand, as two fp16 numbers: its value and what that rounding left (2^-21 of P
//     together; the first alone, 2^-11, showed in outputs whose terms cancel).  Its
//     columns are the heads, in the lanes that hold their scores, times the groups
//     (up to four heads), times the two parts where room is left (one or two heads,
//     or four at head_dim 64); else the second part takes products of its own.  The
//     quad's lanes hold the same weights as often, so that one movmatrix makes all of it.
//     It costs 200 requests 98.3 -> 100.3 us, four heads 45.7 -> 47.5, eight 34.4 -> 36.9.
//   The weights' reference m follows the scores alone, w_t = 2^(x_t - m) up to 2^3, so
//     the softmax sum knows nothing of V.  P stays within fp16 by a factor of its own,
//     a power of two 2^k for each (head, group): P = w_t s_t,g 2^k.  It is lowered (with
//     a rescale of the accumulators) only when a P could pass 2^15, so that the chunk's
//     largest lies at 2^10, and rises again as m does: a P is a normal number down
//     to 2^-24 of the largest w_t s_t,g so far, whatever the scales of V.  Whether one
//     could pass 2^15 is told from the chunk's largest weight and largest scale; the
//     largest product is worked out only then.
// What bounds it: the unpacking.  Per 16 tokens of a KV head (2304 bytes of K and V) a
// launch issues 280 warp instructions in all with one query head, 375 with four and 403
// with eight; the unpacking itself is 64 AND and 64 fp16 FMA (with one or two heads K's
// half of that is 16 AND and 8 shifts).  Measured: one head, 200 requests, 515 MB, 100
// us; 8 x 32768 tokens x 32 heads 209 us (5.8 TB/s; copies alone run at 6.4; K by fp16
// too took about a tenth more).  Under sustained load the 1000 W cap takes the SM clock
// down by a tenth: 104 and 243 us.  Two heads, 200 x 16 KV heads, 258 MB: 68 us; four, 200
// x 8, 129 MB: 47 us; eight, 64 x 8, 77 MB: 37 us, one wave of items (plan entry, table and
// first copies 5 us, about six chunks of 3, merge 5).
// Tried on the fp16 form, when it took 227 us, and slower (the long case): 16 warps an SM at 128 registers
// (241 us), copying warps of their own with four heads a copy (242; with setmaxnreg
// 275), warps that take single heads by themselves (257), K as 64 + n with the constant
// taken off the sums (242), the shifts on the multiply pipe (256), e4m3 operands (285;
// mma.sync turns them into fp16 first).  V by byte products was left out: the
// zero points' share, taken off after the sums, would leave their rounding where n - z is 0.
// ldmatrix reads K rows (token, 16 bytes) as they lie; transposed, it pairs
// two tokens of V in each register.  The pieces of 8 tokens are 128 contiguous
// bytes, so both are free of bank conflicts.
#pragma once

#include <math.h>
#include <stdint.h>

#include "decode.cuh"
#include "decode_gqa.cuh"
#include "device_utils.cuh"
#include "mma_utils.cuh"
#include "quant4.cuh"

namespace pa {

constexpr int kQ4ChunkBlocks = 4;  // blocks a ring stage holds
constexpr int kQ4Chunk = kQ4ChunkBlocks * kBlock;

template <typename T, int D>
struct Q4Config {
  static constexpr int WARPS = 4;
  static constexpr int THREADS = WARPS * 32;
  static constexpr int CTAS_PER_SM = 3;  // by registers (168) and shared memory (74 KB)
  static constexpr int TILE = q4_tile_bytes(D);
  static constexpr int HALF = kQ4ChunkBlocks * TILE;  // the K (or V) tiles of a stage
  static constexpr int STAGE_BYTES = 2 * HALF;
  static constexpr int NSTAGE = D == 128 ? 2 : 4;
  static_assert(STAGE_BYTES % 128 == 0, "stages start 128-byte aligned");
  static size_t smem_bytes(int partition_size) {
    return (size_t)WARPS * NSTAGE * STAGE_BYTES + (size_t)WARPS * NSTAGE * 8 +
           (size_t)(partition_size / kBlock) * 4;
  }
};

// KV heads per work item: the CTA's four warps take four heads, or share two
// heads or one where the pool has no more.
inline int q4_heads_per_item(int heads) { return heads >= 4 ? 4 : heads >= 2 ? 2 : 1; }

template <typename T>
__device__ __forceinline__ void load8(const T* p, float* f) {
  Chunk<T>::to_float(*reinterpret_cast<const uint4*>(p), f);
}

__device__ __forceinline__ __half2 as_half2(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }
__device__ __forceinline__ uint32_t as_u32(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
constexpr uint32_t kMinus2m10 = 0x94009400u;  // -2^-10 in both halves

// (n - z) 2^-10 of the numbers in bits 0-3 (even) or 4-7 (odd) of both halves,
// given nz = -z 2^-10: exact.
__device__ __forceinline__ uint32_t q4_even(uint32_t w, __half2 nz) {
  return as_u32(__hfma2(as_half2(w & 0x000f000fu), as_half2(0x74007400u), nz));  // 2^14
}
__device__ __forceinline__ uint32_t q4_odd(uint32_t w, __half2 nz) {
  return as_u32(__hfma2(as_half2(w & 0x00f000f0u), as_half2(0x64006400u), nz));  // 2^10
}
__device__ __forceinline__ uint32_t pack_half(float a, float b) { return MmaType<__half>::pack(a, b); }

// One 8 x 8 matrix of 16-bit values across the warp, transposed.
__device__ __forceinline__ uint32_t movmatrix(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// 2^p of a whole number from -126 to 127.
__device__ __forceinline__ float pow2(int p) { return __uint_as_float((uint32_t)(p + 127) << 23); }

// scale * 2^p as two factors, for before and after the product with K's scale, which neither then takes out of
// fp32 where the score itself is in it.  The second is 1 but for queries of extreme sizes.
__device__ __forceinline__ float2 split_factor(float scale, int p) {
  return p > 0 ? make_float2(1.f, scale * pow2(p))
               : p < -64 ? make_float2(pow2(-64), scale * pow2(p + 64)) : make_float2(scale * pow2(p), 1.f);
}

// 2^x; results below the normal numbers become zero.
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Products of pairs in one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%2, %3};\n\tmov.b64 q, {%4, %5};\n\t"
      "mul.rn.f32x2 p, p, q;\n\tmov.b64 {%0, %1}, p;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// a - s * (the value that the pair a became in fp16, as the word h)
__device__ __forceinline__ float2 sub_half2(float2 a, uint32_t h, float s) {
  const float2 b = __half22float2(as_half2(h));
  return make_float2(fmaf(-s, b.x, a.x), fmaf(-s, b.y, a.y));
}

// d += a * b for one m16n8k32 tile, a of unsigned bytes, b of signed ones, 32-bit sums.
__device__ __forceinline__ void mma16832_u8s8(int* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
constexpr uint32_t kNibbles = 0x0f0f0f0fu;

// G: query heads per KV head.  NH: those a lane keeps scores of.  I8: the scores by
// byte products, the queries' digits in the columns.
template <typename T, int D, int G, bool MASS>
__global__ void __launch_bounds__(128, 3) paged_decode_q4_kernel(DecodeArgs a, int heads_per_item) {
  using Cfg = Q4Config<T, D>;
  constexpr int TILE = Cfg::TILE, NSTAGE = Cfg::NSTAGE;
  constexpr int PIECES = D / 32, GROUPS = D / 64;
  constexpr int CB = kQ4ChunkBlocks;
  constexpr bool I8 = G <= 2;
  constexpr int NH = G == 1 ? 1 : 2;
  // What the columns of P hold beside the heads: the groups (G <= 4), and what P's rounding left where room is left
  constexpr bool GROUP_COLS = GROUPS == 2 && G <= 4, REST_COLS = G <= 2 || (G == 4 && GROUPS == 1);
  // m follows a score beyond 2^kMove: w s stays below 2^127.2, V's scales being below 2^124.2
  constexpr float kMove = 3.f;
  // P's factor 2^k is at most 2^126, lowered where P may pass kPMove, so that the largest lies in [2^10, 2^11):
  // by biased exponents, that of the largest w s and the factor's add up to kFactorPut
  constexpr float kPMove = 32768.f;
  constexpr int kFactorTop = 126 + 127, kFactorPut = 10 + 2 * 127;
  constexpr int FG = GROUP_COLS ? 1 : GROUPS;  // groups whose factor a lane keeps

  extern __shared__ __align__(128) uint8_t q4_smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(q4_smem + Cfg::WARPS * NSTAGE * Cfg::STAGE_BYTES);
  int32_t* tbl = reinterpret_cast<int32_t*>(bars + Cfg::WARPS * NSTAGE);
  __shared__ int32_t s_item, s_abort, s_merge, s_plan_ok;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = lane >> 2, j = lane & 3;  // fragment row (query head, or dimension) and quad lane
  // the lane's heads are head0 and the next, its columns' group my_group (GROUP_COLS)
  const int head0 = I8 ? 0 : G == 4 ? 2 * (j & 1) : 2 * j, my_group = G == 4 ? j >> 1 : j & 1;
  const int HK = a.heads, HQ = HK * G, PS = a.partition_size;
  const int wph = Cfg::WARPS / heads_per_item;  // warps that share a KV head
  const int part = warp % wph;

  if (a.after_plan) grid_dependency_wait();
  int32_t next = -1;  // thread 0: the next item, once reserved
  if (threadIdx.x == 0) {
    for (int i = 0; i < Cfg::WARPS * NSTAGE; ++i) mbar_init(smem_addr(&bars[i]), 1);
    mbar_init_fence();
    s_abort = 0;
    s_plan_ok = plan_header_ok(a);  // see the MHA kernel
    if (s_plan_ok) next = atomicAdd(&a.plan->work_counter, 1);
    else atomicOr(a.err, PA_DEVERR_PLAN);
  }
  __syncthreads();
  if (!s_plan_ok) return;
  const int32_t num_items = a.plan->num_items;

  uint32_t fills = 0;
  uint8_t* my_stages = q4_smem + warp * NSTAGE * Cfg::STAGE_BYTES;
  uint64_t* my_bars = bars + warp * NSTAGE;

  for (;;) {
    if (threadIdx.x == 0) {
      s_item = next >= 0 ? next : atomicAdd(&a.plan->work_counter, 1);
      next = -1;
    }
    __syncthreads();
    const int item = s_item;
    if (item >= num_items || s_abort) break;
    PlanItem it;
    if (!plan_item(a, item, &it)) {  // a damaged plan entry: report and skip the item
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
      tbl[i] = b;
    }
    __syncthreads();

    const int kvh = g * heads_per_item + warp / wph;
    const bool mine = kvh < HK;
    const int64_t sh0 = (int64_t)s * HQ + kvh * G;
    // the chunks of the partition that this warp takes
    const int chunks = (nblk + CB - 1) / CB;
    const int c_lo = chunks * part / wph, c_n = chunks * (part + 1) / wph - c_lo;

    // of query heads head0 + e; l_run is over this lane's tokens
    float m[NH], l_run[NH];
    float f[FG][NH];
#pragma unroll
    for (int e = 0; e < NH; ++e) {
      m[e] = -INFINITY, l_run[e] = 0.f;
#pragma unroll
      for (int gr = 0; gr < FG; ++gr) f[gr][e] = __uint_as_float((uint32_t)kFactorTop << 23);
    }
    float o[PIECES][2][4];
#pragma unroll
    for (int c = 0; c < PIECES; ++c)
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[c][m][e] = 0.f;

    bool ok = true;
    if (mine) {
      const uint8_t* kbase = static_cast<const uint8_t*>(a.k_pool) + (int64_t)kvh * TILE;
      const uint8_t* vbase = static_cast<const uint8_t*>(a.v_pool) + (int64_t)kvh * TILE;
      const int64_t block_bytes = (int64_t)HK * TILE;
      // fill k with chunk c: lanes 0 .. 7 copy the K and V tiles of its blocks
      auto issue = [&](uint32_t k, int c) {
        const int st = k % NSTAGE;
        const uint32_t bar = smem_addr(&my_bars[st]);
        const int nb = min(CB, nblk - c * CB);
        __syncwarp();  // every lane is done with the stage
        if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)(nb * 2 * TILE));
        __syncwarp();
        if (lane < 2 * nb) {
          fence_proxy_async_shared();
          const int b = lane >> 1;
          const int64_t off = (int64_t)tbl[c * CB + b] * block_bytes;
          const uint32_t dst = smem_addr(my_stages + st * Cfg::STAGE_BYTES) + (lane & 1) * Cfg::HALF + b * TILE;
          bulk_copy_g2s(dst, ((lane & 1) ? vbase : kbase) + off, TILE, bar);
        }
      };
      const uint32_t k0 = fills;
      for (int i = 0; i < NSTAGE && i < c_n; ++i) issue(k0 + i, c_lo + i);

      // Q fragments, column r, dimensions 32 c + 8 j .. + 7: head r % G (I8: digit r / 2 of head r % 2, zero past G)
      uint32_t qb[PIECES][I8 ? 2 : 4];
      float2 kq[NH];         // scores to log2 units, in two factors (I8: of this lane's digit)
      float qs[GROUPS][NH];  // I8: sum of a group's queries in this lane's digit
      {
        const int q_head = I8 ? (r & 1) : r & (G - 1);
        float qf[PIECES][8], top = 0.f;
#pragma unroll
        for (int c = 0; c < PIECES; ++c) {
          if (q_head < G) {
            load8(static_cast<const T*>(a.q) + (sh0 + q_head) * D + 32 * c + 8 * j, qf[c]);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) qf[c][e] = 0.f;
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(qf[c][e]));
        }
        top = fmaxf(top, __shfl_xor_sync(kFullMask, top, 1));
        top = fmaxf(top, __shfl_xor_sync(kFullMask, top, 2));
        const int ex = (int)(__float_as_uint(top) >> 23);  // biased exponent; 255: infinity or NaN
        if constexpr (I8) {
          // as whole numbers, the row's largest in [2^21, 2^22), of three signed base-256 digits; column r
          // is digit r / 2, the leading one first, of head r % 2
          const int term = r >> 1;
          const int qe = ex == 255 ? 0 : 21 + 127 - ex;
          const float fa = pow2(qe >> 1), fb = pow2(qe - (qe >> 1));  // 2^qe
          float probe = 0.f;  // NaN once a query is NaN or infinite
          auto digit = [&](float x, int* sum) {
            probe = fmaf(x, 0.f, probe);
            const int v = __float2int_rn(x * fa * fb);
            const int d0 = (int)(int8_t)v, v1 = (v - d0) >> 8;
            const int d1 = (int)(int8_t)v1, d2 = (v1 - d1) >> 8;
            const int d = term == 0 ? d2 : term == 1 ? d1 : term == 2 ? d0 : 0;
            *sum += d;
            return (uint32_t)d & 0xffu;
          };
#pragma unroll
          for (int gr = 0; gr < GROUPS; ++gr) {
            int sum = 0;
#pragma unroll
            for (int c = 2 * gr; c < 2 * gr + 2; ++c) {
              qb[c][0] = qb[c][1] = 0u;
#pragma unroll
              for (int e = 0; e < 8; ++e)  // as the numbers lie in a register: the even ones, then the odd ones
                qb[c][e & 1] |= digit(qf[c][e], &sum) << (8 * (e / 2));
            }
            sum += __shfl_xor_sync(kFullMask, sum, 1);
            sum += __shfl_xor_sync(kFullMask, sum, 2);
#pragma unroll
            for (int e = 0; e < NH; ++e) qs[gr][e] = (float)__shfl_sync(kFullMask, sum, 4 * (2 * j + e));
          }
          probe += __shfl_xor_sync(kFullMask, probe, 1);
          probe += __shfl_xor_sync(kFullMask, probe, 2);
#pragma unroll
          for (int e = 0; e < NH; ++e)  // 2^(16 - 8 j): the digit's weight
            kq[e] = split_factor(a.scale_log2 + __shfl_sync(kFullMask, probe, 4 * e),
                                 16 - 8 * j - __shfl_sync(kFullMask, qe, 4 * e));
        } else {
          // scaled by 2^qe so that the row's largest value lies in [2^14, 2^15)
          const int qe = ex == 255 ? 0 : 14 + 127 - ex;
          const float fa = pow2(qe >> 1), fb = pow2(qe - (qe >> 1));
#pragma unroll
          for (int e = 0; e < NH; ++e)
            kq[e] = split_factor(a.scale_log2, 10 - __shfl_sync(kFullMask, qe, 8 * j + 4 * e));
#pragma unroll
          for (int c = 0; c < PIECES; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e)  // pairs as the nibbles lie in a register: (0, 4), (1, 5), ...
              qb[c][e] = pack_half(qf[c][e] * fa * fb, qf[c][e + 4] * fa * fb);
        }
      }

      bool second = false;  // a second factor is not 1
#pragma unroll
      for (int e = 0; e < NH; ++e) second |= kq[e].y != 1.f;
      second = __any_sync(kFullMask, second);

      int i = 0;
      for (; i < c_n; ++i) {
        const uint32_t k = k0 + i;
        const int st = k % NSTAGE;
        if (!__all_sync(kFullMask, mbar_wait_bounded(smem_addr(&my_bars[st]), (k / NSTAGE) & 1u))) {
          ok = false;
          break;
        }
        uint8_t* kt = my_stages + st * Cfg::STAGE_BYTES;
        uint8_t* vt = kt + Cfg::HALF;
        const int valid = min(kQ4Chunk, ntok - (c_lo + i) * kQ4Chunk);
        if (valid < kQ4Chunk) {
          // slots past the context hold anything: their V words become zero
          // (scale and zero point), so that they add nothing; their scores
          // are masked below
          for (int t = valid + lane; t < kQ4Chunk; t += 32)
#pragma unroll
            for (int gr = 0; gr < GROUPS; ++gr)
              *reinterpret_cast<uint32_t*>(vt + (t >> 4) * TILE + q4_words_off(D) + (gr * 16 + (t & 15)) * 4) = 0u;
          __syncwarp();
        }

        // ---- scores of the chunk in log2 units: x[b][nt][e] of token 16 b + 8 nt + r, head head0 + e
        float x[CB][2][NH];
#pragma unroll
        for (int b = 0; b < CB; ++b) {
          const uint32_t tile = smem_addr(kt + b * TILE);
          uint32_t kw[2][PIECES];
          if constexpr (D == 128) {
            const uint32_t at = tile + (lane >> 3) * 256 + (lane & 7) * 16;
            ldmatrix_x4(kw[0], at);
            ldmatrix_x4(kw[1], at + 128);
          } else {
            uint32_t w[4];
            ldmatrix_x4(w, tile + ((lane >> 3) & 1) * 256 + (lane >> 4) * 128 + (lane & 7) * 16);
            kw[0][0] = w[0], kw[0][1] = w[1], kw[1][0] = w[2], kw[1][1] = w[3];
          }
          const uint8_t* words = kt + b * TILE + q4_words_off(D) + r * 4;
          if constexpr (I8) {
#pragma unroll
            for (int gr = 0; gr < GROUPS; ++gr) {
              int c[4] = {0, 0, 0, 0};
#pragma unroll
              for (int pc = 2 * gr; pc < 2 * gr + 2; ++pc) {
                const uint32_t w0 = kw[0][pc], w1 = kw[1][pc];
                const uint32_t am[4] = {w0 & kNibbles, w1 & kNibbles, (w0 >> 4) & kNibbles, (w1 >> 4) & kNibbles};
                mma16832_u8s8(c, am, qb[pc][0], qb[pc][1]);
              }
              uint32_t word[2];
#pragma unroll
              for (int nt = 0; nt < 2; ++nt) word[nt] = *reinterpret_cast<const uint32_t*>(words + gr * 64 + nt * 32);
#pragma unroll
              for (int e = 0; e < NH; ++e) {
                const float2 d = mul2(make_float2(fmaf(-q4_zero(word[0]), qs[gr][e], (float)c[e]),
                                                  fmaf(-q4_zero(word[1]), qs[gr][e], (float)c[2 + e])),
                                      make_float2(kq[e].x, kq[e].x));
                x[b][0][e] = gr == 0 ? q4_scale(word[0]) * d.x : fmaf(q4_scale(word[0]), d.x, x[b][0][e]);
                x[b][1][e] = gr == 0 ? q4_scale(word[1]) * d.y : fmaf(q4_scale(word[1]), d.y, x[b][1][e]);
              }
            }
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
              for (int e = 0; e < NH; ++e) {  // the digits, over the quad's lanes
                float v = x[b][nt][e];
                if (second) v *= kq[e].y;
                v += __shfl_xor_sync(kFullMask, v, 1);
                v += __shfl_xor_sync(kFullMask, v, 2);
                x[b][nt][e] = v;
              }
          } else {
#pragma unroll
            for (int gr = 0; gr < GROUPS; ++gr) {
              uint32_t word[2];
              __half2 nz[2];  // -z 2^-10 of the two tokens, in both halves
#pragma unroll
              for (int nt = 0; nt < 2; ++nt) {
                word[nt] = *reinterpret_cast<const uint32_t*>(words + gr * 64 + nt * 32);
                nz[nt] = __hmul2(as_half2(__byte_perm(word[nt], word[nt], 0x1010)), as_half2(kMinus2m10));
              }
              float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int pc = 2 * gr; pc < 2 * gr + 2; ++pc) {
                const uint32_t w0 = kw[0][pc], w1 = kw[1][pc], u0 = w0 >> 8, u1 = w1 >> 8;
                const uint32_t a0[4] = {q4_even(w0, nz[0]), q4_even(w1, nz[1]), q4_odd(w0, nz[0]), q4_odd(w1, nz[1])};
                const uint32_t a1[4] = {q4_even(u0, nz[0]), q4_even(u1, nz[1]), q4_odd(u0, nz[0]), q4_odd(u1, nz[1])};
                mma16816<__half>(c, a0, qb[pc][0], qb[pc][1]);
                mma16816<__half>(c, a1, qb[pc][2], qb[pc][3]);
              }
#pragma unroll
              for (int nt = 0; nt < 2; ++nt) {
                const float sc = q4_scale(word[nt]);
                const float2 d = mul2(make_float2(c[2 * nt], c[2 * nt + 1]), make_float2(kq[0].x, kq[NH - 1].x));
                x[b][nt][0] = gr == 0 ? sc * d.x : fmaf(sc, d.x, x[b][nt][0]);
                x[b][nt][NH - 1] = gr == 0 ? sc * d.y : fmaf(sc, d.y, x[b][nt][NH - 1]);
              }
            }
            if (second) {
#pragma unroll
              for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int e = 0; e < NH; ++e) x[b][nt][e] *= kq[e].y;
            }
          }
        }
        if (valid < kQ4Chunk) {
#pragma unroll
          for (int b = 0; b < CB; ++b)
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
              if (b * 16 + nt * 8 + r >= valid) {
#pragma unroll
                for (int e = 0; e < NH; ++e) x[b][nt][e] = -INFINITY;
              }
        }
        if constexpr (MASS) {
#pragma unroll
          for (int e = 0; e < NH; ++e) {
            float* dst = a.scores + (sh0 + head0 + e) * a.score_stride + tok0 + (c_lo + i) * kQ4Chunk + r;
#pragma unroll
            for (int b = 0; b < CB; ++b)
#pragma unroll
              for (int nt = 0; nt < 2; ++nt)  // lanes that hold the same heads store a block each in turn
                if ((I8 ? (b & 3) == j : G == 8 || (b & 1) == j >> 1) && b * 16 + nt * 8 + r < valid)
                  dst[b * 16 + nt * 8] = x[b][nt][e];
          }
        }

        // ---- softmax: the chunk's maxima, and the weights in the scores' place
        float mx[NH], down[NH];  // down: what m moves the accumulators by, in log2
#pragma unroll
        for (int e = 0; e < NH; ++e) {
          mx[e] = -INFINITY;
#pragma unroll
          for (int b = 0; b < CB; ++b) mx[e] = fmaxf(mx[e], fmaxf(x[b][0][e], x[b][1][e]));
#pragma unroll
          for (int k = 4; k < 32; k <<= 1) mx[e] = fmaxf(mx[e], __shfl_xor_sync(kFullMask, mx[e], k));
          down[e] = 0.f;
          if (mx[e] - m[e] > kMove) {  // by the difference: beyond 2^24 the sum would be rounded
            down[e] = m[e] - mx[e];  // -infinity on the first move
            m[e] = mx[e];
            l_run[e] *= ex2(down[e]);
          }
          const float mb = m[e] == -INFINITY ? 0.f : -m[e];
#pragma unroll
          for (int b = 0; b < CB; ++b)
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
              x[b][nt][e] = ex2(x[b][nt][e] + mb);
              l_run[e] += x[b][nt][e];
            }
        }

        // ---- P's factors
        uint32_t big = 0u;
        constexpr int WPB = 4 * GROUPS;  // 16-byte loads that hold a block's words
        if (lane < CB * WPB) {
          const uint4 w = *reinterpret_cast<const uint4*>(vt + (lane / WPB) * TILE + q4_words_off(D) +
                                                          (lane % WPB) * 16);
          const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (ws[e] < 0x7f800000u) big = max(big, ws[e]);  // NaN scales do not count
        }
        big = __reduce_max_sync(kFullMask, big);  // as a float, the largest scale and a little more
        bool move = false;
#pragma unroll
        for (int e = 0; e < NH; ++e) {
          const float bound = __uint_as_float(big) * ex2(mx[e] - m[e]);
          move |= down[e] < 0.f;
#pragma unroll
          for (int gr = 0; gr < FG; ++gr) move |= bound * f[gr][e] > kPMove;
        }
        if (__any_sync(kFullMask, move)) {
#pragma unroll
          for (int gr = 0; gr < FG; ++gr) {
            float top[NH], alpha[2] = {1.f, 1.f};  // top: the group's largest w s
#pragma unroll
            for (int e = 0; e < NH; ++e) top[e] = 0.f;
#pragma unroll
            for (int b = 0; b < CB; ++b)
#pragma unroll
              for (int nt = 0; nt < 2; ++nt) {
                const float sc = q4_scale(*reinterpret_cast<const uint32_t*>(
                    vt + b * TILE + q4_words_off(D) + (GROUP_COLS ? my_group : gr) * 64 + nt * 32 + r * 4));
#pragma unroll
                for (int e = 0; e < NH; ++e) top[e] = fmaxf(top[e], x[b][nt][e] * sc);  // NaN does not count
              }
#pragma unroll
            for (int e = 0; e < NH; ++e) {
#pragma unroll
              for (int k = 4; k < 32; k <<= 1) top[e] = fmaxf(top[e], __shfl_xor_sync(kFullMask, top[e], k));
              const int was = (int)(__float_as_uint(f[gr][e]) >> 23), ex = (int)(__float_as_uint(top[e]) >> 23);
              int fe = was;
              if (down[e] < 0.f) fe = min(kFactorTop, fe + (int)fminf(-down[e], 512.f));  // rises as m does
              if (top[e] * __uint_as_float((uint32_t)fe << 23) > kPMove) fe = kFactorPut - ex;
              alpha[e] = ex2(down[e] + (float)(fe - was));  // 0 on the first move
              f[gr][e] = __uint_as_float((uint32_t)fe << 23);
            }
#pragma unroll
            for (int c = gr * (PIECES / FG); c < (gr + 1) * (PIECES / FG); ++c)
#pragma unroll
              for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[c][h][e] *= alpha[NH == 2 ? e & 1 : 0];
          }
        }

        // ---- values
#pragma unroll
        for (int b = 0; b < CB; ++b) {
          const uint32_t tile = smem_addr(vt + b * TILE);
          const uint8_t* words = vt + b * TILE + q4_words_off(D);
          uint32_t pb[2], pr[2];  // P, and what its rounding left unless that has columns of its own
          auto weights = [&](int gr) {
            const int fg = FG == 1 ? 0 : gr;
            float sc[2];
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
              sc[nt] = q4_scale(*reinterpret_cast<const uint32_t*>(words + gr * 64 + nt * 32 + r * 4));
            // pairs of two heads, or of a head's two tokens
#pragma unroll
            for (int q = 0; q < NH; ++q) {
              const float2 w = NH == 2 ? make_float2(x[b][q][0], x[b][q][NH - 1]) : make_float2(x[b][0][0], x[b][1][0]);
              const float2 p = mul2(mul2(w, make_float2(sc[q], NH == 2 ? sc[q] : sc[1])), make_float2(f[fg][0], f[fg][NH - 1]));
              const uint32_t hi = pack_half(p.x, p.y);
              const float2 rest = sub_half2(p, hi, REST_COLS && j < 2 ? 0.f : 1.f);
              if constexpr (NH == 1) {
                pb[0] = movmatrix(pack_half(rest.x, 0.f));
                pb[1] = movmatrix(pack_half(rest.y, 0.f));
              } else {
                const uint32_t part = pack_half(rest.x, rest.y);
                pb[q] = movmatrix(REST_COLS ? part : hi);
                if (!REST_COLS) pr[q] = movmatrix(part);
              }
            }
          };
          if (FG == 1) weights(GROUP_COLS ? my_group : 0);
#pragma unroll
          for (int gr = 0; gr < GROUPS; ++gr) {
            if (FG == 2) weights(gr);
            __half2 nz[2];  // -z 2^-10 of tokens 2 j and 2 j + 1
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
              const uint2 two = *reinterpret_cast<const uint2*>(words + gr * 64 + nt * 32 + j * 8);
              nz[nt] = __hmul2(as_half2(__byte_perm(two.x, two.y, 0x5410)), as_half2(kMinus2m10));
            }
            uint32_t v[4];
            ldmatrix_x4_trans(v, tile + (2 * gr + (lane >> 4)) * 256 + ((lane >> 3) & 1) * 128 + (lane & 7) * 16);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t v0 = v[2 * h], v1 = v[2 * h + 1], u0 = v0 >> 8, u1 = v1 >> 8;
              const uint32_t a0[4] = {q4_even(v0, nz[0]), q4_odd(v0, nz[0]), q4_even(v1, nz[1]), q4_odd(v1, nz[1])};
              const uint32_t a1[4] = {q4_even(u0, nz[0]), q4_odd(u0, nz[0]), q4_even(u1, nz[1]), q4_odd(u1, nz[1])};
              mma16816<__half>(o[2 * gr + h][0], a0, pb[0], pb[1]);
              mma16816<__half>(o[2 * gr + h][1], a1, pb[0], pb[1]);
              if constexpr (!REST_COLS) {
                mma16816<__half>(o[2 * gr + h][0], a0, pr[0], pr[1]);
                mma16816<__half>(o[2 * gr + h][1], a1, pr[0], pr[1]);
              }
            }
          }
        }
        if (i + NSTAGE < c_n) issue(k + NSTAGE, c_lo + i + NSTAGE);
        // as in the MHA kernel: the next item is reserved shortly before this one ends
        if (threadIdx.x == 0 && i == max(c_n - 2, 0)) next = atomicAdd(&a.plan->work_counter, 1);
      }
      if (!ok) {
        if (lane == 0) {  // as in the MHA kernel: report, stop, and poison the plan
          atomicOr(a.err, PA_DEVERR_TIMEOUT);
          s_abort = 1;
          a.plan->poisoned = 1;
          __threadfence();
        }
        const int issued = min(c_n, i + NSTAGE);
        for (int jj = i; jj < issued; ++jj) {
          const uint32_t k = k0 + jj;
          mbar_wait_bounded(smem_addr(&my_bars[k % NSTAGE]), (k / NSTAGE) & 1u);
        }
      } else {
        fills = k0 + c_n;
      }
#pragma unroll
      for (int e = 0; e < NH; ++e)
#pragma unroll
        for (int k = 4; k < 32; k <<= 1) l_run[e] += __shfl_xor_sync(kFullMask, l_run[e], k);
      if (wph > 1 && part > 0) {  // for the first warp of the head (this warp's stages are drained)
        float* xs = reinterpret_cast<float*>(my_stages);
#pragma unroll
        for (int c = 0; c < PIECES; ++c)
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) xs[((c * 2 + m) * 4 + e) * 32 + lane] = o[c][m][e];
#pragma unroll
        for (int e = 0; e < NH; ++e) {
          xs[(PIECES * 8 + 2 * e) * 32 + lane] = m[e];
          xs[(PIECES * 8 + 2 * e + 1) * 32 + lane] = l_run[e];
#pragma unroll
          for (int gr = 0; gr < FG; ++gr)
            xs[(PIECES * 8 + 2 * NH + gr * NH + e) * 32 + lane] = f[gr][e];
        }
        fence_proxy_async_shared();  // before the ring's next bulk copies into the same bytes
      }
    }
    if (wph > 1) __syncthreads();
    if (mine && part == 0 && (wph > 1 ? !s_abort : ok)) {
      for (int other = 1; other < wph; ++other) {  // fold in the other warps' states
        const float* xs = reinterpret_cast<const float*>(my_stages + other * NSTAGE * Cfg::STAGE_BYTES);
        float sa[FG][2] = {}, sb[FG][2] = {};  // rescales of the accumulators
#pragma unroll
        for (int e = 0; e < NH; ++e) {
          const float mb = xs[(PIECES * 8 + 2 * e) * 32 + lane], lb = xs[(PIECES * 8 + 2 * e + 1) * 32 + lane];
          const float M = fmaxf(m[e], mb);
          l_run[e] = (m[e] == -INFINITY ? 0.f : l_run[e] * exp2f(m[e] - M)) + (mb == -INFINITY ? 0.f : lb * exp2f(mb - M));
#pragma unroll
          for (int gr = 0; gr < FG; ++gr) {
            // either factor, risen as M lies above its reference; the smaller one serves both
            const float other = xs[(PIECES * 8 + 2 * NH + gr * NH + e) * 32 + lane];
            const int fa = (int)(__float_as_uint(f[gr][e]) >> 23), fb = (int)(__float_as_uint(other) >> 23);
            const int both = min(kFactorTop, min(fa + (int)fminf(M - m[e], 512.f), fb + (int)fminf(M - mb, 512.f)));
            sa[gr][e] = m[e] == -INFINITY ? 0.f : exp2f(m[e] - M + (float)(both - fa));
            sb[gr][e] = mb == -INFINITY ? 0.f : exp2f(mb - M + (float)(both - fb));
            f[gr][e] = __uint_as_float((uint32_t)both << 23);
          }
          m[e] = M;
        }
#pragma unroll
        for (int c = 0; c < PIECES; ++c)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int gr = c / (PIECES / FG), head = NH == 2 ? e & 1 : 0;
              o[c][h][e] = o[c][h][e] * sa[gr][head] + xs[((c * 2 + h) * 4 + e) * 32 + lane] * sb[gr][head];
            }
      }
      if (wph > 1) fence_proxy_async_shared();  // the other warps' rings are refilled after the loop's barrier
      // The accumulators hold 2^(k - 10) of their sums.  Partial results are the sums over (1 to 2) 2^12 of l, with
      // m raised by as much: whatever the values, thousands of them add up in fp32, and small ones stay.
      float inv[NH];
      float2 ml[NH];
#pragma unroll
      for (int e = 0; e < NH; ++e) {
        const int up = (int)(__float_as_uint(l_run[e]) >> 23) - 127 + 12;
        const float by = __uint_as_float((uint32_t)(127 - up) << 23);
        inv[e] = split ? 1024.f * by : m[e] != -INFINITY ? 1024.f / l_run[e] : 0.f;
        ml[e] = make_float2(m[e] + (float)up, l_run[e] * by);
      }
      // 2^-k
      auto back = [&](int gr, int e) { return __uint_as_float((254u << 23) - __float_as_uint(f[FG == 1 ? 0 : gr][e])); };
      // Of a head, this lane writes the pieces from `first` on, dimensions 32 c + 4 r .. + 3 of each.  With REST_COLS
      // lanes 0 and 1 hold the sums of P, 2 and 3 those of what its rounding left: a lane gives the one that holds
      // the other part its share of that one's piece.
      constexpr int WRITES = REST_COLS ? 1 : GROUP_COLS ? 2 : PIECES;
      const int first = REST_COLS ? (GROUP_COLS ? 2 * my_group : 0) + (j >> 1) : GROUP_COLS ? 2 * my_group : 0;
      const bool writes = !(I8 && GROUPS == 1) || (j & 1) == 0;  // two lanes hold the same there
#pragma unroll
      for (int e = 0; e < NH; ++e) {
#pragma unroll
        for (int q = 0; q < WRITES; ++q) {
          float v[4], give[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int h = k >> 1, n = 2 * (k & 1) + e;
            if constexpr (REST_COLS) {
#pragma unroll
              for (int c = 0; c < PIECES; ++c) {
                if (c == first) v[k] = o[c][h][n];
                if (c == (first ^ 1)) give[k] = o[c][h][n];
              }
              v[k] += __shfl_xor_sync(kFullMask, give[k], 2);
            } else {
              v[k] = GROUP_COLS && my_group ? o[(2 + q) % PIECES][h][n] : o[q][h][n];
            }
            v[k] = v[k] * inv[e] * back(q / 2, e);
          }
          if (!writes) continue;
          const int64_t at = sh0 + head0 + e;
          const int d = 32 * (first + q) + 4 * r;
          if (!split)
            *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + at * D + d) =
                make_uint2(MmaType<T>::pack(v[0], v[1]), MmaType<T>::pack(v[2], v[3]));
          else
            *reinterpret_cast<float4*>(a.part_acc + (at * a.max_parts + p) * D + d) = make_float4(v[0], v[1], v[2], v[3]);
        }
        if (r == 0 && j < (G + 1) / 2) {
          if (split) a.part_ml[(sh0 + head0 + e) * a.max_parts + p] = ml[e];
          else if (MASS) a.lse[sh0 + head0 + e] = m[e] + log2f(l_run[e]);
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
        s_merge = arrived == ni && !s_abort && *(volatile int32_t*)&a.plan->poisoned == 0;
        if (arrived == ni) *cnt = 0;
      }
      __syncthreads();
      if (s_merge && mine && part == 0) {
        __threadfence();
        // rounds of at most 8 partitions of every head (each keeps its weights in registers)
        constexpr int RING = NSTAGE * Cfg::STAGE_BYTES, ROUND = 8 * D * 4;
        bool merged = true;
        if constexpr (G == 1) {
          const int used = merge_staged<T, D, NSTAGE, RING, MASS>(a, sh0, np, lane, my_stages, my_bars, fills);
          fills += used > 0 ? used : -used;
          merged = used > 0;
        } else {
          merged = merge_group<T, D, G, NSTAGE, G * ROUND < RING ? G * ROUND : RING, MASS>(a, sh0, np, lane, my_stages,
                                                                                          my_bars, fills);
        }
        if (!merged && lane == 0) {  // as for a copy of the item: report, stop, poison the plan
          atomicOr(a.err, PA_DEVERR_TIMEOUT);
          s_abort = 1;
          a.plan->poisoned = 1;
          __threadfence();
        }
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
