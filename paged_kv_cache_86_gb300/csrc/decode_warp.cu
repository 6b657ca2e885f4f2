// decode_warp.cu -- decode attention in which every warp walks keys of its own:
// over an fp8 E4M3 cache with one scale per (block, KV head), and over the bf16
// cache, both with an optional sliding window behind a few first tokens that stay
// visible (pkv_paged_decode_fp8_block, pkv_paged_decode_window).
//
//   out[i, g] = sum_p softmax_p(scale q[i, g] . K_i[p]) V_i[p] over the seen p:
//   all p < ctx, or with a window of w and s sinks p < s and p >= ctx - w.
//
// The work is HBM-bound: a key and a value of one KV head are 256 bytes (fp8)
// and feed the `group` query heads that share them, 4 * 128 * group operations.
// The tensor core is needed only because the CUDA cores would not keep up with
// group * 2 operations a byte; its rate is not what counts. What counts is that
// no warp waits for another one: decode_tcg.cu feeds the tensor core tiles of all
// KV heads, and its softmax warps meet once a tile; here a warp owns 16 tokens of
// one KV head at a time and the mma.m16n8k16 that work on them,
//   S^T [16 tokens x 8 heads] = K [16 x 128] Q^T      8 MMAs
//   O^T [128 dims x 8 heads] += V^T [128 x 16] P^T    8 MMAs, P^T from S^T by
//                                                     two 8x8 transposes
// and nothing is exchanged before the end of its keys. Codes become f16 (exact) two
// at a time; scales are applied to the scores and to the weights.
//
// The keys come to the warps in one of two ways. Block sizes that 8 divides: a
// producer warp copies tiles of all KV heads, which are contiguous in the cache, by
// TMA into a ring that fills the SM's shared memory (decode_ring_kernel). Others:
// every warp loads its rows straight into the registers that the MMAs take them
// from (decode_direct_kernel). Its pieces of 128 or 256 bytes, read at eight different
// times, DRAM served at 0.45 of its rate; asked for in L2 together, a tile ahead, at
// 0.6 to 0.7. 512 sequences (fp8, 0.59 M tokens): 202 us at block 16, 311 at block 6;
// behind a window of 1024 (bf16) 242-246 and 338. At 0.91 and 0.98 of the copy rate, merge
// included, the rings are bound by HBM; 3 sequences take 13 us, two launches of
// dependent loads, and 17 with direct loads.
//
// Split: the seen tokens of all sequences, in tiles of 16 with kSegTiles of
// overhead in front of each sequence, are one line that is cut into equal ranges;
// a ring (a direct warp) takes one range. A sequence that a cut goes through leaves
// (m, l, O) records that a second launch merges.
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <mutex>

#include "cut_entries.h"
#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "pkv_tc.cuh"

namespace pkv {
namespace {

constexpr int kHD = 128;
constexpr int kTok = 16;                   // tokens of a tile
constexpr int kSegTiles = 2;               // what starting a sequence costs, in tiles
constexpr int kMinTiles = 4;               // shortest range
constexpr int kDirectWarps = 8;            // warps of a CTA, direct loads
// Warps of a CTA with rings, producers included, and so the registers of a thread
// (168). With 18 (96 registers, spills; two rings for 8 KV heads instead of one) 512
// sequences took 263 us (fp8) and 274 us (bf16, window of 1024), with 12 220 and 268.
constexpr int kRingWarps = 12;
constexpr int kCombineWarps = 8;
constexpr int kRingBytes = 220 * 1024;     // of all stages of a CTA
constexpr int kMaxStages = 16;             // of one ring
constexpr float kLog2e = 1.4426950408889634f;
// A reference maximum is kept until a score exceeds it by this (log2): weights
// stay below 2^kGrow (bf16: exact range) and f16 weights, which are also scaled
// by 2^kLift, between 2^-24 and 2^15.
constexpr float kGrow = 8.f;
constexpr float kLift = 7.f;
constexpr float kDrop = 1.f / 128.f;       // 2^-kLift

// n / d for 0 <= n < 2^31 by a multiplication (Granlund and Montgomery, "Division by
// Invariant Integers using Multiplication")
struct FastDiv {
  uint32_t mul, shift, d;
};

struct WarpParams {
  __nv_bfloat16 *out;
  const __nv_bfloat16 *q;
  const uint8_t *k_cache;
  const uint8_t *v_cache;
  const float *k_scales;
  const float *v_scales;
  const int32_t *block_tables;
  const int32_t *context_lens;
  int max_blocks_per_seq;
  int num_seqs;
  int max_context_len;
  int num_q_heads;
  int num_kv_heads;
  int group;
  int chunks;          // warps' head chunks of a KV head
  int per_chunk;       // query heads of a chunk
  int num_blocks;
  FastDiv bs;
  int window;          // 0: none
  int sinks;
  float scale_log2;
  int ranges;          // most ranges the line is cut into
  // shared-memory rings (decode_ring_kernel)
  int unit;            // tokens of a box: 16 or 8
  int heads_per_cta;   // KV heads of a box
  int head_groups;     // boxes over all KV heads
  int rings;           // of a CTA
  int stages;          // of a ring
  // What the second launch merges, an entry (sequence, its first and its last range;
  // sequence -1 or one range: nothing) for each of whichever are fewer: the sequences,
  // or the ranges, which have the sequence that they begin inside of if they are the
  // second of its ranges.
  int4 *cuts;
  bool cuts_by_seq;
  float4 *ml;          // records: (m, l, M)
  float *po;           // and O
  uint32_t *err;
};

__device__ __forceinline__ uint32_t div_of(uint32_t n, const FastDiv &f) {
  return f.d == 1 ? n : __umulhi(n, f.mul) >> f.shift;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// With results below 2^-126: the values' scales go down to 2^-120, and a kept maximum
// may be off by 2^8.
__device__ __forceinline__ float ex2_far(float x) {
  float y;
  asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 16 bytes that are used once: past L1
__device__ __forceinline__ uint4 ld_once(const uint8_t *p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
  return h;
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

template <bool kFp8>
__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                      uint32_t b0, uint32_t b1) {
  if constexpr (kFp8)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The operands of the two products, as a lane of mma.m16n8k16 holds them: fragment
// row (column of B) g = lane / 4, pair kp = lane % 4. The 128 dims of S's
// contraction may come in any order, and so may O's rows: a lane takes runs of
// neighbouring dims, so that it loads 16 bytes at a time.
//   K, Q: fp8 dims 32 kp + 0 .. 31; bf16 64 j + 16 kp + 0 .. 15, j = 0, 1
//   V, O: fp8 dims 16 g + 0 .. 15;  bf16 64 j + 8 g + 0 .. 7,   j = 0, 1
template <bool kFp8, int NT>
struct Heads {
  static constexpr int kKL = kFp8 ? 2 : 4;   // 16-byte loads of a lane's part of a K row
  static constexpr int kVL = kFp8 ? 1 : 2;   // and of a V row

  uint32_t qf[NT][8][2];            // Q^T: element (k, head g) of each of the 8 steps
  float qmul[NT][2];                // score factor of heads 2 kp, 2 kp + 1
  float o[NT][8][4];                // O^T
  // for heads 2 kp, 2 kp + 1: reference maxima of the scores and (fp8) of the scores
  // plus the log of the values' scale, and the lane's part of the sum of weights
  float m[NT][2], mw[NT][2], l[NT][2];

  // First dim of the lane's i-th 8 dims.
  static __device__ __forceinline__ int q_dim(int i, int kp) {
    return kFp8 ? 32 * kp + 8 * i : 64 * (i >> 1) + 16 * kp + 8 * (i & 1);
  }

  // The lane's parts of `heads` query rows, the first one at q.
  static __device__ __forceinline__ void load_q(const __nv_bfloat16 *q, int heads, uint4 (&raw)[NT][4]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, kp = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int h = nt * 8 + g;
        raw[nt][i] = h < heads ? __ldg(reinterpret_cast<const uint4 *>(q + h * kHD + q_dim(i, kp))) : make_uint4(0, 0, 0, 0);
      }
  }

  // A sequence begins, with what load_q has read.
  __device__ __forceinline__ void start(const uint4 (&raw)[NT][4], float scale_log2) {
    const int kp = threadIdx.x & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      uint32_t w[16];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[4 * i] = raw[nt][i].x;
        w[4 * i + 1] = raw[nt][i].y;
        w[4 * i + 2] = raw[nt][i].z;
        w[4 * i + 3] = raw[nt][i].w;
      }
      if constexpr (kFp8) {
        // f16 has three bits more than bf16 but a small range: the head's row is
        // scaled by a power of two to a maximum in [2^13, 2^14), exactly but for
        // entries under 2^-28 of it; rows that are not finite give NaN either way
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < 16; ++e) top = max(top, max(w[e] & 0x7fffu, (w[e] >> 16) & 0x7fffu));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = top >= 0x7f80u || top < 0x80u ? 0 : min(13 + 127 - static_cast<int>(top >> 7), 120);
        const float up = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float2 f = bf16x2_to_float2(w[i]);
          const __half2 hh = __floats2half2_rn(f.x * up, f.y * up);
          w[i] = *reinterpret_cast<const uint32_t *>(&hh);
        }
        const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        qmul[nt][0] = scale_log2 * __shfl_sync(0xffffffffu, down, 8 * kp);
        qmul[nt][1] = scale_log2 * __shfl_sync(0xffffffffu, down, 8 * kp + 4);
      } else {
        qmul[nt][0] = qmul[nt][1] = scale_log2;
      }
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        qf[nt][s][0] = w[2 * s];
        qf[nt][s][1] = w[2 * s + 1];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][i][e] = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[nt][e] = mw[nt][e] = -INFINITY;
        l[nt][e] = 0.f;
      }
    }
  }

  // S^T = K Q^T from the lane's parts of the K rows of tokens g and g + 8: s[0, 1] are
  // token g's scores of heads 2 kp, 2 kp + 1, s[2, 3] token g + 8's. Two chains of four
  // MMAs instead of one of eight.
  __device__ __forceinline__ void scores(const uint4 (&k)[2][kKL], float (&s)[NT][4]) const {
    float odd[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[nt][e] = odd[nt][e] = 0.f;
#pragma unroll
    for (int st = 0; st < 8; ++st) {
      uint32_t a[4];
      if constexpr (kFp8) {
        const uint32_t w0 = (&k[0][st >> 2].x)[st & 3], w1 = (&k[1][st >> 2].x)[st & 3];
        a[0] = e4m3x2_to_f16x2(static_cast<uint16_t>(w0));
        a[1] = e4m3x2_to_f16x2(static_cast<uint16_t>(w1));
        a[2] = e4m3x2_to_f16x2(static_cast<uint16_t>(w0 >> 16));
        a[3] = e4m3x2_to_f16x2(static_cast<uint16_t>(w1 >> 16));
      } else {
        a[0] = (&k[0][st >> 1].x)[2 * (st & 1)];
        a[1] = (&k[1][st >> 1].x)[2 * (st & 1)];
        a[2] = (&k[0][st >> 1].x)[2 * (st & 1) + 1];
        a[3] = (&k[1][st >> 1].x)[2 * (st & 1) + 1];
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        mma16<kFp8>(st & 1 ? odd[nt] : s[nt], a[0], a[1], a[2], a[3], qf[nt][st][0], qf[nt][st][1]);
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[nt][e] += odd[nt][e];
  }

  // The weights of the tile as B fragments of P^T. real, ks, vs: whether tokens g and
  // g + 8 count, their keys' scale and the log2 of their values' scale (fp8).
  __device__ __forceinline__ void weights(float (&s)[NT][4], bool real0, bool real1, float ks0, float ks1,
                                          float vs0, float vs1, uint32_t (&pb)[NT][2]) {
    bool grow = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        // (fp8: the factors first: a score of 2^130 that a scale of 2^-120 takes back must not
        // be infinite in between. Rounded to zero, their product is finite: 0 times it is 0.)
        float x = s[nt][e];
        x *= kFp8 ? __fmul_rz(qmul[nt][e & 1], e < 2 ? ks0 : ks1) : qmul[nt][e & 1];
        x = (e < 2 ? real0 : real1) ? x : -INFINITY;
        s[nt][e] = x;
        grow |= x > m[nt][e & 1] + kGrow;
        if constexpr (kFp8) grow |= x + (e < 2 ? vs0 : vs1) > mw[nt][e & 1] + kGrow;
      }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float top = fmaxf(s[nt][e], s[nt][e + 2]);
          float topw = kFp8 ? fmaxf(s[nt][e] + vs0, s[nt][e + 2] + vs1) : 0.f;
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) {
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
            if constexpr (kFp8) topw = fmaxf(topw, __shfl_xor_sync(0xffffffffu, topw, x));
          }
          top = fmaxf(top, m[nt][e]);
          const float f = top == -INFINITY ? 1.f : ex2(m[nt][e] - top);
          m[nt][e] = top;
          l[nt][e] *= f;
          float fo = f;
          if constexpr (kFp8) {
            topw = fmaxf(topw, mw[nt][e]);
            fo = topw == -INFINITY ? 1.f : ex2(mw[nt][e] - topw);
            mw[nt][e] = topw;
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            o[nt][i][e] *= fo;
            o[nt][i][e + 2] *= fo;
          }
        }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float ref = m[nt][e & 1] == -INFINITY ? 0.f : m[nt][e & 1];
        w[e] = ex2(s[nt][e] - ref);
        if constexpr (kFp8) {
          l[nt][e & 1] += w[e];
          const float refw = mw[nt][e & 1] == -INFINITY ? 0.f : mw[nt][e & 1];
          w[e] = ex2(s[nt][e] + (e < 2 ? vs0 : vs1) - (refw - kLift));
        }
      }
      uint32_t h0, h1;
      if constexpr (kFp8) {
        const __half2 x0 = __floats2half2_rn(w[0], w[1]), x1 = __floats2half2_rn(w[2], w[3]);
        h0 = *reinterpret_cast<const uint32_t *>(&x0);
        h1 = *reinterpret_cast<const uint32_t *>(&x1);
      } else {
        // the sum is of the rounded weights, so that the output stays a mean of V
        h0 = float2_to_bf16x2(w[0], w[1]);
        h1 = float2_to_bf16x2(w[2], w[3]);
        const float2 r0 = bf16x2_to_float2(h0), r1 = bf16x2_to_float2(h1);
        l[nt][0] += r0.x + r1.x;
        l[nt][1] += r0.y + r1.y;
      }
      pb[nt][0] = transpose8x8(h0);
      pb[nt][1] = transpose8x8(h1);
    }
  }

  // O^T += V^T P^T from the lane's parts of the V rows of tokens 2 kp, 2 kp + 1,
  // 2 kp + 8, 2 kp + 9. MMA i has the dims 2 i, 2 i + 1 of each lane's 16.
  __device__ __forceinline__ void accumulate(const uint4 (&v)[4][kVL], const uint32_t (&pb)[NT][2]) {
#pragma unroll
    for (int w = 0; w < (kFp8 ? 4 : 8); ++w) {
      const uint32_t x0 = (&v[0][w >> 2].x)[w & 3], x1 = (&v[1][w >> 2].x)[w & 3];
      const uint32_t x2 = (&v[2][w >> 2].x)[w & 3], x3 = (&v[3][w >> 2].x)[w & 3];
      if constexpr (kFp8) {
        // words of four dims: (token, next token) codes of a dim side by side
        const uint32_t p0 = __byte_perm(x0, x1, 0x5140), p1 = __byte_perm(x0, x1, 0x7362);
        const uint32_t p2 = __byte_perm(x2, x3, 0x5140), p3 = __byte_perm(x2, x3, 0x7362);
        const uint32_t a0 = e4m3x2_to_f16x2(static_cast<uint16_t>(p0));
        const uint32_t a1 = e4m3x2_to_f16x2(static_cast<uint16_t>(p0 >> 16));
        const uint32_t a2 = e4m3x2_to_f16x2(static_cast<uint16_t>(p2));
        const uint32_t a3 = e4m3x2_to_f16x2(static_cast<uint16_t>(p2 >> 16));
        const uint32_t b0 = e4m3x2_to_f16x2(static_cast<uint16_t>(p1));
        const uint32_t b1 = e4m3x2_to_f16x2(static_cast<uint16_t>(p1 >> 16));
        const uint32_t b2 = e4m3x2_to_f16x2(static_cast<uint16_t>(p3));
        const uint32_t b3 = e4m3x2_to_f16x2(static_cast<uint16_t>(p3 >> 16));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma16<kFp8>(o[nt][2 * w], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
          mma16<kFp8>(o[nt][2 * w + 1], b0, b1, b2, b3, pb[nt][0], pb[nt][1]);
        }
      } else {
        const uint32_t a0 = __byte_perm(x0, x1, 0x5410), a1 = __byte_perm(x0, x1, 0x7632);
        const uint32_t a2 = __byte_perm(x2, x3, 0x5410), a3 = __byte_perm(x2, x3, 0x7632);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma16<kFp8>(o[nt][w], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
      }
    }
  }

  // The sequence's output rows (whole), or records of this range's part of it.
  __device__ __forceinline__ void finish(bool whole, int heads, __nv_bfloat16 *out, float4 *ml, float *po) {
    const int lane = threadIdx.x & 31, g = lane >> 2, kp = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float sum = l[nt][e];
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
        const int h = nt * 8 + 2 * kp + e;
        if (h >= heads) continue;
        float v[16];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[2 * i] = o[nt][i][e];
          v[2 * i + 1] = o[nt][i][e + 2];
        }
        const int dim0 = kFp8 ? 16 * g : 8 * g, dim1 = kFp8 ? dim0 + 8 : dim0 + 64;
        if (whole) {
          float f = 1.f / sum, fw = 1.f;            // 0 / 0: every seen score is -inf
          if constexpr (kFp8) {
            f *= kDrop;
            fw = ex2_far(mw[nt][e] == -INFINITY ? 0.f : mw[nt][e] - m[nt][e]);
          }
          uint32_t w[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) w[i] = float2_to_bf16x2(v[2 * i] * f * fw, v[2 * i + 1] * f * fw);
          __nv_bfloat16 *dst = out + h * kHD;
          *reinterpret_cast<uint4 *>(dst + dim0) = make_uint4(w[0], w[1], w[2], w[3]);
          *reinterpret_cast<uint4 *>(dst + dim1) = make_uint4(w[4], w[5], w[6], w[7]);
        } else {
          float *dst = po + h * kHD;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            *reinterpret_cast<float4 *>(dst + dim0 + 4 * i) = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
            *reinterpret_cast<float4 *>(dst + dim1 + 4 * i) =
                make_float4(v[8 + 4 * i], v[9 + 4 * i], v[10 + 4 * i], v[11 + 4 * i]);
          }
          if (g == 0) ml[h] = make_float4(m[nt][e], sum, kFp8 ? mw[nt][e] : m[nt][e], 0.f);
        }
      }
  }
};

// What a sequence's query sees, as a walk of units of `unit` tokens (boxes; 1 for
// direct loads): the first `front` units and, `gap` units further on, the others.
// A unit may hold tokens that are not seen: p counts if p < ctx and (p < sinks or
// p >= first).
struct Seen {
  int ctx, first, units, front, gap;
};

__device__ __forceinline__ Seen seen_of(const WarpParams &p, int i, int unit, bool report) {
  int ctx = __ldg(p.context_lens + i);
  if (ctx < 0 || ctx > p.max_context_len) {
    if (report) raise_error(p.err, PKV_DEVERR_LENGTH);
    ctx = min(max(ctx, 0), p.max_context_len);
  }
  Seen s{ctx, 0, 0, 0, 0};
  if (p.window > 0) s.first = max(ctx - p.window, 0);
  const int shift = unit == 16 ? 4 : unit == 8 ? 3 : 0;
  const int lo = s.first >> shift;
  const int front = (min(p.sinks, ctx) + unit - 1) >> shift;
  if (lo > front) {
    s.front = front;
    s.gap = lo - front;
  }
  s.units = ((ctx + unit - 1) >> shift) - s.gap;
  return s;
}

__device__ __forceinline__ int tiles_of(const Seen &s, int unit) { return (s.units * unit + kTok - 1) / kTok; }
__device__ __forceinline__ int cost_of(const Seen &s, int unit) { return s.units > 0 ? tiles_of(s, unit) + kSegTiles : 0; }

struct Plan {
  int range_len, total;   // tiles of a range, of the line
};

// Where the CTA's ranges start on the line of all sequences: walker w of the CTA
// (w < walkers) takes range range_of(w); its first sequence goes to seq_of[w] (num_seqs:
// none) and that one's start on the line to pos_of[w]. The whole CTA calls it.

template <typename F>
__device__ __forceinline__ Plan plan_ranges(const WarpParams &p, int unit, int walkers, int *part, int *seq_of,
                                            int *pos_of, F range_of) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int threads = blockDim.x, warps = threads >> 5;
  const int per = (p.num_seqs + threads - 1) / threads;
  const int lo = min(tid * per, p.num_seqs), hi = min(lo + per, p.num_seqs);
  int mine = 0;
  for (int i = lo; i < hi; ++i) mine += cost_of(seen_of(p, i, unit, blockIdx.x == 0), unit);
  int inc = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, inc, off);
    if (lane >= off) inc += o;
  }
  if (lane == 31) part[warp] = inc;
  if (tid < walkers) seq_of[tid] = p.num_seqs;
  __syncthreads();
  int before = inc - mine, total = 0;
  for (int w = 0; w < warps; ++w) {
    if (w < warp) before += part[w];
    total += part[w];
  }
  const int range_len = range_length(total, p.ranges, kMinTiles);
  int at = before;
  for (int i = lo; i < hi; ++i) {
    const int end = at + cost_of(seen_of(p, i, unit, false), unit);
    for (int w = 0; w < walkers; ++w) {
      const long long first = static_cast<long long>(range_of(w)) * range_len;
      if (first >= at && first < end) {
        seq_of[w] = i;
        pos_of[w] = at;
      }
    }
    at = end;
  }
  __syncthreads();
  return Plan{range_len, total};
}

// Zeros for the sequences that see nothing, spread over the CTAs; `threads` threads of
// this one call it.
__device__ __forceinline__ void zero_rows(const WarpParams &p, int threads) {
  for (int i = blockIdx.x; i < p.num_seqs; i += gridDim.x) {
    if (__ldg(p.context_lens + i) > 0 && p.max_context_len > 0) continue;
    if (p.cuts_by_seq && threadIdx.x == 0) p.cuts[i] = make_int4(-1, 0, 0, 0);
    uint4 *dst = reinterpret_cast<uint4 *>(p.out + static_cast<int64_t>(i) * p.num_q_heads * kHD);
    for (int x = threadIdx.x; x < p.num_q_heads * (kHD / 8); x += threads) dst[x] = make_uint4(0, 0, 0, 0);
  }
}

// The parts of sequences in one range of the line, one after the other.
struct Walk {
  int seq, pos;
  long long line0;
  int line1, range_len;
  // the current part: tiles [t0, t1) of all `tiles` of sequence `seq`
  Seen seen;
  int t0, t1, tiles;

  __device__ __forceinline__ Walk(const Plan &plan, int range, int seq_at, int pos_at)
      : seq(seq_at - 1), pos(pos_at), range_len(plan.range_len) {
    line0 = static_cast<long long>(range) * plan.range_len;
    line1 = static_cast<int>(min(line0 + plan.range_len, static_cast<long long>(plan.total)));
  }
  // The entry of WarpParams::cuts that this range stands for; before the first next().
  __device__ __forceinline__ void begin(const WarpParams &p, int range, int unit) const {
    if (p.cuts_by_seq) return;
    int4 cut = make_int4(-1, 0, 0, 0);
    if (seq + 1 < p.num_seqs && pos + kSegTiles < line0) {
      const int r0 = (pos + kSegTiles) / range_len;
      const int r1 = (pos + cost_of(seen_of(p, seq + 1, unit, false), unit) - 1) / range_len;
      if (range == r0 + 1) cut = make_int4(seq + 1, r0, r1, 0);
    }
    p.cuts[range] = cut;
  }
  // The entry of the sequence that begins with the current part.
  __device__ __forceinline__ void entry(const WarpParams &p, int range) const {
    if (p.cuts_by_seq && t0 == 0)
      p.cuts[seq] = make_int4(seq, range, static_cast<int>((pos - 1) / range_len), 0);
  }
  __device__ __forceinline__ bool next(const WarpParams &p, int unit) {
    while (++seq < p.num_seqs && pos < line1) {
      seen = seen_of(p, seq, unit, false);
      tiles = tiles_of(seen, unit);
      const int first = pos + kSegTiles;
      t0 = static_cast<int>(max(line0 - first, 0ll));
      t1 = min(line1 - first, tiles);
      pos += cost_of(seen, unit);
      if (t0 < t1) return true;
    }
    return false;
  }
  __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == tiles; }
};

// ----------------------------------------------------------- direct loads --

// Every warp loads its tiles itself, whatever the block size. NT: tiles of 8 query
// heads a warp computes for its KV head.
template <bool kFp8, int NT>
__global__ void __launch_bounds__(kDirectWarps * 32, kFp8 && NT == 1 ? 2 : 1)
decode_direct_kernel(const WarpParams p) {
  using H = Heads<kFp8, NT>;
  __shared__ int s_part[kDirectWarps], s_seq[kDirectWarps], s_pos[kDirectWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, kp = lane & 3;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int vheads = p.num_kv_heads * p.chunks;
  auto range_of = [&](int w) { return (static_cast<int>(blockIdx.x) * kDirectWarps + w) / vheads; };
  const Plan plan = plan_ranges(p, 1, kDirectWarps, s_part, s_seq, s_pos, range_of);
  const int range = range_of(warp), vh = (blockIdx.x * kDirectWarps + warp) % vheads;
  const int kvh = vh / p.chunks, head0 = vh % p.chunks * p.per_chunk;
  const int heads = min(p.per_chunk, p.group - head0);       // of this warp
  constexpr int kRow = kFp8 ? kHD : 2 * kHD;                 // bytes of a head's row
  const int64_t row_bytes = static_cast<int64_t>(p.num_kv_heads) * kRow;
  const uint8_t *kbase = p.k_cache + kvh * kRow + 32 * kp;
  const uint8_t *vbase = p.v_cache + kvh * kRow + 16 * g;
  H x;
  Walk walk(plan, range, s_seq[warp], s_pos[warp]);
  const bool tells = vh == 0 && lane == 0 && range < p.ranges;
  if (tells) walk.begin(p, range, 1);
  zero_rows(p, blockDim.x);
  while (walk.next(p, 1)) {
    if (tells) walk.entry(p, range);
    const Seen &seen = walk.seen;
    const int t1 = walk.t1;
    // the lane's token of a tile: its block and its row in the block
    const int32_t *bt = p.block_tables + static_cast<int64_t>(walk.seq) * p.max_blocks_per_seq;
    auto look_up = [&](int t, int &id, int &off) {
      const int j = t * kTok + (lane & 15);
      id = -1;
      off = 0;
      if (t < t1 && j < seen.units) {
        const uint32_t at = j + (j >= seen.front ? seen.gap : 0);
        const uint32_t b = div_of(at, p.bs);
        off = static_cast<int>(at - b * p.bs.d);
        id = __ldg(bt + b);
      }
    };
    // cache row of the lane's token (-1: none, or one between the sinks and the
    // window; -2: of a bad block, a zero key and value as in the rings); its scale, of K
    // in the lower half of the warp and of V in the upper
    auto resolve = [&](int t, int id, int off, int &row, float &scale) {
      const int j = t * kTok + (lane & 15);
      const int at = j + (j >= seen.front ? seen.gap : 0);
      const bool real = t < t1 && j < seen.units && (at < p.sinks || at >= seen.first);
      const bool good = real && id >= 0 && id < p.num_blocks;
      if (real && !good && lane < 16) raise_error(p.err, PKV_DEVERR_BLOCK_ID);
      row = good ? id * static_cast<int>(p.bs.d) + off : real ? -2 : -1;
      scale = 0.f;
      if constexpr (kFp8)
        if (good) scale = __ldg((lane < 16 ? p.k_scales : p.v_scales) + static_cast<int64_t>(id) * p.num_kv_heads + kvh);
    };
    uint4 kr[2][H::kKL], vr[4][H::kVL];
    auto load_k = [&](int row) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = __shfl_sync(0xffffffffu, row, g + 8 * i);
        const uint8_t *src = kbase + r * row_bytes;
#pragma unroll
        for (int d = 0; d < H::kKL; ++d)
          kr[i][d] = r >= 0 ? ld_once(src + (d >> 1) * 128 + (d & 1) * 16) : make_uint4(0, 0, 0, 0);
      }
    };
    auto load_v = [&](int row) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = __shfl_sync(0xffffffffu, row, 2 * kp + (i & 1) + 8 * (i >> 1));
        const uint8_t *src = vbase + r * row_bytes;
#pragma unroll
        for (int d = 0; d < H::kVL; ++d) vr[i][d] = r >= 0 ? ld_once(src + d * 128) : make_uint4(0, 0, 0, 0);
      }
    };
    // A token's heads lie side by side, but the warps that take them come by at eight
    // different times: a tile ahead of its loads one of them asks L2 for all of them.
    auto ask = [&](int r) {
      if (r >= 0 && (lane & 15) % vheads == vh)
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;"
                     :: "l"((lane < 16 ? p.k_cache : p.v_cache) + r * row_bytes), "r"(static_cast<uint32_t>(row_bytes)));
    };
    int id, off, row, next_row;
    float scale, next_scale;
    look_up(walk.t0, id, off);
    resolve(walk.t0, id, off, row, scale);
    load_k(row);
    load_v(row);
    look_up(walk.t0 + 1, id, off);
    resolve(walk.t0 + 1, id, off, next_row, next_scale);
    ask(next_row);
    look_up(walk.t0 + 2, id, off);
    const int64_t out_row = static_cast<int64_t>(walk.seq) * p.num_q_heads + kvh * p.group + head0;
    uint4 raw[NT][4];
    x.load_q(p.q + out_row * kHD, heads, raw);
    x.start(raw, p.scale_log2);
#pragma unroll 1
    for (int t = walk.t0; t < t1; ++t) {
      float s[NT][4];
      x.scores(kr, s);
      const bool real0 = __shfl_sync(0xffffffffu, row, g) != -1, real1 = __shfl_sync(0xffffffffu, row, g + 8) != -1;
      float ks0 = 1.f, ks1 = 1.f, vs0 = 0.f, vs1 = 0.f;
      if constexpr (kFp8) {
        ks0 = __shfl_sync(0xffffffffu, scale, g);
        ks1 = __shfl_sync(0xffffffffu, scale, g + 8);
        const float ls = lg2(scale);
        vs0 = __shfl_sync(0xffffffffu, ls, g + 16);
        vs1 = __shfl_sync(0xffffffffu, ls, g + 24);
      }
      // the next tile's K is on its way while the softmax runs, its V after the PV
      int row2;
      float scale2;
      resolve(t + 2, id, off, row2, scale2);
      ask(row2);
      look_up(t + 3, id, off);
      if (t + 1 < t1) load_k(next_row);
      uint32_t pb[NT][2];
      x.weights(s, real0, real1, ks0, ks1, vs0, vs1, pb);
      x.accumulate(vr, pb);
      if (t + 1 < t1) load_v(next_row);
      row = next_row;
      scale = next_scale;
      next_row = row2;
      next_scale = scale2;
    }
    const int64_t rec = (static_cast<int64_t>(range * 2 + (walk.t0 == 0 ? 1 : 0)) * vheads + vh) * p.per_chunk;
    x.finish(walk.whole(), heads, p.out + out_row * kHD, p.ml + rec, p.po + rec * kHD);
  }
}

// --------------------------------------------------- shared-memory rings --

// Bytes of one stage: K and V of a tile, all heads of the CTA.
__host__ __device__ constexpr int stage_bytes(bool fp8, int heads) { return 2 * kTok * heads * (fp8 ? kHD : 2 * kHD); }

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, const volatile int *abort) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort));
}

// A producer warp per ring loads tiles of 16 tokens, all KV heads of the CTA at once,
// as one or two boxes (units) of K and of V; vheads warps per ring take one KV head's
// rows each out of shared memory. A box lands as [head][token][128 bytes] (bf16: two
// such halves of 64 dims), swizzled by the token, which makes every 16-byte load
// below free of bank conflicts.
template <bool kFp8, int NT>
__global__ void __launch_bounds__(kRingWarps * 32, 1)
decode_ring_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                   const WarpParams p) {
  using H = Heads<kFp8, NT>;
  constexpr int kHalves = kFp8 ? 1 : 2;       // 128-byte pieces of a head's row
  extern __shared__ uint8_t smem_raw[];
  __shared__ int s_part[kRingWarps], s_seq[kRingWarps], s_pos[kRingWarps];
  __shared__ uint64_t s_bar[2 * kMaxStages * (kRingWarps / 2)];   // full, empty; a ring has two warps at least
  __shared__ int s_abort;
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, kp = lane & 3;
  const int hc = p.heads_per_cta, stages = p.stages;
  const int ring_warps = hc * p.chunks;                       // consumers of a ring
  const int consumers = ring_warps * p.rings;
  const int ring = warp < consumers ? warp / ring_warps : warp - consumers;
  auto full = [&](int s) { return smem_addr(&s_bar[2 * (ring * stages + s)]); };
  auto empty = [&](int s) { return smem_addr(&s_bar[2 * (ring * stages + s) + 1]); };
  volatile int *abort = &s_abort;
  if (threadIdx.x == 0) {
    for (int i = 0; i < p.rings * stages; ++i) {
      mbar_init(smem_addr(&s_bar[2 * i]), 1);
      mbar_init(smem_addr(&s_bar[2 * i + 1]), ring_warps);
    }
    s_abort = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  // launched while the kernel before this one drains: nothing of its is read before here
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // ring r of CTA b: range (b / groups) * rings + r of head group b % groups
  const int hg = blockIdx.x % p.head_groups;
  auto range_of = [&](int r) { return static_cast<int>(blockIdx.x) / p.head_groups * p.rings + r; };
  const Plan plan = plan_ranges(p, p.unit, p.rings, s_part, s_seq, s_pos, range_of);
  const int range = range_of(ring);
  const int bytes = stage_bytes(kFp8, hc);
  const uint32_t ring_base = base + ring * stages * bytes;
  // strides of a stage in bytes: V behind K; dims halves; heads; tokens 8 .. 15
  const uint32_t v_off = bytes / 2, half_dims = kTok * hc * 128;
  const uint32_t head_step = p.unit * 128;
  const uint32_t upper = p.unit == 16 ? 1024u : v_off / 2;
  const uint32_t upper_dims = p.unit == 16 ? half_dims : half_dims / 2;   // dims halves of one box
  Walk walk(plan, range, s_seq[ring], s_pos[ring]);
  int s = 0;                                                  // the ring's next stage,
  uint32_t phase = 0;                                         // and the parity of its turn
  auto advance = [&]() {
    if (++s == stages) {
      s = 0;
      phase ^= 1;
    }
  };
  bool ok = true;

  if (warp >= consumers) {
    // ------------------------------------------------------------- producer
    const bool tells = lane == 0 && hg == 0;
    if (tells) walk.begin(p, range, p.unit);
    const int per_tile = kTok / p.unit, batch = 32 / per_tile;  // units of a tile, tiles of a batch
    int issued = 0;
    const int oob_row = p.num_blocks * static_cast<int>(p.bs.d);
    while (ok && walk.next(p, p.unit)) {
      if (tells) walk.entry(p, range);
      const int32_t *bt = p.block_tables + static_cast<int64_t>(walk.seq) * p.max_blocks_per_seq;
      for (int tb = walk.t0; ok && tb < walk.t1; tb += batch) {
        // the lane's unit of the batch: its first cache row; behind the last one, and
        // for a bad block id, rows behind the pool, which read as zero
        const int u = tb * per_tile + lane;
        int row = oob_row;
        if (u < walk.seen.units && u < walk.t1 * per_tile) {
          const uint32_t at = static_cast<uint32_t>(u + (u >= walk.seen.front ? walk.seen.gap : 0)) * p.unit;
          const uint32_t b = div_of(at, p.bs);
          const int id = __ldg(bt + b);
          if (id >= 0 && id < p.num_blocks) row = id * static_cast<int>(p.bs.d) + static_cast<int>(at - b * p.bs.d);
          else raise_error(p.err, PKV_DEVERR_BLOCK_ID);
        }
        const int n = min(batch, walk.t1 - tb);
        for (int j = 0; j < n; ++j) {
          int good = 1;
          if (lane == 0) {
            // (the turn before an unused barrier's first one counts as done)
            if (!mbar_wait(empty(s), phase ^ 1, abort)) {
              good = 0;
              *abort = 1;
              raise_error(p.err, PKV_DEVERR_TIMEOUT);
            } else {
              mbar_arrive_expect_tx(full(s), bytes);
            }
          }
          ok = __shfl_sync(0xffffffffu, good, 0);
          if (!ok) break;
          // lane: which of K and V, of the dims halves and of the tile's units it loads
          const int unit = lane % per_tile, half = lane / per_tile % kHalves, is_v = lane / (per_tile * kHalves);
          const int r = __shfl_sync(0xffffffffu, row, j * per_tile + unit);
          if (is_v < 2) {
            const uint32_t dst = ring_base + s * bytes + is_v * v_off + unit * (v_off / per_tile) + half * upper_dims;
            tma_load_3d(dst, is_v ? &tm_v : &tm_k, half * 64, r, hg * hc, full(s));
          }
          ++issued;
          advance();
        }
      }
    }
    // every copy lands before the CTA may exit
    if (lane == 0)
      for (int j = max(0, issued - stages); j < issued; ++j) mbar_wait(full(j % stages), (j / stages) & 1, nullptr);
  } else {
    // ------------------------------------------------------------ consumers
    zero_rows(p, consumers * 32);
    const int in_ring = warp % ring_warps;
    const int kvh = hg * hc + in_ring / p.chunks, head0 = in_ring % p.chunks * p.per_chunk;
    const bool real_head = kvh < p.num_kv_heads;              // a group may hang over the last head
    const int heads = real_head ? min(p.per_chunk, p.group - head0) : 0;
    const int vheads = p.num_kv_heads * p.chunks, vh = kvh * p.chunks + in_ring % p.chunks;
    const uint32_t head_base = ring_base + in_ring / p.chunks * head_step;
    // 16-byte pieces of the lane: K row g: pieces 2 kp, 2 kp + 1; V rows 2 kp, 2 kp + 1: piece g
    const uint32_t k0 = g * 128 + (((2 * kp) ^ g) << 4), k1 = g * 128 + (((2 * kp + 1) ^ g) << 4);
    const uint32_t v0 = 2 * kp * 128 + ((g ^ (2 * kp)) << 4), v1 = (2 * kp + 1) * 128 + ((g ^ (2 * kp + 1)) << 4);
    H x;
    while (ok && walk.next(p, p.unit)) {
      const Seen seen = walk.seen;
      const int64_t out_row = static_cast<int64_t>(walk.seq) * p.num_q_heads + kvh * p.group + head0;
      uint4 raw[NT][4];
      x.load_q(p.q + (real_head ? out_row * kHD : 0), heads, raw);
      const int32_t *bt = p.block_tables + static_cast<int64_t>(walk.seq) * p.max_blocks_per_seq;
      // fp8: scales of 8 tiles at a time, lane = (8 tokens, K or V): ids a batch ahead
      float sc = 0.f, next_sc = 0.f;
      auto scale_of = [&](int tb) {
        const int j = tb * kTok + (lane >> 1) * 8;            // first of the 8 tokens on the walk
        const int u = j / p.unit;
        float v = 0.f;
        if (real_head && u < seen.units) {
          const uint32_t at = static_cast<uint32_t>(u + (u >= seen.front ? seen.gap : 0)) * p.unit;
          const int id = __ldg(bt + div_of(at, p.bs));
          if (id >= 0 && id < p.num_blocks)
            v = __ldg((lane & 1 ? p.v_scales : p.k_scales) + static_cast<int64_t>(id) * p.num_kv_heads + kvh);
        }
        return v;
      };
      if constexpr (kFp8) {
        sc = scale_of(walk.t0);
        if (walk.t0 + 8 < walk.t1) next_sc = scale_of(walk.t0 + 8);
        if (lane & 1) sc = lg2(sc);
      }
      x.start(raw, p.scale_log2);
#pragma unroll 1
      for (int t = walk.t0; t < walk.t1; ++t) {
        if (!warp_wait(full(s), phase, abort)) {
          ok = false;
          *abort = 1;
          raise_error(p.err, PKV_DEVERR_TIMEOUT);
          break;
        }
        const uint32_t kt = head_base + s * bytes, vt = kt + v_off;
        uint4 k[2][H::kKL], v[4][H::kVL];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int d = 0; d < H::kKL; ++d)
            k[i][d] = lds128(kt + i * upper + (d >> 1) * upper_dims + (d & 1 ? k1 : k0));
        float sv[NT][4];
        x.scores(k, sv);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int d = 0; d < H::kVL; ++d) v[i][d] = lds128(vt + (i >> 1) * upper + d * upper_dims + (i & 1 ? v1 : v0));
        // first positions of the tile's two eights
        const int j0 = t * kTok, j1 = j0 + 8;
        const int front = seen.front * p.unit, gap = seen.gap * p.unit;
        const int a0 = j0 + (j0 >= front ? gap : 0), a1 = j1 + (j1 >= front ? gap : 0);
        auto counts = [&](int at) { return at < seen.ctx && (at < p.sinks || at >= seen.first); };
        const bool real0 = counts(a0 + g), real1 = counts(a1 + g);
        float ks0 = 1.f, ks1 = 1.f, vs0 = 0.f, vs1 = 0.f;
        if constexpr (kFp8) {
          const int b = (t - walk.t0) & 7;
          ks0 = __shfl_sync(0xffffffffu, sc, 4 * b);
          vs0 = __shfl_sync(0xffffffffu, sc, 4 * b + 1);
          ks1 = __shfl_sync(0xffffffffu, sc, 4 * b + 2);
          vs1 = __shfl_sync(0xffffffffu, sc, 4 * b + 3);
          if (b == 7) {
            sc = lane & 1 ? lg2(next_sc) : next_sc;
            if (t + 9 < walk.t1) next_sc = scale_of(t + 9);
          }
        }
        uint32_t pb[NT][2];
        x.weights(sv, real0, real1, ks0, ks1, vs0, vs1, pb);
        // what a row that does not count holds is not known: 0 times NaN is NaN
        if (!__all_sync(0xffffffffu, real0 && real1)) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (!counts((i >> 1 ? a1 : a0) + 2 * kp + (i & 1)))
#pragma unroll
              for (int d = 0; d < H::kVL; ++d) v[i][d] = make_uint4(0, 0, 0, 0);
        }
        x.accumulate(v, pb);
        __syncwarp();
        if (lane == 0) mbar_arrive(empty(s));
        advance();
      }
      if (!ok) break;
      const int64_t rec = (static_cast<int64_t>(range * 2 + (walk.t0 == 0 ? 1 : 0)) * vheads + vh) * p.per_chunk;
      x.finish(walk.whole(), heads, p.out + out_row * kHD, p.ml + rec, p.po + rec * kHD);
    }
  }
}

// --------------------------------------------------------------- combine --

// `share` warps per (entry of cuts, query head) merge the records of a cut sequence:
// out = sum O_i 2^(M_i - M*) / sum l_i 2^(m_i - m*) * drop * 2^(M* - m*)
__global__ void __launch_bounds__(kCombineWarps * 32) decode_warp_combine_kernel(const WarpParams p, int share, float drop) {
  __shared__ float4 s_acc[kCombineWarps][32];
  __shared__ float s_sum[kCombineWarps];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 cut = p.cuts[blockIdx.x];
  const int seq = cut.x, r0 = cut.y, r1 = cut.z;
  if (!merges_entry(seq, r0, r1, blockIdx.x, p.cuts_by_seq, p.num_seqs, p.ranges)) return;   // the whole CTA
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = warp % share;
  const int qh = blockIdx.y * (kCombineWarps / share) + warp / share;
  const bool row = qh < p.num_q_heads;
  const int in_group = qh % p.group;
  const int vheads = p.num_kv_heads * p.chunks;
  const int vh = qh / p.group * p.chunks + in_group / p.per_chunk, h = in_group % p.per_chunk;
  auto record = [&](int r) { return (static_cast<int64_t>(2 * r + (r == r0 ? 1 : 0)) * vheads + vh) * p.per_chunk + h; };
  const int n = row ? r1 - r0 + 1 : 0;
  // records base + (k + 0 .. 7) * share; the first ones are on their way while their
  // factors are worked out
  float4 x[8];
  auto fetch = [&](int base, int k) {
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int i = base + (k + u) * share;
      x[u] = i < n ? *(reinterpret_cast<const float4 *>(p.po + record(r0 + i) * kHD) + lane)
                   : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  };
  fetch(part, 0);
  float top = -INFINITY, topw = -INFINITY, sum = 0.f;
  for (int i = lane; i < n; i += 32) {
    const float4 v = p.ml[record(r0 + i)];
    top = fmaxf(top, v.x);
    topw = fmaxf(topw, v.z);
  }
#pragma unroll
  for (int x = 16; x >= 1; x >>= 1) {
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    topw = fmaxf(topw, __shfl_xor_sync(0xffffffffu, topw, x));
  }
  const float ref = top == -INFINITY ? 0.f : top, refw = topw == -INFINITY ? 0.f : topw;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  // records part, part + share, ...: 32 at a time, a lane each for their factors
  for (int base = part; base < n; base += 32 * share) {
    float f = 0.f;
    const int own = base + lane * share;
    if (own < n) {
      const float4 v = p.ml[record(r0 + own)];
      sum += v.y * ex2(v.x - ref);
      f = ex2(v.z - refw);
    }
    const int left = min(32, (n - base + share - 1) / share);
    for (int k = 0; k < left; k += 8) {
      if (base != part || k > 0) fetch(base, k);
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const float y = __shfl_sync(0xffffffffu, f, k + u);
        if (k + u < left) {
          acc.x += x[u].x * y;
          acc.y += x[u].y * y;
          acc.z += x[u].z * y;
          acc.w += x[u].w * y;
        }
      }
    }
  }
#pragma unroll
  for (int x = 16; x >= 1; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
  if (share > 1) {
    s_acc[warp][lane] = acc;
    if (lane == 0) s_sum[warp] = sum;
    __syncthreads();
    if (part > 0) return;
    for (int w = 1; w < share; ++w) {
      const float4 x = s_acc[warp + w][lane];
      acc = make_float4(acc.x + x.x, acc.y + x.y, acc.z + x.z, acc.w + x.w);
      sum += s_sum[warp + w];
    }
  }
  if (!row) return;
  const float f = 1.f / sum * drop, fw = ex2_far(refw - ref);
  reinterpret_cast<uint2 *>(p.out + (static_cast<int64_t>(seq) * p.num_q_heads + qh) * kHD)[lane] =
      make_uint2(float2_to_bf16x2(acc.x * f * fw, acc.y * f * fw), float2_to_bf16x2(acc.z * f * fw, acc.w * f * fw));
}

struct Shape {
  int chunks, per_chunk, ranges, grid;
  bool wide;           // two tiles of 8 query heads a warp
  bool ring;
  int unit, heads_per_cta, head_groups, rings, stages, warps;
};

// Ranges: as many as resident walkers of one (KV head, chunk) pair.
bool shape_of(int num_q_heads, int num_kv_heads, int block_size, bool fp8, Shape *s) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const int sms = sm_count(dev);
  if (sms <= 0) return false;
  const int group = num_q_heads / num_kv_heads;
  // fp8 with one or two KV heads: warps of 8 query heads each instead of 16 (512
  // sequences, groups of 16: 62 us against 79 with one KV head, 106 against 122 with
  // two, but 197 against 166 with four and 374 against 301 with eight)
  s->wide = group > 8 && !(fp8 && num_kv_heads <= 2);
  const int most = s->wide ? 16 : 8;
  s->chunks = (group + most - 1) / most;
  s->per_chunk = (group + s->chunks - 1) / s->chunks;
  const int vheads = num_kv_heads * s->chunks;
  s->ring = block_size % 8 == 0 && s->chunks < kRingWarps;
  if (s->ring) {
    s->unit = block_size % 16 == 0 ? 16 : 8;
    int heads = (kRingWarps - 1) / s->chunks;                  // a warp per (head, chunk) and a producer
    if (heads > 8) heads = 8;
    s->head_groups = (num_kv_heads + heads - 1) / heads;
    s->heads_per_cta = (num_kv_heads + s->head_groups - 1) / s->head_groups;
    const int bytes = stage_bytes(fp8, s->heads_per_cta), ring_warps = s->heads_per_cta * s->chunks;
    s->rings = kRingWarps / (ring_warps + 1);
    while (s->rings > 1 && kRingBytes / (s->rings * bytes) < 3) --s->rings;
    s->stages = kRingBytes / (s->rings * bytes);
    if (s->stages > kMaxStages) s->stages = kMaxStages;
    s->warps = s->rings * (ring_warps + 1);
    s->grid = sms / s->head_groups;                            // per head group
    if (s->grid < 1) s->grid = 1;
    s->ranges = s->grid * s->rings;
    s->grid *= s->head_groups;
    return true;
  }
  const int ctas = sms * (fp8 && !s->wide ? 2 : 1);
  s->ranges = ctas * kDirectWarps / vheads;
  if (s->ranges < 1) s->ranges = 1;
  s->grid = (s->ranges * vheads + kDirectWarps - 1) / kDirectWarps;
  return true;
}

size_t cuts_bytes(const Shape &s) { return (sizeof(int4) * s.ranges + 255) & ~size_t(255); }

size_t records_of(const Shape &s, int num_kv_heads) {
  return static_cast<size_t>(s.ranges) * 2 * num_kv_heads * s.chunks * s.per_chunk;
}

size_t bytes_of(const Shape &s, int num_kv_heads) {
  return cuts_bytes(s) + records_of(s, num_kv_heads) * (sizeof(float4) + kHD * sizeof(float));
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

// Boxes of 128 bytes of `unit` tokens of `heads` KV heads.
bool cache_map(CUtensorMap *map, const void *base, uint64_t rows, uint64_t hkv, bool fp8, int unit, int heads) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t row = fp8 ? kHD : 2 * kHD;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(kHD), rows, hkv};
  cuuint64_t strides[2] = {hkv * row, row};
  cuuint32_t box[3] = {fp8 ? 128u : 64u, static_cast<cuuint32_t>(unit), static_cast<cuuint32_t>(heads)};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims,
            strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

using RingKernel = void (*)(CUtensorMap, CUtensorMap, WarpParams);

// Largest dynamic shared memory of kernel `which`, set once a device.
cudaError_t allow_smem(const void *kern, int which, int bytes) {
  static std::atomic<uint64_t> done[4];
  int dev = 0;
  if (cudaError_t e = cudaGetDevice(&dev)) return e;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (dev <= 63 && (done[which].load() & bit)) return cudaSuccess;
  if (cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes)) return e;
  done[which].fetch_or(bit);
  return cudaSuccess;
}

// A launch that may begin while the kernel before it on the stream ends; the kernels
// here wait for that one before they read anything.
template <typename... P, typename... A>
cudaError_t launch_dependent(cudaStream_t stream, dim3 grid, int threads, int smem, void (*kern)(P...), const A &...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace

size_t decode_warp_workspace_bytes(int num_q_heads, int num_kv_heads) {
  size_t need = 0;
  for (bool fp8 : {false, true})
    for (int block_size : {1, 8}) {        // every path
      Shape s;
      if (!shape_of(num_q_heads, num_kv_heads, block_size, fp8, &s)) return 0;
      const size_t b = bytes_of(s, num_kv_heads);
      if (b > need) need = b;
    }
  return need;
}

bool decode_warp_fits(int num_seqs, int max_context_len) {
  const int64_t tiles = (static_cast<int64_t>(max_context_len) + kTok - 1) / kTok + kSegTiles;
  return num_seqs * tiles < (int64_t(1) << 31);
}

cudaError_t launch_decode_warp(const DecodeWarpArgs &a, cudaStream_t stream) {
  const bool fp8 = a.k_scales != nullptr;
  Shape s;
  if (!shape_of(a.num_q_heads, a.num_kv_heads, a.block_size, fp8, &s)) return cudaErrorInvalidValue;
  WarpParams p;
  p.out = static_cast<__nv_bfloat16 *>(a.out);
  p.q = static_cast<const __nv_bfloat16 *>(a.q);
  p.k_cache = static_cast<const uint8_t *>(a.k_cache);
  p.v_cache = static_cast<const uint8_t *>(a.v_cache);
  p.k_scales = a.k_scales;
  p.v_scales = a.v_scales;
  p.block_tables = a.block_tables;
  p.context_lens = a.context_lens;
  p.max_blocks_per_seq = a.max_blocks_per_seq;
  p.num_seqs = a.num_seqs;
  p.max_context_len = a.max_context_len;
  p.num_q_heads = a.num_q_heads;
  p.num_kv_heads = a.num_kv_heads;
  p.group = a.num_q_heads / a.num_kv_heads;
  p.chunks = s.chunks;
  p.per_chunk = s.per_chunk;
  p.num_blocks = a.num_blocks;
  p.bs.d = static_cast<uint32_t>(a.block_size);
  p.bs.mul = p.bs.shift = 0;
  if (a.block_size > 1) {
    // l = ceil(log2 d): n / d = (n * ceil(2^(31 + l) / d)) >> (31 + l) for n < 2^31
    int l = 1;
    while ((int64_t(1) << l) < a.block_size) ++l;
    p.bs.mul = static_cast<uint32_t>(((uint64_t(1) << (31 + l)) + a.block_size - 1) / a.block_size);
    p.bs.shift = static_cast<uint32_t>(l - 1);
  }
  // neither bound can hide a token beyond max_context_len
  p.window = a.window < a.max_context_len ? a.window : a.max_context_len;
  p.sinks = a.sinks < a.max_context_len ? a.sinks : a.max_context_len;
  p.scale_log2 = a.scale * kLog2e;
  p.ranges = s.ranges;
  p.cuts = static_cast<int4 *>(a.workspace);
  p.cuts_by_seq = a.num_seqs <= s.ranges;
  p.ml = reinterpret_cast<float4 *>(static_cast<uint8_t *>(a.workspace) + cuts_bytes(s));
  p.po = reinterpret_cast<float *>(p.ml + records_of(s, a.num_kv_heads));
  p.err = a.err;
  if (s.ring) {
    p.unit = s.unit;
    p.heads_per_cta = s.heads_per_cta;
    p.head_groups = s.head_groups;
    p.rings = s.rings;
    p.stages = s.stages;
    const uint64_t rows = static_cast<uint64_t>(a.num_blocks) * a.block_size;
    CUtensorMap tk, tv;
    if (!cache_map(&tk, a.k_cache, rows, a.num_kv_heads, fp8, s.unit, s.heads_per_cta) ||
        !cache_map(&tv, a.v_cache, rows, a.num_kv_heads, fp8, s.unit, s.heads_per_cta))
      return cudaErrorInvalidValue;
    RingKernel kern = fp8 ? (s.wide ? decode_ring_kernel<true, 2> : decode_ring_kernel<true, 1>)
                          : (s.wide ? decode_ring_kernel<false, 2> : decode_ring_kernel<false, 1>);
    if (cudaError_t e = allow_smem(reinterpret_cast<const void *>(kern), (fp8 ? 1 : 0) + (s.wide ? 2 : 0), kRingBytes + 1024))
      return e;
    const int smem = s.rings * s.stages * stage_bytes(fp8, s.heads_per_cta) + 1024;
    if (cudaError_t e = launch_dependent(stream, dim3(s.grid), s.warps * 32, smem, kern, tk, tv, p)) return e;
  } else {
    auto kern = fp8 ? (s.wide ? decode_direct_kernel<true, 2> : decode_direct_kernel<true, 1>)
                    : (s.wide ? decode_direct_kernel<false, 2> : decode_direct_kernel<false, 1>);
    if (cudaError_t e = launch_dependent(stream, dim3(s.grid), kDirectWarps * 32, 0, kern, p)) return e;
  }
  // warps a merge: one for every 8 records that a sequence has on average
  int share = 1;
  while (share < kCombineWarps && share * 8 * static_cast<int64_t>(a.num_seqs) < s.ranges) share *= 2;
  const int rows = kCombineWarps / share;
  return launch_dependent(stream, dim3(p.cuts_by_seq ? a.num_seqs : s.ranges, (a.num_q_heads + rows - 1) / rows), kCombineWarps * 32, 0,
                          decode_warp_combine_kernel, p, share, fp8 ? kDrop : 1.f);
}

}  // namespace pkv
