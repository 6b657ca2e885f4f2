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
// group * 2 operations a byte; its rate is not what counts. So instead of whole
// tiles through shared memory, with warps meeting at barriers (decode_tcg.cu),
// a warp loads 16 tokens of one KV head straight into the registers that
// mma.m16n8k16 takes them from, and nothing is exchanged with another warp
// before the end of its keys:
//   S^T [16 tokens x 8 heads] = K [16 x 128] Q^T      8 MMAs
//   O^T [128 dims x 8 heads] += V^T [128 x 16] P^T    8 MMAs, P^T from S^T by
//                                                     two 8x8 transposes
// The order of the 128 dims inside the contraction is free, and so is the order
// of O's rows, so both are chosen so that every global load is 16 bytes a lane:
// of S's contraction a lane holds 16 (fp8) or 8 (bf16) neighbouring dims, and of
// V's rows the dims of 16 (8) neighbours of four tokens. Codes become f16 (exact)
// two at a time; scales are applied to the scores and to the weights. Loads of the
// next tile's K are issued when the tile's S has been computed, V's after its PV,
// the block table is looked up one tile further ahead.
//
// Split: the seen tokens of all sequences, in tiles of 16 with kSegTiles of
// overhead in front of each sequence, are one line that is cut into equal ranges;
// a warp takes one range of one KV head, the warps of a CTA neighbouring heads, so
// that a token's heads are read at the same time from one place. A sequence that a
// cut goes through leaves (m, l, O) records that a second launch merges.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <mutex>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kHD = 128;
constexpr int kWarps = 8;                  // of a CTA
constexpr int kThreads = kWarps * 32;
constexpr int kTok = 16;                   // tokens of a tile
constexpr int kSegTiles = 2;               // what starting a sequence costs, in tiles
constexpr int kMinTiles = 4;               // shortest range
constexpr float kLog2e = 1.4426950408889634f;
// A reference maximum is kept until a score exceeds it by this (log2): weights
// stay below 2^kGrow (bf16: exact range) and f16 weights, which are also scaled
// by 2^kLift, between 2^-24 and 2^15.
constexpr float kGrow = 8.f;
constexpr float kLift = 7.f;

// n / d for 0 <= n < 2^31 by a multiplication
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
  int *plan;           // [0] tiles of a range, [1 ..] starts of the sequences on the line
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

// Seen tokens of a sequence, how many positions behind the sinks are left out.
struct Seen {
  int n, shift;
};

__device__ __forceinline__ Seen seen_of(const WarpParams &p, int i, bool report) {
  int ctx = __ldg(p.context_lens + i);
  if (ctx < 0 || ctx > p.max_context_len) {
    if (report) raise_error(p.err, PKV_DEVERR_LENGTH);
    ctx = min(max(ctx, 0), p.max_context_len);
  }
  Seen s{ctx, 0};
  if (p.window > 0) s.shift = max(max(ctx - p.window, 0) - p.sinks, 0);
  s.n = ctx - s.shift;
  return s;
}

__device__ __forceinline__ int tiles_of(int n) { return (n + kTok - 1) / kTok; }
__device__ __forceinline__ int cost_of(int n) { return n > 0 ? tiles_of(n) + kSegTiles : 0; }

template <bool kFp8> constexpr int kLoads = kFp8 ? 2 : 4;   // 16-byte loads of a row's part a lane takes

// First dim of the d-th group of neighbours that a lane holds of a K row (and of
// Q), lane % 4 = kp, and of a V row (and of O), lane / 4 = n.
template <bool kFp8>
__device__ __forceinline__ int k_dim(int d, int kp) { return kFp8 ? 64 * d + 16 * kp : 32 * d + 8 * kp; }

// NT: tiles of 8 query heads a warp computes for its KV head
template <bool kFp8, int NT>
__global__ void __launch_bounds__(kThreads, kFp8 && NT == 1 ? 2 : 1)
decode_warp_kernel(const WarpParams p) {
  __shared__ int s_part[kWarps], s_seq[kWarps], s_pos[kWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, kp = lane & 3;       // MMA fragments: row (column of B) g, pair kp
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // ---- plan: where this CTA's ranges start on the line of all sequences
  const int vheads = p.num_kv_heads * p.chunks;
  const int per = (p.num_seqs + kThreads - 1) / kThreads;
  const int lo = min(tid * per, p.num_seqs), hi = min(lo + per, p.num_seqs);
  int mine = 0;
  for (int i = lo; i < hi; ++i) mine += cost_of(seen_of(p, i, blockIdx.x == 0).n);
  int inc = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, inc, off);
    if (lane >= off) inc += o;
  }
  if (lane == 31) s_part[warp] = inc;
  if (tid < kWarps) s_seq[tid] = p.num_seqs;
  __syncthreads();
  int before = inc - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += s_part[w];
    total += s_part[w];
  }
  const int range_len = max((total + p.ranges - 1) / p.ranges, kMinTiles);
  {
    int at = before;
    for (int i = lo; i < hi; ++i) {
      const int end = at + cost_of(seen_of(p, i, false).n);
      for (int w = 0; w < kWarps; ++w) {
        const long long first = static_cast<long long>((blockIdx.x * kWarps + w) / vheads) * range_len;
        if (first >= at && first < end) {
          s_seq[w] = i;
          s_pos[w] = at;
        }
      }
      if (blockIdx.x == 0) p.plan[1 + i] = at;
      at = end;
    }
    if (blockIdx.x == 0 && tid == 0) {
      p.plan[0] = range_len;
      p.plan[1 + p.num_seqs] = total;
    }
  }
  __syncthreads();

  const int range = (blockIdx.x * kWarps + warp) / vheads;
  const int vh = (blockIdx.x * kWarps + warp) % vheads;
  const int kvh = vh / p.chunks, head0 = vh % p.chunks * p.per_chunk;
  const int heads = min(p.per_chunk, p.group - head0);       // of this warp
  const long long line0 = static_cast<long long>(range) * range_len;
  const int line1 = static_cast<int>(min(line0 + range_len, static_cast<long long>(total)));
  constexpr int kRow = kFp8 ? kHD : 2 * kHD;                 // bytes of a head's row
  const int64_t row_bytes = static_cast<int64_t>(p.num_kv_heads) * kRow;
  const uint8_t *kbase = p.k_cache + kvh * kRow + k_dim<kFp8>(0, kp) * (kRow / kHD);
  const uint8_t *vbase = p.v_cache + kvh * kRow + 16 * g;
  // bytes between a lane's 16-byte loads of one K row / V row
  constexpr int kStepK = 64, kStepV = 128;
  constexpr int kKL = kFp8 ? 2 : 4, kVL = kFp8 ? 1 : 2;

  int seq = s_seq[warp], pos = s_pos[warp];
  for (; seq < p.num_seqs && pos < line1; ++seq) {
    const Seen seen = seen_of(p, seq, false);
    const int tiles = tiles_of(seen.n);
    const int first_tile = pos + kSegTiles;                  // on the line
    const int t0 = static_cast<int>(max(line0 - first_tile, 0ll)), t1 = min(line1 - first_tile, tiles);
    pos += cost_of(seen.n);
    if (t0 >= t1) continue;
    const bool whole = t0 == 0 && t1 == tiles;

    // the lane's token of a tile: its block and its row in the block
    const int32_t *bt = p.block_tables + static_cast<int64_t>(seq) * p.max_blocks_per_seq;
    auto look_up = [&](int t, int &id, int &off) {
      const int j = t * kTok + (lane & 15);
      id = -1;
      off = 0;
      if (t < t1 && j < seen.n) {
        const uint32_t at = j + (j >= p.sinks ? seen.shift : 0);
        const uint32_t b = div_of(at, p.bs);
        off = static_cast<int>(at - b * p.bs.d);
        id = __ldg(bt + b);
      }
    };
    // cache row of the lane's token (-1: none); its scale, of K in the lower half
    // of the warp and of V in the upper
    auto resolve = [&](int t, int id, int off, int &row, float &scale) {
      const bool real = t < t1 && t * kTok + (lane & 15) < seen.n;
      const bool good = real && id >= 0 && id < p.num_blocks;
      if (real && !good && lane < 16) raise_error(p.err, PKV_DEVERR_BLOCK_ID);
      row = good ? id * static_cast<int>(p.bs.d) + off : -1;
      scale = 0.f;
      if constexpr (kFp8)
        if (good) scale = __ldg((lane < 16 ? p.k_scales : p.v_scales) + static_cast<int64_t>(id) * p.num_kv_heads + kvh);
    };
    uint4 kr[2][kKL], vr[4][kVL];
    auto load_k = [&](int row) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int r = __shfl_sync(0xffffffffu, row, g + 8 * x);
        const uint8_t *src = kbase + r * row_bytes;
#pragma unroll
        for (int d = 0; d < kKL; ++d) kr[x][d] = r >= 0 ? ld_once(src + d * kStepK) : make_uint4(0, 0, 0, 0);
      }
    };
    auto load_v = [&](int row) {
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int r = __shfl_sync(0xffffffffu, row, 2 * kp + (x & 1) + 8 * (x >> 1));
        const uint8_t *src = vbase + r * row_bytes;
#pragma unroll
        for (int d = 0; d < kVL; ++d) vr[x][d] = r >= 0 ? ld_once(src + d * kStepV) : make_uint4(0, 0, 0, 0);
      }
    };
    int id, off, row;
    float scale;
    look_up(t0, id, off);
    resolve(t0, id, off, row, scale);
    look_up(t0 + 1, id, off);
    load_k(row);
    load_v(row);

    // ---- Q: B fragments, element (k, head g); qmul of the lane's heads 2 kp, 2 kp + 1
    uint32_t qf[NT][8][2];
    float qmul[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int h = nt * 8 + g;
      uint4 x[4];
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        // fp8: a lane's 16 dims are two loads
        const int dim = kFp8 ? k_dim<kFp8>(d >> 1, kp) + 8 * (d & 1) : k_dim<kFp8>(d, kp);
        x[d] = make_uint4(0, 0, 0, 0);
        if (h < heads)
          x[d] = __ldg(reinterpret_cast<const uint4 *>(
              p.q + (static_cast<int64_t>(seq) * p.num_q_heads + kvh * p.group + head0 + h) * kHD + dim));
      }
      uint32_t w[16];
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        w[4 * d] = x[d].x;
        w[4 * d + 1] = x[d].y;
        w[4 * d + 2] = x[d].z;
        w[4 * d + 3] = x[d].w;
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
        qmul[nt][0] = p.scale_log2 * __shfl_sync(0xffffffffu, down, 8 * kp);
        qmul[nt][1] = p.scale_log2 * __shfl_sync(0xffffffffu, down, 8 * kp + 4);
      } else {
        qmul[nt][0] = qmul[nt][1] = p.scale_log2;
      }
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        qf[nt][s][0] = w[2 * s];
        qf[nt][s][1] = w[2 * s + 1];
      }
    }

    float o[NT][8][4], m[NT][2], mw[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
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

#pragma unroll 1
    for (int t = t0; t < t1; ++t) {
      // ---- S^T = K Q^T
      float s[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[nt][e] = 0.f;
#pragma unroll
      for (int st = 0; st < 8; ++st) {
        uint32_t a[4];
        if constexpr (kFp8) {
          const uint32_t *x0 = &kr[0][st >> 2].x, *x1 = &kr[1][st >> 2].x;
          const uint32_t w0 = x0[st & 3], w1 = x1[st & 3];
          a[0] = e4m3x2_to_f16x2(static_cast<uint16_t>(w0));
          a[1] = e4m3x2_to_f16x2(static_cast<uint16_t>(w1));
          a[2] = e4m3x2_to_f16x2(static_cast<uint16_t>(w0 >> 16));
          a[3] = e4m3x2_to_f16x2(static_cast<uint16_t>(w1 >> 16));
        } else {
          const uint32_t *x0 = &kr[0][st >> 1].x, *x1 = &kr[1][st >> 1].x;
          a[0] = x0[2 * (st & 1)];
          a[1] = x1[2 * (st & 1)];
          a[2] = x0[2 * (st & 1) + 1];
          a[3] = x1[2 * (st & 1) + 1];
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma16<kFp8>(s[nt], a[0], a[1], a[2], a[3], qf[nt][st][0], qf[nt][st][1]);
      }
      // the lane's two tokens, g and g + 8, and their scales
      const bool real0 = __shfl_sync(0xffffffffu, row, g) >= 0, real1 = __shfl_sync(0xffffffffu, row, g + 8) >= 0;
      float ks0 = 1.f, ks1 = 1.f, vs0 = 0.f, vs1 = 0.f;
      if constexpr (kFp8) {
        ks0 = __shfl_sync(0xffffffffu, scale, g);
        ks1 = __shfl_sync(0xffffffffu, scale, g + 8);
        const float ls = lg2(scale);
        vs0 = __shfl_sync(0xffffffffu, ls, g + 16);
        vs1 = __shfl_sync(0xffffffffu, ls, g + 24);
      }
      // next tile's K while the softmax runs
      int next_row = -1;
      float next_scale = 0.f;
      if (t + 1 < t1) {
        resolve(t + 1, id, off, next_row, next_scale);
        look_up(t + 2, id, off);
        load_k(next_row);
      }
      // ---- softmax against the kept maxima
      bool grow = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x = s[nt][e] * qmul[nt][e & 1];
          if constexpr (kFp8) x *= e < 2 ? ks0 : ks1;
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
      uint32_t pb[NT][2];
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
        if constexpr (kFp8) {
          const __half2 h0 = __floats2half2_rn(w[0], w[1]), h1 = __floats2half2_rn(w[2], w[3]);
          pb[nt][0] = transpose8x8(*reinterpret_cast<const uint32_t *>(&h0));
          pb[nt][1] = transpose8x8(*reinterpret_cast<const uint32_t *>(&h1));
        } else {
          // the sum is of the rounded weights, so that the output stays a mean of V
          const uint32_t h0 = float2_to_bf16x2(w[0], w[1]), h1 = float2_to_bf16x2(w[2], w[3]);
          const float2 r0 = bf16x2_to_float2(h0), r1 = bf16x2_to_float2(h1);
          l[nt][0] += r0.x + r1.x;
          l[nt][1] += r0.y + r1.y;
          pb[nt][0] = transpose8x8(h0);
          pb[nt][1] = transpose8x8(h1);
        }
      }
      // ---- O^T += V^T P^T: tile i has the dims 2 i, 2 i + 1 of each lane's 16
#pragma unroll
      for (int w = 0; w < (kFp8 ? 4 : 8); ++w) {
        uint32_t a[8];
        if constexpr (kFp8) {
          // words of four dims: (token, next token) codes of a dim side by side
          const uint32_t x0 = (&vr[0][0].x)[w], x1 = (&vr[1][0].x)[w], x2 = (&vr[2][0].x)[w], x3 = (&vr[3][0].x)[w];
          const uint32_t p0 = __byte_perm(x0, x1, 0x5140), p1 = __byte_perm(x0, x1, 0x7362);
          const uint32_t p2 = __byte_perm(x2, x3, 0x5140), p3 = __byte_perm(x2, x3, 0x7362);
          a[0] = e4m3x2_to_f16x2(static_cast<uint16_t>(p0));
          a[1] = e4m3x2_to_f16x2(static_cast<uint16_t>(p0 >> 16));
          a[2] = e4m3x2_to_f16x2(static_cast<uint16_t>(p2));
          a[3] = e4m3x2_to_f16x2(static_cast<uint16_t>(p2 >> 16));
          a[4] = e4m3x2_to_f16x2(static_cast<uint16_t>(p1));
          a[5] = e4m3x2_to_f16x2(static_cast<uint16_t>(p1 >> 16));
          a[6] = e4m3x2_to_f16x2(static_cast<uint16_t>(p3));
          a[7] = e4m3x2_to_f16x2(static_cast<uint16_t>(p3 >> 16));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma16<kFp8>(o[nt][2 * w], a[0], a[1], a[2], a[3], pb[nt][0], pb[nt][1]);
            mma16<kFp8>(o[nt][2 * w + 1], a[4], a[5], a[6], a[7], pb[nt][0], pb[nt][1]);
          }
        } else {
          const uint32_t x0 = (&vr[0][w >> 2].x)[w & 3], x1 = (&vr[1][w >> 2].x)[w & 3];
          const uint32_t x2 = (&vr[2][w >> 2].x)[w & 3], x3 = (&vr[3][w >> 2].x)[w & 3];
          a[0] = __byte_perm(x0, x1, 0x5410);
          a[1] = __byte_perm(x0, x1, 0x7632);
          a[2] = __byte_perm(x2, x3, 0x5410);
          a[3] = __byte_perm(x2, x3, 0x7632);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16<kFp8>(o[nt][w], a[0], a[1], a[2], a[3], pb[nt][0], pb[nt][1]);
        }
      }
      if (t + 1 < t1) load_v(next_row);
      row = next_row;
      scale = next_scale;
    }

    // ---- the sequence's rows, or a record of this range's part
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float sum = l[nt][e];
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
        const int h = nt * 8 + 2 * kp + e;
        if (h >= heads) continue;
        // lane's dims: fp8 16 g + 0 .. 15; bf16 8 g + 0 .. 7 and 64 + 8 g + 0 .. 7
        float v[16];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[2 * i] = o[nt][i][e];
          v[2 * i + 1] = o[nt][i][e + 2];
        }
        const int dim0 = kFp8 ? 16 * g : 8 * g, dim1 = kFp8 ? dim0 + 8 : dim0 + 64;
        if (whole) {
          float f = 1.f / sum, fw = 1.f;            // 0 / 0: every seen score is -inf
          if constexpr (kFp8) fw = ex2(mw[nt][e] == -INFINITY ? 0.f : mw[nt][e] - m[nt][e] - kLift);
          uint32_t w[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) w[i] = float2_to_bf16x2(v[2 * i] * f * fw, v[2 * i + 1] * f * fw);
          __nv_bfloat16 *dst = p.out + (static_cast<int64_t>(seq) * p.num_q_heads + kvh * p.group + head0 + h) * kHD;
          *reinterpret_cast<uint4 *>(dst + dim0) = make_uint4(w[0], w[1], w[2], w[3]);
          *reinterpret_cast<uint4 *>(dst + dim1) = make_uint4(w[4], w[5], w[6], w[7]);
        } else {
          const int64_t rec = (static_cast<int64_t>(range * 2 + (t0 == 0 ? 1 : 0)) * vheads + vh) * p.per_chunk + h;
          float *dst = p.po + rec * kHD;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            *reinterpret_cast<float4 *>(dst + dim0 + 4 * i) = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
            *reinterpret_cast<float4 *>(dst + dim1 + 4 * i) =
                make_float4(v[8 + 4 * i], v[9 + 4 * i], v[10 + 4 * i], v[11 + 4 * i]);
          }
          if (g == 0) p.ml[rec] = make_float4(m[nt][e], sum, kFp8 ? mw[nt][e] : m[nt][e], 0.f);
        }
      }
  }
}

// --------------------------------------------------------------- combine --

// One warp per (sequence, query head) merges the records of a cut sequence:
// out = sum O_i 2^(M_i - M*) / sum l_i 2^(m_i - m*) * 2^(M* - m* - lift); a
// sequence that sees nothing gets zeros.
__global__ void __launch_bounds__(kThreads) decode_warp_combine_kernel(const WarpParams p, float lift) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const long long w = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int seq = static_cast<int>(w / p.num_q_heads), qh = static_cast<int>(w % p.num_q_heads);
  if (seq >= p.num_seqs) return;
  const int range_len = __ldg(p.plan), a = __ldg(p.plan + 1 + seq), b = __ldg(p.plan + 2 + seq);
  uint2 *dst = reinterpret_cast<uint2 *>(p.out + (static_cast<int64_t>(seq) * p.num_q_heads + qh) * kHD) + lane;
  if (a == b) {
    *dst = make_uint2(0, 0);
    return;
  }
  const int r0 = (a + kSegTiles) / range_len, r1 = (b - 1) / range_len;
  if (r0 == r1) return;
  const int in_group = qh % p.group;
  const int vheads = p.num_kv_heads * p.chunks;
  const int vh = qh / p.group * p.chunks + in_group / p.per_chunk, h = in_group % p.per_chunk;
  auto record = [&](int r) { return (static_cast<int64_t>(2 * r + (r == r0 ? 1 : 0)) * vheads + vh) * p.per_chunk + h; };
  float top = -INFINITY, topw = -INFINITY;
  for (int r = r0 + lane; r <= r1; r += 32) {
    const float4 v = p.ml[record(r)];
    top = fmaxf(top, v.x);
    topw = fmaxf(topw, v.z);
  }
#pragma unroll
  for (int x = 16; x >= 1; x >>= 1) {
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    topw = fmaxf(topw, __shfl_xor_sync(0xffffffffu, topw, x));
  }
  const float ref = top == -INFINITY ? 0.f : top, refw = topw == -INFINITY ? 0.f : topw;
  float sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int base = r0; base <= r1; base += 32) {
    float f = 0.f;
    if (base + lane <= r1) {
      const float4 v = p.ml[record(base + lane)];
      sum += v.y * ex2(v.x - ref);
      f = ex2(v.z - refw);
    }
    const int n = min(32, r1 - base + 1);
    for (int k = 0; k < n; k += 8) {
      float4 x[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        x[u] = k + u < n ? *(reinterpret_cast<const float4 *>(p.po + record(base + k + u) * kHD) + lane)
                         : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const float y = __shfl_sync(0xffffffffu, f, (k + u) & 31);
        if (k + u < n) {
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
  const float f = 1.f / sum, fw = ex2(refw - ref - lift);
  *dst = make_uint2(float2_to_bf16x2(acc.x * f * fw, acc.y * f * fw), float2_to_bf16x2(acc.z * f * fw, acc.w * f * fw));
}

struct Shape {
  int chunks, per_chunk, ranges, grid;
  bool wide;   // two tiles of 8 query heads a warp
};

// Ranges: as many as resident warps, over the (KV head, chunk) pairs.
bool shape_of(int num_q_heads, int num_kv_heads, bool fp8, Shape *s) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const int sms = sm_count(dev);
  if (sms <= 0) return false;
  const int group = num_q_heads / num_kv_heads;
  s->wide = group > 8;
  const int most = s->wide ? 16 : 8;
  s->chunks = (group + most - 1) / most;
  s->per_chunk = (group + s->chunks - 1) / s->chunks;
  const int vheads = num_kv_heads * s->chunks;
  const int ctas = sms * (fp8 && !s->wide ? 2 : 1);
  s->ranges = ctas * kWarps / vheads;
  if (s->ranges < 1) s->ranges = 1;
  s->grid = (s->ranges * vheads + kWarps - 1) / kWarps;
  return true;
}

size_t plan_bytes(int num_seqs) { return (sizeof(int) * (static_cast<size_t>(num_seqs) + 2) + 255) & ~size_t(255); }

size_t records_of(const Shape &s, int num_kv_heads) {
  return static_cast<size_t>(s.ranges) * 2 * num_kv_heads * s.chunks * s.per_chunk;
}

size_t bytes_of(int num_seqs, const Shape &s, int num_kv_heads) {
  return plan_bytes(num_seqs) + records_of(s, num_kv_heads) * (sizeof(float4) + kHD * sizeof(float));
}

}  // namespace

size_t decode_warp_workspace_bytes(int num_seqs, int num_q_heads, int num_kv_heads) {
  size_t need = 0;
  for (bool fp8 : {false, true}) {
    Shape s;
    if (!shape_of(num_q_heads, num_kv_heads, fp8, &s)) return 0;
    const size_t b = bytes_of(num_seqs, s, num_kv_heads);
    if (b > need) need = b;
  }
  return need;
}

bool decode_warp_fits(int num_seqs, int max_context_len, int num_q_heads) {
  const int64_t tiles = (static_cast<int64_t>(max_context_len) + kTok - 1) / kTok + kSegTiles;
  return num_seqs * tiles < (int64_t(1) << 31) && static_cast<int64_t>(num_seqs) * num_q_heads < (int64_t(1) << 31);
}

cudaError_t launch_decode_warp(const DecodeWarpArgs &a, cudaStream_t stream) {
  const bool fp8 = a.k_scales != nullptr;
  Shape s;
  if (!shape_of(a.num_q_heads, a.num_kv_heads, fp8, &s)) return cudaErrorInvalidValue;
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
  p.plan = static_cast<int *>(a.workspace);
  p.ml = reinterpret_cast<float4 *>(static_cast<uint8_t *>(a.workspace) + plan_bytes(a.num_seqs));
  p.po = reinterpret_cast<float *>(p.ml + records_of(s, a.num_kv_heads));
  p.err = a.err;
  auto kern = fp8 ? (s.wide ? decode_warp_kernel<true, 2> : decode_warp_kernel<true, 1>)
                  : (s.wide ? decode_warp_kernel<false, 2> : decode_warp_kernel<false, 1>);
  kern<<<s.grid, kThreads, 0, stream>>>(p);
  if (cudaError_t e = cudaGetLastError()) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((static_cast<int64_t>(a.num_seqs) * a.num_q_heads + kWarps - 1) / kWarps));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, decode_warp_combine_kernel, p, fp8 ? kLift : 0.f);
}

}  // namespace pkv
