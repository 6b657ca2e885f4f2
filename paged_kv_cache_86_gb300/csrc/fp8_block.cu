// fp8_block.cu -- an fp8 E4M3 cache with one scale per (block, KV head), written
// (pkv_store_kvcache_fp8_block) and read back (pkv_load_kvcache_fp8_block)
// (LLM Infra 101 v0.2, KV Quantization: the cache keeps low-bit values).
//
// The scale s of a block and head is a power of two: the smallest 2^e with
// max |x| <= 448 * 2^e over the block's finite values, e in [-120, 119]. E4M3 has
// its own exponent, so a power of two loses nothing against amax / 448 but the
// last factor below 2 of the subnormal range, and three things become exact:
// the product x / s before the one rounding to a code, the value code * s in
// bf16, and the change of a code to a larger scale (but where it becomes
// subnormal), so a block that is appended to a token at a time does not wear.
//
// A call's new tokens of a sequence are the positions context_len - n ..
// context_len - 1. The blocks they touch belong to that sequence alone, so one
// team of half-warps does everything about one (block, head, K or V): the
// maximum of the new rows, the scale, the codes, and, where the block holds older
// rows and the scale has to grow, those rows' codes in the new scale. No atomics,
// and no order between teams matters.
//
// What bounds them: the store reads 2 and writes 1 byte a value. 16384 tokens of 32
// prompts (8 KV heads, block 16) take 20.5 us, 4.9 TB/s, 0.72 of the measured copy
// rate: a third of the time is the chain lengths -> table -> rows of each of its 3.4
// waves of CTAs, the rest is shared by loads and the arithmetic of the codes (issue
// slots 0.66 busy). 64 registers for four CTAs an SM; three took 22.0 us, five (with
// spills) 25.8; 4 or 16 rows a half-warp instead of 8 26.0 and 28.0; one wave of CTAs
// with several blocks each 22.7. 512 tokens of 512 sequences: 4.6 us, the chain alone,
// where no scale grows; 7.7 where all do (block 16), and 68 at block 256, where one
// half-warp re-expresses up to 255 rows, four at a time.
// The read-back: 0.29 M tokens (8 KV heads) 284 us, 6.35 TB/s, 0.93 of the copy rate.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kTeams = kThreads / 16;   // half-warps of a CTA
constexpr int kHold = 8;                // rows a half-warp keeps in registers between its two passes
constexpr int kRowBytes = 128;          // codes of one head's row

// The largest i in [0, n) with a[i] <= t (0 if there is none), for non-decreasing
// a: 32 probes at a time, one a lane. The whole warp calls it.
__device__ __forceinline__ int last_at_or_before(const int32_t *a, int n, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0;
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int at = lane * step;
    const bool le = at < n && __ldg(a + lo + at) <= t;
    const int k = max(__popc(__ballot_sync(0xffffffffu, le)) - 1, 0);
    lo += k * step;
    n = min(step, n - k * step);
  }
  return lo;
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }

// The larger absolute value of two bf16 in a word, as bf16 bits; not finite: 0.
__device__ __forceinline__ uint32_t finite_top(uint32_t w) {
  const uint32_t lo = w & 0x7fffu, hi = (w >> 16) & 0x7fffu;
  return max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u);
}

// 2^e, e as in the header comment, from the bf16 bits of the maximum: with
// amax = 1.f * 2^E, 1.f <= 1.75 fits 448 = 1.75 * 2^8 at e = E - 8.
__device__ __forceinline__ float block_scale(uint32_t amax) {
  const int e = static_cast<int>(amax >> 7) - 127 - 8 + ((amax & 127u) > 96u ? 1 : 0);
  return __uint_as_float(static_cast<uint32_t>(min(max(e, -120), 119) + 127) << 23);
}

__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
  return __half22float2(*reinterpret_cast<__half2 *>(&h));
}

__device__ __forceinline__ uint32_t rescale4(uint32_t codes, float by) {
  const float2 a = e4m3x2_to_float2(codes & 0xffffu), b = e4m3x2_to_float2(codes >> 16);
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(__fmul_rn(a.y, by)), "f"(__fmul_rn(a.x, by)));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(__fmul_rn(b.y, by)), "f"(__fmul_rn(b.x, by)));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// ----------------------------------------------------------------- store --

// CTA (x, y): the touched blocks whose first new row lies in rows
// [x * chunk, (x + 1) * chunk), for the (K or V, head) pairs y * teams_at_once ...
// 2 * Hkv - 1, kTeams / team of them, `team` half-warps each.
__global__ void __launch_bounds__(kThreads, 4) store_fp8_block_kernel(const Fp8BlockStoreArgs a, int chunk,
                                                                   int team) {
  __shared__ uint32_t s_top[2][kTeams];
  const int lane = threadIdx.x & 31, sub = lane & 15;
  const int half = threadIdx.x >> 4;             // this thread's half-warp
  const int member = half & (team - 1);          // team is a power of two
  const int pair = blockIdx.y * (kTeams / team) + half / team;
  const bool active = pair < 2 * a.num_kv_heads;
  const bool is_v = active && pair >= a.num_kv_heads;
  const int head = !active ? 0 : is_v ? pair - a.num_kv_heads : pair;
  const __nv_bfloat16 *src = (is_v ? a.value : a.key) + head * 128 + sub * 8;
  const int64_t stride = is_v ? a.value_stride : a.key_stride;
  uint8_t *cache = is_v ? a.v_cache : a.k_cache;
  float *scales = is_v ? a.v_scales : a.k_scales;
  const bool reports = threadIdx.x == 0 && blockIdx.y == 0;
  const int bs = a.block_size;
  const int64_t cap = static_cast<int64_t>(a.max_blocks_per_seq) * bs;

  int t = blockIdx.x * chunk;                     // the launcher keeps this below total_q
  const int t_end = t + min(chunk, a.total_q - t);
  // a round of one token a sequence: row t is sequence t's
  int seq;
  if (t < a.num_seqs && __ldg(a.cu_seqlens_q + t) == t && __ldg(a.cu_seqlens_q + t + 1) == t + 1)
    seq = t;
  else
    seq = last_at_or_before(a.cu_seqlens_q, a.num_seqs, t);
  int units = 0;                                  // every thread of the CTA counts the same
  for (; seq < a.num_seqs && t < t_end; ++seq) {
    const int q0 = __ldg(a.cu_seqlens_q + seq), q1 = __ldg(a.cu_seqlens_q + seq + 1);
    const int ctx = __ldg(a.context_lens + seq);
    if (q0 < 0 || q1 < q0 || q1 > a.total_q || ctx < q1 - q0 || ctx > cap) {
      if (reports) raise_error(a.err, PKV_DEVERR_LENGTH);
      continue;
    }
    const int start = ctx - (q1 - q0);            // position of the sequence's first new row
    if (t < q0) t = q0;
    // row and block of the position of row t; behind the first row, on to the next block's first
    int blk = (start + (t - q0)) / bs, off0 = (start + (t - q0)) - blk * bs;
    if (t > q0 && off0 > 0) {
      t = bs - off0 < q1 - t ? t + (bs - off0) : q1;
      ++blk;
      off0 = 0;
    }
    for (; t < q1 && t < t_end; ++units, ++blk, off0 = 0) {
      const int n = min(bs - off0, q1 - t);
      const int id = __ldg(a.block_tables + static_cast<int64_t>(seq) * a.max_blocks_per_seq + blk);
      // new row r of the unit: row t + r of the call, row off0 + r of the block
      const __nv_bfloat16 *row = src + t * stride;
      uint4 held[kHold];
#pragma unroll
      for (int i = 0; i < kHold; ++i) {
        const int r = member + i * team;
        held[i] = active && r < n ? __ldg(reinterpret_cast<const uint4 *>(row + r * stride)) : make_uint4(0, 0, 0, 0);
      }
      const bool good = id >= 0 && id < a.num_blocks;
      if (!good && reports) raise_error(a.err, PKV_DEVERR_BLOCK_ID);
      const bool mine = active && good;
      float *scale_at = scales + static_cast<int64_t>(good ? id : 0) * a.num_kv_heads + head;
      float old = 0.f;
      if (off0 > 0 && mine && sub == 0) old = *scale_at;
      old = __shfl_sync(0xffffffffu, old, lane & 16);
      // the maximum: of the absolute bits, and once more without what is not finite
      // where that is among them
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < kHold; ++i)
        top = max_u16x2(top, max_u16x2(max_u16x2(held[i].x & 0x7fff7fffu, held[i].y & 0x7fff7fffu),
                                       max_u16x2(held[i].z & 0x7fff7fffu, held[i].w & 0x7fff7fffu)));
      top = max(top & 0xffffu, top >> 16);
      if (top >= 0x7f80u) {
        top = 0;
#pragma unroll
        for (int i = 0; i < kHold; ++i)
          top = max(max(max(finite_top(held[i].x), finite_top(held[i].y)),
                        max(finite_top(held[i].z), finite_top(held[i].w))), top);
      }
      for (int r = member + kHold * team; r < n && mine; r += team) {
        const uint4 v = __ldg(reinterpret_cast<const uint4 *>(row + r * stride));
        top = max(max(max(finite_top(v.x), finite_top(v.y)), max(finite_top(v.z), finite_top(v.w))), top);
      }
      __syncwarp();
#pragma unroll
      for (int x = 8; x >= 1; x >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, x));
      if (team > 1) {                             // one buffer is free again when the other's barrier is passed
        uint32_t *buf = s_top[units & 1];
        if (sub == 0) buf[half] = top;
        __syncthreads();
        for (int m = 0; m < team; ++m) top = max(top, buf[half - member + m]);
      }
      float now = block_scale(top);
      if (off0 > 0) now = fmaxf(now, old);
      const float inv = 1.f / now;                // exact for a power of two
      if (mine) {
        uint8_t *dst = cache + ((static_cast<int64_t>(id) * bs + off0) * a.num_kv_heads + head) * kRowBytes + sub * 8;
        const int64_t step = static_cast<int64_t>(a.num_kv_heads) * kRowBytes;   // next row of the block
#pragma unroll
        for (int i = 0; i < kHold; ++i) {
          const int r = member + i * team;
          if (r < n)
            *reinterpret_cast<uint2 *>(dst + r * step) =
                make_uint2(quantize4_e4m3(make_uint2(held[i].x, held[i].y), inv),
                           quantize4_e4m3(make_uint2(held[i].z, held[i].w), inv));
        }
        for (int r = member + kHold * team; r < n; r += team) {
          const uint4 v = __ldg(reinterpret_cast<const uint4 *>(row + r * stride));
          *reinterpret_cast<uint2 *>(dst + r * step) = make_uint2(quantize4_e4m3(make_uint2(v.x, v.y), inv),
                                                                  quantize4_e4m3(make_uint2(v.z, v.w), inv));
        }
        if (off0 > 0 && now != old) {
          const float by = old * inv;
          uint8_t *older = dst - off0 * step;
          for (int r = member; r < off0; r += 4 * team) {
            uint2 c[4];                           // on their way together
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (r + i * team < off0) c[i] = *reinterpret_cast<const uint2 *>(older + (r + i * team) * step);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (r + i * team < off0)
                *reinterpret_cast<uint2 *>(older + (r + i * team) * step) =
                    make_uint2(rescale4(c[i].x, by), rescale4(c[i].y, by));
          }
        }
        if (member == 0 && sub == 0) *scale_at = now;
      }
      t += n;
    }
  }
}

// ------------------------------------------------------------------ load --

constexpr int kLoadRows = 16;    // output rows of a CTA
constexpr int kLoadItems = 4;    // 16-code pieces a thread has in flight

// Rows [16 x, 16 x + 16) of the output: sequence i has the rows
// [row_starts[i], row_starts[i] + context_lens[i]), in position order.
__global__ void __launch_bounds__(kThreads) load_fp8_block_kernel(const Fp8BlockLoadArgs a) {
  __shared__ int s_id[kLoadRows], s_off[kLoadRows];
  const int bs = a.block_size;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * kLoadRows;
  const int64_t cap = static_cast<int64_t>(a.max_blocks_per_seq) * bs;
  if (threadIdx.x < 32) {
    const int first = last_at_or_before(a.row_starts, a.num_seqs, row0);
    if (threadIdx.x < kLoadRows) {
      const int64_t row = row0 + threadIdx.x;
      int i = first;
      while (i + 1 < a.num_seqs && __ldg(a.row_starts + i + 1) <= row) ++i;
      const int64_t pos = row - __ldg(a.row_starts + i), ctx = __ldg(a.context_lens + i);
      int id = -1;
      if (row < a.num_rows && pos >= 0 && pos < ctx && ctx <= cap) {
        id = __ldg(a.block_tables + static_cast<int64_t>(i) * a.max_blocks_per_seq + pos / bs);
        if (id < 0 || id >= a.num_blocks) {
          raise_error(a.err, PKV_DEVERR_BLOCK_ID);
          id = -1;
        }
      }
      s_id[threadIdx.x] = id;
      s_off[threadIdx.x] = static_cast<int>(pos % bs);
    }
  } else if (blockIdx.x == 0) {
    // every length once, whichever rows the call has of its sequence
    for (int i = threadIdx.x - 32; i < a.num_seqs; i += kThreads - 32) {
      const int ctx = __ldg(a.context_lens + i);
      if (ctx < 0 || ctx > cap) raise_error(a.err, PKV_DEVERR_LENGTH);
    }
  }
  __syncthreads();
  // pieces of 16 codes: 8 to a head's row, then the heads of K and of V, then the rows
  const int per_row = 2 * a.num_kv_heads * 8;
  const int pieces = kLoadRows * per_row;
  for (int base = threadIdx.x; base < pieces; base += kThreads * kLoadItems) {
    uint4 codes[kLoadItems];
    float scale[kLoadItems];
    __nv_bfloat16 *dst[kLoadItems];
#pragma unroll
    for (int u = 0; u < kLoadItems; ++u) {
      const int p = base + u * kThreads;
      dst[u] = nullptr;
      if (p < pieces) {
        const int r = p / per_row, in_row = p - r * per_row;
        const int pair = in_row >> 3, sub = in_row & 7;
        const int id = s_id[r];
        if (id >= 0) {
          const bool is_v = pair >= a.num_kv_heads;
          const int head = is_v ? pair - a.num_kv_heads : pair;
          const uint8_t *src = (is_v ? a.v_cache : a.k_cache) +
                               ((static_cast<int64_t>(id) * bs + s_off[r]) * a.num_kv_heads + head) * kRowBytes;
          codes[u] = __ldg(reinterpret_cast<const uint4 *>(src) + sub);
          scale[u] = __ldg((is_v ? a.v_scales : a.k_scales) + static_cast<int64_t>(id) * a.num_kv_heads + head);
          dst[u] = (is_v ? a.value_out + (row0 + r) * a.value_stride : a.key_out + (row0 + r) * a.key_stride) +
                   head * 128 + sub * 16;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kLoadItems; ++u) {
      if (dst[u] == nullptr) continue;
      const uint32_t w[4] = {codes[u].x, codes[u].y, codes[u].z, codes[u].w};
      uint32_t o[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 lo = e4m3x2_to_float2(w[i] & 0xffffu), hi = e4m3x2_to_float2(w[i] >> 16);
        o[2 * i] = float2_to_bf16x2(__fmul_rn(lo.x, scale[u]), __fmul_rn(lo.y, scale[u]));
        o[2 * i + 1] = float2_to_bf16x2(__fmul_rn(hi.x, scale[u]), __fmul_rn(hi.y, scale[u]));
      }
      uint4 *d = reinterpret_cast<uint4 *>(dst[u]);
      d[0] = make_uint4(o[0], o[1], o[2], o[3]);
      d[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
  }
}

}  // namespace

cudaError_t launch_store_fp8_block(const Fp8BlockStoreArgs &a, cudaStream_t stream) {
  // From the average of new tokens a sequence: rows a CTA looks for first rows in,
  // and half-warps a (block, head) is spread over, so that a full block's rows stay
  // in registers between the maximum and the codes. The average is wrong for a long
  // chunk among single tokens: 500 of them and one of 2048 take 16.7 us at block 16 and
  // 203 at block 256, where the same rows as five chunks take 7.8 and 17.4.
  const int avg = (a.total_q - 1) / a.num_seqs + 1;
  const int rows = avg < a.block_size ? avg : a.block_size;
  int team = 1;
  while (team < kTeams && team * kHold < rows) team *= 2;
  const int at_once = kTeams / team;
  const dim3 grid(static_cast<unsigned>((a.total_q - 1) / rows + 1),
                  static_cast<unsigned>((2 * a.num_kv_heads + at_once - 1) / at_once));
  store_fp8_block_kernel<<<grid, kThreads, 0, stream>>>(a, rows, team);
  return cudaGetLastError();
}

cudaError_t launch_load_fp8_block(const Fp8BlockLoadArgs &a, cudaStream_t stream) {
  load_fp8_block_kernel<<<static_cast<unsigned>((a.num_rows - 1) / kLoadRows + 1), kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace pkv
