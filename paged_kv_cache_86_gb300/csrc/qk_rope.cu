// qk_rope.cu -- head norm and position rotation of a step's queries and keys,
// in the pass that also writes the keys and values to their cache slots.
//
// For every token t and head row x of D values (query heads with q_weight, key
// heads with k_weight):
//   y  = x * rsqrt(mean(x^2) + eps) * w            (skipped when the weight is absent)
//   y' = y with each pair (a, b) turned by the token's angle row:
//        a' = a cos_i - b sin_i,  b' = b cos_i + a sin_i,  i < rotary_dim / 2
// where pair i is (i, i + rotary_dim/2) or, interleaved, (2i, 2i + 1), and dims
// from rotary_dim on pass through. All of it is fp32 with one rounding to bf16
// at the end; the value rows of the storing variant move bit for bit.
//
// Bound by HBM: each row is read once and written once (the angle row, 4 *
// rotary_dim bytes a token, is shared by all its heads). A row belongs to D/16
// neighbouring lanes and each lane holds the two 8-value chunks whose dims turn
// into one another (chunk l and chunk l + rotary_dim/16), so the turn needs no
// exchange between lanes, the sum of squares log2(D/16) shuffles, and every
// access is 16 bytes. A warp stays with one token, so the angles are loaded
// once and serve all the rows it handles.
//
// Measured, 32 / 8 heads of 128 with the store: 16384 tokens 69.2 us = 5.9 TB/s (its
// 411 MB at 6.78 TB/s: 60.6 us), 512 tokens 4.1 us, 8 tokens 2.5 us (the launch). What
// counts is warps in flight: 28 an SM (72 registers) took 74.5 us, 24 85; the next row
// loaded ahead costs registers and took 92. Stores that evict first save 3 us more but
// evict what the next kernel reads.
#include <cuda_runtime.h>

#include <algorithm>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kWarps = 4;

struct Chunk {
  float v[8];
};

__device__ __forceinline__ Chunk unpack(uint4 r) {
  Chunk c;
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = bf16x2_to_float2(w[i]);
    c.v[2 * i] = f.x;
    c.v[2 * i + 1] = f.y;
  }
  return c;
}

__device__ __forceinline__ uint4 pack(const Chunk &c) {
  return make_uint4(float2_to_bf16x2(c.v[0], c.v[1]), float2_to_bf16x2(c.v[2], c.v[3]),
                    float2_to_bf16x2(c.v[4], c.v[5]), float2_to_bf16x2(c.v[6], c.v[7]));
}

// kD: head_dim. kInter: interleaved pairs. kMany: the angles are read again for each row
// (from L1) instead of held in 16 registers, so that more warps an SM are
// resident: 36 instead of 32 (52 or 56 registers, 64; launch bounds that ask for as many
// give 56 and 63, and cost 1-2 % at 6000 and 12000 tokens).
template <int kD, bool kInter, bool kMany>
__global__ void __launch_bounds__(kWarps * 32) qk_rope_kernel(const QkRopeArgs a) {
  constexpr int kLanes = kD / 16;          // lanes of a row
  constexpr int kRows = 32 / kLanes;       // rows a warp handles at once
  const int lane = threadIdx.x & 31;
  const int64_t gw = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int64_t t = gw / a.parts;          // token
  const int part = static_cast<int>(gw - t * a.parts);
  if (t >= a.num_tokens) return;
  const int pos = __ldg(a.positions + t);
  if (pos < 0 || pos >= a.max_position) {
    if (lane == 0) raise_error(a.err, PKV_DEVERR_LENGTH);
    return;
  }
  int64_t slot = t;                        // row of the key (and value) output
  if (a.slot_mapping != nullptr) {
    slot = __ldg(a.slot_mapping + t);
    if (slot >= a.num_slots) {
      if (lane == 0) raise_error(a.err, PKV_DEVERR_SLOT);
      slot = -1;
    }
  }
  const int l = lane % kLanes, sub = lane / kLanes;
  const int turn = a.rotary_dim / 16;      // lanes whose two chunks turn
  // the lane's two chunks of 8 values, in elements of the row
  const int c0 = (l < turn ? l : 2 * l) * 8;
  const int c1 = l < turn ? c0 + turn * 8 : c0 + 8;
  const float *angles = a.cos_sin + static_cast<int64_t>(pos) * a.rotary_dim;
  float cs[8], sn[8];
  auto load_angles = [&]() {
    const int half = a.rotary_dim / 2;
    // neox: pair i is (c0 + i, c1 + i); interleaved: pairs c0/2 + 0..3 and c1/2 + 0..3
    const int p0 = kInter ? c0 / 2 : c0, p1 = kInter ? c1 / 2 : c0 + 4;
    *reinterpret_cast<float4 *>(cs) = __ldg(reinterpret_cast<const float4 *>(angles + p0));
    *reinterpret_cast<float4 *>(cs + 4) = __ldg(reinterpret_cast<const float4 *>(angles + p1));
    *reinterpret_cast<float4 *>(sn) = __ldg(reinterpret_cast<const float4 *>(angles + half + p0));
    *reinterpret_cast<float4 *>(sn + 4) =
        __ldg(reinterpret_cast<const float4 *>(angles + half + p1));
  };
  if (!kMany && l < turn) load_angles();
  // the lanes of this lane's row
  const unsigned row_lanes = ((1u << kLanes) - 1u) << (sub * kLanes);
  const int heads = a.num_q_heads + a.num_kv_heads;
  const int rows = heads + (a.v != nullptr ? a.num_kv_heads : 0);
  for (int r0 = part * kRows; r0 < rows; r0 += a.parts * kRows) {
    const int r = r0 + sub;
    const __nv_bfloat16 *src = nullptr, *w = nullptr;
    __nv_bfloat16 *dst = nullptr;
    if (r < a.num_q_heads) {
      src = a.q + t * a.q_stride + r * kD;
      dst = a.q_out + t * a.q_out_stride + r * kD;
      w = a.q_weight;
    } else if (r < heads) {
      const int h = r - a.num_q_heads;
      src = a.k + t * a.k_stride + h * kD;
      if (slot >= 0) dst = a.k_out + slot * a.k_out_stride + h * kD;
      w = a.k_weight;
    } else if (r < rows) {
      const int h = r - heads;
      src = a.v + t * a.v_stride + h * kD;
      if (slot >= 0) dst = a.v_out + slot * a.k_out_stride + h * kD;
    }
    uint4 x0 = make_uint4(0u, 0u, 0u, 0u), x1 = x0;
    if (dst != nullptr) {
      x0 = *reinterpret_cast<const uint4 *>(src + c0);
      x1 = *reinterpret_cast<const uint4 *>(src + c1);
    }
    if (dst == nullptr) continue;
    if (r >= heads || (w == nullptr && l >= turn)) {   // bit for bit
      *reinterpret_cast<uint4 *>(dst + c0) = x0;
      *reinterpret_cast<uint4 *>(dst + c1) = x1;
      continue;
    }
    Chunk u = unpack(x0), z = unpack(x1);
    if (w != nullptr) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss += u.v[i] * u.v[i] + z.v[i] * z.v[i];
#pragma unroll
      for (int off = kLanes / 2; off >= 1; off >>= 1) ss += __shfl_xor_sync(row_lanes, ss, off);
      const float inv = rsqrtf(ss * (1.f / kD) + a.eps);
      const Chunk w0 = unpack(__ldg(reinterpret_cast<const uint4 *>(w + c0)));
      const Chunk w1 = unpack(__ldg(reinterpret_cast<const uint4 *>(w + c1)));
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        u.v[i] *= inv * w0.v[i];
        z.v[i] *= inv * w1.v[i];
      }
    }
    if (l < turn) {
      if (kMany) load_angles();
      if constexpr (kInter) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a0 = u.v[2 * i], b0 = u.v[2 * i + 1], a1 = z.v[2 * i], b1 = z.v[2 * i + 1];
          u.v[2 * i] = a0 * cs[i] - b0 * sn[i];
          u.v[2 * i + 1] = b0 * cs[i] + a0 * sn[i];
          z.v[2 * i] = a1 * cs[4 + i] - b1 * sn[4 + i];
          z.v[2 * i + 1] = b1 * cs[4 + i] + a1 * sn[4 + i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float p = u.v[i], s = z.v[i];
          u.v[i] = p * cs[i] - s * sn[i];
          z.v[i] = s * cs[i] + p * sn[i];
        }
      }
    }
    *reinterpret_cast<uint4 *>(dst + c0) = pack(u);
    *reinterpret_cast<uint4 *>(dst + c1) = pack(z);
  }
}

// Warps of an instance that an SM holds at once, 0 on an error.
template <int kD, bool kInter, bool kMany>
int resident() {
  static const int warps = [] {   // built for one architecture: the same on every device
    int ctas = 0;
    const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(
        &ctas, qk_rope_kernel<kD, kInter, kMany>, kWarps * 32, 0);
    return e == cudaSuccess ? ctas * kWarps : 0;
  }();
  return warps;
}

template <int kD>
int resident(bool interleaved, bool many) {
  return interleaved ? (many ? resident<kD, true, true>() : resident<kD, true, false>())
                     : (many ? resident<kD, false, true>() : resident<kD, false, false>());
}

template <int kD, bool kMany>
void launch(const QkRopeArgs &a, unsigned grid, cudaStream_t stream) {
  if (a.interleaved)
    qk_rope_kernel<kD, true, kMany><<<grid, kWarps * 32, 0, stream>>>(a);
  else
    qk_rope_kernel<kD, false, kMany><<<grid, kWarps * 32, 0, stream>>>(a);
}

template <int kD>
void launch(const QkRopeArgs &a, unsigned grid, bool many, cudaStream_t stream) {
  if (many)
    launch<kD, true>(a, grid, stream);
  else
    launch<kD, false>(a, grid, stream);
}

}  // namespace

cudaError_t launch_qk_rope(QkRopeArgs a, int head_dim, cudaStream_t stream) {
  if (a.num_tokens == 0) return cudaSuccess;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  auto held = [&](bool many) {   // warps that the GPU holds at once
    return int64_t(sm_count(dev)) * (head_dim == 64    ? resident<64>(a.interleaved, many)
                                     : head_dim == 128 ? resident<128>(a.interleaved, many)
                                                       : resident<256>(a.interleaved, many));
  };
  const int64_t want = held(false);
  if (want == 0) return cudaErrorInvalidDeviceFunction;
  // With few tokens a token's rows are spread over up to one warp a pass, until the
  // GPU holds no more; with many, a warp takes all the rows of its
  // token and loads its angles once. 32 / 8 heads, us at 8 / 512 / 1024 / 2048 / 16384
  // tokens, with 28 warps resident: 2.4 / 5.2 / 5.6 / 8.6 / 74.5; never spread 7.6 / 8.1 /
  // 8.8 / 10.7 / 74.5; always 2.4 / 5.2 / 7.2 / 11.9 / 115.6; up to 16 warps an SM 2.4 / 4.8 /
  // 6.8 / 10.7 / 74.6, up to 64 2.5 / 5.1 / 7.3 / 9.3 / 74.5.
  const int rows = a.num_q_heads + (a.v != nullptr ? 2 : 1) * a.num_kv_heads;
  const int passes = (rows + 512 / head_dim - 1) / (512 / head_dim);
  int64_t parts = want / a.num_tokens;
  parts = parts < 1 ? 1 : parts > passes ? passes : parts;
  // More tokens than resident warps: the last wave of warps may be nearly empty, so of one
  // warp a token, two, and one with kMany (more of them resident) the one is taken
  // whose waves cost least, by what a wave measured: 32 / 8 heads, us at 5200 / 6000 /
  // 8192 / 12000 / 16384 / 20000 tokens: one 31.8 / 34.0 / 38.7 / 54.9 / 72.6 / 88.2, two
  // 27.9 / 30.3 / 39.6 / 54.0 / 72.1 / 87.9, kMany 24.4 / 35.5 / 39.9 / 57.3 / 69.2 / 84.4. Few passes
  // are not divided: the angles would be loaded for too few rows. The costs are those of
  // 32 / 8 heads of 128. With them, of twelve shapes (head dims 64, 128 and 256, 2 / 1 to
  // 64 / 8 heads, with and without norm, store and interleaving) at 4900 to 32768 tokens the
  // choice is at most 4 % slower than one warp a token and 6 % slower than the best of the
  // three (8 / 2 heads of 256, 6000 tokens: 16.2, 15.3 by two); at 8 to 4096 tokens the
  // parts above are within 8 % of the best of 1, 2, 4, 8 and all.
  bool many = false;
  if (a.num_tokens > want) {
    auto waves = [](int64_t warps, int64_t resident) { return (warps + resident - 1) / resident; };
    const int64_t one = 200 * waves(a.num_tokens, want);
    const int64_t two = passes < 8 ? one : 103 * waves(2 * int64_t(a.num_tokens), want);
    const int64_t more = 229 * waves(a.num_tokens, std::max(want, held(true)));
    many = more < one && more <= two;
    if (!many && two < one) parts = 2;
  }
  a.parts = static_cast<int>(parts);
  const int64_t warps = static_cast<int64_t>(a.num_tokens) * a.parts;
  const unsigned grid = static_cast<unsigned>((warps + kWarps - 1) / kWarps);
  if (warps > (static_cast<int64_t>(1) << 33)) return cudaErrorInvalidValue;
  if (head_dim == 64) launch<64>(a, grid, many, stream);
  else if (head_dim == 128) launch<128>(a, grid, many, stream);
  else launch<256>(a, grid, many, stream);
  return cudaGetLastError();
}

}  // namespace pkv
