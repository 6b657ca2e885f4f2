// tree_decode.cu -- attention of drafted token trees over the paged cache.
//
// Sequence i brings T_i drafted tokens (rows cu_seqlens_q[i] ..) whose K and V
// are given beside the cache. Row t, query head g sees every cached position
// p < context_lens[i] and the drafted tokens u whose bit is set in row t of
// tree_mask:
//   out = sum_x softmax_x(scale * q . K_x) V_x   over those x; zero when there
// are none. One warp per (row, query head), an online softmax over one key at
// a time; each lane holds four of the 128 dims.
#include <cuda_runtime.h>
#include <math.h>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kHD = 128;
constexpr int kWarps = 4;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float4 load4(const void *row, int lane) {
  const uint2 w = reinterpret_cast<const uint2 *>(row)[lane];
  const float2 a = bf16x2_to_float2(w.x), b = bf16x2_to_float2(w.y);
  return make_float4(a.x, a.y, b.x, b.y);
}

__global__ void __launch_bounds__(kWarps * 32) tree_decode_kernel(const TreeDecodeArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t gw = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int row = static_cast<int>(gw / a.num_q_heads);
  const int g = static_cast<int>(gw % a.num_q_heads);
  if (row >= a.total_q || row >= a.cu_seqlens_q[a.num_seqs]) return;
  int lo = 0, hi = a.num_seqs - 1;  // last sequence that starts at or before the row
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.cu_seqlens_q[mid] <= row) lo = mid; else hi = mid - 1;
  }
  const int first = a.cu_seqlens_q[lo], n = a.cu_seqlens_q[lo + 1] - first;
  const int ctx = a.context_lens[lo];
  if (first < 0 || n > a.max_seqlen_q || row >= first + n || first + n > a.total_q || ctx < 0 ||
      ctx > a.max_context_len) {
    if (lane == 0) raise_error(a.err, PKV_DEVERR_LENGTH);
    return;
  }
  const int h = g / (a.num_q_heads / a.num_kv_heads);
  const __nv_bfloat16 *qr = static_cast<const __nv_bfloat16 *>(a.q) +
                            (static_cast<int64_t>(row) * a.num_q_heads + g) * kHD;
  const float4 q = load4(qr, lane);
  const float c = a.scale * kLog2e;
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  auto take = [&](const __nv_bfloat16 *k, const __nv_bfloat16 *v) {
    const float4 kk = load4(k, lane), vv = load4(v, lane);
    float s = q.x * kk.x + q.y * kk.y + q.z * kk.z + q.w * kk.w;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    s *= c;
    const float mn = fmaxf(m, s);
    const float al = m == mn ? 1.f : exp2f(m - mn), p = exp2f(s - mn);
    m = mn;
    l = l * al + p;
    o.x = o.x * al + p * vv.x;
    o.y = o.y * al + p * vv.y;
    o.z = o.z * al + p * vv.z;
    o.w = o.w * al + p * vv.w;
  };
  const __nv_bfloat16 *kc = static_cast<const __nv_bfloat16 *>(a.k_cache);
  const __nv_bfloat16 *vc = static_cast<const __nv_bfloat16 *>(a.v_cache);
  for (int p = 0; p < ctx; ++p) {
    const int blk = a.block_tables[static_cast<int64_t>(lo) * a.max_blocks_per_seq + p / a.block_size];
    if (blk < 0 || blk >= a.num_blocks) {
      if (lane == 0) raise_error(a.err, PKV_DEVERR_BLOCK_ID);
      continue;
    }
    const int64_t at = ((static_cast<int64_t>(blk) * a.block_size + p % a.block_size) *
                        a.num_kv_heads + h) * kHD;
    take(kc + at, vc + at);
  }
  for (int u = 0; u < n; ++u) {
    const uint32_t word = a.tree_mask[static_cast<int64_t>(row) * a.mask_words + (u >> 5)];
    if ((word >> (u & 31)) & 1u)
      take(static_cast<const __nv_bfloat16 *>(a.key) + (first + u) * a.key_stride + h * kHD,
           static_cast<const __nv_bfloat16 *>(a.value) + (first + u) * a.value_stride + h * kHD);
  }
  const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
  uint2 w;
  w.x = float2_to_bf16x2(o.x * inv, o.y * inv);
  w.y = float2_to_bf16x2(o.z * inv, o.w * inv);
  reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) +
                            (static_cast<int64_t>(row) * a.num_q_heads + g) * kHD)[lane] = w;
}

}  // namespace

bool tree_decode_supported(int num_q_heads, int num_kv_heads) {
  return num_q_heads % num_kv_heads == 0 && num_q_heads / num_kv_heads <= 16;
}

size_t tree_decode_workspace_bytes(int max_seqlen_q, int num_q_heads, int num_kv_heads) {
  (void)max_seqlen_q;
  (void)num_q_heads;
  (void)num_kv_heads;
  return 256;
}

cudaError_t launch_tree_decode(const TreeDecodeArgs &a, cudaStream_t stream) {
  const int64_t warps = static_cast<int64_t>(a.total_q) * a.num_q_heads;
  tree_decode_kernel<<<static_cast<unsigned>((warps + kWarps - 1) / kWarps), kWarps * 32, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace pkv
