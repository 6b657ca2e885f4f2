// slots.cu -- a round's index arrays built on the GPU: block tables, slot map,
// positions and prefix sums from request lengths (pkv_plan_slots), and the
// ancestor masks of drafted trees from their parent links (pkv_tree_masks).
//
// With ctx_i cached and n_i new tokens, request i needs ceil((ctx_i + n_i) / bs)
// blocks and has ceil(ctx_i / bs); the missing ones are taken from the free
// list in request order, and token j goes to position p = ctx_i + j, slot
// table[i][p / bs] * bs + p % bs (LLM Infra 101 v0.5, KV Block Manager: FIFO
// free list; Mini-SGLang 源码解析（二）§6.7-6.8: page table, flat index).
//
// A few kilobytes move, so what counts is latency: one launch, no exchange
// between CTAs. Every CTA computes the prefix sums over all requests itself
// and takes its own 1024 tokens. A new block's id is read from the free list,
// not from the table, and the token that starts the block writes it to the
// table, so no CTA reads what another one writes. Measured: 5.4 us for 512 requests of
// one token, 5.2 us for 32 of 512 (17 CTAs); the bytes would take 0.1 us. It is the chain
// lengths -> three block scans -> binary search -> table entry -> store.
#include <cuda_runtime.h>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kThreads = 1024;

// Exclusive prefix sum over the CTA of one value a thread; *total gets the sum.
// Two barriers; `part` is 32 entries of shared memory, free again on return.
__device__ long long block_exclusive(long long v, long long *part, long long *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long inc = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, inc, off);
    if (lane >= off) inc += o;
  }
  if (lane == 31) part[warp] = inc;
  __syncthreads();
  const long long w = part[lane];
  long long winc = w;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, winc, off);
    if (lane >= off) winc += o;
  }
  *total = __shfl_sync(0xffffffffu, winc, 31);
  const long long before = __shfl_sync(0xffffffffu, winc - w, warp);
  __syncthreads();
  return before + inc - v;
}

__global__ void __launch_bounds__(kThreads) plan_slots_kernel(const PlanSlotsArgs a) {
  __shared__ long long part[32];
  // first row, cached tokens, owned blocks and place in the free list of the
  // chunk's requests
  __shared__ int s_row[kThreads + 1], s_ctx[kThreads], s_have[kThreads], s_take[kThreads];
  const int tid = threadIdx.x;
  const long long t = static_cast<long long>(blockIdx.x) * kThreads + tid;  // this thread's row
  const bool writes = blockIdx.x == 0;
  const int bs = a.block_size;
  const long long cap = static_cast<long long>(a.max_blocks_per_seq) * bs;
  const int cursor_in = __ldg(a.free_cursor);
  const int cursor = min(max(cursor_in, 0), a.num_free);
  if (writes && tid == 0 && cursor != cursor_in) raise_error(a.err, PKV_DEVERR_NO_BLOCKS);
  long long rows = 0, keys = 0, taken = 0;  // sums over the requests before the chunk
  bool placed = false;
  for (int base = 0; base < a.num_seqs; base += kThreads) {
    const int i = base + tid;
    long long ctx = 0, n = 0;
    uint32_t bad = 0;
    if (i < a.num_seqs) {
      ctx = __ldg(a.context_lens + i);
      n = __ldg(a.new_lens + i);
      if (ctx < 0 || ctx > cap || n < 0) bad = PKV_DEVERR_LENGTH;
      ctx = min(max(ctx, 0ll), cap);
      n = max(n, 0ll);
      if (n > cap - ctx) {
        bad = PKV_DEVERR_LENGTH;
        n = cap - ctx;
      }
    }
    long long sum;
    long long row = rows + block_exclusive(n, part, &sum);
    // rows past the last one the caller has room for are cut
    const long long end = min(row + n, static_cast<long long>(a.max_tokens));
    if (row + n > a.max_tokens) bad |= n > 0 ? PKV_DEVERR_LENGTH : 0u;
    row = min(row, static_cast<long long>(a.max_tokens));
    n = end - row;
    rows = min(rows + sum, static_cast<long long>(a.max_tokens));
    const int have = static_cast<int>((ctx + bs - 1) / bs);
    const int fresh = static_cast<int>((ctx + n + bs - 1) / bs) - have;
    long long sum_keys, sum_fresh;
    const long long key = keys + block_exclusive(ctx + n, part, &sum_keys);
    const long long take = taken + block_exclusive(fresh, part, &sum_fresh);
    keys += sum_keys;
    taken += sum_fresh;
    if (writes && i < a.num_seqs) {
      if (key + ctx + n > 0x7fffffffll) bad |= PKV_DEVERR_LENGTH;
      if (cursor + take + fresh > a.num_free) bad |= PKV_DEVERR_NO_BLOCKS;
      if (bad) raise_error(a.err, bad);
      a.cu_seqlens_q[i + 1] = static_cast<int>(end);
      a.cu_seqlens_k[i + 1] = static_cast<int>(min(key + ctx + n, 0x7fffffffll));
      a.context_out[i] = static_cast<int>(ctx + n);
    }
    s_row[tid] = static_cast<int>(row);
    s_ctx[tid] = static_cast<int>(ctx);
    s_have[tid] = have;
    s_take[tid] = static_cast<int>(min(take, 0x7fffffffll));
    if (tid == kThreads - 1) s_row[kThreads] = static_cast<int>(end);
    __syncthreads();
    if (!placed && t >= s_row[0] && t < s_row[kThreads]) {
      // the request of row t: the last one of the chunk that starts at or before it
      int lo = 0, hi = min(kThreads, a.num_seqs - base) - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_row[mid] <= t) lo = mid; else hi = mid - 1;
      }
      placed = true;
      const int pos = s_ctx[lo] + static_cast<int>(t - s_row[lo]);
      const int blk = pos / bs, off = pos - blk * bs;
      int32_t *entry = a.block_tables + static_cast<int64_t>(base + lo) * a.max_blocks_per_seq + blk;
      int id = -1;
      if (blk < s_have[lo]) {
        id = *entry;
        if (id < 0 || id >= a.num_blocks) {
          raise_error(a.err, PKV_DEVERR_BLOCK_ID);
          id = -1;
        }
      } else {
        const long long at = static_cast<long long>(cursor) + s_take[lo] + (blk - s_have[lo]);
        if (at < a.num_free) {
          id = __ldg(a.free_blocks + at);
          if (id < 0 || id >= a.num_blocks) {
            raise_error(a.err, PKV_DEVERR_BLOCK_ID);
            id = -1;
          }
        }
        if (off == 0) *entry = id;
      }
      a.slot_mapping[t] = id < 0 ? -1 : id * bs + off;
      a.positions[t] = pos;
    }
    __syncthreads();
  }
  if (!placed && t < a.max_tokens) {  // rows behind the last request
    a.slot_mapping[t] = -1;
    a.positions[t] = 0;
  }
  if (writes && tid == 0) {
    a.cu_seqlens_q[0] = 0;
    a.cu_seqlens_k[0] = 0;
    *a.cursor_out = static_cast<int>(min(cursor + taken, static_cast<long long>(a.num_free)));
  }
}

constexpr int kNodes = 128;          // nodes a CTA handles, one a thread
constexpr int kStagedParents = 1024;

// Row t of a tree's mask has the bits of t and all its ancestors. Parents come
// before their children, so the walk from t to the root meets falling indices:
// each word of the row is complete when the walk leaves it, and is written once.
// Measured: 4.3 us for one tree of 64 nodes, 4.7 us for 512 of up to 64, the latency of
// the launch, the links' load and the walk through shared memory.
__global__ void __launch_bounds__(kNodes) tree_masks_kernel(const TreeMasksArgs a) {
  __shared__ int s_parent[kStagedParents];
  const int seq = blockIdx.x;
  const int first = __ldg(a.cu_seqlens_q + seq);
  const int n = __ldg(a.cu_seqlens_q + seq + 1) - first;
  if (first < 0 || n < 0 || n > a.max_seqlen_q || n > a.total_q - first) {
    if (threadIdx.x == 0) raise_error(a.err, PKV_DEVERR_LENGTH);
    return;
  }
  const int t0 = blockIdx.y * kNodes;
  if (t0 >= n) return;
  // a link that does not point back (or to the root, -1) counts as the root
  auto link = [&](int u) {
    const int p = __ldg(a.parents + first + u);
    if (p < -1 || p >= u) {
      raise_error(a.err, PKV_DEVERR_TREE);
      return -1;
    }
    return p;
  };
  const int staged = min(min(n, t0 + kNodes), kStagedParents);
  for (int u = threadIdx.x; u < staged; u += kNodes) s_parent[u] = link(u);
  __syncthreads();
  const int t = t0 + threadIdx.x;
  if (t >= n) return;
  auto parent = [&](int u) { return u < staged ? s_parent[u] : link(u); };
  int32_t *row = a.tree_mask + static_cast<int64_t>(first + t) * a.mask_words;
  int word = t >> 5, depth = 0;
  uint32_t bits = 1u << (t & 31);
  for (int w = a.mask_words - 1; w > word; --w) row[w] = 0;
  for (int u = parent(t); u >= 0; u = parent(u)) {
    ++depth;
    if ((u >> 5) != word) {
      row[word] = static_cast<int32_t>(bits);
      bits = 0u;
      for (--word; word > (u >> 5); --word) row[word] = 0;
    }
    bits |= 1u << (u & 31);
  }
  row[word] = static_cast<int32_t>(bits);
  for (--word; word >= 0; --word) row[word] = 0;
  a.positions[first + t] = __ldg(a.context_lens + seq) + depth;
}

}  // namespace

cudaError_t launch_plan_slots(const PlanSlotsArgs &a, cudaStream_t stream) {
  const unsigned grid = a.max_tokens > kThreads ? (a.max_tokens - 1) / kThreads + 1 : 1;
  plan_slots_kernel<<<grid, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_tree_masks(const TreeMasksArgs &a, cudaStream_t stream) {
  const dim3 grid(a.num_seqs, (a.max_seqlen_q + kNodes - 1) / kNodes);
  tree_masks_kernel<<<grid, kNodes, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace pkv
