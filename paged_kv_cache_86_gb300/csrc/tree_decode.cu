// tree_decode.cu -- attention of drafted token trees over the paged cache, on
// the tcgen05 tensor cores (sm_103a).
//
// Sequence i brings T_i drafted tokens (rows cu_seqlens_q[i] ..) whose K and V
// are given beside the cache. Row t, query head g sees every cached position
// p < context_lens[i] and the drafted tokens u whose bit is set in row t of
// tree_mask; out = softmax(scale q.K) V over those, zero when there are none.
//
// Every cached K/V byte is needed once per call and serves T_i * G query rows
// (G query heads a KV head), at most 256 of which share one pass: 128 rows are
// 128 flops a byte, below the 282 the GPU has for each byte of HBM, so the
// kernel is bound by reading the cache and everything else has to hide behind
// that stream.
//
// Work. The rows of one KV head of a sequence form row groups of up to two
// 128-row MMA tiles (row = token * G + head of the group). A stream is one
// (KV head, sequence, row group); it is walked in tiles of 128 keys -- the
// cached ones, then the drafts, which share the last cached tile when they fit
// behind its keys. The flat space of all tiles, head-major, is cut into equal
// ranges, one per CTA (one CTA an SM). With 8 KV heads the ranges of different
// heads start at the same tokens, so the CTAs that read the eight 256-byte
// pieces of a token's row run side by side. A stream that a range boundary
// cuts leaves partial records (O, m, l) that tree_combine_kernel merges by the
// log-sum-exp rule.
//
// A CTA runs its tiles through two softmax warpgroups, x = 0 and 1, that
// alternate: an "op" is one key tile met by one MMA row tile, op g belongs to
// x = g & 1, and the tensor core issues PV(g - 2), S(g) for g = 0, 1, 2, ...
// across streams, so while one warpgroup computes its softmax the tensor core
// and the other one work.
//   * streams of one row tile (T_i * G <= 128): consecutive key tiles alternate
//     between the warpgroups, each with its own O, maximum and sum; at the end
//     the one with the last tile merges both, reading the other's O from TMEM.
//   * streams of two row tiles: every key tile is met by both; K and V are
//     loaded once.
// Accumulators S_0, S_1, O_0, O_1 fill the 512 TMEM columns; P is written as
// bf16 over S and is the A operand of the PV MMA from there. P is exp2 of fp32
// scores and enters the fp32 row sum before it is rounded; the one rounding of
// the weights to bf16 (2^-8 of each at most) is what the tensor core's operand
// type asks for. O is rescaled only when a row's maximum grows by over 2^8.
//
// Loads (warps 8 and 10): whole tiles of blocks that are a multiple of 8 rows
// by TMA boxes; partial tiles, other block sizes and the drafts by TMA row
// gathers (four rows an instruction), which put zeros where a tile has no key,
// so no stale cache row ever meets an MMA. Drafted V rows a query row must not
// see may hold anything: their values that are not finite are set to zero in
// shared memory and added back at the end for the rows that do see them.
//
// Every wait is bounded; on a timeout the CTA records PKV_DEVERR_TIMEOUT,
// drains its copies and MMAs, frees its TMEM and exits.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "pkv_tc.cuh"

namespace pkv {
namespace {

constexpr int kTile = 128;
constexpr int kHD = 128;
constexpr int kRegion = 16384;       // 128 rows x 64 dims, 128-byte swizzle
constexpr int kTileBytes = 2 * kRegion;
constexpr int kKStages = 3;
constexpr int kVStages = 2;
constexpr int kThreads = 384;        // softmax 0 (warps 0-3), softmax 1 (4-7), loaders + MMA (8-11)
constexpr int kWarpK = 8, kWarpMma = 9, kWarpV = 10;
// Registers: launched at 168 a thread; warpgroup 2 drops to 104 and the softmax
// warpgroups rise to 200, which adds up to the launch total again.
constexpr int kRegsLaunch = 168, kRegsLow = 104, kRegsHigh = 200;
static_assert(2 * 128 * kRegsHigh + 128 * kRegsLow == kThreads * kRegsLaunch,
              "setmaxnreg split must add up to the launch allocation");
constexpr int kTmemCols = 512;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescaleThreshold = 8.f;
constexpr int kSegRing = 4;
constexpr int kSegReaders = 1 + 1 + 8;   // V loader, MMA issuer, softmax warps

constexpr int kOffQ = 0;                                // two Q tiles
constexpr int kOffK = kOffQ + 2 * kTileBytes;
constexpr int kOffV = kOffK + kKStages * kTileBytes;
constexpr int kOffMl = kOffV + kVStages * kTileBytes;   // float2[128]
constexpr int kOffSeg = kOffMl + kTile * 8;
constexpr int kSegBytes = 64;
constexpr int kOffBar = kOffSeg + kSegRing * kSegBytes;
// q full/empty x2, k and v full/empty, s/p/pv/o_free x2, ml full/free, seg full/empty
constexpr int kNumBars = 4 + 2 * kKStages + 2 * kVStages + 8 + 2 + 2 * kSegRing;
constexpr int kOffMisc = kOffBar + kNumBars * 8;        // TMEM address, abort flag, start
constexpr int kSmemBytes = kOffMisc + 32 + 1024;        // the base is rounded up to 1024 bytes
static_assert(kSmemBytes <= 232448, "shared memory of one CTA");

// One CTA's part of one stream, handed from the K loader to the other roles.
struct Seg {
  int head;     // KV head; -1 ends the walk
  int ctx;      // cached tokens of the sequence
  int drafts;   // drafted tokens of the sequence
  int q0;       // its first drafted row
  int seq;
  int tok0;     // the row group's first token in the tree
  int ntok;     // its tokens
  int t0, t1;   // tiles of the stream
  int slot;     // partial record, -1: the whole stream is here
  int op0;      // first op
  int qtile;    // running number of its first Q tile
  int bad;      // set when a drafted V value was not finite
};
static_assert(sizeof(Seg) <= kSegBytes, "segment ring entry");

struct Boundary {   // what the combine needs about a stream cut at a CTA's range start
  int row0;         // first drafted row of its row group, -1: nothing to combine here
  int ntok;
  int head;
  int first;        // CTA of its first piece
  int last;         // CTA of its last piece
};

struct TreeParams {
  __nv_bfloat16 *out;
  const __nv_bfloat16 *value;
  int64_t value_stride;
  const int32_t *block_tables;
  int max_blocks_per_seq;
  const int32_t *context_lens;
  const int32_t *cu_q;
  const int32_t *tree_mask;
  int mask_words;
  int num_seqs;
  int total_q;
  int max_seqlen_q;
  int max_context_len;
  int num_q_heads;
  int num_kv_heads;
  int group;
  int box_tokens;    // tokens of a Q box: box_tokens * group rows, a multiple of 8
  int tile_tokens;   // tokens of an MMA row tile
  int block_size;
  int num_blocks;
  int box_rows;      // rows of a K/V box; 0: gathers only
  float scale_log2;  // |scale| * log2 e, or 1 with flip == 0
  float flip;        // 1, -1 (negative scale) or 0 (zero scale): factor of the raw scores
  int rows_cap;      // rows of a partial record
  float2 *ml;
  float *po;
  Boundary *bounds;
  uint32_t *err;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The keys of tile j of a stream: cached rows [128 j, 128 j + cached) in rows
// 0 .. of the tile, then drafts [u0, u0 + drafts) from row `at` (a multiple of
// 4) on; rows 0 .. rows - 1 are loaded (a multiple of 16).
struct TileKeys {
  int cached, at, u0, drafts, rows;
};

__device__ __forceinline__ int tree_tiles(int ctx, int drafts) {
  const int full = ctx / kTile, rem = ctx % kTile;
  if (((rem + 3) & ~3) + drafts <= kTile) return full + 1;
  return full + (rem > 0 ? 1 : 0) + (drafts + kTile - 1) / kTile;
}

__device__ __forceinline__ TileKeys tile_keys(int ctx, int drafts, int j) {
  const int full = ctx / kTile, rem = ctx % kTile, rem4 = (rem + 3) & ~3;
  TileKeys k;
  k.at = k.u0 = k.drafts = 0;
  k.cached = kTile;
  k.rows = kTile;
  if (j < full) return k;
  if (rem4 + drafts <= kTile) {
    k.cached = rem;
    k.at = rem4;
    k.drafts = drafts;
  } else if (rem > 0 && j == full) {
    k.cached = rem;
  } else {
    k.cached = 0;
    k.u0 = (j - full - (rem > 0 ? 1 : 0)) * kTile;
    k.drafts = min(kTile, drafts - k.u0);
  }
  k.rows = (max(k.cached, k.at + k.drafts) + 15) & ~15;
  return k;
}

__device__ __forceinline__ uint64_t desc_kmajor(uint32_t tile_base, int kk) {
  return smem_desc_sw128(tile_base + (kk >> 2) * kRegion + (kk & 3) * 32, 16, 1024);
}

// start-address increment (16-byte units) of K step kk of a K-major tile
__device__ __forceinline__ uint32_t kmajor_step(int kk) {
  return static_cast<uint32_t>(((kk >> 2) * kRegion + (kk & 3) * 32) >> 4);
}

__device__ __forceinline__ uint64_t desc_at(uint64_t d, uint32_t step) {
  return (d & 0xFFFFFFFF00000000ull) | static_cast<uint32_t>(static_cast<uint32_t>(d) + step);
}

__device__ __forceinline__ uint64_t desc_v_mnmajor(uint32_t tile_base) {
  return smem_desc_sw128(tile_base, kRegion, 1024);
}

// D[tmem] (+)= A[tmem] * B[smem desc], bf16 inputs, fp32 accumulator.
__device__ __forceinline__ void umma_bf16_tmem_a(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                                 uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      :: "r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate) : "memory");
}

__device__ __forceinline__ void tmem_st32_u(uint32_t taddr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};"
      :: "r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]),
         "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]),
         "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]),
         "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
         "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}

// Four rows r of a [rows, row_elems] array, 64 elements from column x on, to
// 4 x 128 bytes of shared memory (rows outside the array read as zero).
__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap *map, int x, int4 r,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5, %6}], [%7];"
      :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(r.x), "r"(r.y), "r"(r.z),
         "r"(r.w), "r"(bar)
      : "memory");
}

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, const volatile int *abort) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort));
}

// Lengths of sequence i, checked: drafts == 0 when there is nothing to do.
__device__ __forceinline__ bool seq_lengths(const TreeParams &p, int i, int *ctx, int *drafts,
                                            int *q0) {
  *q0 = __ldg(p.cu_q + i);
  const int end = __ldg(p.cu_q + i + 1);
  *ctx = __ldg(p.context_lens + i);
  *drafts = end - *q0;
  if (*q0 < 0 || end < *q0 || *drafts > p.max_seqlen_q || end > p.total_q || *ctx < 0 ||
      *ctx > p.max_context_len) {
    *drafts = 0;
    return false;
  }
  return true;
}

__global__ void __launch_bounds__(kThreads, 1)
tree_decode_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_kg,
                   const __grid_constant__ CUtensorMap tm_vg, const __grid_constant__ CUtensorMap tm_kd,
                   const __grid_constant__ CUtensorMap tm_vd, const TreeParams p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_addr(smem_raw);
  const uint32_t base = (raw_addr + 1023u) & ~1023u;
  uint8_t *smem = smem_raw + (base - raw_addr);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  // let the combine be scheduled early (it waits for this grid's end)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const uint32_t bar0 = base + kOffBar;
  auto q_full = [&](int s) { return bar0 + 8u * s; };
  auto q_empty = [&](int s) { return bar0 + 8u * (2 + s); };
  auto k_full = [&](int s) { return bar0 + 8u * (4 + s); };
  auto k_empty = [&](int s) { return bar0 + 8u * (4 + kKStages + s); };
  constexpr int kBv = 4 + 2 * kKStages;
  auto v_full = [&](int s) { return bar0 + 8u * (kBv + s); };
  auto v_empty = [&](int s) { return bar0 + 8u * (kBv + kVStages + s); };
  constexpr int kBx = kBv + 2 * kVStages;
  auto s_full = [&](int x) { return bar0 + 8u * (kBx + x); };
  auto p_full = [&](int x) { return bar0 + 8u * (kBx + 2 + x); };
  auto pv_done = [&](int x) { return bar0 + 8u * (kBx + 4 + x); };
  auto o_free = [&](int x) { return bar0 + 8u * (kBx + 6 + x); };
  const uint32_t ml_full = bar0 + 8u * (kBx + 8), ml_free = bar0 + 8u * (kBx + 9);
  auto seg_full = [&](int i) { return bar0 + 8u * (kBx + 10 + i); };
  auto seg_empty = [&](int i) { return bar0 + 8u * (kBx + 10 + kSegRing + i); };
  volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(smem + kOffMisc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + kOffMisc + 4);
  volatile int *start = reinterpret_cast<volatile int *>(smem + kOffMisc + 8);  // seq, tile, range, total
  float2 *ml_x = reinterpret_cast<float2 *>(smem + kOffMl);
  auto seg_at = [&](int i) {
    return reinterpret_cast<volatile Seg *>(smem + kOffSeg + (i % kSegRing) * kSegBytes);
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(q_full(s), 1);
      mbar_init(q_empty(s), 1);
      mbar_init(s_full(s), 1);
      mbar_init(p_full(s), 4);
      mbar_init(pv_done(s), 1);
      mbar_init(o_free(s), 4);
    }
    for (int s = 0; s < kKStages; ++s) {
      mbar_init(k_full(s), 1);
      mbar_init(k_empty(s), 1);
    }
    for (int s = 0; s < kVStages; ++s) {
      mbar_init(v_full(s), 1);
      mbar_init(v_empty(s), 1);
    }
    mbar_init(ml_full, 4);
    mbar_init(ml_free, 4);
    for (int i = 0; i < kSegRing; ++i) {
      mbar_init(seg_full(i), 1);
      mbar_init(seg_empty(i), kSegReaders);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kWarpMma) {
    tmem_alloc(smem_addr(const_cast<uint32_t *>(tmem_slot)), kTmemCols);
    tmem_relinquish();
  }

  // ---- the CTA's range: tiles of all sequences (one KV head), counted by every
  // CTA itself; thread t counts sequences [t * per, (t + 1) * per)
  const int pair_tokens = 2 * p.tile_tokens;
  const int per = (p.num_seqs + kThreads - 1) / kThreads;
  auto seq_cost = [&](int i, bool report) {
    int ctx, drafts, q0;
    if (!seq_lengths(p, i, &ctx, &drafts, &q0) && report) raise_error(p.err, PKV_DEVERR_LENGTH);
    return drafts == 0 ? 0 : tree_tiles(ctx, drafts) * ((drafts + pair_tokens - 1) / pair_tokens);
  };
  int mine = 0;
  for (int i = threadIdx.x * per; i < min(p.num_seqs, (static_cast<int>(threadIdx.x) + 1) * per); ++i)
    mine += seq_cost(i, blockIdx.x == 0);
  int inc = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, inc, off);
    if (lane >= off) inc += o;
  }
  int *part = reinterpret_cast<int *>(smem + kOffMl);
  if (lane == 31) part[warp] = inc;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  int before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    const int v = part[w];
    if (w < warp) before += v;
    total += v;
  }
  const int units = total * p.num_kv_heads;
  const int range = max(1, (units + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x));
  const long long lo64 = static_cast<long long>(blockIdx.x) * range;
  const int lo = lo64 < units ? static_cast<int>(lo64) : units;
  const int hi = static_cast<int>(min(lo64 + range, static_cast<long long>(units)));
  const int off0 = lo < hi ? lo % total : -1;   // the range starts at this tile of its head
  {
    int at = before + inc - mine;               // this thread's first tile
    if (off0 >= at && off0 < at + mine) {
      int i = threadIdx.x * per;
      for (;; ++i) {
        const int c = seq_cost(i, false);
        if (off0 < at + c) break;
        at += c;
      }
      start[0] = i;
      start[1] = off0 - at;
    }
  }
  __syncthreads();
  const uint32_t tmem = *tmem_slot;
  auto tmem_s = [&](int x) { return tmem + x * kTile; };           // P over columns 0..63
  auto tmem_o = [&](int x) { return tmem + (2 + x) * kTile; };
  const uint32_t sQ = base + kOffQ;
  auto sK = [&](int s) { return base + kOffK + s * kTileBytes; };
  auto sV = [&](int s) { return base + kOffV + s * kTileBytes; };
  auto fail = [&]() {
    *abort_flag = 1;
    raise_error(p.err, PKV_DEVERR_TIMEOUT);
  };
  // Segment n for a reader: copied out of the ring; false on a timeout. The ring
  // entry is given back by seg_done().
  auto read_seg = [&](int n, Seg &s, bool whole_warp) -> bool {
    const uint32_t par = (n / kSegRing) & 1;
    const bool got = whole_warp ? warp_wait(seg_full(n % kSegRing), par, abort_flag)
                                : mbar_wait(seg_full(n % kSegRing), par, abort_flag);
    if (!got) return false;
    const volatile Seg *v = seg_at(n);
    s.head = v->head;
    s.ctx = v->ctx;
    s.drafts = v->drafts;
    s.q0 = v->q0;
    s.seq = v->seq;
    s.tok0 = v->tok0;
    s.ntok = v->ntok;
    s.t0 = v->t0;
    s.t1 = v->t1;
    s.slot = v->slot;
    s.op0 = v->op0;
    s.qtile = v->qtile;
    return true;
  };
  auto seg_done = [&](int n, bool whole_warp) {
    if (whole_warp) __syncwarp();
    if (!whole_warp || lane == 0) mbar_arrive(seg_empty(n % kSegRing));
  };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kRegsLow));
    if (warp == kWarpK || warp == kWarpV) {
      // ------------------------------------------------------------- loaders
      const bool is_k = warp == kWarpK;
      const int stages = is_k ? kKStages : kVStages;
      const CUtensorMap *map_box = is_k ? &tm_k : &tm_v;
      const CUtensorMap *map_rows = is_k ? &tm_kg : &tm_vg;
      const CUtensorMap *map_draft = is_k ? &tm_kd : &tm_vd;
      const int oob_row = p.num_blocks * p.block_size;
      int issued = 0;
      bool ok = true;
      if (lane == 0) {
        tma_prefetch_desc(map_box);
        tma_prefetch_desc(map_rows);
        tma_prefetch_desc(map_draft);
        if (is_k) tma_prefetch_desc(&tm_q);
      }
      // one key tile of a segment into the next stage
      auto load_tile = [&](const Seg &sg, int j) -> bool {
        const TileKeys tk = tile_keys(sg.ctx, sg.drafts, j);
        const int32_t *bt = p.block_tables + static_cast<int64_t>(sg.seq) * p.max_blocks_per_seq;
        auto cache_row = [&](int key) {
          const int blk = __ldg(bt + key / p.block_size);
          if (blk >= 0 && blk < p.num_blocks) return blk * p.block_size + key % p.block_size;
          if (is_k) raise_error(p.err, PKV_DEVERR_BLOCK_ID);
          return oob_row;
        };
        const bool boxes = p.box_rows > 0 && tk.cached == kTile;
        const int pieces = boxes ? kTile / p.box_rows : tk.rows / 4;
        int4 r = make_int4(oob_row, oob_row, oob_row, oob_row);
        bool draft = false;
        if (lane < pieces) {
          if (boxes) {
            r.x = cache_row(j * kTile + lane * p.box_rows);
          } else {
            const int k0 = 4 * lane;
            draft = tk.drafts > 0 && k0 >= tk.at;
            if (draft) {
              const int u = k0 - tk.at, first = sg.q0 + tk.u0;
              r.x = u < tk.drafts ? first + u : p.total_q;
              r.y = u + 1 < tk.drafts ? first + u + 1 : p.total_q;
              r.z = u + 2 < tk.drafts ? first + u + 2 : p.total_q;
              r.w = u + 3 < tk.drafts ? first + u + 3 : p.total_q;
            } else {
              const int key = j * kTile + k0;
              if (k0 < tk.cached) r.x = cache_row(key);
              if (k0 + 1 < tk.cached) r.y = cache_row(key + 1);
              if (k0 + 2 < tk.cached) r.z = cache_row(key + 2);
              if (k0 + 3 < tk.cached) r.w = cache_row(key + 3);
            }
          }
        }
        const int s = issued % stages, round = issued / stages;
        const uint32_t full = is_k ? k_full(s) : v_full(s);
        int good = 1;
        if (lane == 0) {
          if (round > 0 && !mbar_wait(is_k ? k_empty(s) : v_empty(s), (round - 1) & 1, abort_flag)) {
            good = 0;
            fail();
          } else {
            mbar_arrive_expect_tx(full, tk.rows * kHD * 2);
          }
        }
        if (!__shfl_sync(0xffffffffu, good, 0)) return false;
        const uint32_t dst = is_k ? sK(s) : sV(s);
        if (lane < pieces) {
          if (boxes) {
            tma_load_3d(dst + lane * p.box_rows * 128, map_box, 0, sg.head, r.x, full);
            tma_load_3d(dst + kRegion + lane * p.box_rows * 128, map_box, 64, sg.head, r.x, full);
          } else {
            const CUtensorMap *map = draft ? map_draft : map_rows;
            tma_gather4(dst + lane * 512, map, sg.head * kHD, r, full);
            tma_gather4(dst + kRegion + lane * 512, map, sg.head * kHD + 64, r, full);
          }
        }
        ++issued;
        return true;
      };
      if (is_k) {
        // walk the range: streams of (head, sequence, row group)
        int qtiles = 0, q_issued = 0, op = 0, n = 0;
        int left = hi - lo;
        int head = left > 0 ? lo / total : 0, seq = left > 0 ? start[0] : 0;
        int off = left > 0 ? start[1] : 0;       // tile inside the sequence's row groups
        int seq_base = -32, c_ctx = 0, c_drafts = 0, c_q0 = 0;  // 32 sequences' lengths, one a lane
        Boundary bd;
        bd.row0 = -1;
        bd.ntok = bd.head = bd.first = bd.last = 0;
        bool first_seg = true;
        while (ok && left > 0) {
          if (seq >= p.num_seqs) {               // on to the next KV head
            seq = 0;
            ++head;
          }
          if (seq < seq_base || seq >= seq_base + 32) {
            seq_base = seq & ~31;
            c_drafts = 0;
            if (seq_base + lane < p.num_seqs)
              seq_lengths(p, seq_base + lane, &c_ctx, &c_drafts, &c_q0);
          }
          Seg sg;
          sg.ctx = __shfl_sync(0xffffffffu, c_ctx, seq - seq_base);
          sg.drafts = __shfl_sync(0xffffffffu, c_drafts, seq - seq_base);
          sg.q0 = __shfl_sync(0xffffffffu, c_q0, seq - seq_base);
          if (sg.drafts == 0) {
            ++seq;
            continue;
          }
          const int nt = tree_tiles(sg.ctx, sg.drafts);
          const int groups = (sg.drafts + pair_tokens - 1) / pair_tokens;
          int rg = off / nt;
          sg.t0 = off - rg * nt;
          sg.head = head;
          sg.seq = seq;
          for (; ok && rg < groups && left > 0; ++rg) {
            sg.t1 = min(nt, sg.t0 + left);
            sg.tok0 = rg * pair_tokens;
            sg.ntok = min(pair_tokens, sg.drafts - sg.tok0);
            const bool two = sg.ntok > p.tile_tokens;
            sg.slot = (sg.t0 == 0 && sg.t1 == nt) ? -1
                      : 2 * static_cast<int>(blockIdx.x) + (sg.t0 == 0 ? 1 : 0);
            if (two) op = (op + 1) & ~1;         // both row tiles of a key tile in one op pair
            sg.op0 = op;
            sg.qtile = qtiles;
            const int steps = sg.t1 - sg.t0;
            op += two ? 2 * steps : steps;
            // the stream that the range start cuts is merged at its first cut
            if (first_seg && sg.t0 > 0 && sg.t0 <= range) {
              bd.row0 = sg.q0 + sg.tok0;
              bd.ntok = sg.ntok;
              bd.head = head;
              bd.first = static_cast<int>(blockIdx.x) - 1;
              bd.last = (lo - sg.t0 + nt - 1) / range;
            }
            first_seg = false;
            int good = 1;
            if (lane == 0) {
              if (n >= kSegRing &&
                  !mbar_wait(seg_empty(n % kSegRing), ((n / kSegRing) - 1) & 1, abort_flag)) {
                good = 0;
                fail();
              } else {
                volatile Seg *v = seg_at(n);
                v->head = sg.head;
                v->ctx = sg.ctx;
                v->drafts = sg.drafts;
                v->q0 = sg.q0;
                v->seq = sg.seq;
                v->tok0 = sg.tok0;
                v->ntok = sg.ntok;
                v->t0 = sg.t0;
                v->t1 = sg.t1;
                v->slot = sg.slot;
                v->op0 = sg.op0;
                v->qtile = sg.qtile;
                v->bad = 0;
                mbar_arrive(seg_full(n % kSegRing));
              }
              // Q tiles: box_tokens * group rows a box
              for (int x = 0; good && x < (two ? 2 : 1); ++x) {
                const int s = (qtiles + x) & 1, round = (qtiles + x) >> 1;
                if (round > 0 && !mbar_wait(q_empty(s), (round - 1) & 1, abort_flag)) {
                  good = 0;
                  fail();
                  break;
                }
                const int tok = min(p.tile_tokens, sg.ntok - x * p.tile_tokens);
                const int boxes = (tok + p.box_tokens - 1) / p.box_tokens;
                const int box_rows = p.box_tokens * p.group;
                mbar_arrive_expect_tx(q_full(s), boxes * box_rows * kHD * 2);
                for (int b = 0; b < boxes; ++b) {
                  const int row = sg.q0 + sg.tok0 + x * p.tile_tokens + b * p.box_tokens;
                  const uint32_t dst = sQ + s * kTileBytes + b * box_rows * 128;
                  tma_load_3d(dst, &tm_q, 0, head * p.group, row, q_full(s));
                  tma_load_3d(dst + kRegion, &tm_q, 64, head * p.group, row, q_full(s));
                }
                ++q_issued;
              }
            }
            if (!__shfl_sync(0xffffffffu, good, 0)) {
              ok = false;
              break;
            }
            ++n;
            qtiles += two ? 2 : 1;
            for (int j = sg.t0; ok && j < sg.t1; ++j) ok = load_tile(sg, j);
            left -= steps;
            sg.t0 = 0;
          }
          ++seq;
          off = 0;
        }
        if (lane == 0) {
          p.bounds[blockIdx.x] = bd;
          if (ok) {                              // the walk's end
            if (n >= kSegRing &&
                !mbar_wait(seg_empty(n % kSegRing), ((n / kSegRing) - 1) & 1, abort_flag)) {
              fail();
            } else {
              seg_at(n)->head = -1;
              mbar_arrive(seg_full(n % kSegRing));
            }
          }
          for (int s = max(0, q_issued - 2); s < q_issued; ++s)   // drain
            mbar_wait(q_full(s & 1), (s >> 1) & 1, nullptr);
        }
      } else {
        Seg sg;
        for (int n = 0; ok; ++n) {
          if (!read_seg(n, sg, true)) {
            fail();
            break;
          }
          seg_done(n, true);
          if (sg.head < 0) break;
          for (int j = sg.t0; ok && j < sg.t1; ++j) ok = load_tile(sg, j);
        }
      }
      if (lane == 0)   // the last copies must land before the CTA exits
        for (int j = max(0, issued - stages); j < issued; ++j)
          mbar_wait(is_k ? k_full(j % stages) : v_full(j % stages), (j / stages) & 1, nullptr);
    } else if (warp == kWarpMma) {
      // ---------------------------------------------------------- MMA issuer
      if (lane == 0) {
        constexpr uint32_t idesc_s = umma_idesc_bf16(kTile, kTile, false);
        constexpr uint32_t idesc_pv = umma_idesc_bf16(kTile, kHD, true);  // B (V) MN-major
        bool ok = true;
        int s_count[2] = {0, 0}, pv_count[2] = {0, 0}, o_used[2] = {0, 0};
        // the PV that each x owes: MMA steps (0: none), first of its segment,
        // V tile, last user of it
        int steps[2] = {0, 0}, first[2] = {0, 0}, vtile[2] = {0, 0}, frees[2] = {0, 0};
        auto issue_pv = [&](int x) -> bool {
          if (steps[x] == 0) return true;
          const int s = vtile[x] % kVStages;
          if (!mbar_wait(v_full(s), (vtile[x] / kVStages) & 1, abort_flag) ||
              !mbar_wait(p_full(x), pv_count[x] & 1, abort_flag))
            return false;
          // the first PV of a segment overwrites O_x: the last one must be read out
          if (first[x]) {
            if (o_used[x] > 0 && !mbar_wait(o_free(x), (o_used[x] - 1) & 1, abort_flag)) return false;
            ++o_used[x];
          }
          tc_fence_after();
          const uint64_t dv = desc_v_mnmajor(sV(s));
          for (int kk = 0; kk < steps[x]; ++kk)
            umma_bf16_tmem_a(tmem_o(x), tmem_s(x) + kk * 8, desc_at(dv, kk * (2048 >> 4)), idesc_pv,
                             (first[x] && kk == 0) ? 0u : 1u);
          umma_commit(pv_done(x));
          ++pv_count[x];
          if (frees[x]) umma_commit(v_empty(s));
          steps[x] = 0;
          return true;
        };
        int op = 0, ktile = 0, vbase = 0;
        Seg sg;
        for (int n = 0; ok; ++n) {
          if (!read_seg(n, sg, false)) {
            ok = false;
            break;
          }
          seg_done(n, false);
          if (sg.head < 0) break;
          for (; ok && op < sg.op0; ++op) ok = issue_pv(op & 1);  // an op left out
          const bool two = sg.ntok > p.tile_tokens;
          const int tiles = sg.t1 - sg.t0, ops = two ? 2 * tiles : tiles;
          for (int i = 0; ok && i < ops; ++i, ++op) {
            const int x = op & 1;
            if (!issue_pv(x)) {
              ok = false;
              break;
            }
            const int tile = two ? i >> 1 : i;
            const int qt = sg.qtile + (two ? x : 0);
            const int s = ktile % kKStages;
            if ((i < (two ? 2 : 1) && !mbar_wait(q_full(qt & 1), (qt >> 1) & 1, abort_flag)) ||
                !mbar_wait(k_full(s), (ktile / kKStages) & 1, abort_flag)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint64_t dq = desc_kmajor(sQ + (qt & 1) * kTileBytes, 0), dk = desc_kmajor(sK(s), 0);
#pragma unroll
            for (int kk = 0; kk < kHD / 16; ++kk)
              umma_bf16(tmem_s(x), desc_at(dq, kmajor_step(kk)), desc_at(dk, kmajor_step(kk)), idesc_s,
                        kk > 0 ? 1u : 0u);
            umma_commit(s_full(x));
            ++s_count[x];
            const bool frees_kv = !two || x == 1;
            if (frees_kv) {
              umma_commit(k_empty(s));
              ++ktile;
            }
            if (i >= ops - (two ? 2 : 1)) umma_commit(q_empty(qt & 1));
            steps[x] = tile_keys(sg.ctx, sg.drafts, sg.t0 + tile).rows / 16;
            first[x] = i < 2;
            vtile[x] = vbase + tile;
            frees[x] = frees_kv;
          }
          vbase += tiles;
        }
        if (ok) ok = issue_pv(op & 1) && issue_pv((op + 1) & 1);
        if (!ok) fail();
        for (int x = 0; x < 2; ++x) {  // every issued MMA completes before TMEM is freed
          if (s_count[x] > 0) mbar_wait(s_full(x), (s_count[x] - 1) & 1, nullptr);
          if (pv_count[x] > 0) mbar_wait(pv_done(x), (pv_count[x] - 1) & 1, nullptr);
        }
      }
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(kRegsHigh));
    // ------------------------------------------------------ softmax 0 / 1
    const int x = warp >> 2;
    const int quad = warp & 3;                       // TMEM lanes 32 * quad ..
    const int r = quad * 32 + lane;                  // row of the MMA tile
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const int r_tok = r / p.group, r_head = r - r_tok * p.group;
    const float c = p.scale_log2;
    bool ok = true;
    int s_count = 0, vbase = 0, merges = 0;
    int pv_count[2] = {0, 0};
    Seg sg;
    for (int n = 0; ok; ++n) {
      if (!read_seg(n, sg, true)) {
        ok = false;
        break;
      }
      if (sg.head < 0) break;
      const bool two = sg.ntok > p.tile_tokens;
      const int tiles = sg.t1 - sg.t0;
      const int tok_x = two ? x * p.tile_tokens : 0;             // first token of this row tile
      const int ntok_x = min(p.tile_tokens, sg.ntok - tok_x);
      const bool live = r_tok < ntok_x;                          // this row exists
      const bool warp_live = quad * 32 < ntok_x * p.group;       // some row of the warp does
      const int64_t q_row = static_cast<int64_t>(sg.q0) + sg.tok0 + tok_x + r_tok;
      const int step = two ? 1 : 2;
      const int i0 = two ? 0 : ((x - sg.op0) & 1);
      float m_used = -INFINITY, l_sum = 0.f;         // running maximum of the scores, row sum

      for (int i = i0; ok && i < tiles; i += step) {
        const TileKeys tk = tile_keys(sg.ctx, sg.drafts, sg.t0 + i);
        const bool whole = tk.cached == kTile;
        // the row's visible columns of a tile that is not all cached keys
        uint32_t vis[4] = {0u, 0u, 0u, 0u};
        if (!whole && warp_live) {
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const int left = tk.drafts - 32 * w;
            if (live && left > 0) {
              vis[w] = static_cast<uint32_t>(
                  __ldg(p.tree_mask + q_row * p.mask_words + (tk.u0 >> 5) + w));
              if (left < 32) vis[w] &= (1u << left) - 1u;
            }
          }
          // move the drafts' bits up to their columns and add the cached ones
          if (tk.at & 64) {
            vis[3] = vis[1];
            vis[2] = vis[0];
            vis[1] = vis[0] = 0u;
          }
          if (tk.at & 32) {
            vis[3] = vis[2];
            vis[2] = vis[1];
            vis[1] = vis[0];
            vis[0] = 0u;
          }
          const int sh = tk.at & 31;
          vis[3] = __funnelshift_l(vis[2], vis[3], sh);
          vis[2] = __funnelshift_l(vis[1], vis[2], sh);
          vis[1] = __funnelshift_l(vis[0], vis[1], sh);
          vis[0] <<= sh;
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const int left = tk.cached - 32 * w;
            vis[w] |= left >= 32 ? 0xffffffffu : left > 0 ? (1u << left) - 1u : 0u;
          }
        }
        if (!warp_wait(s_full(x), s_count & 1, abort_flag)) {
          ok = false;
          break;
        }
        ++s_count;
        if (tk.drafts > 0) {
          // drafted V values that are not finite must not meet the weights of
          // rows that do not see them (0 * NaN); thread r takes V row r
          const int vt = vbase + i;
          if (!warp_wait(v_full(vt % kVStages), (vt / kVStages) & 1, abort_flag)) {
            ok = false;
            break;
          }
          if (r >= tk.at && r < tk.at + tk.drafts) {
            const uint32_t row = sV(vt % kVStages) + r * 128;
            uint32_t inf = 0u;
#pragma unroll 4
            for (int e = 0; e < 16; ++e) {
              const uint4 v = lds128(row + (e >> 3) * kRegion + (e & 7) * 16);
              // an all-ones exponent carries into the sign bit
              inf |= ((v.x & 0x7f807f80u) + 0x00800080u) | ((v.y & 0x7f807f80u) + 0x00800080u) |
                     ((v.z & 0x7f807f80u) + 0x00800080u) | ((v.w & 0x7f807f80u) + 0x00800080u);
            }
            if (inf & 0x80008000u) {
              // the flag first: a warpgroup that already finds zeros here sees it too
              seg_at(n)->bad = 1;
              __threadfence_block();
              for (int e = 0; e < 64; ++e) {
                const uint32_t a = row + (e >> 5) * kRegion + (e & 31) * 4;
                uint32_t v;
                asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
                if ((v & 0x7f80u) == 0x7f80u) v &= 0xffff0000u;
                if ((v & 0x7f800000u) == 0x7f800000u) v &= 0xffffu;
                asm volatile("st.shared.u32 [%0], %1;" :: "r"(a), "r"(v) : "memory");
              }
              fence_proxy_async_smem();
            }
          }
          __syncwarp();
        }
        if (warp_live) {
          tc_fence_after();
          float s[kTile];
#pragma unroll
          for (int cc = 0; cc < 4; ++cc)
            tmem_ld32(tmem_s(x) + lane_off + cc * 32, *reinterpret_cast<float(*)[32]>(s + cc * 32));
          tmem_wait_ld();
          if (p.flip != 1.f) {
#pragma unroll
            for (int e = 0; e < kTile; ++e) s[e] *= p.flip;
          }
          if (!whole) {
#pragma unroll
            for (int e = 0; e < kTile; ++e) s[e] = ((vis[e >> 5] >> (e & 31)) & 1u) ? s[e] : -INFINITY;
          }
          const float mt = max128(s);
          const bool grow =
              mt != -INFINITY && (m_used == -INFINITY || (mt - m_used) * c > kRescaleThreshold);
          float alpha = 1.f;
          if (grow) {
            if (m_used != -INFINITY) {
              alpha = ex2((m_used - mt) * c);
              l_sum *= alpha;
            }
            m_used = mt;
          }
          // O_x holds this x's earlier PVs of the segment, complete because S
          // completed after them
          if (i > i0 && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
            for (int cc = 0; cc < 4; ++cc) {
              float o[32];
              tmem_ld32(tmem_o(x) + lane_off + cc * 32, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] *= alpha;
              tmem_st32(tmem_o(x) + lane_off + cc * 32, o);
            }
            tmem_wait_st();
          }
          // a row that has seen nothing yet keeps weights of 0: exp2(-inf - 0)
          const float mc = m_used == -INFINITY ? 0.f : m_used * c;
          float2 rs2[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) rs2[e] = make_float2(0.f, 0.f);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t pk[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float2 xx = ffma2(make_float2(s[half * 64 + 2 * e], s[half * 64 + 2 * e + 1]),
                                      make_float2(c, c), make_float2(-mc, -mc));
              const float2 pp = make_float2(ex2(xx.x), ex2(xx.y));
              rs2[e & 3] = fadd2(rs2[e & 3], pp);
              pk[e] = float2_to_bf16x2(pp.x, pp.y);
            }
            tmem_st32_u(tmem_s(x) + lane_off + half * 32, pk);
          }
          const float2 rs01 = fadd2(rs2[0], rs2[1]), rs23 = fadd2(rs2[2], rs2[3]);
          l_sum += (rs01.x + rs01.y) + (rs23.x + rs23.y);
          tmem_wait_st();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(x));
      }
      if (!ok) break;

      // ---- the segment's end
      int ops_x[2];                                  // ops of each warpgroup in the segment
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int y0 = (y - sg.op0) & 1;
        ops_x[y] = two ? tiles : tiles > y0 ? (tiles - y0 + 1) / 2 : 0;
        pv_count[y] += ops_x[y];
      }
      vbase += tiles;
      const bool merge = !two && tiles > 1;          // both warpgroups hold a part of the rows
      const int owner = two ? x : (sg.op0 + tiles - 1) & 1;
      if (merge && owner != x) {
        // hand the row's maximum and sum to the other warpgroup
        if (merges > 0) ok = warp_wait(ml_free, (merges - 1) & 1, abort_flag);
        if (ok) {
          ml_x[r] = make_float2(m_used, l_sum);
          __syncwarp();
          if (lane == 0) mbar_arrive(ml_full);
        }
      } else if (owner == x) {
        ok = warp_wait(pv_done(x), (pv_count[x] - 1) & 1, abort_flag);
        float own = 1.f, oth = 0.f;                  // factors of O_x and the other's O
        float m_all = m_used;
        if (ok && merge) {
          ok = warp_wait(ml_full, merges & 1, abort_flag) &&
               warp_wait(pv_done(1 - x), (pv_count[1 - x] - 1) & 1, abort_flag);
          const float2 o = ml_x[r];
          m_all = fmaxf(m_used, o.x);
          own = m_used == -INFINITY ? 0.f : ex2((m_used - m_all) * c);
          oth = o.x == -INFINITY ? 0.f : ex2((o.x - m_all) * c);
          l_sum = l_sum * own + o.y * oth;
          __syncwarp();
          if (lane == 0) mbar_arrive(ml_free);
        }
        tc_fence_after();
        const bool bad = seg_at(n)->bad != 0;
        if (ok && warp_live) {
          const float inv = sg.slot >= 0 ? 1.f : l_sum == 0.f ? 0.f : 1.f / l_sum;
          own *= inv;
          oth *= inv;
          __nv_bfloat16 *orow = p.out + (q_row * p.num_q_heads + sg.head * p.group + r_head) * kHD;
          const int64_t rec = static_cast<int64_t>(sg.slot) * p.rows_cap +
                              tok_x * p.group + r;   // partial record's row
          if (sg.slot >= 0 && live)
            p.ml[rec] = make_float2(m_all == -INFINITY ? -INFINITY : m_all * c, l_sum);
#pragma unroll 1
          for (int cc = 0; cc < 4; ++cc) {
            float o[32];
            tmem_ld32(tmem_o(x) + lane_off + cc * 32, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] *= own;
            if (merge) {
              float o2[32];
              tmem_ld32(tmem_o(1 - x) + lane_off + cc * 32, o2);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = fmaf(o2[e], oth, o[e]);
            }
            if (bad && live) {
              // give back what was taken out of V for the drafts this row sees
              for (int j = sg.t0; j < sg.t1; ++j) {
                const TileKeys tk = tile_keys(sg.ctx, sg.drafts, j);
                for (int u = tk.u0; u < tk.u0 + tk.drafts; ++u) {
                  const uint32_t w = __ldg(p.tree_mask + q_row * p.mask_words + (u >> 5));
                  if (!((w >> (u & 31)) & 1u)) continue;
                  const uint32_t *v = reinterpret_cast<const uint32_t *>(
                      p.value + (static_cast<int64_t>(sg.q0) + u) * p.value_stride + sg.head * kHD +
                      cc * 32);
#pragma unroll
                  for (int e = 0; e < 16; ++e) {
                    const uint32_t b = __ldg(v + e);
                    const float2 f = bf16x2_to_float2(b);
                    if ((b & 0x7f80u) == 0x7f80u) o[2 * e] += f.x;
                    if ((b & 0x7f800000u) == 0x7f800000u) o[2 * e + 1] += f.y;
                  }
                }
              }
            }
            if (!live) continue;
            if (sg.slot >= 0) {
              float4 *dst = reinterpret_cast<float4 *>(p.po + rec * kHD + cc * 32);
#pragma unroll
              for (int q4 = 0; q4 < 8; ++q4)
                dst[q4] = make_float4(o[q4 * 4], o[q4 * 4 + 1], o[q4 * 4 + 2], o[q4 * 4 + 3]);
            } else {
              uint4 *dst = reinterpret_cast<uint4 *>(orow + cc * 32);
#pragma unroll
              for (int q4 = 0; q4 < 4; ++q4) {
                uint4 v;
                v.x = float2_to_bf16x2(o[q4 * 8 + 0], o[q4 * 8 + 1]);
                v.y = float2_to_bf16x2(o[q4 * 8 + 2], o[q4 * 8 + 3]);
                v.z = float2_to_bf16x2(o[q4 * 8 + 4], o[q4 * 8 + 5]);
                v.w = float2_to_bf16x2(o[q4 * 8 + 6], o[q4 * 8 + 7]);
                dst[q4] = v;
              }
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(o_free(x));
          if (merge) mbar_arrive(o_free(1 - x));
        }
      }
      if (merge) ++merges;
      seg_done(n, true);
    }
    if (!ok) fail();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Merge the pieces of the streams that range boundaries cut: one warp a row,
// each lane four dims. A stream's pieces lie in CTAs first .. last, in record
// 2c + 1 of the first (it starts there) and 2c of the others.
constexpr int kCombineWarps = 8;

__global__ void __launch_bounds__(kCombineWarps * 32) tree_combine_kernel(const TreeParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Boundary b = p.bounds[blockIdx.x];
  if (b.row0 < 0) return;
  const int lane = threadIdx.x & 31;
  const int rows = b.ntok * p.group;
  for (int row = blockIdx.y * kCombineWarps + (threadIdx.x >> 5); row < rows;
       row += gridDim.y * kCombineWarps) {
    // records hold two row tiles of tile_tokens * group rows back to back
    auto rec = [&](int piece) {
      return static_cast<int64_t>(2 * piece + (piece == b.first ? 1 : 0)) * p.rows_cap + row;
    };
    float m = -INFINITY;
    for (int c = b.first + lane; c <= b.last; c += 32) m = fmaxf(m, p.ml[rec(c)].x);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    float l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (m != -INFINITY) {
#pragma unroll 4
      for (int c = b.first; c <= b.last; ++c) {
        const float2 ml = p.ml[rec(c)];
        const float4 v = reinterpret_cast<const float4 *>(p.po + rec(c) * kHD)[lane];
        const float w = ml.x == -INFINITY ? 0.f : ex2(ml.x - m);
        if (ml.x == -INFINITY) continue;   // a piece the row sees nothing of
        l += w * ml.y;
        o.x += w * v.x;
        o.y += w * v.y;
        o.z += w * v.z;
        o.w += w * v.w;
      }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int tok = row / p.group, g = row - tok * p.group;
    uint2 w;
    w.x = float2_to_bf16x2(o.x * inv, o.y * inv);
    w.y = float2_to_bf16x2(o.z * inv, o.w * inv);
    reinterpret_cast<uint2 *>(p.out + ((static_cast<int64_t>(b.row0) + tok) * p.num_q_heads +
                                       b.head * p.group + g) * kHD)[lane] = w;
  }
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

// [rows, heads, 128] bf16 with a row stride, boxes of 64 dims x box_heads x box_rows
bool box_map(CUtensorMap *map, const void *base, uint64_t rows, uint64_t heads, uint64_t row_bytes,
             uint32_t box_heads, uint32_t box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {kHD, heads, rows};
  cuuint64_t strides[2] = {kHD * 2, row_bytes};
  cuuint32_t box[3] = {64, box_heads, box_rows};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [rows, heads * 128] bf16 with a row stride, for gathers of four rows x 64 elements
bool rows_map(CUtensorMap *map, const void *base, uint64_t rows, uint64_t heads, uint64_t row_bytes) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {heads * kHD, rows};
  cuuint64_t strides[1] = {row_bytes};
  cuuint32_t box[2] = {64, 1};
  cuuint32_t estr[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tokens of a Q box: box_tokens * group rows are whole 8-row swizzle atoms, at
// least 16 rows, so that a short tree loads little more than its own rows.
int box_tokens(int group) {
  int t = 1;
  while (t * group % 8 != 0 || t * group < 16) t *= 2;
  return t;
}

int tile_tokens(int group) {
  const int b = box_tokens(group);
  return b * (kTile / (b * group));
}

int rows_cap(int max_seqlen_q, int group) {
  const int tokens = 2 * tile_tokens(group);
  return (max_seqlen_q < tokens ? max_seqlen_q : tokens) * group;
}

size_t align256(size_t n) { return (n + 255) & ~size_t(255); }

struct TreeWs {
  size_t ml, po, total;
};

TreeWs tree_ws(int max_seqlen_q, int group, int grid) {
  const size_t rows = size_t(2) * grid * rows_cap(max_seqlen_q, group);
  TreeWs w;
  w.ml = align256(sizeof(Boundary) * grid);
  w.po = align256(w.ml + sizeof(float2) * rows);
  w.total = align256(w.po + sizeof(float) * rows * kHD);
  return w;
}

}  // namespace

bool tree_decode_supported(int num_q_heads, int num_kv_heads) {
  return num_q_heads % num_kv_heads == 0 && num_q_heads / num_kv_heads <= 16;
}

bool tree_decode_fits(int num_seqs, int max_seqlen_q, int max_context_len, int num_q_heads,
                      int num_kv_heads) {
  const int64_t pair = 2 * tile_tokens(num_q_heads / num_kv_heads);
  const int64_t tiles = int64_t(max_context_len) / kTile + 1 + (int64_t(max_seqlen_q) + kTile - 1) / kTile;
  const int64_t groups = (int64_t(max_seqlen_q) + pair - 1) / pair;
  // products of four int32 values: in double, whose 2^-53 does not matter here
  return double(tiles) * double(groups) * double(num_seqs) * double(num_kv_heads) < 1073741824.0;
}

size_t tree_decode_workspace_bytes(int max_seqlen_q, int num_q_heads, int num_kv_heads) {
  const int grid = decode_tc_grid();
  return grid > 0 ? tree_ws(max_seqlen_q, num_q_heads / num_kv_heads, grid).total : 0;
}

cudaError_t launch_tree_decode(const TreeDecodeArgs &a, cudaStream_t stream) {
  static std::once_flag attr_once;
  static cudaError_t attr_err = cudaSuccess;
  std::call_once(attr_once, [] {
    attr_err = cudaFuncSetAttribute(tree_decode_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    kSmemBytes);
    // setmaxnreg.inc waits until the registers it asks for are free: refuse a
    // build whose launch allocation is not the one the split adds up to
    cudaFuncAttributes fa;
    if (attr_err == cudaSuccess) attr_err = cudaFuncGetAttributes(&fa, tree_decode_kernel);
    if (attr_err == cudaSuccess && fa.numRegs != kRegsLaunch) attr_err = cudaErrorInvalidConfiguration;
  });
  if (attr_err != cudaSuccess) return attr_err;
  const int grid = decode_tc_grid();
  if (grid <= 0) return cudaErrorInvalidValue;
  const int group = a.num_q_heads / a.num_kv_heads;
  TreeParams p;
  p.box_tokens = box_tokens(group);
  p.tile_tokens = tile_tokens(group);
  // boxes fill whole 8-row swizzle atoms; other block sizes are gathered
  p.box_rows = a.block_size % 8 == 0 ? a.block_size & -a.block_size : 0;
  if (p.box_rows > kTile) p.box_rows = kTile;
  const uint64_t cache_rows = static_cast<uint64_t>(a.num_blocks) * a.block_size;
  const uint64_t cache_bytes = static_cast<uint64_t>(a.num_kv_heads) * kHD * 2;
  CUtensorMap tq, tk, tv, tkg, tvg, tkd, tvd;
  const uint32_t kv_box = p.box_rows > 0 ? p.box_rows : 8;
  if (!box_map(&tq, a.q, a.total_q, a.num_q_heads, static_cast<uint64_t>(a.num_q_heads) * kHD * 2,
               group, p.box_tokens) ||
      !box_map(&tk, a.k_cache, cache_rows, a.num_kv_heads, cache_bytes, 1, kv_box) ||
      !box_map(&tv, a.v_cache, cache_rows, a.num_kv_heads, cache_bytes, 1, kv_box) ||
      !rows_map(&tkg, a.k_cache, cache_rows, a.num_kv_heads, cache_bytes) ||
      !rows_map(&tvg, a.v_cache, cache_rows, a.num_kv_heads, cache_bytes) ||
      !rows_map(&tkd, a.key, a.total_q, a.num_kv_heads, a.key_stride * 2) ||
      !rows_map(&tvd, a.value, a.total_q, a.num_kv_heads, a.value_stride * 2))
    return cudaErrorInvalidValue;
  const TreeWs ws = tree_ws(a.max_seqlen_q, group, grid);
  uint8_t *w = static_cast<uint8_t *>(a.workspace);
  p.out = static_cast<__nv_bfloat16 *>(a.out);
  p.value = static_cast<const __nv_bfloat16 *>(a.value);
  p.value_stride = a.value_stride;
  p.block_tables = a.block_tables;
  p.max_blocks_per_seq = a.max_blocks_per_seq;
  p.context_lens = a.context_lens;
  p.cu_q = a.cu_seqlens_q;
  p.tree_mask = a.tree_mask;
  p.mask_words = a.mask_words;
  p.num_seqs = a.num_seqs;
  p.total_q = a.total_q;
  p.max_seqlen_q = a.max_seqlen_q;
  p.max_context_len = a.max_context_len;
  p.num_q_heads = a.num_q_heads;
  p.num_kv_heads = a.num_kv_heads;
  p.group = group;
  p.block_size = a.block_size;
  p.num_blocks = a.num_blocks;
  p.flip = a.scale > 0.f ? 1.f : a.scale < 0.f ? -1.f : 0.f;
  p.scale_log2 = a.scale == 0.f ? 1.f : fabsf(a.scale) * kLog2e;
  p.rows_cap = rows_cap(a.max_seqlen_q, group);
  p.bounds = reinterpret_cast<Boundary *>(w);
  p.ml = reinterpret_cast<float2 *>(w + ws.ml);
  p.po = reinterpret_cast<float *>(w + ws.po);
  p.err = a.err;
  tree_decode_kernel<<<grid, kThreads, kSmemBytes, stream>>>(tq, tk, tv, tkg, tvg, tkd, tvd, p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, (p.rows_cap + kCombineWarps - 1) / kCombineWarps);
  cfg.blockDim = dim3(kCombineWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_combine_kernel, p);
}

}  // namespace pkv
