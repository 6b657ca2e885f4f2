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
// Two softmax warpgroups x = 0, 1, each with a score region (TMEM columns 128 x
// ..), an output accumulator O_x (256 + 128 x ..), a maximum and a sum a row. A
// step g is one 128-row MMA tile meeting one key tile; it belongs to x = g & 1,
// and the tensor core gets PV(g - 2), S(g) for g = 0, 1, 2, ... across streams:
// while one warpgroup computes its softmax the tensor core and the other work.
//   * streams of one row tile (T_i * G <= 128): consecutive key tiles alternate
//     between the warpgroups; at the end the one with the last tile merges both,
//     reading the other's O from TMEM.
//   * streams of two row tiles: x takes row tile x, and each key tile makes two
//     steps; K and V are loaded once.
// P is written as bf16 over S and is the A operand of the PV MMA from there. P is
// exp2 of fp32 scores and enters the fp32 row sum before it is rounded; the one
// rounding of the weights to bf16 (2^-8 of each at most) is what the tensor
// core's operand type asks for. O is rescaled only when a row's maximum grows by
// over 2^8.
//
// Loads (warp 8 K, warp 10 V, warp 11 Q and the walk; warp 9 issues the MMAs): TMA boxes
// when the block size is a multiple of 8 (whole tiles in boxes of up to a block, partial
// tiles and drafts in boxes of 8 rows), else TMA row gathers, four rows an instruction: 256
// ragged sequences take 221 us at block size 16, 236 at 12 and at 1. Rows of a tile that
// are no key of the sequence may be other rows of a block or other sequences' drafts, and
// drafts that a row does not see may hold anything: their scores are masked, and V values
// among them that are not finite are set to zero in shared memory (0 * NaN is not 0),
// those of drafts to be added back at the end for the rows that see them.
//
// What a tile costs besides its loads is instructions, fetched by eleven warps that each
// do something else: the kernel follows its code size more than its arithmetic (256 ragged
// sequences: 297 us at 129 KB of code, 251 at 72 KB; later 225 -> 221 us from 95 to 82 KB,
// and 233 us with the two softmax passes unrolled; the loop that looks for non-finite
// drafts, unrolled by four, alone costs 2 %). Hence one copy of each role for both x,
// short loops, elected lanes and waits that hardware suspends.
//
// Measured, attention and combine, with floors of bytes at 6.78 TB/s (bf16 products at 1912
// TFLOP/s): 64 sequences U[128, 4096] x 16 drafts, 16 / 8 heads 94-96 us (81); 256 lognormal
// sequences x U[1, 32] drafts, 32 / 8 heads 221-223 us (194; DRAM traffic 1.29 GB read, the
// tensor pipe 31 % active); 8 x 32768 cached tokens x 64 drafts, 32 / 8 heads 213-218 us
// (160, 144 by products; the tensor pipe 57 % active, exp2 30 %, issue slots 39 %: none is
// full, each row tile waits for its chain S, softmax, PV), 239-242 us at the 1.7 GHz that
// the power limit leaves in long runs; one sequence of 5000 tokens 13.5 us (1). The combine
// is 4 to 10 us of it; the loads alone take 87.5 / 205 / 168 us of the first three.
// Figures of a choice, here and below, are its sides measured on the kernel of its time.
//
// Every wait on an mbarrier is bounded; on a timeout the CTA records PKV_DEVERR_TIMEOUT,
// drains its copies and MMAs, frees its TMEM and exits. (tcgen05.alloc waits, before any
// of those, until the SM's CTAs of another kernel have freed their TMEM.)
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <atomic>
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
// Five tiles fit. Three of K against three of V: 64 sequences of 16 drafts 96.0 / 97.9 us,
// 1 x 32768 33.7 / 34.2, 8 x 64 drafts 216.8 / 216.3, 256 ragged sequences the same.
constexpr int kKStages = 3;
constexpr int kVStages = 2;
constexpr int kThreads = 384;        // softmax 0 (warps 0-3), softmax 1 (4-7), loaders + MMA (8-11)
constexpr int kWarpK = 8, kWarpMma = 9, kWarpV = 10, kWarpWalk = 11;
constexpr int kTmemCols = 512;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescaleThreshold = 8.f;
constexpr int kSegRing = 4;
constexpr int kSegReaders = 2 + 1 + 8;   // K and V loaders, MMA issuer, softmax warps

constexpr int kOffMl = 0;                               // float2[128]
constexpr int kOffSeg = kOffMl + kTile * 8;
constexpr int kSegBytes = 64;
constexpr int kOffBar = kOffSeg + kSegRing * kSegBytes;
// q full/empty x2, k and v full/empty, s_full, p_full, o_free, pv_done, wg_end x2, ml
// full/free, drained, seg full/empty
constexpr int kNumBars = 4 + 2 * kKStages + 2 * kVStages + 10 + 3 + 2 * kSegRing;
constexpr int kOffMisc = kOffBar + kNumBars * 8;        // TMEM address, abort flag, start
constexpr int kOffRows = (kOffMisc + 32 + 15) / 16 * 16;      // int4[2][32], of the K and V loaders
constexpr int kOffQ = (kOffRows + 2 * 32 * 16 + 1023) / 1024 * 1024;   // two Q tiles
constexpr int kOffK = kOffQ + 2 * kTileBytes;
constexpr int kOffV = kOffK + kKStages * kTileBytes;
constexpr int kSmemBytes = kOffV + kVStages * kTileBytes;
static_assert(kSmemBytes <= 232448, "shared memory of one CTA");

// One CTA's part of one stream, handed from the walking warp to the other roles.
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
  int step0;    // its first step
  int qtile;    // running number of its first Q tile
  int bad;      // set when a drafted V value was not finite (seen or not)
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
  uint32_t bs_mul, bs_half, bs_shift;   // n / block_size, see block_of
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
// 8) on; rows 0 .. rows - 1 are loaded (a multiple of 16).
struct TileKeys {
  int cached, at, u0, drafts, rows;
};

__device__ __forceinline__ int tree_tiles(int ctx, int drafts) {
  const int full = ctx / kTile, rem = ctx % kTile;
  if (((rem + 7) & ~7) + drafts <= kTile) return full + 1;
  return full + (rem > 0 ? 1 : 0) + (drafts + kTile - 1) / kTile;
}

__device__ __forceinline__ TileKeys tile_keys(int ctx, int drafts, int j) {
  const int full = ctx / kTile, rem = ctx % kTile, rem8 = (rem + 7) & ~7;
  TileKeys k;
  k.at = k.u0 = k.drafts = 0;
  k.cached = kTile;
  k.rows = kTile;
  if (j < full) return k;
  if (rem8 + drafts <= kTile) {
    k.cached = rem;
    k.at = rem8;
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

// Maximum of 32 values, four chains of three-operand maxima (NaN is ignored).
__device__ __forceinline__ float max32(const float (&v)[32]) {
  float a[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) a[i] = fmaxf(v[i], v[i + 4]);
#pragma unroll
  for (int e = 8; e < 32; e += 8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = fmax3(a[i], v[e + i], v[e + 4 + i]);
  }
  return fmaxf(fmax3(a[0], a[1], a[2]), a[3]);
}

// One lane of a converged warp. Copies and MMAs take operands that are the same for the
// warp: inside `if (elect_one())`, in warp-uniform control flow, the compiler knows that
// they are, under `lane == 0` it does not (64 sequences 136 -> 117 us, 256 372 -> 289 us).
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// A value all lanes hold, uniform to the compiler.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

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

// Wait for the phase with the given parity: suspended in hardware for up to kSuspendNs
// at a time (it measured up to 4 us), because a dozen warps that poll take
// shared-memory cycles from the MMAs' operands (256 sequences: 361-429 us polling, 327
// suspended). Gives up when *abort becomes non-zero or after kMaxPolls polls, two
// seconds or so.
constexpr uint32_t kSuspendNs = 1000000u;
constexpr uint32_t kMaxPolls = 1u << 19;

__device__ __forceinline__ bool poll(uint32_t bar, uint32_t parity, uint32_t abort) {
  uint32_t ok;
  // nothing but the first try when the phase is over
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b32 n, f;\n\t"
      "mov.b32 %0, 1;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "@p bra DONE;\n\t"
      "mov.b32 n, 0;\n\t"
      "AGAIN:\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "@p bra DONE;\n\t"
      "ld.volatile.shared.b32 f, [%4];\n\t"
      "add.u32 n, n, 1;\n\t"
      "setp.ne.b32 q, f, 0;\n\t"
      "setp.ge.or.u32 q, n, %5, q;\n\t"
      "@!q bra AGAIN;\n\t"
      "mov.b32 %0, 0;\n\t"
      "DONE:\n\t}"
      : "=&r"(ok) : "r"(bar), "r"(parity), "r"(kSuspendNs), "r"(abort), "r"(kMaxPolls) : "memory");
  return ok != 0;
}

__device__ __forceinline__ void mbar_arrive_count(uint32_t bar, uint32_t n) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" :: "r"(bar), "r"(n) : "memory");
}

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, uint32_t abort) {
  return __all_sync(0xffffffffu, poll(bar, parity, abort));
}

// key / block_size without a division.
__device__ __forceinline__ int block_of(const TreeParams &p, int key) {
  const uint32_t n = key, t = __umulhi(n, p.bs_mul);
  return static_cast<int>((t + ((n - t) >> p.bs_half)) >> p.bs_shift);
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

// Whether a row sees any key. A row without a weight (a sum of 0) is zero if it sees nothing;
// if all its scores are -inf its softmax is NaN.
__device__ __forceinline__ bool sees_any(const TreeParams &p, int64_t q_row, int ctx, int drafts) {
  bool sees = ctx > 0;
#pragma unroll 1
  for (int u = 0; u < drafts && !sees; u += 32) {
    const uint32_t w = __ldg(p.tree_mask + q_row * p.mask_words + (u >> 5));
    sees = (drafts - u < 32 ? w & ((1u << (drafts - u)) - 1u) : w) != 0;
  }
  return sees;
}

__global__ void __launch_bounds__(kThreads, 1)
tree_decode_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_kp,
                   const __grid_constant__ CUtensorMap tm_vp, const __grid_constant__ CUtensorMap tm_kd,
                   const __grid_constant__ CUtensorMap tm_vd, const TreeParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw;
  const uint32_t base = smem_addr(smem_raw);
  if ((base & 1023u) != 0) {   // the swizzled tiles need it, and nothing is left to round up
    if (threadIdx.x == 0) p.bounds[blockIdx.x].row0 = -1;
    raise_error(p.err, PKV_DEVERR_TIMEOUT);
    return;
  }
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
  auto o_free = [&](int x) { return bar0 + 8u * (kBx + 4 + x); };
  auto pv_done = [&](int x) { return bar0 + 8u * (kBx + 6 + x); };
  auto wg_end = [&](int x) { return bar0 + 8u * (kBx + 8 + x); };
  const uint32_t ml_full = bar0 + 8u * (kBx + 10), ml_free = bar0 + 8u * (kBx + 11);
  const uint32_t drained = bar0 + 8u * (kBx + 12);
  auto seg_full = [&](int i) { return bar0 + 8u * (kBx + 13 + i); };
  auto seg_empty = [&](int i) { return bar0 + 8u * (kBx + 13 + kSegRing + i); };
  volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(smem + kOffMisc);
  volatile int *abort_word = reinterpret_cast<volatile int *>(smem + kOffMisc + 4);
  const uint32_t abort_flag = base + kOffMisc + 4;
  volatile int *start = reinterpret_cast<volatile int *>(smem + kOffMisc + 8);  // first sequence, tile
  const uint32_t never = base + kOffMisc + 16;   // stays 0
  float2 *ml = reinterpret_cast<float2 *>(smem + kOffMl);
  auto seg_at = [&](int i) {
    return reinterpret_cast<volatile Seg *>(smem + kOffSeg + (i % kSegRing) * kSegBytes);
  };

  if (warp == kWarpWalk) {
    // barriers counted 4 (a softmax warpgroup's warps), by ring readers, 2 (pv_done), else 1
    static_assert(kNumBars <= 64, "two barriers a lane");
    for (int b = lane; b < kNumBars; b += 32) {
      const uint32_t bar = bar0 + 8u * b;
      int count = 1;
      for (int x = 0; x < 2; ++x)
        if (bar == p_full(x) || bar == o_free(x) || bar == wg_end(x)) count = 4;
        else if (bar == pv_done(x)) count = 2;
      if (bar == ml_full || bar == ml_free) count = 4;
      if (bar >= seg_empty(0) && bar <= seg_empty(kSegRing - 1)) count = kSegReaders;
      mbar_init(bar, count);
    }
    if (lane == 0) *abort_word = *reinterpret_cast<volatile int *>(smem + kOffMisc + 16) = 0;
    fence_barrier_init();
  }
  if (warp == kWarpMma) {
    tmem_alloc(smem_addr(const_cast<uint32_t *>(tmem_slot)), kTmemCols);
    tmem_relinquish();
  }

  // ---- the CTA's range: tiles of all sequences (one KV head), counted by every
  // CTA itself; thread t counts sequences [t * per, (t + 1) * per)
  const int pair_tokens = 2 * p.tile_tokens;
  auto row_groups = [&](int drafts) {   // one but for wide trees
    return drafts <= pair_tokens ? 1 : (drafts + pair_tokens - 1) / pair_tokens;
  };
  const int per = (p.num_seqs + kThreads - 1) / kThreads;
  auto seq_cost = [&](int i, bool report) {
    int ctx, drafts, q0;
    if (!seq_lengths(p, i, &ctx, &drafts, &q0) && report) raise_error(p.err, PKV_DEVERR_LENGTH);
    return drafts == 0 ? 0 : tree_tiles(ctx, drafts) * row_groups(drafts);
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
  int before = 0, total = 0;   // tiles before this thread's and of all sequences
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    const int v = part[w];
    if (w < warp) before += v;
    total += v;
  }
  // range b is [floor(b * units / ctas), floor((b + 1) * units / ctas)), so that
  // with num_kv_heads | ctas every head is cut at the same tiles; no range is empty
  total = uniform(total);
  const int units = total * p.num_kv_heads;
  const int ctas = min(static_cast<int>(gridDim.x), max(units, 1));
  const int bid = static_cast<int>(blockIdx.x);
  const int per_cta = units / ctas, extra = units - per_cta * ctas;
  // n / ctas is the high word of n * ceil(2^32 / ctas) while n * ctas < 2^32; here n < ctas^2,
  // and a GPU has below 1600 SMs. With one CTA extra is 0.
  const uint32_t ctas_mul = 0xffffffffu / static_cast<uint32_t>(ctas) + 1;
  auto range_lo = [&](int b) {   // floor(b * units / ctas)
    b = min(b, ctas);
    return b * per_cta + static_cast<int>(__umulhi(b * extra, ctas_mul));
  };
  auto range_of = [&](int f) {   // the range that tile f lies in
    int a = 0, b = ctas - 1;
    while (a < b) {
      const int m = (a + b + 1) >> 1;
      if (range_lo(m) <= f) a = m; else b = m - 1;
    }
    return a;
  };
  const int lo = range_lo(bid), hi = range_lo(bid + 1);
  const int head0 = lo < hi ? lo / total : 0;
  const int off0 = lo < hi ? lo - head0 * total : -1;   // the range starts at this tile of its head
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
  auto tmem_s = [&](int x) { return tmem + x * kTile; };
  auto tmem_o = [&](int x) { return tmem + (2 + x) * kTile; };
  const uint32_t sQ = base + kOffQ;
  auto sK = [&](int s) { return base + kOffK + s * kTileBytes; };
  auto sV = [&](int s) { return base + kOffV + s * kTileBytes; };
  auto fail = [&]() {   // a whole warp
    if (lane == 0) {
      *abort_word = 1;
      raise_error(p.err, PKV_DEVERR_TIMEOUT);
    }
    __syncwarp();
  };
  // Segment n for a reader (a whole warp): copied out of the ring; false on a
  // timeout. seg_done() gives the ring entry back.
  auto read_seg = [&](int n, Seg &s) -> bool {
    if (!warp_wait(seg_full(n % kSegRing), (n / kSegRing) & 1, abort_flag)) return false;
    const uint32_t at = base + kOffSeg + (n % kSegRing) * kSegBytes;
    const uint4 a = lds128(at), b = lds128(at + 16), c = lds128(at + 32);
    s.head = uniform(a.x);
    s.ctx = uniform(a.y);
    s.drafts = uniform(a.z);
    s.q0 = uniform(a.w);
    s.seq = uniform(b.x);
    s.tok0 = uniform(b.y);
    s.ntok = uniform(b.z);
    s.t0 = uniform(b.w);
    s.t1 = uniform(c.x);
    s.slot = uniform(c.y);
    s.step0 = uniform(c.z);
    s.qtile = uniform(c.w);
    return true;
  };
  auto seg_done = [&](int n) {
    __syncwarp();
    if (lane == 0) mbar_arrive(seg_empty(n % kSegRing));
  };

  if (warp >= 8) {
    if (warp == kWarpK || warp == kWarpV) {
      // ---------------------------------------------------- K and V loaders
      // (one copy of the code for both warps)
      const bool is_k = warp == kWarpK;
      const int stages = is_k ? kKStages : kVStages;
      const uint32_t full0 = is_k ? k_full(0) : v_full(0), empty0 = is_k ? k_empty(0) : v_empty(0);
      const uint32_t dst0 = is_k ? sK(0) : sV(0);
      const CUtensorMap *map_whole = is_k ? &tm_k : &tm_v;
      const CUtensorMap *map_part = is_k ? &tm_kp : &tm_vp;
      const CUtensorMap *map_draft = is_k ? &tm_kd : &tm_vd;
      const int oob_row = p.num_blocks * p.block_size;
      const bool boxes = p.box_rows > 0;
      const int box_shift = __ffs(p.box_rows) - 1;
      int issued = 0, stage = 0, parity = 1;   // the first round finds every stage empty
      bool ok = true;
      if (lane == 0) {
        tma_prefetch_desc(map_whole);
        tma_prefetch_desc(map_part);
        tma_prefetch_desc(map_draft);
      }
      // The rows of a tile are looked up one tile ahead: the block table's latency
      // passes while the tile before waits for its stage and is issued. Lane l holds
      // what belongs to the first row of the tile's l-th box, or to the four rows of its
      // l-th gather; rows are worked out when the tile is issued, not waited for here.
      struct Rows {
        int4 r;       // the lane's block ids as read, or its rows of the drafts
        bool drafted;
        int key, off; // first key of the lane's copy, and its place in its block
        int left;     // cached keys from there on
        int rows;     // of the tile, to be loaded
        int shift;    // log2 of the rows a copy
        int draft;    // first copy of drafts
        int head;     // KV head; -1: no tile
        bool whole;
      };
      Seg sg;
      int n = -1, j = 0;
      sg.t1 = 0;
      auto look_up = [&](Rows &t) -> bool {   // the walk's next tile
        t.head = -1;
        if (j >= sg.t1) {
          if (!read_seg(++n, sg)) return false;
          seg_done(n);
          j = sg.t0;
          if (sg.head < 0) return true;
        }
        const TileKeys tk = tile_keys(sg.ctx, sg.drafts, j);
        t.head = sg.head;
        t.whole = tk.cached == kTile;
        t.rows = tk.rows;
        t.shift = !boxes ? 2 : t.whole ? box_shift : 3;
        t.draft = tk.drafts > 0 ? tk.at >> t.shift : kTile;
        const int k0 = lane << t.shift;
        t.key = j * kTile + k0;
        t.drafted = tk.drafts > 0 && k0 >= tk.at;
        if (t.drafted) {
          const int u = k0 - tk.at, first = sg.q0 + tk.u0;
          t.r.x = u < tk.drafts ? first + u : p.total_q;
          t.r.y = u + 1 < tk.drafts ? first + u + 1 : p.total_q;
          t.r.z = u + 2 < tk.drafts ? first + u + 2 : p.total_q;
          t.r.w = u + 3 < tk.drafts ? first + u + 3 : p.total_q;
        } else {
          const int32_t *bt = p.block_tables + static_cast<int64_t>(sg.seq) * p.max_blocks_per_seq;
          t.left = tk.cached - k0;
          t.r = make_int4(0, 0, 0, 0);
          const int blk = block_of(p, t.key);
          t.off = t.key - blk * p.block_size;
          if (t.left > 0) t.r.x = __ldg(bt + blk);
          if (!boxes) {
            if (t.left > 1) t.r.y = __ldg(bt + block_of(p, t.key + 1));
            if (t.left > 2) t.r.z = __ldg(bt + block_of(p, t.key + 2));
            if (t.left > 3) t.r.w = __ldg(bt + block_of(p, t.key + 3));
          }
        }
        ++j;
        return true;
      };
      int4 *rows_smem = reinterpret_cast<int4 *>(smem + kOffRows) + (is_k ? 0 : 32);
      Rows next;
      next.head = -1;
      next.drafted = true;
      do {                                   // the first turn only looks up
        Rows t = next;
        if (!t.drafted) {
          auto row = [&](int blk, int e) {   // of the lane's e-th key
            if (e >= t.left) return oob_row;
            const int off = e == 0 ? t.off : t.key + e - block_of(p, t.key + e) * p.block_size;
            if (blk >= 0 && blk < p.num_blocks) return blk * p.block_size + off;
            if (is_k) raise_error(p.err, PKV_DEVERR_BLOCK_ID);
            return oob_row;
          };
          t.r.x = row(t.r.x, 0);
          if (!boxes) {
            t.r.y = row(t.r.y, 1);
            t.r.z = row(t.r.z, 2);
            t.r.w = row(t.r.w, 3);
          }
        }
        ok = look_up(next);
        if (t.head < 0) continue;
        ok = ok && warp_wait(empty0 + 8 * stage, parity, abort_flag);
        if (!ok) break;
        // one lane issues the copies, from the rows of all lanes in shared memory
        rows_smem[lane] = t.r;
        __syncwarp();
        if (elect_one()) {
          const uint32_t full = full0 + 8 * stage;
          uint32_t dst = dst0 + stage * kTileBytes;
          mbar_arrive_expect_tx(full, t.rows * kHD * 2);
          const int copies = t.rows >> t.shift;
          const CUtensorMap *map = t.whole ? map_whole : map_part;
          if (boxes) {
            const int dst_step = 128 << t.shift;
            int b = 0;
#pragma unroll 1
            for (int part = 0; part < 2; ++part) {     // cached rows, drafts
              const int end = part == 0 ? min(t.draft, copies) : copies;
#pragma unroll 1
              for (; b < end; ++b, dst += dst_step) {
                const int row = rows_smem[b].x;
                tma_load_3d(dst, map, 0, t.head, row, full);
                tma_load_3d(dst + kRegion, map, 64, t.head, row, full);
              }
              map = map_draft;
            }
          } else {
            // 64 gathers a tile: their issue bounds the loader, so the rows of four
            // are read together (336 -> 251 us for 256 sequences; one at a time waits for
            // shared memory each time, eight are longer code: 283 us). The drafts begin
            // at an even one.
            const int x0 = t.head * kHD, x1 = x0 + 64;
#pragma unroll 1
            for (int b = 0; b < copies; b += 4, dst += 4 * 512) {
              const int4 r0 = rows_smem[b], r1 = rows_smem[b + 1], r2 = rows_smem[b + 2],
                         r3 = rows_smem[b + 3];
              const CUtensorMap *ma = b < t.draft ? map : map_draft;
              const CUtensorMap *mb = b + 2 < t.draft ? map : map_draft;
              tma_gather4(dst, ma, x0, r0, full);
              tma_gather4(dst + kRegion, ma, x1, r0, full);
              tma_gather4(dst + 512, ma, x0, r1, full);
              tma_gather4(dst + 512 + kRegion, ma, x1, r1, full);
              tma_gather4(dst + 1024, mb, x0, r2, full);
              tma_gather4(dst + 1024 + kRegion, mb, x1, r2, full);
              tma_gather4(dst + 1536, mb, x0, r3, full);
              tma_gather4(dst + 1536 + kRegion, mb, x1, r3, full);
            }
          }
        }
        __syncwarp();
        ++issued;
        if (++stage == stages) {
          stage = 0;
          parity ^= 1;
        }
      } while (ok && next.head >= 0);
      if (!ok) fail();
#pragma unroll 1
      for (int j = max(0, issued - stages); j < issued; ++j)   // the last copies must land
        warp_wait(full0 + 8 * (j % stages), (j / stages) & 1, never);
    } else if (warp == kWarpWalk) {
      // ---------------------------------------- the walk, and the Q tiles
      int qtiles = 0, q_issued = 0, step = 0, n = 0;
      bool ok = true;
      int left = hi - lo;
      int head = head0, seq = uniform(left > 0 ? start[0] : 0);
      int off = uniform(left > 0 ? start[1] : 0);   // tile inside the sequence's row groups
      int seq_base = -32, c_ctx = 0, c_drafts = 0, c_q0 = 0;  // 32 sequences' lengths, one a lane
      Boundary bd;
      bd.row0 = -1;
      bd.ntok = bd.head = bd.first = bd.last = 0;
      bool first_seg = true;
      if (lane == 0) tma_prefetch_desc(&tm_q);
      // the end of the walk is one more ring entry
      for (bool more = true; ok && more;) {
        Seg sg = {};
        int nt = 0;
        more = left > 0;
        if (more) {
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
          sg.ctx = __shfl_sync(0xffffffffu, c_ctx, seq - seq_base);
          sg.drafts = __shfl_sync(0xffffffffu, c_drafts, seq - seq_base);
          sg.q0 = __shfl_sync(0xffffffffu, c_q0, seq - seq_base);
          nt = sg.drafts == 0 ? 0 : tree_tiles(sg.ctx, sg.drafts);
          if (off >= nt * row_groups(sg.drafts)) {              // the sequence is done (or has no drafts)
            ++seq;
            off = 0;
            continue;
          }
        }
        bool two = false;
        if (more) {
          const int rg = off < nt ? 0 : off / nt;
          sg.t0 = off - rg * nt;
          sg.t1 = min(nt, sg.t0 + left);
          sg.tok0 = rg * pair_tokens;
          sg.ntok = min(pair_tokens, sg.drafts - sg.tok0);
          two = sg.ntok > p.tile_tokens;
          sg.slot = (sg.t0 == 0 && sg.t1 == nt) ? -1 : 2 * bid + (sg.t0 == 0 ? 1 : 0);
          if (two) step = (step + 1) & ~1;       // row tile x in steps g with g & 1 == x
          sg.step0 = step;
          const int tiles = sg.t1 - sg.t0;
          step += two ? 2 * tiles : tiles;
          off += tiles;
          left -= tiles;
        }
        ok = n < kSegRing || warp_wait(seg_empty(n % kSegRing), ((n / kSegRing) - 1) & 1, abort_flag);
        if (!ok) break;
        if (lane == 0) {
          volatile Seg *v = seg_at(n);
          v->head = more ? head : -1;
          v->ctx = sg.ctx;
          v->drafts = sg.drafts;
          v->q0 = sg.q0;
          v->seq = seq;
          v->tok0 = sg.tok0;
          v->ntok = sg.ntok;
          v->t0 = sg.t0;
          v->t1 = sg.t1;
          v->slot = sg.slot;
          v->step0 = sg.step0;
          v->qtile = qtiles;
          v->bad = 0;
          mbar_arrive(seg_full(n % kSegRing));
        }
        __syncwarp();
        ++n;
        // Q tiles: box_tokens * group rows a box
#pragma unroll 1
        for (int x = 0; more && x < (two ? 2 : 1); ++x) {
          const int s = qtiles & 1, round = qtiles >> 1;
          ok = round == 0 || warp_wait(q_empty(s), (round - 1) & 1, abort_flag);
          if (!ok) break;
          const int tok = min(p.tile_tokens, sg.ntok - x * p.tile_tokens);
          const int boxes = (tok + p.box_tokens - 1) >> (__ffs(p.box_tokens) - 1);
          const int box_rows = p.box_tokens * p.group;
          if (elect_one()) mbar_arrive_expect_tx(q_full(s), boxes * box_rows * kHD * 2);
          uint32_t dst = sQ + s * kTileBytes;
          int row = sg.q0 + sg.tok0 + x * p.tile_tokens;
#pragma unroll 1
          for (int b = 0; b < boxes; ++b) {
            if (elect_one()) {
              tma_load_3d(dst, &tm_q, 0, head * p.group, row, q_full(s));
              tma_load_3d(dst + kRegion, &tm_q, 64, head * p.group, row, q_full(s));
            }
            dst += box_rows * 128;
            row += p.box_tokens;
          }
          ++q_issued;
          ++qtiles;
        }
        if (first_seg && sg.t0 > 0) {
          bd.row0 = sg.q0 + sg.tok0;
          bd.ntok = sg.ntok;
          bd.head = head;
          bd.first = lo - sg.t0;
          bd.last = lo - sg.t0 + nt - 1;
        }
        first_seg = false;
      }
      // the stream that the range start cuts is merged at its first cut (worked out last:
      // nothing waits for it)
      if (bd.row0 >= 0) {
        bd.last = range_of(bd.last);
        if (range_lo(bid - 1) > bd.first) bd.row0 = -1;   // an earlier range cuts it too
        bd.first = bid - 1;
      }
      if (lane == 0) p.bounds[bid] = bd;
      if (!ok) fail();
#pragma unroll 1
      for (int s = max(0, q_issued - 2); s < q_issued; ++s)   // drain
        warp_wait(q_full(s & 1), (s >> 1) & 1, never);
    } else if (warp == kWarpMma) {
      // ---------------------------------------------------------- MMA issuer
      // One elected lane runs the whole role. Its instructions are on the path of every
      // tile, so there are few: one copy for both x, ring positions counted up,
      // descriptors that differ by adds, waits without a vote. MMAs are issued by twos: the
      // tensor core takes longer than a turn of the loop, and the code is 2 KB shorter
      // than unrolled.
      if (elect_one()) {
      constexpr uint32_t idesc_s = umma_idesc_bf16(kTile, 0, false);            // N is added
      constexpr uint32_t idesc_pv = umma_idesc_bf16(kTile, kHD, true);          // B (V) MN-major
      constexpr uint32_t kTileStep = kTileBytes >> 4;
      const uint32_t tm = tmem;
      const uint64_t dq0 = desc_kmajor(sQ, 0), dk0 = desc_kmajor(sK(0), 0), dv0 = desc_v_mnmajor(sV(0));
      // The PV that an x owes: its MMAs (16 keys each, 0: none), the stage and parity of
      // its V tile, and whether it is the x's first of the segment (overwrites O_x), the
      // last one, the last user of the V tile, or one whose V tile x = 0 has waited for.
      constexpr int kMmas = 15, kStageAt = 4, kParity = 64, kFresh = 128, kEnds = 256, kFrees = 512,
                    kWaited = 1024, kPv = 2047;
      // What an x keeps: the parity of p_full(x) and, once a segment has overwritten
      // O_x, that of o_free(x).
      constexpr int kPParity = 1 << 12, kOUsed = 1 << 13, kOParity = 1 << 14;
      int mine = 0, other = 0;               // of this step's x and of the other one
      bool ok = true, two = false, ended = false;
      int x = 0, step = 0, i = 0, steps = 0, whole = 0, flush = 0;
      int ks = 0, kp = 0, vs = 0, vp = 0;    // stage and parity of the next K and V tile
      Seg sg = {};
      for (int n = 0;; ) {
        if (i == steps && !ended) {          // the next segment
          ok = poll(seg_full(n % kSegRing), (n / kSegRing) & 1, abort_flag);
          if (!ok) break;
          const uint32_t at = base + kOffSeg + (n % kSegRing) * kSegBytes;
          const uint4 a = lds128(at), b = lds128(at + 16), c = lds128(at + 32);
          sg.head = a.x;
          sg.ctx = a.y;
          sg.drafts = a.z;
          sg.ntok = b.z;
          sg.t0 = b.w;
          sg.t1 = c.x;
          sg.step0 = c.z;
          sg.qtile = c.w;
          mbar_arrive(seg_empty(n % kSegRing));
          ++n;
          ended = sg.head < 0;
          two = sg.ntok > p.tile_tokens;
          steps = ended ? 0 : (two ? 2 : 1) * (sg.t1 - sg.t0);
          whole = sg.ctx / kTile;
          i = 0;
        }
        // ---- two steps at a time inside a segment: whole tiles, neither the first nor
        // the last PV of an x, so nothing is decided on the way
        if (x == 0 && i >= 4 && i + 4 <= steps && step >= sg.step0 &&
            sg.t0 + (two ? (i + 1) >> 1 : i + 1) < whole) {
          int ps = (mine >> kStageAt) & 3, pp = (mine & kParity) ? 1 : 0;   // V of the owed PVs
          int parity = (mine & kPParity) ? 1 : 0, parity1 = (other & kPParity) ? 1 : 0;
          const uint32_t q0 = (sg.qtile & 1) * kTileStep, q1 = ((sg.qtile + (two ? 1 : 0)) & 1) * kTileStep;
          int stage0 = 0, stage_p0 = 0, stage1 = 0, stage_p1 = 0;
          auto pv_s = [&](const int y, const uint32_t q, bool wait, bool free, int &p_par) -> bool {
            if (wait && !poll(v_full(ps), pp, abort_flag)) return false;
            if (!poll(p_full(y), p_par, abort_flag)) return false;
            p_par ^= 1;
            tc_fence_after();
            const uint64_t dv = desc_at(dv0, ps * kTileStep);
#pragma unroll 2
            for (int kk = 0; kk < kTile / 16; ++kk)
              umma_bf16_tmem_a(tm + (2 + y) * kTile, tm + y * kTile + kk * 8,
                               desc_at(dv, kk * (2048 >> 4)), idesc_pv, 1u);
            if (free) {
              umma_commit(v_empty(ps));
              if (++ps == kVStages) {
                ps = 0;
                pp ^= 1;
              }
            }
            if (wait && !poll(k_full(ks), kp, abort_flag)) return false;
            const uint64_t dq = desc_at(dq0, q), dk = desc_at(dk0, ks * kTileStep);
            constexpr uint32_t idesc = idesc_s | ((kTile >> 3) << 17);
#pragma unroll 2
            for (int kk = 0; kk < kHD / 16; ++kk)
              umma_bf16(tm + y * kTile, desc_at(dq, kmajor_step(kk)), desc_at(dk, kmajor_step(kk)),
                        idesc, kk > 0 ? 1u : 0u);
            umma_commit(s_full(y));
            (y ? stage1 : stage0) = vs;
            (y ? stage_p1 : stage_p0) = vp;
            if (free) {
              umma_commit(k_empty(ks));
              if (++ks == kKStages) {
                ks = 0;
                kp ^= 1;
              }
              if (++vs == kVStages) {
                vs = 0;
                vp ^= 1;
              }
            }
            return true;
          };
          do {
            ok = pv_s(0, q0, true, !two, parity) && pv_s(1, q1, !two, true, parity1);
            i += 2;
            step += 2;
          } while (ok && i + 4 <= steps && sg.t0 + (two ? (i + 1) >> 1 : i + 1) < whole);
          if (!ok) break;
          mine = (mine & (kOUsed | kOParity)) | (parity ? kPParity : 0) | kTile / 16 |
                 stage0 << kStageAt | (stage_p0 ? kParity : 0) | (two ? 0 : kFrees);
          other = (other & (kOUsed | kOParity)) | (parity1 ? kPParity : 0) | kTile / 16 |
                  stage1 << kStageAt | (stage_p1 ? kParity : 0) | kFrees | (two ? kWaited : 0);
          continue;
        }
        if (ended && flush++ == 2) break;
        // ---- what S of the step needs, unless it is left out (step0 is one further) or
        // the walk is over: worked out before the wait for the weights, so that PV and S
        // go to the tensor core one behind the other
        const bool scores = !ended && step >= sg.step0;
        const int qt = sg.qtile + (two ? x : 0);
        const int tile = sg.t0 + (two ? i >> 1 : i);
        const int rows = !scores || tile < whole ? kTile : tile_keys(sg.ctx, sg.drafts, tile).rows;
        const uint32_t idesc = idesc_s | (static_cast<uint32_t>(rows >> 3) << 17);
        const uint64_t dq = desc_at(dq0, (qt & 1) * kTileStep), dk = desc_at(dk0, ks * kTileStep);
        const uint32_t to = tm + (2 + x) * kTile, ts = tm + x * kTile;
        const bool frees = !two || x == 1;
        const bool k_there = (two && x == 1) || mbar_test_wait(k_full(ks), kp);
        // ---- the x's last PV
        const int w = mine;
        if (w & kMmas) {
          const int mmas = w & kMmas, stage = (w >> kStageAt) & 3;
          const uint64_t dv = desc_at(dv0, stage * kTileStep);
          int keep = (w & ~kPv) ^ kPParity;
          ok = (w & kWaited) || poll(v_full(stage), (w & kParity) ? 1 : 0, abort_flag);
          // what the last segment left in O_x must have been read out
          if (ok && (w & kFresh)) {
            if (w & kOUsed) {
              ok = poll(o_free(x), (w & kOParity) ? 1 : 0, abort_flag);
              keep ^= kOParity;
            }
            keep |= kOUsed;
          }
          mine = keep;
          ok = ok && poll(p_full(x), (w & kPParity) ? 1 : 0, abort_flag);
          if (!ok) break;
          tc_fence_after();
          if (mmas == kTile / 16) {
#pragma unroll 2
            for (int kk = 0; kk < kTile / 16; ++kk)
              umma_bf16_tmem_a(to, ts + kk * 8, desc_at(dv, kk * (2048 >> 4)), idesc_pv,
                               kk > 0 || !(w & kFresh));
          } else {
#pragma unroll 1
            for (int kk = 0; kk < mmas; ++kk)
              umma_bf16_tmem_a(to, ts + kk * 8, desc_at(dv, kk * (2048 >> 4)), idesc_pv,
                               kk > 0 || !(w & kFresh));
          }
          if (w & kFrees) umma_commit(v_empty(stage));
          if (w & kEnds) {
            umma_commit(pv_done(x));
            // and an arrival of this thread's own, which has waited for the softmax warps:
            // what they wrote to the segment (bad) is visible behind pv_done
            mbar_arrive(pv_done(x));
          }
        }
        // ---- S of the step
        if (scores) {
          ok = (i >= (two ? 2 : 1) || poll(q_full(qt & 1), (qt >> 1) & 1, abort_flag)) &&
               (k_there || poll(k_full(ks), kp, abort_flag));
          if (!ok) break;
          tc_fence_after();
#pragma unroll 2
          for (int kk = 0; kk < kHD / 16; ++kk)
            umma_bf16(ts, desc_at(dq, kmajor_step(kk)), desc_at(dk, kmajor_step(kk)), idesc,
                      kk > 0 ? 1u : 0u);
          umma_commit(s_full(x));
          if (frees) umma_commit(k_empty(ks));
          if (i >= steps - (two ? 2 : 1)) umma_commit(q_empty(qt & 1));
          mine |= rows / 16 | vs << kStageAt | (vp ? kParity : 0) | (i < 2 ? kFresh : 0) |
                  (i >= steps - 2 ? kEnds : 0) | (frees ? kFrees : 0) | (two && x == 1 ? kWaited : 0);
          if (frees) {
            if (++ks == kKStages) {
              ks = 0;
              kp ^= 1;
            }
            if (++vs == kVStages) {
              vs = 0;
              vp ^= 1;
            }
          }
          ++i;
        }
        ++step;
        x ^= 1;
        const int t = mine;
        mine = other;
        other = t;
      }
      if (!ok) {
        *abort_word = 1;
        raise_error(p.err, PKV_DEVERR_TIMEOUT);
      }
      // every issued MMA completes before TMEM is freed
      umma_commit(drained);
      poll(drained, 0, never);
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------ softmax 0 / 1
    const int x = warp >> 2;
    const int quad = warp & 3;                       // TMEM lanes 32 * quad ..
    const int row = quad * 32 + lane;                // row of the MMA tile
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const int r_tok = row / p.group, r_head = row - r_tok * p.group;
    const float c = p.scale_log2;
    bool ok = true;
    int steps_seen = 0, tbase = 0, merges = 0;
    int segs[2] = {0, 0};                            // segments each warpgroup has had steps in
    Seg sg;
    for (int n = 0; ok; ++n) {
      if (!read_seg(n, sg)) {
        ok = false;
        break;
      }
      if (sg.head < 0) break;
      const bool two = sg.ntok > p.tile_tokens;
      const bool clean = !two || x == 0;                         // looks for non-finite V
      const int tiles = sg.t1 - sg.t0;
      const int tok_x = two ? x * p.tile_tokens : 0;             // first token of this row tile
      const int ntok_x = min(p.tile_tokens, sg.ntok - tok_x);
      const bool live = r_tok < ntok_x;                          // this row exists
      const bool warp_live = quad * 32 < ntok_x * p.group;       // some row of the warp does
      const int64_t q_row = static_cast<int64_t>(sg.q0) + sg.tok0 + tok_x + r_tok;
      const int whole_tiles = sg.ctx / kTile;
      const int i0 = two ? 0 : (x - sg.step0) & 1;   // this warpgroup's first tile
      float m_used = -INFINITY, l_sum = 0.f;         // running maximum of the scores, row sum

      // warps without a row take no part: the first warp arrives for them too
      const int live_warps = min(4, (ntok_x * p.group + 31) / 32);
      const uint32_t arrivals = quad == 0 ? 5 - live_warps : 1;
      const int my_steps = two ? tiles : (tiles - i0 + 1) / 2;
      if (!warp_live) steps_seen += my_steps;
      for (int i = i0; ok && warp_live && i < tiles; i += two ? 1 : 2) {
        const bool whole = sg.t0 + i < whole_tiles;
        TileKeys tk;
        tk.drafts = 0;
        int cols = 4;               // 32-column pieces that hold keys, in pairs
        const int32_t *mask_row = p.tree_mask + q_row * p.mask_words;
        if (!whole) {
          tk = tile_keys(sg.ctx, sg.drafts, sg.t0 + i);
          if (live && tk.drafts > 0)
            asm volatile("prefetch.global.L1 [%0];" :: "l"(mask_row + (tk.u0 >> 5)));
          cols = (tk.rows + 63) >> 6 << 1;
        }
        if (!warp_wait(s_full(x), steps_seen & 1, abort_flag)) {
          ok = false;
          break;
        }
        ++steps_seen;
        {
          tc_fence_after();
          const uint32_t ts = tmem_s(x) + lane_off;
          if (!whole || p.flip != 1.f) {
            // a negative or zero scale and the columns the row does not see, back
            // into TMEM, so that what follows is the same code for every tile
#pragma unroll 1
            for (int cc = 0; cc < cols; ++cc) {
              uint32_t word = 0xffffffffu;             // the row's visible columns of the 32
              if (!whole) {
                const int left = tk.cached - 32 * cc;
                word = left >= 32 ? 0xffffffffu : left > 0 ? (1u << left) - 1u : 0u;
                const int u = 32 * cc - tk.at;         // draft of the first column
                if (live && u > -32 && u < tk.drafts) {
                  const int32_t *m = mask_row + (tk.u0 >> 5) + (u >> 5);
                  const uint32_t lo = u >= 0 ? static_cast<uint32_t>(__ldg(m)) : 0u;
                  const uint32_t hi =
                      (u & ~31) + 32 < tk.drafts ? static_cast<uint32_t>(__ldg(m + 1)) : 0u;
                  uint32_t bits = __funnelshift_r(lo, hi, u & 31);
                  if (tk.drafts - u < 32) bits &= (1u << (tk.drafts - u)) - 1u;
                  word |= bits;
                }
              }
              float s[32];
              tmem_ld32(ts + cc * 32, s);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) s[e] = ((word >> e) & 1u) ? s[e] * p.flip : -INFINITY;
              tmem_st32(ts + cc * 32, s);
            }
            tmem_wait_st();
          }
          // The scores are read twice, 32 columns at a time in short loops: code that
          // holds the whole row in registers is four times as long and its
          // instruction fetches cost more than the second read.
          float mt = -INFINITY;
#pragma unroll 1
          for (int cc = 0; cc < cols; cc += 2) {
            float s0[32], s1[32];
            tmem_ld32(ts + cc * 32, s0);
            tmem_ld32(ts + cc * 32 + 32, s1);
            tmem_wait_ld();
            mt = fmax3(mt, max32(s0), max32(s1));
          }
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
          // O_x holds this x's earlier PVs of the segment, complete because this S
          // was issued behind them
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
          float2 rs2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
          for (int cc = 0; cc < cols; cc += 2) {
            float s0[32], s1[32];
            tmem_ld32(ts + cc * 32, s0);
            tmem_ld32(ts + cc * 32 + 32, s1);
            tmem_wait_ld();
            uint32_t pk[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float2 ss = e < 16 ? make_float2(s0[2 * e], s0[2 * e + 1])
                                       : make_float2(s1[2 * e - 32], s1[2 * e - 31]);
              const float2 xx = ffma2(ss, make_float2(c, c), make_float2(-mc, -mc));
              const float2 pp = make_float2(ex2(xx.x), ex2(xx.y));
              rs2[e & 1] = fadd2(rs2[e & 1], pp);
              pk[e] = float2_to_bf16x2(pp.x, pp.y);
            }
            tmem_st32_u(ts + cc * 16, pk);   // over scores that have been read
          }
          l_sum += (rs2[0].x + rs2[0].y) + (rs2[1].x + rs2[1].y);
          tmem_wait_st();
          tc_fence_before();
        }
        if (clean && !whole) {
          // V values that are not finite must not meet the weights (of 0) of rows that
          // do not see them; the live threads share the 16-byte pieces of the tile's
          // rows behind the cached ones. Of a tile that both warpgroups use the first
          // does it: the MMA warp waits for its weights and issues its PV before the
          // second's, so both PVs come behind its writes and their proxy fences
          const int vt = tbase + i;
          if (!warp_wait(v_full(vt % kVStages), (vt / kVStages) & 1, abort_flag)) {
            ok = false;
            break;
          }
          const uint32_t v0 = sV(vt % kVStages);
#pragma unroll 1
          for (int e = tk.cached * 16 + row; e < tk.rows * 16; e += 32 * live_warps) {
            // piece e & 15 of row e / 16 (swizzled among themselves: any order will do)
            const uint32_t at = v0 + ((e >> 3) & 1) * kRegion + (e >> 4) * 128 + (e & 7) * 16;
            uint4 v = lds128(at);
            // an all-ones exponent carries into the sign bit
            const uint32_t inf =
                ((v.x & 0x7f807f80u) + 0x00800080u) | ((v.y & 0x7f807f80u) + 0x00800080u) |
                ((v.z & 0x7f807f80u) + 0x00800080u) | ((v.w & 0x7f807f80u) + 0x00800080u);
            if (inf & 0x80008000u) {
              if ((e >> 4) >= tk.at && (e >> 4) < tk.at + tk.drafts) seg_at(n)->bad = 1;
              auto finite = [](uint32_t w) {
                if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
                if ((w & 0x7f800000u) == 0x7f800000u) w &= 0xffffu;
                return w;
              };
              asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" :: "r"(at), "r"(finite(v.x)),
                           "r"(finite(v.y)), "r"(finite(v.z)), "r"(finite(v.w)) : "memory");
              fence_proxy_async_smem();
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive_count(p_full(x), arrivals);
      }
      if (!ok) break;

      // ---- the segment's end
      tbase += tiles;
#pragma unroll
      for (int y = 0; y < 2; ++y)
        if (two || tiles > ((y - sg.step0) & 1)) ++segs[y];
      const int owner = two ? x : (sg.step0 + tiles - 1) & 1;
      const bool merge = !two && tiles > 1;          // both warpgroups hold a part of the rows
      if (!warp_live) {
      } else if (owner != x) {
        if (merge) {
          // hand the rows' maxima and sums to the other warpgroup
          if (merges > 0) ok = warp_wait(ml_free, (merges - 1) & 1, abort_flag);
          ml[row] = make_float2(m_used, l_sum);
          __syncwarp();
          if (lane == 0) mbar_arrive_count(ml_full, arrivals);
        }
      } else {
        float own = 1.f, oth = 0.f;                  // factors of O_x and the other's O
        float m_all = m_used;
        if (merge) {
          ok = warp_wait(ml_full, merges & 1, abort_flag);
          const float2 o = ml[row];
          __syncwarp();
          if (lane == 0) mbar_arrive_count(ml_free, arrivals);
          m_all = fmaxf(m_used, o.x);
          own = m_used == -INFINITY ? 0.f : ex2((m_used - m_all) * c);
          oth = o.x == -INFINITY ? 0.f : ex2((o.x - m_all) * c);
          // maxima pass over NaN, so scores of NaN alone leave a maximum of -inf and a sum of
          // NaN, which a factor of 0 keeps: a sum of 0, not the maximum, says "sees nothing"
          l_sum = l_sum * own + o.y * oth;
        }
        ok = ok && warp_wait(pv_done(x), (segs[x] - 1) & 1, abort_flag) &&
             (!merge || warp_wait(pv_done(1 - x), (segs[1 - x] - 1) & 1, abort_flag));
        tc_fence_after();
        const bool bad = seg_at(n)->bad != 0;
        if (ok && warp_live) {
          // no weight: a partial record has -inf for its maximum if the row sees nothing at
          // all, else the lowest number, so that the combine can tell
          float inv = sg.slot >= 0 ? 1.f : 1.f / l_sum, lowest = -INFINITY;
          if (l_sum == 0.f) {
            if (live && sees_any(p, q_row, sg.ctx, sg.drafts)) lowest = -3.402823466e38f;
            if (sg.slot < 0) inv = lowest == -INFINITY ? 0.f : __int_as_float(0x7fc00000);
          }
          own *= inv;
          oth *= inv;
          __nv_bfloat16 *orow = p.out + (q_row * p.num_q_heads + sg.head * p.group + r_head) * kHD;
          const int64_t rec = static_cast<int64_t>(sg.slot) * p.rows_cap +
                              tok_x * p.group + row;   // partial record's row
          if (sg.slot >= 0 && live)
            p.ml[rec] = make_float2(m_all == -INFINITY ? lowest : m_all * c, l_sum);
#pragma unroll 1
          for (int cc = 0; cc < 4; ++cc) {
            float o[32];
            tmem_ld32(tmem_o(x) + lane_off + cc * 32, o);
            tmem_wait_ld();
            // an accumulator the row has no part in may not have been written
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = own == 0.f ? 0.f : o[e] * own;
            if (merge) {
              float o2[32];
              tmem_ld32(tmem_o(1 - x) + lane_off + cc * 32, o2);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = oth == 0.f ? o[e] : fmaf(o2[e], oth, o[e]);
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
          if (bad && live) {
            // give back what was taken out of V for the drafts this row sees, to what the
            // thread has just written: no rounding matters to an infinity or NaN (held in
            // registers it was 3 KB more code, for nearly no row)
            asm volatile("" ::: "memory");
#pragma unroll 1
            for (int j = sg.t0; j < sg.t1; ++j) {
              const TileKeys tk = tile_keys(sg.ctx, sg.drafts, j);
#pragma unroll 1
              for (int u = tk.u0; u < tk.u0 + tk.drafts; ++u) {
                const uint32_t w = __ldg(p.tree_mask + q_row * p.mask_words + (u >> 5));
                if (!((w >> (u & 31)) & 1u)) continue;
                const __nv_bfloat16 *v =
                    p.value + (static_cast<int64_t>(sg.q0) + u) * p.value_stride + sg.head * kHD;
#pragma unroll 1
                for (int e = 0; e < kHD; ++e) {
                  const float f = __bfloat162float(v[e]);
                  if (fabsf(f) < INFINITY) continue;
                  if (sg.slot >= 0)
                    p.po[rec * kHD + e] += f;
                  else
                    orow[e] = __float2bfloat16(__bfloat162float(orow[e]) + f);
                }
              }
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive_count(o_free(x), arrivals);
          if (merge) mbar_arrive_count(o_free(1 - x), arrivals);
        }
      }
      if (merge) ++merges;
      seg_done(n);
      // the warpgroup stays together by segments, so that a warp without a row never
      // misses a phase of the other barriers
      if (lane == 0) mbar_arrive(wg_end(x));
      ok = ok && warp_wait(wg_end(x), n & 1, abort_flag);
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

// Merge the pieces of the streams that range boundaries cut, each lane four dims
// of a row. A stream's pieces lie in CTAs first .. last, in record 2c + 1 of the
// first (it starts there) and 2c of the others. A warp merges a row of up to
// eight pieces; with more, the CTA's eight warps share the row's pieces, so that
// no warp waits for more than a few loads in turn (one sequence of 5000 tokens, 38
// pieces a row: 14.4 us shared, 22.0 not; 256 sequences, two or three pieces: 254 us
// shared, 225 not). Bound by the latency of that chain: lengths, pieces, output.
constexpr int kCombineWarps = 8;
constexpr int kBatch = 6;
constexpr int kPieces = 4;

__global__ void __launch_bounds__(kCombineWarps * 32, 4)
tree_combine_kernel(const TreeParams p, const int num_bounds) {
  __shared__ float2 s_ml[kCombineWarps];
  __shared__ float4 s_o[kCombineWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int index = blockIdx.x;
  if (static_cast<int>(gridDim.x) < num_bounds) {
    // few streams, fewer CTAs than boundaries: CTA x takes the x-th boundary that has
    // something to merge (searched for only then: it costs 1 us of 97)
    int left = blockIdx.x;
    index = -1;
    for (int b0 = 0; b0 < num_bounds && index < 0; b0 += 256) {
      bool cut[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int b = b0 + 32 * j + lane;
        cut[j] = b < num_bounds && p.bounds[b].row0 >= 0;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        unsigned mask = __ballot_sync(0xffffffffu, cut[j]);
        const int n = __popc(mask);
        if (index < 0 && left < n) {
          for (; left > 0; --left) mask &= mask - 1;
          index = b0 + 32 * j + __ffs(mask) - 1;
        } else {
          left -= n;
        }
      }
    }
    if (index < 0) return;
  }
  const Boundary b = p.bounds[index];
  if (b.row0 < 0) return;
  const int rows = b.ntok * p.group;
  const bool shared_row = b.last - b.first >= kCombineWarps;
  const int share = shared_row ? kCombineWarps : 1;   // warps on a row
  const int part = shared_row ? warp : 0;
  const int row0 = shared_row ? blockIdx.y : blockIdx.y * kCombineWarps + warp;
  const int row_step = gridDim.y * (shared_row ? 1 : kCombineWarps);
  auto finish = [&](int row, float m, float l, float4 o) {
    // no weight: zero for a row that sees nothing, else 0 / 0
    const float inv = m == -INFINITY && l == 0.f ? 0.f : 1.f / l;
    const int tok = row / p.group, g = row - tok * p.group;
    uint2 w;
    w.x = float2_to_bf16x2(o.x * inv, o.y * inv);
    w.y = float2_to_bf16x2(o.z * inv, o.w * inv);
    reinterpret_cast<uint2 *>(p.out + ((static_cast<int64_t>(b.row0) + tok) * p.num_q_heads +
                                       b.head * p.group + g) * kHD)[lane] = w;
  };
  if (b.last - b.first < kPieces) {
    // few pieces: two rows' loads in flight
    for (int row = row0; row < rows; row += 2 * row_step) {
      float2 ml[2][kPieces];
      float4 v[2][kPieces];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int j = 0; j < kPieces; ++j) {
          const int c = min(b.first + j, b.last);
          const int64_t rec = static_cast<int64_t>(2 * c + (c == b.first ? 1 : 0)) * p.rows_cap +
                              min(row + e * row_step, rows - 1);
          ml[e][j] = p.ml[rec];
          v[e][j] = reinterpret_cast<const float4 *>(p.po + rec * kHD)[lane];
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float m = -INFINITY, l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int j = 0; j < kPieces; ++j)
          if (b.first + j <= b.last) m = fmaxf(m, ml[e][j].x);
#pragma unroll
        for (int j = 0; j < kPieces; ++j) {
          // of a piece without a maximum only the sum counts: 0, or NaN
          if (b.first + j > b.last) continue;
          const float w = ml[e][j].x == -INFINITY ? 0.f : ex2(ml[e][j].x - m);
          l += w * ml[e][j].y;
          if (ml[e][j].x == -INFINITY) continue;
          o.x += w * v[e][j].x;
          o.y += w * v[e][j].y;
          o.z += w * v[e][j].z;
          o.w += w * v[e][j].w;
        }
        if (row + e * row_step < rows) finish(row + e * row_step, m, l, o);
      }
    }
    return;
  }
  for (int row = row0; row < rows; row += row_step) {
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    // a batch of pieces' loads in flight at a time
    for (int c0 = b.first + part; c0 <= b.last; c0 += kBatch * share) {
      float2 ml[kBatch];
      float4 v[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int c = min(c0 + j * share, b.last);
        const int64_t rec = static_cast<int64_t>(2 * c + (c == b.first ? 1 : 0)) * p.rows_cap + row;
        ml[j] = p.ml[rec];
        v[j] = reinterpret_cast<const float4 *>(p.po + rec * kHD)[lane];
      }
      float mt = m;
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if (c0 + j * share <= b.last) mt = fmaxf(mt, ml[j].x);
      const float a = m == -INFINITY ? 0.f : ex2(m - mt);
      l *= a;
      o = make_float4(o.x * a, o.y * a, o.z * a, o.w * a);
      m = mt;
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        // of a piece without a maximum only the sum counts: 0, or NaN
        if (c0 + j * share > b.last) continue;
        const float w = ml[j].x == -INFINITY ? 0.f : ex2(ml[j].x - m);
        l += w * ml[j].y;
        if (ml[j].x == -INFINITY) continue;
        o.x += w * v[j].x;
        o.y += w * v[j].y;
        o.z += w * v[j].z;
        o.w += w * v[j].w;
      }
    }
    if (shared_row) {
      s_o[warp][lane] = o;
      if (lane == 0) s_ml[warp] = make_float2(m, l);
      __syncthreads();
      if (warp == 0) {
        float mt = -INFINITY;
#pragma unroll
        for (int w = 0; w < kCombineWarps; ++w) mt = fmaxf(mt, s_ml[w].x);
        m = mt;
        l = 0.f;
        o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kCombineWarps; ++w) {
          const float2 ml = s_ml[w];
          const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - mt);
          const float4 v = s_o[w][lane];
          l += f * ml.y;
          o.x += f * v.x;
          o.y += f * v.y;
          o.z += f * v.z;
          o.w += f * v.w;
        }
      }
      __syncthreads();
      if (warp != 0) continue;
    }
    finish(row, m, l, o);
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
  // once a device: the attribute belongs to the device's copy of the kernel
  static std::atomic<uint64_t> attr_set{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t dev_bit = uint64_t(1) << (dev & 63);
  if (dev > 63 || !(attr_set.load() & dev_bit)) {
    e = cudaFuncSetAttribute(tree_decode_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kSmemBytes);
    if (e != cudaSuccess) return e;
    attr_set.fetch_or(dev_bit);
  }
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
  CUtensorMap tq, tk, tv, tkp, tvp, tkd, tvd;
  const uint64_t hkv = a.num_kv_heads, rows_q = a.total_q;
  bool maps = box_map(&tq, a.q, rows_q, a.num_q_heads, static_cast<uint64_t>(a.num_q_heads) * kHD * 2,
                      group, p.box_tokens);
  if (p.box_rows > 0) {
    maps = maps && box_map(&tk, a.k_cache, cache_rows, hkv, cache_bytes, 1, p.box_rows) &&
           box_map(&tv, a.v_cache, cache_rows, hkv, cache_bytes, 1, p.box_rows) &&
           box_map(&tkp, a.k_cache, cache_rows, hkv, cache_bytes, 1, 8) &&
           box_map(&tvp, a.v_cache, cache_rows, hkv, cache_bytes, 1, 8) &&
           box_map(&tkd, a.key, rows_q, hkv, a.key_stride * 2, 1, 8) &&
           box_map(&tvd, a.value, rows_q, hkv, a.value_stride * 2, 1, 8);
  } else {
    maps = maps && rows_map(&tk, a.k_cache, cache_rows, hkv, cache_bytes) &&
           rows_map(&tv, a.v_cache, cache_rows, hkv, cache_bytes) &&
           rows_map(&tkd, a.key, rows_q, hkv, a.key_stride * 2) &&
           rows_map(&tvd, a.value, rows_q, hkv, a.value_stride * 2);
    tkp = tk;
    tvp = tv;
  }
  if (!maps) return cudaErrorInvalidValue;
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
  // division by d = block_size with 2^(l-1) < d <= 2^l, m = 2^32 (2^l - d) / d + 1
  // (Granlund and Montgomery, "Division by Invariant Integers using Multiplication")
  int l = 0;
  while ((int64_t(1) << l) < a.block_size) ++l;
  p.bs_mul = static_cast<uint32_t>((((int64_t(1) << l) - a.block_size) << 32) / a.block_size + 1);
  p.bs_half = l > 0 ? 1 : 0;
  p.bs_shift = l > 0 ? l - 1 : 0;
  p.num_blocks = a.num_blocks;
  p.flip = a.scale > 0.f ? 1.f : a.scale < 0.f ? -1.f : 0.f;
  p.scale_log2 = a.scale == 0.f ? 1.f : fabsf(a.scale) * kLog2e;
  p.rows_cap = rows_cap(a.max_seqlen_q, group);
  p.bounds = reinterpret_cast<Boundary *>(w);
  p.ml = reinterpret_cast<float2 *>(w + ws.ml);
  p.po = reinterpret_cast<float *>(w + ws.po);
  p.err = a.err;
  tree_decode_kernel<<<grid, kThreads, kSmemBytes, stream>>>(tq, tk, tv, tkp, tvp, tkd, tvd, p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  // at most one merge a stream and one a range boundary
  const int64_t streams = static_cast<int64_t>(a.num_seqs) * a.num_kv_heads *
                          ((a.max_seqlen_q + 2 * p.tile_tokens - 1) / (2 * p.tile_tokens));
  const int merges = streams < grid ? static_cast<int>(streams) : grid;
  // four CTAs an SM in all (all resident at once: with 32 a merge the launch alone
  // took 8 us), shared among the merges; more than one a row helps nobody. 64 x 16
  // drafts: 109 us with one an SM, 105.7 with two, 104.5 with four, 104.7 with eight
  int share = 4 * grid / merges;
  share = share < p.rows_cap ? share : p.rows_cap;
  cfg.gridDim = dim3(merges, share > 0 ? share : 1);
  cfg.blockDim = dim3(kCombineWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_combine_kernel, p, grid);
}

}  // namespace pkv
