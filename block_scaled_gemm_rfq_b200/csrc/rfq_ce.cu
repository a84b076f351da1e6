// rfq_ce.cu -- softmax cross entropy at the output head, without the logits.
//
// With z = h . w^T (h [T][D] hidden states, w [V][D] the head, both bf16) and one label
// y_t per row,
//
//     lse_t  = log sum_v exp z_tv            loss_t = lse_t - z_{t,y_t}
//     dz_tv  = dloss_t (exp(z_tv - lse_t) - [v = y_t])
//     dh     = dz . w                         dw     = dz^T . h
//
// A logits matrix would be T x V; here a [256 x 256] tile of it exists only as the fp32
// accumulator of the tensor cores (TMEM).  Forward: the epilogue reduces each tile row to
// (max, sum of exponentials) over 128 (or 32) columns and a second kernel joins those parts.
// Backward: for one piece of the vocabulary at a time the logits are computed again,
// turned into dz with the known lse, rounded to bf16 into the workspace, and multiplied with
// w (dh, accumulated over the pieces in fp32) and h (dw, complete).
//
// All four products run in one persistent, warp-specialized kernel on tcgen05 kind::f16
// MMAs; what differs is how the operands lie in shared memory (along K, or along M/N for
// the products that contract over a matrix's rows: no transposed copy is made) and the
// epilogue:
//   kLogits  A = h (K-major)          B = w piece (K-major)     row statistics
//   kGrad    A = h (K-major)          B = w piece (K-major)     dz in bf16
//   kHidden  A = dz (K-major)         B = w piece (N-major)     dh, fp32 sums or bf16
//   kHead    A = dz (M-major)         B = h (N-major, a copy)   dw in bf16
//
// Roles (per CTA): warp 0 TMA producer, warp 1 MMA issuer (leader CTA of a pair),
// warps 2..9 epilogue.  Two 256-column accumulators, so that the epilogue of a tile runs
// under the mainloop of the next.  CTA pairs (256 x 256 tiles) above 128 rows, single
// CTAs (128 x 256, or 128 x 64 against small heads) up to 128, where the rest of a pair's rows would be padding.
// Every wait on an mbarrier is bounded (rfq_ptx.cuh).  No TMA multicast.
//
// Bounds and rates (a range is that of several cards).  With many rows the tensor cores bound all four products: 4096 x 4096 against
// 8192 entries keeps the tensor pipe 88 % (kLogits), 83 % (kGrad), 90 % (kHidden) and 83 % (kHead) active, 1.45 to
// 1.55 PFLOP/s with a cold start, a single launch each; under seconds of such load the card lowers its clock and
// 2048 x 4096 against 131072 entries take 1.65 to 1.72 ms (1.28 to 1.33 PFLOP/s).  The backward pass computes the logits
// once more, a fourth product to the three that training needs (4096 rows against 32768 x 4096: 3.36 to 3.48 ms forward and
// backward, 1.26 to 1.31 PFLOP/s over the four): the price of holding no T x V matrix between the passes, 537 MB in fp32
// there.  With few rows reading the head bounds them: 1 row against 131072 x 4096 takes 186 to 191 us, 5.6 to 5.8 TB/s; 8
// rows against 32003 x 1024 20 us, half of it the two kernels' start and end.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "rfq_internal.h"
#include "rfq_ptx.cuh"
#include "rfq_tmap.h"

namespace rfq {

__device__ unsigned int g_ce_error = 0;

namespace {

enum Mode { kLogits = 0, kGrad = 1, kHidden = 2, kHead = 3 };

constexpr int kBM = 128;                 // rows of the output per CTA
constexpr int kBN = 256;                 // columns of the output per tile,
constexpr int kNarrow = 64;              // or, for logits of few rows against a small head (see tile_columns())
constexpr int kBK = 64;                  // contraction elements per stage (128 bytes)
constexpr int kThreads = 320;            // warp 0 TMA, warp 1 MMA, warps 2..9 epilogue
constexpr uint32_t kTmemCols = 512;      // two accumulators of up to 256 fp32 columns
constexpr uint32_t kSmemLimit = 232448;
constexpr float kLog2e = 1.4426950408889634f;
// The tensor cores add into the fp32 accumulator by truncation, so a long contraction drifts
// towards zero: 3e-6 of lse at D = 4096 when one accumulator takes all of it.  Where the
// logits themselves are the result (kLogits) the accumulator therefore takes a part of the
// contraction at a time and the epilogue adds those parts with rounding: 1024 elements above 128 rows (512 cost
// 4 % of 2048 rows against 131072 x 4096), 128 up to 128 rows, where reading the head hides it (22.0 us both, then, for
// 8 rows against 32003 x 1024) and a loss of few rows has no others to average with (3e-6 -> 3e-7 for one row).
// The backward pass (kGrad) takes the same parts, so that its logits are those that lse is of: where a label is nearly
// certain p - 1 cancels, and a drift between the two was 17 % of 1 - p = 1e-3 at D = 4096.  It costs dh of 64 rows against 50000 x
// 2048 94 -> 97 us (the epilogue of a tile holds up the parts of the next), of 1000 rows against 50001 x 2048 nothing that shows.
// The gradients are rounded to bf16, but dw sums over up to 2^24 rows and dh over pieces of millions of entries: a sum of one
// sign over 2^24 rows lost 1 %.  They take 4096 at a time.
template <int kPair, int kMode>
constexpr int kPart = kMode == kLogits || kMode == kGrad ? (kPair == 2 ? 16 : 2) : 64;   // k-tiles
// Contractions that fit one part have kernels of their own (kParts false): the sums over parts cost the epilogue registers, and
// where it bounds the product that shows (dw of 64 rows of 50000 x 2048 104 -> 111 us, of 128 of 32768 x 4096 128 -> 141; of
// 1000 rows the same).  Not the forward logits, which have
// registers left, and the backward ones of few rows, whose parts are short.
template <int kPair, int kMode>
constexpr bool kAlwaysParts = kMode == kLogits || (kMode == kGrad && kPair == 1);
// dz is rounded to bf16 for the next products.  Over many rows those roundings average out; a few rows leave
// a gradient that is off by one rounding of its largest entries, beside its own.  Up to 16 rows dz is therefore
// kept as the sum of two bf16 terms: rows T .. 2 T - 1 of dz are what rows 0 .. T - 1 left out.  dh takes both
// in the one tile of 128 rows that it fills anyway and adds its rows at the end; dw takes a second k-tile.  Error
// of dh against 64 bits with one and with two terms: 1 row 0.0031 and 0.0018, 6 rows 0.0020 and 0.0017 (a bf16
// rounding alone is 0.0017).  It cost 1 row of 112492 x 2824 nothing (557 us), 3 of 3863 x 3112 72 -> 82 us; at 64
// rows of 50000 x 2048 189 -> 217 us, for an error that is 0.0020 without.  With more rows (0.0019 at
// 4096) it would be two products beside the four.
constexpr int64_t kTwoTermRows = 16;

// Products that write a matrix pass its rows through 4 KiB of shared memory per epilogue warp, so that
// they leave in whole 128-byte lines: a thread holds 128 columns of one row, and 16-byte stores of
// 32 rows at a time held a head gradient of 64 tokens to 2.1 TB/s.
template <int kPair, int kMode, int kN>
struct Layout {
  static constexpr uint32_t kATile = kBM * kBK * 2;               // 16 KiB
  static constexpr uint32_t kBTile = (kN / kPair) * kBK * 2;      // 32 KiB (single), 16 KiB (pair) or 8 KiB (narrow)
  static constexpr uint32_t kStage = kATile + kBTile;
  static constexpr uint32_t kBarrierBytes = 256;
  static constexpr uint32_t kOut = kMode == kLogits ? 0u : 8u * 4096u;
  static constexpr int kStages = static_cast<int>((kSmemLimit - 1024 - kBarrierBytes - kOut) / kStage);   // 4 (single), 7 or 6 (pair), 9 or 8 (narrow)
  static constexpr uint32_t kSmem = kStages * kStage + kOut + kBarrierBytes + 1024;
  static_assert(kStage % 1024 == 0, "stage buffers must keep 1 KiB alignment");
  static_assert(kSmem <= kSmemLimit, "exceeds the 227 KiB shared-memory limit");
  static constexpr int kAccs = 2;                                 // accumulators
  static_assert((2 * kStages + 2 * kAccs + 1) * 8 + 8 <= kBarrierBytes, "barrier area too small");
};

struct Maps {
  CUtensorMap a, b;
};

// How a product's tiles are shared out.  The first `whole` tiles go round the units (CTAs or
// pairs) one by one.  What is left over when these rounds are full (kHidden alone) is cut along the
// contraction into slices, each leaving the fp32 sums of its tile in a slot of its own; so a product
// of few tiles, or of a few more than a round, keeps the SMs busy.  All tiles of one slice come
// before the next slice: the units at work then read the same part of the contraction, and share it
// through L2 (cut into equal runs of k-tiles instead, with no such order, the units read dz and the
// head several times from memory: 657 against 561 us for 1000 x 2048 x 50001).
struct Share {
  int num_mb, num_nb;     // tiles along M (of kBM * kPair rows) and N
  int group;              // row tiles that pass over the columns together
  int tiles, whole;
  int units;
  int slices, slice_kt;   // of the rest: k-tiles of one slice
};

struct Params {
  int M, N;               // rows and columns of the product
  int num_kt;             // k-tiles of the contraction
  uint32_t a_bytes;       // of A in a stage
  Share share;
  // kLogits, kGrad
  const int64_t* labels;  // [M]
  int64_t ignore;
  int64_t vocab;
  int64_t v0;             // first vocabulary entry of the piece
  float2* stats;          // [2 * num_nb][M]: (max * log2 e, sum of 2^(z log2 e - that))
  float* target;          // [M]: logit of the label
  const float* lse;       // [M]
  const float* dloss;     // [M]
  const float* gmax;      // largest finite |dloss|
  __nv_bfloat16* dz;      // [M][ld_dz]
  int64_t ld_dz;
  // kHidden: whole tiles to bf16 at once (out != nullptr: one piece) or into fp32 sums; the rest to slots
  float* acc;             // [M][N]
  float* slots;           // [tiles - whole][slices][rows of a tile][kBN]
  int accumulate;         // not the first piece
  // kHidden and kHead
  __nv_bfloat16* out;     // [M][N]
  int term;               // kGrad and kHead: rows of dz before its second terms begin, or 0: it has none
  int skip;               // fault injection: 1 + the stage fill that the first CTA leaves out, or 0
};

// Shared-memory operand descriptors (128-byte swizzle).  K-major: rows of 128 bytes, 8-row
// groups 1024 bytes apart.  M/N-major: chunks of 64 M/N elements x kBK contraction rows of
// 128 bytes; 8 contraction rows are 1024 bytes (stride offset), the next 64 M/N elements one
// chunk (8 KiB) further (leading offset).
constexpr uint32_t kChunk = 64u * kBK * 2u;
template <bool kMnMajor>
__device__ __forceinline__ uint64_t operand_desc(const void* p) {
  const uint64_t addr = smem_addr(p);
  const uint64_t lbo = kMnMajor ? (kChunk >> 4) : 1u;
  return ((addr >> 4) & 0x3FFFull) | (lbo << 16) | ((1024ull >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
// Start-address step (16-byte units) of the 16 contraction elements of one MMA.
template <bool kMnMajor>
constexpr uint64_t kDescStep = kMnMajor ? (16u * 128u) >> 4 : 32u >> 4;

template <int kPair, bool kAMn, bool kBMn, int kN>
__device__ __forceinline__ constexpr uint32_t mma_idesc() {
  return (1u << 4)                               // D: fp32
         | (1u << 7) | (1u << 10)                // A, B: bf16
         | (uint32_t(kAMn) << 15) | (uint32_t(kBMn) << 16)
         | (uint32_t(kN >> 3) << 17) | (uint32_t((kBM * kPair) >> 4) << 24);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Tile number -> row and column tile.  Tiles run over groups of `group` row tiles, then column tiles,
// row tile fastest: the CTAs at work share few column tiles of B (the head's rows, which are far
// larger than L2) and one group of rows of A, which L2 holds.
__host__ __device__ __forceinline__ void place(const Share& s, int tile, int* mb, int* nb) {
  const int in_group = s.group * s.num_nb;
  const int g = tile / in_group;
  const int rr = tile - g * in_group;
  const int left = s.num_mb - g * s.group;
  const int rows = s.group < left ? s.group : left;
  *nb = rr / rows;
  *mb = g * s.group + (rr - *nb * rows);
}

struct Work {
  int mb, nb, kt0, kt1;
  int slot;               // -1: a whole tile
};
// Item `item` of a product: the whole tiles, then the slices.  False past the last, and where a slice is
// empty (the last piece of a vocabulary may be shorter than the one the slices were cut for).
__device__ __forceinline__ int num_items(const Share& s) { return s.whole + (s.tiles - s.whole) * s.slices; }
__device__ __forceinline__ bool work_at(const Params& p, int item, Work& w) {
  if (item < p.share.whole) {
    place(p.share, item, &w.mb, &w.nb);
    w.kt0 = 0;
    w.kt1 = p.num_kt;
    w.slot = -1;
    return true;
  }
  const int rest = p.share.tiles - p.share.whole;
  const int slice = (item - p.share.whole) / rest, t = (item - p.share.whole) - slice * rest;
  place(p.share, p.share.whole + t, &w.mb, &w.nb);
  w.kt0 = slice * p.share.slice_kt;
  w.kt1 = min(p.num_kt, w.kt0 + p.share.slice_kt);
  w.slot = t * p.share.slices + slice;
  return w.kt0 < w.kt1;
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&v);
}

template <int kPair, int kMode, int kN, bool kParts>
__global__ void __launch_bounds__(kThreads, 1) rfq_ce_kernel(const __grid_constant__ Maps maps, const Params p) {
  using L = Layout<kPair, kMode, kN>;
  constexpr int kC = kN / 2;   // columns of an epilogue thread
  constexpr bool kAMn = kMode == kHead;
  constexpr bool kBMn = kMode == kHidden || kMode == kHead;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kStages * L::kStage + L::kOut);
  uint64_t* empty = full + L::kStages;
  uint64_t* acc_full = empty + L::kStages;    // [kAccs]
  uint64_t* acc_empty = acc_full + L::kAccs;  // [kAccs]
  uint64_t* drain = acc_empty + L::kAccs;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = kPair == 2 ? cluster_cta_rank() : 0u;
  const bool leader = rank == 0;
  const int unit = static_cast<int>(blockIdx.x) / kPair;
  const int items = num_items(p.share);
  Work t;

  if (threadIdx.x == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < L::kAccs; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 8 * kPair);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&maps.a);
    prefetch_tmap(&maps.b);
  }
  if (warp == 1) {
    tmem_alloc_g<kPair>(tmem_slot, kTmemCols);
    tmem_relinquish_g<kPair>();
  }
  __syncwarp();
  tc_fence_before();
  if (kPair == 2) cluster_sync();
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  griddep_launch_dependents();
  griddep_wait();   // every input may come from the kernel before

  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------------------ TMA producer
      uint32_t stage = 0, phase = 0, filled = 0, last_parity = 0;
      int fill = 0;
      for (int item = unit; item < items; item += p.share.units) {
        if (!work_at(p, item, t)) continue;
        const int row_a = (t.mb * kPair + static_cast<int>(rank)) * kBM;
        const int row_b = t.nb * kN + static_cast<int>(rank) * (kN / kPair);
        for (int kt = t.kt0; kt < t.kt1; ++kt) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, &g_ce_error, kErrWaitEmpty)) goto producer_done;
          if (++fill != p.skip || blockIdx.x != 0) {
            uint8_t* sa = smem + stage * L::kStage;
            uint8_t* sb = sa + L::kATile;
            const uint32_t bar = kPair == 2 ? map_to_cta(smem_addr(&full[stage]), 0) : 0u;
            if (leader) mbar_arrive_expect_tx(&full[stage], (p.a_bytes + L::kBTile) * kPair);
            auto load = [&](uint8_t* dst, const CUtensorMap* map, int x, int y) {
              if constexpr (kPair == 2) tma_load_2d_pair(dst, map, bar, x, y);
              else tma_load_2d(dst, map, &full[stage], x, y);
            };
            if constexpr (kAMn) {
#pragma unroll
              for (int c = 0; c < kBM / 64; ++c) load(sa + c * kChunk, &maps.a, row_a + 64 * c, kt * (p.term > 0 ? p.term : kBK));
            } else {
              load(sa, &maps.a, kt * kBK, row_a);
            }
            if constexpr (kBMn) {
#pragma unroll
              for (int c = 0; c < kN / kPair / 64; ++c)   // the second terms meet the same rows of h; past its end are zeros
                load(sb + c * kChunk, &maps.b, row_b + 64 * c, kMode == kHead && p.term > 0 ? 0 : kt * kBK);
            } else {
              load(sb, &maps.b, kt * kBK, row_b);
            }
            filled |= 1u << stage;
            last_parity = (last_parity & ~(1u << stage)) | (phase << stage);
          }
          if (++stage == static_cast<uint32_t>(L::kStages)) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
    producer_done:
      // Teardown: every copy armed on this CTA's barriers must have landed.
      if (leader)
        for (int s = 0; s < L::kStages; ++s)
          if (filled & (1u << s)) {
            int never = 0;
            mbar_wait(&full[s], (last_parity >> s) & 1u, &never, &g_ce_error, kErrWaitDrain);
          }
    }
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      // ------------------------------------------------------------ MMA issuer
      constexpr uint32_t idesc = mma_idesc<kPair, kAMn, kBMn, kN>();
      uint32_t stage = 0, phase = 0, buf = 0, acc_phase = 0;
      bool ok = true;
      for (int item = unit; item < items && ok; item += p.share.units) {
        if (!work_at(p, item, t)) continue;
        const int part = kParts ? kPart<kPair, kMode> : t.kt1 - t.kt0;
        for (int kp = t.kt0; kp < t.kt1 && ok; kp += part) {
          if (!mbar_wait(&acc_empty[buf], acc_phase ^ 1u, abort_flag, &g_ce_error, kErrWaitAccEmpty)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t acc = tmem + buf * (kTmemCols / L::kAccs);
          const int kp1 = min(kp + part, t.kt1);
          for (int kt = kp; kt < kp1; ++kt) {
            if (!mbar_wait(&full[stage], phase, abort_flag, &g_ce_error, kErrWaitFull)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint8_t* sa = smem + stage * L::kStage;
            const uint64_t da = operand_desc<kAMn>(sa);
            const uint64_t db = operand_desc<kBMn>(sa + L::kATile);
#pragma unroll
            for (uint32_t q = 0; q < kBK / 16; ++q)
              mma_bf16_g<kPair>(acc, da + q * kDescStep<kAMn>, db + q * kDescStep<kBMn>, idesc,
                                (kt != kp || q != 0) ? 1u : 0u);
            tc_commit_g<kPair>(&empty[stage]);
            if (++stage == static_cast<uint32_t>(L::kStages)) {
              stage = 0;
              phase ^= 1u;
            }
          }
          if (!ok) break;
          tc_commit_g<kPair>(&acc_full[buf]);
          if (++buf == static_cast<uint32_t>(L::kAccs)) {
            buf = 0;
            acc_phase ^= 1u;
          }
        }
      }
      if (!ok) {
        // Teardown after an abort: wait for the MMAs already issued.
        tc_commit_g<kPair>(drain);
        int never = 0;
        mbar_wait(drain, 0, &never, &g_ce_error, kErrWaitDrain);
      }
    }
  } else {
    // -------------------------------------------------------------- epilogue
    // 8 warps: two per TMEM lane quadrant, each owning half of the columns; a thread
    // holds its (128 or 32) of one row, so row reductions need no exchange between lanes.
    const int quad = warp & 3;
    const int half = (warp - 2) >> 2;
    uint32_t buf = 0, acc_phase = 0;
    float gmax = 0.f;
    if constexpr (kMode != kLogits) gmax = *p.gmax;
    for (int item = unit; item < items; item += p.share.units) {
      if (!work_at(p, item, t)) continue;
      const int row = (t.mb * kPair + static_cast<int>(rank)) * kBM + quad * 32 + lane;
      const int col0 = t.nb * kN + half * kC;
      uint32_t v[kC / 32][32];
      auto take = [&](bool first) {
        // The lanes agree, so that none waits below for one that gave up; and rows past the end, which leave the loop body
        // early, are with the others again.
        const bool full_now = mbar_wait(&acc_full[buf], acc_phase, abort_flag, &g_ce_error, kErrWaitAccFull, 2 * kWaitLimitNs);
        if (!__all_sync(0xffffffffu, full_now)) return false;
        tc_fence_after();
        const uint32_t taddr = tmem + (static_cast<uint32_t>(quad * 32) << 16) + buf * (kTmemCols / L::kAccs) + half * kC;
        if (first) {
#pragma unroll
          for (int c = 0; c < kC / 32; ++c) tmem_load_32x32b_x32(taddr + 32 * c, v[c]);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int c = 0; c < kC / 16; ++c) {
            uint32_t u[2][8];
            tmem_load_32x32b_x8(taddr + 16 * c, u[0]);
            tmem_load_32x32b_x8(taddr + 16 * c + 8, u[1]);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              uint32_t& w = v[c >> 1][16 * (c & 1) + i];
              w = __float_as_uint(__uint_as_float(w) + __uint_as_float(u[i >> 3][i & 7]));
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (kPair == 2) mbar_arrive_remote(map_to_cta(smem_addr(&acc_empty[buf]), 0));
          else mbar_arrive(&acc_empty[buf]);
        }
        if (++buf == static_cast<uint32_t>(L::kAccs)) {
          buf = 0;
          acc_phase ^= 1u;
        }
        return true;
      };
      bool ok = take(true);
      if constexpr (kParts)
        for (int kp = t.kt0 + kPart<kPair, kMode>; kp < t.kt1 && ok; kp += kPart<kPair, kMode>) ok = take(false);
      if (!ok) break;
      // Hands this warp's rows over for storing, 128 bytes of each at a time: fill(c) gives this thread's
      // 16-byte piece c, keep(r, c, piece) stores piece c of row r of the warp's 32.
      auto turn = [&](int pieces, auto fill, auto keep) {
        int lane = static_cast<int>(threadIdx.x & 31);
        if constexpr (kParts) asm volatile("" : "+r"(lane));   // no address formed of it is kept from tile to tile: registers are short
        uint8_t* mine = smem + L::kStages * L::kStage + (warp - 2) * 4096;
#pragma unroll
        for (int c0 = 0; c0 < pieces; c0 += 8) {
#pragma unroll
          for (int c = 0; c < 8; ++c)
            if (c0 + c < pieces) *reinterpret_cast<uint4*>(mine + lane * 128 + ((c ^ (lane & 7)) << 4)) = fill(c0 + c);
          __syncwarp();
#pragma unroll(kParts ? 4 : 8)
          for (int i = 0; i < 8; ++i) {
            const int r = 4 * i + (lane >> 3), c = lane & 7;
            if (c0 + c < pieces) keep(r, c0 + c, *reinterpret_cast<const uint4*>(mine + r * 128 + ((c ^ (r & 7)) << 4)));
          }
          __syncwarp();
        }
      };
      const int row_w = row - lane;   // the warp's first row
      if (row_w >= p.M) continue;

      if constexpr (kMode == kLogits) {
        if (row >= p.M) continue;
        const int64_t label = p.labels[row] - p.v0 - col0;   // position inside this thread's columns, if 0..kC - 1
        const int cols = min(kC, p.N - col0);               // may be <= 0 in the last column tile
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < kC; ++i) {
          const float z = __uint_as_float(v[i >> 5][i & 31]);
          if (i < cols) m = fmaxf(m, z);
        }
        const float c = (m == -INFINITY ? 0.f : m) * kLog2e;
        float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
        for (int i = 0; i < kC; ++i) {
          const float e = i < cols ? ex2(fmaf(__uint_as_float(v[i >> 5][i & 31]), kLog2e, -c)) : 0.f;
          if ((i & 3) == 0) s0 += e;
          else if ((i & 3) == 1) s1 += e;
          else if ((i & 3) == 2) s2 += e;
          else s3 += e;
        }
        // A part without columns (or of nothing but -inf) is (-inf, 0): it joins as nothing.
        p.stats[static_cast<int64_t>(2 * t.nb + half) * p.M + row] =
            make_float2(m == -INFINITY ? -INFINITY : c, (s0 + s1) + (s2 + s3));
        if (label >= 0 && label < cols && label + p.v0 + col0 < p.vocab) {
          float z = 0.f;
#pragma unroll
          for (int i = 0; i < kC; ++i)
            if (i == label) z = __uint_as_float(v[i >> 5][i & 31]);
          p.target[row] = z;
        }
      } else if constexpr (kMode == kGrad) {
        const int at_row = min(row, p.M - 1);
        const int64_t label = p.labels[at_row];
        const int64_t from = label - p.v0 - col0;
        const int at = from >= 0 && from < kC ? static_cast<int>(from) : -1;   // the label's place among this thread's columns
        const bool counted = label != p.ignore;
        float g = p.dloss[at_row];
        g = gmax > 0.f ? g / gmax : g;          // gmax == 0: every finite entry is zero
        if (label < 0 || label >= p.vocab) g = NAN;
        const float l2 = p.lse[at_row] * kLog2e;
        // dz in the logits' place: of two neighbours the bf16 pair in the first one's register, and what it left out in the second's
        // (of an infinite or NaN entry the first term says all).
#pragma unroll
        for (int k = 0; k < kC; k += 2) {
          float d[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float q = ex2(fmaf(__uint_as_float(v[k >> 5][(k + e) & 31]), kLog2e, -l2));
            if (k + e == at) q -= 1.f;
            d[e] = counted ? q * g : 0.f;
          }
          const uint32_t pair = pack_bf16(d[0], d[1]);
          v[k >> 5][k & 31] = pair;
          if constexpr (kPair == 1) {
            const float l0 = d[0] - __uint_as_float(pair << 16), l1 = d[1] - __uint_as_float(pair & 0xffff0000u);
            v[k >> 5][(k + 1) & 31] = pack_bf16(fabsf(l0) <= 1.f ? l0 : 0.f, fabsf(l1) <= 1.f ? l1 : 0.f);
          }
        }
        auto leave = [&](auto second) {
          constexpr int kSecond = decltype(second)::value;
          turn(kC / 8, [&](int i) {
            const int k = 8 * i + kSecond;
            return make_uint4(v[k >> 5][k & 31], v[k >> 5][(k + 2) & 31], v[k >> 5][(k + 4) & 31], v[k >> 5][(k + 6) & 31]);
          }, [&](int r, int c, const uint4& piece) {
            if (row_w + r < p.M && col0 + 8 * c < p.N)
              *reinterpret_cast<uint4*>(p.dz + static_cast<int64_t>(row_w + r + (kSecond ? p.term : 0)) * p.ld_dz + col0 + 8 * c) = piece;
          });
        };
        leave(std::false_type{});
        if constexpr (kPair == 1)
          if (p.term > 0) leave(std::true_type{});
      } else if (kMode == kHidden && (p.out == nullptr || t.slot >= 0)) {
        float* dst = t.slot < 0 ? p.acc + static_cast<int64_t>(row_w) * p.N + col0
                                : p.slots + (static_cast<int64_t>(t.slot) * (kBM * kPair) + rank * kBM + quad * 32) * kN + half * kC;
        const int64_t ld = t.slot < 0 ? p.N : kN;
        turn(kC / 4, [&](int i) {
          return make_uint4(v[i >> 3][(4 * i) & 31], v[i >> 3][(4 * i + 1) & 31], v[i >> 3][(4 * i + 2) & 31], v[i >> 3][(4 * i + 3) & 31]);
        }, [&](int r, int c, const uint4& piece) {
          if (row_w + r >= p.M || col0 + 4 * c >= p.N) return;
          float4 f = make_float4(__uint_as_float(piece.x), __uint_as_float(piece.y), __uint_as_float(piece.z), __uint_as_float(piece.w));
          float4* o = reinterpret_cast<float4*>(dst + r * ld + 4 * c);
          if (p.accumulate) {
            const float4 was = *o;
            f.x += was.x;
            f.y += was.y;
            f.z += was.z;
            f.w += was.w;
          }
          *o = f;
        });
      } else {   // kHidden (one piece) and kHead
        turn(kC / 8, [&](int i) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int k = 8 * i + 2 * e;
            w[e] = pack_bf16(__uint_as_float(v[k >> 5][k & 31]) * gmax, __uint_as_float(v[(k + 1) >> 5][(k + 1) & 31]) * gmax);
          }
          return make_uint4(w[0], w[1], w[2], w[3]);
        }, [&](int r, int c, const uint4& piece) {
          if (row_w + r < p.M && col0 + 8 * c < p.N)
            *reinterpret_cast<uint4*>(p.out + static_cast<int64_t>(row_w + r) * p.N + col0 + 8 * c) = piece;
        });
      }
    }
  }

  __syncwarp();   // one lane alone had the work, or rows past the end left early: the barrier below takes whole warps
  tc_fence_before();
  if (kPair == 2) cluster_sync();
  else __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_g<kPair>(tmem, kTmemCols);
}

// Joins the parts of each row: C = max c, lse = C ln 2 + log sum s 2^(c - C).  One block per
// 32 rows, 32 strands over the parts; the last steps in double, so that a loss that is a
// small difference of large logits keeps the precision of the fp32 logits.
__global__ void __launch_bounds__(1024) rfq_ce_join_kernel(const float2* stats, const float* target, const int64_t* labels,
                                                           int M, int parts, int64_t ignore, int64_t vocab, float* loss,
                                                           float* lse) {
  __shared__ float sc[32][33], ss[32][33];
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x, strand = threadIdx.y;
  const int row = blockIdx.x * 32 + lane;
  float c = -INFINITY, s = 0.f;
  if (row < M) {
#pragma unroll 4
    for (int k = strand; k < parts; k += 32) {
      const float2 q = stats[static_cast<int64_t>(k) * M + row];
      const float top = fmaxf(c, q.x);
      const float base = top == -INFINITY ? 0.f : top;
      s = s * ex2(c - base) + q.y * ex2(q.x - base);
      c = top;
    }
  }
  sc[strand][lane] = c;
  ss[strand][lane] = s;
  __syncthreads();
  // A warp for each row, a lane for each strand.
  const int out_row = blockIdx.x * 32 + strand;
  if (out_row >= M) return;
  c = sc[lane][strand];
  s = ss[lane][strand];
  float top = c;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  const float base = top == -INFINITY ? 0.f : top;
  s *= ex2(c - base);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
  if (lane == 0) {
    const double l = static_cast<double>(base) * 0.69314718055994530942 + log(static_cast<double>(s));
    lse[out_row] = static_cast<float>(l);
    const int64_t label = labels[out_row];
    float out = 0.f;
    if (label != ignore)
      out = label >= 0 && label < vocab ? static_cast<float>(l - static_cast<double>(target[out_row])) : NAN;
    loss[out_row] = out;
  }
}

// Before the products.  Block 0: gmax = largest finite |dloss| over the rows that count.  The others, where dw is wanted:
// a copy of h whose ignored rows are zero.  dz of such a row is zero, but dw = dz^T h would still take 0 x NaN or
// 0 x inf from padding that nobody wrote.  (A warp for each 2 KiB of a row.  dw of 300 rows against 5000 x 1024 25 -> 28 us, of 64
// against 50000 x 2048 97 -> 104 with the logits' parts, of 4096 against 8192 x 4096 415 -> 435, both gradients against 32768 x 4096
// 2.56 ms as before; a warp for each row took 7 us more for one row.)
constexpr int kCopyRun = 128;   // 16-byte vectors
__global__ void __launch_bounds__(1024) rfq_ce_prepare_kernel(const float* dloss, const int64_t* labels, int M, int64_t ignore, float* gmax,
                                                              const uint4* h, uint4* clean, int vecs) {
  __shared__ float part[32];
  griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (blockIdx.x > 0) {
    const int runs = (vecs + kCopyRun - 1) / kCopyRun;   // of a row; M * runs < 2^30
    for (int i = (static_cast<int>(blockIdx.x) - 1) * 32 + warp; i < M * runs; i += (static_cast<int>(gridDim.x) - 1) * 32) {
      const int row = i / runs, c0 = (i - row * runs) * kCopyRun + lane;
      const int64_t label = labels[row];
      const int64_t at = static_cast<int64_t>(row) * vecs + c0;
      uint4 v[kCopyRun / 32];   // asked for beside the label, not after it
#pragma unroll
      for (int u = 0; u < kCopyRun / 32; ++u) v[u] = c0 + 32 * u < vecs ? h[at + 32 * u] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int u = 0; u < kCopyRun / 32; ++u)
        if (c0 + 32 * u < vecs) clean[at + 32 * u] = label != ignore ? v[u] : make_uint4(0u, 0u, 0u, 0u);
    }
    return;
  }
  float m = 0.f;
  for (int i = threadIdx.x; i < M; i += 1024) {
    const float g = fabsf(dloss[i]);
    if (labels[i] != ignore && g <= 3.402823466e38f) m = fmaxf(m, g);
  }
  for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  if (lane == 0) part[warp] = m;
  __syncthreads();
  if (threadIdx.x < 32) {
    m = part[threadIdx.x];
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    if (threadIdx.x == 0) *gmax = m;
  }
}

// dh of the tiles that the product left in fp32: gmax * the sum of a tile's slots, in order (of two rows where
// dz has two terms), or (whole tiles of a product over several pieces) gmax * its sums.  One block per 4 rows of a tile, so that small
// outputs of many slices have their loads under way at once.
__global__ void __launch_bounds__(256) rfq_ce_hidden_kernel(const Share share, int tile0, int tile_rows, const float* acc, const float* slots,
                                                            const float* gmax, int M, int N, int term, __nv_bfloat16* dh) {
  griddep_launch_dependents();
  griddep_wait();
  const int blocks = tile_rows / 4;
  const int tile = tile0 + static_cast<int>(blockIdx.x) / blocks;
  const int r = static_cast<int>(blockIdx.x) % blocks * 4 + (threadIdx.x >> 6);
  int mb, nb;
  place(share, tile, &mb, &nb);
  const int rest = tile - share.whole;
  const int in_tile = (threadIdx.x & 63) * 4, col = nb * kBN + in_tile, row = mb * tile_rows + r;
  if (col >= N || row >= M) return;
  const float g = *gmax;
  float4 f;
  if (rest < 0) {
    f = *reinterpret_cast<const float4*>(acc + static_cast<int64_t>(row) * N + col);
  } else {
    const float* src = slots + (static_cast<int64_t>(rest) * share.slices * tile_rows + r) * kBN + in_tile;
    f = *reinterpret_cast<const float4*>(src);
#pragma unroll 8
    for (int s = 1; s < share.slices; ++s) {
      const float4 o = *reinterpret_cast<const float4*>(src + static_cast<int64_t>(s) * tile_rows * kBN);
      f.x += o.x;
      f.y += o.y;
      f.z += o.z;
      f.w += o.w;
    }
    if (term > 0) {
      src += static_cast<int64_t>(term) * kBN;
#pragma unroll 8
      for (int s = 0; s < share.slices; ++s) {
        const float4 o = *reinterpret_cast<const float4*>(src + static_cast<int64_t>(s) * tile_rows * kBN);
        f.x += o.x;
        f.y += o.y;
        f.z += o.z;
        f.w += o.w;
      }
    }
  }
  *reinterpret_cast<uint2*>(dh + static_cast<int64_t>(row) * N + col) = make_uint2(pack_bf16(f.x * g, f.y * g), pack_bf16(f.z * g, f.w * g));
}

template <class Kernel, class... Args>
cudaError_t launch_pdl(Kernel kernel, dim3 grid, dim3 block, size_t smem, int cluster, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // see griddep_wait()
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  return e != cudaSuccess ? e : cudaGetLastError();
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int kPlanSms = 148;                      // work is shared out for a B200, whatever runs it

// Pairs of CTAs above 128 rows.
int pair_of(int64_t M) { return M > kBM ? 2 : 1; }

enum Cut { kWhole, kCutRest, kAllSlots };

Share share_out(int64_t M, int64_t N, int64_t K, Cut cut, int columns = kBN) {
  const int pair = pair_of(M);
  Share s = {};
  s.num_mb = static_cast<int>(ceil_div(M, kBM * pair));
  s.num_nb = static_cast<int>(ceil_div(N, columns));
  s.group = 16;
  s.tiles = s.whole = s.num_mb * s.num_nb;
  s.units = kPlanSms / pair;
  s.slices = 1;
  s.slice_kt = static_cast<int>(ceil_div(K, kBK));
  if (cut == kAllSlots || (cut == kCutRest && s.tiles % s.units != 0)) {
    // The number of slices that leaves the fewest k-tiles to the unit with the most, each slice
    // charged 4 for its epilogue.
    s.whole = cut == kAllSlots ? 0 : s.tiles / s.units * s.units;
    const int64_t rest = s.tiles - s.whole, kt = s.slice_kt;
    int64_t best = INT64_MAX;
    for (int n = 1; n <= 32 && n <= kt; ++n) {
      const int64_t per = ceil_div(kt, n);
      if (ceil_div(kt, per) != n) continue;
      const int64_t cost = ceil_div(rest * n, s.units) * (per + 4);
      if (cost < best) {
        best = cost;
        s.slices = n;
        s.slice_kt = static_cast<int>(per);
      }
    }
    if (s.slices == 1 && cut != kAllSlots) s.whole = s.tiles;
  }
  return s;
}

template <int kPair, int kMode, int kN>
cudaError_t launch_mode(const Maps& maps, const Params& p, cudaStream_t stream) {
  using L = Layout<kPair, kMode, kN>;
  const int longest = p.share.whole > 0 ? p.num_kt : p.share.slice_kt;
  auto kernel = rfq_ce_kernel<kPair, kMode, kN, true>;
  if constexpr (!kAlwaysParts<kPair, kMode>)
    if (longest <= kPart<kPair, kMode>) kernel = rfq_ce_kernel<kPair, kMode, kN, false>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
  if (e != cudaSuccess) return e;
  int units = p.share.units;
  if (units > p.share.whole + (p.share.tiles - p.share.whole) * p.share.slices)
    units = p.share.whole + (p.share.tiles - p.share.whole) * p.share.slices;
  return launch_pdl(kernel, dim3(units * kPair), dim3(kThreads), L::kSmem, kPair, stream, maps, p);
}

// Columns of a tile of logits of T rows against n entries: narrow where a row of CTAs then holds them all, because few
// wide tiles leave SMs idle while each CTA waits for its chain of loads.  Measured, narrow against wide: 8 rows, 4096 x
// 1024 11.7 against 14.1 us, 1000 x 4096 27 against 35; 128 rows, 9400 x 4096 33 against 38; two rounds of narrow
// tiles lose what one gains (128 rows, 10000 x 4096 55 against 38).
int tile_columns(int64_t T, int64_t n) { return pair_of(T) == 1 && ceil_div(n, kNarrow) <= kPlanSms ? kNarrow : kBN; }

// A [M] x B [N] product over K; a_ld / b_ld: elements between the rows of the matrix in memory.
template <int kMode>
cudaError_t product(EncodeTiledFn encode, const void* a, int64_t a_ld, const void* b, int64_t b_ld, int64_t M, int64_t N,
                    int64_t K, const Share& share, Params p, cudaStream_t stream, int columns = kBN) {
  constexpr bool kAMn = kMode == kHead;
  constexpr bool kBMn = kMode == kHidden || kMode == kHead;
  const bool pair = pair_of(M) == 2;
  Maps maps;
  const int64_t a_rows = p.term > 0 ? 2 * K : K;
  // Few rows: A's box has no more of them than there are.  The rest of its tile is whatever it was (rows of the
  // product that are not kept); as zeros it took its share of the copies' time (1 row against 131072 x 4096 208 us, not 186).
  const uint32_t box = pair || M > kBM - 8 ? kBM : static_cast<uint32_t>(M + 7) / 8 * 8;
  p.a_bytes = (kAMn ? kBM : box) * kBK * 2;
  const bool ok = (kAMn ? encode_bf16_map(encode, &maps.a, a, a_rows, M, a_ld, kBK) : encode_bf16_map(encode, &maps.a, a, M, K, a_ld, box)) &&
                  (kBMn ? encode_bf16_map(encode, &maps.b, b, K, N, b_ld, kBK)
                        : encode_bf16_map(encode, &maps.b, b, N, K, b_ld, pair ? kBN / 2 : columns));
  if (!ok) return cudaErrorInvalidValue;
  p.M = static_cast<int>(M);
  p.N = static_cast<int>(N);
  p.num_kt = kAMn && p.term > 0 ? 2 : static_cast<int>(ceil_div(K, kBK));
  p.share = share;
  if constexpr (kMode == kLogits || kMode == kGrad)
    if (columns == kNarrow) return launch_mode<1, kMode, kNarrow>(maps, p, stream);
  return pair ? launch_mode<2, kMode, kBN>(maps, p, stream) : launch_mode<1, kMode, kBN>(maps, p, stream);
}

constexpr int64_t kForwardRows = 32768;            // rows of one forward pass, at most (bounds the statistics)
constexpr int64_t kPieceBytes = int64_t(256) << 20;
constexpr int64_t kMinPiece = 2048;

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

// How the backward pass is cut: vocabulary entries per piece, how the dh product is shared out, and
// the offsets of the workspace's parts.
struct Plan {
  int64_t piece, pieces, ld_dz;
  int64_t rows;           // of dz
  Share hidden;
  size_t off_acc, off_slots, off_clean, off_gmax, bytes;
};

Plan plan_backward(int64_t T, int64_t D, int64_t V, bool want_dh, bool want_dw) {
  Plan q;
  q.rows = T <= kTwoTermRows ? 2 * T : T;
  q.piece = kPieceBytes / 2 / q.rows / kBN * kBN;
  if (q.piece < kMinPiece) q.piece = kMinPiece;
  q.pieces = ceil_div(V, q.piece);
  if (q.pieces == 1) q.piece = V;
  else q.piece = ceil_div(ceil_div(V, q.pieces), kBN) * kBN;      // even pieces
  q.pieces = ceil_div(V, q.piece);
  q.ld_dz = (q.piece + 7) / 8 * 8;
  q.hidden = share_out(q.rows, D, q.piece, q.rows > T ? kAllSlots : kCutRest);
  size_t at = align256(static_cast<size_t>(q.rows) * q.ld_dz * 2);
  q.off_acc = at;
  if (want_dh && q.pieces > 1 && q.hidden.whole > 0) at += align256(static_cast<size_t>(T) * D * 4);
  q.off_slots = at;
  if (want_dh) at += static_cast<size_t>(q.hidden.tiles - q.hidden.whole) * q.hidden.slices * (kBM * pair_of(T)) * kBN * 4;
  q.off_clean = at;
  if (want_dw) at += align256(static_cast<size_t>(T) * D * 2);
  q.off_gmax = at;
  q.bytes = at + 256;
  return q;
}

}  // namespace

size_t ce_forward_workspace(int64_t T, int64_t V) {
  const int64_t rows = T < kForwardRows ? T : kForwardRows;
  return align256(static_cast<size_t>(2 * ceil_div(V, tile_columns(rows, V))) * rows * sizeof(float2)) + align256(static_cast<size_t>(rows) * 4);
}

size_t ce_backward_workspace(int64_t T, int64_t D, int64_t V, bool want_dh, bool want_dw) {
  return plan_backward(T, D, V, want_dh, want_dw).bytes;
}

cudaError_t launch_ce_forward(const void* h, const void* w, const int64_t* labels, int64_t T, int64_t D, int64_t V,
                              int64_t ignore, float* loss, float* lse, void* ws, void* encode_tiled, int skip_fill, cudaStream_t stream) {
  EncodeTiledFn encode = reinterpret_cast<EncodeTiledFn>(encode_tiled);
  // Even groups: a last one of few rows would be summed in the parts of few rows (kPart), and the backward pass, which takes all rows at
  // once, would not find the logits that its lse is of (10 % of 1 - p = 1e-3 for logits near 100).
  const int64_t group = ceil_div(T, ceil_div(T, kForwardRows));
  for (int64_t t0 = 0; t0 < T; t0 += group) {
    const int64_t rows = T - t0 < group ? T - t0 : group;
    const int columns = tile_columns(rows, V), parts = static_cast<int>(2 * ceil_div(V, columns));
    Params p = {};
    p.labels = labels + t0;
    p.ignore = ignore;
    p.vocab = V;
    p.stats = static_cast<float2*>(ws);
    p.skip = t0 == 0 ? skip_fill + 1 : 0;
    p.target = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + align256(static_cast<size_t>(parts) * rows * sizeof(float2)));
    cudaError_t e = product<kLogits>(encode, static_cast<const __nv_bfloat16*>(h) + t0 * D, D, w, D, rows, V, D, share_out(rows, V, D, kWhole, columns), p, stream, columns);
    if (e != cudaSuccess) return e;
    e = launch_pdl(rfq_ce_join_kernel, dim3(static_cast<unsigned>(ceil_div(rows, 32))), dim3(32, 32), 0, 1, stream,
                   static_cast<const float2*>(p.stats), static_cast<const float*>(p.target), p.labels, static_cast<int>(rows),
                   parts, ignore, V, loss + t0, lse + t0);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_ce_backward(const void* h, const void* w, const int64_t* labels, const float* lse, const float* dloss,
                               int64_t T, int64_t D, int64_t V, int64_t ignore, void* dh, void* dw, void* ws, void* encode_tiled,
                               int skip_fill, cudaStream_t stream) {
  EncodeTiledFn encode = reinterpret_cast<EncodeTiledFn>(encode_tiled);
  const Plan q = plan_backward(T, D, V, dh != nullptr, dw != nullptr);
  uint8_t* base = static_cast<uint8_t*>(ws);
  __nv_bfloat16* dz = static_cast<__nv_bfloat16*>(ws);
  float* acc = reinterpret_cast<float*>(base + q.off_acc);
  float* slots = reinterpret_cast<float*>(base + q.off_slots);
  float* gmax = reinterpret_cast<float*>(base + q.off_gmax);
  uint4* clean = reinterpret_cast<uint4*>(base + q.off_clean);
  const int64_t copies = dw == nullptr ? 0 : ceil_div(T * ceil_div(D / 8, kCopyRun), 32);   // blocks of 32 warps, at most two of them an SM
  cudaError_t e = launch_pdl(rfq_ce_prepare_kernel, dim3(static_cast<unsigned>(1 + (copies < 2 * kPlanSms ? copies : 2 * kPlanSms))), dim3(1024), 0, 1, stream, dloss,
                             labels, static_cast<int>(T), ignore, gmax, static_cast<const uint4*>(h), clean, static_cast<int>(D / 8));
  for (int64_t v0 = 0; v0 < V && e == cudaSuccess; v0 += q.piece) {
    const int64_t n = V - v0 < q.piece ? V - v0 : q.piece;
    const __nv_bfloat16* wp = static_cast<const __nv_bfloat16*>(w) + v0 * D;
    Params p = {};
    p.labels = labels;
    p.ignore = ignore;
    p.vocab = V;
    p.v0 = v0;
    p.lse = lse;
    p.dloss = dloss;
    p.gmax = gmax;
    p.dz = dz;
    p.ld_dz = q.ld_dz;
    p.term = q.rows > T ? static_cast<int>(T) : 0;
    const int columns = tile_columns(T, n);
    p.skip = v0 == 0 ? skip_fill + 1 : 0;
    e = product<kGrad>(encode, h, D, wp, D, T, n, D, share_out(T, n, D, kWhole, columns), p, stream, columns);
    p.skip = 0;
    if (e == cudaSuccess && dh != nullptr) {
      p.acc = acc;
      p.slots = slots;
      p.accumulate = v0 > 0;
      p.out = q.pieces == 1 ? static_cast<__nv_bfloat16*>(dh) : nullptr;
      e = product<kHidden>(encode, dz, q.ld_dz, wp, D, q.rows, D, n, q.hidden, p, stream);
    }
    if (e == cudaSuccess && dw != nullptr) {
      p.out = static_cast<__nv_bfloat16*>(dw) + v0 * D;
      e = product<kHead>(encode, dz, q.ld_dz, clean, D, n, D, T, share_out(n, D, T, kWhole), p, stream);
    }
  }
  // Tiles of dh still in fp32: all of them after several pieces, else the rest.
  const int tile0 = q.pieces > 1 ? 0 : q.hidden.whole;
  if (e == cudaSuccess && dh != nullptr && tile0 < q.hidden.tiles) {
    const int tile_rows = kBM * pair_of(T);
    e = launch_pdl(rfq_ce_hidden_kernel, dim3(static_cast<unsigned>((q.hidden.tiles - tile0) * (tile_rows / 4))), dim3(256), 0, 1, stream,
                   q.hidden, tile0, tile_rows, static_cast<const float*>(acc), static_cast<const float*>(slots),
                   static_cast<const float*>(gmax), static_cast<int>(T), static_cast<int>(D), q.rows > T ? static_cast<int>(T) : 0,
                   static_cast<__nv_bfloat16*>(dh));
  }
  return e;
}

cudaError_t read_and_clear_ce_error(unsigned int* value) {
  unsigned int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(value, g_ce_error, sizeof(unsigned int));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(g_ce_error, &zero, sizeof(unsigned int));
}

}  // namespace rfq
