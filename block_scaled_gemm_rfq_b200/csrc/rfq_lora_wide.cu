// rfq_lora_wide.cu -- the adapters' products over long batches, on tcgen05.
//
//   shrink   s[m] = scale_a P_a src[m]      rows x wide -> rank
//   expand   out[m] = base[m] + Q_a s[m]    rank -> wide
//   outer    dA, dB                         contraction over rows
//
// (rfq_lora.cu has the operator; P, Q = A, B going forward and B^T, A^T going back.)  All are
// bound by memory: 2 r flops for each element of src, or of base and out, with r <= 128.  What
// the tensor cores buy here is instructions: with warp-level MMAs a [64 x 128] tile of expand
// took 7400 warp instructions and ran at 0.7 TB/s; one thread's tcgen05.mma replaces the
// fragment loads and MMAs of a whole tile, and the epilogue's thread owns a row.
//
// One CTA works on a chunk of 128 neighbouring rows.  A product is formed for all 128 rows once
// for each adapter that the chunk holds, and each row keeps the result of its own: rows of an
// MMA do not mix, so no row is gathered and nothing leaks between rows.  Chunks of one
// adapter, the rule in prompts and training, cost one pass.  (Short batches, where rows
// have adapters of their own, take the kernels of rfq_lora.cu.)
//
// shrink: the contraction is split over a cluster of up to 8 CTAs, whose partial sums are added
// through distributed shared memory in the order of the ranks.  The accumulator takes 256
// elements of the contraction at a time (the tensor cores add by truncation) and the epilogue adds those
// parts with rounding.  shrink leaves s as bf16 terms (two, 16 bits, for a bf16 output; three, 24 bits, for an
// fp32 one), which are expand's operand as they are.
// expand: base tiles come in by TMA (by a warp of its own: behind the loads of Q in one queue, chunks of two
// adapters held the base back and cost 1.3 times those of one), are added to in shared memory and leave from
// there by TMA.
//
// 16384 rows of one adapter of rank 16, 4096 -> 4096: both products 81 us, of which reading src and base and writing
// out needs 63 (402 MB); alone shrink takes 36 us (134 MB, 3.8 TB/s: some 9 us of it are start, first loads and the
// cluster's exchange) and expand 45 (268 MB, 6 TB/s).  4096 rows of 8 adapters of rank 64, 4096 -> 12288: 61 us where
// chunks hold one adapter (floor 39), 65 to 68 where requests end inside them, which are then passed over twice.  What a chunk
// holds decides: in random order 16384 rows of 8, 16, 64 adapters of rank 16 take 362, 680 and 2220 us, sorted 96, 98 and 106.
// Stages of 128 elements of the contraction in shrink, for longer pieces of a row, were no faster.
//
// Roles: warp 0 TMA producer, warp 1 MMA issuer, the others epilogue.  Every wait on an mbarrier
// is bounded (rfq_ptx.cuh); after one that ran out the epilogue runs through its loops without
// waiting, so that no warp is left alone at a barrier.  No TMA multicast.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "rfq_internal.h"
#include "rfq_ptx.cuh"
#include "rfq_terms.cuh"
#include "rfq_tmap.h"

namespace rfq {

__device__ unsigned int g_lora_error = 0;

namespace {

constexpr int kChunk = 128;
constexpr uint32_t kBox = kChunk * 128;    // 128 rows of 128 bytes
constexpr uint32_t kSmemLimit = 232448;
constexpr int kMaxStages = 8;
// k-tiles of 64 per accumulation.  Whatever the results' types, so that s does not depend on them (16 were no faster).
constexpr int kPartTiles = 4;

// Shared-memory operand descriptors, 128-byte swizzle (K-major: 8-row groups 1024 bytes apart;
// M/N-major: chunks of 64 elements `lead` bytes apart, 8 contraction rows 1024 bytes apart).
__device__ __forceinline__ uint64_t k_major_desc(uint32_t addr) {
  return ((addr >> 4) & 0x3FFFull) | (1ull << 16) | ((1024ull >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ uint64_t mn_major_desc(uint32_t addr, uint32_t lead) {
  return ((addr >> 4) & 0x3FFFull) | (static_cast<uint64_t>(lead >> 4) << 16) | ((1024ull >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
// kind::f16, bf16 operands, fp32 accumulator, M = 128.
__device__ __forceinline__ uint32_t idesc(uint32_t n, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (uint32_t(b_mn) << 16) | ((n >> 3) << 17) | ((128u >> 4) << 24);
}

// The adapters of a chunk in the order of their first rows.  A warp's lanes hold the 128 ids (lane + 32 i)
// and the list (adapter d in lane d % 32, word d / 32), so that a look is one shuffle; all lanes of
// the warp call these together.
struct Adapters {
  int id[4];
  int list[4];
  int count;
  __device__ __forceinline__ void load(const int* ids, int64_t row0, int64_t M, int n) {
    const int lane = threadIdx.x & 31;
    unsigned left = 0;   // bit i: row lane + 32 i not yet taken
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t row = row0 + lane + 32 * i;
      const int v = row < M ? ids[row] : -1;
      id[i] = v >= 0 && v < n ? v : -1;
      left |= static_cast<unsigned>(id[i] >= 0) << i;
    }
    count = 0;
    while (true) {
      int a = -1;
#pragma unroll
      for (int i = 3; i >= 0; --i) {
        const unsigned m = __ballot_sync(0xffffffffu, left >> i & 1u);
        const int v = __shfl_sync(0xffffffffu, id[i], m ? __ffs(m) - 1 : 0);
        if (m) a = v;
      }
      if (a < 0) break;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (id[i] == a) left &= ~(1u << i);
        if (lane == (count & 31) && i == count >> 5) list[i] = a;
      }
      ++count;
    }
  }
  __device__ __forceinline__ int at(int d) const {
    const int w = d >> 5;
    return __shfl_sync(0xffffffffu, w == 0 ? list[0] : w == 1 ? list[1] : w == 2 ? list[2] : list[3], d & 31);
  }
};

struct Cursor {
  uint32_t stage = 0, phase = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++stage == static_cast<uint32_t>(stages)) {
      stage = 0;
      phase ^= 1u;
    }
  }
};

// A producer thread's record of what it has asked for, to wait for at the end.
struct Filled {
  uint32_t mask = 0, last = 0;
  __device__ __forceinline__ void add(const Cursor& c) {
    mask |= 1u << c.stage;
    last = (last & ~(1u << c.stage)) | (c.phase << c.stage);
  }
  __device__ __forceinline__ void drain(uint64_t* full, int stages) {
    for (int s = 0; s < stages; ++s)
      if (mask & (1u << s)) {
        int never = 0;
        mbar_wait(&full[s], (last >> s) & 1u, &never, &g_lora_error, kErrWaitDrain);
      }
  }
};

// ---------------------------------------------------------------- shrink
struct ShrinkMaps {
  CUtensorMap src, p;
};
struct ShrinkParams {
  const int* ids;
  const float* scale;
  float* s;                // [M][r] or nullptr
  __nv_bfloat16* terms;    // [M][num_terms][r]: s as a sum of bf16 terms
  int num_terms;
  int* counts;             // [chunks]
  int64_t M;
  int n, r, kt, kt_per_rank, cluster, stages;
};

constexpr int kShrinkThreads = 192;   // TMA, MMA, four epilogue warps

__host__ __device__ constexpr uint32_t shrink_p_bytes(bool trans, int r) {
  const uint32_t r16 = (r + 15) / 16 * 16;
  return trans ? (r > 64 ? 2u : 1u) * 64u * 128u : r16 * 128u;
}
__host__ __device__ constexpr uint32_t shrink_sum_bytes(int r) { return kChunk * (r + 4) * 4; }

template <bool kTrans>
__global__ void __launch_bounds__(kShrinkThreads) rfq_lora_shrink_wide_kernel(const __grid_constant__ ShrinkMaps maps,
                                                                              const ShrinkParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], drained;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t r16 = (p.r + 15) / 16 * 16;
  const uint32_t stage_bytes = kBox + shrink_p_bytes(kTrans, p.r);
  const uint32_t acc_cols = r16 <= 32 ? 32 : r16 <= 64 ? 64 : 128;
  float* sums = reinterpret_cast<float*>(smem + p.stages * stage_bytes);   // [128][r + 4]
  volatile int* abort_flag = &abort_word;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 4);
    }
    mbar_init(&drained, 1);
    abort_word = 0;
    fence_mbar_init();
    prefetch_tmap(&maps.src);
    prefetch_tmap(&maps.p);
  }
  if (warp == 1) {
    tmem_alloc_g<1>(&tmem_slot, 2 * acc_cols);
    tmem_relinquish_g<1>();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  griddep_launch_dependents();
  griddep_wait();

  const uint32_t rank = cluster_cta_rank();
  const int64_t row0 = static_cast<int64_t>(blockIdx.x / p.cluster) * kChunk;
  const int kt0 = static_cast<int>(rank) * p.kt_per_rank;
  const int kt1 = min(p.kt, kt0 + p.kt_per_rank);
  Adapters walk;
  walk.load(p.ids, row0, p.M, p.n);
  if (rank == 0 && threadIdx.x == 0) p.counts[row0 / kChunk] = walk.count;

  if (warp == 0) {
    Cursor c;
    Filled filled;
    bool ok = true;
    for (int d = 0; d < walk.count && ok; ++d) {
      const int a = walk.at(d);
      if (lane == 0) {
        for (int kt = kt0; kt < kt1; ++kt) {
          ok = mbar_wait(&empty[c.stage], c.phase ^ 1u, abort_flag, &g_lora_error, kErrWaitEmpty);
          if (!ok) break;
          uint8_t* sx = smem + c.stage * stage_bytes;
          mbar_arrive_expect_tx(&full[c.stage], stage_bytes);
          tma_load_2d(sx, &maps.src, &full[c.stage], kt * 64, static_cast<int>(row0));
          if constexpr (kTrans) {
            tma_load_3d(sx + kBox, &maps.p, &full[c.stage], 0, kt * 64, a);
            if (p.r > 64) tma_load_3d(sx + kBox + 64 * 128, &maps.p, &full[c.stage], 64, kt * 64, a);
          } else {
            tma_load_3d(sx + kBox, &maps.p, &full[c.stage], kt * 64, 0, a);
          }
          filled.add(c);
          c.next(p.stages);
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
    }
    if (lane == 0) filled.drain(full, p.stages);
    __syncwarp();
  } else if (warp == 1) {
    Cursor c, acc;
    bool ok = true;
    const uint32_t id = idesc(r16, kTrans);
    for (int pass = 0; pass < walk.count && ok; ++pass) {
      if (lane == 0) {
        for (int kp = kt0; kp < kt1 && ok; kp += kPartTiles) {
          ok = mbar_wait(&acc_empty[acc.stage], acc.phase ^ 1u, abort_flag, &g_lora_error, kErrWaitAccEmpty);
          if (!ok) break;
          tc_fence_after();
          const uint32_t d = tmem + acc.stage * acc_cols;
          for (int kt = kp; kt < min(kp + kPartTiles, kt1); ++kt) {
            ok = mbar_wait(&full[c.stage], c.phase, abort_flag, &g_lora_error, kErrWaitFull);
            if (!ok) break;
            tc_fence_after();
            const uint32_t sx = smem_addr(smem) + c.stage * stage_bytes, sp = sx + kBox;
            const uint64_t da = k_major_desc(sx);
            const uint64_t db = kTrans ? mn_major_desc(sp, 64 * 128) : k_major_desc(sp);
#pragma unroll
            for (uint32_t q = 0; q < 4; ++q)
              mma_bf16_g<1>(d, da + 2 * q, db + (kTrans ? 128 : 2) * q, id, (kt != kp || q != 0) ? 1u : 0u);
            tc_commit(&empty[c.stage]);
            c.next(p.stages);
          }
          if (!ok) break;
          tc_commit(&acc_full[acc.stage]);
          acc.next(2);
        }
        if (!ok) {   // teardown after an abort: wait for the MMAs already issued
          tc_commit(&drained);
          int never = 0;
          mbar_wait(&drained, 0, &never, &g_lora_error, kErrWaitDrain);
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
    }
    __syncwarp();
  } else {
    const int quad = warp & 3;
    const int row = quad * 32 + lane;
    const int mine = walk.id[0] * (quad == 0) + walk.id[1] * (quad == 1) + walk.id[2] * (quad == 2) + walk.id[3] * (quad == 3);
    float* out = sums + row * (p.r + 4);
    Cursor acc;
    for (int d = 0; d < walk.count; ++d) {
      const int a = walk.at(d);
      for (int kp = kt0; kp < kt1; kp += kPartTiles) {
        mbar_wait(&acc_full[acc.stage], acc.phase, abort_flag, &g_lora_error, kErrWaitAccFull, 2 * kWaitLimitNs);
        tc_fence_after();
        __syncwarp();
        const uint32_t at = tmem + (static_cast<uint32_t>(quad * 32) << 16) + acc.stage * acc_cols;
        for (int j = __any_sync(0xffffffffu, mine == a) ? 0 : p.r; j < p.r; j += 8) {
          uint32_t v[8];
          tmem_load_32x32b_x8(at + j, v);
          tmem_wait_ld();
          if (mine == a) {
            float4* o = reinterpret_cast<float4*>(out + j);
            float4 x = make_float4(__uint_as_float(v[0]), __uint_as_float(v[1]), __uint_as_float(v[2]), __uint_as_float(v[3]));
            float4 y = make_float4(__uint_as_float(v[4]), __uint_as_float(v[5]), __uint_as_float(v[6]), __uint_as_float(v[7]));
            if (kp != kt0) {
              const float4 u = o[0], w = o[1];
              x.x += u.x; x.y += u.y; x.z += u.z; x.w += u.w;
              y.x += w.x; y.y += w.y; y.z += w.z; y.w += w.w;
            }
            o[0] = x;
            o[1] = y;
          }
          __syncwarp();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&acc_empty[acc.stage]);
        acc.next(2);
      }
    }
  }

  // Each rank adds the cluster's sums for its share of the rows, in the order of the ranks.
  __syncwarp();
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc_g<1>(tmem, 2 * acc_cols);
  }
  const int rows = kChunk / p.cluster, r4 = p.r / 4;
  const uint32_t sums_addr = smem_addr(sums);
  for (int i = threadIdx.x; i < rows * r4; i += kShrinkThreads) {
    const int m = static_cast<int>(rank) * rows + i / r4, j = i % r4 * 4;
    const int64_t row = row0 + m;
    if (row >= p.M) continue;
    const int a = p.ids[row];
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (a >= 0 && a < p.n) {
      const uint32_t at = sums_addr + (m * (p.r + 4) + j) * 4;
      for (int k = 0; k < p.cluster; ++k) {
        const float4 u = ld_shared_cluster_f32x4(map_to_cta(at, k));
        v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
      }
      const float w = p.scale[a];
      v.x *= w; v.y *= w; v.z *= w; v.w *= w;
    }
    if (p.s != nullptr) *reinterpret_cast<float4*>(p.s + row * p.r + j) = v;
    __nv_bfloat16* t = p.terms + row * p.num_terms * p.r + j;
    for (int e = 0; e < p.num_terms; ++e) {   // 8 bits each
      const __nv_bfloat162 lo = {take_term(v.x), take_term(v.y)}, hi = {take_term(v.z), take_term(v.w)};
      *reinterpret_cast<uint2*>(t + e * p.r) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    }
  }
  __syncwarp();     // rows past the end left the loop body early; the barrier takes whole warps
  cluster_sync();   // the others may still be reading this CTA's sums
}

// ---------------------------------------------------------------- expand
struct ExpandMaps {
  CUtensorMap s, q, base, out;
};
struct ExpandParams {
  const int* ids;
  int64_t M;
  int C;
  int n, r;
  int has_base, in_place;
  int tiles;               // column tiles
  int unit_tiles, col_units;   // without counts: tiles of a unit, units along the columns
  int64_t units;
  int64_t chunks;
  const int* counts;       // [chunks]: adapters of each, from shrink, or nullptr
  int s_stages, base_stages, q_stages;
};

constexpr int kExpandThreads = 352;    // TMA of s and Q, MMA, eight epilogue warps, TMA of the base
constexpr int kBaseWarp = 10;
constexpr int kAccs = 4;               // accumulators of 128 columns in tensor memory
// Columns of a tile: 256 bytes of a row, two boxes of 128 bytes.
template <bool kF32>
constexpr int kCols = kF32 ? 64 : 128;
// Bf16 terms in which s enters the MMA, as in short batches (kExpandTerms in rfq_lora.cu): one term would add an error as
// large as a bf16 output's own rounding, in the same direction for a whole row.  The second costs 1 to 5 % (both products of 4096
// rows, 4096 -> 12288: rank 16 51.8 -> 52.0 us, rank 128 84.4 -> 86.1, 8 requests of rank 64 63 -> 66).
template <bool kF32>
constexpr int kTerms = kF32 ? 3 : 2;

// What a CTA works on: runs of column tiles of one chunk each.
// With one adapter (or where shrink left no counts) all chunks are alike: units of 4 to 16 tiles go round the CTAs.
// Else a chunk is passed over once for each adapter in it, and the tiles of all chunks, one chunk after the other, are
// cut into one part for each CTA, of equal work: 2 for a tile and 3 for each pass over it (a tile of two adapters took
// 1.6 times the time of one).  Measured with s in one term, both products of 4096 rows of 8 requests that end inside chunks, rank 64,
// 4096 -> 12288: 61 to 66 us with parts against 70 to 79 with units; 8 requests of 512 rows each 58 against 55; one
// adapter 55 against 53.
struct Place {
  int64_t chunk;
  int tile;
};
__device__ __forceinline__ int tile_work(const ExpandParams& p, int64_t chunk) {
  const int c = p.counts[chunk];
  return c == 0 && p.in_place ? 0 : 2 + 3 * c;
}
// Where this CTA's part begins and ends (end: the first tile that is not its own).  Every warp finds it for itself.
__device__ __forceinline__ void cut_part(const ExpandParams& p, Place& begin, Place& end) {
  const int lane = threadIdx.x & 31;
  const int64_t per = (p.chunks + 31) / 32, first = min(p.chunks, lane * per), last = min(p.chunks, first + per);
  int64_t sum = 0;
#pragma unroll 4
  for (int64_t c = first; c < last; ++c) sum += tile_work(p, c);
  int64_t upto = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t o = __shfl_up_sync(0xffffffffu, upto, d);
    if (lane >= d) upto += o;
  }
  const uint64_t total = __shfl_sync(0xffffffffu, upto, 31) * p.tiles, each = total / gridDim.x, more = total - each * gridDim.x;
  const int64_t before = (upto - sum) * p.tiles;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const uint64_t b = blockIdx.x + e;
    const int64_t at = static_cast<int64_t>(b * each + min(b, more));
    const bool mine = at >= before && at < before + sum * p.tiles;
    Place found = {p.chunks, 0};   // the end of the last run, or nothing to do at all
    if (mine) {
      int64_t from = before;
      for (int64_t c = first; c < last; ++c) {
        const int w = tile_work(p, c);
        const int64_t next = from + static_cast<int64_t>(w) * p.tiles;
        if (at < next) {
          found = {c, (static_cast<int>(at - from) + w - 1) / w};
          if (found.tile == p.tiles) found = {c + 1, 0};   // so that a part has no empty run but the last
          break;
        }
        from = next;
      }
    }
    const unsigned who = __ballot_sync(0xffffffffu, mine);
    const int source = who != 0 ? __ffs(who) - 1 : 0;
    Place& place = e == 0 ? begin : end;
    place.chunk = __shfl_sync(0xffffffffu, found.chunk, source);
    place.tile = __shfl_sync(0xffffffffu, found.tile, source);
  }
}

struct Runs {
  Place begin, end;
  int64_t at;   // the next chunk of the part, or the next unit
  __device__ __forceinline__ explicit Runs(const ExpandParams& p) {
    if (p.counts != nullptr) {
      cut_part(p, begin, end);
      at = begin.chunk;
    } else {
      at = blockIdx.x;
    }
  }
  __device__ __forceinline__ bool next(const ExpandParams& p, int64_t& row0, int& t0, int& t1) {
    if (p.counts != nullptr) {
      if (at > end.chunk) return false;
      t0 = at == begin.chunk ? begin.tile : 0;
      t1 = at == end.chunk ? end.tile : p.tiles;
      row0 = at++ * kChunk;
      return t0 < t1;
    }
    if (at >= p.units) return false;
    row0 = at / p.col_units * kChunk;
    t0 = static_cast<int>(at % p.col_units) * p.unit_tiles;
    t1 = min(p.tiles, t0 + p.unit_tiles);
    at += gridDim.x;
    return true;
  }
};

template <bool kTrans, bool kF32>
__host__ __device__ constexpr uint32_t expand_q_bytes(int r) {
  const uint32_t r16 = (r + 15) / 16 * 16;
  return kTrans ? kCols<kF32> / 64 * r16 * 128u : (r > 64 ? 2u : 1u) * kCols<kF32> * 128u;
}
template <bool kF32>
__host__ __device__ constexpr uint32_t expand_s_bytes(int r) {
  return (r > 64 ? 2u : 1u) * kTerms<kF32> * kBox;
}

template <bool kTrans, bool kF32>
__global__ void __launch_bounds__(kExpandThreads, 1) rfq_lora_expand_wide_kernel(const __grid_constant__ ExpandMaps maps,
                                                                                 const ExpandParams p) {
  constexpr int kT = kTerms<kF32>;
  constexpr int kN = kCols<kF32>;
  constexpr int kBoxCols = kN / 2;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t b_full[kMaxStages], b_empty[kMaxStages], q_full[kMaxStages], q_empty[kMaxStages], acc_full[kAccs], acc_empty[kAccs],
      s_full[2], s_empty[2], drained;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  volatile int* abort_flag = &abort_word;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t r16 = (p.r + 15) / 16 * 16;
  const uint32_t q_bytes = expand_q_bytes<kTrans, kF32>(p.r);
  const uint32_t s_bytes = expand_s_bytes<kF32>(p.r);
  uint8_t* s_mem = smem;                                           // [r / 64][term][128 rows x 128 bytes]
  uint8_t* b_mem = s_mem + p.s_stages * s_bytes;                   // base tiles: two boxes each
  uint8_t* q_mem = b_mem + p.base_stages * 2 * kBox;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(&b_full[s], 1);
      mbar_init(&b_empty[s], 1);
      mbar_init(&q_full[s], 1);
      mbar_init(&q_empty[s], 1);
    }
    for (int b = 0; b < kAccs; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 8);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&s_full[b], 1);
      mbar_init(&s_empty[b], 1);
    }
    mbar_init(&drained, 1);
    abort_word = 0;
    fence_mbar_init();
    prefetch_tmap(&maps.s);
    prefetch_tmap(&maps.q);
    prefetch_tmap(&maps.base);
    prefetch_tmap(&maps.out);
  }
  if (warp == 1) {
    tmem_alloc_g<1>(&tmem_slot, kAccs * 128);
    tmem_relinquish_g<1>();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  griddep_launch_dependents();
  griddep_wait();

  // Where a chunk has no adapter and the base is the output, there is nothing to do; every role finds that out
  // for itself.
  Runs runs(p);
  int64_t row0;
  int t0, t1;
  Adapters walk;
  if (warp == 0) {
    Cursor sc, qc;
    Filled s_filled, q_filled;
    bool ok = true;
    while (ok && runs.next(p, row0, t0, t1)) {
      walk.load(p.ids, row0, p.M, p.n);
      if (walk.count == 0) continue;
      if (lane == 0) {
        ok = mbar_wait(&s_empty[sc.stage], sc.phase ^ 1u, abort_flag, &g_lora_error, kErrWaitEmpty);
        if (ok) {
          uint8_t* ss = s_mem + sc.stage * s_bytes;
          mbar_arrive_expect_tx(&s_full[sc.stage], s_bytes);
          for (int k = 0; k < p.r; k += 64)
            for (int e = 0; e < kT; ++e)
              tma_load_3d(ss + ((k >> 6) * kT + e) * kBox, &maps.s, &s_full[sc.stage], k, e, static_cast<int>(row0));
          s_filled.add(sc);
          sc.next(p.s_stages);
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      for (int t = t0; t < t1 && ok; ++t) {
        const int col = t * kN;
        for (int d = 0; d < walk.count && ok; ++d) {
          const int a = walk.at(d);
          if (lane == 0) {
            ok = mbar_wait(&q_empty[qc.stage], qc.phase ^ 1u, abort_flag, &g_lora_error, kErrWaitEmpty);
            if (ok) {
              uint8_t* sq = q_mem + qc.stage * q_bytes;
              mbar_arrive_expect_tx(&q_full[qc.stage], q_bytes);
              if constexpr (kTrans) {
#pragma unroll
                for (int c = 0; c < kN / 64; ++c) tma_load_3d(sq + c * r16 * 128, &maps.q, &q_full[qc.stage], col + 64 * c, 0, a);
              } else {
                tma_load_3d(sq, &maps.q, &q_full[qc.stage], 0, col, a);
                if (p.r > 64) tma_load_3d(sq + kN * 128, &maps.q, &q_full[qc.stage], 64, col, a);
              }
              q_filled.add(qc);
              qc.next(p.q_stages);
            }
          }
          ok = __shfl_sync(0xffffffffu, ok, 0);
        }
      }
    }
    if (lane == 0) {
      s_filled.drain(s_full, p.s_stages);
      q_filled.drain(q_full, p.q_stages);
    }
    __syncwarp();
  } else if (warp == kBaseWarp) {
    Cursor bc;
    Filled b_filled;
    bool ok = p.has_base != 0;
    while (ok && runs.next(p, row0, t0, t1)) {
      if (p.in_place) {
        walk.load(p.ids, row0, p.M, p.n);
        if (walk.count == 0) continue;
      }
      if (lane == 0) {
        for (int t = t0; t < t1; ++t) {
          ok = mbar_wait(&b_empty[bc.stage], bc.phase ^ 1u, abort_flag, &g_lora_error, kErrWaitEmpty);
          if (!ok) break;
          const int col = t * kN;
          uint8_t* sb = b_mem + bc.stage * 2 * kBox;
          mbar_arrive_expect_tx(&b_full[bc.stage], 2 * kBox);
          tma_load_2d(sb, &maps.base, &b_full[bc.stage], col, static_cast<int>(row0));
          tma_load_2d(sb + kBox, &maps.base, &b_full[bc.stage], col + kBoxCols, static_cast<int>(row0));
          b_filled.add(bc);
          bc.next(p.base_stages);
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
    }
    if (lane == 0) b_filled.drain(b_full, p.base_stages);
    __syncwarp();
  } else if (warp == 1) {
    Cursor sc, qc, acc;
    int last = -1;
    uint32_t last_phase = 0;
    bool ok = true;
    const uint32_t id = idesc(kN, kTrans);
    while (ok && runs.next(p, row0, t0, t1)) {
      walk.load(p.ids, row0, p.M, p.n);
      if (walk.count == 0) continue;
      if (lane == 0) {
        ok = mbar_wait(&s_full[sc.stage], sc.phase, abort_flag, &g_lora_error, kErrWaitFull);
        tc_fence_after();
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      for (int t = t0; t < t1 && ok; ++t) {
        for (int pass = 0; pass < walk.count && ok; ++pass) {
          if (lane == 0) {
            ok = mbar_wait(&acc_empty[acc.stage], acc.phase ^ 1u, abort_flag, &g_lora_error, kErrWaitAccEmpty) &&
                 mbar_wait(&q_full[qc.stage], qc.phase, abort_flag, &g_lora_error, kErrWaitFull);
            if (ok) {
              tc_fence_after();
              const uint32_t d = tmem + acc.stage * 128;
              const uint32_t sq = smem_addr(q_mem) + qc.stage * q_bytes, sa = smem_addr(s_mem) + sc.stage * s_bytes;
              uint32_t more = 0;
              for (uint32_t k = 0; k < r16 / 16; ++k) {
                const uint64_t db = kTrans ? mn_major_desc(sq, r16 * 128) + 128 * k : k_major_desc(sq + (k >> 2) * kN * 128) + 2 * (k & 3);
#pragma unroll
                for (int e = kT - 1; e >= 0; --e) {   // smallest terms first
                  mma_bf16_g<1>(d, k_major_desc(sa + ((k >> 2) * kT + e) * kBox) + 2 * (k & 3), db, id, more);
                  more = 1;
                }
              }
              tc_commit(&q_empty[qc.stage]);
              tc_commit(&acc_full[acc.stage]);
            }
            qc.next(p.q_stages);
            acc.next(kAccs);
          }
          ok = __shfl_sync(0xffffffffu, ok, 0);
        }
      }
      if (lane == 0) {
        if (ok) {
          tc_commit(&s_empty[sc.stage]);   // with the last MMA of the unit
          last = static_cast<int>(sc.stage);
          last_phase = sc.phase;
        } else {                           // teardown after an abort: wait for the MMAs already issued
          tc_commit(&drained);
          int never = 0;
          mbar_wait(&drained, 0, &never, &g_lora_error, kErrWaitDrain);
        }
      }
      sc.next(p.s_stages);
    }
    // The last commit arrives on a barrier of this CTA: it has done so before the CTA leaves.
    if (lane == 0 && ok && last >= 0) {
      int never = 0;
      mbar_wait(&s_empty[last], last_phase, &never, &g_lora_error, kErrWaitDrain);
    }
    __syncwarp();
  } else {
    const int quad = warp & 3, half = (warp - 2) >> 2;
    const int row = quad * 32 + lane;
    Cursor bc, acc;
    int release = -1;   // the stage whose tile may still be on its way out
    while (runs.next(p, row0, t0, t1)) {
      walk.load(p.ids, row0, p.M, p.n);
      const bool any = walk.count > 0;
      if (!any && p.in_place) continue;
      const int mine = quad == 0 ? walk.id[0] : quad == 1 ? walk.id[1] : quad == 2 ? walk.id[2] : walk.id[3];
      for (int t = t0; t < t1; ++t) {
        if (p.has_base) mbar_wait(&b_full[bc.stage], bc.phase, abort_flag, &g_lora_error, kErrWaitFull, 2 * kWaitLimitNs);
        uint8_t* sb = b_mem + bc.stage * 2 * kBox;
        uint8_t* line = sb + half * kBox + row * 128;
        if (!p.has_base) {
          // The stage is free once its last tile has left (one thread waits, all learn of it at the barrier).
          if (threadIdx.x == 64 && release >= 0) bulk_wait_read_all();
          __syncwarp();
          asm volatile("bar.sync 1, 256;" ::: "memory");
          if (mine < 0)
#pragma unroll
            for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4*>(line + c * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
        for (int d = 0; d < walk.count; ++d) {
          const int a = walk.at(d);
          mbar_wait(&acc_full[acc.stage], acc.phase, abort_flag, &g_lora_error, kErrWaitAccFull, 2 * kWaitLimitNs);
          tc_fence_after();
          __syncwarp();
          const uint32_t at = tmem + (static_cast<uint32_t>(quad * 32) << 16) + acc.stage * 128 + half * kBoxCols;
          const bool here = __any_sync(0xffffffffu, mine == a);   // these 32 rows have the adapter
#pragma unroll
          for (int g = 0; g < kBoxCols / 32; ++g) {
            if (!here) break;
            uint32_t v[32];
            tmem_load_32x32b_x32(at + 32 * g, v);
            tmem_wait_ld();
            if (mine == a) {
              if constexpr (kF32) {
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                  float4* o = reinterpret_cast<float4*>(line + (c ^ (row & 7)) * 16);
                  float4 f = make_float4(__uint_as_float(v[4 * c]), __uint_as_float(v[4 * c + 1]), __uint_as_float(v[4 * c + 2]),
                                         __uint_as_float(v[4 * c + 3]));
                  if (p.has_base) {
                    const float4 b = *o;
                    f.x += b.x; f.y += b.y; f.z += b.z; f.w += b.w;
                  }
                  *o = f;
                }
              } else {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                  uint4* o = reinterpret_cast<uint4*>(line + ((4 * g + c) ^ (row & 7)) * 16);
                  uint32_t w[4] = {0u, 0u, 0u, 0u};
                  if (p.has_base) {
                    const uint4 b = *o;
                    w[0] = b.x; w[1] = b.y; w[2] = b.z; w[3] = b.w;
                  }
#pragma unroll
                  for (int h = 0; h < 4; ++h) {
                    const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(w[h] << 16) + __uint_as_float(v[8 * c + 2 * h]),
                                                                   __uint_as_float(w[h] & 0xffff0000u) + __uint_as_float(v[8 * c + 2 * h + 1]));
                    w[h] = *reinterpret_cast<const uint32_t*>(&b);
                  }
                  *o = make_uint4(w[0], w[1], w[2], w[3]);
                }
              }
            }
            __syncwarp();
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&acc_empty[acc.stage]);
          acc.next(kAccs);
        }
        fence_proxy_async_smem();
        __syncwarp();
        asm volatile("bar.sync 1, 256;" ::: "memory");
        if (threadIdx.x == 64) {
          if (*abort_flag == 0) {
            const int col = t * kN;
            tma_store_2d(&maps.out, sb, col, static_cast<int>(row0));
            if (col + kBoxCols < p.C) tma_store_2d(&maps.out, sb + kBox, col + kBoxCols, static_cast<int>(row0));
          }
          bulk_commit_group();
          if (p.has_base) {
            bulk_wait_read_but_one();
            if (release >= 0) mbar_arrive(&b_empty[release]);
          }
        }
        release = static_cast<int>(bc.stage);
        bc.next(p.base_stages);
      }
    }
    if (threadIdx.x == 64) bulk_wait_all();
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc_g<1>(tmem, kAccs * 128);
  }
}

// ---------------------------------------------------------------- outer
// part[range][a][j][c] = sum over the range's rows of adapter a of v[m][j] w[m][c] for the two pairs (v, w) =
// (ds', x) and (s', dy): products that contract over rows, v^T (rank along M, padded to 128) by w (256
// columns along N), both M/N-major.  A CTA sorts its range's rows by adapter (a check where they are neighbours)
// and takes 64 of one adapter a stage: by TMA where they are neighbours, else gathered (the last ones of an adapter too)
// with 16-byte asynchronous copies that lay down the 128-byte swizzle themselves and zeros behind the last.  So rows
// of other adapters never enter a product, in whatever order they come.  Bound by reading x and dy: 8192
// rows, 4096 -> 12288, rank 64 (268 MB) take 64 us, 4.3 TB/s with the tensor pipe 70 % active, 100 us less than on
// warp-level MMAs.  Two terms of up to rank 64 in the two halves of one MMA's M: half the MMAs, but twice the partial
// sums, 147 against 142 us for the whole backward pass.  Seven copy warps for rows that are not neighbours: those 7 %
// faster, neighbours 2 to 4 % slower.
// Roles: warps 0..2 copies, warp 3 MMA issuer, warps 4..11 epilogue (128 columns of a row of the rank each thread).
struct OuterMaps {
  CUtensorMap v[2], w[2];     // of the sides; boxes of 64 elements x 64 rows
};
struct OuterSide {
  const __nv_bfloat16* v;     // [M][ld]: terms of r each, kT or more
  int ld;
  const __nv_bfloat16* w;     // [M][C]
  float* part;                // [ranges][n][r][C]
  int64_t C;
  int tiles;                  // column tiles (0: not wanted)
};
struct OuterParams {
  OuterSide side[2];
  const int* ids;
  int* present;               // [ranges][n]
  int64_t M;
  int n, r, range, stages;
};

constexpr int kOuterThreads = 384, kCopyWarps = 3;
constexpr int kOuterN = 256, kOuterK = 64;                 // columns and rows of a stage
constexpr int kOuterRange = RFQ_LORA_OUTER_RANGE;          // rows of one range, at most
constexpr uint32_t kOuterChunk = kOuterK * 128u;           // 64 elements along M or N
constexpr int kOuterPart = 4;                              // stages of one accumulation, see kPartTiles
static_assert(RFQ_LORA_MAX_ADAPTERS <= 4096 && kOuterRange == 4096, "adapter and row in one key");
constexpr int kNoAdapter = 1 << 24;

template <int kT>
__host__ __device__ constexpr uint32_t outer_stage_bytes(int r) {
  return (kOuterN / 64 + kT * (r > 64 ? 2 : 1)) * kOuterChunk;
}
// First of keys[0 .. count) that is not below `key`.
__device__ __forceinline__ int lower_bound(const int* keys, int count, int key) {
  int lo = 0, hi = count;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (keys[mid] < key) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool valid) {   // zeros (and no read) where not
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
// Waits until at most `groups` (1 to 3, else 0) of this thread's groups of copies are on their way.
__device__ __forceinline__ void copy_wait(int groups) {
  if (groups == 3) asm volatile("cp.async.wait_group 3;" ::: "memory");
  else if (groups == 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
  else if (groups == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
  else asm volatile("cp.async.wait_group 0;" ::: "memory");
}

template <int kT>
__global__ void __launch_bounds__(kOuterThreads, 1) rfq_lora_outer_wide_kernel(const __grid_constant__ OuterMaps maps,
                                                                                const OuterParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ int keys[kOuterRange];
  __shared__ uint64_t full[4], empty[4], acc_full[2], acc_empty[2], drained;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  volatile int* abort_flag = &abort_word;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t stage_bytes = outer_stage_bytes<kT>(p.r);
  const int chunks = p.r > 64 ? 2 : 1;

  if (tid == 0) {
    for (int s = 0; s < 4; ++s) {
      mbar_init(&full[s], kCopyWarps);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 8);
    }
    mbar_init(&drained, 1);
    abort_word = 0;
    fence_mbar_init();
  }
  if (warp == kCopyWarps) {
    tmem_alloc_g<1>(&tmem_slot, 2 * kOuterN);
    tmem_relinquish_g<1>();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  griddep_launch_dependents();
  griddep_wait();

  int tile = static_cast<int>(blockIdx.x);
  const bool second = tile >= p.side[0].tiles;
  if (second) tile -= p.side[0].tiles;
  const OuterSide s = second ? p.side[1] : p.side[0];
  const int64_t row0 = static_cast<int64_t>(blockIdx.y) * p.range;
  const int count = static_cast<int>(min(static_cast<int64_t>(p.range), p.M - row0));
  const int64_t c0 = static_cast<int64_t>(tile) * kOuterN;

  // The range's rows by adapter, then row: keys (adapter << 12) + row, rows without one last.
  int size = 64;
  while (size < count) size <<= 1;
  for (int i = tid; i < size; i += kOuterThreads) {
    int key = 0x7fffffff;
    if (i < count) {
      const int id = p.ids[row0 + i];
      key = (id >= 0 && id < p.n ? id << 12 : kNoAdapter) + i;
    }
    keys[i] = key;
  }
  __syncthreads();
  bool sorted = true;
  for (int i = tid + 1; i < size; i += kOuterThreads) sorted = sorted && keys[i - 1] <= keys[i];
  if (!__syncthreads_and(sorted)) {
    for (int k = 2; k <= size; k <<= 1)
      for (int j = k >> 1; j > 0; j >>= 1) {   // a bitonic sort
        for (int i = tid; i < size / 2; i += kOuterThreads) {
          const int lo = ((i & ~(j - 1)) << 1) | (i & (j - 1)), hi = lo | j;
          const int a = keys[lo], b = keys[hi];
          if ((a > b) == ((lo & k) == 0)) {
            keys[lo] = b;
            keys[hi] = a;
          }
        }
        __syncthreads();
      }
  }
  const int rows = lower_bound(keys, count, kNoAdapter);   // rows with an adapter
  if (blockIdx.x == 0)
    for (int i = tid; i < p.n; i += kOuterThreads) {
      const int at = lower_bound(keys, rows, i << 12);
      p.present[static_cast<int64_t>(blockIdx.y) * p.n + i] = at < rows && (keys[at] >> 12) == i;
    }

  if (warp < kCopyWarps) {
    // ------------------------------------------------------------ copies
    const int lag = p.stages - 1;   // gathered stages that are on their way while one more is asked for
    const int per = kT * p.r / 8, r8 = p.r / 8;
    const bool has_col = c0 + 8 * lane < s.C;
    const __nv_bfloat16* w = has_col ? s.w + row0 * s.C + c0 + 8 * lane : s.w;   // (read only where has_col)
    const __nv_bfloat16* v = s.v + row0 * s.ld + 8 * lane;
    uint32_t v_to[2], v_q[2];       // this lane's pieces of a row of v: chunk, piece in its 128 bytes
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int i = lane + 32 * u, e = i / r8, j = i - e * r8;
      v_to[u] = (e * chunks + (j >> 3)) * kOuterChunk;
      v_q[u] = j & 7;
    }
    const CUtensorMap* map_v = &maps.v[second];
    const CUtensorMap* map_w = &maps.w[second];
    Cursor c, out;
    Filled filled;
    int pending = 0;                // gathered stages not yet handed over
    bool ok = true;
    auto give = [&]() {             // the oldest of them has landed
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[out.stage]);
      out.next(p.stages);
      --pending;
    };
    for (int first = 0; first < rows && ok;) {
      const int end = lower_bound(keys, rows, ((keys[first] >> 12) + 1) << 12);
      for (int at = first; at < end; at += kOuterK) {
        ok = mbar_wait(&empty[c.stage], c.phase ^ 1u, abort_flag, &g_lora_error, kErrWaitEmpty);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        uint8_t* stage = smem + c.stage * stage_bytes;
        filled.add(c);
        if (at + kOuterK <= end && keys[at + kOuterK - 1] - keys[at] == kOuterK - 1) {
          copy_wait(0);
          while (pending > 0) give();
          if (lane == 0) {
            if (warp == 0) {
              const int row = static_cast<int>(row0) + (keys[at] & (kOuterRange - 1));
              mbar_arrive_expect_tx(&full[c.stage], stage_bytes);
              for (int e = 0; e < kT; ++e)
                for (int h = 0; h < chunks; ++h)
                  tma_load_2d(stage + (e * chunks + h) * kOuterChunk, map_v, &full[c.stage], e * p.r + 64 * h, row);
#pragma unroll
              for (int h = 0; h < kOuterN / 64; ++h)
                tma_load_2d(stage + (kT * chunks + h) * kOuterChunk, map_w, &full[c.stage], static_cast<int>(c0) + 64 * h, row);
            } else {
              mbar_arrive(&full[c.stage]);
            }
          }
          out.next(p.stages);
        } else {
          const uint32_t sv = smem_addr(stage), sw = sv + (kT * chunks + (lane >> 3)) * kOuterChunk;
          // A lane looks up one row for all: their addresses then come by shuffles, not one load after the other.
          const int mine = warp + kCopyWarps * lane;
          const int key = mine < kOuterK && at + mine < end ? keys[at + mine] & (kOuterRange - 1) : -1;
          const uint32_t c_off = static_cast<uint32_t>(s.C), ld = static_cast<uint32_t>(s.ld);
#pragma unroll 8
          for (int k = 0; k < (kOuterK + kCopyWarps - 1) / kCopyWarps; ++k) {
            const int m = warp + kCopyWarps * k, row = __shfl_sync(0xffffffffu, key, k);
            if (m >= kOuterK) break;
            const bool has = row >= 0;
            const uint64_t r = has ? row : 0;
            copy16(sw + m * 128 + (((lane & 7) ^ (m & 7)) << 4), w + r * c_off, has && has_col);
#pragma unroll
            for (int u = 0; u < 2; ++u)
              if (lane + 32 * u < per) copy16(sv + v_to[u] + m * 128 + ((v_q[u] ^ (m & 7)) << 4), v + r * ld + 256 * u, has);
          }
          asm volatile("cp.async.commit_group;" ::: "memory");
          if (++pending > lag) {
            copy_wait(lag);
            give();
          }
        }
        c.next(p.stages);
      }
      first = end;
    }
    copy_wait(0);
    while (pending > 0) give();
    if (tid == 0) filled.drain(full, p.stages);
    __syncwarp();
  } else if (warp == kCopyWarps) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t id = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 15) | (1u << 16) | (uint32_t(kOuterN >> 3) << 17) | ((128u >> 4) << 24);
      Cursor c, acc;
      bool ok = true;
      for (int first = 0; first < rows && ok;) {
        const int end = lower_bound(keys, rows, ((keys[first] >> 12) + 1) << 12);
        const int iters = (end - first + kOuterK - 1) / kOuterK;
        for (int i0 = 0; i0 < iters && ok; i0 += kOuterPart) {
          ok = mbar_wait(&acc_empty[acc.stage], acc.phase ^ 1u, abort_flag, &g_lora_error, kErrWaitAccEmpty);
          if (!ok) break;
          tc_fence_after();
          const uint32_t d = tmem + acc.stage * kOuterN;
          for (int i = i0; i < min(i0 + kOuterPart, iters); ++i) {
            ok = mbar_wait(&full[c.stage], c.phase, abort_flag, &g_lora_error, kErrWaitFull);
            if (!ok) break;
            tc_fence_after();
            const uint32_t sv = smem_addr(smem) + c.stage * stage_bytes, sw = sv + kT * chunks * kOuterChunk;
            const uint64_t db = mn_major_desc(sw, kOuterChunk);
#pragma unroll
            for (uint32_t q = 0; q < kOuterK / 16; ++q)
#pragma unroll
              for (int e = kT - 1; e >= 0; --e)   // smallest terms first
                // Up to rank 64 the other half of M is whatever lies behind (inside the stage): its results are not kept.
                mma_bf16_g<1>(d, mn_major_desc(sv + e * chunks * kOuterChunk, kOuterChunk) + 128 * q, db + 128 * q, id,
                              (i != i0 || q != 0 || e != kT - 1) ? 1u : 0u);
            tc_commit(&empty[c.stage]);
            c.next(p.stages);
          }
          if (!ok) break;
          tc_commit(&acc_full[acc.stage]);
          acc.next(2);
        }
        first = end;
      }
      if (!ok) {   // teardown after an abort: wait for the MMAs already issued
        tc_commit(&drained);
        int never = 0;
        mbar_wait(&drained, 0, &never, &g_lora_error, kErrWaitDrain);
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    const int quad = warp & 3, half = (warp - 4) >> 2;
    const int j = quad * 32 + lane;
    const bool here = quad * 32 < p.r;
    Cursor acc;
    bool ok = true;
    for (int first = 0; first < rows && ok;) {
      const int a = keys[first] >> 12;
      const int end = lower_bound(keys, rows, (a + 1) << 12);
      const int iters = (end - first + kOuterK - 1) / kOuterK;
      float sum[128];
      for (int i0 = 0; i0 < iters && ok; i0 += kOuterPart) {
        ok = mbar_wait(&acc_full[acc.stage], acc.phase, abort_flag, &g_lora_error, kErrWaitAccFull, 2 * kWaitLimitNs);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        if (here) {
          const uint32_t at = tmem + (static_cast<uint32_t>(quad * 32) << 16) + acc.stage * kOuterN + half * 128;
#pragma unroll
          for (int c = 0; c < 128; c += 8) {
            uint32_t u[8];
            tmem_load_32x32b_x8(at + c, u);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[c + i] = i0 == 0 ? __uint_as_float(u[i]) : sum[c + i] + __uint_as_float(u[i]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&acc_empty[acc.stage]);
        acc.next(2);
      }
      if (ok && j < p.r) {
        float* out = s.part + ((static_cast<int64_t>(blockIdx.y) * p.n + a) * p.r + j) * s.C;
        const int64_t col = c0 + half * 128;
#pragma unroll
        for (int c = 0; c < 128; c += 4)
          if (col + c < s.C) *reinterpret_cast<float4*>(out + col + c) = make_float4(sum[c], sum[c + 1], sum[c + 2], sum[c + 3]);
      }
      __syncwarp();
      first = end;
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kCopyWarps) {
    __syncwarp();
    tmem_dealloc_g<1>(tmem, 2 * kOuterN);
  }
}

// ---------------------------------------------------------------- host
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// [n][rows][cols] bf16, box 64 columns x box_rows rows of one matrix.
bool encode_pool_map(EncodeTiledFn encode, CUtensorMap* map, const void* base, int64_t n, int64_t rows, int64_t cols, uint32_t box_rows) {
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(n)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(cols) * 2, static_cast<cuuint64_t>(cols) * static_cast<cuuint64_t>(rows) * 2};
  cuuint32_t box[3] = {64u, box_rows, 1u};
  cuuint32_t one[3] = {1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
bool encode_f32_map(EncodeTiledFn encode, CUtensorMap* map, const void* base, int64_t rows, int64_t cols) {
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols) * 4};
  cuuint32_t box[2] = {32u, kChunk};
  cuuint32_t one[2] = {1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Dynamic shared memory that any call may ask of shrink and expand, and of outer.  What is set here belongs to the kernel, not to the
// launch: set to each launch's own size, a smaller call on another host thread could lower it before this one's launch.
constexpr int kMostSmem = kSmemLimit - 1024, kMostOuterSmem = kSmemLimit - 17 * 1024;

template <class Kernel, class Maps, class Params>
cudaError_t launch(Kernel kernel, const Maps& maps, const Params& p, int64_t grid, int threads, size_t smem, int cluster, cudaStream_t stream) {
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(threads);
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
  e = cudaLaunchKernelEx(&cfg, kernel, maps, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <bool kTrans, bool kF32>
cudaError_t expand_typed(const ExpandMaps& maps, ExpandParams p, int num_sms, cudaStream_t stream) {
  const uint32_t q = expand_q_bytes<kTrans, kF32>(p.r), s = expand_s_bytes<kF32>(p.r);
  // 2 KiB: alignment (in the dynamic part) and the static part (368 bytes).  With them four base stages fit beside two of s up to rank 64, three
  // beside one above; with 4 KiB kept back there is one less of each, and 4096 rows of rank 128, 4096 -> 12288, take 111 us, not 86.
  uint32_t room = kSmemLimit - 2048 - s;
  // One stage of s where chunks may hold several adapters: a CTA's part touches few chunks, and the room goes to Q, which
  // then comes once for each adapter (4096 rows of 8 requests of rank 64: 66 us, with two stages of s 70).
  p.s_stages = 1;
  if (p.counts == nullptr && room >= s + 3 * 2 * kBox + 2 * q) {
    p.s_stages = 2;
    room -= s;
  }
  p.q_stages = 2;
  p.base_stages = 2;
  while (p.base_stages < 4 && (p.base_stages + 1) * 2 * kBox + p.q_stages * q <= room) ++p.base_stages;
  while (p.q_stages < 4 && p.base_stages * 2 * kBox + (p.q_stages + 1) * q <= room) ++p.q_stages;
  const size_t smem = 1024 + p.s_stages * s + p.base_stages * 2 * kBox + p.q_stages * q;
  const int64_t parts = p.counts != nullptr ? p.chunks * p.tiles : p.units, grid = parts < num_sms ? parts : num_sms;
  return launch(rfq_lora_expand_wide_kernel<kTrans, kF32>, maps, p, grid, kExpandThreads, smem, 1, stream);
}

}  // namespace

// s [M][r] (or nullptr) = scale (P src), P the pool [n][r][C] or (trans) [n][C][r]; terms [M][num_terms][r];
// counts [chunks of 128 rows]: adapters of each.
cudaError_t launch_lora_shrink_wide(const void* src, const void* pool, bool trans, const int* ids, const float* scale, float* s,
                                    void* terms, int num_terms, int* counts, int64_t M, int64_t C, int64_t n, int64_t r, int num_sms, void* encode_tiled, cudaStream_t stream) {
  EncodeTiledFn encode = reinterpret_cast<EncodeTiledFn>(encode_tiled);
  ShrinkMaps maps;
  const uint32_t r16 = static_cast<uint32_t>((r + 15) / 16 * 16);
  if (!encode_bf16_map(encode, &maps.src, src, M, C, C, kChunk) ||
      !(trans ? encode_pool_map(encode, &maps.p, pool, n, C, r, 64) : encode_pool_map(encode, &maps.p, pool, n, r, C, r16)))
    return cudaErrorInvalidValue;
  ShrinkParams p = {};
  p.ids = ids;
  p.scale = scale;
  p.s = s;
  p.terms = static_cast<__nv_bfloat16*>(terms);
  p.num_terms = num_terms;
  p.counts = counts;
  p.M = M;
  p.n = static_cast<int>(n);
  p.r = static_cast<int>(r);
  p.kt = static_cast<int>(ceil_div(C, 64));
  // A cluster of up to 8 along the contraction while two CTAs per SM are not reached, no rank empty.
  const int64_t chunks = ceil_div(M, kChunk);
  p.cluster = 1;
  while (p.cluster < 8 && chunks * p.cluster * 2 <= 2 * num_sms) {
    const int next = p.cluster * 2, per = static_cast<int>(ceil_div(p.kt, next));
    if (per < 2 || (next - 1) * per >= p.kt) break;
    p.cluster = next;
  }
  p.kt_per_rank = static_cast<int>(ceil_div(p.kt, p.cluster));
  const uint32_t stage = kBox + shrink_p_bytes(trans, p.r), sums = shrink_sum_bytes(p.r);
  // As many stages as leave room for two CTAs per SM; as many as fit one where there are few CTAs (clusters
  // of 8 do not fill every SM alone: 16 of them took two rounds, 27 us for 2000 rows against 24 for 3000)
  // or two would have fewer than three each.
  const uint32_t room = chunks * p.cluster > num_sms / 2 ? kSmemLimit / 2 : kSmemLimit;
  p.stages = sums + 2048 < room ? static_cast<int>((room - 2048 - sums) / stage) : 0;
  if (p.stages < 3) p.stages = static_cast<int>((kSmemLimit - 2048 - sums) / stage);
  if (p.stages > kMaxStages) p.stages = kMaxStages;
  // Never less than 112 KiB.  CTAs that share an SM share its tensor memory too: two of this kernel fit there by their columns, but one
  // beside a CTA of the short-batch GEMM (all 512 columns, 120 KiB, a cluster as well) on another stream would let each of two clusters
  // hold what a CTA of the other waits for, for good.
  constexpr size_t kLeastSmem = 112 * 1024;
  static_assert(2 * (kLeastSmem + 2048) <= 228 * 1024 && kLeastSmem + 120 * 1024 > 228 * 1024, "two of these an SM, none beside a 120 KiB one");
  const size_t need = 1024 + static_cast<size_t>(p.stages) * stage + sums, smem = need > kLeastSmem ? need : kLeastSmem;
  return trans ? launch(rfq_lora_shrink_wide_kernel<true>, maps, p, chunks * p.cluster, kShrinkThreads, smem, p.cluster, stream)
               : launch(rfq_lora_shrink_wide_kernel<false>, maps, p, chunks * p.cluster, kShrinkThreads, smem, p.cluster, stream);
}

// out [M][C] = base + Q s, s from its terms (all of num_terms lie there; the output's type says how many
// are taken), Q the pool [n][C][r] or (trans) [n][r][C].  counts: as left by shrink, or nullptr (only time depends on it).
cudaError_t launch_lora_expand_wide(const void* terms, int num_terms, const int* counts, const void* pool, bool trans, const int* ids, const void* base, void* out, bool f32,
                                    int64_t M, int64_t C, int64_t n, int64_t r, int num_sms, void* encode_tiled, cudaStream_t stream) {
  EncodeTiledFn encode = reinterpret_cast<EncodeTiledFn>(encode_tiled);
  ExpandMaps maps;
  const uint32_t r16 = static_cast<uint32_t>((r + 15) / 16 * 16);
  const int cols = f32 ? kCols<true> : kCols<false>;
  auto wide_map = [&](CUtensorMap* map, const void* at) {
    return f32 ? encode_f32_map(encode, map, at, M, C) : encode_bf16_map(encode, map, at, M, C, C, kChunk);
  };
  // [M][term][r] as (r, term, M): a box is one term of 128 rows, zeros behind r.
  auto s_map = [&](CUtensorMap* map) {
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(r), static_cast<cuuint64_t>(num_terms), static_cast<cuuint64_t>(M)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(r) * 2, static_cast<cuuint64_t>(r) * 2 * num_terms};
    cuuint32_t box[3] = {64u, 1u, kChunk};
    cuuint32_t one[3] = {1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(terms), dims, strides, box, one,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  if (!s_map(&maps.s) || !wide_map(&maps.out, out) || !wide_map(&maps.base, base != nullptr ? base : out) ||
      !(trans ? encode_pool_map(encode, &maps.q, pool, n, r, C, r16) : encode_pool_map(encode, &maps.q, pool, n, C, r, cols)))
    return cudaErrorInvalidValue;
  ExpandParams p = {};
  p.ids = ids;
  p.M = M;
  p.C = static_cast<int>(C);
  p.n = static_cast<int>(n);
  p.r = static_cast<int>(r);
  p.has_base = base != nullptr;
  p.in_place = base == out;
  p.tiles = static_cast<int>(ceil_div(C, cols));
  p.chunks = ceil_div(M, kChunk);
  p.counts = n > 1 ? counts : nullptr;
  // Column tiles of one unit: the length (4 to 16 tiles) that leaves the fewest tiles to the CTA
  // with the most, each unit charged a quarter of one more for the change of rows.
  int64_t best = INT64_MAX;
  p.unit_tiles = p.tiles;
  for (int len = 4; len <= 16; ++len) {
    const int64_t units = p.chunks * ceil_div(p.tiles, len), cost = ceil_div(units, num_sms) * (4 * len + 1);
    if (cost < best) {
      best = cost;
      p.unit_tiles = len;
    }
  }
  p.col_units = static_cast<int>(ceil_div(p.tiles, p.unit_tiles));
  p.units = p.chunks * p.col_units;
  if (trans) return f32 ? expand_typed<true, true>(maps, p, num_sms, stream) : expand_typed<true, false>(maps, p, num_sms, stream);
  return f32 ? expand_typed<false, true>(maps, p, num_sms, stream) : expand_typed<false, false>(maps, p, num_sms, stream);
}

// part of both sides (v [M][ld] of `terms` terms, w [M][C]; a side without w is not wanted), present [ranges][n].
cudaError_t launch_lora_outer_wide(const void* ds, int ds_ld, const void* x, float* part_a, int64_t K, const void* s, int s_ld, const void* dy,
                                   float* part_b, int64_t N, int terms, const int* ids, int* present, int64_t M, int64_t n, int64_t r, int range,
                                   void* encode_tiled, cudaStream_t stream) {
  EncodeTiledFn encode = reinterpret_cast<EncodeTiledFn>(encode_tiled);
  OuterMaps maps = {};
  if (x != nullptr && !(encode_bf16_map(encode, &maps.v[0], ds, M, ds_ld, ds_ld, kOuterK) && encode_bf16_map(encode, &maps.w[0], x, M, K, K, kOuterK)))
    return cudaErrorInvalidValue;
  if (dy != nullptr && !(encode_bf16_map(encode, &maps.v[1], s, M, s_ld, s_ld, kOuterK) && encode_bf16_map(encode, &maps.w[1], dy, M, N, N, kOuterK)))
    return cudaErrorInvalidValue;
  OuterParams p = {};
  p.side[0] = {static_cast<const __nv_bfloat16*>(ds), ds_ld, static_cast<const __nv_bfloat16*>(x), part_a, K, x != nullptr ? static_cast<int>(ceil_div(K, kOuterN)) : 0};
  p.side[1] = {static_cast<const __nv_bfloat16*>(s), s_ld, static_cast<const __nv_bfloat16*>(dy), part_b, N, dy != nullptr ? static_cast<int>(ceil_div(N, kOuterN)) : 0};
  p.ids = ids;
  p.present = present;
  p.M = M;
  p.n = static_cast<int>(n);
  p.r = static_cast<int>(r);
  p.range = range;
  const uint32_t stage = terms == 3 ? outer_stage_bytes<3>(p.r) : outer_stage_bytes<2>(p.r);
  p.stages = static_cast<int>((kMostOuterSmem - 1024) / stage);   // 2 to 4 (beside 17 KiB: the keys and barriers)
  if (p.stages > 4) p.stages = 4;
  const size_t smem = 1024 + static_cast<size_t>(p.stages) * stage;
  auto kernel = terms == 3 ? rfq_lora_outer_wide_kernel<3> : rfq_lora_outer_wide_kernel<2>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostOuterSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.side[0].tiles + p.side[1].tiles), static_cast<unsigned>(ceil_div(M, range)));
  cfg.blockDim = dim3(kOuterThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // see griddep_wait()
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kernel, maps, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t read_and_clear_lora_error(unsigned int* value) {
  unsigned int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(value, g_lora_error, sizeof(unsigned int));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(g_lora_error, &zero, sizeof(unsigned int));
}

}  // namespace rfq
