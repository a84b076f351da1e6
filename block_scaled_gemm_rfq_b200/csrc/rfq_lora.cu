// rfq_lora.cu -- low-rank adapters of many requests beside a shared projection.
//
// Row m of a batch uses adapter a = ids[m] (none if that is outside [0, n)).  With
// A [n][r][K], B [n][N][r] in bf16 and one fp32 scale per adapter:
//
//     s_m = scale_a A_a x_m                       (rank r, fp32)
//     y_m = base_m + B_a s_m
//
// and for the gradient dy (those of the adapters summed over their rows):
//
//     ds_m = scale_a B_a^T dy_m     dx_m = base_m + A_a^T ds_m
//     dA_a = sum ds_m x_m^T         dB_a = sum dy_m s_m^T
//
// With r far below K and N every product is bound by memory: x and dy are read and y and
// dx written once per pass over them, at 2 r flops for each of their elements:
//
//   shrink   s, ds: rows x wide -> rank
//   expand   y, dx: rank -> wide, added to the base
//   split    s, ds as sums of bf16 terms for the next one
//   outer    dA, dB: contraction over rows, split into row ranges
//   reduce   sums the ranges in order and rounds
//
// Long batches take the kernels of rfq_lora_wide.cu (tcgen05; 128 neighbouring rows, or 64 of
// one adapter).  Here are those of short batches, where rows have adapters of their own and time goes
// into reading the adapters' weights; all on warp-level m16n8k16 MMAs.  The rows of a 256-row chunk are grouped by adapter inside the CTA that works on them (no
// host knowledge of the ids, no order asked of them): groups of up to 16 rows share an
// adapter's weights.
//
// Going forward the weights run along the contraction (A in shrink, B in expand) and go from global
// memory straight into MMA fragments, each used by one warp once: a thread's fragment takes any
// four contraction elements of its row as long as the other operand takes the same, so it
// loads neighbouring ones, 8 or 16 bytes at a time.  Both products are one launch.
// Going back they run across it: they, and the operands of the gradients, go through shared memory
// with 16-byte asynchronous copies and are transposed on the way out (ldmatrix).  Each thread
// keeps the addresses of the pieces it copies and steps them along: with the addresses formed anew
// for each copy the kernels issued 1600 instructions a warp for 8 KiB and ran at 1.9 TB/s; with one
// bulk copy for each 256-byte row piece they were slower still (about 65 ns a copy and SM).
//
// No atomics: a result does not depend on timing.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "rfq_internal.h"
#include "rfq_ptx.cuh"
#include "rfq_terms.cuh"

namespace rfq {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 256;                // rows grouped by one CTA
constexpr int kRows = 16;                  // rows of one group
constexpr int kMaxAdapters = RFQ_LORA_MAX_ADAPTERS;
constexpr int kMaxStages = 6;
constexpr int kSmemLimit = 227 * 1024;

__host__ __device__ constexpr int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
// Row stride in shared memory of rows of `bytes` bytes: an odd number of 16-byte units, so that
// eight rows at one column fall into eight different bank groups (ldmatrix without conflicts).
__host__ __device__ constexpr int odd_stride(int bytes) { return ((bytes / 16) | 1) * 16; }
// Rows along which the rank runs (r * 2 bytes) lie back to back in global memory.  Up to 32 bytes,
// or an odd number of 16-byte units, they are copied as one block as they lie (at most two-way
// conflicts); longer ones row by row with a padded stride.
__host__ __device__ constexpr bool rank_block(int r) { return r <= 16 || (r / 8) % 2 == 1; }
__host__ __device__ constexpr int rank_stride(int r) { return rank_block(r) ? 2 * r : odd_stride(2 * r); }

template <bool kTrans>
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
  if constexpr (kTrans)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
template <bool kTrans>
__device__ __forceinline__ void ldsm2(uint32_t (&r)[2], uint32_t a) {
  if constexpr (kTrans)
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(a) : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(a) : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma1688(float (&d)[4], const uint32_t (&a)[2], uint32_t b) {
  asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5}, {%6}, {%0, %1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a[0]), "r"(a[1]), "r"(b));
}
// 16 bytes from global to shared memory; zeros (and no read) where `valid` is false.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async16_bytes(uint32_t dst, const void* src, int bytes) {   // 16, or 0 for zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until at most stages - 2 groups of this thread are on their way (stages: 2 to kMaxStages).
__device__ __forceinline__ void cp_wait_stage(int stages) {
  switch (stages) {
    case 2: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 3: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 4: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    case 5: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 4;" ::: "memory"); break;
  }
}

// The rows of one chunk, grouped by adapter: order[] lists them (as offsets in the chunk) by
// rising adapter, rows without one last; item i is order[start[i] .. start[i + 1]), at most
// kRows rows of one adapter.
struct Groups {
  int ids[kChunk];
  int order[kChunk];
  int start[kChunk + 1];
  int items;
  int keys[kChunk];            // of the grouping alone
  int runs[kChunk / 32];
  int firsts[kChunk / 32];
};
constexpr int kTable = 3 * kChunk + 2;   // words of a Groups that the next kernel reads back

__device__ void group_rows(Groups& g, const int* ids, int64_t row0, int64_t M, int n) {
  static_assert(kThreads == kChunk && kMaxAdapters < 0x7fffff, "a thread for each row, adapter and row in one key");
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int count = static_cast<int>(M - row0 < kChunk ? M - row0 : kChunk);
  int id = INT_MAX;
  if (t < count) {
    const int v = ids[row0 + t];
    if (v >= 0 && v < n) id = v;
  }
  g.ids[t] = id;
  // Adapter, then row: all keys differ; rows past the last sort behind all others.
  int key = t >= count ? 0x7fffffff : (id == INT_MAX ? 0x7fffff00 : id << 8) | t;
  g.keys[t] = key;
  __syncthreads();
  // Rows already in order (neighbours of one request, one adapter for all) need no sorting.
  if (!__syncthreads_and(t == 0 || t >= count || g.keys[t - 1] < key)) {
    for (int k = 2; k < 2 * count; k <<= 1)    // rows past the last are in place
      for (int j = k >> 1; j > 0; j >>= 1) {   // a bitonic sort, through shuffles below 32
        int other;
        if (j < 32) {
          other = __shfl_xor_sync(0xffffffffu, key, j);
        } else {
          __syncthreads();
          g.keys[t] = key;
          __syncthreads();
          other = g.keys[t ^ j];
        }
        key = ((t & j) == 0) == ((t & k) == 0) ? min(key, other) : max(key, other);
      }
    __syncthreads();
    g.keys[t] = key;
    __syncthreads();
  }
  // Runs of one adapter, and in them every kRows-th row, begin an item.
  const bool begins = t < count && (t == 0 || (g.keys[t - 1] >> 8) != (key >> 8));
  const unsigned run = __ballot_sync(0xffffffffu, begins);
  if (lane == 0) g.runs[warp] = static_cast<int>(run);
  __syncthreads();
  bool first = false;
  if (t < count) {
    int w = warp;
    unsigned bits = run & (0xffffffffu >> (31 - lane));
    while (bits == 0) bits = static_cast<unsigned>(g.runs[--w]);   // row 0 begins a run
    first = (t - (w * 32 + 31 - __clz(bits))) % kRows == 0;
    g.order[t] = key & (kChunk - 1);
  }
  const unsigned firsts = __ballot_sync(0xffffffffu, first);
  if (lane == 0) g.firsts[warp] = __popc(firsts);
  __syncthreads();
  int before = 0, items = 0;
#pragma unroll
  for (int w = 0; w < kChunk / 32; ++w) {
    if (w < warp) before += g.firsts[w];
    items += g.firsts[w];
  }
  if (first) g.start[before + __popc(firsts & ((1u << lane) - 1))] = t;
  if (t == 0) {
    g.start[items] = count;
    g.items = items;
  }
  __syncthreads();
}

// The grouping is done by shrink; the first CTA of each chunk leaves it for expand.
__device__ __forceinline__ void leave_groups(const Groups& g, int* table) {
  for (int i = threadIdx.x; i < kTable; i += kThreads) table[i] = reinterpret_cast<const int*>(&g)[i];
}
__device__ __forceinline__ void take_groups(Groups& g, const int* table) {
  for (int i = threadIdx.x; i < kTable; i += kThreads) reinterpret_cast<int*>(&g)[i] = table[i];
  __syncthreads();
}

// ---------------------------------------------------------------- shrink
// ds of short batches: part[split][m][j] = sum over the split's k of src[m][k] B_a[k][j].
struct ShrinkParams {
  const __nv_bfloat16* src;   // [M][C]
  const __nv_bfloat16* p;     // [n][C][r]
  const int* ids;
  float* part;                // [splits][M][r]
  int64_t M, C, c_split;      // c_split: contraction elements of one split (a multiple of kBK)
  int* table;                 // [chunks][kTable]
  int n, r, zs;               // zs: CTAs that share the items of one chunk
  int stages;
};

constexpr int kBK = 128;                         // contraction elements of one stage
constexpr int kRowStride = odd_stride(kBK * 2);  // of a 256-byte row segment
__host__ __device__ constexpr int shrink_p_bytes(int r) { return kBK * rank_stride(r); }
constexpr int kWarps = kThreads / 32;
static_assert(kRows == 16 && kBK / 16 == kWarps, "an item is one MMA tile of rows; each warp takes one k16 step of a stage");
__host__ __device__ constexpr int shrink_red_bytes(int r) { return (kWarps - 1) * kRows * r * 4; }

template <int kJ>   // 8-column tiles of the rank, at most
__global__ void __launch_bounds__(kThreads) rfq_lora_shrink_kernel(const ShrinkParams p) {
  constexpr int kPCopies = kJ * 8 * (kBK / 8) / kThreads;   // of the adapter's weights, at most
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ __align__(16) Groups g;
  griddep_launch_dependents();
  griddep_wait();
  const int64_t row0 = static_cast<int64_t>(blockIdx.x / p.zs) * kChunk;
  const int z = static_cast<int>(blockIdx.x % p.zs);
  group_rows(g, p.ids, row0, p.M, p.n);
  if (z == 0 && blockIdx.y == 0) leave_groups(g, p.table + (blockIdx.x / p.zs) * kTable);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int jt = p.r / 8;
  const int p_stride = rank_stride(p.r);
  const int stage_bytes = kRows * kRowStride + shrink_p_bytes(p.r);
  const uint32_t base = smem_addr(smem);
  float* red = reinterpret_cast<float*>(smem + p.stages * stage_bytes);   // [kWarps - 1][kRows][r]
  const int64_t c0 = static_cast<int64_t>(blockIdx.y) * p.c_split;
  const int64_t c1 = min(p.C, c0 + p.c_split);
  const int iters = static_cast<int>(ceil_div(c1 - c0, kBK));
  const int xm = tid >> 4, qx = tid & 15;       // this thread's 16-byte piece of a stage: row, place in its 256 bytes

  for (int item = z; item < g.items; item += p.zs) {
    const int first = g.start[item], rows = g.start[item + 1] - first;
    const int a = g.ids[g.order[first]];
    if (a == INT_MAX) break;   // rows without an adapter come last
    const bool has_x = xm < rows;
    const __nv_bfloat16* x_at = p.src + (row0 + g.order[has_x ? first + xm : first]) * p.C + c0 + 8 * qx;
    const __nv_bfloat16* pa = p.p + static_cast<int64_t>(a) * p.r * p.C;
    const __nv_bfloat16* p_at[kPCopies];
    uint32_t p_to[kPCopies];
    int p_k[kPCopies];         // contraction element of the piece in its stage; kBK where there is none
#pragma unroll
    for (int u = 0; u < kPCopies; ++u) {
      const int i = tid + kThreads * u;
      const int k = i / jt;
      p_k[u] = k < kBK ? k : kBK;
      p_at[u] = pa + c0 * p.r + 8 * static_cast<int64_t>(i);
      p_to[u] = k * p_stride + (i - k * jt) * 16;
    }
    int load_stage = 0, load_left = static_cast<int>(c1 - c0);   // contraction elements not yet asked for
    auto load = [&]() {
      if (load_left > 0) {
        const uint32_t sx = base + load_stage * stage_bytes, sp = sx + kRows * kRowStride;
        const bool ok_x = has_x && 8 * qx < load_left;
        cp_async16(sx + xm * kRowStride + 16 * qx, ok_x ? x_at : p.src, ok_x);
        x_at += kBK;
#pragma unroll
        for (int u = 0; u < kPCopies; ++u)
          if (p_k[u] < kBK) {
            const bool ok = p_k[u] < load_left;
            cp_async16(sp + p_to[u], ok ? p_at[u] : p.p, ok);
            p_at[u] += kBK * p.r;
          }
      }
      cp_commit();
      load_left -= kBK;
      if (++load_stage == p.stages) load_stage = 0;
    };

    float acc[kJ][4];
#pragma unroll
    for (int j = 0; j < kJ; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
    for (int it = 0; it < p.stages - 1; ++it) load();
    int stage = 0;
    for (int it = 0; it < iters; ++it) {
      cp_wait_stage(p.stages);
      __syncthreads();
      load();
      const uint32_t sx = base + stage * stage_bytes, sp = sx + kRows * kRowStride;
      uint32_t fa[4];
      ldsm4<false>(fa, sx + (lane & 15) * kRowStride + 32 * warp + (lane >> 4) * 16);
#pragma unroll
      for (int j = 0; j < kJ; j += 2) {
        if (j + 1 < jt) {
          uint32_t fb[4];
          ldsm4<true>(fb, sp + (warp * 16 + (lane & 15)) * p_stride + (j + (lane >> 4)) * 16);
          mma16816(acc[j], fa, fb[0], fb[1]);
          mma16816(acc[j + 1], fa, fb[2], fb[3]);
        } else if (j < jt) {
          uint32_t fb[2];
          ldsm2<true>(fb, sp + (warp * 16 + (lane & 15)) * p_stride + j * 16);
          mma16816(acc[j], fa, fb[0], fb[1]);
        }
      }
      if (++stage == p.stages) stage = 0;
    }
    // Join the warps, in order; the first of them writes [rows][r].
    const int ra = lane >> 2, rb = ra + 8;
    if (warp > 0) {
#pragma unroll
      for (int j = 0; j < kJ; ++j)
        if (j < jt) {
          float* at = red + ((warp - 1) * kRows + ra) * p.r + j * 8 + 2 * (lane & 3);
          *reinterpret_cast<float2*>(at) = make_float2(acc[j][0], acc[j][1]);
          *reinterpret_cast<float2*>(at + 8 * p.r) = make_float2(acc[j][2], acc[j][3]);
        }
    }
    __syncthreads();
    if (warp == 0) {
      float* out = p.part + static_cast<int64_t>(blockIdx.y) * p.M * p.r;
      const int64_t row_a = ra < rows ? row0 + g.order[first + ra] : -1, row_b = rb < rows ? row0 + g.order[first + rb] : -1;
#pragma unroll
      for (int j = 0; j < kJ; ++j)
        if (j < jt) {
          const int col = j * 8 + 2 * (lane & 3);
          float2 va = make_float2(acc[j][0], acc[j][1]), vb = make_float2(acc[j][2], acc[j][3]);
#pragma unroll
          for (int w = 0; w < kWarps - 1; ++w) {
            const float2 ua = *reinterpret_cast<const float2*>(red + (w * kRows + ra) * p.r + col);
            const float2 ub = *reinterpret_cast<const float2*>(red + (w * kRows + rb) * p.r + col);
            va.x += ua.x;
            va.y += ua.y;
            vb.x += ub.x;
            vb.y += ub.y;
          }
          if (row_a >= 0) *reinterpret_cast<float2*>(out + row_a * p.r + col) = va;
          if (row_b >= 0) *reinterpret_cast<float2*>(out + row_b * p.r + col) = vb;
        }
    }
    __syncthreads();
  }
}

// s'[m][j] = scale_a * sum of the splits, in order.
__device__ __forceinline__ float join_parts(const float* part, int splits, int64_t stride, int64_t at, float scale) {
  float v = part[at];
#pragma unroll 4
  for (int s = 1; s < splits; ++s) v += part[s * stride + at];
  return v * scale;
}
// v as a sum of kT bf16 terms (8 bits each).
template <int kT>
__device__ __forceinline__ void split_terms(float v, __nv_bfloat16 (&t)[kT]) {
#pragma unroll
  for (int i = 0; i < kT; ++i) t[i] = take_term(v);
}

// ---------------------------------------------------------------- expand
// dx of short batches: out[m][c] = base[m][c] + sum_j ds'[m][j] A_a[j][c].  A stage holds a [kRows][kBN]
// tile of the base and the adapter's weights for its columns; the sum is formed in place and copied
// out from there, in whole row pieces.
struct ExpandParams {
  const float* part;          // [splits][M][r]
  const float* scale;         // [n]
  const __nv_bfloat16* q;     // [n][r][C]
  const int* table;           // [chunks][kTable], from shrink
  const void* base;           // [M][C] or nullptr
  void* out;                  // [M][C]
  int64_t M, C;
  int n, r, splits, zs;
  int tiles;                  // column tiles of one CTA
  int stages;
};

// Columns of one tile: 256 bytes of a row.
template <bool kF32>
constexpr int kBN = kF32 ? 64 : 128;
template <bool kF32>
constexpr int kQStride = odd_stride(kBN<kF32> * 2);
template <bool kF32>
__host__ __device__ constexpr int expand_stage_bytes(int r) {
  return kRows * kRowStride + r * kQStride<kF32>;
}
// The rank-r vector enters the MMA in bf16 terms of 8 bits each: three for an fp32 output (24 bits), two
// for a bf16 one.  One term would add an error as large as the output's own rounding (2^-9 of the adapter's
// share), in the same direction for a whole row, and the few rows of a short batch do not average it away: dx of
// two rows of rank 16 was off by 1.6 times its rounding.  The second costs 26.4 -> 27.8 us for 256 rows of 48
// adapters of rank 32 (4096 -> 12288), nothing for 16 rows.
template <bool kF32>
constexpr int kExpandTerms = kF32 ? 3 : 2;
template <bool kF32>
__host__ __device__ constexpr int expand_s_bytes(int r) {
  return kExpandTerms<kF32> * kRows * odd_stride(2 * r);
}

template <bool kF32>
__global__ void __launch_bounds__(kThreads) rfq_lora_expand_kernel(const ExpandParams p) {
  constexpr int kT = kExpandTerms<kF32>;
  constexpr int kCols = kBN<kF32>;
  constexpr int kPairs = kCols / kWarps / 8;           // 8-column tiles of a warp: two, or one of fp32
  constexpr int kSize = kF32 ? 4 : 2;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ __align__(16) Groups g;
  griddep_launch_dependents();
  griddep_wait();
  const int64_t row0 = static_cast<int64_t>(blockIdx.x / p.zs) * kChunk;
  const int z = static_cast<int>(blockIdx.x % p.zs);
  take_groups(g, p.table + (blockIdx.x / p.zs) * kTable);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int q_stride = kQStride<kF32>;
  const int s_stride = odd_stride(2 * p.r);
  const int stage_bytes = expand_stage_bytes<kF32>(p.r);
  uint8_t* s_mem = smem + p.stages * stage_bytes;
  const uint32_t base = smem_addr(smem), s_base = smem_addr(s_mem);
  const int64_t begin = static_cast<int64_t>(blockIdx.y) * p.tiles * kCols;
  const int64_t end = min(p.C, begin + static_cast<int64_t>(p.tiles) * kCols);
  const int iters = static_cast<int>(ceil_div(end - begin, kCols));
  const int xm = tid >> 4, qx = tid & 15;              // this thread's 16-byte piece of a tile
  constexpr int kPiece = 16 / kSize;                   // its columns
  const uint8_t* from = static_cast<const uint8_t*>(p.base);
  uint8_t* to = static_cast<uint8_t*>(p.out);

  for (int item = z; item < g.items; item += p.zs) {
    const int first = g.start[item], rows = g.start[item + 1] - first;
    const int a = g.ids[g.order[first]];
    const bool with = a != INT_MAX;
    // Rows without an adapter (they come last) keep what they have where the base is the output itself.
    if (!with && p.base == p.out) continue;
    const bool has = xm < rows;
    // Byte offset of this thread's piece, in the base and in the output.
    const int64_t at = ((row0 + g.order[has ? first + xm : first]) * p.C + begin) * kSize + 16 * qx;
    const __nv_bfloat16* qa = p.q + (with ? static_cast<int64_t>(a) * p.r * p.C : 0);
    int load_stage = 0, load_it = 0;
    auto load = [&]() {
      if (load_it < iters) {
        const uint32_t sb = base + load_stage * stage_bytes, sq = sb + kRows * kRowStride;
        const int left = static_cast<int>(min(static_cast<int64_t>(kCols), end - begin - static_cast<int64_t>(load_it) * kCols));
        if (from != nullptr) {
          const bool ok = has && kPiece * qx < left;
          cp_async16(sb + xm * kRowStride + 16 * qx, ok ? from + at + load_it * 256 : from, ok);
        }
        if (with) {
          const int64_t c = begin + static_cast<int64_t>(load_it) * kCols;
          constexpr int kQ = kCols / 8;
          for (int i = tid; i < p.r * kQ; i += kThreads) {
            const int j = i / kQ, q = i % kQ;
            const bool ok = 8 * q < left;
            cp_async16(sq + j * q_stride + 16 * q, ok ? qa + j * p.C + c + 8 * q : p.q, ok);
          }
        }
      }
      cp_commit();
      ++load_it;
      if (++load_stage == p.stages) load_stage = 0;
    };
    for (int it = 0; it < p.stages - 1; ++it) load();
    if (with) {
      const float scale = p.scale[a];
      for (int i = tid; i < rows * p.r; i += kThreads) {
        const int m = i / p.r, j = i - m * p.r;
        const int64_t sat = (row0 + g.order[first + m]) * p.r + j;
        const float v = join_parts(p.part, p.splits, p.M * p.r, sat, scale);
        __nv_bfloat16 t[kT];
        split_terms<kT>(v, t);
#pragma unroll
        for (int e = 0; e < kT; ++e) *reinterpret_cast<__nv_bfloat16*>(s_mem + (e * kRows + m) * s_stride + 2 * j) = t[e];
      }
    }
    int stage = 0;
    for (int it = 0; it < iters; ++it) {
      cp_wait_stage(p.stages);
      __syncthreads();
      load();
      uint8_t* sb = smem + stage * stage_bytes;
      const uint32_t sq = base + stage * stage_bytes + kRows * kRowStride;
      const int left = static_cast<int>(min(static_cast<int64_t>(kCols), end - begin - static_cast<int64_t>(it) * kCols));
      const int col = warp * (8 * kPairs);
      if (col < left && (with || from == nullptr)) {
        float acc[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
        if (with) {
          int ks = 0;
          for (; ks < p.r / 16; ++ks) {
            uint32_t fb[4];
            if constexpr (kPairs == 2) {
              ldsm4<true>(fb, sq + (ks * 16 + (lane & 15)) * q_stride + col * 2 + (lane >> 4) * 16);
            } else {
              uint32_t f2[2];
              ldsm2<true>(f2, sq + (ks * 16 + (lane & 15)) * q_stride + col * 2);
              fb[0] = f2[0];
              fb[1] = f2[1];
            }
#pragma unroll
            for (int e = kT - 1; e >= 0; --e) {   // smallest terms first
              uint32_t fa[4];
              ldsm4<false>(fa, s_base + (e * kRows + (lane & 15)) * s_stride + 32 * ks + (lane >> 4) * 16);
              mma16816(acc[0], fa, fb[0], fb[1]);
              if constexpr (kPairs == 2) mma16816(acc[1], fa, fb[2], fb[3]);
            }
          }
          if (p.r & 8) {   // the last eight of the rank
            uint32_t fb[2];
            // With one 8-column tile both halves of the load read it.
            ldsm2<true>(fb, sq + (ks * 16 + (lane & 7)) * q_stride + col * 2 + (kPairs == 2 ? (lane >> 3) & 1 : 0) * 16);
#pragma unroll
            for (int e = kT - 1; e >= 0; --e) {
              uint32_t fa[2];
              ldsm2<false>(fa, s_base + (e * kRows + (lane & 15)) * s_stride + 32 * ks);
              mma1688(acc[0], fa, fb[0]);
              if constexpr (kPairs == 2) mma1688(acc[1], fa, fb[1]);
            }
          }
        }
#pragma unroll
        for (int i = 0; i < kPairs; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint8_t* o = sb + (8 * h + (lane >> 2)) * kRowStride + (col + 8 * i + 2 * (lane & 3)) * kSize;
            float x = acc[i][2 * h], y = acc[i][2 * h + 1];
            if constexpr (kF32) {
              if (from != nullptr) {
                const float2 b = *reinterpret_cast<const float2*>(o);
                x += b.x;
                y += b.y;
              }
              *reinterpret_cast<float2*>(o) = make_float2(x, y);
            } else {
              if (from != nullptr) {
                const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(o));
                x += b.x;
                y += b.y;
              }
              *reinterpret_cast<__nv_bfloat162*>(o) = __floats2bfloat162_rn(x, y);
            }
          }
      }
      __syncthreads();
      if (has && kPiece * qx < left)
        *reinterpret_cast<uint4*>(to + at + it * 256) = *reinterpret_cast<const uint4*>(sb + xm * kRowStride + 16 * qx);
      if (++stage == p.stages) stage = 0;
    }
    __syncthreads();   // the next group's copies and s' go where this one's were
  }
}

// ---------------------------------------------------------------- forward
// Both products of the forward pass in one launch: a cluster of CTAs takes an item, its ranks the
// contraction of shrink by ranges, exchange their sums through distributed shared memory, and take
// the columns of expand by ranges.  (Asking for the weights' way to L2 ahead of time made it slower, 29.6
// against 26.6 us for 256 rows of 48 adapters: the loads of 16 warps an SM keep memory as busy.)
// 16 rows of 16 adapters of rank 16 (4096 -> 4096, 4.6 MB) take 7.0 us, nearly all of it start, two chains of
// loads and the cluster's exchange; 256 rows of 48 of rank 32 (4096 -> 12288, 65 MB) 27.8 to 28.9 us, 2.3 TB/s: an item is a
// chain of grouping, shrink, exchange and expand, and there are too few of them to hide one's waits under another's.
//
// shrink: each warp takes 32 elements of the contraction at a time: lane (g, q) loads elements
// 8 q .. 8 q + 7 of row g of the adapter (for each eight of the rank) and of the item's rows g and
// g + 8; the halves of these 16 bytes are the fragments of two MMAs.
// expand: a warp takes 32 columns at a time as four 8-column tiles whose columns are interleaved,
// so that lane (g, q) ends up with columns 8 q .. 8 q + 7 of the rows g and g + 8: 16 bytes of bf16.
struct ForwardParams {
  const __nv_bfloat16* x;     // [M][K]
  const __nv_bfloat16* a;     // [n][r][K]
  const __nv_bfloat16* b;     // [n][N][r]
  const float* scale;         // [n]
  const int* ids;
  const void* base;           // [M][N] or nullptr
  void* out;                  // [M][N]
  float* hidden;              // [M][r] or nullptr
  int64_t M, K, N;
  int n, r, zs;               // zs: clusters (or groups of `parts`) that share the items of one chunk
  int cluster, parts;         // parts: clusters that share the columns of one item, each with all of its shrink
};

constexpr int64_t kSumPart = 16384;   // contraction elements that a CTA adds up in the MMAs' accumulators

template <int kJ, bool kF32>   // kJ: 8-column tiles of the rank, at most
__global__ void __launch_bounds__(kThreads, kJ <= 8 ? 2 : 1) rfq_lora_forward_kernel(const ForwardParams p) {
  constexpr int kT = kExpandTerms<kF32>;
  constexpr int kSmRow = kJ * 8 + 8;
  constexpr int kRedBytes = 4 * kRows * kJ * 8 * 4, kSmBytes = kT * kRows * kSmRow * 2;
  __shared__ __align__(16) Groups g;
  __shared__ __align__(16) float sums[kRows * kJ * 8];
  __shared__ __align__(16) uint8_t pool[kRedBytes > kSmBytes ? kRedBytes : kSmBytes];
  float (*red)[kRows][kJ * 8] = reinterpret_cast<float (*)[kRows][kJ * 8]>(pool);              // shrink: [4]
  __nv_bfloat16 (*sm)[kRows][kSmRow] = reinterpret_cast<__nv_bfloat16 (*)[kRows][kSmRow]>(pool);   // expand: [kT]
  griddep_launch_dependents();
  griddep_wait();
  const int rank = static_cast<int>(cluster_cta_rank());
  const int64_t cluster = blockIdx.x / p.cluster;
  const int part = static_cast<int>(cluster % p.parts);
  const int64_t row0 = cluster / p.parts / p.zs * kChunk;
  const int z = static_cast<int>(cluster / p.parts % p.zs);
  group_rows(g, p.ids, row0, p.M, p.n);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quad = lane & 3, line = lane >> 2;
  const int jt = p.r / 8;
  // This rank's part of the contraction (of 32 elements a step) and of the columns (of 32).
  const int64_t k_per = ceil_div(ceil_div(p.K, 32), p.cluster) * 32, k0 = rank * k_per, k1 = min(p.K, k0 + k_per);
  const int64_t n_per = ceil_div(ceil_div(p.N, 32), p.cluster * p.parts) * 32, begin = (part * p.cluster + rank) * n_per,
                end = min(p.N, begin + n_per);
  const uint4 zero4 = make_uint4(0u, 0u, 0u, 0u);

  for (int item = z; item < g.items; item += p.zs) {   // the same items in every rank
    const int first = g.start[item], rows = g.start[item + 1] - first;
    const int a = g.ids[g.order[first]];
    const bool with = a != INT_MAX;
    if (p.hidden != nullptr && rank + part == 0 && !with)
      for (int i = tid; i < rows * p.r; i += kThreads) p.hidden[(row0 + g.order[first + i / p.r]) * p.r + i % p.r] = 0.f;
    // Rows without an adapter (they come last) keep what they have where the base is the output itself.
    if (!with && p.base == p.out) continue;
    const bool has[2] = {line < rows, line + 8 < rows};
    const int64_t row[2] = {row0 + g.order[first + (has[0] ? line : 0)], row0 + g.order[first + (has[1] ? line + 8 : 0)]};
    // Column of this lane's fragment row in tile i of expand: 8 (g / 2) + 2 i + (g & 1).
    const __nv_bfloat16* qa = with ? p.b + (static_cast<int64_t>(a) * p.N + 8 * (line >> 1) + (line & 1)) * p.r : p.b;
    if (with) {
      const __nv_bfloat16* xa = p.x + row[0] * p.K;
      const __nv_bfloat16* xb = p.x + row[1] * p.K;
      const __nv_bfloat16* pa = p.a + (static_cast<int64_t>(a) * p.r + line) * p.K;
      // The MMAs add by truncation (7e-4 of a sum of one sign over 2^20 elements, 2.7e-6 in parts of 16384): a part at a time, added with rounding.
      for (int64_t s0 = k0; s0 == k0 || s0 < k1; s0 += kSumPart) {
        const int64_t s1 = min(k1, s0 + kSumPart);
        float acc[kJ][4];
#pragma unroll
        for (int j = 0; j < kJ; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
#pragma unroll(kJ <= 4 ? 2 : 1)
        for (int64_t c = s0 + 32 * warp + 8 * quad; c < s1 + 8 * quad; c += 8 * 32) {
          const bool ok = c < s1;
          const uint4 ua = ok && has[0] ? *reinterpret_cast<const uint4*>(xa + c) : zero4;
          const uint4 ub = ok && has[1] ? *reinterpret_cast<const uint4*>(xb + c) : zero4;
          const uint32_t f0[4] = {ua.x, ub.x, ua.y, ub.y}, f1[4] = {ua.z, ub.z, ua.w, ub.w};
          uint4 w[kJ];
#pragma unroll
          for (int j = 0; j < kJ; ++j) w[j] = ok && j < jt ? *reinterpret_cast<const uint4*>(pa + 8 * j * p.K + c) : zero4;
#pragma unroll
          for (int j = 0; j < kJ; ++j)
            if (j < jt) {
              mma16816(acc[j], f0, w[j].x, w[j].y);
              mma16816(acc[j], f1, w[j].z, w[j].w);
            }
        }
        // The warps' sums: four and four, then the others to the first.
        auto give = [&](int slot) {
#pragma unroll
          for (int j = 0; j < kJ; ++j) {
            const int col = j * 8 + 2 * quad;
            *reinterpret_cast<float2*>(&red[slot][line][col]) = make_float2(acc[j][0], acc[j][1]);
            *reinterpret_cast<float2*>(&red[slot][line + 8][col]) = make_float2(acc[j][2], acc[j][3]);
          }
        };
        auto take = [&](int slot) {
#pragma unroll
          for (int j = 0; j < kJ; ++j) {
            const int col = j * 8 + 2 * quad;
            const float2 ua = *reinterpret_cast<const float2*>(&red[slot][line][col]);
            const float2 ub = *reinterpret_cast<const float2*>(&red[slot][line + 8][col]);
            acc[j][0] += ua.x;
            acc[j][1] += ua.y;
            acc[j][2] += ub.x;
            acc[j][3] += ub.y;
          }
        };
        if (s0 > k0) __syncthreads();   // the first warp is done with the part before
        if (warp >= 4) give(warp - 4);
        __syncthreads();
        if (warp < 4) take(warp);
        __syncthreads();
        if (warp > 0 && warp < 4) give(warp);
        __syncthreads();
        if (warp == 0) {
          for (int w = 1; w < 4; ++w) take(w);
#pragma unroll
          for (int j = 0; j < kJ; ++j) {
            const int col = j * 8 + 2 * quad;
            float2* at[2] = {reinterpret_cast<float2*>(&sums[line * kJ * 8 + col]), reinterpret_cast<float2*>(&sums[(line + 8) * kJ * 8 + col])};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float2 v = make_float2(acc[j][2 * h], acc[j][2 * h + 1]);
              if (s0 > k0) {
                v.x += at[h]->x;
                v.y += at[h]->y;
              }
              *at[h] = v;
            }
          }
        }
      }
      cluster_sync();   // every rank's sums are there
      const float scale = p.scale[a];
      const uint32_t sums_addr = smem_addr(sums);
      for (int i = tid; i < rows * p.r / 4; i += kThreads) {
        const int m = i / (p.r / 4), j = (i - m * (p.r / 4)) * 4;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int k = 0; k < p.cluster; ++k) {
          const float4 u = ld_shared_cluster_f32x4(map_to_cta(sums_addr + (m * kJ * 8 + j) * 4, k));
          v.x += u.x;
          v.y += u.y;
          v.z += u.z;
          v.w += u.w;
        }
        const float f[4] = {v.x * scale, v.y * scale, v.z * scale, v.w * scale};
        if (p.hidden != nullptr && rank + part == 0) *reinterpret_cast<float4*>(p.hidden + (row0 + g.order[first + m]) * p.r + j) = make_float4(f[0], f[1], f[2], f[3]);
#pragma unroll
        for (int e4 = 0; e4 < 4; ++e4) {
          __nv_bfloat16 t[kT];
          split_terms<kT>(f[e4], t);
#pragma unroll
          for (int e = 0; e < kT; ++e) sm[e][m][j + e4] = t[e];
        }
      }
      __syncthreads();
      cluster_arrive();   // this CTA is done with the others' sums; waited for before its own change
    }

    // All loads of 32 columns, then their MMAs.
    constexpr int kK = kJ / 2;             // steps of 16 along the rank, at most
    constexpr int kRaw = kF32 ? 2 : 1;
    const int whole = p.r / 16;
    const bool half = (p.r & 8) != 0;
    const __nv_bfloat16* q0 = qa + (begin + 32 * warp) * p.r + 4 * quad;
    int64_t at[2] = {(row[0] * p.N + begin + 32 * warp + 8 * quad) * (kF32 ? 4 : 2), (row[1] * p.N + begin + 32 * warp + 8 * quad) * (kF32 ? 4 : 2)};
    for (int64_t c = begin + 32 * warp; c < end; c += 8 * 32) {
      const bool full = c + 32 <= p.N;       // else the last columns, some of them missing
      const bool col_ok = full || c + 8 * quad < p.N;
      uint4 raw[2][kRaw];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < kRaw; ++e)
          raw[h][e] = p.base != nullptr && has[h] && col_ok ? *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.base) + at[h] + 16 * e) : zero4;
      float acc[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
      if (with) {
        uint2 w[kK][4];
        const __nv_bfloat16* q = q0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool ok = full || c + 8 * (line >> 1) + 2 * i + (line & 1) < p.N;
#pragma unroll
          for (int k = 0; k < kK; ++k) {
            w[k][i] = make_uint2(0u, 0u);
            if (k < whole) {
              if (ok) w[k][i] = *reinterpret_cast<const uint2*>(q + 16 * k);
            } else if (k == whole && half) {   // the last eight of the rank
              if (ok) w[k][i].x = *reinterpret_cast<const uint32_t*>(q + 16 * k - 2 * quad);
            }
          }
          q += 2 * p.r;
        }
        q0 += 8 * 32 * p.r;
#pragma unroll
        for (int k = 0; k < kK; ++k) {
          if (k < whole) {
#pragma unroll
            for (int e = kT - 1; e >= 0; --e) {   // smallest terms first
              const uint2 sa = *reinterpret_cast<const uint2*>(&sm[e][line][16 * k + 4 * quad]);
              const uint2 sb = *reinterpret_cast<const uint2*>(&sm[e][line + 8][16 * k + 4 * quad]);
              const uint32_t fa[4] = {sa.x, sb.x, sa.y, sb.y};
#pragma unroll
              for (int i = 0; i < 4; ++i) mma16816(acc[i], fa, w[k][i].x, w[k][i].y);
            }
          } else if (k == whole && half) {
#pragma unroll
            for (int e = kT - 1; e >= 0; --e) {
              const uint32_t fa[2] = {*reinterpret_cast<const uint32_t*>(&sm[e][line][16 * k + 2 * quad]),
                                      *reinterpret_cast<const uint32_t*>(&sm[e][line + 8][16 * k + 2 * quad])};
#pragma unroll
              for (int i = 0; i < 4; ++i) mma1688(acc[i], fa, w[k][i].x);
            }
          }
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint4* o = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) + at[h]);
        at[h] += 8 * 32 * (kF32 ? 4 : 2);
        if (!has[h] || !col_ok) continue;
        if constexpr (kF32) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint4 u = raw[h][e];
            o[e] = make_uint4(__float_as_uint(__uint_as_float(u.x) + acc[2 * e][2 * h]), __float_as_uint(__uint_as_float(u.y) + acc[2 * e][2 * h + 1]),
                              __float_as_uint(__uint_as_float(u.z) + acc[2 * e + 1][2 * h]),
                              __float_as_uint(__uint_as_float(u.w) + acc[2 * e + 1][2 * h + 1]));
          }
        } else {
          const uint32_t u[4] = {raw[h][0].x, raw[h][0].y, raw[h][0].z, raw[h][0].w};
          uint32_t v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(u[i] << 16) + acc[i][2 * h],
                                                           __uint_as_float(u[i] & 0xffff0000u) + acc[i][2 * h + 1]);
            v[i] = *reinterpret_cast<const uint32_t*>(&b);
          }
          *o = make_uint4(v[0], v[1], v[2], v[3]);
        }
      }
    }
    __syncthreads();          // the next item's sums go where this one's terms were
    if (with) cluster_wait();
  }
}

// ---------------------------------------------------------------- split
// The rank-r vectors as bf16 terms [M][term][r]: ds' from its partial sums (after the shrink of short
// batches; that of long ones leaves terms), s' as saved by the forward pass.  Rows without an adapter are never read by what follows.
struct SplitParams {
  const float* part;          // [splits][M][r]
  const float* scale;
  const int* ids;
  const float* hidden;        // [M][r]
  __nv_bfloat16* ds;          // [M][term][r] or nullptr
  __nv_bfloat16* s;           // [M][term][r] or nullptr
  int64_t M;
  int n, r, splits;
};

template <int kT>
__global__ void __launch_bounds__(kThreads) rfq_lora_split_kernel(const SplitParams p) {
  griddep_launch_dependents();
  griddep_wait();
  const int64_t total = p.M * p.r;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < total; i += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int64_t m = i / p.r;
    const int a = p.ids[m];
    if (a < 0 || a >= p.n) continue;
    const int64_t at = m * kT * p.r + (i - m * p.r);
    __nv_bfloat16 t[kT];
    if (p.ds != nullptr) {
      split_terms<kT>(join_parts(p.part, p.splits, total, i, p.scale[a]), t);
#pragma unroll
      for (int e = 0; e < kT; ++e) p.ds[at + e * p.r] = t[e];
    }
    if (p.s != nullptr) {
      split_terms<kT>(p.hidden[i], t);
#pragma unroll
      for (int e = 0; e < kT; ++e) p.s[at + e * p.r] = t[e];
    }
  }
}

// ---------------------------------------------------------------- outer
// part[range][a][j][c] = sum over the range's rows of adapter a of v[m][j] w[m][c], for the two
// pairs (v, w) = (ds', x) and (s', dy).
// Bound by reading x and dy at small ranks: 16384 rows of rank 16 (4096 -> 4096, 268 MB) take 61 us, 4.5 TB/s with
// L1 at 66 % (the transposing loads); stages of 64 rows with two CTAs an SM, in place of 32 with three, took 8 us
// more.  By the MMAs at large ones, which rfq_lora_wide.cu takes where batches are long.
constexpr int kOuterCols = 128;
constexpr int kOuterRows = 32;        // rows of one stage
constexpr int kMaxRange = 4096;       // rows of one range

constexpr int kOuterStatic = kMaxAdapters + 2 * kMaxRange + 64;   // its fixed shared memory

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
  int n, r, range;            // range: rows of one range
};

constexpr int kWStride = odd_stride(kOuterCols * 2);
template <int kT>
__host__ __device__ constexpr int outer_v_stride(int r) {
  return odd_stride(kT * r * 2);
}
template <int kT>
__host__ __device__ constexpr int outer_stage_bytes(int r) {
  return kOuterRows * (kWStride + outer_v_stride<kT>(r));
}
// Stages of the ring (four of the largest, rank 128 in three terms, fill one SM's shared memory).
constexpr int kOuterStages = 4;
constexpr int kMostBesideOuter = kOuterStages * outer_stage_bytes<3>(128) + 64;
static_assert(kMostBesideOuter + kOuterStatic + 1024 <= kSmemLimit, "the largest ring fits");

template <int kJ16, int kT>   // kJ16: 16-row tiles of the rank, at most
__global__ void __launch_bounds__(kThreads) rfq_lora_outer_kernel(const OuterParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ uint8_t here[kMaxAdapters];
  __shared__ uint16_t list[kMaxRange];
  __shared__ int warp_count[8];
  griddep_launch_dependents();
  griddep_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int tile = static_cast<int>(blockIdx.x);
  const bool second = tile >= p.side[0].tiles;
  if (second) tile -= p.side[0].tiles;
  const OuterSide s = second ? p.side[1] : p.side[0];
  const int range = static_cast<int>(blockIdx.y);
  const int64_t row0 = static_cast<int64_t>(range) * p.range;
  const int count = static_cast<int>(min(static_cast<int64_t>(p.range), p.M - row0));
  const int64_t c0 = static_cast<int64_t>(tile) * kOuterCols;
  const int v_stride = outer_v_stride<kT>(p.r);
  const int v_pieces = kT * p.r / 8;            // 16-byte pieces of a row of v
  const int stage_bytes = outer_stage_bytes<kT>(p.r);
  const uint32_t base = smem_addr(smem);
  const int j16 = (p.r + 15) / 16;
  const int qx = tid & 15;
  const bool qx_ok = c0 + 8 * qx < s.C;
  // This thread's 16-byte pieces of a stage's v: row, element in v, place in the stage.
  constexpr int kS = kOuterStages;
  const uint32_t w_to = (tid >> 4) * kWStride + 16 * qx;
  const int w_size = qx_ok ? 16 : 0;
  const int64_t w_step = 16 * s.C;
  constexpr int kVCopies = (kOuterRows * kT * kJ16 * 2 + kThreads - 1) / kThreads;
  int v_m[kVCopies], v_from[kVCopies];
  uint32_t v_to[kVCopies];
#pragma unroll
  for (int u = 0; u < kVCopies; ++u) {
    const int i = tid + kThreads * u, m = i / v_pieces, q = i - m * v_pieces;
    v_m[u] = m < kOuterRows ? m : kOuterRows;
    v_from[u] = m * s.ld + 8 * q;
    v_to[u] = m * v_stride + 16 * q;
  }

  for (int i = tid; i < p.n; i += kThreads) here[i] = 0;
  __syncthreads();
  for (int i = tid; i < count; i += kThreads) {
    const int id = p.ids[row0 + i];
    if (id >= 0 && id < p.n) here[id] = 1;
  }
  __syncthreads();
  if (blockIdx.x == 0 && blockIdx.z == 0)
    for (int i = tid; i < p.n; i += kThreads) p.present[static_cast<int64_t>(range) * p.n + i] = here[i];

  const int per = static_cast<int>(ceil_div(count, kThreads));
  for (int a = static_cast<int>(blockIdx.z); a < p.n; a += gridDim.z) {
    if (!here[a]) continue;
    // The rows of this adapter, in order.
    int mine = 0;
    for (int i = tid * per; i < min(count, (tid + 1) * per); ++i) mine += p.ids[row0 + i] == a;
    int before = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, before, d);
      if (lane >= d) before += o;
    }
    __syncthreads();   // the adapter before this one is done with list, warp_count and the stages
    if (lane == 31) warp_count[warp] = before;
    __syncthreads();
    int total = 0, offset = before - mine;
    for (int w = 0; w < 8; ++w) {
      if (w < warp) offset += warp_count[w];
      total += warp_count[w];
    }
    for (int i = tid * per; i < min(count, (tid + 1) * per); ++i)
      if (p.ids[row0 + i] == a) list[offset++] = static_cast<uint16_t>(i);
    __syncthreads();

    const int iters = (total + kOuterRows - 1) / kOuterRows;
    // Rows that are neighbours (one request, one adapter for all) are stepped through; others are looked
    // up in the list for each copy.
    const bool run = list[total - 1] - list[0] == total - 1;
    const __nv_bfloat16* w_at = qx_ok ? s.w + (row0 + list[0] + (tid >> 4)) * s.C + c0 + 8 * qx : s.w;
    const __nv_bfloat16* v_at = s.v + (row0 + list[0]) * s.ld;
    int load_stage = 0, load_at = 0;
    uint32_t load_to = base;
    auto load = [&]() {
      if (run && load_at + kOuterRows <= total) {   // whole stages of neighbours, the usual ones
        const __nv_bfloat16* from = w_at;
#pragma unroll
        for (int u = 0; u < kOuterRows / 16; ++u) {
          cp_async16_bytes(load_to + w_to + 16 * u * kWStride, from, w_size);
          from += w_step;
        }
        w_at = from;
#pragma unroll
        for (int u = 0; u < kVCopies; ++u)
          if (v_m[u] < kOuterRows) cp_async16_bytes(load_to + kOuterRows * kWStride + v_to[u], v_at + v_from[u], 16);
        v_at += kOuterRows * s.ld;
      } else if (load_at < total) {
        const uint32_t sw = load_to, sv = sw + kOuterRows * kWStride;
#pragma unroll
        for (int u = 0; u < kOuterRows / 16; ++u) {   // rows past the last: zeros
          const int m = (tid >> 4) + 16 * u;
          const bool ok = load_at + m < total && qx_ok;
          const __nv_bfloat16* from = w_at + 16 * u * s.C;
          if (!run && ok) from = s.w + (row0 + list[load_at + m]) * s.C + c0 + 8 * qx;
          cp_async16(sw + m * kWStride + 16 * qx, ok ? from : s.w, ok);
        }
        w_at += kOuterRows * s.C;
#pragma unroll
        for (int u = 0; u < kVCopies; ++u)
          if (v_m[u] < kOuterRows) {
            const bool ok = load_at + v_m[u] < total;
            const __nv_bfloat16* from = v_at + v_from[u];
            if (!run && ok) from = s.v + (row0 + list[load_at + v_m[u]]) * s.ld + v_from[u] - v_m[u] * s.ld;
            cp_async16(sv + v_to[u], ok ? from : s.v, ok);
          }
        v_at += kOuterRows * s.ld;
      }
      cp_commit();
      load_at += kOuterRows;
      load_to += stage_bytes;
      if (++load_stage == kS) {
        load_stage = 0;
        load_to = base;
      }
    };
    // fp32 results: the MMAs add by truncation, so each stage's 32 rows are summed on their own and
    // added to the rest with rounding.
    constexpr bool kFlush = kT == 3;
    float acc[kJ16][2][4], sum[kFlush ? kJ16 : 1][2][4];
#pragma unroll
    for (int j = 0; j < kJ16; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          acc[j][h][e] = 0.f;
          if constexpr (kFlush) sum[j][h][e] = 0.f;
        }
    for (int it = 0; it < kS - 1; ++it) load();
    int stage = 0;
    uint32_t sw = base;
    for (int it = 0; it < iters; ++it) {
      cp_wait_stage(kS);
      __syncthreads();
      load();
      const uint32_t sv = sw + kOuterRows * kWStride;
#pragma unroll
      for (int ks = 0; ks < kOuterRows / 16; ++ks) {
        uint32_t fb[4];   // w: rows along the contraction; tiles of columns 16 * warp, + 8
        ldsm4<true>(fb, sw + (ks * 16 + (lane & 15)) * kWStride + 32 * warp + (lane >> 4) * 16);
#pragma unroll
        for (int j = 0; j < kJ16; ++j)
          if (j < j16) {
#pragma unroll
            for (int e = kT - 1; e >= 0; --e) {
              // v^T: 16 of the rank x 16 rows.  Where the rank ends after 8, the other 8 are whatever
              // lies behind (inside the stages): their results are not kept.
              uint32_t fa[4];
              ldsm4<true>(fa, sv + (ks * 16 + (lane & 7) + ((lane >> 4) << 3)) * v_stride + 2 * e * p.r + 32 * j + ((lane >> 3) & 1) * 16);
              mma16816(acc[j][0], fa, fb[0], fb[1]);
              mma16816(acc[j][1], fa, fb[2], fb[3]);
            }
          }
      }
      if constexpr (kFlush) {
#pragma unroll
        for (int j = 0; j < kJ16; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              sum[j][h][e] += acc[j][h][e];
              acc[j][h][e] = 0.f;
            }
      }
      sw += stage_bytes;
      if (++stage == kS) {
        stage = 0;
        sw = base;
      }
    }
    if constexpr (kFlush) {
#pragma unroll
      for (int j = 0; j < kJ16; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[j][h][e] = sum[j][h][e];
    }
    float* out = s.part + (static_cast<int64_t>(range) * p.n + a) * p.r * s.C;
#pragma unroll
    for (int j = 0; j < kJ16; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t c = c0 + 16 * warp + 8 * h + 2 * (lane & 3);
        const int ja = 16 * j + (lane >> 2), jb = ja + 8;
        if (c < s.C) {
          if (ja < p.r) *reinterpret_cast<float2*>(out + ja * s.C + c) = make_float2(acc[j][h][0], acc[j][h][1]);
          if (jb < p.r) *reinterpret_cast<float2*>(out + jb * s.C + c) = make_float2(acc[j][h][2], acc[j][h][3]);
        }
      }
  }
}

// ---------------------------------------------------------------- reduce
// dA[a][j][k] and dB[a][c][j] = the ranges' sums in order; an adapter without rows gets zeros.  A block takes
// kReduceTile elements of one adapter's dA, in the order in which they lie, or all of the rank for 32 columns of its dB,
// which is written transposed: through shared memory, so that both sides move in whole lines, and each
// thread's loads are under way together (one element after the other they took 43 us for the 17 MB of 5 adapters of
// rank 104, 6640 -> 9296, against 8.5 now).
struct ReduceSide {
  const float* part;
  void* out;
  int64_t C;
  int64_t tiles;              // blocks of one adapter
};
struct ReduceParams {
  ReduceSide side[2];         // dA, dB
  const int* present;
  int n, r, ranges;
};
constexpr int kReduceVecs = 4, kReduceTile = kThreads * kReduceVecs * 4;

template <bool kF32>
__device__ __forceinline__ void put4(void* out, int64_t at, const float4& v) {   // at: a multiple of 4
  if constexpr (kF32) {
    *reinterpret_cast<float4*>(static_cast<float*>(out) + at) = v;
  } else {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(out) + at) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  }
}

template <bool kF32>
__global__ void __launch_bounds__(kThreads) rfq_lora_reduce_kernel(const ReduceParams p) {
  __shared__ float tile[RFQ_LORA_MAX_RANK][33];
  griddep_launch_dependents();
  griddep_wait();
  const int tid = threadIdx.x;
  int64_t b = blockIdx.x;
  const bool second = b >= p.side[0].tiles * p.n;
  if (second) b -= p.side[0].tiles * p.n;
  const ReduceSide s = second ? p.side[1] : p.side[0];
  const int a = static_cast<int>(b / s.tiles);
  const int64_t t = b - a * s.tiles;
  const int64_t size = p.r * s.C;              // of one adapter
  const float* part = s.part + a * size;
  const int64_t step = static_cast<int64_t>(p.n) * size;
  // This thread's vectors: places in the adapter's [r][C], negative where there is none.  (A vector of four
  // lies in one row: C is a multiple of 8.)
  int64_t at[kReduceVecs];
  float4 sum[kReduceVecs];
#pragma unroll
  for (int u = 0; u < kReduceVecs; ++u) {
    sum[u] = make_float4(0.f, 0.f, 0.f, 0.f);
    const int i = tid + kThreads * u;
    if (!second) {
      at[u] = t * kReduceTile + 4 * i;
      if (at[u] >= size) at[u] = -1;
    } else {
      const int64_t c = t * 32 + (i & 7) * 4;
      at[u] = i >> 3 < p.r && c < s.C ? (i >> 3) * s.C + c : -1;
    }
  }
  for (int g = 0; g < p.ranges; ++g) {
    if (!p.present[static_cast<int64_t>(g) * p.n + a]) continue;
    const float* from = part + g * step;
    float4 v[kReduceVecs];
#pragma unroll
    for (int u = 0; u < kReduceVecs; ++u) v[u] = at[u] >= 0 ? *reinterpret_cast<const float4*>(from + at[u]) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int u = 0; u < kReduceVecs; ++u) {
      sum[u].x += v[u].x;
      sum[u].y += v[u].y;
      sum[u].z += v[u].z;
      sum[u].w += v[u].w;
    }
  }
  if (!second) {
#pragma unroll
    for (int u = 0; u < kReduceVecs; ++u)
      if (at[u] >= 0) put4<kF32>(s.out, a * size + at[u], sum[u]);
    return;
  }
#pragma unroll
  for (int u = 0; u < kReduceVecs; ++u) {
    const int i = tid + kThreads * u;
    if (i >> 3 < p.r) {
      float* to = &tile[i >> 3][(i & 7) * 4];
      to[0] = sum[u].x;
      to[1] = sum[u].y;
      to[2] = sum[u].z;
      to[3] = sum[u].w;
    }
  }
  __syncthreads();
  const int cols = static_cast<int>(min(static_cast<int64_t>(32), s.C - t * 32)), r4 = p.r / 4;
  const int64_t base = a * size + t * 32 * p.r;
  for (int i = tid; i < cols * r4; i += kThreads) {
    const int c = i / r4, j = (i - c * r4) * 4;
    put4<kF32>(s.out, base + 4 * i, make_float4(tile[j][c], tile[j + 1][c], tile[j + 2][c], tile[j + 3][c]));
  }
}
static_assert(kThreads * kReduceVecs >= RFQ_LORA_MAX_RANK * 8, "a block's vectors cover the rank for 32 columns");

// ---------------------------------------------------------------- host
constexpr int kPlanSms = 148;   // the cut does not depend on the device that runs it

// `most`: the dynamic shared memory that any call may ask of this kernel.  The limit that it sets belongs to the kernel, not to
// the launch: set to each launch's own size, a call of a smaller rank on another host thread could lower it between
// the two and make this launch fail.
template <class Kernel, class Params>
cudaError_t launch(Kernel kernel, const Params& p, dim3 grid, size_t smem, int most, cudaStream_t stream) {
  if (most > 0) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // see griddep_wait()
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// Dynamic shared memory of the kernels that have a Groups beside it, at most (1 KiB is the system's).
constexpr int kMostBesideGroups = kSmemLimit - 1024 - static_cast<int>(sizeof(Groups));

// Stages of a ring: three or four if two CTAs then share an SM, else as many as fit one (2 to 6).
int ring_stages(int stage_bytes, int other_bytes) {   // other_bytes: besides the ring and the Groups
  const int half = (kSmemLimit / 2 - 1024 - static_cast<int>(sizeof(Groups)) - other_bytes) / stage_bytes;
  if (half >= 3) return half < 4 ? half : 4;
  const int whole = (kMostBesideGroups - other_bytes) / stage_bytes;
  return whole < kMaxStages ? whole : kMaxStages;
}

// Whether a batch goes by chunks of 128 neighbouring rows (rfq_lora_wide.cu) or by groups of up to 16
// rows of one adapter.  A chunk is passed over once for each adapter in it, so there have to be more
// than 32 rows for each on average; and the two wide kernels take 15 us whatever they do, which is
// worth it from a size on.  Measured with one adapter, groups against chunks.  Forward, K = N = 4096:
// rank 16, 1000 rows 11 against 16 us, 3000 rows 31 against 24; rank 64, 300 rows 15 against 17,
// 1000 rows 21 against 18; 5120 -> 13824, rank 8, 1111 rows 30 against 25; an fp32 y counts half as
// much again (rank 16, 1000 rows 15 against 19 us, 2000 rows 24 against 26).  Backward (dx), K = N =
// 4096: rank 16, 128 rows 12 against 15 us, 1000 rows 25 against 16; rank 64, 128 rows 19 against 17.
// Rows sorted by adapter, that is.  The ids are on the device, so a batch whose rows are not goes by the same rule, and a chunk of it costs a
// pass for each adapter that it happens to hold: 4096 rows of 8 adapters of rank 16 in random order, 4096 -> 12288, 204 us against 60 sorted,
// of 100 adapters 1493 against 106 (include/rfq.h asks for sorted rows).
bool wide_forward(int64_t M, int64_t K, int64_t N, int64_t r, int64_t n, bool f32) {
  return M > 64 && M > 32 * n && M * (r + 8) * (K + N) / 2 * (f32 ? 3 : 2) > 330000000;
}
bool wide_backward(int64_t M, int64_t K, int64_t N, int64_t r, int64_t n) {
  return M > 64 && M > 32 * n && M * r * (K + N) > 60000000;
}

// Whether ds of a long batch comes from chunks too: a cluster of eight CTAs works on each, which leaves SMs
// idle below 2400 rows and passes over N / 8 once for each adapter in it.  Measured, whole backward pass, ds by groups
// against chunks: 5120 -> 13824, rank 8 of 3 adapters, 1000 rows 48 against 63 us, 2000 rows 69 against 76, 2900 rows 96 against 94; rank 16,
// 1000 rows 43 against 45, 2000 rows 63 against 57; rank 64, 300 rows 48 against 49, 1000 rows 84 against 71.
bool wide_ds(int64_t M, int64_t K, int64_t N, int64_t r, int64_t n) {
  return wide_backward(M, K, N, r, n) && M * r > 20000;
}

// Whether the adapters' gradients of a long batch go over tcgen05 too (rfq_lora_wide.cu): 64 rows of one adapter a
// stage, where the kernel here takes 32 and is bound by warp-level MMAs as the rank grows.  Measured, whole backward
// pass, there against here, K = N = 4096: rank 32, 1500 rows 42 against 46 us; rank 64, 2000 rows 51 against 65, 2500
// rows of 10 adapters 105 against 125, 300 rows of 4 66 against 51; rank 128, 400 rows 47 against 55, 2500 rows of 20
// 287 against 339; rows in random order are gathered and want the kernel here (dB alone, 16384 rows of 8 adapters, rank 32 209
// against 105, rank 64 224 against 153; of 16, rank 128 354 against 377).  At rank 16 both read x and dy at nearly the same rate and the one here gathers rows that are
// not neighbours faster: one adapter, 4000 rows 60 against 59, 8000 rows 86 against 88, 16384 rows 140 against 147; 4
// adapters row by row, 16384 rows 373 against 286.
bool wide_outer(int64_t M, int64_t K, int64_t N, int64_t r, int64_t n) {
  return wide_backward(M, K, N, r, n) && (r > 16 ? M > 96 * n : n == 1 && M > 6000);
}

// CTAs that share the groups of one chunk: one for each there can be, up to `most` over all chunks.
int64_t chunk_ctas(int64_t M, int64_t n, int64_t most) {
  const int64_t chunks = ceil_div(M, kChunk), rows = M < kChunk ? M : kChunk;
  int64_t z = n + 1 + rows / kRows;   // every adapter, the rows without one, and groups that are full
  if (z > rows) z = rows;
  if (chunks * z > most) z = most / chunks;
  return z > 1 ? z : 1;
}

// Splits of the shrink product's contraction: one wave of three CTAs per SM, 256 elements each at least, kSumPart at most.
int shrink_splits(int64_t M, int64_t C, int64_t n, int64_t* c_split, int* zs) {
  const int64_t chunks = ceil_div(M, kChunk), z = chunk_ctas(M, n, 2 * kPlanSms);
  const int64_t most = ceil_div(C, 256);
  int64_t s = 3 * kPlanSms / (chunks * z);
  if (s > most) s = most;
  if (s > 32) s = 32;
  if (s < ceil_div(C, kSumPart)) s = ceil_div(C, kSumPart);
  *c_split = ceil_div(ceil_div(C, s), 256) * 256;
  *zs = static_cast<int>(z);
  return static_cast<int>(ceil_div(C, *c_split));
}

cudaError_t shrink(const void* src, const void* w, const int* ids, int* table, float* part, int64_t M, int64_t C, int64_t n, int64_t r,
                   int* splits, cudaStream_t stream) {
  ShrinkParams p = {};
  p.src = static_cast<const __nv_bfloat16*>(src);
  p.p = static_cast<const __nv_bfloat16*>(w);
  p.ids = ids;
  p.table = table;
  p.part = part;
  p.M = M;
  p.C = C;
  p.n = static_cast<int>(n);
  p.r = static_cast<int>(r);
  *splits = shrink_splits(M, C, n, &p.c_split, &p.zs);
  const dim3 grid(static_cast<unsigned>(ceil_div(M, kChunk) * p.zs), static_cast<unsigned>(*splits));
  const int stage = kRows * kRowStride + shrink_p_bytes(p.r), red = shrink_red_bytes(p.r);
  p.stages = ring_stages(stage, red);
  const size_t smem = static_cast<size_t>(p.stages) * stage + red;
  if (r <= 16) return launch(rfq_lora_shrink_kernel<2>, p, grid, smem, kMostBesideGroups, stream);
  if (r <= 32) return launch(rfq_lora_shrink_kernel<4>, p, grid, smem, kMostBesideGroups, stream);
  if (r <= 64) return launch(rfq_lora_shrink_kernel<8>, p, grid, smem, kMostBesideGroups, stream);
  return launch(rfq_lora_shrink_kernel<16>, p, grid, smem, kMostBesideGroups, stream);
}

template <bool kF32>
cudaError_t expand_typed(ExpandParams p, cudaStream_t stream) {
  const int64_t chunks = ceil_div(p.M, kChunk), z = chunk_ctas(p.M, p.n, 2 * kPlanSms);
  p.zs = static_cast<int>(z);
  // Column tiles of a CTA: one wave of two CTAs per SM.
  const int64_t tiles = ceil_div(p.C, kBN<kF32>);
  int64_t parts = 2 * kPlanSms / (chunks * z);
  if (parts > tiles) parts = tiles;
  if (parts < 1) parts = 1;
  p.tiles = static_cast<int>(ceil_div(tiles, parts));
  const dim3 grid(static_cast<unsigned>(chunks * z), static_cast<unsigned>(ceil_div(tiles, p.tiles)));
  const int stage = expand_stage_bytes<kF32>(p.r), other = expand_s_bytes<kF32>(p.r);
  p.stages = ring_stages(stage, other);
  return launch(rfq_lora_expand_kernel<kF32>, p, grid, static_cast<size_t>(p.stages) * stage + other, kMostBesideGroups, stream);
}

cudaError_t expand(const float* part, int splits, const float* scale, const void* w, const int* table, const void* base, void* out,
                   bool f32, int64_t M, int64_t C, int64_t n, int64_t r, cudaStream_t stream) {
  ExpandParams p = {};
  p.part = part;
  p.scale = scale;
  p.q = static_cast<const __nv_bfloat16*>(w);
  p.table = table;
  p.base = base;
  p.out = out;
  p.M = M;
  p.C = C;
  p.n = static_cast<int>(n);
  p.r = static_cast<int>(r);
  p.splits = splits;
  return f32 ? expand_typed<true>(p, stream) : expand_typed<false>(p, stream);
}

template <bool kF32>
cudaError_t forward_typed(const ForwardParams& p, int64_t clusters, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * p.cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // see griddep_wait()
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaError_t e = p.r <= 16   ? cudaLaunchKernelEx(&cfg, rfq_lora_forward_kernel<2, kF32>, p)
                  : p.r <= 32 ? cudaLaunchKernelEx(&cfg, rfq_lora_forward_kernel<4, kF32>, p)
                  : p.r <= 64 ? cudaLaunchKernelEx(&cfg, rfq_lora_forward_kernel<8, kF32>, p)
                              : cudaLaunchKernelEx(&cfg, rfq_lora_forward_kernel<16, kF32>, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int kJ16, int kT>
cudaError_t outer_typed(const OuterParams& p, dim3 grid, cudaStream_t stream) {
  // The last row's fragments may reach past its end.
  return launch(rfq_lora_outer_kernel<kJ16, kT>, p, grid, static_cast<size_t>(kOuterStages) * outer_stage_bytes<kT>(p.r) + 64,
                kMostBesideOuter, stream);
}
template <int kT>
cudaError_t outer_rank(const OuterParams& p, dim3 grid, cudaStream_t stream) {
  if (p.r <= 16) return outer_typed<1, kT>(p, grid, stream);
  if (p.r <= 32) return outer_typed<2, kT>(p, grid, stream);
  if (p.r <= 64) return outer_typed<4, kT>(p, grid, stream);
  return outer_typed<8, kT>(p, grid, stream);
}

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

// Rows of one range of the outer products: one wave of three CTAs per SM over all column tiles.
int outer_range(int64_t M, int64_t tiles) {
  const int64_t want = tiles < 3 * kPlanSms ? 3 * kPlanSms / tiles : 1;
  int64_t rows = ceil_div(ceil_div(M, want), kOuterRows) * kOuterRows;
  if (rows < 256) rows = 256;
  if (rows > kMaxRange) rows = kMaxRange;
  return static_cast<int>(rows);
}

// The same for the tcgen05 kernel: one wave of one CTA per SM, 256 columns each.
int outer_range_wide(int64_t M, int64_t tiles) {
  const int64_t want = tiles < kPlanSms ? kPlanSms / tiles : 1;
  int64_t rows = ceil_div(ceil_div(M, want), 64) * 64;
  if (rows < 256) rows = 256;
  if (rows > RFQ_LORA_OUTER_RANGE) rows = RFQ_LORA_OUTER_RANGE;
  return static_cast<int>(rows);
}

struct BackwardPlan {
  size_t table, part, counts, ds, s, part_a, part_b, present, bytes;
  int range, ranges;
};
// fp32 results take three terms, bf16 ones two; the workspace is sized for three.
BackwardPlan plan_backward(int64_t M, int64_t K, int64_t N, int64_t r, int64_t n) {
  BackwardPlan b;
  int64_t cs;
  int z;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += align256(bytes);
    return o;
  };
  b.range = wide_outer(M, K, N, r, n) ? outer_range_wide(M, ceil_div(K, 256) + ceil_div(N, 256)) : outer_range(M, ceil_div(K, kOuterCols) + ceil_div(N, kOuterCols));
  b.ranges = static_cast<int>(ceil_div(M, b.range));
  const bool chunks = wide_ds(M, K, N, r, n);
  b.table = take(chunks ? 0 : static_cast<size_t>(ceil_div(M, kChunk)) * kTable * 4);
  b.part = take(chunks ? 0 : static_cast<size_t>(shrink_splits(M, N, n, &cs, &z)) * M * r * 4);
  b.counts = take(chunks ? static_cast<size_t>(ceil_div(M, 128)) * 4 : 0);
  b.ds = take(static_cast<size_t>(3) * M * r * 2);
  b.s = take(static_cast<size_t>(3) * M * r * 2);
  b.part_a = take(static_cast<size_t>(b.ranges) * n * r * K * 4);
  b.part_b = take(static_cast<size_t>(b.ranges) * n * r * N * 4);
  b.present = take(static_cast<size_t>(b.ranges) * n * 4);
  b.bytes = at;
  return b;
}

}  // namespace

// Long batches leave s as bf16 terms, and how many adapters each chunk has; short ones need nothing (256 bytes, so
// that a workspace is one).
size_t lora_forward_workspace(int64_t M, int64_t K, int64_t N, int64_t r, int64_t n) {
  if (!wide_forward(M, K, N, r, n, true)) return 256;   // whatever y's type
  return align256(static_cast<size_t>(3) * M * r * 2) + align256(static_cast<size_t>(ceil_div(M, 128)) * 4);
}

size_t lora_backward_workspace(int64_t M, int64_t K, int64_t N, int64_t r, int64_t n) {
  return plan_backward(M, K, N, r, n).bytes;
}

cudaError_t launch_lora_forward(const void* x, const void* a, const void* b, const float* scale, const int* ids, const void* base,
                                void* y, bool y_bf16, float* hidden, int64_t M, int64_t K, int64_t N, int64_t r, int64_t n,
                                void* ws, int num_sms, void* encode_tiled, cudaStream_t stream) {
  cudaError_t e;
  if (wide_forward(M, K, N, r, n, !y_bf16)) {
    const int terms = y_bf16 ? 2 : 3;
    int* counts = reinterpret_cast<int*>(static_cast<uint8_t*>(ws) + align256(static_cast<size_t>(3) * M * r * 2));
    e = launch_lora_shrink_wide(x, a, false, ids, scale, hidden, ws, terms, counts, M, K, n, r, num_sms, encode_tiled, stream);
    if (e != cudaSuccess) return e;
    return launch_lora_expand_wide(ws, terms, counts, b, false, ids, base, y, !y_bf16, M, N, n, r, num_sms, encode_tiled, stream);
  }
  ForwardParams p = {};
  p.x = static_cast<const __nv_bfloat16*>(x);
  p.a = static_cast<const __nv_bfloat16*>(a);
  p.b = static_cast<const __nv_bfloat16*>(b);
  p.scale = scale;
  p.ids = ids;
  p.base = base;
  p.out = y;
  p.hidden = hidden;
  p.M = M;
  p.K = K;
  p.N = N;
  p.n = static_cast<int>(n);
  p.r = static_cast<int>(r);
  // Clusters of up to eight, as many as are resident at once.
  const int64_t chunks = ceil_div(M, kChunk), z = chunk_ctas(M, n, 2 * kPlanSms);
  p.zs = static_cast<int>(z);
  const int64_t slots = (r <= 64 ? 2 : 1) * kPlanSms;   // CTAs that are resident at once
  const int64_t ranks = slots / (chunks * z);
  p.cluster = static_cast<int>(ranks < 1 ? 1 : ranks > 8 ? 8 : ranks);
  // Few items: several clusters share the columns of one (256 columns a CTA at least).
  int64_t parts = slots / (chunks * z * p.cluster);
  const int64_t most = ceil_div(N, 256 * p.cluster);
  p.parts = static_cast<int>(parts < most ? parts : most);
  if (p.parts < 1) p.parts = 1;
  return y_bf16 ? forward_typed<false>(p, chunks * z * p.parts, stream) : forward_typed<true>(p, chunks * z * p.parts, stream);
}

cudaError_t launch_lora_backward(const void* x, const void* a, const void* b, const float* scale, const int* ids, const void* dy,
                                 const float* hidden, const void* dx_base, void* dx, bool dx_bf16, void* da, void* db,
                                 bool grad_bf16, int64_t M, int64_t K, int64_t N, int64_t r, int64_t n, void* ws, int num_sms,
                                 void* encode_tiled, cudaStream_t stream) {
  const BackwardPlan pl = plan_backward(M, K, N, r, n);
  uint8_t* base = static_cast<uint8_t*>(ws);
  float* part = reinterpret_cast<float*>(base + pl.part);
  int* table = reinterpret_cast<int*>(base + pl.table);
  int* counts = reinterpret_cast<int*>(base + pl.counts);
  __nv_bfloat16* ds = reinterpret_cast<__nv_bfloat16*>(base + pl.ds);
  __nv_bfloat16* s = reinterpret_cast<__nv_bfloat16*>(base + pl.s);
  const bool chunks = wide_backward(M, K, N, r, n), chunks_ds = wide_ds(M, K, N, r, n);
  const int terms = grad_bf16 ? 2 : 3;
  // Terms of ds' for expand and the adapters' gradients: what an fp32 dx or they need.
  const int ds_terms = chunks && dx != nullptr && !dx_bf16 ? 3 : terms;
  int splits = 1;
  cudaError_t e = cudaSuccess;
  if (dx != nullptr || da != nullptr) {
    e = chunks_ds ? launch_lora_shrink_wide(dy, b, true, ids, scale, nullptr, ds, ds_terms, counts, M, N, n, r, num_sms, encode_tiled, stream)
                  : shrink(dy, b, ids, table, part, M, N, n, r, &splits, stream);
    if (e != cudaSuccess) return e;
  }
  SplitParams sp = {};
  sp.part = part;
  sp.scale = scale;
  sp.ids = ids;
  sp.hidden = hidden;
  sp.M = M;
  sp.n = static_cast<int>(n);
  sp.r = static_cast<int>(r);
  sp.splits = splits;
  sp.ds = !chunks_ds && (da != nullptr || (chunks && dx != nullptr)) ? ds : nullptr;
  sp.s = db != nullptr ? s : nullptr;
  auto split = [&](int kind) {
    if (sp.ds == nullptr && sp.s == nullptr) return cudaSuccess;
    const int64_t blocks = ceil_div(M * r, kThreads);
    const dim3 sgrid(static_cast<unsigned>(blocks < 8 * kPlanSms ? blocks : 8 * kPlanSms));
    return kind == 2 ? launch(rfq_lora_split_kernel<2>, sp, sgrid, 0, 0, stream) : launch(rfq_lora_split_kernel<3>, sp, sgrid, 0, 0, stream);
  };
  // Expand over chunks reads ds' as terms, expand of groups forms them itself.
  const bool split_first = chunks && !chunks_ds;
  const int s_terms = split_first ? ds_terms : terms;
  if (split_first && (e = split(s_terms)) != cudaSuccess) return e;
  if (dx != nullptr) {
    e = chunks ? launch_lora_expand_wide(ds, ds_terms, chunks_ds ? counts : nullptr, a, true, ids, dx_base, dx, !dx_bf16, M, K, n, r, num_sms, encode_tiled, stream)
               : expand(part, splits, scale, a, table, dx_base, dx, !dx_bf16, M, K, n, r, stream);
    if (e != cudaSuccess) return e;
  }
  if (da == nullptr && db == nullptr) return e;
  if (!split_first && (e = split(s_terms)) != cudaSuccess) return e;
  float* part_a = reinterpret_cast<float*>(base + pl.part_a);
  float* part_b = reinterpret_cast<float*>(base + pl.part_b);
  int* present = reinterpret_cast<int*>(base + pl.present);
  const int ds_ld = static_cast<int>(ds_terms * r), s_ld = static_cast<int>(s_terms * r);
  if (wide_outer(M, K, N, r, n)) {
    e = launch_lora_outer_wide(ds, ds_ld, da != nullptr ? x : nullptr, part_a, K, s, s_ld, db != nullptr ? dy : nullptr, part_b, N, terms, ids, present,
                               M, n, r, pl.range, encode_tiled, stream);
  } else {
    OuterParams o = {};
    o.side[0] = {ds, ds_ld, static_cast<const __nv_bfloat16*>(x), part_a, K, da != nullptr ? static_cast<int>(ceil_div(K, kOuterCols)) : 0};
    o.side[1] = {s, s_ld, static_cast<const __nv_bfloat16*>(dy), part_b, N, db != nullptr ? static_cast<int>(ceil_div(N, kOuterCols)) : 0};
    o.ids = ids;
    o.present = present;
    o.M = M;
    o.n = static_cast<int>(n);
    o.r = static_cast<int>(r);
    o.range = pl.range;
    // Few CTAs and several adapters (short batches): the adapters are shared out too.
    const int64_t ctas = static_cast<int64_t>(o.side[0].tiles + o.side[1].tiles) * pl.ranges;
    int64_t zs = 2 * kPlanSms / ctas;
    if (zs > n) zs = n;
    if (zs < 1) zs = 1;
    const dim3 grid(static_cast<unsigned>(o.side[0].tiles + o.side[1].tiles), static_cast<unsigned>(pl.ranges), static_cast<unsigned>(zs));
    e = grad_bf16 ? outer_rank<2>(o, grid, stream) : outer_rank<3>(o, grid, stream);
  }
  if (e != cudaSuccess) return e;
  ReduceParams q = {};
  q.side[0] = {part_a, da, K, da != nullptr ? ceil_div(r * K, kReduceTile) : 0};
  q.side[1] = {part_b, db, N, db != nullptr ? ceil_div(N, 32) : 0};
  q.present = present;
  q.n = static_cast<int>(n);
  q.r = static_cast<int>(r);
  q.ranges = pl.ranges;
  const dim3 rgrid(static_cast<unsigned>((q.side[0].tiles + q.side[1].tiles) * n));
  return grad_bf16 ? launch(rfq_lora_reduce_kernel<false>, q, rgrid, 0, 0, stream) : launch(rfq_lora_reduce_kernel<true>, q, rgrid, 0, 0, stream);
}

}  // namespace rfq
