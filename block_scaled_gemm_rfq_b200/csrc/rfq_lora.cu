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
// dx written once per pass over them, at 2 r flops for each of their elements.  So the
// kernels are built around the wide matrices' rows and use warp-level m16n8k16 MMAs, whose
// operands may be transposed on the way from shared memory (A and B are each needed in
// both directions) and whose rows can be gathered:
//
//   shrink   s, ds: rows x wide -> rank, the contraction split over CTAs, partial sums fp32
//   expand   y, dx: rank -> wide, adds the partial sums in order, adds the base
//   split    s, ds as sums of bf16 terms for the next one
//   outer    dA, dB: contraction over rows, split into row ranges
//   reduce   sums the ranges in order and rounds
//
// The rows of a 128-row chunk are grouped by adapter inside the CTA that works on them (no
// host knowledge of the ids, no order asked of them): groups of up to kRows rows share an
// adapter's weights.  No atomics: a result does not depend on timing.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "rfq_internal.h"
#include "rfq_ptx.cuh"

namespace rfq {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 128;      // rows grouped by one CTA
constexpr int kStages = 4;

__host__ __device__ constexpr int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
// Row stride in shared memory, in 16-byte units: odd, so that eight rows at one column fall
// into eight different bank groups (ldmatrix without conflicts).
__host__ __device__ constexpr int odd_stride(int chunks16) { return chunks16 | 1; }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kN>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kN) : "memory");
}
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

// The rows of one chunk, grouped by adapter: order[] lists them (as offsets in the chunk) by
// rising adapter, rows without one last; item i is order[start[i] .. start[i + 1]), at most
// kRows rows of one adapter.
struct Groups {
  int ids[kChunk];
  int order[kChunk];
  int flag[kChunk];
  int start[kChunk + 1];
  int items;
};

template <int kRows>
__device__ void group_rows(Groups& g, const int* ids, int64_t row0, int64_t M, int n) {
  const int t = threadIdx.x;
  const int count = static_cast<int>(M - row0 < kChunk ? M - row0 : kChunk);
  int id = INT_MAX;
  if (t < kChunk) {
    if (t < count) {
      const int v = ids[row0 + t];
      if (v >= 0 && v < n) id = v;
    }
    g.ids[t] = id;
  }
  __syncthreads();
  if (t < count) {
    int less = 0, before = 0;
#pragma unroll 8
    for (int j = 0; j < count; ++j) {
      const int v = g.ids[j];
      less += v < id;
      before += v == id && j < t;
    }
    g.order[less + before] = t;
    g.flag[less + before] = before % kRows == 0;
  }
  __syncthreads();
  if (t < 32) {
    int items = 0;
    for (int w = 0; w < kChunk; w += 32) {
      const bool f = w + t < count && g.flag[w + t] != 0;
      const unsigned bits = __ballot_sync(0xffffffffu, f);
      if (f) g.start[items + __popc(bits & ((1u << t) - 1))] = w + t;
      items += __popc(bits);
    }
    if (t == 0) {
      g.start[items] = count;
      g.items = items;
    }
  }
  __syncthreads();
}

// ---------------------------------------------------------------- shrink
// part[split][m][j] = sum over the split's k of src[m][k] P_a[j][k], P = A (rows j, k along the
// row) or, kTrans, B (rows k, j along the row).
struct ShrinkParams {
  const __nv_bfloat16* src;   // [M][C]
  const __nv_bfloat16* p;     // [n][r][C] or [n][C][r]
  const int* ids;
  float* part;                // [splits][M][r]
  int64_t M, C, c_split;      // c_split: contraction elements of one split (a multiple of kBK)
  int n, r, zs;               // zs: CTAs that share the items of one chunk
};

template <int kRows>
struct ShrinkTile {
  static constexpr int kWm = kRows / 16;         // warps along the rows
  static constexpr int kWk = 8 / kWm;            // warps along a stage's contraction
  static constexpr int kBK = kWk == 8 ? 128 : 64;
  static constexpr int kSteps = kBK / 16 / kWk;  // k16 steps of a warp in one stage
  static constexpr int kXStride = odd_stride(kBK / 8);
  static constexpr int kXBytes = kRows * kXStride * 16;
};
template <int kRows, bool kTrans>
__host__ __device__ constexpr int shrink_p_stride(int r) {
  return kTrans ? odd_stride(r / 8) : odd_stride(ShrinkTile<kRows>::kBK / 8);
}
template <int kRows, bool kTrans>
__host__ __device__ constexpr int shrink_p_bytes(int r) {
  return (kTrans ? ShrinkTile<kRows>::kBK : r) * shrink_p_stride<kRows, kTrans>(r) * 16;
}

template <int kRows, bool kTrans, int kJ>   // kJ: 8-column tiles of the rank, at most
__global__ void __launch_bounds__(kThreads) rfq_lora_shrink_kernel(const ShrinkParams p) {
  using T = ShrinkTile<kRows>;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Groups g;
  __shared__ int64_t row_of[kRows];
  griddep_launch_dependents();
  griddep_wait();
  const int64_t row0 = static_cast<int64_t>(blockIdx.x / p.zs) * kChunk;
  const int z = static_cast<int>(blockIdx.x % p.zs);
  group_rows<kRows>(g, p.ids, row0, p.M, p.n);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int wm = warp % T::kWm, wk = warp / T::kWm;
  const int p_stride = shrink_p_stride<kRows, kTrans>(p.r);
  const int p_bytes = shrink_p_bytes<kRows, kTrans>(p.r);
  const int stage_bytes = T::kXBytes + p_bytes;
  const uint32_t base = smem_addr(smem);
  const int jt = p.r / 8;
  const int64_t c0 = static_cast<int64_t>(blockIdx.y) * p.c_split;
  const int64_t c1 = min(p.C, c0 + p.c_split);
  const int iters = static_cast<int>(ceil_div(c1 - c0, T::kBK));

  for (int item = z; item < g.items; item += p.zs) {
    const int first = g.start[item], rows = g.start[item + 1] - first;
    const int a = g.ids[g.order[first]];
    if (a == INT_MAX) break;   // rows without an adapter come last
    for (int i = tid; i < kRows; i += kThreads) row_of[i] = i < rows ? row0 + g.order[first + i] : -1;
    __syncthreads();
    const __nv_bfloat16* pa = p.p + static_cast<int64_t>(a) * p.r * p.C;

    auto load = [&](int it) {
      if (it < iters) {
        const uint32_t sx = base + (it % kStages) * stage_bytes, sp = sx + T::kXBytes;
        const int64_t c = c0 + static_cast<int64_t>(it) * T::kBK;
        for (int i = tid; i < kRows * (T::kBK / 8); i += kThreads) {
          const int m = i / (T::kBK / 8), q = i % (T::kBK / 8);
          const int64_t row = row_of[m];
          const bool ok = row >= 0 && c + 8 * q < c1;
          cp_async16(sx + (m * T::kXStride + q) * 16, ok ? p.src + row * p.C + c + 8 * q : p.src, ok);
        }
        if constexpr (kTrans) {
          for (int i = tid; i < T::kBK * jt; i += kThreads) {
            const int k = i / jt, q = i - k * jt;
            const bool ok = c + k < c1;
            cp_async16(sp + (k * p_stride + q) * 16, ok ? pa + (c + k) * p.r + 8 * q : p.p, ok);
          }
        } else {
          for (int i = tid; i < p.r * (T::kBK / 8); i += kThreads) {
            const int j = i / (T::kBK / 8), q = i % (T::kBK / 8);
            const bool ok = c + 8 * q < c1;
            cp_async16(sp + (j * p_stride + q) * 16, ok ? pa + static_cast<int64_t>(j) * p.C + c + 8 * q : p.p, ok);
          }
        }
      }
      cp_commit();
    };

    float acc[kJ][4];
#pragma unroll
    for (int j = 0; j < kJ; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
    for (int it = 0; it < kStages - 1; ++it) load(it);
    for (int it = 0; it < iters; ++it) {
      cp_wait<kStages - 2>();
      __syncthreads();
      load(it + kStages - 1);
      const uint32_t sx = base + (it % kStages) * stage_bytes, sp = sx + T::kXBytes;
#pragma unroll
      for (int s = 0; s < T::kSteps; ++s) {
        const int ks = wk * T::kSteps + s;
        uint32_t fa[4];
        ldsm4<false>(fa, sx + ((wm * 16 + (lane & 15)) * T::kXStride + 2 * ks + (lane >> 4)) * 16);
#pragma unroll
        for (int j = 0; j < kJ; j += 2) {
          if (j + 1 < jt) {
            uint32_t fb[4];
            if constexpr (kTrans) ldsm4<true>(fb, sp + ((ks * 16 + (lane & 15)) * p_stride + j + (lane >> 4)) * 16);
            else ldsm4<false>(fb, sp + ((j * 8 + (lane & 7) + ((lane >> 4) << 3)) * p_stride + 2 * ks + ((lane >> 3) & 1)) * 16);
            mma16816(acc[j], fa, fb[0], fb[1]);
            if constexpr (kJ > 1) mma16816(acc[j + 1], fa, fb[2], fb[3]);
          } else if (j < jt) {
            uint32_t fb[2];
            if constexpr (kTrans) ldsm2<true>(fb, sp + ((ks * 16 + (lane & 15)) * p_stride + j) * 16);
            else ldsm2<false>(fb, sp + ((j * 8 + (lane & 7)) * p_stride + 2 * ks + ((lane >> 3) & 1)) * 16);
            mma16816(acc[j], fa, fb[0], fb[1]);
          }
        }
      }
    }
    cp_wait<0>();
    __syncthreads();
    // Join the warps that shared a row tile (in order) and write [rows][r].
    float* red = reinterpret_cast<float*>(smem);   // [kWk][kRows][r]
#pragma unroll
    for (int j = 0; j < kJ; ++j)
      if (j < jt) {
        const int col = j * 8 + 2 * (lane & 3);
        float* at = red + (static_cast<int64_t>(wk) * kRows + wm * 16 + (lane >> 2)) * p.r + col;
        *reinterpret_cast<float2*>(at) = make_float2(acc[j][0], acc[j][1]);
        *reinterpret_cast<float2*>(at + 8 * p.r) = make_float2(acc[j][2], acc[j][3]);
      }
    __syncthreads();
    for (int i = tid; i < rows * p.r; i += kThreads) {
      const int m = i / p.r, j = i - m * p.r;
      float v = red[i];
#pragma unroll
      for (int w = 1; w < T::kWk; ++w) v += red[w * kRows * p.r + i];
      p.part[(static_cast<int64_t>(blockIdx.y) * p.M + row_of[m]) * p.r + j] = v;
    }
    __syncthreads();
  }
}

// s'[m][j] = scale_a * sum of the splits, in order.
__device__ __forceinline__ float join_parts(const float* part, int splits, int64_t stride, int64_t at, float scale) {
  float v = part[at];
  for (int s = 1; s < splits; ++s) v += part[s * stride + at];
  return v * scale;
}
// v as a sum of kT bf16 terms (8 bits each).
template <int kT>
__device__ __forceinline__ void split_terms(float v, __nv_bfloat16 (&t)[kT]) {
#pragma unroll
  for (int i = 0; i < kT; ++i) {
    t[i] = __float2bfloat16_rn(v);
    if (i + 1 < kT) v -= __bfloat162float(t[i]);
  }
}

// ---------------------------------------------------------------- expand
// out[m][c] = base[m][c] + sum_j s'[m][j] Q_a, Q = B (rows c, j along the row) or, kTrans, A
// (rows j, c along the row).
struct ExpandParams {
  const float* part;          // [splits][M][r]
  const float* scale;         // [n]
  const __nv_bfloat16* q;     // [n][C][r] or [n][r][C]
  const int* ids;
  const void* base;           // [M][C] or nullptr
  void* out;                  // [M][C]
  float* hidden;              // [M][r] or nullptr
  int64_t M, C;
  int n, r, splits, zs;
};

constexpr int kExpandCols = 256;
template <bool kTrans>
__host__ __device__ constexpr int expand_q_bytes(int r) {
  const int r16 = (r + 15) / 16 * 16;
  return kTrans ? r16 * odd_stride(kExpandCols / 8) * 16 : kExpandCols * odd_stride(r16 / 8) * 16;
}
template <int kRows, int kT>
__host__ __device__ constexpr int expand_s_bytes(int r) {
  return kT * kRows * odd_stride((r + 15) / 16 * 2) * 16;
}

template <int kRows, bool kTrans, bool kF32>
__global__ void __launch_bounds__(kThreads) rfq_lora_expand_kernel(const ExpandParams p) {
  // The rank-r vector enters the MMA in bf16: one term (2^-8 of the adapter's share, below the
  // rounding of a bf16 output) or, for an fp32 output, three (24 bits).
  constexpr int kT = kF32 ? 3 : 1;
  constexpr int kWm = kRows / 16, kWn = 8 / kWm;
  constexpr int kWarpCols = kExpandCols / kWn;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Groups g;
  __shared__ int64_t row_of[kRows];
  griddep_launch_dependents();
  griddep_wait();
  const int64_t row0 = static_cast<int64_t>(blockIdx.x / p.zs) * kChunk;
  const int z = static_cast<int>(blockIdx.x % p.zs);
  group_rows<kRows>(g, p.ids, row0, p.M, p.n);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int wm = warp % kWm, wn = warp / kWm;
  const int r16 = (p.r + 15) / 16 * 16;
  const int q_stride = kTrans ? odd_stride(kExpandCols / 8) : odd_stride(r16 / 8);
  const int s_stride = odd_stride(r16 / 8);
  const uint32_t sq = smem_addr(smem);
  uint8_t* s_bytes = smem + expand_q_bytes<kTrans>(p.r);
  const uint32_t ss = smem_addr(s_bytes);
  const int64_t c0 = static_cast<int64_t>(blockIdx.y) * kExpandCols;
  const int cols = static_cast<int>(min(static_cast<int64_t>(kExpandCols), p.C - c0));

  for (int item = z; item < g.items; item += p.zs) {
    const int first = g.start[item], rows = g.start[item + 1] - first;
    const int a = g.ids[g.order[first]];
    const bool with = a != INT_MAX;
    for (int i = tid; i < kRows; i += kThreads) row_of[i] = i < rows ? row0 + g.order[first + i] : -1;
    __syncthreads();
    if (with) {
      if constexpr (kTrans) {
        const __nv_bfloat16* qa = p.q + static_cast<int64_t>(a) * p.r * p.C;
        for (int i = tid; i < r16 * (kExpandCols / 8); i += kThreads) {
          const int j = i / (kExpandCols / 8), c = i % (kExpandCols / 8);
          const bool ok = j < p.r && 8 * c < cols;
          cp_async16(sq + (j * q_stride + c) * 16, ok ? qa + j * p.C + c0 + 8 * c : p.q, ok);
        }
      } else {
        const __nv_bfloat16* qa = p.q + (static_cast<int64_t>(a) * p.C + c0) * p.r;
        const int jc = r16 / 8;
        for (int i = tid; i < kExpandCols * jc; i += kThreads) {
          const int c = i / jc, j = i - c * jc;
          const bool ok = c < cols && 8 * j < p.r;
          cp_async16(sq + (c * q_stride + j) * 16, ok ? qa + static_cast<int64_t>(c) * p.r + 8 * j : p.q, ok);
        }
      }
      cp_commit();
      const float scale = p.scale[a];
      for (int i = tid; i < kRows * r16; i += kThreads) {
        const int m = i / r16, j = i - m * r16;
        float v = 0.f;
        if (m < rows && j < p.r) {
          v = join_parts(p.part, p.splits, p.M * p.r, row_of[m] * p.r + j, scale);
          if (p.hidden != nullptr && blockIdx.y == 0) p.hidden[row_of[m] * p.r + j] = v;
        }
        __nv_bfloat16 t[kT];
        split_terms<kT>(v, t);
#pragma unroll
        for (int e = 0; e < kT; ++e)
          *reinterpret_cast<__nv_bfloat16*>(s_bytes + ((e * kRows + m) * s_stride * 16) + 2 * j) = t[e];
      }
      cp_wait<0>();
    } else if (p.hidden != nullptr && blockIdx.y == 0) {
      for (int i = tid; i < rows * p.r; i += kThreads) p.hidden[row_of[i / p.r] * p.r + i % p.r] = 0.f;
    }
    __syncthreads();
    if (with || p.base != p.out) {
      // Each thread ends up with 8 neighbouring columns of two rows (16 bytes of bf16): it holds
      // two columns of each of four 8-column tiles, and the four lanes of a quad exchange them.
      const int quad = lane & 3;
      const int64_t row_a = row_of[wm * 16 + (lane >> 2)], row_b = row_of[wm * 16 + 8 + (lane >> 2)];
      // Before the loop over column groups: whether this thread has rows at all.
#pragma unroll 2
      for (int gcol = wn * kWarpCols; gcol < (wn + 1) * kWarpCols; gcol += 32) {
        if (gcol >= cols) break;
        const int col = gcol + 8 * quad;
        const bool col_ok = col < cols;
        float base_a[8], base_b[8];
        auto load_base = [&](float (&f)[8], int64_t row) {
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = 0.f;
          if (p.base == nullptr || row < 0 || !col_ok) return;
          const int64_t at = row * p.C + c0 + col;
          if constexpr (kF32) {
            const float4 u = *reinterpret_cast<const float4*>(static_cast<const float*>(p.base) + at);
            const float4 w = *reinterpret_cast<const float4*>(static_cast<const float*>(p.base) + at + 4);
            f[0] = u.x; f[1] = u.y; f[2] = u.z; f[3] = u.w;
            f[4] = w.x; f[5] = w.y; f[6] = w.z; f[7] = w.w;
          } else {
            const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.base) + at);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              f[2 * e] = __uint_as_float(w[e] << 16);
              f[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
            }
          }
        };
        load_base(base_a, row_a);
        load_base(base_b, row_b);
        if (with) {
          float acc[4][4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
          for (int ks = 0; ks < r16 / 16; ++ks) {
            uint32_t fb[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int c = gcol + 16 * h;
              if constexpr (kTrans) ldsm4<true>(fb[h], sq + ((ks * 16 + (lane & 15)) * q_stride + c / 8 + (lane >> 4)) * 16);
              else ldsm4<false>(fb[h], sq + ((c + (lane & 7) + ((lane >> 4) << 3)) * q_stride + 2 * ks + ((lane >> 3) & 1)) * 16);
            }
#pragma unroll
            for (int e = kT - 1; e >= 0; --e) {   // smallest terms first
              uint32_t fa[4];
              ldsm4<false>(fa, ss + ((e * kRows + wm * 16 + (lane & 15)) * s_stride + 2 * ks + (lane >> 4)) * 16);
              mma16816(acc[0], fa, fb[0][0], fb[0][1]);
              mma16816(acc[1], fa, fb[0][2], fb[0][3]);
              mma16816(acc[2], fa, fb[1][0], fb[1][1]);
              mma16816(acc[3], fa, fb[1][2], fb[1][3]);
            }
          }
          // 4 x 4 exchange inside each quad: lane q gives tile i to lane i and gets tile q from all.
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            // In step d lane q sends the pair of tile q ^ d and receives that of its own tile from lane q ^ d.
            const int from = quad ^ i;
            float send[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              send[e] = from == 0 ? acc[0][e] : from == 1 ? acc[1][e] : from == 2 ? acc[2][e] : acc[3][e];
#pragma unroll
            for (int e = 0; e < 4; ++e) send[e] = __shfl_xor_sync(0xffffffffu, send[e], i);
            // `from` is also the lane it came from: columns 2 * from, 2 * from + 1 of the tile.
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (from == k) {
                base_a[2 * k] += send[0];
                base_a[2 * k + 1] += send[1];
                base_b[2 * k] += send[2];
                base_b[2 * k + 1] += send[3];
              }
          }
        }
        auto store = [&](const float (&f)[8], int64_t row) {
          if (row < 0 || !col_ok) return;
          const int64_t at = row * p.C + c0 + col;
          if constexpr (kF32) {
            float* o = static_cast<float*>(p.out) + at;
            *reinterpret_cast<float4*>(o) = make_float4(f[0], f[1], f[2], f[3]);
            *reinterpret_cast<float4*>(o + 4) = make_float4(f[4], f[5], f[6], f[7]);
          } else {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * e], f[2 * e + 1]);
              w[e] = *reinterpret_cast<uint32_t*>(&b);
            }
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + at) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        };
        store(base_a, row_a);
        store(base_b, row_b);
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------- split
// The rank-r vectors as bf16 terms [term][M][r]: ds' from its partial sums, s' as saved by the
// forward pass.  Rows without an adapter are never read by what follows.
template <int kT>
__global__ void __launch_bounds__(kThreads) rfq_lora_split_kernel(const float* part, const float* scale, const int* ids, int n, int64_t M,
                                                                  int r, int splits, __nv_bfloat16* ds, const float* hidden,
                                                                  __nv_bfloat16* s) {
  griddep_launch_dependents();
  griddep_wait();
  const int64_t total = M * r;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < total; i += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int a = ids[i / r];
    if (a < 0 || a >= n) continue;
    __nv_bfloat16 t[kT];
    if (ds != nullptr) {
      split_terms<kT>(join_parts(part, splits, total, i, scale[a]), t);
#pragma unroll
      for (int e = 0; e < kT; ++e) ds[e * total + i] = t[e];
    }
    if (s != nullptr) {
      split_terms<kT>(hidden[i], t);
#pragma unroll
      for (int e = 0; e < kT; ++e) s[e * total + i] = t[e];
    }
  }
}

// ---------------------------------------------------------------- outer
// part[range][a][j][c] = sum over the range's rows of adapter a of v[m][j] w[m][c], for the two
// pairs (v, w) = (ds', x) and (s', dy).
constexpr int kOuterCols = 128;
constexpr int kOuterRows = 32;        // rows of one stage
constexpr int kMaxRange = 4096;       // rows of one range
constexpr int kMaxAdapters = 4096;

struct OuterSide {
  const __nv_bfloat16* v;     // [term][M][r]
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

template <int kT>
__host__ __device__ constexpr int outer_stage_bytes(int r) {
  return kOuterRows * odd_stride(kOuterCols / 8) * 16 + kT * kOuterRows * odd_stride((r + 15) / 16 * 2) * 16;
}

template <int kJ16, int kT>   // kJ16: 16-row tiles of the rank, at most
__global__ void __launch_bounds__(kThreads) rfq_lora_outer_kernel(const OuterParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ uint8_t here[kMaxAdapters];
  __shared__ uint16_t list[kMaxRange];
  __shared__ int16_t rid[kMaxRange];
  __shared__ int warp_count[8];
  griddep_launch_dependents();
  griddep_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int tile = static_cast<int>(blockIdx.x);
  const int which = tile >= p.side[0].tiles;
  if (which) tile -= p.side[0].tiles;
  const OuterSide s = which ? p.side[1] : p.side[0];
  const int range = static_cast<int>(blockIdx.y);
  const int64_t row0 = static_cast<int64_t>(range) * p.range;
  const int count = static_cast<int>(min(static_cast<int64_t>(p.range), p.M - row0));
  const int64_t c0 = static_cast<int64_t>(tile) * kOuterCols;
  const int r16 = (p.r + 15) / 16 * 16;
  const int j16 = r16 / 16;
  constexpr int kWStride = odd_stride(kOuterCols / 8);
  const int v_stride = odd_stride(r16 / 8);
  constexpr int kWBytes = kOuterRows * kWStride * 16;
  const int stage_bytes = outer_stage_bytes<kT>(p.r);
  const uint32_t base = smem_addr(smem);

  for (int i = tid; i < p.n; i += kThreads) here[i] = 0;
  __syncthreads();
  for (int i = tid; i < count; i += kThreads) {
    const int id = p.ids[row0 + i];
    const bool ok = id >= 0 && id < p.n;
    rid[i] = ok ? static_cast<int16_t>(id) : int16_t(-1);
    if (ok) here[id] = 1;
  }
  __syncthreads();
  if (blockIdx.x == 0)
    for (int i = tid; i < p.n; i += kThreads) p.present[static_cast<int64_t>(range) * p.n + i] = here[i];

  for (int a = 0; a < p.n; ++a) {
    if (!here[a]) continue;
    // The rows of this adapter, in order.
    const int per = static_cast<int>(ceil_div(count, kThreads));
    int mine = 0;
    for (int i = tid * per; i < min(count, (tid + 1) * per); ++i) mine += rid[i] == a;
    int before = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, before, d);
      if (lane >= d) before += o;
    }
    if (lane == 31) warp_count[warp] = before;
    __syncthreads();
    int total = 0, offset = before - mine;
    for (int w = 0; w < 8; ++w) {
      if (w < warp) offset += warp_count[w];
      total += warp_count[w];
    }
    for (int i = tid * per; i < min(count, (tid + 1) * per); ++i)
      if (rid[i] == a) list[offset++] = static_cast<uint16_t>(i);
    __syncthreads();

    const int iters = (total + kOuterRows - 1) / kOuterRows;
    auto load = [&](int it) {
      if (it < iters) {
        const uint32_t sw = base + (it % kStages) * stage_bytes, sv = sw + kWBytes;
        for (int i = tid; i < kOuterRows * (kOuterCols / 8); i += kThreads) {
          const int m = i / (kOuterCols / 8), q = i % (kOuterCols / 8);
          const int at = it * kOuterRows + m;
          const bool ok = at < total && c0 + 8 * q < s.C;
          cp_async16(sw + (m * kWStride + q) * 16, ok ? s.w + (row0 + list[at]) * s.C + c0 + 8 * q : s.w, ok);
        }
        const int jc = r16 / 8;
        for (int i = tid; i < kT * kOuterRows * jc; i += kThreads) {
          const int em = i / jc, j = i - em * jc;
          const int e = em / kOuterRows, m = em - e * kOuterRows;
          const int at = it * kOuterRows + m;
          const bool ok = at < total && 8 * j < p.r;
          cp_async16(sv + (em * v_stride + j) * 16, ok ? s.v + (e * p.M + row0 + list[at]) * p.r + 8 * j : s.v, ok);
        }
      }
      cp_commit();
    };
    float acc[kJ16][2][4];
#pragma unroll
    for (int j = 0; j < kJ16; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[j][h][e] = 0.f;
    for (int it = 0; it < kStages - 1; ++it) load(it);
    for (int it = 0; it < iters; ++it) {
      cp_wait<kStages - 2>();
      __syncthreads();
      load(it + kStages - 1);
      const uint32_t sw = base + (it % kStages) * stage_bytes, sv = sw + kWBytes;
#pragma unroll
      for (int ks = 0; ks < kOuterRows / 16; ++ks) {
        uint32_t fb[4];   // w: rows along the contraction; tiles of columns 16 * warp, + 8
        ldsm4<true>(fb, sw + ((ks * 16 + (lane & 15)) * kWStride + 2 * warp + (lane >> 4)) * 16);
#pragma unroll
        for (int j = 0; j < kJ16; ++j)
          if (j < j16) {
#pragma unroll
            for (int e = kT - 1; e >= 0; --e) {
              uint32_t fa[4];   // v^T: 16 of the rank x 16 rows
              ldsm4<true>(fa, sv + ((e * kOuterRows + ks * 16 + (lane & 7) + ((lane >> 4) << 3)) * v_stride + 2 * j + ((lane >> 3) & 1)) * 16);
              mma16816(acc[j][0], fa, fb[0], fb[1]);
              mma16816(acc[j][1], fa, fb[2], fb[3]);
            }
          }
      }
    }
    cp_wait<0>();
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
    __syncthreads();
  }
}

// ---------------------------------------------------------------- reduce
// dA[a][j][k] and dB[a][c][j] = the ranges' sums in order; an adapter without rows gets zeros.
// One block per 32 x 32 tile of [r][C] of one adapter; dB is written transposed.
struct ReduceSide {
  const float* part;
  void* out;
  int64_t C;
  int64_t tiles;              // blocks of this side
  int transposed;
};
struct ReduceParams {
  ReduceSide side[2];
  const int* present;
  int n, r, ranges;
};

template <bool kF32>
__device__ __forceinline__ void put(void* out, int64_t at, float v) {
  if constexpr (kF32) static_cast<float*>(out)[at] = v;
  else static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(v);
}

template <bool kF32>
__global__ void __launch_bounds__(kThreads) rfq_lora_reduce_kernel(const ReduceParams p) {
  __shared__ float tile[32][33];
  griddep_launch_dependents();
  griddep_wait();
  int64_t b = blockIdx.x;
  const int which = b >= p.side[0].tiles;
  if (which) b -= p.side[0].tiles;
  const ReduceSide s = which ? p.side[1] : p.side[0];
  const int64_t ct = ceil_div(s.C, 32);
  const int jt = (p.r + 31) / 32;
  const int a = static_cast<int>(b / (ct * jt));
  const int64_t rest = b - a * ct * jt;
  const int j0 = static_cast<int>(rest / ct) * 32;
  const int64_t c0 = (rest % ct) * 32;
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  for (int y = ty; y < 32; y += 8) {
    float v = 0.f;
    const int j = j0 + y;
    const int64_t c = c0 + tx;
    if (j < p.r && c < s.C)
      for (int g = 0; g < p.ranges; ++g)
        if (p.present[static_cast<int64_t>(g) * p.n + a]) v += s.part[((static_cast<int64_t>(g) * p.n + a) * p.r + j) * s.C + c];
    if (s.transposed) tile[y][tx] = v;
    else if (j < p.r && c < s.C) put<kF32>(s.out, (static_cast<int64_t>(a) * p.r + j) * s.C + c, v);
  }
  if (s.transposed) {
    __syncthreads();
    for (int y = ty; y < 32; y += 8) {
      const int64_t c = c0 + y;
      const int j = j0 + tx;
      if (j < p.r && c < s.C) put<kF32>(s.out, (static_cast<int64_t>(a) * s.C + c) * p.r + j, tile[tx][y]);
    }
  }
}

// ---------------------------------------------------------------- host
constexpr int kPlanSms = 148;   // the cut does not depend on the device that runs it

template <class Kernel, class Params>
cudaError_t launch(Kernel kernel, const Params& p, dim3 grid, size_t smem, cudaStream_t stream) {
  if (smem > 24 * 1024) {   // with the static part (at most 21 KiB) it may pass the default limit of 48 KiB
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
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

// Rows of one group: 16 where an adapter has few rows of a batch, else 64.
int group_size(int64_t M, int64_t n) { return M <= 32 * n || M <= 64 ? 16 : 64; }

// Splits of the shrink product's contraction: enough CTAs for four per SM, at least two stages each.
int shrink_splits(int64_t M, int64_t C, int64_t n, int64_t* c_split, int* zs) {
  const int rows = group_size(M, n), bk = rows == 16 ? 128 : 64;
  const int64_t chunks = ceil_div(M, kChunk);
  // CTAs per chunk: as many as it can have groups, while the chunks alone do not fill the device.
  int64_t z = ceil_div(M < kChunk ? M : kChunk, rows == 16 ? 1 : rows);
  while (z > 1 && chunks * z > 2 * kPlanSms) z = (z + 1) / 2;
  const int64_t most = ceil_div(C, 2 * bk);
  int64_t s = ceil_div(4 * kPlanSms, chunks * (z < 16 ? z : 16));
  if (s > most) s = most;
  if (s > 32) s = 32;
  if (s < 1) s = 1;
  *c_split = ceil_div(ceil_div(C, s), bk) * bk;
  *zs = static_cast<int>(z);
  return static_cast<int>(ceil_div(C, *c_split));
}

template <int kRows, bool kTrans>
cudaError_t shrink_rank(const ShrinkParams& p, dim3 grid, cudaStream_t stream) {
  using T = ShrinkTile<kRows>;
  size_t smem = static_cast<size_t>(kStages) * (T::kXBytes + shrink_p_bytes<kRows, kTrans>(p.r));
  const size_t red = static_cast<size_t>(T::kWk) * kRows * p.r * 4;
  if (red > smem) smem = red;
  if (p.r <= 16) return launch(rfq_lora_shrink_kernel<kRows, kTrans, 2>, p, grid, smem, stream);
  if (p.r <= 32) return launch(rfq_lora_shrink_kernel<kRows, kTrans, 4>, p, grid, smem, stream);
  if (p.r <= 64) return launch(rfq_lora_shrink_kernel<kRows, kTrans, 8>, p, grid, smem, stream);
  return launch(rfq_lora_shrink_kernel<kRows, kTrans, 16>, p, grid, smem, stream);
}

template <bool kTrans>
cudaError_t shrink(const void* src, const void* w, const int* ids, float* part, int64_t M, int64_t C, int64_t n, int64_t r,
                   int* splits, cudaStream_t stream) {
  ShrinkParams p = {};
  p.src = static_cast<const __nv_bfloat16*>(src);
  p.p = static_cast<const __nv_bfloat16*>(w);
  p.ids = ids;
  p.part = part;
  p.M = M;
  p.C = C;
  p.n = static_cast<int>(n);
  p.r = static_cast<int>(r);
  *splits = shrink_splits(M, C, n, &p.c_split, &p.zs);
  const dim3 grid(static_cast<unsigned>(ceil_div(M, kChunk) * p.zs), static_cast<unsigned>(*splits));
  return group_size(M, n) == 16 ? shrink_rank<16, kTrans>(p, grid, stream) : shrink_rank<64, kTrans>(p, grid, stream);
}

template <int kRows, bool kTrans>
cudaError_t expand_rows(const ExpandParams& p, bool f32, dim3 grid, cudaStream_t stream) {
  const size_t q = expand_q_bytes<kTrans>(p.r);
  return f32 ? launch(rfq_lora_expand_kernel<kRows, kTrans, true>, p, grid, q + expand_s_bytes<kRows, 3>(p.r), stream)
             : launch(rfq_lora_expand_kernel<kRows, kTrans, false>, p, grid, q + expand_s_bytes<kRows, 1>(p.r), stream);
}

template <bool kTrans>
cudaError_t expand(const float* part, int splits, const float* scale, const void* w, const int* ids, const void* base, void* out,
                   bool f32, float* hidden, int64_t M, int64_t C, int64_t n, int64_t r, cudaStream_t stream) {
  ExpandParams p = {};
  p.part = part;
  p.scale = scale;
  p.q = static_cast<const __nv_bfloat16*>(w);
  p.ids = ids;
  p.base = base;
  p.out = out;
  p.hidden = hidden;
  p.M = M;
  p.C = C;
  p.n = static_cast<int>(n);
  p.r = static_cast<int>(r);
  p.splits = splits;
  const int rows = group_size(M, n);
  const int64_t chunks = ceil_div(M, kChunk), tiles = ceil_div(C, kExpandCols);
  int64_t z = ceil_div(M < kChunk ? M : kChunk, rows == 16 ? 1 : rows);
  while (z > 1 && chunks * z * tiles > 4 * kPlanSms) z = (z + 1) / 2;
  p.zs = static_cast<int>(z);
  const dim3 grid(static_cast<unsigned>(chunks * z), static_cast<unsigned>(tiles));
  return rows == 16 ? expand_rows<16, kTrans>(p, f32, grid, stream) : expand_rows<64, kTrans>(p, f32, grid, stream);
}

template <int kT>
cudaError_t outer_rank(const OuterParams& p, dim3 grid, cudaStream_t stream) {
  const size_t smem = static_cast<size_t>(kStages) * outer_stage_bytes<kT>(p.r);
  if (p.r <= 16) return launch(rfq_lora_outer_kernel<1, kT>, p, grid, smem, stream);
  if (p.r <= 32) return launch(rfq_lora_outer_kernel<2, kT>, p, grid, smem, stream);
  if (p.r <= 64) return launch(rfq_lora_outer_kernel<4, kT>, p, grid, smem, stream);
  return launch(rfq_lora_outer_kernel<8, kT>, p, grid, smem, stream);
}

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

// Rows of one range of the outer products: about four CTAs per SM over all column tiles.
int outer_range(int64_t M, int64_t tiles) {
  const int64_t want = ceil_div(4 * kPlanSms, tiles);
  int64_t rows = ceil_div(ceil_div(M, want), kOuterRows) * kOuterRows;
  if (rows < 256) rows = 256;
  if (rows > kMaxRange) rows = kMaxRange;
  return static_cast<int>(rows);
}

struct BackwardPlan {
  size_t part, ds, s, part_a, part_b, present, bytes;
  int range, ranges;
};
// fp32 outputs take three terms, bf16 ones two; the workspace is sized for three.
BackwardPlan plan_backward(int64_t M, int64_t K, int64_t N, int64_t r, int64_t n) {
  BackwardPlan b;
  int64_t cs;
  int z;
  const int splits = shrink_splits(M, N, n, &cs, &z);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += align256(bytes);
    return o;
  };
  b.range = outer_range(M, ceil_div(K, kOuterCols) + ceil_div(N, kOuterCols));
  b.ranges = static_cast<int>(ceil_div(M, b.range));
  b.part = take(static_cast<size_t>(splits) * M * r * 4);
  b.ds = take(static_cast<size_t>(3) * M * r * 2);
  b.s = take(static_cast<size_t>(3) * M * r * 2);
  b.part_a = take(static_cast<size_t>(b.ranges) * n * r * K * 4);
  b.part_b = take(static_cast<size_t>(b.ranges) * n * r * N * 4);
  b.present = take(static_cast<size_t>(b.ranges) * n * 4);
  b.bytes = at;
  return b;
}

}  // namespace

size_t lora_forward_workspace(int64_t M, int64_t K, int64_t r, int64_t n) {
  int64_t cs;
  int z;
  return align256(static_cast<size_t>(shrink_splits(M, K, n, &cs, &z)) * M * r * 4);
}

size_t lora_backward_workspace(int64_t M, int64_t K, int64_t N, int64_t r, int64_t n) {
  return plan_backward(M, K, N, r, n).bytes;
}

cudaError_t launch_lora_forward(const void* x, const void* a, const void* b, const float* scale, const int* ids, const void* base,
                                void* y, bool y_bf16, float* hidden, int64_t M, int64_t K, int64_t N, int64_t r, int64_t n,
                                void* ws, cudaStream_t stream) {
  float* part = static_cast<float*>(ws);
  int splits = 1;
  cudaError_t e = shrink<false>(x, a, ids, part, M, K, n, r, &splits, stream);
  if (e != cudaSuccess) return e;
  return expand<false>(part, splits, scale, b, ids, base, y, !y_bf16, hidden, M, N, n, r, stream);
}

cudaError_t launch_lora_backward(const void* x, const void* a, const void* b, const float* scale, const int* ids, const void* dy,
                                 const float* hidden, const void* dx_base, void* dx, bool dx_bf16, void* da, void* db,
                                 bool grad_bf16, int64_t M, int64_t K, int64_t N, int64_t r, int64_t n, void* ws,
                                 cudaStream_t stream) {
  const BackwardPlan pl = plan_backward(M, K, N, r, n);
  uint8_t* base = static_cast<uint8_t*>(ws);
  float* part = reinterpret_cast<float*>(base + pl.part);
  __nv_bfloat16* ds = reinterpret_cast<__nv_bfloat16*>(base + pl.ds);
  __nv_bfloat16* s = reinterpret_cast<__nv_bfloat16*>(base + pl.s);
  int splits = 1;
  cudaError_t e = cudaSuccess;
  if (dx != nullptr || da != nullptr) {
    e = shrink<true>(dy, b, ids, part, M, N, n, r, &splits, stream);
    if (e != cudaSuccess) return e;
  }
  if (dx != nullptr) {
    e = expand<true>(part, splits, scale, a, ids, dx_base, dx, !dx_bf16, nullptr, M, K, n, r, stream);
    if (e != cudaSuccess) return e;
  }
  if (da == nullptr && db == nullptr) return e;
  {
    const int64_t blocks = ceil_div(M * r, kThreads);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks < 8 * kPlanSms ? blocks : 8 * kPlanSms));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    __nv_bfloat16* ds_out = da != nullptr ? ds : nullptr;
    __nv_bfloat16* s_out = db != nullptr ? s : nullptr;
    const float* cpart = part;
    e = grad_bf16 ? cudaLaunchKernelEx(&cfg, rfq_lora_split_kernel<2>, cpart, scale, ids, static_cast<int>(n), M, static_cast<int>(r),
                                       splits, ds_out, hidden, s_out)
                  : cudaLaunchKernelEx(&cfg, rfq_lora_split_kernel<3>, cpart, scale, ids, static_cast<int>(n), M, static_cast<int>(r),
                                       splits, ds_out, hidden, s_out);
    if (e != cudaSuccess) return e;
  }
  OuterParams o = {};
  o.side[0].v = ds;
  o.side[0].w = static_cast<const __nv_bfloat16*>(x);
  o.side[0].part = reinterpret_cast<float*>(base + pl.part_a);
  o.side[0].C = K;
  o.side[0].tiles = da != nullptr ? static_cast<int>(ceil_div(K, kOuterCols)) : 0;
  o.side[1].v = s;
  o.side[1].w = static_cast<const __nv_bfloat16*>(dy);
  o.side[1].part = reinterpret_cast<float*>(base + pl.part_b);
  o.side[1].C = N;
  o.side[1].tiles = db != nullptr ? static_cast<int>(ceil_div(N, kOuterCols)) : 0;
  o.ids = ids;
  o.present = reinterpret_cast<int*>(base + pl.present);
  o.M = M;
  o.n = static_cast<int>(n);
  o.r = static_cast<int>(r);
  o.range = pl.range;
  const dim3 grid(static_cast<unsigned>(o.side[0].tiles + o.side[1].tiles), static_cast<unsigned>(pl.ranges));
  e = grad_bf16 ? outer_rank<2>(o, grid, stream) : outer_rank<3>(o, grid, stream);
  if (e != cudaSuccess) return e;
  ReduceParams q = {};
  const int64_t jt = ceil_div(r, 32);
  q.side[0] = {o.side[0].part, da, K, da != nullptr ? n * jt * ceil_div(K, 32) : 0, 0};
  q.side[1] = {o.side[1].part, db, N, db != nullptr ? n * jt * ceil_div(N, 32) : 0, 1};
  q.present = o.present;
  q.n = o.n;
  q.r = o.r;
  q.ranges = pl.ranges;
  const dim3 rgrid(static_cast<unsigned>(q.side[0].tiles + q.side[1].tiles));
  return grad_bf16 ? launch(rfq_lora_reduce_kernel<false>, q, rgrid, 0, stream) : launch(rfq_lora_reduce_kernel<true>, q, rgrid, 0, stream);
}

}  // namespace rfq
