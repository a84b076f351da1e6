// rfq_clip.cu -- global norm of a list of gradients, and the list scaled to a largest norm.
//
//     norm = sqrt(sum over all elements of all tensors of x^2)
//     c = min(1, max_norm / (norm + 1e-6)),   out = c x
//
// Bound by memory: the list is read once for the norm and once more, written once, for the
// scaling (which cannot start before the norm is known).  The tensors' addresses travel in
// the kernels' parameters (a table of up to kTable tensors a launch), so nothing is copied
// to the device and a captured graph keeps them.  Every CTA walks over pieces of 16 KiB,
// all tensors' pieces numbered through, and leaves one partial sum; the scaling
// kernel's CTAs each add the partial sums in the same order.  The scaling walks the pieces
// backwards: the end of the list, read last, is what L2 still holds.
//
// Sums: the squares of a thread's elements of one piece (32 of bf16, 16 of fp32) in fp32, these sums in fp64.
// Where the fp32 sum leaves [1e-30, 1e37] (values near 1e19 or below 1e-15) the piece is
// added again in fp64, so the norm neither overflows nor underflows before its own value does.
//
// 40 tensors of 1.87 GB of bf16 in all: 0.93 to 0.97 ms for the three passes (5.6 GB), 5.75 to 6.0 TB/s by the card; a shorter
// list stays in L2 between the norm and the scaling (37 tensors of 90 MB, odd sizes and both types: 51 us).
// Whole pieces go without a check at their vectors: with one at each, the same list took 1.22 ms.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "rfq_internal.h"
#include "rfq_ptx.cuh"

namespace rfq {
namespace {

constexpr int kThreads = 256;
constexpr int kVecs = 4;                     // 16-byte vectors of a thread in one piece
constexpr int kPieceBytes = kThreads * kVecs * 16;   // 16 KiB
constexpr int kTable = 512;                  // tensors of one launch (14 KiB of parameters)
constexpr int kPlanSms = 148;
constexpr int kGrid = 6 * kPlanSms;

struct Table {
  const void* in[kTable];
  void* out[kTable];
  int64_t numel[kTable];       // negative: fp32, -numel elements; else bf16
  int first[kTable + 1];       // first piece of each tensor
  int count;
};

// Moves `t` to the tensor that holds piece `k` (pieces are visited in one direction).
__device__ __forceinline__ void find(const Table& tab, int k, int& t) {
  while (t + 1 < tab.count && k >= tab.first[t + 1]) ++t;
  while (t > 0 && k < tab.first[t]) --t;
}

// One element type: a 16-byte vector as floats, and single elements.
template <bool kF32>
struct Type {
  static constexpr int kPer = kF32 ? 4 : 8;                  // elements of a vector
  static constexpr int kPiece = kPieceBytes / (kF32 ? 4 : 2);
  __device__ static __forceinline__ void open(const uint4& u, float (&f)[kPer]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (kF32) {
        f[e] = __uint_as_float(w[e]);
      } else {
        f[2 * e] = __uint_as_float(w[e] << 16);
        f[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
      }
    }
  }
  __device__ static __forceinline__ uint4 close(const float (&f)[kPer]) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (kF32) {
        w[e] = __float_as_uint(f[e]);
      } else {
        const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * e], f[2 * e + 1]);
        w[e] = *reinterpret_cast<const uint32_t*>(&b);
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ static __forceinline__ float get(const void* p, int i) {
    if constexpr (kF32) return static_cast<const float*>(p)[i];
    else return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  }
  __device__ static __forceinline__ void put(void* p, int i, float x) {
    if constexpr (kF32) static_cast<float*>(p)[i] = x;
    else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(x);
  }
};

// Sum of the threads' values in a fixed order; the result in every thread.
__device__ double block_sum(double v) {
  __shared__ double part[kThreads / 32];
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) s += part[w];
  return s;
}

// The squares of this thread's share of n elements at `in`.  Vectors as far as the piece is whole and
// on a 16-byte boundary (pieces are multiples of 16 bytes from the tensor's start), else one by one.
template <bool kF32>
__device__ __forceinline__ double sum_piece(const uint8_t* in, int n) {
  using T = Type<kF32>;
  float s = 0.f, top = 0.f;
  auto add = [&](float x) {
    s = fmaf(x, x, s);
    top = fmaxf(top, fabsf(x));
  };
  const uint4* v = reinterpret_cast<const uint4*>(in);
  const int vecs = (reinterpret_cast<uintptr_t>(in) & 15u) == 0 ? n / T::kPer : 0;
  if (vecs == kVecs * kThreads) {
    uint4 u[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) u[i] = v[i * kThreads + threadIdx.x];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      float f[T::kPer];
      T::open(u[i], f);
#pragma unroll
      for (int e = 0; e < T::kPer; ++e) add(f[e]);
    }
  } else {
    for (int i = threadIdx.x; i < vecs; i += kThreads) {
      float f[T::kPer];
      T::open(v[i], f);
#pragma unroll
      for (int e = 0; e < T::kPer; ++e) add(f[e]);
    }
    for (int i = vecs * T::kPer + threadIdx.x; i < n; i += kThreads) add(T::get(in, i));
  }
  if (s >= 1e-30f && s <= 1e37f) return s;
  if (s == s && top == 0.f) return 0.0;
  // Out of fp32's comfortable range (or NaN): the same elements once more.
  double d = 0.0;
  for (int i = threadIdx.x; i < vecs; i += kThreads) {
    float f[T::kPer];
    T::open(v[i], f);
    for (int e = 0; e < T::kPer; ++e) d += static_cast<double>(f[e]) * f[e];
  }
  for (int i = vecs * T::kPer + threadIdx.x; i < n; i += kThreads) {
    const double x = T::get(in, i);
    d += x * x;
  }
  return d;
}

template <bool kF32>
__device__ __forceinline__ void scale_piece(const uint8_t* in, uint8_t* out, int n, float c) {
  using T = Type<kF32>;
  const uint4* v = reinterpret_cast<const uint4*>(in);
  uint4* w = reinterpret_cast<uint4*>(out);
  const int vecs = ((reinterpret_cast<uintptr_t>(in) | reinterpret_cast<uintptr_t>(out)) & 15u) == 0 ? n / T::kPer : 0;
  auto scaled = [&](const uint4& u) {
    float f[T::kPer];
    T::open(u, f);
#pragma unroll
    for (int e = 0; e < T::kPer; ++e) f[e] *= c;
    return T::close(f);
  };
  if (vecs == kVecs * kThreads) {
    uint4 u[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) u[i] = v[i * kThreads + threadIdx.x];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) w[i * kThreads + threadIdx.x] = scaled(u[i]);
  } else {
    for (int i = threadIdx.x; i < vecs; i += kThreads) w[i] = scaled(v[i]);
    for (int i = vecs * T::kPer + threadIdx.x; i < n; i += kThreads) T::put(out, i, T::get(in, i) * c);
  }
}

// Calls f(byte offset, elements, is fp32) for piece k of the list, which lies in tensor t.
template <class F>
__device__ __forceinline__ void with_piece(const Table& tab, int k, int t, F f) {
  const int64_t numel = tab.numel[t];
  const bool f32 = numel < 0;
  const int per = f32 ? Type<true>::kPiece : Type<false>::kPiece;
  const int64_t at = static_cast<int64_t>(k - tab.first[t]);
  const int64_t left = (f32 ? -numel : numel) - at * per;
  f(at * kPieceBytes, static_cast<int>(left < per ? left : per), f32);
}

__global__ void __launch_bounds__(kThreads) rfq_clip_norm_kernel(const __grid_constant__ Table tab, double* partial) {
  griddep_launch_dependents();
  griddep_wait();
  const int pieces = tab.first[tab.count];
  double sum = 0.0;
  int t = 0;
  for (int k = blockIdx.x; k < pieces; k += gridDim.x) {
    find(tab, k, t);
    with_piece(tab, k, t, [&](int64_t at, int n, bool f32) {
      const uint8_t* in = static_cast<const uint8_t*>(tab.in[t]) + at;
      sum += f32 ? sum_piece<true>(in, n) : sum_piece<false>(in, n);
    });
  }
  sum = block_sum(sum);
  if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

__device__ __forceinline__ float join_norm(const double* partial, int parts) {
  double v = 0.0;
  for (int i = threadIdx.x; i < parts; i += kThreads) v += partial[i];
  return static_cast<float>(sqrt(block_sum(v)));
}

__global__ void __launch_bounds__(kThreads) rfq_clip_finish_kernel(const double* partial, int parts, float* norm) {
  griddep_launch_dependents();
  griddep_wait();
  const float n = join_norm(partial, parts);
  if (threadIdx.x == 0) *norm = n;
}

__global__ void __launch_bounds__(kThreads) rfq_clip_scale_kernel(const __grid_constant__ Table tab, const double* partial, int parts,
                                                                  float max_norm, float* norm) {
  griddep_launch_dependents();
  griddep_wait();
  const float n = join_norm(partial, parts);
  if (blockIdx.x == 0 && threadIdx.x == 0) *norm = n;
  float c = max_norm / (n + 1e-6f);
  if (c > 1.f || max_norm == INFINITY) c = 1.f;   // a NaN stays one
  const int pieces = tab.first[tab.count];
  int t = tab.count - 1;
  for (int k = pieces - 1 - static_cast<int>(blockIdx.x); k >= 0; k -= gridDim.x) {
    find(tab, k, t);
    if (c == 1.f && tab.in[t] == tab.out[t]) continue;   // multiplying by one changes nothing
    with_piece(tab, k, t, [&](int64_t at, int n, bool f32) {
      const uint8_t* in = static_cast<const uint8_t*>(tab.in[t]) + at;
      uint8_t* out = static_cast<uint8_t*>(tab.out[t]) + at;
      if (f32) scale_piece<true>(in, out, n, c);
      else scale_piece<false>(in, out, n, c);
    });
  }
}

template <class Kernel, class... Args>
cudaError_t launch(Kernel kernel, int grid, cudaStream_t stream, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // see griddep_wait()
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// Fills one table from the list, from tensor `i` on; returns the tensor to go on with.
int64_t fill(Table& tab, const void* const* in, void* const* out, const int64_t* numels, const rfq_out_t* types, int64_t count,
             int64_t i) {
  tab.count = 0;
  int64_t pieces = 0;
  tab.first[0] = 0;
  for (; i < count && tab.count < kTable; ++i) {
    if (numels[i] == 0) continue;
    const int t = tab.count++;
    tab.in[t] = in[i];
    tab.out[t] = out != nullptr ? out[i] : const_cast<void*>(in[i]);
    tab.numel[t] = types[i] == RFQ_OUT_F32 ? -numels[i] : numels[i];
    const int64_t per = types[i] == RFQ_OUT_F32 ? Type<true>::kPiece : Type<false>::kPiece;
    pieces += (numels[i] + per - 1) / per;
    tab.first[t + 1] = static_cast<int>(pieces);
  }
  return i;
}

int grid_of(const Table& tab) { return tab.first[tab.count] < kGrid ? tab.first[tab.count] : kGrid; }

}  // namespace

size_t clip_workspace(int64_t count) {
  const int64_t tables = (count + kTable - 1) / kTable;
  return static_cast<size_t>(tables > 0 ? tables : 1) * kGrid * sizeof(double);
}

cudaError_t launch_clip(const void* const* in, void* const* out, const int64_t* numels, const rfq_out_t* types, int64_t count,
                        bool scale, float max_norm, float* norm, void* ws, cudaStream_t stream) {
  double* partial = static_cast<double*>(ws);
  Table tab;
  int parts = 0;
  cudaError_t e = cudaSuccess;
  for (int64_t i = 0; i < count && e == cudaSuccess;) {
    i = fill(tab, in, out, numels, types, count, i);
    if (tab.count == 0) break;
    const int grid = grid_of(tab);
    e = launch(rfq_clip_norm_kernel, grid, stream, tab, partial + parts);
    parts += grid;
  }
  if (e != cudaSuccess) return e;
  const double* cpartial = partial;
  if (!scale || parts == 0) return launch(rfq_clip_finish_kernel, 1, stream, cpartial, parts, norm);
  for (int64_t i = 0; i < count && e == cudaSuccess;) {
    i = fill(tab, in, out, numels, types, count, i);
    if (tab.count == 0) break;
    e = launch(rfq_clip_scale_kernel, grid_of(tab), stream, tab, cpartial, parts, max_norm, norm);
  }
  return e;
}

}  // namespace rfq
