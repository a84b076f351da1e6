// rfq_clip.cu -- global norm of a list of gradients, and the list scaled to a largest norm.
//
//     norm = sqrt(sum over all elements of all tensors of x^2)
//     c = min(1, max_norm / (norm + 1e-6)),   out = c x
//
// Bound by memory: the list is read once for the norm and once more, written once, for the
// scaling (which cannot start before the norm is known).  The tensors' addresses travel in
// the kernels' parameters (a table of up to kTable tensors a launch), so nothing is copied
// to the device and a captured graph keeps them.  Every CTA walks over pieces of kPiece
// elements, all tensors' pieces numbered through, and leaves one partial sum; the scaling
// kernel's CTAs each add the partial sums in the same order.  The scaling walks the pieces
// backwards: the end of the list, read last, is what L2 still holds.
//
// Sums: the squares of a thread's elements of one piece (32) in fp32, these sums in fp64.
// Where the fp32 sum leaves [1e-30, 1e37] (values near 1e19 or below 1e-15) the piece is
// added again in fp64, so the norm neither overflows nor underflows before its own value does.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "rfq_internal.h"
#include "rfq_ptx.cuh"

namespace rfq {
namespace {

constexpr int kThreads = 256;
constexpr int kPiece = 8192;                 // elements: four 8-element vectors a thread
constexpr int kVecs = kPiece / 8 / kThreads;
constexpr int kTable = 512;                  // tensors of one launch (14 KiB of parameters)
constexpr int kPlanSms = 148;
constexpr int kGrid = 4 * kPlanSms;

struct Table {
  const void* in[kTable];
  void* out[kTable];
  int64_t numel[kTable];       // negative: fp32, -numel elements; else bf16
  int first[kTable + 1];       // first piece of each tensor
  int count;
};

struct Piece {
  int64_t at;                  // first element
  int n;                       // elements
  bool f32;
};

// Moves `t` to the tensor that holds piece `k` (pieces are visited in one direction).
__device__ __forceinline__ Piece find(const Table& tab, int k, int& t) {
  while (t + 1 < tab.count && k >= tab.first[t + 1]) ++t;
  while (t > 0 && k < tab.first[t]) --t;
  Piece p;
  const int64_t numel = tab.numel[t];
  p.f32 = numel < 0;
  p.at = static_cast<int64_t>(k - tab.first[t]) * kPiece;
  const int64_t left = (p.f32 ? -numel : numel) - p.at;
  p.n = static_cast<int>(left < kPiece ? left : kPiece);
  return p;
}

__device__ __forceinline__ float element(const void* base, int64_t i, bool f32) {
  return f32 ? static_cast<const float*>(base)[i] : __bfloat162float(static_cast<const __nv_bfloat16*>(base)[i]);
}

// Eight elements as floats; `base` + i on a 16-byte boundary.
__device__ __forceinline__ void load8(const void* base, int64_t i, bool f32, float (&f)[8]) {
  if (f32) {
    const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(base) + i);
    const float4 b = *reinterpret_cast<const float4*>(static_cast<const float*>(base) + i + 4);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  } else {
    const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + i);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[2 * e] = __uint_as_float(w[e] << 16);
      f[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
  }
}

__device__ __forceinline__ void store8(void* base, int64_t i, bool f32, const float (&f)[8]) {
  if (f32) {
    float* o = static_cast<float*>(base) + i;
    *reinterpret_cast<float4*>(o) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4*>(o + 4) = make_float4(f[4], f[5], f[6], f[7]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * e], f[2 * e + 1]);
      w[e] = *reinterpret_cast<uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(base) + i) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

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

__global__ void __launch_bounds__(kThreads) rfq_clip_norm_kernel(const __grid_constant__ Table tab, double* partial) {
  griddep_launch_dependents();
  griddep_wait();
  const int pieces = tab.first[tab.count];
  double sum = 0.0;
  int t = 0;
  for (int k = blockIdx.x; k < pieces; k += gridDim.x) {
    const Piece p = find(tab, k, t);
    const void* in = tab.in[t];
    float s = 0.f, top = 0.f;
    // Vectors of eight as far as they go (p.at is a multiple of kPiece), the rest one by one.
    const int whole = (reinterpret_cast<uintptr_t>(in) & 15u) == 0 ? p.n & ~7 : 0;
    float f[kVecs][8];
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      const int i = (v * kThreads + threadIdx.x) * 8;
#pragma unroll
      for (int e = 0; e < 8; ++e) f[v][e] = 0.f;
      if (i < whole) load8(in, p.at + i, p.f32, f[v]);
    }
#pragma unroll
    for (int v = 0; v < kVecs; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        s = fmaf(f[v][e], f[v][e], s);
        top = fmaxf(top, fabsf(f[v][e]));
      }
    for (int i = whole + threadIdx.x; i < p.n; i += kThreads) {
      const float x = element(in, p.at + i, p.f32);
      s = fmaf(x, x, s);
      top = fmaxf(top, fabsf(x));
    }
    if (s >= 1e-30f && s <= 1e37f) {
      sum += s;
    } else if (s != s || top > 0.f) {
      // Out of fp32's comfortable range (or NaN): this thread's elements once more.
      for (int i = threadIdx.x * 8; i < whole; i += kThreads * 8)
        for (int e = 0; e < 8; ++e) {
          const double x = element(in, p.at + i + e, p.f32);
          sum += x * x;
        }
      for (int i = whole + threadIdx.x; i < p.n; i += kThreads) {
        const double x = element(in, p.at + i, p.f32);
        sum += x * x;
      }
    }
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
    const Piece p = find(tab, k, t);
    const void* in = tab.in[t];
    void* out = tab.out[t];
    if (c == 1.f && in == out) continue;   // multiplying by one changes nothing
    const int whole = ((reinterpret_cast<uintptr_t>(in) | reinterpret_cast<uintptr_t>(out)) & 15u) == 0 ? p.n & ~7 : 0;
    float f[kVecs][8];
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      const int i = (v * kThreads + threadIdx.x) * 8;
      if (i < whole) load8(in, p.at + i, p.f32, f[v]);
    }
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      const int i = (v * kThreads + threadIdx.x) * 8;
      if (i < whole) {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[v][e] *= c;
        store8(out, p.at + i, p.f32, f[v]);
      }
    }
    for (int i = whole + threadIdx.x; i < p.n; i += kThreads) {
      const float x = element(in, p.at + i, p.f32) * c;
      if (p.f32) static_cast<float*>(out)[p.at + i] = x;
      else static_cast<__nv_bfloat16*>(out)[p.at + i] = __float2bfloat16_rn(x);
    }
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
    pieces += (numels[i] + kPiece - 1) / kPiece;
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
