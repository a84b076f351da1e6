// rfq_internal.h -- launchers shared between the kernels' .cu files and the C ABI.
// Arguments are validated by the C ABI (rfq_api.cu) before these are called.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "rfq.h"

namespace rfq {

// Kernel 1: fused quantizer.  qr_codes == nullptr selects plain MXFP4.
// `encode_tiled` is the driver's cuTensorMapEncodeTiled.
cudaError_t launch_quantize(const void* x, int64_t M, int64_t K, void* qx_codes, void* qx_scales, void* qr_codes,
                            void* qr_scales, int num_sms, void* encode_tiled, cudaStream_t stream);

// Kernel 1 as the MXFP8 (E4M3) comparator quantizer: codes one byte per element.
cudaError_t launch_quantize_mxfp8(const void* x, int64_t M, int64_t K, void* codes, void* scales, int num_sms,
                                  void* encode_tiled, cudaStream_t stream);

// Kernel 1t: quantizer of X^T for a row-major X [R][C] (blocks along R).
cudaError_t launch_quantize_t(const void* x, int64_t R, int64_t C, void* qt_codes, void* qt_scales, void* qr_codes,
                              void* qr_scales, int num_sms, void* encode_tiled, cudaStream_t stream);

// Kernel 2: RFQ GEMM (y_transposed: Y written as [N][M]).  qr_codes == nullptr selects the plain MXFP4 GEMM.
// `encode_tiled` is the driver's cuTensorMapEncodeTiled.  `skip_fill` >= 0 makes
// the producer of CTA 0 skip that stage fill (fault injection for the bounded
// waits; -1 in normal use).
cudaError_t launch_gemm(const void* qx_codes, const void* qx_scales, const void* qr_codes, const void* qr_scales,
                        const void* qw_codes, const void* qw_scales, int64_t M, int64_t N, int64_t K, void* y,
                        bool y_bf16, bool y_transposed, int num_sms, void* encode_tiled, int skip_fill,
                        cudaStream_t stream);

// Single-kernel RFQ linear layer for M <= 64 (quantizer inside the GEMM).
cudaError_t launch_linear_fused(const void* x, int64_t M, int64_t K, const void* qw_codes, const void* qw_scales,
                                int64_t N, void* y, bool y_bf16, bool residual, int num_sms, void* encode_tiled,
                                cudaStream_t stream);
void set_fused_split_override(int split);   // 0 = automatic

// The same kernel for pre-quantized operands (M <= 256): Q(X), Q(R) as written by
// the quantizer come in by TMA; the GEMM's M <= 256 path when its tiles are few.
cudaError_t launch_gemm_short(const void* qx_codes, const void* qx_scales, const void* qr_codes,
                              const void* qr_scales, const void* qw_codes, const void* qw_scales, int64_t M,
                              int64_t N, int64_t K, void* y, bool y_bf16, int num_sms, void* encode_tiled,
                              int skip_fill, cudaStream_t stream);
constexpr int64_t kShortGemmMaxM = 256;

// The MXFP8 comparator GEMM: E4M3 codes (one byte per element) with E8M0 scales in
// the same MMA layout, plain (no residual term).
cudaError_t launch_gemm_mxfp8(const void* qx_codes, const void* qx_scales, const void* qw_codes,
                              const void* qw_scales, int64_t M, int64_t N, int64_t K, void* y, bool y_bf16,
                              int num_sms, void* encode_tiled, cudaStream_t stream);

// Tensor-core rate probe: up to `max_clusters` clusters (of 2 CTAs for variants 0
// and 2), no more than can be resident at once, issue `iters` x 8 MMAs of the
// GEMM's shapes on shared-memory-resident operands; variant 0 = kind::mxf4 CTA
// pair (M 256), 1 = kind::mxf4 single CTA (M 128), 2 = kind::mxf8f6f4 CTA pair.
// cycles[cluster] = the issuing thread's clock64 span; *clusters_used = clusters launched.
cudaError_t launch_mma_rate_probe(int variant, int iters, unsigned long long* cycles, int max_clusters,
                                  int* clusters_used, cudaStream_t stream);

// Softmax cross entropy at the output head (rfq_ce.cu).  dh / dw may be nullptr.  `skip_fill` as for launch_gemm, in the
// product that forms the logits.
size_t ce_forward_workspace(int64_t T, int64_t V);
size_t ce_backward_workspace(int64_t T, int64_t D, int64_t V, bool want_dh, bool want_dw);
cudaError_t launch_ce_forward(const void* h, const void* w, const int64_t* labels, int64_t T, int64_t D, int64_t V,
                              int64_t ignore, float* loss, float* lse, void* ws, void* encode_tiled, int skip_fill, cudaStream_t stream);
cudaError_t launch_ce_backward(const void* h, const void* w, const int64_t* labels, const float* lse, const float* dloss,
                               int64_t T, int64_t D, int64_t V, int64_t ignore, void* dh, void* dw, void* ws, void* encode_tiled,
                               int skip_fill, cudaStream_t stream);

// Low-rank adapters beside a projection (rfq_lora.cu).  base, hidden, dx, da, db may be nullptr.
size_t lora_forward_workspace(int64_t M, int64_t K, int64_t N, int64_t r, int64_t n);
size_t lora_backward_workspace(int64_t M, int64_t K, int64_t N, int64_t r, int64_t n);
cudaError_t launch_lora_forward(const void* x, const void* a, const void* b, const float* scale, const int* ids, const void* base,
                                void* y, bool y_bf16, float* hidden, int64_t M, int64_t K, int64_t N, int64_t r, int64_t n,
                                void* ws, int num_sms, void* encode_tiled, cudaStream_t stream);
cudaError_t launch_lora_backward(const void* x, const void* a, const void* b, const float* scale, const int* ids, const void* dy,
                                 const float* hidden, const void* dx_base, void* dx, bool dx_bf16, void* da, void* db,
                                 bool grad_bf16, int64_t M, int64_t K, int64_t N, int64_t r, int64_t n, void* ws, int num_sms,
                                 void* encode_tiled, cudaStream_t stream);
// Their two products over long batches (rfq_lora_wide.cu).  shrink: s [M][r] fp32 (or nullptr) = scale
// (P src) and s as bf16 terms [M][num_terms][r], the pool [n][r][C] or, transposed, [n][C][r].  expand:
// out = base + Q s from the terms, the pool [n][C][r] or, transposed, [n][r][C].
cudaError_t launch_lora_shrink_wide(const void* src, const void* pool, bool trans, const int* ids, const float* scale, float* s,
                                    void* terms, int num_terms, int* counts, int64_t M, int64_t C, int64_t n, int64_t r, int num_sms,
                                    void* encode_tiled, cudaStream_t stream);
cudaError_t launch_lora_expand_wide(const void* terms, int num_terms, const int* counts, const void* pool, bool trans, const int* ids,
                                    const void* base, void* out, bool f32, int64_t M, int64_t C, int64_t n, int64_t r,
                                    int num_sms, void* encode_tiled, cudaStream_t stream);
constexpr int RFQ_LORA_OUTER_RANGE = 4096;   // rows of one range of launch_lora_outer_wide, at most (a multiple of 64)
cudaError_t launch_lora_outer_wide(const void* ds, int ds_ld, const void* x, float* part_a, int64_t K, const void* s, int s_ld,
                                   const void* dy, float* part_b, int64_t N, int terms, const int* ids, int* present, int64_t M,
                                   int64_t n, int64_t r, int range, void* encode_tiled, cudaStream_t stream);

// Global norm of a list of tensors (host arrays) and, where `scale`, the list scaled to it (rfq_clip.cu).
// out == nullptr scales in place.
size_t clip_workspace(int64_t count);
cudaError_t launch_clip(const void* const* in, void* const* out, const int64_t* numels, const rfq_out_t* types, int64_t count,
                        bool scale, float max_norm, float* norm, void* ws, cudaStream_t stream);

// Read and clear the device error words (GEMM, quantizer, fused layer, output head, adapters) of the current device.
cudaError_t read_and_clear_device_error(unsigned int* value);
cudaError_t read_and_clear_quant_error(unsigned int* value);
cudaError_t read_and_clear_fused_error(unsigned int* value);
cudaError_t read_and_clear_ce_error(unsigned int* value);
cudaError_t read_and_clear_lora_error(unsigned int* value);

}  // namespace rfq
