// Internal launchers behind the C ABI (host side, one translation unit each).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/sgpt.h"

namespace sgpt {

// factor.cu
size_t factor_ws_bytes(int d);
cudaError_t launch_factor(const float* H, long long n_total, int d, float damp, float* U, void* ws,
                          int* info, cudaStream_t st);

// sweep.cu
size_t prune_ws_bytes(int d_out, int d_in);
cudaError_t launch_prune(float* W, int rows, int d, long long ldw, const float* U,
                         const sgpt_params& p, uint32_t* mask, float* row_loss, void* ws,
                         int* info, cudaStream_t st);
cudaError_t launch_quant_grid(const float* W, long long ldw, int rows, int d, int bits, float* grid,
                              cudaStream_t st);
cudaError_t launch_prune_noalloc(float* W, int rows, int d, long long ldw, const float* U,
                                 const sgpt_params& p, uint32_t* mask, float* row_loss, int* info,
                                 cudaStream_t st);

// pack.cu
cudaError_t launch_pack24(const float* W, long long ldw, int rows, int d, const uint32_t* mask,
                          float* values, uint32_t* meta, int* info, cudaStream_t st);
int packnm_meta_words(int d, int n, int m);
cudaError_t launch_packnm(const float* W, long long ldw, int rows, int d, const uint32_t* mask, int n, int m,
                          float* values, uint32_t* meta, int* info, cudaStream_t st);
size_t recon_ws_bytes(int rows, int d);
cudaError_t launch_recon(const float* W0, const float* W, int rows, int d, long long ldw,
                         const float* H, double* num_den, void* ws, cudaStream_t st);

// driver.cu
cudaError_t launch_to_bf16(const float* W, long long ld, long long rows, int cols, uint16_t* Wb, const int* info,
                           cudaStream_t st);
cudaError_t launch_linear_bf16(const uint16_t* X, const uint16_t* Wb, long long n, int d_in, int d_out, float* Y,
                               int* info, cudaStream_t st);
size_t mlp_block_ws_bytes(int h, int f, long long n);
cudaError_t launch_prune_mlp_block(const sgpt_mlp_block& blk, int h, int f, const uint16_t* X, long long n,
                                   int mode, const sgpt_params& p, uint16_t* X_next, uint16_t* Z, void* ws,
                                   int* info, cudaStream_t st);

size_t attn_block_ws_bytes(int hidden, int heads, int kv_heads, int width, long long n);
cudaError_t launch_prune_attn_block(const sgpt_attn_block& blk, int hidden, int heads, int kv_heads, int width,
                                    float scale, const uint16_t* X, long long n, const int32_t* offsets, int n_seq,
                                    int mode, const sgpt_params& p, uint16_t* X_next, uint16_t* A, void* ws, int* info,
                                    cudaStream_t st);

// consumer.cu
size_t sparse24_meta_tiles_bytes(int rows, int d);
cudaError_t launch_tile_meta(const uint32_t* meta, int rows, int d, uint32_t* tiles, cudaStream_t st);
cudaError_t launch_sparse24_gemm(const uint16_t* values_bf16, const uint32_t* tiles, int rows, int d,
                                 const uint16_t* X, long long n, float* Y, int* info, cudaStream_t st);

// quant.cu
cudaError_t launch_quant_codes(const float* W, long long ldw, int rows, int d, const float* grid, int bits,
                               int8_t* codes, int* info, cudaStream_t st);
cudaError_t launch_quant_tokens(const uint16_t* X, long long n, int d, long long ldx, int8_t* Xq, float* scale,
                                int32_t* sums, int* info, cudaStream_t st);
cudaError_t launch_quant_tokens_silu(const uint16_t* G, const uint16_t* U, long long n, int d, long long ldg,
                                     long long ldu, int8_t* Xq, float* scale, int32_t* sums, int* info,
                                     cudaStream_t st);

// linear_i8.cu
cudaError_t launch_linear_i8(const int8_t* Xq, const float* xs, const int32_t* xsum, long long n, const int8_t* codes,
                             const float* grid, int bits, int d, int rows, void* Y, bool y_bf16, int* info,
                             cudaStream_t st);

// attention.cu
long long attention_ctas(long long n_tok, int n_seq, int heads, int kv_heads);
cudaError_t launch_attention(const uint16_t* Q, long long ldq, const uint16_t* K, long long ldk, const uint16_t* V,
                             long long ldv, const int32_t* cu, int n_seq, long long n_tok, int heads, int kv_heads,
                             int D, float scale, uint16_t* O, long long ldo, int* info, cudaStream_t st);

// hessian_tc.cu
size_t hessian_ws_bytes(int d, long long n);
cudaError_t launch_hessian_tc(float* H, const uint16_t* X, long long n, int d, void* ws, int* info,
                              cudaStream_t st, bool set);

}  // namespace sgpt
