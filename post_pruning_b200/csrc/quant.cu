// Tokens and weights in 8 bits, for the integer product of linear_i8.cu.
//
// quant_tokens_kernel: a row x of n activations becomes
//   a = max_k |x_k|,  s = a / 127,  q_k = rint(127 x_k / a)  (ties to even),
// and t = sum_k q_k (the product needs it for the weights' zero points). A
// row of zeros has s = 0 and q = 0. With the gate (GATED), x is
// silu(g) * u = g / (1 + e^-g) * u, formed and kept in fp32: nothing is
// rounded to bf16 in between.
//   For bf16 x the codes are the exact ones. 127 x is exact in fp32. A
// quotient that is no tie cannot round across one: with x = X 2^i and
// a = A 2^j (X and A integers below 256, e = j - i) its distance to a tie is
// |254 X - (2k+1) A 2^e| / (2 A 2^e), at least 1/254/255 of it. And a tie
// Q = k + 1/2 comes out as itself: t = 127 x (1/a), with the reciprocal
// rounded once, is within two units in the last place of Q, so the remainder
// 127 x - t a is a small multiple of a's and t's units and exact in one fused
// multiply-add, and t + remainder (1/a) rounds to Q (the residual step of
// Markstein, IBM J. Res. Dev. 34, 1990). The gated x are no short numbers:
// they take one product with the rounded 127/a.
//   Bound by memory: 2 (gated: 4) bytes read and 1 written per element. A row
// is read once: its threads hold it in registers between the maximum and the
// codes. A warp takes a row up to 1024 elements, a CTA of 128 to 512 threads a
// longer one, small enough that several rows are in flight per SM. A few long
// rows (above 8192, n <= 64: decoding) are split over clusters of eight CTAs, which
// exchange their maxima and sums.
//
// quant_codes_kernel: the integer codes of weights on their rows' grid
// (scale, zero point), less half the levels so that they fit a signed byte.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/sgpt.h"
#include "common.cuh"
#include "kernels.h"
#include "tc_ptx.cuh"

namespace sgpt {

namespace {

// silu(g) * u. The reciprocal instruction is off by at most one unit in the
// last place.
__device__ __forceinline__ float silu_mul(float g, float u) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + expf(-g)));
  return g * r * u;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ __forceinline__ uint32_t pack4(int a, int b, int c, int d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// Largest of the row's v (over the group of NT threads, and the cluster).
// Everything above infinity's bits is NaN's; kSkip above all says that a CTA
// of the cluster has seen an error recorded and does nothing.
constexpr uint32_t kSkip = 0xffffffffu;
template <int NT, int CL>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* red, uint32_t* shared_by_cluster) {
  v = __reduce_max_sync(0xffffffffu, v);
  if constexpr (NT > 32) {
    const int t = threadIdx.x;
    if ((t & 31) == 0) red[t >> 5] = v;
    __syncthreads();
    v = __reduce_max_sync(0xffffffffu, (t & 31) < NT / 32 ? red[t & 31] : 0u);
  }
  if constexpr (CL > 1) {
    if (threadIdx.x == 0) {
      shared_by_cluster[0] = v;
      shared_by_cluster[1] = 0;                    // the codes' sum follows there
    }
    ptx::cluster_sync();
    v = 0;
#pragma unroll
    for (int p = 0; p < CL; ++p) v = max(v, (uint32_t)ptx::ld_cluster(ptx::map_rank(ptx::smem_u32(shared_by_cluster), p)));
  }
  return v;
}

// A row per group of NT threads (CL > 1: per cluster of CL CTAs of NT), at
// most VPT vectors of 8 elements per thread.
template <int NT, int VPT, int CL, bool GATED>
__global__ void __launch_bounds__(NT == 32 ? 256 : NT) quant_tokens_kernel(
    const uint16_t* __restrict__ X, const uint16_t* __restrict__ Uu, long long n, int d, long long ldx, long long ldu,
    int8_t* __restrict__ Xq, float* __restrict__ scale, int32_t* __restrict__ sums, int* info) {
  constexpr int kRows = NT == 32 ? 8 : 1;          // rows per CTA
  __shared__ uint32_t red[2][32], mine[2];
  const int part = CL > 1 ? (int)ptx::cluster_rank() : 0;
  ptx::let_next_start();
  ptx::after_previous();
  const bool skip = cta_info_set(info);
  if (CL == 1 && skip) return;
  const int t = threadIdx.x % NT;
  const long long row = (long long)(blockIdx.x / CL) * kRows + threadIdx.x / NT;
  if (kRows > 1 && row >= n) return;
  const int vecs = d / 8, v0 = part * NT + t, step = NT * CL;
  const uint4* x4 = reinterpret_cast<const uint4*>(X + row * ldx);
  const uint4* u4 = reinterpret_cast<const uint4*>(GATED ? Uu + row * ldu : nullptr);

  uint4 raw[VPT];                  // the row, bf16 (GATED: z holds it in fp32)
  float z[GATED ? VPT * 8 : 1];
  uint32_t top = 0;                // bits of the largest magnitude; NaN and infinity compare above all numbers
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    raw[i] = make_uint4(0, 0, 0, 0);
    if (v0 + i * step < vecs) raw[i] = __ldcs(x4 + v0 + i * step);
  }
  if constexpr (GATED) {
    uint4 rawu[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      rawu[i] = make_uint4(0, 0, 0, 0);
      if (v0 + i * step < vecs) rawu[i] = __ldcs(u4 + v0 + i * step);
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const uint32_t g[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
      const uint32_t u[4] = {rawu[i].x, rawu[i].y, rawu[i].z, rawu[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        z[8 * i + 2 * j] = silu_mul(bf16_lo(g[j]), bf16_lo(u[j]));
        z[8 * i + 2 * j + 1] = silu_mul(bf16_hi(g[j]), bf16_hi(u[j]));
        top = max(top, max(__float_as_uint(z[8 * i + 2 * j]) & 0x7fffffffu,
                           __float_as_uint(z[8 * i + 2 * j + 1]) & 0x7fffffffu));
      }
    }
  } else {
    uint32_t m2 = 0;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) m2 = __vmaxu2(m2, w[j] & 0x7fff7fffu);
    }
    top = max(m2 & 0xffff0000u, m2 << 16);
  }
  top = row_max<NT, CL>(CL > 1 && skip ? kSkip : top, red[0], &mine[0]);
  if (CL > 1 && top == kSkip) {                    // one decision for the cluster
    ptx::cluster_sync();                           // no CTA leaves while its word is read
    return;
  }
  const bool finite = top < 0x7f800000u;
  const float a = __uint_as_float(top);
  // 127 a and 1 / a stay numbers: rows above 2^119 are scaled by 2^-8, rows
  // below 2^-100 by 2^64, exactly (what the first flushes is far below half a code)
  const float pre = a > 0x1p119f ? 0x1p-8f : a < 0x1p-100f ? 0x1p64f : 1.f;
  const float k = 127.f * pre, den = a * pre;
  const bool some = finite && top != 0u;
  const float inv = some ? __frcp_rn(den) : 0.f;
  const float ratio = GATED ? k * inv : 0.f;

  int sum = 0;
  uint2* q2 = reinterpret_cast<uint2*>(Xq + row * d);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    if (v0 + i * step >= vecs) continue;
    uint2 o = make_uint2(0, 0);
    if (some) {
      int c[8];
      if constexpr (GATED) {
#pragma unroll
        for (int j = 0; j < 8; ++j) c[j] = __float2int_rn(z[8 * i + j] * ratio);
      } else {
        const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float u = (j & 1 ? bf16_hi(w[j / 2]) : bf16_lo(w[j / 2])) * k;
          const float q = u * inv;
          c[j] = __float2int_rn(fmaf(fmaf(-q, den, u), inv, q));
        }
      }
      o = make_uint2(pack4(c[0], c[1], c[2], c[3]), pack4(c[4], c[5], c[6], c[7]));
      sum = __dp4a((int)o.x, 0x01010101, sum);
      sum = __dp4a((int)o.y, 0x01010101, sum);
    }
    q2[v0 + i * step] = o;
  }
  sum = __reduce_add_sync(0xffffffffu, sum);
  if constexpr (NT > 32) {
    if ((t & 31) == 0) red[1][t >> 5] = (uint32_t)sum;
    __syncthreads();
    if (t < 32) sum = __reduce_add_sync(0xffffffffu, t < NT / 32 ? (int)red[1][t] : 0);
  }
  if constexpr (CL > 1) {
    // mine[1] of the first CTA was cleared before the maxima were exchanged
    if (t == 0) ptx::add_cluster(ptx::map_rank(ptx::smem_u32(&mine[1]), 0), sum);
    ptx::cluster_sync();
    sum = (int)mine[1];
  }
  if (t == 0 && part == 0) {
    scale[row] = finite ? __fdiv_rn(a, 127.f) : __uint_as_float(0x7fc00000u);
    sums[row] = sum;
    if (!finite) set_info(info, SGPT_INFO_NONFINITE);
  }
}

__global__ void __launch_bounds__(256) quant_codes_kernel(const float* __restrict__ W, long long ldw, int rows, int d,
                                                          const float* __restrict__ grid, float maxq, float half,
                                                          int8_t* __restrict__ codes, int* info) {
  if (cta_info_set(info)) return;
  const long long quads = (long long)rows * (d / 4);
  bool bad = false;
  for (long long q = (long long)blockIdx.x * blockDim.x + threadIdx.x; q < quads;
       q += (long long)gridDim.x * blockDim.x) {
    const long long r = q / (d / 4);
    const int c = (int)(q - r * (d / 4)) * 4;
    const float4 w = ld4(W + r * ldw + c);
    const float scale = grid[2 * r], zero = grid[2 * r + 1];
    const float v[4] = {w.x, w.y, w.z, w.w};
    int o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float x = rintf(__fdiv_rn(v[j], scale)) + zero;
      bad |= !(fabsf(x) < INFINITY);
      o[j] = (int)(fminf(fmaxf(x, 0.f), maxq) - half);
    }
    *reinterpret_cast<uint32_t*>(codes + r * d + c) = pack4(o[0], o[1], o[2], o[3]);
  }
  if (__syncthreads_or(bad) && threadIdx.x == 0) set_info(info, SGPT_INFO_NONFINITE);
}

template <int NT, int VPT, int CL, bool GATED>
cudaError_t launch_as(const uint16_t* X, const uint16_t* U, long long n, int d, long long ldx, long long ldu,
                      int8_t* Xq, float* scale, int32_t* sums, int* info, cudaStream_t st) {
  static_assert(NT == 32 || NT % 32 == 0, "whole warps");
  return launch_after(quant_tokens_kernel<NT, VPT, CL, GATED>, (unsigned)(NT == 32 ? cdivll(n, 8) : n * CL),
                      NT == 32 ? 256 : NT, 0, CL, st, X, U, n, d, ldx, ldu, Xq, scale, sums, info);
}

constexpr int kFewRows = 64;   // rows that do not fill the SMs with a CTA each

template <bool GATED>
cudaError_t launch(const uint16_t* X, const uint16_t* U, long long n, int d, long long ldx, long long ldu, int8_t* Xq,
                   float* scale, int32_t* sums, int* info, cudaStream_t st) {
  const auto as = [&](auto f) { return f(X, U, n, d, ldx, ldu, Xq, scale, sums, info, st); };
  if (d <= 1024) return as(launch_as<32, 4, 1, GATED>);
  if (d <= 4096) return as(launch_as<128, 4, 1, GATED>);
  if (d <= 8192) return as(launch_as<256, 4, 1, GATED>);
  if (n <= kFewRows) return as(launch_as<256, 2, 8, GATED>);
  if (d <= 16384) return as(launch_as<256, 8, 1, GATED>);
  if constexpr (GATED) return as(launch_as<512, 8, 1, GATED>);
  if (d <= 26624) return as(launch_as<256, 13, 1, false>);
  return as(launch_as<256, 16, 1, false>);
}

}  // namespace

cudaError_t launch_quant_tokens(const uint16_t* X, long long n, int d, long long ldx, int8_t* Xq, float* scale,
                                int32_t* sums, int* info, cudaStream_t st) {
  return launch<false>(X, nullptr, n, d, ldx, 0, Xq, scale, sums, info, st);
}

cudaError_t launch_quant_tokens_silu(const uint16_t* G, const uint16_t* U, long long n, int d, long long ldg,
                                     long long ldu, int8_t* Xq, float* scale, int32_t* sums, int* info,
                                     cudaStream_t st) {
  return launch<true>(G, U, n, d, ldg, ldu, Xq, scale, sums, info, st);
}

cudaError_t launch_quant_codes(const float* W, long long ldw, int rows, int d, const float* grid, int bits,
                               int8_t* codes, int* info, cudaStream_t st) {
  const long long quads = (long long)rows * (d / 4);
  const int ctas = (int)std::max<long long>(1, std::min<long long>(cdivll(quads, 256), 16LL * kNumSMs));
  quant_codes_kernel<<<ctas, 256, 0, st>>>(W, ldw, rows, d, grid, (float)((1 << bits) - 1), (float)(1 << (bits - 1)),
                                           codes, info);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace sgpt
