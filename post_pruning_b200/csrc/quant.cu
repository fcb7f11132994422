// Tokens and weights in 8 bits, for the integer product of linear_i8.cu.
//
// quant_tokens_kernel: a row x of n activations becomes
//   a = max_k |x_k|,  s = a / 127,  q_k = rint(127 x_k / a)  (ties to even),
// and t = sum_k q_k (the product needs it for the weights' zero points). A
// row of zeros has s = 0 and q = 0. With the gate (GATED), x is
// silu(g) * u = g / (1 + e^-g) * u, formed and kept in fp32: nothing is
// rounded to bf16 in between.
//   For bf16 x the codes are the exact ones: 127 x and the division's
// operands are exact in fp32, the division rounds correctly, and a quotient
// that is no tie cannot round onto one: with x = X 2^i and a = A 2^j (X and A
// integers below 256, e = j - i) the distance to a tie is
// |254 X - (2k+1) A 2^e| / (2 A 2^e) >= 1 / (2 A 2^e), at least 1/254/255 of
// the quotient, far above the 2^-24 of the rounding.
//   Bound by memory: 2 (gated: 4) bytes read and 1 written per element. A row
// is read once: its group of threads holds it in registers between the
// maximum and the codes (at most 32 elements per thread), a warp per row up
// to 1024 elements, a CTA of 256 up to 8192, of 1024 up to 32768.
//
// quant_codes_kernel: the integer codes of weights on their rows' grid
// (scale, zero point), less half the levels so that they fit a signed byte.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/sgpt.h"
#include "common.cuh"
#include "kernels.h"

namespace sgpt {

namespace {

constexpr int kVec = 4;        // 16-byte vectors (8 elements) of a row per thread, at most

__device__ __forceinline__ float silu_mul(float g, float u) { return g / (1.f + expf(-g)) * u; }

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// The code of x in a row of largest magnitude a = den / pre: k = 127 pre.
__device__ __forceinline__ int code_of(float x, float k, float den) { return __float2int_rn(__fdiv_rn(x * k, den)); }

__device__ __forceinline__ uint32_t pack4(int a, int b, int c, int d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

template <int NT, bool GATED>
__global__ void __launch_bounds__(NT == 32 ? 256 : NT) quant_tokens_kernel(
    const uint16_t* __restrict__ X, const uint16_t* __restrict__ Uu, long long n, int d, long long ldx, long long ldu,
    int8_t* __restrict__ Xq, float* __restrict__ scale, int32_t* __restrict__ sums, int* info) {
  constexpr int kRows = NT == 32 ? 8 : 1;          // rows per CTA
  constexpr int kWarps = NT / 32;
  __shared__ uint32_t red[2][32];
  if (cta_info_set(info)) return;
  const int t = threadIdx.x % NT;
  const long long row = (long long)blockIdx.x * kRows + threadIdx.x / NT;
  if (kRows > 1 && row >= n) return;
  const int vecs = d / 8;
  const uint4* x4 = reinterpret_cast<const uint4*>(X + row * ldx);
  const uint4* u4 = reinterpret_cast<const uint4*>(GATED ? Uu + row * ldu : nullptr);

  uint4 raw[kVec];                 // the row, bf16 (GATED: z holds it in fp32)
  float z[GATED ? kVec * 8 : 1];
  uint32_t top = 0;                // bits of the largest magnitude; NaN and infinity compare above all numbers
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    raw[i] = make_uint4(0, 0, 0, 0);
    if (t + i * NT < vecs) raw[i] = x4[t + i * NT];
  }
  if constexpr (GATED) {
    uint4 rawu[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      rawu[i] = make_uint4(0, 0, 0, 0);
      if (t + i * NT < vecs) rawu[i] = u4[t + i * NT];
    }
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
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
    for (int i = 0; i < kVec; ++i) {
      const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) m2 = __vmaxu2(m2, w[j] & 0x7fff7fffu);
    }
    top = max(m2 & 0xffff0000u, m2 << 16);
  }
  top = __reduce_max_sync(0xffffffffu, top);
  if (kWarps > 1) {
    if ((t & 31) == 0) red[0][t >> 5] = top;
    __syncthreads();
    top = __reduce_max_sync(0xffffffffu, (t & 31) < kWarps ? red[0][t & 31] : 0u);
  }
  const bool finite = top < 0x7f800000u;
  const float a = __uint_as_float(top);
  // 127 a stays a number: rows above 2^119 are scaled by 2^-8, exactly (what
  // that flushes is far below half a code)
  const float pre = a > 0x1p119f ? 0x1p-8f : 1.f;
  const float k = 127.f * pre, den = a * pre;
  const bool some = finite && top != 0u;

  int sum = 0;
  uint2* q2 = reinterpret_cast<uint2*>(Xq + row * d);
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    if (t + i * NT >= vecs) continue;
    uint2 o = make_uint2(0, 0);
    if (some) {
      int c[8];
      if constexpr (GATED) {
#pragma unroll
        for (int j = 0; j < 8; ++j) c[j] = code_of(z[8 * i + j], k, den);
      } else {
        const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          c[2 * j] = code_of(bf16_lo(w[j]), k, den);
          c[2 * j + 1] = code_of(bf16_hi(w[j]), k, den);
        }
      }
      o = make_uint2(pack4(c[0], c[1], c[2], c[3]), pack4(c[4], c[5], c[6], c[7]));
      sum = __dp4a((int)o.x, 0x01010101, sum);
      sum = __dp4a((int)o.y, 0x01010101, sum);
    }
    q2[t + i * NT] = o;
  }
  sum = __reduce_add_sync(0xffffffffu, sum);
  if (kWarps > 1) {
    if ((t & 31) == 0) red[1][t >> 5] = (uint32_t)sum;
    __syncthreads();
    if (t < 32) sum = __reduce_add_sync(0xffffffffu, t < kWarps ? (int)red[1][t] : 0);
  }
  if (t == 0) {
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

template <bool GATED>
cudaError_t launch(const uint16_t* X, const uint16_t* U, long long n, int d, long long ldx, long long ldu, int8_t* Xq,
                   float* scale, int32_t* sums, int* info, cudaStream_t st) {
  if (d <= 32 * 8 * kVec)
    quant_tokens_kernel<32, GATED><<<(unsigned)cdivll(n, 8), 256, 0, st>>>(X, U, n, d, ldx, ldu, Xq, scale, sums, info);
  else if (d <= 256 * 8 * kVec)
    quant_tokens_kernel<256, GATED><<<(unsigned)n, 256, 0, st>>>(X, U, n, d, ldx, ldu, Xq, scale, sums, info);
  else
    quant_tokens_kernel<1024, GATED><<<(unsigned)n, 1024, 0, st>>>(X, U, n, d, ldx, ldu, Xq, scale, sums, info);
  count_launches(1);
  return cudaGetLastError();
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
