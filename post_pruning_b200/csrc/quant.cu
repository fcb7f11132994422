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
// codes. A warp takes a row up to 1024 elements, a CTA of 128 to 1024 threads a
// longer one, small enough that several rows are in flight per SM, with no
// more registers than the row needs (16384 gated rows of 5120 with four
// vectors of eight per thread: 92 us; with the three that they need: 75; 2048
// rows of 16416 with 13 vectors: 21.1, with their nine 19.2). Of
// 4096 rows on a warp takes up to 2048 elements too (gated: 1280): it has no
// barrier to wait at (8192 rows of 1248 in a CTA each 10.2 us, in a warp 6.9;
// 2048 rows 3.4 and 3.8). A few long rows (above 8192, n <= 64: decoding) are
// split over clusters of eight CTAs, which exchange their maxima and sums.
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

// A sum with kRound (1.5 * 2^23) is rounded to an integer, ties to even, and
// holds it in its low bits. (The conversion instruction shares the quarter
// rate unit with the gate's exponential and reciprocal.)
constexpr float kRound = 12582912.f;

__device__ __forceinline__ uint32_t pack4(int a, int b, int c, int d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// Eight gated values and the largest magnitude's bits so far.
__device__ __forceinline__ void gated8(const uint4& graw, const uint4& uraw, float* z, uint32_t& top) {
  const uint32_t g[4] = {graw.x, graw.y, graw.z, graw.w};
  const uint32_t u[4] = {uraw.x, uraw.y, uraw.z, uraw.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    z[2 * j] = silu_mul(bf16_lo(g[j]), bf16_lo(u[j]));
    z[2 * j + 1] = silu_mul(bf16_hi(g[j]), bf16_hi(u[j]));
    top = max(top, max(__float_as_uint(z[2 * j]) & 0x7fffffffu, __float_as_uint(z[2 * j + 1]) & 0x7fffffffu));
  }
}

// What a row's codes need of its largest magnitude (given by its bits).
struct RowScale {
  float a, pre, k, den, inv;     // code of x = rint(x k / den), k = 127 pre, den = a pre, inv = 1 / den
  bool finite, some;             // all values are numbers; one is not zero
};
__device__ __forceinline__ RowScale row_scale(uint32_t top) {
  RowScale r;
  r.finite = top < 0x7f800000u;
  r.some = r.finite && top != 0u;
  r.a = __uint_as_float(top);
  // 127 a and 1 / a stay numbers: rows above 2^119 are scaled by 2^-8, rows
  // below 2^-100 by 2^64, exactly (what the first flushes is far below half a code)
  r.pre = r.a > 0x1p119f ? 0x1p-8f : r.a < 0x1p-100f ? 0x1p64f : 1.f;
  r.k = 127.f * r.pre;
  r.den = r.a * r.pre;
  r.inv = r.some ? __frcp_rn(r.den) : 0.f;
  return r;
}

// Eight codes, and their part of the row's sum.
__device__ __forceinline__ uint2 pack8(const int (&c)[8], int& sum) {
  const uint2 o = make_uint2(pack4(c[0], c[1], c[2], c[3]), pack4(c[4], c[5], c[6], c[7]));
  sum = __dp4a((int)o.x, 0x01010101, sum);
  sum = __dp4a((int)o.y, 0x01010101, sum);
  return o;
}
__device__ __forceinline__ uint2 gated_codes(const float* z, const RowScale& r, int& sum) {
  if (!r.some) return make_uint2(0, 0);
  const float ratio = 127.f * r.inv;
  int c[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) c[j] = __float_as_int(fmaf(z[j], ratio, kRound));
  return pack8(c, sum);
}
// The row's gated values as gated_codes() takes them, times pre.
template <int N>
__device__ __forceinline__ void prescale(float (&z)[N], const RowScale& r) {
  if (r.pre != 1.f) {
#pragma unroll
    for (int j = 0; j < N; ++j) z[j] *= r.pre;
  }
}
__device__ __forceinline__ uint2 exact_codes(const uint4& raw, const RowScale& r, int& sum) {
  if (!r.some) return make_uint2(0, 0);
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  int c[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float u = (j & 1 ? bf16_hi(w[j / 2]) : bf16_lo(w[j / 2])) * r.k;
    const float q = u * r.inv;
    c[j] = __float_as_int(fmaf(fmaf(-q, r.den, u), r.inv, q) + kRound);
  }
  return pack8(c, sum);
}

// A row's scale and sum, and the report of values that are not finite.
__device__ __forceinline__ void finish_row(const RowScale& r, int sum, float* scale, int32_t* sums, int* info) {
  *scale = r.finite ? __fdiv_rn(r.a, 127.f) : __uint_as_float(0x7fc00000u);
  *sums = sum;
  if (!r.finite) set_info(info, SGPT_INFO_NONFINITE);
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
    const uint16_t* X, const uint16_t* Uu, long long n, int d, long long ldx, long long ldu, int8_t* __restrict__ Xq,
    float* __restrict__ scale, int32_t* __restrict__ sums, int* info) {
  constexpr int kRows = NT == 32 ? 8 : 1;          // rows per CTA
  __shared__ uint32_t red[2][32], mine[2];
  const int part = CL > 1 ? (int)ptx::cluster_rank() : 0;
  ptx::let_next_start();
  ptx::after_previous();
  const int t = threadIdx.x % NT;
  const long long row = (long long)(blockIdx.x / CL) * kRows + threadIdx.x / NT;
  const int vecs = kRows > 1 && row >= n ? 0 : d / 8, v0 = part * NT + t, step = NT * CL;
  const uint4* x4 = reinterpret_cast<const uint4*>(X + row * ldx);
  const uint4* u4 = reinterpret_cast<const uint4*>(GATED ? Uu + row * ldu : nullptr);

  uint4 raw[VPT];                  // the row, bf16 (GATED: z holds it in fp32)
  float z[GATED ? VPT * 8 : 1];
  uint32_t top = 0;                // bits of the largest magnitude; NaN and infinity compare above all numbers
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    raw[i] = make_uint4(0, 0, 0, 0);
    if (v0 + i * step < vecs) raw[i] = ptx::ld_once(x4 + v0 + i * step);
  }
  uint4 rawu[GATED ? VPT : 1];
  if constexpr (GATED) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      rawu[i] = make_uint4(0, 0, 0, 0);
      if (v0 + i * step < vecs) rawu[i] = ptx::ld_once(u4 + v0 + i * step);
    }
  }
  const bool skip = cta_info_set(info);            // under the row's loads
  if (CL == 1 && (skip || vecs == 0)) return;
  if constexpr (GATED) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) gated8(raw[i], rawu[i], z + 8 * i, top);
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
  const RowScale rs = row_scale(top);
  if constexpr (GATED) prescale(z, rs);
  int sum = 0;
  uint2* q2 = reinterpret_cast<uint2*>(Xq + row * d);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    if (v0 + i * step >= vecs) continue;
    if constexpr (GATED)
      q2[v0 + i * step] = gated_codes(z + 8 * i, rs, sum);
    else
      q2[v0 + i * step] = exact_codes(raw[i], rs, sum);
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
  if (t == 0 && part == 0) finish_row(rs, sum, scale + row, sums + row, info);
}

// The gated rows of 20481 to 28672 elements, when there are many. A row takes 4
// bytes per element in and more arithmetic than a CTA can hide behind its own
// loads: persistent CTAs of 512 keep two rows of G and U in shared memory, one
// copied in (bulk copies) while the other is quantized (8192 x 25600: 181 us,
// 5.8 TB/s; with a row per CTA 273 us). Shorter rows are quicker with several
// CTAs an SM (8192 x 20480: 132 us and 146), longer ones find no room for two.
constexpr int kGatedThreads = 512, kGatedVec = 7;                    // vectors of a thread at most
constexpr int kGatedMax = 28672;                                     // elements: two rows fill the shared memory
static_assert(kGatedMax == kGatedThreads * kGatedVec * 8, "a row in registers");
static_assert(2 * 4 * kGatedMax + 256 <= 232448, "dynamic shared memory per CTA");

template <int VPT>
__global__ void __launch_bounds__(kGatedThreads, 1) quant_gated_kernel(
    const uint16_t* G, const uint16_t* Uu, long long n, int d, long long ldg, long long ldu, int8_t* __restrict__ Xq,
    float* __restrict__ scale, int32_t* __restrict__ sums, int* info, long long wait_cycles) {
  extern __shared__ __align__(128) unsigned char rows_smem[];         // [2][G row, U row]
  __shared__ uint64_t full[2];
  __shared__ uint32_t red[2][32];
  __shared__ int failed;
  ptx::let_next_start();
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const uint32_t row_bytes = 2u * (uint32_t)d;
  const uint32_t s0 = ptx::smem_u32(rows_smem), bar0 = ptx::smem_u32(full);
  if (t == 0) {
    failed = 0;
    ptx::mbar_init(bar0, 1);
    ptx::mbar_init(bar0 + 8, 1);
    ptx::mbar_init_fence();
  }
  ptx::after_previous();
  auto load = [&](long long row, int b) {
    ptx::mbar_expect(bar0 + 8 * b, 2 * row_bytes);
    ptx::bulk_copy(s0 + 2 * b * row_bytes, G + row * ldg, row_bytes, bar0 + 8 * b);
    ptx::bulk_copy(s0 + (2 * b + 1) * row_bytes, Uu + row * ldu, row_bytes, bar0 + 8 * b);
  };
  if (t == 0)
    for (int b = 0; b < 2; ++b) {
      const long long row = blockIdx.x + (long long)b * gridDim.x;
      if (row < n) load(row, b);
    }
  const int vecs = d / 8;
  uint32_t use = 0;
  if (cta_info_set(info)) {                        // under the first copies, which land before the CTA ends
    if (t == 0)
      for (int b = 0; b < 2; ++b)
        if (blockIdx.x + (long long)b * gridDim.x < n) ptx::mbar_wait(bar0 + 8 * b, 0, kDrainCycles);
    return;
  }
  for (long long row = blockIdx.x; row < n; row += gridDim.x, ++use) {
    const int b = use & 1;
    if (!ptx::mbar_wait(bar0 + 8 * b, (use >> 1) & 1, wait_cycles)) failed = 1;
    __syncthreads();
    if (failed) break;
    const uint4* g4 = reinterpret_cast<const uint4*>(rows_smem + 2 * b * row_bytes);
    const uint4* u4 = reinterpret_cast<const uint4*>(rows_smem + (2 * b + 1) * row_bytes);
    float z[VPT * 8];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      uint4 graw = make_uint4(0, 0, 0, 0), uraw = graw;
      if (t + i * kGatedThreads < vecs) {
        graw = g4[t + i * kGatedThreads];
        uraw = u4[t + i * kGatedThreads];
      }
      gated8(graw, uraw, z + 8 * i, top);
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) red[0][warp] = top;
    __syncthreads();                               // and everyone has read the row
    top = __reduce_max_sync(0xffffffffu, lane < kGatedThreads / 32 ? red[0][lane] : 0u);
    const long long later = row + 2LL * gridDim.x;
    if (t == 0 && later < n) {
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      load(later, b);
    }
    const RowScale rs = row_scale(top);
    prescale(z, rs);
    int sum = 0;
    uint2* q2 = reinterpret_cast<uint2*>(Xq + row * d);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      if (t + i * kGatedThreads >= vecs) continue;
      q2[t + i * kGatedThreads] = gated_codes(z + 8 * i, rs, sum);
    }
    sum = __reduce_add_sync(0xffffffffu, sum);
    if (lane == 0) red[1][warp] = (uint32_t)sum;
    __syncthreads();
    if (warp == 0) {
      sum = __reduce_add_sync(0xffffffffu, lane < kGatedThreads / 32 ? (int)red[1][lane] : 0);
      if (lane == 0) finish_row(rs, sum, scale + row, sums + row, info);
    }
  }
  if (failed) {
    // the copies in flight land before the CTA ends
    if (t == 0) {
      for (uint32_t x = use; x < use + 2; ++x)
        if (blockIdx.x + (long long)x * gridDim.x < n) ptx::mbar_wait(bar0 + 8 * (x & 1), (x >> 1) & 1, kDrainCycles);
      set_info(info, SGPT_INFO_TIMEOUT);
    }
    __syncthreads();
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

template <int VPT>
cudaError_t launch_gated(const uint16_t* G, const uint16_t* U, long long n, int d, long long ldg, long long ldu,
                         int8_t* Xq, float* scale, int32_t* sums, int* info, cudaStream_t st) {
  static PerDevice attrs;
  const cudaError_t e = once_per_device(attrs, [] {
    return cudaFuncSetAttribute(quant_gated_kernel<VPT>, cudaFuncAttributeMaxDynamicSharedMemorySize, 2 * 4 * kGatedMax);
  });
  if (e != cudaSuccess) return e;
  return launch_after(quant_gated_kernel<VPT>, (unsigned)std::min<long long>(n, kNumSMs), kGatedThreads,
                      2 * 4 * (size_t)d, 1, st, G, U, n, d, ldg, ldu, Xq, scale, sums, info, wait_limit_cycles());
}

using LaunchFn = cudaError_t (*)(const uint16_t*, const uint16_t*, long long, int, long long, long long, int8_t*, float*,
                                 int32_t*, int*, cudaStream_t);
// The fewest vectors per thread, from VPT on, that hold the row.
template <int NT, int VPT, int MOST, bool GATED>
LaunchFn fit(int vecs) {
  if constexpr (VPT < MOST)
    if (vecs > NT * VPT) return fit<NT, VPT + 1, MOST, GATED>(vecs);
  return launch_as<NT, VPT, 1, GATED>;
}

constexpr int kFewRows = 64;   // rows that do not fill the SMs with a CTA each
constexpr int kManyRows = 4096;              // rows that suit a warp each up to kWarpVecs vectors per lane
template <bool GATED>
constexpr int kWarpVecs = GATED ? 5 : 8;

template <bool GATED>
cudaError_t launch(const uint16_t* X, const uint16_t* U, long long n, int d, long long ldx, long long ldu, int8_t* Xq,
                   float* scale, int32_t* sums, int* info, cudaStream_t st) {
  const auto as = [&](auto f) { return f(X, U, n, d, ldx, ldu, Xq, scale, sums, info, st); };
  const int vecs = d / 8;
  if (vecs <= 32 * 4) return as(fit<32, 1, 4, GATED>(vecs));
  if (n >= kManyRows && vecs <= 32 * kWarpVecs<GATED>) return as(fit<32, 5, kWarpVecs<GATED>, GATED>(vecs));
  if (vecs <= 128 * 4) return as(fit<128, 2, 4, GATED>(vecs));
  if (vecs <= 256 * 4) return as(fit<256, 3, 4, GATED>(vecs));
  if (n <= kFewRows) return as(launch_as<256, 2, 8, GATED>);
  if (vecs <= 256 * 8) return as(fit<256, 5, 8, GATED>(vecs));
  if constexpr (GATED) {
    if (vecs <= 512 * 5) return as(launch_as<512, 5, 1, true>);
    if (vecs <= kGatedThreads * 6) return as(launch_gated<6>);
    if (vecs <= kGatedThreads * kGatedVec) return as(launch_gated<kGatedVec>);
    return as(launch_as<1024, 4, 1, true>);
  }
  return as(fit<256, 9, 16, false>(vecs));
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
