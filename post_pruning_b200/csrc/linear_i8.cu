// The integer product of 8-bit tokens and 8-bit weights with a scale per
// token and per output channel:
//   y_tr = s_t scale_r ( sum_k q_tk c_rk - z_r t_t ),   z_r = zero_r - 2^(b-1),
// q, s, t from quant_tokens (t_t = sum_k q_tk), c the codes and (scale, zero)
// the grid of the joint sparse and quantized sweep. The bracket is an exact
// int32: |q| <= 127, |c|, |z| <= 128 and K <= 32768 bound it by
// 2 * 127 * 128 * 32768 < 2^31. It is then rounded to fp32 once and
// multiplied by scale_r and s_t in fp32 (and, for a bf16 Y, rounded once more).
//
// Orientation: A = codes (M = 128 output channels), B = tokens (N), both
// K-major int8, tcgen05.mma.kind::i8 into int32 accumulators in TMEM. A lane
// of the epilogue holds one output channel, so its scale and zero point are
// registers and a warp writes 32 consecutive channels of a token; and one
// token costs a product of N = 16, not a row tile of 128.
//
// Persistent, one CTA per SM, warp-specialized: warp 0 feeds a ring of
// 128-byte K stages by TMA (128-byte swizzle, out of range reads give zero
// codes), warp 1 issues four MMAs (K = 32) per stage into one of two
// accumulators, warps 2-5 drain the other. Tiles are walked in groups of 16
// tile rows (rows fastest) so that resident CTAs share panels in L2. Every
// wait is bounded as everywhere in this library.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/sgpt.h"
#include "common.cuh"
#include "kernels.h"
#include "tc_ptx.cuh"

namespace sgpt {

namespace {

using namespace ptx;

constexpr int kBM = 128, kBK = 128;             // output channels per tile; codes (bytes) of K per stage
constexpr int kThreads = 192;                   // producer, MMA, 4 epilogue warps
constexpr int kGroupRows = 16;
constexpr int kABytes = kBM * kBK;

__host__ __device__ constexpr int stage_bytes(int bn) { return kABytes + bn * kBK; }
__host__ __device__ constexpr int stages_for(int bn) { return bn > 128 ? 4 : bn > 64 ? 6 : 8; }
__host__ __device__ constexpr size_t smem_for(int bn) {
  return (size_t)stages_for(bn) * stage_bytes(bn) + 1024 + 256 + 2 * 8 * bn;
}
// accumulator columns: two of max(bn, 16), allocated as a power of two >= 32
__host__ __device__ constexpr uint32_t tmem_cols(int bn) { return bn <= 16 ? 32u : 2u * bn; }

// D int32, A and B signed bytes, both K-major.
__host__ __device__ constexpr uint32_t idesc(int bn) {
  return (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(bn >> 3) << 17) | ((uint32_t)(kBM >> 4) << 24);
}

__device__ __forceinline__ void mma_i8(uint32_t acc, uint64_t ad, uint64_t bd, uint32_t id, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n}\n" ::"r"(acc),
      "l"(ad), "l"(bd), "r"(id), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void store_y(float* y, float v) { *y = v; }
__device__ __forceinline__ void store_y(uint16_t* y, float v) { *y = __bfloat16_as_ushort(__float2bfloat16_rn(v)); }

template <int BN, class T>
__global__ void __launch_bounds__(kThreads, 1) linear_i8_kernel(
    const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap, int rows, int d, int n,
    const float* __restrict__ grid, int half, const float* __restrict__ xs, const int32_t* __restrict__ xsum,
    T* __restrict__ Y, int* info, const long long wait_cycles) {
  constexpr int kStages = stages_for(BN), kStage = stage_bytes(BN);
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kStages * kStage);
  float* tok_scale = reinterpret_cast<float*>(smem + kStages * kStage + 256);       // [2][BN]
  int32_t* tok_sum = reinterpret_cast<int32_t*>(tok_scale + 2 * BN);                // [2][BN]
  __shared__ uint32_t tmem_slot;
  __shared__ int failed;
  if (cta_info_set(info)) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int mt_count = cdiv(rows, kBM), nt_count = cdiv(n, BN), kt_count = cdiv(d, kBK);
  const long long items = (long long)mt_count * nt_count;
  const uint32_t s0 = smem_u32(smem);
  const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * kStages;
  const uint32_t tfull0 = empty0 + 8 * kStages, tempty0 = tfull0 + 16, mdone = tempty0 + 16;
  if (threadIdx.x == 0) {
    prefetch_map(&wmap);
    prefetch_map(&xmap);
    failed = 0;
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull0 + 8 * b, 1);
      mbar_init(tempty0 + 8 * b, 4);
    }
    mbar_init(mdone, 1);
    mbar_init_fence();
  }
  if (warp == 0) tmem_alloc(smem_u32(&tmem_slot), tmem_cols(BN));
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = tmem_slot;

  auto decode = [&](long long w, int& mt, int& nt) {
    const long long per_group = (long long)kGroupRows * nt_count;
    const int g = (int)(w / per_group);
    const int first = g * kGroupRows;
    const int grows = min(kGroupRows, mt_count - first);
    const long long r = w - g * per_group;
    mt = first + (int)(r % grows);
    nt = (int)(r / grows);
  };

  if (warp == 0) {
    if (lane == 0) {
      long long g = 0;
      for (long long w = blockIdx.x; w < items && !failed; w += gridDim.x) {
        int mt, nt;
        decode(w, mt, nt);
        for (int i = 0; i < kt_count; ++i, ++g) {
          const int s = (int)(g % kStages);
          if (g >= kStages && !mbar_wait(empty0 + 8 * s, (uint32_t)((g / kStages) & 1) ^ 1, wait_cycles)) {
            failed = 1;
            break;
          }
          const uint32_t bar = full0 + 8 * s, sa = s0 + s * kStage;
          mbar_expect(bar, kStage);
          tma_2d(sa, &wmap, bar, i * kBK, mt * kBM);
          tma_2d(sa + kABytes, &xmap, bar, i * kBK, nt * BN);
        }
      }
      // the copies in flight land before the CTA ends
      for (long long x = (g > kStages ? g - kStages : 0); x < g; ++x)
        if (!mbar_wait(full0 + 8 * (int)(x % kStages), (uint32_t)(x / kStages) & 1, kDrainCycles)) failed = 1;
    }
  } else if (warp == 1) {
    if (lane == 0) {
      long long g = 0;
      int u = 0;
      for (long long w = blockIdx.x; w < items && !failed; w += gridDim.x, ++u) {
        const int b = u & 1;
        if (u >= 2 && !mbar_wait(tempty0 + 8 * b, ((u >> 1) & 1) ^ 1, wait_cycles)) {
          failed = 1;
          break;
        }
        fence_after();
        for (int i = 0; i < kt_count; ++i, ++g) {
          const int s = (int)(g % kStages);
          if (!mbar_wait(full0 + 8 * s, (uint32_t)(g / kStages) & 1, wait_cycles)) {
            failed = 1;
            break;
          }
          fence_after();
          const uint32_t sa = s0 + s * kStage;
#pragma unroll
          for (int j = 0; j < kBK / 32; ++j)
            mma_i8(tmem + b * BN, sw128_desc(sa + 32 * j), sw128_desc(sa + kABytes + 32 * j), idesc(BN),
                   (i > 0 || j > 0) ? 1u : 0u);
          mma_commit(empty0 + 8 * s);
        }
        if (failed) break;
        mma_commit(tfull0 + 8 * b);
      }
      // never free TMEM under a running MMA
      mma_commit(mdone);
      if (!mbar_wait(mdone, 0, kDrainCycles)) failed = 1;
    }
  } else {
    const int q = warp & 3, et = threadIdx.x - 64;       // TMEM lanes 32 q .. of this warp; epilogue thread
    int u = 0;
    for (long long w = blockIdx.x; w < items; w += gridDim.x, ++u) {
      int mt, nt;
      decode(w, mt, nt);
      const int b = u & 1, n0 = nt * BN, row = mt * kBM + q * 32 + lane;
      for (int e = et; e < BN; e += 128) {
        const bool in = n0 + e < n;
        tok_scale[b * BN + e] = in ? xs[n0 + e] : 0.f;
        tok_sum[b * BN + e] = in ? xsum[n0 + e] : 0;
      }
      float sr = 0.f;
      int zr = 0;
      if (row < rows) {
        const float2 gz = *reinterpret_cast<const float2*>(grid + 2 * (long long)row);
        sr = gz.x;
        zr = (int)gz.y - half;
      }
      asm volatile("bar.sync 1, 128;" ::: "memory");
      int bad = failed;
      if (!bad) bad = !mbar_wait(tfull0 + 8 * b, (u >> 1) & 1, wait_cycles);
      bad = __any_sync(0xffffffffu, bad);      // one decision per warp: the TMEM loads are warp-collective
      if (bad) failed = 1;
      fence_after();
      if (!bad) {
        T* yp = Y + (long long)n0 * rows + row;
#pragma unroll 1
        for (int c = 0; c < BN; c += 16) {
          uint32_t v[16];
          tmem_ld16(tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(b * BN + c), v);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            if (row >= rows || n0 + c + e >= n) continue;
            const int acc = (int)v[e] - zr * tok_sum[b * BN + c + e];
            store_y(yp + (long long)(c + e) * rows, (float)acc * sr * tok_scale[b * BN + c + e]);
          }
        }
      }
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(tempty0 + 8 * b);
      // a warp that gave up still meets the others at the named barrier of the remaining tiles
    }
  }
  fence_before();
  __syncthreads();
  if (failed && threadIdx.x == 0) set_info(info, SGPT_INFO_TIMEOUT);
  if (warp == 0) tmem_free(tmem, tmem_cols(BN));
}

// int8 [rows x d], boxes of 128 bytes x `box` rows with the 128-byte swizzle.
bool map_i8(CUtensorMap* m, const int8_t* p, long long rows, long long d, int box_rows) {
  const TmaEncodeFn enc = tma_encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)d, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)d};
  const cuuint32_t box[2] = {(cuuint32_t)kBK, (cuuint32_t)box_rows};
  const cuuint32_t es[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t*>(p), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Args {
  const int8_t* Xq;
  const float* xs;
  const int32_t* xsum;
  long long n;
  const int8_t* codes;
  const float* grid;
  int half, d, rows;
  void* Y;
  int* info;
  cudaStream_t st;
};

template <int BN, class T>
cudaError_t launch(const Args& a) {
  CUtensorMap wm, xm;
  if (!map_i8(&wm, a.codes, a.rows, a.d, kBM) || !map_i8(&xm, a.Xq, a.n, a.d, BN)) return cudaErrorInvalidValue;
  static PerDevice attrs;
  const cudaError_t e = once_per_device(attrs, [] {
    return cudaFuncSetAttribute(linear_i8_kernel<BN, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_for(BN));
  });
  if (e != cudaSuccess) return e;
  const long long items = (long long)cdiv(a.rows, kBM) * cdivll(a.n, BN);
  const int ctas = (int)std::min<long long>(items, kNumSMs);
  linear_i8_kernel<BN, T><<<ctas, kThreads, smem_for(BN), a.st>>>(wm, xm, a.rows, a.d, (int)a.n, a.grid, a.half, a.xs,
                                                                 a.xsum, static_cast<T*>(a.Y), a.info,
                                                                 wait_limit_cycles());
  count_launches(1);
  return cudaGetLastError();
}

template <class T>
cudaError_t dispatch(const Args& a) {
  if (a.n <= 16) return launch<16, T>(a);
  if (a.n <= 32) return launch<32, T>(a);
  if (a.n <= 64) return launch<64, T>(a);
  if (a.n <= 128) return launch<128, T>(a);
  return launch<256, T>(a);
}

}  // namespace

cudaError_t launch_linear_i8(const int8_t* Xq, const float* xs, const int32_t* xsum, long long n, const int8_t* codes,
                             const float* grid, int bits, int d, int rows, void* Y, bool y_bf16, int* info,
                             cudaStream_t st) {
  const Args a{Xq, xs, xsum, n, codes, grid, 1 << (bits - 1), d, rows, Y, info, st};
  return y_bf16 ? dispatch<uint16_t>(a) : dispatch<float>(a);
}

}  // namespace sgpt
