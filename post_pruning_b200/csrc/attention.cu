// Causal attention over packed prompts with grouped heads:
//   o_i = sum_{j <= i} p_ij v_j / sum_{j <= i} p_ij,  p_ij = exp(scale q_i . k_j)
// for every sequence of the packed rows and every query head h, which reads
// key/value head h / (heads / kv_heads). One pass over the keys with the
// running maximum m_i and sum l_i of the softmax (fp32); scores and outputs
// accumulate in fp32 on the tensor cores, the weights p_ij of a key block are
// rounded to bf16 for the second product (relative to the running maximum,
// so to 2^-9 of each weight; the sum l_i takes them unrounded).
//
// A CTA owns two 128-row query tiles: the same rows of two heads that share
// a key/value head, or, where the group of heads is odd, two consecutive
// tiles of one head. Both run over the same K and V blocks of 128 keys, so
// while one tile's four softmax warps exponentiate, the tensor cores work for
// the other tile. Warp 8 loads Q and a ring of K and V blocks by TMA, warp 9
// issues the products: S = Q K^T into 128 TMEM columns per tile, then, once
// the softmax warps have replaced S by the bf16 weights in the same columns,
// O += P V with P read from TMEM, followed by the next S.
//   The running maximum is only raised when a row's maximum has grown by more
// than 2^8 in the exponent's base (weights up to 256 are as exact as weights
// up to 1); then the warp rescales its rows of O in TMEM itself: S of block j
// is complete only after the product of block j - 1.
//
// Masked places never reach a result: scores after the diagonal are replaced
// by -inf whatever they are, and rows of V after the end of the sequence are
// zeroed in shared memory before the product that would read them. Rows
// outside every sequence are neither read for a result nor written.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/sgpt.h"
#include "common.cuh"
#include "kernels.h"
#include "tc_ptx.cuh"

namespace sgpt {

namespace {

using namespace ptx;

constexpr int kT = 128;                         // query rows per tile, keys per block
constexpr int kThreads = 320;                   // 2 x 4 softmax warps, TMA, MMA
constexpr int kBox = kT * 128;                  // 16 KB: 128 rows x 64 bf16
constexpr float kGrow = 8.f;                    // exponent growth that moves the running maximum

__host__ __device__ constexpr int tile_bytes(int D) { return D / 64 * kBox; }
__host__ __device__ constexpr int stages_for(int D) { return D == 128 ? 5 : 8; }
__host__ __device__ constexpr size_t smem_for(int D) {
  return (size_t)(2 + stages_for(D)) * tile_bytes(D) + 1024 + 256;
}
static_assert(smem_for(128) <= 232448, "dynamic shared memory per CTA");

constexpr uint32_t kTmemCols = 512;             // S0, S1 (P over them), O0, O1 at 128 columns each

// D fp32, A and B bf16, M = 128; B K-major (S) or MN-major (O).
__host__ __device__ constexpr uint32_t idesc(int n, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(kT >> 4) << 24);
}

__device__ __forceinline__ void mma_ss(uint32_t acc, uint64_t ad, uint64_t bd, uint32_t id, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(acc),
      "l"(ad), "l"(bd), "r"(id), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t acc, uint32_t a_tmem, uint64_t bd, uint32_t id, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(acc),
      "r"(a_tmem), "l"(bd), "r"(id), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two fp32 in one 64-bit register, for the packed fp32 instructions.
__device__ __forceinline__ uint64_t pair_of(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 pair_to(uint64_t p) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(p));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Largest of 32 scores and a.
__device__ __forceinline__ float max32(const uint32_t (&s)[32], float a) {
  float m[4] = {a, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int i = 0; i < 32; i += 8)
#pragma unroll
    for (int x = 0; x < 4; ++x) m[x] = max3(m[x], __uint_as_float(s[i + 2 * x]), __uint_as_float(s[i + 2 * x + 1]));
  return fmaxf(max3(m[0], m[1], m[2]), m[3]);
}

// Scores of 64 keys after column r of them become -inf.
__device__ __forceinline__ void mask64(uint32_t (&a)[32], uint32_t (&b)[32], int r) {
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    if (i > r) a[i] = 0xff800000u;
    if (i + 32 > r) b[i] = 0xff800000u;
  }
}

struct Shape {
  long long ldo;             // elements between rows of O
  int n_tok, n_seq, heads, group;
  int pair;                  // 1: a CTA's two tiles are two heads of one group; 0: two row tiles of one head
  float c;                   // scale * log2(e)
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1) attention_kernel(
    const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
    const __grid_constant__ CUtensorMap vmap, const int32_t* __restrict__ cu, const Shape sh,
    uint16_t* __restrict__ O, int* info, const long long wait_cycles) {
  constexpr int kTile = tile_bytes(D), kStages = stages_for(D);
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + (2 + kStages) * kTile);
  __shared__ uint32_t tmem_slot;
  __shared__ int failed;
  __shared__ int where[3];                       // first row, length, unit of the sequence
  if (cta_info_set(info)) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int head_units = sh.pair ? sh.heads / 2 : sh.heads;
  const int unit_rows = sh.pair ? kT : 2 * kT;

  if (blockIdx.x == 0) {                         // every offset is checked once
    bool bad = false;
    for (int b = threadIdx.x; b < sh.n_seq; b += kThreads) bad |= cu[b] < 0 || cu[b + 1] < cu[b] || cu[b + 1] > sh.n_tok;
    if (__syncthreads_or(bad) && threadIdx.x == 0) set_info(info, SGPT_INFO_BAD_LENGTHS);
  }
  if (warp == 0) {
    // the sequence that holds this unit of rows; a sequence's offsets are
    // used only if they lie inside the packed rows
    const int unit = blockIdx.x / head_units;
    int before = 0;
    if (lane == 0) where[1] = 0;
    __syncwarp();
    for (int b0 = 0; b0 < sh.n_seq; b0 += 32) {
      const int b = b0 + lane;
      int first = 0, len = 0;
      if (b < sh.n_seq) {
        first = cu[b];
        const int end = cu[b + 1];
        len = first >= 0 && end >= first && end <= sh.n_tok ? end - first : 0;
      }
      const int units = cdiv(len, unit_rows);
      int upto = units;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
      }
      const bool mine = unit >= before + upto - units && unit < before + upto;
      if (mine) {
        where[0] = first;
        where[1] = len;
        where[2] = units - 1 - (unit - (before + upto - units));   // the longest rows of keys first
      }
      if (__any_sync(0xffffffffu, mine)) break;
      before += __shfl_sync(0xffffffffu, upto, 31);
    }
  }
  const uint32_t s0 = smem_u32(smem);
  const uint32_t ring = s0 + 2 * kTile;
  const uint32_t qfull = smem_u32(bars), full0 = qfull + 16, empty0 = full0 + 8 * kStages;
  const uint32_t sfull = empty0 + 8 * kStages, pfull = sfull + 16, ofull = pfull + 32, mdone = ofull + 16;
  if (threadIdx.x == 0) {
    prefetch_map(&qmap);
    prefetch_map(&kmap);
    prefetch_map(&vmap);
    failed = 0;
    for (int h = 0; h < 2; ++h) {
      mbar_init(qfull + 8 * h, 1);
      mbar_init(sfull + 8 * h, 1);
      mbar_init(pfull + 16 * h, 4);             // the weights of the block's first 64 keys
      mbar_init(pfull + 16 * h + 8, 4);         // and of its last 64
      mbar_init(ofull + 8 * h, 1);
    }
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    mbar_init(mdone, 1);
    mbar_init_fence();
  }
  __syncthreads();
  const int first = where[0], len = where[1], unit = where[2];
  if (len == 0) return;                          // a CTA past the last unit
  if (warp == 8) tmem_alloc(smem_u32(&tmem_slot), kTmemCols);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_slot, 0);
  const int hu = blockIdx.x % head_units;

  // tile h: its head, its first row in the sequence, its key blocks
  auto head_of = [&](int h) { return sh.pair ? 2 * hu + h : hu; };
  auto row_of = [&](int h) { return unit * unit_rows + (sh.pair ? 0 : h * kT); };
  auto blocks_of = [&](int h) { return row_of(h) < len ? row_of(h) / kT + 1 : 0; };
  const int nb0 = blocks_of(0), nb1 = blocks_of(1), nb = max(nb0, nb1);

  if (warp == 8) {
    if (lane == 0) {
      const int kvh = head_of(0) / sh.group;
      for (int h = 0; h < 2; ++h) {
        if (!blocks_of(h)) continue;
        mbar_expect(qfull + 8 * h, kTile);
        for (int x = 0; x < D / 64; ++x)
          tma_3d(s0 + h * kTile + x * kBox, &qmap, qfull + 8 * h, 64 * x, head_of(h), first + row_of(h));
      }
      int g = 0;                                 // ring slots used: K0 V0 K1 V1 ...
      for (; g < 2 * nb; ++g) {
        const int s = g % kStages;
        if (g >= kStages && !mbar_wait(empty0 + 8 * s, ((g / kStages) & 1) ^ 1, wait_cycles)) {
          failed = 1;
          break;
        }
        mbar_expect(full0 + 8 * s, kTile);
        for (int x = 0; x < D / 64; ++x)
          tma_3d(ring + s * kTile + x * kBox, (g & 1) ? &vmap : &kmap, full0 + 8 * s, 64 * x, kvh, first + (g >> 1) * kT);
      }
      // the copies in flight land before the CTA ends
      for (int h = 0; h < 2; ++h)
        if (blocks_of(h) && !mbar_wait(qfull + 8 * h, 0, kDrainCycles)) failed = 1;
      for (int x = max(g - kStages, 0); x < g; ++x)
        if (!mbar_wait(full0 + 8 * (x % kStages), (x / kStages) & 1, kDrainCycles)) failed = 1;
    }
  } else if (warp == 9) {
    bool ok = true;
    auto wait = [&](uint32_t bar, uint32_t parity) {      // one decision for the warp
      if (ok && __any_sync(0xffffffffu, !mbar_wait(bar, parity, wait_cycles))) ok = false;
      fence_after();
      return ok;
    };
    auto wait_slot = [&](int g) { return wait(full0 + 8 * (g % kStages), (g / kStages) & 1); };
    const uint64_t q_desc = sw128_desc(s0), k_desc = sw128_desc(ring), v_desc = sw128_desc(ring, kBox);
    auto score = [&](int h, int g) {                       // S_h = Q_h K^T
      if (elect_one()) {
        const uint64_t qd = q_desc + (uint64_t)(h * kTile >> 4), kd = k_desc + (uint64_t)((g % kStages) * kTile >> 4);
        const uint32_t acc = tmem + h * kT;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint64_t off = ((ks >> 2) * kBox + 32 * (ks & 3)) >> 4;
          mma_ss(acc, qd + off, kd + off, idesc(kT, false), ks > 0);
        }
        mma_commit(sfull + 8 * h);
      }
      __syncwarp();
    };
    auto signal = [&](uint32_t bar) {
      if (elect_one()) mma_commit(bar);
      __syncwarp();
    };
    if (wait_slot(0)) {
      for (int h = 0; h < 2; ++h)
        if (blocks_of(h) && wait(qfull + 8 * h, 0)) score(h, 0);
      signal(empty0);
    }
    const int ragged = len % kT;                           // keys of the sequence's last block (0: all)
    for (int j = 0; j < nb && ok; ++j) {
      const int gv = 2 * j + 1, gk = 2 * j + 2;
      if (!wait_slot(gv)) break;
      if (ragged && j == len / kT) {
        // rows of V after the sequence's end: their weights are zero, but
        // zero times a NaN or an infinity is not
        for (int x = 0; x < D / 64; ++x)
          for (int i = ragged * 8 + lane; i < kT * 8; i += 32)
            *reinterpret_cast<uint4*>(smem + 2 * kTile + (gv % kStages) * kTile + x * kBox + 16 * i) =
                make_uint4(0, 0, 0, 0);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
      }
      for (int h = 0; h < 2 && ok; ++h) {
        const int mine = h ? nb1 : nb0;
        if (j >= mine) continue;
        const uint64_t vd = v_desc + (uint64_t)((gv % kStages) * kTile >> 4);
        for (int half = 0; half < 2 && ok; ++half) {
          if (!wait(pfull + 16 * h + 8 * half, j & 1)) break;
          if (elect_one()) {
            const uint32_t acc = tmem + 2 * kT + h * kT, pd = tmem + h * kT + 32 * half;
            const uint64_t vh = vd + (uint64_t)(2048 * 4 * half >> 4);
#pragma unroll
            for (int x = 0; x < 4; ++x)
              mma_ts(acc, pd + 8 * x, vh + (uint64_t)(2048 * x >> 4), idesc(D, true), x > 0 ? 1u : (uint32_t)(j + half > 0));
          }
          __syncwarp();
        }
        if (!ok) break;
        if (j + 1 < mine) {
          if (!wait_slot(gk)) break;
          score(h, gk);
        } else {
          signal(ofull + 8 * h);
        }
      }
      if (!ok) break;
      signal(empty0 + 8 * (gv % kStages));
      if (j + 1 < nb) signal(empty0 + 8 * (gk % kStages));
    }
    if (!ok) failed = 1;
    // never free TMEM under a running MMA
    signal(mdone);
    if (!mbar_wait(mdone, 0, kDrainCycles)) failed = 1;
  } else {
    const int h = warp >> 2, q = warp & 3;
    const int mine = h ? nb1 : nb0;
    const uint32_t lanes = (uint32_t)(q * 32) << 16;
    const uint32_t ts = tmem + lanes + h * kT, to = tmem + lanes + 2 * kT + h * kT;
    const int r = q * 32 + lane, row = row_of(h) + r;      // row in the tile and in the sequence
    float m = -INFINITY;
    uint64_t l2[2] = {0, 0};                               // the row's sum, in four parts
    const uint64_t c2 = pair_of(sh.c, sh.c);
    bool ok = true;
    for (int j = 0; j < mine && ok; ++j) {
      if (__any_sync(0xffffffffu, !mbar_wait(sfull + 8 * h, j & 1, wait_cycles))) {
        ok = false;
        break;
      }
      fence_after();
      const bool diagonal = j == mine - 1;
      uint32_t s[4][32];
      tmem_ld32(ts, s[0]);
      tmem_ld32(ts + 32, s[1]);
      tmem_ld_wait();
      tmem_ld32(ts + 64, s[2]);
      tmem_ld32(ts + 96, s[3]);
      if (diagonal) mask64(s[0], s[1], r);
      float top = max32(s[1], max32(s[0], -INFINITY));
      tmem_ld_wait();
      if (diagonal) mask64(s[2], s[3], r - 64);
      top = max32(s[3], max32(s[2], top));
      const bool grow = j == 0 || (top - m) * sh.c > kGrow;
      if (__any_sync(0xffffffffu, grow)) {
        const float mnew = grow ? top : m;
        if (j > 0) {
          const float alpha = ex2((m - mnew) * sh.c);      // 1 where the maximum stays
          const uint64_t a2 = pair_of(alpha, alpha);
#pragma unroll
          for (int x = 0; x < 2; ++x) l2[x] = fma2(l2[x], a2, 0);
#pragma unroll 1
          for (int i = 0; i < D / 16; ++i) {
            uint32_t o[16];
            tmem_ld16(to + 16 * i, o);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st16(to + 16 * i, o);
          }
        }
        m = mnew;
      }
      const float mc = m * sh.c;
      const uint64_t mc2 = pair_of(-mc, -mc);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t p[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const int i = 64 * half + 2 * e;
          const float2 x = pair_to(
              fma2(pair_of(__uint_as_float(s[i / 32][i % 32]), __uint_as_float(s[i / 32][i % 32 + 1])), c2, mc2));
          const float a = ex2(x.x), b = ex2(x.y);
          l2[e & 1] = add2(l2[e & 1], pair_of(a, b));
          p[e] = pack_bf16(a, b);
        }
        tmem_st32(ts + 32 * half, p);
        tmem_st_wait();
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(pfull + 16 * h + 8 * half);
      }
    }
    const float2 la = pair_to(l2[0]), lb = pair_to(l2[1]);
    const float l = (la.x + la.y) + (lb.x + lb.y);
    if (mine && ok && __any_sync(0xffffffffu, !mbar_wait(ofull + 8 * h, 0, wait_cycles))) ok = false;
    if (!ok) failed = 1;
    if (mine && ok) {
      fence_after();
      const float inv = 1.f / l;
      bool bad = false;
      uint16_t* op = O + (long long)(first + row) * sh.ldo + head_of(h) * D;
#pragma unroll 1
      for (int i = 0; i < D / 32; ++i) {
        uint32_t o[32];
        tmem_ld32(to + 32 * i, o);
        tmem_ld_wait();
        uint32_t v[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float a = __uint_as_float(o[2 * e]) * inv, b = __uint_as_float(o[2 * e + 1]) * inv;
          bad |= !(fabsf(a) < INFINITY) || !(fabsf(b) < INFINITY);
          v[e] = pack_bf16(a, b);
        }
        if (row < len) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            *reinterpret_cast<uint4*>(op + 32 * i + 8 * e) = make_uint4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
        }
      }
      if (bad && row < len) set_info(info, SGPT_INFO_NONFINITE);
    }
  }
  fence_before();
  __syncthreads();
  if (failed && threadIdx.x == 0) set_info(info, SGPT_INFO_TIMEOUT);
  if (warp == 8) tmem_free(tmem, kTmemCols);
}

// bf16 [rows x heads x D], row stride ld elements: boxes of 64 columns of one
// head x 128 rows with the 128-byte swizzle.
bool map_heads(CUtensorMap* m, const uint16_t* p, long long rows, int heads, int D, long long ld) {
  const TmaEncodeFn enc = tma_encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)ld * 2};
  const cuuint32_t box[3] = {64, 1, kT};
  const cuuint32_t es[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(p), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch(const CUtensorMap& qm, const CUtensorMap& km, const CUtensorMap& vm, const int32_t* cu,
                   const Shape& sh, long long ctas, uint16_t* O, int* info, cudaStream_t st) {
  static PerDevice attrs;
  const cudaError_t e = once_per_device(attrs, [] {
    return cudaFuncSetAttribute(attention_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_for(D));
  });
  if (e != cudaSuccess) return e;
  attention_kernel<D><<<(unsigned)ctas, kThreads, smem_for(D), st>>>(qm, km, vm, cu, sh, O, info, wait_limit_cycles());
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace

// CTAs of a launch: the units of rows that n_seq sequences of n_tok rows in
// all can have, for each unit of heads.
long long attention_ctas(long long n_tok, int n_seq, int heads, int kv_heads) {
  const bool pair = heads / kv_heads % 2 == 0;
  const long long units = n_tok / (pair ? kT : 2 * kT) + std::min<long long>(n_seq, n_tok);
  return units * (pair ? heads / 2 : heads);
}

cudaError_t launch_attention(const uint16_t* Q, long long ldq, const uint16_t* K, long long ldk, const uint16_t* V,
                             long long ldv, const int32_t* cu, int n_seq, long long n_tok, int heads, int kv_heads,
                             int D, float scale, uint16_t* O, long long ldo, int* info, cudaStream_t st) {
  CUtensorMap qm, km, vm;
  if (!map_heads(&qm, Q, n_tok, heads, D, ldq) || !map_heads(&km, K, n_tok, kv_heads, D, ldk) ||
      !map_heads(&vm, V, n_tok, kv_heads, D, ldv))
    return cudaErrorInvalidValue;
  Shape sh;
  sh.ldo = ldo;
  sh.n_tok = (int)n_tok;
  sh.n_seq = n_seq;
  sh.heads = heads;
  sh.group = heads / kv_heads;
  sh.pair = sh.group % 2 == 0;
  sh.c = (float)((double)scale * 1.4426950408889634);
  const long long ctas = attention_ctas(n_tok, n_seq, heads, kv_heads);
  return D == 128 ? launch<128>(qm, km, vm, cu, sh, ctas, O, info, st)
                  : launch<64>(qm, km, vm, cu, sh, ctas, O, info, st);
}

}  // namespace sgpt
