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
// Two kernels, both warp-specialized: warp 0 feeds a ring of 128-byte K
// stages by TMA (128-byte swizzle, out of range reads give zero codes), warp 1
// issues four MMAs (K = 32) per stage, the others are the epilogue: four in the
// split kernel, eight (two for the columns of each TMEM quarter) in the pair
// kernel, where K is short and the epilogue not hidden: 480 -> 15000 with 2000
// tokens took 43 us with four and 36 with eight; 25600 wide either takes the
// same. Every wait is bounded as everywhere in this library.
//   What a tile's epilogue has beside its stores is kept short for the same
// reason: its scales are fetched a tile ahead, its accumulator is handed back
// without a release, tiles are decoded in 32 bits (those 36 us: 29; 608 ->
// 23264 with 8192 tokens 215 us: 165). The stores are then what is left.
//
// linear_i8_pair_kernel, many tiles: persistent CTA pairs (cta_group::2) on
// tiles of 256 channels x 256 (or 128) tokens, each CTA with half of the rows of both
// operands, two accumulators so that one is drained under the other's MMAs.
// A single CTA on 128 x 256 tiles is bound by shared memory (48 KB written and
// 48 KB read per 512 cycles of MMA, above its 128 bytes per cycle): 2,890
// TOP/s on 16384 x 5120 x 25600 as a single launch; the pair needs 32 + 32 KB:
// 3,420, its tensor cores busy for 91 % of the time. In a row the power limit
// leaves the pair 2,870 to 3,100. K in two parts where there are few tiles.
// Tiles are walked in groups of 8 tile rows (rows fastest) so that resident
// pairs share panels in L2.
//
// linear_i8_split_kernel, few tiles: one tile of 128 channels x 16..64 tokens
// per CTA, or per cluster of CTAs that split K and add their int32 accumulators
// through distributed shared memory. Bound by reading the codes, by the
// kernel's start and end where they are few: 25600 -> 5120 with 16 tokens in
// 25 us (5.2 TB/s), 768 -> 768 in 2.9.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/sgpt.h"
#include "common.cuh"
#include "kernels.h"
#include "tc_ptx.cuh"

namespace sgpt {

namespace {

using namespace ptx;

constexpr int kBM = 128, kBK = 128;             // output channels per CTA; codes (bytes) of K per stage
constexpr int kThreads = 192;                   // producer, MMA, 4 epilogue warps
constexpr int kABytes = kBM * kBK;
constexpr long long kGraceCycles = 20000000ll;  // a failed pair's copies land within this (about 10 ms)

// D int32, A and B signed bytes, both K-major.
__host__ __device__ constexpr uint32_t idesc(int m, int n) {
  return (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

template <int PAIR>
__device__ __forceinline__ void mma_i8(uint32_t acc, uint64_t ad, uint64_t bd, uint32_t id, uint32_t accumulate) {
  if constexpr (PAIR)
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n}\n" ::"r"(acc),
        "l"(ad), "l"(bd), "r"(id), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n}\n" ::"r"(acc),
        "l"(ad), "l"(bd), "r"(id), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void store_y(float* y, float v) { *y = v; }
__device__ __forceinline__ void store_y(uint16_t* y, float v) { *y = __bfloat16_as_ushort(__float2bfloat16_rn(v)); }

// What the epilogues need beside the accumulators.
struct Out {
  const float* grid;         // [rows][2] scale, zero point
  const float* xs;           // [n] token scales
  const int32_t* xsum;       // [n] token code sums
  void* Y;                   // [n][rows]
  int rows, n, half;
};

struct Channel {             // one output channel's scale and shifted zero point
  float scale;
  int zero;
};
__device__ __forceinline__ float2 grid_of(const Out& o, int row) {
  return row < o.rows ? *reinterpret_cast<const float2*>(o.grid + 2 * (long long)row) : make_float2(0.f, 0.f);
}
__device__ __forceinline__ Channel channel(const Out& o, float2 g) { return Channel{g.x, (int)g.y - o.half}; }

constexpr int kMaxSplit = 8;                    // parts of K at most

// y of one token and channel from the exact sum of products.
__device__ __forceinline__ float result(int sum, const Channel& ch, float tok_scale, int tok_sum) {
  return (float)(sum - ch.zero * tok_sum) * ch.scale * tok_scale;
}

// Scales and code sums of 16 tokens from shared memory (16-byte aligned).
// Taken before a block's stores: the compiler has to assume that a store to Y
// may reach the arrays, and would load them column by column between the
// stores (105 cycles a column instead of under 20).
__device__ __forceinline__ void load16(const float* tok_scale, const int32_t* tok_sum, float (&ts)[16], int (&tz)[16]) {
#pragma unroll
  for (int i = 0; i < 16; i += 4) {
    const float4 a = *reinterpret_cast<const float4*>(tok_scale + i);
    const int4 b = *reinterpret_cast<const int4*>(tok_sum + i);
    ts[i] = a.x;
    ts[i + 1] = a.y;
    ts[i + 2] = a.z;
    ts[i + 3] = a.w;
    tz[i] = b.x;
    tz[i + 1] = b.y;
    tz[i + 2] = b.z;
    tz[i + 3] = b.w;
  }
}

// One channel (row) of 16 tokens, `left` of which there are.
template <class T>
__device__ __forceinline__ void store16(T* y, long long rows, const uint32_t (&v)[16], const Channel& ch,
                                        const float (&ts)[16], const int (&tz)[16], int left) {
  float r[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) r[e] = result((int)v[e], ch, ts[e], tz[e]);
  if (left >= 16) {
#pragma unroll
    for (int e = 0; e < 16; ++e) store_y(y + e * rows, r[e]);
  } else {
#pragma unroll
    for (int e = 0; e < 16; ++e)
      if (e < left) store_y(y + e * rows, r[e]);
  }
}

// Four consecutive channels of a token.
__device__ __forceinline__ void store4(float* y, const float (&v)[4]) {
  *reinterpret_cast<float4*>(y) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4(uint16_t* y, const float (&v)[4]) {
  ushort4 o;
  store_y(&o.x, v[0]);
  store_y(&o.y, v[1]);
  store_y(&o.z, v[2]);
  store_y(&o.w, v[3]);
  *reinterpret_cast<ushort4*>(y) = o;
}

// The split sums: every CTA of the cluster holds its part of a tile, token by
// token, at `part` ([tokens][128] int32); this one's epilogue warps (w of WARPS)
// add up and write every `split`-th token. first + step * p: the CTA of part
// p. A lane takes four channels: 16 bytes of distributed shared memory at a
// time, 16 loads in flight, are what keeps this short.
template <class T, int WARPS>
__device__ __forceinline__ void add_parts(uint32_t part, int split, int sp, int first, int step, int w, int lane,
                                          int row0, int n0, int cols, const Out& out, const Channel (&ch)[4],
                                          const float* tok_scale, const int32_t* tok_sum) {
  const int rows = out.rows, row = row0 + 4 * lane;
  const bool whole = rows % 4 == 0 && row + 3 < rows;
  T* Y = static_cast<T*>(out.Y) + (long long)n0 * rows + row;
  const int every = WARPS * split;
  for (int c0 = sp + split * w; c0 < cols; c0 += 4 * every) {
    int4 acc[4] = {};
    float ts[4];
    int tz[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = min(c0 + i * every, cols - 1);
      ts[i] = tok_scale[c];
      tz[i] = tok_sum[c];
    }
#pragma unroll 4
    for (int p = 0; p < split; ++p) {
      const uint32_t from = map_rank(part + 16 * lane, first + step * p);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = c0 + i * every;
        if (c >= cols) continue;
        const int4 v = ld_cluster4(from + 4 * kBM * c);
        acc[i].x += v.x;
        acc[i].y += v.y;
        acc[i].z += v.z;
        acc[i].w += v.w;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = c0 + i * every;
      if (c >= cols) continue;
      const int sum[4] = {acc[i].x, acc[i].y, acc[i].z, acc[i].w};
      float v[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) v[x] = result(sum[x], ch[x], ts[i], tz[i]);
      T* y = Y + (long long)c * rows;
      if (whole) {
        store4(y, v);
      } else {
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (row + x < rows) store_y(y + x, v[x]);
      }
    }
  }
}

// ------------------------------------------------------------------ CTA pairs

__host__ __device__ constexpr int pair_stage(int bn) { return kABytes + bn / 2 * kBK; }   // per CTA
__host__ __device__ constexpr int pair_stages(int bn) { return bn > 128 ? 6 : 8; }
__host__ __device__ constexpr size_t pair_smem(int bn) {
  return (size_t)pair_stages(bn) * pair_stage(bn) + 1024 + 256 + 2 * 8 * bn;
}
constexpr int kPairThreads = 320;               // producer, MMA, 8 epilogue warps
constexpr int kGroupRows = 8;                   // 256-channel tile rows walked together

template <int BN, class T>
__global__ void __launch_bounds__(kPairThreads, 1) linear_i8_pair_kernel(const __grid_constant__ CUtensorMap wmap,
                                                                         const __grid_constant__ CUtensorMap xmap, int d,
                                                                         int split, const Out out, int* info,
                                                                         const long long wait_cycles) {
  constexpr int kStages = pair_stages(BN), kStage = pair_stage(BN);
  static_assert(BN * kBM * 4 <= kStages * kStage, "the parts of a split sum fit the ring");
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  // both CTAs lay their shared memory out alike: the pair's barriers and
  // operands are addressed by the same offsets
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kStages * kStage);
  float* tok_scale = reinterpret_cast<float*>(smem + kStages * kStage + 256);       // [2][BN]
  int32_t* tok_sum = reinterpret_cast<int32_t*>(tok_scale + 2 * BN);                // [2][BN]
  __shared__ uint32_t tmem_slot;
  __shared__ int failed;
  let_next_start();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank(), leader = rank & ~1u, half = rank & 1u;   // the pair's first CTA; this one's half
  const int sp = (int)(rank >> 1);                           // this pair's part of K
  const uint16_t both = (uint16_t)(3u << leader);
  const int rows = out.rows, n = out.n;
  const int mt_count = cdiv(rows, 2 * kBM), nt_count = cdiv(n, BN), kt_count = cdiv(d, kBK);
  const int k0 = (int)((long long)kt_count * sp / split), k1 = (int)((long long)kt_count * (sp + 1) / split);
  const uint32_t items = (uint32_t)mt_count * (uint32_t)nt_count;             // below 2^31, as the launch checks
  const uint32_t first_item = blockIdx.x / (2 * split), step = gridDim.x / (2 * split);
  const uint32_t s0 = smem_u32(smem);
  const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * kStages;
  const uint32_t tfull0 = empty0 + 8 * kStages, tempty0 = tfull0 + 16, mdone = tempty0 + 16;
  auto decode = [&](uint32_t w, int& mt, int& nt) {
    const uint32_t per_group = (uint32_t)kGroupRows * (uint32_t)nt_count;
    const uint32_t first = w / per_group * kGroupRows, r = w % per_group;
    const uint32_t grows = min((uint32_t)kGroupRows, (uint32_t)mt_count - first);
    mt = (int)(first + r % grows);
    nt = (int)(r / grows);
  };
  if (threadIdx.x == 0) {
    prefetch_map(&wmap);
    prefetch_map(&xmap);
    failed = 0;
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full0 + 8 * s, 1);              // used in the pair's first CTA
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull0 + 8 * b, 1);
      mbar_init(tempty0 + 8 * b, 16);           // used in the pair's first CTA: eight warps of each
    }
    mbar_init(mdone, 1);
    mbar_init_fence();
  }
  after_previous();
  if (warp == 0) tmem_alloc2(smem_u32(&tmem_slot), 2 * BN);
  fence_before();
  cluster_sync();
  fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_slot, 0);
  // an error recorded by an earlier call: everything runs, nothing is written
  // (the look at *info is under the products)
  const bool write = warp < 2 || !info_set(info);

  if (warp == 0) {
    if (elect_one()) {
      const uint32_t leader_full0 = map_rank(full0, leader);
      long long g = 0;
      for (uint32_t w = first_item; w < items && !failed; w += step) {
        int mt, nt;
        decode(w, mt, nt);
        for (int i = k0; i < k1; ++i, ++g) {
          const int s = (int)(g % kStages);
          if (g >= kStages && !mbar_wait(empty0 + 8 * s, (uint32_t)((g / kStages) & 1) ^ 1, wait_cycles)) {
            failed = 1;
            break;
          }
          const uint32_t bar = leader_full0 + 8 * s, sa = s0 + s * kStage;
          if (half == 0) mbar_expect(full0 + 8 * s, 2 * kStage);      // both CTAs' copies
          tma_2d_pair(sa, &wmap, bar, i * kBK, mt * 2 * kBM + (int)half * kBM);
          tma_2d_pair(sa + kABytes, &xmap, bar, i * kBK, nt * BN + (int)half * (BN / 2));
        }
      }
      // the last stages' releases, which reach into this CTA, arrive before it ends
      for (long long x = (g > kStages ? g - kStages : 0); x < g && !failed; ++x)
        if (!mbar_wait(empty0 + 8 * (int)(x % kStages), (uint32_t)(x / kStages) & 1, wait_cycles)) failed = 1;
    }
  } else if (warp == 1) {
    if (half == 0 && elect_one()) {
      const uint64_t a_desc = sw128_desc(s0), b_desc = sw128_desc(s0 + kABytes);
      long long g = 0;
      int u = 0;
      for (uint32_t w = first_item; w < items && !failed; w += step, ++u) {
        const int b = u & 1;
        if (u >= 2 && !mbar_wait(tempty0 + 8 * b, ((u >> 1) & 1) ^ 1, wait_cycles)) {
          failed = 1;
          break;
        }
        fence_after();
        for (int i = k0; i < k1; ++i, ++g) {
          const int s = (int)(g % kStages);
          if (!mbar_wait(full0 + 8 * s, (uint32_t)(g / kStages) & 1, wait_cycles)) {
            failed = 1;
            break;
          }
          fence_after();
          const uint64_t off = (uint64_t)(s * kStage >> 4);
#pragma unroll
          for (int j = 0; j < kBK / 32; ++j)
            mma_i8<1>(tmem + b * BN, a_desc + off + 2 * j, b_desc + off + 2 * j, idesc(2 * kBM, BN),
                      j > 0 ? 1u : (uint32_t)(i > k0));
          mma_commit2(empty0 + 8 * s, both);
        }
        if (failed) break;
        mma_commit2(tfull0 + 8 * b, both);
      }
      // never free TMEM under a running MMA
      mma_commit2(mdone, (uint16_t)(1u << leader));
      if (!mbar_wait(mdone, 0, kDrainCycles)) failed = 1;
    }
  } else {
    // TMEM lanes 32 q .. of this warp, and its half of the columns; epilogue thread
    const int q = warp & 3, part_of = (warp - 2) >> 2, et = threadIdx.x - 64;
    const uint32_t leader_tempty0 = map_rank(tempty0, leader);
    // A tile's channel and token scales are asked for before the stores of the
    // tile before it (asked for after them, they came 3300 cycles later) and
    // touched after them.
    float2 grid_next = make_float2(0.f, 0.f);
    float scale_next = 0.f;
    int sum_next = 0;
    int mt_next = 0, nt_next = 0;
    auto fetch = [&](uint32_t w) {
      decode(w, mt_next, nt_next);
      grid_next = grid_of(out, mt_next * 2 * kBM + (int)half * kBM + q * 32 + lane);
      const int tok = nt_next * BN + et;
      const bool in = et < BN && tok < n;
      scale_next = in ? out.xs[tok] : 0.f;
      sum_next = in ? out.xsum[tok] : 0;
    };
    if (first_item < items) fetch(first_item);
    int u = 0;
    for (uint32_t w = first_item; w < items; w += step, ++u) {
      const int mt = mt_next, nt = nt_next;
      const int b = u & 1, n0 = nt * BN, row = mt * 2 * kBM + (int)half * kBM + q * 32 + lane;
      const int cols = min(BN, n - n0);
      if (et < BN) {
        tok_scale[b * BN + et] = scale_next;
        tok_sum[b * BN + et] = sum_next;
      }
      const Channel ch = channel(out, grid_next);
      asm volatile("bar.sync 1, 256;" ::: "memory");
      if (w + step < items) fetch(w + step);
      int bad = failed;
      if (!bad) bad = !mbar_wait(tfull0 + 8 * b, (u >> 1) & 1, wait_cycles);
      bad = __any_sync(0xffffffffu, bad);      // one decision per warp: the TMEM loads are warp-collective
      if (bad) failed = 1;
      fence_after();
      if (!bad) {
        T* yp = static_cast<T*>(out.Y) + (long long)n0 * rows + row;
        int32_t* part = reinterpret_cast<int32_t*>(smem) + q * 32 + lane;
        const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(b * BN);
#pragma unroll 1
        for (int c = part_of * (BN / 2); c < min(cols, (part_of + 1) * (BN / 2)); c += 32) {
          uint32_t v[2][16];
          tmem_ld16(acc + c, v[0]);
          tmem_ld16(acc + c + 16, v[1]);
          if (split > 1) {
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) part[(c + e) * kBM] = (int32_t)v[e / 16][e % 16];
          } else {
            float ts[2][16];
            int tz[2][16];
            load16(tok_scale + b * BN + c, tok_sum + b * BN + c, ts[0], tz[0]);
            load16(tok_scale + b * BN + c + 16, tok_sum + b * BN + c + 16, ts[1], tz[1]);
            tmem_ld_wait();
            if (row < rows && write) {
              store16(yp + (long long)c * rows, rows, v[0], ch, ts[0], tz[0], cols - c);
              store16(yp + (long long)(c + 16) * rows, rows, v[1], ch, ts[1], tz[1], cols - c - 16);
            }
          }
        }
      }
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(leader_tempty0 + 8 * b);
      // a warp that gave up still meets the others at the named barrier of the remaining tiles
    }
  }
  if (split > 1) {                              // one tile per cluster
    int mt, nt;
    decode(first_item, mt, nt);
    const int row0 = mt * 2 * kBM + (int)half * kBM;
    Channel ch4[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) ch4[x] = channel(out, grid_of(out, row0 + 4 * lane + x));
    cluster_sync();
    bool all = write;
    for (int p = 0; p < 2 * split; ++p) all = all && ld_cluster(map_rank(smem_u32(&failed), p)) == 0;
    if (warp >= 2 && all)
      add_parts<T, 8>(s0, split, sp, (int)half, 2, warp - 2, lane, row0, nt * BN, min(BN, n - nt * BN), out, ch4,
                      tok_scale, tok_sum);
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  if (failed && threadIdx.x == 0) {
    set_info(info, SGPT_INFO_TIMEOUT);
    // copies of this CTA may still be in flight on a barrier that nothing waits for any more
    const long long t0 = clock64();
    while (clock64() - t0 < kGraceCycles) {
    }
  }
  __syncthreads();
  cluster_sync();                               // the cluster ends together: MMAs, barriers and sums reach into its CTAs
  if (warp == 0) tmem_free2(tmem, 2 * BN);
}

// ---------------------------------------------------- one tile, split over K

// the most that leaves room for two CTAs on an SM
__host__ __device__ constexpr int split_stages(int bn) { return bn <= 16 ? 6 : bn <= 32 ? 5 : 4; }
__host__ __device__ constexpr int split_stage(int bn) { return kABytes + bn * kBK; }
__host__ __device__ constexpr size_t split_smem(int bn) {
  return (size_t)split_stages(bn) * split_stage(bn) + 1024 + 128;
}
constexpr int kSplitPerSM = 2;
static_assert(2 * (split_smem(16) + 2048) <= 233472 && 2 * (split_smem(32) + 2048) <= 233472 &&
                  2 * (split_smem(64) + 2048) <= 233472, "CTAs per SM");

template <int BN, class T>
__global__ void __launch_bounds__(kThreads) linear_i8_split_kernel(const __grid_constant__ CUtensorMap wmap,
                                                                   const __grid_constant__ CUtensorMap xmap, int d,
                                                                   int split, const Out out, int* info,
                                                                   const long long wait_cycles) {
  constexpr int kStages = split_stages(BN), kStage = split_stage(BN);
  constexpr uint32_t kCols = BN < 32 ? 32 : BN;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kStages * kStage);
  __shared__ uint32_t tmem_slot;
  __shared__ int failed;
  __shared__ __align__(16) float tok_scale[BN];
  __shared__ __align__(16) int32_t tok_sum[BN];
  let_next_start();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank();                    // this CTA's part of K
  const int tile = blockIdx.x / split;
  const int rows = out.rows, n = out.n;
  const int nt_count = cdiv(n, BN), kt_count = cdiv(d, kBK);
  const int mt = tile / nt_count, nt = tile % nt_count;      // token tiles fastest: they read the same codes together
  const int k0 = (int)((long long)kt_count * rank / split), k1 = (int)((long long)kt_count * (rank + 1) / split);
  const uint32_t s0 = smem_u32(smem);
  const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * kStages, tfull = empty0 + 8 * kStages, mdone = tfull + 8;
  if (threadIdx.x == 0) {
    prefetch_map(&wmap);
    prefetch_map(&xmap);
    failed = 0;
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    mbar_init(tfull, 1);
    mbar_init(mdone, 1);
    mbar_init_fence();
  }
  after_previous();
  if (warp == 0) tmem_alloc(smem_u32(&tmem_slot), kCols);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = tmem_slot;
  const bool write = warp < 2 || !info_set(info);            // as above

  if (warp == 0) {
    if (elect_one()) {
      int g = 0;
      for (int i = k0; i < k1; ++i, ++g) {
        const int s = g % kStages;
        if (g >= kStages && !mbar_wait(empty0 + 8 * s, ((g / kStages) & 1) ^ 1, wait_cycles)) {
          failed = 1;
          break;
        }
        const uint32_t bar = full0 + 8 * s, sa = s0 + s * kStage;
        mbar_expect(bar, kStage);
        tma_2d(sa, &wmap, bar, i * kBK, mt * kBM);
        tma_2d(sa + kABytes, &xmap, bar, i * kBK, nt * BN);
      }
      // the copies in flight land before the CTA ends
      for (int x = max(g - kStages, 0); x < g; ++x)
        if (!mbar_wait(full0 + 8 * (x % kStages), (x / kStages) & 1, kDrainCycles)) failed = 1;
    }
  } else if (warp == 1) {
    if (elect_one()) {
      const uint64_t a_desc = sw128_desc(s0), b_desc = sw128_desc(s0 + kABytes);
      for (int g = 0; g < k1 - k0; ++g) {
        const int s = g % kStages;
        if (!mbar_wait(full0 + 8 * s, (g / kStages) & 1, wait_cycles)) {
          failed = 1;
          break;
        }
        fence_after();
        const uint64_t off = (uint64_t)(s * kStage >> 4);
#pragma unroll
        for (int j = 0; j < kBK / 32; ++j)
          mma_i8<0>(tmem, a_desc + off + 2 * j, b_desc + off + 2 * j, idesc(kBM, BN), j > 0 ? 1u : (uint32_t)(g > 0));
        mma_commit(empty0 + 8 * s);
      }
      if (!failed) mma_commit(tfull);
      // never free TMEM under a running MMA
      mma_commit(mdone);
      if (!mbar_wait(mdone, 0, kDrainCycles)) failed = 1;
    }
  }
  const int q = warp & 3, r = q * 32 + lane;               // epilogue warps: TMEM lane = channel in the tile
  const int row = mt * kBM + r, n0 = nt * BN, cols = min(BN, n - n0);
  const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16);
  T* Y = static_cast<T*>(out.Y) + (long long)n0 * rows + row;
  Channel ch{0.f, 0}, ch4[4];                              // this lane's channel, or its four of the split sums
  bool ok = true;
  if (warp >= 2) {
    for (int e = threadIdx.x - 64; e < cols; e += 128) {
      tok_scale[e] = out.xs[n0 + e];
      tok_sum[e] = out.xsum[n0 + e];
    }
    ch = channel(out, grid_of(out, row));
#pragma unroll
    for (int x = 0; x < 4; ++x) ch4[x] = channel(out, grid_of(out, mt * kBM + 4 * lane + x));
    asm volatile("bar.sync 1, 128;" ::: "memory");
    if (__any_sync(0xffffffffu, !mbar_wait(tfull, 0, wait_cycles))) {
      failed = 1;
      ok = false;
    }
    fence_after();
  }
  if (split == 1) {
    if (warp >= 2 && ok) {
#pragma unroll 1
      for (int c = 0; c < cols; c += 16) {
        uint32_t v[16];
        float ts[16];
        int tz[16];
        tmem_ld16(lanes + c, v);
        load16(tok_scale + c, tok_sum + c, ts, tz);
        tmem_ld_wait();
        if (row < rows && write) store16(Y + (long long)c * rows, rows, v, ch, ts, tz, cols - c);
      }
    }
  } else {
    // the parts of the sum, token by token, in the ring that the products
    // have left; each CTA of the cluster then adds up and writes its share
    // of the tokens (int32 sums: any order gives the same bits)
    int32_t* part = reinterpret_cast<int32_t*>(smem);      // [BN][128]
    if (warp >= 2 && ok) {
#pragma unroll 1
      for (int c = 0; c < cols; c += 16) {
        uint32_t v[16];
        tmem_ld16(lanes + c, v);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 16; ++e) part[(c + e) * kBM + r] = (int32_t)v[e];
      }
    }
    cluster_sync();
    bool all = write;
    for (int p = 0; p < split; ++p) all = all && ld_cluster(map_rank(smem_u32(&failed), p)) == 0;
    if (warp >= 2 && all)
      add_parts<T, 4>(s0, split, rank, 0, 1, warp - 2, lane, mt * kBM, n0, cols, out, ch4, tok_scale, tok_sum);
    cluster_sync();                                        // no CTA leaves while its sums are read
  }
  fence_before();
  __syncthreads();
  if (failed && threadIdx.x == 0) set_info(info, SGPT_INFO_TIMEOUT);
  if (warp == 0) tmem_free(tmem, kCols);
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
  const int8_t* codes;
  int d;
  Out out;
  int* info;
  cudaStream_t st;
};

// Which kernel, how many tokens a tile, K in how many parts: the least of the
// times (us) that these lines, fitted to every variant on 18 layers (256 to
// 28672 wide) with 1 to 8000 tokens, expect; over those the choice was 1.7 %
// off the best one. One token of 768 -> 768 took 4.3 us in clusters of three
// and takes 2.9 in single CTAs, 333 tokens 5.8 in pairs and 3.1.
//   The split kernel: a wave of 296 CTAs costs its start and epilogue, and
// each K stage its time in every layer of 148 CTAs (two on an SM share it);
// adding K's parts up costs a cluster's two barriers and grows with its size.
// The pair kernel: waves of 74 pairs; K in more than two is not tried there:
// clusters of eight such CTAs do not all find room at once (16 of them took
// two waves); clusters of seven CTAs of the split kernel did not either.
//   Codes that the L2 does not hold come at 6.2 TB/s, and at 70 GB/s a CTA;
// another tile of tokens that reads them at about the same time costs 0.45 as
// much again (17 tokens of 20608 -> 25568: 120 us in two tiles of 16 one after
// the other, 93 side by side, 80 in one of 32).
struct Plan {
  bool pair;
  int bn, split;
};
struct PlanLine {
  bool pair;
  int bn;
  float start, wave, stage, split, part;
};
constexpr PlanLine kPlanLines[] = {{false, 16, 0.f, 2.6f, 0.13f, 1.0f, 0.46f},   {false, 32, 0.f, 2.8f, 0.141f, 0.8f, 0.55f},
                                   {false, 64, 0.f, 2.9f, 0.196f, 1.16f, 0.51f}, {true, 128, 3.1f, 1.7f, 0.161f, 2.8f, 0.f},
                                   {true, 256, 2.7f, 2.9f, 0.289f, 2.3f, 0.f}};

Plan plan(int rows, int n, int d) {
  const int kt = cdiv(d, kBK);
  const float codes = (float)rows * (float)d;
  Plan best{true, 256, 1};
  float least = INFINITY;
  for (const PlanLine& l : kPlanLines) {
    const long long tiles = (long long)cdiv(rows, l.pair ? 2 * kBM : kBM) * cdiv(n, l.bn);
    const long long room = l.pair ? kNumSMs / 2 : kSplitPerSM * kNumSMs;      // clusters of a part each
    if (!l.pair && tiles > 64 * room) continue;
    for (int split = 1; split <= (l.pair ? 2 : kMaxSplit) && split <= kt; split *= 2) {
      if (split > 1 && tiles * split > room) break;
      const long long units = tiles * split, waves = cdivll(units, room), rest = units - (waves - 1) * room;
      const long long layers = l.pair ? waves : 2 * (waves - 1) + (rest > kNumSMs ? 2 : 1);
      float t = l.start + l.wave * waves + l.stage * layers * cdiv(kt, split);
      if (split > 1) t += l.split + l.part * (split - 1);
      if (codes > 32e6f) {
        const float ctas = (float)std::min(units, room) * (l.pair ? 2 : 1);
        // (of two that wait for the codes alike, the one with less else to do)
        const float reads = 1.f + 0.45f * (cdiv(n, l.bn) - 1);
        t = std::max(t, 3.2f + codes * reads / std::min(6.2e6f, ctas * 7.0e4f) + 0.001f * t);
      }
      if (t < least) {
        least = t;
        best = Plan{l.pair, l.bn, split};
      }
    }
  }
  return best;
}

template <int BN, class T>
cudaError_t launch_pair(const Args& a, int split) {
  CUtensorMap wm, xm;
  if (!map_i8(&wm, a.codes, a.out.rows, a.d, kBM) || !map_i8(&xm, a.Xq, a.out.n, a.d, BN / 2))
    return cudaErrorInvalidValue;
  static PerDevice attrs;
  const cudaError_t e = once_per_device(attrs, [] {
    return cudaFuncSetAttribute(linear_i8_pair_kernel<BN, T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)pair_smem(BN));
  });
  if (e != cudaSuccess) return e;
  const long long items = (long long)cdiv(a.out.rows, 2 * kBM) * cdiv(a.out.n, BN);
  if (items > INT32_MAX - kNumSMs) return cudaErrorInvalidValue;       // a Y of 2^47 values
  const int pairs = split > 1 ? (int)items * split : (int)std::min<long long>(items, kNumSMs / 2);
  return launch_after(linear_i8_pair_kernel<BN, T>, 2 * pairs, kPairThreads, pair_smem(BN), 2 * split, a.st, wm, xm, a.d,
                      split, a.out, a.info, wait_limit_cycles());
}

template <int BN, class T>
cudaError_t launch_split(const Args& a, int split) {
  CUtensorMap wm, xm;
  if (!map_i8(&wm, a.codes, a.out.rows, a.d, kBM) || !map_i8(&xm, a.Xq, a.out.n, a.d, BN)) return cudaErrorInvalidValue;
  static PerDevice attrs;
  cudaError_t e = once_per_device(attrs, [] {
    return cudaFuncSetAttribute(linear_i8_split_kernel<BN, T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)split_smem(BN));
  });
  if (e != cudaSuccess) return e;
  const long long tiles = (long long)cdiv(a.out.rows, kBM) * cdiv(a.out.n, BN);
  if (tiles * split > INT32_MAX) return cudaErrorInvalidValue;
  return launch_after(linear_i8_split_kernel<BN, T>, (unsigned)(tiles * split), kThreads, split_smem(BN), split, a.st, wm,
                      xm, a.d, split, a.out, a.info, wait_limit_cycles());
}

template <class T>
cudaError_t dispatch(const Args& a) {
  const Plan p = plan(a.out.rows, a.out.n, a.d);
  if (p.pair) return p.bn == 256 ? launch_pair<256, T>(a, p.split) : launch_pair<128, T>(a, p.split);
  return p.bn == 16 ? launch_split<16, T>(a, p.split)
                    : p.bn == 32 ? launch_split<32, T>(a, p.split) : launch_split<64, T>(a, p.split);
}

}  // namespace

cudaError_t launch_linear_i8(const int8_t* Xq, const float* xs, const int32_t* xsum, long long n, const int8_t* codes,
                             const float* grid, int bits, int d, int rows, void* Y, bool y_bf16, int* info,
                             cudaStream_t st) {
  const Args a{Xq, codes, d, Out{grid, xs, xsum, Y, rows, (int)n, 1 << (bits - 1)}, info, st};
  return y_bf16 ? dispatch<uint16_t>(a) : dispatch<float>(a);
}

}  // namespace sgpt
