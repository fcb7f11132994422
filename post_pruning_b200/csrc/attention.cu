// Causal attention over packed prompts with grouped heads:
//   o_i = sum_{j <= i} p_ij v_j / sum_{j <= i} p_ij,  p_ij = exp(scale q_i . k_j)
// for every sequence of the packed rows and every query head h, which reads
// key/value head h / (heads / kv_heads). One pass over the keys with the
// running maximum m_i and sum l_i of the softmax (fp32); scores and outputs
// accumulate in fp32 on the tensor cores, the weights p_ij of a key block are
// rounded to bf16 for the second product (relative to the running maximum,
// so to 2^-9 of each weight; the sum l_i takes them unrounded).
//
// A unit of work is two 128-row query tiles: the same rows of two heads that
// share a key/value head, or, where the group of heads is odd, two
// consecutive tiles of one head. Both run over the same K and V blocks of 128
// keys, so while one tile's four softmax warps exponentiate, the tensor cores
// work for the other tile. CTAs are persistent and take the units of CTAs
// that have not started yet (the longest ones first), so a unit's operands
// load under the one before it. Warp 8 finds the units and loads Q
// and a ring of K and V blocks by TMA, warp 9 issues the products:
// S = Q K^T into 128 TMEM columns per tile, then, as the softmax warps
// replace S by the bf16 weights in the same columns, half a block at a time,
// O += P V with P read from TMEM, followed by the next S.
//   The running maximum is only raised when a row's maximum has grown by more
// than 2^8 in the exponent's base (weights up to 256 are as exact as weights
// up to 1); then the warp rescales its rows of O in TMEM itself: S of block j
// is complete only after the product of block j - 1.
//
// Few units (few heads, long sequences) leave SMs idle: there a cluster of 2, 4
// or 8 CTAs shares a unit, each with a part of its keys and a maximum, sum
// and O of its own, which are joined through distributed shared memory: each
// CTA writes its share of the rows, O = sum_p f_p O_p / sum_p f_p l_p with
// f_p = exp(m_p - max m). Those CTAs take one unit only.
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
constexpr int kThreads = 384;                   // 2 x 4 softmax warps, TMA, MMA, two idle
// registers a thread after the split: 2 x 200 + 104 = 3 x 168, what the block is launched with
constexpr int kSoftmaxRegs = 200, kOtherRegs = 104;
constexpr int kBox = kT * 128;                  // 16 KB: 128 rows x 64 bf16
// Barriers that free ring slots, one for each group of slots that is freed
// together: at most kStages groups are outstanding (each holds a slot), so with
// as many barriers a wait is never more than one phase behind.
constexpr int kFree = 8;
constexpr float kGrow = 8.f;                    // exponent growth that moves the running maximum

__host__ __device__ constexpr int tile_bytes(int D) { return D / 64 * kBox; }
__host__ __device__ constexpr int stages_for(int D) { return D == 128 ? 5 : 8; }
__host__ __device__ constexpr size_t smem_for(int D) {
  return (size_t)(2 + stages_for(D)) * tile_bytes(D) + 1024 + 512;
}
static_assert(kFree >= stages_for(128) && kFree >= stages_for(64) && 8 * (22 + kFree + stages_for(64)) <= 512, "barriers");
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

// The weights exp2(c s - mc) of 64 scores, as bf16 pairs, and their sums.
__device__ __forceinline__ void weights(const uint32_t (&a)[32], const uint32_t (&b)[32], uint64_t c2, float mc,
                                        uint32_t (&p)[32], uint64_t (&sum)[2]) {
  const uint64_t mc2 = pair_of(-mc, -mc);
  sum[0] = sum[1] = 0;
#pragma unroll
  for (int e = 0; e < 32; ++e) {
    const uint32_t lo = e < 16 ? a[2 * e] : b[2 * e - 32], hi = e < 16 ? a[2 * e + 1] : b[2 * e - 31];
    const float2 x = pair_to(fma2(pair_of(__uint_as_float(lo), __uint_as_float(hi)), c2, mc2));
    const float u = ex2(x.x), v = ex2(x.y);
    sum[e & 1] = add2(sum[e & 1], pair_of(u, v));
    p[e] = pack_bf16(u, v);
  }
}

struct Shape {
  long long ldo;             // elements between rows of O
  int n_tok, n_seq, heads, group;
  int pair;                  // 1: a unit's two tiles are two heads of one group; 0: two row tiles of one head
  int wide;                  // 1: rows of O start on 32-byte boundaries
  float c;                   // scale * log2(e)
};

// A unit of work: two tiles. len == 0 ends the CTA.
struct Work {
  int first, len, unit, head_unit;
  __device__ int head(const Shape& sh, int h) const { return sh.pair ? 2 * head_unit + h : head_unit; }
  // tile h's first row in the sequence, and its key blocks
  __device__ int row(const Shape& sh, int h) const { return sh.pair ? unit * kT : (2 * unit + h) * kT; }
  __device__ int all_blocks(const Shape& sh, int h) const { return row(sh, h) < len ? row(sh, h) / kT + 1 : 0; }
  // of these, the ones of CTA `part` of the unit's cluster, from first_block on
  template <int PARTS>
  __device__ int first_block(const Shape& sh, int part) const {
    return PARTS > 1 ? max(all_blocks(sh, 0), all_blocks(sh, 1)) * part / PARTS : 0;
  }
  template <int PARTS>
  __device__ int blocks(const Shape& sh, int h, int part) const {
    if (PARTS == 1) return all_blocks(sh, h);
    return max(0, min(all_blocks(sh, h), first_block<PARTS>(sh, part + 1)) - first_block<PARTS>(sh, part));
  }
};

// Where the last search ended: the first of 32 sequences, and the units before it.
struct Search {
  int b0 = 0;
  long long before = 0;
};

// The unit `index` of the launch, by a whole warp, which goes on from its last
// search (a CTA's indices mostly grow). Units of rows are taken from 32
// sequences after 32, a lane each, the longest rows of keys of all of them
// first: f(u) units have the number u or a later one in their sequence, and
// the search halves the interval of u. (One sequence after the other left the
// long units of the last one to the end: ten prompts of 2 to 1355 rows took
// 39 us instead of 27, 8 x 2048 rows a twentieth longer.) A sequence's offsets
// are used only if they lie inside the packed rows.
__device__ Work find_work(const Shape& sh, const int32_t* cu, int index, int lane, Search& at_seq) {
  const int head_units = sh.pair ? sh.heads / 2 : sh.heads;
  const int unit_rows = sh.pair ? kT : 2 * kT;
  const int unit = index / head_units;
  Work w{0, 0, 0, index % head_units};
  if (unit < at_seq.before) at_seq = Search();
  for (; at_seq.b0 < sh.n_seq; at_seq.b0 += 32) {
    const int b = at_seq.b0 + lane;
    int first = 0, len = 0;
    if (b < sh.n_seq) {
      first = cu[b];
      const int end = cu[b + 1];
      len = first >= 0 && end >= first && end <= sh.n_tok ? end - first : 0;
    }
    const int units = cdiv(len, unit_rows);
    auto f = [&](int u) { return (int)__reduce_add_sync(0xffffffffu, (unsigned)max(0, units - u)); };
    const int all = f(0);
    const long long at = unit - at_seq.before;
    if (at < all) {
      int lo = 0, hi = (int)__reduce_max_sync(0xffffffffu, (unsigned)units), later = 0;      // f(lo) > at >= f(hi) = later
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2, n = f(mid);
        if (n > at) {
          lo = mid;
        } else {
          hi = mid;
          later = n;
        }
      }
      const unsigned with = __ballot_sync(0xffffffffu, units > lo);
      const int rank = __popc(with & ((1u << lane) - 1));
      const int src = __ffs(__ballot_sync(0xffffffffu, units > lo && rank == (int)at - later)) - 1;
      w.first = __shfl_sync(0xffffffffu, first, src);
      w.len = __shfl_sync(0xffffffffu, len, src);
      w.unit = lo;
      return w;
    }
    at_seq.before += all;
  }
  return w;
}

// Every offset is looked at once, by one warp.
__device__ void check_offsets(const Shape& sh, const int32_t* cu, int lane, int* info) {
  bool bad = false;
  for (int b = lane; b < sh.n_seq; b += 32) bad |= cu[b] < 0 || cu[b + 1] < cu[b] || cu[b + 1] > sh.n_tok;
  if (__any_sync(0xffffffffu, bad) && lane == 0) set_info(info, SGPT_INFO_BAD_LENGTHS);
}

__device__ __forceinline__ void store32(uint16_t* p, const uint32_t* v, bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}

// Transposes four 32-byte pieces of a row over the four lanes of a quad: in,
// lane x has the pieces 0..3 of row x; out, lane x has piece x of the rows
// 0..3. A store then writes 128 consecutive bytes of eight rows instead of 32
// bytes of each of 32 rows, a quarter of the lines. For a width of 128 those
// lines took 1900 of the epilogue's 2700 cycles (8 x 2048 rows in a row, 64
// heads on 8: 632 -> 616 us; 16 on 2: 157.6 -> 155.5; eight ragged prompts, 32
// on 32: 144.5 -> 147.3). It costs more than it saves for a width of 64 (half
// the lines) and in units of one or two blocks, whose epilogue nothing hides.
__device__ __forceinline__ void quad_transpose(uint32_t (&v)[32], int lane) {
#pragma unroll
  for (int bit = 1; bit < 4; bit <<= 1) {
    const bool odd = lane & bit;
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      if (a & bit) continue;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int lo = 8 * a + i, hi = 8 * (a | bit) + i;
        const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? v[lo] : v[hi], bit);
        if (odd)
          v[lo] = got;
        else
          v[hi] = got;
      }
    }
  }
}

// One wait's count on a barrier: the n-th wait takes parity n & 1.
struct Phase {
  uint32_t n = 0;
  __device__ uint32_t next() { return n++ & 1u; }
};

template <int D, int PARTS>
__global__ void __launch_bounds__(kThreads, 1) attention_kernel(
    const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
    const __grid_constant__ CUtensorMap vmap, const int32_t* cu, const Shape sh, uint16_t* O, int* info, const long long wait_cycles) {
  constexpr int kTile = tile_bytes(D), kStages = stages_for(D);
  constexpr bool SPLIT = PARTS > 1;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + (2 + kStages) * kTile);
  __shared__ __align__(16) uint32_t answer[4];
  __shared__ uint32_t tmem_slot;
  __shared__ int failed;
  __shared__ Work work[2];
  __shared__ int group_of[kStages];              // producer's: what frees each ring slot
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = SPLIT ? (int)cluster_rank() : 0;
  const uint32_t s0 = smem_u32(smem);
  const uint32_t ring = s0 + 2 * kTile;
  // [2]: one per tile or per work slot
  const uint32_t qfull = smem_u32(bars), qempty = qfull + 16, sfull = qempty + 16, ofull = sfull + 16;
  const uint32_t pfull = ofull + 16;             // [2][2]: a block's first 64 keys, its last 64
  const uint32_t wfull = pfull + 32, wempty = wfull + 16;
  const uint32_t full0 = wempty + 16, free0 = full0 + 8 * kStages;    // [kStages], [kFree]
  const uint32_t vask = free0 + 8 * kFree, vready = vask + 8, stolen = vready + 8, mdone = stolen + 8;
  if (threadIdx.x == 0) {
    prefetch_map(&qmap);
    prefetch_map(&kmap);
    prefetch_map(&vmap);
    failed = 0;
    for (int h = 0; h < 2; ++h) {
      mbar_init(qfull + 8 * h, 1);
      mbar_init(qempty + 8 * h, 1);
      mbar_init(sfull + 8 * h, 1);
      mbar_init(ofull + 8 * h, 1);
      mbar_init(pfull + 16 * h, 4);
      mbar_init(pfull + 16 * h + 8, 4);
      mbar_init(wfull + 8 * h, 1);
      mbar_init(wempty + 8 * h, 10);             // eight softmax warps, the MMA warp, the V tail warp
    }
    for (int s = 0; s < kStages; ++s) mbar_init(full0 + 8 * s, 1);
    for (int s = 0; s < kFree; ++s) mbar_init(free0 + 8 * s, 1);
    mbar_init(vask, 1);
    mbar_init(vready, 1);
    mbar_init(stolen, 1);
    mbar_init(mdone, 1);
    mbar_init_fence();
  }
  let_next_start();
  after_previous();
  Search at_seq;
  Work w0{0, 0, 0, 0};                           // warp 8's first unit: its offsets load under the set-up
  if (warp == 8) w0 = find_work(sh, cu, blockIdx.x / PARTS, lane, at_seq);
  if (warp == 9) tmem_alloc(smem_u32(&tmem_slot), kTmemCols);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_slot, 0);

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == 8) {
      // Units of work, one after the other, and their operands. The next
      // unit's index is asked for while this one's operands are loaded.
      int index = blockIdx.x;
      uint32_t g = 0, units = 0, groups = 0;     // ring slots, units and groups of slots so far
      uint32_t q_used[2] = {0, 0};
      bool ok = true, asked = false, first = true;
      Phase answers;
      while (ok) {
        const Work w = index < 0 ? Work{0, 0, 0, 0} : first ? w0 : find_work(sh, cu, index, lane, at_seq);
        first = false;
        if (!SPLIT && index >= 0) {
          if (lane == 0) {
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");    // this lane has read the last answer
            mbar_expect(stolen, 16);
            steal_cta(smem_u32(answer), stolen);
          }
          asked = true;
        }
        if (index < 0 || w.len) {
          const int slot = units & 1;
          if (lane == 0) {
            if (units >= 2 && !mbar_wait(wempty + 8 * slot, (units / 2 - 1) & 1, wait_cycles)) ok = false;
            if (ok) {
              work[slot] = w;
              mbar_arrive(wfull + 8 * slot);
            }
          }
          ok = __all_sync(0xffffffffu, ok);
          ++units;
        }
        if (index < 0 || !ok) break;
        if (w.len && lane == 0) {
          const int nb0 = w.blocks<PARTS>(sh, 0, part), nb1 = w.blocks<PARTS>(sh, 1, part), nb = max(nb0, nb1);
          const int kvh = w.head(sh, 0) / sh.group, key0 = w.first + w.first_block<PARTS>(sh, part) * kT;
          for (int x = 0; x < 2 * nb && ok; ++x, ++g) {             // K0 V0 K1 V1 ...
            const uint32_t s = g % kStages;
            if (g >= kStages) {
              const uint32_t f = group_of[s];
              if (!mbar_wait(free0 + 8 * (f % kFree), (f / kFree) & 1, wait_cycles)) {
                ok = false;
                break;
              }
            }
            group_of[s] = groups + (x + 1) / 2;                      // K0 | V0 K1 | V1 K2 | ... | the last V
            mbar_expect(full0 + 8 * s, kTile);
            for (int c = 0; c < D / 64; ++c)
              tma_3d(ring + s * kTile + c * kBox, (x & 1) ? &vmap : &kmap, full0 + 8 * s, 64 * c, kvh, key0 + (x >> 1) * kT);
            if (x == 0) {
              for (int h = 0; h < 2 && ok; ++h) {
                if (!(h ? nb1 : nb0)) continue;
                if (q_used[h] && !mbar_wait(qempty + 8 * h, (q_used[h] - 1) & 1, wait_cycles)) {
                  ok = false;
                  break;
                }
                ++q_used[h];
                mbar_expect(qfull + 8 * h, kTile);
                for (int c = 0; c < D / 64; ++c)
                  tma_3d(s0 + h * kTile + c * kBox, &qmap, qfull + 8 * h, 64 * c, w.head(sh, h), w.first + w.row(sh, h));
              }
            }
          }
          groups += nb + 1;
        }
        __syncwarp();
        if (SPLIT) {                             // one unit per cluster
          ok = __all_sync(0xffffffffu, ok);
          index = -1;
          continue;
        }
        const uint32_t parity = answers.next();
        bool got = mbar_wait(stolen, parity, wait_cycles);
        if (!got) mbar_wait(stolen, parity, kDrainCycles);
        asked = false;
        ok = __all_sync(0xffffffffu, ok && got);
        // by lane 0 alone: no other lane's read has to be ordered before the next answer
        index = __shfl_sync(0xffffffffu, lane == 0 ? stolen_cta(smem_u32(answer)) : 0, 0);
        // the first CTA looks at the offsets; which CTAs are taken is not
        // specified, so whoever takes that one does it instead
        if (index == 0) check_offsets(sh, cu, lane, info);
      }
      if (!ok && lane == 0) {
        failed = 1;
        // what is still in flight lands before the CTA ends
        if (asked) mbar_wait(stolen, answers.next(), kDrainCycles);
        for (int h = 0; h < 2; ++h)
          if (q_used[h]) mbar_wait(qfull + 8 * h, (q_used[h] - 1) & 1, kDrainCycles);
        for (uint32_t x = g > kStages ? g - kStages : 0; x < g; ++x)
          mbar_wait(full0 + 8 * (x % kStages), (x / kStages) & 1, kDrainCycles);
      }
    } else if (warp == 9) {
      if (elect_one()) {
        const uint64_t q_desc = sw128_desc(s0), k_desc = sw128_desc(ring), v_desc = sw128_desc(ring, kBox);
        // No instruction more than needed between the products: the tensor
        // cores idle while this thread is late.
        struct Slot {                                      // of the ring, in the order of use
          uint32_t s, parity;
          __device__ void step() {
            if (++s == kStages) {
              s = 0;
              parity ^= 1;
            }
          }
        };
        auto loaded = [&](Slot x) { return mbar_wait(full0 + 8 * x.s, x.parity, wait_cycles); };
        auto is_loaded = [&](Slot x) { return mbar_test(full0 + 8 * x.s, x.parity); };
        auto score = [&](int h, Slot x, bool last) {       // S_h = Q_h K^T
          const uint64_t qd = q_desc + (uint64_t)(h * kTile >> 4), kd = k_desc + (uint64_t)(x.s * (kTile >> 4));
          const uint32_t acc = tmem + h * kT;
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint64_t off = ((ks >> 2) * kBox + 32 * (ks & 3)) >> 4;
            mma_ss(acc, qd + off, kd + off, idesc(kT, false), ks > 0);
          }
          mma_commit(sfull + 8 * h);
          if (last) mma_commit(qempty + 8 * h);
        };
        auto units_done = [&]() -> bool {                  // false: a wait ran out
          Slot at{0, 0};                                   // the next slot to use
          uint32_t groups = 0;
          // parities of the next waits on qfull, pfull (per tile) and vready
          uint32_t parities = 0;
          constexpr uint32_t kQ = 1, kP = 4, kV = 16;
          auto next_of = [&](uint32_t bit) {
            const uint32_t p = (parities & bit) != 0;
            parities ^= bit;
            return p;
          };
          bool ahead = false;                              // the first tile's first scores are under way
          for (uint32_t u = 0;; ++u) {
            if (!mbar_wait(wfull + 8 * (u & 1), (u >> 1) & 1, wait_cycles)) return false;
            const Work w = work[u & 1];
            mbar_arrive(wempty + 8 * (u & 1));
            if (!w.len) return true;
            const int nb0 = w.blocks<PARTS>(sh, 0, part), nb1 = w.blocks<PARTS>(sh, 1, part), nb = max(nb0, nb1);
            if (SPLIT && !nb) continue;
            // the block inside which the sequence ends
            const int tail = w.len % kT ? w.len / kT - w.first_block<PARTS>(sh, part) : nb;
            if (!loaded(at)) return false;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int mine = h ? nb1 : nb0;
              if (!mine || (h == 0 && ahead)) continue;
              if (!mbar_wait(qfull + 8 * h, next_of(kQ << h), wait_cycles)) return false;
              score(h, at, mine == 1);
            }
            ahead = false;
            mma_commit(free0 + 8 * (groups++ % kFree));
            at.step();
            bool v_here = false, k_here = false;           // this block's V and the next one's K have been seen
            for (int j = 0; j < nb; ++j) {
              if (!v_here && !loaded(at)) return false;
              if (j == tail) {
                mbar_arrive(vask);
                if (!mbar_wait(vready, next_of(kV), wait_cycles)) return false;
              }
              const uint64_t vd = v_desc + (uint64_t)(at.s * (kTile >> 4));
              at.step();
              const Slot k = at;                           // the next block's K (or the next unit's)
              v_here = false;
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int mine = h ? nb1 : nb0;
                if (j >= mine) continue;
                const uint32_t acc = tmem + 2 * kT + h * kT, pd = tmem + h * kT, par = next_of(kP << h);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                  if (!mbar_wait(pfull + 16 * h + 8 * half, par, wait_cycles)) return false;
                  fence_after();
#pragma unroll
                  for (int x = 4 * half; x < 4 * half + 4; ++x)
                    mma_ts(acc, pd + 8 * x, vd + (uint64_t)(2048 * x >> 4), idesc(D, true), x > 0 ? 1u : (uint32_t)(j > 0));
                  if (half == 0 && j + 1 < nb) {
                    // looked for here, where there is time until the second half
                    if (h == 0) {
                      k_here = is_loaded(k);
                    } else {
                      Slot v = k;
                      v.step();
                      v_here = is_loaded(v);
                    }
                  }
                }
                if (j + 1 < mine) {
                  if (!k_here && !loaded(k)) return false;
                  k_here = true;
                  score(h, k, j + 2 == mine);
                } else {
                  mma_commit(ofull + 8 * h);
                  // the first tile goes on to the next unit, if that is here,
                  // while the second one is still at this unit's last block
                  if (!SPLIT && h == 0) {
                    Slot first = k;                        // of the next unit
                    if (nb1 > nb0) {
                      first.step();
                      first.step();
                    }
                    const uint32_t v = (u + 1) & 1;
                    if (mbar_test(wfull + 8 * v, ((u + 1) >> 1) & 1) && work[v].len && is_loaded(first) &&
                        mbar_test(qfull, parities & kQ)) {
                      parities ^= kQ;
                      score(0, first, work[v].blocks<PARTS>(sh, 0, part) == 1);
                      ahead = true;
                    }
                  }
                }
              }
              mma_commit(free0 + 8 * (groups++ % kFree));
              if (j + 1 < nb) at.step();
              k_here = false;
            }
          }
        };
        if (!units_done()) failed = 1;
        // never free TMEM under a running MMA
        mma_commit(mdone);
        if (!mbar_wait(mdone, 0, kDrainCycles)) failed = 1;
      }
    } else if (warp == 10) {
      // Zeroes the rows of V after the end of a sequence in the block that
      // holds it: their weights are zero, but zero times a NaN is not.
      uint32_t g = 0;
      Phase asked;
      for (uint32_t u = 0;; ++u) {
        if (__any_sync(0xffffffffu, !mbar_wait(wfull + 8 * (u & 1), (u >> 1) & 1, wait_cycles))) break;
        const Work w = work[u & 1];
        __syncwarp();
        if (lane == 0) mbar_arrive(wempty + 8 * (u & 1));
        if (!w.len) break;
        const int nb = max(w.blocks<PARTS>(sh, 0, part), w.blocks<PARTS>(sh, 1, part)), keys = w.len % kT;
        if (keys && nb && w.first_block<PARTS>(sh, part) + nb - 1 == w.len / kT) {
          const uint32_t s = (g + 2 * nb - 1) % kStages;
          if (__any_sync(0xffffffffu, !mbar_wait(vask, asked.next(), wait_cycles))) break;
          for (int c = 0; c < D / 64; ++c)
            for (int i = keys * 8 + lane; i < kT * 8; i += 32)
              *reinterpret_cast<uint4*>(smem + (2 + s) * kTile + c * kBox + 16 * i) = make_uint4(0, 0, 0, 0);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(vready);
        }
        g += 2 * nb;
      }
    } else if (blockIdx.x == 0) {
      check_offsets(sh, cu, lane, info);
    }
    if (SPLIT) cluster_sync();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int h = warp >> 2, q = warp & 3;
    const uint32_t lanes = (uint32_t)(q * 32) << 16;
    const uint32_t ts = tmem + lanes + h * kT, to = tmem + lanes + 2 * kT + h * kT;
    const int r = q * 32 + lane;                           // row in the tile
    const uint64_t c2 = pair_of(sh.c, sh.c);
    Phase sn, on;
    bool ok = true;
    Work shared_unit{0, 0, 0, 0};                          // SPLIT: the unit, and the row's maximum and sum here
    float shared_m = 0.f, shared_l = 0.f;
    // an error recorded by an earlier call: everything runs, nothing is
    // written (the look at *info is under the first products)
    const bool write = !info_set(info);
    auto wait = [&](uint32_t bar, uint32_t parity) {       // one decision for the warp
      ok = !__any_sync(0xffffffffu, !mbar_wait(bar, parity, wait_cycles));
      fence_after();
      return ok;
    };
    for (uint32_t u = 0;; ++u) {
      if (!wait(wfull + 8 * (u & 1), (u >> 1) & 1)) break;
      const Work w = work[u & 1];
      __syncwarp();
      if (lane == 0) mbar_arrive(wempty + 8 * (u & 1));
      if (!w.len) break;
      const int mine = w.blocks<PARTS>(sh, h, part);
      if (SPLIT) shared_unit = w;
      if (!mine) continue;
      const int last = SPLIT ? w.row(sh, h) / kT - w.first_block<PARTS>(sh, part) : mine - 1;
      float m = -INFINITY;
      uint64_t l2[2] = {0, 0};                             // the row's sum, in four parts
      for (int j = 0; j < mine; ++j) {
        if (!wait(sfull + 8 * h, sn.next())) break;
        const bool diagonal = j == last;
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
        // The first half of the weights is formed with the maximum that the
        // row had before this block, under the search for the block's own;
        // they are formed again in the rare block that moves the maximum (the
        // first block has no maximum before it).
        uint32_t p[32];
        uint64_t sum[2];
        if (j > 0) weights(s[0], s[1], c2, m * sh.c, p, sum);
        const bool grow = j == 0 || (top - m) * sh.c > kGrow;
        if (__any_sync(0xffffffffu, grow)) {
          const float mnew = grow ? top : m;
          if (j > 0) {
            const float alpha = ex2((m - mnew) * sh.c);    // 1 where the maximum stays
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
          weights(s[0], s[1], c2, m * sh.c, p, sum);
        }
        tmem_st32(ts, p);
        l2[0] = add2(l2[0], sum[0]);
        l2[1] = add2(l2[1], sum[1]);
        tmem_st_wait();
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(pfull + 16 * h);
        weights(s[2], s[3], c2, m * sh.c, p, sum);
        tmem_st32(ts + 32, p);
        l2[0] = add2(l2[0], sum[0]);
        l2[1] = add2(l2[1], sum[1]);
        tmem_st_wait();
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(pfull + 16 * h + 8);
      }
      if (!ok || !wait(ofull + 8 * h, on.next())) break;
      const float2 la = pair_to(l2[0]), lb = pair_to(l2[1]);
      const float l = (la.x + la.y) + (lb.x + lb.y);
      if (SPLIT) {
        shared_m = m;
        shared_l = l;
        continue;
      }
      const float inv = 1.f / l;
      const int row = w.row(sh, h) + r;
      uint64_t bad = 0;                                    // a sum of o * 0: NaN if one is not finite
      const uint64_t inv2 = pair_of(inv, inv);
      uint16_t* op = O + (long long)(w.first + row) * sh.ldo + w.head(sh, h) * D;
      auto chunk = [&](int i, uint32_t* v) {               // 32 columns of the row
        uint32_t o[32];
        tmem_ld32(to + 32 * i, o);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const uint64_t y = fma2(pair_of(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1])), inv2, 0);
          bad = fma2(y, 0, bad);
          v[e] = pack_bf16(pair_to(y).x, pair_to(y).y);
        }
      };
      if (D == 128 && mine > 2) {
        const int quad = lane & 3;
        // a warp without a row of the sequence has nothing to write
#pragma unroll 1
        for (int i = row - lane < w.len ? 0 : 2; i < 2; ++i) {
          uint32_t v[32];
          chunk(2 * i, v);
          chunk(2 * i + 1, v + 16);
          quad_transpose(v, lane);
#pragma unroll
          for (int x = 0; x < 4; ++x)
            if (row - quad + x < w.len && write) store32(op + (x - quad) * sh.ldo + 64 * i + 16 * quad, v + 8 * x, sh.wide);
        }
      } else {
#pragma unroll 1
        for (int i = 0; i < D / 32; ++i) {
          uint32_t v[16];
          chunk(i, v);
          if (row < w.len && write) {
            store32(op + 32 * i, v, sh.wide);
            store32(op + 32 * i + 16, v + 8, sh.wide);
          }
        }
      }
      fence_before();                                      // O is read: the next unit's weights follow
      if (!(pair_to(bad).x + pair_to(bad).y == 0.f) && row < w.len) set_info(info, SGPT_INFO_NONFINITE);
    }
    if (!ok) failed = 1;
    if constexpr (SPLIT) {
      // Both tiles' products are done: their operands' place takes this
      // part's O (fp32, rows of D with their 16-byte pieces swapped about so
      // that neither side meets bank conflicts) and, behind it, m and l.
      asm volatile("bar.sync 1, 256;" ::: "memory");
      const Work w = shared_unit;
      const uint32_t ml = s0 + 2 * kT * D * 4;             // [2][kT] pairs
      if (ok && w.blocks<PARTS>(sh, h, part)) {
        const uint32_t line = s0 + (h * kT + r) * D * 4;
#pragma unroll 1
        for (int i = 0; i < D / 16; ++i) {
          uint32_t o[16];
          tmem_ld16(to + 16 * i, o);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int piece = (4 * i + e) ^ (lane & 7);
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(line + 16 * piece), "r"(o[4 * e]),
                         "r"(o[4 * e + 1]), "r"(o[4 * e + 2]), "r"(o[4 * e + 3])
                         : "memory");
          }
        }
        asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(ml + 8 * (h * kT + r)), "f"(shared_m), "f"(shared_l)
                     : "memory");
      }
      cluster_sync();
      bool all = write && w.len;
      for (int p = 0; p < PARTS; ++p) all = all && ld_cluster(map_rank(smem_u32(&failed), p)) == 0;
      // A warp takes whole rows, four columns a lane, with 16 loads of O in
      // flight: one row at a time took 4 (width 64) to 8 us more in two parts.
      constexpr int kAtOnce = 128 / D, kRows = 16 / PARTS;
      const int piece = lane % (D / 4);
#pragma unroll 1
      for (int x0 = (part * 8 + warp) * kAtOnce + lane / (D / 4); x0 < 2 * kT && all; x0 += 16 * 8 * kAtOnce) {
        int4 o[kRows][PARTS];
        float pm[kRows][PARTS], pl[kRows][PARTS];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          const int x = x0 + 8 * PARTS * kAtOnce * i, g = x / kT;
#pragma unroll
          for (int p = 0; p < PARTS; ++p) {
            if (w.blocks<PARTS>(sh, g, p)) {
              ld_cluster2(map_rank(ml + 8 * x, p), pm[i][p], pl[i][p]);
              o[i][p] = ld_cluster4(map_rank(s0 + x * D * 4 + 16 * (piece ^ (x & 7)), p));
            } else {
              pm[i][p] = -INFINITY;
              pl[i][p] = 0.f;
              o[i][p] = make_int4(0, 0, 0, 0);
            }
          }
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          const int x = x0 + 8 * PARTS * kAtOnce * i, g = x / kT, row = w.row(sh, g) + x % kT;
          float top = pm[i][0], l = 0.f, y[4] = {}, bad = 0.f;
#pragma unroll
          for (int p = 1; p < PARTS; ++p) top = fmaxf(top, pm[i][p]);
#pragma unroll
          for (int p = 0; p < PARTS; ++p) {
            const float f = ex2((pm[i][p] - top) * sh.c);
            l = fmaf(f, pl[i][p], l);
            y[0] = fmaf(f, __int_as_float(o[i][p].x), y[0]);
            y[1] = fmaf(f, __int_as_float(o[i][p].y), y[1]);
            y[2] = fmaf(f, __int_as_float(o[i][p].z), y[2]);
            y[3] = fmaf(f, __int_as_float(o[i][p].w), y[3]);
          }
          if (row >= w.len) continue;
          const float inv = 1.f / l;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            y[e] *= inv;
            bad = fmaf(y[e], 0.f, bad);
          }
          *reinterpret_cast<uint2*>(O + (long long)(w.first + row) * sh.ldo + w.head(sh, g) * D + 4 * piece) =
              make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
          if (!(bad == 0.f)) set_info(info, SGPT_INFO_NONFINITE);
        }
      }
    }
  }
  fence_before();
  __syncthreads();
  if (failed && threadIdx.x == 0) set_info(info, SGPT_INFO_TIMEOUT);
  if (SPLIT) cluster_sync();                               // no CTA leaves while its part is read
  if (warp == 9) tmem_free(tmem, kTmemCols);
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

template <int D, int PARTS>
cudaError_t launch(const CUtensorMap& qm, const CUtensorMap& km, const CUtensorMap& vm, const int32_t* cu,
                   const Shape& sh, long long units, uint16_t* O, int* info, cudaStream_t st) {
  static PerDevice attrs;
  const cudaError_t e = once_per_device(attrs, [] {
    return cudaFuncSetAttribute(attention_kernel<D, PARTS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)smem_for(D));
  });
  if (e != cudaSuccess) return e;
  return launch_after(attention_kernel<D, PARTS>, (unsigned)(units * PARTS), kThreads, smem_for(D), PARTS, st, qm, km,
                      vm, cu, sh, O, info, wait_limit_cycles());
}

template <int D>
cudaError_t launch_parts(int parts, const CUtensorMap& qm, const CUtensorMap& km, const CUtensorMap& vm,
                         const int32_t* cu, const Shape& sh, long long units, uint16_t* O, int* info, cudaStream_t st) {
  return parts == 8   ? launch<D, 8>(qm, km, vm, cu, sh, units, O, info, st)
         : parts == 4 ? launch<D, 4>(qm, km, vm, cu, sh, units, O, info, st)
         : parts == 2 ? launch<D, 2>(qm, km, vm, cu, sh, units, O, info, st)
                      : launch<D, 1>(qm, km, vm, cu, sh, units, O, info, st);
}

// Into how many parts the keys of a unit are split: the least of the times
// (us) that this expects for sequences of one length (the longest of several
// taken as a quarter longer: it decides, and only the device knows it). A unit
// takes `block` for each block of its two tiles' keys and `start` once; the
// launch takes its longest part, or all parts over the SMs. Clusters of four
// or eight CTAs find room for 32 and 14 at once (16 of eight took two waves),
// and each further wave of them waits for the one before. Fitted to 336
// launches of 1 to 32 heads on 1 to 32, 64 to 8192 rows; over these the choice
// was 1.3 % off the best part count, and 1 part 23 %. One head of 8192 rows:
// 105 us in 1 part, 59 in 2, 35 in 4 (width 64); 8 heads on 2 of 3000 rows: 45
// in 1, 28 in 2; 512 rows 12.0 in 1, 10.1 in 4.
int parts_for(long long n_tok, int n_seq, int head_units, bool pair, int D) {
  constexpr float kStart[2][4] = {{5.8f, 8.3f, 8.3f, 9.2f}, {6.3f, 10.9f, 10.9f, 11.7f}};    // width; 1, 2, 4, 8 parts
  constexpr int kRoom[4] = {kNumSMs, kNumSMs / 2, 32, 14};
  const float block = D == 64 ? 1.6f : 1.7f;
  const float* start = kStart[D == 128];
  const long long seqs = std::min<long long>(n_seq, n_tok);
  const int rows = pair ? kT : 2 * kT;
  const int of_seq = (int)cdivll(cdivll(n_tok, n_seq), rows);                // units of rows
  const float units = (float)seqs * of_seq * head_units;
  const float blocks = units * 0.5f * (pair ? of_seq + 1 : 2 * (of_seq + 1));    // of all units
  int longest = (int)cdivll(n_seq > 1 ? cdivll(5 * n_tok, 4ll * n_seq) : n_tok, kT);
  if (!pair && longest > 1) longest -= longest & 1;                          // one tile alone takes less than two
  if (longest < 4) return 1;                                                 // at 3 blocks nothing gains 3 %
  int best = 1;
  float least = start[0] + std::max(block * longest, (block * blocks + 2 * (units - kNumSMs)) / kNumSMs);
  for (int i = 1; i < 4; ++i) {
    const int parts = 1 << i;
    const float part = block * cdiv(longest, parts), all = (block * blocks + units * parts * start[i]) / kNumSMs;
    float t = std::max(start[i] + part, all);
    if (units > kRoom[i]) {
      t = std::max(t, 1.1f * all);
      if (i > 1) t = std::max(t, std::ceil(units / kRoom[i]) * start[i] + part);
    }
    if (t < least) {
      least = t;
      best = parts;
    }
  }
  return best;
}

}  // namespace

// CTAs of a launch: the units of rows that n_seq sequences of n_tok rows in
// all can have, for each unit of heads.
long long attention_ctas(long long n_tok, int n_seq, int heads, int kv_heads) {
  const bool pair = heads / kv_heads % 2 == 0;
  const int unit_rows = pair ? kT : 2 * kT;      // a sequence's last unit may have one row only
  const long long units = (n_tok + std::min<long long>(n_seq, n_tok) * (unit_rows - 1)) / unit_rows;
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
  sh.wide = (reinterpret_cast<uintptr_t>(O) & 31u) == 0 && ldo % 16 == 0;
  sh.c = (float)((double)scale * 1.4426950408889634);
  const long long units = attention_ctas(n_tok, n_seq, heads, kv_heads);
  const int parts = parts_for(n_tok, n_seq, sh.pair ? heads / 2 : heads, sh.pair, D);
  return D == 128 ? launch_parts<128>(parts, qm, km, vm, cu, sh, units, O, info, st)
                  : launch_parts<64>(parts, qm, km, vm, cu, sh, units, O, info, st);
}

}  // namespace sgpt
