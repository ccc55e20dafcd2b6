// Choosing the cache blocks a query attends to.
//
// summarize: when a block is full, each KV head's keys in it are bounded per
// channel, lo_d <= k_d <= hi_d, in 8 bits: with u the smallest power of two,
// at least 2^-50, for which max |k| / u <= 127,
//   hi_d = ceil(max_t k_td / u),  lo_d = floor(min_t k_td / u)
// (rounded outward, so that the bound holds), u kept as fp32.
//
// select: the logit of any key in block j is at most
//   sum_d max(q_d hi_d, q_d lo_d) u_j,
// and a block's score is the largest of these over the KV head's query
// heads, each query rounded to 8 bits under a power-of-two scale of its own.
// The sum is a whole number below 2^22 and the scales are powers of two, so
// a score is exact in fp32 whatever the order of its sums: the selection is
// the same on every run and for every launch shape, ties to the lowest index.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "launch.cuh"
#include "pa_device.cuh"
#include "pa_kernels.cuh"
#include "tc_ptx.cuh"

namespace pa {

namespace {

constexpr float kClamp = 1125899906842624.f;  // 2^50: larger keys and queries count as this
constexpr int kMinExp = -50;

// The exponent of the smallest power of two u >= 2^-50 with amax / u <= 127.
__device__ __forceinline__ int exponent_for(float amax) {
  if (!(amax > 0.f)) return kMinExp;
  int e;
  const float m = frexpf(amax, &e);  // amax = m 2^e, m in [0.5, 1)
  e = m * 128.f <= 127.f ? e - 7 : e - 6;
  return e < kMinExp ? kMinExp : e;
}
__device__ __forceinline__ float exp2i(int e) { return __int_as_float((127 + e) << 23); }

// ------------------------------------------------------------- summarize

constexpr int kSumWarps = 8;

// Extremes of packed pairs (NaN loses against a number).
template <bool FP8>
struct Pair;
template <>
struct Pair<false> {
  using T = __nv_bfloat162;
  static __device__ __forceinline__ float2 f(T v) { return __bfloat1622float2(v); }
};
template <>
struct Pair<true> {
  using T = __half2;
  static __device__ __forceinline__ float2 f(T v) { return __half22float2(v); }
};

// Bound: the keys' bytes, read once.  The unit of work is a full block's
// column of 32 consecutive 16-byte pieces (512 bytes of each token's row,
// whole heads): a warp reads it with 8 loads in flight, and the extremes
// stay packed in the cache's own precision, where they are exact.  A CTA
// looks at up to 32 consecutive tokens of the step and takes the blocks
// whose last slot is among them.  kSplit = 1: each warp takes a column of
// its own, and no warp waits for another.  kSplit = 8 (blocks of 64 tokens
// and more, where one warp's walk would be the call's time): all 8 warps of
// the CTA share a column's tokens and their results meet in shared memory.
template <int D, bool FP8, int kSplit>
__global__ void __launch_bounds__(32 * kSumWarps, FP8 ? 2 : 4)
    summarize_kernel(const __grid_constant__ SummaryParams p, int tokens_per_cta) {
  using P2 = typename Pair<FP8>::T;
  constexpr int kPieces = D * (FP8 ? 1 : 2) / 16;  // 16-byte pieces per head
  constexpr int kPairs = FP8 ? 8 : 4;              // channel pairs per piece
  constexpr int kLoads = 8;                        // in flight per lane
  __shared__ P2 s_hi[kSplit > 1 ? kSplit : 1][kPairs][32];
  __shared__ P2 s_lo[kSplit > 1 ? kSplit : 1][kPairs][32];
  ptx::grid_dependency_wait();
  ptx::grid_launch_dependents();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int block = 1 << p.log2_block_size;
  const int pieces = p.num_kv_heads * kPieces;  // of a token's row
  const int columns = (pieces + 31) / 32;
  const int64_t tok = (int64_t)blockIdx.x * tokens_per_cta + lane;
  int slot = -1;
  if (lane < tokens_per_cta && tok < p.num_tokens) slot = p.slot_mapping[tok];
  const bool last = slot >= 0 && slot < p.num_slots && (slot & (block - 1)) == block - 1;
  const unsigned hits = __ballot_sync(0xffffffffu, last);  // the same in every warp
  const int work = __popc(hits) * columns;
  // (blockIdx.y: CTAs that share these tokens' columns)
  constexpr int kUnits = kSumWarps / kSplit;  // columns a CTA takes at a time
  for (int w = blockIdx.y * kUnits + warp / kSplit; w < work; w += gridDim.y * kUnits) {
    const int hit = w / columns, piece = (w - hit * columns) * 32 + lane;
    unsigned left = hits;
    for (int i = 0; i < hit; ++i) left &= left - 1;
    const int64_t blk = __shfl_sync(0xffffffffu, slot, __ffs(left) - 1) >> p.log2_block_size;
    const int part = kSplit > 1 ? warp : 0;  // this warp's tokens: part, part + kSplit, ...
    P2 hi[kPairs], lo[kPairs];
    const bool in = piece < pieces;
    const uint4* base =
        static_cast<const uint4*>(p.k_cache) + blk * block * pieces + (in ? piece : 0);
    bool first = true;
    for (int t0 = part; t0 < block; t0 += kLoads * kSplit) {
      uint4 v[kLoads];
#pragma unroll
      for (int i = 0; i < kLoads; ++i)  // (those past the block's end are not looked at below)
        if (i == 0 || t0 + i * kSplit < block) v[i] = base[(int64_t)(t0 + i * kSplit) * pieces];
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        if (i > 0 && t0 + i * kSplit >= block) break;  // uniform
        P2 x[kPairs];
        if constexpr (FP8) {
          const uint32_t c[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            uint32_t h2;
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n"
                : "=r"(h2)
                : "h"((uint16_t)(c[k / 2] >> (16 * (k % 2)))));
            x[k] = *reinterpret_cast<P2*>(&h2);
          }
        } else {
          *reinterpret_cast<uint4*>(x) = v[i];
        }
#pragma unroll
        for (int k = 0; k < kPairs; ++k) {
          hi[k] = first ? x[k] : __hmax2(hi[k], x[k]);
          lo[k] = first ? x[k] : __hmin2(lo[k], x[k]);
        }
        first = false;
      }
    }
    if constexpr (kSplit > 1) {  // blocks of kSplit tokens and more: every warp has some
#pragma unroll
      for (int k = 0; k < kPairs; ++k) {
        s_hi[part][k][lane] = hi[k];
        s_lo[part][k][lane] = lo[k];
      }
      __syncthreads();
      if (part == 0) {
#pragma unroll
        for (int k = 0; k < kPairs; ++k)
#pragma unroll
          for (int j = 1; j < kSplit; ++j) {
            hi[k] = __hmax2(hi[k], s_hi[j][k][lane]);
            lo[k] = __hmin2(lo[k], s_lo[j][k][lane]);
          }
      }
    }
    if (part == 0) {
      float h[2 * kPairs], l[2 * kPairs], amax = 0.f;
#pragma unroll
      for (int k = 0; k < kPairs; ++k) {
        const float2 a = Pair<FP8>::f(hi[k]), b = Pair<FP8>::f(lo[k]);
        h[2 * k] = a.x;
        h[2 * k + 1] = a.y;
        l[2 * k] = b.x;
        l[2 * k + 1] = b.y;
      }
#pragma unroll
      for (int k = 0; k < 2 * kPairs; ++k) {
        // a channel without a number counts as 0
        h[k] = h[k] == h[k] ? fminf(fmaxf(h[k], -kClamp), kClamp) : 0.f;
        l[k] = l[k] == l[k] ? fminf(fmaxf(l[k], -kClamp), kClamp) : 0.f;
        amax = fmaxf(amax, fmaxf(fabsf(h[k]), fabsf(l[k])));
      }
#pragma unroll
      for (int o = 1; o < kPieces; o *= 2)  // over the head's pieces
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      const int e = exponent_for(amax);
      const float inv = exp2i(-e);
      uint32_t ch[kPairs / 2], cl[kPairs / 2];
#pragma unroll
      for (int k = 0; k < kPairs / 2; ++k) {
        ch[k] = cl[k] = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // (the products too are rounded outward: exact but below the smallest
          // float, where a tiny key beside a huge one would become 0)
          ch[k] |= ((uint32_t)__float2int_ru(__fmul_ru(h[4 * k + i], inv)) & 255u) << (8 * i);
          cl[k] |= ((uint32_t)__float2int_rd(__fmul_rd(l[4 * k + i], inv)) & 255u) << (8 * i);
        }
      }
      if (in) {
        const int head = piece / kPieces, c0 = (piece % kPieces) * 2 * kPairs;
        int8_t* row = p.codes + (blk * p.num_kv_heads + head) * 2 * D + c0;
        if constexpr (FP8) {
          *reinterpret_cast<uint4*>(row) = make_uint4(ch[0], ch[1], ch[2], ch[3]);
          *reinterpret_cast<uint4*>(row + D) = make_uint4(cl[0], cl[1], cl[2], cl[3]);
        } else {
          *reinterpret_cast<uint2*>(row) = make_uint2(ch[0], ch[1]);
          *reinterpret_cast<uint2*>(row + D) = make_uint2(cl[0], cl[1]);
        }
        if (piece % kPieces == 0) p.scales[blk * p.num_kv_heads + head] = exp2i(e);
      }
    }
    if constexpr (kSplit > 1) __syncthreads();  // the partial extremes have been read
  }
}

// ---------------------------------------------------------------- select

// Order of floats as unsigned integers.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x);
  return min(b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u), 0xfffffffeu);  // (a NaN's is cut)
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;\n" ::: "memory");
}
// A 32-bit word of another CTA's shared memory.
__device__ __forceinline__ uint32_t load_peer(const void* own, uint32_t rank) {
  uint32_t a, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(a) : "r"(smem_u32(own)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];\n" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// Four codes of a word as two f16 pairs (exact): with the sign bit flipped a
// byte is code + 128, which behind 0x64 reads as the f16 1024 + code + 128.
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  w ^= 0x80808080u;
  const __half2 bias = __half2half2(__ushort_as_half(0x6480));  // 1152
  uint32_t a = __byte_perm(w, 0x64646464u, 0x4140), b = __byte_perm(w, 0x64646464u, 0x4342);
  const __half2 x = __hsub2(*reinterpret_cast<__half2*>(&a), bias);
  const __half2 y = __hsub2(*reinterpret_cast<__half2*>(&b), bias);
  lo = *reinterpret_cast<const uint32_t*>(&x);
  hi = *reinterpret_cast<const uint32_t*>(&y);
}

// The 16-byte pieces of a block row (maxima, then minima) that lane c of a
// quad takes.
template <int D>
__device__ __forceinline__ int piece_of(int c, int i) {
  constexpr int kHalf = D / 64;  // pieces of the maxima per lane
  return (i / kHalf) * (D / 16) + c + 4 * (i % kHalf);
}

// The unit's query heads in 8 bits: per head the codes above zero, then
// those below (zero elsewhere), and the head's power of two.
template <int D, int G>
struct __align__(16) QueryCodes {
  uint32_t word[G][2 * D / 4];
  float u[G];
};

// A warp codes one head, four channels (the registers w) to each of the first
// D / 4 lanes.
template <int D, int G>
__device__ __forceinline__ void code_query(QueryCodes<D, G>& q, int head, int lane, uint2 w) {
  float x[4] = {bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y)}, amax = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = x[i] == x[i] ? fminf(fmaxf(x[i], -kClamp), kClamp) : 0.f;
    amax = fmaxf(amax, fabsf(x[i]));
  }
  amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
  const int e = exponent_for(amax);
  const float inv = exp2i(-e);
  uint32_t pos = 0, neg = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int v = __float2int_rn(x[i] * inv);
    pos |= (uint32_t)max(v, 0) << (8 * i);
    neg |= ((uint32_t)min(v, 0) & 255u) << (8 * i);
  }
  if (lane < D / 4) {
    q.word[head][lane] = pos;
    q.word[head][D / 4 + lane] = neg;
  }
  if (lane == 0) q.u[head] = exp2i(e);
}

// The products of 16 block rows with the unit's query heads.  Lane 4 g + c
// takes its pieces of rows g and g + 8, the maxima in the first half of them
// and the minima in the second, and the same channels of the queries' codes
// above and below zero; sum() leaves in every lane of a quad the largest
// product of rows g and g + 8, scaled by the heads' powers of two.  code is
// row g in shared memory, whose pieces lie at index ^ flip.
//
// G >= 4: f16 MMAs, the heads in the 8 columns (code and query whole numbers
// up to 127, sums below 2^22: exact).  The MMA's k order is free as long as
// both operands share it, so the pieces are operand A as they lie.
template <int D, int G, bool MMA>
struct Scorer {
  static constexpr int kPieces = D / 32;
  uint32_t qb[kPieces][4][2];
  float u0, u1;  // the powers of two of columns 2c and 2c + 1

  __device__ __forceinline__ void take(const QueryCodes<D, G>& q, int g, int c) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      uint4 w = make_uint4(0, 0, 0, 0);
      if (g < G) w = *reinterpret_cast<const uint4*>(&q.word[g][4 * piece_of<D>(c, i)]);
      codes_to_f16(w.x, qb[i][0][0], qb[i][0][1]);
      codes_to_f16(w.y, qb[i][1][0], qb[i][1][1]);
      codes_to_f16(w.z, qb[i][2][0], qb[i][2][1]);
      codes_to_f16(w.w, qb[i][3][0], qb[i][3][1]);
    }
    u0 = q.u[2 * c < G ? 2 * c : 0];
    u1 = q.u[2 * c + 1 < G ? 2 * c + 1 : 0];
  }
  __device__ __forceinline__ void sum(const uint8_t* code, int flip, int c, float (&best)[2]) {
    float part[4][4] = {};  // four chains of MMAs
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const uint8_t* at = code + (piece_of<D>(c, i) ^ flip) * 16;
      const uint4 x = *reinterpret_cast<const uint4*>(at);
      const uint4 y = *reinterpret_cast<const uint4*>(at + 8 * 2 * D);
      const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t a0, a1, a2, a3;
        codes_to_f16(xs[k], a0, a2);
        codes_to_f16(ys[k], a1, a3);
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
            "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};\n"
            : "+f"(part[k][0]), "+f"(part[k][1]), "+f"(part[k][2]), "+f"(part[k][3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(qb[i][k][0]), "r"(qb[i][k][1]));
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float d0 = (part[0][2 * h] + part[1][2 * h]) + (part[2][2 * h] + part[3][2 * h]);
      const float d1 = (part[0][2 * h + 1] + part[1][2 * h + 1]) +
                       (part[2][2 * h + 1] + part[3][2 * h + 1]);
      best[h] = 2 * c < G ? d0 * u0 : -INFINITY;
      if (2 * c + 1 < G) best[h] = fmaxf(best[h], d1 * u1);
      best[h] = fmaxf(best[h], __shfl_xor_sync(0xffffffffu, best[h], 1));
      best[h] = fmaxf(best[h], __shfl_xor_sync(0xffffffffu, best[h], 2));
      best[h] += 0.f;  // -0 counts as 0
    }
  }
};

// G <= 2: 8-bit dot products, 2 D / 16 words a lane, row and head: fewer
// instructions than the MMAs, whose columns would be mostly empty.
template <int D, int G>
struct Scorer<D, G, false> {
  static constexpr int kPieces = D / 32;
  uint32_t qb[G][kPieces][4];
  float u[G];

  __device__ __forceinline__ void take(const QueryCodes<D, G>& q, int, int c) {
#pragma unroll
    for (int h = 0; h < G; ++h) {
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const uint4 w = *reinterpret_cast<const uint4*>(&q.word[h][4 * piece_of<D>(c, i)]);
        qb[h][i][0] = w.x;
        qb[h][i][1] = w.y;
        qb[h][i][2] = w.z;
        qb[h][i][3] = w.w;
      }
      u[h] = q.u[h];
    }
  }
  __device__ __forceinline__ void sum(const uint8_t* code, int flip, int c, float (&best)[2]) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
#pragma unroll
      for (int h = 0; h < G; ++h) {
        int s[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
          const uint4 x = *reinterpret_cast<const uint4*>(code + r * 8 * 2 * D +
                                                          (piece_of<D>(c, i) ^ flip) * 16);
          s[0] = __dp4a((int)x.x, (int)qb[h][i][0], s[0]);
          s[1] = __dp4a((int)x.y, (int)qb[h][i][1], s[1]);
          s[0] = __dp4a((int)x.z, (int)qb[h][i][2], s[0]);
          s[1] = __dp4a((int)x.w, (int)qb[h][i][3], s[1]);
        }
        int t = s[0] + s[1];
        t += __shfl_xor_sync(0xffffffffu, t, 1);
        t += __shfl_xor_sync(0xffffffffu, t, 2);
        const float v = (float)t * u[h];
        best[r] = h ? fmaxf(best[r], v) : v;
      }
    }
  }
};

constexpr int kMaxCluster = 8;  // CTAs that share a unit
constexpr int kHeld = 8;        // keys a lane holds where one warp finds the cut
constexpr int kStages = 2;      // steps of 16 rows in a warp's ring (3 and 4: no faster)

// One cluster of CTAs per (query row, KV head).  Each CTA scores an equal
// run of the candidate blocks and keeps their keys in its shared memory;
// the cut is found by radix selection over the cluster (8 bits a pass, from
// the top bit in which any two keys differ, ending as soon as a pass leaves
// nothing to decide), and each CTA writes its share in rising order.
// Scoring reads 2 D + 4 bytes a block and head, which bounds the large
// calls; the rest of a call is a chain of dependent loads and barriers.
// With many units a CTA is one or two warps and the units in flight on an SM
// hide each other's chains; with few, 8 warps shorten the chain itself.
template <int D, int G, int NT>
__global__ void __launch_bounds__(NT, NT == 32 ? 24 : 1)
    select_kernel(const __grid_constant__ SelectParams p, int clusters) {
  constexpr int kPieces = D / 32;  // 16-byte pieces of a row per lane
  constexpr int kWarps = NT / 32;
  constexpr bool kShared = NT >= 256;  // a cluster may share the unit
  constexpr int kEarly = NT == 32 ? 4 : 1;  // ids per thread loaded before the length is known
  // (a copy whose 32-byte sectors were split in shared memory would fetch them twice)
  extern __shared__ __align__(128) uint8_t s_ring[];
  uint32_t* s_key = reinterpret_cast<uint32_t*>(s_ring + kWarps * kStages * 32 * D);
  __shared__ uint32_t s_hists[kShared ? 2 : 1][256];
  __shared__ uint32_t s_total[kShared ? 256 : 1];
  __shared__ uint32_t s_pub[2];  // what peers read: least key, largest key
  __shared__ uint32_t s_warp[kWarps][4];
  __shared__ uint32_t s_cut[3];
  __shared__ QueryCodes<D, G> s_q;
  auto sync = [] {
    if constexpr (NT == 32)
      __syncwarp();
    else
      __syncthreads();
  };
  ptx::grid_dependency_wait();
  ptx::grid_launch_dependents();
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int g = lane / 4, c = lane % 4;
  const int rank = clusters > 1 ? (int)cluster_rank() : 0;
  const int unit = blockIdx.x / clusters;
  const int row = unit / p.num_kv_heads, kvh = unit - row * p.num_kv_heads;
  const int seq = p.row_seqs ? p.row_seqs[row] : row;
  const int block = 1 << p.log2_block_size;
  int n = p.context_lens[row];
  // loads that do not depend on the length: queries, and the first ids
  constexpr int kHeads = (G + kWarps - 1) / kWarps;  // query heads a warp codes
  uint2 qw[kHeads];
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    const int h = warp + i * kWarps;
    qw[i] = make_uint2(0, 0);
    if (h < G && lane < D / 4)
      qw[i] = *reinterpret_cast<const uint2*>(p.q + ((int64_t)unit * G + h) * D + 4 * lane);
  }
  const bool known = (unsigned)seq < (unsigned)p.num_seqs;
  const int32_t* table = p.block_tables + (known ? (int64_t)seq * p.max_blocks : 0);
  const int first = p.sink;
  int32_t early[kEarly];
  if (clusters == 1 && known) {
#pragma unroll
    for (int i = 0; i < kEarly; ++i) {
      const int64_t j = (int64_t)first + i * NT + tid;
      early[i] = j < p.max_blocks ? table[j] : 0;
    }
  }
  n = max(n, 0);
  int nb = (int)min(((int64_t)n + block - 1) >> p.log2_block_size, (int64_t)p.max_blocks);
  if (!known) nb = 0;
  int32_t* out = p.selected + (int64_t)unit * p.top;
  if (nb <= p.top) {  // every block (the same in all CTAs of the cluster)
    if (rank == 0)
      for (int i = tid; i < p.top; i += NT) out[i] = i < nb ? i : -1;
    return;
  }
  const int cand = nb - p.sink - p.recent;
  const uint32_t want = (uint32_t)(p.top - p.sink - p.recent);  // < cand
  if (rank == 0) {
    for (int i = tid; i < p.sink; i += NT) out[i] = i;
    for (int i = tid; i < p.recent; i += NT) out[p.top - p.recent + i] = nb - p.recent + i;
  }
  if (want == 0) return;

  // this CTA's run of candidates: their block ids, in the words that the
  // keys will take
  const int per = (cand + clusters - 1) / clusters;
  const int j0 = min(rank * per, cand), count = min(per, cand - j0);
  int from = 0;
  if (clusters == 1) {
#pragma unroll
    for (int i = 0; i < kEarly; ++i)
      if (i * NT + tid < count) s_key[i * NT + tid] = (uint32_t)early[i];
    from = kEarly * NT;
  }
  for (int j = from + tid; j < count; j += NT) s_key[j] = (uint32_t)table[first + j0 + j];
#pragma unroll
  for (int i = 0; i < kHeads; ++i)
    if (warp + i * kWarps < G) code_query<D, G>(s_q, warp + i * kWarps, lane, qw[i]);
  sync();  // ids, query codes

  // A warp scores 16 rows a step.  It copies them, kStages - 1 steps ahead,
  // whole rows side by side (a copy instruction asks for full lines), into a
  // ring of its own in shared memory; odd rows' halves are exchanged there so
  // that a quad-wise read finds every bank once.
  constexpr int kRowBytes = 2 * D, kRowLanes = kRowBytes / 16, kRowsPer = 32 / kRowLanes;
  uint32_t kmin = 0xffffffffu, kmax = 0;
  Scorer<D, G, (G >= 4)> scorer;
  uint8_t* const ring = s_ring + warp * kStages * 16 * kRowBytes;
  float su[kStages];         // lane r < 16: row r's scale
  uint32_t inside[kStages];  // bit r: row r's block is in the pool
  constexpr int kStep = 16 * kWarps;
  auto load = [&](int r0, int stage) {
    if (r0 < count) {
      const uint32_t blk = lane < 16 && r0 + lane < count ? s_key[r0 + lane] : 0xffffffffu;
      const bool in = blk < (uint32_t)p.num_blocks;
      inside[stage] = __ballot_sync(0xffffffffu, in);
      // (block, head) pairs number below 2^32: each has 64 bytes of keys or more
      const uint32_t at = in ? blk * (uint32_t)p.num_kv_heads + kvh : 0u;
      if (lane < 16) su[stage] = p.scales[at];
#pragma unroll
      for (int m = 0; m < 16; m += kRowsPer) {
        const int r = m + lane / kRowLanes, piece = lane % kRowLanes;
        const uint32_t a = __shfl_sync(0xffffffffu, at, r);
        cp_async_16(smem_u32(ring + (stage * 16 + r) * kRowBytes + (piece ^ ((r & 1) << 2)) * 16),
                    p.codes + (int64_t)a * kRowBytes + piece * 16, 16);
      }
    }
    cp_async_commit();
  };
  auto score = [&](int r0, int stage) {
    float best[2];
    scorer.sum(ring + (stage * 16 + g) * kRowBytes, (g & 1) << 2, c, best);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int j = r0 + g + 8 * h;
      const float u = __shfl_sync(0xffffffffu, su[stage], g + 8 * h);
      const bool in = inside[stage] >> (g + 8 * h) & 1;
      const uint32_t key = order_key(in ? best[h] * u : -INFINITY);  // outside the pool: last
      if (j < count) {
        kmin = min(kmin, key);
        kmax = max(kmax, key);
        if (c == 0) s_key[j] = key;  // (its id was read a step ago)
      }
    }
  };
#pragma unroll
  for (int k = 0; k < kStages - 1; ++k) load(16 * warp + k * kStep, k);
  scorer.take(s_q, g, c);
  for (int r0 = 16 * warp; r0 < count; r0 += kStages * kStep) {  // uniform in the warp
#pragma unroll
    for (int k = 0; k < kStages; ++k) {
      if (r0 + k * kStep < count) {
        load(r0 + (k + kStages - 1) * kStep, (k + kStages - 1) % kStages);
        cp_async_wait<kStages - 1>();
        __syncwarp();
        score(r0 + k * kStep, k);
        __syncwarp();
      }
    }
  }
  // Few candidates: one warp holds their keys in registers and halves the
  // range in which the cut lies until the keys from `mid` on are as many as
  // wanted (or one value is left, shared by some that are not).
  if (clusters == 1 && count <= 32 * kHeld) {
    sync();
    if (warp > 0) return;
    uint32_t key[kHeld];
    uint32_t low = 0xffffffffu, high = 0;
#pragma unroll
    for (int r = 0; r < kHeld; ++r) {
      // behind the last 0: never counted, mid is above the least key
      const bool in = r * 32 + lane < count;
      key[r] = in ? s_key[r * 32 + lane] : 0u;
      low = min(low, in ? key[r] : 0xffffffffu);
      high = max(high, key[r]);
    }
    low = __reduce_min_sync(0xffffffffu, low);  // more than wanted are >= low
    high = __reduce_max_sync(0xffffffffu, high) + 1;  // fewer are >= high
    uint32_t over = 0;  // keys >= high
    while (high - low > 1) {
      const uint32_t mid = low + (high - low) / 2;
      uint32_t n = 0;
#pragma unroll
      for (int r = 0; r < kHeld; ++r) n += key[r] >= mid;
      n = __reduce_add_sync(0xffffffffu, n);
      if (n > want) {
        low = mid;
      } else {
        high = mid;
        over = n;
        if (n == want) break;
      }
    }
    uint32_t ties = want - over;  // of the keys equal to low, the first ones
    int at = first;
    const uint32_t before = (1u << lane) - 1;
#pragma unroll
    for (int r = 0; r < kHeld; ++r) {
      const uint32_t equal = __ballot_sync(0xffffffffu, r * 32 + lane < count && key[r] == low);
      const bool take = key[r] >= high || ((equal >> lane & 1) && __popc(equal & before) < ties);
      const uint32_t taken = __ballot_sync(0xffffffffu, take);
      if (take) out[at + __popc(taken & before)] = first + r * 32 + lane;
      at += __popc(taken);
      ties -= min(ties, (uint32_t)__popc(equal));
    }
    return;
  }

  kmin = __reduce_min_sync(0xffffffffu, kmin);
  kmax = __reduce_max_sync(0xffffffffu, kmax);
  if constexpr (NT > 32) {
    if (lane == 0) {
      s_warp[warp][0] = kmin;
      s_warp[warp][1] = kmax;
    }
    __syncthreads();
    kmin = __reduce_min_sync(0xffffffffu, s_warp[lane % kWarps][0]);
    kmax = __reduce_max_sync(0xffffffffu, s_warp[lane % kWarps][1]);
  }
  if (kShared && clusters > 1) {
    if (tid == 0) {
      s_pub[0] = kmin;
      s_pub[1] = kmax;
    }
    cluster_sync();
    if (lane < clusters) {
      kmin = load_peer(&s_pub[0], lane);
      kmax = load_peer(&s_pub[1], lane);
    }
    kmin = __reduce_min_sync(0xffffffffu, kmin);
    kmax = __reduce_max_sync(0xffffffffu, kmax);
  }

  // The cut: keys (less the least one) are compared in their top bits
  // `key >> shift`; `prefix` is the cut's, `left` how many of the keys equal
  // to it there are still wanted.
  int shift = 32 - __clz(kmax - kmin);
  uint32_t prefix = 0, left = want, equal = (uint32_t)cand;
  // keys of the cluster's lower ranks above the cut and equal to it, as this
  // thread's bins show them (before any pass all are equal)
  uint32_t lower_gt = 0, lower_eq = tid == 0 ? (uint32_t)j0 : 0u;
  for (int pass = 0; shift > 0 && equal != left; ++pass) {
    // two histograms in turn: peers may still read the last pass's
    uint32_t* s_hist = s_hists[kShared ? pass & 1 : 0];
    const int bits = min(shift, 8);
    for (int i = tid; i < 256; i += NT) s_hist[i] = 0;
    sync();
    const int next = shift - bits;
    for (int i = tid; i < count; i += NT) {
      const uint32_t k = s_key[i] - kmin;
      // (a shift by 32 in two steps)
      if (((k >> (shift - 1)) >> 1) == prefix) atomicAdd(&s_hist[(k >> next) & ((1u << bits) - 1)], 1u);
    }
    const uint32_t* total = s_hist;
    uint32_t lower = 0;  // lower ranks' keys in bin tid
    if (kShared && clusters > 1) {
      cluster_sync();
      if (tid < 256) {
        uint32_t t[kMaxCluster], sum = 0;
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) t[r] = r < clusters ? load_peer(&s_hist[tid], r) : 0u;
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) {
          sum += t[r];
          lower += r < rank ? t[r] : 0u;
        }
        s_total[tid] = sum;
      }
      total = s_total;
      __syncthreads();
    } else {
      sync();
    }
    if (warp == 0) {
      // lane l holds bins 255 - 8 l down to 248 - 8 l
      uint32_t c[8], sum = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        c[i] = total[255 - 8 * lane - i];
        sum += c[i];
      }
      uint32_t above = sum;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, above, o);
        if (lane >= o) above += v;
      }
      above -= sum;  // keys in the lanes before, all larger
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (above < left && above + c[i] >= left) {  // one bin of one lane
          s_cut[0] = 255 - 8 * lane - i;
          s_cut[1] = left - above;
          s_cut[2] = c[i];
        }
        above += c[i];
      }
    }
    sync();
    if (kShared) {
      lower_gt += tid > (int)s_cut[0] ? lower : 0u;
      lower_eq = tid == (int)s_cut[0] ? lower : 0u;
    }
    prefix = (prefix << bits) | s_cut[0];
    left = s_cut[1];
    equal = s_cut[2];
    shift = next;
    // (the next pass writes s_cut only after two more barriers)
  }
  // nothing of a peer's memory is read from here on; no CTA leaves before all
  // have come here
  if (kShared && clusters > 1) asm volatile("barrier.cluster.arrive.aligned;\n" ::: "memory");

  // write: keys above the cut, and the first `left` of those equal to it;
  // each thread owns a run of the CTA's keys
  const int run = (count + NT - 1) / NT | 1;  // odd: threads' words in different banks
  const int i0 = min(tid * run, count), i1 = min(i0 + run, count);
  uint32_t gt = 0, eq = 0;
  for (int i = i0; i < i1; ++i) {
    const uint32_t k = shift ? ((s_key[i] - kmin) >> (shift - 1)) >> 1 : s_key[i] - kmin;
    gt += k > prefix;
    eq += k == prefix;
  }
  uint32_t a = gt, b = eq;  // inclusive sums over the warp, then the CTA
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const uint32_t v = __shfl_up_sync(0xffffffffu, a, o), w = __shfl_up_sync(0xffffffffu, b, o);
    if (lane >= o) {
      a += v;
      b += w;
    }
  }
  if (kShared) {
    lower_gt = __reduce_add_sync(0xffffffffu, lower_gt);
    lower_eq = __reduce_add_sync(0xffffffffu, lower_eq);
  }
  sync();  // s_warp's extremes have been read
  if (lane == 31) {
    s_warp[warp][0] = a;
    s_warp[warp][1] = b;
    s_warp[warp][2] = lower_gt;
    s_warp[warp][3] = lower_eq;
  }
  sync();
  a -= gt;
  b -= eq;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) {
      a += s_warp[w][0];
      b += s_warp[w][1];
    }
    if (kShared && clusters > 1) {
      a += s_warp[w][2];
      b += s_warp[w][3];
    }
  }
  for (int i = i0; i < i1; ++i) {
    const uint32_t k = shift ? ((s_key[i] - kmin) >> (shift - 1)) >> 1 : s_key[i] - kmin;
    const bool is_eq = k == prefix;
    if (k > prefix || (is_eq && b < left)) out[first + a + min(b, left)] = first + j0 + i;
    a += k > prefix;
    b += is_eq;
  }
  if (kShared && clusters > 1) asm volatile("barrier.cluster.wait.aligned;\n" ::: "memory");
}

template <int D, int G, int NT>
cudaError_t launch_select_nt(const SelectParams& p, int c, cudaStream_t stream) {
  // the warps' rings, then a word for each candidate
  const size_t smem = (size_t)NT / 32 * kStages * 32 * D +
                      (size_t)((p.max_blocks + c - 1) / c) * sizeof(uint32_t);
  const int64_t units = (int64_t)p.num_rows * p.num_kv_heads;
  const cudaError_t e = allow_large<select_kernel<D, G, NT>>();
  if (e != cudaSuccess) return e;
  return launch_dependent<select_kernel<D, G, NT>>(dim3((unsigned)(units * c)), dim3(NT), smem,
                                                   stream, c, p, c);
}

// CTAs per unit and threads per CTA (us at 128 channels, 16-token blocks):
//  - few units share theirs among up to 8 CTAs while that leaves each 100
//    blocks and one to an SM, or 256 blocks and two to an SM: 16 units of 4000
//    blocks 33.1 alone, 11.3 by 8; 16 of 500 7.7, 6.5 by 4; 64 of 2000 18.9,
//    12.1 by 4, 18.4 by 8; 128 of 500 8.2, 9.1 by 2;
//  - a unit's chain of waits is shortest with 8 warps, while all fit: 256
//    units of 180 blocks 6.6 with 256 threads, 7.0 with 128; 512 of 180 10.8
//    and 8.6; 1024 of 180 19.6, 13.3, and 12.7 with 64;
//  - with more than 8 to an SM and few query heads a warp each is best, as
//    long as many keep their keys on an SM: 8192 units of 180 blocks, one
//    query head, 63.0 with 64 threads, 56.6 with 32 (four query heads, 2048
//    units: 23.3 and 27.6).
template <int D, int G>
cudaError_t launch_select(const SelectParams& p, int num_sms, cudaStream_t stream) {
  const int64_t units = (int64_t)p.num_rows * p.num_kv_heads;
  int c = 1;
  while (c < kMaxCluster && units * 2 * c <= 2 * num_sms &&
         p.max_blocks / (2 * c) >= (units * 2 * c <= num_sms ? 100 : 256))
    c *= 2;
  while (c < kMaxCluster && p.max_blocks > c * (kSelectMaxBlocks / kMaxCluster)) c *= 2;
  if (c > 1 || units <= 2 * num_sms) return launch_select_nt<D, G, 256>(p, c, stream);
  if (units <= 4 * num_sms || p.max_blocks > 4096) return launch_select_nt<D, G, 128>(p, c, stream);
  if constexpr (G <= 2)
    if (units > 8 * num_sms && p.max_blocks <= 1024) return launch_select_nt<D, G, 32>(p, c, stream);
  return launch_select_nt<D, G, 64>(p, c, stream);
}

template <int D>
cudaError_t launch_select_d(const SelectParams& p, int group, int num_sms, cudaStream_t stream) {
  switch (group) {
    case 1: return launch_select<D, 1>(p, num_sms, stream);
    case 2: return launch_select<D, 2>(p, num_sms, stream);
    case 4: return launch_select<D, 4>(p, num_sms, stream);
    case 8: return launch_select<D, 8>(p, num_sms, stream);
  }
  return cudaErrorInvalidValue;
}

template <int D, bool FP8>
cudaError_t launch_summarize(const SummaryParams& p, cudaStream_t stream) {
  const int columns = (p.num_kv_heads * D * (FP8 ? 1 : 2) / 16 + 31) / 32;
  const int block = 1 << p.log2_block_size;
  // A short step's tokens are their sequences' newest, any of which may end
  // a block, so a CTA looks at one; a long one's come in runs, with one full
  // block among block_size tokens, so a CTA looks at 32.
  const int per = p.num_tokens <= 1024 ? 1 : 32;
  const unsigned groups = (unsigned)((p.num_tokens + per - 1) / per);
  const dim3 b(32 * kSumWarps);
  if (block < 64) {
    // (a grid's y ends at 65535; CTAs stride over what is left)
    const int y = (columns * (per == 1 ? 1 : (32 + block - 1) / block) + kSumWarps - 1) / kSumWarps;
    const dim3 grid(groups, (unsigned)(y < 65535 ? y : 65535));
    return launch_dependent<summarize_kernel<D, FP8, 1>>(grid, b, 0, stream, 1, p, per);
  }
  return launch_dependent<summarize_kernel<D, FP8, 8>>(dim3(groups, (unsigned)columns), b, 0,
                                                       stream, 1, p, per);
}

}  // namespace

cudaError_t launch_summarize_blocks(const SummaryParams& p, int head_dim, bool fp8,
                                    cudaStream_t stream) {
  if (head_dim == 128)
    return fp8 ? launch_summarize<128, true>(p, stream) : launch_summarize<128, false>(p, stream);
  return fp8 ? launch_summarize<64, true>(p, stream) : launch_summarize<64, false>(p, stream);
}

cudaError_t launch_select_blocks(const SelectParams& p, int head_dim, int group, int num_sms,
                                 cudaStream_t stream) {
  return head_dim == 128 ? launch_select_d<128>(p, group, num_sms, stream)
                         : launch_select_d<64>(p, group, num_sms, stream);
}

}  // namespace pa
