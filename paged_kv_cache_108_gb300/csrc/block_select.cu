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

constexpr int kSumThreads = 256;
constexpr int kSumWarps = kSumThreads / 32;

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

// Bound: the keys' bytes, read once.  A CTA looks at up to 32 consecutive
// tokens of the step and summarises the blocks whose last slot is among
// them.  A warp reads 32 consecutive 16-byte pieces of a token's row (512
// bytes, whole heads) and walks every 8th token with up to 8 loads in
// flight; the extremes stay packed in the cache's own precision, where they
// are exact, and the warps' results meet in shared memory.
template <int D, bool FP8>
__global__ void __launch_bounds__(kSumThreads)
    summarize_kernel(const __grid_constant__ SummaryParams p, int tokens_per_cta) {
  using P2 = typename Pair<FP8>::T;
  constexpr int kPieces = D * (FP8 ? 1 : 2) / 16;  // 16-byte pieces per head
  constexpr int kPairs = FP8 ? 8 : 4;              // channel pairs per piece
  __shared__ P2 s_hi[kSumWarps][kPairs][32], s_lo[kSumWarps][kPairs][32];
  ptx::grid_dependency_wait();
  ptx::grid_launch_dependents();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int block = 1 << p.log2_block_size;
  const int pieces = p.num_kv_heads * kPieces;  // of a token's row
  const int piece = blockIdx.y * 32 + lane;
  const int64_t tok = (int64_t)blockIdx.x * tokens_per_cta + lane;
  int slot = -1;
  if (lane < tokens_per_cta && tok < p.num_tokens) slot = p.slot_mapping[tok];
  const bool last = slot >= 0 && slot < p.num_slots && (slot & (block - 1)) == block - 1;
  unsigned hits = __ballot_sync(0xffffffffu, last);
  while (hits) {  // the same blocks in every warp
    const int src = __ffs(hits) - 1;
    hits &= hits - 1;
    const int64_t blk = __shfl_sync(0xffffffffu, slot, src) >> p.log2_block_size;
    if (piece < pieces) {
      const uint4* base = static_cast<const uint4*>(p.k_cache) + blk * block * pieces + piece;
      P2 hi[kPairs], lo[kPairs];
      bool first = true;
      for (int t0 = warp; t0 < block; t0 += 8 * kSumWarps) {
        uint4 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          // past the end the warp's first token again: no effect on extremes
          const int t = t0 + i * kSumWarps;
          v[i] = base[(int64_t)(t < block ? t : t0) * pieces];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          P2 x[kPairs];
          if constexpr (FP8) {
            const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              uint32_t h2;
              asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n"
                  : "=r"(h2)
                  : "h"((uint16_t)(w[k / 2] >> (16 * (k % 2)))));
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
      if (warp < block) {
#pragma unroll
        for (int k = 0; k < kPairs; ++k) {
          s_hi[warp][k][lane] = hi[k];
          s_lo[warp][k][lane] = lo[k];
        }
      }
    }
    __syncthreads();
    if (warp == 0) {
      float h[2 * kPairs], l[2 * kPairs], amax = 0.f;
      const int n = block < kSumWarps ? block : kSumWarps;
#pragma unroll
      for (int k = 0; k < kPairs; ++k) {
        P2 a = s_hi[0][k][lane], b = s_lo[0][k][lane];
        for (int w = 1; w < n; ++w) {
          a = __hmax2(a, s_hi[w][k][lane]);
          b = __hmin2(b, s_lo[w][k][lane]);
        }
        const float2 fa = Pair<FP8>::f(a), fb = Pair<FP8>::f(b);
        h[2 * k] = fa.x;
        h[2 * k + 1] = fa.y;
        l[2 * k] = fb.x;
        l[2 * k + 1] = fb.y;
      }
#pragma unroll
      for (int k = 0; k < 2 * kPairs; ++k) {
        // a channel without a number counts as 0
        h[k] = h[k] == h[k] ? fminf(fmaxf(h[k], -kClamp), kClamp) : 0.f;
        l[k] = l[k] == l[k] ? fminf(fmaxf(l[k], -kClamp), kClamp) : 0.f;
        amax = fmaxf(amax, fmaxf(fabsf(h[k]), fabsf(l[k])));
      }
      if (piece >= pieces) amax = 0.f;
#pragma unroll
      for (int o = 1; o < kPieces; o *= 2) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      if (piece < pieces) {
        const int e = exponent_for(amax);
        const float inv = exp2i(-e);
        uint32_t ch[kPairs / 2], cl[kPairs / 2];
#pragma unroll
        for (int k = 0; k < kPairs / 2; ++k) {
          ch[k] = cl[k] = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            ch[k] |= ((uint32_t)__float2int_ru(h[4 * k + i] * inv) & 255u) << (8 * i);
            cl[k] |= ((uint32_t)__float2int_rd(l[4 * k + i] * inv) & 255u) << (8 * i);
          }
        }
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
    if (hits) __syncthreads();  // warp 0 has read the partial extremes
  }
}

// ---------------------------------------------------------------- select

// Order of floats as unsigned integers.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x);
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
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

// One cluster of CTAs per (query row, KV head).  Each CTA scores an equal
// run of the candidate blocks and keeps their keys in its shared memory;
// the cut is found by radix selection over the cluster (8 bits a pass, from
// the top bit in which any two keys differ, ending as soon as a pass leaves
// nothing to decide), and each CTA writes its share in rising order.
// Scoring reads (2 D + 4) bytes a block and head, which bounds the large
// calls; D / 16 lanes take a block's row, 16 bytes of maxima and 16 of
// minima each, with the queries' codes in registers and __dp4a.
template <int D, int G, int NT>
__global__ void __launch_bounds__(NT)
    select_kernel(const __grid_constant__ SelectParams p, int clusters) {
  constexpr int kLanes = D / 16;       // lanes per block row
  constexpr int kRows = NT / kLanes;   // rows per step of the CTA
  constexpr int kUnroll = 4;
  constexpr int kWarps = NT / 32;
  extern __shared__ uint32_t s_key[];
  __shared__ uint32_t s_q[G][2][D / 4];  // codes above zero, codes below
  __shared__ float s_qu[G];
  __shared__ uint32_t s_hist[256];
  __shared__ uint32_t s_total[256];
  __shared__ uint32_t s_pub[4];  // what peers read: least key, largest key, counts
  __shared__ uint32_t s_warp[kWarps][2];
  __shared__ uint32_t s_cut[3];
  ptx::grid_dependency_wait();
  ptx::grid_launch_dependents();
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int rank = clusters > 1 ? (int)cluster_rank() : 0;
  const int unit = blockIdx.x / clusters;
  const int row = unit / p.num_kv_heads, kvh = unit - row * p.num_kv_heads;
  const int seq = p.row_seqs ? p.row_seqs[row] : row;
  const int block = 1 << p.log2_block_size;
  int n = p.context_lens[row];
  n = max(n, 0);
  int nb = (int)min(((int64_t)n + block - 1) >> p.log2_block_size, (int64_t)p.max_blocks);
  if ((unsigned)seq >= (unsigned)p.num_seqs) nb = 0;
  int32_t* out = p.selected + (int64_t)unit * p.top;
  if (nb <= p.top) {  // every block (the same in all CTAs of the cluster)
    if (rank == 0)
      for (int i = tid; i < p.top; i += NT) out[i] = i < nb ? i : -1;
    return;
  }
  const int32_t* table = p.block_tables + (int64_t)seq * p.max_blocks;
  const int first = p.sink, cand = nb - p.sink - p.recent;
  const uint32_t want = (uint32_t)(p.top - p.sink - p.recent);  // < cand
  if (rank == 0) {
    for (int i = tid; i < p.sink; i += NT) out[i] = i;
    for (int i = tid; i < p.recent; i += NT) out[p.top - p.recent + i] = nb - p.recent + i;
  }
  if (want == 0) return;

  // the queries' codes, one warp per query head
  for (int g = warp; g < G; g += kWarps) {
    const __nv_bfloat16* q = p.q + ((int64_t)(row * p.num_kv_heads + kvh) * G + g) * D;
    float x[4] = {0.f, 0.f, 0.f, 0.f}, amax = 0.f;
    if (lane < D / 4) {
      const uint2 w = *reinterpret_cast<const uint2*>(q + 4 * lane);
      x[0] = bf16_lo(w.x);
      x[1] = bf16_hi(w.x);
      x[2] = bf16_lo(w.y);
      x[3] = bf16_hi(w.y);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = x[i] == x[i] ? fminf(fmaxf(x[i], -kClamp), kClamp) : 0.f;
      amax = fmaxf(amax, fabsf(x[i]));
    }
#pragma unroll
    for (int o = 16; o; o /= 2) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const int e = exponent_for(amax);
    const float inv = exp2i(-e);
    uint32_t pos = 0, neg = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = __float2int_rn(x[i] * inv);
      pos |= ((uint32_t)max(c, 0) & 255u) << (8 * i);
      neg |= ((uint32_t)min(c, 0) & 255u) << (8 * i);
    }
    if (lane < D / 4) {
      s_q[g][0][lane] = pos;
      s_q[g][1][lane] = neg;
    }
    if (lane == 0) s_qu[g] = exp2i(e);
  }
  __syncthreads();
  const int part = lane % kLanes;
  int qp[G][4], qn[G][4];
  float qu[G];
#pragma unroll
  for (int g = 0; g < G; ++g) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      qp[g][i] = (int)s_q[g][0][4 * part + i];
      qn[g][i] = (int)s_q[g][1][4 * part + i];
    }
    qu[g] = s_qu[g];
  }

  // scores of this CTA's run of candidates
  const int per = (cand + clusters - 1) / clusters;
  const int j0 = min(rank * per, cand), count = min(per, cand - j0);
  uint32_t kmin = 0xffffffffu, kmax = 0;
  const int sub = tid / kLanes;
  for (int b0 = 0; b0 < count; b0 += kRows * kUnroll) {  // uniform in the CTA
    int blk[kUnroll];
    uint4 hi[kUnroll], lo[kUnroll];
    float bu[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int j = b0 + u * kRows + sub;
      blk[u] = j < count ? table[first + j0 + j] : -1;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      hi[u] = lo[u] = make_uint4(0, 0, 0, 0);
      bu[u] = -INFINITY;  // a block id outside the pool comes last
      if ((unsigned)blk[u] < (unsigned)p.num_blocks) {
        const int64_t at = (int64_t)blk[u] * p.num_kv_heads + kvh;
        const uint4* r = reinterpret_cast<const uint4*>(p.codes + at * 2 * D);
        hi[u] = r[part];
        lo[u] = r[kLanes + part];
        bu[u] = p.scales[at];
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      float best = -INFINITY;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        int s = __dp4a((int)hi[u].x, qp[g][0], 0);
        s = __dp4a((int)hi[u].y, qp[g][1], s);
        s = __dp4a((int)hi[u].z, qp[g][2], s);
        s = __dp4a((int)hi[u].w, qp[g][3], s);
        s = __dp4a((int)lo[u].x, qn[g][0], s);
        s = __dp4a((int)lo[u].y, qn[g][1], s);
        s = __dp4a((int)lo[u].z, qn[g][2], s);
        s = __dp4a((int)lo[u].w, qn[g][3], s);
#pragma unroll
        for (int o = 1; o < kLanes; o *= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
        best = fmaxf(best, (float)s * qu[g]);
      }
      const int j = b0 + u * kRows + sub;
      const uint32_t key = order_key(bu[u] == -INFINITY ? -INFINITY : best * bu[u]);
      if (j < count) {
        kmin = min(kmin, key);
        kmax = max(kmax, key);
        if (part == 0) s_key[j] = key;
      }
    }
  }
  kmin = __reduce_min_sync(0xffffffffu, kmin);
  kmax = __reduce_max_sync(0xffffffffu, kmax);
  if (lane == 0) {
    s_warp[warp][0] = kmin;
    s_warp[warp][1] = kmax;
  }
  __syncthreads();
  for (int w = 0; w < kWarps; ++w) {
    kmin = min(kmin, s_warp[w][0]);
    kmax = max(kmax, s_warp[w][1]);
  }
  if (clusters > 1) {
    if (tid == 0) {
      s_pub[0] = kmin;
      s_pub[1] = kmax;
    }
    cluster_sync();
    for (int r = 0; r < clusters; ++r) {
      kmin = min(kmin, load_peer(&s_pub[0], r));
      kmax = max(kmax, load_peer(&s_pub[1], r));
    }
  }

  // The cut: keys (less the least one) are compared in their top bits
  // `key >> shift`; `prefix` is the cut's, `left` how many of the keys equal
  // to it there are still wanted.
  int shift = 32 - __clz(kmax - kmin);
  uint32_t prefix = 0, left = want, equal = (uint32_t)cand;
  while (shift > 0 && equal != left) {
    const int bits = min(shift, 8);
    for (int i = tid; i < 256; i += NT) s_hist[i] = 0;
    __syncthreads();
    const int next = shift - bits;
    for (int i = tid; i < count; i += NT) {
      const uint32_t k = s_key[i] - kmin;
      // (a shift by 32 in two steps)
      if (((k >> (shift - 1)) >> 1) == prefix) atomicAdd(&s_hist[(k >> next) & ((1u << bits) - 1)], 1u);
    }
    if (clusters > 1) cluster_sync(); else __syncthreads();
    for (int i = tid; i < 256; i += NT) {
      uint32_t t = s_hist[i];
      if (clusters > 1) {
        t = 0;
        for (int r = 0; r < clusters; ++r) t += load_peer(&s_hist[i], r);
      }
      s_total[i] = t;
    }
    if (clusters > 1) cluster_sync(); else __syncthreads();  // peers have read s_hist
    if (warp == 0) {
      // lane l holds bins 255 - 8 l down to 248 - 8 l
      uint32_t c[8], sum = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        c[i] = s_total[255 - 8 * lane - i];
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
    __syncthreads();
    prefix = (prefix << bits) | s_cut[0];
    left = s_cut[1];
    equal = s_cut[2];
    shift = next;
    // (the next pass writes s_cut only after two more barriers)
  }

  // write: keys above the cut, and the first `left` of those equal to it;
  // each thread owns a run of the CTA's keys
  const int run = (count + NT - 1) / NT;
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
  __syncthreads();  // s_warp's extremes have been read
  if (lane == 31) {
    s_warp[warp][0] = a;
    s_warp[warp][1] = b;
  }
  __syncthreads();
  a -= gt;
  b -= eq;
  uint32_t all_gt = 0, all_eq = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w == warp) {
      a += all_gt;
      b += all_eq;
    }
    all_gt += s_warp[w][0];
    all_eq += s_warp[w][1];
  }
  if (clusters > 1) {
    if (tid == 0) {
      s_pub[2] = all_gt;
      s_pub[3] = all_eq;
    }
    cluster_sync();
    for (int r = 0; r < rank; ++r) {
      a += load_peer(&s_pub[2], r);
      b += load_peer(&s_pub[3], r);
    }
  }
  for (int i = i0; i < i1; ++i) {
    const uint32_t k = shift ? ((s_key[i] - kmin) >> (shift - 1)) >> 1 : s_key[i] - kmin;
    const bool is_eq = k == prefix;
    if (k > prefix || (is_eq && b < left)) out[first + a + min(b, left)] = first + j0 + i;
    a += k > prefix;
    b += is_eq;
  }
  if (clusters > 1) cluster_sync();  // no CTA leaves while a peer may read its memory
}

template <int D, int G>
cudaError_t launch_select(const SelectParams& p, int num_sms, cudaStream_t stream) {
  constexpr int NT = 256;
  const int64_t units = (int64_t)p.num_rows * p.num_kv_heads;
  int c = 1;
  while (c < 8 && units * c < num_sms && p.max_blocks / (2 * c) >= 64) c *= 2;
  while (c < 8 && p.max_blocks > c * 32768) c *= 2;
  const size_t smem = (size_t)((p.max_blocks + c - 1) / c) * sizeof(uint32_t);
  return launch_dependent(select_kernel<D, G, NT>, dim3((unsigned)(units * c)), dim3(NT), smem,
                          stream, c, p, c);
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

}  // namespace

cudaError_t launch_summarize_blocks(const SummaryParams& p, int head_dim, bool fp8,
                                    cudaStream_t stream) {
  const int pieces = p.num_kv_heads * head_dim * (fp8 ? 1 : 2) / 16;
  // A short step's tokens are their sequences' newest, so a CTA looks at one;
  // a long one's come in runs, with one full block in block_size tokens.
  const int block = 1 << p.log2_block_size;
  const int per = p.num_tokens <= 512 ? 1 : (block < 16 ? 16 : (block > 32 ? 32 : block));
  const dim3 grid((unsigned)((p.num_tokens + per - 1) / per), (unsigned)((pieces + 31) / 32));
  auto kernel = head_dim == 128
                    ? (fp8 ? summarize_kernel<128, true> : summarize_kernel<128, false>)
                    : (fp8 ? summarize_kernel<64, true> : summarize_kernel<64, false>);
  return launch_dependent(kernel, grid, dim3(kSumThreads), 0, stream, 1, p, per);
}

cudaError_t launch_select_blocks(const SelectParams& p, int head_dim, int group, int num_sms,
                                 cudaStream_t stream) {
  return head_dim == 128 ? launch_select_d<128>(p, group, num_sms, stream)
                         : launch_select_d<64>(p, group, num_sms, stream);
}

}  // namespace pa
