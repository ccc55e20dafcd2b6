// Prompt attention with changed scores on the 5th-generation tensor cores,
// for a bf16 or e4m3 cache with head_dim 128: the tiles of pa_varlen_scored.
//
// Request r's new tokens are q[qsl[r] .. qsl[r+1]), the last T of its context;
// the token at position i sees keys below i + 1, or below the request's prefix
// if i is inside it, and of those the last `window` up to its own position:
//   s = scale q . k;  s <- cap tanh(s / cap);  s <- s - slope |i - j|
//   out = softmax(s) V.
//
// Bound: each tile's chain of products and softmax; two tiles are all that
// tensor memory holds.  A chunk of 128 keys takes a tile 5200 clocks (capped
// bf16): 1370 of waiting for its two products (1024 on the tensor cores), 2950 of
// softmax, the rest of an item's epilogue (650 a chunk, with 6 chunks an item).
// The tensor cores are busy 0.4 of it, issue slots a third.
//
// A work item is a pair of neighbouring query tiles of one request and KV head:
// 2 x 128 rows, row = token * G + query head in the group.  Both tiles use
// each K and V chunk of 128 keys while it is in shared memory, and alternate on
// the tensor cores: while one tile's softmax runs, the other's products do.
//   S_t = Q_t K^T     M = 128 rows, N = 128 keys, K = 128, into tensor memory
//   P_t               two threads a row, 64 logits each, 32 at a time: changed,
//                     masked, exponentiated; 16-bit weights back over them
//   O_t += P_t V      A = P_t from tensor memory, B = V's rows, MN-major
// Tensor memory is full: S_0, S_1 (P over them), O_0, O_1 of 128 columns.
// (One thread a row, 8 softmax warps in place of 16: 136 us for four capped
// prompts of up to 2048 tokens, where that took 121.  Halves with products of
// their own, N = 64, under 16 warps: 131.)  The two halves of a row agree on its
// largest logit, and add up its sum, through shared memory.
// Capped logits without a bias need no running max over a bf16 cache: they lie
// within the cap, and for a cap up to 55 weights from 2^-80 to 2^80 leave bf16
// and the fp32 sums room for values and counts (2^127 = 2^80 2^17 keys 2^30 of a
// value).  Elsewhere O is rescaled only when a row's running max grows by more
// than 2^8; all lanes of the row's warps take part (by 1), as tensor memory
// accesses are a warp's.
//
// The cap.  tanh(u) for |u| <= 3/4 is an odd polynomial of degree 7 (fitted to
// the smallest largest error over that range: 3.6e-6, which a cap of 50 makes
// 1.8e-4 of a weight, a tenth of its 16-bit rounding), five FMAs a logit; a half
// chunk with a larger |u| in one of the warp's rows takes 1 - 2 / (1 + e^2u), one
// exponential and one reciprocal.  Both are off by a fixed share of the cap: above
// a cap of 64 each score is capped by itself, to within 2^-20 of the score.
//
// An e4m3 cache: two warps widen each chunk to f16 (exact) in shared memory;
// q, scaled by a power of two a row that puts its largest |q| in [1, 2), is
// rounded to f16 in place by the row's threads (11 bits for bf16's 8: exact down
// to 2^-14 of the row's largest); weights are f16, raised by 2^7.
//
// Keys that no token of the item sees (behind the last, before a window, in part
// not loaded) and their values are zeroed in shared memory, so that nothing they
// hold reaches a sum or chooses a formula for the cap; logits are masked by a
// select.
//
// Roles (640 threads): warps 0-7 and 8-15 softmax and epilogue of tile 0 and 1,
// four warps a half of the columns; warp 16 loads (q, K, V) and hands out items;
// warp 17 issues the MMAs; warps 18-19 widen or zero.  (Two more warps would leave
// 80 registers a thread, and spills.)  Every wait is bounded: error word 0, the
// CTA gives up.
//
// Work split: the chunks of all items of a head in a row, K in all, are cut
// into equal ranges, each taken by H_kv neighbouring CTAs, one a head (ragged
// chunks of 168 items on 152 SMs, an item a CTA: 134 us, half the SMs idle in
// the second round).  An item's chunks are visited from its last keys to its
// first: a bias by distance has its largest weights there, and the running max
// hardly grows.  A CTA's range splits at most two items: their sums go to the
// workspace in fp32, and the CTA that holds an item's end (its first keys) adds
// them up once its own range is done and the others' flags, tagged with the
// call, are up; those are CTAs before it, which have all been started.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "launch.cuh"
#include "mma_ptx.cuh"
#include "pa_device.cuh"
#include "pa_kernels.cuh"
#include "tc_ptx.cuh"
#include "tc_sched.cuh"

namespace pa {
namespace ps {

using tc::Smem;
using tc::drain_bar;

constexpr int D = 128, CHK = 128;       // keys per chunk
constexpr int kMaxReqs = 256;
constexpr int HALF_B = 128 * 128;       // 128 rows of 64 16-bit columns
constexpr int TILE_B = 2 * HALF_B;      // a q tile, a K or V chunk in 16 bits
constexpr int RAW_B = CHK * D;          // a K or V chunk in e4m3
constexpr int NTHREADS = 640;
constexpr int PROD_WARP = 16, MMA_WARP = 17, FIX_WARP = 18;
constexpr int NITEM = 4;                // items published ahead
// Of an item, in chunks, when CTAs' shares are made equal.  (Four capped prompts
// with 1 and 2: 116.5, 115.5 us; 512 new tokens behind 8 K 75.8, 78.4.)
constexpr int kItemCost = 1;
// Units of a CTA at least, where there are few: parts cost their joining.  (64
// tokens at the end of 1000 with 1, 2, 3 and 4: 25.4, 22.6, 23.2, 22.6 us; 20 of
// 300 16.2, 15.2, 13.8, 13.8.)
constexpr int kMinUnits = 2;
constexpr int NFIX = 4;                 // zeroed chunks ahead of their MMA, at most
constexpr int S_COL = 0, O_COL = 256;   // tile t: + 128 t; logits of the h-th half: + 64 h
constexpr float kRescaleLog2 = 8.f;
constexpr float kBoundedLog2 = 80.f;    // caps up to this need no running max

constexpr int kItemBytes = 80;
// Sums of an item's 2 x 128 rows: [tile][column / 4][row] float4, then
// [tile][row] (max, sum)
constexpr int kPartWords = 2 * 128 * (D + 2);

template <bool FP8>
struct Cfg {
  static constexpr int NST = FP8 ? 3 : 4;   // 16-bit chunks in shared memory
  static constexpr int NRAW = FP8 ? 3 : 0;  // e4m3 chunks
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_ST = OFF_Q + 2 * TILE_B;
  static constexpr int OFF_RAW = OFF_ST + NST * TILE_B;
  static constexpr int OFF_X = OFF_RAW + NRAW * RAW_B;  // [2 uses][tile][half][row] words exchanged
  static constexpr int OFF_BAR = OFF_X + 2 * 2 * 2 * 128 * 4;
  static constexpr int NLOAD = FP8 ? NRAW : NST;  // stages that TMA fills
  static constexpr int B_Q_FULL = 0, B_Q_EMPTY = 1, B_Q_READY = 2 /* [2] */, B_FULL = 4,
                       B_EMPTY = B_FULL + NLOAD, B_WIDE = B_EMPTY + NLOAD,
                       B_WIDE_EMPTY = B_WIDE + NST, B_FIX = B_WIDE_EMPTY + NST,
                       B_S_FULL = B_FIX + NFIX, B_P_FULL = B_S_FULL + 2, B_O_FULL = B_P_FULL + 2,
                       B_O_EMPTY = B_O_FULL + 2, B_X = B_O_EMPTY + 2, B_ITEM_FULL = B_X + 2,
                       B_ITEM_EMPTY = B_ITEM_FULL + NITEM, B_PART = B_ITEM_EMPTY + NITEM,
                       B_MERGE = B_PART + 1, NBARS = B_MERGE + 1;
  static constexpr int OFF_TMEM = OFF_BAR + NBARS * 8;
  static constexpr int OFF_ABORT = OFF_TMEM + 4;
  static constexpr int OFF_RING = (OFF_ABORT + 4 + 15) / 16 * 16;
  // pairs of tiles before each request, [R + 1]: 16 bits (prefill_scored_fits)
  static constexpr int OFF_TP = OFF_RING + NITEM * kItemBytes;
  static constexpr int SMEM_BYTES = OFF_TP + (kMaxReqs + 1) * 2 + 1024;  // + alignment slack
  static constexpr float kRaise = FP8 ? 7.f : 0.f;  // log2 of the factor of P and its sum
  static_assert(SMEM_BYTES <= 232448, "shared memory per CTA");
  static_assert(OFF_BAR % 1024 == 0, "tiles stay 1024-byte aligned");
};

struct Params {
  __nv_bfloat16* out;           // [num_tokens, H, D]
  const int32_t* block_tables;  // [R, max_blocks]
  const int32_t* seq_lens;      // [R]
  const int32_t* qsl;           // [R + 1]
  int* err;                     // workspace word 0
  unsigned long long* flags;    // [CTAs][2]: the call's tag once a part is written
  float* parts;                 // [CTAs][2][kPartWords]
  unsigned long long epoch;
  int ranges;                   // CTAs of a head
  int num_seqs, num_tokens, num_heads, num_kv_heads, max_blocks, num_blocks, block_size, log2_bs;
  int box_tok, log2_box;
  float scale_log2;
  const float* k_scale;  // e4m3: device scalars
  const float* v_scale;
  ScoreMod mod;
};

// A wait that the other side usually has ended: the test comes first.
__device__ __forceinline__ bool wait_at(const Smem& sm, uint32_t bar, uint32_t parity, int* err,
                                        int code) {
  return ptx::mbar_try_wait(bar, parity) || tc::wait_bar(sm, bar, parity, err, code);
}
// A stage of a ring and the parity of its use.
template <int N>
struct Stage {
  int s = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next() {
    if (++s == N) {
      s = 0;
      ph ^= 1;
    }
  }
};

// Two lanes of fp32 arithmetic an instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  unsigned long long ra, rb, rc, rd;
  asm("mov.b64 %0, {%1, %2};" : "=l"(ra) : "f"(a.x), "f"(a.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(rb) : "f"(b.x), "f"(b.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(rc) : "f"(c.x), "f"(c.y));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(rd) : "l"(ra), "l"(rb), "l"(rc));
  float2 d;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(rd));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  unsigned long long ra, rb, rd;
  asm("mov.b64 %0, {%1, %2};" : "=l"(ra) : "f"(a.x), "f"(a.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(rb) : "f"(b.x), "f"(b.y));
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(rd) : "l"(ra), "l"(rb));
  float2 d;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(rd));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  unsigned long long ra, rb, rd;
  asm("mov.b64 %0, {%1, %2};" : "=l"(ra) : "f"(a.x), "f"(a.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(rb) : "f"(b.x), "f"(b.y));
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(rd) : "l"(ra), "l"(rb));
  float2 d;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(rd));
  return d;
}
// The largest of three (a NaN is passed over).
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// D[tmem] (+)= A[tmem] * B[smem]^T, kind::f16: a column of A holds two 16-bit
// elements of each row.
__device__ __forceinline__ void mma_from_tmem(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                              uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void store_32(void* to, const uint32_t (&w)[8], bool aligned) {
  if (!aligned) {
    static_cast<uint4*>(to)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    static_cast<uint4*>(to)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    return;
  }
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(to), "r"(w[0]),
               "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// An item, or the part of its chunks that falls to a CTA.
struct __align__(16) Item {
  int r, g;      // request (-1: there are no more items), KV head
  int q0;        // first q row of the pair
  int pos;       // position of its first token
  int ntok[2];   // new tokens of each tile
  int kv_lo, kv_end;  // keys that the pair's tokens see lie in [kv_lo, kv_end)
  int prefix;
  int jl, n;     // the last chunk's keys, count (0: zero rows); chunk c has keys jl - c
  int a[2], b[2];  // chunks of each tile: [a, b)
  int part;      // slot of its sums in the workspace, or -1
  int merge;     // the first of the CTAs that share the item, where this one adds up; or -1
};
static_assert(sizeof(Item) == kItemBytes, "");

template <int G>
__device__ __forceinline__ Item item_of(int pair, int g, const uint16_t* tp, const Params& p) {
  constexpr int MQ = 128 / G;
  Item it;
  it.g = g;
  int lo = 0, hi = p.num_seqs;  // the request of this pair: tp[r] <= pair < tp[r + 1]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (tp[mid] <= pair) lo = mid;
    else hi = mid;
  }
  it.r = lo;
  const int first = __ldg(&p.qsl[lo]), T = __ldg(&p.qsl[lo + 1]) - first;
  const int sl = __ldg(&p.seq_lens[lo]), ctx = sl - T;
  const int tok = (pair - tp[lo]) * 2 * MQ;
  it.q0 = first + tok;
  it.pos = ctx + tok;
  it.prefix = p.mod.prefix_lens ? min(__ldg(&p.mod.prefix_lens[lo]), sl) : 0;
  int end[2], low[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    it.ntok[t] = min(MQ, max(0, T - tok - t * MQ));
    const int p0 = it.pos + t * MQ;
    end[t] = p0 + it.ntok[t];
    if (p0 < it.prefix) end[t] = max(end[t], it.prefix);
    low[t] = p.mod.window > 0 ? max(0, p0 - p.mod.window + 1) : 0;
  }
  it.kv_lo = low[0];
  it.kv_end = it.ntok[1] ? max(end[0], end[1]) : end[0];
  const bool none = ctx < 0 || it.kv_end > (p.max_blocks << p.log2_bs);
  it.jl = (it.kv_end + CHK - 1) / CHK - 1;
  it.n = none ? 0 : it.jl + 1 - it.kv_lo / CHK;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const bool some = it.ntok[t] > 0 && !none;
    it.a[t] = some ? it.jl - (end[t] - 1) / CHK : 0;
    it.b[t] = some ? it.jl + 1 - low[t] / CHK : 0;
  }
  it.part = it.merge = -1;
  return it;
}
// Its chunks [from, to) alone.
__device__ __forceinline__ void restrict_to(Item& it, int from, int to) {
  it.jl -= from;
  it.n = to - from;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    it.a[t] = min(max(it.a[t] - from, 0), it.n);
    it.b[t] = min(max(it.b[t] - from, 0), it.n);
  }
}
// Whether a chunk holds keys that no token of the item sees.
__device__ __forceinline__ bool ragged(const Item& it, int c) {
  const int key0 = (it.jl - c) * CHK;
  return key0 < it.kv_lo || key0 + CHK > it.kv_end;
}

// cap tanh(s rs / cap) + bias in log2 units for |s rs| <= 3/4 cap, the cap's
// and the scale's factors being in the coefficients.
__device__ __forceinline__ float2 capped_poly(float2 s, const float (&k)[4], float2 bias) {
  const float2 z = mul2(s, s);
  float2 f = fma2(both(k[3]), z, both(k[2]));
  f = fma2(f, z, both(k[1]));
  f = fma2(f, z, both(k[0]));
  return fma2(f, s, bias);
}
// Without a bias, adding s^4 to `fourth`.
__device__ __forceinline__ float2 capped_poly_sum(float2 s, const float (&k)[4], float2& fourth) {
  const float2 z = mul2(s, s);
  fourth = fma2(z, z, fourth);
  float2 f = fma2(both(k[3]), z, both(k[2]));
  f = fma2(f, z, both(k[1]));
  f = fma2(f, z, both(k[0]));
  return mul2(f, s);
}

// LARGE: a cap above 64.  (A kernel of its own: with the branch in one, ragged
// e4m3 chunks under a cap of 30 took 78.3 us, where this takes 75.3.)
template <int G, bool FP8, bool LARGE>
__global__ void __launch_bounds__(NTHREADS, 1)
    prefill_scored_kernel(const __grid_constant__ CUtensorMap tm_k,
                          const __grid_constant__ CUtensorMap tm_v,
                          const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ Params p) {
  using C = Cfg<FP8>;
  constexpr int MQ = 128 / G;
  constexpr int NST = C::NST, NLOAD = C::NLOAD;
  extern __shared__ unsigned char smem_raw[];
  Smem sm;
  {
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t aligned = (raw + 1023u) & ~1023u;
    sm.base = smem_raw + (aligned - raw);
    sm.base_u32 = aligned;
    sm.off_bar = C::OFF_BAR;
    sm.off_abort = C::OFF_ABORT;
  }
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int R = p.num_seqs;
  uint16_t* tp = reinterpret_cast<uint16_t*>(sm.base + C::OFF_TP);

  ptx::grid_dependency_wait();
  if (warp == MMA_WARP) {
    ptx::tmem_alloc(sm.base_u32 + C::OFF_TMEM, 512);
    ptx::tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < C::NBARS; ++i) {
      uint32_t cnt = 1;
      if (i >= C::B_Q_READY && i < C::B_Q_READY + 2) cnt = 256;
      // a tile's softmax warps
      if ((i >= C::B_P_FULL && i < C::B_P_FULL + 2) || (i >= C::B_O_EMPTY && i < C::B_O_EMPTY + 2) ||
          (i >= C::B_X && i < C::B_X + 2))
        cnt = 8;
      // the MMAs, and the two zeroing warps
      if (!FP8 && i >= C::B_EMPTY && i < C::B_EMPTY + NLOAD) cnt = 3;
      // the two widening or zeroing warps' threads
      if ((FP8 && i >= C::B_EMPTY && i < C::B_EMPTY + NLOAD) ||
          (i >= C::B_WIDE && i < C::B_WIDE + NST) || (i >= C::B_FIX && i < C::B_FIX + NFIX))
        cnt = 64;
      // the softmax warps
      if (i == C::B_PART || i == C::B_MERGE) cnt = 16;
      // an item is read by the MMA thread, 16 softmax warps and those two
      if (i >= C::B_ITEM_EMPTY && i < C::B_ITEM_EMPTY + NITEM) cnt = 19;
      ptx::mbar_init(sm.bar(i), cnt);
    }
    *sm.abort_flag() = 0;
    ptx::fence_mbar_init();
  }
  if (warp == PROD_WARP && lane == 0) {
    ptx::prefetch_tmap(&tm_k);
    ptx::prefetch_tmap(&tm_v);
    ptx::prefetch_tmap(&tm_q);
  }
  for (int r = tid; r < R; r += NTHREADS) {
    const int T = __ldg(&p.qsl[r + 1]) - __ldg(&p.qsl[r]);
    tp[r] = (uint16_t)(T > 0 ? (T + 2 * MQ - 1) / (2 * MQ) : 0);
  }
  __syncthreads();
  if (warp == 0) {  // exclusive prefix
    int carry = 0;
    for (int base = 0; base < R; base += 32) {
      const int i = base + lane, v = i < R ? tp[i] : 0;
      int incl = v;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += o;
      }
      if (i < R) tp[i] = (uint16_t)(carry + incl - v);
      carry += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) tp[R] = (uint16_t)carry;
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sm.base + C::OFF_TMEM);
  // This CTA's head and range of chunks: [lo, hi) of K, from chunk off0 of a pair.
  __shared__ long long s_sum[NTHREADS / 32], s_others[NTHREADS / 32], s_before;
  __shared__ int s_pair, s_last;  // the pairs of its first and last unit
  const int j = blockIdx.x / p.num_kv_heads, g = blockIdx.x - j * p.num_kv_heads;
  const int pairs = tp[R];
  // A pair's chunks, and kItemCost more for what an item takes besides (the
  // first units of a pair; one without keys has its zeros written).
  auto units_of = [&](int pair) -> int { return item_of<G>(pair, g, tp, p).n + kItemCost; };
  long long K = 0, lo = 0, hi = 0;
  int ranges = 1;
  {
    long long others = 0, before = 0;
    for (int x = tid + NTHREADS; x < pairs; x += NTHREADS) others += units_of(x);
    for (int base = 0; base < pairs; base += NTHREADS) {
      const int n = base + tid < pairs ? units_of(base + tid) : 0;
      long long incl = n;
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const long long up = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += up;
      }
      if (base == 0) {
#pragma unroll
        for (int d = 16; d; d /= 2) others += __shfl_xor_sync(0xffffffffu, others, d);
      } else {
        __syncthreads();  // s_sum is free
      }
      if (lane == 31) s_sum[warp] = incl;
      if (base == 0 && lane == 0) s_others[warp] = others;
      if (tid == 0 && base == 0) s_pair = s_last = -1;
      __syncthreads();
      long long start = before + incl - n, end = before;
      for (int w = 0; w < NTHREADS / 32; ++w) {
        if (w < warp) start += s_sum[w];
        end += s_sum[w];
      }
      if (base == 0) {
        K = end;
        for (int w = 0; w < NTHREADS / 32; ++w) K += s_others[w];
        ranges = (int)min((long long)p.ranges, max(1ll, K / kMinUnits));
        if (j < ranges) {
          lo = tc::range_lo(j, K, ranges);
          hi = tc::range_lo(j + 1, K, ranges);
        }
      }
      if (j < ranges && start <= lo && lo < start + n) s_pair = base + tid;
      if (j < ranges && start < hi && hi <= start + n) {
        s_last = base + tid;
        s_before = start;
      }
      __syncthreads();
      if (j >= ranges || s_last >= 0) break;
      before = end;
    }
  }
  Item* items = reinterpret_cast<Item*>(sm.base + C::OFF_RING);
  // the k-th item of this CTA; by a whole warp
  auto read_item = [&](int k) -> Item {
    const int slot = k % NITEM;
    Item it;
    it.r = -1;
    if (wait_at(sm, sm.bar(C::B_ITEM_FULL + slot), (uint32_t)(k / NITEM) & 1, p.err, 60))
      it = items[slot];
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(sm.bar(C::B_ITEM_EMPTY + slot));
    return it;
  };

  if (warp >= PROD_WARP) {
    if (warp == PROD_WARP) {
      // ================= loads =================
      Stage<NLOAD> st;  // K and V chunks in turn
      long long ns = 0;  // those filled
      int nq = 0;        // q pairs
      // from the last pair to the first: what a later CTA waits for is done first,
      // what is joined here last
      const int lowest = hi > lo ? s_pair : 0;
      int pair = hi > lo ? s_last : -1;
      long long u0 = hi > lo ? s_before : 0;  // the pair's first unit
      for (int k = 0;; ++k) {
        const int slot = k % NITEM;
        if (!wait_at(sm, sm.bar(C::B_ITEM_EMPTY + slot), ((uint32_t)(k / NITEM) & 1) ^ 1, p.err, 61))
          break;
        Item it;
        it.r = -1;
        for (bool found = false; pair >= lowest && !found; --pair) {
          it = item_of<G>(pair, g, tp, p);
          const int all = it.n + kItemCost;
          if (pair < s_last) u0 -= all;
          const int off = (int)max(lo - u0, 0ll), upto = (int)min((long long)all, hi - u0);
          const int from = max(off - kItemCost, 0), to = upto - kItemCost;
          found = it.n == 0 || to > from;
          if (it.n == 0) continue;  // zeros
          if (!found) {
            it.r = -1;  // (none of the pair's chunks)
          } else if (from > 0 || to < it.n) {
            if (from > 0 && to == it.n)
              it.merge = tc::cta_of(u0 + kItemCost, K, ranges);
            else
              it.part = from > 0 ? 0 : 1;
            restrict_to(it, from, to);
          }
        }
        if (lane == 0) {
          items[slot] = it;
          ptx::mbar_arrive(sm.bar(C::B_ITEM_FULL + slot));
        }
        if (it.r < 0) break;
        bool ok = true;
        const int q_at = nq > 0 ? 1 : 0;
        for (int x = 0; x < 2 * it.n; ++x) {
          if (x == q_at) {  // the q tiles: behind the first keys, once the last ones are free
            if (nq > 0 && !wait_at(sm, sm.bar(C::B_Q_EMPTY), (nq - 1) & 1, p.err, 62)) {
              ok = false;
              break;
            }
            if (lane == 0) {
              // rows token * G + i: box {64 of d, G heads, MQ tokens} per half;
              // tokens behind the batch read as zeros
              ptx::mbar_arrive_expect_tx(sm.bar(C::B_Q_FULL), 2 * TILE_B);
              for (int t = 0; t < 2; ++t)
                for (int h = 0; h < 2; ++h)
                  ptx::tma_load_3d(sm.base_u32 + C::OFF_Q + t * TILE_B + h * HALF_B, &tm_q,
                                   sm.bar(C::B_Q_FULL), 64 * h, it.g * G, it.q0 + t * MQ);
            }
            ++nq;
          }
          const int s = st.s;
          const int key0 = (it.jl - x / 2) * CHK;
          const int keys = min(CHK, it.kv_end - key0);
          const int nbox = (keys + p.box_tok - 1) >> p.log2_box;
          // blocks that lie before every window are not read
          const int box0 = max(0, it.kv_lo - key0) >> p.log2_box;
          const bool mine = lane >= box0 && lane < nbox;
          int phys = 0;
          if (mine)
            phys = __ldg(&p.block_tables[(int64_t)it.r * p.max_blocks +
                                         ((key0 + lane * p.box_tok) >> p.log2_bs)]);
          if (!wait_at(sm, sm.bar(C::B_EMPTY + s), st.ph ^ 1, p.err, 63)) {
            ok = false;
            break;
          }
          if (mine && (unsigned)phys >= (unsigned)p.num_blocks) {
            atomicExch(p.err, 3);  // bad block id: block 0 instead of a fault
            phys = 0;
          }
          if (lane == 0)
            ptx::mbar_arrive_expect_tx(sm.bar(C::B_FULL + s), (uint32_t)(nbox - box0) * p.box_tok *
                                                                  (uint32_t)(D * (FP8 ? 1 : 2)));
          __syncwarp();
          if (mine) {
            const void* tm = x & 1 ? (const void*)&tm_v : (const void*)&tm_k;
            const uint32_t dst = sm.base_u32 + (FP8 ? C::OFF_RAW + s * RAW_B : C::OFF_ST + s * TILE_B) +
                                 (uint32_t)(lane * p.box_tok) * 128u;
            const int off = (key0 + lane * p.box_tok) & (p.block_size - 1);
            ptx::tma_load_4d(dst, tm, sm.bar(C::B_FULL + s), 0, it.g, off, phys);
            if (!FP8)
              ptx::tma_load_4d(dst + HALF_B, tm, sm.bar(C::B_FULL + s), 64, it.g, off, phys);
          }
          st.next();
          ++ns;
        }
        if (!ok) break;
      }
      // drain: the last loads must have landed before the CTA ends
      __syncwarp();
      if (lane == 0) {
        for (long long l = ns > NLOAD ? ns - NLOAD : 0; l < ns; ++l)
          drain_bar(sm.bar(C::B_FULL + (int)(l % NLOAD)), (uint32_t)(l / NLOAD) & 1);
        if (nq > 0) drain_bar(sm.bar(C::B_Q_FULL), (nq - 1) & 1);
      }
    } else if (warp == MMA_WARP) {
      // ================= MMAs =================
      // The whole warp walks the chunks with values it knows to be the same in all
      // lanes, one lane issues.
      constexpr uint32_t kIdescBf16 = ptx::idesc_bf16_f32_ab(128, 128, false, false);
      constexpr uint32_t kIdescBf16T = ptx::idesc_bf16_f32_ab(128, 128, false, true);
      // f16 operands: format 0 in both fields
      constexpr uint32_t kFormat = (1u << 7) | (1u << 10);
      constexpr uint32_t IDESC_QK = FP8 ? kIdescBf16 & ~kFormat : kIdescBf16;
      constexpr uint32_t IDESC_PV = FP8 ? kIdescBf16T & ~kFormat : kIdescBf16T;
      constexpr int b_staged = FP8 ? C::B_WIDE : C::B_FULL;
      constexpr int b_free = FP8 ? C::B_WIDE_EMPTY : C::B_EMPTY;
      Stage<NST> st;     // of the next chunk: K_0 V_0 K_1 V_1 ... of every item
      long long ns = 0;  // chunks used
      int nq = 0, nfix = 0;
      int np[2] = {0, 0}, ni[2] = {0, 0};  // chunks done, items with some, of each tile
      // descriptors of the first tile or stage: others lie so many 16-byte units on
      const uint32_t base = __reduce_or_sync(0xffffffffu, sm.base_u32);
      const uint32_t tm = __reduce_or_sync(0xffffffffu, tmem);
      const uint64_t q_desc = ptx::smem_desc_sw128(base + C::OFF_Q, 16, 1024);
      const uint64_t k_desc = ptx::smem_desc_sw128(base + C::OFF_ST, 16, 1024);
      const uint64_t v_desc = ptx::smem_desc_sw128(base + C::OFF_ST, HALF_B, 1024);
      const bool leader = ptx::elect_one();
      auto wait = [&](int bar, uint32_t parity, int code) -> bool {
        return __all_sync(0xffffffffu, wait_at(sm, sm.bar(bar), parity, p.err, code)) != 0;
      };
      bool ok = true;
      for (int k = 0; ok; ++k) {
        const int slot = k % NITEM;
        if (!wait(C::B_ITEM_FULL + slot, (uint32_t)(k / NITEM) & 1, 66)) break;
        auto field = [&](const int& x) { return (int)__reduce_or_sync(0xffffffffu, (unsigned)x); };
        const Item& in = items[slot];
        Item it;
        it.r = field(in.r), it.n = field(in.n), it.jl = field(in.jl);
        it.kv_lo = field(in.kv_lo), it.kv_end = field(in.kv_end);
        const int from[2] = {field(in.a[0]), field(in.a[1])}, to[2] = {field(in.b[0]), field(in.b[1])};
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(sm.bar(C::B_ITEM_EMPTY + slot));
        if (it.r < 0) break;
        if (it.n == 0) continue;
        ok = wait(C::B_Q_FULL, nq & 1, 67);
        if (FP8)
          for (int t = 0; t < 2; ++t) ok = ok && wait(C::B_Q_READY + t, nq & 1, 68);
        int v_st = 0;  // the chunk before's values
        for (int c = 0; c <= it.n && ok; ++c) {
          const int pc = c - 1;
          const bool keys = c < it.n, values = c > 0;
          if (values) {
            v_st = st.s;
            ok = wait(b_staged + v_st, st.ph, 64);
            if (!FP8 && ragged(it, pc)) {
              ok = ok && wait(C::B_FIX + nfix % NFIX, (uint32_t)(nfix / NFIX) & 1, 69);
              ++nfix;
            }
            st.next();
          }
          if (keys) {
            ok = ok && wait(b_staged + st.s, st.ph, 65);
            if (!FP8 && ragged(it, c)) {
              ok = ok && wait(C::B_FIX + nfix % NFIX, (uint32_t)(nfix / NFIX) & 1, 69);
              ++nfix;
            }
          }
          if (!ok) break;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const uint32_t s_tm = tm + S_COL + 128 * t, o_tm = tm + O_COL + 128 * t;
            if (pc >= from[t] && pc < to[t]) {  // P V of the chunk before
              if (pc == from[t] && ni[t] > 0) ok = ok && wait(C::B_O_EMPTY + t, (ni[t] - 1) & 1, 70);
              ok = ok && wait(C::B_P_FULL + t, np[t] & 1, 71);
              if (!ok) break;
              ptx::tc_fence_after();
              const uint64_t v = v_desc + (uint32_t)v_st * (TILE_B >> 4);
              const uint32_t add = pc > from[t];
              if (leader) {
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)  // weights lie over the first half of their logits
                  mma_from_tmem(o_tm, s_tm + 64 * (kk >> 2) + 8 * (kk & 3), v + kk * (2048 >> 4),
                                IDESC_PV, kk > 0 ? 1u : add);
                ptx::tc_commit(sm.bar(C::B_O_FULL + t));
              }
              __syncwarp();
              ++np[t];
            }
            if (c >= from[t] && c < to[t]) {  // Q K^T, over the weights just used
              ptx::tc_fence_after();
              const uint64_t q = q_desc + t * (TILE_B >> 4);
              const uint64_t kb = k_desc + (uint32_t)st.s * (TILE_B >> 4);
              if (leader) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                  const int at = (kk >> 2) * (HALF_B >> 4) + (kk & 3) * 2;
                  ptx::tc_mma_f16(s_tm, q + at, kb + at, IDESC_QK, kk > 0);
                }
                ptx::tc_commit(sm.bar(C::B_S_FULL + t));
              }
              __syncwarp();
            }
          }
          if (!ok) break;
          if (leader) {
            if (values) ptx::tc_commit(sm.bar(b_free + v_st));
            if (keys) ptx::tc_commit(sm.bar(b_free + st.s));
            if (c == it.n - 1) ptx::tc_commit(sm.bar(C::B_Q_EMPTY));
          }
          __syncwarp();
          if (keys) st.next();
        }
        if (!ok) break;
        ns += 2 * it.n;
        ++nq;
#pragma unroll
        for (int t = 0; t < 2; ++t) ni[t] += to[t] > from[t];
      }
      // drain: every product and commit issued must have landed before the end
      if (leader) {
        for (int t = 0; t < 2; ++t)
          if (np[t] > 0) drain_bar(sm.bar(C::B_O_FULL + t), (np[t] - 1) & 1);
        if (nq > 0) drain_bar(sm.bar(C::B_Q_EMPTY), (nq - 1) & 1);
        for (long long l = ns > NST ? ns - NST : 0; l < ns; ++l)
          drain_bar(sm.bar(b_free + (int)(l % NST)), (uint32_t)(l / NST) & 1);
      }
      __syncwarp();
    } else {
      // ================= widening (e4m3) and zeroing =================
      const int x = tid - FIX_WARP * 32;
      Stage<NST> st;
      Stage<FP8 ? C::NRAW : 1> raw_st;
      int nfix = 0;
      // e4m3: 16 elements at a time, of rows row0, row0 + 8 ...; 8 lanes take 4
      // pieces of two neighbouring rows, whose stores then fall in different banks
      const int row0 = ((x >> 3) & ~1) | ((x >> 2) & 1), piece = x & 3, side = (x >> 3) & 1;
      const int from = row0 * 128 + (((4 * side + piece) ^ row0) << 4);
      const int to0 = side * HALF_B + row0 * 128 + (((2 * piece) ^ row0) << 4);
      const int to1 = side * HALF_B + row0 * 128 + (((2 * piece + 1) ^ row0) << 4);
      for (int k = 0;; ++k) {
        const Item it = read_item(k);
        if (it.r < 0) break;
        bool ok = true;
        if constexpr (FP8) {
          for (int c = 0; c < 2 * it.n && ok; ++c, raw_st.next(), st.next()) {
            const int s = raw_st.s, w = st.s;
            const int key0 = (it.jl - c / 2) * CHK;
            ok = wait_at(sm, sm.bar(C::B_FULL + s), raw_st.ph, p.err, 72) &&
                 wait_at(sm, sm.bar(C::B_WIDE_EMPTY + w), st.ph ^ 1, p.err, 73);
            __syncwarp();
            if (!ok) break;
            const unsigned char* raw = sm.base + C::OFF_RAW + s * RAW_B + from;
            unsigned char* wide = sm.base + C::OFF_ST + w * TILE_B;
            const int low = it.kv_lo - key0 - row0, end = it.kv_end - key0 - row0;
            auto widen_all = [&](auto cut) {
#pragma unroll 4
              for (int i = 0; i < CHK / 8; ++i) {
                uint4 v = *reinterpret_cast<const uint4*>(raw + i * 1024);
                if (cut.value && (8 * i < low || 8 * i >= end)) v = make_uint4(0, 0, 0, 0);
                *reinterpret_cast<uint4*>(wide + to0 + i * 1024) =
                    make_uint4(widen((uint16_t)v.x), widen((uint16_t)(v.x >> 16)),
                               widen((uint16_t)v.y), widen((uint16_t)(v.y >> 16)));
                *reinterpret_cast<uint4*>(wide + to1 + i * 1024) =
                    make_uint4(widen((uint16_t)v.z), widen((uint16_t)(v.z >> 16)),
                               widen((uint16_t)v.w), widen((uint16_t)(v.w >> 16)));
              }
            };
            if (ragged(it, c / 2)) widen_all(std::true_type());
            else widen_all(std::false_type());
            ptx::fence_proxy_async_smem();
            ptx::mbar_arrive(sm.bar(C::B_WIDE + w));
            ptx::mbar_arrive(sm.bar(C::B_EMPTY + s));
          }
        } else {
          // Every chunk is waited for and let go, whether zeroed or not, so that
          // these warps are never a stage's whole round ahead or behind.
          for (int x2 = 0; x2 < 2 * it.n && ok; ++x2, st.next()) {
            const int s = st.s, c = x2 / 2;
            ok = wait_at(sm, sm.bar(C::B_FULL + s), st.ph, p.err, 74);
            __syncwarp();
            if (!ok) break;
            if (!ragged(it, c)) {
              if (lane == 0) ptx::mbar_arrive(sm.bar(C::B_EMPTY + s));
              continue;
            }
            unsigned char* v = sm.base + C::OFF_ST + s * TILE_B;
            const int key0 = (it.jl - c) * CHK;
            for (int u = x; u < CHK * 16; u += 64) {
              const int row = u >> 4;
              if (key0 + row < it.kv_lo || key0 + row >= it.kv_end)
                *reinterpret_cast<uint4*>(v + ((u >> 3) & 1) * HALF_B + row * 128 + (u & 7) * 16) =
                    make_uint4(0, 0, 0, 0);
            }
            ptx::fence_proxy_async_smem();
            ptx::mbar_arrive(sm.bar(C::B_FIX + nfix % NFIX));
            ++nfix;
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(sm.bar(C::B_EMPTY + s));
          }
        }
        if (!ok) break;
      }
    }
  } else {
    // ================= softmax and epilogue =================
    const int t = warp >> 3, half = (warp >> 2) & 1;
    const int row = tid & 127, tok = row / G, hd = row % G;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_col = tmem + lane_base + S_COL + 128 * t + 64 * half;
    const uint32_t o_col = tmem + lane_base + O_COL + 128 * t + 64 * half;
    const float ksc = FP8 ? __ldg(p.k_scale) : 1.f;
    const float vsc = FP8 ? __ldg(p.v_scale) : 1.f;
    const bool out_aligned = reinterpret_cast<uintptr_t>(p.out) % 32 == 0;
    int nc = 0, nq = 0, nx = 0;  // chunks of this tile, items with chunks, exchanges
    int np = 0;  // parts written
    int merge = -1;  // the item to join: its first CTA, this CTA's max and sum, if any
    float m_own = -INFINITY, l_own = 0.f;
    bool some = false;
    __nv_bfloat16* own_row = nullptr;
    auto part_at = [&](int cta, int slot) -> float* {
      return p.parts + (2 * (int64_t)cta + slot) * kPartWords;
    };
    bool ok = true;
    // By a whole warp: whether all of its lanes' waits ended.
    auto wait = [&](int bar, uint32_t parity, int code) -> bool {
      const bool mine = wait_at(sm, sm.bar(bar), parity, p.err, code);
      __syncwarp();
      return __all_sync(0xffffffffu, mine);
    };
    // A word of the row's other half for one of this half's.
    auto exchange = [&](float mine) -> float {
      float* at = reinterpret_cast<float*>(sm.base + C::OFF_X) + ((nx & 1) * 2 + t) * 256 + row;
      at[128 * half] = mine;
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(sm.bar(C::B_X + t));
      ok = wait(C::B_X + t, nx & 1, 82);
      ++nx;
      return at[128 * (half ^ 1)];
    };
    auto store_row = [&](__nv_bfloat16* to, const float (&o)[32], float inv) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
          w[e] = pack_bf16x2_rn(o[16 * c + 2 * e] * inv * vsc, o[16 * c + 2 * e + 1] * inv * vsc);
        store_32(to + 16 * c, w, out_aligned);  // (rows lie apart: whole sectors)
      }
    };
    for (int k = 0; ok; ++k) {
      const Item it = read_item(k);
      if (it.r < 0) break;
      const int ntok = t ? it.ntok[1] : it.ntok[0];
      const int first = t ? it.a[1] : it.a[0], last = t ? it.b[1] : it.b[0];
      // (nothing is written outside the batch, whatever the starts say)
      const bool row_ok = tok < ntok && (unsigned)(it.q0 + t * MQ + tok) < (unsigned)p.num_tokens;
      const int pos = it.pos + t * MQ + tok;
      __nv_bfloat16* orow = p.out +
                            ((int64_t)(it.q0 + t * MQ + tok) * p.num_heads + it.g * G + hd) * D +
                            64 * half;
      if (it.n == 0) {
        if (row_ok) {
#pragma unroll
          for (int c = 0; c < 8; ++c) reinterpret_cast<uint4*>(orow)[c] = make_uint4(0, 0, 0, 0);
        }
        continue;
      }
      float rs = p.scale_log2;
      if constexpr (FP8) {
        // the row's half of q as f16, in place, under the row's own power of two
        ok = wait(C::B_Q_FULL, nq & 1, 75);
        if (!ok) break;
        unsigned char* qrow = sm.base + C::OFF_Q + t * TILE_B + half * HALF_B + row * 128;
        float amax = 0.f;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const uint4 v = *reinterpret_cast<const uint4*>(qrow + (((c ^ row) & 7) << 4));
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(w[e])), fabsf(bf16_hi(w[e]))));
        }
        amax = fmaxf(amax, exchange(amax));
        if (!ok) break;
        // (kept within the normal floats; an infinite or NaN q stays what it is)
        const int e2 = min(max((int)(__float_as_uint(amax) >> 23), 1), 253) - 127;
        const float inv = __int_as_float((127 - e2) << 23);
        rs *= ksc * __int_as_float((127 + e2) << 23);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          uint4* at = reinterpret_cast<uint4*>(qrow + (((c ^ row) & 7) << 4));
          const uint4 v = *at;
          *at = make_uint4(pack2<true>(bf16_lo(v.x) * inv, bf16_hi(v.x) * inv),
                           pack2<true>(bf16_lo(v.y) * inv, bf16_hi(v.y) * inv),
                           pack2<true>(bf16_lo(v.z) * inv, bf16_hi(v.z) * inv),
                           pack2<true>(bf16_lo(v.w) * inv, bf16_hi(v.w) * inv));
        }
        ptx::fence_proxy_async_smem();
        ptx::mbar_arrive(sm.bar(C::B_Q_READY + t));
      }
      ++nq;
      // keys [low, lim) are visible to the row
      int lim = row_ok ? pos + 1 : 0, low = 0;
      if (row_ok && pos < it.prefix) lim = max(lim, it.prefix);
      if (p.mod.window > 0) low = max(0, pos - p.mod.window + 1);
      const unsigned seen = (unsigned)max(0, lim - low);
      const float slope =
          p.mod.slopes ? __ldg(&p.mod.slopes[it.g * G + hd]) * 1.4426950408889634f : 0.f;
      const int pos0 = it.pos + t * MQ;  // of the tile's first token
      const bool cap = LARGE || p.mod.cap_log2 > 0.f;
      const float ru = rs * p.mod.inv_cap;  // to u = score / cap
      // The polynomial's coefficients, with the powers of ru in them; where the
      // highest leaves the normal floats, the cap is taken the other way.  (Rows
      // under e4m3's scales are multiplied by ru first.)
      const float ru2 = ru * ru;
      const bool ru_fits = FP8 || (fabsf(ru) >= 0x1p-13f && fabsf(ru) <= 0x1p13f);
      float poly_k[4];
      {
        float r = ru;
#pragma unroll
        for (int x = 0; x < 4; ++x, r *= ru2) poly_k[x] = p.mod.tanh_poly[x] * (FP8 ? 1.f : r);
      }
      // capped, without a bias, over bf16: weights are 2^s as it is
      const bool bounded = !FP8 && !LARGE && cap && !p.mod.slopes && p.mod.cap_log2 <= kBoundedLog2;
      float m_ref = bounded && first < last ? 0.f : -INFINITY;
      float2 l2 = make_float2(0.f, 0.f);
      for (int c = first; c < last; ++c) {
        ok = wait(C::B_S_FULL + t, nc & 1, 76);
        if (!ok) break;
        ptx::tc_fence_after();
        const int key0 = (it.jl - c) * CHK + 64 * half;
        // every row of a full tile sees every key between the last token's
        // window and the first token
        const bool whole = ntok == MQ && key0 + 64 <= pos0 + 1 &&
                           (p.mod.window <= 0 || key0 >= pos0 + MQ - p.mod.window);
        // 32 logits at a time, from key 32 x of the half on
        auto load = [&](float2 (&s)[16], int x) {
          float v[32];
          ptx::tmem_ld_x32(s_col + 32 * x, v);
          ptx::tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 16; ++e) s[e] = make_float2(v[2 * e], v[2 * e + 1]);
        };
        auto largest = [](const float2 (&s)[16]) {
          float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int e = 0; e < 16; ++e) top[e & 1] = max3(top[e & 1], s[e].x, s[e].y);
          return fmaxf(top[0], top[1]);
        };
        auto largest_size = [](const float2 (&s)[16]) {
          float top[2] = {0.f, 0.f};
#pragma unroll
          for (int e = 0; e < 16; ++e)
            top[e & 1] = max3(top[e & 1], fabsf(s[e].x), fabsf(s[e].y));
          return fmaxf(top[0], top[1]);
        };
        auto fits = [&](float size) {
          return __all_sync(0xffffffffu, !row_ok || (ru_fits && size * fabsf(ru) <= 0.75f)) != 0;
        };
        auto by_poly = [&](float2 (&s)[16], float2 plus) {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            s[e] = capped_poly(FP8 ? mul2(s[e], both(ru)) : s[e], poly_k, plus);
        };
        auto by_exp = [&](float2 (&s)[16]) {
          const float re = rs * p.mod.inv_cap_log2, two = -2.f * p.mod.cap_log2;
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            s[e].x = fmaf(two, fast_reciprocal(1.f + fast_exp2(s[e].x * re)), p.mod.cap_log2);
            s[e].y = fmaf(two, fast_reciprocal(1.f + fast_exp2(s[e].y * re)), p.mod.cap_log2);
          }
        };
        auto by_either = [&](float2 (&s)[16]) {
          const float to_u = p.mod.inv_cap;
#pragma unroll
          for (int e = 0; e < 16; ++e) s[e] = mul2(s[e], both(rs));
          if (__all_sync(0xffffffffu, largest_size(s) * to_u <= kTanhSmall)) {  // (the same scores)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              s[e].x = capped_small(s[e].x, s[e].x * to_u);
              s[e].y = capped_small(s[e].y, s[e].y * to_u);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              s[e].x = capped(s[e].x, s[e].x * to_u, p.mod.cap_log2);
              s[e].y = capped(s[e].y, s[e].y * to_u, p.mod.cap_log2);
            }
          }
        };
        auto mask = [&](float2 (&s)[16], int x) {
          const int kf = low - key0 - 32 * x;
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            if ((unsigned)(2 * e - kf) >= seen) s[e].x = -INFINITY;
            if ((unsigned)(2 * e + 1 - kf) >= seen) s[e].y = -INFINITY;
          }
        };
        auto weigh = [&](float2 (&s)[16], int x) {  // 2^s as weights over the logits
          float2 sum = make_float2(0.f, 0.f);
          float w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 q = make_float2(fast_exp2(s[e].x), fast_exp2(s[e].y));
            const uint32_t w2 = pack2<FP8>(q.x, q.y);
            w[e] = __uint_as_float(w2);
            // bf16: the sum is of the weights as rounded, so that a large one's
            // rounding (2^-9) leaves the quotient; f16's 2^-12 may stay in
            sum = add2(sum, FP8 ? q : make_float2(bf16_lo(w2), bf16_hi(w2)));
          }
          ptx::tmem_st_x16(s_col + 16 * x, w);
          l2 = add2(l2, sum);
        };
        if (bounded) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            float2 s[16];
            load(s, x);
            // Whether the polynomial holds, after the fact: no |u| is above 3/4 where
            // the u^4 sum to less than (3/4)^4.  (The largest |u|, before: 122 us for
            // four capped prompts, where this takes 118.)
            float2 fourth = make_float2(0.f, 0.f);
#pragma unroll
            for (int e = 0; e < 16; ++e) s[e] = capped_poly_sum(s[e], poly_k, fourth);
            if (!__all_sync(0xffffffffu,
                            !row_ok || (ru_fits && (fourth.x + fourth.y) * (ru2 * ru2) <=
                                                       0.31640625f))) {
              load(s, x);
              by_exp(s);
            }
            if (!whole) mask(s, x);
            weigh(s, x);
          }
        } else {
          // The row's largest logit: of whole halves without a bias that of the
          // raw ones, changed (the cap is monotonic); others are changed first.
          float cm = -INFINITY;
          bool late = whole && !p.mod.slopes && rs >= 0.f && !LARGE;
          if (late) {
            float size = 0.f;
#pragma unroll 1
            for (int x = 0; x < 2; ++x) {
              float2 s[16];
              load(s, x);
              cm = fmaxf(cm, largest(s));
              if (cap) size = fmaxf(size, largest_size(s));
            }
            cm *= rs;
            if (cap) {
              cm = p.mod.cap_log2 *
                   (1.f - 2.f * fast_reciprocal(1.f + fast_exp2(cm * p.mod.inv_cap_log2)));
              late = fits(size);
              if (!late) cm = -INFINITY;
            }
          }
          if (!late) {
            // no key behind a row's own: the bias is a line over the keys
            const float at = (float)(pos - key0);
#pragma unroll 1
            for (int x = 0; x < 2; ++x) {
              float2 s[16];
              load(s, x);
              if (!cap) {
#pragma unroll
                for (int e = 0; e < 16; ++e) s[e] = mul2(s[e], both(rs));
              } else if (LARGE) {
                by_either(s);
              } else if (fits(largest_size(s))) {
                by_poly(s, both(0.f));
              } else {
                by_exp(s);
              }
              if (p.mod.slopes) {
                const float d = at - 32.f * x;
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                  s[e].x = fmaf(-slope, fabsf(d - (float)(2 * e)), s[e].x);
                  s[e].y = fmaf(-slope, fabsf(d - (float)(2 * e + 1)), s[e].y);
                }
              }
              if (!whole) mask(s, x);
              cm = fmaxf(cm, largest(s));
              float v[32];
#pragma unroll
              for (int e = 0; e < 16; ++e) v[2 * e] = s[e].x, v[2 * e + 1] = s[e].y;
              ptx::tmem_st_x32(s_col + 32 * x, v);
            }
            ptx::tmem_st_wait();
          }
          cm = fmaxf(cm, exchange(cm));
          if (!ok) break;
          float alpha = 1.f;
          if (cm > m_ref + kRescaleLog2) {
            if (m_ref != -INFINITY) alpha = fast_exp2(m_ref - cm);
            m_ref = cm;
          }
          if (__any_sync(0xffffffffu, alpha != 1.f)) {  // (never at an item's first keys)
            ok = wait(C::B_O_FULL + t, (nc - 1) & 1, 77);  // the products of the chunk before
            if (!ok) break;
            ptx::tc_fence_after();
#pragma unroll 1
            for (int x = 0; x < 2; ++x) {
              float o[32];
              ptx::tmem_ld_x32(o_col + 32 * x, o);
              ptx::tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] *= alpha;
              ptx::tmem_st_x32(o_col + 32 * x, o);
            }
            l2.x *= alpha;
            l2.y *= alpha;
          }
          const float2 plus = both(C::kRaise - (m_ref == -INFINITY ? 0.f : m_ref));
          const float2 factor = both(late ? rs : 1.f);
#pragma unroll 1
          for (int x = 0; x < 2; ++x) {
            float2 s[16];
            load(s, x);
            if (late && cap) {
              by_poly(s, plus);
            } else {
#pragma unroll
              for (int e = 0; e < 16; ++e) s[e] = fma2(s[e], factor, plus);
            }
            weigh(s, x);
          }
        }
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(sm.bar(C::B_P_FULL + t));
        ++nc;
      }
      if (!ok) break;
      float l = l2.x + l2.y;
      l += exchange(l);
      if (!ok) break;
      if (first < last) {  // (a tile may have no tokens, or no chunks in this part)
        ok = wait(C::B_O_FULL + t, (nc - 1) & 1, 78);
        if (!ok) break;
        ptx::tc_fence_after();
      }
      if (it.merge >= 0) {  // the CTA's last item
        merge = it.merge;
        m_own = m_ref;
        l_own = l;
        some = first < last;
        own_row = row_ok ? orow : nullptr;
        break;
      }
      float* part = nullptr;
      if (it.part >= 0) {
        part = part_at(blockIdx.x, it.part);
        if (half == 0)
          __stcg(reinterpret_cast<float2*>(part + 256 * D) + 128 * t + row, make_float2(m_ref, l));
      }
      if (first < last) {
        const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
#pragma unroll 1
        for (int x = 0; x < 2; ++x) {
          float o[32];
          ptx::tmem_ld_x32(o_col + 32 * x, o);
          ptx::tmem_ld_wait();
          if (it.part >= 0 && row_ok) {
            float4* to = reinterpret_cast<float4*>(part) + (t * 32 + 16 * half + 8 * x) * 128 + row;
#pragma unroll
            for (int e = 0; e < 8; ++e)
              __stcg(to + 128 * e, make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]));
          } else if (it.part < 0 && row_ok) {
            store_row(orow + 32 * x, o, inv);
          }
          __syncwarp();
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(sm.bar(C::B_O_EMPTY + t));
      }
      if (it.part >= 0) {
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(sm.bar(C::B_PART));
        if (warp == 0) {  // once both tiles' sums are written
          ok = wait(C::B_PART, np & 1, 80);
          if (ok && lane == 0) {
            ptx::fence_acq_rel_gpu();
            st_release(&p.flags[2 * blockIdx.x + it.part], p.epoch);
          }
        }
        ++np;
      }
    }
    // The item whose end this CTA holds: its own sums (in tensor memory, if it
    // has some) and the parts of the CTAs before it, in their order.
    if (ok && merge >= 0) {
      const int count = j - merge;
      auto cta = [&](int k) { return (merge + k) * p.num_kv_heads + g; };
      // the first CTA's part starts the item, the others' go on with it
      for (int k = lane; k < count; k += 32) {  // (each warp for itself)
        const long long begun = clock64();
        while (ld_acquire(&p.flags[2 * cta(k) + (k == 0 ? 1 : 0)]) != p.epoch) {
          if (clock64() - begun > tc::kWaitClocks) {
            atomicExch(p.err, 79);
            ok = false;
            break;
          }
        }
      }
      ok = __all_sync(0xffffffffu, ok);
      if (lane == 0) ptx::mbar_arrive(sm.bar(C::B_MERGE));
      // Both tiles' warps are done with their products: shared memory is free (an
      // item may have some for one tile alone), and all have seen the flags.
      const bool all = wait(C::B_MERGE, 0, 81);
      ok = ok && all;
      if (ok && warp == 0) {  // down, for a replay of this launch
        for (int k = lane; k < count; k += 32) p.flags[2 * cta(k) + (k == 0 ? 1 : 0)] = 0;
      }
      __syncwarp();
      if (ok) {
        // Sums come through shared memory, in pieces of 32 columns of a part: 8
        // copies a thread, of its own row, three pieces ahead.  (By plain loads,
        // two or three parts took 15 us.)
        constexpr int kAhead = 3;
        static_assert(kAhead * 512 * 128 <= C::OFF_X, "the pieces' room");
        const uint32_t own = sm.base_u32 + tid * 16;
        auto ml_of = [&](int k) {
          return __ldcg(reinterpret_cast<const float2*>(part_at(cta(k), k == 0 ? 1 : 0) + 256 * D) +
                        128 * t + row);
        };
        const int pieces = 2 * count;
        auto fetch = [&](int i) {  // piece i: columns 32 (i / count) on, of part i % count
          if (i < pieces && own_row) {
            const int x = i >= count, k = i - x * count;
            const float4* from = reinterpret_cast<const float4*>(part_at(cta(k), k == 0 ? 1 : 0)) +
                                 (t * 32 + 16 * half + 8 * x) * 128 + row;
#pragma unroll
            for (int e = 0; e < 8; ++e)
              cp_async_16(own + ((i % kAhead) * 8 + e) * 8192, from + 128 * e, 16);
          }
          cp_async_commit();
        };
#pragma unroll
        for (int i = 0; i < kAhead; ++i) fetch(i);
        float most = m_own;
#pragma unroll 4
        for (int k = 0; k < count; ++k) most = fmaxf(most, ml_of(k).x);
        // (a part without keys has no sums written)
        const bool mine = some && (m_own != -INFINITY || l_own != 0.f);
        const float f_own = mine ? fast_exp2(m_own - most) : 0.f;
        float l = mine ? f_own * l_own : 0.f;
#pragma unroll 4
        for (int k = 0; k < count; ++k) {
          const float2 ml = ml_of(k);
          if (ml.x != -INFINITY || ml.y != 0.f) l += fast_exp2(ml.x - most) * ml.y;
        }
        const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
        float2 ml = ml_of(0);
#pragma unroll 1
        for (int x = 0; x < 2; ++x) {
          float o[32];
          if (some) {
            ptx::tmem_ld_x32(o_col + 32 * x, o);
            ptx::tmem_ld_wait();
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = mine ? o[e] * f_own : 0.f;
#pragma unroll 1
          for (int k = 0; k < count; ++k) {
            const int i = x * count + k;
            const float2 now = ml;
            ml = ml_of(k + 1 < count ? k + 1 : 0);
            cp_async_wait<kAhead - 1>();
            if (own_row && (now.x != -INFINITY || now.y != 0.f)) {
              const float f = fast_exp2(now.x - most);
              const float4* v =
                  reinterpret_cast<const float4*>(sm.base) + (i % kAhead) * 8 * 512 + tid;
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float4 w = v[512 * e];
                o[4 * e] += f * w.x, o[4 * e + 1] += f * w.y;
                o[4 * e + 2] += f * w.z, o[4 * e + 3] += f * w.w;
              }
            }
            fetch(i + kAhead);
          }
          if (own_row) store_row(own_row + 32 * x, o, inv);
          __syncwarp();
        }
        cp_async_wait<0>();
      }
    }
  }

  // ---------------- teardown ----------------
  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == MMA_WARP) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

// Ranges per head: those whose CTAs fill the SMs best in one round or two.
int ranges_of(int heads, int num_sms) {
  int best = 1;
  auto rounds = [&](int64_t r) { return (r * heads + num_sms - 1) / num_sms; };
  for (int r = 2; (int64_t)r * heads <= 2 * num_sms; ++r)
    if (rounds(r) * best < rounds(best) * r) best = r;
  return best;
}
size_t flag_bytes(int64_t ctas) { return (size_t)(ctas * 16 + 255) / 256 * 256; }

template <int G, bool FP8, bool LARGE>
cudaError_t launch_one(const Params& prm, const CUtensorMap& mk, const CUtensorMap& mv,
                     const CUtensorMap& mq, cudaStream_t stream) {
  const cudaError_t e = allow_large<prefill_scored_kernel<G, FP8, LARGE>>();
  if (e != cudaSuccess) return e;
  return launch_dependent<prefill_scored_kernel<G, FP8, LARGE>>(
      dim3(prm.ranges * prm.num_kv_heads), dim3(NTHREADS), Cfg<FP8>::SMEM_BYTES, stream, 1, mk, mv, mq,
      prm);
}

template <int G, bool FP8>
cudaError_t launch_g(const Params& prm, const CUtensorMap& mk, const CUtensorMap& mv,
                     const CUtensorMap& mq, cudaStream_t stream) {
  return prm.mod.large_cap ? launch_one<G, FP8, true>(prm, mk, mv, mq, stream)
                           : launch_one<G, FP8, false>(prm, mk, mv, mq, stream);
}

template <bool FP8>
cudaError_t launch_f(const Params& prm, const CUtensorMap& mk, const CUtensorMap& mv,
                     const CUtensorMap& mq, int group, cudaStream_t stream) {
  switch (group) {
    case 1: return launch_g<1, FP8>(prm, mk, mv, mq, stream);
    case 2: return launch_g<2, FP8>(prm, mk, mv, mq, stream);
    case 4: return launch_g<4, FP8>(prm, mk, mv, mq, stream);
    case 8: return launch_g<8, FP8>(prm, mk, mv, mq, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace ps

// A pair holds 2 * 128 / group tokens of one request; the last of each request
// may hold fewer.
bool prefill_scored_fits(int64_t num_tokens, int group, int num_seqs) {
  return num_tokens * group / 256 + num_seqs <= 65535;
}

size_t prefill_scored_workspace_bytes(int num_kv_heads, int num_sms) {
  const int64_t ranges = ps::ranges_of(num_kv_heads, num_sms), ctas = ranges * num_kv_heads;
  if (ranges == 1) return 0;  // nothing is split
  return ps::flag_bytes(ctas) + (size_t)ctas * 2 * ps::kPartWords * 4;
}

cudaError_t launch_prefill_scored(const PrefillLaunch& a, cudaStream_t stream) {
  using namespace ps;
  tc::EncodeTiledFn enc = tc::encode_fn();
  if (!enc) return cudaErrorNotSupported;
  const int group = a.num_heads / a.num_kv_heads;
  const int box_tok = a.block_size < 128 ? a.block_size : 128;
  CUtensorMap mk, mv, mq;
  {
    // [blocks, block_size, H_kv, d]: a box is 128 bytes (64 bf16 or all 128
    // e4m3 of d) of box_tok tokens of one KV head
    const cuuint64_t elt = a.fp8 ? 1 : 2;
    const CUtensorMapDataType dt =
        a.fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const CUtensorMapL2promotion promo =
        a.fp8 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B;
    cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)a.num_kv_heads, (cuuint64_t)a.block_size,
                          (cuuint64_t)a.num_blocks};
    cuuint64_t strides[3] = {(cuuint64_t)D * elt, (cuuint64_t)a.num_kv_heads * D * elt,
                             (cuuint64_t)a.block_size * a.num_kv_heads * D * elt};
    cuuint32_t box[4] = {(cuuint32_t)(128 / elt), 1, (cuuint32_t)box_tok, 1};
    cuuint32_t es[4] = {1, 1, 1, 1};
    for (auto [map, base] : {std::pair<CUtensorMap*, const void*>(&mk, a.k_cache), {&mv, a.v_cache}})
      if (enc(map, dt, 4, const_cast<void*>(base), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, promo,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
  }
  {
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)a.num_heads, (cuuint64_t)a.num_tokens};
    cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)a.num_heads * D * 2};
    cuuint32_t box[3] = {64, (cuuint32_t)group, (cuuint32_t)(128 / group)};
    cuuint32_t es[3] = {1, 1, 1};
    if (enc(&mq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(a.q), dims, strides, box,
            es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  Params prm{};
  prm.out = static_cast<__nv_bfloat16*>(a.out);
  prm.block_tables = a.block_tables;
  prm.seq_lens = a.seq_lens;
  prm.qsl = a.query_start_loc;
  prm.err = static_cast<int*>(a.workspace);
  prm.ranges = ranges_of(a.num_kv_heads, a.num_ctas);
  char* ws = static_cast<char*>(a.workspace) + 256;
  prm.flags = reinterpret_cast<unsigned long long*>(ws);
  prm.parts = reinterpret_cast<float*>(ws + flag_bytes(prm.ranges * a.num_kv_heads));
  prm.epoch = tc::next_call_epoch();
  prm.num_seqs = a.num_seqs;
  prm.num_tokens = a.num_tokens;
  prm.num_heads = a.num_heads;
  prm.num_kv_heads = a.num_kv_heads;
  prm.max_blocks = a.max_blocks;
  prm.num_blocks = a.num_blocks;
  prm.block_size = a.block_size;
  while ((1 << prm.log2_bs) < a.block_size) ++prm.log2_bs;
  prm.box_tok = box_tok;
  while ((1 << prm.log2_box) < box_tok) ++prm.log2_box;
  prm.scale_log2 = a.scale * 1.4426950408889634f;
  prm.k_scale = a.k_scale;
  prm.v_scale = a.v_scale;
  prm.mod = a.mod;
  return a.fp8 ? launch_f<true>(prm, mk, mv, mq, group, stream)
               : launch_f<false>(prm, mk, mv, mq, group, stream);
}

}  // namespace pa
