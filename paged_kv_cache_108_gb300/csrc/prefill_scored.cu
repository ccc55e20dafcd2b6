// Prompt attention with changed scores on the 5th-generation tensor cores,
// for a bf16 or e4m3 cache with head_dim 128: the tiles of pa_varlen_scored.
//
// Request r's new tokens are q[qsl[r] .. qsl[r+1]), the last T of its context;
// the token at position i sees keys below i + 1, or below the request's prefix
// if i is inside it, and of those the last `window` up to its own position:
//   s = scale q . k;  s <- cap tanh(s / cap);  s <- s - slope |i - j|
//   out = softmax(s) V.
//
// Bound: with a cap the issue of the softmax's instructions (about 9 a logit,
// 128 x 128 logits a tile and chunk), then the MMAs (4 d flop a logit).
//
// A work item is a pair of neighbouring query tiles of one request and KV head:
// 2 x 128 rows, row = token * G + query head in the group.  Both tiles use
// each K and V chunk of 128 keys while it is in shared memory, and alternate
// on the tensor cores: while one tile's softmax runs, the other's products do.
//   S_t = Q_t K^T   M = 128 rows, N = 128 keys, K = 128, into tensor memory
//   P_t             one thread a row: 128 logits from tensor memory, changed,
//                   masked, exponentiated; 16-bit weights written back over S_t
//   O_t += P_t V    A = P_t from tensor memory, B = the V chunk, MN-major
// Tensor memory is full: S_0, S_1 (P over them), O_0, O_1 of 128 columns.
// O is rescaled only when a row's running max grows by more than 2^8; all lanes
// of the row's warp take part (by 1), as tensor memory accesses are a warp's.
//
// The cap.  tanh(u) for |u| <= 1 is an odd polynomial of degree 11 (fitted to
// the smallest largest error over [0, 1]: 2.5e-7), which runs on the FMA pipe
// two logits an instruction; a chunk with a larger |u| in one of the warp's
// rows takes 1 - 2 / (1 + e^2u), one exponential and one reciprocal.
//
// An e4m3 cache: two warps widen each chunk to f16 (exact) in shared memory;
// q, scaled by a power of two a row that puts its largest |q| in [1, 2), is
// rounded to f16 in place by the row's thread (11 bits for bf16's 8: exact down
// to 2^-14 of the row's largest); weights are f16, raised by 2^7.
//
// Values of keys that no token of the item sees (behind the last, before a
// window, in part not loaded) are zeroed in shared memory, so that nothing
// they hold reaches a sum; their logits are masked by a select.
//
// Roles (384 threads): warps 0-3 and 4-7 softmax and epilogue of tile 0 and 1;
// warp 8 loads (q, K, V) and hands out items; warp 9 issues the MMAs; warps
// 10-11 widen or zero.  Items come from a counter in the workspace (word 1,
// zeroed by the host before the launch), each request's longest first.  Every
// mbarrier wait is bounded: error word 0, the CTA gives up.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

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
using tc::wait_bar;

constexpr int D = 128, CHK = 128;       // keys per chunk
constexpr int kMaxReqs = 256;
constexpr int HALF_B = 128 * 128;       // 128 rows of 64 16-bit columns
constexpr int TILE_B = 2 * HALF_B;      // a q tile, a K or V chunk in 16 bits
constexpr int RAW_B = CHK * D;          // a K or V chunk in e4m3
constexpr int NTHREADS = 384;
constexpr int PROD_WARP = 8, MMA_WARP = 9, FIX_WARP = 10;
constexpr int NITEM = 4;                // items published ahead
constexpr int NFIX = 4;                 // zeroed V chunks ahead of their MMA, at most
constexpr int S_COL = 0, O_COL = 256;   // tile t: + 128 t
constexpr float kRescaleLog2 = 8.f;

template <bool FP8>
struct Cfg {
  static constexpr int NST = FP8 ? 3 : 5;   // 16-bit chunks in shared memory
  static constexpr int NRAW = FP8 ? 3 : 0;  // e4m3 chunks
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_ST = OFF_Q + 2 * TILE_B;
  static constexpr int OFF_RAW = OFF_ST + NST * TILE_B;
  static constexpr int OFF_BAR = OFF_RAW + NRAW * RAW_B;
  static constexpr int NLOAD = FP8 ? NRAW : NST;  // stages that TMA fills
  static constexpr int B_Q_FULL = 0, B_Q_EMPTY = 1, B_Q_READY = 2 /* [2] */, B_FULL = 4,
                       B_EMPTY = B_FULL + NLOAD, B_WIDE = B_EMPTY + NLOAD,
                       B_WIDE_EMPTY = B_WIDE + NST, B_FIX = B_WIDE_EMPTY + NST,
                       B_S_FULL = B_FIX + NFIX, B_P_FULL = B_S_FULL + 2, B_O_FULL = B_P_FULL + 2,
                       B_O_EMPTY = B_O_FULL + 2, B_ITEM_FULL = B_O_EMPTY + 2,
                       B_ITEM_EMPTY = B_ITEM_FULL + NITEM, NBARS = B_ITEM_EMPTY + NITEM;
  static constexpr int OFF_TMEM = OFF_BAR + NBARS * 8;
  static constexpr int OFF_ABORT = OFF_TMEM + 4;
  static constexpr int OFF_RING = OFF_ABORT + 4;
  // pairs of tiles before each request, [R + 1]; at most 65535 new tokens
  static constexpr int OFF_TP = OFF_RING + NITEM * 4;
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
  unsigned* next_item;          // workspace word 1
  int num_seqs, num_heads, num_kv_heads, max_blocks, num_blocks, block_size, log2_bs;
  int box_tok, log2_box;
  float scale_log2;
  const float* k_scale;  // e4m3: device scalars
  const float* v_scale;
  ScoreMod mod;
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

// One work item.
struct Item {
  int r, g;
  int q0;        // first q row of the pair
  int pos;       // position of its first token
  int ntok[2];   // new tokens of each tile
  int kv_lo, kv_end;  // keys that the pair's tokens see lie in [kv_lo, kv_end)
  int prefix;
  int j0, n;     // chunks of the pair: first, count (0: zero rows)
  int a[2], b[2];  // those of each tile, relative to j0: [a, b)
};

template <int G>
__device__ __forceinline__ Item item_of(int i, const uint16_t* tp, const Params& p) {
  constexpr int MQ = 128 / G;
  Item it;
  const int pair = i / p.num_kv_heads;
  it.g = i - pair * p.num_kv_heads;
  int lo = 0, hi = p.num_seqs;  // the request of this pair: tp[r] <= pair < tp[r + 1]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (tp[mid] <= pair) lo = mid;
    else hi = mid;
  }
  it.r = lo;
  const int first = __ldg(&p.qsl[lo]), T = __ldg(&p.qsl[lo + 1]) - first;
  const int sl = __ldg(&p.seq_lens[lo]), ctx = sl - T;
  const int tok = (tp[lo + 1] - 1 - pair) * 2 * MQ;  // the last tokens, which see most, first
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
  it.j0 = it.kv_lo / CHK;
  const bool none = ctx < 0 || it.kv_end > (p.max_blocks << p.log2_bs);
  it.n = none ? 0 : (it.kv_end + CHK - 1) / CHK - it.j0;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const bool some = it.ntok[t] > 0 && !none;
    it.a[t] = some ? low[t] / CHK - it.j0 : 0;
    it.b[t] = some ? (end[t] + CHK - 1) / CHK - it.j0 : 0;
  }
  return it;
}
// Whether a chunk holds keys that no token of the item sees.
__device__ __forceinline__ bool ragged(const Item& it, int c) {
  const int key0 = (it.j0 + c) * CHK;
  return key0 < it.kv_lo || key0 + CHK > it.kv_end;
}

// The logits s (times rs: in log2 units) as changed ones in log2 units; the
// row's own position is `at` keys behind the first of them.
__device__ __forceinline__ void change_scores(float2 (&s)[64], float rs, const ScoreMod& mod,
                                              float slope, float at) {
  if (mod.cap_log2 > 0.f) {
    const float ru = rs * mod.inv_cap;  // to u = score / cap
    float most = 0.f;
#pragma unroll
    for (int e = 0; e < 64; ++e) most = fmaxf(most, fmaxf(fabsf(s[e].x), fabsf(s[e].y)));
    const float2 ru2 = both(ru);
    if (__all_sync(0xffffffffu, most * fabsf(ru) <= 1.f)) {
      float2 c[6];
#pragma unroll
      for (int k = 0; k < 6; ++k) c[k] = both(mod.tanh_poly[k]);
#pragma unroll
      for (int e = 0; e < 64; ++e) {
        const float2 u = mul2(s[e], ru2), z = mul2(u, u);
        float2 h = fma2(c[5], z, c[4]);
        h = fma2(h, z, c[3]);
        h = fma2(h, z, c[2]);
        h = fma2(h, z, c[1]);
        h = fma2(h, z, c[0]);
        s[e] = mul2(h, u);
      }
    } else {
      const float re = ru * 2.f * 1.4426950408889634f, cap = mod.cap_log2;
#pragma unroll
      for (int e = 0; e < 64; ++e) {
        s[e].x = cap - 2.f * cap * fast_reciprocal(1.f + fast_exp2(s[e].x * re));
        s[e].y = cap - 2.f * cap * fast_reciprocal(1.f + fast_exp2(s[e].y * re));
      }
    }
  } else {
    const float2 rs2 = both(rs);
#pragma unroll
    for (int e = 0; e < 64; ++e) s[e] = mul2(s[e], rs2);
  }
  if (mod.slopes) {
#pragma unroll
    for (int e = 0; e < 64; ++e) {
      s[e].x -= slope * fabsf(at - (float)(2 * e));
      s[e].y -= slope * fabsf(at - (float)(2 * e + 1));
    }
  }
}

template <int G, bool FP8>
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
      if ((i >= C::B_Q_READY && i < C::B_Q_READY + 2) || (i >= C::B_P_FULL && i < C::B_P_FULL + 2) ||
          (i >= C::B_O_EMPTY && i < C::B_O_EMPTY + 2))
        cnt = 128;
      // the MMAs, and the two zeroing warps
      if (!FP8 && i >= C::B_EMPTY && i < C::B_EMPTY + NLOAD) cnt = 3;
      // the two widening or zeroing warps' threads
      if ((FP8 && i >= C::B_EMPTY && i < C::B_EMPTY + NLOAD) ||
          (i >= C::B_WIDE && i < C::B_WIDE + NST) || (i >= C::B_FIX && i < C::B_FIX + NFIX))
        cnt = 64;
      // an item is read by the MMA thread, 8 softmax warps and those two
      if (i >= C::B_ITEM_EMPTY && i < C::B_ITEM_EMPTY + NITEM) cnt = 11;
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
  const int total = (int)min((long long)tp[R] * p.num_kv_heads, (long long)0x7fffffff);
  volatile int* ring_s = reinterpret_cast<volatile int*>(sm.base + C::OFF_RING);
  // the k-th item of this CTA (total: no more); by a whole warp
  auto read_item = [&](int k) -> int {
    const int slot = k % NITEM;
    if (!wait_bar(sm, sm.bar(C::B_ITEM_FULL + slot), (uint32_t)(k / NITEM) & 1, p.err, 60))
      return total;
    const int i = ring_s[slot];
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(sm.bar(C::B_ITEM_EMPTY + slot));
    return i;
  };

  // Registers: 384 threads were launched with 168, 64512 in all; 256 go on with
  // 208 and 128 with 88, which is as many.
  if (warp >= PROD_WARP) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;\n");
    if (warp == PROD_WARP) {
      // ================= loads =================
      long long ns = 0;  // stages filled: K and V chunks in turn
      int nq = 0;        // q pairs
      for (int k = 0;; ++k) {
        const int slot = k % NITEM;
        if (!wait_bar(sm, sm.bar(C::B_ITEM_EMPTY + slot), ((uint32_t)(k / NITEM) & 1) ^ 1, p.err, 61))
          break;
        int i = 0;
        if (lane == 0) {
          const unsigned got = atomicAdd(p.next_item, 1u);
          i = got < (unsigned)total ? (int)got : total;
          ring_s[slot] = i;
          ptx::mbar_arrive(sm.bar(C::B_ITEM_FULL + slot));
        }
        i = __shfl_sync(0xffffffffu, i, 0);
        if (i >= total) break;
        const Item it = item_of<G>(i, tp, p);
        bool ok = true;
        for (int x = 0; x < 2 * it.n; ++x) {
          if (x == 1) {  // the q tiles, behind the first keys
            if (nq > 0 && !wait_bar(sm, sm.bar(C::B_Q_EMPTY), (nq - 1) & 1, p.err, 62)) {
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
          const int s = (int)(ns % NLOAD);
          const uint32_t ph = (uint32_t)(ns / NLOAD) & 1;
          const int key0 = (it.j0 + x / 2) * CHK;
          const int keys = min(CHK, it.kv_end - key0);
          const int nbox = (keys + p.box_tok - 1) >> p.log2_box;
          // blocks that lie before every window are not read
          const int box0 = max(0, it.kv_lo - key0) >> p.log2_box;
          const bool mine = lane >= box0 && lane < nbox;
          int phys = 0;
          if (mine)
            phys = __ldg(&p.block_tables[(int64_t)it.r * p.max_blocks +
                                         ((key0 + lane * p.box_tok) >> p.log2_bs)]);
          if (!wait_bar(sm, sm.bar(C::B_EMPTY + s), ph ^ 1, p.err, 63)) {
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
            if (!FP8) ptx::tma_load_4d(dst + HALF_B, tm, sm.bar(C::B_FULL + s), 64, it.g, off, phys);
          }
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
      if (lane == 0) {
        constexpr uint32_t kIdescBf16 = ptx::idesc_bf16_f32_ab(128, 128, false, false);
        constexpr uint32_t kIdescBf16T = ptx::idesc_bf16_f32_ab(128, 128, false, true);
        // f16 operands: format 0 in both fields
        constexpr uint32_t kFormat = (1u << 7) | (1u << 10);
        constexpr uint32_t IDESC_QK = FP8 ? kIdescBf16 & ~kFormat : kIdescBf16;
        constexpr uint32_t IDESC_PV = FP8 ? kIdescBf16T & ~kFormat : kIdescBf16T;
        long long ns = 0;            // stages before this item
        int nq = 0, nfix = 0;
        int np[2] = {0, 0}, ni[2] = {0, 0};  // PV products, items with some, of each tile
        bool ok = true;
        auto staged = [&](long long s) {  // chunk s is in shared memory, in 16 bits
          return FP8 ? wait_bar(sm, sm.bar(C::B_WIDE + (int)(s % NST)), (uint32_t)(s / NST) & 1, p.err, 64)
                     : wait_bar(sm, sm.bar(C::B_FULL + (int)(s % NST)), (uint32_t)(s / NST) & 1, p.err, 65);
        };
        auto release = [&](long long s) {
          ptx::tc_commit(sm.bar((FP8 ? C::B_WIDE_EMPTY : C::B_EMPTY) + (int)(s % NST)));
        };
        for (int k = 0; ok; ++k) {
          const int slot = k % NITEM;
          if (!wait_bar(sm, sm.bar(C::B_ITEM_FULL + slot), (uint32_t)(k / NITEM) & 1, p.err, 66)) break;
          const int i = ring_s[slot];
          ptx::mbar_arrive(sm.bar(C::B_ITEM_EMPTY + slot));
          if (i >= total) break;
          const Item it = item_of<G>(i, tp, p);
          if (it.n == 0) continue;
          ok = wait_bar(sm, sm.bar(C::B_Q_FULL), nq & 1, p.err, 67);
          if (FP8)
            for (int t = 0; t < 2; ++t)
              ok = ok && wait_bar(sm, sm.bar(C::B_Q_READY + t), nq & 1, p.err, 68);
          for (int c = 0; c <= it.n && ok; ++c) {
  #pragma unroll
            for (int t = 0; t < 2; ++t) {
              const int pc = c - 1;
              if (pc >= it.a[t] && pc < it.b[t]) {  // P V of the chunk before
                const long long s = ns + 2 * pc + 1;
                ok = ok && staged(s);
                const bool first = t == 0 || !(pc >= it.a[0] && pc < it.b[0]);
                if (!FP8 && first && ragged(it, pc)) {
                  ok = ok && wait_bar(sm, sm.bar(C::B_FIX + nfix % NFIX), (uint32_t)(nfix / NFIX) & 1,
                                      p.err, 69);
                  ++nfix;
                }
                if (pc == it.a[t] && ni[t] > 0)
                  ok = ok && wait_bar(sm, sm.bar(C::B_O_EMPTY + t), (ni[t] - 1) & 1, p.err, 70);
                ok = ok && wait_bar(sm, sm.bar(C::B_P_FULL + t), np[t] & 1, p.err, 71);
                if (!ok) break;
                ptx::tc_fence_after();
                const uint32_t v = sm.base_u32 + C::OFF_ST + (int)(s % NST) * TILE_B;
  #pragma unroll
                for (int kk = 0; kk < CHK / 16; ++kk)
                  mma_from_tmem(tmem + O_COL + 128 * t, tmem + S_COL + 128 * t + 8 * kk,
                                ptx::smem_desc_sw128(v + kk * 2048, HALF_B, 1024), IDESC_PV,
                                pc > it.a[t] || kk > 0);
                ptx::tc_commit(sm.bar(C::B_O_FULL + t));
                ++np[t];
                if (t == 1 || !(pc >= it.a[1] && pc < it.b[1])) release(s);
              }
              if (c >= it.a[t] && c < it.b[t]) {  // Q K^T, over the weights just used
                const long long s = ns + 2 * c;
                ok = ok && staged(s);
                if (!ok) break;
                ptx::tc_fence_after();
                const uint32_t q = sm.base_u32 + C::OFF_Q + t * TILE_B;
                const uint32_t kb = sm.base_u32 + C::OFF_ST + (int)(s % NST) * TILE_B;
  #pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                  const uint32_t at = (kk >> 2) * HALF_B + (kk & 3) * 32;
                  ptx::tc_mma_f16(tmem + S_COL + 128 * t, ptx::smem_desc_sw128(q + at, 16, 1024),
                                  ptx::smem_desc_sw128(kb + at, 16, 1024), IDESC_QK, kk > 0);
                }
                ptx::tc_commit(sm.bar(C::B_S_FULL + t));
                if (t == 1 || !(c >= it.a[1] && c < it.b[1])) release(s);
              }
            }
            if (c == it.n - 1 && ok) ptx::tc_commit(sm.bar(C::B_Q_EMPTY));
          }
          if (!ok) break;
          ns += 2 * it.n;
          ++nq;
  #pragma unroll
          for (int t = 0; t < 2; ++t) ni[t] += it.b[t] > it.a[t];
        }
        // drain: every product and commit issued must have landed before the end
  #pragma unroll
        for (int t = 0; t < 2; ++t)
          if (np[t] > 0) drain_bar(sm.bar(C::B_O_FULL + t), (np[t] - 1) & 1);
        if (nq > 0) drain_bar(sm.bar(C::B_Q_EMPTY), (nq - 1) & 1);
        for (long long l = ns > NST ? ns - NST : 0; l < ns; ++l)
          drain_bar(sm.bar((FP8 ? C::B_WIDE_EMPTY : C::B_EMPTY) + (int)(l % NST)), (uint32_t)(l / NST) & 1);
      }
    } else {
      // ================= widening (e4m3) and zeroing =================
      const int x = tid - FIX_WARP * 32;
      long long ns = 0;
      int nfix = 0;
      for (int k = 0;; ++k) {
        const int i = read_item(k);
        if (i >= total) break;
        const Item it = item_of<G>(i, tp, p);
        bool ok = true;
        if constexpr (FP8) {
          for (int st = 0; st < 2 * it.n && ok; ++st, ++ns) {
            const int s = (int)(ns % NLOAD), w = (int)(ns % NST);
            const int key0 = (it.j0 + st / 2) * CHK;
            ok = wait_bar(sm, sm.bar(C::B_FULL + s), (uint32_t)(ns / NLOAD) & 1, p.err, 72) &&
                 wait_bar(sm, sm.bar(C::B_WIDE_EMPTY + w), ((uint32_t)(ns / NST) & 1) ^ 1, p.err, 73);
            __syncwarp();
            if (!ok) break;
            const unsigned char* raw = sm.base + C::OFF_RAW + s * RAW_B;
            unsigned char* wide = sm.base + C::OFF_ST + w * TILE_B;
            // 16 elements at a time; 8 lanes take 4 pieces of two neighbouring
            // rows, whose stores then fall in different banks
  #pragma unroll 4
            for (int u = x; u < CHK * 8; u += 64) {
              const int pc = u & 3, row = ((u >> 3) & ~1) | ((u >> 2) & 1), half = (u >> 3) & 1;
              const int piece = 4 * half + pc;
              uint4 v = *reinterpret_cast<const uint4*>(raw + row * 128 + ((piece ^ (row & 7)) << 4));
              if (key0 + row < it.kv_lo || key0 + row >= it.kv_end) v = make_uint4(0, 0, 0, 0);
              unsigned char* to = wide + half * HALF_B + row * 128;
              *reinterpret_cast<uint4*>(to + (((2 * pc) ^ (row & 7)) << 4)) =
                  make_uint4(widen((uint16_t)v.x), widen((uint16_t)(v.x >> 16)),
                             widen((uint16_t)v.y), widen((uint16_t)(v.y >> 16)));
              *reinterpret_cast<uint4*>(to + (((2 * pc + 1) ^ (row & 7)) << 4)) =
                  make_uint4(widen((uint16_t)v.z), widen((uint16_t)(v.z >> 16)),
                             widen((uint16_t)v.w), widen((uint16_t)(v.w >> 16)));
            }
            ptx::fence_proxy_async_smem();
            ptx::mbar_arrive(sm.bar(C::B_WIDE + w));
            ptx::mbar_arrive(sm.bar(C::B_EMPTY + s));
          }
        } else {
          // Every chunk is waited for and let go, whether zeroed or not, so that
          // these warps are never a stage's whole round ahead or behind.
          for (int st = 0; st < 2 * it.n && ok; ++st, ++ns) {
            const int s = (int)(ns % NST), c = st / 2;
            ok = wait_bar(sm, sm.bar(C::B_FULL + s), (uint32_t)(ns / NST) & 1, p.err, 74);
            __syncwarp();
            if (!ok) break;
            if (!(st & 1) || !ragged(it, c)) {
              if (lane == 0) ptx::mbar_arrive(sm.bar(C::B_EMPTY + s));
              continue;
            }
            unsigned char* v = sm.base + C::OFF_ST + s * TILE_B;
            const int key0 = (it.j0 + c) * CHK;
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
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;\n");
    // ================= softmax and epilogue =================
    const int t = warp >> 2;
    const int row = tid & 127, tok = row / G, hd = row % G;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_col = tmem + lane_base + S_COL + 128 * t;
    const uint32_t o_col = tmem + lane_base + O_COL + 128 * t;
    const float ksc = FP8 ? __ldg(p.k_scale) : 1.f;
    const float vsc = FP8 ? __ldg(p.v_scale) : 1.f;
    int nc = 0, nq = 0;  // chunks of this tile, items with chunks
    bool ok = true;
    for (int k = 0; ok; ++k) {
      const int i = read_item(k);
      if (i >= total) break;
      const Item it = item_of<G>(i, tp, p);
      const int ntok = t ? it.ntok[1] : it.ntok[0];
      const int first = t ? it.a[1] : it.a[0], last = t ? it.b[1] : it.b[0];
      const bool row_ok = tok < ntok;
      const int pos = it.pos + t * MQ + tok;
      __nv_bfloat16* orow = p.out + ((int64_t)(it.q0 + t * MQ + tok) * p.num_heads + it.g * G + hd) * D;
      if (it.n == 0) {
        if (row_ok) {
#pragma unroll
          for (int c = 0; c < 16; ++c) reinterpret_cast<uint4*>(orow)[c] = make_uint4(0, 0, 0, 0);
        }
        continue;
      }
      float rs = p.scale_log2;
      if constexpr (FP8) {
        // the row of q as f16, in place, under a power of two of its own
        ok = wait_bar(sm, sm.bar(C::B_Q_FULL), nq & 1, p.err, 75);
        __syncwarp();
        if (!ok) break;
        unsigned char* qrow = sm.base + C::OFF_Q + t * TILE_B + row * 128;
        float amax = 0.f;
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const uint4 v = *reinterpret_cast<const uint4*>(qrow + (c >> 3) * HALF_B + ((c & 7) << 4));
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(w[e])), fabsf(bf16_hi(w[e]))));
        }
        // (kept within the normal floats; an infinite or NaN q stays what it is)
        const int e2 = min(max((int)(__float_as_uint(amax) >> 23), 1), 253) - 127;
        const float inv = __int_as_float((127 - e2) << 23);
        rs *= ksc * __int_as_float((127 + e2) << 23);
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          uint4* at = reinterpret_cast<uint4*>(qrow + (c >> 3) * HALF_B + ((c & 7) << 4));
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
      const float slope =
          p.mod.slopes ? __ldg(&p.mod.slopes[it.g * G + hd]) * 1.4426950408889634f : 0.f;
      const int pos0 = it.pos + t * MQ;  // of the tile's first token
      float m_ref = -INFINITY;
      float2 l2 = make_float2(0.f, 0.f);
      for (int c = first; c < last; ++c, ++nc) {
        float2 s[64];
        ok = wait_bar(sm, sm.bar(C::B_S_FULL + t), nc & 1, p.err, 76);
        __syncwarp();
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        {
          float v[4][32];
#pragma unroll
          for (int h = 0; h < 4; ++h) ptx::tmem_ld_x32(s_col + 32 * h, v[h]);
          ptx::tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 64; ++e) s[e] = make_float2(v[e >> 4][2 * (e & 15)], v[e >> 4][2 * (e & 15) + 1]);
        }
        const int key0 = (it.j0 + c) * CHK;
        change_scores(s, rs, p.mod, slope, (float)(pos - key0));
        // every row of a full tile sees every key of a chunk between the last
        // token's window and the first token
        const bool whole = ntok == MQ && key0 + CHK <= pos0 + 1 &&
                           (p.mod.window <= 0 || key0 >= pos0 + MQ - p.mod.window);
        if (!whole) {
          const int kf = low - key0;
          const unsigned kn = (unsigned)max(0, lim - max(low, 0));
#pragma unroll
          for (int e = 0; e < 64; ++e) {
            if ((unsigned)(2 * e - kf) >= kn) s[e].x = -INFINITY;
            if ((unsigned)(2 * e + 1 - kf) >= kn) s[e].y = -INFINITY;
          }
        }
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int e = 0; e < 64; ++e) m4[e & 3] = fmaxf(m4[e & 3], fmaxf(s[e].x, s[e].y));
        const float cm = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        float alpha = 1.f;
        if (cm > m_ref + kRescaleLog2) {
          if (m_ref != -INFINITY) alpha = fast_exp2(m_ref - cm);
          m_ref = cm;
        }
        if (__any_sync(0xffffffffu, alpha != 1.f)) {  // (never at an item's first chunk)
          ok = wait_bar(sm, sm.bar(C::B_O_FULL + t), (nc - 1) & 1, p.err, 77);
          __syncwarp();
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            float o[32];
            ptx::tmem_ld_x32(o_col + 32 * h, o);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] *= alpha;
            ptx::tmem_st_x32(o_col + 32 * h, o);
          }
          ptx::tmem_st_wait();
          l2.x *= alpha;
          l2.y *= alpha;
        }
        const float2 bias = both(C::kRaise - (m_ref == -INFINITY ? 0.f : m_ref));
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float w[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const float2 y = add2(s[32 * h + e], bias);
            const float2 q = make_float2(fast_exp2(y.x), fast_exp2(y.y));
            sum[e & 1] = add2(sum[e & 1], q);  // before the 16-bit rounding the MMA sees
            w[e] = __uint_as_float(pack2<FP8>(q.x, q.y));
          }
          ptx::tmem_st_x32(s_col + 32 * h, w);
        }
        l2 = add2(l2, add2(sum[0], sum[1]));
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
        ptx::mbar_arrive(sm.bar(C::B_P_FULL + t));
      }
      if (!ok) break;
      if (first == last) continue;  // a tile without tokens
      ok = wait_bar(sm, sm.bar(C::B_O_FULL + t), (nc - 1) & 1, p.err, 78);
      __syncwarp();
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      ptx::tc_fence_after();
      const float l = l2.x + l2.y;
      const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        float o[32];
        ptx::tmem_ld_x32(o_col + 32 * h, o);
        ptx::tmem_ld_wait();
        if (row_ok) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[e] = pack_bf16x2_rn(o[8 * c + 2 * e] * inv * vsc, o[8 * c + 2 * e + 1] * inv * vsc);
            reinterpret_cast<uint4*>(orow)[4 * h + c] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
        __syncwarp();
      }
      ptx::tc_fence_before();
      ptx::mbar_arrive(sm.bar(C::B_O_EMPTY + t));
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

template <int G, bool FP8>
cudaError_t launch_g(const Params& prm, const CUtensorMap& mk, const CUtensorMap& mv,
                     const CUtensorMap& mq, int num_ctas, cudaStream_t stream) {
  const cudaError_t e = allow_large<prefill_scored_kernel<G, FP8>>();
  if (e != cudaSuccess) return e;
  return launch_dependent<prefill_scored_kernel<G, FP8>>(dim3(num_ctas), dim3(NTHREADS),
                                                         Cfg<FP8>::SMEM_BYTES, stream, 1, mk, mv,
                                                         mq, prm);
}

template <bool FP8>
cudaError_t launch_f(const Params& prm, const CUtensorMap& mk, const CUtensorMap& mv,
                     const CUtensorMap& mq, int group, int num_ctas, cudaStream_t stream) {
  switch (group) {
    case 1: return launch_g<1, FP8>(prm, mk, mv, mq, num_ctas, stream);
    case 2: return launch_g<2, FP8>(prm, mk, mv, mq, num_ctas, stream);
    case 4: return launch_g<4, FP8>(prm, mk, mv, mq, num_ctas, stream);
    case 8: return launch_g<8, FP8>(prm, mk, mv, mq, num_ctas, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace ps

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
  prm.next_item = reinterpret_cast<unsigned*>(static_cast<char*>(a.workspace) + 4);
  const cudaError_t ez = cudaMemsetAsync(prm.next_item, 0, sizeof(unsigned), stream);
  if (ez != cudaSuccess) return ez;
  prm.num_seqs = a.num_seqs;
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
  return a.fp8 ? launch_f<true>(prm, mk, mv, mq, group, a.num_ctas, stream)
               : launch_f<false>(prm, mk, mv, mq, group, a.num_ctas, stream);
}

}  // namespace pa
