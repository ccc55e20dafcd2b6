// Decode attention with changed scores: capped, biased by distance, kept to
// a window; over a bf16 cache, an e4m3 one, or 8-bit rows with a unit for
// each token and head.
//
// For a row at position i of its sequence (its newest token: i = n - 1) and
// KV head h,
//   s_j = scale q . k_j;  s_j <- cap tanh(s_j / cap);  s_j <- s_j - slope |i - j|
//   out = softmax(s_j, j in [i - window + 1, end)) V
// for the head's G query heads together, so that each K and V byte is read
// once.  end is i + 1, or the sequence's prefix for a row inside it.
//
// Bound: the visible tokens' bytes (at G = 4, 4 flop a byte in bf16, 8 in 8
// bits).  Each warp streams 16-token chunks through a cp.async ring of its own
// and keeps its own softmax state, as in the decode over listed blocks:
//   S^T [16 tokens x 8 columns] = K q^T     (mma m16n8k16, K by ldmatrix)
//   O^T [D x 8 columns] += V^T P^T          (V by ldmatrix.trans)
// with the query heads in the 8 columns; for G <= 4 columns 4..7 repeat the
// heads and carry what rounding takes from P, for G = 8 a second MMA does.
// 8-bit elements are widened to f16 in registers (exact); q then enters in
// f16 under a power of two per head, and P is raised by 2^14 (f16 ends at
// 2^-24).  The unit of an 8-bit row multiplies its logit, and its weight in
// P V, relative to the largest unit the warp has met (a running maximum like
// the softmax's), so that f16 holds those products whatever the units' size.
//
// The cap's tanh(u) is 1 - 2 / (1 + e^2u): one exponential and one reciprocal,
// off by about 2^-22 of the cap.
//
// Work split: a unit is a (row, KV head); its visible tokens are cut into
// steps of one chunk per warp, and the steps of all units in a row, K in all,
// into equal ranges, one for each CTA that runs at once, whatever the lengths.
// Loads run ahead across the ends of units.  A CTA's range splits at most two
// units (the one it starts in, the one it ends in): their partial sums go to
// the workspace, and the last CTA to arrive at a unit adds them up in order of
// their CTAs, so the result does not depend on who is last.  Where units are
// many times the CTAs (kWholeUnits), each CTA takes one whole unit.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "launch.cuh"
#include "mma_ptx.cuh"
#include "pa_device.cuh"
#include "pa_kernels.cuh"
#include "tc_ptx.cuh"
#include "tc_sched.cuh"

namespace pa {

namespace {

constexpr int kChunk = 16;        // tokens a warp handles at a time
constexpr int kCtasPerSm = 2;     // what registers and shared memory are kept to
constexpr int kWholeUnits = 6;    // units per CTA from which none is split
constexpr int kMinSteps = 2;      // steps of a CTA at least, where units are split

template <int D, KvFormat F>
struct Cfg {
  static constexpr int kRow = D * (F == kBf16 ? 2 : 1);  // bytes of a token's channels
  static constexpr int kPieces = kRow / 16;
  static constexpr int kTile = kChunk * kRow;  // K (or V) bytes of a chunk
  static constexpr int kWarps = F == kBf16 ? 4 : 8;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kStages = F == kBf16 ? 3 : 2;
  static constexpr int kUnits = F == kInt8 ? 2 * kChunk * 4 : 0;  // bytes of a chunk's units
  static constexpr int kStage = 2 * kTile + kUnits;
  static constexpr int kRing = kWarps * kStages * kStage;
  // 16-byte pieces of a tile's row, permuted so that 8 rows' pieces of one
  // column (ldmatrix) fall in different banks
  static __device__ __forceinline__ int swizzle(int row, int piece) {
    if constexpr (kPieces >= 8)
      return piece ^ (row & 7);
    else
      return piece ^ ((row >> 1) & 3);
  }
};

// The two codes of a 16-bit half, low byte first, as an f16 pair: 1024 + 128 +
// code has the biased code in its low bits.
__device__ __forceinline__ uint32_t widen_int8(uint32_t codes, uint32_t pick) {
  const uint32_t w = __byte_perm(codes ^ 0x80808080u, 0x64646464u, pick);
  const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&w), __float2half2_rn(1152.f));
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Bytes 0 and 1 (hi false) or 2 and 3 of a word of 8-bit elements.
template <KvFormat F>
__device__ __forceinline__ uint32_t widen_half(uint32_t w, bool hi) {
  if constexpr (F == kInt8)
    return widen_int8(w, hi ? 0x4342 : 0x4140);
  else
    return widen((uint16_t)(hi ? w >> 16 : w));
}
// Bytes 0 and 2 (odd false) or 1 and 3.
template <KvFormat F>
__device__ __forceinline__ uint32_t widen_alternate(uint32_t w, bool odd) {
  if constexpr (F == kInt8)
    return widen_int8(w, odd ? 0x4341 : 0x4240);
  else
    return widen((uint16_t)__byte_perm(w, 0, odd ? 0x4431 : 0x4420));
}

// The factor of a part whose running max is m under the whole's max; 1 where
// neither has a token, so that a NaN among the logits still reaches the sums.
__device__ __forceinline__ float weight(float m, float whole) {
  return whole == -INFINITY ? 1.f : fast_exp2(m - whole);
}
// What sums over 8-bit rows are relative to at least: the smallest normal
// float, whose reciprocal is finite.
constexpr float kLeastUnit = 1.17549435e-38f;
// Units are >= 0, so they order like their bits, NaN above all.
__device__ __forceinline__ float larger_unit(float a, float b) {
  return __uint_as_float(max(__float_as_uint(a), __float_as_uint(b)));
}

// A row's sequence, its position and the keys it sees, [first, end).
struct Row {
  int seq;  // -1: none
  int pos, first, end;
};
__device__ __forceinline__ Row row_of(const ScoredParams& p, int row) {
  Row r;
  const int64_t room = (int64_t)p.max_blocks << p.log2_block_size;
  int64_t end, pos;
  if (!p.starts) {
    r.seq = row;
    end = p.lens[row];
    pos = end - 1;
  } else {
    int lo = 0, hi = p.num_seqs;  // the last sequence that starts at or before the row
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.starts[mid] <= row) lo = mid;
      else hi = mid;
    }
    const int64_t s0 = p.starts[lo], s1 = p.starts[lo + 1], len = p.lens[lo];
    r.seq = row >= s0 && row < s1 ? lo : -1;
    pos = len - (s1 - s0) + (row - s0);
    end = pos + 1;
    if (s1 - s0 > len) end = 0;  // more new tokens than the sequence has
    if (p.mod.prefix_lens && end > 0) {
      const int64_t prefix = min((int64_t)p.mod.prefix_lens[lo], len);
      if (pos < prefix) end = prefix;
    }
  }
  end = r.seq < 0 ? 0 : min(end, room);
  r.pos = (int)pos;
  r.end = (int)max(end, (int64_t)0);
  r.first = p.mod.window > 0 ? (int)max((int64_t)0, pos - p.mod.window + 1) : 0;
  r.first = min(r.first, r.end);
  return r;
}
// Tokens are visited from a multiple of the chunk on.
__device__ __forceinline__ int first_chunk(const Row& r) { return r.first & ~(kChunk - 1); }
template <int kStep>
__device__ __forceinline__ int steps_of(const Row& r) {
  const int n = r.end - first_chunk(r);
  return n <= 0 ? 1 : (n + kStep - 1) / kStep;  // a row without keys has its zeros written
}

// What a warp knows of a chunk that it has asked for.
struct __align__(16) Chunk {
  int row, kvh, tok, first;
  int seen, pos, flags, steps;  // seen: a bit per token; steps: of the unit
};
enum { kOpens = 1, kCloses = 2, kNobody = 4 };

template <int D, int G, KvFormat F>
__global__ void __launch_bounds__(Cfg<D, F>::kThreads, kCtasPerSm)
    decode_scored_kernel(const __grid_constant__ ScoredParams p, bool whole_units) {
  using C = Cfg<D, F>;
  constexpr bool F16 = F != kBf16;
  constexpr int kWarps = C::kWarps, kThreads = C::kThreads;
  constexpr int kStep = kWarps * kChunk;  // tokens of a step
  constexpr int kSteps = D / 16;          // k16 steps of q . k; m16 tiles of O^T
  constexpr int kColHeads = G <= 4 ? 4 : 8;
  constexpr int kPart = G * (D + 2) + 1;  // a partial: sums, then max and sum per head, unit
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Chunk s_chunk[kWarps][C::kStages];
  __shared__ float s_o[kWarps][kColHeads][D];
  __shared__ float s_ml[kWarps][kColHeads][2];
  __shared__ float s_unit[kWarps];
  __shared__ long long s_sum[kWarps], s_before;
  __shared__ int s_row, s_last;
  ptx::grid_dependency_wait();
  ptx::grid_launch_dependents();
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int g = lane / 4, c = lane % 4;  // MMA fragment coordinates
  const int hkv = p.num_kv_heads;

  // ---- this CTA's range of steps: [lo, hi) of K, from step `at` of a unit ----
  long long K = 0, lo = 0, hi = 0;
  int ctas = 1, row = 0, kvh = 0, at = 0;
  Row cur;
  if (whole_units) {
    row = blockIdx.x / hkv;
    kvh = blockIdx.x - row * hkv;
    cur = row_of(p, row);
    hi = K = steps_of<kStep>(cur);
  } else {
    long long sum = 0;
    for (int r = tid; r < p.num_rows; r += kThreads) sum += steps_of<kStep>(row_of(p, r));
    for (int d = 16; d; d /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (lane == 0) s_sum[warp] = sum;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) K += s_sum[w];
    K *= hkv;
    ctas = (int)min((long long)gridDim.x, max(1ll, K / kMinSteps));
    if ((int)blockIdx.x >= ctas) return;
    lo = tc::range_lo(blockIdx.x, K, ctas);
    hi = tc::range_lo(blockIdx.x + 1, K, ctas);
    // the row that step lo lies in
    long long before = 0;
    for (int base = 0; base < p.num_rows; base += kThreads) {
      const int r = base + tid;
      const long long n = r < p.num_rows ? (long long)steps_of<kStep>(row_of(p, r)) * hkv : 0;
      long long incl = n;
      for (int d = 1; d < 32; d *= 2) {
        const long long o = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += o;
      }
      __syncthreads();  // s_sum is free
      if (lane == 31) s_sum[warp] = incl;
      if (tid == 0) s_row = -1;
      __syncthreads();
      long long mine = before + incl - n, end = before;
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) mine += s_sum[w];
        end += s_sum[w];
      }
      if (mine <= lo && lo < mine + n) {
        s_row = r;
        s_before = mine;
      }
      __syncthreads();
      if (s_row >= 0) break;
      before = end;
    }
    row = s_row;
    cur = row_of(p, row);
    const int n = steps_of<kStep>(cur);
    const long long in = lo - s_before;
    kvh = (int)(in / n);
    at = (int)(in - (long long)kvh * n);
  }
  const int total = (int)(hi - lo);

  const uint32_t ring = smem_u32(smem) + warp * C::kStages * C::kStage;
  const int64_t stride = (int64_t)hkv * C::kRow;  // between tokens
  const int lb = p.log2_block_size;
  float ks = 1.f, post = 1.f;  // e4m3's scales
  if constexpr (F == kE4m3) {
    ks = *p.k_scale;
    post = *p.v_scale;
  }

  // ---- loads: the chunk of step `asked`, and the slot of the one behind it ----
  int asked = 0;
  auto slot_of = [&]() -> int {  // of this lane's token of the cursor's chunk
    const int tok = first_chunk(cur) + (at * kWarps + warp) * kChunk + (lane & 15);
    if (asked >= total || tok < cur.first || tok >= cur.end) return -1;
    const int phys = p.block_tables[(int64_t)cur.seq * p.max_blocks + (tok >> lb)];
    return (unsigned)phys < (unsigned)p.num_blocks ? (phys << lb) + (tok & ((1 << lb) - 1)) : -1;
  };
  int slot = slot_of();
  auto load = [&]() {
    if (asked < total) {
      const int n = steps_of<kStep>(cur);
      const int st = asked % C::kStages;
      const uint32_t stage = ring + st * C::kStage;
      const unsigned seen = __ballot_sync(0xffffffffu, slot >= 0) & 0xffff;
      if (lane == 0) {
        Chunk& k = s_chunk[warp][st];
        k.row = row;
        k.kvh = kvh;
        k.tok = first_chunk(cur) + (at * kWarps + warp) * kChunk;
        k.first = cur.first;
        k.seen = (int)seen;
        k.pos = cur.pos;
        k.steps = n;
        k.flags = (asked == 0 || at == 0 ? kOpens : 0) |
                  (asked == total - 1 || at == n - 1 ? kCloses : 0) |
                  // a row of no sequence: nothing is written
                  (cur.seq < 0 ? kNobody : 0);
      }
      const uint8_t* kbase = static_cast<const uint8_t*>(p.k_cache) + (int64_t)kvh * C::kRow;
      const uint8_t* vbase = static_cast<const uint8_t*>(p.v_cache) + (int64_t)kvh * C::kRow;
      constexpr int kRowsPer = 32 / C::kPieces;  // tokens per instruction
      const int piece = lane % C::kPieces;
#pragma unroll
      for (int r = 0; r < kChunk / kRowsPer; ++r) {
        const int t = r * kRowsPer + lane / C::kPieces;
        const int s = __shfl_sync(0xffffffffu, slot, t);
        const int64_t from = (int64_t)max(s, 0) * stride + piece * 16;
        const uint32_t dst = stage + t * C::kRow + C::swizzle(t, piece) * 16;
        cp_async_16(dst, kbase + from, s >= 0 ? 16 : 0);  // zeros where there is no token
        cp_async_16(dst + C::kTile, vbase + from, s >= 0 ? 16 : 0);
      }
      if constexpr (F == kInt8) {  // units: the keys' by lanes 0..15, the values' by 16..31
        const float* u = lane < 16 ? p.k_scale : p.v_scale;
        const uint32_t dst = stage + 2 * C::kTile + lane * 4;
        if (slot >= 0)
          cp_async_4(dst, u + (int64_t)slot * hkv + kvh);
        else
          asm volatile("st.shared.f32 [%0], %1;\n" ::"r"(dst), "f"(0.f) : "memory");
      }
      // the next step's cursor
      ++asked;
      if (++at == n) {
        at = 0;
        if (++kvh == hkv) {
          kvh = 0;
          ++row;
          if (asked < total) cur = row_of(p, row);
        }
      }
      slot = slot_of();
    }
    cp_async_commit();
  };

  // ---- a unit's queries, as MMA operand B: column `col` is query head col
  // (mod 4 when G <= 4); what its logits are multiplied by; its slopes ----
  const int qh = g % kColHeads;
  uint2 qw[kSteps];
  uint32_t qb[kSteps][2];
  float f0 = 0.f, f1 = 0.f, slope0 = 0.f, slope1 = 0.f;
  auto fetch_q = [&](int unit_row, int unit_kvh) {
    const int64_t unit = (int64_t)unit_row * hkv + unit_kvh;
    const __nv_bfloat16* q = p.q + (unit * G + qh) * D;
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      qw[k] = make_uint2(0, 0);
      if (qh < G) {
        if (F16) {
          qw[k] = *reinterpret_cast<const uint2*>(q + 16 * k + 4 * c);
        } else {
          qw[k].x = *reinterpret_cast<const uint32_t*>(q + 16 * k + 2 * c);
          qw[k].y = *reinterpret_cast<const uint32_t*>(q + 16 * k + 8 + 2 * c);
        }
      }
    }
    if (p.mod.slopes) {
      const int h0 = (2 * c) % kColHeads, h1 = (2 * c + 1) % kColHeads;
      constexpr float kLog2e = 1.4426950408889634f;
      slope0 = h0 < G ? p.mod.slopes[unit_kvh * G + h0] * kLog2e : 0.f;
      slope1 = h1 < G ? p.mod.slopes[unit_kvh * G + h1] * kLog2e : 0.f;
    }
  };
  auto place_q = [&]() {
    f0 = f1 = p.scale_log2;
    if constexpr (F16) {
      float amax = 0.f;
#pragma unroll
      for (int k = 0; k < kSteps; ++k)
        amax = fmaxf(amax, fmaxf(fmaxf(fabsf(bf16_lo(qw[k].x)), fabsf(bf16_hi(qw[k].x))),
                                 fmaxf(fabsf(bf16_lo(qw[k].y)), fabsf(bf16_hi(qw[k].y)))));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      // 2^floor(log2 amax); kept within the normal floats so that its
      // reciprocal is exact (an infinite or NaN q stays what it is)
      const int e = min(max((int)(__float_as_uint(amax) >> 23), 1), 253) - 127;
      const float q_scale = __int_as_float((127 + e) << 23), inv = __int_as_float((127 - e) << 23);
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        qb[k][0] = pack2<true>(bf16_lo(qw[k].x) * inv, bf16_hi(qw[k].x) * inv);
        qb[k][1] = pack2<true>(bf16_lo(qw[k].y) * inv, bf16_hi(qw[k].y) * inv);
      }
      f0 *= ks * __shfl_sync(0xffffffffu, q_scale, 4 * (2 * c));
      f1 *= ks * __shfl_sync(0xffffffffu, q_scale, 4 * (2 * c + 1));
    } else {
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        qb[k][0] = qw[k].x;
        qb[k][1] = qw[k].y;
      }
    }
  };

  float o[kSteps][4];
  float m0, m1, l0, l1;
  float unit_max, unit_inverse;  // int8: the largest unit of a value row so far
  auto open = [&]() {
#pragma unroll
    for (int i = 0; i < kSteps; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    m0 = m1 = -INFINITY;
    l0 = l1 = 0.f;
    unit_max = kLeastUnit;
    unit_inverse = 1.f / kLeastUnit;
  };

  fetch_q(row, kvh);
#pragma unroll
  for (int s = 0; s < C::kStages - 1; ++s) load();
  for (int it = 0; it < total; ++it) {
    load();
    cp_async_wait<C::kStages - 1>();
    __syncwarp();
    const Chunk ch = s_chunk[warp][it % C::kStages];
    if (ch.flags & kOpens) {
      place_q();
      open();
    }
    const uint32_t kt = ring + (it % C::kStages) * C::kStage;
    const uint32_t vt = kt + C::kTile;
    if (ch.seen) {
      float s[4] = {0.f, 0.f, 0.f, 0.f};
      {
        const int r = (lane & 7) + ((lane >> 3) & 1) * 8;
        const uint32_t base = kt + r * C::kRow;
        if constexpr (F16) {
#pragma unroll
          for (int k = 0; k < kSteps; k += 2) {
            uint32_t w[4];
            ldmatrix_x4(w, base + C::swizzle(r, k + (lane >> 4)) * 16);
#pragma unroll
            for (int h = 0; h < 2; ++h) {  // the two 16-channel pieces
              const uint32_t x = w[2 * h], y = w[2 * h + 1];
              const uint32_t a[4] = {widen_half<F>(x, false), widen_half<F>(y, false),
                                     widen_half<F>(x, true), widen_half<F>(y, true)};
              mma16816<true>(s, a, qb[k + h][0], qb[k + h][1]);
            }
          }
        } else {
#pragma unroll
          for (int k = 0; k < kSteps; ++k) {
            uint32_t a[4];
            ldmatrix_x4(a, base + C::swizzle(r, 2 * k + (lane >> 4)) * 16);
            mma16816<false>(s, a, qb[k][0], qb[k][1]);
          }
        }
      }
      // tokens g and g + 8 of the chunk, columns 2c and 2c + 1
      const int t0 = ch.tok + g, t1 = t0 + 8;
      float x[4] = {s[0] * f0, s[1] * f1, s[2] * f0, s[3] * f1};
      float vu0 = 1.f, vu1 = 1.f;
      if constexpr (F == kInt8) {
        const float* u = reinterpret_cast<const float*>(
            smem + (warp * C::kStages + it % C::kStages) * C::kStage + 2 * C::kTile);
        x[0] *= u[g];
        x[1] *= u[g];
        x[2] *= u[g + 8];
        x[3] *= u[g + 8];
        vu0 = u[16 + g];
        vu1 = u[16 + g + 8];
      }
      if (p.mod.cap_log2 > 0.f) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          x[i] = p.mod.cap_log2 *
                 (1.f - 2.f * fast_reciprocal(1.f + fast_exp2(x[i] * p.mod.inv_cap_log2)));
      }
      if (p.mod.slopes) {
        const float d0 = (float)abs(ch.pos - t0), d1 = (float)abs(ch.pos - t1);
        x[0] -= slope0 * d0;
        x[1] -= slope1 * d0;
        x[2] -= slope0 * d1;
        x[3] -= slope1 * d1;
      }
      const bool in0 = ch.seen >> g & 1, in1 = ch.seen >> (g + 8) & 1;
      const float x00 = in0 ? x[0] : -INFINITY, x01 = in0 ? x[1] : -INFINITY;
      const float x10 = in1 ? x[2] : -INFINITY, x11 = in1 ? x[3] : -INFINITY;
      float n0 = fmaxf(x00, x10), n1 = fmaxf(x01, x11);
#pragma unroll
      for (int d = 4; d < 32; d *= 2) {
        n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, d));
        n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, d));
      }
      n0 = fmaxf(n0, m0);
      n1 = fmaxf(n1, m1);
      float grown = unit_max;
      if constexpr (F == kInt8) {
        const uint32_t most =
            __reduce_max_sync(0xffffffffu, max(__float_as_uint(vu0), __float_as_uint(vu1)));
        grown = larger_unit(unit_max, __uint_as_float(most));
      }
      if (__any_sync(0xffffffffu, n0 > m0 || n1 > m1) || (F == kInt8 && grown != unit_max)) {
        float a0 = m0 == -INFINITY ? 0.f : fast_exp2(m0 - n0);
        float a1 = m1 == -INFINITY ? 0.f : fast_exp2(m1 - n1);
        l0 *= a0;
        l1 *= a1;
        if constexpr (F == kInt8) {
          unit_inverse = 1.f / grown;
          a0 *= unit_max * unit_inverse;
          a1 *= unit_max * unit_inverse;
          unit_max = grown;
        }
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          o[i][0] *= a0;
          o[i][1] *= a1;
          o[i][2] *= a0;
          o[i][3] *= a1;
        }
        m0 = n0;
        m1 = n1;
      }
      constexpr float kRaise = F16 ? 16384.f : 1.f;  // the factor that P and its sum carry
      const float z0 = m0 == -INFINITY ? 0.f : m0, z1 = m1 == -INFINITY ? 0.f : m1;
      float p00 = fast_exp2(x00 - z0) * kRaise, p01 = fast_exp2(x01 - z1) * kRaise;
      float p10 = fast_exp2(x10 - z0) * kRaise, p11 = fast_exp2(x11 - z1) * kRaise;
      l0 += p00 + p10;
      l1 += p01 + p11;
      if constexpr (F == kInt8) {
        const float w0 = vu0 * unit_inverse, w1 = vu1 * unit_inverse;
        p00 *= w0;
        p01 *= w0;
        p10 *= w1;
        p11 *= w1;
      }
      uint32_t hi0 = pack2<F16>(p00, p01), hi1 = pack2<F16>(p10, p11);
      const float2 r0 = unpack2<F16>(hi0), r1 = unpack2<F16>(hi1);
      uint32_t lo0 = pack2<F16>(p00 - r0.x, p01 - r0.y), lo1 = pack2<F16>(p10 - r1.x, p11 - r1.y);
      if constexpr (G <= 4) {  // columns 4..7 carry the remainders
        if (c >= 2) {
          hi0 = lo0;
          hi1 = lo1;
        }
      }
      const uint32_t b0 = movmatrix_trans(hi0), b1 = movmatrix_trans(hi1);
      uint32_t d0 = 0, d1 = 0;
      if constexpr (G > 4) {
        d0 = movmatrix_trans(lo0);
        d1 = movmatrix_trans(lo1);
      }
      if constexpr (F16) {
        // a transposed 16-bit unit holds channels 2g and 2g + 1 of a token: the
        // even ones become row g of the tile, the odd ones row g + 8
        const int r = (lane & 7) + ((lane >> 3) & 1) * 8;
#pragma unroll
        for (int k = 0; k < kSteps; k += 2) {
          uint32_t w[4];
          ldmatrix_x4_trans(w, vt + r * C::kRow + C::swizzle(r, k + (lane >> 4)) * 16);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t x = w[2 * h], y = w[2 * h + 1];
            const uint32_t a[4] = {widen_alternate<F>(x, false), widen_alternate<F>(x, true),
                                   widen_alternate<F>(y, false), widen_alternate<F>(y, true)};
            mma16816<true>(o[k + h], a, b0, b1);
            if constexpr (G > 4) mma16816<true>(o[k + h], a, d0, d1);
          }
        }
      } else {
        const int r = (lane & 7) + (lane >> 4) * 8;
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          uint32_t a[4];
          ldmatrix_x4_trans(a, vt + r * C::kRow + C::swizzle(r, 2 * k + ((lane >> 3) & 1)) * 16);
          mma16816<false>(o[k], a, b0, b1);
          if constexpr (G > 4) mma16816<false>(o[k], a, d0, d1);
        }
      }
    }
    const bool closes = ch.flags & kCloses;
    if (closes && it + 1 < total) {  // the next unit's queries, while this one is added up
      const Chunk& k = s_chunk[warp][(it + 1) % C::kStages];
      fetch_q(k.row, k.kvh);
    }
    __syncwarp();  // the stage may be filled again
    if (!closes) continue;

    // ---- the piece is done: the warps' sums meet ----
#pragma unroll
    for (int d = 4; d < 32; d *= 2) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, d);
      l1 += __shfl_xor_sync(0xffffffffu, l1, d);
    }
    if constexpr (G <= 4) {
#pragma unroll
      for (int i = 0; i < kSteps; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[i][j] += __shfl_xor_sync(0xffffffffu, o[i][j], 2);
    }
    __syncthreads();  // the last piece's sums have been read
    if (2 * c < kColHeads) {
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int d0 = 16 * i + (F16 ? 2 * g : g), d1 = F16 ? d0 + 1 : d0 + 8;
        s_o[warp][2 * c][d0] = o[i][0];
        s_o[warp][2 * c + 1][d0] = o[i][1];
        s_o[warp][2 * c][d1] = o[i][2];
        s_o[warp][2 * c + 1][d1] = o[i][3];
      }
      if (g == 0) {
        s_ml[warp][2 * c][0] = m0;
        s_ml[warp][2 * c][1] = l0;
        s_ml[warp][2 * c + 1][0] = m1;
        s_ml[warp][2 * c + 1][1] = l1;
      }
    }
    if (lane == 0) s_unit[warp] = unit_max;
    __syncthreads();
    const int64_t unit = (int64_t)ch.row * hkv + ch.kvh;
    // the unit's steps in the order of all, [u0, u1)
    const int in = ch.tok - warp * kChunk - (ch.first & ~(kChunk - 1));  // tokens before this step
    const long long u0 = lo + it - in / kStep, u1 = u0 + ch.steps;
    const bool split = u0 < lo || u1 > hi;
    // CTA k's part of the unit: it goes on with the unit, or starts it
    auto part_of = [&](int k) -> float* {
      return p.parts + (2 * (int64_t)k + (tc::range_lo(k, K, ctas) > u0 ? 0 : 1)) * kPart;
    };
    float* part = split ? part_of(blockIdx.x) : nullptr;
    float whole_unit = kLeastUnit;
    if constexpr (F == kInt8) {
#pragma unroll
      for (int w = 0; w < kWarps; ++w) whole_unit = larger_unit(whole_unit, s_unit[w]);
    }
    for (int i = tid; i < G * D; i += kThreads) {
      const int h = i / D, d = i % D;
      float mm = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, s_ml[w][h][0]);
      float acc = 0.f, l = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float a = weight(s_ml[w][h][0], mm);
        const float u = F == kInt8 ? s_unit[w] / whole_unit : 1.f;
        acc += a * u * s_o[w][h][d];
        l += a * s_ml[w][h][1];
      }
      if (split) {
        part[i] = acc;
        if (d == 0) {
          part[G * D + 2 * h] = mm;
          part[G * D + 2 * h + 1] = l;
          if (h == 0) part[G * (D + 2)] = whole_unit;
        }
      } else if (!(ch.flags & kNobody)) {
        // the division first: acc is a sum over all tokens, and the factor may
        // bring it past the largest float where the result is in range
        p.out[unit * G * D + i] =
            __float2bfloat16_rn(l == 0.f ? 0.f : acc / l * (F == kInt8 ? whole_unit : post));
      }
    }
    if (!split) continue;

    // ---- a split unit: the last of its CTAs to arrive adds the parts up ----
    const int c0 = tc::cta_of(u0, K, ctas), c1 = tc::cta_of(u1 - 1, K, ctas);
    __syncthreads();  // the part is written
    if (tid == 0) {
      ptx::fence_acq_rel_gpu();
      const int n = tc::arrive(&p.counters[unit], p.epoch);
      s_last = n == c1 - c0 + 1;
      if (s_last) p.counters[unit] = p.epoch << 16;  // none, for a replay of this launch
      ptx::fence_acq_rel_gpu();
    }
    __syncthreads();
    if (!s_last) continue;
    for (int i = tid; i < G * D; i += kThreads) {
      const int h = i / D;
      float mm = -INFINITY, uu = kLeastUnit;
      for (int k = c0; k <= c1; ++k) {
        const float* q = part_of(k);
        mm = fmaxf(mm, __ldcg(q + G * D + 2 * h));
        if constexpr (F == kInt8) uu = larger_unit(uu, __ldcg(q + G * (D + 2)));
      }
      float acc = 0.f, l = 0.f;
      for (int k = c0; k <= c1; ++k) {
        const float* q = part_of(k);
        const float a = weight(__ldcg(q + G * D + 2 * h), mm);
        const float u = F == kInt8 ? __ldcg(q + G * (D + 2)) / uu : 1.f;
        acc += a * u * __ldcg(q + i);
        l += a * __ldcg(q + G * D + 2 * h + 1);
      }
      p.out[unit * G * D + i] =
          __float2bfloat16_rn(l == 0.f ? 0.f : acc / l * (F == kInt8 ? uu : post));
    }
  }
  cp_async_wait<0>();
}

int64_t parts_bytes(int group, int head_dim, int num_sms) {
  return (int64_t)kCtasPerSm * num_sms * 2 * (group * (head_dim + 2) + 1) * 4;
}

template <int D, int G, KvFormat F>
cudaError_t launch_one(const ScoredParams& p, int num_sms, cudaStream_t stream) {
  using C = Cfg<D, F>;
  const int64_t units = (int64_t)p.num_rows * p.num_kv_heads;
  const int64_t at_once = (int64_t)kCtasPerSm * num_sms;
  const bool whole = units >= kWholeUnits * at_once;
  const cudaError_t e = allow_large<decode_scored_kernel<D, G, F>>();
  if (e != cudaSuccess) return e;
  return launch_dependent<decode_scored_kernel<D, G, F>>(
      dim3((unsigned)(whole ? units : at_once)), dim3(C::kThreads), C::kRing, stream, 1, p, whole);
}

template <int D, KvFormat F>
cudaError_t launch_g(const ScoredParams& p, int group, int num_sms, cudaStream_t stream) {
  switch (group) {
    case 1: return launch_one<D, 1, F>(p, num_sms, stream);
    case 2: return launch_one<D, 2, F>(p, num_sms, stream);
    case 4: return launch_one<D, 4, F>(p, num_sms, stream);
    case 8: return launch_one<D, 8, F>(p, num_sms, stream);
  }
  return cudaErrorInvalidValue;
}

template <int D>
cudaError_t launch_f(const ScoredParams& p, int group, KvFormat format, int num_sms,
                     cudaStream_t stream) {
  switch (format) {
    case kBf16: return launch_g<D, kBf16>(p, group, num_sms, stream);
    case kE4m3: return launch_g<D, kE4m3>(p, group, num_sms, stream);
    case kInt8: return launch_g<D, kInt8>(p, group, num_sms, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

// Parts of the CTAs that run at once, then a counter for each unit that may
// be split.
size_t scored_workspace_bytes(int64_t num_rows, int64_t num_heads, int64_t num_kv_heads,
                              int head_dim, int num_sms) {
  const int64_t units = num_rows * num_kv_heads;
  if (units >= (int64_t)kWholeUnits * kCtasPerSm * num_sms) return 0;
  const int64_t parts = parts_bytes((int)(num_heads / num_kv_heads), head_dim, num_sms);
  return (size_t)((parts + 255) / 256 * 256 + units * 8);
}

cudaError_t launch_decode_scored(ScoredParams p, void* workspace, int head_dim, int group,
                                 KvFormat format, int num_sms, cudaStream_t stream) {
  const int64_t parts = parts_bytes(group, head_dim, num_sms);
  p.parts = static_cast<float*>(workspace);
  p.counters = reinterpret_cast<unsigned long long*>(static_cast<char*>(workspace) +
                                                     (parts + 255) / 256 * 256);
  p.epoch = tc::next_call_epoch();
  return head_dim == 128 ? launch_f<128>(p, group, format, num_sms, stream)
                         : launch_f<64>(p, group, format, num_sms, stream);
}

}  // namespace pa
