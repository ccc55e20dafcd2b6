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
// bits).  Each warp streams chunks of 16 or 32 tokens through a cp.async ring of its own
// and keeps its own softmax state, as in the decode over listed blocks:
//   S^T [16 tokens x 8 columns] = K q^T     (mma m16n8k16, K by ldmatrix)
//   O^T [D x 8 columns] += V^T P^T          (V by ldmatrix.trans)
// with the query heads in the 8 columns.  Over bf16, columns 4..7 repeat the
// heads for G <= 4 and carry what rounding takes from P, for G = 8 a second
// MMA does.  8-bit elements are widened to f16 in registers (exact); q then
// enters in f16 under a power of two per head, and P is raised by 2^14 (f16
// ends at 2^-24) and rounded once: up to 2^-11 of a weight, an eighth of
// the output's own rounding.  The unit of an 8-bit row multiplies its logit, and
// its weight in P V, relative to the largest product of a weight and a unit that
// the warp has met in the head, about (a running maximum like the softmax's, beside
// its own): f16 then holds each product to half a step or to 2^-37 of that largest
// one, whatever the units' size.  (Relative to the largest unit alone, one for all
// heads, a token with all the weight was lost beside values 2^40 larger that hardly
// counted; one int8 row of 128 K tokens took 57.9 us, where this takes 58.2, 64
// windowed rows 38.4 and 38.9.)
//
// The cap leaves small scores as they are, to within 2^-22 of themselves, and
// large ones to within 2^-20 (capped()).
//
// Work split: a unit is a (row, KV head); its visible tokens are cut into
// steps of one chunk per warp, and the steps of all rows, K in all, into equal
// ranges, whatever the lengths.  Each range is taken by H_kv neighbouring CTAs,
// one a head, as many in all as run at once: they read the same tokens at the
// same time, whose heads lie side by side (with ranges over the units' steps in
// a row, heads far apart, 8 e4m3 rows of 64 K tokens took 152 us).  Loads run
// ahead across the ends of units.  A CTA's range splits at most two units, and
// it goes through its units from the last to the first: the last one's partial
// sums go to the workspace early, and the first one, whose end it holds, is joined
// from its own sums in shared memory and the parts of the CTAs before it, in their
// order, once their flags are up.  (From the first unit to the last, with all
// parts through memory: 64 capped rows 98.7 us, where this takes 97.6, 64 windowed
// int8 rows 39.2 for 38.3, one int8 row of 128 K tokens the same.  A counter of
// arrivals, exchanged with the call's tag, made 38 CTAs of one unit queue for it.)  Flags carry a tag of the
// call, so the workspace needs no initialisation.  Where there is no room for
// parts, and where takes_whole() says so, each CTA takes one whole unit.
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

// What registers and shared memory are kept to.  (64 channels over bf16 with two:
// 2000 rows of 300 tokens 91 us, with three 80.)
constexpr int ctas_per_sm(int head_dim, KvFormat f) { return head_dim == 64 && f == kBf16 ? 3 : 2; }

template <int D, int G, KvFormat F>
struct Cfg {
  static constexpr int kCtasPerSm = ctas_per_sm(D, F);
  static constexpr int kRow = D * (F == kBf16 ? 2 : 1);  // bytes of a token's channels
  static constexpr int kPieces = kRow / 16;
  static constexpr int kChunk = F == kBf16 ? 16 : 32;  // tokens a warp handles at a time
  static constexpr int kTile = kChunk * kRow;  // K (or V) bytes of a chunk
  // What shared memory holds of two CTAs.  (One int8 row of 128 K tokens with 4, 5
  // and 6 warps: 64, 69, 59 us.)
  static constexpr int kWarps = F == kBf16 ? 4 : (D == 64 ? 8 : (G > 4 ? 5 : 6));
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
// Products of weights and units that enter P V are raised by 2^12 over their
// reference, which leaves room for products 8 times as large before it must grow;
// it is at least 2^-112, so that what they are multiplied by is finite.
constexpr float kRaiseUnits = 4096.f, kRoomUnits = 8.f, kLeastProduct = 1.92592994e-34f;

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
// Tokens are visited from a multiple of 16 on.
__device__ __forceinline__ int first_visited(int first) { return first & ~15; }
template <int kStep>
__device__ __forceinline__ int steps_of(const Row& r) {
  const int n = r.end - first_visited(r.first);
  return n <= 0 ? 1 : (n + kStep - 1) / kStep;  // a row without keys has its zeros written
}

// (whole 16-byte pieces)
constexpr int part_words(int group, int head_dim) { return (group * (head_dim + 3) + 3) / 4 * 4; }

// What a warp knows of a chunk that it has asked for.
struct __align__(16) Chunk {
  int row, tok, first;
  unsigned seen;  // a bit per token
  int pos, flags, steps, rel;  // steps of the unit, its first one from this CTA's lo on
};
enum { kOpens = 1, kCloses = 2, kNobody = 4 };

template <int D, int G, KvFormat F>
__global__ void __launch_bounds__(Cfg<D, G, F>::kThreads, Cfg<D, G, F>::kCtasPerSm)
    decode_scored_kernel(const __grid_constant__ ScoredParams p, bool whole_units) {
  using C = Cfg<D, G, F>;
  constexpr bool F16 = F != kBf16;
  constexpr int kWarps = C::kWarps, kThreads = C::kThreads, kChunk = C::kChunk;
  constexpr int kGroups = kChunk / 16;    // 16-token MMA tiles of a chunk
  constexpr int kStep = kWarps * kChunk;  // tokens of a step
  constexpr int kSteps = D / 16;          // k16 steps of q . k; m16 tiles of O^T
  constexpr int kColHeads = G <= 4 ? 4 : 8;
  constexpr int kPart = part_words(G, D);  // a partial: sums, then max, sum, reference per head
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr int kInfos = 4;  // steps asked for at a time, at most: kStages + 1
  static_assert(C::kStages < kInfos, "");
  __shared__ Chunk s_chunk[kWarps][kInfos];
  __shared__ __align__(16) float s_o[kWarps][kColHeads][D];
  __shared__ float s_ml[kWarps][kColHeads][2];
  __shared__ float s_ref[kWarps][kColHeads];
  __shared__ long long s_sum[kWarps], s_before;
  __shared__ Row s_cur;
  __shared__ float s_factor[kWarps][G], s_max[G], s_l[G], s_post[G];
  __shared__ int s_row;
  ptx::grid_dependency_wait();
  ptx::grid_launch_dependents();
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int g = lane / 4, c = lane % 4;  // MMA fragment coordinates
  const int hkv = p.num_kv_heads;

  // ---- this CTA's head and range of steps: [lo, hi) of K, from step `at` of a row ----
  const int part = blockIdx.x / hkv, kvh = blockIdx.x - part * hkv;
  long long K = 0, lo = 0, hi = 0;
  int ctas = 1, row = 0, rel = 0;  // ctas: those of a head; rel: the row's first step - lo
  Row cur;  // the last of this CTA's rows
  if (whole_units) {
    row = part;
    cur = row_of(p, row);
    hi = K = steps_of<kStep>(cur);
  } else {
    // K, and the row that this CTA's last step lies in; each thread counts the steps
    // of rows side by side (by tiles of kThreads rows, one behind the other: 10000 rows
    // of 40 tokens 745 us, where this takes 713)
    const int per = (p.num_rows + kThreads - 1) / kThreads;
    const int r0 = min(tid * per, p.num_rows), r1 = min(r0 + per, p.num_rows);
    Row mine = {-1, 0, 0, 0};
    int n = 0;  // steps of this thread's last row
    long long steps = 0;
#pragma unroll 4
    for (int r = r0; r < r1; ++r) {
      mine = row_of(p, r);
      n = steps_of<kStep>(mine);
      steps += n;
    }
    long long end = steps;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const long long up = __shfl_up_sync(0xffffffffu, end, d);
      if (lane >= d) end += up;
    }
    if (lane == 31) s_sum[warp] = end;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) end += s_sum[w];
      K += s_sum[w];
    }
    ctas = (int)min((long long)(gridDim.x / hkv), K);  // (K is not 0)
    if (part >= ctas) return;
    lo = tc::range_lo(part, K, ctas);
    hi = tc::range_lo(part + 1, K, ctas);
    if (end - steps < hi && hi <= end) {
      int r = r1 - 1;
      for (end -= n; hi <= end; end -= n) {
        mine = row_of(p, --r);
        n = steps_of<kStep>(mine);
      }
      s_row = r;
      s_before = end;
      s_cur = mine;
    }
    __syncthreads();
    row = s_row;
    cur = s_cur;
    rel = (int)(s_before - lo);
  }
  const int total = (int)(hi - lo);

  const uint32_t ring = smem_u32(smem) + warp * C::kStages * C::kStage;
  const int stride = hkv * C::kRow;  // between tokens: bytes, below 2^24
  const int lb = p.log2_block_size;
  float ks = 1.f, post = 1.f;  // e4m3's scales
  if constexpr (F == kE4m3) {
    ks = *p.k_scale;
    post = *p.v_scale;
  }

  // ---- loads.  ask() looks up the slot of this lane's token of the cursor's
  // chunk (-1: none) and goes on to the next; load_keys() and load_values() of
  // the step then need no other address ----
  int asked = 0, n = steps_of<kStep>(cur);
  int at = max(-rel, 0), stop = min(total - rel, n);  // the row's steps that are this CTA's
  auto ask = [&]() -> int {
    if (asked >= total) return -1;
    const int tok0 = first_visited(cur.first) + (at * kWarps + warp) * kChunk;
    if (lane == 0) {
      Chunk& k = s_chunk[warp][asked % kInfos];
      k.row = row;
      k.tok = tok0;
      k.first = cur.first;
      k.pos = cur.pos;
      k.steps = n;
      k.rel = rel;
      k.flags = (at == max(-rel, 0) ? kOpens : 0) | (at == stop - 1 ? kCloses : 0) |
                // a row of no sequence: nothing is written
                (cur.seq < 0 ? kNobody : 0);
    }
    const int tok = tok0 + (lane & (kChunk - 1));
    int slot = -1;
    if (tok >= cur.first && tok < cur.end) {
      const int phys = p.block_tables[(int64_t)cur.seq * p.max_blocks + (tok >> lb)];
      if ((unsigned)phys < (unsigned)p.num_blocks) slot = (phys << lb) + (tok & ((1 << lb) - 1));
    }
    ++asked;
    if (++at == stop && asked < total) {  // rows from the last to the first
      cur = row_of(p, --row);
      stop = n = steps_of<kStep>(cur);
      rel -= n;
      at = max(-rel, 0);
    }
    return slot;
  };
  constexpr int kRowsPer = 32 / C::kPieces;  // tokens per instruction
  const int piece = lane % C::kPieces;
  const int64_t lane_at = (int64_t)kvh * C::kRow + piece * 16;
  const uint8_t* const kbase = static_cast<const uint8_t*>(p.k_cache) + lane_at;
  const uint8_t* const vbase = static_cast<const uint8_t*>(p.v_cache) + lane_at;
  auto load_rows = [&](uint32_t to, const uint8_t* base, int slot) {
#pragma unroll
    for (int r = 0; r < kChunk / kRowsPer; ++r) {
      const int t = r * kRowsPer + lane / C::kPieces;
      const int s = __shfl_sync(0xffffffffu, slot, t);
      cp_async_16(to + t * C::kRow + C::swizzle(t, piece) * 16, base + (int64_t)max(s, 0) * stride,
                  s >= 0 ? 16 : 0);  // zeros where there is no token
    }
  };
  auto load_units = [&](uint32_t to, const float* units, int slot) {
    cp_async_4_or_zero(to + lane * 4, units + (int64_t)max(slot, 0) * hkv + kvh, slot >= 0 ? 4 : 0);
  };
  auto load_keys = [&](int step, int slot) {
    if (step < total) {
      unsigned seen = __ballot_sync(0xffffffffu, slot >= 0);
      if constexpr (kChunk == 16) seen &= 0xffff;
      if (lane == 0) s_chunk[warp][step % kInfos].seen = seen;
      const uint32_t stage = ring + step % C::kStages * C::kStage;
      load_rows(stage, kbase, slot);
      if constexpr (F == kInt8) load_units(stage + 2 * C::kTile, p.k_scale, slot);
    }
    cp_async_commit();
  };
  auto load_values = [&](int step, int slot) {
    if (step < total) {
      const uint32_t stage = ring + step % C::kStages * C::kStage;
      load_rows(stage + C::kTile, vbase, slot);
      if constexpr (F == kInt8) load_units(stage + 2 * C::kTile + 4 * kChunk, p.v_scale, slot);
    }
    cp_async_commit();
  };

  // ---- a unit's queries, as MMA operand B: column `col` is query head col
  // (mod 4 when G <= 4); what its logits are multiplied by; its slopes ----
  const int qh = g % kColHeads;
  uint2 qw[kSteps];
  uint32_t qb[kSteps][2];
  float f0 = 0.f, f1 = 0.f, slope0 = 0.f, slope1 = 0.f;
  auto fetch_q = [&](int unit_row) {
    const int64_t unit = (int64_t)unit_row * hkv + kvh;
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
      slope0 = h0 < G ? p.mod.slopes[kvh * G + h0] * kLog2e : 0.f;
      slope1 = h1 < G ? p.mod.slopes[kvh * G + h1] * kLog2e : 0.f;
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
  // int8: the largest weight times unit so far, about, under the weights' own
  // reference m; and what such products are multiplied by
  float r0, r1, by0, by1;
  auto open = [&]() {
#pragma unroll
    for (int i = 0; i < kSteps; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    m0 = m1 = -INFINITY;
    l0 = l1 = 0.f;
    r0 = r1 = kLeastProduct;
    by0 = by1 = kRaiseUnits / kLeastProduct;
  };

  constexpr float kPost = F == kInt8 ? 1.f / kRaiseUnits : 1.f;
  // Two outputs.  The division first: x and y are sums over all tokens, and
  // the factor may bring them past the largest float where the result is in
  // range.
  auto store = [&](int64_t at, float x, float y, float l, float factor) {
    if (l == 0.f) x = y = 0.f;
    else x = x / l * factor, y = y / l * factor;
    *reinterpret_cast<uint32_t*>(p.out + at) = pack_bf16x2_rn(x, y);
  };

  int64_t merge_unit = -1;  // the split unit whose end this CTA holds, and
  int merge_rel = 0;        // the first of its steps
  fetch_q(row);
  int slot;  // of the step that is loaded next
  {
    int early[C::kStages];
#pragma unroll
    for (int s = 0; s < C::kStages; ++s) early[s] = ask();
    slot = ask();
#pragma unroll
    for (int s = 0; s < C::kStages; ++s) {
      load_keys(s, early[s]);
      load_values(s, early[s]);
    }
  }
  // groups behind a step's keys, or behind its values with the keys that took
  // their place in between
  constexpr int kBehind = 2 * C::kStages - 1;
  for (int it = 0; it < total; ++it) {
    cp_async_wait<kBehind>();
    __syncwarp();
    const Chunk ch = s_chunk[warp][it % kInfos];
    if (ch.flags & kOpens) {
      place_q();
      open();
    }
    const uint32_t kt = ring + (it % C::kStages) * C::kStage;
    const uint32_t vt = kt + C::kTile;
    // logits of tokens g, g + 8, g + 16 ... of the chunk, columns 2c and 2c + 1
    float x[2 * kGroups][2];
    const float* units = reinterpret_cast<const float*>(
        smem + (warp * C::kStages + it % C::kStages) * C::kStage + 2 * C::kTile);
    if (ch.seen) {
      float ku[2 * kGroups];
#pragma unroll
      for (int i = 0; i < 2 * kGroups; ++i) ku[i] = F == kInt8 ? units[g + 8 * i] : 1.f;
#pragma unroll
      for (int gr = 0; gr < kGroups; ++gr) {
        float s[4] = {0.f, 0.f, 0.f, 0.f};
        const int r = 16 * gr + (lane & 7) + ((lane >> 3) & 1) * 8;
        const uint32_t base = kt + r * C::kRow;
        if constexpr (F16) {
#pragma unroll
          for (int k = 0; k < kSteps; k += 2) {
            uint32_t w[4];
            ldmatrix_x4(w, base + C::swizzle(r, k + (lane >> 4)) * 16);
#pragma unroll
            for (int h = 0; h < 2; ++h) {  // the two 16-channel pieces
              const uint32_t y = w[2 * h], z = w[2 * h + 1];
              const uint32_t a[4] = {widen_half<F>(y, false), widen_half<F>(z, false),
                                     widen_half<F>(y, true), widen_half<F>(z, true)};
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
        x[2 * gr][0] = s[0];
        x[2 * gr][1] = s[1];
        x[2 * gr + 1][0] = s[2];
        x[2 * gr + 1][1] = s[3];
      }
      if constexpr (F == kInt8) {
#pragma unroll
        for (int i = 0; i < 2 * kGroups; ++i) {
          x[i][0] *= ku[i];
          x[i][1] *= ku[i];
        }
      }
    }
    float n0 = -INFINITY, n1 = -INFINITY;  // each column's largest logit so far
    __syncwarp();
    load_keys(it + C::kStages, slot);  // in the place of the keys just used
    if (ch.seen) {
      if (p.mod.cap_log2 > 0.f) {
        bool small = true;
#pragma unroll
        for (int i = 0; i < 2 * kGroups; ++i) {
          x[i][0] *= f0;
          x[i][1] *= f1;
          small &= fabsf(x[i][0] * p.mod.inv_cap) <= kTanhSmall &&
                   fabsf(x[i][1] * p.mod.inv_cap) <= kTanhSmall;
        }
        if (__all_sync(0xffffffffu, small)) {  // (either way the same scores)
#pragma unroll
          for (int i = 0; i < 2 * kGroups; ++i) {
            x[i][0] = capped_small(x[i][0], x[i][0] * p.mod.inv_cap);
            x[i][1] = capped_small(x[i][1], x[i][1] * p.mod.inv_cap);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 2 * kGroups; ++i) {
            x[i][0] = capped(x[i][0], x[i][0] * p.mod.inv_cap, p.mod.cap_log2);
            x[i][1] = capped(x[i][1], x[i][1] * p.mod.inv_cap, p.mod.cap_log2);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < 2 * kGroups; ++i) {
          x[i][0] *= f0;
          x[i][1] *= f1;
        }
      }
      if (p.mod.slopes) {
#pragma unroll
        for (int i = 0; i < 2 * kGroups; ++i) {
          const float d = (float)abs(ch.pos - (ch.tok + g + 8 * i));
          x[i][0] -= slope0 * d;
          x[i][1] -= slope1 * d;
        }
      }
      if (ch.seen != (kChunk == 32 ? 0xffffffffu : 0xffffu)) {
#pragma unroll
        for (int i = 0; i < 2 * kGroups; ++i)
          if (!(ch.seen >> (g + 8 * i) & 1)) x[i][0] = x[i][1] = -INFINITY;
      }
      n0 = x[0][0];
      n1 = x[0][1];
#pragma unroll
      for (int i = 1; i < 2 * kGroups; ++i) {
        n0 = fmaxf(n0, x[i][0]);
        n1 = fmaxf(n1, x[i][1]);
      }
#pragma unroll
      for (int d = 4; d < 32; d *= 2) {
        n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, d));
        n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, d));
      }
      n0 = fmaxf(n0, m0);
      n1 = fmaxf(n1, m1);
    }
    cp_async_wait<kBehind>();
    __syncwarp();
    if (ch.seen) {
      float vu[4] = {1.f, 1.f, 1.f, 1.f};
      if constexpr (F == kInt8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) vu[i] = units[kChunk + g + 8 * i];
      }
      auto scale_sums = [&](float a0, float a1) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          o[i][0] *= a0;
          o[i][1] *= a1;
          o[i][2] *= a0;
          o[i][3] *= a1;
        }
      };
      if (__any_sync(0xffffffffu, n0 > m0 || n1 > m1)) {
        const float a0 = m0 == -INFINITY ? 0.f : fast_exp2(m0 - n0);
        const float a1 = m1 == -INFINITY ? 0.f : fast_exp2(m1 - n1);
        l0 *= a0;
        l1 *= a1;
        if constexpr (F == kInt8) {
          // the products' reference falls with the weights: their sums stay as they
          // are, unless it would fall below the least
          const float t0 = r0 * a0, t1 = r1 * a1;
          r0 = fmaxf(t0, kLeastProduct);
          r1 = fmaxf(t1, kLeastProduct);
          by0 = kRaiseUnits * fast_reciprocal(r0);
          by1 = kRaiseUnits * fast_reciprocal(r1);
          if (__any_sync(0xffffffffu, t0 < kLeastProduct || t1 < kLeastProduct))
            scale_sums(t0 < kLeastProduct ? t0 / kLeastProduct : 1.f,
                       t1 < kLeastProduct ? t1 / kLeastProduct : 1.f);
        } else {
          scale_sums(a0, a1);
        }
        m0 = n0;
        m1 = n1;
      }
      // log2 of the factor that P and its sum carry (int8: the products alone)
      constexpr float kRaise = F == kE4m3 ? 14.f : 0.f;
      const float z0 = (m0 == -INFINITY ? 0.f : m0) - kRaise;
      const float z1 = (m1 == -INFINITY ? 0.f : m1) - kRaise;
#pragma unroll
      for (int i = 0; i < 2 * kGroups; ++i) {
        x[i][0] = fast_exp2(x[i][0] - z0);
        x[i][1] = fast_exp2(x[i][1] - z1);
        l0 += x[i][0];
        l1 += x[i][1];
      }
      if constexpr (F == kInt8) {
        // (a NaN is passed over here, and stays in x)
        const float most = fmaxf(fmaxf(vu[0], vu[1]), fmaxf(vu[2], vu[3]));
        if (!__any_sync(0xffffffffu, most > kRoomUnits * fminf(r0, r1))) {  // weights are at most 1
#pragma unroll
          for (int i = 0; i < 2 * kGroups; ++i) {
            x[i][0] *= vu[i] * by0;
            x[i][1] *= vu[i] * by1;
          }
        } else {
          float top0 = 0.f, top1 = 0.f;
#pragma unroll
          for (int i = 0; i < 2 * kGroups; ++i) {
            x[i][0] *= vu[i];
            x[i][1] *= vu[i];
            top0 = fmaxf(top0, x[i][0]);
            top1 = fmaxf(top1, x[i][1]);
          }
#pragma unroll
          for (int d = 4; d < 32; d *= 2) {
            top0 = fmaxf(top0, __shfl_xor_sync(0xffffffffu, top0, d));
            top1 = fmaxf(top1, __shfl_xor_sync(0xffffffffu, top1, d));
          }
          if (__any_sync(0xffffffffu, top0 > r0 || top1 > r1)) {
            const float t0 = fmaxf(top0, r0), t1 = fmaxf(top1, r1);
            const float i0 = fast_reciprocal(t0), i1 = fast_reciprocal(t1);
            scale_sums(t0 > r0 ? r0 * i0 : 1.f, t1 > r1 ? r1 * i1 : 1.f);
            r0 = t0;
            r1 = t1;
            by0 = kRaiseUnits * i0;
            by1 = kRaiseUnits * i1;
          }
#pragma unroll
          for (int i = 0; i < 2 * kGroups; ++i) {
            x[i][0] *= by0;
            x[i][1] *= by1;
          }
        }
      }
#pragma unroll
      for (int gr = 0; gr < kGroups; ++gr) {
        uint32_t hi0 = pack2<F16>(x[2 * gr][0], x[2 * gr][1]);
        uint32_t hi1 = pack2<F16>(x[2 * gr + 1][0], x[2 * gr + 1][1]);
        if constexpr (F16) {
          const uint32_t b0 = movmatrix_trans(hi0), b1 = movmatrix_trans(hi1);
          // a transposed 16-bit unit holds channels 2g and 2g + 1 of a token: the
          // even ones become row g of the tile, the odd ones row g + 8
          const int r = 16 * gr + (lane & 7) + ((lane >> 3) & 1) * 8;
#pragma unroll
          for (int k = 0; k < kSteps; k += 2) {
            uint32_t w[4];
            ldmatrix_x4_trans(w, vt + r * C::kRow + C::swizzle(r, k + (lane >> 4)) * 16);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t y = w[2 * h], z = w[2 * h + 1];
              const uint32_t a[4] = {widen_alternate<F>(y, false), widen_alternate<F>(y, true),
                                     widen_alternate<F>(z, false), widen_alternate<F>(z, true)};
              mma16816<true>(o[k + h], a, b0, b1);
            }
          }
        } else {
          const float2 r0 = unpack2<false>(hi0), r1 = unpack2<false>(hi1);
          uint32_t lo0 = pack2<false>(x[2 * gr][0] - r0.x, x[2 * gr][1] - r0.y);
          uint32_t lo1 = pack2<false>(x[2 * gr + 1][0] - r1.x, x[2 * gr + 1][1] - r1.y);
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
          const int r = 16 * gr + (lane & 7) + (lane >> 4) * 8;
#pragma unroll
          for (int k = 0; k < kSteps; ++k) {
            uint32_t a[4];
            ldmatrix_x4_trans(a, vt + r * C::kRow + C::swizzle(r, 2 * k + ((lane >> 3) & 1)) * 16);
            mma16816<false>(o[k], a, b0, b1);
            if constexpr (G > 4) mma16816<false>(o[k], a, d0, d1);
          }
        }
      }
    }
    const bool closes = ch.flags & kCloses;
    if (closes && it + 1 < total) {  // the next unit's queries, while this one is added up
      fetch_q(s_chunk[warp][(it + 1) % kInfos].row);
    }
    __syncwarp();
    load_values(it + C::kStages, slot);
    slot = ask();
    if (!closes) continue;

    // ---- the piece is done: the warps' sums meet ----
#pragma unroll
    for (int d = 4; d < 32; d *= 2) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, d);
      l1 += __shfl_xor_sync(0xffffffffu, l1, d);
    }
    if constexpr (!F16 && G <= 4) {  // the remainders' columns
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
        if constexpr (F == kInt8) {
          s_ref[warp][2 * c] = r0;
          s_ref[warp][2 * c + 1] = r1;
        }
      }
    }
    __syncthreads();
    const int64_t unit = (int64_t)ch.row * hkv + kvh;
    const bool starts = ch.rel >= 0, ends = ch.rel + ch.steps <= total;
    const bool split = !starts || !ends;
    // the factors of the warps' sums, and each head's max and sum over them
    if (tid < kWarps * G) {
      const int w = tid / G, h = tid % G;
      float mm = -INFINITY, rr = kLeastProduct, l = 0.f;
#pragma unroll
      for (int x = 0; x < kWarps; ++x) mm = fmaxf(mm, s_ml[x][h][0]);
      if constexpr (F == kInt8) {
#pragma unroll
        for (int x = 0; x < kWarps; ++x) rr = fmaxf(rr, weight(s_ml[x][h][0], mm) * s_ref[x][h]);
      }
      const float a = weight(s_ml[w][h][0], mm);
      s_factor[w][h] = F == kInt8 ? a * s_ref[w][h] / rr : a;
      if (w == 0) {
#pragma unroll
        for (int x = 0; x < kWarps; ++x) l += weight(s_ml[x][h][0], mm) * s_ml[x][h][1];
        s_max[h] = mm;
        s_l[h] = l;
        s_post[h] = F == kInt8 ? rr : post;
      }
    }
    __syncthreads();
    if (!starts && ends) {  // its last piece: what is here is joined from shared memory
      merge_unit = unit;
      merge_rel = ch.rel;
      break;
    }
    float* mine = p.parts + (2 * (int64_t)blockIdx.x + (starts ? 1 : 0)) * kPart;
    for (int i = 2 * tid; i < G * D; i += 2 * kThreads) {
      const int h = i / D, d = i % D;
      float x = 0.f, y = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float a = s_factor[w][h];
        x += a * s_o[w][h][d];
        y += a * s_o[w][h][d + 1];
      }
      if (split)
        *reinterpret_cast<float2*>(mine + i) = make_float2(x, y);
      else if (!(ch.flags & kNobody))
        store(unit * G * D + i, x, y, s_l[h], s_post[h] * kPost);
    }
    if (!split) continue;
    if (tid < G) {
      mine[G * D + 3 * tid] = s_max[tid];
      mine[G * D + 3 * tid + 1] = s_l[tid];
      mine[G * D + 3 * tid + 2] = s_post[tid];
    }

    __syncthreads();  // the part is written
    if (tid == 0) {
      ptx::fence_acq_rel_gpu();
      st_release(&p.flags[2 * blockIdx.x + (starts ? 1 : 0)], p.epoch);
    }
  }
  cp_async_wait<0>();
  if (merge_unit < 0) return;

  // ---- the CTA that holds a split unit's end adds the unit's parts up: those
  // of CTAs before it, which have all been started, so that the wait ends ----
  const int first = tc::cta_of(lo + merge_rel, K, ctas), count = part - first;
  // the first CTA's part starts the unit, the others' go on with it
  auto index_of = [&](int k) { return 2 * ((first + k) * hkv + kvh) + (k == 0 ? 1 : 0); };
  bool all = true;
  for (int k = tid; k < count; k += kThreads) {
    unsigned long long* flag = &p.flags[index_of(k)];
    const long long begun = clock64();
    while (ld_acquire(flag) != p.epoch) {
      if (clock64() - begun > tc::kWaitClocks) {
        atomicExch(p.err, 41);
        all = false;
        break;
      }
    }
    *flag = 0;  // for a replay of this launch
  }
  if (!__syncthreads_and(all)) return;
  // As many parts as the ring holds are brought in at once: one trip to memory
  // for up to 38 (D = 128, G = 4).  (Eight at a time in registers: 4.3 us for 38
  // parts, where this takes 2.)
  constexpr int kBatch = C::kRing / (kPart * 4);
  constexpr int kItems = (G * D / 4 + kThreads - 1) / kThreads;
  float4 sum[kItems];
  float top[kItems], l[kItems], rr[kItems];
#pragma unroll
  for (int j = 0; j < kItems; ++j) {  // this CTA's own sums
    sum[j] = make_float4(0.f, 0.f, 0.f, 0.f);
    top[j] = -INFINITY;
    l[j] = 0.f;
    rr[j] = kLeastProduct;
    const int i = 4 * (tid + j * kThreads), h = i / D, d = i % D;
    if (i >= G * D) break;
    top[j] = s_max[h];
    l[j] = s_l[h];
    if constexpr (F == kInt8) rr[j] = s_post[h];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float a = s_factor[w][h];
      const float4 v = *reinterpret_cast<const float4*>(&s_o[w][h][d]);
      sum[j].x += a * v.x, sum[j].y += a * v.y, sum[j].z += a * v.z, sum[j].w += a * v.w;
    }
  }
  const float* held = reinterpret_cast<const float*>(smem);
  for (int k0 = 0; k0 < count; k0 += kBatch) {
    const int n = min(kBatch, count - k0);
    __syncthreads();  // the ring is free
    for (int i = tid; i < n * (kPart / 4); i += kThreads) {
      const int k = i / (kPart / 4), w = i - k * (kPart / 4);
      cp_async_16(smem_u32(smem) + 16 * i,
                  p.parts + (int64_t)index_of(k0 + k) * kPart + 4 * w, 16);
    }
    cp_async_commit();
    cp_async_wait<0>();
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kItems; ++j) {
      const int i = 4 * (tid + j * kThreads), h = i / D;
      if (i >= G * D) break;
      const float* ml = held + G * D + 3 * h;
      float most = top[j], ref = kLeastProduct;
      for (int k = 0; k < n; ++k) most = fmaxf(most, ml[k * kPart]);
      float a = weight(top[j], most);
      l[j] *= a;
      if constexpr (F == kInt8) {
        for (int k = 0; k < n; ++k)
          ref = fmaxf(ref, weight(ml[k * kPart], most) * ml[k * kPart + 2]);
        a *= rr[j];
        ref = fmaxf(ref, a);
        a /= ref;
      }
      const float inverse = 1.f / ref;
      sum[j].x *= a, sum[j].y *= a, sum[j].z *= a, sum[j].w *= a;
#pragma unroll 4
      for (int k = 0; k < n; ++k) {
        const float* q = held + k * kPart;
        a = weight(ml[k * kPart], most);
        l[j] += a * ml[k * kPart + 1];
        if constexpr (F == kInt8) a = a * ml[k * kPart + 2] * inverse;
        const float4 v = *reinterpret_cast<const float4*>(q + i);
        sum[j].x += a * v.x, sum[j].y += a * v.y, sum[j].z += a * v.z, sum[j].w += a * v.w;
      }
      top[j] = most;
      rr[j] = ref;
    }
  }
#pragma unroll
  for (int j = 0; j < kItems; ++j) {
    const int i = 4 * (tid + j * kThreads);
    if (i >= G * D) break;
    const float factor = F == kInt8 ? rr[j] * kPost : post;
    store(merge_unit * G * D + i, sum[j].x, sum[j].y, l[j], factor);
    store(merge_unit * G * D + i + 2, sum[j].z, sum[j].w, l[j], factor);
  }
}

// Units per CTA, for two an SM, from which no room for parts is asked for.  (657,
// rows of 400 tokens and 64 channels, whole and split, us: bf16 4043, 3796, int8
// 4078, 3585.)
constexpr int kManyUnits = 512;

// Whether each unit goes to one CTA although its parts have room.  CTAs handed out
// as others end, a row's heads to neighbours, keep many heads closer together than
// equal ranges do; but a row much longer than the others is then one CTA's, so only
// where the longest that there may be is short beside a CTA's share.  (Whole and
// split, us, e4m3 rows of 32 heads: 256 of 2900 tokens 937, 978, 600 of 2900 2130,
// 2280, 350 of 1200 578, 586, of lengths up to 1200 369, 353, 1000 of 300 617, 582;
// 8 heads: 1000 rows of 2000 674, 670, 512 of up to 2000 250, 238; 228 rows of 300
// with one of 128 K among them, bf16: 2250, 162.)
constexpr int kWholeHeads = 16, kWholeTokens = 1024, kTokensPerUnit = 128;
bool takes_whole(const ScoredParams& p, int64_t at_once) {
  const int64_t longest = (int64_t)p.max_blocks << p.log2_block_size;
  return p.num_kv_heads >= kWholeHeads && longest >= kWholeTokens &&
         longest * at_once <= (int64_t)p.num_rows * p.num_kv_heads * kTokensPerUnit;
}

// Ranges per head: such that the fewest rounds of the CTAs that run at once
// do the most.
int ranges_of(int64_t heads, int64_t at_once) {
  int64_t best = 1;
  auto rounds = [&](int64_t r) { return (r * heads + at_once - 1) / at_once; };
  for (int64_t r = at_once / heads < 1 ? 1 : at_once / heads; r <= 16 || r * heads <= at_once; ++r)
    if (rounds(r) * best < rounds(best) * r) best = r;
  return (int)best;
}

template <int D, int G, KvFormat F>
cudaError_t launch_one(const ScoredParams& p, int num_sms, cudaStream_t stream) {
  using C = Cfg<D, G, F>;
  const int64_t units = (int64_t)p.num_rows * p.num_kv_heads;
  const int64_t at_once = (int64_t)C::kCtasPerSm * num_sms;
  const bool whole = !p.flags || takes_whole(p, at_once);
  const cudaError_t e = allow_large<decode_scored_kernel<D, G, F>>();
  if (e != cudaSuccess) return e;
  return launch_dependent<decode_scored_kernel<D, G, F>>(
      dim3((unsigned)(whole ? units
                            : ranges_of(p.num_kv_heads, at_once) * (int64_t)p.num_kv_heads)),
      dim3(C::kThreads), C::kRing, stream, 1, p, whole);
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

// Flags of two parts for each CTA, then the parts.
static int64_t split_ctas(int64_t num_kv_heads, int num_sms, int per_sm) {
  return ranges_of(num_kv_heads, (int64_t)per_sm * num_sms) * num_kv_heads;
}
static size_t flag_bytes(int64_t ctas) { return (size_t)(ctas * 16 + 255) / 256 * 256; }
static size_t split_bytes(int64_t num_kv_heads, int group, int head_dim, int num_sms, int per_sm) {
  const int64_t ctas = split_ctas(num_kv_heads, num_sms, per_sm);
  return flag_bytes(ctas) + (size_t)ctas * 2 * part_words(group, head_dim) * 4;
}

size_t scored_workspace_bytes(int64_t num_rows, int64_t num_heads, int64_t num_kv_heads,
                              int head_dim, int num_sms) {
  if (num_rows * num_kv_heads >= (int64_t)kManyUnits * 2 * num_sms) return 0;
  const int group = (int)(num_heads / num_kv_heads);
  size_t most = 0;
  for (KvFormat f : {kBf16, kE4m3, kInt8}) {
    const size_t n = split_bytes(num_kv_heads, group, head_dim, num_sms, ctas_per_sm(head_dim, f));
    if (n > most) most = n;
  }
  return most;
}

cudaError_t launch_decode_scored(ScoredParams p, void* workspace, size_t bytes, int head_dim,
                                 int group, KvFormat format, int num_sms, cudaStream_t stream) {
  const int per_sm = ctas_per_sm(head_dim, format);
  p.flags = nullptr;
  if (bytes >= split_bytes(p.num_kv_heads, group, head_dim, num_sms, per_sm)) {
    p.flags = static_cast<unsigned long long*>(workspace);
    p.parts = reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                       flag_bytes(split_ctas(p.num_kv_heads, num_sms, per_sm)));
    p.epoch = tc::next_call_epoch();
  }
  return head_dim == 128 ? launch_f<128>(p, group, format, num_sms, stream)
                         : launch_f<64>(p, group, format, num_sms, stream);
}

}  // namespace pa
