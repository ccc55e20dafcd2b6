// Decode attention over listed cache blocks.
//
// For query row r and KV head h with the listed blocks J,
//   out = softmax(scale q . K_T^T) V_T,  T = the tokens of J's blocks below
// the row's context length, for the head's G query heads together, so that
// each K and V byte is read once.
//
// Bound: the listed blocks' bytes (at G = 4, 4 flop a byte).  Every KV head
// of a row has a list of its own, so what is contiguous in memory is one
// token's channels of one head (64 to 256 bytes); rows of that size are
// gathered by 16-byte cp.async, and the matrix work beside them is small
// enough for warp-level MMAs: each warp streams 16-token chunks through a
// ring of its own in shared memory and keeps its own softmax state, so the
// stream needs no barrier.  A warp's chunk:
//   S^T [16 tokens x 8 columns] = K q^T     (mma m16n8k16, K by ldmatrix)
//   p = 2^(s - m) per column, running max and sum in fp32
//   O^T [D x 8 columns] += V^T P^T          (V by ldmatrix.trans)
// Transposed so that the 16-row side of the MMA holds tokens and channels
// and the query heads sit in the 8 columns; P turns from accumulator to
// operand layout by movmatrix.  With G <= 4 the columns 4..7 repeat the
// heads of columns 0..3 and carry what rounding takes from P (p - round(p)),
// so P V keeps about 16 bits of P at no cost; with G = 8 a second MMA does.
// (The sum of the weights is of P before that rounding; 2^-17 of a weight is
// far below the outputs' half step, 2^-9.)
// An e4m3 cache is widened to f16 in registers (exact); q then enters in f16
// under a power-of-two scale per head that puts its largest channel in
// [1, 2) (f16 keeps 11 bits, bf16 q has 8, so channels down to 2^-16 of the
// largest stay exact).  f16 ends at 2^-24, so its P is 2^14 2^(s - m), below
// its largest value 65504: what is lost of a weight is below 2^-39 of the
// largest, and 2^22 listed tokens lose less than 2^-17 together (2^(s - m)
// itself would drop each weight below 2^-25, 2^-3 together).
// The warps' results meet in shared memory, those of the CTAs that share a
// (row, KV head) in a cluster's distributed shared memory: no workspace, no
// second kernel, and sums in a fixed order.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "launch.cuh"
#include "pa_device.cuh"
#include "pa_kernels.cuh"
#include "tc_ptx.cuh"

namespace pa {

namespace {

constexpr int kChunk = 16;      // tokens a warp handles at a time
// CTAs that share a (row, KV head): what every device runs, and what this one does
constexpr int kMaxCluster = 8, kLargeCluster = 12;

__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
  return y;
}
template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (F16) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    return pack_bf16x2_rn(lo, hi);
  }
}
template <bool F16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (F16)
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  else
    return make_float2(bf16_lo(w), bf16_hi(w));
}
// The two e4m3 values of a 16-bit half as an f16 pair.
__device__ __forceinline__ uint32_t widen(uint16_t codes) {
  uint32_t h2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(h2) : "h"(codes));
  return h2;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;\n" ::: "memory");
}
// Writes a word of another CTA's shared memory.
__device__ __forceinline__ void store_peer(float* own, uint32_t rank, float v) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(a) : "r"(smem_u32(own)), "r"(rank));
  asm volatile("st.shared::cluster.f32 [%0], %1;\n" ::"r"(a), "f"(v) : "memory");
}

// The factor of a part whose running max is m under the whole's max; 1 where
// neither has a token, so that a NaN among the logits still reaches the sums.
__device__ __forceinline__ float weight(float m, float whole) {
  return whole == -INFINITY ? 1.f : fast_exp2(m - whole);
}
// (o / l) scale, and zero for a row without tokens.  The division first: o is
// a sum over up to 2^22 tokens, and scale may bring it past the largest float
// where the result is in range.
__device__ __forceinline__ __nv_bfloat16 quotient(float o, float l, float scale) {
  return __float2bfloat16_rn(l == 0.f ? 0.f : o / l * scale);
}

template <int D, bool FP8>
struct Cfg {
  static constexpr int kRow = D * (FP8 ? 1 : 2);  // bytes of a token's channels
  static constexpr int kPieces = kRow / 16;
  static constexpr int kTile = kChunk * kRow;  // K (or V) bytes of a chunk
  // A warp's stage is 8 KB of bf16 or 4 KB of e4m3 (D = 128), and e4m3 has
  // twice the instructions a byte, so twice the warps to hide them behind
  // (8 rows of 8192 tokens: 33.3 us with 4 warps of 3 stages, 28.4 with 8 of
  // 2; 64 rows of 1024 tokens in bf16: 46.5 with 4 of 3, 56.1 with 8 of 2).
  static constexpr int kWarps = FP8 ? 8 : 4;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kStages = FP8 ? 2 : 3;
  static constexpr int kRing = kWarps * kStages * 2 * kTile;
  static constexpr int kMerge = kWarps * 8 * (D + 2) * 4;  // reuses the ring
  static_assert(kMerge <= kRing, "the merge reuses the ring");
  // 16-byte pieces of a tile's row, permuted so that 8 rows' pieces of one
  // column (ldmatrix) fall in different banks
  static __device__ __forceinline__ int swizzle(int row, int piece) {
    if constexpr (kPieces >= 8)
      return piece ^ (row & 7);
    else
      return piece ^ ((row >> 1) & 3);
  }
};

template <int D, int G, bool FP8>
__global__ void __launch_bounds__(Cfg<D, FP8>::kThreads)
    decode_selected_kernel(const __grid_constant__ SelectedParams p, int clusters) {
  using C = Cfg<D, FP8>;
  constexpr int kWarps = C::kWarps, kThreads = C::kThreads;
  constexpr int kSteps = D / 16;  // k16 steps of q . k; m16 tiles of O^T
  constexpr int kEarly = 2;       // list entries per thread in the first loads
  extern __shared__ __align__(128) uint8_t smem[];
  // listed entries of this CTA's share: first slot of the block, tokens in use
  int2* s_entry = reinterpret_cast<int2*>(smem + C::kRing);
  __shared__ int s_last;
  // what the cluster's CTAs hand this one: their sums of its share of the
  // outputs, and every head's max and sum
  __shared__ float s_part[G * D + kLargeCluster];
  __shared__ float s_state[kLargeCluster][G][2];
  // the first half of a cluster barrier: peers may be written to once all run
  if (clusters > 1) asm volatile("barrier.cluster.arrive.aligned;\n" ::: "memory");
  ptx::grid_dependency_wait();
  ptx::grid_launch_dependents();
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int g = lane / 4, c = lane % 4;  // MMA fragment coordinates
  const int unit = blockIdx.x / clusters, rank = blockIdx.x % clusters;
  const int row = unit / p.num_kv_heads, kvh = unit - row * p.num_kv_heads;
  const int lb = p.log2_block_size, block = 1 << lb;

  // What depends on nothing is loaded first: the list's first entries, the
  // length, the queries; then the entries' physical blocks.
  const int32_t* list = p.selected + (int64_t)unit * p.top;
  int j_early[kEarly], phys_early[kEarly];
#pragma unroll
  for (int k = 0; k < kEarly; ++k) {
    const int i = k * kThreads + tid;
    j_early[k] = i < p.top ? list[i] : -1;
  }
  const int seq = p.row_seqs ? p.row_seqs[row] : row;
  int64_t n = p.context_lens[row];
  const bool known = (unsigned)seq < (unsigned)p.num_seqs;
  const int32_t* table = p.block_tables + (known ? (int64_t)seq * p.max_blocks : 0);
  constexpr int kColHeads = G <= 4 ? 4 : 8;
  const int qh = g % kColHeads;  // the query head of this lane's MMA column
  uint2 qw[kSteps];              // its channels, as operand B takes them
  {
    const __nv_bfloat16* q = p.q + ((int64_t)unit * G + qh) * D;
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      qw[k] = make_uint2(0, 0);
      if (qh < G) {
        if (FP8) {
          qw[k] = *reinterpret_cast<const uint2*>(q + 16 * k + 4 * c);
        } else {
          qw[k].x = *reinterpret_cast<const uint32_t*>(q + 16 * k + 2 * c);
          qw[k].y = *reinterpret_cast<const uint32_t*>(q + 16 * k + 8 + 2 * c);
        }
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kEarly; ++k)
    phys_early[k] = known && (unsigned)j_early[k] < (unsigned)p.max_blocks ? table[j_early[k]] : -1;
  n = known ? min(n, (int64_t)p.max_blocks << lb) : 0;

  // entries up to the last that names a block below the context's end
  auto inside = [&](int j) { return j >= 0 && ((int64_t)j << lb) < n; };
  if (tid == 0) s_last = 0;
  __syncthreads();
  int last = 0;
#pragma unroll
  for (int k = 0; k < kEarly; ++k)
    if (inside(j_early[k])) last = k * kThreads + tid + 1;
  for (int i = kEarly * kThreads + tid; i < p.top; i += kThreads)
    if (inside(list[i])) last = i + 1;
  last = __reduce_max_sync(0xffffffffu, last);
  if (lane == 0 && last) atomicMax(&s_last, last);
  __syncthreads();
  last = s_last;
  // this CTA's share: an equal run of 16-token chunks
  const int all_chunks = ((last << lb) + kChunk - 1) / kChunk;  // top << lb is below 2^23
  const int per = (all_chunks + clusters - 1) / clusters;
  const int c0 = min(rank * per, all_chunks);
  const int chunks = min(c0 + per, all_chunks) - c0;
  const int slot0 = c0 * kChunk;  // in list order
  const int e0 = slot0 >> lb;
  const int e1 = chunks ? min(last, ((slot0 + chunks * kChunk - 1) >> lb) + 1) : e0;
  auto enter = [&](int i, int j, int phys) {
    if (i < e0 || i >= e1) return;
    s_entry[i - e0] = inside(j) && (unsigned)phys < (unsigned)p.num_blocks
                          ? make_int2(phys << lb, (int)min((int64_t)block, n - ((int64_t)j << lb)))
                          : make_int2(0, 0);
  };
#pragma unroll
  for (int k = 0; k < kEarly; ++k) enter(k * kThreads + tid, j_early[k], phys_early[k]);
  for (int i = max(e0, kEarly * kThreads) + tid; i < e1; i += kThreads) {
    const int j = list[i];
    enter(i, j, inside(j) ? table[j] : -1);
  }

  // q as MMA operand B: column `col` is query head col (mod 4 when G <= 4)
  uint32_t qb[kSteps][2];
  float q_scale = 1.f;  // FP8: what q's columns were divided by
  if constexpr (FP8) {
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
    q_scale = __int_as_float((127 + e) << 23);
    const float inv = __int_as_float((127 - e) << 23);
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      qb[k][0] = pack2<true>(bf16_lo(qw[k].x) * inv, bf16_hi(qw[k].x) * inv);
      qb[k][1] = pack2<true>(bf16_lo(qw[k].y) * inv, bf16_hi(qw[k].y) * inv);
    }
  } else {
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      qb[k][0] = qw[k].x;
      qb[k][1] = qw[k].y;
    }
  }
  // the logit factors of this lane's two accumulator columns 2c, 2c + 1
  float f0 = p.scale_log2, f1 = p.scale_log2, v_scale = 1.f;
  if constexpr (FP8) {
    const float ks = *p.k_scale;
    v_scale = *p.v_scale;
    f0 *= ks * __shfl_sync(0xffffffffu, q_scale, 4 * (2 * c));
    f1 *= ks * __shfl_sync(0xffffffffu, q_scale, 4 * (2 * c + 1));
  }
  __syncthreads();  // entries

  const uint32_t ring = smem_u32(smem) + warp * C::kStages * 2 * C::kTile;
  const int64_t stride = (int64_t)p.num_kv_heads * C::kRow;  // between tokens
  const uint8_t* kbase = static_cast<const uint8_t*>(p.k_cache) + (int64_t)kvh * C::kRow;
  const uint8_t* vbase = static_cast<const uint8_t*>(p.v_cache) + (int64_t)kvh * C::kRow;
  const int my = chunks > warp ? (chunks - warp + kWarps - 1) / kWarps : 0;  // this warp's chunks

  auto load = [&](int it) {
    if (it < my) {
      const int s0 = slot0 + (warp + it * kWarps) * kChunk;
      const uint32_t stage = ring + (it % C::kStages) * 2 * C::kTile;
      constexpr int kRowsPer = 32 / C::kPieces;  // tokens per instruction
      const int piece = lane % C::kPieces;
#pragma unroll
      for (int r = 0; r < kChunk / kRowsPer; ++r) {
        const int t = r * kRowsPer + lane / C::kPieces;
        const int e = ((s0 + t) >> lb) - e0, off = (s0 + t) & (block - 1);
        int2 en = make_int2(0, 0);
        if (e < e1 - e0) en = s_entry[e];
        const bool in = off < en.y;
        const int64_t at = (int64_t)(in ? en.x + off : 0) * stride + piece * 16;
        const uint32_t dst = stage + t * C::kRow + C::swizzle(t, piece) * 16;
        cp_async_16(dst, kbase + at, in ? 16 : 0);  // zeros where there is no token
        cp_async_16(dst + C::kTile, vbase + at, in ? 16 : 0);
      }
    }
    cp_async_commit();
  };

  float o[kSteps][4];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;

#pragma unroll
  for (int s = 0; s < C::kStages - 1; ++s) load(s);
  for (int it = 0; it < my; ++it) {
    load(it + C::kStages - 1);
    cp_async_wait<C::kStages - 1>();
    __syncwarp();
    const uint32_t kt = ring + (it % C::kStages) * 2 * C::kTile;
    const uint32_t vt = kt + C::kTile;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    {
      const int r = (lane & 7) + ((lane >> 3) & 1) * 8;
      const uint32_t base = kt + r * C::kRow;
      if constexpr (FP8) {
#pragma unroll
        for (int k = 0; k < kSteps; k += 2) {
          uint32_t w[4];
          ldmatrix_x4(w, base + C::swizzle(r, k + (lane >> 4)) * 16);
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // the two 16-channel pieces
            const uint32_t x = w[2 * h], y = w[2 * h + 1];
            const uint32_t a[4] = {widen((uint16_t)x), widen((uint16_t)y),
                                   widen((uint16_t)(x >> 16)), widen((uint16_t)(y >> 16))};
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
    const int s0 = slot0 + (warp + it * kWarps) * kChunk;
    bool in[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int sl = s0 + g + 8 * h;
      const int e = (sl >> lb) - e0;
      in[h] = e < e1 - e0 && (sl & (block - 1)) < s_entry[e].y;
    }
    const float x00 = in[0] ? s[0] * f0 : -INFINITY, x01 = in[0] ? s[1] * f1 : -INFINITY;
    const float x10 = in[1] ? s[2] * f0 : -INFINITY, x11 = in[1] ? s[3] * f1 : -INFINITY;
    float n0 = fmaxf(x00, x10), n1 = fmaxf(x01, x11);
#pragma unroll
    for (int d = 4; d < 32; d *= 2) {
      n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, d));
      n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, d));
    }
    n0 = fmaxf(n0, m0);
    n1 = fmaxf(n1, m1);
    if (__any_sync(0xffffffffu, n0 > m0 || n1 > m1)) {
      const float a0 = m0 == -INFINITY ? 0.f : fast_exp2(m0 - n0);
      const float a1 = m1 == -INFINITY ? 0.f : fast_exp2(m1 - n1);
      l0 *= a0;
      l1 *= a1;
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
    constexpr float kRaise = FP8 ? 16384.f : 1.f;  // the factor that P and its sum carry
    const float z0 = m0 == -INFINITY ? 0.f : m0, z1 = m1 == -INFINITY ? 0.f : m1;
    const float p00 = fast_exp2(x00 - z0) * kRaise, p01 = fast_exp2(x01 - z1) * kRaise;
    const float p10 = fast_exp2(x10 - z0) * kRaise, p11 = fast_exp2(x11 - z1) * kRaise;
    l0 += p00 + p10;
    l1 += p01 + p11;
    uint32_t hi0 = pack2<FP8>(p00, p01), hi1 = pack2<FP8>(p10, p11);
    const float2 r0 = unpack2<FP8>(hi0), r1 = unpack2<FP8>(hi1);
    uint32_t lo0 = pack2<FP8>(p00 - r0.x, p01 - r0.y), lo1 = pack2<FP8>(p10 - r1.x, p11 - r1.y);
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
    if constexpr (FP8) {
      // a transposed 16-bit unit holds channels 2g and 2g + 1 of a token: the
      // even ones become row g of the tile, the odd ones row g + 8
      const int r = (lane & 7) + ((lane >> 3) & 1) * 8;
#pragma unroll
      for (int k = 0; k < kSteps; k += 2) {
        uint32_t w[4];
        ldmatrix_x4_trans(w, vt + r * C::kRow + C::swizzle(r, k + (lane >> 4)) * 16);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t x = __byte_perm(w[2 * h], 0, 0x3120), y = __byte_perm(w[2 * h + 1], 0, 0x3120);
          const uint32_t a[4] = {widen((uint16_t)x), widen((uint16_t)(x >> 16)),
                                 widen((uint16_t)y), widen((uint16_t)(y >> 16))};
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
    __syncwarp();  // the stage may be filled again
  }
  cp_async_wait<0>();

  // the warps' results: max, sum and channels per column
#pragma unroll
  for (int d = 4; d < 32; d *= 2) {
    l0 += __shfl_xor_sync(0xffffffffu, l0, d);
    l1 += __shfl_xor_sync(0xffffffffu, l1, d);
  }
  __syncthreads();  // the ring is free
  float* mo = reinterpret_cast<float*>(smem);  // [warp][column][D]
  float* ml = mo + kWarps * 8 * D;             // [warp][column][2]
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int d0 = 16 * i + (FP8 ? 2 * g : g), d1 = FP8 ? d0 + 1 : d0 + 8;
    float* w0 = mo + (warp * 8 + 2 * c) * D;
    w0[d0] = o[i][0];
    w0[D + d0] = o[i][1];
    w0[d1] = o[i][2];
    w0[D + d1] = o[i][3];
  }
  if (g == 0) {
    float* w = ml + (warp * 8 + 2 * c) * 2;
    w[0] = m0;
    w[1] = l0;
    w[2] = m1;
    w[3] = l1;
  }
  __syncthreads();
  // the CTA's own result, unnormalised; in a cluster each CTA owns a share of
  // the outputs and is handed the others' parts of it
  const int share = (G * D + clusters - 1) / clusters;
  if (clusters > 1) asm volatile("barrier.cluster.wait.aligned;\n" ::: "memory");
  for (int i = tid; i < G * D; i += kThreads) {
    const int h = i / D, d = i % D;
    float mm = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, ml[(w * 8 + h) * 2]);
    float acc = 0.f, l = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float a = weight(ml[(w * 8 + h) * 2], mm);
      float x = mo[(w * 8 + h) * D + d];
      if (G <= 4) x += mo[(w * 8 + h + 4) * D + d];
      acc += a * x;
      l += a * ml[(w * 8 + h) * 2 + 1];
    }
    if (clusters == 1) {
      p.out[(int64_t)unit * G * D + i] = quotient(acc, l, v_scale);
    } else {
      const int owner = i / share;
      store_peer(&s_part[rank * share + i - owner * share], owner, acc);
      if (d < clusters) {
        store_peer(&s_state[rank][h][0], d, mm);
        store_peer(&s_state[rank][h][1], d, l);
      }
    }
  }
  if (clusters == 1) return;
  cluster_sync();  // all parts have arrived; peers' memory is not touched again
  for (int i = tid; i < share; i += kThreads) {
    const int o = rank * share + i;
    if (o >= G * D) break;
    const int h = o / D;
    float mm = -INFINITY;
    for (int r = 0; r < clusters; ++r) mm = fmaxf(mm, s_state[r][h][0]);
    float acc = 0.f, l = 0.f;
    for (int r = 0; r < clusters; ++r) {
      const float a = weight(s_state[r][h][0], mm);
      acc += a * s_part[r * share + i];
      l += a * s_state[r][h][1];
    }
    p.out[(int64_t)unit * G * D + o] = quotient(acc, l, v_scale);
  }
}

template <int D, int G, bool FP8>
cudaError_t launch_one(const SelectedParams& p, int num_sms, cudaStream_t stream) {
  using C = Cfg<D, FP8>;
  const int64_t units = (int64_t)p.num_rows * p.num_kv_heads;
  const int64_t tokens = (int64_t)p.top << p.log2_block_size;  // of a unit, at most
  // CTAs per unit: as many as run at two to an SM, while each has a chunk for
  // every warp (8 rows of 8 heads, 8192 tokens each in e4m3: 51.9 us with 1,
  // 31.1 with 2, 28.4 with 4, and 40.7 with 5, which no longer run at once).
  // Up to 8, and 12 where these few units' lists leave each CTA four chunks a
  // warp and the SMs are not yet full (one row of 8 heads in bf16: 2048 blocks
  // 58.0 us with 8, 41.5 with 12, 63.6 with 16; 256 blocks 10.1, 8.6, 7.9; 64
  // blocks 5.1, 5.2, 5.1; 4 rows of 256 blocks 15.5, 22.2, 27.2).
  const int64_t chunks = tokens / (kChunk * C::kWarps);  // for every warp of a CTA
  const bool large = units * kLargeCluster <= 3 * num_sms / 2 && chunks >= 4 * kLargeCluster;
  int64_t c = 2 * num_sms / units;
  if (c > chunks) c = chunks;
  if (c > kMaxCluster) c = large ? kLargeCluster : kMaxCluster;
  if (c < 1) c = 1;
  const size_t smem = C::kRing + (size_t)p.top * sizeof(int2);
  const cudaError_t e = allow_large<decode_selected_kernel<D, G, FP8>>();
  if (e != cudaSuccess) return e;
  return launch_dependent<decode_selected_kernel<D, G, FP8>>(
      dim3((unsigned)(units * c)), dim3(C::kThreads), smem, stream, (int)c, p, (int)c);
}

template <int D, bool FP8>
cudaError_t launch_g(const SelectedParams& p, int group, int num_sms, cudaStream_t stream) {
  switch (group) {
    case 1: return launch_one<D, 1, FP8>(p, num_sms, stream);
    case 2: return launch_one<D, 2, FP8>(p, num_sms, stream);
    case 4: return launch_one<D, 4, FP8>(p, num_sms, stream);
    case 8: return launch_one<D, 8, FP8>(p, num_sms, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_decode_selected(const SelectedParams& p, int head_dim, int group, bool fp8,
                                   int num_sms, cudaStream_t stream) {
  if (head_dim == 128)
    return fp8 ? launch_g<128, true>(p, group, num_sms, stream)
               : launch_g<128, false>(p, group, num_sms, stream);
  return fp8 ? launch_g<64, true>(p, group, num_sms, stream)
             : launch_g<64, false>(p, group, num_sms, stream);
}

}  // namespace pa
