// Reading a paged cache back: rows [num_rows, H_kv, d] of bf16 keys and
// values, sequence i's tokens first_tokens[i] .. context_lens[i] - 1 from row
// out_start_loc[i] on.
//   value = element (bf16) | element * scale (e4m3) | code * unit[token, head]
// (int8), in fp32, rounded once.
//
// Bound: bytes, each read or written once (8-bit caches: 1 in, 2 out).  All
// heads of a token lie in one row of the cache and of the output, so a CTA
// takes a few tokens and streams their rows in 16-byte pieces; what a row
// needs first -- its sequence, then that one's start and length, then the
// block -- is looked up once per token, by one warp for all its tokens with
// 32 boundaries compared at a time.
#include <cuda_bf16.h>

#include "launch.cuh"
#include "pa_device.cuh"
#include "pa_kernels.cuh"
#include "tc_ptx.cuh"

namespace pa {

namespace {

constexpr int kThreads = 256;
// Pieces in flight per thread.  (e4m3 with four: 8187 tokens of 8 heads 13.3 us,
// with two 11.2; bf16 64 contexts 172 us with four, 177 with two.)
constexpr int unroll_of(KvFormat f) { return f == kBf16 ? 4 : 2; }
constexpr int kMaxTokens = 32;  // tokens per CTA at most

// The sequence whose rows hold `row`: the number of starts[1 ..] <= row, by
// the whole warp, 32 boundaries at a time.
__device__ __forceinline__ int sequence_of(const int32_t* starts, int num_seqs, int row,
                                           int lane) {
  int lo = 0, n = num_seqs;  // among the sequences lo .. lo + n
  while (n > 0) {
    const int step = n / 32 + 1;
    const int at = lane * step;  // boundary lo + at + step ends that many sequences
    const bool passed = at + step <= n && starts[lo + at + step] <= row;
    const int whole = __popc(__ballot_sync(0xffffffffu, passed)) * step;
    lo += whole;
    n = min(step - 1, n - whole);
  }
  return lo;
}

// Eight elements, times f, as bf16.
template <KvFormat F>
__device__ __forceinline__ uint4 widen8(uint2 w, float f) {
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t x = i ? w.y : w.x;
    float a, b, c, d;
    if constexpr (F == kE4m3) {
      const float2 lo = e4m3x2_to_float2((uint16_t)x), hi = e4m3x2_to_float2((uint16_t)(x >> 16));
      a = lo.x, b = lo.y, c = hi.x, d = hi.y;
    } else {
      a = (float)(int8_t)x, b = (float)(int8_t)(x >> 8);
      c = (float)(int8_t)(x >> 16), d = (float)((int)x >> 24);
    }
    r[2 * i] = pack_bf16x2_rn(a * f, b * f);
    r[2 * i + 1] = pack_bf16x2_rn(c * f, d * f);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// A piece is 16 bytes of the cache: 8 bf16 or 16 8-bit elements.
template <int D, KvFormat F>
__global__ void __launch_bounds__(kThreads)
    gather_cache_kernel(const __grid_constant__ GatherParams p, int tokens_per_cta,
                        uint32_t pieces_inverse) {
  constexpr int kElems = F == kBf16 ? 8 : 16, kUnroll = unroll_of(F);
  __shared__ int s_slot[kMaxTokens];
  ptx::grid_dependency_wait();
  ptx::grid_launch_dependents();
  const int tid = threadIdx.x, lane = tid % 32;
  const int64_t row0 = (int64_t)blockIdx.x * tokens_per_cta;
  const int ntok = (int)min((int64_t)tokens_per_cta, p.num_rows - row0);
  for (int t = tid / 32; t < ntok; t += kThreads / 32) {  // a warp per token
    const int row = (int)row0 + t;
    const int seq = sequence_of(p.out_start_loc, p.num_seqs, row, lane);
    int slot = -1;
    if (lane == 0 && seq < p.num_seqs) {
      // (three loads at once, then the block's)
      const int64_t first = p.first_tokens ? p.first_tokens[seq] : 0;
      const int64_t start = p.out_start_loc[seq], end = p.context_lens[seq];
      const int64_t tok = first + row - start;
      if (first >= 0 && tok >= first && tok < end &&
          tok < (int64_t)p.max_blocks << p.log2_block_size) {
        const int phys =
            p.block_tables[(int64_t)seq * p.max_blocks + (tok >> p.log2_block_size)];
        if ((unsigned)phys < (unsigned)p.num_blocks)
          slot = (phys << p.log2_block_size) + (int)(tok & ((1 << p.log2_block_size) - 1));
      }
    }
    if (lane == 0) s_slot[t] = slot;
  }
  float ks = 1.f, vs = 1.f;
  if constexpr (F == kE4m3) {
    ks = *p.k_scale;
    vs = *p.v_scale;
  }
  __syncthreads();
  // a thread's 16 elements of an 8-bit cache are 32 bytes of the output
  const bool whole_sectors =
      (reinterpret_cast<uintptr_t>(p.k_out) | reinterpret_cast<uintptr_t>(p.v_out)) % 32 == 0;
  const int per_row = p.num_kv_heads * (D / kElems);  // pieces of a token's keys
  const int pieces = 2 * per_row;                     // and values
  const int64_t all = (int64_t)ntok * pieces;
  for (int64_t base = tid; base < all; base += kThreads * kUnroll) {
    uint4 w[kUnroll];
    float f[kUnroll];
    int64_t to[kUnroll];  // element of the output, or -1
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t i = base + u * kThreads;
      to[u] = -1;
      f[u] = 1.f;
      if (i >= all) continue;
      const int t = tokens_per_cta == 1 ? 0 : (int)__umulhi((unsigned)i, pieces_inverse);
      const int x = (int)(i - (int64_t)t * pieces);
      const int slot = s_slot[t];
      if (slot < 0) continue;
      const bool is_v = x >= per_row;
      const int piece = is_v ? x - per_row : x;
      const int64_t row = (int64_t)slot * per_row + piece;
      w[u] = __ldcs(reinterpret_cast<const uint4*>(is_v ? p.v_cache : p.k_cache) + row);
      if constexpr (F == kE4m3) f[u] = is_v ? vs : ks;
      if constexpr (F == kInt8)
        f[u] = (is_v ? p.v_scale : p.k_scale)[(int64_t)slot * p.num_kv_heads + piece / (D / 16)];
      to[u] = ((row0 + t) * per_row + piece) * kElems;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (to[u] < 0) continue;
      const int64_t i = base + u * kThreads;
      const int t = tokens_per_cta == 1 ? 0 : (int)__umulhi((unsigned)i, pieces_inverse);
      const bool is_v = i - (int64_t)t * pieces >= per_row;
      uint4* o = reinterpret_cast<uint4*>((is_v ? p.v_out : p.k_out) + to[u]);
      if constexpr (F == kBf16) {
        __stcs(o, w[u]);
      } else {
        const uint4 x = widen8<F>(make_uint2(w[u].x, w[u].y), f[u]);
        const uint4 y = widen8<F>(make_uint2(w[u].z, w[u].w), f[u]);
        if (whole_sectors) {
          asm volatile("st.global.cs.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(o),
                       "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w), "r"(y.x), "r"(y.y), "r"(y.z),
                       "r"(y.w)
                       : "memory");
        } else {
          __stcs(o, x);
          __stcs(o + 1, y);
        }
      }
    }
  }
}

template <int D, KvFormat F>
cudaError_t launch_one(const GatherParams& p, int num_sms, cudaStream_t stream) {
  const int64_t pieces = 2 * (int64_t)p.num_kv_heads * (D / (F == kBf16 ? 8 : 16));
  int64_t t = kThreads * unroll_of(F) / pieces;
  t = t < 1 ? 1 : (t > kMaxTokens ? kMaxTokens : t);
  const int64_t spread = p.num_rows / (4 * num_sms);  // a short call uses every SM
  if (t > spread) t = spread < 1 ? 1 : spread;
  // ceil(2^32 / pieces): i / pieces is the high half of i * it while i <
  // t * pieces <= 1024
  const uint32_t inverse = (uint32_t)((((uint64_t)1 << 32) + pieces - 1) / pieces);
  return launch_dependent<gather_cache_kernel<D, F>>(
      dim3((unsigned)((p.num_rows + t - 1) / t)), dim3(kThreads), 0, stream, 1, p, (int)t, inverse);
}

template <int D>
cudaError_t launch_d(const GatherParams& p, KvFormat format, int num_sms, cudaStream_t stream) {
  switch (format) {
    case kBf16: return launch_one<D, kBf16>(p, num_sms, stream);
    case kE4m3: return launch_one<D, kE4m3>(p, num_sms, stream);
    case kInt8: return launch_one<D, kInt8>(p, num_sms, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_gather_cache(const GatherParams& p, int head_dim, KvFormat format, int num_sms,
                                cudaStream_t stream) {
  return head_dim == 128 ? launch_d<128>(p, format, num_sms, stream)
                         : launch_d<64>(p, format, num_sms, stream);
}

}  // namespace pa
