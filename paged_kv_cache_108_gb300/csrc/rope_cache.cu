// Rotary position embedding fused with the cache write; optionally behind an
// RMS norm of each query and key head, and into a cache of 8-bit rows.
//
// For the pair (x, y) that pair index i < rot_dim / 2 names in a head, with
// p the token's position on that pair's axis and (c, s) = (cos, sin) from
// row p of the caller's table,
//   x' = x c - y s,   y' = y c + x s
// in fp32, rounded once: queries to bf16 in q_out, keys to bf16 or e4m3 at
// the token's slot of the cache; values go to their slot unrotated.  Fusing
// the rotation with the write saves the rotated keys' trip through memory
// (one write and one read of [N, H_kv, d]) and a launch.
//
// Bound: bytes.  Each input is read once and each output written once.  A
// CTA takes a few tokens; its threads first issue the 16-byte loads of the
// queries, keys and values they own (two 8-element pieces holding 8 whole
// pairs, so that a rotation needs no exchange between threads), and while
// these are in flight the tokens' cosines and sines -- shared by all heads --
// are gathered into shared memory, one (pair, axis) per thread, which serves
// every assignment of axes to pairs alike.
//
// The norm, x / sqrt(mean x^2 + eps) * w per head, and the 8-bit rows' unit,
// max |x| / 127 per token and head, are sums and maxima over a head, which
// d / 16 neighbouring threads hold between them: three shuffles (two at 64
// channels) each, in fp32, and no further pass over memory.  A code is
// x / unit rounded to the nearest whole number (IEEE division, ties to even).
#include <cuda_bf16.h>

#include "launch.cuh"
#include "pa_device.cuh"
#include "pa_kernels.cuh"
#include "tc_ptx.cuh"

namespace pa {

namespace {

constexpr int kRopeThreads = 128;
constexpr int kRopeCtas = 8;       // per SM: what the registers are kept to
// Items in flight per thread: three, or two where a head's threads exchange (a
// prompt of 8192 tokens with the norm: bf16 50.5 us with three, 48.5 with two,
// 50.6 with one; into 8-bit rows and read back 71, 66, 70).
constexpr int kRopeUnroll = 3;
constexpr int unroll_of(bool together) { return together ? 2 : kRopeUnroll; }
constexpr int kRopeMaxTokens = 8;  // tokens per CTA at most

// The position axis of pair i: one axis, sections in a row, or axes in turn
// (pair i takes axis i % num_axes while that axis has pairs left, else 0).
__device__ __forceinline__ int axis_of_pair(const RopeParams& p, int i) {
  if (p.num_axes == 1) return 0;
  if (p.in_turn) {
    const int a = i % p.num_axes;
    return i < p.num_axes * p.sections[a] ? a : 0;
  }
  int a = 0, end = p.sections[0];
#pragma unroll
  for (int k = 1; k < 4; ++k)
    if (k < p.num_axes && i >= end) {
      a = k;
      end += p.sections[k];
    }
  return a;
}

// x / unit as a code: whole numbers up to 127, ties to even.  A row's largest
// |x| gives 127 exactly.  (A row of zeros has unit 0; one that holds an
// infinity or a NaN an infinite or NaN one, whose product with 0 is NaN: their
// codes are 0.)
__device__ __forceinline__ uint32_t code_of(float x, float unit) {
  const float r = rintf(__fdiv_rn(x, unit));
  return (uint32_t)(int)fminf(fmaxf(r, -127.f), 127.f) & 255;
}

// Stores a piece: rounded from f, or, for a bf16 destination whose channels
// are unchanged, as it was loaded, so that a NaN keeps its bits.
template <KvFormat F>
__device__ __forceinline__ void store_piece(void* cache, int64_t elem, const float* f, float scale,
                                            const uint4& loaded, bool changed) {
  if constexpr (F == kBf16) {
    uint4 w;
    w.x = changed ? pack_bf16x2_rn(f[0], f[1]) : loaded.x;
    w.y = changed ? pack_bf16x2_rn(f[2], f[3]) : loaded.y;
    w.z = changed ? pack_bf16x2_rn(f[4], f[5]) : loaded.z;
    w.w = changed ? pack_bf16x2_rn(f[6], f[7]) : loaded.w;
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(cache) + elem) = w;
  } else if constexpr (F == kInt8) {
    uint2 w = make_uint2(0, 0);
    if (scale > 0.f && scale < INFINITY) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w.x |= code_of(f[i], scale) << (8 * i);
        w.y |= code_of(f[4 + i], scale) << (8 * i);
      }
    }
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(cache) + elem) = w;
  } else {
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      h[i] = pack_e4m3x2_rn(__fdiv_rn(f[2 * i], scale), __fdiv_rn(f[2 * i + 1], scale));
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(cache) + elem) =
        make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
  }
}

__device__ __forceinline__ void turn(float& x, float& y, float c, float s) {
  const float u = x * c - y * s;
  y = y * c + x * s;
  x = u;
}

// Over the kCols neighbouring threads that hold a head between them.
template <int kCols>
__device__ __forceinline__ float head_sum(float x) {
#pragma unroll
  for (int d = 1; d < kCols; d *= 2) x += __shfl_xor_sync(0xffffffffu, x, d);
  return x;
}
template <int kCols>
__device__ __forceinline__ uint32_t head_max(uint32_t x) {
#pragma unroll
  for (int d = 1; d < kCols; d *= 2) x = max(x, __shfl_xor_sync(0xffffffffu, x, d));
  return x;
}

template <int D, KvFormat F, bool NORM, int kUnroll>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas)
    rope_and_cache_kernel(const __grid_constant__ RopeParams p) {
  constexpr bool FP8 = F == kE4m3;
  constexpr bool kTogether = NORM || F == kInt8;  // a head's threads exchange: none leaves early
  constexpr int kCols = D / 16;  // items (two 8-element pieces) per head
  constexpr int kRows = kRopeThreads / kCols;  // heads the CTA takes at a time
  __shared__ __align__(16) float2 s_cs[kRopeMaxTokens][D / 2];
  __shared__ int s_slot[kRopeMaxTokens];
  __shared__ int s_ok[kRopeMaxTokens];
  __shared__ __align__(16) float s_weight[NORM ? 2 : 1][NORM ? D : 4];  // queries', keys'
  ptx::grid_dependency_wait();
  ptx::grid_launch_dependents();
  const int tid = threadIdx.x;
  const int64_t tok0 = (int64_t)blockIdx.x * p.tokens_per_cta;
  const int ntok = (int)min((int64_t)p.tokens_per_cta, p.num_tokens - tok0);
  const int half = p.rot_dim / 2;
  const int kv0 = p.num_heads, v0 = kv0 + p.num_kv_heads, heads = v0 + p.num_kv_heads;
  // a thread's two pieces start at the same channels in every head: column c
  // and its partner half the rotated width on, or two neighbours where pairs
  // are adjacent and where nothing is rotated
  const int c = tid % kCols;
  const bool turned = c < p.rot_dim / 16;
  const bool split = turned && !p.adjacent;
  const int e0 = split ? 8 * c : 16 * c, e1 = split ? half + 8 * c : 16 * c + 8;
  const int first = tid / kCols, rows = ntok * heads;
  float ks = 1.f, vs = 1.f;
  if (FP8) {
    ks = *p.k_scale;
    vs = *p.v_scale;
  }
  const int base0 = blockIdx.y * kRows * kUnroll;
  for (int base = base0; base < rows; base += gridDim.y * kRows * kUnroll) {
    uint4 a[kUnroll], b[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int r = base + u * kRows + first;
      if (r >= rows) continue;
      const int t = (int)__umulhi((unsigned)r, p.heads_inverse), h = r - t * heads;
      const __nv_bfloat16* row =
          h < kv0 ? p.query + (tok0 + t) * p.q_stride + h * D
                  : (h < v0 ? p.key + (tok0 + t) * p.k_stride + (h - kv0) * D
                            : p.value + (tok0 + t) * p.v_stride + (h - v0) * D);
      a[u] = *reinterpret_cast<const uint4*>(row + e0);
      b[u] = *reinterpret_cast<const uint4*>(row + e1);
    }
    if (base == base0) {
      if (tid < ntok) {
        const int64_t tok = tok0 + tid;
        s_slot[tid] = p.slot_mapping[tok];
        bool ok = true;
        for (int x = 0; x < p.num_axes; ++x)
          ok &= (unsigned)p.positions[x * p.num_tokens + tok] < (unsigned)p.max_position;
        s_ok[tid] = ok;
      }
      if constexpr (NORM) {
        for (int i = tid; i < 2 * D; i += kRopeThreads)
          s_weight[i / D][i % D] = (i < D ? p.q_weight : p.k_weight)[i % D];
      }
      for (int i = tid; i < ntok * half; i += kRopeThreads) {
        const int t = ntok == 1 ? 0 : i / half, pair = i - t * half;
        const int pos = p.positions[axis_of_pair(p, pair) * p.num_tokens + tok0 + t];
        float2 cs = make_float2(1.f, 0.f);
        if ((unsigned)pos < (unsigned)p.max_position) {
          const float* row = p.cos_sin + (int64_t)pos * p.rot_dim;
          cs = make_float2(row[pair], row[half + pair]);
        }
        s_cs[t][pair] = cs;
      }
      __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int r = base + u * kRows + first;
      if (!kTogether && r >= rows) continue;
      const bool there = r < rows;
      const int t = there ? (int)__umulhi((unsigned)r, p.heads_inverse) : 0;
      const int h = there ? r - t * heads : 0;
      if (!kTogether && !s_ok[t]) continue;
      if (kTogether && !there) a[u] = b[u] = make_uint4(0, 0, 0, 0);
      float x[8], y[8];
      Unpack16<false>::run(a[u], x);
      Unpack16<false>::run(b[u], y);
      const bool turns = h < v0 && turned;
      const bool changed = turns || (NORM && h < v0);
      if constexpr (NORM) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss += x[i] * x[i] + y[i] * y[i];
        ss = head_sum<kCols>(ss);
        if (h < v0) {
          const float f = rsqrtf(ss * (1.f / D) + p.eps);
          const float4* w = reinterpret_cast<const float4*>(s_weight[h >= kv0]);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float4 u = w[e0 / 4 + i], v = w[e1 / 4 + i];
            x[4 * i] *= f * u.x, x[4 * i + 1] *= f * u.y;
            x[4 * i + 2] *= f * u.z, x[4 * i + 3] *= f * u.w;
            y[4 * i] *= f * v.x, y[4 * i + 1] *= f * v.y;
            y[4 * i + 2] *= f * v.z, y[4 * i + 3] *= f * v.w;
          }
        }
      }
      if (turns) {
        const float4* cs = reinterpret_cast<const float4*>(&s_cs[t][8 * c]);
        if (p.adjacent) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float4 m = cs[i], n = cs[2 + i];
            turn(x[4 * i], x[4 * i + 1], m.x, m.y);
            turn(x[4 * i + 2], x[4 * i + 3], m.z, m.w);
            turn(y[4 * i], y[4 * i + 1], n.x, n.y);
            turn(y[4 * i + 2], y[4 * i + 3], n.z, n.w);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 m = cs[i];
            turn(x[2 * i], y[2 * i], m.x, m.y);
            turn(x[2 * i + 1], y[2 * i + 1], m.z, m.w);
          }
        }
      }
      float unit = 0.f;
      if constexpr (F == kInt8) {
        // |x| as bits orders like |x|, infinities and then NaNs above all
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          m = max(m, max(__float_as_uint(x[i]) & 0x7fffffffu, __float_as_uint(y[i]) & 0x7fffffffu));
        unit = __fdiv_rn(__uint_as_float(head_max<kCols>(m)), 127.f);
      }
      if (kTogether && (!there || !s_ok[t])) continue;
      if (h < kv0) {
        const int64_t row = ((tok0 + t) * kv0 + h) * D;
        store_piece<kBf16>(p.q_out, row + e0, x, 1.f, a[u], changed);
        store_piece<kBf16>(p.q_out, row + e1, y, 1.f, b[u], changed);
      } else {
        const int slot = s_slot[t];
        if (slot < 0 || slot >= p.num_slots) continue;  // padding token or bad slot
        const bool is_v = h >= v0;
        const int64_t at = (int64_t)slot * p.num_kv_heads + h - (is_v ? v0 : kv0);
        const int64_t row = at * D;
        void* cache = is_v ? p.v_cache : p.k_cache;
        const float scale = F == kInt8 ? unit : (is_v ? vs : ks);
        store_piece<F>(cache, row + e0, x, scale, a[u], changed);
        store_piece<F>(cache, row + e1, y, scale, b[u], changed);
        if (F == kInt8 && c == 0) (is_v ? p.v_units : p.k_units)[at] = unit;
      }
    }
  }
}

template <int D, KvFormat F, bool NORM>
cudaError_t launch(RopeParams p, int num_sms, cudaStream_t stream) {
  // tokens per CTA: enough items for every thread's loads in flight
  const int heads = p.num_heads + 2 * p.num_kv_heads;
  const int64_t per_token = (int64_t)heads * (D / 16);
  int64_t t = kRopeThreads * kRopeUnroll / per_token;
  t = t < 1 ? 1 : (t > kRopeMaxTokens ? kRopeMaxTokens : t);
  // A long call's CTAs take two tokens at least: the wait for positions, then
  // table rows, then the barrier is paid once for both (8192 tokens of 48
  // heads: 49.1 us with one, 40.2 with two, 40.5 with four).  A short call is
  // spread over the SMs instead.
  if (p.num_tokens >= 2 * kRopeCtas * num_sms && t < 2) t = 2;
  const int64_t spread = p.num_tokens / (2 * num_sms);
  if (t > spread) t = spread < 1 ? 1 : spread;
  // ceil(2^32 / heads): r / heads is the high half of r * it while r * heads
  // is below 2^32 (r < 2 * heads <= 2^16, or 8 * heads <= 2^9)
  p.heads_inverse = (uint32_t)((((uint64_t)1 << 32) + heads - 1) / heads);
  p.tokens_per_cta = (int)t;
  const dim3 b(kRopeThreads);
  const unsigned ctas = (unsigned)((p.num_tokens + t - 1) / t);
  // A short call's tokens are shared by as many CTAs as give each thread one
  // item: less work behind each wait (1 token of 48 heads: 2.96 us alone, 1.98
  // by 3; 64 in e4m3 3.63, 2.66; 300 4.04, 3.70; 600 4.95, 5.62, where the
  // CTAs no longer run at once).
  const int at_once = kRopeThreads / (D / 16);  // heads of a CTA
  const int64_t parts = (t * heads + at_once - 1) / at_once;
  if (ctas * parts <= 6 * num_sms)
    return launch_dependent<rope_and_cache_kernel<D, F, NORM, 1>>(dim3(ctas, (unsigned)parts), b, 0,
                                                                  stream, 1, p);
  constexpr int U = unroll_of(NORM || F == kInt8);
  return launch_dependent<rope_and_cache_kernel<D, F, NORM, U>>(dim3(ctas), b, 0, stream, 1, p);
}

template <int D, KvFormat F>
cudaError_t launch_norm(const RopeParams& p, int num_sms, cudaStream_t stream) {
  return p.q_weight ? launch<D, F, true>(p, num_sms, stream) : launch<D, F, false>(p, num_sms, stream);
}

}  // namespace

cudaError_t launch_rope_and_cache(RopeParams p, int head_dim, bool fp8, int num_sms,
                                  cudaStream_t stream) {
  if (head_dim == 128)
    return fp8 ? launch<128, kE4m3, false>(p, num_sms, stream)
               : launch<128, kBf16, false>(p, num_sms, stream);
  return fp8 ? launch<64, kE4m3, false>(p, num_sms, stream)
             : launch<64, kBf16, false>(p, num_sms, stream);
}

cudaError_t launch_norm_rope_and_cache(RopeParams p, int head_dim, KvFormat format, int num_sms,
                                       cudaStream_t stream) {
  switch (format) {
    case kBf16:
      return head_dim == 128 ? launch_norm<128, kBf16>(p, num_sms, stream)
                             : launch_norm<64, kBf16>(p, num_sms, stream);
    case kE4m3:
      return head_dim == 128 ? launch_norm<128, kE4m3>(p, num_sms, stream)
                             : launch_norm<64, kE4m3>(p, num_sms, stream);
    case kInt8:
      return head_dim == 128 ? launch_norm<128, kInt8>(p, num_sms, stream)
                             : launch_norm<64, kInt8>(p, num_sms, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace pa
