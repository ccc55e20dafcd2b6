// Rotary position embedding fused with the cache write.
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
#include <cuda_bf16.h>

#include "launch.cuh"
#include "pa_device.cuh"
#include "pa_kernels.cuh"
#include "tc_ptx.cuh"

namespace pa {

namespace {

constexpr int kRopeThreads = 128;
constexpr int kRopeCtas = 8;       // per SM: what the registers are kept to
constexpr int kRopeUnroll = 3;     // items in flight per thread
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

// Stores a piece: rounded from f, or, for a bf16 destination whose channels
// are not rotated, as it was loaded, so that a NaN keeps its bits.
__device__ __forceinline__ void store_piece(void* cache, int64_t elem, const float* f, bool fp8,
                                            float scale, const uint4& loaded, bool rotated) {
  if (!fp8) {
    uint4 w;
    w.x = rotated ? pack_bf16x2_rn(f[0], f[1]) : loaded.x;
    w.y = rotated ? pack_bf16x2_rn(f[2], f[3]) : loaded.y;
    w.z = rotated ? pack_bf16x2_rn(f[4], f[5]) : loaded.z;
    w.w = rotated ? pack_bf16x2_rn(f[6], f[7]) : loaded.w;
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(cache) + elem) = w;
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

template <int D, bool FP8, int kUnroll>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas)
    rope_and_cache_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kCols = D / 16;  // items (two 8-element pieces) per head
  constexpr int kRows = kRopeThreads / kCols;  // heads the CTA takes at a time
  __shared__ __align__(16) float2 s_cs[kRopeMaxTokens][D / 2];
  __shared__ int s_slot[kRopeMaxTokens];
  __shared__ int s_ok[kRopeMaxTokens];
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
      if (r >= rows) continue;
      const int t = (int)__umulhi((unsigned)r, p.heads_inverse), h = r - t * heads;
      if (!s_ok[t]) continue;
      float x[8], y[8];
      Unpack16<false>::run(a[u], x);
      Unpack16<false>::run(b[u], y);
      const bool turns = h < v0 && turned;
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
      if (h < kv0) {
        const int64_t row = ((tok0 + t) * kv0 + h) * D;
        store_piece(p.q_out, row + e0, x, false, 1.f, a[u], turns);
        store_piece(p.q_out, row + e1, y, false, 1.f, b[u], turns);
      } else {
        const int slot = s_slot[t];
        if (slot < 0 || slot >= p.num_slots) continue;  // padding token or bad slot
        const bool is_v = h >= v0;
        const int64_t row = ((int64_t)slot * p.num_kv_heads + h - (is_v ? v0 : kv0)) * D;
        void* cache = is_v ? p.v_cache : p.k_cache;
        const float scale = is_v ? vs : ks;
        store_piece(cache, row + e0, x, FP8, scale, a[u], turns);
        store_piece(cache, row + e1, y, FP8, scale, b[u], turns);
      }
    }
  }
}

}  // namespace

cudaError_t launch_rope_and_cache(RopeParams p, int head_dim, bool fp8, int num_sms,
                                  cudaStream_t stream) {
  // tokens per CTA: enough items for every thread's loads in flight
  const int heads = p.num_heads + 2 * p.num_kv_heads;
  const int64_t per_token = (int64_t)heads * (head_dim / 16);
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
  const int at_once = kRopeThreads / (head_dim / 16);  // heads of a CTA
  const int64_t parts = (t * heads + at_once - 1) / at_once;
  if (ctas * parts <= 6 * num_sms) {
    const dim3 g(ctas, (unsigned)parts);
    if (head_dim == 128)
      return fp8 ? launch_dependent<rope_and_cache_kernel<128, true, 1>>(g, b, 0, stream, 1, p)
                 : launch_dependent<rope_and_cache_kernel<128, false, 1>>(g, b, 0, stream, 1, p);
    return fp8 ? launch_dependent<rope_and_cache_kernel<64, true, 1>>(g, b, 0, stream, 1, p)
               : launch_dependent<rope_and_cache_kernel<64, false, 1>>(g, b, 0, stream, 1, p);
  }
  const dim3 g(ctas);
  constexpr int U = kRopeUnroll;
  if (head_dim == 128)
    return fp8 ? launch_dependent<rope_and_cache_kernel<128, true, U>>(g, b, 0, stream, 1, p)
               : launch_dependent<rope_and_cache_kernel<128, false, U>>(g, b, 0, stream, 1, p);
  return fp8 ? launch_dependent<rope_and_cache_kernel<64, true, U>>(g, b, 0, stream, 1, p)
             : launch_dependent<rope_and_cache_kernel<64, false, U>>(g, b, 0, stream, 1, p);
}

}  // namespace pa
