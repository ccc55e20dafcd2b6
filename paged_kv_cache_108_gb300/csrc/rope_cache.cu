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
constexpr int kRopeUnroll = 4;     // work items in flight per thread
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

__device__ __forceinline__ void store_piece(void* cache, int64_t elem, const float* f, bool fp8,
                                            float scale) {
  if (!fp8) {
    uint4 w;
    w.x = pack_bf16x2_rn(f[0], f[1]);
    w.y = pack_bf16x2_rn(f[2], f[3]);
    w.z = pack_bf16x2_rn(f[4], f[5]);
    w.w = pack_bf16x2_rn(f[6], f[7]);
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

template <int D, bool FP8>
__global__ void __launch_bounds__(kRopeThreads)
    rope_and_cache_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kCols = D / 16;  // items (two 8-element pieces) per head
  __shared__ float2 s_cs[kRopeMaxTokens][D / 2];
  __shared__ int s_slot[kRopeMaxTokens];
  __shared__ int s_ok[kRopeMaxTokens];
  ptx::grid_dependency_wait();
  ptx::grid_launch_dependents();
  const int tid = threadIdx.x;
  const int64_t tok0 = (int64_t)blockIdx.x * p.tokens_per_cta;
  const int ntok = (int)min((int64_t)p.tokens_per_cta, p.num_tokens - tok0);
  const int half = p.rot_dim / 2;
  const int rot_cols = p.rot_dim / 16;
  const int heads = p.num_heads + 2 * p.num_kv_heads;
  const int per_token = heads * kCols;
  const int items = ntok * per_token;
  float ks = 1.f, vs = 1.f;
  if (FP8) {
    ks = *p.k_scale;
    vs = *p.v_scale;
  }
  bool staged = false;
  for (int base = 0; base < items; base += kRopeThreads * kRopeUnroll) {
    uint4 a[kRopeUnroll], b[kRopeUnroll];
    int tl[kRopeUnroll], hd[kRopeUnroll], e0[kRopeUnroll], e1[kRopeUnroll], col[kRopeUnroll];
#pragma unroll
    for (int u = 0; u < kRopeUnroll; ++u) {
      const int it = base + u * kRopeThreads + tid;
      tl[u] = -1;
      if (it >= items) continue;
      const int t = it / per_token, r = it - t * per_token;
      const int h = r / kCols, c = r % kCols;
      tl[u] = t;
      hd[u] = h;
      col[u] = c;
      // the pieces' first elements: c and its partner half the rotated width
      // on; neighbours for adjacent pairs and for channels left unrotated
      const bool split = !p.adjacent && c < rot_cols;
      e0[u] = split ? 8 * c : 16 * c;
      e1[u] = split ? half + 8 * c : 16 * c + 8;
      const __nv_bfloat16* row;
      if (h < p.num_heads)
        row = p.query + (tok0 + t) * p.q_stride + h * D;
      else if (h < p.num_heads + p.num_kv_heads)
        row = p.key + (tok0 + t) * p.k_stride + (h - p.num_heads) * D;
      else
        row = p.value + (tok0 + t) * p.v_stride + (h - p.num_heads - p.num_kv_heads) * D;
      a[u] = *reinterpret_cast<const uint4*>(row + e0[u]);
      b[u] = *reinterpret_cast<const uint4*>(row + e1[u]);
    }
    if (!staged) {  // the same for every thread of the CTA
      staged = true;
      if (tid < ntok) {
        const int64_t tok = tok0 + tid;
        s_slot[tid] = p.slot_mapping[tok];
        bool ok = true;
        for (int x = 0; x < p.num_axes; ++x)
          ok &= (unsigned)p.positions[x * p.num_tokens + tok] < (unsigned)p.max_position;
        s_ok[tid] = ok;
      }
      for (int i = tid; i < ntok * half; i += kRopeThreads) {
        const int t = i / half, pair = i - t * half;
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
    for (int u = 0; u < kRopeUnroll; ++u) {
      if (tl[u] < 0 || !s_ok[tl[u]]) continue;
      const int64_t tok = tok0 + tl[u];
      const bool is_q = hd[u] < p.num_heads;
      const bool is_v = hd[u] >= p.num_heads + p.num_kv_heads;
      float x[8], y[8];
      Unpack16<false>::run(a[u], x);
      Unpack16<false>::run(b[u], y);
      if (!is_v && col[u] < rot_cols) {
        const float2* cs = &s_cs[tl[u]][8 * col[u]];
        if (p.adjacent) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 c0 = cs[i], c1 = cs[4 + i];
            const float x0 = x[2 * i], x1 = x[2 * i + 1], y0 = y[2 * i], y1 = y[2 * i + 1];
            x[2 * i] = x0 * c0.x - x1 * c0.y;
            x[2 * i + 1] = x1 * c0.x + x0 * c0.y;
            y[2 * i] = y0 * c1.x - y1 * c1.y;
            y[2 * i + 1] = y1 * c1.x + y0 * c1.y;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 c = cs[i];
            const float xi = x[i], yi = y[i];
            x[i] = xi * c.x - yi * c.y;
            y[i] = yi * c.x + xi * c.y;
          }
        }
      }
      if (is_q) {
        const int64_t row = (tok * p.num_heads + hd[u]) * D;
        store_piece(p.q_out, row + e0[u], x, false, 1.f);
        store_piece(p.q_out, row + e1[u], y, false, 1.f);
      } else {
        const int slot = s_slot[tl[u]];
        if (slot < 0 || slot >= p.num_slots) continue;  // padding token or bad slot
        const int h = hd[u] - p.num_heads - (is_v ? p.num_kv_heads : 0);
        const int64_t row = ((int64_t)slot * p.num_kv_heads + h) * D;
        void* cache = is_v ? p.v_cache : p.k_cache;
        const float scale = is_v ? vs : ks;
        store_piece(cache, row + e0[u], x, FP8, scale);
        store_piece(cache, row + e1[u], y, FP8, scale);
      }
    }
  }
}

}  // namespace

cudaError_t launch_rope_and_cache(RopeParams p, int head_dim, bool fp8, cudaStream_t stream) {
  // tokens per CTA: enough items for every thread's loads in flight
  const int64_t per_token = (int64_t)(p.num_heads + 2 * p.num_kv_heads) * (head_dim / 16);
  int64_t t = kRopeThreads * kRopeUnroll / per_token;
  t = t < 1 ? 1 : (t > kRopeMaxTokens ? kRopeMaxTokens : t);
  p.tokens_per_cta = (int)t;
  const int64_t grid = (p.num_tokens + t - 1) / t;
  const dim3 g((unsigned)grid), b(kRopeThreads);
  if (head_dim == 128)
    return fp8 ? launch_dependent<rope_and_cache_kernel<128, true>>(g, b, 0, stream, 1, p)
               : launch_dependent<rope_and_cache_kernel<128, false>>(g, b, 0, stream, 1, p);
  return fp8 ? launch_dependent<rope_and_cache_kernel<64, true>>(g, b, 0, stream, 1, p)
             : launch_dependent<rope_and_cache_kernel<64, false>>(g, b, 0, stream, 1, p);
}

}  // namespace pa
