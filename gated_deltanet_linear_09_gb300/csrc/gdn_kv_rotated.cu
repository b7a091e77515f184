// gdn_kv_rotated.cu -- the cache's append with the heads' RMSNorm and rotary positions on the way.
//
// Between an attention layer's projection and its cache every query and key vector is normed and turned:
// a chain of element-wise steps, so one pass does them all, and q, k and v are read once.  The floor is
// the bytes.  A CTA takes neighbouring tokens; a vector is D / 8 neighbouring lanes with 16 bytes each, so
// the norm's sum is a few shuffles.  In the half layout a lane's partner elements are loaded a second time,
// as raw bf16 (a hit in L1: the lines are the warp's own), which costs one instruction where exchanging
// them costs four.  Angles belong to tokens: they are computed once into shared memory, while the vectors'
// first loads are under way.
#include "gdn_kv.cuh"
#include "gdn_rotary.cuh"

namespace gdn {

namespace {

constexpr int kMostTokens = 32;
constexpr int kMostTurns = 2048;       // (cos, sin) of a CTA: tokens * half

__device__ __forceinline__ void unpack8(const uint4 u, float* v) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float* v) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The scale byte of a vector whose largest magnitude is `top`: the least 2^(b - 127), b >= 10, with
// top <= 448 * 2^(b - 127); 127 for a zero vector, 255 for one with an infinity or a NaN.
__device__ __forceinline__ int scale_byte_f32(float top) {
  const uint32_t u = __float_as_uint(top);
  if (u >= 0x7f800000u) return 255;
  if (u == 0) return 127;
  // 448 = 1.75 * 2^8
  const int e = (int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e < 10 ? 10 : e;
}

// 8 elements with this scale byte -> codes (the factor 2^(127 - b) is exact: 7 <= 254 - b <= 244).
__device__ __forceinline__ uint2 codes8(const float* v, int b) {
  if (b == 255) return make_uint2(0, 0);
  const float f = __uint_as_float((uint32_t)(254 - b) << 23);
  uint16_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h[i]) : "f"(v[2 * i + 1] * f), "f"(v[2 * i] * f));
  return make_uint2((uint32_t)h[0] | ((uint32_t)h[1] << 16), (uint32_t)h[2] | ((uint32_t)h[3] << 16));
}

template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// of magnitudes; a NaN is above all (as bits they order like numbers)
template <int L>
__device__ __forceinline__ float lanes_max(float v) {
  uint32_t u = __float_as_uint(v);
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) u = max(u, __shfl_xor_sync(0xffffffffu, u, o));
  return __uint_as_float(u);
}

template <int D, bool Q8, bool INTER>
__global__ void __launch_bounds__(256) append_rotated_kernel(const KvView c, const KvBatchView bt, int tokens,
                                                             const RotatedAppend a) {
  constexpr int L = D / 8, kSide = 32 / L;       // lanes of a vector, vectors of a warp at a time
  __shared__ long long place[kMostTokens];
  __shared__ int angle_at[kMostTokens];
  __shared__ __align__(16) float cs[kMostTurns], sn[kMostTurns];
  const int t0 = blockIdx.x * tokens, count = min(tokens, bt.total - t0);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, l = lane % L;
  const int heads = a.Hq + 2 * c.H, vectors = count * heads;
  pdl_begin();
  struct Item {
    uint4 x, y;          // the lane's elements, and in the half layout their partners
    int tok, head;
  };
  const bool turned = l * 8 < 2 * a.half;
  const int away = INTER ? 0 : (l * 8 < a.half ? a.half : -a.half);
  auto load = [&](int v, Item& it) {
    it.x = it.y = make_uint4(0, 0, 0, 0);
    it.tok = v / heads;
    it.head = v - it.tok * heads;
    if (v >= vectors) return;
    const long long row = t0 + it.tok;
    const __nv_bfloat16* p = it.head < a.Hq ? a.q + row * a.q_ld + it.head * a.q_head_ld
                             : it.head < a.Hq + c.H ? a.k + row * a.k_ld + (it.head - a.Hq) * D
                                                    : a.v + row * a.v_ld + (it.head - a.Hq - c.H) * D;
    it.x = __ldg(reinterpret_cast<const uint4*>(p) + l);
    if (!INTER && turned && it.head < a.Hq + c.H) it.y = __ldg(reinterpret_cast<const uint4*>(p + away) + l);
  };
  const int first = warp * kSide + lane / L, step = 8 * kSide;
  Item it;
  load(first, it);
  if (warp == 0) {
    const Place p = find_place(c, bt, min(t0 + lane, bt.total - 1));
    if (lane < count) {
      place[lane] = p.page < 0 ? -1 : (((long long)p.page * c.H) << c.page_shift) + p.off;
      angle_at[lane] = a.positions ? __ldg(a.positions + t0 + lane) : p.pos;
    }
  }
  __syncthreads();
  for (int i = tid; i < count * a.half; i += 256) {
    const int t = i / a.half;
    const float2 r = rotary_turn(__ldg(a.turns + i - t * a.half), angle_at[t], a.scale);
    cs[i] = r.x;
    sn[i] = r.y;
  }
  __syncthreads();
  // (whole warps go round together: the shuffles take every lane)
  for (int v = first; v - lane / L < vectors; v += step) {
    Item next;
    load(v + step, next);
    const bool live = v < vectors;
    const long long base = live ? place[it.tok] : -1;
    const bool is_q = it.head < a.Hq, is_v = it.head >= a.Hq + c.H;
    float x[8];
    unpack8(it.x, x);
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
    ss = lanes_sum<L>(ss);                        // (every lane, whatever its vector)
    if (!is_v) {
      const __nv_bfloat16* w = is_q ? a.q_norm : a.k_norm;
      float y[8];
      if constexpr (!INTER) unpack8(it.y, y);
      if (w) {
        const float rs = rsqrtf(ss * (1.0f / D) + a.eps);
        float g[8];
        unpack8(__ldg(reinterpret_cast<const uint4*>(w) + l), g);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] *= rs * (a.w0 + g[j]);
        if (!INTER && turned) {
          unpack8(__ldg(reinterpret_cast<const uint4*>(w + away) + l), g);
#pragma unroll
          for (int j = 0; j < 8; ++j) y[j] *= rs * (a.w0 + g[j]);
        }
      }
      if (turned && live) {
        if constexpr (INTER) {
          const float4 co = *reinterpret_cast<const float4*>(cs + it.tok * a.half + l * 4);
          const float4 si = *reinterpret_cast<const float4*>(sn + it.tok * a.half + l * 4);
          const float cc[4] = {co.x, co.y, co.z, co.w}, sc[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float u = x[2 * j], z = x[2 * j + 1];
            x[2 * j] = turned_a(u, z, cc[j], sc[j]);
            x[2 * j + 1] = turned_b(u, z, cc[j], sc[j]);
          }
        } else {
          const int at = it.tok * a.half + (away > 0 ? l * 8 : l * 8 - a.half);
          const float sign = away > 0 ? -1.f : 1.f;
#pragma unroll
          for (int j0 = 0; j0 < 8; j0 += 4) {
            const float4 co = *reinterpret_cast<const float4*>(cs + at + j0);
            const float4 si = *reinterpret_cast<const float4*>(sn + at + j0);
            const float cc[4] = {co.x, co.y, co.z, co.w}, sc[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j0 + j] = fmaf(x[j0 + j], cc[j], sign * __fmul_rn(y[j0 + j], sc[j]));
          }
        }
      }
    }
    if (is_q) {
      if (live) {
        const uint4 o = base < 0 ? make_uint4(0, 0, 0, 0) : pack8(x);
        reinterpret_cast<uint4*>(a.q_out + ((long long)(t0 + it.tok) * a.Hq + it.head) * D)[l] = o;
      }
    }
    if constexpr (Q8) {
      float top = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) top = __uint_as_float(max(__float_as_uint(top), __float_as_uint(x[j]) & 0x7fffffffu));
      top = lanes_max<L>(top);
      if (!is_q && base >= 0) {
        const int h = it.head - a.Hq - (is_v ? c.H : 0), b = scale_byte_f32(top);
        const long long at = base + ((long long)h << c.page_shift);
        reinterpret_cast<uint2*>(static_cast<uint8_t*>(is_v ? c.v : c.k) + at * D)[l] = codes8(x, b);
        if (l == 0) (is_v ? c.vs : c.ks)[at] = (uint8_t)b;
      }
    } else if (!is_q && base >= 0) {
      const int h = it.head - a.Hq - (is_v ? c.H : 0);
      const long long at = base + ((long long)h << c.page_shift);
      reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(is_v ? c.v : c.k) + at * D)[l] = is_v ? it.x : pack8(x);
    }
    it = next;
  }
}

}  // namespace

int launch_kv_append_rotated(const KvView& c, const KvBatchView& bt, const RotatedAppend& a, cudaStream_t stream) {
  // tokens of a CTA: two rounds of its warps, more (up to eight times that) where that leaves the SMs
  // their fill of CTAs
  const long long lanes = (long long)(a.Hq + 2 * c.H) * (c.D / 8);
  const int most = kMostTurns / a.half < kMostTokens ? kMostTurns / a.half : kMostTokens;
  long long t = (512 + lanes - 1) / lanes;
  const long long top = t * 8;
  while (2 * t <= top && bt.total > 2048 * t) t *= 2;
  const int tokens = t < most ? (int)t : most;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((bt.total + tokens - 1) / tokens));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  cudaError_t e = cudaSuccess;
#define GDN_RUN(DD)                                                                                           \
  e = c.ks ? (a.interleaved ? cudaLaunchKernelEx(&cfg, append_rotated_kernel<DD, true, true>, c, bt, tokens, a)   \
                            : cudaLaunchKernelEx(&cfg, append_rotated_kernel<DD, true, false>, c, bt, tokens, a)) \
           : (a.interleaved ? cudaLaunchKernelEx(&cfg, append_rotated_kernel<DD, false, true>, c, bt, tokens, a)  \
                            : cudaLaunchKernelEx(&cfg, append_rotated_kernel<DD, false, false>, c, bt, tokens, a))
  if (c.D == 64) GDN_RUN(64);
  else if (c.D == 128) GDN_RUN(128);
  else GDN_RUN(256);
#undef GDN_RUN
  return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace gdn
