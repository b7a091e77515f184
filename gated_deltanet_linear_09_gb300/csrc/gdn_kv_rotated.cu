// gdn_kv_rotated.cu -- the cache's append with the heads' RMSNorm and rotary positions on the way.
//
// Between an attention layer's projection and its cache every query and key vector is normed and turned:
// a chain of element-wise steps, so one pass does them all, and q, k and v are read once.  The floor is
// the bytes.  A CTA takes neighbouring tokens; a vector is a few neighbouring lanes, so the norm's sum is a
// few shuffles.  A lane holds both elements of its pairs in either layout, so nothing is exchanged.  Angles
// belong to tokens: they are computed once into shared memory, while the vectors' first loads are under way.
// 33,965 tokens of 16 query and twice 2 heads of 256, a quarter of them turned: 122 us, 5.7 TB/s, 84 % of a copy: the
// start of a CTA (16 tokens of it; with 8 142 us, with 32 122).
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

enum Part { kQueries, kKeys, kValues };

// A vector is L = D / 16 neighbouring lanes, each with two pieces of 8 elements: what a vector costs beside its
// elements (its place, its sum) is spread over many.  In the half layout lane l's are pieces l and l + half / 8,
// each other's partners, for the rotated part, and for the rest l + half / 8 and l + L; else l and l + L.
template <int D, bool Q8, bool INTER>
struct Kernel {
  static constexpr int L = D / 16, kSide = 32 / L;      // lanes of a vector, vectors of a warp at a time
  static constexpr int kStep = 8 * kSide;               // vectors of the CTA's warps at a time
  static constexpr int kBatch = 2;                      // of these in flight, and as many ahead

  // The rotation of one piece of pairs, or of two whose elements are each other's partners (half layout).
  static __device__ __forceinline__ void turn(float* x, float* y, const float* cp, const float* sp) {
#pragma unroll
    for (int j0 = 0; j0 < (INTER ? 4 : 8); j0 += 4) {
      const float4 co = *reinterpret_cast<const float4*>(cp + j0), si = *reinterpret_cast<const float4*>(sp + j0);
      const float cc[4] = {co.x, co.y, co.z, co.w}, sc[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float& p = INTER ? x[2 * j] : x[j0 + j];
        float& q = INTER ? x[2 * j + 1] : y[j0 + j];
        const float u = p, z = q;
        p = turned_a(u, z, cc[j], sc[j]);
        q = turned_b(u, z, cc[j], sc[j]);
      }
    }
  }

  // All vectors of one part of the CTA's tokens.  ready(): called by all threads between the first loads and
  // the first use of places and angles.
  template <int PART, typename F>
  static __device__ __forceinline__ void run(const KvView& c, const RotatedAppend& a, int t0, int count,
                                             const long long* place, const float* cs, const float* sn, F ready) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % L;
    const int heads = PART == kQueries ? a.Hq : c.H, n = count * heads;
    if (n == 0) {
      ready();
      return;
    }
    const __nv_bfloat16* src = PART == kQueries ? a.q : PART == kKeys ? a.k : a.v;
    const long long ld = PART == kQueries ? a.q_ld : PART == kKeys ? a.k_ld : a.v_ld;
    const long long head_ld = PART == kQueries ? a.q_head_ld : D;
    src += (long long)t0 * ld;
    const __nv_bfloat16* weight = PART == kQueries ? a.q_norm : PART == kKeys ? a.k_norm : nullptr;
    // the pieces' places in the vector, whether they are turned and which angles are theirs
    int at[2], angle[2];
    bool turned[2];
    float g[2][8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (INTER) {
        at[h] = (l + h * L) * 8;
        turned[h] = at[h] < 2 * a.half;
        angle[h] = at[h] / 2;
      } else {
        turned[h] = l * 8 < a.half;
        at[h] = turned[h] ? l * 8 + h * a.half : h == 0 ? l * 8 + a.half : (L + l) * 8;
        angle[h] = l * 8;
      }
      turned[h] = turned[h] && PART != kValues;
      if (PART != kValues && weight) {
        unpack8(__ldg(reinterpret_cast<const uint4*>(weight + at[h])), g[h]);
#pragma unroll
        for (int j = 0; j < 8; ++j) g[h][j] += a.w0;
      }
    }
    const int first = warp * kSide + lane / L, skip_tok = kStep / heads, skip_head = kStep % heads;
    int tok = first / heads, head = first % heads;
    // a step along the vectors, and back from the last head to the next token's first
    src += tok * ld + head * head_ld;
    const long long skip = skip_tok * ld + skip_head * head_ld, wrap = ld - heads * head_ld;
    struct Batch {
      uint4 raw[kBatch][2];
      int tok[kBatch], head[kBatch];
    };
    auto load = [&](Batch& b) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        b.tok[i] = tok;
        b.head[i] = head;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          b.raw[i][h] = tok < count ? __ldg(reinterpret_cast<const uint4*>(src + at[h])) : make_uint4(0, 0, 0, 0);
        src += skip;
        tok += skip_tok;
        head += skip_head;
        if (head >= heads) {
          head -= heads;
          ++tok;
          src += wrap;
        }
      }
    };
    Batch now, next;
    load(now);
    ready();
    // (whole warps go round together: the shuffles take every lane)
#pragma unroll 1
    for (int v = warp * kSide; v < n; v += kStep * kBatch) {
      load(next);                       // (nothing past the last token)
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const bool live = now.tok[i] < count;
        const long long base = live ? place[now.tok[i]] : -1;
        float x[2][8];
        if (PART != kValues || Q8) {
          unpack8(now.raw[i][0], x[0]);
          unpack8(now.raw[i][1], x[1]);
        }
        if constexpr (PART != kValues) {
          float rs = 1.f;
          if (weight) {
            float s0 = 0.f, s1 = 0.f;
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
              float u = x[j >> 3][j & 7], z = x[j >> 3][(j & 7) + 1];
              fma_pair(u, z, u, z, s0, s1);
              s0 = u;
              s1 = z;
            }
            rs = rsqrtf(lanes_sum<L>(s0 + s1) * (1.0f / D) + a.eps);
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
              float* u = &x[j >> 3][j & 7];
              mul_pair(u[0], u[1], g[j >> 3][j & 7], g[j >> 3][(j & 7) + 1]);
              mul_pair(u[0], u[1], rs, rs);
            }
          }
          const float* cp = cs + (live ? now.tok[i] * a.half : 0);
          const float* sp = sn + (live ? now.tok[i] * a.half : 0);
          if (INTER) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
              if (turned[h]) turn(x[h], nullptr, cp + angle[h], sp + angle[h]);
          } else if (turned[0]) {
            turn(x[0], x[1], cp + angle[0], sp + angle[0]);
          }
        }
        if constexpr (PART == kQueries) {
          if (live) {
            uint4* out = reinterpret_cast<uint4*>(a.q_out) + ((long long)t0 * a.Hq + v + i * kStep + lane / L) * (2 * L);
#pragma unroll
            for (int h = 0; h < 2; ++h) out[at[h] / 8] = base < 0 ? make_uint4(0, 0, 0, 0) : pack8(x[h]);
          }
        } else {
          const long long slot = base + ((long long)now.head[i] << c.page_shift);
          if constexpr (Q8) {
            uint32_t top = 0;
#pragma unroll
            for (int j = 0; j < 16; ++j) top = max(top, __float_as_uint(x[j >> 3][j & 7]) & 0x7fffffffu);
            const int b = scale_byte_f32(lanes_max<L>(__uint_as_float(top)));
            if (base >= 0) {
              uint2* out = reinterpret_cast<uint2*>(static_cast<uint8_t*>(PART == kValues ? c.v : c.k) + slot * D);
#pragma unroll
              for (int h = 0; h < 2; ++h) out[at[h] / 8] = codes8(x[h], b);
              if (l == 0) (PART == kValues ? c.vs : c.ks)[slot] = (uint8_t)b;
            }
          } else if (base >= 0) {
            uint4* out = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(PART == kValues ? c.v : c.k) + slot * D);
#pragma unroll
            for (int h = 0; h < 2; ++h) out[at[h] / 8] = PART == kValues ? now.raw[i][h] : pack8(x[h]);
          }
        }
      }
      now = next;
    }
  }
};

template <int D, bool Q8, bool INTER>
__global__ void __launch_bounds__(256, 2) append_rotated_kernel(const KvView c, const KvBatchView bt, int tokens,
                                                             const RotatedAppend a) {
  __shared__ long long place[kMostTokens];
  __shared__ int angle_at[kMostTokens];
  __shared__ __align__(16) float cs[kMostTurns], sn[kMostTurns];
  const int t0 = blockIdx.x * tokens, count = min(tokens, bt.total - t0);
  const int tid = threadIdx.x;
  pdl_begin();
  if (tid < 32) {
    const Place p = find_place(c, bt, min(t0 + tid, bt.total - 1));
    if (tid < count) {
      place[tid] = p.page < 0 ? -1 : (((long long)p.page * c.H) << c.page_shift) + p.off;
      angle_at[tid] = a.positions ? __ldg(a.positions + t0 + tid) : p.pos;
    }
  }
  using K = Kernel<D, Q8, INTER>;
  K::template run<kValues>(c, a, t0, count, place, cs, sn, [&]() {
    __syncthreads();
    for (int i = tid; i < count * a.half; i += 256) {
      const int t = i / a.half;
      const float2 r = rotary_turn(__ldg(a.turns + i - t * a.half), angle_at[t], a.scale);
      cs[i] = r.x;
      sn[i] = r.y;
    }
  });
  K::template run<kKeys>(c, a, t0, count, place, cs, sn, []() { __syncthreads(); });
  K::template run<kQueries>(c, a, t0, count, place, cs, sn, []() {});
}

}  // namespace

int launch_kv_append_rotated(const KvView& c, const KvBatchView& bt, const RotatedAppend& a, cudaStream_t stream) {
  // tokens of a CTA: a round of its warps, more where that leaves the SMs some waves of CTAs
  const long long lanes = (long long)(a.Hq + 2 * c.H) * (c.D / 16);
  const int most = kMostTurns / a.half < kMostTokens ? kMostTurns / a.half : kMostTokens;
  long long t = (256 + lanes - 1) / lanes;
  while (t < 16 && bt.total > 2048 * t) t *= 2;
  const int tokens = t < most ? (int)t : most;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((bt.total - 1) / tokens + 1));
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
