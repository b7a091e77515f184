// gdn_rotary.cu -- rotary positions of queries and keys.
//
// Three flops per element: the floor is the bytes, every element read and written once.  An angle
// belongs to a token and a pair, whatever the head: a CTA takes a few neighbouring tokens, computes
// their sines and cosines into shared memory, and then walks all heads of q and k with them.  An item of
// work is a vector of one head, or for the half layout the two vectors that hold its pairs, so nothing is
// read twice.  16384 tokens of 40 bf16 heads of 128: 53.0 us, 6.3 TB/s, 93 % of a copy.
#include "gdn_rotary.cuh"

namespace gdn {

namespace {

// Division by a constant of the launch: (x * mul) >> 32, corrected once; exact for x < 2^31 and any d.
struct FastDiv {
  uint32_t d, mul;
  explicit FastDiv(uint32_t n) : d(n), mul((uint32_t)((1ull << 32) / n > 0xffffffffull ? 0xffffffffu : (1ull << 32) / n)) {}
  // (mul is at most 2^32 / d and short of it by less than 1: the quotient is at most one too small)
  __device__ __forceinline__ uint32_t div(uint32_t x) const {
    const uint32_t q = __umulhi(x, mul);
    return x - q * d >= d ? q + 1 : q;
  }
};

struct RotaryArgs {
  const void* q;
  const void* k;
  void* q_out;
  void* k_out;
  long long q_ld, q_head_ld, k_ld, k_head_ld;
  const uint64_t* turns;
  const int32_t* pos;
  float scale;
  int tokens, per_cta, dim, half, q_heads, heads;   // half: pairs of a head; heads: q's and k's
  FastDiv items, all_heads, pairs;                  // items of a head, heads, pairs
  int step_item, step_head, step_token;             // 256 items on
  int rest;                                         // items past the rotated part
};

constexpr int kTurns = 2048;      // (cos, sin) of a CTA: tokens * pairs of a head

template <typename T, int V>
struct Vec {
  float v[V];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (V == 1) {
      v[0] = Act<T>::load(p);
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < V; i += 2) {
        if constexpr (V == 2) {
          const float2 f = *reinterpret_cast<const float2*>(p);
          v[0] = f.x; v[1] = f.y;
        } else if (i % 4 == 0) {
          const float4 f = *reinterpret_cast<const float4*>(p + i);
          v[i] = f.x; v[i + 1] = f.y; v[i + 2] = f.z; v[i + 3] = f.w;
        }
      }
    } else {
      uint32_t w[V / 2];
      if constexpr (V == 8) {
        const uint4 u = *reinterpret_cast<const uint4*>(p);
        w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
      } else if constexpr (V == 2) {
        w[0] = *reinterpret_cast<const uint32_t*>(p);
      } else {
        const uint2 u = *reinterpret_cast<const uint2*>(p);
        w[0] = u.x; w[1] = u.y;
      }
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (V == 1) {
      Act<T>::store(p, v[0]);
    } else if constexpr (sizeof(T) == 4) {
      if constexpr (V == 2) *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
      else *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
      uint32_t w[V / 2];
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
      }
      if constexpr (V == 8) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
      else if constexpr (V == 2) *reinterpret_cast<uint32_t*>(p) = w[0];
      else *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    }
  }
};

// V elements a vector.  Half layout: items 0 .. half / V - 1 of a head are its pairs' vectors, the others two vectors
// each past the rotated part (the last perhaps one).  Interleaved (V > 1): an item is two vectors, holding whole pairs;
// V = 1: items 0 .. half - 1 are the pairs, the others two elements each.  WHOLE: nothing past the rotated part.
template <typename T, int V, bool INTER, bool WHOLE>
__global__ void __launch_bounds__(256) rotary_kernel(const RotaryArgs a) {
  __shared__ __align__(16) float2 turn[kTurns];
  const int t0 = blockIdx.x * a.per_cta, count = min(a.per_cta, a.tokens - t0), tid = threadIdx.x;
  pdl_begin();
  for (int i = tid; i < count * a.half; i += 256) {
    const int t = a.pairs.div(i), p = i - t * a.half;
    turn[i] = rotary_turn(__ldg(a.turns + p), __ldg(a.pos + t0 + t), a.scale);
  }
  __syncthreads();
  const int paired = INTER && V > 1 ? 0 : a.half / V;
  const int th = a.items.div(tid);
  int e = tid - th * (int)a.items.d, t = a.all_heads.div(th), head = th - t * a.heads;
  auto next = [&]() {
    e += a.step_item;
    head += a.step_head;
    t += a.step_token;
    if (e >= (int)a.items.d) {
      e -= a.items.d;
      ++head;
    }
    if (head >= a.heads) {
      head -= a.heads;
      ++t;
    }
  };
  // (unrolled by two 54.5 us for the 53 above)
#pragma unroll 1
  for (; t < count; next()) {
    const bool is_q = head < a.q_heads;
    const int h = is_q ? head : head - a.q_heads;
    const long long row = t0 + t;
    const T* src = is_q ? static_cast<const T*>(a.q) + row * a.q_ld + h * a.q_head_ld
                        : static_cast<const T*>(a.k) + row * a.k_ld + h * a.k_head_ld;
    T* dst = is_q ? static_cast<T*>(a.q_out) + (row * a.q_heads + h) * a.dim
                  : static_cast<T*>(a.k_out) + (row * (a.heads - a.q_heads) + h) * a.dim;
    const float2* cs = turn + t * a.half;
    if constexpr (INTER && V > 1) {
      const int at[2] = {e * V, (e + (int)a.items.d) * V};
      const bool two = at[1] < a.dim;
      Vec<T, V> x[2];
      x[0].load(src + at[0]);
      if (two) x[1].load(src + at[1]);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int p = at[i] / 2;
        if (p < a.half) {
#pragma unroll
          for (int j = 0; j < V / 2; ++j) {
            const float2 c = cs[p + j];
            const float u = x[i].v[2 * j], w = x[i].v[2 * j + 1];
            x[i].v[2 * j] = turned_a(u, w, c.x, c.y);
            x[i].v[2 * j + 1] = turned_b(u, w, c.x, c.y);
          }
        }
      }
      x[0].store(dst + at[0]);
      if (two) x[1].store(dst + at[1]);
    } else {
      // (all lanes' loads alike, whether their vectors are turned or not: a warp's lanes hold both kinds, and a quarter
      // of heads of 256 turned takes 83 us of 537 MB, in branches of their own 133)
      const bool turned = WHOLE || e < paired;
      const int lo = !turned ? 2 * a.half + (e - paired) * V : INTER ? 2 * e : e * V;
      const int hi = lo + (!turned ? a.rest * V : INTER ? 1 : a.half);
      const bool two = turned || hi < a.dim;
      Vec<T, V> x, y;
      x.load(src + lo);
      if (two) y.load(src + hi);
      if (turned) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float2 c = cs[e * V + j];
          const float u = x.v[j], w = y.v[j];
          x.v[j] = turned_a(u, w, c.x, c.y);
          y.v[j] = turned_b(u, w, c.x, c.y);
        }
      }
      x.store(dst + lo);
      if (two) y.store(dst + hi);
    }
  }
}

template <typename T, int V>
int launch_as(const RotaryArgs& a, bool inter, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.tokens - 1) / a.per_cta + 1));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = inter            ? cudaLaunchKernelEx(&cfg, rotary_kernel<T, V, true, false>, a)
                        : a.rest == 0 ? cudaLaunchKernelEx(&cfg, rotary_kernel<T, V, false, true>, a)
                                      : cudaLaunchKernelEx(&cfg, rotary_kernel<T, V, false, false>, a);
  return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

template <typename T>
int launch_typed(const RotaryLaunch& r, cudaStream_t stream) {
  const int half = r.rot / 2;
  // whole vectors of V elements everywhere: bases, rows, heads, and the pairs' halves (or the rotated part)
  auto fits = [&](int v) {
    const uintptr_t bases = reinterpret_cast<uintptr_t>(r.q) | reinterpret_cast<uintptr_t>(r.k) |
                            reinterpret_cast<uintptr_t>(r.q_out) | reinterpret_cast<uintptr_t>(r.k_out);
    const long long n = r.dim | r.q_ld | r.q_head_ld | r.k_ld | r.k_head_ld | (r.interleaved ? r.rot : half);
    return bases % (v * sizeof(T)) == 0 && n % v == 0;
  };
  constexpr int kWide = 16 / sizeof(T), kMid = 8 / sizeof(T);
  const int v = fits(kWide) ? kWide : fits(kMid) ? kMid : fits(2) ? 2 : 1;
  const int heads = r.q_heads + r.k_heads;
  const int rest = ((r.dim - r.rot) / v + 1) / 2, items = r.interleaved && v > 1 ? (r.dim / v + 1) / 2 : half / v + rest;
  // (16 bytes, 8, 4 of bf16, or an element: of 537 MB of bf16, vectors of 16 bytes take 82 to 93 us, of 8 98, of 4 128,
  // elements 240)
  // tokens of a CTA: some four items a thread, as far as their sines fit
  const long long per_token = (long long)heads * items;
  long long per = (1024 + per_token - 1) / per_token;
  if (per > kTurns / half) per = kTurns / half;
  const RotaryArgs a{r.q, r.k, r.q_out, r.k_out, r.q_ld, r.q_head_ld, r.k_ld, r.k_head_ld, r.turns, r.positions,
                     r.scale, r.tokens, (int)per, r.dim, half, r.q_heads, heads, FastDiv((uint32_t)items),
                     FastDiv((uint32_t)heads), FastDiv((uint32_t)half), 256 % items, 256 / items % heads, 256 / items / heads, rest};
  if (v == kWide) return launch_as<T, kWide>(a, r.interleaved, stream);
  if (v == kMid) return launch_as<T, kMid>(a, r.interleaved, stream);
  if (v == 2) return launch_as<T, 2>(a, r.interleaved, stream);
  return launch_as<T, 1>(a, r.interleaved, stream);
}

}  // namespace

int launch_rotary(const RotaryLaunch& r, gdn_dtype act, cudaStream_t stream) {
  return act == GDN_BF16 ? launch_typed<__nv_bfloat16>(r, stream) : launch_typed<float>(r, stream);
}

}  // namespace gdn
