// gdn_block.cu -- a block's output on its way to the next block: its norm, gate and scale, the residual's
// addition, and the next block's norm.
//
//   b = x / rms_g(x) (w0 + post),  h = r + s c b act(z),  y = h / rms(h) (w0 + pre)
//
// A dozen flops per element: the floor is the bytes, x, z and r read once, h and y written once.  A row stays
// in registers from the first load to the last store, between the two sums that it waits for.
#include "gdn_internal.h"

namespace gdn {

namespace {

struct BlockArgs {
  gdn_block_args p;
  float inv_n, inv_g;
  int rows, n;
};

// VEC (8 or 1) consecutive elements as they are in memory: what is loaded ahead is held so.
template <typename T, int VEC>
struct Raw {
  T v;
  __device__ __forceinline__ void load(const T* p) { v = *p; }
  __device__ __forceinline__ void get(float* x) const { x[0] = Act<T>::load(&v); }
  static __device__ __forceinline__ void put(T* p, const float* x) { Act<T>::store(p, x[0]); }
};
template <>
struct Raw<float, 8> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void get(float* x) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
  static __device__ __forceinline__ void put(float* p, const float* x) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
};
template <>
struct Raw<__nv_bfloat16, 8> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float* x) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void put(__nv_bfloat16* p, const float* x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// Element-wise steps on VEC elements, two at a time where there are two.
template <int VEC>
__device__ __forceinline__ void mul_by(float* x, const float* a) {
  if constexpr (VEC == 1) x[0] *= a[0];
  else
#pragma unroll
    for (int e = 0; e < VEC; e += 2) mul_pair(x[e], x[e + 1], a[e], a[e + 1]);
}
template <int VEC>
__device__ __forceinline__ void mul_by(float* x, float a) {
  if constexpr (VEC == 1) x[0] *= a;
  else
#pragma unroll
    for (int e = 0; e < VEC; e += 2) mul_pair(x[e], x[e + 1], a, a);
}
// x * a + b
template <int VEC>
__device__ __forceinline__ void fma_by(float* x, float a, const float* b) {
  if constexpr (VEC == 1) x[0] = fmaf(x[0], a, b[0]);
  else
#pragma unroll
    for (int e = 0; e < VEC; e += 2) fma_pair(x[e], x[e + 1], a, a, b[e], b[e + 1]);
}
// x * (rs * (offset + w))
template <int VEC>
__device__ __forceinline__ void weigh(float* x, float* w, float rs, float offset) {
  if constexpr (VEC == 1) {
    x[0] *= rs * (offset + w[0]);
  } else {
    const float base = rs * offset;      // (fused: rs w + rs offset, rounded once)
#pragma unroll
    for (int e = 0; e < VEC; e += 2) {
      fma_pair(w[e], w[e + 1], rs, rs, base, base);
      mul_pair(x[e], x[e + 1], w[e], w[e + 1]);
    }
  }
}
template <int VEC>
__device__ __forceinline__ void add_squares(const float* x, float& a, float& b) {
  if constexpr (VEC == 1) a = fmaf(x[0], x[0], a);
  else
#pragma unroll
    for (int e = 0; e < VEC; e += 2) {
      float u = x[e], v = x[e + 1];
      fma_pair(u, v, x[e], x[e + 1], a, b);
      a = u;
      b = v;
    }
}
// sigmoid for a result that is rounded to bf16: both approximations are off by about 2^-22.
__device__ __forceinline__ float sigmoid_fast(float z) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return r;
}

// A row's sum over its threads (SHARED: the CTA's, else a warp's); `part` is this sum's own.
template <bool SHARED>
__device__ __forceinline__ float row_sum(float v, float* part) {
  v = warp_sum(v);
  if constexpr (SHARED) {
    const int lane = threadIdx.x & 31;
    if (lane == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = warp_sum(lane < (int)blockDim.x / 32 ? part[lane] : 0.f);
  }
  return v;
}

// A row is held by a CTA (SHARED; as many threads as it takes) or a warp, NV vectors of VEC elements a thread:
// vector j of thread t is vector j * threads + t of the row.  Everything that does not depend on a sum is
// loaded before it: what bounds this is the bytes in flight, and a row waits for two sums.  GROUPED: the
// first norm is over runs of 32 to 256 columns, 4 to 32 neighbouring lanes.
template <typename T, int VEC, int NV, bool SHARED, bool GROUPED, int MOST>
__global__ void __launch_bounds__(MOST) block_kernel(const BlockArgs a) {
  using R = Raw<T, VEC>;
  __shared__ float part[2][32];
  const gdn_block_args& p = a.p;
  const int threads = SHARED ? (int)blockDim.x : 32, t = SHARED ? threadIdx.x : threadIdx.x & 31, n = a.n;
  const long long row = SHARED ? blockIdx.x : (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  pdl_begin();
  if (!SHARED && row >= a.rows) return;     // whole warps leave; no barrier follows
  R x[NV], z[NV], r[NV], w[NV];
  auto load = [&](R* to, const void* from, long long at) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * threads + t) * VEC;
      if (c < n) to[j].load(static_cast<const T*>(from) + at + c);
    }
  };
  load(x, p.x, row * p.x_ld);
  if (p.gate) load(z, p.gate, row * p.gate_ld);
  if (p.residual) load(r, p.residual, row * p.residual_ld);
  if (p.post) {
    if constexpr (GROUPED) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (j * threads + t) * VEC;
        if (c < n) w[j].load(static_cast<const T*>(p.post) + (c & (p.group - 1)));
      }
    } else {
      load(w, p.post, 0);
    }
  }
  float h[NV][VEC];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if ((j * threads + t) * VEC < n) {
      x[j].get(h[j]);
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) h[j][e] = 0.f;
    }
  }
  if (p.post) {
    float rs = 0.f;
    if constexpr (!GROUPED) {
      float ss = 0.f, s2 = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j) add_squares<VEC>(h[j], ss, s2);
      rs = rsqrtf(row_sum<SHARED>(ss + s2, part[0]) * a.inv_n + p.eps);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if constexpr (GROUPED) {
        float ss = 0.f, s2 = 0.f;
        add_squares<VEC>(h[j], ss, s2);
        ss += s2;
        for (int o = p.group / (2 * VEC); o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        rs = rsqrtf(ss * a.inv_g + p.eps);
      }
      if ((j * threads + t) * VEC < n) {
        float g[VEC];
        w[j].get(g);
        weigh<VEC>(h[j], g, rs, p.weight_offset);
      }
    }
  }
  if (p.channel_scale) load(x, p.channel_scale, 0);
  if (p.pre) load(w, p.pre, 0);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * threads + t) * VEC;
    if (c >= n) continue;
    float g[VEC];
    if (p.gate) {
      z[j].get(g);
      float s[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) s[e] = sizeof(T) == 4 ? sigmoidf_(g[e]) : sigmoid_fast(g[e]);
      if (p.gate_act == GDN_GATE_SILU) mul_by<VEC>(s, g);
      mul_by<VEC>(h[j], s);
    }
    if (p.channel_scale) {
      x[j].get(g);
      mul_by<VEC>(h[j], g);
    }
    if (p.residual) {
      r[j].get(g);
      fma_by<VEC>(h[j], p.scale, g);
    } else {
      mul_by<VEC>(h[j], p.scale);
    }
    if (p.total) R::put(static_cast<T*>(p.total) + row * n + c, h[j]);
  }
  if (!p.pre) return;
  float ss = 0.f, s2 = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j) add_squares<VEC>(h[j], ss, s2);         // (zeros past the row's end)
  const float rs = rsqrtf(row_sum<SHARED>(ss + s2, part[1]) * a.inv_n + p.eps);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * threads + t) * VEC;
    if (c >= n) continue;
    float g[VEC];
    w[j].get(g);
    weigh<VEC>(h[j], g, rs, p.weight_offset);
    R::put(static_cast<T*>(p.y) + row * n + c, h[j]);
  }
}

template <typename T, int VEC, int NV, bool SHARED, int MOST>
int launch_one(const BlockArgs& a, cudaStream_t stream) {
  const int vectors = (a.n + VEC - 1) / VEC;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(SHARED ? a.rows : (a.rows + 3) / 4));
  cfg.blockDim = dim3(SHARED ? (unsigned)((vectors + NV * 32 - 1) / (NV * 32) * 32) : 128);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  cudaError_t e = cudaSuccess;
  if constexpr (VEC == 8) {
    if (a.p.post && a.p.group < a.n) {
      e = cudaLaunchKernelEx(&cfg, block_kernel<T, VEC, NV, SHARED, true, MOST>, a);
      return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
    }
  }
  e = cudaLaunchKernelEx(&cfg, block_kernel<T, VEC, NV, SHARED, false, MOST>, a);
  return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

// A warp to a row up to 32 vectors (256 elements), then a CTA with four vectors of bf16 a thread, or two of f32
// (its registers hold twice as much), more where a row would not fit 512 threads.
template <typename T>
int launch_wide(const BlockArgs& a, cudaStream_t s) {
  constexpr int NV = sizeof(T) == 4 ? 2 : 4;
  const int nv = a.n / 8;
  if (nv <= 32) return launch_one<T, 8, 1, false, 128>(a, s);
  if (nv <= NV * 256) return launch_one<T, 8, NV, true, 256>(a, s);
  if (nv <= NV * 512) return launch_one<T, 8, NV, true, 512>(a, s);
  return launch_one<T, 8, 4, true, 1024>(a, s);
}

// Rows off the 16-byte grid, an element per access.
template <typename T>
int launch_narrow(const BlockArgs& a, cudaStream_t s) {
  if (a.n <= 128) return launch_one<T, 1, 4, false, 128>(a, s);
  if (a.n <= 8192) return launch_one<T, 1, 8, true, 1024>(a, s);
  return launch_one<T, 1, 32, true, 1024>(a, s);
}

template <typename T>
int launch_typed(const BlockArgs& a, cudaStream_t s) {
  const long long bits = a.n | a.p.x_ld | (a.p.gate ? a.p.gate_ld : 0) | (a.p.residual ? a.p.residual_ld : 0);
  return bits % 8 == 0 ? launch_wide<T>(a, s) : launch_narrow<T>(a, s);
}

}  // namespace

int launch_block_norm(const gdn_block_args& p, int rows, int n, gdn_dtype act, cudaStream_t stream) {
  const BlockArgs a{p, 1.0f / (float)n, 1.0f / (float)p.group, rows, n};
  return act == GDN_BF16 ? launch_typed<__nv_bfloat16>(a, stream) : launch_typed<float>(a, stream);
}

}  // namespace gdn
