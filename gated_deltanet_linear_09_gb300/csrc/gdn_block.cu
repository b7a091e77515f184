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

// VEC (8 or 1) consecutive elements at p.
template <typename T, int VEC>
__device__ __forceinline__ void load_vec(const T* p, float* v) {
  if constexpr (VEC == 1) {
    v[0] = Act<T>::load(p);
  } else if constexpr (sizeof(T) == 4) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}

template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T* p, const float* v) {
  if constexpr (VEC == 1) {
    Act<T>::store(p, v[0]);
  } else if constexpr (sizeof(T) == 4) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// A row's sum over TPR threads; `part` is this sum's own.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* part) {
  v = warp_sum(v);
  if constexpr (TPR > 32) {
    constexpr int WARPS = TPR / 32;
    const int lane = threadIdx.x & 31;
    if (lane == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = warp_sum(lane < WARPS ? part[lane] : 0.f);
  }
  return v;
}

// TPR threads hold one row, NV vectors of VEC elements each (vector j of thread t is vector j * TPR + t of
// the row); TPR = 32 puts several rows into a CTA.  GROUPED: the first norm is over runs of 32 to 256
// columns, 4 to 32 neighbouring lanes.
template <typename T, int VEC, int TPR, int NV, bool GROUPED>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR) block_kernel(const BlockArgs a) {
  constexpr int CTA = TPR < 128 ? 128 : TPR;
  __shared__ float part[2][CTA / 32];
  const gdn_block_args& p = a.p;
  const int tid = threadIdx.x, t = TPR < 128 ? tid % TPR : tid, n = a.n;
  const long long row = (long long)blockIdx.x * (CTA / TPR) + (TPR < 128 ? tid / TPR : 0);
  pdl_begin();
  if (TPR < 128 && row >= a.rows) return;   // whole warps leave; no barrier follows for TPR = 32
  const T* x = static_cast<const T*>(p.x) + row * p.x_ld;
  float h[NV][VEC];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * TPR + t) * VEC;
#pragma unroll
    for (int e = 0; e < VEC; ++e) h[j][e] = 0.f;
    if (c < n) load_vec<T, VEC>(x + c, h[j]);
  }
  float z[NV][VEC], r[NV][VEC];
  if (p.gate) {
    const T* src = static_cast<const T*>(p.gate) + row * p.gate_ld;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * TPR + t) * VEC;
      if (c < n) load_vec<T, VEC>(src + c, z[j]);
    }
  }
  if (p.residual) {
    const T* src = static_cast<const T*>(p.residual) + row * p.residual_ld;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * TPR + t) * VEC;
      if (c < n) load_vec<T, VEC>(src + c, r[j]);
    }
  }
  if (p.post) {
    const T* w = static_cast<const T*>(p.post);
    float rs = 0.f;
    if constexpr (!GROUPED) {
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e) ss = fmaf(h[j][e], h[j][e], ss);
      rs = rsqrtf(row_sum<TPR>(ss, part[0]) * a.inv_n + p.eps);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * TPR + t) * VEC;
      if constexpr (GROUPED) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < VEC; ++e) ss = fmaf(h[j][e], h[j][e], ss);
        for (int o = p.group / (2 * VEC); o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        rs = rsqrtf(ss * a.inv_g + p.eps);
      }
      float g[VEC];
      if (c < n) {
        load_vec<T, VEC>(w + (GROUPED ? c & (p.group - 1) : c), g);
#pragma unroll
        for (int e = 0; e < VEC; ++e) h[j][e] *= rs * (p.weight_offset + g[e]);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * TPR + t) * VEC;
    if (c >= n) continue;
    if (p.gate) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        // (fast division and exponential, off by 2^-21, where the result is rounded to bf16)
        const float s = sizeof(T) == 4 ? sigmoidf_(z[j][e]) : __fdividef(1.0f, 1.0f + __expf(-z[j][e]));
        h[j][e] *= p.gate_act == GDN_GATE_SILU ? z[j][e] * s : s;
      }
    }
    if (p.channel_scale) {
      float g[VEC];
      load_vec<T, VEC>(static_cast<const T*>(p.channel_scale) + c, g);
#pragma unroll
      for (int e = 0; e < VEC; ++e) h[j][e] *= g[e];
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) h[j][e] = p.residual ? fmaf(p.scale, h[j][e], r[j][e]) : p.scale * h[j][e];
    if (p.total) store_vec<T, VEC>(static_cast<T*>(p.total) + row * n + c, h[j]);
  }
  if (!p.pre) return;
  float ss = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < VEC; ++e) ss = fmaf(h[j][e], h[j][e], ss);     // (zeros past the row's end)
  const float rs = rsqrtf(row_sum<TPR>(ss, part[1]) * a.inv_n + p.eps);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * TPR + t) * VEC;
    if (c >= n) continue;
    float g[VEC];
    load_vec<T, VEC>(static_cast<const T*>(p.pre) + c, g);
#pragma unroll
    for (int e = 0; e < VEC; ++e) g[e] = h[j][e] * rs * (p.weight_offset + g[e]);
    store_vec<T, VEC>(static_cast<T*>(p.y) + row * n + c, g);
  }
}

template <typename T, int VEC, int TPR, int NV>
int launch_one(const BlockArgs& a, cudaStream_t stream) {
  const int per = TPR < 128 ? 128 / TPR : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.rows + per - 1) / per));
  cfg.blockDim = dim3(TPR < 128 ? 128 : TPR);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  cudaError_t e = cudaSuccess;
  if constexpr (VEC == 8) {
    if (a.p.post && a.p.group < a.n) {
      e = cudaLaunchKernelEx(&cfg, block_kernel<T, VEC, TPR, NV, true>, a);
      return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
    }
  }
  e = cudaLaunchKernelEx(&cfg, block_kernel<T, VEC, TPR, NV, false>, a);
  return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

// A warp to a row up to 512 elements, then 128 to 1,024 threads with two to four vectors each.
template <typename T>
int launch_wide(const BlockArgs& a, cudaStream_t s) {
  const int nv = a.n / 8;
  if (nv <= 32) return launch_one<T, 8, 32, 1>(a, s);
  if (nv <= 64) return launch_one<T, 8, 32, 2>(a, s);
  if (nv <= 256) return launch_one<T, 8, 128, 2>(a, s);
  if (nv <= 512) return launch_one<T, 8, 256, 2>(a, s);
  if (nv <= 768) return launch_one<T, 8, 256, 3>(a, s);
  if (nv <= 1024) return launch_one<T, 8, 512, 2>(a, s);
  if (nv <= 2048) return launch_one<T, 8, 1024, 2>(a, s);
  return launch_one<T, 8, 1024, 4>(a, s);
}

// Rows off the 16-byte grid, an element per access.
template <typename T>
int launch_narrow(const BlockArgs& a, cudaStream_t s) {
  if (a.n <= 128) return launch_one<T, 1, 32, 4>(a, s);
  if (a.n <= 1024) return launch_one<T, 1, 128, 8>(a, s);
  if (a.n <= 4096) return launch_one<T, 1, 512, 8>(a, s);
  if (a.n <= 8192) return launch_one<T, 1, 1024, 8>(a, s);
  return launch_one<T, 1, 1024, 32>(a, s);
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
