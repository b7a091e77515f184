// gdn_norm.cu -- RMSNorm with the residual's addition; activation-dtype or scaled 8-bit output.
//
// h = x + r, y = h / sqrt(mean h^2 + eps) * (w0 + w).  Two or three flops per element, so the
// floor is the bytes: x and r read once, the sum and y written once.  A row therefore stays in
// registers between the pass that sums h^2 and the one that scales: nothing is read twice.
// Measured: 16384 x 4096 bf16 with residual to block-scaled 8 bits 71.0 us, 99 % of the copy bandwidth
// (6.65 of 6.69 TB/s); one row of 5120 2.0 us on the GPU, below what a call takes on the host.
#include "gdn_internal.h"

#include <cuda_fp8.h>

namespace gdn {

namespace {

// VEC consecutive elements at p: 16 bytes, two elements, or one.
template <typename T, int VEC>
__device__ __forceinline__ void load_vec(const T* p, float* v) {
  if constexpr (VEC == 1) {
    v[0] = Act<T>::load(p);
  } else if constexpr (VEC == 2 && sizeof(T) == 4) {
    const float2 f = *reinterpret_cast<const float2*>(p);
    v[0] = f.x; v[1] = f.y;
  } else if constexpr (VEC == 2) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(p);
    v[0] = __uint_as_float(w << 16);
    v[1] = __uint_as_float(w & 0xffff0000u);
  } else if constexpr (sizeof(T) == 4) {
    const float4 f = *reinterpret_cast<const float4*>(p);
    v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
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
  } else if constexpr (VEC == 2 && sizeof(T) == 4) {
    *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
  } else if constexpr (VEC == 2) {
    *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(v[0], v[1]);
  } else if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
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

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// a / b, rounded once: the product with the rounded reciprocal and Markstein's correction by its
// remainder.  (Codes of the product alone fall to the other side of a halfway point 2.4 times as often as
// the quotient's.)
__device__ __forceinline__ float quotient(float a, float b, float inv) {
  const float q = a * inv;
  return fmaf(fmaf(-q, b, a), inv, q);
}

// A group's scale and its reciprocal.  An infinite scale is divided by as the reciprocal 0 alone (the
// correction by the remainder of 0 times infinity would be NaN).
struct __align__(8) Scale {
  float by, inv;
  __device__ __forceinline__ Scale() {}
  __device__ __forceinline__ explicit Scale(float s) : by(s == INFINITY ? 0.f : s), inv(1.0f / s) {}
  __device__ __forceinline__ float of(float v) const { return quotient(v, by, inv); }
  // two at once, as codes
  __device__ __forceinline__ uint32_t codes(float v0, float v1) const {
    uint64_t v, q, r;
    const uint64_t i = pair(inv, inv), b = pair(-by, -by);
    v = pair(v0, v1);
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(q) : "l"(v), "l"(i));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(q), "l"(b), "l"(v));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(q) : "l"(r), "l"(i), "l"(q));
    float q0, q1;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(q0), "=f"(q1) : "l"(q));
    return e4m3x2(q0, q1);
  }
  static __device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(lo), "f"(hi));
    return p;
  }
};

// PAIRS: quotients two at once (16384 x 4096 by blocks 71.0 us, one at a time 71.5); not where a warp's
// scales differ from vector to vector and are held ahead (16384 x 2046 47.5 us, one at a time 45.6).
template <int VEC, bool PAIRS = true>
__device__ __forceinline__ void store_e4m3(uint8_t* p, const float* v, const Scale& s) {
  if constexpr (VEC == 1) {
    *p = (uint8_t)e4m3x2(s.of(v[0]), 0.f);
  } else if constexpr (VEC == 2) {
    *reinterpret_cast<uint16_t*>(p) = (uint16_t)(PAIRS ? s.codes(v[0], v[1]) : e4m3x2(s.of(v[0]), s.of(v[1])));
  } else {
    uint32_t w[VEC / 4];
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i)
      w[i] = s.codes(v[4 * i], v[4 * i + 1]) | (s.codes(v[4 * i + 2], v[4 * i + 3]) << 16);
    if constexpr (VEC == 4) *reinterpret_cast<uint32_t*>(p) = w[0];
    else *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  }
}

// max that keeps a NaN, so that a group holding one gets a NaN scale.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// The same over a warp, of magnitudes: as bits they order like numbers, a NaN above all.
__device__ __forceinline__ float warp_max_nan(float m) {
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m) & 0x7fffffffu));
}

__device__ __forceinline__ float scale_of(float amax) {
  return max_nan(amax == INFINITY ? amax : quotient(amax, 448.0f, 1.0f / 448.0f), 0x1p-120f);
}

struct NormArgs {
  const void* x;
  const void* r;
  const void* w;
  void* sum;
  void* y;
  float* scales;
  long long x_ld, r_ld;
  float w0, eps, inv_n;
  int rows, n;
};

// TPR threads hold one row, NV vectors of VEC elements each (vector j of thread t is vector
// j * TPR + t of the row).  TPR = 32 puts several rows into a CTA and needs no shared memory.
// KIND is a gdn_norm_out.
template <typename T, int VEC, int TPR, int NV, int KIND>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR) norm_kernel(const NormArgs a) {
  constexpr int CTA = TPR < 128 ? 128 : TPR;
  constexpr int WARPS = CTA / 32;
  __shared__ float part[WARPS];
  // One or two elements a lane: a warp's columns are a part of a group.  Group maxima, as the bits of
  // non-negative floats (a NaN's are above all), then the groups' scales.
  constexpr bool SMEM_GROUPS = KIND == GDN_NORM_E4M3_BLOCK && VEC <= 2 && TPR > 32;
  __shared__ uint32_t gmax[SMEM_GROUPS ? TPR * NV * VEC / 128 : 1];
  __shared__ Scale gscale[SMEM_GROUPS ? TPR * NV * VEC / 128 : 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int t = TPR < 128 ? tid % TPR : tid;
  const long long row = (long long)blockIdx.x * (CTA / TPR) + (TPR < 128 ? tid / TPR : 0);
  pdl_begin();
  if (TPR < 128 && row >= a.rows) return;   // whole warps leave; no barrier follows for TPR = 32
  const int n = a.n;
  const T* x = static_cast<const T*>(a.x) + row * a.x_ld;
  const T* r = a.r ? static_cast<const T*>(a.r) + row * a.r_ld : nullptr;
  float h[NV][VEC];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * TPR + t) * VEC;
#pragma unroll
    for (int e = 0; e < VEC; ++e) h[j][e] = 0.f;
    if (c < n) load_vec<T, VEC>(x + c, h[j]);
  }
  if (r) {
    float v[NV][VEC];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * TPR + t) * VEC;
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[j][e] = 0.f;
      if (c < n) load_vec<T, VEC>(r + c, v[j]);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < VEC; ++e) h[j][e] += v[j][e];
  }
  float ss = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < VEC; ++e) ss = fmaf(h[j][e], h[j][e], ss);
  if (a.sum) {
    T* s = static_cast<T*>(a.sum) + row * n;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * TPR + t) * VEC;
      if (c < n) store_vec<T, VEC>(s + c, h[j]);
    }
  }
  if constexpr (SMEM_GROUPS)
    for (int i = tid; i < TPR * NV * VEC / 128; i += CTA) gmax[i] = 0;
  ss = warp_sum(ss);
  if constexpr (TPR > 32) {
    if (lane == 0) part[warp] = ss;
    __syncthreads();
    ss = lane < WARPS ? part[lane] : 0.f;
    ss = warp_sum(ss);
  }
  const float rs = rsqrtf(ss * a.inv_n + a.eps);
  const T* w = static_cast<const T*>(a.w);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * TPR + t) * VEC;
    float g[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) g[e] = 0.f;
    if (c < n) load_vec<T, VEC>(w + c, g);
    // past the row's end h and the weight are zero: those lanes add nothing to a group's maximum
#pragma unroll
    for (int e = 0; e < VEC; ++e) h[j][e] = c < n ? h[j][e] * rs * (a.w0 + g[e]) : 0.f;
  }
  if constexpr (KIND == GDN_NORM_ACT) {
    T* y = static_cast<T*>(a.y) + row * n;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * TPR + t) * VEC;
      if (c < n) store_vec<T, VEC>(y + c, h[j]);
    }
  } else {
    uint8_t* y = static_cast<uint8_t*>(a.y) + row * n;
    float m[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      m[j] = 0.f;
#pragma unroll
      for (int e = 0; e < VEC; ++e) m[j] = max_nan(m[j], fabsf(h[j][e]));
    }
    if constexpr (KIND == GDN_NORM_E4M3_ROW) {
      float mr = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j) mr = max_nan(mr, m[j]);
      mr = warp_max_nan(mr);
      if constexpr (TPR > 32) {
        __syncthreads();   // part[] of the sum has been read
        if (lane == 0) part[warp] = mr;
        __syncthreads();
        mr = lane < WARPS ? part[lane] : 0.f;
        mr = warp_max_nan(mr);
      }
      const float s = scale_of(mr);
      const Scale scale(s);
      if (t == 0) a.scales[row] = s;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (j * TPR + t) * VEC;
        if (c < n) store_e4m3<VEC>(y + c, h[j], scale);
      }
    } else {
      const int groups = (n + 127) >> 7;
      if constexpr (VEC > 2) {
        // 128 columns are the vectors of 128 / VEC neighbouring lanes
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const int c = (j * TPR + t) * VEC;
          float mg = m[j];
#pragma unroll
          for (int o = 64 / VEC; o > 0; o >>= 1) mg = max_nan(mg, __shfl_xor_sync(0xffffffffu, mg, o));
          const float s = scale_of(mg);
          const Scale scale(s);
          if (c < n) {
            if ((c & 127) == 0) a.scales[row * groups + (c >> 7)] = s;
            store_e4m3<VEC>(y + c, h[j], scale);
          }
        }
      } else if constexpr (TPR == 32) {
        // the warp's next few vectors
        constexpr int kOf = 4 / VEC;
#pragma unroll
        for (int j0 = 0; j0 < NV; j0 += kOf) {
          float mg = 0.f;
#pragma unroll
          for (int j = j0; j < j0 + kOf; ++j) mg = max_nan(mg, m[j]);
          mg = warp_max_nan(mg);
          const float s = scale_of(mg);
          const Scale scale(s);
          if (t == 0 && j0 / kOf < groups) a.scales[row * groups + j0 / kOf] = s;
#pragma unroll
          for (int j = j0; j < j0 + kOf; ++j) {
            const int c = (j * TPR + t) * VEC;
            if (c < n) store_e4m3<VEC>(y + c, h[j], scale);
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          float mg = m[j];
          mg = warp_max_nan(mg);
          if (lane == 0) atomicMax(&gmax[(j * TPR + t) * VEC >> 7], __float_as_uint(mg));
        }
        __syncthreads();
        for (int i = tid; i < groups; i += CTA) {
          const float s = scale_of(__uint_as_float(gmax[i]));
          a.scales[row * groups + i] = s;
          gscale[i] = Scale(s);
        }
        __syncthreads();
        Scale scale[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) scale[j] = gscale[(j * TPR + t) * VEC >> 7];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const int c = (j * TPR + t) * VEC;
          if (c < n) store_e4m3<VEC, false>(y + c, h[j], scale[j]);
        }
      }
    }
  }
}

template <typename T, int VEC, int TPR, int NV>
int launch_one(const NormArgs& a, int kind, cudaStream_t stream) {
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
  cudaError_t e;
  if (kind == GDN_NORM_ACT) e = cudaLaunchKernelEx(&cfg, norm_kernel<T, VEC, TPR, NV, GDN_NORM_ACT>, a);
  else if (kind == GDN_NORM_E4M3_ROW) e = cudaLaunchKernelEx(&cfg, norm_kernel<T, VEC, TPR, NV, GDN_NORM_E4M3_ROW>, a);
  else e = cudaLaunchKernelEx(&cfg, norm_kernel<T, VEC, TPR, NV, GDN_NORM_E4M3_BLOCK>, a);
  return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

// A warp per row up to 1,024 elements (bf16; 512 f32), then 128 to 1,024 threads.
template <typename T, int VEC>
int launch_vec(const NormArgs& a, int kind, cudaStream_t s) {
  const int nv = (a.n + VEC - 1) / VEC;
  if (nv <= 32) return launch_one<T, VEC, 32, 1>(a, kind, s);
  if (nv <= 128) return launch_one<T, VEC, 32, 4>(a, kind, s);
  if (nv <= 256) return launch_one<T, VEC, 128, 2>(a, kind, s);
  if (nv <= 512) return launch_one<T, VEC, 128, 4>(a, kind, s);
  if (nv <= 1024) return launch_one<T, VEC, 256, 4>(a, kind, s);
  if (nv <= 2048) return launch_one<T, VEC, 512, 4>(a, kind, s);
  if (nv <= 4096) return launch_one<T, VEC, 1024, 4>(a, kind, s);
  return launch_one<T, VEC, 1024, 8>(a, kind, s);
}

// Rows off the 16-byte grid: two elements per access where they are all even, else one; a warp to a row
// up to 512 accesses.  (100,000 rows of 130, bf16 with residual: 103 us with a CTA to a row and one
// element an access, 28 so; 16384 x 2046 to 8 bits by rows 54 and 42 us; 16384 x 2047, which leaves one
// element an access, 53 us against 41 for 2048.)
template <typename T, int VEC>
int launch_narrow(const NormArgs& a, int kind, cudaStream_t s) {
  const int nv = (a.n + VEC - 1) / VEC;
  if (nv <= 128) return launch_one<T, VEC, 32, 4>(a, kind, s);
  if (nv <= 256) return launch_one<T, VEC, 32, 8>(a, kind, s);
  if (nv <= 512) return launch_one<T, VEC, 32, 16>(a, kind, s);
  if (nv <= 1024) return launch_one<T, VEC, 128, 8>(a, kind, s);
  if (nv <= 2048) return launch_one<T, VEC, 256, 8>(a, kind, s);
  if (nv <= 4096) return launch_one<T, VEC, 512, 8>(a, kind, s);
  if (nv <= 8192) return launch_one<T, VEC, 1024, 8>(a, kind, s);
  return launch_one<T, VEC, 1024, VEC == 1 ? 32 : 16>(a, kind, s);
}

template <typename T>
int launch_typed(const NormArgs& a, int kind, cudaStream_t s) {
  constexpr int kVec = 16 / sizeof(T);
  const long long bits = a.n | a.x_ld | (a.r ? a.r_ld : 0);
  if (bits % kVec == 0) return launch_vec<T, kVec>(a, kind, s);
  return bits % 2 == 0 ? launch_narrow<T, 2>(a, kind, s) : launch_narrow<T, 1>(a, kind, s);
}

}  // namespace

int launch_rms_norm(const void* x, long long x_ld, const void* residual, long long residual_ld,
                    const void* weight, float weight_offset, float eps, int rows, int n,
                    gdn_dtype act, int kind, void* sum_out, void* y, float* scales,
                    cudaStream_t stream) {
  const NormArgs a{x, residual, weight, sum_out, y, scales, x_ld, residual_ld, weight_offset, eps,
                   1.0f / (float)n, rows, n};
  return act == GDN_BF16 ? launch_typed<__nv_bfloat16>(a, kind, stream) : launch_typed<float>(a, kind, stream);
}

}  // namespace gdn
