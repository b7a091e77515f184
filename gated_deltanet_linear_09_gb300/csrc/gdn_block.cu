// gdn_block.cu -- a block's output on its way to the next block: its norm, gate and scale, the residual's
// addition, and the next block's norm.
//
//   b = x / rms_g(x) (w0 + post),  h = r + s c b act(z),  y = h / rms(h) (w0 + pre)
//
// A dozen flops per element: the floor is the bytes, x, z and r read once, h and y written once.  A row stays
// in registers from the first load to the last store, between the two sums that it waits for.
#include "gdn_internal.h"
#include "gdn_tc.cuh"

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

// The same for many rows: CTAs that stay, with the next row's x, gate and residual on their way into shared memory
// by bulk copies while a row is worked on.  (A CTA to a row has nothing in flight while it starts, waits for its
// sums and stores: 8192 rows of 4096 with a gate 46 us, so 36.)  Two vectors a thread (NV)
// leave room for the weights in registers; with four they come from L1.
template <typename T, int NV, bool GROUPED, int MOST>
__global__ void __launch_bounds__(MOST) block_rows_kernel(const BlockArgs a, int stages) {
  using R = Raw<T, 8>;
  constexpr int kMostStages = 4;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ float part[4][32];
  __shared__ __align__(8) uint64_t full[kMostStages];
  const gdn_block_args& p = a.p;
  const int threads = blockDim.x, t = threadIdx.x, n = a.n;
  const uint32_t plane = (uint32_t)n * sizeof(T), planes = 1 + (p.gate != nullptr) + (p.residual != nullptr);
  const uint32_t gate_at = plane, residual_at = p.gate ? 2 * plane : plane;
  if (t == 0) {
    for (int i = 0; i < stages; ++i) tc::mbar_init(&full[i], 1);
    tc::mbar_fence_init();
  }
  __syncthreads();
  pdl_begin();
  constexpr bool kHold = NV <= 2;
  R post[NV], channel[NV], pre[NV];
#pragma unroll
  for (int j = 0; j < NV && kHold; ++j) {
    const int c = (j * threads + t) * 8;
    if (c >= n) continue;
    if (p.post) post[j].load(static_cast<const T*>(p.post) + (GROUPED ? c & (p.group - 1) : c));
    if (p.channel_scale) channel[j].load(static_cast<const T*>(p.channel_scale) + c);
    if (p.pre) pre[j].load(static_cast<const T*>(p.pre) + c);
  }
  auto fetch = [&](long long row, int st) {            // one thread
    if (row >= a.rows) return;
    uint8_t* to = ring + (size_t)st * planes * plane;
    tc::mbar_arrive_expect_tx(&full[st], planes * plane);
    tc::bulk_g2s(to, static_cast<const T*>(p.x) + row * p.x_ld, plane, &full[st]);
    if (p.gate) tc::bulk_g2s(to + gate_at, static_cast<const T*>(p.gate) + row * p.gate_ld, plane, &full[st]);
    if (p.residual) tc::bulk_g2s(to + residual_at, static_cast<const T*>(p.residual) + row * p.residual_ld, plane, &full[st]);
  };
  if (t == 0)
    for (int i = 0; i < stages; ++i) fetch(blockIdx.x + (long long)i * gridDim.x, i);
  int st = 0, turn = 0;
  uint32_t phase = 0;
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
    const uint8_t* in = ring + (size_t)st * planes * plane;
    tc::mbar_wait(&full[st], phase);
    float h[NV][8];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * threads + t) * 8;
#pragma unroll
      for (int e = 0; e < 8; ++e) h[j][e] = 0.f;
      if (c < n) {
        R x;
        x.load(reinterpret_cast<const T*>(in) + c);
        x.get(h[j]);
      }
    }
    if (p.post) {
      float rs = 0.f;
      if constexpr (!GROUPED) {
        float ss = 0.f, s2 = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) add_squares<8>(h[j], ss, s2);
        rs = rsqrtf(row_sum<true>(ss + s2, part[turn]) * a.inv_n + p.eps);
      }
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (j * threads + t) * 8;
        if constexpr (GROUPED) {
          float ss = 0.f, s2 = 0.f;
          add_squares<8>(h[j], ss, s2);
          ss += s2;
          for (int o = p.group / 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          rs = rsqrtf(ss * a.inv_g + p.eps);
        }
        if (c < n) {
          float g[8];
          if (!kHold) post[j].load(static_cast<const T*>(p.post) + (GROUPED ? c & (p.group - 1) : c));
          post[j].get(g);
          weigh<8>(h[j], g, rs, p.weight_offset);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * threads + t) * 8;
      if (c >= n) continue;
      R w;
      float g[8];
      if (p.gate) {
        w.load(reinterpret_cast<const T*>(in + gate_at) + c);
        w.get(g);
        float s[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] = sizeof(T) == 4 ? sigmoidf_(g[e]) : sigmoid_fast(g[e]);
        if (p.gate_act == GDN_GATE_SILU) mul_by<8>(s, g);
        mul_by<8>(h[j], s);
      }
      if (p.channel_scale) {
        if (!kHold) channel[j].load(static_cast<const T*>(p.channel_scale) + c);
        channel[j].get(g);
        mul_by<8>(h[j], g);
      }
      if (p.residual) {
        w.load(reinterpret_cast<const T*>(in + residual_at) + c);
        w.get(g);
        fma_by<8>(h[j], p.scale, g);
      } else {
        mul_by<8>(h[j], p.scale);
      }
      if (p.total) R::put(static_cast<T*>(p.total) + row * n + c, h[j]);
    }
    float rs = 0.f;
    if (p.pre) {
      float ss = 0.f, s2 = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j) add_squares<8>(h[j], ss, s2);
      rs = rsqrtf(row_sum<true>(ss + s2, part[2 + turn]) * a.inv_n + p.eps);
    } else {
      __syncthreads();
    }
    // (every thread has read the row)
    if (t == 0) fetch(row + (long long)stages * gridDim.x, st);
    if (++st == stages) {
      st = 0;
      phase ^= 1u;
    }
    if (p.pre) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (j * threads + t) * 8;
        if (c >= n) continue;
        float g[8];
        if (!kHold) pre[j].load(static_cast<const T*>(p.pre) + c);
        pre[j].get(g);
        weigh<8>(h[j], g, rs, p.weight_offset);
        R::put(static_cast<T*>(p.y) + row * n + c, h[j]);
      }
    }
  }
}

// Launches it where the rows are many and a few fit an SM's shared memory; GDN_ERR_UNSUPPORTED_SHAPE: use the other.
template <typename T, int NV>
int launch_rows(const BlockArgs& a, int ctas, int sms, size_t stage, cudaStream_t stream) {
  constexpr int kRing = 208 * 1024;
  const int threads = (a.n / 8 + NV * 32 - 1) / (NV * 32) * 32;
  if (ctas > 1024 / threads) ctas = 1024 / threads;
  if (a.rows < 4 * ctas * sms) return GDN_ERR_UNSUPPORTED_SHAPE;
  int stages = (int)(kRing / (ctas * stage));
  if (stages > 4) stages = 4;
  const bool grouped = a.p.post && a.p.group < a.n;
  auto kern = grouped ? block_rows_kernel<T, NV, true, 512> : block_rows_kernel<T, NV, false, 512>;
  static OncePerDevice once[2];
  const int rc = raise_smem(once[grouped], kern, kRing);
  if (rc != GDN_OK) return rc;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(ctas * sms));
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = stages * stage;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a, stages) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

// Two rows' ring for each of as many CTAs as fit an SM.  Four vectors a thread (of bf16) where that makes CTAs small
// and they are four or more: many rows at once hide a row's sums (8192 x 4096 with a gate 36 us, with two
// vectors 40); else two, so that a row is done sooner (8192 x 5120 with everything 74 us, with four 84).
template <typename T>
int launch_ring(const BlockArgs& a, cudaStream_t stream) {
  const int sms = sm_count(), planes = 1 + (a.p.gate != nullptr) + (a.p.residual != nullptr);
  const size_t stage = (size_t)planes * a.n * sizeof(T);
  const int ctas = (int)(208 * 1024 / (2 * stage));
  if (sms <= 0 || ctas < 2) return GDN_ERR_UNSUPPORTED_SHAPE;
  if (sizeof(T) == 2 && ctas >= 4) return launch_rows<T, 4>(a, ctas, sms, stage, stream);
  return launch_rows<T, 2>(a, ctas, sms, stage, stream);
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
  if (nv <= 1024) {
    const int rc = launch_ring<T>(a, s);
    if (rc != GDN_ERR_UNSUPPORTED_SHAPE) return rc;
  }
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
