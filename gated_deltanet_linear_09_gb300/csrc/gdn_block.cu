// gdn_block.cu -- a block's output on its way to the next block: its norm, gate and scale, the residual's
// addition, and the next block's norm.
//
//   b = x / rms_g(x) (w0 + post),  h = r + s c b act(z),  y = h / rms(h) (w0 + pre)
//
// A dozen flops per element: the floor is the bytes, x, z and r read once, h and y written once.  A row stays
// in registers from the first load to the last store, between the two sums that it waits for.  bf16: 8192 x 5120 with
// everything 72.5 us, 5.8 TB/s, 85 % of a copy; 8192 x 4096 in heads of 128 with a gate 37 us, 81 %; 13107 x 4096 with
// everything 87 us, 91 %.  bf16 rows off the boundaries run at half of that, bound by the instructions of single
// elements and pairs.
#include <type_traits>

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
// s = sigmoid(z).  For a result that is rounded to bf16 by approximations, off by about 2^-22 of it for z of a few units and
// by |z| 2^-24 far below (its argument's rounding): less than 2^-17 as long as it is not 0.  Two elements at a time where
// there are two.
template <typename T, int VEC>
__device__ __forceinline__ void sigmoids(const float* z, float* s) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) s[e] = sigmoidf_(z[e]);
  } else {
    constexpr float kMinusLog2e = -1.4426950408889634f;
#pragma unroll
    for (int e = 0; e < VEC; ++e) s[e] = z[e];
    mul_by<VEC>(s, kMinusLog2e);
#pragma unroll
    for (int e = 0; e < VEC; ++e) asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(s[e]));
    if constexpr (VEC == 1) s[0] += 1.0f;
    else
#pragma unroll
      for (int e = 0; e < VEC; e += 2) add_pair(s[e], s[e + 1], 1.0f, 1.0f);
#pragma unroll
    for (int e = 0; e < VEC; ++e) asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(s[e]));
  }
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];\n" ::"l"(p)); }

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
// loaded before it: what bounds this is the bytes in flight, and a row waits for two sums.  Where a thread's
// registers do not hold all of that (HOLD false), it is on its way to L2 meanwhile.  GROUPED: the first norm is
// over runs of 32 to 256 columns, 4 to 32 neighbouring lanes.
template <typename T, int VEC, int NV, bool SHARED, bool GROUPED, int MOST>
__global__ void __launch_bounds__(MOST) block_kernel(const BlockArgs a) {
  using R = Raw<T, VEC>;
  constexpr bool HOLD = NV * VEC * (int)sizeof(T) <= 64 && MOST < 1024;
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
  if constexpr (HOLD) {
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
  } else {
    constexpr int kLine = 128 / sizeof(T);
    for (int c = t * kLine; c < n; c += threads * kLine) {
      if (p.gate) prefetch_l2(static_cast<const T*>(p.gate) + row * p.gate_ld + c);
      if (p.residual) prefetch_l2(static_cast<const T*>(p.residual) + row * p.residual_ld + c);
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
      const int c = (j * threads + t) * VEC;
      if (c < n) {
        float g[VEC];
        if constexpr (!HOLD) w[j].load(static_cast<const T*>(p.post) + (GROUPED ? c & (p.group - 1) : c));
        w[j].get(g);
        weigh<VEC>(h[j], g, rs, p.weight_offset);
      }
    }
  }
  if constexpr (HOLD) {
    if (p.channel_scale) load(x, p.channel_scale, 0);
    if (p.pre) load(w, p.pre, 0);
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * threads + t) * VEC;
    if (c >= n) continue;
    float g[VEC];
    if (p.gate) {
      if constexpr (!HOLD) z[j].load(static_cast<const T*>(p.gate) + row * p.gate_ld + c);
      z[j].get(g);
      float s[VEC];
      sigmoids<T, VEC>(g, s);
      if (p.gate_act == GDN_GATE_SILU) mul_by<VEC>(s, g);
      mul_by<VEC>(h[j], s);
    }
    if (p.channel_scale) {
      if constexpr (!HOLD) x[j].load(static_cast<const T*>(p.channel_scale) + c);
      x[j].get(g);
      mul_by<VEC>(h[j], g);
    }
    if (p.residual) {
      if constexpr (!HOLD) r[j].load(static_cast<const T*>(p.residual) + row * p.residual_ld + c);
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
    if constexpr (!HOLD) w[j].load(static_cast<const T*>(p.pre) + c);
    w[j].get(g);
    weigh<VEC>(h[j], g, rs, p.weight_offset);
    R::put(static_cast<T*>(p.y) + row * n + c, h[j]);
  }
}

// How rows lie: on 16-byte boundaries; bf16 rows that begin on the same 4-byte offset in every tensor; anywhere.
enum Lie { kAligned, kPaired, kAnywhere };

// A row's bytes in the ring, and those of the weights beside it (not for aligned rows; for paired rows of odd
// length twice, once as for a row that begins in the middle of four bytes).
template <typename T, Lie LIE>
__host__ __device__ __forceinline__ uint32_t ring_plane(int n) {
  return LIE == kAligned ? n * (uint32_t)sizeof(T) : (n * (uint32_t)sizeof(T) + 30) / 16 * 16;
}
template <Lie LIE>
__host__ __device__ __forceinline__ int weight_elements(int n) {
  return LIE == kPaired ? (n % 2 ? 2 : 1) * ((n + 3) / 2 * 2) : n;
}
template <typename T, Lie LIE>
__host__ __device__ __forceinline__ uint32_t ring_weights(const gdn_block_args& p, int n) {
  if (LIE == kAligned) return 0;
  const uint32_t count = (p.post != nullptr) + (p.channel_scale != nullptr) + (p.pre != nullptr);
  return (count * weight_elements<LIE>(n) * (uint32_t)sizeof(T) + 15) / 16 * 16;
}
// Bytes from the 16-byte boundary before it.
__device__ __forceinline__ uint32_t lead(const void* p) { return (uint32_t)reinterpret_cast<uintptr_t>(p) & 15u; }

__device__ __forceinline__ uint32_t lds32(uint32_t at) {
  uint32_t u;
  asm volatile("ld.shared.b32 %0, [%1];\n" : "=r"(u) : "r"(at));
  return u;
}
template <typename T>
__device__ __forceinline__ float lds_one(uint32_t at) {
  if constexpr (sizeof(T) == 4) {
    return __uint_as_float(lds32(at));
  } else {
    uint16_t u;
    asm volatile("ld.shared.b16 %0, [%1];\n" : "=h"(u) : "r"(at));
    return __uint_as_float((uint32_t)u << 16);
  }
}

// A thread's vector in the kernel below, from element c on, of a row in shared memory (its address) or in global
// memory.
template <typename T, Lie LIE>
struct Piece {                       // 8 neighbouring elements
  static constexpr int VEC = 8;
  static __device__ __forceinline__ void get(uint32_t row, int c, int, int, float* x) {
    uint4 u[sizeof(T) / 2];
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i)
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];\n"
                   : "=r"(u[i].x), "=r"(u[i].y), "=r"(u[i].z), "=r"(u[i].w)
                   : "r"(row + c * (uint32_t)sizeof(T) + i * 16));
    reinterpret_cast<const Raw<T, 8>*>(u)->get(x);
  }
  static __device__ __forceinline__ void get(const T* row, int c, int, int, float* x) {
    Raw<T, 8> r;
    r.load(row + c);
    r.get(x);
  }
  static __device__ __forceinline__ void put(T* row, int c, int, int, const float* x) { Raw<T, 8>::put(row + c, x); }
};
template <>
struct Piece<__nv_bfloat16, kPaired> {   // two neighbours in four bytes, the row's first or last perhaps alone
  static constexpr int VEC = 2;
  static __device__ __forceinline__ void get(uint32_t row, int c, int, int n, float* x) {
    const uint32_t u = lds32(row + c * 2);
    x[0] = c >= 0 ? __uint_as_float(u << 16) : 0.f;
    x[1] = c + 1 < n ? __uint_as_float(u & 0xffff0000u) : 0.f;
  }
  static __device__ __forceinline__ void put(__nv_bfloat16* row, int c, int, int n, const float* x) {
    if (c >= 0 && c + 1 < n) {
      *reinterpret_cast<__nv_bfloat162*>(row + c) = __floats2bfloat162_rn(x[0], x[1]);
    } else {
      row[c < 0 ? 0 : c] = __float2bfloat16_rn(c < 0 ? x[1] : x[0]);
    }
  }
};
template <typename T>
struct Piece<T, kAnywhere> {             // the element and the one `step` on, which may be past the row's end
  static constexpr int VEC = 2;
  static __device__ __forceinline__ void get(uint32_t row, int c, int step, int n, float* x) {
    x[0] = lds_one<T>(row + c * (uint32_t)sizeof(T));
    x[1] = c + step < n ? lds_one<T>(row + (c + step) * (uint32_t)sizeof(T)) : 0.f;
  }
  static __device__ __forceinline__ void get(const T* row, int c, int step, int n, float* x) {
    x[0] = Act<T>::load(row + c);
    x[1] = c + step < n ? Act<T>::load(row + c + step) : 0.f;
  }
  static __device__ __forceinline__ void put(T* row, int c, int step, int n, const float* x) {
    Act<T>::store(row + c, x[0]);
    if (c + step < n) Act<T>::store(row + c + step, x[1]);
  }
};

// What is left to do for a CTA that stopped at a row whose copies did not come within the wait's limit: NaN in its outputs
// of that row and the later ones (there is no status word to set, and nothing that looks like a result is left), and a
// wait, with a limit too, for copies under way, whose stages follow from the row's turn.
template <typename T>
__device__ __noinline__ void leave_stopped(T* total, T* y, int row, int rows, int n, uint64_t* full, int stages) {
  const float nan = __uint_as_float(0x7fffffffu);
  for (long long r = row; r < rows; r += gridDim.x)
    for (int c = threadIdx.x; c < n; c += blockDim.x) {
      if (total) Act<T>::store(total + r * n + c, nan);
      if (y) Act<T>::store(y + r * n + c, nan);
    }
  if (threadIdx.x != 0) return;
  int turn = (row - (int)blockIdx.x) / (int)gridDim.x;
  for (long long r = row; r < rows && r < row + (long long)stages * gridDim.x; r += gridDim.x, ++turn)
    tc::mbar_wait(&full[turn % stages], (uint32_t)(turn / stages) & 1u, 100000000ull);
}

// The same for many rows: CTAs that stay, with the next row's x, gate and residual on their way into shared memory
// by bulk copies while a row is worked on.  (A CTA to a row has nothing in flight while it starts, waits for its
// sums and stores: 8192 x 4096 with a gate 46 us, so 37.)  The weights of aligned rows come from L1.  Other rows are
// copied from the 16-byte boundary before them to the one behind them, and read an element or two at a time; their
// weights lie beside the ring (KEPT: `weights` bytes), or come from L1 and L2 where there is no room.
template <typename T, Lie LIE, int NV, bool GROUPED, bool KEPT, int MOST>
__global__ void __launch_bounds__(MOST, 1024 / MOST) block_rows_kernel(const BlockArgs a, int stages, uint32_t weights) {
  using P = Piece<T, LIE>;
  constexpr int VEC = P::VEC;
  constexpr int kMostStages = 4;
  constexpr bool WIDE = LIE == kAligned;
  static_assert(!(WIDE && KEPT) && (KEPT || LIE != kPaired), "weights");
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ float part[4][32];
  __shared__ __align__(8) uint64_t full[kMostStages];
  __shared__ int stopped;              // the row whose copies did not come, or -1
  const gdn_block_args& p = a.p;
  const int threads = blockDim.x, t = threadIdx.x, n = a.n;
  const uint32_t plane = ring_plane<T, LIE>(n), planes = 1 + (p.gate != nullptr) + (p.residual != nullptr);
  const uint32_t gate_at = plane, residual_at = p.gate ? 2 * plane : plane;
  uint8_t* const rows_at = ring + weights;
  if (t == 0) {
    for (int i = 0; i < stages; ++i) tc::mbar_init(&full[i], 1);
    stopped = -1;
    tc::mbar_fence_init();
  }
  __syncthreads();
  pdl_begin();
  // (addresses in shared memory or in global memory)
  using At = std::conditional_t<KEPT, uint32_t, const T*>;
  At post_at, channel_at, pre_at;
  if constexpr (KEPT) {
    T* w = reinterpret_cast<T*>(ring);
    auto keep = [&](const void* from) {
      const uint32_t at = tc::smem_u32(w);
      if (!from) return at;
      for (int c = t; c < n; c += threads) {
        const T x = static_cast<const T*>(from)[c];
        w[c] = x;
        if (LIE == kPaired && n % 2) w[weight_elements<LIE>(n) / 2 + 1 + c] = x;
      }
      w += weight_elements<LIE>(n);
      return at;
    };
    post_at = keep(p.post);
    channel_at = keep(p.channel_scale);
    pre_at = keep(p.pre);
    __syncthreads();
  } else {
    post_at = static_cast<const T*>(p.post);
    channel_at = static_cast<const T*>(p.channel_scale);
    pre_at = static_cast<const T*>(p.pre);
  }
  auto fetch = [&](long long row, int st) {            // one thread
    if (row >= a.rows) return;
    uint8_t* to = rows_at + (size_t)st * planes * plane;
    const T* from[3] = {static_cast<const T*>(p.x) + row * p.x_ld, static_cast<const T*>(p.gate) + row * p.gate_ld,
                        static_cast<const T*>(p.residual) + row * p.residual_ld};
    if constexpr (WIDE) {
      tc::mbar_arrive_expect_tx(&full[st], planes * plane);
      tc::bulk_g2s(to, from[0], plane, &full[st]);
      if (p.gate) tc::bulk_g2s(to + gate_at, from[1], plane, &full[st]);
      if (p.residual) tc::bulk_g2s(to + residual_at, from[2], plane, &full[st]);
    } else {
      // (behind a row comes the next; behind the last, nothing that may be read)
      const bool have[3] = {true, p.gate != nullptr, p.residual != nullptr};
      const uint32_t at[3] = {0, gate_at, residual_at};
      uint32_t bytes[3], all = 0;
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        const uint32_t head = lead(from[i]), end = head + n * (uint32_t)sizeof(T);
        bytes[i] = !have[i] ? 0 : row + 1 < a.rows ? (end + 15) & ~15u : end & ~15u;
        all += bytes[i];
      }
      tc::mbar_arrive_expect_tx(&full[st], all);
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (bytes[i]) tc::bulk_g2s(to + at[i], reinterpret_cast<const uint8_t*>(from[i]) - lead(from[i]), bytes[i], &full[st]);
    }
  };
  if (t == 0)
    for (int i = 0; i < stages; ++i) fetch(blockIdx.x + (long long)i * gridDim.x, i);
  const int step = VEC * threads, mine = LIE == kAnywhere ? t : t * VEC;
  const int shifted = LIE == kPaired ? weight_elements<LIE>(n) + 2 : 0;      // bytes to the weights of a row that begins odd
  int st = 0, turn = 0;
  uint32_t phase = 0;
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
    uint8_t* const in = rows_at + (size_t)st * planes * plane;
    uint32_t x_in = tc::smem_u32(in), gate_in = x_in + gate_at, residual_in = x_in + residual_at;
    tc::mbar_wait(&full[st], phase);
    if constexpr (!WIDE) {
      auto begin = [&](uint32_t& at, uint32_t off, const void* base, long long ld) {
        if (!base) return;
        const T* from = static_cast<const T*>(base) + row * ld;
        const uint32_t head = lead(from) / sizeof(T);
        at += head * sizeof(T);
        if (row + 1 == a.rows) {                          // what the copy left out
          const int c = (int)((head + n) & ~(uint32_t)(16 / sizeof(T) - 1)) - (int)head + t;
          if (c >= 0 && c < n) reinterpret_cast<T*>(in + off)[head + c] = from[c];
        }
      };
      begin(x_in, 0, p.x, p.x_ld);
      begin(gate_in, gate_at, p.gate, p.gate_ld);
      begin(residual_in, residual_at, p.residual, p.residual_ld);
      if (row + 1 == a.rows) __syncthreads();
    }
    // paired: vectors begin with the element before a row that begins in the middle of four bytes
    const int odd = LIE == kPaired ? (int)(row & n & 1) : 0, first = mine - odd;
    const int w_at = odd ? shifted : 0;
    float h[NV][VEC];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = j * step + first;
#pragma unroll
      for (int e = 0; e < VEC; ++e) h[j][e] = 0.f;
      if (c < n) P::get(x_in, c, threads, n, h[j]);
    }
    if (p.post) {
      float rs = 0.f;
      if constexpr (!GROUPED) {
        float ss = 0.f, s2 = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) add_squares<VEC>(h[j], ss, s2);
        rs = rsqrtf(row_sum<true>(ss + s2, part[turn]) * a.inv_n + p.eps);
      }
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = j * step + first;
        if constexpr (GROUPED) {
          float ss = 0.f, s2 = 0.f;
          add_squares<VEC>(h[j], ss, s2);
          ss += s2;
          for (int o = p.group / 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          rs = rsqrtf(ss * a.inv_g + p.eps);
        }
        if (c < n) {
          float g[VEC];
          P::get(post_at + w_at, GROUPED ? c & (p.group - 1) : c, threads, n, g);
          weigh<VEC>(h[j], g, rs, p.weight_offset);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = j * step + first;
      if (c >= n) continue;
      float g[VEC];
      if (p.gate) {
        P::get(gate_in, c, threads, n, g);
        float s[VEC];
        sigmoids<T, VEC>(g, s);
        if (p.gate_act == GDN_GATE_SILU) mul_by<VEC>(s, g);
        mul_by<VEC>(h[j], s);
      }
      if (p.channel_scale) {
        P::get(channel_at + w_at, c, threads, n, g);
        mul_by<VEC>(h[j], g);
      }
      if (p.residual) {
        P::get(residual_in, c, threads, n, g);
        fma_by<VEC>(h[j], p.scale, g);
      } else {
        mul_by<VEC>(h[j], p.scale);
      }
      if (p.total) P::put(static_cast<T*>(p.total) + row * n, c, threads, n, h[j]);
    }
    // (one thread looks whether the wait ran out: every thread keeping what its own said costs rows off the boundaries 5 %)
    if (t == threads - 1 && !tc::mbar_try_wait(&full[st], phase)) stopped = (int)row;
    float rs = 0.f;
    if (p.pre) {
      float ss = 0.f, s2 = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j) add_squares<VEC>(h[j], ss, s2);
      rs = rsqrtf(row_sum<true>(ss + s2, part[2 + turn]) * a.inv_n + p.eps);
    } else {
      __syncthreads();
    }
    if ((uint32_t)*(volatile int*)&stopped <= (uint32_t)row) break;     // (the next row's is above it: the same for all threads)
    // (every thread has read the row)
    if (t == 0) fetch(row + (long long)stages * gridDim.x, st);
    if (++st == stages) {
      st = 0;
      phase ^= 1u;
    }
    if (p.pre) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = j * step + first;
        if (c >= n) continue;
        float g[VEC];
        P::get(pre_at + w_at, c, threads, n, g);
        weigh<VEC>(h[j], g, rs, p.weight_offset);
        P::put(static_cast<T*>(p.y) + row * n, c, threads, n, h[j]);
      }
    }
  }
  __syncthreads();
  if (stopped >= 0) leave_stopped<T>(static_cast<T*>(p.total), static_cast<T*>(p.y), stopped, a.rows, n, full, stages);
}

// Launches it where the rows are many and a few fit an SM's shared memory; GDN_ERR_UNSUPPORTED_SHAPE: use the other.
constexpr int kRing = 208 * 1024;
template <typename T, Lie LIE, int NV, bool KEPT, int MOST>
int launch_rows(const BlockArgs& a, int ctas, int sms, cudaStream_t stream) {
  constexpr int kOne = NV * Piece<T, LIE>::VEC * 32;      // elements of a warp
  const size_t stage = (size_t)(1 + (a.p.gate != nullptr) + (a.p.residual != nullptr)) * ring_plane<T, LIE>(a.n);
  const size_t weights = KEPT ? ring_weights<T, LIE>(a.p, a.n) : 0;
  const int threads = (a.n + (LIE == kPaired) + kOne - 1) / kOne * 32;
  if (threads > MOST) return GDN_ERR_UNSUPPORTED_SHAPE;
  if (ctas > 1024 / threads) ctas = 1024 / threads;
  if (a.rows / 4 < ctas * sms) return GDN_ERR_UNSUPPORTED_SHAPE;
  int stages = (int)((kRing / ctas - weights) / stage);
  if (stages > 4) stages = 4;
  const bool grouped = LIE == kAligned && a.p.post && a.p.group < a.n;
  auto kern = grouped ? block_rows_kernel<T, LIE, NV, LIE == kAligned, KEPT, MOST> : block_rows_kernel<T, LIE, NV, false, KEPT, MOST>;
  static OncePerDevice once[2];
  const int rc = raise_smem(once[grouped], kern, kRing);
  if (rc != GDN_OK) return rc;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(ctas * sms));
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = weights + stages * stage;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a, stages, (uint32_t)weights) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

// Two rows' ring for each of as many CTAs as fit an SM.  Aligned rows: two vectors a thread, so that a row is done
// soon (13107 bf16 x 4096 with everything 87 us, with four vectors 111), four where 512 threads need that.  Other
// rows: 8 elements a thread, of bf16 rows above 256 elements, which take half the instructions, 16, so that more rows
// are under way (43669 x 2049 156 us, with 8 elements 184; 6989 f32 x 6401 104 us, with 16 elements 193), unless
// there is one CTA to an SM (10483 bf16 x 5121 with everything 185 us, with 16 elements 231).  Rows too long for 1024
// threads of these: 16 elements, or 32.
template <typename T, Lie LIE>
int launch_ring(const BlockArgs& a, cudaStream_t stream) {
  const int sms = sm_count();
  const size_t row = (size_t)(1 + (a.p.gate != nullptr) + (a.p.residual != nullptr)) * ring_plane<T, LIE>(a.n);
  const size_t weights = ring_weights<T, LIE>(a.p, a.n);
  const int ctas = (int)(kRing / (2 * row + weights));
  if (sms <= 0) return GDN_ERR_UNSUPPORTED_SHAPE;
  if constexpr (LIE == kAligned) {
    if (ctas < 1) return GDN_ERR_UNSUPPORTED_SHAPE;
    if (a.n <= 8192) return launch_rows<T, LIE, 2, false, 512>(a, ctas, sms, stream);
    return launch_rows<T, LIE, 4, false, 512>(a, ctas, sms, stream);
  } else {
    if (ctas < 1 || a.n > 16384) {
      if (row > kRing) return GDN_ERR_UNSUPPORTED_SHAPE;
      if constexpr (LIE == kPaired) return launch_ring<T, kAnywhere>(a, stream);
      else if (a.n <= 16384) return launch_rows<T, LIE, 8, false, 1024>(a, 1, sms, stream);
      else return launch_rows<T, LIE, 16, false, 1024>(a, 1, sms, stream);
    }
    if (a.n > 8192 || (sizeof(T) == 2 && a.n > 256 && ctas > 1)) return launch_rows<T, LIE, 8, true, 1024>(a, ctas, sms, stream);
    return launch_rows<T, LIE, 4, true, 1024>(a, ctas, sms, stream);
  }
}

template <typename T, int VEC, int NV, bool SHARED, int MOST>
int launch_one(const BlockArgs& a, cudaStream_t stream) {
  const int vectors = (a.n + VEC - 1) / VEC;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(SHARED ? a.rows : (a.rows - 1) / 4 + 1));
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

// A warp to a row of up to 512 elements, for f32 1024 (43690 x 1024 79 us, by the rows kernel 99; 87381 bf16 x 1024
// 95 us, by the rows kernel 90).  Above that the rows kernel, where there are rows enough, else a CTA to a row with
// four vectors of bf16 a thread, or two of f32 (its registers hold twice as much), more where a row would not fit 512
// threads.
template <typename T>
int launch_wide(const BlockArgs& a, cudaStream_t s) {
  constexpr int NV = sizeof(T) == 4 ? 2 : 4;
  const int nv = a.n / 8;
  if (nv <= 32) return launch_one<T, 8, 1, false, 128>(a, s);
  if (nv <= 64) return launch_one<T, 8, 2, false, 128>(a, s);
  if constexpr (sizeof(T) == 4)
    if (nv <= 128) return launch_one<T, 8, 4, false, 128>(a, s);
  const int rc = launch_ring<T, kAligned>(a, s);
  if (rc != GDN_ERR_UNSUPPORTED_SHAPE) return rc;
  if (nv <= NV * 256) return launch_one<T, 8, NV, true, 256>(a, s);
  if (nv <= NV * 512) return launch_one<T, 8, NV, true, 512>(a, s);
  return launch_one<T, 8, 4, true, 1024>(a, s);
}

// Rows off the 16-byte grid, an element per access.
template <typename T>
int launch_narrow(const BlockArgs& a, cudaStream_t s) {
  if (a.n > 128) {
    const long long odd = (a.n ^ a.p.x_ld) | (a.p.gate ? a.n ^ a.p.gate_ld : 0) | (a.p.residual ? a.n ^ a.p.residual_ld : 0);
    int rc = GDN_ERR_UNSUPPORTED_SHAPE;
    if constexpr (sizeof(T) == 2) rc = odd % 2 == 0 ? launch_ring<T, kPaired>(a, s) : launch_ring<T, kAnywhere>(a, s);
    else rc = launch_ring<T, kAnywhere>(a, s);
    if (rc != GDN_ERR_UNSUPPORTED_SHAPE) return rc;
  }
  if (a.n <= 128) return launch_one<T, 1, 4, false, 128>(a, s);
  if (a.n <= 4096) return launch_one<T, 1, 8, true, 512>(a, s);
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
