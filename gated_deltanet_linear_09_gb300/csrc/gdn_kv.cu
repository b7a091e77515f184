// gdn_kv.cu -- the paged key/value cache: storing new tokens' vectors (bf16, or quantised to e4m3
// with a power-of-two scale per vector) and reading places back.
//
// The scale of a vector is the least power of two that brings its largest magnitude to 448.  A
// power of two leaves the mantissas alone, so it quantises as well as any scale does (it can only
// cost the topmost binade of the exponent range), and an 8-bit value times it is exactly a bf16
// value: reading is exact, and attention runs on the same numbers however the cache is held.
#include "gdn_internal.h"
#include "gdn_kv.cuh"

namespace gdn {

namespace {

__device__ __forceinline__ uint32_t e4m3x4(const float* v) {
  uint16_t a, b;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(a) : "f"(v[1]), "f"(v[0]));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(b) : "f"(v[3]), "f"(v[2]));
  return (uint32_t)a | ((uint32_t)b << 16);
}

__device__ __forceinline__ void unpack8(const uint4 u, float* v) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// 8 e4m3 codes -> 8 bf16 (4 words), times the scale of exponent byte b.
__device__ __forceinline__ uint4 dequant8(uint2 u, uint32_t b) {
  uint32_t w[4];
  e4m3x4_to_bf16(u.x, w[0], w[1]);
  e4m3x4_to_bf16(u.y, w[2], w[3]);
  const uint32_t s = scale_bits(b);
  const uint32_t s2 = s | (s << 16);
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = mul_bf16x2(w[i], s2);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// One thread per 8 elements of the key and the value vector of U (token, head) pairs: D / 8
// neighbouring lanes share a vector, whose maximum they find by shuffles.  Bound by the bytes; what
// keeps a thread from its stores is the chain of lookups to its place (sequence, length, page), so
// the vectors are loaded first, for all U at once, and sequences are found by a 32-way search per
// warp (two steps up to 1,024 sequences) instead of a binary one.
template <int D>
struct Lane {
  long long vec;      // (token, head) pair
  int part, tok, head;
  bool live;
  __device__ __forceinline__ Lane(const KvView& c, const KvBatchView& bt, int u) {
    constexpr int L = D / 8;
    const long long gid = ((long long)u * gridDim.x + blockIdx.x) * blockDim.x + threadIdx.x;
    vec = gid / L;
    part = (int)(gid % L);
    live = vec < (long long)bt.total * c.H;
    tok = live ? (int)((unsigned long long)vec >> 32 == 0 ? (unsigned)vec / (unsigned)c.H : vec / c.H) : bt.total - 1;
    head = live ? (int)(vec - (long long)tok * c.H) : 0;
  }
};

template <int D, bool Q, int U>
__global__ void __launch_bounds__(256) append_kernel(const KvView c, const KvBatchView bt,
                                                     const __nv_bfloat16* __restrict__ k, long long k_ld,
                                                     const __nv_bfloat16* __restrict__ v, long long v_ld) {
  pdl_begin();
  uint4 kx[U], vx[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const Lane<D> a(c, bt, u);
    kx[u] = vx[u] = make_uint4(0, 0, 0, 0);
    if (a.live) {
      kx[u] = __ldcs(reinterpret_cast<const uint4*>(k + (long long)a.tok * k_ld + a.head * D + a.part * 8));
      vx[u] = __ldcs(reinterpret_cast<const uint4*>(v + (long long)a.tok * v_ld + a.head * D + a.part * 8));
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const Lane<D> a(c, bt, u);
    const Place p = find_place(c, bt, a.tok);
    const bool store = a.live && p.page >= 0;
    const long long at = store ? (((long long)p.page * c.H + a.head) << c.page_shift) + p.off : 0;
    if constexpr (!Q) {
      if (store) {
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(c.k) + at * D + a.part * 8) = kx[u];
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(c.v) + at * D + a.part * 8) = vx[u];
      }
    } else {
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        const uint4 x = which ? vx[u] : kx[u];
        uint32_t m = 0;
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          m = max(m, w[i] & 0x7fffu);
          m = max(m, (w[i] >> 16) & 0x7fffu);
        }
#pragma unroll
        for (int o = D / 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        const int b = scale_byte(m);
        // 2^(127 - b): exponent field 254 - b, at least 7 (b <= 247 for finite vectors)
        const float inv = __uint_as_float((uint32_t)(254 - (b == 255 ? 127 : b)) << 23);
        float f[8];
        unpack8(x, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] *= inv;
        uint2 q = make_uint2(e4m3x4(f), e4m3x4(f + 4));
        if (store) {
          // codes of a vector that reads as NaN: any finite ones
          if (b == 255) q = make_uint2(0, 0);
          *reinterpret_cast<uint2*>(static_cast<uint8_t*>(which ? c.v : c.k) + at * D + a.part * 8) = q;
          if (a.part == 0) (which ? c.vs : c.ks)[at] = (uint8_t)b;
        }
      }
    }
  }
}

template <int D, bool Q, int U>
__global__ void __launch_bounds__(256) read_kernel(const KvView c, const KvBatchView bt,
                                                   __nv_bfloat16* __restrict__ k,
                                                   __nv_bfloat16* __restrict__ v) {
  pdl_begin();
  uint4 kx[U], vx[U];
  uint2 kq[U], vq[U];
  uint32_t kb[U], vb[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const Lane<D> a(c, bt, u);
    const Place p = find_place(c, bt, a.tok);
    kx[u] = vx[u] = make_uint4(0, 0, 0, 0);
    kq[u] = vq[u] = make_uint2(0, 0);
    kb[u] = vb[u] = 0;
    if (a.live && p.page >= 0) {
      const long long at = (((long long)p.page * c.H + a.head) << c.page_shift) + p.off;
      if constexpr (!Q) {
        kx[u] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(c.k) + at * D + a.part * 8));
        vx[u] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(c.v) + at * D + a.part * 8));
      } else {
        kq[u] = __ldcs(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(c.k) + at * D + a.part * 8));
        vq[u] = __ldcs(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(c.v) + at * D + a.part * 8));
        kb[u] = c.ks[at];
        vb[u] = c.vs[at];
      }
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const Lane<D> a(c, bt, u);
    if (!a.live) continue;
    if constexpr (Q) {
      kx[u] = dequant8(kq[u], kb[u]);      // (codes 0 and byte 0 give zeros)
      vx[u] = dequant8(vq[u], vb[u]);
    }
    const long long o = a.vec * D + a.part * 8;
    __stcs(reinterpret_cast<uint4*>(k + o), kx[u]);
    __stcs(reinterpret_cast<uint4*>(v + o), vx[u]);
  }
}

template <typename... KArgs, typename... Args>
int launch(void (*kern)(KArgs...), int each, long long threads, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((threads + 256 * each - 1) / (256 * each)));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

// More than one pair a thread once there are far more threads than the SMs hold at a time.
constexpr long long kManyThreads = 1 << 20;

}  // namespace

int launch_kv_append(const KvView& c, const KvBatchView& bt, const void* k, long long k_ld,
                     const void* v, long long v_ld, cudaStream_t stream) {
  const auto* kp = static_cast<const __nv_bfloat16*>(k);
  const auto* vp = static_cast<const __nv_bfloat16*>(v);
  const long long n = (long long)bt.total * c.H * (c.D / 8);
#define GDN_RUN_U(DD, U)                                                                    \
  return c.ks ? launch(append_kernel<DD, true, U>, U, n, stream, c, bt, kp, k_ld, vp, v_ld) \
              : launch(append_kernel<DD, false, U>, U, n, stream, c, bt, kp, k_ld, vp, v_ld)
#define GDN_RUN(DD)               \
  if (n > kManyThreads) GDN_RUN_U(DD, 2); \
  else GDN_RUN_U(DD, 1)
  if (c.D == 64) { GDN_RUN(64); }
  if (c.D == 128) { GDN_RUN(128); }
  GDN_RUN(256);
#undef GDN_RUN
#undef GDN_RUN_U
}

int launch_kv_read(const KvView& c, const KvBatchView& bt, void* k, void* v, cudaStream_t stream) {
  auto* kp = static_cast<__nv_bfloat16*>(k);
  auto* vp = static_cast<__nv_bfloat16*>(v);
  const long long n = (long long)bt.total * c.H * (c.D / 8);
#define GDN_RUN_U(DD, U)                                                          \
  return c.ks ? launch(read_kernel<DD, true, U>, U, n, stream, c, bt, kp, vp)     \
              : launch(read_kernel<DD, false, U>, U, n, stream, c, bt, kp, vp)
#define GDN_RUN(DD)               \
  if (n > kManyThreads) GDN_RUN_U(DD, 2); \
  else GDN_RUN_U(DD, 1)
  if (c.D == 64) { GDN_RUN(64); }
  if (c.D == 128) { GDN_RUN(128); }
  GDN_RUN(256);
#undef GDN_RUN
#undef GDN_RUN_U
}

}  // namespace gdn
