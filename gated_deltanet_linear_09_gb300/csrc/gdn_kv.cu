// gdn_kv.cu -- the paged key/value cache: storing new tokens' vectors (bf16, or quantised to e4m3
// with a power-of-two scale per vector) and reading places back.
//
// The scale of a vector is the least power of two that brings its largest magnitude to 448.  A
// power of two leaves the mantissas alone, so it quantises as well as any scale does (it can only
// cost the topmost binade of the exponent range), and an 8-bit value times it is exactly a bf16
// value: reading is exact, and attention runs on the same numbers however the cache is held.
#include <type_traits>

#include "gdn_internal.h"
#include "gdn_kv.cuh"

namespace gdn {

namespace {

// 8 e4m3 codes -> 8 bf16 (4 words), times the scale of exponent byte b.  The codes' bits are the
// values times 2^-120: one multiply by 2^120 times the scale where that is a bf16 value, else two.
__device__ __forceinline__ uint4 dequant8(uint2 u, uint32_t b) {
  const uint32_t f = b <= 134 ? (b + 120) << 7 : 0x7b80u, f2 = f | (f << 16);
  uint32_t w[4];
  w[0] = mul_bf16x2(e4m3_hi_bits(__byte_perm(u.x, 0, 0x1404)), f2);
  w[1] = mul_bf16x2(e4m3_hi_bits(__byte_perm(u.x, 0, 0x3424)), f2);
  w[2] = mul_bf16x2(e4m3_hi_bits(__byte_perm(u.y, 0, 0x1404)), f2);
  w[3] = mul_bf16x2(e4m3_hi_bits(__byte_perm(u.y, 0, 0x3424)), f2);
  if (b > 134) {
    const uint32_t s = scale_bits(b), s2 = s | (s << 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = mul_bf16x2(w[i], s2);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// A CTA takes neighbouring tokens, a warp a token at a time (or a few narrow ones): the lanes walk its
// heads' vectors in pieces of 16 elements (8 from each half of the vector, so that a warp's loads and
// stores are whole), D / 16 neighbouring lanes to a vector.  Bound by the bytes as long as the work
// per piece is small: the places (a 32-way search, a length, a page) are looked up once per token by
// one warp, into shared memory, while the others' first loads are under way.  (Looked up by every
// thread with 64-bit pair indices, the instructions were the bound: 68 % of the issue slots and
// 3.6 TB/s.  With 8 elements a lane: 4.5 TB/s on seven prompts of 34,000 tokens in all, 2 x 256,
// 8-bit; with 16, 5.4.)
constexpr int kMostTokens = 32;

// The pieces of a CTA's tokens as its 8 warps walk them: every eighth run of 32 pieces each (narrow
// tokens side by side in a run where they divide a warp).
struct Walk {
  int width, side, turns, count;
  int tok, turn;                   // this run's first token, and run in the token
  int lane_tok, lane_piece;
  __device__ __forceinline__ Walk(int pieces, int tokens) {
    const int lane = threadIdx.x & 31;
    width = pieces;
    count = tokens;
    side = pieces < 32 && 32 % pieces == 0 ? 32 / pieces : 1;
    turns = (pieces + 31) >> 5;
    lane_tok = side > 1 ? lane / pieces : 0;
    lane_piece = side > 1 ? lane % pieces : lane;
    tok = 0;
    turn = threadIdx.x >> 5;
    settle();
  }
  __device__ __forceinline__ void settle() {
    while (turn >= turns) { turn -= turns; tok += side; }
  }
  __device__ __forceinline__ bool more() const { return tok < count; }
  __device__ __forceinline__ void next() { turn += 8; settle(); }
  __device__ __forceinline__ int token() const { return tok + lane_tok; }
  __device__ __forceinline__ int piece() const { return turn * 32 + lane_piece; }
  __device__ __forceinline__ bool live() const { return token() < count && piece() < width; }
};

// Places of tokens t0 .. t0 + count - 1 (count <= 32) into shared memory, by one warp: the vector
// index of head 0, or -1.
__device__ __forceinline__ void find_places(const KvView& c, const KvBatchView& bt, int t0, int count,
                                            long long* place) {
  const int lane = threadIdx.x & 31;
  const Place p = find_place(c, bt, min(t0 + lane, bt.total - 1));
  if (lane < count) place[lane] = p.page < 0 ? -1 : (((long long)p.page * c.H) << c.page_shift) + p.off;
}

// The largest magnitude's bits among 16 elements.
__device__ __forceinline__ uint32_t top_of(const uint4* x) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    m = __vmaxu2(m, __vmaxu2(__vmaxu2(x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu),
                             __vmaxu2(x[i].z & 0x7fff7fffu, x[i].w & 0x7fff7fffu)));
  return max(m & 0xffffu, m >> 16);
}

// 8 elements of a vector with this scale byte -> codes.  The factor 2^(127 - b) is a bf16 value
// (exponent field 254 - b, 7 to 244) and the products are exact; the codes of a vector that reads as
// NaN: any finite ones.
__device__ __forceinline__ uint2 quantise8(const uint4 x, int b) {
  if (b == 255) return make_uint2(0, 0);
  const uint32_t f = (uint32_t)(254 - b) << 7, f2 = f | (f << 16);
  const uint32_t w[4] = {mul_bf16x2(x.x, f2), mul_bf16x2(x.y, f2), mul_bf16x2(x.z, f2), mul_bf16x2(x.w, f2)};
  uint16_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
        : "=h"(h[i])
        : "f"(__uint_as_float(w[i] & 0xffff0000u)), "f"(__uint_as_float(w[i] << 16)));
  return make_uint2((uint32_t)h[0] | ((uint32_t)h[1] << 16), (uint32_t)h[2] | ((uint32_t)h[3] << 16));
}

template <int D, bool Q>
__global__ void __launch_bounds__(256) append_kernel(const KvView c, const KvBatchView bt, int tokens,
                                                     const __nv_bfloat16* __restrict__ k, long long k_ld,
                                                     const __nv_bfloat16* __restrict__ v, long long v_ld) {
  constexpr int L = D / 16;
  __shared__ long long place[kMostTokens];
  const int t0 = blockIdx.x * tokens, count = min(tokens, bt.total - t0);
  Walk w(c.H * L, count);
  pdl_begin();
  struct Piece {
    uint4 k[2], v[2];
    int head, part;
  };
  auto load = [&](Piece& x) {
    x.head = w.piece() / L;
    x.part = w.piece() % L;
#pragma unroll
    for (int i = 0; i < 2; ++i) x.k[i] = x.v[i] = make_uint4(0, 0, 0, 0);
    if (!w.live()) return;
    const long long row = t0 + w.token();
    const uint4* kp = reinterpret_cast<const uint4*>(k + row * k_ld + x.head * D) + x.part;
    const uint4* vp = reinterpret_cast<const uint4*>(v + row * v_ld + x.head * D) + x.part;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      x.k[i] = __ldcs(kp + i * L);
      x.v[i] = __ldcs(vp + i * L);
    }
  };
  Piece x;
  load(x);
  if (threadIdx.x < 32) find_places(c, bt, t0, count, place);
  __syncthreads();
  while (w.more()) {
    const long long base = w.live() ? place[w.token()] : -1;
    w.next();
    Piece next;
    load(next);
    const long long at = base + ((long long)x.head << c.page_shift);
    if constexpr (!Q) {
      if (base >= 0) {
        uint4* kp = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(c.k) + at * D) + x.part;
        uint4* vp = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(c.v) + at * D) + x.part;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          kp[i * L] = x.k[i];
          vp[i * L] = x.v[i];
        }
      }
    } else {
      uint32_t top = top_of(x.k) | (top_of(x.v) << 16);      // both vectors' in one word
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, o));
      if (base >= 0) {
        const int kb = scale_byte(top & 0xffffu), vb = scale_byte(top >> 16);
        uint2* kp = reinterpret_cast<uint2*>(static_cast<uint8_t*>(c.k) + at * D) + x.part;
        uint2* vp = reinterpret_cast<uint2*>(static_cast<uint8_t*>(c.v) + at * D) + x.part;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          kp[i * L] = quantise8(x.k[i], kb);
          vp[i * L] = quantise8(x.v[i], vb);
        }
        if (x.part == 0) {
          c.ks[at] = (uint8_t)kb;
          c.vs[at] = (uint8_t)vb;
        }
      }
    }
    x = next;
  }
}

template <int D, bool Q>
__global__ void __launch_bounds__(256) read_kernel(const KvView c, const KvBatchView bt, int tokens,
                                                   __nv_bfloat16* __restrict__ k,
                                                   __nv_bfloat16* __restrict__ v) {
  constexpr int L = D / 16;
  __shared__ long long place[kMostTokens];
  const int t0 = blockIdx.x * tokens, count = min(tokens, bt.total - t0);
  Walk w(c.H * L, count);
  pdl_begin();
  if (threadIdx.x < 32) find_places(c, bt, t0, count, place);
  __syncthreads();
  // what a piece is loaded as: bf16, or codes and the scale bytes
  using Raw = typename std::conditional<Q, uint2, uint4>::type;
  struct Piece {
    Raw k[2], v[2];
    uint32_t kb, vb;
  };
  auto load = [&](Piece& x) {
#pragma unroll
    for (int i = 0; i < 2; ++i) x.k[i] = x.v[i] = Raw{};
    x.kb = x.vb = 0;
    const long long base = w.live() ? place[w.token()] : -1;
    if (base < 0) return;
    const int p = w.piece();
    const long long at = base + ((long long)(p / L) << c.page_shift);
    const Raw* kp = reinterpret_cast<const Raw*>(static_cast<const uint8_t*>(c.k) + at * (D * (Q ? 1 : 2))) + p % L;
    const Raw* vp = reinterpret_cast<const Raw*>(static_cast<const uint8_t*>(c.v) + at * (D * (Q ? 1 : 2))) + p % L;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      x.k[i] = __ldcs(kp + i * L);
      x.v[i] = __ldcs(vp + i * L);
    }
    if constexpr (Q) {
      x.kb = c.ks[at];
      x.vb = c.vs[at];
    }
  };
  Piece x;
  load(x);
  while (w.more()) {
    const bool live = w.live();
    const int p = w.piece();
    const long long o = ((long long)(t0 + w.token()) * c.H + p / L) * (2 * L) + p % L;
    w.next();
    Piece next;
    load(next);
    if (live) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint4 ky, vy;
        if constexpr (Q) {                     // (codes 0 and byte 0 give zeros)
          ky = dequant8(x.k[i], x.kb);
          vy = dequant8(x.v[i], x.vb);
        } else {
          ky = x.k[i];
          vy = x.v[i];
        }
        __stcs(reinterpret_cast<uint4*>(k) + o + i * L, ky);
        __stcs(reinterpret_cast<uint4*>(v) + o + i * L, vy);
      }
    }
    x = next;
  }
}

template <typename... KArgs, typename... Args>
int launch(void (*kern)(KArgs...), int blocks, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

// Tokens of a CTA: one run of 32 pieces for each warp, more (up to eight) where that leaves the SMs
// their fill of CTAs.  (96 tokens of 8 x 128, 8-bit: 6.5 us so, 8.5 us with eight tokens a CTA.)
int tokens_per_cta(const KvView& c, const KvBatchView& bt) {
  const int width = c.H * (c.D / 16);
  const int side = width < 32 && 32 % width == 0 ? 32 / width : 1, turns = (width + 31) / 32;
  int t = side * (turns < 8 ? 8 / turns : 1);
  const long long most = (long long)t * 8;
  while (t < kMostTokens && 2LL * t <= most && bt.total > 2048LL * t) t *= 2;
  return t < kMostTokens ? t : kMostTokens;
}

}  // namespace

int launch_kv_append(const KvView& c, const KvBatchView& bt, const void* k, long long k_ld,
                     const void* v, long long v_ld, cudaStream_t stream) {
  const auto* kp = static_cast<const __nv_bfloat16*>(k);
  const auto* vp = static_cast<const __nv_bfloat16*>(v);
  const int tokens = tokens_per_cta(c, bt), blocks = (bt.total + tokens - 1) / tokens;
#define GDN_RUN(DD)                                                                                \
  return c.ks ? launch(append_kernel<DD, true>, blocks, stream, c, bt, tokens, kp, k_ld, vp, v_ld) \
              : launch(append_kernel<DD, false>, blocks, stream, c, bt, tokens, kp, k_ld, vp, v_ld)
  if (c.D == 64) GDN_RUN(64);
  if (c.D == 128) GDN_RUN(128);
  GDN_RUN(256);
#undef GDN_RUN
}

int launch_kv_read(const KvView& c, const KvBatchView& bt, void* k, void* v, cudaStream_t stream) {
  auto* kp = static_cast<__nv_bfloat16*>(k);
  auto* vp = static_cast<__nv_bfloat16*>(v);
  const int tokens = tokens_per_cta(c, bt), blocks = (bt.total + tokens - 1) / tokens;
#define GDN_RUN(DD)                                                                    \
  return c.ks ? launch(read_kernel<DD, true>, blocks, stream, c, bt, tokens, kp, vp)   \
              : launch(read_kernel<DD, false>, blocks, stream, c, bt, tokens, kp, vp)
  if (c.D == 64) GDN_RUN(64);
  if (c.D == 128) GDN_RUN(128);
  GDN_RUN(256);
#undef GDN_RUN
}

}  // namespace gdn
