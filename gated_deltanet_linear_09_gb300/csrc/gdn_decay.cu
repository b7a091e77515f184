// gdn_decay.cu -- linear attention with a decay for each head, token by token.
//
//   S_t = e^g S_(t-1) + k v^T,   o_t = scale S_t^T q
//
// A step reads and writes every state once (8 dk dv bytes) for 4 dk dv flops: the floor is the bytes.  The
// columns of a state are independent, so a CTA takes CW of one state's dv columns, all dk rows: its
// threads hold them in registers from the first load to the last store, whatever the number of tokens, and
// the sum over the rows is the only thing that meets in shared memory.  64 rows of 48 heads of 128 x 128: 60.5 us,
// 6.7 TB/s, 98 % of a copy.  From some four tokens on the instructions are the longer part (256 rows of 32 heads:
// 2 tokens 158 us, 8 tokens 224), so sums go two elements at a time and vectors are loaded 8 at a time (317).
#include "gdn_internal.h"

namespace gdn {

namespace {

constexpr int kThreads = 256;
constexpr int kBlock = GDN_MAX_DECODE_TOKENS;     // tokens whose vectors are held at a time

struct StepArgs {
  DecayView l;
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  const float* g;
  __nv_bfloat16* out;
  long long q_ld, k_ld, v_ld, g_ld;
  const int32_t* slots;
  int T;
};

// (x, y) += f * (a, b)
__device__ __forceinline__ void add_product(float& x, float& y, float f, float a, float b) {
  float u = f, w = f;
  fma_pair(u, w, a, b, x, y);
  x = u;
  y = w;
}

template <int DK, int DV, int CW>
__global__ void __launch_bounds__(kThreads) step_kernel(const StepArgs a) {
  constexpr int LPR = CW / 4;                // lanes (of float4) to a row
  constexpr int R = kThreads / LPR;          // rows at a time
  constexpr int N = DK / R;                  // rows of a thread
  static_assert(DK % R == 0, "rows of a thread");
  constexpr int SUMS = R < 8 ? R : 8;        // partial sums that meet: a warp's rows are added by shuffles
  __shared__ __align__(16) float qs[kBlock][DK], ks[kBlock][DK], vs[kBlock][CW], sums[kBlock][SUMS][CW];
  __shared__ float gs[kBlock];
  const int tid = threadIdx.x, row = blockIdx.z, h = blockIdx.y, c0 = blockIdx.x * CW;
  const int r0 = tid / LPR, c = (tid % LPR) * 4;
  pdl_begin();
  const long long t0 = (long long)row * a.T;
  const int slot = __ldg(a.slots + row);
  if (tid == 0 && slot >= a.l.num_slots) set_status(a.l.status, GDN_STATUS_SLOT_RANGE);
  const int hk = h / (a.l.Hv / a.l.Hk);
  if (slot < 0 || slot >= a.l.num_slots) {
    for (int i = tid; i < a.T * CW; i += kThreads)
      a.out[((t0 + i / CW) * a.l.Hv + h) * DV + c0 + i % CW] = __float2bfloat16_rn(0.f);
    return;
  }
  float* state = a.l.state + ((long long)slot * a.l.Hv + h) * (DK * DV) + c0;
  float4 s[N];
#pragma unroll
  for (int i = 0; i < N; ++i)
    s[i] = __ldcs(reinterpret_cast<const float4*>(state + (size_t)(r0 + i * R) * DV + c));
  // vectors of 8: queries, keys and values of all tokens
  constexpr int KV = DK / 8, VV = CW / 8;
  for (int i = tid; i < a.T * (2 * KV + VV); i += kThreads) {
    const int t = i / (2 * KV + VV), p = i % (2 * KV + VV);
    const bool q = p < KV, k = !q && p < 2 * KV;
    const int d = (q ? p : k ? p - KV : p - 2 * KV) * 8;
    const __nv_bfloat16* src = q ? a.q + (t0 + t) * a.q_ld + hk * DK : k ? a.k + (t0 + t) * a.k_ld + hk * DK
                                                                      : a.v + (t0 + t) * a.v_ld + h * DV + c0;
    float* dst = q ? qs[t] : k ? ks[t] : vs[t];
    const uint4 u = *reinterpret_cast<const uint4*>(src + d);
    const float f = q ? a.l.scale : 1.f;
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; e += 2)
      *reinterpret_cast<float4*>(dst + d + 2 * e) =
          make_float4(__uint_as_float(w[e] << 16) * f, __uint_as_float(w[e] & 0xffff0000u) * f,
                      __uint_as_float(w[e + 1] << 16) * f, __uint_as_float(w[e + 1] & 0xffff0000u) * f);
  }
  if (tid < a.T) gs[tid] = expf(__ldg(a.g + (t0 + tid) * a.g_ld + h));
  __syncthreads();
  for (int t = 0; t < a.T; ++t) {
    const float e = gs[t];
    const float4 v = *reinterpret_cast<const float4*>(&vs[t][c]);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (e == 0.f) {                  // a decay of zero empties the state whatever it held
#pragma unroll
      for (int i = 0; i < N; ++i) s[i] = o;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float k = ks[t][r0 + i * R], q = qs[t][r0 + i * R];
      mul_pair(s[i].x, s[i].y, e, e);
      mul_pair(s[i].z, s[i].w, e, e);
      add_product(s[i].x, s[i].y, k, v.x, v.y);
      add_product(s[i].z, s[i].w, k, v.z, v.w);
      add_product(o.x, o.y, q, s[i].x, s[i].y);
      add_product(o.z, o.w, q, s[i].z, s[i].w);
    }
#pragma unroll
    for (int m = LPR; m < 32; m <<= 1) {
      o.x += __shfl_xor_sync(0xffffffffu, o.x, m);
      o.y += __shfl_xor_sync(0xffffffffu, o.y, m);
      o.z += __shfl_xor_sync(0xffffffffu, o.z, m);
      o.w += __shfl_xor_sync(0xffffffffu, o.w, m);
    }
    if ((tid & 31) < LPR) *reinterpret_cast<float4*>(&sums[t][tid >> 5][c]) = o;
  }
  __syncthreads();
  for (int i = tid; i < a.T * CW; i += kThreads) {
    const int t = i / CW, d = i % CW;
    float o = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) o += sums[t][w][d];
    a.out[((long long)(t0 + t) * a.l.Hv + h) * DV + c0 + d] = __float2bfloat16_rn(o);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) __stcs(reinterpret_cast<float4*>(state + (size_t)(r0 + i * R) * DV + c), s[i]);
}

template <int DK, int DV, int CW>
int launch_cols(const StepArgs& a, int rows, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(DV / CW, (unsigned)a.l.Hv, (unsigned)rows);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, step_kernel<DK, DV, CW>, a) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

// 64 columns: with 128 the batch above takes 62.0 us, 8 tokens 244; with 32 60.5 and 288, states of 64 x 128 91 for 80.
template <int DK, int DV>
int launch_dims(const StepArgs& a, int rows, cudaStream_t stream) {
  return launch_cols<DK, DV, 64>(a, rows, stream);
}

int launch_rows(const StepArgs& a, int rows, cudaStream_t stream) {
  if (a.l.dk == 128) return a.l.dv == 128 ? launch_dims<128, 128>(a, rows, stream) : launch_dims<128, 64>(a, rows, stream);
  return a.l.dv == 128 ? launch_dims<64, 128>(a, rows, stream) : launch_dims<64, 64>(a, rows, stream);
}

StepArgs step_args(const DecayView& l, const gdn_decay_tokens& t) {
  StepArgs a = {};
  a.l = l;
  a.q = static_cast<const __nv_bfloat16*>(t.q);
  a.k = static_cast<const __nv_bfloat16*>(t.k);
  a.v = static_cast<const __nv_bfloat16*>(t.v);
  a.g = t.log_decay;
  a.out = static_cast<__nv_bfloat16*>(t.out);
  a.q_ld = t.q_ld;
  a.k_ld = t.k_ld;
  a.v_ld = t.v_ld;
  a.g_ld = t.decay_ld;
  return a;
}

}  // namespace

int launch_decay_step(const DecayView& l, const gdn_decay_tokens& t, const int32_t* slot_idx, int B, int T,
                      cudaStream_t stream) {
  StepArgs a = step_args(l, t);
  a.slots = slot_idx;
  a.T = T;
  return launch_rows(a, B, stream);
}

}  // namespace gdn
