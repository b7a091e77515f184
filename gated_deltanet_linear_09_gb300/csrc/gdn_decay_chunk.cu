// gdn_decay_chunk.cu -- linear attention with a decay for each head over whole prompts, on the tcgen05 tensor
// cores in chunks of 128 tokens.
//
// With G_i the sum of the chunk's log decays up to token i, S the state before the chunk:
//   o_i = scale ( e^G_i S^T q_i + sum_{j <= i} e^(G_i - G_j) (q_i . k_j) v_j )
//   S  <- e^G_C S + sum_j e^(G_C - G_j) k_j v_j^T
// Five matrix products a chunk: scores Q K^T, their product with V, Q with the state, and the state's update
// twice, as the decayed keys are two bf16 parts (exact to 2^-16; the state is an f32 result).
//
// The chunks of all heads of all sequences, laid end to end, form one line (a constant per sequence and
// head beside its chunks), and CTA w of G takes the w-th of G equal pieces: long and short prompts, many heads
// or one, are balanced alike with no plan from the host.  Where pieces cut a sequence, three kernels: the
// first sums up what each cut piece adds to the state (its keys weighted to the piece's end, so nothing is
// rescaled), the second chains these along the pieces, the third computes the outputs, each piece from the
// state it begins with.
#include <math.h>

#include "gdn_internal.h"
#include "gdn_tmap.h"

namespace gdn {

using namespace tc;

namespace {

constexpr int kC = 128;               // tokens of a chunk
constexpr int kRunCost = 4, kChunkCost = 4;   // the line's units: beginning and ending a run, a chunk of it
constexpr int kLeast = 16;            // units of a piece at least (whole chunks in every piece of a long run)
constexpr int kRing = 4;              // runs known ahead
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLowest = -105.f;     // exp of it is 0 in f32

struct ChunkArgs {
  DecayView l;
  const float* g;
  long long g_ld;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  long long k_ld, v_ld;
  __nv_bfloat16* out;
  const int32_t* cu;
  const int32_t* slots;
  const uint8_t* init;
  // [grid] states of the pieces' ends, [grid] states that cut runs began with (the slot is written by the run's
  // last piece, whenever that comes to it), [grid] log2 decays, [grid] flags
  float* ws;
  float log2_scale;
  int num_seqs, total, grid;
};

struct Maps {
  CUtensorMap q, k, v;
};

// A piece's share of one head of one sequence: chunks [c0, c1) of n.
struct Run {
  int t0, len, head, slot, c0, c1, n, kind, init;
};
enum { kEnd = 0, kRun = 1, kZeros = 2 };      // no more runs; a run; one without a usable slot

// ------------------------------------------------------------------ the line

struct Line {
  long long x0, x1;       // this piece
  int pieces;
};

__device__ __forceinline__ int chunks_of(int len) { return (len + kC - 1) / kC; }
__device__ __forceinline__ long long head_cost(int len) { return kRunCost + (long long)kChunkCost * chunks_of(len); }
// chunks of a run before offset o
__device__ __forceinline__ int chunk_at(long long o, int n) {
  const long long c = (o - kRunCost + kChunkCost - 1) / kChunkCost;
  return o <= kRunCost ? 0 : c < n ? (int)c : n;
}

struct Walk {
  const ChunkArgs* a;
  long long x0, x1, r0;    // the piece, and the current run's place on the line
  int s, h, t0, len, slot, init;

  __device__ __forceinline__ void load() {
    t0 = __ldg(a->cu + s);
    len = __ldg(a->cu + s + 1) - t0;
    slot = __ldg(a->slots + s);
    init = a->init != nullptr && __ldg(a->init + s) != 0;
  }
  // `into`: the place x of the line, as an offset into sequence `seq`
  __device__ __forceinline__ void start(const ChunkArgs& args, const Line& line, long long x, int seq, long long into) {
    a = &args;
    x0 = line.x0;
    x1 = line.x1;
    s = seq;
    load();
    h = (int)(into / head_cost(len));
    r0 = x - (into - h * head_cost(len));
  }
  // The piece's share of the current run.
  __device__ __forceinline__ Run here() const {
    const int n = chunks_of(len);
    const bool usable = slot >= 0 && slot < a->l.num_slots;
    return Run{t0, len, h, slot, chunk_at(x0 - r0, n), chunk_at(x1 - r0, n), n, usable ? kRun : kZeros, init};
  }
  // The next run with something to do in this piece.
  __device__ __forceinline__ bool next(Run* r) {
    while (r0 < x1) {
      const long long at = r0;
      *r = here();
      r0 += head_cost(len);
      if (++h == a->l.Hv) {
        h = 0;
        if (++s < a->num_seqs) load();
        else r0 = x1;
      }
      if (r->n == 0 ? at >= x0 : r->c1 > r->c0) return true;
    }
    return false;
  }
};

struct Scan {
  long long warp_sum[32];
  long long into;
  int seq;
};

// Cuts the line (all NT threads).  False: the ranges do not fit together.  sc->seq and sc->into: where this
// CTA's piece begins (END: its last unit).
template <int NT, bool END>
__device__ __forceinline__ bool locate(const ChunkArgs& a, int index, Line* line, Scan* sc) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.num_seqs + NT - 1) / NT, s0 = tid * per, s1 = min(a.num_seqs, s0 + per);
  long long sum = 0;
  bool wrong = tid == 0 && (__ldg(a.cu) != 0 || __ldg(a.cu + a.num_seqs) > a.total);
  for (int s = s0; s < s1; ++s) {
    const int len = __ldg(a.cu + s + 1) - __ldg(a.cu + s);
    wrong |= len < 0;
    sum += head_cost(max(len, 0)) * a.l.Hv;
  }
  long long incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 31) sc->warp_sum[warp] = incl;
  if (__syncthreads_or(wrong)) return false;
  long long total = 0;
  for (int w = 0; w < NT / 32; ++w) {
    if (w < warp) incl += sc->warp_sum[w];
    total += sc->warp_sum[w];
  }
  const long long most = total / kLeast;
  const int pieces = (int)(most < 1 ? 1 : most < a.grid ? most : a.grid);
  line->pieces = pieces;
  const long long each = total / pieces;
  const int more = (int)(total - each * pieces);
  line->x0 = each * index + min(index, more);
  line->x1 = each * (index + 1) + min(index + 1, more);
  if (index < pieces) {
    const long long x = END ? line->x1 - 1 : line->x0;
    long long at = incl - sum;
    if (at <= x && x < incl) {
      for (int s = s0; s < s1; ++s) {
        const long long c = head_cost(__ldg(a.cu + s + 1) - __ldg(a.cu + s)) * a.l.Hv;
        if (x < at + c) {
          sc->seq = s;
          sc->into = x - at;
          break;
        }
        at += c;
      }
    }
  }
  __syncthreads();
  return true;
}

// Zeros in tokens [begin, end), shared by the grid's CTAs.
__device__ __forceinline__ void zero_tokens(const ChunkArgs& a, long long begin, long long end) {
  const long long row = (long long)a.l.Hv * a.l.dv / 8, n = (end - begin) * row;
  uint4* p = reinterpret_cast<uint4*>(a.out) + begin * row;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (long long)gridDim.x * blockDim.x)
    p[i] = make_uint4(0, 0, 0, 0);
}

// ------------------------------------------------------------------ waits that give up

// The first wait that runs out marks the CTA dead and sets the status; from then on no wait blocks, no copy or
// product is issued, and every role runs through to the end of its loops.
__device__ __forceinline__ void wait_bar(uint64_t* bar, uint32_t parity, volatile int* dead, int32_t* status) {
  if (mbar_try_wait(bar, parity)) return;
  if (*dead == 0 && !mbar_wait(bar, parity)) {
    *dead = 1;
    set_status(status, GDN_STATUS_TIMEOUT);
  }
}

// ------------------------------------------------------------------ operands

constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);          // SBO, version, 128-byte swizzle
constexpr uint32_t kDescK = (16u >> 4) << 16;                                  // K-major: LBO unused
constexpr uint32_t kDescMN = ((128u * 128u) >> 4) << 16;                       // MN-major: 64-column blocks

__device__ __forceinline__ uint64_t desc(uint32_t saddr, uint32_t kind) {
  return ((uint64_t)kDescHi << 32) | (((saddr & 0x3FFFFu) >> 4) | kind);
}
// bf16 operands, A MN-major too (bit 15).
__host__ __device__ constexpr uint32_t idesc_bf16_mnmn(int M, int N) { return idesc_bf16_bmn(M, N) | (1u << 15); }

__device__ __forceinline__ float ex2f(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ float lo_f32(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f32(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
// Whether a pair of bf16 (magnitude bits, larger of several) holds an infinity or a NaN.
__device__ __forceinline__ bool not_finite(uint32_t m) { return (m & 0xffffu) >= 0x7f80u || (m >> 16) >= 0x7f80u; }
__device__ __forceinline__ void tmem_ld32_nw(uint32_t addr, uint32_t* r) {
  tmem_ld16_nw(addr, r);
  tmem_ld16_nw(addr + 16, r + 16);
}
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int x0, int x1, int x2, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];\n" ::"r"(
          smem_u32(dst)),
      "l"(map), "r"(smem_u32(bar)), "r"(x0), "r"(x1), "r"(x2)
      : "memory");
}

// A token's log decay, in log2 units.
__device__ __forceinline__ float decay_log2(const ChunkArgs& a, long long t, int h) {
  const float g = __ldg(a.g + t * a.g_ld + h);
  return (g < kLowest ? kLowest : g) * kLog2e;
}

// The decays of `rows` tokens from t on (a whole warp, lane = 4 tokens): up to and with each token, and of
// what follows each in the chunk plus `rest`, as a factor (0 past the rows).  Returns the chunk's sum.
__device__ __forceinline__ float chunk_decays(const ChunkArgs& a, int t, int rows, int h, float rest, float* upto,
                                              float* after) {
  const int lane = threadIdx.x & 31;
  float g[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int j = lane * 4 + e;
    g[e] = j < rows ? decay_log2(a, t + j, h) : 0.f;
  }
  const float own = (g[0] + g[1]) + (g[2] + g[3]);
  float up = own, down = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float u = __shfl_up_sync(0xffffffffu, up, o), d = __shfl_down_sync(0xffffffffu, down, o);
    if (lane >= o) up += u;
    if (lane + o < 32) down += d;
  }
  const float all = __shfl_sync(0xffffffffu, up, 31);
  float before = __shfl_up_sync(0xffffffffu, up, 1), behind = __shfl_down_sync(0xffffffffu, down, 1);
  if (lane == 0) before = 0.f;
  if (lane == 31) behind = 0.f;
  float4 p, w;
  p.x = before + g[0]; p.y = p.x + g[1]; p.z = p.y + g[2]; p.w = p.z + g[3];
  behind += rest;
  w.w = behind; w.z = w.w + g[3]; w.y = w.z + g[2]; w.x = w.y + g[1];
  w.x = lane * 4 + 0 < rows ? ex2f(w.x) : 0.f;
  w.y = lane * 4 + 1 < rows ? ex2f(w.y) : 0.f;
  w.z = lane * 4 + 2 < rows ? ex2f(w.z) : 0.f;
  w.w = lane * 4 + 3 < rows ? ex2f(w.w) : 0.f;
  if (upto) *reinterpret_cast<float4*>(upto + lane * 4) = p;
  *reinterpret_cast<float4*>(after + lane * 4) = w;
  return all;
}

// Turns a K tile [DK / 64][128 rows][128 bytes], 128-byte swizzled, into the high parts of its rows times w, in
// place, and the low parts beside it.  NT threads, this one the t-th.
template <int DK, int NT>
__device__ __forceinline__ void split_keys(uint8_t* k, uint8_t* lo, const float* w, int t) {
#pragma unroll 4
  for (int i = 0; i < DK * kC / 8 / NT; ++i) {
    const int at = i * NT + t;
    const float f = w[(at >> 3) & (kC - 1)];
    uint4* p = reinterpret_cast<uint4*>(k) + at;
    const uint4 u = *p;
    const uint32_t x[4] = {u.x, u.y, u.z, u.w};
    uint32_t h[4], l[4], top = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float a = lo_f32(x[e]) * f, b = hi_f32(x[e]) * f;
      h[e] = pack2(a, b);
      l[e] = pack2(a - lo_f32(h[e]), b - hi_f32(h[e]));
      top = __vmaxu2(top, h[e] & 0x7fff7fffu);
    }
    if (f == 0.f) {
#pragma unroll
      for (int e = 0; e < 4; ++e) h[e] = l[e] = 0;      // (whatever the key)
    } else if (not_finite(top)) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {                      // no low part beside an infinity or a NaN
        if ((h[e] & 0x7f80u) == 0x7f80u) l[e] &= 0xffff0000u;
        if ((h[e] & 0x7f800000u) == 0x7f800000u) l[e] &= 0xffffu;
      }
    }
    *p = make_uint4(h[0], h[1], h[2], h[3]);
    reinterpret_cast<uint4*>(lo)[at] = make_uint4(l[0], l[1], l[2], l[3]);
  }
}

// Zeros in the place of a V tile's non-finite values and rows past the sequence; whether there were any of
// the former.
template <int BLOCKS, int NT>
__device__ __forceinline__ bool clean_values(uint8_t* v, int rows, int t) {
  bool bad = false;
#pragma unroll 4
  for (int i = 0; i < BLOCKS * 1024 / NT; ++i) {
    const int at = i * NT + t, row = (at >> 3) & (kC - 1);
    uint4* p = reinterpret_cast<uint4*>(v) + at;
    const uint4 u = *p;
    uint32_t x[4] = {u.x, u.y, u.z, u.w};
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) top = __vmaxu2(top, x[e] & 0x7fff7fffu);
    if (row >= rows) {
      *p = make_uint4(0, 0, 0, 0);
    } else if (not_finite(top)) {
      bad = true;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if ((x[e] & 0x7f80u) == 0x7f80u) x[e] &= 0xffff0000u;
        if ((x[e] & 0x7f800000u) == 0x7f800000u) x[e] &= 0xffffu;
      }
      *p = make_uint4(x[0], x[1], x[2], x[3]);
    }
  }
  return bad;
}

// Barrier over n threads that returns whether any of them passed true.
__device__ __forceinline__ bool bar_any(int id, int n, bool v) {
  uint32_t r;
  __syncwarp();
  asm volatile(
      "{\n.reg .pred p, q;\nsetp.ne.u32 p, %3, 0;\nbar.red.or.pred q, %1, %2, p;\nselp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"(id), "r"(n), "r"((uint32_t)v)
      : "memory");
  return r != 0;
}

// Which of the columns c .. c + 31 a value not finite of tokens t - back .. t has reached by token t.
__device__ __noinline__ uint32_t reached_columns(const ChunkArgs& a, long long t, int back, int head, int dv, int c) {
  uint32_t m = 0;
  float sum = 0.f;
  for (int j = 0; j <= back && ex2f(sum) != 0.f; ++j) {
    for (int e = 0; e < 32; ++e)
      if (!(fabsf(__bfloat162float(a.v[(t - j) * a.v_ld + head * dv + c + e])) < INFINITY)) m |= 1u << e;
    sum += decay_log2(a, t - j, head);
  }
  return m;
}

// What the non-finite values of column c among tokens [t, t + rows) add to N elements of the state's column from
// row d0 on: infinities and NaN, told apart as the recurrence does.
template <int N>
__device__ __noinline__ void add_non_finite(const ChunkArgs& a, long long t, int rows, int head, int dk, int dv, int c, int d0,
                                            float* s) {
  const int hk = head / (a.l.Hv / a.l.Hk);
  float sum = 0.f;
  for (int j = rows - 1; j >= 0; --j) {
    const float w = ex2f(sum);
    if (w == 0.f) break;
    const float v = __bfloat162float(a.v[(t + j) * a.v_ld + head * dv + c]);
    if (!(fabsf(v) < INFINITY))
      for (int e = 0; e < N; ++e) s[e] += __bfloat162float(a.k[(t + j) * a.k_ld + hk * dk + d0 + e]) * w * v;
    sum += decay_log2(a, t + j, head);
  }
}

template <typename... KArgs, typename... Args>
int launch(void (*kern)(KArgs...), dim3 grid, int threads, size_t smem, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

// A dv-by-dk state (transposed: a TMEM lane is a column of the state) as 128 threads hold it: lane r is
// column r, or for 64 columns column r % 64 and half of the rows.
template <int DK, int DV>
struct StateRows {
  static constexpr int kCols = DV == 128 ? DK : DK / 2;       // state rows of a thread
  static __device__ __forceinline__ int column(int r) { return r & (DV - 1); }
  static __device__ __forceinline__ int first(int r) { return DV == 128 ? 0 : (r >> 6) * kCols; }
};

// ------------------------------------------------------------------ what a cut piece adds to the state

template <int DK, int DV>
struct __align__(1024) SumSmem {
  uint8_t k[2][DK * kC * 2];
  uint8_t lo[2][DK * kC * 2];
  uint8_t v[2][128 * kC * 2];         // 64 columns twice, so that they fill the product's 128 rows
  float w[2][kC];
  Scan scan;
  Run run;
  float decay;
  uint32_t tmem;
  int dead, bad;
  uint64_t full[2], ready[2], empty[2], weights[2], done;
};

constexpr int kSumThreads = 320;      // two warpgroups that split keys, MMA, loader

template <int DK, int DV>
__global__ void __launch_bounds__(kSumThreads, 1) sum_kernel(const ChunkArgs a, const __grid_constant__ Maps maps) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  SumSmem<DK, DV>& sm = *reinterpret_cast<SumSmem<DK, DV>*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, piece = blockIdx.x;
  pdl_begin();
  float* decays = a.ws + 2 * (size_t)a.grid * (DK * DV);
  int* flags = reinterpret_cast<int*>(decays + a.grid);
  Line line;
  if (!locate<kSumThreads, true>(a, piece, &line, &sm.scan)) return;
  if (tid == 0) {
    // only the run that holds the piece's last unit can go on after it
    Run last = {};
    bool cut = false;
    if (piece < line.pieces) {
      Walk walk;
      walk.start(a, line, line.x1 - 1, sm.scan.seq, sm.scan.into);
      last = walk.here();
      cut = last.kind == kRun && last.c1 > last.c0 && last.c1 < last.n;
    }
    if (!cut) last.kind = kEnd;
    sm.run = last;
    flags[piece] = !cut ? 0 : last.c0 == 0 ? 1 : 2;
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.ready[i], 8);
      mbar_init(&sm.empty[i], 1);
      mbar_init(&sm.weights[i], 1);
    }
    mbar_init(&sm.done, 1);
    sm.dead = sm.bad = 0;
    mbar_fence_init();
  }
  __syncthreads();
  const Run run = sm.run;
  if (run.kind == kEnd) return;
  if (warp == 8) tmem_alloc(&sm.tmem, 128);
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = sm.tmem;
  const int n = run.c1 - run.c0;
  auto wait = [&](uint64_t* bar, uint32_t parity) { wait_bar(bar, parity, &sm.dead, a.l.status); };
  auto dead = [&]() { return *(volatile int*)&sm.dead != 0; };
  // chunks from the last to the first, so that each one's weights to the piece's end are known
  if (warp == 9) {
    const int hk = run.head / (a.l.Hv / a.l.Hk);
    float rest = 0.f;
    for (int i = 0; i < n; ++i) {
      const int st = i & 1, t = run.t0 + (run.c1 - 1 - i) * kC;
      if (i >= 2) wait(&sm.empty[st], ((i >> 1) & 1) ^ 1u);
      __syncwarp();
      if (lane == 0 && !dead()) {
        mbar_arrive_expect_tx(&sm.full[st], DK * kC * 2 + 128 * kC * 2);
        tma_load_3d(sm.k[st], &maps.k, 0, t, hk * (DK / 64), &sm.full[st]);
        tma_load_3d(sm.v[st], &maps.v, 0, t, run.head * (DV / 64), &sm.full[st]);
        if (DV == 64) tma_load_3d(sm.v[st] + 64 * kC * 2, &maps.v, 0, t, run.head, &sm.full[st]);
      }
      rest += chunk_decays(a, t, kC, run.head, rest, nullptr, sm.w[st]);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.weights[st]);
    }
    if (lane == 0) sm.decay = rest;
    // no copy outlives the CTA
    for (int i = max(0, n - 2); i < n; ++i) mbar_wait(&sm.full[i & 1], (i >> 1) & 1, 100000000ull);
  } else if (warp == 8) {
    if (lane == 0) {
      for (int i = 0; i < n && !dead(); ++i) {
        const int st = i & 1;
        wait(&sm.ready[st], (i >> 1) & 1);
        if (dead()) break;
        fence_after_sync();
        const uint64_t va = desc(smem_u32(sm.v[st]), kDescMN);
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          const uint64_t kb = desc(smem_u32(part ? sm.lo[st] : sm.k[st]), kDescMN);
#pragma unroll
          for (int ks = 0; ks < kC / 16; ++ks)
            mma_bf16(tmem, desc_add(va, ks * 2048), desc_add(kb, ks * 2048), idesc_bf16_mnmn(128, DK), i > 0 || part > 0 || ks > 0);
        }
        mma_commit(&sm.empty[st]);
      }
      mma_commit(&sm.done);
    }
    __syncwarp();
  } else {
    for (int i = 0; i < n; ++i) {
      const int st = i & 1;
      wait(&sm.weights[st], (i >> 1) & 1);
      wait(&sm.full[st], (i >> 1) & 1);
      __syncwarp();
      split_keys<DK, 256>(sm.k[st], sm.lo[st], sm.w[st], tid);
      if (clean_values<2, 256>(sm.v[st], kC, tid)) sm.bad = 1;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.ready[st]);
    }
  }
  __syncthreads();
  wait(&sm.done, 0);
  __syncthreads();
  fence_after_sync();
  if (warp < 4) {
    using L = StateRows<DK, DV>;
    const int c = L::column(tid), d0 = L::first(tid);
    const bool begins = run.c0 == 0 && run.init;        // with a state
    const float f = ex2f(sm.decay);
    float* kept = a.ws + (size_t)(a.grid + piece) * (DK * DV);
    const float* src = a.l.state + ((long long)run.slot * a.l.Hv + run.head) * (DK * DV);
    float* dst = a.ws + (size_t)piece * (DK * DV);
#pragma unroll
    for (int b = 0; b < L::kCols; b += 32) {
      uint32_t r[32];
      tmem_ld32_nw(tmem + ((uint32_t)(warp * 32) << 16) + d0 + b, r);
      tmem_wait_ld();
      reg_fence16(r);
      reg_fence16(r + 16);
      float s[32];
#pragma unroll
      for (int e = 0; e < 32; ++e) s[e] = __uint_as_float(r[e]);
      if (begins) {
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const float x = src[(d0 + b + e) * DV + c];
          kept[(d0 + b + e) * DV + c] = x;
          if (f != 0.f) s[e] = fmaf(f, x, s[e]);
        }
      }
      if (sm.bad) {
        float more[32];
        for (int e = 0; e < 32; ++e) more[e] = 0.f;
        add_non_finite<32>(a, run.t0 + run.c0 * kC, n * kC, run.head, DK, DV, c, d0 + b, more);
#pragma unroll
        for (int e = 0; e < 32; ++e) s[e] += more[e];
      }
#pragma unroll
      for (int e = 0; e < 32; ++e) dst[(d0 + b + e) * DV + c] = s[e];
    }
  }
  if (tid == 0) decays[piece] = sm.decay;
  fence_before_sync();
  __syncthreads();
  if (warp == 8) tmem_dealloc(tmem, 128);
}

// ------------------------------------------------------------------ along the pieces

// S_p <- e^g_p S_(p-1) + S_p over each run's pieces, 1,024 elements a CTA.
__global__ void __launch_bounds__(256) chain_kernel(const ChunkArgs a) {
  pdl_begin();
  const int size = a.l.dk * a.l.dv;
  const float* decays = a.ws + 2 * (size_t)a.grid * size;
  const int* flags = reinterpret_cast<const int*>(decays + a.grid);
  if (__ldcg(flags + blockIdx.x) != 1) return;
  float4* p = reinterpret_cast<float4*>(a.ws) + ((size_t)blockIdx.x * size / 4) + blockIdx.y * 256 + threadIdx.x;
  float4 s = __ldcg(p);
  for (int i = blockIdx.x + 1; i < a.grid && __ldcg(flags + i) == 2; ++i) {
    p += size / 4;
    float4 x = __ldcg(p);
    const float f = ex2f(__ldcg(decays + i));
    if (f != 0.f) {
      x.x = fmaf(f, s.x, x.x); x.y = fmaf(f, s.y, x.y);
      x.z = fmaf(f, s.z, x.z); x.w = fmaf(f, s.w, x.w);
    }
    __stcg(p, x);
    s = x;
  }
}

// ------------------------------------------------------------------ outputs

template <int DK, int DV>
struct __align__(1024) OutSmem {
  uint8_t q[DK * kC * 2];
  uint8_t k[2][DK * kC * 2];
  uint8_t v[2][128 * kC * 2];         // 64 columns twice, so that they fill the state product's 128 rows
  uint8_t state[DK * DV * 2];         // bf16 [DK / 64][DV rows][128 bytes]
  uint8_t lo[DK * kC * 2];
  float upto[2][kC], w[2][kC];
  Run runs[kRing];
  uint32_t tmem;
  int dead;
  int bad[2];
  uint64_t kv_full[2], kv_empty[2], g_full[2], q_full, q_empty, s_done, p_ready, st_ready, ks_ready, o_done, o_empty, g_done;
  uint64_t run_full[kRing], run_empty[kRing], drained;
};

constexpr int kOutThreads = 384;      // scores and outputs; keys and state; MMA, K and V loader, Q loader, runs
constexpr int kReaders = 11;

// TMEM columns: scores (their decayed bf16 form in the lower half), the two parts of the output, the state.
constexpr int kTmS = 0, kTmO = 128, kTmI = 256, kTmState = 384;

template <int DK, int DV>
__global__ void __launch_bounds__(kOutThreads, 1) out_kernel(const ChunkArgs a, const __grid_constant__ Maps maps) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  OutSmem<DK, DV>& sm = *reinterpret_cast<OutSmem<DK, DV>*>(smem_raw);
  Scan& scan = *reinterpret_cast<Scan*>(sm.lo);          // (before the roles begin)
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, piece = blockIdx.x;
  pdl_begin();
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.kv_full[i], 1);
      mbar_init(&sm.kv_empty[i], 1);
      mbar_init(&sm.g_full[i], 1);
    }
    mbar_init(&sm.q_full, 1);
    mbar_init(&sm.q_empty, 1);
    mbar_init(&sm.s_done, 1);
    mbar_init(&sm.p_ready, 4);
    mbar_init(&sm.st_ready, 4);
    mbar_init(&sm.ks_ready, 4);
    mbar_init(&sm.o_done, 1);
    mbar_init(&sm.o_empty, 4);
    mbar_init(&sm.g_done, 1);
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&sm.run_full[i], 1);
      mbar_init(&sm.run_empty[i], kReaders);
    }
    mbar_init(&sm.drained, 1);
    sm.dead = 0;
    mbar_fence_init();
  }
  Line line;
  if (!locate<kOutThreads, false>(a, piece, &line, &scan)) {
    if (tid == 0) set_status(a.l.status, GDN_STATUS_BAD_SEQLENS);
    zero_tokens(a, 0, a.total);
    return;
  }
  const int seq = scan.seq;
  const long long into = scan.into;
  zero_tokens(a, __ldg(a.cu + a.num_seqs), a.total);
  if (piece >= line.pieces) return;
  if (warp == 8) tmem_alloc(&sm.tmem, 512);
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = sm.tmem;
  auto wait = [&](uint64_t* bar, uint32_t parity) { wait_bar(bar, parity, &sm.dead, a.l.status); };
  auto wait_warp = [&](uint64_t* bar, uint32_t parity) {
    wait(bar, parity);
    __syncwarp();
  };
  auto dead = [&]() { return *(volatile int*)&sm.dead != 0; };
  auto warp_dead = [&]() { return __any_sync(0xffffffffu, dead()) != 0; };
  int ring = 0;
  uint32_t ring_phase = 0;
  // the next run of a role (a whole warp); kind kEnd when there is none
  auto next_run = [&]() -> Run {
    wait_warp(&sm.run_full[ring], ring_phase);
    Run r = sm.runs[ring];
    if (warp_dead()) r.kind = kEnd;
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.run_empty[ring]);
    if (++ring == kRing) { ring = 0; ring_phase ^= 1u; }
    return r;
  };
  auto arrive_warp = [&](uint64_t* bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };
  int n = 0;                          // chunks so far
  const int group = a.l.Hv / a.l.Hk;

  if (warp == 11) {
    // ---------------------------------------------------------------- runs
    Walk walk;
    walk.start(a, line, line.x0, seq, into);
    Run r;
    for (bool more = true; more;) {
      more = walk.next(&r);
      wait_warp(&sm.run_empty[ring], ring_phase ^ 1u);
      if (warp_dead()) break;
      if (lane == 0) {
        if (more && r.slot >= a.l.num_slots) set_status(a.l.status, GDN_STATUS_SLOT_RANGE);
        if (!more) r.kind = kEnd;
        sm.runs[ring] = r;
        mbar_arrive(&sm.run_full[ring]);
      }
      __syncwarp();
      if (++ring == kRing) { ring = 0; ring_phase ^= 1u; }
    }
  } else if (warp == 9) {
    // ---------------------------------------------------------------- keys, values, decays
    for (Run r = next_run(); r.kind != kEnd; r = next_run()) {
      if (r.kind != kRun) continue;
      const int hk = r.head / group;
      for (int c = r.c0; c < r.c1; ++c, ++n) {
        const int st = n & 1, t = r.t0 + c * kC;
        if (n >= 2) wait_warp(&sm.kv_empty[st], ((n >> 1) & 1) ^ 1u);
        if (lane == 0 && !dead()) {
          mbar_arrive_expect_tx(&sm.kv_full[st], DK * kC * 2 + 128 * kC * 2);
          tma_load_3d(sm.k[st], &maps.k, 0, t, hk * (DK / 64), &sm.kv_full[st]);
          tma_load_3d(sm.v[st], &maps.v, 0, t, r.head * (DV / 64), &sm.kv_full[st]);
          if (DV == 64) tma_load_3d(sm.v[st] + 64 * kC * 2, &maps.v, 0, t, r.head, &sm.kv_full[st]);
        }
        __syncwarp();
        chunk_decays(a, t, min(kC, r.len - c * kC), r.head, 0.f, sm.upto[st], sm.w[st]);
        arrive_warp(&sm.g_full[st]);
      }
    }
    for (int i = max(0, n - 2); i < n; ++i) mbar_wait(&sm.kv_full[i & 1], (i >> 1) & 1, 100000000ull);
  } else if (warp == 10) {
    // ---------------------------------------------------------------- queries
    for (Run r = next_run(); r.kind != kEnd; r = next_run()) {
      if (r.kind != kRun) continue;
      for (int c = r.c0; c < r.c1; ++c, ++n) {
        if (n >= 1) wait_warp(&sm.q_empty, (n & 1) ^ 1u);
        if (lane == 0 && !dead()) {
          mbar_arrive_expect_tx(&sm.q_full, DK * kC * 2);
          tma_load_3d(sm.q, &maps.q, 0, r.t0 + c * kC, r.head / group * (DK / 64), &sm.q_full);
        }
        __syncwarp();
      }
    }
    if (n > 0) mbar_wait(&sm.q_full, (n - 1) & 1, 100000000ull);
  } else if (warp == 8) {
    // ---------------------------------------------------------------- MMA (one thread)
    const uint64_t qd = desc(smem_u32(sm.q), kDescK), sd = desc(smem_u32(sm.state), kDescK);
    const uint64_t lod = desc(smem_u32(sm.lo), kDescMN);
    while (lane == 0) {
      wait(&sm.run_full[ring], ring_phase);
      const Run r = sm.runs[ring];
      mbar_arrive(&sm.run_empty[ring]);
      if (++ring == kRing) { ring = 0; ring_phase ^= 1u; }
      if (dead() || r.kind == kEnd) break;
      if (r.kind != kRun) continue;
      for (int c = r.c0; c < r.c1; ++c, ++n) {
        const int st = n & 1;
        const uint64_t kk = desc(smem_u32(sm.k[st]), kDescK), km = desc(smem_u32(sm.k[st]), kDescMN);
        const uint64_t vm = desc(smem_u32(sm.v[st]), kDescMN);
        wait(&sm.q_full, n & 1);
        wait(&sm.kv_full[st], (n >> 1) & 1);
        if (dead()) break;
        fence_after_sync();
        // scores (the product with the last chunk's, which holds these columns, was issued before)
#pragma unroll
        for (int ks = 0; ks < DK / 16; ++ks) {
          const uint32_t o = (ks >> 2) * (128 * kC) + (ks & 3) * 32;
          mma_bf16(tmem + kTmS, desc_add(qd, o), desc_add(kk, o), idesc_bf16(128, kC), ks > 0);
        }
        mma_commit(&sm.s_done);
        // queries and the state before the chunk
        wait(&sm.st_ready, n & 1);
        if (n > 0) wait(&sm.o_empty, (n & 1) ^ 1u);
        if (dead()) break;
        fence_after_sync();
#pragma unroll
        for (int ks = 0; ks < DK / 16; ++ks)
          mma_bf16(tmem + kTmI, desc_add(qd, (ks >> 2) * (128 * kC) + (ks & 3) * 32),
                   desc_add(sd, (ks >> 2) * (128 * DV) + (ks & 3) * 32), idesc_bf16(128, DV), ks > 0);
        mma_commit(&sm.q_empty);
        // the state's update, lanes = its columns
        wait(&sm.ks_ready, n & 1);
        if (dead()) break;
        fence_after_sync();
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
          for (int ks = 0; ks < kC / 16; ++ks)
            mma_bf16(tmem + kTmState, desc_add(vm, ks * 2048), desc_add(part ? lod : km, ks * 2048), idesc_bf16_mnmn(128, DK), 1);
        mma_commit(&sm.g_done);
        wait(&sm.p_ready, n & 1);
        if (dead()) break;
        fence_after_sync();
#pragma unroll
        for (int ks = 0; ks < kC / 16; ++ks)
          mma_bf16_tmem_a(tmem + kTmO, tmem + kTmS + ks * 8, desc_add(vm, ks * 2048), idesc_bf16_bmn(128, DV), ks > 0);
        mma_commit(&sm.o_done);
        mma_commit(&sm.kv_empty[st]);
      }
    }
    if (lane == 0) {                  // no product outlives the TMEM
      mma_commit(&sm.drained);
      mbar_wait(&sm.drained, 0, 100000000ull);
    }
    __syncwarp();
  } else if (warp < 4) {
    // ---------------------------------------------------------------- scores and outputs: a thread to a token
    const int i = tid;
    const uint32_t tl = tmem + ((uint32_t)(warp * 32) << 16);
    for (Run r = next_run(); r.kind != kEnd; r = next_run()) {
      if (r.kind == kZeros) {
        const int begin = r.c0 * kC, end = min(r.len, r.c1 * kC);
        for (int t = begin + i; t < end; t += 128)
          for (int d = 0; d < DV; d += 8)
            *reinterpret_cast<uint4*>(a.out + ((long long)(r.t0 + t) * a.l.Hv + r.head) * DV + d) = make_uint4(0, 0, 0, 0);
        continue;
      }
      for (int c = r.c0; c < r.c1; ++c, ++n) {
        const int st = n & 1, rows = min(kC, r.len - c * kC);
        wait_warp(&sm.g_full[st], (n >> 1) & 1);
        const float* upto = sm.upto[st];
        const float mine = upto[i] + a.log2_scale;
        wait_warp(&sm.s_done, n & 1);
        fence_after_sync();
#pragma unroll
        for (int b = 0; b < kC / 32; ++b) {
          uint32_t x[32], p[16];
          if (b > warp) {                                   // later tokens only
#pragma unroll
            for (int e = 0; e < 16; ++e) p[e] = 0;
          } else {
            tmem_ld32_nw(tl + kTmS + b * 32, x);
            tmem_wait_ld();
            reg_fence16(x);
            reg_fence16(x + 16);
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const float4 g = *reinterpret_cast<const float4*>(upto + b * 32 + e);
              const float gg[4] = {g.x, g.y, g.z, g.w};
              float y[4];
#pragma unroll
              for (int f = 0; f < 4; ++f) {
                y[f] = __uint_as_float(x[e + f]) * ex2f(mine - gg[f]);
                if (b == warp && b * 32 + e + f > i) y[f] = 0.f;
              }
              p[e / 2] = pack2(y[0], y[1]);
              p[e / 2 + 1] = pack2(y[2], y[3]);
            }
          }
          tmem_st16w_nw(tl + kTmS + b * 16, p);
        }
        tmem_wait_st();
        fence_before_sync();
        arrive_warp(&sm.p_ready);
        wait_warp(&sm.o_done, n & 1);
        fence_after_sync();
        const float f = ex2f(mine);
        const bool bad = *(volatile int*)&sm.bad[st] != 0;
        const long long t = r.t0 + c * kC + i;
        __nv_bfloat16* dst = a.out + (t * a.l.Hv + r.head) * DV;
#pragma unroll
        for (int b = 0; b < DV / 32; ++b) {
          uint32_t x[32], y[32];
          tmem_ld32_nw(tl + kTmO + b * 32, x);
          tmem_ld32_nw(tl + kTmI + b * 32, y);
          tmem_wait_ld();
          reg_fence16(x);
          reg_fence16(x + 16);
          reg_fence16(y);
          reg_fence16(y + 16);
          float o[32];
#pragma unroll
          for (int e = 0; e < 32; ++e)
            o[e] = f == 0.f ? __uint_as_float(x[e]) : fmaf(f, __uint_as_float(y[e]), __uint_as_float(x[e]));
          if (bad && i < rows) {
            const uint32_t m = reached_columns(a, t, i, r.head, DV, b * 32);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (m >> e & 1) o[e] = NAN;
          }
          if (i < rows) {
#pragma unroll
            for (int e = 0; e < 32; e += 8)
              *reinterpret_cast<uint4*>(dst + b * 32 + e) = make_uint4(pack2(o[e], o[e + 1]), pack2(o[e + 2], o[e + 3]),
                                                                       pack2(o[e + 4], o[e + 5]), pack2(o[e + 6], o[e + 7]));
          }
        }
        fence_before_sync();
        arrive_warp(&sm.o_empty);
      }
    }
  } else {
    // ---------------------------------------------------------------- keys and state: a thread to a state column
    using L = StateRows<DK, DV>;
    const int t = tid - 128, col = L::column(t), d0 = L::first(t);
    const uint32_t tl = tmem + kTmState + ((uint32_t)((warp - 4) * 32) << 16) + d0;
    constexpr long long kSize = DK * DV;
    // the state as the products have left it, with what its last chunk's non-finite values add
    auto held = [&](const Run& r, int c, bool bad, int b, float* s) {
      uint32_t x[32];
      tmem_ld32_nw(tl + b, x);
      tmem_wait_ld();
      reg_fence16(x);
      reg_fence16(x + 16);
#pragma unroll
      for (int e = 0; e < 32; ++e) s[e] = __uint_as_float(x[e]);
      if (bad) {
        float more[32];               // (a copy, so that s stays in registers)
        for (int e = 0; e < 32; ++e) more[e] = 0.f;
        add_non_finite<32>(a, r.t0 + c * kC, min(kC, r.len - c * kC), r.head, DK, DV, col, d0 + b, more);
#pragma unroll
        for (int e = 0; e < 32; ++e) s[e] += more[e];
      }
    };
    while (true) {
      const Run r = next_run();
      if (bar_any(1, 128, r.kind == kEnd)) break;         // (together: they meet in barriers)
      if (r.kind != kRun) continue;
      float* state = a.l.state + ((long long)r.slot * a.l.Hv + r.head) * kSize;
      const float* from = r.c0 > 0                ? a.ws + (size_t)(piece - 1) * kSize
                          : !r.init              ? nullptr
                          : r.c1 < r.n           ? a.ws + (size_t)(a.grid + piece) * kSize
                                                 : state;
      if (r.n == 0 && !r.init) {
        for (int e = 0; e < L::kCols; ++e) state[(d0 + e) * DV + col] = 0.f;
      }
      bool bad = false;               // the last chunk's values
      for (int c = r.c0; c < r.c1; ++c, ++n) {
        const int st = n & 1;
        if (c > r.c0) {
          wait_warp(&sm.g_done, (n & 1) ^ 1u);
          fence_after_sync();
        }
        wait_warp(&sm.g_full[st], (n >> 1) & 1);
        const float f = ex2f(sm.upto[st][kC - 1]);
#pragma unroll
        for (int b = 0; b < L::kCols; b += 32) {
          float s[32];
          if (c > r.c0) {
            held(r, c - 1, bad, b, s);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) s[e] = from ? __ldcg(from + (d0 + b + e) * DV + col) : 0.f;
          }
          uint8_t* row = sm.state + ((d0 + b) >> 6) * (128 * DV) + col * 128;
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            const int at = (((d0 + b) & 63) + e) >> 3;
            *reinterpret_cast<uint4*>(row + ((at ^ (col & 7)) << 4)) = make_uint4(
                pack2(s[e], s[e + 1]), pack2(s[e + 2], s[e + 3]), pack2(s[e + 4], s[e + 5]), pack2(s[e + 6], s[e + 7]));
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) s[e] = f == 0.f ? 0.f : s[e] * f;
          tmem_st16_nw(tl + b, s);
          tmem_st16_nw(tl + b + 16, s + 16);
        }
        tmem_wait_st();
        fence_before_sync();
        fence_proxy_async_smem();
        arrive_warp(&sm.st_ready);
        wait_warp(&sm.kv_full[st], (n >> 1) & 1);
        bad = clean_values<2, 128>(sm.v[st], min(kC, r.len - c * kC), t);
        wait_warp(&sm.s_done, n & 1);
        split_keys<DK, 128>(sm.k[st], sm.lo, sm.w[st], t);
        bad = bar_any(1, 128, bad);
        if (t == 0) sm.bad[st] = bad;
        fence_proxy_async_smem();
        arrive_warp(&sm.ks_ready);
      }
      if (r.c1 > r.c0) {
        wait_warp(&sm.g_done, (n & 1) ^ 1u);
        fence_after_sync();
        if (r.c1 == r.n) {
#pragma unroll
          for (int b = 0; b < L::kCols; b += 32) {
            float s[32];
            held(r, r.c1 - 1, bad, b, s);
#pragma unroll
            for (int e = 0; e < 32; ++e) state[(d0 + b + e) * DV + col] = s[e];
          }
        }
        fence_before_sync();
      }
    }
  }
  __syncthreads();
  if (warp == 8) tmem_dealloc(tmem, 512);
}

template <int DK, int DV>
int launch_dims(const ChunkArgs& a, const Maps& maps, cudaStream_t stream) {
  static_assert(sizeof(SumSmem<DK, DV>) <= 227 * 1024 && sizeof(OutSmem<DK, DV>) <= 227 * 1024, "shared memory of a block");
  static OncePerDevice once_sum, once_out;
  int rc;
  if ((rc = raise_smem(once_sum, sum_kernel<DK, DV>, sizeof(SumSmem<DK, DV>))) != GDN_OK) return rc;
  if ((rc = raise_smem(once_out, out_kernel<DK, DV>, sizeof(OutSmem<DK, DV>))) != GDN_OK) return rc;
  if ((rc = launch(sum_kernel<DK, DV>, dim3((unsigned)a.grid), kSumThreads, sizeof(SumSmem<DK, DV>), stream, a, maps)) != GDN_OK)
    return rc;
  if ((rc = launch(chain_kernel, dim3((unsigned)a.grid, DK * DV / 1024), 256, 0, stream, a)) != GDN_OK) return rc;
  return launch(out_kernel<DK, DV>, dim3((unsigned)a.grid), kOutThreads, sizeof(OutSmem<DK, DV>), stream, a, maps);
}

}  // namespace

size_t decay_prefill_ws_bytes(const DecayView& l, int, int) {
  const int sms = sm_count();
  const size_t grid = sms > 0 ? sms : 160;      // without a device (host-side sizing): at least the part's SMs
  return grid * (2 * (size_t)l.dk * l.dv * 4 + 8);
}

int launch_decay_prefill(const DecayView& l, const gdn_decay_tokens& t, const int32_t* cu_seqlens,
                         const int32_t* slot_idx, const uint8_t* has_init, int num_seqs, int total_tokens,
                         void* workspace, cudaStream_t stream) {
  ChunkArgs a = {};
  a.l = l;
  a.g = t.log_decay;
  a.g_ld = t.decay_ld;
  a.k = static_cast<const __nv_bfloat16*>(t.k);
  a.v = static_cast<const __nv_bfloat16*>(t.v);
  a.k_ld = t.k_ld;
  a.v_ld = t.v_ld;
  a.out = static_cast<__nv_bfloat16*>(t.out);
  a.cu = cu_seqlens;
  a.slots = slot_idx;
  a.init = has_init;
  a.ws = static_cast<float*>(workspace);
  a.log2_scale = log2f(l.scale);
  a.num_seqs = num_seqs;
  a.total = total_tokens;
  a.grid = sm_count();
  if (a.grid <= 0) return GDN_ERR_CUDA;
  Maps maps = {};
  if (total_tokens > 0 && !(make_rows_map(t.q, total_tokens, t.q_ld, l.Hk * l.dk, kC, l.dk / 64, &maps.q) &&
                            make_rows_map(t.k, total_tokens, t.k_ld, l.Hk * l.dk, kC, l.dk / 64, &maps.k) &&
                            make_rows_map(t.v, total_tokens, t.v_ld, l.Hv * l.dv, kC, l.dv / 64, &maps.v)))
    return GDN_ERR_CUDA;
  if (l.dk == 128) return l.dv == 128 ? launch_dims<128, 128>(a, maps, stream) : launch_dims<128, 64>(a, maps, stream);
  return l.dv == 128 ? launch_dims<64, 128>(a, maps, stream) : launch_dims<64, 64>(a, maps, stream);
}

}  // namespace gdn
