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
// or one, are balanced alike with no plan from the host.  Where pieces cut a sequence, a first kernel sums up what
// each cut piece adds to the state (its keys weighted to the piece's end, so nothing is rescaled), and the outputs'
// kernel starts each piece from its state: the sums of a run's pieces before it, which it adds up itself, or with few
// heads, where a run has many pieces, finds chained by a kernel between the two (a prompt of 16384 tokens of 6 heads 50
// us, without that kernel 54; 4096 of 32 heads 53, without it 52, before the checks below).  Runs that lie in one piece need no sums, and the
// outputs' kernel begins with them as soon as the sums' kernel leaves an SM.
//
// 4096 tokens of 32 heads of 128 x 128: 52.4 us, of which the sums take 15 and the outputs 33; 14 ragged prompts of 2924
// tokens, 448 runs in all: 62, and 8 more when the outputs waited for all sums.  A chunk takes the outputs 5,700 clocks:
// shared memory's bandwidth, 2,300 wavefronts of operands, 2,600 of the threads' accesses and some 1,000 of copies, of
// 128 bytes a clock.  (The tensor pipe is busy for 2,560 of them.)  A run of one chunk takes 9,300: the roles' steps one
// after another, as no chunk of the same run keeps them busy meanwhile.
//
// Fewer than 32 bits: the decayed scores and, for the outputs, the state are operands in bf16 (2^-8 of each at most, in
// f32 sums; more bits would take a second product each and shared memory that is not there), the decayed keys two bf16
// parts.  Tokens before one whose decay is 0 count nothing, whatever they hold, where scores and sums come out not finite
// too (looking for those takes 1 % of the time).
#include <math.h>

#include "gdn_internal.h"
#include "gdn_tmap.h"

namespace gdn {

using namespace tc;

namespace {

constexpr int kC = 128;               // tokens of a chunk
// The line's units: beginning and ending a run, the same of a run of one chunk, which does not wait for sums, and a
// chunk.  (The prompts above, before the looks for what is not finite: at 4, 1 52 and 61 us; at 3, 1 52 and 65; at 5, 1 52
// and 68; at 4, 2 52 and 62.)
constexpr int kRunCost = 4, kShortCost = 1, kChunkCost = 4;
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
  // last piece, whenever that comes to it), [grid] states that pieces begin with, [grid] log2 decays, [grid] flags
  float* ws;
  float log2_scale;
  int num_seqs, total, grid;
  int cut;                            // pieces may cut sequences: the sums come before the outputs
  int chained;                        // and a kernel that chains them; else each piece adds up what came before it
};

struct Maps {
  CUtensorMap q, k, v, out;
};

// A piece's share of one head of one sequence: chunks [c0, c1) of n.
struct Run {
  int t0, len, head, slot, c0, c1, n, kind, init;
  // chunk c is the first of a sequence that begins without a state
  __device__ __forceinline__ bool fresh(int c) const { return c == 0 && !init; }
};
enum { kEnd = 0, kRun = 1, kZeros = 2 };      // no more runs; a run; one without a usable slot

// ------------------------------------------------------------------ the line

struct Line {
  long long x0, x1;       // this piece
  int pieces;
};

__device__ __forceinline__ int chunks_of(int len) { return (len + kC - 1) / kC; }
__device__ __forceinline__ int run_cost(int n) { return n == 1 ? kShortCost : kRunCost; }
__device__ __forceinline__ long long head_cost(int len) {
  const int n = chunks_of(len);
  return run_cost(n) + (long long)kChunkCost * n;
}
// chunks of a run before offset o
__device__ __forceinline__ int chunk_at(long long o, int n) {
  const int begin = run_cost(n);
  const long long c = (o - begin + kChunkCost - 1) / kChunkCost;
  return o <= begin ? 0 : c < n ? (int)c : n;
}

// Where a place of the line lies: in which sequence, how far into it, and the sequence.
struct Found {
  long long into;
  int seq, t0, len, slot, init;
};

struct Walk {
  const ChunkArgs* a;
  long long x0, x1, r0;    // the piece, and the current run's place on the line
  int s, h, t0, len, slot, init;

  __device__ __forceinline__ void load() {
    t0 = __ldcg(a->cu + s);
    len = __ldcg(a->cu + s + 1) - t0;
    slot = __ldcg(a->slots + s);
    init = a->init != nullptr && __ldcg(a->init + s) != 0;
  }
  // from the place x of the line
  __device__ __forceinline__ void start(const ChunkArgs& args, const Line& line, long long x, const Found& at) {
    a = &args;
    x0 = line.x0;
    x1 = line.x1;
    s = at.seq;
    t0 = at.t0;
    len = at.len;
    slot = at.slot;
    init = at.init;
    h = (int)(at.into / head_cost(len));
    r0 = x - (at.into - h * head_cost(len));
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
  Line line;
  Found found;
  int end;              // the tokens of the sequences
  int wrong;
};

__device__ __forceinline__ Line cut_line(long long total, int grid, int index) {
  Line line;
  const long long most = total / kLeast;
  line.pieces = (int)(most < 1 ? 1 : most < grid ? most : grid);
  const long long each = total / line.pieces;
  const int more = (int)(total - each * line.pieces);
  line.x0 = each * index + min(index, more);
  line.x1 = each * (index + 1) + min(index + 1, more);
  return line;
}

// Cuts the line and finds where this CTA's piece begins (END: its last unit; all NT threads).  False: the
// ranges do not fit together.
template <int NT, bool END>
__device__ __forceinline__ bool locate(const ChunkArgs& a, int index, Scan* sc) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (a.num_seqs <= 32) {                 // one warp, all that it needs loaded at once
    if (warp == 0) {
      const bool on = lane < a.num_seqs;
      const int c0 = on ? __ldcg(a.cu + lane) : 0, c1 = on ? __ldcg(a.cu + lane + 1) : 0, slot = on ? __ldcg(a.slots + lane) : -1;
      const int init = on && a.init && __ldcg(a.init + lane) != 0;
      const bool wrong = (lane == 0 && c0 != 0) || c1 < c0 || c1 > a.total;
      const long long cost = on ? head_cost(c1 > c0 ? c1 - c0 : 0) * a.l.Hv : 0;
      long long incl = cost;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += u;
      }
      const Line line = cut_line(__shfl_sync(0xffffffffu, incl, 31), a.grid, index);
      const long long x = END ? line.x1 - 1 : line.x0, before = incl - cost;
      if (on && before <= x && x < incl) sc->found = Found{x - before, lane, c0, c1 - c0, slot, init};
      if (lane == a.num_seqs - 1) sc->end = c1;
      if (lane == 0) sc->line = line;
      const bool any = __any_sync(0xffffffffu, wrong);
      if (lane == 0) sc->wrong = any;
    }
    __syncthreads();
    return !sc->wrong;
  }
  const int per = (a.num_seqs + NT - 1) / NT, s0 = tid * per, s1 = min(a.num_seqs, s0 + per);
  long long sum = 0;
  bool wrong = tid == 0 && __ldcg(a.cu) != 0;
  for (int s = s0; s < s1; ++s) {
    const int c0 = __ldcg(a.cu + s), c1 = __ldcg(a.cu + s + 1);
    wrong |= c1 < c0 || c1 > a.total;
    sum += head_cost(c1 > c0 ? c1 - c0 : 0) * a.l.Hv;
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
  const Line line = cut_line(total, a.grid, index);
  if (tid == 0) {
    sc->line = line;
    sc->end = __ldcg(a.cu + a.num_seqs);
  }
  const long long x = END ? line.x1 - 1 : line.x0;
  long long at = incl - sum;
  if (at <= x && x < incl) {
    for (int s = s0; s < s1; ++s) {
      const int c0 = __ldcg(a.cu + s), len = __ldcg(a.cu + s + 1) - c0;
      const long long c = head_cost(len) * a.l.Hv;
      if (x < at + c) {
        sc->found = Found{x - at, s, c0, len, __ldcg(a.slots + s), a.init && __ldcg(a.init + s) != 0};
        break;
      }
      at += c;
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
// product is issued, and every role runs through to the end of its loops.  (Out of line, like all that is rare:
// the roles' code together has to fit the instruction caches.  With everything inlined and unrolled 38 % of
// the fetches missed, and the outputs of 4096 tokens of 32 heads took 59 us, so 33.)
__device__ __noinline__ void wait_long(uint64_t* bar, uint32_t parity, volatile int* dead, int32_t* status) {
  const long long t0 = clock64();
  while (*dead == 0) {
    // (asleep until the phase completes, or for some time: polling takes a part of shared memory's bandwidth)
    uint32_t ok;
    asm volatile(
        "{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\nselp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(100000u)
        : "memory");
    if (ok) return;
    if (clock64() - t0 > 4000000000ll) {            // two seconds
      *dead = 1;
      set_status(status, GDN_STATUS_TIMEOUT);
    }
  }
}
__device__ __forceinline__ void wait_bar(uint64_t* bar, uint32_t parity, volatile int* dead, int32_t* status) {
  if (!mbar_try_wait(bar, parity)) wait_long(bar, parity, dead, status);
}

// ------------------------------------------------------------------ operands

constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);          // SBO, version, 128-byte swizzle
constexpr uint32_t kDescK = (16u >> 4) << 16;                                  // K-major: LBO unused
constexpr uint32_t kDescMN = ((128u * 128u) >> 4) << 16;                       // MN-major: 64-column blocks

__device__ __forceinline__ uint32_t desc(uint32_t saddr, uint32_t kind) { return ((saddr & 0x3FFFFu) >> 4) | kind; }
// Products of operands whose descriptors' low words (the start address in sixteen-byte units, beside a
// constant) are these.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n.reg .pred p;\n.reg .b64 a, b;\nmov.b64 a, {%1, %5};\nmov.b64 b, {%2, %5};\nsetp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n}\n" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(acc), "n"(kDescHi)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n.reg .pred p;\n.reg .b64 b;\nmov.b64 b, {%2, %5};\nsetp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(idesc), "r"(acc), "n"(kDescHi)
      : "memory");
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
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
__device__ __forceinline__ bool any_nan(uint32_t w) { return (w & 0x7fffu) > 0x7f80u || (w & 0x7fff0000u) > 0x7f800000u; }
__device__ __forceinline__ bool finite_lo(uint32_t w) { return (w & 0x7f80u) != 0x7f80u; }
__device__ __forceinline__ bool finite_hi(uint32_t w) { return (w & 0x7f800000u) != 0x7f800000u; }
// Pairs of f32 in one instruction.
__device__ __forceinline__ void mul2(float& x, float& y, float f) {
  asm("{\n.reg .b64 a, b;\nmov.b64 a, {%0, %1};\nmov.b64 b, {%2, %2};\nmul.rn.f32x2 a, a, b;\nmov.b64 {%0, %1}, a;\n}\n"
      : "+f"(x), "+f"(y)
      : "f"(f));
}
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

__device__ __forceinline__ void tma_prefetch_3d(const CUtensorMap* map, int x0, int x1, int x2) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global [%0, {%1, %2, %3}];\n" ::"l"(map), "r"(x0), "r"(x1), "r"(x2) : "memory");
}

__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, int x0, int x1, int x2, const void* src) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];\n" ::"l"(map), "r"(x0), "r"(x1),
               "r"(x2), "r"(smem_u32(src))
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;\n" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;\n" ::: "memory"); }
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;\n" ::: "memory"); }

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];\n" ::"l"(p)); }

// A token's log decay, in log2 units.
__device__ __forceinline__ float decay_log2(const ChunkArgs& a, long long t, int h) {
  const float g = __ldcg(a.g + t * a.g_ld + h);
  return (g < kLowest ? kLowest : g) * kLog2e;
}

// A factor as the sum of two bf16 (exact to 2^-17), the larger in the low half.
__device__ __forceinline__ uint32_t two_parts(float w) {
  const __nv_bfloat16 hi = __float2bfloat16_rn(w);
  return pack2(w, w - __bfloat162float(hi));
}

// The log decays of `rows` tokens from t on, four to a lane (0 past the rows).
struct Decays {
  float g[4];
  __device__ __forceinline__ Decays(const ChunkArgs& a, int t, int rows, int h) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int j = lane * 4 + e;
      g[e] = j < rows ? decay_log2(a, t + j, h) : 0.f;
    }
  }
};

// Their sums (a whole warp): up to and with each token, and of what follows each in the chunk plus `rest`, as a factor
// in two parts (0 past the rows).  Returns the chunk's sum.
__device__ __forceinline__ float chunk_decays(const Decays& d, int rows, float rest, float* upto, uint32_t* after) {
  const int lane = threadIdx.x & 31;
  const float* g = d.g;
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
  *reinterpret_cast<uint4*>(after + lane * 4) = make_uint4(two_parts(w.x), two_parts(w.y), two_parts(w.z), two_parts(w.w));
  return all;
}

// Turns a K tile [DK / 64][128 rows][128 bytes], 128-byte swizzled, into the high parts of its rows times w, in
// place, and the low parts beside it.  NT threads, this one the t-th.  With w = w1 + w2 in bf16, all of it is
// bf16 arithmetic on pairs: h = k w1 rounded, k w1 - h exactly, and l = that plus k w2.  The factor of a 16-byte
// piece is its row's.
template <int DK, int NT>
__device__ __noinline__ void fix_split(uint8_t* k, uint8_t* lo, const uint32_t* w, int t) {
  // rows of weight 0 are 0 whatever the key; no low part beside an infinity or a NaN
  for (int at = t; at < DK * kC / 8; at += NT) {
    uint32_t* h = reinterpret_cast<uint32_t*>(k) + 4 * at;
    uint32_t* l = reinterpret_cast<uint32_t*>(lo) + 4 * at;
    const bool none = (w[(at >> 3) & (kC - 1)] & 0x7fffu) == 0;
    for (int e = 0; e < 4; ++e) {
      if (none) h[e] = l[e] = 0;
      if (!finite_lo(h[e])) l[e] &= 0xffff0000u;
      if (!finite_hi(h[e])) l[e] &= 0xffffu;
    }
  }
}
template <int DK, int NT>
__device__ __forceinline__ void split_keys(uint8_t* k, uint8_t* lo, const uint32_t* w, int t) {
  constexpr int kPer = DK * kC / 8 / NT;
  uint32_t sum = 0;                        // of the low parts: a NaN beside every key that is not finite
  uint4* kp = reinterpret_cast<uint4*>(k) + t;
  uint4* lp = reinterpret_cast<uint4*>(lo) + t;
  uint4 u = *kp;
  uint32_t f = w[(t >> 3) & (kC - 1)];
#pragma unroll 2
  for (int i = 0; i < kPer; ++i) {
    const int next = (i + 1 < kPer ? i + 1 : i) * NT;        // (ahead of the stores, which may alias it)
    const uint4 un = reinterpret_cast<const uint4*>(k)[next + t];
    const uint32_t fn = w[((next + t) >> 3) & (kC - 1)];
    const uint32_t w1 = __byte_perm(f, 0, 0x1010), w2 = __byte_perm(f, 0, 0x3232);
    const uint32_t x[4] = {u.x, u.y, u.z, u.w};
    uint32_t h[4], l[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      h[e] = mul_bf16x2(x[e], w1);
      l[e] = fma_bf16x2(x[e], w2, fma_bf16x2(x[e], w1, h[e] ^ 0x80008000u));
      sum = fma_bf16x2(l[e], 0, sum);
    }
    *kp = make_uint4(h[0], h[1], h[2], h[3]);
    *lp = make_uint4(l[0], l[1], l[2], l[3]);
    kp += NT;
    lp += NT;
    u = un;
    f = fn;
  }
  if (any_nan(sum)) fix_split<DK, NT>(k, lo, w, t);
}

// Zeros in the place of a V tile's non-finite values and rows past the sequence; whether there were any of
// the former.
template <int NT>
__device__ __noinline__ void clean_slowly(uint8_t* v, int t) {
  for (int at = t; at < 2048; at += NT) {
    uint32_t* x = reinterpret_cast<uint32_t*>(v) + 4 * at;
    for (int e = 0; e < 4; ++e) {
      if (!finite_lo(x[e])) x[e] &= 0xffff0000u;
      if (!finite_hi(x[e])) x[e] &= 0xffffu;
    }
  }
}
template <int NT>
__device__ __forceinline__ bool clean_values(uint8_t* v, int rows, int t) {
  uint32_t sum[4] = {0, 0, 0, 0};          // NaN with any value that is not finite
  constexpr int kBatch = 8;
#pragma unroll 1
  for (int i0 = 0; i0 < 2048 / NT; i0 += kBatch) {
    uint4 u[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int at = (i0 + i) * NT + t;    // (of a row past the sequence: row 0)
      u[i] = reinterpret_cast<const uint4*>(v)[((at >> 3) & (kC - 1)) < rows ? at : at & 7];
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      sum[0] = fma_bf16x2(u[i].x, 0, sum[0]);
      sum[1] = fma_bf16x2(u[i].y, 0, sum[1]);
      sum[2] = fma_bf16x2(u[i].z, 0, sum[2]);
      sum[3] = fma_bf16x2(u[i].w, 0, sum[3]);
    }
  }
  if (rows < kC)
    for (int block = 0; block < 2; ++block)
      for (int at = rows * 8 + t; at < 1024; at += NT) reinterpret_cast<uint4*>(v)[block * 1024 + at] = make_uint4(0, 0, 0, 0);
  const bool odd = any_nan(sum[0]) || any_nan(sum[1]) || any_nan(sum[2]) || any_nan(sum[3]);
  if (odd) clean_slowly<NT>(v, t);
  return odd;
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

// Byte of 16-byte piece `piece` of a row in an output tile [DV / 64][128 rows][128 bytes], 128-byte swizzled.
__device__ __forceinline__ int tile_at(int row, int piece) {
  return (piece >> 3) * (128 * kC) + row * 128 + (((piece & 7) ^ (row & 7)) << 4);
}

// NaN in those of `columns` columns from c on of an output tile's row that a value not finite of tokens
// t - row .. t has reached by token t.
__device__ __noinline__ void mark_reached(const ChunkArgs& a, long long t, int row, int head, int c, int columns, uint8_t* tile) {
  float sum = 0.f;
  for (int j = 0; j <= row && ex2f(sum) != 0.f; ++j) {
    for (int e = c; e < c + columns; ++e)
      if (!(fabsf(__bfloat162float(__ldcg(a.v + (t - j) * a.v_ld + head * a.l.dv + e))) < INFINITY))
        reinterpret_cast<__nv_bfloat16*>(tile + tile_at(row, e >> 3))[e & 7] = __float2bfloat16_rn(NAN);
    sum += decay_log2(a, t - j, head);
  }
}

// The first rows of an output tile (a sequence's last, when they are fewer than the tile's), by a warp.
template <int DV>
__device__ __noinline__ void store_rows(const ChunkArgs& a, int t, int rows, int head, const uint8_t* tile, int lane) {
  constexpr int kPieces = DV / 8, kStep = 32 / kPieces, kBatch = 8;
  const int piece = lane % kPieces;
  const long long ld = (long long)a.l.Hv * DV;
  __nv_bfloat16* out = a.out + ((long long)t * a.l.Hv + head) * DV + piece * 8;
  for (int row0 = lane / kPieces; row0 < rows; row0 += kStep * kBatch) {
    uint4 x[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) x[i] = *reinterpret_cast<const uint4*>(tile + tile_at(min(row0 + i * kStep, kC - 1), piece));
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (row0 + i * kStep < rows) *reinterpret_cast<uint4*>(out + (row0 + i * kStep) * ld) = x[i];
  }
}

// What the non-finite values of column c among tokens [t, t + rows) add to element d of the state's column: infinities
// and NaN, told apart as the recurrence does.  ALL: what all of its values add.
template <bool ALL>
__device__ __noinline__ float column_part(const ChunkArgs& a, long long t, int rows, int head, int c, int d) {
  const int hk = head / (a.l.Hv / a.l.Hk);
  float sum = 0.f, s = 0.f;
  for (int j = rows - 1; j >= 0; --j) {
    const float w = ex2f(sum);
    if (w != 0.f) {
      const float v = __bfloat162float(__ldcg(a.v + (t + j) * a.v_ld + head * a.l.dv + c));
      if (ALL || !(fabsf(v) < INFINITY)) s += __bfloat162float(__ldcg(a.k + (t + j) * a.k_ld + hk * a.l.dk + d)) * w * v;
    }
    sum += decay_log2(a, t + j, head);
  }
  return s;
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

// A dv-by-dk state (transposed: a TMEM lane is a column of the state) as eight warps hold it: lane r of the
// warps r / 32 and r / 32 + 4 is column r, half of the rows each, or for 64 columns column r % 64 and a quarter
// of the rows.
template <int DK, int DV>
struct StateRows {
  static constexpr int kRows = DK * DV / 256, kBlock = kRows < 16 ? kRows : 16;
  int lanes, column, first;
  __device__ __forceinline__ explicit StateRows(int t) {
    const int r = t & 127, half = t >> 7;
    lanes = r & ~31;
    column = r & (DV - 1);
    first = (DV == 128 ? half : (r >> 6) * 2 + half) * kRows;
  }
};

// kBlock columns of the lane's row.
template <int N>
__device__ __forceinline__ void tmem_row(uint32_t addr, float* s) {
  uint32_t x[N];
  if constexpr (N == 32) tmem_ld32_nw(addr, x);
  else tmem_ld16_nw(addr, x);
  tmem_wait_ld();
  reg_fence16(x);
  if constexpr (N == 32) reg_fence16(x + 16);
#pragma unroll
  for (int e = 0; e < N; ++e) s[e] = __uint_as_float(x[e]);
}

// ------------------------------------------------------------------ what a cut piece adds to the state

template <int DK, int DV>
struct __align__(1024) SumSmem {
  uint8_t k[2][DK * kC * 2];
  uint8_t lo[2][DK * kC * 2];
  uint8_t v[2][128 * kC * 2];         // 64 columns twice, so that they fill the product's 128 rows
  uint32_t w[2][kC];
  Scan scan;
  Run run;
  float decay;
  uint32_t tmem;
  int dead;
  uint64_t full[2], ready[2], empty[2], weights[2], done;
};

constexpr int kSumThreads = 320;      // two warpgroups that split keys, MMA, loader

template <int DK, int DV>
__global__ void __launch_bounds__(kSumThreads, 1) sum_kernel(const ChunkArgs a, const __grid_constant__ Maps maps) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  SumSmem<DK, DV>& sm = *reinterpret_cast<SumSmem<DK, DV>*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, piece = blockIdx.x;
  pdl_begin();
  float* decays = a.ws + 3 * (size_t)a.grid * (DK * DV);
  int* flags = reinterpret_cast<int*>(decays + a.grid);
  if (!locate<kSumThreads, true>(a, piece, &sm.scan)) return;
  if (tid == 0) {
    // only the run that holds the piece's last unit can go on after it
    Run last = {};
    bool cut = false;
    const Line line = sm.scan.line;
    if (piece < line.pieces) {
      Walk walk;
      walk.start(a, line, line.x1 - 1, sm.scan.found);
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
    sm.dead = 0;
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
      const Decays own(a, t, kC, run.head);                 // (on their way while the stage is waited for)
      if (i >= 2) wait(&sm.empty[st], ((i >> 1) & 1) ^ 1u);
      __syncwarp();
      if (lane == 0 && !dead()) {
        mbar_arrive_expect_tx(&sm.full[st], DK * kC * 2 + 128 * kC * 2);
        tma_load_3d(sm.k[st], &maps.k, 0, t, hk * (DK / 64), &sm.full[st]);
        tma_load_3d(sm.v[st], &maps.v, 0, t, run.head * (DV / 64), &sm.full[st]);
        if (DV == 64) tma_load_3d(sm.v[st] + 64 * kC * 2, &maps.v, 0, t, run.head, &sm.full[st]);
      }
      rest += chunk_decays(own, kC, rest, nullptr, sm.w[st]);
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
        const uint32_t va = desc(smem_u32(sm.v[st]), kDescMN);
#pragma unroll 1
        for (int part = 0; part < 2; ++part) {
          const uint32_t kb = desc(smem_u32(part ? sm.lo[st] : sm.k[st]), kDescMN);
#pragma unroll
          for (int ks = 0; ks < kC / 16; ++ks)
            mma_ss(tmem, va + ks * 128, kb + ks * 128, idesc_bf16_mnmn(128, DK), i > 0 || part > 0 || ks > 0);
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
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.ready[st]);
    }
  }
  __syncthreads();
  wait(&sm.done, 0);
  __syncthreads();
  fence_after_sync();
  if (warp < 8) {
    using L = StateRows<DK, DV>;
    constexpr int N = L::kBlock;
    const L at(tid);
    const bool begins = run.c0 == 0 && run.init;        // with a state
    const float f = ex2f(sm.decay);
    float* kept = a.ws + (size_t)(a.grid + piece) * (DK * DV) + at.column;
    const float* src = a.l.state + ((long long)run.slot * a.l.Hv + run.head) * (DK * DV) + at.column;
    float* dst = a.ws + (size_t)piece * (DK * DV) + at.column;
#pragma unroll 1
    for (int b = 0; b < L::kRows; b += N) {
      const int d = at.first + b;
      float s[N], x[N];
      if (begins) {
#pragma unroll
        for (int e = 0; e < N; ++e) x[e] = __ldcg(src + (d + e) * DV);
      }
      tmem_row<N>(tmem + ((uint32_t)at.lanes << 16) + d, s);
      if (begins) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
          kept[(d + e) * DV] = x[e];
          if (f != 0.f) s[e] = fmaf(f, x[e], s[e]);
        }
      }
      bool odd = false;
#pragma unroll
      for (int e = 0; e < N; ++e) {
        dst[(d + e) * DV] = s[e];
        odd |= !(fabsf(s[e]) < INFINITY);
      }
      // (a value that is not finite times a zero, which may be a part of a key or a key that a decay of zero has cut off:
      // such elements are summed again, from the tokens that do count)
      if (odd)
#pragma unroll 1
        for (int e = 0; e < N; ++e) {
          if (fabsf(__ldcg(dst + (d + e) * DV)) < INFINITY) continue;
          float x = column_part<true>(a, run.t0 + run.c0 * kC, n * kC, run.head, at.column, d + e);
          if (begins && f != 0.f) x = fmaf(f, __ldcg(src + (d + e) * DV), x);
          dst[(d + e) * DV] = x;
        }
    }
  }
  if (tid == 0) decays[piece] = sm.decay;
  fence_before_sync();
  __syncthreads();
  if (warp == 8) tmem_dealloc(tmem, 128);
}

// ------------------------------------------------------------------ along the pieces

// S_p <- e^g_p S_(p-1) + S_p over each run's pieces.  Every CTA reads which pieces begin a chain and how it goes on,
// takes its share of the chains (4,096 elements of one at a time), and loads the states ahead: the chain
// itself waits for no load.
constexpr int kChainThreads = 1024, kMostGrid = 1024;

__global__ void __launch_bounds__(kChainThreads) chain_kernel(const ChunkArgs a) {
  constexpr int kAhead = 6;
  __shared__ float decay[kMostGrid];
  __shared__ int flag[kMostGrid + 1], start[kMostGrid], before[33];
  pdl_begin();
  const int size = a.l.dk * a.l.dv, slices = size / 4096, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float* decays = a.ws + 3 * (size_t)a.grid * size;
  const int mine = tid < a.grid ? __ldcg(reinterpret_cast<const int*>(decays + a.grid) + tid) : 0;
  if (mine == 2) decay[tid] = ex2f(__ldcg(decays + tid));
  flag[tid] = mine;
  const uint32_t starts = __ballot_sync(0xffffffffu, mine == 1);
  if (lane == 0) before[warp] = __popc(starts);
  if (tid == 0) flag[kMostGrid] = 0;
  __syncthreads();
  if (warp == 0) {
    const int n = before[lane];
    int incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += u;
    }
    before[lane] = incl - n;
    if (lane == 31) before[32] = incl;
  }
  __syncthreads();
  if (mine == 1) start[before[warp] + __popc(starts & ((1u << lane) - 1u))] = tid;
  __syncthreads();
  for (int i = blockIdx.x; i < before[32] * slices; i += gridDim.x) {
    int piece = start[i / slices];
    float4* p = reinterpret_cast<float4*>(a.ws) + ((size_t)piece * size + (i % slices) * 4096) / 4 + tid;
    float4 s = __ldcg(p);
    while (flag[piece + 1] == 2) {
      float4 x[kAhead];
      int n = 0;
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        if (n == j && flag[piece + 1 + j] == 2) {
          x[j] = __ldcg(p + (size_t)(j + 1) * (size / 4));
          ++n;
        }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        if (j >= n) break;
        const float f = decay[++piece];
        p += size / 4;
        if (f != 0.f) {
          x[j].x = fmaf(f, s.x, x[j].x); x[j].y = fmaf(f, s.y, x[j].y);
          x[j].z = fmaf(f, s.z, x[j].z); x[j].w = fmaf(f, s.w, x[j].w);
        }
        s = x[j];
        __stcg(p, s);
      }
    }
  }
}

// The same for one piece that a run cut before it reaches: the state that it begins with, from the sums of the
// run's pieces before it (at most 32), by T threads of whole warps.
template <int SIZE, int T>
__device__ __noinline__ void carry(const ChunkArgs& a, int piece, int t) {
  constexpr int kSlots = SIZE / 4 / T;
  const int lane = t & 31;
  const float* decays = a.ws + 3 * (size_t)a.grid * SIZE;
  const int flag = lane < piece ? __ldcg(reinterpret_cast<const int*>(decays + a.grid) + piece - 1 - lane) : 0;
  const float mine = ex2f(lane < piece ? __ldcg(decays + piece - 1 - lane) : 0.f);
  const uint32_t first = __ballot_sync(0xffffffffu, flag == 1);
  int i = first ? __ffs(first) - 1 : 0;                       // pieces from the run's first to the last but one
  const float4* p = reinterpret_cast<const float4*>(a.ws) + (size_t)(piece - 1 - i) * (SIZE / 4) + t;
  float4 s[kSlots];
#pragma unroll
  for (int j = 0; j < kSlots; ++j) s[j] = __ldcg(p + j * T);
#pragma unroll 1
  while (--i >= 0) {
    const float f = __shfl_sync(0xffffffffu, mine, i);
    p += SIZE / 4;
#pragma unroll
    for (int j = 0; j < kSlots; ++j) {
      float4 x = __ldcg(p + j * T);
      if (f != 0.f) {
        x.x = fmaf(f, s[j].x, x.x); x.y = fmaf(f, s[j].y, x.y);
        x.z = fmaf(f, s[j].z, x.z); x.w = fmaf(f, s[j].w, x.w);
      }
      s[j] = x;
    }
  }
  float4* to = reinterpret_cast<float4*>(a.ws) + (size_t)(2 * a.grid + piece) * (SIZE / 4) + t;
#pragma unroll
  for (int j = 0; j < kSlots; ++j) __stcg(to + j * T, s[j]);
  __threadfence();
}

// ------------------------------------------------------------------ outputs

// The decayed scores of 32 columns (from `from` on) to `to`, for a warp of which some came out not finite: a token that a
// decay of zero keeps from this one counts nothing, whatever the score (a factor of zero would make it NaN).  `last`: the
// last column that the token sees.
__device__ __noinline__ void scores_slowly(uint32_t from, uint32_t to, const float* upto, float mine, int last) {
  uint32_t x[32], p[16];
  tmem_ld32_nw(from, x);
  tmem_wait_ld();
  reg_fence16(x);
  reg_fence16(x + 16);
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    const float f0 = e <= last ? ex2f(mine - upto[e]) : 0.f, f1 = e + 1 <= last ? ex2f(mine - upto[e + 1]) : 0.f;
    p[e / 2] = pack2(f0 != 0.f ? __uint_as_float(x[e]) * f0 : 0.f, f1 != 0.f ? __uint_as_float(x[e + 1]) * f1 : 0.f);
  }
  tmem_st16w_nw(to, p);
}

template <int DK, int DV>
struct __align__(1024) OutSmem {
  uint8_t q[DK * kC * 2];
  uint8_t k[2][DK * kC * 2];
  uint8_t v[2][128 * kC * 2];         // 64 columns twice, so that they fill the state product's 128 rows
  uint8_t state[DK * DV * 2];         // bf16 [DK / 64][DV rows][128 bytes]
  uint8_t lo[DK * kC * 2];
  float upto[2][kC];
  uint32_t w[2][kC];
  Run runs[kRing];
  uint32_t tmem;
  int dead;
  int bad[4];
  uint64_t k_full[2], v_full[2], v_ready[2], k_empty[2], v_empty[2], g_full[2], q_full, q_empty, s_done, p_ready, st_ready, ks_ready, o_done, o_empty, g_done, t_ready;
  uint64_t run_full[kRing], run_empty[kRing], drained;
};

// Eight warps for scores and outputs, eight for keys and state; MMA, K and V loader, runs, Q loader and check of V, outputs.
constexpr int kOutThreads = 640;
constexpr int kMmaWarp = 16, kLoadWarp = 17, kLoadQWarp = 18, kStoreWarp = 19;
constexpr int kReaders = 19;

// TMEM columns: scores (their decayed bf16 form in the lower half of each half), the two parts of the output, the state.
constexpr int kTmS = 0, kTmO = 128, kTmI = 256, kTmState = 384;

template <int DK, int DV>
__global__ void __launch_bounds__(kOutThreads, 1) out_kernel(const ChunkArgs a, const __grid_constant__ Maps maps) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  OutSmem<DK, DV>& sm = *reinterpret_cast<OutSmem<DK, DV>*>(smem_raw);
  Scan& scan = *reinterpret_cast<Scan*>(sm.lo);          // (before the roles begin)
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, piece = blockIdx.x;
  // After the sums or the chain only the states of cut runs depend on the kernel before this one: everything else begins
  // at once, beside it.  (That kernel let this one start when everything before this call was done and written back.
  // This one has not waited for that itself, which is what makes writes visible to all of its loads, so what it reads of
  // the call's inputs comes from L2, by tensor copies and loads past L1, whose lines may be from before.)
  if (!a.cut) pdl_wait_primary();
  pdl_launch_dependents();
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.k_full[i], 1);
      mbar_init(&sm.v_full[i], 1);
      mbar_init(&sm.k_empty[i], 1);
      mbar_init(&sm.v_empty[i], 1);
      mbar_init(&sm.v_ready[i], 1);
      mbar_init(&sm.g_full[i], 1);
    }
    mbar_init(&sm.q_full, 1);
    mbar_init(&sm.q_empty, 1);
    mbar_init(&sm.s_done, 1);
    mbar_init(&sm.p_ready, 8);
    mbar_init(&sm.st_ready, 8);
    mbar_init(&sm.ks_ready, 8);
    mbar_init(&sm.o_done, 1);
    mbar_init(&sm.o_empty, 8);
    mbar_init(&sm.t_ready, 8);
    mbar_init(&sm.g_done, 1);
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&sm.run_full[i], 1);
      mbar_init(&sm.run_empty[i], kReaders);
    }
    mbar_init(&sm.drained, 1);
    sm.dead = 0;
    mbar_fence_init();
  }
  if (!locate<kOutThreads, false>(a, piece, &scan)) {
    if (tid == 0) set_status(a.l.status, GDN_STATUS_BAD_SEQLENS);
    zero_tokens(a, 0, a.total);
    pdl_wait_primary();
    return;
  }
  const Line line = scan.line;
  const Found found = scan.found;
  zero_tokens(a, scan.end, a.total);
  if (piece >= line.pieces) {
    pdl_wait_primary();
    return;
  }
  if (warp == kMmaWarp) tmem_alloc(&sm.tmem, 512);
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
  // A run that was cut before this piece: the state that it begins with here.  (In front of the roles: called from
  // within them, it costs their loops registers, and the prompts above 53 and 64 us.)
  if (warp < kMmaWarp && a.cut && !a.chained) {
    Walk walk;
    walk.start(a, line, line.x0, found);
    const Run r = walk.here();
    if (r.kind == kRun && r.c0 > 0 && r.c1 > r.c0) {
      pdl_wait_primary();
      carry<DK * DV, 512>(a, piece, tid);
      bar_any(2, 512, false);
    }
  }

  if (warp == kStoreWarp) {
    // ---------------------------------------------------------------- outputs to memory
    for (Run r = next_run(); r.kind != kEnd; r = next_run()) {
      if (r.kind != kRun) continue;
      for (int c = r.c0; c < r.c1; ++c, ++n) {
        const int st = n & 1, rows = min(kC, r.len - c * kC);
        wait_warp(&sm.t_ready, n & 1);
        if (rows < kC) {
          store_rows<DV>(a, r.t0 + c * kC, rows, r.head, sm.v[st], lane);
          fence_proxy_async_smem();                         // (the next values come by the other proxy)
        } else if (lane == 0 && !dead()) {
          tma_store_3d(&maps.out, 0, r.t0 + c * kC, r.head * (DV / 64), sm.v[st]);
          bulk_commit();
          bulk_wait_read();
        }
        arrive_warp(&sm.v_empty[st]);
      }
    }
    if (lane == 0) bulk_wait();
  } else if (warp == kLoadWarp) {
    // ---------------------------------------------------------------- keys, values, decays
    for (Run r = next_run(); r.kind != kEnd; r = next_run()) {
      if (r.kind != kRun) continue;
      const int hk = r.head / group;
      for (int c = r.c0; c < r.c1; ++c, ++n) {
        const int st = n & 1, t = r.t0 + c * kC, rows = min(kC, r.len - c * kC);
        const Decays own(a, t, rows, r.head);               // (on their way while the stage is waited for)
        if (n >= 2) wait_warp(&sm.k_empty[st], ((n >> 1) & 1) ^ 1u);
        if (lane == 0 && !dead()) {
          mbar_arrive_expect_tx(&sm.k_full[st], DK * kC * 2);
          tma_load_3d(sm.k[st], &maps.k, 0, t, hk * (DK / 64), &sm.k_full[st]);
        }
        __syncwarp();
        chunk_decays(own, rows, 0.f, sm.upto[st], sm.w[st]);
        arrive_warp(&sm.g_full[st]);
        if (n >= 2) wait_warp(&sm.v_empty[st], ((n >> 1) & 1) ^ 1u);
        if (lane == 0 && !dead()) {
          mbar_arrive_expect_tx(&sm.v_full[st], 128 * kC * 2);
          tma_load_3d(sm.v[st], &maps.v, 0, t, r.head * (DV / 64), &sm.v_full[st]);
          if (DV == 64) tma_load_3d(sm.v[st] + 64 * kC * 2, &maps.v, 0, t, r.head, &sm.v_full[st]);
        }
        __syncwarp();
      }
    }
    for (int i = max(0, n - 2); i < n; ++i) {
      mbar_wait(&sm.k_full[i & 1], (i >> 1) & 1, 100000000ull);
      mbar_wait(&sm.v_full[i & 1], (i >> 1) & 1, 100000000ull);
    }
  } else if (warp == kLoadQWarp) {
    // ---------------------------------------------------------------- runs, one ahead, queries, check of the values
    Walk walk;
    walk.start(a, line, line.x0, found);
    auto publish = [&](Run* r) {
      if (!walk.next(r)) r->kind = kEnd;
      // the state that it begins with comes from DRAM: on its way to L2
      if (r->kind == kRun && r->c0 == 0 && r->c1 == r->n && r->init) {
        const float* state = a.l.state + ((long long)r->slot * a.l.Hv + r->head) * (DK * DV);
        for (int i = lane * 32; i < DK * DV; i += 32 * 32) prefetch_l2(state + i);
      }
      wait_warp(&sm.run_empty[ring], ring_phase ^ 1u);
      if (lane == 0 && !dead()) {
        if (r->kind != kEnd && r->slot >= a.l.num_slots) set_status(a.l.status, GDN_STATUS_SLOT_RANGE);
        sm.runs[ring] = *r;
        mbar_arrive(&sm.run_full[ring]);
      }
      __syncwarp();
      if (++ring == kRing) { ring = 0; ring_phase ^= 1u; }
    };
    Run r, ahead;
    publish(&r);
    while (r.kind != kEnd && !warp_dead()) {
      publish(&ahead);
      for (int c = r.c0; r.kind == kRun && c < r.c1; ++c, ++n) {
        if (n >= 1) wait_warp(&sm.q_empty, (n & 1) ^ 1u);
        if (lane == 0 && !dead()) {
          mbar_arrive_expect_tx(&sm.q_full, DK * kC * 2);
          tma_load_3d(sm.q, &maps.q, 0, r.t0 + c * kC, r.head / group * (DK / 64), &sm.q_full);
          // (one place for queries: the next ones wait in L2)
          if (c + 1 < r.c1) tma_prefetch_3d(&maps.q, 0, r.t0 + (c + 1) * kC, r.head / group * (DK / 64));
        }
        __syncwarp();
        // values that are not finite
        const int st = n & 1;
        wait_warp(&sm.v_full[st], (n >> 1) & 1);
        const bool bad = __any_sync(0xffffffffu, clean_values<32>(sm.v[st], min(kC, r.len - c * kC), lane));
        if (lane == 0) sm.bad[n & 3] = bad;
        fence_proxy_async_smem();
        arrive_warp(&sm.v_ready[st]);
      }
      r = ahead;
    }
    if (n > 0) mbar_wait(&sm.q_full, (n - 1) & 1, 100000000ull);
  } else if (warp == kMmaWarp) {
    // ---------------------------------------------------------------- MMA (one thread)
    const uint32_t qd = desc(smem_u32(sm.q), kDescK), sd = desc(smem_u32(sm.state), kDescK);
    const uint32_t lod = desc(smem_u32(sm.lo), kDescMN);
    while (lane == 0) {
      wait(&sm.run_full[ring], ring_phase);
      const Run r = sm.runs[ring];
      mbar_arrive(&sm.run_empty[ring]);
      if (++ring == kRing) { ring = 0; ring_phase ^= 1u; }
      if (dead() || r.kind == kEnd) break;
      if (r.kind != kRun) continue;
      for (int c = r.c0; c < r.c1; ++c, ++n) {
        const int st = n & 1;
        const uint32_t kk = desc(smem_u32(sm.k[st]), kDescK), km = desc(smem_u32(sm.k[st]), kDescMN);
        const uint32_t vm = desc(smem_u32(sm.v[st]), kDescMN);
        wait(&sm.q_full, n & 1);
        wait(&sm.k_full[st], (n >> 1) & 1);
        if (dead()) break;
        fence_after_sync();
        // scores (the product with the last chunk's, which holds these columns, was issued before)
#pragma unroll
        for (int ks = 0; ks < DK / 16; ++ks) {
          const uint32_t o = ((ks >> 2) * (128 * kC) + (ks & 3) * 32) / 16;
          mma_ss(tmem + kTmS, qd + o, kk + o, idesc_bf16(128, kC), ks > 0);
        }
        mma_commit(&sm.s_done);
        // queries and the state before the chunk (first: the place of its bf16 form is free once the update is done)
        wait(&sm.st_ready, n & 1);
        if (n > 0) wait(&sm.o_empty, (n & 1) ^ 1u);
        if (dead()) break;
        fence_after_sync();
        const bool fresh = r.fresh(c);
#pragma unroll
        for (int ks = 0; ks < DK / 16 && !fresh; ++ks)
          mma_ss(tmem + kTmI, qd + ((ks >> 2) * (128 * kC) + (ks & 3) * 32) / 16,
                 sd + ((ks >> 2) * (128 * DV) + (ks & 3) * 32) / 16, idesc_bf16(128, DV), ks > 0);
        mma_commit(&sm.q_empty);
        // the state's update, lanes = its columns
        wait(&sm.v_ready[st], (n >> 1) & 1);
        wait(&sm.ks_ready, n & 1);
        if (dead()) break;
        fence_after_sync();
#pragma unroll 1
        for (int part = 0; part < 2; ++part) {
          const uint32_t kb = part ? lod : km;
#pragma unroll
          for (int ks = 0; ks < kC / 16; ++ks)
            mma_ss(tmem + kTmState, vm + ks * 128, kb + ks * 128, idesc_bf16_mnmn(128, DK), !fresh || part > 0 || ks > 0);
        }
        mma_commit(&sm.g_done);
        wait(&sm.p_ready, n & 1);
        if (dead()) break;
        fence_after_sync();
#pragma unroll
        for (int ks = 0; ks < kC / 16; ++ks)
          mma_ts(tmem + kTmO, tmem + kTmS + (ks >> 2) * 64 + (ks & 3) * 8, vm + ks * 128, idesc_bf16_bmn(128, DV), ks > 0);
        mma_commit(&sm.o_done);
        mma_commit(&sm.k_empty[st]);
      }
    }
    if (lane == 0) {                  // no product outlives the TMEM
      mma_commit(&sm.drained);
      mbar_wait(&sm.drained, 0, 100000000ull);
    }
    __syncwarp();
  } else if (warp < 8) {
    // ------------------------------- scores and outputs: a token to a thread and the one 128 on, half of its columns each
    const int i = tid & 127, quad = warp & 3, half = warp >> 2;
    const uint32_t tl = tmem + ((uint32_t)(quad * 32) << 16);
    for (Run r = next_run(); r.kind != kEnd; r = next_run()) {
      if (r.kind == kZeros) {
        const int begin = r.c0 * kC, end = min(r.len, r.c1 * kC);
        for (int t = begin + tid; t < end; t += 256)
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
#pragma unroll 1
        for (int bb = 0; bb < 2; ++bb) {
          const int b = half * 2 + bb;
          const int last = b == quad ? lane : 31;           // the last column that the token sees
          float x[32];
          uint32_t p[16], odd[2] = {0, 0};                  // odd: NaN with any that is not finite
          if (b > quad) {                                   // later tokens only
#pragma unroll
            for (int e = 0; e < 16; ++e) p[e] = 0;
          } else {
            tmem_row<32>(tl + kTmS + b * 32, x);
            const float4* g4 = reinterpret_cast<const float4*>(upto + b * 32);
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const float4 g = g4[e / 4];
              x[e] *= ex2f(mine - g.x);
              x[e + 1] *= ex2f(mine - g.y);
              x[e + 2] *= ex2f(mine - g.z);
              x[e + 3] *= ex2f(mine - g.w);
            }
#pragma unroll
            for (int e = 0; e < 32; e += 2) p[e / 2] = pack2(e <= last ? x[e] : 0.f, e + 1 <= last ? x[e + 1] : 0.f);
#pragma unroll
            for (int e = 0; e < 16; ++e) odd[e & 1] = fma_bf16x2(p[e], 0, odd[e & 1]);
          }
          // (over scores that this warp has read)
          const uint32_t to = tl + kTmS + half * 64 + bb * 16;
          if (__any_sync(0xffffffffu, any_nan(odd[0]) || any_nan(odd[1]))) scores_slowly(tl + kTmS + b * 32, to, upto + b * 32, mine, last);
          else tmem_st16w_nw(to, p);
        }
        tmem_wait_st();
        fence_before_sync();
        arrive_warp(&sm.p_ready);
        wait_warp(&sm.o_done, n & 1);
        fence_after_sync();
        const float f = r.fresh(c) ? 0.f : ex2f(mine);
        // into the place of the values, which the chunk's products have read; a warp of its own sends them off
        uint8_t* tile = sm.v[st];
#pragma unroll 1
        for (int b = 0; b < DV / 2; b += 16) {
          float o[16];
          uint32_t x[16], z[16];
          tmem_ld16_nw(tl + kTmO + half * (DV / 2) + b, x);
          tmem_ld16_nw(tl + kTmI + half * (DV / 2) + b, z);
          tmem_wait_ld();
          reg_fence16(x);
          reg_fence16(z);
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            o[e] = __uint_as_float(x[e]);
            if (f != 0.f) o[e] = fmaf(f, __uint_as_float(z[e]), o[e]);   // (no state, or one that has decayed to nothing: nothing)
          }
          const int piece = (half * (DV / 2) + b) / 8;
          *reinterpret_cast<uint4*>(tile + tile_at(i, piece)) =
              make_uint4(pack2(o[0], o[1]), pack2(o[2], o[3]), pack2(o[4], o[5]), pack2(o[6], o[7]));
          *reinterpret_cast<uint4*>(tile + tile_at(i, piece + 1)) =
              make_uint4(pack2(o[8], o[9]), pack2(o[10], o[11]), pack2(o[12], o[13]), pack2(o[14], o[15]));
        }
        fence_before_sync();
        arrive_warp(&sm.o_empty);
        if (*(volatile int*)&sm.bad[n & 3] && i < rows)
          mark_reached(a, r.t0 + c * kC + i, i, r.head, half * (DV / 2), DV / 2, tile);
        fence_proxy_async_smem();
        arrive_warp(&sm.t_ready);
      }
    }
  } else {
    // ------------------------------- keys and state
    if (a.chained) pdl_wait_primary();
    using L = StateRows<DK, DV>;
    constexpr int N = L::kBlock;
    const int t = tid - 256;
    const L at(t);
    const uint32_t tl = tmem + kTmState + ((uint32_t)at.lanes << 16) + at.first;
    constexpr long long kSize = DK * DV;
    // adds what the non-finite values of chunk c of a run add to N rows of the state's column
    auto add_bad = [&](const Run& r, int c, int d, float* s) {
      float more[N];                  // (a copy, so that s stays in registers)
#pragma unroll 1
      for (int e = 0; e < N; ++e)
        more[e] = column_part<false>(a, r.t0 + c * kC, min(kC, r.len - c * kC), r.head, at.column, d + e);
#pragma unroll
      for (int e = 0; e < N; ++e) s[e] += more[e];
    };
    while (true) {
      const Run r = next_run();
      if (bar_any(1, 256, r.kind == kEnd)) break;         // (together: they meet in barriers)
      if (r.kind != kRun) continue;
      float* state = a.l.state + ((long long)r.slot * a.l.Hv + r.head) * kSize + at.column;
      if (!a.chained && r.c1 < r.n && r.init) pdl_wait_primary();
      const float* from = r.c0 > 0     ? a.ws + (size_t)(a.chained ? piece - 1 : 2 * a.grid + piece) * kSize + at.column
                          : r.c1 < r.n ? a.ws + (size_t)(a.grid + piece) * kSize + at.column
                                       : state;
      if (r.n == 0 && !r.init) {
        for (int e = 0; e < L::kRows; ++e) state[(at.first + e) * DV] = 0.f;
      }
      for (int c = r.c0; c < r.c1; ++c, ++n) {
        const int st = n & 1;
        if (c > r.c0) {
          wait_warp(&sm.g_done, (n & 1) ^ 1u);
          fence_after_sync();
        }
        wait_warp(&sm.g_full[st], (n >> 1) & 1);
        const float f = ex2f(sm.upto[st][kC - 1]);
#pragma unroll 1
        for (int b = 0; b < L::kRows && !r.fresh(c); b += N) {
          const int d = at.first + b;
          float s[N];
          if (c > r.c0) {
            tmem_row<N>(tl + b, s);
            if (*(volatile int*)&sm.bad[(n - 1) & 3]) add_bad(r, c - 1, d, s);
          } else {
#pragma unroll
            for (int e = 0; e < N; ++e) s[e] = __ldcg(from + (d + e) * DV);
          }
          uint8_t* row = sm.state + (d >> 6) * (128 * DV) + at.column * 128;
          const int chunk = (d & 63) >> 3;
#pragma unroll
          for (int e = 0; e < N; e += 8)
            *reinterpret_cast<uint4*>(row + (((chunk + e / 8) ^ (at.column & 7)) << 4)) = make_uint4(
                pack2(s[e], s[e + 1]), pack2(s[e + 2], s[e + 3]), pack2(s[e + 4], s[e + 5]), pack2(s[e + 6], s[e + 7]));
#pragma unroll
          for (int e = 0; e < N; e += 2) mul2(s[e], s[e + 1], f);
          if (f == 0.f) {                                   // (whatever it was)
#pragma unroll
            for (int e = 0; e < N; ++e) s[e] = 0.f;
          }
          tmem_st16_nw(tl + b, s);
          if constexpr (N == 32) tmem_st16_nw(tl + b + 16, s + 16);
        }
        tmem_wait_st();
        fence_before_sync();
        fence_proxy_async_smem();
        arrive_warp(&sm.st_ready);
        wait_warp(&sm.s_done, n & 1);
        split_keys<DK, 256>(sm.k[st], sm.lo, sm.w[st], t);
        fence_proxy_async_smem();
        arrive_warp(&sm.ks_ready);
      }
      if (r.c1 > r.c0) {
        wait_warp(&sm.g_done, (n & 1) ^ 1u);
        fence_after_sync();
        if (r.c1 == r.n) {
#pragma unroll 1
          for (int b = 0; b < L::kRows; b += N) {
            float s[N];
            tmem_row<N>(tl + b, s);
            if (*(volatile int*)&sm.bad[(n - 1) & 3]) add_bad(r, r.c1 - 1, at.first + b, s);
#pragma unroll
            for (int e = 0; e < N; ++e) state[(at.first + b + e) * DV] = s[e];
          }
        }
        fence_before_sync();
      }
    }
    pdl_wait_primary();                 // (this kernel ends after the one before it)
  }
  __syncthreads();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

template <int DK, int DV>
int launch_dims(const ChunkArgs& a, const Maps& maps, cudaStream_t stream) {
  static_assert(sizeof(SumSmem<DK, DV>) <= 227 * 1024 && sizeof(OutSmem<DK, DV>) <= 227 * 1024, "shared memory of a block");
  static OncePerDevice once_sum, once_out;
  int rc;
  if ((rc = raise_smem(once_sum, sum_kernel<DK, DV>, sizeof(SumSmem<DK, DV>))) != GDN_OK) return rc;
  if ((rc = raise_smem(once_out, out_kernel<DK, DV>, sizeof(OutSmem<DK, DV>))) != GDN_OK) return rc;
  if (a.cut) {
    rc = launch(sum_kernel<DK, DV>, dim3((unsigned)a.grid), kSumThreads, sizeof(SumSmem<DK, DV>), stream, a, maps);
    if (rc != GDN_OK) return rc;
  }
  if (a.chained) {
    rc = launch(chain_kernel, dim3((unsigned)a.grid), kChainThreads, 0, stream, a);
    if (rc != GDN_OK) return rc;
  }
  return launch(out_kernel<DK, DV>, dim3((unsigned)a.grid), kOutThreads, sizeof(OutSmem<DK, DV>), stream, a, maps);
}

}  // namespace

size_t decay_prefill_ws_bytes(const DecayView& l, int, int) {
  const int sms = sm_count();
  const size_t grid = sms > 0 ? sms : 160;      // without a device (host-side sizing): at least the part's SMs
  return grid * (3 * (size_t)l.dk * l.dv * 4 + 8);
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
  if (a.grid <= 0 || a.grid >= kMostGrid) return GDN_ERR_CUDA;
  a.cut = total_tokens > kC;          // (one chunk is not cut)
  // a sequence's heads share the line equally, so a run lies in at most grid / Hv + 2 pieces
  a.chained = a.cut && a.grid > 10 * l.Hv;
  Maps maps = {};
  if (total_tokens > 0 && !(make_rows_map(t.q, total_tokens, t.q_ld, l.Hk * l.dk, kC, l.dk / 64, &maps.q) &&
                            make_rows_map(t.k, total_tokens, t.k_ld, l.Hk * l.dk, kC, l.dk / 64, &maps.k) &&
                            make_rows_map(t.v, total_tokens, t.v_ld, l.Hv * l.dv, kC, l.dv / 64, &maps.v) &&
                            make_rows_map(t.out, total_tokens, (long long)l.Hv * l.dv, l.Hv * l.dv, kC, l.dv / 64, &maps.out)))
    return GDN_ERR_CUDA;
  if (l.dk == 128) return l.dv == 128 ? launch_dims<128, 128>(a, maps, stream) : launch_dims<128, 64>(a, maps, stream);
  return l.dv == 128 ? launch_dims<64, 128>(a, maps, stream) : launch_dims<64, 64>(a, maps, stream);
}

}  // namespace gdn
