// gdn_attn_chunk.cu -- attention of runs of new tokens (prompts, chunks of prompts) over the paged
// cache, on the tcgen05 tensor cores.
//
//   S = Q K^T,   P = 2^(scale log2(e) S - m),   O += P V,   o = O / l,   l = sum P
//
// in one pass over 128-key tiles.  A CTA holds a tile of query rows (row = new token x head of the
// key/value head's group): two blocks of 128 rows for head dims up to 128, one for 256 and where no
// sequence has rows for a second.  S and O live in TMEM (256 + 2 D columns, or 2 x 128 + D), P
// replaces S in place as the TMEM operand of the second product.
//
// What bounds it: 4 D flops per (row, key) on the tensor pipe and one exponential per (row, key)
// on the special-function units, of which D = 128 takes about as long for both; so neither may
// wait for the other:
//  * a softmax warpgroup per block of rows (a thread owns a row: no shuffles), one thread issuing
//    MMAs, a warp each issuing the TMA copies of keys and values, and for 8-bit caches a warpgroup
//    (two for D = 256) that turns the values' codes into bf16 operands; the keys' codes are operands
//    of e4m3 MMAs as they are, against the queries in two e4m3 parts;
//  * the MMA order PV_0(i), QK_0(i+1), PV_1(i), QK_1(i+1) keeps the pipe on one block while the
//    other block's softmax runs (one block: two S buffers, PV(i), QK(i+2));
//  * the reference m follows the running maximum only when that outgrows it by 2^8, so O is almost
//    never rescaled, and never by a warpgroup of its own;
//  * a tile's queries have the place that its gate and its output then pass through, so the next tile's
//    are loaded, and its first product issued, after the output has left: between two tiles of rows the
//    pipe stands still for 9 us (bf16, D = 128 or 256), 13 to 14 us where queries are split for an 8-bit
//    cache, and 3.5 us more with a gate at D = 256 (5 and 1 tiles a CTA compared, 2 and 18 key tiles each).
// Measured, 4096 tokens on 16384 cached ones (1.24 TFLOP at 32 heads of 128 and 16 of 256), a few calls
// in a row: bf16 D = 128 836 to 849 us, 1457 to 1480 TFLOP/s (77 to 78 % of the dense bf16 rate, 63 % of
// the cycles with the pipe busy at its nominal rate; 899 us in a long row of calls, under the power
// cap); D = 256 812 us, 1523; D = 64 697 us, 887, where the exponentials bound it.  8-bit: 1120 us, 1183
// to 1205 us and 909 us, bound by the conversion of the values, whose instructions share the issue slots
// and instruction caches with the softmax.  32 rows on 8000 keys (64 sequences of 8 tokens): bf16 318 to
// 322 us, 98 % of the copy bandwidth; 8-bit 354 us, 45 %.
// Fewer bits: the probabilities become bf16, the type of the second product's other operand (half a step
// of each, 2^-9 to 2^-8 of it; tf32 products run at half the rate); their sum takes them unrounded.  An
// 8-bit cache's queries become two e4m3 parts (see split_e4m3).
// Values whose key some rows do not see must be finite for the product to leave those rows alone:
// in tiles that the causal edge crosses, the first warpgroup replaces non-finite ones (and
// whatever lies past the sequence's end) by zero, and notes column and position, so that the rows
// that do see them get their infinity or NaN.
#include "gdn_attn.cuh"
#include "gdn_tmap.h"

namespace gdn {

using namespace tc;

namespace attn {

constexpr int kKeys = 128;         // keys of a tile
// B: 128-row query blocks.  One where TMEM holds no more (D = 256), or where a tile has no rows for
// two: S then has two buffers, so that the products of one key tile run beside the softmax of another.
template <int D, bool Q8, int B>
struct ChunkCfg {
  static_assert(B == 1 || (B == 2 && D < 256), "TMEM: S and O of each block");
  static constexpr int kBlocks = B;
  static constexpr int kRows = 128 * kBlocks;
  static constexpr int kCols = D == 64 ? 64 : 128;          // columns of a ring stage
  static constexpr int kHalves = D / kCols;                 // stages of a K or V tile
  // K stages: bf16, or the e4m3 codes themselves; V stages: bf16; R stages: the codes of V
  static constexpr int kKBytes = kKeys * kCols * (Q8 ? 1 : 2), kVBytes = kKeys * kCols * 2, kRBytes = kKeys * kCols;
  static constexpr int kKStages = D == 64 ? (B == 1 ? 6 : 4) : Q8 ? (D == 256 ? 2 : B == 1 ? 4 : 3) : D == 128 && B == 2 ? 2 : 3;
  static constexpr int kVStages = Q8 ? 2 : D == 64 ? (B == 1 ? 6 : 4) : D == 128 && B == 2 ? 3 : 2;
  static constexpr int kRStages = !Q8 ? 0 : B == 1 && D < 256 ? 3 : 2;
  // tiles whose scales are held: a tile's place is taken after the values of two tiles before it
  // have been converted, which with two V stages means that four before it are through
  static constexpr int kScales = Q8 ? 4 : 0;
  static constexpr int kSoftWarps = 4 * kBlocks;
  static constexpr int kMmaWarp = kSoftWarps, kLoadWarp = kSoftWarps + 1, kSchedWarp = kSoftWarps + 2, kLoadVWarp = kSoftWarps + 3,
                       kConvWarp = kSoftWarps + 4;
  // whole warpgroups: softmax (one per block), control (MMA and TMA warps), conversion
  static constexpr int kConvGroups = Q8 ? kHalves : 0;      // one for each half of a V tile
  static constexpr int kGroups = kBlocks + 1 + kConvGroups;
  static constexpr int kThreads = kGroups * 128;
  static constexpr int kReaders = kSoftWarps + 3 + 4 * kConvGroups;   // warps that read a segment
  // registers per thread at launch (65,536 shared by the CTA's threads, in eights) and after the
  // warpgroups have traded: their sum over the warpgroups is the launch's
  static constexpr int kLaunchRegs = kGroups == 2 ? 255 : kGroups == 3 ? 168 : 128;
  static constexpr int kSoftRegs = kGroups == 2 ? 0 : kGroups == 3 ? 208 : B == 2 ? 176 : 216;
  static constexpr int kCtrlRegs = kGroups == 2 ? 0 : kGroups == 3 ? 88 : B == 2 ? 64 : 88;
  static constexpr int kConvRegs = kGroups == 3 ? 168 : B == 2 ? 96 : 104;
  static_assert(kGroups == 2 || B * kSoftRegs + kCtrlRegs + kConvGroups * kConvRegs <= kGroups * kLaunchRegs,
                "a share above the launch's registers would wait for ever");
  static constexpr int kQBytes = 128 * D * 2;               // one block
  static constexpr int kO = 256;                            // TMEM column of O (block b: + b D)
};

template <int D, bool Q8, int B>
struct __align__(1024) ChunkSmem {
  using C = ChunkCfg<D, Q8, B>;
  uint8_t q[C::kBlocks][C::kQBytes];
  uint8_t k[C::kKStages][C::kKBytes];
  uint8_t v[C::kVStages][C::kVBytes];
  uint8_t raw[Q8 ? C::kRStages : 1][Q8 ? C::kRBytes : 128];
  uint8_t scales[Q8 ? C::kScales : 1][2][kKeys];             // bytes of a tile's keys and values
  float k_scale[Q8 ? C::kScales : 1][kKeys];
  float q_scale[C::kBlocks][Q8 ? 128 : 1];
  LineScan<C::kRows, C::kThreads> scan;
  uint32_t bad[D];                  // a Notes of each column
  SegDesc segs[kSegs];
  int any_bad;
  uint32_t tmem;
  int dead, stopped;
  uint64_t k_full[C::kKStages], k_empty[C::kKStages], v_full[C::kVStages], v_empty[C::kVStages];
  uint64_t r_full[Q8 ? C::kRStages : 1], r_empty[Q8 ? C::kRStages : 1];
  uint64_t s_bytes[Q8 ? C::kScales : 1], s_free[Q8 ? C::kScales : 1], s_ready[Q8 ? C::kScales : 1];
  uint64_t q_ready[2], s_full[2], p_ready[2], o_done[2];
  uint64_t seg_full[kSegs], seg_empty[kSegs];
  uint64_t drained;
};

// Where in a column of values the first +inf, -inf and NaN lie that some rows of a tile do not see, as
// positions past its first row's (at most 256 rows and 128 keys on), ten bits each.  An 8-bit cache has
// vectors that are NaN throughout and no infinities: there it is one absolute position.
struct Notes {
  static constexpr uint32_t kNone = 0xffffffffu;
  static __device__ __forceinline__ int first(uint32_t notes, int kind) { return (notes >> (10 * kind)) & 1023; }
  // the bf16 `value` at position `at`
  static __device__ __forceinline__ void add(uint32_t* notes, uint32_t value, int at) {
    const int kind = value == 0x7f80u ? 0 : value == 0xff80u ? 1 : 2;
    uint32_t old = *(volatile uint32_t*)notes;
    while (first(old, kind) > at) {
      const uint32_t seen = old;
      old = atomicCAS(notes, seen, (seen & ~(1023u << (10 * kind))) | ((uint32_t)at << (10 * kind)));
      if (old == seen) break;
    }
  }
};

// Operand descriptors of 128-byte-swizzled tiles (8-row groups 1,024 bytes apart).  Only the low
// word changes from one MMA to the next: the start address, in sixteen-byte units, beside a constant.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);          // SBO, version, swizzle
constexpr uint32_t kDescHi64 = (512u >> 4) | (1u << 14) | (4u << 29);          // 64-byte rows and swizzle
constexpr uint32_t kDescK = (16u >> 4) << 16;                                  // K-major: LBO unused
constexpr uint32_t kDescMN = ((128u * 128u) >> 4) << 16;                       // MN-major: 64-column blocks

__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t kind) { return ((saddr & 0x3FFFFu) >> 4) | kind; }

// The issuing thread's instructions between two MMAs are what the tensor pipe waits for when they
// are many: 32-bit operands, constants where possible.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n.reg .pred p;\n.reg .b64 a, b;\nmov.b64 a, {%1, %5};\nmov.b64 b, {%2, %5};\nsetp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n}\n" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(acc), "n"(kDescHi)
      : "memory");
}
// The same on e4m3 operands (32 columns an MMA); HI as above.
template <uint32_t HI>
__device__ __forceinline__ void mma_ss_e4m3(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n.reg .pred p;\n.reg .b64 a, b;\nmov.b64 a, {%1, %5};\nmov.b64 b, {%2, %5};\nsetp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, p;\n}\n" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(acc), "n"(HI)
      : "memory");
}
// kind::f8f6f4, e4m3 A and B (both K-major), f32 accumulator.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n.reg .pred p;\n.reg .b64 b;\nmov.b64 b, {%2, %5};\nsetp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(idesc), "r"(acc), "n"(kDescHi)
      : "memory");
}

__device__ __forceinline__ uint32_t globaltimer_lo() {
  uint32_t t;
  asm volatile("mov.u32 %0, %globaltimer_lo;" : "=r"(t));
  return t;
}
// A wait of the roles that compute.  One that gives up waits (again with a limit) until both loading
// warps have stopped, of themselves or because nothing comes back to them; then nothing that the role
// still hands back, on its way through its segment, is taken for a free place.  Few instructions: they
// stand at every wait, and the 8-bit kernels are bound by their instruction caches (with two more
// 64-bit loops here 1116 -> 1200 us).  The status is set at the end.
__device__ __forceinline__ void wait_held(uint64_t* bar, uint32_t parity, volatile int* dead, volatile int* stopped) {
  if (mbar_try_wait(bar, parity)) return;
  const uint32_t t0 = globaltimer_lo();
  while (*dead == 0) {
    if (mbar_try_wait(bar, parity)) return;
    if (globaltimer_lo() - t0 > 2000000000u) *dead = 1;
  }
  while (*stopped < 2 && globaltimer_lo() - t0 < 3000000000u) {}
}
__device__ __forceinline__ float ex2f(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N));
}

// 32 lanes x 32 columns; no wait.
__device__ __forceinline__ void tmem_ld32_nw(uint32_t addr, uint32_t* r) {
  tmem_ld16_nw(addr, r);
  tmem_ld16_nw(addr + 16, r + 16);
}

// Pairs of f32 in one instruction.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t p, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool fill) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(fill ? 16 : 0) : "memory");
}
// An arrival once this thread's copies so far are there.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];\n" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;\n" ::: "memory"); }

template <int N>
struct Int {
  static constexpr int value = N;
};

// Position of a stage in the ring.
template <int N>
struct RingPos {
  int stage = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void step() {
    if (++stage == N) { stage = 0; phase ^= 1u; }
  }
};

// The ring's order within a segment of n tiles: K0, K1, V0, K2, V1, ... (each kHalves stages).
// Calls f(is_v, tile index from 0, half).
template <int HALVES, typename F>
__device__ __forceinline__ void ring_order(int n, F f) {
  for (int h = 0; h < HALVES; ++h) f(false, 0, h);
  for (int i = 0; i < n; ++i) {
    if (i + 1 < n)
      for (int h = 0; h < HALVES; ++h) f(false, i + 1, h);
    for (int h = 0; h < HALVES; ++h) f(true, i, h);
  }
}

template <int D, bool Q8, int B>
__global__ void __launch_bounds__(ChunkCfg<D, Q8, B>::kThreads, 1)
chunk_kernel(const KvView c, const KvBatchView b, const AttnArgs a, int grid, int fix, int least,
             const __grid_constant__ KvMaps maps) {
  using C = ChunkCfg<D, Q8, B>;
  constexpr int R = C::kRows, TK = kKeys;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  ChunkSmem<D, Q8, B>& sm = *reinterpret_cast<ChunkSmem<D, Q8, B>*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < C::kKStages; ++i) {
      mbar_init(&sm.k_full[i], 1);
      mbar_init(&sm.k_empty[i], 1);
    }
    for (int i = 0; i < C::kVStages; ++i) {
      mbar_init(&sm.v_full[i], Q8 ? 4 : 1);
      mbar_init(&sm.v_empty[i], 1);
    }
    for (int i = 0; i < C::kRStages; ++i) {
      mbar_init(&sm.r_full[i], 1);
      mbar_init(&sm.r_empty[i], 4);
    }
    for (int i = 0; i < C::kScales; ++i) {
      mbar_init(&sm.s_bytes[i], 16);
      mbar_init(&sm.s_free[i], 4 * C::kConvGroups);
      mbar_init(&sm.s_ready[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.q_ready[i], 4);
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_ready[i], 4);
      mbar_init(&sm.o_done[i], 1);
    }
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(&sm.seg_full[i], 1);
      mbar_init(&sm.seg_empty[i], C::kReaders);
    }
    mbar_init(&sm.drained, 1);
    sm.dead = sm.stopped = 0;
    sm.any_bad = 0;
    mbar_fence_init();
  }
  for (int i = tid; i < D; i += C::kThreads) sm.bad[i] = Q8 ? INT32_MAX : Notes::kNone;
  pdl_begin();
  const RowRange batch = batch_rows(b);
  // (never before the wait in pdl_begin: a kernel that this one waits for may need the columns)
  if (warp == C::kMmaWarp) tmem_alloc(&sm.tmem, 512);
  fence_before_sync();
  bool bad_len = false;
  Pieces pieces;
  const int cta = blockIdx.x;
  locate_piece<R, C::kThreads>(c, b, a.g, fix, grid, least, cta, &pieces, &sm.scan, &bad_len);
  zero_outside(a, b, D, batch, &bad_len);
  if (bad_len) set_status(c.status, GDN_STATUS_BAD_SEQLENS);
  // (locate_piece has synchronised the block)
  if (cta >= pieces.count) {
    if (tid == 0) Partials<R, D>::note(a.ws, grid, cta, a.g, nullptr, 0);
    if (warp == C::kMmaWarp) tmem_dealloc(sm.tmem, 512);
    return;
  }
  fence_after_sync();
  // all 512 columns: they start at column 0, and TMEM addresses are constants from here on
  constexpr uint32_t tmem = 0;
  if (sm.tmem != 0) {
    if (tid == 0) {
      set_status(c.status, GDN_STATUS_TIMEOUT);
      Partials<R, D>::note(a.ws, grid, cta, a.g, nullptr, 0);
    }
    if (warp == C::kMmaWarp) tmem_dealloc(sm.tmem, 512);
    return;
  }
  auto dead = [&]() { return *(volatile int*)&sm.dead != 0; };
  auto warp_dead = [&]() { return __any_sync(0xffffffffu, dead()) != 0; };
  auto wait = [&](uint64_t* bar, uint32_t parity) { wait_held(bar, parity, &sm.dead, &sm.stopped); };
  auto wait_warp = [&](uint64_t* bar, uint32_t parity) {
    wait(bar, parity);
    __syncwarp();
  };
  auto seg_wait = [&](const RingPos<kSegs>& p) -> const SegDesc& {
    wait_warp(&sm.seg_full[p.stage], p.phase);
    return sm.segs[p.stage];
  };
  auto seg_done = [&](RingPos<kSegs>& p) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.seg_empty[p.stage]);
    p.step();
  };
  RingPos<kSegs> seg;

  // All four warps of the control warpgroup give their registers up together.
  if (C::kGroups > 2 && warp >= C::kMmaWarp && warp < C::kConvWarp) regs_down<C::kCtrlRegs ? C::kCtrlRegs : 24>();
  if (warp == C::kSchedWarp) {
    // ---------------------------------------------------------------- segments
    SegIter<R, TK> it;
    it.start(&b, c.page_shift, c.H, a.g, fix, pieces, cta, sm.scan.at);
    Segment s;
    s.split = false;
    bool alive = true;
    for (bool more = true; more;) {
      more = it.next(&s);
      if (more && idle(s)) continue;
      alive = wait_bar(&sm.seg_empty[seg.stage], seg.phase ^ 1u, &sm.dead, c.status);
      if (!alive) break;
      if (lane == 0) {
        SegDesc d = {};
        d.n = -1;
        sm.segs[seg.stage] = more ? describe<R>(s, a.g) : d;
        mbar_arrive(&sm.seg_full[seg.stage]);
      }
      __syncwarp();
      seg.step();
    }
    // the piece's last tile may be shared with the next ones
    if (lane == 0) Partials<R, D>::note(a.ws, grid, cta, a.g, &s, alive && s.split ? it.sharing(s.nt) : 0);
  } else if (warp == C::kLoadWarp || warp == C::kLoadVWarp) {
    // ---------------------------------------------------------------- TMA
    // Copies of one warp go out one after another (some 150 cycles each), hence a warp for the keys
    // and one for the values (64 sequences of 8000, pages of 16, D = 128, bf16: 359 us with one, 322 us).
    const bool values = warp == C::kLoadVWarp;
    const int box = min(1 << c.page_shift, TK);            // keys of one copy
    constexpr int kBoxCols = Q8 ? C::kCols : 64;
    constexpr int kBlk = C::kCols / kBoxCols;
    const int pages = TK / box;                             // 1 to 8
    RingPos<C::kKStages> kp;
    RingPos<Q8 ? C::kRStages : C::kVStages> vp;
    RingPos<Q8 ? C::kScales : 1> sp;
    uint64_t* v_full = Q8 ? sm.r_full : sm.v_full;
    uint64_t* v_empty = Q8 ? sm.r_empty : sm.v_empty;
    const int my_page = lane / kBlk, my_blk = lane % kBlk;
    bool alive = true;
    while (alive) {
      alive = wait_bar(&sm.seg_full[seg.stage], seg.phase, &sm.dead, c.status);
      const SegDesc& sd = sm.segs[seg.stage];
      const int n = sd.n, ta = sd.ta, len = sd.len, head = sd.head;
      const int* table = b.table + (long long)sd.seq * b.table_ld;
      seg_done(seg);
      if (!alive || n < 0) break;
      if (n == 0) continue;
      auto lookup = [&](int i) {                            // this lane's page of tile i
        const int k = (ta + i) * TK + my_page * box;
        if (i >= n || my_page >= pages || k >= len) return c.num_pages;   // zeros
        int p = __ldg(table + (k >> c.page_shift));
        if (p < 0 || p >= c.num_pages) {
          set_status(c.status, GDN_STATUS_PAGE_RANGE);
          p = c.num_pages;
        }
        return p;
      };
      int p_next = lookup(0), p_ahead = lookup(1);          // pages of tiles i + 1, i + 2
#pragma unroll 1
      for (int i = 0; i < n && alive; ++i) {
        const int page = p_next;
        p_next = p_ahead;
        p_ahead = lookup(i + 2);
        const int off = (((ta + i) * TK) & ((1 << c.page_shift) - 1));   // 0 unless pages exceed a tile
        if (Q8 && !values) {                                // the tile's scale bytes, keys and values
          alive = wait_bar(&sm.s_free[sp.stage], sp.phase ^ 1u, &sm.dead, c.status);
          if (!alive) break;
          const int key = (lane & 7) * 16, at = key & (box - 1);
          const int p = __shfl_sync(0xffffffffu, page, (key / box) * kBlk);
          const uint8_t* src = (lane & 8 ? c.vs : c.ks) + (((long long)p * c.H + head) << c.page_shift) + off + at;
          if (lane < 16) {
            const bool there = p < c.num_pages;             // zeros if not
            cp_async16(smem_u32(sm.scales[sp.stage][lane >> 3] + key), there ? src : c.ks, there);
            cp_async_arrive(&sm.s_bytes[sp.stage]);
          }
          __syncwarp();
          sp.step();
        }
#pragma unroll
        for (int half = 0; half < C::kHalves; ++half) {
          uint64_t* full = values ? &v_full[vp.stage] : &sm.k_full[kp.stage];
          alive = wait_bar(values ? &v_empty[vp.stage] : &sm.k_empty[kp.stage], (values ? vp.phase : kp.phase) ^ 1u,
                           &sm.dead, c.status);
          if (!alive) break;
          if (lane == 0) mbar_arrive_expect_tx(full, values ? (Q8 ? C::kRBytes : C::kVBytes) : C::kKBytes);
          __syncwarp();
          if (my_page < pages) {
            uint8_t* dst = values ? (Q8 ? sm.raw[vp.stage] : sm.v[vp.stage]) : sm.k[kp.stage];
            dst += Q8 ? my_page * box * C::kCols : my_blk * (TK * 128) + my_page * box * 128;
            tma_load_5d(dst, values ? &maps.v : &maps.k, 0, off, half * kBlk + my_blk, head, page, full);
          }
          __syncwarp();
          if (values) vp.step();
          else kp.step();
        }
      }
    }
    if (lane == 0) atomicAdd(&sm.stopped, 1);
    // no copy outlives the CTA, whoever has stopped waiting for it
    cp_async_wait_all();
    if (values) drain_ring<(Q8 ? C::kRStages : C::kVStages)>(v_full, vp.stage, vp.phase);
    else drain_ring<C::kKStages>(sm.k_full, kp.stage, kp.phase);
  } else if (warp == C::kMmaWarp) {
    // ---------------------------------------------------------------- MMA (one thread)
    // The tensor pipe queues only a few MMAs, so what this thread does between them leaves the pipe
    // idle (a commit costs some 40 cycles, a wait that finds its phase complete twice that): it
    // waits for p_ready alone where that implies the tiles are there, and (two blocks) leaves it to
    // the softmax to hand the rings' stages back.
    if (lane == 0) {
      RingPos<C::kKStages> kp;
      RingPos<C::kVStages> vp;
      uint32_t cnt[2] = {0, 0};          // tiles of each block
      uint32_t s_cnt = 0;                // S buffers filled (one block)
      uint32_t q_phase[2] = {0, 0};
      constexpr uint32_t kIdQK = Q8 ? idesc_e4m3(128, 128) : idesc_bf16(128, 128);
      constexpr uint32_t kIdPV = idesc_bf16_bmn(128, C::kCols);
      const uint32_t k0 = desc_lo(smem_u32(sm.k[0]), kDescK), v0 = desc_lo(smem_u32(sm.v[0]), kDescMN);
      const uint32_t q0 = desc_lo(smem_u32(sm.q[0]), kDescK);
      auto k_lo = [&]() { return k0 + kp.stage * (C::kKBytes / 16); };
      auto v_lo = [&]() { return v0 + vp.stage * (C::kVBytes / 16); };
      // S[buf] (+)= Q K^T over the columns of one stage; O += P[buf] V into those columns
      auto qk_half = [&](int blk, int buf, uint32_t k, int half) {
        if constexpr (!Q8) {
          const uint32_t q = q0 + (blk * C::kQBytes + half * (C::kCols / 64) * (128 * 128)) / 16;
#pragma unroll
          for (int ks = 0; ks < C::kCols / 16; ++ks) {
            const uint32_t o = ((ks >> 2) * (128 * 128) + (ks & 3) * 32) / 16;
            mma_ss(buf * 128, q + o, k + o, kIdQK, half > 0 || ks > 0);
          }
        } else {
          // both parts of the queries against the same codes
#pragma unroll
          for (int part = 0; part < 2; ++part) {
            const uint32_t q = q0 + (blk * C::kQBytes + part * (C::kQBytes / 2) + half * (128 * C::kCols)) / 16;
#pragma unroll
            for (int ks = 0; ks < C::kCols / 32; ++ks)
              mma_ss_e4m3<C::kCols == 128 ? kDescHi : kDescHi64>(buf * 128, q + ks * 2, k + ks * 2, kIdQK,
                                                                half > 0 || part > 0 || ks > 0);
          }
        }
      };
      auto pv_half = [&](int blk, int buf, uint32_t v, int half, bool acc) {
#pragma unroll
        for (int ks = 0; ks < TK / 16; ++ks)
          mma_ts(C::kO + blk * D + half * C::kCols, buf * 128 + ks * 8, v + ks * (2048 / 16), kIdPV, acc || ks > 0);
      };
      while (true) {
        wait(&sm.seg_full[seg.stage], seg.phase);
        const SegDesc& sd = sm.segs[seg.stage];
        const int n = sd.n;
        const bool two = sd.rows > 128;
        mbar_arrive(&sm.seg_empty[seg.stage]);
        seg.step();
        if (dead() || n < 0) break;
        if (n == 0) continue;
        wait(&sm.q_ready[0], q_phase[0]);
        q_phase[0] ^= 1u;
        if (C::kBlocks == 2 && two) {
          wait(&sm.q_ready[1], q_phase[1]);
          q_phase[1] ^= 1u;
        }
        if constexpr (C::kBlocks == 2) {
          wait(&sm.k_full[kp.stage], kp.phase);
          fence_after_sync();
          qk_half(0, 0, k_lo(), 0);
          mma_commit(&sm.s_full[0]);
          if (two) {
            qk_half(1, 1, k_lo(), 0);
            mma_commit(&sm.s_full[1]);
          }
          kp.step();
          // Block 0's softmax of tile i has seen V(i) and K(i + 1) arrive before it says p_ready.
          for (int i = 0; i + 1 < n; ++i) {
            wait(&sm.p_ready[0], cnt[0]++ & 1u);
            fence_after_sync();
            pv_half(0, 0, v_lo(), 0, i > 0);
            qk_half(0, 0, k_lo(), 0);
            mma_commit(&sm.s_full[0]);
            if (two) {
              wait(&sm.p_ready[1], cnt[1]++ & 1u);
              fence_after_sync();
              pv_half(1, 1, v_lo(), 0, i > 0);
              qk_half(1, 1, k_lo(), 0);
              mma_commit(&sm.s_full[1]);
            }
            vp.step();
            kp.step();
          }
          wait(&sm.p_ready[0], cnt[0]++ & 1u);
          fence_after_sync();
          pv_half(0, 0, v_lo(), 0, n > 1);
          mma_commit(&sm.o_done[0]);
          if (two) {
            wait(&sm.p_ready[1], cnt[1]++ & 1u);
            fence_after_sync();
            pv_half(1, 1, v_lo(), 0, n > 1);
            mma_commit(&sm.o_done[1]);
          }
          vp.step();
        } else {
          auto qk_tile = [&]() {
            const int buf = (int)(s_cnt & 1u);
#pragma unroll
            for (int h = 0; h < C::kHalves; ++h) {
              wait(&sm.k_full[kp.stage], kp.phase);
              fence_after_sync();
              qk_half(0, buf, k_lo(), h);
              mma_commit(&sm.k_empty[kp.stage]);
              kp.step();
            }
            mma_commit(&sm.s_full[buf]);
            ++s_cnt;
          };
          qk_tile();
          if (n > 1) qk_tile();
          for (int i = 0; i < n; ++i) {
            const int buf = (int)(cnt[0] & 1u);
            wait(&sm.p_ready[0], cnt[0]++ & 1u);
            fence_after_sync();
#pragma unroll
            for (int h = 0; h < C::kHalves; ++h) {
              pv_half(0, buf, v_lo(), h, i > 0);
              mma_commit(&sm.v_empty[vp.stage]);
              vp.step();
            }
            mma_commit(&sm.o_done[0]);
            if (i + 2 < n) qk_tile();
          }
        }
      }
      mma_commit(&sm.drained);          // nor does a product outlive the TMEM
      mbar_wait(&sm.drained, 0, kDrainNs);
    }
    __syncwarp();
  } else if (Q8 && warp >= C::kConvWarp) {
    // ---------------------------------------------------------------- e4m3 -> bf16
    if constexpr (C::kConvRegs < C::kLaunchRegs) regs_down<C::kConvRegs>();
    const int ct = (tid - C::kConvWarp * 32) & 127, group = (warp - C::kConvWarp) >> 2;
    RingPos<Q8 ? C::kRStages : 1> src;
    RingPos<C::kVStages> dst;
    RingPos<Q8 ? C::kScales : 1> ks, vs;
    // A warp converts its own 32 rows, so that a row's multiplier comes from the lane that holds it.
    // A lane takes 16 codes of a row in two halves, the first of which differs from lane to lane so
    // that neither the 8-byte loads nor the 16-byte swizzled stores meet in a bank.  The loop is kept
    // rolled (D = 256: two rows), with the next row's loads ahead: unrolled eight times it does not
    // fit an SM quarter's instruction cache next to the softmax, and both ran at a third of the speed
    // (one prompt piece of 4096 on 16384 tokens, D = 256 with one group: 3147 us, rolled 1481 us).
    // A group of warps for each half of a V tile: 1481 -> 1388 us, two rows 1284 us.  The conversion
    // instruction (to f16 operands, for tiles whose scales f16 holds) is fewer instructions and slower
    // (1210 -> 1244 us; D = 128 1107 -> 1420): bit operations.
    constexpr int kPer = C::kCols / 16, kStep = 32 / kPer, kSteps = 32 / kStep;
    const int piece = lane % kPer, sub = lane / kPer, warp_row = (ct >> 5) * 32 + sub;
    constexpr int kUnroll = D == 256 ? 2 : 1;
    const int odd = kPer == 8 ? (piece >> 2) ^ (sub & 1) : (sub >> 1) & 1;
    while (true) {
      const int n = seg_wait(seg).n;
      seg_done(seg);
      if (warp_dead() || n < 0) break;
      if (n == 0) continue;
      ring_order<C::kHalves>(n, [&](bool is_v, int, int half) {
        if (!is_v) {
          // The scales of a tile's keys, one per thread.  Their place was last read by the softmax
          // four tiles ago, which is over: a V stage of a later tile has come back since.
          if (half == 0) {
            wait_warp(&sm.s_bytes[ks.stage], ks.phase);
            if (group == 0) {
              sm.k_scale[ks.stage][ct] = scale_f32(sm.scales[ks.stage][0][ct]);
              __syncwarp();
              if (lane == 0) mbar_arrive(&sm.s_ready[ks.stage]);
            }
            ks.step();
          }
          return;
        }
        if (half == group) {
          wait_warp(&sm.r_full[src.stage], src.phase);
          const uint32_t bb = sm.scales[vs.stage][1][ct];
          // the code's bits are the value times 2^-120: one multiply by 2^120 times the scale where that
          // is a bf16 value, else two
          const uint32_t f = bb <= 134 ? (bb + 120) << 7 : 0x7b80u;
          const bool large = __any_sync(0xffffffffu, bb > 134);
          wait_warp(&sm.v_empty[dst.stage], dst.phase ^ 1u);
          const uint8_t* raw = sm.raw[src.stage] + warp_row * C::kCols + piece * 16 + odd * 8;
          const int other = odd ? -8 : 8;
          uint8_t* out = sm.v[dst.stage];
          uint2 u[2] = {*reinterpret_cast<const uint2*>(raw), *reinterpret_cast<const uint2*>(raw + other)};
#pragma unroll kUnroll
          for (int j = 0; j < kSteps; ++j) {
            const int row = warp_row + j * kStep, src_lane = sub + j * kStep;
            const uint32_t fr = __shfl_sync(0xffffffffu, f, src_lane), f2 = fr | (fr << 16);
            uint2 next[2];
            raw += j + 1 < kSteps ? kStep * C::kCols : 0;
            next[0] = *reinterpret_cast<const uint2*>(raw);
            next[1] = *reinterpret_cast<const uint2*>(raw + other);
            uint32_t w[2][4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              w[e][0] = mul_bf16x2(e4m3_hi_bits(__byte_perm(u[e].x, 0, 0x1404)), f2);
              w[e][1] = mul_bf16x2(e4m3_hi_bits(__byte_perm(u[e].x, 0, 0x3424)), f2);
              w[e][2] = mul_bf16x2(e4m3_hi_bits(__byte_perm(u[e].y, 0, 0x1404)), f2);
              w[e][3] = mul_bf16x2(e4m3_hi_bits(__byte_perm(u[e].y, 0, 0x3424)), f2);
            }
            if (large) {
              const uint32_t b2 = __shfl_sync(0xffffffffu, bb, src_lane);
              const uint32_t s2 = b2 > 134 ? scale_bits(b2) | (scale_bits(b2) << 16) : 0x3f803f80u;
#pragma unroll
              for (int k = 0; k < 8; ++k) w[k >> 2][k & 3] = mul_bf16x2(w[k >> 2][k & 3], s2);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int at = 2 * piece + (odd ^ e);
              *reinterpret_cast<uint4*>(out + (at >> 3) * (TK * 128) + row * 128 + (((at & 7) ^ (row & 7)) << 4)) =
                  make_uint4(w[e][0], w[e][1], w[e][2], w[e][3]);
              u[e] = next[e];
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&sm.v_full[dst.stage]);
            mbar_arrive(&sm.r_empty[src.stage]);
            mbar_arrive(&sm.s_free[vs.stage]);
          }
        }
        if (half == C::kHalves - 1) vs.step();
        src.step();
        dst.step();
      });
    }
  } else if (warp < C::kSoftWarps) {
    // ---------------------------------------------------------------- softmax and output
    if constexpr (C::kSoftRegs > 0) regs_up<C::kSoftRegs>();
    const int blk = warp >> 2, r = tid & 127, lbase = (warp & 3) * 32;
    const uint32_t tl = tmem + ((uint32_t)lbase << 16);
    uint32_t cnt = 0;                  // tiles of this block so far
    uint32_t segments = 0;
    RingPos<C::kVStages> vp;           // block 0 follows the rings
    RingPos<C::kKStages> kp, k_out;    // (two blocks) and hands their stages back, or block 1 does
    RingPos<C::kVStages> v_out, v_at;
    RingPos<Q8 ? C::kScales : 1> sp;   // 8-bit: the scales' ring
    // 16-byte piece p of row rr of this warp's 32 rows in the queries' place: the rows that this warp
    // loads, so warps do not meet in it
    auto row_piece = [&](int rr, int p) {
      constexpr bool kNarrow = Q8 && D == 64;                 // 64-byte query rows, in two parts
      return reinterpret_cast<uint4*>(
          sm.q[blk] + (kNarrow ? (p >> 2) * 8192 + (lbase + rr) * 64 + (((p & 3) ^ ((rr >> 1) & 3)) << 4)
                               : (p >> 3) * 16384 + (lbase + rr) * 128 + (((p & 7) ^ (rr & 7)) << 4)));
    };
    auto load_q = [&](const SegDesc& s) {
      // A warp loads its own 32 rows (lane i knows where row i is), D / 8 lanes a row at a time:
      // 16-byte pieces, swizzled, all in flight at once.
      const int base = s.tile * R + blk * 128 + lbase;
      const int rows = (int)min(32LL, (long long)s.tokens * a.g - base);      // may be negative
      constexpr int kPer = D / 8, kStep = 32 / kPer;
      const int piece = lane % kPer, first = lane / kPer;
      const int mine = min(base + lane, s.tokens * a.g - 1);
      const int t = mine / a.g;
      const long long where = (s.row0 + t) * a.q_ld + (s.head * a.g + (mine - t * a.g)) * a.q_head_ld;
#pragma unroll 8
      for (int j = 0; j < 32 / kStep; ++j) {
        const int row = j * kStep + first;
        const long long w = __shfl_sync(0xffffffffu, where, row);
        cp_async16(smem_u32(row_piece(row, piece)), a.q + w + piece * 8, row < rows);
      }
      cp_async_wait_all();
      __syncwarp();
      if constexpr (Q8) {
        // The rows become their two e4m3 parts (see split_e4m3), which take the same place: the warp
        // has a row before it writes it.  Rows past the tile's last are zeros in either form.
        sm.q_scale[blk][r] = a.scale_log2;
        uint4 ahead = *row_piece(first, piece);
#pragma unroll 1
        for (int j = 0; j * kStep < rows; ++j) {
          const int row = j * kStep + first;
          const uint4 u = ahead;
          ahead = *row_piece(min(row + kStep, 31), piece);
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
          const uint32_t m = __vmaxu2(__vmaxu2(u.x & 0x7fff7fffu, u.y & 0x7fff7fffu),
                                      __vmaxu2(u.z & 0x7fff7fffu, u.w & 0x7fff7fffu));
          uint32_t top = max(m & 0xffffu, m >> 16);
          if constexpr (kPer == 32) {
            top = __reduce_max_sync(0xffffffffu, top);
          } else {
#pragma unroll
            for (int o = kPer / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
          }
          __syncwarp();
          const int bb = scale_byte(top);
          const uint32_t inv = split_factor(bb);
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) split_e4m3(mul_bf16x2(w[e], inv), hi[e], lo[e]);
          if (piece == 0) sm.q_scale[blk][lbase + row] = scale_f32(bb) * a.scale_log2;
          const int col = piece * 8;                                 // byte in the row
          uint8_t* d = sm.q[blk] + (col >> 7) * (128 * 128) +
                       (C::kCols == 128 ? (lbase + row) * 128 + ((((col & 127) >> 4) ^ (row & 7)) << 4)
                                        : (lbase + row) * 64 + (((col >> 4) ^ ((row >> 1) & 3)) << 4)) + (col & 8);
          *reinterpret_cast<uint2*>(d) = make_uint2(hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16));
          *reinterpret_cast<uint2*>(d + C::kQBytes / 2) = make_uint2(lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16));
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.q_ready[blk]);
    };
    auto active = [&](const SegDesc& s) {
      return s.n > 0 && s.rows > 128 * blk;
    };
    {
      const SegDesc& first = seg_wait(seg);
      if (!warp_dead() && active(first)) load_q(first);
    }
    // The warps leave together: none acts on a segment that another did not get.
    bool stop = bar_any(1, C::kSoftWarps * 32, dead());
    while (!stop) {
      const SegDesc& cur = sm.segs[seg.stage];                   // released at the end
      const int n = cur.n;
      if (n < 0) break;
      const int rows = cur.rows;
      const int row = cur.tile * R + blk * 128 + r;              // this thread's row
      const bool live = blk * 128 + r < rows;
      const int before = cur.len - cur.tokens;
      RingPos<kSegs> ahead_seg = seg;
      ahead_seg.step();
      if (!active(cur)) {
        if (cur.owns_empty && live) {
          int tok, head;
          row_of(SeqInfo{cur.row0, cur.tokens, cur.len}, a.g, cur.head, row, &tok, &head);
          uint4* o = reinterpret_cast<uint4*>(a.out + ((long long)tok * a.Hq + head) * D);
          for (int i = 0; i < D / 8; ++i) o[i] = make_uint4(0, 0, 0, 0);
        }
        if (n == 0 && !cur.owns_empty && live)         // an empty share of a split tile
          __stcg(reinterpret_cast<float2*>(Partials<R, D>::ml(a.ws, cta, cur.slot) + 2 * (blk * 128 + r)),
                 make_float2(-INFINITY, 0.f));
        for (int i = 0; i < n; ++i) {                   // the other block's tiles
          if (Q8) sp.step();
          k_out.step();
          v_out.step();
        }
        const SegDesc& next = seg_wait(ahead_seg);
        if (!warp_dead() && active(next)) load_q(next);
      } else {
        const int last_row = cur.tokens * a.g - 1, len = cur.len, ta = cur.ta;
        const int pos = before + min(row, last_row) / a.g;
        const int pos_min = before + min(cur.tile * R + blk * 128, last_row) / a.g;
        const bool releases = blk == (rows > 128 ? 1 : 0);
        float m = -INFINITY, l = 0.f;
        for (int i = 0; i < n; ++i, ++cnt) {
          const int buf = C::kBlocks == 2 ? blk : (int)(cnt & 1u);
          // A parity wait tells a phase from the one before it only when no phase is skipped: so
          // block 0 waits for every stage of the rings, needed or not.  Its p_ready then tells the
          // MMA thread that V(i) (and, with two blocks, K(i + 1)) are there.
          auto rings = [&]() {
            if (C::kBlocks != 2 || blk != 0) return;
            v_at = vp;
            wait_warp(&sm.v_full[vp.stage], vp.phase);
            vp.step();
            if (i == 0) kp.step();
            if (i + 1 < n) {
              wait_warp(&sm.k_full[kp.stage], kp.phase);
              kp.step();
            }
          };
          // D = 128 waits after the exponentials, D = 64, which those bound, before the scores (4096
          // tokens on 16384, before and after: bf16 D = 128 890 and 847 us, D = 64 683 and 749; 8-bit
          // D = 128 1160 and 1107 us, D = 64 922 and 978)
          if (D == 64) rings();
          if (Q8) wait_warp(&sm.s_ready[sp.stage], sp.phase);
          wait_warp(&sm.s_full[buf], (C::kBlocks == 2 ? cnt : cnt >> 1) & 1u);
          fence_after_sync();
          if (C::kBlocks == 2 && releases && warp == 4 * blk && lane == 0) {
            // the last block's scores are there: K(i) has been read, and V(i - 1)
            mbar_arrive(&sm.k_empty[k_out.stage]);
            if (i > 0) mbar_arrive(&sm.v_empty[v_out.stage]);
          }
          k_out.step();
          if (i > 0) v_out.step();
          const uint32_t s_addr = tl + buf * 128;
          const int k0 = (ta + i) * TK;
          const bool partial = k0 + TK - 1 > pos_min;
          const int lim = pos - k0;                               // columns 0..lim are seen
          // 8-bit, D = 256: S has two buffers, so the products run ahead, and the scores are read twice,
          // 32 at a time in rolled loops, which leaves the instruction caches to the conversion (4096
          // tokens on 16384: 1388 -> 1219 us).  Else once, into registers: with two blocks a block's
          // products wait for its softmax (read twice, D = 128: 1107 -> 1411 us; one block, 32 rows on
          // 8000 keys: 426 -> 434 us).
          constexpr bool kTwice = Q8 && D == 256;
          uint32_t v[kTwice ? 32 : 128];
          float xs[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
          const float scale = Q8 ? sm.q_scale[blk][r] : a.scale_log2;
          // 8-bit: n / 32 scores of 32, each times its key's scale (the row's is in the softmax scale)
          // with the next 32 under way; a hidden key's scale may be anything, so hide after scaling
          auto scores = [&](int first, auto count) {
            constexpr int kCount = decltype(count)::value;
            if constexpr (!Q8) {
#pragma unroll
              for (int cc = 0; cc < kCount; ++cc) tmem_ld32_nw(s_addr + cc * 32, v + cc * 32);
              tmem_wait_ld();
#pragma unroll
              for (int cc = 0; cc < 2 * kCount; ++cc) reg_fence16(v + cc * 16);
            } else {
              const float4* f = reinterpret_cast<const float4*>(sm.k_scale[sp.stage] + first);
              tmem_ld32_nw(s_addr + first, v);
#pragma unroll
              for (int cc = 0; cc < kCount; ++cc) {
                float4 g[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) g[e] = f[cc * 8 + e];
                tmem_wait_ld();
                reg_fence16(v + cc * 32);
                reg_fence16(v + cc * 32 + 16);
                if (cc + 1 < kCount) tmem_ld32_nw(s_addr + first + (cc + 1) * 32, v + (cc + 1) * 32);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  uint32_t* y = v + cc * 32 + 4 * e;
                  float z[4];
                  unpair(mul2(pair(__uint_as_float(y[0]), __uint_as_float(y[1])), pair(g[e].x, g[e].y)), z[0], z[1]);
                  unpair(mul2(pair(__uint_as_float(y[2]), __uint_as_float(y[3])), pair(g[e].z, g[e].w)), z[2], z[3]);
#pragma unroll
                  for (int k = 0; k < 4; ++k) y[k] = __float_as_uint(z[k]);
                }
              }
            }
            if (partial) {
#pragma unroll
              for (int e = 0; e < 32 * kCount; ++e)
                if (first + e > lim) v[e] = 0xff800000u;
            }
          };
          auto maxima = [&](int n) {
#pragma unroll
            for (int e = 0; e < n; e += 8)
#pragma unroll
              for (int j = 0; j < 4; ++j)
                xs[j] = fmaxf(xs[j], fmaxf(__uint_as_float(v[e + 2 * j]), __uint_as_float(v[e + 2 * j + 1])));
          };
          if constexpr (kTwice) {
#pragma unroll 1
            for (int k = 0; k < TK; k += 32) {
              scores(k, Int<1>{});
              maxima(32);
            }
          } else {
            scores(0, Int<4>{});
            maxima(TK);
          }
          const float x = fmaxf(fmaxf(xs[0], xs[1]), fmaxf(xs[2], xs[3])) * scale;
          if (__any_sync(0xffffffffu, x > m + 8.f)) {
            // only a row whose own maximum asks for it: no bit of a row depends on another's keys
            const float mn = x > m + 8.f ? x : m;
            const float f = mn == m ? 1.f : ex2f(m - mn);
            m = mn;
            l *= f;
            if (i > 0) {
              // two blocks: s_full of this tile came after the product of the one before
              if (C::kBlocks == 1) wait_warp(&sm.o_done[blk], (cnt - 1) & 1u);
              fence_after_sync();
#pragma unroll 1
              for (int d = 0; d < D; d += 16) {
                float o[16];
                tmem_ld16(tl + C::kO + blk * D + d, o);
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] *= f;
                tmem_st16_nw(tl + C::kO + blk * D + d, o);
              }
              tmem_wait_st();
            }
          }
          const float ref = m == -INFINITY ? 0.f : m;
          const uint64_t sc2 = pair(scale, scale), ref2 = pair(-ref, -ref);
          uint64_t l2[2] = {pair(l, 0.f), pair(0.f, 0.f)};
          auto exps = [&](const uint32_t* y, uint32_t at) {        // of 16 scores
            uint32_t w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              float p0, p1;
              unpair(fma2(pair(__uint_as_float(y[2 * e]), __uint_as_float(y[2 * e + 1])), sc2, ref2), p0, p1);
              p0 = ex2f(p0);
              p1 = ex2f(p1);
              l2[e & 1] = add2(l2[e & 1], pair(p0, p1));
              w[e] = pack2(p0, p1);
            }
            tmem_st8w_nw(at, w);
          };
          if constexpr (kTwice) {
#pragma unroll 1
            for (int k = 0; k < TK; k += 32) {
              scores(k, Int<1>{});
              exps(v, s_addr + k / 2);                             // the columns of scores read before
              exps(v + 16, s_addr + k / 2 + 8);
            }
          } else {
#pragma unroll
            for (int cc = 0; cc < 8; ++cc) exps(v + cc * 16, s_addr + cc * 8);
          }
          if (Q8) sp.step();
          {
            float l0, l1, l3, l4;
            unpair(l2[0], l0, l1);
            unpair(l2[1], l3, l4);
            l = (l0 + l1) + (l3 + l4);
          }
          if (D != 64) rings();
          // for its parity's sake every tile: one block's s_full does not imply the product before
          if (C::kBlocks == 1 && i > 0) wait_warp(&sm.o_done[blk], (cnt - 1) & 1u);
          if (C::kBlocks == 1) {         // (one block: two V stages hold one tile, which comes late)
            v_at = vp;
            for (int h = 0; h < C::kHalves; ++h, vp.step()) wait_warp(&sm.v_full[vp.stage], vp.phase);
          }
          if (blk == 0 && partial) {
            // a causal-edge tile's values: zero past the end, zero and noted where not finite
            for (int h = 0; h < C::kHalves; ++h, v_at.step()) {
              // keys from the first row's position on (earlier ones are seen by all rows)
              const int j0 = max(0, pos_min + 1 - k0), j1 = TK;
              constexpr int kPer = C::kCols / 8;
              const int piece = r % kPer;
              for (int j = j0 + r / kPer; j < j1; j += 128 / kPer) {
                uint4* p = reinterpret_cast<uint4*>(sm.v[v_at.stage] + (piece >> 3) * (TK * 128) + j * 128 +
                                                    (((piece & 7) ^ (j & 7)) << 4));
                if (k0 + j >= len) {
                  *p = make_uint4(0, 0, 0, 0);
                  continue;
                }
                const uint4 u = *p;
                uint32_t w[4] = {u.x, u.y, u.z, u.w};
                uint32_t hit = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) hit |= ((w[e] & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
                if (hit) {
#pragma unroll
                  for (int e = 0; e < 8; ++e)
                    if (((w[e >> 1] >> (16 * (e & 1))) & 0x7f80u) == 0x7f80u) {
                      const uint32_t y = (w[e >> 1] >> (16 * (e & 1))) & 0xffffu;
                      w[e >> 1] &= e & 1 ? 0x0000ffffu : 0xffff0000u;
                      if constexpr (Q8) atomicMin((int*)&sm.bad[h * C::kCols + piece * 8 + e], k0 + j);
                      else Notes::add(&sm.bad[h * C::kCols + piece * 8 + e], y, k0 + j - pos_min);
                    }
                  sm.any_bad = 1;
                  *p = make_uint4(w[0], w[1], w[2], w[3]);
                }
              }
            }
            fence_proxy_async_smem();
          }
          __syncwarp();
          tmem_wait_st();
          fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.p_ready[blk]);
        }
        int tok = 0, head = 0;
        row_of(SeqInfo{cur.row0, cur.tokens, cur.len}, a.g, cur.head, min(row, last_row), &tok, &head);
        if (a.gate && cur.whole) {
          // every product with these queries is through: their place takes the gate in
          const long long grow = tok * a.gate_ld + head * a.gate_head_ld;
          constexpr int kPer = D / 8, kStep = 32 / kPer;
          const int piece = lane % kPer, first = lane / kPer;
#pragma unroll 8
          for (int j = 0; j < 32 / kStep; ++j) {
            const int rr = j * kStep + first;
            const long long at = __shfl_sync(0xffffffffu, grow, rr);
            cp_async16(smem_u32(row_piece(rr, piece)), a.gate + at + piece * 8, true);
          }
        }
        // two blocks: one phase of o_done a segment
        wait_warp(&sm.o_done[blk], (C::kBlocks == 2 ? segments++ : cnt - 1) & 1u);
        fence_after_sync();
        if (C::kBlocks == 2) {
          if (releases && warp == 4 * blk && lane == 0) mbar_arrive(&sm.v_empty[v_out.stage]);
          v_out.step();
        }
        const bool whole = cur.whole, bad = *(volatile int*)&sm.any_bad != 0;
        const float inv = !whole ? 1.f : l == 0.f ? 0.f : 1.0f / l;
        const int pr = blk * 128 + r;
        const int rows32 = min(32, rows - blk * 128 - lbase);
        auto read_o = [&](int d, uint32_t* o) {
          tmem_ld32_nw(tl + C::kO + blk * D + d, o);
          tmem_wait_ld();
          reg_fence16(o);
          reg_fence16(o + 16);
          if (bad) {
            if constexpr (Q8) {
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if ((int)sm.bad[d + e] <= pos) o[e] = 0x7fffffffu;
            } else {
              const int mine = pos - (cur.len - cur.tokens + min(cur.tile * R, last_row) / a.g);
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const uint32_t notes = sm.bad[d + e];
                float y = __uint_as_float(o[e]);           // (infinities of both signs add up to NaN)
                if (Notes::first(notes, 0) <= mine) y += INFINITY;
                if (Notes::first(notes, 1) <= mine) y -= INFINITY;
                o[e] = Notes::first(notes, 2) <= mine ? 0x7fffffffu : __float_as_uint(y);
              }
            }
          }
        };
        if (whole) {
          // The queries have been read: the place of this warp's 32 rows (a piece is 16 bytes) took
          // the gate in meanwhile, and turns rows held by a thread each into rows of consecutive lanes.
          if (a.gate) {
            cp_async_wait_all();
            __syncwarp();
          }
#pragma unroll 1
          for (int d = 0; d < D; d += 32) {
            uint32_t o[32];
            read_o(d, o);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint4* at = row_piece(lane, d / 8 + e);
              float y[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) y[k] = __uint_as_float(o[8 * e + k]) * inv;
              if (a.gate) {
                const uint4 z = *at;
                const uint32_t zw[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
                for (int k = 0; k < 8; ++k)
                  y[k] *= gate_of(__uint_as_float(k & 1 ? zw[k >> 1] & 0xffff0000u : zw[k >> 1] << 16));
              }
              *at = make_uint4(pack2(y[0], y[1]), pack2(y[2], y[3]), pack2(y[4], y[5]), pack2(y[6], y[7]));
            }
          }
          __syncwarp();
          const long long orow = ((long long)tok * a.Hq + head) * D;
          constexpr int kPer = D / 8, kStep = 32 / kPer;
          const int piece = lane % kPer, first = lane / kPer;
#pragma unroll 8
          for (int j = 0; j < 32 / kStep; ++j) {
            const int rr = j * kStep + first;
            const long long at = __shfl_sync(0xffffffffu, orow, rr);
            const uint4 y = *row_piece(rr, piece);
            if (rr < rows32) *reinterpret_cast<uint4*>(a.out + at + piece * 8) = y;
          }
          __syncwarp();
        } else {
          float4* part = reinterpret_cast<float4*>(Partials<R, D>::rows(a.ws, cta, cur.slot)) + pr;
#pragma unroll 1
          for (int d = 0; d < D; d += 32) {
            uint32_t o[32];
            read_o(d, o);
            if (live)
#pragma unroll
              for (int e = 0; e < 32; e += 4)
                __stcg(part + (size_t)(d + e) / 4 * R,
                       make_float4(__uint_as_float(o[e]), __uint_as_float(o[e + 1]), __uint_as_float(o[e + 2]),
                                   __uint_as_float(o[e + 3])));
            __syncwarp();
          }
        }
        if (!whole && live) {
          // a NaN sum must survive the merge even when its reference never left -infinity
          __stcg(reinterpret_cast<float2*>(Partials<R, D>::ml(a.ws, cta, cur.slot) + 2 * pr),
                 make_float2(l != l ? INFINITY : m, l));
        }
        fence_before_sync();           // O has been read before the next segment's p_ready
        __syncwarp();
        const SegDesc& next = seg_wait(ahead_seg);
        if (!warp_dead() && active(next)) load_q(next);
      }
      // both blocks are done with the notes on non-finite values
      if (bar_any(1, C::kSoftWarps * 32, *(volatile int*)&sm.any_bad != 0 || dead())) {
        for (int i = tid; i < D; i += C::kSoftWarps * 32) sm.bad[i] = Q8 ? INT32_MAX : Notes::kNone;
        if (tid == 0) sm.any_bad = 0;
        stop = bar_any(1, C::kSoftWarps * 32, dead());
      }
      seg_done(seg);
    }
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  if (tid == 0 && dead()) set_status(c.status, GDN_STATUS_TIMEOUT);
  if (warp == C::kMmaWarp) tmem_dealloc(tmem, 512);
}

template <int D, bool Q8, int B>
int launch_chunk(const KvView& c, const KvBatchView& b, const AttnArgs& a, int sms, cudaStream_t stream) {
  using C = ChunkCfg<D, Q8, B>;
  constexpr size_t smem = sizeof(ChunkSmem<D, Q8, B>);
  static_assert(smem <= 232448, "shared memory of a CTA");
  static OncePerDevice once;
  int rc = raise_smem(once, chunk_kernel<D, Q8, B>, smem);
  if (rc != GDN_OK) return rc;
  KvMaps maps;
  const int P = 1 << c.page_shift;
  if (!make_tile_maps(c, P < kKeys ? P : kKeys, Q8 ? C::kCols : 64, &maps)) return GDN_ERR_CUDA;
  // What a tile of rows costs beside its keys, in keys (the gate's share grows with the columns), and
  // the fewest keys worth a piece of their own (14 tokens on 8481: 21.5 us at 512, 24.2 at 256).  12
  // sequences of 3 to 1456 new tokens at 512, 640, 768, 896, 1024 keys: D = 256 bf16 97, 92, 94, 96,
  // 98 us, 8-bit 139, 133, 128, 128, 131, gated -, 162, 145, 142, 138; D = 128 bf16 54, 56, 58, -, 58.
  // A tile's time beside its keys alone (5 and 1 tiles a CTA compared): D = 256 bf16 441 keys' time, 8-bit
  // 724, a gate 180 more; D = 128 716 and 824.
  const int base = D < 256 ? 512 : Q8 ? 896 : 640;
  const int grid = sms, fix = (base + (a.gate ? D / 2 : 0)) * a.g;
  const int least = 512 * a.g;
  rc = launch_dependent(chunk_kernel<D, Q8, B>, dim3((unsigned)grid), C::kThreads, smem, stream, c, b, a, grid,
                            fix, least, maps);
  if (rc != GDN_OK) return rc;
  return launch_dependent(merge_kernel<C::kRows, D>, dim3((unsigned)(6 * sms)), kMergeWarps * 32, 0, stream, a, grid);
}

size_t chunk_ws_bytes(int D, int sms) {
  return D == 64 ? Partials<256, 64>::bytes(sms)
       : D == 128 ? Partials<256, 128>::bytes(sms)
                  : Partials<128, 256>::bytes(sms);
}

template <int D, int B>
int launch_chunk(const KvView& c, const KvBatchView& b, const AttnArgs& a, int sms, cudaStream_t stream) {
  return c.ks != nullptr ? launch_chunk<D, true, B>(c, b, a, sms, stream) : launch_chunk<D, false, B>(c, b, a, sms, stream);
}

int launch_chunk(const KvView& c, const KvBatchView& b, const AttnArgs& a, int sms, cudaStream_t stream) {
  // One block where no tile has rows for a second (64 sequences of 8 tokens and 8000 keys, 32 rows:
  // bf16 D = 128 374 us with two, 359 with one; 8-bit 464 and 426).
  const bool one = (long long)(b.max_tokens > 0 ? b.max_tokens : b.total) * a.g <= 128;
  if (c.D == 64) return one ? launch_chunk<64, 1>(c, b, a, sms, stream) : launch_chunk<64, 2>(c, b, a, sms, stream);
  if (c.D == 128) return one ? launch_chunk<128, 1>(c, b, a, sms, stream) : launch_chunk<128, 2>(c, b, a, sms, stream);
  return launch_chunk<256, 1>(c, b, a, sms, stream);
}

}  // namespace attn
}  // namespace gdn
