// gdn_attn_rows.cu -- attention of a few query rows per key/value head over the paged cache: the
// decode step (one token per sequence), and short runs of new tokens.
//
//   o_r = sum_j p_rj v_j / sum_j p_rj,   p_rj = 2^(s_rj - m_r),   s_rj = scale log2(e) q_r . k_j
//
// with one pass over the keys: m_r is a reference that follows the running maximum (it only has to
// stay within 2^8 of it, or 2^4, so the accumulator is rescaled when a maximum outgrows it by that much,
// not at every step) and every sum is f32.
//
// What bounds it: the cache is read once, 2 D elements per key and head, for 8 or 16 rows, so the
// floor is its bytes at the HBM rate.  Everything else must hide behind the loads:
//  * two producer warps (keys, values) keep a ring of stages full with TMA tensor copies (a box is a
//    page's part of a stage, 128-byte swizzled), page numbers fetched one stage ahead;
//  * each consumer warp takes its own 16 or 32 keys of a stage and runs its own softmax, so warps
//    meet only at the end of a tile, where their results are added in a fixed order;
//  * the products are MMAs on registers, in the transposed form: S^T = K Q^T and O^T = V^T P^T have
//    the keys (columns) as their 16 rows and 8 query rows as their columns, which fits the groups of
//    4 and 8 that share a key/value head without empty rows (the other way round half the MMAs and
//    half the accumulators were).  P^T becomes an operand by a transposing register move.  The
//    128-row tcgen05 shape would run 15/16 empty, needs the probabilities to cross TMEM, and could
//    not be faster than the loads;
//  * 8-bit caches: the keys' codes are e4m3 MMA operands as they are (the queries as two e4m3
//    parts, whose sum is exact), their scales applied to the scores; the values' codes become f16 by
//    the conversion instruction, their scales applied to the probabilities.
// Measured (the copy bandwidth is 6.69 TB/s): 64 sequences of 8000 positions, 8 x 128, 4 rows, bf16
// 302 to 310 us, 6.8 TB/s, 8-bit 167 to 171 us, 6.2 TB/s; ragged 8-bit batch of 64, 200 to 16,000 positions, 87 us,
// 5.7 TB/s; two sequences of 100,000 to 131,000, 2 x 256, bf16, 76 us, 5.9 TB/s.  16 rows on 8 bits:
// 257 us, 4.1 TB/s, bound by the instructions of two row tiles.
// Fewer bits: the probabilities become bf16, or f16 over 8-bit values (see kNear), as the matrix
// instructions' operands are; their sum takes them unrounded, and all sums are f32.
#include "gdn_attn.cuh"
#include "gdn_tmap.h"

namespace gdn {

using namespace tc;

namespace attn {


// NT: tiles of 8 query rows.
template <int D, bool Q8, int NT>
struct RowsCfg {
  static constexpr int kRows = 8 * NT;
  static constexpr int kElem = Q8 ? 1 : 2;
  // D = 256: twice the accumulators and bytes, so one CTA of an SM, with more warps where they fit
  static constexpr int kCtas = D == 256 ? 1 : 2;
  static constexpr int kConsumers = D == 256 && Q8 && NT == 1 ? 8 : 4;
  static constexpr int kThreads = (kConsumers + 2) * 32;
  // Groups of 16 keys that a warp takes of a stage: with half the bytes to wait for, an 8-bit cache
  // wants the chains of two side by side (16 rows on 64 x 8000 keys: D = 64 196 us with one, 160 with
  // two, D = 256 162 and 136), as far as two CTAs' registers go: with D = 128 and 16 rows they spill
  // (285 us with two, 258 with one).
  static constexpr int kGroups = Q8 && kConsumers == 4 && !(NT == 2 && D == 128) ? 2 : 1;
  static constexpr int kKeys = 16 * kGroups * kConsumers;        // of a stage
  static constexpr int kHalfBytes = kKeys * D * kElem;           // a stage's keys
  static constexpr int kStageBytes = 2 * kHalfBytes;
  static constexpr int kRing = kCtas == 1 ? 196608 : 98304;
  static constexpr int kStages = kRing / kStageBytes;
  static constexpr bool kQRegs = NT * D <= 128;                  // query operands stay in registers
  static constexpr int kBox = D * kElem >= 128 ? 128 : 64;       // swizzle span, bytes
  static constexpr int kQLd = 2 * D + 16;                        // bytes of a staged query row
  // columns merged at a time, as the shared memory beside the ring allows
  static constexpr int kChunk = NT == 1 ? (D == 256 && !Q8 ? 128 : 64) : D / (Q8 && D > 64 ? 8 : 4);
  static constexpr int kReaders = kConsumers + 1;                // warps that read a published segment
  static constexpr int kMLd = kChunk + 4;
};

template <int D, bool Q8, int NT>
struct __align__(1024) RowsSmem {
  using C = RowsCfg<D, Q8, NT>;
  uint8_t ring[C::kStages][C::kStageBytes];
  uint8_t scales[Q8 ? C::kStages : 1][2][C::kKeys];     // scale bytes of a stage's keys and values
  uint8_t q[C::kRows][C::kQLd];                         // the rows, as copied
  uint2 q_part[Q8 ? D / 16 : 1][NT][32];                // 8-bit caches: operands of their two e4m3 parts
  float q_scale[C::kRows];
  float o[C::kConsumers][C::kRows][C::kMLd];
  float ml[C::kConsumers][C::kRows][2];
  LineScan<C::kRows, C::kThreads> scan;
  uint64_t full[C::kStages];
  uint64_t empty[C::kStages];
  SegDesc segs[kSegs];
  uint64_t seg_full[kSegs], seg_empty[kSegs];
  uint64_t q_full, q_empty;
  int dead;
};

// How far (as a power of two) a maximum may outgrow its reference.  f32 and bf16 hold 2^8 times the
// reference's probability alike; with an 8-bit cache the probabilities become f16, to which the
// factor 2^kUp moves them.
template <bool Q8>
constexpr int kLag = Q8 ? 4 : 8;
constexpr int kUp = 15 - kLag<true>;
// Scale byte whose unit 2^(b - 127 - kUp) is 1, and the least that is used as a unit.
constexpr int kUnitOne = 127 + kUp, kLeastUnit = kUnitOne - 40;
// How far below the unit a scale may lie for f16 products, and how many keys a warp may add to a tile
// so: a probability p becomes p 2^(b - unit + kUp), at least 2 p, which f16 holds to 2^-11 of itself
// from 2^-14 up and to 2^-25 below, so all small ones together are off by kMostNear 2^-26 = 2^-10 of
// the row's sum, which is at least 1.  (64 x 8000 keys of 8 x 128, 4 rows: 167 us where all keys are
// so, 193 us where none are; D = 64 102 and 130; two tokens, 16 rows 256 and 322.)
constexpr uint32_t kNear = kUp - 1;
constexpr int kMostNear = 1 << 16;

__device__ __forceinline__ void mma16816(float* c, const uint4& a, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816_f16(float* c, const uint4& a, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16832_e4m3(float* c, const uint4& a, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}
// Two 16 x 16 byte matrices, transposed: lane (n, t) gets columns n and n + 8 of the first, then of
// the second, each word four consecutive rows 4 t .. 4 t + 3.
__device__ __forceinline__ void ldsm2t_b8(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// The e4m3 codes of w's low or high half as f16 values.
__device__ __forceinline__ uint32_t e4m3_to_f16x2(uint16_t h) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(h));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// The 8 x 8 matrix of 16-bit elements that the warp holds (lane (g, t): row g, columns 2 t, 2 t + 1),
// transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ float lds_bf16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];\n" : "=h"(v) : "r"(addr) : "memory");
  return __uint_as_float((uint32_t)v << 16);
}
// The sign bits of the halves that hold an infinity or a NaN, of two bf16.
__device__ __forceinline__ uint32_t non_finite(uint32_t w) { return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u; }
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;\n" ::"r"(id), "r"(threads) : "memory");
}

// 16 bytes (zeros when !fill) by cp.async, and one arrival on bar when they are there.
__device__ __forceinline__ void cp_async16_mbar(uint32_t dst, const void* src, bool fill, uint64_t* bar) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;\n"
               "cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%3];\n" ::"r"(dst),
               "l"(src), "r"(fill ? 16 : 0), "r"(smem_u32(bar))
               : "memory");
}

template <int D, bool Q8, int NT>
__global__ void __launch_bounds__(RowsCfg<D, Q8, NT>::kThreads, RowsCfg<D, Q8, NT>::kCtas)
rows_kernel(const KvView c, const KvBatchView b, const AttnArgs a, int grid, int fix, int least,
            const __grid_constant__ KvMaps maps) {
  using C = RowsCfg<D, Q8, NT>;
  constexpr int R = C::kRows, TK = C::kKeys, NC = C::kConsumers * 32;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  RowsSmem<D, Q8, NT>& sm = *reinterpret_cast<RowsSmem<D, Q8, NT>*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&sm.full[i], Q8 ? 2 + TK / 8 : 2);
      mbar_init(&sm.empty[i], C::kConsumers);
    }
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(&sm.seg_full[i], 1);
      mbar_init(&sm.seg_empty[i], C::kReaders);
    }
    mbar_init(&sm.q_full, 1);
    mbar_init(&sm.q_empty, C::kConsumers);
    sm.dead = 0;
    mbar_fence_init();
  }
  // rows past a tile's last are multiplied too: nothing comes of them, but what they hold must not
  // differ from run to run (all rows of a warp move their references together)
  for (int i = tid; i < R * C::kQLd / 16; i += C::kThreads)
    reinterpret_cast<uint4*>(sm.q)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  pdl_begin();
  const RowRange batch = batch_rows(b);
  bool bad = false;
  Pieces pieces;
  const int cta = blockIdx.x;
  locate_piece<R, C::kThreads>(c, b, a.g, fix, grid, least, cta, &pieces, &sm.scan, &bad);
  zero_outside(a, b, D, batch, &bad);
  if (bad) set_status(c.status, GDN_STATUS_BAD_SEQLENS);
  if (cta >= pieces.count) {
    if (tid == 0) Partials<R, D>::note(a.ws, grid, cta, a.g, nullptr, 0);
    return;
  }
  int seg = 0;                    // place in the ring of segments
  uint32_t seg_phase = 0;
  auto seg_step = [&]() {
    if (++seg == kSegs) { seg = 0; seg_phase ^= 1u; }
  };

  if (warp >= C::kConsumers) {
    // ---------------------------------------------------------------- producers
    // Copies of one warp go out one after another (some 150 cycles each), hence a warp for the keys
    // and one for the values.
    const bool values = warp > C::kConsumers;
    int stage = 0;
    uint32_t phase = 0, q_phase = 0;
    SegIter<R, TK> it;
    Segment sg;
    sg.split = false;
    bool first = true, alive = true;
    if (!values) it.start(&b, c.page_shift, c.H, a.g, fix, pieces, cta, sm.scan.at);
    while (alive) {
      // the keys' producer walks the piece, for all
      SegDesc d = {};
      d.n = -1;
      if (!values) {
        bool more = it.next(&sg);
        while (more && idle(sg)) more = it.next(&sg);
        if (more) d = describe<R>(sg, a.g);
        alive = wait_bar(&sm.seg_empty[seg], seg_phase ^ 1u, &sm.dead, c.status);
        if (alive && lane == 0) {
          sm.segs[seg] = d;
          mbar_arrive(&sm.seg_full[seg]);
        }
      } else {
        alive = wait_bar(&sm.seg_full[seg], seg_phase, &sm.dead, c.status);
        d = sm.segs[seg];
        __syncwarp();
        if (alive && lane == 0) mbar_arrive(&sm.seg_empty[seg]);
      }
      __syncwarp();
      seg_step();
      if (!alive || d.n < 0) break;
      if (d.n == 0) continue;
      const int tb = d.ta + d.n, keys = d.keys;
      // The queries' place is free when the tile before has been scored: after what the ring takes, or
      // (the piece's first tile) at once (23 sequences of up to 1054, 64 heads over 8 x 64 of 8 bits: 17.9 -> 15.8 us).
      auto load_queries = [&]() {
        alive = wait_bar(&sm.q_empty, q_phase ^ 1u, &sm.dead, c.status);
        if (!alive) return;
        q_phase ^= 1u;
        if (lane == 0) mbar_arrive_expect_tx(&sm.q_full, (uint32_t)d.rows * 2 * D);
        __syncwarp();
        if (lane < d.rows) {
          int tok, head;
          row_of(SeqInfo{d.row0, d.tokens, d.len}, a.g, d.head, d.tile * R + lane, &tok, &head);
          bulk_g2s(sm.q[lane], a.q + tok * a.q_ld + head * a.q_head_ld, 2 * D, &sm.q_full);
        }
        __syncwarp();
      };
      const int q_after = first ? -1 : min(tb, d.ta + C::kStages - 1) - 1;
      if (values && first) load_queries();
      first = false;
      const int* table = b.table + (long long)d.seq * b.table_ld;
      // Lane i < TK / 16 looks after the i-th 16 keys of a stage: their page, fetched a stage ahead,
      // the box that begins with them (a box is a page's part of the stage), and their scale bytes.
      constexpr int kLanes = TK / 16;
      const int box = min(1 << c.page_shift, TK);
      int k0 = d.ta * TK + (lane % kLanes) * 16;
      int page = k0 < keys ? __ldg(table + (k0 >> c.page_shift)) : 0;
      for (int i = d.ta; i < tb && alive; ++i) {
        const int k1 = k0 + TK;
        int page_next = 0;
        if (i + 1 < tb && k1 < keys) page_next = __ldg(table + (k1 >> c.page_shift));
        alive = wait_bar(&sm.empty[stage], phase ^ 1u, &sm.dead, c.status);
        if (!alive) break;
        uint64_t* full = &sm.full[stage];
        const int live = (min(TK, keys - i * TK) + box - 1) / box;            // boxes
        if (lane == 0) mbar_arrive_expect_tx(full, (uint32_t)(live * box * D * C::kElem));
        __syncwarp();
        if (k0 < keys && (page < 0 || page >= c.num_pages)) {
          set_status(c.status, GDN_STATUS_PAGE_RANGE);
          page = c.num_pages;            // outside the map: the copy fills zeros
        }
        const int off = k0 & ((1 << c.page_shift) - 1);
        if (lane < kLanes && k0 < keys && ((lane * 16) & (box - 1)) == 0)
          tma_load_5d(sm.ring[stage] + (values ? C::kHalfBytes : 0) + lane * 16 * D * C::kElem,
                      values ? &maps.v : &maps.k, 0, off, 0, d.head, page, full);
        if (Q8 && lane < kLanes) {
          const bool in = k0 < keys && page < c.num_pages;
          const uint8_t* src = values ? c.vs : c.ks;
          if (in) src += (((long long)page * c.H + d.head) << c.page_shift) + off;
          cp_async16_mbar(smem_u32(&sm.scales[stage][values][lane * 16]), src, in, full);
        }
        __syncwarp();
        if (values && i == q_after) load_queries();
        page = page_next;
        k0 = k1;
        if (++stage == C::kStages) { stage = 0; phase ^= 1u; }
      }
    }
    // no copy outlives the CTA, whoever has stopped waiting for it
    asm volatile("cp.async.wait_all;\n" ::: "memory");
    drain_ring<C::kStages>(sm.full, stage, phase);
    if (values) mbar_wait(&sm.q_full, q_phase ^ 1u, kDrainNs);
    // the piece's last tile may be shared with the next ones
    if (!values && lane == 0)
      Partials<R, D>::note(a.ws, grid, cta, a.g, &sg, alive && sg.split ? it.sharing(sg.nt) : 0);
    return;
  }

  // ------------------------------------------------------------------ consumers
  const int t = lane & 3, g = lane >> 2;
  constexpr int G = C::kGroups;
  // a box of `box` keys is [column blocks][box][128 bytes]
  const int box = min(1 << c.page_shift, TK);
  const uint32_t blk_bytes = box * C::kBox;
  uint32_t at[G];                                        // this warp's groups in a stage's half
#pragma unroll
  for (int u = 0; u < G; ++u) {
    const int k = (warp * G + u) * 16;
    at[u] = (k / box) * (box * D * C::kElem) + (k % box) * C::kBox;
  }
  int stage = 0;
  uint32_t phase = 0, q_phase = 0;
  bool alive = true;
  SegDesc sg;
  // The next segment, for all consumers or for none.
  auto next_segment = [&]() {
    alive = wait_bar(&sm.seg_full[seg], seg_phase, &sm.dead, c.status) && alive;
    sg = sm.segs[seg];
    __syncwarp();
    if (alive && lane == 0) mbar_arrive(&sm.seg_empty[seg]);
    seg_step();
    return !bar_any(1, NC, !alive) && sg.n >= 0;
  };
  for (bool more = next_segment(); more; more = next_segment()) {
    const SeqInfo info{sg.row0, sg.tokens, sg.len};
    const int row_base = sg.tile * R, rows = sg.rows, keys = sg.keys;
    if (sg.n == 0) {
      if (sg.owns_empty) {
        for (int i = tid; i < rows * (D / 8); i += NC) {
          int tok, head;
          row_of(info, a.g, sg.head, row_base + i / (D / 8), &tok, &head);
          *reinterpret_cast<uint4*>(a.out + ((long long)tok * a.Hq + head) * D + (i % (D / 8)) * 8) =
              make_uint4(0, 0, 0, 0);
        }
      } else {                                             // an empty share of a split tile
        for (int i = tid; i < rows; i += NC)
          __stcg(reinterpret_cast<float2*>(Partials<R, D>::ml(a.ws, cta, sg.slot) + 2 * i), make_float2(-INFINITY, 0.f));
      }
      continue;
    }
    const int before = info.len - info.tokens;          // position of the first new token
    alive = alive && wait_one(&sm.q_full, q_phase, &sm.dead, c.status);
    q_phase ^= 1u;
    if constexpr (Q8) {
      // A warp splits some rows into their parts (see split_e4m3), a lane some columns of them.
      constexpr int kEl = D == 256 ? 8 : 4;              // columns of a lane (D = 64: half the lanes)
      const int d0 = lane * kEl;
#pragma unroll
      for (int j = 0; j < R / C::kConsumers; ++j) {
        const int r = warp * (R / C::kConsumers) + j;
        uint32_t w[kEl / 2], top = 0;
#pragma unroll
        for (int e = 0; e < kEl / 4; ++e) {
          const uint2 u = d0 < D ? reinterpret_cast<const uint2*>(sm.q[r] + 2 * d0)[e] : make_uint2(0, 0);
          w[2 * e] = u.x;
          w[2 * e + 1] = u.y;
        }
#pragma unroll
        for (int e = 0; e < kEl / 2; ++e) top = max(top, max(w[e] & 0x7fffu, (w[e] >> 16) & 0x7fffu));
        top = __reduce_max_sync(0xffffffffu, top);
        const int bb = scale_byte(top);
        const uint32_t inv = split_factor(bb);
        if (lane == 0) sm.q_scale[r] = scale_f32(bb) * a.scale_log2;
#pragma unroll
        for (int e = 0; e < kEl / 4; ++e) {
          uint32_t hi[2], lo[2];
#pragma unroll
          for (int k = 0; k < 2; ++k)
            split_e4m3(mul_bf16x2(w[2 * e + k], inv), hi[k], lo[k]);
          if (d0 < D) {
            const int d = d0 + 4 * e, ks = d / 64 * 2 + ((d >> 3) & 1), ln = (r & 7) * 4 + ((d >> 4) & 3);
            uint32_t* at0 = &sm.q_part[ks][r >> 3][ln].x + ((d >> 2) & 1);
            at0[0] = hi[0] | (hi[1] << 16);
            at0[D / 32 * NT * 64] = lo[0] | (lo[1] << 16);
          }
        }
      }
      bar_sync(1, NC);
      if (alive && lane == 0) mbar_arrive(&sm.q_empty);
    }
    // Query operands of k-step ks and row tile nt: column g is the row, and the columns of the
    // k-step are 16 ks + 2 t, + 1, + 8, + 9; for 8-bit keys (k-step (part, ks)) the eight from
    // 64 (ks / 2) + 16 t + 8 (ks % 2) on, so that a lane's columns of a key are sixteen together.
    constexpr int kSteps = D / 16;                       // of a score: D / 32 for each part, or D / 16
    auto query = [&](int ks, int nt) {
      if constexpr (!Q8) {
        const uint8_t* q = sm.q[8 * nt + g] + 2 * (16 * ks + 2 * t);
        return make_uint2(*reinterpret_cast<const uint32_t*>(q), *reinterpret_cast<const uint32_t*>(q + 16));
      } else {
        return sm.q_part[ks][nt][lane];
      }
    };
    uint2 qr[C::kQRegs ? kSteps : 1][NT];
    if constexpr (C::kQRegs) {
#pragma unroll
      for (int ks = 0; ks < kSteps; ++ks)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) qr[ks][nt] = query(ks, nt);
    }
    // When a row outgrows its reference, the others' go along where all see the same keys: one visit
    // instead of several (ragged 8-bit batch, 64 sequences: 70.0 -> 69.2 us in a graph).  Rows of several
    // tokens move by their own maximum alone, and rows past the tile's last have no scores.
    const float own_lag = info.tokens > 1 ? kLag<Q8> : 0.f;
    // this thread's rows: 8 nt + 2 t + e; the last position each sees
    const int pos_min = before + row_base / a.g;
    int pos[NT][2];
    float scale[NT][2], m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * nt + 2 * t + e;
        pos[nt][e] = before + (row_base + r) / a.g;
        scale[nt][e] = r >= rows ? 0.f : Q8 ? sm.q_scale[r] : a.scale_log2;
        m[nt][e] = -INFINITY;
        l[nt][e] = 0.f;
      }
    // 8-bit values: the accumulators count in 2^(v_ref - kUnitOne) (0: nothing added yet)
    int v_ref = 0;
    const bool few = sg.n * 16 * G <= kMostNear;
    float o[D / 16][NT][4];       // (columns 16 i + g and + 8) x (rows 2 t, 2 t + 1)
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) o[i][nt][0] = o[i][nt][1] = o[i][nt][2] = o[i][nt][3] = 0.f;

    for (int i = sg.ta; i < sg.ta + sg.n; ++i) {
      const int st = stage;
      alive = alive && wait_one(&sm.full[st], phase, &sm.dead, c.status);
      if (++stage == C::kStages) { stage = 0; phase ^= 1u; }
      const int k0 = i * TK + warp * G * 16;
      if (k0 < keys) {
        const uint8_t* kb = sm.ring[st];
        const uint32_t vb = smem_u32(kb) + C::kHalfBytes;
        // The key, of a group's 16, of MMA row g + 8 f.  8-bit caches: the order that gives the
        // transposed value loads (whose lane t holds four neighbouring rows) and the keys' 16-byte
        // loads alike eight different bank groups.
        auto key_in = [&](int f) { return Q8 ? (g & 1) << 2 | f << 1 | ((g >> 1) & 1) | (g >> 2) << 3 : g + 8 * f; };
        // ---- scores: element (f, e) is key f of row e
        float s[G][NT][4];
#pragma unroll
        for (int u = 0; u < G; ++u)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) s[u][nt][0] = s[u][nt][1] = s[u][nt][2] = s[u][nt][3] = 0.f;
        if constexpr (!Q8) {
          const int key = ((lane >> 3) & 1) * 8 + (lane & 7), half = lane >> 4;
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
            for (int u = 0; u < G; ++u) {
              uint32_t r[4];
              ldsm4(smem_u32(kb) + at[u] + key * 128 + (ks >> 2) * blk_bytes +
                        ((((ks & 3) * 2 + half) ^ (key & 7)) << 4), r);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                const uint2 q = C::kQRegs ? qr[C::kQRegs ? ks : 0][nt] : query(ks, nt);
                mma16816(s[u][nt], make_uint4(r[0], r[1], r[2], r[3]), q.x, q.y);
              }
            }
        } else {
#pragma unroll
          for (int cb = 0; cb < D / 64; ++cb) {
            uint4 w[G][2];
#pragma unroll
            for (int u = 0; u < G; ++u)
#pragma unroll
              for (int f = 0; f < 2; ++f) {
                const int key = key_in(f);
                const int chunk = (C::kBox == 128) ? (((cb & 1) * 4 + t) ^ (key & 7)) : (t ^ ((key >> 1) & 3));
                w[u][f] = *reinterpret_cast<const uint4*>(kb + at[u] + (C::kBox == 128 ? (cb >> 1) * blk_bytes : 0) +
                                                          key * C::kBox + chunk * 16);
              }
#pragma unroll
            for (int part = 0; part < 2; ++part)
#pragma unroll
              for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  constexpr int kPart = D / 32;
                  const int ks = part * kPart + cb * 2 + e;
                  const uint2 q = C::kQRegs ? qr[C::kQRegs ? ks : 0][nt] : query(ks, nt);
#pragma unroll
                  for (int u = 0; u < G; ++u)
                    mma16832_e4m3(s[u][nt], e ? make_uint4(w[u][0].z, w[u][1].z, w[u][0].w, w[u][1].w)
                                              : make_uint4(w[u][0].x, w[u][1].x, w[u][0].y, w[u][1].y), q.x, q.y);
                }
          }
        }
        uint32_t v_byte[G][2];
#pragma unroll
        for (int u = 0; u < G; ++u)
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            float ks = 1.f;
            v_byte[u][f] = 0;
            if constexpr (Q8) {
              ks = scale_f32(sm.scales[st][0][(warp * G + u) * 16 + key_in(f)]);
              v_byte[u][f] = sm.scales[st][1][(warp * G + u) * 16 + key_in(f)];
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              s[u][nt][2 * f] *= ks * scale[nt][0];
              s[u][nt][2 * f + 1] *= ks * scale[nt][1];
            }
          }
        const bool partial = k0 + 16 * G - 1 > pos_min;       // some row does not see all keys
        if (partial) {
#pragma unroll
          for (int u = 0; u < G; ++u)
#pragma unroll
            for (int f = 0; f < 2; ++f)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  if (k0 + 16 * u + key_in(f) > pos[nt][e]) s[u][nt][2 * f + e] = -INFINITY;
        }
        // ---- softmax of this warp's keys
        float x[NT][2];
        bool above = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float v = -INFINITY;
#pragma unroll
            for (int u = 0; u < G; ++u) v = fmaxf(v, fmaxf(s[u][nt][e], s[u][nt][2 + e]));
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
            x[nt][e] = v;
            above |= v > m[nt][e] + kLag<Q8>;
          }
        if (__any_sync(0xffffffffu, above)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              // no bit of a row depends on keys that it does not see
              const float to = x[nt][e] > m[nt][e] + own_lag ? x[nt][e] : m[nt][e];
              const float f = m[nt][e] == to ? 1.f : ex2(m[nt][e] - to);
              m[nt][e] = to;
              l[nt][e] *= f;
#pragma unroll
              for (int d = 0; d < D / 16; ++d) {
                o[d][nt][e] *= f;
                o[d][nt][2 + e] *= f;
              }
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float ref = m[nt][e] == -INFINITY ? 0.f : m[nt][e];
#pragma unroll
            for (int u = 0; u < G; ++u)
#pragma unroll
              for (int f = 0; f < 2; ++f) {
                const float p = ex2(s[u][nt][2 * f + e] - ref);
                s[u][nt][2 * f + e] = p;
                l[nt][e] += p;
              }
          }
        // ---- values
        if constexpr (!Q8) {
          static_assert(Q8 || G == 1, "the bf16 values are written for one group");
          uint2 p[NT];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            p[nt] = make_uint2(transpose8x8(pack_bf16(s[0][nt][0], s[0][nt][1])),
                               transpose8x8(pack_bf16(s[0][nt][2], s[0][nt][3])));
          const int key = (lane >> 4) * 8 + (lane & 7), half = (lane >> 3) & 1;
          const uint32_t row = vb + at[0] + key * 128;
          auto load_v = [&](int d, uint32_t* r) {         // columns 16 d + g, + 8; keys 2 t, + 1, + 8, + 9
            ldsm4t(row + (d >> 2) * blk_bytes + ((((d & 3) * 2 + half) ^ (key & 7)) << 4), r);
          };
          // keys past the sequence's end: their rows may hold anything, and 0 x NaN is NaN
          const bool tail = k0 + 16 > keys;
          uint32_t z0 = 0xffffffffu, z1 = 0xffffffffu;
          if (tail) {
            const int y = k0 + 2 * t;
            z0 = (y < keys ? 0xffffu : 0u) | (y + 1 < keys ? 0xffff0000u : 0u);
            z1 = (y + 8 < keys ? 0xffffu : 0u) | (y + 9 < keys ? 0xffff0000u : 0u);
          }
          // A key hidden from some rows and seen by others: its value must be finite for the matrix
          // product to leave the former alone.  Non-finite ones are taken out of it and added to the
          // rows that see them.
          uint32_t seen = 0;
          if (partial && info.tokens > 1) {
#pragma unroll 4
            for (int d = 0; d < D / 16; ++d) {
              uint32_t r[4];
              load_v(d, r);
              seen |= non_finite(r[0] & z0) | non_finite(r[1] & z0) | non_finite(r[2] & z1) | non_finite(r[3] & z1);
            }
          }
          if (!__any_sync(0xffffffffu, seen != 0)) {
#pragma unroll
            for (int d = 0; d < D / 16; ++d) {
              uint32_t r[4];
              load_v(d, r);
              if (tail) { r[0] &= z0; r[1] &= z0; r[2] &= z1; r[3] &= z1; }
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma16816(o[d][nt], make_uint4(r[0], r[1], r[2], r[3]), p[nt].x, p[nt].y);
            }
          } else {
#pragma unroll
            for (int d = 0; d < D / 16; ++d) {
              uint32_t r[4];
              load_v(d, r);
              r[0] &= z0; r[1] &= z0; r[2] &= z1; r[3] &= z1;
#pragma unroll
              for (int y = 0; y < 4; ++y) r[y] &= ~((non_finite(r[y]) >> 15) * 0xffffu);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma16816(o[d][nt], make_uint4(r[0], r[1], r[2], r[3]), p[nt].x, p[nt].y);
            }
#pragma unroll 1
            for (int j = 0; j < 16 && k0 + j < keys; ++j) {
              const int src = (j & 7) * 4 + t;
              float pj[NT][2];
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  pj[nt][e] = __shfl_sync(0xffffffffu, j & 8 ? s[0][nt][2 + e] : s[0][nt][e], src);
#pragma unroll
              for (int d = 0; d < D / 16; ++d) {
                const uint32_t v = vb + at[0] + j * 128 + (d >> 2) * blk_bytes + g * 2;
                const float v0 = lds_bf16(v + ((((d & 3) * 2) ^ (j & 7)) << 4));
                const float v1 = lds_bf16(v + ((((d & 3) * 2 + 1) ^ (j & 7)) << 4));
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                  for (int e = 0; e < 2; ++e)
                    if (k0 + j <= pos[nt][e]) {
                      if (!isfinite(v0)) o[d][nt][e] = fmaf(pj[nt][e], v0, o[d][nt][e]);
                      if (!isfinite(v1)) o[d][nt][2 + e] = fmaf(pj[nt][e], v1, o[d][nt][2 + e]);
                    }
              }
            }
          }
        } else {
          // The probabilities take the values' scales 2^(b - 127) as 2^(b - v_ref + kUp).  The unit is
          // chosen by the first keys that all rows see, two binades above their largest scale, and stays:
          // what a key adds then depends on no other key.  f16 holds the products of nearby scales;
          // the other keys', and those of keys that some row does not see or that lie past the
          // sequence's end (codes there may be NaN's, which the bit conversion makes 480), are bf16,
          // whose exponents hold any.  Where hidden keys begin, or scales come that the unit is far
          // too small for (the sum would leave f32), the unit becomes 1 for good, in which a sum holds what
          // an f32 sum of the values themselves does.
          bool wide = partial || v_ref == 0 || !few;
#pragma unroll
          for (int u = 0; u < G; ++u)
#pragma unroll
            for (int f = 0; f < 2; ++f) wide |= (uint32_t)(v_ref - (int)v_byte[u][f]) > kNear;
          if (__any_sync(0xffffffffu, wide)) {
            uint32_t most = 0, least = 255;
            if (!partial) {
#pragma unroll
              for (int u = 0; u < G; ++u)
#pragma unroll
                for (int f = 0; f < 2; ++f)
                  if (v_byte[u][f] != 255) {
                    most = max(most, v_byte[u][f]);
                    least = min(least, v_byte[u][f]);
                  }
              most = __reduce_max_sync(0xffffffffu, most);
              least = __reduce_min_sync(0xffffffffu, least);
              if (v_ref == 0) v_ref = min(max((int)most + 2, kLeastUnit), kUnitOne);
            }
            if (partial || (int)most > v_ref + 24) {
              if (v_ref != 0 && v_ref != kUnitOne) {
                const float f = __uint_as_float((uint32_t)(127 + v_ref - kUnitOne) << 23);
#pragma unroll
                for (int y = 0; y < D / 16; ++y)
#pragma unroll
                  for (int nt = 0; nt < NT; ++nt) {
                    o[y][nt][0] *= f; o[y][nt][1] *= f; o[y][nt][2] *= f; o[y][nt][3] *= f;
                  }
              }
              v_ref = kUnitOne;
            }
            wide = partial || !few || (int)most > v_ref || v_ref - (int)least > (int)kNear;
          }
#pragma unroll
          for (int u = 0; u < G; ++u)
#pragma unroll
            for (int f = 0; f < 2; ++f) {
              const int bb = (int)v_byte[u][f];
              const float y = bb == 255 ? __int_as_float(0x7fffffff)
                                        : __uint_as_float((uint32_t)max(bb - v_ref + kUnitOne, 0) << 23);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  s[u][nt][2 * f + e] *= y;
                  // a hidden key stays at zero even if its vector reads as NaN
                  if (partial && k0 + 16 * u + key_in(f) > pos[nt][e]) s[u][nt][2 * f + e] = 0.f;
                }
            }
          // lane i & 15 points at the key of matrix row i: rows 4 t + 2 f + e are MMA rows 2 t + e + 8 f
          const int key = (lane & 1) << 2 | (lane & 2) | ((lane >> 2) & 1) | (lane & 8);
          auto load_v = [&](int u, int d, uint32_t* r) {  // columns 32 d + g, + 8, + 16, + 24
            const int chunk = 2 * d + (lane >> 4);
            ldsm2t_b8(vb + at[u] + key * C::kBox +
                          (C::kBox == 128 ? (d >> 2) * blk_bytes + (((chunk & 7) ^ (key & 7)) << 4)
                                          : (chunk ^ ((key >> 1) & 3)) << 4), r);
          };
          uint2 p[G][NT];
#pragma unroll
          for (int u = 0; u < G; ++u)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const float* y = s[u][nt];
              p[u][nt] = wide ? make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]))
                              : make_uint2(pack_f16(y[0], y[1]), pack_f16(y[2], y[3]));
              p[u][nt].x = transpose8x8(p[u][nt].x);
              p[u][nt].y = transpose8x8(p[u][nt].y);
            }
          if (!wide) {
#pragma unroll
            for (int d = 0; d < D / 32; ++d) {
              uint32_t r[G][4];
#pragma unroll
              for (int u = 0; u < G; ++u) load_v(u, d, r[u]);
#pragma unroll
              for (int u = 0; u < G; ++u)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const uint32_t r0 = r[u][2 * h], r1 = r[u][2 * h + 1];
                  const uint4 v = make_uint4(e4m3_to_f16x2((uint16_t)r0), e4m3_to_f16x2((uint16_t)r1),
                                             e4m3_to_f16x2((uint16_t)(r0 >> 16)), e4m3_to_f16x2((uint16_t)(r1 >> 16)));
#pragma unroll
                  for (int nt = 0; nt < NT; ++nt) mma16816_f16(o[2 * d + h][nt], v, p[u][nt].x, p[u][nt].y);
                }
            }
          } else {
#pragma unroll
            for (int u = 0; u < G; ++u)
#pragma unroll
              for (int d = 0; d < D / 32; ++d) {
                uint32_t r[4];
                load_v(u, d, r);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  uint4 v;
                  e4m3x4_to_bf16(r[2 * h], v.x, v.z);
                  e4m3x4_to_bf16(r[2 * h + 1], v.y, v.w);
#pragma unroll
                  for (int nt = 0; nt < NT; ++nt) mma16816(o[2 * d + h][nt], v, p[u][nt].x, p[u][nt].y);
                }
              }
          }
        }
      }
      __syncwarp();
      if (alive && lane == 0) mbar_arrive(&sm.empty[st]);
    }

    if (!Q8 && alive && lane == 0) mbar_arrive(&sm.q_empty);

    // ---- the warps' results of this tile become one
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], d);
        // a NaN sum must survive the merge even when its reference never left -infinity
        if (l[nt][e] != l[nt][e]) m[nt][e] = INFINITY;
        if (g == 0) {
          sm.ml[warp][8 * nt + 2 * t + e][0] = m[nt][e];
          sm.ml[warp][8 * nt + 2 * t + e][1] = l[nt][e];
        }
      }
    bar_sync(1, NC);
    float f[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < C::kConsumers; ++w) top = fmaxf(top, sm.ml[w][8 * nt + 2 * t + e][0]);
        f[nt][e] = m[nt][e] == -INFINITY ? 0.f : ex2(m[nt][e] - top);
        if (Q8) f[nt][e] *= v_ref == 0 ? 0.f : __uint_as_float((uint32_t)(v_ref - kUp) << 23);   // 2^(v_ref - kUnitOne)
      }
    const bool whole = sg.whole;
    float* prow = Partials<R, D>::rows(a.ws, cta, sg.slot);
    // Some of the columns at a time: every warp lays its part down, and each thread adds the
    // warps' values of the four columns it then writes.
    constexpr int kPieces = C::kChunk / 4, kStep = NC / kPieces;
    const int piece = tid % kPieces;
#pragma unroll
    for (int ch = 0; ch < D / C::kChunk; ++ch) {
#pragma unroll
      for (int d = 0; d < C::kChunk / 16; ++d)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float* v = o[ch * (C::kChunk / 16) + d][nt];
            sm.o[warp][8 * nt + 2 * t + e][16 * d + g] = v[e] * f[nt][e];
            sm.o[warp][8 * nt + 2 * t + e][16 * d + g + 8] = v[2 + e] * f[nt][e];
          }
      bar_sync(1, NC);
      for (int r = tid / kPieces; r < rows; r += kStep) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < C::kConsumers; ++w) {
          const float4 u = *reinterpret_cast<const float4*>(&sm.o[w][r][piece * 4]);
          v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
        }
        const int d = ch * C::kChunk + piece * 4;
        if (whole || (ch == 0 && piece == 0)) {
          float M = -INFINITY, sum = 0.f;
#pragma unroll
          for (int w = 0; w < C::kConsumers; ++w) M = fmaxf(M, sm.ml[w][r][0]);
#pragma unroll
          for (int w = 0; w < C::kConsumers; ++w) {
            const float mw = sm.ml[w][r][0];
            if (mw != -INFINITY) sum += sm.ml[w][r][1] * ex2(mw - M);
          }
          if (whole) {
            const float inv = sum == 0.f ? 0.f : 1.0f / sum;
            v.x *= inv; v.y *= inv; v.z *= inv; v.w *= inv;
          } else {
            __stcg(reinterpret_cast<float2*>(Partials<R, D>::ml(a.ws, cta, sg.slot) + 2 * r), make_float2(M, sum));
          }
        }
        if (whole) {
          int tok, head;
          row_of(info, a.g, sg.head, row_base + r, &tok, &head);
          store_out4(a, D, tok, head, d, v);
        } else {
          __stcg(reinterpret_cast<float4*>(prow + (size_t)r * D + d), v);
        }
      }
      if (ch + 1 < D / C::kChunk) bar_sync(1, NC);
    }
    // (next_segment has the barrier that frees the warps' results)
  }
}

template <int D, bool Q8, int NT>
int launch_rows(const KvView& c, const KvBatchView& b, const AttnArgs& a, int sms, cudaStream_t stream) {
  using C = RowsCfg<D, Q8, NT>;
  constexpr size_t smem = sizeof(RowsSmem<D, Q8, NT>);
  static_assert(smem <= 232448 && (smem + 1024) * C::kCtas <= 233472, "shared memory of an SM");
  static OncePerDevice once;
  int rc = raise_smem(once, rows_kernel<D, Q8, NT>, smem);
  if (rc != GDN_OK) return rc;
  KvMaps maps;
  const int P = 1 << c.page_shift;
  if (!make_kv_maps(c, P < C::kKeys ? P : C::kKeys, &maps)) return GDN_ERR_CUDA;
  // What a tile costs beside its keys, in keys: some 3 us, in which an 8-bit cache gives twice the
  // keys.  (64 sequences of 255 to 15859: 8-bit 133 us at 64, 121 at 192, 111 at 384; bf16 193, 193,
  // 195.)  And the fewest keys worth a piece of their own (777 keys: 14.7 us at 128, 15.5 at 256, 18.4 at 512).
  const int grid = rows_grid(D, sms), fix = (Q8 ? 384 : 128) * a.g;
  const int least = 128 * a.g;
  rc = launch_dependent(rows_kernel<D, Q8, NT>, dim3((unsigned)grid), C::kThreads, smem, stream, c, b, a, grid,
                            fix, least, maps);
  if (rc != GDN_OK) return rc;
  return launch_dependent(merge_kernel<C::kRows, D>, dim3((unsigned)(2 * sms)), kMergeWarps * 32, 0, stream, a, grid);
}

int rows_grid(int D, int sms) { return min(kMaxPieces, D == 256 ? sms : 2 * sms); }

size_t rows_ws_bytes(int D, int sms) {
  const int grid = rows_grid(D, sms);
  return D == 64 ? Partials<16, 64>::bytes(grid)
       : D == 128 ? Partials<16, 128>::bytes(grid) : Partials<16, 256>::bytes(grid);
}

template <int D>
int launch_rows(const KvView& c, const KvBatchView& b, const AttnArgs& a, int rows, int sms, cudaStream_t stream) {
  if (rows <= 8)
    return c.ks ? launch_rows<D, true, 1>(c, b, a, sms, stream) : launch_rows<D, false, 1>(c, b, a, sms, stream);
  return c.ks ? launch_rows<D, true, 2>(c, b, a, sms, stream) : launch_rows<D, false, 2>(c, b, a, sms, stream);
}

int launch_rows(const KvView& c, const KvBatchView& b, const AttnArgs& a, int rows, int sms, cudaStream_t stream) {
  return c.D == 64    ? launch_rows<64>(c, b, a, rows, sms, stream)
         : c.D == 128 ? launch_rows<128>(c, b, a, rows, sms, stream)
                      : launch_rows<256>(c, b, a, rows, sms, stream);
}

}  // namespace attn
}  // namespace gdn
