// gdn_attn_rows.cu -- attention of a few query rows per key/value head over the paged cache: the
// decode step (one token per sequence), and short runs of new tokens.
//
//   o_r = sum_j p_rj v_j / sum_j p_rj,   p_rj = 2^(s_rj - m_r),   s_rj = scale log2(e) q_r . k_j
//
// with one pass over the keys: m_r is a reference that follows the running maximum (it only has to
// stay within 2^8 of it, so the accumulator is rescaled when a maximum outgrows it by that much,
// not at every step) and every sum is f32.
//
// What bounds it: the cache is read once, 2 D elements per key and head, for at most 16 rows, so
// the floor is its bytes at the HBM rate.  Everything else must hide behind the loads:
//  * a producer warp keeps a ring of 64-key stages full with TMA tensor copies (a box is 16 keys of
//    one page, 128-byte swizzled), page numbers fetched one stage ahead;
//  * each consumer warp takes 16 keys of a stage and runs its own softmax, so warps meet only at
//    the end of a tile, where their accumulators are added in a fixed order;
//  * the products are m16n8k16 MMAs on registers.  Sixteen rows fill that shape; the 128-row
//    tcgen05 shape would run 7/8 empty here, needs the probabilities to cross TMEM, and could not
//    be faster than the loads, which already set the pace;
//  * 8-bit caches: the keys' codes are e4m3 MMA operands as they are (the queries as two e4m3
//    parts, whose sum is exact), their scales applied to the scores; the values' codes become f16 by
//    the conversion instruction, their scales applied to the probabilities.  Halving the bytes
//    halves the time the arithmetic may take: converting both to bf16 by bit operations, 2.5 per
//    element, held the kernel to 3.7 of the 6.7 TB/s.
#include "gdn_attn.cuh"
#include "gdn_tmap.h"

namespace gdn {

using namespace tc;

namespace attn {

constexpr int kRows = 16;

template <int D, bool Q8>
struct RowsCfg {
  // D = 256: the accumulators take 128 registers of a thread, and a stage twice the bytes.
  static constexpr int kConsumers = 4;
  static constexpr int kCtas = D == 256 ? 1 : 2;
  static constexpr int kThreads = (kConsumers + 2) * 32;         // and two producers: keys, values
  static constexpr int kElem = Q8 ? 1 : 2;
  // Groups of 16 keys that a warp takes of a stage.  An MMA's result takes some 70 cycles; with half
  // the bytes to wait for, an 8-bit cache wants the chains of two groups side by side.
  static constexpr int kGroups = Q8 ? 2 : 1;
  static constexpr int kKeys = 64 * kGroups;                     // of a stage
  static constexpr int kHalfBytes = kKeys * D * kElem;           // a stage's keys
  static constexpr int kStageBytes = 2 * kHalfBytes;
  static constexpr int kRing = kCtas == 1 ? 196608 : 98304;
  static constexpr int kStages = kRing / kStageBytes;
  static constexpr int kBox = D * kElem >= 128 ? 128 : 64;       // swizzle span, bytes
  static constexpr int kQLd = 2 * D + 16;                        // bytes of a staged query row
  static constexpr int kChunk = D / (Q8 && D > 64 ? 8 : 4);      // columns merged at a time
  static constexpr int kMLd = kChunk + 4;
};

template <int D, bool Q8>
struct __align__(1024) RowsSmem {
  using C = RowsCfg<D, Q8>;
  uint8_t ring[C::kStages][C::kStageBytes];
  uint8_t scales[Q8 ? C::kStages : 1][2][C::kKeys];    // scale bytes of a stage's keys and values
  uint8_t q[kRows][C::kQLd];              // the rows, as copied
  uint4 q_parts[Q8 ? D / 16 : 1][32];     // 8-bit caches: A fragments of their two e4m3 parts
  float q_scale[kRows];
  float o[C::kConsumers][kRows][C::kMLd];
  float ml[C::kConsumers][kRows][2];
  LineScan<kRows, C::kThreads> scan;
  uint64_t full[C::kStages];
  uint64_t empty[C::kStages];
  uint64_t q_full, q_empty;
  int dead;
};

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
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];\n" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
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

// A bounded wait: a timeout marks the CTA dead, after which no wait blocks and the (wrong) results
// are flagged by the status bit.
__device__ __forceinline__ void wait_or_die(uint64_t* bar, uint32_t parity, volatile int* dead, int32_t* status) {
  if (*dead) return;
  if (!mbar_wait(bar, parity)) {
    *dead = 1;
    set_status(status, GDN_STATUS_TIMEOUT);
  }
}

template <int D, bool Q8>
__global__ void __launch_bounds__(RowsCfg<D, Q8>::kThreads, RowsCfg<D, Q8>::kCtas)
rows_kernel(const KvView c, const KvBatchView b, const AttnArgs a, int grid, int fix, int least,
            const __grid_constant__ KvMaps maps) {
  using C = RowsCfg<D, Q8>;
  constexpr int R = kRows, TK = C::kKeys, NC = C::kConsumers * 32;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  RowsSmem<D, Q8>& sm = *reinterpret_cast<RowsSmem<D, Q8>*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&sm.full[i], Q8 ? 2 + TK / 8 : 2);
      mbar_init(&sm.empty[i], 4);
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
  zero_padding(a, b, D);
  bool bad = false;
  Pieces pieces;
  const int cta = blockIdx.x;
  locate_piece<R, C::kThreads>(c, b, a.g, fix, grid, least, cta, &pieces, &sm.scan, &bad);
  if (bad) set_status(c.status, GDN_STATUS_BAD_SEQLENS);
  if (cta >= pieces.count) {
    if (tid == 0) Partials<R, D>::note(a.ws, grid, cta, a.g, nullptr, 0);
    return;
  }
  SegIter<R, TK> it;
  it.start(&b, c.page_shift, c.H, a.g, fix, pieces, cta, sm.scan.at);
  Segment sg;
  sg.split = false;

  if (warp >= C::kConsumers) {
    // ---------------------------------------------------------------- producers
    // Copies of one warp go out one after another (some 150 cycles each), hence a warp for the keys
    // and one for the values.
    const bool values = warp > C::kConsumers;
    int stage = 0;
    uint32_t phase = 0, q_phase = 0;
    while (it.next(&sg)) {
      if (sg.ta >= sg.tb) continue;
      const int rows = (int)min((long long)R, (long long)sg.info.tokens * a.g - sg.tile * R);
      // the queries' place is free when the tile before has been scored: after what the ring takes
      const int q_after = min(sg.tb, sg.ta + C::kStages - 1) - 1;
      const int* table = b.table + (long long)sg.seq * b.table_ld;
      const int keys = min(sg.info.len, tile_keys<R>(sg.info, a.g, sg.tile));
      // Lane i < TK / 16 looks after the i-th 16 keys of a stage: their page, fetched a stage ahead,
      // the box that begins with them (a box is a page's part of the stage), and their scale bytes.
      constexpr int kLanes = TK / 16;
      const int box = min(1 << c.page_shift, TK);
      int k0 = sg.ta * TK + (lane % kLanes) * 16;
      int page = k0 < keys ? __ldg(table + (k0 >> c.page_shift)) : 0;
      for (int i = sg.ta; i < sg.tb; ++i) {
        const int k1 = k0 + TK;
        int page_next = 0;
        if (i + 1 < sg.tb && k1 < keys) page_next = __ldg(table + (k1 >> c.page_shift));
        wait_or_die(&sm.empty[stage], phase ^ 1u, &sm.dead, c.status);
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
                      values ? &maps.v : &maps.k, 0, off, 0, sg.head, page, full);
        if (Q8 && lane < kLanes) {
          const bool in = k0 < keys && page < c.num_pages;
          const uint8_t* src = values ? c.vs : c.ks;
          if (in) src += (((long long)page * c.H + sg.head) << c.page_shift) + off;
          cp_async16_mbar(smem_u32(&sm.scales[stage][values][lane * 16]), src, in, full);
        }
        __syncwarp();
        if (values && i == q_after) {
          wait_or_die(&sm.q_empty, q_phase ^ 1u, &sm.dead, c.status);
          q_phase ^= 1u;
          if (lane == 0) mbar_arrive_expect_tx(&sm.q_full, (uint32_t)rows * 2 * D);
          __syncwarp();
          if (lane < rows) {
            int tok, head;
            row_of(sg.info, a.g, sg.head, sg.tile * R + lane, &tok, &head);
            bulk_g2s(sm.q[lane], a.q + tok * a.q_ld + head * a.q_head_ld, 2 * D, &sm.q_full);
          }
          __syncwarp();
        }
        page = page_next;
        k0 = k1;
        if (++stage == C::kStages) { stage = 0; phase ^= 1u; }
      }
    }
    // the piece's last tile may be shared with the next ones
    if (!values && lane == 0) Partials<R, D>::note(a.ws, grid, cta, a.g, &sg, sg.split ? it.sharing(sg.nt) : 0);
    return;
  }

  // ------------------------------------------------------------------ consumers
  const int t = lane & 3, n = lane >> 2;
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
  while (it.next(&sg)) {
    const SeqInfo info = sg.info;
    const int row_base = sg.tile * R;
    const int rows = min((long long)R, (long long)info.tokens * a.g - row_base);
    if (sg.ta >= sg.tb) {
      if (sg.owns_empty)
        for (int i = tid; i < rows * (D / 8); i += NC) {
          int tok, head;
          row_of(info, a.g, sg.head, row_base + i / (D / 8), &tok, &head);
          *reinterpret_cast<uint4*>(a.out + ((long long)tok * a.Hq + head) * D + (i % (D / 8)) * 8) =
              make_uint4(0, 0, 0, 0);
        }
      else if (sg.nt > 0)                                // an empty share of a split tile
        for (int i = tid; i < rows; i += NC)
          __stcg(reinterpret_cast<float2*>(Partials<R, D>::ml(a.ws, cta, sg.slot) + 2 * i), make_float2(-INFINITY, 0.f));
      continue;
    }
    const int keys = min(info.len, tile_keys<R>(info, a.g, sg.tile));
    const int before = info.len - info.tokens;          // position of the first new token
    wait_or_die(&sm.q_full, q_phase, &sm.dead, c.status);
    q_phase ^= 1u;
    if constexpr (Q8) {
      // A warp splits four rows into their parts (see split_e4m3).  The k order inside a 64-column
      // block follows the keys' loads: lane t of a quad reads 16 consecutive columns, eight to a
      // k-step.
      constexpr int kEl = D == 256 ? 8 : 4;              // columns of a lane (D = 64: half the lanes)
      const int d0 = lane * kEl;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = warp * 4 + j;
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
        const float inv = __uint_as_float((uint32_t)(254 - (bb == 255 ? 127 : bb)) << 23);
        if (lane == 0) sm.q_scale[r] = scale_f32(bb) * a.scale_log2;
#pragma unroll
        for (int e = 0; e < kEl / 4; ++e) {
          uint32_t hi[2], lo[2];
#pragma unroll
          for (int k = 0; k < 2; ++k)
            split_e4m3(__uint_as_float(w[2 * e + k] << 16) * inv, __uint_as_float(w[2 * e + k] & 0xffff0000u) * inv,
                       hi[k], lo[k]);
          const int d = d0 + 4 * e;
          if (d < D) {
            const int ks = (d >> 6) * 2 + ((d >> 3) & 1), ln = (r & 7) * 4 + ((d >> 4) & 3);
            const int reg = (r >> 3) + 2 * ((d >> 2) & 1);
            reinterpret_cast<uint32_t*>(&sm.q_parts[ks][ln])[reg] = hi[0] | (hi[1] << 16);
            reinterpret_cast<uint32_t*>(&sm.q_parts[D / 32 + ks][ln])[reg] = lo[0] | (lo[1] << 16);
          }
        }
      }
      bar_sync(1, NC);
      if (lane == 0) mbar_arrive(&sm.q_empty);
    }
    // last position each of this thread's two rows sees
    const int pos0 = before + (row_base + n) / a.g, pos1 = before + (row_base + n + 8) / a.g;
    const int pos_min = before + row_base / a.g;
    const float scale0 = Q8 ? sm.q_scale[n] : a.scale_log2, scale1 = Q8 ? sm.q_scale[n + 8] : a.scale_log2;
    // 8-bit values: the accumulators count in 2^(v_ref - 134), v_ref the largest scale byte so far
    int v_ref = 0;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;

    for (int i = sg.ta; i < sg.tb; ++i) {
      const int st = stage;
      wait_or_die(&sm.full[st], phase, &sm.dead, c.status);
      if (++stage == C::kStages) { stage = 0; phase ^= 1u; }
      const int k0 = i * TK + warp * G * 16;
      if (k0 < keys) {
        const uint8_t* kb = sm.ring[st];
        const uint32_t vb = smem_u32(kb) + C::kHalfBytes;
        // ---- scores: 16 rows x 2 columns of 8 keys, for each group
        float s[G][2][4];
#pragma unroll
        for (int u = 0; u < G; ++u)
#pragma unroll
          for (int j = 0; j < 2; ++j) s[u][j][0] = s[u][j][1] = s[u][j][2] = s[u][j][3] = 0.f;
        if constexpr (!Q8) {
          const int key = ((lane >> 4) << 3) + (lane & 7), half = (lane >> 3) & 1;
          const uint32_t q_row = smem_u32(sm.q[lane & 15]) + (lane >> 4) * 16;
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            uint4 q;
            ldsm4(q_row + ks * 32, &q.x);
#pragma unroll
            for (int u = 0; u < G; ++u) {
              uint32_t r[4];
              ldsm4(smem_u32(kb) + at[u] + key * 128 + (ks >> 2) * blk_bytes +
                        ((((ks & 3) * 2 + half) ^ (key & 7)) << 4), r);
              mma16816(s[u][0], q, r[0], r[1]);
              mma16816(s[u][1], q, r[2], r[3]);
            }
          }
        } else {
          // column n of score tile j is key 4 (n >> 1) + 2 j + (n & 1): the order in which the
          // transposed loads below hand out the values
#pragma unroll
          for (int cb = 0; cb < D / 64; ++cb) {
            uint4 w[G][2];
#pragma unroll
            for (int u = 0; u < G; ++u)
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const int key = 4 * (n >> 1) + 2 * j + (n & 1);
                const int chunk = (C::kBox == 128) ? (((cb & 1) * 4 + t) ^ (key & 7)) : (t ^ ((key >> 1) & 3));
                w[u][j] = *reinterpret_cast<const uint4*>(kb + at[u] + (C::kBox == 128 ? (cb >> 1) * blk_bytes : 0) +
                                                          key * C::kBox + chunk * 16);
              }
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int part = 0; part < 2; ++part) {
                const uint4 q = sm.q_parts[part * (D / 32) + cb * 2 + e][lane];
#pragma unroll
                for (int u = 0; u < G; ++u)
#pragma unroll
                  for (int j = 0; j < 2; ++j)
                    mma16832_e4m3(s[u][j], q, e ? w[u][j].z : w[u][j].x, e ? w[u][j].w : w[u][j].y);
              }
          }
        }
        uint32_t v_bytes[G];                           // scale bytes of the values of keys 4 t .. 4 t + 3
#pragma unroll
        for (int u = 0; u < G; ++u) {
          uint32_t k_bytes = 0;
          v_bytes[u] = 0;
          if constexpr (Q8) {
            k_bytes = *reinterpret_cast<const uint32_t*>(&sm.scales[st][0][(warp * G + u) * 16 + 4 * t]);
            v_bytes[u] = *reinterpret_cast<const uint32_t*>(&sm.scales[st][1][(warp * G + u) * 16 + 4 * t]);
          }
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float f = Q8 ? scale_f32((k_bytes >> (8 * (2 * j + e))) & 0xffu) : 1.f;
              s[u][j][e] *= f * scale0;
              s[u][j][e + 2] *= f * scale1;
            }
        }
        // the key of a lane's score (u, j, e)
        auto key_of = [&](int u, int j, int e) { return k0 + 16 * u + (Q8 ? 4 * t + 2 * j + e : j * 8 + 2 * t + e); };
        const bool partial = k0 + 16 * G - 1 > pos_min;       // some row does not see all keys
        if (partial) {
#pragma unroll
          for (int u = 0; u < G; ++u)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                if (key_of(u, j, e) > pos0) s[u][j][e] = -INFINITY;
                if (key_of(u, j, e) > pos1) s[u][j][e + 2] = -INFINITY;
              }
        }
        // ---- softmax of this warp's keys
        float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
        for (int u = 0; u < G; ++u) {
          x0 = fmaxf(x0, fmaxf(fmaxf(s[u][0][0], s[u][0][1]), fmaxf(s[u][1][0], s[u][1][1])));
          x1 = fmaxf(x1, fmaxf(fmaxf(s[u][0][2], s[u][0][3]), fmaxf(s[u][1][2], s[u][1][3])));
        }
        x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 1));
        x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 1));
        x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 2));
        x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 2));
        // 2^8 above the reference is harmless in f32 and in the 16-bit probabilities alike
        if (__any_sync(0xffffffffu, x0 > m0 + 8.f || x1 > m1 + 8.f)) {
          const float n0 = fmaxf(m0, x0), n1 = fmaxf(m1, x1);
          const float f0 = m0 == n0 ? 1.f : ex2(m0 - n0), f1 = m1 == n1 ? 1.f : ex2(m1 - n1);
          m0 = n0; m1 = n1;
          l0 *= f0; l1 *= f1;
#pragma unroll
          for (int d = 0; d < D / 8; ++d) {
            o[d][0] *= f0; o[d][1] *= f0; o[d][2] *= f1; o[d][3] *= f1;
          }
        }
        const float r0 = m0 == -INFINITY ? 0.f : m0, r1 = m1 == -INFINITY ? 0.f : m1;
#pragma unroll
        for (int u = 0; u < G; ++u)
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              s[u][j][e] = ex2(s[u][j][e] - r0);
              s[u][j][e + 2] = ex2(s[u][j][e + 2] - r1);
              l0 += s[u][j][e];
              l1 += s[u][j][e + 2];
            }
        // ---- values
        if constexpr (!Q8) {
          static_assert(Q8 || G == 1, "the bf16 values are written for one group");
          const float(&p4)[2][4] = s[0];
          const uint4 p = make_uint4(pack_bf16(p4[0][0], p4[0][1]), pack_bf16(p4[0][2], p4[0][3]),
                                     pack_bf16(p4[1][0], p4[1][1]), pack_bf16(p4[1][2], p4[1][3]));
          const int key = (((lane >> 3) & 1) << 3) + (lane & 7), half = lane >> 4;
          const uint32_t row = vb + at[0] + key * 128;
          // keys past the sequence's end: their rows may hold anything, and 0 x NaN is NaN
          const bool tail = k0 + 16 > keys;
          uint32_t z0 = 0xffffffffu, z1 = 0xffffffffu;
          if (tail) {
            const int u = k0 + 2 * t;
            z0 = (u < keys ? 0xffffu : 0u) | (u + 1 < keys ? 0xffff0000u : 0u);
            z1 = (u + 8 < keys ? 0xffffu : 0u) | (u + 9 < keys ? 0xffff0000u : 0u);
          }
          bool finite = true;
          if (partial && info.tokens > 1) {
            // a key hidden from some rows and seen by others: its value must be finite for the
            // matrix product to leave the former alone
            uint32_t seen = 0;
#pragma unroll 4
            for (int d = 0; d < D / 16; ++d) {
              uint32_t r[4];
              ldsm4t(row + (d >> 2) * blk_bytes + ((((d & 3) * 2 + half) ^ (key & 7)) << 4), r);
              seen |= ((r[0] & z0 & 0x7f807f80u) + 0x00800080u) | ((r[1] & z1 & 0x7f807f80u) + 0x00800080u) |
                      ((r[2] & z0 & 0x7f807f80u) + 0x00800080u) | ((r[3] & z1 & 0x7f807f80u) + 0x00800080u);
            }
            finite = !__any_sync(0xffffffffu, (seen & 0x80008000u) != 0);
          }
          if (finite) {
#pragma unroll
            for (int d = 0; d < D / 16; ++d) {
              uint32_t r[4];
              ldsm4t(row + (d >> 2) * blk_bytes + ((((d & 3) * 2 + half) ^ (key & 7)) << 4), r);
              if (tail) { r[0] &= z0; r[1] &= z1; r[2] &= z0; r[3] &= z1; }
              mma16816(o[2 * d], p, r[0], r[1]);
              mma16816(o[2 * d + 1], p, r[2], r[3]);
            }
          } else {
#pragma unroll 1
            for (int j = 0; j < 16 && k0 + j < keys; ++j) {
              const int src = (lane & ~3) | ((j & 7) >> 1);
              const float u0 = j & 8 ? (j & 1 ? p4[1][1] : p4[1][0]) : (j & 1 ? p4[0][1] : p4[0][0]);
              const float u1 = j & 8 ? (j & 1 ? p4[1][3] : p4[1][2]) : (j & 1 ? p4[0][3] : p4[0][2]);
              const float p0 = __shfl_sync(0xffffffffu, u0, src), p1 = __shfl_sync(0xffffffffu, u1, src);
              const bool see0 = k0 + j <= pos0, see1 = k0 + j <= pos1;
#pragma unroll
              for (int d = 0; d < D / 8; ++d) {
                const uint32_t w = lds32(vb + at[0] + j * 128 + (d >> 3) * blk_bytes + (((d & 7) ^ (j & 7)) << 4) + t * 4);
                const float v0 = __uint_as_float(w << 16), v1 = __uint_as_float(w & 0xffff0000u);
                if (see0) { o[d][0] = fmaf(p0, v0, o[d][0]); o[d][1] = fmaf(p0, v1, o[d][1]); }
                if (see1) { o[d][2] = fmaf(p1, v0, o[d][2]); o[d][3] = fmaf(p1, v1, o[d][3]); }
              }
            }
          }
        } else {
          // The probabilities take the values' scales 2^(b - 127) as 2^(b - v_ref + 7), v_ref the
          // largest b so far: f16 has eleven bits for them from 2^15 down to 2^-14, which is room
          // for scales 2^18 apart.  Where they are further apart, and past the sequence's end (codes
          // there may be NaN's, which the bit conversion makes 480), bf16 operands instead.
          uint32_t most = 0, least = 255;
#pragma unroll
          for (int u = 0; u < G; ++u)
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const uint32_t bb = (v_bytes[u] >> (8 * y)) & 0xffu;
              if (k0 + 16 * u + 4 * t + y < keys && bb != 255) {
                most = max(most, bb);
                least = min(least, bb);
              }
            }
          most = __reduce_max_sync(0xffffffffu, most);
          least = __reduce_min_sync(0xffffffffu, least);
          if ((int)most > v_ref) {
            const int d = v_ref - (int)most;
            const float f = d < -126 ? 0.f : __uint_as_float((uint32_t)(127 + d) << 23);
            v_ref = (int)most;
#pragma unroll
            for (int y = 0; y < D / 8; ++y) {
              o[y][0] *= f; o[y][1] *= f; o[y][2] *= f; o[y][3] *= f;
            }
          }
          const bool wide = v_ref - (int)least > 18 || k0 + 16 * G > keys;
#pragma unroll
          for (int u = 0; u < G; ++u)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int bb = (int)((v_bytes[u] >> (8 * (2 * j + e))) & 0xffu);
                const float f = bb == 255 ? __int_as_float(0x7fffffff)
                                          : __uint_as_float((uint32_t)max(bb - v_ref + 134, 0) << 23);
                s[u][j][e] *= f;
                s[u][j][e + 2] *= f;
              }
          if (partial) {       // a hidden key stays at zero even if its vector reads as NaN
#pragma unroll
            for (int u = 0; u < G; ++u)
#pragma unroll
              for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  if (key_of(u, j, e) > pos0) s[u][j][e] = 0.f;
                  if (key_of(u, j, e) > pos1) s[u][j][e + 2] = 0.f;
                }
          }
          const int key = lane & 15;
          auto value_at = [&](int u, int d) {           // 16 keys x 32 columns from column 32 d on
            const int chunk = 2 * d + (lane >> 4);
            return vb + at[u] + key * C::kBox +
                   (C::kBox == 128 ? (d >> 2) * blk_bytes + (((chunk & 7) ^ (key & 7)) << 4)
                                   : (chunk ^ ((key >> 1) & 3)) << 4);
          };
          if (!wide) {
            uint4 p[G];
#pragma unroll
            for (int u = 0; u < G; ++u)
              p[u] = make_uint4(pack_f16(s[u][0][0], s[u][0][1]), pack_f16(s[u][0][2], s[u][0][3]),
                                pack_f16(s[u][1][0], s[u][1][1]), pack_f16(s[u][1][2], s[u][1][3]));
#pragma unroll
            for (int d = 0; d < D / 32; ++d) {
              uint32_t r[G][4];
#pragma unroll
              for (int u = 0; u < G; ++u) ldsm2t_b8(value_at(u, d), r[u]);
#pragma unroll
              for (int u = 0; u < G; ++u)
#pragma unroll
                for (int y = 0; y < 4; ++y)
                  mma16816_f16(o[4 * d + y], p[u], e4m3_to_f16x2((uint16_t)r[u][y]),
                               e4m3_to_f16x2((uint16_t)(r[u][y] >> 16)));
            }
          } else {
#pragma unroll
            for (int u = 0; u < G; ++u) {
              const uint4 p = make_uint4(pack_bf16(s[u][0][0], s[u][0][1]), pack_bf16(s[u][0][2], s[u][0][3]),
                                         pack_bf16(s[u][1][0], s[u][1][1]), pack_bf16(s[u][1][2], s[u][1][3]));
#pragma unroll
              for (int d = 0; d < D / 32; ++d) {
                uint32_t r[4];
                ldsm2t_b8(value_at(u, d), r);
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                  uint32_t b0, b1;
                  e4m3x4_to_bf16(r[y], b0, b1);
                  mma16816(o[4 * d + y], p, b0, b1);
                }
              }
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.empty[st]);
    }

    if (!Q8 && lane == 0) mbar_arrive(&sm.q_empty);

    // ---- the warps' results of this tile become one
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
    // a NaN sum must survive the merge even when its reference never left -infinity
    if (l0 != l0) m0 = INFINITY;
    if (l1 != l1) m1 = INFINITY;
    if (t == 0) {
      sm.ml[warp][n][0] = m0; sm.ml[warp][n][1] = l0;
      sm.ml[warp][n + 8][0] = m1; sm.ml[warp][n + 8][1] = l1;
    }
    bar_sync(1, NC);
    float M0 = -INFINITY, M1 = -INFINITY;
#pragma unroll
    for (int w = 0; w < C::kConsumers; ++w) {
      M0 = fmaxf(M0, sm.ml[w][n][0]);
      M1 = fmaxf(M1, sm.ml[w][n + 8][0]);
    }
    float f0 = m0 == -INFINITY ? 0.f : ex2(m0 - M0), f1 = m1 == -INFINITY ? 0.f : ex2(m1 - M1);
    if (Q8) {
      const float unit = v_ref == 0 ? 0.f : __uint_as_float((uint32_t)(v_ref - 7) << 23);   // 2^(v_ref - 134)
      f0 *= unit;
      f1 *= unit;
    }
    const bool whole = sg.whole();
    float* prow = Partials<R, D>::rows(a.ws, cta, sg.slot);
    // Some of the columns at a time: every warp lays its part down, and each thread adds the
    // warps' values of the four columns it then writes.
    constexpr int kPieces = C::kChunk / 4, kStep = NC / kPieces;
    const int piece = tid % kPieces;
#pragma unroll
    for (int ch = 0; ch < D / C::kChunk; ++ch) {
#pragma unroll
      for (int d = 0; d < C::kChunk / 8; ++d) {
        const float* v = o[ch * (C::kChunk / 8) + d];
        *reinterpret_cast<float2*>(&sm.o[warp][n][d * 8 + 2 * t]) = make_float2(v[0] * f0, v[1] * f0);
        *reinterpret_cast<float2*>(&sm.o[warp][n + 8][d * 8 + 2 * t]) = make_float2(v[2] * f1, v[3] * f1);
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
          float M = -INFINITY, l = 0.f;
#pragma unroll
          for (int w = 0; w < C::kConsumers; ++w) M = fmaxf(M, sm.ml[w][r][0]);
#pragma unroll
          for (int w = 0; w < C::kConsumers; ++w) {
            const float mw = sm.ml[w][r][0];
            if (mw != -INFINITY) l += sm.ml[w][r][1] * ex2(mw - M);
          }
          if (whole) {
            const float inv = l == 0.f ? 0.f : 1.0f / l;
            v.x *= inv; v.y *= inv; v.z *= inv; v.w *= inv;
          } else {
            __stcg(reinterpret_cast<float2*>(Partials<R, D>::ml(a.ws, cta, sg.slot) + 2 * r), make_float2(M, l));
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
    bar_sync(1, NC);
  }
}

template <int D, bool Q8>
int launch_rows(const KvView& c, const KvBatchView& b, const AttnArgs& a, int sms, cudaStream_t stream) {
  using C = RowsCfg<D, Q8>;
  constexpr size_t smem = sizeof(RowsSmem<D, Q8>);
  static_assert(smem <= 232448 && (smem + 1024) * C::kCtas <= 233472, "shared memory of an SM");
  static const cudaError_t set = cudaFuncSetAttribute(
      rows_kernel<D, Q8>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (set != cudaSuccess) return GDN_ERR_CUDA;
  KvMaps maps;
  const int P = 1 << c.page_shift;
  if (!make_kv_maps(c, P < C::kKeys ? P : C::kKeys, &maps)) return GDN_ERR_CUDA;
  const int grid = rows_grid(D, sms), fix = 64 * a.g;
  const int least = 256 * a.g;
  int rc = launch_dependent(rows_kernel<D, Q8>, dim3((unsigned)grid), C::kThreads, smem, stream, c, b, a, grid,
                            fix, least, maps);
  if (rc != GDN_OK) return rc;
  return launch_dependent(merge_kernel<kRows, D>, dim3((unsigned)(2 * sms)), kMergeWarps * 32, 0, stream, a, grid);
}

int rows_grid(int D, int sms) { return min(kMaxPieces, D == 256 ? sms : 2 * sms); }

size_t rows_ws_bytes(int D, int sms) {
  const int grid = rows_grid(D, sms);
  return D == 64 ? Partials<kRows, 64>::bytes(grid)
       : D == 128 ? Partials<kRows, 128>::bytes(grid) : Partials<kRows, 256>::bytes(grid);
}

int launch_rows(const KvView& c, const KvBatchView& b, const AttnArgs& a, int sms, cudaStream_t stream) {
  const bool q8 = c.ks != nullptr;
  if (c.D == 64) return q8 ? launch_rows<64, true>(c, b, a, sms, stream) : launch_rows<64, false>(c, b, a, sms, stream);
  if (c.D == 128) return q8 ? launch_rows<128, true>(c, b, a, sms, stream) : launch_rows<128, false>(c, b, a, sms, stream);
  return q8 ? launch_rows<256, true>(c, b, a, sms, stream) : launch_rows<256, false>(c, b, a, sms, stream);
}

}  // namespace attn
}  // namespace gdn
