// gdn_attn.cuh -- how the attention kernels split their work, and what they share.
//
// The queries of a sequence under one key/value head are T * g rows (row r = token r / g, head
// r % g of the group), cut into tiles of R rows.  A tile's work is a run over the keys its last
// row sees.  All tiles of all sequences, laid end to end and measured in (keys x g) plus a
// constant per tile, form one line, and CTA w of G takes the w-th of G equal pieces of it: long
// and short sequences, many heads or one, are balanced alike, with no plan from the host.  A piece
// that begins or ends inside a tile leaves that tile's partial result (reference m, sum l and the
// unnormalised rows) in the workspace, and a second kernel merges them; a tile that lies inside
// one piece is finished in place.
#pragma once

#include "gdn_kv.cuh"
#include "gdn_tc.cuh"

namespace gdn {
namespace attn {

// 64-bit division that is a 32-bit one whenever it can be.
__device__ __forceinline__ long long div_small(long long a, int b) {
  return (unsigned long long)a >> 32 == 0 ? (long long)((unsigned)a / (unsigned)b) : a / b;
}

struct SeqInfo {
  int row0;        // first packed token
  int tokens;      // new tokens
  int len;         // cached positions, 0 when the sequence is not usable
};

// A sequence whose tokens do not lie in the batch's keeps those that do, without cached positions: their
// rows are written (zeros) like all others.
__device__ __forceinline__ SeqInfo load_seq(const KvBatchView& b, int page_shift, int s, bool* bad) {
  const int c0 = __ldg(b.cu + s), c1 = __ldg(b.cu + s + 1), len = __ldg(b.lens + s);
  SeqInfo r{c0, c1 - c0, len};
  if (c0 < 0 || c1 < c0 || c1 > b.total) {
    *bad = true;
    r.row0 = max(0, min(c0, b.total));
    r.tokens = max(0, min(c1, b.total) - r.row0);
    r.len = 0;
  } else if (len < 0 || len > ((long long)b.table_cols << page_shift)) {
    *bad = true;
    r.len = 0;
  }
  return r;
}

// Work of one sequence under one head: tiles of R rows, the k-th costing fix + base + (k+1) R.
struct SeqWork {
  int tiles;
  long long base;   // keys before the new tokens, times g, plus the constant per tile
  __device__ __forceinline__ long long prefix(long long k, int R) const {
    return k * base + (long long)R * (k * (k + 1) / 2);
  }
};

template <int R>
__device__ __forceinline__ SeqWork seq_work(const SeqInfo& s, int g, int fix) {
  SeqWork w;
  w.tiles = (s.tokens * g + R - 1) / R;
  w.base = (long long)max(s.len - s.tokens, 0) * g + fix;
  return w;
}

// One CTA's share of one tile.
struct Segment {
  int seq, head, tile;
  SeqInfo info;
  int ta, tb, nt;       // key tiles [ta, tb) of the tile's nt
  bool owns_empty;      // the tile sees no key and this piece holds its start: write zeros
  int slot;             // partial slot: 0 when the piece begins inside the tile, else 1
  bool split;           // the tile begins in this piece and ends in a later one
  __device__ __forceinline__ bool whole() const { return ta == 0 && tb == nt; }
};

// Keys the rows of a tile see at most: those of its last row.
template <int R>
__device__ __forceinline__ int tile_keys(const SeqInfo& s, int g, int tile) {
  const int last = min((tile + 1) * R, s.tokens * g) - 1;        // rows fit 31 bits
  return max(0, s.len - s.tokens + last / g + 1);
}

// The line cut into pieces as equal as whole units allow: the first `more` are one unit longer.
struct Pieces {
  int count, more;
  long long each;
  __device__ __forceinline__ long long bound(int i) const { return each * i + min(i, more); }
  // the piece that holds line position x
  __device__ __forceinline__ int at(long long x) const {
    const long long longer = (each + 1) * more;
    return x < longer ? (int)(x / (each + 1)) : more + (int)((x - longer) / each);
  }
};

// A place on the line.
struct Located {
  int seq;
  long long into;     // offset inside the sequence
};

// Walks the tiles of a piece of the line.  All arithmetic is 64-bit and the same in every thread.
template <int R, int TK>
struct SegIter {
  const KvBatchView* b;
  int page_shift, H, g, fix;
  long long left;           // work left in the piece
  long long off;            // offset of the piece inside the current tile
  long long line;           // the current tile's place on the line
  Pieces pieces;
  int piece;
  int s, h, k;              // current sequence, head, tile
  SeqInfo info;
  SeqWork work;
  bool bad;

  __device__ __forceinline__ void start(const KvBatchView* bt, int shift, int heads, int group, int fix_,
                                        const Pieces& p, int index, const Located& at) {
    b = bt; page_shift = shift; H = heads; g = group; fix = fix_; pieces = p; piece = index; bad = false;
    left = p.bound(index + 1) - p.bound(index);
    if (left <= 0) return;
    s = at.seq;
    info = load_seq(*b, page_shift, s, &bad);
    work = seq_work<R>(info, g, fix);
    const long long per = work.prefix(work.tiles, R);
    long long into = at.into;
    h = 0;
    if (into >= per && per > 0) {
      h = (per >> 32) == 0 && (into >> 32) == 0 ? (int)((unsigned)into / (unsigned)per) : (int)(into / per);
      into -= (long long)h * per;
    }
    // largest k with prefix(k) <= into: the root of R/2 k^2 + (base + R/2) k = into, then exactly
    const float bb = (float)work.base + 0.5f * R;
    k = (int)(2.f * (float)into / (bb + sqrtf(bb * bb + 2.f * R * (float)into)));
    k = max(0, min(k, work.tiles - 1));
    while (k > 0 && work.prefix(k, R) > into) --k;
    while (k + 1 < work.tiles && work.prefix(k + 1, R) <= into) ++k;
    off = into - work.prefix(k, R);
    line = p.bound(index) - off;
  }

  __device__ __forceinline__ int key_tile(long long o, int nt) const {
    return o <= fix ? 0 : (int)min((long long)nt, div_small(o - fix, g * TK));
  }

  // Key tiles of piece p in the tile at `line` of this cost.
  __device__ __forceinline__ void share(int p, long long cost, int nt, int* ta, int* tb) const {
    const long long o0 = max(0LL, pieces.bound(p) - line), o1 = min(cost, pieces.bound(p + 1) - line);
    *ta = key_tile(o0, nt);
    *tb = o1 == cost ? nt : key_tile(o1, nt);
  }

  // After next() gave a split tile: the pieces that share it; 0 when one of them has all its key
  // tiles (and finishes it) or it has none.
  __device__ __forceinline__ int sharing(int nt) {
    if (nt == 0) return 0;
    const long long cost = work.base + (long long)k * R;    // next() went past the tile
    line -= cost;
    int ta = 0, tb = 0;
    for (int p = piece; p < pieces.count && ta == 0; ++p) {
      share(p, cost, nt, &ta, &tb);
      if (ta == 0 && tb == nt) return 0;
      if (tb > 0) break;
    }
    return pieces.at(line + cost - 1) - piece + 1;
  }

  // The next segment; false at the end of the piece.
  __device__ __forceinline__ bool next(Segment* out) {
    if (left <= 0) return false;
    while (k >= work.tiles) {          // next head, then the next sequence with rows
      k = 0;
      if (work.tiles > 0 && h + 1 < H) { ++h; break; }
      h = 0;
      ++s;
      if (s >= b->num_seqs) { left = 0; return false; }
      info = load_seq(*b, page_shift, s, &bad);
      work = seq_work<R>(info, g, fix);
    }
    const long long cost = work.base + (long long)(k + 1) * R;
    const long long end = min(cost, off + left);
    const int keys = tile_keys<R>(info, g, k);
    out->seq = s;
    out->head = h;
    out->tile = k;
    out->info = info;
    out->nt = (keys + TK - 1) / TK;
    out->ta = key_tile(off, out->nt);
    out->tb = end == cost ? out->nt : key_tile(end, out->nt);
    out->owns_empty = out->nt == 0 && off == 0;
    out->slot = off > 0 ? 0 : 1;
    out->split = off == 0 && end < cost;
    left -= end - off;
    off = 0;
    line += cost;
    ++k;
    return true;
  }
};

// The number of pieces worth cutting a line of this length into.
__device__ __forceinline__ Pieces make_pieces(long long total, int grid, int least) {
  Pieces p;
  p.count = (int)min((long long)grid, max(1LL, div_small(total, least)));
  p.each = div_small(total, p.count);
  p.more = (int)(total - p.each * p.count);
  return p;
}

// Block-wide (NT threads, NT a multiple of 32, at most 1,024) view of the line.
template <int R, int NT>
struct LineScan {
  long long warp_sum[32];
  Located at;
};

template <int R, int NT>
__device__ __forceinline__ long long seq_cost(const KvView& c, const KvBatchView& b, int g, int fix, int s,
                                              bool* bad) {
  if (s >= b.num_seqs) return 0;
  const SeqInfo i = load_seq(b, c.page_shift, s, bad);
  const SeqWork w = seq_work<R>(i, g, fix);
  return w.prefix(w.tiles, R) * c.H;
}

// Inclusive prefix sum over the block of v; *total = the block's sum.
template <int NT>
__device__ __forceinline__ long long block_scan(long long v, long long* warp_sum, long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();
  if (lane == 31) warp_sum[warp] = v;
  __syncthreads();
  long long before = 0, sum = 0;
  for (int i = 0; i < NT / 32; ++i) {
    if (i < warp) before += warp_sum[i];
    sum += warp_sum[i];
  }
  *total = sum;
  return v + before;
}

// Cuts the line and finds where piece `index` begins (all NT threads).
template <int R, int NT>
__device__ __forceinline__ void locate_piece(const KvView& c, const KvBatchView& b, int g, int fix, int grid,
                                             int least, int index, Pieces* pieces, LineScan<R, NT>* sc, bool* bad) {
  if (b.num_seqs <= 32) {              // every warp by itself; one of them writes
    const int lane = threadIdx.x & 31;
    const long long v = seq_cost<R, NT>(c, b, g, fix, lane, bad);
    long long incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += u;
    }
    *pieces = make_pieces(__shfl_sync(0xffffffffu, incl, 31), grid, least);
    if (threadIdx.x < 32 && index < pieces->count) {
      const long long x = pieces->bound(index), lo = incl - v;
      if (v > 0 && lo <= x && x < incl) {
        sc->at.seq = lane;
        sc->at.into = x - lo;
      }
    }
    __syncthreads();
    return;
  }
  long long total = 0, v0 = 0, incl0 = 0;
  for (int s0 = 0; s0 < b.num_seqs; s0 += NT) {
    const long long v = seq_cost<R, NT>(c, b, g, fix, s0 + (int)threadIdx.x, bad);
    long long sum;
    const long long incl = block_scan<NT>(v, sc->warp_sum, &sum);
    if (s0 == 0) { v0 = v; incl0 = incl; }
    total += sum;
  }
  const Pieces p = make_pieces(total, grid, least);
  *pieces = p;
  if (index < p.count) {
    const long long x = p.bound(index);
    long long before = 0;
    for (int s0 = 0; s0 < b.num_seqs; s0 += NT) {
      long long v = v0, incl = incl0, sum = 0;
      if (b.num_seqs > NT) {
        bool ignore = false;
        v = seq_cost<R, NT>(c, b, g, fix, s0 + (int)threadIdx.x, &ignore);
        incl = block_scan<NT>(v, sc->warp_sum, &sum);
      }
      const long long lo = before + incl - v;
      if (v > 0 && lo <= x && x < lo + v) {
        sc->at.seq = s0 + (int)threadIdx.x;
        sc->at.into = x - lo;
      }
      before += sum;
    }
  }
  __syncthreads();
}

// ------------------------------------------------------------------ waits that give up

// Every wait of the attention kernels is bounded.  The first that runs out marks the CTA dead and sets
// GDN_STATUS_TIMEOUT; from then on no wait blocks, no segment is begun and no copy issued; warps that
// meet in barriers go on to where they vote to leave.  Copies and products under way are waited for,
// with a limit, before the CTA ends, and an arrival never meets a phase that only its bytes keep open
// (it would be one too many).  The results are wrong, in bounds, and told by the status.
__device__ __forceinline__ bool wait_one(uint64_t* bar, uint32_t parity, volatile int* dead, int32_t* status) {
  if (tc::mbar_try_wait(bar, parity)) return true;
  if (*dead == 0) {
    if (tc::mbar_wait(bar, parity)) return true;
    *dead = 1;
    set_status(status, GDN_STATUS_TIMEOUT);
  }
  return false;
}
// The same for a whole warp, with one answer.
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* dead, int32_t* status) {
  return __all_sync(0xffffffffu, wait_one(bar, parity, dead, status));
}

constexpr uint64_t kDrainNs = 100000000;
// The copies into a ring of N stages that was left at (stage, phase).
template <int N>
__device__ __forceinline__ void drain_ring(uint64_t* full, int stage, uint32_t phase) {
  for (int i = 0; i < N; ++i) tc::mbar_wait(&full[i], i < stage ? phase : phase ^ 1u, kDrainNs);
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

// ------------------------------------------------------------------ segments, published

constexpr int kSegs = 4;           // segments known ahead

// A segment as the roles of a CTA need it: one warp walks the piece and publishes them in a ring.
struct SegDesc {
  int seq, row0, tokens, len;      // the sequence
  int head, tile, rows;            // key/value head, tile of rows and its rows
  int keys;                        // keys that the tile's last row sees
  int ta, n;                       // first key tile, number of them; n < 0: no more segments
  int whole, owns_empty, slot;
};

template <int R>
__device__ __forceinline__ SegDesc describe(const Segment& s, int g) {
  return SegDesc{s.seq, s.info.row0, s.info.tokens, s.info.len, s.head, s.tile,
                 min(R, s.info.tokens * g - s.tile * R), min(s.info.len, tile_keys<R>(s.info, g, s.tile)),
                 s.ta, max(s.tb - s.ta, 0), s.whole(), s.owns_empty, s.slot};
}

// Nothing to do for a segment: no key tiles, no zeros to write, no split tile to leave an empty
// share of.
__device__ __forceinline__ bool idle(const Segment& s) { return s.tb <= s.ta && !s.owns_empty && s.nt == 0; }

// ------------------------------------------------------------------ partial results

// A split tile, noted by the piece it begins in: its pieces are first (slot 1) and the count - 1
// after it (slot 0).
struct MergeDesc {
  int row0, tokens, head, tile, rows, count;
};

constexpr int kMaxPieces = 1024;
constexpr int kMergeWarps = 8;

// Warps of a merging block that share a row: all when many pieces have to be read one after
// another, else one each.
__host__ __device__ constexpr bool whole_block_rows(int count) { return count > 16; }

// Workspace: [G][2 slots] x (R x D floats, then R (m, l) pairs), then G descriptors and G counts
// of merging work.  The floats are rows of D for tiles of few rows, which are written and read by
// rows; for R >= 128, where a thread holds a row, [D / 4][R] groups of four columns, so that both
// sides move 32 rows' groups at a time.
template <int R, int D>
struct Partials {
  static constexpr bool kByColumns = R >= 128;
  // merging work of a tile: units of 32 rows x 32 columns, or 8 rows, or a row for a whole block
  static __host__ __device__ int work(int rows, int count) {
    return kByColumns ? (rows + 31) / 32 * (D / 32)
                      : whole_block_rows(count) ? rows : (rows + kMergeWarps - 1) / kMergeWarps;
  }
  static constexpr size_t kSlotFloats = (size_t)R * D + 2 * R;
  static __host__ __device__ size_t slots_bytes(int grid) { return (size_t)grid * 2 * kSlotFloats * 4; }
  static __host__ __device__ size_t bytes(int grid) {
    return slots_bytes(grid) + (size_t)grid * (sizeof(MergeDesc) + sizeof(int));
  }
  static __device__ __forceinline__ float* rows(float* ws, int cta, int slot) {
    return ws + ((size_t)cta * 2 + slot) * kSlotFloats;
  }
  static __device__ __forceinline__ float* ml(float* ws, int cta, int slot) {
    return rows(ws, cta, slot) + (size_t)R * D;
  }
  static __device__ __forceinline__ MergeDesc* desc(float* ws, int grid) {
    return reinterpret_cast<MergeDesc*>(reinterpret_cast<char*>(ws) + slots_bytes(grid));
  }
  static __device__ __forceinline__ int* units(float* ws, int grid) {
    return reinterpret_cast<int*>(desc(ws, grid) + grid);
  }
  // One thread of CTA cta: what the merge has to do for the tile that begins in the piece and is
  // shared by `count` (0: nothing).
  static __device__ __forceinline__ void note(float* ws, int grid, int cta, int g, const Segment* s, int count) {
    int n = 0;
    if (count > 0) {
      const int r = min(R, s->info.tokens * g - s->tile * R);
      desc(ws, grid)[cta] = MergeDesc{s->info.row0, s->info.tokens, s->head, s->tile, r, count};
      n = work(r, count);
    }
    units(ws, grid)[cta] = n;
  }
};

// ------------------------------------------------------------------ output rows

// A row (of the T * g rows under key/value head h) in the query-shaped tensors.
__device__ __forceinline__ void row_of(const SeqInfo& s, int g, int h, int r, int* tok, int* head) {
  const int t = r / g;
  *tok = s.row0 + t;
  *head = h * g + (r - t * g);
}

// sigmoid, to a few units of f32 (zero below -87); its product is rounded to bf16.  With an IEEE
// division the gate took a third of a mixed batch's time (D = 256, 2720 tokens: 205 us, so 146 us).
__device__ __forceinline__ float gate_of(float x) { return __fdividef(1.0f, 1.0f + __expf(-x)); }

// Writes 4 consecutive output elements (d a multiple of 4), gated.
__device__ __forceinline__ void store_out4(const AttnArgs& a, int D, int tok, int head, int d, float4 o) {
  if (a.gate) {
    const float4 z = Act<__nv_bfloat16>::ldg4(a.gate + tok * a.gate_ld + head * a.gate_head_ld + d);
    o.x *= gate_of(z.x); o.y *= gate_of(z.y); o.z *= gate_of(z.z); o.w *= gate_of(z.w);
  }
  Act<__nv_bfloat16>::store4(a.out + ((long long)tok * a.Hq + head) * D + d, o);
}

// The rows of the sequences: [begin, end) (loaded early, used late).
struct RowRange {
  int begin, end;
};
__device__ __forceinline__ RowRange batch_rows(const KvBatchView& b) {
  return b.num_seqs > 0 ? RowRange{__ldg(b.cu), __ldg(b.cu + b.num_seqs)} : RowRange{0, 0};
}

// Zeros in rows [begin, end).
__device__ __forceinline__ void zero_rows(const AttnArgs& a, int D, int begin, int end) {
  const long long n = (long long)(end - begin) * a.Hq * (D / 8);
  uint4* p = reinterpret_cast<uint4*>(a.out + (long long)begin * a.Hq * D);
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < n;
       i += (long long)gridDim.x * blockDim.x)
    p[i] = make_uint4(0, 0, 0, 0);
}

// In the padding rows past the last sequence, and in rows before the first (there should be none).
__device__ __forceinline__ void zero_outside(const AttnArgs& a, const KvBatchView& b, int D, RowRange rows, bool* bad) {
  if (rows.begin != 0) {
    *bad = true;
    zero_rows(a, D, 0, min(rows.begin, b.total));
  }
  if (rows.end < b.total) zero_rows(a, D, max(rows.end, 0), b.total);
}

// ------------------------------------------------------------------ merging split tiles

// A running merge of partial results (reference, sum and Q groups of four columns), a few at a time so
// that their loads are in flight together.
constexpr int kMergeBatch = 4;

template <int Q>
struct Merged {
  float top = -INFINITY, l = 0.f;
  float4 o[Q];
  __device__ __forceinline__ Merged() {
#pragma unroll
    for (int q = 0; q < Q; ++q) o[q] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __device__ __forceinline__ void add(const float2 (&ml)[kMergeBatch], const float4 (&p)[kMergeBatch][Q]) {
    float to = top;
#pragma unroll
    for (int y = 0; y < kMergeBatch; ++y) to = fmaxf(to, ml[y].x);
    if (to == -INFINITY) return;
    const float f = exp2f(top - to);      // 0 at first
    const bool first = top == -INFINITY;
    top = to;
    l = first ? 0.f : l * f;
#pragma unroll
    for (int q = 0; q < Q; ++q)
      o[q] = first ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(o[q].x * f, o[q].y * f, o[q].z * f, o[q].w * f);
#pragma unroll
    for (int y = 0; y < kMergeBatch; ++y) {
      if (ml[y].x == -INFINITY) continue;
      const float w = exp2f(ml[y].x - to);
      l = fmaf(w, ml[y].y, l);
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        o[q].x = fmaf(w, p[y][q].x, o[q].x); o[q].y = fmaf(w, p[y][q].y, o[q].y);
        o[q].z = fmaf(w, p[y][q].z, o[q].z); o[q].w = fmaf(w, p[y][q].w, o[q].w);
      }
    }
  }
};

// Merges the split tiles: each piece's rows count 2^(m - M), M the largest reference of the row.
// The work (8 rows, or one row read by all 8 warps) is spread over the grid by the counts that
// every CTA of the attention kernel left.
template <int R, int D>
__global__ void __launch_bounds__(kMergeWarps * 32) merge_kernel(const AttnArgs a, int grid) {
  constexpr int NT = kMergeWarps * 32, Q = (D + 127) / 128, kPer = kMaxPieces / NT;
  __shared__ int before[kMaxPieces + 1];
  __shared__ int warp_total[kMergeWarps];
  __shared__ float4 acc[kMergeWarps][D / 4];
  __shared__ float2 acc_ml[kMergeWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_begin();
  // prefix sums of the counts, kPer per thread
  {
    const int* units = Partials<R, D>::units(a.ws, grid);
    int v[kPer], sum = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int i = tid * kPer + j;
      v[j] = i < grid ? __ldcg(units + i) : 0;
      sum += v[j];
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += u;
    }
    if (lane == 31) warp_total[warp] = incl;
    __syncthreads();
    int base = incl - sum;
    for (int w = 0; w < warp; ++w) base += warp_total[w];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      before[tid * kPer + j] = base;
      base += v[j];
    }
    if (tid == NT - 1) before[kMaxPieces] = base;
    __syncthreads();
  }
  const int total = before[kMaxPieces];
  for (int u = blockIdx.x; u < total; u += gridDim.x) {
    int lo = 0, hi = kMaxPieces;            // the piece whose work holds u
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (before[mid] <= u) lo = mid; else hi = mid;
    }
    const MergeDesc d = Partials<R, D>::desc(a.ws, grid)[lo];
    if constexpr (Partials<R, D>::kByColumns) {
      // lane = row, warp = four columns
      const int v = u - before[lo], r = v / (D / 32) * 32 + lane, col = (v % (D / 32)) * 32 + warp * 4;
      if (r < d.rows) {
        Merged<1> acc;
        for (int j0 = 0; j0 < d.count; j0 += kMergeBatch) {
          float2 ml[kMergeBatch];
          float4 p[kMergeBatch][1];
#pragma unroll
          for (int y = 0; y < kMergeBatch; ++y) {
            const int j = j0 + y, slot = j == 0 ? 1 : 0;
            ml[y] = make_float2(-INFINITY, 0.f);
            if (j < d.count) {
              ml[y] = __ldcg(reinterpret_cast<const float2*>(Partials<R, D>::ml(a.ws, lo + j, slot) + 2 * r));
              // (where the share was empty this is whatever was there, and not used)
              p[y][0] = __ldcg(reinterpret_cast<const float4*>(Partials<R, D>::rows(a.ws, lo + j, slot)) +
                               (size_t)(col / 4) * R + r);
            }
          }
          acc.add(ml, p);
        }
        const float l = acc.l;
        const float4 o = acc.o[0];
        const float inv = l == 0.f ? 0.f : 1.0f / l;
        int tok, head;
        row_of(SeqInfo{d.row0, d.tokens, 0}, a.g, d.head, d.tile * R + r, &tok, &head);
        store_out4(a, D, tok, head, col, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
      }
      continue;
    }
    const bool together = whole_block_rows(d.count);
    const int r = together ? u - before[lo] : (u - before[lo]) * kMergeWarps + warp;
    const int j0 = together ? warp : 0, step = together ? kMergeWarps : 1;
    Merged<Q> part;
    if (r < d.rows)
      for (int jb = j0; jb < d.count; jb += step * kMergeBatch) {
        float2 ml[kMergeBatch];
        float4 p[kMergeBatch][Q];
#pragma unroll
        for (int y = 0; y < kMergeBatch; ++y) {
          const int j = jb + y * step, slot = j == 0 ? 1 : 0;
          ml[y] = make_float2(-INFINITY, 0.f);
          if (j < d.count) {
            ml[y] = __ldcg(reinterpret_cast<const float2*>(Partials<R, D>::ml(a.ws, lo + j, slot) + 2 * r));
            const float4* src = reinterpret_cast<const float4*>(Partials<R, D>::rows(a.ws, lo + j, slot) + (size_t)r * D);
#pragma unroll
            for (int q = 0; q < Q; ++q)
              if (q * 32 + lane < D / 4) p[y][q] = __ldcg(src + q * 32 + lane);
          }
        }
        part.add(ml, p);
      }
    const float4(&sum)[Q] = part.o;
    const float l = part.l, top = part.top;
    const SeqInfo info{d.row0, d.tokens, 0};
    int tok = 0, head = 0;
    if (!together) {
      if (r < d.rows) {
        const float inv = l == 0.f ? 0.f : 1.0f / l;
        row_of(info, a.g, d.head, d.tile * R + r, &tok, &head);
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          const int col = q * 32 + lane;
          if (col < D / 4)
            store_out4(a, D, tok, head, col * 4,
                       make_float4(sum[q].x * inv, sum[q].y * inv, sum[q].z * inv, sum[q].w * inv));
        }
      }
    } else {
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const int col = q * 32 + lane;
        if (col < D / 4) acc[warp][col] = sum[q];
      }
      if (lane == 0) acc_ml[warp] = make_float2(top, l);
      __syncthreads();
      if (tid < D / 4) {
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        float lt = 0.f, most = -INFINITY;
#pragma unroll
        for (int w = 0; w < kMergeWarps; ++w) most = fmaxf(most, acc_ml[w].x);
#pragma unroll
        for (int w = 0; w < kMergeWarps; ++w) {
          if (acc_ml[w].x == -INFINITY) continue;
          const float f = exp2f(acc_ml[w].x - most);
          const float4 v = acc[w][tid];
          o.x = fmaf(f, v.x, o.x); o.y = fmaf(f, v.y, o.y);
          o.z = fmaf(f, v.z, o.z); o.w = fmaf(f, v.w, o.w);
          lt = fmaf(f, acc_ml[w].y, lt);
        }
        const float inv = lt == 0.f ? 0.f : 1.0f / lt;
        row_of(info, a.g, d.head, d.tile * R + r, &tok, &head);
        store_out4(a, D, tok, head, tid * 4, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
      }
      __syncthreads();
    }
  }
}

// ------------------------------------------------------------------ launches

template <typename... KArgs, typename... Args>
inline int launch_dependent(void (*kern)(KArgs...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                            Args... args) {
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

}  // namespace attn
}  // namespace gdn
