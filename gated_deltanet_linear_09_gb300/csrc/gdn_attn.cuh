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

__device__ __forceinline__ SeqInfo load_seq(const KvBatchView& b, int page_shift, int s, bool* bad) {
  const int c0 = __ldg(b.cu + s), c1 = __ldg(b.cu + s + 1), len = __ldg(b.lens + s);
  SeqInfo r{c0, c1 - c0, len};
  if (c0 < 0 || c1 < c0 || c1 > b.total) {
    *bad = true;
    r.row0 = r.tokens = r.len = 0;
  } else if (len < 0 || len > ((long long)b.table_ld << page_shift)) {
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
  w.tiles = (int)(((long long)s.tokens * g + R - 1) / R);
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
  __device__ __forceinline__ bool whole() const { return ta == 0 && tb == nt; }
};

// Keys the rows of a tile see at most: those of its last row.
template <int R>
__device__ __forceinline__ int tile_keys(const SeqInfo& s, int g, int tile) {
  const long long last = min((long long)(tile + 1) * R, (long long)s.tokens * g) - 1;
  return max(0, s.len - s.tokens + (int)(last / g) + 1);
}

// Walks the tiles of a piece of the line.  All arithmetic is 64-bit and the same in every thread.
template <int R, int TK>
struct SegIter {
  const KvBatchView* b;
  int page_shift, H, g, fix;
  long long left;           // work left in the piece
  long long off;            // offset of the piece inside the current tile
  int s, h, k;              // current sequence, head, tile
  SeqInfo info;
  SeqWork work;
  bool bad;

  __device__ __forceinline__ void start(const KvBatchView* bt, int shift, int heads, int group, int fix_,
                                        int seq, long long into, long long amount) {
    b = bt; page_shift = shift; H = heads; g = group; fix = fix_; left = amount; s = seq; bad = false;
    if (left <= 0) return;
    info = load_seq(*b, page_shift, s, &bad);
    work = seq_work<R>(info, g, fix);
    const long long per = work.prefix(work.tiles, R);
    h = 0;
    if (into >= per && per > 0) {        // heads are few: a division would cost as much
      h = (int)(into / per);
    }
    into -= (long long)h * per;
    int lo = 0, hi = work.tiles;      // largest k with prefix(k) <= into
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (work.prefix(mid, R) <= into) lo = mid; else hi = mid;
    }
    k = lo;
    off = into - work.prefix(k, R);
  }

  __device__ __forceinline__ int key_tile(long long o, int nt) const {
    return o <= fix ? 0 : (int)min((long long)nt, div_small(o - fix, g * TK));
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
    left -= end - off;
    off = 0;
    ++k;
    return true;
  }
};

// The line cut into pieces as equal as whole units allow: the first `more` are one unit longer.
struct Pieces {
  int count, more;
  long long each;
  __device__ __forceinline__ long long bound(int i) const { return each * i + min(i, more); }
};

// The number of pieces worth cutting a line of this length into.
__device__ __forceinline__ Pieces make_pieces(long long total, int grid, int least) {
  Pieces p;
  p.count = (int)min((long long)grid, max(1LL, div_small(total, least)));
  p.each = div_small(total, p.count);
  p.more = (int)(total - p.each * p.count);
  return p;
}

// Block-wide (NT threads, NT a multiple of 32, at most 1,024): the total work of all sequences,
// and where the line positions x[0..NX) (given as functions of the total by `bounds`) fall.
struct Located {
  int seq;
  long long into;     // offset inside the sequence
};

template <int R, int NT>
struct LineScan {
  long long warp_sum[32];
  long long total;
  Located at[2];
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

// Fills sc->total and sc->at[i] for the piece bounds first, first + 1 (all NT threads).  A bound at
// the very end of the line is located past the last sequence.
template <int R, int NT>
__device__ __forceinline__ void locate_piece(const KvView& c, const KvBatchView& b, int g, int fix, int grid,
                                             int least, int first, Pieces* pieces, LineScan<R, NT>* sc,
                                             bool* bad) {
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
  if (threadIdx.x == 0) {
    sc->total = total;
    sc->at[0].seq = sc->at[1].seq = b.num_seqs;
    sc->at[0].into = sc->at[1].into = 0;
  }
  __syncthreads();
  long long before = 0;
  for (int s0 = 0; s0 < b.num_seqs; s0 += NT) {
    long long v = v0, incl = incl0, sum = 0;
    if (s0 > 0 || b.num_seqs > NT) {
      bool ignore = false;
      v = seq_cost<R, NT>(c, b, g, fix, s0 + (int)threadIdx.x, &ignore);
      incl = block_scan<NT>(v, sc->warp_sum, &sum);
    }
    const long long lo = before + incl - v, hi = before + incl;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (first + i > p.count) continue;
      const long long x = p.bound(first + i);
      if (v > 0 && lo <= x && x < hi) {
        sc->at[i].seq = s0 + (int)threadIdx.x;
        sc->at[i].into = x - lo;
      }
    }
    before += sum;
  }
  __syncthreads();
}

// ------------------------------------------------------------------ partial results

// Slot layout: [G][2 slots] x ( R x D floats, then R (m, l) pairs ).
template <int R, int D>
struct Partials {
  static constexpr size_t kSlotFloats = (size_t)R * D + 2 * R;
  static __host__ __device__ size_t bytes(int grid) { return (size_t)grid * 2 * kSlotFloats * 4; }
  static __device__ __forceinline__ float* rows(float* ws, int cta, int slot) {
    return ws + ((size_t)cta * 2 + slot) * kSlotFloats;
  }
  static __device__ __forceinline__ float* ml(float* ws, int cta, int slot) {
    return rows(ws, cta, slot) + (size_t)R * D;
  }
};

// ------------------------------------------------------------------ output rows

// A row (of the T * g rows under key/value head h) in the query-shaped tensors.
__device__ __forceinline__ void row_of(const SeqInfo& s, int g, int h, int r, int* tok, int* head) {
  const int t = r / g;
  *tok = s.row0 + t;
  *head = h * g + (r - t * g);
}

__device__ __forceinline__ float gate_of(float x) { return 1.0f / (1.0f + __expf(-x)); }

// Writes 4 consecutive output elements (d a multiple of 4), gated.
__device__ __forceinline__ void store_out4(const AttnArgs& a, int D, int tok, int head, int d, float4 o) {
  if (a.gate) {
    const float4 z = Act<__nv_bfloat16>::ldg4(a.gate + tok * a.gate_ld + head * a.gate_head_ld + d);
    o.x *= gate_of(z.x); o.y *= gate_of(z.y); o.z *= gate_of(z.z); o.w *= gate_of(z.w);
  }
  Act<__nv_bfloat16>::store4(a.out + ((long long)tok * a.Hq + head) * D + d, o);
}

// Zeros in the padding rows past the last sequence.
__device__ __forceinline__ void zero_padding(const AttnArgs& a, const KvBatchView& b, int D) {
  const int end = b.num_seqs > 0 ? __ldg(b.cu + b.num_seqs) : 0;
  if (end < 0 || end >= b.total) return;
  const long long n = (long long)(b.total - end) * a.Hq * (D / 8);
  uint4* p = reinterpret_cast<uint4*>(a.out + (long long)end * a.Hq * D);
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < n;
       i += (long long)gridDim.x * blockDim.x)
    p[i] = make_uint4(0, 0, 0, 0);
}

// ------------------------------------------------------------------ merging split tiles

// Block (i, y) looks at the bound between pieces i and i + 1.  If it falls inside a tile and is the
// first to do so, the block merges rows y, y + gridDim.y, ... of the tile over the pieces that
// share it: each piece's rows count 2^(m - M), M the largest reference.
constexpr int kMaxPieces = 1024;

template <int R, int TK, int D>
__global__ void __launch_bounds__(256) merge_kernel(const KvView c, const KvBatchView b, const AttnArgs a,
                                                    int grid, int fix, int least) {
  constexpr int NT = 256, W = NT / 32, Q = (D + 127) / 128;
  __shared__ LineScan<R, NT> scan;
  __shared__ float4 acc[W][D / 4];
  __shared__ float acc_l[W];
  __shared__ int source[kMaxPieces];      // partial slot of each piece of the tile, -1: it left none
  __shared__ float weight[kMaxPieces];
  pdl_begin();
  bool bad = false;
  Pieces pieces;
  const int i = blockIdx.x;
  locate_piece<R, NT>(c, b, a.g, fix, grid, least, i, &pieces, &scan, &bad);
  if (i + 1 >= pieces.count) return;
  const long long x = pieces.bound(i + 1), x_prev = pieces.bound(i);
  if (x == x_prev) return;
  // the tile that holds x
  SegIter<R, TK> it;
  it.start(&b, c.page_shift, c.H, a.g, fix, scan.at[1].seq, scan.at[1].into, 1);
  if (it.off == 0) return;                              // a tile begins at the bound
  const long long t0 = x - it.off;                      // the tile's place on the line
  if (x_prev > t0) return;                              // an earlier bound lies inside this tile
  const long long cost = it.work.base + (long long)(it.k + 1) * R;
  const int keys = tile_keys<R>(it.info, a.g, it.k);
  const int nt = (keys + TK - 1) / TK;
  if (nt == 0) return;                                  // zeros, written by piece i
  const int rows = (int)min((long long)R, (long long)it.info.tokens * a.g - (long long)it.k * R);
  if ((int)blockIdx.y >= rows) return;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // the pieces i .. i + count - 1 share the tile
  int count = 0;
  bool one = false;
  for (int j0 = 0;; j0 += NT) {
    const int j = j0 + tid, p = i + j;
    const bool in = p < pieces.count && pieces.bound(p) < t0 + cost;
    if (in) {
      const long long o0 = max(0LL, pieces.bound(p) - t0), o1 = min(cost, pieces.bound(p + 1) - t0);
      const int ta = it.key_tile(o0, nt), tb = o1 == cost ? nt : it.key_tile(o1, nt);
      source[j] = ta < tb ? 2 * p + (o0 > 0 ? 0 : 1) : -1;
      one |= ta == 0 && tb == nt;                       // one piece did it all and finished it
    }
    const int n = __syncthreads_count(in);
    count += n;
    if (n < NT) break;
  }
  if (__syncthreads_or(one)) return;
  for (int r = blockIdx.y; r < rows; r += gridDim.y) {
    float top = -INFINITY;
    for (int j = tid; j < count; j += NT) {
      const int s = source[j];
      const float m = s < 0 ? -INFINITY : __ldcg(Partials<R, D>::ml(a.ws, s >> 1, s & 1) + 2 * r);
      weight[j] = m;
      top = fmaxf(top, m);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) acc_l[warp] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < W; ++w) top = fmaxf(top, acc_l[w]);
    __syncthreads();
    float4 sum[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) sum[q] = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
#pragma unroll 4
    for (int j = warp; j < count; j += W) {
      const float m = weight[j];
      if (m == -INFINITY) continue;
      const int s = source[j];
      const float w = exp2f(m - top);
      l += w * __ldcg(Partials<R, D>::ml(a.ws, s >> 1, s & 1) + 2 * r + 1);
      const float4* src = reinterpret_cast<const float4*>(Partials<R, D>::rows(a.ws, s >> 1, s & 1) + (size_t)r * D);
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const int col = q * 32 + lane;
        if (col < D / 4) {
          const float4 v = __ldcg(src + col);
          sum[q].x = fmaf(w, v.x, sum[q].x); sum[q].y = fmaf(w, v.y, sum[q].y);
          sum[q].z = fmaf(w, v.z, sum[q].z); sum[q].w = fmaf(w, v.w, sum[q].w);
        }
      }
    }
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int col = q * 32 + lane;
      if (col < D / 4) acc[warp][col] = sum[q];
    }
    if (lane == 0) acc_l[warp] = l;
    __syncthreads();
    if (tid < D / 4) {
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      float lt = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float4 v = acc[w][tid];
        o.x += v.x; o.y += v.y; o.z += v.z; o.w += v.w;
        lt += acc_l[w];
      }
      const float inv = lt == 0.f ? 0.f : 1.0f / lt;
      o.x *= inv; o.y *= inv; o.z *= inv; o.w *= inv;
      int tok, head;
      row_of(it.info, a.g, it.h, it.k * R + r, &tok, &head);
      store_out4(a, D, tok, head, tid * 4, o);
    }
    __syncthreads();
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
