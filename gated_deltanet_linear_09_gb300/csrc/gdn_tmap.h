// gdn_tmap.h -- TMA tensor maps of the paged cache, and the tensor copies that use them.
#pragma once

#include <cuda.h>

#include "gdn_internal.h"
#include "gdn_tc.cuh"

namespace gdn {

// Keys, values and (8-bit caches) their scale bytes.
struct KvMaps {
  CUtensorMap k, v;
};

// Maps whose box is `rows` keys of one page and head, all of head_dim: [D-blocks][rows][128 bytes]
// in shared memory, 128-byte swizzled (64-byte rows and swizzle when head_dim is 64 bytes).
bool make_kv_maps(const KvView& c, int rows, KvMaps* maps);

// Maps whose box is `rows` keys by `cols` columns: [rows][cols], swizzled over the row's bytes -- all
// but 8-bit values, which a warp reads to convert them.
bool make_tile_maps(const KvView& c, int rows, int cols, KvMaps* maps);

// A map of bf16 rows `ld` elements apart whose box is box_rows rows of box_blocks blocks of 64 columns:
// [blocks][rows][128 bytes] in shared memory, 128-byte swizzled.  Rows past the last read as zeros.
bool make_rows_map(const void* base, long long rows, long long ld, int cols, int box_rows, int box_blocks, CUtensorMap* map);

namespace attn {
int rows_grid(int D, int sms);
size_t rows_ws_bytes(int D, int sms);
// `rows` (at most 16): the most query rows of a sequence under one key/value head.
int launch_rows(const KvView& c, const KvBatchView& b, const AttnArgs& a, int rows, int sms, cudaStream_t stream);
size_t chunk_ws_bytes(int D, int sms);
int launch_chunk(const KvView& c, const KvBatchView& b, const AttnArgs& a, int sms, cudaStream_t stream);
}  // namespace attn

#ifdef __CUDACC__
namespace tc {

// Coordinates outside the map read as zero; the innermost one is always a multiple of 16 bytes.
__device__ __forceinline__ void tma_load_5d(void* dst, const CUtensorMap* map, int x0, int x1, int x2, int x3,
                                            int x4, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6, %7}], [%2];\n" ::"r"(
          smem_u32(dst)),
      "l"(map), "r"(smem_u32(bar)), "r"(x0), "r"(x1), "r"(x2), "r"(x3), "r"(x4)
      : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(smem_u32(bar)) : "memory");
}

}  // namespace tc
#endif

}  // namespace gdn
