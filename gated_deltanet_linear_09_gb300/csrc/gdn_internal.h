// gdn_internal.h -- declarations shared by the host API and the kernel translation units.
#pragma once

#include "gdn_common.cuh"
#include "gdn_device.h"

// NVTX ranges around the C-ABI calls: a profiler or tracer attached to the process sees each call
// as a named range on the calling thread (with none attached a range costs a few nanoseconds).
// Compiled out when the NVTX headers are not available.
#if defined(__has_include)
#if __has_include(<nvtx3/nvToolsExt.h>)
#include <nvtx3/nvToolsExt.h>
#define GDN_NVTX 1
#endif
#endif

namespace gdn {

struct CallRange {
  explicit CallRange(const char* name) {
#ifdef GDN_NVTX
    nvtxRangePushA(name);
#else
    (void)name;
#endif
  }
  ~CallRange() {
#ifdef GDN_NVTX
    nvtxRangePop();
#endif
  }
  CallRange(const CallRange&) = delete;
  CallRange& operator=(const CallRange&) = delete;
};
#define GDN_CALL_RANGE(name) ::gdn::CallRange gdn_call_range_(name)

int launch_decode(const KDims& d, const gdn_weights* w, const gdn_pool* pool,
                  const int32_t* slot_idx, int B, const void* qkv, const void* z, const void* a,
                  const void* b, void* out, cudaStream_t stream);

int launch_decode_multi(const KDims& d, const gdn_weights* w, const gdn_pool* pool,
                        const int32_t* slot_idx, int B, int TT, const void* qkv, const void* z,
                        const void* a, const void* b, void* out, cudaStream_t stream);

int launch_conv1d_update(const KDims& d, const gdn_weights* w, const gdn_pool* pool,
                         const int32_t* slot_idx, int B, const void* in, void* out,
                         cudaStream_t stream);

struct CompactPairs {
  int32_t src[GDN_MAX_COMPACT_PAIRS];
  int32_t dst[GDN_MAX_COMPACT_PAIRS];
};

int launch_compact(const CompactPairs& pairs, int n, void* rec, size_t rec_slot_bytes, void* conv,
                   size_t conv_slot_bytes, cudaStream_t stream);

// Workspace carve-up of the chunkwise prefill.
struct PrefillWs {
  float* qk;      // [T][Hk][2][dk]   l2-normalised q (scaled) and k
  float* vu;      // [T][Hv][dv]      v after conv+SiLU, then U~ = T diag(beta) V, then U
  float* w;       // [T][Hv][dk]      W = T diag(beta e^gamma) K
  float* gb;      // [T][Hv][2]       (g, beta), g replaced by the in-chunk cumulative gamma
  float* sc;      // [NCmax][Hv][dk][dv] state at the start of every chunk
  size_t bytes;
};

PrefillWs prefill_ws_layout(const KDims& d, int num_seqs, int total_tokens, void* base);

int launch_prefill(const KDims& d, const gdn_weights* w, const gdn_pool* pool,
                   const int32_t* cu_seqlens, const int32_t* slot_idx, const uint8_t* has_init,
                   int num_seqs, int total_tokens, const void* qkv, const void* z, const void* a,
                   const void* b, void* out, const PrefillWs& ws, cudaStream_t stream);

// Tensor-core (tcgen05) prefill for dk = dv = 128.
bool prefill_tc_supported(const KDims& d);
size_t prefill_tc_ws_bytes(const KDims& d, int num_seqs, int total_tokens);
// The smallest workspace the tensor-core prefill accepts: the records of one chunk.  Smaller
// workspaces than prefill_tc_ws_bytes run the call in windows of whole chunks.
size_t prefill_tc_ws_min_bytes(const KDims& d);
int launch_prefill_tc(const KDims& d, const gdn_weights* w, const gdn_pool* pool,
                      const int32_t* cu_seqlens, const int32_t* slot_idx, const uint8_t* has_init,
                      int num_seqs, int total_tokens, const void* qkv, const void* z, const void* a,
                      const void* b, void* out, void* ws, size_t ws_bytes, cudaStream_t stream);

// Dense bf16 projection (tcgen05 GEMM) with a routing epilogue: output feature n of row m goes
// to ptr[s][m * ld[s] + n - start[s]] for the segment s holding n.
struct ProjRoute {
  int nseg;
  int start[GDN_MAX_PROJ_SEGMENTS];
  int ld[GDN_MAX_PROJ_SEGMENTS];
  __nv_bfloat16* ptr[GDN_MAX_PROJ_SEGMENTS];
};

// Contraction split the library picks for an M x N x K projection (1 to 8).
int proj_auto_split(int M, int N, int K);
size_t proj_packed_bytes(int N, int K);
int launch_proj_pack(const void* w, int N, int K, void* packed, cudaStream_t stream);
int launch_proj(const void* x, const void* wp, int M, int N, int K, int ks, const ProjRoute& route,
                int32_t* status, cudaStream_t stream);

// Raises a kernel's dynamic shared memory to `bytes` (0: to the most a block can have) on the current
// device, once on each, so that launches -- also those recorded into a CUDA graph -- need not.
template <typename K>
int raise_smem(OncePerDevice& once, K kern, size_t bytes) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return GDN_ERR_CUDA;
  return once.run(dev, [&]() -> int {
    int most = (int)bytes;
    if (bytes == 0 && cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) != cudaSuccess)
      return GDN_ERR_CUDA;
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most) == cudaSuccess ? GDN_OK
                                                                                                  : GDN_ERR_CUDA;
  });
}

// Number of SMs of the current device (looked up once per device); 0 without one.
int sm_count();

// RMSNorm with the residual's addition (kind: a gdn_norm_out).
int launch_rms_norm(const void* x, long long x_ld, const void* residual, long long residual_ld,
                    const void* weight, float weight_offset, float eps, int rows, int n,
                    gdn_dtype act, int kind, void* sum_out, void* y, float* scales,
                    cudaStream_t stream);

// The paged key/value cache and the new tokens of a call, by value to every kernel.
struct KvView {
  void* k;
  void* v;
  uint8_t* ks;    // exponent bytes; NULL for a bf16 cache
  uint8_t* vs;
  int32_t* status;
  int num_pages, page_shift, H, D;
};

struct KvBatchView {
  const int32_t* cu;
  const int32_t* lens;
  const int32_t* table;
  int num_seqs, total, table_ld, max_tokens, table_cols;
};

int launch_kv_append(const KvView& c, const KvBatchView& b, const void* k, long long k_ld,
                     const void* v, long long v_ld, cudaStream_t stream);
int launch_kv_read(const KvView& c, const KvBatchView& b, void* k, void* v, cudaStream_t stream);

// Rotary positions of queries and keys (outputs dense).
struct RotaryLaunch {
  const void* q;
  const void* k;
  void* q_out;
  void* k_out;
  long long q_ld, q_head_ld, k_ld, k_head_ld;
  const uint64_t* turns;
  const int32_t* positions;
  float scale;
  int rot, interleaved, tokens, dim, q_heads, k_heads;
};
int launch_rotary(const RotaryLaunch& r, gdn_dtype act, cudaStream_t stream);

// The cache's append with the heads' norm and rotation.
struct RotatedAppend {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  __nv_bfloat16* q_out;
  long long q_ld, q_head_ld, k_ld, v_ld;
  const __nv_bfloat16* q_norm;
  const __nv_bfloat16* k_norm;
  const uint64_t* turns;
  const int32_t* positions;
  float scale, w0, eps;
  int Hq, half, interleaved;
};
int launch_kv_append_rotated(const KvView& c, const KvBatchView& b, const RotatedAppend& a, cudaStream_t stream);

int launch_block_norm(const gdn_block_args& a, int rows, int n, gdn_dtype act, cudaStream_t stream);

// Linear attention with a decay for each head.
struct DecayView {
  float* state;
  int32_t* status;
  int num_slots, Hk, Hv, dk, dv;
  float scale;
};
int launch_decay_step(const DecayView& l, const gdn_decay_tokens& t, const int32_t* slot_idx, int B, int T,
                      cudaStream_t stream);
size_t decay_prefill_ws_bytes(const DecayView& l, int num_seqs, int total_tokens);
int launch_decay_prefill(const DecayView& l, const gdn_decay_tokens& t, const int32_t* cu_seqlens,
                         const int32_t* slot_idx, const uint8_t* has_init, int num_seqs, int total_tokens,
                         void* workspace, cudaStream_t stream);

struct AttnArgs {
  const __nv_bfloat16* q;
  const __nv_bfloat16* gate;
  __nv_bfloat16* out;
  long long q_ld, q_head_ld, gate_ld, gate_head_ld;
  int Hq, g;           // query heads; query heads per key/value head
  float scale_log2;    // softmax scale times log2(e)
  float* ws;
};

size_t attn_ws_bytes(const KvView& c, int Hq);
int launch_attn(const KvView& c, const KvBatchView& b, const AttnArgs& a, cudaStream_t stream);

}  // namespace gdn
