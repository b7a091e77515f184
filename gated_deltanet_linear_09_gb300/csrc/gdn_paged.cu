// gdn_paged.cu -- the extern "C" boundary of the full-attention layers' operators: argument
// checks, tensor maps, and the choice of the attention kernel.
#include <math.h>

#include <cudaTypedefs.h>

#include "gdn_internal.h"
#include "gdn_tmap.h"

namespace gdn {

namespace {

// Number of SMs of the current device (looked up once per device).
int sm_count() {
  constexpr int kMax = 64;
  static int count[kMax] = {};   // written with the same value by every thread that finds it empty
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMax) return 0;
  int n = __atomic_load_n(&count[dev], __ATOMIC_RELAXED);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    __atomic_store_n(&count[dev], n, __ATOMIC_RELAXED);
  }
  return n;
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  return fn;
}

// The maps of keys and values (same geometry).
bool encode_all(const KvView& c, PFN_cuTensorMapEncodeTiled_v12000 encode, const cuuint64_t* dims,
                const cuuint64_t* strides, const cuuint32_t* box, CUtensorMapSwizzle swizzle_k,
                CUtensorMapSwizzle swizzle_v, KvMaps* maps) {
  const bool q8 = c.ks != nullptr;
  const cuuint32_t one[5] = {1, 1, 1, 1, 1};
  for (int i = 0; i < 2; ++i)
    if (encode(i ? &maps->v : &maps->k, q8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5,
               i ? c.v : c.k, dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, i ? swizzle_v : swizzle_k,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return false;
  return true;
}

}  // namespace

bool make_tile_maps(const KvView& c, int rows, int cols, KvMaps* maps) {
  const auto encode = encode_fn();
  if (!encode) return false;
  const bool q8 = c.ks != nullptr;
  const uint64_t elem = q8 ? 1 : 2, row = c.D * elem, span = cols * elem;
  const uint64_t P = 1ull << c.page_shift;
  const cuuint64_t dims[5] = {(cuuint64_t)cols, P, row / span, (cuuint64_t)c.H, (cuuint64_t)c.num_pages};
  const cuuint64_t strides[4] = {row, span, P * row, c.H * P * row};
  const cuuint32_t box[5] = {(cuuint32_t)cols, (cuuint32_t)rows, 1, 1, 1};
  const CUtensorMapSwizzle swizzle = span == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  return encode_all(c, encode, dims, strides, box, swizzle, q8 ? CU_TENSOR_MAP_SWIZZLE_NONE : swizzle, maps);
}

bool make_kv_maps(const KvView& c, int rows, KvMaps* maps) {
  const auto encode = encode_fn();
  if (!encode) return false;
  const bool q8 = c.ks != nullptr;
  const uint64_t elem = q8 ? 1 : 2, row = c.D * elem, span = row < 128 ? row : 128;
  const uint64_t P = 1ull << c.page_shift;
  const cuuint64_t dims[5] = {span / elem, P, row / span, (cuuint64_t)c.H, (cuuint64_t)c.num_pages};
  const cuuint64_t strides[4] = {row, span, P * row, c.H * P * row};
  const cuuint32_t box[5] = {(cuuint32_t)(span / elem), (cuuint32_t)rows, (cuuint32_t)(row / span), 1, 1};
  const CUtensorMapSwizzle swizzle = span == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  return encode_all(c, encode, dims, strides, box, swizzle, swizzle, maps);
}

size_t attn_ws_bytes(const KvView& c, int) {
  const int sms = sm_count();
  const int n = sms > 0 ? sms : 160;   // without a device (host-side sizing): at least the part's SMs
  const size_t few = attn::rows_ws_bytes(c.D, n), many = attn::chunk_ws_bytes(c.D, n);
  return few > many ? few : many;
}

int launch_attn(const KvView& c, const KvBatchView& b, const AttnArgs& a, cudaStream_t stream) {
  const int sms = sm_count();
  if (sms <= 0) return GDN_ERR_CUDA;
  const long long most = b.max_tokens > 0 ? b.max_tokens : b.total;
  if (most * a.g <= 16) return attn::launch_rows(c, b, a, (int)(most * a.g), sms, stream);
  return attn::launch_chunk(c, b, a, sms, stream);
}

}  // namespace gdn

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int check_cache(const gdn_kv_cache* cache, gdn::KvView* v, bool need_memory) {
  if (!cache) return GDN_ERR_INVALID_ARG;
  const gdn_kv_cache& c = *cache;
  if (c.type != GDN_KV_BF16 && c.type != GDN_KV_E4M3) return GDN_ERR_INVALID_ARG;
  if (c.num_kv_heads <= 0 || c.num_pages < 0 || c.page_size <= 0) return GDN_ERR_INVALID_ARG;
  if (c.head_dim != 64 && c.head_dim != 128 && c.head_dim != 256) return GDN_ERR_UNSUPPORTED_SHAPE;
  if (c.page_size < 16 || c.page_size > 256 || (c.page_size & (c.page_size - 1)) != 0)
    return GDN_ERR_UNSUPPORTED_SHAPE;
  // a page's bytes are a stride of the tensor maps (below 2^40)
  if (c.num_kv_heads > (1 << 20)) return GDN_ERR_TOO_LARGE;
  if (need_memory) {
    if (c.num_pages == 0 || !c.k_pages || !c.v_pages) return GDN_ERR_INVALID_ARG;
    if ((c.type == GDN_KV_E4M3) != (c.k_scales != nullptr) || (c.type == GDN_KV_E4M3) != (c.v_scales != nullptr))
      return GDN_ERR_INVALID_ARG;
    if (!aligned(c.k_pages, 16) || !aligned(c.v_pages, 16) || !aligned(c.k_scales, 16) || !aligned(c.v_scales, 16))
      return GDN_ERR_MISALIGNED;
  }
  int shift = 4;
  while ((1 << shift) < c.page_size) ++shift;
  *v = gdn::KvView{c.k_pages, c.v_pages, c.k_scales, c.v_scales, c.status, c.num_pages, shift, c.num_kv_heads,
                   c.head_dim};
  return GDN_OK;
}

int check_batch(const gdn_kv_batch* batch, gdn::KvBatchView* v) {
  if (!batch) return GDN_ERR_INVALID_ARG;
  const gdn_kv_batch& b = *batch;
  if (b.num_seqs < 0 || b.total_tokens < 0 || b.table_ld < 0 || b.max_tokens < 0 || b.table_cols < 0)
    return GDN_ERR_INVALID_ARG;
  const int cols = b.table_cols > 0 ? b.table_cols : b.table_ld;
  if (b.num_seqs > 65535) return GDN_ERR_TOO_LARGE;
  if (b.num_seqs == 0 && b.total_tokens > 0) return GDN_ERR_INVALID_ARG;
  if (b.num_seqs > 0 && (!b.cu_seqlens || !b.kv_lens || (cols > 0 && !b.block_table))) return GDN_ERR_INVALID_ARG;
  if (!aligned(b.cu_seqlens, 4) || !aligned(b.kv_lens, 4) || !aligned(b.block_table, 4)) return GDN_ERR_MISALIGNED;
  *v = gdn::KvBatchView{b.cu_seqlens, b.kv_lens, b.block_table, b.num_seqs, b.total_tokens, b.table_ld, b.max_tokens, cols};
  return GDN_OK;
}

}  // namespace

extern "C" {

int gdn_rms_norm(const void* x, int64_t x_ld, const void* residual, int64_t residual_ld, const void* weight,
                 float weight_offset, float eps, int32_t rows, int32_t n, gdn_dtype act, gdn_norm_out out_kind,
                 void* sum_out, void* y, float* scales, cudaStream_t stream) {
  GDN_CALL_RANGE("gdn_rms_norm");
  if (act != GDN_F32 && act != GDN_BF16) return GDN_ERR_INVALID_ARG;
  if (out_kind != GDN_NORM_ACT && out_kind != GDN_NORM_E4M3_ROW && out_kind != GDN_NORM_E4M3_BLOCK)
    return GDN_ERR_INVALID_ARG;
  if (rows < 0 || n < 1 || !(eps >= 0.f) || !isfinite(eps) || !isfinite(weight_offset)) return GDN_ERR_INVALID_ARG;
  if (n > GDN_MAX_NORM_WIDTH) return GDN_ERR_TOO_LARGE;
  if (rows == 0) return GDN_OK;
  if (!x || !weight || !y || (out_kind != GDN_NORM_ACT && !scales)) return GDN_ERR_INVALID_ARG;
  if (x_ld < n || (residual && residual_ld < n)) return GDN_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(sum_out, 16) ||
      !aligned(y, 16) || !aligned(scales, 16))
    return GDN_ERR_MISALIGNED;
  return gdn::launch_rms_norm(x, x_ld, residual, residual_ld, weight, weight_offset, eps, rows, n, act,
                              (int)out_kind, sum_out, y, scales, stream);
}

int gdn_kv_append(const gdn_kv_cache* cache, const gdn_kv_batch* batch, const void* k, int64_t k_ld, const void* v,
                  int64_t v_ld, cudaStream_t stream) {
  GDN_CALL_RANGE("gdn_kv_append");
  gdn::KvView c;
  gdn::KvBatchView b;
  int rc;
  if ((rc = check_cache(cache, &c, true)) != GDN_OK) return rc;
  if ((rc = check_batch(batch, &b)) != GDN_OK) return rc;
  const int64_t width = (int64_t)c.H * c.D;
  if (k_ld < width || v_ld < width) return GDN_ERR_INVALID_ARG;
  if (b.total == 0) return GDN_OK;
  if (!k || !v) return GDN_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || k_ld % 8 != 0 || v_ld % 8 != 0) return GDN_ERR_MISALIGNED;
  if ((int64_t)b.total * width > (1LL << 38)) return GDN_ERR_TOO_LARGE;
  return gdn::launch_kv_append(c, b, k, k_ld, v, v_ld, stream);
}

int gdn_kv_read(const gdn_kv_cache* cache, const gdn_kv_batch* batch, void* k, void* v, cudaStream_t stream) {
  GDN_CALL_RANGE("gdn_kv_read");
  gdn::KvView c;
  gdn::KvBatchView b;
  int rc;
  if ((rc = check_cache(cache, &c, true)) != GDN_OK) return rc;
  if ((rc = check_batch(batch, &b)) != GDN_OK) return rc;
  if (b.total == 0) return GDN_OK;
  if (!k || !v) return GDN_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16)) return GDN_ERR_MISALIGNED;
  if ((int64_t)b.total * c.H * c.D > (1LL << 38)) return GDN_ERR_TOO_LARGE;
  return gdn::launch_kv_read(c, b, k, v, stream);
}

size_t gdn_paged_attention_workspace_bytes(const gdn_kv_cache* cache, int32_t num_q_heads) {
  gdn::KvView c;
  if (check_cache(cache, &c, false) != GDN_OK || num_q_heads <= 0 || num_q_heads % c.H != 0) return 0;
  return gdn::attn_ws_bytes(c, num_q_heads);
}

int gdn_paged_attention(const gdn_kv_cache* cache, const gdn_kv_batch* batch, int32_t num_q_heads, const void* q,
                        int64_t q_ld, int64_t q_head_ld, const void* gate, int64_t gate_ld, int64_t gate_head_ld,
                        float scale, void* out, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  GDN_CALL_RANGE("gdn_paged_attention");
  gdn::KvView c;
  gdn::KvBatchView b;
  int rc;
  if ((rc = check_cache(cache, &c, true)) != GDN_OK) return rc;
  if ((rc = check_batch(batch, &b)) != GDN_OK) return rc;
  if (num_q_heads <= 0 || !(scale >= 0.f) || !isfinite(scale)) return GDN_ERR_INVALID_ARG;
  if (num_q_heads % c.H != 0) return GDN_ERR_HEAD_DIVISIBILITY;
  // (a group's factor of the work's units: thousands of keys times it fit 31 bits)
  if ((int64_t)b.total * num_q_heads > (1LL << 30) || num_q_heads / c.H > (1 << 20)) return GDN_ERR_TOO_LARGE;
  if (b.total == 0) return GDN_OK;
  if (!q || !out) return GDN_ERR_INVALID_ARG;
  if (q_ld < c.D || q_head_ld < c.D || (gate && (gate_ld < c.D || gate_head_ld < c.D))) return GDN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(out, 16) || q_ld % 8 != 0 || q_head_ld % 8 != 0) return GDN_ERR_MISALIGNED;
  if (gate && (!aligned(gate, 16) || gate_ld % 8 != 0 || gate_head_ld % 8 != 0)) return GDN_ERR_MISALIGNED;
  if (!workspace || workspace_bytes < gdn::attn_ws_bytes(c, num_q_heads)) return GDN_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned(workspace, 256)) return GDN_ERR_MISALIGNED;
  gdn::AttnArgs a;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.gate = static_cast<const __nv_bfloat16*>(gate);
  a.out = static_cast<__nv_bfloat16*>(out);
  a.q_ld = q_ld;
  a.q_head_ld = q_head_ld;
  a.gate_ld = gate_ld;
  a.gate_head_ld = gate_head_ld;
  a.Hq = num_q_heads;
  a.g = num_q_heads / c.H;
  a.scale_log2 = (float)((scale > 0.f ? (double)scale : 1.0 / sqrt((double)c.D)) * 1.4426950408889634);
  a.ws = static_cast<float*>(workspace);
  return gdn::launch_attn(c, b, a, stream);
}

}  // extern "C"
