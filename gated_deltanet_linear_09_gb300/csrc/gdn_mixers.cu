// gdn_mixers.cu -- the extern "C" boundary of the operators between a layer's projections (the cache's
// rotated append stands with the cache's other calls): argument checks, one launch each.
#include <math.h>

#include "gdn_internal.h"

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

bool dense(int tokens, int heads, int dim, int64_t ld, int64_t head_ld) {
  return (heads == 1 || head_ld == dim) && (tokens == 1 || ld == (int64_t)heads * dim);
}

int check_layer(const gdn_decay_layer* layer, gdn::DecayView* v, bool need_memory) {
  if (!layer) return GDN_ERR_INVALID_ARG;
  const gdn_decay_layer& l = *layer;
  if (l.num_k_heads <= 0 || l.num_v_heads <= 0 || !(l.scale >= 0.f) || !isfinite(l.scale)) return GDN_ERR_INVALID_ARG;
  if (l.num_v_heads % l.num_k_heads != 0) return GDN_ERR_HEAD_DIVISIBILITY;
  if ((l.head_k_dim != 64 && l.head_k_dim != 128) || (l.head_v_dim != 64 && l.head_v_dim != 128))
    return GDN_ERR_UNSUPPORTED_SHAPE;
  if (l.num_v_heads > 65535) return GDN_ERR_TOO_LARGE;      // (a dimension of the grids)
  if (need_memory) {
    if (!l.state || l.num_slots <= 0) return GDN_ERR_INVALID_ARG;
    if (!aligned(l.state, 16)) return GDN_ERR_MISALIGNED;
  }
  *v = gdn::DecayView{l.state, l.status, l.num_slots, l.num_k_heads, l.num_v_heads, l.head_k_dim, l.head_v_dim,
                      l.scale > 0.f ? l.scale : 1.0f / sqrtf((float)l.head_k_dim)};
  return GDN_OK;
}

int check_tokens(const gdn_decay_tokens* tokens, const gdn::DecayView& l, long long count) {
  if (!tokens) return GDN_ERR_INVALID_ARG;
  if (count == 0) return GDN_OK;
  const gdn_decay_tokens& t = *tokens;
  if (!t.q || !t.k || !t.v || !t.log_decay || !t.out) return GDN_ERR_INVALID_ARG;
  const int64_t kw = (int64_t)l.Hk * l.dk, vw = (int64_t)l.Hv * l.dv;
  if (t.q_ld < kw || t.k_ld < kw || t.v_ld < vw || (t.decay_ld != 0 && t.decay_ld < l.Hv)) return GDN_ERR_INVALID_ARG;
  if (!aligned(t.q, 16) || !aligned(t.k, 16) || !aligned(t.v, 16) || !aligned(t.out, 16) || !aligned(t.log_decay, 4) ||
      t.q_ld % 8 != 0 || t.k_ld % 8 != 0 || t.v_ld % 8 != 0)
    return GDN_ERR_MISALIGNED;
  return GDN_OK;
}

// The outputs are not the inputs.
bool apart(const gdn_decay_tokens& t, long long count) { return count == 0 || (t.out != t.q && t.out != t.k && t.out != t.v); }

}  // namespace

extern "C" {

int gdn_rotary_apply(const gdn_rotary* rotary, const int32_t* positions, int32_t tokens, int32_t head_dim,
                     gdn_dtype act, const void* q, int64_t q_ld, int64_t q_head_ld, int32_t q_heads, void* q_out,
                     const void* k, int64_t k_ld, int64_t k_head_ld, int32_t k_heads, void* k_out,
                     cudaStream_t stream) {
  GDN_CALL_RANGE("gdn_rotary_apply");
  if (!rotary || (act != GDN_F32 && act != GDN_BF16)) return GDN_ERR_INVALID_ARG;
  if (tokens < 0 || head_dim < 1 || q_heads < 0 || k_heads < 0 || !isfinite(rotary->scale)) return GDN_ERR_INVALID_ARG;
  if (rotary->rot_dim < 2 || rotary->rot_dim % 2 != 0 || rotary->rot_dim > head_dim) return GDN_ERR_UNSUPPORTED_SHAPE;
  if (head_dim > GDN_MAX_ROTARY_DIM || q_heads > 65536 || k_heads > 65536) return GDN_ERR_TOO_LARGE;
  if (tokens == 0 || q_heads + k_heads == 0) return GDN_OK;
  if (!rotary->turns || !positions) return GDN_ERR_INVALID_ARG;
  if (!aligned(rotary->turns, 8) || !aligned(positions, 4)) return GDN_ERR_MISALIGNED;
  const uintptr_t size = act == GDN_BF16 ? 2 : 4;
  if (q_heads > 0) {
    if (!q || !q_out || q_ld < head_dim || q_head_ld < head_dim) return GDN_ERR_INVALID_ARG;
    if (!aligned(q, size) || !aligned(q_out, size)) return GDN_ERR_MISALIGNED;
    if (q_out == q && !dense(tokens, q_heads, head_dim, q_ld, q_head_ld)) return GDN_ERR_INVALID_ARG;
  }
  if (k_heads > 0) {
    if (!k || !k_out || k_ld < head_dim || k_head_ld < head_dim) return GDN_ERR_INVALID_ARG;
    if (!aligned(k, size) || !aligned(k_out, size)) return GDN_ERR_MISALIGNED;
    if (k_out == k && !dense(tokens, k_heads, head_dim, k_ld, k_head_ld)) return GDN_ERR_INVALID_ARG;
  }
  if (q_heads > 0 && k_heads > 0 && (q_out == k || k_out == q || q_out == k_out)) return GDN_ERR_INVALID_ARG;
  const gdn::RotaryLaunch r{q_heads ? q : nullptr, k_heads ? k : nullptr, q_heads ? q_out : nullptr, k_heads ? k_out : nullptr,
                            q_heads ? q_ld : 0, q_heads ? q_head_ld : 0, k_heads ? k_ld : 0, k_heads ? k_head_ld : 0,
                            rotary->turns, positions, rotary->scale, rotary->rot_dim, rotary->interleaved != 0, tokens,
                            head_dim, q_heads, k_heads};
  return gdn::launch_rotary(r, act, stream);
}

int gdn_block_norm(const gdn_block_args* args, int32_t rows, int32_t n, gdn_dtype act, cudaStream_t stream) {
  GDN_CALL_RANGE("gdn_block_norm");
  if (!args || (act != GDN_F32 && act != GDN_BF16) || rows < 0 || n < 1) return GDN_ERR_INVALID_ARG;
  const gdn_block_args& a = *args;
  if (!(a.eps >= 0.f) || !isfinite(a.eps) || !isfinite(a.weight_offset) || !isfinite(a.scale)) return GDN_ERR_INVALID_ARG;
  if (a.gate_act != GDN_GATE_NONE && a.gate_act != GDN_GATE_SIGMOID && a.gate_act != GDN_GATE_SILU) return GDN_ERR_INVALID_ARG;
  if (n > GDN_MAX_NORM_WIDTH) return GDN_ERR_TOO_LARGE;
  if (a.group != n && ((a.group != 32 && a.group != 64 && a.group != 128 && a.group != 256) || n % a.group != 0))
    return GDN_ERR_UNSUPPORTED_SHAPE;
  if (rows == 0) return GDN_OK;
  if (!a.x || (a.gate != nullptr) != (a.gate_act != GDN_GATE_NONE) || (a.pre != nullptr) != (a.y != nullptr))
    return GDN_ERR_INVALID_ARG;
  if (!a.total && !a.y) return GDN_ERR_INVALID_ARG;
  if (a.x_ld < n || (a.gate && a.gate_ld < n) || (a.residual && a.residual_ld < n)) return GDN_ERR_INVALID_ARG;
  for (const void* p : {a.x, a.gate, a.residual, a.post, a.pre, a.channel_scale, (const void*)a.total, (const void*)a.y})
    if (!aligned(p, 16)) return GDN_ERR_MISALIGNED;
  if (a.post && a.group != n && (a.x_ld % 8 != 0 || (a.gate && a.gate_ld % 8 != 0) || (a.residual && a.residual_ld % 8 != 0)))
    return GDN_ERR_MISALIGNED;
  if (a.total == a.y) return GDN_ERR_INVALID_ARG;
  // (dense outputs in the place of rows further apart: over rows that other CTAs have yet to read)
  for (const void* out : {(const void*)a.total, (const void*)a.y})
    if (rows > 1 && out && ((out == a.x && a.x_ld != n) || (out == a.gate && a.gate_ld != n) || (out == a.residual && a.residual_ld != n)))
      return GDN_ERR_INVALID_ARG;
  return gdn::launch_block_norm(a, rows, n, act, stream);
}

int gdn_decay_step(const gdn_decay_layer* layer, const gdn_decay_tokens* tokens, const int32_t* slot_idx, int32_t B,
                   int32_t T, cudaStream_t stream) {
  GDN_CALL_RANGE("gdn_decay_step");
  gdn::DecayView l;
  int rc;
  if ((rc = check_layer(layer, &l, true)) != GDN_OK) return rc;
  if (T < 1 || T > GDN_MAX_DECODE_TOKENS || B < 0) return GDN_ERR_INVALID_ARG;
  if (B > 65535) return GDN_ERR_TOO_LARGE;
  if ((rc = check_tokens(tokens, l, B)) != GDN_OK) return rc;
  if (B == 0) return GDN_OK;
  if (!slot_idx) return GDN_ERR_INVALID_ARG;
  if (!aligned(slot_idx, 4)) return GDN_ERR_MISALIGNED;
  if (!apart(*tokens, B)) return GDN_ERR_INVALID_ARG;
  return gdn::launch_decay_step(l, *tokens, slot_idx, B, T, stream);
}

size_t gdn_decay_prefill_workspace_bytes(const gdn_decay_layer* layer, int32_t num_seqs, int32_t total_tokens) {
  gdn::DecayView l;
  if (check_layer(layer, &l, false) != GDN_OK || num_seqs < 0 || total_tokens < 0) return 0;
  return gdn::decay_prefill_ws_bytes(l, num_seqs, total_tokens);
}

int gdn_decay_prefill(const gdn_decay_layer* layer, const gdn_decay_tokens* tokens, const int32_t* cu_seqlens,
                      const int32_t* slot_idx, const uint8_t* has_initial_state, int32_t num_seqs,
                      int32_t total_tokens, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  GDN_CALL_RANGE("gdn_decay_prefill");
  gdn::DecayView l;
  int rc;
  if ((rc = check_layer(layer, &l, true)) != GDN_OK) return rc;
  if (num_seqs < 0 || total_tokens < 0) return GDN_ERR_INVALID_ARG;
  if (num_seqs > 65535) return GDN_ERR_TOO_LARGE;
  if (num_seqs == 0) return total_tokens == 0 ? GDN_OK : GDN_ERR_INVALID_ARG;
  if ((rc = check_tokens(tokens, l, total_tokens)) != GDN_OK) return rc;
  if (!cu_seqlens || !slot_idx) return GDN_ERR_INVALID_ARG;
  if (!aligned(cu_seqlens, 4) || !aligned(slot_idx, 4)) return GDN_ERR_MISALIGNED;
  if (!workspace || workspace_bytes < gdn::decay_prefill_ws_bytes(l, num_seqs, total_tokens))
    return GDN_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned(workspace, 256)) return GDN_ERR_MISALIGNED;
  if (!apart(*tokens, total_tokens)) return GDN_ERR_INVALID_ARG;
  return gdn::launch_decay_prefill(l, *tokens, cu_seqlens, slot_idx, has_initial_state, num_seqs, total_tokens,
                                   workspace, stream);
}

}  // extern "C"
