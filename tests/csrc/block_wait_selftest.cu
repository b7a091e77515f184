// block_wait_selftest.cu -- the block norm's rows kernel on two SMs' CTAs, with one row's copy left out: the wait for it
// gives up after two seconds.
#include "gdn_tc.cuh"

namespace gdn {
__device__ unsigned long long left_out;
namespace tc {
__device__ __forceinline__ void some_bulk_g2s(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  if (reinterpret_cast<unsigned long long>(src) != left_out) bulk_g2s(dst, src, bytes, bar);
}
}  // namespace tc
}  // namespace gdn
#define bulk_g2s some_bulk_g2s
#include "gdn_block.cu"
#undef bulk_g2s

int gdn::sm_count() { return 2; }

// bf16 rows of n elements on 16-byte boundaries; `lost`: an x row's address (0: none).  The rows' share of a CTA in *ctas.
extern "C" int block_rows(const gdn_block_args* args, int rows, int n, unsigned long long lost, int* ctas) {
  if (cudaMemcpyToSymbol(gdn::left_out, &lost, sizeof lost) != cudaSuccess) return -1;
  const gdn::BlockArgs a{*args, 1.0f / (float)n, 1.0f / (float)args->group, rows, n};
  *ctas = 2;
  const int rc = gdn::launch_rows<__nv_bfloat16, gdn::kAligned, 2, false, 512>(a, 1, 2, nullptr);
  if (rc != GDN_OK) return rc;
  return cudaDeviceSynchronize() == cudaSuccess ? 0 : -2;
}
