// attn_wait_selftest.cu -- the attention kernels' bounded waits on a small ring: a producing warp
// copies tiles into two stages, four consuming warps hand them back, and one of them waits for an
// arrival that never comes.  Every wait gives up after two seconds.
#include "gdn_attn.cuh"
#include "gdn_tmap.h"

using namespace gdn;
using namespace gdn::tc;
using namespace gdn::attn;

constexpr int kStages = 2, kFloats = 256, kWarps = 4;

// out: tiles issued, consuming warps that left by the vote, tiles whose sum was right in every warp
__global__ void __launch_bounds__((kWarps + 1) * 32) ring_kernel(const float* src, int tiles, int stuck_at, int32_t* status,
                                                               int* out) {
  __shared__ __align__(128) float ring[kStages][kFloats];
  __shared__ uint64_t full[kStages], empty[kStages], never;
  __shared__ int dead;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kWarps);
    }
    mbar_init(&never, 1);
    dead = 0;
    mbar_fence_init();
  }
  __syncthreads();
  bool alive = true;
  int stage = 0;
  uint32_t phase = 0;
  auto step = [&]() {
    if (++stage == kStages) { stage = 0; phase ^= 1u; }
  };
  if (warp == kWarps) {
    for (int i = 0; i < tiles; ++i) {
      alive = wait_bar(&empty[stage], phase ^ 1u, &dead, status);
      if (!alive) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&full[stage], kFloats * 4);
        bulk_g2s(ring[stage], src + i * kFloats, kFloats * 4, &full[stage]);
        atomicAdd(out, 1);
      }
      __syncwarp();
      step();
    }
    drain_ring<kStages>(full, stage, phase);
    return;
  }
  for (int i = 0; i < tiles; ++i) {
    alive = alive && wait_one(&full[stage], phase, &dead, status);
    if (warp == 1 && i == stuck_at) alive = alive && wait_one(&never, 0, &dead, status);
    __syncwarp();
    float sum = 0.f;
    for (int k = lane; k < kFloats; k += 32) sum += ring[stage][k];
    sum = warp_sum(sum);
    if (alive && lane == 0) {
      if (sum == (float)(kFloats * i)) atomicAdd(out + 2, 1);
      mbar_arrive(&empty[stage]);
    }
    step();
  }
  if (bar_any(1, kWarps * 32, !alive) && lane == 0) atomicAdd(out + 1, 1);
}

extern "C" int attn_ring(const float* src, int tiles, int stuck_at, int32_t* status, int* out) {
  ring_kernel<<<1, (kWarps + 1) * 32>>>(src, tiles, stuck_at, status, out);
  if (cudaGetLastError() != cudaSuccess) return -1;
  return cudaDeviceSynchronize() == cudaSuccess ? 0 : -2;
}
