// A ring of two rows whose second one is never asked for, so that the wait for it runs out.
#include <cuda_runtime.h>

#include "row_ring.cuh"

namespace {

constexpr int kRow = 1024;  // floats
constexpr uint64_t kLimit = 20000000;  // 20 ms

// Warp 0 waits for both rows and has to leave; warp 1 goes through the barriers to the end.
// out: the first row's sum by warp 1, then a word for each thread that came to the end.
__global__ void ring_wait_probe(const float *row, float *out, int *status) {
  using namespace nabla;
  __shared__ alignas(128) float rows[2][kRow];
  __shared__ RowRing ring;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) tc::mbar_init(&ring.full[i], 1);
    ring.abort = 0;
    ring.stages = 2;
    tc::fence_barrier_init();
    tc::mbar_expect_tx(&ring.full[0], sizeof(rows[0]));
    tc::bulk_load(rows[0], row, sizeof(rows[0]), &ring.full[0]);
  }
  __syncthreads();
  if (!tc::mbar_try_wait(&ring.full[0], 0)) wait_for_row<kLimit>(&ring.full[0], 0, &ring, status);
  float sum = 0.f;
  for (int i = threadIdx.x & 31; i < kRow; i += 32) sum += rows[0][i];
  __syncthreads();
  if (threadIdx.x == 0) {  // the stage's next row is in flight when the wait below gives up
    tc::mbar_expect_tx(&ring.full[0], sizeof(rows[0]));
    tc::bulk_load(rows[0], row, sizeof(rows[0]), &ring.full[0]);
  }
  if (threadIdx.x < 32 && !tc::mbar_try_wait(&ring.full[1], 0))
    wait_for_row<kLimit>(&ring.full[1], 0, &ring, status);
  __syncthreads();
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (threadIdx.x == 32) out[0] = sum;
  out[1 + threadIdx.x] = 1.f;
}

}  // namespace

extern "C" int ring_wait(const float *row, float *out, int *status, cudaStream_t st) {
  ring_wait_probe<<<1, 64, 0, st>>>(row, out, status);
  return (int)cudaGetLastError();
}
