// The tree attention's host guard (a GPU, but no kernel is launched): a kernel with
// static shared memory, whose dynamic shared memory starts later, is refused, and one
// without is not.  Built and run by tests/test_gpu_tree_guard.py.
#include "tq_tree_impl.cuh"

#include <cstdio>

__global__ void shifted(int* out) {
  __shared__ int x[64];
  x[threadIdx.x & 63] = (int)threadIdx.x;
  __syncthreads();
  out[threadIdx.x] = x[63 - (threadIdx.x & 63)];
}
__global__ void plain(int* out) {
  extern __shared__ int y[];
  y[threadIdx.x] = (int)threadIdx.x;
  __syncthreads();
  out[threadIdx.x] = y[0];
}

int main() {
  std::atomic<uint64_t> a{0}, b{0};
  const cudaError_t no = tq::check_smem_base(shifted, a), yes = tq::check_smem_base(plain, b);
  const bool ok = no == cudaErrorNotSupported && yes == cudaSuccess && a == 0 && b == 1 &&
                  tq::check_smem_base(plain, b) == cudaSuccess && tq::check_smem_base(shifted, a) == no;
  std::printf("%s (%s, %s)\n", ok ? "guard ok" : "guard BAD", cudaGetErrorString(no), cudaGetErrorString(yes));
  return !ok;
}
