// The fused step with its bf16 output: the instances of fused_forms.cuh, the
// launch-shape query, the device error word and the bounded-wait diagnostic.
#define TW_FUSED_Q8 0
#include "fused_forms.cuh"

namespace tw {
namespace {

// Diagnostic: one CTA waits, with the kernels' bounded wait, on an mbarrier
// phase that nothing completes (one pending arrival that never comes). The
// wait gives up after limit_ns and reports through the device error word.
__global__ void wait_timeout_probe(unsigned long long limit_ns) {
  __shared__ __align__(8) uint64_t bar;
  __shared__ int abort_flag;
  if (threadIdx.x == 0) {
    mbar_init(&bar, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  if (threadIdx.x == 0) wait_phase(&bar, 0u, &abort_flag, 1u, limit_ns);
}

}  // namespace

int plan_launch(int64_t rows, int64_t hidden, int n, int sm_budget, LaunchShape* shape) {
  DeviceInfo* d = nullptr;
  int st = device_info(&d);
  if (st != TW_OK) return st;
  Choice c;
  return shape_for(*d, rows, hidden, n, sm_budget, &c, shape);
}

int launch_fused(const FusedArgs& a, cudaStream_t stream, int sm_budget, int* smid_out) {
  return launch_forms(a, stream, sm_budget, smid_out);
}

int launch_wait_probe(long long limit_ns, cudaStream_t stream) {
  wait_timeout_probe<<<1, 32, 0, stream>>>(static_cast<unsigned long long>(limit_ns));
  return cudaGetLastError() == cudaSuccess ? TW_OK : TW_ERR_CUDA;
}

int read_device_error(int reset, int* code) {
  if (cudaDeviceSynchronize() != cudaSuccess) return TW_ERR_CUDA;
  unsigned fused = 0, q8 = 0, combine = 0;
  int st = read_ring_error(reset, &fused);
  if (st == TW_OK) st = read_fused_q8_error(reset, &q8);
  if (st == TW_OK) st = read_combine_error(reset, &combine);
  if (st != TW_OK) return st;
  if (code) *code = static_cast<int>(fused | q8 | combine);
  return TW_OK;
}

}  // namespace tw
