// Internal interface between the C-ABI layer (abi.cpp) and the kernels
// (fused_kernel.cu). Not installed; not part of the public boundary.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "tw.h"

namespace tw {

// Arguments of one fused launch, already validated by the ABI layer.
struct FusedArgs {
  const void* partials[TW_MAX_PARTIALS];
  int n;
  void* residual;
  const void* gamma;
  void* out;
  float eps;
  int64_t rows;
  int64_t hidden;
  // e4m3 output only
  void* scales;
  int group;  // values per scale (H for a whole row)
  int scale_type;
};

struct LaunchShape {
  int grid;        // CTAs (one per SM)
  int threads;     // threads per CTA
  int smem_bytes;  // dynamic shared memory per CTA
  int stages;      // staging-ring depth
  int kmax;        // row chunks held in registers (template instance)
};

// Launch shape on the current device (queries and caches device attributes).
int plan_launch(int64_t rows, int64_t hidden, int n, int sm_budget, LaunchShape* shape);

// Enqueue the fused kernel on `stream`. smid_out: optional device int32[grid].
int launch_fused(const FusedArgs& a, cudaStream_t stream, int sm_budget, int* smid_out);
// The same with an e4m3 output and scales.
int launch_fused_q8(const FusedArgs& a, cudaStream_t stream, int sm_budget);

// Unfused baseline (unfused_kernels.cu): S = bf16(sum of partials), then the
// residual add + RMSNorm of the stored residual.
int launch_reduce(const void* const* partials, int n, int64_t rows, int64_t hidden, void* sum,
                  cudaStream_t stream);
int launch_add_rmsnorm(const void* sum, void* residual, const void* gamma, float eps, int64_t rows,
                       int64_t hidden, void* out, cudaStream_t stream);

// Arguments of one combine launch, already validated. scale_type < 0: bf16
// output; otherwise e4m3 with scales. k == 0 (with n >= 1): the dense step, its
// vectors given to threads as in the fused step's kernels, so that the rows are
// bitwise theirs.
struct CombineArgs {
  const void* experts;
  int64_t m;
  const int32_t* rows;
  const float* weights;
  int k;
  const void* partials[TW_MAX_PARTIALS];
  int n;
  void* residual;
  const void* gamma;
  void* out;
  void* scales;
  int group;  // values per scale (H for a whole row)
  int scale_type;
  float eps;
  int64_t tokens;
  int64_t hidden;
};
int launch_combine(const CombineArgs& a, cudaStream_t stream, int sm_budget);
// Read (and optionally clear) the device-side error words of the 8-bit step's
// and the combine kernels, after the device was synchronised.
int read_fused_q8_error(int reset, unsigned* code);
int read_combine_error(int reset, unsigned* code);

// Arguments of one routing launch, already validated.
struct RouteArgs {
  const void* logits;
  int logits_type;
  const float* bias;
  int64_t tokens;
  int experts;
  int k;
  int scoring;
  int n_groups, top_groups, group_top;
  int renormalize;
  float scale;
  float* weights;
  int32_t* ids;
};
int launch_route(const RouteArgs& a, cudaStream_t stream);

// Diagnostic kernel: a bounded wait on an mbarrier nothing completes.
int launch_wait_probe(long long limit_ns, cudaStream_t stream);

// Read (and optionally clear) the device-side error word of the current device.
int read_device_error(int reset, int* code);

}  // namespace tw
