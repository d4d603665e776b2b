// Combine + residual + RMSNorm kernel for sm_103a: the step after the experts
// of a mixture-of-experts layer, in one pass.
//
//   z = sum_k w[t,k] X[rows[t,k]] + P_0[t] + ... + P_{N-1}[t] + R[t]   fp32
//   R[t] = bf16(z);  y = (z * rsqrt(mean z^2 + eps)) * gamma
//   out  = bf16(y), or e4m3 codes with scales (row_ops.cuh)
//
// Bound: HBM. Every source row is read once and z stays in registers between
// the sum and the norm, so the bytes are (K + N + 1) rows read and two rows
// (one and a half with 8-bit output) written per token.
//
// One CTA per token row at a time. Thread t owns the 16-byte vectors t, t +
// 256, ... of the row, as in the fused step, so the order of every sum depends
// on H alone.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "row_ops.cuh"
#include "tw_internal.h"

namespace tw {

// Bit 3: a row index outside the expert rows.
__device__ unsigned int g_combine_error = 0;

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

struct CombineParams {
  const uint4* experts;
  const int32_t* rows;
  const float* weights;
  const uint4* partials[TW_MAX_PARTIALS];
  uint4* residual;
  const uint4* gamma;
  void* out;
  void* scales;
  long long m;
  long long tokens;
  int vec_per_row;
  int k;
  int n;
  int group;  // values per scale; 8 * vec_per_row for a whole row
  int scale_type;
  float eps;
  float hidden;
};

template <int KMAX, bool Q8>
__global__ void __launch_bounds__(kThreads) combine_kernel(const __grid_constant__ CombineParams p) {
  __shared__ int s_row[2][TW_MAX_TOPK];
  __shared__ float s_weight[2][TW_MAX_TOPK];
  __shared__ __align__(16) float s_sum[2][kWarps];
  __shared__ __align__(16) float s_max[2][kWarps];
  grid_dependency_wait();
  grid_launch_dependents();
  const int t = threadIdx.x;
  const int lane = t & 31;
  const int warp = t >> 5;
  const int vpr = p.vec_per_row;
  const bool row_scale = p.group == 8 * vpr;
  int buf = 0;
  for (long long row = blockIdx.x; row < p.tokens; row += gridDim.x, buf ^= 1) {
    // The two buffers alternate: a thread writes buffer b for row i + 2 only
    // after the barriers of row i + 1, which every thread reaches after it has
    // read b for row i.
    if (t < p.k) {
      int r = p.rows[row * p.k + t];
      if (r < -1 || r >= p.m) {
        atomicOr(&g_combine_error, 8u);
        r = -1;
      }
      s_row[buf][t] = r;
      s_weight[buf][t] = r >= 0 ? p.weights[row * p.k + t] : 0.0f;
    }
    __syncthreads();
    float z[KMAX][8];
    float ss = 0.0f, am = 0.0f;
    uint4* res_row = p.residual + row * vpr;
#pragma unroll
    for (int j = 0; j < KMAX; ++j) {
      const int v = j * kThreads + t;
#pragma unroll
      for (int i = 0; i < 8; ++i) z[j][i] = 0.0f;
      if (v < vpr) {
        for (int k = 0; k < p.k; ++k) {
          const int r = s_row[buf][k];
          if (r < 0) continue;
          float x[8];
          load8(__ldg(p.experts + static_cast<long long>(r) * vpr + v), x);
          const float w = s_weight[buf][k];
#pragma unroll
          for (int i = 0; i < 8; ++i) z[j][i] = fmaf(w, x[i], z[j][i]);
        }
        for (int n = 0; n < p.n; ++n) add8(p.partials[n][row * vpr + v], z[j]);
        add8(res_row[v], z[j]);
        res_row[v] = pack8(z[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(z[j][i], z[j][i], ss);
        if (Q8 && row_scale) {
          float g[8];
          load8(__ldg(p.gamma + v), g);
#pragma unroll
          for (int i = 0; i < 8; ++i) am = fmaxf(am, fabsf(z[j][i] * g[i]));
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (Q8) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
    }
    if (lane == 0) {
      s_sum[buf][warp] = ss;
      if (Q8) s_max[buf][warp] = am;
    }
    __syncthreads();
    const float rs = rsqrtf(warp_total(s_sum[buf]) / p.hidden + p.eps);
    GroupScale gs = {};
    if (Q8 && row_scale) {
#pragma unroll
      for (int w = 0; w < kWarps; ++w) am = fmaxf(am, s_max[buf][w]);
      gs = group_scale(am * rs, p.scale_type);
      if (t == 0) store_scale(p.scales, row, gs, p.scale_type);
    }
#pragma unroll
    for (int j = 0; j < KMAX; ++j) {
      const int v = j * kThreads + t;
      if constexpr (Q8) {
        float y[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
        if (v < vpr) scale8(z[j], rs, __ldg(p.gamma + v), y);
        if (!row_scale) {
          float a = amax8(y);
          for (int o = p.group >> 4; o > 0; o >>= 1)
            a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
          gs = group_scale(a, p.scale_type);
          const int per = p.group >> 3;  // vectors per group
          if (v < vpr && (v & (per - 1)) == 0)
            store_scale(p.scales, row * (vpr / per) + v / per, gs, p.scale_type);
        }
        if (v < vpr) static_cast<uint2*>(p.out)[row * vpr + v] = pack_e4m3(y, gs.inv);
      } else if (v < vpr) {
        float y[8];
        scale8(z[j], rs, __ldg(p.gamma + v), y);
        static_cast<uint4*>(p.out)[row * vpr + v] = pack8(y);
      }
    }
  }
}

using CombineFn = void (*)(CombineParams);
#define TW_COMBINE(Q) {combine_kernel<1, Q>, combine_kernel<2, Q>, combine_kernel<4, Q>, \
                       combine_kernel<8, Q>, combine_kernel<16, Q>}
const CombineFn kCombine[2][5] = {TW_COMBINE(false), TW_COMBINE(true)};
#undef TW_COMBINE

}  // namespace

int launch_combine(const CombineArgs& a, cudaStream_t stream, int sm_budget) {
  CombineParams p;
  p.experts = static_cast<const uint4*>(a.experts);
  p.rows = a.rows;
  p.weights = a.weights;
  for (int r = 0; r < TW_MAX_PARTIALS; ++r)
    p.partials[r] = r < a.n ? static_cast<const uint4*>(a.partials[r]) : nullptr;
  p.residual = static_cast<uint4*>(a.residual);
  p.gamma = static_cast<const uint4*>(a.gamma);
  p.out = a.out;
  p.scales = a.scales;
  p.m = a.m;
  p.tokens = a.tokens;
  p.vec_per_row = static_cast<int>(a.hidden / 8);
  p.k = a.k;
  p.n = a.n;
  p.group = a.group;
  p.scale_type = a.scale_type;
  p.eps = a.eps;
  p.hidden = static_cast<float>(a.hidden);
  int kc = 0;
  while ((1 << kc) * kThreads < p.vec_per_row) ++kc;
  int64_t grid = sm_budget > 0 ? sm_budget : (1 << 16);
  if (grid > a.tokens) grid = a.tokens;
  const CombineFn fn = kCombine[a.scale_type >= 0 ? 1 : 0][kc];
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, fn, p) != cudaSuccess) {
    cudaGetLastError();
    return TW_ERR_CUDA;
  }
  return TW_OK;
}

int read_combine_error(int reset, unsigned* code) {
  if (cudaMemcpyFromSymbol(code, g_combine_error, sizeof(*code)) != cudaSuccess) return TW_ERR_CUDA;
  if (reset && *code) {
    const unsigned zero = 0;
    if (cudaMemcpyToSymbol(g_combine_error, &zero, sizeof(zero)) != cudaSuccess) return TW_ERR_CUDA;
  }
  return TW_OK;
}

}  // namespace tw
