// Expert routing kernel for sm_103a: scores of E experts per token, the K best
// and their weights (the formulas are in tw.h at tw_route_experts).
//
// One warp per token row, the row's E order values in registers: lane l owns
// experts l * V .. l * V + V - 1, so a group of consecutive experts is a run of
// lanes and the lowest index of a tie is the lowest lane's. K rounds of a warp
// maximum (redux.sync on order-preserving integer keys) give the experts in
// order.
//
// Order. Without a bias the scores are increasing in the logits, so experts
// are compared by their logits, which is exact. With a bias, or with group
// values that are sums, fp32 values can differ from the exact ones by more than
// two candidates differ from each other. Each value therefore carries an error
// bound; where a decision (the next of the K, the last of the K against the
// rest, the last group against the rest) is closer than its bounds and the two
// candidates' inputs are not the same, the warp does the row again in fp64.
// With random logits that is well under 1% of the rows.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cfloat>
#include <cstdint>

#include "row_ops.cuh"
#include "tw_internal.h"

namespace tw {
namespace {

constexpr int kRouteWarps = 4;
constexpr unsigned kAll = 0xffffffffu;

// Relative error of an fp32 score. Sigmoid: expf 2^-22, the sum 2^-24, the
// division 2^-24; together below 2^-21. Softmax: the exponent's argument x -
// max is rounded at |x - max| 2^-24, at most 2^-17.5 where exp is not 0; expf,
// the sum over E and the division add below 2^-18.
constexpr float kSigmoidErr = 0x1p-20f;
constexpr float kSoftmaxErr = 0x1p-16f;
constexpr float kRoundErr = 0x1p-22f;  // rounding of s + b and of c - b, in units of |c| + |b|

struct RouteParams {
  const void* logits;
  const float* bias;
  float* weights;
  int32_t* ids;
  long long tokens;
  int experts;
  int k;
  int n_groups, top_groups, group_top, group_size;
  int renormalize;
  float scale;
};

// A logit as fp32: NaN counts as -inf (left out), +inf as the largest finite
// value; -0 becomes +0 so that equal values have equal bits.
__device__ __forceinline__ float clean(float x) {
  if (!(x > -INFINITY)) return -INFINITY;
  return fminf(x, FLT_MAX) + 0.0f;
}

// Order-preserving integer of a float; 0 stands for "not a candidate" (-inf).
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x);
  const uint32_t k = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
  return x > -INFINITY ? k : 0u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}
template <typename F>
__device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

template <bool BF16>
__device__ __forceinline__ float load_logit(const RouteParams& p, long long row, int e) {
  const long long at = row * p.experts + e;
  if constexpr (BF16)
    return clean(__bfloat162float(static_cast<const __nv_bfloat16*>(p.logits)[at]));
  else
    return clean(static_cast<const float*>(p.logits)[at]);
}

__device__ __forceinline__ float load_bias(const RouteParams& p, int e) {
  return p.bias ? clean(__ldg(p.bias + e)) : 0.0f;
}

// The larger of two 64-bit keys over the warp.
__device__ __forceinline__ unsigned long long warp_max64(unsigned long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const unsigned long long u = __shfl_xor_sync(kAll, v, o);
    v = u > v ? u : v;
  }
  return v;
}
__device__ __forceinline__ unsigned long long order_key64(double x) {
  const unsigned long long b = static_cast<unsigned long long>(__double_as_longlong(x));
  const unsigned long long k = (b >> 63) ? ~b : (b | 0x8000000000000000ull);
  return x > -INFINITY ? k : 0ull;
}

// The row's selection in fp64. Returns in lane k the k-th expert (-1: none).
template <int V, bool SIGMOID, bool BF16>
__device__ __noinline__ int select_fp64(const RouteParams& p, long long row, int lane) {
  double c[V];
  double top = -INFINITY, sum = 0.0;
  if constexpr (!SIGMOID) {
    for (int i = 0; i < V; ++i) {
      const int e = lane * V + i;
      if (e < p.experts) top = fmax(top, static_cast<double>(load_logit<BF16>(p, row, e)));
    }
    for (int o = 16; o > 0; o >>= 1) top = fmax(top, __shfl_xor_sync(kAll, top, o));
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane * V + i;
    const double x = e < p.experts ? static_cast<double>(load_logit<BF16>(p, row, e)) : -INFINITY;
    double s = 0.0;
    if (x > -INFINITY) {
      if constexpr (SIGMOID) s = x > -700.0 ? 1.0 / (1.0 + exp(-x)) : exp(x);  // exp(700) is finite
      else s = exp(x - top);
    }
    sum += s;
    c[i] = x > -INFINITY ? s : -INFINITY;
  }
  if constexpr (!SIGMOID) sum = warp_sum(sum);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane * V + i;
    if (c[i] > -INFINITY) {
      if constexpr (!SIGMOID) c[i] /= sum;
      if (p.bias) c[i] += static_cast<double>(load_bias(p, e));
    }
  }
  if (p.top_groups < p.n_groups) {
    double mine = -INFINITY;  // lane g: group g's value
    for (int g = 0; g < p.n_groups; ++g) {
      double best = -INFINITY, second = -INFINITY;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = lane * V + i;
        if (e / p.group_size == g && c[i] > second) {
          if (c[i] > best) { second = best; best = c[i]; }
          else second = c[i];
        }
      }
      for (int o = 16; o > 0; o >>= 1) {
        const double b2 = __shfl_xor_sync(kAll, best, o), s2 = __shfl_xor_sync(kAll, second, o);
        second = fmax(fmin(best, b2), fmax(second, s2));
        best = fmax(best, b2);
      }
      double v = best;
      if (p.group_top == 2 && second > -INFINITY) v += second;
      if (lane == g) mine = v;
    }
    unsigned kept = 0;
    unsigned long long key = lane < p.n_groups ? order_key64(mine) : 0ull;
    for (int r = 0; r < p.top_groups; ++r) {
      const unsigned long long m = warp_max64(key);
      if (m == 0ull) break;
      const int g = __ffs(__ballot_sync(kAll, key == m)) - 1;
      kept |= 1u << g;
      if (lane == g) key = 0ull;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane * V + i;
      if (e < p.experts && !((kept >> (e / p.group_size)) & 1u)) c[i] = -INFINITY;
    }
  }
  int mine = -1;
  for (int r = 0; r < p.k; ++r) {
    unsigned long long best = 0ull;
    int at = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      // without a bias the logits order the experts
      const int e = lane * V + i;
      const double o = (p.bias || !(c[i] > -INFINITY))
                           ? c[i] : static_cast<double>(load_logit<BF16>(p, row, e));
      const unsigned long long key = order_key64(o);
      if (key > best) { best = key; at = e; }
    }
    const unsigned long long m = warp_max64(best);
    if (m == 0ull) break;
    const int e = __reduce_min_sync(kAll, best == m ? at : 0x7fffffff);
    if (lane == r) mine = e;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (lane * V + i == e) c[i] = -INFINITY;
  }
  return mine;
}

// Whether a (larger, with error bound ea) and b (eb) may be out of order; so
// may two that overflowed.
__device__ __forceinline__ bool too_close(float a, float ea, float b, float eb) {
  return !(a - b > ea + eb);
}

template <int V, bool SIGMOID, bool BF16>
__global__ void __launch_bounds__(kRouteWarps * 32)
    route_kernel(const __grid_constant__ RouteParams p) {
  __shared__ float s_value[kRouteWarps][32 * V];
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  const bool grouped = p.top_groups < p.n_groups;
  // fp32 values (not the logits) decide something
  const bool by_value = p.bias != nullptr || (grouped && p.group_top == 2);
  const float rel = SIGMOID ? kSigmoidErr : kSoftmaxErr;
  const long long stride = static_cast<long long>(gridDim.x) * kRouteWarps;
  for (long long row = static_cast<long long>(blockIdx.x) * kRouteWarps + warp; row < p.tokens;
       row += stride) {
    float x[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane * V + i;
      x[i] = e < p.experts ? load_logit<BF16>(p, row, e) : -INFINITY;
    }
    // softmax statistics, where scores or the unrenormalised weights need them
    float top = 0.0f, total = 1.0f;
    if (!SIGMOID && (by_value || !p.renormalize)) {
      top = x[0];
#pragma unroll
      for (int i = 1; i < V; ++i) top = fmaxf(top, x[i]);
      top = warp_max(top);
      total = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) total += x[i] > -INFINITY ? expf(x[i] - top) : 0.0f;
      total = warp_sum(total);
    }
    // values c; a masked expert keeps -inf
    float c[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      c[i] = x[i];
      if (by_value && x[i] > -INFINITY) {
        const float s = SIGMOID ? 1.0f / (1.0f + expf(-x[i])) : expf(x[i] - top) / total;
        c[i] = s + load_bias(p, lane * V + i);
      }
    }
    bool unsure = false;
    if (grouped) {
#pragma unroll
      for (int i = 0; i < V; ++i) s_value[warp][lane * V + i] = c[i];
      __syncwarp();
      float value = -INFINITY, err = 0.0f;
      if (lane < p.n_groups) {
        float best = -INFINITY, second = -INFINITY;
        int at = 0, at2 = 0;
        for (int i = 0; i < p.group_size; ++i) {
          const int e = lane * p.group_size + i;
          const float v = s_value[warp][e];
          if (v > best) { second = best; at2 = at; best = v; at = e; }
          else if (v > second) { second = v; at2 = e; }
        }
        value = best;
        if (by_value && best > -INFINITY) {
          const float b = load_bias(p, at);
          err = rel * fabsf(best - b) + kRoundErr * (fabsf(best) + fabsf(b));
        }
        if (p.group_top == 2 && second > -INFINITY) {
          const float b = load_bias(p, at2);
          value += second;
          err += rel * fabsf(second - b) + kRoundErr * (fabsf(second) + fabsf(b) + fabsf(value));
        }
      }
      __syncwarp();
      uint32_t key = lane < p.n_groups ? order_key(value) : 0u;
      unsigned kept = 0;
      int last = -1;
      for (int r = 0; r < p.top_groups; ++r) {
        const uint32_t m = __reduce_max_sync(kAll, key);
        if (m == 0u) break;
        last = __ffs(__ballot_sync(kAll, key == m)) - 1;
        kept |= 1u << last;
        if (lane == last) key = 0u;
      }
      if (by_value && last >= 0) {
        const float v = __shfl_sync(kAll, value, last), ev = __shfl_sync(kAll, err, last);
        // any group left against any kept one: the kept with the lowest value
        // decides, and kept groups' bounds are at most max(ev, err of theirs)
        const float worst = warp_max(((kept >> lane) & 1u) ? err : ev);
        unsure = key != 0u && too_close(v, worst, value, err);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = lane * V + i;
        if (e < p.experts && !((kept >> (e / p.group_size)) & 1u)) c[i] = -INFINITY;
        else if (p.bias == nullptr) c[i] = x[i];  // without a bias: ordered by the logits
      }
    }
    // K rounds: lane r keeps the r-th expert
    uint32_t key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = order_key(c[i]);
    int id = -1;
    float value = -INFINITY;
    for (int r = 0; r < p.k; ++r) {
      uint32_t best = key[0];
      int at = lane * V;
#pragma unroll
      for (int i = 1; i < V; ++i)
        if (key[i] > best) { best = key[i]; at = lane * V + i; }
      const uint32_t m = __reduce_max_sync(kAll, best);
      if (m == 0u) break;
      const int e = __reduce_min_sync(kAll, best == m ? at : 0x7fffffff);
      if (lane == r) { id = e; value = key_value(m); }
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (lane * V + i == e) key[i] = 0u;
    }
    if (p.bias != nullptr) {
      // each chosen expert against the one before it, and the last against
      // every expert that is left
      const float b = id >= 0 ? load_bias(p, id) : 0.0f;
      const float xv = id >= 0 ? load_logit<BF16>(p, row, id) : 0.0f;
      const float err =
          id >= 0 ? rel * fabsf(value - b) + kRoundErr * (fabsf(value) + fabsf(b)) : 0.0f;
      const float pv = __shfl_up_sync(kAll, value, 1), pe = __shfl_up_sync(kAll, err, 1);
      const float pb = __shfl_up_sync(kAll, b, 1), px = __shfl_up_sync(kAll, xv, 1);
      if (lane > 0 && id >= 0 && too_close(pv, pe, value, err) && !(px == xv && pb == b))
        unsure = true;
      const float lv = __shfl_sync(kAll, value, p.k - 1), le = __shfl_sync(kAll, err, p.k - 1);
      const float lb = __shfl_sync(kAll, b, p.k - 1), lx = __shfl_sync(kAll, xv, p.k - 1);
      if (lv > -INFINITY) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          if (key[i] == 0u) continue;
          const float v = key_value(key[i]);
          const int e = lane * V + i;
          const float be = load_bias(p, e);
          const float ee = rel * fabsf(v - be) + kRoundErr * (fabsf(v) + fabsf(be));
          if (too_close(lv, le, v, ee) && !(lb == be && lx == load_logit<BF16>(p, row, e)))
            unsure = true;
        }
      }
    }
    if (__any_sync(kAll, unsure)) id = select_fp64<V, SIGMOID, BF16>(p, row, lane);

    // weights of the chosen, lane k the k-th
    float w = 0.0f;
    const float xv = id >= 0 ? load_logit<BF16>(p, row, id) : -INFINITY;
    if (p.renormalize) {
      // Both scores are e^x times a factor; where every chosen logit is far
      // below 0 (sigmoid, e^-60 and less) the factor 1 / (1 + e^x) is 1 and e^x
      // is taken relative to the largest, so that nothing underflows.
      const float m = warp_max(xv);
      if (id >= 0) w = (SIGMOID && m > -60.0f) ? 1.0f / (1.0f + expf(-xv)) : expf(xv - m);
      const float sum = warp_sum(w);
      if (id >= 0) w = w / sum * p.scale;
    } else if (id >= 0) {
      w = (SIGMOID ? 1.0f / (1.0f + expf(-xv)) : expf(xv - top) / total) * p.scale;
    }
    if (lane < p.k) {
      p.weights[row * p.k + lane] = w;
      p.ids[row * p.k + lane] = id;
    }
  }
}

using RouteFn = void (*)(RouteParams);
#define TW_ROUTE(S, B) {route_kernel<1, S, B>, route_kernel<2, S, B>, route_kernel<4, S, B>, \
                        route_kernel<8, S, B>, route_kernel<16, S, B>, route_kernel<32, S, B>}
const RouteFn kRoute[2][2][6] = {{TW_ROUTE(false, false), TW_ROUTE(false, true)},
                                 {TW_ROUTE(true, false), TW_ROUTE(true, true)}};
#undef TW_ROUTE

}  // namespace

int launch_route(const RouteArgs& a, cudaStream_t stream) {
  RouteParams p;
  p.logits = a.logits;
  p.bias = a.bias;
  p.weights = a.weights;
  p.ids = a.ids;
  p.tokens = a.tokens;
  p.experts = a.experts;
  p.k = a.k;
  p.n_groups = a.n_groups;
  p.top_groups = a.top_groups;
  p.group_top = a.group_top;
  p.group_size = a.experts / a.n_groups;
  p.renormalize = a.renormalize;
  p.scale = a.scale;
  int v = 0;
  while ((32 << v) < a.experts) ++v;
  int64_t blocks = (a.tokens + kRouteWarps - 1) / kRouteWarps;
  if (blocks > (1 << 20)) blocks = 1 << 20;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(kRouteWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const RouteFn fn = kRoute[a.scoring == TW_SCORE_SIGMOID][a.logits_type == TW_LOGITS_BF16][v];
  if (cudaLaunchKernelEx(&cfg, fn, p) != cudaSuccess) {
    cudaGetLastError();
    return TW_ERR_CUDA;
  }
  return TW_OK;
}

}  // namespace tw
