// Expert routing kernels for sm_103a: scores of E experts per token, the K best
// and their weights (the formulas are in tw.h at tw_route_experts).
//
// Bound: instruction issue. A row of 256 fp32 logits is 1 KiB, 0.15 ns of HBM
// time, but selecting 8 of 256 in order costs hundreds of instructions per
// warp, half of them minima, maxima and compares, which issue at half rate.
// The design therefore counts instructions:
//
//   Keys. Every candidate becomes one 32-bit integer, 22 bits of its value and
//   10 bits of 1023 - index: one integer maximum finds the best and its index
//   and sends ties to the lowest index. The 22 bits are a fixed-point value
//   taken with one fused multiply-add onto 2^23 (quantise()), relative to the
//   row's largest value; bf16 logits are their own 16 bits.
//
//   Selection. A lane sorts its 8 keys (19 compare-exchanges); then K rounds of
//   a maximum over the lanes' first keys, the winner's list moving up by one.
//   Rows of up to 64 experts take 1 to 8 lanes, so that 4 to 32 rows share a
//   warp; longer rows take the warp (redux.sync).
//
// Order. The result's order is that of exact arithmetic. Without a bias the
// scores are increasing in the logits, so logits are compared, and quantise()
// is monotone: only equal keys of different logits are open. With a bias, or
// with group values that are sums, fp32 values carry an error bound. Where a
// decision is closer than its bound, and the two experts' inputs are not the
// same, it is made again exactly: the few candidates in fp64 (settle,
// settle_groups), or the whole row where they are too many to list
// (select_exact). With random logits that is about 0.2% of the rows of 256
// experts with a bias.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cstdint>

#include "row_ops.cuh"
#include "tw_internal.h"

namespace tw {
namespace {

constexpr int kRouteWarps = 4;
constexpr int kRouteBlocks = 152 * 12;  // about what is resident at once; larger batches loop
// From this many tokens on, rows of 65 to 256 experts share a warp four by
// four, which halves the instructions per row but has four rows wait for one
// that is settled in fp64. Measured against one row per warp (256 experts, K =
// 8): bf16, no bias 3.0 against 3.1 us at 2048 tokens, 3.5 / 4.1 at 4096, 7.5 /
// 11.1 at 16384; sigmoid with bias and groups 11.2 / 7.8 at 4096, 14.3 / 11.7 at
// 8192, 17.9 / 19.6 at 16384, 27.1 / 33.6 at 32768.
constexpr int64_t kLongTokens = 4096;
constexpr int64_t kLongTokensByValue = 12288;
// Resident blocks per SM that several rows per warp leave registers for: the
// 32 fp32 values of a lane (168 registers, three blocks, without a bound: 256
// experts, sigmoid + bias + groups 18.8 against 17.9 us at 16384 tokens, 29.6 /
// 27.1 at 32768), and 8 values (108 registers; 64 experts, bf16 8.1 against 7.3
// us at 32768). The other lengths are left to the compiler (0): a bound made
// them slower.
constexpr int kBlocks32 = 5, kBlocks8 = 8;
constexpr unsigned kAll = 0xffffffffu;
constexpr uint32_t kNone = 1024u;          // fixed-point keys below: no candidate
constexpr uint32_t kNone16 = 0x00800000u;  // the same for keys of bf16 logits

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

// ------------------------------------------------------------------ inputs

// A logit or bias: NaN counts as -inf (left out), +inf as the largest finite
// value (which no bf16 logit is).
__device__ __forceinline__ float clean(float x) { return fminf(fmaxf(x, -INFINITY), FLT_MAX); }

template <bool BF16>
__device__ __forceinline__ float load_logit(const RouteParams& p, long long row, int e) {
  const long long at = row * p.experts + e;
  if constexpr (BF16)
    return clean(__bfloat162float(static_cast<const __nv_bfloat16*>(p.logits)[at]));
  else
    return clean(__ldg(static_cast<const float*>(p.logits) + at));
}

__device__ __forceinline__ float load_bias(const RouteParams& p, int e) {
  return p.bias ? clean(__ldg(p.bias + e)) : 0.0f;
}

// The V logits from expert e0 on; experts beyond E are -inf. VEC: E is a
// multiple of V and rows start on 16 bytes, so a lane's run is whole 16-byte
// vectors or nothing.
template <int V, bool BF16, bool VEC>
__device__ __forceinline__ void load_row(const RouteParams& p, long long row, int e0, bool there,
                                         float (&x)[V]) {
  constexpr int kPer = BF16 ? 8 : 4;  // values in 16 bytes
  if constexpr (VEC && V % kPer == 0) {
    uint4 q[V / kPer];
    const uint32_t out = BF16 ? 0xff80ff80u : 0xff800000u;  // -inf
#pragma unroll
    for (int v = 0; v < V / kPer; ++v) q[v] = make_uint4(out, out, out, out);
    if (there && e0 < p.experts) {
      const char* at = static_cast<const char*>(p.logits) +
                       (row * p.experts + e0) * static_cast<long long>(BF16 ? 2 : 4);
#pragma unroll
      for (int v = 0; v < V / kPer; ++v) q[v] = __ldg(reinterpret_cast<const uint4*>(at) + v);
    }
#pragma unroll
    for (int v = 0; v < V / kPer; ++v) {
      if constexpr (BF16) {
        load8(q[v], &x[8 * v]);
      } else {
        x[4 * v] = __uint_as_float(q[v].x);
        x[4 * v + 1] = __uint_as_float(q[v].y);
        x[4 * v + 2] = __uint_as_float(q[v].z);
        x[4 * v + 3] = __uint_as_float(q[v].w);
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = clean(x[i]);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      x[i] = there && e0 + i < p.experts ? load_logit<BF16>(p, row, e0 + i) : -INFINITY;
  }
}

// The same for the 4 rows of a warp with 8 lanes each, through shared memory:
// the rows are one run of bytes, read 512 at a time by the whole warp; a lane
// then takes its C 16-byte pieces in an order that depends on the lane (order()),
// so that 8 lanes read from all banks. Straight from global memory every lane
// would touch a line of its own in every load, 8 times the L1 wavefronts. The
// order of a lane's values does not matter: keys carry the index.
template <int V, bool BF16>
struct Staged {
  static constexpr int kPer = BF16 ? 8 : 4;  // values per piece
  static constexpr int C = V / kPer;         // pieces per lane
  static __device__ __forceinline__ int order(int sub, int i) { return i ^ ((sub * C / 8) & (C - 1)); }
  // the expert of a lane's i-th value
  static __device__ __forceinline__ int expert(int sub, int i) {
    return sub * V + order(sub, i / kPer) * kPer + i % kPer;
  }
  static __device__ __forceinline__ void load(const RouteParams& p, long long first, int rows,
                                              int lane, bool there, uint4* stage, float (&x)[V]) {
    const int row_pieces = p.experts / kPer;
    const uint4* from = reinterpret_cast<const uint4*>(
        static_cast<const char*>(p.logits) + first * row_pieces * 16);
    const int all = rows * row_pieces;
    uint4 q[C];
#pragma unroll
    for (int i = 0; i < C; ++i) q[i] = i * 32 + lane < all ? __ldg(from + i * 32 + lane) : uint4{};
    __syncwarp();  // the last rows have been read
#pragma unroll
    for (int i = 0; i < C; ++i) stage[i * 32 + lane] = q[i];
    __syncwarp();
    const int sub = lane & 7;
    there = there && sub * V < p.experts;
    const uint32_t out = BF16 ? 0xff80ff80u : 0xff800000u;  // -inf
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const uint4 v = there ? stage[(lane >> 3) * row_pieces + sub * C + order(sub, i)]
                            : make_uint4(out, out, out, out);
      if constexpr (BF16) {
        load8(v, &x[8 * i]);
      } else {
        x[4 * i] = __uint_as_float(v.x);
        x[4 * i + 1] = __uint_as_float(v.y);
        x[4 * i + 2] = __uint_as_float(v.z);
        x[4 * i + 3] = __uint_as_float(v.w);
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = clean(x[i]);
  }
};

// ------------------------------------------------------------------ across lanes
//
// L: lanes of a row, a power of two; its rows lie side by side in the warp.

template <int L>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  if constexpr (L == 32) {
    return __reduce_max_sync(kAll, v);
  } else {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(kAll, v, o));
    return v;
  }
}
template <int L>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}
template <int L, typename F>
__device__ __forceinline__ F lanes_sum(F v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// ------------------------------------------------------------------ values

// Fast e^x and 1 / x (2 ulp and 1 ulp; subnormals count as 0).
__device__ __forceinline__ float fast_exp(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.44269504f));
  return r;
}
__device__ __forceinline__ float fast_rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Absolute errors of the scores that the choice uses, in units of the row's
// largest possible score (1, or 1 / total for softmax), and of an addition:
//   sigmoid  1 / (1 + e^-x): the exponential's relative error d = |x| 2^-23 +
//            2^-22 moves s by s (1 - s) d, at most 2^-23; the sum, the reciprocal
//            and the subnormals that count as 0 add less than 2^-22.
//   softmax  e^(x - top) / total: the exponential's error falls with its value,
//            at most 2^-22 of the largest; the total has at most 37 roundings.
constexpr float kSigmoidErr = 0x1p-21f;
constexpr float kSoftmaxErr = 0x1p-18f;
constexpr float kAddErr = 0x1p-22f;  // rounding of s + b, in units of |s| + |b|

// Order-preserving integer of a float, 0 for -inf, and back.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);  // -0 and +0 are equal
  const uint32_t k = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
  return x > -INFINITY ? k : 0u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}
__device__ __forceinline__ unsigned long long order_key64(double x) {
  const unsigned long long b = static_cast<unsigned long long>(__double_as_longlong(x + 0.0));
  const unsigned long long k = (b >> 63) ? ~b : (b | 0x8000000000000000ull);
  return x > -INFINITY ? k : 0ull;
}
__device__ __forceinline__ double key_value64(unsigned long long k) {
  return __longlong_as_double(static_cast<long long>((k >> 63) ? (k & 0x7fffffffffffffffull) : ~k));
}

// ------------------------------------------------------------------ keys

// Fixed point of the values of one row: fma(c, inv, add) is an integer on top
// of 2^23, so its low 22 bits are the value in steps of 1 / inv, the row's
// largest value near 2^22 - 32. Values more than about R below the largest
// give 0, as -inf does. The fma rounds once, so the mapping is monotone. R
// grows with |hi| so that add keeps steps of at most 8 and nothing reaches
// 2^22.
struct Fixed {
  float inv, add;
};
__device__ __forceinline__ Fixed fixed_for(float hi, float reach) {
  const float r = fmaxf(reach, fabsf(hi) * 0.0625f);
  Fixed f;
  f.inv = __fdividef(4194304.0f, r);  // r <= 2^124, within the fast division's range
  f.add = fmaf(-hi, f.inv, 8388608.0f + 4194304.0f - 32.0f);
  return f;
}
__device__ __forceinline__ uint32_t fixed_key(float c, const Fixed& f, uint32_t tail) {
  const float t = fmaxf(fmaf(c, f.inv, f.add), 8388608.0f);  // a NaN gives 2^23
  return (__float_as_uint(t) << 10) + tail;
}

// bf16 logits: their 16 bits in order, exactly, above the index. Keys below
// kNone16 are -inf.
__device__ __forceinline__ uint32_t bf16_key(float x, uint32_t tail) {
  // what stands for +inf rounds up to 0x7f80, above every bf16
  const uint32_t b = __float_as_uint(x + 0.0f) + 0x8000u;
  const uint32_t o = b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
  return (o & 0xffff0000u) | tail;
}

__device__ __forceinline__ void exchange(uint32_t& a, uint32_t& b) {
  const uint32_t hi = max(a, b);
  b = min(a, b);
  a = hi;
}

template <int D>
__device__ __forceinline__ void sort_descending(uint32_t (&k)[D]) {
  static_assert(D == 1 || D == 2 || D == 4 || D == 8, "one to eight keys");
  if constexpr (D == 2) {
    exchange(k[0], k[1]);
  } else if constexpr (D == 4) {
    exchange(k[0], k[2]); exchange(k[1], k[3]);
    exchange(k[0], k[1]); exchange(k[2], k[3]);
    exchange(k[1], k[2]);
  } else if constexpr (D == 8) {
    exchange(k[0], k[2]); exchange(k[1], k[3]); exchange(k[4], k[6]); exchange(k[5], k[7]);
    exchange(k[0], k[4]); exchange(k[1], k[5]); exchange(k[2], k[6]); exchange(k[3], k[7]);
    exchange(k[0], k[1]); exchange(k[2], k[3]); exchange(k[4], k[5]); exchange(k[6], k[7]);
    exchange(k[2], k[4]); exchange(k[3], k[5]);
    exchange(k[1], k[4]); exchange(k[3], k[6]);
    exchange(k[1], k[2]); exchange(k[3], k[4]); exchange(k[5], k[6]);
  }
}

// The 8 largest of two descending lists of 8, descending, in a: the larger of
// a[i] and b[7 - i] are those 8 and fall, then rise; three levels sort them.
__device__ __forceinline__ void merge8(uint32_t (&a)[8], const uint32_t (&b)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] = max(a[i], b[7 - i]);
#pragma unroll
  for (int d = 4; d > 0; d >>= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if ((i & d) == 0) exchange(a[i], a[i + d]);
}

// A lane's keys in descending order: all V of them, or the 8 largest.
template <int V, int D, bool EXACT16>
__device__ __forceinline__ void lane_keys(const float (&c)[V], const Fixed& f, int e0,
                                          uint32_t (&k)[D]) {
  const uint32_t tail = 1023u - static_cast<uint32_t>(e0);
#pragma unroll
  for (int v = 0; v < V; v += D) {
    uint32_t part[D];
#pragma unroll
    for (int i = 0; i < D; ++i)
      part[i] = EXACT16 ? bf16_key(c[v + i], tail - (v + i)) : fixed_key(c[v + i], f, tail - (v + i));
    sort_descending<D>(part);
    if (v == 0) {
#pragma unroll
      for (int i = 0; i < D; ++i) k[i] = part[i];
    } else if constexpr (D == 8) {
      merge8(k, part);
    }
  }
}

template <int D>
__device__ __forceinline__ void pop(uint32_t (&k)[D], bool mine) {
#pragma unroll
  for (int i = 0; i + 1 < D; ++i) k[i] = mine ? k[i + 1] : k[i];
  k[D - 1] = mine ? 0u : k[D - 1];
}

__device__ __forceinline__ int key_expert(uint32_t k) { return 1023 - static_cast<int>(k & 1023u); }

// Whether two near experts are in the order of their keys: their inputs are the
// same, so that their values are. Without a bias the loaded logits tell; fp32
// logits with a bias are hardly ever the same and go to settle unseen.
template <bool BF16>
__device__ __forceinline__ bool same_inputs(const RouteParams& p, long long row, int a, int b) {
  if (!BF16 && p.bias) return false;
  return load_logit<BF16>(p, row, a) == load_logit<BF16>(p, row, b) &&
         (!p.bias || load_bias(p, a) == load_bias(p, b));
}

// Without a bias: whether one of a lane's logits has the last chosen one's key
// but is not the same.
template <int V, bool BF16>
__device__ __forceinline__ bool near_last(const RouteParams& p, long long row, uint32_t last,
                                          const float (&c)[V], const Fixed& f) {
  const float x = load_logit<BF16>(p, row, key_expert(last));
  bool near = false;
#pragma unroll
  for (int i = 0; i < V; ++i)
    near = near || ((fixed_key(c[i], f, 0u) >> 10) == (last >> 10) && c[i] != x);
  return near;
}

// ------------------------------------------------------------------ exact rows

template <bool SIGMOID>
__device__ __forceinline__ double score64(double x, double top) {
  if constexpr (!SIGMOID) return exp(x - top);
  return x > -700.0 ? 1.0 / (1.0 + exp(-x)) : exp(x);  // exp(700) is finite
}

__device__ __forceinline__ unsigned long long lanes_max64(unsigned long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const unsigned long long u = __shfl_xor_sync(kAll, v, o);
    v = u > v ? u : v;
  }
  return v;
}

// The row's selection in fp64 (logits are compared as they are), by the whole
// warp, V experts per lane. Returns in lane k the k-th expert (-1: none).
template <int V, bool SIGMOID, bool BF16>
__device__ __noinline__ int select_exact(const RouteParams& p, long long row, int lane) {
  const bool grouped = p.top_groups < p.n_groups;
  const bool by_value = p.bias != nullptr || (grouped && p.group_top == 2);
  unsigned long long c[V];  // order keys of the values
  if (by_value) {
    double top = 0.0, total = 1.0;
    if constexpr (!SIGMOID) {
      top = -INFINITY;
      for (int i = 0; i < V; ++i) {
        const int e = lane * V + i;
        if (e < p.experts) top = fmax(top, static_cast<double>(load_logit<BF16>(p, row, e)));
      }
      for (int o = 16; o > 0; o >>= 1) top = fmax(top, __shfl_xor_sync(kAll, top, o));
      total = 0.0;
      for (int i = 0; i < V; ++i) {
        const int e = lane * V + i;
        const float x = e < p.experts ? load_logit<BF16>(p, row, e) : -INFINITY;
        if (x > -INFINITY) total += score64<SIGMOID>(x, top);
      }
      total = lanes_sum<32>(total);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane * V + i;
      const float x = e < p.experts ? load_logit<BF16>(p, row, e) : -INFINITY;
      double v = -INFINITY;
      if (x > -INFINITY) {
        v = score64<SIGMOID>(x, top);
        if constexpr (!SIGMOID) v /= total;
        if (p.bias) v += static_cast<double>(load_bias(p, e));
      }
      c[i] = order_key64(v);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane * V + i;
      c[i] = e < p.experts ? order_key64(load_logit<BF16>(p, row, e)) : 0ull;
    }
  }
  if (grouped) {
    unsigned long long mine = 0ull;  // lane g: group g's value
    for (int g = 0; g < p.n_groups; ++g) {
      unsigned long long best = 0ull, second = 0ull;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = lane * V + i;
        if (e / p.group_size == g && c[i] > second) {
          second = c[i] > best ? best : c[i];
          best = c[i] > best ? c[i] : best;
        }
      }
      for (int o = 16; o > 0; o >>= 1) {
        const unsigned long long b = __shfl_xor_sync(kAll, best, o);
        const unsigned long long s = __shfl_xor_sync(kAll, second, o);
        const unsigned long long low = b > best ? best : b;
        second = s > second ? s : second;
        second = low > second ? low : second;
        best = b > best ? b : best;
      }
      if (p.group_top == 2 && second != 0ull)
        best = order_key64(key_value64(best) + key_value64(second));
      if (lane == g) mine = best;
    }
    unsigned kept = 0;
    for (int r = 0; r < p.top_groups; ++r) {
      const unsigned long long m = lanes_max64(mine);
      if (m == 0ull) break;
      const int g = __ffs(__ballot_sync(kAll, mine == m)) - 1;
      kept |= 1u << g;
      if (lane == g) mine = 0ull;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane * V + i;
      if (e < p.experts && !((kept >> (e / p.group_size)) & 1u)) c[i] = 0ull;
      // without a bias the logits order the experts
      else if (!p.bias && c[i] != 0ull) c[i] = order_key64(load_logit<BF16>(p, row, e));
    }
  }
  int mine = -1;
  for (int r = 0; r < p.k; ++r) {
    unsigned long long best = c[0];
    int at = lane * V;
#pragma unroll
    for (int i = 1; i < V; ++i)
      if (c[i] > best) { best = c[i]; at = lane * V + i; }
    const unsigned long long m = lanes_max64(best);
    if (m == 0ull) break;
    const int e = __reduce_min_sync(kAll, best == m ? at : 0x7fffffff);
    if (lane == r) mine = e;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (lane * V + i == e) c[i] = 0ull;
  }
  return mine;
}

// Softmax statistics of a row in fp64, by the whole warp.
template <bool BF16>
__device__ __forceinline__ void softmax64(const RouteParams& p, long long row, int lane,
                                          double& top, double& total) {
  float most = -FLT_MAX;
  for (int e = lane; e < p.experts; e += 32) most = fmaxf(most, load_logit<BF16>(p, row, e));
  top = lanes_max<32>(most);
  total = 0.0;
  for (int e = lane; e < p.experts; e += 32)
    total += score64<false>(load_logit<BF16>(p, row, e), top);  // e^-inf is 0
  total = lanes_sum<32>(total);
}

// The place of one of up to 32 candidates, lane l's expert e (-1: none), in
// their order by exact values; without a bias by their logits. The count of
// candidates before it is its place: no rounds, and no lane waits for another.
template <bool SIGMOID, bool BF16>
__device__ __noinline__ int settle(const RouteParams& p, long long row, int lane, int e) {
  double top = 0.0, total = 1.0;
  if (!SIGMOID && p.bias) softmax64<BF16>(p, row, lane, top, total);
  unsigned long long key = 0ull;
  if (e >= 0) {
    double v = load_logit<BF16>(p, row, e);
    if (p.bias) {
      v = score64<SIGMOID>(v, top);
      if constexpr (!SIGMOID) v /= total;
      v += static_cast<double>(load_bias(p, e));
    }
    key = order_key64(v);
  }
  int before = 0;
  for (unsigned left = __ballot_sync(kAll, e >= 0); left != 0u; left &= left - 1) {
    const int l = __ffs(left) - 1;
    const unsigned long long u = __shfl_sync(kAll, key, l);
    const int f = __shfl_sync(kAll, e, l);
    before += u > key || (u == key && f < e) ? 1 : 0;
  }
  return before;
}

// Which groups stay, as a mask, where fp32 cannot tell: lane g holds group g's
// value (-inf: none), whether it would stay, and `bound`, how far two values
// must be apart to be in order. Only groups near the border are done exactly,
// each by the whole warp.
template <bool SIGMOID, bool BF16>
__device__ __noinline__ unsigned settle_groups(const RouteParams& p, long long row, int lane,
                                               float value, bool stays, float bound) {
  const float low = -lanes_max<32>(stays ? -value : -INFINITY);
  const float high = lanes_max<32>(stays ? -INFINITY : value);
  const bool border = value > -INFINITY && !((stays ? value - high : low - value) > bound);
  const unsigned kept = __ballot_sync(kAll, stays && !border);
  double top = 0.0, total = 1.0;
  // without a bias the total is a common factor
  if constexpr (!SIGMOID) softmax64<BF16>(p, row, lane, top, total);
  unsigned long long mine = 0ull;
  for (unsigned left = __ballot_sync(kAll, border); left != 0u; left &= left - 1) {
    const int g = __ffs(left) - 1;
    unsigned long long best = 0ull, second = 0ull;
    for (int i = lane; i < p.group_size; i += 32) {
      const int e = g * p.group_size + i;
      const float x = load_logit<BF16>(p, row, e);
      double v = -INFINITY;
      if (x > -INFINITY) {
        v = score64<SIGMOID>(x, top);
        if (p.bias) {
          if constexpr (!SIGMOID) v /= total;
          v += static_cast<double>(load_bias(p, e));
        }
      }
      const unsigned long long key = order_key64(v);
      if (key > best) {
        second = best;
        best = key;
      } else if (key > second) {
        second = key;
      }
    }
    for (int o = 16; o > 0; o >>= 1) {
      const unsigned long long b = __shfl_xor_sync(kAll, best, o);
      const unsigned long long s = __shfl_xor_sync(kAll, second, o);
      const unsigned long long less = b > best ? best : b;
      second = s > second ? s : second;
      second = less > second ? less : second;
      best = b > best ? b : best;
    }
    if (p.group_top == 2 && second != 0ull)
      best = order_key64(key_value64(best) + key_value64(second));
    if (lane == g) mine = best;
  }
  unsigned all = kept;
  for (int r = __popc(kept); r < p.top_groups; ++r) {
    const unsigned long long m = lanes_max64(mine);
    if (m == 0ull) break;
    const int g = __ffs(__ballot_sync(kAll, mine == m)) - 1;
    all |= 1u << g;
    if (lane == g) mine = 0ull;
  }
  return all;
}

// ------------------------------------------------------------------ weights

// 1 / (1 + e^-x) as a quotient whose divisor is between 1 and 2, so that the
// fast division holds and small scores keep their last bits.
__device__ __forceinline__ float sigmoid(float x) {
  const float t = expf(-fabsf(x));
  return __fdividef(x >= 0.0f ? 1.0f : t, 1.0f + t);
}

// Unnormalised weight of a chosen expert with logit x; m: the largest chosen
// logit of the row. Renormalised, both scores are e^x times a factor, taken
// relative to the largest; a sigmoid's factor 1 / (1 + e^x) is 1 where every
// chosen logit is far below 0 (m <= -60) and part of the score elsewhere, so
// nothing underflows that should not.
template <bool SIGMOID>
__device__ __forceinline__ float relative_weight(float x, float m) {
  if (SIGMOID && m > -60.0f) return sigmoid(x);
  return expf(x - m);
}
template <bool SIGMOID>
__device__ __forceinline__ float plain_weight(float x, float top, float total) {
  return SIGMOID ? sigmoid(x) : __fdividef(expf(x - top), total);
}

// Weights of a row's chosen experts, one per lane (-1: none) with its place
// among the K, and the stores. Every place below K is some lane's. top and
// total: the row's softmax statistics, used without renormalisation.
template <bool SIGMOID, bool BF16>
__device__ __forceinline__ void store_choice(const RouteParams& p, long long row, int place, int id,
                                             float top, float total) {
  float w = 0.0f;
  if (place >= p.k) id = -1;
  const float x = id >= 0 ? load_logit<BF16>(p, row, id) : -INFINITY;
  if (p.renormalize) {
    const float m = lanes_max<32>(x);
    if (id >= 0) w = relative_weight<SIGMOID>(x, m);
    const float sum = lanes_sum<32>(w);
    if (id >= 0) w *= __fdividef(p.scale, sum);
  } else if (id >= 0) {
    w = plain_weight<SIGMOID>(x, top, total) * p.scale;
  }
  if (place < p.k) {
    p.weights[row * p.k + place] = w;
    p.ids[row * p.k + place] = id;
  }
}

// Softmax statistics of a row's logits.
template <int V, int L>
__device__ __forceinline__ void softmax_stats(const float (&x)[V], float& top, float& total) {
  top = x[0];
#pragma unroll
  for (int i = 1; i < V; ++i) top = fmaxf(top, x[i]);
  top = fmaxf(lanes_max<L>(top), -FLT_MAX);  // a row of -inf: every e^(x - top) is 0
  total = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) total += expf(x[i] - top);
  total = lanes_sum<L>(total);
}

// score + bias of a logit; a masked expert keeps -inf.
template <bool SIGMOID>
__device__ __forceinline__ float value_of(float x, float b, float top, float inv_total) {
  const float s = SIGMOID ? fast_rcp(1.0f + fast_exp(-x)) : fast_exp(x - top) * inv_total;
  return x > -INFINITY ? s + b : -INFINITY;
}

constexpr float kLogitReach = 32.0f;  // R of Fixed: logits, and values (scores are in [0, 1])
constexpr float kValueReach = 2.0f;

// ------------------------------------------------------------------ one row per warp

// The two largest of a group's values, spread over `lanes` lanes (a power of
// two) that hold V each, in every one of those lanes.
template <int V>
__device__ __forceinline__ void group_best(const float (&c)[V], int lanes, float& best,
                                           float& second) {
  best = c[0];
  second = -INFINITY;
#pragma unroll
  for (int i = 1; i < V; ++i) {
    second = fmaxf(second, fminf(best, c[i]));
    best = fmaxf(best, c[i]);
  }
  for (int o = 1; o < lanes; o <<= 1) {
    const float b = __shfl_xor_sync(kAll, best, o), s = __shfl_xor_sync(kAll, second, o);
    second = fmaxf(fminf(best, b), fmaxf(second, s));
    best = fmaxf(best, b);
  }
}

// One row of up to 32 V experts by the whole warp, with or without groups.
// bias: the lane's biases, where V is small enough to hold them; s_value: 32 V
// floats of the warp's own, for groups that are not runs of lanes.
template <int V, bool SIGMOID, bool BF16, bool VEC>
__device__ __forceinline__ void route_row(const RouteParams& p, long long row, int lane,
                                          const float (&bias)[V <= 8 ? V : 1], float* s_value) {
  constexpr int D = V < 8 ? V : 8;
  constexpr bool kKeepBias = V <= 8;
  const int e0 = lane * V;
  const bool grouped = p.top_groups < p.n_groups;
  const bool biased = p.bias != nullptr;
  // fp32 values (not the logits) decide something
  const bool by_value = biased || (grouped && p.group_top == 2);
  // lanes per group where groups are whole runs of a power of two of lanes
  const int per = p.group_size / V;
  const bool aligned = p.group_size % V == 0 && (per & (per - 1)) == 0;
  const uint32_t none = BF16 && !biased ? kNone16 : kNone;
  float c[V];
  load_row<V, BF16, VEC>(p, row, e0, true, c);
  float top = 0.0f, total = 1.0f, inv_total = 1.0f;
  if (!SIGMOID && (by_value || !p.renormalize)) {
    softmax_stats<V, 32>(c, top, total);
    inv_total = __fdividef(1.0f, total);
  }
  const float largest = SIGMOID ? 1.0f : inv_total;  // of all scores
  // With a bias c becomes the values; without one the logits order the
  // experts and only groups need scores.
  if (biased) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float b;
      if constexpr (kKeepBias) b = bias[i];
      else b = e0 + i < p.experts ? load_bias(p, e0 + i) : 0.0f;
      c[i] = value_of<SIGMOID>(c[i], b, top, inv_total);
    }
  }
  bool stays = true;  // this lane's group (aligned groups)
  if (grouped) {
    // value of a group: in every lane of it (aligned), else in lane g
    float value = -INFINITY, second = -INFINITY;
    bool leader = lane < p.n_groups;
    if (aligned) {
      if (by_value && !biased) {
        float s[V];
#pragma unroll
        for (int i = 0; i < V; ++i) s[i] = value_of<SIGMOID>(c[i], 0.0f, top, inv_total);
        group_best<V>(s, per, value, second);
      } else {
        group_best<V>(c, per, value, second);
      }
      leader = (lane & (per - 1)) == 0 && e0 < p.experts;
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        s_value[e0 + i] =
            by_value && !biased ? value_of<SIGMOID>(c[i], 0.0f, top, inv_total) : c[i];
      __syncwarp();
      if (leader) {
        for (int i = 0; i < p.group_size; ++i) {
          const float v = s_value[lane * p.group_size + i];
          second = fmaxf(second, fminf(value, v));
          value = fmaxf(value, v);
        }
      }
      __syncwarp();
    }
    float size = fabsf(value);
    if (p.group_top == 2 && second > -INFINITY) {
      value += second;
      size += fabsf(second);
    }
    uint32_t key = leader ? order_key(value) : 0u;
    unsigned kept = 0;  // leader lanes of the groups that stay
    uint32_t last = 0u;
    for (int r = 0; r < p.top_groups; ++r) {
      const uint32_t m = __reduce_max_sync(kAll, key);
      if (m == 0u) break;
      last = m;
      const int who = __ffs(__ballot_sync(kAll, key == m)) - 1;
      kept |= 1u << who;
      if (lane == who) key = 0u;
    }
    if (by_value) {
      // |b| <= |c| + largest; the sum of two is rounded once more
      const float err =
          value > -INFINITY ? 2.0f * (SIGMOID ? kSigmoidErr : kSoftmaxErr) * largest +
                                  kAddErr * (2.0f * size + 4.0f * largest + fabsf(value))
                            : 0.0f;
      const float worst = __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(err)));
      if (__any_sync(kAll, key != 0u && !(key_value(last) - value > 2.0f * worst))) {
        // lane g gets group g's value; its leader is lane g * per (aligned)
        const int from = aligned ? lane * per : lane;
        const float v = __shfl_sync(kAll, leader ? value : -INFINITY, from & 31);
        const bool in = lane < p.n_groups;
        const unsigned groups = settle_groups<SIGMOID, BF16>(
            p, row, lane, in ? v : -INFINITY, in && ((kept >> (from & 31)) & 1u), 2.0f * worst);
        if (aligned) kept = __ballot_sync(kAll, leader && ((groups >> (lane / per)) & 1u));
        else kept = groups;
      }
    }
    if (aligned) {
      stays = (kept >> (lane & ~(per - 1))) & 1u;
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (e0 + i < p.experts && !((kept >> ((e0 + i) / p.group_size)) & 1u)) c[i] = -INFINITY;
    }
  }
  // keys
  uint32_t k[D];
  float margin = 0.0f;  // in steps of the keys
  Fixed f = {};
  if (BF16 && !biased) {
    lane_keys<V, D, true>(c, Fixed{}, e0, k);
    if (!stays) {
#pragma unroll
      for (int i = 0; i < D; ++i) k[i] = 0u;
    }
  } else {
    float hi = c[0];
#pragma unroll
    for (int i = 1; i < V; ++i) hi = fmaxf(hi, c[i]);
    const uint32_t hk = __reduce_max_sync(kAll, stays ? order_key(hi) : 0u);
    hi = hk != 0u ? key_value(hk) : -FLT_MAX;
    f = fixed_for(hi, biased ? kValueReach : kLogitReach);
    if (biased)
      margin = 2.0f * f.inv *
                   ((SIGMOID ? kSigmoidErr : kSoftmaxErr) * largest +
                    kAddErr * (2.0f * largest + 4.0f * kValueReach + 4.0f * fabsf(hi))) + 1.0f;
    if (!stays) f.inv = f.add = 0.0f;  // every key of the lane is "none"
    lane_keys<V, D, false>(c, f, e0, k);
  }
  // K rounds: lane r keeps the r-th key
  uint32_t mine = 0u, m = 0u;
  int found = 0, popped = 0;
  for (; found < p.k; ++found) {
    m = __reduce_max_sync(kAll, k[0]);
    if (m < none) break;
    if (lane == found) mine = m;
    const bool won = k[0] == m;
    pop<D>(k, won);
    if (V > D && won) ++popped;
  }
  // a list of 8 that ran empty may have lost larger keys than the last
  bool open = V > D && popped == D;
  if (found < p.k) {
    // out of keys: fewer than K candidates, or some that lie below the
    // fixed-point range
    int valid = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) valid += stays && c[i] > -INFINITY ? 1 : 0;
    if (__reduce_add_sync(kAll, valid) != found) open = true;
  }
  bool near = false;
  if (!(BF16 && !biased)) {
    // each chosen expert against the one before it, and the last against
    // those that are left
    const uint32_t steps = margin < 4194304.0f ? static_cast<uint32_t>(margin) : 4194304u;
    const uint32_t before = __shfl_up_sync(kAll, mine, 1);
    if (lane > 0 && lane < found && (before >> 10) - (mine >> 10) <= steps)
      near = !same_inputs<BF16>(p, row, key_expert(before), key_expert(mine));
    const uint32_t last = __shfl_sync(kAll, mine, found > 0 ? found - 1 : 0);
    uint32_t low = 0u;
    if ((last >> 10) > steps) low = (last >> 10) - steps;
    else if (biased && found > 0) open = true;  // the margin reaches below the range
    int n = found;
    while (found == p.k) {  // usually ends at once
      m = __reduce_max_sync(kAll, k[0]);
      if (m < kNone || (m >> 10) < low) break;
      if (!biased) {
        open = open || near_last<V, BF16>(p, row, last, c, f);
        break;
      }
      if (n == 32) {
        open = true;
        break;
      }
      if (!same_inputs<BF16>(p, row, key_expert(m), key_expert(last))) near = true;
      if (lane == n) mine = m;
      ++n;
      const bool won = k[0] == m;
      pop<D>(k, won);
      if (V > D && won) ++popped;
    }
    if (V > D && popped == D) open = true;
    near = __any_sync(kAll, near);
    open = __any_sync(kAll, open);
    if (near && !open) {
      // every candidate within the margin of the last is in a lane below n
      const int e = lane < n ? key_expert(mine) : -1;
      const int place = settle<SIGMOID, BF16>(p, row, lane, e);
      // fewer than K: the other lanes' places are theirs
      store_choice<SIGMOID, BF16>(p, row, e >= 0 ? place : lane, e, top, total);
      return;
    }
  } else {
    open = __any_sync(kAll, open);
  }
  int id = lane < found ? key_expert(mine) : -1;
  if (open) id = select_exact<V, SIGMOID, BF16>(p, row, lane);
  store_choice<SIGMOID, BF16>(p, row, lane, id, top, total);
}

template <int V>
__device__ __forceinline__ void lane_bias(const RouteParams& p, int e0,
                                          float (&bias)[V <= 8 ? V : 1]) {
  if constexpr (V <= 8) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      bias[i] = p.bias != nullptr && e0 + i < p.experts ? load_bias(p, e0 + i) : 0.0f;
  }
}

template <int V, bool SIGMOID, bool BF16, bool VEC>
__global__ void __launch_bounds__(kRouteWarps * 32)
    route_kernel(const __grid_constant__ RouteParams p) {
  __shared__ float s_value[kRouteWarps][32 * V];
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  float bias[V <= 8 ? V : 1];
  lane_bias<V>(p, lane * V, bias);
  const long long stride = static_cast<long long>(gridDim.x) * kRouteWarps;
  for (long long row = static_cast<long long>(blockIdx.x) * kRouteWarps + warp; row < p.tokens;
       row += stride)
    route_row<V, SIGMOID, BF16, VEC>(p, row, lane, bias, s_value[warp]);
}

// A row of a warp that holds several, where its lists do not reach.
template <int V, bool SIGMOID, bool BF16>
__device__ __noinline__ void route_again(const RouteParams& p, long long row, int lane,
                                         float* s_value) {
  float bias[V <= 8 ? V : 1];
  lane_bias<V>(p, lane * V, bias);
  route_row<V, SIGMOID, BF16, false>(p, row, lane, bias, s_value);
}

// ------------------------------------------------------------------ several rows per warp

// The 8 largest keys of a row in every one of its L lanes, descending, from
// the lanes' 8 largest; next (if wanted): the largest key that is not among
// them.
template <int L>
__device__ __forceinline__ void merge_lanes(uint32_t (&k)[8], uint32_t& next, bool wanted) {
#pragma unroll
  for (int o = 1; o < L; o <<= 1) {
    uint32_t b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = __shfl_xor_sync(kAll, k[i], o);
    if (wanted) {
#pragma unroll
      for (int i = 0; i < 8; ++i) next = max(next, min(k[i], b[7 - i]));
      next = max(next, __shfl_xor_sync(kAll, next, o));
    }
    merge8(k, b);
  }
}

// Rows of V L experts at most, L lanes each, 32 / L rows per warp. Groups are
// whole runs of lanes. SMALLK: K <= 8, the lanes' sorted lists are merged (40
// instructions a level, for all rows of the warp at once); otherwise (V = 8)
// K rounds of a maximum over the lanes' first keys.
template <int V, int L, bool SMALLK, bool SIGMOID, bool BF16, bool VEC>
__global__ void __launch_bounds__(kRouteWarps * 32, V == 8 ? kBlocks8 : V == 32 && !BF16 ? kBlocks32 : 0)
    route_rows_kernel(const __grid_constant__ RouteParams p) {
  static_assert(V == 8 || SMALLK, "longer lists keep their 8 largest keys");
  constexpr int kRows = 32 / L;  // rows of a warp
  // chosen experts per lane: K <= 8, or K <= min(32, 8 L)
  constexpr int kSlots = SMALLK ? 8 / L : (L < 8 ? 8 : 32 / L);
  constexpr int kWide = V * L / 32 < 2 ? 2 : V * L / 32;  // experts per lane, a row per warp
  __shared__ float s_value[kRouteWarps][32 * kWide];
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int sub = lane % L;
  const int e0 = sub * V;
  const bool grouped = p.top_groups < p.n_groups;
  const bool biased = p.bias != nullptr;
  const bool by_value = biased || (grouped && p.group_top == 2);
  const bool check = !(BF16 && !biased);  // bf16 logits have exact keys
  const uint32_t none = check ? kNone : kNone16;
  const int per = p.group_size / V;  // lanes per group
  // Longer lists come through shared memory, as their biases do (padded, so
  // that 8 lanes read from all banks); 8 biases stay in registers.
  constexpr bool kStaged = V > 8;
  using Stage = Staged<V, BF16>;
  __shared__ __align__(16) uint4 s_stage[kStaged ? kRouteWarps : 1][kStaged ? 32 * Stage::C : 1];
  __shared__ __align__(16) float s_bias[kStaged ? L * (V + 4) : 1];
  float bias[kStaged ? 1 : V];
  if constexpr (kStaged) {
    if (biased) {
      for (int e = threadIdx.x; e < p.experts; e += kRouteWarps * 32)
        s_bias[e / V * (V + 4) + e % V] = load_bias(p, e);
      __syncthreads();
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) bias[i] = biased && e0 + i < p.experts ? load_bias(p, e0 + i) : 0.0f;
  }
  // the expert of the lane's i-th value
  auto expert = [&](int i) {
    if constexpr (kStaged) return Stage::expert(sub, i);
    else return e0 + i;
  };
  const long long stride = static_cast<long long>(gridDim.x) * kRouteWarps * kRows;
  for (long long first = (static_cast<long long>(blockIdx.x) * kRouteWarps + (threadIdx.x >> 5)) *
                         kRows;
       first < p.tokens; first += stride) {
    const long long row = first + lane / L;
    const bool there = row < p.tokens;
    float c[V];
    if constexpr (kStaged) {
      const long long rows = p.tokens - first;
      Stage::load(p, first, rows < kRows ? static_cast<int>(rows) : kRows, lane, there,
                  s_stage[threadIdx.x >> 5], c);
    } else {
      load_row<V, BF16, VEC>(p, row, e0, there, c);
    }
    float top = 0.0f, total = 1.0f, inv_total = 1.0f;
    if (!SIGMOID && (by_value || !p.renormalize)) {
      softmax_stats<V, L>(c, top, total);
      inv_total = __fdividef(1.0f, total);
    }
    const float largest = SIGMOID ? 1.0f : inv_total;
    if (biased) {
      if constexpr (kStaged) {
        // four at a time: a piece holds 4 or 8
#pragma unroll
        for (int i = 0; i < V; i += 4) {
          const float4 b =
              sub * V < p.experts
                  ? *reinterpret_cast<const float4*>(&s_bias[sub * (V + 4) + expert(i) % V])
                  : float4{};
          c[i] = value_of<SIGMOID>(c[i], b.x, top, inv_total);
          c[i + 1] = value_of<SIGMOID>(c[i + 1], b.y, top, inv_total);
          c[i + 2] = value_of<SIGMOID>(c[i + 2], b.z, top, inv_total);
          c[i + 3] = value_of<SIGMOID>(c[i + 3], b.w, top, inv_total);
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) c[i] = value_of<SIGMOID>(c[i], bias[i], top, inv_total);
      }
    }
    bool stays = true;  // this lane's group
    if (L > 1 && grouped) {
      float value, second;
      if (by_value && !biased) {
        float s[V];
#pragma unroll
        for (int i = 0; i < V; ++i) s[i] = value_of<SIGMOID>(c[i], 0.0f, top, inv_total);
        group_best<V>(s, per, value, second);
      } else {
        group_best<V>(c, per, value, second);
      }
      float size = fabsf(value);
      if (p.group_top == 2 && second > -INFINITY) {
        value += second;
        size += fabsf(second);
      }
      // rank among the row's groups; ties go to the lower lane
      const uint32_t key = order_key(value);
      int rank = 0;
      for (int d = per; d < L; d += per) {
        const uint32_t other = __shfl_xor_sync(kAll, key, d);
        rank += other > key || (other == key && (sub ^ d) < sub) ? 1 : 0;
      }
      stays = rank < p.top_groups && key != 0u;
      if (by_value) {
        const float err =
            value > -INFINITY ? 2.0f * (SIGMOID ? kSigmoidErr : kSoftmaxErr) * largest +
                                    kAddErr * (2.0f * size + 4.0f * largest + fabsf(value))
                              : 0.0f;
        const float worst = lanes_max<L>(err);
        const float low = -lanes_max<L>(stays ? -value : -INFINITY);  // of those kept
        const float high = lanes_max<L>(stays ? -INFINITY : value);   // of the others
        unsigned todo = __ballot_sync(
            kAll, there && sub == 0 && high > -INFINITY && !(low - high > 2.0f * worst));
        for (; todo != 0u; todo &= todo - 1) {
          // lane g gets group g's value of the row whose first lane is `at`
          const int at = __ffs(todo) - 1;
          const int from = (at + lane * per) & 31;
          const float v = __shfl_sync(kAll, value, from);
          const bool kept = __shfl_sync(kAll, stays ? 1 : 0, from) != 0, in = lane < p.n_groups;
          const float bound = 2.0f * __shfl_sync(kAll, worst, at);
          const unsigned groups = settle_groups<SIGMOID, BF16>(
              p, first + at / L, lane, in ? v : -INFINITY, in && kept, bound);
          if (lane - sub == at) stays = (groups >> (sub / per)) & 1u;
        }
      }
    }
    // keys
    uint32_t k[8];
    uint32_t next = 0u;  // the largest key that is in no list
    uint32_t steps = 0u;
    Fixed f = {};
    if (check) {
      float hi = c[0];
#pragma unroll
      for (int i = 1; i < V; ++i) hi = fmaxf(hi, c[i]);
      hi = fmaxf(lanes_max<L>(stays ? hi : -INFINITY), -FLT_MAX);
      f = fixed_for(hi, biased ? kValueReach : kLogitReach);
      if (biased) {
        const float margin = 2.0f * f.inv *
                                 ((SIGMOID ? kSigmoidErr : kSoftmaxErr) * largest +
                                  kAddErr * (2.0f * largest + 4.0f * kValueReach + 4.0f * fabsf(hi))) +
                             1.0f;
        steps = margin < 4194304.0f ? static_cast<uint32_t>(margin) : 4194304u;
      }
      if (!stays) f.inv = f.add = 0.0f;  // every key of the lane is "none"
    }
#pragma unroll
    for (int v = 0; v < V; v += 8) {
      uint32_t part[8];
      if (check) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          part[i] = fixed_key(c[v + i], f, 1023u - static_cast<uint32_t>(expert(v + i)));
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          part[i] = stays ? bf16_key(c[v + i], 1023u - static_cast<uint32_t>(expert(v + i))) : 0u;
      }
      sort_descending<8>(part);
      if (v == 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) k[i] = part[i];
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) next = max(next, min(k[i], part[7 - i]));
        merge8(k, part);
      }
    }
    uint32_t keep[kSlots];  // lane l: keys l, l + L, ...
    uint32_t last = 0u;
    int found = 0;
    bool near = false, open = false;
    if constexpr (SMALLK) {
      merge_lanes<L>(k, next, check || V > 8);  // a branch costs long lists more than it saves
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool is = i < p.k && k[i] >= none;
        found += is ? 1 : 0;
        last = is ? k[i] : last;
      }
#pragma unroll
      for (int s = 0; s < kSlots; ++s) {
        keep[s] = k[s * L];
#pragma unroll
        for (int l = 1; l < L; ++l)
          if (s * L + l < 8) keep[s] = sub == l ? k[s * L + l] : keep[s];
      }
      if (check) {
        // the smallest distance between keys in a row down to the first that
        // is left out; the index part is worth less than a step
        uint32_t least = 0xffffffffu;
#pragma unroll
        for (int i = 1; i < 8; ++i)
          if (i <= p.k && k[i] >= none) least = min(least, k[i - 1] - k[i]);
        if (p.k == 8 && next >= none) least = min(least, k[7] - next);
        const bool close = there && found > 0 && (least >> 10) <= steps;
        if (biased && found > 0 && (last >> 10) <= steps) open = true;  // below the range
        if (__any_sync(kAll, close)) {
          if (close) {
#pragma unroll
            for (int i = 1; i < 8; ++i)
              if (i < found && (k[i - 1] >> 10) - (k[i] >> 10) <= steps)
                near = near || !same_inputs<BF16>(p, row, key_expert(k[i - 1]), key_expert(k[i]));
            // the last against the rest; past the lists only another look helps
            const uint32_t low = (last >> 10) > steps ? (last >> 10) - steps : 0u;
            if (found == p.k && !biased) {
              open = open || near_last<V, BF16>(p, row, last, c, f);
            } else if (found == p.k) {
#pragma unroll
              for (int i = 1; i < 8; ++i)
                if (i >= p.k && k[i] >= none && (k[i] >> 10) >= low)
                  near = near || !same_inputs<BF16>(p, row, key_expert(last), key_expert(k[i]));
              if (next >= none && (next >> 10) >= low)
                open = open || near ||
                       !same_inputs<BF16>(p, row, key_expert(last), key_expert(next));
            }
          }
          open = lanes_max<L>(open ? 1u : 0u) != 0u;  // near_last looks at one lane's
        }
      }
    } else {
#pragma unroll
      for (int s = 0; s < kSlots; ++s) {
        keep[s] = 0u;
        if (s * L < p.k) {
          for (int l = 0; l < L && s * L + l < p.k; ++l) {
            const uint32_t m = lanes_max<L>(k[0]);
            if (m >= none) {
              if (check && found > 0 && (last >> 10) - (m >> 10) <= steps)
                near = near || !same_inputs<BF16>(p, row, key_expert(last), key_expert(m));
              if (sub == l) keep[s] = m;
              last = m;
              ++found;
              pop<8>(k, k[0] == m);
            }
          }
        }
      }
      if (check) {
        // the last against those that are left
        uint32_t low = 0u;
        if ((last >> 10) > steps) low = (last >> 10) - steps;
        else if (biased && found > 0) open = true;  // the margin reaches below the range
        while (true) {  // usually ends at once
          const uint32_t m = lanes_max<L>(k[0]);
          const bool close = found == p.k && !near && m >= none && (m >> 10) >= low;
          if (!__any_sync(kAll, close)) break;
          if (close) {
            near = !same_inputs<BF16>(p, row, key_expert(m), key_expert(last));
            pop<8>(k, k[0] == m);
          }
        }
      }
    }
    if (__any_sync(kAll, found < p.k)) {
      // out of keys: fewer than K candidates, or some below the fixed-point range
      int valid = 0;
#pragma unroll
      for (int i = 0; i < V; ++i) valid += stays && c[i] > -INFINITY ? 1 : 0;
      valid = lanes_sum<L>(valid);
      open = open || (found < p.k && valid != found);
    }
    const bool again = there && (near || open);
    // weights
    float x[kSlots], w[kSlots];
    float m = -INFINITY;
#pragma unroll
    for (int s = 0; s < kSlots; ++s) {
      x[s] = -INFINITY;
      if (s * L + sub < p.k && keep[s] >= none) {
        x[s] = load_logit<BF16>(p, row, key_expert(keep[s]));
        m = fmaxf(m, x[s]);
      }
    }
    float factor = p.scale;
    if (p.renormalize) {
      m = lanes_max<L>(m);
      float sum = 0.0f;
#pragma unroll
      for (int s = 0; s < kSlots; ++s) {
        w[s] = 0.0f;
        if (s * L < p.k && x[s] > -INFINITY) w[s] = relative_weight<SIGMOID>(x[s], m);
        sum += w[s];
      }
      sum = lanes_sum<L>(sum);
      factor = sum > 0.0f ? __fdividef(p.scale, sum) : 0.0f;
    } else {
#pragma unroll
      for (int s = 0; s < kSlots; ++s) {
        w[s] = 0.0f;
        if (s * L < p.k && x[s] > -INFINITY) w[s] = plain_weight<SIGMOID>(x[s], top, total);
      }
    }
    if (there && !again) {
      float* w_at = p.weights + row * p.k;
      int32_t* id_at = p.ids + row * p.k;
#pragma unroll
      for (int s = 0; s < kSlots; ++s) {
        const int r = s * L + sub;
        if (r < p.k) {
          w_at[r] = w[s] * factor;
          id_at[r] = keep[s] >= none ? key_expert(keep[s]) : -1;
        }
      }
    }
    // rows that fp32 could not decide, by the whole warp
    unsigned todo = __ballot_sync(kAll, again && sub == 0);
    while (todo != 0u) {
      const int at = __ffs(todo) - 1;
      todo &= todo - 1;
      const long long r = first + at / L;
      if (!SMALLK || __shfl_sync(kAll, open ? 1 : 0, at) != 0) {
        route_again<kWide, SIGMOID, BF16>(p, r, lane, s_value[threadIdx.x >> 5]);
        continue;
      }
      // every candidate is among the 8 keys: lane l takes the l-th
      uint32_t cand = 0u;
#pragma unroll
      for (int s = 0; s < kSlots; ++s) {
        const uint32_t v = __shfl_sync(kAll, keep[s], at + (lane & (L - 1)));
        cand = lane / L == s ? v : cand;
      }
      const int id = lane < 8 && cand >= none ? key_expert(cand) : -1;
      const int place = settle<SIGMOID, BF16>(p, r, lane, id);
      // fewer than K: the other lanes' places are theirs
      store_choice<SIGMOID, BF16>(p, r, id >= 0 ? place : lane, id, __shfl_sync(kAll, top, at),
                                  __shfl_sync(kAll, total, at));
    }
  }
}

using RouteFn = void (*)(RouteParams);

// One row per warp, V = 1 .. 32 experts per lane; whole 16-byte loads exist
// where a lane's run is at least 16 bytes (V = 4 fp32, V = 8 both).
#define TW_ROUTE(S, B, X) {route_kernel<1, S, B, false>, route_kernel<2, S, B, false>, \
                           route_kernel<4, S, B, (X) && !(B)>, route_kernel<8, S, B, X>, \
                           route_kernel<16, S, B, X>, route_kernel<32, S, B, X>}
#define TW_ROUTE2(S, B) {TW_ROUTE(S, B, false), TW_ROUTE(S, B, true)}
const RouteFn kRoute[2][2][2][6] = {{TW_ROUTE2(false, false), TW_ROUTE2(false, true)},
                                    {TW_ROUTE2(true, false), TW_ROUTE2(true, true)}};
#undef TW_ROUTE2
#undef TW_ROUTE
// Several rows per warp, 8 experts per lane, L = 1 .. 8 lanes; K <= 8, or more
// (not for L = 1).
#define TW_ROWS(S, B, X) \
  {{route_rows_kernel<8, 1, true, S, B, X>, route_rows_kernel<8, 2, true, S, B, X>, \
    route_rows_kernel<8, 4, true, S, B, X>, route_rows_kernel<8, 8, true, S, B, X>}, \
   {nullptr, route_rows_kernel<8, 2, false, S, B, X>, route_rows_kernel<8, 4, false, S, B, X>, \
    route_rows_kernel<8, 8, false, S, B, X>}}
#define TW_ROWS2(S, B) {TW_ROWS(S, B, false), TW_ROWS(S, B, true)}
const RouteFn kRows[2][2][2][2][4] = {{TW_ROWS2(false, false), TW_ROWS2(false, true)},
                                      {TW_ROWS2(true, false), TW_ROWS2(true, true)}};
#undef TW_ROWS2
#undef TW_ROWS
// 16 and 32 experts per lane, 8 lanes, whole vectors, K <= 8.
#define TW_LONG(S, B) {route_rows_kernel<16, 8, true, S, B, true>, \
                       route_rows_kernel<32, 8, true, S, B, true>}
const RouteFn kLong[2][2][2] = {{TW_LONG(false, false), TW_LONG(false, true)},
                                {TW_LONG(true, false), TW_LONG(true, true)}};
#undef TW_LONG

// Whether groups are runs of a power of two of lanes with v experts each.
bool groups_fit(const RouteArgs& a, int v) {
  if (a.top_groups == a.n_groups) return true;
  const int size = a.experts / a.n_groups, per = size / v;
  return size % v == 0 && (per & (per - 1)) == 0;
}

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
  const int sigmoid = a.scoring == TW_SCORE_SIGMOID, bf16 = a.logits_type == TW_LOGITS_BF16;
  const int64_t row_bytes = static_cast<int64_t>(a.experts) * (bf16 ? 2 : 4);
  const bool on16 = reinterpret_cast<uintptr_t>(a.logits) % 16 == 0 && row_bytes % 16 == 0;
  RouteFn fn;
  int64_t rows_per_block = kRouteWarps;
  const int v_long = a.experts <= 128 ? 16 : 32;
  const bool by_value = a.bias != nullptr || (a.top_groups < a.n_groups && a.group_top == 2);
  if (a.experts <= 64 && groups_fit(a, 8)) {
    int l = 0;
    while ((8 << l) < a.experts) ++l;
    fn = kRows[sigmoid][bf16][on16 && a.experts % 8 == 0][a.k > 8][l];
    rows_per_block *= 32 >> l;
  } else if (a.experts <= 256 && a.k <= 8 && on16 && a.experts % v_long == 0 &&
             groups_fit(a, v_long) &&
             a.tokens >= (by_value ? kLongTokensByValue : kLongTokens)) {
    fn = kLong[sigmoid][bf16][v_long == 32];
    rows_per_block *= 4;
  } else {
    int v = 0;
    while ((32 << v) < a.experts) ++v;
    fn = kRoute[sigmoid][bf16][on16 && a.experts % (1 << v) == 0][v];
  }
  int64_t blocks = (a.tokens + rows_per_block - 1) / rows_per_block;
  if (blocks > kRouteBlocks) blocks = kRouteBlocks;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(kRouteWarps * 32);
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

}  // namespace tw
