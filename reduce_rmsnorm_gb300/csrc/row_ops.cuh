// Device helpers shared by the row kernels (fused_forms.cuh, combine_kernel.cu):
// programmatic dependent launch, the L2 prefetch hint, bf16 vectors of 8, the
// e4m3 output with its scales and the end of a row.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "tw.h"

namespace tw {
namespace {

// ------------------------------------------------------------------ launch order, prefetch

// Asks L2 to fetch [src, src + bytes) (16-byte aligned, bytes a multiple of
// 16). A hint only: nothing is returned to the thread and no memory is written.
__device__ __forceinline__ void prefetch_l2(const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ void grid_dependency_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

__device__ __forceinline__ void grid_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// ------------------------------------------------------------------ bf16 x 8

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ __forceinline__ void load8(const uint4 q, float a[8]) {
  a[0] = bf16_lo(q.x); a[1] = bf16_hi(q.x);
  a[2] = bf16_lo(q.y); a[3] = bf16_hi(q.y);
  a[4] = bf16_lo(q.z); a[5] = bf16_hi(q.z);
  a[6] = bf16_lo(q.w); a[7] = bf16_hi(q.w);
}

// a[2i], a[2i+1] += the two bf16 values of word w, as one packed fp32x2 add
// (add.rn.f32x2: two independent IEEE round-to-nearest fp32 additions, the
// same results as two scalar adds, in one instruction).
__device__ __forceinline__ void add2(float& lo, float& hi, uint32_t w) {
  uint64_t acc, v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(acc) : "f"(lo), "f"(hi));
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(w << 16), "r"(w & 0xffff0000u));
  asm("add.rn.f32x2 %0, %0, %1;" : "+l"(acc) : "l"(v));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(acc));
}

__device__ __forceinline__ void add8(const uint4 q, float a[8]) {
  add2(a[0], a[1], q.x);
  add2(a[2], a[3], q.y);
  add2(a[4], a[5], q.z);
  add2(a[6], a[7], q.w);
}

// y[i] = (z[i] * rs) * gamma[i] for the 8 bf16 gamma values of q, as packed
// fp32x2 multiplies (mul.rn.f32x2: two IEEE round-to-nearest products per
// instruction, the same results as scalar multiplies in the same order).
__device__ __forceinline__ void scale8(const float z[8], float rs, const uint4 q, float y[8]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  uint64_t r2;
  asm("mov.b64 %0, {%1, %1};" : "=l"(r2) : "f"(rs));
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint64_t a, g;
    asm("mov.b64 %0, {%1, %2};" : "=l"(a) : "f"(z[2 * k]), "f"(z[2 * k + 1]));
    asm("mov.b64 %0, {%1, %2};" : "=l"(g) : "r"(w[k] << 16), "r"(w[k] & 0xffff0000u));
    asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(a) : "l"(r2));
    asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(a) : "l"(g));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(y[2 * k]), "=f"(y[2 * k + 1]) : "l"(a));
  }
}

// Sum of the 8 warp partials in warp order, read as two 16-byte loads.
__device__ __forceinline__ float warp_total(const float* w8) {
  const float4 a = *reinterpret_cast<const float4*>(w8);
  const float4 b = *reinterpret_cast<const float4*>(w8 + 4);
  return ((((((a.x + a.y) + a.z) + a.w) + b.x) + b.y) + b.z) + b.w;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint4 pack8(const float a[8]) {
  return make_uint4(pack2(a[0], a[1]), pack2(a[2], a[3]), pack2(a[4], a[5]), pack2(a[6], a[7]));
}

// ------------------------------------------------------------------ e4m3 with scales
//
// A group of g consecutive values (or the whole row) has one scale s and codes
// q = e4m3_rne_sat(y / s). With a = max |y| over the group:
//   fp32 scales  s = max(a / 448, 2^-126)
//   e8m0 scales  s = the smallest power of two >= a / 448, at least 2^-126
// 448 is e4m3's largest value, so no finite code saturates; the lower bound
// keeps 1 / s finite and gives a group of zeros the codes 0. y is the unrounded
// fp32 value: rounding it to bf16 first would put a second rounding (2^-9) under
// the 8-bit one (2^-4) for nothing.
constexpr float kE4m3Max = 448.0f;
constexpr float kScaleMin = 1.17549435082228750797e-38f;  // 2^-126

// The stored scale of a group and the factor 1 / s that its values take.
struct GroupScale {
  float scale;     // TW_SCALE_F32
  uint32_t code;   // TW_SCALE_E8M0: the biased exponent
  float inv;
};

// 448 = 1.75 * 2^8, so for a = m * 2^e (1 <= m < 2) the smallest power of two
// >= a / 448 is 2^(e - 8) for m <= 1.75 and 2^(e - 7) above: an exact rule on
// a's bits, with no division whose rounding could cross the border. An infinite
// a has an infinite (fp32) or NaN (e8m0) scale; fmaxf drops a NaN.
// FAST: a product and an approximate reciprocal, each within an ulp, for the
// two divisions of an fp32 scale (see finish_row).
template <bool FAST>
__device__ __forceinline__ GroupScale group_scale(float amax, int scale_type) {
  GroupScale g;
  if (scale_type == TW_SCALE_E8M0) {
    const uint32_t b = __float_as_uint(fmaxf(amax, 0.0f));
    const int e = static_cast<int>(b >> 23) - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
    const bool inf = b == 0x7f800000u;
    g.code = inf ? 255u : static_cast<uint32_t>(e < 1 ? 1 : e);
    g.inv = inf ? 0.0f : __uint_as_float((254u - g.code) << 23);  // code <= 247
    g.scale = 0.0f;
  } else {
    g.scale = fmaxf(FAST ? amax * (1.0f / kE4m3Max) : amax / kE4m3Max, kScaleMin);
    if constexpr (FAST) asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(g.inv) : "f"(g.scale));
    else g.inv = 1.0f / g.scale;
    g.code = 0u;
  }
  return g;
}

__device__ __forceinline__ void store_scale(void* scales, long long at, const GroupScale& g,
                                            int scale_type) {
  if (scale_type == TW_SCALE_E8M0) static_cast<unsigned char*>(scales)[at] = static_cast<unsigned char>(g.code);
  else static_cast<float*>(scales)[at] = g.scale;
}

// Eight values times inv as e4m3 (round to nearest even, saturating; a NaN
// stays NaN), in memory order.
__device__ __forceinline__ uint2 pack_e4m3(const float y[8], float inv) {
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
        : "=h"(lo)
        : "f"(y[4 * h + 1] * inv), "f"(y[4 * h] * inv));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
        : "=h"(hi)
        : "f"(y[4 * h + 3] * inv), "f"(y[4 * h + 2] * inv));
    w[h] = static_cast<uint32_t>(lo) | static_cast<uint32_t>(hi) << 16;
  }
  return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ float amax8(const float y[8]) {
  float m = fabsf(y[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) m = fmaxf(m, fabsf(y[i]));
  return m;
}

// ------------------------------------------------------------------ the end of a row

constexpr int kConsumerWarps = 8;  // of a pipeline
constexpr int kConsumerThreads = kConsumerWarps * 32;
constexpr int kConsumerBarrierId = 1;            // named barrier of the consumer warps

// The end of a row, shared by every kernel form: the sum of squares is
// reduced across the warp (xor shuffle) and then across the pipeline's 8
// warps in warp order (through `wsum`, this row's 8 floats), r = rsqrt(mean +
// eps), and Y = (z * r) * gamma is stored as bf16. With evict-first loads the
// output is stored streaming too, so its lines drain during this launch; with
// normal loads the store policy measured within 0.2%. A kernel that reads Y
// right after still finds it unless L2 needs the room. The residual keeps the
// default policy (evict-first there measured -1%).
//
// Q8: a group's largest |y| comes from an xor shuffle, since its group / 8
// vectors lie in adjacent lanes of one warp and slot. One scale for the row
// needs no second barrier: max |z gamma| is reduced beside the sum of squares
// (`wmax`), and r times it is max |y| up to the products' roundings (2^-23,
// against the codes' 2^-4).
//
// Thread t of `threads` (a multiple of 32, at most 256) owns the vectors t, t +
// threads, ...: slot j is vector j * threads + t. With fewer than 8 warps the
// others' wsum and wmax are 0.
//
// gamma(j, v): the thread's j-th vector of gamma, which is the row's vector v.
// Rows of more than 2 vectors a thread that do not fill whole slots take the
// fast scale (3 to 10% of a combine launch); the others do not, where the
// largest (T = 8192, H = 16384, N = 8) took 418 us with it and 400 without. The
// choice depends on H alone, as every bit of a row does.
template <int KMAX, bool EXACT, bool Q8, typename P, typename Gamma>
__device__ __forceinline__ void finish_row(const P& p, float ss, const float (&z)[KMAX][8],
                                           const Gamma& gamma, float* wsum, float* wmax,
                                           int bar_id, int threads, int lane, int wg, int t,
                                           int vpr, long long row) {
  constexpr bool FAST = KMAX > 2 && !EXACT;
  const bool row_scale = Q8 && p.group == 8 * vpr;
  float am = 0.0f;
  if constexpr (Q8) {
    if (row_scale) {
#pragma unroll
      for (int j = 0; j < KMAX; ++j) {
        const int v = j * threads + t;
        if (EXACT || v < vpr) {
          float y[8];
          scale8(z[j], 1.0f, gamma(j, v), y);
          am = fmaxf(am, amax8(y));
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  if (lane == 0) {
    wsum[wg] = ss;
    if constexpr (Q8) wmax[wg] = am;
  }
  asm volatile("bar.sync %0, %1;" ::"r"(bar_id), "r"(threads) : "memory");
  const float total = warp_total(wsum);
  const float rs = rsqrtf(total / p.hidden + p.eps);
  if constexpr (Q8) {
    uint2* out_row = static_cast<uint2*>(p.out) + row * vpr;
    GroupScale gs = {};
    if (row_scale) {
      const float4 a = *reinterpret_cast<const float4*>(wmax);
      const float4 b = *reinterpret_cast<const float4*>(wmax + 4);
      am = fmaxf(fmaxf(fmaxf(a.x, a.y), fmaxf(a.z, a.w)), fmaxf(fmaxf(b.x, b.y), fmaxf(b.z, b.w)));
      gs = group_scale<FAST>(am * rs, p.scale_type);
      if (t == 0) store_scale(p.scales, row, gs, p.scale_type);
    }
    const int per = p.group >> 3;  // vectors per group, a power of two unless it is the row
    const int per_log2 = 31 - __clz(per);
    // a few slots at a time, so that their shuffles overlap: T = 8192, H =
    // 16384, N = 8 takes 404 us with one slot at a time, 400 with two, 418 with
    // four
    constexpr int B = KMAX <= 4 ? KMAX : 2;
#pragma unroll
    for (int j0 = 0; j0 < KMAX; j0 += B) {
      if (!EXACT && j0 * threads >= vpr) break;
      float y[B][8], a[B];
#pragma unroll
      for (int u = 0; u < B; ++u) {
        const int j = j0 + u, v = j * threads + t;
#pragma unroll
        for (int i = 0; i < 8; ++i) y[u][i] = 0.0f;
        if (EXACT || v < vpr) {
          scale8(z[j], rs, gamma(j, v), y[u]);
        }
        a[u] = amax8(y[u]);
      }
      if (!row_scale) {
        for (int o = per >> 1; o > 0; o >>= 1)
#pragma unroll
          for (int u = 0; u < B; ++u) a[u] = fmaxf(a[u], __shfl_xor_sync(0xffffffffu, a[u], o));
      }
#pragma unroll
      for (int u = 0; u < B; ++u) {
        const int v = (j0 + u) * threads + t;
        if (EXACT || v < vpr) {
          if (!row_scale) {
            gs = group_scale<FAST>(a[u], p.scale_type);
            if ((v & (per - 1)) == 0)
              store_scale(p.scales, (row * vpr + v) >> per_log2, gs, p.scale_type);
          }
          const uint2 q = pack_e4m3(y[u], gs.inv);
          if (p.l2_stream) __stcs(out_row + v, q);
          else out_row[v] = q;
        }
      }
    }
  } else {
    uint4* out_row = static_cast<uint4*>(p.out) + row * vpr;
#pragma unroll
    for (int j = 0; j < KMAX; ++j) {
      const int v = j * threads + t;
      if (EXACT || v < vpr) {
        float y[8];
        scale8(z[j], rs, gamma(j, v), y);
        if (p.l2_stream) __stcs(out_row + v, pack8(y));
        else out_row[v] = pack8(y);
      }
    }
  }
}

}  // namespace
}  // namespace tw
