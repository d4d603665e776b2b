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
// A CTA has `threads` consumer threads (a multiple of 32, at most 256), chosen
// so that KMAX vectors each just cover the row: thread t owns the 16-byte
// vectors t, t + threads, ... The choice depends on H alone, so the order of
// every sum does too, and both forms below give bitwise the same rows under
// every grid.
//
//   Ring    (up to 32 sources): each CTA owns a contiguous range of rows. A
//           producer warp reads the indices a row ahead and copies a row
//           chunk by chunk into a ring of shared-memory stages, a stage holding
//           one chunk (4 or 8 KiB) of every source, one bulk copy per lane
//           (mbarrier completion): about 200 KB in flight per SM whatever the
//           consumers do. The consumers read the same indices, and both sides
//           count chunks alone, so a wait that gives up leaves every barrier
//           matched. (A stage per source row instead, with a wait per source,
//           took 280 ns a stage whatever its size.) A CTA finishes a row
//           before it adds up the next, so short rows share an SM among several
//           CTAs: at T = 4800, H = 1024, K = 8 one CTA took 27 us, three 18.9.
//   Direct  (more than 32 sources, which do not fit a warp's lanes or a
//           stage): one CTA per row; a thread's vectors of U sources at a time
//           go straight into registers. Every warp reads the row's K indices
//           and weights itself (lane k slot k) and hands them round by shuffle,
//           so no barrier stands between the indices and the gathers. Where
//           both fit it is 5 to 50% slower (T = 1, H = 4096, K = 8 3.2 against
//           2.8 us; T = 1024, H = 8192, K = 8 40.9 against 29.9).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <mutex>

#include "ring_ops.cuh"
#include "row_ops.cuh"
#include "tw_internal.h"

namespace tw {

namespace {

constexpr int kMaxGrid = 1 << 16;
constexpr uint32_t kPrefetchDense = 16u * 1024u;  // per dense source and CTA
constexpr int kMaxShare = 8;  // ring CTAs per SM
// Stages that each of several ring CTAs on an SM has at least. Two against one:
// H = 2048, K = 8 at T = 1000 8.5 / 10.4 us, at T = 2000 15.1 / 16.8; the same
// elsewhere.
constexpr int kMinStages = 2;
constexpr int kStaticSmemReserve = 4096;  // barriers, sums, weights, flag, slack

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
  int l2_stream;  // 1: evict-first loads and a streaming output (ring)
  int threads;    // consumer threads
  int stages;     // ring
  float eps;
  float hidden;
};

// Sources whose loads are in flight at once, by vectors per thread: 8 to 16
// loads, 128 to 256 bytes a thread.
template <int KMAX>
constexpr int kBatch = KMAX == 1 ? 8 : KMAX <= 4 ? 4 : KMAX == 8 ? 2 : 1;

// z[j] += w * (the thread's vectors of a source row), one fma per value; a
// partial has w = 1, which makes it an addition.
template <int KMAX>
__device__ __forceinline__ void add_source(const uint4 (&q)[KMAX], float w, float (&z)[KMAX][8]) {
#pragma unroll
  for (int j = 0; j < KMAX; ++j) {
    float x[8];
    load8(q[j], x);
#pragma unroll
    for (int i = 0; i < 8; ++i) z[j][i] = fmaf(w, x[i], z[j][i]);
  }
}

// Lane k's slot of a row: its index (-1: nothing to add) and weight.
struct Slot {
  int index;
  float weight;
};
__device__ __forceinline__ Slot load_slot(const CombineParams& p, long long row, int lane) {
  Slot s = {-1, 0.0f};
  if (lane < p.k) {
    s.index = __ldg(p.rows + row * p.k + lane);
    s.weight = __ldg(p.weights + row * p.k + lane);
  }
  return s;
}
// The slots that add something, as a mask; the first warp of the row reports
// indices outside the expert rows.
__device__ __forceinline__ unsigned kept_slots(const CombineParams& p, const Slot& s, bool report) {
  const bool kept = s.index >= 0 && s.index < p.m;
  if (report && !kept && s.index != -1) atomicOr(&g_device_error, 8u);
  return __ballot_sync(0xffffffffu, kept);
}

template <int KMAX, bool EXACT>
__device__ __forceinline__ float square_sum(const float (&z)[KMAX][8], int t, int threads, int vpr) {
  float ss = 0.0f;
#pragma unroll
  for (int j = 0; j < KMAX; ++j)
    if (EXACT || j * threads + t < vpr) {
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(z[j][i], z[j][i], ss);
    }
  return ss;
}

template <int KMAX, bool Q8>
__global__ void __launch_bounds__(kConsumerThreads)
    combine_kernel(const __grid_constant__ CombineParams p) {
  __shared__ __align__(16) float s_sum[2][kConsumerWarps];
  __shared__ __align__(16) float s_max[2][kConsumerWarps];
  constexpr int U = kBatch<KMAX>;
  const int t = threadIdx.x;
  const int lane = t & 31;
  const int warp = t >> 5;
  const int threads = p.threads;
  const int vpr = p.vec_per_row;
  if (t < 2 * kConsumerWarps) {
    s_sum[t / kConsumerWarps][t % kConsumerWarps] = 0.0f;
    s_max[t / kConsumerWarps][t % kConsumerWarps] = 0.0f;
  }
  __syncthreads();
  grid_dependency_wait();
  grid_launch_dependents();
  auto gamma = [&](int, int v) { return __ldg(p.gamma + v); };
  int buf = 0;
  for (long long row = blockIdx.x; row < p.tokens; row += gridDim.x, buf ^= 1) {
    const Slot slot = load_slot(p, row, lane);
    uint4* res_row = p.residual + row * vpr;
    // the residual's loads go out before the indices arrive, registers allowing
    constexpr bool kEarly = KMAX <= 8;
    uint4 res[kEarly ? KMAX : 1];
    if constexpr (kEarly) {
#pragma unroll
      for (int j = 0; j < KMAX; ++j) {
        const int v = j * threads + t;
        res[j] = v < vpr ? res_row[v] : make_uint4(0, 0, 0, 0);
      }
    }
    float z[KMAX][8];
#pragma unroll
    for (int j = 0; j < KMAX; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) z[j][i] = -0.0f;  // -0 + x is x, -0 too
    // the kept slots in order, U at a time
    for (unsigned left = kept_slots(p, slot, warp == 0); left != 0u;) {
      uint4 q[U][KMAX];
      float w[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const bool there = left != 0u;
        const int l = there ? __ffs(left) - 1 : 0;
        left &= left - 1;
        const long long r = __shfl_sync(0xffffffffu, slot.index, l);
        const float weight = __shfl_sync(0xffffffffu, slot.weight, l);
        w[u] = there ? weight : 0.0f;
        const uint4* src = p.experts + r * vpr;
#pragma unroll
        for (int j = 0; j < KMAX; ++j) {
          const int v = j * threads + t;
          q[u][j] = there && v < vpr ? __ldg(src + v) : make_uint4(0, 0, 0, 0);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) add_source<KMAX>(q[u], w[u], z);
    }
    for (int n = 0; n < p.n; n += U) {
      uint4 q[U][KMAX];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint4* src = p.partials[n + u < p.n ? n + u : 0] + row * vpr;
#pragma unroll
        for (int j = 0; j < KMAX; ++j) {
          const int v = j * threads + t;
          q[u][j] = n + u < p.n && v < vpr ? src[v] : make_uint4(0, 0, 0, 0);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (n + u < p.n) {
#pragma unroll
          for (int j = 0; j < KMAX; ++j) add8(q[u][j], z[j]);
        }
    }
#pragma unroll
    for (int j = 0; j < KMAX; ++j) {
      const int v = j * threads + t;
      if (v < vpr) {
        if constexpr (kEarly) add8(res[j], z[j]);
        else add8(res_row[v], z[j]);
        res_row[v] = pack8(z[j]);
      }
    }
    const float ss = square_sum<KMAX, false>(z, t, threads, vpr);
    // The two buffers alternate: a warp writes buffer b for row i + 2 only after
    // row i + 1's barrier, which every warp reaches after it has read b for row i.
    finish_row<KMAX, false, Q8>(p, ss, z, gamma, s_sum[buf], s_max[buf], kConsumerBarrierId,
                                threads, lane, warp, t, vpr, row);
  }
}

// acc += w * (the eight bf16 values of q), as packed fp32x2 fmas (each two
// IEEE fmas, the same results as scalar ones). w = 1 is an addition.
__device__ __forceinline__ void fma8(const uint4 q, float w, float a[8]) {
  const uint32_t x[4] = {q.x, q.y, q.z, q.w};
  uint64_t w2;
  asm("mov.b64 %0, {%1, %1};" : "=l"(w2) : "f"(w));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint64_t acc, v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(acc) : "f"(a[2 * i]), "f"(a[2 * i + 1]));
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(x[i] << 16), "r"(x[i] & 0xffff0000u));
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(v), "l"(w2));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a[2 * i]), "=f"(a[2 * i + 1]) : "l"(acc));
  }
}

// VPT:   vectors of a thread per chunk. KMAX: per row.
// EXACT: the threads' vectors are the row, with none left over.
template <int KMAX, int VPT, bool EXACT, bool Q8>
__global__ void __launch_bounds__(kConsumerThreads + 32, 1)
    combine_ring_kernel(const __grid_constant__ CombineParams p) {
  extern __shared__ __align__(128) unsigned char ring[];
  __shared__ __align__(8) uint64_t full_bar[kMaxStages];
  __shared__ __align__(8) uint64_t empty_bar[kMaxStages];
  __shared__ __align__(16) float s_sum[2][kConsumerWarps];
  __shared__ __align__(16) float s_max[2][kConsumerWarps];
  __shared__ __align__(16) float s_weight[kConsumerWarps][32];  // by place in the row's order
  __shared__ int abort_flag;
  static_assert(KMAX % VPT == 0, "vectors must fill whole chunks");
  const int tid = threadIdx.x;
  const int lane = tid & 31;
  const int warp = tid >> 5;
  const int threads = p.threads;
  const int vpr = EXACT ? KMAX * threads : p.vec_per_row;
  const int chunk_vec = VPT * threads;
  const uint32_t chunk_bytes = static_cast<uint32_t>(chunk_vec) * 16u;
  const int chunks = EXACT ? KMAX / VPT : (vpr + chunk_vec - 1) / chunk_vec;
  const int stages = p.stages;
  const uint32_t stage_bytes = chunk_bytes * static_cast<uint32_t>(p.k + p.n + 1);
  const long long grid = gridDim.x;
  const long long row0 = static_cast<long long>(blockIdx.x) * p.tokens / grid;
  const long long row1 = static_cast<long long>(blockIdx.x + 1) * p.tokens / grid;
  if (tid < 2 * kConsumerWarps) {
    s_sum[tid / kConsumerWarps][tid % kConsumerWarps] = 0.0f;
    s_max[tid / kConsumerWarps][tid % kConsumerWarps] = 0.0f;
  }
  if (tid == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], static_cast<uint32_t>(threads / 32));
    }
    abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  // L2 warm-up before the dependency wait, a hint that reads nothing: the first
  // dense rows (which expert rows are needed is not known yet)
  if (tid >= threads && lane <= p.n && row1 > row0) {
    const uint4* src = (lane < p.n ? p.partials[lane] : p.residual) + row0 * vpr;
    const long long avail = (row1 - row0) * vpr * 16;
    prefetch_l2(src, static_cast<uint32_t>(avail < kPrefetchDense ? avail : kPrefetchDense));
  }
  grid_dependency_wait();
  grid_launch_dependents();
  volatile int* abort = &abort_flag;
  Slot next = load_slot(p, row0, lane);

  if (tid >= threads) {
    // ---------------- producer warp. Lane k < K copies slot k's expert row,
    // lane K + n partial n, lane K + N the residual (K + N + 1 <= 32).
    const uint64_t policy = p.l2_stream ? l2_evict_first_policy() : l2_evict_normal_policy();
    const int dense = lane - p.k;  // 0 .. N
    const uint4* dense_base = dense >= 0 && dense < p.n ? p.partials[dense] : p.residual;
    const bool is_dense = dense >= 0 && dense <= p.n;
    long long issued = 0;
    int s = 0;
    uint32_t round_parity = 0;
    bool first_pass = true, ok = true;
    for (long long row = row0; row < row1 && ok; ++row) {
      const Slot slot = next;
      if (row + 1 < row1) next = load_slot(p, row + 1, lane);
      const unsigned kept = kept_slots(p, slot, true);
      const int n_kept = __popc(kept);
      const bool mine = is_dense || ((kept >> lane) & 1u);
      const int place = is_dense ? n_kept + dense : __popc(kept & ((1u << lane) - 1u));
      const uint4* src = is_dense ? dense_base + row * vpr
                                  : p.experts + static_cast<long long>(mine ? slot.index : 0) * vpr;
      const uint32_t sources = static_cast<uint32_t>(n_kept + p.n + 1);
      for (int c = 0; c < chunks; ++c) {
        const int v0 = c * chunk_vec;
        const uint32_t bytes =
            EXACT ? chunk_bytes : static_cast<uint32_t>(min(chunk_vec, vpr - v0)) * 16u;
        int good = 1;
        if (lane == 0) {
          if (!first_pass) good = wait_phase(&empty_bar[s], round_parity ^ 1u, abort, 2u);
          if (good) mbar_arrive_expect_tx(&full_bar[s], bytes * sources);
        }
        ok = __shfl_sync(0xffffffffu, good, 0) != 0;
        if (!ok) break;
        if (mine)
          bulk_load(ring + static_cast<size_t>(s) * stage_bytes +
                        static_cast<uint32_t>(place) * chunk_bytes,
                    src + v0, bytes, &full_bar[s], policy);
        ++issued;
        if (++s == stages) {
          s = 0;
          round_parity ^= 1u;
          first_pass = false;
        }
      }
    }
    if (lane == 0) drain_ring(full_bar, stages, issued);
    return;
  }

  // ---------------- consumers
  const uint32_t base = smem_addr(ring) + static_cast<uint32_t>(tid) * 16u;
  // gamma for the CTA's whole range: in registers, or for long rows in shared
  // memory behind the ring (with the z of a long row the registers would spill,
  // and read again from L2 every row it cost 10% at H = 16384)
  constexpr bool kGammaRegs = KMAX <= 4;
  uint4 g_reg[kGammaRegs ? KMAX : 1];
  const uint4* s_gamma =
      reinterpret_cast<const uint4*>(ring + static_cast<size_t>(stages) * stage_bytes);
#pragma unroll
  for (int j = 0; j < KMAX; ++j) {
    const int v = j * threads + tid;
    const uint4 g = (EXACT || v < vpr) ? __ldg(p.gamma + v) : make_uint4(0, 0, 0, 0);
    if constexpr (kGammaRegs) g_reg[j] = g;
    else if (EXACT || v < vpr) const_cast<uint4*>(s_gamma)[v] = g;  // read by this thread only
  }
  auto gamma = [&](int j, int v) {
    if constexpr (kGammaRegs) return g_reg[j];
    else return s_gamma[v];
  };
  int s = 0;
  uint32_t parity = 0;
  float z[KMAX][8];
  for (long long row = row0; row < row1; ++row) {
    const Slot slot = next;
    if (row + 1 < row1) next = load_slot(p, row + 1, lane);
    const unsigned kept = kept_slots(p, slot, false);
    const int sources = __popc(kept) + p.n + 1;
    __syncwarp();  // the last row's weights have been read
    s_weight[warp][lane] = 1.0f;  // of the partials and the residual
    __syncwarp();
    if ((kept >> lane) & 1u) s_weight[warp][__popc(kept & ((1u << lane) - 1u))] = slot.weight;
    __syncwarp();
    uint4* res_row = p.residual + row * vpr;
    float ss = 0.0f;
#pragma unroll
    for (int c = 0; c < KMAX / VPT; ++c) {
      if (c < chunks) {
        wait_phase(&full_bar[s], parity, abort, 1u);
        const uint32_t at = base + static_cast<uint32_t>(s) * stage_bytes;
#pragma unroll
        for (int u = 0; u < VPT; ++u)
#pragma unroll
          for (int i = 0; i < 8; ++i) z[c * VPT + u][i] = -0.0f;  // -0 + x is x, -0 too
        // four sources at a time, then the one to three left
        int i = 0;
        for (; i + 3 < sources; i += 4) {
          const float4 w = *reinterpret_cast<const float4*>(&s_weight[warp][i]);
          const uint32_t from = at + static_cast<uint32_t>(i) * chunk_bytes;
#pragma unroll
          for (int u = 0; u < VPT; ++u) {
            if (EXACT || (c * VPT + u) * threads + tid < vpr) {
              float(&acc)[8] = z[c * VPT + u];
              const uint32_t v = from + static_cast<uint32_t>(u * threads) * 16u;
              const uint4 q0 = lds128(v), q1 = lds128(v + chunk_bytes);
              const uint4 q2 = lds128(v + 2 * chunk_bytes), q3 = lds128(v + 3 * chunk_bytes);
              fma8(q0, w.x, acc);
              fma8(q1, w.y, acc);
              fma8(q2, w.z, acc);
              fma8(q3, w.w, acc);
            }
          }
        }
        for (; i < sources; ++i) {
          const float w = s_weight[warp][i];
#pragma unroll
          for (int u = 0; u < VPT; ++u)
            if (EXACT || (c * VPT + u) * threads + tid < vpr)
              fma8(lds128(at + static_cast<uint32_t>(i) * chunk_bytes +
                          static_cast<uint32_t>(u * threads) * 16u),
                   w, z[c * VPT + u]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty_bar[s]);
#pragma unroll
        for (int u = 0; u < VPT; ++u) {
          const int j = c * VPT + u;
          const int v = j * threads + tid;
          if (EXACT || v < vpr) {
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(z[j][e], z[j][e], ss);
            res_row[v] = pack8(z[j]);
          }
        }
        if (++s == stages) {
          s = 0;
          parity ^= 1u;
        }
      }
    }
    finish_row<KMAX, EXACT, Q8>(p, ss, z, gamma, s_sum[row & 1], s_max[row & 1],
                                kConsumerBarrierId, threads, lane, warp, tid, vpr, row);
  }
}

using CombineFn = void (*)(CombineParams);
#define TW_COMBINE(Q) {combine_kernel<1, Q>, combine_kernel<2, Q>, combine_kernel<4, Q>, \
                       combine_kernel<8, Q>, combine_kernel<16, Q>}
const CombineFn kDirect[2][5] = {TW_COMBINE(false), TW_COMBINE(true)};
#undef TW_COMBINE
// Ring instances by vectors per row and per chunk.
#define TW_RING(E, Q) \
  {{combine_ring_kernel<1, 1, E, Q>, combine_ring_kernel<2, 1, E, Q>, combine_ring_kernel<4, 1, E, Q>, \
    combine_ring_kernel<8, 1, E, Q>, combine_ring_kernel<16, 1, E, Q>}, \
   {nullptr, combine_ring_kernel<2, 2, E, Q>, combine_ring_kernel<4, 2, E, Q>, \
    combine_ring_kernel<8, 2, E, Q>, combine_ring_kernel<16, 2, E, Q>}}
const CombineFn kRing[2][2][2][5] = {{TW_RING(false, false), TW_RING(true, false)},
                                     {TW_RING(false, true), TW_RING(true, true)}};
#undef TW_RING

// Registers per thread of a ring instance, queried once (0: not yet known, or
// the query failed). They are the same on every device.
std::atomic<int> g_ring_regs[2][2][2][5];

int ring_regs(int q8, int exact, int vpt2, int kc) {
  std::atomic<int>& known = g_ring_regs[q8][exact][vpt2][kc];
  int r = known.load(std::memory_order_relaxed);
  if (r == 0) {
    cudaFuncAttributes a;
    if (cudaFuncGetAttributes(&a, kRing[q8][exact][vpt2][kc]) != cudaSuccess) {
      cudaGetLastError();
      return 0;
    }
    r = a.numRegs;
    known.store(r, std::memory_order_relaxed);
  }
  return r;
}

constexpr int kMaxDevices = 64;

// Per device: SM count and shared memory, queried once, and which ring
// instances may use it (static storage, so the flags start false).
struct DeviceInfo {
  std::atomic<bool> ready;
  int sms;
  int l2_bytes;
  int regs_per_sm;
  int smem_optin;
  std::atomic<bool> attr_done[2][2][2][5];
};
DeviceInfo g_devices[kMaxDevices];
std::mutex g_mutex;

int device_info(DeviceInfo** out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return TW_ERR_CUDA;
  DeviceInfo& d = g_devices[dev];
  if (!d.ready.load(std::memory_order_acquire)) {
    std::lock_guard<std::mutex> lock(g_mutex);
    if (!d.ready.load(std::memory_order_relaxed)) {
      if (cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
          cudaDeviceGetAttribute(&d.l2_bytes, cudaDevAttrL2CacheSize, dev) != cudaSuccess ||
          cudaDeviceGetAttribute(&d.regs_per_sm, cudaDevAttrMaxRegistersPerMultiprocessor, dev) !=
              cudaSuccess ||
          cudaDeviceGetAttribute(&d.smem_optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) !=
              cudaSuccess)
        return TW_ERR_CUDA;
      d.ready.store(true, std::memory_order_release);
    }
  }
  *out = &d;
  return TW_OK;
}

}  // namespace

int launch_combine(const CombineArgs& a, cudaStream_t stream, int sm_budget) {
  DeviceInfo* d = nullptr;
  const int st = device_info(&d);
  if (st != TW_OK) return st;
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
  p.l2_stream = 0;
  p.eps = a.eps;
  p.hidden = static_cast<float>(a.hidden);
  int kc = 0;
  while ((kConsumerThreads << kc) < p.vec_per_row) ++kc;
  const int kmax = 1 << kc;
  p.threads = ((p.vec_per_row + kmax - 1) / kmax + 31) / 32 * 32;
  if (kmax >= 8 || (a.k == 0 && kmax > 1))  // a.k == 0: the fused step's layout
    p.threads = kConsumerThreads;
  const int q8 = a.scale_type >= 0 ? 1 : 0;
  int64_t grid = d->sms;
  if (sm_budget > 0 && sm_budget < grid) grid = sm_budget;
  const int exact = p.vec_per_row == kmax * p.threads ? 1 : 0;
  const int sources = a.k + a.n + 1;
  const int chunk = p.threads * 16;
  // Ring CTAs per SM: a CTA takes a row at a time, and with short rows its
  // consumers, not HBM, set the pace. As many as the registers hold with at
  // least kMinStages stages each, while each still has a row. An SM budget
  // means one per SM.
  const int gamma_bytes = kmax > 4 ? p.vec_per_row * 16 : 0;
  int share = sm_budget == 0 ? kMaxShare : 1, vpt2 = 0, stage = 0, stages = 0;
  for (; share >= 1; --share) {
    const int room = d->smem_optin / share - kStaticSmemReserve - gamma_bytes;
    // 8 KiB chunks where at least three stages of them fit
    vpt2 = kmax >= 2 && 3 * 2 * chunk * sources <= room ? 1 : 0;
    stage = chunk * (vpt2 + 1) * sources;
    stages = room / stage;
    if (share == 1) break;
    if (stages < kMinStages || a.tokens < share * grid) continue;
    // registers are given per warp, in units of 8 a thread, on four partitions
    const int regs = (ring_regs(q8, exact, vpt2, kc) + 7) / 8 * 8;
    const int warps = (share * (p.threads + 32) / 32 + 3) / 4;
    if (regs > 0 && warps * 32 * regs <= d->regs_per_sm / 4) break;
  }
  const int64_t ring_grid = grid * share;
  if (stages > kMaxStages) stages = kMaxStages;
  // one row per CTA stages that row and leaves the rest of the SM's shared
  // memory to the next launch's CTAs
  if (a.tokens <= ring_grid && stages > kmax >> vpt2) stages = kmax >> vpt2;
  p.stages = stages;
  // Evict-first loads and a streaming output while the output is at most a
  // quarter of the L2, normal loads above. Measured evict-first against
  // normal: T = 1024, H = 8192, K = 8 30.8 / 33.0 us, T = 512, H = 5120 12.3 /
  // 13.9; T = 8192, H = 8192, K = 8 240 / 227, T = 4096, H = 16384 164 / 156.
  p.l2_stream = a.tokens * a.hidden * (q8 ? 1 : 2) * 4 <= d->l2_bytes ? 1 : 0;
  CombineFn fn;
  cudaLaunchConfig_t cfg = {};
  if (stages >= 1 && sources <= 32) {
    fn = kRing[q8][exact][vpt2][kc];
    std::atomic<bool>& done = d->attr_done[q8][exact][vpt2][kc];
    if (!done.load(std::memory_order_acquire)) {
      std::lock_guard<std::mutex> lock(g_mutex);
      if (!done.load(std::memory_order_relaxed)) {
        if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 d->smem_optin - kStaticSmemReserve) !=
            cudaSuccess) {
          cudaGetLastError();
          return TW_ERR_CUDA;
        }
        done.store(true, std::memory_order_release);
      }
    }
    grid = ring_grid < a.tokens ? ring_grid : a.tokens;
    cfg.blockDim = dim3(static_cast<unsigned>(p.threads + 32));
    cfg.dynamicSmemBytes = static_cast<size_t>(stages) * stage + gamma_bytes;
  } else {
    fn = kDirect[q8][kc];
    if (sm_budget == 0) grid = kMaxGrid;
    if (grid > a.tokens) grid = a.tokens;
    cfg.blockDim = dim3(static_cast<unsigned>(p.threads));
  }
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
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

int read_combine_error(int reset, unsigned* code) { return read_ring_error(reset, code); }

}  // namespace tw
