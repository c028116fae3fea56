// fs_verify.cu -- fs_probs and fs_verify (fs_speculate.h): probabilities from logits,
// and the verification of drafted tokens against the target's.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <climits>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "fs_ptx.cuh"
#include "fs_speculate.h"

namespace fs {
int* device_error_word();  // fs_sample.cu

namespace verify {
namespace {

constexpr uint64_t kWaitLimitNs = 2000000000ull;  // 2 s
constexpr int kErrWaitTimeout = 1;                // the library's device error word, bit 0

__device__ __forceinline__ float wide(float x) { return x; }
__device__ __forceinline__ float wide(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void narrow(float* out, float x) { *out = x; }
__device__ __forceinline__ void narrow(__nv_bfloat16* out, float x) { *out = __float2bfloat16_rn(x); }

// ---------------------------------------------------------------------------
// Probabilities
// ---------------------------------------------------------------------------
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// exp((l - m) / T) for l <= m, to 2^-22 relative at any distance: l - m, and its
// product with log2(e) / T, are held in two floats, the exponent's whole part goes in
// as bits (Cody and Waite's reduction; an argument off by 2^-24 at most; the rest is the hardware's base-2 exponential).
// At T past 2^100, where c_lo falls among the subnormals, to 2^-20.  Below 2^-126 it is 0.
struct Exp {
  float m, c_hi, c_lo;  // the maximum, log2(e) / T
  __device__ __forceinline__ Exp(float max, float T) : m(max) {
    constexpr float kHi = 1.44269502f, kLo = 1.92596299e-8f;  // log2(e)
    const float t = fmaxf(T, 0x1p-126f);
    c_hi = __fdiv_rn(kHi, t);
    c_lo = __fdiv_rn(fmaf(-c_hi, t, kHi) + kLo, t);
  }
  __device__ __forceinline__ float operator()(float l) const {
    const float t = l - m;
    const float b = t - l;
    const float t_lo = (l - (t - b)) - (m + b);
    const float y = t * c_hi;
    if (y < -126.0f) return 0.0f;  // -inf too, whose t_lo is NaN
    const float n = rintf(y);
    const float f = fmaf(t, c_hi, -n) + fmaf(t, c_lo, t_lo * c_hi);
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(f));
    return e * __int_as_float((int(n) + 127) << 23);
  }
};

struct ProbsParams {
  const void* logits;
  int64_t ldl;
  const float* temperature;
  const uint32_t* mask;
  int64_t mask_ld;
  void* out;
  int64_t ldo;
  int32_t N, V;
  int32_t part;  // a CTA's elements of a row, a multiple of 32
  uint64_t wait_limit_ns;
  int* error_word;
};

// exp for a whole row in registers.  p = 2^(l c - K) / sum of the same for any K, so K is
// the whole number nearest m c, c = log2(e) / T in two floats: then l c - K - n, n a whole
// number too, is one rounding of a number of little over 1/2 (off by 2^-24), and 2^n goes into
// the exponent.  8 operations; where m c is too large for that, Exp.
struct FastExp {
  static constexpr float kMagic = 0x1.8p23f;  // adding it rounds to a whole number, in the low bits
  float at, c_hi, c_lo;                       // kMagic - K
  static __device__ __forceinline__ bool can(float m, float c_hi) { return fabsf(m * c_hi) < 0x1p22f; }
  __device__ __forceinline__ FastExp(float m, float hi, float lo)
      : at(kMagic - rintf(m * hi)), c_hi(hi), c_lo(lo) {}
  __device__ __forceinline__ float operator()(float l) const {
    const float r = fmaf(l, c_hi, at);  // kMagic + n
    const float f = fmaf(l, c_lo, fmaf(l, c_hi, at - r));
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(f));
    // 0 below 2^-126 (off by up to a third of that right above it), of -infinity too, whose f is NaN.
    return r < kMagic - 126.0f
               ? 0.0f
               : __uint_as_float(__float_as_uint(e) + (__float_as_uint(r) << 23));
  }
};

constexpr int kProbThreads = 512;
constexpr int kProbWarps = kProbThreads / 32;
constexpr int kMaxProbCluster = 16;  // more than 8 need the kernel's leave
constexpr int kMaxProbGroups = 8;
constexpr int kMaxPart = kMaxProbGroups * 4 * kProbThreads;  // a CTA's elements of a row

// Four elements at x, of which n exist, the others -infinity.
template <class T, bool kWhole>
__device__ __forceinline__ void load4(const T* x, int n, float (&l)[4]) {
  if (kWhole && n >= 4) {
    if constexpr (sizeof(T) == 2) {
      const uint2 w = *reinterpret_cast<const uint2*>(x);
      l[0] = __uint_as_float(w.x << 16), l[1] = __uint_as_float(w.x & 0xFFFF0000u);
      l[2] = __uint_as_float(w.y << 16), l[3] = __uint_as_float(w.y & 0xFFFF0000u);
    } else {
      const float4 w = *reinterpret_cast<const float4*>(x);
      l[0] = w.x, l[1] = w.y, l[2] = w.z, l[3] = w.w;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) l[i] = i < n ? wide(x[i]) : -INFINITY;
}
template <class TO, bool kWhole>
__device__ __forceinline__ void store4(TO* out, int n, const float (&p)[4]) {
  if (kWhole && n >= 4) {
    if constexpr (sizeof(TO) == 2) {
      const __nv_bfloat162 a = __floats2bfloat162_rn(p[0], p[1]), b = __floats2bfloat162_rn(p[2], p[3]);
      *reinterpret_cast<uint2*>(out) = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                                  *reinterpret_cast<const uint32_t*>(&b));
    } else {
      *reinterpret_cast<float4*>(out) = make_float4(p[0], p[1], p[2], p[3]);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < n) narrow(out + i, p[i]);
}

struct alignas(16) ProbsShared {
  // What the warps of a row's cluster tell one another: maxima; sums, or of a greedy row
  // the ids.  Slots that no warp has hold what changes nothing.
  uint32_t first[kMaxProbCluster * kProbWarps], second[kMaxProbCluster * kProbWarps];
  uint32_t mask[2][kMaxPart / 32];  // this row's and the next one's words
  uint64_t full;                    // the row's elements have arrived
  uint64_t told[2];                 // every CTA's word has
  uint32_t copies;                  // issued so far
  uint32_t gave_up;
};

// A barrier's phase has completed, or the wait's limit has passed: then the error word says
// so, and no later wait waits.
__device__ __forceinline__ void wait_for(const ProbsParams& p, ProbsShared& sm, uint64_t* bar,
                                         uint32_t phase) {
  if (ptx::mbar_try_wait(bar, phase)) return;
  const uint64_t t0 = ptx::global_timer_ns();
  while (!ptx::mbar_try_wait(bar, phase) && !*static_cast<volatile uint32_t*>(&sm.gave_up)) {
    if (ptx::global_timer_ns() - t0 > p.wait_limit_ns) {
      *static_cast<volatile uint32_t*>(&sm.gave_up) = 1u;
      atomicOr(p.error_word, kErrWaitTimeout);
    }
  }
}
// Behind a wait of this thread: whether it has ended well, and so the phase is complete.
__device__ __forceinline__ bool waited_well(ProbsShared& sm) {
  return !*static_cast<volatile uint32_t*>(&sm.gave_up);
}
// This warp's word into its slot in every CTA of the cluster, by stores that count on the
// receiver's barrier.  (A cluster's barrier would also wait for the stores of the row before.)
// A word of the next row cannot overtake: its sender has had this row's words from everyone.
// After a wait that ran out nothing is told, so that the others' waits run out too.
__device__ __forceinline__ void tell(uint32_t* slots, uint64_t* bar, int rank, int n_ctas,
                                     uint32_t v, bool well) {
  const uint32_t lane = threadIdx.x & 31;
  if (!well) return;
  if (threadIdx.x == 0) ptx::mbar_arrive_expect_tx(bar, uint32_t(n_ctas * kProbWarps) * 4u);
  if (int(lane) < n_ctas)
    asm volatile(
        "st.async.shared::cluster.mbarrier::complete_tx::bytes.u32 [%0], %1, [%2];" ::"r"(
            ptx::cluster_addr(slots + rank * kProbWarps + int(threadIdx.x >> 5), lane)),
        "r"(v), "r"(ptx::cluster_addr(bar, lane))
        : "memory");
}
// All slots in one, in a fixed order; the whole warp.
template <class Op>
__device__ __forceinline__ float of_slots(const uint32_t* slots, int n_ctas, Op op) {
  const int lane = int(threadIdx.x & 31);
  const uint4* at = reinterpret_cast<const uint4*>(slots) + lane;
  uint4 v = at[0];
  float r = op(op(__uint_as_float(v.x), __uint_as_float(v.y)),
               op(__uint_as_float(v.z), __uint_as_float(v.w)));
  if (n_ctas > 8) {
    v = at[32];
    r = op(r, op(op(__uint_as_float(v.x), __uint_as_float(v.y)),
                 op(__uint_as_float(v.z), __uint_as_float(v.w))));
  }
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) r = op(r, __shfl_xor_sync(0xFFFFFFFFu, r, s));
  return r;
}
// `bytes` (a multiple of 16) from global to shared memory, arriving on `bar`.
__device__ __forceinline__ void copy_async(void* to, const void* from, uint32_t bytes,
                                           uint64_t* bar) {
  ptx::mbar_arrive_expect_tx(bar, bytes);
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(ptx::smem_u32(to)),
      "l"(from), "r"(bytes), "r"(ptx::smem_u32(bar))
      : "memory");
}

// A row to a cluster of CTAs, kGroups times 4 elements a thread in registers: read once,
// written once.  Bound: memory.  The clusters stay for many rows: a row's elements are copied
// to shared memory while the row before is summed and written (without that a cluster's life
// was a chain of waits: 320 rows of 128256, masked, 139 us, now 57).  The maximum and the
// sum go through the cluster's shared memory, in the order of its CTAs.
// Rows of 128256 go 36 at a time (clusters of 8, two CTAs an SM): the first 36 take 11.2 us from
// masked bf16 to fp32, every 36 more 6.0 (their bytes 4.1), bf16 to bf16 without masks 8.7 and 4.4
// (2.7), fp32 to fp32 12.1 and 5.4 (5.4, bound by them).
// kAsync: rows on 16-byte boundaries; else they are read element by element and not ahead (320 rows
// of 50257 in bf16 57 us, 26 where they lie 50264 apart).
template <class T, class TO, bool kAsync, int kGroups>
__global__ void __launch_bounds__(kProbThreads, 2) probs_kernel(const ProbsParams p) {
  __shared__ ProbsShared sm;
  extern __shared__ __align__(16) uint8_t buffer_raw[];
  T* buffer = reinterpret_cast<T*>(buffer_raw);
  uint32_t n_ctas_u;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n_ctas_u));
  const int n_ctas = int(n_ctas_u);
  const int rank = int(ptx::cluster_ctarank());
  const int lane = threadIdx.x & 31;
  const int n_clusters = int(gridDim.x / n_ctas_u);
  const int begin = min(rank * p.part, p.V);
  const int n = min(p.part, p.V - begin);  // this CTA's elements
  constexpr int kWholeCopy = 16 / int(sizeof(T));
  const int copied = kAsync ? n / kWholeCopy * kWholeCopy : 0;
  const int words = (n + 31) / 32;
  if (threadIdx.x == 0) {
    ptx::mbar_init(&sm.full, 1);
    ptx::mbar_init(&sm.told[0], 1);
    ptx::mbar_init(&sm.told[1], 1);
    ptx::fence_barrier_init();
    sm.copies = sm.gave_up = 0u;
  }
  if (threadIdx.x < kMaxProbCluster * kProbWarps) {
    sm.first[threadIdx.x] = 0xFF800000u;  // -infinity
    sm.second[threadIdx.x] = 0u;
  }
  auto row_of = [&](int64_t row) { return static_cast<const T*>(p.logits) + row * p.ldl + begin; };
  auto mask_word = [&](int64_t row) {
    return int(threadIdx.x) < words ? p.mask[row * p.mask_ld + begin / 32 + threadIdx.x] : 0u;
  };
  ptx::grid_dependency_wait();  // the launch overlaps the kernel before it on the stream
  // The few elements behind the last whole 16 bytes come one by one, and behind them lies
  // -infinity.
  const int at_end = copied + int(threadIdx.x);
  auto copy_end = [&](const T* x) {
    if (kAsync && at_end < n) buffer[at_end] = x[at_end];
  };
  int64_t row = blockIdx.x / n_ctas_u;
  if (kAsync) {
    for (int i = n + int(threadIdx.x); i < kGroups * 4 * kProbThreads; i += kProbThreads)
      narrow(buffer + i, -INFINITY);
    copy_end(row_of(row));
  }
  if (p.mask) sm.mask[0][threadIdx.x] = mask_word(row);
  float temp = p.temperature ? p.temperature[row] : 1.0f;
  __syncthreads();
  auto copy_row = [&](int64_t row) {  // one thread
    copy_async(buffer, row_of(row), uint32_t(copied) * sizeof(T), &sm.full);
    ++sm.copies;
  };
  if (copied > 0 && threadIdx.x == 0) copy_row(row);
  ptx::cluster_sync();  // every CTA has started before another one writes its memory
  const int i0 = int(threadIdx.x) * 4;
  for (int turn = 0; row < p.N; ++turn) {
    const T* x = row_of(row);
    const int64_t next = row + n_clusters;
    const bool more = next < p.N;
    const uint32_t* mask = sm.mask[turn & 1];
    const bool greedy = !(temp > 0.0f && temp < INFINITY);
    const uint32_t phase = uint32_t(turn & 1);
    if (copied > 0) wait_for(p, sm, &sm.full, phase);
    float l[kGroups][4];
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const int i = i0 + g * kProbThreads * 4;
      if constexpr (kAsync)
        load4<T, true>(buffer + i, 4, l[g]);
      else
        load4<T, false>(x + i, n - i, l[g]);
    }
    if (p.mask) {
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        const int i = i0 + g * kProbThreads * 4;
        const uint32_t bits = mask[i >> 5] >> (i & 31);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (!(bits >> k & 1u)) l[g][k] = -INFINITY;
      }
    }
    float m = -INFINITY;
    if (greedy) {
#pragma unroll
      for (int g = 0; g < kGroups; ++g)
#pragma unroll
        for (int k = 0; k < 4; ++k) m = fmaxf(m, l[g][k]);  // of a number and NaN the number
    } else {
#pragma unroll
      for (int g = 0; g < kGroups; ++g)
#pragma unroll
        for (int k = 0; k < 4; ++k) m = max_nan(m, l[g][k]);
    }
    const bool well = waited_well(sm);
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, s));
    tell(sm.first, &sm.told[0], rank, n_ctas, __float_as_uint(m), well);
    __syncthreads();  // every thread has read the buffer
    if (more && copied > 0 && threadIdx.x == 0 && well) copy_row(next);
    if (more) copy_end(row_of(next));
    const uint32_t next_word = more && p.mask ? mask_word(next) : 0u;
    const float next_temp = more && p.temperature ? p.temperature[next] : 1.0f;
    Exp exact(0.0f, temp);
    wait_for(p, sm, &sm.told[0], phase);
    m = of_slots(sm.first, n_ctas, max_nan);
    TO* out = static_cast<TO*>(p.out) + row * p.ldo + begin;
    if (greedy) {
      int at = INT_MAX;
      if (m > -INFINITY) {
#pragma unroll
        for (int g = kGroups - 1; g >= 0; --g)
#pragma unroll
          for (int k = 3; k >= 0; --k)
            if (l[g][k] == m) at = begin + i0 + g * kProbThreads * 4 + k;
      }
      at = INT_MAX - __reduce_min_sync(0xFFFFFFFFu, at);
      sm.mask[phase ^ 1u][threadIdx.x] = next_word;
      tell(sm.second, &sm.told[1], rank, n_ctas, uint32_t(at), waited_well(sm));
      __syncthreads();
      wait_for(p, sm, &sm.told[1], phase);
      at = 0;
      for (int c = lane; c < n_ctas * kProbWarps; c += 32) at = max(at, int(sm.second[c]));
      at = INT_MAX - __reduce_max_sync(0xFFFFFFFFu, at);
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        const int i = i0 + g * kProbThreads * 4, v = begin + i;
        const float one[4] = {v == at ? 1.0f : 0.0f, v + 1 == at ? 1.0f : 0.0f,
                              v + 2 == at ? 1.0f : 0.0f, v + 3 == at ? 1.0f : 0.0f};
        store4<TO, kAsync>(out + i, n - i, one);
      }
    } else {
      float sum = 0.0f;
      if (m > -INFINITY && m < INFINITY) {
        exact.m = m;
        if (FastExp::can(m, exact.c_hi)) {
          const FastExp e(m, exact.c_hi, exact.c_lo);
#pragma unroll
          for (int g = 0; g < kGroups; ++g)
#pragma unroll
            for (int k = 0; k < 4; ++k) sum += l[g][k] = e(l[g][k]);
        } else {
#pragma unroll
          for (int g = 0; g < kGroups; ++g)
#pragma unroll
            for (int k = 0; k < 4; ++k) sum += l[g][k] = exact(l[g][k]);
        }
      } else {
        // No allowed id: all 0.  A NaN or +inf among them: all of them NaN.
        const float nan = __int_as_float(0x7FFFFFFF);
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
          const int i = i0 + g * kProbThreads * 4;
          const uint32_t bits = !p.mask ? 15u : mask[i >> 5] >> (i & 31);
#pragma unroll
          for (int k = 0; k < 4; ++k) l[g][k] = m == -INFINITY || !(bits >> k & 1u) ? 0.0f : nan;
        }
        sum = 1.0f;
      }
      const bool well = waited_well(sm);
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, s);
      sm.mask[phase ^ 1u][threadIdx.x] = next_word;
      tell(sm.second, &sm.told[1], rank, n_ctas, __float_as_uint(sum), well);
      __syncthreads();
      wait_for(p, sm, &sm.told[1], phase);
      sum = of_slots(sm.second, n_ctas, [](float a, float b) { return a + b; });
      const float inv = __fdiv_rn(1.0f, sum);
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        const int i = i0 + g * kProbThreads * 4;
#pragma unroll
        for (int k = 0; k < 4; ++k) l[g][k] *= inv;
        store4<TO, kAsync>(out + i, n - i, l[g]);
      }
    }
    row = next;
    temp = next_temp;
  }
  // After a wait that ran out a copy may be on its way, and the others may still store here: this
  // CTA ends behind them (the barrier is of those that have not ended).
  __syncthreads();
  if (sm.gave_up) {
    if (threadIdx.x == 0 && sm.copies > 0) {
      const uint64_t t0 = ptx::global_timer_ns();
      while (!ptx::mbar_try_wait(&sm.full, (sm.copies - 1u) & 1u) &&
             ptx::global_timer_ns() - t0 <= p.wait_limit_ns) {
      }
    }
    ptx::cluster_sync();
  }
}

// Rows longer than a cluster's registers: one CTA, three passes, the later two mostly from L2.
// Slow for few rows: 5 rows of 262208 take 260 us (of 262144, in a cluster, 7), 320 600 (135), less
// than a tenth of the copy rate; the largest vocabulary in use here has 262144 ids.
template <class T, class TO>
__global__ void __launch_bounds__(kProbThreads) long_probs_kernel(const ProbsParams p) {
  __shared__ float s_val[kProbThreads / 32];
  __shared__ int s_idx[kProbThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(p.logits) + row * p.ldl;
  TO* out = static_cast<TO*>(p.out) + row * p.ldo;
  const uint32_t* mask = p.mask ? p.mask + row * p.mask_ld : nullptr;
  const float temp = p.temperature ? p.temperature[row] : 1.0f;
  const bool greedy = !(temp > 0.0f && temp < INFINITY);
  auto allowed = [&](int v) { return mask == nullptr || (mask[v >> 5] >> (v & 31) & 1u) != 0u; };

  float m = -INFINITY;
  int at = INT_MAX;
  for (int v = threadIdx.x; v < p.V; v += kProbThreads) {
    if (!allowed(v)) continue;
    const float l = wide(x[v]);
    if (greedy) {
      if (l > m) m = l, at = v;
    } else {
      m = max_nan(m, l);
    }
  }
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) {
    const float om = __shfl_xor_sync(0xFFFFFFFFu, m, s);
    const int oa = __shfl_xor_sync(0xFFFFFFFFu, at, s);
    if (greedy) {
      if (om > m || (om == m && oa < at)) m = om, at = oa;
    } else {
      m = max_nan(m, om);
    }
  }
  if (lane == 0) s_val[warp] = m, s_idx[warp] = at;
  __syncthreads();
  m = s_val[0], at = s_idx[0];
  for (int w = 1; w < kProbThreads / 32; ++w) {
    if (greedy) {
      if (s_val[w] > m || (s_val[w] == m && s_idx[w] < at)) m = s_val[w], at = s_idx[w];
    } else {
      m = max_nan(m, s_val[w]);
    }
  }
  if (greedy || m == -INFINITY) {
    __syncthreads();
    for (int v = threadIdx.x; v < p.V; v += kProbThreads)
      narrow(out + v, greedy && v == at ? 1.0f : 0.0f);
    return;
  }
  const Exp exact(m, temp);
  // Where l - m may be past the largest number and T is not far below it, FastExp, which makes
  // no difference of the two.
  const FastExp fast(m, exact.c_hi, exact.c_lo);
  const bool far = -FLT_MAX - m == -INFINITY && FastExp::can(m, exact.c_hi);
  auto e = [&](float l) { return far ? fast(l) : exact(l); };
  float sum = 0.0f;
  for (int v = threadIdx.x; v < p.V; v += kProbThreads)
    if (allowed(v)) sum += e(wide(x[v]));
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, s);
  __syncthreads();
  if (lane == 0) s_val[warp] = sum;
  __syncthreads();
  sum = 0.0f;
  for (int w = 0; w < kProbThreads / 32; ++w) sum += s_val[w];
  const float inv = __fdiv_rn(1.0f, sum);
  for (int v = threadIdx.x; v < p.V; v += kProbThreads)
    narrow(out + v, allowed(v) ? e(wide(x[v])) * inv : 0.0f);
}

// ---------------------------------------------------------------------------
// Verification
// ---------------------------------------------------------------------------
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kSegment = 1024;      // elements of a segment, doubled until there are
constexpr int kMaxSegments = 1024;  // at most so many
constexpr int kMaxCluster = 16;     // more than 8 need the kernel's leave

struct VerifyParams {
  const void* p;
  const void* q;
  const int64_t* ids;
  const float* u;
  int64_t p_seq, p_pos, q_seq, q_pos, ld_ids, ldu;
  int64_t* out_ids;
  int64_t ld_out;
  int64_t* accepted;
  int32_t K, V;
  int32_t segment, n_segments;
  uint64_t wait_limit_ns;
  int* error_word;
};

// A sum in two floats, the second at most half the last place of the first (Knuth's two-sum): to
// 2^-46 or so of the total.  (64-bit arithmetic is slow on this GPU: a scan by 16 warps in it took as
// long as reading the row.)
struct Sum {
  float hi = 0.0f, lo = 0.0f;
  // A term; `lo` is only gathered, for normal() after a few dozen at most.
  __device__ __forceinline__ void add(float w) {
    const float s = hi + w;
    const float b = s - hi;
    lo += (hi - (s - b)) + (w - b);
    hi = s;
  }
  __device__ __forceinline__ Sum normal() const {
    Sum r;
    r.hi = hi + lo;
    r.lo = lo - (r.hi - hi);
    return r;
  }
  __device__ __forceinline__ Sum operator+(const Sum& o) const {
    Sum r = *this;
    r.add(o.hi);
    r.lo += o.lo;
    return r.normal();
  }
  __device__ __forceinline__ bool operator>(const Sum& o) const {
    return hi > o.hi || (hi == o.hi && lo > o.lo);
  }
  __device__ __forceinline__ Sum operator*(float u) const {
    Sum r;
    r.hi = hi * u;
    r.lo = fmaf(lo, u, fmaf(hi, u, -r.hi));
    return r.normal();
  }
};
__device__ __forceinline__ Sum shfl_xor(const Sum& v, int d) {
  Sum r;
  r.hi = __shfl_xor_sync(0xFFFFFFFFu, v.hi, d);
  r.lo = __shfl_xor_sync(0xFFFFFFFFu, v.lo, d);
  return r;
}
// The sum of the lanes up to and with this one.
__device__ __forceinline__ Sum scan(Sum v, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    Sum o;
    o.hi = __shfl_up_sync(0xFFFFFFFFu, v.hi, d);
    o.lo = __shfl_up_sync(0xFFFFFFFFu, v.lo, d);
    if (lane >= d) v = o + v;
  }
  return v;
}
// The sum before it, given that.
__device__ __forceinline__ Sum exclusive(const Sum& inclusive, int lane) {
  Sum r;
  r.hi = __shfl_up_sync(0xFFFFFFFFu, inclusive.hi, 1);
  r.lo = __shfl_up_sync(0xFFFFFFFFu, inclusive.lo, 1);
  if (lane == 0) r = Sum();
  return r;
}

enum Mode { kTarget = 0, kResidual = 1, kWithout = 2 };

// Negative, infinite and NaN weights are 0.
__device__ __forceinline__ float weight(float w) {
  w = fmaxf(w, 0.0f);
  return w < INFINITY ? w : 0.0f;
}

// The weights that a sequence's last token is drawn with.
template <class T>
struct Weights {
  const T* p;
  const T* q;
  int mode, without;
  __device__ __forceinline__ float at(int v) const {
    if (mode == kWithout && v == without) return 0.0f;
    return weight(mode == kResidual ? wide(p[v]) - wide(q[v]) : wide(p[v]));
  }
};

template <class T>
__device__ __forceinline__ void unpack(const uint4& v, float (&x)[16 / sizeof(T)]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 2) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    } else {
      x[i] = __uint_as_float(w[i]);
    }
  }
}

// A warp's sum of a segment, 1024 elements at a time.  Every lane takes runs of 16 bytes, 32
// runs side by side, in the same order however they are read: 16 bytes at a time where rows allow
// it, four runs of each row in flight.  What a lane's 32 terms lose is gathered, no more: after
// 65536 terms (a segment of the longest rows) it would itself be off, by 2^-23 of a sum of equal
// weights.
constexpr int kTerms = 32;
template <class T, bool kTwo>
__device__ __forceinline__ Sum whole_piece(const T* p, const T* q, int lane) {
  constexpr int kRun = 16 / int(sizeof(T));
  const uint4* pv = reinterpret_cast<const uint4*>(p) + lane;
  const uint4* qv = reinterpret_cast<const uint4*>(q) + lane;
  Sum s;
  for (int j = 0; j < kSegment / (32 * kRun); j += 4) {
    uint4 a[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = __ldcs(pv + 32 * (j + i));
    if (kTwo) {
#pragma unroll
      for (int i = 0; i < 4; ++i) b[i] = __ldcs(qv + 32 * (j + i));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float x[kRun], y[kRun];
      unpack<T>(a[i], x);
      if (kTwo) unpack<T>(b[i], y);
#pragma unroll
      for (int k = 0; k < kRun; ++k) s.add(weight(kTwo ? x[k] - y[k] : x[k]));
    }
  }
  return s.normal();
}
template <class T, bool kTwo>
__device__ __forceinline__ Sum whole_segment(const T* p, const T* q, int segment, int lane) {
  static_assert(kSegment == 32 * kTerms, "terms of a lane");
  Sum s = whole_piece<T, kTwo>(p, q, lane);
  for (int v = kSegment; v < segment; v += kSegment)
    s = s + whole_piece<T, kTwo>(p + v, kTwo ? q + v : q, lane);
  return s;
}
template <class T>
__device__ __forceinline__ Sum segment_sum(const Weights<T>& w, int begin, int length, int segment,
                                           bool vec, int lane) {
  constexpr int kRun = 16 / int(sizeof(T));
  Sum s;
  if (vec && length == segment &&
      !(w.mode == kWithout && w.without >= begin && w.without - begin < length)) {
    s = w.mode == kResidual ? whole_segment<T, true>(w.p + begin, w.q + begin, segment, lane)
                            : whole_segment<T, false>(w.p + begin, nullptr, segment, lane);
  } else {
    auto add_up = [&](int at, int end) {
      Sum piece;
      for (int v0 = at + lane * kRun; v0 < end; v0 += 32 * kRun) {
#pragma unroll
        for (int i = 0; i < kRun; ++i)
          if (v0 + i < end) piece.add(w.at(begin + v0 + i));
      }
      return piece.normal();
    };
    s = add_up(0, min(length, kSegment));
    for (int at = kSegment; at < length; at += kSegment)
      s = s + add_up(at, min(length, at + kSegment));
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) s = s + shfl_xor(s, d);
  return s;
}

struct alignas(16) Shared {
  Sum sums[kMaxSegments];
  Sum warps[kWarps];
  Sum before;  // sum of the segments before the chosen one
  Sum target;
  uint64_t arrived;  // the segments' sums have
  int accepted, mode, without;
  int segment, first, last, found;
  int gave_up;
};

// The segments' sums are there, or (false) the wait's limit has passed: then the error word
// says so.  One warp.
__device__ __forceinline__ bool wait_arrived(const VerifyParams& a, Shared& sm) {
  bool there = ptx::mbar_try_wait(&sm.arrived, 0);
  if (!there) {
    const uint64_t t0 = ptx::global_timer_ns();
    while (!(there = ptx::mbar_try_wait(&sm.arrived, 0))) {
      if (ptx::global_timer_ns() - t0 > a.wait_limit_ns) {
        atomicOr(a.error_word, kErrWaitTimeout);
        break;
      }
    }
  }
  return __all_sync(0xFFFFFFFFu, there);
}

// How many drafts pass, and what the next token is drawn from.  One warp.
template <class T>
__device__ __forceinline__ void accept(const VerifyParams& a, int64_t b, Shared& sm, int lane) {
  int n = 0;
  bool rejected = false;
  int without = -1;
  for (int i0 = 0; i0 < a.K; i0 += 32) {
    const int i = i0 + lane;
    bool pass = false, none = true;
    int x32 = -1;
    if (i < a.K) {
      const int64_t x = a.ids[b * a.ld_ids + i];
      const float u = a.u[b * a.ldu + i];
      none = x < 0;
      if (x >= 0 && x < a.V) {
        x32 = int(x);
        const float uc = u > 0.0f ? fminf(u, 0x1.fffffep-1f) : 0.0f;
        const float px = wide(static_cast<const T*>(a.p)[b * a.p_seq + i * a.p_pos + x]);
        const float qx =
            a.q ? wide(static_cast<const T*>(a.q)[b * a.q_seq + i * a.q_pos + x]) : 1.0f;
        pass = double(uc) * double(qx) < double(px);
      }
    }
    const uint32_t stop = __ballot_sync(0xFFFFFFFFu, !pass);
    if (stop != 0u) {
      const int at = __ffs(stop) - 1;
      n = i0 + at;  // K where the lanes past the last draft stop
      rejected = !__shfl_sync(0xFFFFFFFFu, int(none), at);
      without = __shfl_sync(0xFFFFFFFFu, x32, at);
      break;
    }
    n = i0 + 32;
  }
  if (lane == 0) {
    sm.accepted = n;
    sm.mode = !rejected ? kTarget : a.q ? kResidual : kWithout;
    sm.without = without;
  }
}

// The segment in which the sums pass u times their total; false if all are 0.  One warp.
__device__ __forceinline__ bool find_segment(const VerifyParams& a, float u, Shared& sm,
                                             int lane) {
  const int per = (a.n_segments + 31) / 32;
  const int s0 = min(lane * per, a.n_segments), s1 = min(s0 + per, a.n_segments);
  Sum own;
  for (int s = s0; s < s1; ++s) own = own + sm.sums[s];
  const Sum upto = scan(own, lane), ahead = exclusive(upto, lane);
  Sum total;
  total.hi = __shfl_sync(0xFFFFFFFFu, upto.hi, 31);
  total.lo = __shfl_sync(0xFFFFFFFFu, upto.lo, 31);
  const uint32_t some = __ballot_sync(0xFFFFFFFFu, own.hi > 0.0f);
  if (some == 0u) return false;
  const Sum target = total * (u > 0.0f ? fminf(u, 0x1.fffffep-1f) : 0.0f);
  const uint32_t past = __ballot_sync(0xFFFFFFFFu, own.hi > 0.0f && upto > target);
  // Past every sum (by their rounding): the last one that is not 0.
  const int at = past != 0u ? __ffs(past) - 1 : 31 - __clz(some);
  if (lane == at) {
    Sum before = ahead, run = ahead;
    int chosen = s0;
    for (int s = s0; s < s1; ++s) {
      const Sum x = sm.sums[s];
      if (!(x.hi > 0.0f)) continue;
      before = run;
      run = run + x;
      chosen = s;
      if (run > target) break;
    }
    sm.segment = chosen;
    sm.before = before;
    sm.target = target;
    sm.first = INT_MAX;
    sm.last = -1;
  }
  return true;
}

// The first element of the chosen segment whose sum passes the target.  All threads.
template <class T>
__device__ __forceinline__ int find_element(const VerifyParams& a, const Weights<T>& w, Shared& sm) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = a.segment / kThreads;
  const int v0 = sm.segment * a.segment + int(threadIdx.x) * per;
  const int v1 = v0 < a.V ? v0 + min(per, a.V - v0) : v0;
  // kTerms at a time, as in a segment's sum; mostly there are 2 in all.
  int last = -1;
  auto add_up = [&](int from, int to) {
    Sum t;
    for (int v = from; v < to; ++v) {
      const float x = w.at(v);
      t.add(x);
      if (x > 0.0f) last = v;
    }
    return t.normal();
  };
  Sum own;
  if (per <= kTerms) {
    own = add_up(v0, v1);
  } else {
    for (int at = v0; at < v1; at += kTerms) own = own + add_up(at, min(v1, at + kTerms));
  }
  const Sum upto = scan(own, lane);
  if (lane == 31) sm.warps[warp] = upto;
  __syncthreads();
  const Sum warps = scan(lane < kWarps ? sm.warps[lane] : Sum(), lane);
  Sum ahead;  // of the warps before this one
  ahead.hi = __shfl_sync(0xFFFFFFFFu, warps.hi, max(warp - 1, 0));
  ahead.lo = __shfl_sync(0xFFFFFFFFu, warps.lo, max(warp - 1, 0));
  if (warp == 0) ahead = Sum();
  ahead = sm.before + ahead;
  // Only lanes where the target may be passed look again; the lowest counts.
  const uint32_t past = __ballot_sync(0xFFFFFFFFu, last >= 0 && ahead + upto > sm.target);
  const Sum base = ahead + exclusive(upto, lane);
  if (past != 0u && lane == __ffs(past) - 1) {
    int first = last;
    auto search = [&](Sum run, int from, int to) {
      for (int v = from; v < to; ++v) {
        const float x = w.at(v);
        if (!(x > 0.0f)) continue;
        Sum term;
        term.hi = x;
        run = run + term;
        if (run > sm.target) {
          first = v;
          return true;
        }
      }
      return false;
    };
    if (per <= kTerms) {
      search(base, v0, v1);
    } else {
      Sum done;  // of the terms before
      for (int at = v0; at < v1 && !search(base + done, at, min(v1, at + kTerms)); at += kTerms)
        done = done + add_up(at, min(v1, at + kTerms));
    }
    atomicMin(&sm.first, first);
  }
  last = __reduce_max_sync(0xFFFFFFFFu, last);
  if (lane == 0) atomicMax(&sm.last, last);
  __syncthreads();
  return sm.first != INT_MAX ? sm.first : sm.last;
}

// The token drawn with the weights w, once the segments' sums have arrived; -1 if all of them
// are 0.  After a wait that ran out it is -1 too: what lies in the sums' places is not looked at,
// and not written either, since others may still store there.  All threads.
template <class T>
__device__ __forceinline__ int draw(const VerifyParams& a, Weights<T>& w, float u, bool vec,
                                    Shared& sm) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (warp == 0) {
    const bool there = wait_arrived(a, sm);
    const bool some = there && find_segment(a, u, sm, lane);
    if (lane == 0) sm.found = some, sm.gave_up = !there;
  }
  __syncthreads();
  if (!sm.found && !sm.gave_up && w.mode != kTarget) {
    // Nothing is left of p after a rejection: the draw is from p.
    w.mode = kTarget;
    for (int s = warp; s < a.n_segments; s += kWarps) {
      const int begin = s * a.segment;
      const Sum t = segment_sum(w, begin, min(a.segment, a.V - begin), a.segment, vec, lane);
      if (lane == 0) sm.sums[s] = t;
    }
    __syncthreads();
    if (warp == 0) {
      const bool some = find_segment(a, u, sm, lane);
      if (lane == 0) sm.found = some;
    }
    __syncthreads();
  }
  return sm.found ? find_element(a, w, sm) : -1;
}

// A sequence to a cluster of CTAs.  Each finds out which drafts pass (that is 2 dependent reads,
// and less than telling one another); the row's segments go around their warps; the first CTA
// gathers the segments' sums, finds the segment that u falls into and sums that again, element
// by element.  Bound: memory for large batches, for small ones the chain of those reads.
template <class T>
__global__ void __launch_bounds__(kThreads, 2) verify_kernel(const VerifyParams a) {
  __shared__ Shared sm;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t n_ctas;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n_ctas));
  const int rank = int(ptx::cluster_ctarank());
  const int64_t b = blockIdx.x / n_ctas;
  if (threadIdx.x == 0) {
    ptx::mbar_init(&sm.arrived, 1);
    ptx::fence_barrier_init();
    if (rank == 0) ptx::mbar_arrive_expect_tx(&sm.arrived, uint32_t(a.n_segments) * 8u);
  }
  ptx::cluster_arrive();
  ptx::grid_dependency_wait();  // the launch overlaps the kernel before it on the stream
  if (warp == 0) accept<T>(a, b, sm, lane);
  const float u = a.u[b * a.ldu + a.K];
  __syncthreads();
  const int n = sm.accepted;
  Weights<T> w;
  w.p = static_cast<const T*>(a.p) + b * a.p_seq + n * a.p_pos;
  w.mode = sm.mode;
  w.without = sm.without;
  w.q = w.mode == kResidual ? static_cast<const T*>(a.q) + b * a.q_seq + n * a.q_pos : nullptr;
  const bool vec =
      ((reinterpret_cast<uintptr_t>(w.p) | reinterpret_cast<uintptr_t>(w.q)) & 15) == 0;
  ptx::cluster_wait();  // the first CTA's barrier is there
  const uint32_t sums0 = ptx::cluster_addr(sm.sums, 0), arrived0 = ptx::cluster_addr(&sm.arrived, 0);
  for (int s = rank * kWarps + warp; s < a.n_segments; s += int(n_ctas) * kWarps) {
    const int begin = s * a.segment;
    const Sum t = segment_sum(w, begin, min(a.segment, a.V - begin), a.segment, vec, lane);
    if (lane == 0)
      asm volatile(
          "st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(
              sums0 + uint32_t(s) * 8u),
          "f"(t.hi), "f"(t.lo), "r"(arrived0)
          : "memory");
  }
  if (rank != 0) return;
  const int drawn = draw(a, w, u, vec, sm);
  for (int i = threadIdx.x; i <= a.K; i += kThreads)
    a.out_ids[b * a.ld_out + i] = i < n ? a.ids[b * a.ld_ids + i] : i == n ? int64_t(drawn) : -1;
  if (threadIdx.x == 0 && a.accepted) a.accepted[b] = n;
  // After a wait that ran out the others may still store here: this CTA ends behind them
  // (the barrier is of those that have not ended) and their stores.
  if (sm.gave_up) {
    ptx::cluster_sync();
    if (warp == 0) wait_arrived(a, sm);
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
constexpr int kMaxDevices = 64;
std::mutex g_mu;
struct Device {
  bool known = false;
  fs_status status = FS_ERR_UNSUPPORTED;
  int sms = 0;
  bool wide_clusters = false;  // of kMaxCluster CTAs fit
  int* error_word = nullptr;
};
Device g_devices[kMaxDevices];

// Whether clusters of kMaxCluster CTAs of a verification kernel can run here at all.
bool wide_clusters_fit(void (*kernel)(VerifyParams)) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = kMaxCluster;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kMaxCluster);
  cfg.blockDim = dim3(kThreads);
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int n = 0;
  const bool fit =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) ==
          cudaSuccess &&
      cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess && n >= 1;
  cudaGetLastError();
  return fit;
}

// The current device, if it is a GB300 (sm_103).
fs_status device_setup(const Device** out) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
    cudaGetLastError();
    return FS_ERR_UNSUPPORTED;
  }
  std::lock_guard<std::mutex> lock(g_mu);
  Device& d = g_devices[dev];
  if (!d.known) {
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
      cudaGetLastError();
      return FS_ERR_CUDA;
    }
    d.status = FS_ERR_UNSUPPORTED;
    if (major == 10 && minor == 3) {
      d.error_word = device_error_word();
      d.wide_clusters = wide_clusters_fit(verify_kernel<float>) &&
                        wide_clusters_fit(verify_kernel<__nv_bfloat16>);
      const bool ok = d.error_word != nullptr;
      cudaGetLastError();
      d.status = ok ? FS_OK : FS_ERR_CUDA;
    }
    d.known = true;
  }
  *out = &d;
  return d.status;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
uintptr_t element(int dtype) { return dtype == FS_F32 ? 4 : 2; }
bool known(int dtype) { return dtype == FS_BF16 || dtype == FS_F32; }
constexpr int64_t kMostV = INT_MAX - 65536;  // a segment's end fits 32 bits

template <class T, class TO, bool kAsync, int kGroups>
cudaError_t launch_probs(ProbsParams p, int ctas, cudaStream_t stream) {
  auto kernel = probs_kernel<T, TO, kAsync, kGroups>;
  // How many clusters fit, once for each kernel, device and size of cluster.
  static std::mutex mu;
  static int fit[kMaxDevices][kMaxProbCluster + 1];
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(ctas);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kProbThreads);
  cfg.gridDim = dim3(unsigned(ctas));
  cfg.dynamicSmemBytes = kAsync ? kGroups * 4 * kProbThreads * sizeof(T) : 0;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int clusters;
  {
    std::lock_guard<std::mutex> lock(mu);
    int& f = fit[dev][ctas];
    if (f == 0) {
      if (kAsync)
        err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   int(cfg.dynamicSmemBytes));
      if (err == cudaSuccess && ctas > 8)
        err = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      int n = 0;
      if (err == cudaSuccess) err = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
      if (err != cudaSuccess) return err;
      if (n < 1) return cudaErrorInvalidConfiguration;
      f = n;
    }
    clusters = f;
  }
  // No more than the rows need in as many turns.
  const int64_t turns = ceil_div(p.N, clusters);
  cfg.gridDim = dim3(unsigned(ceil_div(p.N, turns) * ctas));
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <class T, class TO>
cudaError_t launch_probs(ProbsParams p, cudaStream_t stream) {
  // CTAs of a row's cluster by V alone, so that a row's sum does not depend on what else is
  // computed: as few as hold it, of any number, since a row's chain of waits costs each CTA
  // the same (320 rows of 151936 in fp32: 10 CTAs 72 us, 16 of 19 elements a thread 98; 1000 of
  // 40000: 3 CTAs 60, 8 88); two where that makes a single row faster (16000: 7.8 and 9.7).
  const int ctas = int(std::max<int64_t>(std::min<int64_t>(kMaxProbCluster, ceil_div(p.V, kMaxPart)),
                                         p.V > kMaxPart / 2 ? 2 : 1));
  const int64_t part = ceil_div(ceil_div(p.V, ctas), 32) * 32;
  if (part > kMaxPart) {
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kProbThreads);
    cfg.gridDim = dim3(unsigned(p.N));
    cfg.stream = stream;
    return cudaLaunchKernelEx(&cfg, long_probs_kernel<T, TO>, p);
  }
  p.part = int32_t(part);
  const bool whole = aligned(p.logits, 16) && p.ldl * sizeof(T) % 16 == 0 && aligned(p.out, 16) &&
                     p.ldo * sizeof(TO) % 16 == 0;
  const int64_t per = ceil_div(part, kProbThreads * 4);
  if (per <= 1)
    return whole ? launch_probs<T, TO, true, 1>(p, ctas, stream)
                 : launch_probs<T, TO, false, 1>(p, ctas, stream);
  if (per <= 2)
    return whole ? launch_probs<T, TO, true, 2>(p, ctas, stream)
                 : launch_probs<T, TO, false, 2>(p, ctas, stream);
  if (per <= 4)
    return whole ? launch_probs<T, TO, true, 4>(p, ctas, stream)
                 : launch_probs<T, TO, false, 4>(p, ctas, stream);
  if (per <= 6)
    return whole ? launch_probs<T, TO, true, 6>(p, ctas, stream)
                 : launch_probs<T, TO, false, 6>(p, ctas, stream);
  return whole ? launch_probs<T, TO, true, 8>(p, ctas, stream)
               : launch_probs<T, TO, false, 8>(p, ctas, stream);
}

}  // namespace
}  // namespace verify
}  // namespace fs

using namespace fs::verify;

extern "C" fs_status fs_probs(const fs_probs_args* args, void* stream_ptr) {
  if (!args) return FS_ERR_INVALID_ARG;
  const fs_probs_args& a = *args;
  // (A long row is a CTA; of the others' grid there are never more CTAs than fit at once.)
  if (a.N < 0 || a.N >= (1 << 28) || a.V < 1 || a.V > kMostV || !known(a.dtype) ||
      !known(a.out_dtype))
    return FS_ERR_INVALID_ARG;
  if (a.N == 0) return FS_OK;
  if (a.N > 1 && (a.ldl < a.V || a.ldo < a.V || (a.vocab_mask && a.mask_ld < ceil_div(a.V, 32))))
    return FS_ERR_INVALID_ARG;
  if (!a.logits || !a.out || !aligned(a.logits, element(a.dtype)) ||
      !aligned(a.out, element(a.out_dtype)) || !aligned(a.temperature, 4) ||
      !aligned(a.vocab_mask, 4))
    return FS_ERR_INVALID_ARG;
  if (a.out == a.logits && (a.dtype != a.out_dtype || (a.N > 1 && a.ldl != a.ldo)))
    return FS_ERR_INVALID_ARG;
  const Device* dev = nullptr;
  const fs_status st = device_setup(&dev);
  if (st != FS_OK) return st;
  ProbsParams p = {};
  p.logits = a.logits;
  p.ldl = a.N > 1 ? a.ldl : 0;
  p.temperature = a.temperature;
  p.mask = a.vocab_mask;
  p.mask_ld = a.mask_ld;
  p.out = a.out;
  p.ldo = a.N > 1 ? a.ldo : 0;
  p.N = int32_t(a.N);
  p.V = int32_t(a.V);
  p.wait_limit_ns = kWaitLimitNs;
  p.error_word = dev->error_word;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  const cudaError_t err =
      a.dtype == FS_F32
          ? (a.out_dtype == FS_F32 ? launch_probs<float, float>(p, stream)
                                   : launch_probs<float, __nv_bfloat16>(p, stream))
          : (a.out_dtype == FS_F32 ? launch_probs<__nv_bfloat16, float>(p, stream)
                                   : launch_probs<__nv_bfloat16, __nv_bfloat16>(p, stream));
  if (err != cudaSuccess) {
    cudaGetLastError();
    return FS_ERR_CUDA;
  }
  return FS_OK;
}

extern "C" fs_status fs_verify(const fs_verify_args* args, void* stream_ptr) {
  if (!args) return FS_ERR_INVALID_ARG;
  const fs_verify_args& a = *args;
  if (a.B < 0 || a.B >= (1 << 24) || a.K < 0 || a.K > FS_VERIFY_DRAFTS_MAX || a.V < 1 ||
      a.V > kMostV || !known(a.dtype))
    return FS_ERR_INVALID_ARG;
  if (a.B == 0) return FS_OK;
  if (!a.p || !a.u || !a.out_ids || (a.K > 0 && !a.draft_ids) || !aligned(a.p, element(a.dtype)) ||
      !aligned(a.q, element(a.dtype)) || !aligned(a.u, 4) || !aligned(a.draft_ids, 8) ||
      !aligned(a.out_ids, 8) || !aligned(a.out_accepted, 8))
    return FS_ERR_INVALID_ARG;
  if (a.p_seq < 0 || a.p_pos < 0 || a.q_seq < 0 || a.q_pos < 0 ||
      (a.B > 1 && (a.ld_ids < a.K || a.ldu < a.K + 1 || a.ld_out < a.K + 1)))
    return FS_ERR_INVALID_ARG;
  const Device* dev = nullptr;
  const fs_status st = device_setup(&dev);
  if (st != FS_OK) return st;
  VerifyParams p = {};
  p.p = a.p;
  p.q = a.K > 0 ? a.q : nullptr;
  p.ids = a.draft_ids;
  p.u = a.u;
  p.p_seq = a.p_seq;
  p.p_pos = a.p_pos;
  p.q_seq = a.q_seq;
  p.q_pos = a.q_pos;
  p.ld_ids = a.ld_ids;
  p.ldu = a.ldu;
  p.out_ids = a.out_ids;
  p.ld_out = a.ld_out;
  p.accepted = a.out_accepted;
  p.K = int32_t(a.K);
  p.V = int32_t(a.V);
  int64_t segment = kSegment;
  while (ceil_div(a.V, segment) > kMaxSegments) segment *= 2;
  p.segment = int32_t(segment);
  p.n_segments = int32_t(ceil_div(a.V, segment));
  p.wait_limit_ns = kWaitLimitNs;
  p.error_word = dev->error_word;
  // A sequence's row over as many CTAs as fit beside the others' (two an SM), and over twice as
  // many again while each one's part stays worth its place: kPlaceKb for every turn that they
  // take on the SMs (what a CTA would read, at 22 KB a us, in the 5 to 7 us that it is there before
  // and after it reads).  Up to 16 where that leaves a sequence's CTAs an SM each.
  // Measured, in us, calls behind one another on inputs past L2, 1 / 2 / 4 / 8 CTAs: 128256 in
  // bf16 without q, 16 sequences 18.3 / 13.0 / 10.2 / 9.6, 64: 19.4 / 13.8 / 13.2 / 17.4, 152: 19.8 /
  // 18.2 / 25.6 / 32.7, 256: 27.2 / 33.9 / 40.4 / 50.9; alone and from memory 25 / 19 / 17 / 16, 25 /
  // 21 / 19 / 23, 27 / 24 / 33 / 42, 33 / 42 / 48 / 60.  8 and 16 CTAs, 151936 in fp32 with q: 1
  // sequence 8.1 and 6.6, 9: 9.6 and 8.8, 16: 11.4 and 11.8.  Where rows are long and batches large
  // it takes too many by up to a fifth: 256 sequences of 151936 in fp32 41.5 with 2 CTAs, 33.9 with 1.
  constexpr int64_t kPlaceKb = 150;
  const int64_t slots = 2 * int64_t(dev->sms);
  const int64_t row_kb = (a.V * int64_t(element(a.dtype)) * (p.q ? 2 : 1)) >> 10;
  int ctas = 1;
  while (ctas < 8 && ctas * kWarps < p.n_segments &&
         (a.B * ctas * 2 <= slots || a.B * (ctas * 2) * (ctas * 2) * kPlaceKb <= slots * row_kb))
    ctas *= 2;
  if (a.B * kMaxCluster <= dev->sms && 8 * kWarps < p.n_segments && dev->wide_clusters)
    ctas = kMaxCluster;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(ctas);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(a.B * ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = static_cast<cudaStream_t>(stream_ptr);
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t err = a.dtype == FS_F32
                              ? cudaLaunchKernelEx(&cfg, verify_kernel<float>, p)
                              : cudaLaunchKernelEx(&cfg, verify_kernel<__nv_bfloat16>, p);
  if (err != cudaSuccess) {
    cudaGetLastError();
    return FS_ERR_CUDA;
  }
  return FS_OK;
}
