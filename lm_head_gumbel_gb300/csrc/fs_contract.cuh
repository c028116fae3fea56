// fs_contract.cuh -- one persistent tcgen05 contraction kernel, D[m,n] =
// sum_k A[m,k] B[n,k] in fp32, with the operand layouts and the epilogue as
// template parameters.  The log-probability operators are four uses of it:
//   scores     A = H (k contiguous), B = W (k contiguous)  -> row statistics
//   gradient G A = H,                B = W                 -> bf16 [B, V]
//   dH = G W   A = G (k contiguous), B = W (n contiguous)  -> bf16 / partial sums
//   dW = G^T H A = G (m contiguous), B = H (n contiguous)  -> bf16 [V, d]
// so no operand is ever transposed in memory: TMA brings 64 x 64 boxes of the
// contiguous dimension with the 128-byte swizzle either way, and the matrix
// descriptors say which dimension that is.
//
// Warp roles as in the sampler's stage 1: warp 0 issues TMA copies into a ring
// of 64-wide k slices, warp 1 issues the MMAs (M = 128 per CTA and N = 256; for
// CTA pairs cta_group::2, M = 256 over both), warps 2-9 read finished
// accumulators (two of them, so an epilogue overlaps the next unit's MMAs).
// Every wait is bounded: past the limit the roles wind down and the device
// error word records it.
//
// Bound: W's bytes for few rows, the tensor cores for many.  Measured (GB300, copy
// 6.7 TB/s, bf16 1900 TFLOP/s in bursts, 1730 held at the power limit): scores of 64
// rows at d = 4096, V = 151936 read W at 6.6 TB/s with what follows them; of 1000
// rows 1470 TFLOP/s held, 1640 in bursts (a slice of a CTA pair takes 600 cycles, 544
// at the unit's nominal rate); dH of 96 rows at d = 2048 6.5 TB/s; dW of 96 rows
// writes 5.4 TB/s: 2 slices a unit, its epilogue and stores bound it.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "fs_ptx.cuh"

namespace fs {
namespace ptx {

// 2-D tiled store of one box from shared memory (bulk async group).
__device__ __forceinline__ void tma_store_2d(const void* tmap, const void* smem_src, int32_t x,
                                             int32_t y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::
                   "l"(reinterpret_cast<uint64_t>(tmap)),
               "r"(x), "r"(y), "r"(smem_u32(smem_src))
               : "memory");
}
__device__ __forceinline__ void bulk_commit() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// All of this thread's bulk stores have read their shared memory.
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}
__device__ __forceinline__ void bulk_wait() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}
// Order this thread's shared-memory writes before later async-proxy reads.
__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Shared-memory matrix descriptor of an operand whose M (or N) dimension is
// contiguous, stored with the 128-byte swizzle: atoms of 64 bf16 along it by 8
// along K (1024 bytes), K-neighbouring atoms 1024 bytes apart, neighbours along
// M (N) `lead` bytes apart.
__device__ __forceinline__ uint64_t smem_desc_sw128_mn(uint32_t saddr, uint32_t lead) {
  uint64_t desc = 0;
  desc |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  desc |= static_cast<uint64_t>(lead >> 4) << 16;
  desc |= static_cast<uint64_t>(1024u >> 4) << 32;
  desc |= static_cast<uint64_t>(1u) << 46;
  desc |= static_cast<uint64_t>(2u) << 61;
  return desc;
}

// Store to an address from cluster_addr, in this or another CTA of the cluster.
__device__ __forceinline__ void st_cluster(uint32_t addr, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

// Arrive on an mbarrier given by its shared::cluster address, ordering no
// memory: what it reports is that tensor-memory loads have completed (their
// wait has returned).  The releasing form first waits for the thread's earlier
// stores, 2100 cycles beside this kernel's TMA stores.
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t bar_cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                   bar_cluster_addr)
               : "memory");
}

// max that returns NaN if either input is NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float ex2(float a) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(a));
  return r;
}

}  // namespace ptx

namespace vocab {

constexpr int kBM = 128;  // M rows per CTA = tensor-memory lanes
constexpr int kBN = 256;  // N columns per unit = accumulator columns (fewer: Epi::kN)
constexpr int kBK = 64;   // k slice: 64 bf16 = one 128-byte swizzle row
constexpr int kUK = 16;   // k of one MMA
constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (2 + kEpiWarps);
constexpr int kMaxStages = 8;
constexpr uint32_t kChunkBytes = 64 * kBK * 2;  // one 64 x 64 box, 8 KB
constexpr uint32_t kBoxBytes = 2 * 4096;  // an epilogue warp's two 32 x 64 bf16 boxes
constexpr uint32_t kStagingBytes = kEpiWarps * kBoxBytes;
constexpr uint32_t kBarrierBytes = 256;
static_assert((2 * kMaxStages + 5) * 8 + 8 <= kBarrierBytes, "barriers, tensor-memory address, flag");
constexpr int kErrWaitTimeout = 1;  // the library's device error word, bit 0

template <class Epi>
__host__ __device__ constexpr uint32_t ring_bytes() {
  return Epi::kStaged ? 160u * 1024u : 224u * 1024u;
}
template <class Epi>
__host__ __device__ constexpr size_t smem_bytes() {
  return 1024 /* alignment slack */ + ring_bytes<Epi>() + (Epi::kStaged ? kStagingBytes : 0) +
         kBarrierBytes;
}

// k slices per ring stage: narrow units have small slices, and a slice of its
// own stage costs the producer about 450 cycles (8 rows at d = 2048, V = 4096:
// 32 slices, 7.6 of 14 us) -- as long as 64 columns of W take to stream.
template <class Epi>
__host__ __device__ constexpr int slices() {
  return kBN / Epi::kN;
}

// Ring stages for a box of `a_bytes` of A per slice.  An MMA reads kBM rows of A, 16 KB,
// whatever the box holds (rows past it feed accumulator rows that no epilogue reads),
// so the ring leaves room for the last slice's: with a short box and 64 columns of B
// that reach goes past the slice (48 rows: 2 KB; 3 stages of 4 slices instead of 4).
template <class Epi, bool kPair>
__host__ __device__ constexpr uint32_t ring_stages(uint32_t a_bytes) {
  const uint32_t slice = a_bytes + (kPair ? Epi::kN / 2 : Epi::kN) * kBK * 2;
  const uint32_t a_read = kBM * kBK * 2;
  const uint32_t past = a_read > slice ? a_read - slice : 0;
  const uint32_t n = (ring_bytes<Epi>() - past) / (slices<Epi>() * slice);
  return n < kMaxStages ? n : kMaxStages;
}
// Where the MMAs' reads of the ring end, from its start.
template <class Epi, bool kPair>
__host__ __device__ constexpr uint32_t ring_reach(uint32_t a_bytes) {
  const uint32_t slice = a_bytes + (kPair ? Epi::kN / 2 : Epi::kN) * kBK * 2;
  const uint32_t a_read = kBM * kBK * 2;
  const uint32_t all = ring_stages<Epi, kPair>(a_bytes) * slices<Epi>() * slice;
  return all - slice + (slice > a_read ? slice : a_read);
}
// For every height of A's box (8 rows to kBM): at least two stages, in the ring.
template <class Epi, bool kPair>
__host__ __device__ constexpr bool ring_fits() {
  for (uint32_t rows = 8; rows <= kBM; rows += 8)
    if (ring_stages<Epi, kPair>(rows * 128u) < 2 ||
        ring_reach<Epi, kPair>(rows * 128u) > ring_bytes<Epi>())
      return false;
  return true;
}

enum : uint32_t { kPolicyNormal = 0, kPolicyFirst = 1, kPolicyLast = 2 };

struct Shape {
  int32_t n_mt, n_nt;      // tiles along M (128 rows, 256 for CTA pairs) and N (Epi::kN)
  int32_t n_units;         // n_mt * n_nt * number of k splits
  int32_t n_kb;            // 64-wide k slices in all
  int32_t n_splits;        // split i takes slices i, i + n_splits, ... of them
  uint32_t k_descending;   // counted from the last slice: what the kernel before read last is in L2
  int32_t m_rows, n_cols;  // extents of M and N
  uint32_t m_fastest;      // unit order: M tiles (else N tiles) innermost, k splits outermost
  uint32_t a_box_rows;     // rows of A's box when k is contiguous (a multiple of 8)
  uint32_t a_bytes, stage_bytes, n_stages;  // A's part of a slice; a stage holds slices<Epi>()
  uint32_t policy_a, policy_b;  // L2 eviction hints
  // The launch overlaps the kernel before it on the stream, which writes A and
  // the epilogue's inputs: B streams at once, the rest waits for that kernel.
  uint32_t pdl;
  // A dependent kernel may be scheduled from the start (it takes SMs as this
  // one's CTAs leave them) instead of as the last CTAs end.
  uint32_t early_trigger;
  uint64_t wait_limit_ns;
  int* error_word;
};

struct Unit {
  int mt, nt, split;
  int kb0, n_kb;  // first k slice, number of them
};

// A worker's units, every n_workers-th of the list, without a division each.
struct Units {
  int u, step;              // unit, stride
  int inner, outer, split;  // of unit u
  int inner_step, outer_step;
  __device__ __forceinline__ Units(const Shape& s, int worker, int n_workers)
      : u(worker), step(n_workers) {
    const int n_inner = s.m_fastest ? s.n_mt : s.n_nt, n_outer = s.m_fastest ? s.n_nt : s.n_mt;
    const int t = worker / n_inner;
    inner = worker - t * n_inner;
    split = t / n_outer;
    outer = t - split * n_outer;
    outer_step = n_workers / n_inner;
    inner_step = n_workers - outer_step * n_inner;
  }
  __device__ __forceinline__ bool more(const Shape& s) const { return u < s.n_units; }
  __device__ __forceinline__ Unit get(const Shape& s) const {
    Unit r;
    r.mt = s.m_fastest ? inner : outer;
    r.nt = s.m_fastest ? outer : inner;
    r.split = split;
    r.kb0 = s.k_descending ? s.n_kb - 1 - split : split;
    r.n_kb = (s.n_kb - split + s.n_splits - 1) / s.n_splits;
    return r;
  }
  __device__ __forceinline__ void next(const Shape& s) {
    const int n_inner = s.m_fastest ? s.n_mt : s.n_nt, n_outer = s.m_fastest ? s.n_nt : s.n_mt;
    u += step;
    inner += inner_step;
    outer += outer_step;
    if (inner >= n_inner) {
      inner -= n_inner;
      ++outer;
    }
    while (outer >= n_outer) {
      outer -= n_outer;
      ++split;
    }
  }
};

// Bounded mbarrier waits, with the sampler's semantics: past the limit the
// CTA raises its abort flag and the device error word, and every role winds
// down instead of spinning.
struct BoundedWait {
  volatile uint32_t* abort_flag;
  uint64_t limit_ns;
  int* error_word;

  __device__ bool wait(uint64_t* bar, uint32_t parity) const {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = ptx::global_timer_ns();
    while (true) {
      if (ptx::mbar_try_wait(bar, parity)) return true;
      if (*abort_flag) return false;
      if (ptx::global_timer_ns() - t0 > limit_ns) {
        *abort_flag = 1u;
        atomicOr(error_word, kErrWaitTimeout);
        return false;
      }
    }
  }
  __device__ bool wait_warp(uint64_t* bar, uint32_t parity) const {
    return __all_sync(0xFFFFFFFFu, wait(bar, parity));
  }
  // While winding down: ignores the abort flag, still bounded.
  __device__ bool drain(uint64_t* bar, uint32_t parity) const {
    const uint64_t t0 = ptx::global_timer_ns();
    while (!ptx::mbar_try_wait(bar, parity)) {
      if (ptx::global_timer_ns() - t0 > limit_ns) {
        atomicOr(error_word, kErrWaitTimeout);
        return false;
      }
    }
    return true;
  }
};

__device__ __forceinline__ uint64_t policy_of(uint32_t code) {
  return code == kPolicyFirst  ? ptx::policy_evict_first()
         : code == kPolicyLast ? ptx::policy_evict_last()
                               : ptx::policy_evict_normal();
}

// What an epilogue call knows about its 32 rows x kN / 2 columns.
struct TileAt {
  Unit unit;
  int row0;         // first M row of the warp's 32 lanes
  int col0;         // first N column of the warp's columns
  int rank;         // CTA of the pair
  int quad, half;   // rows quad*32.. and which half of the CTA's tile's columns
  uint32_t taddr;   // tensor-memory address of (row0, col0)
};

// kAmn / kBmn: A's M (B's N) dimension is the contiguous one in memory.
// before() runs ahead of the wait for a unit's accumulator and gets the first row of
// the warp's next unit too; start() and finish() get the thread's M row in its
// worker's first unit.
// Epi: struct with Params, State, kN (columns of a unit: 256, or 64 / 128 where
// 256 would leave CTAs without units), kStaged (uses bf16 boxes in shared memory
// and tmap_d), and static device functions start / before / tile / finish.
// The tensor maps and parameters are the kernel's own; `block` of `n_blocks` CTAs.
template <class Epi, bool kPair, bool kAmn, bool kBmn>
__device__ __forceinline__ void contract(const CUtensorMap& tmap_a, const CUtensorMap& tmap_b,
                                         const CUtensorMap& tmap_d, const Shape& s,
                                         const typename Epi::Params& ep, int block,
                                         int n_blocks) {
  constexpr int kCtas = kPair ? 2 : 1;
  constexpr int kN = Epi::kN;
  constexpr uint32_t kTmemCols = 2 * kN;
  static_assert(kN == 256 || (!kPair && !kBmn && (kN == 64 || kN == 128)), "unit columns");
  static_assert(ring_fits<Epi, kPair>(), "MMAs read no further than the ring");
  constexpr int kBRows = kN / kCtas;  // B rows in this CTA's shared memory
  constexpr uint32_t kBBytes = kBRows * kBK * 2;
  constexpr int kS = slices<Epi>();
  constexpr uint32_t kIdesc = ptx::idesc_bf16_f32(kBM * kCtas, kN) | (kAmn ? 1u << 15 : 0u) |
                              (kBmn ? 1u << 16 : 0u);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* staging = smem + ring_bytes<Epi>();
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(staging + (Epi::kStaged ? kStagingBytes : 0));
  uint64_t* empty_bar = full_bar + kMaxStages;
  uint64_t* tfull_bar = empty_bar + kMaxStages;
  uint64_t* tempty_bar = tfull_bar + 2;
  uint64_t* drain_bar = tempty_bar + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain_bar + 1);
  volatile uint32_t* abort_flag = tmem_holder + 1;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = kPair ? int(ptx::cluster_ctarank()) : 0;
  const bool leader = rank == 0;
  const int worker = block / kCtas;
  const int n_workers = n_blocks / kCtas;

  if (threadIdx.x == 0) {
    for (uint32_t i = 0; i < s.n_stages; ++i) {
      ptx::mbar_init(&full_bar[i], 1);
      ptx::mbar_init(&empty_bar[i], 1);
    }
    for (int a = 0; a < 2; ++a) {
      ptx::mbar_init(&tfull_bar[a], 1);
      ptx::mbar_init(&tempty_bar[a], kCtas * kEpiWarps);
    }
    ptx::mbar_init(drain_bar, 1);
    *abort_flag = 0u;
    ptx::fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    ptx::prefetch_tmap(&tmap_a);
    ptx::prefetch_tmap(&tmap_b);
    if (Epi::kStaged) ptx::prefetch_tmap(&tmap_d);
  }
  if (warp == 1) {
    if constexpr (kPair) {
      ptx::tmem_alloc_pair(tmem_holder, kTmemCols);
      ptx::tmem_relinquish_pair();
    } else {
      ptx::tmem_alloc(tmem_holder, kTmemCols);
      ptx::tmem_relinquish();
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if constexpr (kPair) ptx::cluster_sync();
  ptx::tc_fence_after();
  if (s.early_trigger) ptx::grid_launch_dependents();
  const uint32_t tmem_base = *tmem_holder;
  const BoundedWait waiter{abort_flag, s.wait_limit_ns, s.error_word};

  if (warp == 0) {
    // ---------------- TMA producer ----------------
    const bool issuer = ptx::elect_one();
    const uint64_t pol_a = policy_of(s.policy_a), pol_b = policy_of(s.policy_b);
    auto load = [&](uint8_t* dst, const CUtensorMap* map, uint32_t stage, int x, int y,
                    uint64_t pol) {
      if constexpr (kPair)
        ptx::tma_load_2d_pair(dst, map, ptx::cluster_addr(&full_bar[stage], 0), x, y, pol);
      else
        ptx::tma_load_2d(dst, map, &full_bar[stage], x, y, pol);
    };
    // Rows (k contiguous) or 64-wide chunks (M or N contiguous) past the end
    // are read from the last valid ones instead: they only feed accumulator
    // rows or columns that no epilogue reads.
    auto load_a = [&](uint32_t stage, int i, int kb, int mt) {
      uint8_t* dst = smem + size_t(stage) * s.stage_bytes + i * (s.a_bytes + kBBytes);
      const int m0 = (mt * kCtas + rank) * kBM;
      if constexpr (kAmn) {
#pragma unroll
        for (int i = 0; i < kBM / 64; ++i)
          load(dst + i * kChunkBytes, &tmap_a, stage, min(m0 + 64 * i, (s.m_rows - 1) & ~63),
               kb * kBK, pol_a);
      } else {
        load(dst, &tmap_a, stage, kb * kBK, min(m0, s.m_rows - 1), pol_a);
      }
    };
    auto load_b = [&](uint32_t stage, int i, int kb, int nt) {
      uint8_t* dst = smem + size_t(stage) * s.stage_bytes + i * (s.a_bytes + kBBytes) + s.a_bytes;
      const int n0 = nt * kN + rank * kBRows;
      if constexpr (kBmn) {
#pragma unroll
        for (int i = 0; i < kBRows / 64; ++i)
          load(dst + i * kChunkBytes, &tmap_b, stage, min(n0 + 64 * i, (s.n_cols - 1) & ~63),
               kb * kBK, pol_b);
      } else {
        load(dst, &tmap_b, stage, kb * kBK, min(n0, s.n_cols - 1), pol_b);
      }
    };
    uint32_t stage = 0, phase = 0, issued = 0;
    bool ok = true;
    // The first ring fill's A copies, held back until the kernel before is done.
    bool deferring = s.pdl != 0;
    int n_held = 0, held_kb[kMaxStages], held_n[kMaxStages], held_mt[kMaxStages];
    const int kb_step = s.k_descending ? -s.n_splits : s.n_splits;
    auto release = [&]() {
      ptx::grid_dependency_wait();
      if (issuer)
        for (int h = 0; h < n_held; ++h)
          for (int i = 0; i < held_n[h]; ++i) load_a(uint32_t(h), i, held_kb[h] + i * kb_step, held_mt[h]);
      deferring = false;
    };
    for (Units it(s, worker, n_workers); ok && it.more(s); it.next(s)) {
      const Unit t = it.get(s);
      for (int k = 0; k < t.n_kb; k += kS) {
        if (!waiter.wait_warp(&empty_bar[stage], phase ^ 1u)) {
          ok = false;
          break;
        }
        const int n = min(kS, t.n_kb - k);
        if (issuer) {
          if (leader)
            ptx::mbar_arrive_expect_tx(&full_bar[stage],
                                       uint32_t(n) * kCtas * (s.a_bytes + kBBytes));
#pragma unroll
          for (int i = 0; i < kS; ++i) {
            if (i >= n) break;
            const int kb = t.kb0 + (k + i) * kb_step;
            load_b(stage, i, kb, t.nt);
            if (!deferring) load_a(stage, i, kb, t.mt);
          }
        }
        if (deferring) {  // the first fill: stage n_held
          held_kb[n_held] = t.kb0 + k * kb_step;
          held_n[n_held] = n;
          held_mt[n_held++] = t.mt;
        }
        ++issued;
        if (++stage == s.n_stages) {
          stage = 0;
          phase ^= 1u;
        }
        if (deferring && n_held == int(s.n_stages)) release();
      }
    }
    if (deferring) release();
    // Every issued copy lands before the CTA's shared memory goes away (the
    // leader's barriers see both CTAs' copies).
    if (leader) {
      for (uint32_t i = 0; i < s.n_stages; ++i) {
        const uint32_t fills = issued / s.n_stages + (i < issued % s.n_stages ? 1u : 0u);
        if (fills) waiter.drain(&full_bar[i], (fills - 1u) & 1u);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------- MMA issuer (the leader CTA's) ----------------
    if (leader) {
      const bool issuer = ptx::elect_one();
      uint32_t stage = 0, phase = 0, acc = 0, acc_phase = 0;
      bool ok = true;
      const uint32_t s0 = ptx::smem_u32(smem);
      // Descriptors of stage 0; stages and k steps only add to the start
      // address (addresses stay below 256 KB, so the 14-bit field never carries).
      const uint64_t desc_a0 =
          kAmn ? ptx::smem_desc_sw128_mn(s0, kChunkBytes) : ptx::smem_desc_sw128(s0);
      const uint64_t desc_b0 = kBmn ? ptx::smem_desc_sw128_mn(s0 + s.a_bytes, kChunkBytes)
                                    : ptx::smem_desc_sw128(s0 + s.a_bytes);
      constexpr uint64_t kStepA = kAmn ? 2048 >> 4 : (kUK * 2) >> 4;
      constexpr uint64_t kStepB = kBmn ? 2048 >> 4 : (kUK * 2) >> 4;
      auto commit = [&](uint64_t* bar) {
        if constexpr (kPair)
          ptx::mma_commit_pair_multicast(bar, 0x3);
        else
          ptx::mma_commit(bar);
      };
      for (Units it(s, worker, n_workers); ok && it.more(s); it.next(s)) {
        const Unit t = it.get(s);
        if (!waiter.wait_warp(&tempty_bar[acc], acc_phase ^ 1u)) break;
        ptx::tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * kN;
        for (int kb = 0; kb < t.n_kb; kb += kS) {
          if (!waiter.wait_warp(&full_bar[stage], phase)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          if (issuer) {
#pragma unroll
            for (int i = 0; i < kS; ++i) {
              if (i >= t.n_kb - kb) break;
              const uint64_t off =
                  uint64_t((stage * s.stage_bytes + i * (s.a_bytes + kBBytes)) >> 4);
#pragma unroll
              for (int k = 0; k < kBK / kUK; ++k) {
                const uint64_t da = desc_a0 + off + kStepA * k, db = desc_b0 + off + kStepB * k;
                const uint32_t more = (kb | i | k) != 0 ? 1u : 0u;
                if constexpr (kPair)
                  ptx::mma_bf16_pair(d_tmem, da, db, kIdesc, more);
                else
                  ptx::mma_bf16(d_tmem, da, db, kIdesc, more);
              }
            }
            commit(&empty_bar[stage]);
          }
          __syncwarp();
          if (++stage == s.n_stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        if (issuer) commit(&tfull_bar[acc]);
        __syncwarp();
        acc ^= 1u;
        if (acc == 0) acc_phase ^= 1u;
      }
      // All MMAs complete before tensor memory is released.
      if (issuer) {
        if constexpr (kPair)
          ptx::mma_commit_pair(drain_bar);
        else
          ptx::mma_commit(drain_bar);
      }
      __syncwarp();
      waiter.drain(drain_bar, 0);
    }
    __syncwarp();
  } else {
    // ---------------- epilogue ----------------
    if (s.pdl) ptx::grid_dependency_wait();  // its inputs may still be in flight
    const int e = warp - 2;
    const int quad = warp & 3;  // the tensor-memory lane quadrant this warp may read
    const int half = e >> 2;
    uint8_t* box = staging + e * kBoxBytes;
    uint32_t acc = 0, acc_phase = 0;
    typename Epi::State st;
    Units it(s, worker, n_workers);
    const int first_row = (it.get(s).mt * kCtas + rank) * kBM + quad * 32 + lane;
    Epi::start(ep, st, first_row, lane, s);
    for (; it.more(s); it.next(s)) {
      TileAt at;
      at.unit = it.get(s);
      at.rank = rank;
      at.quad = quad;
      at.half = half;
      at.row0 = (at.unit.mt * kCtas + rank) * kBM + quad * 32;
      at.col0 = at.unit.nt * kN + half * (kN / 2);
      at.taddr = tmem_base + (uint32_t(quad * 32) << 16) + acc * kN + uint32_t(half * (kN / 2));
      Units ahead = it;
      ahead.next(s);
      Epi::before(ep, st, at, (ahead.get(s).mt * kCtas + rank) * kBM + quad * 32, lane, s);
      int ok = 0;
      if (lane == 0) ok = waiter.wait(&tfull_bar[acc], acc_phase) ? 1 : 0;
      ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
      if (!ok) break;
      ptx::tc_fence_after();
      // The epilogue calls this once its last tensor-memory load has completed:
      // the next MMAs into this accumulator need not wait for its stores.
      auto release = [&]() {
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (kPair)
            ptx::mbar_arrive_cluster_relaxed(ptx::cluster_addr(&tempty_bar[acc], 0));
          else
            ptx::mbar_arrive(&tempty_bar[acc]);
        }
      };
      if (at.row0 < s.m_rows && at.col0 < s.n_cols)
        Epi::tile(ep, st, at, lane, box, &tmap_d, s, release);
      else
        release();
      acc ^= 1u;
      if (acc == 0) acc_phase ^= 1u;
    }
    Epi::finish(ep, st, worker, first_row, half, s);
    if (Epi::kStaged && lane == 0) ptx::bulk_wait();
  }

  ptx::tc_fence_before();
  __syncthreads();
  // Both CTAs are done with each other's barriers and the MMAs have drained
  // before the pair's tensor memory is released.
  if constexpr (kPair) ptx::cluster_sync();
  if (warp == 1) {
    ptx::tc_fence_after();
    if constexpr (kPair)
      ptx::tmem_dealloc_pair(tmem_base, kTmemCols);
    else
      ptx::tmem_dealloc(tmem_base, kTmemCols);
  }
  if constexpr (kPair) ptx::cluster_sync();
  // A dependent kernel waits for the whole grid before it reads anything of it.
  if (!s.early_trigger) ptx::grid_launch_dependents();
}

template <class Epi, bool kPair, bool kAmn, bool kBmn>
__global__ void __launch_bounds__(kThreads, 1)
    contract_kernel(const __grid_constant__ CUtensorMap tmap_a,
                    const __grid_constant__ CUtensorMap tmap_b,
                    const __grid_constant__ CUtensorMap tmap_d, const Shape s,
                    const __grid_constant__ typename Epi::Params ep) {
  contract<Epi, kPair, kAmn, kBmn>(tmap_a, tmap_b, tmap_d, s, ep, int(blockIdx.x),
                                   int(gridDim.x));
}

// ---------------------------------------------------------------------------
// A bf16 tile through shared memory: the warp's 32 rows x 128 columns are
// written as two boxes of 64 columns in the store's 128-byte swizzle (16-byte
// chunk c of row r at chunk c ^ (r & 7), so a warp's writes touch every bank
// equally often) and TMA stores take them out, clipped at the tensor's edges.
__device__ __forceinline__ void box_begin(int lane) {
  if (lane == 0) ptx::bulk_wait_read();  // the boxes' last stores have been read
  __syncwarp();
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Columns [8c, 8c + 8) of the lane's row, as bf16 pairs.
__device__ __forceinline__ void box_put(uint8_t* box, int lane, int c, uint32_t v0, uint32_t v1,
                                        uint32_t v2, uint32_t v3) {
  *reinterpret_cast<uint4*>(box + (c >> 3) * 4096 + lane * 128 + (((c & 7) ^ (lane & 7)) << 4)) =
      make_uint4(v0, v1, v2, v3);
}
// Store the boxes whose first column lies below `cols`.
__device__ __forceinline__ void box_end(uint8_t* box, const void* tmap, int lane, int x, int y,
                                        int cols) {
  ptx::fence_async_smem();
  __syncwarp();
  if (lane == 0) {
    if (x < cols) ptx::tma_store_2d(tmap, box, x, y);
    if (x + 64 < cols) ptx::tma_store_2d(tmap, box + 4096, x + 64, y);
    ptx::bulk_commit();
  }
}

// The accumulator rounded to bf16 (once, to nearest even) and stored.  A TMA
// store writes whole 16-byte pieces, so tmap_d covers the columns below whole_n
// (a multiple of 8); the up to 7 columns behind are stored one by one, and
// nothing past a row's end is touched.
//
// With few k slices per unit this epilogue is what bounds the kernel (dW of 96
// rows: 2 slices): its steps -- load, wait for the boxes, write them, fence,
// store -- depend on one another, so they are taken once per 128 columns, and
// the accumulator is given back before the boxes are written.
//
// What bf16 rounded away of G at the rows' tokens (Rounding) is added here, in fp32
// and in the order of H's rows.  kByRow (dH): the lane's row is a row of H, its
// token names a row of W.  Else (dW): the lane's row is a row of W; the words the
// logits' pass left for the warp's 32 rows say which rows of H have one of them as
// their token -- usually none, B 32 / V on average.  They are read a unit ahead, and
// the first such row of H before the wait for the accumulator.
struct Rounding {
  const float* delta;  // [B]: G at the row's token, less what is stored of it
  // [V / 32][ceil(B / 32)]: for 32 ids and 32 rows of H, a bit for each row whose
  // token is among the ids, and the first one's token (of the 32) and delta.
  const uint4* marks;
  const int64_t* tokens;
  int64_t vocab_offset;
  int32_t B, V;
  const __nv_bfloat16* X;  // W for dH, H for dW
  int64_t ldx;
  // The token of H's row b as a row of W, or -1.
  __device__ __forceinline__ int32_t row_of_w(int b) const {
    const int64_t local = tokens[b] - vocab_offset;
    return local >= 0 && local < V ? int32_t(local) : -1;
  }
  // The marks of the 32 ids from row0 and the lane's of 32 blocks of H's rows.
  __device__ __forceinline__ uint4 load_marks(int block0, int row0, int lane) const {
    const int blocks = (B + 31) / 32;
    if (block0 + lane >= blocks || row0 >= V) return make_uint4(0u, 0u, 0u, 0u);
    return marks[int64_t(row0 >> 5) * blocks + block0 + lane];
  }
};

// r += f * x for 8 columns from x, of which `n` exist.
__device__ __forceinline__ void add_scaled8(uint32_t* r, float f, const __nv_bfloat16* x, int n) {
  if (n >= 8) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(x));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r[2 * i] = __float_as_uint(fmaf(f, __uint_as_float(w[i] << 16), __uint_as_float(r[2 * i])));
      r[2 * i + 1] = __float_as_uint(
          fmaf(f, __uint_as_float(w[i] & 0xFFFF0000u), __uint_as_float(r[2 * i + 1])));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n)
        r[i] = __float_as_uint(fmaf(f, __bfloat162float(x[i]), __uint_as_float(r[i])));
  }
}

template <bool kByRow>
struct StoreEpi {
  static constexpr int kN = kBN;
  static constexpr bool kStaged = true;
  struct Params {
    __nv_bfloat16* out;
    int64_t ld;
    int32_t whole_n;
    Rounding g;
  };
  struct State {
    float delta;             // kByRow: the row's, 0 for no token
    const __nv_bfloat16* x;  // kByRow: the row of W its token names
    uint4 marks, next;       // else: the first 32 blocks' marks of this unit, the next
    uint32_t some;           // else: which blocks have any
    uint2 quad;              // the first marked row of H: columns 4 lane .. + 3 of 128
  };
  // Columns 4 lane .. + 3 of the 128 from col of H's row b.
  static __device__ __forceinline__ uint2 load_quad(const Params& p, int b, int col, int lane,
                                                    int n_cols) {
    const __nv_bfloat16* x = p.g.X + int64_t(b) * p.g.ldx + col + 4 * lane;
    const int n = n_cols - (col + 4 * lane);
    if (n >= 4) return __ldg(reinterpret_cast<const uint2*>(x));
    uint32_t v[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) v[i] = i < n ? __bfloat16_as_ushort(x[i]) : 0u;
    return make_uint2(v[0] | v[1] << 16, v[2]);
  }
  static __device__ __forceinline__ void start(const Params& p, State& st, int row, int lane,
                                               const Shape&) {
    if constexpr (!kByRow) st.next = p.g.load_marks(0, row - lane, lane);
  }
  static __device__ __forceinline__ void before(const Params& p, State& st, const TileAt& at,
                                                int next_row0, int lane, const Shape& s) {
    if constexpr (kByRow) {
      const int b = at.row0 + lane;
      const int32_t v = b < s.m_rows ? p.g.row_of_w(b) : -1;
      st.delta = v >= 0 ? p.g.delta[b] : 0.0f;
      st.x = p.g.X + int64_t(max(v, 0)) * p.g.ldx;
    } else {
      st.marks = st.next;
      st.next = p.g.load_marks(0, next_row0, lane);
      st.some = __ballot_sync(0xFFFFFFFFu, st.marks.x != 0u);
      if (st.some != 0u) {
        const int k = __ffs(st.some) - 1;
        const int b = k * 32 + __ffs(__shfl_sync(0xFFFFFFFFu, st.marks.x, k)) - 1;
        st.quad = load_quad(p, b, at.col0, lane, s.n_cols);
      }
    }
  }
  // The accumulator of lane `row`, 128 columns, += f times H's (quad).  Short loops:
  // code that few units run comes from far away, and unrolled it took longer to
  // fetch than to run (2 us a unit).
  static __device__ __forceinline__ void add_row(uint32_t taddr, bool here, float f, uint2 quad) {
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
      uint32_t r[32];
      ptx::tmem_ld_32x32b_x32(taddr + uint32_t(c * 32), r);
      ptx::tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const uint32_t w =
            __shfl_sync(0xFFFFFFFFu, (j & 1) ? quad.y : quad.x, c * 8 + (j >> 1));
        const float h0 = __uint_as_float(w << 16), h1 = __uint_as_float(w & 0xFFFF0000u);
        if (here) {
          r[2 * j] = __float_as_uint(fmaf(f, h0, __uint_as_float(r[2 * j])));
          r[2 * j + 1] = __float_as_uint(fmaf(f, h1, __uint_as_float(r[2 * j + 1])));
        }
      }
      ptx::tmem_st_32x32b_x32(taddr + uint32_t(c * 32), r);
    }
    ptx::tmem_wait_st();
  }
  // G's rounding at the tokens among the warp's rows, into the accumulator.
  static __device__ __forceinline__ void add_marked(const Params& p, const State& st,
                                                    const TileAt& at, int lane, int n_cols) {
    bool first = st.some != 0u;  // quad holds its row
#pragma unroll 1
    for (int block0 = 0; block0 < (p.g.B + 31) / 32; block0 += 32) {
      const uint4 m = block0 == 0 ? st.marks : p.g.load_marks(block0, at.row0, lane);
#pragma unroll 1
      for (uint32_t some = __ballot_sync(0xFFFFFFFFu, m.x != 0u); some != 0u; some &= some - 1u) {
        const int k = __ffs(some) - 1, b0 = (block0 + k) * 32;
        uint32_t word = __shfl_sync(0xFFFFFFFFu, m.x, k);
        int32_t row = int32_t(__shfl_sync(0xFFFFFFFFu, m.y, k));
        float f = __uint_as_float(__shfl_sync(0xFFFFFFFFu, m.z, k));
#pragma unroll 1
        while (true) {
          const uint2 quad =
              first ? st.quad : load_quad(p, b0 + __ffs(word) - 1, at.col0, lane, n_cols);
          first = false;
          add_row(at.taddr, row == lane, f, quad);
          word &= word - 1u;
          if (word == 0u) break;
          row = p.g.row_of_w(b0 + __ffs(word) - 1) - at.row0;
          f = p.g.delta[b0 + __ffs(word) - 1];
        }
      }
    }
  }
  // 8 columns of the lane's row, from col: into the box or, from whole_n on, out.
  static __device__ __forceinline__ void put8(const Params& p, const TileAt& at, int lane,
                                              uint8_t* box, const Shape& s, int q, uint32_t v0,
                                              uint32_t v1, uint32_t v2, uint32_t v3) {
    box_put(box, lane, q, v0, v1, v2, v3);
    if (at.col0 + 8 * q == p.whole_n && p.whole_n < s.n_cols && at.row0 + lane < s.m_rows) {
      uint16_t* out = reinterpret_cast<uint16_t*>(p.out + int64_t(at.row0 + lane) * p.ld);
      const uint32_t v[4] = {v0, v1, v2, v3};
#pragma unroll
      for (int i = 0; i < 7; ++i)
        if (p.whole_n + i < s.n_cols) out[p.whole_n + i] = uint16_t(v[i / 2] >> (16 * (i & 1)));
    }
  }
  template <class Release>
  static __device__ __forceinline__ void tile(const Params& p, State& st, const TileAt& at,
                                              int lane, uint8_t* box, const void* tmap,
                                              const Shape& s, Release release) {
    if constexpr (!kByRow)
      if (st.some != 0u || p.g.B > 32 * 32) add_marked(p, st, at, lane, s.n_cols);
    uint32_t v[64];  // the row's 128 columns as bf16 pairs
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      uint32_t r[64];
      ptx::tmem_ld_32x32b_x32(at.taddr + uint32_t(c * 64), reinterpret_cast<uint32_t(&)[32]>(r));
      ptx::tmem_ld_32x32b_x32(at.taddr + uint32_t(c * 64 + 32),
                              reinterpret_cast<uint32_t(&)[32]>(r[32]));
      ptx::tmem_wait_ld();
      if constexpr (kByRow) {
        const int col = at.col0 + c * 64;
        if (st.delta != 0.0f)
#pragma unroll
          for (int q = 0; q < 8; ++q)
            add_scaled8(r + 8 * q, st.delta, st.x + col + 8 * q, s.n_cols - (col + 8 * q));
      }
#pragma unroll
      for (int i = 0; i < 32; ++i)
        v[c * 32 + i] = pack_bf16(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
    }
    release();
    box_begin(lane);
#pragma unroll
    for (int q = 0; q < 16; ++q)
      put8(p, at, lane, box, s, q, v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
    box_end(box, tmap, lane, at.col0, at.row0, p.whole_n);
  }
  static __device__ __forceinline__ void finish(const Params&, State&, int, int, int,
                                                const Shape&) {}
};

// One k split's fp32 accumulator, for a later sum in split order.  A CTA tile
// (128 x 256) is stored as [64 column quads][128 rows] float4, so a warp's
// 16-byte stores are contiguous.  Once a unit of dozens of slices: 94 us at 96 rows,
// d = 2048, V = 151936, of which W's stream is 93.
struct PartialEpi {
  static constexpr int kN = kBN;
  static constexpr bool kStaged = false;
  struct Params {
    float4* partial;
    int32_t ctas;  // CTAs per tile
  };
  struct State {};
  static __device__ __forceinline__ void start(const Params&, State&, int, int, const Shape&) {}
  static __device__ __forceinline__ void before(const Params&, State&, const TileAt&, int, int,
                                                const Shape&) {}
  template <class Release>
  static __device__ __forceinline__ void tile(const Params& p, State&, const TileAt& at, int lane,
                                              uint8_t*, const void*, const Shape& s,
                                              Release release) {
    const int64_t slot =
        (int64_t(at.unit.split) * s.n_mt * s.n_nt + int64_t(at.unit.mt) * s.n_nt + at.unit.nt) *
            p.ctas + at.rank;
    float4* out = p.partial + slot * (kBM * kBN / 4) + at.quad * 32 + lane;
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
      uint32_t r[32];
      ptx::tmem_ld_32x32b_x32(at.taddr + uint32_t(c * 32), r);
      ptx::tmem_wait_ld();
#pragma unroll
      for (int q = 0; q < 8; ++q)
        out[int64_t(at.half * 32 + c * 8 + q) * kBM] =
            make_float4(__uint_as_float(r[4 * q]), __uint_as_float(r[4 * q + 1]),
                        __uint_as_float(r[4 * q + 2]), __uint_as_float(r[4 * q + 3]));
    }
    release();
  }
  static __device__ __forceinline__ void finish(const Params&, State&, int, int, int,
                                                const Shape&) {}
};

}  // namespace vocab
}  // namespace fs
