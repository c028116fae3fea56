// fs_embed.cu -- embedding lookup with scaling, and its gradient to the table by
// sorted tokens (fs_vocab.h).
//
// Lookup: a copy bound by memory; a warp takes 2 KB of one row, 64 bytes a
// lane in flight (16384 ids at d = 5120, bf16: 35 us with what L2 holds, 42 with
// none of it, 5.8 TB/s), or 16 columns a lane, one at a time, of rows that are not
// aligned (16384 ids at d = 5119: 65 us, 114 with 4 at a time; d = 5120 52).
//
// Gradient, up to 1024 ids, one kernel (512 ids, d = 256: 11.1 us, 13.1 by the
// kernels below; 1024 ids, d = 2048: 14.7, 14.3): every CTA sorts the (id, position)
// pairs in shared memory, a warp sums each run of 32 sorted positions over the
// CTA's 64 columns, and ids that cross runs are joined; other CTAs zero the rows
// that no id names.
//
// Gradient, more ids, three or four kernels:
//   sort_kernel       a cluster of 8 CTAs sorts the pairs, stably (4099 ids 8 us,
//                     32768 ids 29: latency)
//   zero_kernel       beside it, when the whole table is written: zeroes it
//   run_sum_kernel    the sorted positions in runs: a warp sums one run over 256
//                     columns, writes the ids that begin and end in the run, and
//                     leaves a partial sum for those that cross into its
//                     neighbours (32768 rows of d = 4096: 54 us, the rows at 5 TB/s
//                     while the table's are written)
//   run_join_kernel   the ids that cross runs, from their partial sums in order
//                     (5 us at 4099 ids, 10 at 32768: latency)
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "fs_ptx.cuh"
#include "fs_vocab.h"

namespace fs {
namespace embed {
namespace {

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// C columns of a row from p, as loaded (C = 8: 16-byte loads, p on a 16-byte
// boundary; C = 2: a pair; C = 1: one element).  Loading and converting are apart so that a
// warp's loads of several rows are all in flight before the first is used.
template <typename T, int C>
struct Piece;
template <typename T>
struct Piece<T, 1> {
  T v;
  __device__ __forceinline__ void load(const T* p) { v = *p; }
  __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = to_float(v); }
};
template <>
struct Piece<__nv_bfloat16, 2> {
  uint32_t v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    v = *reinterpret_cast<const uint32_t*>(p);
  }
  __device__ __forceinline__ void get(float (&f)[2]) const {
    f[0] = __uint_as_float(v << 16);
    f[1] = __uint_as_float(v & 0xFFFF0000u);
  }
};
template <>
struct Piece<float, 2> {
  float2 v;
  __device__ __forceinline__ void load(const float* p) {
    v = *reinterpret_cast<const float2*>(p);
  }
  __device__ __forceinline__ void get(float (&f)[2]) const { f[0] = v.x, f[1] = v.y; }
};
template <>
struct Piece<__nv_bfloat16, 8> {
  uint4 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    v = *reinterpret_cast<const uint4*>(p);
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
};
template <>
struct Piece<float, 8> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
    f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
};
template <>
struct Piece<float, 4> {
  float4 v;
  __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ void get(float (&f)[4]) const {
    f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
  }
};
template <typename T>
__device__ __forceinline__ void store(T* p, const float (&f)[1]) {
  put(p, f[0]);
}
__device__ __forceinline__ void store(__nv_bfloat16* p, const float (&f)[2]) {
  *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(f[0], f[1]);
}
__device__ __forceinline__ void store(float* p, const float (&f)[2]) {
  *reinterpret_cast<float2*>(p) = make_float2(f[0], f[1]);
}
__device__ __forceinline__ void store(float* p, const float (&f)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
}
__device__ __forceinline__ void store(__nv_bfloat16* p, const float (&f)[8]) {
  __nv_bfloat162 h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
  *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(h);
}
__device__ __forceinline__ void store(float* p, const float (&f)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}

// Eight columns 32 apart of a row (kStrided), a warp's next to one another: rows that
// do not start on 16-byte boundaries.  `n` columns are left from p; a column past the
// end is read from p instead and not written.  (8377 fp32 ids, d = 2229, into a whole
// table: 53.6 us; one column a lane 69.7, d = 2232 on 16-byte boundaries 40.8.)
constexpr int kStrided = -8;
template <typename T>
struct Piece<T, kStrided> {
  T v[8];
  __device__ __forceinline__ void load(const T* p, int n) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = p[32 * i < n ? 32 * i : 0];
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = to_float(v[i]);
  }
};
// C columns, or with C = kStrided 8.
template <int C>
constexpr int kColumns = C < 0 ? -C : C;
template <int C, typename T>
__device__ __forceinline__ void load_piece(Piece<T, C>& piece, const T* p, int n) {
  if constexpr (C < 0)
    piece.load(p, n);
  else
    piece.load(p);
}
template <int C, typename T>
__device__ __forceinline__ void store_piece(T* p, const float (&f)[kColumns<C>], int n) {
  if constexpr (C < 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (32 * i < n) put(p + 32 * i, f[i]);
  } else {
    store(p, f);
  }
}

// How a row's columns are divided among warps: columns below `vec` (a multiple
// of 8; 0 where rows do not start on 16-byte boundaries) in segments of C columns
// a lane and G groups of lanes, the rest in segments of R columns a lane.  A
// warp works on one segment, so its path is uniform.
struct Columns {
  int32_t d, vec, vec_segments, segments;
};
__host__ Columns columns_of(int64_t d, bool vec, int C, int groups, int R) {
  Columns c;
  c.d = int32_t(d);
  c.vec = vec ? int32_t(d & ~int64_t(7)) : 0;
  c.vec_segments = (c.vec + 32 * C * groups - 1) / (32 * C * groups);
  c.segments = c.vec_segments + (c.d - c.vec + 32 * R - 1) / (32 * R);
  return c;
}

// ---------------------------------------------------------------------------
// Lookup
// ---------------------------------------------------------------------------
constexpr int kLookupThreads = 128;
constexpr int kLookupGroups = 4;    // of 16 bytes a lane
constexpr int kLookupSingles = 16;  // of one column a lane

// G pieces of C columns from col0, 32 C apart, of one row.
template <typename T, int C, int G>
__device__ __forceinline__ void lookup_piece(const T* src, T* dst, int col0, int end, bool held,
                                             float scale) {
  Piece<T, C> piece[G];
  if (held) {
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int col = col0 + g * 32 * C;
      if (col < end) piece[g].load(src + col);
    }
  }
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int col = col0 + g * 32 * C;
    if (col >= end) break;
    float v[C] = {};
    if (held) {
      piece[g].get(v);
#pragma unroll
      for (int i = 0; i < C; ++i) v[i] *= scale;
    }
    store(dst + col, v);
  }
}

template <typename T>
__global__ void __launch_bounds__(kLookupThreads)
    lookup_kernel(const int64_t* __restrict__ ids, int64_t N, const T* __restrict__ E, int32_t V,
                  int64_t lde, float scale, int64_t vocab_offset, T* __restrict__ out,
                  int64_t ldo, const Columns cols) {
  constexpr int C = 16 / sizeof(T);
  const int lane = threadIdx.x & 31;
  const int64_t item = (int64_t(blockIdx.x) * kLookupThreads + threadIdx.x) >> 5;
  const int64_t n = item / cols.segments;
  if (n >= N) return;
  const int seg = int(item - n * cols.segments);
  const int64_t id = ids[n] - vocab_offset;
  const bool held = id >= 0 && id < V;
  const T* src = E + (held ? id : 0) * lde;
  T* dst = out + n * ldo;
  if (seg < cols.vec_segments)
    lookup_piece<T, C, kLookupGroups>(src, dst, seg * (32 * C * kLookupGroups) + lane * C,
                                      cols.vec, held, scale);
  else
    lookup_piece<T, 1, kLookupSingles>(
        src, dst, cols.vec + (seg - cols.vec_segments) * (32 * kLookupSingles) + lane, cols.d,
        held, scale);
}

// ---------------------------------------------------------------------------
// Gradient: sort, and zero the rows that stay 0
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kCluster = 8;
constexpr int kMaxBits = 9;  // of a radix digit
constexpr int kBins = 1 << kMaxBits;
constexpr int kFillRows = 1 << 16;   // rows of a zeroing CTA, at most
constexpr int kFillBytes = 1 << 18;  // and bytes, about
constexpr int kSmallMax = 1024;      // ids of the one-kernel gradient

struct SortParams {
  const int64_t* ids;
  int32_t N, V;
  int64_t vocab_offset;
  int32_t bits, passes;  // digit width, number of passes
  uint32_t* key[2];      // [N] ping-pong; the result is in [passes & 1]
  uint32_t* pos[2];
  // When the whole table is written (else null):
  uint8_t* table;
  int64_t table_ld, row_bytes;
  int32_t fill_rows;  // rows of a zeroing CTA
};

// An id as a row of the table, V where the table has no such row.
__device__ __forceinline__ uint32_t row_of(const SortParams& p, int64_t id) {
  const int64_t v = id - p.vocab_offset;
  return (v >= 0 && v < p.V) ? uint32_t(v) : uint32_t(p.V);
}

// The lanes of the warp that hold an element with the same digit, for a lane that
// holds one: a vote per digit bit (bits past the digit's width are 0 everywhere).
// __match_any_sync takes several times as long where most lanes differ.
template <int kBits>
__device__ __forceinline__ uint32_t same_digit(uint32_t digit, bool has) {
  uint32_t peers = __ballot_sync(0xFFFFFFFFu, has);
#pragma unroll
  for (int b = 0; b < kBits; ++b) {
    const bool one = (digit >> b) & 1u;
    const uint32_t ones = __ballot_sync(0xFFFFFFFFu, one);
    peers &= one ? ones : ~ones;
  }
  return peers;
}

__device__ __forceinline__ uint32_t load_cluster(const uint32_t* p, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(ptx::cluster_addr(p, rank))
               : "memory");
  return v;
}

// Stable LSD radix sort by one cluster.  CTA c holds elements [c * per, ...).
// A pass: digit counts per CTA; every CTA reads all counts and places its own
// after those of smaller digits and of earlier CTAs; then tiles of 1024
// elements in order, each element ranked among the equal digits of its warp
// (by votes), of the tile's earlier warps (a scan over the warps' counts) and of
// earlier tiles (the running base).
struct ClusterSort {
  uint32_t hist[kBins];          // this CTA's digit counts
  uint32_t base[kBins];          // next place of each digit
  uint32_t scan[kSortWarps];
  uint16_t wc[kSortWarps][kBins];  // a tile's counts per warp, then offsets
};
__device__ void sort_cluster(const SortParams& p, uint32_t rank, ClusterSort& sm) {
  auto &hist = sm.hist, &base = sm.base;
  auto& scan = sm.scan;
  auto& wc = sm.wc;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.N + kCluster - 1) / kCluster;
  const int e0 = min(int(rank) * per, p.N), e1 = min(e0 + per, p.N);
  const int bins = 1 << p.bits;
  const int warps = min(kSortWarps, (e1 - e0 + 31) / 32);  // that hold elements of a tile
  for (int pass = 0; pass < p.passes; ++pass) {
    const int shift = pass * p.bits;
    const uint32_t* kin = p.key[pass & 1];
    const uint32_t* pin = p.pos[pass & 1];
    uint32_t* kout = p.key[(pass + 1) & 1];
    uint32_t* pout = p.pos[(pass + 1) & 1];
    auto key_at = [&](int i) { return pass == 0 ? row_of(p, p.ids[i]) : __ldcg(kin + i); };
    // The first tile's elements stay in registers from the count to the move.
    uint32_t key = 0u, at = 0u;
    if (e0 + tid < e1) {
      key = key_at(e0 + tid);
      at = pass == 0 ? uint32_t(e0 + tid) : __ldcg(pin + e0 + tid);
    }
    for (int i = tid; i < bins; i += kSortThreads) hist[i] = 0u;
    __syncthreads();
    if (e0 + tid < e1) atomicAdd(&hist[(key >> shift) & (bins - 1)], 1u);
#pragma unroll 4
    for (int i = e0 + kSortThreads + tid; i < e1; i += kSortThreads)
      atomicAdd(&hist[(key_at(i) >> shift) & (bins - 1)], 1u);
    ptx::cluster_sync();  // every CTA's counts are complete
    // Thread b: the digit's total, and its count in earlier CTAs.
    uint32_t total = 0u, before = 0u;
    if (tid < bins) {
#pragma unroll
      for (int c = 0; c < kCluster; ++c) {
        const uint32_t n = load_cluster(&hist[tid], uint32_t(c));
        total += n;
        if (c < int(rank)) before += n;
      }
    }
    // Exclusive sum of the totals over the digits.
    uint32_t incl = total;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, incl, off);
      if (lane >= off) incl += o;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    const uint32_t prev = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? scan[lane] : 0u);
    if (tid < bins) base[tid] = prev + incl - total + before;
    for (int t0 = e0; t0 < e1; t0 += kSortThreads) {
      for (int w = warp; w < warps; w += kSortWarps)  // bins is even: 4 bytes at a time
        for (int i = lane; i < bins / 2; i += 32) reinterpret_cast<uint32_t*>(wc[w])[i] = 0u;
      const int i = t0 + tid;
      const bool has = i < e1;
      if (t0 != e0) {
        key = has ? key_at(i) : 0u;
        at = !has ? 0u : pass == 0 ? uint32_t(i) : __ldcg(pin + i);
      }
      __syncthreads();
      const uint32_t digit = (key >> shift) & (bins - 1);
      const uint32_t peers = same_digit<kMaxBits>(digit, has);
      const uint32_t earlier = __popc(peers & ((1u << lane) - 1u));
      if (has && earlier == 0u) wc[warp][digit] = uint16_t(__popc(peers));
      __syncthreads();
      if (tid < bins) {
        uint32_t run = 0u;
#pragma unroll 8
        for (int w = 0; w < warps; ++w) {
          const uint32_t n = wc[w][tid];
          wc[w][tid] = uint16_t(run);
          run += n;
        }
        total = run;  // of this tile
      }
      __syncthreads();
      if (has) {
        const uint32_t to = base[digit] + wc[warp][digit] + earlier;
        __stcg(kout + to, key);
        __stcg(pout + to, at);
      }
      __syncthreads();
      if (tid < bins) base[tid] += total;
    }
    // The next pass reads what all CTAs wrote; no CTA's counts change before
    // all have been read.
    __threadfence();
    ptx::cluster_sync();
  }
}

__device__ __forceinline__ void store_cluster(uint32_t* p, uint32_t rank, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(ptx::cluster_addr(p, rank)), "r"(v)
               : "memory");
}

// The same for up to 1024 pairs a CTA, which stay in registers and shared memory:
// a pass ranks the CTA's pairs, sends its digit counts to every CTA, and then each
// pair to the CTA that holds its place.  (4099 ids: 4 us less than through L2.)
struct SmallClusterSort {
  uint32_t hist[kCluster][kBins];  // every CTA's digit counts
  uint32_t base[kBins];            // first place of this CTA's pairs of a digit
  uint32_t scan[kSortWarps];
  uint32_t in_key[kSortThreads], in_pos[kSortThreads];  // this CTA's pairs
  uint16_t wc[kSortWarps][kBins];  // counts per warp, then offsets
};
__device__ void sort_cluster_small(const SortParams& p, uint32_t rank, SmallClusterSort& sm) {
  auto& hist = sm.hist;
  auto& base = sm.base;
  auto& scan = sm.scan;
  auto &in_key = sm.in_key, &in_pos = sm.in_pos;
  auto& wc = sm.wc;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.N + kCluster - 1) / kCluster;
  const int e0 = min(int(rank) * per, p.N), n = min(per, p.N - e0);
  const int bins = 1 << p.bits;
  const int warps = (n + 31) / 32;
  const bool has = tid < n;
  // Every CTA has started before any writes to another's shared memory; the first
  // pass's counts are taken meanwhile.
  ptx::cluster_arrive();
  uint32_t key = has ? row_of(p, p.ids[e0 + tid]) : 0u;
  uint32_t pos = uint32_t(e0 + tid);
  for (int pass = 0; pass < p.passes; ++pass) {
    if (warp < warps)
      for (int i = lane; i < bins / 2; i += 32) reinterpret_cast<uint32_t*>(wc[warp])[i] = 0u;
    __syncwarp();
    const uint32_t digit = (key >> (pass * p.bits)) & (bins - 1);
    const uint32_t peers = same_digit<kMaxBits>(digit, has);
    const uint32_t earlier = __popc(peers & ((1u << lane) - 1u));
    if (has && earlier == 0u) wc[warp][digit] = uint16_t(__popc(peers));
    __syncthreads();
    if (pass == 0) ptx::cluster_wait();
    if (tid < bins) {
      uint32_t run = 0u;
#pragma unroll 8
      for (int w = 0; w < warps; ++w) {
        const uint32_t c = wc[w][tid];
        wc[w][tid] = uint16_t(run);
        run += c;
      }
#pragma unroll
      for (int c = 0; c < kCluster; ++c) store_cluster(&hist[rank][tid], uint32_t(c), run);
    }
    ptx::cluster_sync();  // every CTA's counts have arrived, and its pairs have been read
    uint32_t total = 0u, before = 0u;
    if (tid < bins) {
#pragma unroll
      for (int c = 0; c < kCluster; ++c) {
        const uint32_t h = hist[c][tid];
        total += h;
        if (c < int(rank)) before += h;
      }
    }
    uint32_t incl = total;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, incl, off);
      if (lane >= off) incl += o;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    const uint32_t prev = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? scan[lane] : 0u);
    if (tid < bins) base[tid] = prev + incl - total + before;
    __syncthreads();
    if (has) {
      const uint32_t to = base[digit] + wc[warp][digit] + earlier;
      const uint32_t c = to / uint32_t(per);
      store_cluster(&in_key[to - c * per], c, key);
      store_cluster(&in_pos[to - c * per], c, pos);
    }
    ptx::cluster_sync();  // every pair has arrived; no counts change before all were read
    if (has) {
      key = in_key[tid];
      pos = in_pos[tid];
    }
  }
  if (has) {
    p.key[p.passes & 1][e0 + tid] = key;
    p.pos[p.passes & 1][e0 + tid] = pos;
  }
}

// Stable LSD radix sort of up to 1024 pairs by one CTA, a pair a thread, in shared
// memory.  A pass counts the digits of every warp's pairs, sums the counts in
// (digit, warp) order -- each count becomes the first place of its digit's pairs
// -- and moves the pairs there.  Ends with the sorted pairs in key and pos.
constexpr int kBlockBits = 7;  // of a digit, at most
struct BlockSort {
  uint16_t count[(1 << kBlockBits) * kSortWarps];
  uint32_t key[kSortThreads];
  uint32_t pos[kSortThreads];
  uint32_t total[kSortWarps];
};
__device__ void sort_block(const SortParams& p, BlockSort& sm) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int bins = 1 << p.bits, n_counts = bins * kSortWarps;
  const int chunk = max(1, n_counts / kSortThreads);  // counts of a thread's part of the sum
  const int c0 = tid * chunk;
  const bool has = tid < p.N;
  uint32_t key = has ? row_of(p, p.ids[tid]) : 0u;
  uint32_t pos = uint32_t(tid);
  for (int pass = 0; pass < p.passes; ++pass) {
    const uint32_t digit = (key >> (pass * p.bits)) & (bins - 1);
    for (int i = tid; i < n_counts; i += kSortThreads) sm.count[i] = 0;
    __syncthreads();
    const uint32_t peers = same_digit<kBlockBits>(digit, has);
    const uint32_t earlier = __popc(peers & ((1u << lane) - 1u));
    if (has && earlier == 0u) sm.count[digit * kSortWarps + warp] = uint16_t(__popc(peers));
    __syncthreads();
    // Exclusive sums of the counts.
    uint32_t mine = 0u;
    if (c0 < n_counts)
      for (int c = 0; c < chunk; ++c) mine += sm.count[c0 + c];
    uint32_t incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, incl, off);
      if (lane >= off) incl += o;
    }
    if (lane == 31) sm.total[warp] = incl;
    __syncthreads();
    const uint32_t before = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? sm.total[lane] : 0u);
    uint32_t run = before + incl - mine;
    if (c0 < n_counts)
      for (int c = 0; c < chunk; ++c) {
        const uint32_t n = sm.count[c0 + c];
        sm.count[c0 + c] = uint16_t(run);
        run += n;
      }
    __syncthreads();
    if (has) {
      const uint32_t to = sm.count[digit * kSortWarps + warp] + earlier;
      sm.key[to] = key;
      sm.pos[to] = pos;
    }
    __syncthreads();
    if (has) {
      key = sm.key[tid];
      pos = sm.pos[tid];
    }
  }
}

// Zeros: two bytes at a time up to a 16-byte boundary, 16 at a time from there,
// by `n` threads of which this is number i.
__device__ __forceinline__ void zero_span(uint8_t* to, int64_t bytes, int i, int n) {
  const int64_t head =
      min(int64_t((16u - uint32_t(reinterpret_cast<uintptr_t>(to) & 15u)) & 15u), bytes);
  const int64_t n16 = (bytes - head) / 16, tail = head + n16 * 16;
  for (int64_t k = i * 2; k < head; k += n * 2) *reinterpret_cast<uint16_t*>(to + k) = 0;
#pragma unroll 4
  for (int64_t k = i; k < n16; k += n)
    reinterpret_cast<uint4*>(to + head)[k] = make_uint4(0u, 0u, 0u, 0u);
  for (int64_t k = tail + i * 2; k < bytes; k += n * 2)
    *reinterpret_cast<uint16_t*>(to + k) = 0;
}

// CTA `part` zeroes its fill_rows rows of the table (about 256 KB, in the order
// the CTAs start: 7.6 TB/s; as few CTAs as SMs, each on rows far apart, wrote at
// 4.9).  kMarked: all but those that some id names, found by one pass over the ids.
template <bool kMarked>
__device__ void fill_rows(const SortParams& p, int64_t part) {
  const int64_t r0 = part * p.fill_rows;
  if (r0 >= p.V) return;
  const int rows = int(min(int64_t(p.fill_rows), p.V - r0));
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint8_t* first = p.table + r0 * p.table_ld;
  __shared__ uint32_t marks[kMarked ? kFillRows / 32 : 1];
  if (kMarked) {
    for (int i = threadIdx.x; i < (rows + 31) / 32; i += kSortThreads) marks[i] = 0u;
    __syncthreads();
    int any = 0;
    for (int i = threadIdx.x; i < p.N; i += kSortThreads) {
      const int64_t r = int64_t(row_of(p, p.ids[i])) - r0;
      if (r >= 0 && r < rows) {
        atomicOr(&marks[r >> 5], 1u << (r & 31));
        any = 1;
      }
    }
    if (__syncthreads_or(any)) {
      for (int r = warp; r < rows; r += kSortWarps)
        if (!((marks[r >> 5] >> (r & 31)) & 1u))
          zero_span(first + r * p.table_ld, p.row_bytes, lane, 32);
      return;
    }
  }
  if (p.table_ld == p.row_bytes)
    zero_span(first, rows * p.row_bytes, threadIdx.x, kSortThreads);
  else
    for (int r = warp; r < rows; r += kSortWarps)
      zero_span(first + r * p.table_ld, p.row_bytes, lane, 32);
}

constexpr size_t kSortSmem = std::max(sizeof(ClusterSort), sizeof(SmallClusterSort));

// One cluster.  Its dependent may start at once: the sums wait for its end, and
// the zeroing needs nothing of it.
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kSortThreads)
    sort_kernel(const SortParams p) {
  extern __shared__ __align__(16) uint8_t dyn[];
  ptx::grid_launch_dependents();
  if (p.N <= kCluster * kSortThreads)
    sort_cluster_small(p, ptx::cluster_ctarank(), *reinterpret_cast<SmallClusterSort*>(dyn));
  else
    sort_cluster(p, ptx::cluster_ctarank(), *reinterpret_cast<ClusterSort*>(dyn));
}

// Zeroes the table while the ids are sorted, as a programmatic dependent of the
// sort: it may start once the sort has (so everything before the sort is done)
// and reads nothing.  Its last CTA ends after the sort, so what waits for this
// kernel waits for both.  (In one launch with the sort, as clusters of 8, the
// zeroing took 242 us instead of 170 at V = 151936, d = 4096.)
__global__ void __launch_bounds__(kSortThreads, 2) zero_kernel(const SortParams p) {
  fill_rows<false>(p, int64_t(blockIdx.x));
  if (blockIdx.x == gridDim.x - 1) ptx::grid_dependency_wait();
}

// ---------------------------------------------------------------------------
// Gradient: sums over the sorted positions
// ---------------------------------------------------------------------------
constexpr int kRunThreads = 128;
constexpr int kRunWarps = kRunThreads / 32;
constexpr int kAhead = 8;  // rows in flight per warp (16 at 2 columns a lane: no gain)

struct RunParams {
  const uint32_t* key;  // sorted rows of the table, V at the end for dropped ids
  const uint32_t* pos;
  int32_t N, V, run, n_runs;  // sorted positions of a run (16 or a multiple of 32), runs
  Columns cols;
  const void* dY;
  int64_t ldy;
  void* dE;
  int64_t lde;
  float scale;
  float* partial;  // [n_runs][2][ldp]: sums of the ids crossing a run's start, end
  int64_t ldp;
};

__device__ __forceinline__ float* partial_at(const RunParams& p, int run, int end, int col) {
  return p.partial + (int64_t(run) * 2 + end) * p.ldp + col;
}

template <typename TO>
__device__ __forceinline__ TO* table_at(const RunParams& p, uint32_t row, int col) {
  return static_cast<TO*>(p.dE) + int64_t(row) * p.lde + col;
}

// A row's finished sum, scaled and (kAdd) added to what the row held.
template <bool kAdd, typename TO, int C>
__device__ __forceinline__ void write_sum(const RunParams& p, TO* dst, const Piece<TO, C>& old,
                                          const float (&sum)[kColumns<C>], int n) {
  float v[kColumns<C>];
#pragma unroll
  for (int i = 0; i < kColumns<C>; ++i) v[i] = sum[i] * p.scale;
  if (kAdd) {
    float o[kColumns<C>];
    old.get(o);
#pragma unroll
    for (int i = 0; i < kColumns<C>; ++i) v[i] += o[i];
  }
  store_piece<C>(dst, v, n);
}

// One warp, one run, C columns a lane from col, of which n are left (lanes without
// any, n <= 0, follow along on the row's first columns).  The run's ids come in order; the
// first may continue the previous run's last (then its sum is the run's start
// partial), the last may go on in the next run (the end partial; a run that is
// one id crossing both ways has a start partial only).  The rows of dY, and
// with kAdd the table's rows that are finished here, are loaded kAhead at once.
template <typename TY, typename TO, int C, bool kAdd>
__device__ __forceinline__ void sum_run(const RunParams& p, int run, int col, int n, int lane) {
  const bool in = n > 0;
  const int i0 = run * p.run, i1 = min(i0 + p.run, p.N);
  const uint32_t dropped = uint32_t(p.V);
  const TY* src = static_cast<const TY*>(p.dY) + (in ? col : 0);
  float sum[kColumns<C>] = {};
  uint32_t prev = i0 > 0 ? p.key[i0 - 1] : dropped;
  bool crosses_start = false;  // the sum continues the previous run's
  bool open = false;           // the sum goes on past the last position seen
  for (int j0 = i0; j0 < i1; j0 += 32) {
    // Lane i holds sorted position j0 + i and whether its id ends there.
    uint32_t key = dropped, pos = 0u, next = dropped;
    const int j = j0 + lane;
    if (j < i1) {
      key = p.key[j];
      pos = p.pos[j];
    }
    if (j + 1 < p.N && j < i1) next = p.key[j + 1];
    const int live = __popc(__ballot_sync(0xFFFFFFFFu, key != dropped));
    const uint32_t ends = __ballot_sync(0xFFFFFFFFu, key != dropped && next != key);
    if (live == 0) break;
    if (j0 == i0) crosses_start = i0 > 0 && prev == __shfl_sync(0xFFFFFFFFu, key, 0);
#pragma unroll 1
    for (int g = 0; g < live; g += kAhead) {
      Piece<TY, C> piece[kAhead];
      Piece<TO, C> old[kAdd ? kAhead : 1];
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {  // past the end: the last row again, unused
        const int i = min(g + a, live - 1);
        load_piece<C>(piece[a], src + int64_t(__shfl_sync(0xFFFFFFFFu, pos, i)) * p.ldy, n);
        if (kAdd && ((ends >> i) & 1u))
          load_piece<C>(old[a], table_at<TO>(p, __shfl_sync(0xFFFFFFFFu, key, i), in ? col : 0),
                        n);
      }
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        if (g + a >= live) break;
        float v[kColumns<C>];
        piece[a].get(v);
#pragma unroll
        for (int i = 0; i < kColumns<C>; ++i) sum[i] += v[i];
        if (!((ends >> (g + a)) & 1u)) continue;  // warp-uniform
        const uint32_t row = __shfl_sync(0xFFFFFFFFu, key, g + a);
        if (in) {
          if (crosses_start)
            store_piece<C>(partial_at(p, run, 0, col), sum, n);
          else
            write_sum<kAdd, TO, C>(p, table_at<TO>(p, row, col), old[kAdd ? a : 0], sum, n);
        }
        crosses_start = false;
#pragma unroll
        for (int i = 0; i < kColumns<C>; ++i) sum[i] = 0.0f;
      }
    }
    open = !((ends >> (live - 1)) & 1u);
  }
  if (open && in) store_piece<C>(partial_at(p, run, crosses_start ? 0 : 1, col), sum, n);
}

// The id that begins in run `run` and goes on up to run `last`: its partial
// sums in order.
template <typename TO, int C, bool kAdd>
__device__ __forceinline__ void join_runs(const RunParams& p, int run, int last, uint32_t id,
                                          int col, int n) {
  float sum[kColumns<C>];
  Piece<TO, C> old;
  if (kAdd) load_piece<C>(old, static_cast<const TO*>(table_at<TO>(p, id, col)), n);
  Piece<float, C> piece;
  load_piece<C>(piece, static_cast<const float*>(partial_at(p, run, 1, col)), n);
  piece.get(sum);
#pragma unroll 8
  for (int r = run + 1; r <= last; ++r) {
    float v[kColumns<C>];
    load_piece<C>(piece, static_cast<const float*>(partial_at(p, r, 0, col)), n);
    piece.get(v);
#pragma unroll
    for (int i = 0; i < kColumns<C>; ++i) sum[i] += v[i];
  }
  write_sum<kAdd, TO, C>(p, table_at<TO>(p, id, col), old, sum, n);
}

// kVec: rows on 16-byte boundaries.  (A kernel for each: the strided loads take twice
// the registers of the bf16 ones.)
template <typename TY, typename TO, bool kAdd, bool kVec>
__global__ void __launch_bounds__(kRunThreads) run_sum_kernel(const RunParams p) {
  ptx::grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  const int64_t item = (int64_t(blockIdx.x) * kRunThreads + threadIdx.x) >> 5;
  const int run = int(item / p.cols.segments);
  if (run >= p.n_runs) return;
  const int seg = int(item - int64_t(run) * p.cols.segments);
  if constexpr (!kVec) {
    const int col = seg * 256 + lane;
    sum_run<TY, TO, kStrided, kAdd>(p, run, col, p.cols.d - col, lane);
  } else if (seg < p.cols.vec_segments) {
    const int col = seg * 256 + lane * 8;
    sum_run<TY, TO, 8, kAdd>(p, run, col, p.cols.vec - col, lane);
  } else {
    const int col = p.cols.vec + (seg - p.cols.vec_segments) * 32 + lane;
    sum_run<TY, TO, 1, kAdd>(p, run, col, p.cols.d - col, lane);
  }
}

// The last run that goes on with the id that run `run` ends in (by a warp; 32 runs
// looked at at once), or -1 if no id begins in the run and goes on.
__device__ __forceinline__ int last_run(const RunParams& p, int run, int lane) {
  if (run >= p.n_runs - 1) return -1;  // the last run's ids end in it
  const int i0 = run * p.run, i1 = i0 + p.run;  // a run before the last is full
  const uint32_t id = p.key[i1 - 1];
  if (id == uint32_t(p.V) || p.key[i1] != id) return -1;
  if (p.key[i0] == id && i0 > 0 && p.key[i0 - 1] == id) return -1;  // began earlier
  int last = run;
  while (true) {
    const int r = last + 1 + lane;
    const bool on = r < p.n_runs && p.key[int64_t(r) * p.run] == id;
    const uint32_t all = __ballot_sync(0xFFFFFFFFu, on);
    last += all == 0xFFFFFFFFu ? 32 : __ffs(~all) - 1;
    if (all != 0xFFFFFFFFu) return last;
  }
}

template <typename TO, bool kAdd>
__global__ void __launch_bounds__(kRunThreads) run_join_kernel(const RunParams p) {
  ptx::grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  const int64_t item = (int64_t(blockIdx.x) * kRunThreads + threadIdx.x) >> 5;
  const int run = int(item / p.cols.segments);
  const int seg = int(item - int64_t(run) * p.cols.segments);
  const int last = last_run(p, run, lane);
  if (last < 0) return;
  const uint32_t id = p.key[(run + 1) * p.run - 1];
  if (seg < p.cols.vec_segments) {
    const int col = seg * 256 + lane * 8;
    if (col < p.cols.vec) join_runs<TO, 8, kAdd>(p, run, last, id, col, p.cols.vec - col);
  } else if (p.cols.vec == 0) {
    const int col = seg * 256 + lane;
    if (col < p.cols.d) join_runs<TO, kStrided, kAdd>(p, run, last, id, col, p.cols.d - col);
  } else {
    const int col = p.cols.vec + (seg - p.cols.vec_segments) * 32 + lane;
    if (col < p.cols.d) join_runs<TO, 1, kAdd>(p, run, last, id, col, p.cols.d - col);
  }
}

// ---------------------------------------------------------------------------
// Gradient of up to kSmallMax ids, one kernel
// ---------------------------------------------------------------------------
constexpr int kSmallCols = 64;  // columns of a CTA: two a lane (one where rows are not aligned)
struct SmallShared {
  BlockSort sort;
  float partial[kSmallMax / 32 * 2 * kSmallCols];
};

template <typename TY, typename TO, int C, bool kAdd>
__device__ __forceinline__ void small_segment(const RunParams& p, int warp, int lane, int col,
                                              int n) {
  if (warp < p.n_runs) sum_run<TY, TO, C, kAdd>(p, warp, col, n, lane);
  __syncthreads();
  const int last = last_run(p, warp, lane);
  if (last >= 0 && n > 0)
    join_runs<TO, C, kAdd>(p, warp, last, p.key[(warp + 1) * p.run - 1], col, n);
}

// CTAs 0 .. segments - 1: a segment of the columns, a warp for each run of 32
// sorted positions; the others zero rows.  The sort is done by every CTA for
// itself (about 1.5 us), so that none waits for another.
template <typename TY, typename TO, bool kAdd>
__global__ void __launch_bounds__(kSortThreads)
    small_grad_kernel(const SortParams sp, const RunParams rp) {
  __shared__ SmallShared sm;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int seg = blockIdx.x;
  if (seg >= rp.cols.segments) {
    fill_rows<true>(sp, int64_t(seg) - rp.cols.segments);
    return;
  }
  sort_block(sp, sm.sort);
  __syncthreads();
  RunParams p = rp;
  p.key = sm.sort.key;
  p.pos = sm.sort.pos;
  p.ldp = kSmallCols;
  if (seg < p.cols.vec_segments) {
    const int col0 = seg * 64, col = col0 + lane * 2;
    p.partial = sm.partial - col0;
    small_segment<TY, TO, 2, kAdd>(p, warp, lane, col, p.cols.vec - col);
  } else {
    const int col0 = p.cols.vec + (seg - p.cols.vec_segments) * 32, col = col0 + lane;
    p.partial = sm.partial - col0;
    small_segment<TY, TO, 1, kAdd>(p, warp, lane, col, p.cols.d - col);
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
constexpr int kMaxDevices = 64;
std::mutex g_mu;
fs_status g_status[kMaxDevices];
bool g_known[kMaxDevices] = {};

// FS_OK on a GB300 (sm_103), as the library's other entry points.
fs_status device_check() {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
    cudaGetLastError();
    return FS_ERR_UNSUPPORTED;
  }
  std::lock_guard<std::mutex> lock(g_mu);
  if (!g_known[dev]) {
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess) {
      cudaGetLastError();
      return FS_ERR_CUDA;
    }
    g_status[dev] = major == 10 && minor == 3 ? FS_OK : FS_ERR_UNSUPPORTED;
    if (g_status[dev] == FS_OK &&
        cudaFuncSetAttribute(sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             int(kSortSmem)) != cudaSuccess) {
      cudaGetLastError();
      g_status[dev] = FS_ERR_CUDA;
    }
    g_known[dev] = true;
  }
  return g_status[dev];
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t round256(size_t n) { return (n + 255u) & ~size_t(255u); }
int64_t element(int dtype) { return dtype == FS_F32 ? 4 : 2; }
// Partial rows start on 16-byte boundaries: d rounded up to 8.
int64_t partial_ld(int64_t d) { return (d + 7) / 8 * 8; }
bool rows_vec(const void* p, int64_t ld, int dtype) {
  return aligned(p, 16) && ld * element(dtype) % 16 == 0;
}
constexpr int64_t kMaxN = INT_MAX - 65536;  // the loops over positions step past N by a block
bool sizes_ok(int64_t N, int64_t V, int64_t d, int64_t vocab_offset) {
  return N >= 0 && N <= kMaxN && d >= 1 && d <= INT_MAX - 2048 && V >= 1 && vocab_offset >= 0 &&
         V <= INT_MAX && vocab_offset + V <= INT_MAX;
}

// `after`: as a programmatic dependent of the kernel before.
cudaError_t launch(const void* kernel, int64_t blocks, int threads, size_t smem, bool after,
                   void** args, cudaStream_t stream) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(blocks), 1, 1);
  cfg.blockDim = dim3(unsigned(threads), 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = after ? 1 : 0;
  return cudaLaunchKernelExC(&cfg, kernel, args);
}

}  // namespace
}  // namespace embed
}  // namespace fs

using namespace fs::embed;

extern "C" fs_status fs_embed(const int64_t* ids, int64_t N, const void* E, int64_t V, int64_t d,
                              int64_t lde, int dtype, float scale, int64_t vocab_offset,
                              void* out, int64_t ldo, void* stream_ptr) {
  if (!sizes_ok(N, V, d, vocab_offset) || lde < d || ldo < d) return FS_ERR_INVALID_ARG;
  if (dtype != FS_BF16 && dtype != FS_F32) return FS_ERR_INVALID_ARG;
  if (N == 0) return FS_OK;
  if (!ids || !E || !out || !aligned(ids, 8) || !aligned(E, element(dtype)) ||
      !aligned(out, element(dtype)))
    return FS_ERR_INVALID_ARG;
  const Columns cols =
      columns_of(d, rows_vec(E, lde, dtype) && rows_vec(out, ldo, dtype),
                 int(16 / element(dtype)), kLookupGroups,
                 kLookupSingles);
  const int64_t blocks = ceil_div(N * cols.segments, kLookupThreads / 32);
  if (blocks > INT_MAX) return FS_ERR_INVALID_ARG;
  const fs_status st = device_check();
  if (st != FS_OK) return st;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  if (dtype == FS_BF16)
    lookup_kernel<__nv_bfloat16><<<unsigned(blocks), kLookupThreads, 0, stream>>>(
        ids, N, static_cast<const __nv_bfloat16*>(E), int32_t(V), lde, scale, vocab_offset,
        static_cast<__nv_bfloat16*>(out), ldo, cols);
  else
    lookup_kernel<float><<<unsigned(blocks), kLookupThreads, 0, stream>>>(
        ids, N, static_cast<const float*>(E), int32_t(V), lde, scale, vocab_offset,
        static_cast<float*>(out), ldo, cols);
  return cudaGetLastError() == cudaSuccess ? FS_OK : FS_ERR_CUDA;
}

namespace fs {
namespace embed {
namespace {

// Sorted positions of a run (32 in the one-kernel gradient): long ones leave fewer
// partial sums to join, short ones more warps.  Measured with ids at frequencies
// 1 / rank, in us a call, runs of 16 / 32 / 64 / 128:
//   2048 ids, d = 2048   16.1 / 17.9 / 23.6 / 35.4     3000 ids  18.8 / 20.8 / 25.0 / 37.3
//   4099 ids, d = 2048   22.2 / 21.4 / 25.4 / 37.9    12000 ids  44.7 / 39.0 / 39.0 / 51.3
//   (4099 with nothing in L2 24.2 / 25.1)
//   16384 ids, d = 2048  63.0 / 47.3 / 45.1           32768 ids, d = 4096  178 / 143 / 131 / 123
//   16384 ids, d = 512   36.1 / 32.8 / 36.2 / 47.9    32768 ids, d = 256    - /  50 /  56 /  69
// (the last two: a warp takes 256 columns, so long runs leave too few warps).
int64_t run_length(int64_t N, int64_t d) {
  if (N <= kSmallMax) return 32;
  int64_t run = N <= 5000 ? 16 : N <= 12000 ? 32 : N <= 20000 ? 64 : 128;
  while (run > 16 && N / run * ceil_div(d, 256) < 1000) run /= 2;
  return run;
}

template <bool kAdd>
const void* small_kernel(int y_dtype, int e_dtype) {
  if (y_dtype == FS_F32)
    return reinterpret_cast<const void*>(&small_grad_kernel<float, float, kAdd>);
  if (e_dtype == FS_F32)
    return reinterpret_cast<const void*>(&small_grad_kernel<__nv_bfloat16, float, kAdd>);
  return reinterpret_cast<const void*>(&small_grad_kernel<__nv_bfloat16, __nv_bfloat16, kAdd>);
}

template <bool kAdd, bool kVec>
const void* sum_kernel(int y_dtype, int e_dtype) {
  if (y_dtype == FS_F32)
    return reinterpret_cast<const void*>(&run_sum_kernel<float, float, kAdd, kVec>);
  if (e_dtype == FS_F32)
    return reinterpret_cast<const void*>(&run_sum_kernel<__nv_bfloat16, float, kAdd, kVec>);
  return reinterpret_cast<const void*>(&run_sum_kernel<__nv_bfloat16, __nv_bfloat16, kAdd, kVec>);
}
template <bool kAdd>
const void* join_kernel_of(int e_dtype) {
  return e_dtype == FS_F32 ? reinterpret_cast<const void*>(&run_join_kernel<float, kAdd>)
                           : reinterpret_cast<const void*>(&run_join_kernel<__nv_bfloat16, kAdd>);
}

}  // namespace
}  // namespace embed
}  // namespace fs

// Workspace: two buffers of sorted rows, two of positions, the runs' partial sums.
extern "C" size_t fs_embed_grad_workspace_size(int64_t N, int64_t d) {
  if (N < 1 || !sizes_ok(N, 1, d, 0)) return 0;
  return 4 * round256(size_t(N) * 4u) +
         round256(size_t(ceil_div(N, run_length(N, d))) * 2u * size_t(partial_ld(d)) * 4u);
}

extern "C" fs_status fs_embed_grad(const int64_t* ids, int64_t N, const void* dY, int64_t V,
                                   int64_t d, int64_t ldy, int y_dtype, float scale,
                                   int64_t vocab_offset, void* dE, int64_t lde, int e_dtype,
                                   int accumulate, void* workspace, size_t workspace_bytes,
                                   void* stream_ptr) {
  if (!sizes_ok(N, V, d, vocab_offset) || ldy < d || lde < d) return FS_ERR_INVALID_ARG;
  if ((y_dtype != FS_BF16 && y_dtype != FS_F32) || (e_dtype != FS_BF16 && e_dtype != FS_F32) ||
      (y_dtype == FS_F32 && e_dtype != FS_F32))
    return FS_ERR_INVALID_ARG;
  if (!dE || !aligned(dE, element(e_dtype))) return FS_ERR_INVALID_ARG;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  if (N == 0) {
    if (accumulate) return FS_OK;
    const fs_status st = device_check();
    if (st != FS_OK) return st;
    if (cudaMemset2DAsync(dE, size_t(lde * element(e_dtype)), 0, size_t(d * element(e_dtype)),
                          size_t(V), stream) != cudaSuccess) {
      cudaGetLastError();
      return FS_ERR_CUDA;
    }
    return FS_OK;
  }
  if (!ids || !dY || !aligned(ids, 8) || !aligned(dY, element(y_dtype))) return FS_ERR_INVALID_ARG;
  const bool small = N <= kSmallMax;
  const int64_t run = run_length(N, d), n_runs = ceil_div(N, run);
  const bool vec = d >= 8 && rows_vec(dY, ldy, y_dtype) && rows_vec(dE, lde, e_dtype);
  const Columns cols = columns_of(d, vec, small ? 2 : 8, 1, small || vec ? 1 : 8);  // kStrided's 8
  const int64_t blocks = ceil_div(n_runs * cols.segments, kRunWarps);
  if (blocks > INT_MAX) return FS_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256) ||
      workspace_bytes < fs_embed_grad_workspace_size(N, d))
    return FS_ERR_WORKSPACE;
  const fs_status st = device_check();
  if (st != FS_OK) return st;

  SortParams sp = {};
  sp.ids = ids;
  sp.N = int32_t(N);
  sp.V = int32_t(V);
  sp.vocab_offset = vocab_offset;
  int bits = 1;
  while (bits < 31 && (int64_t(1) << bits) <= V) ++bits;  // rows 0 .. V
  const int most = small ? kBlockBits : kMaxBits;
  sp.passes = (bits + most - 1) / most;
  sp.bits = (bits + sp.passes - 1) / sp.passes;
  if (!accumulate) {
    sp.table = static_cast<uint8_t*>(dE);
    sp.table_ld = lde * element(e_dtype);
    sp.row_bytes = d * element(e_dtype);
    sp.fill_rows =
        int32_t(std::min<int64_t>(kFillRows, std::max<int64_t>(1, kFillBytes / sp.row_bytes)));
  }
  const int64_t fill = accumulate ? 0 : ceil_div(V, sp.fill_rows);  // CTAs that zero rows
  if (fill > INT_MAX - cols.segments - 2 * kCluster) return FS_ERR_INVALID_ARG;
  RunParams rp = {};
  rp.N = int32_t(N);
  rp.V = int32_t(V);
  rp.run = int32_t(run);
  rp.n_runs = int32_t(n_runs);
  rp.cols = cols;
  rp.dY = dY;
  rp.ldy = ldy;
  rp.dE = dE;
  rp.lde = lde;
  rp.scale = scale;
  cudaError_t err;

  if (small) {
    void* args[] = {&sp, &rp};
    err = launch(accumulate ? small_kernel<true>(y_dtype, e_dtype)
                            : small_kernel<false>(y_dtype, e_dtype),
                 cols.segments + fill, kSortThreads, 0, false, args, stream);
    if (err != cudaSuccess) {
      cudaGetLastError();
      return FS_ERR_CUDA;
    }
    return FS_OK;
  }

  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const size_t one = round256(size_t(N) * 4u);
  for (int i = 0; i < 2; ++i) {
    sp.key[i] = reinterpret_cast<uint32_t*>(ws + one * i);
    sp.pos[i] = reinterpret_cast<uint32_t*>(ws + one * (2 + i));
  }
  rp.key = sp.key[sp.passes & 1];
  rp.pos = sp.pos[sp.passes & 1];
  rp.partial = reinterpret_cast<float*>(ws + 4 * one);
  rp.ldp = partial_ld(d);
  void* sort_args[] = {&sp};
  err = launch(reinterpret_cast<const void*>(&sort_kernel), kCluster, kSortThreads, kSortSmem,
               false, sort_args, stream);
  // All rows are zeroed: those that ids name are written twice, which is less
  // than telling them apart costs (every zeroing CTA would read all ids).
  if (err == cudaSuccess && !accumulate)
    err = launch(reinterpret_cast<const void*>(&zero_kernel), fill, kSortThreads, 0, true,
                 sort_args, stream);
  const void* sum = accumulate ? (vec ? sum_kernel<true, true>(y_dtype, e_dtype)
                                      : sum_kernel<true, false>(y_dtype, e_dtype))
                               : (vec ? sum_kernel<false, true>(y_dtype, e_dtype)
                                      : sum_kernel<false, false>(y_dtype, e_dtype));
  const void* join = accumulate ? join_kernel_of<true>(e_dtype) : join_kernel_of<false>(e_dtype);
  void* args[] = {&rp};
  if (err == cudaSuccess) err = launch(sum, blocks, kRunThreads, 0, true, args, stream);
  if (err == cudaSuccess && n_runs > 1)
    err = launch(join, blocks, kRunThreads, 0, true, args, stream);
  if (err != cudaSuccess) {
    cudaGetLastError();
    return FS_ERR_CUDA;
  }
  return FS_OK;
}
