// fs_embed.cu -- embedding lookup with scaling, and its gradient to the table by
// sorted tokens (fs_vocab.h).
//
// Lookup: a copy bound by memory; a warp takes 2 KB of one row, 64 bytes a
// lane in flight.
//
// Gradient, three kernels:
//   sort_fill_kernel  a cluster of 8 CTAs sorts (id, position) stably; when the
//                     whole table is written, the other CTAs meanwhile zero
//                     the rows that no id names
//   run_sum_kernel    the sorted positions in runs of 32: a warp sums one run
//                     over 256 columns, writes the ids that begin and end in
//                     the run, and leaves a partial sum for those that cross
//                     into its neighbours
//   run_join_kernel   the ids that cross runs, from their partial sums in order
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

constexpr int kCols = 8;  // columns a lane works on

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }

// Eight columns from `col` of a row of d, in fp32; `vec`: the row starts on a
// 16-byte boundary (col is a multiple of 8).  Columns past d read as 0.
__device__ __forceinline__ void load8(const __nv_bfloat16* row, int col, int d, bool vec,
                                      float (&v)[kCols]) {
  if (vec && col + kCols <= d) {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(row + col));
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kCols; ++i) v[i] = col + i < d ? to_float(row[col + i]) : 0.0f;
  }
}
__device__ __forceinline__ void load8(const float* row, int col, int d, bool vec,
                                      float (&v)[kCols]) {
  if (vec && col + kCols <= d) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(row + col));
    const float4 b = __ldg(reinterpret_cast<const float4*>(row + col) + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < kCols; ++i) v[i] = col + i < d ? row[col + i] : 0.0f;
  }
}
__device__ __forceinline__ void store8(__nv_bfloat16* row, int col, int d, bool vec,
                                       const float (&v)[kCols]) {
  if (vec && col + kCols <= d) {
    __nv_bfloat162 h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<uint4*>(row + col) = *reinterpret_cast<const uint4*>(h);
  } else {
#pragma unroll
    for (int i = 0; i < kCols; ++i)
      if (col + i < d) row[col + i] = __float2bfloat16_rn(v[i]);
  }
}
__device__ __forceinline__ void store8(float* row, int col, int d, bool vec,
                                       const float (&v)[kCols]) {
  if (vec && col + kCols <= d) {
    reinterpret_cast<float4*>(row + col)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(row + col)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
#pragma unroll
    for (int i = 0; i < kCols; ++i)
      if (col + i < d) row[col + i] = v[i];
  }
}

// ---------------------------------------------------------------------------
// Lookup
// ---------------------------------------------------------------------------
constexpr int kLookupThreads = 128;
constexpr int kLookupGroups = 4;  // 8-column groups per lane

template <typename T>
__global__ void __launch_bounds__(kLookupThreads)
    lookup_kernel(const int64_t* __restrict__ ids, int64_t N, const T* __restrict__ E, int32_t V,
                  int32_t d, int64_t lde, float scale, int64_t vocab_offset, T* __restrict__ out,
                  int64_t ldo, int32_t segments, int vec_in, int vec_out) {
  const int lane = threadIdx.x & 31;
  const int64_t item = (int64_t(blockIdx.x) * kLookupThreads + threadIdx.x) >> 5;
  const int64_t n = item / segments;
  if (n >= N) return;
  const int col0 = int(item - n * segments) * (32 * kLookupGroups * kCols) + lane * kCols;
  const int64_t id = ids[n] - vocab_offset;
  const bool held = id >= 0 && id < V;
  const T* src = E + (held ? id : 0) * lde;
  T* dst = out + n * ldo;
  float v[kLookupGroups][kCols];
#pragma unroll
  for (int g = 0; g < kLookupGroups; ++g) {
    const int col = col0 + g * 32 * kCols;
    if (held && col < d) {
      load8(src, col, d, vec_in != 0, v[g]);
    } else {
#pragma unroll
      for (int i = 0; i < kCols; ++i) v[g][i] = 0.0f;
    }
  }
#pragma unroll
  for (int g = 0; g < kLookupGroups; ++g) {
    const int col = col0 + g * 32 * kCols;
    if (col >= d) break;
    if (held) {
#pragma unroll
      for (int i = 0; i < kCols; ++i) v[g][i] *= scale;
    }
    store8(dst, col, d, vec_out != 0, v[g]);
  }
}

// ---------------------------------------------------------------------------
// Gradient: sort, and zero the rows that stay 0
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kCluster = 8;
constexpr int kMaxBits = 9;  // of a radix digit
constexpr int kBins = 1 << kMaxBits;
constexpr int kFillRows = 1 << 16;  // rows whose marks a fill CTA holds at once

struct SortParams {
  const int64_t* ids;
  int32_t N, V;
  int64_t vocab_offset;
  int32_t bits, passes;  // digit width, number of passes
  uint32_t* key[2];      // [N] ping-pong; the result is in [passes & 1]
  uint32_t* pos[2];
  uint8_t* fill;  // rows to zero (null: none), strides and lengths in bytes
  int64_t fill_ld;
  int64_t fill_row;
};

// An id as a row of the table, V where the table has no such row.
__device__ __forceinline__ uint32_t row_of(const SortParams& p, int64_t id) {
  const int64_t v = id - p.vocab_offset;
  return (v >= 0 && v < p.V) ? uint32_t(v) : uint32_t(p.V);
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
// (match), of the tile's earlier warps (a scan over the warps' counts) and of
// earlier tiles (the running base).
__device__ void sort_cluster(const SortParams& p, uint32_t rank) {
  __shared__ uint32_t hist[kBins];          // this CTA's digit counts
  __shared__ uint32_t base[kBins];          // next place of each digit
  __shared__ uint32_t scan[kSortWarps];
  __shared__ uint16_t wc[kSortWarps][kBins];  // a tile's counts per warp, then offsets
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.N + kCluster - 1) / kCluster;
  const int e0 = min(int(rank) * per, p.N), e1 = min(e0 + per, p.N);
  const int bins = 1 << p.bits;
  for (int pass = 0; pass < p.passes; ++pass) {
    const int shift = pass * p.bits;
    const uint32_t* kin = p.key[pass & 1];
    const uint32_t* pin = p.pos[pass & 1];
    uint32_t* kout = p.key[(pass + 1) & 1];
    uint32_t* pout = p.pos[(pass + 1) & 1];
    auto key_at = [&](int i) { return pass == 0 ? row_of(p, p.ids[i]) : __ldcg(kin + i); };
    for (int i = tid; i < bins; i += kSortThreads) hist[i] = 0u;
    __syncthreads();
    for (int i = e0 + tid; i < e1; i += kSortThreads)
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
    uint32_t prev = 0u;
    for (int w = 0; w < warp; ++w) prev += scan[w];
    if (tid < bins) base[tid] = prev + incl - total + before;
    for (int t0 = e0; t0 < e1; t0 += kSortThreads) {
      for (int i = tid; i < kSortWarps * bins; i += kSortThreads)
        wc[i / bins][i & (bins - 1)] = 0;
      __syncthreads();
      const int i = t0 + tid;
      const bool has = i < e1;
      uint32_t key = 0u, digit = 0xFFFFFFFFu, at = 0u;
      if (has) {
        key = key_at(i);
        at = pass == 0 ? uint32_t(i) : __ldcg(pin + i);
        digit = (key >> shift) & (bins - 1);
      }
      const uint32_t peers = __match_any_sync(0xFFFFFFFFu, digit);
      const uint32_t earlier = __popc(peers & ((1u << lane) - 1u));
      if (has && earlier == 0u) wc[warp][digit] = uint16_t(__popc(peers));
      __syncthreads();
      if (tid < bins) {
        uint32_t run = 0u;
#pragma unroll 8
        for (int w = 0; w < kSortWarps; ++w) {
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

// CTA `part` of `parts` zeroes its share of the rows that no id names: it marks
// the named ones of its range in shared memory (one pass over the ids), then
// writes the others, a warp per row.
__device__ void fill_rows(const SortParams& p, int part, int parts) {
  __shared__ uint32_t marks[kFillRows / 32];
  const int64_t per = (int64_t(p.V) + parts - 1) / parts;
  const int64_t r0 = int64_t(part) * per, r1 = min(r0 + per, int64_t(p.V));
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int64_t b0 = r0; b0 < r1; b0 += kFillRows) {
    const int rows = int(min(int64_t(kFillRows), r1 - b0));
    __syncthreads();
    for (int i = threadIdx.x; i < (rows + 31) / 32; i += kSortThreads) marks[i] = 0u;
    __syncthreads();
    for (int i = threadIdx.x; i < p.N; i += kSortThreads) {
      const int64_t r = int64_t(row_of(p, p.ids[i])) - b0;
      if (r >= 0 && r < rows) atomicOr(&marks[r >> 5], 1u << (r & 31));
    }
    __syncthreads();
    for (int r = warp; r < rows; r += kSortWarps) {
      if ((marks[r >> 5] >> (r & 31)) & 1u) continue;
      // Two bytes at a time up to a 16-byte boundary, 16 at a time from there.
      uint8_t* row = p.fill + (b0 + r) * p.fill_ld;
      const int64_t head =
          min(int64_t((16u - uint32_t(reinterpret_cast<uintptr_t>(row) & 15u)) & 15u), p.fill_row);
      const int64_t n16 = (p.fill_row - head) / 16, tail = head + n16 * 16;
      for (int64_t i = lane * 2; i < head; i += 64) *reinterpret_cast<uint16_t*>(row + i) = 0;
      for (int64_t i = lane; i < n16; i += 32)
        reinterpret_cast<uint4*>(row + head)[i] = make_uint4(0u, 0u, 0u, 0u);
      for (int64_t i = tail + lane * 2; i < p.fill_row; i += 64)
        *reinterpret_cast<uint16_t*>(row + i) = 0;
    }
  }
}

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kSortThreads)
    sort_fill_kernel(const SortParams p) {
  if (blockIdx.x < kCluster)
    sort_cluster(p, ptx::cluster_ctarank());
  else
    fill_rows(p, int(blockIdx.x) - kCluster, int(gridDim.x) - kCluster);
  ptx::grid_launch_dependents();
}

// ---------------------------------------------------------------------------
// Gradient: sums over the sorted positions
// ---------------------------------------------------------------------------
constexpr int kRun = 32;        // sorted positions of a run
constexpr int kRunThreads = 128;
constexpr int kAhead = 8;       // rows in flight per warp

struct RunParams {
  const uint32_t* key;  // sorted rows of the table, V at the end for dropped ids
  const uint32_t* pos;
  int32_t N, V, d, n_runs, segments;
  const void* dY;
  int64_t ldy;
  void* dE;
  int64_t lde;
  float scale;
  float* partial;  // [n_runs][2][d]: sums of the ids crossing a run's start, end
  int vec_in, vec_out, accumulate;
};

template <typename TO>
__device__ __forceinline__ void write_row(const RunParams& p, uint32_t row, int col,
                                          float (&sum)[kCols]) {
  TO* dst = static_cast<TO*>(p.dE) + int64_t(row) * p.lde;
#pragma unroll
  for (int i = 0; i < kCols; ++i) sum[i] *= p.scale;
  if (p.accumulate) {
    float old[kCols];
    if (p.vec_out && col + kCols <= p.d) {  // not __ldg: this launch writes the row
      if constexpr (sizeof(TO) == 4) {
        const float4 a = reinterpret_cast<const float4*>(dst + col)[0];
        const float4 b = reinterpret_cast<const float4*>(dst + col)[1];
        old[0] = a.x, old[1] = a.y, old[2] = a.z, old[3] = a.w;
        old[4] = b.x, old[5] = b.y, old[6] = b.z, old[7] = b.w;
      } else {
        const uint4 a = *reinterpret_cast<const uint4*>(dst + col);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          old[2 * i] = __uint_as_float(w[i] << 16);
          old[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < kCols; ++i) old[i] = col + i < p.d ? to_float(dst[col + i]) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < kCols; ++i) sum[i] += old[i];
  }
  store8(dst, col, p.d, p.vec_out != 0, sum);
}

// Partial rows start on 16-byte boundaries: d rounded up to 8.
__host__ __device__ __forceinline__ int64_t partial_ld(int64_t d) { return (d + 7) / 8 * 8; }

__device__ __forceinline__ float4* partial_at(const RunParams& p, int run, int end, int col) {
  return reinterpret_cast<float4*>(p.partial + (int64_t(run) * 2 + end) * partial_ld(p.d) + col);
}

// One warp: run `run`, columns [seg * 256, ...).  The run's ids come in order;
// the first may continue the previous run's last (then its sum is the run's
// start partial), the last may go on in the next run (the end partial; a run
// that is one id crossing both ways has a start partial only).
template <typename TY, typename TO>
__global__ void __launch_bounds__(kRunThreads) run_sum_kernel(const RunParams p) {
  ptx::grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  const int64_t item = (int64_t(blockIdx.x) * kRunThreads + threadIdx.x) >> 5;
  const int run = int(item / p.segments);
  if (run >= p.n_runs) return;
  const int col = int(item - int64_t(run) * p.segments) * (32 * kCols) + lane * kCols;
  const int i0 = run * kRun, n = min(kRun, p.N - i0);
  const uint32_t dropped = uint32_t(p.V);
  // Lane i holds sorted position i0 + i.
  uint32_t key = dropped, pos = 0u;
  if (lane < n) {
    key = p.key[i0 + lane];
    pos = p.pos[i0 + lane];
  }
  const uint32_t before = i0 > 0 ? p.key[i0 - 1] : dropped;
  const uint32_t after = i0 + n < p.N ? p.key[i0 + n] : dropped;
  const int live = __popc(__ballot_sync(0xFFFFFFFFu, lane < n && key != dropped));
  const bool in = col < p.d;
  const TY* dY = static_cast<const TY*>(p.dY);
  float sum[kCols] = {};
  uint32_t cur = __shfl_sync(0xFFFFFFFFu, key, 0);
  bool crosses_start = live > 0 && i0 > 0 && before == cur;
  for (int g = 0; g < live; g += kAhead) {
    float v[kAhead][kCols];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const uint32_t at = __shfl_sync(0xFFFFFFFFu, pos, (g + a) & 31);
      if (g + a < live && in) {
        load8(dY + int64_t(at) * p.ldy, col, p.d, p.vec_in != 0, v[a]);
      } else {
#pragma unroll
        for (int i = 0; i < kCols; ++i) v[a][i] = 0.0f;
      }
    }
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const uint32_t k = __shfl_sync(0xFFFFFFFFu, key, (g + a) & 31);
      if (g + a >= live) break;
      if (k != cur) {  // warp-uniform: `cur` ends here
        if (in) {
          if (crosses_start) {
            partial_at(p, run, 0, col)[0] = make_float4(sum[0], sum[1], sum[2], sum[3]);
            partial_at(p, run, 0, col)[1] = make_float4(sum[4], sum[5], sum[6], sum[7]);
          } else {
            write_row<TO>(p, cur, col, sum);
          }
        }
        crosses_start = false;
        cur = k;
#pragma unroll
        for (int i = 0; i < kCols; ++i) sum[i] = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < kCols; ++i) sum[i] += v[a][i];
    }
  }
  if (live == 0 || !in) return;
  const bool crosses_end = live == n && after == cur;
  if (crosses_start || crosses_end) {
    float4* to = partial_at(p, run, crosses_start ? 0 : 1, col);
    to[0] = make_float4(sum[0], sum[1], sum[2], sum[3]);
    to[1] = make_float4(sum[4], sum[5], sum[6], sum[7]);
  } else {
    write_row<TO>(p, cur, col, sum);
  }
}

// One warp: the id that begins in run `run` and goes on past its end, if there
// is one: its partial sums in order.
template <typename TO>
__global__ void __launch_bounds__(kRunThreads) run_join_kernel(const RunParams p) {
  ptx::grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  const int64_t item = (int64_t(blockIdx.x) * kRunThreads + threadIdx.x) >> 5;
  const int run = int(item / p.segments);
  if (run >= p.n_runs - 1) return;  // the last run's ids end in it
  const int col = int(item - int64_t(run) * p.segments) * (32 * kCols) + lane * kCols;
  const int i0 = run * kRun, i1 = i0 + kRun;  // a run before the last is full
  const uint32_t id = p.key[i1 - 1];
  if (id == uint32_t(p.V) || p.key[i1] != id) return;
  if (p.key[i0] == id && i0 > 0 && p.key[i0 - 1] == id) return;  // began earlier
  // The runs that go on with the id (32 looked at at once).
  int last = run;
  while (true) {
    const int r = last + 1 + lane;
    const bool on = r < p.n_runs && p.key[int64_t(r) * kRun] == id;
    const uint32_t all = __ballot_sync(0xFFFFFFFFu, on);
    last += all == 0xFFFFFFFFu ? 32 : __ffs(~all) - 1;
    if (all != 0xFFFFFFFFu) break;
  }
  if (col >= p.d) return;
  const float4* first = partial_at(p, run, 1, col);
  float4 a = first[0], b = first[1];
  float sum[kCols] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll 8
  for (int r = run + 1; r <= last; ++r) {
    const float4* q = partial_at(p, r, 0, col);
    a = q[0], b = q[1];
    sum[0] += a.x, sum[1] += a.y, sum[2] += a.z, sum[3] += a.w;
    sum[4] += b.x, sum[5] += b.y, sum[6] += b.z, sum[7] += b.w;
  }
  write_row<TO>(p, id, col, sum);
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
    g_known[dev] = true;
  }
  return g_status[dev];
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t round256(size_t n) { return (n + 255u) & ~size_t(255u); }
int64_t element(int dtype) { return dtype == FS_F32 ? 4 : 2; }
bool rows_vec(const void* p, int64_t ld, int dtype) {
  return aligned(p, 16) && ld * element(dtype) % 16 == 0;
}
constexpr int64_t kMaxN = INT_MAX - 65536;  // the loops over positions step past N by a block
bool sizes_ok(int64_t N, int64_t V, int64_t d, int64_t vocab_offset) {
  return N >= 0 && N <= kMaxN && d >= 1 && d <= INT_MAX - 2048 && V >= 1 && vocab_offset >= 0 &&
         V <= INT_MAX && vocab_offset + V <= INT_MAX;
}

cudaError_t launch_after(const void* kernel, int64_t blocks, int threads, void** args,
                         cudaStream_t stream) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(blocks), 1, 1);
  cfg.blockDim = dim3(unsigned(threads), 1, 1);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
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
  const int64_t segments = ceil_div(d, 32 * kLookupGroups * kCols);
  const int64_t blocks = ceil_div(N * segments, kLookupThreads / 32);
  if (blocks > INT_MAX) return FS_ERR_INVALID_ARG;
  const fs_status st = device_check();
  if (st != FS_OK) return st;
  const int vi = rows_vec(E, lde, dtype), vo = rows_vec(out, ldo, dtype);
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  if (dtype == FS_BF16)
    lookup_kernel<__nv_bfloat16><<<unsigned(blocks), kLookupThreads, 0, stream>>>(
        ids, N, static_cast<const __nv_bfloat16*>(E), int32_t(V), int32_t(d), lde, scale,
        vocab_offset, static_cast<__nv_bfloat16*>(out), ldo, int32_t(segments), vi, vo);
  else
    lookup_kernel<float><<<unsigned(blocks), kLookupThreads, 0, stream>>>(
        ids, N, static_cast<const float*>(E), int32_t(V), int32_t(d), lde, scale, vocab_offset,
        static_cast<float*>(out), ldo, int32_t(segments), vi, vo);
  return cudaGetLastError() == cudaSuccess ? FS_OK : FS_ERR_CUDA;
}

// Workspace: two buffers of sorted rows, two of positions, the runs' partial sums.
extern "C" size_t fs_embed_grad_workspace_size(int64_t N, int64_t d) {
  if (N <= 0 || N > kMaxN || d < 1 || d > INT_MAX - 2048) return 0;
  return 4 * round256(size_t(N) * 4u) +
         round256(size_t(ceil_div(N, kRun)) * 2u * size_t(partial_ld(d)) * 4u);
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
  if (N > 0 && (!ids || !dY || !aligned(ids, 8) || !aligned(dY, element(y_dtype))))
    return FS_ERR_INVALID_ARG;
  if (N == 0 && accumulate) return FS_OK;
  const int64_t n_runs = ceil_div(N, kRun), segments = ceil_div(d, 32 * kCols);
  const int64_t blocks = ceil_div(n_runs * segments, kRunThreads / 32);
  if (blocks > INT_MAX) return FS_ERR_INVALID_ARG;
  if (N > 0 && (!workspace || !aligned(workspace, 256) ||
                workspace_bytes < fs_embed_grad_workspace_size(N, d)))
    return FS_ERR_WORKSPACE;
  const fs_status st = device_check();
  if (st != FS_OK) return st;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);

  SortParams sp = {};
  sp.ids = ids;
  sp.N = int32_t(N);
  sp.V = int32_t(V);
  sp.vocab_offset = vocab_offset;
  int bits = 1;
  while (bits < 31 && (int64_t(1) << bits) <= V) ++bits;  // rows 0 .. V
  sp.passes = (bits + kMaxBits - 1) / kMaxBits;
  sp.bits = (bits + sp.passes - 1) / sp.passes;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const size_t one = round256(size_t(N) * 4u);
  if (N > 0) {
    for (int i = 0; i < 2; ++i) {
      sp.key[i] = reinterpret_cast<uint32_t*>(ws + one * i);
      sp.pos[i] = reinterpret_cast<uint32_t*>(ws + one * (2 + i));
    }
  } else {
    sp.passes = 0;
  }
  if (!accumulate) {
    sp.fill = static_cast<uint8_t*>(dE);
    sp.fill_ld = lde * element(e_dtype);
    sp.fill_row = d * element(e_dtype);
  }
  // One cluster sorts; 19 more (152 CTAs) zero rows.
  sort_fill_kernel<<<accumulate ? kCluster : 20 * kCluster, kSortThreads, 0, stream>>>(sp);
  if (cudaGetLastError() != cudaSuccess) return FS_ERR_CUDA;
  if (N == 0) return FS_OK;

  RunParams rp = {};
  rp.key = sp.key[sp.passes & 1];
  rp.pos = sp.pos[sp.passes & 1];
  rp.N = int32_t(N);
  rp.V = int32_t(V);
  rp.d = int32_t(d);
  rp.n_runs = int32_t(n_runs);
  rp.segments = int32_t(segments);
  rp.dY = dY;
  rp.ldy = ldy;
  rp.dE = dE;
  rp.lde = lde;
  rp.scale = scale;
  rp.partial = reinterpret_cast<float*>(ws + 4 * one);
  rp.vec_in = rows_vec(dY, ldy, y_dtype);
  rp.vec_out = rows_vec(dE, lde, e_dtype);
  rp.accumulate = accumulate ? 1 : 0;
  const void* sum = y_dtype == FS_F32 ? reinterpret_cast<const void*>(&run_sum_kernel<float, float>)
                    : e_dtype == FS_F32
                        ? reinterpret_cast<const void*>(&run_sum_kernel<__nv_bfloat16, float>)
                        : reinterpret_cast<const void*>(
                              &run_sum_kernel<__nv_bfloat16, __nv_bfloat16>);
  const void* join = e_dtype == FS_F32
                         ? reinterpret_cast<const void*>(&run_join_kernel<float>)
                         : reinterpret_cast<const void*>(&run_join_kernel<__nv_bfloat16>);
  void* args[] = {&rp};
  cudaError_t err = launch_after(sum, blocks, kRunThreads, args, stream);
  if (err == cudaSuccess && n_runs > 1)
    err = launch_after(join, blocks, kRunThreads, args, stream);
  if (err != cudaSuccess) {
    cudaGetLastError();
    return FS_ERR_CUDA;
  }
  return FS_OK;
}
