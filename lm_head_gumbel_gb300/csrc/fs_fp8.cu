// fs_fp8.cu -- fs_quantize and fs_matmul_fp8 (fs_speculate.h): matrices in 8-bit
// floating point (e4m3) with a scale for each block of 128, and their product.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>
#include <mutex>
#include <type_traits>

#include "fs_contract.cuh"
#include "fs_pieces.h"
#include "fs_ptx.cuh"
#include "fs_speculate.h"

namespace fs {
int* device_error_word();  // fs_sample.cu

namespace ptx {

// kind::f8f6f4: 8-bit A and B (one byte an element, 32 along k), fp32 accumulate.
__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_f8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Instruction descriptor of kind::f8f6f4 with e4m3 A/B (format 0), fp32 D, both K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(uint32_t M, uint32_t N) {
  return (1u << 4) | ((N >> 3) << 17) | ((M >> 4) << 24);
}
// d += a * b on two fp32 values at once (a register pair each).
__device__ __forceinline__ void fma2(uint64_t& d, uint64_t a, uint64_t b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(d) : "l"(a), "l"(b));
}
__device__ __forceinline__ uint64_t pack2(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
// Barriers and values in shared memory by 32-bit addresses.
__device__ __forceinline__ bool mbar_try_wait_at(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ void mbar_arrive_at(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ float ld_shared_f32(uint32_t at) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}
// Two values in e4m3, to nearest even, past 448 to 448; lo in the low byte.
__device__ __forceinline__ uint32_t cvt_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

}  // namespace ptx

namespace fp8 {
namespace {

constexpr int kBlock = FS_FP8_BLOCK;
constexpr float kMostE4m3 = 448.0f;

// ---------------------------------------------------------------------------
// Quantisation
// ---------------------------------------------------------------------------
// Bound: memory.  A head of 151936 x 4096 in bf16 (1.87 GB read and written) takes 264 us,
// 7.1 TB/s, in fp32 439; 16384 x 5120 hidden states 40 us, 6.4 TB/s, in fp32 62.  Rows off 16-byte
// boundaries go element by element: 103 and 133 us for those hidden states.  Elements stay bits until they are
// scaled, so that a thread's loads are all in flight (branches between them: 779 us for the
// head), and the largest magnitude is an unsigned maximum: a NaN's bits are above every
// number's.
constexpr uint32_t kLeastMaxBits = 0x0D800000u;  // 2^-100

// 8 elements as they lie in memory.
template <class T>
struct Eight {
  uint32_t w[2 * sizeof(T)];
};
// Those from x, of which n exist, the others 0, are read in two steps, so that the first
// of several pieces can be in flight at once: whole ones (fs_pieces.h), then what is left.
template <class T, bool kVec>
__device__ __forceinline__ bool load_whole(Eight<T>& e, const T* x, int n, bool last) {
  const bool can = kVec && whole_piece(n, last);
#pragma unroll
  for (int i = 0; i < int(sizeof(T)) / 2; ++i) {
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (can) v = __ldcs(reinterpret_cast<const uint4*>(x) + i);
    e.w[4 * i] = v.x, e.w[4 * i + 1] = v.y, e.w[4 * i + 2] = v.z, e.w[4 * i + 3] = v.w;
  }
  return can;
}
template <class T>
__device__ __forceinline__ void load_rest(Eight<T>& e, const T* x, int n, bool whole) {
  if (n <= 0 || (whole && n >= 8)) return;
  if constexpr (sizeof(T) == 2) {
    const uint16_t* p = reinterpret_cast<const uint16_t*>(x);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      e.w[i] = (2 * i < n ? p[2 * i] : 0u) | (2 * i + 1 < n ? uint32_t(p[2 * i + 1]) << 16 : 0u);
  } else {
    const uint32_t* p = reinterpret_cast<const uint32_t*>(x);
#pragma unroll
    for (int i = 0; i < 8; ++i) e.w[i] = i < n ? p[i] : 0u;
  }
}
// The bits of the largest magnitude, as fp32.
__device__ __forceinline__ uint32_t most(const Eight<__nv_bfloat16>& e) {
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("max.u16x2 %0, %1, %2;" : "=r"(m) : "r"(m), "r"(e.w[i] & 0x7FFF7FFFu));
  return max(m & 0xFFFF0000u, m << 16);
}
__device__ __forceinline__ uint32_t most(const Eight<float>& e) {
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, e.w[i] & 0x7FFFFFFFu);
  return m;
}
__device__ __forceinline__ float element_of(const Eight<__nv_bfloat16>& e, int i) {
  return __uint_as_float((i & 1) ? e.w[i / 2] & 0xFFFF0000u : e.w[i / 2] << 16);
}
__device__ __forceinline__ float element_of(const Eight<float>& e, int i) {
  return __uint_as_float(e.w[i]);
}

template <bool kVec, class E>
__device__ __forceinline__ void store8(uint8_t* out, int n, const E& e, float inv) {
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    h[i] = ptx::cvt_e4m3x2(element_of(e, 2 * i) * inv, element_of(e, 2 * i + 1) * inv);
  const uint2 w = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
  if (kVec && n >= 8) {
    *reinterpret_cast<uint2*>(out) = w;
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) out[i] = uint8_t((i < 4 ? w.x : w.y) >> (8 * (i & 3)));
}

struct QuantParams {
  const void* x;
  int64_t ldx;
  uint8_t* values;
  int64_t ldv;
  float* scale;
  int64_t lds;
  int32_t N, d, col_blocks;
};

// Blocks of 1 x 128 to 8 lanes, which take pieces l and l + 8 of a block's 16; kPer blocks
// side by side in a thread's registers.  16 lanes a block, a division of the block's number
// and two for the scales in every lane left 16384 x 5120 bound by instructions: 59 us.
constexpr int kRowThreads = 128;
constexpr int kRowLanes = 8;
constexpr int kRowBlocks = kRowThreads / kRowLanes;  // a CTA's side by side
template <class T, bool kVec, int kPer>
__global__ void __launch_bounds__(kRowThreads) quantize_rows_kernel(const QuantParams p) {
  const int lane = threadIdx.x % kRowLanes;
  int64_t block = int64_t(blockIdx.x) * (kRowBlocks * kPer) + threadIdx.x / kRowLanes;
  int64_t row = int64_t(p.N) * p.col_blocks <= UINT_MAX - 4096  // past it by a CTA
                    ? int64_t(uint32_t(block) / uint32_t(p.col_blocks))
                    : block / p.col_blocks;
  int cb = int(block - row * p.col_blocks);
  int64_t rows[kPer];
  int cbs[kPer];
  Eight<T> e[kPer][2];
  bool whole[kPer][2];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    rows[i] = row;
    cbs[i] = cb;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int col = cb * kBlock + (lane + kRowLanes * j) * 8;
      whole[i][j] = load_whole<T, kVec>(e[i][j], static_cast<const T*>(p.x) + row * p.ldx + col,
                                        row < p.N ? p.d - col : 0, row == p.N - 1);
    }
    for (cb += kRowBlocks; cb >= p.col_blocks; cb -= p.col_blocks) ++row;
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const bool here = rows[i] < p.N;
    const int col = cbs[i] * kBlock + lane * 8;
    const T* x = static_cast<const T*>(p.x) + rows[i] * p.ldx + col;
    uint32_t m = kLeastMaxBits;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      load_rest(e[i][j], x + 64 * j, here ? p.d - col - 64 * j : 0, whole[i][j]);
      m = max(m, most(e[i][j]));
    }
#pragma unroll
    for (int s = kRowLanes / 2; s > 0; s >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, s));
    // One division for both: the first lane's is the scale, the others' its inverse.
    const float top = __uint_as_float(m);
    const float ratio = __fdiv_rn(lane == 0 ? top : kMostE4m3, lane == 0 ? kMostE4m3 : top);
    const float inv = __shfl_sync(0xFFFFFFFFu, ratio, (threadIdx.x & 31) | 1);
    if (!here) continue;
    if (lane == 0) p.scale[rows[i] * p.lds + cbs[i]] = ratio;
    uint8_t* out = p.values + rows[i] * p.ldv + col;
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (p.d - col > 64 * j) store8<kVec>(out + 64 * j, p.d - col - 64 * j, e[i][j], inv);
  }
}

// A block of 128 x 128 to a CTA, kTileLoads pieces of 8 elements a thread.
constexpr int kTileThreads = 256;
constexpr int kTileLoads = 8;
template <class T, bool kVec>
__global__ void __launch_bounds__(kTileThreads) quantize_tile_kernel(const QuantParams p) {
  __shared__ uint32_t warp_max[kTileThreads / 32];
  const int rb = int(blockIdx.x / unsigned(p.col_blocks));
  const int cb = int(blockIdx.x - unsigned(rb) * unsigned(p.col_blocks));
  const int col = cb * kBlock + int(threadIdx.x & 15) * 8;
  const int row0 = rb * kBlock + int(threadIdx.x >> 4);
  const T* x = static_cast<const T*>(p.x) + int64_t(row0) * p.ldx + col;
  uint8_t* out = p.values + int64_t(row0) * p.ldv + col;
  Eight<T> e[kTileLoads];
  const bool whole = kVec && rb * kBlock + kBlock <= p.N && cb * kBlock + kBlock <= p.d;
  if (whole) {
#pragma unroll
    for (int i = 0; i < kTileLoads; ++i) load_whole<T, kVec>(e[i], x + 16 * i * p.ldx, 8, true);
  } else {
#pragma unroll
    for (int i = 0; i < kTileLoads; ++i) {
      const int n = row0 + 16 * i < p.N ? p.d - col : 0;
      load_rest(e[i], x + 16 * i * p.ldx, n,
                load_whole<T, kVec>(e[i], x + 16 * i * p.ldx, n, row0 + 16 * i == p.N - 1));
    }
  }
  uint32_t m = kLeastMaxBits;
#pragma unroll
  for (int i = 0; i < kTileLoads; ++i) m = max(m, most(e[i]));
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kTileThreads / 32; ++i) m = max(m, warp_max[i]);
  const float top = __uint_as_float(m);
  if (threadIdx.x == 0) p.scale[int64_t(rb) * p.lds + cb] = __fdiv_rn(top, kMostE4m3);
  const float inv = __fdiv_rn(kMostE4m3, top);
  if (whole) {
#pragma unroll
    for (int i = 0; i < kTileLoads; ++i) store8<kVec>(out + 16 * i * p.ldv, 8, e[i], inv);
  } else {
#pragma unroll
    for (int i = 0; i < kTileLoads; ++i)
      if (row0 + 16 * i < p.N) store8<kVec>(out + 16 * i * p.ldv, p.d - col, e[i], inv);
  }
}

// ---------------------------------------------------------------------------
// Product
//
// Warp roles as in fs_contract.cuh: warp 0 issues TMA copies into a ring of 128-wide
// k slices (128 bytes a row, so the swizzle and the descriptors are those of 64 bf16),
// warp 1 issues the MMAs (M = 128 per CTA, kN vocabulary columns; for CTA pairs M = 256
// over both), warp 2 brings the scales, warps 4-11 take the sums out.  The scales change
// with every slice, so a slice is an accumulator of its own: the MMAs alternate over kAcc of
// them in tensor memory, and the warps add each, times the product of the two scales, to
// sums in registers.
//
// Bound: W's bytes for few rows (one row at d = 4096, V = 151936 takes 92 us, 6.75 TB/s; 128
// rows of 128256 90).  For many, what follows the MMAs: 1000 rows (CTA pairs) take 459 us in
// bursts, 2720 TFLOP/s, 800 cycles a slice; by leaving parts out in copies of the kernel, the MMAs
// with their waits alone 550 (512 at the nominal rate; a CTA's copies are 60 bytes a cycle
// then), with loads from tensor memory but no additions 733, with additions but no loads 729, all but
// outputs 752.  So neither loads nor additions by themselves bound it, but the way of an
// accumulator from the MMAs to the sums' warps and back, of which two overlap; which part of it stays
// uncovered is not known.  320 rows (single CTAs): 1012 cycles, of which 857 without the sums, at
// 57 bytes of copies a cycle.  ptxas spills 44 bytes of stores and 188 of loads in the pairs'
// kernel, 8 and 72 to 80 in the single CTAs' (in which warps is not known).
// First 1045 us: tensor-memory loads one at a time with their additions between, scales read by
// the same warps (a wait for tensor-memory loads waits for those too), outputs stored from
// registers, all lanes at every wait.  Polling is not free here: the same waits without the clock
// reads between their tries took 790 us.
// ---------------------------------------------------------------------------
using vocab::BoundedWait;
using vocab::kEpiWarps;

// Three groups of four warps, so that registers can be moved between them: the
// copying and issuing warps give theirs to the sums, 128 registers a thread.
constexpr int kThreads = 384;
constexpr int kFirstSum = 4;  // the first warp of the sums
constexpr int kIssueRegs = 56, kSumRegs = 224;
static_assert(kIssueRegs * 128 + kSumRegs * 256 <= 168 * kThreads, "registers at launch");

constexpr int kBM = 128;
constexpr int kBK = 128;          // k slice: 128 e4m3 = one 128-byte swizzle row
constexpr int kUK = 32;           // k of one MMA
constexpr int kMaxStages = 8;
constexpr uint32_t kARead = kBM * kBK;  // bytes of A an MMA reads, whatever the box holds
constexpr uint32_t kBarrierBytes = 256;
// The scales of some slices: of A's 128 rows, times W's of either half's columns.
constexpr int kGroups = 2;
constexpr int kGroupSlices = 16;
struct ScaleGroup {
  float product[2][kGroupSlices][kBM];
};
// Shared memory.  CTA pairs: 4 stages of 32 KB do as well as 6, and a second box lets a warp
// fill one while the other is stored.  Single CTAs: as much as fits, 3 to 4 stages.
constexpr uint32_t kBoxBytes = 4096;  // a warp's 32 rows x 128 bytes of output
template <bool kPair>
struct Layout {
  static constexpr uint32_t kRing = (kPair ? 128u : 160u) * 1024u;
  static constexpr int kBoxes = kPair ? 2 : 1;
  static constexpr uint32_t kBoxesAt = kRing;
  static constexpr uint32_t kScalesAt = kBoxesAt + kEpiWarps * kBoxes * kBoxBytes;
  static constexpr uint32_t kBarriersAt = kScalesAt + kGroups * uint32_t(sizeof(ScaleGroup));
  static constexpr size_t kBytes = 1024 /* alignment slack */ + kBarriersAt + kBarrierBytes;
  static_assert(kBytes <= 227 * 1024 && kScalesAt % 16 == 0 && kBarriersAt % 8 == 0, "layout");
};

template <int kN>
__host__ __device__ constexpr int accumulators() {
  return kN == 256 ? 2 : 4;
}
// Parts of an accumulator, side by side, with barriers of their own: the second part's
// MMAs run while the first one's sums are taken out, by the warps of one group each.
template <int kN>
__host__ __device__ constexpr int parts() {
  return kN == 256 ? 2 : 1;
}
// Ring stages for a box of `a_bytes` of A: the last stage's MMAs read kARead of A too.
template <int kN, bool kPair>
__host__ __device__ constexpr uint32_t ring_stages(uint32_t a_bytes) {
  const uint32_t stage = a_bytes + (kPair ? kN / 2 : kN) * kBK;
  const uint32_t past = kARead > stage ? kARead - stage : 0;
  const uint32_t n = (Layout<kPair>::kRing - past) / stage;
  return n < kMaxStages ? n : kMaxStages;
}

struct Plan {
  int32_t n_mt, n_nt, n_units;  // tiles along M (128 rows, 256 for pairs) and V; their product
  int32_t n_kb;                 // k slices
  int32_t M, V;
  uint32_t a_bytes, stage_bytes, n_stages;
  uint32_t pdl;
  const float* a_scale;
  int64_t lda_scale;
  const float* w_scale;
  int64_t ldw_scale;
  void* out;
  int64_t ldo;
  uint32_t out_f32;
  int32_t whole_v;  // columns below it go by TMA, in whole 16-byte pieces
  uint32_t scale_vec;         // both scales' rows on 16-byte boundaries
  uint64_t wait_limit_ns;
  int* error_word;
};

// How a box of output lies in shared memory: 32 columns of fp32 or 64 of bf16 a row (32
// where a warp has no more), in the store's swizzle.
template <int kCols, bool kF32>
struct Box {
  static constexpr int kSize = kF32 ? 4 : 2;
  static constexpr int kWidth = kCols * kSize < 128 ? kCols : 128 / kSize;
  static constexpr int kPitch = kWidth * kSize;
  static_assert(kPitch == 128 || kPitch == 64, "rows of the swizzle");
  // Of 16-byte chunk c of a row.
  static __device__ __forceinline__ uint32_t at(int row, int c) {
    return uint32_t(row * kPitch + ((c ^ (kPitch == 128 ? row & 7 : (row >> 1) & 3)) << 4));
  }
};

// A warp's 32 rows x kCols sums, rounded once, through its box: a lane has a row, whose
// pieces stored from registers would be 32 rows' 16 bytes at a time (4 times the store
// traffic's time; 300 cycles a slice at d = 4096).  TMA stores take them out; columns
// that it cannot write, behind the last whole 16 bytes or of rows off 16-byte boundaries,
// go row by row.
template <int kCols, bool kF32, int kBoxes>
__device__ __forceinline__ void store_sums(const Plan& s, const void* tmap, uint8_t* boxes,
                                           int lane, const float (&sum)[kCols], int row0,
                                           int col0) {
  using B = Box<kCols, kF32>;
#pragma unroll
  for (int part = 0; part < kCols / B::kWidth; ++part) {
    const int x = col0 + part * B::kWidth;
    uint8_t* box = boxes + part % kBoxes * kBoxBytes;
    // The box's last store has been read (kBoxes - 1 later ones may not).
    if (lane == 0)
      asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kBoxes - 1) : "memory");
    __syncwarp();
#pragma unroll
    for (int c = 0; c < B::kPitch / 16; ++c) {
      const float* v = sum + part * B::kWidth + c * (16 / B::kSize);
      uint4 w;
      if constexpr (kF32)
        w = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                       __float_as_uint(v[3]));
      else
        w = make_uint4(vocab::pack_bf16(v[0], v[1]), vocab::pack_bf16(v[2], v[3]),
                       vocab::pack_bf16(v[4], v[5]), vocab::pack_bf16(v[6], v[7]));
      *reinterpret_cast<uint4*>(box + B::at(lane, c)) = w;
    }
    ptx::fence_async_smem();
    __syncwarp();
    if (lane == 0) {
      if (x < s.whole_v) ptx::tma_store_2d(tmap, box, x, row0);
      ptx::bulk_commit();  // (perhaps an empty group: a box is always so many groups ago)
    }
    const int from = max(x, s.whole_v), to = min(x + B::kWidth, s.V);
    if (from < to) {
      for (int r = 0; r < 32 && row0 + r < s.M; ++r) {
        const int64_t out = int64_t(row0 + r) * s.ldo;
        for (int v = from + lane; v < to; v += 32) {
          const int byte = (v - x) * B::kSize;
          const uint8_t* p = box + B::at(r, byte >> 4) + (byte & 15);
          if constexpr (kF32)
            static_cast<float*>(s.out)[out + v] = *reinterpret_cast<const float*>(p);
          else
            static_cast<uint16_t*>(s.out)[out + v] = *reinterpret_cast<const uint16_t*>(p);
        }
      }
      __syncwarp();
    }
  }
}

// The rest of a wait whose first try failed, with BoundedWait's limit and abort flag.
__device__ __forceinline__ void wait_on(const BoundedWait& w, uint32_t bar, uint32_t parity) {
  const uint64_t t0 = ptx::global_timer_ns();
  while (!ptx::mbar_try_wait_at(bar, parity) && !*w.abort_flag) {
    if (ptx::global_timer_ns() - t0 > w.limit_ns) {
      *w.abort_flag = 1u;
      atomicOr(w.error_word, vocab::kErrWaitTimeout);
    }
  }
}

template <int kN, bool kPair>
__global__ void __launch_bounds__(kThreads, 1)
    matmul_kernel(const __grid_constant__ CUtensorMap tmap_a,
                  const __grid_constant__ CUtensorMap tmap_b,
                  const __grid_constant__ CUtensorMap tmap_o, const __grid_constant__ Plan s) {
  using L = Layout<kPair>;
  constexpr int kCtas = kPair ? 2 : 1;
  constexpr int kAcc = accumulators<kN>();
  constexpr uint32_t kTmemCols = kAcc * kN;
  constexpr int kBRows = kN / kCtas;
  constexpr uint32_t kBBytes = kBRows * kBK;
  constexpr int kCols = kN / 2;  // columns of a summing warp
  constexpr int kParts = parts<kN>();
  constexpr int kPartRows = kBRows / kParts;  // of B in this CTA's shared memory
  constexpr uint32_t kIdesc = ptx::idesc_e4m3_f32(kBM * kCtas, kN / kParts);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(smem + L::kBarriersAt);
  uint64_t* empty_bar = full_bar + kMaxStages;
  uint64_t* tfull_bar = empty_bar + kMaxStages;
  uint64_t* tempty_bar = tfull_bar + 4;  // of accumulator a, part h: [a * kParts + h]
  uint64_t* sfull_bar = tempty_bar + 4;
  uint64_t* sempty_bar = sfull_bar + kGroups;
  uint64_t* drain_bar = sempty_bar + kGroups;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain_bar + 1);
  volatile uint32_t* abort_flag = tmem_holder + 1;
  static_assert((2 * kMaxStages + 9 + 2 * kGroups) * 8 + 8 <= kBarrierBytes,
                "barriers, tensor-memory address, flag");
  ScaleGroup* groups = reinterpret_cast<ScaleGroup*>(smem + L::kScalesAt);

  // The same in all lanes, which the compiler cannot see: addresses that depend on it then
  // stay in uniform registers, as tensor-memory loads take them.
  const int warp = __shfl_sync(0xFFFFFFFFu, int(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31;
  const int rank = kPair ? int(ptx::cluster_ctarank()) : 0;
  const bool leader = rank == 0;
  const int worker = int(blockIdx.x) / kCtas;
  const int n_workers = int(gridDim.x) / kCtas;

  if (threadIdx.x == 0) {
    for (uint32_t i = 0; i < s.n_stages; ++i) {
      ptx::mbar_init(&full_bar[i], 1);
      ptx::mbar_init(&empty_bar[i], 1);
    }
    for (int a = 0; a < kAcc * kParts; ++a) {
      ptx::mbar_init(&tfull_bar[a], 1);
      ptx::mbar_init(&tempty_bar[a], kCtas * kEpiWarps / kParts);
    }
    for (int g = 0; g < kGroups; ++g) {
      ptx::mbar_init(&sfull_bar[g], 1);
      ptx::mbar_init(&sempty_bar[g], kEpiWarps);
    }
    ptx::mbar_init(drain_bar, 1);
    *abort_flag = 0u;
    ptx::fence_barrier_init();
    ptx::prefetch_tmap(&tmap_a);
    ptx::prefetch_tmap(&tmap_b);
    ptx::prefetch_tmap(&tmap_o);
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
  // The launch always overlaps the kernel before it on the stream; without the caller's
  // word only this set-up does.  Its own dependents may start once that kernel has ended (with
  // the caller's word a warp says so later): what they read ahead cannot be what a kernel
  // further back still writes.
  if (!s.pdl) {
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
  }
  const uint32_t tmem_base = *tmem_holder;
  const BoundedWait waiter{abort_flag, s.wait_limit_ns, s.error_word};

  if (warp < kFirstSum) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
    if (warp == 0) {
      // ---------------- TMA producer ----------------
      // One thread: with votes of all lanes at its waits it took 40 cycles a slice longer
      // than the MMAs.
      uint32_t issued = 0;
      if (ptx::elect_one()) {
        const uint64_t pol_a = ptx::policy_evict_last();
        const uint64_t pol_b = s.n_mt > 1 ? ptx::policy_evict_normal() : ptx::policy_evict_first();
        auto load = [&](uint8_t* dst, const CUtensorMap* map, uint32_t stage, int x, int y,
                        uint64_t pol) {
          if constexpr (kPair)
            ptx::tma_load_2d_pair(dst, map, ptx::cluster_addr(&full_bar[stage], 0), x, y, pol);
          else
            ptx::tma_load_2d(dst, map, &full_bar[stage], x, y, pol);
        };
        // Rows past the end read as 0.
        auto load_a = [&](uint32_t stage, int kb, int mt) {
          load(smem + size_t(stage) * s.stage_bytes, &tmap_a, stage, kb * kBK,
               (mt * kCtas + rank) * kBM, pol_a);
        };
        uint32_t stage = 0, phase = 0;
        bool ok = true;
        // The first ring fill's A copies, held back until the kernel before is done.
        bool deferring = s.pdl != 0;
        int n_held = 0, held_kb[kMaxStages], held_mt[kMaxStages];
        auto release = [&]() {
          ptx::grid_dependency_wait();
          for (int h = 0; h < n_held; ++h) load_a(uint32_t(h), held_kb[h], held_mt[h]);
          deferring = false;
        };
        for (int u = worker; ok && u < s.n_units; u += n_workers) {
          const int nt = u / s.n_mt, mt = u - nt * s.n_mt;
          for (int kb = 0; kb < s.n_kb; ++kb) {
            if (!waiter.wait(&empty_bar[stage], phase ^ 1u)) {
              ok = false;
              break;
            }
            if (leader)
              ptx::mbar_arrive_expect_tx(&full_bar[stage], kCtas * (s.a_bytes + kBBytes));
            // A part's columns of a pair's tile lie half in each CTA.
#pragma unroll
            for (int h = 0; h < kParts; ++h)
              load(smem + size_t(stage) * s.stage_bytes + s.a_bytes + h * kPartRows * kBK, &tmap_b,
                   stage, kb * kBK, nt * kN + h * (kN / kParts) + rank * kPartRows, pol_b);
            if (!deferring) load_a(stage, kb, mt);
            if (deferring) {  // the first fill: stage n_held
              held_kb[n_held] = kb;
              held_mt[n_held++] = mt;
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
      }
      issued = __reduce_max_sync(0xFFFFFFFFu, issued);
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
      // One thread does it all: what it takes from an accumulator's return to its next MMAs is
      // on the chain that bounds the kernel (votes of the warp's lanes at its waits: 20 cycles a
      // slice of 890).
      if (leader && ptx::elect_one()) {
        // A's copies come behind the kernel before; its time does not count against a wait's limit.
        if (s.pdl) ptx::grid_dependency_wait();
        uint32_t stage = 0, phase = 0, acc_phases = 0;  // a bit for each accumulator
        bool ok = true;
        const uint32_t s0 = ptx::smem_u32(smem);
        const uint64_t desc_a0 = ptx::smem_desc_sw128(s0);
        const uint64_t desc_b0 = ptx::smem_desc_sw128(s0 + s.a_bytes);
        auto commit = [&](uint64_t* bar) {
          if constexpr (kPair)
            ptx::mma_commit_pair_multicast(bar, 0x3);
          else
            ptx::mma_commit(bar);
        };
        for (int u = worker; ok && u < s.n_units; u += n_workers) {
          for (int kb = 0; ok && kb < s.n_kb; ++kb) {
            const uint64_t off = uint64_t((stage * s.stage_bytes) >> 4);
            const uint32_t acc = uint32_t(kb) % kAcc;  // a unit begins with the first one
            ok = waiter.wait(&full_bar[stage], phase);
#pragma unroll
            for (int h = 0; h < kParts; ++h) {
              ok = ok && waiter.wait(&tempty_bar[acc * kParts + h], (acc_phases >> acc & 1u) ^ 1u);
              if (!ok) break;
              ptx::tc_fence_after();
              const uint32_t d_tmem = tmem_base + acc * kN + h * (kN / kParts);
#pragma unroll
              for (int k = 0; k < kBK / kUK; ++k) {
                const uint64_t da = desc_a0 + off + uint64_t(kUK >> 4) * k;
                const uint64_t db =
                    desc_b0 + off + uint64_t(h * ((kPartRows * kBK) >> 4) + (kUK >> 4) * k);
                if constexpr (kPair)
                  ptx::mma_f8_pair(d_tmem, da, db, kIdesc, k != 0 ? 1u : 0u);
                else
                  ptx::mma_f8(d_tmem, da, db, kIdesc, k != 0 ? 1u : 0u);
              }
              commit(&tfull_bar[acc * kParts + h]);
              if (h == kParts - 1) commit(&empty_bar[stage]);
            }
            if (++stage == s.n_stages) {
              stage = 0;
              phase ^= 1u;
            }
            acc_phases ^= 1u << acc;
          }
        }
        // All MMAs complete before tensor memory is released.
        if constexpr (kPair)
          ptx::mma_commit_pair(drain_bar);
        else
          ptx::mma_commit(drain_bar);
      }
      __syncwarp();
      if (leader) waiter.drain(drain_bar, 0);
      __syncwarp();
    } else if (warp == 2) {
      // ---------------- scales ----------------
      // From memory by a warp of its own: a wait for tensor-memory loads waits for a
      // warp's loads from memory too (450 cycles every four slices).
      if (s.pdl) {
        ptx::grid_dependency_wait();
        ptx::grid_launch_dependents();
      }
      uint32_t g = 0, phase = 0;
      bool ok = true;
      for (int u = worker; ok && u < s.n_units; u += n_workers) {
        const int nt = u / s.n_mt, mt = u - nt * s.n_mt;
        const int row0 = (mt * kCtas + rank) * kBM;
        for (int kb0 = 0; kb0 < s.n_kb; kb0 += kGroupSlices) {
          if (!waiter.wait_warp(&sempty_bar[g], phase ^ 1u)) {
            ok = false;
            break;
          }
          const int end = min(s.n_kb, kb0 + kGroupSlices);
          for (int kb = kb0; kb < end; kb += 4) {
            const int n = min(4, end - kb);
            float v[4][4], w[2][4];
            auto four = [&](const float* p, float (&x)[4]) {
              if (s.scale_vec && n == 4) {
                const float4 f = *reinterpret_cast<const float4*>(p);
                x[0] = f.x, x[1] = f.y, x[2] = f.z, x[3] = f.w;
              } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = i < n ? p[i] : 0.0f;
              }
            };
#pragma unroll
            for (int j = 0; j < 4; ++j)
              four(s.a_scale + int64_t(min(row0 + 32 * j + lane, s.M - 1)) * s.lda_scale + kb,
                   v[j]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int row = min(nt * kN + h * kCols, s.V - 1) / kBlock;
              four(s.w_scale + int64_t(row) * s.ldw_scale + kb, w[h]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                groups[g].product[0][kb - kb0 + i][32 * j + lane] = v[j][i] * w[0][i];
                groups[g].product[1][kb - kb0 + i][32 * j + lane] = v[j][i] * w[1][i];
              }
            }
          }
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&sfull_bar[g]);
          if (++g == kGroups) {
            g = 0;
            phase ^= 1u;
          }
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSumRegs));
    // ---------------- sums ----------------
    if (s.pdl) ptx::grid_dependency_wait();  // before the first output
    const int quad = warp & 3;  // the tensor-memory lane quadrant this warp may read
    const int half = (warp - kFirstSum) >> 2;
    constexpr int kChunks = kCols / 32;
    const uint32_t taddr0 = tmem_base + (uint32_t(quad * 32) << 16) + uint32_t(half * kCols);
    const int part = kParts == 2 ? half : 0;
    const uint32_t tfull0 = ptx::smem_u32(tfull_bar + part);
    const uint32_t tempty0 = ptx::cluster_addr(tempty_bar + part, 0);
    const uint32_t sfull0 = ptx::smem_u32(sfull_bar), sempty0 = ptx::smem_u32(sempty_bar);
    const uint32_t scales0 = ptx::smem_u32(&groups[0].product[half][0][quad * 32 + lane]);
    uint32_t acc_phases = 0, group = 0, group_phase = 0;
    // Past its limit a wait raises the abort flag and returns, and so does every later one
    // at once: the loops end, with the error reported and sums of no use.
    auto wait = [&](uint32_t bar, uint32_t parity) {
      if (!ptx::mbar_try_wait_at(bar, parity)) wait_on(waiter, bar, parity);
      __syncwarp();
    };
    // An accumulator goes back once its last load has completed (the wait for that is
    // the whole warp's), a group of scales with its last one.
    auto arrive = [&](uint32_t bar) {
      if (lane == 0) ptx::mbar_arrive_cluster_relaxed(bar);
    };
    auto next_group = [&]() {
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive_at(sempty0 + 8u * group);
      if (++group == kGroups) {
        group = 0;
        group_phase ^= 1u;
      }
    };
    for (int u = worker; u < s.n_units; u += n_workers) {
      const int nt = u / s.n_mt, mt = u - nt * s.n_mt;
      const int row0 = (mt * kCtas + rank) * kBM + quad * 32;
      const int col0 = nt * kN + half * kCols;
      if (row0 >= s.M || col0 >= s.V) {  // nothing here
        for (int kb = 0; kb < s.n_kb; ++kb) {
          const uint32_t acc = uint32_t(kb) % kAcc;
          wait(tfull0 + 8u * kParts * acc, acc_phases >> acc & 1u);
          acc_phases ^= 1u << acc;
          ptx::tc_fence_before();
          arrive(tempty0 + 8u * kParts * acc);
          if (kb % kGroupSlices == kGroupSlices - 1 || kb + 1 == s.n_kb) {
            wait(sfull0 + 8u * group, group_phase);
            next_group();
          }
        }
        continue;
      }
      uint64_t sums[kCols / 2];
#pragma unroll
      for (int i = 0; i < kCols / 2; ++i) sums[i] = 0ull;
      uint32_t r[2][32];
      auto add = [&](int c, float scale) {
        const uint64_t f = ptx::pack2(__float_as_uint(scale), __float_as_uint(scale));
#pragma unroll
        for (int i = 0; i < 16; ++i)
          ptx::fma2(sums[c * 16 + i], ptx::pack2(r[c & 1][2 * i], r[c & 1][2 * i + 1]), f);
      };
      wait(sfull0 + 8u * group, group_phase);
      uint32_t scale_at = scales0 + group * uint32_t(sizeof(ScaleGroup));
      float scale = ptx::ld_shared_f32(scale_at);
      wait(tfull0, acc_phases & 1u);
      acc_phases ^= 1u;
      ptx::tc_fence_after();
      ptx::tmem_ld_32x32b_x32(taddr0, r[0]);
      if (kChunks > 1) ptx::tmem_ld_32x32b_x32(taddr0 + 32u, r[1]);
      // A slice, from accumulator a; `more`: another one of the unit follows.  Loads go out as
      // soon as their registers are free, 32 columns at a time, the next slice's first ones
      // beside the last additions of this one's.  A unit begins with the first accumulator,
      // so that every address is known ahead (made from a counter they held the loads up by
      // 100 cycles).
      auto slice = [&](int kb, auto which, bool more) {
        constexpr int a = decltype(which)::value;
        constexpr int next = (a + 1) % kAcc;
        float scale_next = 0.0f;
        if (more) {
          scale_at += kBM * 4;
          if (kb % kGroupSlices == kGroupSlices - 1) {
            next_group();
            wait(sfull0 + 8u * group, group_phase);
            scale_at = scales0 + group * uint32_t(sizeof(ScaleGroup));
          }
        }
        ptx::tmem_wait_ld();
#pragma unroll
        for (int c = 2; c < kChunks; ++c) {
          add(c - 2, scale);
          ptx::tmem_ld_32x32b_x32(taddr0 + uint32_t(a * kN + c * 32), r[c & 1]);
        }
        if (more) scale_next = ptx::ld_shared_f32(scale_at);
        if (kChunks > 2) ptx::tmem_wait_ld();
        ptx::tc_fence_before();
        arrive(tempty0 + uint32_t(8 * kParts * a));
        if (kChunks > 1) add(kChunks - 2, scale);
        if (more) {
          wait(tfull0 + uint32_t(8 * kParts * next), acc_phases >> next & 1u);
          acc_phases ^= 1u << next;
          ptx::tc_fence_after();
          if (kChunks > 1) ptx::tmem_ld_32x32b_x32(taddr0 + uint32_t(next * kN), r[0]);
        }
        add(kChunks - 1, scale);
        if (more) {
          if (kChunks > 1)
            ptx::tmem_ld_32x32b_x32(taddr0 + uint32_t(next * kN) + 32u, r[1]);
          else
            ptx::tmem_ld_32x32b_x32(taddr0 + uint32_t(next * kN), r[0]);
        }
        scale = scale_next;
      };
#pragma unroll 1
      for (int kb = 0; kb < s.n_kb; kb += kAcc) {
        slice(kb, std::integral_constant<int, 0>(), kb + 1 < s.n_kb);
        if (kb + 1 < s.n_kb) slice(kb + 1, std::integral_constant<int, 1>(), kb + 2 < s.n_kb);
        if constexpr (kAcc == 4) {
          if (kb + 2 < s.n_kb) slice(kb + 2, std::integral_constant<int, 2>(), kb + 3 < s.n_kb);
          if (kb + 3 < s.n_kb) slice(kb + 3, std::integral_constant<int, 3>(), kb + 4 < s.n_kb);
        }
      }
      next_group();
      float sum[kCols];
#pragma unroll
      for (int i = 0; i < kCols / 2; ++i) ptx::unpack2(sums[i], sum[2 * i], sum[2 * i + 1]);
      uint8_t* box = smem + L::kBoxesAt + (warp - kFirstSum) * (L::kBoxes * kBoxBytes);
      if (s.out_f32)
        store_sums<kCols, true, L::kBoxes>(s, &tmap_o, box, lane, sum, row0, col0);
      else
        store_sums<kCols, false, L::kBoxes>(s, &tmap_o, box, lane, sum, row0, col0);
    }
    if (lane == 0) ptx::bulk_wait();
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
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

constexpr int kMaxDevices = 64;
constexpr int64_t kMost = INT_MAX - 512;  // sizes, so that a tile's end fits 32 bits
constexpr uint64_t kWaitLimitNs = 2000000000ull;  // 2 s

struct Device {
  bool initialised = false;
  fs_status status = FS_ERR_UNSUPPORTED;
  int sms = 0, pairs = 0;
  EncodeTiledFn encode = nullptr;
  int* error_word = nullptr;
};
std::mutex g_mu;
Device g_devices[kMaxDevices];

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t element(int dtype) { return dtype == FS_F32 ? 4 : 2; }
bool known(int dtype) { return dtype == FS_BF16 || dtype == FS_F32; }

template <int kN, bool kPair>
bool prepare_kernel(int sms, int* pairs) {
  auto k = matmul_kernel<kN, kPair>;
  if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           int(Layout<kPair>::kBytes)) != cudaSuccess)
    return false;
  if (!kPair) return true;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 2;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.gridDim = dim3(unsigned(sms / 2 * 2), 1, 1);
  cfg.dynamicSmemBytes = Layout<kPair>::kBytes;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, k, &cfg) != cudaSuccess || n < 1) return false;
  *pairs = std::min(*pairs, n);
  return true;
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
  if (!d.initialised) {
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
      cudaGetLastError();
      return FS_ERR_CUDA;
    }
    d.status = FS_ERR_UNSUPPORTED;
    if (major == 10 && minor == 3) {
      d.pairs = d.sms / 2;
      void* fn = nullptr;
      cudaDriverEntryPointQueryResult q;
      d.error_word = device_error_word();
      const bool ok = d.error_word != nullptr && prepare_kernel<64, false>(d.sms, &d.pairs) &&
                      prepare_kernel<128, false>(d.sms, &d.pairs) &&
                      prepare_kernel<256, false>(d.sms, &d.pairs) &&
                      prepare_kernel<256, true>(d.sms, &d.pairs) &&
                      cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000,
                                                       cudaEnableDefault, &q) == cudaSuccess &&
                      q == cudaDriverEntryPointSuccess && fn != nullptr;
      cudaGetLastError();
      d.encode = reinterpret_cast<EncodeTiledFn>(fn);
      d.status = ok ? FS_OK : FS_ERR_CUDA;
    }
    d.initialised = true;
  }
  *out = &d;
  return d.status;
}

// 2-D tensor map with boxes of `width` x `rows` elements, swizzled over their rows of 64
// or 128 bytes; elements past the extents read as zero and are not written.
bool encode(const Device& dev, CUtensorMap* m, CUtensorMapDataType type, int size,
            const void* base, int64_t inner, int64_t outer, int64_t ld, int width, int rows) {
  const cuuint64_t dims[2] = {cuuint64_t(inner), cuuint64_t(outer)};
  const cuuint64_t strides[1] = {cuuint64_t(ld) * unsigned(size)};
  const cuuint32_t box[2] = {cuuint32_t(width), cuuint32_t(rows)};
  const cuuint32_t estr[2] = {1, 1};
  return dev.encode(m, type, 2, const_cast<void*>(base), dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE,
                    width * size == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The smallest number of workers that needs no more waves than all of them.
int balanced(int64_t units, int workers) {
  if (units <= workers) return int(units);
  return int(ceil_div(units, ceil_div(units, workers)));
}

template <int kN, bool kPair>
fs_status launch(const Device& dev, const fs_matmul_fp8_args& a, Plan s, cudaStream_t stream) {
  const int64_t n_mt = ceil_div(a.M, kPair ? 2 * kBM : kBM), n_nt = ceil_div(a.V, kN);
  if (n_mt * n_nt > INT_MAX - 1024) return FS_ERR_INVALID_ARG;  // past it by a stride
  s.n_mt = int32_t(n_mt);
  s.n_nt = int32_t(n_nt);
  s.n_units = int32_t(n_mt * n_nt);
  const int box_rows = int(std::min<int64_t>(kBM, ceil_div(a.M, 8) * 8));
  s.a_bytes = uint32_t(box_rows) * kBK;
  s.stage_bytes = s.a_bytes + (kPair ? kN / 2 : kN) * kBK;
  s.n_stages = ring_stages<kN, kPair>(s.a_bytes);
  CUtensorMap ta, tb, to;
  // Of a single row the stride is any that the map takes.
  const int64_t lda = a.M > 1 ? a.lda : ceil_div(a.d, 16) * 16;
  const int64_t ldw = a.V > 1 ? a.ldw : ceil_div(a.d, 16) * 16;
  const auto bytes = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  if (!encode(dev, &ta, bytes, 1, a.A, a.d, a.M, lda, kBK, box_rows) ||
      !encode(dev, &tb, bytes, 1, a.W, a.d, a.V, ldw, kBK,
              (kPair ? kN / 2 : kN) / parts<kN>()))
    return FS_ERR_CUDA;
  to = tb;  // where nothing goes by it
  if (s.whole_v > 0) {
    const int64_t ldo = a.M > 1 ? a.ldo : ceil_div(a.V, 8) * 8;
    const auto type =
        s.out_f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const int width = s.out_f32 ? Box<kN / 2, true>::kWidth : Box<kN / 2, false>::kWidth;
    if (!encode(dev, &to, type, s.out_f32 ? 4 : 2, a.out, s.whole_v, a.M, ldo, width, 32))
      return FS_ERR_CUDA;
  }
  cudaLaunchAttribute attr[2];
  unsigned n = 0;
  if (kPair) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = 2;
    attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
    ++n;
  }
  attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[n].val.programmaticStreamSerializationAllowed = 1;
  ++n;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(balanced(s.n_units, kPair ? dev.pairs : dev.sms) * (kPair ? 2 : 1)));
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = Layout<kPair>::kBytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = n;
  if (cudaLaunchKernelEx(&cfg, matmul_kernel<kN, kPair>, ta, tb, to, s) != cudaSuccess) {
    cudaGetLastError();
    return FS_ERR_CUDA;
  }
  return FS_OK;
}

// Rows' blocks a thread takes: one while they leave SMs without work, else two (four loads
// in flight).
int64_t blocks_per_thread(int64_t blocks, int sms) {
  return blocks >= int64_t(sms) * 16 * kRowBlocks * 2 ? 2 : 1;
}

template <class T, bool kVec>
void launch_quantize(const QuantParams& p, int block_rows, int64_t per, unsigned ctas,
                     cudaStream_t stream) {
  if (block_rows != 1)
    quantize_tile_kernel<T, kVec><<<ctas, kTileThreads, 0, stream>>>(p);
  else if (per == 2)
    quantize_rows_kernel<T, kVec, 2><<<ctas, kRowThreads, 0, stream>>>(p);
  else
    quantize_rows_kernel<T, kVec, 1><<<ctas, kRowThreads, 0, stream>>>(p);
}

}  // namespace
}  // namespace fp8
}  // namespace fs

using namespace fs::fp8;

extern "C" fs_status fs_quantize(const void* x, int64_t N, int64_t d, int64_t ldx, int x_dtype,
                                 int block_rows, void* values, int64_t ldv, float* scale,
                                 int64_t lds, void* stream_ptr) {
  if (N < 0 || N > INT_MAX - kBlock || d < 1 || d > INT_MAX - kBlock || !known(x_dtype) ||
      (block_rows != 1 && block_rows != kBlock))
    return FS_ERR_INVALID_ARG;
  if (N == 0) return FS_OK;
  const int64_t col_blocks = ceil_div(d, kBlock);
  if ((N > 1 && (ldx < d || ldv < d)) || (N > block_rows && lds < col_blocks))
    return FS_ERR_INVALID_ARG;
  if (!x || !values || !scale || !aligned(x, element(x_dtype)) || !aligned(scale, 4))
    return FS_ERR_INVALID_ARG;
  const int64_t all = N * col_blocks;
  if ((block_rows == 1 ? ceil_div(all, kRowBlocks) : ceil_div(N, kBlock) * col_blocks) >
      INT_MAX)
    return FS_ERR_INVALID_ARG;
  const Device* dev = nullptr;
  const fs_status st = device_setup(&dev);
  if (st != FS_OK) return st;
  const int64_t per = blocks_per_thread(all, dev->sms);
  const unsigned ctas = unsigned(block_rows == 1 ? ceil_div(all, kRowBlocks * per)
                                                 : ceil_div(N, kBlock) * col_blocks);
  QuantParams p = {};
  p.x = x;
  p.ldx = N > 1 ? ldx : 0;
  p.values = static_cast<uint8_t*>(values);
  p.ldv = N > 1 ? ldv : 0;
  p.scale = scale;
  p.lds = lds;
  p.N = int32_t(N);
  p.d = int32_t(d);
  p.col_blocks = int32_t(col_blocks);
  const bool vec = whole_pieces(reinterpret_cast<uintptr_t>(x), N, p.ldx, int(element(x_dtype))) &&
                   aligned(values, 8) && p.ldv % 8 == 0;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  if (x_dtype == FS_F32)
    vec ? launch_quantize<float, true>(p, block_rows, per, ctas, stream)
        : launch_quantize<float, false>(p, block_rows, per, ctas, stream);
  else
    vec ? launch_quantize<__nv_bfloat16, true>(p, block_rows, per, ctas, stream)
        : launch_quantize<__nv_bfloat16, false>(p, block_rows, per, ctas, stream);
  return cudaGetLastError() == cudaSuccess ? FS_OK : FS_ERR_CUDA;
}

extern "C" fs_status fs_matmul_fp8(const fs_matmul_fp8_args* args, void* stream_ptr) {
  if (!args) return FS_ERR_INVALID_ARG;
  const fs_matmul_fp8_args& a = *args;
  if (a.M < 0 || a.M > kMost || a.d < 1 || a.d > kMost || a.V < 1 || a.V > kMost ||
      !known(a.out_dtype) || (a.flags & ~FS_FLAG_OVERLAP_PREVIOUS))
    return FS_ERR_INVALID_ARG;
  if (ceil_div(a.M, kBM) * ceil_div(a.V, 64) > INT_MAX) return FS_ERR_INVALID_ARG;
  if (a.M == 0) return FS_OK;
  const int64_t n_kb = ceil_div(a.d, kBK);
  if ((a.M > 1 && (a.lda < a.d || a.lda % 16 || a.lda_scale < n_kb || a.ldo < a.V)) ||
      (a.V > 1 && (a.ldw < a.d || a.ldw % 16)) || (a.V > kBlock && a.ldw_scale < n_kb))
    return FS_ERR_INVALID_ARG;
  if (!a.A || !a.a_scale || !a.W || !a.w_scale || !a.out || !aligned(a.A, 16) ||
      !aligned(a.W, 16) || !aligned(a.a_scale, 4) || !aligned(a.w_scale, 4) ||
      !aligned(a.out, element(a.out_dtype)))
    return FS_ERR_INVALID_ARG;
  const Device* dev = nullptr;
  const fs_status st = device_setup(&dev);
  if (st != FS_OK) return st;
  Plan s = {};
  s.n_kb = int32_t(n_kb);
  s.M = int32_t(a.M);
  s.V = int32_t(a.V);
  s.pdl = (a.flags & FS_FLAG_OVERLAP_PREVIOUS) ? 1u : 0u;
  s.a_scale = a.a_scale;
  s.lda_scale = a.lda_scale;
  s.w_scale = a.w_scale;
  s.ldw_scale = a.ldw_scale;
  s.out = a.out;
  s.ldo = a.M > 1 ? a.ldo : 0;
  s.out_f32 = a.out_dtype == FS_F32;
  const int64_t piece = 16 / element(a.out_dtype);
  if (aligned(a.out, 16) && s.ldo % piece == 0) s.whole_v = int32_t(a.V / piece * piece);
  s.scale_vec = aligned(a.a_scale, 16) && aligned(a.w_scale, 16) &&
                (a.M == 1 || a.lda_scale % 4 == 0) && (a.V <= kBlock || a.ldw_scale % 4 == 0);
  s.wait_limit_ns = kWaitLimitNs;
  s.error_word = dev->error_word;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  // Few units leave SMs without work: the widest that still gives each SM one.
  const int64_t n_mt = ceil_div(a.M, kBM);
  if (n_mt * ceil_div(a.V, 64) <= dev->sms) return launch<64, false>(*dev, a, s, stream);
  if (n_mt * ceil_div(a.V, 128) <= dev->sms) return launch<128, false>(*dev, a, s, stream);
  if (a.M <= kBM) return launch<256, false>(*dev, a, s, stream);
  // CTA pairs read W once for 256 rows, but take 256 at a time.  Where the last ones are few,
  // single CTAs need fewer turns, each 1.25 times as long: at d = 4096, V = 128256, pairs / single
  // CTAs in bursts (held at the power limit), 200 rows 111 / 136 us (123 / 141), 320 200 / 181 (213 /
  // 193), 384 202 / 184, 450 205 / 242, 600 286 / 292 (317 / 312), 1000 (V = 151936) 458 / 537 (528 /
  // 592).
  const int64_t n_nt = ceil_div(a.V, 256);
  const int64_t pair_turns = ceil_div(ceil_div(a.M, 2 * kBM) * n_nt, dev->pairs);
  const int64_t single_turns = ceil_div(n_mt * n_nt, dev->sms);
  return single_turns * 5 < pair_turns * 4 ? launch<256, false>(*dev, a, s, stream)
                                           : launch<256, true>(*dev, a, s, stream);
}
