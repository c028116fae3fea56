// fs_logprobs.cu -- token log-probabilities, entropy and top alternatives from
// hidden states and the LM head, and their gradient (fs_vocab.h).
//
// Forward, two kernels.  The contraction kernel (fs_contract.cuh) streams W
// past a block of rows; a CTA (pair) keeps its block of rows for the whole
// launch, so each epilogue thread owns one row and half of the vocabulary
// blocks its CTA visits, and carries in registers, in one pass over its logits,
//   m = max x,  S = sum 2^(x-m),  U = sum 2^(x-m) (x-m)      (x in base-2 units)
// and the best KC raw logits with their ids (without alternatives, one id near the
// maximum).  A second kernel joins the threads' states of a row, sums the logits of the
// ids that decide it again in compensated fp32, puts their terms into the sums in place of
// the tensor core's, and ranks the alternatives.
//
// Backward, three contractions: G = dLoss/dlogits in bf16 (the logits again,
// turned into G in the epilogue), dH = G W, dW = G^T H.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "fs_contract.cuh"
#include "fs_vocab.h"

namespace fs {

int* device_error_word();  // fs_sample.cu

namespace vocab {
namespace {

// Workspaces and k splits are planned for this many SMs (GB300); a device that
// offers fewer co-resident CTA pairs uses less of them.
constexpr int kPlanSms = 152;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// The tensor core adds 16 products to the fp32 accumulator at a time and cuts
// the sum off towards zero, so a logit comes out short by about half a unit in
// the accumulator's last place per step: measured over heads of d = 256 to 5120,
// 1.55e-8 (0.26 2^-24) of the logit per step of 16 -- 4e-6 at d = 4096, a bias
// that does not average out of the log-sum-exp.  The scale that turns logits
// into base-2 units carries the mean of it.  That mean is a fact of sums of many
// terms of either sign: one logit differs from it by a quarter, and sums that are
// exact on the way (hidden states of few non-zeros) are not cut off at all.  So
// what single ids decide does not rest on it: the terms of the token, the
// candidates (without any, of an id near the row's maximum) in a row's sums, and G
// at the token, come from logits summed again in compensated fp32.
constexpr float kCutPerStep = 1.55e-8f;
__device__ __forceinline__ float mean_cut(int n_kb) {
  return kCutPerStep * float(n_kb * (kBK / kUK));
}
__device__ __forceinline__ float scale_to_log2(float T, int n_kb) {
  return kLog2e / T * (1.0f + mean_cut(n_kb));
}

__device__ __forceinline__ float row_temperature(const float* temperature, int row) {
  const float T = temperature ? temperature[row] : 1.0f;
  // (1 / T has to be finite.)
  return (T > 0.0f && !isinf(T)) ? fmaxf(T, 0x1p-126f) : 1.0f;
}

// The allow-words of one row's 128 ids from v0, ids at or past V cleared.
struct AllowWords {
  uint32_t w[4];
  __device__ __forceinline__ AllowWords(const uint32_t* mrow, int v0, int V) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int n = V - (v0 + c * 32);
      w[c] = n <= 0 ? 0u : (mrow != nullptr ? mrow[(v0 >> 5) + c] : 0xFFFFFFFFu);
      if (n > 0 && n < 32) w[c] &= (1u << n) - 1u;
    }
  }
  __device__ __forceinline__ uint32_t at(int c) const {
    return c == 0 ? w[0] : c == 1 ? w[1] : c == 2 ? w[2] : w[3];
  }
};

// ---------------------------------------------------------------------------
// Forward: row statistics and candidates
// ---------------------------------------------------------------------------

// One thread's state of a row, as left in the workspace: m the largest raw logit.
struct RowPart {
  float m, S, U;
  float at_token;  // the raw logit of the row's token, -inf if it is not the thread's
};
// Without lists, an id near the thread's maximum.
struct RowRef {
  float val;  // its raw logit
  int32_t id;  // -1 for none
};

// Insert (v, id) into a list sorted by decreasing value whose last entry it
// beats; equal values keep their order, so with ids visited in increasing
// order the lower id stays first.
template <int KC>
__device__ __forceinline__ void list_insert(float (&ts)[KC], int32_t (&ti)[KC], float v,
                                            int32_t id) {
#pragma unroll
  for (int q = KC - 1; q > 0; --q) {
    const bool here = v > ts[q], above = v > ts[q - 1];
    ts[q] = above ? ts[q - 1] : here ? v : ts[q];
    ti[q] = above ? ti[q - 1] : here ? id : ti[q];
  }
  const bool first = v > ts[0];
  ts[0] = first ? v : ts[0];
  ti[0] = first ? id : ti[0];
}

// v[j] for a lane-varying j without local memory.
__device__ __forceinline__ float pick32(const uint32_t (&v)[32], uint32_t j) {
  uint32_t a[16];
#pragma unroll
  for (int q = 0; q < 16; ++q) a[q] = (j & 16u) ? v[q + 16] : v[q];
#pragma unroll
  for (int q = 0; q < 8; ++q) a[q] = (j & 8u) ? a[q + 8] : a[q];
#pragma unroll
  for (int q = 0; q < 4; ++q) a[q] = (j & 4u) ? a[q + 4] : a[q];
#pragma unroll
  for (int q = 0; q < 2; ++q) a[q] = (j & 2u) ? a[q + 2] : a[q];
  return __uint_as_float((j & 1u) ? a[1] : a[0]);
}

// A logit as a sort key: an order-preserving unsigned integer whose low 7 bits
// hold 127 - j, so that of equal values the one at the lower column j < 128 is
// the greater.  The value's own low 7 bits go (it is rounded down to 17 bits), so
// keys only show an order between different steps of 2^-16 of the value: see
// ScoreEpi::fill.  0: no candidate (-inf, NaN).
__device__ __forceinline__ uint32_t sort_key(uint32_t bits, int j) {
  const float f = __uint_as_float(bits) + 0.0f;  // -0 counts as +0
  const uint32_t b = __float_as_uint(f);
  const uint32_t u = b ^ (uint32_t(int32_t(b) >> 31) | 0x80000000u);
  return f > -INFINITY ? (u & ~127u) | uint32_t(127 - j) : 0u;
}
__device__ __forceinline__ int key_column(uint32_t key) { return 127 - int(key & 127u); }

// Bitonic networks on 32 keys in registers, largest first.
__device__ __forceinline__ void order_pair(uint32_t& a, uint32_t& b) {
  const uint32_t hi = max(a, b), lo = min(a, b);
  a = hi;
  b = lo;
}
__device__ __forceinline__ void sort32(uint32_t (&k)[32]) {
#pragma unroll
  for (int size = 2; size <= 32; size *= 2) {
#pragma unroll
    for (int step = size / 2; step > 0; step /= 2) {
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        if ((i & step) != 0) continue;
        if ((i & size) == 0)
          order_pair(k[i], k[i + step]);
        else
          order_pair(k[i + step], k[i]);
      }
    }
  }
}
// The 32 largest of two sorted lists, sorted, into a.
__device__ __forceinline__ void merge32(uint32_t (&a)[32], const uint32_t (&b)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) a[i] = max(a[i], b[31 - i]);
#pragma unroll
  for (int step = 16; step > 0; step /= 2) {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if ((i & step) == 0) order_pair(a[i], a[i + step]);
  }
}

struct ScoreParams {
  int32_t B, V;  // rows of this launch, ids
  const float* temperature;
  const uint32_t* mask;
  int64_t mask_ld;
  const int64_t* tokens;  // or null
  int64_t vocab_offset;
  RowPart* part;     // [B][n_slots]
  RowRef* ref;       // KC = 0: [B][n_slots]
  float* cand_val;   // [B][n_slots][KC] raw logits, best first
  int32_t* cand_id;  // ids from 0, -1 past the end
  int32_t n_slots;
  bool sorted_start;  // the lists are filled by ScoreEpi::fill
};

template <int KC, int kCols>
struct ScoreEpi {
  static constexpr int kN = kCols;
  static constexpr bool kStaged = false;
  using Params = ScoreParams;
  struct State {
    float m = -INFINITY, S = 0.0f, U = 0.0f;  // m: the largest raw logit
    float scale2 = 0.0f;                      // log2(e) / T
    const uint32_t* mrow = nullptr;
    int row = -1;
    int32_t token = -1;  // id from 0, -1 for none
    float at_token = -INFINITY;
    RowRef ref{-INFINITY, -1};  // KC = 0
    bool first = true;  // no unit seen yet
    float ts[KC > 0 ? KC : 1];
    int32_t ti[KC > 0 ? KC : 1];
  };
  static __device__ __forceinline__ void start(const Params&, State& st, int, int,
                                               const Shape&) {
#pragma unroll
    for (int q = 0; q < KC; ++q) {
      st.ts[q] = -INFINITY;
      st.ti[q] = -1;
    }
  }
  static __device__ __forceinline__ void before(const Params&, State&, const TileAt&, int, int,
                                                const Shape&) {}
  // 32 logits; returns the largest.  kMasked: a cleared id's logit counts as -inf,
  // whatever it is.
  template <bool kMasked>
  static __device__ __forceinline__ float chunk(State& st, uint32_t (&r)[32], uint32_t allow) {
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      if (kMasked) r[j] = ((allow >> j) & 1u) ? r[j] : 0xFF800000u;
      top = ptx::max_nan(top, __uint_as_float(r[j]));
    }
    if (top == -INFINITY) return top;  // nothing allowed (false for NaN)
    const float m = ptx::max_nan(st.m, top);
    float acc = 0.0f, ent = 0.0f;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      // Far below the maximum 2^t is 0 in fp32; the bound keeps 0 * -inf out of
      // U.  (The difference first: the maximum's own t is exactly 0, so a row
      // that allows one id has entropy 0.)
      const float t = ptx::max_nan((__uint_as_float(r[j]) - m) * st.scale2, -16384.0f);
      const float e = ptx::ex2(t);
      acc += e;
      ent = fmaf(e, t, ent);
    }
    const float shift = ptx::max_nan((st.m - m) * st.scale2, -16384.0f);
    if (st.m == -INFINITY) {  // the row's first chunk
      st.S = acc;
      st.U = ent;
    } else {
      const float f = ptx::ex2(shift);
      st.U = fmaf(f, fmaf(shift, st.S, st.U), ent);
      st.S = fmaf(f, st.S, acc);
    }
    st.m = m;
    return top;
  }
  // The list from the first unit's logits: sorted by key, 32 at a time, and merged; then
  // the values of the KC + 4 best keys are fetched (by their columns, from a copy of each
  // chunk in local memory) and put in order where they share a step.  False, with the
  // list empty, if for some lane more than 4 keys beyond those it keeps share the step
  // of the last it keeps: a larger logit may have been dropped.  Inserting one by one, as is done
  // then, is slower where the first unit's logits hold the rest up (16 rows, d = 1024,
  // V = 30000, K = 20, one unit a CTA: 56 us a call against 34.5, 1.7 of these for the
  // values); so is sorting whole values with their columns, 64-bit keys (18 us more).
  static __device__ __forceinline__ bool fill(const Params& p, State& st, const TileAt& at,
                                              const AllowWords& allow, bool valid) {
    constexpr int kFetch = KC + 4;
    uint32_t best[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) best[i] = 0u;
#pragma unroll 1
    for (int c = 0; c < kN / 64; ++c) {
      if (at.col0 + c * 32 >= p.V) break;
      uint32_t r[32];
      ptx::tmem_ld_32x32b_x32(at.taddr + uint32_t(c * 32), r);
      ptx::tmem_wait_ld();
      const uint32_t w = valid ? allow.at(c) : 0u;
#pragma unroll
      for (int j = 0; j < 32; ++j) r[j] = ((w >> j) & 1u) ? sort_key(r[j], c * 32 + j) : 0u;
      sort32(r);
      merge32(best, r);
    }
    const bool open = best[kFetch] != 0u && (best[kFetch] ^ best[KC - 1]) < 128u;
    if (__any_sync(0xFFFFFFFFu, open)) return false;
    float v[kFetch];
#pragma unroll
    for (int q = 0; q < kFetch; ++q) v[q] = -INFINITY;
#pragma unroll 1
    for (int c = 0; c < kN / 64; ++c) {
      if (at.col0 + c * 32 >= p.V) break;
      uint32_t r[32];
      ptx::tmem_ld_32x32b_x32(at.taddr + uint32_t(c * 32), r);
      ptx::tmem_wait_ld();
#pragma unroll
      for (int q = 0; q < kFetch; ++q) {
        const int col = key_column(best[q]);
        if (best[q] != 0u && (col >> 5) == c) v[q] = __uint_as_float(r[col & 31]) + 0.0f;
      }
    }
    // Neighbours of one step change places, at most kFetch rounds; equal values stay in
    // the order of their columns.
    while (true) {
      bool rising = false;
#pragma unroll
      for (int q = 0; q + 1 < kFetch; ++q) rising |= v[q] < v[q + 1];
      if (!__any_sync(0xFFFFFFFFu, rising)) break;
#pragma unroll
      for (int odd = 0; odd < 2; ++odd)
#pragma unroll
        for (int q = odd; q + 1 < kFetch; q += 2) {
          const bool swap = v[q] < v[q + 1];
          const float a = v[q], b = v[q + 1];
          const uint32_t ka = best[q], kb = best[q + 1];
          v[q] = swap ? b : a;
          v[q + 1] = swap ? a : b;
          best[q] = swap ? kb : ka;
          best[q + 1] = swap ? ka : kb;
        }
    }
#pragma unroll
    for (int q = 0; q < KC; ++q) {
      st.ts[q] = v[q];
      st.ti[q] = best[q] != 0u ? at.col0 + key_column(best[q]) : -1;
    }
    return true;
  }
  template <class Release>
  static __device__ __forceinline__ void tile(const Params& p, State& st, const TileAt& at,
                                              int lane, uint8_t*, const void*, const Shape& s,
                                              Release release) {
    const int row = at.row0 + lane;
    const bool valid = row < p.B;
    if (valid && st.row < 0) {  // the thread's row, the same in every unit
      st.row = row;
      st.scale2 = scale_to_log2(row_temperature(p.temperature, row), s.n_kb);
      if (p.mask) st.mrow = p.mask + int64_t(row) * p.mask_ld;
      if (p.tokens) {
        const int64_t local = p.tokens[row] - p.vocab_offset;
        if (local >= 0 && local < p.V) st.token = int32_t(local);
      }
    }
    const AllowWords allow(st.mrow, at.col0, p.V);
    auto load = [&](int c, uint32_t (&r)[32]) {
      ptx::tmem_ld_32x32b_x32(at.taddr + uint32_t(c * 32), r);
      ptx::tmem_wait_ld();
      const uint32_t w = allow.at(c);
      const bool full = __all_sync(0xFFFFFFFFu, !valid || w == 0xFFFFFFFFu);
      if (!valid) return;
      const float top = full ? chunk<false>(st, r, w) : chunk<true>(st, r, w);
      const uint32_t tok = uint32_t(st.token - (at.col0 + c * 32));
      if (tok < 32u) st.at_token = pick32(r, tok);
      // Any id within 2^4 of the row's largest term serves: looking for the column
      // costs 64 instructions a chunk, so small rises are passed over.
      if (KC == 0 && (top - st.ref.val) * st.scale2 > 4.0f) {
        uint32_t hit = 0u;
#pragma unroll
        for (int j = 0; j < 32; ++j) hit |= __uint_as_float(r[j]) == top ? 1u << j : 0u;
        st.ref = RowRef{top, at.col0 + c * 32 + __ffs(hit) - 1};
      }
    };
    bool filled = false;
    if constexpr (KC > 0) {
      if (st.first && p.sorted_start) filled = fill(p, st, at, allow, valid);
      st.first = false;
    }
#pragma unroll 1
    for (int c = 0; c < kN / 64; ++c) {
      if (at.col0 + c * 32 >= p.V) break;
      uint32_t r[32];
      load(c, r);
      if constexpr (KC > 0) {
        if (filled) continue;
        // Every lane marks the logits that beat its list's last entry; the
        // warp then inserts one per lane and round, lowest id first.  (An
        // entry of the row's best is among the best of any subset holding it.)
        uint32_t want = 0u;
        if (valid) {
          const float least = st.ts[KC - 1];
#pragma unroll
          for (int j = 0; j < 32; ++j) want |= __uint_as_float(r[j]) > least ? 1u << j : 0u;
        }
        while (__any_sync(0xFFFFFFFFu, want != 0u)) {
          if (want != 0u) {
            const uint32_t j = uint32_t(__ffs(want) - 1);
            want &= want - 1u;
            const float v = pick32(r, j) + 0.0f;  // -0 counts as +0
            if (v > st.ts[KC - 1]) list_insert<KC>(st.ts, st.ti, v, at.col0 + c * 32 + int(j));
          }
        }
      }
    }
    release();
  }
  static __device__ __forceinline__ void finish(const Params& p, State& st, int worker, int row,
                                                int half, const Shape& s) {
    // A slot per (group of workers on the same vocabulary blocks, half); every
    // one is written, also by a thread whose columns lay past V.
    if (row >= p.B) return;
    const int64_t slot = int64_t(row) * p.n_slots + (worker / s.n_mt) * 2 + half;
    p.part[slot] = RowPart{st.m, st.S, st.U, st.at_token};
    if constexpr (KC == 0) {
      p.ref[slot] = st.ref;
    } else {
      float4* v4 = reinterpret_cast<float4*>(p.cand_val + slot * KC);
      int4* i4 = reinterpret_cast<int4*>(p.cand_id + slot * KC);
#pragma unroll
      for (int q = 0; q < KC; q += 4) {
        v4[q / 4] = make_float4(st.ts[q], st.ts[q + 1], st.ts[q + 2], st.ts[q + 3]);
        i4[q / 4] = make_int4(st.ti[q], st.ti[q + 1], st.ti[q + 2], st.ti[q + 3]);
      }
    }
  }
};

// ---------------------------------------------------------------------------
// Forward: join a row's parts, rank its alternatives
// ---------------------------------------------------------------------------

struct JoinParams {
  const __nv_bfloat16* H;  // of this launch's first row
  const __nv_bfloat16* W;
  int64_t ldh, ldw;
  int32_t d, V, n_slots, K;
  int32_t n_kb;  // k slices of the contraction
  int32_t ctas;  // blocks (a cluster) per row
  const float* temperature;
  const uint32_t* mask;
  int64_t mask_ld;
  const int64_t* tokens;
  int64_t vocab_offset;
  const RowPart* part;
  const RowRef* ref;
  const float* cand_val;
  const int32_t* cand_id;
  float *out_logp, *out_entropy, *out_lse;
  int64_t* out_topk_idx;
  float* out_topk_logp;
};

// a + b = s + err exactly (Knuth's two-sum).
__device__ __forceinline__ float two_sum(float a, float b, float& err) {
  const float s = __fadd_rn(a, b);
  const float bb = __fsub_rn(s, a);
  err = __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb));
  return s;
}

// One logit by a warp: bf16 products are exact in fp32, and their sum is kept
// as an unevaluated pair hi + lo, good to about 2^-45 of the terms' magnitude.
// Every lane returns it, normalised (hi is the sum rounded to fp32); the order
// of the terms depends on d alone.  kDeep 16-byte loads of w are in flight per lane
// (a warp usually reads its row from DRAM); h is shared by the row's warps and
// comes from L1.
template <int kDeep>
__device__ __forceinline__ float2 warp_logit(const __nv_bfloat16* __restrict__ h,
                                             const __nv_bfloat16* __restrict__ w, int d,
                                             int lane) {
  const uint4* h4 = reinterpret_cast<const uint4*>(h);
  const uint4* w4 = reinterpret_cast<const uint4*>(w);
  float hi = 0.0f, lo = 0.0f;
  auto add = [&](float x) {
    float err;
    hi = two_sum(hi, x, err);
    lo = __fadd_rn(lo, err);
  };
  const int n8 = d >> 3;
  for (int i0 = lane; i0 < n8; i0 += 32 * kDeep) {
    uint4 wv[kDeep];
#pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      const int i = i0 + 32 * u;
      wv[u] = i < n8 ? __ldg(w4 + i) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      const int i = i0 + 32 * u;
      if (i >= n8) break;
      const uint4 hv = __ldg(h4 + i);
      const uint32_t av[4] = {hv.x, hv.y, hv.z, hv.w};
      const uint32_t bv[4] = {wv[u].x, wv[u].y, wv[u].z, wv[u].w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        add(__fmul_rn(__uint_as_float(av[q] << 16), __uint_as_float(bv[q] << 16)));
        add(__fmul_rn(__uint_as_float(av[q] & 0xFFFF0000u),
                      __uint_as_float(bv[q] & 0xFFFF0000u)));
      }
    }
  }
  const int tail = n8 * 8 + lane;
  if (tail < d) add(__fmul_rn(__bfloat162float(h[tail]), __bfloat162float(w[tail])));
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    const float ohi = __shfl_xor_sync(0xFFFFFFFFu, hi, off);
    const float olo = __shfl_xor_sync(0xFFFFFFFFu, lo, off);
    float err;
    hi = two_sum(hi, ohi, err);
    lo = __fadd_rn(__fadd_rn(lo, olo), err);
  }
  // Infinite or NaN: hi alone.
  if (!isfinite(hi)) return make_float2(hi, 0.0f);
  float err;
  const float sum = two_sum(hi, lo, err);
  return make_float2(sum, err);
}

// A row's normaliser: lse = L / T + log_sum, L one id's logit as an exact pair.
struct Norm {
  float2 L;
  float log_sum;
};
// (logit - L) / T - log_sum, so that neither the logits' size nor the rounding of lse
// enters; at most 0 (log_sum is off by its own rounding where one token has nearly all
// the mass).  NaN stays.
__device__ __forceinline__ float scaled_logp(float2 logit, float T, const Norm& n) {
  const float logp = ((logit.x - n.L.x) + (logit.y - n.L.y)) / T - n.log_sum;
  return logp > 0.0f ? 0.0f : logp;
}
// a / T + b without the quotient's rounding.
__device__ __forceinline__ float scaled_sum(float2 a, float T, float b) {
  const float q = __fdiv_rn(a.x, T);
  if (!isfinite(q)) return q + b;
  return q + ((__fmaf_rn(-q, T, a.x) + a.y) / T + b);
}

// An order-preserving map of floats to unsigned integers; NaN counts as +inf
// (it ranks first, so that every place is filled; the row's lse is NaN too).
__device__ __forceinline__ uint32_t order_bits(float f) {
  if (!(f == f)) f = INFINITY;
  const uint32_t u = __float_as_uint(f + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// (value, id) as one unsigned integer whose order is: higher value first, then
// lower id; 0 (no entry) comes last.  -0 counts as +0; values are not NaN.
__device__ __forceinline__ uint64_t entry_key(float f, int32_t id) {
  if (id < 0) return 0u;
  return (uint64_t(order_bits(f)) << 32) | (0xFFFFFFFFu - uint32_t(id));
}

// The value of an entry's key.
__device__ __forceinline__ float entry_value(uint64_t key) {
  const uint32_t u = uint32_t(key >> 32);
  return __uint_as_float((u & 0x80000000u) ? u ^ 0x80000000u : ~u);
}

// How many of the n keys in shared memory exceed `key`.
__device__ __forceinline__ int count_above(const uint64_t* keys, int n, uint64_t key) {
  int above[4] = {};
  int i = 0;
  for (; i + 4 <= n; i += 4) {
    uint64_t k[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) k[q] = keys[i + q];
#pragma unroll
    for (int q = 0; q < 4; ++q) above[q] += k[q] > key ? 1 : 0;
  }
  for (; i < n; ++i) above[0] += keys[i] > key ? 1 : 0;
  return above[0] + above[1] + above[2] + above[3];
}

// Fold the state (m1, S1, U1) into (m0, S0, U0); raw logits times scale2 are in base 2.
__device__ __forceinline__ void join_state(float& m0, float& S0, float& U0, float m1, float S1,
                                           float U1, float scale2) {
  if (m1 == -INFINITY) return;
  if (m0 == -INFINITY) {
    m0 = m1, S0 = S1, U0 = U1;
    return;
  }
  const float mm = ptx::max_nan(m0, m1);
  const float d0 = ptx::max_nan((m0 - mm) * scale2, -16384.0f);
  const float d1 = ptx::max_nan((m1 - mm) * scale2, -16384.0f);
  const float f0 = exp2f(d0), f1 = exp2f(d1);
  U0 = f0 * fmaf(d0, S0, U0) + f1 * fmaf(d1, S1, U1);
  S0 = f0 * S0 + f1 * S1;
  m0 = mm;
}
__device__ __forceinline__ void join_lanes(float& m, float& S, float& U, float scale2) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    const float om = __shfl_xor_sync(0xFFFFFFFFu, m, off);
    const float oS = __shfl_xor_sync(0xFFFFFFFFu, S, off);
    const float oU = __shfl_xor_sync(0xFFFFFFFFu, U, off);
    join_state(m, S, U, om, oS, oU, scale2);
  }
}
__device__ __forceinline__ uint64_t max_lanes(uint64_t key) {
  const uint32_t hi = __reduce_max_sync(0xFFFFFFFFu, uint32_t(key >> 32));
  const uint32_t lo = uint32_t(key >> 32) == hi ? uint32_t(key) : 0u;
  return (uint64_t(hi) << 32) | __reduce_max_sync(0xFFFFFFFFu, lo);
}
__device__ __forceinline__ float sum_lanes(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
  return v;
}

// Blocks of the join kernel: a thread per slot at least.  Up to a block per SM
// what counts is a row's latency: a warp for every logit of K <= 5, whole rows
// of W in flight.  Beyond (CTA pairs: half the slots) it is the number of rows
// in flight: small blocks of fewer registers (1000 rows at d = 4096, K = 5: 35 us,
// with the large blocks 63).
struct JoinWide {
  static constexpr int kThreads = 320, kDeep = 16, kBlocks = 2;
};
struct JoinNarrow {
  static constexpr int kThreads = 160, kDeep = 4, kBlocks = 8;
};
constexpr int kMaxSlots = 2 * kPlanSms;
static_assert(kMaxSlots <= JoinWide::kThreads && kPlanSms <= JoinNarrow::kThreads,
              "a thread per slot");

// A row's block, or with more logits to sum than a block has warps and few
// rows, its cluster of `ctas` blocks: every block selects the candidates, the
// logits are dealt out to all warps, and block 0 sums, ranks and writes.
// Launched as a programmatic dependent of the contraction.
//
// The n = K + 4 best entries of the row's lists, in three steps:
//   heads     the largest head of every 8 lists bounds the n-th best head from
//             below (n of these reach it); the few heads that reach the bound
//             are ranked by counting;
//   entries   an entry in place q of the list with the r-th best head has r + q
//             better ones, so only r + q < n can matter, and only entries that
//             reach the n-th best head;
//   ranks     those (rarely more than n + a few) are ranked by counting.
// Keys are all different, so counting gives each its place whatever order the
// threads came in.
//
// What bounds it is latency: dependent loads, barriers and short loops, hidden
// behind other rows where there are more rows than SMs.  In a call, in part while the
// contraction ends: 12 us of 64 rows at d = 4096 with K = 5, 8 with K = 0; 35 of 1000
// rows, 14 with K = 0.
template <int KC, class Block>
__global__ void __launch_bounds__(Block::kThreads, Block::kBlocks)
    join_kernel(const JoinParams p) {
  constexpr int kJoinThreads = Block::kThreads;
  constexpr int kJoinWarps = kJoinThreads / 32;
  constexpr int kList = KC > 0 ? KC : 1;
  constexpr int kGroups = kJoinThreads / 8;
  constexpr int kEntries = kList * (kList + 1) / 2;
  static_assert(KC < 31, "a lane per candidate, and the last one for the token");
  __shared__ float s_m[kJoinWarps], s_S[kJoinWarps], s_U[kJoinWarps];
  __shared__ uint32_t s_at[kJoinWarps];  // order_bits of the token's raw logit
  __shared__ float2 s_token;
  __shared__ Norm s_norm;
  __shared__ uint32_t s_group[kGroups];
  __shared__ uint32_t s_bound;
  __shared__ int32_t s_heads, s_entries;
  __shared__ uint64_t s_head[KC > 0 ? kJoinThreads : kJoinWarps];
  __shared__ int32_t s_slot[KC > 0 ? kJoinThreads : 1];
  __shared__ uint64_t s_entry[kEntries];
  __shared__ int32_t s_list[kList];
  __shared__ uint64_t s_least;
  __shared__ int32_t s_id[kList], s_rank[kList];
  __shared__ float s_raw[kList];  // the candidates' fp32 sums
  __shared__ uint64_t s_key[kList];
  __shared__ float2 s_logit[kList];
  const int cta = int(blockIdx.x) % p.ctas;
  const int row = int(blockIdx.x) / p.ctas;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n_cand = KC > 0 ? p.K + 4 : 1;  // at most KC; without lists, the reference id
  if (tid < kList) s_list[tid] = s_id[tid] = -1, s_rank[tid] = 0, s_key[tid] = 0u;
  if (tid == 0) s_bound = 0u, s_heads = s_entries = 0, s_least = 0u;
  if (KC > 0 && p.ctas > 1) ptx::cluster_sync();  // block 0's keys are cleared before any arrives
  ptx::grid_dependency_wait();

  // ---- what the row needs from memory, at once
  const int64_t slot0 = int64_t(row) * p.n_slots;
  float m = -INFINITY, S = 0.0f, U = 0.0f, at_token = -INFINITY;
  uint64_t head = 0u;
  if (tid < p.n_slots) {
    const RowPart r = p.part[slot0 + tid];
    if constexpr (KC > 0) {
      head = entry_key(p.cand_val[(slot0 + tid) * KC], p.cand_id[(slot0 + tid) * KC]);
    } else {
      const RowRef ref = p.ref[slot0 + tid];
      head = entry_key(ref.val, ref.id);
    }
    m = r.m, S = r.S, U = r.U, at_token = r.at_token;
  }
  const float T = row_temperature(p.temperature, row), scale2 = scale_to_log2(T, p.n_kb);
  int64_t token = -1, local = -1;
  bool scored = false;  // the token has a logit
  if (p.tokens) {
    token = p.tokens[row];
    local = token - p.vocab_offset;
    scored = token >= 0 && local >= 0 && local < p.V;
    if (scored && p.mask)
      scored = (p.mask[int64_t(row) * p.mask_ld + (local >> 5)] >> (local & 31)) & 1u;
  }

  // ---- statistics: lanes, then (below) warps
  join_lanes(m, S, U, scale2);
  const uint32_t at = __reduce_max_sync(0xFFFFFFFFu, order_bits(at_token));
  if (lane == 0) s_m[warp] = m, s_S[warp] = S, s_U[warp] = U, s_at[warp] = at;

  // ---- candidates
  if constexpr (KC == 0) {
    head = max_lanes(head);
    if (lane == 0) s_head[warp] = head;
    __syncthreads();
    head = max_lanes(lane < kJoinWarps ? s_head[lane] : 0u);  // the row's, in every warp
  } else {
    const uint32_t value = uint32_t(head >> 32);
    uint32_t top = value;
#pragma unroll
    for (int off = 4; off > 0; off >>= 1)
      top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, off));
    if ((lane & 7) == 0) s_group[tid >> 3] = top;
    __syncthreads();
    if (tid < kGroups) {  // the group whose largest head is the n-th largest
      const uint32_t mine = s_group[tid];
      int above = 0, reach = 0;
#pragma unroll 8
      for (int i = 0; i < kGroups; ++i) {
        const uint32_t g = s_group[i];
        above += g > mine ? 1 : 0;
        reach += g >= mine ? 1 : 0;
      }
      if (above < n_cand && reach >= n_cand) s_bound = mine;
    }
    __syncthreads();
    if (head != 0u && value >= s_bound) {
      const int i = atomicAdd(&s_heads, 1);
      s_head[i] = head;
      s_slot[i] = tid;
    }
    __syncthreads();
    if (tid < s_heads) {
      const uint64_t key = s_head[tid];
      const int r = count_above(s_head, s_heads, key);
      if (r < n_cand) s_list[r] = s_slot[tid];
      if (r == n_cand - 1) s_least = key;
    }
    __syncthreads();
    for (int r = warp; r < n_cand; r += kJoinWarps) {
      const int32_t list = s_list[r];
      if (list < 0 || lane >= n_cand - r) continue;
      const int64_t at = (slot0 + list) * KC + lane;
      const uint64_t key = entry_key(p.cand_val[at], p.cand_id[at]);
      if (key != 0u && key >= s_least) s_entry[atomicAdd(&s_entries, 1)] = key;
    }
    __syncthreads();
    for (int i = tid; i < s_entries; i += kJoinThreads) {
      const uint64_t key = s_entry[i];
      const int r = count_above(s_entry, s_entries, key);
      if (r < n_cand) {
        s_id[r] = int32_t(0xFFFFFFFFu - uint32_t(key));
        s_raw[r] = entry_value(key);
      }
    }
    __syncthreads();
  }

  // ---- the logits again, a warp each (0: the token, from 1: candidates), dealt
  // out to the warps of all blocks
  const __nv_bfloat16* h = p.H + int64_t(row) * p.ldh;
  auto cand_id = [&](int i) {
    if constexpr (KC == 0) return head != 0u ? int32_t(0xFFFFFFFFu - uint32_t(head)) : -1;
    return s_id[min(i, kList - 1)];
  };
  auto cand_raw = [&](int i) {
    if constexpr (KC == 0) return entry_value(head);
    return s_raw[min(i, kList - 1)];
  };
  // The last warp of block 0 joins the row's sums meanwhile and takes the terms of the
  // known ids out: the candidates, a lane each, and the token in the last lane.
  const bool sums = cta == 0 && warp == kJoinWarps - 1;
  float rest_S = 0.0f, rest_U = 0.0f;
  bool known = false;  // the lane has such an id
  if (sums) {
    m = lane < kJoinWarps ? s_m[lane] : -INFINITY;
    S = lane < kJoinWarps ? s_S[lane] : 0.0f;
    U = lane < kJoinWarps ? s_U[lane] : 0.0f;
    const uint32_t all_at = __reduce_max_sync(0xFFFFFFFFu, lane < kJoinWarps ? s_at[lane] : 0u);
    join_lanes(m, S, U, scale2);
    const bool held = lane < n_cand && cand_id(lane) >= 0;
    const bool listed = __any_sync(0xFFFFFFFFu, held && cand_id(lane) == local);
    const float raw = held ? cand_raw(lane)
                      : lane == 31 && scored && !listed ? entry_value(uint64_t(all_at) << 32)
                                                        : -INFINITY;
    known = isfinite(raw);
    const float t = fmaxf((raw - m) * scale2, -16384.0f), e = known ? exp2f(t) : 0.0f;
    rest_S = ptx::max_nan(S - sum_lanes(e), 0.0f);
    rest_U = -ptx::max_nan(sum_lanes(e * t) - U, 0.0f);
  }
  for (int j = cta * kJoinWarps + warp; j <= n_cand; j += p.ctas * kJoinWarps) {
    if (j == 0) {
      if (scored) {
        const float2 l = warp_logit<Block::kDeep>(h, p.W + local * p.ldw, p.d, lane);
        if (lane == 0) s_token = l;
      }
      continue;
    }
    const int32_t id = cand_id(j - 1);
    if (id < 0) continue;
    const float2 l = warp_logit<Block::kDeep>(h, p.W + int64_t(id) * p.ldw, p.d, lane);
    if (lane == 0) {
      const uint64_t key = (uint64_t(order_bits(l.x)) << 32) | order_bits(l.y);
      if (cta == 0) {
        s_logit[j - 1] = l;
        s_key[j - 1] = key;
      } else {
        ptx::st_cluster(ptx::cluster_addr(&s_logit[j - 1], 0),
                        *reinterpret_cast<const uint64_t*>(&l));
        ptx::st_cluster(ptx::cluster_addr(&s_key[j - 1], 0), key);
      }
    }
  }
  if (KC > 0 && p.ctas > 1) {
    ptx::cluster_sync();
    if (cta != 0) return;
  } else {
    __syncthreads();
  }

  // ---- the row's sums, with the known ids' terms from their exact logits in place of
  // those the contraction added: relative to the largest of them, L, so that a row that
  // one token decides is as exact as L.
  if (sums) {
    const float2 l = !known ? make_float2(0.0f, 0.0f) : lane == 31 ? s_token : s_logit[min(lane, kList - 1)];
    const uint64_t key =
        known ? (uint64_t(order_bits(l.x)) << 32) | order_bits(l.y) : 0u;
    const uint64_t top = max_lanes(key);
    const int lead = __ffs(__ballot_sync(0xFFFFFFFFu, key == top)) - 1;
    Norm norm;
    norm.L = make_float2(__shfl_sync(0xFFFFFFFFu, l.x, lead), __shfl_sync(0xFFFFFFFFu, l.y, lead));
    if (top == 0u) norm.L = make_float2(m, 0.0f);  // none known
    // The others' terms relative to L (m in base 2 is m scale2), and the known ids' own.
    const float unit = kLog2e / T;
    // At a temperature near 0 the one cut-off more is any number of units: bounded, so
    // that where there are no other terms they stay 0.
    const float up = fminf(
        fmaxf(unit * ((norm.L.x - m) + (norm.L.y - m * mean_cut(p.n_kb))), -100.0f), 100.0f);
    const float f = exp2f(-up);
    const float t = fmaxf(unit * ((l.x - norm.L.x) + (l.y - norm.L.y)), -16384.0f);
    const float e = known ? exp2f(t) : 0.0f;
    S = fmaf(rest_S, f, sum_lanes(e));
    U = fmaf(f, fmaf(-up, rest_S, rest_U), sum_lanes(e * t));
    const bool none = m == -INFINITY;
    const float log2S = log2f(S);
    norm.log_sum = none ? -INFINITY : kLn2 * log2S;
    if (lane == 0) {
      s_norm = norm;
      if (p.out_lse) p.out_lse[row] = none ? -INFINITY : scaled_sum(norm.L, T, norm.log_sum);
      if (p.out_entropy) {
        const float entropy = kLn2 * (log2S - U / S);
        p.out_entropy[row] = none || entropy < 0.0f ? 0.0f : entropy;
      }
      if (p.tokens)
        p.out_logp[row] =
            scored ? scaled_logp(s_token, T, norm) : token < 0 ? 0.0f : -INFINITY;
    }
  }
  if constexpr (KC > 0) {
    for (int pair = tid; pair < n_cand * n_cand; pair += kJoinThreads) {
      const int j = pair / n_cand, i = pair - j * n_cand;
      const uint64_t a = s_key[i], b = s_key[j];  // 0: absent
      if (a != 0u && (a > b || (a == b && s_id[i] < s_id[j]))) atomicAdd(&s_rank[j], 1);
    }
    __syncthreads();
    if (tid < n_cand) {
      const int32_t id = s_id[tid];
      const int rank = id < 0 ? tid : s_rank[tid];  // absent ones come last, in place
      if (rank < p.K) {
        const int64_t o = int64_t(row) * p.K + rank;
        p.out_topk_idx[o] = id < 0 ? -1 : p.vocab_offset + id;
        // Missing ones have -inf, but NaN as all of the row has if a logit is not a number.
        p.out_topk_logp[o] = id >= 0 ? scaled_logp(s_logit[tid], T, s_norm)
                             : isnan(s_norm.log_sum) ? s_norm.log_sum : -INFINITY;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Backward: G = dLoss / dlogits
// ---------------------------------------------------------------------------

struct GradParams {
  int32_t B, V, d;
  const __nv_bfloat16* H;
  const __nv_bfloat16* W;
  int64_t ldh, ldw;
  const float* temperature;
  const uint32_t* mask;
  int64_t mask_ld;
  const int64_t* tokens;
  const float *lse, *entropy, *grad_logp, *grad_entropy;
  int64_t vocab_offset;
  float* delta;  // [B]: what rounding took from G at the row's token, where W has it
  uint4* marks;  // as Rounding's
};

template <int kCols>
struct GradEpi {
  static constexpr int kN = kCols;
  static constexpr bool kStaged = true;
  using Params = GradParams;
  // With a, e the row's upstream gradients over T, P = 2^x the probability and
  // x = log2 p = l scale2 - lse2:  G = P (c0 + c1 x), + a at the token, where
  // c1 = -e ln2, c0 = -a - e entropy.  The token's element is the largest of its
  // row by far and repeats its rounding error in all of dH's row and dW's, where
  // the others' average out; so what bf16 leaves of it is kept (delta) and added
  // to those rows in fp32: with it the results are as close as their own bf16
  // rounding allows where the rest of the row is spread out (4 to 512 rows: 1.0 times
  // the error of that rounding alone, without it 1.3 to 1.6).  Another id that holds
  // much of a row repeats its rounding in the same way, and that is left: such an id
  // of probability 0.3 in every row takes the error to 1.02 to 1.05 times (1.25 in
  // the worst row of dH), of 0.9 to 1.2 to 1.5 (1.9), of 0.99 to 1.2 to 1.35 (2.0).
  // At a likely token the element is a (1 - P), which the
  // tensor core's sum is not good enough for beside an exact lse: it is taken from
  // the token's logit summed again.
  struct State {
    int row = -1;
    float scale2, lse2, c0, c1, a;
    float T, lse;
    int32_t token;  // id from 0, -1 for none among W's
    const uint32_t* mrow;
    bool live;  // false: the row's G is 0
    bool far;   // the logits' error, in units of T, is not small
    float at_token;  // G at the token, if that is among the unit's columns
  };
  static __device__ __forceinline__ void start(const Params&, State&, int, int, const Shape&) {}
  static __device__ __forceinline__ void load_row(const Params& p, State& st, int row,
                                                  int n_kb) {
    st.row = row;
    st.mrow = nullptr;
    st.live = st.far = false;
    st.token = -1;
    st.scale2 = st.lse2 = st.c0 = st.c1 = st.a = st.lse = 0.0f;
    st.T = 1.0f;
    if (row >= p.B) return;
    const float T = st.T = row_temperature(p.temperature, row);
    const float lse = st.lse = p.lse[row];
    if (p.mask) st.mrow = p.mask + int64_t(row) * p.mask_ld;
    st.scale2 = scale_to_log2(T, n_kb);
    st.lse2 = lse * kLog2e;
    st.live = lse != -INFINITY;
    st.far = fabsf(st.lse2) * mean_cut(n_kb) > 0x1p-10f;
    float a = p.grad_logp[row] / T;
    const int64_t token = p.tokens[row], local = token - p.vocab_offset;
    if (token < 0) {
      a = 0.0f;
    } else if (local >= 0 && local < p.V) {
      st.token = int32_t(local);
      if (st.mrow && !((st.mrow[local >> 5] >> (local & 31)) & 1u)) a = 0.0f;
    }
    st.a = a;
    st.c0 = -a;
    if (p.grad_entropy) {
      const float e = p.grad_entropy[row] / T;
      st.c0 = fmaf(-e, p.entropy[row], -a);
      st.c1 = -e * kLn2;
    }
  }
  // G at the row's token, whose logit is l.
  static __device__ __forceinline__ float token_gradient(const State& st, float2 l) {
    const float logp = scaled_sum(l, st.T, -st.lse), x = (logp > 0.0f ? 0.0f : logp) * kLog2e;
    return fmaf(exp2f(x), fmaf(st.c1, ptx::max_nan(x, -16384.0f), st.c0), st.a);
  }
  // The tokens among the warp's columns, while the unit's MMAs run (their logits one by
  // one: behind the wait, 128 rows at d = 2048, V = 30000 took 98 us instead of 92).
  static __device__ __forceinline__ void before(const Params& p, State& st, const TileAt& at, int,
                                                int lane, const Shape& s) {
    const int row = at.row0 + lane;
    if (row != st.row) load_row(p, st, row, s.n_kb);
    const uint32_t tok = uint32_t(st.token - at.col0);
#pragma unroll 1
    for (uint32_t left = __ballot_sync(0xFFFFFFFFu, tok < uint32_t(kN / 2)); left != 0u;
         left &= left - 1u) {
      const int i = __ffs(left) - 1;
      const int64_t id = at.col0 + int(__shfl_sync(0xFFFFFFFFu, tok, i));
      const float2 l = warp_logit<8>(p.H + int64_t(at.row0 + i) * p.ldh, p.W + id * p.ldw, p.d,
                                     lane);
      if (lane == i) st.at_token = token_gradient(st, l);
    }
  }
  // 32 columns of G into the box; kCareful: `at_token` at the token's, if it is among
  // them, and no probability above 1 (the tensor core's logit of an id that has all the
  // mass may be above lse by more than ex2 takes, at temperatures near 0).
  template <bool kCareful>
  static __device__ __forceinline__ void put_chunk(const State& st, const uint32_t (&r)[32],
                                                   uint32_t w, uint32_t tok, float at_token,
                                                   uint8_t* box, int lane, int c) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float g[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int j = q * 8 + i;
        // Far below 1, p is 0 in fp32; the bound keeps 0 * -inf out of G.
        float x = ptx::max_nan(fmaf(__uint_as_float(r[j]), st.scale2, -st.lse2), -16384.0f);
        if (kCareful) x = x > 0.0f ? 0.0f : x;
        float v = ptx::ex2(x) * fmaf(st.c1, x, st.c0);
        if (kCareful && tok == uint32_t(j)) v = at_token;
        g[i] = ((w >> j) & 1u) ? v : 0.0f;
      }
      box_put(box, lane, c * 4 + q, pack_bf16(g[0], g[1]), pack_bf16(g[2], g[3]),
              pack_bf16(g[4], g[5]), pack_bf16(g[6], g[7]));
    }
  }
  template <class Release>
  static __device__ __forceinline__ void tile(const Params& p, State& st, const TileAt& at,
                                              int lane, uint8_t* box, const void* tmap,
                                              const Shape& s, Release release) {
    const int row = at.row0 + lane;
    const AllowWords allow(st.mrow, at.col0, p.V);
    box_begin(lane);
    const int blocks = (p.B + 31) / 32;
    const bool far = __any_sync(0xFFFFFFFFu, st.far);
#pragma unroll 1
    for (int c = 0; c < kN / 64; ++c) {
      const uint32_t w = st.live ? allow.at(c) : 0u;  // 0 past V
      const uint32_t tok = uint32_t(st.token - (at.col0 + c * 32));
      // The rows with their token here: dW's epilogue looks for them, and a warp
      // without one need not.
      const uint32_t marked = __ballot_sync(0xFFFFFFFFu, tok < 32u);
      uint32_t r[32];
      ptx::tmem_ld_32x32b_x32(at.taddr + uint32_t(c * 32), r);
      ptx::tmem_wait_ld();
      uint4 mark = make_uint4(marked, 0u, 0u, 0u);
      if (marked == 0u && !far) {
        put_chunk<false>(st, r, w, tok, 0.0f, box, lane, c);
      } else {
        const bool held = tok < 32u && ((w >> (tok & 31u)) & 1u);  // not masked, a live row
        const float at_token = held ? st.at_token : 0.0f;
        put_chunk<true>(st, r, w, tok, at_token, box, lane, c);
        float delta = at_token - __bfloat162float(__float2bfloat16_rn(at_token));
        if (!isfinite(delta)) delta = 0.0f;
        if (tok < 32u) p.delta[row] = delta;  // one thread of the grid for each row
        mark.y = __shfl_sync(0xFFFFFFFFu, tok, __ffs(marked) - 1);
        mark.z = __float_as_uint(__shfl_sync(0xFFFFFFFFu, delta, __ffs(marked) - 1));
      }
      if (lane == 0) p.marks[int64_t((at.col0 >> 5) + c) * blocks + (at.row0 >> 5)] = mark;
    }
    release();
    box_end(box, tmap, lane, at.col0, at.row0, min(p.V, at.col0 + kN / 2));
  }
  static __device__ __forceinline__ void finish(const Params&, State&, int, int, int,
                                                const Shape&) {}
};

// dH from its k splits, in split order, with G's rounding at the row's token, rounded
// to bf16 once.  A thread takes 4 columns of one row; neighbouring threads take
// neighbouring rows, the order the partial tiles are stored in (PartialEpi).  The
// partials come from L2: 9 us alone and cold for 19 splits of 96 rows at d = 2048.
constexpr int kSumThreads = 256;
constexpr int kSumBlocksPerTile = kBM * kBN / 4 / kSumThreads;  // of one CTA's tile
__global__ void __launch_bounds__(kSumThreads)
    sum_splits_kernel(const float4* __restrict__ partial, int32_t n_splits, int32_t n_tiles,
                      int32_t n_nt, int32_t ctas, int32_t B, int32_t d, const Rounding g,
                      __nv_bfloat16* __restrict__ dH, int64_t lddh) {
  ptx::grid_launch_dependents();
  constexpr int kTile = kBM * kBN / 4;              // float4 of a CTA's tile
  const int tile = blockIdx.x / kSumBlocksPerTile;  // (tile of the grid, CTA)
  const int at = blockIdx.x % kSumBlocksPerTile * kSumThreads + threadIdx.x;
  const int r = at % kBM, c4 = at / kBM;  // row, group of 4 columns
  const int t = tile / ctas, rank = tile - t * ctas;
  const int row = (t / n_nt * ctas + rank) * kBM + r;
  const int col = t % n_nt * kBN + c4 * 4;
  const bool in = row < B && col < d;
  // The row of W that G's rounding at the token belongs to.
  const int32_t v = in ? g.row_of_w(row) : -1;
  uint32_t x[4] = {};
  if (v >= 0) {
    const __nv_bfloat16* w = g.X + int64_t(v) * g.ldx + col;
    if (col + 4 <= d) {
      const uint2 two = __ldg(reinterpret_cast<const uint2*>(w));
      x[0] = two.x << 16, x[1] = two.x & 0xFFFF0000u;
      x[2] = two.y << 16, x[3] = two.y & 0xFFFF0000u;
    } else {
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (col + i < d) x[i] = __float_as_uint(__bfloat162float(w[i]));
    }
  }
  ptx::grid_dependency_wait();
  if (!in) return;
  const float delta = v >= 0 ? g.delta[row] : 0.0f;
  const float4* src = partial + (int64_t(t) * ctas + rank) * kTile + at;
  const int64_t step = int64_t(n_tiles) * ctas * kTile;
  float sum[4] = {};
#pragma unroll 8
  for (int s = 0; s < n_splits; ++s) {
    const float4 a = src[s * step];
    sum[0] += a.x, sum[1] += a.y, sum[2] += a.z, sum[3] += a.w;
  }
  if (delta != 0.0f)
#pragma unroll
    for (int i = 0; i < 4; ++i) sum[i] = fmaf(delta, __uint_as_float(x[i]), sum[i]);
  __nv_bfloat16* out = dH + int64_t(row) * lddh + col;
  if (col + 4 <= d) {
    __nv_bfloat162 h[2] = {__floats2bfloat162_rn(sum[0], sum[1]),
                               __floats2bfloat162_rn(sum[2], sum[3])};
    *reinterpret_cast<uint2*>(out) = *reinterpret_cast<const uint2*>(h);
  } else {
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (col + i < d) out[i] = __float2bfloat16_rn(sum[i]);
  }
}

// dH's partial tiles and dW in one launch, the first `n_h` CTAs the former's, one unit
// each, and the others dW's, where these have few: then a launch's start and end are
// much of its time (a call in two launches / in one, us: 4 rows at d = 256, V = 4096
// 20.5 / 16.4; 60 at 1024, 11137 29.4 / 24.1; 12 at 3214, 5280 37.1 / 35.3, dW's CTAs
// with 7 units each; but 15 at 142, 125310, 11 units each, 53.3 / 56.8).
constexpr size_t kBothSmem = std::max(smem_bytes<PartialEpi>(), smem_bytes<StoreEpi<false>>());
template <bool kPair>
__global__ void __launch_bounds__(kThreads, 1)
    both_kernel(const __grid_constant__ CUtensorMap h_a, const __grid_constant__ CUtensorMap h_b,
                const __grid_constant__ CUtensorMap w_a, const __grid_constant__ CUtensorMap w_b,
                const __grid_constant__ CUtensorMap w_d, const __grid_constant__ Shape h,
                const __grid_constant__ Shape w, const __grid_constant__ PartialEpi::Params hp,
                const __grid_constant__ StoreEpi<false>::Params wp, int n_h) {
  if (int(blockIdx.x) < n_h)
    contract<PartialEpi, kPair, false, true>(h_a, h_b, w_d, h, hp, int(blockIdx.x), n_h);
  else
    contract<StoreEpi<false>, kPair, true, true>(w_a, w_b, w_d, w, wp, int(blockIdx.x) - n_h,
                                                 int(gridDim.x) - n_h);
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

constexpr int kMaxDevices = 64;
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
size_t round256(size_t n) { return (n + 255u) & ~size_t(255u); }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <class Epi, bool kPair, bool kAmn, bool kBmn>
bool prepare_kernel(int sms, int* pairs) {
  auto k = contract_kernel<Epi, kPair, kAmn, kBmn>;
  if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           int(smem_bytes<Epi>())) != cudaSuccess)
    return false;
  if (!kPair) return true;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 2;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.gridDim = dim3(unsigned(sms / 2 * 2), 1, 1);
  cfg.dynamicSmemBytes = smem_bytes<Epi>();
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, k, &cfg) != cudaSuccess || n < 1) return false;
  *pairs = std::min(*pairs, n);
  return true;
}

template <int KC>
bool prepare_scores(int sms, int* pairs) {
  return prepare_kernel<ScoreEpi<KC, 64>, false, false, false>(sms, pairs) &&
         prepare_kernel<ScoreEpi<KC, 128>, false, false, false>(sms, pairs) &&
         prepare_kernel<ScoreEpi<KC, 256>, false, false, false>(sms, pairs) &&
         prepare_kernel<ScoreEpi<KC, 256>, true, false, false>(sms, pairs);
}

template <int KC>
cudaError_t launch_join(JoinParams j, int64_t rows, cudaStream_t stream) {
  const bool wide = rows <= kPlanSms || j.n_slots > JoinNarrow::kThreads;
  // More logits than a block has warps: as many blocks as leave every SM at
  // most one.
  j.ctas = 1;
  while (wide && j.ctas < 4 && (j.K > 0 ? j.K + 5 : 2) > j.ctas * (JoinWide::kThreads / 32) &&
         rows * j.ctas * 2 <= kPlanSms)
    j.ctas *= 2;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(j.ctas);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(rows * j.ctas), 1, 1);
  cfg.blockDim = dim3(unsigned(wide ? JoinWide::kThreads : JoinNarrow::kThreads), 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = j.ctas > 1 ? 2 : 1;
  return wide ? cudaLaunchKernelEx(&cfg, join_kernel<KC, JoinWide>, j)
              : cudaLaunchKernelEx(&cfg, join_kernel<KC, JoinNarrow>, j);
}

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
      d.sms = std::min(d.sms, kPlanSms);
      d.pairs = d.sms / 2;
      void* fn = nullptr;
      cudaDriverEntryPointQueryResult q;
      d.error_word = device_error_word();
      const bool ok =
          d.error_word != nullptr && prepare_scores<0>(d.sms, &d.pairs) &&
          prepare_scores<8>(d.sms, &d.pairs) && prepare_scores<16>(d.sms, &d.pairs) &&
          prepare_scores<24>(d.sms, &d.pairs) &&
          prepare_kernel<GradEpi<128>, false, false, false>(d.sms, &d.pairs) &&
          prepare_kernel<GradEpi<256>, false, false, false>(d.sms, &d.pairs) &&
          prepare_kernel<GradEpi<256>, true, false, false>(d.sms, &d.pairs) &&
          prepare_kernel<StoreEpi<true>, false, false, true>(d.sms, &d.pairs) &&
          prepare_kernel<StoreEpi<true>, true, false, true>(d.sms, &d.pairs) &&
          prepare_kernel<PartialEpi, false, false, true>(d.sms, &d.pairs) &&
          prepare_kernel<PartialEpi, true, false, true>(d.sms, &d.pairs) &&
          prepare_kernel<StoreEpi<false>, false, true, true>(d.sms, &d.pairs) &&
          prepare_kernel<StoreEpi<false>, true, true, true>(d.sms, &d.pairs) &&
          cudaFuncSetAttribute(both_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               int(kBothSmem)) == cudaSuccess &&
          cudaFuncSetAttribute(both_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               int(kBothSmem)) == cudaSuccess &&
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

// 2-D bf16 tensor map with 128-byte-swizzled boxes of 64 x rows; elements past
// the extents read as zero and are not written.
bool encode(const Device& dev, CUtensorMap* m, const void* base, int64_t inner, int64_t outer,
            int64_t ld, int box_rows) {
  const cuuint64_t dims[2] = {cuuint64_t(inner), cuuint64_t(outer)};
  const cuuint64_t strides[1] = {cuuint64_t(ld) * 2u};
  const cuuint32_t box[2] = {64u, cuuint32_t(box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  return dev.encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides,
                    box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class Epi, bool kPair, bool kAmn>
void fill_ring(const Device& dev, Shape& s) {
  constexpr uint32_t kBBytes = (kPair ? Epi::kN / 2 : Epi::kN) * kBK * 2;
  s.a_bytes = kAmn ? kBM * kBK * 2 : s.a_box_rows * 128u;
  s.stage_bytes = slices<Epi>() * (s.a_bytes + kBBytes);
  s.n_stages = ring_stages<Epi, kPair>(s.a_bytes);
  s.wait_limit_ns = kWaitLimitNs;
  s.error_word = dev.error_word;
}

template <class Epi, bool kPair, bool kAmn, bool kBmn>
fs_status launch(const Device& dev, const CUtensorMap& a, const CUtensorMap& b,
                 const CUtensorMap& d, Shape s, const typename Epi::Params& ep, int workers,
                 bool overlap, cudaStream_t stream) {
  fill_ring<Epi, kPair, kAmn>(dev, s);
  cudaLaunchAttribute attr[2];
  unsigned n = 0;
  if (kPair) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = 2;
    attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
    ++n;
  }
  if (overlap) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(workers * (kPair ? 2 : 1)), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem_bytes<Epi>();
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = n;
  if (cudaLaunchKernelEx(&cfg, contract_kernel<Epi, kPair, kAmn, kBmn>, a, b, d, s, ep) !=
      cudaSuccess) {
    cudaGetLastError();
    return FS_ERR_CUDA;
  }
  return FS_OK;
}

// The smallest number of workers that needs no more waves than all of them.
int balanced(int64_t units, int workers) {
  if (units <= workers) return int(units);
  const int64_t waves = ceil_div(units, workers);
  return int(ceil_div(units, waves));
}

// Rows per forward launch.  A worker keeps its block of rows, so the workers
// are split into as many groups as divide evenly among the blocks: 3, 4 or 5
// pair blocks (256 rows) use 75 or 76 of 76 pairs and share each W tile in L2,
// and W is streamed once per launch.
int64_t rows_per_launch(int64_t B) {
  const int64_t blocks = ceil_div(B, 2 * kBM);
  return ceil_div(blocks, ceil_div(blocks, 5)) * 2 * kBM;
}

// A thread's list: K + 4 at least; longer ones cost registers, time and what the join
// reads (64 rows at d = 4096, V = 151936, K = 4: 8 entries 194 us, 16 196, 24 200).
int list_cap(int64_t K) { return K <= 0 ? 0 : K <= 4 ? 8 : K <= 12 ? 16 : 24; }

// Columns of a single-CTA unit of the logits' kernels: the narrowest that still
// gives every SM at most one unit, so that a small vocabulary starts as many
// CTAs as it can (6 rows at d = 1790, V = 11137, K = 5: 256 wide 30.6 us, 128 24.1, 64,
// which needs two units of some CTAs, 26.3).  Else 256: wide units read H least often and
// need the fewest barriers, narrow ones have fewer logits before a CTA's first list is
// full, and neither is better throughout (256 / 128 wide, us: 6 rows, d = 1790, V = 38281,
// K = 0 30.7 / 29.9, K = 5 43.3 / 39.6, K = 20 46.2 / 46.5; 100 rows, d = 256, V = 60000,
// K = 20 47.0 / 52.6; 8 rows, d = 512, V = 151936, K = 20 67.4 / 71.0).
int unit_cols(int64_t V, int least) {
  int n = least;
  while (n < kBN && ceil_div(V, n) > kPlanSms) n *= 2;
  return n;
}

// Upper bound of a row's slots: groups of workers x 2 halves.
int64_t plan_slots(int64_t rows, int64_t V) {
  if (rows <= kBM) return 2 * std::min<int64_t>(ceil_div(V, unit_cols(V, 64)), kPlanSms);
  return 2 * std::min<int64_t>(ceil_div(V, kBN), kPlanSms / 2 / ceil_div(rows, 2 * kBM));
}

bool sizes_ok(int64_t B, int64_t d, int64_t V) {
  return B >= 1 && B <= 65535 && d >= 1 && d <= int64_t(INT_MAX) - kBK && V >= 1 && V <= INT_MAX;
}

bool inputs_ok(const void* H, const void* W, const float* temperature, const uint32_t* mask,
               int64_t mask_ld, int64_t B, int64_t d, int64_t V, int64_t ldh, int64_t ldw,
               int64_t vocab_offset) {
  if (!sizes_ok(B, d, V) || !H || !W || !aligned(H, 16) || !aligned(W, 16)) return false;
  if (ldh < d || ldw < d || ldh % 8 != 0 || ldw % 8 != 0) return false;
  if (temperature && !aligned(temperature, 4)) return false;
  if (mask && (!aligned(mask, 4) || mask_ld < ceil_div(V, 32))) return false;
  return vocab_offset >= 0 && vocab_offset + V <= INT_MAX;
}

template <int KC>
fs_status run_scores(const fs_logprobs_args* a, const Device& dev, cudaStream_t stream) {
  const int64_t chunk = rows_per_launch(a->B);
  for (int64_t b0 = 0; b0 < a->B; b0 += chunk) {
    const int64_t rows = std::min(chunk, a->B - b0);
    const bool pair = rows > kBM;
    const int n_mt = pair ? int(ceil_div(rows, 2 * kBM)) : 1;
    const int cols = pair ? kBN : unit_cols(a->V, 64);
    const int n_nt = int(ceil_div(a->V, cols));
    const int groups = balanced(n_nt, (pair ? dev.pairs : dev.sms) / n_mt);
    const int n_slots = 2 * groups;
    const int box_rows = pair ? kBM : int(std::min<int64_t>(kBM, (rows + 7) / 8 * 8));
    const auto* H = static_cast<const __nv_bfloat16*>(a->H) + b0 * a->ldh;
    CUtensorMap mh, mw;
    if (!encode(dev, &mh, H, a->d, rows, a->ldh, box_rows) ||
        !encode(dev, &mw, a->W, a->d, a->V, a->ldw, pair ? kBN / 2 : cols))
      return FS_ERR_INVALID_ARG;
    Shape s = {};
    s.n_mt = n_mt;
    s.n_nt = n_nt;
    s.n_units = n_mt * n_nt;
    s.n_kb = int32_t(ceil_div(a->d, kBK));
    s.n_splits = 1;
    s.m_rows = int32_t(rows);
    s.n_cols = int32_t(a->V);
    s.m_fastest = 1;
    s.a_box_rows = uint32_t(box_rows);
    s.policy_a = kPolicyLast;
    s.policy_b = n_mt > 1 ? kPolicyNormal : kPolicyFirst;
    s.pdl = (a->flags & FS_FLAG_OVERLAP_PREVIOUS) && b0 == 0;
    ScoreParams ep = {};
    ep.B = int32_t(rows);
    ep.V = int32_t(a->V);
    ep.temperature = a->temperature ? a->temperature + b0 : nullptr;
    ep.mask = a->vocab_mask ? a->vocab_mask + b0 * a->mask_ld : nullptr;
    ep.mask_ld = a->mask_ld;
    ep.n_slots = n_slots;
    // A unit of few rows and a long k takes longer to stream than its logits to insert one
    // by one, and the code of the sorting start is not fetched (start sorted / inserted, us:
    // 64 rows, d = 4096, V = 151936, K = 5 197.1 / 195.0, 1 row, K = 20 198.7 / 196.9; with
    // fewer units a CTA, 64 rows, V = 60000, K = 20 103.0 / 108.6, or a shorter k, 1 row,
    // d = 2048, V = 100000, K = 20 75.1 / 83.7, the first unit's logits hold the rest up).
    ep.sorted_start = pair || s.n_kb < 64 || s.n_units < 3 * groups;
    ep.tokens = a->tokens ? a->tokens + b0 : nullptr;
    ep.vocab_offset = a->vocab_offset;
    uint8_t* ws = static_cast<uint8_t*>(a->workspace);
    ep.part = reinterpret_cast<RowPart*>(ws);
    ep.ref = reinterpret_cast<RowRef*>(ep.part + size_t(rows) * n_slots);  // without lists
    ws += round256(size_t(rows) * n_slots * sizeof(RowPart));
    ep.cand_val = reinterpret_cast<float*>(ws);
    ws += round256(size_t(rows) * n_slots * KC * 4u);
    ep.cand_id = reinterpret_cast<int32_t*>(ws);
    const bool overlap = s.pdl != 0;
    const int workers = groups * n_mt;
    fs_status st;
    if (pair)
      st = launch<ScoreEpi<KC, 256>, true, false, false>(dev, mh, mw, mh, s, ep, workers, overlap,
                                                         stream);
    else if (cols == 256)
      st = launch<ScoreEpi<KC, 256>, false, false, false>(dev, mh, mw, mh, s, ep, workers, overlap,
                                                          stream);
    else if (cols == 128)
      st = launch<ScoreEpi<KC, 128>, false, false, false>(dev, mh, mw, mh, s, ep, workers, overlap,
                                                          stream);
    else
      st = launch<ScoreEpi<KC, 64>, false, false, false>(dev, mh, mw, mh, s, ep, workers, overlap,
                                                         stream);
    if (st != FS_OK) return st;
    JoinParams j = {};
    j.H = H;
    j.W = static_cast<const __nv_bfloat16*>(a->W);
    j.ldh = a->ldh;
    j.ldw = a->ldw;
    j.d = int32_t(a->d);
    j.V = int32_t(a->V);
    j.n_slots = n_slots;
    j.K = int32_t(a->K);
    j.temperature = ep.temperature;
    j.mask = ep.mask;
    j.mask_ld = a->mask_ld;
    j.n_kb = s.n_kb;
    j.tokens = ep.tokens;
    j.vocab_offset = a->vocab_offset;
    j.part = ep.part;
    j.ref = ep.ref;
    j.cand_val = ep.cand_val;
    j.cand_id = ep.cand_id;
    j.out_logp = a->out_logp ? a->out_logp + b0 : nullptr;
    j.out_entropy = a->out_entropy ? a->out_entropy + b0 : nullptr;
    j.out_lse = a->out_lse ? a->out_lse + b0 : nullptr;
    j.out_topk_idx = KC ? a->out_topk_idx + b0 * a->K : nullptr;
    j.out_topk_logp = KC ? a->out_topk_logp + b0 * a->K : nullptr;
    if (launch_join<KC>(j, rows, stream) != cudaSuccess) {
      cudaGetLastError();
      return FS_ERR_CUDA;
    }
  }
  return FS_OK;
}

// ---- gradient ------------------------------------------------------------

// How dH = G W is split along k (the vocabulary).  Unsplit, the tiles of
// [B, d] leave workers idle or in a thin last wave; each split adds partial tiles
// written and read in fp32 and a kernel to sum them.  Costs in us as measured: a
// k slice 0.33 (0.45 unsplit: its ring is shorter by the store's staging; 6 rows at
// d = 4193, V = 1940, 31 slices, unsplit 18.7 us with G's 19, in 4 splits 5.5), 8
// slices to fill the pipeline and drain a tile, 4 for the sum kernel and 0.06 for
// each partial tile.
int64_t plan_split(int64_t B, int64_t d, int64_t V) {
  const bool pair = B > kBM;
  const int64_t workers = pair ? kPlanSms / 2 : kPlanSms;
  const int64_t tiles = ceil_div(B, pair ? 2 * kBM : kBM) * ceil_div(d, kBN);
  const int64_t n_kb = ceil_div(V, kBK);
  int64_t best = 1;
  double best_cost = 1e300;
  for (int64_t want = 1; want <= 64 && want <= n_kb; ++want) {
    const int64_t kb = ceil_div(n_kb, want), n = ceil_div(n_kb, kb);
    const int64_t waves = ceil_div(tiles * n, workers);
    const double sum = n > 1 ? 4.0 + 0.06 * double(n * tiles * (pair ? 2 : 1)) : 0.0;
    const double cost = double(waves * (kb + 8)) * (n > 1 ? 0.33 : 0.45) + sum;
    if (cost < best_cost) {
      best_cost = cost;
      best = n;
    }
  }
  return best;
}

// Columns of a result's store map (StoreEpi::Params::whole_n; unused below 8).
int64_t store_cols(int64_t d) { return d < 8 ? 8 : d & ~int64_t(7); }

size_t g_bytes(int64_t B, int64_t V) { return round256(size_t(B) * size_t((V + 7) / 8 * 8) * 2u); }
size_t delta_bytes(int64_t B) { return round256(size_t(B) * 4u); }
size_t marks_bytes(int64_t B, int64_t V) {  // whole units of ids
  return round256(size_t(ceil_div(V, kBN)) * (kBN / 32) * size_t(ceil_div(B, 32)) * sizeof(uint4));
}
size_t partial_bytes(int64_t B, int64_t d, int64_t V) {
  const int64_t n = plan_split(B, d, V);
  if (n == 1) return 0;
  const int64_t ctas = B > kBM ? 2 : 1;
  return size_t(n * ceil_div(B, kBM * ctas) * ceil_div(d, kBN) * ctas) * kBM * kBN * 4u;
}

}  // namespace
}  // namespace vocab
}  // namespace fs

using namespace fs::vocab;

extern "C" size_t fs_logprobs_workspace_size(int64_t B, int64_t V, int64_t K) {
  if (!sizes_ok(B, 1, V) || K < 0 || K > FS_LOGPROBS_TOPK_MAX) return 0;
  const int64_t rows = std::min(B, rows_per_launch(B));
  const int KC = list_cap(K);
  size_t most = 0;
  // The last launch may have fewer rows, and so more slots a row.
  for (const int64_t r : {rows, B % rows == 0 ? rows : B % rows}) {
    const size_t entries = size_t(r) * size_t(plan_slots(r, V));
    const size_t own = sizeof(RowPart) + (KC == 0 ? sizeof(RowRef) : 0);
    most = std::max(most, round256(entries * own) + 2 * round256(entries * KC * 4u));
  }
  return most;
}

extern "C" fs_status fs_logprobs(const fs_logprobs_args* a, void* stream_ptr) {
  if (a == nullptr) return FS_ERR_INVALID_ARG;
  if (!inputs_ok(a->H, a->W, a->temperature, a->vocab_mask, a->mask_ld, a->B, a->d, a->V, a->ldh,
                 a->ldw, a->vocab_offset))
    return FS_ERR_INVALID_ARG;
  if ((a->flags & ~uint32_t(FS_FLAG_OVERLAP_PREVIOUS)) != 0) return FS_ERR_INVALID_ARG;
  if (a->K < 0 || a->K > FS_LOGPROBS_TOPK_MAX) return FS_ERR_INVALID_ARG;
  if ((a->tokens == nullptr) != (a->out_logp == nullptr)) return FS_ERR_INVALID_ARG;
  if ((a->K > 0) != (a->out_topk_idx != nullptr) || (a->K > 0) != (a->out_topk_logp != nullptr))
    return FS_ERR_INVALID_ARG;
  if (!a->out_logp && !a->out_entropy && !a->out_lse && a->K == 0) return FS_ERR_INVALID_ARG;
  if ((a->tokens && !aligned(a->tokens, 8)) || (a->out_logp && !aligned(a->out_logp, 4)) ||
      (a->out_entropy && !aligned(a->out_entropy, 4)) || (a->out_lse && !aligned(a->out_lse, 4)) ||
      (a->out_topk_idx && !aligned(a->out_topk_idx, 8)) ||
      (a->out_topk_logp && !aligned(a->out_topk_logp, 4)))
    return FS_ERR_INVALID_ARG;
  if (!a->workspace || !aligned(a->workspace, 256) ||
      a->workspace_bytes < fs_logprobs_workspace_size(a->B, a->V, a->K))
    return FS_ERR_WORKSPACE;
  const Device* dev = nullptr;
  const fs_status st = device_setup(&dev);
  if (st != FS_OK) return st;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  switch (list_cap(a->K)) {
    case 0: return run_scores<0>(a, *dev, stream);
    case 8: return run_scores<8>(a, *dev, stream);
    case 16: return run_scores<16>(a, *dev, stream);
    default: return run_scores<24>(a, *dev, stream);
  }
}

namespace {
// Sizes whose units or partial tiles would overflow the kernels' 32-bit counts.
bool grad_sizes_ok(int64_t B, int64_t d, int64_t V) {
  return sizes_ok(B, d, V) && ceil_div(V, kBM) * ceil_div(d, kBN) <= INT_MAX &&
         ceil_div(V, kBN) * ceil_div(B, kBM) <= INT_MAX &&
         (ceil_div(B, kBM) + 1) * ceil_div(d, kBN) * 64 <= INT_MAX;
}
}  // namespace

extern "C" size_t fs_logprobs_grad_workspace_size(int64_t B, int64_t d, int64_t V) {
  if (!grad_sizes_ok(B, d, V)) return 0;
  return g_bytes(B, V) + delta_bytes(B) + marks_bytes(B, V) + partial_bytes(B, d, V);
}

extern "C" fs_status fs_logprobs_grad(const fs_logprobs_grad_args* a, void* stream_ptr) {
  if (a == nullptr) return FS_ERR_INVALID_ARG;
  if (!inputs_ok(a->H, a->W, a->temperature, a->vocab_mask, a->mask_ld, a->B, a->d, a->V, a->ldh,
                 a->ldw, a->vocab_offset) ||
      !grad_sizes_ok(a->B, a->d, a->V))
    return FS_ERR_INVALID_ARG;
  if (!a->tokens || !a->lse || !a->grad_logp || !aligned(a->tokens, 8) || !aligned(a->lse, 4) ||
      !aligned(a->grad_logp, 4))
    return FS_ERR_INVALID_ARG;
  if ((a->entropy == nullptr) != (a->grad_entropy == nullptr) ||
      (a->entropy && (!aligned(a->entropy, 4) || !aligned(a->grad_entropy, 4))))
    return FS_ERR_INVALID_ARG;
  if (!a->out_dH && !a->out_dW) return FS_ERR_INVALID_ARG;
  if (a->out_dH && (!aligned(a->out_dH, 16) || a->lddh < a->d || a->lddh % 8 != 0))
    return FS_ERR_INVALID_ARG;
  if (a->out_dW && (!aligned(a->out_dW, 16) || a->lddw < a->d || a->lddw % 8 != 0))
    return FS_ERR_INVALID_ARG;
  if (!a->workspace || !aligned(a->workspace, 256) ||
      a->workspace_bytes < fs_logprobs_grad_workspace_size(a->B, a->d, a->V))
    return FS_ERR_WORKSPACE;
  const Device* dp = nullptr;
  fs_status st = device_setup(&dp);
  if (st != FS_OK) return st;
  const Device& dev = *dp;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  const int64_t B = a->B, d = a->d, V = a->V, ldg = (V + 7) / 8 * 8;
  void* G = a->workspace;
  uint8_t* behind_g = static_cast<uint8_t*>(G) + g_bytes(B, V);
  float* delta = reinterpret_cast<float*>(behind_g);
  uint4* marks = reinterpret_cast<uint4*>(behind_g + delta_bytes(B));
  const bool pair = B > kBM;
  const int ctas = pair ? 2 : 1;
  const int workers = pair ? dev.pairs : dev.sms;

  // G: the logits again, as in the forward pass.
  {
    const int box_rows = pair ? kBM : int(std::min<int64_t>(kBM, (B + 7) / 8 * 8));
    const int cols = pair ? kBN : unit_cols(V, 128);  // a box of 64 columns a half
    CUtensorMap mh, mw, mg;
    if (!encode(dev, &mh, a->H, d, B, a->ldh, box_rows) ||
        !encode(dev, &mw, a->W, d, V, a->ldw, pair ? kBN / 2 : cols) ||
        !encode(dev, &mg, G, ldg, B, ldg, 32))  // its padding columns are written (as 0)
      return FS_ERR_INVALID_ARG;
    Shape s = {};
    s.n_mt = int32_t(ceil_div(B, kBM * ctas));
    s.n_nt = int32_t(ceil_div(V, cols));
    s.n_units = s.n_mt * s.n_nt;
    s.n_kb = int32_t(ceil_div(d, kBK));
    s.n_splits = 1;
    s.m_rows = int32_t(B);
    s.n_cols = int32_t(V);
    s.m_fastest = 1;
    s.a_box_rows = uint32_t(box_rows);
    s.policy_a = kPolicyLast;
    s.policy_b = kPolicyNormal;
    s.early_trigger = 1;
    GradParams ep = {};
    ep.B = int32_t(B);
    ep.V = int32_t(V);
    ep.d = int32_t(d);
    ep.H = static_cast<const __nv_bfloat16*>(a->H);
    ep.W = static_cast<const __nv_bfloat16*>(a->W);
    ep.ldh = a->ldh;
    ep.ldw = a->ldw;
    ep.temperature = a->temperature;
    ep.mask = a->vocab_mask;
    ep.mask_ld = a->mask_ld;
    ep.tokens = a->tokens;
    ep.lse = a->lse;
    ep.entropy = a->entropy;
    ep.grad_logp = a->grad_logp;
    ep.grad_entropy = a->grad_entropy;
    ep.vocab_offset = a->vocab_offset;
    ep.delta = delta;
    ep.marks = marks;
    const int n = balanced(s.n_units, workers);
    if (pair)
      st = launch<GradEpi<256>, true, false, false>(dev, mh, mw, mg, s, ep, n, false, stream);
    else if (cols == 256)
      st = launch<GradEpi<256>, false, false, false>(dev, mh, mw, mg, s, ep, n, false, stream);
    else
      st = launch<GradEpi<128>, false, false, false>(dev, mh, mw, mg, s, ep, n, false, stream);
    if (st != FS_OK) return st;
  }

  // dH = G W.
  const int64_t n_splits = a->out_dH ? plan_split(B, d, V) : 1;
  CUtensorMap hg, hw, ho;
  Shape h = {};
  if (a->out_dH) {
    const int box_rows = pair ? kBM : int(std::min<int64_t>(kBM, (B + 7) / 8 * 8));
    if (!encode(dev, &hg, G, V, B, ldg, box_rows) || !encode(dev, &hw, a->W, d, V, a->ldw, kBK) ||
        !encode(dev, &ho, a->out_dH, store_cols(d), B, a->lddh, 32))
      return FS_ERR_INVALID_ARG;
    h.n_mt = int32_t(ceil_div(B, kBM * ctas));
    h.n_nt = int32_t(ceil_div(d, kBN));
    h.n_units = int32_t(h.n_mt * h.n_nt * n_splits);
    h.n_kb = int32_t(ceil_div(V, kBK));
    h.n_splits = int32_t(n_splits);
    h.k_descending = 1;  // from the ids whose rows of W and columns of G came last
    h.m_rows = int32_t(B);
    h.n_cols = int32_t(d);
    h.m_fastest = 1;
    h.a_box_rows = uint32_t(box_rows);
    h.pdl = h.early_trigger = 1;  // W streams while the kernel before ends
  }

  // dW = G^T H: M is the vocabulary, so the units of one vocabulary block
  // (its slice of G) run over the columns of H next to one another.
  const bool both = a->out_dH && a->out_dW && n_splits > 1 && h.n_units * 3 <= workers * 2 &&
                    ceil_div(V, kBM * ctas) * ceil_div(d, kBN) <= 8 * (workers - h.n_units);
  const bool wpair = both ? pair : V > kBM;
  CUtensorMap wg, wh, wo;
  Shape w = {};
  if (a->out_dW) {
    if (!encode(dev, &wg, G, V, B, ldg, kBK) || !encode(dev, &wh, a->H, d, B, a->ldh, kBK) ||
        !encode(dev, &wo, a->out_dW, store_cols(d), V, a->lddw, 32))
      return FS_ERR_INVALID_ARG;
    w.n_mt = int32_t(ceil_div(V, wpair ? 2 * kBM : kBM));
    w.n_nt = int32_t(ceil_div(d, kBN));
    w.n_units = w.n_mt * w.n_nt;
    w.n_kb = int32_t(ceil_div(B, kBK));
    w.n_splits = 1;
    w.m_rows = int32_t(V);
    w.n_cols = int32_t(d);
    w.policy_b = kPolicyLast;
    w.pdl = 1;  // H streams while the kernel before ends
    w.early_trigger = both;
  }
  const int32_t whole_d = int32_t(d & ~int64_t(7));
  const Rounding h_rounding = {delta, marks, a->tokens, a->vocab_offset, int32_t(B), int32_t(V),
                               static_cast<const __nv_bfloat16*>(a->W), a->ldw};
  const PartialEpi::Params hp = {
      reinterpret_cast<float4*>(behind_g + delta_bytes(B) + marks_bytes(B, V)), ctas};
  const StoreEpi<false>::Params wp = {static_cast<__nv_bfloat16*>(a->out_dW), a->lddw, whole_d,
                                      {delta, marks, a->tokens, a->vocab_offset, int32_t(B),
                                       int32_t(V), static_cast<const __nv_bfloat16*>(a->H),
                                       a->ldh}};

  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;  // of pairs
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (both) {
    if (pair) {
      fill_ring<PartialEpi, true, false>(dev, h);
      fill_ring<StoreEpi<false>, true, true>(dev, w);
    } else {
      fill_ring<PartialEpi, false, false>(dev, h);
      fill_ring<StoreEpi<false>, false, true>(dev, w);
    }
    const int n_w = balanced(w.n_units, workers - h.n_units);
    cfg.gridDim = dim3(unsigned((h.n_units + n_w) * ctas), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = kBothSmem;
    cfg.numAttrs = pair ? 2 : 1;
    const int n_h = h.n_units * ctas;
    if (cudaLaunchKernelEx(&cfg, pair ? both_kernel<true> : both_kernel<false>, hg, hw, wg, wh,
                           wo, h, w, hp, wp, n_h) != cudaSuccess) {
      cudaGetLastError();
      return FS_ERR_CUDA;
    }
    cfg.numAttrs = 1;
  } else if (a->out_dH) {
    const int n = balanced(h.n_units, workers);
    if (n_splits == 1) {
      using Epi = StoreEpi<true>;
      const Epi::Params ep = {static_cast<__nv_bfloat16*>(a->out_dH), a->lddh, whole_d,
                              h_rounding};
      st = pair ? launch<Epi, true, false, true>(dev, hg, hw, ho, h, ep, n, true, stream)
                : launch<Epi, false, false, true>(dev, hg, hw, ho, h, ep, n, true, stream);
    } else {
      st = pair ? launch<PartialEpi, true, false, true>(dev, hg, hw, ho, h, hp, n, true, stream)
                : launch<PartialEpi, false, false, true>(dev, hg, hw, ho, h, hp, n, true, stream);
    }
    if (st != FS_OK) return st;
  }
  if (n_splits > 1) {
    cfg.gridDim = dim3(unsigned(h.n_mt * h.n_nt * ctas * kSumBlocksPerTile), 1, 1);
    cfg.blockDim = dim3(kSumThreads, 1, 1);
    cfg.dynamicSmemBytes = 0;
    if (cudaLaunchKernelEx(&cfg, sum_splits_kernel, static_cast<const float4*>(hp.partial),
                           int32_t(n_splits), h.n_mt * h.n_nt, h.n_nt, int32_t(ctas), int32_t(B),
                           int32_t(d), h_rounding, static_cast<__nv_bfloat16*>(a->out_dH),
                           a->lddh) != cudaSuccess) {
      cudaGetLastError();
      return FS_ERR_CUDA;
    }
  }
  if (a->out_dW && !both) {
    using Epi = StoreEpi<false>;
    const int n = balanced(w.n_units, wpair ? dev.pairs : dev.sms);
    st = wpair ? launch<Epi, true, true, true>(dev, wg, wh, wo, w, wp, n, true, stream)
               : launch<Epi, false, true, true>(dev, wg, wh, wo, w, wp, n, true, stream);
    if (st != FS_OK) return st;
  }
  return FS_OK;
}
