// fs_logprobs.cu -- token log-probabilities, entropy and top alternatives from
// hidden states and the LM head, and their gradient (fs_vocab.h).
//
// Forward, two kernels.  The contraction kernel (fs_contract.cuh) streams W
// past a block of rows; a CTA (pair) keeps its block of rows for the whole
// launch, so each epilogue thread owns one row and half of the vocabulary
// blocks its CTA visits, and carries in registers, in one pass over its logits,
//   m = max x,  S = sum 2^(x-m),  U = sum 2^(x-m) (x-m)      (x in base-2 units)
// and the best KC raw logits with their ids.  A second kernel joins the
// threads' states of a row and ranks its alternatives.
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

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float row_temperature(const float* temperature, int row) {
  const float T = temperature ? temperature[row] : 1.0f;
  return (T > 0.0f && !isinf(T)) ? T : 1.0f;
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

// One thread's state of a row, as left in the workspace.
struct RowPart {
  float m, S, U, unused;
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

template <int KC>
struct ScoreEpi {
  static constexpr bool kStaged = false;
  struct Params {
    int32_t B, V;  // rows of this launch, ids
    const float* temperature;
    const uint32_t* mask;
    int64_t mask_ld;
    RowPart* part;     // [B][n_slots]
    float* cand_val;   // [B][n_slots][KC] raw logits, best first
    int32_t* cand_id;  // ids from 0, -1 past the end
    int32_t n_slots;
  };
  struct State {
    float m = -INFINITY, S = 0.0f, U = 0.0f;  // m: the largest raw logit
    float scale2 = 0.0f;                      // log2(e) / T
    const uint32_t* mrow = nullptr;
    int row = -1;
    float ts[KC > 0 ? KC : 1];
    int32_t ti[KC > 0 ? KC : 1];
  };
  static __device__ __forceinline__ void start(const Params&, State& st) {
#pragma unroll
    for (int q = 0; q < KC; ++q) {
      st.ts[q] = -INFINITY;
      st.ti[q] = -1;
    }
  }
  // 32 logits.  kMasked: a cleared id's logit counts as -inf, whatever it is.
  template <bool kMasked>
  static __device__ __forceinline__ void chunk(State& st, uint32_t (&r)[32], uint32_t allow) {
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      if (kMasked) r[j] = ((allow >> j) & 1u) ? r[j] : 0xFF800000u;
      top = ptx::max_nan(top, __uint_as_float(r[j]));
    }
    if (top == -INFINITY) return;  // nothing allowed (false for NaN)
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
  }
  static __device__ __forceinline__ void tile(const Params& p, State& st, const TileAt& at,
                                              int lane, uint8_t*, const void*, const Shape&) {
    const int row = at.row0 + lane;
    const bool valid = row < p.B;
    if (valid && st.row < 0) {  // the thread's row, the same in every unit
      st.row = row;
      st.scale2 = kLog2e / row_temperature(p.temperature, row);
      if (p.mask) st.mrow = p.mask + int64_t(row) * p.mask_ld;
    }
    const AllowWords allow(st.mrow, at.col0, p.V);
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
      if (at.col0 + c * 32 >= p.V) break;
      uint32_t r[32];
      ptx::tmem_ld_32x32b_x32(at.taddr + uint32_t(c * 32), r);
      ptx::tmem_wait_ld();
      const uint32_t w = allow.at(c);
      const bool full = __all_sync(0xFFFFFFFFu, !valid || w == 0xFFFFFFFFu);
      if (valid) {
        if (full)
          chunk<false>(st, r, w);
        else
          chunk<true>(st, r, w);
      }
      if constexpr (KC > 0) {
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
            const float v = pick32(r, j);
            if (v > st.ts[KC - 1]) list_insert<KC>(st.ts, st.ti, v, at.col0 + c * 32 + int(j));
          }
        }
      }
    }
  }
  static __device__ __forceinline__ void finish(const Params& p, State& st, int worker, int row,
                                                int half, const Shape& s) {
    // A slot per (group of workers on the same vocabulary blocks, half); every
    // one is written, also by a thread whose 128 columns lay past V.
    if (row >= p.B) return;
    const int64_t slot = int64_t(row) * p.n_slots + (worker / s.n_mt) * 2 + half;
    const float m2 = st.m == -INFINITY ? st.m : st.m * st.scale2;
    p.part[slot] = RowPart{m2, st.S, st.U, 0.0f};
    if constexpr (KC > 0) {
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
  const float* temperature;
  const uint32_t* mask;
  int64_t mask_ld;
  const int64_t* tokens;
  int64_t vocab_offset;
  const RowPart* part;
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
// as an unevaluated pair (hi, lo), so the result is good to about 2^-45 of the
// terms' magnitude.  Every lane returns it; the order of the terms depends on
// d alone.
__device__ __forceinline__ double warp_logit(const __nv_bfloat16* __restrict__ h,
                                             const __nv_bfloat16* __restrict__ w, int d,
                                             int lane) {
  float hi = 0.0f, lo = 0.0f;
  const int n8 = d >> 3;
#pragma unroll 4
  for (int i = lane; i < n8; i += 32) {
    const uint4 a = reinterpret_cast<const uint4*>(h)[i];
    const uint4 b = reinterpret_cast<const uint4*>(w)[i];
    const uint32_t av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float err;
      hi = two_sum(hi, __fmul_rn(__uint_as_float(av[q] << 16), __uint_as_float(bv[q] << 16)), err);
      lo = __fadd_rn(lo, err);
      hi = two_sum(hi,
                   __fmul_rn(__uint_as_float(av[q] & 0xFFFF0000u),
                             __uint_as_float(bv[q] & 0xFFFF0000u)),
                   err);
      lo = __fadd_rn(lo, err);
    }
  }
  const int tail = n8 * 8 + lane;
  if (tail < d) {
    float err;
    hi = two_sum(hi, __fmul_rn(__bfloat162float(h[tail]), __bfloat162float(w[tail])), err);
    lo = __fadd_rn(lo, err);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    const float ohi = __shfl_xor_sync(0xFFFFFFFFu, hi, off);
    const float olo = __shfl_xor_sync(0xFFFFFFFFu, lo, off);
    float err;
    hi = two_sum(hi, ohi, err);
    lo = __fadd_rn(__fadd_rn(lo, olo), err);
  }
  return isfinite(hi) ? double(hi) + double(lo) : double(hi);
}

// An order-preserving map of non-NaN floats to unsigned integers above 0 (-0
// folded into +0).
__device__ __forceinline__ uint32_t order_key(float f) {
  const uint32_t u = __float_as_uint(f + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

// The warp's n best entries of up to 32 sorted lists, one per lane, in shared
// memory: n rounds of the best head, lower id on ties, popped by its lane.
template <typename Emit>
__device__ __forceinline__ void warp_best(const float* val, const int32_t* id, int len, bool has,
                                          int n, Emit emit) {
  int pos = 0;
  uint32_t key = 0u;
  int32_t head = INT_MAX;
  auto load = [&]() {
    const bool more = has && pos < len && id[pos] >= 0;
    key = more ? order_key(val[pos]) : 0u;
    head = more ? id[pos] : INT_MAX;
  };
  load();
  for (int j = 0; j < n; ++j) {
    const uint32_t best = __reduce_max_sync(0xFFFFFFFFu, key);
    const int32_t who = __reduce_min_sync(0xFFFFFFFFu, key == best ? head : INT_MAX);
    if (best == 0u) {
      emit(j, -INFINITY, -1);
      continue;
    }
    emit(j, key_value(best), who);
    if (key == best && head == who) {
      ++pos;
      load();
    }
  }
}

template <int KC>
constexpr int kJoinThreads = KC > 0 ? 320 : 128;
// At most one slot per thread of a warp-select: 2 * 152 slots in 10 warps.
constexpr int kMaxSlots = 320;

// One block per row.  Launched as a programmatic dependent of the contraction.
template <int KC>
__global__ void __launch_bounds__(kJoinThreads<KC>) join_kernel(const JoinParams p) {
  constexpr int kThreadsJ = kJoinThreads<KC>;
  constexpr int kWarps = kThreadsJ / 32;
  constexpr int kList = KC > 0 ? KC : 1;
  extern __shared__ __align__(16) uint8_t dyn[];  // the row's lists
  __shared__ float s_m[kWarps], s_S[kWarps], s_U[kWarps];
  __shared__ float s_wv[kWarps * kList];
  __shared__ int32_t s_wi[kWarps * kList];
  __shared__ int32_t s_id[kList + 1];
  __shared__ double s_logit[kList + 1];
  const int row = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  ptx::grid_dependency_wait();

  // ---- the row's lists into shared memory
  float* lv = reinterpret_cast<float*>(dyn);
  int32_t* li = reinterpret_cast<int32_t*>(lv + p.n_slots * KC);
  if constexpr (KC > 0) {
    const float4* v4 = reinterpret_cast<const float4*>(p.cand_val + int64_t(row) * p.n_slots * KC);
    const int4* i4 = reinterpret_cast<const int4*>(p.cand_id + int64_t(row) * p.n_slots * KC);
    for (int i = threadIdx.x; i < p.n_slots * KC / 4; i += kThreadsJ) {
      reinterpret_cast<float4*>(lv)[i] = v4[i];
      reinterpret_cast<int4*>(li)[i] = i4[i];
    }
  }

  // ---- statistics: threads in slot order, then lanes, then warps
  const RowPart* part = p.part + int64_t(row) * p.n_slots;
  float m = -INFINITY, S = 0.0f, U = 0.0f;
  auto join = [](float& m0, float& S0, float& U0, float m1, float S1, float U1) {
    if (m1 == -INFINITY) return;
    if (m0 == -INFINITY) {
      m0 = m1, S0 = S1, U0 = U1;
      return;
    }
    const float mm = ptx::max_nan(m0, m1);
    const float d0 = ptx::max_nan(m0 - mm, -16384.0f), d1 = ptx::max_nan(m1 - mm, -16384.0f);
    const float f0 = exp2f(d0), f1 = exp2f(d1);
    U0 = f0 * fmaf(d0, S0, U0) + f1 * fmaf(d1, S1, U1);
    S0 = f0 * S0 + f1 * S1;
    m0 = mm;
  };
  for (int i = threadIdx.x; i < p.n_slots; i += kThreadsJ) {
    const RowPart r = part[i];
    join(m, S, U, r.m, r.S, r.U);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    const float om = __shfl_xor_sync(0xFFFFFFFFu, m, off);
    const float oS = __shfl_xor_sync(0xFFFFFFFFu, S, off);
    const float oU = __shfl_xor_sync(0xFFFFFFFFu, U, off);
    join(m, S, U, om, oS, oU);
  }
  if (lane == 0) s_m[warp] = m, s_S[warp] = S, s_U[warp] = U;
  __syncthreads();
  m = s_m[0], S = s_S[0], U = s_U[0];
  for (int w = 1; w < kWarps; ++w) join(m, S, U, s_m[w], s_S[w], s_U[w]);
  const bool none = m == -INFINITY;
  const float log2S = log2f(S);
  const float lse = none ? -INFINITY : kLn2 * (m + log2S);

  // ---- candidates: the K + 4 best fp32 sums of all lists
  const int n_cand = KC > 0 ? p.K + 4 : 0;  // at most KC
  if constexpr (KC > 0) {
    const int slot = threadIdx.x;
    warp_best(lv + slot * KC, li + slot * KC, KC, slot < p.n_slots, n_cand,
              [&](int j, float v, int32_t id) {
                if (lane == 0) s_wv[warp * KC + j] = v, s_wi[warp * KC + j] = id;
              });
    __syncthreads();
    if (warp == 0)
      warp_best(s_wv + lane * KC, s_wi + lane * KC, n_cand, lane < kWarps, n_cand,
                [&](int j, float, int32_t id) {
                  if (lane == 0) s_id[j] = id;
                });
  }
  // ---- the token
  int64_t token = -1, local = -1;
  bool scored = false;  // its logit is wanted
  if (p.tokens) {
    token = p.tokens[row];
    local = token - p.vocab_offset;
    scored = token >= 0 && local >= 0 && local < p.V;
    if (scored && p.mask)
      scored = (p.mask[int64_t(row) * p.mask_ld + (local >> 5)] >> (local & 31)) & 1u;
  }
  if (threadIdx.x == 0) s_id[n_cand] = scored ? int32_t(local) : -1;
  __syncthreads();
  // ---- their logits again, compensated
  for (int j = warp; j <= n_cand; j += kWarps) {
    const int32_t id = s_id[j];
    if (id < 0) continue;
    const double l = warp_logit(p.H + int64_t(row) * p.ldh, p.W + int64_t(id) * p.ldw, p.d, lane);
    // NaN (the row's lse is NaN too) ranks first, so every place is filled.
    if (lane == 0) s_logit[j] = l == l ? l : double(INFINITY);
  }
  __syncthreads();
  const double inv_t = 1.0 / double(row_temperature(p.temperature, row));
  if (threadIdx.x == 0) {
    if (p.out_lse) p.out_lse[row] = lse;
    if (p.out_entropy) p.out_entropy[row] = none ? 0.0f : kLn2 * (log2S - U / S);
    if (p.tokens)
      p.out_logp[row] = token < 0 ? 0.0f
                        : !scored ? -INFINITY
                                  : float(s_logit[n_cand] * inv_t - double(lse));
  }
  if constexpr (KC > 0) {
    if (int(threadIdx.x) < n_cand) {
      const int j = threadIdx.x;
      const int32_t id = s_id[j];
      const double l = id < 0 ? 0.0 : s_logit[j];
      int rank = 0;
      for (int i = 0; i < n_cand; ++i) {
        const int32_t oi = s_id[i];
        if (oi < 0 || i == j) continue;
        rank += (id < 0 || s_logit[i] > l || (s_logit[i] == l && oi < id)) ? 1 : 0;
      }
      if (id < 0) rank = j;  // absent entries come last, in place
      if (rank < p.K) {
        const int64_t o = int64_t(row) * p.K + rank;
        p.out_topk_idx[o] = id < 0 ? -1 : p.vocab_offset + id;
        p.out_topk_logp[o] = id < 0 ? -INFINITY : float(l * inv_t - double(lse));
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Backward: G = dLoss / dlogits
// ---------------------------------------------------------------------------

struct GradEpi {
  static constexpr bool kStaged = true;
  struct Params {
    int32_t B, V;
    const float* temperature;
    const uint32_t* mask;
    int64_t mask_ld;
    const int64_t* tokens;
    const float *lse, *entropy, *grad_logp, *grad_entropy;
    int64_t vocab_offset;
  };
  // With a, e the row's upstream gradients over T, P = 2^x the probability and
  // x = log2 p = l scale2 - lse2:  G = P (c0 + c1 x), + a at the token, where
  // c1 = -e ln2, c0 = -a - e entropy.
  struct State {
    int row = -1;
    float scale2, lse2, c0, c1, a;
    int32_t token;  // id from 0, -1 for none
    const uint32_t* mrow;
    bool live;  // false: the row's G is 0
  };
  static __device__ __forceinline__ void start(const Params&, State&) {}
  static __device__ __forceinline__ void load_row(const Params& p, State& st, int row) {
    st.row = row;
    st.mrow = nullptr;
    st.live = false;
    st.token = -1;
    st.scale2 = st.lse2 = st.c0 = st.c1 = st.a = 0.0f;
    if (row >= p.B) return;
    const float T = row_temperature(p.temperature, row);
    const float lse = p.lse[row];
    if (p.mask) st.mrow = p.mask + int64_t(row) * p.mask_ld;
    st.scale2 = kLog2e / T;
    st.lse2 = lse * kLog2e;
    st.live = lse != -INFINITY;
    float a = p.grad_logp[row] / T;
    const int64_t token = p.tokens[row], local = token - p.vocab_offset;
    if (token < 0) {
      a = 0.0f;
    } else if (local >= 0 && local < p.V) {
      st.token = int32_t(local);
      if (st.mrow && !((st.mrow[local >> 5] >> (local & 31)) & 1u)) {
        a = 0.0f;
        st.token = -1;
      }
    }
    st.a = a;
    st.c0 = -a;
    if (p.grad_entropy) {
      const float e = p.grad_entropy[row] / T;
      st.c0 = fmaf(-e, p.entropy[row], -a);
      st.c1 = -e * kLn2;
    }
  }
  static __device__ __forceinline__ void tile(const Params& p, State& st, const TileAt& at,
                                              int lane, uint8_t* box, const void* tmap,
                                              const Shape&) {
    const int row = at.row0 + lane;
    if (row != st.row) load_row(p, st, row);
    const AllowWords allow(st.mrow, at.col0, p.V);
#pragma unroll 1
    for (int c = 0; c < 2; ++c) {
      if (at.col0 + c * 64 >= p.V) break;
      box_begin(lane);
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        uint32_t r[32];
        ptx::tmem_ld_32x32b_x32(at.taddr + uint32_t(c * 64 + h * 32), r);
        ptx::tmem_wait_ld();
        const uint32_t w = st.live ? allow.at(2 * c + h) : 0u;
        const uint32_t tok = uint32_t(st.token - (at.col0 + c * 64 + h * 32));
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float g[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int j = q * 8 + i;
            // Far below 1, p is 0 in fp32; the bound keeps 0 * -inf out of G.
            const float x =
                ptx::max_nan(fmaf(__uint_as_float(r[j]), st.scale2, -st.lse2), -16384.0f);
            float v = ptx::ex2(x) * fmaf(st.c1, x, st.c0);
            if (tok == uint32_t(j)) v += st.a;
            g[i] = ((w >> j) & 1u) ? v : 0.0f;
          }
          box_put(box, lane, h * 4 + q, g);
        }
      }
      box_end(box, tmap, lane, at.col0 + c * 64, at.row0);
    }
  }
  static __device__ __forceinline__ void finish(const Params&, State&, int, int, int,
                                                const Shape&) {}
};

// dH from its k splits, in split order, rounded to bf16 once.  A thread takes
// 8 columns of one row; neighbouring threads take neighbouring rows, the order
// the partial tiles are stored in (PartialEpi).
constexpr int kSumThreads = 256;
__global__ void __launch_bounds__(kSumThreads)
    sum_splits_kernel(const float4* __restrict__ partial, int32_t n_splits, int32_t n_tiles,
                      int32_t n_nt, int32_t ctas, int32_t B, int32_t d,
                      __nv_bfloat16* __restrict__ dH, int64_t lddh) {
  ptx::grid_dependency_wait();
  constexpr int kTile = kBM * kBN / 4;               // float4 of a CTA's tile
  const int tile = blockIdx.x / (kBN / 8 * kBM / kSumThreads);  // (tile of the grid, CTA)
  const int in = blockIdx.x % (kBN / 8 * kBM / kSumThreads) * kSumThreads + threadIdx.x;
  const int r = in % kBM, c8 = in / kBM;  // row, group of 8 columns
  const int t = tile / ctas, rank = tile - t * ctas;
  const int row = (t / n_nt * ctas + rank) * kBM + r;
  const int col = t % n_nt * kBN + c8 * 8;
  if (row >= B || col >= d) return;
  float v[8] = {};
  for (int s = 0; s < n_splits; ++s) {
    const float4* src = partial + ((int64_t(s) * n_tiles + t) * ctas + rank) * kTile +
                        int64_t(c8 * 2) * kBM + r;
    const float4 a = src[0], b = src[kBM];
    v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
    v[4] += b.x, v[5] += b.y, v[6] += b.z, v[7] += b.w;
  }
  __nv_bfloat16* out = dH + int64_t(row) * lddh + col;
  if (col + 8 <= d) {
    __nv_bfloat162 h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<uint4*>(out) = *reinterpret_cast<const uint4*>(h);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (col + i < d) out[i] = __float2bfloat16_rn(v[i]);
  }
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
// Workspaces and k splits are planned for this many SMs (GB300); a device that
// offers fewer co-resident CTA pairs uses less of them.
constexpr int kPlanSms = 152;

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
  return prepare_kernel<ScoreEpi<KC>, false, false, false>(sms, pairs) &&
         prepare_kernel<ScoreEpi<KC>, true, false, false>(sms, pairs) &&
         cudaFuncSetAttribute(join_kernel<KC>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              std::max(1, kMaxSlots * KC * 8)) == cudaSuccess;
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
          prepare_scores<8>(d.sms, &d.pairs) && prepare_scores<24>(d.sms, &d.pairs) &&
          prepare_kernel<GradEpi, false, false, false>(d.sms, &d.pairs) &&
          prepare_kernel<GradEpi, true, false, false>(d.sms, &d.pairs) &&
          prepare_kernel<StoreEpi, false, false, true>(d.sms, &d.pairs) &&
          prepare_kernel<StoreEpi, true, false, true>(d.sms, &d.pairs) &&
          prepare_kernel<PartialEpi, false, false, true>(d.sms, &d.pairs) &&
          prepare_kernel<PartialEpi, true, false, true>(d.sms, &d.pairs) &&
          prepare_kernel<StoreEpi, false, true, true>(d.sms, &d.pairs) &&
          prepare_kernel<StoreEpi, true, true, true>(d.sms, &d.pairs) &&
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

template <class Epi, bool kPair, bool kAmn, bool kBmn>
fs_status launch(const Device& dev, const CUtensorMap& a, const CUtensorMap& b,
                 const CUtensorMap& d, Shape s, const typename Epi::Params& ep, int workers,
                 bool overlap, cudaStream_t stream) {
  constexpr uint32_t kBBytes = (kPair ? kBN / 2 : kBN) * kBK * 2;
  s.a_bytes = kAmn ? kBM * kBK * 2 : s.a_box_rows * 128u;
  s.stage_bytes = s.a_bytes + kBBytes;
  s.n_stages = std::min<uint32_t>(kMaxStages, ring_bytes<Epi>() / s.stage_bytes);
  s.wait_limit_ns = kWaitLimitNs;
  s.error_word = dev.error_word;
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

int list_cap(int64_t K) { return K <= 0 ? 0 : K <= 4 ? 8 : 24; }

// Upper bound of a row's slots: groups of workers x 2 halves.
int64_t plan_slots(int64_t rows, int64_t V) {
  const int64_t workers = rows <= kBM ? kPlanSms : kPlanSms / 2;
  const int64_t n_mt = rows <= kBM ? 1 : ceil_div(rows, 2 * kBM);
  return 2 * std::min(ceil_div(V, kBN), workers / n_mt);
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
    const int n_nt = int(ceil_div(a->V, kBN));
    const int groups = balanced(n_nt, (pair ? dev.pairs : dev.sms) / n_mt);
    const int n_slots = 2 * groups;
    const int box_rows = pair ? kBM : int(std::min<int64_t>(kBM, (rows + 7) / 8 * 8));
    const auto* H = static_cast<const __nv_bfloat16*>(a->H) + b0 * a->ldh;
    CUtensorMap mh, mw;
    if (!encode(dev, &mh, H, a->d, rows, a->ldh, box_rows) ||
        !encode(dev, &mw, a->W, a->d, a->V, a->ldw, pair ? kBN / 2 : kBN))
      return FS_ERR_INVALID_ARG;
    Shape s = {};
    s.n_mt = n_mt;
    s.n_nt = n_nt;
    s.n_units = n_mt * n_nt;
    s.n_kb = s.kb_per_split = int32_t(ceil_div(a->d, kBK));
    s.m_rows = int32_t(rows);
    s.n_cols = int32_t(a->V);
    s.m_fastest = 1;
    s.a_box_rows = uint32_t(box_rows);
    s.policy_a = kPolicyLast;
    s.policy_b = n_mt > 1 ? kPolicyNormal : kPolicyFirst;
    s.pdl = (a->flags & FS_FLAG_OVERLAP_PREVIOUS) && b0 == 0;
    typename ScoreEpi<KC>::Params ep = {};
    ep.B = int32_t(rows);
    ep.V = int32_t(a->V);
    ep.temperature = a->temperature ? a->temperature + b0 : nullptr;
    ep.mask = a->vocab_mask ? a->vocab_mask + b0 * a->mask_ld : nullptr;
    ep.mask_ld = a->mask_ld;
    ep.n_slots = n_slots;
    uint8_t* ws = static_cast<uint8_t*>(a->workspace);
    ep.part = reinterpret_cast<RowPart*>(ws);
    ws += round256(size_t(rows) * n_slots * sizeof(RowPart));
    ep.cand_val = reinterpret_cast<float*>(ws);
    ws += round256(size_t(rows) * n_slots * KC * 4u);
    ep.cand_id = reinterpret_cast<int32_t*>(ws);
    const fs_status st =
        pair ? launch<ScoreEpi<KC>, true, false, false>(dev, mh, mw, mh, s, ep, groups * n_mt,
                                                        s.pdl != 0, stream)
             : launch<ScoreEpi<KC>, false, false, false>(dev, mh, mw, mh, s, ep, groups,
                                                         s.pdl != 0, stream);
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
    j.tokens = a->tokens ? a->tokens + b0 : nullptr;
    j.vocab_offset = a->vocab_offset;
    j.part = ep.part;
    j.cand_val = ep.cand_val;
    j.cand_id = ep.cand_id;
    j.out_logp = a->out_logp ? a->out_logp + b0 : nullptr;
    j.out_entropy = a->out_entropy ? a->out_entropy + b0 : nullptr;
    j.out_lse = a->out_lse ? a->out_lse + b0 : nullptr;
    j.out_topk_idx = KC ? a->out_topk_idx + b0 * a->K : nullptr;
    j.out_topk_logp = KC ? a->out_topk_logp + b0 * a->K : nullptr;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(rows), 1, 1);
    cfg.blockDim = dim3(kJoinThreads<KC>, 1, 1);
    cfg.dynamicSmemBytes = size_t(n_slots) * KC * 8u;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, join_kernel<KC>, j) != cudaSuccess) {
      cudaGetLastError();
      return FS_ERR_CUDA;
    }
  }
  return FS_OK;
}

// ---- gradient ------------------------------------------------------------

// How dH = G W is split along k (the vocabulary).  Unsplit, the tiles of
// [B, d] leave workers idle or in a thin last wave; each split adds a partial
// tile written and read in fp32.  Costs are in k slices of a worker's MMAs.
struct Split {
  int64_t n, kb;  // splits, k slices of each
};
Split plan_split(int64_t B, int64_t d, int64_t V) {
  const bool pair = B > kBM;
  const int64_t workers = pair ? kPlanSms / 2 : kPlanSms;
  const int64_t tiles = ceil_div(B, pair ? 2 * kBM : kBM) * ceil_div(d, kBN);
  const int64_t n_kb = ceil_div(V, kBK);
  Split best = {1, n_kb};
  double best_cost = 1e300;
  for (int64_t want = 1; want <= 64 && want <= n_kb; ++want) {
    const int64_t kb = ceil_div(n_kb, want), n = ceil_div(n_kb, kb);
    const int64_t waves = ceil_div(tiles * n, workers);
    const double partial_mb = n > 1 ? double(n * tiles) * (pair ? 2 : 1) * 0.131 : 0.0;
    const double cost = double(waves * (kb + 8)) + partial_mb * 2.2;
    if (cost < best_cost) {
      best_cost = cost;
      best = {n, kb};
    }
  }
  return best;
}

// Columns of a result's store map (StoreEpi::Params::whole_n; unused below 8).
int64_t store_cols(int64_t d) { return d < 8 ? 8 : d & ~int64_t(7); }

size_t g_bytes(int64_t B, int64_t V) { return round256(size_t(B) * size_t((V + 7) / 8 * 8) * 2u); }
size_t partial_bytes(int64_t B, int64_t d, int64_t V) {
  const Split sp = plan_split(B, d, V);
  if (sp.n == 1) return 0;
  const int64_t ctas = B > kBM ? 2 : 1;
  return size_t(sp.n * ceil_div(B, kBM * ctas) * ceil_div(d, kBN) * ctas) * kBM * kBN * 4u;
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
    most = std::max(most, round256(entries * sizeof(RowPart)) + 2 * round256(entries * KC * 4u));
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
    default: return run_scores<24>(a, *dev, stream);
  }
}

namespace {
// Sizes whose units or partial tiles would overflow the kernels' 32-bit counts.
bool grad_sizes_ok(int64_t B, int64_t d, int64_t V) {
  return sizes_ok(B, d, V) && ceil_div(V, kBM) * ceil_div(d, kBN) <= INT_MAX &&
         ceil_div(V, kBN) * ceil_div(B, kBM) <= INT_MAX &&
         ceil_div(B, kBM) * ceil_div(d, kBN) * 64 <= INT_MAX;
}
}  // namespace

extern "C" size_t fs_logprobs_grad_workspace_size(int64_t B, int64_t d, int64_t V) {
  if (!grad_sizes_ok(B, d, V)) return 0;
  return g_bytes(B, V) + partial_bytes(B, d, V);
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
  const bool pair = B > kBM;
  const int ctas = pair ? 2 : 1;
  const int workers = pair ? dev.pairs : dev.sms;

  // G: the logits again, as in the forward pass.
  {
    const int box_rows = pair ? kBM : int(std::min<int64_t>(kBM, (B + 7) / 8 * 8));
    CUtensorMap mh, mw, mg;
    if (!encode(dev, &mh, a->H, d, B, a->ldh, box_rows) ||
        !encode(dev, &mw, a->W, d, V, a->ldw, pair ? kBN / 2 : kBN) ||
        !encode(dev, &mg, G, ldg, B, ldg, 32))  // its padding columns are written (as 0)
      return FS_ERR_INVALID_ARG;
    Shape s = {};
    s.n_mt = int32_t(ceil_div(B, kBM * ctas));
    s.n_nt = int32_t(ceil_div(V, kBN));
    s.n_units = s.n_mt * s.n_nt;
    s.n_kb = s.kb_per_split = int32_t(ceil_div(d, kBK));
    s.m_rows = int32_t(B);
    s.n_cols = int32_t(V);
    s.m_fastest = 1;
    s.a_box_rows = uint32_t(box_rows);
    s.policy_a = kPolicyLast;
    s.policy_b = kPolicyNormal;
    GradEpi::Params ep = {};
    ep.B = int32_t(B);
    ep.V = int32_t(V);
    ep.temperature = a->temperature;
    ep.mask = a->vocab_mask;
    ep.mask_ld = a->mask_ld;
    ep.tokens = a->tokens;
    ep.lse = a->lse;
    ep.entropy = a->entropy;
    ep.grad_logp = a->grad_logp;
    ep.grad_entropy = a->grad_entropy;
    ep.vocab_offset = a->vocab_offset;
    const int n = balanced(s.n_units, workers);
    st = pair ? launch<GradEpi, true, false, false>(dev, mh, mw, mg, s, ep, n, false, stream)
              : launch<GradEpi, false, false, false>(dev, mh, mw, mg, s, ep, n, false, stream);
    if (st != FS_OK) return st;
  }

  // dH = G W.
  if (a->out_dH) {
    const Split sp = plan_split(B, d, V);
    const int box_rows = pair ? kBM : int(std::min<int64_t>(kBM, (B + 7) / 8 * 8));
    CUtensorMap mg, mw, mo;
    if (!encode(dev, &mg, G, V, B, ldg, box_rows) || !encode(dev, &mw, a->W, d, V, a->ldw, kBK) ||
        !encode(dev, &mo, a->out_dH, store_cols(d), B, a->lddh, 32))
      return FS_ERR_INVALID_ARG;
    Shape s = {};
    s.n_mt = int32_t(ceil_div(B, kBM * ctas));
    s.n_nt = int32_t(ceil_div(d, kBN));
    s.n_units = int32_t(s.n_mt * s.n_nt * sp.n);
    s.n_kb = int32_t(ceil_div(V, kBK));
    s.kb_per_split = int32_t(sp.kb);
    s.m_rows = int32_t(B);
    s.n_cols = int32_t(d);
    s.m_fastest = 1;
    s.a_box_rows = uint32_t(box_rows);
    const int n = balanced(s.n_units, workers);
    if (sp.n == 1) {
      const StoreEpi::Params ep = {static_cast<__nv_bfloat16*>(a->out_dH), a->lddh,
                                   int32_t(d & ~int64_t(7))};
      st = pair ? launch<StoreEpi, true, false, true>(dev, mg, mw, mo, s, ep, n, false, stream)
                : launch<StoreEpi, false, false, true>(dev, mg, mw, mo, s, ep, n, false, stream);
      if (st != FS_OK) return st;
    } else {
      PartialEpi::Params ep = {};
      ep.partial = reinterpret_cast<float4*>(static_cast<uint8_t*>(G) + g_bytes(B, V));
      ep.ctas = ctas;
      st = pair ? launch<PartialEpi, true, false, true>(dev, mg, mw, mo, s, ep, n, false, stream)
                : launch<PartialEpi, false, false, true>(dev, mg, mw, mo, s, ep, n, false, stream);
      if (st != FS_OK) return st;
      const int64_t blocks = int64_t(s.n_mt) * s.n_nt * ctas * (kBM * kBN / 8 / kSumThreads);
      if (blocks > INT_MAX) return FS_ERR_INVALID_ARG;
      sum_splits_kernel<<<unsigned(blocks), kSumThreads, 0, stream>>>(
          ep.partial, int32_t(sp.n), s.n_mt * s.n_nt, s.n_nt, ctas, int32_t(B), int32_t(d),
          static_cast<__nv_bfloat16*>(a->out_dH), a->lddh);
      if (cudaGetLastError() != cudaSuccess) return FS_ERR_CUDA;
    }
  }

  // dW = G^T H: M is the vocabulary, so the units of one vocabulary block
  // (its slice of G) run over the columns of H next to one another.
  if (a->out_dW) {
    const bool wpair = V > kBM;
    CUtensorMap mg, mh, mo;
    if (!encode(dev, &mg, G, V, B, ldg, kBK) || !encode(dev, &mh, a->H, d, B, a->ldh, kBK) ||
        !encode(dev, &mo, a->out_dW, store_cols(d), V, a->lddw, 32))
      return FS_ERR_INVALID_ARG;
    Shape s = {};
    s.n_mt = int32_t(ceil_div(V, wpair ? 2 * kBM : kBM));
    s.n_nt = int32_t(ceil_div(d, kBN));
    s.n_units = s.n_mt * s.n_nt;
    s.n_kb = s.kb_per_split = int32_t(ceil_div(B, kBK));
    s.m_rows = int32_t(V);
    s.n_cols = int32_t(d);
    s.m_fastest = 0;
    s.a_box_rows = 0;
    s.policy_b = kPolicyLast;
    const StoreEpi::Params ep = {static_cast<__nv_bfloat16*>(a->out_dW), a->lddw,
                                 int32_t(d & ~int64_t(7))};
    const int n = balanced(s.n_units, wpair ? dev.pairs : dev.sms);
    st = wpair ? launch<StoreEpi, true, true, true>(dev, mg, mh, mo, s, ep, n, false, stream)
               : launch<StoreEpi, false, true, true>(dev, mg, mh, mo, s, ep, n, false, stream);
    if (st != FS_OK) return st;
  }
  return FS_OK;
}
