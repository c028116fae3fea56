// Waits that run out: verification's draw behind a barrier that nothing arrives on, over sums
// that nobody wrote; probabilities whose CTAs have half their warps, so that the other half's
// words never come (every access stays in its buffers, every wait ends).
#include "fs_verify.cu"

namespace test_of_waits {
__device__ int g_word = 0;

__global__ void __launch_bounds__(fs::verify::kThreads)
    stale_draw_kernel(const fs::verify::VerifyParams a, int mode, int* out) {
  using namespace fs::verify;
  __shared__ Shared sm;
  if (threadIdx.x == 0) {
    fs::ptx::mbar_init(&sm.arrived, 1);
    fs::ptx::fence_barrier_init();
    fs::ptx::mbar_arrive_expect_tx(&sm.arrived, uint32_t(a.n_segments) * 8u);  // none come
  }
  // What shared memory may hold: pairs whose sum is above 0 without any first part that is.
  for (int s = threadIdx.x; s < a.n_segments; s += kThreads)
    sm.sums[s].hi = s % 3 ? -5.0f : 0.0f, sm.sums[s].lo = s % 2 ? 10.0f : 3.0f;
  __syncthreads();
  if (threadIdx.x < 32) {  // even a search finds no segment that there is none of
    sm.segment = 0;
    find_segment(a, 0.5f, sm, int(threadIdx.x));
    if (threadIdx.x == 0) out[2] = sm.segment;
  }
  __syncthreads();
  Weights<float> w;
  w.p = static_cast<const float*>(a.p);
  w.q = static_cast<const float*>(a.q);
  w.mode = mode;
  w.without = 0;
  const int drawn = draw(a, w, 0.5f, true, sm);
  if (threadIdx.x == 0) {
    out[0] = drawn;
    out[1] = sm.gave_up;
    bool kept = true;
    for (int s = 0; s < a.n_segments; ++s)
      kept = kept && sm.sums[s].hi == (s % 3 ? -5.0f : 0.0f) && sm.sums[s].lo == (s % 2 ? 10.0f : 3.0f);
    out[3] = kept;
  }
}
}  // namespace test_of_waits

namespace fs {
int* device_error_word() { return nullptr; }  // this file's calls go to the kernel above only
}  // namespace fs

// out (device): the drawn id, whether the wait ran out, the segment of a search, whether the
// sums were left alone.  Returns the error word, or -1.
extern "C" int stale_draw(const float* p, const float* q, int V, int mode, uint64_t limit_ns,
                          int* out, void* stream) {
  fs::verify::VerifyParams a = {};
  a.p = p;
  a.q = q;
  a.V = V;
  a.segment = fs::verify::kSegment;
  a.n_segments = (V + a.segment - 1) / a.segment;
  if (a.n_segments > fs::verify::kMaxSegments || limit_ns > 1000000000ull) return -1;
  a.wait_limit_ns = limit_ns;
  int word = 0;
  void* at = nullptr;
  if (cudaGetSymbolAddress(&at, test_of_waits::g_word) != cudaSuccess) return -1;
  a.error_word = static_cast<int*>(at);
  test_of_waits::stale_draw_kernel<<<1, fs::verify::kThreads, 0, static_cast<cudaStream_t>(stream)>>>(a, mode, out);
  if (cudaGetLastError() != cudaSuccess ||
      cudaMemcpyFromSymbol(&word, test_of_waits::g_word, sizeof(int)) != cudaSuccess)
    return -1;
  return word;
}

// N rows of 8000 logits, more than one row to a cluster of two CTAs.  Returns the error word, or -1.
extern "C" int half_probs(const float* logits, float* out, int N, int clusters, uint64_t limit_ns,
                          void* stream) {
  using namespace fs::verify;
  if (limit_ns > 1000000000ull || N < 1 || clusters < 1 || clusters > N) return -1;
  int word = 0;
  void* at = nullptr;
  if (cudaGetSymbolAddress(&at, test_of_waits::g_word) != cudaSuccess ||
      cudaMemcpyToSymbol(test_of_waits::g_word, &word, sizeof(int)) != cudaSuccess)
    return -1;
  ProbsParams p = {};
  p.logits = logits;
  p.out = out;
  p.ldl = p.ldo = p.V = 8000;
  p.N = N;
  p.part = 4000;
  p.wait_limit_ns = limit_ns;
  p.error_word = static_cast<int*>(at);
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 2;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(2 * clusters));
  cfg.blockDim = dim3(kProbThreads / 2);
  cfg.dynamicSmemBytes = 2 * 4 * kProbThreads * sizeof(float);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, probs_kernel<float, float, true, 2>, p) != cudaSuccess ||
      cudaMemcpyFromSymbol(&word, test_of_waits::g_word, sizeof(int)) != cudaSuccess)
    return -1;
  return word;
}
