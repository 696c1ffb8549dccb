// Gated linear scan: the decoding step and the states of sequences without tokens.
//
// The step is one token of every sequence: x, decay, gate and the float32 state are read once, y
// and the state written once, one element (or two) per thread: 8 sequences of 2048 channels 2.8 us, which is a
// launch's own time; 4096 of 2048 float32 30 us (5.6 TB/s; one channel per thread 36).
#include "dynconv_internal.hpp"
#include "dynconv_scan_kernels.hpp"

namespace dynconv {

namespace {

constexpr int kStepThreads = 256;

template <typename ET, int V>
__global__ __launch_bounds__(kStepThreads) void k_scan_step(const ScanStepParams p) {
  typedef scan::Elems<ET, V> E;
  const uint32_t per = uint32_t(p.D) / V;  // whole lanes of a row
  const uint64_t i = (uint64_t(blockIdx.y) * gridDim.x + blockIdx.x) * kStepThreads + threadIdx.x;
  const uint64_t b = i / per;
  if (b >= uint64_t(p.B)) return;
  const uint32_t c = uint32_t(i - b * per) * V;
  auto at = [&](const void* t, int64_t s) {
    return *reinterpret_cast<const typename E::W*>(static_cast<const char*>(t) + (int64_t(b) * s + c) * int64_t(sizeof(ET)));
  };
  float x[V], r[V], g[V], y[V];
  float* st = p.state + int64_t(b) * p.sts + c;
  E::get(at(p.x, p.xs), x);
  E::get(at(p.decay, p.as), r);
  if (p.gate != nullptr) E::get(at(p.gate, p.gs), g);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const scan::Decay d = scan::decay_of(scan::sigmoid(r[v]), p.rate[c + v] * scan::kLog2e);
    y[v] = __builtin_fmaf(d.a, st[v], d.b * (p.gate != nullptr ? scan::sigmoid(g[v]) : 1.f) * x[v]);
  }
#pragma unroll
  for (int v = 0; v < V; ++v) st[v] = y[v];
  *reinterpret_cast<typename E::W*>(static_cast<char*>(p.y) + (int64_t(b) * p.ys + c) * int64_t(sizeof(ET))) = E::put(y);
}

__global__ __launch_bounds__(kStepThreads) void k_scan_copy_state(const float* src, int64_t ss, float* dst, int64_t ds,
                                                                   int32_t B, int32_t D) {
  const uint64_t i = (uint64_t(blockIdx.y) * gridDim.x + blockIdx.x) * kStepThreads + threadIdx.x;
  const uint64_t b = i / uint32_t(D);
  if (b >= uint64_t(B)) return;
  const uint32_t c = uint32_t(i - b * uint32_t(D));
  dst[int64_t(b) * ds + c] = src != nullptr ? src[int64_t(b) * ss + c] : 0.f;
}

dim3 grid_for(int64_t threads) {
  constexpr int64_t most = int64_t(1) << 23;  // a dimension of a launch has fewer than 2^32 threads
  const int64_t blocks = (threads + kStepThreads - 1) / kStepThreads;
  return dim3(unsigned(blocks < most ? blocks : most), unsigned((blocks + most - 1) / most));
}

template <typename ET>
void launch_step(const ScanStepParams& p, int vec, hipStream_t s) {
  const dim3 grid = grid_for(int64_t(p.B) * (p.D / vec));
  if (vec == 2) {
    hipLaunchKernelGGL((k_scan_step<ET, 2>), grid, dim3(kStepThreads), 0, s, p);
  } else {
    hipLaunchKernelGGL((k_scan_step<ET, 1>), grid, dim3(kStepThreads), 0, s, p);
  }
}

}  // namespace

hipError_t scan_step(const ScanStepParams& p, dynconv_dtype dt, int vec, hipStream_t s) {
  if (dt == DYNCONV_BF16) {
    launch_step<bf16_t>(p, vec, s);
  } else if (dt == DYNCONV_F16) {
    launch_step<f16_t>(p, vec, s);
  } else {
    launch_step<float>(p, vec, s);
  }
  return hipGetLastError();
}

hipError_t scan_copy_state(const float* src, int64_t ss, float* dst, int64_t ds, int32_t B, int32_t D, hipStream_t s) {
  hipLaunchKernelGGL(k_scan_copy_state, grid_for(int64_t(B) * D), dim3(kStepThreads), 0, s, src, ss, dst, ds, B, D);
  return hipGetLastError();
}

}  // namespace dynconv
