// Internal declarations of the low-rank adapters and of the routers' balance loss:
// argument structs shared by the C entry points (mx_api.cu) and the kernel files.
#pragma once

#include <atomic>

#include "mx_internal.cuh"

namespace imc {
namespace mx {

constexpr int kMaxRank = 128;

constexpr int kBlockSharedMemory = 232448;  // bytes that a block may take, static ones included

// Launches Kernel in clusters of `ctas` blocks (1: none) as the programmatic dependent of
// the stream's previous kernel.  What the kernel may take of shared memory is set once per
// device (0.5 us a call), to the most there is: the same value whichever call comes first, so
// that host threads may make first calls of different sizes at once.
template <auto Kernel, typename... Args>
cudaError_t launch_clusters(dim3 grid, int ctas, int threads, size_t smem, cudaStream_t s, Args... args) {
  static std::atomic<bool> ready[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !ready[dev].load(std::memory_order_acquire)) {
    cudaFuncAttributes own;
    e = cudaFuncGetAttributes(&own, Kernel);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               kBlockSharedMemory - (int)own.sharedSizeBytes);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready[dev].store(true, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ctas > 1 ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, Kernel, args...);
  note_launch();
  return e;
}

// Rows of x in adapter order: bucket l of `offsets` [L + 2] holds the places in
// `order` of adapter l's rows, bucket L those of the rows without an adapter
// (the layout of moe_layout with one choice per row).
struct AdapterArgs {
  const void* x;        // [T, K], rows ld elements apart
  int64_t ld;
  const void *a, *b;    // [L, r, K], [L, N, r]
  const float* scale;   // [L] or null: ones
  const int32_t *offsets, *order;
  const void* base;     // [T, N] or null: zeros
  void* out;            // [T, N]; may be base
  int64_t T, K, N;
  int L, r;
  void* workspace;      // adapters_bytes
};
size_t adapters_bytes(int64_t T, int64_t L, int64_t r);
cudaError_t launch_adapters(const AdapterArgs& a, int dtype, cudaStream_t s);

struct AdapterGradArgs {
  const void *grad, *x;  // [T, N], [T, K]
  const void *a, *b;
  const float* scale;
  const int32_t *offsets, *order;
  const void* base;      // [T, K] or null: zeros
  void *grad_x, *grad_a, *grad_b;  // each may be null
  int64_t T, K, N;
  int L, r;
  void* workspace;       // adapters_backward_bytes
};
size_t adapters_backward_bytes(int64_t T, int64_t r);
cudaError_t launch_adapters_backward(const AdapterGradArgs& a, int dtype, cudaStream_t s);

struct BalanceArgs {
  const void* logits;    // [T, E], rows ld elements apart
  int64_t T, ld;
  int E, k, S, sigmoid;
  const int32_t* experts;  // [T, k]
  const int32_t* offsets;  // [S + 1] or null: one sequence of all tokens
  float* loss;             // [S]
  int32_t* counts;         // [S, E]
  // backward
  const float* grad_loss;     // [S]
  const float* grad_weights;  // [T, k] or null
  int renorm;
  float scale;
  void* grad;              // [T, E]
  void* workspace;         // balance_bytes
};
size_t balance_bytes(int64_t T, int64_t S, int64_t E);
cudaError_t launch_balance(const BalanceArgs& a, int dtype, cudaStream_t s);
cudaError_t launch_balance_backward(const BalanceArgs& a, int dtype, cudaStream_t s);

}  // namespace mx
}  // namespace imc
