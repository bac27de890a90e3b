// Device helpers and launch code shared by the translation units of libkvq.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <utility>

#include "kvq_internal.h"

namespace kvq {

// Per-device error word (KVQ_DEVERR_* bits): one for each translation unit with
// kernels; kvq_device_error() reads them all.
static __device__ unsigned int g_error_word;

__device__ __forceinline__ void flag_error(unsigned int bit) { atomicOr(&g_error_word, bit); }

// ------------------------------------------------------------------ helpers
// Byte offset, inside a K page whose token rows are ROWB bytes, of 16-byte
// chunk c of token t: tokens come in two groups of 8, and a group stores its
// chunk 0 for tokens 0..7, then chunk 1, ... (8 x 16-byte core matrices, the
// K-major operand layout of the tensor cores).
template <int ROWB>
__host__ __device__ __forceinline__ int k_chunk_offset(int c, int t) {
  return (t >> 3) * (8 * ROWB) + c * 128 + (t & 7) * 16;
}

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Reads this translation unit's error word on the current device (after the
// device has been synchronized) into *flags, clearing it on request.
static inline cudaError_t read_error_word(uint32_t* flags, int clear) {
  unsigned int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_error_word, sizeof(v));
  if (e != cudaSuccess) return e;
  *flags = v;
  if (clear && v) {
    const unsigned int zero = 0;
    e = cudaMemcpyToSymbol(g_error_word, &zero, sizeof(zero));
  }
  return e;
}

// What is set up once per context (a new one, after a device reset, has another
// id): the attributes of a kernel, which cost as much as a launch to set.
class OncePerContext {
 public:
  bool done(int dev) const {
    const unsigned long long id = context_id();
    return id != 0 && dev < 64 && ids_[dev].load(std::memory_order_acquire) == id;
  }
  void set(int dev) {
    const unsigned long long id = context_id();
    if (id != 0 && dev < 64) ids_[dev].store(id, std::memory_order_release);
  }

 private:
  std::atomic<unsigned long long> ids_[64] = {};
};

// Launch as the programmatic dependent of the kernel ahead on the stream: it
// may start (and run up to its grid_dep_wait) before that kernel finishes.
template <typename... KArgs, typename... Args>
static inline cudaError_t launch_pdl(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                       Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

}  // namespace kvq
