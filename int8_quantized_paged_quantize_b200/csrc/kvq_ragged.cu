// Attention of ragged chunks of new tokens over the paged cache
// (kvq_ragged_attn): launchers of kvq_ragged.cuh.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <climits>
#include <cstdint>
#include <type_traits>

#include "kvq_common.cuh"
#include "kvq_internal.h"
#include "kvq_quant.cuh"
#include "kvq_decode_mma.cuh"
#include "kvq_prefill.cuh"
#include "kvq_ragged.cuh"

namespace kvq {

namespace {
constexpr float kLog2e = 1.4426950408889634f;
size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

// Workspace pieces: two places per CTA of `rows` rows each.
struct RgSpace {
  int rows;
  size_t o, ml, total;
};
RgSpace rg_space(int32_t total_q, const kvq_dims& d) {
  RgSpace w;
  const int G = d.n_q_heads / d.n_kv_heads;
  w.rows = int(std::min<int64_t>(256, int64_t(total_q) * G));
  const size_t places = 2 * size_t(device_sm_count());
  w.o = round256(places * w.rows * d.head_dim * sizeof(float));
  w.ml = round256(places * w.rows * 2 * sizeof(float));
  w.total = w.o + w.ml + round256(places * sizeof(RgPiece));
  return w;
}

// Shared-memory limit of the kernel, and the check that its registers are those
// that it shares out anew. Both cost as much as a launch, so they are done once
// per context (a new one, after a reset, has another id).
template <int D, int FMT, bool HP>
cudaError_t prepare() {
  auto kern = ragged_mma_kernel<D, FMT, HP>;
  static std::atomic<unsigned long long> done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long id = context_id();
  if (id != 0 && dev < 64 && done[dev].load(std::memory_order_acquire) == id) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, RgCfg<D, FMT, HP>::SMEM);
  if (e != cudaSuccess) return e;
  cudaFuncAttributes fa;
  e = cudaFuncGetAttributes(&fa, kern);
  if (e != cudaSuccess) return e;
  if (fa.numRegs != kRgRegs) return cudaErrorInvalidConfiguration;
  if (id != 0 && dev < 64) done[dev].store(id, std::memory_order_release);
  return cudaSuccess;
}

template <int D, int FMT, bool HP>
cudaError_t ragged_dispatch(const RaggedArgs& a, const kvq_dims& d, int per_tensor, cudaStream_t st) {
  using C = RgCfg<D, FMT, HP>;
  using OutT = typename std::conditional<HP, float, __nv_bfloat16>::type;
  auto kern = ragged_mma_kernel<D, FMT, HP>;
  cudaError_t e = prepare<D, FMT, HP>();
  if (e != cudaSuccess) return e;
  const int G = d.n_q_heads / d.n_kv_heads;
  const RgSpace w = rg_space(a.total_q, d);
  char* ws = static_cast<char*>(a.workspace);
  float* po = reinterpret_cast<float*>(ws);
  float* pml = reinterpret_cast<float*>(ws + w.o);
  RgPiece* pieces = reinterpret_cast<RgPiece*>(ws + w.o + w.ml);
  RgBatch b;
  b.cu = a.cu_q;
  b.ctx_lens = a.ctx;
  b.B = a.n_seqs;
  b.T = a.total_q;
  b.Hk = d.n_kv_heads;
  b.W = d.max_blocks_per_seq;
  b.max_ctx = a.max_ctx;
  b.p.g_log = G == 8 ? 3 : G == 4 ? 2 : G == 2 ? 1 : 0;
  b.p.pos_log = (C::RPB == 256 ? 8 : 7) - b.p.g_log;
  b.p.window = a.window;
  const int grid = device_sm_count();                    // one CTA per SM
  e = launch_pdl(kern, dim3(unsigned(grid)), dim3(kRgThreads), C::SMEM, st,
                 static_cast<const __nv_bfloat16*>(a.q), a.q_stride, static_cast<const uint8_t*>(a.kc),
                 static_cast<const uint8_t*>(a.vc), static_cast<const __nv_bfloat16*>(a.ks),
                 static_cast<const __nv_bfloat16*>(a.vs), a.tables, b, int(d.num_blocks),
                 a.sm_scale * kLog2e, per_tensor, decode_wait_limit(), a.out, po, pml, pieces, w.rows);
  if (e != cudaSuccess) return e;
  e = launch_pdl(ragged_merge_kernel<D, OutT>, dim3(unsigned(grid), unsigned((std::min(w.rows, C::RPB) + 31) / 32)),
                 dim3(256), 0, st, static_cast<const float*>(po), static_cast<const float*>(pml),
                 static_cast<const RgPiece*>(pieces), grid, w.rows, b.p, int(d.n_q_heads),
                 static_cast<OutT*>(a.out));
  return e;
}
}  // namespace

size_t ragged_workspace(int32_t total_q, const kvq_dims& d) { return rg_space(total_q, d).total; }

int launch_ragged(const RaggedArgs& a, kvq_fmt fmt, const kvq_dims& d, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int pt = fmt == KVQ_INT8_TENSOR;
  cudaError_t e;
#define KVQ_RG(DD, FF) \
  e = a.out_f32 ? ragged_dispatch<DD, FF, true>(a, d, pt, st) : ragged_dispatch<DD, FF, false>(a, d, pt, st)
#define KVQ_RG_D(DD)                                       \
  switch (fmt) {                                           \
    case KVQ_FP8_E4M3: KVQ_RG(DD, KVQ_FP8_E4M3); break;    \
    case KVQ_FP8_E5M2: KVQ_RG(DD, KVQ_FP8_E5M2); break;    \
    case KVQ_INT8_ASYM: KVQ_RG(DD, KVQ_INT8_ASYM); break;  \
    case KVQ_BF16: KVQ_RG(DD, KVQ_BF16); break;            \
    default: KVQ_RG(DD, KVQ_INT8_CHANNEL); break;          \
  }
  if (d.head_dim == 128) {
    KVQ_RG_D(128)
  } else {
    KVQ_RG_D(64)
  }
#undef KVQ_RG_D
#undef KVQ_RG
  return int(e);
}

int read_ragged_error(uint32_t* flags, int clear) { return int(read_error_word(flags, clear)); }

}  // namespace kvq
