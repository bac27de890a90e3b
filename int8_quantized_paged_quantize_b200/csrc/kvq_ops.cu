// The cache write with rotary embedding (kvq_append_rope) and the dequantizing
// read-back (kvq_read): launchers of kvq_rope.cuh / kvq_append.cuh and
// kvq_read.cuh.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kvq_common.cuh"
#include "kvq_internal.h"
#include "kvq_rope.cuh"
#include "kvq_decode_mma.cuh"
#include "kvq_prefill.cuh"
#include "kvq_read.cuh"

namespace kvq {

namespace {
template <int D, int FMT>
cudaError_t rope_dispatch(const RopeArgs& a, const int64_t* slots, int32_t T, void* kc, void* vc,
                          void* ks, void* vs, const kvq_dims& d, int per_tensor, cudaStream_t st) {
  RopeRows<D> rows;
  rows.q = static_cast<const __nv_bfloat16*>(a.q);
  rows.k = static_cast<const __nv_bfloat16*>(a.k);
  rows.v = static_cast<const __nv_bfloat16*>(a.v);
  rows.qs = a.q_stride;
  rows.kst = a.k_stride;
  rows.vst = a.v_stride;
  rows.slots = slots;
  rows.positions = a.positions;
  rows.cos_sin = a.cos_sin;
  rows.q_out = static_cast<__nv_bfloat16*>(a.q_out);
  rows.Hq = a.q ? d.n_q_heads : 0;
  rows.max_pos = a.max_position;
  rows.rotary = a.rotary_dim;
  rows.interleaved = a.interleaved;
  const int qy = (rows.Hq + RopeRows<D>::kHeads - 1) / RopeRows<D>::kHeads;
  const dim3 grid(unsigned((int64_t(T) + kBlockSize - 1) / kBlockSize), unsigned(d.n_kv_heads + qy));
  append_kernel<D, FMT, RopeRows<D>><<<grid, 256, 0, st>>>(
      rows, T, d.n_kv_heads, d.num_blocks, static_cast<uint8_t*>(kc), static_cast<uint8_t*>(vc),
      static_cast<__nv_bfloat16*>(ks), static_cast<__nv_bfloat16*>(vs), per_tensor);
  return cudaGetLastError();
}

template <int D, int FMT, typename OutT>
cudaError_t read_dispatch(const ReadArgs& a, const kvq_dims& d, int per_tensor, cudaStream_t st) {
  const int64_t items = (int64_t(a.total) + kBlockSize - 1) / kBlockSize * d.n_kv_heads;
  const unsigned grid = unsigned((items + ReadCfg<D, FMT>::WARPS - 1) / ReadCfg<D, FMT>::WARPS);
  return launch_pdl(read_kernel<D, FMT, OutT>, dim3(grid), dim3(256), 0, st,
                    static_cast<const uint8_t*>(a.kc), static_cast<const uint8_t*>(a.vc),
                    static_cast<const __nv_bfloat16*>(a.ks), static_cast<const __nv_bfloat16*>(a.vs),
                    a.tables, a.starts, a.cu, int(a.n_seqs), int(a.total), int(d.n_kv_heads),
                    int(d.num_blocks), int(d.max_blocks_per_seq), per_tensor,
                    static_cast<OutT*>(a.k_out), static_cast<OutT*>(a.v_out));
}

template <int D, int FMT>
cudaError_t read_dispatch2(const ReadArgs& a, const kvq_dims& d, int per_tensor, cudaStream_t st) {
  return a.out_f32 ? read_dispatch<D, FMT, float>(a, d, per_tensor, st)
                   : read_dispatch<D, FMT, __nv_bfloat16>(a, d, per_tensor, st);
}
}  // namespace

int launch_append_rope(const RopeArgs& a, const int64_t* slots, int32_t T, void* kc, void* vc,
                       void* ks, void* vs, kvq_fmt fmt, const kvq_dims& d, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int pt = fmt == KVQ_INT8_TENSOR;
  cudaError_t e;
#define KVQ_ROPE(DD)                                                                              \
  switch (fmt) {                                                                                  \
    case KVQ_FP8_E4M3: e = rope_dispatch<DD, KVQ_FP8_E4M3>(a, slots, T, kc, vc, ks, vs, d, pt, st); break;   \
    case KVQ_FP8_E5M2: e = rope_dispatch<DD, KVQ_FP8_E5M2>(a, slots, T, kc, vc, ks, vs, d, pt, st); break;   \
    case KVQ_INT8_ASYM: e = rope_dispatch<DD, KVQ_INT8_ASYM>(a, slots, T, kc, vc, ks, vs, d, pt, st); break; \
    case KVQ_BF16: e = rope_dispatch<DD, KVQ_BF16>(a, slots, T, kc, vc, ks, vs, d, pt, st); break;           \
    default: e = rope_dispatch<DD, KVQ_INT8_CHANNEL>(a, slots, T, kc, vc, ks, vs, d, pt, st); break;         \
  }
  if (d.head_dim == 128) {
    KVQ_ROPE(128)
  } else {
    KVQ_ROPE(64)
  }
#undef KVQ_ROPE
  return int(e);
}

int launch_read(const ReadArgs& a, kvq_fmt fmt, const kvq_dims& d, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int pt = fmt == KVQ_INT8_TENSOR;
  cudaError_t e;
#define KVQ_READ(DD)                                                             \
  switch (fmt) {                                                                 \
    case KVQ_FP8_E4M3: e = read_dispatch2<DD, KVQ_FP8_E4M3>(a, d, pt, st); break;   \
    case KVQ_FP8_E5M2: e = read_dispatch2<DD, KVQ_FP8_E5M2>(a, d, pt, st); break;   \
    case KVQ_INT8_ASYM: e = read_dispatch2<DD, KVQ_INT8_ASYM>(a, d, pt, st); break; \
    case KVQ_BF16: e = read_dispatch2<DD, KVQ_BF16>(a, d, pt, st); break;           \
    case KVQ_KIVI2: e = read_dispatch2<DD, KVQ_KIVI2>(a, d, pt, st); break;         \
    case KVQ_KIVI4: e = read_dispatch2<DD, KVQ_KIVI4>(a, d, pt, st); break;         \
    default: e = read_dispatch2<DD, KVQ_INT8_CHANNEL>(a, d, pt, st); break;         \
  }
  if (d.head_dim == 128) {
    KVQ_READ(128)
  } else {
    KVQ_READ(64)
  }
#undef KVQ_READ
  return int(e);
}

int read_ops_error(uint32_t* flags, int clear) { return int(read_error_word(flags, clear)); }

}  // namespace kvq
