// CUDA kernels of libkvq for sm_100a: quantize-on-append, the launch of the
// paged GQA decode attention kernel (kvq_decode_mma.cuh, split-K partials) and
// the log-sum-exp merge.
//
// Sources (web pages, by title and section):
//  "KV cache quantization: what FP8/INT8 K and V really give, and their limits"
//     - "What KV cache quantization actually is": quantize only when storing,
//       scale from the full BF16 values, BF16 per-token scales, dequantization
//       fused into the attention kernel right before the matmuls.
//     - "Formats you will actually meet": E4M3 for K/V; INT8 per-token
//       asymmetric (scale, zero_point).
//  "Fitting 76x concurrent requests with an FP8 KV cache" - "4. Precision
//     loss?": 8-bit storage, FP32 accumulation of the attention dot products.
//  "KV Cache compression" - "5.1 Quantization pipeline" (a separate dequant
//     kernel gives the bandwidth gain back), "6.3" (quantize right after K/V
//     are computed).
//  "From FP8 KV cache to INT4 weight-only" - "Core concepts" 1) decode reads the
//     whole cache once per step and is memory bound; 2) PagedAttention.
//
// Numerics that must match the oracle bit for bit (codes and scales):
//  IEEE f32 division (__fdiv_rn), BF16 round-to-nearest-even of the scale,
//  hardware E4M3 conversion with round-to-nearest-even and saturation, rint
//  (ties to even) for INT8. This file is compiled without fast-math.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

#include <algorithm>
#include <utility>

#include "kvq_common.cuh"
#include "kvq_internal.h"
#include "kvq_append.cuh"
#include "kvq_decode_mma.cuh"
#include "kvq_decode_kivi.cuh"
#include "kvq_kivi.cuh"
#include "kvq_merge.cuh"
#include "kvq_prefill.cuh"

namespace kvq {

// ------------------------------------------------------------------ launchers
namespace {
constexpr float kLog2e = 1.4426950408889634f;

template <int D, int FMT>
cudaError_t append_dispatch(const void* k, const void* v, const int64_t* slots, int32_t T, void* kc,
                            void* vc, void* ks, void* vs, const kvq_dims& d, int per_tensor,
                            cudaStream_t st) {
  const dim3 grid(unsigned((int64_t(T) + kBlockSize - 1) / kBlockSize), unsigned(d.n_kv_heads));
  const PlainRows<D> rows{static_cast<const __nv_bfloat16*>(k), static_cast<const __nv_bfloat16*>(v),
                          slots};
  append_kernel<D, FMT, PlainRows<D>><<<grid, 256, 0, st>>>(
      rows, T, d.n_kv_heads, d.num_blocks, static_cast<uint8_t*>(kc), static_cast<uint8_t*>(vc),
      static_cast<__nv_bfloat16*>(ks), static_cast<__nv_bfloat16*>(vs), per_tensor);
  return cudaGetLastError();
}

template <int D, int G, int FMT>
cudaError_t decode_mma_dispatch3(const void* q, int32_t B, const void* kc, const void* vc,
                                 const void* ks, const void* vs, const int32_t* tables,
                                 const int32_t* ctx, int32_t max_ctx, float sm_scale,
                                 const DecodePlan& plan, void* ws, const kvq_dims& d,
                                 int per_tensor, int n_query, int nrg, cudaStream_t st) {
  using C = MmaCfg<D, G, FMT>;
  auto kern = decode_mma_kernel<D, G, FMT>;
  static OncePerContext once;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!once.done(dev)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout,
                             int(cudaSharedmemCarveoutMaxShared));
    if (e != cudaSuccess) return e;
    once.set(dev);
  }
  // resident CTAs per SM: shared memory bounds it (registers are capped so
  // that two 8-bit CTAs fit); the BF16 ring takes a whole SM
  int smem_sm = 0, reserved = 0;
  e = cudaDeviceGetAttribute(&smem_sm, cudaDevAttrMaxSharedMemoryPerMultiprocessor, dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&reserved, cudaDevAttrReservedSharedMemoryPerBlock, dev);
  if (e != cudaSuccess) return e;
  const int per_sm = std::max(1, std::min(FMT == KVQ_BF16 ? 1 : 2, smem_sm / (C::SMEM + reserved)));
  float* po = static_cast<float*>(ws);
  float* pml = reinterpret_cast<float*>(static_cast<char*>(ws) + plan.o_bytes);
  int32_t* pcnt = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + plan.o_bytes + plan.ml_bytes);
  // one CTA per resident slot, in groups of nrg (one CTA per row group) that
  // walk the same share of the tile list; at least one group
  const int64_t slots_resident = int64_t(device_sm_count()) * per_sm;
  const int64_t grid = std::max<int64_t>(1, slots_resident / nrg) * nrg;
  e = launch_pdl(kern, dim3(unsigned(grid)), dim3(192), C::SMEM, st,
      static_cast<const __nv_bfloat16*>(q), static_cast<const uint8_t*>(kc),
      static_cast<const uint8_t*>(vc), static_cast<const __nv_bfloat16*>(ks),
      static_cast<const __nv_bfloat16*>(vs), tables, ctx, B, d.n_kv_heads, nrg, d.num_blocks,
      d.max_blocks_per_seq, max_ctx, plan.partition / kTileTokens, plan.slots, sm_scale * kLog2e,
      per_tensor, n_query, decode_wait_limit(), po, pml, pcnt);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

template <int D, int FMT>
cudaError_t decode_dispatch2(int R, const void* q, int32_t B, const void* kc, const void* vc,
                             const void* ks, const void* vs, const int32_t* tables,
                             const int32_t* ctx, int32_t max_ctx, float sm_scale,
                             const DecodePlan& plan, void* ws, const kvq_dims& d, int per_tensor,
                             int n_query, cudaStream_t st) {
  // R query rows per KV head, taken in groups of gp rows (one instantiation per gp)
  int gp = 1;
  const int nrg = row_groups(R, &gp);
  switch (gp) {
    case 1: return decode_mma_dispatch3<D, 1, FMT>(q, B, kc, vc, ks, vs, tables, ctx, max_ctx, sm_scale, plan, ws, d, per_tensor, n_query, nrg, st);
    case 2: return decode_mma_dispatch3<D, 2, FMT>(q, B, kc, vc, ks, vs, tables, ctx, max_ctx, sm_scale, plan, ws, d, per_tensor, n_query, nrg, st);
    case 4: return decode_mma_dispatch3<D, 4, FMT>(q, B, kc, vc, ks, vs, tables, ctx, max_ctx, sm_scale, plan, ws, d, per_tensor, n_query, nrg, st);
    default: return decode_mma_dispatch3<D, 8, FMT>(q, B, kc, vc, ks, vs, tables, ctx, max_ctx, sm_scale, plan, ws, d, per_tensor, n_query, nrg, st);
  }
}

template <int D, int FMT>
cudaError_t prefill_dispatch2(const void* q, int32_t B, const void* kc, const void* vc,
                              const void* ks, const void* vs, const int32_t* tables,
                              const int32_t* ctx, int32_t max_ctx, float sm_scale,
                              const DecodePlan& plan, void* ws, const kvq_dims& d, int per_tensor,
                              int n_query, cudaStream_t st) {
  using C = PfCfg<D, FMT>;
  auto kern = prefill_mma_kernel<D, FMT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  const int G = d.n_q_heads / d.n_kv_heads;
  const int R = G * n_query;                         // query rows of a KV head
  const int nrb = (R + 127) / 128;                   // 128-row blocks, one CTA each
  float* po = static_cast<float*>(ws);
  float* pml = reinterpret_cast<float*>(static_cast<char*>(ws) + plan.o_bytes);
  int32_t* pcnt = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + plan.o_bytes + plan.ml_bytes);
  // one CTA per SM, in groups of nrb that walk the same share of the tile list
  const int64_t grid = std::max<int64_t>(1, int64_t(device_sm_count()) / nrb) * nrb;
  e = launch_pdl(kern, dim3(unsigned(grid)), dim3(448), C::SMEM, st,
      static_cast<const __nv_bfloat16*>(q), static_cast<const uint8_t*>(kc),
      static_cast<const uint8_t*>(vc), static_cast<const __nv_bfloat16*>(ks),
      static_cast<const __nv_bfloat16*>(vs), tables, ctx, B, d.n_kv_heads, G, n_query, nrb,
      d.num_blocks, d.max_blocks_per_seq, max_ctx, plan.partition / kTileTokens, plan.slots,
      sm_scale * kLog2e, per_tensor, decode_wait_limit(), po, pml, pcnt);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}
}  // namespace

int launch_prefill_partial(const void* q, int32_t B, const void* kc, const void* vc,
                           const void* ks, const void* vs, const int32_t* tables,
                           const int32_t* ctx, int32_t max_ctx, float sm_scale,
                           const DecodePlan& plan, void* ws, kvq_fmt fmt, const kvq_dims& d,
                           void* stream, int n_query) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  const int pt = fmt == KVQ_INT8_TENSOR;
#define KVQ_PF(DD, FF) prefill_dispatch2<DD, FF>(q, B, kc, vc, ks, vs, tables, ctx, max_ctx, sm_scale, plan, ws, d, pt, n_query, st)
  if (d.head_dim == 128) {
    if (fmt == KVQ_FP8_E4M3) e = KVQ_PF(128, KVQ_FP8_E4M3);
    else if (fmt == KVQ_FP8_E5M2) e = KVQ_PF(128, KVQ_FP8_E5M2);
    else if (fmt == KVQ_INT8_ASYM) e = KVQ_PF(128, KVQ_INT8_ASYM);
    else if (fmt_static(fmt)) e = KVQ_PF(128, KVQ_INT8_CHANNEL);
    else e = KVQ_PF(128, KVQ_BF16);
  } else {
    if (fmt == KVQ_FP8_E4M3) e = KVQ_PF(64, KVQ_FP8_E4M3);
    else if (fmt == KVQ_FP8_E5M2) e = KVQ_PF(64, KVQ_FP8_E5M2);
    else if (fmt == KVQ_INT8_ASYM) e = KVQ_PF(64, KVQ_INT8_ASYM);
    else if (fmt_static(fmt)) e = KVQ_PF(64, KVQ_INT8_CHANNEL);
    else e = KVQ_PF(64, KVQ_BF16);
  }
#undef KVQ_PF
  return int(e);
}

int launch_append(const void* k, const void* v, const int64_t* slots, int32_t T, void* kc,
                  void* vc, void* ks, void* vs, kvq_fmt fmt, const kvq_dims& d, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int pt = fmt == KVQ_INT8_TENSOR;
  cudaError_t e;
#define KVQ_APP(DD, FF) append_dispatch<DD, FF>(k, v, slots, T, kc, vc, ks, vs, d, pt, st)
  if (d.head_dim == 128) {
    if (fmt == KVQ_FP8_E4M3) e = KVQ_APP(128, KVQ_FP8_E4M3);
    else if (fmt == KVQ_FP8_E5M2) e = KVQ_APP(128, KVQ_FP8_E5M2);
    else if (fmt == KVQ_INT8_ASYM) e = KVQ_APP(128, KVQ_INT8_ASYM);
    else if (fmt_static(fmt)) e = KVQ_APP(128, KVQ_INT8_CHANNEL);
    else e = KVQ_APP(128, KVQ_BF16);
  } else {
    if (fmt == KVQ_FP8_E4M3) e = KVQ_APP(64, KVQ_FP8_E4M3);
    else if (fmt == KVQ_FP8_E5M2) e = KVQ_APP(64, KVQ_FP8_E5M2);
    else if (fmt == KVQ_INT8_ASYM) e = KVQ_APP(64, KVQ_INT8_ASYM);
    else if (fmt_static(fmt)) e = KVQ_APP(64, KVQ_INT8_CHANNEL);
    else e = KVQ_APP(64, KVQ_BF16);
  }
#undef KVQ_APP
  return int(e);
}

int launch_decode_partial(const void* q, int32_t B, const void* kc, const void* vc,
                          const void* ks, const void* vs, const int32_t* tables,
                          const int32_t* ctx, int32_t max_ctx, float sm_scale,
                          const DecodePlan& plan, void* ws, kvq_fmt fmt, const kvq_dims& d,
                          void* stream, int n_query) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int G = d.n_q_heads / d.n_kv_heads;
  cudaError_t e;
#define KVQ_DEC(DD, FF) decode_dispatch2<DD, FF>(G, q, B, kc, vc, ks, vs, tables, ctx, max_ctx, sm_scale, plan, ws, d, pt, n_query, st)
  const int pt = fmt == KVQ_INT8_TENSOR;
  if (d.head_dim == 128) {
    if (fmt == KVQ_FP8_E4M3) e = KVQ_DEC(128, KVQ_FP8_E4M3);
    else if (fmt == KVQ_FP8_E5M2) e = KVQ_DEC(128, KVQ_FP8_E5M2);
    else if (fmt == KVQ_INT8_ASYM) e = KVQ_DEC(128, KVQ_INT8_ASYM);
    else if (fmt_static(fmt)) e = KVQ_DEC(128, KVQ_INT8_CHANNEL);
    else e = KVQ_DEC(128, KVQ_BF16);
  } else {
    if (fmt == KVQ_FP8_E4M3) e = KVQ_DEC(64, KVQ_FP8_E4M3);
    else if (fmt == KVQ_FP8_E5M2) e = KVQ_DEC(64, KVQ_FP8_E5M2);
    else if (fmt == KVQ_INT8_ASYM) e = KVQ_DEC(64, KVQ_INT8_ASYM);
    else if (fmt_static(fmt)) e = KVQ_DEC(64, KVQ_INT8_CHANNEL);
    else e = KVQ_DEC(64, KVQ_BF16);
  }
#undef KVQ_DEC
  return int(e);
}

int launch_decode_merge(int32_t B, const int32_t* ctx, int32_t max_ctx, void* out, bool out_f32,
                        const void* ws, const DecodePlan& plan, const kvq_dims& d, void* stream,
                        int rows_per_count, const int32_t* dst_row) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const float* po = static_cast<const float*>(ws);
  const float* pml = reinterpret_cast<const float*>(static_cast<const char*>(ws) + plan.o_bytes);
  const int32_t* pcnt =
      reinterpret_cast<const int32_t*>(static_cast<const char*>(ws) + plan.o_bytes + plan.ml_bytes);
  const int rows = int(int64_t(B) * d.n_q_heads);
  const dim3 grid(unsigned((rows + 3) / 4));
  // G: query rows per row group, the unit part_cnt is kept for
  const int W = d.max_blocks_per_seq, Hq = d.n_q_heads;
  int G = rows_per_count;
  if (G <= 0) row_groups(d.n_q_heads / d.n_kv_heads, &G);
  cudaError_t e;
  if (d.head_dim == 128) {
    if (out_f32)
      e = launch_pdl(merge_kernel<128, float>, grid, dim3(128), 0, st, ctx, Hq, G, plan.slots,
                     max_ctx, W, po, pml, pcnt, static_cast<float*>(out), rows, dst_row);
    else
      e = launch_pdl(merge_kernel<128, __nv_bfloat16>, grid, dim3(128), 0, st, ctx, Hq, G,
                     plan.slots, max_ctx, W, po, pml, pcnt, static_cast<__nv_bfloat16*>(out), rows, dst_row);
  } else {
    if (out_f32)
      e = launch_pdl(merge_kernel<64, float>, grid, dim3(128), 0, st, ctx, Hq, G, plan.slots,
                     max_ctx, W, po, pml, pcnt, static_cast<float*>(out), rows, dst_row);
    else
      e = launch_pdl(merge_kernel<64, __nv_bfloat16>, grid, dim3(128), 0, st, ctx, Hq, G,
                     plan.slots, max_ctx, W, po, pml, pcnt, static_cast<__nv_bfloat16*>(out), rows, dst_row);
  }
  if (e != cudaSuccess) return int(e);
  return int(cudaGetLastError());
}

namespace {
template <int D, int G, int BITS>
cudaError_t kivi_dispatch3(const void* q, int32_t B, const void* kc, const void* vc, const void* km,
                           const void* vm, const int32_t* tables, const int32_t* lens,
                           int32_t max_len, float sm_scale, const DecodePlan& plan, void* ws,
                           const kvq_dims& d, cudaStream_t st) {
  using C = KiviCfg<D, G, BITS>;
  auto kern = decode_kivi_kernel<D, G, BITS>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout,
                           int(cudaSharedmemCarveoutMaxShared));
  if (e != cudaSuccess) return e;
  int dev = 0, smem_sm = 0, reserved = 0;
  e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&smem_sm, cudaDevAttrMaxSharedMemoryPerMultiprocessor, dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&reserved, cudaDevAttrReservedSharedMemoryPerBlock, dev);
  if (e != cudaSuccess) return e;
  const int per_sm = std::max(1, std::min(2, smem_sm / (C::SMEM + reserved)));
  float* po = static_cast<float*>(ws);
  float* pml = reinterpret_cast<float*>(static_cast<char*>(ws) + plan.o_bytes);
  int32_t* pcnt = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + plan.o_bytes + plan.ml_bytes);
  const int64_t grid = int64_t(device_sm_count()) * per_sm;
  kern<<<dim3(unsigned(grid)), 256, C::SMEM, st>>>(
      static_cast<const __nv_bfloat16*>(q), static_cast<const uint8_t*>(kc),
      static_cast<const uint8_t*>(vc), static_cast<const __nv_bfloat16*>(km),
      static_cast<const __nv_bfloat16*>(vm), tables, lens, B, d.n_kv_heads, d.num_blocks,
      d.max_blocks_per_seq, max_len, plan.partition / kTileTokens, plan.slots, sm_scale * kLog2e,
      decode_wait_limit(), po, pml, pcnt);
  return cudaGetLastError();
}

template <int D, int BITS>
cudaError_t kivi_dispatch2(int G, const void* q, int32_t B, const void* kc, const void* vc,
                           const void* km, const void* vm, const int32_t* tables,
                           const int32_t* lens, int32_t max_len, float sm_scale,
                           const DecodePlan& plan, void* ws, const kvq_dims& d, cudaStream_t st) {
  switch (G) {
    case 1: return kivi_dispatch3<D, 1, BITS>(q, B, kc, vc, km, vm, tables, lens, max_len, sm_scale, plan, ws, d, st);
    case 2: return kivi_dispatch3<D, 2, BITS>(q, B, kc, vc, km, vm, tables, lens, max_len, sm_scale, plan, ws, d, st);
    case 4: return kivi_dispatch3<D, 4, BITS>(q, B, kc, vc, km, vm, tables, lens, max_len, sm_scale, plan, ws, d, st);
    default: return kivi_dispatch3<D, 8, BITS>(q, B, kc, vc, km, vm, tables, lens, max_len, sm_scale, plan, ws, d, st);
  }
}
}  // namespace

int launch_kivi_decode(const void* q, int32_t B, const void* kc, const void* vc, const void* km,
                       const void* vm, const int32_t* tables, const int32_t* qlens,
                       int32_t max_qlen, const void* rk, const void* rv,
                       const int32_t* rtables, const int32_t* rlens, int32_t max_rlen,
                       float sm_scale, void* out, bool out_f32, void* ws, const DecodePlan& pa,
                       const DecodePlan& pb, int bits, const kvq_dims& d, const kvq_dims& rd,
                       void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int G = d.n_q_heads / d.n_kv_heads;
  void* ws_b = static_cast<char*>(ws) + pa.total;
  cudaError_t e;
  // the quantized groups
  if (d.head_dim == 128)
    e = bits == 2 ? kivi_dispatch2<128, 2>(G, q, B, kc, vc, km, vm, tables, qlens, max_qlen, sm_scale, pa, ws, d, st)
                  : kivi_dispatch2<128, 4>(G, q, B, kc, vc, km, vm, tables, qlens, max_qlen, sm_scale, pa, ws, d, st);
  else
    e = bits == 2 ? kivi_dispatch2<64, 2>(G, q, B, kc, vc, km, vm, tables, qlens, max_qlen, sm_scale, pa, ws, d, st)
                  : kivi_dispatch2<64, 4>(G, q, B, kc, vc, km, vm, tables, qlens, max_qlen, sm_scale, pa, ws, d, st);
  if (e != cudaSuccess) return int(e);
  // the residual tokens and the merge, one CTA per (sequence, KV head),
  // launched as a programmatic dependent of the groups kernel
  (void)pb;
  const float* poa = static_cast<const float*>(ws);
  const float* pmla = reinterpret_cast<const float*>(static_cast<const char*>(ws) + pa.o_bytes);
  const int32_t* pca = reinterpret_cast<const int32_t*>(static_cast<const char*>(ws) + pa.o_bytes + pa.ml_bytes);
  const dim3 grid(unsigned(int64_t(B) * d.n_kv_heads));
  const float qk = sm_scale * kLog2e;
  auto go = [&](auto kern, auto* o) {
    return launch_pdl(kern, grid, dim3(128), 0, st, static_cast<const __nv_bfloat16*>(q), d.n_kv_heads,
                      qlens, pa.slots, max_qlen, d.max_blocks_per_seq, poa, pmla, pca,
                      static_cast<const __nv_bfloat16*>(rk), static_cast<const __nv_bfloat16*>(rv), rtables,
                      rlens, rd.num_blocks, rd.max_blocks_per_seq, max_rlen, qk, o);
  };
#define KVQ_RM(DD, GG)                                                                        \
  e = out_f32 ? go(kivi_residual_merge_kernel<DD, GG, float>, static_cast<float*>(out))       \
              : go(kivi_residual_merge_kernel<DD, GG, __nv_bfloat16>, static_cast<__nv_bfloat16*>(out))
#define KVQ_RM_G(DD)        \
  switch (G) {              \
    case 1: KVQ_RM(DD, 1); break; \
    case 2: KVQ_RM(DD, 2); break; \
    case 4: KVQ_RM(DD, 4); break; \
    default: KVQ_RM(DD, 8); break; \
  }
  if (d.head_dim == 128) {
    KVQ_RM_G(128)
  } else {
    KVQ_RM_G(64)
  }
#undef KVQ_RM_G
#undef KVQ_RM
  if (e != cudaSuccess) return int(e);
  return int(cudaGetLastError());
}

int read_kernels_error(uint32_t* flags, int clear) { return int(read_error_word(flags, clear)); }

}  // namespace kvq
