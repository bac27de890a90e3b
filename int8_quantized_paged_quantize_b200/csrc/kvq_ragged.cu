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

// Single new tokens, in a call without a window, can go through the decode kernels, which
// multiply the codes as they are stored: the ragged kernel's converters and producer take
// some 2,000 cycles a step of 64 tokens however few rows there are. The lengths are on the
// device, so the choice is by the call's shape; the ragged kernel always runs, leaves the
// single tokens out and hands their rows on.
//   total_q = n_seqs, a decode step: always (32/8 heads; 64 sequences of 1,024 to 8,192
//     tokens: FP8 108 against 304 us, INT8 107 / 359, BF16 194 / 244; 8 of up to 256, FP8:
//     16 / 25; 1 of 100: 15 / 22; 257 of 1,500: 146 / 454, 1,024 of 50 to 1,500: 373 / 1,294);
//   total_q > n_seqs, single tokens perhaps beside chunks: 8-bit caches from kRtWork
//     (sequence, KV head, token)s on. FP8, 63 single tokens and a chunk of 512 at up to
//     8,000 tokens: 179 / 347 us, 15 and 450 at up to 4,096: 58 / 73, 3 and 500 at 12,000: 198
//     / 226. Where no sequence has one token, two launches find nothing to do: 8 chunks of 200
//     200 / 201, 4 of 1,000 596 / 596, 16 of 30 91 / 80; the lengths are on the device, so that
//     the shape of the last call is that of 15 and 450. BF16: 277 / 277, 63 / 62, 171 / 170:
//     not worth it.
// Not with FP32 output over 8-bit caches: their weights have 18 bits (FP8), or 24 below the
// largest one (INT8: tokens 12 nats below a dominant one came out 1e-2 off), the ragged
// kernel's 24 of their own (64 of 1,024 to 8,192 tokens, INT8: 393 us). Nor with contexts
// above kRtLong for each (sequence, KV head), of which the decode kernels' at most 15 splits
// leave SMs idle (1 of 60,000 tokens, 1 KV head: 56 / 50 us).
// At most kRtSeqs sequences: the workspace has kRtRows partials a head, two a sequence then.
constexpr int kRtSeqs = 1024, kRtSlots = 16, kRtRows = 2048;
constexpr int64_t kRtLong = 32768, kRtWork = 1 << 18;

// The decode kernels' plan: at most kRtSlots partials a row (the automatic plan's
// number), and kRtRows of them over all sequences. max_ctx is what the caller allows, in a
// captured graph the model's maximum, so it sizes the slots only: partition 0 lets the
// kernel size its shares by the longest sequence of the batch. Contexts of 2,000 tokens, FP8,
// 32/8 heads, max_ctx exact / 131,072: 1 sequence 15 / 15 us, 8 20 / 20, 64 57 / 57 (shares
// sized by max_ctx: 15 / 164, 19 / 94, 56 / 96).
int rt_plan(int32_t n, int32_t max_ctx, const kvq_dims& d, DecodePlan* plan) {
  const int32_t tiles = std::max(1, (max_ctx + kTileTokens - 1) / kTileTokens);
  const int32_t splits = std::min(kRtSlots, kRtRows / n) - 1;
  const int rc = make_plan(n, max_ctx, kTileTokens * ((tiles + splits - 1) / splits), &d, plan);
  plan->partition = 0;
  return rc;
}
// Its workspace for up to n sequences (not falling with n).
size_t rt_bytes(int32_t n, const kvq_dims& d) {
  const size_t rows = size_t(std::min(n * kRtSlots, kRtRows)) * d.n_q_heads;
  return round256(rows * d.head_dim * sizeof(float)) + round256(rows * 2 * sizeof(float)) +
         round256(size_t(n) * d.n_q_heads * sizeof(int32_t));
}

// Workspace pieces: two places per CTA of `rows` rows each; the sums of its two slots; for a
// decode step each sequence's context and output row, its query and the decode kernels' workspace.
struct RgSpace {
  int rows;
  size_t o, ml, pieces, sums, seqs, q1, total;
};
RgSpace rg_space(int32_t total_q, const kvq_dims& d) {
  RgSpace w;
  const int G = d.n_q_heads / d.n_kv_heads;
  w.rows = int(std::min<int64_t>(256, int64_t(total_q) * G));
  const size_t places = 2 * size_t(device_sm_count());
  w.o = round256(places * w.rows * d.head_dim * sizeof(float));
  w.ml = round256(places * w.rows * 2 * sizeof(float));
  w.pieces = round256(places * sizeof(RgPiece));
  w.sums = round256(places * 128 * d.head_dim * sizeof(float));
  w.total = w.o + w.ml + w.pieces + w.sums;
  const int32_t n = total_q < 256 ? total_q : kRtSeqs;   // from 256 tokens on, the largest size
  w.seqs = round256(size_t(n) * sizeof(int32_t));
  w.q1 = round256(size_t(n) * d.n_q_heads * d.head_dim * 2);
  w.total += 2 * w.seqs + w.q1 + rt_bytes(n, d);
  return w;
}

// Shared-memory limit of the kernel, and the check that its registers are those
// that it shares out anew.
template <int D, int FMT, bool HP>
cudaError_t prepare() {
  auto kern = ragged_mma_kernel<D, FMT, HP>;
  static OncePerContext once;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (once.done(dev)) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, RgCfg<D, FMT, HP>::SMEM);
  if (e != cudaSuccess) return e;
  cudaFuncAttributes fa;
  e = cudaFuncGetAttributes(&fa, kern);
  if (e != cudaSuccess) return e;
  if (fa.numRegs != kRgRegs) return cudaErrorInvalidConfiguration;
  once.set(dev);
  return cudaSuccess;
}

template <int D, int FMT, bool HP>
cudaError_t ragged_dispatch(const RaggedArgs& a, kvq_fmt fmt, const kvq_dims& d, int per_tensor, cudaStream_t st) {
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
  b.ctx1 = b.row1 = nullptr;
  b.q1 = nullptr;
  DecodePlan plan;
  const bool step = !(HP && !C::BF) && a.window == 0 && a.n_seqs <= kRtSeqs &&
                    (a.total_q == a.n_seqs || (!C::BF && a.total_q > a.n_seqs && int64_t(a.n_seqs) * d.n_kv_heads * a.max_ctx >= kRtWork)) &&
                    a.max_ctx <= kRtLong * a.n_seqs * d.n_kv_heads && rt_plan(a.n_seqs, a.max_ctx, d, &plan) == KVQ_OK &&
                    plan.total <= rt_bytes(a.n_seqs, d);
  float* sums = reinterpret_cast<float*>(ws + w.o + w.ml + w.pieces);
  char* at = ws + w.o + w.ml + w.pieces + w.sums;
  if (step) {
    b.ctx1 = reinterpret_cast<int32_t*>(at);
    b.row1 = reinterpret_cast<int32_t*>(at + w.seqs);
    b.q1 = reinterpret_cast<uint4*>(at + 2 * w.seqs);
  }
  const int grid = device_sm_count();                    // one CTA per SM
  e = launch_pdl(kern, dim3(unsigned(grid)), dim3(kRgThreads), C::SMEM, st,
                 static_cast<const __nv_bfloat16*>(a.q), a.q_stride, static_cast<const uint8_t*>(a.kc),
                 static_cast<const uint8_t*>(a.vc), static_cast<const __nv_bfloat16*>(a.ks),
                 static_cast<const __nv_bfloat16*>(a.vs), a.tables, b, int(d.num_blocks),
                 a.sm_scale * kLog2e, per_tensor, decode_wait_limit(), a.out, po, pml, pieces, w.rows, sums);
  if (e != cudaSuccess) return e;
  e = launch_pdl(ragged_merge_kernel<D, OutT>, dim3(unsigned(grid), unsigned((std::min(w.rows, C::RPB) + 31) / 32)),
                 dim3(256), 0, st, static_cast<const float*>(po), static_cast<const float*>(pml),
                 static_cast<const RgPiece*>(pieces), grid, w.rows, b.p, int(d.n_q_heads),
                 static_cast<OutT*>(a.out));
  if (e != cudaSuccess || !step) return e;
  void* dws = at + 2 * w.seqs + w.q1;
  e = cudaError_t(launch_decode_partial(b.q1, a.n_seqs, a.kc, a.vc, a.ks, a.vs, a.tables, b.ctx1, a.max_ctx, a.sm_scale, plan, dws,
                                        fmt, d, st, 1));
  if (e != cudaSuccess) return e;
  return cudaError_t(launch_decode_merge(a.n_seqs, b.ctx1, a.max_ctx, a.out, a.out_f32, dws, plan, d, st, 0, b.row1));
}
}  // namespace

size_t ragged_workspace(int32_t total_q, const kvq_dims& d) { return rg_space(total_q, d).total; }

int launch_ragged(const RaggedArgs& a, kvq_fmt fmt, const kvq_dims& d, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int pt = fmt == KVQ_INT8_TENSOR;
  cudaError_t e;
#define KVQ_RG(DD, FF) \
  e = a.out_f32 ? ragged_dispatch<DD, FF, true>(a, fmt, d, pt, st) : ragged_dispatch<DD, FF, false>(a, fmt, d, pt, st)
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
