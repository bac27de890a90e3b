// Dequantizing read-back of cached tokens (kvq_read): runs of tokens of each
// sequence out of the pages, as BF16 or FP32 rows [token][KV head][D].
//
// A warp takes the (up to 16) output rows of one window for one KV head: it
// finds their sequences, and walks them in segments (consecutive tokens of one
// page). Of a segment's K page a lane holds 16 channels of a token, as the
// page stores them, and writes them as one 32-byte piece. The V page is
// transposed, so it passes through shared memory: a lane takes 4 tokens x 16 channels and turns them by
// byte permutes, with the chunks placed so that the 8 channel groups read
// different banks. Nothing is computed in fewer than 32 bits; the values are
// rounded once, to the output type.
//
// Bound: HBM (the pages' bytes in, 2 D Hk values out per token).
#pragma once

#include <cuda_fp16.h>

#include "kvq_common.cuh"
#include "kvq_prefill.cuh"

namespace kvq {

template <int D, int FMT>
struct ReadCfg {
  static constexpr bool KIVI = FMT == KVQ_KIVI2 || FMT == KVQ_KIVI4;
  static constexpr int BITS = FMT == KVQ_KIVI2 ? 2 : FMT == KVQ_KIVI4 ? 4 : FMT == KVQ_BF16 ? 16 : 8;
  static constexpr int PAGE = kBlockSize * D * BITS / 8;
  static constexpr int WARPS = 8;
  // the V page of a warp; low-bit pages: 16 bytes apart after every 16 channels, so that
  // the 8 channel groups of a warp's reads lie in different banks
  static constexpr int GROUPB = 4 * BITS * 8;                    // bytes of 16 channels of a V page
  static constexpr int SMEM = KIVI ? PAGE + (D / 16) * 16 : PAGE;
};

// 16 output values as one row piece.
template <typename OutT>
__device__ __forceinline__ void store16(OutT* dst, const float (&x)[16], bool wide) {
  if constexpr (sizeof(OutT) == 2) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
    if (wide) {                                   // a whole 32-byte sector by one store
      asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(w[0]), "r"(w[1]),
                   "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                   : "memory");
    } else {
      reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
      reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
  } else {
    (void)wide;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      reinterpret_cast<float4*>(dst)[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
  }
}

// Four 8-bit codes (packed little-endian) as floats.
template <int FMT>
__device__ __forceinline__ void codes4_to_f32(uint32_t w, float* x) {
  uint32_t lo, hi;
  if constexpr (FMT == KVQ_FP8_E4M3) fp8x4_to_f16x4<true>(w, lo, hi);
  else if constexpr (FMT == KVQ_FP8_E5M2) fp8x4_to_f16x4<false>(w, lo, hi);
  else s8x4_to_f16x4(w, lo, hi);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
}

// Largest index i of cu[0 .. n-1] with cu[i] <= r (-1 if none), for a
// non-decreasing cu, by the whole warp: 32 probes a step.
__device__ __forceinline__ int warp_upper(const int32_t* cu, int n, int r, int lane) {
  int lo = -1, hi = n;                            // cu[lo] <= r < cu[hi]
  while (hi - lo > 1) {
    const int step = max(1, (hi - lo + 31) / 32);
    const int i = lo + (lane + 1) * step;
    const bool le = i < hi && cu[i] <= r;
    const unsigned m = __ballot_sync(0xffffffffu, le);
    const int c = __popc(m & ~(m + 1u));          // probes from the first on that hold
    const int nlo = lo + c * step;
    hi = min(hi, nlo + step);
    lo = nlo;
  }
  return lo;
}

// 3 CTAs an SM (80 registers; BF16 pages and static scales, which spill at 3: 2). 32 whole
// contexts of 4,100 tokens, 8 KV heads, in a graph: INT8 167 us against 198 at 128 registers
// and 212 with K and V in CTAs of their own; 4-bit 57 against 66; static scales 265 with 2,
// 286 with 3. At 4 the spills cost more.
template <int D, int FMT, typename OutT>
__global__ void __launch_bounds__(256, FMT == KVQ_BF16 || FMT == KVQ_INT8_CHANNEL ? 2 : 3) read_kernel(
    const uint8_t* __restrict__ kc, const uint8_t* __restrict__ vc,
    const __nv_bfloat16* __restrict__ ks, const __nv_bfloat16* __restrict__ vs,
    const int32_t* __restrict__ tables, const int32_t* __restrict__ starts,
    const int32_t* __restrict__ cu, int B, int total, int Hk, int NB, int W, int per_tensor,
    OutT* __restrict__ ko, OutT* __restrict__ vo) {
  using C = ReadCfg<D, FMT>;
  constexpr bool F8 = FMT == KVQ_FP8_E4M3 || FMT == KVQ_FP8_E5M2;
  constexpr bool SI = FMT == KVQ_INT8_CHANNEL;
  constexpr int NCH = D / 16;                     // 16-channel pieces of a row
  __shared__ __align__(16) uint8_t smem[C::WARPS][C::SMEM];
  // a programmatic dependent of the append ahead of it
  tc::grid_dep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (blockIdx.x == 0)                            // lengths that do not describe rows
    for (int b = threadIdx.x; b <= B; b += blockDim.x) {
      const int c = cu[b];
      if (c < 0 || c > total || (b > 0 && c < cu[b - 1])) flag_error(KVQ_DEVERR_RANGE);
    }
  const int64_t item = int64_t(blockIdx.x) * C::WARPS + warp;
  const int64_t win = item / Hk;
  const int h = int(item % Hk);
  if (win * kBlockSize >= total) return;
  const int r0 = int(win * kBlockSize), n = min(kBlockSize, total - r0);

  // ---- the rows: sequence, token, page (lanes 0 .. 15)
  int bs = warp_upper(cu, B + 1, r0, lane);
  int64_t tok = -1;                               // token of this lane's row (-1: no such row)
  int blk = -1;                                   // its block (-1: none, zeros are written)
  int seq = -1;
  if (lane < n) {
    const int r = r0 + lane;
    int b = max(bs, 0);
    while (b < B && cu[b + 1] <= r) ++b;
    if (b < B && cu[b] >= 0 && cu[b] <= r) {
      seq = b;
      const int s = starts[b];
      tok = int64_t(s) + (r - cu[b]);
      if (s < 0 || tok >= int64_t(W) * kBlockSize) {
        if (h == 0) flag_error(KVQ_DEVERR_CONTEXT);
        tok = 0;
      } else {
        blk = tables[int64_t(b) * W + tok / kBlockSize];
        if (blk < 0 || blk >= NB) {
          if (h == 0) flag_error(KVQ_DEVERR_BLOCK);
          blk = -1;
        }
      }
    }
  }
  // segments: a row continues its predecessor's when it is the next token of
  // the same page
  const int64_t ptok = __shfl_up_sync(0xffffffffu, tok, 1);
  const int pblk = __shfl_up_sync(0xffffffffu, blk, 1), pseq = __shfl_up_sync(0xffffffffu, seq, 1);
  const bool valid = lane < n && seq >= 0;
  const bool start = valid && !(lane > 0 && pseq == seq && pblk == blk && tok == ptok + 1 && tok % kBlockSize != 0);
  const unsigned vmask = __ballot_sync(0xffffffffu, valid);
  unsigned smask = __ballot_sync(0xffffffffu, start);
  const bool wide = sizeof(OutT) == 2 && ((reinterpret_cast<uintptr_t>(ko) | reinterpret_cast<uintptr_t>(vo)) & 31) == 0;

  for (unsigned left = smask; left != 0u; left &= left - 1u) {
    const int i0 = __ffs(left) - 1;
    const unsigned stop = (smask | ~vmask) & ~((2u << i0) - 1u);
    const int len = (stop ? __ffs(stop) - 1 : 32) - i0;
    const int64_t t0 = __shfl_sync(0xffffffffu, tok, i0);
    const int pb = __shfl_sync(0xffffffffu, blk, i0);
    const int sq = __shfl_sync(0xffffffffu, seq, i0);
    const int o0 = int(t0 % kBlockSize);          // the segment's tokens o0 .. o0 + len - 1 of the page
    const int64_t row0 = r0 + i0;
    if (pb < 0) {                                 // no such page: zeros
      for (int j = lane; j < len * NCH; j += 32) {
        float z[16] = {};
        const int64_t at = ((row0 + j / NCH) * Hk + h) * D + (j % NCH) * 16;
        if (ko) store16(ko + at, z, wide);
        if (vo) store16(vo + at, z, wide);
      }
      continue;
    }
    const int64_t page = int64_t(pb) * Hk + h;
    const uint8_t* kp = kc + page * C::PAGE;
    const uint8_t* vp = vc + page * C::PAGE;

    // ---- V: its loads first, so that they are in flight under K's
    constexpr int VL = (C::PAGE + 511) / 512;     // 2 bits at D = 64: half a warp's chunks
    uint4 vraw[VL];
    if (vo) {
#pragma unroll
      for (int i = 0; i < VL; ++i)
        if (C::PAGE >= 512 * (i + 1) || (lane + 32 * i) * 16 < C::PAGE) vraw[i] = reinterpret_cast<const uint4*>(vp)[lane + 32 * i];
    }

    // ---- K: item j = (token group, piece c, token): 16 channels of a token
    if (ko) {
      constexpr int KI = 16 * NCH / 32;
      uint4 ka[KI], kb[KI];
#pragma unroll
      for (int i = 0; i < KI; ++i) {
        const int j = lane + 32 * i;
        if constexpr (C::BITS == 16) {            // chunks of 8 channels: 2c and 2c + 1
          const int g = j / (8 * NCH), c = (j >> 3) % NCH, t = j & 7;
          const uint8_t* src = kp + g * 16 * D + 2 * c * 128 + t * 16;
          ka[i] = *reinterpret_cast<const uint4*>(src);
          kb[i] = *reinterpret_cast<const uint4*>(src + 128);
        } else if constexpr (C::BITS == 8) {
          ka[i] = reinterpret_cast<const uint4*>(kp)[j];
        } else if constexpr (C::BITS == 4) {
          const uint2 w = reinterpret_cast<const uint2*>(kp)[j];
          ka[i] = make_uint4(w.x, w.y, 0u, 0u);
        } else {
          ka[i] = make_uint4(reinterpret_cast<const uint32_t*>(kp)[j], 0u, 0u, 0u);
        }
      }
#pragma unroll
      for (int i = 0; i < KI; ++i) {
        const int j = lane + 32 * i;
        const int c = (j >> 3) % NCH, t = (j / (8 * NCH)) * 8 + (j & 7);
        if (t < o0 || t >= o0 + len) continue;
        float x[16];
        if constexpr (C::BITS == 16) {
          const uint32_t w[8] = {ka[i].x, ka[i].y, ka[i].z, ka[i].w, kb[i].x, kb[i].y, kb[i].z, kb[i].w};
#pragma unroll
          for (int e = 0; e < 8; ++e) { x[2 * e] = bf16_lo(w[e]); x[2 * e + 1] = bf16_hi(w[e]); }
        } else if constexpr (C::BITS == 8) {
          const uint32_t w[4] = {ka[i].x, ka[i].y, ka[i].z, ka[i].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) codes4_to_f32<FMT>(w[e], x + 4 * e);
          if constexpr (F8) {
            const float s = __bfloat162float(ks[page * kBlockSize + t]);
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] *= s;
          } else if constexpr (FMT == KVQ_INT8_ASYM) {
            const __nv_bfloat162 m = reinterpret_cast<const __nv_bfloat162*>(ks)[page * kBlockSize + t];
            const float s = __low2float(m), z = __high2float(m);
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = (x[e] - z) * s;
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e)
              x[e] *= __bfloat162float(ks[per_tensor ? 0 : h * D + 16 * c + e]);
          }
        } else {
          // unit (t, c): codes 4m + jj at bit 8jj + 2m, or in word m/2 at bit 8jj + 4(m%2)
          uint32_t w4[4];
          if constexpr (C::BITS == 2) {
#pragma unroll
            for (int m = 0; m < 4; ++m) w4[m] = (ka[i].x >> (2 * m)) & 0x03030303u;
          } else {
            w4[0] = ka[i].x & 0x0f0f0f0fu; w4[1] = (ka[i].x >> 4) & 0x0f0f0f0fu;
            w4[2] = ka[i].y & 0x0f0f0f0fu; w4[3] = (ka[i].y >> 4) & 0x0f0f0f0fu;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) codes4_to_f32<FMT>(w4[e], x + 4 * e);
          // (s, z) of the channels: block i of the group holds channels i D/8 ..
          const int64_t g8 = (t0 / kBlockSize) & ~int64_t(7);
          constexpr int PER = D / 8;              // channels per block
#pragma unroll
          for (int e0 = 0; e0 < 16; e0 += (PER < 16 ? PER : 16)) {
            const int ch = 16 * c + e0;
            const int64_t bi = g8 + ch / PER;
            int mb = bi < W ? tables[int64_t(sq) * W + bi] : -1;
            if (mb < 0 || mb >= NB) {
              flag_error(KVQ_DEVERR_BLOCK);
              mb = -1;
            }
#pragma unroll
            for (int e = 0; e < (PER < 16 ? PER : 16); e += 4) {   // four (s, z) pairs
              uint4 m = make_uint4(0, 0, 0, 0);
              if (mb >= 0)
                m = __ldg(reinterpret_cast<const uint4*>(ks + ((int64_t(mb) * Hk + h) * kBlockSize + ch % PER + e) * 2));
              x[e0 + e] = __fmaf_rn(x[e0 + e], bf16_lo(m.x), bf16_hi(m.x));
              x[e0 + e + 1] = __fmaf_rn(x[e0 + e + 1], bf16_lo(m.y), bf16_hi(m.y));
              x[e0 + e + 2] = __fmaf_rn(x[e0 + e + 2], bf16_lo(m.z), bf16_hi(m.z));
              x[e0 + e + 3] = __fmaf_rn(x[e0 + e + 3], bf16_lo(m.w), bf16_hi(m.w));
            }
          }
        }
        store16(ko + ((row0 + t - o0) * Hk + h) * D + 16 * c, x, wide);
      }
    }

    // ---- V: lane = 4 tokens (quarter tq) x 16 channels (piece g)
    if (vo) {
      const int g = lane & 7, tq = lane >> 3;
      uint32_t cw[16];                            // codes: 4 tokens of channel 16 g + i (8 bits each)
      uint32_t cw2[C::BITS == 16 ? 16 : 1];       // BF16: tokens 4 tq, +1 in cw, +2, +3 in cw2
      __syncwarp();
      if constexpr (C::KIVI) {
#pragma unroll
        for (int i = 0; i < VL; ++i) {
          const int at = (lane + 32 * i) * 16;
          if (at < C::PAGE) *reinterpret_cast<uint4*>(smem[warp] + at + at / C::GROUPB * 16) = vraw[i];
        }
      } else {
        // chunk x (channel x % D) at x with its low 3 bits xored by the piece
#pragma unroll
        for (int i = 0; i < VL; ++i) {
          const int xch = lane + 32 * i;
          *reinterpret_cast<uint4*>(smem[warp] + (xch ^ ((xch >> 4) & 7)) * 16) = vraw[i];
        }
      }
      __syncwarp();
      if (g < NCH && 4 * tq < o0 + len && 4 * tq + 4 > o0) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int ch = 16 * g + i;
          if constexpr (C::BITS == 16) {
            const int xch = (tq >> 1) * D + ch;
            const uint2 w = *reinterpret_cast<const uint2*>(smem[warp] + (xch ^ ((xch >> 4) & 7)) * 16 + (tq & 1) * 8);
            cw[i] = w.x;
            cw2[i] = w.y;
          } else if constexpr (C::BITS == 8) {
            cw[i] = *reinterpret_cast<const uint32_t*>(smem[warp] + (ch ^ ((ch >> 4) & 7)) * 16 + tq * 4);
          } else if constexpr (C::BITS == 4) {
            const uint32_t w = *reinterpret_cast<const uint32_t*>(smem[warp] + 8 * ch + 16 * g + 4 * (tq >> 1));
            cw[i] = (w >> (4 * (tq & 1))) & 0x0f0f0f0fu;
          } else {
            cw[i] = (*reinterpret_cast<const uint32_t*>(smem[warp] + 4 * ch + 16 * g) >> (2 * tq)) & 0x03030303u;
          }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {             // token 4 tq + k
          const int t = 4 * tq + k;
          if (t < o0 || t >= o0 + len) continue;
          float x[16];
          if constexpr (C::BITS == 16) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const uint32_t w = k < 2 ? cw[i] : cw2[i];
              x[i] = (k & 1) ? bf16_hi(w) : bf16_lo(w);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
              // byte k of four channels' words
              const uint32_t a = __byte_perm(cw[i], cw[i + 1], k | ((k + 4) << 4));
              const uint32_t b = __byte_perm(cw[i + 2], cw[i + 3], k | ((k + 4) << 4));
              codes4_to_f32<FMT>(__byte_perm(a, b, 0x5410), x + i);
            }
            if constexpr (F8) {
              const float s = __bfloat162float(vs[page * kBlockSize + t]);
#pragma unroll
              for (int e = 0; e < 16; ++e) x[e] *= s;
            } else if constexpr (FMT == KVQ_INT8_ASYM) {
              const __nv_bfloat162 m = reinterpret_cast<const __nv_bfloat162*>(vs)[page * kBlockSize + t];
              const float s = __low2float(m), z = __high2float(m);
#pragma unroll
              for (int e = 0; e < 16; ++e) x[e] = (x[e] - z) * s;
            } else if constexpr (SI) {
#pragma unroll
              for (int e = 0; e < 16; ++e)
                x[e] *= __bfloat162float(vs[per_tensor ? 0 : h * D + 16 * g + e]);
            } else {
              const __nv_bfloat162 m = reinterpret_cast<const __nv_bfloat162*>(vs)[page * kBlockSize + t];
              const float s = __low2float(m), z = __high2float(m);
#pragma unroll
              for (int e = 0; e < 16; ++e) x[e] = __fmaf_rn(x[e], s, z);
            }
          }
          store16(vo + ((row0 + t - o0) * Hk + h) * D + 16 * g, x, wide);
        }
      }
      __syncwarp();
    }
  }
}

}  // namespace kvq
