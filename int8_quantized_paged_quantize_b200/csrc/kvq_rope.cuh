// Rows of kvq_append_rope: K and V rows at a token stride (views of one fused
// projection), the rotary embedding applied to K on the way to the quantizer
// of the append kernel, and CTAs that rotate the query's rows.
//
//   pair (a, b) of a row at position p, angle i:
//     a' = a cos[p][i] - b sin[p][i],   b' = b cos[p][i] + a sin[p][i]
//   pairs (i, i + rotary/2), or (2i, 2i + 1) when interleaved; channels from
//   `rotary` on pass through.
// Products and sums are rounded one by one in FP32 (no fused multiply-add), so
// the result does not depend on which of a pair a thread holds, and then to
// BF16: what a separate rotary kernel with BF16 output followed by kvq_append
// stores, bit for bit.
//
// Bound: HBM ((2 Hq + 2 Hk) rows of 2D bytes and the pages per token).
#pragma once

#include "kvq_append.cuh"

namespace kvq {

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// own * cos -+ partner * sin of a BF16 pair (minus for the first of the pair).
__device__ __forceinline__ float rope_first(float a, float b, float c, float s) {
  return __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
}
__device__ __forceinline__ float rope_second(float a, float b, float c, float s) {
  return __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
}

// Eight angles' cosines and sines.
struct Angles8 {
  float c[8], s[8];
  __device__ __forceinline__ void load(const float* row, int half, int i) {
#pragma unroll
    for (int x = 0; x < 8; x += 4) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(row + i + x));
      const float4 b = __ldg(reinterpret_cast<const float4*>(row + half + i + x));
      c[x] = a.x; c[x + 1] = a.y; c[x + 2] = a.z; c[x + 3] = a.w;
      s[x] = b.x; s[x + 1] = b.y; s[x + 2] = b.z; s[x + 3] = b.w;
    }
  }
};

template <int D>
struct RopeRows {
  const __nv_bfloat16* __restrict__ q;
  const __nv_bfloat16* __restrict__ k;
  const __nv_bfloat16* __restrict__ v;
  int64_t qs, kst, vst;                        // elements between tokens
  const int64_t* __restrict__ slots;
  const int32_t* __restrict__ positions;
  const float* __restrict__ cos_sin;           // [max_pos][rotary]: cosines, then sines
  __nv_bfloat16* __restrict__ q_out;
  int Hq, max_pos, rotary;
  bool interleaved;

  static constexpr bool kQuery = true;
  static constexpr int kHeads = 16;            // query heads per CTA
  // 64 registers: the rows of a pair and its angles are in flight together
  template <int FMT>
  static constexpr int ctas_per_sm() { return 4; }

  // position of token t, or -1 outside the table
  __device__ __forceinline__ int position(int64_t t) const {
    const int p = positions[t];
    return p >= 0 && p < max_pos ? p : -1;
  }
  // a token without a position in the table is not written
  __device__ __forceinline__ int64_t slot(int64_t t, int h) const {
    const int64_t s = slots[t];
    if (s < 0 || position(t) >= 0) return s;
    if (h == 0) flag_error(KVQ_DEVERR_POSITION);
    return -1;
  }

  __device__ __forceinline__ void load(int64_t t, int which, int Hk, int h, int d0,
                                       uint32_t (&raw)[D / (2 * kRowLanes)]) const {
    (void)Hk;
    if (which) {
      load_row<D>(v + t * vst + int64_t(h) * D + d0, raw);
      return;
    }
    const __nv_bfloat16* row = k + t * kst + int64_t(h) * D;
    const float* cs = cos_sin + int64_t(max(position(t), 0)) * rotary;
    const int half = rotary >> 1;
    load_row<D>(row + d0, raw);
#pragma unroll
    for (int c = 0; c < D / (8 * kRowLanes); ++c) {
      const int d = d0 + 8 * c;                // a chunk of 8 channels: rotated or not as a whole
      if (d >= rotary) continue;
      if (interleaved) {
        const float4 co = __ldg(reinterpret_cast<const float4*>(cs + (d >> 1)));
        const float4 si = __ldg(reinterpret_cast<const float4*>(cs + half + (d >> 1)));
        const float cc[4] = {co.x, co.y, co.z, co.w}, ss[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float a = bf16_lo(raw[4 * c + e]), b = bf16_hi(raw[4 * c + e]);
          raw[4 * c + e] = pack_bf16x2(rope_first(a, b, cc[e], ss[e]), rope_second(a, b, cc[e], ss[e]));
        }
      } else {
        // the other chunk of the pair: the same row, so mostly an L1 hit
        const bool first = d < half;
        const uint4 o = *reinterpret_cast<const uint4*>(row + (first ? d + half : d - half));
        const uint32_t ow[4] = {o.x, o.y, o.z, o.w};
        Angles8 an;
        an.load(cs, half, first ? d : d - half);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x0 = bf16_lo(raw[4 * c + e]), x1 = bf16_hi(raw[4 * c + e]);
          const float y0 = bf16_lo(ow[e]), y1 = bf16_hi(ow[e]);
          const float r0 = first ? rope_first(x0, y0, an.c[2 * e], an.s[2 * e])
                                 : rope_second(y0, x0, an.c[2 * e], an.s[2 * e]);
          const float r1 = first ? rope_first(x1, y1, an.c[2 * e + 1], an.s[2 * e + 1])
                                 : rope_second(y1, x1, an.c[2 * e + 1], an.s[2 * e + 1]);
          raw[4 * c + e] = pack_bf16x2(r0, r1);
        }
      }
    }
  }

  // The query rows of tokens tb .. tb + n - 1, heads 16 y .. 16 y + 15: a warp
  // takes two tokens, a lane the pairs of eight angles (two 16-byte chunks) of
  // every fourth (D = 128) or eighth head, so the angles are loaded once.
  __device__ __forceinline__ void query(int64_t tb, int n, int y) const {
    constexpr int UNITS = D / 16, HPI = 32 / UNITS, IT = kHeads / HPI;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int u = lane % UNITS, h0 = y * kHeads + lane / UNITS;
    const int half = rotary >> 1;
    const bool rot = u < (rotary >> 4);
    // the unit's chunks: a pair of chunks half a rotation apart, or 16
    // neighbouring channels (interleaved pairs, and what passes through)
    const int c0 = rot && !interleaved ? 8 * u : 16 * u;
    const int c1 = rot && !interleaved ? 8 * u + half : 16 * u + 8;
    for (int i = 0; i < 2; ++i) {
      const int ti = 2 * warp + i;
      if (ti >= n) break;
      const int64_t t = tb + ti;
      const int p = position(t);
      uint4 x0[IT], x1[IT];
      const __nv_bfloat16* row = q + t * qs;
#pragma unroll
      for (int j = 0; j < IT; ++j) {
        const int h = h0 + j * HPI;
        if (h < Hq) {
          x0[j] = *reinterpret_cast<const uint4*>(row + int64_t(h) * D + c0);
          x1[j] = *reinterpret_cast<const uint4*>(row + int64_t(h) * D + c1);
        }
      }
      if (p < 0) {                             // left as it is
        if (y == 0 && lane == 0 && slots[t] >= 0) flag_error(KVQ_DEVERR_POSITION);
        continue;
      }
      Angles8 an;
      if (rot) an.load(cos_sin + int64_t(p) * rotary, half, 8 * u);
#pragma unroll
      for (int j = 0; j < IT; ++j) {
        const int h = h0 + j * HPI;
        if (h >= Hq) continue;
        if (rot) {
          uint32_t* a = reinterpret_cast<uint32_t*>(&x0[j]);
          uint32_t* b = reinterpret_cast<uint32_t*>(&x1[j]);
          if (interleaved) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float a0 = bf16_lo(a[e]), b0 = bf16_hi(a[e]), a1 = bf16_lo(b[e]), b1 = bf16_hi(b[e]);
              a[e] = pack_bf16x2(rope_first(a0, b0, an.c[e], an.s[e]), rope_second(a0, b0, an.c[e], an.s[e]));
              b[e] = pack_bf16x2(rope_first(a1, b1, an.c[4 + e], an.s[4 + e]),
                                 rope_second(a1, b1, an.c[4 + e], an.s[4 + e]));
            }
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float a0 = bf16_lo(a[e]), a1 = bf16_hi(a[e]), b0 = bf16_lo(b[e]), b1 = bf16_hi(b[e]);
              a[e] = pack_bf16x2(rope_first(a0, b0, an.c[2 * e], an.s[2 * e]),
                                 rope_first(a1, b1, an.c[2 * e + 1], an.s[2 * e + 1]));
              b[e] = pack_bf16x2(rope_second(a0, b0, an.c[2 * e], an.s[2 * e]),
                                 rope_second(a1, b1, an.c[2 * e + 1], an.s[2 * e + 1]));
            }
          }
        }
        __nv_bfloat16* o = q_out + (t * Hq + h) * D;
        *reinterpret_cast<uint4*>(o + c0) = x0[j];
        *reinterpret_cast<uint4*>(o + c1) = x1[j];
      }
    }
  }
};

}  // namespace kvq
