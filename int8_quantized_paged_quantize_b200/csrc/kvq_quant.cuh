// The row quantizers of the append kernels: one (token, KV head) row of BF16
// values to codes and scale on a group of 8 lanes.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cstdint>

#include "kvq_common.cuh"

namespace kvq {

// A (token, KV head) row of D BF16 values is quantized by a group of
// kRowLanes = 8 lanes with E = D/8 consecutive values each (two 16-byte loads
// at D = 128), so a warp instruction serves four rows and the per-row work
// (range, scale, reciprocal, zero point) is shared by 16 values per lane. The
// range is an integer max over the group, the BF16 scale (+ zero point) is
// formed on each of its lanes, and the lane's codes are packed little-endian
// in d order into `w`.
constexpr int kRowLanes = 8;

template <int D, int FMT>
struct RowCodes {
  static constexpr int E = D / kRowLanes;
  static constexpr int ELT = (FMT == KVQ_BF16) ? 2 : 1;
  static constexpr int WORDS = E * ELT / 4;
  uint32_t w[WORDS];
  __nv_bfloat16 s;
  int zp;
};

// This lane's D/8 BF16 values of a row, as packed pairs.
template <int D>
__device__ __forceinline__ void load_row(const __nv_bfloat16* src, uint32_t (&raw)[D / (2 * kRowLanes)]) {
#pragma unroll
  for (int c = 0; c < D / (8 * kRowLanes); ++c) {
    const uint4 u = reinterpret_cast<const uint4*>(src)[c];
    raw[4 * c] = u.x; raw[4 * c + 1] = u.y; raw[4 * c + 2] = u.z; raw[4 * c + 3] = u.w;
  }
}

// a / c for a constant c > 0 and a >= 0: RN(a * RN(1/c)) corrected once on the
// exact FMA residual. For c = 448 and c = 57344 over every BF16 a, and for
// c = 255 over every a = RN(hi - lo) of BF16 hi >= 0 >= lo, this is the IEEE
// quotient bit for bit (tests/test_scale_division.py enumerates all of them),
// so the row scales are those of a plain division.
template <int C>
__device__ __forceinline__ float div_by_const(float a) {
  constexpr float c = float(C), r = 1.0f / float(C);
  const float q = __fmul_rn(a, r);
  return __fmaf_rn(__fmaf_rn(-q, c, a), r, q);
}

// x / s for the row's BF16 scale s > 0, as the codes need it. For s >= 2^-100
// it is RN(x * RN(1/s)) corrected once on the exact FMA residual (Markstein's
// method), with the residual's sign folded so that a zero x keeps its sign
// (-0 / s = -0) without a test: it may differ from the IEEE quotient in the
// last bit, but the E4M3, E5M2 and rint codes taken from it are the IEEE
// quotient's for every BF16 x with |x| <= 65536 s, subnormal x included
// (enumerated by tests/test_scale_division.py). Rows with a smaller scale take
// the IEEE division.
struct ScaleDiv {
  float s, r;
  bool fast;
  __device__ __forceinline__ explicit ScaleDiv(float s_) {
    s = s_;
    fast = s_ >= 7.88860905e-31f;                   // 2^-100
    r = fast ? __frcp_rn(s_) : 0.f;
  }
  __device__ __forceinline__ float operator()(float x) const {
    if (!fast) return __fdiv_rn(x, s);
    const float q = __fmul_rn(x, r);
    const float e = __fmaf_rn(q, s, -x);             // minus the residual x - q s (exact)
    return __fmaf_rn(-e, r, q);
  }
};

// Integer rounding by one addition: for |q| < 2^22, q + 1.5 * 2^23 lies in
// [2^23, 2^24), where the float spacing is 1, so the sum is rint(q) (round to
// nearest even) and its bit pattern is kRintBits + rint(q).
constexpr float kRintMagic = 12582912.0f;
constexpr int kRintBits = 0x4B400000;

// The low bytes of four ints, packed little-endian.
__device__ __forceinline__ uint32_t pack_low_bytes(int a, int b, int c, int d) {
  const uint32_t lo = __byte_perm(uint32_t(a), uint32_t(b), 0x0040);
  const uint32_t hi = __byte_perm(uint32_t(c), uint32_t(d), 0x0040);
  return __byte_perm(lo, hi, 0x5410);
}


// Lane-wise max of two pairs of 16-bit fields, unsigned or signed (the
// signed form with a floor of 0).
__device__ __forceinline__ uint32_t vmax_u16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t vmax_relu_s16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.relu.s16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Field-wise max of a u16x2 word over the kRowLanes lanes of this row group
// (the four groups of the warp reduce at once).
__device__ __forceinline__ uint32_t row_vmax_u16x2(uint32_t v) {
#pragma unroll
  for (int o = kRowLanes / 2; o > 0; o >>= 1) v = vmax_u16x2(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// The two BF16 values of a packed pair as floats (low half first).
__device__ __forceinline__ float2 bf16x2_to_float2(uint32_t w) { return make_float2(bf16_lo(w), bf16_hi(w)); }

// Markstein's corrected quotient on a pair: q = RN(x r), e = RN(q s - x)
// (exact), q' = RN(q - e r), with -x and -r passed in so that a zero x keeps
// its sign; the same arithmetic as ScaleDiv, two lanes per instruction.
__device__ __forceinline__ float2 div_pair(float2 x, float2 r2, float2 nr2, float2 s2) {
  const float2 nx = __fmul2_rn(x, make_float2(-1.f, -1.f));
  const float2 q = __fmul2_rn(x, r2);
  const float2 e = __ffma2_rn(q, s2, nx);
  return __ffma2_rn(e, nr2, q);
}

// Two pairs of quotients as four E4M3 / E5M2 codes (RNE, satfinite),
// little-endian: a.x in the low byte.
template <bool E4>
__device__ __forceinline__ uint32_t fp8x4(float2 a, float2 b) {
  uint32_t w;
  if constexpr (E4)
    asm("{\n .reg .b16 lo, hi;\n cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n"
        " cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n mov.b32 %0, {lo, hi};\n}"
        : "=r"(w) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  else
    asm("{\n .reg .b16 lo, hi;\n cvt.rn.satfinite.e5m2x2.f32 lo, %2, %1;\n"
        " cvt.rn.satfinite.e5m2x2.f32 hi, %4, %3;\n mov.b32 %0, {lo, hi};\n}"
        : "=r"(w) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return w;
}

// Two ints saturated to [-128, 127] in bytes 0 (b) and 1 (a), bytes 2-3 from
// the low half of c.
__device__ __forceinline__ uint32_t pack_sat_s8x2(int a, int b, uint32_t c) {
  uint32_t d;
  asm("cvt.pack.sat.s8.s32.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

// The row maximum is taken on bit patterns: non-negative floats (and BF16
// values) order as their bits read as integers and every negative one (-0
// included) reads as a negative signed integer, so an integer max with a floor
// of 0 gives the float maximum, +0 when nothing is positive. The lane's BF16
// pairs are reduced as 16-bit fields, two values per instruction. Every lane
// of the warp must call the quantizers (the half-warp reductions are warp-wide
// shuffles); a row that is not stored is still quantized, from whatever its
// lanes hold.
template <int D, int FMT>
__device__ __forceinline__ void quantize_row(const uint32_t (&raw)[D / (2 * kRowLanes)], RowCodes<D, FMT>& rc) {
  constexpr int E = D / kRowLanes;
  constexpr int NW = E / 2;                          // BF16 pairs of the lane
  rc.zp = 0;
  rc.s = __float2bfloat16_rn(0.f);
  if constexpr (FMT == KVQ_BF16) {
#pragma unroll
    for (int i = 0; i < NW; ++i) rc.w[i] = raw[i];
    return;
  } else {
#pragma unroll
    for (int i = 0; i < RowCodes<D, FMT>::WORDS; ++i) rc.w[i] = 0u;
    if constexpr (FMT == KVQ_FP8_E4M3 || FMT == KVQ_FP8_E5M2) {
      // s = bf16(amax / max code), code = fp8_rne_satfinite(x / s)
      constexpr bool E4 = FMT == KVQ_FP8_E4M3;
      uint32_t m = raw[0] & 0x7fff7fffu;             // |x| of both halves
#pragma unroll
      for (int i = 1; i < NW; ++i) m = vmax_u16x2(m, raw[i] & 0x7fff7fffu);
      m = row_vmax_u16x2(m);
      const float amax = __uint_as_float(max(m & 0xffffu, m >> 16) << 16);
      rc.s = __float2bfloat16_rn(E4 ? div_by_const<448>(amax) : div_by_const<57344>(amax));
      const float s = __bfloat162float(rc.s);
      if (s >= 7.88860905e-31f) {                    // 2^-100: the corrected quotient
        const float r = __frcp_rn(s);
        const float2 r2 = make_float2(r, r), nr2 = make_float2(-r, -r), s2 = make_float2(s, s);
#pragma unroll
        for (int i = 0; i < NW; i += 2)
          rc.w[i >> 1] = fp8x4<E4>(div_pair(bf16x2_to_float2(raw[i]), r2, nr2, s2),
                                   div_pair(bf16x2_to_float2(raw[i + 1]), r2, nr2, s2));
      } else if (s != 0.f) {                         // tiny scale: the IEEE quotient
#pragma unroll
        for (int i = 0; i < NW; i += 2) {
          const float2 a = bf16x2_to_float2(raw[i]), b = bf16x2_to_float2(raw[i + 1]);
          rc.w[i >> 1] = fp8x4<E4>(make_float2(__fdiv_rn(a.x, s), __fdiv_rn(a.y, s)),
                                   make_float2(__fdiv_rn(b.x, s), __fdiv_rn(b.y, s)));
        }
      }
    } else {  // INT8 asymmetric: range [lo, hi] widened to hold 0
      // hi = max(0, max x) and nlo = max(0, max -x), as 16-bit fields
      uint32_t hw = vmax_relu_s16x2(raw[0], 0u), nw = vmax_relu_s16x2(raw[0] ^ 0x80008000u, 0u);
#pragma unroll
      for (int i = 1; i < NW; ++i) {
        hw = vmax_relu_s16x2(hw, raw[i]);
        nw = vmax_relu_s16x2(nw, raw[i] ^ 0x80008000u);
      }
      // both maxima in one word (hi low, nlo high), reduced over the row group
      const uint32_t hn = row_vmax_u16x2(vmax_u16x2(__byte_perm(hw, nw, 0x5410),
                                                     __byte_perm(hw, nw, 0x7632)));
      const float hi = bf16_lo(hn), nlo = bf16_hi(hn);
      rc.s = __float2bfloat16_rn(div_by_const<255>(__fadd_rn(hi, nlo)));
      const float s = __bfloat162float(rc.s);
      if (s != 0.f) {
        const ScaleDiv div(s);
        const float zq = fminf(fmaxf(-div(nlo), -1024.f), 1024.f);   // lo / s
        rc.zp = min(127, max(-128, -128 - __float2int_rn(zq)));
        // code = clamp(rint(x / s) + zp, -128, 127): every x of the row lies in
        // [lo, hi], so |x / s| stays near 255 and the rounding addition
        // applies; the sum's bits less kRintBits are rint(x / s), zp is added
        // as an integer and the pack saturates
        const int off = rc.zp - kRintBits;
        int c[E];
        if (div.fast) {
          const float2 r2 = make_float2(div.r, div.r), nr2 = make_float2(-div.r, -div.r);
          const float2 s2 = make_float2(s, s), mg = make_float2(kRintMagic, kRintMagic);
#pragma unroll
          for (int i = 0; i < NW; ++i) {
            const float2 t = __fadd2_rn(div_pair(bf16x2_to_float2(raw[i]), r2, nr2, s2), mg);
            c[2 * i] = __float_as_int(t.x) + off;
            c[2 * i + 1] = __float_as_int(t.y) + off;
          }
        } else {
#pragma unroll
          for (int i = 0; i < NW; ++i) {
            const float2 x = bf16x2_to_float2(raw[i]);
            c[2 * i] = __float_as_int(__fadd_rn(__fdiv_rn(x.x, s), kRintMagic)) + off;
            c[2 * i + 1] = __float_as_int(__fadd_rn(__fdiv_rn(x.y, s), kRintMagic)) + off;
          }
        }
#pragma unroll
        for (int i = 0; i < E; i += 4) rc.w[i >> 2] = pack_sat_s8x2(c[i + 1], c[i], pack_sat_s8x2(c[i + 3], c[i + 2], 0u));
      }
    }
  }
}

// Static-scale INT8 (one given scale per channel, or one per cache): code =
// clamp(rint(x / s), -127, 127), 0 where s <= 0 or s is NaN. sc[i] and rc_[i]
// (shared memory) are the scale of this lane's element i and its reciprocal
// RN(1/s), 0 when s is below 2^-100 (those take the IEEE division). x is first clamped to
// +-65536 s, which changes only quotients that saturate anyway and keeps the
// corrected quotient inside the range where its rint equals that of the IEEE
// quotient (tests/test_scale_division.py).
template <int D>
__device__ __forceinline__ void quantize_row_static(const uint32_t (&raw)[D / (2 * kRowLanes)],
                                                    const float* sc, const float* rc_,
                                                    RowCodes<D, KVQ_INT8_CHANNEL>& rc) {
  constexpr int E = D / kRowLanes;
  rc.zp = 0;
  rc.s = __float2bfloat16_rn(0.f);
#pragma unroll
  for (int i = 0; i < RowCodes<D, KVQ_INT8_CHANNEL>::WORDS; ++i) rc.w[i] = 0u;
  // the lane's scales and reciprocals as 16-byte reads (sc, rc_ are 64-byte aligned)
  float scv[E], rcv[E];
#pragma unroll
  for (int i = 0; i < E; i += 4) {
    const float4 a = *reinterpret_cast<const float4*>(sc + i);
    const float4 b = *reinterpret_cast<const float4*>(rc_ + i);
    scv[i] = a.x; scv[i + 1] = a.y; scv[i + 2] = a.z; scv[i + 3] = a.w;
    rcv[i] = b.x; rcv[i + 1] = b.y; rcv[i + 2] = b.z; rcv[i + 3] = b.w;
  }
  int c[E];
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const float x = (i & 1) ? bf16_hi(raw[i / 2]) : bf16_lo(raw[i / 2]);
    const float s = scv[i], r = rcv[i];
    c[i] = 0;
    if (s > 0.f) {
      const float lim = s * 65536.f;
      const float xc = fminf(fmaxf(x, -lim), lim);
      float q;
      if (r != 0.f) {
        const float q0 = __fmul_rn(xc, r);
        const float e = __fmaf_rn(q0, s, -xc);
        q = __fmaf_rn(-e, r, q0);
      } else {
        q = __fdiv_rn(xc, s);
      }
      // |q| <= 65536 (x clamped above): the rounding addition applies
      c[i] = min(kRintBits + 127, max(kRintBits - 127, __float_as_int(__fadd_rn(q, kRintMagic))));
    }
  }
#pragma unroll
  for (int i = 0; i < E; i += 4) rc.w[i >> 2] = pack_low_bytes(c[i], c[i + 1], c[i + 2], c[i + 3]);
}

// Bytes [p, e) of the 16-byte chunk at dst (16-byte aligned) from w, with the
// widest aligned stores the range allows: one 16-byte store for a whole chunk,
// else 8-, 4-, 2- and 1-byte pieces. Bytes outside [p, e) are not touched, so
// writers of disjoint byte ranges of one chunk never clobber each other.
__device__ __forceinline__ void store_bytes16(uint8_t* dst, const uint32_t (&w)[4], int p, int e) {
  if (p == 0 && e == 16) {
    *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    return;
  }
#pragma unroll
  for (int h8 = 0; h8 < 2; ++h8) {
    const int a8 = max(p, 8 * h8), b8 = min(e, 8 * h8 + 8);
    if (a8 >= b8) continue;
    if (a8 == 8 * h8 && b8 == 8 * h8 + 8) {
      *reinterpret_cast<uint2*>(dst + 8 * h8) = make_uint2(w[2 * h8], w[2 * h8 + 1]);
      continue;
    }
#pragma unroll
    for (int h4 = 0; h4 < 2; ++h4) {
      const int base4 = 8 * h8 + 4 * h4;
      const int a4 = max(a8, base4), b4 = min(b8, base4 + 4);
      if (a4 >= b4) continue;
      const uint32_t word = w[2 * h8 + h4];
      if (a4 == base4 && b4 == base4 + 4) {
        *reinterpret_cast<uint32_t*>(dst + base4) = word;
        continue;
      }
#pragma unroll
      for (int h2 = 0; h2 < 2; ++h2) {
        const int base2 = base4 + 2 * h2;
        const int a2 = max(a4, base2), b2 = min(b4, base2 + 2);
        if (a2 >= b2) continue;
        const uint32_t half = word >> (16 * h2);
        if (a2 == base2 && b2 == base2 + 2)
          *reinterpret_cast<uint16_t*>(dst + base2) = uint16_t(half);
        else
          dst[a2] = uint8_t(half >> (8 * (a2 - base2)));
      }
    }
  }
}

}  // namespace kvq
