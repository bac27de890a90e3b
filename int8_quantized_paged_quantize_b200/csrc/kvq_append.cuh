// Quantize-on-append: the kernel behind kvq_append and kvq_append_rope.
#pragma once

#include "kvq_quant.cuh"
#include "kvq_tc.cuh"

namespace kvq {

// Contiguous K and V rows [T][Hk][D].
template <int D>
struct PlainRows {
  const __nv_bfloat16* __restrict__ k;
  const __nv_bfloat16* __restrict__ v;
  const int64_t* __restrict__ slots;
  static constexpr bool kQuery = false;
  template <int FMT>
  static constexpr int ctas_per_sm() { return FMT == KVQ_INT8_CHANNEL ? 5 : 8; }
  // values d0 .. d0 + D/8 - 1 of the K (which = 0) or V row of token t, head h
  __device__ __forceinline__ void load(int64_t t, int which, int Hk, int h, int d0,
                                       uint32_t (&raw)[D / (2 * kRowLanes)]) const {
    load_row<D>((which ? v : k) + (t * Hk + h) * D + d0, raw);
  }
  __device__ __forceinline__ int64_t slot(int64_t t, int) const { return slots[t]; }
};

// One CTA of 8 warps per (16 consecutive input tokens, KV head). Warp w takes
// tokens 2w and 2w+1: its four lane groups quantize their K rows (lanes 0-15)
// and V rows (lanes 16-31) into shared memory in one pass. The input rows are
// requested before the slots arrive (a skipped token's row is read and
// dropped), so the loads overlap. The window is then written in page-sized
// pieces:
//   - the 16 tokens fill one page in order (the bulk / prefill case): the page
//     is written as whole 16-byte chunks, K in its chunk-major layout and V
//     transposed with byte permutes;
//   - otherwise each token writes its K chunks, and the tokens are grouped into
//     segments (runs of consecutive slots inside one page); a segment writes its
//     byte range of each transposed V chunk once, with the widest aligned
//     stores that range allows. A page continued from an offset (chunked
//     prefill) thus costs one partial chunk per channel, not one byte store per
//     token and channel.
// Where a row comes from is the template parameter ROWS: contiguous K and V
// (PlainRows), or strided ones with the rotary embedding applied to K
// (kvq_append_rope).
// Register use is capped at 32 so that 8 CTAs (64 warps) fit on an SM (a few
// bytes of spills for INT8 with its zero point cost less than 6 CTAs did); the
// static-scale format takes 48 (5 CTAs), its scales in shared memory.
template <int D, int FMT, class ROWS>
__global__ void __launch_bounds__(256, ROWS::template ctas_per_sm<FMT>())
append_kernel(const ROWS rows, int T, int Hk, int NB, uint8_t* __restrict__ kc,
              uint8_t* __restrict__ vc, __nv_bfloat16* __restrict__ ks, __nv_bfloat16* __restrict__ vs,
              int per_tensor) {
  using RC = RowCodes<D, FMT>;
  constexpr int E = RC::E, ELT = RC::ELT;
  constexpr int ROWB = D * ELT;                 // bytes of one token row
  constexpr int PADB = ROWB + 16;               // padded smem row (bank spread)
  constexpr int PAGEB = kBlockSize * ROWB;
  constexpr int NC = ROWB / 16;                 // 16-byte chunks of a K row
  constexpr int UC = ELT;                       // 16-byte V chunks per channel
  constexpr int TPC = 16 / ELT;                 // tokens per V chunk
  constexpr int MV = (FMT == KVQ_FP8_E4M3 || FMT == KVQ_FP8_E5M2) ? 1 : (FMT == KVQ_INT8_ASYM ? 2 : 0);
  __shared__ __align__(16) uint8_t kbuf[kBlockSize * PADB];
  __shared__ __align__(16) uint8_t vbuf[kBlockSize * PADB];
  __shared__ __nv_bfloat16 kmb[kBlockSize][2], vmb[kBlockSize][2];
  __shared__ int64_t sl[kBlockSize];
  __shared__ int seg_i0[kBlockSize], seg_len[kBlockSize], nseg, page_fast;
  // static scales of the head's K (0) and V (1) channels and their reciprocals
  __shared__ __align__(16) float sscale[FMT == KVQ_INT8_CHANNEL ? 2 * D : 4];
  __shared__ __align__(16) float srcp[FMT == KVQ_INT8_CHANNEL ? 2 * D : 4];

  // the decode kernel of the step may start its set-up now; it reads the
  // cache only after this grid has finished
  tc::grid_dep_launch_dependents();
  const int h = blockIdx.y;
  const int64_t tb = int64_t(blockIdx.x) * kBlockSize;
  const int n = int(min(int64_t(kBlockSize), int64_t(T) - tb));
  if constexpr (ROWS::kQuery) {
    if (h >= Hk) {                              // a CTA of the query's rows
      rows.query(tb, n, h - Hk);
      return;
    }
  }
  const int64_t nslots = int64_t(NB) * kBlockSize;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // lane group g = lane / 8: the K row (g = 0, 1) or the V row (g = 2, 3) of
  // token 2 warp + (g & 1); requested before the slots arrive
  const int which = lane >> 4;                  // 0: K row, 1: V row
  const int ti = 2 * warp + ((lane >> 3) & 1);  // token of the window
  const int d0 = (lane & (kRowLanes - 1)) * E;
  uint32_t raw[D / (2 * kRowLanes)];
#pragma unroll
  for (int e = 0; e < D / (2 * kRowLanes); ++e) raw[e] = 0u;
  if (ti < n) rows.load(tb + ti, which, Hk, h, d0, raw);
  if (threadIdx.x < kBlockSize) sl[threadIdx.x] = threadIdx.x < n ? rows.slot(tb + threadIdx.x, h) : -1;
  if constexpr (FMT == KVQ_INT8_CHANNEL) {
    for (int i = threadIdx.x; i < 2 * D; i += blockDim.x) {
      const float sv = __bfloat162float((i >= D ? vs : ks)[per_tensor ? 0 : h * D + i % D]);
      sscale[i] = sv;
      srcp[i] = sv >= 7.88860905e-31f ? __frcp_rn(sv) : 0.f;   // 2^-100
    }
  }
  __syncthreads();

  if (warp == 0) {
    const int64_t si = lane < kBlockSize ? sl[lane] : -1;
    const int64_t sp = (lane > 0 && lane < kBlockSize) ? sl[lane - 1] : -1;
    const int64_t s0 = sl[0];
    // whole page in order: slot i = s0 + i for all 16 tokens, s0 page-aligned
    const bool inpage = lane >= kBlockSize || (si == s0 + lane && s0 >= 0 && s0 % kBlockSize == 0 &&
                                               s0 < nslots && n == kBlockSize);
    const bool fast = __all_sync(0xffffffffu, inpage);
    // segments: a token starts one unless it continues the previous token's
    // slot inside the same page
    const bool valid = si >= 0 && si < nslots;
    const bool start = valid && !(sp >= 0 && sp < nslots && si == sp + 1 && si % kBlockSize != 0);
    const unsigned vmask = __ballot_sync(0xffffffffu, valid);
    const unsigned smask = __ballot_sync(0xffffffffu, start);
    if (start) {
      const int idx = __popc(smask & ((1u << lane) - 1u));
      // the run ends at the next start or at the first invalid token
      const unsigned stop = (smask | ~vmask) & ~((2u << lane) - 1u);
      seg_i0[idx] = lane;
      seg_len[idx] = (stop ? __ffs(stop) - 1 : 32) - lane;
    }
    if (lane == 0) {
      nseg = __popc(smask);
      page_fast = fast;
    }
  }

  {
    // every lane quantizes (the reductions span the warp); only real rows store
    RC rc;
    if constexpr (FMT == KVQ_INT8_CHANNEL)
      quantize_row_static<D>(raw, sscale + which * D + d0, srcp + which * D + d0, rc);
    else quantize_row<D, FMT>(raw, rc);
    const int64_t slot = ti < n ? sl[ti] : -1;
    if (slot >= nslots) {
      if ((lane & (kRowLanes - 1)) == 0) flag_error(KVQ_DEVERR_SLOT);
    } else if (slot >= 0) {
      uint8_t* dst = (which ? vbuf : kbuf) + ti * PADB + d0 * ELT;
#pragma unroll
      for (int c = 0; c < E * ELT / 16; ++c)
        reinterpret_cast<uint4*>(dst)[c] = make_uint4(rc.w[4 * c], rc.w[4 * c + 1], rc.w[4 * c + 2], rc.w[4 * c + 3]);
      if constexpr (E * ELT == 8) *reinterpret_cast<uint2*>(dst) = make_uint2(rc.w[0], rc.w[1]);
      if ((lane & (kRowLanes - 1)) == 0) {
        (which ? vmb : kmb)[ti][0] = rc.s;
        (which ? vmb : kmb)[ti][1] = __int2bfloat16_rn(rc.zp);
      }
    }
  }
  __syncthreads();

  if (page_fast) {                                   // uniform over the CTA
    const int64_t page = (sl[0] / kBlockSize) * Hk + h;
    uint8_t* kp = kc + page * PAGEB;
    uint8_t* vp = vc + page * PAGEB;
    // items [0, KN): K chunk j = (token group t/8, c, t%8) <- bytes [16c, 16c+16)
    // of token t's row. Items [KN, KN + VN): a V piece, from 32-bit words of
    // the staged rows transposed with byte permutes.
    constexpr int KN = PAGEB / 16;
    constexpr int VN = ELT == 1 ? 2 * (D / 4) : 2 * (D / 2);
    for (int j = threadIdx.x; j < KN + VN; j += blockDim.x) {
      if (j < KN) {
        const int c = (j >> 3) % NC, t = (j / (8 * NC)) * 8 + (j & 7);
        *reinterpret_cast<uint4*>(kp + j * 16) = *reinterpret_cast<const uint4*>(kbuf + t * PADB + c * 16);
        continue;
      }
      const int jv = j - KN;
      if constexpr (ELT == 1) {
        // channels 4c..4c+3, tokens 8h..8h+7: two 4x4 byte transposes; the
        // result is the low or high 8 bytes of four channels' chunks
        const int c = jv % (D / 4), hh = jv / (D / 4);
        uint32_t o[4][2];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const int t0 = 8 * hh + 4 * g;
          const uint32_t r0 = *reinterpret_cast<const uint32_t*>(vbuf + (t0 + 0) * PADB + 4 * c);
          const uint32_t r1 = *reinterpret_cast<const uint32_t*>(vbuf + (t0 + 1) * PADB + 4 * c);
          const uint32_t r2 = *reinterpret_cast<const uint32_t*>(vbuf + (t0 + 2) * PADB + 4 * c);
          const uint32_t r3 = *reinterpret_cast<const uint32_t*>(vbuf + (t0 + 3) * PADB + 4 * c);
          const uint32_t a01 = __byte_perm(r0, r1, 0x5140), a23 = __byte_perm(r2, r3, 0x5140);
          const uint32_t b01 = __byte_perm(r0, r1, 0x7362), b23 = __byte_perm(r2, r3, 0x7362);
          o[0][g] = __byte_perm(a01, a23, 0x5410);
          o[1][g] = __byte_perm(a01, a23, 0x7632);
          o[2][g] = __byte_perm(b01, b23, 0x5410);
          o[3][g] = __byte_perm(b01, b23, 0x7632);
        }
#pragma unroll
        for (int m = 0; m < 4; ++m)
          *reinterpret_cast<uint2*>(vp + (4 * c + m) * 16 + 8 * hh) = make_uint2(o[m][0], o[m][1]);
      } else {
        // channels 2c, 2c+1, tokens 8u..8u+7: 2x2 transposes of 16-bit halves
        const int c = jv % (D / 2), u = jv / (D / 2);
        uint32_t lo4[4], hi4[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int t0 = 8 * u + 2 * q;
          const uint32_t w0 = *reinterpret_cast<const uint32_t*>(vbuf + t0 * PADB + 4 * c);
          const uint32_t w1 = *reinterpret_cast<const uint32_t*>(vbuf + (t0 + 1) * PADB + 4 * c);
          lo4[q] = __byte_perm(w0, w1, 0x5410);
          hi4[q] = __byte_perm(w0, w1, 0x7632);
        }
        *reinterpret_cast<uint4*>(vp + (u * D + 2 * c) * 16) = make_uint4(lo4[0], lo4[1], lo4[2], lo4[3]);
        *reinterpret_cast<uint4*>(vp + (u * D + 2 * c + 1) * 16) = make_uint4(hi4[0], hi4[1], hi4[2], hi4[3]);
      }
    }
  } else {
    // K: whole 16-byte chunks of each token's row
    for (int j = threadIdx.x; j < n * NC; j += blockDim.x) {
      const int i = j / NC, c = j % NC;
      const int64_t slot = sl[i];
      if (slot < 0 || slot >= nslots) continue;
      const int64_t page = (slot / kBlockSize) * Hk + h;
      *reinterpret_cast<uint4*>(kc + page * PAGEB + k_chunk_offset<ROWB>(c, int(slot % kBlockSize))) =
          *reinterpret_cast<const uint4*>(kbuf + i * PADB + c * 16);
    }
    // V: per (segment, channel d, chunk u) the segment's bytes of that chunk
    const int ns = nseg;
    for (int j = threadIdx.x; j < ns * D * UC; j += blockDim.x) {
      const int sg = j / (D * UC), d = (j / UC) % D, u = j % UC;
      const int i0 = seg_i0[sg], len = seg_len[sg];
      const int64_t slot0 = sl[i0];
      const int o0 = int(slot0 % kBlockSize);
      // token offsets of the segment inside chunk u
      const int ta = max(o0, u * TPC), tz = min(o0 + len, (u + 1) * TPC);
      if (ta >= tz) continue;
      uint8_t* chunk = vc + ((slot0 / kBlockSize) * Hk + h) * PAGEB + (u * D + d) * 16;
      if (tz - ta == 1) {                            // one token: one element
        const int i = i0 + (ta - o0), b = (ta - u * TPC) * ELT;
        if constexpr (ELT == 1) chunk[b] = vbuf[i * PADB + d];
        else *reinterpret_cast<uint16_t*>(chunk + b) = *reinterpret_cast<const uint16_t*>(vbuf + i * PADB + 2 * d);
        continue;
      }
      uint32_t wv[4];
#pragma unroll
      for (int q4 = 0; q4 < 4; ++q4) {
        uint32_t word = 0;
        const int w0 = u * TPC + q4 * (4 / ELT);      // first token offset of this word
        if (w0 + 4 / ELT > ta && w0 < tz) {
#pragma unroll
          for (int bb = 0; bb < 4 / ELT; ++bb) {
            const int t = w0 + bb;
            if (t >= ta && t < tz) {
              const int i = i0 + (t - o0);
              if constexpr (ELT == 1)
                word |= uint32_t(vbuf[i * PADB + d]) << (8 * bb);
              else
                word |= uint32_t(*reinterpret_cast<const uint16_t*>(vbuf + i * PADB + 2 * d)) << (16 * bb);
            }
          }
        }
        wv[q4] = word;
      }
      store_bytes16(chunk, wv, (ta - u * TPC) * ELT, (tz - u * TPC) * ELT);
    }
  }
  // metadata: one thread per (token, K or V)
  if (MV > 0 && threadIdx.x < 2 * kBlockSize) {
    const int t = threadIdx.x & 15;
    const int64_t slot = sl[t];
    if (t < n && slot >= 0 && slot < nslots) {
      const bool isv = threadIdx.x >= kBlockSize;
      __nv_bfloat16* meta = isv ? vs : ks;
      const __nv_bfloat16 (*mb)[2] = isv ? vmb : kmb;
      const int64_t row = ((slot / kBlockSize) * Hk + h) * kBlockSize + slot % kBlockSize;
      if (MV == 1) {
        meta[row] = mb[t][0];
      } else {
        *reinterpret_cast<__nv_bfloat162*>(meta + row * 2) = __halves2bfloat162(mb[t][0], mb[t][1]);
      }
    }
  }
}

}  // namespace kvq
