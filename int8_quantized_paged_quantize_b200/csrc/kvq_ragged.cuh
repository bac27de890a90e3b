// Attention of ragged chunks of new tokens over the paged quantized cache
// (kvq_ragged_attn): sequence b brings n_b new tokens, the last n_b of its
// cached context, and row i of them, at position p = ctx_b - n_b + i, attends
// the cached tokens t <= p (with a window w: p - w < t <= p):
//   out = sum_t softmax_t(sm_scale q . K_t) V_t, K and V as the codes stand for.
//
// A flash-attention loop on the 5th-generation tensor cores. A CTA takes a
// block of up to 256 query rows of one (sequence, KV head) (rows of the G query
// heads that share the head, token by token) and walks the cached tokens in
// steps of 64:
//   S[128 x 64] = Q . K^T      Q in shared memory, K codes expanded to f16
//   P = 2^(S f - m)            FP32 registers, one row a thread
//   O[128 x D] += P . V        P as bf16 parts in tensor memory, V codes as bf16
// The query is exact in f16 after a power-of-two scaling of its row (the elements
// below 2^-29 of the largest aside), the 8-bit codes of K (INT8: less the zero point)
// are exact in f16 and those of V in bf16, and the products accumulate in FP32. A BF16
// cache is multiplied as it is stored. Running maximum, sum and O are FP32.
// The scales of the tokens are applied in FP32: K's to the scores, V's to the weights.
// A weight is rounded to 16 bits, as two bf16 parts, for BF16 output, which is itself
// rounded to 8, and to 24, as three, for FP32 output (HP). bf16 has the range of FP32, so a
// weight keeps its bits however far below the largest one it lies. What was less:
//   f16 weights (two parts for FP32 output) end at 2^-24: thousands of tokens 12 nats
//     below a token without a value came out 6e-3 (FP32 output 4e-3) off, and 20 nats
//     below it they were lost;
//   K and V expanded to f16 code * scale, with weights of 11 bits, spare the softmax
//     warps two factors a score from shared memory (1,024 new tokens at 4,096, 64/8 heads:
//     INT8 202 us, 245 now; FP8 170, 219 now), but 13% of the values came out rounded
//     otherwise than the exact ones (now 0.2%);
//   one bf16 part over a BF16 cache: 145 us, 175 now, 40% of the values.
// With static INT8 scales the K scale of each channel multiplies the query, which is kept
// as two f16 parts, and the V scale the finished channel. (One part: 4% to 5% of the values
// at D = 64 rounded otherwise; the second takes the place of slot B's rows, so a block has
// 128: 1,024 new tokens at 4,096, 64/8 heads, 218 us then, 310 to 330 now.)
//
// The two halves of the CTA work on different products at the same time, so
// that one's exponentials cover the other's matrix products: slot A and slot B
// have their own S, P and O in tensor memory and four softmax warps each. A
// block of more than 128 rows puts its first 128 rows in slot A and the others
// in slot B, and every step runs in both (the codes are expanded once for 256
// rows). A block of at most 128 rows runs its even steps in slot A and its odd
// ones in slot B, over the same rows, and joins the two at its end. A block of at most 16
// rows (a token or two of a sequence) has its rows in each of the four warps of a
// slot, every warp with 16 of a step's tokens: a row's exponentials are spread
// over four threads, and eight softmaxes join.
//
// The online softmax moves a row's reference m only when the largest weight a
// step could give, the largest score times 2^eV, passes 2^8 relative to it (O is
// then rescaled in tensor memory).
//
// Work split: see kvq_ragged_plan.h. A block that lies in one CTA's share is
// finished there; the first and the last of a share may be pieces, whose
// (m, l, O) go to the workspace (two places a CTA) for ragged_merge_kernel.
//
// 16 warps per CTA, one CTA per SM:
//   0       producer: 1-D bulk copies of 4 K and 4 V pages a step into a ring
//           of raw stages, the scales beside them by plain loads
//   1       tensor memory, and one thread that issues the products
//   2       walks the CTA's share of the work list, hands the pieces to the other
//           roles through a ring and writes the rows that attend nothing; 3: none
//   4..7    softmax of slot A (thread = row = TMEM lane), 8..11 of slot B
//   12..15  converters: codes of a step to f16 (K) and bf16 (V; BF16 cache: none), V of
//           tokens past the end zeroed, the scales as FP32 column factors
// The registers are shared out by role: 168 a thread for the softmax warps
// (64 scores and the weights made of them), 88 for the others.
//
// A V row that holds a NaN or an infinity (with a per-token scale: whose scale is
// one) reaches the rows that attend it, in its channels or in all of them, and
// no other row: in a step that some row does not attend as a whole its V is
// zeroed in the operand, where 0 x NaN would reach every row, and the rows that
// do attend it get a NaN sum.
//
// Every wait is bounded, as in the other attention kernels: on expiry the CTA
// stops issuing, drains, writes NaN to every row of its share and returns.
#pragma once

#include "kvq_common.cuh"
#include "kvq_prefill.cuh"
#include "kvq_ragged_plan.h"

namespace kvq {

constexpr int kRgRing = 4;                     // pieces handed ahead
constexpr int kRgGroup = 4;                    // steps of a group of the producer (4 pages a step, a lane each)
constexpr int kRgNarrow = 16;                  // rows that every warp of a slot has a copy of

template <int D, int FMT, bool HP>
struct RgCfg {
  static constexpr bool BF = FMT == KVQ_BF16;
  static constexpr bool F8 = FMT == KVQ_FP8_E4M3 || FMT == KVQ_FP8_E5M2;
  static constexpr bool SI = FMT == KVQ_INT8_CHANNEL;            // static per channel / per tensor
  static constexpr bool ZP = FMT == KVQ_INT8_ASYM;
  static constexpr int E = BF ? 2 : 1;
  static constexpr int PAGE = kBlockSize * D * E;                // raw page bytes
  static constexpr int MV = F8 ? 1 : (ZP ? 2 : 0);
  static constexpr int METAB = kBlockSize * MV * 2;              // raw scale bytes of a page
  static constexpr int ST = kRgStep, PPS = kRgStep / kBlockSize; // tokens, pages per step
  static constexpr int QP = SI ? 2 : 1;                          // query parts
  // weight parts. The third one has the columns of the slot's S, which its softmax warps have
  // read by then; a slot's next scores are issued behind its values.
  static constexpr int PP = HP ? 3 : 2;
  // Steps of a slot that the tensor cores add up, before its O is added to FP32 sums in the
  // workspace: they round their sums down, so that what is lost would grow with the context
  // (0.1% to 0.2% of a value at 524,288 tokens).
  // BF16 output, INT8, 2 x 2,048 rows at 8,192: 1,613 us with 128 steps, 1,653 with 64, 1,721
  // with 32; of the values 0.22%, 0.11%, 0.05% are rounded otherwise than by the plain form.
  // FP32 output, FP8, 1,024 rows at 4,096: 355 us with 8 steps, 367 with 6, 392 with 4 (BF16
  // cache: 289, 307, 330); rows that see 8,192 tokens are off by 0.9e-6 with 6 (BF16 cache
  // 0.9e-6 with 4), and with the parts in the other order by 1.5e-6, 1.2e-6, 0.8e-6 with 8, 6, 4
  // (BF16 cache 1.9e-6, 1.5e-6, 1.1e-6).
  // A narrow block's warps have weights for 16 of a step's tokens each, a quarter of the
  // additions.
  static constexpr int FLUSH = !HP ? 64 : BF ? 4 : 6;
  static __device__ __forceinline__ int flush(int rows) { return rows <= kRgNarrow ? 4 * FLUSH : FLUSH; }
  static constexpr int RPB = QP == 2 ? 128 : 256;     // rows per block
  static constexpr int NRAW = BF ? 4 : 3;                        // raw stages (steps)
  static constexpr int NC = BF ? NRAW : 3;                       // operand stages
  static constexpr int CPAGE = kBlockSize * D * 2;               // page at 16 bits
  static constexpr bool COLS = MV > 0;                           // scores and weights scaled token by token
  static constexpr int CMETA = (COLS ? 2 * ST * 4 : 0) + 16;     // K and V scale per token; eV, 2^-eV of the step
  static constexpr int CSTAGE = (BF ? 0 : 2 * PPS * CPAGE) + CMETA;
  static constexpr int QBYTES = 128 * D * 2;
  static constexpr uint32_t K_LBO = 128, K_SBO = 16 * D;
  static constexpr uint32_t V_LBO = 16 * D, V_SBO = 128;
  static constexpr uint32_t Q_LBO = 128, Q_SBO = 16 * D;
  // tensor memory: O of slots A and B, then S and P of each
  static constexpr int COL_O = 0, COL_S = 2 * D, COL_P = 2 * D + 128, TMEM_COLS = 512;
  static constexpr int RSTAGE = 2 * PPS * PAGE;                  // K pages, V pages
  static constexpr int RMETA = 2 * PPS * METAB;
  static constexpr int OFF_R = 0;
  static constexpr int OFF_Q = OFF_R + NRAW * RSTAGE;
  static constexpr int OFF_C = OFF_Q + 2 * QBYTES;
  static constexpr int OFF_RM = (OFF_C + NC * CSTAGE + 15) / 16 * 16;
  static constexpr int OFF_X = OFF_RM + NRAW * RMETA;            // float [16][128]: joining the slots
  static constexpr int OFF_XS = OFF_X + 16 * 128 * 4;            // float2 [128]: m, l of slot B
  static constexpr int OFF_BAR = OFF_XS + 128 * 8;
  static constexpr int NBAR = 2 * NRAW + 2 * NC + 8 + 2 + 2 * kRgRing;
  static constexpr int OFF_MASK = (OFF_BAR + 8 * NBAR + 15) / 16 * 16;   // page masks [NRAW], [NC], then [NC][12]
  static constexpr int OFF_RED = OFF_MASK + 16 * ((NRAW + NC + 3) / 4) + 48 * NC;
  static constexpr int OFF_MISC = OFF_RED + 128;
  static constexpr int OFF_ITEM = OFF_MISC + 48;                 // RgItem [kRgRing]
  static constexpr int USED = OFF_ITEM + kRgRing * 64;
  // one CTA per SM (it takes all tensor memory): never less than half of an SM's shared memory
  static constexpr int SMEM = USED < 118 * 1024 ? 118 * 1024 : USED;
  static_assert(OFF_C % 128 == 0 && OFF_Q % 128 == 0 && CSTAGE % 16 == 0 && OFF_BAR % 8 == 0, "alignment");
  static_assert(SMEM <= 227 * 1024, "shared memory");
};

// A piece as the roles see it: the block's sequence, head and rows, its steps.
struct __align__(16) RgItem {
  int b, h, k, rows;                           // rows 0: no more pieces
  int row0, n, ctx, first;                     // first: token step of the block's step 0
  int lo, hi, count, pad;
};

// What describes the batch (device memory) and the shape.
struct RgBatch {
  const int32_t* cu;
  const int32_t* ctx_lens;
  int B, T, Hk, W, max_ctx;
  // null, or (a decode step) the sequences with one new token are the decode kernels':
  // their context (0 for the others), output row (-1) and query row, for these to read
  int32_t *ctx1, *row1;
  uint4* q1;
  RgShape p;

  // sequence b: its new tokens and context; a range or a context that is not
  // legal counts as empty
  __device__ __forceinline__ RgSeq seq(int b, int* row0, unsigned* bad, bool all = false) const {
    const int c0 = cu[b], c1 = cu[b + 1], x = ctx_lens[b];
    RgSeq s;
    s.n = c1 - c0;
    s.ctx = x;
    unsigned f = 0;
    if (c0 < 0 || c1 < c0 || c1 > T) {
      f = KVQ_DEVERR_RANGE;
      s.n = 0;
    }
    if (x < 0 || x > max_ctx || int64_t(x) > int64_t(W) * kBlockSize) {
      f |= KVQ_DEVERR_CONTEXT;
      s.ctx = 0;
    }
    if (!all && ctx1 && s.n == 1) s.n = 0;
    *row0 = c0;
    if (bad) *bad = f;
    return s;
  }
};

// Cursor over the pieces of one CTA's share.
struct RgWalk {
  RgSeq s;
  int b, h, k, nb, row0;
  long long pos, start, end;
  int first, count, lo, hi, rows;
  bool done;

  __device__ __forceinline__ void load(const RgBatch& a) {          // the next sequence with rows, from b on
    nb = 0;
    while (b < a.B) {
      s = a.seq(b, &row0, nullptr);
      nb = rg_blocks(s, a.p);
      if (nb > 0) return;
      ++b;
    }
  }
  __device__ __forceinline__ int weight() const { return rows > 128 ? 2 : 1; }
  __device__ __forceinline__ bool item(const RgBatch& a) {
    rg_block(s, k, a.p, &first, &count);
    rows = rg_rows(s, k, a.p);
    return rg_piece(pos, count, weight(), start, end, &lo, &hi);
  }
  __device__ __forceinline__ void step(const RgBatch& a) {
    pos += kRgPiece + (long long)weight() * count;
    if (++k < nb) return;
    k = 0;
    if (++h < a.Hk) return;
    h = 0;
    ++b;
    load(a);
  }
  __device__ __forceinline__ void settle(const RgBatch& a) {
    while (true) {
      if (pos >= end || nb == 0) {
        done = true;
        return;
      }
      if (item(a)) {
        done = false;
        return;
      }
      step(a);
    }
  }
  // P0: cost per KV head of the sequences before b0
  __device__ __forceinline__ void init(const RgBatch& a, int b0, long long P0, long long start_, long long end_) {
    b = b0;
    start = start_;
    end = end_;
    load(a);
    const long long L = rg_cost(s, a.p);
    long long off = start - P0 * a.Hk;
    for (h = 0; off >= L; ++h) off -= L;
    k = nb > 1 ? rg_find(s, off, a.p) : 0;
    pos = start - off + (k > 0 ? rg_prefix(s, k, a.p) : 0);
    settle(a);
  }
  __device__ __forceinline__ void next(const RgBatch& a) {
    step(a);
    settle(a);
  }
  __device__ __forceinline__ bool whole() const { return lo == 0 && hi == count; }
};

// A piece's place in the workspace: what the joining kernel has to know.
struct RgPiece {
  int valid, last, row0, n, h, k, pad0, pad1;
};
static_assert(sizeof(RgPiece) == 32, "layout");

__device__ __forceinline__ void rg_record(RgPiece* p, bool last, int row0, int n, int h, int k) {
  RgPiece r;
  r.valid = 1;
  r.last = last;
  r.row0 = row0;
  r.n = n;
  r.h = h;
  r.k = k;
  r.pad0 = r.pad1 = 0;
  *p = r;
}

// 1-D bulk copy global -> shared. No L2 hint: the pages of a sequence are read
// again for its other blocks.
__device__ __forceinline__ void bulk_g2s_keep(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          tc::smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(tc::smem_u32(bar))
      : "memory");
}

// 32 lanes x 32 columns.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

// 32 lanes x 8 columns.
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// Shared memory by its 32-bit address.
__device__ __forceinline__ uint4 lds_u4(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ void sts_u4(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ uint32_t rg_pack(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t f16x2_to_bf16x2(uint32_t w) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  return rg_pack(f.x, f.y);
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// One arrival for the whole warp, after what its lanes did.
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
  __syncwarp();
  // predicated, not branched around
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.eq.s32 p, %1, 0;\n\t"
      "@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}\n" ::"r"(tc::smem_u32(bar)),
      "r"(lane)
      : "memory");
}

// A product must cost the thread that issues it few instructions (the 64-bit
// descriptors built anew for each took it a thousand cycles a step). The
// high words of the shared-memory descriptors (stride, version; see sdesc_plain) are
// constants, the low words (address / 16, leading offset) advance by additions.
template <uint32_t SBO>
__host__ __device__ constexpr uint32_t rg_desc_hi() { return (SBO >> 4) | (1u << 14); }
template <uint32_t LBO>
__device__ __forceinline__ uint32_t rg_desc_lo(uint32_t saddr) { return ((saddr & 0x3FFFFu) >> 4) | ((LBO >> 4) << 16); }
template <uint32_t AHI, uint32_t BHI>
__device__ __forceinline__ void rg_mma_ss(uint32_t d, uint32_t alo, uint32_t blo, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %6};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}\n" ::"r"(d),
      "r"(alo), "r"(blo), "r"(idesc), "r"(acc), "n"(AHI), "n"(BHI)
      : "memory");
}
template <uint32_t BHI>
__device__ __forceinline__ void rg_mma_ts(uint32_t d, uint32_t a, uint32_t blo, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 b, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}\n" ::"r"(d),
      "r"(a), "r"(blo), "r"(idesc), "r"(acc), "n"(BHI)
      : "memory");
}

__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(e));
  return e != 0u;
}

// Four int8 codes less a zero point as f16 (exact): 1024 + (c + 128) by a byte
// permute, minus z = 1152 + zero point, an integer of [1024, 1279]; z0 for codes
// 0 and 1, z1 for 2 and 3.
__device__ __forceinline__ void s8x4_less(uint32_t w, uint32_t z0, uint32_t z1, uint32_t& lo, uint32_t& hi) {
  const uint32_t x = w ^ 0x80808080u;
  const uint32_t p0 = __byte_perm(x, 0x64646464u, 0x4140), p1 = __byte_perm(x, 0x64646464u, 0x4342);
  const __half2 h0 = __hsub2(*reinterpret_cast<const __half2*>(&p0), *reinterpret_cast<const __half2*>(&z0));
  const __half2 h1 = __hsub2(*reinterpret_cast<const __half2*>(&p1), *reinterpret_cast<const __half2*>(&z1));
  lo = *reinterpret_cast<const uint32_t*>(&h0);
  hi = *reinterpret_cast<const uint32_t*>(&h1);
}
// 16 codes: the same zero point for all, or one for each.
__device__ __forceinline__ void codes16_less(const uint4 c, uint32_t z, uint4& o0, uint4& o1) {
  s8x4_less(c.x, z, z, o0.x, o0.y);
  s8x4_less(c.y, z, z, o0.z, o0.w);
  s8x4_less(c.z, z, z, o1.x, o1.y);
  s8x4_less(c.w, z, z, o1.z, o1.w);
}
__device__ __forceinline__ void codes16_less_pairs(const uint4 c, const uint32_t* z, uint4& o0, uint4& o1) {
  s8x4_less(c.x, z[0], z[1], o0.x, o0.y);
  s8x4_less(c.y, z[2], z[3], o0.z, o0.w);
  s8x4_less(c.z, z[4], z[5], o1.x, o1.y);
  s8x4_less(c.w, z[6], z[7], o1.z, o1.w);
}

constexpr int kRgThreads = 512;
constexpr int kRgRegs = 128;                   // registers a thread at launch: 168 + 168 + 88 + 88 = 4 x 128

template <int D, int FMT, bool HP>
__global__ void __launch_bounds__(kRgThreads, 1) ragged_mma_kernel(
    const __nv_bfloat16* __restrict__ q, int64_t q_stride, const uint8_t* __restrict__ kc,
    const uint8_t* __restrict__ vc, const __nv_bfloat16* __restrict__ ks,
    const __nv_bfloat16* __restrict__ vs, const int32_t* __restrict__ tables, const RgBatch bt, int NB,
    float qk_scale, int per_tensor, long long wait_limit, void* __restrict__ out_,
    float* __restrict__ part_o, float* __restrict__ part_ml, RgPiece* __restrict__ pieces, int rows_cap,
    float* __restrict__ sums) {
  using C = RgCfg<D, FMT, HP>;
  using namespace tc;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int NWARPS = kRgThreads / 32;

  uint8_t* raw = smem + C::OFF_R;
  uint8_t* rmeta = smem + C::OFF_RM;
  uint8_t* cst = smem + C::OFF_C;
  uint8_t* qop = smem + C::OFF_Q;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* rfull = bars;                     // [NRAW] producer -> converters
  uint64_t* rfree = rfull + C::NRAW;          // [NRAW]
  uint64_t* cfull = rfree + C::NRAW;          // [NC] converters -> MMA, softmax
  uint64_t* cfree = cfull + C::NC;            // [NC] the step's products have completed
  uint64_t* sfull = cfree + C::NC;            // [2] S of a slot in tensor memory
  uint64_t* sfree = sfull + 2;                // [2] S read by the slot's softmax warps
  uint64_t* pready = sfree + 2;               // [2] P of a slot in tensor memory
  uint64_t* pvdone = pready + 2;              // [2] the slot's last PV product has completed
  uint64_t* qready = pvdone + 2;              // the query operand of the next piece
  uint64_t* drain = qready + 1;
  uint64_t* pfull = drain + 1;                // [kRgRing] a piece is in the ring
  uint64_t* pfree = pfull + kRgRing;          // [kRgRing] every role has read it
  RgItem* items = reinterpret_cast<RgItem*>(smem + C::OFF_ITEM);
  volatile uint32_t* rmask = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_MASK);
  // per operand stage, as each converter warp saw them: {whether some page is
  // missing or some V is not finite}, {not-finite V tokens 0..31}, {.. 32..63}
  volatile uint32_t* cpages = rmask + C::NRAW;   // [NC] valid pages of an operand stage
  uint4* cmask = reinterpret_cast<uint4*>(smem + C::OFF_MASK + 16 * ((C::NRAW + C::NC + 3) / 4));
  long long* red64 = reinterpret_cast<long long*>(smem + C::OFF_RED);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  int* misci = reinterpret_cast<int*>(smem + C::OFF_MISC + 8);
  long long* miscll = reinterpret_cast<long long*>(smem + C::OFF_MISC + 16);

  // ------------------------------------------------------------ set-up
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::NRAW; ++s) {
      mbar_init(rfull + s, 1);
      mbar_init(rfree + s, C::BF ? 1 : 4);
    }
    for (int j = 0; j < C::NC; ++j) {
      mbar_init(cfull + j, 4);
      mbar_init(cfree + j, 1);
    }
    for (int j = 0; j < 2; ++j) {
      mbar_init(sfull + j, 1);
      mbar_init(sfree + j, 4);
      mbar_init(pready + j, 4);
      mbar_init(pvdone + j, 1);
    }
    mbar_init(qready, 8);
    mbar_init(drain, 1);
    for (int j = 0; j < kRgRing; ++j) {
      mbar_init(pfull + j, 1);
      mbar_init(pfree + j, 14);                // producer, MMA, 8 softmax and 4 converter warps
    }
    for (int j = 0; j < 3 * C::NC; ++j) cmask[j] = make_uint4(0, 0, 0, 0);
    *abort_flag = 0;
    misci[0] = -1;
    mbar_init_fence();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // every argument in device memory is read, and the workspace written, after
  // the kernel ahead on the stream has finished
  grid_dep_wait();
  grid_dep_launch_dependents();

  if (bt.ctx1) {
    const int n16 = (bt.Hk << bt.p.g_log) * D / 8;         // 16-byte pieces of a query row
    for (int b = blockIdx.x; b < bt.B; b += gridDim.x) {
      int row0;
      const RgSeq sq = bt.seq(b, &row0, nullptr, true);
      const bool one = sq.n == 1;
      if (threadIdx.x == 0) {
        bt.ctx1[b] = one ? sq.ctx : 0;
        bt.row1[b] = one ? row0 : -1;
      }
      const uint4* src = reinterpret_cast<const uint4*>(q + int64_t(row0) * q_stride);
      for (int i = threadIdx.x; one && i < n16; i += kRgThreads) bt.q1[int64_t(b) * n16 + i] = src[i];
    }
  }

  // ------------------------------------------------------------ the share
  // Each thread has one sequence (or, in rounds, every 512th): its cost, the
  // sum before it, and with that whether the share begins in it.
  long long T = 0;                             // cost per KV head of the whole list
  long long mine = 0, before = 0;              // of this thread's sequence in the last round
  if (threadIdx.x < 2) pieces[2 * blockIdx.x + threadIdx.x].valid = 0;
  auto round = [&](int base, bool check) {
    const int bb = base + threadIdx.x;
    mine = 0;
    if (bb < bt.B) {
      int row0;
      unsigned bad;
      const RgSeq s = bt.seq(bb, &row0, &bad);
      if (check && bad && blockIdx.x == 0) flag_error(bad);
      mine = rg_cost(s, bt.p);
    }
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) red64[warp] = incl;
    __syncthreads();
    before = T + incl - mine;
#pragma unroll
    for (int w = 0; w < NWARPS; ++w) {
      const long long x = red64[w];
      before += w < warp ? x : 0;
      T += x;
    }
    __syncthreads();
  };
  for (int base = 0; base < bt.B; base += kRgThreads) round(base, true);
  const long long all = T * bt.Hk;
  const long long N = ll_min((long long)gridDim.x, ll_max(1, all / kRgMinShare));
  if (all == 0 || blockIdx.x >= N) {           // uniform for the CTA
    if (warp == 1) tmem_dealloc(tmem, C::TMEM_COLS);
    return;
  }
  const long long start = (blockIdx.x * all) / N, end = ((blockIdx.x + 1) * all) / N;
  if (bt.B > kRgThreads) T = 0;
  for (int base = 0; base < bt.B; base += kRgThreads) {
    if (bt.B > kRgThreads) round(base, false);
    if (mine > 0 && before * bt.Hk <= start && start < (before + mine) * bt.Hk) {
      misci[0] = base + threadIdx.x;
      miscll[0] = before;
    }
  }
  __syncthreads();

  // piece i of the share; false when there is none (or the kernel gave up). By
  // one lane, or by a whole warp (`whole`).
  auto fetch = [&](int i, RgItem& it, bool whole) -> bool {
    const int s = i % kRgRing;
    bool got = mbar_wait(pfull + s, (i / kRgRing) & 1, abort_flag, wait_limit);
    if (whole) got = __all_sync(0xffffffffu, got);
    if (!got) return false;
    const uint32_t a = smem_u32(items + s);
    const uint4 x = lds_u4(a), y = lds_u4(a + 16), z = lds_u4(a + 32);
    it.b = int(x.x); it.h = int(x.y); it.k = int(x.z); it.rows = int(x.w);
    it.row0 = int(y.x); it.n = int(y.y); it.ctx = int(y.z); it.first = int(y.w);
    it.lo = int(z.x); it.hi = int(z.y); it.count = int(z.z);
    if (whole) __syncwarp();
    if (!whole || lane == 0) mbar_arrive(pfree + s);
    return it.rows > 0;
  };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == 0) {
      // ---------------------------------------------------------- producer
      // Steps go in groups of kRgGroup: a lane holds the block id of one page of a group, two
      // groups ahead of the copies. The scales of a step are loaded a step ahead. (Pages
      // asked into L2 a group ahead cost more than they gave: decode of 64 sequences, FP8,
      // 298 against 262 us.)
      constexpr int CPP = C::METAB > 0 ? C::METAB / 16 : 1;    // 16-byte scale chunks per page
      const int sp = lane / CPP, sc = lane % CPP;
      RgItem it;
      int np = 0, i0 = 0;
      bool more = true;
      struct Group {
        int id, h, n, np;                      // this lane's block id, head, steps (0: no more), pages
      };
      auto next_item = [&]() {
        more = fetch(np++, it, true);
        i0 = it.lo;
      };
      auto next_group = [&]() -> Group {
        Group g{-1, 0, 0, 0};
        if (!more) return g;
        g.h = it.h;
        g.n = min(kRgGroup, it.hi - i0);
        const int pg = (it.first + i0) * C::PPS;
        g.np = min(g.n * C::PPS, (it.ctx + kBlockSize - 1) / kBlockSize - pg);
        if (lane < g.np) g.id = tables[int64_t(it.b) * bt.W + pg + lane];
        i0 += g.n;
        if (i0 >= it.hi) next_item();
        return g;
      };
      uint4 kv = make_uint4(0, 0, 0, 0), vv = kv;
      // this lane's chunk of the scales of step j of a group
      auto scales = [&](const Group& g, int j, uint4& a, uint4& b) {
        if constexpr (C::MV > 0) {
          const int blk = __shfl_sync(0xffffffffu, g.id, j * C::PPS + (sp & 3));
          if (sp < C::PPS && blk >= 0 && blk < NB) {
            const int64_t off = (int64_t(blk) * bt.Hk + g.h) * C::METAB + sc * 16;
            a = __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(ks) + off));
            b = __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(vs) + off));
          }
        }
      };
      next_item();
      Group cur = next_group(), nxt = next_group();
      scales(cur, 0, kv, vv);
      int issued = 0, s = 0;
      bool ok = true;
      while (ok && cur.n > 0) {
        const Group far = next_group();
        for (int j = 0; j < cur.n; ++j, s = s + 1 == C::NRAW ? 0 : s + 1) {
          const int u = issued;
          const int id0 = __shfl_sync(0xffffffffu, cur.id, j * C::PPS + (lane & 3));
          const bool valid = lane < C::PPS && id0 >= 0 && id0 < NB;
          if (lane < C::PPS && j * C::PPS + lane < cur.np && !valid) flag_error(KVQ_DEVERR_BLOCK);
          const uint32_t mask = __ballot_sync(0xffffffffu, valid) & 0xFu;
          const int64_t page = int64_t(id0) * bt.Hk + cur.h;
          uint4 kn = make_uint4(0, 0, 0, 0), vn = kn;
          if (j + 1 < cur.n) scales(cur, j + 1, kn, vn);
          else scales(nxt, 0, kn, vn);
          if (lane == 0) {
            ok = u < C::NRAW || mbar_wait(rfree + s, ((u / C::NRAW) & 1) ^ 1, abort_flag, wait_limit);
            if (ok) mbar_expect_tx(rfull + s, 2u * uint32_t(__popc(mask)) * uint32_t(C::PAGE));
          }
          ok = __shfl_sync(0xffffffffu, int(ok), 0);
          if (!ok) break;
          uint8_t* st = raw + s * C::RSTAGE;
          if (valid) {
            bulk_g2s_keep(st + lane * C::PAGE, kc + page * C::PAGE, C::PAGE, rfull + s);
            bulk_g2s_keep(st + (C::PPS + lane) * C::PAGE, vc + page * C::PAGE, C::PAGE, rfull + s);
          }
          if constexpr (C::MV > 0) {
            if (sp < C::PPS && ((mask >> (sp & 3)) & 1u) != 0u) {
              uint8_t* m = rmeta + s * C::RMETA;
              *reinterpret_cast<uint4*>(m + sp * C::METAB + sc * 16) = kv;
              *reinterpret_cast<uint4*>(m + (C::PPS + sp) * C::METAB + sc * 16) = vv;
            }
          }
          __syncwarp();
          if (lane == 0) {
            rmask[s] = mask;
            mbar_arrive(rfull + s);
          }
          issued = u + 1;
          kv = kn;
          vv = vn;
        }
        cur = nxt;
        nxt = far;
      }
      if (lane == 0) {
        // The copies already issued land before the CTA's shared memory goes away. Not
        // only where a wait has run out by now: another role's may run out later, with
        // the last copies still on their way.
        volatile int no_abort = 0;
        for (int u = issued > C::NRAW ? issued - C::NRAW : 0; u < issued; ++u)
          mbar_wait(rfull + u % C::NRAW, (u / C::NRAW) & 1, &no_abort, kMmaWaitLimitCycles);
      }
    } else if (warp == 1) {
      // ---------------------------------------------------------- MMA issuer
      // One elected lane issues the products. Order of a step i:
      //   two blocks of rows  S_A(i), O_A(i-1), S_B(i), O_B(i-1)
      //   one                 S_x(i), O_y(i-1)   (x, y the slots of the steps)
      // so that a slot's next scores are in the making while its softmax warps
      // are still at work on the last ones. With three weight parts S has to wait
      // for O, which reads the third from S's columns:
      //   two blocks of rows  O_A(i-1), S_A(i), O_B(i-1), S_B(i)
      // and a slot's softmax overlaps the other slot's products only.
      // The smallest part comes first: sums are rounded down, by less while they are small.
      if (elect_one()) {
      constexpr uint32_t id_s = idesc_f16(C::ST, C::BF);
      constexpr uint32_t id_pv = idesc_f16(D, true);
      // operand stages: K pages, then V pages
      const uint32_t q_lo = rg_desc_lo<C::Q_LBO>(smem_u32(qop));
      const uint32_t k_lo = rg_desc_lo<C::K_LBO>(smem_u32(C::BF ? raw : cst));
      const uint32_t v_lo = rg_desc_lo<C::V_LBO>(smem_u32(C::BF ? raw : cst) + C::PPS * C::CPAGE);
      constexpr uint32_t STAGE16 = (C::BF ? C::RSTAGE : C::CSTAGE) / 16;
      uint32_t par_c = 0, par_q = 0;                       // phases of cfull (bit per stage), qready
      uint32_t par_s = 0, par_p = 0;                       // sfree, pready (bit per slot)
      uint32_t fresh = 3;                                  // slots whose S has never been written
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        return mbar_wait(bar, parity, abort_flag, wait_limit);
      };
      auto scores = [&](int x, int stage, int qx) -> bool {
        if (fresh & (1u << x)) {
          fresh &= ~(1u << x);
        } else {
          if (!wait(sfree + x, (par_s >> x) & 1u)) return false;
          par_s ^= 1u << x;
        }
        tc_fence_after();
        {
          const uint32_t kb = k_lo + uint32_t(stage) * STAGE16;
          const uint32_t qa = q_lo + uint32_t(qx) * (C::QBYTES / 16), ds = tmem + C::COL_S + x * 64;
#pragma unroll
          for (int qp = C::QP - 1; qp >= 0; --qp)
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              rg_mma_ss<rg_desc_hi<C::Q_SBO>(), rg_desc_hi<C::K_SBO>()>(
                  ds, qa + qp * (C::QBYTES / 16) + kk * 16, kb + kk * 16, id_s, qp < C::QP - 1 || kk ? 1u : 0u);
          mma_commit(sfull + x);
        }
        return true;
      };
      auto values = [&](int x, int stage, bool first, bool frees) -> bool {
        if (!wait(pready + x, (par_p >> x) & 1u)) return false;
        par_p ^= 1u << x;
        tc_fence_after();
        {
          const uint32_t vb = v_lo + uint32_t(stage) * STAGE16;
          const uint32_t od = tmem + C::COL_O + x * D, pa = tmem + C::COL_P + x * 64;
#pragma unroll
          for (int j = C::PP - 1; j >= 0; --j)
#pragma unroll
            for (int kk = 0; kk < C::PPS; ++kk)
              rg_mma_ts<rg_desc_hi<C::V_SBO>()>(od, (j < 2 ? pa + j * 32 : tmem + C::COL_S + x * 64) + 8 * kk, vb + kk * (C::CPAGE / 16), id_pv,
                                                j < C::PP - 1 || kk ? 1u : uint32_t(!first));
          mma_commit(pvdone + x);
          if (frees) mma_commit(C::BF ? rfree + stage : cfree + stage);   // the step's last product
        }
        return true;
      };
      int stage = 0;
      RgItem w;
      for (int np = 0; ok && fetch(np, w, false); ++np) {
        const int steps = w.hi - w.lo;
        const bool two = w.rows > 128;
        ok = wait(qready, par_q);
        par_q ^= 1u;
        int last = 0;                                      // the stage of the step before
        // whether the values of step v are the first of their slot's O
        auto first = [&](int v) -> bool {
          const int k = two ? v : v >> 1;
          return k % C::flush(w.rows) == 0;
        };
        for (int i = 0; ok && i < steps; ++i) {
          ok = wait(cfull + stage, (par_c >> stage) & 1u);
          if (!ok) break;
          par_c ^= 1u << stage;
          if (two && C::PP == 3) {
            if (i > 0) ok = values(0, last, first(i - 1), false);
            if (ok) ok = scores(0, stage, 0);
            if (ok && i > 0) ok = values(1, last, first(i - 1), true);
            if (ok) ok = scores(1, stage, 1);
          } else if (two) {
            ok = scores(0, stage, 0);
            if (ok && i > 0) ok = values(0, last, first(i - 1), false);
            if (ok) ok = scores(1, stage, 1);
            if (ok && i > 0) ok = values(1, last, first(i - 1), true);
          } else {
            ok = scores(i & 1, stage, 0);
            if (ok && i > 0) ok = values((i & 1) ^ 1, last, first(i - 1), true);
          }
          last = stage;
          stage = stage + 1 == C::NC ? 0 : stage + 1;
        }
        if (ok && two) ok = values(0, last, first(steps - 1), false) && values(1, last, first(steps - 1), true);
        if (ok && !two) ok = values((steps - 1) & 1, last, first(steps - 1), true);
      }
      // every product issued completes before tensor memory is released
      volatile int no_abort = 0;
      mma_commit(drain);
      mbar_wait(drain, 0, &no_abort, kMmaWaitLimitCycles);
      }
      __syncwarp();
    } else if (warp == 2) {
      // ---------------------------------------------------------- the pieces
      // The whole warp walks, all lanes alike. Blocks in which no row attends anything get
      // their zero rows here and are not handed on: a role looks at most kRgRing pieces
      // ahead of the one that it holds up, so it may not skip any number of them.
      using OutT = typename std::conditional<HP, float, __nv_bfloat16>::type;
      RgWalk w;
      w.init(bt, misci[0], miscll[0], start, end);
      for (int i = 0;; w.next(bt)) {
        if (!w.done && w.count == 0) {
          constexpr int PER = D * int(sizeof(OutT)) / 16;      // 16-byte pieces of a row
          for (int j = lane; j < w.rows * PER; j += 32) {
            const int rr = j / PER;
            const int64_t row = int64_t(w.row0 + (w.k << bt.p.pos_log) + (rr >> bt.p.g_log)) * (bt.Hk << bt.p.g_log) +
                                (w.h << bt.p.g_log) + (rr & ((1 << bt.p.g_log) - 1));
            reinterpret_cast<uint4*>(static_cast<OutT*>(out_) + row * D)[j % PER] = make_uint4(0, 0, 0, 0);
          }
          continue;
        }
        const int s = i % kRgRing;
        bool got = true;
        if (lane == 0) {
          got = i < kRgRing || mbar_wait(pfree + s, (i / kRgRing - 1) & 1, abort_flag, wait_limit);
          if (got) {
            RgItem it;
            it.b = w.b; it.h = w.h; it.k = w.k; it.rows = w.done ? 0 : w.rows;
            it.row0 = w.row0; it.n = w.s.n; it.ctx = w.s.ctx; it.first = w.first;
            it.lo = w.lo; it.hi = w.hi; it.count = w.count; it.pad = 0;
            items[s] = it;
            mbar_arrive(pfull + s);
          }
        }
        if (!__shfl_sync(0xffffffffu, int(got), 0) || w.done) break;
        ++i;
      }
    }
  } else if (warp >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    // ---------------------------------------------------------- converters
    const int ct = threadIdx.x - 384;                      // 0 .. 127
    bool ok = true;
    int u = 0, s = 0, cs = 0;                              // step, its raw and operand stage
    RgItem w;
    for (int np = 0; ok && fetch(np, w, true); ++np) {
      // tokens that every row of the block attends
      const int j0 = w.k << bt.p.pos_log, base = w.ctx - w.n;
      const int all_end = base + j0 + 1;
      const int all_beg = bt.p.window > 0 ? base + j0 + (w.rows >> bt.p.g_log) - bt.p.window : 0;
      for (int i = w.lo; ok && i < w.hi; ++i, ++u, s = s + 1 == C::NRAW ? 0 : s + 1, cs = cs + 1 == C::NC ? 0 : cs + 1) {
        if (ok) ok = mbar_wait(rfull + s, (u / C::NRAW) & 1, abort_flag, wait_limit);
        if (ok && !C::BF && u >= C::NC) ok = mbar_wait(cfree + cs, (u / C::NC - 1) & 1, abort_flag, wait_limit);
        ok = __all_sync(0xffffffffu, ok);                  // what follows votes and reduces over the warp
        const uint32_t pm = rmask[s];
        const int tok0 = (w.first + i) * C::ST;
        if (ct == 0) cpages[cs] = pm;
        const bool plain = tok0 >= all_beg && tok0 + C::ST <= all_end && pm == 0xFu;   // no mask, nothing missing
        uint8_t* rk = raw + s * C::RSTAGE;
        uint8_t* rv = rk + C::PPS * C::PAGE;
        uint8_t* cb = cst + cs * C::CSTAGE;
        uint32_t* cmw = reinterpret_cast<uint32_t*>(cmask + 3 * cs);
        // tokens of page p that hold cache entries
        auto nvalid = [&](int p) -> int {
          if (((pm >> p) & 1u) == 0u) return 0;
          return max(0, min(16, w.ctx - (tok0 + 16 * p)));
        };
        if (ok) {
          if constexpr (C::BF) {
            // V as it is stored; where some row does not attend every token, tokens that
            // hold nothing and tokens with a NaN or an infinity are zeroed
            uint32_t bad0 = 0u, bad1 = 0u;
            constexpr int NIT = C::PPS * 2 * D / 128;
#pragma unroll 2
            for (int it = plain ? NIT : 0; it < NIT; ++it) {
              const int x = ct + 128 * it;                 // chunk: 8 tokens of a channel
              const int p = x / (2 * D), o8 = ((x / D) & 1) * 8;
              const int keep = max(0, min(8, nvalid(p) - o8));
              uint4* ch = reinterpret_cast<uint4*>(rv + x * 16);
              const uint4 c4 = *ch;
              uint32_t wv[4] = {c4.x, c4.y, c4.z, c4.w};
              uint32_t mx = 0u;
#pragma unroll
              for (int e = 0; e < 4; ++e) mx = vmax_u16x2(mx, wv[e] & 0x7fff7fffu);
              const bool wild = max(mx & 0xffffu, mx >> 16) >= 0x7f80u;
              if (keep == 8 && !wild) continue;
              uint32_t bad = 0u;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                uint32_t m = 0u;
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                  const uint32_t v16 = (wv[e] >> (16 * z)) & 0x7fffu;
                  const int t = 2 * e + z;
                  if (t < keep && v16 < 0x7f80u) m |= 0xffffu << (16 * z);
                  if (t < keep && v16 >= 0x7f80u) bad |= 1u << t;
                }
                wv[e] &= m;
              }
              *ch = make_uint4(wv[0], wv[1], wv[2], wv[3]);
              bad <<= (p & 1) * 16 + o8;
              if (p < 2) bad0 |= bad;
              else bad1 |= bad;
            }
            bad0 = __reduce_or_sync(0xffffffffu, bad0);
            bad1 = __reduce_or_sync(0xffffffffu, bad1);
            if (lane == 0) {
              cmw[ct >> 5] = (pm ^ 0xFu) | bad0 | bad1;
              cmw[4 + (ct >> 5)] = bad0;
              cmw[8 + (ct >> 5)] = bad1;
            }
          } else {
            // A warp has one page of the step. The loops stay rolled: the kernel's roles
            // share the instruction caches, and unrolled they cost all of them more than
            // their own latency (FP8 chunks: 205 against 163 us).
            const int pw = ct >> 5;
            const uint32_t rka = smem_u32(rk) + pw * C::PAGE, rva = smem_u32(rv) + pw * C::PAGE;
            const uint32_t cka = smem_u32(cb) + pw * C::CPAGE, cva = cka + C::PPS * C::CPAGE;
            float* cm = reinterpret_cast<float*>(cb + 2 * C::PPS * C::CPAGE);
            const uint8_t* mk = rmeta + s * C::RMETA;
            const uint8_t* mv = mk + C::PPS * C::METAB;
            constexpr int NIT = D / 32;
            const int nv = nvalid(pw);
            uint32_t keep = nv >= 16 ? 0xffffu : (1u << nv) - 1u;   // tokens of the page that count
            // f16 pairs of neighbouring tokens' V zero points; K zero point of token
            // `lane % 16`, twice
            uint32_t vz[C::ZP ? 8 : 1];
            uint32_t kz = 0u;
            if constexpr (C::MV > 0) {
              // the step's largest finite V scale
              constexpr int MB = 2 * C::MV;
              uint32_t top = 0u;
#pragma unroll
              for (int z = 0; z < 2; ++z) {
                const int t = lane + 32 * z;
                uint32_t v = 0u;                             // for a token that holds nothing
                if (((pm >> (t >> 4)) & 1u) != 0u && tok0 + t < w.ctx) v = *reinterpret_cast<const uint16_t*>(mv + t * MB) & 0x7fffu;
                if (v < 0x7f80u) top = max(top, v);
              }
              top = __reduce_max_sync(0xffffffffu, top);
              // an exponent is taken out of the step's scales when they are beyond 2^60 or
              // 2^-60 only, so that weights times scales, and their sums, stay within FP32
              const int e = int(top >> 7) - 127;
              const int ev = top == 0u ? 0 : e > 60 ? e - 60 : e < -60 ? e + 60 : 0;
              const float vdn = __int_as_float((127 - ev) << 23);
              // this page's tokens: lane % 16
              const int t = 16 * pw + (lane & 15);
              const bool there = (lane & 15) < nv;
              float sk = 0.f, sv = 0.f;
              if (there) {
                sk = __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(mk + t * MB));
                sv = __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(mv + t * MB));
              }
              const bool wild = !(fabsf(sv) < INFINITY);
              const uint32_t wm = __ballot_sync(0xffffffffu, wild) & 0xffffu;
              if (wild) sv = plain ? __int_as_float(0x7fc00000) : 0.f;
              if (!plain) keep &= ~wm;
              if (lane < 16) {
                cm[t] = sk * qk_scale;
                cm[C::ST + t] = sv * vdn;
              }
              if constexpr (C::ZP) {
                float zk = 0.f, zv = 0.f;
                if (there) {
                  zk = __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(mk + t * MB + 2));
                  zv = __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(mv + t * MB + 2));
                }
                auto half_bits = [](float x) -> uint32_t { return __half_as_ushort(__float2half_rn(x)); };
                const uint32_t own = half_bits(1152.f + zv);
                const uint32_t two = own | (__shfl_xor_sync(0xffffffffu, own, 1) << 16);
#pragma unroll
                for (int j = 0; j < 8; ++j) vz[j] = __shfl_sync(0xffffffffu, two, 2 * j);
                kz = half_bits(1152.f + zk) * 0x10001u;
              }
              if (lane == 0) {
                if (pw == 0)
                  *reinterpret_cast<float2*>(cm + 2 * C::ST) = make_float2(float(ev), vdn);
                const uint32_t bad = plain ? 0u : wm;
                cmw[4 + pw] = pw < 2 ? bad << (16 * pw) : 0u;
                cmw[8 + pw] = pw < 2 ? 0u : bad << (16 * (pw - 2));
                cmw[pw] = (pm ^ 0xFu) | bad;
              }
            } else {
              if (lane == 0) cmw[pw] = pm ^ 0xFu;
            }
#pragma unroll 1
            for (int it = 0; it < NIT; ++it) {               // 16 channels of a token
              const int k = lane + 32 * it;
              const uint4 codes = lds_u4(rka + k * 16);
              const int g = k / (D / 2), rem = k % (D / 2), c = rem >> 3, tt = rem & 7;
              uint4 o0, o1;
              if constexpr (C::ZP) codes16_less(codes, __shfl_sync(0xffffffffu, kz, 8 * g + tt), o0, o1);
              else codes16_to_f16<FMT>(codes, o0, o1);
              const uint32_t dst = cka + g * 16 * D + (2 * c) * 128 + tt * 16;
              sts_u4(dst, o0.x, o0.y, o0.z, o0.w);
              sts_u4(dst + 128, o1.x, o1.y, o1.z, o1.w);
            }
#pragma unroll 1
            for (int it = 0; it < NIT; ++it) {               // 16 tokens of a channel
              const int d = lane + 32 * it;
              const uint4 codes = lds_u4(rva + d * 16);
              uint4 o0, o1;
              if constexpr (C::ZP) codes16_less_pairs(codes, vz, o0, o1);
              else codes16_to_f16<FMT>(codes, o0, o1);
              uint32_t wv[8] = {o0.x, o0.y, o0.z, o0.w, o1.x, o1.y, o1.z, o1.w};
#pragma unroll
              for (int j = 0; j < 8; ++j) wv[j] = f16x2_to_bf16x2(wv[j]);   // exact: codes less zero points
              if (!plain) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                  wv[j] &= ((keep >> (2 * j)) & 1u ? 0x0000FFFFu : 0u) | ((keep >> (2 * j + 1)) & 1u ? 0xFFFF0000u : 0u);
              }
              sts_u4(cva + d * 16, wv[0], wv[1], wv[2], wv[3]);
              sts_u4(cva + (D + d) * 16, wv[4], wv[5], wv[6], wv[7]);
            }
          }
          fence_proxy_async_smem();
        }
        warp_arrive(cfull + cs, lane);
        if constexpr (!C::BF) {
          if (lane == 0) mbar_arrive(rfree + s);
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
    // ---------------------------------------------------------- softmax warps
    const int quarter = warp & 3;
    const int x = (warp - 4) >> 2;                         // slot
    const int r = quarter * 32 + lane;                     // row of the slot, TMEM lane
    const uint32_t lane_base = uint32_t(quarter * 32) << 16;
    const uint32_t t_o = tmem + lane_base + C::COL_O + x * D;
    const uint32_t t_s = tmem + lane_base + C::COL_S + x * 64;
    const uint32_t t_p = tmem + lane_base + C::COL_P + x * 64;
    float* xch = reinterpret_cast<float*>(smem + C::OFF_X);              // [16][128]
    float2* xsum = reinterpret_cast<float2*>(smem + C::OFF_XS);          // [128]
    const int pair_bar = 2 + quarter;                      // the two warps of this lane quarter
    const int gshift = bt.p.g_log, G = 1 << gshift;
    bool ok = true;
    auto wait_all = [&](uint64_t* bar, uint32_t parity) {  // tcgen05.ld / st are warp-wide
      if (ok) ok = mbar_wait(bar, parity, abort_flag, wait_limit);
      ok = __all_sync(0xffffffffu, ok);
    };
    // this thread's row of a block: the block row, its token of the sequence's new ones
    auto block_row = [&](const RgItem& w) -> int {
      return w.rows > 128 ? x * 128 + r : w.rows <= kRgNarrow ? lane : r;
    };
    auto token_of = [&](const RgItem& w, int rr) -> int { return (w.k << bt.p.pos_log) + (rr >> gshift); };
    auto head_of = [&](const RgItem& w, int rr) -> int { return (w.h << gshift) + (rr & (G - 1)); };

    // The query rows of a piece into the operand (K-major 8-row groups of
    // 16-byte chunks). A warp takes its 32 rows eight at a time, a lane one row
    // (lane % 8) of them and every fourth chunk: 64 contiguous bytes a row from
    // global memory, 512 to shared memory. `down` takes the scores of this thread's own
    // row (lane = 8 (lane / 8) + lane % 8) back to the row's units. With one block
    // of rows for both slots, slot A's warps write it.
    auto store_q = [&](const RgItem& w, float& down) {
      down = 1.f;
      const bool two = w.rows > 128;
      const int rs = lane & 7, cs = lane >> 3;
      const bool wr = two || x == 0;
      constexpr int NI = D / 32;
      uint4 c[4][NI];
#pragma unroll
      for (int rg = 0; rg < 4; ++rg) {
        const int rr = (two ? x * 128 : 0) + (w.rows <= kRgNarrow ? 0 : quarter * 32) + 8 * rg + rs;
        const bool have = rr < w.rows;
        const uint4* src = reinterpret_cast<const uint4*>(
            q + int64_t(w.row0 + (have ? token_of(w, rr) : 0)) * q_stride + int64_t(head_of(w, rr)) * D) + cs;
#pragma unroll
        for (int i = 0; i < NI; ++i) c[rg][i] = have ? src[4 * i] : make_uint4(0, 0, 0, 0);
      }
      uint8_t* dst = qop + (two ? x : 0) * C::QBYTES + quarter * 4 * C::Q_SBO + rs * 16 + cs * C::Q_LBO;
      // sm_scale is the row factor's, its sign the query's (scales per token: their factors have it)
      if constexpr (C::BF) {
        down = fabsf(qk_scale);
        const uint32_t sg = qk_scale < 0.f ? 0x80008000u : 0u;
        if (wr) {
#pragma unroll
          for (int rg = 0; rg < 4; ++rg)
#pragma unroll
            for (int i = 0; i < NI; ++i)
              *reinterpret_cast<uint4*>(dst + rg * C::Q_SBO + 4 * i * C::Q_LBO) =
                  make_uint4(c[rg][i].x ^ sg, c[rg][i].y ^ sg, c[rg][i].z ^ sg, c[rg][i].w ^ sg);
        }
      } else {
        // static INT8: q times the K scale of the channel
        uint4 sc[C::SI ? NI : 1];
        if constexpr (C::SI) {
          const uint32_t one = per_tensor ? *reinterpret_cast<const uint16_t*>(ks) * 0x10001u : 0u;
#pragma unroll
          for (int i = 0; i < NI; ++i)
            sc[i] = per_tensor ? make_uint4(one, one, one, one)
                               : reinterpret_cast<const uint4*>(ks + w.h * D)[4 * i + cs];
        }
        auto pair = [&](int rg, int i, int e) -> float2 {
          const uint32_t v = e == 0 ? c[rg][i].x : e == 1 ? c[rg][i].y : e == 2 ? c[rg][i].z : c[rg][i].w;
          float2 f = make_float2(bf16_lo(v), bf16_hi(v));
          if constexpr (C::SI) {
            const uint32_t k = e == 0 ? sc[i].x : e == 1 ? sc[i].y : e == 2 ? sc[i].z : sc[i].w;
            f.x *= bf16_lo(k);
            f.y *= bf16_hi(k);
          }
          return f;
        };
#pragma unroll
        for (int rg = 0; rg < 4; ++rg) {
          float amax = 0.f;
          if constexpr (C::SI) {
#pragma unroll
            for (int i = 0; i < NI; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 f = pair(rg, i, e);
                amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
              }
          } else {
            uint32_t m = 0u;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
              m = vmax_u16x2(m, c[rg][i].x & 0x7fff7fffu);
              m = vmax_u16x2(m, c[rg][i].y & 0x7fff7fffu);
              m = vmax_u16x2(m, c[rg][i].z & 0x7fff7fffu);
              m = vmax_u16x2(m, c[rg][i].w & 0x7fff7fffu);
            }
            amax = __uint_as_float(max(m & 0xffffu, m >> 16) << 16);
          }
          amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 8));
          amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 16));
          // power-of-two scaling: the largest element lands in [2^14, 2^15)
          int e2 = 0;
          if (amax > 0.f && amax < INFINITY) e2 = 14 - ilogbf(amax);
          e2 = max(-113, min(100, e2));
          float up = __int_as_float((127 + e2) << 23);
          if (rg == cs) down = __int_as_float((127 - e2) << 23);
          if constexpr (!C::COLS) {
            up = copysignf(up, qk_scale);
            if (rg == cs) down *= fabsf(qk_scale);
          }
#pragma unroll
          for (int i = 0; i < NI; ++i) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 f = pair(rg, i, e);
              const float a = f.x * up, b = f.y * up;
              const __half2 h2 = __floats2half2_rn(a, b);
              hi[e] = *reinterpret_cast<const uint32_t*>(&h2);
              if constexpr (C::QP == 2) {
                const __half2 l2 = __floats2half2_rn(a - __low2float(h2), b - __high2float(h2));
                lo[e] = *reinterpret_cast<const uint32_t*>(&l2);
              }
            }
            if (wr) {
              *reinterpret_cast<uint4*>(dst + rg * C::Q_SBO + 4 * i * C::Q_LBO) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
              if constexpr (C::QP == 2)
                *reinterpret_cast<uint4*>(dst + C::QBYTES + rg * C::Q_SBO + 4 * i * C::Q_LBO) =
                    make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
          }
        }
      }
      fence_proxy_async_smem();
    };
    using OutT = typename std::conditional<HP, float, __nv_bfloat16>::type;
    OutT* out = static_cast<OutT*>(out_);
    const bool wide = (reinterpret_cast<uintptr_t>(out_) & 31) == 0;
    auto st32 = [&](void* dst, const uint32_t (&v)[8]) {   // 32 bytes of one row
      if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                     "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                     : "memory");
      } else {
        reinterpret_cast<uint4*>(dst)[0] = make_uint4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<uint4*>(dst)[1] = make_uint4(v[4], v[5], v[6], v[7]);
      }
    };
    auto store_row16 = [&](OutT* dst, const float (&o)[16]) {
      uint32_t v[8];
      if constexpr (HP) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = __float_as_uint(o[8 * i + e]);
          st32(dst + 8 * i, v);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const __nv_bfloat162 w2 = __floats2bfloat162_rn(o[2 * e], o[2 * e + 1]);
          v[e] = *reinterpret_cast<const uint32_t*>(&w2);
        }
        st32(dst, v);
      }
    };
    // The next piece. The eight warps meet at barriers, so they go on together or
    // not at all.
    int np = 0;
    auto next_item = [&](RgItem& w) -> bool {
      const bool mine = ok && fetch(np++, w, true);
      uint32_t both;
      asm volatile(
          "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
          "barrier.cta.red.and.pred q, 1, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}\n"
          : "=r"(both)
          : "r"(uint32_t(mine))
          : "memory");
      return both != 0u;
    };

    RgItem pw;
    bool more = next_item(pw);
    float down = 1.f;
    if (more) {
      store_q(pw, down);
      warp_arrive(qready, lane);
    }
    int u0 = 0;                                            // the piece's first step
    uint32_t cnt = 0, cnt_other = 0;                       // steps of this slot and of the other so far
    while (more) {
      const bool two = pw.rows > 128;
      const int rr = block_row(pw);
      const bool row_ok = rr < pw.rows;
      const bool active = __any_sync(0xffffffffu, row_ok);
      const int nsteps = pw.hi - pw.lo;
      const int p = pw.ctx - pw.n + token_of(pw, rr);
      // tokens lo_t <= t < lim are attended; rows past the block's see everything
      // (nothing of them is written)
      const int lim = row_ok ? max(0, p + 1) : INT_MAX;
      const int lo_t = row_ok && bt.p.window > 0 ? max(0, p + 1 - bt.p.window) : 0;
      const int lim_min = __reduce_min_sync(0xffffffffu, lim), lo_max = __reduce_max_sync(0xffffffffu, lo_t);
      float m_run = -INFINITY, mref = 0.f, l = 0.f;   // mref: m_run, or 0 where it is -inf
      bool any_step = false;
      // The tensor cores round their sums down, by up to a last bit for each
      // product added; so a slot's O goes to the workspace every FLUSH steps (rows side by
      // side, each thread its own) and is added up there in FP32. m_sum: their reference.
      float* sum = sums + (int64_t(blockIdx.x) * 2 + x) * 128 * D + r;
      float m_sum = -INFINITY;
      bool summed = false;
      // A narrow block: all four warps of a slot have its rows, each for 16 of a
      // step's tokens, as a softmax of their own (P is zero in the others' columns).
      const bool narrow = pw.rows <= kRgNarrow;
      if (narrow) {
        const uint32_t z[16] = {};
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_st16(t_p + 16 * c, z);
        tmem_st_wait();
      }
      // operand stage, and its phase, of this slot's first step
      int stage = (two ? u0 : u0 + x) % C::NC;
      uint32_t phase = ((two ? u0 : u0 + x) / C::NC) & 1;
      // One step: the scores of this warp's rows for `width` tokens (all 64, or with
      // narrow blocks the warp's 16) to weights. Nothing moves the reference in
      // most steps, and most have no mask.
      auto softmax_step = [&](auto width, int i, int ck) {
        constexpr int NT = decltype(width)::value;         // tokens of the step that are this warp's
        const int col0 = NT == C::ST ? 0 : NT * quarter;   // the first of them
        uint32_t sr[NT];
        if constexpr (NT == C::ST) {
          tmem_ld32(t_s, sr);
          tmem_ld32(t_s + 32, sr + 32);
        } else {
          tmem_ld16(t_s + col0, sr);
        }
        tmem_ld_wait();
        tc_fence_before();
        warp_arrive(sfree + x, lane);
        // the tokens' K and V scales, four at a time; then {eV, 2^-eV}
        const float4* cm4 = reinterpret_cast<const float4*>(smem + C::OFF_C + ck * C::CSTAGE + (C::BF ? 0 : 2 * C::PPS * C::CPAGE));
        const int q0 = col0 / 4;
        const uint4 odd = cmask[3 * ck];
        const int t0 = (pw.first + pw.lo + i) * C::ST;
        // every row of the warp attends every token (the same for all its lanes)
        const bool full = t0 >= lo_max && t0 + C::ST <= lim_min && (odd.x | odd.y | odd.z | odd.w) == 0u;
        // Scores in the operand's units (times f: base-2 scores), in place of S.
        float2* x2 = reinterpret_cast<float2*>(sr);
        if constexpr (C::COLS) {
          float4 fa[2][4];
#pragma unroll
          for (int j = 0; j < 4; ++j) fa[0][j] = cm4[q0 + j];
#pragma unroll
          for (int c = 0; c < NT / 16; ++c) {
            if (c + 1 < NT / 16) {
#pragma unroll
              for (int j = 0; j < 4; ++j) fa[(c + 1) & 1][j] = cm4[q0 + 4 * (c + 1) + j];
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int k = 8 * c + 2 * j;
              const float4 a = fa[c & 1][j];
              x2[k] = __fmul2_rn(x2[k], make_float2(a.x, a.y));
              x2[k + 1] = __fmul2_rn(x2[k + 1], make_float2(a.z, a.w));
            }
          }
        }
        bool wild = false;
        if (!full) {
          // the tokens this row attends, as bits
          auto low = [](int n) -> uint64_t { return n >= 64 ? ~0ull : n <= 0 ? 0ull : (1ull << n) - 1ull; };
          uint64_t vis = low(lim - t0) & ~low(lo_t - t0);
          const uint32_t pages_ok = cpages[ck];
          const uint4 wl = cmask[3 * ck + 1], wh = cmask[3 * ck + 2];
          const uint32_t wild0 = wl.x | wl.y | wl.z | wl.w, wild1 = wh.x | wh.y | wh.z | wh.w;
#pragma unroll
          for (int pg = 0; pg < C::PPS; ++pg)
            if (((pages_ok >> pg) & 1u) == 0u) vis &= ~(0xffffull << (16 * pg));
          uint64_t bad = uint64_t(wild0) | (uint64_t(wild1) << 32);
          if constexpr (NT < C::ST) {
            vis = (vis >> col0) & 0xffffull;
            bad >>= col0;
          }
          wild = (vis & bad) != 0ull;
          const uint32_t v0 = uint32_t(vis), v1 = uint32_t(vis >> 32);
#pragma unroll
          for (int c = 0; c < NT; ++c)
            if (!(((c < 32 ? v0 : v1) >> (c & 31)) & 1u)) sr[c] = 0xff800000u;
        }
        float2 ee = make_float2(0.f, 1.f);                 // eV, 2^-eV
        if constexpr (C::COLS) ee = *reinterpret_cast<const float2*>(cm4 + C::ST / 2);
        // takes x to the base-2 score; never 0 (a score scale of 0, or an underflow), so that
        // masked scores stay -inf
        const float f = fmaxf(down, 1.17549435e-38f);
        float mt;
        {
          float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int k = 0; k < NT; k += 8)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              m4[j] = max3(m4[j], __uint_as_float(sr[k + 2 * j]), __uint_as_float(sr[k + 2 * j + 1]));
          mt = max3(fmaxf(m4[0], m4[1]), m4[2], m4[3]) * f + ee.x;
        }
        bool pv_seen = false;
        if (__any_sync(0xffffffffu, mt > m_run + 8.f)) {
          const bool move = mt > m_run + 8.f;
          const float alpha = move && m_run != -INFINITY ? ex2_ftz(m_run - mt) : 1.f;
          m_run = move ? mt : m_run;
          mref = m_run == -INFINITY ? 0.f : m_run;
          l *= alpha;
          if (__any_sync(0xffffffffu, alpha != 1.f)) {
            wait_all(pvdone + x, (cnt - 1) & 1);
            tc_fence_after();
            pv_seen = true;
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
              uint32_t ov[16];
              tmem_ld16(t_o + 16 * c, ov);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 16; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
              tmem_st16(t_o + 16 * c, ov);
            }
            tmem_st_wait();
          }
        }
        // weights 2^(x f - m + eV) times the token's V scale 2^-eV, in parts
        const float mx = ee.x - mref;
        const float2 dn2 = make_float2(f, f), nm2 = make_float2(mx, mx);
        float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        constexpr int NCH = NT / 16;
        auto expo = [&](int c) {
#pragma unroll
          for (int k = 8 * c; k < 8 * c + 8; ++k) x2[k] = __ffma2_rn(x2[k], dn2, nm2);
#pragma unroll
          for (int k = 8 * c; k < 8 * c + 8; ++k) x2[k] = make_float2(ex2_ftz(x2[k].x), ex2_ftz(x2[k].y));
        };
        constexpr int STC = C::PP == 3 || NCH == 1 ? 1 : 2;  // chunks stored together
        uint32_t ph[8 * STC], pl[8 * STC], pt[8 * STC];
        float4 fs[4];
        expo(0);
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
          if constexpr (C::COLS) {
#pragma unroll
            for (int j = 0; j < 4; ++j) fs[j] = cm4[C::ST / 4 + q0 + 4 * c + j];
          }
          if (c + 1 < NCH) expo(c + 1);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int kk = 8 * c + k, o = 8 * (c % STC) + k;
            const float2 p2 = x2[kk];
            ls[k & 1] = __fadd2_rn(ls[k & 1], p2);
            float2 wv = p2;
            if constexpr (C::COLS)
              wv = __fmul2_rn(p2, (k & 1) ? make_float2(fs[k / 2].z, fs[k / 2].w) : make_float2(fs[k / 2].x, fs[k / 2].y));
            ph[o] = rg_pack(wv.x, wv.y);
            const float2 rest = __ffma2_rn(make_float2(bf16_lo(ph[o]), bf16_hi(ph[o])), make_float2(-1.f, -1.f), wv);   // exact
            pl[o] = rg_pack(rest.x, rest.y);
            if constexpr (C::PP == 3) pt[o] = rg_pack(rest.x - bf16_lo(pl[o]), rest.y - bf16_hi(pl[o]));
          }
          if (c % STC == STC - 1) {
            // the last product has read P
            if (c < STC && cnt > 0 && !pv_seen) {
              wait_all(pvdone + x, (cnt - 1) & 1);
              tc_fence_after();
            }
            if constexpr (NCH == 1) {
              tmem_st8(t_p + col0 / 2, ph);
              tmem_st8(t_p + 32 + col0 / 2, pl);
              if constexpr (C::PP == 3) {
                const uint32_t z[8] = {};                  // S was in the other warps' columns
#pragma unroll
                for (int w = 0; w < 4; ++w)
                  if (w != quarter) tmem_st8(t_s + 8 * w, z);
                tmem_st8(t_s + col0 / 2, pt);
              }
            } else if constexpr (STC == 1) {
              tmem_st8(t_p + 8 * c, ph);
              tmem_st8(t_p + 32 + 8 * c, pl);
              tmem_st8(t_s + 8 * c, pt);
            } else {
              tmem_st16(t_p + 8 * (c - 1), ph);
              tmem_st16(t_p + 32 + 8 * (c - 1), pl);
            }
          }
        }
        const float2 ls2 = __fadd2_rn(ls[0], ls[1]);
        l += (ls2.x + ls2.y) * ee.y;
        if (wild) l = __int_as_float(0x7fc00000);
        tmem_st_wait();
        tc_fence_before();
        warp_arrive(pready + x, lane);
      };
      for (int i = two ? 0 : x; i < nsteps; i += two ? 1 : 2) {
        const int ck = stage;
        const uint32_t cpar = phase;
        const int ahead = two ? 1 : 2;                     // to this slot's next step
        stage += ahead;
        if (stage >= C::NC) {
          stage -= C::NC;
          phase ^= 1u;
        }
        // both at once: they are mostly complete
        if (!__all_sync(0xffffffffu, mbar_test_wait(sfull + x, cnt & 1) & mbar_test_wait(cfull + ck, cpar))) {
          wait_all(sfull + x, cnt & 1);
          wait_all(cfull + ck, cpar);
        }
        tc_fence_after();
        if (!active) {
          warp_arrive(sfree + x, lane);
          if (cnt > 0) wait_all(pvdone + x, (cnt - 1) & 1);
          warp_arrive(pready + x, lane);
          ++cnt;
          continue;
        }
        if ((two ? i : i >> 1) % C::flush(pw.rows) == 0 && any_step) {
          wait_all(pvdone + x, (cnt - 1) & 1);
          tc_fence_after();
          const float f = ex2_ftz(m_sum - mref);
#pragma unroll 1
          for (int c = 0; c < D / 16; ++c) {
            uint32_t ov[16];
            tmem_ld16(t_o + 16 * c, ov);
            float was[16] = {};
            if (summed) {
#pragma unroll
              for (int e = 0; e < 16; ++e) was[e] = sum[(16 * c + e) * 128] * f;
            }
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) sum[(16 * c + e) * 128] = was[e] + __uint_as_float(ov[e]);
          }
          m_sum = m_run;
          summed = true;
        }
        if (narrow) softmax_step(std::integral_constant<int, 16>{}, i, ck);
        else softmax_step(std::integral_constant<int, C::ST>{}, i, ck);
        ++cnt;
        any_step = true;
      }
      if (!active) any_step = (two ? 0 : x) < nsteps;
      cnt_other += two ? nsteps : (x ? (nsteps + 1) / 2 : nsteps / 2);
      u0 += nsteps;

      // the next piece's query, once the products that read this one's have completed
      RgItem nxt;
      const bool more_n = next_item(nxt);
      float down_n = 1.f;
      if (more_n) {
        if (!two && x == 0 && nsteps > 1) wait_all(sfull + 1, (cnt_other - 1) & 1);
        store_q(nxt, down_n);
        warp_arrive(qready, lane);
      }

      // ---- the piece's end: O of the last step
      if (any_step) wait_all(pvdone + x, (cnt - 1) & 1);
      tc_fence_after();
      const float f_sum = summed ? ex2_ftz(m_sum - mref) : 0.f;
      auto add_sums = [&](uint32_t (&ov)[16], int c) {
        if (summed) {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            ov[e] = __float_as_uint(__uint_as_float(ov[e]) + sum[(16 * c + e) * 128] * f_sum);
        }
      };
      const bool whole = pw.lo == 0 && pw.hi == pw.count;
      const int64_t place = int64_t(blockIdx.x) * 2 + (pw.lo == 0 ? 1 : 0);
      auto out_row = [&](int row) -> int64_t {
        return int64_t(pw.row0 + token_of(pw, row)) * (bt.Hk << gshift) + head_of(pw, row);
      };
      auto v_scale = [&](int d) -> float {
        if constexpr (C::SI) return __bfloat162float(vs[per_tensor ? 0 : pw.h * D + d]);
        return 1.f;
      };
      if (narrow) {
        // eight softmaxes of the same rows: their references and sums first, then O
        // 16 channels at a time, each warp adding up two channels for all rows
        const int strm = x * 4 + quarter;
        if (lane < kRgNarrow) xsum[strm * kRgNarrow + lane] = any_step ? make_float2(m_run, l) : make_float2(-INFINITY, 0.f);
        named_bar_sync(1, 256);
        const int row = lane & (kRgNarrow - 1);
        float m = -INFINITY;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = fmaxf(m, xsum[j * kRgNarrow + row].x);
        const float ref = m == -INFINITY ? 0.f : m;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 o = xsum[j * kRgNarrow + row];
          sum += o.y * ex2_ftz(o.x - ref);
        }
        const float mine = any_step ? ex2_ftz(m_run - ref) : 0.f;
        const float inv = whole ? (sum == 0.f ? 0.f : 1.f / sum) : 1.f;
#pragma unroll 1
        for (int c = 0; c < D / 16; ++c) {
          uint32_t ov[16];
          tmem_ld16(t_o + 16 * c, ov);
          tmem_ld_wait();
          add_sums(ov, c);
          if (lane < kRgNarrow) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
              xch[(strm * 16 + e) * kRgNarrow + lane] = any_step ? __uint_as_float(ov[e]) * mine : 0.f;
          }
          named_bar_sync(1, 256);
          const int e = 2 * strm + (lane >> 4), d = 16 * c + e;
          float o = 0.f;
#pragma unroll
          for (int j = 0; j < 8; ++j) o += xch[(j * 16 + e) * kRgNarrow + row];
          o *= v_scale(d) * inv;
          if (row < pw.rows) {
            if (whole) {
              if constexpr (HP) out[out_row(row) * D + d] = o;
              else out[out_row(row) * D + d] = __float2bfloat16_rn(o);
            } else {
              part_o[(place * D + d) * rows_cap + row] = o;
            }
          }
          named_bar_sync(1, 256);
        }
        if (!whole && strm == 0 && lane < pw.rows)
          *reinterpret_cast<float2*>(part_ml + (place * rows_cap + row) * 2) = make_float2(m, sum);
      } else if (active) {
        float ma = 1.f, mb = 0.f;                          // O = ma O_A + mb O_B (one block of rows)
        if (!two) {
          if (x == 1) xsum[r] = any_step ? make_float2(m_run, l) : make_float2(-INFINITY, 0.f);
          named_bar_sync(pair_bar, 64);
          if (x == 0) {
            const float2 o = xsum[r];
            const float m = fmaxf(m_run, o.x);
            const float mr = m == -INFINITY ? 0.f : m;
            ma = ex2_ftz(m_run - mr);
            mb = ex2_ftz(o.x - mr);
            l = l * ma + o.y * mb;
            m_run = m;
          }
        }
        const float inv = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
#pragma unroll 1
        for (int c = 0; c < D / 16; ++c) {
          uint32_t ov[16];
          tmem_ld16(t_o + 16 * c, ov);
          tmem_ld_wait();
          add_sums(ov, c);
          float o[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = any_step ? __uint_as_float(ov[e]) : 0.f;
          if (!two) {
            if (x == 1) {
#pragma unroll
              for (int e = 0; e < 16; ++e) xch[e * 128 + r] = o[e];
            }
            named_bar_sync(pair_bar, 64);
            if (x == 0) {
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = o[e] * ma + xch[e * 128 + r] * mb;
            }
            named_bar_sync(pair_bar, 64);
          }
          if (row_ok && (two || x == 0)) {
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] *= v_scale(16 * c + e) * inv;
            if (whole) {
              store_row16(out + out_row(rr) * D + 16 * c, o);
            } else {
              // channel by channel, the rows side by side
              float* po = part_o + (place * D + 16 * c) * rows_cap + rr;
#pragma unroll
              for (int e = 0; e < 16; ++e) po[int64_t(e) * rows_cap] = o[e];
            }
          }
        }
        if (!whole && row_ok && (two || x == 0))
          *reinterpret_cast<float2*>(part_ml + (place * rows_cap + rr) * 2) = make_float2(m_run, l);
      }
      if (!whole && x == 0 && r == 0)
        rg_record(pieces + place, pw.hi == pw.count, pw.row0, pw.n, pw.h, pw.k);
      tc_fence_before();
      down = down_n;
      pw = nxt;
      more = more_n;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
  if (*abort_flag) {
    // what this CTA was to write becomes NaN
    if (threadIdx.x == 0) flag_error(KVQ_DEVERR_TIMEOUT);
    using OutT = typename std::conditional<HP, float, __nv_bfloat16>::type;
    OutT* out = static_cast<OutT*>(out_);
    const float nan = __int_as_float(0x7fc00000);
    RgWalk w;
    for (w.init(bt, misci[0], miscll[0], start, end); !w.done; w.next(bt)) {
      const int slot = w.lo == 0 ? 1 : 0;
      for (int j = threadIdx.x; j < w.rows * D; j += blockDim.x) {
        const int rr = j / D, d = j % D;
        if (w.whole()) {
          const int64_t row = int64_t(w.row0 + (w.k << bt.p.pos_log) + (rr >> bt.p.g_log)) * (bt.Hk << bt.p.g_log) +
                              (w.h << bt.p.g_log) + (rr & ((1 << bt.p.g_log) - 1));
          if constexpr (HP) out[row * D + d] = nan;
          else out[row * D + d] = __float2bfloat16_rn(nan);
        } else if (d < 2) {
          part_ml[((int64_t(blockIdx.x) * 2 + slot) * rows_cap + rr) * 2 + d] = d ? nan : INFINITY;
        }
      }
      if (!w.whole() && threadIdx.x == 0)
        rg_record(pieces + 2 * blockIdx.x + slot, w.hi == w.count, w.row0, w.s.n, w.h, w.k);
    }
  }
}

// Joins the pieces of the blocks that were cut: a block's pieces are the second
// place of the CTA where it begins and the first places of the CTAs after it,
// up to the one marked last.
//   m = max m_i, l = sum l_i 2^(m_i - m), out = sum O_i 2^(m_i - m) / l.
// The order of the pieces is that of the tokens, so the result does not depend
// on timing. A CTA takes 32 rows (lane = row), a warp D/8 of the channels; the
// places hold the rows side by side, so a warp's loads are whole lines.
template <int D, typename OutT>
__global__ void __launch_bounds__(256) ragged_merge_kernel(
    const float* part_o, const float* part_ml, const RgPiece* pieces, int n_ctas, int rows_cap,
    RgShape p, int Hq, OutT* __restrict__ out) {
  tc::grid_dep_wait();
  const int c0 = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  RgPiece pc;
  {
    const int4 a = __ldcg(reinterpret_cast<const int4*>(pieces + 2 * c0 + 1));
    const int4 b = __ldcg(reinterpret_cast<const int4*>(pieces + 2 * c0 + 1) + 1);
    pc.valid = a.x; pc.last = a.y; pc.row0 = a.z; pc.n = a.w;
    pc.h = b.x; pc.k = b.y;
  }
  if (!pc.valid) return;
  RgSeq sq;
  sq.n = pc.n;
  sq.ctx = 0;
  const int rows = rg_rows(sq, pc.k, p);
  if (blockIdx.y * 32 >= rows) return;
  // how many pieces follow: up to the first place marked last, 32 CTAs at a time
  int n = 0;
  for (int base = c0 + 1; base < n_ctas; base += 32) {
    const int c = base + lane;
    int2 v = make_int2(0, 0);
    if (c < n_ctas) v = __ldcg(reinterpret_cast<const int2*>(pieces + 2 * c));
    const unsigned stop = __ballot_sync(0xffffffffu, v.x == 0 || v.y != 0);
    if (stop) {
      const int f = __ffs(stop) - 1;
      n += f + (__shfl_sync(0xffffffffu, v.x, f) ? 1 : 0);
      break;
    }
    n += 32;
  }
  const int total = n + 1, rr = blockIdx.y * 32 + lane;
  if (rr >= rows) return;
  auto place = [&](int i) -> int64_t { return int64_t(c0 + i) * 2 + (i == 0 ? 1 : 0); };
  constexpr int NV = D / 8, U = 4;             // channels a thread; pieces in flight
  float o[NV] = {};
  float m = -INFINITY, l = 0.f;
  for (int base = 0; base < total; base += U) {
    float2 ml[U];
    float v[U][NV];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      ml[i] = make_float2(-INFINITY, 0.f);
      if (base + i < total) {
        const int64_t pl = place(base + i);
        ml[i] = __ldcg(reinterpret_cast<const float2*>(part_ml) + pl * rows_cap + rr);
        const float* src = part_o + (pl * D + warp * NV) * rows_cap + rr;
#pragma unroll
        for (int e = 0; e < NV; ++e) v[i][e] = __ldcg(src + int64_t(e) * rows_cap);
      }
    }
    float mn = m;
#pragma unroll
    for (int i = 0; i < U; ++i) mn = fmaxf(mn, ml[i].x);
    const float ref = mn == -INFINITY ? 0.f : mn, keep = exp2f(m - ref);
    m = mn;
    l *= keep;
#pragma unroll
    for (int e = 0; e < NV; ++e) o[e] *= keep;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (base + i < total) {
        const float w = exp2f(ml[i].x - ref);
        l += ml[i].y * w;
#pragma unroll
        for (int e = 0; e < NV; ++e) o[e] += v[i][e] * w;
      }
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int G = 1 << p.g_log;
  OutT* dst = out + (int64_t(pc.row0 + (pc.k << p.pos_log) + (rr >> p.g_log)) * Hq + pc.h * G + (rr & (G - 1))) * D + warp * NV;
  if constexpr (sizeof(OutT) == 4) {
#pragma unroll
    for (int e = 0; e < NV; e += 4)
      *reinterpret_cast<float4*>(dst + e) = make_float4(o[e] * inv, o[e + 1] * inv, o[e + 2] * inv, o[e + 3] * inv);
  } else {
#pragma unroll
    for (int e = 0; e < NV; e += 8)
      *reinterpret_cast<uint4*>(dst + e) =
          make_uint4(rg_pack(o[e] * inv, o[e + 1] * inv), rg_pack(o[e + 2] * inv, o[e + 3] * inv),
                     rg_pack(o[e + 4] * inv, o[e + 5] * inv), rg_pack(o[e + 6] * inv, o[e + 7] * inv));
  }
}

}  // namespace kvq
