// Work list of the ragged attention kernel, in integers shared by the kernel
// and its host test.
//
// The query rows of one (sequence, KV head) are its n new tokens times the G
// query heads of the head, token by token: row = token * G + g. They are taken
// in blocks of `rpb` rows (256, or 128); a block reads the cached tokens that
// any of its rows attends, in steps of 64. The list is every (sequence, KV
// head, block) in that order; a block costs kRgPiece units (opening and closing
// it) plus 1 or 2 units a step (2 when it holds more than 128 rows, twice the
// products). A CTA takes an equal, contiguous share of the total cost and with
// it the steps whose first unit lies in the share; a block may thus be cut
// into pieces, which a second kernel joins.
#pragma once

#if defined(__CUDACC__)
#define KVQ_HD __host__ __device__ __forceinline__
#else
#define KVQ_HD inline
#endif

namespace kvq {

constexpr int kRgStep = 64;      // tokens per step
constexpr int kRgPiece = 6;      // cost of opening and closing a block's piece
constexpr int kRgMinShare = 12;  // smallest share of a CTA (above 2, so that a cut
                                 // block continues in the next CTA)

// The new tokens of one sequence: n of them, the last of its ctx tokens.
struct RgSeq {
  int n, ctx;
};

// Steps [first, first + count) that block k reads: tokens from the first row's
// window (window 0: all) to the last row's own position.
KVQ_HD void rg_block(const RgSeq& s, int k, int pos_per_block, int window, int* first, int* count) {
  const int base = s.ctx - s.n;
  const int j0 = k * pos_per_block;
  const int j1 = s.n - j0 < pos_per_block ? s.n : j0 + pos_per_block;
  const int end = base + j1;
  if (end <= 0) {
    *first = *count = 0;
    return;
  }
  int beg = window > 0 ? base + j0 + 1 - window : 0;
  if (beg < 0) beg = 0;
  *first = beg / kRgStep;
  *count = (end - 1) / kRgStep + 1 - *first;
}

KVQ_HD int rg_rows(const RgSeq& s, int k, int pos_per_block, int G) {
  const int left = s.n - k * pos_per_block;
  return (left < pos_per_block ? left : pos_per_block) * G;
}

// sum over k < m of ceil(max(0, a + k P) / 64); P divides 64 or is a multiple of it.
KVQ_HD long long rg_sum_ceil(int a, int P, long long m) {
  long long k1 = a > 0 ? 0 : (-(long long)a) / P + 1;   // first positive term
  if (k1 >= m) return 0;
  const long long x = a + k1 * P, c = m - k1;
  if (P >= kRgStep) return c * ((x + kRgStep - 1) / kRgStep) + (P / kRgStep) * (c * (c - 1) / 2);
  const long long r = kRgStep / P, h = (x + P - 1) / P;
  // ceil((x + k P) / 64) = ceil((h + k) / r); Q(n) = sum of ceil(i / r), i = 1 .. n
  const long long n1 = h + c - 1, n0 = h - 1;
  const long long q1 = n1 / r, q0 = n0 / r;
  return (r * (q1 * (q1 + 1) / 2) + (n1 % r) * (q1 + 1)) - (r * (q0 * (q0 + 1) / 2) + (n0 % r) * (q0 + 1));
}

// Cost of blocks 0 .. k-1 of a sequence, all of them full (k < number of blocks).
KVQ_HD long long rg_prefix(const RgSeq& s, int k, int pos_per_block, int G, int window) {
  const int base = s.ctx - s.n;
  const int w = pos_per_block * G > 128 ? 2 : 1;
  long long steps = rg_sum_ceil(base + pos_per_block, pos_per_block, k);
  // floor(x / 64) = ceil((x - 63) / 64)
  if (window > 0) steps -= rg_sum_ceil(base + 1 - window - (kRgStep - 1), pos_per_block, k);
  return (long long)k * kRgPiece + w * steps;
}

KVQ_HD int rg_blocks(const RgSeq& s, int pos_per_block) { return (s.n + pos_per_block - 1) / pos_per_block; }

KVQ_HD long long rg_block_cost(const RgSeq& s, int k, int pos_per_block, int G, int window) {
  int first, count;
  rg_block(s, k, pos_per_block, window, &first, &count);
  return kRgPiece + (long long)(rg_rows(s, k, pos_per_block, G) > 128 ? 2 : 1) * count;
}

// Cost of all blocks of one (sequence, KV head).
KVQ_HD long long rg_cost(const RgSeq& s, int pos_per_block, int G, int window) {
  const int nb = rg_blocks(s, pos_per_block);
  if (nb == 0) return 0;
  return rg_prefix(s, nb - 1, pos_per_block, G, window) + rg_block_cost(s, nb - 1, pos_per_block, G, window);
}

// The block that holds cost position x of the (sequence, KV head)'s blocks.
KVQ_HD int rg_find(const RgSeq& s, long long x, int pos_per_block, int G, int window) {
  int lo = 0, hi = rg_blocks(s, pos_per_block);         // prefix(lo) <= x < prefix(hi)
  while (hi - lo > 1) {
    const int mid = lo + (hi - lo) / 2;
    if (rg_prefix(s, mid, pos_per_block, G, window) <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Steps [lo, hi) of a block's `count` that a share [start, end) holds, the block
// beginning at cost position pos. True if the share has a piece of the block:
// for a block without steps, the share that holds its first unit.
KVQ_HD bool rg_piece(long long pos, int count, int w, long long start, long long end, int* lo, int* hi) {
  if (count == 0) {
    *lo = *hi = 0;
    return start <= pos && pos < end;
  }
  long long a = start - pos - kRgPiece, b = end - pos - kRgPiece;
  a = a <= 0 ? 0 : (a + w - 1) >> (w - 1);               // w is 1 or 2
  b = b <= 0 ? 0 : (b + w - 1) >> (w - 1);
  if (a > count) a = count;
  if (b > count) b = count;
  *lo = int(a);
  *hi = int(b);
  return a < b;
}

}  // namespace kvq
