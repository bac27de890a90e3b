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

// The shape of a block: pos = 1 << pos_log tokens of the sequence's new ones, G = 1 << g_log
// query heads each. All sizes are powers of two, so that the list needs no division.
struct RgShape {
  int pos_log, g_log, window;
};

// Steps [first, first + count) that block k reads: tokens from the first row's
// window (window 0: all) to the last row's own position.
KVQ_HD void rg_block(const RgSeq& s, int k, const RgShape& p, int* first, int* count) {
  const int base = s.ctx - s.n;
  const int j0 = k << p.pos_log;
  const int j1 = s.n - j0 < (1 << p.pos_log) ? s.n : j0 + (1 << p.pos_log);
  const int end = base + j1;
  if (end <= 0) {
    *first = *count = 0;
    return;
  }
  int beg = p.window > 0 ? base + j0 + 1 - p.window : 0;
  if (beg < 0) beg = 0;
  *first = beg >> 6;
  *count = ((end - 1) >> 6) + 1 - *first;
}

KVQ_HD int rg_rows(const RgSeq& s, int k, const RgShape& p) {
  const int left = s.n - (k << p.pos_log);
  return (left < (1 << p.pos_log) ? left : 1 << p.pos_log) << p.g_log;
}

// Q(n) = sum of ceil(i / 2^r) over i = 1 .. n.
KVQ_HD long long rg_q(long long n, int r) {
  const long long q = n >> r;
  return ((q * (q + 1) / 2) << r) + (n - (q << r)) * (q + 1);
}

// sum over k < m of ceil(max(0, a + (k << pos_log)) / 64).
KVQ_HD long long rg_sum_ceil(int a, int pos_log, long long m) {
  const long long k1 = a > 0 ? 0 : ((-(long long)a) >> pos_log) + 1;   // first positive term
  if (k1 >= m) return 0;
  const long long x = a + (k1 << pos_log), c = m - k1;
  if (pos_log >= 6) return c * ((x + 63) >> 6) + ((c * (c - 1) / 2) << (pos_log - 6));
  // ceil((x + (k << pos_log)) / 64) = ceil((h + k) / 2^r)
  const int r = 6 - pos_log;
  const long long h = (x + (1 << pos_log) - 1) >> pos_log;
  return rg_q(h + c - 1, r) - rg_q(h - 1, r);
}

// Cost of blocks 0 .. k-1 of a sequence, all of them full (k < number of blocks).
KVQ_HD long long rg_prefix(const RgSeq& s, int k, const RgShape& p) {
  const int base = s.ctx - s.n;
  long long steps = rg_sum_ceil(base + (1 << p.pos_log), p.pos_log, k);
  // floor(x / 64) = ceil((x - 63) / 64)
  if (p.window > 0) steps -= rg_sum_ceil(base + 1 - p.window - (kRgStep - 1), p.pos_log, k);
  return (long long)k * kRgPiece + (steps << (p.pos_log + p.g_log > 7 ? 1 : 0));
}

KVQ_HD int rg_blocks(const RgSeq& s, const RgShape& p) { return int(((long long)s.n + (1 << p.pos_log) - 1) >> p.pos_log); }

KVQ_HD long long rg_block_cost(const RgSeq& s, int k, const RgShape& p) {
  int first, count;
  rg_block(s, k, p, &first, &count);
  return kRgPiece + (rg_rows(s, k, p) > 128 ? 2LL : 1LL) * count;
}

// Cost of all blocks of one (sequence, KV head).
KVQ_HD long long rg_cost(const RgSeq& s, const RgShape& p) {
  const int nb = rg_blocks(s, p);
  if (nb == 0) return 0;
  return (nb > 1 ? rg_prefix(s, nb - 1, p) : 0) + rg_block_cost(s, nb - 1, p);
}

// The block that holds cost position x of the (sequence, KV head)'s blocks.
KVQ_HD int rg_find(const RgSeq& s, long long x, const RgShape& p) {
  int lo = 0, hi = rg_blocks(s, p);                     // prefix(lo) <= x < prefix(hi)
  while (hi - lo > 1) {
    const int mid = lo + (hi - lo) / 2;
    if (rg_prefix(s, mid, p) <= x) lo = mid;
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
