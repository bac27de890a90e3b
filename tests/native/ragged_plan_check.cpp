// Host check of csrc/kvq_ragged_plan.h: the work list of the ragged attention
// kernel on random batches. Restates the kernel's walk (a CTA finds its first
// block from the cost position of its share and takes the pieces that follow)
// and compares it with a list built block by block.
//   usage: ragged_plan_check <seed> <cases>; prints "ok <pieces> <cut blocks>".
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <map>
#include <random>
#include <tuple>
#include <vector>

#include "kvq_ragged_plan.h"

using namespace kvq;

#define CHECK(x)                                                       \
  do {                                                                 \
    if (!(x)) {                                                        \
      std::printf("line %d: %s (case %d)\n", __LINE__, #x, g_case);    \
      std::exit(1);                                                    \
    }                                                                  \
  } while (0)
static int g_case = 0;

struct Piece {
  int cta, lo, hi, count;
};

int main(int argc, char** argv) {
  std::mt19937_64 rng(argc > 1 ? std::strtoull(argv[1], nullptr, 10) : 1);
  const int cases = argc > 2 ? std::atoi(argv[2]) : 1000;
  auto pick = [&](long long lo, long long hi) { return lo + (long long)(rng() % (unsigned long long)(hi - lo + 1)); };
  long long n_pieces = 0, n_cut = 0;
  for (g_case = 0; g_case < cases; ++g_case) {
    const int Bs[] = {1, 2, 3, 16, 64, 130};
    const int grids[] = {1, 3, 148};
    const int B = Bs[pick(0, 5)], Hk = int(pick(1, 8)), grid = grids[pick(0, 2)];
    RgShape p;
    p.g_log = int(pick(0, 3));
    p.pos_log = (pick(0, 3) ? 8 : 7) - p.g_log;
    const int max_ctx = int(pick(1, 1) + pick(0, 1) * pick(0, 200) + pick(0, 1) * pick(0, 6000));
    p.window = pick(0, 2) ? 0 : int(pick(1, max_ctx));
    if (p.window >= max_ctx) p.window = 0;               // as the host does
    std::vector<RgSeq> seqs(B);
    for (auto& s : seqs) {
      s.ctx = int(pick(0, max_ctx));
      const int kind = int(pick(0, 4));
      s.n = kind == 0 ? 0 : kind == 1 ? 1 : kind == 2 ? int(pick(0, 40)) : int(pick(0, s.ctx + (pick(0, 9) ? 0 : 300)));
    }
    // ---- the list, block by block
    struct Blk {
      int b, h, k, first, count, w;
      long long pos;
    };
    std::vector<Blk> list;
    long long pos = 0;
    std::vector<long long> cost(B);
    for (int b = 0; b < B; ++b) {
      const RgSeq& s = seqs[b];
      const int nb = rg_blocks(s, p), P = 1 << p.pos_log;
      CHECK(nb == (s.n + P - 1) / P);
      long long one = 0;
      for (int h = 0; h < Hk; ++h) {
        one = 0;
        for (int k = 0; k < nb; ++k) {
          int first, count;
          rg_block(s, k, p, &first, &count);
          // every token that a row of the block attends lies in the steps
          const int base = s.ctx - s.n, j1 = std::min(s.n, (k + 1) * P);
          int lo = 1 << 30, hi = -1;
          for (int j = k * P; j < j1; ++j) {
            const int at = base + j;
            if (at < 0) continue;
            lo = std::min(lo, p.window ? std::max(0, at - p.window + 1) : 0);
            hi = std::max(hi, at);
          }
          if (hi < 0) {
            CHECK(count == 0);
          } else {
            CHECK(first * kRgStep <= lo && hi < (first + count) * kRgStep);
            CHECK(hi >= (first + count - 1) * kRgStep);   // no step too many behind
          }
          const int rows = rg_rows(s, k, p), w = rows > 128 ? 2 : 1;
          CHECK(rows == ((j1 - k * P) << p.g_log) && rows <= (1 << (p.pos_log + p.g_log)));
          const long long c = kRgPiece + (long long)w * count;
          CHECK(rg_block_cost(s, k, p) == c);
          if (k < nb - 1 || (s.n & (P - 1)) == 0) {       // full blocks: the closed form
            CHECK(rg_prefix(s, k, p) == one);
            if (h == 0) CHECK(rg_find(s, one, p) == k || k == nb);
            if (h == 0) CHECK(rg_find(s, one + c - 1, p) == k);
          }
          list.push_back({b, h, k, first, count, w, pos});
          pos += c;
          one += c;
        }
      }
      cost[b] = one;
      CHECK(rg_cost(s, p) == one);
    }
    const long long all = pos;
    if (all == 0) continue;
    const long long N = std::min<long long>(grid, std::max<long long>(1, all / kRgMinShare));
    // ---- the walk of each CTA
    std::map<std::tuple<int, int, int>, std::vector<Piece>> got;
    for (int c = 0; c < N; ++c) {
      const long long start = c * all / N, end = (c + 1) * all / N;
      long long P0 = 0;
      int b = 0;
      while (!(cost[b] > 0 && P0 * Hk <= start && start < (P0 + cost[b]) * Hk)) {
        P0 += cost[b++];
        CHECK(b < B);
      }
      long long off = start - P0 * Hk;
      int h = 0;
      for (; off >= cost[b]; ++h) off -= cost[b];
      CHECK(h < Hk);
      int nb = rg_blocks(seqs[b], p);
      int k = nb > 1 ? rg_find(seqs[b], off, p) : 0;
      long long at = start - off + (k > 0 ? rg_prefix(seqs[b], k, p) : 0);
      int first_places = 0, last_places = 0;
      while (at < end) {
        int first, count, lo, hi;
        rg_block(seqs[b], k, p, &first, &count);
        const int w = rg_rows(seqs[b], k, p) > 128 ? 2 : 1;
        if (rg_piece(at, count, w, start, end, &lo, &hi)) {
          got[{b, h, k}].push_back({c, lo, hi, count});
          ++n_pieces;
          if (!(lo == 0 && hi == count)) ++(lo == 0 ? last_places : first_places);
        }
        at += kRgPiece + (long long)w * count;
        if (++k < nb) continue;
        k = 0;
        if (++h < Hk) continue;
        h = 0;
        do ++b; while (b < B && rg_blocks(seqs[b], p) == 0);
        if (b == B) break;
        nb = rg_blocks(seqs[b], p);
      }
      CHECK(first_places <= 1 && last_places <= 1);       // one place each in the workspace
    }
    // ---- every block once, its pieces in adjacent CTAs
    CHECK(got.size() == list.size());
    for (const Blk& x : list) {
      const auto& v = got[{x.b, x.h, x.k}];
      CHECK(!v.empty() && v.front().lo == 0 && v.back().hi == x.count);
      for (size_t i = 1; i < v.size(); ++i) CHECK(v[i].lo == v[i - 1].hi && v[i].cta == v[i - 1].cta + 1 && v[i].hi > v[i].lo);
      if (v.size() > 1) {
        ++n_cut;
        CHECK(v.front().hi > 0);
      }
    }
  }
  std::printf("ok %lld %lld\n", n_pieces, n_cut);
  return 0;
}
