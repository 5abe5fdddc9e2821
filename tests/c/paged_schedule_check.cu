// Host-only check of the paged decode's schedule (no kernel is launched): over many
// batches, every CTA's run is walked as the kernel walks it.  Each visible position of
// each (sequence, KV head) lies in exactly one tile of one segment, the segments'
// partial slots pair + CTA are distinct and inside the workspace, and a pair's
// segments are the consecutive CTAs that its first one announces.  Prints "ok" or the
// first failure.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "../../learnable_sink_b200/csrc/paged.cuh"

using sk::kPairUnits;
using sk::Runs;
using sk::SeqTiles;

int main() {
  std::srand(5);
  long long checked = 0;
  const int grids[] = {1, 7, 148, 296, 320};
  for (int round = 0; round < 400; ++round) {
    const int B = 1 + std::rand() % (round % 5 == 0 ? 300 : 9), Hkv = 1 + std::rand() % 5;
    const int tp = round % 2 ? 128 : 256, cap = 128 * (1 + std::rand() % 40);
    const int lg = 4 + std::rand() % 4, ppt = tp >> lg, pl = (tp == 128 ? 7 : 8) - lg;
    const int n_sink = round % 3 ? 0 : std::rand() % 300, window = round % 4 ? 0 : 1 + std::rand() % 2000;
    std::vector<int> len(B);
    for (int& n : len) n = std::rand() % (cap + 200) - 20;
    const int n_cta = grids[round % 5];
    long long total = 0;
    std::vector<long long> first(B);
    for (int b = 0; b < B; ++b) {
      first[b] = total;
      total += (long long)Hkv * (SeqTiles(len[b], cap, n_sink, window, lg, pl).count + kPairUnits);
    }
    const Runs runs((int)total, n_cta);
    if (runs.begin(0) != 0 || runs.begin(n_cta) != total) return std::printf("runs do not cover\n"), 1;
    std::vector<std::vector<char>> seen((size_t)B * Hkv);
    std::vector<int> next_cta((size_t)B * Hkv, -1), left((size_t)B * Hkv, -1);
    std::vector<char> slot((size_t)B * Hkv + n_cta, 0);
    for (int c = 0; c < n_cta; ++c) {
      long long u = runs.begin(c);
      const long long end = runs.begin(c + 1);
      while (u < end) {
        int b = 0;
        while (b + 1 < B && first[b + 1] <= u) ++b;
        const SeqTiles s(len[b], cap, n_sink, window, lg, pl);
        const int units = s.count + kPairUnits, rem = (int)(u - first[b]);
        const int kvh = rem / units, t0 = rem % units;
        const size_t pair = (size_t)b * Hkv + kvh;
        const int cnt = (int)((end - u) < s.count - t0 ? end - u : s.count - t0);
        if (cnt > 0) {
          if (t0 == 0) {
            next_cta[pair] = c;
            left[pair] = runs.cta_of((int)u + s.count - 1) - c + 1;
          }
          if (next_cta[pair] != c || left[pair] < 1) return std::printf("segment not announced\n"), 1;
          ++next_cta[pair];
          --left[pair];
          if (pair + c >= slot.size() || slot[pair + c]) return std::printf("partial slot\n"), 1;
          slot[pair + c] = 1;
          seen[pair].resize((size_t)cap);
          for (int k = t0 * ppt; k < (t0 + cnt) * ppt && k < s.pages; ++k) {
            const long long at = (long long)s.page(k) << lg;
            if (at < 0 || at + (1 << lg) > cap) return std::printf("page outside the table\n"), 1;
            for (int i = 0; i < 1 << lg; ++i) ++seen[pair][at + i];
          }
        }
        u += units - t0;
        if (u > end) u = end;
      }
    }
    for (int b = 0; b < B; ++b)
      for (int h = 0; h < Hkv; ++h) {
        const size_t pair = (size_t)b * Hkv + h;
        if (left[pair] != 0) return std::printf("a pair has no segment, or too few\n"), 1;
        const int n = len[b] < 0 ? 0 : len[b] > cap ? cap : len[b];
        for (int j = 0; j < (int)seen[pair].size(); ++j) {
          const bool vis = j < n && (window <= 0 || j < n_sink || j >= n - window);
          if (seen[pair][j] > 1 || (vis && seen[pair][j] != 1))
            return std::printf("position %d of length %d covered %d times\n", j, n, seen[pair][j]), 1;
          ++checked;
        }
      }
  }
  std::printf("ok %lld\n", checked);
  return 0;
}
