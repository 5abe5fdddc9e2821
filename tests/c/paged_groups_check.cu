// Host-only check of the paged decode's schedule of CTA groups (no kernel is launched), by
// the functions that the kernels call: for many batches every CTA's run is walked as its
// roles walk it.  Each visible position of each (sequence, KV head) lies in exactly one
// tile of one segment; the segments' partial slots are distinct and inside the workspace;
// the join, which derives a pair's segments for itself, finds the groups that have one, and
// a segment that holds all of its row is the only one.  Rows left whole and rows cut, both
// sides of the rule between them.  Prints "ok" or the first failure.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "../../learnable_sink_b200/csrc/paged.cuh"

using namespace sk;

#define CHECK(x, what)                                                                       \
  if (!(x)) return std::printf("round %d: %s\n", round, what), 1

int main() {
  std::srand(11);
  long long checked = 0;
  int whole_rounds = 0, cut_rounds = 0, near[2] = {0, 0}, idle_rounds = 0;
  const int heads[] = {1, 2, 3, 5, 8, 9, 10, 11, 16, 24, 40};
  const int sm_counts[] = {148, 148, 148, 132, 160, 200};
  for (int round = 0; round < 1500; ++round) {
    const int Hkv = heads[std::rand() % 11], lanes = group_lanes(Hkv), chunks = Hkv / lanes;
    CHECK(lanes >= 1 && lanes <= kMaxLanes && lanes * chunks == Hkv, "lanes");
    const int sms = sm_counts[std::rand() % 6], per_sm = 1 + std::rand() % 2;
    const int slack = per_sm == 2 && std::rand() % 2 ? 6 : 3;
    const int tp = std::rand() % 2 ? 128 : 256, lg = 4 + std::rand() % 4;
    const int ppt = tp >> lg, pl = (tp == 128 ? 7 : 8) - lg;
    const int max_pages = 1 + std::rand() % (4000 >> lg), cap = max_pages << lg;
    const int kind = std::rand() % 4;  // unequal, equal, about equal, many
    const int B = kind == 3 ? 100 + std::rand() % 200 : 1 + std::rand() % (kind == 0 ? 12 : 40);
    const int n_sink = std::rand() % 3 ? 0 : std::rand() % 300;
    const int window = std::rand() % 4 ? 0 : 1 + std::rand() % 2000;
    std::vector<int> len(B);
    const int base = std::rand() % (cap + 1);
    for (int& n : len)
      n = kind == 1 ? base : kind == 2 ? base - std::rand() % (tp * 4) : std::rand() % (cap + 200) - 20;
    auto seq_of = [&](int b) { return SeqTiles(len[b], cap, n_sink, window, lg, pl); };

    // what the host launches
    const long long most = ((long long)cap + tp - 1) / tp + kPairUnits;
    const int groups = schedule_groups(most * B * chunks, per_sm * sms, lanes);
    CHECK(groups >= 1 && groups * lanes <= kMaxCtas, "groups");
    const long long pairs = (long long)B * Hkv, slots = part_slots(pairs, sms);

    // what every CTA adds up
    std::vector<int> before(B + 1, 0);
    int longest = 0;
    for (int b = 0; b < B; ++b) {
      const int units = seq_of(b).count + kPairUnits;
      CHECK(units <= most, "more tiles than the table has");
      before[b + 1] = before[b] + units * chunks;
      longest = units > longest ? units : longest;
    }
    const int total = before[B];
    const Runs runs(total, groups);
    CHECK(runs.begin(0) == 0 && runs.begin(groups) == total, "runs do not cover");
    const bool whole = rows_whole(B * chunks, longest, runs.per, groups, slack);
    (whole ? whole_rounds : cut_rounds) += 1;
    if (B * chunks <= groups && !whole) ++near[0];
    if (whole && longest > runs.per) ++near[1];
    if (total < groups) ++idle_rounds;

    std::vector<std::vector<char>> seen((size_t)pairs, std::vector<char>(cap, 0));
    std::vector<char> slot((size_t)slots, 0);
    std::vector<int> begun((size_t)pairs, -1), had((size_t)pairs, 0), alone((size_t)pairs, 0);
    const int slice = 1 + std::rand() % 3;  // sequences that a thread adds up
    for (int g = 0; g < groups; ++g)
      for (int lane = 0; lane < lanes; ++lane) {
        Walk w;
        const int f0 = runs.begin(g), units = runs.begin(g + 1) - f0;
        if (whole) {
          w = whole_walk(g, lane, B, lanes, chunks, seq_of);
        } else if (f0 == total) {
          w.left = 0;
        } else {
          int b = 0;
          while (before[b + 1] <= f0) ++b;
          b = b / slice * slice;
          w = cut_walk(f0, units, b, before[b], lane, lanes, chunks, seq_of);
        }
        const int run = w.left;
        if (!w.begin(Hkv, lanes, seq_of)) continue;
        do {
          CHECK(w.b >= 0 && w.b < B && w.kvh >= 0 && w.kvh < Hkv && w.kvh % lanes == lane, "pair");
          CHECK(w.t0 >= 0 && w.cnt >= 1 && w.t0 + w.cnt <= w.seq.count, "tiles");
          const size_t pair = (size_t)w.b * Hkv + w.kvh;
          if (w.t0 == 0) {  // what the decode kernel notes for the join
            const int first = f0 + run - w.left;
            begun[pair] = g;
            const int parts = whole ? 1 : parts_of(runs, g, first, w.seq.count);
            CHECK(parts >= 1 && parts <= kMaxCtas, "parts");
            had[pair] -= parts;
          }
          CHECK(begun[pair] >= 0, "a later segment before the first");
          alone[pair] += w.cnt == w.seq.count;
          ++had[pair];
          const long long at = part_slot((long long)pair, g, lanes);
          CHECK(at >= 0 && at < slots && !slot[at], "partial slot");
          slot[at] = 1;
          for (int k = w.t0 * ppt; k < (w.t0 + w.cnt) * ppt && k < w.seq.pages; ++k) {
            const long long row = (long long)w.seq.page(k) << lg;
            CHECK(row >= 0 && row + (1 << lg) <= cap, "page outside the table");
            for (int i = 0; i < 1 << lg; ++i) ++seen[pair][row + i];
          }
        } while (w.next(Hkv, lanes, seq_of));
      }

    for (int b = 0; b < B; ++b)
      for (int h = 0; h < Hkv; ++h) {
        const size_t pair = (size_t)b * Hkv + h;
        CHECK(begun[pair] >= 0 && had[pair] == 0, "a pair's segments are not those announced");
        // what the join finds from the lengths
        const int units = seq_of(b).count + kPairUnits;
        int first_group = 0, parts = 0;
        if (!whole) {
          const int first = before[b] + (chunks == 1 ? 0 : h / lanes * units);
          first_group = runs.cta_of(first);
          parts = parts_of(runs, first_group, first, units - kPairUnits);
          CHECK(first_group == begun[pair], "the join's first group");
          for (int i = 0; i < parts; ++i) {
            const long long at = part_slot((long long)pair, first_group + i, lanes);
            CHECK(at < slots && slot[at], "the join reads a slot that nobody has");
          }
        }
        CHECK(alone[pair] == (parts <= 1), "who writes the result");
        const int n = len[b] < 0 ? 0 : len[b] > cap ? cap : len[b];
        for (int j = 0; j < cap; ++j) {
          const bool vis = j < n && (window <= 0 || j < n_sink || j >= n - window);
          CHECK(seen[pair][j] <= 1 && (!vis || seen[pair][j] == 1), "a position's tiles");
          ++checked;
        }
      }
  }
  const int round = -1;
  CHECK(whole_rounds > 100 && cut_rounds > 100 && near[0] > 100 && near[1] > 50 && idle_rounds > 0,
        "the batches do not reach every kind of schedule");
  std::printf("ok %lld (%d whole, %d cut; %d %d %d)\n", checked, whole_rounds, cut_rounds, near[0],
              near[1], idle_rounds);
  return 0;
}
