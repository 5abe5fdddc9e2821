// Paged K/V cache: what the append and decode kernels share.  Position p of
// sequence b is row p % page_size of page block_table[b, p / page_size]; a
// page of one KV head is a contiguous block of page_size rows
// ([n_pages, Hkv, page_size, D]), which has one scale in the 8-bit cache.
#pragma once
#include "common.cuh"

namespace sk {

struct PagedView {
  void* k_pages;
  void* v_pages;
  float* k_scale;  // [n_pages, Hkv], 8-bit cache only
  float* v_scale;
  const int32_t* table;    // [B, max_pages]
  const int32_t* seqlens;  // [B], the call's new tokens included
  int B, n_pages, page_size, page_log2, max_pages, Hkv;
  int* status;
};

// The paged kernels may be on an SM while the kernel before them still writes what they
// read behind their wait (lengths, tables, scales, queries, even a rotation table): the
// read-only path, __ldg, is for what nobody writes while a kernel lives, and is not used.
// Plain loads cost the same.  Scales, of which other blocks write the neighbours in a
// sector, come from L2 (in the decode; all of these from L2 cost an 8-bit prefill 14 %).
template <class T>
__device__ __forceinline__ T fresh(const T* p) {
  return *p;
}

struct PagedAppendProblem {
  PagedView c;
  int dt, T, Hq, D, rot, n_pos, interleaved;
  const void* k;
  const void* v;
  const void* q;  // or nullptr
  long long k_stride, v_stride, q_stride;  // elements between tokens
  const int32_t* cu;   // [B + 1], or nullptr: one token a sequence
  const float* rope;   // [n_pos, rot]: cos, then sin; or nullptr
  void* q_out;
  void* k_out;  // or nullptr
};
int launch_paged_append(const PagedAppendProblem& p, cudaStream_t stream);
int launch_paged_append_fp8(const PagedAppendProblem& p, cudaStream_t stream);

struct PagedDecodeProblem {
  PagedView c;
  int dt, Hq, D, n_sink, window, fp8;
  float scale;
  const void* q;
  const float* sink;
  void* out;
  float* lse;
  float* sink_s;
  float* part;  // workspace
  int lanes, chunks;  // KV heads that a group of CTAs works on side by side; Hkv / lanes
};
int launch_paged_decode(const PagedDecodeProblem& p, cudaStream_t stream);
size_t paged_decode_part_floats(int B, int Hq, int Hkv, int D, int sms);

constexpr int kPagedMaxGroup = 16;  // query heads per KV head

// ---- the decode's schedule (host and device) --------------------------------
constexpr int kMaxCtas = 320;

// The pages of a sequence that hold visible positions, [0, sp) for the sink tokens
// and then fp, fp + 1, ..., cut into tiles of so many pages: a window's tiles begin at
// its own first page, behind the sink tokens' (so four sink tokens cost a page of a
// tile, not a tile).  There is always a tile, which writes the result of a sequence
// without a key.
struct SeqTiles {
  int n, sp, fp, pages, count;
  SeqTiles() = default;
  // ppt_log2: pages per tile (shifts: every CTA's start waits for this)
  __host__ __device__ SeqTiles(int len, int cap, int n_sink, int window, int page_log2,
                               int ppt_log2) {
    n = len < 0 ? 0 : len > cap ? cap : len;
    const int rest = (1 << page_log2) - 1;
    pages = (n >> page_log2) + ((n & rest) != 0);
    sp = pages;
    fp = 0;
    const int w0 = n - window;  // first position of the window
    if (window > 0 && w0 > n_sink) {
      sp = (n_sink >> page_log2) + ((n_sink & rest) != 0);
      fp = w0 >> page_log2 > sp ? w0 >> page_log2 : sp;
      pages = sp + pages - fp;
    }
    count = (pages >> ppt_log2) + ((pages & ((1 << ppt_log2) - 1)) != 0);
    if (count < 1) count = 1;
  }
  // the i-th of the pages
  __host__ __device__ int page(int i) const { return i < sp ? i : fp + i - sp; }
};

// A (sequence, KV head) pair is worth its tiles and kPairUnits more, for what its
// ends cost (queries, first references, result) whatever its length: with 1 a
// StreamingLLM band over unequal lengths takes 25 us, with 0 30; 2 gives nothing.
constexpr int kPairUnits = 1;

// CTA i of n takes `per` units, the first `more` CTAs one more; with fewer units
// than CTAs the first ones take one each, so that a pair's CTAs are consecutive.
// (Units are counted in 32 bits, which the host has checked: a 64-bit division is a
// long subroutine, and every CTA's start waits for it.)
struct Runs {
  int per, more;
  __host__ __device__ Runs(int total, int n) : per(total / n), more(total % n) {}
  __host__ __device__ int begin(int i) const { return i * per + (i < more ? i : more); }
  __host__ __device__ int cta_of(int unit) const {
    const int fat = more * (per + 1);
    return unit < fat ? unit / (per + 1) : more + (unit - fat) / per;
  }
};

// CTAs work in groups, one KV head each of the same tiles: the largest divisor of Hkv
// up to 8.
constexpr int kMaxLanes = 8;
__host__ __device__ inline int group_lanes(int Hkv) {
  int n = Hkv < kMaxLanes ? Hkv : kMaxLanes;
  while (Hkv % n != 0) --n;
  return n;
}

// Whether every row of the schedule is left whole, to a group of its own (no partials, no
// join), given the groups' even share: a cut costs two ends, and a lone CTA on an SM is
// faster than two.  Break-even, measured over 4 to 37 equal sequences of 8 KV heads, lies
// at rows longer by 3 to 4 units, and by 6 where two CTAs with a tile row a position
// share an SM; 32 sequences of 1,024 tokens in 8 bits take 18 us so and 21 evenly cut.
__host__ __device__ inline bool rows_whole(int rows, int longest, int share, int groups, int slack) {
  return rows <= groups && longest <= share + share / 8 + (share + 3 < slack ? share + 3 : slack);
}

// Groups of a grid of at most `ctas` CTAs: no more than the tables have units.
__host__ __device__ inline int schedule_groups(long long units, int ctas, int lanes) {
  const int most = (ctas < kMaxCtas ? ctas : kMaxCtas) / lanes;
  return units < most ? (int)units : most;
}

// A row of the schedule is a sequence's tiles for a chunk of `lanes` KV heads.  A CTA's
// run of units is walked segment by segment; seq_of(b) gives the tiles of sequence b.
struct Walk {
  int b, kvh, t0, cnt;  // the segment: tiles [t0, t0 + cnt) of (b, kvh)
  SeqTiles seq;
  int left;             // units of the run from the segment on
  __host__ __device__ void cut() { cnt = seq.count - t0 < left ? seq.count - t0 : left; }
  // a run that begins behind a row's tiles begins with the next row
  template <class F>
  __host__ __device__ bool begin(int Hkv, int lanes, F seq_of) {
    return left > 0 && (cnt > 0 || next(Hkv, lanes, seq_of));
  }
  template <class F>
  __host__ __device__ bool next(int Hkv, int lanes, F seq_of) {
    left -= seq.count + kPairUnits - t0;
    if (left <= 0) return false;
    t0 = 0;
    if ((kvh += lanes) >= Hkv) {
      kvh -= Hkv;
      seq = seq_of(++b);
    }
    cut();
    return true;
  }
};
// The run of CTA `lane` of a group that has row `group` to itself (none: left = 0).
template <class F>
__host__ __device__ inline Walk whole_walk(int group, int lane, int B, int lanes, int chunks,
                                           F seq_of) {
  Walk w;
  w.b = group / chunks;
  w.kvh = (group - w.b * chunks) * lanes + lane;
  w.t0 = w.left = 0;
  if (w.b < B) {
    w.seq = seq_of(w.b);
    w.left = w.seq.count + kPairUnits;
    w.cut();
  }
  return w;
}
// The run of `units` units from f0 on, which lies at or behind unit `before`, the first of
// sequence b.
template <class F>
__host__ __device__ inline Walk cut_walk(int f0, int units, int b, int before, int lane, int lanes,
                                         int chunks, F seq_of) {
  Walk w;
  w.b = b;
  for (;;) {
    w.seq = seq_of(w.b);
    const int of_all = (w.seq.count + kPairUnits) * chunks;
    if (f0 < before + of_all) break;
    before += of_all;
    ++w.b;
  }
  const int rem = f0 - before, row = w.seq.count + kPairUnits;
  const int chunk = rem / row;
  w.kvh = chunk * lanes + lane;
  w.t0 = rem - chunk * row;
  w.left = units;
  w.cut();
  return w;
}
// Groups that have a part of a row's tiles, whose first unit `first` lies in group `group`.
__host__ __device__ inline int parts_of(const Runs& runs, int group, int first, int tiles) {
  return runs.cta_of(first + tiles - 1) - group + 1;
}
// Partials of pair (b, kvh) = b Hkv + kvh: rows come in order along the groups, so no two
// segments share a slot.
__host__ __device__ inline long long part_slot(long long pair, int group, int lanes) {
  return pair + group * lanes;
}
__host__ __device__ inline long long part_slots(long long pairs, int sms) {
  return pairs + (2 * sms < kMaxCtas ? 2 * sms : kMaxCtas);
}

}  // namespace sk
