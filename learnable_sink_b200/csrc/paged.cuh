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
};
int launch_paged_decode(const PagedDecodeProblem& p, cudaStream_t stream);
size_t paged_decode_part_floats(int B, int Hq, int Hkv, int D, int sms);

constexpr int kPagedMaxGroup = 16;  // query heads per KV head

// ---- the decode's schedule (host and device) --------------------------------
constexpr int kMaxCtas = 320;

// The tiles (of tp positions) of a sequence of length n that hold visible
// positions: [0, ts), then f, f + 1, ...; never none, so that a sequence without a
// key still has a (masked) tile, which writes its result.
struct SeqTiles {
  int n, ts, f, count;
  SeqTiles() = default;
  __host__ __device__ SeqTiles(int len, int cap, int n_sink, int window, int tp) {
    n = len < 0 ? 0 : len > cap ? cap : len;
    const int all = n / tp + (n % tp != 0);
    ts = all > 1 ? all : 1;
    f = 0;
    count = ts;
    const int w0 = n - window;  // first position of the window
    if (window > 0 && w0 > n_sink) {
      ts = n_sink / tp + (n_sink % tp != 0);
      f = w0 / tp > ts ? w0 / tp : ts;
      count = ts + all - f;
    }
  }
  __host__ __device__ int tile(int i) const { return i < ts ? i : f + i - ts; }
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

}  // namespace sk
