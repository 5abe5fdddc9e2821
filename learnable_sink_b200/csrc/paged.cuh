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

}  // namespace sk
