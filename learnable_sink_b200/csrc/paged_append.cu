// Appending keys and values to a paged cache, the position rotation applied on
// the way.
//
// A token's position is p = cache_seqlens[b] - n_b + i (the i-th of the n_b new
// tokens of sequence b; cache_seqlens counts them).  With c_i, s_i the cosine
// and sine of the position's i-th angle (a float32 table [n_pos, rot]: cosines,
// then sines), the pair (a, b) of a key or query becomes
//   a' = a c - b s,   b' = b c + a s,
// pairs being elements (i, i + rot/2), or (2i, 2i + 1) when interleaved; the
// elements past rot are copied.  16-bit results are rounded once, from float32.
//
// 8-bit cache: a block (page, KV head) holds E4M3 codes of value / s.  s is a
// power of two, the smallest 2^e (e >= -126) with amax <= 448 2^e over the
// finite magnitudes written to the block, 0 while they are all 0.  A power of
// two makes the product code * s exact in 16 bits, and moving a block's earlier
// codes to a larger scale exact but for codes that become subnormal.
#include <cuda_fp8.h>

#include "internal.h"
#include "paged.cuh"

namespace sk {

namespace {

// Sequence of packed token t: the last b with cu[b] <= t (32-way search by the
// lanes of a warp: one load a step for up to 32 sequences).
__device__ __forceinline__ int find_sequence(const int32_t* cu, int B, int t, int lane) {
  int lo = 0, n = B;  // the answer is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int i = lane * step;
    const bool le = i < n && fresh(cu + lo + i) <= t;
    const int hit = __popc(__ballot_sync(0xffffffffu, le));
    const int skip = hit > 0 ? (hit - 1) * step : 0;
    lo += skip;
    n = min(step, n - skip);
  }
  return lo;
}

// Page id of position `pos` of sequence b, or -1 with the status set when the
// table's row does not reach it or names no page of the pool.
__device__ __forceinline__ int page_of(const PagedView& c, int b, int page_idx) {
  int id = -1;
  if (page_idx >= 0 && page_idx < c.max_pages)
    id = fresh(c.table + (long long)b * c.max_pages + page_idx);
  if (id < 0 || id >= c.n_pages) {
    set_status(c.status, SINKATTN_ERR_BOUNDS);
    return -1;
  }
  return id;
}

// The two 8-element column chunks that a thread owns in every row, so that each
// rotated pair lies in one thread, and neighbouring threads' chunks side by side
// (16-byte accesses that meet in one 32-byte sector from one thread instead cost
// a D = 64 append 10 %).  Thread j of the row's D/16.
struct Chunks {
  int a, b;             // first columns
  bool rot_a, rot_b;    // whether they are rotated
};
template <int D>
__device__ __forceinline__ Chunks row_chunks(int j, int rot, int interleaved) {
  Chunks c;
  if (interleaved) {
    c.a = 8 * j;
    c.b = D / 2 + 8 * j;
    c.rot_a = c.a < rot;
    c.rot_b = c.b < rot;
  } else {
    // the pairs (i, i + rot/2), then the halves of what is not rotated
    const int nr = rot / 16;
    c.rot_a = c.rot_b = j < nr;
    c.a = j < nr ? 8 * j : rot + 8 * (j - nr);
    c.b = c.a + (j < nr ? rot / 2 : (D - rot) / 2);
  }
  return c;
}

// cosines and sines of a position for the thread's sixteen elements: eight
// consecutive angles, or four for each chunk of neighbouring pairs
struct Angles {
  float c[8], s[8];
};
__device__ __forceinline__ void load_angles(Angles& t, const float* rope, long long pos, int rot,
                                            const Chunks& ch, int interleaved) {
  const float* row = rope + pos * rot;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int at = interleaved ? (i ? ch.b : ch.a) / 2 : ch.a + 4 * i;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
    if (i ? ch.rot_b : ch.rot_a) {
      x = fresh(reinterpret_cast<const float4*>(row + at));
      y = fresh(reinterpret_cast<const float4*>(row + rot / 2 + at));
    }
    t.c[4 * i] = x.x; t.c[4 * i + 1] = x.y; t.c[4 * i + 2] = x.z; t.c[4 * i + 3] = x.w;
    t.s[4 * i] = y.x; t.s[4 * i + 1] = y.y; t.s[4 * i + 2] = y.z; t.s[4 * i + 3] = y.w;
  }
}

template <class E>
__device__ __forceinline__ void widen8(const uint4& u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = E::widen(w[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
template <class E>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(E::pack(x[0], x[1]), E::pack(x[2], x[3]), E::pack(x[4], x[5]),
                    E::pack(x[6], x[7]));
}

// x c - y s and x c + y s.  EXACT adds the products' own rounding errors back (a
// fused multiply-add gives them), which leaves half a unit in the last place or
// little more whatever cancels: an 8-bit code next to a tie then falls as the exact
// value does.  16-bit results do not show the difference.  The error of an infinite
// product is not a number, or infinite where the product overflowed; it is left out, and
// the sum stays infinite, or NaN where two infinities cancel.
template <bool EXACT>
__device__ __forceinline__ float turn(float x, float c, float y, float s) {
  if constexpr (!EXACT) return x * c + y * s;
  const float w = y * s, e = fmaf(y, s, -w);
  const float r = fmaf(x, c, w);
  return fabsf(w) < INFINITY ? r + e : r;
}
template <bool EXACT>
__device__ __forceinline__ void rotate_pairs(float (&x)[8], const float* c, const float* s) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float x0 = x[2 * i], x1 = x[2 * i + 1];
    x[2 * i] = turn<EXACT>(x0, c[i], -x1, s[i]);
    x[2 * i + 1] = turn<EXACT>(x1, c[i], x0, s[i]);
  }
}
template <bool EXACT>
__device__ __forceinline__ void rotate16(float (&a)[8], float (&b)[8], const Angles& t,
                                         const Chunks& ch, int interleaved) {
  if (interleaved) {
    if (ch.rot_a) rotate_pairs<EXACT>(a, t.c, t.s);
    if (ch.rot_b) rotate_pairs<EXACT>(b, t.c + 4, t.s + 4);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = a[i], y = b[i];
      a[i] = turn<EXACT>(x, t.c[i], -y, t.s[i]);
      b[i] = turn<EXACT>(y, t.c[i], x, t.s[i]);
    }
  }
}

// Both kernels are programmatic dependents (their launch lies under the end of the
// kernel before them, whose writes the wait makes visible) and let the next one be
// scheduled at once.
__device__ __forceinline__ void join_stream() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Offsets that leave the call's rows and may name none of them, so that no token's thread
// meets them: one thread of the grid looks at the first and the last.
__device__ __forceinline__ void check_offsets(const PagedAppendProblem& p) {
  if (p.cu && blockIdx.x == 0 && threadIdx.x == 0 && (fresh(p.cu) < 0 || fresh(p.cu + p.c.B) > p.T))
    set_status(p.c.status, SINKATTN_ERR_BOUNDS);
}

// Where a packed token goes.
struct Place {
  int b, pos;  // b < 0: no sequence of the call has it, or it is out of bounds
};
__device__ __forceinline__ Place place_token(const PagedAppendProblem& p, int t, int lane) {
  Place r{-1, 0};
  if (p.cu) {
    const int b = find_sequence(p.cu, p.c.B, t, lane);
    const int c0 = fresh(p.cu + b), c1 = fresh(p.cu + b + 1);
    if (t < c0 || t >= c1) return r;  // rows behind the last sequence
    if (c0 < 0 || c1 > p.T) {         // offsets that leave the call's rows
      set_status(p.c.status, SINKATTN_ERR_BOUNDS);
      return r;
    }
    r.pos = max(fresh(p.c.seqlens + b), 0) - (c1 - t);
    r.b = b;
  } else {
    const int n = fresh(p.c.seqlens + t);
    if (n <= 0) return r;  // a slot without a new token
    r.pos = n - 1;
    r.b = t;
  }
  if (r.pos < 0 || (p.rope && r.pos >= p.n_pos)) {
    set_status(p.c.status, SINKATTN_ERR_BOUNDS);
    r.b = -1;
  }
  return r;
}

// Copy or rotate the 16-bit rows of one token: rows [0, Hq) are its queries,
// then Hkv keys, then Hkv values (only the queries when kv = false).  Thread
// (j, g) of the token's D/16 x NG takes chunk pair j of rows g, g + NG, ...;
// its angles are loaded once for all of them, and four rows are in flight.  A token
// whose page is not in the pool has its queries rotated all the same.
template <class E, int D, int U>
__device__ __forceinline__ void token_rows(const PagedAppendProblem& p, int t, int j, int g,
                                           int NG, bool kv, int lane) {
  using T = typename E::T;
  const int Hq = p.q ? p.Hq : 0, Hkv = p.c.Hkv;
  int rows = kv ? Hq + 2 * Hkv : Hq;
  const Chunks ch = row_chunks<D>(j, p.rot, p.interleaved);
  const T* q = static_cast<const T*>(p.q) + t * p.q_stride;
  const T* k = static_cast<const T*>(p.k) + t * p.k_stride;
  const T* v = static_cast<const T*>(p.v) + t * p.v_stride;
  uint4 xa[U], xb[U];
  auto load = [&](int r0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * NG;
      if (r < rows) {
        const T* src = r < Hq ? q + r * D : r < Hq + Hkv ? k + (r - Hq) * D : v + (r - Hq - Hkv) * D;
        xa[u] = *reinterpret_cast<const uint4*>(src + ch.a);
        xb[u] = *reinterpret_cast<const uint4*>(src + ch.b);
      }
    }
  };
  load(g);  // under way while the token's place is looked up
  const Place pl = place_token(p, t, lane);
  if (pl.b < 0) return;
  T* kdst = nullptr;
  T* vdst = nullptr;
  if (kv) {
    const int page = page_of(p.c, pl.b, pl.pos >> p.c.page_log2);
    if (page < 0) rows = Hq;
    const long long at =
        (((long long)page * Hkv << p.c.page_log2) + (pl.pos & (p.c.page_size - 1))) * D;
    kdst = static_cast<T*>(p.c.k_pages) + at;
    vdst = static_cast<T*>(p.c.v_pages) + at;
  }
  const long long head_step = (long long)D << p.c.page_log2;
  Angles an;
  if (ch.rot_a) load_angles(an, p.rope, pl.pos, p.rot, ch, p.interleaved);
  T* qo = static_cast<T*>(p.q_out) + (long long)t * p.Hq * D;
  T* ko = p.k_out && kv ? static_cast<T*>(p.k_out) + (long long)t * Hkv * D : nullptr;
  for (int r0 = g; r0 < rows; r0 += U * NG) {
    if (r0 != g) load(r0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * NG;
      if (r >= rows) break;
      if (ch.rot_a && r < Hq + Hkv) {
        float a[8], b[8];
        widen8<E>(xa[u], a);
        widen8<E>(xb[u], b);
        rotate16<false>(a, b, an, ch, p.interleaved);
        xa[u] = pack8<E>(a);
        xb[u] = pack8<E>(b);
      }
      T* dst = r < Hq ? qo + r * D
                      : r < Hq + Hkv ? kdst + (r - Hq) * head_step : vdst + (r - Hq - Hkv) * head_step;
      *reinterpret_cast<uint4*>(dst + ch.a) = xa[u];
      *reinterpret_cast<uint4*>(dst + ch.b) = xb[u];
      if (ko && r >= Hq && r < Hq + Hkv) {
        *reinterpret_cast<uint4*>(ko + (r - Hq) * D + ch.a) = xa[u];
        *reinterpret_cast<uint4*>(ko + (r - Hq) * D + ch.b) = xb[u];
      }
    }
  }
}

constexpr int kAppendThreads = 256;
// Bound by HBM: 411 MB (4 x 4,096 tokens, 32 query and 2 x 8 key and value heads of
// 128) in 66 to 67 us, 6.2 TB/s, 0.94 of a plain copy's rate.  Rows in flight a thread and
// blocks an SM: more rows hide latency within a thread, but their registers cost the
// threads that hide it beside them.  (2, 4) takes 66 us there, (4, 3) 69, (4, 2) 78,
// (1, 6) 71; a ragged batch at D = 64 takes 36 us with (4, 3) and 40 with (4, 2), (4, 4).
template <int D>
struct AppendCfg {
  static constexpr int ROWS = D == 128 ? 2 : 4, BLOCKS = D == 128 ? 4 : 3;
};

template <class E, int D>
__global__ void __launch_bounds__(kAppendThreads, AppendCfg<D>::BLOCKS)
    paged_append_kernel(PagedAppendProblem p, int NG) {
  join_stream();
  constexpr int NC = D / 16;
  const int per_token = NC * NG;  // a multiple of 32: a warp stays in one token
  const long long t =
      (long long)blockIdx.x * (kAppendThreads / per_token) + threadIdx.x / per_token;
  if (t >= p.T) return;
  const int i = threadIdx.x % per_token;
  token_rows<E, D, AppendCfg<D>::ROWS>(p, (int)t, i % NC, i / NC, NG, true, threadIdx.x & 31);
  check_offsets(p);
}

// ---------------------------------------------------------------- 8-bit cache
// The smallest power of two s >= 2^-126 with amax <= 448 s (448 = 1.75 2^8),
// 0 for amax = 0.
__device__ __forceinline__ float block_scale(float amax) {
  if (!(amax > 0.f)) return 0.f;
  const uint32_t u = __float_as_uint(amax);
  int e = int(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);  // biased exponent of s
  if (e < 1) e = 1;
  return __uint_as_float(uint32_t(e) << 23);
}
__device__ __forceinline__ float finite_abs(float x) {
  const uint32_t u = __float_as_uint(x) & 0x7fffffffu;
  return u < 0x7f800000u ? __uint_as_float(u) : 0.f;
}
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return (lo & 0xffffu) | (hi << 16);
}
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float m) {
  return make_uint2(encode4(x[0] * m, x[1] * m, x[2] * m, x[3] * m),
                    encode4(x[4] * m, x[5] * m, x[6] * m, x[7] * m));
}
__device__ __forceinline__ float2 decode2(uint32_t two) {
  const __half2_raw h =
      __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two & 0xffffu), __NV_E4M3);
  return __half22float2(__half2(h));
}
__device__ __forceinline__ uint32_t rescale4(uint32_t codes, float m) {
  const float2 a = decode2(codes), b = decode2(codes >> 16);
  return encode4(a.x * m, a.y * m, b.x * m, b.y * m);
}

// A block of the grid per touched page and KV head (D = 64: two heads) of K, and one
// of V, of page/8 warps with eight rows each.  The new rows are read once and stay in
// registers between the block's amax and the encoding: two passes of a warp over a
// head of 128, or one over two heads of 64, which then share their angles and the
// block's beginning.  That is what 64 registers hold.  A prefill of 4 x 4,096 tokens, 8
// heads of 128, takes 68 to 70 us so, 88 with sixteen rows a warp (128 registers), 76 with
// four rows of two heads; a ragged batch at D = 64 26 us, 28 with one head.  It is bound
// by its instructions and by the chain of small loads (offsets, length, table) that a
// block begins with: the prefill without queries takes 30 us for 100 MB, 25 without the
// rotation, whose angles every head's block reads again.  Other blocks rotate the
// queries.
//
// The pages that a sequence touches need no prefix sum: n tokens touch at most
// n/page + 2 pages (rounded down), so sequence b owns items
// [cu[b]/page + 2b, cu[b + 1]/page + 2(b + 1)) and the rest of them are idle.
template <int D>
struct BlockCfg {
  static constexpr int HEADS = D == 128 ? 1 : 2;   // of a block
  static constexpr int PASSES = D == 128 ? 2 : 1;  // of a warp
  static constexpr int ROWS = PASSES * 32 / (D / 16);
};
template <class E, int D>
__global__ void __launch_bounds__(512, 2) paged_append_fp8_kernel(PagedAppendProblem p,
                                                                  unsigned q_per_item, int NG) {
  using T = typename E::T;
  constexpr int NC = D / 16;         // threads per row
  constexpr int RPP = 32 / NC;       // rows per pass of a warp
  constexpr int PASSES = BlockCfg<D>::PASSES, HP = BlockCfg<D>::HEADS;
  __shared__ float s_max[HP][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  join_stream();
  check_offsets(p);
  const PagedView& c = p.c;
  // an item's blocks: K and V of every head, then its share of the query blocks, so
  // that one kind's waits lie under the other's traffic
  const unsigned kv_blocks = 2 * ((c.Hkv + HP - 1) / HP), per_item = kv_blocks + q_per_item;
  const unsigned item = blockIdx.x / per_item, part = blockIdx.x - item * per_item;
  if (part >= kv_blocks) {
    const int per_token = NC * NG;
    const long long t = ((long long)item * q_per_item + (part - kv_blocks)) * (blockDim.x / per_token) +
                        threadIdx.x / per_token;
    const int i = threadIdx.x % per_token;
    if (t < p.T) token_rows<E, D, 2>(p, (int)t, i % NC, i / NC, NG, false, lane);
    return;
  }
  const bool is_v = part & 1;
  const int h0 = (part >> 1) * HP, nh = min(HP, c.Hkv - h0);  // its heads
  // the sequence, and the new tokens [t0, t1) that fall in the item's page
  int b, c0, c1;
  if (p.cu) {
    int lo = 0, n = c.B;
    while (n > 1) {
      const int step = (n + 31) / 32, i = lane * step;
      const bool le = i < n && (fresh(p.cu + lo + i) >> c.page_log2) + 2 * (lo + i) <= (int)item;
      const int hit = __popc(__ballot_sync(0xffffffffu, le));
      const int skip = hit > 0 ? (hit - 1) * step : 0;
      lo += skip;
      n = min(step, n - skip);
    }
    b = lo;
    c0 = fresh(p.cu + b);
    c1 = fresh(p.cu + b + 1);
  } else {
    b = item;
    c0 = b;
    c1 = b + 1;
  }
  const int n_new = c1 - c0;
  const int len = max(fresh(c.seqlens + b), 0);
  if (n_new <= 0 || (!p.cu && len == 0)) return;
  if (c0 < 0 || c1 > p.T) {  // offsets that leave the call's rows
    if (threadIdx.x == 0) set_status(c.status, SINKATTN_ERR_BOUNDS);
    return;
  }
  const int start = len - n_new;  // position of token c0
  const int end = p.rope ? min(len, p.n_pos) : len;
  if ((start < 0 || end < len) && threadIdx.x == 0) set_status(c.status, SINKATTN_ERR_BOUNDS);
  const int first = start >> c.page_log2;  // page of the sequence's first new token
  const int page_idx = first + (p.cu ? (int)item - ((c0 >> c.page_log2) + 2 * b) : 0);
  const int pos0 = page_idx << c.page_log2;  // position of the page's row 0
  const int r0 = max(start - pos0, 0), r1 = min(end - pos0, c.page_size);
  if (page_idx < max(first, 0) || r0 >= r1) return;

  const int row_base = warp * BlockCfg<D>::ROWS;
  const int j = lane % NC, sub = lane / NC;
  const Chunks ch = row_chunks<D>(j, is_v ? 0 : p.rot, p.interleaved);
  const T* src = is_v ? static_cast<const T*>(p.v) : static_cast<const T*>(p.k);
  const long long tstride = is_v ? p.v_stride : p.k_stride;
  uint4 ua[HP][PASSES], ub[HP][PASSES];
#pragma unroll
  for (int u = 0; u < PASSES; ++u) {
    const int r = row_base + u * RPP + sub;
    const long long t = (long long)c0 + (pos0 + r - start);
    const T* row = src + t * tstride + h0 * D;
#pragma unroll
    for (int e = 0; e < HP; ++e) {
      ua[e][u] = ub[e][u] = make_uint4(0, 0, 0, 0);
      if (r >= r0 && r < r1 && e < nh) {
        ua[e][u] = *reinterpret_cast<const uint4*>(row + e * D + ch.a);
        ub[e][u] = *reinterpret_cast<const uint4*>(row + e * D + ch.b);
      }
    }
  }
  const int page = page_of(c, b, page_idx);  // looked up under the rows' loads
  if (page < 0) return;
  const long long blk = (long long)page * c.Hkv + h0;
  float* scale_at = (is_v ? c.v_scale : c.k_scale) + blk;
  float s_old[HP], amax[HP];
#pragma unroll
  for (int e = 0; e < HP; ++e) s_old[e] = r0 > 0 && e < nh ? scale_at[e] : 0.f;
  float xa[HP][PASSES][8], xb[HP][PASSES][8];
#pragma unroll
  for (int e = 0; e < HP; ++e) amax[e] = 0.f;
#pragma unroll
  for (int u = 0; u < PASSES; ++u) {
    const int r = row_base + u * RPP + sub;
    const bool on = r >= r0 && r < r1;
    Angles an;
    if (on && ch.rot_a) load_angles(an, p.rope, pos0 + r, p.rot, ch, p.interleaved);
#pragma unroll
    for (int e = 0; e < HP; ++e) {
      widen8<E>(ua[e][u], xa[e][u]);
      widen8<E>(ub[e][u], xb[e][u]);
      if (on && ch.rot_a) rotate16<true>(xa[e][u], xb[e][u], an, ch, p.interleaved);
      if (on && !is_v && p.k_out && e < nh) {
        T* ko = static_cast<T*>(p.k_out) +
                ((long long)(c0 + (pos0 + r - start)) * c.Hkv + h0 + e) * D;
        *reinterpret_cast<uint4*>(ko + ch.a) = pack8<E>(xa[e][u]);
        *reinterpret_cast<uint4*>(ko + ch.b) = pack8<E>(xb[e][u]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
        amax[e] = fmaxf(amax[e], fmaxf(fabsf(xa[e][u][i]), fabsf(xb[e][u][i])));
    }
  }
#pragma unroll
  for (int e = 0; e < HP; ++e) {
    if (amax[e] == INFINITY) {  // rare (a NaN has dropped out already): the finite ones alone
      amax[e] = 0.f;
#pragma unroll
      for (int u = 0; u < PASSES; ++u)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          amax[e] = fmaxf(amax[e], fmaxf(finite_abs(xa[e][u][i]), finite_abs(xb[e][u][i])));
    }
    // magnitudes are ordered as their bits are
    const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(amax[e]));
    if (lane == 0) s_max[e][warp] = __uint_as_float(top);
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < HP; ++e) {
    if (e >= nh) break;
    float top = 0.f;
    for (int w = 0; w < (int)(blockDim.x >> 5); ++w) top = fmaxf(top, s_max[e][w]);
    const float s = fmaxf(block_scale(top), s_old[e]);
    uint8_t* dst = static_cast<uint8_t*>(is_v ? c.v_pages : c.k_pages) +
                   ((blk + e) << c.page_log2) * D;
    // where every value is 0 (or not finite) any factor will do
    const float inv = s > 0.f ? __frcp_rn(s) : 1.f;
    const bool grow = s > s_old[e] && r0 > 0;
    const float ratio = s_old[e] * inv;
#pragma unroll
    for (int u = 0; u < PASSES; ++u) {
      const int r = row_base + u * RPP + sub;
      uint2* da = reinterpret_cast<uint2*>(dst + (long long)r * D + ch.a);
      uint2* db = reinterpret_cast<uint2*>(dst + (long long)r * D + ch.b);
      if (r >= r0 && r < r1) {
        *da = encode8(xa[e][u], inv);
        *db = encode8(xb[e][u], inv);
      } else if (grow && r < r0) {
        const uint2 a = *da, bq = *db;
        *da = make_uint2(rescale4(a.x, ratio), rescale4(a.y, ratio));
        *db = make_uint2(rescale4(bq.x, ratio), rescale4(bq.y, ratio));
      }
    }
    if (threadIdx.x == 0) scale_at[e] = s;
  }
}

template <class... A>
int launch_dependent(void (*kern)(A...), unsigned blocks, int threads, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = stream;
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(threads);
  return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess ? SINKATTN_OK : SINKATTN_ERR_CUDA;
}

// Row groups of a token's threads: eight leave a thread several rows, whose loads
// overlap and share its angles (a prefill takes 66 us, with sixteen 73).  While all
// tokens fit the SMs with a block of 256 threads each (four blocks an SM), they get one
// each, which ends sooner.
int row_groups(int T, int D) { return T < 4 * 148 ? kAppendThreads / (D / 16) : 8; }

template <class E, int D>
int append_typed(const PagedAppendProblem& p, cudaStream_t stream) {
  const int NG = row_groups(p.T, D), per_token = D / 16 * NG;
  const long long blocks = ((long long)p.T * per_token + kAppendThreads - 1) / kAppendThreads;
  if (blocks > 0x7fffffffLL) return SINKATTN_ERR_INVALID_ARG;
  return launch_dependent(paged_append_kernel<E, D>, (unsigned)blocks, kAppendThreads, stream, p, NG);
}

template <class E, int D>
int append_fp8_typed(const PagedAppendProblem& p, cudaStream_t stream) {
  const int threads = p.c.page_size / BlockCfg<D>::ROWS * 32;
  const long long items = p.cu ? p.T / p.c.page_size + 2LL * p.c.B : p.c.B;
  const int NG = 128 / D * 8;  // 64 threads a token: every block size holds whole tokens
  const int tokens = threads / (D / 16 * NG);
  const long long q_blocks = p.q ? (p.T + tokens - 1) / tokens : 0;
  const long long q_per_item = (q_blocks + items - 1) / items;
  const long long kv_blocks = 2 * ((p.c.Hkv + BlockCfg<D>::HEADS - 1) / BlockCfg<D>::HEADS);
  const long long blocks = items * (kv_blocks + q_per_item);
  if (blocks > 0x7fffffffLL) return SINKATTN_ERR_INVALID_ARG;
  return launch_dependent(paged_append_fp8_kernel<E, D>, (unsigned)blocks, threads, stream, p,
                          (unsigned)q_per_item, NG);
}

}  // namespace

int launch_paged_append(const PagedAppendProblem& p, cudaStream_t s) {
  if (p.dt == SINKATTN_FP16)
    return p.D == 128 ? append_typed<ElemF16, 128>(p, s) : append_typed<ElemF16, 64>(p, s);
  return p.D == 128 ? append_typed<ElemBf16, 128>(p, s) : append_typed<ElemBf16, 64>(p, s);
}
int launch_paged_append_fp8(const PagedAppendProblem& p, cudaStream_t s) {
  if (p.dt == SINKATTN_FP16)
    return p.D == 128 ? append_fp8_typed<ElemF16, 128>(p, s) : append_fp8_typed<ElemF16, 64>(p, s);
  return p.D == 128 ? append_fp8_typed<ElemBf16, 128>(p, s) : append_fp8_typed<ElemBf16, 64>(p, s);
}

}  // namespace sk
