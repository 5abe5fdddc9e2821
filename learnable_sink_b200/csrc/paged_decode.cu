// Single-token attention with a learnable sink over a paged cache, 16-bit or
// E4M3 with a scale for each page and KV head:
//   x_j = scale <q, k_j>,  l = sum_j e^{x_j - m},  O = sum_j e^{x_j - m} v_j / (l + e^{a - m})
// over the visible positions j < n, and with a window also j < n_sink or
// j >= n - window.
//
// Bound by HBM (a visible row of K and V is read once and shared by the G query
// heads of its KV head), as long as the arithmetic stays off the CUDA cores: 16
// sequences of 8 to 32 thousand tokens, 8 KV heads of 128, take 195 to 202 us (6.6 to
// 6.9 TB/s; a plain copy reaches 6.5), 4 of 98 to 131 thousand in 8 bits 139 to 144 us
// (6.5 to 6.8 TB/s).  A call of little work takes 7.2 us: 1 to find its place from the
// lengths, 1.6 until the first scores, 1.5 for a tile and its result, 1 to end the
// kernel, 1.7 to join.  So
// both products run on tcgen05 with the cache as the M side, where its rows lie
// in shared memory as TMA brought them, whatever their type:
//   S^T[128 positions x N] = K Q^T     A = K tile, K-major; B = Q, K-major
//   O^T[D x N]            += V^T P^T   A = V tile, MN-major; B = P, MN-major
// An instruction costs the same for any N <= 64, so the columns are cheap, and
// they carry the precision that 8-bit operands lack: a value x is split in
// rounded terms t0 = r(x), t1 = r((x - t0) c), ..., each in columns of its own and
// summed, with its factor, in float32.  E4M3 keeps four significant bits: two
// terms hold a bf16 query exactly (three an f16 one) down to 2^-23 of its row's
// largest; four terms hold a probability to 2^-16 of itself and 2^-30 of the largest
// (with three, 2^-12 and 2^-26, a hundred thousand weights beside a dominant one went
// missing from O, while l had them).  With a 16-bit cache the queries go in as they are
// and a probability takes two terms (16 bits of it for bf16, 22 for f16).
//
// One thread owns one position of a tile and four query heads: softmax statistics
// are per thread (l) or voted (the reference maximum moves, for all positions, when
// a score passes it by more than 2^2), so a tile needs one barrier among four warps
// and no shuffles.  Up to 16 heads take that many warpgroups, each with columns of
// its own: a tile's time is latency, and four heads fit 80 registers, so the SM
// holds enough warps to hide it (eight heads a thread: 1.6 times the time a tile).
// Long sums are taken in two steps: the tensor cores truncate as they add, and a thread's
// l takes a tile after the other, so every 16 tiles O and l are folded into sums that
// are rounded (262,144 equal weights in one row: the result is up to 1.4e-3 too small
// without).
// In the 8-bit cache the value scale goes into the probability: e^{x - m} is
// multiplied by it in the exponent, with a reference of its own.
//
// Schedule: CTAs work in groups of up to eight, one KV head each of the same tiles of
// the same sequence, at about the same time: the heads' rows of a page are neighbours
// in memory, and DRAM likes them together (the long calls above: 209 and 147 us if every
// CTA goes its own way, 195 and 139 in groups of eight, 203 and 144 of four; pages of 16
// gain nothing).  A row of the schedule is a sequence's tiles for a group's heads, with
// a unit for the row's own cost behind them; the rows, in order, are dealt in equal runs
// to the groups.  Lengths are on the device, so every CTA adds them up for itself.  A run
// is cut into segments where the row changes.  A segment that holds all of its row writes
// the result; others write (O, m, l) at slot pair + first CTA of the group, which no two
// segments share, and a second kernel joins them.  Rows of about the same length are left
// whole.
#include <cuda_fp8.h>

#include <algorithm>
#include <climits>

#include "internal.h"
#include "paged.cuh"

namespace sk {

namespace {

constexpr int kRows = 128;     // rows of a K or V tile
constexpr int kHeads = 4;      // query heads per softmax warpgroup
constexpr int kJoinThreads = 128;

// ------------------------------------------------------------------ schedule
template <int TP>  // positions per tile, 128 or 256
__device__ __forceinline__ SeqTiles tiles_of(const PagedDecodeProblem& p, int len) {
  return SeqTiles(len, p.c.max_pages << p.c.page_log2, p.n_sink, p.window, p.c.page_log2,
                  (TP == 128 ? 7 : 8) - p.c.page_log2);
}
template <int TP>
__device__ __forceinline__ SeqTiles seq_tiles(const PagedDecodeProblem& p, int b) {
  return tiles_of<TP>(p, fresh(p.c.seqlens + b));
}
__device__ __forceinline__ bool visible(const PagedDecodeProblem& p, int n, int pos) {
  return pos < n && (p.window <= 0 || pos < p.n_sink || pos >= n - p.window);
}

// Every role walks the CTA's run for itself.
template <int TP>
__device__ __forceinline__ bool next_segment(const PagedDecodeProblem& p, Walk& w) {
  return w.next(p.c.Hkv, p.lanes, [&](int b) { return seq_tiles<TP>(p, b); });
}
struct Start {
  Walk walk;
  int first, total;  // the run's first unit; units of all
  bool whole;        // a pair a CTA
};

// Adds up the lengths (a slice of the sequences a thread) and finds where this
// CTA's run begins; the thread whose slice it is in sets the walk up for all.
template <int THREADS, int TP, int SLACK>
__device__ __forceinline__ void find_start(const PagedDecodeProblem& p, Start* st, int2* s_warp) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per_thread = (p.c.B + THREADS - 1) / THREADS;
  const int b0 = tid * per_thread, b1 = min(b0 + per_thread, p.c.B);
  int sum = 0, longest = 0;
  for (int b = b0; b < b1; ++b) {
    const int units = seq_tiles<TP>(p, b).count + kPairUnits;
    sum += units;
    longest = max(longest, units);
  }
  longest = __reduce_max_sync(0xffffffffu, longest);
  int inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) s_warp[warp] = make_int2(inc, longest);
  __syncthreads();
  int before = inc - sum, total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    const int2 v = s_warp[w];
    if (w < warp) before += v.x;
    total += v.x;
    longest = max(longest, v.y);
  }
  const int chunks = p.chunks, group = blockIdx.y, groups = gridDim.y;
  total *= chunks;
  before *= chunks;
  const Runs runs(total, groups);
  auto seq_of = [&](int b) { return seq_tiles<TP>(p, b); };
  if (rows_whole(p.c.B * chunks, longest, runs.per, groups, SLACK)) {
    if (tid == 0) {
      st->walk = whole_walk(group, blockIdx.x, p.c.B, p.lanes, chunks, seq_of);
      st->whole = true;
    }
    return;
  }
  const int f0 = runs.begin(group);
  if (f0 >= before && f0 < before + sum * chunks) {
    st->walk = cut_walk(f0, runs.begin(group + 1) - f0, b0, before, blockIdx.x, p.lanes, chunks, seq_of);
    st->first = f0;
    st->total = total;
    st->whole = false;
  } else if (f0 == total && tid == 0) {
    st->walk.left = 0;  // less work than CTAs
  }
}

// ------------------------------------------------------------------ geometry
// NWG softmax warpgroups, of four query heads each.
template <class E, int D, bool F8, int NWG>
struct Geo {
  static constexpr int EB = F8 ? 1 : 2;
  static constexpr int CB = D * EB;                    // bytes of a position
  // Positions per row of a tile.  A warp spends about 85 cycles on a copy of 1 KB and
  // 125 on one of 4 KB, and a tile has its barriers and votes whatever it holds; so two
  // positions of 64 bytes, neighbours in memory, share a row: K's halves are multiplied
  // apart, into columns of their own, and V's half rows with the probabilities of their
  // own positions (a StreamingLLM band, with the leaner softmax that it made room for:
  // 24.7 -> 23.1 us).
  static constexpr int PP = CB == 64 ? 2 : 1;
  static constexpr int TP = kRows * PP;                // positions per tile
  static constexpr int RB = CB * PP;                   // bytes of a row
  static constexpr int BW = 128;                       // of a TMA box's row
  static constexpr int NB = RB / BW;                   // boxes per row
  static constexpr int QW = CB < 128 ? CB : 128;       // width of a query's rows
  static constexpr int TILE = kRows * RB;              // K or V tile
  static constexpr int QT = F8 ? (E::kFmt == 0 ? 3 : 2) : 1;  // terms of a query
  static constexpr int PT = F8 ? 4 : 2;                // terms of a probability
  // A warpgroup's columns: term t of head h at 4 t + h of 16 bytes' worth, so that
  // a thread's probabilities are one 16-byte store.
  static constexpr int COLS = 16 / EB;
  static constexpr int N = COLS * NWG < 16 ? 16 : COLS * NWG;  // of the queries
  static constexpr int NT = N * PP;                    // columns of S^T and of O^T
  static constexpr int PBYTES = NT / COLS * kRows * 16;
  static constexpr int QBYTES = N * CB;
  static constexpr int KE = 32 / EB;                   // K extent of an instruction
  static constexpr int TMEM = 4 * NT;                  // two S^T, O^T and its folded sum
  static constexpr int WARPS = 4 * NWG + 4, THREADS = WARPS * 32;
  // CTAs an SM: one's segment ends and waits overlap the other's work.  32 KB tiles
  // (or sixteen heads) leave room for one.
  static constexpr int CTAS = TILE < 32768 && NWG < 4 ? 2 : 1;
  static constexpr int SLACK = CTAS == 2 && PP == 1 ? 6 : 3;  // of rows_whole
  // A ring of tiles, K and V in turn.
  static constexpr int SLOTS =
      ((CTAS == 2 ? 112640 : 227328) - 2 * QBYTES - 2 * PBYTES - 1024) / TILE;
  static constexpr int OFF_Q = SLOTS * TILE;
  static constexpr int OFF_P = OFF_Q + 2 * QBYTES;
  static constexpr int SMEM = OFF_P + 2 * PBYTES + 1024;  // + room to align the base
  // factor from one term to the next: the residue of a rounding to EB bytes is
  // at most 2^-5 (E4M3), 2^-11 (f16) of the value's power of two; bf16 has range
  // to spare and needs none.  Queries move by 2^4, which keeps every term of a
  // 448-scaled row in range.
  static constexpr float TERM = F8 ? 32.f : (E::kFmt == 0 ? 2048.f : 1.f);
  static_assert((PT > QT ? PT : QT) * kHeads <= COLS, "a warpgroup's columns");
  static_assert(QBYTES % 1024 == 0 && TILE % 1024 == 0, "swizzled tiles start on their pattern");
  static_assert(TMEM >= 32 && TMEM * CTAS <= 512 && (TMEM & (TMEM - 1)) == 0, "tensor memory");
  static_assert(SLOTS >= 3, "S of a tile goes ahead of P V of the last one");
};

// Probabilities are held as 2^kBase e^{x - m}: with a reference that lags by at
// most 2^kLag they stay within 2^8 (E4M3 reaches 448), as high as they can: f16 and E4M3
// lose small ones.  bf16 does not, and its values reach as far as O, so there they stay
// within 1.
// The 8-bit terms are split in f16 pairs, where a residue and its move by 2^5 are exact
// and take half the instructions of float32.  What the rounding to f16 left is moved by 2^10
// and goes into the third term, whose own residue is the fourth: at worst that is 512
// and saturates, 64 2^-15 of a weight above 128, 2^-16 (a weight below its reference keeps
// 2^-17.6).  The fourth term's last bit is 2^-24 in these units; half of it, and half of
// that for f16's own subnormals, are below 2^-30 of the largest weight.
constexpr float kLag = 2.f;
template <class E, bool F8>
constexpr float kBase = F8 || E::kFmt == 0 ? 6.f : -kLag;

// Tiles whose sums O and l are held as the tensor cores and the threads add them up: at
// most 128 steps of O, each truncated by less than 2^-23 of it.  (Folding costs a long 8-bit
// decode 0.4 %, a 16-bit one nothing.)
constexpr int kFold = 16;

template <bool F8>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
  if constexpr (F8)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(id), "r"(acc)
        : "memory");
  else
    mma_ss(d, a, b, id, acc);
}
// Instruction descriptor: the 16-bit one; kind::f8f6f4 has its fields in the same
// places (format 0 = E4M3).
template <class E, bool F8>
__host__ __device__ constexpr uint32_t idesc(int M, int N, int a_mn, int b_mn) {
  return idesc_16_f32(F8 ? 0u : E::kFmt, M, N, a_mn, b_mn);
}
// Shared-memory descriptor of a K or V tile or a Q block: rows of BW bytes under
// the swizzle of that width, 8-row groups BW * 8 apart, boxes lbo apart.
template <int BW>
__device__ __forceinline__ uint64_t sdesc_rows(uint32_t addr, uint32_t lbo) {
  const uint64_t type = BW == 128 ? 2 : 4;
  return uint64_t((addr >> 4) & 0x3FFFu) | (uint64_t((lbo >> 4) & 0x3FFFu) << 16) |
         (uint64_t((BW * 8) >> 4) << 32) | (uint64_t(1) << 46) | (type << 61);
}
// P: row k's 16-byte unit i at i 2048 + 16 k, no swizzle: 8-row groups 128 bytes
// apart, units 2048.  A thread stores a position with one vector store, free of
// bank conflicts.
__device__ __forceinline__ uint64_t sdesc_p(uint32_t addr) {
  return uint64_t((addr >> 4) & 0x3FFFu) | (uint64_t(128 >> 4) << 16) |
         (uint64_t((kRows * 16) >> 4) << 32) | (uint64_t(1) << 46);
}

// the same between E4M3 pairs and f16 pairs
__device__ __forceinline__ uint32_t e4m3x2_of_f16x2(__half2 v) {
  return __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(v), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ __half2 f16x2_of_e4m3x2(uint32_t two) {
  return __half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two), __NV_E4M3));
}
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 e4m3x2_value(uint32_t two) {
  const __half2_raw h =
      __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two), __NV_E4M3);
  return __half22float2(__half2(h));
}

// true on all 128 threads of the warpgroup (barrier 1 + wg) if it is on any
__device__ __forceinline__ bool any_of_128(bool f, int wg) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}\n"
      : "=r"(r)
      : "r"(uint32_t(f)), "r"(wg + 1)
      : "memory");
  return r != 0;
}
// Lane's row, N consecutive columns (4, 8 or 16).
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t (&r)[N]) {
  if constexpr (N == 16) tmem_ld16(addr, r);
  else if constexpr (N == 8)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                   "=r"(r[6]), "=r"(r[7])
                 : "r"(addr));
  else
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
template <int N>
__device__ __forceinline__ void tmem_st(uint32_t addr, const uint32_t (&r)[N]) {
  if constexpr (N == 16) tmem_st16(addr, r);
  else tmem_st8(addr, r);
}
// the warp's largest x (NaN only if every x is)
__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}
// The mark of a page that is not in the pool, a NaN that log2f does not return.
constexpr uint32_t kOutside = 0xffffffffu;
// The reference of a row that has seen nothing: low enough that every score
// raises it, and finite, so that -inf minus it is -inf and not NaN.
constexpr float kNone = -3e38f;
// 2^(a - b), 0 from a = -inf (also over b = -inf)
__device__ __forceinline__ float ratio2(float a, float b) {
  return a == -INFINITY ? 0.f : fast_exp2(a - b);
}
// the sink's over the maximum, which it may be itself, at +inf too
__device__ __forceinline__ float sink_ratio(float a2, float mt) {
  return a2 == INFINITY ? 1.f : ratio2(a2, mt);
}
// log(lw 2^mt + e^a), den = lw + e^a / 2^mt: a itself, whatever its size, where the keys have
// no weight beside it
__device__ __forceinline__ float lse_of(float lw, float den, float mt, float a) {
  return lw == 0.f ? a : (mt + log2f(den)) * kLn2;
}

template <int SLOTS>
struct Bars {
  uint64_t full[SLOTS], empty[SLOTS];
  uint64_t s_full[2], p_full[2], pv_done[2], q_full[2], q_free[2], drain;
};

// workspace: [B Hkv] (first CTA, segments; B > kJoinThreads), then the partials
__host__ __device__ inline size_t meta_floats(long long pairs) {
  return (size_t)((2 * pairs + 63) / 64 * 64);
}

// ------------------------------------------------------------------ kernel
template <class E, int D, bool F8, int NWG>
__global__ void __launch_bounds__(Geo<E, D, F8, NWG>::THREADS, Geo<E, D, F8, NWG>::CTAS)
    paged_decode_kernel(const __grid_constant__ CUtensorMap tmap_k,
                        const __grid_constant__ CUtensorMap tmap_v,
                        const __grid_constant__ PagedDecodeProblem p) {
  using G_ = Geo<E, D, F8, NWG>;
  constexpr int SLOTS = G_::SLOTS, N = G_::N, NT = G_::NT, PP = G_::PP, TP = G_::TP, COLS = G_::COLS, GP = NWG * kHeads, H = kHeads;
  constexpr int W_TMA = 4 * NWG, W_MMA = W_TMA + 1, W_Q = W_TMA + 2;
  extern __shared__ uint8_t dsm_raw[];
  uint8_t* sm =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dsm_raw) + 1023) & ~uintptr_t(1023));
  __shared__ Bars<SLOTS> bar;
  __shared__ int abort_s;
  __shared__ uint32_t tmem_s;
  __shared__ Start start_s;
  __shared__ int2 warp_s[G_::WARPS];
  __shared__ __align__(16) float qs_s[8][GP];  // query scales of the last eight segments
  __shared__ float sink_sm[8][GP];             // their sink logits
  // (A segment's entries are read up to its result.  The queries of segment s + 8
  // are written once the scores of s + 6 are done, which follow the probabilities
  // of a tile behind segment s + 4.)
  // For each warpgroup: reference maxima of x and of x + log2(value scale), what they
  // were raised by last (a factor), each warp's maxima or sums, and the factors of
  // the result.
  __shared__ __align__(16) float ref_s[NWG][2][H], corr_s[NWG][2][H], red_s[NWG][4][2 * H], fac_s[NWG][H];
  __shared__ float fold_s[NWG][4][H];  // each warp's folded l
  // a tile's pages: score factor and log2 of the value scale (kOutside: not in the pool)
  __shared__ float2 page_s[2][TP / 16];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = p.Hq / p.c.Hkv;
  const PagedView& c = p.c;

  if (warp == W_MMA) {
    tmem_alloc(&tmem_s, G_::TMEM);
    tmem_relinquish();
  }
  if (tid == W_TMA * 32) {
    prefetch_tensormap(&tmap_k);
    prefetch_tensormap(&tmap_v);
    for (int i = 0; i < SLOTS; ++i) {
      mbar_init(&bar.full[i], 1);
      mbar_init(&bar.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.s_full[i], 2);  // scores, and their pages' scales
      mbar_init(&bar.p_full[i], 4 * NWG);
      mbar_init(&bar.pv_done[i], 1);
      mbar_init(&bar.q_full[i], 1);
      mbar_init(&bar.q_free[i], 1);
    }
    mbar_init(&bar.drain, 1);
    fence_mbar_init();
    abort_s = 0;
  }
  if (tid < 8 * GP) qs_s[tid / GP][tid % GP] = 0.f;
  // columns that no head or term owns stay zero
  for (int i = tid * 16; i < 2 * G_::QBYTES + 2 * G_::PBYTES; i += G_::THREADS * 16)
    *reinterpret_cast<uint4*>(sm + G_::OFF_Q + i) = make_uint4(0u, 0u, 0u, 0u);
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  // up to here nothing that another kernel writes was read: this kernel is itself
  // a programmatic dependent, and its start lies under the end of the last one
  asm volatile("griddepcontrol.wait;" ::: "memory");
  find_start<G_::THREADS, TP, G_::SLACK>(p, &start_s, warp_s);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_s;
  const uint32_t tm_s = tmem, tm_o = tmem + 2 * NT, tm_fold = tmem + 3 * NT;

  Walk w = start_s.walk;
  const int total = start_s.total, f0 = start_s.first, run = w.left;
  const bool work = w.begin(c.Hkv, p.lanes, [&](int b) { return seq_tiles<TP>(p, b); });

  if (!work) {
    // less work than CTAs
  } else if (warp == W_TMA) {
    // ---------------------------------------------------------------- TMA
    const int ppt = TP >> c.page_log2;  // pages per tile
    int ld = 0;                         // tiles (K or V) issued
    bool ok = true;
    do {
      auto load_id = [&](int i) {  // lane's page of tile i, -1: none to bring
        const int k = (w.t0 + i) * ppt + lane;
        int id = -1;
        if (lane < ppt && i < w.cnt && k < w.seq.pages)
          id = fresh(c.table + (long long)w.b * c.max_pages + w.seq.page(k));
        return id < c.n_pages ? id : -1;
      };
      int next = load_id(0);
      for (int i = 0; i < w.cnt && ok; ++i) {
        const int id = next;
        next = load_id(i + 1);
        const uint32_t need = __ballot_sync(0xffffffffu, id >= 0);
        const uint32_t bytes = __popc(need) * (uint32_t)(c.page_size * G_::CB);
        const int src = lane / G_::NB, nb = lane % G_::NB;  // this lane's page and box
        const int my = __shfl_sync(0xffffffffu, id, src);
        const int row = ((my * c.Hkv + w.kvh) << c.page_log2) / PP;
        const int at = nb * (kRows * G_::BW) + (src << c.page_log2) / PP * G_::BW;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv, ++ld) {
          const int slot = ld % SLOTS;
          if (ld >= SLOTS) ok = ok && mbar_wait(&bar.empty[slot], (ld / SLOTS - 1) & 1, &abort_s, c.status);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (lane == 0) mbar_expect_tx(&bar.full[slot], bytes);
          __syncwarp();
          if (src < ppt && my >= 0)
            tma_load_3d(sm + slot * G_::TILE + at, kv ? &tmap_v : &tmap_k, &bar.full[slot],
                        nb * (G_::BW / G_::EB), 0, row);
        }
      }
    } while (ok && next_segment<TP>(p, w));
    // The join's CTAs come up under the last tiles (let up at the start, the work before
    // their wait is in this kernel's way: 0.2 to 0.4 us).
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (!ok)  // leave no copy in flight
      for (int k = max(ld - SLOTS, 0); k < ld; ++k) {
        const long long t0 = clock64();
        while (!mbar_try_wait(&bar.full[k % SLOTS], (k / SLOTS) & 1))
          if (clock64() - t0 > kWaitBudgetCycles) break;
      }
  } else if (warp == W_MMA) {
    // ---------------------------------------------------------------- MMA
    if (lane == 0) {
      const uint32_t base = smem_u32(sm);
      bool ok = true;
      int j = 0, seg = 0;   // tiles, segments begun
      int pend = -1;        // tile whose P V is not issued yet
      bool pend_first = false;
      auto issue_pv = [&]() {
        const int slot = (2 * pend + 1) % SLOTS;
        ok = ok && mbar_wait(&bar.p_full[pend & 1], (pend >> 1) & 1, &abort_s, c.status) &&
             mbar_wait(&bar.full[slot], ((2 * pend + 1) / SLOTS) & 1, &abort_s, c.status);
        if (!ok) return;
        tc_fence_after();
        const uint64_t ad = sdesc_rows<G_::BW>(base + slot * G_::TILE, kRows * G_::BW);
        const uint64_t bd = sdesc_p(base + G_::OFF_P + (pend & 1) * G_::PBYTES);
#pragma unroll
        for (int k = 0; k < kRows / G_::KE; ++k)
          mma<F8>(tm_o, sdesc_add(ad, k * G_::KE * G_::BW), sdesc_add(bd, k * G_::KE * 16),
                  idesc<E, F8>(D * PP, NT, 1, 1), k > 0 || !pend_first);
        mma_commit(&bar.empty[slot]);
        mma_commit(&bar.pv_done[pend & 1]);
        pend = -1;
      };
      do {
        for (int i = 0; i < w.cnt && ok; ++i, ++j) {
          const int slot = (2 * j) % SLOTS;
          if (i == 0) ok = ok && mbar_wait(&bar.q_full[seg & 1], (seg >> 1) & 1, &abort_s, c.status);
          // the next scores ahead of the last tile's values, unless K is late
          if (pend >= 0 && !mbar_try_wait(&bar.full[slot], ((2 * j) / SLOTS) & 1)) issue_pv();
          ok = ok && mbar_wait(&bar.full[slot], ((2 * j) / SLOTS) & 1, &abort_s, c.status);
          if (!ok) break;
          tc_fence_after();
          const uint64_t ad = sdesc_rows<G_::BW>(base + slot * G_::TILE, 16);
          const uint64_t bd = sdesc_rows<G_::QW>(base + G_::OFF_Q + (seg & 1) * G_::QBYTES, 16);
#pragma unroll
          for (int q = 0; q < PP; ++q)
#pragma unroll
            for (int k = 0; k < G_::CB / 32; ++k) {
              const int a_at = q * G_::CB + k * 32, b_at = k * 32;
              mma<F8>(tm_s + (j & 1) * NT + q * N,
                      sdesc_add(ad, a_at / G_::BW * kRows * G_::BW + a_at % G_::BW),
                      sdesc_add(bd, b_at / G_::QW * N * G_::QW + b_at % G_::QW),
                      idesc<E, F8>(kRows, N, 0, 0), k > 0);
            }
          mma_commit(&bar.empty[slot]);
          mma_commit(&bar.s_full[j & 1]);
          if (i == w.cnt - 1) mma_commit(&bar.q_free[seg & 1]);
          if (pend >= 0) issue_pv();
          pend = j;
          pend_first = i % kFold == 0;
        }
        ++seg;
      } while (ok && next_segment<TP>(p, w));
      if (ok && pend >= 0) issue_pv();
      if (!ok) {  // no product may be running when the tensor memory is freed
        mma_commit(&bar.drain);
        const long long t0 = clock64();
        while (!mbar_try_wait(&bar.drain, 0))
          if (clock64() - t0 > kWaitBudgetCycles) break;
      }
    }
    __syncwarp();
  } else if (warp == W_Q) {
    // ---------------------------------------------------------------- queries
    constexpr int CPL = D / 32;  // columns per lane
    int seg = 0;
    bool ok = true;
    do {
      uint8_t* qd = sm + G_::OFF_Q + (seg & 1) * G_::QBYTES;
      const float a = p.sink && lane < G ? fresh(p.sink + w.kvh * G + lane) : -INFINITY;
      const typename E::T* q =
          static_cast<const typename E::T*>(p.q) + ((long long)w.b * p.Hq + w.kvh * G) * D + lane * CPL;
      auto at = [&](int r, int byte) {  // row r of the block, swizzled as the tiles are
        const int box = byte / G_::QW, in = byte % G_::QW, ch = in >> 4;
        const int x = G_::QW == 128 ? ch ^ (r & 7) : ch ^ ((r >> 1) & 3);
        return qd + box * (N * G_::QW) + r * G_::QW + (x << 4) + (in & 15);
      };
      uint32_t raws[GP][CPL / 2];
#pragma unroll
      for (int h = 0; h < GP; ++h) {  // every head's loads in flight at once
        if (h >= G) continue;
        if constexpr (CPL == 4) {
          const uint2 u = fresh(reinterpret_cast<const uint2*>(q + h * D));
          raws[h][0] = u.x;
          raws[h][CPL / 2 - 1] = u.y;
        } else {
          raws[h][0] = fresh(reinterpret_cast<const uint32_t*>(q + h * D));
        }
      }
      if (seg >= 2) ok = mbar_wait(&bar.q_free[seg & 1], ((seg >> 1) - 1) & 1, &abort_s, c.status);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      if (lane < GP) sink_sm[seg & 7][lane] = a;
#pragma unroll
      for (int h = 0; h < GP; ++h) {
        if (h >= G) continue;
        const uint32_t(&raw)[CPL / 2] = raws[h];
        if constexpr (!F8) {
#pragma unroll
          for (int i = 0; i < CPL / 2; ++i)
            *reinterpret_cast<uint32_t*>(at(h / H * COLS + h % H, (lane * CPL + 2 * i) * 2)) = raw[i];
          if (lane == 0) qs_s[seg & 7][h] = 1.f;
        } else {
          float x[CPL];
          float mx = 0.f;
          bool odd = false;
#pragma unroll
          for (int i = 0; i < CPL / 2; ++i) {
            const float2 f = E::widen(raw[i]);
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
            mx = fmaxf(mx, fmaxf(fabsf(f.x), fabsf(f.y)));
            odd = odd || !(fabsf(f.x) < INFINITY) || !(fabsf(f.y) < INFINITY);
          }
          mx = warp_max(mx);
          odd = __any_sync(0xffffffffu, odd);
          // the smallest power of two s with mx <= 448 s (the row's terms reach
          // 448); an infinity or NaN in the row makes its scores NaN
          const uint32_t u = __float_as_uint(mx);
          const int e = max(int(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0), 1);
          const float inv = odd || mx == 0.f ? 0.f : __uint_as_float(uint32_t(254 - e) << 23);
          if (lane == 0)
            qs_s[seg & 7][h] = odd ? __uint_as_float(0x7fffffffu) : __uint_as_float(uint32_t(e) << 23);
#pragma unroll
          for (int t = 0; t < G_::QT; ++t) {
            uint32_t code = 0;
#pragma unroll
            for (int i = 0; i < CPL / 2; ++i) {
              if (t == 0) {
                x[2 * i] *= inv;
                x[2 * i + 1] *= inv;
              }
              const uint32_t two = e4m3x2(x[2 * i], x[2 * i + 1]);
              const float2 v = e4m3x2_value(two);
              x[2 * i] = (x[2 * i] - v.x) * 16.f;
              x[2 * i + 1] = (x[2 * i + 1] - v.y) * 16.f;
              code |= two << (16 * i);
            }
            uint8_t* dst = at(h / H * COLS + t * H + h % H, lane * CPL);
            if constexpr (CPL == 4) *reinterpret_cast<uint32_t*>(dst) = code;
            else *reinterpret_cast<uint16_t*>(dst) = (uint16_t)code;
          }
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.q_full[seg & 1]);
      ++seg;
    } while (next_segment<TP>(p, w));
  } else if (warp == W_Q + 1) {
    // ---------------------------------------------------------------- page scales
    const int ppt = TP >> c.page_log2;
    const float scale_log2 = p.scale * kLog2e;
    int j = 0;
    bool ok = true;
    do {
      auto load_id = [&](int i) {
        const int k = (w.t0 + i) * ppt + lane;
        int id = -2;  // no page here
        if (lane < ppt && i < w.cnt && k < w.seq.pages) {
          id = fresh(c.table + (long long)w.b * c.max_pages + w.seq.page(k));
          if (id < 0 || id >= c.n_pages) {
            set_status(c.status, SINKATTN_ERR_BOUNDS);
            id = -1;
          }
        }
        return id;
      };
      int id = load_id(0);
      if (w.t0 == 0 && lane == 0) {
        if (c.B > kJoinThreads) {  // where the join finds the pair's segments
          const long long pair = (long long)w.b * c.Hkv + w.kvh;
          const int first = f0 + run - w.left, group = blockIdx.y;
          const Runs runs(total, gridDim.y);
          reinterpret_cast<int2*>(p.part)[pair] = make_int2(
              group, start_s.whole ? 1 : parts_of(runs, group, first, w.seq.count));
        }
        if (fresh(c.seqlens + w.b) > w.seq.n) set_status(c.status, SINKATTN_ERR_BOUNDS);
      }
      for (int i = 0; i < w.cnt; ++i, ++j) {
        float2 v = make_float2(scale_log2, 1.f);
        if (F8 && id >= 0) {
          const long long blk = (long long)id * c.Hkv + w.kvh;
          v.x *= __ldcg(c.k_scale + blk);
          v.y = __ldcg(c.v_scale + blk);
        }
        const bool outside = id == -1;
        id = load_id(i + 1);
        v.y = outside ? __uint_as_float(kOutside) : F8 ? log2f(v.y) : 0.f;
        if (j >= 2) ok = mbar_wait(&bar.p_full[j & 1], ((j >> 1) - 1) & 1, &abort_s, c.status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane < ppt) page_s[j & 1][lane] = v;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.s_full[j & 1]);
      }
    } while (ok && next_segment<TP>(p, w));
  } else {
    // ---------------------------------------------------------------- softmax
    const int wg = NWG == 1 ? 0 : warp >> 2, wt = tid & 127, ww = warp & 3;
    const int h0 = wg * H;                                    // its first query head
    const uint32_t my_lane = uint32_t(ww * 32) << 16;
    const uint32_t my_s = tm_s + wg * COLS + my_lane, my_o = tm_o + wg * COLS + my_lane;
    const uint32_t my_fold = tm_fold + wg * COLS + my_lane;
    float(&ref)[2][H] = ref_s[wg];
    float(&corr)[2][H] = corr_s[wg];
    float(&red)[4][2 * H] = red_s[wg];
    const int ppt = TP >> c.page_log2;
    const long long pairs = (long long)c.B * c.Hkv;
    float* parts = p.part + meta_floats(pairs);
    // l over the warp: lanes 8 h .. 8 h + 7 get head h's sum
    auto warp_sums = [&](const float(&l)[H]) {
      const bool hi = lane & 16, hj = lane & 8;
      float a = hi ? l[2] : l[0], b = hi ? l[3] : l[1];
      a += __shfl_xor_sync(0xffffffffu, hi ? l[0] : l[2], 16);
      b += __shfl_xor_sync(0xffffffffu, hi ? l[1] : l[3], 16);
      float t = hj ? b : a;
      t += __shfl_xor_sync(0xffffffffu, hj ? a : b, 8);
#pragma unroll
      for (int o = 4; o >= 1; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
      return t;
    };
    float& my_fold_l = fold_s[wg][ww][lane >> 3];  // of lanes 0, 8, 16, 24
    int j = 0, seg = 0;
    // No wait that runs out breaks the loops (each returns at once after the
    // first): every thread meets every barrier, and the results are undefined.
    do {
      float l[H];
#pragma unroll
      for (int h = 0; h < H; ++h) l[h] = 0.f;
      if (wt < 2 * H) ref[wt / H][wt % H] = kNone;
      if ((lane & 7) == 0) my_fold_l = 0.f;
      for (int i = 0; i < w.cnt; ++i, ++j) {
        // the thread's positions (past the last page: past the sequence)
        const int at_page = (w.t0 + i) * ppt + (wt * PP >> c.page_log2);
        const int pos0 = at_page < w.seq.pages ? (w.seq.page(at_page) << c.page_log2) +
                                                     (wt * PP & (c.page_size - 1))
                                               : w.seq.n;
        mbar_wait(&bar.s_full[j & 1], (j >> 1) & 1, &abort_s, c.status);
        tc_fence_after();
        if (i > 0 && i % kFold == 0) {  // rare: O starts afresh with this tile's product
          mbar_wait(&bar.pv_done[(j - 1) & 1], ((j - 1) >> 1) & 1, &abort_s, c.status);
          tc_fence_after();
#pragma unroll
          for (int q = 0; q < PP; ++q) {
            uint32_t r[COLS], f[COLS];
            tmem_ld(my_o + q * N, r);
            tmem_ld(my_fold + q * N, f);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < COLS; ++k)
              r[k] = __float_as_uint(__uint_as_float(r[k]) + (i > kFold ? __uint_as_float(f[k]) : 0.f));
            tmem_st(my_fold + q * N, r);
          }
          tmem_st_wait();
          const float t = warp_sums(l);
          if ((lane & 7) == 0) my_fold_l += t;
#pragma unroll
          for (int h = 0; h < H; ++h) l[h] = 0.f;
        }
        const float2 page = page_s[j & 1][wt * PP >> c.page_log2];
        const bool held = __float_as_uint(page.y) != kOutside;
        const float lvs = held ? page.y : 0.f;
        // scores in log2 units; hidden positions at -inf whatever their rows hold
        bool seen[PP];
        float x[PP][H];
        if constexpr (F8) {
          uint32_t r[PP][16];
#pragma unroll
          for (int q = 0; q < PP; ++q) tmem_ld(my_s + (j & 1) * NT + q * N, r[q]);
          tmem_ld_wait();
#pragma unroll
          for (int h = 0; h < H; ++h) {
            const float f = page.x * qs_s[seg & 7][h0 + h];
#pragma unroll
            for (int q = 0; q < PP; ++q) {
              float v = __uint_as_float(r[q][H + h]);
              if constexpr (G_::QT == 3) v += __uint_as_float(r[q][2 * H + h]) * 0.0625f;
              x[q][h] = (__uint_as_float(r[q][h]) + v * 0.0625f) * f;
            }
          }
        } else {
          uint32_t r[4];
          tmem_ld(my_s + (j & 1) * NT, r);
          tmem_ld_wait();
#pragma unroll
          for (int h = 0; h < H; ++h) x[0][h] = __uint_as_float(r[h]) * page.x;
        }
#pragma unroll
        for (int q = 0; q < PP; ++q) {
          seen[q] = held && visible(p, w.seq.n, pos0 + q);
#pragma unroll
          for (int h = 0; h < H; ++h) x[q][h] = seen[q] ? x[q][h] : -INFINITY;
        }
        bool moves = i == 0;
#pragma unroll
        for (int h = 0; h < H; ++h) {
          const float xm = PP == 2 ? fmaxf(x[0][h], x[PP - 1][h]) : x[0][h];
          moves |= xm - ref[0][h] > kLag;
          if constexpr (F8) moves |= xm + (lvs - ref[1][h]) > kLag;
        }
        if (any_of_128(moves, wg)) {
          // rare: raise the references to the maxima so far, and bring l, O and their
          // folded sums along
          float mine = 0.f;
#pragma unroll
          for (int h = 0; h < H; ++h) {
            const float xm = PP == 2 ? fmaxf(x[0][h], x[PP - 1][h]) : x[0][h];
            const float a = warp_max(xm);
            mine = lane == h ? a : mine;
            if constexpr (F8) {
              const float b = warp_max(xm + lvs);
              mine = lane == H + h ? b : mine;
            }
          }
          if (lane < (F8 ? 2 : 1) * H) red[ww][lane] = mine;
          named_bar_sync(1 + wg, 128);
          if (wt < (F8 ? 2 : 1) * H) {
            const int k = wt / H, h = wt % H;
            const float old = ref[k][h];
            const float now =
                fmaxf(fmaxf(fmaxf(red[0][wt], red[1][wt]), fmaxf(red[2][wt], red[3][wt])), old);
            ref[k][h] = now;
            corr[k][h] = ratio2(old, now);
          }
          named_bar_sync(1 + wg, 128);
          if (i > 0) {
            mbar_wait(&bar.pv_done[(j - 1) & 1], ((j - 1) >> 1) & 1, &abort_s, c.status);
            tc_fence_after();
#pragma unroll
            for (int h = 0; h < H; ++h) l[h] *= corr[0][h];
            if ((lane & 7) == 0) my_fold_l *= corr[0][lane >> 3];
            for (uint32_t at = my_o; at <= (i < kFold ? my_o : my_fold); at += NT) {
#pragma unroll
              for (int q = 0; q < PP; ++q) {
                uint32_t r[COLS];
                tmem_ld(at + q * N, r);
                tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < COLS; ++k)
                  r[k] = __float_as_uint(__uint_as_float(r[k]) * corr[F8][k % H]);
                tmem_st(at + q * N, r);
              }
            }
            tmem_st_wait();
          }
        }
        // P's buffer is free: the commit behind these scores covers the products
        // issued before them, P V of two tiles ago among them
#pragma unroll
        for (int q = 0; q < PP; ++q) {
          uint32_t pk[4] = {0u, 0u, 0u, 0u};
#pragma unroll
          for (int h = 0; h < H; h += 2) {
            float e[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float pr = fast_exp2(x[q][h + k] - ref[0][h + k]);
              l[h + k] += pr;
              e[k] = F8 ? fast_exp2(x[q][h + k] + (lvs - ref[1][h + k] + kBase<E, F8>)) : pr * (E::kFmt == 0 ? 64.f : 0.25f);
            }
            if constexpr (F8) {
              __half2 v = __floats2half2_rn(e[0], e[1]);
              const float2 f = __half22float2(v);
              const __half2 rest = __floats2half2_rn((e[0] - f.x) * (G_::TERM * G_::TERM),
                                                     (e[1] - f.y) * (G_::TERM * G_::TERM));
#pragma unroll
              for (int t = 0; t < G_::PT; ++t) {
                if (t == 2) v = __hadd2(v, rest);
                const uint32_t two = e4m3x2_of_f16x2(v);
                pk[t] = h == 0 ? two : __byte_perm(pk[t], two, 0x5410);
                if (t + 1 < G_::PT)
                  v = __hmul2(__hsub2(v, f16x2_of_e4m3x2(two)), __float2half2_rn(G_::TERM));
              }
            } else {
#pragma unroll
              for (int t = 0; t < G_::PT; ++t) {
                const uint32_t two = E::pack(e[0], e[1]);
                const float2 v = E::widen(two);
                pk[2 * t + h / 2] = two;
                e[0] = (e[0] - v.x) * G_::TERM;
                e[1] = (e[1] - v.y) * G_::TERM;
              }
            }
          }
          *reinterpret_cast<uint4*>(sm + G_::OFF_P + (j & 1) * G_::PBYTES +
                                    (q * (N / COLS) + wg) * (kRows * 16) + wt * 16) =
              make_uint4(pk[0], pk[1], pk[2], pk[3]);
        }
        if (wg == 0 && (!seen[0] || !seen[PP - 1])) {
          // a hidden row may hold NaN, and 0 NaN is not 0: clear its values
          const int slot = (2 * j + 1) % SLOTS;
          mbar_wait(&bar.full[slot], ((2 * j + 1) / SLOTS) & 1, &abort_s, c.status);
          uint8_t* row = sm + slot * G_::TILE + wt * G_::BW;
#pragma unroll
          for (int k = 0; k < G_::RB / 16; ++k)
            if (!seen[k * 16 / G_::CB])  // 16-byte unit k of the row, where the swizzle puts it
              *reinterpret_cast<uint4*>(row + k / 8 * (kRows * G_::BW) + ((k % 8 ^ (wt & 7)) << 4)) =
                  make_uint4(0u, 0u, 0u, 0u);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.p_full[j & 1]);
      }
      // ------------------------------------------------ the segment's result
      {
        const float t = warp_sums(l);
        if ((lane & 7) == 0) red[ww][lane >> 3] = t + my_fold_l;
      }
      named_bar_sync(1 + wg, 128);
      const long long pair = (long long)w.b * c.Hkv + w.kvh;
      const bool final = w.cnt == w.seq.count;
      float* part = parts + part_slot(pair, blockIdx.y, p.lanes) * G * (D + 2);
      const long long row0 = (long long)w.b * p.Hq + w.kvh * G;
      if (wt < H && h0 + wt < G) {
        const int h = h0 + wt;
        const float m = ref[0][wt], lt = (red[0][wt] + red[1][wt]) + (red[2][wt] + red[3][wt]);
        // O is in units of 2^ref less the base (a head whose value scales are all 0
        // has none, and an O of 0 or NaN)
        const float mo = F8 ? ref[1][wt] : m;
        float f;
        if (final) {
          const float a = sink_sm[seg & 7][h], a2 = a * kLog2e;
          const float mt = fmaxf(m, a2);
          const float lw = lt * ratio2(m, mt), den = lw + sink_ratio(a2, mt);
          const float inv = den != 0.f ? 1.f / den : 0.f;
          f = mo == kNone ? inv : fast_exp2(mo - mt - kBase<E, F8>) * inv;
          p.lse[row0 + h] = lse_of(lw, den, mt, a);
          if (p.sink_s) p.sink_s[row0 + h] = lw * inv;
        } else {
          f = mo == kNone ? 1.f : fast_exp2(mo - m - kBase<E, F8>);
          part[h * (D + 2) + D] = m;
          part[h * (D + 2) + D + 1] = lt;
        }
        fac_s[wg][wt] = f;
      }
      named_bar_sync(1 + wg, 128);
      mbar_wait(&bar.pv_done[(j - 1) & 1], ((j - 1) >> 1) & 1, &abort_s, c.status);
      tc_fence_after();
      // O^T's row of this thread.  M = 64 has sixteen rows a warp; with two positions
      // a row, rows 64 to 127 are the second ones' (in columns of their own), and come
      // to the first ones' threads through this warpgroup's part of a P buffer.
      uint32_t r[COLS];
      tmem_ld(my_o + (PP == 2 ? (ww >> 1) * N : 0), r);
      tmem_ld_wait();
      if (w.cnt > kFold) {
        uint32_t f[COLS];
        tmem_ld(my_fold + (PP == 2 ? (ww >> 1) * N : 0), f);
        tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < COLS; ++k)
          r[k] = __float_as_uint(__uint_as_float(r[k]) + __uint_as_float(f[k]));
      }
      tc_fence_before();
      float o[H];
#pragma unroll
      for (int h = 0; h < H; ++h) {
        o[h] = __uint_as_float(r[(G_::PT - 1) * H + h]);
#pragma unroll
        for (int t = G_::PT - 2; t >= 0; --t)
          o[h] = __uint_as_float(r[t * H + h]) + o[h] * (1.f / G_::TERM);
      }
      if constexpr (PP == 2) {
        float4* half = reinterpret_cast<float4*>(sm + G_::OFF_P + wg * (kRows * 16)) + (wt & 63);
        if (wt >= 64) *half = make_float4(o[0], o[1], o[2], o[3]);
        named_bar_sync(1 + wg, 128);
        if (wt < 64) {
          const float4 v = *half;
          o[0] += v.x;
          o[1] += v.y;
          o[2] += v.z;
          o[3] += v.w;
        }
      }
      const int d = D == 128 || PP == 2 ? wt : ww * 16 + lane;
      if (D == 128 || (PP == 2 ? wt < 64 : lane < 16)) {
#pragma unroll
        for (int h = 0; h < H; ++h) {
          if (h0 + h >= G) break;
          const float v = o[h] * fac_s[wg][h];
          if (final) static_cast<typename E::T*>(p.out)[(row0 + h0 + h) * D + d] = (typename E::T)v;
          else part[(h0 + h) * (D + 2) + d] = v;
        }
      }
      ++seg;
    } while (next_segment<TP>(p, w));
  }
  __syncthreads();
  if (warp == W_MMA) {
    tc_fence_after();
    tmem_dealloc(tmem, G_::TMEM);
  }
}

// Join a pair's segments and the sink: one CTA per (sequence, query head), a
// thread a column.  Launched as a programmatic dependent, which starts when every CTA
// of the decode kernel is past its own wait: what earlier kernels wrote (lengths,
// sinks) may be read at once, from L2, and where the pair's segments are is known before they
// are done (0.5 to 1 us of a call).  With more sequences than threads, whose lengths
// would take long to add up, the decode kernel's note says it.
template <class E, int D, int TP, int SLACK>
__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(PagedDecodeProblem p, int groups) {
  __shared__ float wt_s[kMaxCtas], red_s[2][4];
  __shared__ int sum_s[4], before_s[4], longest_s[4], mine_s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / p.Hq, h = blockIdx.x % p.Hq, G = p.Hq / p.c.Hkv;
  const long long pair = (long long)b * p.c.Hkv + h / G;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const float a = p.sink ? __ldcg(p.sink + h) : -INFINITY, a2 = a * kLog2e;
  int2 meta = make_int2(0, 0);
  if (p.c.B <= kJoinThreads) {
    const int units = tid < p.c.B ? tiles_of<TP>(p, __ldcg(p.c.seqlens + tid)).count + kPairUnits : 0;
    const int sum = __reduce_add_sync(0xffffffffu, units);
    const int before = __reduce_add_sync(0xffffffffu, tid < b ? units : 0);
    const int longest = __reduce_max_sync(0xffffffffu, units);
    if (lane == 0) {
      sum_s[warp] = sum;
      before_s[warp] = before;
      longest_s[warp] = longest;
    }
    if (tid == b) mine_s = units;
    __syncthreads();
    const int chunks = p.chunks;
    const int total = (sum_s[0] + sum_s[1] + sum_s[2] + sum_s[3]) * chunks;
    const Runs runs(total, groups);
    const int first = (before_s[0] + before_s[1] + before_s[2] + before_s[3]) * chunks +
                      (chunks == 1 ? 0 : h / (G * p.lanes) * mine_s);
    if (!rows_whole(p.c.B * chunks, max(max(longest_s[0], longest_s[1]), max(longest_s[2], longest_s[3])),
                    runs.per, groups, SLACK)) {
      meta.x = runs.cta_of(first);
      meta.y = parts_of(runs, meta.x, first, mine_s - kPairUnits);
    }
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (p.c.B > kJoinThreads) meta = __ldcg(reinterpret_cast<const int2*>(p.part) + pair);
  const int ns = min(meta.y, kMaxCtas);
  if (ns <= 1) return;
  const float* parts = p.part + meta_floats((long long)p.c.B * p.c.Hkv);
  const long long row = (long long)G * (D + 2), step = row * p.lanes;
  const float* part = parts + part_slot(pair, meta.x, p.lanes) * row + (long long)(h % G) * (D + 2);
  // the first segments' columns are on their way while the weights are made
  constexpr int U = 16;
  float v[U];
  auto load = [&](int i0) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      v[u] = tid < D && i0 + u < ns ? __ldcg(part + (i0 + u) * step + tid) : 0.f;
  };
  load(0);
  constexpr int R = (kMaxCtas + kJoinThreads - 1) / kJoinThreads;
  float m[R], l[R], mt = a2;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int i = r * kJoinThreads + tid;
    m[r] = i < ns ? __ldcg(part + i * step + D) : -INFINITY;
    l[r] = i < ns ? __ldcg(part + i * step + D + 1) : 0.f;
    mt = fmaxf(mt, m[r]);
  }
  mt = warp_max(mt);
  if (lane == 0) red_s[0][warp] = mt;
  __syncthreads();
  mt = fmaxf(fmaxf(red_s[0][0], red_s[0][1]), fmaxf(red_s[0][2], red_s[0][3]));
  float lt = 0.f;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int i = r * kJoinThreads + tid;
    const float wt = ratio2(m[r], mt);
    if (i < ns) wt_s[i] = wt;
    lt += l[r] * wt;
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) lt += __shfl_xor_sync(0xffffffffu, lt, o);
  if (lane == 0) red_s[1][warp] = lt;
  __syncthreads();
  lt = (red_s[1][0] + red_s[1][1]) + (red_s[1][2] + red_s[1][3]);
  const float den = lt + sink_ratio(a2, mt);
  const long long at = (long long)b * p.Hq + h;
  if (tid < D) {
    float o = 0.f;
    for (int i0 = 0; i0 < ns; i0 += U) {
      if (i0 > 0) load(i0);
#pragma unroll
      for (int u = 0; u < U; ++u) o += i0 + u < ns ? v[u] * wt_s[i0 + u] : 0.f;
    }
    static_cast<typename E::T*>(p.out)[at * D + tid] = (typename E::T)(den != 0.f ? o / den : 0.f);
  }
  if (tid == 0) {
    p.lse[at] = lse_of(lt, den, mt, a);
    if (p.sink_s) p.sink_s[at] = den != 0.f ? lt / den : 0.f;
  }
}

template <class E, int D, bool F8, int NWG>
int decode_cfg(PagedDecodeProblem p, cudaStream_t stream) {
  using G_ = Geo<E, D, F8, NWG>;
  const PagedView& c = p.c;
  const int rows = c.n_pages * c.Hkv * c.page_size;
  CUtensorMap mk, mv;
  constexpr int PP = G_::PP;
  if (F8 ? !make_tmap_codes(&mk, c.k_pages, rows / PP, 1, D * PP, c.page_size / PP) ||
               !make_tmap_codes(&mv, c.v_pages, rows / PP, 1, D * PP, c.page_size / PP)
         : !make_tmap_3d(&mk, c.k_pages, rows, 1, D, 1, c.page_size) ||
               !make_tmap_3d(&mv, c.v_pages, rows, 1, D, 1, c.page_size))
    return SINKATTN_ERR_CUDA;
  auto kern = paged_decode_kernel<E, D, F8, NWG>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, G_::SMEM) !=
      cudaSuccess)
    return SINKATTN_ERR_CUDA;
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  // no more groups than the tables have units
  const long long tiles = ((long long)c.max_pages * c.page_size + G_::TP - 1) / G_::TP;
  if ((tiles + kPairUnits) * c.B * c.Hkv > INT_MAX) return SINKATTN_ERR_UNSUPPORTED;
  p.lanes = group_lanes(c.Hkv);
  p.chunks = c.Hkv / p.lanes;
  const int groups = schedule_groups((tiles + kPairUnits) * c.B * p.chunks, G_::CTAS * sms, p.lanes);
  record_start(SINKATTN_KERNEL_DECODE, stream);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = stream;
  cfg.gridDim = dim3(p.lanes, (unsigned)groups);
  cfg.blockDim = dim3(G_::THREADS);
  cfg.dynamicSmemBytes = G_::SMEM;
  const cudaError_t rc = cudaLaunchKernelEx(&cfg, kern, mk, mv, p);
  record_stop(SINKATTN_KERNEL_DECODE, stream);
  if (rc != cudaSuccess) return SINKATTN_ERR_CUDA;
  if (tiles == 1) return SINKATTN_OK;  // every pair is one segment
  cfg.gridDim = dim3(c.B * p.Hq);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = 0;
  if (cudaLaunchKernelEx(&cfg, paged_join_kernel<E, D, G_::TP, G_::SLACK>, p, groups) != cudaSuccess) return SINKATTN_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? SINKATTN_OK : SINKATTN_ERR_CUDA;
}

template <class E, int D, bool F8>
int decode_group(const PagedDecodeProblem& p, cudaStream_t stream) {
  const int G = p.Hq / p.c.Hkv;
  if (G <= kHeads) return decode_cfg<E, D, F8, 1>(p, stream);
  if (G <= 2 * kHeads) return decode_cfg<E, D, F8, 2>(p, stream);
  return decode_cfg<E, D, F8, 4>(p, stream);
}
template <class E, int D>
int decode_typed(const PagedDecodeProblem& p, cudaStream_t stream) {
  return p.fp8 ? decode_group<E, D, true>(p, stream) : decode_group<E, D, false>(p, stream);
}

}  // namespace

size_t paged_decode_part_floats(int B, int Hq, int Hkv, int D, int sms) {
  const long long pairs = (long long)B * Hkv;
  return meta_floats(pairs) + (size_t)part_slots(pairs, sms) * (Hq / Hkv) * (D + 2);
}

int launch_paged_decode(const PagedDecodeProblem& p, cudaStream_t s) {
  if (p.dt == SINKATTN_FP16)
    return p.D == 128 ? decode_typed<ElemF16, 128>(p, s) : decode_typed<ElemF16, 64>(p, s);
  return p.D == 128 ? decode_typed<ElemBf16, 128>(p, s) : decode_typed<ElemBf16, 64>(p, s);
}

}  // namespace sk
