// decode_runs.cuh -- paged decode attention with the keys of the whole batch cut
// into equal runs: over the 8-bit cache (attn_decode_paged_e4m3), over the rows' own
// bf16 pages in attn_decode_paged_shared, and over the pages that a sliding window
// and a few first tokens leave of a row, of either cache (attn_decode_paged_window,
// attn_decode_paged_window_e4m3).
//
// One query token per row; the online recurrence of "Naive attention and the
// online softmax" in base 2. Both contractions are mma.m16n8k16 with the keys
// (S^T = K q^T) or the value dimensions (O^T = V^T P^T) as the 16 rows and up to
// 8 query heads of the KV head as the 8 columns: one MMA covers 16 keys x 8
// heads x 16 dims.
//   * K: the contraction index may be permuted freely, so a lane reads 16-byte
//     chunks of a key with one shared load each and takes them as its A
//     fragment; no ldmatrix, no shuffles.
//   * V: ldmatrix.trans. P^T: the S^T accumulator holds key rows; movmatrix
//     transposes the 8x8 block of weights into the B fragment.
//
// 8-bit cache (e4m3.cuh). With c_j, e_j the codes and exponent of key j, w_j,
// f_j those of its value,
//   s_j = scale * 2^e_j (q . c_j),  o = sum_j exp(s_j) 2^f_j w_j / sum_j exp(s_j).
// Codes go to fp16 (exact) in registers. Each head has two references: m for
// the normaliser (a running max of s) and r for the accumulator (a running max
// of s + f, the log2 weight with which a code of V enters). Any common shift
// is legal, and a weight 2^(s + f - r) fits fp16 whatever the values'
// magnitudes are, so P V is one fp16 product against the codes themselves. r is
// held as d = r - m and scores enter as rounded products minus m: both are
// exact for the heaviest keys at any magnitude of the logits, where the spacing
// of fp32 numbers passes 2^15's exponent (from 2^27 on). q
// is scaled per head by a power of two to a largest magnitude in
// [2^14, 2^15), where fp16 holds bf16's 8 significant bits down to 2^-28 of
// that maximum. ldmatrix moves byte pairs (two dims of a key); one prmt puts
// the same dim of two keys side by side.
//
// bf16 cache: q, K and V enter as they are; P is the two-term bf16 split
// P_hi + P_lo (a single bf16 weight would cost up to 2^-8 of itself).
//
// Bound by memory: 2 (d_h + 1) or 4 d_h bytes per key and KV head. A warp owns
// a ring of NST stages, each one page of K and V, for the 8-bit cache with their
// exponents, filled by its own 16-byte cp.async into a swizzled layout. (Four
// TMA boxes a page cost the warp 850 cycles to issue, operands differing from
// lane to lane, a third of a page's time and more than its arithmetic.)
//
// Work split: the (row, KV head, head block) units, laid end to end with a
// weight of np + kUnit for np pages, are cut into equal runs, one per warp, so
// any mix of lengths fills the machine and the launch does not depend on the
// lengths. A warp works through its run unit by unit on its own (no barrier, no
// join between units) and finishes each unit that lies inside its run. Units
// cut by a run border are joined at the CTA's end from shared memory, in run
// order, each warp taking the sums of 16 dims (one warp adding all parts of its
// unit took 2.3 us of a 32768-key row's 20). What reaches past the CTA leaves at
// most two partial states per CTA (a unit that began before it, one that goes
// on behind it), which the merge kernel joins in run order. (Splitting a unit over all warps of a CTA and joining at every unit's
// end instead took 57 us for 64 rows of up to 1000 keys, 131 MB: rows of a few
// pages cost a CTA as much as rows of hundreds.)
//
// Windows are bound by the visible pages' bytes in the same way: 66 rows of up to
// 16384 keys, window 4096 and 4 sinks, 32 query heads over 8 of 128, take 153 to 157 us of
// the bf16 cache, 0.94 to 0.91 of the copy rate; 200 rows of the 8-bit cache, window 2001
// and 18 sinks, 134.5 us, 0.86 (a unit is 128 pages, and has its query and its output).
// Masking only the pages at a part's ends took the first from 158 to 154 us.
#pragma once

#include "common.cuh"
#include "e4m3.cuh"
#include "internal.h"

namespace attn {

namespace {

using e4m3::kPage;

// Weights are at most 2^15 (fp16's largest finite number is 65504): the
// reference r is set to 13 below a new running max's weight and moves once a
// weight would pass 2^15. Weights down to 2^-27 of the largest are then normal
// fp16 numbers, and what fp16 drops below 2^-38 of it is under 2^-20 of the sum
// even for 2^18 keys.
constexpr float kTop = 13.0f, kSlack = 2.0f;
constexpr float kNone = -3.402823466e38f;  // reference before the first key: below every score

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t movmatrix_t(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t lds_u8(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=h"(v) : "r"(addr));
  return v;
}
// 16 bytes to shared memory, zeros if !live.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool live, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint.L2::256B [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src),
               "r"(live ? 16 : 0), "l"(policy)
               : "memory");
}
// The same for exponents: a page's bytes of 8 heads fill a 128-byte line, which
// is fetched whole and kept for the other heads' runs. (As 16-byte reads that L2
// drops first they cost a DRAM access each, as many as the codes' slabs.)
__device__ __forceinline__ void copy16_line(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(live ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the newest N groups of this thread's copies have landed.
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Two fp32 numbers' upper halves (bf16, truncated) and what they leave out.
__device__ __forceinline__ uint32_t split_hi(float a, float b) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, 0x7632;" : "=r"(r) : "r"(__float_as_uint(a)), "r"(__float_as_uint(b)));
  return r;
}
__device__ __forceinline__ uint32_t split_lo(float a, float b) {
  return pack_bf16x2(a - __uint_as_float(__float_as_uint(a) & 0xffff0000u),
                     b - __uint_as_float(__float_as_uint(b) & 0xffff0000u));
}

// E8: the 8-bit cache. NW warps per CTA, NST stages per warp.
template <bool E8, int D, int NW, int NST>
struct Cfg {
  static constexpr int PAGE_BYTES = kPage * D * (E8 ? 1 : 2);  // one page of one KV head
  static constexpr int STAGE_BYTES = 2 * PAGE_BYTES;           // K then V
  static constexpr int RING_BYTES = NW * NST * STAGE_BYTES;
  static constexpr int EXP_OFF = RING_BYTES;                   // [warp][stage][K 16 | V 16]
  static constexpr int EXP_BYTES = E8 ? 32 : 0;
  static constexpr int NREG = D / 4;                           // accumulators per lane
  static constexpr int JOIN_OFF = EXP_OFF + NW * NST * EXP_BYTES;
  static constexpr int JOIN_BYTES = NW * 32 * NREG * 4;        // a warp's part of a cut unit
  static constexpr int ML_OFF = JOIN_OFF + JOIN_BYTES;         // [2][warp][8 heads] floats
  static constexpr int SMEM = ML_OFF + 2 * NW * 8 * 4;         // from a 1024-byte boundary
  // The unit that goes on behind a warp's run is kept in the warp's ring, free by then.
  static_assert(NST * STAGE_BYTES >= 32 * NREG * 4 + 64 && NW >= D / 16, "join");
};

// 16-byte chunk `c` of key row `r` of a page, swizzled so that the loads of K
// (two rows x four chunks a quarter warp) and ldmatrix (eight rows of one chunk)
// find distinct banks. 8-bit codes: rows of 128 or 64 bytes; bf16: halves of 64
// elements, rows of 128 bytes.
template <bool E8, int D>
__device__ __forceinline__ uint32_t chunk_at(uint32_t page, int r, int c) {
  if constexpr (E8)
    return page + r * D + ((c ^ (D == 128 ? (r & 7) : ((r >> 1) & 3))) << 4);
  else
    return page + (c >> 3) * (kPage * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

// What a merge reads of the unit that begins in a CTA and goes on behind it: parts
// (0: there is none), first (row, head), heads.
struct alignas(16) RunCut {
  int parts, row0, nh;
};

// Where states and results go. Units cut by a run border: part (two slots of 8
// heads per CTA). Other units: o and lse themselves (8-bit decode), or a state
// per (row, head) in row_* (shared-prefix decode, whose merge adds the prefix).
struct RunOut {
  long long* plan;
  float *o_part, *m_part, *l_part;
  float *o_row, *m_row, *l_row;
  __nv_bfloat16* o;
  float* lse;
  RunCut* cut = nullptr;  // [CTAs] (windows)
};

constexpr int kMinRun = 1;      // least weight of a warp's run
constexpr int kLenCache = 128;  // row lengths kept in shared memory

template <int NW>
struct RunShared {
  long long warp[NW];
  long long off[NW];  // weight between a warp's first row and its run
  int b[NW];          // its first row
  int kind[NW];       // its stored part: 0 none, 1 the unit goes on, 2 it ends
  int own[NW];        // the unit behind it: 0 none, 1 began in its run, 2 before the CTA
  int own_row[NW], own_nh[NW], own_left[NW];  // left: its pages behind the warp's run
  int len[kLenCache];
};

struct Rows {
  const int32_t* seq_lens;
  int B, max_len, upr, n_gb;  // units per row, and per (row, KV head)
  static constexpr bool kWindow = false;
  static constexpr int kUnit = kRunsUnit;  // a unit's query, state and epilogue, in pages
  __device__ __forceinline__ int pages(int len) const { return (len + kPage - 1) / kPage; }
  __device__ __forceinline__ int page_at(int, int i) const { return i; }
};
// Rows that see their last `window` keys and the first `sinks`. What the kernel
// walks are the pages that hold such keys, laid end to end: sink_pages of them,
// then the window's from page first on. Every one of them holds a visible key, so
// no page's scores are all masked, and pages in between are never looked up.
template <int UNIT>
struct WindowRows : Rows {
  int window, sinks;
  static constexpr bool kWindow = true;
  static constexpr int kUnit = UNIT;
  __device__ __forceinline__ int first_key(int len) const { return max(len - window, 0); }
  __device__ __forceinline__ int sink_pages(int len) const {
    return (min(sinks, len) + kPage - 1) / kPage;
  }
  __device__ __forceinline__ int skipped(int len) const {  // pages between the two parts
    return max(first_key(len) / kPage - sink_pages(len), 0);
  }
  __device__ __forceinline__ int pages(int len) const {
    return (len + kPage - 1) / kPage - skipped(len);
  }
  __device__ __forceinline__ int page_at(int len, int i) const {
    return i < sink_pages(len) ? i : i + skipped(len);
  }
  // Which of the 16 slots of page p a row of len keys sees, one bit each.
  __device__ __forceinline__ uint32_t visible(int len, int p) const {
    auto below = [](int n) { return (1u << min(max(n, 0), kPage)) - 1u; };  // slots 0 .. n - 1
    const int at = p * kPage;
    return below(len - at) & (~below(first_key(len) - at) | below(min(sinks, len) - at));
  }
};

// A warp's run, unit by unit. Warp-uniform.
struct Walk {
  int b, u, len, np;   // row, unit within the row, its keys and pages
  int lo, hi;          // pages of the unit that lie in the run
  long long rem;       // weight of the run behind this unit
};

__device__ __forceinline__ int row_len(const Rows& rw, int b) {
  const int n = __ldcg(rw.seq_lens + b);
  return min(max(n, 0), rw.max_len);
}
__device__ __forceinline__ int row_len(const Rows& rw, const int* cached, int b) {
  return rw.B <= kLenCache ? cached[b] : row_len(rw, b);
}
template <class R>
__device__ __forceinline__ int row_weight(const R& rw, int len) {  // of one unit of the row
  return len > 0 ? rw.pages(len) + R::kUnit : 0;
}
// a / b for a >= 0, b > 0: in 32 bits where both fit (64-bit division costs
// several hundred cycles).
__device__ __forceinline__ long long div_ll(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}
// Opens unit w.u of row w.b at weight `off` within it.
template <int kUnit>
__device__ __forceinline__ void walk_open(Walk& w, long long off) {
  const long long take = min(w.np + kUnit - off, w.rem);
  w.lo = static_cast<int>(max(off - kUnit, 0ll));
  w.hi = static_cast<int>(max(off + take - kUnit, 0ll));
  w.rem -= take;
}
// Next unit of the run; false at its end.
template <class R>
__device__ __forceinline__ bool walk_next(Walk& w, const R& rw, const int* cached) {
  if (w.rem <= 0) return false;
  if (++w.u == rw.upr) {
    w.u = 0;
    do {
      ++w.b;
      if (w.b >= rw.B) return false;
      w.len = row_len(rw, cached, w.b);
    } while (w.len == 0);
    w.np = rw.pages(w.len);
  }
  walk_open<R::kUnit>(w, 0);
  return true;
}

// A warp's run: weight (0: none; -1: none for the whole CTA), first row and its
// length, weight between that row's first unit and the run.
struct RunPlan {
  long long rem, off;
  int b, len;
  long long per;  // weight of every run
};

// Plans the runs, one per warp; CTA 0 leaves the plan for a merge that reads it (else
// nullptr).
template <int NW, class R, class Sync>
__device__ __forceinline__ RunPlan plan_runs(const R rw, long long* plan, RunShared<NW>& sh, int cta,
                                          int n_cta, unsigned int* err, Sync sync) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // ---- the runs: prefix sums of the rows' weights (per unit) ----
  const long long n_runs = static_cast<long long>(n_cta) * NW;
  auto per_of = [&](long long all) {
    return max(static_cast<long long>(kMinRun), div_ll(all + n_runs - 1, n_runs));
  };
  if (lane == 0) sh.kind[warp] = sh.own[warp] = 0;  // read behind the join's barrier
  long long all, per, p0;
  bool have;
  RunPlan r;
  if (rw.B <= 32) {
    // A row per lane: every warp plans for itself, without a barrier (9.0 us a
    // call for a row of 1000 keys; the form below 9.4).
    int len = 0;
    if (lane < rw.B) {
      const int raw = __ldcg(rw.seq_lens + lane);
      len = min(max(raw, 0), rw.max_len);
      if (cta == 0 && warp == 0 && raw != len) atomicOr(err, ATTN_DEVERR_BAD_SEQ_LEN);
    }
    sh.len[lane] = len;  // (every warp writes the same)
    const uint32_t w = row_weight(rw, len);
    uint32_t incl = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    all = static_cast<long long>(__shfl_sync(0xffffffffu, incl, 31)) * rw.upr;
    per = per_of(all);
    if (cta == 0 && warp == 0 && plan != nullptr) {  // for the merge
      if (lane == 0) plan[0] = per * NW;
      if (lane < rw.B) plan[1 + lane] = incl - w;
      if (lane == rw.B - 1) plan[1 + rw.B] = incl;
    }
    if (per * NW * cta >= all) return RunPlan{-1, 0, 0, 0, 0};
    p0 = per * (static_cast<long long>(NW) * cta + warp);
    have = p0 < all;
    const long long at = static_cast<long long>(incl - w) * rw.upr;
    const uint32_t mine =
        __ballot_sync(0xffffffffu, p0 >= at && p0 < static_cast<long long>(incl) * rw.upr);
    r.b = have ? __ffs(mine) - 1 : 0;
    r.off = have ? p0 - __shfl_sync(0xffffffffu, at, r.b) : 0;
    r.len = __shfl_sync(0xffffffffu, len, r.b);
    __syncwarp();
  } else {
    const int per_t = (rw.B + NW * 32 - 1) / (NW * 32);
    const int b0 = min(tid * per_t, rw.B), b1 = min(b0 + per_t, rw.B);
    long long sum = 0;
    for (int b = b0; b < b1; ++b) {
      const int raw = __ldcg(rw.seq_lens + b);
      const int len = min(max(raw, 0), rw.max_len);
      if (cta == 0 && raw != len) atomicOr(err, ATTN_DEVERR_BAD_SEQ_LEN);
      if (b < kLenCache) sh.len[b] = len;
      sum += row_weight(rw, len);
    }
    long long incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) sh.warp[warp] = incl;
    sync();
    long long before = incl - sum, total = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      if (w < warp) before += sh.warp[w];
      total += sh.warp[w];
    }
    all = total * rw.upr;
    per = per_of(all);
    const long long cta0 = per * NW * cta;
    if (cta == 0 && plan != nullptr) {  // for the merge
      if (tid == 0) plan[0] = per * NW;
      long long at = before;
      for (int b = b0; b < b1; ++b) {
        plan[1 + b] = at;
        at += row_weight(rw, row_len(rw, sh.len, b));
        if (b == rw.B - 1) plan[1 + rw.B] = at;
      }
    }
    if (cta0 >= all) return RunPlan{-1, 0, 0, 0, 0};
    long long at = before * rw.upr;
    const long long end = (before + sum) * rw.upr;
    if (cta0 + per * NW > at && cta0 < end) {
      for (int b = b0; b < b1; ++b) {
        const long long next = at + static_cast<long long>(row_weight(rw, row_len(rw, sh.len, b))) * rw.upr;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          const long long p = cta0 + per * w;
          if (p >= at && p < next) {
            sh.b[w] = b;
            sh.off[w] = p - at;
          }
        }
        at = next;
      }
    }
    sync();
    p0 = cta0 + per * warp;
    have = p0 < all;
    r.b = have ? sh.b[warp] : 0;
    r.off = have ? sh.off[warp] : 0;
    r.len = row_len(rw, sh.len, r.b);
  }
  r.rem = have ? min(per, all - p0) : 0;
  r.per = per;
  return r;
}

// The same out of line, for shared_kernel, whose two phases miss the instruction
// cache as it is (a third of its warps' waits with 64 rows over 8192 keys). With
// the plan inlined 256 rows over a prefix of 32768 keys took 192 us instead of
// 182, 64 over 8192 50.9 instead of 50.3; the 8-bit decode takes it inlined (a row
// of 32768 keys 20.7 us, this way 20.9).
template <int NW, class R, class Sync>
__device__ __noinline__ RunPlan plan_runs_apart(const R rw, long long* plan, RunShared<NW>& sh,
                                                int cta, int n_cta, unsigned int* err, Sync sync) {
  return plan_runs(rw, plan, sh, cta, n_cta, err, sync);
}

// The whole of CTA `cta` of `n_cta`, by NW warps (threads 0 .. NW * 32 - 1), which
// `sync` joins; `smem` starts at a 1024-byte boundary. Returns with every copy
// landed.
template <bool E8, int D, int NW, int NST, class R, class Sync>
__device__ __forceinline__ void runs_body(
    const uint8_t* __restrict__ kc, const uint8_t* __restrict__ vc, const uint8_t* __restrict__ ks,
    const uint8_t* __restrict__ vs, const __nv_bfloat16* __restrict__ q,
    const int32_t* __restrict__ block_table, const R rw, int h, int h_kv, int g, int max_blocks,
    int num_blocks, float qscale, const RunOut& out, uint8_t* smem, RunShared<NW>& sh, int cta,
    int n_cta, unsigned int* err, Sync sync) {
  using C = Cfg<E8, D, NW, NST>;
  constexpr bool WIN = R::kWindow;
  constexpr bool FINAL = E8 || WIN;  // units that no border cuts: o and lse, else row states
  constexpr int KS = D / 16;  // MMA steps over d_h
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gid = lane >> 2, tq = lane & 3;
  const int n_gb = rw.n_gb;

  const uint32_t sbase = smem_u32(smem);
  float* join = reinterpret_cast<float*>(smem + C::JOIN_OFF);
  float* ms = reinterpret_cast<float*>(smem + C::ML_OFF);  // [warp][8]
  float* ls = ms + NW * 8;
  auto& s_kind = sh.kind;
  auto& s_own = sh.own;
  auto& s_own_row = sh.own_row;
  auto& s_own_nh = sh.own_nh;
  auto& s_len = sh.len;
  // The unit that goes on behind a warp's run: accumulators, then m and l, in
  // the warp's ring, free by then.
  auto tail_of = [&](int w) { return reinterpret_cast<float*>(smem + w * NST * C::STAGE_BYTES); };

  RunPlan plan;
  if constexpr (FINAL)
    plan = plan_runs(rw, out.plan, sh, cta, n_cta, err, sync);
  else
    plan = plan_runs_apart(rw, out.plan, sh, cta, n_cta, err, sync);
  if (plan.rem < 0) return;  // nothing for this CTA
  bool have = plan.rem > 0;
  Walk cw;
  cw.b = plan.b;
  cw.len = plan.len;
  const long long off = plan.off;
  cw.np = rw.pages(cw.len);
  cw.rem = plan.rem;
  {
    const int wu = cw.np + R::kUnit;
    cw.u = static_cast<int>(div_ll(off, wu));
    walk_open<R::kUnit>(cw, off - static_cast<long long>(cw.u) * wu);
  }

  // ---- producer state: the same walk, NST pages ahead ----
  Walk pw = cw;
  bool more = have;
  int pi = pw.lo;  // next page to issue
  int bt = -1;     // table entries of the next pages, 32 at a time
  int issued = 0;
  auto load_bt = [&](int i) {
    bt = i + lane < pw.hi
             ? __ldcg(block_table + static_cast<size_t>(pw.b) * max_blocks + rw.page_at(pw.len, i + lane))
             : -1;
  };
  const uint32_t ring = sbase + warp * NST * C::STAGE_BYTES;
  const uint32_t exps = sbase + C::EXP_OFF + warp * NST * C::EXP_BYTES;
  const uint64_t policy = policy_evict_first();
  int bt_i = 0;  // pages taken from bt
  if (more) load_bt(pi);
  // Copies of this warp's next page, if there is one, into stage issued % NST;
  // one group of copies either way.
  auto issue_next = [&]() {
    while (more && pi >= pw.hi) {
      more = walk_next(pw, rw, s_len);
      pi = pw.lo;
      bt_i = 0;
      if (more) load_bt(pi);
    }
    if (more) {
      if (bt_i == 32) {
        bt_i = 0;
        load_bt(pi);
      }
      const int phys = __shfl_sync(0xffffffffu, bt, bt_i);
      const bool live = phys >= 0 && phys < num_blocks;  // else the page reads as zeros
      if (!live && lane == 0) atomicOr(err, ATTN_DEVERR_BAD_PAGE);
      const int st = issued % NST, kvh = pw.u / n_gb;
      const size_t page = live ? phys : 0;
      const uint32_t kd = ring + st * C::STAGE_BYTES, vd = kd + C::PAGE_BYTES;
      constexpr int CPR = C::PAGE_BYTES / (kPage * 16);  // chunks per row
      constexpr int RPI = 32 / CPR;                      // rows per instruction
      const int r = lane / CPR, c = lane % CPR;
      const size_t row_bytes = E8 ? D : static_cast<size_t>(h_kv) * D * 2;
      const size_t off = (E8 ? (page * h_kv + kvh) * C::PAGE_BYTES
                             : (page * kPage * h_kv + kvh) * (D * 2)) +
                         r * row_bytes + c * 16;
#pragma unroll
      for (int j = 0; j < kPage / RPI; ++j)
        copy16(chunk_at<E8, D>(kd, j * RPI + r, c), kc + off + j * RPI * row_bytes, live, policy);
#pragma unroll
      for (int j = 0; j < kPage / RPI; ++j)
        copy16(chunk_at<E8, D>(vd, j * RPI + r, c), vc + off + j * RPI * row_bytes, live, policy);
      if constexpr (E8) {
        if (lane < 2)
          copy16_line(exps + st * 32 + lane * 16, (lane ? vs : ks) + (page * h_kv + kvh) * kPage, live);
      }
      ++issued;
      ++bt_i;
      ++pi;
    }
    copies_commit();
  };
  for (int i = 0; i < NST; ++i) issue_next();

  float m0 = kNone, m1 = kNone, l0 = 0.f, l1 = 0.f;
  float acc[KS][4];

  // Emits dims 16k .. 16k + 15 of a state (accumulators relative to 2^m, in
  // log2 units): into `slot` of the partial states, or (slot < 0) as the row's
  // final output (8-bit) or its own-keys state (bf16); with k = 0 the scalars.
  auto emit = [&](long long slot, size_t row0, int nh, int k, const float (&x)[4], float M0, float M1,
                  float L0, float L1) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int head = 2 * tq + e;
      if (head >= nh) continue;
      const float L = e ? L1 : L0, M = e ? M1 : M0;
      const size_t row = row0 + head;
      if (!ATTN_GUARD(row < static_cast<size_t>(rw.B) * h, err)) continue;
      if (FINAL && slot < 0) {
        const bool empty = L == 0.f;  // every logit -inf
        const float inv = empty ? 0.f : 1.f / L;
        if constexpr (E8) {
          *reinterpret_cast<uint32_t*>(out.o + row * D + 16 * k + 2 * gid) =
              empty ? 0u : pack_bf16x2(x[e] * inv, x[2 + e] * inv);
        } else {
          out.o[row * D + 16 * k + gid] = __float2bfloat16(empty ? 0.f : x[e] * inv);
          out.o[row * D + 16 * k + 8 + gid] = __float2bfloat16(empty ? 0.f : x[2 + e] * inv);
        }
        if (k == 0 && out.lse != nullptr && gid == 0)
          out.lse[row] = empty ? -INFINITY : M * kLn2 + logf(L);
        continue;
      }
      const size_t at = slot < 0 ? row : static_cast<size_t>(slot) * 8 + head;
      if (!ATTN_GUARD(slot < 0 || at < static_cast<size_t>(n_cta) * 16, err)) continue;
      float* so = (slot < 0 ? out.o_row : out.o_part) + at * D;
      if constexpr (E8) {
        *reinterpret_cast<float2*>(so + 16 * k + 2 * gid) = make_float2(x[e], x[2 + e]);
      } else {
        so[16 * k + gid] = x[e];
        so[16 * k + 8 + gid] = x[2 + e];
      }
      if (k == 0 && gid == 0) {
        (slot < 0 ? out.m_row : out.m_part)[at] = M;
        (slot < 0 ? out.l_row : out.l_part)[at] = L;
      }
    }
  };
  auto emit_all = [&](long long slot, size_t row0, int nh) {
#pragma unroll
    for (int k = 0; k < KS; ++k) emit(slot, row0, nh, k, acc[k], m0, m1, l0, l1);
  };
  float* const tail = tail_of(warp);

  int used = 0;      // stages consumed
  const int v_row = 8 * ((lane >> 3) & 1) + (lane & 7), v_dc = lane >> 4;

  while (have) {  // ---- one unit of the run ----
    if (cw.hi <= cw.lo) {  // the run ends before the unit's first page
      have = walk_next(cw, rw, s_len);
      continue;
    }
    const int kvh = cw.u / n_gb, gb = cw.u % n_gb;
    const int hq0 = kvh * g + gb * 8;     // first query head of the block
    const int nh = min(8, g - gb * 8);    // heads in the block

    // q as the B operand: lane (gid, tq) holds head gid's dims of the chunks
    // that lanes tq read of K (8-bit: 32 or 16 consecutive dims).
    uint32_t qb[KS][2];
    float hc = qscale;
    if constexpr (E8) {
      constexpr int NC = D / 64;  // 16-dim chunks per lane
      float x[NC * 16];
#pragma unroll
      for (int c = 0; c < NC * 2; ++c) {
        uint4 t = make_uint4(0u, 0u, 0u, 0u);
        if (gid < nh)
          t = __ldcg(reinterpret_cast<const uint4*>(
              q + (static_cast<size_t>(cw.b) * h + hq0 + gid) * D + tq * (NC * 16) + c * 8));
        const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[c * 8 + 2 * i] = bf16lo(w[i]);
          x[c * 8 + 2 * i + 1] = bf16hi(w[i]);
        }
      }
      uint32_t a = 0;
#pragma unroll
      for (int i = 0; i < NC * 16; ++i) {
        const uint32_t b = __float_as_uint(x[i]) & 0x7fffffffu;
        a = max(a, b >= 0x7f800000u ? 0u : b);
      }
      a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
      a = max(a, __shfl_xor_sync(0xffffffffu, a, 2));
      // Largest finite magnitude to [2^14, 2^15); exponents below 2^-112 (and
      // zero rows) are treated as 2^-112.
      const int be = max(static_cast<int>(a >> 23), 15);     // biased exponent
      const float up = __uint_as_float(static_cast<uint32_t>(min(254, 127 + 14 + 127 - be)) << 23);
      const int down = min(be - 14, 240);
      hc = qscale * __uint_as_float(static_cast<uint32_t>(max(down, 1)) << 23);
#pragma unroll
      for (int ksi = 0; ksi < KS; ++ksi) {
        qb[ksi][0] = pack_f16x2(x[ksi * 4] * up, x[ksi * 4 + 1] * up);
        qb[ksi][1] = pack_f16x2(x[ksi * 4 + 2] * up, x[ksi * 4 + 3] * up);
      }
    } else {
      // bf16: chunks 2tq, 2tq + 1 (8 dims each) of every 64-element half.
#pragma unroll
      for (int c = 0; c < KS / 2; ++c) {
        uint4 t = make_uint4(0u, 0u, 0u, 0u);
        if (gid < nh)
          t = __ldcg(reinterpret_cast<const uint4*>(
              q + (static_cast<size_t>(cw.b) * h + hq0 + gid) * D + (c >> 1) * 64 +
              (2 * tq + (c & 1)) * 8));
        qb[2 * c][0] = t.x;
        qb[2 * c][1] = t.y;
        qb[2 * c + 1][0] = t.z;
        qb[2 * c + 1][1] = t.w;
      }
    }
    const float hc0 = __shfl_sync(0xffffffffu, hc, (2 * tq) * 4);
    const float hc1 = __shfl_sync(0xffffffffu, hc, (2 * tq + 1) * 4);
    const float lo0 = fminf(hc0, 1.f), lo1 = fminf(hc1, 1.f), up0 = fmaxf(hc0, 1.f), up1 = fmaxf(hc1, 1.f);

    // State of heads 2tq, 2tq + 1: normaliser share l of this lane's keys
    // relative to 2^m, accumulators relative to 2^r.
    m0 = m1 = kNone;
    l0 = l1 = 0.f;
    float d0 = 0.f, d1 = 0.f, c0 = 1.f, c1 = 1.f;  // d: r - m, c: 2^-d
#pragma unroll
    for (int i = 0; i < KS; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;

    int sink_pages = 0;
    if constexpr (WIN) sink_pages = rw.sink_pages(cw.len);

    for (int i = cw.lo; i < cw.hi; ++i) {
      const int st = used % NST;
      copies_wait<NST - 1>();
      __syncwarp();
      const uint32_t kp = ring + st * C::STAGE_BYTES, vp = kp + C::PAGE_BYTES;
      // Slots that the row sees: below `valid`, or (window) the bits of `vis`.
      const int valid = WIN ? kPage : min(kPage, cw.len - i * kPage);
      uint32_t vis = 0xffffu;
      if constexpr (WIN) {  // only a part's first and last page can be seen in part
        if (i + 1 == sink_pages || i == sink_pages || i + 1 == cw.np)
          vis = rw.visible(cw.len, rw.page_at(cw.len, i));
      }
      const bool partial = WIN ? vis != 0xffffu : valid < kPage;
      auto live = [&](int slot) { return WIN ? ((vis >> slot) & 1u) != 0u : slot < valid; };
      if (partial) {
        // Slots out of sight hold whatever the cache holds there (NaN codes
        // among it); their weights are 0, but 0 * NaN is not.
        constexpr int CPR = C::PAGE_BYTES / (kPage * 16);
        for (int c = lane; c < (WIN ? kPage : kPage - valid) * CPR; c += 32)
          if (!WIN || !live(c / CPR))
            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(
                             chunk_at<E8, D>(vp, (WIN ? 0 : valid) + c / CPR, c % CPR)),
                         "r"(0u)
                         : "memory");
        __syncwarp();
      }

      // ---- S^T = K q^T: keys gid and gid + 8, heads 2tq and 2tq + 1 ----
      // s[2 i + e]: key gid + 8 i, head 2 tq + e.
      float s[4] = {0.f, 0.f, 0.f, 0.f};
      uint32_t fa = 0, fb = 0;  // exponent bytes of the values
      if constexpr (E8) {
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          const int ch = tq * (D / 64) + c;
          const uint4 x = lds128(chunk_at<E8, D>(kp, gid, ch));
          const uint4 y = lds128(chunk_at<E8, D>(kp, gid + 8, ch));
          const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t a0 = e4m3::decode2(static_cast<uint16_t>(xw[j]));
            const uint32_t a1 = e4m3::decode2(static_cast<uint16_t>(yw[j]));
            const uint32_t a2 = e4m3::decode2(static_cast<uint16_t>(xw[j] >> 16));
            const uint32_t a3 = e4m3::decode2(static_cast<uint16_t>(yw[j] >> 16));
            mma_f16(s, a0, a1, a2, a3, qb[c * 4 + j][0], qb[c * 4 + j][1]);
          }
        }
        const uint32_t ep = exps + st * 32;
        const float ka = e4m3::scale_of(lds_u8(ep + gid)), kb = e4m3::scale_of(lds_u8(ep + gid + 8));
        fa = lds_u8(ep + 16 + gid);
        fb = lds_u8(ep + 24 + gid);
        // hc ka may be infinite where the score is not, its two parts' products cannot.
        // (Rounded here, and not joined with the differences from the reference below.)
        s[0] = __fmul_rn(s[0] * (lo0 * ka), up0);
        s[1] = __fmul_rn(s[1] * (lo1 * ka), up1);
        s[2] = __fmul_rn(s[2] * (lo0 * kb), up0);
        s[3] = __fmul_rn(s[3] * (lo1 * kb), up1);
      } else {
        float s2[4] = {0.f, 0.f, 0.f, 0.f};  // two chains: half the latency
#pragma unroll
        for (int c = 0; c < KS / 2; ++c) {
          const int ch = (c >> 1) * 8 + 2 * tq + (c & 1);
          const uint4 x = lds128(chunk_at<E8, D>(kp, gid, ch));
          const uint4 y = lds128(chunk_at<E8, D>(kp, gid + 8, ch));
          mma_bf16(s, x.x, y.x, x.y, y.y, qb[2 * c][0], qb[2 * c][1]);
          mma_bf16(s2, x.z, y.z, x.w, y.w, qb[2 * c + 1][0], qb[2 * c + 1][1]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] = __fmul_rn(s[i] + s2[i], i & 1 ? hc1 : hc0);  // (as above)
      }

      // ---- weights: p relative to m, w (8-bit) relative to r ----
      float p0, p1, p2, p3, w0, w1, w2, w3;
      auto weights = [&] {
        float x[4] = {s[0] - m0, s[1] - m1, s[2] - m0, s[3] - m1};
        float va = e4m3::scale_of(fa), vb = e4m3::scale_of(fb);
        if (partial) {  // slots out of sight: weight 0, whatever they hold
          if (!live(gid)) x[0] = x[1] = -INFINITY, va = 0.f;
          if (!live(gid + 8)) x[2] = x[3] = -INFINITY, vb = 0.f;
        }
        p0 = ex2_approx(x[0]);
        p1 = ex2_approx(x[1]);
        p2 = ex2_approx(x[2]);
        p3 = ex2_approx(x[3]);
        if constexpr (E8) {  // 2^(s + f - r) = p * 2^-d * 2^f, in the order whose
          w0 = (p0 * c0) * va;  // first product is finite (2^f 2^-d may not be)
          w1 = (p1 * c1) * va;
          w2 = (p2 * c0) * vb;
          w3 = (p3 * c1) * vb;
        }
      };
      weights();
      // The references move only when a weight passes 2^kSlack (or a fp16
      // weight 2^15); a NaN never compares, and reaches l and O as it is.
      bool up = fmaxf(fmaxf(p0, p1), fmaxf(p2, p3)) > 4.f;
      if constexpr (E8) up = up || fmaxf(fmaxf(w0, w1), fmaxf(w2, w3)) > 32768.f;
      if (__any_sync(0xffffffffu, up)) {
        const bool la = live(gid), lb = live(gid + 8);
        const float s0 = la ? s[0] : -INFINITY, s1 = la ? s[1] : -INFINITY;
        const float s2 = lb ? s[2] : -INFINITY, s3 = lb ? s[3] : -INFINITY;
        const float ga = static_cast<float>(static_cast<int>(fa) - 127);
        const float gb2 = static_cast<float>(static_cast<int>(fb) - 127);
        float n0 = fmaxf(s0, s2), n1 = fmaxf(s1, s3);
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
          n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, off));
          n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, off));
        }
        n0 = fmaxf(n0, m0);
        n1 = fmaxf(n1, m1);
        float a0 = ex2_approx(m0 - n0), a1 = ex2_approx(m1 - n1);
        l0 *= a0;
        l1 *= a1;
        if constexpr (E8) {
          float t0 = fmaxf(s0 - n0 + ga, s2 - n0 + gb2), t1 = fmaxf(s1 - n1 + ga, s3 - n1 + gb2);
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) {
            t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, off));
            t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, off));
          }
          // d stays above -120, so that 2^-d is finite: values all below 2^-107
          // (rows of zeros among them) then have weights up to 2^3 instead of 2^13.
          const float b0 = d0 + (m0 - n0), b1 = d1 + (m1 - n1);  // the old r, from the new m
          d0 = fmaxf(fmaxf(t0 - kTop, b0), -120.f);
          d1 = fmaxf(fmaxf(t1 - kTop, b1), -120.f);
          a0 = ex2_approx(b0 - d0);
          a1 = ex2_approx(b1 - d1);
          c0 = ex2_approx(-d0);
          c1 = ex2_approx(-d1);
        }
        m0 = n0;
        m1 = n1;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          acc[k][0] *= a0;
          acc[k][1] *= a1;
          acc[k][2] *= a0;
          acc[k][3] *= a1;
        }
        weights();
      }
      l0 += p0 + p2;
      l1 += p1 + p3;
      if constexpr (E8) {
        const uint32_t pb0 = movmatrix_t(pack_f16x2(w0, w1)), pb1 = movmatrix_t(pack_f16x2(w2, w3));
        // O^T += V^T P^T: rows gid, gid + 8 of step k are dims 16k + 2 gid and
        // 16k + 2 gid + 1.
#pragma unroll
        for (int k = 0; k < KS; k += 2) {
          uint32_t r[4];
          ldsm_x4_t(chunk_at<E8, D>(vp, v_row, k + v_dc), r);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            uint32_t x, y;
            asm("prmt.b32 %0, %1, %1, 0x3120;" : "=r"(x) : "r"(r[2 * e]));
            asm("prmt.b32 %0, %1, %1, 0x3120;" : "=r"(y) : "r"(r[2 * e + 1]));
            mma_f16(acc[k + e], e4m3::decode2(static_cast<uint16_t>(x)),
                    e4m3::decode2(static_cast<uint16_t>(x >> 16)),
                    e4m3::decode2(static_cast<uint16_t>(y)),
                    e4m3::decode2(static_cast<uint16_t>(y >> 16)), pb0, pb1);
          }
        }
      } else {
        const uint32_t h0 = movmatrix_t(split_hi(p0, p1)), h1 = movmatrix_t(split_hi(p2, p3));
        const uint32_t e0 = movmatrix_t(split_lo(p0, p1)), e1 = movmatrix_t(split_lo(p2, p3));
        // Rows gid, gid + 8 of step k are dims 16k + gid and 16k + 8 + gid.
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          uint32_t r[4];
          ldsm_x4_t(chunk_at<E8, D>(vp, v_row, 2 * k + v_dc), r);
          mma_bf16(acc[k], r[0], r[2], r[1], r[3], h0, h1);
          mma_bf16(acc[k], r[0], r[2], r[1], r[3], e0, e1);
        }
      }
      __syncwarp();
      ++used;
      issue_next();
    }

    // ---- the unit's state: normaliser over all keys, accumulators relative
    // to 2^m ----
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, off);
      l1 += __shfl_xor_sync(0xffffffffu, l1, off);
    }
    if constexpr (E8) {
      const float f0 = ex2_approx(d0), f1 = ex2_approx(d1);
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        acc[k][0] *= f0;
        acc[k][1] *= f1;
        acc[k][2] *= f0;
        acc[k][3] *= f1;
      }
    }
    const size_t row0 = static_cast<size_t>(cw.b) * h + hq0;
    const bool begins = cw.lo == 0, ends = cw.hi == cw.np;
    if (begins && ends) {
      emit_all(-1, row0, nh);
    } else if (warp == 0 && !begins && ends) {  // began before the CTA
      emit_all(2ll * cta, row0, nh);
    } else {
      // Cut: kept for the join. A part that began in this run, or before the
      // CTA and goes on, starts a chain (always the run's last unit: the ring
      // is free); others continue one.
      const bool starts = begins || warp == 0;
      float* dst = starts ? tail : join + warp * C::NREG * 32;
#pragma unroll
      for (int i = 0; i < C::NREG; ++i) dst[i * 32 + lane] = acc[i >> 2][i & 3];
      if (gid == 0) {
        float* md = starts ? tail + C::NREG * 32 : ms + warp * 8;
        float* ld = starts ? tail + C::NREG * 32 + 8 : ls + warp * 8;
        md[2 * tq] = m0;
        md[2 * tq + 1] = m1;
        ld[2 * tq] = l0;
        ld[2 * tq + 1] = l1;
      }
      if (lane == 0) {
        if (starts) {
          s_own[warp] = begins ? 1 : 2;
          s_own_row[warp] = static_cast<int>(row0);
          s_own_nh[warp] = nh;
          if constexpr (WIN) sh.own_left[warp] = cw.np - cw.hi;
        } else {
          s_kind[warp] = ends ? 2 : 1;
        }
      }
    }
    have = walk_next(cw, rw, s_len);
  }

  // ---- join the units cut between this CTA's warps ----
  sync();
  if (warp < KS) {
    const int k = warp;
    int open = 0, row0 = 0, nh = 0, opened = 0;  // the chain: 0 none, else its s_own; its warp
    float x[4] = {0.f, 0.f, 0.f, 0.f};
    float M0 = 0.f, M1 = 0.f, L0 = 0.f, L1 = 0.f;
#pragma unroll 1
    for (int w = 0; w < NW; ++w) {
      const int kind = s_kind[w], own = s_own[w];
      if (kind != 0 && open != 0) {
        const float n0 = ms[w * 8 + 2 * tq], n1 = ms[w * 8 + 2 * tq + 1];
        const float T0 = fmaxf(M0, n0), T1 = fmaxf(M1, n1);
        const float a0 = ex2_approx(M0 - T0), a1 = ex2_approx(M1 - T1);
        const float c0 = ex2_approx(n0 - T0), c1 = ex2_approx(n1 - T1);
        L0 = L0 * a0 + ls[w * 8 + 2 * tq] * c0;
        L1 = L1 * a1 + ls[w * 8 + 2 * tq + 1] * c1;
        M0 = T0;
        M1 = T1;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          x[i] = x[i] * ((i & 1) ? a1 : a0) +
                 join[(w * C::NREG + 4 * k + i) * 32 + lane] * ((i & 1) ? c1 : c0);
        if (kind == 2) {
          emit(open == 2 ? 2ll * cta : -1ll, row0, nh, k, x, M0, M1, L0, L1);
          open = 0;
        }
      }
      if (own != 0) {
        const float* t = tail_of(w);
        open = own;
        opened = w;
        row0 = s_own_row[w];
        nh = s_own_nh[w];
        M0 = t[C::NREG * 32 + 2 * tq];
        M1 = t[C::NREG * 32 + 2 * tq + 1];
        L0 = t[C::NREG * 32 + 8 + 2 * tq];
        L1 = t[C::NREG * 32 + 8 + 2 * tq + 1];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = t[(4 * k + i) * 32 + lane];
      }
    }
    if (open != 0)
      emit(2ll * cta + (open == 1 ? 1 : 0), row0, nh, k, x, M0, M1, L0, L1);
    if constexpr (WIN) {
      // The unit that began in this CTA and goes on behind it: the weight that is left
      // of it is spread over the CTAs behind.
      if (out.cut != nullptr && tid == 0 && open == 1) {
        const long long left = sh.own_left[opened] - plan.per * (NW - 1 - opened);
        out.cut[cta] = RunCut{static_cast<int>(1 + div_ll(left + plan.per * NW - 1, plan.per * NW)), row0, nh};
      }
    }
  }
}

}  // namespace
}  // namespace attn
