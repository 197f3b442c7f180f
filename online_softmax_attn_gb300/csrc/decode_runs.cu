// decode_runs.cu -- paged decode attention with the keys of the whole batch cut
// into equal runs: over the 8-bit cache (attn_decode_paged_e4m3), and over the
// rows' own bf16 pages in attn_decode_paged_shared.
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
// magnitudes are, so P V is one fp16 product against the codes themselves. q
// is scaled per head by a power of two to a largest magnitude in
// [2^14, 2^15), where fp16 holds bf16's 8 significant bits down to 2^-28 of
// that maximum. ldmatrix moves byte pairs (two dims of a key); one prmt puts
// the same dim of two keys side by side.
//
// bf16 cache: q, K and V enter as they are; P is the two-term bf16 split
// P_hi + P_lo (a single bf16 weight would cost up to 2^-8 of itself).
//
// Bound by memory: 2 (d_h + 1) or 4 d_h bytes per key and KV head. A warp owns
// a ring of NST stages, each one page of K and V (TMA, swizzled), for the 8-bit
// cache with their exponents (16-byte bulk copies).
//
// Work split: the (row, KV head, head block) units, laid end to end with a
// weight of np + kUnit for np pages, are cut into equal runs, one per warp, so
// any mix of lengths fills the machine and the launch does not depend on the
// lengths. A warp works through its run unit by unit on its own (no barrier, no
// join between units) and finishes each unit that lies inside its run. Units
// cut by a run border are joined at the CTA's end: the warp that has a unit's
// first part adds the following warps' parts from shared memory. What reaches
// past the CTA leaves at most two partial states per CTA (a unit that began
// before it, one that goes on behind it), which the merge kernel joins in run
// order. (Splitting a unit over all warps of a CTA and joining at every unit's
// end instead took 57 us for 64 rows of up to 1000 keys, 131 MB: rows of a few
// pages cost a CTA as much as rows of hundreds.)
#include "common.cuh"
#include "e4m3.cuh"
#include "internal.h"
#include "pdl.cuh"

namespace attn {

static __device__ unsigned int g_decode_runs_err;
// Exponents of a page outside the cache (its codes read as zeros).
static __device__ __align__(16) const uint8_t g_unit_exp[16] = {127, 127, 127, 127, 127, 127, 127, 127,
                                                                127, 127, 127, 127, 127, 127, 127, 127};

namespace {

using e4m3::kPage;

// Weights are at most 2^15 (fp16's largest finite number is 65504): the
// reference r is set to 13 below a new running max's weight and moves once a
// weight would pass 2^15. Weights down to 2^-27 of the largest are then normal
// fp16 numbers, and what fp16 drops below 2^-38 of it is under 2^-20 of the sum
// even for 2^18 keys.
constexpr float kTop = 13.0f, kSlack = 2.0f;
constexpr float kNone = -1e30f;  // reference before the first key

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
__device__ __forceinline__ void tma_load_3d_hint(uint32_t dst, const void* tmap, uint32_t bar,
                                                 int c0, int c1, int c2, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void bulk_load16(uint32_t dst, const void* src, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], 16, [%2];" ::"r"(dst),
      "l"(src), "r"(bar)
      : "memory");
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
  static constexpr int BAR_OFF = ML_OFF + 2 * NW * 8 * 4;
  static constexpr int SMEM = BAR_OFF + NW * NST * 8 + 1024;
  static_assert(NW * NST <= 32, "one lane initialises each barrier");
  // Static shared memory (kLenCache lengths and some words, 1248) and the driver's
  // 1 KB come on top.
  static constexpr int CTAS = E8 ? 2 : 1;  // per SM
  static_assert(CTAS * (SMEM + 1248 + 1024) <= 228 * 1024, "shared memory of the CTAs on an SM");
};

// 16-byte chunk `c` of key row `r` of a page: the TMA's swizzle. 8-bit codes:
// rows of 128 (128-byte swizzle) or 64 bytes (64-byte swizzle); bf16: halves
// of 64 elements, rows of 128 bytes.
template <bool E8, int D>
__device__ __forceinline__ uint32_t chunk_at(uint32_t page, int r, int c) {
  if constexpr (E8)
    return page + r * D + ((c ^ (D == 128 ? (r & 7) : ((r >> 1) & 3))) << 4);
  else
    return page + (c >> 3) * (kPage * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

// Where states and results go. Units cut by a run border: part (two slots of 8
// heads per CTA). Other units: o and lse themselves (8-bit decode), or a state
// per (row, head) in row_* (shared-prefix decode, whose merge adds the prefix).
struct RunOut {
  long long* plan;
  float *o_part, *m_part, *l_part;
  float *o_row, *m_row, *l_row;
  __nv_bfloat16* o;
  float* lse;
};

constexpr int kUnit = kRunsUnit;  // a unit's query, state and epilogue, in pages
constexpr int kMinRun = 1;      // least weight of a warp's run
constexpr int kLenCache = 256;  // row lengths kept in shared memory

struct Rows {
  const int32_t* seq_lens;
  int B, max_len, upr;  // upr: units per row
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
__device__ __forceinline__ int row_weight(int len) {  // of one unit of the row
  return len > 0 ? (len + kPage - 1) / kPage + kUnit : 0;
}
// Opens unit w.u of row w.b at weight `off` within it.
__device__ __forceinline__ void walk_open(Walk& w, long long off) {
  const long long take = min(w.np + kUnit - off, w.rem);
  w.lo = static_cast<int>(max(off - kUnit, 0ll));
  w.hi = static_cast<int>(max(off + take - kUnit, 0ll));
  w.rem -= take;
}
// Next unit of the run; false at its end.
__device__ __forceinline__ bool walk_next(Walk& w, const Rows& rw, const int* cached) {
  if (w.rem <= 0) return false;
  if (++w.u == rw.upr) {
    w.u = 0;
    do {
      ++w.b;
      if (w.b >= rw.B) return false;
      w.len = row_len(rw, cached, w.b);
    } while (w.len == 0);
    w.np = (w.len + kPage - 1) / kPage;
  }
  walk_open(w, 0);
  return true;
}

template <bool E8, int D, int NW, int NST>
__global__ void __launch_bounds__(NW * 32, Cfg<E8, D, NW, NST>::CTAS)
    decode_runs_kernel(const __grid_constant__ CUtensorMap tmap_k,
                   const __grid_constant__ CUtensorMap tmap_v, const uint8_t* __restrict__ ks,
                   const uint8_t* __restrict__ vs, const __nv_bfloat16* __restrict__ q,
                   const int32_t* __restrict__ block_table, Rows rw, int h, int h_kv, int g,
                   int max_blocks, int num_blocks, float qscale, const RunOut out) {
  using C = Cfg<E8, D, NW, NST>;
  constexpr int KS = D / 16;  // MMA steps over d_h
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gid = lane >> 2, tq = lane & 3;
  const int n_gb = rw.upr / h_kv;

  extern __shared__ __align__(16) uint8_t smem_raw[];  // (1024 would pad the static part)
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  float* join = reinterpret_cast<float*>(smem + C::JOIN_OFF);
  float* ms = reinterpret_cast<float*>(smem + C::ML_OFF);  // [warp][8]
  float* ls = ms + NW * 8;
  __shared__ long long s_warp[NW];
  __shared__ long long s_off[NW];  // weight between a warp's first row and its run
  __shared__ int s_b[NW];          // its first row
  __shared__ int s_kind[NW];       // its stored part: 0 none, 1 the unit goes on, 2 it ends
  __shared__ int s_len[kLenCache];

  if (warp == 0) {
    if (lane < NW * NST) mbar_init(sbase + C::BAR_OFF + lane * 8, 1);
    fence_barrier_init();
    if (lane == 0) {
      prefetch_tmap(&tmap_k);
      prefetch_tmap(&tmap_v);
    }
  }
  pdl_wait();     // lengths, table, q and the cache are earlier kernels' output
  pdl_trigger();

  // ---- the runs: prefix sums of the rows' weights (per unit) ----
  const int per_t = (rw.B + NW * 32 - 1) / (NW * 32);
  const int b0 = min(tid * per_t, rw.B), b1 = min(b0 + per_t, rw.B);
  long long sum = 0;
  for (int b = b0; b < b1; ++b) {
    const int raw = __ldcg(rw.seq_lens + b);
    const int len = min(max(raw, 0), rw.max_len);
    if (blockIdx.x == 0 && raw != len) atomicOr(&g_decode_runs_err, ATTN_DEVERR_BAD_SEQ_LEN);
    if (b < kLenCache) s_len[b] = len;
    sum += row_weight(len);
  }
  long long incl = sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += y;
  }
  if (lane == 31) s_warp[warp] = incl;
  if (tid < NW) s_kind[tid] = 0;
  __syncthreads();
  long long before = incl - sum, total = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    if (w < warp) before += s_warp[w];
    total += s_warp[w];
  }
  const long long all = total * rw.upr;
  const long long n_runs = static_cast<long long>(gridDim.x) * NW;
  const long long per = max(static_cast<long long>(kMinRun), (all + n_runs - 1) / n_runs);
  const long long cta0 = per * NW * blockIdx.x;
  if (blockIdx.x == 0) {  // for the merge
    if (tid == 0) out.plan[0] = per * NW;
    long long at = before;
    for (int b = b0; b < b1; ++b) {
      out.plan[1 + b] = at;
      at += row_weight(row_len(rw, s_len, b));
      if (b == rw.B - 1) out.plan[1 + rw.B] = at;
    }
  }
  if (cta0 >= all) return;
  {
    long long at = before * rw.upr;
    const long long end = (before + sum) * rw.upr;
    if (cta0 + per * NW > at && cta0 < end) {
      for (int b = b0; b < b1; ++b) {
        const long long next = at + static_cast<long long>(row_weight(row_len(rw, s_len, b))) * rw.upr;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          const long long p = cta0 + per * w;
          if (p >= at && p < next) {
            s_b[w] = b;
            s_off[w] = p - at;
          }
        }
        at = next;
      }
    }
  }
  __syncthreads();
  const long long p0 = cta0 + per * warp;
  bool have = p0 < all;
  Walk cw;
  cw.b = have ? s_b[warp] : 0;
  cw.len = row_len(rw, s_len, cw.b);
  cw.np = (cw.len + kPage - 1) / kPage;
  cw.rem = have ? min(per, all - p0) : 0;
  cw.u = 0;
  {
    const long long off = have ? s_off[warp] : 0;
    const int wu = cw.np + kUnit;
    cw.u = static_cast<int>(off / wu);
    walk_open(cw, off % wu);
  }

  // ---- producer state: the same walk, NST pages ahead ----
  Walk pw = cw;
  bool more = have;
  int pi = pw.lo;  // next page to issue
  int bt = -1;     // table entries of the next pages, 32 at a time
  int issued = 0;
  auto load_bt = [&](int i) {
    bt = i + lane < pw.hi
             ? __ldcg(block_table + static_cast<size_t>(pw.b) * max_blocks + i + lane)
             : -1;
  };
  const uint32_t ring = sbase + warp * NST * C::STAGE_BYTES;
  const uint32_t exps = sbase + C::EXP_OFF + warp * NST * C::EXP_BYTES;
  const uint32_t bars = sbase + C::BAR_OFF + warp * NST * 8;
  const uint64_t policy = policy_evict_first();
  int bt_i = 0;  // pages taken from bt
  if (more) load_bt(pi);
  // Issues this warp's next page, if there is one, into stage issued % NST.
  auto issue_next = [&]() {
    while (more && pi >= pw.hi) {
      more = walk_next(pw, rw, s_len);
      pi = pw.lo;
      bt_i = 0;
      if (more) load_bt(pi);
    }
    if (!more) return;
    if (bt_i == 32) {
      bt_i = 0;
      load_bt(pi);
    }
    const int phys = __shfl_sync(0xffffffffu, bt, bt_i);
    if (lane == 0) {
      const int st = issued % NST;
      const uint32_t dst = ring + st * C::STAGE_BYTES, bar = bars + st * 8;
      const int kvh = pw.u / n_gb;
      const bool bad = phys < 0 || phys >= num_blocks;
      if (bad) atomicOr(&g_decode_runs_err, ATTN_DEVERR_BAD_PAGE);
      // An out-of-range coordinate is filled with zeros by the copy engine.
      mbar_arrive_expect_tx(bar, C::STAGE_BYTES + C::EXP_BYTES);
      if constexpr (E8) {
        const int slab = bad ? -1 : phys * h_kv + kvh;
        const size_t eo = static_cast<size_t>(bad ? 0 : slab) * kPage;
        tma_load_3d_hint(dst, &tmap_k, bar, 0, 0, slab, policy);
        tma_load_3d_hint(dst + C::PAGE_BYTES, &tmap_v, bar, 0, 0, slab, policy);
        bulk_load16(exps + st * 32, bad ? g_unit_exp : ks + eo, bar);
        bulk_load16(exps + st * 32 + 16, bad ? g_unit_exp : vs + eo, bar);
      } else {
#pragma unroll
        for (int hf = 0; hf < D / 64; ++hf) {
          tma_load_4d_hint(dst + hf * (kPage * 128), &tmap_k, bar, hf * 64, kvh, 0, bad ? -1 : phys,
                           policy);
          tma_load_4d_hint(dst + C::PAGE_BYTES + hf * (kPage * 128), &tmap_v, bar, hf * 64, kvh, 0,
                           bad ? -1 : phys, policy);
        }
      }
    }
    ++issued;
    ++bt_i;
    ++pi;
  };
  for (int i = 0; i < NST; ++i) issue_next();

  // A unit cut at the end of this warp's run stays in registers and is joined
  // with the next warps' parts at the end of the CTA: 1 if it began in this
  // run, 2 if it began before the CTA.
  int own = 0, own_nh = 0;
  size_t own_row = 0;
  float m0 = kNone, m1 = kNone, l0 = 0.f, l1 = 0.f;
  float acc[KS][4];

  // Emits a state (accumulators relative to 2^m, in log2 units): into `slot`
  // of the partial states, or (slot < 0) as the row's final output (8-bit) or
  // its own-keys state (bf16).
  auto emit = [&](long long slot, size_t row0, int nh) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int head = 2 * tq + e;
      if (head >= nh) continue;
      const float L = e ? l1 : l0, M = e ? m1 : m0;
      const size_t row = row0 + head;
      if (!ATTN_GUARD(row < static_cast<size_t>(rw.B) * h, &g_decode_runs_err)) continue;
      if (E8 && slot < 0) {
        const bool empty = L == 0.f;  // every logit -inf
        const float inv = empty ? 0.f : 1.f / L;
#pragma unroll
        for (int k = 0; k < KS; ++k)
          *reinterpret_cast<uint32_t*>(out.o + row * D + 16 * k + 2 * gid) =
              empty ? 0u : pack_bf16x2(acc[k][e] * inv, acc[k][2 + e] * inv);
        if (out.lse != nullptr && gid == 0) out.lse[row] = empty ? -INFINITY : M * kLn2 + logf(L);
        continue;
      }
      const size_t at = slot < 0 ? row : static_cast<size_t>(slot) * 8 + head;
      if (!ATTN_GUARD(slot < 0 || at < static_cast<size_t>(gridDim.x) * 16, &g_decode_runs_err)) continue;
      float* so = (slot < 0 ? out.o_row : out.o_part) + at * D;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        if constexpr (E8) {
          *reinterpret_cast<float2*>(so + 16 * k + 2 * gid) = make_float2(acc[k][e], acc[k][2 + e]);
        } else {
          so[16 * k + gid] = acc[k][e];
          so[16 * k + 8 + gid] = acc[k][2 + e];
        }
      }
      if (gid == 0) {
        (slot < 0 ? out.m_row : out.m_part)[at] = M;
        (slot < 0 ? out.l_row : out.l_part)[at] = L;
      }
    }
  };

  int used = 0;      // stages consumed
  bool dead = false; // a wait gave up: results are void, the error word says so
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

    // State of heads 2tq, 2tq + 1: normaliser share l of this lane's keys
    // relative to 2^m, accumulators relative to 2^r.
    m0 = m1 = kNone;
    l0 = l1 = 0.f;
    float r0 = kNone, r1 = kNone;
#pragma unroll
    for (int i = 0; i < KS; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;

    for (int i = cw.lo; i < cw.hi; ++i) {
      const int st = used % NST;
      if (!dead && !mbar_wait(bars + st * 8, (used / NST) & 1, &g_decode_runs_err)) dead = true;
      dead = __any_sync(0xffffffffu, dead);
      if (dead) break;
      const uint32_t kp = ring + st * C::STAGE_BYTES, vp = kp + C::PAGE_BYTES;
      const int valid = min(kPage, cw.len - i * kPage);
      if (valid < kPage) {
        // Slots past the row's end hold whatever the cache holds there (NaN
        // codes among it); their weights are 0, but 0 * NaN is not.
        constexpr int CPR = C::PAGE_BYTES / (kPage * 16);
        for (int c = lane; c < (kPage - valid) * CPR; c += 32)
          asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(
                           chunk_at<E8, D>(vp, valid + c / CPR, c % CPR)),
                       "r"(0u)
                       : "memory");
        fence_proxy_async_smem();  // before the stage is refilled by the copy engine
        __syncwarp();
      }

      // ---- S^T = K q^T: keys gid and gid + 8, heads 2tq and 2tq + 1 ----
      float sa[4] = {0.f, 0.f, 0.f, 0.f}, sb[4] = {0.f, 0.f, 0.f, 0.f};
      float va = 0.f, vb = 0.f, ka = 1.f, kb = 1.f;
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
            mma_f16((j & 1) ? sb : sa, a0, a1, a2, a3, qb[c * 4 + j][0], qb[c * 4 + j][1]);
          }
        }
        const uint32_t ep = exps + st * 32;
        ka = e4m3::scale_of(lds_u8(ep + gid));
        kb = e4m3::scale_of(lds_u8(ep + gid + 8));
        va = static_cast<float>(static_cast<int>(lds_u8(ep + 16 + gid)) - 127);
        vb = static_cast<float>(static_cast<int>(lds_u8(ep + 24 + gid)) - 127);
      } else {
#pragma unroll
        for (int c = 0; c < KS / 2; ++c) {
          const int ch = (c >> 1) * 8 + 2 * tq + (c & 1);
          const uint4 x = lds128(chunk_at<E8, D>(kp, gid, ch));
          const uint4 y = lds128(chunk_at<E8, D>(kp, gid + 8, ch));
          mma_bf16(sa, x.x, y.x, x.y, y.y, qb[2 * c][0], qb[2 * c][1]);
          mma_bf16(sb, x.z, y.z, x.w, y.w, qb[2 * c + 1][0], qb[2 * c + 1][1]);
        }
      }
      float s0 = (sa[0] + sb[0]) * hc0 * ka, s1 = (sa[1] + sb[1]) * hc1 * ka;
      float s2 = (sa[2] + sb[2]) * hc0 * kb, s3 = (sa[3] + sb[3]) * hc1 * kb;
      if (valid < kPage) {
        if (gid >= valid) s0 = s1 = -INFINITY;
        if (gid + 8 >= valid) s2 = s3 = -INFINITY;
      }
      const float t0 = s0 + va, t1 = s1 + va, t2 = s2 + vb, t3 = s3 + vb;

      // ---- references: they move only when a score passes them by kSlack ----
      // (a NaN never compares, and reaches l and O through its weight)
      bool up = s0 > m0 + kSlack || s2 > m0 + kSlack || s1 > m1 + kSlack || s3 > m1 + kSlack;
      if constexpr (E8)
        up = up || t0 > r0 + (kTop + kSlack) || t2 > r0 + (kTop + kSlack) ||
             t1 > r1 + (kTop + kSlack) || t3 > r1 + (kTop + kSlack);
      if (__any_sync(0xffffffffu, up)) {
        float n0 = fmaxf(s0, s2), n1 = fmaxf(s1, s3), w0 = fmaxf(t0, t2), w1 = fmaxf(t1, t3);
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
          n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, off));
          n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, off));
          if constexpr (E8) {
            w0 = fmaxf(w0, __shfl_xor_sync(0xffffffffu, w0, off));
            w1 = fmaxf(w1, __shfl_xor_sync(0xffffffffu, w1, off));
          }
        }
        n0 = fmaxf(n0, m0);
        n1 = fmaxf(n1, m1);
        const float am0 = ex2_approx(m0 - n0), am1 = ex2_approx(m1 - n1);
        l0 *= am0;
        l1 *= am1;
        m0 = n0;
        m1 = n1;
        float a0 = am0, a1 = am1;
        if constexpr (E8) {
          w0 = fmaxf(w0 - kTop, r0);
          w1 = fmaxf(w1 - kTop, r1);
          a0 = ex2_approx(r0 - w0);
          a1 = ex2_approx(r1 - w1);
          r0 = w0;
          r1 = w1;
        }
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          acc[k][0] *= a0;
          acc[k][1] *= a1;
          acc[k][2] *= a0;
          acc[k][3] *= a1;
        }
      }
      const float p0 = ex2_approx(s0 - m0), p1 = ex2_approx(s1 - m1);
      const float p2 = ex2_approx(s2 - m0), p3 = ex2_approx(s3 - m1);
      l0 += p0 + p2;
      l1 += p1 + p3;
      if constexpr (E8) {
        const uint32_t pb0 = movmatrix_t(pack_f16x2(ex2_approx(t0 - r0), ex2_approx(t1 - r1)));
        const uint32_t pb1 = movmatrix_t(pack_f16x2(ex2_approx(t2 - r0), ex2_approx(t3 - r1)));
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
      if (lane == 0) fence_proxy_async_smem();  // generic reads (and zeroing) before the refill
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
      const float f0 = ex2_approx(r0 - m0), f1 = ex2_approx(r1 - m1);
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
      emit(-1, row0, nh);
    } else if (begins || (warp == 0 && !ends)) {  // the run's last unit
      own = begins ? 1 : 2;
      own_row = row0;
      own_nh = nh;
    } else if (warp == 0) {  // began before the CTA, ends here
      emit(2ll * blockIdx.x, row0, nh);
    } else {  // for the warp that has the unit's first part in this CTA
#pragma unroll
      for (int i = 0; i < C::NREG; ++i) join[(warp * C::NREG + i) * 32 + lane] = acc[i >> 2][i & 3];
      if (gid == 0) {
        ms[warp * 8 + 2 * tq] = m0;
        ms[warp * 8 + 2 * tq + 1] = m1;
        ls[warp * 8 + 2 * tq] = l0;
        ls[warp * 8 + 2 * tq + 1] = l1;
      }
      if (lane == 0) s_kind[warp] = ends ? 2 : 1;
    }
    have = walk_next(cw, rw, s_len);
  }

  // ---- join the units cut between this CTA's warps ----
  __syncthreads();
  if (own != 0) {
    bool ends = false;
    for (int w = warp + 1; w < NW && !ends; ++w) {
      const int kind = s_kind[w];
      if (kind == 0) break;  // (only after a wait that gave up)
      ends = kind == 2;
      const float n0 = ms[w * 8 + 2 * tq], n1 = ms[w * 8 + 2 * tq + 1];
      const float M0 = fmaxf(m0, n0), M1 = fmaxf(m1, n1);
      const float a0 = ex2_approx(m0 - M0), a1 = ex2_approx(m1 - M1);
      const float c0 = ex2_approx(n0 - M0), c1 = ex2_approx(n1 - M1);
      l0 = l0 * a0 + ls[w * 8 + 2 * tq] * c0;
      l1 = l1 * a1 + ls[w * 8 + 2 * tq + 1] * c1;
      m0 = M0;
      m1 = M1;
#pragma unroll
      for (int i = 0; i < C::NREG; ++i)
        acc[i >> 2][i & 3] = acc[i >> 2][i & 3] * ((i & 1) ? a1 : a0) +
                             join[(w * C::NREG + i) * 32 + lane] * ((i & 1) ? c1 : c0);
    }
    emit(own == 2 ? 2ll * blockIdx.x : ends ? -1ll : 2ll * blockIdx.x + 1, own_row, own_nh);
  }
  if (dead) {
    // Bounded chance for the copies in flight to land before the CTA exits.
    for (int j = used; j < issued; ++j)
      (void)mbar_wait(bars + (j % NST) * 8, (j / NST) & 1, &g_decode_runs_err);
  }
}

// Joins the partial states of each (row, head) that a run border cut, and
// writes empty rows. One CTA per (row, head), warps take its partials in turn.
template <int D>
__global__ void __launch_bounds__(128)
    decode_runs_merge_kernel(const float* __restrict__ o_part, const float* __restrict__ m_part,
                         const float* __restrict__ l_part, const long long* __restrict__ plan,
                         int h, int g, int n_gb, int upr, __nv_bfloat16* __restrict__ o,
                         float* __restrict__ lse) {
  constexpr int VEC = D / 32, U = 4, NW = 4;
  __shared__ float sm[NW], sl[NW], so[NW][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = blockIdx.x / h, hq = blockIdx.x % h;
  pdl_wait();
  pdl_trigger();
  const long long per = __ldcg(plan), at = __ldcg(plan + 1 + b);
  const long long wu = __ldcg(plan + 2 + b) - at;  // weight of one unit: its pages + kUnit
  const size_t row = static_cast<size_t>(b) * h + hq;
  if (wu == 0) {
    for (int i = threadIdx.x; i < D / 2; i += 128) reinterpret_cast<uint32_t*>(o + row * D)[i] = 0u;
    if (lse != nullptr && threadIdx.x == 0) lse[row] = -INFINITY;
    return;
  }
  const int u = (hq / g) * n_gb + (hq % g) / 8;
  const long long s = at * upr + u * wu;
  const long long c0 = (s + kUnit) / per;  // CTAs of the unit's first and last page
  const int n = static_cast<int>((s + wu - 1) / per - c0) + 1;
  if (n == 1) return;  // finished by its CTA
  float M = kNone, L = 0.f, acc[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
  for (int base = warp; base < n; base += NW * U) {
    float m[U], l[U], x[U][VEC];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int j = base + i * NW;
      m[i] = kNone;
      l[i] = 0.f;
#pragma unroll
      for (int e = 0; e < VEC; ++e) x[i][e] = 0.f;
      if (j < n) {
        const size_t slot = (2 * (c0 + j) + (j == 0 ? 1 : 0)) * 8 + (hq % g) % 8;
        m[i] = __ldcg(m_part + slot);
        l[i] = __ldcg(l_part + slot);
        const float* src = o_part + slot * D + lane * VEC;
        if constexpr (VEC == 4) {
          const float4 t = __ldcg(reinterpret_cast<const float4*>(src));
          x[i][0] = t.x; x[i][1] = t.y; x[i][2] = t.z; x[i][3] = t.w;
        } else {
          const float2 t = __ldcg(reinterpret_cast<const float2*>(src));
          x[i][0] = t.x; x[i][1] = t.y;
        }
      }
    }
    float Mn = M;
#pragma unroll
    for (int i = 0; i < U; ++i) Mn = fmaxf(Mn, m[i]);
    const float sc = ex2_approx(M - Mn);
    M = Mn;
    L *= sc;
#pragma unroll
    for (int e = 0; e < VEC; ++e) acc[e] *= sc;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const float w = ex2_approx(m[i] - Mn);
      L = fmaf(w, l[i], L);
#pragma unroll
      for (int e = 0; e < VEC; ++e) acc[e] = fmaf(w, x[i][e], acc[e]);
    }
  }
  if (lane == 0) {
    sm[warp] = M;
    sl[warp] = L;
  }
#pragma unroll
  for (int e = 0; e < VEC; ++e) so[warp][lane * VEC + e] = acc[e];
  __syncthreads();
  float Mt = kNone, Lt = 0.f;
#pragma unroll
  for (int w = 0; w < NW; ++w) Mt = fmaxf(Mt, sm[w]);
#pragma unroll
  for (int w = 0; w < NW; ++w) Lt = fmaf(sl[w], ex2_approx(sm[w] - Mt), Lt);
  const bool empty = Lt == 0.f;
  const float inv = empty ? 0.f : 1.f / Lt;
  for (int e = threadIdx.x; e < D; e += 128) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) v = fmaf(so[w][e], ex2_approx(sm[w] - Mt), v);
    o[row * D + e] = __float2bfloat16(empty ? 0.f : v * inv);
  }
  if (lse != nullptr && threadIdx.x == 0) lse[row] = empty ? -INFINITY : Mt * kLn2 + logf(Lt);
}

template <bool E8, int D, int NW, int NST>
cudaError_t launch_cfg(const DecodeRunsArgs& a, int sms, cudaStream_t stream) {
  using C = Cfg<E8, D, NW, NST>;
  CUtensorMap tk, tv;
  CUresult r;
  if constexpr (E8) {
    const uint64_t dims[3] = {uint64_t(D), uint64_t(kPage), uint64_t(a.num_blocks) * a.h_kv};
    const uint64_t strides[2] = {uint64_t(D), uint64_t(kPage) * D};
    const uint32_t box[3] = {uint32_t(D), uint32_t(kPage), 1u};
    const CUtensorMapSwizzle sw = D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
    r = encode_tensor_map(&tk, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(a.k_cache), dims,
                          strides, box, sw);
    if (r == CUDA_SUCCESS)
      r = encode_tensor_map(&tv, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(a.v_cache), dims,
                            strides, box, sw);
  } else {
    const uint64_t dims[4] = {uint64_t(D), uint64_t(a.h_kv), uint64_t(kPage), uint64_t(a.num_blocks)};
    const uint64_t strides[3] = {uint64_t(D) * 2, uint64_t(a.h_kv) * D * 2,
                                 uint64_t(kPage) * a.h_kv * D * 2};
    const uint32_t box[4] = {64u, 1u, uint32_t(kPage), 1u};
    r = encode_tensor_map(&tk, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(a.k_cache), dims,
                          strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
    if (r == CUDA_SUCCESS)
      r = encode_tensor_map(&tv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(a.v_cache),
                            dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
  }
  if (r != CUDA_SUCCESS) return cudaErrorInvalidValue;
  auto kern = decode_runs_kernel<E8, D, NW, NST>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  const int grid = C::CTAS * sms < kRunsMaxCtas ? C::CTAS * sms : kRunsMaxCtas;
  const int g = a.h / a.h_kv, n_gb = (g + 7) / 8;
  const Rows rw{a.seq_lens, a.B, a.max_blocks * kPage, a.h_kv * n_gb};
  const RunOut out{a.plan,  a.o_part, a.m_part, a.l_part, a.o_row,
                   a.m_row, a.l_row,  static_cast<__nv_bfloat16*>(a.o), a.lse};
  return launch_pdl(kern, dim3(grid), dim3(NW * 32), size_t(C::SMEM), stream, tk, tv, a.k_exp, a.v_exp,
                    static_cast<const __nv_bfloat16*>(a.q), a.block_table, rw, a.h, a.h_kv, g,
                    a.max_blocks, a.num_blocks, a.scale * kLog2e, out);
}

cudaError_t sm_count(int* sms) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
  return e;
}

}  // namespace

cudaError_t launch_decode8(const DecodeRunsArgs& a, cudaStream_t stream) {
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  e = a.d_h == 128 ? launch_cfg<true, 128, 8, 2>(a, sms, stream)
                   : launch_cfg<true, 64, 8, 3>(a, sms, stream);
  if (e != cudaSuccess) return e;
  const int g = a.h / a.h_kv, n_gb = (g + 7) / 8;
  auto merge = a.d_h == 128 ? decode_runs_merge_kernel<128> : decode_runs_merge_kernel<64>;
  return launch_pdl(merge, dim3(unsigned(a.B) * a.h), dim3(128), 0, stream,
                    static_cast<const float*>(a.o_part), static_cast<const float*>(a.m_part),
                    static_cast<const float*>(a.l_part), static_cast<const long long*>(a.plan), a.h,
                    g, n_gb, a.h_kv * n_gb, static_cast<__nv_bfloat16*>(a.o), a.lse);
}

cudaError_t launch_decode_runs_bf16(const DecodeRunsArgs& a, cudaStream_t stream) {
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  return a.d_h == 128 ? launch_cfg<false, 128, 8, 3>(a, sms, stream)
                      : launch_cfg<false, 64, 8, 4>(a, sms, stream);
}

unsigned int decode_runs_read_and_clear_error(cudaStream_t stream, cudaError_t* st) {
  unsigned int v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(&v, g_decode_runs_err, sizeof(v), 0,
                                            cudaMemcpyDeviceToHost, stream);
  if (e == cudaSuccess)
    e = cudaMemcpyToSymbolAsync(g_decode_runs_err, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice,
                                stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
  if (st) *st = e;
  return v;
}

}  // namespace attn
