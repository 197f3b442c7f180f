// decode_tree.cu -- attn_decode_paged_tree: paged attention of each row's drafted
// tokens, which form a tree.
//
// Row b has n drafted tokens at the last n of its len positions; every one of them
// sees the ctx = len - n keys in front of them, and of the drafts those whose bits
// its mask sets. The online recurrence of "Naive attention and the online softmax"
// in base 2, its states joined where a row's keys are cut ("Merge normalized
// attention without averaging tile outputs").
//
// The n * g query rows (token, head of the group) of a KV head share its keys, so
// they are the rows of dense products against tiles of 128 keys: up to n g of about
// 256 the keys' bytes bound the time (2 * 128 * d_h * 2 bytes a tile and head at
// 1 / 152 of the memory rate are about 1.5 us, the two products with two 128-row
// tiles and the two-term P less), and a key is read once for all of them.
//
// A unit is (row, KV head, block of up to two 128-row tiles) and its key tiles. A
// CTA has two softmax warpgroups ("streams"; thread = query row), warps that load Q,
// K and V, and an MMA warp. Where the unit has two row tiles the streams have one each
// and share every key tile; where it has one, the streams take its key tiles in turn,
// each with an accumulator of its own, and join the two at the end, half of the
// dimensions each (either reads both accumulators from tensor memory: the same lanes).
// Steps alternate between the streams; per step S = Q K^T (SS), weights over S in
// tensor memory, O += P V (TS), with S of step e + 2 issued behind P V of step e. Q has
// two slots, so that a unit's queries, like its first keys, land while the one in
// front is still at work.
//
// V stays bf16 and P is the two-term bf16 split P_hi + P_lo, so q, K and V enter as
// they are, whatever their magnitudes.
//
// Work split: the units of all rows, laid end to end with a weight of their key tiles
// + kTreeUnit, are cut into equal runs, one per CTA, so any mix of lengths and of
// drafts fills the machine and the launch depends on neither. A unit inside a run is
// finished by its CTA; one that a border cuts leaves a partial state per CTA, at most
// two in a CTA (one that began before it, one that goes on behind it), which
// tree_merge_kernel joins in run order.
//
// Masked drafts never reach a row: their scores are set to -inf, and since 0 * NaN
// is not 0, non-finite numbers among the drafts' values are taken out of the V tile
// and put back as NaN, at the end, in the rows that see them. Only tiles that hold
// drafts are looked at for that, and for slots past the row's end.
//
// Measured (GB300): 64 rows of up to 16384 keys and 24 drafts, 32 query heads over 8
// of 128: 341 to 370 us, GPU to GPU, the keys' bytes at 0.95 to 0.87 of the copy rate. One
// row of 32768 keys and 26 drafts: 36 us, 20 of them the bytes; the others are the
// launch, the CTA's set-up, the first keys' way and the merge. 24 rows of up to 8192 keys,
// 61 drafts, 8 heads over one of 64 (two row tiles each): 27 to 33 us, GPU to GPU, where
// the two streams' chain S, weights, P V takes 2.1 us a key tile. One row of 500 keys and
// 8 drafts: 11 us, latency. (Figures beside a choice below compare two forms on
// one GPU, at the state of the kernel when it was made.)
#include "decode_runs.cuh"
#include "pdl.cuh"
#include "tc.cuh"

namespace attn {

static __device__ unsigned int g_tree_err;
#ifdef ATTN_DEBUG
// The key tile, in each CTA's own order, and which of its loads is not requested
// (attn_selftest_tree_stall): 0 K, 1 V.
static __device__ int g_tree_stall[2] = {-1, 0};
#endif

namespace {

constexpr int kBM = 128, kBN = 128;
// A unit's weight beside its key tiles: query, states, output. (64 rows of up to 16384
// keys: 341 us with 2 to 4, 343 with 6; 24 rows, two row tiles: 32 with 2 and 3, 34 with
// 4 and 6.)
constexpr int kTreeUnit = 3;
// A row's reference moves, to the largest score so far, when one passes it by more
// than this (log2 units).
constexpr float kRise = 8.0f;

// A row: drafts, keys, first query token, key tiles, row blocks (0: no work).
struct TreeRow {
  int n, len, tok0, nt, n_rb;
};
// Where the CTA's run starts, a run's weight, and the warps' sums of the rows' weights.
struct TreePlan {
  long long sum[12];
  long long off, per;
  int b;
  TreeRow row;
};
// A unit's key tiles [t0, t0 + nt) in a CTA's run.
struct TreeSeg {
  int b, kvh;         // row, KV head
  int n, len, tok0;   // the row's drafts, keys and first query token
  int first;          // first draft of the unit's query rows
  int t0, nt, left;   // left: key tiles of the unit behind these; nt 0: the run has ended
  int begins;         // the unit's first tile is among them
  int two;            // more drafts than one 128-row tile holds
};

template <int D>
struct TrCfg {
  static constexpr int SUBS = D / 64;
  static constexpr int SUB_BYTES = 128 * 128;
  static constexpr int TILE = kBN * D * 2;
  static constexpr int NSK = D == 128 ? 2 : 4, NSV = D == 128 ? 3 : 4;
  static constexpr int Q_OFF = 0;
  static constexpr int K_OFF = Q_OFF + 2 * TILE;
  static constexpr int V_OFF = K_OFF + NSK * TILE;
  static constexpr int ML_OFF = V_OFF + NSV * TILE;  // (reference, sum) [stream][row]
  // q_full[2], q_empty[2], seg_full[2], seg_empty[2], k_full[], k_empty[], v_full[],
  // v_empty[], s_full[2], p_full[2], o_final[2], ml_full, ml_empty, mma_done
  static constexpr int B_QF = 0, B_QE = 2, B_GF = 4, B_GE = 6, B_KF = 8, B_KE = B_KF + NSK,
                       B_VF = B_KE + NSK, B_VE = B_VF + NSV, B_SF = B_VE + NSV, B_PF = B_SF + 2,
                       B_OF = B_PF + 2, B_MF = B_OF + 2, B_ME = B_MF + 1, B_DONE = B_ME + 1,
                       NBAR = B_DONE + 1;
  static_assert(NBAR <= 384, "a thread initialises each barrier");
  static constexpr int BAR_OFF = ML_OFF + 2 * kBM * 8;
  static constexpr int MISC_OFF = BAR_OFF + NBAR * 8;  // tensor-memory slot, abort flag, poison[2]
  static constexpr int PLAN_OFF = (MISC_OFF + 16 + 15) / 16 * 16;
  static constexpr int SEG_OFF = PLAN_OFF + (sizeof(TreePlan) + 15) / 16 * 16;  // two segments
  static constexpr int SMEM = SEG_OFF + 2 * sizeof(TreeSeg);
  static_assert(SMEM <= 227 * 1024, "shared memory of an SM");
  static constexpr int THREADS = 384;
  static constexpr int K_WARP = 8, MMA_WARP = 9, V_WARP = 10, Q_WARP = 11;
  static constexpr int REG_LAUNCH = 168, REG_CONTROL = 120, REG_SOFTMAX = 192;
  static_assert(2 * 128 * REG_SOFTMAX + 128 * REG_CONTROL <= THREADS * REG_LAUNCH,
                "register split exceeds the launch allocation");
};

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// Packed fp32 pairs.
__device__ __forceinline__ uint64_t f2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unf2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Bounded wait that also gives up at once when another role has aborted.
__device__ __forceinline__ bool wait_or_abort(uint32_t bar, uint32_t parity,
                                              volatile int* abort_flag) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if (globaltimer_ns() - t0 > ATTN_WAIT_LIMIT_NS) {
      atomicOr(&g_tree_err, ATTN_DEVERR_WAIT_TIMEOUT);
      *abort_flag = 1;
      return false;
    }
  }
}

struct TreeRows {
  const int32_t* block_table;
  const int32_t* cu_q;
  const int32_t* seq_lens;
  const int32_t* mask;  // [total_q, words]
  int B, total_q, max_q_len, words, h, h_kv, g, max_blocks, num_blocks;
  int tpt;  // tokens per 128-row tile: 128 / g
};

struct TreeRaw {  // a row's offsets and length as they are
  int begin, end, len;
};
__device__ __forceinline__ TreeRaw tree_raw(const TreeRows& a, int b) {
  return TreeRaw{__ldcg(a.cu_q + b), __ldcg(a.cu_q + b + 1), __ldcg(a.seq_lens + b)};
}
__device__ __forceinline__ TreeRow tree_row(const TreeRows& a, const TreeRaw& raw, bool report) {
  TreeRow r;
  r.tok0 = raw.begin;
  const int end = raw.end;
  r.len = raw.len;
  const int cap = a.max_blocks * kPage;
  const long long n = static_cast<long long>(end) - r.tok0;
  if (r.tok0 < 0 || end > a.total_q || n < 0 || n > a.max_q_len || n > cap) {
    if (report) atomicOr(&g_tree_err, ATTN_DEVERR_BAD_SEQ_LEN);
    r.n = r.len = r.nt = r.n_rb = 0;
    return r;
  }
  r.n = static_cast<int>(n);
  if (r.n > 0 && (r.len < r.n || r.len > cap)) {
    if (report) atomicOr(&g_tree_err, ATTN_DEVERR_BAD_SEQ_LEN);
    r.len = r.len < r.n ? r.n : cap;
  }
  r.nt = (r.len + kBN - 1) / kBN;
  r.n_rb = (r.n + 2 * a.tpt - 1) / (2 * a.tpt);
  return r;
}
__device__ __forceinline__ long long tree_weight(const TreeRows& a, const TreeRow& r) {
  return static_cast<long long>(r.n_rb) * a.h_kv * (r.nt + kTreeUnit);
}

// A CTA's run.
struct TreeWalk {
  long long rem, off;  // weight of the run left; the run's start within the unit
  int b, u;            // row, unit within it
  TreeRow r;
  TreeRaw ahead;       // row b + 1
  TreeRaw held;        // few rows (B <= 32): that of row `lane`
  __device__ __forceinline__ void look_ahead(const TreeRows& a) {
    if (a.B <= 32)
      ahead = TreeRaw{__shfl_sync(0xffffffffu, held.begin, b + 1), __shfl_sync(0xffffffffu, held.end, b + 1),
                      __shfl_sync(0xffffffffu, held.len, b + 1)};
    else
      ahead = b + 1 < a.B ? tree_raw(a, b + 1) : TreeRaw{0, 0, 0};
  }
  __device__ __forceinline__ bool next(const TreeRows& a, TreeSeg& s) {
    while (rem > 0) {
      while (u >= r.n_rb * a.h_kv) {
        if (++b >= a.B) return false;
        r = tree_row(a, ahead, false);
        u = 0;
        look_ahead(a);
      }
      const long long take = min(r.nt + kTreeUnit - off, rem);
      s.t0 = static_cast<int>(max(off - kTreeUnit, 0ll));
      const int hi = static_cast<int>(max(off + take - kTreeUnit, 0ll));
      s.nt = hi - s.t0;
      s.left = r.nt - hi;
      s.b = b;
      s.kvh = u / r.n_rb;
      s.n = r.n;
      s.len = r.len;
      s.tok0 = r.tok0;
      s.first = (u % r.n_rb) * 2 * a.tpt;
      s.begins = s.t0 == 0;
      s.two = r.n - s.first > a.tpt;
      rem -= take;
      off = 0;
      ++u;
      if (s.nt > 0) return true;
    }
    return false;
  }
};

// What the merge reads of the unit that begins in a CTA and goes on behind it.
struct TreeCut {
  int parts, tok, n_tok, kvh;  // parts 0: none
};
struct TreeOut {
  TreeCut* cut;  // [CTAs]
  // Partial states, slot 2 c: the unit that began before CTA c, 2 c + 1: the one that
  // goes on behind it. Accumulators [slot][tile 2][d_h / 4][128 rows][4] (a warp
  // stores 512 contiguous bytes), m (log2 units) and l [slot][tile][128].
  float *o_part, *m_part, *l_part;
  __nv_bfloat16* o;
  float* lse;
};

// Which keys the query row with mask words `mask` sees, 32 from key ctx + 32 w on, one
// bit each: all of them in front of the drafts (w < 0), draft t where bit t is set
// (t < n).
__device__ __forceinline__ uint32_t tree_word(const int32_t* mask, int n, int w) {
  if (w < 0) return 0xffffffffu;
  if (w * 32 >= n) return 0u;
  const uint32_t x = static_cast<uint32_t>(__ldcg(mask + w));
  return n - w * 32 >= 32 ? x : x & ((1u << (n - w * 32)) - 1u);
}

// Chunk c of 16 bytes of key `row` of the V tile at `base`.
__device__ __forceinline__ uint32_t v_chunk(uint32_t base, int row, int c) {
  // (any order will do: eight neighbouring rows read distinct banks)
  return base + (c >> 3) * (128 * 128) + row * 128 + (((c ^ row) & 7) << 4);
}
// Non-finite numbers of a V tile's key become zeros. Rare.
template <int D>
__device__ __noinline__ void drop_nonfinite(uint32_t base, int row) {
#pragma unroll 1
  for (int c = 0; c < D / 8; ++c) {
    const uint32_t at = v_chunk(base, row, c);
    const uint4 x = lds128(at);
    uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if ((w[k] & 0x7f80u) == 0x7f80u) w[k] &= 0xffff0000u;
      if ((w[k] & 0x7f800000u) == 0x7f800000u) w[k] &= 0xffffu;
    }
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3])
                 : "memory");
  }
}
// The tile's V, in shared memory at `base`, before a P V that gives some of its keys
// weight 0: key `row` of the tile. Keys from `lim` on become zeros. Non-finite numbers
// of keys from `draft` on become zeros too; returns whether there were any. (Chunk by
// chunk with a branch each this took 3 us, at every unit's end.)
template <int D>
__device__ __forceinline__ bool clean_v(uint32_t base, int row, int draft, int lim) {
  if (row >= lim) {
#pragma unroll
    for (int c = 0; c < D / 8; ++c)
      asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(v_chunk(base, row, c)), "r"(0u) : "memory");
    return false;
  }
  if (row < draft) return false;
  uint32_t most = 0u;  // largest exponent fields, of either half
#pragma unroll
  for (int c = 0; c < D / 8; ++c) {
    const uint4 x = lds128(v_chunk(base, row, c));
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) asm("max.u16x2 %0, %0, %1;" : "+r"(most) : "r"(w[k] & 0x7f807f80u));
  }
  if ((most & 0xffffu) != 0x7f80u && (most >> 16) != 0x7f80u) return false;
  drop_nonfinite<D>(base, row);
  return true;
}

// Which dims are non-finite in the value of a draft that the row sees, among keys
// k0 .. k1 - 1 (one bit each). Rare: the values are read again from the cache.
template <int D>
__device__ __noinline__ uint4 poisoned_dims(const __nv_bfloat16* vc, const TreeRows& a, int b, int kvh,
                                            const int32_t* mask, int n, int ctx, int k0, int k1) {
  uint32_t out[4] = {0u, 0u, 0u, 0u};
#pragma unroll 1
  for (int j = max(k0, ctx); j < k1; ++j) {
    if (!((tree_word(mask, n, (j - ctx) >> 5) >> ((j - ctx) & 31)) & 1u)) continue;
    const int phys = __ldcg(a.block_table + static_cast<size_t>(b) * a.max_blocks + j / kPage);
    if (phys < 0 || phys >= a.num_blocks) continue;
    const uint4* v = reinterpret_cast<const uint4*>(
        vc + ((static_cast<size_t>(phys) * kPage + j % kPage) * a.h_kv + kvh) * D);
#pragma unroll
    for (int c = 0; c < D / 8; ++c) {
      const uint4 x = __ldcg(v + c);
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if ((w[k] & 0x7f80u) == 0x7f80u) out[c >> 2] |= 1u << ((c & 3) * 8 + 2 * k);
        if ((w[k] & 0x7f800000u) == 0x7f800000u) out[c >> 2] |= 2u << ((c & 3) * 8 + 2 * k);
      }
    }
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}

// Inclusive sums over the warp.
__device__ __forceinline__ long long warp_sums(long long x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

template <int D>
__global__ void __launch_bounds__(384, 1)
    tree_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                const __grid_constant__ CUtensorMap tmap_v, const __nv_bfloat16* __restrict__ v_cache,
                const TreeRows a, const TreeOut out, float scale_log2) {
  using C = TrCfg<D>;
  // Aligned by its declaration (there is no room for slack, nor anything static in
  // front of it).
  extern __shared__ __align__(1024) uint8_t smem[];
  TreePlan& plan = *reinterpret_cast<TreePlan*>(smem + C::PLAN_OFF);
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) { return sbase + C::BAR_OFF + 8 * i; };
  float2* ml = reinterpret_cast<float2*>(smem + C::ML_OFF);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::MISC_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::MISC_OFF + 4);
  // Segment (counted from 1) whose V had non-finite drafts, by its count's parity.
  volatile int* poison = reinterpret_cast<volatile int*>(smem + C::MISC_OFF + 8);
  // Segment i of the run lies in slot i & 1: the Q warp walks the run and leaves what
  // the other warps need, which keeps the walk out of their registers (what they spill
  // does not stay in the 28 KB of L1 that the tiles leave).
  TreeSeg* segs = reinterpret_cast<TreeSeg*>(smem + C::SEG_OFF);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x;

  ATTN_DCHECK((sbase & 1023u) == 0u, &g_tree_err);
  if (tid == 0) {
    prefetch_tmap(&tmap_q);
    prefetch_tmap(&tmap_k);
    prefetch_tmap(&tmap_v);
    *abort_flag = 0;
    poison[0] = poison[1] = 0;
  }
  if (tid < C::NBAR) {
    const bool both = tid == C::B_MF || tid == C::B_ME, p = tid >= C::B_PF && tid < C::B_PF + 2;
    const bool seg = tid >= C::B_GE && tid < C::B_GE + 2;  // eleven warps read a segment
    mbar_init(bar(tid), both ? 256u : p ? 128u : seg ? 11u : 1u);
    fence_barrier_init();
  }
  if (warp == C::MMA_WARP) tc::alloc(smem_u32(tmem_slot), 512);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();  // q, lengths, tables, masks and pages are earlier kernels' output

  // ---- the runs: prefix sums of the rows' weights. Of at most 32 rows the Q warp, which
  // alone walks them, has one a lane and plans for itself (one row of 500 keys 11.8 -> 11.1
  // us, 24 rows 34.1 -> 32.8) ----
  long long per = 0, all = 0;  // the weight of a run and of all
  if (a.B > 32) {
    const int per_t = (a.B + C::THREADS - 1) / C::THREADS;
    const int b0 = min(tid * per_t, a.B), b1 = min(b0 + per_t, a.B);
    long long sum = 0;
    TreeRow mine{0, 0, 0, 0, 0};
    for (int b = b0; b < b1; ++b) {
      mine = tree_row(a, tree_raw(a, b), cta == 0);
      sum += tree_weight(a, mine);
    }
    const long long incl = warp_sums(sum, lane);
    if (lane == 31) plan.sum[warp] = incl;
    __syncthreads();
    long long at = incl - sum;
#pragma unroll
    for (int w = 0; w < 12; ++w) {
      if (w < warp) at += plan.sum[w];
      all += plan.sum[w];
    }
    per = max(1ll, div_ll(all + gridDim.x - 1, gridDim.x));
    const long long p0 = per * cta;
    if (p0 >= at && p0 < at + sum) {
      for (int b = b0; b < b1; ++b) {
        if (per_t > 1) mine = tree_row(a, tree_raw(a, b), false);
        const long long w = tree_weight(a, mine);
        if (p0 >= at && p0 < at + w) {
          plan.b = b;
          plan.off = p0 - at;
          plan.row = mine;
        }
        at += w;
      }
    }
    __syncthreads();
  }
  // Steps e = 0, 1, ... of a segment alternate between the streams (stream e & 1), which
  // share its key tiles, or have them in turn.
  auto n_of = [](int nt, bool two, int t) { return two ? nt : (nt + 1 - t) >> 1; };
  // Key tile of 8 pages into dst: lane i < 8 * SUBS issues the box of page i % 8,
  // half i / 8. Whole warp.
  auto load_tile = [&](uint32_t dst, const CUtensorMap* map, uint32_t b, int kvh, int ent, int sel,
                       int page0, int n_pages) {
    int phys = __shfl_sync(0xffffffffu, ent, sel + (lane & 7));
    if (phys < 0 || phys >= a.num_blocks) {
      if (page0 + (lane & 7) < n_pages) atomicOr(&g_tree_err, ATTN_DEVERR_BAD_PAGE);
      phys = -1;
    }
    if (lane == 0) mbar_arrive_expect_tx(b, C::TILE);
    __syncwarp();
    if (lane < 8 * C::SUBS)
      tma_load_4d(dst + (lane >> 3) * C::SUB_BYTES + (lane & 7) * kPage * 128, map, b, (lane >> 3) * 64,
                  kvh, 0, phys);
    __syncwarp();
  };
  auto warp_wait = [&](uint32_t b, uint32_t parity) {
    return __all_sync(0xffffffffu, wait_or_abort(b, parity, abort_flag));
  };
  // Segment i, or false: none is left, or an abort. Once a warp has read what it needs
  // it lets go of it. Whole warp.
  auto open = [&](int i) {
    return warp_wait(bar(C::B_GF + (i & 1)), (i >> 1) & 1) && segs[i & 1].nt > 0;
  };
  auto close = [&](int i) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(C::B_GE + (i & 1)));
  };

  if (warp >= C::K_WARP) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REG_CONTROL));
    if (warp == C::K_WARP || warp == C::V_WARP) {
      // --------------------------------------------------------- producers
      const bool is_k = warp == C::K_WARP;
      const int ns = is_k ? C::NSK : C::NSV, full = is_k ? C::B_KF : C::B_VF,
                empty = is_k ? C::B_KE : C::B_VE;
      const uint32_t ring = sbase + (is_k ? C::K_OFF : C::V_OFF);
      const CUtensorMap* map = is_k ? &tmap_k : &tmap_v;
      int g = 0;
      bool ok = true;
#ifdef ATTN_DEBUG
      const int stall = g_tree_stall[1] == (is_k ? 0 : 1) ? g_tree_stall[0] : -1;
#else
      constexpr int stall = -1;
#endif
      for (int it = 0; ok && open(it); ++it) {
        const TreeSeg s = segs[it & 1];
        close(it);
        const int n_pages = (s.len + kPage - 1) / kPage;
        const int32_t* table = a.block_table + static_cast<size_t>(s.b) * a.max_blocks;
        // Table entries of the 32 pages from `page` on, one per lane.
        auto entries = [&](int page) { return page + lane < n_pages ? __ldcg(table + page + lane) : -1; };
        int ent = entries(s.t0 * 8), next = -1;
        for (int j = 0; j < s.nt; ++j, ++g) {
          const int st = g % ns, page0 = (s.t0 + j) * 8;
          if ((j & 3) == 0) {  // entries four tiles at a time, fetched four tiles ahead
            if (j > 0) ent = next;
            next = entries(page0 + 32);
          }
          if (g >= ns && !warp_wait(bar(empty + st), (g / ns - 1) & 1)) {
            ok = false;
            break;
          }
          if (g != stall)
            load_tile(ring + st * C::TILE, map, bar(full + st), s.kvh, ent, (j & 3) * 8, page0, n_pages);
        }
      }
      if (*abort_flag) {
        // Drain: the newest load of each stage is the only one that can still be in
        // flight. Bounded waits, error already recorded.
        for (int i = max(0, g - ns); i < g; ++i)
          if (i != stall) (void)mbar_wait(bar(full + i % ns), (i / ns) & 1, &g_tree_err);
      }
    } else if (warp == C::Q_WARP) {
      // The run's segments, and query tile q (counted over them) in slot q & 1.
      TreeWalk walk;
      walk.off = 0;
      walk.b = walk.u = 0;
      walk.r = TreeRow{0, 0, 0, 0, 0};
      walk.ahead = walk.held = TreeRaw{0, 0, 0};
      if (lane == 0) out.cut[cta].parts = 0;
      long long off = 0;  // the run's start within its first row
      if (a.B <= 32) {
        if (lane < a.B) walk.held = tree_raw(a, lane);
        TreeRow mine{0, 0, 0, 0, 0};
        if (lane < a.B) mine = tree_row(a, walk.held, cta == 0);
        const long long w = tree_weight(a, mine), incl = warp_sums(w, lane);
        all = __shfl_sync(0xffffffffu, incl, 31);
        per = max(1ll, div_ll(all + gridDim.x - 1, gridDim.x));
        const long long p0 = per * cta;
        if (p0 >= incl - w && p0 < incl) {
          plan.b = lane;
          plan.off = p0 - (incl - w);
          plan.row = mine;
        }
        __syncwarp();
      }
      if (per * cta < all) {
        walk.b = plan.b;
        walk.r = plan.row;
        off = plan.off;
      }
      if (lane == 0) plan.per = per;
      walk.rem = per * cta < all ? min(per, all - per * cta) : 0;
      if (walk.rem > 0) {
        walk.look_ahead(a);
        const long long wu = walk.r.nt + kTreeUnit;
        walk.u = static_cast<int>(div_ll(off, wu));
        walk.off = off - walk.u * wu;
      }
      int q = 0;
      bool ok = true;
      for (int it = 0; ok; ++it) {
        TreeSeg s;
        if (!walk.next(a, s)) s.nt = 0;
        if (it >= 2 && !warp_wait(bar(C::B_GE + (it & 1)), ((it >> 1) - 1) & 1)) break;
        if (lane == 0) {
          segs[it & 1] = s;
          mbar_arrive(bar(C::B_GF + (it & 1)));
        }
        __syncwarp();
        if (s.nt == 0) break;
        const int tiles = s.two ? 2 : 1;
        for (int i = 0; i < tiles; ++i, ++q) {
          const int slot = q & 1;
          if (q >= 2 && !warp_wait(bar(C::B_QE + slot), ((q >> 1) - 1) & 1)) {
            ok = false;
            break;
          }
          if (lane == 0) mbar_arrive_expect_tx(bar(C::B_QF + slot), C::SUBS * 128 * a.g * a.tpt);
          __syncwarp();
          if (lane < C::SUBS)
            tma_load_4d(sbase + C::Q_OFF + slot * C::TILE + lane * C::SUB_BYTES, &tmap_q, bar(C::B_QF + slot),
                        lane * 64, 0, s.kvh, s.tok0 + s.first + i * a.tpt);
          __syncwarp();
        }
      }
      if (*abort_flag)
        for (int i = max(0, q - 2); i < q; ++i)
          (void)mbar_wait(bar(C::B_QF + (i & 1)), (i >> 1) & 1, &g_tree_err);
    } else if (warp == C::MMA_WARP) {
      // -------------------------------------------------------- MMA issuer
      constexpr uint32_t idS = tc::idesc_bf16_f32(kBM, kBN, false, false);
      constexpr uint32_t idO = tc::idesc_bf16_f32(kBM, D, false, true);
      const uint64_t dq0 = tc::sw128_desc(sbase + C::Q_OFF, 16, 1024);
      const uint64_t dk0 = tc::sw128_desc(sbase + C::K_OFF, 16, 1024);
      const uint64_t dv0 = tc::sw128_desc(sbase + C::V_OFF, C::SUB_BYTES, 1024);
      bool ok = true;
      int g0 = 0, q = 0, base[2] = {0, 0};
      for (int it = 0; ok && open(it); ++it) {
        const bool two = segs[it & 1].two;
        const int nt = segs[it & 1].nt, n = two ? 2 * nt : nt;
        close(it);
        ok = warp_wait(bar(C::B_QF + (q & 1)), (q >> 1) & 1) &&
             (!two || warp_wait(bar(C::B_QF + ((q + 1) & 1)), ((q + 1) >> 1) & 1));
        // S of step e once its K tile is there, then what it frees.
        auto s_step = [&](int e) {
          const int t = e & 1, g = g0 + (two ? e >> 1 : e), st = g % C::NSK;
          if (!warp_wait(bar(C::B_KF + st), (g / C::NSK) & 1)) return false;
          tc::fence_after();
          const int slot = (q + (two ? t : 0)) & 1;
          const uint64_t da = dq0 + uint64_t((slot * C::TILE) >> 4);
          const uint64_t db = dk0 + uint64_t((st * C::TILE) >> 4);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off16 = ((kk >> 2) * C::SUB_BYTES + (kk & 3) * 32) >> 4;
            tc::mma_ss_elect(tmem + t * 256, da + off16, db + off16, idS, kk > 0 ? 1u : 0u);
          }
          tc::commit_elect(bar(C::B_SF + t));
          if (!two || t == 1) tc::commit_elect(bar(C::B_KE + st));
          if (e == n - 1 || (two && e == n - 2)) tc::commit_elect(bar(C::B_QE + slot));  // its last reader
          return true;
        };
        for (int e = -2; ok && e < n; ++e) {
          if (e >= 0) {
            const int t = e & 1, g = g0 + (two ? e >> 1 : e), sv = g % C::NSV;
            ok = warp_wait(bar(C::B_PF + t), (base[t] + (e >> 1)) & 1) &&
                 warp_wait(bar(C::B_VF + sv), (g / C::NSV) & 1);
            if (!ok) break;
            tc::fence_after();
            const uint64_t db = dv0 + uint64_t((sv * C::TILE) >> 4);
            const uint32_t dO = tmem + t * 256 + 128, aP = tmem + t * 256;
#pragma unroll
            for (int kk = 0; kk < kBN / 16; ++kk) {
              const uint64_t b = db + uint64_t((kk * 16 * 128) >> 4);
              tc::mma_ts_elect(dO, aP + kk * 8, b, idO, (e >= 2 || kk > 0) ? 1u : 0u);
              tc::mma_ts_elect(dO, aP + 64 + kk * 8, b, idO, 1u);
            }
            if (!two || t == 1) tc::commit_elect(bar(C::B_VE + sv));
            if (e + 2 >= n) tc::commit_elect(bar(C::B_OF + t));  // the stream's last step
          }
          if (e + 2 < n) ok = s_step(e + 2);
        }
        g0 += nt;
        q += two ? 2 : 1;
        base[0] += n_of(nt, two, 0);
        base[1] += n_of(nt, two, 1);
      }
      tc::commit_elect(bar(C::B_DONE));
      (void)__all_sync(0xffffffffu, mbar_wait(bar(C::B_DONE), 0, &g_tree_err));
    }
  } else {
    // ------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REG_SOFTMAX));
    const int t = warp >> 2, wq = warp & 3, r = wq * 32 + lane;
    const uint32_t tS = tmem + (uint32_t(wq * 32) << 16) + t * 256, tO = tS + 128;
    const int row_tok = r / a.g, hh = r % a.g;  // token of the tile, head of the group
    int g0 = 0, cnt = 0, fin[2] = {0, 0}, handed = 0;
    bool ok = true;
    for (int it = 0; ok && open(it); ++it) {
      const TreeSeg& s = segs[it & 1];
      const bool two = s.two;
      const int n = n_of(s.nt, two, t), n1 = n_of(s.nt, two, 1);
      const int ctx = s.len - s.n;
      // This thread's query row: draft `tok` of the row.
      const int tok = s.first + (two ? t * a.tpt : 0) + row_tok;
      const bool valid = row_tok < a.tpt && tok < s.n;
      const bool busy = __any_sync(0xffffffffu, valid);
      const int32_t* mask = a.mask + static_cast<size_t>(s.tok0 + (valid ? tok : 0)) * a.words;
      float ref = kNone, l = 0.f;
      // The accumulators and ml are the other stream's to read until it says so.
      if (handed > 0 &&
          !__all_sync(0xffffffffu, wait_or_abort(bar(C::B_ME), (handed - 1) & 1, abort_flag)))
        break;
      // The words that hold an edge tile's bits are asked for a step ahead: a load takes
      // 2 us beside the pages' traffic.
      uint32_t words[5];
      auto fetch_words = [&](int i) {
        const int key = (s.t0 + (two ? i : 2 * i + t)) * kBN;
        if (i < n && key + kBN > ctx) {
#pragma unroll
          for (int k = 0; k < 5; ++k) words[k] = tree_word(mask, s.n, ((key - ctx) >> 5) + k);
        }
      };
      fetch_words(0);
      for (int i = 0; i < n; ++i, ++cnt) {
        const int j = two ? i : 2 * i + t;  // key tile within the segment
        const int k0 = (s.t0 + j) * kBN;
        const bool edge = k0 + kBN > ctx;  // drafts, and perhaps slots past the row's end
        if (!warp_wait(bar(C::B_SF + t), cnt & 1)) {
          ok = false;
          break;
        }
        if (busy) {
          tc::fence_after();
          uint32_t sr[4][32];
#pragma unroll
          for (int c = 0; c < 4; ++c) tc::ld32(tS + c * 32, sr[c]);
          tc::wait_ld();
          if (edge) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const uint32_t bits = __funnelshift_r(words[c], words[c + 1], (k0 - ctx) & 31);
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (!((bits >> k) & 1u)) sr[c][k] = __float_as_uint(-INFINITY);
            }
          }
          float cm[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            auto x = [&](int k) { return __uint_as_float(sr[c][k]); };
            float m8[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) m8[k] = max3(x(4 * k), x(4 * k + 1), fmaxf(x(4 * k + 2), x(4 * k + 3)));
            cm[c] = fmaxf(max3(max3(m8[0], m8[1], m8[2]), max3(m8[3], m8[4], m8[5]), m8[6]), m8[7]);
          }
          const float cand = __fmul_rn(fmaxf(max3(cm[0], cm[1], cm[2]), cm[3]), scale_log2);
          float alpha = 1.f;
          if (cand - ref > kRise) {
            alpha = ex2_approx(ref - cand);
            l *= alpha;
            ref = cand;
          }
          const bool rescale = i > 0 && __any_sync(0xffffffffu, alpha != 1.f);
          // Scores enter as rounded products minus the reference, which is exact near it
          // at any magnitude of the logits: with the product's residual left in, up to half
          // a step of the logit, the largest weight passed fp32 from logits of 2^30 on. (So
          // the products are not packed: a packed product and sum are joined to one fma
          // whatever their rounding modifiers; 24 rows of two row tiles took 30.0 us so, and
          // 31.4 now, the other cases 1 % more at most. The exact form out of line, for
          // large references alone: 64 rows 370 us instead of 346.) P_hi is p's upper 16
          // bits, P_lo = bf16(p - P_hi); keys 2k, 2k + 1 of half h in columns 32 h + k,
          // 64 + 32 h + k.
          const uint64_t n2 = f2(-ref, -ref);
          uint64_t sumA = f2(0.f, 0.f), sumB = f2(0.f, 0.f);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t hi[32], lo[32];
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              const int key = 64 * half + 2 * k;
              float y0, y1;
              unf2(add2(f2(__fmul_rn(__uint_as_float(sr[key >> 5][key & 31]), scale_log2),
                           __fmul_rn(__uint_as_float(sr[key >> 5][(key & 31) + 1]), scale_log2)),
                        n2),
                   y0, y1);
              const float q0 = ex2_approx(y0), q1 = ex2_approx(y1);
              if (k & 1) sumB = add2(sumB, f2(q0, q1)); else sumA = add2(sumA, f2(q0, q1));
              hi[k] = split_hi(q0, q1);
              lo[k] = split_lo(q0, q1);
            }
            tc::st32(tS + 32 * half, hi);
            tc::st32(tS + 64 + 32 * half, lo);
          }
          float s0, s1;
          unf2(add2(sumA, sumB), s0, s1);
          l += s0 + s1;
          if (rescale) {
            const uint64_t a2 = f2(alpha, alpha);
#pragma unroll
            for (int c = 0; c < D / 32; ++c) tc::ld32(tO + c * 32, sr[c]);
            tc::wait_ld();
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                float x0, x1;
                unf2(mul2(f2(__uint_as_float(sr[c][2 * k]), __uint_as_float(sr[c][2 * k + 1])), a2), x0, x1);
                sr[c][2 * k] = __float_as_uint(x0);
                sr[c][2 * k + 1] = __float_as_uint(x1);
              }
              tc::st32(tO + c * 32, sr[c]);
            }
          }
          tc::wait_st();
          tc::fence_before();
        }
        if (edge && (t == 0 || !two)) {
          const int g = g0 + j, sv = g % C::NSV;
          if (!warp_wait(bar(C::B_VF + sv), (g / C::NSV) & 1)) {
            ok = false;
            break;
          }
          if (clean_v<D>(sbase + C::V_OFF + sv * C::TILE, r, max(ctx - k0, 0), s.len - k0))
            poison[it & 1] = it + 1;
          fence_proxy_async_smem();  // the MMA reads V through the async proxy
        }
        mbar_arrive(bar(C::B_PF + t));
        fetch_words(i + 1);
      }
      g0 += s.nt;
      if (!ok) break;
      // The P V that this thread reads are done. (n > 0 but for stream 1 of a single
      // tile; stream 0 has one at least.)
      float w0 = 1.f, w1 = 0.f;
      uint32_t acc = tO;             // what w0 weighs
      int c0 = 0, c1 = D / 32;       // 32-column blocks of the output that this thread has
      const bool join = !two && n1 > 0;
      if (!two) {
        ml[t * kBM + r] = make_float2(ref, l);
        mbar_arrive(bar(C::B_MF));
        if (!__all_sync(0xffffffffu, wait_or_abort(bar(C::B_MF), handed & 1, abort_flag))) break;
        ++handed;
        const float2 x = ml[r], y = ml[kBM + r];
        const float m = fmaxf(x.x, y.x);
        w0 = ex2_approx(x.x - m);
        w1 = ex2_approx(y.x - m);
        l = x.y * w0 + y.y * w1;
        ref = m;
        acc = tmem + (uint32_t(wq * 32) << 16) + 128;
        c0 = t * (D / 64);
        c1 = c0 + D / 64;
        if (!__all_sync(0xffffffffu, wait_or_abort(bar(C::B_OF), fin[0] & 1, abort_flag))) break;
        if (join && !__all_sync(0xffffffffu, wait_or_abort(bar(C::B_OF + 1), fin[1] & 1, abort_flag))) break;
      } else if (!__all_sync(0xffffffffu, wait_or_abort(bar(C::B_OF + t), fin[t] & 1, abort_flag))) {
        break;
      }
      ++fin[0];
      if (n1 > 0) ++fin[1];
      tc::fence_after();
      const bool whole = s.begins && s.left == 0;
      uint4 bad = make_uint4(0u, 0u, 0u, 0u);
      if (busy && poison[it & 1] == it + 1 && valid)
        bad = poisoned_dims<D>(v_cache, a, s.b, s.kvh, mask, s.n, ctx, s.t0 * kBN,
                               min((s.t0 + s.nt) * kBN, s.len));
      const int slot = 2 * cta + (s.begins ? 1 : 0);
      const size_t pt = static_cast<size_t>(slot) * 2 + (two ? t : 0);
      const bool empty = l == 0.f;
      const float inv = whole ? (empty ? 0.f : 1.f / l) : 1.f;
      const size_t row = static_cast<size_t>(s.tok0 + tok) * a.h + s.kvh * a.g + hh;
      const bool store = valid && ATTN_GUARD(row < static_cast<size_t>(a.total_q) * a.h, &g_tree_err) &&
                         ATTN_GUARD(slot < 2 * kRunsMaxCtas, &g_tree_err);
      const int out_row = store ? static_cast<int>(row) : -1;
#pragma unroll 1
      for (int c = c0; c < c1; ++c) {
        if (!busy) break;
        uint32_t ov[32];
        float x[32];
        tc::ld32(acc + c * 32, ov);
        tc::wait_ld();
#pragma unroll
        for (int k = 0; k < 32; ++k) x[k] = __uint_as_float(ov[k]) * w0;
        if (join) {
          tc::ld32(acc + 256 + c * 32, ov);
          tc::wait_ld();
#pragma unroll
          for (int k = 0; k < 32; ++k) x[k] = fmaf(__uint_as_float(ov[k]), w1, x[k]);
        }
        const uint32_t nan = c < 2 ? (c == 0 ? bad.x : bad.y) : (c == 2 ? bad.z : bad.w);
        if (nan != 0u)
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if ((nan >> k) & 1u) x[k] = __uint_as_float(0x7fc00000u);
        if (whole) {
          // 64 bytes of a row per thread; turned among four lanes so that they store
          // 64 contiguous bytes, of the four lanes' rows in turn.
          uint32_t y[4][4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int w = 0; w < 4; ++w)
              y[k][w] = empty ? 0u : pack_bf16x2(x[8 * k + 2 * w] * inv, x[8 * k + 2 * w + 1] * inv);
#pragma unroll
          for (int bit = 1; bit < 4; bit <<= 1)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if (k & bit) continue;
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                const bool up = lane & bit;
                const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? y[k][w] : y[k | bit][w], bit);
                y[k][w] = up ? got : y[k][w];
                y[k | bit][w] = up ? y[k | bit][w] : got;
              }
            }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int to = __shfl_sync(0xffffffffu, out_row, (lane & ~3) + k);
            if (to >= 0)
              *reinterpret_cast<uint4*>(out.o + static_cast<size_t>(to) * D + c * 32 + (lane & 3) * 8) =
                  make_uint4(y[k][0], y[k][1], y[k][2], y[k][3]);
          }
        } else if (store) {
          float4* dst = reinterpret_cast<float4*>(out.o_part + pt * (kBM * D)) + r;
#pragma unroll
          for (int k = 0; k < 8; ++k)
            dst[(c * 8 + k) * kBM] = make_float4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
        }
      }
      if (store && (two || t == 0)) {
        if (whole) {
          if (out.lse != nullptr) out.lse[row] = empty ? -INFINITY : ref * kLn2 + logf(l);
        } else {
          out.m_part[pt * kBM + r] = ref;
          out.l_part[pt * kBM + r] = l;
        }
      }
      if (tid == 0 && s.begins && s.left > 0)
        out.cut[cta] = TreeCut{static_cast<int>(1 + div_ll(s.left + plan.per - 1, plan.per)), s.tok0 + s.first,
                               min(2 * a.tpt, s.n - s.first), s.kvh};
      close(it);
      // O is read out before the next segment's first P V, which waits for this
      // thread's next P (behind ml_empty, where the other stream read it too).
      tc::fence_before();
      if (!two) mbar_arrive(bar(C::B_ME));
    }
  }

  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == C::MMA_WARP) tc::dealloc(tmem, 512);
}

// Joins the partial states of each unit that begins in an attention CTA and goes on
// behind it, in run order. An item is kMergeThreads / (D / 4) query rows of a cut unit,
// a thread 4 dims of one over all parts, kMergeUnroll of them in flight. One CTA per
// attention CTA: it looks at all cuts, and its groups take their share of the items. (On
// one GPU one row of 32768 keys took 35.9 us all in all, 24 rows with two row tiles 32.2;
// with a CTA per cut and 8 rows, most of them without work, 38.0 and 34.0; with 8 parts in
// flight 36.5 and 31.9, with 20 38.1 and 32.1; with two CTAs 2 us more (what the looks at the
// cuts cost: all read the same lines; a look per warp 5 us more).)
constexpr int kMergeThreads = 128, kMergeGroups = 4, kMergeUnroll = 10;
template <int D>
__global__ void __launch_bounds__(kMergeThreads* kMergeGroups)
    tree_merge_kernel(const TreeOut out, int h, int g, int tpt, int total_q) {
  constexpr int U = kMergeUnroll, R = kMergeThreads / (D / 4);
  constexpr int PER = kRunsMaxCtas / 32;  // cuts a lane: lane + 32 k
  static_assert(kRunsMaxCtas % 32 == 0, "a warp looks at the cuts");
  __shared__ TreeCut cuts[kRunsMaxCtas];  // [lane][k], and the items up to each one's end
  __shared__ int ends[kRunsMaxCtas];
  pdl_wait();
  pdl_trigger();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    TreeCut mine[PER];
    int sum = 0;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int i = lane + 32 * k;
      int4 x = make_int4(0, 0, 0, 0);
      if (i < static_cast<int>(gridDim.x)) x = __ldcg(reinterpret_cast<const int4*>(out.cut) + i);
      mine[k] = TreeCut{x.x, x.y, x.z, x.w};
    }
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      sum += mine[k].parts > 0 ? (mine[k].n_tok * g + R - 1) / R : 0;
      cuts[lane * PER + k] = mine[k];
      ends[lane * PER + k] = sum;
    }
    int before = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += y;
    }
    before -= sum;
#pragma unroll
    for (int k = 0; k < PER; ++k) ends[lane * PER + k] += before;
  }
  __syncthreads();
  const int total = ends[kRunsMaxCtas - 1], lane = threadIdx.x & 31;
  const int tid = threadIdx.x % kMergeThreads, group = threadIdx.x / kMergeThreads;
  for (int item = blockIdx.x + gridDim.x * group; item < total; item += gridDim.x * kMergeGroups) {
    int at = 0;  // the cut that the item is of
#pragma unroll
    for (int k = 0; k < PER; ++k)
      at += __popc(__ballot_sync(0xffffffffu, ends[lane * PER + k] <= item));
    const int cta = at / PER + 32 * (at % PER), first = at > 0 ? ends[at - 1] : 0;
    const TreeCut cut = cuts[at];
    const int parts = cut.parts, tok = cut.tok, n_tok = cut.n_tok, kvh = cut.kvh;
    const int c = tid / R, r = (item - first) * R + tid % R;
    if (r >= n_tok * g) continue;
    const int tile = r / (tpt * g), in_tile = r % (tpt * g);
    const size_t row = static_cast<size_t>(tok + r / g) * h + kvh * g + r % g;
    if (!ATTN_GUARD(row < static_cast<size_t>(total_q) * h, &g_tree_err)) continue;
    float M = kNone, L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int base = 0; base < parts; base += U) {
      float m[U], l[U];
      float4 x[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int j = base + i;
        m[i] = kNone;
        l[i] = 0.f;
        x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (j < parts) {
          const int slot = 2 * (cta + j) + (j == 0 ? 1 : 0);
          ATTN_DCHECK(slot < 2 * kRunsMaxCtas, &g_tree_err);
          const size_t pt = static_cast<size_t>(slot) * 2 + tile;
          m[i] = __ldcg(out.m_part + pt * kBM + in_tile);
          l[i] = __ldcg(out.l_part + pt * kBM + in_tile);
          x[i] = __ldcg(reinterpret_cast<const float4*>(out.o_part + pt * (kBM * D)) + c * kBM + in_tile);
        }
      }
      float Mn = M;
#pragma unroll
      for (int i = 0; i < U; ++i) Mn = fmaxf(Mn, m[i]);
      const float sc = ex2_approx(M - Mn);
      M = Mn;
      L *= sc;
      acc.x *= sc; acc.y *= sc; acc.z *= sc; acc.w *= sc;
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const float w = ex2_approx(m[i] - Mn);
        L = fmaf(w, l[i], L);
        acc.x = fmaf(w, x[i].x, acc.x);
        acc.y = fmaf(w, x[i].y, acc.y);
        acc.z = fmaf(w, x[i].z, acc.z);
        acc.w = fmaf(w, x[i].w, acc.w);
      }
    }
    const bool empty = L == 0.f;
    const float inv = empty ? 0.f : 1.f / L;
    uint2 y = make_uint2(0u, 0u);
    if (!empty) {
      y.x = pack_bf16x2(acc.x * inv, acc.y * inv);
      y.y = pack_bf16x2(acc.z * inv, acc.w * inv);
    }
    *reinterpret_cast<uint2*>(out.o + row * D + c * 4) = y;
    if (out.lse != nullptr && c == 0) out.lse[row] = empty ? -INFINITY : M * kLn2 + logf(L);
  }
}

template <int D>
cudaError_t launch_d(const TreeDecode& t, cudaStream_t stream) {
  using C = TrCfg<D>;
  const int g = t.h / t.h_kv, tpt = kBM / g;
  CUtensorMap tq, tk, tv;
  // Rows (token, head of the group): box of g heads x 128 / g tokens; map order (d, g,
  // KV head, token).
  const uint64_t qd[4] = {uint64_t(D), uint64_t(g), uint64_t(t.h_kv), uint64_t(t.total_q)};
  const uint64_t qs[3] = {uint64_t(D) * 2, uint64_t(g) * D * 2, uint64_t(t.h) * D * 2};
  const uint32_t qb[4] = {64u, uint32_t(g), 1u, uint32_t(tpt)};
  const uint64_t dims[4] = {uint64_t(D), uint64_t(t.h_kv), uint64_t(kPage), uint64_t(t.num_blocks)};
  const uint64_t strides[3] = {uint64_t(D) * 2, uint64_t(t.h_kv) * D * 2, uint64_t(kPage) * t.h_kv * D * 2};
  const uint32_t box[4] = {64u, 1u, uint32_t(kPage), 1u};
  if (encode_tensor_map(&tq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(t.q), qd, qs, qb,
                        CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS ||
      encode_tensor_map(&tk, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(t.k_cache), dims, strides,
                        box, CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS ||
      encode_tensor_map(&tv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(t.v_cache), dims, strides,
                        box, CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int grid = sms < kRunsMaxCtas ? sms : kRunsMaxCtas;
  const TreeRows a{t.block_table, t.cu_q, t.seq_lens, t.mask, t.B, t.total_q, t.max_q_len, t.words,
                   t.h, t.h_kv, g, t.max_blocks, t.num_blocks, tpt};
  uint8_t* ws = static_cast<uint8_t*>(t.workspace);
  const TreeLayout L = tree_layout(D);
  const TreeOut out{reinterpret_cast<TreeCut*>(ws), reinterpret_cast<float*>(ws + L.o_off),
                    reinterpret_cast<float*>(ws + L.m_off), reinterpret_cast<float*>(ws + L.l_off),
                    static_cast<__nv_bfloat16*>(t.o), t.lse};
  static_assert(sizeof(TreeCut) <= kTreeCutBytes, "workspace");
  auto kern = tree_kernel<D>;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kern, dim3(unsigned(grid)), dim3(C::THREADS), size_t(C::SMEM), stream, tq, tk, tv,
                 static_cast<const __nv_bfloat16*>(t.v_cache), a, out, t.scale * kLog2e);
  if (e != cudaSuccess) return e;
  return launch_pdl(tree_merge_kernel<D>, dim3(unsigned(grid)), dim3(kMergeThreads * kMergeGroups), 0, stream, out,
                    t.h, g, tpt, t.total_q);
}

}  // namespace

cudaError_t launch_decode_tree(const TreeDecode& t, cudaStream_t stream) {
  return t.d_h == 128 ? launch_d<128>(t, stream) : launch_d<64>(t, stream);
}

cudaError_t tree_set_stall(int key_tile, int what) {
#ifdef ATTN_DEBUG
  const int v[2] = {key_tile, what};
  return cudaMemcpyToSymbol(g_tree_stall, v, sizeof(v));
#else
  (void)key_tile;
  (void)what;
  return cudaErrorNotSupported;
#endif
}

unsigned int tree_read_and_clear_error(cudaStream_t stream, cudaError_t* st) {
  unsigned int v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(&v, g_tree_err, sizeof(v), 0, cudaMemcpyDeviceToHost, stream);
  if (e == cudaSuccess)
    e = cudaMemcpyToSymbolAsync(g_tree_err, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
  if (st) *st = e;
  return v;
}

}  // namespace attn
