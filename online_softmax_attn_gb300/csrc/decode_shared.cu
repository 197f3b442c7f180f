// decode_shared.cu -- decode of a batch whose rows share a prefix of keys.
//
// Row b attends to the prefix's keys and to its own. The two key sets are
// disjoint, so their states merge ("Merge normalized attention without
// averaging tile outputs"); the prefix's state is computed for all rows at
// once: the B * g query rows of a KV head are the M rows of dense products
// against each key tile, and the prefix is read once for all of them.
//
//   shared_kernel: in two phases, the prefix's states of every row by tcgen05,
//     and the states over the rows' own pages (runs_body of decode_runs.cuh on
//     the softmax warps). Every other group of CTAs takes the phases in the
//     other order, so that the products of one half run beside the memory
//     traffic of the other; as kernels behind each other the two took 127 +
//     66 us for 256 rows over 32768 keys and up to 700 of their own.
//   shared_merge_kernel: the states of a row, joined in a fixed order and
//     divided once.
//
// Prefix phase. Query rows of a KV head are ordered (token, head of the
// group), so a 128-row tile is one TMA box of 128 / g tokens x g heads. A CTA
// has two softmax warpgroups ("streams"; thread = row), a TMA warp and an MMA
// warp. NT = 2 (more than 128 rows): the streams are two row tiles that share
// each key tile. NT = 1: the streams take the key tiles of one row tile in
// turn, each with an accumulator of its own, so that one stream's exponentials
// overlap the other's MMAs in this case too. Steps alternate between the
// streams; per step S = Q K^T (SS), weights over S in tensor memory, O += P V
// (TS), with S of step e + 2 issued behind P V of step e.
//
// Work split: `groups` runs of equal length over the (KV head, key tile) pairs,
// times the row blocks (NT * 128 rows) as neighbouring CTAs, which read the
// same tiles at the same time, so the L2 serves all but one of them. A run that
// crosses a head border gives two states.
//
// P V is one fp16 MMA chain where V's tile is a tile of fp16 numbers: two warps
// convert each V tile in shared memory as it lands, times a power of two, and put
// ones into the slots past the last key. A tile with a number that does not convert
// exactly (kVShift) is loaded again and stays bf16, with P = P_hi + P_lo in two MMAs;
// so V enters as it is everywhere, however small a column's or a key's values are
// beside the rest of their tile. With the two-term P everywhere the prefix of 256
// rows over 32768 keys took 205 us.
#include "decode_runs.cuh"
#include "pdl.cuh"
#include "tc.cuh"

namespace attn {

static __device__ unsigned int g_shared_err;
#ifdef ATTN_DEBUG
// The key tile, in each CTA's own order, and which of its loads is not requested
// (attn_selftest_shared_stall): 0 K, 1 V, 2 V's second load.
static __device__ int g_shared_stall[2] = {-1, 0};
#endif

namespace {

constexpr int kBM = 128, kBN = 128;
// kTop, kSlack (decode_runs.cuh): a row's reference is set kTop below a new
// maximum and moves when a score passes it by kTop + kSlack. fp16 weights need
// that room below them. fp16 tiles hold V times 2^kVShift, and tiles that stay bf16
// have it in their weights instead, so that one accumulator serves both. With
// weights of up to 2^15 a sum over V passes fp32's range from |v| = 2^105 on, where
// its result need not: once a tile holds a magnitude of 2^kHuge the segment's rows
// go on with the maximum itself as reference and without kVShift, and its tiles
// stay bf16 with the two-term P. Up to 2^kHuge sums over 2^30 keys stay below 2^117.
constexpr int kHuge = 64;
// fp16 holds a bf16 number's 8 bits, times 2^kVShift, from 2^(-17 - kVShift) (8 bits
// above its smallest step, 2^-24) to below 2^(16 - kVShift). The lower 32 of these 33
// binades, 2^-25 to below 128, are the window that tiles are checked for: with kVWindow
// added the numbers in it, and no others, have 111 as their exponents' first bits, so
// the check is an addition and half an AND a pair. Zero, which converts, lies outside:
// a batch with anything outside is looked at again in the registers. (Exact limits for
// every pair, as minima and maxima of magnitudes, took 188 us for 256 rows over 32768
// keys, this way 186.6, without a check 182.3; rounding both to nearest and towards
// zero, 182.5, misses what both take to zero. A tile that goes on as bf16 costs its CTA
// 9 us.) Of tiles of 128 x 128 values from N(0, 1) one in 2500 holds a number that is
// too small, of N(0, 0.02^2) one in 50.
constexpr int kVShift = 8;
constexpr float kVScale = 1 << kVShift;
constexpr uint32_t kVLeast = (127 - 17 - kVShift) << 7, kVMost = (127 + 16 - kVShift) << 7;  // bits
constexpr uint32_t kVWindow = (224 - (127 - 17 - kVShift)) * 0x00800080u;
constexpr uint32_t kOnes = 0x3f803f80u;  // in slots past the last key, whose weights are 0
constexpr int kVFp16 = 0, kVWide = 1, kVHuge = 2;  // a V tile's format (wide[])

template <int D, int NT>
struct SpCfg {
  static constexpr int SUBS = D / 64;
  static constexpr int SUB_BYTES = 128 * 128;
  static constexpr int TILE = kBN * D * 2;
  static constexpr int NSK = NT == 2 ? 2 : 3;
  static constexpr int NSV = 3;
  static constexpr int Q_OFF = 0;
  static constexpr int K_OFF = Q_OFF + NT * TILE;
  static constexpr int V_OFF = K_OFF + NSK * TILE;
  // q_full, q_empty, k_full[], k_empty[], v_full[] (landed), v_ready[]
  // (converted), v_empty[], v_again (a tile loaded once more), s_full[2],
  // p_full[2], o_final[2], mma_done
  static constexpr int B_KF = 2, B_KE = B_KF + NSK, B_VF = B_KE + NSK, B_VR = B_VF + NSV,
                       B_VE = B_VR + NSV, B_VA = B_VE + NSV, B_SF = B_VA + 1, B_PF = B_SF + 2,
                       B_OF = B_PF + 2, B_DONE = B_OF + 2, NBAR = B_DONE + 1;
  static_assert(NBAR <= 32, "one warp initialises the barriers, one per lane");
  static constexpr int NST = D == 128 ? 3 : 4;
  using Own = Cfg<false, D, 8, NST>;  // the other phase, from offset 0
  static constexpr int TILES_END = V_OFF + NSV * TILE;
  static constexpr int BAR_OFF = TILES_END > Own::SMEM ? TILES_END : Own::SMEM;
  static constexpr int MISC_OFF = BAR_OFF + NBAR * 8;  // tensor-memory slot, abort flag, wide[NSV]
  static constexpr int SMEM = MISC_OFF + 32 + 1024;
  static_assert(SMEM + sizeof(RunShared<8>) <= 227 * 1024, "shared memory of an SM");
  static constexpr int THREADS = 384;  // two softmax warpgroups, one of control
  static constexpr int PRODUCER_WARP = 8, MMA_WARP = 9, CONV_WARP = 10;  // to 11
  static constexpr int CONV_THREADS = 64;
  static constexpr int REG_LAUNCH = 168, REG_CONTROL = 120, REG_SOFTMAX = 192;
  static_assert(2 * 128 * REG_SOFTMAX + 128 * REG_CONTROL <= THREADS * REG_LAUNCH,
                "register split exceeds the launch allocation");
};

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
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
      atomicOr(&g_shared_err, ATTN_DEVERR_WAIT_TIMEOUT);
      *abort_flag = 1;
      return false;
    }
  }
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
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
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

// Weights of a key tile in the rare cases, out of line: where V stays bf16
// (`two`) P_hi (upper 16 bits) in columns 0-63 of the S tile and P_lo =
// bf16(p - P_hi) in columns 64-127, of weights times v_scale (what fp16 tiles hold V
// times), else fp16 as in the common case. The scores enter as rounded products
// minus the reference, which is exact near it at any magnitude of the logits. Reads
// the S tile again (keys from lim on masked) and returns the weights' sum (without
// v_scale). Warp-collective.
__device__ __noinline__ float rare_weights(uint32_t tS, int lim, float scale_log2, float ref, bool two,
                                           float v_scale) {
  float sum0 = 0.f, sum1 = 0.f;
  uint32_t sr[4][32];
#pragma unroll
  for (int c = 0; c < 4; ++c) tc::ld32(tS + c * 32, sr[c]);
  tc::wait_ld();
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t hi[32], lo[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const int key = 64 * half + 2 * i;
      float x0 = __uint_as_float(sr[key >> 5][key & 31]);
      float x1 = __uint_as_float(sr[key >> 5][(key & 31) + 1]);
      if (key >= lim) x0 = -INFINITY;
      if (key + 1 >= lim) x1 = -INFINITY;
      const float p0 = ex2_approx(__fsub_rn(__fmul_rn(x0, scale_log2), ref));
      const float p1 = ex2_approx(__fsub_rn(__fmul_rn(x1, scale_log2), ref));
      sum0 += p0;
      sum1 += p1;
      if (!two) {
        hi[i] = pack_f16x2(p0, p1);
        lo[i] = 0u;
        continue;
      }
      const float y0 = p0 * v_scale, y1 = p1 * v_scale;
      hi[i] = split_hi(y0, y1);
      lo[i] = split_lo(y0, y1);
    }
    tc::st32(tS + 32 * half, hi);
    if (two) tc::st32(tS + 64 + 32 * half, lo);
  }
  return sum0 + sum1;
}

// Bits, but the sign, of the largest magnitude in a converter thread's chunks of a V
// tile (every 64th from `base` on, the thread's first), of keys before lim.
template <int D>
__device__ __noinline__ uint32_t largest_bits(uint32_t base, int ct, int lim) {
  uint32_t m = 0x80008000u;  // behind a set sign bit the bits are in order as signed halves
#pragma unroll 1
  for (int i = 0; i < D / 4; ++i) {
    if ((((i * 64 + ct) >> 3) & (kBN - 1)) >= lim) continue;
    const uint4 x = lds128(base + i * (64 * 16));
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) asm("max.s16x2 %0, %0, %1;" : "+r"(m) : "r"(w[k] | 0x80008000u));
  }
  return max(m & 0x7fffu, (m >> 16) & 0x7fffu);
}

// Two bf16 numbers times 2^kVShift as fp16 numbers.
__device__ __forceinline__ __nv_bfloat162 v_scaled(uint32_t w) {
  return __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w), __floats2bfloat162_rn(kVScale, kVScale));
}
__device__ __forceinline__ uint32_t v_fp16(__nv_bfloat162 y) {
  const uint32_t u = *reinterpret_cast<const uint32_t*>(&y);
  return pack_f16x2(bf16lo(u), bf16hi(u));
}

struct PrefixArgs {
  const int32_t* table;
  const int32_t* len;
  int max_blocks, num_blocks, h_kv, groups, n_rb, s_cap, rows;  // rows = B * g per KV head
  float *o, *m, *l;
};

// The run of key tiles of one CTA group.
struct PrefixRun {
  int len, tiles;       // prefix length, key tiles per head
  long long per, lo, hi;
};
__device__ __forceinline__ PrefixRun prefix_run(const PrefixArgs& a, int group) {
  PrefixRun r;
  r.len = min(max(__ldcg(a.len), 0), a.max_blocks * kPage);
  r.tiles = (r.len + kBN - 1) / kBN;
  const long long all = static_cast<long long>(r.tiles) * a.h_kv;
  r.per = max(1ll, (all + a.groups - 1) / a.groups);
  r.lo = min(all, r.per * group);
  r.hi = min(all, r.lo + r.per);
  return r;
}

// The rows' own pages (runs_body's arguments).
struct OwnArgs {
  const uint8_t* kc;
  const uint8_t* vc;
  const __nv_bfloat16* q;
  const int32_t* block_table;
  Rows rw;
  int h, g, max_blocks;
  RunOut out;
};

template <int D, int NT>
__global__ void __launch_bounds__(384, 1)
    shared_kernel(const __grid_constant__ CUtensorMap tmap_q,
                  const __grid_constant__ CUtensorMap tmap_k,
                  const __grid_constant__ CUtensorMap tmap_v, const PrefixArgs a,
                  const OwnArgs own, int tok_per_tile, float scale_log2) {
  using C = SpCfg<D, NT>;
  extern __shared__ __align__(16) uint8_t smem_raw[];  // (1024 would pad the static part)
  __shared__ RunShared<8> sh;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) { return sbase + C::BAR_OFF + 8 * i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::MISC_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::MISC_OFF + 4);
  volatile int* wide = reinterpret_cast<volatile int*>(smem + C::MISC_OFF + 8);  // [NSV]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rb = blockIdx.x % a.n_rb, group = blockIdx.x / a.n_rb;

  if (threadIdx.x == 0) {
    prefetch_tmap(&tmap_q);
    prefetch_tmap(&tmap_k);
    prefetch_tmap(&tmap_v);
    *abort_flag = 0;
  }
  if (warp == 0 && lane < C::NBAR) {
    mbar_init(bar(lane), lane == C::B_PF || lane == C::B_PF + 1          ? 128u
                         : lane >= C::B_VR && lane < C::B_VR + C::NSV ? uint32_t(C::CONV_THREADS)
                                                                      : 1u);
    fence_barrier_init();
  }
  if (warp == C::MMA_WARP) tc::alloc(smem_u32(tmem_slot), 512);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = *tmem_slot;
  // q, the prefix's length, table and pages are earlier kernels' output. The
  // merge is not let in before this kernel's end: its waiting CTAs gather on the
  // SMs that fall free first, and it then runs on half of them (56.5 us instead of
  // 49.9 for 64 rows over 8192 keys, wherever this kernel triggers).
  pdl_wait();
  const PrefixRun run = prefix_run(a, group);
  if (blockIdx.x == 0 && threadIdx.x == 0)
    (void)clamp_seq_len(__ldcg(a.len), a.max_blocks * kPage, &g_shared_err);

#ifdef ATTN_DEBUG
  const int stall_tile = g_shared_stall[0], stall_what = g_shared_stall[1];
  auto stalled = [=](int g, int what) { return g == stall_tile && what == stall_what; };
#else
  auto stalled = [](int, int) { return false; };
#endif

  // A segment: key tiles [t0, t0 + nt) of KV head kvh. Every role walks the
  // same segments.
  struct Seg {
    int kvh, t0, nt;
  };
  auto seg_at = [&](long long p) -> Seg {
    Seg s;
    s.kvh = static_cast<int>(p / run.tiles);
    s.t0 = static_cast<int>(p % run.tiles);
    s.nt = static_cast<int>(min(static_cast<long long>(run.tiles - s.t0), run.hi - p));
    return s;
  };
  // Steps e = 0, 1, ... of a segment alternate between the streams: stream
  // e & 1; key tile e (NT = 1) or e / 2 (NT = 2).
  auto n_steps = [](const Seg& s) { return NT == 2 ? 2 * s.nt : s.nt; };
  auto tile_of = [](int e) { return NT == 2 ? e >> 1 : e; };
  auto n_of = [&](const Seg& s, int t) { return (n_steps(s) + 1 - t) >> 1; };
  const int n_pages = (run.len + kPage - 1) / kPage;
  // Table entries of the 32 pages from `page` on, one per lane; -1 (reads as
  // zeros) behind the prefix.
  auto entries = [&](int page) { return page + lane < n_pages ? __ldcg(a.table + page + lane) : -1; };
  // Key tile of 8 pages into dst: lane i < 8 * SUBS issues the box of page
  // i % 8, half i / 8 (one thread issuing all of them took 90 cycles a box).
  // `ent` holds the tile's entries in lanes at .. at + 7. Whole warp.
  auto load_tile = [&](uint32_t dst, const CUtensorMap* map, uint32_t b, int kvh, int ent, int at,
                       int page0) {
    int phys = __shfl_sync(0xffffffffu, ent, at + (lane & 7));
    if (phys < 0 || phys >= a.num_blocks) {
      if (page0 + (lane & 7) < n_pages) atomicOr(&g_shared_err, ATTN_DEVERR_BAD_PAGE);
      phys = -1;
    }
    if (lane == 0) mbar_arrive_expect_tx(b, C::TILE);
    if (lane < 8 * C::SUBS)
      tma_load_4d(dst + (lane >> 3) * C::SUB_BYTES + (lane & 7) * kPage * 128, map, b,
                  (lane >> 3) * 64, kvh, 0, phys);
    __syncwarp();
  };

  // The rows' own pages, before the prefix in every other group of CTAs (the
  // row blocks of a group read the same key tiles and stay together). Both
  // phases use the same shared memory: all warps meet between them, and the
  // generic accesses of one come before the copies of the other.
  const bool own_first = group & 1;
  auto own_phase = [&] {
    // Runs are handed out from the last CTA on: where there is little work of
    // either kind, no CTA gets both.
    const int n_cta = min(int(gridDim.x), kRunsMaxCtas), cta = int(gridDim.x) - 1 - int(blockIdx.x);
    if (cta < n_cta)
      runs_body<false, D, 8, C::NST>(own.kc, own.vc, nullptr, nullptr, own.q, own.block_table, own.rw,
                                     own.h, a.h_kv, own.g, own.max_blocks, a.num_blocks, scale_log2,
                                     own.out, smem, sh, cta, n_cta, &g_shared_err,
                                     [] { asm volatile("barrier.cta.sync 2, 256;" ::: "memory"); });
  };
  auto meet = [] {
    fence_proxy_async_smem();
    __syncthreads();
  };

  if (warp >= C::PRODUCER_WARP) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REG_CONTROL));
    if (own_first) meet();
    if (warp == C::PRODUCER_WARP) {
      // ---------------------------------------------------------- producer
      auto wait = [&](uint32_t b, uint32_t parity) {
        return __all_sync(0xffffffffu, wait_or_abort(b, parity, abort_flag));
      };
      int it = 0, g0 = 0, q_issued = 0, k_issued = 0, v_issued = 0;
      bool ok = true;
      for (long long p = run.lo; ok && p < run.hi; ++it) {
        const Seg s = seg_at(p);
        p += s.nt;
        int ent = entries(s.t0 * 8), next = -1;
        if (it > 0 && !wait(bar(1), (it - 1) & 1)) break;
        if (lane == 0) mbar_arrive_expect_tx(bar(0), NT * C::TILE);
        if (lane < NT * C::SUBS)
          tma_load_4d(sbase + C::Q_OFF + lane * C::SUB_BYTES, &tmap_q, bar(0), (lane % C::SUBS) * 64, 0,
                      s.kvh, (rb * NT + lane / C::SUBS) * tok_per_tile);
        __syncwarp();
        q_issued = it + 1;
        for (int j = 0; j < s.nt; ++j) {
          const int g = g0 + j, sk = g % C::NSK, sv = g % C::NSV, page0 = (s.t0 + j) * 8;
          if ((j & 3) == 0) {  // entries four tiles at a time, fetched four tiles ahead
            if (j > 0) ent = next;
            next = entries(page0 + 32);
          }
          if (g >= C::NSK && !wait(bar(C::B_KE + sk), (g / C::NSK - 1) & 1)) {
            ok = false;
            break;
          }
          if (!stalled(g, 0))
            load_tile(sbase + C::K_OFF + sk * C::TILE, &tmap_k, bar(C::B_KF + sk), s.kvh, ent, (j & 3) * 8,
                      page0);
          k_issued = g + 1;
          if (g >= C::NSV && !wait(bar(C::B_VE + sv), (g / C::NSV - 1) & 1)) {
            ok = false;
            break;
          }
          if (!stalled(g, 1))
            load_tile(sbase + C::V_OFF + sv * C::TILE, &tmap_v, bar(C::B_VF + sv), s.kvh, ent, (j & 3) * 8,
                      page0);
          v_issued = g + 1;
        }
        g0 += s.nt;
      }
      if (*abort_flag) {
        // Drain: the newest load of each stage is the only one that can still
        // be in flight. Bounded waits, error already recorded.
        if (q_issued > 0) (void)mbar_wait(bar(0), (q_issued - 1) & 1, &g_shared_err);
        for (int g = max(0, k_issued - C::NSK); g < k_issued; ++g)
          if (!stalled(g, 0)) (void)mbar_wait(bar(C::B_KF + g % C::NSK), (g / C::NSK) & 1, &g_shared_err);
        for (int g = max(0, v_issued - C::NSV); g < v_issued; ++g)
          if (!stalled(g, 1)) (void)mbar_wait(bar(C::B_VF + g % C::NSV), (g / C::NSV) & 1, &g_shared_err);
      }
    } else if (warp == C::MMA_WARP) {
      // -------------------------------------------------------- MMA issuer
      constexpr uint32_t idS = tc::idesc_bf16_f32(kBM, kBN, false, false);
      constexpr uint32_t idO = tc::idesc_bf16_f32(kBM, D, false, true);
      const uint64_t dq0 = tc::sw128_desc(sbase + C::Q_OFF, 16, 1024);
      const uint64_t dk0 = tc::sw128_desc(sbase + C::K_OFF, 16, 1024);
      const uint64_t dv0 = tc::sw128_desc(sbase + C::V_OFF, C::SUB_BYTES, 1024);
      auto issue_s = [&](int t, int st) {
        const uint64_t da = dq0 + uint64_t(((NT == 2 ? t : 0) * C::TILE) >> 4);
        const uint64_t db = dk0 + uint64_t((st * C::TILE) >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off16 = ((kk >> 2) * C::SUB_BYTES + (kk & 3) * 32) >> 4;
          tc::mma_ss_elect(tmem + t * 256, da + off16, db + off16, idS, kk > 0 ? 1u : 0u);
        }
        tc::commit_elect(bar(C::B_SF + t));
      };
      constexpr uint32_t idO16 = tc::idesc_f16_f32(kBM, D, false, true);
      auto issue_pv = [&](int t, int st, bool acc, bool two) {
        const uint64_t db = dv0 + uint64_t((st * C::TILE) >> 4);
        const uint32_t dO = tmem + t * 256 + 128, aP = tmem + t * 256;
        if (!two) {
#pragma unroll
          for (int kk = 0; kk < kBN / 16; ++kk)
            tc::mma_ts_elect(dO, aP + kk * 8, db + uint64_t((kk * 16 * 128) >> 4), idO16,
                             (acc || kk > 0) ? 1u : 0u);
        } else {
#pragma unroll
          for (int kk = 0; kk < kBN / 16; ++kk) {
            const uint64_t b = db + uint64_t((kk * 16 * 128) >> 4);
            tc::mma_ts_elect(dO, aP + kk * 8, b, idO, (acc || kk > 0) ? 1u : 0u);
            tc::mma_ts_elect(dO, aP + 64 + kk * 8, b, idO, 1u);
          }
        }
      };
      auto wait = [&](uint32_t b, uint32_t parity) {
        return __all_sync(0xffffffffu, wait_or_abort(b, parity, abort_flag));
      };
      bool ok = true;
      int it = 0, g0 = 0, base[2] = {0, 0};
      for (long long p = run.lo; ok && p < run.hi; ++it) {
        const Seg s = seg_at(p);
        p += s.nt;
        const int n = n_steps(s);
        ok = wait(bar(0), it & 1);
        // S of step e once its K tile is there (first use) and, behind it,
        // what it frees.
        auto s_step = [&](int e) {
          const int g = g0 + tile_of(e), st = g % C::NSK;
          if (!wait(bar(C::B_KF + st), (g / C::NSK) & 1)) return false;
          tc::fence_after();
          issue_s(e & 1, st);
          if (NT == 1 || (e & 1)) tc::commit_elect(bar(C::B_KE + st));
          if (e == n - 1) tc::commit_elect(bar(1));  // Q's last reader
          return true;
        };
        for (int e = -2; ok && e < n; ++e) {
          if (e >= 0) {
            const int t = e & 1, g = g0 + tile_of(e), sv = g % C::NSV;
            ok = wait(bar(C::B_PF + t), (base[t] + (e >> 1)) & 1) &&
                 wait(bar(C::B_VR + sv), (g / C::NSV) & 1);
            if (!ok) break;
            tc::fence_after();
            issue_pv(t, sv, e >= 2, __shfl_sync(0xffffffffu, wide[sv], 0) != 0);
            if (NT == 1 || t == 1) tc::commit_elect(bar(C::B_VE + sv));
            if (e + 2 >= n) tc::commit_elect(bar(C::B_OF + t));  // the stream's last step
          }
          if (e + 2 < n) ok = s_step(e + 2);
        }
        g0 += s.nt;
        base[0] += n_of(s, 0);
        base[1] += n_of(s, 1);
      }
      tc::commit_elect(bar(C::B_DONE));
      (void)__all_sync(0xffffffffu, mbar_wait(bar(C::B_DONE), 0, &g_shared_err));
    } else {
      // -------------------------------------------------------- V to fp16
      const int ct = threadIdx.x - C::CONV_WARP * 32;  // 0 .. 63
      constexpr int CHUNKS = C::TILE / 16, PER = CHUNKS / C::CONV_THREADS, UN = 4;
      int g0 = 0, again = 0;
      bool ok = true;
      for (long long p = run.lo; ok && p < run.hi;) {
        const Seg s = seg_at(p);
        p += s.nt;
        bool huge = false;  // a tile of the segment so far
        for (int j = 0; j < s.nt; ++j) {
          const int g = g0 + j, sv = g % C::NSV;
          if (!__all_sync(0xffffffffu, wait_or_abort(bar(C::B_VF + sv), (g / C::NSV) & 1, abort_flag)))
            ok = false;
          const uint32_t base = sbase + C::V_OFF + sv * C::TILE + ct * 16;
          const int lim = min(kBN, run.len - (s.t0 + j) * kBN);  // keys that exist
          bool off = false;
          uint32_t in = 0xffffffffu;  // the window's bits: cleared by a number outside it
          if (ok) {
#pragma unroll 1
            for (int i0 = 0; i0 < PER; i0 += UN) {
              uint4 x[UN];
#pragma unroll
              for (int u = 0; u < UN; ++u)
                asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(x[u].x), "=r"(x[u].y), "=r"(x[u].z), "=r"(x[u].w)
                             : "r"(base + (i0 + u) * (C::CONV_THREADS * 16)));
#pragma unroll
              for (int u = 0; u < UN; ++u) {
                // Chunk index (i0 + u) * 64 + ct, 8 chunks per 128-byte row.
                const int row = (((i0 + u) * C::CONV_THREADS + ct) >> 3) & (kBN - 1);
                if (row >= lim) x[u] = make_uint4(kOnes, kOnes, kOnes, kOnes);
                const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
                uint32_t hh[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  hh[k] = v_fp16(v_scaled(w[k]));
                  in &= w[k] + kVWindow;
                }
                asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                                 base + (i0 + u) * (C::CONV_THREADS * 16)),
                             "r"(hh[0]), "r"(hh[1]), "r"(hh[2]), "r"(hh[3])
                             : "memory");
              }
              if ((in & 0x70007000u) != 0x70007000u) {  // zeros do convert
                // Behind a set sign bit the bits are in order as signed halves; with 1
                // taken off, zero becomes the largest.
                uint32_t most = 0x80008000u, least = 0x7fff7fffu;
#pragma unroll
                for (int u = 0; u < UN; ++u) {
                  const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
                  for (int k = 0; k < 4; ++k) {
                    const uint32_t m = w[k] | 0x80008000u;
                    asm("max.s16x2 %0, %0, %1;" : "+r"(most) : "r"(m));
                    asm("min.s16x2 %0, %0, %1;" : "+r"(least) : "r"(m - 0x00010001u));
                  }
                }
                off = off || min(least & 0x7fffu, (least >> 16) & 0x7fffu) + 1 < kVLeast ||
                      max(most & 0x7fffu, (most >> 16) & 0x7fffu) >= kVMost;
                in = 0xffffffffu;
              }
            }
          }
          // Agreed by the 64 threads.
          auto any = [](bool mine) {
            int r;
            asm volatile(
                "{\n\t.reg .pred p, q;\n\t"
                "setp.ne.s32 p, %1, 0;\n\t"
                "barrier.cta.red.or.pred q, 1, 64, p;\n\t"
                "selp.s32 %0, 1, 0, q;\n\t}"
                : "=r"(r)
                : "r"(mine ? 1 : 0)
                : "memory");
            return r != 0;
          };
          int fmt = kVFp16;
          if (any(huge || off)) {
            // The tile as it was. The generic writes above come before the
            // copy engine's.
            fence_proxy_async_smem();
            asm volatile("barrier.cta.sync 1, 64;" ::: "memory");
            if (warp == C::CONV_WARP && !stalled(g, 2) && __all_sync(0xffffffffu, ok)) {
              const int page0 = (s.t0 + j) * 8;
              load_tile(sbase + C::V_OFF + sv * C::TILE, &tmap_v, bar(C::B_VA), s.kvh, entries(page0), 0,
                        page0);
            }
            if (ok && !__all_sync(0xffffffffu, wait_or_abort(bar(C::B_VA), again & 1, abort_flag))) {
              ok = false;
              (void)mbar_wait(bar(C::B_VA), again & 1, &g_shared_err);  // bounded: let it land
            }
            ++again;
            huge = any(huge || largest_bits<D>(base, ct, lim) >= (127u + kHuge) << 7);
            fmt = huge ? kVHuge : kVWide;
            // Slots past the last key hold whatever the cache holds (possibly
            // NaN or inf); their weights are 0, but 0 * NaN is not.
            if (lim < kBN)
              for (int c = lim * 8 + ct; c < kBN * 8; c += C::CONV_THREADS)
#pragma unroll
                for (int u = 0; u < C::SUBS; ++u)
                  asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(
                                   sbase + C::V_OFF + sv * C::TILE + u * C::SUB_BYTES + c * 16),
                               "r"(0u)
                               : "memory");
          }
          if (ct == 0) wide[sv] = fmt;
          fence_proxy_async_smem();  // the MMA reads V through the async proxy
          mbar_arrive(bar(C::B_VR + sv));
          // Agreed by both warps before either goes on (an abort ends both).
          int all_ok;
          asm volatile(
              "{\n\t.reg .pred p, q;\n\t"
              "setp.ne.s32 p, %1, 0;\n\t"
              "barrier.cta.red.and.pred q, 1, 64, p;\n\t"
              "selp.s32 %0, 1, 0, q;\n\t}"
              : "=r"(all_ok)
              : "r"(ok ? 1 : 0)
              : "memory");
          ok = all_ok != 0;
          if (!ok) break;
        }
        g0 += s.nt;
      }
    }
    if (!own_first) meet();
  } else {
    // ------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REG_SOFTMAX));
    if (own_first) {
      own_phase();
      meet();
    }
    const int t = warp >> 2, wq = warp & 3, r = wq * 32 + lane;
    const uint32_t tS = tmem + (uint32_t(wq * 32) << 16) + t * 256, tO = tS + 128;
    const long long row = (static_cast<long long>(rb) * NT + (NT == 2 ? t : 0)) * kBM + r;
    int g0 = 0, cnt = 0, ofin = 0;
    bool ok = true;
    for (long long p = run.lo; ok && p < run.hi;) {
      const Seg s = seg_at(p);
      const int touch = group - static_cast<int>((static_cast<long long>(s.kvh) * run.tiles) / run.per);
      p += s.nt;
      const int n = n_of(s, t);
      float ref = kNone, l = 0.f, top = kTop;
      for (int i = 0; i < n; ++i, ++cnt) {
        const int j = NT == 2 ? i : 2 * i + t;  // key tile within the segment
        if (!__all_sync(0xffffffffu, wait_or_abort(bar(C::B_SF + t), cnt & 1, abort_flag))) {
          ok = false;
          break;
        }
        const int lim = min(kBN, run.len - (s.t0 + j) * kBN);  // keys that exist
        tc::fence_after();
        uint32_t sr[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tc::ld32(tS + c * 32, sr[c]);
        tc::wait_ld();
        if (lim < kBN) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int i2 = 0; i2 < 32; ++i2)
              if (c * 32 + i2 >= lim) sr[c][i2] = __float_as_uint(-INFINITY);
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
        const float cand = fmaxf(max3(cm[0], cm[1], cm[2]), cm[3]) * scale_log2;
        float alpha = 1.f;
        if (cand - ref > top + kSlack) {
          float next = cand - top;  // where fp32's spacing is too wide for that, cand itself
          if (cand - next > top + kSlack) next = cand;
          alpha = ex2_approx(ref - next);
          l *= alpha;
          ref = next;
        }
        const int g = g0 + j, sv = g % C::NSV;
        if (!__all_sync(0xffffffffu, wait_or_abort(bar(C::B_VR + sv), (g / C::NSV) & 1, abort_flag))) {
          ok = false;
          break;
        }
        const int fmt = __shfl_sync(0xffffffffu, wide[sv], 0);
        if (fmt == kVHuge && top != 0.f) {  // from here on weights of at most 2^kSlack,
          const float next = ref + top, down = ex2_approx(ref - next);  // and V as it is
          alpha *= down * (1.f / kVScale);
          l *= down;
          ref = next;
          top = 0.f;
        }
        const bool two = fmt != kVFp16, rescale = i > 0 && __any_sync(0xffffffffu, alpha != 1.f);
        // Below 2^20 the products' and the reference's roundings cannot take a
        // weight past fp16's range.
        if (!two && !__any_sync(0xffffffffu, fabsf(ref) >= 0x1p20f)) {
          // fp16 weights: key pair (2k, 2k + 1) of chunk c in column 16c + k,
          // staged in registers whose scores are used up.
          const uint64_t c2 = f2(scale_log2, scale_log2), n2 = f2(-ref, -ref);
          uint64_t sumA = f2(0.f, 0.f), sumB = f2(0.f, 0.f);
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              float y0, y1;
              unf2(fma2(f2(__uint_as_float(sr[c][2 * k]), __uint_as_float(sr[c][2 * k + 1])), c2, n2), y0, y1);
              const float p0 = ex2_approx(y0), p1 = ex2_approx(y1);
              if (k & 1) sumB = add2(sumB, f2(p0, p1)); else sumA = add2(sumA, f2(p0, p1));
              sr[c][k] = pack_f16x2(p0, p1);
            }
          uint32_t pw[32];
#pragma unroll
          for (int half = 0; half < 2; ++half) {
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              pw[k] = sr[2 * half][k];
              pw[16 + k] = sr[2 * half + 1][k];
            }
            tc::st32(tS + 32 * half, pw);
          }
          float s0, s1;
          unf2(add2(sumA, sumB), s0, s1);
          l += s0 + s1;
        } else {
          l += rare_weights(tS, lim, scale_log2, ref, two, top != 0.f ? kVScale : 1.f);
        }
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
        mbar_arrive(bar(C::B_PF + t));
      }
      if (!ok) break;
      if (n > 0) {
        if (!__all_sync(0xffffffffu, wait_or_abort(bar(C::B_OF + t), ofin & 1, abort_flag))) break;
        ++ofin;
        tc::fence_after();
      }
      // The state of this row over the segment (m in log2 units).
      // Accumulators as [d_h / 4][128 rows][4], so that a warp stores 512
      // contiguous bytes.
      const size_t slot =
          ((static_cast<size_t>(s.kvh) * a.s_cap + touch) * a.n_rb + rb) * 2 + t;
      const size_t pi = slot * kBM + r;
      float* so = a.o + slot * kBM * D + r * 4;
      const bool store = row < a.rows && touch >= 0 && touch < a.s_cap;
      const float v_inv = top != 0.f ? 1.f / kVScale : 1.f;
      ATTN_DCHECK(touch >= 0 && touch < a.s_cap, &g_shared_err);
      ATTN_DCHECK(!store || pi < static_cast<size_t>(a.h_kv) * a.s_cap * a.n_rb * (2 * kBM), &g_shared_err);
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t ov[32];
        if (n > 0) {
          tc::ld32(tO + c * 32, ov);
          tc::wait_ld();
        }
        if (store && n > 0) {
#pragma unroll
          for (int i2 = 0; i2 < 8; ++i2)
            *reinterpret_cast<float4*>(so + (c * 8 + i2) * (kBM * 4)) =
                make_float4(__uint_as_float(ov[4 * i2]) * v_inv, __uint_as_float(ov[4 * i2 + 1]) * v_inv,
                            __uint_as_float(ov[4 * i2 + 2]) * v_inv, __uint_as_float(ov[4 * i2 + 3]) * v_inv);
        }
      }
      if (store) {
        a.m[pi] = ref;
        a.l[pi] = l;
      }
      // O is read out before the next segment's first P V, which waits for
      // this thread's next P.
      tc::fence_before();
      g0 += s.nt;
    }
    if (!own_first) {
      meet();
      own_phase();
    }
  }

  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == C::MMA_WARP) tc::dealloc(tmem, 512);
}

// Joins a row's states: the prefix's (one per CTA that had a part of the head's
// tiles, two with NT = 1), then its own, in that order, and divides once. A CTA
// takes kMergeRows neighbouring (token, head) rows of a KV head; a thread has 4
// dims of one row over all its states, kMergeUnroll of them in flight.
constexpr int kMergeRows = 8, kMergeUnroll = 8;
struct MergeArgs {
  PrefixArgs p;
  int NT, h, g, upr;
  const long long* plan;
  const float *o_part, *m_part, *l_part, *o_row, *m_row, *l_row;
  __nv_bfloat16* out;
  float* lse;
};

template <int D>
__global__ void __launch_bounds__(kMergeRows* D / 4) shared_merge_kernel(const MergeArgs a) {
  constexpr int U = kMergeUnroll;
  const int kvh = blockIdx.y, c = threadIdx.x / kMergeRows;
  const long long pr = static_cast<long long>(blockIdx.x) * kMergeRows + threadIdx.x % kMergeRows;
  pdl_wait();
  // The next kernel may start once every CTA of this one runs. With more CTAs
  // than the GPU holds at a time (three per SM) it would come in on whichever
  // SMs fall free: the next call's row blocks, neighbours that share key tiles,
  // then lie scattered (256 rows over 32768 keys: 215 us a call, else 181),
  // while 64 rows over 8192 keys gain (55.0 us without, 50.0 with).
  if (gridDim.x * gridDim.y <= 3 * 152) pdl_trigger();
  if (pr >= a.p.rows) return;
  const int b = static_cast<int>(pr / a.g), hh = static_cast<int>(pr % a.g);
  const size_t row = static_cast<size_t>(b) * a.h + kvh * a.g + hh;
  if (!ATTN_GUARD(row < static_cast<size_t>(a.p.rows / a.g) * a.h, &g_shared_err)) return;
  // Own states' place (loads first: the prefix's length is one round trip too).
  const long long per = __ldcg(a.plan), at = __ldcg(a.plan + 1 + b);
  const long long wu = __ldcg(a.plan + 2 + b) - at;  // weight of one unit
  const PrefixRun run = prefix_run(a.p, 0);
  int n_pre = 0, per_touch = 1;
  size_t pre0 = 0;
  if (run.tiles > 0) {
    const long long s = static_cast<long long>(kvh) * run.tiles;
    n_pre = static_cast<int>((s + run.tiles - 1) / run.per - s / run.per) + 1;
    const int rb = static_cast<int>(pr / (a.NT * kBM)), rt = static_cast<int>(pr % (a.NT * kBM));
    pre0 = ((static_cast<size_t>(kvh) * a.p.s_cap * a.p.n_rb + rb) * 2 + rt / kBM) * kBM + rt % kBM;
    per_touch = a.NT == 1 ? 2 : 1;
    n_pre *= per_touch;
  }
  int n_own = 0;
  long long c0 = 0;
  if (wu > 0) {
    const long long s = at * a.upr + kvh * wu;
    c0 = (s + kRunsUnit) / per;
    n_own = static_cast<int>((s + wu - 1) / per - c0) + 1;
  }
  const int n = n_pre + n_own;
  float M = kNone, L = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int base = 0; base < n; base += U) {
    float m[U], l[U];
    float4 x[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int j = base + i;
      m[i] = kNone;
      l[i] = 0.f;
      x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (j < n_pre) {
        const size_t idx = pre0 + ((j / per_touch) * static_cast<size_t>(a.p.n_rb) * 2 + j % per_touch) * kBM;
        m[i] = __ldcg(a.p.m + idx);
        l[i] = __ldcg(a.p.l + idx);
        // (a stream without key tiles stores no accumulators: not used then)
        x[i] = __ldcg(reinterpret_cast<const float4*>(a.p.o + (idx - idx % kBM) * D + (idx % kBM) * 4 +
                                                      c * (kBM * 4)));
      } else if (j < n) {
        const bool cut = n_own > 1;
        const size_t idx = cut ? (2 * (c0 + j - n_pre) + (j == n_pre ? 1 : 0)) * 8 + hh : row;
        m[i] = __ldcg((cut ? a.m_part : a.m_row) + idx);
        l[i] = __ldcg((cut ? a.l_part : a.l_row) + idx);
        x[i] = __ldcg(reinterpret_cast<const float4*>((cut ? a.o_part : a.o_row) + idx * D + c * 4));
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
      if (m[i] != kNone) {
        acc.x = fmaf(w, x[i].x, acc.x);
        acc.y = fmaf(w, x[i].y, acc.y);
        acc.z = fmaf(w, x[i].z, acc.z);
        acc.w = fmaf(w, x[i].w, acc.w);
      }
    }
  }
  const bool empty = L == 0.f;
  const float inv = empty ? 0.f : 1.f / L;
  uint2 y = make_uint2(0u, 0u);
  if (!empty) {
    y.x = pack_bf16x2(acc.x * inv, acc.y * inv);
    y.y = pack_bf16x2(acc.z * inv, acc.w * inv);
  }
  *reinterpret_cast<uint2*>(a.out + row * D + c * 4) = y;
  if (a.lse != nullptr && c == 0) a.lse[row] = empty ? -INFINITY : M * kLn2 + logf(L);
}

template <int D, int NT>
cudaError_t launch_states(const SharedArgs& s, const SharedPlan& pl, const PrefixArgs& a,
                          cudaStream_t stream) {
  using C = SpCfg<D, NT>;
  const DecodeRunsArgs& r = s.own;
  const int g = r.h / r.h_kv;
  CUtensorMap tq, tk, tv;
  const uint64_t qd[4] = {uint64_t(D), uint64_t(g), uint64_t(r.h_kv), uint64_t(r.B)};
  const uint64_t qs[3] = {uint64_t(D) * 2, uint64_t(g) * D * 2, uint64_t(r.h) * D * 2};
  // Rows (token, head): box of g heads x 128 / g tokens; map order (d, g, KV
  // head, token).
  const uint32_t qb[4] = {64u, uint32_t(g), 1u, uint32_t(kBM / g)};
  const uint64_t dims[4] = {uint64_t(D), uint64_t(r.h_kv), uint64_t(kPage), uint64_t(r.num_blocks)};
  const uint64_t strides[3] = {uint64_t(D) * 2, uint64_t(r.h_kv) * D * 2,
                               uint64_t(kPage) * r.h_kv * D * 2};
  const uint32_t box[4] = {64u, 1u, uint32_t(kPage), 1u};
  if (encode_tensor_map(&tq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(r.q), qd, qs, qb,
                        CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS ||
      encode_tensor_map(&tk, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(r.k_cache), dims,
                        strides, box, CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS ||
      encode_tensor_map(&tv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(r.v_cache), dims,
                        strides, box, CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  OwnArgs own;
  own.kc = static_cast<const uint8_t*>(r.k_cache);
  own.vc = static_cast<const uint8_t*>(r.v_cache);
  own.q = static_cast<const __nv_bfloat16*>(r.q);
  own.block_table = r.block_table;
  own.rw = Rows{r.seq_lens, r.B, r.max_blocks * kPage, r.h_kv, 1};
  own.h = r.h;
  own.g = g;
  own.max_blocks = r.max_blocks;
  own.out = RunOut{r.plan, r.o_part, r.m_part, r.l_part, r.o_row, r.m_row, r.l_row, nullptr, nullptr};
  auto kern = shared_kernel<D, NT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(unsigned(pl.groups) * pl.n_rb), dim3(C::THREADS), size_t(C::SMEM), stream,
                    tq, tk, tv, a, own, kBM / g, r.scale * kLog2e);
}

}  // namespace

cudaError_t launch_shared(const SharedArgs& s, cudaStream_t stream) {
  const DecodeRunsArgs& r = s.own;
  const int g = r.h / r.h_kv;
  const SharedPlan pl = shared_plan(r.B, g, r.h_kv);
  PrefixArgs a;
  a.table = s.prefix_table;
  a.len = s.prefix_len;
  a.max_blocks = s.max_prefix_blocks;
  a.num_blocks = r.num_blocks;
  a.h_kv = r.h_kv;
  a.groups = pl.groups;
  a.n_rb = pl.n_rb;
  a.s_cap = pl.s_cap;
  a.rows = r.B * g;
  a.o = s.pre_o;
  a.m = s.pre_m;
  a.l = s.pre_l;
  cudaError_t e;
  if (r.d_h == 128)
    e = pl.nt == 2 ? launch_states<128, 2>(s, pl, a, stream) : launch_states<128, 1>(s, pl, a, stream);
  else
    e = pl.nt == 2 ? launch_states<64, 2>(s, pl, a, stream) : launch_states<64, 1>(s, pl, a, stream);
  if (e != cudaSuccess) return e;
  MergeArgs m;
  m.p = a;
  m.NT = pl.nt;
  m.h = r.h;
  m.g = g;
  m.upr = r.h_kv;
  m.plan = r.plan;
  m.o_part = r.o_part;
  m.m_part = r.m_part;
  m.l_part = r.l_part;
  m.o_row = r.o_row;
  m.m_row = r.m_row;
  m.l_row = r.l_row;
  m.out = static_cast<__nv_bfloat16*>(r.o);
  m.lse = r.lse;
  auto merge = r.d_h == 128 ? shared_merge_kernel<128> : shared_merge_kernel<64>;
  return launch_pdl(merge, dim3(unsigned((a.rows + kMergeRows - 1) / kMergeRows), unsigned(r.h_kv)),
                    dim3(unsigned(kMergeRows * r.d_h / 4)), 0, stream, m);
}

cudaError_t shared_set_stall(int key_tile, int what) {
#ifdef ATTN_DEBUG
  const int v[2] = {key_tile, what};
  return cudaMemcpyToSymbol(g_shared_stall, v, sizeof(v));
#else
  (void)key_tile;
  (void)what;
  return cudaErrorNotSupported;
#endif
}

unsigned int shared_read_and_clear_error(cudaStream_t stream, cudaError_t* st) {
  unsigned int v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(&v, g_shared_err, sizeof(v), 0, cudaMemcpyDeviceToHost,
                                            stream);
  if (e == cudaSuccess)
    e = cudaMemcpyToSymbolAsync(g_shared_err, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
  if (st) *st = e;
  return v;
}

}  // namespace attn
