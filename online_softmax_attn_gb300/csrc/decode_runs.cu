// decode_runs.cu -- attn_decode_paged_e4m3: the run decode (decode_runs.cuh) over
// the 8-bit cache, and the merge of the rows that its runs cut; for few keys both
// in one kernel. attn_decode_paged_window and attn_decode_paged_window_e4m3 are the
// same kernels over the pages that a row's window and its first tokens leave.
#include "decode_runs.cuh"
#include "pdl.cuh"

namespace attn {

static __device__ unsigned int g_decode_runs_err;

namespace {

// 8 warps and one CTA per SM, 4 stages (d_h = 128). Two CTAs of 2 stages took
// 22.4 instead of 20.9 us for a row of 32768 keys (twice as many parts to join)
// and 170.8 instead of 173.0 for 66 rows of up to 16384; 12 warps of 3 stages
// 21.5 and 173.4, 16 of 2 24.0 and 170.7.
template <bool E8, int D, int NST, class R>
__global__ void __launch_bounds__(256, 1)
    decode_runs_kernel(const uint8_t* __restrict__ kc, const uint8_t* __restrict__ vc,
                       const uint8_t* __restrict__ ks, const uint8_t* __restrict__ vs, const __nv_bfloat16* __restrict__ q,
                       const int32_t* __restrict__ block_table, R rw, int h, int h_kv, int g,
                       int max_blocks, int num_blocks, float qscale, const RunOut out) {
  extern __shared__ __align__(16) uint8_t smem_raw[];  // (1024 would pad the static part)
  __shared__ RunShared<8> sh;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  pdl_wait();     // lengths, table, q and the cache are earlier kernels' output
  pdl_trigger();
  if constexpr (R::kWindow) {
    if (threadIdx.x == 0) out.cut[blockIdx.x].parts = 0;
  }
  runs_body<E8, D, 8, NST>(kc, vc, ks, vs, q, block_table, rw, h, h_kv, g, max_blocks,
                           num_blocks, qscale, out, smem, sh, blockIdx.x, gridDim.x,
                           &g_decode_runs_err, [] { __syncthreads(); });
}

// Joins the n partial states of (row, head) `row`, head hh of its block, that the CTAs
// from c0 on hold, and divides once. A CTA of 128 threads: warps take the states in
// turn (a row alone on the GPU has 38 per head: one round trip).
template <int D>
__device__ __forceinline__ void merge_parts(const float* __restrict__ o_part, const float* __restrict__ m_part,
                                            const float* __restrict__ l_part, long long c0, int n, int hh,
                                            size_t row, __nv_bfloat16* __restrict__ o,
                                            float* __restrict__ lse) {
  constexpr int VEC = D / 32, U = 10, NW = 4;  // 40 states in flight
  __shared__ float sm[NW], sl[NW], so[NW][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
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
        const size_t slot = (2 * (c0 + j) + (j == 0 ? 1 : 0)) * 8 + hh;
        ATTN_DCHECK(slot < 2 * kRunsMaxCtas * 8, &g_decode_runs_err);
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

// Merge of the rows that the runs' borders cut, and of empty rows. One CTA per (row,
// head).
template <int D>
__global__ void __launch_bounds__(128)
    decode_runs_merge_kernel(const float* __restrict__ o_part, const float* __restrict__ m_part,
                         const float* __restrict__ l_part, const long long* __restrict__ plan,
                         int h, int g, int n_gb, int upr, __nv_bfloat16* __restrict__ o,
                         float* __restrict__ lse) {
  const int b = blockIdx.x / h, hq = blockIdx.x % h;
  pdl_wait();
  pdl_trigger();
  const long long per = __ldcg(plan), at = __ldcg(plan + 1 + b);
  const long long wu = __ldcg(plan + 2 + b) - at;  // weight of one unit: its pages + kRunsUnit
  const size_t row = static_cast<size_t>(b) * h + hq;
  if (!ATTN_GUARD(row < gridDim.x && per > 0 && wu >= 0, &g_decode_runs_err)) return;
  if (wu == 0) {
    for (int i = threadIdx.x; i < D / 2; i += 128) reinterpret_cast<uint32_t*>(o + row * D)[i] = 0u;
    if (lse != nullptr && threadIdx.x == 0) lse[row] = -INFINITY;
    return;
  }
  const int u = (hq / g) * n_gb + (hq % g) / 8;
  const long long s = at * upr + u * wu;
  const long long c0 = (s + kRunsUnit) / per;  // CTAs of the unit's first and last page
  const int n = static_cast<int>((s + wu - 1) / per - c0) + 1;
  if (n == 1) return;  // finished by its CTA
  merge_parts<D>(o_part, m_part, l_part, c0, n, (hq % g) % 8, row, o, lse);
}

// The same for windows, whose units are many and short: head blockIdx.y of the unit
// that begins in CTA blockIdx.x of the runs and goes on behind it, and empty rows. (A
// CTA per (row, head) took 6 us for 66 rows of 32 heads and 10 for 200, most of them
// finished already.)
template <int D>
__global__ void __launch_bounds__(128)
    decode_window_merge_kernel(const float* __restrict__ o_part, const float* __restrict__ m_part,
                               const float* __restrict__ l_part, const RunCut* __restrict__ cut,
                               const Rows rw, int h, __nv_bfloat16* __restrict__ o,
                               float* __restrict__ lse) {
  const int hh = blockIdx.y;
  pdl_wait();
  pdl_trigger();
  const int parts = __ldcg(&cut[blockIdx.x].parts);
  if (parts > 0) {
    const int row0 = __ldcg(&cut[blockIdx.x].row0), nh = __ldcg(&cut[blockIdx.x].nh);
    const size_t row = static_cast<size_t>(row0) + hh;
    if (hh < nh && ATTN_GUARD(row < static_cast<size_t>(rw.B) * h, &g_decode_runs_err))
      merge_parts<D>(o_part, m_part, l_part, blockIdx.x, parts, hh, row, o, lse);
  }
  for (int b = blockIdx.x + gridDim.x * hh; b < rw.B; b += gridDim.x * gridDim.y) {
    if (row_len(rw, b) > 0) continue;
    const size_t row = static_cast<size_t>(b) * h;
    for (int i = threadIdx.x; i < h * (D / 8); i += 128)
      reinterpret_cast<uint4*>(o + row * D)[i] = make_uint4(0u, 0u, 0u, 0u);
    if (lse != nullptr)
      for (int i = threadIdx.x; i < h; i += 128) lse[row + i] = -INFINITY;
  }
}

// Few rows of few keys: one kernel. A cluster of 8 CTAs has one unit (row, KV
// head, head block), cut into 64 runs; the CTAs' states go through L2, and CTA
// i joins head i's behind a cluster barrier, where a second kernel's launch and
// its reads of the plan took as long as the pages. Taken up to kUnitMost units
// and tables of kUnitBlocks pages (the lengths are on the device), us a call,
// else with two kernels: one row of 16, 1000, 4000, 8000 keys, 8 KV heads of 128
// 6.7, 7.5, 9.4, 12.0, else 8.1, 9.0, 10.1, 11.8; of 64 1000, 4000 keys 6.7, 8.0,
// else 7.7, 8.5; 14 units of 1000 keys 7.6, else 9.3; 16 units 12.7, else 9.4 (not
// all clusters fit at a time). Windows of the bf16 cache, whose pages are twice as long,
// have the same borders: one row, 8 KV heads of 128, windows of 1000, 2000, 4000 keys 7.8,
// 8.0, 9.8, else 8.5, 9.1, 10.0; 14 units 8.2, 8.7, 10.7, else 9.1, 10.3, 12.0; 16 units
// 13.7, 14.4, 18.0, else 9.2, 10.4, 12.8 (one head alone crosses at 3500: 8.8, else 8.6).
constexpr int kClusterCtas = 8;
constexpr int kUnitMost = 14, kUnitBlocks = 256;
static_assert(kUnitMost * kClusterCtas <= kRunsMaxCtas, "workspace of the partial states");
template <bool E8, int D, int NST, class R>
__global__ void __launch_bounds__(256, 1) __cluster_dims__(kClusterCtas)
    decode_unit_kernel(const uint8_t* __restrict__ kc, const uint8_t* __restrict__ vc,
                       const uint8_t* __restrict__ ks, const uint8_t* __restrict__ vs, const __nv_bfloat16* __restrict__ q,
                       const int32_t* __restrict__ block_table, R rw, int h, int h_kv, int g, int n_gb,
                       int max_blocks, int num_blocks, float qscale, const RunOut out) {
  using C = Cfg<E8, D, 8, NST>;
  constexpr size_t kHead = E8 ? C::PAGE_BYTES : D * 2;  // bytes from one head of a page to the next
  extern __shared__ __align__(16) uint8_t smem_raw[];  // (1024 would pad the static part)
  __shared__ RunShared<8> sh;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const int unit = blockIdx.x / kClusterCtas, cta = blockIdx.x % kClusterCtas;
  const int upr = h_kv * n_gb, b = unit / upr, kvh = unit % upr / n_gb, gb = unit % n_gb;
  const int nh = min(8, g - gb * 8);
  const size_t row0 = static_cast<size_t>(b) * h + kvh * g + gb * 8;
  RunOut mine = out;  // this unit alone
  mine.plan = nullptr;
  mine.o_part += static_cast<size_t>(unit) * (2 * kClusterCtas * 8) * D;
  mine.m_part += unit * (2 * kClusterCtas * 8);
  mine.l_part += unit * (2 * kClusterCtas * 8);
  mine.o += row0 * D;
  if (mine.lse != nullptr) mine.lse += row0;
  pdl_wait();     // lengths, table, q and the cache are earlier kernels' output
  pdl_trigger();
  rw.seq_lens += b;
  rw.B = rw.upr = rw.n_gb = 1;
  runs_body<E8, D, 8, NST>(kc + kvh * kHead, vc + kvh * kHead, ks + kvh * kPage, vs + kvh * kPage,
                           q + row0 * D, block_table + static_cast<size_t>(b) * max_blocks, rw, h,
                           h_kv, nh, max_blocks, num_blocks, qscale, mine, smem, sh, cta, kClusterCtas,
                           &g_decode_runs_err, [] { __syncthreads(); });
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
  if (cta >= nh || threadIdx.x >= 32) return;
  constexpr int VEC = D / 32;
  const int lane = threadIdx.x, wu = row_weight(rw, row_len(rw, 0));
  if (!ATTN_GUARD(row0 + cta < static_cast<size_t>(gridDim.x / (kClusterCtas * upr)) * h, &g_decode_runs_err))
    return;
  if (wu == 0) {  // an empty row
    for (int i = lane; i < D / 2; i += 32) reinterpret_cast<uint32_t*>(mine.o + cta * D)[i] = 0u;
    if (mine.lse != nullptr && lane == 0) mine.lse[cta] = -INFINITY;
    return;
  }
  const int per = max(kMinRun, (wu + kClusterCtas * 8 - 1) / (kClusterCtas * 8)) * 8;
  const int c0 = R::kUnit / per, n = (wu - 1) / per - c0 + 1;
  if (n == 1) return;  // finished by its CTA
  float m[kClusterCtas], l[kClusterCtas], x[kClusterCtas][VEC];
  float M = kNone;
#pragma unroll
  for (int j = 0; j < kClusterCtas; ++j) {
    m[j] = kNone;
    l[j] = 0.f;
#pragma unroll
    for (int e = 0; e < VEC; ++e) x[j][e] = 0.f;
    if (j < n) {
      const int slot = (2 * (c0 + j) + (j == 0 ? 1 : 0)) * 8 + cta;
      m[j] = __ldcg(mine.m_part + slot);
      l[j] = __ldcg(mine.l_part + slot);
      const float* src = mine.o_part + slot * D + lane * VEC;
      if constexpr (VEC == 4) {
        const float4 t = __ldcg(reinterpret_cast<const float4*>(src));
        x[j][0] = t.x; x[j][1] = t.y; x[j][2] = t.z; x[j][3] = t.w;
      } else {
        const float2 t = __ldcg(reinterpret_cast<const float2*>(src));
        x[j][0] = t.x; x[j][1] = t.y;
      }
    }
  }
#pragma unroll
  for (int j = 0; j < kClusterCtas; ++j) M = fmaxf(M, m[j]);
  float L = 0.f, acc[VEC] = {};
#pragma unroll
  for (int j = 0; j < kClusterCtas; ++j) {
    const float w = ex2_approx(m[j] - M);
    L = fmaf(w, l[j], L);
#pragma unroll
    for (int e = 0; e < VEC; ++e) acc[e] = fmaf(w, x[j][e], acc[e]);
  }
  const bool empty = L == 0.f;
  const float inv = empty ? 0.f : 1.f / L;
#pragma unroll
  for (int e = 0; e < VEC; e += 2)
    *reinterpret_cast<uint32_t*>(mine.o + cta * D + lane * VEC + e) =
        empty ? 0u : pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
  if (mine.lse != nullptr && lane == 0) mine.lse[cta] = empty ? -INFINITY : M * kLn2 + logf(L);
}

template <class R>
R rows_of(const DecodeRunsArgs& a) {
  const int n_gb = (a.h / a.h_kv + 7) / 8;
  R rw{};
  static_cast<Rows&>(rw) = Rows{a.seq_lens, a.B, a.max_blocks * kPage, a.h_kv * n_gb, n_gb};
  if constexpr (R::kWindow) {
    rw.window = a.window;
    rw.sinks = a.sinks;
  }
  return rw;
}

template <bool E8, int D, int NST, class R>
cudaError_t launch_unit(const DecodeRunsArgs& a, cudaStream_t stream) {
  constexpr int kSmem = Cfg<E8, D, 8, NST>::SMEM + 1024;
  static_assert(kSmem + sizeof(RunShared<8>) <= 227 * 1024, "shared memory of an SM");
  auto kern = decode_unit_kernel<E8, D, NST, R>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  const R rw = rows_of<R>(a);
  const RunOut out{nullptr, a.o_part, a.m_part, a.l_part, nullptr,
                   nullptr, nullptr,  static_cast<__nv_bfloat16*>(a.o), a.lse};
  return launch_pdl(kern, dim3(unsigned(a.B * rw.upr * kClusterCtas)), dim3(256), size_t(kSmem), stream,
                    static_cast<const uint8_t*>(a.k_cache), static_cast<const uint8_t*>(a.v_cache), a.k_exp, a.v_exp,
                    static_cast<const __nv_bfloat16*>(a.q), a.block_table, rw, a.h, a.h_kv, a.h / a.h_kv, rw.n_gb,
                    a.max_blocks, a.num_blocks, a.scale * kLog2e, out);
}

template <bool E8, int D, int NST, class R>
cudaError_t launch_cfg(const DecodeRunsArgs& a, int sms, cudaStream_t stream) {
  using C = Cfg<E8, D, 8, NST>;
  constexpr int kSmem = C::SMEM + 1024;
  static_assert(kSmem + sizeof(RunShared<8>) <= 227 * 1024, "shared memory of an SM");
  static_assert(sizeof(RunCut) * kRunsMaxCtas <= kRunsCutBytes, "workspace");
  auto kern = decode_runs_kernel<E8, D, NST, R>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  const int grid = sms < kRunsMaxCtas ? sms : kRunsMaxCtas;
  const RunOut out{R::kWindow ? nullptr : a.plan, a.o_part, a.m_part, a.l_part, nullptr,
                   nullptr, nullptr,  static_cast<__nv_bfloat16*>(a.o), a.lse,
                   static_cast<RunCut*>(a.cut)};
  return launch_pdl(kern, dim3(grid), dim3(256), size_t(kSmem), stream,
                    static_cast<const uint8_t*>(a.k_cache), static_cast<const uint8_t*>(a.v_cache), a.k_exp, a.v_exp,
                    static_cast<const __nv_bfloat16*>(a.q), a.block_table, rows_of<R>(a), a.h, a.h_kv,
                    a.h / a.h_kv, a.max_blocks, a.num_blocks, a.scale * kLog2e, out);
}

cudaError_t sm_count(int* sms) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
  return e;
}

}  // namespace

namespace {
// `most`: pages that a row can have, known on the host.
template <bool E8, int NST128, int NST64, class One, class R>
cudaError_t launch_runs(const DecodeRunsArgs& a, int most, cudaStream_t stream) {
  const long long units = static_cast<long long>(a.B) * a.h_kv * ((a.h / a.h_kv + 7) / 8);
  if (units <= kUnitMost && most <= kUnitBlocks)
    return a.d_h == 128 ? launch_unit<E8, 128, NST128, One>(a, stream) : launch_unit<E8, 64, NST64, One>(a, stream);
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  e = a.d_h == 128 ? launch_cfg<E8, 128, NST128, R>(a, sms, stream)
                   : launch_cfg<E8, 64, NST64, R>(a, sms, stream);
  if (e != cudaSuccess) return e;
  const int g = a.h / a.h_kv, n_gb = (g + 7) / 8;
  if constexpr (R::kWindow) {
    const int ctas = sms < kRunsMaxCtas ? sms : kRunsMaxCtas;
    auto merge = a.d_h == 128 ? decode_window_merge_kernel<128> : decode_window_merge_kernel<64>;
    const Rows rw = rows_of<Rows>(a);
    return launch_pdl(merge, dim3(unsigned(ctas), unsigned(g < 8 ? g : 8)), dim3(128), 0, stream,
                      static_cast<const float*>(a.o_part), static_cast<const float*>(a.m_part),
                      static_cast<const float*>(a.l_part), static_cast<const RunCut*>(a.cut), rw, a.h,
                      static_cast<__nv_bfloat16*>(a.o), a.lse);
  }
  auto merge = a.d_h == 128 ? decode_runs_merge_kernel<128> : decode_runs_merge_kernel<64>;
  return launch_pdl(merge, dim3(unsigned(a.B) * a.h), dim3(128), 0, stream,
                    static_cast<const float*>(a.o_part), static_cast<const float*>(a.m_part),
                    static_cast<const float*>(a.l_part), static_cast<const long long*>(a.plan), a.h,
                    g, n_gb, a.h_kv * n_gb, static_cast<__nv_bfloat16*>(a.o), a.lse);
}
}  // namespace

cudaError_t launch_decode8(const DecodeRunsArgs& a, cudaStream_t stream) {
  return launch_runs<true, 4, 6, Rows, Rows>(a, a.max_blocks, stream);
}

// Units of windows are short, so what one weighs beside its pages matters: 200 rows of
// the 8-bit cache, window 2001, took 157.8 us with 1, 147.7 with 3, 142.2 with 5, 142.8
// with 8 (66 rows of the bf16 cache, window 4096: 158.2, 159.0, 158.9, 159.4), before the
// merge went by the runs' borders (now 134.5 and 155.5).
constexpr int kWindowUnit = 5;
cudaError_t launch_decode_window(const DecodeRunsArgs& a, cudaStream_t stream) {
  // The window's pages (one more where it starts inside a page) and the sinks'.
  const long long seen = (a.window + 14ll) / kPage + 1 + (a.sinks + 15ll) / kPage;
  const int most = seen < a.max_blocks ? static_cast<int>(seen) : a.max_blocks;
  using One = WindowRows<kRunsUnit>;  // a unit on its own is cut as a whole row's
  using Many = WindowRows<kWindowUnit>;
  return a.k_exp != nullptr ? launch_runs<true, 4, 6, One, Many>(a, most, stream)
                            : launch_runs<false, 3, 6, One, Many>(a, most, stream);
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
