// decode_runs.cu -- attn_decode_paged_e4m3: the run decode (decode_runs.cuh) over
// the 8-bit cache, and the merge of the rows that its runs cut; for few keys both
// in one kernel.
#include "decode_runs.cuh"
#include "pdl.cuh"

namespace attn {

static __device__ unsigned int g_decode_runs_err;

namespace {

// 8 warps and one CTA per SM, 4 stages (d_h = 128). Two CTAs of 2 stages took
// 22.4 instead of 20.9 us for a row of 32768 keys (twice as many parts to join)
// and 170.8 instead of 173.0 for 66 rows of up to 16384; 12 warps of 3 stages
// 21.5 and 173.4, 16 of 2 24.0 and 170.7.
template <int D, int NST>
__global__ void __launch_bounds__(256, 1)
    decode_runs_kernel(const uint8_t* __restrict__ kc, const uint8_t* __restrict__ vc,
                       const uint8_t* __restrict__ ks, const uint8_t* __restrict__ vs, const __nv_bfloat16* __restrict__ q,
                       const int32_t* __restrict__ block_table, Rows rw, int h, int h_kv, int g,
                       int max_blocks, int num_blocks, float qscale, const RunOut out) {
  extern __shared__ __align__(16) uint8_t smem_raw[];  // (1024 would pad the static part)
  __shared__ RunShared<8> sh;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  pdl_wait();     // lengths, table, q and the cache are earlier kernels' output
  pdl_trigger();
  runs_body<true, D, 8, NST>(kc, vc, ks, vs, q, block_table, rw, h, h_kv, g, max_blocks,
                             num_blocks, qscale, out, smem, sh, blockIdx.x, gridDim.x,
                             &g_decode_runs_err, [] { __syncthreads(); });
}

// Joins the partial states of each (row, head) that a run border cut, and
// writes empty rows. One CTA per (row, head), warps take its partials in turn
// (a row alone on the GPU has 38 per head: one round trip).
template <int D>
__global__ void __launch_bounds__(128)
    decode_runs_merge_kernel(const float* __restrict__ o_part, const float* __restrict__ m_part,
                         const float* __restrict__ l_part, const long long* __restrict__ plan,
                         int h, int g, int n_gb, int upr, __nv_bfloat16* __restrict__ o,
                         float* __restrict__ lse) {
  constexpr int VEC = D / 32, U = 10, NW = 4;  // 40 states in flight
  __shared__ float sm[NW], sl[NW], so[NW][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = blockIdx.x / h, hq = blockIdx.x % h;
  pdl_wait();
  pdl_trigger();
  const long long per = __ldcg(plan), at = __ldcg(plan + 1 + b);
  const long long wu = __ldcg(plan + 2 + b) - at;  // weight of one unit: its pages + kUnit
  const size_t row = static_cast<size_t>(b) * h + hq;
  if (!ATTN_GUARD(row < gridDim.x && per > 0 && wu >= 0, &g_decode_runs_err)) return;
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

// Few rows of few keys: one kernel. A cluster of 8 CTAs has one unit (row, KV
// head, head block), cut into 64 runs; the CTAs' states go through L2, and CTA
// i joins head i's behind a cluster barrier, where a second kernel's launch and
// its reads of the plan took as long as the pages. Taken up to kUnitMost units
// and tables of kUnitBlocks pages (the lengths are on the device), us a call,
// else with two kernels: one row of 16, 1000, 4000, 8000 keys, 8 KV heads of 128
// 6.7, 7.5, 9.4, 12.0, else 8.1, 9.0, 10.1, 11.8; of 64 1000, 4000 keys 6.7, 8.0,
// else 7.7, 8.5; 14 units of 1000 keys 7.6, else 9.3; 16 units 12.7, else 9.4 (not
// all clusters fit at a time).
constexpr int kClusterCtas = 8;
constexpr int kUnitMost = 14, kUnitBlocks = 256;
static_assert(kUnitMost * kClusterCtas <= kRunsMaxCtas, "workspace of the partial states");
template <int D, int NST>
__global__ void __launch_bounds__(256, 1) __cluster_dims__(kClusterCtas)
    decode_unit_kernel(const uint8_t* __restrict__ kc, const uint8_t* __restrict__ vc,
                       const uint8_t* __restrict__ ks, const uint8_t* __restrict__ vs, const __nv_bfloat16* __restrict__ q,
                       const int32_t* __restrict__ block_table, const int32_t* __restrict__ seq_lens, int h, int h_kv,
                       int g, int n_gb, int max_blocks, int num_blocks, float qscale, const RunOut out) {
  using C = Cfg<true, D, 8, NST>;
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
  const Rows rw{seq_lens + b, 1, max_blocks * kPage, 1, 1};
  runs_body<true, D, 8, NST>(kc + static_cast<size_t>(kvh) * C::PAGE_BYTES,
                             vc + static_cast<size_t>(kvh) * C::PAGE_BYTES, ks + kvh * kPage,
                             vs + kvh * kPage, q + row0 * D,
                             block_table + static_cast<size_t>(b) * max_blocks, rw, h, h_kv, nh,
                             max_blocks, num_blocks, qscale, mine, smem, sh, cta, kClusterCtas,
                             &g_decode_runs_err, [] { __syncthreads(); });
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
  if (cta >= nh || threadIdx.x >= 32) return;
  constexpr int VEC = D / 32;
  const int lane = threadIdx.x, wu = row_weight(row_len(rw, 0));
  if (!ATTN_GUARD(row0 + cta < static_cast<size_t>(gridDim.x / (kClusterCtas * upr)) * h, &g_decode_runs_err))
    return;
  if (wu == 0) {  // an empty row
    for (int i = lane; i < D / 2; i += 32) reinterpret_cast<uint32_t*>(mine.o + cta * D)[i] = 0u;
    if (mine.lse != nullptr && lane == 0) mine.lse[cta] = -INFINITY;
    return;
  }
  const int per = max(kMinRun, (wu + kClusterCtas * 8 - 1) / (kClusterCtas * 8)) * 8;
  const int c0 = kUnit / per, n = (wu - 1) / per - c0 + 1;
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

template <int D, int NST>
cudaError_t launch_unit(const DecodeRunsArgs& a, cudaStream_t stream) {
  constexpr int kSmem = Cfg<true, D, 8, NST>::SMEM + 1024;
  auto kern = decode_unit_kernel<D, NST>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  const int g = a.h / a.h_kv, n_gb = (g + 7) / 8;
  const RunOut out{nullptr, a.o_part, a.m_part, a.l_part, nullptr,
                   nullptr, nullptr,  static_cast<__nv_bfloat16*>(a.o), a.lse};
  return launch_pdl(kern, dim3(unsigned(a.B * a.h_kv * n_gb * kClusterCtas)), dim3(256), size_t(kSmem), stream,
                    static_cast<const uint8_t*>(a.k_cache), static_cast<const uint8_t*>(a.v_cache), a.k_exp, a.v_exp,
                    static_cast<const __nv_bfloat16*>(a.q), a.block_table, a.seq_lens, a.h, a.h_kv, g, n_gb,
                    a.max_blocks, a.num_blocks, a.scale * kLog2e, out);
}

template <int D, int NST>
cudaError_t launch_cfg(const DecodeRunsArgs& a, int sms, cudaStream_t stream) {
  using C = Cfg<true, D, 8, NST>;
  constexpr int kSmem = C::SMEM + 1024;
  static_assert(kSmem + sizeof(RunShared<8>) <= 227 * 1024, "shared memory of an SM");
  auto kern = decode_runs_kernel<D, NST>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  const int grid = sms < kRunsMaxCtas ? sms : kRunsMaxCtas;
  const int g = a.h / a.h_kv, n_gb = (g + 7) / 8;
  const Rows rw{a.seq_lens, a.B, a.max_blocks * kPage, a.h_kv * n_gb, n_gb};
  const RunOut out{a.plan,  a.o_part, a.m_part, a.l_part, nullptr,
                   nullptr, nullptr,  static_cast<__nv_bfloat16*>(a.o), a.lse};
  return launch_pdl(kern, dim3(grid), dim3(256), size_t(kSmem), stream,
                    static_cast<const uint8_t*>(a.k_cache), static_cast<const uint8_t*>(a.v_cache), a.k_exp, a.v_exp,
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
  const long long units = static_cast<long long>(a.B) * a.h_kv * ((a.h / a.h_kv + 7) / 8);
  if (units <= kUnitMost && a.max_blocks <= kUnitBlocks)
    return a.d_h == 128 ? launch_unit<128, 4>(a, stream) : launch_unit<64, 6>(a, stream);
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  e = a.d_h == 128 ? launch_cfg<128, 4>(a, sms, stream)
                   : launch_cfg<64, 6>(a, sms, stream);
  if (e != cudaSuccess) return e;
  const int g = a.h / a.h_kv, n_gb = (g + 7) / 8;
  auto merge = a.d_h == 128 ? decode_runs_merge_kernel<128> : decode_runs_merge_kernel<64>;
  return launch_pdl(merge, dim3(unsigned(a.B) * a.h), dim3(128), 0, stream,
                    static_cast<const float*>(a.o_part), static_cast<const float*>(a.m_part),
                    static_cast<const float*>(a.l_part), static_cast<const long long*>(a.plan), a.h,
                    g, n_gb, a.h_kv * n_gb, static_cast<__nv_bfloat16*>(a.o), a.lse);
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
