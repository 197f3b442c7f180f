// cache_e4m3.cu -- writing new tokens into the 8-bit paged cache and reading
// tokens back from it.
//
// Tokens are packed row after row as in attn_prefill_paged: row b's tokens
// cu[b] .. cu[b+1]-1 are the last of its seq_lens[b] key positions, and
// position p lives in slot p % 16 of page block_table[b][p / 16]. The cache is
// head-major inside a page, [num_blocks, h_kv, 16, d_h] codes and
// [num_blocks, h_kv, 16] exponent bytes, so the keys that one decode CTA reads
// (a page of one KV head) are one run of 16 * d_h bytes.
//
// Both kernels move bytes and compute almost nothing: a group of d_h / 8 lanes
// takes one row (8 numbers a lane: 16 or 32 bytes on the wide side, 8 on the
// code side), the largest magnitude is a shuffle over the group.
#include "common.cuh"
#include "e4m3.cuh"
#include "internal.h"
#include "pdl.cuh"

namespace attn {

static __device__ unsigned int g_cache8_err;

namespace {

using e4m3::kPage;

// Flat slot (page * h_kv + head) * 16 + slot of token t, or -1 where it has
// none: a token before or behind the sequences (silently: padding), one whose
// position lies outside its table row, or one on a page outside the cache
// (both with an error bit; *bad_page tells the latter apart).
struct TokenMap {
  const int32_t* block_table;
  const int32_t* cu;
  const int32_t* seq_lens;
  int B, max_blocks, num_blocks;
};

__device__ __forceinline__ int last_row_at(const TokenMap& m, int t) {
  int lo = 0, hi = m.B;  // rows [0, lo) start at or before t's row
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(m.cu + mid) <= t) lo = mid; else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ bool locate(const TokenMap& m, int t, int* page, int* slot,
                                       bool* bad_page) {
  *bad_page = false;
  const int b = last_row_at(m, t);
  const int end = __ldg(m.cu + b + 1);
  if (t < __ldg(m.cu + b) || t >= end) return false;  // no sequence's token
  const long long pos = static_cast<long long>(__ldg(m.seq_lens + b)) - end + t;
  if (pos < 0 || pos >= static_cast<long long>(m.max_blocks) * kPage) {
    atomicOr(&g_cache8_err, ATTN_DEVERR_BAD_SEQ_LEN);
    return false;
  }
  const int p = __ldg(m.block_table + static_cast<size_t>(b) * m.max_blocks + pos / kPage);
  *slot = static_cast<int>(pos % kPage);
  *page = p;
  if (p < 0 || p >= m.num_blocks) {
    atomicOr(&g_cache8_err, ATTN_DEVERR_BAD_PAGE);
    *bad_page = true;
  }
  return true;
}

template <bool BF16>
__device__ __forceinline__ void load_row8(const void* base, long long off, float (&x)[8]) {
  if constexpr (BF16) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + off));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = bf16lo(w[i]);
      x[2 * i + 1] = bf16hi(w[i]);
    }
  } else {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + off);
    const float4 a = __ldg(p), b = __ldg(p + 1);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
}

struct RowStrides {
  long long tok, head;  // elements
};

// One group of D / 8 lanes quantises U tokens of one head of K or V.
template <int D, bool BF16, int U>
__global__ void __launch_bounds__(256)
    cache_write_kernel(const void* __restrict__ k, const void* __restrict__ v, RowStrides sk,
                       RowStrides sv, TokenMap m, int total, int h_kv, uint8_t* __restrict__ kc,
                       uint8_t* __restrict__ vc, uint8_t* __restrict__ ks,
                       uint8_t* __restrict__ vs) {
  constexpr int L = D / 8;  // lanes per row
  const int sub = threadIdx.x % L;
  const long long gid = (static_cast<long long>(blockIdx.x) * 256 + threadIdx.x) / L;
  const int rows = 2 * h_kv;
  const int t0 = static_cast<int>(gid / rows) * U;
  const int r = static_cast<int>(gid % rows);
  const bool is_v = r >= h_kv;
  const int head = is_v ? r - h_kv : r;
  const void* src = is_v ? v : k;
  const RowStrides st = is_v ? sv : sk;
  uint8_t* codes = is_v ? vc : kc;
  uint8_t* exps = is_v ? vs : ks;
  pdl_wait();
  pdl_trigger();

  float x[U][8];
#pragma unroll
  for (int u = 0; u < U; ++u) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[u][i] = 0.f;
    if (t0 + u < total) load_row8<BF16>(src, (t0 + u) * st.tok + head * st.head + sub * 8, x[u]);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    // Largest finite magnitude over the row, as bits (ordered like the
    // numbers). A NaN or an infinity has no e4m3 code of its own: it is
    // stored as NaN, so that it cannot turn into a finite key, and does not
    // take part in the scale.
    uint32_t a = 0;
    bool odd = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t b = __float_as_uint(x[u][i]) & 0x7fffffffu;
      odd |= b >= 0x7f800000u;
      a = max(a, b >= 0x7f800000u ? 0u : b);
    }
    if (odd) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if ((__float_as_uint(x[u][i]) & 0x7f800000u) == 0x7f800000u)
          x[u][i] = __uint_as_float(0x7fffffffu);
    }
#pragma unroll
    for (int o = 1; o < L; o <<= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
    const uint32_t e = e4m3::scale_byte(a);
    const float inv = e4m3::inv_scale_of(e);
    uint2 w;
    w.x = e4m3::encode2(x[u][0] * inv, x[u][1] * inv) |
          (e4m3::encode2(x[u][2] * inv, x[u][3] * inv) << 16);
    w.y = e4m3::encode2(x[u][4] * inv, x[u][5] * inv) |
          (e4m3::encode2(x[u][6] * inv, x[u][7] * inv) << 16);
    int page, slot;
    bool bad_page;
    if (t0 + u >= total || !locate(m, t0 + u, &page, &slot, &bad_page) || bad_page) continue;
    const size_t row = (static_cast<size_t>(page) * h_kv + head) * kPage + slot;
    if (!ATTN_GUARD(row < static_cast<size_t>(m.num_blocks) * h_kv * kPage, &g_cache8_err)) continue;
    *reinterpret_cast<uint2*>(codes + row * D + sub * 8) = w;
    if (sub == 0) exps[row] = static_cast<uint8_t>(e);
  }
}

// The reverse: one group of D / 8 lanes reads U tokens of one head back.
template <int D, bool BF16, int U>
__global__ void __launch_bounds__(256)
    cache_read_kernel(const uint8_t* __restrict__ kc, const uint8_t* __restrict__ vc,
                      const uint8_t* __restrict__ ks, const uint8_t* __restrict__ vs, TokenMap m,
                      int total, int h_kv, void* __restrict__ k, void* __restrict__ v,
                      RowStrides sk, RowStrides sv) {
  constexpr int L = D / 8;
  const int sub = threadIdx.x % L;
  const long long gid = (static_cast<long long>(blockIdx.x) * 256 + threadIdx.x) / L;
  const int rows = 2 * h_kv;
  const int t0 = static_cast<int>(gid / rows) * U;
  const int r = static_cast<int>(gid % rows);
  const bool is_v = r >= h_kv;
  const int head = is_v ? r - h_kv : r;
  const uint8_t* codes = is_v ? vc : kc;
  const uint8_t* exps = is_v ? vs : ks;
  const RowStrides st = is_v ? sv : sk;
  pdl_wait();
  pdl_trigger();
  uint2 w[U];
  uint32_t e[U];
  bool live[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    int page = 0, slot = 0;
    bool bad_page = false;
    live[u] = t0 + u < total && locate(m, t0 + u, &page, &slot, &bad_page);
    w[u] = make_uint2(0u, 0u);  // a page outside the cache reads as zeros
    e[u] = 127u;
    if (live[u] && !bad_page) {
      const size_t row = (static_cast<size_t>(page) * h_kv + head) * kPage + slot;
      w[u] = __ldg(reinterpret_cast<const uint2*>(codes + row * D + sub * 8));
      e[u] = __ldg(exps + row);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (!live[u]) continue;
    const float sc = e4m3::scale_of(e[u]);
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t c = ((i & 2) ? w[u].y : w[u].x) >> ((i & 1) * 16);
      const uint32_t hh = e4m3::decode2(static_cast<uint16_t>(c & 0xffffu));
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hh));
      x[2 * i] = f.x * sc;
      x[2 * i + 1] = f.y * sc;
    }
    const long long off = (t0 + u) * st.tok + head * st.head + sub * 8;
    void* dst = is_v ? v : k;
    if constexpr (BF16) {
      uint4 y;
      y.x = pack_bf16x2(x[0], x[1]);
      y.y = pack_bf16x2(x[2], x[3]);
      y.z = pack_bf16x2(x[4], x[5]);
      y.w = pack_bf16x2(x[6], x[7]);
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(dst) + off) = y;
    } else {
      float4* p = reinterpret_cast<float4*>(static_cast<float*>(dst) + off);
      p[0] = make_float4(x[0], x[1], x[2], x[3]);
      p[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
  }
}

template <int D, bool BF16, int U>
cudaError_t launch_write_u(const CacheTokens& a, cudaStream_t stream) {
  const long long groups = (static_cast<long long>(a.total) + U - 1) / U * 2 * a.h_kv;
  const long long blocks = (groups * (D / 8) + 255) / 256;
  if (blocks > 0x7fffffffll) return cudaErrorNotSupported;
  const TokenMap m{a.block_table, a.cu, a.seq_lens, a.B, a.max_blocks, a.num_blocks};
  return launch_pdl(cache_write_kernel<D, BF16, U>, dim3(unsigned(blocks)), dim3(256), 0, stream,
                    static_cast<const void*>(a.k), static_cast<const void*>(a.v),
                    RowStrides{a.k_tok, a.k_head}, RowStrides{a.v_tok, a.v_head}, m, a.total,
                    a.h_kv, a.k_codes, a.v_codes, a.k_exp, a.v_exp);
}

template <int D, bool BF16, int U>
cudaError_t launch_read_u(const CacheTokens& a, cudaStream_t stream) {
  const long long groups = (static_cast<long long>(a.total) + U - 1) / U * 2 * a.h_kv;
  const long long blocks = (groups * (D / 8) + 255) / 256;
  if (blocks > 0x7fffffffll) return cudaErrorNotSupported;
  const TokenMap m{a.block_table, a.cu, a.seq_lens, a.B, a.max_blocks, a.num_blocks};
  return launch_pdl(cache_read_kernel<D, BF16, U>, dim3(unsigned(blocks)), dim3(256), 0, stream,
                    static_cast<const uint8_t*>(a.k_codes), static_cast<const uint8_t*>(a.v_codes),
                    static_cast<const uint8_t*>(a.k_exp), static_cast<const uint8_t*>(a.v_exp), m,
                    a.total, a.h_kv, a.k, a.v, RowStrides{a.k_tok, a.k_head},
                    RowStrides{a.v_tok, a.v_head});
}

}  // namespace

cudaError_t launch_cache_write(const CacheTokens& a, cudaStream_t stream) {
  const bool bf = a.dtype == ATTN_DTYPE_BF16;
  if (a.d_h == 128)
    return bf ? launch_write_u<128, true, 4>(a, stream) : launch_write_u<128, false, 4>(a, stream);
  return bf ? launch_write_u<64, true, 4>(a, stream) : launch_write_u<64, false, 4>(a, stream);
}

cudaError_t launch_cache_read(const CacheTokens& a, cudaStream_t stream) {
  const bool bf = a.dtype == ATTN_DTYPE_BF16;
  if (a.d_h == 128)
    return bf ? launch_read_u<128, true, 4>(a, stream) : launch_read_u<128, false, 4>(a, stream);
  return bf ? launch_read_u<64, true, 4>(a, stream) : launch_read_u<64, false, 4>(a, stream);
}

unsigned int cache8_read_and_clear_error(cudaStream_t stream, cudaError_t* st) {
  unsigned int v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(&v, g_cache8_err, sizeof(v), 0,
                                            cudaMemcpyDeviceToHost, stream);
  if (e == cudaSuccess)
    e = cudaMemcpyToSymbolAsync(g_cache8_err, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice,
                                stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
  if (st) *st = e;
  return v;
}

}  // namespace attn
