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
// Both kernels move bytes and compute little: what bounds them is the bytes in
// flight and, once those are there, the instructions per value. A group of
// d_h / 16 lanes takes one row (one token of one head of K or V), two 8-number
// chunks a lane d_h / 2 numbers apart, so that every load and store of a warp is
// contiguous; the largest magnitude is a shuffle over the group. A thread has U
// rows in flight. Rows are ordered (block of 16 tokens, K heads then V heads,
// token): neighbouring groups then write (read) neighbouring slots of one page
// and head, runs of 16 * d_h bytes with their exponents, while the tensors'
// side comes in whole rows of 128 bytes or more. A CTA's first warp looks its
// tokens up (cu, lengths, block table) while the others' loads are under way. Both
// sides' inputs are read once and marked so (streaming loads took 7% off the write
// of 8192 tokens, now 9.7 us a call, and 4% off the read of 32768, 33.6).
//
// Both kernels may become resident while the kernel in front still writes what
// they read, so that none of it is constant for their lifetime: nothing is read
// before pdl_wait, and no load is a non-coherent one. Offsets, lengths, table and
// exponents come from L2.
#include "common.cuh"
#include "e4m3.cuh"
#include "internal.h"
#include "pdl.cuh"

namespace attn {

static __device__ unsigned int g_cache8_err;

namespace {

using e4m3::kPage;

struct TokenMap {
  const int32_t* block_table;
  const int32_t* cu;
  const int32_t* seq_lens;
  int B, max_blocks, num_blocks;
};

// Offsets and lengths of 32 rows from `lo` on, one per lane; a token's row is
// among them or behind them. Everything of the lookup comes from L2, so round
// trips count: these are one, the table another (each lane searching its row for
// itself took 31.9 us for the write of 24 ragged rows, 33000 tokens of 64 in fp32,
// this way 24.3). Beyond 32 rows it is one more for each factor of 32.
struct NearRows {
  int lo, cu, len;
};
__device__ __forceinline__ NearRows near_rows(const TokenMap& m, int t0) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = m.B;  // t0's row is one of [lo, lo + n)
  while (n > 32) {
    const int step = (n + 31) >> 5, i = lane * step;
    const bool le = lane == 0 || (i < n && __ldcg(m.cu + lo + i) <= t0);
    const int k = __ffs(~__ballot_sync(0xffffffffu, le));  // lanes 0 .. k - 2, or all (0)
    const int at = ((k == 0 ? 33 : k) - 2) * step;
    lo += at;
    n = min(step, n - at);
  }
  NearRows x;
  x.lo = lo;
  x.cu = lo + lane <= m.B ? __ldcg(m.cu + lo + lane) : 0x7fffffff;
  x.len = lo + lane < m.B ? __ldcg(m.seq_lens + lo + lane) : 0;
  return x;
}

// Page and slot of token t, false where it has none: a token before or behind the
// sequences (silently: padding) or one whose position lies outside its table row.
// One on a page outside the cache has a slot, and *bad_page (both of these with an
// error bit). By a whole warp, each lane with a token at or behind x's.
__device__ __forceinline__ bool locate(const TokenMap& m, const NearRows& x, int t, int* page,
                                       int* slot, bool* bad_page) {
  *bad_page = false;
  int r = 0;  // the last of the 32 rows that starts at or before t
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) {
    if (s >= m.B) continue;
    const int v = __shfl_sync(0xffffffffu, x.cu, r + s);
    if (x.lo + r + s < m.B && v <= t) r += s;
  }
  int begin = __shfl_sync(0xffffffffu, x.cu, r), end = __shfl_sync(0xffffffffu, x.cu, (r + 1) & 31);
  int len = __shfl_sync(0xffffffffu, x.len, r), b = x.lo + r;
  if (r == 31) {  // its end, or its row, lies behind them (empty rows between the tokens)
    int hi = m.B;
    while (hi - b > 1) {
      const int mid = b + ((hi - b) >> 1);
      if (__ldcg(m.cu + mid) <= t) b = mid; else hi = mid;
    }
    begin = __ldcg(m.cu + b);
    end = __ldcg(m.cu + b + 1);
    len = __ldcg(m.seq_lens + b);
  }
  const long long pos = static_cast<long long>(len) - end + t;
  if (t < begin || t >= end) return false;  // no sequence's token
  if (pos < 0 || pos >= static_cast<long long>(m.max_blocks) * kPage) {
    atomicOr(&g_cache8_err, ATTN_DEVERR_BAD_SEQ_LEN);
    return false;
  }
  const int p = __ldcg(m.block_table + static_cast<size_t>(b) * m.max_blocks + pos / kPage);
  *slot = static_cast<int>(pos % kPage);
  *page = p;
  if (p < 0 || p >= m.num_blocks) {
    atomicOr(&g_cache8_err, ATTN_DEVERR_BAD_PAGE);
    *bad_page = true;
  }
  return true;
}

struct RowStrides {
  long long tok, head;  // elements
};

// Place of a CTA's tokens: page and slot; page -1: no place, -2: a page outside
// the cache.
constexpr int kBlk = 16;  // tokens per block
// Threads per CTA and rows in flight per thread. Write of 8192 tokens (bf16, 8
// heads of 128), us a call: 64 and 2 10.3, 128 and 2 9.7, 256 and 2 10.6. Read of
// 32768: 64 and 2 34.6, 128 and 2 33.6, 256 and 2 35.8; 4 rows no faster (and
// 40 rows of heads of 64 read in fp32 22.0, else 20.9).
constexpr int kWriteThreads = 128, kReadThreads = 128, kU = 2;

// A CTA's rows lie in one block of 16 tokens: grid (parts of a block, blocks in y
// and z), so that no index needs a division (with rows numbered through and
// divided by a block's, the write of 8192 tokens took 10.9 us, else 10.2).
template <int D, int U, int T>
struct Cta {
  static constexpr int L = D / 16;         // lanes per row
  static constexpr int G = T / L;   // rows at a time
  static constexpr int ROWS = U * G;       // rows per CTA
  static_assert(ROWS % kBlk == 0, "whole heads");
};

__device__ __forceinline__ long long block_of() {
  return static_cast<long long>(blockIdx.z) * gridDim.y + blockIdx.y;
}

// Both by a CTA's first warp: the lookup's first loads, and what is left of it.
__device__ __forceinline__ NearRows tokens_near(const TokenMap& m, int total) {
  const long long t0 = block_of() * kBlk;
  return threadIdx.x < 32 && t0 < total ? near_rows(m, static_cast<int>(t0)) : NearRows{0, 0, 0};
}
__device__ __forceinline__ void locate_tokens(const TokenMap& m, const NearRows& x, int total,
                                              int* s_page, int* s_slot) {
  const long long t0 = block_of() * kBlk;
  if (threadIdx.x >= 32 || t0 >= total) return;
  // Lanes without a token of their own have the last one's place.
  const int i = min(static_cast<int>(threadIdx.x), min(kBlk, static_cast<int>(total - t0)) - 1);
  int page = -1, slot = 0;
  bool bad_page = false;
  if (!locate(m, x, static_cast<int>(t0) + i, &page, &slot, &bad_page)) page = -1;
  s_page[i] = bad_page ? -2 : page;  // (lanes of one token write the same)
  s_slot[i] = slot;
}

// Row `it` of a CTA's rows: its token, that token's index within the CTA, head,
// K or V.
struct RowId {
  long long t;
  int ti, head;
  bool is_v, live;
};
template <int D, int U, int T>
__device__ __forceinline__ RowId row_id(int it, int total, int h_kv) {
  RowId x;
  x.ti = it % kBlk;
  x.t = block_of() * kBlk + x.ti;
  x.head = static_cast<int>(blockIdx.x) * (Cta<D, U, T>::ROWS / kBlk) + it / kBlk;
  x.is_v = x.head >= h_kv;
  if (x.is_v) x.head -= h_kv;
  x.live = x.t < total && x.head < h_kv;
  return x;
}

// 16 numbers of a row (two chunks) as loaded.
template <bool BF16>
struct Raw {
  uint4 w[BF16 ? 2 : 4];
};

// Codes of chunk c of a lane's numbers, times 2^-e. Exact in bf16 too, whose
// exponents are fp32's.
template <bool BF16>
__device__ __forceinline__ uint2 encode8(const Raw<BF16>& r, int c, uint32_t e) {
  uint32_t y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF16) {
      const uint32_t w[4] = {r.w[c].x, r.w[c].y, r.w[c].z, r.w[c].w};
      const uint32_t inv = (254u - e) * 0x00800080u;  // 2^-e twice
      const __nv_bfloat162 p = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]),
                                       *reinterpret_cast<const __nv_bfloat162*>(&inv));
      const uint32_t u = *reinterpret_cast<const uint32_t*>(&p);
      y[i] = e4m3::encode2(bf16lo(u), bf16hi(u));
    } else {
      const uint4 q = r.w[2 * c + (i >> 1)];
      const float inv = e4m3::inv_scale_of(e);
      y[i] = e4m3::encode2(__uint_as_float(i & 1 ? q.z : q.x) * inv, __uint_as_float(i & 1 ? q.w : q.y) * inv);
    }
  }
  return make_uint2(y[0] | (y[1] << 16), y[2] | (y[3] << 16));
}

// fp32 bits of the largest magnitude among a lane's 16 numbers (NaN and
// infinities count, as the largest).
template <bool BF16>
__device__ __forceinline__ uint32_t max_bits(const Raw<BF16>& r) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < (BF16 ? 2 : 4); ++i) {
    const uint32_t w[4] = {r.w[i].x, r.w[i].y, r.w[i].z, r.w[i].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (BF16)
        asm("max.u16x2 %0, %0, %1;" : "+r"(m) : "r"(w[k] & 0x7fff7fffu));
      else
        m = max(m, w[k] & 0x7fffffffu);
    }
  }
  return BF16 ? max(m & 0xffffu, m >> 16) << 16 : m;
}

template <int D, bool BF16, int U>
__global__ void __launch_bounds__(kWriteThreads)
    cache_write_kernel(const void* k, const void* v, RowStrides sk, RowStrides sv, TokenMap m,
                       int total, int h_kv, uint8_t* __restrict__ kc, uint8_t* __restrict__ vc,
                       uint8_t* __restrict__ ks, uint8_t* __restrict__ vs) {
  constexpr int T = kWriteThreads;
  using C = Cta<D, U, T>;
  __shared__ int s_page[kBlk], s_slot[kBlk];
  const int sub = threadIdx.x % C::L, grp = threadIdx.x / C::L;
  pdl_wait();
  pdl_trigger();

  Raw<BF16> x[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const RowId id = row_id<D, U, T>(u * C::G + grp, total, h_kv);
    if (id.live) {
      const RowStrides st = id.is_v ? sv : sk;
      const long long off = id.t * st.tok + id.head * st.head + sub * 8;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        if constexpr (BF16) {
          x[u].w[c] = __ldcs(reinterpret_cast<const uint4*>(
              static_cast<const __nv_bfloat16*>(id.is_v ? v : k) + off + c * (D / 2)));
        } else {
          const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(id.is_v ? v : k) +
                                                          off + c * (D / 2));
          x[u].w[2 * c] = __ldcs(p);
          x[u].w[2 * c + 1] = __ldcs(p + 1);
        }
      }
    } else {
#pragma unroll
      for (int c = 0; c < (BF16 ? 2 : 4); ++c) x[u].w[c] = make_uint4(0u, 0u, 0u, 0u);
    }
  }
  locate_tokens(m, tokens_near(m, total), total, s_page, s_slot);
  __syncthreads();
#pragma unroll
  for (int u = 0; u < U; ++u) {
    uint32_t a = max_bits<BF16>(x[u]);
#pragma unroll
    for (int o = 1; o < C::L; o <<= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
    if (__any_sync(0xffffffffu, a >= 0x7f800000u)) {
      // A NaN or an infinity has no e4m3 code of its own: it is stored as NaN,
      // so that it cannot turn into a finite key, and has no part in the scale.
      a = 0;
#pragma unroll
      for (int c = 0; c < (BF16 ? 2 : 4); ++c) {
        uint32_t* const w[4] = {&x[u].w[c].x, &x[u].w[c].y, &x[u].w[c].z, &x[u].w[c].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (BF16) {
#pragma unroll
            for (int s = 0; s < 32; s += 16) {
              const uint32_t b = (*w[i] >> s) & 0x7fffu;
              if (b >= 0x7f80u)
                *w[i] |= 0x7fffu << s;
              else
                a = max(a, b << 16);
            }
          } else {
            const uint32_t b = *w[i] & 0x7fffffffu;
            if (b >= 0x7f800000u)
              *w[i] |= 0x7fffffffu;
            else
              a = max(a, b);
          }
        }
      }
#pragma unroll
      for (int o = 1; o < C::L; o <<= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
    }
    const uint32_t e = e4m3::scale_byte(a);
    const RowId id = row_id<D, U, T>(u * C::G + grp, total, h_kv);
    if (!id.live || s_page[id.ti] < 0) continue;
    const size_t row =
        (static_cast<size_t>(s_page[id.ti]) * h_kv + id.head) * kPage + s_slot[id.ti];
    if (!ATTN_GUARD(row < static_cast<size_t>(m.num_blocks) * h_kv * kPage, &g_cache8_err)) continue;
    uint8_t* dst = (id.is_v ? vc : kc) + row * D + sub * 8;
    *reinterpret_cast<uint2*>(dst) = encode8<BF16>(x[u], 0, e);
    *reinterpret_cast<uint2*>(dst + D / 2) = encode8<BF16>(x[u], 1, e);
    if (sub == 0) (id.is_v ? vs : ks)[row] = static_cast<uint8_t>(e);
  }
}

// The reverse. fp32 results: four chunks of 4 numbers a lane, so that each store
// of a warp fills its sectors (two halves of a sector in two stores took 28.1 us
// for 86 MB of them, 40 rows of up to 1999 tokens).
template <int D, bool BF16, int U>
__global__ void __launch_bounds__(kReadThreads)
    cache_read_kernel(const uint8_t* kc, const uint8_t* vc, const uint8_t* ks, const uint8_t* vs,
                      TokenMap m, int total, int h_kv, void* __restrict__ k, void* __restrict__ v,
                      RowStrides sk, RowStrides sv) {
  constexpr int T = kReadThreads;
  using C = Cta<D, U, T>;
  __shared__ int s_page[kBlk], s_slot[kBlk];
  const int sub = threadIdx.x % C::L, grp = threadIdx.x / C::L;
  pdl_wait();
  pdl_trigger();
  locate_tokens(m, tokens_near(m, total), total, s_page, s_slot);
  __syncthreads();
  uint32_t w[U][4];  // codes: two chunks of 8, or four of 4
  uint32_t e[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const RowId id = row_id<D, U, T>(u * C::G + grp, total, h_kv);
    w[u][0] = w[u][1] = w[u][2] = w[u][3] = 0u;  // a page outside the cache reads as zeros
    e[u] = 127u;
    if (id.live && s_page[id.ti] >= 0) {
      const size_t row =
          (static_cast<size_t>(s_page[id.ti]) * h_kv + id.head) * kPage + s_slot[id.ti];
      const uint8_t* src = (id.is_v ? vc : kc) + row * D + sub * (BF16 ? 8 : 4);
      if constexpr (BF16) {
        const uint2 a = __ldcs(reinterpret_cast<const uint2*>(src));
        const uint2 b = __ldcs(reinterpret_cast<const uint2*>(src + D / 2));
        w[u][0] = a.x; w[u][1] = a.y; w[u][2] = b.x; w[u][3] = b.y;
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) w[u][c] = __ldcs(reinterpret_cast<const uint32_t*>(src + c * (D / 4)));
      }
      e[u] = __ldcg((id.is_v ? vs : ks) + row);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const RowId id = row_id<D, U, T>(u * C::G + grp, total, h_kv);
    if (!id.live || s_page[id.ti] == -1) continue;
    if (!ATTN_GUARD(id.t < total && id.head < h_kv && id.ti < kBlk, &g_cache8_err)) continue;
    const float sc = e4m3::scale_of(e[u]);
    const RowStrides st = id.is_v ? sv : sk;
    const long long off = id.t * st.tok + id.head * st.head + sub * (BF16 ? 8 : 4);
    float x[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t hh = e4m3::decode2(static_cast<uint16_t>(w[u][i >> 1] >> ((i & 1) * 16)));
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hh));
      x[2 * i] = f.x * sc;
      x[2 * i + 1] = f.y * sc;
    }
    if constexpr (BF16) {
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(id.is_v ? v : k) + off;
#pragma unroll
      for (int c = 0; c < 2; ++c)
        *reinterpret_cast<uint4*>(dst + c * (D / 2)) =
            make_uint4(pack_bf16x2(x[8 * c], x[8 * c + 1]), pack_bf16x2(x[8 * c + 2], x[8 * c + 3]),
                       pack_bf16x2(x[8 * c + 4], x[8 * c + 5]), pack_bf16x2(x[8 * c + 6], x[8 * c + 7]));
    } else {
      float* dst = static_cast<float*>(id.is_v ? v : k) + off;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        *reinterpret_cast<float4*>(dst + c * (D / 4)) =
            make_float4(x[4 * c], x[4 * c + 1], x[4 * c + 2], x[4 * c + 3]);
    }
  }
}

template <int D, int U, int T>
dim3 grid_of(const CacheTokens& a) {
  constexpr int kHeads = Cta<D, U, T>::ROWS / kBlk;  // per CTA, K and V counted apart
  const long long blocks = (static_cast<long long>(a.total) + kBlk - 1) / kBlk;
  const unsigned y = static_cast<unsigned>(blocks < 65535 ? blocks : 65535);
  return dim3(unsigned((2 * a.h_kv + kHeads - 1) / kHeads), y, unsigned((blocks + y - 1) / y));
}

template <int D, bool BF16, int U>
cudaError_t launch_write_u(const CacheTokens& a, cudaStream_t stream) {
  const TokenMap m{a.block_table, a.cu, a.seq_lens, a.B, a.max_blocks, a.num_blocks};
  return launch_pdl(cache_write_kernel<D, BF16, U>, grid_of<D, U, kWriteThreads>(a), dim3(kWriteThreads), 0, stream,
                    static_cast<const void*>(a.k), static_cast<const void*>(a.v),
                    RowStrides{a.k_tok, a.k_head}, RowStrides{a.v_tok, a.v_head}, m, a.total,
                    a.h_kv, a.k_codes, a.v_codes, a.k_exp, a.v_exp);
}

template <int D, bool BF16, int U>
cudaError_t launch_read_u(const CacheTokens& a, cudaStream_t stream) {
  const TokenMap m{a.block_table, a.cu, a.seq_lens, a.B, a.max_blocks, a.num_blocks};
  return launch_pdl(cache_read_kernel<D, BF16, U>, grid_of<D, U, kReadThreads>(a), dim3(kReadThreads), 0, stream,
                    static_cast<const uint8_t*>(a.k_codes), static_cast<const uint8_t*>(a.v_codes),
                    static_cast<const uint8_t*>(a.k_exp), static_cast<const uint8_t*>(a.v_exp), m,
                    a.total, a.h_kv, a.k, a.v, RowStrides{a.k_tok, a.k_head},
                    RowStrides{a.v_tok, a.v_head});
}

}  // namespace

cudaError_t launch_cache_write(const CacheTokens& a, cudaStream_t stream) {
  const bool bf = a.dtype == ATTN_DTYPE_BF16;
  if (a.d_h == 128)
    return bf ? launch_write_u<128, true, kU>(a, stream) : launch_write_u<128, false, kU>(a, stream);
  return bf ? launch_write_u<64, true, kU>(a, stream) : launch_write_u<64, false, kU>(a, stream);
}

cudaError_t launch_cache_read(const CacheTokens& a, cudaStream_t stream) {
  const bool bf = a.dtype == ATTN_DTYPE_BF16;
  if (a.d_h == 128)
    return bf ? launch_read_u<128, true, kU>(a, stream) : launch_read_u<128, false, kU>(a, stream);
  return bf ? launch_read_u<64, true, kU>(a, stream) : launch_read_u<64, false, kU>(a, stream);
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
