// cache_kernels.cu — the paged key/value cache: new tokens' keys and values
// written into it (copied, or quantised row by row) and rows read back as bf16.
//
// Layout: pages [P, H_kv, page, d] of bf16, E4M3 or int8 elements, and for the
// 8-bit kinds one fp32 scale per row of a page and head, [P, H_kv, page]. A
// sequence's position p lies in slot p % page of page table[s, p / page].
//
// Quantisation of a row x of d values (per token and head, so a row written
// today never changes an earlier one): amax = max |x|, a = max(amax,
// M 2^-126), scale = a / M, r = M / a with M = 448 (E4M3) or 127 (int8), both 1
// for a zero row; code = x * r rounded to fp32, then to the code's type, ties
// to even. The bound on a keeps r finite and the scale normal.
//
// Both kernels only move data, and are bound by the memory. A block takes some
// tokens and up to 128 heads of them, about 128 rows: its first warp finds the
// sequence, page and slot of each token (a 32-way search over the offsets and two
// dependent loads, once for all of a token's rows), then d / 8 threads hold a row of
// K and one of V, 16 bytes each on the bf16 side, with four rows' loads in flight.
// Writing 22,640 tokens of 8 heads as E4M3 (d = 128, 140 MB moved) takes 35 us, reading
// 25,740 (159 MB) 32 us.
#include <algorithm>
#include <type_traits>

#include "sa_internal.h"

namespace sa {

namespace cache {
constexpr int kThreads = 256;
}

// Largest s in [0, n] with off[s] <= t for ascending off[0 .. n] and off[0] <= t
// (0 if even off[0] > t): 32 probes a round by the lanes of a warp. All lanes
// of the warp take part and get the result.
__device__ __forceinline__ int find_segment(const int* __restrict__ off, int n, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = n;   // the result lies in [lo, hi]
  while (lo < hi) {
    const int step = (hi - lo + 31) >> 5;
    const int probe = lo + (lane + 1) * step;
    const bool le = probe <= hi && __ldg(off + min(probe, hi)) <= t;
    const int c = __popc(__ballot_sync(0xFFFFFFFFu, le));   // probes 1..c hold (ascending offsets)
    const int nlo = lo + c * step;
    hi = min(hi, nlo + step - 1);
    lo = min(nlo, hi);
  }
  return lo;
}

// Element sizes and value bounds of the cache kinds.
template <int KIND>
struct CacheKind {
  static constexpr int ES = KIND == kCacheBf16 ? 2 : 1;
  static constexpr float M = KIND == kCacheE4m3 ? 448.f : 127.f;
};

// 8 bf16 values as floats.
__device__ __forceinline__ void unpack8(const uint4 w, float (&x)[8]) {
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x[2 * j] = __uint_as_float(v[j] << 16);
    x[2 * j + 1] = __uint_as_float(v[j] & 0xFFFF0000u);
  }
}

template <int KIND>
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float r) {
  uint32_t c[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float a = x[2 * j] * r, b = x[2 * j + 1] * r;
    if constexpr (KIND == kCacheE4m3) {
      c[j] = pack_e4m3x2(a, b);
    } else {
      const int ia = max(-127, min(127, __float2int_rn(a))), ib = max(-127, min(127, __float2int_rn(b)));
      c[j] = (ia & 0xFF) | ((ib & 0xFF) << 8);
    }
  }
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// The 8 values of 8 codes, times the row's scale.
template <int KIND>
__device__ __forceinline__ void decode8(const uint2 w, float s, float (&x)[8]) {
  const uint32_t v[2] = {w.x, w.y};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t b = (v[j >> 2] >> (8 * (j & 3))) & 0xFF;
    if constexpr (KIND == kCacheE4m3) {
      const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(b), __NV_E4M3);
      x[j] = __half2float(__half(h)) * s;
    } else {
      x[j] = static_cast<float>(static_cast<int8_t>(b)) * s;
    }
  }
}

// Where the tokens t0 .. t0 + n - 1 lie: page * H * page size + slot of each in `at`
// (the row of head h is h * page size further), or -1 where the token has no sequence,
// -2 where it has one but its position has no slot (before 0, behind the
// table, or in an entry outside the cache). By the lanes of one warp.
template <bool WRITE>
__device__ __forceinline__ void resolve(const CacheArgs& a, int t0, int n, long long* at) {
  int s = find_segment(a.off, a.n_seqs, t0);
  const int lane = threadIdx.x & 31, t = t0 + lane;
  if (lane >= n) return;
  long long r = -1;
  if (t < a.n_rows && t >= __ldg(a.off)) {
    while (s < a.n_seqs && __ldg(a.off + s + 1) <= t) ++s;
    if (s < a.n_seqs) {
      // written tokens are their sequence's last ones; rows read start at its first position
      // (of the length clamped to [0, the table's positions], as the attention counts them)
      const int full = a.width * a.page;
      const int pos = WRITE ? min(max(__ldg(a.len + s), 0), full) - (min(__ldg(a.off + s + 1), a.n_rows) - t) : t - __ldg(a.off + s);
      r = -2;
      if (pos >= 0 && pos < full) {
        const int pg = __ldg(a.table + static_cast<long long>(s) * a.width + pos / a.page);
        if (pg >= 0 && pg < a.n_pages) r = static_cast<long long>(pg) * a.H * a.page + pos % a.page;
      }
    }
  }
  at[lane] = r;
}

// The larger magnitudes of two pairs of bf16, NaN if one is: a row with a NaN gets a
// scale of NaN and is read as NaN, whatever its codes.
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a & 0x7FFF7FFFu), "r"(b & 0x7FFF7FFFu));
  return r;
}

// Largest magnitudes of a thread's 8 values of K and of V, over the TPR threads of
// the row (neighbours in a warp).
template <int TPR>
__device__ __forceinline__ void row_amax(const uint4 k, const uint4 v, float& ka, float& va) {
  const uint32_t k2 = max_abs2(max_abs2(k.x, k.y), max_abs2(k.z, k.w)), v2 = max_abs2(max_abs2(v.x, v.y), max_abs2(v.z, v.w));
  // one pair of both: K's in the low half
  uint32_t m = max_abs2(__byte_perm(k2, v2, 0x5410), __byte_perm(k2, v2, 0x7632));
#pragma unroll
  for (int o = TPR / 2; o > 0; o >>= 1) m = max_abs2(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  ka = __uint_as_float(m << 16);
  va = __uint_as_float(m & 0xFFFF0000u);
}

template <int D, int KIND>
__global__ void __launch_bounds__(cache::kThreads) cache_write_kernel(const __grid_constant__ CacheArgs a, int toks, int heads) {
  constexpr int TPR = D / 8;                         // threads per row
  constexpr int RPP = cache::kThreads / TPR;         // rows a pass
  constexpr int U = 4;
  __shared__ long long at[32];
  const int t0 = blockIdx.x * toks, h0 = blockIdx.y * heads, nh = min(heads, a.H - h0), c = threadIdx.x % TPR;
  if (threadIdx.x < 32) resolve<true>(a, t0, toks, at);
  __syncthreads();
  const int rows = toks * nh;
  for (int r0 = threadIdx.x / TPR; r0 - threadIdx.x / TPR < rows; r0 += U * RPP) {
    uint4 kw[U], vw[U];
    long long dst[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * RPP, i = r / nh, h = h0 + r - i * nh;
      dst[u] = -1;
      kw[u] = vw[u] = make_uint4(0, 0, 0, 0);
      if (r < rows && at[i] >= 0) {
        const long long t = t0 + i;
        dst[u] = at[i] + static_cast<long long>(h) * a.page;
        kw[u] = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.k) + t * a.k_st + h * a.k_sh + 8 * c));
        vw[u] = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.v) + t * a.v_st + h * a.v_sh + 8 * c));
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if constexpr (KIND == kCacheBf16) {
        if (dst[u] >= 0) {
          reinterpret_cast<uint4*>(a.k_cache)[dst[u] * TPR + c] = kw[u];
          reinterpret_cast<uint4*>(a.v_cache)[dst[u] * TPR + c] = vw[u];
        }
      } else {
        constexpr float M = CacheKind<KIND>::M;
        constexpr float kTiny = M * 1.17549435e-38f;   // M 2^-126
        float ka, va, kx[8], vx[8];
        row_amax<TPR>(kw[u], vw[u], ka, va);
        if (dst[u] < 0) continue;
        const float kb = fmax_nan(ka, kTiny), vb = fmax_nan(va, kTiny);
        const float kr = ka != 0.f ? M / kb : 1.f, vr = va != 0.f ? M / vb : 1.f;
        unpack8(kw[u], kx);
        unpack8(vw[u], vx);
        reinterpret_cast<uint2*>(a.k_cache)[dst[u] * TPR + c] = encode8<KIND>(kx, kr);
        reinterpret_cast<uint2*>(a.v_cache)[dst[u] * TPR + c] = encode8<KIND>(vx, vr);
        if (c == 0) {
          a.k_scale[dst[u]] = ka != 0.f ? kb / M : 1.f;
          a.v_scale[dst[u]] = va != 0.f ? vb / M : 1.f;
        }
      }
    }
  }
}

template <int D, int KIND>
__global__ void __launch_bounds__(cache::kThreads) cache_read_kernel(const __grid_constant__ CacheArgs a, int toks, int heads) {
  constexpr int TPR = D / 8;
  constexpr int RPP = cache::kThreads / TPR;
  constexpr int U = 4;
  __shared__ long long at[32];
  const int t0 = blockIdx.x * toks, h0 = blockIdx.y * heads, nh = min(heads, a.H - h0), c = threadIdx.x % TPR;
  if (threadIdx.x < 32) resolve<false>(a, t0, toks, at);
  __syncthreads();
  const int rows = toks * nh;
  using W = typename std::conditional<KIND == kCacheBf16, uint4, uint2>::type;
  for (int r0 = threadIdx.x / TPR; r0 < rows; r0 += U * RPP) {
    W kc[U], vc[U];
    float ks[U], vs[U];
    long long src[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * RPP, i = r / nh, h = h0 + r - i * nh;
      src[u] = -1;
      kc[u] = vc[u] = W{};             // a position without a slot reads as zeros
      ks[u] = vs[u] = 0.f;
      if (r < rows) {
        src[u] = at[i];
        if (src[u] >= 0) {
          const long long at_row = src[u] + static_cast<long long>(h) * a.page;
          kc[u] = __ldg(reinterpret_cast<const W*>(a.k_cache) + at_row * TPR + c);
          vc[u] = __ldg(reinterpret_cast<const W*>(a.v_cache) + at_row * TPR + c);
          if constexpr (KIND != kCacheBf16) {
            ks[u] = __ldg(a.k_scale + at_row);
            vs[u] = __ldg(a.v_scale + at_row);
          }
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * RPP, i = r / nh, h = h0 + r - i * nh;
      if (r >= rows || src[u] == -1) continue;
      const long long t = t0 + i;
      uint4 kw, vw;
      if constexpr (KIND == kCacheBf16) {
        kw = kc[u];
        vw = vc[u];
      } else {
        float x[8];
        decode8<KIND>(kc[u], ks[u], x);
        kw = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
        decode8<KIND>(vc[u], vs[u], x);
        vw = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
      }
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.k_out) + t * a.k_st + h * a.k_sh + 8 * c) = kw;
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.v_out) + t * a.v_st + h * a.v_sh + 8 * c) = vw;
    }
  }
}

template <int D, int KIND>
static cudaError_t launch_cache_d(const CacheArgs& a, bool write, cudaStream_t st) {
  if (a.n_rows == 0) return cudaSuccess;
  // about 128 rows a block; fewer where the call would not give every SM a block
  const int heads = std::min(a.H, 128);
  int toks = std::max(1, std::min(32, 128 / heads));
  toks = std::min<long long>(toks, std::max<long long>(1, static_cast<long long>(a.n_rows) * ceil_div(a.H, heads) / sm_count_cached()));
  const dim3 grid(ceil_div(a.n_rows, toks), ceil_div(a.H, heads));
  if (write) cache_write_kernel<D, KIND><<<grid, cache::kThreads, 0, st>>>(a, toks, heads);
  else cache_read_kernel<D, KIND><<<grid, cache::kThreads, 0, st>>>(a, toks, heads);
  return cudaGetLastError();
}

cudaError_t launch_cache(const CacheArgs& a, int d, int kind, bool write, cudaStream_t st) {
  if (d == 64) {
    if (kind == kCacheBf16) return launch_cache_d<64, kCacheBf16>(a, write, st);
    if (kind == kCacheE4m3) return launch_cache_d<64, kCacheE4m3>(a, write, st);
    return launch_cache_d<64, kCacheInt8>(a, write, st);
  }
  if (kind == kCacheBf16) return launch_cache_d<128, kCacheBf16>(a, write, st);
  if (kind == kCacheE4m3) return launch_cache_d<128, kCacheE4m3>(a, write, st);
  return launch_cache_d<128, kCacheInt8>(a, write, st);
}

}  // namespace sa
