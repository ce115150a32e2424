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
// Both kernels only move data: a thread holds 8 elements (one 16-byte access
// on the bf16 side) of a row of K and of V, d / 8 threads a row, rows in (token,
// head) order. A block finds the sequence of its first token by a 32-way search
// over the offsets and its threads step on from there.
#include <algorithm>

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

// The larger of two numbers, NaN if one is: a row with a NaN gets a scale of NaN
// and is read as NaN, whatever its codes.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
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

// Row (page * H + head) * page_size + slot of a position, or -1 where the
// position has no slot (before 0, behind the table, or in an entry outside the
// cache).
__device__ __forceinline__ long long cache_row(const CacheArgs& a, int s, int pos, int h) {
  if (pos < 0 || pos >= a.width * static_cast<long long>(a.page)) return -1;
  const int pg = __ldg(a.table + static_cast<long long>(s) * a.width + pos / a.page);
  if (pg < 0 || pg >= a.n_pages) return -1;
  return (static_cast<long long>(pg) * a.H + h) * a.page + pos % a.page;
}

template <int D, int KIND>
__global__ void __launch_bounds__(cache::kThreads) cache_write_kernel(const __grid_constant__ CacheArgs a) {
  constexpr int TPR = D / 8;                         // threads per row
  constexpr int RPB = cache::kThreads / TPR;         // rows per block
  const long long row = static_cast<long long>(blockIdx.x) * RPB + threadIdx.x / TPR;
  const int c = threadIdx.x % TPR;
  const int t0 = static_cast<int>(static_cast<long long>(blockIdx.x) * RPB / a.H);
  int s = find_segment(a.off, a.n_seqs, t0);
  const int t = static_cast<int>(row / a.H), h = static_cast<int>(row % a.H);
  const bool in = t < a.n_rows && t >= __ldg(a.off);
  if (in)
    while (s < a.n_seqs && __ldg(a.off + s + 1) <= t) ++s;
  long long dst = -1;
  if (in && s < a.n_seqs) {
    const int left = min(__ldg(a.off + s + 1), a.n_rows) - t;   // this token and those behind it
    dst = cache_row(a, s, __ldg(a.len + s) - left, h);
  }
  uint4 kw = make_uint4(0, 0, 0, 0), vw = kw;
  if (dst >= 0) {
    kw = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.k) + t * a.k_st + h * a.k_sh + 8 * c));
    vw = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.v) + t * a.v_st + h * a.v_sh + 8 * c));
  }
  if constexpr (KIND == kCacheBf16) {
    if (dst >= 0) {
      reinterpret_cast<uint4*>(a.k_cache)[dst * TPR + c] = kw;
      reinterpret_cast<uint4*>(a.v_cache)[dst * TPR + c] = vw;
    }
  } else {
    constexpr float M = CacheKind<KIND>::M;
    float kx[8], vx[8];
    unpack8(kw, kx);
    unpack8(vw, vx);
    float ka = 0.f, va = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      ka = max_nan(ka, fabsf(kx[j]));
      va = max_nan(va, fabsf(vx[j]));
    }
#pragma unroll
    for (int o = TPR / 2; o > 0; o >>= 1) {   // the TPR threads of a row are neighbours in a warp
      ka = max_nan(ka, __shfl_xor_sync(0xFFFFFFFFu, ka, o));
      va = max_nan(va, __shfl_xor_sync(0xFFFFFFFFu, va, o));
    }
    if (dst < 0) return;
    constexpr float kTiny = M * 1.17549435e-38f;   // M 2^-126
    const float kb = max_nan(ka, kTiny), vb = max_nan(va, kTiny);
    const float kr = ka != 0.f ? M / kb : 1.f, vr = va != 0.f ? M / vb : 1.f;
    reinterpret_cast<uint2*>(a.k_cache)[dst * TPR + c] = encode8<KIND>(kx, kr);
    reinterpret_cast<uint2*>(a.v_cache)[dst * TPR + c] = encode8<KIND>(vx, vr);
    if (c == 0) {
      a.k_scale[dst] = ka != 0.f ? kb / M : 1.f;
      a.v_scale[dst] = va != 0.f ? vb / M : 1.f;
    }
  }
}

template <int D, int KIND>
__global__ void __launch_bounds__(cache::kThreads) cache_read_kernel(const __grid_constant__ CacheArgs a) {
  constexpr int TPR = D / 8;
  constexpr int RPB = cache::kThreads / TPR;
  const long long row = static_cast<long long>(blockIdx.x) * RPB + threadIdx.x / TPR;
  const int c = threadIdx.x % TPR;
  const int t0 = static_cast<int>(static_cast<long long>(blockIdx.x) * RPB / a.H);
  int s = find_segment(a.off, a.n_seqs, t0);
  const int t = static_cast<int>(row / a.H), h = static_cast<int>(row % a.H);
  if (t >= a.n_rows || t < __ldg(a.off)) return;
  while (s < a.n_seqs && __ldg(a.off + s + 1) <= t) ++s;
  if (s >= a.n_seqs) return;
  const long long src = cache_row(a, s, t - __ldg(a.off + s), h);
  uint4 kw = make_uint4(0, 0, 0, 0), vw = kw;   // a position without a slot reads as zeros
  if (src >= 0) {
    if constexpr (KIND == kCacheBf16) {
      kw = __ldg(reinterpret_cast<const uint4*>(a.k_cache) + src * TPR + c);
      vw = __ldg(reinterpret_cast<const uint4*>(a.v_cache) + src * TPR + c);
    } else {
      const uint2 kc = __ldg(reinterpret_cast<const uint2*>(a.k_cache) + src * TPR + c);
      const uint2 vc = __ldg(reinterpret_cast<const uint2*>(a.v_cache) + src * TPR + c);
      const float ks = __ldg(a.k_scale + src), vs = __ldg(a.v_scale + src);
      float x[8];
      decode8<KIND>(kc, ks, x);
      kw = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
      decode8<KIND>(vc, vs, x);
      vw = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    }
  }
  *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.k_out) + t * a.k_st + h * a.k_sh + 8 * c) = kw;
  *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.v_out) + t * a.v_st + h * a.v_sh + 8 * c) = vw;
}

template <int D, int KIND>
static cudaError_t launch_cache_d(const CacheArgs& a, bool write, cudaStream_t st) {
  constexpr int RPB = cache::kThreads / (D / 8);
  const long long blocks = ceil_div_ll(static_cast<long long>(a.n_rows) * a.H, RPB);
  if (blocks == 0) return cudaSuccess;
  if (blocks > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
  if (write) cache_write_kernel<D, KIND><<<static_cast<unsigned>(blocks), cache::kThreads, 0, st>>>(a);
  else cache_read_kernel<D, KIND><<<static_cast<unsigned>(blocks), cache::kThreads, 0, st>>>(a);
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
