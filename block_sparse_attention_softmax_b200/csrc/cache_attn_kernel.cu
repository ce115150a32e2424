// cache_attn_kernel.cu — attention of new tokens over the paged cache:
//   o_i = sum_j softmax_j(scale q_i . k_j) v_j  over the cached positions j that
// token i of a chunk sees (all of them, or with `causal` those up to its own),
// query head h reading key/value head h / G.
#include "sa_internal.h"

namespace sa {

// A warp per (token, query head): d / 32 channels a lane, one key at a time,
// running maximum and sum.
template <int D, int KIND>
__global__ void __launch_bounds__(128) cache_attn_simple_kernel(const __grid_constant__ CacheAttnArgs p) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int Hq = p.H * p.G;
  const long long item = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int t = static_cast<int>(item / Hq), hq = static_cast<int>(item % Hq);
  if (t >= p.n_rows) return;
  if (t < __ldg(p.cu_q)) return;
  const int s = find_segment(p.cu_q, p.n_seqs, t);
  if (s >= p.n_seqs) return;
  const int q1 = min(__ldg(p.cu_q + s + 1), p.n_rows);
  const int L = static_cast<int>(max(0ll, min(static_cast<long long>(__ldg(p.kv_len + s)), static_cast<long long>(p.width) * p.page)));
  const int vis = p.causal ? max(0, L - (q1 - t) + 1) : L;
  const __nv_bfloat16* qp = static_cast<const __nv_bfloat16*>(p.q) + t * p.q_st + hq * p.q_sh;
  CacheArgs ca;
  ca.table = p.table; ca.width = p.width; ca.page = p.page; ca.n_pages = p.n_pages; ca.H = p.H;
  float q[E], o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = __bfloat162float(qp[lane * E + e]) * p.scale_log2;
    o[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j < vis; ++j) {
    const long long row = cache_row(ca, s, j, hq / p.G);
    float k[E], v[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const long long i = row * D + lane * E + e;
      if (row < 0) {
        k[e] = v[e] = 0.f;
      } else if constexpr (KIND == kCacheBf16) {
        k[e] = __bfloat162float(static_cast<const __nv_bfloat16*>(p.k_cache)[i]);
        v[e] = __bfloat162float(static_cast<const __nv_bfloat16*>(p.v_cache)[i]);
      } else if constexpr (KIND == kCacheE4m3) {
        k[e] = static_cast<float>(static_cast<const __nv_fp8_e4m3*>(p.k_cache)[i]) * __ldg(p.k_scale + row);
        v[e] = static_cast<float>(static_cast<const __nv_fp8_e4m3*>(p.v_cache)[i]) * __ldg(p.v_scale + row);
      } else {
        k[e] = static_cast<const int8_t*>(p.k_cache)[i] * __ldg(p.k_scale + row);
        v[e] = static_cast<const int8_t*>(p.v_cache)[i] * __ldg(p.v_scale + row);
      }
    }
    float x = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) x = fmaf(q[e], k[e], x);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, d);
    const float mn = fmaxf(m, x);
    const float corr = exp2f(m - mn), w = exp2f(x - mn);
    l = l * corr + w;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = fmaf(o[e], corr, w * v[e]);
    m = mn;
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  __nv_bfloat16* op = static_cast<__nv_bfloat16*>(p.o) + t * p.o_st + hq * p.o_sh;
#pragma unroll
  for (int e = 0; e < E; ++e) op[lane * E + e] = __float2bfloat16(o[e] * inv);
  if (p.lse && lane == 0)
    p.lse[static_cast<long long>(t) * Hq + hq] = l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

size_t cache_attn_ws_bytes(int d) { return 0; }

template <int D>
static cudaError_t launch_cache_attn_d(const CacheAttnArgs& a, int kind, cudaStream_t st) {
  const unsigned grid = static_cast<unsigned>(ceil_div_ll(static_cast<long long>(a.n_rows) * a.H * a.G, 4));
  if (kind == kCacheBf16) cache_attn_simple_kernel<D, kCacheBf16><<<grid, 128, 0, st>>>(a);
  else if (kind == kCacheE4m3) cache_attn_simple_kernel<D, kCacheE4m3><<<grid, 128, 0, st>>>(a);
  else cache_attn_simple_kernel<D, kCacheInt8><<<grid, 128, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_cache_attn(const CacheAttnArgs& a, int d, int kind, cudaStream_t st) {
  return d == 64 ? launch_cache_attn_d<64>(a, kind, st) : launch_cache_attn_d<128>(a, kind, st);
}

}  // namespace sa
