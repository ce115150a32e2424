// decay_kernels.cu — causal linear attention with a decay for each head, its
// gradients, and its form for single tokens.
//
//   S_t = e^{g_h} S_{t-1} + k_t v_t^T,   o_t = scale * S_t^T q_t,   g_h <= 0
//
// One recurrence serves the forward and the three gradients. Along time
//   X_t = e^g X_{t-1} + s_upd b_t c_t^T,     y_t = (s_out X_t)^T a_t
// and against it
//   E_t = X_{t+1} + s_upd b_t c_t^T,  y_t = E_t^T a_t,  X_t = e^g E_t
// where X enters from x_in and leaves to x_out:
//   o          (a, b, c) = (q, k, v) along time, from S_in to S_out
//   dq = scale S_t do_t:      (do, v, k) along time, from S_in^T
//   dk = E_t v_t:             (v, do, q) against time, from dS_out^T
//   dv = E_t^T k_t:           (k, q, do) against time, from dS_out to dS_in
// with E_t = dL/dS_t = sum_{i >= t} e^{g (i - t)} scale q_i do_i^T + e^{g (N-1-t)} dS_out.
#include <algorithm>

#include "sa_internal.h"

namespace sa {

namespace decay {
constexpr float kMinLog = -1e4f;   // below, e^g is 0 in fp32 all the same, and 0 * g stays 0 for g = -inf
}

// One thread per column of X, its d entries in registers, one step per token.
template <int D>
__global__ void __launch_bounds__(D) decay_recurrent_kernel(const __grid_constant__ DecayArgs p) {
  __shared__ float sa_[D], sb[D];
  const int bh = blockIdx.x, v = threadIdx.x;
  const float w = expf(fmaxf(__ldg(p.log_decay + bh % p.H), decay::kMinLog));
  float x[D];
  const long long so = static_cast<long long>(bh) * D * D;
#pragma unroll
  for (int k = 0; k < D; ++k) x[k] = p.x_in ? p.x_in[so + (p.in_t ? v * D + k : k * D + v)] : 0.f;
  const __nv_bfloat16* A = static_cast<const __nv_bfloat16*>(p.a);
  const __nv_bfloat16* B = static_cast<const __nv_bfloat16*>(p.b);
  const __nv_bfloat16* C = static_cast<const __nv_bfloat16*>(p.c);
  for (int n = 0; n < p.N; ++n) {
    const long long t = (static_cast<long long>(bh) * p.N + (p.reverse ? p.N - 1 - n : n)) * D;
    __syncthreads();
    sa_[v] = __bfloat162float(A[t + v]);
    sb[v] = __bfloat162float(B[t + v]) * p.s_upd;
    __syncthreads();
    const float c = __bfloat162float(C[t + v]);
    float y = 0.f;
    if (p.reverse) {
#pragma unroll
      for (int k = 0; k < D; ++k) {
        x[k] = fmaf(sb[k], c, x[k]);
        y = fmaf(sa_[k], x[k], y);
        x[k] *= w;
      }
    } else {
#pragma unroll
      for (int k = 0; k < D; ++k) {
        x[k] = fmaf(x[k], w, sb[k] * c);
        y = fmaf(sa_[k], x[k], y);
      }
    }
    static_cast<__nv_bfloat16*>(p.y)[t + v] = __float2bfloat16(y * p.s_inter);
  }
  if (p.x_out)
#pragma unroll
    for (int k = 0; k < D; ++k) p.x_out[so + k * D + v] = x[k];
}

// Single token: S' = e^g S + k v^T and o = scale S'^T q, moving S once. A block
// takes a strip of 32 columns of one head's state (8 threads of 16 bytes to a
// row of the strip, 16 rows a pass), so that few heads still give many blocks.
// Every load of the strip is issued before the first is used.
template <int D>
__global__ void __launch_bounds__(128) decay_step_kernel(const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ k,
                                                         const __nv_bfloat16* __restrict__ v, const float* __restrict__ log_decay,
                                                         const float* state, float* state_out, __nv_bfloat16* __restrict__ o,
                                                         int H, float scale) {
  constexpr int NP = D / 16;
  __shared__ float red[4][32];
  const int bh = blockIdx.x / (D / 32), strip = blockIdx.x % (D / 32);
  const int r = threadIdx.x >> 3, c4 = threadIdx.x & 7;
  const long long base = static_cast<long long>(bh) * D;
  const long long so = base * D + strip * 32 + c4 * 4;
  float4 s[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) s[i] = *reinterpret_cast<const float4*>(state + so + static_cast<long long>(r + 16 * i) * D);
  const float w = expf(fmaxf(__ldg(log_decay + bh % H), decay::kMinLog));
  const uint2 vw = __ldg(reinterpret_cast<const uint2*>(v + base + strip * 32 + c4 * 4));
  const float v0 = __uint_as_float(vw.x << 16), v1 = __uint_as_float(vw.x & 0xFFFF0000u);
  const float v2 = __uint_as_float(vw.y << 16), v3 = __uint_as_float(vw.y & 0xFFFF0000u);
  float a0 = 0.f, a1 = 0.f, a2 = 0.f, a3 = 0.f;
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int row = r + 16 * i;
    const float kk = __bfloat162float(k[base + row]), qq = __bfloat162float(q[base + row]);
    s[i].x = fmaf(s[i].x, w, kk * v0);
    s[i].y = fmaf(s[i].y, w, kk * v1);
    s[i].z = fmaf(s[i].z, w, kk * v2);
    s[i].w = fmaf(s[i].w, w, kk * v3);
    *reinterpret_cast<float4*>(state_out + so + static_cast<long long>(row) * D) = s[i];
    a0 = fmaf(qq, s[i].x, a0);
    a1 = fmaf(qq, s[i].y, a1);
    a2 = fmaf(qq, s[i].z, a2);
    a3 = fmaf(qq, s[i].w, a3);
  }
  // sums over the 4 rows of a warp, then over the 4 warps
#pragma unroll
  for (int m = 8; m <= 16; m <<= 1) {
    a0 += __shfl_xor_sync(0xFFFFFFFFu, a0, m);
    a1 += __shfl_xor_sync(0xFFFFFFFFu, a1, m);
    a2 += __shfl_xor_sync(0xFFFFFFFFu, a2, m);
    a3 += __shfl_xor_sync(0xFFFFFFFFu, a3, m);
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane < 8) *reinterpret_cast<float4*>(&red[warp][lane * 4]) = make_float4(a0, a1, a2, a3);
  __syncthreads();
  if (threadIdx.x < 32)
    o[base + strip * 32 + threadIdx.x] =
        __float2bfloat16((red[0][lane] + red[1][lane] + red[2][lane] + red[3][lane]) * scale);
}

size_t decay_ws_bytes(int BH, int N, int d) { return 0; }

cudaError_t launch_decay(const DecayArgs& a, int d, cudaStream_t st) {
  if (d == 64) decay_recurrent_kernel<64><<<a.BH, 64, 0, st>>>(a);
  else decay_recurrent_kernel<128><<<a.BH, 128, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_decay_step(const void* q, const void* k, const void* v, const float* log_decay, const float* state,
                              float* state_out, void* o, int BH, int H, int d, float scale, cudaStream_t st) {
  const auto* Q = static_cast<const __nv_bfloat16*>(q);
  const auto* K = static_cast<const __nv_bfloat16*>(k);
  const auto* V = static_cast<const __nv_bfloat16*>(v);
  auto* O = static_cast<__nv_bfloat16*>(o);
  if (d == 64) decay_step_kernel<64><<<BH * 2, 128, 0, st>>>(Q, K, V, log_decay, state, state_out, O, H, scale);
  else decay_step_kernel<128><<<BH * 4, 128, 0, st>>>(Q, K, V, log_decay, state, state_out, O, H, scale);
  return cudaGetLastError();
}

}  // namespace sa
