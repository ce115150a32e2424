// decay_kernels.cu — causal linear attention with a decay for each head, its
// gradients, and its form for single tokens.
//
//   S_t = e^{g_h} S_{t-1} + k_t v_t^T,   o_t = scale * S_t^T q_t,   g_h <= 0
//
// One recurrence serves the forward and the three gradients. Along time
//   X_t = e^g X_{t-1} + s_upd b_t c_t^T,     y_t = (s_inter X_t)^T a_t
// and against it
//   E_t = X_{t+1} + s_upd b_t c_t^T,  y_t = s_inter E_t^T a_t,  X_t = e^g E_t
// where X enters from x_in and leaves to x_out:
//   o          (a, b, c) = (q, k, v) along time, from S_in to S_out
//   dq = scale S_t do_t:      (do, v, k) along time, from S_in^T
//   dk = E_t v_t:             (v, do, q) against time, from dS_out^T
//   dv = E_t^T k_t:           (k, q, do) against time, from dS_out to dS_in
// with E_t = dL/dS_t = sum_{i >= t} e^{g (i - t)} scale q_i do_i^T + e^{g (N-1-t)} dS_out.
//
// Chunked form. With w = e^g and X the state before a chunk of 128 tokens (along
// time; against it i and j change places, and the exponents are those of the
// E_t above):
//   y_i = s_intra sum_{j <= i} w^{i-j} (a_i . b_j) c_j + s_inter w^{i+1} X^T a_i
//   X'  = w^128 X + sum_j (s_upd w^{127-j} b_j) c_j^T
// Four matrix products of a chunk on tcgen05 (a b^T, P c, a X, b'^T c). All powers
// of w have exponents of at least 0, so a decay that leaves nothing of a token's
// neighbour is as good as any. States stay in fp32; for those that leave the call the
// operand b' is split into three bf16 numbers (exactly), for the others into two
// (2^-16 of it is lost at most). The decay of a chunk multiplies such a state again
// and again and is a pair of fp32 numbers there (decay_pair). P and the state's copy
// that meets a are rounded to bf16 once, as q, k and v are.
//
// Split of the work: the chunks of all heads, head after head, are cut into equal
// contiguous ranges, one per SM. Where a head is cut, the states at the cuts are
// needed first: decay_state_kernel forms each range's own contribution (a weighted
// product b'^T c with weights relative to the range's end, so no step depends on
// another), decay_join_kernel steps over the ranges of a head, and
// decay_chunk_kernel then runs every range from its state. Where heads are many
// enough to fill the SMs whole (see decay_geom), it runs alone.
#include <algorithm>

#include "sa_internal.h"

namespace sa {

namespace decay {

constexpr float kMinLog = -1e4f;   // below, e^g is 0 in fp32 all the same, and 0 * g stays 0 for g = -inf
constexpr int kTok = 128;          // tokens of a chunk
constexpr int kThreads = 1024;     // decay_chunk_kernel: 4 warps for loads, issue and stores, 8 for P, 4 for y, 8 each for the state and b'
constexpr int kStateThreads = 640; // decay_state_kernel: 4 warps of loads and issue, 16 that scale b
constexpr int kPow = 32 + kTok;    // a table of w^0 .. w^127 behind 32 entries that are read but not used

struct Geom {
  int tph;     // chunks of a head
  int total;   // of all heads
  int grid;    // ranges
  int tpc;     // chunks of a range
  int hpc;     // heads that a range can touch
  int whole;   // ranges are whole heads
};

// A range of whole heads costs its chunks; cut heads cost half a chunk more for
// each (two of four operands are read twice) and two more launches with the states
// between them, about 8 us or three chunks.
inline Geom decay_geom(int BH, int N) {
  const int sms = sm_count_cached();
  Geom g;
  g.tph = ceil_div(N, kTok);
  g.total = BH * g.tph;
  const int hpr = ceil_div(BH, sms);
  g.whole = 2ll * hpr * g.tph <= 3ll * ceil_div(g.total, sms) + 6;
  g.tpc = g.whole ? hpr * g.tph : ceil_div(g.total, sms);
  g.grid = ceil_div(g.total, g.tpc);
  g.hpc = (g.tpc + g.tph - 2) / g.tph + 1;
  return g;
}

__device__ __forceinline__ float clamped(float g) { return g < kMinLog ? kMinLog : g; }

// log2 of a head's decay.
__device__ __forceinline__ float log2_decay(const float* log_decay, int h) {
  return clamped(__ldg(log_decay + h)) * 1.4426950408889634f;
}

// e^y, y <= 0, as the sum of two fp32 numbers, for states that are multiplied with it again and again: the rounding of
// one number near 1 is the same every time and adds up over a state's memory (5.7e-6 of a state after 79 chunks). With
// e^y - 1 accurate to its own size, the sum is off by 2^-23 over any memory.
__device__ __forceinline__ float2 decay_pair(float y) {
  const float m = expm1f(y), hi = 1.f + m, e = expf(y);
  const bool near1 = y >= -0.5f;   // (else a memory of two steps, and e^y - 1 would lose e^y)
  return make_float2(near1 ? hi : e, near1 ? m - (hi - 1.f) : 0.f);   // (the difference is exact)
}

// x e^y + u for that pair.
__device__ __forceinline__ float decayed(float x, float2 w, float u) { return fmaf(x, w.x, fmaf(x, w.y, u)); }

__device__ __forceinline__ uint8_t* align1k(uint8_t* p) {
  return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(p) + 1023) & ~uintptr_t(1023));
}

// 8 bf16 values times w as three bf16 numbers each: 24 bits, exactly.
__device__ __forceinline__ void split8(const uint4 x, float w, uint4& hi, uint4& lo, uint4& lo2) {
  const uint32_t v[4] = {x.x, x.y, x.z, x.w};
  uint32_t h[4], l[4], m[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float a = __uint_as_float(v[j] << 16) * w, b = __uint_as_float(v[j] & 0xFFFF0000u) * w;
    h[j] = pack_bf16x2(a, b);
    a -= __uint_as_float(h[j] << 16);
    b -= __uint_as_float(h[j] & 0xFFFF0000u);
    l[j] = pack_bf16x2(a, b);
    m[j] = pack_bf16x2(a - __uint_as_float(l[j] << 16), b - __uint_as_float(l[j] & 0xFFFF0000u));
  }
  hi = make_uint4(h[0], h[1], h[2], h[3]);
  lo = make_uint4(l[0], l[1], l[2], l[3]);
  lo2 = make_uint4(m[0], m[1], m[2], m[3]);
}

// 8 bf16 values times w as two bf16 numbers each.
__device__ __forceinline__ void split8(const uint4 x, float w, uint4& hi, uint4& lo) {
  const uint32_t v[4] = {x.x, x.y, x.z, x.w};
  uint32_t h[4], l[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float a = __uint_as_float(v[j] << 16) * w, b = __uint_as_float(v[j] & 0xFFFF0000u) * w;
    h[j] = pack_bf16x2(a, b);
    l[j] = pack_bf16x2(a - __uint_as_float(h[j] << 16), b - __uint_as_float(h[j] & 0xFFFF0000u));
  }
  hi = make_uint4(h[0], h[1], h[2], h[3]);
  lo = make_uint4(l[0], l[1], l[2], l[3]);
}

template <int D>
struct Tiles {
  static constexpr int NCH = D / 64;                  // 128-byte chunks of a row
  static constexpr uint32_t CHUNK = kTok * 128;
  static constexpr uint32_t TILE = NCH * CHUNK;
  // mapping of NT threads to the 16-byte units of a tile: rows a pass, passes
  static constexpr int CPR = D / 8;
  static constexpr int rows(int nt) { return nt / CPR; }
  static constexpr int passes(int nt) { return kTok * CPR / nt; }
  __device__ static uint32_t unit(int row, int c) { return (c >> 3) * CHUNK + row * 128 + (((c & 7) ^ (row & 7)) << 4); }
};

template <int D>
struct ChunkLayout : Tiles<D> {
  using T = Tiles<D>;
  static constexpr uint32_t OFF_X = 0;                            // the state in bf16, then the low parts of b'
  static constexpr uint32_t OFF_A = T::TILE, OFF_B = OFF_A + 2 * T::TILE, OFF_C = OFF_B + 2 * T::TILE;
  static constexpr uint32_t OFF_POW = OFF_C + 2 * T::TILE;        // powers of w, two tables
  static constexpr uint32_t OFF_BAR = OFF_POW + 2 * kPow * 4;
  static constexpr uint32_t SMEM = OFF_BAR + 256 + 1024;
  static_assert(OFF_BAR % 8 == 0 && SMEM <= 227 * 1024, "shared memory per CTA");
};

template <int D, bool EXACT>
struct StateLayout : Tiles<D> {
  using T = Tiles<D>;
  static constexpr int kStages = D == 128 && EXACT ? 2 : 3;       // (what the shared memory holds)
  static constexpr uint32_t OFF_LO = 0;                           // second and third numbers of b'
  static constexpr uint32_t OFF_B = (EXACT ? 2 : 1) * T::TILE, OFF_C = OFF_B + kStages * T::TILE;
  static constexpr uint32_t OFF_BAR = OFF_C + kStages * T::TILE;
  static constexpr uint32_t SMEM = OFF_BAR + 256 + 1024;
  static_assert(SMEM <= 227 * 1024, "shared memory per CTA");
};

// The chunks of a range one after the other, in order of time or against it.
template <bool REV>
struct Chunks {
  int bh, r, tph, N;
  __device__ Chunks(const Geom& g, int N_, int c0, int c1) : tph(g.tph), N(N_) {
    const int t = REV ? c1 - 1 : c0;
    bh = t / tph;
    r = t - bh * tph;
  }
  __device__ void next() {
    if (REV) {
      if (--r < 0) {
        r = tph - 1;
        --bh;
      }
    } else if (++r == tph) {
      r = 0;
      ++bh;
    }
  }
  __device__ int row() const { return r * kTok; }
  __device__ int len() const { return min(kTok, N - r * kTok); }
  __device__ bool first() const { return REV ? r == tph - 1 : r == 0; }   // of the head
};

// Part of a head that lies in one range: its chunks [lo, hi) and tokens [n0, n1).
struct Part {
  int lo, hi, n0, n1;
};
__device__ __forceinline__ Part part_of(const Geom& g, int cta, int bh, int N) {
  Part p;
  p.lo = max(bh * g.tph, cta * g.tpc);
  p.hi = min(min(g.total, (cta + 1) * g.tpc), (bh + 1) * g.tph);
  p.n0 = (p.lo - bh * g.tph) * kTok;
  p.n1 = min(N, (p.hi - bh * g.tph) * kTok);
  return p;
}
__device__ __forceinline__ long long slot_of(const Geom& g, int cta, int bh) {
  return static_cast<long long>(cta) * g.hpc + bh - cta * g.tpc / g.tph;
}

}  // namespace decay

// ---------------------------------------------------------------- a range's own contribution
// X_part = sum_j (s_upd w^{dist_j} b_j) c_j^T over the tokens of a range's share of a
// head, dist_j the steps from token j to the share's end (against time: its start).
// Chunks so far back that w^dist is 0 in fp32 for every token add nothing and are
// not read. Over the chunks the sum is made in registers, in fp32 rounded to nearest:
// the tensor pipe's adds truncate, and a long sum drifts (9e-6 off over 160 chunks,
// 1.5e-6 over four at a time). EXACT: b' in three bf16 numbers, for states that leave
// the call (1.9e-7 off, against 2.5e-6 with two; 720p 787 -> 870 us). A chunk is 64 KB
// (d = 128) against 1024 cycles of the tensor pipe (EXACT: 1536), but what bounds it is
// the splitting of b and the sums, which take turns with the products: of 40 heads x
// 75,600 it reads 1.12 GB in 234 us with two numbers (4.8 TB/s) and in 329 us with
// three (3.4 TB/s).
template <int D, bool EXACT>
__global__ void __launch_bounds__(decay::kStateThreads, 1)
    decay_state_kernel(const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmC,
                       const __grid_constant__ DecayArgs p, const __grid_constant__ decay::Geom geo) {
  using namespace decay;
  using L = StateLayout<D, EXACT>;
  constexpr int kStages = L::kStages;
  constexpr int kSum = EXACT ? 1 : 4;   // chunks that the tensor pipe sums
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1k(smem_raw);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);   // [kStages] landed
  uint64_t* empty = full + kStages;                                  // [kStages] products done
  uint64_t* ready = empty + kStages;                                 // b' written
  uint64_t* drain = ready + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  // a warp's wait (all lanes poll: with one of them polling apart from the others every wait cost some hundred cycles more)
  const auto warp_wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait_asleep(bar, parity, p.wait_tries); };
  const int c0 = blockIdx.x * geo.tpc, c1 = min(geo.total, c0 + geo.tpc);
  const bool rev = p.reverse != 0;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(ready, 16);
    mbar_init(drain, 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = __shfl_sync(0xFFFFFFFFu, *tmem_slot, 0);
  // With `early` the kernel before this one is of the same call: b and c were there before it, and the loader starts
  // at once. Everyone else waits here, so that no bounded wait has to outlast that kernel.
  if (!p.early || warp != 0) grid_dep_wait();
  grid_dep_trigger();

  // the shares of the range, and of each the chunks [t0, t1) that add something
  const int bh0 = c0 / geo.tph, bh1 = (c1 - 1) / geo.tph;
  auto share = [&](int bh, Part& q, float& g2, int& t0, int& t1) {
    q = part_of(geo, blockIdx.x, bh, p.N);
    g2 = log2_decay(p.log_decay, bh % p.H);
    t0 = q.lo;
    t1 = q.hi;
    // the head's last share matters for x_out alone
    if (!p.x_out && (rev ? q.lo == bh * geo.tph : q.hi == (bh + 1) * geo.tph)) t1 = t0;
    else if (g2 < 0.f) {
      // 2^-150 and below is 0 in fp32; the nearest token of chunk t is (q.hi - 1 - t) kTok - 127 steps or more away
      const float far = 150.f / -g2 + 128.f;
      const int keep = far < 1e9f ? static_cast<int>(far) / kTok + 2 : 0x3FFFFFFF;
      if (rev) t1 = min(q.hi, keep < q.hi - q.lo ? q.lo + keep : q.hi);
      else t0 = keep < q.hi - q.lo ? q.hi - keep : q.lo;
    }
  };

  if (warp == 0) {
    int m = 0;
    bool ok = true;
    for (int bh = bh0; ok && bh <= bh1; ++bh) {
      Part q;
      float g2;
      int t0, t1;
      share(bh, q, g2, t0, t1);
      for (int t = t0; t < t1; ++t, ++m) {
        const int s = m % kStages;
        if (m == kStages) grid_dep_wait();
        if (!(ok = warp_wait(&empty[s], ((m / kStages) & 1) ^ 1))) break;
        const int row = (t - bh * geo.tph) * kTok;
        if (elect_one()) {
          mbar_arrive_expect_tx(&full[s], 2 * L::TILE);
#pragma unroll
          for (int c = 0; c < L::NCH; ++c) {
            tma_load_3d(smem + L::OFF_B + s * L::TILE + c * L::CHUNK, &tmB, &full[s], c * 64, row, bh);
            tma_load_3d(smem + L::OFF_C + s * L::TILE + c * L::CHUNK, &tmC, &full[s], c * 64, row, bh);
          }
        }
        __syncwarp();
      }
    }
    if (lane == 0)
      for (int i = 1; i <= kStages && i <= m; ++i) mbar_drain(&full[(m - i) % kStages], ((m - i) / kStages) & 1);
    __syncwarp();
  } else if (warp == 1) {
    // (for d = 64 the upper 64 rows of the 128 are products of whatever lies behind the tile; nothing reads them)
    const uint32_t idesc = idesc_bf16_f32(128, D, true, true);
    const uint64_t lo0 = sw128_desc(smem_u32(smem + L::OFF_LO), L::CHUNK, 1024);
    const uint64_t b0 = sw128_desc(smem_u32(smem + L::OFF_B), L::CHUNK, 1024);
    const uint64_t cd0 = sw128_desc(smem_u32(smem + L::OFF_C), L::CHUNK, 1024);
    int m = 0, sums = 0;
    bool ok = true;
    for (int bh = bh0; ok && bh <= bh1; ++bh) {
      Part q;
      float g2;
      int t0, t1;
      share(bh, q, g2, t0, t1);
      for (int t = t0; t < t1; ++t, ++m) {
        const int s = m % kStages;
        if (!(ok = warp_wait(ready, m & 1))) break;
        tc_fence_after();
        const uint64_t bd = b0 + ((s * L::TILE) >> 4), cd = cd0 + ((s * L::TILE) >> 4);
        const bool fresh = (t - t0) % kSum == 0;   // a new sum, in the other accumulator
        sums += fresh ? 1 : 0;
        const uint32_t td = tm + (sums & 1) * 128;
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < kTok / 16; ++kk) umma_ss(td, lo0 + kk * 128, cd + kk * 128, idesc, !fresh || kk > 0 ? 1u : 0u);
          if constexpr (EXACT) {
#pragma unroll
            for (int kk = 0; kk < kTok / 16; ++kk) umma_ss(td, lo0 + (L::TILE >> 4) + kk * 128, cd + kk * 128, idesc, 1u);
          }
#pragma unroll
          for (int kk = 0; kk < kTok / 16; ++kk) umma_ss(td, bd + kk * 128, cd + kk * 128, idesc, 1u);
          tc_commit(&empty[s]);
        }
        __syncwarp();
      }
    }
    if (elect_one()) {
      tc_commit(drain);
      mbar_drain(drain, 0);
    }
    __syncwarp();
  } else if (warp >= 4) {
    const int st = threadIdx.x - 128;
    constexpr int R2 = L::rows(512), N2 = L::passes(512);
    const int c = st % L::CPR, r0 = st / L::CPR;
    const int quad = warp & 3, col0 = ((warp - 4) >> 2) * (D / 4);
    const int row_x = quad * 32 + lane;
    int m = 0;
    bool ok = true;
    float x_acc[D / 4];   // this thread's part of a row of X_part
    // the sums lie in one of two accumulators in turn
    int sums = 0;
    auto add_product = [&](int n) {
      if (quad * 32 >= D) return;
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < D / 4; c += 16) {
        uint32_t r[16];
        tmem_ld16_wait(tm + (n & 1) * 128 + (static_cast<uint32_t>(quad * 32) << 16) + col0 + c, r);
#pragma unroll
        for (int e = 0; e < 16; ++e) x_acc[c + e] += __uint_as_float(r[e]);
      }
      tc_fence_before();
    };
    for (int bh = bh0; ok && bh <= bh1; ++bh) {
      Part q;
      float g2;
      int t0, t1;
      share(bh, q, g2, t0, t1);
#pragma unroll
      for (int e = 0; e < D / 4; ++e) x_acc[e] = 0.f;
      for (int t = t0; t < t1; ++t, ++m) {
        const int s = m % kStages;
        const int row = (t - bh * geo.tph) * kTok;
        if (!(ok = warp_wait(&full[s], (m / kStages) & 1))) break;
        uint4 x[N2], lo[N2], lo2[N2];
        uint8_t* sb = smem + L::OFF_B + s * L::TILE;
#pragma unroll
        for (int i = 0; i < N2; ++i) x[i] = *reinterpret_cast<const uint4*>(sb + L::unit(r0 + i * R2, c));
#pragma unroll
        for (int i = 0; i < N2; ++i) {
          const int r = r0 + i * R2, n = row + r;
          const float dist = static_cast<float>(rev ? n + 1 - q.n0 : q.n1 - 1 - n);
          const float w = n < q.n1 ? fast_exp2(dist * g2) * p.s_upd : 0.f;
          uint4 hi;
          if constexpr (EXACT) split8(x[i], w, hi, lo[i], lo2[i]);
          else split8(x[i], w, hi, lo[i]);
          *reinterpret_cast<uint4*>(sb + L::unit(r, c)) = hi;
        }
        // the other parts' buffers: the products before have read them
        if (m > 0 && !(ok = warp_wait(&empty[(m - 1) % kStages], ((m - 1) / kStages) & 1))) break;
#pragma unroll
        for (int i = 0; i < N2; ++i) {
          *reinterpret_cast<uint4*>(smem + L::OFF_LO + L::unit(r0 + i * R2, c)) = lo[i];
          if constexpr (EXACT) *reinterpret_cast<uint4*>(smem + L::OFF_LO + L::TILE + L::unit(r0 + i * R2, c)) = lo2[i];
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(ready);
        if ((t - t0) % kSum == 0) {
          if (t > t0) add_product(sums);
          ++sums;
        }
      }
      if (!ok || t0 >= t1) continue;
      if (!(ok = warp_wait(&empty[(m - 1) % kStages], ((m - 1) / kStages) & 1))) break;
      add_product(sums);
      if (quad * 32 < D) {
        float* out = static_cast<float*>(p.ws) + slot_of(geo, blockIdx.x, bh) * (D * D) + row_x * D + col0;
#pragma unroll
        for (int e = 0; e < D / 4; e += 4)
          *reinterpret_cast<float4*>(out + e) = make_float4(x_acc[e], x_acc[e + 1], x_acc[e + 2], x_acc[e + 3]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tm, 256);
  }
}

// Steps over the shares of a head: each slot's contribution becomes the state that
// enters the share, and the state behind the last one goes to x_out. A thread
// holds 4 columns of a row; 8 shares' loads are in flight at a time.
template <int D>
__global__ void __launch_bounds__(256) decay_join_kernel(const __grid_constant__ DecayArgs p, const __grid_constant__ decay::Geom geo) {
  using namespace decay;
  grid_dep_wait();
  grid_dep_trigger();
  const int bh = blockIdx.y, e = (blockIdx.x * 256 + threadIdx.x) * 4;
  const int row = e / D, col = e % D;
  const long long so = static_cast<long long>(bh) * D * D;
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  if (p.x_in) {
    if (p.in_t) {
      const float* s = p.x_in + so + static_cast<long long>(col) * D + row;
      x = make_float4(s[0], s[D], s[2 * D], s[3 * D]);
    } else {
      x = *reinterpret_cast<const float4*>(p.x_in + so + e);
    }
  }
  const float g = clamped(__ldg(p.log_decay + bh % p.H));
  const int ca = bh * geo.tph / geo.tpc, cb = ((bh + 1) * geo.tph - 1) / geo.tpc, n = cb - ca + 1;
  float* ws = static_cast<float*>(p.ws);
  // decays over the head's first share, its last one, and those between, which are all of one length
  const Part qa = part_of(geo, ca, bh, p.N), qb = part_of(geo, cb, bh, p.N);
  const float2 wa = decay_pair(static_cast<float>(qa.n1 - qa.n0) * g), wb = decay_pair(static_cast<float>(qb.n1 - qb.n0) * g);
  const float2 wi = decay_pair(static_cast<float>(geo.tpc) * kTok * g);
  for (int i0 = 0; i0 < n; i0 += 8) {
    float4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // (the head's last share is only formed, and needed, where x_out is)
      if (i0 + i < n && (i0 + i + 1 < n || p.x_out))
        v[i] = *reinterpret_cast<const float4*>(ws + slot_of(geo, p.reverse ? cb - i0 - i : ca + i0 + i, bh) * (D * D) + e);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i0 + i < n) {
        const int c = p.reverse ? cb - i0 - i : ca + i0 + i;
        *reinterpret_cast<float4*>(ws + slot_of(geo, c, bh) * (D * D) + e) = x;
        if (i0 + i + 1 < n || p.x_out) {
          const float2 w = c == ca ? wa : c == cb ? wb : wi;
          x = make_float4(decayed(x.x, w, v[i].x), decayed(x.y, w, v[i].y), decayed(x.z, w, v[i].z), decayed(x.w, w, v[i].w));
        }
      }
    }
  }
  if (p.x_out) *reinterpret_cast<float4*>(p.x_out + so + e) = x;
}

// ---------------------------------------------------------------- the chunks
// Persistent over a range's chunks. Warp 0 loads a, b, c (two slots each), warps 1
// and 3 issue the products of the two chains below, warp 2 stores y; eight turn a b^T into P and four each form y,
// keep the state (its bf16 copy for the product with a, and its decay) and form b',
// so that the groups work on different chunks at a time. Per chunk:
//   A = a b^T, P, Y1 = P c, the next A   and   X, Y2 = a X, U = b'_lo^T c + b'_hi^T c, X = w X + U
// (2560 cycles of the tensor pipe at d = 128 against 128 KB moved, some 5500
// cycles of the memory's rate; it takes 6,700, the shared memory being busy for some
// 4,900 of them: 3.1 GB in 0.53 ms at 40 heads x 75,600). b' takes b's place in its slot once A is done, its
// low parts the place of the state's copy; y is staged in a's slot.
// EXACT: a third number of b' follows the second one in its place, and the chunk's
// decay is a pair, for ranges of whole heads, whose last state is the caller's (all of
// them take it, so that y has the same bits whether that state is asked for or not).
// Elsewhere the states that leave the call come from the two kernels above.
template <int D, bool REV, bool EXACT>
__global__ void __launch_bounds__(decay::kThreads, 1)
    decay_chunk_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                       const __grid_constant__ CUtensorMap tmC, const __grid_constant__ CUtensorMap tmY,
                       const __grid_constant__ DecayArgs p, const __grid_constant__ decay::Geom geo) {
  using namespace decay;
  using L = ChunkLayout<D>;
  constexpr uint32_t TM_A = 0, TM_U = 128, TM_Y1 = 256, TM_Y2 = 384;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1k(smem_raw);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  uint64_t* ab_full = bars;           // [2] a and b landed
  uint64_t* c_full = bars + 4;        // [2]
  uint64_t* a_empty = bars + 6;       // [2] y left the slot
  uint64_t* upd = bars + 8;           // [2] U done: slot of b free, and of c with p_done
  uint64_t* a_done = bars + 10;       // [2] A = a b^T
  uint64_t* x_ready = bars + 12;      // state's copy written, last update read
  uint64_t* x_read = bars + 13;       // Y2 = a X
  uint64_t* p_ready = bars + 14;
  uint64_t* b_ready = bars + 15;      // [2] b' written
  uint64_t* y_full = bars + 17;       // Y1 and Y2 done
  uint64_t* y_empty = bars + 18;      // and read
  uint64_t* y_staged = bars + 19;     // y in a's slot
  uint64_t* drain = bars + 20;        // [2]
  uint64_t* p_done = bars + 22;       // [2] P and c are read by Y1 = P c
  uint64_t* lo_read = bars + 24;      // (EXACT) b'_lo is read
  uint64_t* lo2_ready = bars + 25;    // (EXACT) b'_lo2 written
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 26);
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  // a warp's wait (all lanes poll: with one of them polling apart from the others every wait cost some hundred cycles more)
  const auto warp_wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait_asleep(bar, parity, p.wait_tries); };
  constexpr bool rev = REV;
  const int c0 = blockIdx.x * geo.tpc, c1 = min(geo.total, c0 + geo.tpc), n_chunks = c1 - c0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ab_full[i], 2);
      mbar_init(&c_full[i], 1);
      mbar_init(&a_empty[i], 1);
      mbar_init(&upd[i], 1);
      mbar_init(&a_done[i], 1);
    }
    mbar_init(x_ready, 8);
    mbar_init(x_read, 1);
    mbar_init(p_ready, 8);
    mbar_init(&b_ready[0], 8);
    mbar_init(&b_ready[1], 8);
    mbar_init(y_full, 2);
    mbar_init(y_empty, 4);
    mbar_init(y_staged, 4);
    mbar_init(&drain[0], 1);
    mbar_init(&drain[1], 1);
    mbar_init(&p_done[0], 1);
    mbar_init(&p_done[1], 1);
    mbar_init(lo_read, 1);
    mbar_init(lo2_ready, 8);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = __shfl_sync(0xFFFFFFFFu, *tmem_slot, 0);
  // Behind the join (or another such kernel of the same call) a, b and c were there before it: the first chunks load and
  // the first A is made while it ends. Everyone else waits here, so that no bounded wait has to outlast that kernel.
  if (geo.whole || warp > 1) grid_dep_wait();
  grid_dep_trigger();

  // registers a thread: 32 (4 x 32 + 8 x 56 + 4 x 48 + 8 x 96 + 8 x 64) = 65536, the launch's 1024 x 64
  if (warp < 4) {
    reg_dealloc<32>();
    if (warp == 0) {
      int n = 0;           // chunks loaded
      int part = 0;        // of one more: 1 its b, 2 its c too
      Chunks<REV> k(geo, p.N, c0, c1);
      for (int i = 0; i < n_chunks; ++i, k.next()) {
        const int s = i & 1, row = k.row(), bh = k.bh;
        const uint32_t ph = ((i >> 1) & 1) ^ 1;
        if (i == 2) grid_dep_wait();
        if (!warp_wait(&upd[s], ph)) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(&ab_full[s], L::TILE);
#pragma unroll
          for (int c = 0; c < L::NCH; ++c) tma_load_3d(smem + L::OFF_B + s * L::TILE + c * L::CHUNK, &tmB, &ab_full[s], c * 64, row, bh);
        }
        __syncwarp();
        part = 1;
        if (!warp_wait(&p_done[s], ph)) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(&c_full[s], L::TILE);
#pragma unroll
          for (int c = 0; c < L::NCH; ++c) tma_load_3d(smem + L::OFF_C + s * L::TILE + c * L::CHUNK, &tmC, &c_full[s], c * 64, row, bh);
        }
        __syncwarp();
        part = 2;
        if (!warp_wait(&a_empty[s], ph)) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(&ab_full[s], L::TILE);
#pragma unroll
          for (int c = 0; c < L::NCH; ++c) tma_load_3d(smem + L::OFF_A + s * L::TILE + c * L::CHUNK, &tmA, &ab_full[s], c * 64, row, bh);
        }
        __syncwarp();
        part = 0;
        ++n;
      }
      // loads in flight land before the CTA gives up its shared memory
      if (lane == 0) {
        for (int i = 1; i <= 2 && i <= n; ++i) {
          mbar_drain(&ab_full[(n - i) & 1], ((n - i) >> 1) & 1);
          mbar_drain(&c_full[(n - i) & 1], ((n - i) >> 1) & 1);
        }
        if (part > 0) {
          mbar_arrive(&ab_full[n & 1]);   // in place of a's
          mbar_drain(&ab_full[n & 1], (n >> 1) & 1);
          if (part > 1) mbar_drain(&c_full[n & 1], (n >> 1) & 1);
        }
      }
      __syncwarp();
    } else if (warp == 1) {
      // A = a b^T of a chunk, then Y1 = P c of it, and the next A in P's place
      const uint32_t id_a = idesc_bf16_f32(128, 128, false, false);
      const uint32_t id_y = idesc_bf16_f32(128, D, false, true);
      const uint64_t ak = sw128_desc(smem_u32(smem + L::OFF_A), 16, 1024);
      const uint64_t bk = sw128_desc(smem_u32(smem + L::OFF_B), 16, 1024);
      const uint64_t cm = sw128_desc(smem_u32(smem + L::OFF_C), L::CHUNK, 1024);
      for (int i = 0; i <= n_chunks; ++i) {
        if (i > 0) {
          const int s = (i - 1) & 1;
          if (i == 1) grid_dep_wait();
          if (!warp_wait(p_ready, (i - 1) & 1)) break;
          if (!warp_wait(&c_full[s], ((i - 1) >> 1) & 1)) break;
          if (i > 1 && !warp_wait(y_empty, i & 1)) break;
          tc_fence_after();
          const uint64_t cd = cm + ((s * L::TILE) >> 4);
          if (elect_one()) {
#pragma unroll 4
            for (int kk = 0; kk < kTok / 16; ++kk) umma_ts(tm + TM_Y1, tm + TM_A + kk * 8, cd + kk * 128, id_y, kk > 0 ? 1u : 0u);
            tc_commit(y_full);
            tc_commit(&p_done[s]);
          }
          __syncwarp();
        }
        if (i == n_chunks) break;
        const int s = i & 1;
        if (!warp_wait(&ab_full[s], (i >> 1) & 1)) break;
        if (i > 0 && !warp_wait(&p_done[s ^ 1], ((i - 1) >> 1) & 1)) break;
        tc_fence_after();
        const uint64_t ad = ak + ((s * L::TILE) >> 4), bd = bk + ((s * L::TILE) >> 4);
        if (elect_one()) {
#pragma unroll 4
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = ((kk >> 2) * L::CHUNK + (kk & 3) * 32u) >> 4;
            umma_ss(tm + TM_A, ad + off, bd + off, id_a, kk > 0 ? 1u : 0u);
          }
          tc_commit(&a_done[s]);
        }
        __syncwarp();
      }
      if (elect_one()) {
        tc_commit(&drain[0]);
        mbar_drain(&drain[0], 0);
      }
      __syncwarp();
    } else if (warp == 3) {
      // Y2 = a X of a chunk, then U = b'_lo^T c + b'_hi^T c (d = 64: U's rows 64.. are not read)
      const uint32_t id_y = idesc_bf16_f32(128, D, false, true);
      const uint32_t id_x = idesc_bf16_f32(128, D, true, true);
      const uint64_t ak = sw128_desc(smem_u32(smem + L::OFF_A), 16, 1024);
      const uint64_t bm = sw128_desc(smem_u32(smem + L::OFF_B), L::CHUNK, 1024);
      const uint64_t cm = sw128_desc(smem_u32(smem + L::OFF_C), L::CHUNK, 1024);
      const uint64_t xm = sw128_desc(smem_u32(smem + L::OFF_X), D * 128, 1024);
      const uint64_t lm = sw128_desc(smem_u32(smem + L::OFF_X), L::CHUNK, 1024);
      for (int i = 0; i < n_chunks; ++i) {
        const int s = i & 1;
        const uint64_t ad = ak + ((s * L::TILE) >> 4), bd = bm + ((s * L::TILE) >> 4), cd = cm + ((s * L::TILE) >> 4);
        if (!warp_wait(&ab_full[s], (i >> 1) & 1)) break;
        if (!warp_wait(x_ready, i & 1)) break;
        if (i > 0 && !warp_wait(y_empty, (i - 1) & 1)) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll 4
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = ((kk >> 2) * L::CHUNK + (kk & 3) * 32u) >> 4;
            umma_ss(tm + TM_Y2, ad + off, xm + kk * 128, id_y, kk > 0 ? 1u : 0u);
          }
          tc_commit(x_read);
          tc_commit(y_full);
        }
        __syncwarp();
        if (!warp_wait(&c_full[s], (i >> 1) & 1)) break;
        if (!warp_wait(&b_ready[s], (i >> 1) & 1)) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll 4
          for (int kk = 0; kk < kTok / 16; ++kk) umma_ss(tm + TM_U, lm + kk * 128, cd + kk * 128, id_x, kk > 0 ? 1u : 0u);
#pragma unroll 4
          for (int kk = 0; kk < kTok / 16; ++kk) umma_ss(tm + TM_U, bd + kk * 128, cd + kk * 128, id_x, 1u);
          tc_commit(EXACT ? lo_read : &upd[s]);
        }
        __syncwarp();
        if constexpr (EXACT) {
          if (!warp_wait(lo2_ready, i & 1)) break;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll 4
            for (int kk = 0; kk < kTok / 16; ++kk) umma_ss(tm + TM_U, lm + kk * 128, cd + kk * 128, id_x, 1u);
            tc_commit(&upd[s]);
          }
          __syncwarp();
        }
      }
      if (elect_one()) {
        tc_commit(&drain[1]);
        mbar_drain(&drain[1], 0);
      }
      __syncwarp();
    } else {
      // y leaves from a's slot, which is free once the store has read it
      Chunks<REV> k(geo, p.N, c0, c1);
      for (int i = 0; i < n_chunks; ++i, k.next()) {
        const int s = i & 1, row = k.row(), bh = k.bh;
        if (!warp_wait(y_staged, i & 1)) break;
        if (elect_one()) {
#pragma unroll
          for (int c = 0; c < L::NCH; ++c) tma_store_3d(&tmY, smem + L::OFF_A + s * L::TILE + c * L::CHUNK, c * 64, row, bh);
          bulk_commit();
          bulk_wait_read_all();
          mbar_arrive(&a_empty[s]);
        }
        __syncwarp();
      }
      if (elect_one()) bulk_wait_all();
      __syncwarp();
    }
  } else {
    const int quad = warp & 3, row = quad * 32 + lane, st = threadIdx.x & 255;
    const uint32_t tq = tm + (static_cast<uint32_t>(quad * 32) << 16);
    if (warp < 12) {
      reg_dealloc<56>();
      // ---------------------------------------------------------- P
      // Row i = token, column j: times w^|i-j| from a table. Two tables take turns from head to head (no warp is
      // more than a chunk ahead of another); every warp writes all of a table, and the same numbers.
      Chunks<REV> k(geo, p.N, c0, c1);
      float* pw = reinterpret_cast<float*>(smem + L::OFF_POW);
      int heads = 0;
      const int wrow = quad * 32 + ((warp - 4) >> 2) * 16, j4 = lane & 3, ra = wrow + (lane >> 2);   // 16 rows a warp
      const uint32_t ta = tm + TM_A + (static_cast<uint32_t>(wrow) << 16);
      for (int i = 0; i < n_chunks; ++i, k.next()) {
        const int s = i & 1;
        if (i == 0 || k.first()) {
          const float g2 = log2_decay(p.log_decay, k.bh % p.H);
          pw = reinterpret_cast<float*>(smem + L::OFF_POW) + (heads++ & 1) * kPow + 32;
          for (int e = lane - 32; e < kTok; e += 32) pw[e] = e < 0 ? 0.f : fast_exp2(e * g2);
          __syncwarp();
        }
        if (!warp_wait(&a_done[s], (i >> 1) & 1)) break;
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < kTok; c += 32) {
          // (P's words take the columns of A that this warp has read by then)
          uint32_t w[8];
          if (rev ? c + 31 < wrow : c > wrow + 15) {
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = 0u;
          } else {
            uint32_t r[16];
            tmem_ld_16x256b_x4(ta + c, r);
            tmem_wait_ld();
            reg_fence16(r);
            const int d0 = rev ? c + 2 * j4 - ra : ra - c - 2 * j4;   // steps from token to token
#pragma unroll
            for (int e = 0; e < 8; ++e) {                             // columns 8 (e / 2), rows ra and ra + 8
              const int d = rev ? d0 + 8 * (e >> 1) - 8 * (e & 1) : d0 - 8 * (e >> 1) + 8 * (e & 1), d1 = rev ? d + 1 : d - 1;
              const float x0 = __uint_as_float(r[2 * e]) * pw[d], x1 = __uint_as_float(r[2 * e + 1]) * pw[d1];
              w[e] = pack_bf16x2(d >= 0 ? x0 : 0.f, d1 >= 0 ? x1 : 0.f);
            }
          }
          tmem_st_16x128b_x4(ta + c / 2, w);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_ready);
      }
    } else if (warp < 16) {
      reg_dealloc<48>();
      // ---------------------------------------------------------- y
      Chunks<REV> k(geo, p.N, c0, c1);
      float g2 = 0.f;
      for (int i = 0; i < n_chunks; ++i, k.next()) {
        const int s = i & 1;
        if (i == 0 || k.first()) g2 = log2_decay(p.log_decay, k.bh % p.H);
        const int steps = rev ? k.len() - 1 - row : row + 1;   // from the state to the token
        const float f1 = p.s_intra, f2 = steps >= 0 ? p.s_inter * fast_exp2(steps * g2) : 0.f;
        if (!warp_wait(y_full, i & 1)) break;
        tc_fence_after();
        uint8_t* stage = smem + L::OFF_A + s * L::TILE;
#pragma unroll 1
        for (int b = 0; b < D / 16; ++b) {
          uint32_t y1[16], y2[16];
          tmem_ld16(tq + TM_Y1 + 16 * b, y1);
          tmem_ld16(tq + TM_Y2 + 16 * b, y2);
          tmem_wait_ld();
          reg_fence16(y1);
          reg_fence16(y2);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int x = 8 * u + 2 * e;
              w[e] = pack_bf16x2(fmaf(__uint_as_float(y2[x]), f2, __uint_as_float(y1[x]) * f1),
                                 fmaf(__uint_as_float(y2[x + 1]), f2, __uint_as_float(y1[x + 1]) * f1));
            }
            *reinterpret_cast<uint4*>(stage + L::unit(row, 2 * b + u)) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
        tc_fence_before();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(y_empty);
          mbar_arrive(y_staged);
        }
      }
    } else if (warp < 24) {
      reg_alloc<96>();
      // ---------------------------------------------------------- the state (row: feature of b)
      // Two warps share a row's columns; the state is in their registers, so that its sums are rounded to nearest.
      uint8_t* sx = smem + L::OFF_X;
      const int col0 = ((warp - 16) >> 2) * (D / 2);
      float x[D / 2];
      const bool out = geo.whole && p.x_out;   // the states behind whole heads
      Chunks<REV> k(geo, p.N, c0, c1);
      float g = 0.f;
      float2 w = make_float2(0.f, 0.f);   // decay over the chunk before
      for (int i = 0; i < n_chunks + (out ? 1 : 0); ++i, k.next()) {
        if (i > 0) {
          if (!warp_wait(&upd[(i - 1) & 1], ((i - 1) >> 1) & 1)) break;
          if (quad * 32 < D) {   // X = w X + b'^T c
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < D / 2; c += 8) {
              uint32_t r[8];
              tmem_ld8_wait(tq + TM_U + col0 + c, r);
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float u = __uint_as_float(r[e]);
                if constexpr (EXACT) x[c + e] = decayed(x[c + e], w, u);
                else x[c + e] = fmaf(x[c + e], w.x, u);
              }
            }
            tc_fence_before();
          }
        }
        if (i == 0 || i == n_chunks || k.first()) {
          if (i > 0 && out && quad * 32 < D) {
            float* dst = p.x_out + (static_cast<long long>(k.bh + (rev ? 1 : -1)) * D + row) * D + col0;
#pragma unroll
            for (int e = 0; e < D / 2; e += 4) *reinterpret_cast<float4*>(dst + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
          }
          if (i == n_chunks) break;
          g = clamped(__ldg(p.log_decay + k.bh % p.H));
          const float* src = geo.whole ? (p.x_in ? p.x_in + static_cast<long long>(k.bh) * D * D : nullptr)
                                       : static_cast<const float*>(p.ws) + slot_of(geo, blockIdx.x, k.bh) * (D * D);
          if (!src || quad * 32 >= D) {
#pragma unroll
            for (int e = 0; e < D / 2; ++e) x[e] = 0.f;
          } else if (geo.whole ? p.in_t : p.slot_t) {
            src += col0 * D + row;
#pragma unroll
            for (int e = 0; e < D / 2; ++e) x[e] = src[e * D];
          } else {
            src += row * D + col0;
#pragma unroll
            for (int e = 0; e < D / 2; e += 4) {
              const float4 v = *reinterpret_cast<const float4*>(src + e);
              x[e] = v.x;
              x[e + 1] = v.y;
              x[e + 2] = v.z;
              x[e + 3] = v.w;
            }
          }
        }
        if (quad * 32 < D) {
#pragma unroll
          for (int u = 0; u < D / 16; ++u) {
            uint32_t v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = pack_bf16x2(x[8 * u + 2 * e], x[8 * u + 2 * e + 1]);
            const int un = col0 / 8 + u;
            *reinterpret_cast<uint4*>(sx + (un >> 3) * (D * 128) + row * 128 + (((un & 7) ^ (row & 7)) << 4)) =
                make_uint4(v[0], v[1], v[2], v[3]);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(x_ready);
        // (EXACT: a state that leaves the call; inside a range the one rounding of w is far below that of the bf16 copy)
        if constexpr (EXACT) w = decay_pair(k.len() * g);
        else w.x = fast_exp2(k.len() * (g * 1.4426950408889634f));
      }
    } else {
      // ---------------------------------------------------------- b'
      // Its high parts take b's place at once, its low parts the place of the state's copy once Y2 has read that.
      constexpr int RPP = L::rows(256), NP = L::passes(256);
      const int c = st % L::CPR, r0 = st / L::CPR;
      Chunks<REV> k(geo, p.N, c0, c1);
      float g2 = 0.f;
      for (int i = 0; i < n_chunks; ++i, k.next()) {
        const int s = i & 1;
        if (i == 0 || k.first()) g2 = log2_decay(p.log_decay, k.bh % p.H);
        if (!warp_wait(&a_done[s], (i >> 1) & 1)) break;
        uint8_t* sb = smem + L::OFF_B + s * L::TILE;
        uint8_t* sl = smem + L::OFF_X;
        uint4 lo[NP];   // EXACT: b as it was
        auto weight = [&](int r) {
          return r < k.len() ? fast_exp2(static_cast<float>(rev ? r + 1 : k.len() - 1 - r) * g2) * p.s_upd : 0.f;
        };
#pragma unroll
        for (int e = 0; e < NP; ++e) {
          const int r = r0 + e * RPP;
          uint4* b = reinterpret_cast<uint4*>(sb + L::unit(r, c));
          const uint4 x = *b;
          uint4 hi;
          split8(x, weight(r), hi, lo[e]);
          if constexpr (EXACT) lo[e] = x;
          *b = hi;
        }
        if (!warp_wait(x_read, i & 1)) break;
#pragma unroll
        for (int e = 0; e < NP; ++e) {
          uint4 l = lo[e], hi;
          if constexpr (EXACT) split8(lo[e], weight(r0 + e * RPP), hi, l);
          *reinterpret_cast<uint4*>(sl + L::unit(r0 + e * RPP, c)) = l;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&b_ready[s]);
        if constexpr (EXACT) {
          if (!warp_wait(lo_read, i & 1)) break;
#pragma unroll
          for (int e = 0; e < NP; ++e) {
            uint4 hi, l, l2;
            split8(lo[e], weight(r0 + e * RPP), hi, l, l2);
            *reinterpret_cast<uint4*>(sl + L::unit(r0 + e * RPP, c)) = l2;
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(lo2_ready);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tm, 512);
  }
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
  const float2 w = decay::decay_pair(decay::clamped(__ldg(log_decay + bh % H)));
  const uint2 vw = __ldg(reinterpret_cast<const uint2*>(v + base + strip * 32 + c4 * 4));
  const uint64_t v01 = f2_make(__uint_as_float(vw.x << 16), __uint_as_float(vw.x & 0xFFFF0000u));
  const uint64_t v23 = f2_make(__uint_as_float(vw.y << 16), __uint_as_float(vw.y & 0xFFFF0000u));
  const uint64_t wh = f2_make(w.x, w.x), wl = f2_make(w.y, w.y);
  uint64_t a01 = 0ull, a23 = 0ull;
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int row = r + 16 * i;
    const float kk = __bfloat162float(k[base + row]), qq = __bfloat162float(q[base + row]);
    const uint64_t k2 = f2_make(kk, kk), q2 = f2_make(qq, qq);
    uint64_t s01 = f2_make(s[i].x, s[i].y), s23 = f2_make(s[i].z, s[i].w);
    s01 = ffma2(s01, wh, ffma2(s01, wl, fmul2(k2, v01)));
    s23 = ffma2(s23, wh, ffma2(s23, wl, fmul2(k2, v23)));
    f2_split(s01, s[i].x, s[i].y);
    f2_split(s23, s[i].z, s[i].w);
    *reinterpret_cast<float4*>(state_out + so + static_cast<long long>(row) * D) = s[i];
    a01 = ffma2(q2, s01, a01);
    a23 = ffma2(q2, s23, a23);
  }
  float a0, a1, a2, a3;
  f2_split(a01, a0, a1);
  f2_split(a23, a2, a3);
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

size_t decay_ws_bytes(int BH, int N, int d) {
  const decay::Geom g = decay::decay_geom(BH, N);
  return g.whole ? 0 : static_cast<size_t>(g.grid) * g.hpc * d * d * sizeof(float);
}

template <int D>
static CUresult decay_map(CUtensorMap* m, const void* x, const DecayArgs& a) {
  return encode_tensor_map_3d_bf16(m, x, D, a.N, a.BH, 64, decay::kTok);
}

// The states that enter the ranges, in the workspace, and x_out.
template <int D, bool EXACT>
static cudaError_t launch_decay_states(const DecayArgs& a, const decay::Geom& g, cudaStream_t st) {
  using L = decay::StateLayout<D, EXACT>;
  CUtensorMap mb, mc;
  if (decay_map<D>(&mb, a.b, a) != CUDA_SUCCESS || decay_map<D>(&mc, a.c, a) != CUDA_SUCCESS) return cudaErrorInvalidValue;
  cudaError_t e = allow_smem<decay_state_kernel<D, EXACT>>(L::SMEM);
  if (e == cudaSuccess) e = launch_pdl(decay_state_kernel<D, EXACT>, dim3(g.grid), dim3(decay::kStateThreads), L::SMEM, st, mb, mc, a, g);
  if (e == cudaSuccess) e = launch_pdl(decay_join_kernel<D>, dim3(D * D / 1024, a.BH), dim3(256), 0, st, a, g);
  return e;
}

template <int D, bool REV, bool EXACT>
static cudaError_t launch_decay_chunks_d(const DecayArgs& a, const decay::Geom& g, cudaStream_t st) {
  using L = decay::ChunkLayout<D>;
  CUtensorMap ma, mb, mc, my;
  if (decay_map<D>(&ma, a.a, a) != CUDA_SUCCESS || decay_map<D>(&mb, a.b, a) != CUDA_SUCCESS ||
      decay_map<D>(&mc, a.c, a) != CUDA_SUCCESS || decay_map<D>(&my, a.y, a) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  cudaError_t e = allow_smem<decay_chunk_kernel<D, REV, EXACT>>(L::SMEM);
  if (e == cudaSuccess)
    e = launch_pdl(decay_chunk_kernel<D, REV, EXACT>, dim3(g.grid), dim3(decay::kThreads), L::SMEM, st, ma, mb, mc, my, a, g);
  return e;
}

template <int D>
static cudaError_t launch_decay_chunks(const DecayArgs& a, const decay::Geom& g, cudaStream_t st) {
  if (g.whole) return a.reverse ? launch_decay_chunks_d<D, true, true>(a, g, st) : launch_decay_chunks_d<D, false, true>(a, g, st);
  return a.reverse ? launch_decay_chunks_d<D, true, false>(a, g, st) : launch_decay_chunks_d<D, false, false>(a, g, st);
}

template <int D>
static cudaError_t launch_decay_d(DecayArgs a, const DecayArgs* same_state, cudaStream_t st) {
  const decay::Geom g = decay::decay_geom(a.BH, a.N);
  cudaError_t e = cudaSuccess;
  if (!g.whole) e = a.exact ? launch_decay_states<D, true>(a, g, st) : launch_decay_states<D, false>(a, g, st);
  if (e == cudaSuccess) e = launch_decay_chunks<D>(a, g, st);
  if (e == cudaSuccess && same_state) {
    DecayArgs b = *same_state;
    b.slot_t = 1;
    e = launch_decay_chunks<D>(b, g, st);
  }
  return e;
}

cudaError_t launch_decay(const DecayArgs& a, const DecayArgs* same_state, int d, cudaStream_t st) {
  return d == 64 ? launch_decay_d<64>(a, same_state, st) : launch_decay_d<128>(a, same_state, st);
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
