// cache_attn_kernel.cu — attention of new tokens over the paged cache:
//   o_i = sum_j softmax_j(scale q_i . k_j) v_j  over the cached positions j that
// token i of a chunk sees (all of them, or with `causal` those up to its own),
// query head h reading key/value head h / G.
//
// One kernel for single tokens, chunks and whole prompts. An item is a key head
// of a sequence and a tile of its new tokens: the G query heads that share the
// key head are rows of the same tile (row = token * G + head in the group, up to
// 128 rows), so a key or value is fetched once for all of them. A single token
// uses only G of the 128 rows; the tensor pipe is then far from its limit (the
// two products of a 128-key tile take 1024 cycles, the tile's 64 KB of bf16
// arrive in about 2800 at the memory's rate) and softmax warps whose rows hold
// no token skip their work, so a batch of single tokens is bound by the memory.
//
// Split of the work. A CTA per SM; the items' key ranges, each with kOver keys'
// worth of work for its start and end, are laid end to end and cut into equal
// parts, one per CTA. An item whose keys fall to several CTAs leaves partial
// results (unnormalised O, running maximum, sum) in the workspace, two slots per
// CTA at most (its first and its last item), which a second kernel joins in a
// fixed order. Long contexts of few rows thus occupy every SM, ragged batches
// balance, and no length has to be known on the host: every CTA finds its part
// from cu_q and kv_len itself (closed-form prefix sums, no list of items).
//
// Roles (as in the block-sparse kernel, which found the two MMA issuers and the
// 16-lane softmax layout by measurement):
//   warp 0       walks the items, posts their facts, loads Q and K tiles by TMA
//   warp 1       issues S = Q K^T
//   warp 2       loads V tiles by TMA (8-bit: K and V codes go into a ring of their
//                own)
//   warp 3       issues O += P V
//   warps 4..11  softmax: 16 rows a warp, 128 columns
//   warps 12..19 8-bit only: codes to fp16 (exact for E4M3 and int8, and one
//                instruction for two codes where bf16 takes five), written as the
//                swizzled tiles that the products read; q to fp16 likewise. Scales
//                stay out of the products: the key's multiplies its score column,
//                the value's its weight.
// fp16 and its range (8-bit caches). A row of q is scaled by a power of two so that
// its largest value lies in [2^13, 2^14) (or below, where that power times the score
// scale would leave fp32): q's 8 bits are exact in fp16's 11 down to
// 2^-28 of that, and what is lost below is under 2^-38 of it. A weight times its
// value's scale is held relative to C, the power of two at or above the largest
// scale of the keys so far (raised like the running maximum, O following), times
// 2^7: at most 2^15, and with all 11 bits down to 2^-21 of a weight of 1 at C.
// Measured (d = 128): 64 single tokens over up to 8,192 bf16 keys 243 us, 0.96 of the
// memory's rate; 48 tokens over up to 32,768 E4M3 keys 353 us, 0.48 of it (the turning
// of codes); 4,680 tokens over 32,760 keys 820 us alone, 0.70 of the tensor pipe's burst
// rate, and 920 to 960 us called back to back under the power cap, 0.60 to 0.62 of it
// (0.70 to 0.73 of the sustained one).
// Pages are fetched in boxes of the largest power of two of rows that divides the
// page (128 at most), so a page may end anywhere in a tile. A table entry that
// names no page is fetched from outside the tensor, which fills zeros.
//
// Keys behind the last visible one of an item: their score columns are replaced
// by -inf whatever they hold, and their value rows (which may be NaN: unused
// cache) are not part of the product except the rest of the last group of 16
// rows, which is zeroed in shared memory first.
#include <algorithm>

#include <cuda_fp16.h>

#include "sa_internal.h"

namespace sa {

namespace cattn {

constexpr int kBM = 128;
constexpr int kBN = 128;
constexpr int kSBufs = 3;
constexpr int kItemRing = 4;
constexpr int kRingWords = 12;
constexpr int kSoftWarps = 8;
constexpr int kSoft0 = 4;         // first softmax warp
constexpr int kDeq0 = 12;         // first dequantising warp
constexpr int kDeqWarps = 8;      // four for keys, four for values
// Work of an item besides its keys, in keys (start, drain and store of its rows).
constexpr int kOver = 128;
// Least work of a CTA, in keys: below, fewer CTAs share the call.
constexpr int kMinKeys = 256;
constexpr int kMaxCtas = 160;
// Blocks at most that share the join of an item (one block alone took 7 us longer over tiles of 126 rows).
constexpr int kJoinY = 4;
constexpr uint32_t kPolyPairs = 0x88u;   // exponentials on the FMA pipe, as in the block-sparse kernel

template <int D, int KIND>
struct Layout {
  static constexpr bool Q8 = KIND != kCacheBf16;
  static constexpr int THREADS = Q8 ? 640 : 384;
  static constexpr int NCH = D / 64;                       // 128-byte chunks of a bf16 row
  static constexpr uint32_t CHUNK = 128 * 128;             // bytes of a chunk of 128 rows
  static constexpr uint32_t TILE = NCH * CHUNK;            // Q, K or V tile in bf16
  static constexpr uint32_t RAW = 128 * D;                 // codes of a K or V tile
  static constexpr int QS = (Q8 && D == 128) ? 1 : 2;
  static constexpr int KST = (!Q8) ? 3 : 2;
  static constexpr int VST = (!Q8 && D == 64) ? 3 : 2;
  static constexpr int RST = Q8 ? (D == 128 ? 3 : 6) : 0;
  static constexpr uint32_t OFF_Q = 0;
  static constexpr uint32_t OFF_K = OFF_Q + QS * TILE;
  static constexpr uint32_t OFF_V = OFF_K + KST * TILE;
  static constexpr uint32_t OFF_RAW = OFF_V + VST * TILE;
  static constexpr uint32_t OFF_SC = OFF_RAW + RST * RAW;  // key and value scales [kSBufs][2][128] fp32
  static constexpr uint32_t OFF_QSC = OFF_SC + (Q8 ? kSBufs * 2 * 128 * 4 : 0);   // 2^-k of q's rows [kItemRing][128]
  static constexpr uint32_t OFF_VMAX = OFF_QSC + (Q8 ? kItemRing * 128 * 4 : 0);  // largest value scales [kSBufs][4]
  static constexpr uint32_t OFF_BASE = OFF_VMAX + (Q8 ? 64 : 0);                  // rows of a key tile's boxes [RST][8]
  static constexpr uint32_t OFF_BAR = OFF_BASE + RST * 8 * 4;
  static constexpr uint32_t OFF_RING = OFF_BAR + 512;
  static constexpr uint32_t USED = OFF_RING + kItemRing * kRingWords * 4;
  // more than half of the SM's shared memory, so that a CTA (which takes all of the tensor memory) is alone
  static constexpr uint32_t SMEM = (USED + 1024 > 120 * 1024) ? USED + 1024 : 120 * 1024;
  static_assert(SMEM <= 227 * 1024, "shared memory per CTA");
  static_assert(KST <= kSBufs && VST <= kSBufs, "slots are freed by barriers indexed by S buffer");
};

__host__ __device__ constexpr uint32_t tm_s(int b) { return static_cast<uint32_t>(b) * 128u; }
constexpr uint32_t TM_O = 384;
constexpr uint32_t TM_COLS = 512;

enum {
  B_QFULL = 0,                 // [2]
  B_QEMPTY = B_QFULL + 2,      // [2]
  B_KFULL = B_QEMPTY + 2,      // [3]
  B_VFULL = B_KFULL + 3,       // [3]
  // Codes of a tile landed, and read: [6] for key tiles, [6] for value tiles each. A stage of the ring holds tiles of
  // both kinds in turn (3 stages) or of one (6), r = 2 tile + kind in stage r % RST. With one barrier a warp could ask
  // for a phase whose predecessor it has not seen end, and a parity cannot tell that phase from the last but one; a
  // kind's own barrier completes once in six tiles, and whoever waits for it waits for every phase.
  B_RFULL = B_VFULL + 3,
  B_REMPTY = B_RFULL + 12,
  B_SFULL = B_REMPTY + 12,      // [kSBufs] S ready, the K slot free
  B_PFULL = B_SFULL + kSBufs,  // [kSBufs]
  B_PVDONE = B_PFULL + kSBufs, // [kSBufs] O updated, the S buffer and V slot free
  B_OFULL = B_PVDONE + kSBufs,
  B_OEMPTY = B_OFULL + 1,
  B_IFULL = B_OEMPTY + 1,      // [kItemRing]
  B_IEMPTY = B_IFULL + kItemRing,
  B_DRAIN = B_IEMPTY + kItemRing,   // [2]
  B_QREADY = B_DRAIN + 2,           // [2] q in fp16 (8-bit)
  B_COUNT = B_QREADY + 2
};
static_assert(B_COUNT * 8 + 8 <= 512, "barrier region");

// ---------------------------------------------------------------- the plan
// Facts of a sequence: its first row, new rows n, cached tokens L, query tiles.
struct Seq {
  int row0, n, L, nqt;
};

__device__ __forceinline__ Seq load_seq(const CacheAttnArgs& a, int tpt, int s) {
  Seq q;
  const int r0 = min(max(__ldg(a.cu_q + s), 0), a.n_rows);
  const int r1 = min(max(__ldg(a.cu_q + s + 1), r0), a.n_rows);
  q.row0 = r0;
  q.n = r1 - r0;
  q.L = static_cast<int>(min(max(static_cast<long long>(__ldg(a.kv_len + s)), 0ll), static_cast<long long>(a.width) * a.page));
  q.nqt = (q.n + tpt - 1) / tpt;
  return q;
}

// Work of the first m query tiles of a key head (m < nqt): kOver and the visible
// keys of the last token of each, max(0, L - n + (i + 1) tpt) with `causal`.
__device__ __forceinline__ long long prefix_work(const CacheAttnArgs& a, int tpt, const Seq& q, int m) {
  if (!a.causal) return static_cast<long long>(m) * (q.L + kOver);
  const long long c = q.L - q.n;
  long long m0 = 0;                                        // tiles that see nothing
  if (c < 0) m0 = min(static_cast<long long>(m), -c / tpt);
  const long long mm = m;
  return (mm - m0) * c + tpt * (mm * (mm + 1) - m0 * (m0 + 1)) / 2 + mm * kOver;
}

__device__ __forceinline__ long long head_work(const CacheAttnArgs& a, int tpt, const Seq& q) {
  return q.n == 0 ? 0 : prefix_work(a, tpt, q, q.nqt - 1) + q.L + kOver;
}

struct Item {
  int s, h, qt;
  int kend;       // keys of the item: the last token's visible ones
  int T;          // its tiles (at least one, so that rows that see nothing are written too)
  int tok0, ntok;
};

__device__ __forceinline__ Item make_item(const CacheAttnArgs& a, int tpt, const Seq& q, int s, int h, int qt) {
  Item it;
  it.s = s;
  it.h = h;
  it.qt = qt;
  it.tok0 = qt * tpt;
  it.ntok = min(tpt, q.n - it.tok0);
  it.kend = a.causal ? max(0, q.L - q.n + it.tok0 + it.ntok) : q.L;
  it.T = max(1, (it.kend + kBN - 1) / kBN);
  return it;
}

__device__ __forceinline__ long long item_work(const CacheAttnArgs& a, const Item& it) { return static_cast<long long>(it.kend) + kOver; }

// Total work W, how many CTAs share it (ctas), the part [k0, k1) of CTA c, and
// the item that covers offset k0 with its first offset.
struct Plan {
  long long W, k0, k1, base;
  int ctas, s, h, qt;
  long long red[20];
};

template <int NT>
__device__ __forceinline__ void make_plan(const CacheAttnArgs& a, int tpt, int c, int grid, Plan* sp) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.n_seqs + NT - 1) / NT;
  const int s0 = min(a.n_seqs, tid * per), s1 = min(a.n_seqs, s0 + per);
  long long own = 0;
#pragma unroll 1
  for (int s = s0; s < s1; ++s) own += a.H * head_work(a, tpt, load_seq(a, tpt, s));
  long long inc = own;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long v = __shfl_up_sync(0xFFFFFFFFu, inc, d);
    if (lane >= d) inc += v;
  }
  if (lane == 31) sp->red[warp] = inc;
  if (tid == 0) sp->s = -1;
  __syncthreads();
  long long W = 0, before = 0;
#pragma unroll 1
  for (int w = 0; w < NT / 32; ++w) {
    if (w == warp) before = W;
    W += sp->red[w];
  }
  before += inc - own;
  const int ctas = static_cast<int>(max(1ll, min(static_cast<long long>(grid), W / kMinKeys)));
  const long long k0 = c < ctas ? W * c / ctas : W, k1 = c < ctas ? W * (c + 1) / ctas : W;
  if (tid == 0) {
    sp->W = W;
    sp->k0 = k0;
    sp->k1 = k1;
    sp->ctas = ctas;
  }
  const long long x = k0;
  if (k0 < k1 && x >= before && x < before + own) {
    long long at = before;
#pragma unroll 1
    for (int s = s0; s < s1; ++s) {
      const Seq q = load_seq(a, tpt, s);
      const long long hw = head_work(a, tpt, q), all = a.H * hw;
      if (x < at + all) {
        const int h = static_cast<int>((x - at) / hw);
        const long long rem = x - at - h * hw;
        int lo = 0, hi = q.nqt - 1;                          // the last tile whose work begins at or before rem
#pragma unroll 1
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (prefix_work(a, tpt, q, mid) <= rem) lo = mid;
          else hi = mid - 1;
        }
        sp->s = s;
        sp->h = h;
        sp->qt = lo;
        sp->base = x - rem + prefix_work(a, tpt, q, lo);
        break;
      }
      at += all;
    }
  }
  __syncthreads();
}

// First tile of an item (first offset `base`) whose start lies at or behind k.
__device__ __forceinline__ int first_tile(long long base, long long k) {
  return k <= base ? 0 : static_cast<int>((k - base + kBN - 1) / kBN);
}

// Partial results of a CTA's first (0) and last (1) item.
template <int D>
__device__ __forceinline__ float* slot_o(const CacheAttnArgs& a, int slot) {
  return static_cast<float*>(a.ws) + static_cast<long long>(slot) * kBM * D;
}
template <int D>
__device__ __forceinline__ float2* slot_ml(const CacheAttnArgs& a, int slot) {
  return reinterpret_cast<float2*>(static_cast<float*>(a.ws) + 2ll * kMaxCtas * kBM * D) + slot * kBM;
}

// The item that a CTA began and did not finish, for the second kernel (rows 0: none).
struct Begun {
  long long base, W;   // its first offset; the work of the call
  int ctas, tiles;     // CTAs that share it; the item's tiles
  int row0, rows, h;   // its first row, rows of its tile (tokens times G), key head
  int vis0;            // keys that its first token sees
};
template <int D>
__device__ __forceinline__ Begun* begun(const CacheAttnArgs& a, int cta) {
  return reinterpret_cast<Begun*>(static_cast<float*>(a.ws) + 2ll * kMaxCtas * kBM * (D + 2)) + cta;
}

// Two codes (the low or the high two bytes of w) as fp16, exactly. int8: with its
// top bit turned a code u is value + 128, 0x6400 | u is 1024 + u.
template <int KIND, int HI>
__device__ __forceinline__ uint32_t decode2(uint32_t w) {
  if constexpr (KIND == kCacheE4m3) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(HI ? w >> 16 : w & 0xFFFFu), __NV_E4M3);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const uint32_t x = __byte_perm(w ^ 0x80808080u, 0x64646464u, HI ? 0x4342 : 0x4140);
    const uint32_t off = 0x64806480u;   // 1152
    const __half2 v = __hsub2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&off));
    return *reinterpret_cast<const uint32_t*>(&v);
  }
}

// 2^ceil(log2 x) of a positive x.
__device__ __forceinline__ float pow2_above(float x) { return __uint_as_float((__float_as_uint(x) + 0x007FFFFFu) & 0x7F800000u); }
constexpr float kMinC = 7.52316385e-37f;   // 2^-120: 2^7 / C stays finite

}  // namespace cattn

template <int D, int KIND>
__global__ void __launch_bounds__(cattn::Layout<D, KIND>::THREADS, 1)
    cache_attn_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CacheAttnArgs a, int tpt, int box_rows) {
  using namespace cattn;
  using L = Layout<D, KIND>;
  constexpr bool Q8 = L::Q8;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Plan plan;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem + L::OFF_Q;
  uint8_t* sK = smem + L::OFF_K;
  uint8_t* sV = smem + L::OFF_V;
  uint8_t* sR = smem + L::OFF_RAW;
  float* sSc = reinterpret_cast<float*>(smem + L::OFF_SC);
  float* sQsc = reinterpret_cast<float*>(smem + L::OFF_QSC);
  float* sVmax = reinterpret_cast<float*>(smem + L::OFF_VMAX);
  volatile int* sBase = reinterpret_cast<volatile int*>(smem + L::OFF_BASE);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + B_COUNT);
  // facts of an item: [0] 1 (0: no more), [1] sequence, [2] key head, [3] first and [4] last-but-one-past tile,
  // [5] keys, [6] first row, [7] rows' tokens, [8] keys the first token sees, [9] 0 whole, 1 / 2 partial in slot 0 / 1,
  // [10] keys that no token goes beyond
  volatile int* ring = reinterpret_cast<volatile int*>(smem + L::OFF_RING);

  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  // a warp's wait (all lanes poll: with one of them polling apart from the others every wait cost some hundred cycles more)
  const auto warp_wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait_asleep(bar, parity, a.wait_tries); };
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars[B_QFULL + i], 1);
      mbar_init(&bars[B_QEMPTY + i], 1);
      mbar_init(&bars[B_DRAIN + i], 1);
      mbar_init(&bars[B_QREADY + i], kDeqWarps);
    }
    for (int i = 0; i < 3; ++i) {
      mbar_init(&bars[B_KFULL + i], Q8 ? kDeqWarps / 2 : 1);
      mbar_init(&bars[B_VFULL + i], Q8 ? kDeqWarps / 2 : 1);
    }
    for (int i = 0; i < 6; ++i) {
      mbar_init(&bars[B_RFULL + i], 1);
      mbar_init(&bars[B_RFULL + 6 + i], 1);
      mbar_init(&bars[B_REMPTY + i], kDeqWarps / 2);
      mbar_init(&bars[B_REMPTY + 6 + i], kDeqWarps / 2);
    }
    for (int i = 0; i < kSBufs; ++i) {
      mbar_init(&bars[B_SFULL + i], 1);
      mbar_init(&bars[B_PFULL + i], kSoftWarps);
      mbar_init(&bars[B_PVDONE + i], 1);
    }
    mbar_init(&bars[B_OFULL], 1);
    mbar_init(&bars[B_OEMPTY], kSoftWarps);
    for (int i = 0; i < kItemRing; ++i) {
      mbar_init(&bars[B_IFULL + i], 1);
      // readers: the two issuers, the V loader, the softmax warps and those that turn codes
      mbar_init(&bars[B_IEMPTY + i], 3 + kSoftWarps + (Q8 ? kDeqWarps : 0));
    }
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, TM_COLS);
    tmem_relinquish();
  }
  grid_dep_wait();
  grid_dep_trigger();
  tc_fence_before();
  make_plan<L::THREADS>(a, tpt, blockIdx.x, gridDim.x, &plan);   // (ends with a barrier of the block)
  tc_fence_after();
  const uint32_t tm = __shfl_sync(0xFFFFFFFFu, *tmem_slot, 0);

  if (warp < kSoft0) {
    // 8-bit, registers a thread: 32 (4 x 56 + 8 x 152 + 8 x 56) = 60416 of the launch's 640 x 96 = 61440
    if constexpr (Q8) reg_dealloc<56>();
    if (warp == 0) {
      // ---------------------------------------------------------- items, Q, K (8-bit: codes)
      if (lane == 0) {
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmK);
      }
      bool ok = true;
      int qi = 0, g = 0, q_armed = 0;
      const long long k1 = plan.k1;
      Begun left{};
      if (plan.s >= 0) {
        int s = plan.s;
        Seq sq = load_seq(a, tpt, s);
        Item it = make_item(a, tpt, sq, s, plan.h, plan.qt);
        long long base = plan.base;
        int t0 = first_tile(base, plan.k0);
        while (ok && base < k1) {
          const int t1 = min(it.T, first_tile(base, k1));
          if (t0 < t1) {
            const int rs = qi % kItemRing;
            if (!(ok = warp_wait(&bars[B_IEMPTY + rs], ((qi / kItemRing) & 1) ^ 1))) break;
            if (lane == 0) {
              volatile int* f = ring + rs * kRingWords;
              f[0] = 1;
              f[1] = s;
              f[2] = it.h;
              f[3] = t0;
              f[4] = t1;
              f[5] = it.kend;
              f[6] = sq.row0 + it.tok0;
              f[7] = it.ntok;
              f[8] = a.causal ? sq.L - sq.n + it.tok0 + 1 : sq.L;
              f[9] = t0 > 0 ? 1 : (t1 < it.T ? 2 : 0);
              if (t0 == 0 && t1 < it.T) left = {base, plan.W, plan.ctas, it.T, f[6], it.ntok * a.G, it.h, f[8]};
              f[10] = sq.L;
              mbar_arrive(&bars[B_IFULL + rs]);
            }
            const int qs = qi % L::QS;
            if (!(ok = warp_wait(&bars[B_QEMPTY + qs], ((qi / L::QS) & 1) ^ 1))) break;
            if (lane == 0) {
              mbar_arrive_expect_tx(&bars[B_QFULL + qs], L::NCH * 128u * a.G * tpt);
              for (int c = 0; c < L::NCH; ++c)
                tma_load_4d(sQ + qs * L::TILE + c * L::CHUNK, &tmQ, &bars[B_QFULL + qs], c * 64, 0, sq.row0 + it.tok0, it.h);
            }
            q_armed = qi + 1;
            // boxes of this item's tiles: the table's entries 32 boxes at a time, one per lane
            const int per_tile = kBN / box_rows;
            const int n_box = (it.kend + box_rows - 1) / box_rows;
            const int* row = a.table + static_cast<long long>(s) * a.width;
            int have = -1, my_plane = 0, my_off = 0;
            for (int t = t0; t < t1; ++t, ++g) {
              const int b0 = t * per_tile, nb = min(per_tile, max(n_box - b0, 0));
              if (b0 / 32 != have) {
                have = b0 / 32;
                const int key = (have * 32 + lane) * box_rows;
                my_plane = a.n_pages * a.H;   // outside the tensor: zeros
                my_off = 0;
                if (key < it.kend) {
                  const int pg = __ldg(row + key / a.page);
                  if (pg >= 0 && pg < a.n_pages) my_plane = pg * a.H + it.h;
                  my_off = key % a.page;
                }
              }
              if constexpr (!Q8) {
                const int ks = g % L::KST;
                if (g >= L::KST) {
                  const int gp = g - L::KST;
                  if (!(ok = warp_wait(&bars[B_SFULL + gp % kSBufs], (gp / kSBufs) & 1))) break;
                }
                if (lane == 0) mbar_arrive_expect_tx(&bars[B_KFULL + ks], nb * box_rows * D * 2u);
                __syncwarp();
                for (int i0 = 0; i0 < nb * L::NCH; i0 += 32) {
                  const int i = i0 + lane, b = i / L::NCH, c = i % L::NCH;
                  const int src = (b0 + b) & 31;
                  const int plane = __shfl_sync(0xFFFFFFFFu, my_plane, src), off = __shfl_sync(0xFFFFFFFFu, my_off, src);
                  if (i < nb * L::NCH)
                    tma_load_3d(sK + ks * L::TILE + c * L::CHUNK + b * box_rows * 128, &tmK, &bars[B_KFULL + ks], c * 64, off, plane);
                }
              } else {
                const int r = 2 * g, ss = r % L::RST, pr = r - L::RST;
                if (pr >= 0 && !(ok = warp_wait(&bars[B_REMPTY + 6 * (pr & 1) + ss], (pr / 6) & 1))) break;
                const int src = (b0 + lane) & 31;
                const int plane = __shfl_sync(0xFFFFFFFFu, my_plane, src), off = __shfl_sync(0xFFFFFFFFu, my_off, src);
                // the cache row of each box, for the scales; -1 without a page
                if (lane < per_tile) sBase[ss * 8 + lane] = lane < nb && plane < a.n_pages * a.H ? plane * a.page + off : -1;
                __syncwarp();
                if (lane == 0) mbar_arrive_expect_tx(&bars[B_RFULL + ss], box_rows * nb * static_cast<uint32_t>(D));
                __syncwarp();
                if (lane < nb) tma_load_3d(sR + ss * L::RAW + lane * box_rows * D, &tmK, &bars[B_RFULL + ss], 0, off, plane);
              }
            }
            ++qi;
          }
          if (!ok) break;
          // next item
          base += item_work(a, it);
          t0 = 0;
          int h = it.h, qt = it.qt + 1;
          if (qt == sq.nqt) {
            qt = 0;
            if (++h == a.H) {
              h = 0;
              if (base >= k1) break;
              do {
                if (++s >= a.n_seqs) break;
                sq = load_seq(a, tpt, s);
              } while (sq.n == 0);
              if (s >= a.n_seqs) break;
            }
          }
          it = make_item(a, tpt, sq, s, h, qt);
        }
      }
      if (lane == 0) *begun<D>(a, blockIdx.x) = left;
      if (ok) {
        const int rs = qi % kItemRing;
        if (warp_wait(&bars[B_IEMPTY + rs], ((qi / kItemRing) & 1) ^ 1) && lane == 0) {
          ring[rs * kRingWords] = 0;
          mbar_arrive(&bars[B_IFULL + rs]);
        }
      }
      if (lane == 0) {
        // loads in flight land before the CTA gives up its shared memory (g counts what was armed)
        if constexpr (!Q8) {
          for (int i = 1; i <= L::KST && i <= g; ++i) mbar_drain(&bars[B_KFULL + (g - i) % L::KST], ((g - i) / L::KST) & 1);
        } else {
          for (int t = max(0, g - 3); t < g; ++t) mbar_drain(&bars[B_RFULL + 2 * t % L::RST], (2 * t / 6) & 1);
        }
        for (int i = 1; i <= L::QS && i <= q_armed; ++i)
          mbar_drain(&bars[B_QFULL + (q_armed - i) % L::QS], ((q_armed - i) / L::QS) & 1);
      }
    } else if (warp == 2) {
      // ---------------------------------------------------------- V (8-bit: codes)
      if (lane == 0) tma_prefetch_desc(&tmV);
      bool ok = true;
      int qi = 0, g = 0;
      while (ok) {
        const int rs = qi % kItemRing;
        if (!(ok = warp_wait(&bars[B_IFULL + rs], (qi / kItemRing) & 1))) break;
        volatile int* f = ring + rs * kRingWords;
        const int more = f[0], s = f[1], h = f[2], t0 = f[3], t1 = f[4], kend = f[5];
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[B_IEMPTY + rs]);
        if (!more) break;
        const int per_tile = kBN / box_rows;
        const int n_box = (kend + box_rows - 1) / box_rows;
        const int* row = a.table + static_cast<long long>(s) * a.width;
        int have = -1, my_plane = 0, my_off = 0;
        for (int t = t0; t < t1; ++t, ++g) {
          const int b0 = t * per_tile, nb = min(per_tile, max(n_box - b0, 0));
          if (b0 / 32 != have) {
            have = b0 / 32;
            const int key = (have * 32 + lane) * box_rows;
            my_plane = a.n_pages * a.H;
            my_off = 0;
            if (key < kend) {
              const int pg = __ldg(row + key / a.page);
              if (pg >= 0 && pg < a.n_pages) my_plane = pg * a.H + h;
              my_off = key % a.page;
            }
          }
          if constexpr (!Q8) {
            const int vs = g % L::VST;
            if (g >= L::VST) {
              const int gp = g - L::VST;
              if (!(ok = warp_wait(&bars[B_PVDONE + gp % kSBufs], (gp / kSBufs) & 1))) break;
            }
            if (lane == 0) mbar_arrive_expect_tx(&bars[B_VFULL + vs], nb * box_rows * D * 2u);
            __syncwarp();
            for (int i0 = 0; i0 < nb * L::NCH; i0 += 32) {
              const int i = i0 + lane, b = i / L::NCH, c = i % L::NCH;
              const int src = (b0 + b) & 31;
              const int plane = __shfl_sync(0xFFFFFFFFu, my_plane, src), off = __shfl_sync(0xFFFFFFFFu, my_off, src);
              if (i < nb * L::NCH)
                tma_load_3d(sV + vs * L::TILE + c * L::CHUNK + b * box_rows * 128, &tmV, &bars[B_VFULL + vs], c * 64, off, plane);
            }
          } else {
            const int r = 2 * g + 1, ss = r % L::RST, pr = r - L::RST;
            if (pr >= 0 && !(ok = warp_wait(&bars[B_REMPTY + 6 * (pr & 1) + ss], (pr / 6) & 1))) break;
            const int src = (b0 + lane) & 31;
            const int plane = __shfl_sync(0xFFFFFFFFu, my_plane, src), off = __shfl_sync(0xFFFFFFFFu, my_off, src);
            if (lane == 0) mbar_arrive_expect_tx(&bars[B_RFULL + 6 + ss], box_rows * nb * static_cast<uint32_t>(D));
            __syncwarp();
            if (lane < nb) tma_load_3d(sR + ss * L::RAW + lane * box_rows * D, &tmV, &bars[B_RFULL + 6 + ss], 0, off, plane);
          }
        }
        ++qi;
      }
      if (lane == 0) {
        if constexpr (!Q8) {
          for (int i = 1; i <= L::VST && i <= g; ++i) mbar_drain(&bars[B_VFULL + (g - i) % L::VST], ((g - i) / L::VST) & 1);
        } else {
          for (int t = max(0, g - 3); t < g; ++t) mbar_drain(&bars[B_RFULL + 6 + (2 * t + 1) % L::RST], ((2 * t + 1) / 6) & 1);
        }
      }
    } else if (warp == 1) {
      // ---------------------------------------------------------- S = Q K^T
      const uint64_t qdesc0 = sw128_desc(smem_u32(sQ), 16, 1024);
      const uint64_t kdesc0 = sw128_desc(smem_u32(sK), 16, 1024);
      const uint32_t idesc = Q8 ? idesc_f16_f32(kBM, kBN, false, false) : idesc_bf16_f32(kBM, kBN, false, false);
      int g = 0, qi = 0;
      bool ok = true;
      while (ok) {
        const int rs = qi % kItemRing;
        if (!(ok = warp_wait(&bars[B_IFULL + rs], (qi / kItemRing) & 1))) break;
        volatile int* f = ring + rs * kRingWords;
        const int more = f[0], n = f[4] - f[3], qs = qi % L::QS;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[B_IEMPTY + rs]);
        if (!more) break;
        if (!(ok = warp_wait(&bars[(Q8 ? B_QREADY : B_QFULL) + qs], (qi / L::QS) & 1))) break;
        for (int t = 0; t < n; ++t, ++g) {
          const int b = g % kSBufs, ks = g % L::KST;
          if (g >= kSBufs && !(ok = warp_wait(&bars[B_PVDONE + b], ((g / kSBufs) & 1) ^ 1))) break;
          if (!(ok = warp_wait(&bars[B_KFULL + ks], (g / L::KST) & 1))) break;
          tc_fence_after();
          const uint64_t qd = qdesc0 + ((qs * L::TILE) >> 4), kd = kdesc0 + ((ks * L::TILE) >> 4);
          const uint32_t ts = tm + tm_s(b);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = (((kk >> 2) * L::CHUNK) + (kk & 3) * 32u) >> 4;
              umma_ss(ts, qd + off, kd + off, idesc, kk > 0 ? 1u : 0u);
            }
            tc_commit(&bars[B_SFULL + b]);
            if (t + 1 == n) tc_commit(&bars[B_QEMPTY + qs]);
          }
          __syncwarp();
        }
        ++qi;
      }
      if (elect_one()) {
        tc_commit(&bars[B_DRAIN]);
        mbar_drain(&bars[B_DRAIN], 0);
      }
      __syncwarp();
    } else {
      // ---------------------------------------------------------- O += P V
      const uint64_t vdesc0 = sw128_desc(smem_u32(sV), L::CHUNK, 1024);
      const uint32_t idesc = Q8 ? idesc_f16_f32(kBM, D, false, true) : idesc_bf16_f32(kBM, D, false, true);
      int g = 0, qi = 0;
      bool ok = true;
      while (ok) {
        const int rs = qi % kItemRing;
        if (!(ok = warp_wait(&bars[B_IFULL + rs], (qi / kItemRing) & 1))) break;
        volatile int* f = ring + rs * kRingWords;
        const int more = f[0], t0 = f[3], t1 = f[4], kend = f[5];
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[B_IEMPTY + rs]);
        if (!more) break;
        for (int t = t0; t < t1; ++t, ++g) {
          const int b = g % kSBufs, vs = g % L::VST;
          if (!(ok = warp_wait(&bars[B_PFULL + b], (g / kSBufs) & 1))) break;
          if (!(ok = warp_wait(&bars[B_VFULL + vs], (g / L::VST) & 1))) break;
          if (t == t0 && !(ok = warp_wait(&bars[B_OEMPTY], (qi & 1) ^ 1))) break;
          tc_fence_after();
          const int nk = (min(kBN, max(kend - t * kBN, 0)) + 15) / 16;   // groups of 16 keys
          const uint64_t vd = vdesc0 + ((vs * L::TILE) >> 4);
          const uint32_t ts = tm + tm_s(b);
          const uint32_t more_o = t > t0 ? 1u : 0u;
          if (elect_one()) {
            if (nk == kBN / 16) {
#pragma unroll
              for (int kk = 0; kk < kBN / 16; ++kk) umma_ts(tm + TM_O, ts + kk * 8, vd + kk * 128, idesc, kk > 0 ? 1u : more_o);
            } else {
#pragma unroll 1
              for (int kk = 0; kk < nk; ++kk) umma_ts(tm + TM_O, ts + kk * 8, vd + kk * 128, idesc, kk > 0 ? 1u : more_o);
            }
            tc_commit(&bars[B_PVDONE + b]);
            if (t + 1 == t1) tc_commit(&bars[B_OFULL]);
          }
          __syncwarp();
        }
        ++qi;
      }
      if (elect_one()) {
        tc_commit(&bars[B_DRAIN + 1]);
        mbar_drain(&bars[B_DRAIN + 1], 0);
      }
      __syncwarp();
    }
  } else if (Q8 && warp >= kDeq0) {
    if constexpr (Q8) {
      // ---------------------------------------------------------- q and codes to fp16
      reg_dealloc<56>();
      const int dt = threadIdx.x - kDeq0 * 32;               // 0..255
      constexpr int CPR = D / 16;                            // 16-byte pieces of a row of codes
      constexpr int RPP = 128 / CPR;                         // rows a pass (four warps)
      const int kv = dt >> 7, c = dt % CPR, r0 = (dt & 127) / CPR;
      // the two 16-byte units of a piece; lanes of the other 128-byte chunk store them the other way round, so that
      // the eight lanes of a row hit eight units of the 128 bytes
      const int first = (c >> 2) & 1, u0 = 2 * (c & 3);
      const int off0 = ((u0 + first) ^ (r0 & 7)) << 4, off1 = ((u0 + 1 - first) ^ (r0 & 7)) << 4;
      bool ok = true;
      int qi = 0, g = 0;
      while (ok) {
        const int rs = qi % kItemRing;
        if (!(ok = warp_wait(&bars[B_IFULL + rs], (qi / kItemRing) & 1))) break;
        volatile int* f = ring + rs * kRingWords;
        const int more = f[0], t0 = f[3], t1 = f[4], kend = f[5], rows = f[7] * a.G;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[B_IEMPTY + rs]);
        if (!more) break;
        {
          // q's rows in place: D / 8 threads a row, 16 bytes each
          const int qs = qi % L::QS;
          if (!(ok = warp_wait(&bars[B_QFULL + qs], (qi / L::QS) & 1))) break;
          constexpr int QPR = D / 8;
          const int qc = dt % QPR;
          // scale_log2 2^-k stays a normal number (a factor of 0 would make masked scores NaN). A row whose k this cuts
          // loses 2^-25 of 2^-k a channel, which with that factor is below 2^-150 of a key's size: no score.
          const int k_max = min(static_cast<int>(__float_as_uint(a.scale_log2) >> 23) - 1, 126);
#pragma unroll 1
          for (int r1 = 0; r1 < rows; r1 += 32 * kDeqWarps / QPR) {
            const int qr = r1 + dt / QPR;                    // (up to 127: a whole pass lies in the tile)
            uint4* p = reinterpret_cast<uint4*>(sQ + qs * L::TILE + (qc >> 3) * L::CHUNK + qr * 128 + (((qc & 7) ^ (qr & 7)) << 4));
            const uint4 w = *p;
            const uint32_t v[4] = {w.x, w.y, w.z, w.w};
            float x[8], m = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              x[2 * e] = __uint_as_float(v[e] << 16);
              x[2 * e + 1] = __uint_as_float(v[e] & 0xFFFF0000u);
              m = fmax3(m, fabsf(x[2 * e]), fabsf(x[2 * e + 1]));
            }
#pragma unroll
            for (int o = QPR / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
            const int e = static_cast<int>(__float_as_uint(m) >> 23);          // 2^(e - 127) <= m
            const int k = e == 255 ? 0 : min(13 + 127 - e, k_max);
            const float up = __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
            *p = make_uint4(pack_f16x2(x[0] * up, x[1] * up), pack_f16x2(x[2] * up, x[3] * up), pack_f16x2(x[4] * up, x[5] * up),
                            pack_f16x2(x[6] * up, x[7] * up));
            if (qc == 0) sQsc[rs * 128 + qr] = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[B_QREADY + qs]);
        }
        for (int t = t0; ok && t < t1; ++t, ++g) {
          const int valid = min(kBN, max(kend - t * kBN, 0));
          const int r = 2 * g + kv, ss = r % L::RST;
          // the slot written: a K slot is free once the QK that read it has completed, a V slot once its PV has
          const int st = kv ? L::VST : L::KST, sl = g % st, gp = g - st;
          if (gp >= 0 && !(ok = warp_wait(&bars[(kv ? B_PVDONE : B_SFULL) + gp % kSBufs], (gp / kSBufs) & 1))) break;
          // (a stage of 3 or 6 holds a tile of the same kind again six tiles later)
          if (!(ok = warp_wait(&bars[B_RFULL + 6 * kv + ss], (r / 6) & 1))) break;
          // scales of key gt, zero where there is no key or page; asked for before the codes are turned
          const int gt = dt & 127;
          float ks = 0.f, vs = 0.f;
          if (kv == 0) {
            const int base = sBase[ss * 8 + gt / box_rows];
            if (gt < valid && base >= 0) {
              ks = __ldg(a.k_scale + base + gt % box_rows);
              vs = __ldg(a.v_scale + base + gt % box_rows);
            }
          }
          const uint8_t* src = sR + ss * L::RAW;
          uint8_t* dst = (kv ? sV : sK) + sl * L::TILE + (c >> 2) * L::CHUNK + r0 * 128;
          constexpr int NB = 2;   // rows a thread holds at a time (more are no faster, 8 a third slower)
          static_assert(RPP % 8 == 0, "a thread's rows have one place in the swizzle");
#pragma unroll 1
          for (int rr = r0; rr < 128; rr += NB * RPP, dst += NB * RPP * 128) {
            uint4 w[NB];
#pragma unroll
            for (int e = 0; e < NB; ++e) {
              w[e] = *reinterpret_cast<const uint4*>(src + (rr + e * RPP) * D + c * 16);
              if (kv && rr + e * RPP >= valid) w[e] = make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int e = 0; e < NB; ++e) {
              const uint4 lo = make_uint4(decode2<KIND, 0>(w[e].x), decode2<KIND, 1>(w[e].x), decode2<KIND, 0>(w[e].y), decode2<KIND, 1>(w[e].y));
              const uint4 hi = make_uint4(decode2<KIND, 0>(w[e].z), decode2<KIND, 1>(w[e].z), decode2<KIND, 0>(w[e].w), decode2<KIND, 1>(w[e].w));
              *reinterpret_cast<uint4*>(dst + e * RPP * 128 + off0) = first ? hi : lo;
              *reinterpret_cast<uint4*>(dst + e * RPP * 128 + off1) = first ? lo : hi;
            }
          }
          if (kv == 0) {
            // largest value scale of the tile
            float m = vs;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
            // (the buffers' last reader is the softmax of tile g - 3)
            if (g >= kSBufs && !(ok = warp_wait(&bars[B_PVDONE + g % kSBufs], ((g / kSBufs) & 1) ^ 1))) break;
            sSc[(g % kSBufs) * 256 + gt] = ks;
            sSc[(g % kSBufs) * 256 + 128 + gt] = vs;
            if (lane == 0) sVmax[(g % kSBufs) * 4 + (gt >> 5)] = m;
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&bars[B_REMPTY + 6 * kv + ss]);
            mbar_arrive(&bars[(kv ? B_VFULL : B_KFULL) + sl]);
          }
        }
        ++qi;
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    if constexpr (Q8) reg_alloc<152>();
    const int quad = warp & 3, half = (warp - kSoft0) >> 2, sw = warp - kSoft0;
    const int j4 = lane & 3;
    const int wrow = quad * 32 + half * 16;               // the warp's 16 rows
    const int ra = wrow + (lane >> 2);                    // this thread's rows: ra and ra + 8
    const uint32_t lane_addr = static_cast<uint32_t>(wrow) << 16;
    int g = 0, qi = 0;
    bool ok = true;
    while (ok) {
      const int rs = qi % kItemRing;
      if (!(ok = warp_wait(&bars[B_IFULL + rs], (qi / kItemRing) & 1))) break;
      volatile int* f = ring + rs * kRingWords;
      const int more = f[0], h = f[2], t0 = f[3], t1 = f[4], kend = f[5], row0 = f[6], ntok = f[7], vis0 = f[8], mode = f[9];
      const int L_ = f[10];
      __syncwarp();
      if ((!Q8 || !more) && lane == 0) mbar_arrive(&bars[B_IEMPTY + rs]);   // (8-bit: once q's scales are read)
      if (!more) break;
      const int rows = ntok * a.G;
      const int tok_a = ra / a.G, tok_b = (ra + 8) / a.G;
      // visible keys of the two rows (all of them without `causal`: vis0 = L)
      const int vis_a = min(L_, max(0, a.causal ? vis0 + tok_a : vis0));
      const int vis_b = min(L_, max(0, a.causal ? vis0 + tok_b : vis0));
      const int vis_min = min(L_, max(0, a.causal ? vis0 + wrow / a.G : vis0));
      const bool active = wrow < rows;
      float m_a = -INFINITY, m_b = -INFINITY, l_a = 0.f, l_b = 0.f;
      float f_a = a.scale_log2, f_b = a.scale_log2;         // of the rows' scores
      float C = kMinC;                                       // (8-bit)
      for (int t = t0; t < t1; ++t, ++g) {
        const int b = g % kSBufs;
        if (!(ok = warp_wait(&bars[B_SFULL + b], (g / kSBufs) & 1))) break;
        if (Q8 && t == t0) {
          // (finite, so that scores of 0 stay 0 under a scale above 2^13 of queries near the end of fp32)
          f_a = fminf(f_a * sQsc[rs * 128 + ra], 3.40282347e38f);
          f_b = fminf(f_b * sQsc[rs * 128 + ra + 8], 3.40282347e38f);
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[B_IEMPTY + rs]);
        }
        if (active) {
          tc_fence_after();
          float xa[32], xb[32];   // [2 k + e]: column 8 k + 2 j4 + e of rows ra, ra + 8
          {
            uint32_t r0[32], r1[32];
            tmem_ld_16x256b_x8(tm + lane_addr + tm_s(b), r0);
            tmem_ld_16x256b_x8(tm + lane_addr + tm_s(b) + 64, r1);
            tmem_wait_ld();
            reg_fence(r0);
            reg_fence(r1);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              xa[2 * k] = __uint_as_float(r0[4 * k]);
              xa[2 * k + 1] = __uint_as_float(r0[4 * k + 1]);
              xb[2 * k] = __uint_as_float(r0[4 * k + 2]);
              xb[2 * k + 1] = __uint_as_float(r0[4 * k + 3]);
              xa[16 + 2 * k] = __uint_as_float(r1[4 * k]);
              xa[16 + 2 * k + 1] = __uint_as_float(r1[4 * k + 1]);
              xb[16 + 2 * k] = __uint_as_float(r1[4 * k + 2]);
              xb[16 + 2 * k + 1] = __uint_as_float(r1[4 * k + 3]);
            }
          }
          if constexpr (Q8) {
            const uint64_t* ksc = reinterpret_cast<const uint64_t*>(sSc + b * 256) + j4;
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const uint64_t ks = ksc[4 * k];
              f2_split(fmul2(f2_make(xa[2 * k], xa[2 * k + 1]), ks), xa[2 * k], xa[2 * k + 1]);
              f2_split(fmul2(f2_make(xb[2 * k], xb[2 * k + 1]), ks), xb[2 * k], xb[2 * k + 1]);
            }
          }
          if ((t + 1) * kBN > vis_min) {
            const int la = vis_a - t * kBN, lb = vis_b - t * kBN;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const int col = 8 * (i >> 1) + 2 * j4 + (i & 1);
              if (col >= la) xa[i] = -INFINITY;
              if (col >= lb) xb[i] = -INFINITY;
            }
          }
          float mx_a, mx_b;
          {
            float ma4[4], mb4[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              ma4[j] = fmax3_nan(fmax3_nan(xa[j], xa[4 + j], xa[8 + j]), fmax3_nan(xa[12 + j], xa[16 + j], xa[20 + j]), fmax_nan(xa[24 + j], xa[28 + j]));
              mb4[j] = fmax3_nan(fmax3_nan(xb[j], xb[4 + j], xb[8 + j]), fmax3_nan(xb[12 + j], xb[16 + j], xb[20 + j]), fmax_nan(xb[24 + j], xb[28 + j]));
            }
            mx_a = fmax_nan(fmax_nan(ma4[0], ma4[1]), fmax_nan(ma4[2], ma4[3]));
            mx_b = fmax_nan(fmax_nan(mb4[0], mb4[1]), fmax_nan(mb4[2], mb4[3]));
            mx_a = fmax_nan(mx_a, __shfl_xor_sync(0xFFFFFFFFu, mx_a, 1));
            mx_b = fmax_nan(mx_b, __shfl_xor_sync(0xFFFFFFFFu, mx_b, 1));
            mx_a = fmax_nan(mx_a, __shfl_xor_sync(0xFFFFFFFFu, mx_a, 2));
            mx_b = fmax_nan(mx_b, __shfl_xor_sync(0xFFFFFFFFu, mx_b, 2));
          }
          // the running maximum is raised only when a tile's exceeds it by more than 8 (weights stay below 2^8)
          float corr_a = 1.f, corr_b = 1.f;
          {
            const float mt_a = mx_a * f_a, mt_b = mx_b * f_b;
            if (mt_a > m_a + 8.f) {
              corr_a = fast_exp2(m_a - mt_a);
              m_a = mt_a;
              l_a *= corr_a;
            }
            if (mt_b > m_b + 8.f) {
              corr_b = fast_exp2(m_b - mt_b);
              m_b = mt_b;
              l_b *= corr_b;
            }
            // a visible score of NaN or +inf (or beyond fp32) makes the row NaN, as inf - inf does in the formula: the
            // exponentials on the FMA pipe would lose it, and the row would be an average that has nothing to do with it
            if (!(mt_a < INFINITY)) l_a = NAN;
            if (!(mt_b < INFINITY)) l_b = NAN;
          }
          const uint64_t fa2 = f2_make(f_a, f_a), fb2 = f2_make(f_b, f_b);
          float invC = 1.f;
          if constexpr (Q8) {
            const float4 vm = *reinterpret_cast<const float4*>(sVmax + b * 4);
            const float c = pow2_above(fmaxf(fmaxf(vm.x, vm.y), fmaxf(vm.z, vm.w)));
            if (c > C) {
              corr_a *= C / c;
              corr_b *= C / c;
              C = c;
            }
            invC = __uint_as_float((261u << 23) - __float_as_uint(C));   // 2^7 / C
          }
          // a row that has seen no key yet keeps m = -inf, and its weights are 0
          const float na = m_a == -INFINITY ? 0.f : -m_a, nb = m_b == -INFINITY ? 0.f : -m_b;
          const uint64_t negm_a = f2_make(na, na), negm_b = f2_make(nb, nb);
          uint64_t acc_a[2] = {0ull, 0ull}, acc_b[2] = {0ull, 0ull};
          uint32_t p[32];   // bf16 pairs: [2 k] row ra, [2 k + 1] row ra + 8, column 4 k + j4
          const uint64_t* vsc = reinterpret_cast<const uint64_t*>(sSc + b * 256 + 128) + j4;
          const uint64_t invC2 = f2_make(invC, invC);
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            uint64_t vs = 0;
            if constexpr (Q8) vs = fmul2(vsc[4 * k], invC2);
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              const float* xr = w ? xb : xa;
              const uint64_t a2 = ffma2(f2_make(xr[2 * k], xr[2 * k + 1]), w ? fb2 : fa2, w ? negm_b : negm_a);
              float e0, e1;
              if ((kPolyPairs >> (k & 7)) & 1) {
                exp2_poly2(a2, e0, e1);
                // its least value is a subnormal that bf16 would round up to 2^-126: times a value of 2^127 no longer
                // nothing, and masked positions have it too (fp16 rounds it to 0)
                if constexpr (!Q8) f2_split(fmul2_ftz(f2_make(e0, e1), f2_make(1.f, 1.f)), e0, e1);
              } else {
                float a0, a1;
                f2_split(a2, a0, a1);
                e0 = fast_exp2(a0);
                e1 = fast_exp2(a1);
              }
              if (w) acc_b[k & 1] = fadd2(acc_b[k & 1], f2_make(e0, e1));
              else acc_a[k & 1] = fadd2(acc_a[k & 1], f2_make(e0, e1));
              if constexpr (Q8) f2_split(fmul2(f2_make(e0, e1), vs), e0, e1);
              p[2 * k + w] = Q8 ? pack_f16x2(e0, e1) : pack_bf16x2(e0, e1);
            }
          }
          {
            float s0, s1;
            f2_split(fadd2(acc_a[0], acc_a[1]), s0, s1);
            l_a += s0 + s1;
            f2_split(fadd2(acc_b[0], acc_b[1]), s0, s1);
            l_b += s0 + s1;
          }
          tmem_st_16x128b_x16(tm + lane_addr + tm_s(b), p);
          if (t > t0 && __any_sync(0xFFFFFFFFu, corr_a != 1.f || corr_b != 1.f)) {
            const int pb = (g - 1) % kSBufs;
            if (!(ok = warp_wait(&bars[B_PVDONE + pb], ((g - 1) / kSBufs) & 1))) {
              tmem_wait_st();
              break;
            }
            tc_fence_after();
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 64) {
              uint32_t o[32];
              const uint32_t oa = tm + lane_addr + TM_O + c0;
              tmem_ld_16x256b_x8(oa, o);
              tmem_wait_ld();
              reg_fence(o);
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                o[4 * k] = __float_as_uint(__uint_as_float(o[4 * k]) * corr_a);
                o[4 * k + 1] = __float_as_uint(__uint_as_float(o[4 * k + 1]) * corr_a);
                o[4 * k + 2] = __float_as_uint(__uint_as_float(o[4 * k + 2]) * corr_b);
                o[4 * k + 3] = __float_as_uint(__uint_as_float(o[4 * k + 3]) * corr_b);
              }
              tmem_st_16x256b_x8(oa, o);
            }
          }
          tmem_wait_st();
          tc_fence_before();
        }
        if constexpr (!Q8) {
          // value rows between the last key and the end of its group of 16: zero (they may hold anything)
          const int valid = kend - t * kBN;
          if (valid < kBN && (valid & 15) != 0) {
            const int vs = g % L::VST, gp = g - L::VST;
            // (the slot's tile before: a wait for this one's phase may only begin when that one has ended)
            if (gp >= 0 && !(ok = warp_wait(&bars[B_PVDONE + gp % kSBufs], (gp / kSBufs) & 1))) break;
            if (!(ok = warp_wait(&bars[B_VFULL + vs], (g / L::VST) & 1))) break;
            const int end = (valid + 15) & ~15;
            for (int z = valid + sw; z < end; z += kSoftWarps)
              for (int i = lane; i < L::NCH * 8; i += 32)
                *reinterpret_cast<uint4*>(sV + vs * L::TILE + (i >> 3) * L::CHUNK + z * 128 + (i & 7) * 16) = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[B_PFULL + b]);
      }
      if (!ok) break;
      // ---------------------------------------------------------- rows out
      if (!(ok = warp_wait(&bars[B_OFULL], qi & 1))) break;
      if (active) {
        l_a += __shfl_xor_sync(0xFFFFFFFFu, l_a, 1);
        l_b += __shfl_xor_sync(0xFFFFFFFFu, l_b, 1);
        l_a += __shfl_xor_sync(0xFFFFFFFFu, l_a, 2);
        l_b += __shfl_xor_sync(0xFFFFFFFFu, l_b, 2);
        // rows that saw a key here; one whose scores were all NaN or -inf keeps m = -inf and gives NaN, as the
        // formula does (a part of a row that has only -inf scores adds nothing to the others)
        const bool some_a = vis_a > t0 * kBN, some_b = vis_b > t0 * kBN;
        const bool none_a = m_a == -INFINITY && !isnan(l_a), none_b = m_b == -INFINITY && !isnan(l_b);
        tc_fence_after();
        const float oc = Q8 ? C * 0.0078125f : 1.f;
        const float o_a = mode != 0 ? oc : none_a ? NAN : oc / l_a, o_b = mode != 0 ? oc : none_b ? NAN : oc / l_b;
        const int slot = 2 * blockIdx.x + (mode == 2 ? 1 : 0);
        float* po = slot_o<D>(a, slot);
        __nv_bfloat16* oa = static_cast<__nv_bfloat16*>(a.o) + (row0 + tok_a) * a.o_st + (static_cast<long long>(h) * a.G + ra % a.G) * a.o_sh;
        __nv_bfloat16* ob = static_cast<__nv_bfloat16*>(a.o) + (row0 + tok_b) * a.o_st + (static_cast<long long>(h) * a.G + (ra + 8) % a.G) * a.o_sh;
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 64) {
          uint32_t o[32];
          tmem_ld_16x256b_x8(tm + lane_addr + TM_O + c0, o);
          tmem_wait_ld();
          reg_fence(o);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int col = c0 + 8 * k + 2 * j4;
            // (a row without a key: its O was never written, 0 whatever it holds)
            const float va0 = some_a ? __uint_as_float(o[4 * k]) * o_a : 0.f, va1 = some_a ? __uint_as_float(o[4 * k + 1]) * o_a : 0.f;
            const float vb0 = some_b ? __uint_as_float(o[4 * k + 2]) * o_b : 0.f, vb1 = some_b ? __uint_as_float(o[4 * k + 3]) * o_b : 0.f;
            if (mode == 0) {
              if (ra < rows) *reinterpret_cast<uint32_t*>(oa + col) = pack_bf16x2(va0, va1);
              if (ra + 8 < rows) *reinterpret_cast<uint32_t*>(ob + col) = pack_bf16x2(vb0, vb1);
            } else {
              if (ra < rows) *reinterpret_cast<float2*>(po + ra * D + col) = make_float2(va0, va1);
              if (ra + 8 < rows) *reinterpret_cast<float2*>(po + (ra + 8) * D + col) = make_float2(vb0, vb1);
            }
          }
        }
        tc_fence_before();
        if (j4 == 0) {
          if (mode != 0) {
            float2* ml = slot_ml<D>(a, slot);
            if (ra < rows) ml[ra] = make_float2(m_a, some_a && !none_a ? l_a : 0.f);
            if (ra + 8 < rows) ml[ra + 8] = make_float2(m_b, some_b && !none_b ? l_b : 0.f);
          } else if (a.lse) {
            const long long Hq = static_cast<long long>(a.H) * a.G;
            if (ra < rows)
              a.lse[(row0 + tok_a) * Hq + static_cast<long long>(h) * a.G + ra % a.G] =
                  some_a ? (m_a + log2f(l_a)) * 0.69314718055994531f : -INFINITY;
            if (ra + 8 < rows)
              a.lse[(row0 + tok_b) * Hq + static_cast<long long>(h) * a.G + (ra + 8) % a.G] =
                  some_b ? (m_b + log2f(l_b)) * 0.69314718055994531f : -INFINITY;
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[B_OEMPTY]);
      ++qi;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tm, TM_COLS);
  }
}

// Joins the partial results of the item that a CTA of the first kernel began and
// did not finish: slot 1 of that CTA, then slot 0 of the CTAs behind it up to the
// item's last tile, in that order (so results do not depend on timing).
template <int D>
__global__ void __launch_bounds__(256) cache_attn_join_kernel(const __grid_constant__ CacheAttnArgs a) {
  using namespace cattn;
  grid_dep_wait();
  const int c = blockIdx.x;
  const Begun it = *begun<D>(a, c);
  if (it.rows * (D / 4) <= static_cast<int>(blockIdx.y) * 256) return;
  // the parts: this CTA's slot 1, then slot 0 of the CTAs behind it up to the item's last tile (one whose share
  // holds no start of a tile left nothing). A share k0 = W e / ctas begins at or before `last` for e up to this:
  const long long last = it.base + static_cast<long long>(it.tiles - 1) * kBN;   // start of its last tile
  const int c_last = static_cast<int>(((last + 1) * it.ctas - 1) / it.W);
  __shared__ int slots[kMaxCtas];
  __shared__ int n_slots;
  if (threadIdx.x < 32) {
    int n = 0;
#pragma unroll 1
    for (int e0 = c; e0 <= c_last; e0 += 32) {
      const int e = e0 + threadIdx.x;
      const long long k0 = it.W * e / it.ctas, k1 = it.W * (e + 1) / it.ctas;
      const bool has = e == c || (e <= c_last && it.base + static_cast<long long>(first_tile(it.base, k0)) * kBN < k1);
      const unsigned m = __ballot_sync(0xFFFFFFFFu, has);
      if (has) slots[n + __popc(m & ((1u << threadIdx.x) - 1))] = 2 * e + (e == c ? 1 : 0);
      n += __popc(m);
    }
    if (threadIdx.x == 0) n_slots = n;
  }
  __syncthreads();
  const int n = n_slots;
#pragma unroll 1
  for (int i = blockIdx.y * 256 + threadIdx.x; i < it.rows * (D / 4); i += gridDim.y * 256) {
    const int row = i / (D / 4), col = i % (D / 4) * 4;
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int e0 = 0; e0 < n; e0 += 4) {
      float2 ml[4];
      float4 v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (e0 + e < n) {
          ml[e] = slot_ml<D>(a, slots[e0 + e])[row];
          v[e] = *reinterpret_cast<const float4*>(slot_o<D>(a, slots[e0 + e]) + row * D + col);
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (e0 + e >= n || (ml[e].x == -INFINITY && ml[e].y == 0.f)) continue;   // (a sum of NaN stays)
        const float mn = fmaxf(m, ml[e].x);
        const float wo = fast_exp2(m - mn), wn = fast_exp2(ml[e].x - mn);   // (m = -inf gives 0)
        o.x = o.x * wo + v[e].x * wn;
        o.y = o.y * wo + v[e].y * wn;
        o.z = o.z * wo + v[e].z * wn;
        o.w = o.w * wo + v[e].w * wn;
        l = l * wo + ml[e].y * wn;
        m = mn;
      }
    }
    // visible keys of the row: none gives zeros, keys whose scores are all NaN or -inf give NaN
    const int vis = it.vis0 + (a.causal ? row / a.G : 0);
    const float f = vis <= 0 ? 0.f : m != -INFINITY ? 1.f / l : NAN;
    const long long tok = it.row0 + row / a.G, hq = static_cast<long long>(it.h) * a.G + row % a.G;
    __nv_bfloat16* op = static_cast<__nv_bfloat16*>(a.o) + tok * a.o_st + hq * a.o_sh + col;
    *reinterpret_cast<uint2*>(op) = make_uint2(pack_bf16x2(o.x * f, o.y * f), pack_bf16x2(o.z * f, o.w * f));
    if (a.lse && col == 0)
      a.lse[tok * a.H * a.G + hq] = vis > 0 ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
  }
}

size_t cache_attn_ws_bytes(int d) {
  return cattn::kMaxCtas * (2ull * cattn::kBM * (static_cast<size_t>(d) * 4 + 8) + sizeof(cattn::Begun));
}

template <int D, int KIND>
static cudaError_t launch_cache_attn_d(const CacheAttnArgs& a, cudaStream_t st) {
  using namespace cattn;
  using L = Layout<D, KIND>;
  int tpt = kBM / a.G;
  if (a.max_q > 0) tpt = std::min(tpt, a.max_q);
  int box = a.page & -a.page;                              // largest power of two that divides the page
  box = std::min(box, kBN);
  CUtensorMap mq, mk, mv;
  if (encode_tensor_map_q_bf16(&mq, a.q, D, a.G, a.n_rows, a.H, a.q_st, a.q_sh, tpt) != CUDA_SUCCESS) return cudaErrorInvalidValue;
  const uint64_t planes = static_cast<uint64_t>(a.n_pages) * a.H;
  if constexpr (L::Q8) {
    if (encode_tensor_map_3d_u8_plain(&mk, a.k_cache, D, a.page, planes, box) != CUDA_SUCCESS) return cudaErrorInvalidValue;
    if (encode_tensor_map_3d_u8_plain(&mv, a.v_cache, D, a.page, planes, box) != CUDA_SUCCESS) return cudaErrorInvalidValue;
  } else {
    if (encode_tensor_map_3d_bf16(&mk, a.k_cache, D, a.page, planes, 64, box) != CUDA_SUCCESS) return cudaErrorInvalidValue;
    if (encode_tensor_map_3d_bf16(&mv, a.v_cache, D, a.page, planes, 64, box) != CUDA_SUCCESS) return cudaErrorInvalidValue;
  }
  cudaError_t e = allow_smem<cache_attn_kernel<D, KIND>>(L::SMEM);
  if (e != cudaSuccess) return e;
  const int grid = std::min(sm_count_cached(), kMaxCtas);
  e = launch_pdl(cache_attn_kernel<D, KIND>, dim3(grid), dim3(L::THREADS), L::SMEM, st, mq, mk, mv, a, tpt, box);
  if (e != cudaSuccess) return e;
  return launch_pdl(cache_attn_join_kernel<D>, dim3(grid, std::min(kJoinY, ceil_div(tpt * a.G * (D / 4), 512))), dim3(256), 0, st, a);
}

cudaError_t launch_cache_attn(const CacheAttnArgs& a, int d, int kind, cudaStream_t st) {
  if (d == 64) {
    if (kind == kCacheBf16) return launch_cache_attn_d<64, kCacheBf16>(a, st);
    if (kind == kCacheE4m3) return launch_cache_attn_d<64, kCacheE4m3>(a, st);
    return launch_cache_attn_d<64, kCacheInt8>(a, st);
  }
  if (kind == kCacheBf16) return launch_cache_attn_d<128, kCacheBf16>(a, st);
  if (kind == kCacheE4m3) return launch_cache_attn_d<128, kCacheE4m3>(a, st);
  return launch_cache_attn_d<128, kCacheInt8>(a, st);
}

}  // namespace sa
