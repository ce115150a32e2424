// cache_api.cu — the extern "C" boundary of the calls that keep state: the
// paged key/value cache, attention over it and linear attention with decay.
// Included from libsa.cu after sa_api.cu, whose argument checks and error
// reporting it uses.

#include <algorithm>
#include <initializer_list>

namespace sa {

namespace {

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// The cache's own facts: sizes, kind and buffers.
int check_cache(const char* fn, int n_rows, int n_seqs, int H, int d, int kind, int n_pages, int page, int width,
                const void* k_cache, const void* v_cache, const void* k_scale, const void* v_scale) {
  if (n_rows < 0 || n_seqs <= 0 || H <= 0 || n_pages <= 0 || page <= 0 || width <= 0)
    return fail(SA_ERR_INVALID_ARG, "%s: sizes must be positive (n_rows at least 0)", fn);
  if (kind != SA_CACHE_BF16 && kind != SA_CACHE_E4M3 && kind != SA_CACHE_INT8)
    return fail(SA_ERR_INVALID_ARG, "%s: unknown cache kind %d", fn, kind);
  if (d != 64 && d != 128) return fail(SA_ERR_UNSUPPORTED, "head dim %d unsupported (64 or 128)", d);
  if (page % 16 != 0) return fail(SA_ERR_UNSUPPORTED, "%s: page of %d tokens unsupported (a multiple of 16)", fn, page);
  if (H > 65535) return fail(SA_ERR_UNSUPPORTED, "%s: %d heads exceed 65535", fn, H);
  // (the loader of the attention works out up to 32 boxes of 128 positions behind the last one)
  if (static_cast<long long>(width) * page > 0x7FFFE000LL)
    return fail(SA_ERR_UNSUPPORTED, "%s: a table of %d pages of %d tokens exceeds 2^31 - 8192 positions", fn, width, page);
  if (static_cast<double>(n_pages) * H * page * d >= 1099511627776.0)
    return fail(SA_ERR_UNSUPPORTED, "%s: cache too large", fn);
  if (static_cast<double>(n_pages) * H * page > 2147483392.0)
    return fail(SA_ERR_UNSUPPORTED, "%s: cache of more than 2^31 - 256 rows", fn);
  if (!k_cache || !v_cache) return fail(SA_ERR_INVALID_ARG, "%s: null pointer", fn);
  const bool scaled = kind != SA_CACHE_BF16;
  if (scaled && (!k_scale || !v_scale)) return fail(SA_ERR_INVALID_ARG, "%s: an 8-bit cache needs k_scale and v_scale", fn);
  if (!scaled && (k_scale || v_scale)) return fail(SA_ERR_INVALID_ARG, "%s: a bf16 cache has no scales", fn);
  const void* ptrs[] = {k_cache, v_cache, k_scale, v_scale};
  for (const void* p : ptrs)
    if (p && !aligned16(p)) return fail(SA_ERR_ALIGN, "%s: pointers must be 16-byte aligned", fn);
  return SA_OK;
}

// Token and head strides of a [rows, heads, d] operand, in elements.
int check_strides(const char* fn, const char* name, long long st, long long sh, int d) {
  if (st < d || sh < d || st % 8 != 0 || sh % 8 != 0 || st >= (1LL << 38) || sh >= (1LL << 38))
    return fail(SA_ERR_INVALID_ARG, "%s: strides of %s must be multiples of 8 elements, at least d (got %lld, %lld)", fn, name, st, sh);
  return SA_OK;
}

// The score scale in base 2: `scale`, or 1/sqrt(d) where it is not positive. It
// has to be a normal fp32 number: a product of 0 or infinity with a score would
// not be the softmax asked for.
int check_scale(const char* fn, double scale, int d, double factor, float* out) {
  if (isnan(scale)) return fail(SA_ERR_INVALID_ARG, "%s: scale is NaN", fn);
  const double x = (scale > 0 ? scale : 1.0 / sqrt(static_cast<double>(d))) * factor;
  if (!(x >= 1.2e-38 && x <= 3.4e38)) return fail(SA_ERR_INVALID_ARG, "%s: scale %g is outside fp32", fn, scale);
  *out = static_cast<float>(x);
  return SA_OK;
}

// Whether `bytes` at p and at q have one in common (a null pointer has none).
bool overlap(const void* p, size_t np, const void* q, size_t nq) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return p && q && a < b + nq && b < a + np;
}

struct Range {
  const void* p;
  size_t bytes;
};

// Refuses outputs that overlap an input or another output.
int check_apart(const char* fn, std::initializer_list<Range> outs, std::initializer_list<Range> ins) {
  for (const Range* o = outs.begin(); o != outs.end(); ++o) {
    for (const Range& i : ins)
      if (overlap(o->p, o->bytes, i.p, i.bytes)) return fail(SA_ERR_INVALID_ARG, "%s: outputs must not overlap inputs", fn);
    for (const Range* x = outs.begin(); x != o; ++x)
      if (overlap(o->p, o->bytes, x->p, x->bytes)) return fail(SA_ERR_INVALID_ARG, "%s: outputs must not overlap each other", fn);
  }
  return SA_OK;
}

// A [rows, heads, d] bf16 operand.
struct Rows {
  const void* p;
  long long st, sh;
};

// Whether two of them have an element in common. Views of one buffer may interleave: with equal strides, or if one of
// the two has no gaps, that is found exactly; others count as apart.
bool rows_overlap(const Rows& x, const Rows& y, long long rows, long long heads, int d) {
  if (rows == 0) return false;
  const auto span = [&](const Rows& r) { return (rows - 1) * r.st + (heads - 1) * r.sh + d; };
  if (!overlap(x.p, 2 * span(x), y.p, 2 * span(y))) return false;
  const long long delta = (reinterpret_cast<intptr_t>(y.p) - reinterpret_cast<intptr_t>(x.p)) / 2;   // (both 16-byte aligned)
  if (x.st == y.st && x.sh == y.sh) {
    // rows that lie t tokens and h heads apart begin delta + h sh + t st elements apart: fewer than d for some t and h?
    for (long long h = -(heads - 1); h < heads; ++h) {
      const long long at = delta + h * x.sh, t0 = -at / x.st;
      for (long long t = std::max(t0 - 1, 1 - rows); t <= std::min(t0 + 1, rows - 1); ++t)
        if (at + t * x.st < d && at + t * x.st > -d) return true;
    }
    return false;
  }
  // does a row of the one begin in the other's [-d + 1, its end)?
  const auto meets = [&](long long end, const Rows& r, long long off) {
    for (long long h = 0; h < heads; ++h) {
      const long long at = off + h * r.sh, t = at > -d ? 0 : (-d - at) / r.st + 1;
      if (t < rows && at + t * r.st < end) return true;
    }
    return false;
  };
  if (span(x) == rows * heads * d) return meets(span(x), y, delta);
  if (span(y) == rows * heads * d) return meets(span(y), x, -delta);
  return false;
}

int check_decay(int B, int H, int N, int d) {
  if (B <= 0 || H <= 0 || N <= 0) return fail(SA_ERR_INVALID_ARG, "B, H and N must be positive (got %d, %d, %d)", B, H, N);
  if (d != 64 && d != 128) return fail(SA_ERR_UNSUPPORTED, "head dim %d unsupported (64 or 128)", d);
  const long long BH = static_cast<long long>(B) * H;
  if (BH > 65535) return fail(SA_ERR_UNSUPPORTED, "B*H = %lld exceeds 65535", BH);
  if (N > 0x7FFFFF00 || BH * N * d >= (1LL << 40)) return fail(SA_ERR_UNSUPPORTED, "tensor too large");
  return SA_OK;
}

size_t decay_tensor_bytes(int B, int H, int N, int d) { return static_cast<size_t>(B) * H * N * d * 2; }
size_t decay_state_bytes(int B, int H, int d) { return static_cast<size_t>(B) * H * d * d * 4; }

int check_rows(const char* fn, int n_rows, long long heads, int d) {
  if (static_cast<double>(n_rows) * heads * d >= 1099511627776.0) return fail(SA_ERR_UNSUPPORTED, "%s: tensor too large", fn);
  return SA_OK;
}

}  // namespace

}  // namespace sa

extern "C" {

int sa_cache_write(const uint16_t* k, const uint16_t* v, long long k_stride_t, long long k_stride_h,
                   long long v_stride_t, long long v_stride_h, int n_rows, int n_seqs, int H_kv, int d, int kind,
                   int n_pages, int page, int table_width, const int32_t* table, const int32_t* cu_q,
                   const int32_t* kv_len, void* k_cache, void* v_cache, float* k_scale, float* v_scale, void* stream) {
  const char* fn = "sa_cache_write";
  int rc = check_cache(fn, n_rows, n_seqs, H_kv, d, kind, n_pages, page, table_width, k_cache, v_cache, k_scale, v_scale);
  if (!rc) rc = check_strides(fn, "k", k_stride_t, k_stride_h, d);
  if (!rc) rc = check_strides(fn, "v", v_stride_t, v_stride_h, d);
  if (!rc) rc = check_rows(fn, n_rows, H_kv, d);
  if (rc) return rc;
  if (!k || !v || !table || !cu_q || !kv_len) return fail(SA_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (!aligned16(k) || !aligned16(v) || !aligned4(table) || !aligned4(cu_q) || !aligned4(kv_len))
    return fail(SA_ERR_ALIGN, "%s: tensors must be 16-byte aligned, index arrays 4-byte", fn);
  CacheArgs a{k, v, nullptr, nullptr, k_stride_t, k_stride_h, v_stride_t, v_stride_h, k_cache, v_cache, k_scale, v_scale,
              table, cu_q, kv_len, n_rows, n_seqs, H_kv, n_pages, page, table_width};
  cudaError_t e = launch_cache(a, d, kind, true, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SA_OK : cuda_fail(e, fn);
}

int sa_cache_read(const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale, int n_rows,
                  int n_seqs, int H_kv, int d, int kind, int n_pages, int page, int table_width, const int32_t* table,
                  const int32_t* cu_r, long long k_stride_t, long long k_stride_h, long long v_stride_t,
                  long long v_stride_h, uint16_t* k, uint16_t* v, void* stream) {
  const char* fn = "sa_cache_read";
  int rc = check_cache(fn, n_rows, n_seqs, H_kv, d, kind, n_pages, page, table_width, k_cache, v_cache, k_scale, v_scale);
  if (!rc) rc = check_strides(fn, "k", k_stride_t, k_stride_h, d);
  if (!rc) rc = check_strides(fn, "v", v_stride_t, v_stride_h, d);
  if (!rc) rc = check_rows(fn, n_rows, H_kv, d);
  if (rc) return rc;
  if (!k || !v || !table || !cu_r) return fail(SA_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (!aligned16(k) || !aligned16(v) || !aligned4(table) || !aligned4(cu_r))
    return fail(SA_ERR_ALIGN, "%s: tensors must be 16-byte aligned, index arrays 4-byte", fn);
  CacheArgs a{nullptr, nullptr, k, v, k_stride_t, k_stride_h, v_stride_t, v_stride_h, const_cast<void*>(k_cache),
              const_cast<void*>(v_cache), const_cast<float*>(k_scale), const_cast<float*>(v_scale), table, cu_r, nullptr,
              n_rows, n_seqs, H_kv, n_pages, page, table_width};
  cudaError_t e = launch_cache(a, d, kind, false, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SA_OK : cuda_fail(e, fn);
}

size_t sa_cache_attn_workspace_size(int d) { return d == 64 || d == 128 ? cache_attn_ws_bytes(d) : 0; }

int sa_cache_attn(const uint16_t* q, long long q_stride_t, long long q_stride_h, int n_rows, int n_seqs, int H_q, int H_kv,
                  int d, int kind, int n_pages, int page, int table_width, const int32_t* table, const int32_t* cu_q,
                  const int32_t* kv_len, int max_q, const void* k_cache, const void* v_cache, const float* k_scale,
                  const float* v_scale, int causal, double scale, uint16_t* o, long long o_stride_t,
                  long long o_stride_h, float* lse_opt, void* workspace, size_t ws_bytes, void* stream) {
  const char* fn = "sa_cache_attn";
  int rc = check_cache(fn, n_rows, n_seqs, H_kv, d, kind, n_pages, page, table_width, k_cache, v_cache, k_scale, v_scale);
  if (!rc) rc = check_strides(fn, "q", q_stride_t, q_stride_h, d);
  if (!rc) rc = check_strides(fn, "o", o_stride_t, o_stride_h, d);
  if (!rc) rc = check_rows(fn, n_rows, H_q, d);
  if (rc) return rc;
  if (H_q <= 0 || H_q % H_kv != 0)
    return fail(SA_ERR_INVALID_ARG, "%s: %d query heads are no multiple of %d key heads", fn, H_q, H_kv);
  if (H_q / H_kv > 128) return fail(SA_ERR_UNSUPPORTED, "%s: more than 128 query heads to a key head", fn);
  if (max_q < 0) return fail(SA_ERR_INVALID_ARG, "%s: max_q must not be negative", fn);
  float scale_log2 = 0.f;
  rc = check_scale(fn, scale, d, 1.4426950408889634, &scale_log2);
  if (rc) return rc;
  if (!q || !o || !table || !cu_q || !kv_len) return fail(SA_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (!aligned16(q) || !aligned16(o) || !aligned4(table) || !aligned4(cu_q) || !aligned4(kv_len) || !aligned4(lse_opt) ||
      !aligned16(workspace))
    return fail(SA_ERR_ALIGN, "%s: tensors must be 16-byte aligned, index arrays and lse 4-byte", fn);
  if (rows_overlap({q, q_stride_t, q_stride_h}, {o, o_stride_t, o_stride_h}, n_rows, H_q, d))
    return fail(SA_ERR_INVALID_ARG, "%s: o must not overlap q", fn);
  const size_t need = cache_attn_ws_bytes(d);
  if (need && (!workspace || ws_bytes < need)) return fail(SA_ERR_WORKSPACE, "%s: workspace of %zu bytes needed", fn, need);
  if (n_rows == 0) return SA_OK;
  CacheAttnArgs a{};
  a.q = q; a.q_st = q_stride_t; a.q_sh = q_stride_h;
  a.o = o; a.o_st = o_stride_t; a.o_sh = o_stride_h;
  a.lse = lse_opt;
  a.k_cache = k_cache; a.v_cache = v_cache; a.k_scale = k_scale; a.v_scale = v_scale;
  a.table = table; a.cu_q = cu_q; a.kv_len = kv_len;
  a.n_rows = n_rows; a.n_seqs = n_seqs; a.H = H_kv; a.G = H_q / H_kv;
  a.n_pages = n_pages; a.page = page; a.width = table_width; a.causal = causal != 0;
  a.max_q = max_q;
  a.scale_log2 = scale_log2;
  a.ws = workspace;
  cudaError_t e = launch_cache_attn(a, d, kind, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SA_OK : cuda_fail(e, fn);
}

size_t sa_decay_attn_workspace_size(int B, int H, int N, int d) {
  if (check_decay(B, H, N, d)) return 0;
  return decay_ws_bytes(B * H, N, d);
}

int sa_decay_attn_fwd(const uint16_t* q, const uint16_t* k, const uint16_t* v, const float* log_decay, int B, int H,
                      int N, int d, double scale, const float* state_opt, uint16_t* o, float* state_out_opt,
                      void* workspace, size_t ws_bytes, void* stream) {
  const char* fn = "sa_decay_attn_fwd";
  int rc = check_decay(B, H, N, d);
  if (rc) return rc;
  if (!q || !k || !v || !log_decay || !o) return fail(SA_ERR_INVALID_ARG, "%s: null pointer", fn);
  float sc = 0.f;
  rc = check_scale(fn, scale, d, 1.0, &sc);
  if (rc) return rc;
  const size_t nx = decay_tensor_bytes(B, H, N, d), ns = decay_state_bytes(B, H, d), nl = static_cast<size_t>(H) * 4;
  rc = check_apart(fn, {{o, nx}, {state_out_opt, ns}}, {{q, nx}, {k, nx}, {v, nx}, {log_decay, nl}, {state_opt, ns}});
  if (rc) return rc;
  const void* ptrs[] = {q, k, v, state_opt, o, state_out_opt, workspace};
  for (const void* p : ptrs)
    if (p && !aligned16(p)) return fail(SA_ERR_ALIGN, "%s: pointers must be 16-byte aligned", fn);
  if (!aligned4(log_decay)) return fail(SA_ERR_ALIGN, "%s: log_decay must be 4-byte aligned", fn);
  const size_t need = decay_ws_bytes(B * H, N, d);
  if (need && (!workspace || ws_bytes < need)) return fail(SA_ERR_WORKSPACE, "%s: workspace of %zu bytes needed", fn, need);
  DecayArgs a{q, k, v, o, log_decay, state_opt, state_out_opt, 0, 0, B * H, H, N, sc, sc, 1.f, workspace};
  cudaError_t e = launch_decay(a, nullptr, d, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SA_OK : cuda_fail(e, fn);
}

int sa_decay_attn_bwd(const uint16_t* q, const uint16_t* k, const uint16_t* v, const float* log_decay,
                      const uint16_t* dout, int B, int H, int N, int d, double scale, const float* state_opt,
                      const float* dstate_out_opt, uint16_t* dq, uint16_t* dk, uint16_t* dv, float* dstate_opt,
                      void* workspace, size_t ws_bytes, void* stream) {
  const char* fn = "sa_decay_attn_bwd";
  int rc = check_decay(B, H, N, d);
  if (rc) return rc;
  if (!q || !k || !v || !log_decay || !dout || !dq || !dk || !dv) return fail(SA_ERR_INVALID_ARG, "%s: null pointer", fn);
  float sc = 0.f;
  rc = check_scale(fn, scale, d, 1.0, &sc);
  if (rc) return rc;
  const size_t nx = decay_tensor_bytes(B, H, N, d), ns = decay_state_bytes(B, H, d), nl = static_cast<size_t>(H) * 4;
  rc = check_apart(fn, {{dq, nx}, {dk, nx}, {dv, nx}, {dstate_opt, ns}},
                   {{q, nx}, {k, nx}, {v, nx}, {dout, nx}, {log_decay, nl}, {state_opt, ns}, {dstate_out_opt, ns}});
  if (rc) return rc;
  const void* ptrs[] = {q, k, v, dout, state_opt, dstate_out_opt, dq, dk, dv, dstate_opt, workspace};
  for (const void* p : ptrs)
    if (p && !aligned16(p)) return fail(SA_ERR_ALIGN, "%s: pointers must be 16-byte aligned", fn);
  if (!aligned4(log_decay)) return fail(SA_ERR_ALIGN, "%s: log_decay must be 4-byte aligned", fn);
  const size_t need = decay_ws_bytes(B * H, N, d);
  if (need && (!workspace || ws_bytes < need)) return fail(SA_ERR_WORKSPACE, "%s: workspace of %zu bytes needed", fn, need);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  DecayArgs aq{dout, v, k, dq, log_decay, state_opt, nullptr, 1, 0, B * H, H, N, sc, sc, 1.f, workspace};
  DecayArgs ak{v, dout, q, dk, log_decay, dstate_out_opt, nullptr, 1, 1, B * H, H, N, sc, 1.f, sc, workspace};
  DecayArgs av{k, q, dout, dv, log_decay, dstate_out_opt, dstate_opt, 0, 1, B * H, H, N, sc, 1.f, sc, workspace};
  av.early = 1;
  aq.exact = 0;
  cudaError_t e = launch_decay(aq, nullptr, d, st);
  if (e == cudaSuccess) e = launch_decay(av, &ak, d, st);   // both gradients step the same E_t
  return e == cudaSuccess ? SA_OK : cuda_fail(e, fn);
}

int sa_decay_attn_step(const uint16_t* q, const uint16_t* k, const uint16_t* v, const float* log_decay,
                       const float* state, int B, int H, int d, double scale, uint16_t* o, float* state_out,
                       void* stream) {
  const char* fn = "sa_decay_attn_step";
  int rc = check_decay(B, H, 1, d);
  if (rc) return rc;
  if (!q || !k || !v || !log_decay || !state || !o || !state_out) return fail(SA_ERR_INVALID_ARG, "%s: null pointer", fn);
  float sc = 0.f;
  rc = check_scale(fn, scale, d, 1.0, &sc);
  if (rc) return rc;
  const size_t nx = decay_tensor_bytes(B, H, 1, d), ns = decay_state_bytes(B, H, d), nl = static_cast<size_t>(H) * 4;
  rc = check_apart(fn, {{o, nx}, {state_out, ns}}, {{q, nx}, {k, nx}, {v, nx}, {log_decay, nl}});
  if (!rc) rc = check_apart(fn, {{o, nx}}, {{state, ns}});
  if (rc) return rc;
  if (state != state_out && overlap(state, ns, state_out, ns))
    return fail(SA_ERR_INVALID_ARG, "%s: state_out is state itself or does not overlap it", fn);
  const void* ptrs[] = {q, k, v, state, o, state_out};
  for (const void* p : ptrs)
    if (!aligned16(p)) return fail(SA_ERR_ALIGN, "%s: pointers must be 16-byte aligned", fn);
  if (!aligned4(log_decay)) return fail(SA_ERR_ALIGN, "%s: log_decay must be 4-byte aligned", fn);
  cudaError_t e = launch_decay_step(q, k, v, log_decay, state, state_out, o, B * H, H, d, sc,
                                    static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SA_OK : cuda_fail(e, fn);
}

}  // extern "C"
