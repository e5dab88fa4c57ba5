// C-ABI entry points of the paged-cache operators: host-side argument checks,
// then the launchers.
#include <cmath>

#include "paged.cuh"
#include "paged_tc.cuh"

namespace ts {

namespace {

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Checks what every call shares and fills the batch description.
int paged_batch(const char* W, int n, int Hq, int Hkv, int d, const int32_t* cu_q,
                const int32_t* seq_lens, int n_seq, const int32_t* table, int max_pages,
                int page_size, int64_t n_pages, int flags, int known_flags, PagedBatch* b) {
  if (flags & ~known_flags) return fail(TS_ERR_INVALID_ARG, "%s: unknown flags 0x%x", W, flags);
  if (n < 0 || n_seq < 0) return fail(TS_ERR_INVALID_ARG, "%s: n=%d, n_seq=%d", W, n, n_seq);
  if (Hq < 1 || Hkv < 1) return fail(TS_ERR_INVALID_ARG, "%s: Hq=%d, Hkv=%d", W, Hq, Hkv);
  if (Hq % Hkv) return fail(TS_ERR_INVALID_ARG, "%s: Hq=%d not a multiple of Hkv=%d", W, Hq, Hkv);
  if (Hq > 1024) return fail(TS_ERR_UNSUPPORTED, "%s: Hq=%d > 1024", W, Hq);
  if (d != 64 && d != 128) return fail(TS_ERR_UNSUPPORTED, "%s: head dim %d not in {64,128}", W, d);
  if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128)
    return fail(TS_ERR_UNSUPPORTED, "%s: page_size %d not in {16,32,64,128}", W, page_size);
  if (max_pages < 1 || n_pages < 1)
    return fail(TS_ERR_INVALID_ARG, "%s: max_pages=%d, n_pages=%lld", W, max_pages,
                (long long)n_pages);
  // a wait for the work before it must stay well inside the bounded waits' second
  if ((int64_t)max_pages * page_size > (int64_t(1) << 25))
    return fail(TS_ERR_UNSUPPORTED, "%s: max_pages * page_size > 2^25", W);
  if (n_seq > (1 << 20)) return fail(TS_ERR_UNSUPPORTED, "%s: n_seq=%d > 2^20", W, n_seq);
  if (n_pages >= (int64_t(1) << 31) / page_size / Hkv)
    return fail(TS_ERR_UNSUPPORTED, "%s: n_pages * Hkv * page_size >= 2^31", W);
  if ((int64_t)n * Hq >= (int64_t(1) << 31))
    return fail(TS_ERR_UNSUPPORTED, "%s: n * Hq >= 2^31", W);
  if (n > 0 && n_seq > 0 && (!cu_q || !seq_lens || !table))
    return fail(TS_ERR_INVALID_ARG, "%s: NULL cu_q, seq_lens or page_table", W);
  b->cu_q = cu_q;
  b->seq_lens = seq_lens;
  b->table = table;
  b->n = n;
  b->n_seq = n_seq;
  b->max_pages = max_pages;
  b->page_shift = page_size == 16 ? 4 : page_size == 32 ? 5 : page_size == 64 ? 6 : 7;
  b->n_pages = n_pages;
  return TS_OK;
}

int check_paged_ws(const void* ws, size_t have, size_t need, const char* W) {
  if (need == 0) return TS_OK;
  if (!ws) return fail(TS_ERR_WORKSPACE, "%s: workspace is NULL (%zu bytes needed)", W, need);
  if (reinterpret_cast<uintptr_t>(ws) % 256)
    return fail(TS_ERR_WORKSPACE, "%s: workspace must be 256-byte aligned", W);
  if (have < need)
    return fail(TS_ERR_WORKSPACE, "%s: workspace has %zu bytes, %zu needed", W, have, need);
  return TS_OK;
}

int64_t bound_kv(int max_pages, int page_size, int64_t max_kv) {
  const int64_t cap = (int64_t)max_pages * page_size;
  return max_kv > 0 && max_kv < cap ? max_kv : cap;
}

// Which kernel takes a dense call.  The row kernel reads the keys once a block
// of 16 packed rows of a KV head, the tensor-core tiles once for 256 rows but
// after a plan and with a join (~20 us in all).  One block always takes the row
// kernel, up to four where they are at most 13 trips of 128 keys a SM in all, any
// number at 8.  Measured: 24 rows of 2 KV heads over 32K rows (7 a SM) 22.6 us
// against 26.9; 6 streams of 94 tokens and at most 491 rows (24 blocks, 4 a SM)
// 7.6 against 19.1, of 154 tokens and 1000 rows (39 blocks, 12 a SM) 29.1 against
// 27.0; 32 rows of 8 KV heads over 100K rows (84 a SM) 127 against 83.
bool few_rows(int n_seq, int max_q, int Hq, int Hkv, int64_t kv) {
  const int64_t blocks = ((int64_t)max_q * (Hq / Hkv) + 15) / 16;
  const int64_t trips = (int64_t)n_seq * Hkv * blocks * ((kv + 127) / 128);
  return blocks <= 1 || trips <= 8 * kGb300Sms || (blocks <= 4 && trips <= 13 * kGb300Sms);
}

}  // namespace

}  // namespace ts

using namespace ts;

extern "C" {

int ts_rope_frequencies(int rot_dim, double base, int scaling, double factor, double original_len,
                        double low, double high, double* freqs, float* rope_scale) {
  clear_error();
  const char* W = "ts_rope_frequencies";
  if (rot_dim < 2 || rot_dim > 1024 || rot_dim % 2)
    return fail(TS_ERR_INVALID_ARG, "%s: rot_dim %d not even in 2 .. 1024", W, rot_dim);
  if (!freqs) return fail(TS_ERR_INVALID_ARG, "%s: NULL freqs", W);
  if (!(base > 1.0) || !std::isfinite(base))
    return fail(TS_ERR_INVALID_ARG, "%s: base %g must be above 1", W, base);
  if (scaling < TS_ROPE_PLAIN || scaling > TS_ROPE_RAMP)
    return fail(TS_ERR_INVALID_ARG, "%s: unknown scaling %d", W, scaling);
  if (scaling != TS_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor)))
    return fail(TS_ERR_INVALID_ARG, "%s: factor %g must be at least 1", W, factor);
  if (scaling == TS_ROPE_BASE && rot_dim < 4)
    return fail(TS_ERR_INVALID_ARG, "%s: a stretched base needs rot_dim >= 4", W);
  if (scaling >= TS_ROPE_WAVELENGTH &&
      (!(original_len > 0.0) || !(low > 0.0) || !(high > low) || !std::isfinite(original_len) ||
       !std::isfinite(high)))
    return fail(TS_ERR_INVALID_ARG, "%s: need original_len > 0 and 0 < low < high", W);
  const double two_pi = 6.283185307179586476925;
  if (scaling == TS_ROPE_BASE) base *= std::pow(factor, rot_dim / (double)(rot_dim - 2));
  double first = 0.0, last = 0.0;
  if (scaling == TS_ROPE_RAMP) {
    auto index = [&](double turns) {
      return rot_dim * std::log(original_len / (two_pi * turns)) / (2.0 * std::log(base));
    };
    first = std::fmax(std::floor(index(high)), 0.0);
    last = std::fmin(std::ceil(index(low)), rot_dim - 1.0);
  }
  for (int c = 0; c < rot_dim / 2; ++c) {
    double f = std::pow(base, -2.0 * c / rot_dim);
    if (scaling == TS_ROPE_LINEAR) {
      f /= factor;
    } else if (scaling == TS_ROPE_WAVELENGTH) {
      const double turns = original_len * f / two_pi;
      const double w = std::fmin(std::fmax((turns - low) / (high - low), 0.0), 1.0);
      f = (1.0 - w) * (f / factor) + w * f;
    } else if (scaling == TS_ROPE_RAMP) {
      const double w = std::fmin(std::fmax((c - first) / std::fmax(last - first, 0.001), 0.0), 1.0);
      f = (1.0 - w) * f + w * (f / factor);
    }
    freqs[c] = f;
  }
  if (rope_scale)
    *rope_scale = scaling == TS_ROPE_RAMP ? (float)(0.1 * std::log(factor) + 1.0) : 1.0f;
  return TS_OK;
}

int ts_paged_rope_append(const void* q, const void* k, const void* v, int64_t q_stride,
                         int64_t k_stride, int64_t v_stride, int n, int Hq, int Hkv, int d,
                         const int32_t* cu_q, const int32_t* seq_lens, int n_seq,
                         const int32_t* page_table, int max_pages, int page_size, int64_t n_pages,
                         const int32_t* positions, const double* freqs, int rot_dim,
                         float rope_scale, void* q_out, void* k_pages, void* v_pages,
                         void* key_min, void* key_max, int flags, int32_t* status, void* stream) {
  clear_error();
  const char* W = "ts_paged_rope_append";
  PagedBatch b;
  int rc = paged_batch(W, n, Hq, Hkv, d, cu_q, seq_lens, n_seq, page_table, max_pages, page_size,
                       n_pages, flags, TS_PAGED_FP16 | TS_ROPE_INTERLEAVED, &b);
  if (rc) return rc;
  if (rot_dim < 0 || rot_dim > d)
    return fail(TS_ERR_INVALID_ARG, "%s: rot_dim %d not in 0 .. d=%d", W, rot_dim, d);
  if (rot_dim % 16)
    return fail(TS_ERR_UNSUPPORTED, "%s: rot_dim %d not a multiple of 16", W, rot_dim);
  if (!key_min != !key_max)
    return fail(TS_ERR_INVALID_ARG, "%s: key_min and key_max go together", W);
  if (n == 0 || n_seq == 0) return TS_OK;
  if (!q || !k || !v || !q_out || !k_pages || !v_pages || (rot_dim > 0 && !freqs))
    return fail(TS_ERR_INVALID_ARG, "%s: NULL tensor", W);
  if (q_stride < (int64_t)Hq * d || k_stride < (int64_t)Hkv * d || v_stride < (int64_t)Hkv * d)
    return fail(TS_ERR_INVALID_ARG, "%s: a token stride is shorter than its row", W);
  if (q_stride % 8 || k_stride % 8 || v_stride % 8)
    return fail(TS_ERR_INVALID_ARG, "%s: token strides must be multiples of 8 elements", W);
  for (const void* p : {q, k, v, (const void*)q_out, (const void*)k_pages, (const void*)v_pages,
                        (const void*)key_min, (const void*)key_max})
    if (!aligned16(p)) return fail(TS_ERR_INVALID_ARG, "%s: a tensor is not 16-byte aligned", W);
  if (q_out == q && q_stride != (int64_t)Hq * d)
    return fail(TS_ERR_INVALID_ARG, "%s: q_out may be q only where q is dense", W);
  AppendArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_out = q_out;
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.key_min = key_min;
  a.key_max = key_max;
  a.positions = positions;
  a.freqs = freqs;
  a.rope_scale = rope_scale;
  a.rot = rot_dim;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.interleaved = (flags & TS_ROPE_INTERLEAVED) != 0;
  return launch_paged_append(b, a, d, (flags & TS_PAGED_FP16) != 0, status,
                             static_cast<cudaStream_t>(stream));
}

size_t ts_paged_attention_workspace_bytes(int n, int n_seq, int Hq, int Hkv, int d, int max_pages,
                                          int page_size, int max_q, int64_t max_kv) {
  if (n < 1 || n_seq < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv || max_pages < 1 || page_size < 1 ||
      max_q < 1)
    return 0;
  const int64_t kv = bound_kv(max_pages, page_size, max_kv);
  if (few_rows(n_seq, max_q, Hq, Hkv, kv))
    return rows_plan((int64_t)n_seq * Hkv, max_q * (Hq / Hkv), d, kv).ws_bytes;
  return tc_plan(n, n_seq, Hq, Hkv, d, max_q, kv).ws_bytes;
}

int ts_paged_attention(const void* q, const void* k_pages, const void* v_pages, int n, int Hq,
                       int Hkv, int d, const int32_t* cu_q, const int32_t* seq_lens, int n_seq,
                       const int32_t* page_table, int max_pages, int page_size, int64_t n_pages,
                       int max_q, int64_t max_kv, void* o, float* lse, void* workspace,
                       size_t workspace_bytes, int flags, int32_t* status, void* stream) {
  clear_error();
  const char* W = "ts_paged_attention";
  PagedBatch b;
  int rc = paged_batch(W, n, Hq, Hkv, d, cu_q, seq_lens, n_seq, page_table, max_pages, page_size,
                       n_pages, flags, TS_PAGED_FP16, &b);
  if (rc) return rc;
  if (n == 0 || n_seq == 0) return TS_OK;
  if (max_q < 1 || max_q > n)
    return fail(TS_ERR_INVALID_ARG, "%s: max_q=%d not in 1 .. n=%d", W, max_q, n);
  if (!q || !k_pages || !v_pages || !o) return fail(TS_ERR_INVALID_ARG, "%s: NULL tensor", W);
  for (const void* p : {q, k_pages, v_pages, (const void*)o})
    if (!aligned16(p)) return fail(TS_ERR_INVALID_ARG, "%s: a tensor is not 16-byte aligned", W);
  const int64_t kv = bound_kv(max_pages, page_size, max_kv);
  if (!few_rows(n_seq, max_q, Hq, Hkv, kv)) {
    const TcPlan p = tc_plan(n, n_seq, Hq, Hkv, d, max_q, kv);
    rc = check_paged_ws(workspace, workspace_bytes, p.ws_bytes, W);
    if (rc) return rc;
    const TcArgs a{q, k_pages, v_pages, Hq, Hkv, max_q, o, lse};
    return launch_paged_tc(b, a, p, d, (flags & TS_PAGED_FP16) != 0, workspace, status,
                           static_cast<cudaStream_t>(stream));
  }
  const RowsPlan p = rows_plan((int64_t)n_seq * Hkv, max_q * (Hq / Hkv), d, kv);
  rc = check_paged_ws(workspace, workspace_bytes, p.ws_bytes, W);
  if (rc) return rc;
  RowsArgs a{};
  a.q = q;
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.max_q = max_q;
  a.o = o;
  a.lse = lse;
  return launch_paged_rows(b, a, p, d, (flags & TS_PAGED_FP16) != 0, workspace, status,
                           static_cast<cudaStream_t>(stream));
}

size_t ts_paged_select_workspace_bytes(int n, int Hkv, int max_pages) {
  if (n < 1 || Hkv < 1 || max_pages < 1) return 0;
  return paged_select_ws_bytes(n, Hkv, max_pages);
}

int ts_paged_select_pages(const void* q, const void* key_min, const void* key_max, int n, int Hq,
                          int Hkv, int d, const int32_t* cu_q, const int32_t* seq_lens, int n_seq,
                          const int32_t* page_table, int max_pages, int page_size,
                          int64_t n_pages, int n_top, int n_sink, int n_recent, int32_t* pages,
                          int32_t* counts, void* workspace, size_t workspace_bytes, int flags,
                          int32_t* status, void* stream) {
  clear_error();
  const char* W = "ts_paged_select_pages";
  PagedBatch b;
  int rc = paged_batch(W, n, Hq, Hkv, d, cu_q, seq_lens, n_seq, page_table, max_pages, page_size,
                       n_pages, flags, TS_PAGED_FP16, &b);
  if (rc) return rc;
  if (n_top < 0 || n_sink < 0 || n_recent < 1)
    return fail(TS_ERR_INVALID_ARG, "%s: need n_top, n_sink >= 0 and n_recent >= 1", W);
  if ((int64_t)n_top + n_sink + n_recent > (1 << 24))
    return fail(TS_ERR_UNSUPPORTED, "%s: more than 2^24 pages a token", W);
  if (n > 65535) return fail(TS_ERR_UNSUPPORTED, "%s: n=%d > 65535 tokens", W, n);
  if (n == 0 || n_seq == 0) return TS_OK;
  if (!q || !key_min || !key_max || !pages || !counts)
    return fail(TS_ERR_INVALID_ARG, "%s: NULL tensor", W);
  for (const void* p : {q, key_min, key_max})
    if (!aligned16(p)) return fail(TS_ERR_INVALID_ARG, "%s: a tensor is not 16-byte aligned", W);
  rc = check_paged_ws(workspace, workspace_bytes, paged_select_ws_bytes(n, Hkv, max_pages), W);
  if (rc) return rc;
  return launch_paged_select(b, q, key_min, key_max, Hq, Hkv, d, (flags & TS_PAGED_FP16) != 0,
                             n_top, n_sink, n_recent, pages, counts, workspace, status,
                             static_cast<cudaStream_t>(stream));
}

size_t ts_paged_selected_workspace_bytes(int n, int Hq, int Hkv, int d, int page_size, int n_sel) {
  if (n < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv || page_size < 1 || n_sel < 1) return 0;
  return rows_plan((int64_t)n * Hkv, Hq / Hkv, d, (int64_t)n_sel * page_size).ws_bytes;
}

int ts_paged_attention_selected(const void* q, const void* k_pages, const void* v_pages, int n,
                                int Hq, int Hkv, int d, const int32_t* cu_q,
                                const int32_t* seq_lens, int n_seq, const int32_t* page_table,
                                int max_pages, int page_size, int64_t n_pages,
                                const int32_t* pages, const int32_t* counts, int n_sel, void* o,
                                float* lse, void* workspace, size_t workspace_bytes, int flags,
                                int32_t* status, void* stream) {
  clear_error();
  const char* W = "ts_paged_attention_selected";
  PagedBatch b;
  int rc = paged_batch(W, n, Hq, Hkv, d, cu_q, seq_lens, n_seq, page_table, max_pages, page_size,
                       n_pages, flags, TS_PAGED_FP16, &b);
  if (rc) return rc;
  if (n_sel < 1) return fail(TS_ERR_INVALID_ARG, "%s: n_sel=%d", W, n_sel);
  if ((int64_t)n_sel * page_size > (int64_t(1) << 25))
    return fail(TS_ERR_UNSUPPORTED, "%s: n_sel * page_size > 2^25", W);
  if (n == 0 || n_seq == 0) return TS_OK;
  if (!q || !k_pages || !v_pages || !pages || !counts || !o)
    return fail(TS_ERR_INVALID_ARG, "%s: NULL tensor", W);
  for (const void* p : {q, k_pages, v_pages, (const void*)o})
    if (!aligned16(p)) return fail(TS_ERR_INVALID_ARG, "%s: a tensor is not 16-byte aligned", W);
  const RowsPlan p =
      rows_plan((int64_t)n * Hkv, Hq / Hkv, d, (int64_t)n_sel * page_size);
  rc = check_paged_ws(workspace, workspace_bytes, p.ws_bytes, W);
  if (rc) return rc;
  RowsArgs a{};
  a.q = q;
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.pages = pages;
  a.counts = counts;
  a.n_sel = n_sel;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.max_q = 1;
  a.o = o;
  a.lse = lse;
  return launch_paged_rows(b, a, p, d, (flags & TS_PAGED_FP16) != 0, workspace, status,
                           static_cast<cudaStream_t>(stream));
}

}  // extern "C"
