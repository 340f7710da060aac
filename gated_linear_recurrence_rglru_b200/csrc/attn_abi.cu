// The extern "C" boundary of the local attention operators: argument checks,
// kernel choice and launches on the caller's stream. See include/rglru_attn.h.
#include <math.h>

#include "attn_kernels.h"
#include "common.cuh"

using namespace rglru;

namespace {

constexpr long long kMaxInt = (1ll << 31) - 1;

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool given(const void *p) { return p != nullptr && aligned16(p); }
bool optional_ok(const void *p) { return p == nullptr || aligned16(p); }
size_t io_bytes(int io) { return io == RGLRU_IO_F32 ? 4 : 2; }

// A span of device memory that a call reads or writes.
struct Span {
  const void *p;
  size_t n;
};

bool meets(const Span &a, const Span &b) {
  if (a.p == nullptr || b.p == nullptr || a.n == 0 || b.n == 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  return a0 < b0 + b.n && b0 < a0 + a.n;
}

// Whether an output span meets an input span or another output span.
template <int NI, int NO> bool overlapping(const Span (&ins)[NI], const Span (&outs)[NO]) {
  for (int o = 0; o < NO; ++o) {
    for (int i = 0; i < NI; ++i)
      if (meets(ins[i], outs[o])) return true;
    for (int x = 0; x < o; ++x)
      if (meets(outs[x], outs[o])) return true;
  }
  return false;
}

// The strided view of a (B, T, H, dh) tensor and the span it covers (a slice's
// span covers what lies between its rows too: an output there is refused). A
// stride of a dimension of one is not looked at.
bool view(const void *p, const rglru_strides *s, int B, int T, int H, int dh, int io, Strided *v,
          Span *span) {
  const long long per16 = 16 / static_cast<long long>(io_bytes(io));
  rglru_strides d = {static_cast<long long>(T) * H * dh, static_cast<long long>(H) * dh, dh};
  if (s != nullptr) {
    if (B > 1) d.batch = s->batch;
    if (T > 1) d.token = s->token;
    if (H > 1) d.head = s->head;
    if (B > 1 && (d.batch < dh || d.batch % per16 != 0)) return false;
    if (T > 1 && (d.token < dh || d.token % per16 != 0)) return false;
    if (H > 1 && (d.head < dh || d.head % per16 != 0)) return false;
    // 2^38 elements are past any device's memory: no stride and no dimension's whole
    // reach is longer, so that the sums below and the copies' 40-bit byte strides stay
    // in range
    constexpr long long kMost = 1ll << 38;
    const auto far = [](long long stride, int n) { return stride > kMost / (n > 2 ? n - 1 : 1); };
    if (far(d.batch, B) || far(d.token, T) || far(d.head, H)) return false;
  }
  *v = {p, d.batch, d.token, d.head};
  const long long last = (B - 1ll) * d.batch + (T - 1ll) * d.token + (H - 1ll) * d.head + dh;
  *span = {p, static_cast<size_t>(last) * io_bytes(io)};
  return true;
}

Span dense(const void *p, long long n, int io) { return {p, static_cast<size_t>(n) * io_bytes(io)}; }
Span bytes_of(const void *p, long long n) { return {p, static_cast<size_t>(n)}; }

int check_heads(int B, int T, int Hq, int Hkv, int dh, int io) {
  if (B < 1 || T < 1 || Hq < 1 || Hkv < 1 || dh < 1) return RGLRU_ERR_INVALID_ARG;
  if (io != RGLRU_IO_F32 && io != RGLRU_IO_BF16) return RGLRU_ERR_INVALID_ARG;
  if (dh % 8 != 0) return RGLRU_ERR_INVALID_ARG;
  if (dh > 256) return RGLRU_ERR_UNSUPPORTED;
  if (static_cast<long long>(B) * T > kMaxInt || static_cast<long long>(B) * Hq > kMaxInt ||
      static_cast<long long>(B) * Hkv > 65535 || static_cast<long long>(Hq) + Hkv > kMaxInt)
    return RGLRU_ERR_UNSUPPORTED;
  if (static_cast<long long>(B) * T > (1ll << 40) / Hq) return RGLRU_ERR_UNSUPPORTED;
  return RGLRU_OK;
}

// The rotation's turn per position of each pair, as a fraction of one turn
// times 2^64: base^(-2i/rot) / (2 pi), by repeated products in long double (64
// bits of fraction on the host).
int set_rotation(QkArgs *a, int rot, double base, float eps) {
  if (rot < 0 || rot > a->dh || rot % 16 != 0) return RGLRU_ERR_INVALID_ARG;
  if (!(eps >= 0.0f) || !isfinite(eps)) return RGLRU_ERR_INVALID_ARG;
  if (!(base >= 1.0) || !isfinite(base)) return RGLRU_ERR_INVALID_ARG;
  a->rot = rot;
  a->eps = eps;
  if (rot > 0) {
    const long double ratio = expl(-2.0L * logl(static_cast<long double>(base)) / rot);
    long double f = 0.159154943091895335768883763372514362L;  // 1 / (2 pi)
    for (int i = 0; i < rot / 2; ++i, f *= ratio)
      a->phase[i] = static_cast<unsigned long long>(f * 18446744073709551616.0L);
  }
  return RGLRU_OK;
}

int check_attn(AttnArgs *a, int io) {
  int st = check_heads(a->B, a->T, a->Hq, a->Hkv, a->dh, io);
  if (st != RGLRU_OK) return st;
  if (a->S < 1 || a->Hq % a->Hkv != 0) return RGLRU_ERR_INVALID_ARG;
  if (a->window < 0 || a->sinks < 0) return RGLRU_ERR_INVALID_ARG;
  if (static_cast<long long>(a->B) * a->S > kMaxInt) return RGLRU_ERR_UNSUPPORTED;
  // tiles of at least 32 rows along a grid dimension; B * Hq heads along another
  if (a->T > 32ll * 65535 || a->S > 32ll * 65535) return RGLRU_ERR_UNSUPPORTED;
  if (static_cast<long long>(a->T) * a->Hq > kMaxInt) return RGLRU_ERR_UNSUPPORTED;
  // a window that reaches the first key hides nothing, and sinks past the last
  // key are no keys
  if (a->window >= a->S) a->window = 0;
  if (a->sinks > a->S) a->sinks = a->S;
  return RGLRU_OK;
}

bool scale_ok(float s) { return isfinite(s) && s > 0.0f; }

}  // namespace

extern "C" {

int rglru_qk_norm_rope_fwd(const void *q, const rglru_strides *q_strides, const void *k,
                           const rglru_strides *k_strides, const void *w_q, const void *w_k,
                           const int *positions, void *q_out, void *k_out, int B, int T, int Hq,
                           int Hkv, int dh, int rot, double base, float eps, int io,
                           void *stream) {
  int st = check_heads(B, T, Hq, Hkv, dh, io);
  if (st != RGLRU_OK) return st;
  QkArgs a = {};
  a.B = B;
  a.T = T;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.dh = dh;
  if ((st = set_rotation(&a, rot, base, eps)) != RGLRU_OK) return st;
  if (!given(q) || !given(k) || !given(q_out) || !given(k_out) || !optional_ok(w_q) ||
      !optional_ok(w_k) || !optional_ok(positions))
    return RGLRU_ERR_INVALID_ARG;
  Span sq, sk;
  if (!view(q, q_strides, B, T, Hq, dh, io, &a.q, &sq) ||
      !view(k, k_strides, B, T, Hkv, dh, io, &a.k, &sk))
    return RGLRU_ERR_INVALID_ARG;
  const long long rows = static_cast<long long>(B) * T;
  const Span ins[] = {sq, sk, dense(w_q, dh, io), dense(w_k, dh, io), bytes_of(positions, 4 * rows)};
  const Span outs[] = {dense(q_out, rows * Hq * dh, io), dense(k_out, rows * Hkv * dh, io)};
  if (overlapping(ins, outs)) return RGLRU_ERR_INVALID_ARG;
  a.w_q = w_q;
  a.w_k = w_k;
  a.positions = positions;
  a.q_out = q_out;
  a.k_out = k_out;
  return launch_qk_fwd(a, io, static_cast<cudaStream_t>(stream)) == cudaSuccess ? RGLRU_OK
                                                                               : RGLRU_ERR_CUDA;
}

int rglru_qk_norm_rope_append(const void *q, const rglru_strides *q_strides, const void *k,
                              const rglru_strides *k_strides, const void *v,
                              const rglru_strides *v_strides, const void *w_q, const void *w_k,
                              const int *positions, void *q_out, void *k_cache, void *v_cache,
                              const int *page_table, int num_pages, int page_size, int max_pages,
                              int B, int T, int Hq, int Hkv, int dh, int rot, double base,
                              float eps, int io, int *dev_status, void *stream) {
  int st = check_heads(B, T, Hq, Hkv, dh, io);
  if (st != RGLRU_OK) return st;
  if (num_pages < 1 || page_size < 1 || max_pages < 1) return RGLRU_ERR_INVALID_ARG;
  QkArgs a = {};
  a.B = B;
  a.T = T;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.dh = dh;
  if ((st = set_rotation(&a, rot, base, eps)) != RGLRU_OK) return st;
  if (!given(q) || !given(k) || !given(v) || !given(positions) || !given(q_out) ||
      !given(k_cache) || !given(v_cache) || !given(page_table) || !optional_ok(w_q) ||
      !optional_ok(w_k) || !optional_ok(dev_status))
    return RGLRU_ERR_INVALID_ARG;
  Span sq, sk, sv;
  if (!view(q, q_strides, B, T, Hq, dh, io, &a.q, &sq) ||
      !view(k, k_strides, B, T, Hkv, dh, io, &a.k, &sk) ||
      !view(v, v_strides, B, T, Hkv, dh, io, &a.v, &sv))
    return RGLRU_ERR_INVALID_ARG;
  const long long rows = static_cast<long long>(B) * T;
  const long long slots = static_cast<long long>(num_pages) * page_size;
  if (slots > (1ll << 46) / (static_cast<long long>(Hkv) * dh)) return RGLRU_ERR_UNSUPPORTED;
  const long long cache = slots * Hkv * dh;
  const Span ins[] = {sq, sk, sv, dense(w_q, dh, io), dense(w_k, dh, io),
                      bytes_of(positions, 4 * rows),
                      bytes_of(page_table, 4ll * B * max_pages)};
  const Span outs[] = {dense(q_out, rows * Hq * dh, io), dense(k_cache, cache, io),
                       dense(v_cache, cache, io), bytes_of(dev_status, 4)};
  if (overlapping(ins, outs)) return RGLRU_ERR_INVALID_ARG;
  a.w_q = w_q;
  a.w_k = w_k;
  a.positions = positions;
  a.q_out = q_out;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.page_table = page_table;
  a.num_pages = num_pages;
  a.page_size = page_size;
  a.max_pages = max_pages;
  a.dev_status = dev_status;
  return launch_qk_append(a, io, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? RGLRU_OK
             : RGLRU_ERR_CUDA;
}

size_t rglru_qk_norm_rope_bwd_workspace_bytes(int B, int T, int Hq, int Hkv, int dh, int io) {
  if (check_heads(B, T, Hq, Hkv, dh, io) != RGLRU_OK) return 0;
  return align_up(qk_bwd_workspace_bytes(B, T, Hq, Hkv, dh), 256);
}

int rglru_qk_norm_rope_bwd(const void *q, const rglru_strides *q_strides, const void *k,
                           const rglru_strides *k_strides, const void *w_q, const void *w_k,
                           const int *positions, const void *dq_out, const void *dk_out, void *dq,
                           void *dk, float *dw_q, float *dw_k, int B, int T, int Hq, int Hkv,
                           int dh, int rot, double base, float eps, int io, void *workspace,
                           size_t workspace_bytes, void *stream) {
  int st = check_heads(B, T, Hq, Hkv, dh, io);
  if (st != RGLRU_OK) return st;
  QkArgs a = {};
  a.B = B;
  a.T = T;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.dh = dh;
  if ((st = set_rotation(&a, rot, base, eps)) != RGLRU_OK) return st;
  if (!given(q) || !given(k) || !given(dq_out) || !given(dk_out) || !given(dq) || !given(dk) ||
      !optional_ok(w_q) || !optional_ok(w_k) || !optional_ok(positions) || !optional_ok(dw_q) ||
      !optional_ok(dw_k))
    return RGLRU_ERR_INVALID_ARG;
  Span sq, sk;
  if (!view(q, q_strides, B, T, Hq, dh, io, &a.q, &sq) ||
      !view(k, k_strides, B, T, Hkv, dh, io, &a.k, &sk))
    return RGLRU_ERR_INVALID_ARG;
  const size_t need = rglru_qk_norm_rope_bwd_workspace_bytes(B, T, Hq, Hkv, dh, io);
  if (!given(workspace) || workspace_bytes < need) return RGLRU_ERR_WORKSPACE;
  const long long rows = static_cast<long long>(B) * T;
  const Span ins[] = {sq, sk, dense(w_q, dh, io), dense(w_k, dh, io), bytes_of(positions, 4 * rows),
                      dense(dq_out, rows * Hq * dh, io), dense(dk_out, rows * Hkv * dh, io)};
  const Span outs[] = {dense(dq, rows * Hq * dh, io), dense(dk, rows * Hkv * dh, io),
                       bytes_of(dw_q, 4 * dh), bytes_of(dw_k, 4 * dh),
                       {workspace, need}};
  if (overlapping(ins, outs)) return RGLRU_ERR_INVALID_ARG;
  a.w_q = w_q;
  a.w_k = w_k;
  a.positions = positions;
  a.dq_out = dq_out;
  a.dk_out = dk_out;
  a.q_out = dq;
  a.k_out = dk;
  a.dw_q = dw_q;
  a.dw_k = dw_k;
  return launch_qk_bwd(a, io, workspace, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? RGLRU_OK
             : RGLRU_ERR_CUDA;
}

int rglru_local_attn_fwd(const void *q, const rglru_strides *q_strides, const void *k,
                         const rglru_strides *k_strides, const void *v,
                         const rglru_strides *v_strides, const int *lens, void *out, float *lse,
                         int B, int T, int S, int Hq, int Hkv, int dh, int window, int sinks,
                         float scale, int io, int *dev_status, void *stream) {
  AttnArgs a = {};
  a.B = B;
  a.T = T;
  a.S = S;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.dh = dh;
  a.window = window;
  a.sinks = sinks;
  a.scale = scale;
  int st = check_attn(&a, io);
  if (st != RGLRU_OK) return st;
  if (!scale_ok(scale) || (lens != nullptr && S != T)) return RGLRU_ERR_INVALID_ARG;
  if (!given(q) || !given(k) || !given(v) || !given(out) || !optional_ok(lens) ||
      !optional_ok(lse) || !optional_ok(dev_status))
    return RGLRU_ERR_INVALID_ARG;
  Span sq, sk, sv;
  if (!view(q, q_strides, B, T, Hq, dh, io, &a.q, &sq) ||
      !view(k, k_strides, B, S, Hkv, dh, io, &a.k, &sk) ||
      !view(v, v_strides, B, S, Hkv, dh, io, &a.v, &sv))
    return RGLRU_ERR_INVALID_ARG;
  const long long rows = static_cast<long long>(B) * T * Hq;
  const Span ins[] = {sq, sk, sv, bytes_of(lens, 4ll * B)};
  const Span outs[] = {dense(out, rows * dh, io), bytes_of(lse, 4 * rows), bytes_of(dev_status, 4)};
  if (overlapping(ins, outs)) return RGLRU_ERR_INVALID_ARG;
  a.lens = lens;
  a.out = out;
  a.lse = lse;
  a.dev_status = dev_status;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e =
      attn_tc_supported(a, io) ? launch_attn_fwd_tc(a, s) : launch_attn_fwd_generic(a, io, s);
  return e == cudaSuccess ? RGLRU_OK : RGLRU_ERR_CUDA;
}

size_t rglru_local_attn_bwd_workspace_bytes(int B, int T, int S, int Hq, int Hkv, int dh,
                                            int window, int sinks, int io) {
  AttnArgs a = {};
  a.B = B;
  a.T = T;
  a.S = S;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.dh = dh;
  a.window = window;
  a.sinks = sinks;
  if (check_attn(&a, io) != RGLRU_OK) return 0;
  return align_up(attn_tc_supported(a, io) ? attn_bwd_tc_workspace_bytes(a)
                                           : attn_bwd_generic_workspace_bytes(a),
                  256);
}

int rglru_local_attn_bwd(const void *q, const rglru_strides *q_strides, const void *k,
                         const rglru_strides *k_strides, const void *v,
                         const rglru_strides *v_strides, const void *out, const float *lse,
                         const void *dout, const int *lens, void *dq, void *dk, void *dv, int B,
                         int T, int S, int Hq, int Hkv, int dh, int window, int sinks,
                         float scale, int io, void *workspace, size_t workspace_bytes,
                         int *dev_status, void *stream) {
  AttnArgs a = {};
  a.B = B;
  a.T = T;
  a.S = S;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.dh = dh;
  a.window = window;
  a.sinks = sinks;
  a.scale = scale;
  int st = check_attn(&a, io);
  if (st != RGLRU_OK) return st;
  if (!scale_ok(scale) || (lens != nullptr && S != T)) return RGLRU_ERR_INVALID_ARG;
  if (!given(q) || !given(k) || !given(v) || !given(out) || !given(lse) || !given(dout) ||
      !given(dq) || !given(dk) || !given(dv) || !optional_ok(lens) || !optional_ok(dev_status))
    return RGLRU_ERR_INVALID_ARG;
  Span sq, sk, sv;
  if (!view(q, q_strides, B, T, Hq, dh, io, &a.q, &sq) ||
      !view(k, k_strides, B, S, Hkv, dh, io, &a.k, &sk) ||
      !view(v, v_strides, B, S, Hkv, dh, io, &a.v, &sv))
    return RGLRU_ERR_INVALID_ARG;
  const size_t need = rglru_local_attn_bwd_workspace_bytes(B, T, S, Hq, Hkv, dh, window, sinks, io);
  if (!given(workspace) || workspace_bytes < need) return RGLRU_ERR_WORKSPACE;
  const long long rows = static_cast<long long>(B) * T * Hq, keys = static_cast<long long>(B) * S * Hkv;
  const Span ins[] = {sq, sk, sv, dense(out, rows * dh, io), bytes_of(lse, 4 * rows),
                      dense(dout, rows * dh, io), bytes_of(lens, 4ll * B)};
  const Span outs[] = {dense(dq, rows * dh, io), dense(dk, keys * dh, io), dense(dv, keys * dh, io),
                       {workspace, need}, bytes_of(dev_status, 4)};
  if (overlapping(ins, outs)) return RGLRU_ERR_INVALID_ARG;
  a.lens = lens;
  a.out = const_cast<void *>(out);
  a.lse = const_cast<float *>(lse);
  a.dout = dout;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  a.dev_status = dev_status;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = attn_tc_supported(a, io) ? launch_attn_bwd_tc(a, workspace, s)
                                                 : launch_attn_bwd_generic(a, io, workspace, s);
  return e == cudaSuccess ? RGLRU_OK : RGLRU_ERR_CUDA;
}

}  // extern "C"

namespace {

int check_decode(const DecodeArgs &a, int io) {
  const int st = check_heads(a.B, 1, a.Hq, a.Hkv, a.dh, io);
  if (st != RGLRU_OK) return st;
  if (a.Hq % a.Hkv != 0 || a.page_size < 1 || a.max_pages < 1 || a.window < 0 || a.sinks < 0)
    return RGLRU_ERR_INVALID_ARG;
  if (static_cast<long long>(a.page_size) * a.max_pages > kMaxInt) return RGLRU_ERR_UNSUPPORTED;
  return RGLRU_OK;
}

}  // namespace

extern "C" {

size_t rglru_paged_attn_decode_workspace_bytes(int B, int Hq, int Hkv, int dh, int page_size,
                                               int max_pages, int window, int sinks, int io) {
  DecodeArgs a = {};
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.dh = dh;
  a.page_size = page_size;
  a.max_pages = max_pages;
  a.window = window;
  a.sinks = sinks;
  if (check_decode(a, io) != RGLRU_OK) return 0;
  const size_t need = align_up(paged_decode_workspace_bytes(a, io), 256);
  return need < 256 ? 256 : need;
}

int rglru_paged_attn_decode(const void *q, const void *k_cache, const void *v_cache,
                            const int *page_table, const int *lens, void *out, int num_pages,
                            int page_size, int max_pages, int B, int Hq, int Hkv, int dh,
                            int window, int sinks, float scale, int io, void *workspace,
                            size_t workspace_bytes, int *dev_status, void *stream) {
  DecodeArgs a = {q, k_cache, v_cache, page_table, lens, out, num_pages, page_size, max_pages,
                  B, Hq, Hkv, dh, window, sinks, scale, dev_status};
  const int st = check_decode(a, io);
  if (st != RGLRU_OK) return st;
  if (num_pages < 1 || !scale_ok(scale)) return RGLRU_ERR_INVALID_ARG;
  if (!given(q) || !given(k_cache) || !given(v_cache) || !given(page_table) || !given(lens) ||
      !given(out) || !optional_ok(dev_status))
    return RGLRU_ERR_INVALID_ARG;
  const long long slots = static_cast<long long>(num_pages) * page_size;
  if (slots > (1ll << 46) / (static_cast<long long>(Hkv) * dh)) return RGLRU_ERR_UNSUPPORTED;
  const size_t need =
      rglru_paged_attn_decode_workspace_bytes(B, Hq, Hkv, dh, page_size, max_pages, window, sinks, io);
  if (!given(workspace) || workspace_bytes < need) return RGLRU_ERR_WORKSPACE;
  const long long rows = static_cast<long long>(B) * Hq, cache = slots * Hkv * dh;
  const Span ins[] = {dense(q, rows * dh, io), dense(k_cache, cache, io), dense(v_cache, cache, io),
                      bytes_of(page_table, 4ll * B * max_pages), bytes_of(lens, 4ll * B)};
  const Span outs[] = {dense(out, rows * dh, io), {workspace, need}, bytes_of(dev_status, 4)};
  if (overlapping(ins, outs)) return RGLRU_ERR_INVALID_ARG;
  return launch_paged_decode(a, io, workspace, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? RGLRU_OK
             : RGLRU_ERR_CUDA;
}

}  // extern "C"
