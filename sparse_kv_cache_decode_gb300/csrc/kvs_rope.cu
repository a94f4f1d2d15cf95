// Rotation of query and key rows, host side: the handle, and the C-ABI entry point over dense rows.
#include <math.h>

#include <new>

#include "kvs_rope.cuh"

using namespace kvs;

namespace {

bool rope_dims(const kvs_rope_config* c, RopeDims* d) {
  if (!c || (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)) return false;
  if (c->rot_dim < 0 || c->rot_dim > c->head_dim || c->rot_dim % 16) return false;
  if ((c->adjacent != 0 && c->adjacent != 1) || c->n_axis < 1 || c->n_axis > kRopeMaxAxes) return false;
  if (!(c->rot_scale >= 0.f) || isinf(c->rot_scale) || !(c->norm_eps >= 0.f) || isinf(c->norm_eps)) return false;
  const int n = c->rot_dim / 2;
  if (n && c->n_axis > 1 && !c->axis) return false;
  if (n && !c->inv_freq && (!(c->theta > 0) || isinf(c->theta))) return false;
  *d = RopeDims{};
  d->d = c->head_dim;
  d->rot = c->rot_dim;
  d->n_axis = c->n_axis;
  d->adjacent = c->adjacent;
  d->rot_scale = c->rot_scale > 0.f ? c->rot_scale : 1.f;
  d->eps = c->norm_eps;
  for (int i = 0; i < n; ++i) {
    const double f = c->inv_freq ? c->inv_freq[i] : pow(c->theta, -2.0 * i / c->rot_dim);
    if (!isfinite(f)) return false;
    // turns per position, to [-1/2, 1/2): the error is a rounding of f / (2 pi), 2^-53 of it
    double turns = f / 6.283185307179586476925286766559;
    turns -= nearbyint(turns);
    if (turns >= 0.5) turns -= 1.0;
    d->freq[i] = (unsigned long long)(long long)ldexp(turns, 64);
    d->axis[i] = c->axis ? c->axis[i] : 0;
    if (d->axis[i] >= c->n_axis) return false;
  }
  return true;
}

// Rows of `n` heads of d elements of n_tok tokens: 16-byte aligned vectors, no two rows sharing an element (a token's heads
// together, or a head's tokens together).
bool rows_ok(const void* p, long long tok, long long head, int n, int d, int n_tok) {
  if (!p || (reinterpret_cast<uintptr_t>(p) & 15u) || tok % 8 || head % 8) return false;
  if ((n > 1 && head < d) || (n_tok > 1 && tok < d)) return false;
  constexpr long long most = 1ll << 40;      // (extents stay in 64 bits, and within any memory)
  if ((n > 1 && head > most / n) || (n_tok > 1 && tok > most / n_tok)) return false;
  return n == 1 || n_tok <= 1 || tok >= (n - 1) * head + d || head >= (n_tok - 1) * tok + d;
}

struct Span {
  uintptr_t p;
  long long tok, head;   // bytes
  int n, n_tok, d;       // d: bytes of a head
  uintptr_t end() const { return p + (size_t)(n_tok - 1) * tok + (size_t)(n - 1) * head + d; }
};
Span span(const void* p, long long tok, long long head, int n, int d, int n_tok) {
  Span s = {reinterpret_cast<uintptr_t>(p), tok * 2, head * 2, n, n_tok, d * 2};
  if (n == 1) s.head = s.d;
  if (n_tok == 1) s.tok = (n - 1) * s.head + s.d;
  return s;
}
// Whether `at` + i * step lies within (-d, d) for a whole i in [lo, hi] (lo <= 0 <= hi, step >= d).
bool comes_near(long long at, long long step, int lo, int hi, int d) {
  if (at > -d && at < d) return true;
  const long long i = at > 0 ? -(at / step) : -at / step;      // rounded towards `at`'s side; the other neighbour is one further
  for (const long long k : {i, at > 0 ? i - 1 : i + 1})
    if (k >= lo && k <= hi && at + k * step > -d && at + k * step < d) return true;
  return false;
}
// Whether the two may share a byte.  Apart are: all of both; columns of rows of the same length; heads of the same stride
// between one another's; and, found row by row, the rows of two of the same strides or of single tokens.  (A stride that
// only one of them has, because the other has a single head, is the stride of both.)  Strides that differ otherwise: they may.
bool may_meet(const Span& a, const Span& b) {
  if (a.end() <= b.p || b.end() <= a.p) return false;
  const Span &x = a.p <= b.p ? a : b, &y = a.p <= b.p ? b : a;
  const long long off = (long long)(y.p - x.p);
  const int d = x.d, n_tok = x.n_tok;      // (the same of both)
  auto apart = [](long long off, long long period, long long wx, long long wy) {
    const long long o = off % period;
    return o >= wx && o + wy <= period;
  };
  if (n_tok > 1 && x.tok == y.tok && apart(off, x.tok, (x.n - 1) * x.head + d, (y.n - 1) * y.head + d)) return false;
  if (x.n == 1 || y.n == 1 || x.head == y.head) {
    const long long head = x.n > 1 ? x.head : y.head;
    if ((n_tok == 1 || (x.tok == y.tok && x.tok % head == 0)) && apart(off, head, d, d)) return false;
    if (n_tok > 1 && x.tok != y.tok) return true;
    const int ahead = n_tok - 1;
    for (int j = 1 - x.n; j < y.n; ++j)      // y's head less x's
      if (comes_near(off + j * head, n_tok > 1 ? x.tok : d, -ahead, ahead, d)) return true;
    return false;
  }
  if (n_tok > 1) return true;
  for (int j = 0; j < x.n; ++j)
    if (comes_near(off - j * x.head, y.head, 0, y.n - 1, d)) return true;
  return false;
}
bool same(const Span& a, const Span& b) { return a.p == b.p && a.n == b.n && a.tok == b.tok && a.head == b.head; }

}  // namespace

extern "C" {

kvs_status kvs_rope_create(const kvs_rope_config* cfg, kvs_rope** out) try {
  if (!out) return KVS_ERR_INVALID_ARG;
  *out = nullptr;
  RopeDims d;
  if (!rope_dims(cfg, &d)) return KVS_ERR_INVALID_ARG;
  kvs_rope* r = new (std::nothrow) kvs_rope;
  if (!r) return KVS_ERR_INVALID_ARG;
  r->d = d;
  *out = r;
  return KVS_OK;
} catch (...) {      // out of host memory
  return KVS_ERR_CUDA;
}

kvs_status kvs_rope_destroy(kvs_rope* rope) {
  if (!rope) return KVS_ERR_INVALID_ARG;
  delete rope;
  return KVS_OK;
}

kvs_status kvs_rotate(const kvs_rope* rope, const void* d_q, long long q_stride, long long q_head_stride, int n_q_head,
                      const float* d_q_norm, void* d_q_out, long long q_out_stride, long long q_out_head_stride, const void* d_k,
                      long long k_stride, long long k_head_stride, int n_k_head, const float* d_k_norm, void* d_k_out,
                      long long k_out_stride, long long k_out_head_stride, const int* d_pos, long long pos_stride, int n_tok,
                      kvs_stream_t stream) try {
  if (!rope || n_tok < 0 || n_q_head < 0 || n_k_head < 0 || n_q_head > 1024 || n_k_head > 1024 || pos_stride < 0) return KVS_ERR_INVALID_ARG;
  if (n_tok == 0 || n_q_head + n_k_head == 0) return KVS_OK;
  if (!d_pos) return KVS_ERR_INVALID_ARG;
  const int d = rope->d.d;
  const void* src[2] = {d_q, d_k};
  void* dst[2] = {d_q_out, d_k_out};
  const float* norm[2] = {d_q_norm, d_k_norm};
  const int n[2] = {n_q_head, n_k_head};
  const long long s_tok[2] = {q_stride, k_stride}, s_head[2] = {q_head_stride, k_head_stride};
  const long long o_tok[2] = {q_out_stride, k_out_stride}, o_head[2] = {q_out_head_stride, k_out_head_stride};
  Span in[2], out[2];
  for (int i = 0; i < 2; ++i) {
    if (!n[i]) continue;
    if (!rows_ok(src[i], s_tok[i], s_head[i], n[i], d, n_tok) || !rows_ok(dst[i], o_tok[i], o_head[i], n[i], d, n_tok)) return KVS_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(norm[i]) & 15u) return KVS_ERR_INVALID_ARG;
    in[i] = span(src[i], s_tok[i], s_head[i], n[i], d, n_tok);
    out[i] = span(dst[i], o_tok[i], o_head[i], n[i], d, n_tok);
  }
  // rows are written while others are still read: in place, or apart
  for (int o = 0; o < 2; ++o)
    for (int i = 0; i < 2; ++i)
      if (n[o] && n[i] && ((!(o == i && same(out[o], in[i])) && may_meet(out[o], in[i])) || (o < i && may_meet(out[o], out[i]))))
        return KVS_ERR_INVALID_ARG;
  RopeRows a = {};
  a.q = {static_cast<const __nv_bfloat16*>(d_q), static_cast<__nv_bfloat16*>(d_q_out), q_stride, q_head_stride, q_out_stride,
         q_out_head_stride, d_q_norm, n_q_head};
  a.k = {static_cast<const __nv_bfloat16*>(d_k), static_cast<__nv_bfloat16*>(d_k_out), k_stride, k_head_stride, k_out_stride,
         k_out_head_stride, d_k_norm, n_k_head};
  a.pos = d_pos;
  a.pos_stride = pos_stride;
  a.n_tok = n_tok;
  return launch_rope_rows(rope->d, a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? KVS_OK : KVS_ERR_CUDA;
} catch (...) {      // out of host memory
  return KVS_ERR_CUDA;
}

}  // extern "C"
