// Host-side argument checks shared by the token operators' C entry points: views of
// heads, overlaps of outputs, workspaces, the norm's and rotation's arguments.
#pragma once
#include <cmath>
#include <cstdint>

#include "tokens.h"
#include "tr_sparseconv.h"

namespace trsc {

constexpr int64_t kMaxTokens = int64_t(1) << 30;
constexpr int kMaxHeads = 4096;

inline size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

inline int elem_bytes(int dtype) { return dtype == TR_SC_F32 ? 4 : 2; }

inline int check_kind(const char* who, int64_t tokens, int dim, int dtype) {
  if (dtype != TR_SC_F32 && dtype != TR_SC_BF16 && dtype != TR_SC_F16)
    return fail(TR_SC_ERR_UNSUPPORTED, "%s: dtype %d", who, dtype);
  if (dim <= 0) return fail(TR_SC_ERR_INVALID_ARG, "%s: dim = %d", who, dim);
  if (dim % 8 != 0 || dim > kMaxHeadDim)
    return fail(TR_SC_ERR_UNSUPPORTED, "%s: dim = %d is no multiple of 8 up to %d", who, dim, kMaxHeadDim);
  if (tokens < 0 || tokens > kMaxTokens)
    return fail(TR_SC_ERR_INVALID_ARG, "%s: tokens = %lld out of [0, 2^30]", who, (long long)tokens);
  return TR_SC_OK;
}

// A [tokens, heads, dim] view: 16-byte aligned rows; strides in elements,
// multiples of 16 bytes. `out`: rows must not overlap each other.
inline int check_heads(const char* who, const char* name, const tr_sc_heads* t, int64_t tokens, int heads, int dim,
                       int dtype, bool out) {
  if (t == nullptr) return fail(TR_SC_ERR_INVALID_ARG, "%s: %s is NULL", who, name);
  if (t->heads != heads)
    return fail(TR_SC_ERR_INVALID_ARG, "%s: %s has %d heads, expected %d", who, name, t->heads, heads);
  if (tokens == 0) return TR_SC_OK;
  if (t->data == nullptr) return fail(TR_SC_ERR_INVALID_ARG, "%s: %s is a NULL pointer", who, name);
  const int per = 16 / elem_bytes(dtype);
  if (reinterpret_cast<uintptr_t>(t->data) % 16 != 0 || t->token_stride % per != 0 || t->head_stride % per != 0)
    return fail(TR_SC_ERR_INVALID_ARG, "%s: %s must be 16-byte aligned in pointer and strides", who, name);
  if (t->token_stride < 0 || t->head_stride < 0 || t->token_stride > (int64_t(1) << 40) ||
      t->head_stride > (int64_t(1) << 40))
    return fail(TR_SC_ERR_INVALID_ARG, "%s: %s has a stride out of [0, 2^40]", who, name);
  if (out && ((tokens > 1 && t->token_stride < dim) || (heads > 1 && t->head_stride < dim)))
    return fail(TR_SC_ERR_INVALID_ARG, "%s: rows of %s overlap", who, name);
  return TR_SC_OK;
}

// ---------------------------------------------------------------------------
// Outputs that overlap. A view's elements are, in bytes, `dim` from each of
// at + t ts + h hs, t < tokens, h < heads.
// ---------------------------------------------------------------------------
typedef __int128 wide_t;  // strides up to 2^42 bytes times 2^30 tokens
struct View {
  const char* name;
  int64_t at, ts, hs, tokens, heads, dim;
  wide_t end() const { return wide_t(tokens - 1) * ts + wide_t(heads - 1) * hs + at + dim; }
};

inline View view_of(const char* name, const tr_sc_heads* t, int64_t tokens, int dim, int dtype) {
  const int64_t b = elem_bytes(dtype);
  return View{name, reinterpret_cast<int64_t>(t->data), t->token_stride * b, t->head_stride * b, tokens, t->heads, dim * b};
}
inline View packed_view(const char* name, const void* p, int64_t tokens, int64_t heads, int64_t dim, int64_t bytes) {
  return View{name, reinterpret_cast<int64_t>(p), heads * dim * bytes, dim * bytes, tokens, heads, dim * bytes};
}

// Whether a step s of [lo, hi] brings [d + s ts, d + s ts + len) onto [0, width).
inline bool meets(wide_t d, int64_t ts, int64_t lo, int64_t hi, int64_t len, int64_t width) {
  if (ts == 0) return d < width && d + len > 0;
  // the first step whose end passes 0
  wide_t s = -(d + len) / ts - 1;
  while (d + s * ts + len <= 0) ++s;
  s = s < lo ? lo : s;
  return s <= hi && d + s * ts + len > 0 && d + s * ts < width;
}

inline bool overlap(const View& a, const View& b) {
  if (a.tokens == 0 || b.tokens == 0 || a.heads == 0 || b.heads == 0 || a.dim == 0 || b.dim == 0) return false;
  if (a.end() <= b.at || b.end() <= a.at) return false;
  // Tokens at unlike strides in one range: taken to overlap.
  if (a.tokens > 1 && b.tokens > 1 && a.ts != b.ts) return true;
  const int64_t ts = a.tokens > 1 ? a.ts : b.ts;
  // Slices of the same rows, side by side.
  if (ts > 0) {
    const int64_t d = ((b.at - a.at) % ts + ts) % ts;
    if ((a.heads - 1) * a.hs + a.dim <= d && d + (b.heads - 1) * b.hs + b.dim <= ts) return false;
  }
  // Heads that alternate: each with each, within reason.
  if (a.heads * b.heads > 65536) return true;
  for (int64_t i = 0; i < a.heads; ++i)
    for (int64_t j = 0; j < b.heads; ++j)
      if (meets(b.at + j * b.hs - a.at - i * a.hs, ts, 1 - a.tokens, b.tokens - 1, b.dim, a.dim)) return true;
  return false;
}

inline bool rows_overlap(const View& a) {  // of one view
  if (a.tokens == 0 || (a.heads - 1) * a.hs + a.dim <= a.ts || (a.tokens - 1) * a.ts + a.dim <= a.hs) return false;
  if (a.tokens > 1 && a.ts < a.dim) return true;
  for (int64_t h = 1; h < a.heads; ++h)
    if (meets(h * a.hs, a.ts, 1 - a.tokens, a.tokens - 1, a.dim, a.dim)) return true;
  return false;
}

inline bool same_view(const View& a, const View& b) {
  return a.at == b.at && a.tokens == b.tokens && a.heads == b.heads && (a.tokens <= 1 || a.ts == b.ts) &&
         (a.heads <= 1 || a.hs == b.hs);
}

// Each output's own rows, and each against the inputs and the outputs before it. in_place[i] (may be null): views
// that output i may be itself.
struct Output {
  View view;
  const View* in_place[2];
};
inline int check_overlap(const char* who, const Output* outs, int n_outs, const View* ins, int n_ins) {
  for (int i = 0; i < n_outs; ++i) {
    const View& o = outs[i].view;
    if (rows_overlap(o)) return fail(TR_SC_ERR_INVALID_ARG, "%s: rows of %s overlap", who, o.name);
    for (int j = 0; j < n_ins + i; ++j) {
      const View& x = j < n_ins ? ins[j] : outs[j - n_ins].view;
      const bool allowed = (outs[i].in_place[0] == &x || outs[i].in_place[1] == &x) && same_view(o, x);
      if (!allowed && overlap(o, x)) return fail(TR_SC_ERR_INVALID_ARG, "%s: %s overlaps %s", who, o.name, x.name);
    }
  }
  return TR_SC_OK;
}

inline int check_workspace(const char* who, const void* ws, size_t have, size_t need) {
  if (have < need) return fail(TR_SC_ERR_WORKSPACE, "%s: workspace %zu bytes < %zu needed", who, have, need);
  if (need > 0 && (ws == nullptr || reinterpret_cast<uintptr_t>(ws) % 256 != 0))
    return fail(TR_SC_ERR_INVALID_ARG, "%s: workspace NULL or not 256-byte aligned", who);
  return TR_SC_OK;
}

// The sides, sinks and scale of a window.
inline int check_window(const char* who, const tr_sc_window* win) {
  if (win->left < -1 || win->right < -1)
    return fail(TR_SC_ERR_INVALID_ARG, "%s: window (%lld, %lld): a side is >= 0, or -1 for no limit", who,
                (long long)win->left, (long long)win->right);
  if (win->sinks < 0 || win->sinks > kMaxSinks)
    return fail(TR_SC_ERR_INVALID_ARG, "%s: sinks = %d out of [0, %d]", who, win->sinks, kMaxSinks);
  if (!(win->scale > 0.f) || std::isinf(win->scale))
    return fail(TR_SC_ERR_INVALID_ARG, "%s: scale = %g, a positive number is needed", who, double(win->scale));
  return TR_SC_OK;
}

inline int check_head_count(const char* who, const tr_sc_heads* t, const char* name) {
  if (t == nullptr) return fail(TR_SC_ERR_INVALID_ARG, "%s: %s is NULL", who, name);
  if (t->heads < 1 || t->heads > kMaxHeads)
    return fail(TR_SC_ERR_INVALID_ARG, "%s: %s has %d heads, out of [1, %d]", who, name, t->heads, kMaxHeads);
  return TR_SC_OK;
}

// The rotation's and gains' part of a norm call.
inline int fill_norm(const char* who, const tr_sc_heads* q, const tr_sc_heads* k, const tr_sc_rotation* rot,
                     const float* q_gain, int q_gain_rows, const float* k_gain, int k_gain_rows, float eps, int64_t tokens,
                     int dim, int dtype, NormArgs* a) {
  int c = check_kind(who, tokens, dim, dtype);
  if (c == TR_SC_OK) c = check_head_count(who, q, "q");
  if (c == TR_SC_OK) c = check_head_count(who, k, "k");
  if (c == TR_SC_OK) c = check_heads(who, "q", q, tokens, q->heads, dim, dtype, false);
  if (c == TR_SC_OK) c = check_heads(who, "k", k, tokens, k->heads, dim, dtype, false);
  if (c != TR_SC_OK) return c;
  if (!(eps >= 0.f) || std::isinf(eps)) return fail(TR_SC_ERR_INVALID_ARG, "%s: eps = %g", who, double(eps));
  if (rot == nullptr) return fail(TR_SC_ERR_INVALID_ARG, "%s: rotation is NULL", who);
  if (rot->axes < 1 || rot->axes > 3) return fail(TR_SC_ERR_INVALID_ARG, "%s: %d axes, out of 1 .. 3", who, rot->axes);
  int64_t pairs = 0;
  for (int i = 0; i < rot->axes; ++i) {
    if (rot->pairs[i] < 0) return fail(TR_SC_ERR_INVALID_ARG, "%s: negative pair count", who);
    pairs += rot->pairs[i];
  }
  if (pairs > dim / 2)
    return fail(TR_SC_ERR_INVALID_ARG, "%s: %lld rotated pairs, %d in a head", who, (long long)pairs, dim / 2);
  if (pairs > 0 && tokens > 0 && (rot->pos == nullptr || rot->freqs == nullptr))
    return fail(TR_SC_ERR_INVALID_ARG, "%s: positions or frequencies are NULL", who);
  if (rot->pos_stride < 0 || rot->pos_stride > (int64_t(1) << 40))
    return fail(TR_SC_ERR_INVALID_ARG, "%s: position stride out of [0, 2^40]", who);
  if ((q_gain != nullptr && q_gain_rows != 1 && q_gain_rows != q->heads) ||
      (k_gain != nullptr && k_gain_rows != 1 && k_gain_rows != k->heads))
    return fail(TR_SC_ERR_INVALID_ARG, "%s: a gain has one row or one a head", who);
  // the rows of a gain that is not there are whatever the caller left
  a->q = NormSide{q->data, q->token_stride, q->head_stride, nullptr, 0, 0, nullptr, 0, 0, q_gain,
                  q_gain != nullptr ? q_gain_rows : 1, nullptr, q->heads};
  a->k = NormSide{k->data, k->token_stride, k->head_stride, nullptr, 0, 0, nullptr, 0, 0, k_gain,
                  k_gain != nullptr ? k_gain_rows : 1, nullptr, k->heads};
  a->pos = rot->pos;
  a->pos_ts = rot->pos_stride;
  a->freqs = rot->freqs;
  a->c1 = rot->pairs[0];
  a->c2 = a->c1 + (rot->axes > 1 ? rot->pairs[1] : 0);
  a->c3 = a->c2 + (rot->axes > 2 ? rot->pairs[2] : 0);
  a->interleaved = rot->interleaved != 0;
  a->eps = eps;
  a->tokens = tokens;
  a->dim = dim;
  a->dtype = dtype;
  a->partials = nullptr;
  return TR_SC_OK;
}

inline void set_out(NormSide* s, const tr_sc_heads* t) {
  s->y = t->data;
  s->yts = t->token_stride;
  s->yhs = t->head_stride;
}

inline void set_grad(NormSide* s, const tr_sc_heads* t) {
  s->dy = t->data;
  s->dts = t->token_stride;
  s->dhs = t->head_stride;
}

inline HeadsRef ref(const tr_sc_heads* t) { return HeadsRef{t->data, t->token_stride, t->head_stride}; }

// Whether 32 rows of a query-like tensor (rows: token by token, in a token the
// heads that share a key-value head) lie within 2^30 bytes of the first.
inline bool rows_reach(const tr_sc_heads* t, const tr_sc_heads* k, int bytes) {
  const int64_t group = t->heads / k->heads, tokens = 32 / group + 2;
  const int64_t most = int64_t(1) << 30;
  return t->token_stride * bytes < most / tokens && t->head_stride * bytes < most / group &&
         tokens * t->token_stride * bytes + group * t->head_stride * bytes < most;
}

}  // namespace trsc
