// C ABI of the token operators (declared in include/tr_sparseconv.h): argument
// checks, workspace layout, launches.
#include <cmath>
#include <cstdint>

#include "tokens.h"
#include "tr_sparseconv.h"

using namespace trsc;

namespace {

constexpr int64_t kMaxTokens = int64_t(1) << 30;
constexpr int kMaxHeads = 4096;

inline size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

int elem_bytes(int dtype) { return dtype == TR_SC_F32 ? 4 : 2; }

int check_kind(const char* who, int64_t tokens, int dim, int dtype) {
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
int check_heads(const char* who, const char* name, const tr_sc_heads* t, int64_t tokens, int heads, int dim,
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

View view_of(const char* name, const tr_sc_heads* t, int64_t tokens, int dim, int dtype) {
  const int64_t b = elem_bytes(dtype);
  return View{name, reinterpret_cast<int64_t>(t->data), t->token_stride * b, t->head_stride * b, tokens, t->heads, dim * b};
}
View packed_view(const char* name, const void* p, int64_t tokens, int64_t heads, int64_t dim, int64_t bytes) {
  return View{name, reinterpret_cast<int64_t>(p), heads * dim * bytes, dim * bytes, tokens, heads, dim * bytes};
}

// Whether a step s of [lo, hi] brings [d + s ts, d + s ts + len) onto [0, width).
bool meets(wide_t d, int64_t ts, int64_t lo, int64_t hi, int64_t len, int64_t width) {
  if (ts == 0) return d < width && d + len > 0;
  // the first step whose end passes 0
  wide_t s = -(d + len) / ts - 1;
  while (d + s * ts + len <= 0) ++s;
  s = s < lo ? lo : s;
  return s <= hi && d + s * ts + len > 0 && d + s * ts < width;
}

bool overlap(const View& a, const View& b) {
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

bool rows_overlap(const View& a) {  // of one view
  if (a.tokens == 0 || (a.heads - 1) * a.hs + a.dim <= a.ts || (a.tokens - 1) * a.ts + a.dim <= a.hs) return false;
  if (a.tokens > 1 && a.ts < a.dim) return true;
  for (int64_t h = 1; h < a.heads; ++h)
    if (meets(h * a.hs, a.ts, 1 - a.tokens, a.tokens - 1, a.dim, a.dim)) return true;
  return false;
}

bool same_view(const View& a, const View& b) {
  return a.at == b.at && a.tokens == b.tokens && a.heads == b.heads && (a.tokens <= 1 || a.ts == b.ts) &&
         (a.heads <= 1 || a.hs == b.hs);
}

// Each output's own rows, and each against the inputs and the outputs before it. in_place[i] (may be null): views
// that output i may be itself.
struct Output {
  View view;
  const View* in_place[2];
};
int check_overlap(const char* who, const Output* outs, int n_outs, const View* ins, int n_ins) {
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

int check_workspace(const char* who, const void* ws, size_t have, size_t need) {
  if (have < need) return fail(TR_SC_ERR_WORKSPACE, "%s: workspace %zu bytes < %zu needed", who, have, need);
  if (need > 0 && (ws == nullptr || reinterpret_cast<uintptr_t>(ws) % 256 != 0))
    return fail(TR_SC_ERR_INVALID_ARG, "%s: workspace NULL or not 256-byte aligned", who);
  return TR_SC_OK;
}

int check_head_count(const char* who, const tr_sc_heads* t, const char* name) {
  if (t == nullptr) return fail(TR_SC_ERR_INVALID_ARG, "%s: %s is NULL", who, name);
  if (t->heads < 1 || t->heads > kMaxHeads)
    return fail(TR_SC_ERR_INVALID_ARG, "%s: %s has %d heads, out of [1, %d]", who, name, t->heads, kMaxHeads);
  return TR_SC_OK;
}

// The rotation's and gains' part of a norm call.
int fill_norm(const char* who, const tr_sc_heads* q, const tr_sc_heads* k, const tr_sc_rotation* rot,
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

void set_out(NormSide* s, const tr_sc_heads* t) {
  s->y = t->data;
  s->yts = t->token_stride;
  s->yhs = t->head_stride;
}

void set_grad(NormSide* s, const tr_sc_heads* t) {
  s->dy = t->data;
  s->dts = t->token_stride;
  s->dhs = t->head_stride;
}

HeadsRef ref(const tr_sc_heads* t) { return HeadsRef{t->data, t->token_stride, t->head_stride}; }

// Whether 32 rows of a query-like tensor (rows: token by token, in a token the
// heads that share a key-value head) lie within 2^30 bytes of the first.
bool rows_reach(const tr_sc_heads* t, const tr_sc_heads* k, int bytes) {
  const int64_t group = t->heads / k->heads, tokens = 32 / group + 2;
  const int64_t most = int64_t(1) << 30;
  return t->token_stride * bytes < most / tokens && t->head_stride * bytes < most / group &&
         tokens * t->token_stride * bytes + group * t->head_stride * bytes < most;
}

// Everything of an attention call but its outputs.
int fill_attn(const char* who, const tr_sc_heads* q, const tr_sc_heads* k, const tr_sc_heads* v,
              const tr_sc_window* win, int64_t nq, int64_t nk, int dim, int dtype, AttnArgs* a) {
  int c = check_kind(who, nq, dim, dtype);
  if (c == TR_SC_OK) c = check_kind(who, nk, dim, dtype);
  if (c == TR_SC_OK) c = check_head_count(who, q, "q");
  if (c == TR_SC_OK) c = check_head_count(who, k, "k");
  if (c == TR_SC_OK) c = check_heads(who, "q", q, nq, q->heads, dim, dtype, false);
  if (c == TR_SC_OK) c = check_heads(who, "k", k, nk, k->heads, dim, dtype, false);
  if (c == TR_SC_OK) c = check_heads(who, "v", v, nk, k->heads, dim, dtype, false);
  if (c != TR_SC_OK) return c;
  if (q->heads % k->heads != 0)
    return fail(TR_SC_ERR_INVALID_ARG, "%s: %d query heads are no multiple of %d key-value heads", who, q->heads,
                k->heads);
  if (win == nullptr) return fail(TR_SC_ERR_INVALID_ARG, "%s: window is NULL", who);
  if (win->batch < 1 || win->batch > (1 << 20))
    return fail(TR_SC_ERR_INVALID_ARG, "%s: batch = %d out of [1, 2^20]", who, win->batch);
  if (win->batch > 1 && (win->cu_q == nullptr || win->cu_k == nullptr))
    return fail(TR_SC_ERR_INVALID_ARG, "%s: more than one sequence needs cu_q and cu_k", who);
  if (win->left < -1 || win->right < -1)
    return fail(TR_SC_ERR_INVALID_ARG, "%s: window (%lld, %lld): a side is >= 0, or -1 for no limit", who,
                (long long)win->left, (long long)win->right);
  if (win->sinks < 0 || win->sinks > kMaxSinks)
    return fail(TR_SC_ERR_INVALID_ARG, "%s: sinks = %d out of [0, %d]", who, win->sinks, kMaxSinks);
  if (!(win->scale > 0.f) || std::isinf(win->scale))
    return fail(TR_SC_ERR_INVALID_ARG, "%s: scale = %g, a positive number is needed", who, double(win->scale));
  if (int64_t(win->batch) * k->heads * (win->sinks + 1) >= (int64_t(1) << 31) ||
      nq * (q->heads / k->heads) + int64_t(1024) * (win->batch + 1) >= (int64_t(1) << 31) ||
      nq * q->heads >= (int64_t(1) << 33) || nk + int64_t(128) * (win->batch + 1) >= (int64_t(1) << 31))
    return fail(TR_SC_ERR_UNSUPPORTED, "%s: too many rows", who);
  // a tile's rows lie within 32-bit offsets of its first
  const int64_t reach = int64_t(1) << 30;
  const int bytes = elem_bytes(dtype);
  if (k->token_stride * bytes >= reach / 64 || v->token_stride * bytes >= reach / 64 || !rows_reach(q, k, bytes))
    return fail(TR_SC_ERR_UNSUPPORTED, "%s: strides too large", who);
  *a = AttnArgs{};
  a->q = ref(q);
  a->k = ref(k);
  a->v = ref(v);
  a->cu_q = win->cu_q;
  a->cu_k = win->cu_k;
  a->k_len = win->k_len;
  a->batch = win->batch;
  a->nq = int32_t(nq);
  a->nk = int32_t(nk);
  a->hq = q->heads;
  a->hk = k->heads;
  a->dim = dim;
  a->dtype = dtype;
  a->left = win->left < 0 || win->left > kFar ? kFar : int32_t(win->left);
  a->right = win->right < 0 || win->right > kFar ? kFar : int32_t(win->right);
  a->sinks = win->sinks;
  a->scale = win->scale;
  return TR_SC_OK;
}

// The sizes of a workspace query, as the arguments of a call that has them; false if no call has.
bool sizes_only(const tr_sc_window* win, int64_t nq, int64_t nk, int q_heads, int kv_heads, int dim, int dtype,
                AttnArgs* a) {
  const tr_sc_heads q{reinterpret_cast<void*>(16), 0, 0, q_heads}, k{reinterpret_cast<void*>(16), 0, 0, kv_heads};
  return fill_attn("workspace", &q, &k, &k, win, nq, nk, dim, dtype, a) == TR_SC_OK;
}

struct BackwardLayout {
  size_t stat, exps, sinks, parts, total;
};
BackwardLayout backward_layout(const AttnArgs& a) {
  BackwardLayout l{};
  l.stat = 0;
  l.exps = align_up(attention_backward_stat_floats(a) * 4, 256);
  l.sinks = l.exps + align_up(attention_backward_exponents(a) * 4, 256);
  l.parts = l.sinks + align_up(attention_backward_sink_floats(a) * 4, 256);
  l.total = l.parts + align_up(attention_backward_part_floats(a) * 4, 256);
  return l;
}

}  // namespace

extern "C" {

int tr_sparseconv_qk_norm_rope(const tr_sc_heads* q, const tr_sc_heads* k, const tr_sc_rotation* rot,
                               const float* q_gain, int q_gain_rows, const float* k_gain, int k_gain_rows, float eps,
                               const tr_sc_heads* q_out, const tr_sc_heads* k_out, int64_t tokens, int dim, int dtype,
                               void* stream) {
  const char* who = "qk_norm_rope";
  NormArgs a;
  int c = fill_norm(who, q, k, rot, q_gain, q_gain_rows, k_gain, k_gain_rows, eps, tokens, dim, dtype, &a);
  if (c == TR_SC_OK) c = check_heads(who, "q_out", q_out, tokens, q->heads, dim, dtype, true);
  if (c == TR_SC_OK) c = check_heads(who, "k_out", k_out, tokens, k->heads, dim, dtype, true);
  if (c != TR_SC_OK) return c;
  const View ins[] = {view_of("q", q, tokens, dim, dtype), view_of("k", k, tokens, dim, dtype)};
  const Output outs[] = {{view_of("q_out", q_out, tokens, dim, dtype), {&ins[0], nullptr}},
                         {view_of("k_out", k_out, tokens, dim, dtype), {&ins[1], nullptr}}};
  c = check_overlap(who, outs, 2, ins, 2);
  if (c != TR_SC_OK) return c;
  set_out(&a.q, q_out);
  set_out(&a.k, k_out);
  const hipError_t e = launch_norm_rope(a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? TR_SC_OK : hip_fail(e, who);
}

size_t tr_sparseconv_qk_norm_rope_backward_workspace_bytes(int64_t tokens, int q_heads, int kv_heads, int dim) {
  if (tokens < 0 || tokens > kMaxTokens || q_heads < 1 || kv_heads < 1 || q_heads > kMaxHeads ||
      kv_heads > kMaxHeads || dim <= 0 || dim % 8 != 0 || dim > kMaxHeadDim)
    return 0;
  return align_up(size_t(norm_rope_partials(tokens, q_heads + kv_heads, dim)) * 4, 256);
}

int tr_sparseconv_qk_norm_rope_backward(const tr_sc_heads* dq_out, const tr_sc_heads* dk_out, const tr_sc_heads* q,
                                        const tr_sc_heads* k, const tr_sc_rotation* rot, const float* q_gain,
                                        int q_gain_rows, const float* k_gain, int k_gain_rows, float eps,
                                        const tr_sc_heads* dq, const tr_sc_heads* dk, float* dq_gain, float* dk_gain,
                                        int64_t tokens, int dim, int dtype, void* workspace, size_t ws_bytes,
                                        void* stream) {
  const char* who = "qk_norm_rope_backward";
  NormArgs a;
  int c = fill_norm(who, q, k, rot, q_gain, q_gain_rows, k_gain, k_gain_rows, eps, tokens, dim, dtype, &a);
  if (c == TR_SC_OK) c = check_heads(who, "dq_out", dq_out, tokens, q->heads, dim, dtype, false);
  if (c == TR_SC_OK) c = check_heads(who, "dk_out", dk_out, tokens, k->heads, dim, dtype, false);
  if (c == TR_SC_OK) c = check_heads(who, "dq", dq, tokens, q->heads, dim, dtype, true);
  if (c == TR_SC_OK) c = check_heads(who, "dk", dk, tokens, k->heads, dim, dtype, true);
  if (c == TR_SC_OK)
    c = check_workspace(who, workspace, ws_bytes,
                        tr_sparseconv_qk_norm_rope_backward_workspace_bytes(tokens, q->heads, k->heads, dim));
  if (c != TR_SC_OK) return c;
  const View ins[] = {view_of("q", q, tokens, dim, dtype), view_of("k", k, tokens, dim, dtype),
                      view_of("dq_out", dq_out, tokens, dim, dtype), view_of("dk_out", dk_out, tokens, dim, dtype)};
  const Output outs[] = {{view_of("dq", dq, tokens, dim, dtype), {&ins[0], &ins[2]}},
                         {view_of("dk", dk, tokens, dim, dtype), {&ins[1], &ins[3]}}};
  c = check_overlap(who, outs, 2, ins, 4);
  if (c != TR_SC_OK) return c;
  if ((dq_gain != nullptr && q_gain == nullptr) || (dk_gain != nullptr && k_gain == nullptr))
    return fail(TR_SC_ERR_INVALID_ARG, "%s: the gradient of a gain that is not there", who);
  if (reinterpret_cast<uintptr_t>(dq_gain) % 16 != 0 || reinterpret_cast<uintptr_t>(dk_gain) % 16 != 0)
    return fail(TR_SC_ERR_INVALID_ARG, "%s: dq_gain and dk_gain must be 16-byte aligned", who);
  set_grad(&a.q, dq_out);
  set_grad(&a.k, dk_out);
  set_out(&a.q, dq);
  set_out(&a.k, dk);
  a.q.dgain = dq_gain;
  a.k.dgain = dk_gain;
  a.partials = static_cast<float*>(workspace);
  const hipError_t e = launch_norm_rope_backward(a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? TR_SC_OK : hip_fail(e, who);
}

size_t tr_sparseconv_window_attention_workspace_bytes(const tr_sc_window* win, int64_t tokens_q, int64_t tokens_k,
                                                      int q_heads, int kv_heads, int dim, int dtype) {
  AttnArgs a;
  if (!sizes_only(win, tokens_q, tokens_k, q_heads, kv_heads, dim, dtype, &a)) return 0;
  return align_up(plan_attention(a).part_floats * 4, 256);
}

int tr_sparseconv_window_attention(const tr_sc_heads* q, const tr_sc_heads* k, const tr_sc_heads* v,
                                   const tr_sc_window* win, const tr_sc_heads* out, float* lse, int64_t tokens_q,
                                   int64_t tokens_k, int dim, int dtype, void* workspace, size_t ws_bytes,
                                   void* stream) {
  const char* who = "window_attention";
  AttnArgs a;
  int c = fill_attn(who, q, k, v, win, tokens_q, tokens_k, dim, dtype, &a);
  if (c == TR_SC_OK) c = check_heads(who, "out", out, tokens_q, q->heads, dim, dtype, true);
  if (c != TR_SC_OK) return c;
  const AttnPlan plan = plan_attention(a);
  c = check_workspace(who, workspace, ws_bytes, align_up(plan.part_floats * 4, 256));
  if (c != TR_SC_OK) return c;
  const View ins[] = {view_of("q", q, tokens_q, dim, dtype), view_of("k", k, tokens_k, dim, dtype),
                      view_of("v", v, tokens_k, dim, dtype)};
  const Output outs[] = {{view_of("out", out, tokens_q, dim, dtype), {nullptr, nullptr}},
                         {packed_view("lse", lse, lse != nullptr ? q->heads : 0, 1, tokens_q, 4), {nullptr, nullptr}}};
  c = check_overlap(who, outs, 2, ins, 3);
  if (c != TR_SC_OK) return c;
  a.o = ref(out);
  a.lse = lse;
  a.part = static_cast<float*>(workspace);
  const hipError_t e = launch_attention(a, plan, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? TR_SC_OK : hip_fail(e, who);
}

size_t tr_sparseconv_window_attention_backward_workspace_bytes(const tr_sc_window* win, int64_t tokens_q,
                                                               int64_t tokens_k, int q_heads, int kv_heads, int dim,
                                                               int dtype) {
  AttnArgs a;
  if (!sizes_only(win, tokens_q, tokens_k, q_heads, kv_heads, dim, dtype, &a)) return 0;
  return backward_layout(a).total;
}

int tr_sparseconv_window_attention_backward(const tr_sc_heads* dout, const tr_sc_heads* q, const tr_sc_heads* k,
                                            const tr_sc_heads* v, const tr_sc_heads* out, const float* lse,
                                            const tr_sc_window* win, void* dq, void* dk, void* dv, int64_t tokens_q,
                                            int64_t tokens_k, int dim, int dtype, void* workspace, size_t ws_bytes,
                                            void* stream) {
  const char* who = "window_attention_backward";
  AttnArgs a;
  int c = fill_attn(who, q, k, v, win, tokens_q, tokens_k, dim, dtype, &a);
  if (c == TR_SC_OK) c = check_heads(who, "dout", dout, tokens_q, q->heads, dim, dtype, false);
  if (c == TR_SC_OK) c = check_heads(who, "out", out, tokens_q, q->heads, dim, dtype, false);
  if (c != TR_SC_OK) return c;
  if (!rows_reach(dout, k, elem_bytes(dtype))) return fail(TR_SC_ERR_UNSUPPORTED, "%s: strides too large", who);
  if ((tokens_q > 0 && (lse == nullptr || dq == nullptr)) || (tokens_k > 0 && (dk == nullptr || dv == nullptr)))
    return fail(TR_SC_ERR_INVALID_ARG, "%s: NULL tensor", who);
  if (reinterpret_cast<uintptr_t>(dq) % 16 != 0 || reinterpret_cast<uintptr_t>(dk) % 16 != 0 ||
      reinterpret_cast<uintptr_t>(dv) % 16 != 0)
    return fail(TR_SC_ERR_INVALID_ARG, "%s: dq, dk and dv must be 16-byte aligned", who);
  const BackwardLayout l = backward_layout(a);
  c = check_workspace(who, workspace, ws_bytes, l.total);
  if (c != TR_SC_OK) return c;
  const View ins[] = {view_of("q", q, tokens_q, dim, dtype),       view_of("k", k, tokens_k, dim, dtype),
                      view_of("v", v, tokens_k, dim, dtype),       view_of("out", out, tokens_q, dim, dtype),
                      view_of("dout", dout, tokens_q, dim, dtype), packed_view("lse", lse, q->heads, 1, tokens_q, 4)};
  const int b = elem_bytes(dtype);
  const Output outs[] = {{packed_view("dq", dq, tokens_q, q->heads, dim, b), {nullptr, nullptr}},
                         {packed_view("dk", dk, tokens_k, k->heads, dim, b), {nullptr, nullptr}},
                         {packed_view("dv", dv, tokens_k, k->heads, dim, b), {nullptr, nullptr}}};
  c = check_overlap(who, outs, 3, ins, 6);
  if (c != TR_SC_OK) return c;
  a.dout = ref(dout);
  a.o = ref(out);
  a.lse = const_cast<float*>(lse);
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  a.stat = reinterpret_cast<float2*>(static_cast<char*>(workspace) + l.stat);
  a.score_exp = reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + l.exps);
  a.dkv_part = reinterpret_cast<float*>(static_cast<char*>(workspace) + l.parts);
  a.sink_part = reinterpret_cast<float*>(static_cast<char*>(workspace) + l.sinks);
  const hipError_t e = launch_attention_backward(a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? TR_SC_OK : hip_fail(e, who);
}

}  // extern "C"
