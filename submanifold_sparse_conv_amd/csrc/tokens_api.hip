// C ABI of the token operators (declared in include/tr_sparseconv.h): argument
// checks, workspace layout, launches.
#include "token_checks.h"

using namespace trsc;

namespace {

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
  c = check_window(who, win);
  if (c != TR_SC_OK) return c;
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
