// C ABI of the operators over a paged cache (declared in include/tr_sparseconv.h):
// argument checks, workspace layout, launches.
#include "paged.h"
#include "token_checks.h"

using namespace trsc;

namespace {

// One tensor of pages: elements (page, slot, head, 0 .. dim - 1).
struct PoolView {
  const char* name;
  int64_t at;                // address
  int64_t step[3], count[3];  // page, slot, head; bytes
  int64_t row;
  wide_t end() const {
    wide_t e = at + row;
    for (int i = 0; i < 3; ++i) e += wide_t(count[i] - 1) * step[i];
    return e;
  }
  bool empty() const { return count[0] == 0; }
};

// The levels of more than one element, the inner ones first; returns their number.
int levels_of(const PoolView& p, int (&order)[3]) {
  int n = 0;
  for (int i = 0; i < 3; ++i) {
    if (p.count[i] <= 1) continue;
    int at = n++;
    for (; at > 0 && p.step[order[at - 1]] > p.step[i]; --at) order[at] = order[at - 1];
    order[at] = i;
  }
  return n;
}

// Whether each level's elements fit between two of the next: no element is another's.
bool pool_rows_overlap(const PoolView& p) {
  if (p.empty()) return false;
  int order[3];
  const int n = levels_of(p, order);
  wide_t extent = p.row;
  for (int i = 0; i < n; ++i) {
    if (p.step[order[i]] < extent) return true;
    extent += wide_t(p.count[order[i]] - 1) * p.step[order[i]];
  }
  return false;
}

// Whether two pools whose own rows do not overlap share an element. Of equal strides: rows that are i_l steps apart at
// level l have the distance d + sum i_l step_l. What the inner levels add to is less than a step, so two i_l at each
// level can bring it within a row. Unlike strides in one range are taken to overlap.
bool rows_meet(const PoolView& p, const int* order, int levels, wide_t d) {
  if (levels == 0) return -p.row < d && d < p.row;
  const int64_t step = p.step[order[levels - 1]], most = p.count[order[levels - 1]] - 1;
  const wide_t i = -(d / step) - (d % step > 0 ? 1 : 0);  // the last with d + i step <= 0
  for (int k = 0; k < 2; ++k)
    if (-most <= i + k && i + k <= most && rows_meet(p, order, levels - 1, d + (i + k) * step)) return true;
  return false;
}
bool pools_overlap(const PoolView& a, const PoolView& b) {
  if (a.empty() || a.end() <= b.at || b.end() <= a.at) return false;
  for (int i = 0; i < 3; ++i)
    if (a.count[i] > 1 && a.step[i] != b.step[i]) return true;
  int order[3];
  const int n = levels_of(a, order);
  return rows_meet(a, order, n, wide_t(b.at) - a.at);
}

bool meets_pool(const View& v, const PoolView& p) {
  if (v.tokens == 0 || v.heads == 0 || p.empty()) return false;
  return v.at < p.end() && p.at < v.end();
}

// The pages of a call.
int fill_pool(const char* who, const tr_sc_pages* p, int heads, int dim, int dtype, PoolRef* r, PoolView* k, PoolView* v) {
  if (p == nullptr) return fail(TR_SC_ERR_INVALID_ARG, "%s: pages is NULL", who);
  if (p->heads != heads)
    return fail(TR_SC_ERR_INVALID_ARG, "%s: the pages have %d heads, expected %d", who, p->heads, heads);
  int log2 = 0;
  while (log2 < kMaxPageLog2 && (1 << log2) < p->page_size) ++log2;
  if (p->page_size != 1 << log2 || log2 < kMinPageLog2)
    return fail(TR_SC_ERR_UNSUPPORTED, "%s: page_size = %d is no power of two in [8, 65536]", who, p->page_size);
  if (p->pages < 0 || p->pages >= (int64_t(1) << 31))
    return fail(TR_SC_ERR_INVALID_ARG, "%s: %lld pages, out of [0, 2^31)", who, (long long)p->pages);
  if (p->batch < 1 || p->batch > (1 << 20))
    return fail(TR_SC_ERR_INVALID_ARG, "%s: batch = %d out of [1, 2^20]", who, p->batch);
  if (p->table_pages < 0 || int64_t(p->table_pages) << log2 > kMaxTokens)
    return fail(TR_SC_ERR_INVALID_ARG, "%s: a table of %d pages of %d, out of [0, 2^30] tokens", who, p->table_pages,
                p->page_size);
  if (p->table_stride < 0 || p->table_stride > (int64_t(1) << 40))
    return fail(TR_SC_ERR_INVALID_ARG, "%s: table stride out of [0, 2^40]", who);
  if (p->len == nullptr || (p->table == nullptr && p->table_pages > 0))
    return fail(TR_SC_ERR_INVALID_ARG, "%s: the page table or the lengths are NULL", who);
  const int64_t b = elem_bytes(dtype);
  const int64_t ks[3] = {p->k_page_stride, p->k_slot_stride, p->k_head_stride};
  const int64_t vs[3] = {p->v_page_stride, p->v_slot_stride, p->v_head_stride};
  if (p->pages > 0) {
    if (p->k == nullptr || p->v == nullptr) return fail(TR_SC_ERR_INVALID_ARG, "%s: k or v pages are a NULL pointer", who);
    bool aligned = reinterpret_cast<uintptr_t>(p->k) % 16 == 0 && reinterpret_cast<uintptr_t>(p->v) % 16 == 0;
    for (int i = 0; i < 3; ++i) {
      aligned = aligned && ks[i] * b % 16 == 0 && vs[i] * b % 16 == 0;
      if (ks[i] < 0 || vs[i] < 0 || ks[i] > (int64_t(1) << 40) || vs[i] > (int64_t(1) << 40))
        return fail(TR_SC_ERR_INVALID_ARG, "%s: the pages have a stride out of [0, 2^40]", who);
    }
    if (!aligned)
      return fail(TR_SC_ERR_INVALID_ARG, "%s: the pages must be 16-byte aligned in pointers and strides", who);
    // rows of a page within 32-bit offsets, in units of 16 bytes; those of a copy to LDS in bytes
    const int64_t most = int64_t(1) << 24;
    if (ks[1] * b >= most || vs[1] * b >= most || ks[1] * b * p->page_size >= (most << 12) ||
        vs[1] * b * p->page_size >= (most << 12) || ks[0] * b >= (most << 12) || vs[0] * b >= (most << 12))
      return fail(TR_SC_ERR_UNSUPPORTED, "%s: slot or page strides too large", who);
  }
  *r = PoolRef{p->k, p->v, ks[0], ks[1], ks[2], vs[0], vs[1], vs[2], int32_t(p->pages), log2, p->table, p->table_stride,
               p->pages > 0 ? p->table_pages : 0, p->len};
  *k = PoolView{"k pages", reinterpret_cast<int64_t>(p->k), {}, {p->pages, p->page_size, heads}, dim * b};
  *v = PoolView{"v pages", reinterpret_cast<int64_t>(p->v), {}, {p->pages, p->page_size, heads}, dim * b};
  for (int i = 0; i < 3; ++i) {
    k->step[i] = ks[i] * b;
    v->step[i] = vs[i] * b;
  }
  return TR_SC_OK;
}

int fill_packed(const char* who, const int32_t* cu_q, int batch, int64_t tokens, Packed* s) {
  if (cu_q == nullptr && tokens % batch != 0)
    return fail(TR_SC_ERR_INVALID_ARG, "%s: without cu_q %lld tokens do not divide into %d sequences", who,
                (long long)tokens, batch);
  *s = Packed{cu_q, batch, cu_q == nullptr ? int32_t(tokens / batch) : 0};
  return TR_SC_OK;
}

// Everything of an attention call but its outputs.
int fill_paged(const char* who, const tr_sc_heads* q, const tr_sc_pages* pages, const int32_t* prefix,
               int64_t prefix_len, const tr_sc_window* win, int64_t nq, int dim, int dtype, PagedArgs* a, PoolView* k,
               PoolView* v) {
  int c = check_kind(who, nq, dim, dtype);
  if (c == TR_SC_OK) c = check_head_count(who, q, "q");
  if (c == TR_SC_OK) c = check_heads(who, "q", q, nq, q->heads, dim, dtype, false);
  if (c != TR_SC_OK) return c;
  if (pages == nullptr) return fail(TR_SC_ERR_INVALID_ARG, "%s: pages is NULL", who);
  if (pages->heads < 1 || pages->heads > kMaxHeads)
    return fail(TR_SC_ERR_INVALID_ARG, "%s: the pages have %d heads, out of [1, %d]", who, pages->heads, kMaxHeads);
  if (q->heads % pages->heads != 0)
    return fail(TR_SC_ERR_INVALID_ARG, "%s: %d query heads are no multiple of %d key-value heads", who, q->heads,
                pages->heads);
  *a = PagedArgs{};
  c = fill_pool(who, pages, pages->heads, dim, dtype, &a->pool, k, v);
  if (c != TR_SC_OK) return c;
  if (win == nullptr) return fail(TR_SC_ERR_INVALID_ARG, "%s: window is NULL", who);
  if (win->cu_k != nullptr || win->k_len != nullptr || win->batch != pages->batch)
    return fail(TR_SC_ERR_INVALID_ARG, "%s: a window over pages has their batch, and no cu_k and k_len", who);
  c = check_window(who, win);
  if (c == TR_SC_OK) c = fill_packed(who, win->cu_q, pages->batch, nq, &a->seqs);
  if (c != TR_SC_OK) return c;
  if (prefix_len < 0 || prefix_len + (int64_t(pages->table_pages) << a->pool.log2) > kMaxTokens)
    return fail(TR_SC_ERR_INVALID_ARG, "%s: a prefix of %lld keys, out of [0, 2^30] with the table's", who,
                (long long)prefix_len);
  if (prefix_len > 0 && prefix == nullptr) return fail(TR_SC_ERR_INVALID_ARG, "%s: the prefix's pages are NULL", who);
  if (prefix_len > 0 && pages->pages == 0)
    return fail(TR_SC_ERR_INVALID_ARG, "%s: a prefix without pages", who);
  const int group = q->heads / pages->heads;
  if (nq * group + int64_t(1024) * (win->batch + 1) >= (int64_t(1) << 31) || nq * q->heads >= (int64_t(1) << 33))
    return fail(TR_SC_ERR_UNSUPPORTED, "%s: too many rows", who);
  a->q = ref(q);
  a->prefix = prefix;
  a->prefix_len = int32_t(prefix_len);
  a->nq = int32_t(nq);
  a->hq = q->heads;
  a->hk = pages->heads;
  a->dim = dim;
  a->dtype = dtype;
  a->left = win->left < 0 || win->left > kFar ? kFar : int32_t(win->left);
  a->right = win->right < 0 || win->right > kFar ? kFar : int32_t(win->right);
  a->sinks = win->sinks;
  a->scale = win->scale;
  return TR_SC_OK;
}

int attend(const char* who, const tr_sc_heads* q, const tr_sc_pages* pages, const int32_t* prefix, int64_t prefix_len,
           const tr_sc_window* win, const tr_sc_heads* out, float* lse, int64_t nq, int dim, int dtype, void* workspace,
           size_t ws_bytes, void* stream) {
  PagedArgs a;
  PoolView k, v;
  int c = fill_paged(who, q, pages, prefix, prefix_len, win, nq, dim, dtype, &a, &k, &v);
  if (c == TR_SC_OK) c = check_heads(who, "out", out, nq, q->heads, dim, dtype, true);
  if (c != TR_SC_OK) return c;
  const PagedPlan plan = plan_paged_attention(a);
  if (!plan.fits) return fail(TR_SC_ERR_UNSUPPORTED, "%s: too many rows and keys", who);
  c = check_workspace(who, workspace, ws_bytes, align_up(plan.part_floats * 4, 256));
  if (c != TR_SC_OK) return c;
  const View ins[] = {view_of("q", q, nq, dim, dtype)};
  const Output outs[] = {{view_of("out", out, nq, dim, dtype), {nullptr, nullptr}},
                         {packed_view("lse", lse, lse != nullptr ? q->heads : 0, 1, nq, 4), {nullptr, nullptr}}};
  c = check_overlap(who, outs, 2, ins, 1);
  if (c != TR_SC_OK) return c;
  for (const Output& o : outs)
    if (meets_pool(o.view, k) || meets_pool(o.view, v))
      return fail(TR_SC_ERR_INVALID_ARG, "%s: %s overlaps the pages", who, o.view.name);
  a.o = ref(out);
  a.lse = lse;
  a.part = static_cast<float*>(workspace);
  const hipError_t e = launch_paged_attention(a, plan, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? TR_SC_OK : hip_fail(e, who);
}

}  // namespace

extern "C" {

int tr_sparseconv_qk_norm_rope_append(const tr_sc_heads* q, const tr_sc_heads* k, const tr_sc_heads* v,
                                      const tr_sc_rotation* rot, const float* q_gain, int q_gain_rows,
                                      const float* k_gain, int k_gain_rows, int norm, float eps,
                                      const tr_sc_heads* q_out, const tr_sc_pages* pages, const int32_t* cu_q,
                                      int64_t tokens, int dim, int dtype, void* stream) {
  const char* who = "qk_norm_rope_append";
  NormArgs n;
  int c = fill_norm(who, q, k, rot, q_gain, q_gain_rows, k_gain, k_gain_rows, norm ? eps : 0.f, tokens, dim, dtype, &n);
  if (c == TR_SC_OK) c = check_heads(who, "v", v, tokens, k->heads, dim, dtype, false);
  if (c == TR_SC_OK) c = check_heads(who, "q_out", q_out, tokens, q->heads, dim, dtype, true);
  if (c != TR_SC_OK) return c;
  if (!norm && (q_gain != nullptr || k_gain != nullptr))
    return fail(TR_SC_ERR_INVALID_ARG, "%s: a gain without the norm", who);
  AppendArgs a{};
  PoolView pk, pv;
  c = fill_pool(who, pages, k->heads, dim, dtype, &a.pool, &pk, &pv);
  if (c == TR_SC_OK) c = fill_packed(who, cu_q, pages->batch, tokens, &a.seqs);
  if (c != TR_SC_OK) return c;
  const View ins[] = {view_of("q", q, tokens, dim, dtype), view_of("k", k, tokens, dim, dtype),
                      view_of("v", v, tokens, dim, dtype)};
  const Output outs[] = {{view_of("q_out", q_out, tokens, dim, dtype), {&ins[0], nullptr}}};
  c = check_overlap(who, outs, 1, ins, 3);
  if (c != TR_SC_OK) return c;
  if (pool_rows_overlap(pk) || pool_rows_overlap(pv))
    return fail(TR_SC_ERR_INVALID_ARG, "%s: rows of the pages overlap", who);
  if (pools_overlap(pk, pv)) return fail(TR_SC_ERR_INVALID_ARG, "%s: k pages overlap v pages", who);
  for (const View* x : {&ins[0], &ins[1], &ins[2], &outs[0].view})
    if (meets_pool(*x, pk) || meets_pool(*x, pv))
      return fail(TR_SC_ERR_INVALID_ARG, "%s: %s overlaps the pages", who, x->name);
  a.q = n.q;
  a.k = n.k;
  set_out(&a.q, q_out);
  a.v = ref(v);
  a.pos = n.pos;
  a.pos_ts = n.pos_ts;
  a.freqs = n.freqs;
  a.c1 = n.c1;
  a.c2 = n.c2;
  a.c3 = n.c3;
  a.interleaved = n.interleaved;
  a.norm = norm != 0;
  a.eps = n.eps;
  a.tokens = tokens;
  a.dim = dim;
  a.dtype = dtype;
  const hipError_t e = launch_norm_rope_append(a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? TR_SC_OK : hip_fail(e, who);
}

size_t tr_sparseconv_paged_attention_workspace_bytes(const tr_sc_pages* pages, const tr_sc_window* win,
                                                     int64_t prefix_len, int64_t tokens_q, int q_heads, int dim,
                                                     int dtype) {
  const tr_sc_heads q{reinterpret_cast<void*>(16), 0, 0, q_heads};
  PagedArgs a;
  PoolView k, v;
  const int32_t* const some = reinterpret_cast<const int32_t*>(16);  // not read
  if (fill_paged("workspace", &q, pages, some, prefix_len, win, tokens_q, dim, dtype, &a, &k, &v) != TR_SC_OK) return 0;
  return align_up(plan_paged_attention(a).part_floats * 4, 256);
}

int tr_sparseconv_paged_window_attention(const tr_sc_heads* q, const tr_sc_pages* pages, const tr_sc_window* win,
                                         const tr_sc_heads* out, float* lse, int64_t tokens_q, int dim, int dtype,
                                         void* workspace, size_t ws_bytes, void* stream) {
  return attend("paged_window_attention", q, pages, nullptr, 0, win, out, lse, tokens_q, dim, dtype, workspace, ws_bytes,
                stream);
}

int tr_sparseconv_shared_prefix_attention(const tr_sc_heads* q, const tr_sc_pages* pages, const int32_t* prefix_pages,
                                          int64_t prefix_len, const tr_sc_window* win, const tr_sc_heads* out,
                                          float* lse, int64_t tokens_q, int dim, int dtype, void* workspace,
                                          size_t ws_bytes, void* stream) {
  return attend("shared_prefix_attention", q, pages, prefix_pages, prefix_len, win, out, lse, tokens_q, dim, dtype,
                workspace, ws_bytes, stream);
}

}  // extern "C"
