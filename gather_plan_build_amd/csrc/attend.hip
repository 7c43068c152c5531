// attend.hip -- attention over composed or paged rows: the calls, and the kernels
// of rows of 16 bits a value (gfx950).
#include "attend_kernel.h"

namespace gpb {
namespace {

int attend(const gpb_attend_plan *p, const int32_t *d_list, const gpb_attend_io *io,
           const void *d_rows, int64_t n_rows, const int32_t *d_pages, int64_t n_listed,
           const int32_t *d_base, int64_t pages_stride, bool paged, void *d_workspace,
           int64_t workspace_bytes, int32_t *d_status, void *stream) {
  if (!p || !io) return GPB_EINVAL;
  int rc = check_format(&p->format);
  if (rc != GPB_OK) return rc;
  const int which = attend_kernel(p->format);
  if (which < 0 || p->bs < 0 || p->n_heads < 1 || p->n_heads % p->format.n_kv_heads ||
      p->n_tokens < 0 || p->max_keys < 0 || p->n_items < 0 || p->n_wide < 0 || p->n_joins < 0 || p->n_refs < 0 ||
      p->n_partial_rows < 0 || p->window < 0 || p->sinks < 0 || p->page_rows < 1 ||
      p->list_ints < 0)
    return GPB_EINVAL;
  const int64_t items = static_cast<int64_t>(p->n_items) * kItemInts;
  if (p->joins_at != items ||
      p->refs_at != items + static_cast<int64_t>(p->n_joins) * kJoinInts ||
      p->positions_at != static_cast<int64_t>(p->refs_at) + p->n_refs ||
      p->list_ints != static_cast<int64_t>(p->positions_at) + p->n_tokens ||
      p->workspace_bytes !=
          static_cast<int64_t>(p->n_partial_rows) * (p->format.v_dim + 2) * 4)
    return GPB_EINVAL;
  if (!(io->scale > 0.0f) || std::isinf(io->scale)) return GPB_EINVAL;
  if (!paged && p->n_groups > 0) return GPB_EINVAL;
  if (n_rows < 0 || n_listed < 0 || pages_stride < 0 || workspace_bytes < 0) return GPB_EINVAL;
  if (n_rows > INT32_MAX) return GPB_ERANGE;
  if (p->n_tokens == 0) return GPB_OK;
  if (p->bs == 0) return GPB_EINVAL;
  if (!d_list || !io->d_q || !io->d_out) return GPB_EINVAL;
  if (workspace_bytes < p->workspace_bytes || (p->workspace_bytes > 0 && !d_workspace))
    return GPB_EINVAL;
  int64_t usable = n_rows;
  if (paged) usable = n_rows / p->page_rows * p->page_rows;
  if (p->max_keys > 0) {
    if (!d_rows || usable < 1) return GPB_EINVAL;
    if (!paged && !d_base) return GPB_EINVAL;
    if (paged) {
      if (!d_pages || n_listed < 1) return GPB_EINVAL;
      if (!d_base && (pages_stride < ceil_div64(p->max_keys, p->page_rows) ||
                      pages_stride > n_listed / p->bs))
        return GPB_EINVAL;
    }
  }
  if (!aligned(d_list, 16) || !aligned(io->d_q, 16) || !aligned(io->d_out, 8) ||
      !aligned(io->d_lse, 4) || !aligned(d_rows, 16) || !aligned(d_pages, 4) ||
      !aligned(d_base, 4) || !aligned(d_workspace, 16) || !aligned(d_status, 4) ||
      io->q_token_stride % 8 || io->q_head_stride % 8 || io->out_token_stride % 4 ||
      io->out_head_stride % 4)
    return GPB_EALIGN;
  if (!apart(p->n_tokens, p->n_heads, p->format.v_dim, io->out_token_stride, io->out_head_stride))
    return GPB_EINVAL;

  AttendArgs a = {};
  a.list = d_list;
  a.q = static_cast<const uint16_t *>(io->d_q);
  a.q_ts = io->q_token_stride; a.q_hs = io->q_head_stride;
  a.rows = static_cast<const uint8_t *>(d_rows);
  a.n_rows = usable;
  a.pages = paged ? d_pages : nullptr;
  a.base = d_base; a.n_listed = n_listed; a.pages_stride = pages_stride;
  a.out = static_cast<uint16_t *>(io->d_out);
  a.o_ts = io->out_token_stride; a.o_hs = io->out_head_stride;
  a.lse = io->d_lse;
  a.sums = static_cast<float *>(d_workspace);
  a.ml = a.sums + static_cast<int64_t>(p->n_partial_rows) * p->format.v_dim;
  a.status = d_status;
  a.c = io->scale * 1.44269504088896341f;
  plan_args(*p, &a);
  a.n_pages = static_cast<int32_t>(usable / p->page_rows);
  const bool narrow = p->n_wide == 0;
  if (held(&p->format))
    return launch_attend_held(type_of(&p->format), which, a, narrow, as_stream(stream));
  return p->format.dtype == GPB_BF16
             ? launch_format<__bf16, Attend>(which, a, narrow, as_stream(stream))
             : launch_format<_Float16, Attend>(which, a, narrow, as_stream(stream));
}

}  // namespace
}  // namespace gpb

extern "C" int gpb_attend_dense(const gpb_attend_plan *plan, const int32_t *d_list,
                                const gpb_attend_io *io, const void *d_dense,
                                int64_t n_dense_rows, const int32_t *d_k_bases,
                                void *d_workspace, int64_t workspace_bytes, int32_t *d_status,
                                void *stream) {
  return gpb::attend(plan, d_list, io, d_dense, n_dense_rows, nullptr, 0, d_k_bases, 0, false,
                     d_workspace, workspace_bytes, d_status, stream);
}

extern "C" int gpb_attend_paged(const gpb_attend_plan *plan, const int32_t *d_list,
                                const gpb_attend_io *io, const void *d_pool,
                                int64_t n_pool_rows, const int32_t *d_pages,
                                int64_t n_pages_listed, const int32_t *d_page_base,
                                int64_t pages_stride, void *d_workspace,
                                int64_t workspace_bytes, int32_t *d_status, void *stream) {
  return gpb::attend(plan, d_list, io, d_pool, n_pool_rows, d_pages, n_pages_listed,
                     d_page_base, pages_stride, true, d_workspace, workspace_bytes, d_status,
                     stream);
}
