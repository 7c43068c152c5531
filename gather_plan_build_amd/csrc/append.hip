// append.hip -- cache rows made from keys and values, the keys and the
// queries of the same tokens rotated by their positions (gfx950).
//
// Pair (x, y) of a head at position p becomes (x cos a - y sin a,
// y cos a + x sin a), a = p * inv_freq[i], computed in fp32 from the row's
// type and rounded to it once.  The angle is the one place where fp32 is not
// enough: at position 10^6 the product's rounding alone is 0.03 rad.  It is
// formed in fp64 as a fraction of a turn and its nearest whole turn taken off;
// the fraction, at most one half, then goes to fp32 sine and cosine of
// pi * 2 fraction, so every position has the error of a first turn.
//
// Bound by HBM: every key, value and query is read once and written once (the
// rows twice when the compose wants them token-packed).  A workgroup takes one
// token: its first rot_dim / 2 lanes make the sines into LDS, shared by all
// heads, then every lane moves 16-byte chunks, two chunks where the pair's
// halves lie rot_dim / 2 apart, so that a head can be rotated in place.
// 44,600 tokens of latent rows and 16 query heads of 576 values to the pool and
// token-packed: 316 us for 1.80 GB, 5.7 TB/s, where large copies reach 4.9 to 6.7;
// 4,099 tokens of 28 query and 4 + 4 other heads of 128: 15.7 us for 75.6 MB (4.8
// TB/s); 8 tokens: 4 us, the launch and two trips to HBM.
#include "append.h"

namespace gpb {
namespace {

template <typename T>
__global__ __launch_bounds__(kBlock) void k_row_append(AppendArgs a) {
  __shared__ __attribute__((aligned(16))) float s_cos[kMaxPairs], s_sin[kMaxPairs];
  const int64_t t = blockIdx.x;
  find_turns<float>(a, t, threadIdx.x, s_cos, s_sin);
  __syncthreads();
  const int64_t loc = a.locs ? a.locs[t] : -1;
  const bool stored = loc >= 0 && loc < a.n_pool_rows;
  if (a.locs && !stored && loc != -1 && threadIdx.x == 0 && a.status)
    atomicOr(a.status, GPB_STATUS_BAD_STAGING_ROW);
  uint8_t *to_pool = stored ? a.pool + loc * a.row_bytes : nullptr;
  uint8_t *to_rows = a.rows ? a.rows + t * a.row_bytes : nullptr;

  const int n_k = a.hkv * a.head_units, n_q = a.hq * a.head_units;
  const int v_units = a.has_v ? a.vd / 8 : 0;
  const int total = n_k + n_q + a.hkv * v_units;
  for (int u = threadIdx.x; u < total; u += kBlock) {
    if (u >= n_k + n_q) {  // a value chunk
      const int x = u - n_k - n_q;
      const int h = x / v_units, c = x - h * v_units;
      const u32x4 val = load16(a.v + t * a.v_ts + h * a.v_hs + c * 8);
      const int64_t off = 2ll * (a.hkv * a.kd + h * a.vd + c * 8);
      if (to_pool) store16(to_pool + off, val);
      if (to_rows) store16(to_rows + off, val);
      continue;
    }
    const bool key = u < n_k;
    const int x = key ? u : u - n_k;
    const int h = x / a.head_units, j = x - h * a.head_units;
    const uint16_t *src = key ? a.k + t * a.k_ts + h * a.k_hs : a.q + t * a.q_ts + h * a.q_hs;
    int e0, e1;
    u32x4 lo, hi;
    rotate_unit<T>(a, src, j, s_cos, s_sin, &e0, &e1, &lo, &hi);
    if (key) {
      const int64_t off = 2ll * (h * a.kd + e0), off1 = 2ll * (h * a.kd + e1);
      if (to_pool) {
        store16(to_pool + off, lo);
        if (e1 >= 0) store16(to_pool + off1, hi);
      }
      if (to_rows) {
        store16(to_rows + off, lo);
        if (e1 >= 0) store16(to_rows + off1, hi);
      }
    } else {
      uint8_t *dst = reinterpret_cast<uint8_t *>(a.q_out + t * a.qo_ts + h * a.qo_hs);
      store16(dst + 2 * e0, lo);
      if (e1 >= 0) store16(dst + 2 * e1, hi);
    }
  }
}

bool whole_chunks(int64_t stride) { return stride % 8 == 0; }

int row_append(const gpb_row_format *f, const gpb_append *p, int32_t *d_status, void *stream) {
  int rc = check_format(f);
  if (rc != GPB_OK) return rc;
  if (!p || p->n_rows < 0 || p->n_q_heads < 0 || p->n_q_heads > 65536 ||
      p->n_pool_rows < 0) return GPB_EINVAL;
  // (a launch has fewer than 2^32 threads)
  if (p->n_pool_rows > INT32_MAX || p->n_rows > static_cast<int64_t>(UINT32_MAX / kBlock))
    return GPB_ERANGE;
  if (p->rot_dim < 0 || p->rot_dim > 2 * kMaxPairs || p->rot_dim % 16 || p->rot_start < 0 ||
      p->rot_start % 8 || p->rot_start > f->k_dim - p->rot_dim ||
      (p->interleaved != 0 && p->interleaved != 1))
    return GPB_EINVAL;
  if (p->rot_dim > 0) {
    if (p->n_axes < 1 || p->n_axes > GPB_MAX_AXES) return GPB_EINVAL;
    int64_t sum = 0;
    for (int x = 0; x < p->n_axes; ++x) {
      if (p->section[x] < 0) return GPB_EINVAL;
      sum += p->section[x];
    }
    if (sum != p->rot_dim / 2) return GPB_EINVAL;
  }
  if (p->n_rows == 0) return GPB_OK;
  const bool has_v = !f->values_in_key, has_q = p->d_q != nullptr;
  if (!p->d_k || (has_v && !p->d_v) || (has_q && (!p->d_q_out || p->n_q_heads < 1)))
    return GPB_EINVAL;
  if ((p->d_pool != nullptr) != (p->d_pool_locs != nullptr) || (!p->d_pool && p->n_pool_rows))
    return GPB_EINVAL;
  if (!p->d_pool && !p->d_rows) return GPB_EINVAL;
  if (p->rot_dim > 0 && (!p->d_inv_freq || !p->d_positions)) return GPB_EINVAL;
  if (has_q && p->d_q == p->d_q_out &&
      (p->q_token_stride != p->qo_token_stride || p->q_head_stride != p->qo_head_stride))
    return GPB_EINVAL;
  if (!aligned(p->d_k, 16) || !aligned(p->d_v, 16) || !aligned(p->d_pool, 16) ||
      !aligned(p->d_rows, 16) || !aligned(p->d_q, 16) || !aligned(p->d_q_out, 16) ||
      !aligned(p->d_pool_locs, 4) || !aligned(p->d_inv_freq, 4) ||
      !aligned(p->d_positions, 4) || !aligned(d_status, 4))
    return GPB_EALIGN;
  if (!whole_chunks(p->k_token_stride) || !whole_chunks(p->k_head_stride) ||
      (has_v && (!whole_chunks(p->v_token_stride) || !whole_chunks(p->v_head_stride))) ||
      (has_q && (!whole_chunks(p->q_token_stride) || !whole_chunks(p->q_head_stride) ||
                 !whole_chunks(p->qo_token_stride) || !whole_chunks(p->qo_head_stride))))
    return GPB_EALIGN;
  if (has_q && !apart(p->n_rows, p->n_q_heads, f->k_dim, p->qo_token_stride, p->qo_head_stride))
    return GPB_EINVAL;

  AppendArgs a = {};
  a.k = static_cast<const uint16_t *>(p->d_k);
  a.v = static_cast<const uint16_t *>(p->d_v);
  a.q = static_cast<const uint16_t *>(p->d_q);
  a.q_out = static_cast<uint16_t *>(p->d_q_out);
  a.pool = static_cast<uint8_t *>(p->d_pool);
  a.rows = static_cast<uint8_t *>(p->d_rows);
  a.locs = p->d_pool_locs; a.positions = p->d_positions; a.inv_freq = p->d_inv_freq;
  a.k_ts = p->k_token_stride; a.k_hs = p->k_head_stride;
  a.v_ts = p->v_token_stride; a.v_hs = p->v_head_stride;
  a.q_ts = p->q_token_stride; a.q_hs = p->q_head_stride;
  a.qo_ts = p->qo_token_stride; a.qo_hs = p->qo_head_stride;
  a.positions_stride = p->positions_stride;
  a.n_pool_rows = p->n_pool_rows;
  a.row_bytes = f->row_bytes; a.hkv = f->n_kv_heads; a.hq = has_q ? p->n_q_heads : 0;
  a.kd = f->k_dim; a.vd = f->v_dim; a.has_v = has_v;
  a.rot_start = p->rot_start; a.pairs = p->rot_dim / 2; a.interleaved = p->interleaved;
  int32_t end = 0;
  for (int x = 0; x < GPB_MAX_AXES; ++x) {
    end = x < p->n_axes - 1 ? end + p->section[x] : INT32_MAX;
    a.axis_end[x] = end;
  }
  a.pair_units = p->interleaved ? 0 : p->rot_dim / 16;
  a.head_units = f->k_dim / 8 - a.pair_units;
  a.status = d_status;
  if (held(f)) return launch_append_held(*f, a, p->n_rows, as_stream(stream));
  const dim3 grid(static_cast<uint32_t>(p->n_rows));
  return f->dtype == GPB_BF16
             ? launch(k_row_append<__bf16>, grid, dim3(kBlock), as_stream(stream), a)
             : launch(k_row_append<_Float16>, grid, dim3(kBlock), as_stream(stream), a);
}

}  // namespace
}  // namespace gpb

extern "C" int gpb_row_append(const gpb_row_format *format, const gpb_append *append,
                              int32_t *d_status, void *stream) {
  return gpb::row_append(format, append, d_status, stream);
}
