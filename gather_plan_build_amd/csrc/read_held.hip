// read_held.hip -- rows held in 8 bits back as rows of their type (gfx950).
//
// A code times its head's scale, a power of two: exact in the row's type, no
// rounding.  Bound by HBM: a held row is read once, a plain one, twice as long,
// written once.  A lane takes eight codes, so that its 16 bytes of result are next
// to its neighbour's; a workgroup takes some rows, the chunks of all of them
// numbered through.  217,280 latent rows (143 MB to 250): 68 us repeated without
// pause, 5.7 TB/s.  72 with plain stores, 74 and 70 with eight and two chunks of a
// lane under way, 68 with the divisions as products.
#include "held.h"

namespace gpb {
namespace {

constexpr int kAhead = 4;  // chunks of a lane under way at once

struct ReadArgs {
  const uint8_t *rows;
  const int32_t *locs;
  uint8_t *out;
  int64_t n_src_rows;
  int32_t n_rows, row_bytes, out_row_bytes;
  int32_t chunks, code_chunks;    // of a row: all, and those of codes
  int32_t k_chunks, v_chunks;     // of a head
  int32_t k_end;                  // chunks of all key heads
  int32_t hkv, plain_at, scales_at;
  int32_t per_block;              // rows of a workgroup
  int32_t *status;
};

template <typename T>
__global__ __launch_bounds__(kBlock) void k_rows_read(ReadArgs a) {
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * a.per_block;
  const int n = static_cast<int>(std::min<int64_t>(a.per_block, a.n_rows - row0));
  const int total = n * a.chunks;
  for (int u0 = threadIdx.x; u0 < total; u0 += kAhead * kBlock) {
    u32x4 raw[kAhead];
    uint32_t scale[kAhead];
    bool code[kAhead], some[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int u = min(u0 + i * kBlock, total - 1);
      const int r = u / a.chunks, c = u - r * a.chunks;
      const int64_t loc = a.locs ? a.locs[row0 + r] : row0 + r;
      some[i] = loc >= 0 && loc < a.n_src_rows;
      if (!some[i] && loc != -1 && c == 0 && a.status) atomicOr(a.status, GPB_STATUS_BAD_DESCRIPTOR);
      const uint8_t *src = a.rows + (some[i] ? loc : 0) * a.row_bytes;
      code[i] = c < a.code_chunks;
      raw[i] = u32x4{};
      scale[i] = 0;
      if (!some[i]) continue;
      if (code[i]) {
        const bool key = c < a.k_end;
        const int head = key ? c / a.k_chunks : a.hkv + (c - a.k_end) / a.v_chunks;
        const u32x2 eight = *reinterpret_cast<const u32x2 *>(src + 8 * c);
        raw[i][0] = eight[0];
        raw[i][1] = eight[1];
        scale[i] = src[a.scales_at + head];
      } else {
        typedef u32x4 Loose4 __attribute__((aligned(8)));
        raw[i] = *reinterpret_cast<const Loose4 *>(src + a.plain_at + 16 * (c - a.code_chunks));
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int u = u0 + i * kBlock;
      if (u >= total) break;
      const int r = u / a.chunks, c = u - r * a.chunks;
      u32x4 x = raw[i];
      if (code[i])
        x = some[i] ? __builtin_bit_cast(u32x4, values8<T>(u32x2{raw[i][0], raw[i][1]},
                                                           scale_of(scale[i])))
                    : u32x4{};
      __builtin_nontemporal_store(
          x, reinterpret_cast<u32x4 *>(a.out + (row0 + r) * a.out_row_bytes + 16 * c));
    }
  }
}

int rows_read(const gpb_row_format *f, const void *d_rows, int64_t n_src_rows,
              const int32_t *d_locs, int32_t n_rows, void *d_out, int32_t out_row_bytes,
              int32_t *d_status, void *stream) {
  int rc = check_format(f);
  if (rc != GPB_OK) return rc;
  if (!held(f) || n_src_rows < 0 || n_rows < 0) return GPB_EINVAL;
  if (n_src_rows > INT32_MAX) return GPB_ERANGE;
  gpb_row_format plain = *f;
  plain.dtype = type_of(f);
  plain.row_bytes = out_row_bytes;
  rc = check_format(&plain);
  if (rc != GPB_OK) return rc;
  if (n_rows == 0) return GPB_OK;
  if (!d_out || (n_src_rows > 0 && !d_rows) || (!d_locs && n_rows > n_src_rows)) return GPB_EINVAL;
  if (!aligned(d_rows, 16) || !aligned(d_out, 16) || !aligned(d_locs, 4) || !aligned(d_status, 4))
    return GPB_EALIGN;
  const HeldRow row(*f);
  ReadArgs a = {};
  a.rows = static_cast<const uint8_t *>(d_rows);
  a.locs = d_locs;
  a.out = static_cast<uint8_t *>(d_out);
  a.n_src_rows = n_src_rows; a.n_rows = n_rows;
  a.row_bytes = f->row_bytes; a.out_row_bytes = out_row_bytes;
  a.code_chunks = static_cast<int32_t>(row.codes / 8);
  a.chunks = a.code_chunks + static_cast<int32_t>(row.plain / 16);
  a.hkv = f->n_kv_heads;
  a.k_chunks = (f->values_in_key ? f->v_dim : f->k_dim) / 8;
  a.v_chunks = f->v_dim / 8;
  a.k_end = a.hkv * a.k_chunks;
  a.plain_at = static_cast<int32_t>(row.codes);
  a.scales_at = static_cast<int32_t>(row.codes + row.plain);
  a.per_block = std::max(1, kAhead * kBlock / a.chunks);
  a.status = d_status;
  const int64_t blocks = ceil_div64(n_rows, a.per_block);
  if (blocks > UINT32_MAX / kBlock) return GPB_ERANGE;  // (a launch has fewer than 2^32 threads)
  const dim3 grid(static_cast<uint32_t>(blocks));
  return plain.dtype == GPB_BF16
             ? launch(k_rows_read<__bf16>, grid, dim3(kBlock), as_stream(stream), a)
             : launch(k_rows_read<_Float16>, grid, dim3(kBlock), as_stream(stream), a);
}

}  // namespace
}  // namespace gpb

extern "C" int gpb_rows_read(const gpb_row_format *format, const void *d_rows,
                             int64_t n_src_rows, const int32_t *d_locs, int32_t n_rows,
                             void *d_out, int32_t out_row_bytes, int32_t *d_status,
                             void *stream) {
  return gpb::rows_read(format, d_rows, n_src_rows, d_locs, n_rows, d_out, out_row_bytes,
                        d_status, stream);
}
