// The row formats that the append and the attention know, and the vector
// types their values are moved in.
#pragma once

#include "gpb_common.h"

namespace gpb {

// Values of a row's type, eight to a 16-byte chunk (one MFMA operand).
template <typename T>
struct Vec;
template <>
struct Vec<__bf16> {
  typedef __bf16 x8 __attribute__((ext_vector_type(8)));
  typedef __bf16 x4 __attribute__((ext_vector_type(4)));
};
template <>
struct Vec<_Float16> {
  typedef _Float16 x8 __attribute__((ext_vector_type(8)));
  typedef _Float16 x4 __attribute__((ext_vector_type(4)));
};
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// A row's type, and whether its values are held in 8 bits.
inline int type_of(const gpb_row_format *f) { return f->dtype & ~GPB_HELD_E4M3; }
inline bool held(const gpb_row_format *f) { return (f->dtype & GPB_HELD_E4M3) != 0; }

// Bytes of a held row: codes, values in the row's type, scales.
struct HeldRow {
  int64_t codes, plain, scales;
  explicit HeldRow(const gpb_row_format &f)
      : codes(static_cast<int64_t>(f.n_kv_heads) *
              (f.values_in_key ? f.v_dim : f.k_dim + f.v_dim)),
        plain(f.values_in_key ? 2ll * (f.k_dim - f.v_dim) : 0),
        scales(f.values_in_key ? 1 : 2ll * f.n_kv_heads) {}
};

// Bytes of a row's keys and values, or 0 where the format is not valid.
inline int64_t payload_bytes(const gpb_row_format *f) {
  if (type_of(f) != GPB_BF16 && type_of(f) != GPB_FP16) return 0;
  if (f->n_kv_heads < 1 || f->n_kv_heads > 1024 || f->k_dim < 8 || f->k_dim > 1024 ||
      f->k_dim % 8 || f->v_dim < 8 || f->v_dim > 1024 || f->v_dim % 8)
    return 0;
  if (f->values_in_key != 0 && f->values_in_key != 1) return 0;
  if (f->values_in_key && (f->n_kv_heads != 1 || f->v_dim > f->k_dim)) return 0;
  if (held(f)) {
    const HeldRow row(*f);
    return row.codes + row.plain + row.scales;
  }
  return 2ll * f->n_kv_heads * (f->k_dim + (f->values_in_key ? 0 : f->v_dim));
}

inline int check_format(const gpb_row_format *f) {
  if (!f) return GPB_EINVAL;
  const int64_t payload = payload_bytes(f);
  if (payload == 0 || f->row_bytes < payload) return GPB_EINVAL;
  return f->row_bytes % 16 ? GPB_EALIGN : GPB_OK;
}

// Whether results [tokens][heads] of `dim` values have a place each: heads
// within tokens, or tokens within heads.
inline bool apart(int64_t tokens, int64_t heads, int64_t dim, int64_t token_stride,
                  int64_t head_stride) {
  const auto within = [dim](int64_t n, int64_t stride, int64_t others, int64_t outer) {
    return (n <= 1 || stride >= dim) &&
           (others <= 1 || (outer >= dim && (n <= 1 || stride <= (outer - dim) / (n - 1))));
  };
  return within(heads, head_stride, tokens, token_stride) ||
         within(tokens, token_stride, heads, head_stride);
}

}  // namespace gpb
