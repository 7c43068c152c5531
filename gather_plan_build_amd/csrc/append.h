// What the appends of plain and of held rows share: arguments, sines, and the
// rotation of a head's chunks.
#pragma once

#include "row_format.h"

namespace gpb {

constexpr int kMaxPairs = 256;

struct AppendArgs {
  const uint16_t *k, *v, *q;
  uint16_t *q_out;
  uint8_t *pool, *rows;
  const int32_t *locs, *positions;
  const float *inv_freq;
  int64_t k_ts, k_hs, v_ts, v_hs, q_ts, q_hs, qo_ts, qo_hs, positions_stride;
  int64_t n_pool_rows;
  int32_t row_bytes, hkv, hq, kd, vd, has_v;
  int32_t rot_start, pairs, interleaved;
  int32_t axis_end[GPB_MAX_AXES];
  int32_t head_units;   // units of one key or query head
  int32_t pair_units;   // of them, units of two chunks (halves apart)
  int32_t *status;
};

template <typename T>
__device__ __forceinline__ f32x8 widen(u32x4 v) {
  return __builtin_convertvector(__builtin_bit_cast(typename Vec<T>::x8, v), f32x8);
}
template <typename T>
__device__ __forceinline__ u32x4 narrow(f32x8 v) {
  return __builtin_bit_cast(u32x4, __builtin_convertvector(v, typename Vec<T>::x8));
}

// Both past the caches: nothing is touched twice here, and rows that fill whole
// lines need not be fetched first.  44,600 latent rows: 316 us so, 333 with plain
// stores, 328 with plain loads and stores; 4,099 tokens of 36 heads: 14.8, 17.0
// and 14.5, which plain ones win by 2%: one form, the large case's.
__device__ __forceinline__ u32x4 load16(const uint16_t *p) {
  return __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p));
}
__device__ __forceinline__ void store16(uint8_t *p, u32x4 v) {
  __builtin_nontemporal_store(v, reinterpret_cast<u32x4 *>(p));
}

// Cosines and sines of the token's pairs into LDS, for all its heads, behind the next
// barrier; lane `id` of the workgroup begins with pair id.
template <typename T>
__device__ __forceinline__ void find_turns(const AppendArgs &a, int64_t t, int id, T *s_cos,
                                           T *s_sin) {
  for (int i = id; i < a.pairs; i += kBlock) {
    int axis = 0;
#pragma unroll
    for (int x = 0; x < GPB_MAX_AXES - 1; ++x) axis += i >= a.axis_end[x];
    const double pos = a.positions[axis * a.positions_stride + t];
    double turns = pos * (static_cast<double>(a.inv_freq[i]) * 0.15915494309189533577);
    turns -= __builtin_rint(turns);
    if constexpr (__is_same(T, double)) {
      double sn, cs;
      sincospi(2.0 * turns, &sn, &cs);
      s_cos[i] = cs;
      s_sin[i] = sn;
    } else {
      float sn, cs;
      sincospif(static_cast<float>(2.0 * turns), &sn, &cs);
      s_cos[i] = cs;
      s_sin[i] = sn;
    }
  }
}

// Unit j of a key or query head at src: two chunks of pairs whose halves lie
// apart (e1 >= 0), or one chunk (pairs side by side, or not rotated).
template <typename T>
__device__ __forceinline__ void rotate_unit(const AppendArgs &a, const uint16_t *src, int j,
                                            const float *s_cos, const float *s_sin, int *e0_out,
                                            int *e1_out, u32x4 *lo_out, u32x4 *hi_out) {
  int e0, e1 = -1;
  if (j < a.pair_units) {
    e0 = a.rot_start + 8 * j;
    e1 = e0 + a.pairs;
  } else {
    e0 = 8 * (j - a.pair_units);
    if (a.pair_units && e0 >= a.rot_start) e0 += 2 * a.pairs;
  }
  u32x4 lo = load16(src + e0), hi = {};
  if (e1 >= 0) {
    hi = load16(src + e1);
    const f32x8 p = widen<T>(lo), q = widen<T>(hi);
    f32x8 y0, y1;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float cs = s_cos[8 * j + i], sn = s_sin[8 * j + i];
      y0[i] = p[i] * cs - q[i] * sn;
      y1[i] = q[i] * cs + p[i] * sn;
    }
    lo = narrow<T>(y0);
    hi = narrow<T>(y1);
  } else if (a.interleaved && e0 >= a.rot_start && e0 < a.rot_start + 2 * a.pairs) {
    const f32x8 p = widen<T>(lo);
    const int i0 = (e0 - a.rot_start) / 2;
    f32x8 y;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float cs = s_cos[i0 + i], sn = s_sin[i0 + i];
      y[2 * i] = p[2 * i] * cs - p[2 * i + 1] * sn;
      y[2 * i + 1] = p[2 * i + 1] * cs + p[2 * i] * sn;
    }
    lo = narrow<T>(y);
  }
  *e0_out = e0;
  *e1_out = e1;
  *lo_out = lo;
  *hi_out = hi;
}

// append_held.hip
int launch_append_held(const gpb_row_format &f, const AppendArgs &a, int32_t n_rows,
                       hipStream_t stream);

}  // namespace gpb
