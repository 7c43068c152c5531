// append_held.hip -- cache rows held in 8 bits, made from keys and values
// (gfx950).
//
// A turned key is not rounded to the row's type on its way: the code is the one
// rounding.  A code on the wrong side of a middle is an eighth of its value off, so
// the turns of coded values are computed in 64 bits: of 6,144,000 codes 20 were not
// the nearest in fp32, 12 with sines in 64 bits alone, none so.  Queries and values
// in 16 bits have k_row_append's turns, and so its very bits.  A head's
// values share a scale, the least power of two 2^e with max |x| <= 448 2^e,
// found by an exchange between the lanes that hold them; x 2^-e is exact, and
// the conversion to e4m3 rounds it to nearest, ties to even.
//
// Bound by HBM, as the plain append.  A workgroup takes one token.  A head's
// 16 values go to a lane, so that it stores 16 bytes, and a head to the next
// power of two of lanes within one wave; keys first, then values, each from the
// start of a wave, so that the exchange has all its lanes.  A lane whose pairs'
// other halves are with another lane reads those again, which the caches hold.
// Queries, and a latent's values in 16 bits, go as in the plain append.  44,600
// latent rows to the pool and packed, 16 query heads: 1.75 GB in 298 us, 5.9 TB/s;
// 4,099 tokens of 28 + 4 + 4 heads of 64: 15.3 us, 2.3 TB/s (14.0 with turns in fp32);
// eight tokens: 5.7 us on the GPU (4.9).
#include "append.h"
#include "held.h"

namespace gpb {
namespace {

struct HeldArgs {
  int32_t k_codes;          // values of a key head that are held in codes
  int32_t k_lanes, v_lanes; // lanes of a head, log2
  int32_t k_end, v_end;     // lanes of all key heads, and of value heads behind them
  int32_t rest_units;       // chunks of eight values of the row's type
  int32_t plain_at, scales_at;  // bytes from a row's start
};

// x in fp32, for a rounding to fewer bits that is to come out as if from x: where fp32
// does not have x, of its two neighbours the one whose last bit is 1.
__device__ __forceinline__ float odd(double x) {
  const float f = static_cast<float>(x);
  const double rest = x - static_cast<double>(f);
  const uint32_t bits = __builtin_bit_cast(uint32_t, f);
  if (!(rest > 0.0 || rest < 0.0) || (bits & 1) || f == 0.0f) return f;
  return __builtin_bit_cast(float, (rest > 0.0) == (f > 0.0f) ? bits + 1 : bits - 1);
}
__device__ __forceinline__ float odd(float x) { return x; }

// Eight values at e of a key head, turned in A.
template <typename T, typename A>
__device__ __forceinline__ f32x8 turned8(const AppendArgs &a, const uint16_t *src, int e,
                                         const A *s_cos, const A *s_sin) {
  const u32x4 own = *reinterpret_cast<const u32x4 *>(src + e);
  f32x8 x = widen<T>(own);
  const int at = e - a.rot_start;
  if (at < 0 || at >= 2 * a.pairs) return x;
  if (a.interleaved) {
    f32x8 y;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const A cs = s_cos[at / 2 + i], sn = s_sin[at / 2 + i];
      y[2 * i] = odd(x[2 * i] * cs - x[2 * i + 1] * sn);
      y[2 * i + 1] = odd(x[2 * i + 1] * cs + x[2 * i] * sn);
    }
    return y;
  }
  const bool first = at < a.pairs;
  const int pair = first ? at : at - a.pairs;
  const f32x8 other =
      widen<T>(*reinterpret_cast<const u32x4 *>(src + (first ? e + a.pairs : e - a.pairs)));
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const A cs = s_cos[pair + i], sn = s_sin[pair + i];
    x[i] = odd(first ? x[i] * cs - other[i] * sn : x[i] * cs + other[i] * sn);
  }
  return x;
}

template <typename T>
__global__ __launch_bounds__(kBlock) void k_row_append_held(AppendArgs a, HeldArgs h) {
  __shared__ __attribute__((aligned(16))) float s_cos[kMaxPairs], s_sin[kMaxPairs];
  __shared__ __attribute__((aligned(16))) double c_cos[kMaxPairs], c_sin[kMaxPairs];
  const int64_t t = blockIdx.x;
  find_turns<float>(a, t, threadIdx.x, s_cos, s_sin);
  if (a.rot_start < h.k_codes)  // (beside them, by other waves if there are few pairs)
    find_turns<double>(a, t, (threadIdx.x + kBlock / 2) % kBlock, c_cos, c_sin);
  __syncthreads();
  const int64_t loc = a.locs ? a.locs[t] : -1;
  const bool stored = loc >= 0 && loc < a.n_pool_rows;
  if (a.locs && !stored && loc != -1 && threadIdx.x == 0 && a.status)
    atomicOr(a.status, GPB_STATUS_BAD_STAGING_ROW);
  uint8_t *to_pool = stored ? a.pool + loc * a.row_bytes : nullptr;
  uint8_t *to_rows = a.rows ? a.rows + t * a.row_bytes : nullptr;

  const int total = h.v_end + h.rest_units + a.hq * a.head_units;
  for (int u = threadIdx.x; u < total; u += kBlock) {
    if (u < h.v_end) {  // 16 values of a head to codes (whole waves come here)
      const bool key = u < h.k_end;
      const int x = key ? u : u - h.k_end, shift = key ? h.k_lanes : h.v_lanes;
      const int head = x >> shift, e = (x & ((1 << shift) - 1)) * 16;
      const int dim = key ? h.k_codes : a.vd;
      const bool one = head < a.hkv && e < dim, two = head < a.hkv && e + 8 < dim;
      f32x8 lo = {}, hi = {};
      if (key) {
        const uint16_t *src = a.k + t * a.k_ts + head * a.k_hs;
        if (one) lo = turned8<T>(a, src, e, c_cos, c_sin);
        if (two) hi = turned8<T>(a, src, e + 8, c_cos, c_sin);
      } else {
        const uint16_t *src = a.v + t * a.v_ts + head * a.v_hs;
        if (one) lo = widen<T>(load16(src + e));
        if (two) hi = widen<T>(load16(src + e + 8));
      }
      float top = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        lo[i] = within<T>(lo[i]);
        hi[i] = within<T>(hi[i]);
        top = __builtin_fmaxf(top, __builtin_fmaxf(__builtin_fabsf(lo[i]), __builtin_fabsf(hi[i])));
      }
      for (int d = 1; d < 1 << shift; d <<= 1) top = __builtin_fmaxf(top, __shfl_xor(top, d, 64));
      const int exponent = scale_exponent<T>(top);
      const float up = power_of_two(-exponent);
      u32x4 codes;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        codes[i] = codes4(lo[4 * i] * up, lo[4 * i + 1] * up, lo[4 * i + 2] * up, lo[4 * i + 3] * up);
        codes[2 + i] = codes4(hi[4 * i] * up, hi[4 * i + 1] * up, hi[4 * i + 2] * up, hi[4 * i + 3] * up);
      }
      const int64_t off = key ? static_cast<int64_t>(head) * h.k_codes + e
                              : static_cast<int64_t>(a.hkv) * a.kd + static_cast<int64_t>(head) * a.vd + e;
      const int64_t scale = h.scales_at + (key ? 0 : a.hkv) + head;
      const uint8_t byte = static_cast<uint8_t>(exponent + 127);
      for (int to = 0; to < 2; ++to) {
        uint8_t *row = to ? to_rows : to_pool;
        if (!row || !one) continue;
        typedef u32x4 Loose4 __attribute__((aligned(8)));  // heads of 8 (2 n + 1) values
        typedef u32x2 Loose2 __attribute__((aligned(8)));
        if (two) *reinterpret_cast<Loose4 *>(row + off) = codes;
        else *reinterpret_cast<Loose2 *>(row + off) = u32x2{codes[0], codes[1]};
        if (e == 0) row[scale] = byte;
      }
      continue;
    }
    const int x = u - h.v_end;
    if (x < h.rest_units) {  // the key's values behind the value
      const int e = a.vd + 8 * x;
      const u32x4 val = narrow<T>(turned8<T>(a, a.k + t * a.k_ts, e, s_cos, s_sin));
      typedef u32x4 Loose4 __attribute__((aligned(8)));
      if (to_pool) *reinterpret_cast<Loose4 *>(to_pool + h.plain_at + 16 * x) = val;
      if (to_rows) *reinterpret_cast<Loose4 *>(to_rows + h.plain_at + 16 * x) = val;
      continue;
    }
    const int y = x - h.rest_units;
    const int head = y / a.head_units, j = y - head * a.head_units;
    int e0, e1;
    u32x4 lo, hi;
    rotate_unit<T>(a, a.q + t * a.q_ts + head * a.q_hs, j, s_cos, s_sin, &e0, &e1, &lo, &hi);
    uint8_t *dst = reinterpret_cast<uint8_t *>(a.q_out + t * a.qo_ts + head * a.qo_hs);
    store16(dst + 2 * e0, lo);
    if (e1 >= 0) store16(dst + 2 * e1, hi);
  }
}

// Lanes for the 16s of `dim` values (at most 1024), as a power of two.
int lanes_log2(int dim) {
  int n = 0;
  while ((16 << n) < dim) ++n;
  return n;
}

}  // namespace

int launch_append_held(const gpb_row_format &f, const AppendArgs &a, int32_t n_rows,
                       hipStream_t stream) {
  const HeldRow row(f);
  HeldArgs h = {};
  h.k_codes = f.values_in_key ? f.v_dim : f.k_dim;
  h.k_lanes = lanes_log2(h.k_codes);
  h.v_lanes = lanes_log2(f.v_dim);
  const auto waves = [&](int lanes) { return static_cast<int32_t>(ceil_div64(f.n_kv_heads << lanes, 64) * 64); };
  h.k_end = waves(h.k_lanes);
  h.v_end = h.k_end + (a.has_v ? waves(h.v_lanes) : 0);
  h.rest_units = static_cast<int32_t>(row.plain / 16);
  h.plain_at = static_cast<int32_t>(row.codes);
  h.scales_at = static_cast<int32_t>(row.codes + row.plain);
  const dim3 grid(static_cast<uint32_t>(n_rows));
  return type_of(&f) == GPB_BF16
             ? launch(k_row_append_held<__bf16>, grid, dim3(kBlock), stream, a, h)
             : launch(k_row_append_held<_Float16>, grid, dim3(kBlock), stream, a, h);
}

}  // namespace gpb
