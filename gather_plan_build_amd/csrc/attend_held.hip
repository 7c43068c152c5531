// attend_held.hip -- the attention kernels of rows held in 8 bits (gfx950).
//
// The kernels of attend_kernel.h with other ways for a row from HBM to the matrix
// instruction, whose operands stay of 16 bits: a code times its scale is a number
// of the row's type, so nothing is rounded on that way, and results are off by what
// they would be off over the rows read back.
//
// Latent rows and narrow items keep the codes in LDS and turn eight of them into an
// operand when it is read: four conversions, which fit into the 32 clocks of the
// matrix instruction before (35.5 clocks for both).  LDS then holds and gives half
// the bytes, by which the latent kernel of 16-bit rows is bound.  Wide items of
// 64- and 128-wide heads are bound by the vector unit, and their four waves read
// each key: there a wave turns its share of a tile on its way to LDS, once.
//
// A key's scale goes with the conversion, since a lane has one key of an operand.
// A value operand holds eight keys to a lane, so there codes are taken at scale 1.
// bf16: the scale goes to the key's weight, which is rounded as it would be without.
// Only a weight below 2^-18 of the largest, of a scale near 2^-100, comes out below
// the least normal number, 2^-126, and loses places: a result is off by less than
// 2^-109 a key for that.  fp16 has not the exponents: scales of 2^-15 and 2^8 side
// by side would leave the one key's weight nothing.  There the eight codes are
// multiplied by their keys' scales, four vector instructions more, which round
// nothing: the products are those of the rows read back (44,600 queries over latent
// rows: 30.5 ms so, 28.6 with the scales in the weights; 32 single tokens: 39 and 37.5
// us; narrow items the same within 1%).
#include <type_traits>

#include "attend_kernel.h"
#include "held.h"

namespace gpb {
namespace {

// The same load with OFF bytes added to the lane's place.  The instruction adds them
// to the LDS place as well.
template <int OFF>
__device__ __forceinline__ void load_to_lds(const uint8_t *from, lds_u8 *to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off offset:%2"
               :
               : "s"(lds_at(to) - OFF), "v"(from), "n"(OFF)
               : "memory");
}
__device__ __forceinline__ void load4_to_lds(const uint8_t *from, lds_u8 *to) {
  load4_to_lds(reinterpret_cast<const int32_t *>(from), to);
}

// A number of the launch's that loops use, kept in a register: left to itself the
// compiler, short of scalar registers, asks for the argument again in the loop, and
// the wait for it is one for all that LDS owes as well.  What it then has to lay
// aside goes to a vector register's lanes, without a wait.  44,600 queries over
// latent rows: 25.6 ms, 25.8 without.
//
// Not of a pointer that is read or written through: the compiler would forget that
// it is one to global memory, and an access to any memory may be one to LDS, so that
// every wait for LDS becomes one for all of it (26.2 ms against 25.1 with waits that
// count).
template <typename V>
__device__ __forceinline__ void keep(V &x) {
  asm volatile("" : "+s"(x));
}
__device__ __forceinline__ AttendArgs kept(AttendArgs a) {
  keep(a.window);
  keep(a.sinks);
  return a;
}

// What runs beside step I of a product: f(integral_constant I).
template <typename F>
struct Beside {
  F f;
  template <int I>
  __device__ __forceinline__ void issue() const {
    f(std::integral_constant<int, I>());
  }
};
template <typename F>
__device__ __forceinline__ Beside<F> beside(F f) {
  return {f};
}

template <typename T, int DK, int DV, bool IN_KEY, bool NARROW>
struct AttendHeld : Attend<T, DK, DV, IN_KEY, NARROW> {
  typedef Attend<T, DK, DV, IN_KEY, NARROW> Plain;
  typedef typename Plain::State State;
  typedef typename Plain::Source Source;
  typedef typename Plain::Sight Sight;
  typedef typename Plain::NoLoader NoLoader;
  typedef typename Plain::x8 x8;
  using Plain::NT;
  using Plain::R0;
  using Plain::R1;
  using Plain::ROW;
  using Plain::RING;
  using Plain::TILES_LDS;
  using Plain::WAVE_XCHG;
  using Plain::SHIFT;
  using Plain::kRows;
  static constexpr bool kHalf = __is_same(T, _Float16);
  // Behind the plain kernel's LDS, a KiB a wave: scales as they come (two tiles of
  // 256 bytes), and by key, as lay_scale has them.  A latent's tiles leave room.
  static constexpr int SCALES = IN_KEY ? 3 * kWideTile * 640 : Plain::LDS;
  static constexpr int LDS = IN_KEY ? Plain::LDS : Plain::LDS + 4096;

  // Bytes from a held row's start: of a key head, of a value head, of its scales.
  static __device__ __forceinline__ int64_t key_at(const AttendItem &it) {
    return IN_KEY ? 0 : static_cast<int64_t>(it.kv_head) * DK;
  }
  static __device__ __forceinline__ int64_t value_at(const AttendArgs &a, const AttendItem &it) {
    return IN_KEY ? 0
                  : static_cast<int64_t>(a.hkv) * DK + static_cast<int64_t>(it.kv_head) * DV;
  }
  static __device__ __forceinline__ int64_t key_scale_at(const AttendArgs &a,
                                                         const AttendItem &it) {
    return IN_KEY ? DV + 2 * (DK - DV)
                  : static_cast<int64_t>(a.hkv) * (DK + DV) + it.kv_head;
  }
  static __device__ __forceinline__ int64_t value_scale_at(const AttendArgs &a,
                                                           const AttendItem &it) {
    return key_scale_at(a, it) + (IN_KEY ? 0 : a.hkv);
  }

  // The largest scale byte an append makes.  A larger one is taken for it in tiles
  // of codes, so that a weight of 0 meets no infinity.
  static constexpr uint32_t kMostByte = Held<T>::kMost + 127;
  // Whether a code comes out of a tile of codes as infinity or NaN (of fp16 a code
  // beyond 240 does at the largest scale, which no append makes).
  static __device__ __forceinline__ bool odd_code(uint32_t code, uint32_t scale) {
    code &= 127;
    return code == 127 || (kHalf && code > 0x77 && scale >= kMostByte);
  }

  // For `careful`.  A tile is odd where its codes are (tiles of codes), or where the
  // values are that went to LDS.
  struct Values {
    int64_t key_at, val_at, key_scale, val_scale;
    const uint8_t *src;
    bool codes;
    __device__ __forceinline__ Values(const AttendArgs &a, const AttendItem &it,
                                      const uint8_t *src)
        : key_at(AttendHeld::key_at(it)), val_at(value_at(a, it)), key_scale(key_scale_at(a, it)),
          val_scale(value_scale_at(a, it)), src(src), codes(IN_KEY || !it.wide) {}
    static __device__ __forceinline__ T one(uint8_t code, uint8_t scale) {
      return values8<T>(u32x2{code, 0}, scale_of(scale))[0];
    }
    __device__ __forceinline__ float key(int64_t off, int e) const {
      const uint8_t *row = src + off;
      if (IN_KEY && e >= DV)
        return static_cast<float>(reinterpret_cast<const T *>(row + DV)[e - DV]);
      return static_cast<float>(one(row[key_at + e], row[key_scale]));
    }
    __device__ __forceinline__ float value(int64_t off, int e) const {
      return static_cast<float>(one(src[off + val_at + e], src[off + val_scale]));
    }
    __device__ __forceinline__ bool odd(int64_t off, int e) const {
      const uint8_t code = src[off + val_at + e], scale = src[off + val_scale];
      return codes ? odd_code(code, scale)
                   : Plain::not_finite(__builtin_bit_cast(uint16_t, one(code, scale)));
    }
  };

  // ---- tiles of codes

  // A tile of n held rows in LDS: blocks of n times 64 bytes of a row, 64 bytes a
  // key, their four chunks moved by bits 2 and 3 of the row.  Sixteen rows at one
  // chunk, the read of a key operand, then meet in no bank, nor do the rows 0 to 3
  // and 8 to 11 (or the next four) at two chunks, that of a value operand.  Four
  // lanes load a row, 64 bytes at a time, so all loads of a lane are of one row (or
  // two), at constant offsets.
  static constexpr int BLOCKS = IN_KEY ? (DV + 2 * (DK - DV)) / 64 : (DK + DV) / 64;
  static constexpr int KEY_BLOCKS = IN_KEY ? BLOCKS : DK / 64;
  static constexpr int VALUES_FROM = IN_KEY ? 0 : DK / 64;  // block of the first value
  static constexpr int CODE_STEPS = (IN_KEY ? DV : DK) / 32;  // chunks of codes to a lane
  static constexpr int KEY_STEPS = KEY_BLOCKS * 2;            // all its chunks of a key

  // Where in a tile the lane reads: key chunk 2 D + half of row lane % 32, even and
  // odd D; value tile t, even and odd t.
  struct Spots {
    uint32_t k[2], v[2];
    __device__ __forceinline__ Spots(int lane) {
      const int n = lane & 31, half = lane >> 5, pair = (lane & 15) >> 1;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        k[x] = n * 64 + ((2 * x + half) ^ ((n >> 2) & 3)) * 16;
        // of 16 lanes, two read eight bytes each of one key; lane i gets value i
        const int row = 4 * half + (pair & 3) + 8 * (pair >> 2);
        v[x] = row * 64 + ((2 * x + ((lane >> 4) & 1)) ^ ((row >> 2) & 3)) * 16 + (lane & 1) * 8;
      }
    }
  };

  template <int TILE>
  static __device__ __forceinline__ u32x4 key_chunk(const lds_u8 *tile, int row0, const Spots &w,
                                                    int D) {
    typedef __attribute__((address_space(3))) u32x4 lds16;
    return *(const lds16 *)(tile + row0 * 64 + w.k[D & 1] + D / 2 * TILE * 64);
  }
  template <int TILE>
  static __device__ __forceinline__ u32x2 value_codes(const lds_u8 *tile, const Spots &w, int key0,
                                                      int t) {
    typedef int v2i __attribute__((ext_vector_type(2)));
    typedef __attribute__((address_space(3))) v2i lds8;
    return __builtin_bit_cast(
        u32x2, __builtin_amdgcn_ds_read_tr8_b64_v2i32(
                   (lds8 *)(tile + w.v[t & 1] + (VALUES_FROM + t / 2) * TILE * 64 + key0 * 64)));
  }
  // Operand E of a lane's chunk D: eight codes of it, or eight values of 16 bits.
  template <int D, int E>
  static __device__ __forceinline__ x8 operand(u32x4 chunk, float scale) {
    if constexpr (D >= CODE_STEPS) return __builtin_bit_cast(x8, chunk);
    else return values8<T>(u32x2{chunk[2 * E], chunk[2 * E + 1]}, scale);
  }
  // The query operand that meets it (see load_queries): steps are two to a chunk of
  // codes and one to a chunk of values.
  static constexpr int step_of(int D) { return D < CODE_STEPS ? 2 * D : D + CODE_STEPS; }

  // The first chunks of a product's keys.
  template <int TILE>
  struct KeyAhead {
    static constexpr int N = KEY_STEPS < 4 ? KEY_STEPS : 4;
    u32x4 raw[N];
    __device__ __forceinline__ void read(const lds_u8 *tile, int row0, const Spots &w) {
#pragma unroll
      for (int d = 0; d < N; ++d) raw[d] = key_chunk<TILE>(tile, row0, w, d);
    }
  };
  // q.k of the 32 keys in rows row0 .. of a tile, whose first chunks are in `ahead`, and
  // the lane's query row.  Conversions and reads stand behind the product they run
  // beside.
  template <int TILE, typename L>
  static __device__ __forceinline__ void products(const x8 *q, const lds_u8 *tile, int row0,
                                                  const Spots &w, float scale,
                                                  KeyAhead<TILE> &ahead, const L &next,
                                                  f32x16 *s) {
    *s = f32x16{};
    x8 k[2];
    k[0] = operand<0, 0>(ahead.raw[0], scale);
    k[1] = operand<0, 1>(ahead.raw[0], scale);
    product_steps<TILE, 0>(q, tile, row0, w, scale, ahead.raw, k, next, s);
  }
  template <int TILE, int D, typename L>
  static __device__ __forceinline__ void product_steps(const x8 *q, const lds_u8 *tile, int row0,
                                                       const Spots &w, float scale, u32x4 *raw,
                                                       x8 *k, const L &next, f32x16 *s) {
    constexpr int AHEAD = KeyAhead<TILE>::N;
    if constexpr (D < KEY_STEPS) {
      constexpr bool MORE = D + 1 < KEY_STEPS;
      *s = mma<T>(k[0], q[step_of(D)], *s);
      in_order();
      if constexpr (MORE) k[0] = operand<D + 1, 0>(raw[(D + 1) % AHEAD], scale);
      next.template issue<D>();
      in_order();
      if constexpr (D < CODE_STEPS) {
        *s = mma<T>(k[1], q[step_of(D) + 1], *s);
        in_order();
      }
      if constexpr (MORE && D + 1 < CODE_STEPS) k[1] = operand<D + 1, 1>(raw[(D + 1) % AHEAD], scale);
      if constexpr (D + AHEAD < KEY_STEPS) raw[D % AHEAD] = key_chunk<TILE>(tile, row0, w, D + AHEAD);
      in_order();
      product_steps<TILE, D + 1>(q, tile, row0, w, scale, raw, k, next, s);
    }
  }

  // Value operand of eight codes; fp16: times their keys' scales.
  static __device__ __forceinline__ x8 value_operand(u32x2 codes, const x8 &by) {
    const x8 x = values8<T>(codes, 1.0f);
    if constexpr (kHalf) return x * by;
    else return x;
  }

  // Sums of N output tiles (values 32 t0 ..) += weights p of 16 NP keys, from row0 on,
  // fp16: with their scales `by`: the first codes, then steps FROM .. TO, with each of
  // which one of the loads of `next` goes out.
  template <int TILE, int NP, int N>
  struct ValueAhead {
    static constexpr int AHEAD = NP * N < 6 ? NP * N : 6;
    u32x2 raw[AHEAD];
    __device__ __forceinline__ void read(const lds_u8 *tile, int row0, const Spots &w, int t0) {
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) raw[i] = codes(tile, row0, w, t0, i);
    }
    static __device__ __forceinline__ u32x2 codes(const lds_u8 *tile, int row0, const Spots &w,
                                                  int t0, int i) {
      return value_codes<TILE>(tile + t0 / 2 * TILE * 64 + row0 * 64, w, i / N * 16, i % N);
    }
    template <int FROM, int TO, typename L>
    __device__ __forceinline__ void add(const x8 *p, const x8 *by, const lds_u8 *tile,
                                        int row0, const Spots &w, int t0, State *st,
                                        const L &next) {
      steps<FROM, TO>(p, by, tile, row0, w, t0, st, next,
                      value_operand(raw[FROM % AHEAD], by[FROM / N]));
    }
    template <int I, int TO, typename L>
    __device__ __forceinline__ void steps(const x8 *p, const x8 *by, const lds_u8 *tile,
                                          int row0, const Spots &w, int t0, State *st,
                                          const L &next, x8 now) {
      if constexpr (I < TO) {
        st->o[I % N] = mma<T>(now, p[I / N], st->o[I % N]);
        in_order();
        if constexpr (I + 1 < TO) now = value_operand(raw[(I + 1) % AHEAD], by[(I + 1) / N]);
        if constexpr (I + AHEAD < NP * N) raw[I % AHEAD] = codes(tile, row0, w, t0, I + AHEAD);
        next.template issue<I>();
        in_order();
        steps<I + 1, TO>(p, by, tile, row0, w, t0, st, next, now);
      }
    }
  };

  // Whether these lanes' share of a tile's value codes holds an odd one (see odd_code);
  // scale(r) is the scale byte of row r's values.
  template <int TILE, typename S>
  static __device__ __forceinline__ bool odd_codes(const lds_u8 *tile, int id, int ids,
                                                   const S &scale) {
    typedef __attribute__((address_space(3))) u32x4 lds16;
    const lds_u8 *v = tile + VALUES_FROM * TILE * 64;
    bool odd = false;
    for (int c = id; c < TILE * DV / 16; c += ids) {
      const u32x4 x = *(const lds16 *)(v + c * 16);
      const uint32_t by = kHalf ? scale(c / 4 % TILE) : 0;
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) odd |= odd_code(x[j] >> 8 * i, by);
    }
    return odd;
  }

  // Scales of the values of a lane's 16 keys of 32: bf16, as its weights take them,
  // fp16, as its value operands do.
  struct ValueScales {
    f32x16 a;
    x8 by[2];
  };
  // The lane has the scale byte of key `lane`'s values, of 32 keys in bf16 and up to 64 in
  // fp16; `room` is 128 bytes of LDS.
  static __device__ __forceinline__ void lay_scale(lds_u8 *room, int lane, uint32_t byte) {
    typedef __attribute__((address_space(3))) float lds_float;
    typedef __attribute__((address_space(3))) T lds_value;
    if (!kHalf && lane >= 32) return;
    const float x = __builtin_amdgcn_ldexpf(1.0f, static_cast<int>(min(byte, kMostByte)) - 127);
    if constexpr (kHalf) ((lds_value *)room)[lane] = static_cast<T>(x);
    else ((lds_float *)room)[lane] = x;
  }
  // Of the 32 keys from key0 on.
  static __device__ __forceinline__ void take_scales(const lds_u8 *room, int key0, int half,
                                                     ValueScales *x) {
    if constexpr (kHalf) {
      typedef typename Vec<T>::x4 x4;
      typedef __attribute__((address_space(3))) x4 lds8;
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const lds_u8 *at = room + (key0 + 16 * b + 4 * half) * 2;
        x->by[b] = __builtin_shufflevector(*(const lds8 *)at, *(const lds8 *)(at + 16), 0, 1, 2, 3,
                                           4, 5, 6, 7);
      }
    } else {
      typedef __attribute__((address_space(3))) f32x4 lds16;
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const f32x4 u = *(const lds16 *)(room + (key0 + 8 * y + 4 * half) * 4);
#pragma unroll
        for (int j = 0; j < 4; ++j) x->a[4 * y + j] = u[j];
      }
    }
  }
  // As Attend::weights, bf16: as operands times their keys' scales.
  static __device__ __forceinline__ float weights(const f32x16 &s, float c, float m,
                                                  const ValueScales &scales, x8 *p) {
    if constexpr (kHalf) {
      return Plain::weights(s, c, m, p);
    } else {
      float sum[4] = {};
      const float ref = Plain::finite_m(m) - SHIFT;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], c, -ref));
        sum[i % 4] += x;
        p[i / 8][i % 8] = static_cast<T>(x * scales.a[i]);
      }
      return (sum[0] + sum[1]) + (sum[2] + sum[3]);
    }
  }

  // The rows of a wave's KEYS keys of tiles of TILE (see Attend::Rows).  Where they
  // are all to be read as they are, and a page has 2^n rows, their places take a few
  // instructions; the loops have no room for more.
  template <int TILE, int KEYS>
  struct Rows : Source {
    const AttendItem &it;
    lds_u8 *ring;
    int first, lane;

    __device__ __forceinline__ Rows(const AttendArgs &a, const AttendItem &it, lds_u8 *lds,
                                    int wave, int lane)
        : Source(a, it), it(it), ring(lds + RING + wave * 1024),
          first(TILE == KEYS ? 0 : wave * KEYS), lane(lane) {
      keep(this->src);
      keep(this->pages);
      keep(this->stride);
      keep(this->page_rows);
      keep(this->page_shift);
      keep(this->n_pages);
    }
    // The first of the wave's keys of tile v.
    __device__ __forceinline__ int key0(int v) const {
      return Plain::first_key(it, v, TILE) + first;
    }
    __device__ __forceinline__ bool easy(int v) const {
      const int k = key0(v), end = k + KEYS - 1;
      return v < it.n_tiles && k >= this->lo && end <= this->last &&
             (k >= this->near || end < this->sunk) && this->page_shift >= 0;
    }
    __device__ __forceinline__ int key(int v, int i) const {
      return v < it.n_tiles ? key0(v) + i : this->lo;
    }
    __device__ __forceinline__ void ask(int v, int slot) const {
      if (!this->pages) return;
      lds_u8 *to = ring + (slot & 3) * 256;
      if (easy(v)) {
        const uint32_t at = static_cast<uint32_t>(key0(v) + lane % KEYS) >> this->page_shift;
        load4_to_lds(this->pages + at, to);
      } else {
        load4_to_lds(this->place(key(v, lane % KEYS)), to);
      }
    }
    // Of key i of the wave's: its page's number, and its place.
    __device__ __forceinline__ uint32_t page(int slot, int i) const {
      typedef __attribute__((address_space(3))) uint32_t lds_u32;
      return this->pages ? ((const lds_u32 *)(ring + (slot & 3) * 256))[i] : 0;
    }
    __device__ __forceinline__ const uint8_t *row(int v, uint32_t page, int i) const {
      uint64_t off;
      if (easy(v) && !__any(page >= this->n_pages && this->pages)) {
        uint32_t r = key0(v) + i;
        if (this->pages)
          r = (page << this->page_shift) | (r & (this->page_rows - 1));
        off = static_cast<uint64_t>(r) * this->stride;
      } else {
        off = this->offset(key(v, i), page);
      }
      return this->src + off;
    }
  };

  // The rows of a wave's 16 keys of wide tiles.  The page numbers and the places of four
  // tiles are found at once, a key to a lane: finding them takes some 70 instructions.
  // 2,723 queries of 128-wide heads, a tile at a time and so: 375 and 351 us; 32
  // requests behind one prefix: 65 and 60 us; 44,600 queries over latent rows: 26.7
  // and 26.2 ms.
  struct FourTiles : Source {
    const AttendItem &it;
    lds_u8 *ring;
    int first, lane;
    uint64_t off;  // of key lane % 16 of tile 4 b + lane / 16

    __device__ __forceinline__ FourTiles(const AttendArgs &a, const AttendItem &it, lds_u8 *lds,
                                         int wave, int lane)
        : Source(a, it), it(it), ring(lds + RING + wave * 1024), first(wave * 16), lane(lane) {
      keep(this->src);
      keep(this->pages);
      keep(this->stride);
      keep(this->page_rows);
      keep(this->page_shift);
      keep(this->n_pages);
    }
    __device__ __forceinline__ int key(int b) const {
      const int v = 4 * b + (lane >> 4);
      return v < it.n_tiles ? Plain::first_key(it, v, kWideTile) + first + (lane & 15) : this->lo;
    }
    __device__ __forceinline__ void ask(int b) const {
      if (this->pages) load4_to_lds(this->place(key(b)), ring);
    }
    __device__ __forceinline__ void find(int b) {
      typedef __attribute__((address_space(3))) uint32_t lds_u32;
      off = this->offset(key(b), this->pages ? ((const lds_u32 *)ring)[lane] : 0);
    }
    // Of key i of tile v, one of the four.
    __device__ __forceinline__ const uint8_t *row(int v, int i) const {
      const int from = (v & 3) * 16 + i;
      const uint32_t lo = __shfl(static_cast<uint32_t>(off), from, 64);
      const uint32_t hi = __shfl(static_cast<uint32_t>(off >> 32), from, 64);
      return this->src + (lo | static_cast<uint64_t>(hi) << 32);
    }
    // Tile v's turn: the row of tile v + 2, and every fourth time the work for the next
    // four.  `asked` comes before the tile's wait for loads, which is before `found`
    // of the next.
    __device__ __forceinline__ void asked(int v) const {
      if ((v & 3) == 0) ask(v / 4 + 1);
    }
    __device__ __forceinline__ const uint8_t *found(int v, int i) {
      const uint8_t *r = row(v + 2, i);
      if ((v & 3) == 1) find(v / 4 + 1);
      return r;
    }
  };

  // ---- narrow items

  // The loads of a wave's tile of 32 keys: rows lane / 4 and 16 + lane / 4, chunk
  // lane % 4 of 64 bytes at a time; and the four bytes around a scale, of key
  // lane % 32, the key's (lanes below 32) or the value's.
  struct NarrowLoader {
    static constexpr int N = 2 * BLOCKS + 1;
    static __device__ __forceinline__ void all(const AttendArgs &a, const AttendItem &it,
                                               const uint8_t *own, lds_u8 *tile,
                                               lds_u8 *scales, int lane) {
      const int64_t scale = lane < 32 ? key_scale_at(a, it) : value_scale_at(a, it);
      gpb::load4_to_lds(own + (scale & ~3ll), scales);
      const uint64_t at = reinterpret_cast<uint64_t>(own);
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const int r = 16 * g + (lane >> 2);
        const uint32_t lo = __shfl(static_cast<uint32_t>(at), r, 64);
        const uint32_t hi = __shfl(static_cast<uint32_t>(at >> 32), r, 64);
        const uint8_t *row = reinterpret_cast<const uint8_t *>(lo | static_cast<uint64_t>(hi) << 32) +
                             ((lane & 3) ^ ((r >> 2) & 3)) * 16;
        blocks<DK / 64>(row + key_at(it), tile + g * 1024);
        blocks<DV / 64>(row + value_at(a, it), tile + DK / 64 * 2048 + g * 1024);
      }
    }
    template <int NB, int J = 0>
    static __device__ __forceinline__ void blocks(const uint8_t *from, lds_u8 *to) {
      if constexpr (J < NB) {
        gpb::load_to_lds<J * 64>(from, to + J * 2048);
        blocks<NB, J + 1>(from, to);
      }
    }
  };

  // As Attend::narrow.  A wave has two tiles' room, so that the loads of the tile
  // after next go out as soon as one has been read.  Page numbers are asked for two
  // tiles before the loads that need them: the wait for the tile between has them.
  template <bool SCAN>
  static __device__ __forceinline__ bool narrow(const AttendArgs &args, const AttendItem &it,
                                                lds_u8 *lds) {
    const AttendArgs a = kept(args);
    const int lane = threadIdx.x & 63, wave = wave_id();
    const int row = lane & 31, half = lane >> 5;
    constexpr int BUF = kNarrowTile * 64 * BLOCKS;
    static_assert(8 * BUF <= TILES_LDS, "two tiles a wave");
    lds_u8 *own = lds + wave * 2 * BUF, *scales = lds + SCALES + wave * 1024;
    const Rows<kNarrowTile, kNarrowTile> rows(a, it, lds, wave, lane);
    if (wave < it.n_tiles) {
      rows.ask(wave, 0);
      rows.ask(wave + 4, 1);
    }
    x8 q[DK / 16];
    int pos;
    load_queries(a, it, row, half, q, &pos);
    const Spots w(lane);
    const Sight see = Plain::sight(a, it, pos);
    State st;
    st.clear();
    bool left = false;  // SCAN: a tile is left to `careful`
    const float c = a.c;
    const auto load = [&](int v, int n) {
      rows.ask(v + 8, n + 2);
      NarrowLoader::all(a, it, rows.row(v, rows.page(n, lane & 31), lane & 31),
                        own + (n & 1) * BUF, scales + (n & 1) * 256, lane);
    };
    if (wave < it.n_tiles) {
      typedef __attribute__((address_space(3))) uint32_t lds_u32;
      loads_done();
      load(wave, 0);
      if (wave + 4 < it.n_tiles) load(wave + 4, 1);
      const int key_shift = static_cast<int>(key_scale_at(a, it) & 3) * 8;
      const int value_shift = static_cast<int>(value_scale_at(a, it) & 3) * 8;
      int n = 0;  // tiles of the wave so far
      lds_reads_done();
      loop_aligned();
      for (int v = wave; v < it.n_tiles; v += 4, ++n) {
        const lds_u8 *now = own + (n & 1) * BUF;
        const int key0 = Plain::first_key(it, v, kNarrowTile);
        const bool whole = Plain::whole_tile(a, it, key0, kNarrowTile);
        if (v + 4 >= it.n_tiles) loads_done();
        else if (rows.pages) loads_done<NarrowLoader::N + 1>();
        else loads_done<NarrowLoader::N>();
        const lds_u8 *sc = scales + (n & 1) * 256;
        const auto value_scale = [&](int r) {
          return ((const lds_u32 *)sc)[32 + r] >> value_shift & 255;
        };
        if (SCAN && !whole && __any(odd_codes<kNarrowTile>(now, lane, 64, value_scale))) {
          left = true;
        } else {
          const uint32_t ks = ((const lds_u32 *)sc)[row] >> key_shift & 255;
          lay_scale(scales + 512, lane, value_scale(row));
          KeyAhead<kNarrowTile> keys;
          keys.read(now, 0, w);
          f32x16 s;
          products<kNarrowTile>(q, now, 0, w, scale_of(ks), keys, NoLoader(), &s);
          ValueAhead<kNarrowTile, 2, NT> values;
          values.read(now, 0, w, 0);
          ValueScales scale;
          take_scales(scales + 512, 0, half, &scale);
          Plain::take_top(
              st, Plain::template masked_top<1>(a, it, &s, key0, whole, see, half), false);
          x8 p[2];
          st.l += weights(s, c, st.m, scale, p);
          values.template add<0, 2 * NT>(p, scale.by, now, 0, w, 0, &st, NoLoader());
        }
        lds_reads_done();
        if (v + 8 < it.n_tiles) load(v + 8, n + 2);
      }
    }
    return Plain::template narrow_end<SCAN, Values>(a, it, lds, wave, lane, st, left);
  }

  // The lane's query row, in the order of its key chunks' codes: of 32 values, the
  // first half of the lanes have the first 16.
  static __device__ __forceinline__ void load_queries(const AttendArgs &a, const AttendItem &it,
                                                      int row, int half, x8 *q, int *pos) {
    const bool has = row < it.n_rows;
    const int g = it.row0 + (has ? row : 0);
    const int t = g / a.G, h = g - t * a.G + it.kv_head * a.G;
    *pos = has ? a.list[a.positions_at + t] : -1;
    const uint16_t *src = a.q + t * a.q_ts + h * a.q_hs + half * 16;
#pragma unroll
    for (int d = 0; d < DK / 16; ++d)
      q[d] = has ? *reinterpret_cast<const x8 *>(src + d / 2 * 32 + d % 2 * 8) : x8{};
    // (arrived before the tiles' loads start, as in Attend::load_queries)
#pragma unroll
    for (int d = 0; d < DK / 16; ++d) asm volatile("" : "+v"(q[d]));
    asm volatile("" : "+v"(*pos));
  }

  // ---- latent rows

  // The loads of a wave's 16 keys of a tile: row lane / 4, chunk lane % 4 of 64 bytes
  // at a time, then the four bytes from its scale on.
  struct LatentLoader {
    static constexpr int N = BLOCKS + 1;
    const uint8_t *row;
    lds_u8 *to, *scales;
    int chunk;
    __device__ __forceinline__ LatentLoader(const uint8_t *row, lds_u8 *tile, lds_u8 *scales,
                                            int wave, int lane)
        : row(row), to(tile + wave * 1024), scales(scales + wave * 256),
          chunk(((lane & 3) ^ ((lane >> 4) & 3)) * 16) {}
    template <int I>
    __device__ __forceinline__ void issue() const {
      if constexpr (I < BLOCKS) gpb::load_to_lds<I * 64>(row + chunk, to + I * kWideTile * 64);
      else if constexpr (I == BLOCKS) gpb::load4_to_lds(row + DV + 2 * (DK - DV), scales);
    }
    template <int I = 0, int END = N>
    __device__ __forceinline__ void all() const {
      if constexpr (I < END) {
        issue<I>();
        all<I + 1, END>();
      }
    }
  };

  // As Attend::latent, over tiles of codes.  Three of them fit, and the weights that
  // pass between the waves of a pair have two places, so that one barrier a tile
  // serves both: behind it the next tile is there, and nobody reads the last one,
  // whose place the loads of the tile after next take.  What a product needs first
  // from LDS is asked for before what comes ahead of the product.
  template <bool SCAN>
  static __device__ __forceinline__ bool latent(const AttendArgs &args, const AttendItem &it,
                                                lds_u8 *lds) {
    const AttendArgs a = kept(args);
    const int lane = threadIdx.x & 63, wave = wave_id();
    const int part = wave & 1, half = lane >> 5;
    const int row = (wave >> 1) * 32 + (lane & 31);
    FourTiles rows(a, it, lds, wave, lane);
    const bool idle = (wave >> 1) * 32 >= it.n_rows;  // a pair without rows only loads
    constexpr int BUF = kWideTile * 64 * BLOCKS, BY_KEY = SCALES + 3 * 1024, XCHG = BY_KEY + 1024;
    static_assert(3 * BUF == SCALES && XCHG + 8 * WAVE_XCHG <= TILES_LDS, "room");
    constexpr int EARLY = 5;  // loads of a tile that go out before its turn begins
    lds_u8 *by_key = lds + BY_KEY + wave * 256;
    typedef __attribute__((address_space(3))) x8 lds8;
    typedef __attribute__((address_space(3))) float lds_float;
    typedef __attribute__((address_space(3))) uint32_t lds_u32;
    x8 q[DK / 16] = {};
    const Spots w(lane);
    const Sight see = Plain::sight(a, it, Plain::position(a, it, row));
    State st;
    st.clear();
    bool left = false;  // SCAN: a tile is left to `careful`
    const float c = a.c;
    const auto loader = [&](const uint8_t *row, int buf) {
      return LatentLoader(row, lds + buf * BUF, lds + SCALES + buf * 1024, wave, lane);
    };
    if (it.n_tiles > 0) {
      typedef typename Plain::template Loader<kWideTile, 4> Queries;
      rows.ask(0);
      {
        // the queries come as a tile of 16-bit rows, behind the first tile
        const int g = it.row0 + min(wave * 16 + (lane & 15), it.n_rows - 1);
        const int t = g / a.G, h = g - t * a.G + it.kv_head * a.G;
        Queries(reinterpret_cast<const uint8_t *>(a.q),
                static_cast<uint64_t>(t * a.q_ts + h * a.q_hs) * 2, lds + BUF, wave, lane)
            .all();
      }
      loads_done<Queries::N>();
      rows.find(0);
      loader(rows.row(0, lane >> 2), 0).all();
      loads_done<LatentLoader::N>();
      __syncthreads();
      const int n = 32 * (wave >> 1) + (lane & 31);
      static_assert(BUF + kWideTile * ROW <= TILES_LDS, "room for the queries");
#pragma unroll
      for (int d = 0; d < DK / 16; ++d) {
        if (d < 2 * CODE_STEPS) {
          const int c = d / 2 * 4 + half * 2 + d % 2;
          q[d] = *(const lds8 *)(lds + BUF + n * R0 + place_of<R0>(n, c) * 16);
        } else {
          const int c = (d - 2 * CODE_STEPS) * 2 + half;
          q[d] = *(const lds8 *)(lds + BUF + kWideTile * R0 + n * R1 + place_of<R1>(n, c) * 16);
        }
        // to the accumulation registers, from which a matrix instruction takes
        // an operand as well: the sums need the others
        asm volatile("" : "+a"(q[d]));
      }
      lds_reads_done();
      loads_done();
      __syncthreads();
      LatentLoader load = loader(rows.row(1, lane >> 2), 1);  // of the tile after this one
      load.template all<0, EARLY>();
      int buf = 0, odd_turn = 0;
      KeyAhead<kWideTile> keys;
      uint32_t scale, laid;  // of the lane's key; of the one that it lays (fp16: of all 64)
      const auto scale_in = [&](int b, int key) {
        return ((const lds_u32 *)(lds + SCALES + b * 1024))[key * 4] & 255;
      };
      const auto begin = [&]() {  // the first reads of the tile in `buf`
        scale = scale_in(buf, 32 * part + (lane & 31));
        laid = kHalf ? scale_in(buf, lane) : scale;
        keys.read(lds + buf * BUF, 32 * part, w);
      };
      begin();
      lds_reads_done();
      loop_aligned();
      for (int v = 0; v < it.n_tiles; ++v) {
        const lds_u8 *now = lds + buf * BUF;
        lds_u8 *mine = lds + XCHG + (odd_turn * 4 + wave) * WAVE_XCHG;
        const lds_u8 *theirs = lds + XCHG + (odd_turn * 4 + (wave ^ 1)) * WAVE_XCHG;
        odd_turn ^= 1;
        const int key0 = Plain::first_key(it, v, kWideTile);
        const int used = buf, after = buf == 0 ? 2 : buf - 1;  // after: of tile v + 2, and v - 1
        buf = buf == 2 ? 0 : buf + 1;
        bool whole, odd = false;
        if constexpr (SCAN) {
          whole = Plain::whole_tile(a, it, key0, kWideTile);
          odd = !whole && __syncthreads_or(odd_codes<kWideTile>(
                              now, threadIdx.x, 256, [&](int r) { return scale_in(used, r); }));
          left |= odd;
        }
        if (odd || idle) {
          whole = Plain::whole_tile(a, it, key0, kWideTile);
          load.template all<EARLY>();
          if (!odd && (v == 0 || !whole)) __syncthreads();
          load = loader(rows.found(v, lane >> 2), after);
          rows.asked(v);
          loads_done();
          __syncthreads();
          load.template all<0, EARLY>();
          begin();
          continue;
        }
        f32x16 s;
        const uint8_t *next_row;
        products<kWideTile>(
            q, now, 32 * part, w, scale_of(scale), keys, beside([&](auto d) {
              constexpr int D = decltype(d)::value;
              if constexpr (D % 2 == 0) load.template issue<EARLY + D / 2>();
              if constexpr (D == 1) lay_scale(by_key, lane, laid);
              if constexpr (D == 5) whole = Plain::whole_tile(a, it, key0, kWideTile);
              if constexpr (D == 13) next_row = rows.found(v, lane >> 2);
              if constexpr (D == 15) rows.asked(v);
            }),
            &s);
        const bool agree = v == 0 || !whole;
        ValueScales mine_by;
        take_scales(by_key, kHalf ? 32 * part : 0, half, &mine_by);
        ValueAhead<kWideTile, 2, NT> first;
        first.read(now, 32 * part, w, part * NT);
        float top =
            Plain::template masked_top<1>(a, it, &s, key0 + 32 * part, whole, see, half);
        if (agree) {
          if (half == 0) ((lds_float *)(mine + 2048 + 128))[lane] = top;
          __syncthreads();
          top = fmaxf(top, ((const lds_float *)(theirs + 2048 + 128))[lane & 31]);
        }
        Plain::take_top(st, top, !agree);
        x8 p[2];
        st.l += weights(s, c, st.m, mine_by, p);
        const float m = st.m;
        ((lds8 *)mine)[lane] = p[0];
        ((lds8 *)mine)[64 + lane] = p[1];
        if (half == 0) ((lds_float *)(mine + 2048))[lane] = m;
        first.template add<0, 2 * NT - 4>(p, mine_by.by, now, 32 * part, w, part * NT, &st,
                                          NoLoader());
        ValueAhead<kWideTile, 2, NT> second;
        second.read(now, 32 * (1 - part), w, part * NT);
        loads_done();
        __syncthreads();
        x8 p2[2];
        p2[0] = ((const lds8 *)theirs)[lane];
        p2[1] = ((const lds8 *)theirs)[64 + lane];
        const float m2 = ((const lds_float *)(theirs + 2048))[lane & 31];
        ValueScales their_by;  // (bf16: in the weights)
        if constexpr (kHalf) take_scales(by_key, 32 * (1 - part), half, &their_by);
        first.template add<2 * NT - 4, 2 * NT>(p, mine_by.by, now, 32 * part, w, part * NT, &st,
                                               NoLoader());
        if (__any(m2 != m)) {
          const float both = fmaxf(m, m2);
          const float f2 = __builtin_amdgcn_exp2f(m2 - Plain::finite_m(both));
          Plain::template rescale<NT>(st.o, &st.l,
                                      __builtin_amdgcn_exp2f(m - Plain::finite_m(both)));
          st.m = both;
#pragma unroll
          for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int j = 0; j < 8; ++j)
              p2[b][j] = static_cast<T>(static_cast<float>(p2[b][j]) * f2);
        }
        load = loader(next_row, after);
        second.template add<0, 2 * NT - 4>(
            p2, their_by.by, now, 32 * (1 - part), w, part * NT, &st, beside([&](auto i) {
              constexpr int I = decltype(i)::value;
              if constexpr (I % 2 == 0 && I / 2 < EARLY) load.template issue<I / 2>();
            }));
        begin();
        second.template add<2 * NT - 4, 2 * NT>(p2, their_by.by, now, 32 * (1 - part), w,
                                                part * NT, &st, NoLoader());
      }
      loads_done();
    }
    // each wave has summed the weights of its own keys
    lds_u8 *mine = lds + TILES_LDS + wave * WAVE_XCHG;
    const lds_u8 *theirs = lds + TILES_LDS + (wave ^ 1) * WAVE_XCHG;
    float l = st.l + other_half(st.l, half);
    __syncthreads();
    ((lds_float *)mine)[lane] = l;
    __syncthreads();
    l += ((const lds_float *)theirs)[lane];
    if constexpr (SCAN) {
      if (__syncthreads_or(left)) {
        Plain::lay_down(it, lds, row, half, st, l, part * NT, true);
        Plain::template careful<Values>(a, it, lds);
        return true;
      }
    } else if (__syncthreads_or(row < it.n_rows && Plain::odd_sums(st.o, l))) {
      return false;
    }
    Plain::store(a, it, lds + wave * 128 * NT * 32, (wave >> 1) * 32, lane, st, l, part * NT);
    return true;
  }

  // ---- wide items

  // A wave's share of a tile, 16 keys: its codes come to registers while an earlier
  // tile is worked on, and go to LDS as the values they stand for, to where a tile of
  // 16-bit rows has them.  Four lanes have a row, chunk lane % 4 of 64 bytes at a time,
  // of keys and then of values.  A wave's write of 1 KiB then takes 16 clocks of LDS, and
  // of rows of 256 bytes 32 with row lane / 4 (of 128 bytes 16 as well).  8 would do: lanes
  // next to each other meet in a bank twice, which are the conflicts that the counters of
  // these kernels show.
  struct Share {
    static constexpr int N0 = DK / 64, N = (DK + DV) / 64;
    u32x4 raw[N];
    uint32_t scale[2];
    int i;        // of the wave's 16 rows, the lane's
    uint32_t to;  // in a tile, of the lane's first chunk

    __device__ __forceinline__ Share(int wave, int lane) {
      const int b0 = lane >> 2 & 1, b1 = lane >> 3 & 1, b2 = lane >> 4 & 1, b3 = lane >> 5;
      i = R0 % 256 ? b0 | b1 << 2 | b2 << 1 | b3 << 3 : b0 << 3 | b1 << 1 | b2 | b3 << 2;
      const int row = wave * 16 + i;
      to = row * R0 + place_of<R0>(row, lane % 4 * 2) * 16;
    }
    template <int J>
    __device__ __forceinline__ void ask(const AttendArgs &a, const AttendItem &it,
                                        const uint8_t *row, int lane) {
      // (said to be global memory, which `keep` has made the compiler forget)
      typedef const __attribute__((address_space(1))) u32x4 global16;
      const int64_t at = J < N0 ? key_at(it) + 64 * J : value_at(a, it) + 64 * (J - N0);
      raw[J] = *(global16 *)(row + at + lane % 4 * 16);
    }
    __device__ __forceinline__ void ask_scales(const AttendArgs &a, const AttendItem &it,
                                               const uint8_t *row) {
      typedef const __attribute__((address_space(1))) uint8_t global1;
      scale[0] = *(global1 *)(row + key_scale_at(a, it));
      scale[1] = *(global1 *)(row + value_scale_at(a, it));
    }
    // (place_of is an exclusive or of what row and chunk give)
    template <int J>
    __device__ __forceinline__ void put(lds_u8 *tile) const {
      typedef __attribute__((address_space(3))) x8 lds8;
      constexpr int C = 8 * (J < N0 ? J : J - N0);
      const float f = scale_of(scale[J < N0 ? 0 : 1]);
      lds_u8 *at = tile + (J < N0 ? 0 : kWideTile * R0);
      *(lds8 *)(at + (to ^ place_of<R0>(0, C) * 16)) = values8<T>(u32x2{raw[J][0], raw[J][1]}, f);
      *(lds8 *)(at + (to ^ place_of<R0>(0, C + 1) * 16)) =
          values8<T>(u32x2{raw[J][2], raw[J][3]}, f);
    }
  };

  // As Attend::thirty_two: parts 4 B .. of what runs beside, two with each product.
  template <int B, int RH, typename L>
  static __device__ __forceinline__ void thirty_two(const AttendArgs &a, const AttendItem &it,
                                                    const x8 *q, const lds_u8 *now,
                                                    const typename Plain::Places &w, int key0,
                                                    bool whole, const Sight *see, State *st,
                                                    int half, const L &parts) {
    f32x16 s[RH];
    Plain::template products<kWideTile, 4 * B, 2, RH>(q, now, 32 * B, w, parts, s);
    x8 p[2 * RH];
#pragma unroll
    for (int r = 0; r < RH; ++r)
      Plain::template weigh<1>(a, it, s + r, key0 + 32 * B, whole, see[r], st[r], half, p + 2 * r);
    Plain::template add_values<2, NT, 4 * B + 2, RH>(p, now + kWideTile * R0 + 32 * B * R1, w, 0, st,
                                                     parts);
  }

  // As Attend::wide.
  template <bool SCAN>
  static __device__ __forceinline__ bool wide(const AttendArgs &args, const AttendItem &it,
                                              lds_u8 *lds) {
    const AttendArgs a = kept(args);
    constexpr int RH = kRows / 128, BUF = kWideTile * ROW;
    const int lane = threadIdx.x & 63, wave = wave_id();
    const int row = wave * 32 * RH + (lane & 31), half = lane >> 5;
    const bool idle = wave * 32 * RH >= it.n_rows;  // a wave without rows only loads
    FourTiles rows(a, it, lds, wave, lane);
    if (it.n_tiles > 0) rows.ask(0);
    x8 q[RH * (DK / 16)];
    Sight see[RH];
    State st[RH];
#pragma unroll
    for (int r = 0; r < RH; ++r) {
      int pos;
      Plain::load_queries(a, it, row + 32 * r, half, q + r * (DK / 16), &pos);
      see[r] = Plain::sight(a, it, pos);
      st[r].clear();
    }
    typename Plain::Places w;
    Plain::find_places(w, lane);
    bool left = false;  // SCAN: a tile is left to `careful`
    if (it.n_tiles > 0) {
      Share share(wave, lane);
      const uint8_t *row_at;
      lds_u8 *to;
      // What runs beside a tile's products, in eight parts: towards the end the next
      // tile goes to LDS, then the loads of the one after it go out, to arrive while
      // five parts pass.  (17,337 queries of 64-wide heads: 441 us so, 485 with the next
      // tile to LDS first and 585 right before the loads.)  Page numbers asked for
      // behind the rows are looked at a tile later.
      int next_v = 0;
      const auto part = [&](auto i) {
        constexpr int I = decltype(i)::value, M = Share::N / 2;
        if constexpr (I >= 6 - M && I < 6) {
          share.template put<2 * (I - 6 + M)>(to);
          share.template put<2 * (I - 6 + M) + 1>(to);
        }
        if constexpr (I == 6) {
          loads_done();
          row_at = next_v == 0 ? rows.row(1, share.i) : rows.found(next_v - 1, share.i);
          share.ask_scales(a, it, row_at);
          share.template ask<0>(a, it, row_at, lane);
          share.template ask<1>(a, it, row_at, lane);
        }
        if constexpr (I == 7) {
          if constexpr (M > 1) {
            share.template ask<2>(a, it, row_at, lane);
            share.template ask<3>(a, it, row_at, lane);
          }
          rows.asked(next_v - 1);
        }
      };
      const auto all_parts = [&]() {
        part(std::integral_constant<int, 0>());
        part(std::integral_constant<int, 1>());
        part(std::integral_constant<int, 2>());
        part(std::integral_constant<int, 3>());
        part(std::integral_constant<int, 4>());
        part(std::integral_constant<int, 5>());
        part(std::integral_constant<int, 6>());
        part(std::integral_constant<int, 7>());
      };
      loads_done();
      rows.find(0);
      row_at = rows.row(0, share.i);
      share.ask_scales(a, it, row_at);
      share.template ask<0>(a, it, row_at, lane);
      share.template ask<1>(a, it, row_at, lane);
      if constexpr (Share::N > 2) {
        share.template ask<2>(a, it, row_at, lane);
        share.template ask<3>(a, it, row_at, lane);
      }
      to = lds;
      all_parts();
      lds_reads_done();
      loop_aligned();
      for (int v = 0; v < it.n_tiles; ++v) {
        __syncthreads();
        lds_u8 *now = lds + (v & 1) * BUF;
        to = lds + (~v & 1) * BUF;
        next_v = v + 1;
        const int key0 = Plain::first_key(it, v, kWideTile);
        const bool whole = Plain::whole_tile(a, it, key0, kWideTile);
        const bool odd =
            SCAN && !whole &&
            __syncthreads_or(Plain::template odd_values<kWideTile>(now, threadIdx.x, 256));
        left |= odd;
        if (odd || idle) {
          all_parts();
          continue;
        }
        if constexpr (RH == 1) {
          f32x16 s[2];
          Plain::template products<kWideTile, 0, 2>(q, now, 0, w, beside(part), s);
          Plain::template products<kWideTile, DK / 32, 2>(q, now, 32, w, beside(part), s + 1);
          x8 p[4];
          Plain::template weigh<2>(a, it, s, key0, whole, see[0], st[0], half, p);
          Plain::template add_values<4, NT, 0>(p, now + kWideTile * R0, w, 0, st, NoLoader());
        } else {
          // (of 64-wide heads a product has four steps, and a tile four products)
          thirty_two<0, RH>(a, it, q, now, w, key0, whole, see, st, half, beside(part));
          thirty_two<1, RH>(a, it, q, now, w, key0, whole, see, st, half, beside(part));
        }
      }
      loads_done();
    }
    float l[RH];
    bool bad = false;
#pragma unroll
    for (int r = 0; r < RH; ++r) {
      l[r] = st[r].l + other_half(st[r].l, half);
      bad |= row + 32 * r < it.n_rows && Plain::odd_sums(st[r].o, l[r]);
    }
    if constexpr (SCAN) {
      if (__syncthreads_or(left)) {
#pragma unroll
        for (int r = 0; r < RH; ++r)
          Plain::lay_down(it, lds, row + 32 * r, half, st[r], l[r], 0, true);
        Plain::template careful<Values>(a, it, lds);
        return true;
      }
    } else if (__syncthreads_or(bad)) {
      return false;
    }
#pragma unroll
    for (int r = 0; r < RH; ++r)
      Plain::store(a, it, lds + wave * 128 * NT * 32, (wave * RH + r) * 32, lane, st[r], l[r], 0);
    return true;
  }

  template <bool SCAN>
  static __device__ __forceinline__ bool item(const AttendArgs &a, const AttendItem &it,
                                              lds_u8 *lds) {
    if constexpr (IN_KEY) return latent<SCAN>(a, it, lds);
    else if constexpr (NARROW) return narrow<SCAN>(a, it, lds);
    else return it.wide ? wide<SCAN>(a, it, lds) : narrow<SCAN>(a, it, lds);
  }
  // Apart, so that the registers of the common case are allotted without it.
  static __device__ __attribute__((noinline)) void again(AttendArgs a, AttendItem it,
                                                         lds_u8 *lds) {
    item<true>(uniform(a), uniform(it), uniform(lds));
  }
};

}  // namespace

int launch_attend_held(int type, int which, const AttendArgs &a, bool narrow,
                       hipStream_t stream) {
  return type == GPB_BF16 ? launch_format<__bf16, AttendHeld>(which, a, narrow, stream)
                          : launch_format<_Float16, AttendHeld>(which, a, narrow, stream);
}

}  // namespace gpb
