// attend.hip -- attention over composed or paged rows (gfx950).
//
// For a query q at position p and the keys k_x, values v_x it sees:
// s_x = scale q.k_x, out = sum exp(s_x) v_x / sum exp(s_x), and
// lse = log sum exp(s_x).  One pass over the keys with a running maximum m
// and sum l (the sums of earlier keys are multiplied by 2^(m_old - m_new) when
// m grows), scores in units of log2 so that exp is one v_exp_f32.
//
// Both products run on the 32x32x16 matrix instruction, transposed: the
// scores as K Q^T, so a lane holds 16 keys' scores of one query row and the
// row's maximum and sum need one exchange, with lane + 32; and the output as
// V^T P^T, whose right operand then is what the lane holds already, and whose
// rescaling is by a number of the lane's own.  The product over keys does not
// mind their order, so V^T is read in the order the scores came out in:
// operand element j of lane half h is key 8 (j / 4) + 4 h + j % 4 of 16, two
// transposing LDS reads (ds_read_b64_tr_b16) of four keys each.
//
// Keys and values go to LDS by direct loads, 16 bytes a lane, a row's 16-byte
// chunks permuted within the row so that reads do not meet in a bank: the
// direct load fixes the LDS place of a lane, so the lane picks its source.  A
// wait then is for LDS alone, and the next tile's loads go out one by one
// between the matrix instructions of this one.
//
// Three kernels, by what bounds them (each beside its function): `wide`, many
// query rows over one tile, by the matrix and vector units; `narrow`, few rows
// (decoding), by the latency of rows from HBM; `latent`, whose 512-value sums
// fill the registers of a CU, by LDS reads and matrix instructions in turn.
// Long ranges of keys are cut into parts, joined by their log-sums in a second
// launch in the order of the work list.
//
// Scores, m, l and the sums are fp32.  P is rounded to the row's type for the
// second product, once, because the matrix instruction's operands have one type;
// l sums the unrounded weights.  Results are then off by 2.3e-3 of their norm in
// bf16 and 2.9e-4 in fp16 (normal keys and values), where their own rounding
// alone makes 1.7e-3 and 2.1e-4: the rest would take a second operand for what P
// loses, and with it twice the second product's instructions.
#include <algorithm>
#include <cmath>

#include "attend.h"

namespace gpb {
namespace {

typedef __attribute__((address_space(3))) uint8_t lds_u8;
typedef short s16x4 __attribute__((ext_vector_type(4)));

// The same in every lane: arguments of a function that is not inlined arrive in
// vector registers.
template <typename V>
__device__ __forceinline__ V uniform(V v) {
  struct Words {
    int w[sizeof(V) / 4];
  };
  Words x = __builtin_bit_cast(Words, v);
#pragma unroll
  for (unsigned i = 0; i < sizeof(V) / 4; ++i) x.w[i] = __builtin_amdgcn_readfirstlane(x.w[i]);
  return __builtin_bit_cast(V, x);
}

template <typename T>
__device__ __forceinline__ f32x16 mma(typename Vec<T>::x8 a, typename Vec<T>::x8 b, f32x16 c);
template <>
__device__ __forceinline__ f32x16 mma<__bf16>(Vec<__bf16>::x8 a, Vec<__bf16>::x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
template <>
__device__ __forceinline__ f32x16 mma<_Float16>(Vec<_Float16>::x8 a, Vec<_Float16>::x8 b,
                                                f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

// The value of lane ^ 32.
__device__ __forceinline__ float other_half(float x, int half) {
  const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(unsigned, x),
                                                  __builtin_bit_cast(unsigned, x), false, false);
  return __builtin_bit_cast(float, half ? r[0] : r[1]);
}

__device__ __forceinline__ int wave_id() {
  return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);  // the same in every lane
}

// Direct loads of 16 bytes a lane into 1 KiB of LDS.  Written out because the
// compiler, which cannot tell the two buffers of a tile apart, lets every LDS
// read wait for all such loads; `loads_done` waits for them where the tile is
// needed.  The loads have no register to write, so nothing of the compiler's can
// be overtaken, and are memory to it, so LDS reads stay on their side of each.
// m0 is not named among what they write: the compiler keeps nothing of its own
// there (a register it has reserved, and refuses in that list), it sets it right
// before an instruction that needs it.  No other instruction here does, which
// tests/test_rows_code.py looks for in the machine code.
__device__ __forceinline__ uint32_t lds_at(lds_u8 *p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p));
}
__device__ __forceinline__ void load_to_lds(const uint8_t *from, lds_u8 *to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
               :
               : "s"(lds_at(to)), "v"(from)
               : "memory");
}
// Four bytes a lane, 256 bytes in all.
__device__ __forceinline__ void load4_to_lds(const int32_t *from, lds_u8 *to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off"
               :
               : "s"(lds_at(to)), "v"(from)
               : "memory");
}
// The lane's place is `lane16` ^ X bytes from base + off, which all lanes
// share; the LDS place is `to` + TO.
template <int X, int TO>
__device__ __forceinline__ void load_to_lds(const uint8_t *base, uint64_t off, uint32_t lane16,
                                            lds_u8 *to) {
  uint32_t at;
  const uint64_t b = reinterpret_cast<uint64_t>(base);
  asm volatile("s_add_u32 m0, %1, %7\n\ts_add_u32 s96, %2, %3\n\ts_addc_u32 s97, %4, %5\n\t"
               "v_xor_b32 %0, %8, %6\n\tglobal_load_lds_dwordx4 %0, s[96:97]"
               : "=&v"(at)
               : "s"(lds_at(to)), "s"(static_cast<uint32_t>(b)), "s"(static_cast<uint32_t>(off)),
                 "s"(static_cast<uint32_t>(b >> 32)), "s"(static_cast<uint32_t>(off >> 32)),
                 "v"(lane16), "n"(TO), "n"(X)
               : "s96", "s97", "scc", "memory");
}
// What the wave asked of LDS has arrived (and what it asked of the scalar
// cache: as long as such a load may be under way the compiler cannot tell how
// many LDS reads are, and has each product wait for all of them).  The builtin
// is the s_waitcnt lgkmcnt(0) that the compiler reckons with.
__device__ __forceinline__ void lds_reads_done() {
  __builtin_amdgcn_s_waitcnt(0xc07f);
  asm volatile("" ::: "memory");
}
// All but the newest LEFT of the wave's loads have arrived.
template <int LEFT = 0>
__device__ __forceinline__ void loads_done() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(LEFT) : "memory");
}

// The loop that follows begins on a line of instruction memory.  Measured on the
// same instructions moved by some bytes: 44,600 queries over latent rows, 25.3 ms
// from a line's start and 25.7 from 60 bytes into it.
__device__ __forceinline__ void loop_aligned() { asm volatile(".p2align 6"); }

// Keeps instructions on their side.  The products below read their operands
// some steps ahead, and with this after every step the compiler, which would
// put each read next to its use to save registers, leaves them there.
__device__ __forceinline__ void in_order() { __builtin_amdgcn_sched_barrier(0); }

// A row's 16-byte chunks are moved within groups so that the LDS reads meet in
// no bank: of a key operand, 16 rows at one chunk; of a value operand, 16 lanes
// at a time, four rows at 32 bytes, which have to fall into different 32 bytes
// of 128 (and the next 16 lanes' into the other 128).  Rows of whole 256 bytes
// all start at bank 0: the chunk's bits are turned (`turned`) so that those two
// columns lie 128 bytes apart, and the row's four low bits added.  Rows of 128
// bytes start half way through the banks in turn and take three.  Measured on
// the value reads: 130 and 149 bytes a clock, 89 with the row's bits alone.
template <int ROW_BYTES>
__device__ __forceinline__ constexpr int row_bits(int r) {
  return ROW_BYTES % 256 ? ((r >> 2) & 1) | (((r ^ (r >> 3)) & 1) << 1) | (((r >> 1) & 1) << 2)
                         : ((r & 7) << 1) | ((r >> 3) & 1);
}
template <int ROW_BYTES>
__device__ __forceinline__ constexpr int turned(int c) {
  if (ROW_BYTES % 256) return c;
  return (c & ~15) | (((c >> 1) & 1) << 3) | (((c >> 2) & 3) << 1) | (c & 1);
}
template <int ROW_BYTES>
__device__ __forceinline__ constexpr int turned_back(int c) {
  if (ROW_BYTES % 256) return c;
  return (c & ~15) | (((c >> 1) & 3) << 2) | (((c >> 3) & 1) << 1) | (c & 1);
}
// Place of chunk c of row r, and the chunk in a place.
template <int ROW_BYTES>
__device__ __forceinline__ constexpr int place_of(int r, int c) {
  return turned<ROW_BYTES>(c) ^ row_bits<ROW_BYTES>(r);
}
template <int ROW_BYTES>
__device__ __forceinline__ constexpr int chunk_at(int r, int place) {
  return turned_back<ROW_BYTES>(place ^ row_bits<ROW_BYTES>(r));
}

// NARROW: a kernel of narrow items alone, with the LDS of those.
template <typename T, int DK, int DV, bool IN_KEY, bool NARROW>
struct Attend {
  static constexpr int KB = DK * 2, VB = DV * 2;              // bytes of a key, a value
  // A tile of n keys in LDS: n rows of K0 bytes (a key, or the value part of a
  // latent), then n rows of R1 bytes (a value, or the rest of a latent).
  static constexpr int R0 = IN_KEY ? VB : KB, R1 = IN_KEY ? KB - VB : VB;
  static constexpr int ROW = R0 + R1;                          // LDS bytes per key
  static constexpr int kRows = rows_of(IN_KEY ? 2 : DK / 128, !NARROW);  // of an item, at most
  // the tile in use and the one under way, or in the end a row's sums
  static constexpr int TILES_LDS =
      NARROW ? 4 * kNarrowTile * ROW : std::max(2 * kWideTile * ROW, kRows * DV * 4);
  static constexpr int WAVE_XCHG = 2048 + 2 * 128;             // latent: a wave's weights, m, maxima
  static constexpr int RING = TILES_LDS + (IN_KEY ? 4 * WAVE_XCHG : 8 * kRows);
  static constexpr int LDS = RING + 4096;
  static constexpr int NT = DV / 32 / (IN_KEY ? 2 : 1);        // output tiles of a wave
  // chunks among which a row's are moved, and steps of 16 values they make
  static constexpr int VS = IN_KEY ? R0 : R1;                  // LDS stride of values
  static constexpr int G0 = R0 % 256 ? 8 : 16, G1 = R1 % 256 ? 8 : 16;
  typedef typename Vec<T>::x8 x8;
  typedef typename Vec<T>::x4 x4;
  // P is held times 2^SHIFT, l with it.  fp16: weights down to 2^-31 of the
  // largest keep a value, where fp16 alone ends at 2^-25.  bf16: an m that stays
  // (see take_top) lets weights grow by 2^8; so held they are at most 1, and sums
  // of the largest values do not pass fp32 before the result does.
  static constexpr float SHIFT = __is_same(T, _Float16) ? 6.0f : -8.0f;

  // Where an item's keys are: key x is `offset` bytes from src, found through
  // its page's number (paged).  A base that leads outside the rows, or outside
  // the page list, is reported and all the item's keys read row 0; so is a page
  // outside the pool, and its keys read page 0.
  struct Source : AttendKeys {
    const uint8_t *src;
    const int32_t *pages;  // of the request's first page
    int32_t *status;
    uint32_t stride;
    int page_rows, page_shift;
    uint32_t n_pages;

    __device__ __forceinline__ Source(const AttendArgs &a, const AttendItem &it)
        : AttendKeys(a, it), src(a.rows), pages(nullptr), status(a.status), stride(a.row_bytes),
          page_rows(a.page_rows), page_shift(a.page_shift), n_pages(0) {
      const int64_t base = uniform<int64_t>(a.base ? a.base[it.req] : it.req * a.pages_stride);
      bool ok;
      if (a.pages) {
        ok = base >= 0 && base + page_of(last) < a.n_listed;
        if (ok) pages = a.pages + base;
        n_pages = a.n_pages;
      } else {
        ok = base + lo >= 0 && base + last < a.n_rows;
        if (ok) src += base * a.row_bytes;
      }
      if (!ok) {
        stride = 0;
        if (status && it.n_tiles > 0) atomicOr(status, GPB_STATUS_BAD_DESCRIPTOR);
      }
    }
    __device__ __forceinline__ uint32_t page_of(uint32_t key) const {
      return page_shift >= 0 ? key >> page_shift : key / static_cast<uint32_t>(page_rows);
    }
    __device__ __forceinline__ const int32_t *place(int key) const {
      return pages + page_of(in_range(key));
    }
    __device__ __forceinline__ uint64_t offset(int key, uint32_t page) const {
      uint32_t row = in_range(key);
      if (pages) {
        if (page >= n_pages) {
          page = 0;
          if (status) atomicOr(status, GPB_STATUS_BAD_DESCRIPTOR);
        }
        row = page * page_rows + (row - page_of(row) * page_rows);
      }
      return static_cast<uint64_t>(row) * stride;
    }
    // At once, waiting for the page's number.
    __device__ __forceinline__ uint64_t offset(int key) const {
      return offset(key, pages ? *place(key) : 0);
    }
  };

  static __device__ __forceinline__ int first_key(const AttendItem &it, int v, int tile) {
    return (v < it.n_first ? it.tile0 + v : it.tile1 + v - it.n_first) * tile;
  }

  // The places of a wave's keys of tiles of TILE, of which it loads KEYS.  Page
  // numbers come through LDS as the rows do, some tiles before those are asked
  // for, so that no wait for a page number is a wait for the loads of rows
  // behind it.  A wave has room for four tiles' numbers.
  template <int TILE, int KEYS>
  struct Rows : Source {
    const AttendItem &it;
    lds_u8 *ring;
    int mine;  // the key of a tile whose row the lane finds

    __device__ __forceinline__ Rows(const AttendArgs &a, const AttendItem &it, lds_u8 *lds,
                                    int wave, int lane)
        : Source(a, it), it(it), ring(lds + RING + wave * 1024),
          mine((TILE == KEYS ? 0 : wave * KEYS) + lane % KEYS) {}
    // A tile's loads go out with the products of an earlier one; where no tile
    // follows they all read one row, which costs less than a second form of
    // the products without them.
    __device__ __forceinline__ int key(int v) const {
      return v < it.n_tiles ? first_key(it, v, TILE) + mine : this->lo;
    }
    // For the page numbers of tile v in room `slot`.
    __device__ __forceinline__ void ask(int v, int slot) const {
      if (this->pages) load4_to_lds(this->place(key(v)), ring + (slot & 3) * 256);
    }
    __device__ __forceinline__ uint64_t row(int v, int slot, int lane) const {
      typedef __attribute__((address_space(3))) int lds_int;
      return this->offset(key(v),
                          this->pages ? ((const lds_int *)(ring + (slot & 3) * 256))[lane] : 0);
    }
  };

  // The loads of one tile of TILE keys, WAVES waves sharing them, each TILE /
  // WAVES keys.  Lane r of `off` holds the place of the wave's key r.
  // Instruction i of the wave, of N, goes out by issue<i>: the products of one
  // tile are under way meanwhile.
  template <int TILE, int WAVES>
  struct Loader {
    static constexpr int N0 = TILE * R0 / 1024 / WAVES, N1 = TILE * R1 / 1024 / WAVES;
    static constexpr int N = N0 + N1;
    // Rows of 1 KiB are loaded one at a time, from where a lane says; shorter
    // ones several at a time, a lane taking its chunk of its own row, the same
    // of keys and values.
    static constexpr bool LONG = R0 == 1024;
    static constexpr int C = (LONG ? R1 : R0) / 16, SHORT = LONG ? N1 : N0;
    static_assert(LONG || R0 == R1, "keys and values of one width, or a latent");
    const uint8_t *src[2];  // of the rows of R0 and of R1 bytes
    lds_u8 *to;
    uint64_t off;           // of the lane's row
    uint64_t chunk[SHORT];
    int wave, lane;

    __device__ __forceinline__ Loader(const AttendArgs &a, const AttendItem &it,
                                      const Source &from, uint64_t off, lds_u8 *tile, int wave,
                                      int lane)
        : Loader(from.src + static_cast<int64_t>(it.kv_head) * KB, off, tile, wave, lane) {
      if (!IN_KEY)
        src[1] = from.src + static_cast<int64_t>(a.hkv) * KB +
                 static_cast<int64_t>(it.kv_head) * VB;
    }
    // Latent rows, or queries of their form, at off from `first`.
    __device__ __forceinline__ Loader(const uint8_t *first, uint64_t off, lds_u8 *tile, int wave,
                                      int lane)
        : to(tile), off(off), wave(wave), lane(lane) {
      src[0] = uniform(first);
      src[1] = src[0] + VB;
#pragma unroll
      for (int j = 0; j < SHORT; ++j) {
        const int r = j * (64 / C) + lane / C;  // its low bits are those of its LDS row
        const uint32_t lo = __shfl(static_cast<uint32_t>(off), r, 64);
        const uint32_t hi = __shfl(static_cast<uint32_t>(off >> 32), r, 64);
        chunk[j] = (lo | static_cast<uint64_t>(hi) << 32) + chunk_at<C * 16>(r, lane % C) * 16;
      }
    }
    template <int I>
    __device__ __forceinline__ void issue() const {
      if constexpr (I < N) {
        constexpr int J = I < N0 ? I : I - N0;
        lds_u8 *at = to + (I < N0 ? wave * N0 : TILE * R0 / 1024 + wave * N1) * 1024;
        if constexpr (LONG && I < N0) {  // (16 a wave: a row's swizzle is that of J)
          const uint32_t lo = __builtin_amdgcn_readlane(static_cast<uint32_t>(off), J);
          const uint32_t hi = __builtin_amdgcn_readlane(static_cast<uint32_t>(off >> 32), J);
          load_to_lds<turned_back<R0>(row_bits<R0>(J)) * 16, J * 1024>(
              src[0], lo | static_cast<uint64_t>(hi) << 32, turned_back<R0>(lane) * 16, at);
        } else {
          load_to_lds(src[I < N0 ? 0 : 1] + chunk[J], at + J * 1024);
        }
      }
    }
    template <int I = 0, int END = N>
    __device__ __forceinline__ void all() const {
      if constexpr (I < END) {
        issue<I>();
        all<I + 1, END>();
      }
    }
  };
  // In place of a Loader where no tile follows.
  struct NoLoader {
    template <int I>
    __device__ __forceinline__ void issue() const {}
  };

  struct State {
    f32x16 o[NT];
    float m, l;
    __device__ __forceinline__ void clear() {
#pragma unroll
      for (int t = 0; t < NT; ++t) o[t] = f32x16{};
      m = -INFINITY;
      l = 0.0f;
    }
  };

  // Where in a tile the lane reads its operands.  The swizzle moves a chunk
  // within its group only, so a few places serve every step, the rest being
  // constant offsets.
  struct Places {
    uint32_t k0[G0 / 2], k1[IN_KEY ? G1 / 2 : 1];
    uint32_t v[2][(IN_KEY ? G0 : G1) / 4];
  };
  static constexpr int VG = IN_KEY ? G0 : G1;  // group of a row of values

  static __device__ __forceinline__ void find_places(Places &w, int lane) {
    const int n = lane & 31, half = lane >> 5, i = lane & 15;
#pragma unroll
    for (int d = 0; d < G0 / 2; ++d) w.k0[d] = n * R0 + place_of<R0>(n, 2 * d + half) * 16;
    if constexpr (IN_KEY)
#pragma unroll
      for (int d = 0; d < G1 / 2; ++d) w.k1[d] = n * R1 + place_of<R1>(n, 2 * d + half) * 16;
    // V^T operand of 16 keys and 32 values: lane l gets value l % 32 of keys
    // 4 half .. + 3 and 8 + 4 half .. + 3; of each 16 lanes, lane i reads four
    // values of key i / 4
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int t = 0; t < VG / 4; ++t) {
        const int row = 8 * x + 4 * half + (i >> 2);
        const int chunk = 4 * t + 2 * ((lane >> 4) & 1) + ((i & 3) >> 1);
        w.v[x][t] = row * VS + place_of<VS>(row, chunk) * 16 + (i & 1) * 8;
      }
  }

  static __device__ __forceinline__ x8 value_operand(const lds_u8 *v, const Places &w, int key0,
                                                     int t) {
    typedef __attribute__((address_space(3))) s16x4 lds4;
    const int off = key0 * VS + t / (VG / 4) * VG * 16;
    const s16x4 a0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(v + w.v[0][t % (VG / 4)] + off));
    const s16x4 a1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(v + w.v[1][t % (VG / 4)] + off));
    return __builtin_bit_cast(x8, __builtin_shufflevector(a0, a1, 0, 1, 2, 3, 4, 5, 6, 7));
  }

  // 16 values of the 32 keys in LDS rows row0 .. of a tile of TILE.
  template <int TILE>
  static __device__ __forceinline__ x8 key_operand(const lds_u8 *tile, int row0, const Places &w,
                                                   int d) {
    typedef __attribute__((address_space(3))) x8 lds8;
    constexpr int D0 = R0 / 32;  // steps in the rows of R0 bytes
    if (d < D0)
      return *(const lds8 *)(tile + row0 * R0 + w.k0[d % (G0 / 2)] + d / (G0 / 2) * G0 * 16);
    return *(const lds8 *)(tile + TILE * R0 + row0 * R1 +
                           w.k1[IN_KEY ? (d - D0) % (G1 / 2) : 0] +
                           (d - D0) / (G1 / 2) * G1 * 16);
  }

  // q.k of the 32 keys in LDS rows row0 .. of a tile of TILE and RH query rows
  // of the lane; with every EVERY steps one of the next tile's loads goes out,
  // the first FIRST.
  template <int TILE, int FIRST, int EVERY, int RH = 1, typename L>
  static __device__ __forceinline__ void products(const x8 *q, const lds_u8 *tile, int row0,
                                                  const Places &w, const L &next, f32x16 *s) {
    constexpr int AHEAD = DK / 16 < 6 ? DK / 16 : 6;
    x8 k[AHEAD];
#pragma unroll
    for (int d = 0; d < AHEAD; ++d) k[d] = key_operand<TILE>(tile, row0, w, d);
#pragma unroll
    for (int r = 0; r < RH; ++r) s[r] = f32x16{};
    product_steps<TILE, FIRST, EVERY, RH, 0, AHEAD>(q, tile, row0, w, next, k, s);
  }
  template <int TILE, int FIRST, int EVERY, int RH, int D, int AHEAD, typename L>
  static __device__ __forceinline__ void product_steps(const x8 *q, const lds_u8 *tile, int row0,
                                                       const Places &w, const L &next, x8 *k,
                                                       f32x16 *s) {
    if constexpr (D < DK / 16) {
#pragma unroll
      for (int r = 0; r < RH; ++r) s[r] = mma<T>(k[D % AHEAD], q[r * (DK / 16) + D], s[r]);
      if constexpr (D + AHEAD < DK / 16)
        k[D % AHEAD] = key_operand<TILE>(tile, row0, w, D + AHEAD);
      if constexpr (D % EVERY == EVERY - 1) next.template issue<FIRST + D / EVERY>();
      in_order();
      product_steps<TILE, FIRST, EVERY, RH, D + 1, AHEAD>(q, tile, row0, w, next, k, s);
    }
  }

  // What a row sees of an item's keys: n keys from `from` on and, of a window's
  // first tokens, `sunk` from key_lo on.
  struct Sight {
    int from;
    unsigned n, sunk;
  };
  static __device__ __forceinline__ Sight sight(const AttendArgs &a, const AttendItem &it,
                                                int pos) {
    const int end = min(pos + 1, it.key_hi);  // pos < 2^30
    Sight x;
    x.from = a.window > 0 ? max(it.key_lo, pos + 1 - a.window) : it.key_lo;
    x.n = max(end - x.from, 0);
    x.sunk = a.window > 0 ? max(min(end, a.sinks) - it.key_lo, 0) : 0;
    return x;
  }

  // The keys that the row does not see go to -infinity.
  static __device__ __forceinline__ void mask(const AttendArgs &a, const AttendItem &it,
                                              const Sight &see, int key0, int half, f32x16 &s) {
    const unsigned at = key0 + 4 * half - see.from;
    if (a.window == 0 || key0 >= a.sinks) {
#pragma unroll
      for (int i = 0; i < 16; ++i) s[i] = at + 8 * (i / 4) + i % 4 < see.n ? s[i] : -INFINITY;
    } else {
      const unsigned first = key0 + 4 * half - it.key_lo;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const unsigned x = 8 * (i / 4) + i % 4;
        s[i] = at + x < see.n || first + x < see.sunk ? s[i] : -INFINITY;
      }
    }
  }

  static __device__ __forceinline__ float largest(const f32x16 &s) {
    float top[4];  // four chains: a wave may be alone on its SIMD
#pragma unroll
    for (int i = 0; i < 4; ++i) top[i] = fmaxf(fmaxf(s[i], s[i + 4]), fmaxf(s[i + 8], s[i + 12]));
    return fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
  }

  static __device__ __forceinline__ float finite_m(float m) {
    return m == -INFINITY ? 0.0f : m;  // nothing seen so far: every weight is 0
  }

  // Weights 2^(c s - m) of 32 keys, as two right operands of the second
  // product; returns their sum.
  static __device__ __forceinline__ float weights(const f32x16 &s, float c, float m, x8 *p) {
    float sum[4] = {};
    const float ref = finite_m(m) - SHIFT;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], c, -ref));
      sum[i % 4] += x;
      p[i / 8][i % 8] = static_cast<T>(x);
    }
    return (sum[0] + sum[1]) + (sum[2] + sum[3]);
  }

  // Sums of N output tiles (values 32 t0 ..) of RH rows += weights p of 16 * NP
  // keys (LDS rows 0 .. of v); with every second step one of the next tile's
  // loads from FIRST on goes out.
  template <int NP, int N, int FIRST, int RH = 1, typename L>
  static __device__ __forceinline__ void add_values(const x8 *p, const lds_u8 *v, const Places &w,
                                                    int t0, State *st, const L &next) {
    constexpr int AHEAD = 4;
    const lds_u8 *at = v + t0 / (VG / 4) * VG * 16;
    x8 x[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) x[i] = value_operand(at, w, i / N * 16, i % N);
    value_steps<NP, N, FIRST, RH, 0, AHEAD>(p, at, w, st, next, x);
  }
  template <int NP, int N, int FIRST, int RH, int I, int AHEAD, typename L>
  static __device__ __forceinline__ void value_steps(const x8 *p, const lds_u8 *at,
                                                     const Places &w, State *st, const L &next,
                                                     x8 *x) {
    if constexpr (I < NP * N) {
#pragma unroll
      for (int r = 0; r < RH; ++r)
        st[r].o[I % N] = mma<T>(x[I % AHEAD], p[r * NP + I / N], st[r].o[I % N]);
      if constexpr (I + AHEAD < NP * N)
        x[I % AHEAD] = value_operand(at, w, (I + AHEAD) / N * 16, (I + AHEAD) % N);
      if constexpr (I % 2 == 0) next.template issue<FIRST + I / 2>();
      in_order();
      value_steps<NP, N, FIRST, RH, I + 1, AHEAD>(p, at, w, st, next, x);
    }
  }

  // A key that one row sees and another does not has weight 0 in the other's
  // product, and 0 times infinity or NaN is NaN.  An item whose sums end up
  // with such a value is therefore done again: the tiles that are not whole are
  // looked through, those that hold one are left out of the products, and
  // `careful` adds them at the end, row by row.  These lanes' share (id of
  // ids) of a tile's values:
  template <int TILE>
  static __device__ __forceinline__ bool odd_values(const lds_u8 *tile, int id, int ids) {
    typedef __attribute__((address_space(3))) u32x4 lds16;
    const lds_u8 *v = IN_KEY ? tile : tile + TILE * R0;
    bool odd = false;
    for (int c = id; c < TILE * VS / 16; c += ids) {
      const u32x4 x = *(const lds16 *)(v + c * 16);
#pragma unroll
      for (int j = 0; j < 4; ++j) odd |= not_finite(x[j]) || not_finite(x[j] >> 16);
    }
    return odd;
  }
  static __device__ __forceinline__ bool not_finite(unsigned bits) {
    constexpr unsigned kExp = __is_same(T, _Float16) ? 0x7c00u : 0x7f80u;
    return (bits & kExp) == kExp;
  }

  // Whether a row's sums hold an infinity or NaN.
  static __device__ __forceinline__ bool odd_sums(const f32x16 *o, float l) {
    float x = l * 0.0f;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) x = __builtin_fmaf(o[t][i], 0.0f, x);
    return !(x == 0.0f);
  }

  template <int N>
  static __device__ __forceinline__ void rescale(f32x16 *o, float *l, float f) {
    *l *= f;
#pragma unroll
    for (int t = 0; t < N; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[t][i] *= f;
  }

  // The largest score of 32 * NB keys from their products, the first at position
  // key0, those that the row does not see masked.
  template <int NB>
  static __device__ __forceinline__ float masked_top(const AttendArgs &a, const AttendItem &it,
                                                     f32x16 *s, int key0, bool whole,
                                                     const Sight &see, int half) {
    if (!whole) {
#pragma unroll
      for (int b = 0; b < NB; ++b) mask(a, it, see, key0 + 32 * b, half, s[b]);
    }
    float top = largest(s[0]);
    if constexpr (NB == 2) top = fmaxf(top, largest(s[1]));
    top *= a.c;
    return fmaxf(top, other_half(top, half));
  }
  // The m to weigh by, given the largest score of new keys, and the sums so far
  // brought to it: m stays until it is passed by more than 8, so that the sums are
  // rescaled now and then and not with every new maximum.  Weights then reach 1
  // (fp16: 2^14).  m grows to the new maximum, whose weight then is a power of two
  // (a row of one key has its value exactly), or by whole steps: weights rounded
  // for one m are brought to another by a power of two, which rounds nothing.
  static __device__ __forceinline__ void take_top(State &st, float top, bool by_steps) {
    const bool more = top > st.m + 8.0f;
    if (__any(more)) {
      const float from = finite_m(st.m);
      float m = by_steps ? from + __builtin_ceilf(top - from) : top;
      m = more ? m : st.m;
      rescale<NT>(st.o, &st.l, __builtin_amdgcn_exp2f(st.m - finite_m(m)));
      st.m = m;
    }
  }
  // The weights of the keys, as operands p; the sums so far brought to their m.
  template <int NB>
  static __device__ __forceinline__ void weigh(const AttendArgs &a, const AttendItem &it,
                                               f32x16 *s, int key0, bool whole, const Sight &see,
                                               State &st, int half, x8 *p) {
    take_top(st, masked_top<NB>(a, it, s, key0, whole, see, half), false);
#pragma unroll
    for (int b = 0; b < NB; ++b) st.l += weights(s[b], a.c, st.m, p + 2 * b);
  }

  static __device__ __forceinline__ bool whole_tile(const AttendArgs &a, const AttendItem &it,
                                                    int key0, int n) {
    return key0 >= it.key_lo && key0 + n <= it.key_hi && key0 + n - 1 <= it.pos_min &&
           (a.window == 0 || it.pos_max - key0 < a.window || key0 + n <= a.sinks);
  }

  static __device__ __forceinline__ int position(const AttendArgs &a, const AttendItem &it,
                                                 int row) {
    return row < it.n_rows ? a.list[a.positions_at + (it.row0 + row) / a.G] : -1;
  }

  // The lane's query row: its token, its head, its queries in registers.
  static __device__ __forceinline__ void load_queries(const AttendArgs &a, const AttendItem &it,
                                                      int row, int half, x8 *q, int *pos) {
    const bool has = row < it.n_rows;
    const int g = it.row0 + (has ? row : 0);
    const int t = g / a.G, h = g - t * a.G + it.kv_head * a.G;
    *pos = has ? a.list[a.positions_at + t] : -1;
    const uint16_t *src = a.q + t * a.q_ts + h * a.q_hs + half * 8;
#pragma unroll
    for (int d = 0; d < DK / 16; ++d)
      q[d] = has ? *reinterpret_cast<const x8 *>(src + d * 16) : x8{};
    // arrived before the tiles' loads start: a wait for them later would wait
    // for those too
#pragma unroll
    for (int d = 0; d < DK / 16; ++d) asm volatile("" : "+v"(q[d]));
    asm volatile("" : "+v"(*pos));
  }

  // What turns a row's sums and its m and l into results; a row that sees
  // nothing has l = 0.
  static __device__ __forceinline__ float inverse(float l) { return l == 0.0f ? 0.0f : 1.0f / l; }
  static __device__ __forceinline__ float log_sum(float m, float l) {
    return l == 0.0f ? -INFINITY
                     : (m + __builtin_amdgcn_logf(l) - SHIFT) * 0.69314718055994531f;
  }

  // Results of the row at `g` (token * G + head of the KV head's group).
  static __device__ __forceinline__ int64_t out_place(const AttendArgs &a, const AttendItem &it,
                                                      int g, int64_t *lse_at) {
    const int token = g / a.G, h = g - token * a.G + it.kv_head * a.G;
    *lse_at = static_cast<int64_t>(token) * a.n_heads + h;
    return token * a.o_ts + h * a.o_hs;
  }

  // The sums (or results) of the wave's 32 rows from row0 on, output tiles t0
  // ..; t0 = 0 also their m and l (or log-sums).  They go by way of 32 W * 4
  // bytes of LDS of the wave's own, so that rows are written in whole: a lane
  // holds 16 bytes of every 64 of one row.
  static __device__ __forceinline__ void store(const AttendArgs &a, const AttendItem &it,
                                               lds_u8 *room, int row0, int lane, const State &st,
                                               float l, int t0) {
    if (row0 >= it.n_rows) return;
    constexpr int W = NT * 32;  // values of a row here
    const int n = lane & 31, half = lane >> 5, row = row0 + n;
    typedef __attribute__((address_space(3))) u32x4 lds16;
    if (it.partial >= 0) {
      constexpr int C = W / 4, M = C < 32 ? C - 1 : 31;  // 16-byte chunks, four values
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          f32x4 x;
#pragma unroll
          for (int j = 0; j < 4; ++j) x[j] = st.o[t][4 * y + j];
          *(lds16 *)(room + (n * C + ((8 * t + 2 * y + half) ^ (n & M))) * 16) =
              __builtin_bit_cast(u32x4, x);
        }
      lds_reads_done();
      float *to = a.sums + static_cast<int64_t>(it.partial) * DV + 32 * t0;
#pragma unroll
      for (int i = 0; i < 32 * C / 64; ++i) {
        const int r = i * (64 / C) + lane / C, c = lane % C;
        const u32x4 x = *(const lds16 *)(room + (r * C + (c ^ (r & M))) * 16);
        if (row0 + r < it.n_rows)
          *reinterpret_cast<u32x4 *>(to + static_cast<int64_t>(row0 + r) * DV + c * 4) = x;
      }
      if (half == 0 && t0 == 0 && row < it.n_rows)
        *reinterpret_cast<f32x2 *>(a.ml + 2 * (static_cast<int64_t>(it.partial) + row)) =
            f32x2{st.m, l};
      lds_reads_done();
      return;
    }
    constexpr int C = W / 8, M = C < 32 ? C - 1 : 31;  // chunks of eight values
    const float inv = inverse(l);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        x4 x;
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = static_cast<T>(st.o[t][4 * y + j] * inv);
        typedef __attribute__((address_space(3))) x4 lds8;
        *(lds8 *)(room + (n * C + ((4 * t + y) ^ (n & M))) * 16 + half * 8) = x;
      }
    lds_reads_done();
    int64_t lse_at;
    const uint64_t at = out_place(a, it, it.row0 + min(row, it.n_rows - 1), &lse_at);
    typedef u32x4 Loose __attribute__((aligned(8)));  // out is 8-byte aligned
#pragma unroll
    for (int i = 0; i < 32 * C / 64; ++i) {
      const int r = i * (64 / C) + lane / C, c = lane % C;
      const u32x4 x = *(const lds16 *)(room + (r * C + (c ^ (r & M))) * 16);
      const uint64_t to = __shfl(static_cast<uint32_t>(at), r, 64) |
                          static_cast<uint64_t>(__shfl(static_cast<uint32_t>(at >> 32), r, 64))
                              << 32;
      if (row0 + r < it.n_rows)  // past the caches: 3% of the windowed prefill's time
        __builtin_nontemporal_store(
            x, reinterpret_cast<Loose *>(a.out + static_cast<int64_t>(to) + 32 * t0 + c * 8));
    }
    if (half == 0 && t0 == 0 && a.lse && row < it.n_rows) a.lse[lse_at] = log_sum(st.m, l);
    lds_reads_done();
  }

  // The end of an item whose products left tiles out (see odd_values): the
  // sums so far are laid down in LDS, and a wave takes a row at a time through the left
  // tiles, key by key, only those that the row sees.
  static __device__ __forceinline__ void lay_down(const AttendItem &it, lds_u8 *lds, int row,
                                                  int half, const State &st, float l, int t0,
                                                  bool holds) {
    typedef __attribute__((address_space(3))) float lds_float;
    lds_float *sums = (lds_float *)lds, *ml = (lds_float *)(lds + TILES_LDS);
    if (!holds || row >= it.n_rows) return;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i)
        sums[row * DV + 32 * (t0 + t) + 8 * (i / 4) + 4 * half + i % 4] = st.o[t][i];
    if (half == 0 && t0 == 0) {
      ml[2 * row] = st.m;
      ml[2 * row + 1] = l;
    }
  }
  static __device__ void careful(const AttendArgs &a, const AttendItem &it, lds_u8 *lds) {
    typedef __attribute__((address_space(3))) float lds_float;
    lds_float *sums = (lds_float *)lds, *ml = (lds_float *)(lds + TILES_LDS);
    const int lane = threadIdx.x & 63;
    constexpr int PK = DK / 64, PV = DV / 64;
    __syncthreads();
    const int tile = it.wide ? kWideTile : kNarrowTile;
    const Source from(a, it);
    const T *keys = reinterpret_cast<const T *>(from.src) + static_cast<int64_t>(it.kv_head) * DK;
    const T *vals = IN_KEY ? keys : reinterpret_cast<const T *>(from.src) +
                                        static_cast<int64_t>(a.hkv) * DK +
                                        static_cast<int64_t>(it.kv_head) * DV;
    for (int r = threadIdx.x >> 6; r < it.n_rows; r += 4) {
      const int g = it.row0 + r;
      const int token = g / a.G, h = g - token * a.G + it.kv_head * a.G;
      const Sight see = sight(a, it, a.list[a.positions_at + token]);
      const T *src = reinterpret_cast<const T *>(a.q + token * a.q_ts + h * a.q_hs);
      float q[PK], o[PV], m = ml[2 * r], sum = ml[2 * r + 1];
#pragma unroll
      for (int e = 0; e < PK; ++e) q[e] = static_cast<float>(src[e * 64 + lane]);
#pragma unroll
      for (int e = 0; e < PV; ++e) o[e] = sums[r * DV + e * 64 + lane];
      for (int v = 0; v < it.n_tiles; ++v) {
        const int key0 = first_key(it, v, tile);
        if (whole_tile(a, it, key0, tile)) continue;
        bool odd = false;
        for (int x = 0; x < tile; ++x) {
          const T *val = vals + from.offset(key0 + x) / 2;
          for (int e = lane; e < DV; e += 64)
            odd |= not_finite(__builtin_bit_cast(uint16_t, val[e]));
        }
        if (!__any(odd)) continue;
        for (int x = 0; x < tile; ++x) {
          const unsigned key = key0 + x;
          if (key - see.from >= see.n && key - it.key_lo >= see.sunk) continue;
          const int64_t at = from.offset(key) / 2;
          float s = 0.0f;
#pragma unroll
          for (int e = 0; e < PK; ++e) s += q[e] * static_cast<float>(keys[at + e * 64 + lane]);
#pragma unroll
          for (int d = 1; d < 64; d <<= 1) s += __shfl_xor(s, d, 64);
          s *= a.c;
          const float top = fmaxf(m, s), ref = top == -INFINITY ? 0.0f : top;
          const float f = __builtin_amdgcn_exp2f(m - ref);
          const float w = __builtin_amdgcn_exp2f(s - (ref - SHIFT));
          sum = sum * f + w;
#pragma unroll
          for (int e = 0; e < PV; ++e)
            o[e] = o[e] * f + w * static_cast<float>(vals[at + e * 64 + lane]);
          m = top;
        }
      }
      if (it.partial >= 0) {
        const int64_t at = static_cast<int64_t>(it.partial) + r;
#pragma unroll
        for (int e = 0; e < PV; ++e) a.sums[at * DV + e * 64 + lane] = o[e];
        if (lane == 0) *reinterpret_cast<f32x2 *>(a.ml + 2 * at) = f32x2{m, sum};
      } else {
        T *dst = reinterpret_cast<T *>(a.out + token * a.o_ts + h * a.o_hs);
        const float inv = inverse(sum);
#pragma unroll
        for (int e = 0; e < PV; ++e) dst[e * 64 + lane] = static_cast<T>(o[e] * inv);
        if (lane == 0 && a.lse)
          a.lse[static_cast<int64_t>(token) * a.n_heads + h] = log_sum(m, sum);
      }
    }
  }

  // Four waves, 32 RH rows each, tiles of 64 keys in two LDS buffers.  Of
  // 64-wide heads a wave has room for 64 rows: every operand read from LDS then
  // serves two matrix instructions, and a tile's loads and addresses twice the
  // weights.
  //
  // 128-wide heads, 2,723 queries over 3,481 to 8,153 keys, 32 heads over 8: 320
  // us and a join of 9, 0.78 PFLOP/s; the matrix unit is busy 45% of the time that
  // a CU has work, the vector unit 54%, and CUs have none for a fifth of it (776
  // items on 512 places).  64-wide heads have half the products per weight:
  // 17,337 queries, 64 heads over 8, window 1024: 438 us, 0.63 PFLOP/s, the
  // vector unit busy 76% of the time with maxima, exponentials and sums.
  template <bool SCAN>
  static __device__ __forceinline__ bool wide(const AttendArgs &a, const AttendItem &it,
                                              lds_u8 *lds) {
    constexpr int RH = kRows / 128, BUF = kWideTile * ROW;
    const int lane = threadIdx.x & 63, wave = wave_id();
    const int row = wave * 32 * RH + (lane & 31), half = lane >> 5;
    const bool idle = wave * 32 * RH >= it.n_rows;  // a wave without rows only loads
    typedef Loader<kWideTile, 4> Load;
    const Rows<kWideTile, kWideTile / 4> rows(a, it, lds, wave, lane);
    if (it.n_tiles > 0) rows.ask(0, 0);
    x8 q[RH * (DK / 16)];
    Sight see[RH];
    State st[RH];
#pragma unroll
    for (int r = 0; r < RH; ++r) {
      int pos;
      load_queries(a, it, row + 32 * r, half, q + r * (DK / 16), &pos);
      see[r] = sight(a, it, pos);
      st[r].clear();
    }
    Places w;
    find_places(w, lane);
    bool left = false;  // SCAN: a tile is left to `careful`
    if (it.n_tiles > 0) {
      loads_done();
      Load(a, it, rows, rows.row(0, 0, lane), lds, wave, lane).all();
      rows.ask(1, 1);
      lds_reads_done();
      loop_aligned();
      for (int v = 0; v < it.n_tiles; ++v) {
        loads_done();
        __syncthreads();
        lds_u8 *now = lds + (v & 1) * BUF;
        const int key0 = first_key(it, v, kWideTile);
        const bool whole = whole_tile(a, it, key0, kWideTile);
        const bool odd = SCAN && !whole &&
                         __syncthreads_or(odd_values<kWideTile>(now, threadIdx.x, 256));
        left |= odd;
        const Load load(a, it, rows, rows.row(v + 1, v + 1, lane), lds + (~v & 1) * BUF, wave, lane);
        rows.ask(v + 2, v + 2);
        if (odd || idle) {
          load.all();
          continue;
        }
        if constexpr (RH == 1) {
          f32x16 s[2];
          products<kWideTile, 0, 2>(q, now, 0, w, load, s);
          products<kWideTile, DK / 32, 2>(q, now, 32, w, load, s + 1);
          x8 p[4];
          weigh<2>(a, it, s, key0, whole, see[0], st[0], half, p);
          add_values<4, NT, 0>(p, now + kWideTile * R0, w, 0, st, NoLoader());
        } else {
          thirty_two<0, RH>(a, it, q, now, w, key0, whole, see, st, half, load);
          thirty_two<1, RH>(a, it, q, now, w, key0, whole, see, st, half, load);
        }
      }
      loads_done();
    }
    float l[RH];
    bool bad = false;
#pragma unroll
    for (int r = 0; r < RH; ++r) {
      l[r] = st[r].l + other_half(st[r].l, half);
      bad |= row + 32 * r < it.n_rows && odd_sums(st[r].o, l[r]);
    }
    if constexpr (SCAN) {
      if (__syncthreads_or(left)) {
#pragma unroll
        for (int r = 0; r < RH; ++r) lay_down(it, lds, row + 32 * r, half, st[r], l[r], 0, true);
        careful(a, it, lds);
        return true;
      }
    } else if (__syncthreads_or(bad)) {
      return false;
    }
#pragma unroll
    for (int r = 0; r < RH; ++r)
      store(a, it, lds + wave * 128 * NT * 32, (wave * RH + r) * 32, lane, st[r], l[r], 0);
    return true;
  }
  // Keys 32 B .. + 31 of a wide tile and RH rows of the lane.
  template <int B, int RH, typename L>
  static __device__ __forceinline__ void thirty_two(const AttendArgs &a, const AttendItem &it,
                                                    const x8 *q, const lds_u8 *now,
                                                    const Places &w, int key0, bool whole,
                                                    const Sight *see, State *st, int half,
                                                    const L &load) {
    f32x16 s[RH];
    products<kWideTile, B *(DK / 32), 2, RH>(q, now, 32 * B, w, load, s);
    x8 p[2 * RH];
#pragma unroll
    for (int r = 0; r < RH; ++r)
      weigh<1>(a, it, s + r, key0 + 32 * B, whole, see[r], st[r], half, p + 2 * r);
    add_values<2, NT, 0, RH>(p, now + kWideTile * R0 + 32 * B * VS, w, 0, st, NoLoader());
  }

  // Latent rows: 64 query rows, two waves to each 32 of them.  The sums of a
  // row are 512 values, too many registers beside its 576 of query for one
  // wave, so of a tile's 64 keys each wave of a pair scores 32, hands its
  // weights to the other through LDS, and both add all 64 keys to their half
  // of the values, their own keys first.  A pair ends every tile with one m.  In
  // an item's first tile and in those that some row sees in part, where rows see
  // their first keys, the two exchange their maxima first and take the same m; in
  // the others, where the exchange would be a wait, m grows by whole steps, and
  // where it grows apart each wave brings its sums, and the weights it was handed,
  // to the larger: by a power of two, so a weight is still rounded once (fp16
  // weights below 2^-20 of the largest, whose last places are lost, a second
  // time).
  template <bool SCAN>
  static __device__ __forceinline__ bool latent(const AttendArgs &a, const AttendItem &it,
                                              lds_u8 *lds) {
    const int lane = threadIdx.x & 63, wave = wave_id();
    const int part = wave & 1, half = lane >> 5;
    const int row = (wave >> 1) * 32 + (lane & 31);
    const Rows<kWideTile, kWideTile / 4> rows(a, it, lds, wave, lane);
    const bool idle = (wave >> 1) * 32 >= it.n_rows;  // a pair without rows only loads
    constexpr int BUF = kWideTile * ROW;
    lds_u8 *mine = lds + TILES_LDS + wave * WAVE_XCHG;
    const lds_u8 *theirs = lds + TILES_LDS + (wave ^ 1) * WAVE_XCHG;
    typedef __attribute__((address_space(3))) x8 lds8;
    typedef __attribute__((address_space(3))) float lds_float;
    x8 q[DK / 16] = {};
    Places w;
    find_places(w, lane);
    const Sight see = sight(a, it, position(a, it, row));
    State st;
    st.clear();
    bool left = false;  // SCAN: a tile is left to `careful`
    if (it.n_tiles > 0) {
      typedef Loader<kWideTile, 4> Load;
      rows.ask(0, 0);
      {
        // the queries come as a tile of their own, in the second buffer, since
        // a key's place in LDS is a query's too
        const int g = it.row0 + min(wave * 16 + (lane & 15), it.n_rows - 1);
        const int t = g / a.G, h = g - t * a.G + it.kv_head * a.G;
        Load(reinterpret_cast<const uint8_t *>(a.q),
             static_cast<uint64_t>(t * a.q_ts + h * a.q_hs) * 2, lds + BUF, wave, lane)
            .all();
      }
      loads_done<Load::N>();
      Load(a, it, rows, rows.row(0, 0, lane), lds, wave, lane).all();
      rows.ask(1, 1);
      if (rows.pages) loads_done<Load::N + 1>();
      else loads_done<Load::N>();
      __syncthreads();
#pragma unroll
      for (int d = 0; d < DK / 16; ++d) {
        q[d] = key_operand<kWideTile>(lds + BUF, 32 * (wave >> 1), w, d);
        // to the accumulation registers, from which a matrix instruction takes
        // an operand as well: the sums need the others
        asm volatile("" : "+a"(q[d]));
      }
      lds_reads_done();
      loop_aligned();
      for (int v = 0; v < it.n_tiles; ++v) {
        loads_done();
        __syncthreads();
        lds_u8 *now = lds + (v & 1) * BUF;
        const int key0 = first_key(it, v, kWideTile);
        const bool whole = whole_tile(a, it, key0, kWideTile);
        const bool agree = v == 0 || !whole;
        const bool odd =
            SCAN && !whole && __syncthreads_or(odd_values<kWideTile>(now, threadIdx.x, 256));
        left |= odd;
        const Load load(a, it, rows, rows.row(v + 1, v + 1, lane), lds + (~v & 1) * BUF, wave, lane);
        rows.ask(v + 2, v + 2);
        if (odd || idle) {
          load.all();
          if (!odd && agree) __syncthreads();
          if (!odd) __syncthreads();
          continue;
        }
        x8 p[2];
        f32x16 s;
        products<kWideTile, 0, 3>(q, now, 32 * part, w, load, &s);
        float top = masked_top<1>(a, it, &s, key0 + 32 * part, whole, see, half);
        if (agree) {
          if (half == 0) ((lds_float *)(mine + 2048 + 128))[lane] = top;
          __syncthreads();
          top = fmaxf(top, ((const lds_float *)(theirs + 2048 + 128))[lane & 31]);
        }
        take_top(st, top, !agree);
        st.l += weights(s, a.c, st.m, p);
        const float m = st.m;
        ((lds8 *)mine)[lane] = p[0];
        ((lds8 *)mine)[64 + lane] = p[1];
        if (half == 0) ((lds_float *)(mine + 2048))[lane] = m;
        add_values<2, NT, DK / 48>(p, now + 32 * part * VS, w, part * NT, &st, load);
        __syncthreads();
        p[0] = ((const lds8 *)theirs)[lane];
        p[1] = ((const lds8 *)theirs)[64 + lane];
        const float m2 = ((const lds_float *)(theirs + 2048))[lane & 31];
        if (__any(m2 != m)) {
          const float both = fmaxf(m, m2), f2 = __builtin_amdgcn_exp2f(m2 - finite_m(both));
          rescale<NT>(st.o, &st.l, __builtin_amdgcn_exp2f(m - finite_m(both)));
          st.m = both;
#pragma unroll
          for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int j = 0; j < 8; ++j)
              p[b][j] = static_cast<T>(static_cast<float>(p[b][j]) * f2);
        }
        add_values<2, NT, 0>(p, now + 32 * (1 - part) * VS, w, part * NT, &st, NoLoader());
      }
      loads_done();
    }
    // each wave has summed the weights of its own keys
    float l = st.l + other_half(st.l, half);
    __syncthreads();
    ((lds_float *)mine)[lane] = l;
    __syncthreads();
    l += ((const lds_float *)theirs)[lane];
    if constexpr (SCAN) {
      if (__syncthreads_or(left)) {
        lay_down(it, lds, row, half, st, l, part * NT, true);
        careful(a, it, lds);
        return true;
      }
    } else if (__syncthreads_or(row < it.n_rows && odd_sums(st.o, l))) {
      return false;
    }
    store(a, it, lds + wave * 128 * NT * 32, (wave >> 1) * 32, lane, st, l, part * NT);
    return true;
  }

  // Four waves over the same rows, each with tiles of 32 keys of its own;
  // their sums meet in LDS at the end, the waves in order.  A wave waits for no
  // other before that, so eight waves of a CU have their loads under way at
  // different times, and a tile's loads are out before its predecessor's
  // products.  Eight queries over windows of 4096 keys, 64 heads over 8, 64
  // wide: 17.5 us and a join of 4 for 67 MB, 3.8 TB/s with the start (item, page
  // numbers, first rows: three trips to HBM).  One query over 737 keys is start
  // and join alone: 13.4 us.
  template <bool SCAN>
  static __device__ __forceinline__ bool narrow(const AttendArgs &a, const AttendItem &it,
                                              lds_u8 *lds) {
    const int lane = threadIdx.x & 63, wave = wave_id();
    const int row = lane & 31, half = lane >> 5;
    x8 q[DK / 16];
    int pos;
    const Rows<kNarrowTile, kNarrowTile> rows(a, it, lds, wave, lane);
    if (wave < it.n_tiles) {
      rows.ask(wave, 0);
      rows.ask(wave + 4, 1);
    }
    load_queries(a, it, row, half, q, &pos);
    Places w;
    find_places(w, lane);
    const Sight see = sight(a, it, pos);
    State st;
    lds_u8 *own = lds + wave * kNarrowTile * ROW;
    typedef __attribute__((address_space(3))) float lds_float;
    st.clear();
    bool left = false;  // SCAN: a tile is left to `careful`
    if (wave < it.n_tiles) {
      typedef Loader<kNarrowTile, 1> Load;
      loads_done();
      Load(a, it, rows, rows.row(wave, 0, lane), own, 0, lane).all();
      int n = 0;  // tiles of the wave so far
      lds_reads_done();
      loop_aligned();
      for (int v = wave; v < it.n_tiles; v += 4, ++n) {
        const int key0 = first_key(it, v, kNarrowTile);
        const bool whole = whole_tile(a, it, key0, kNarrowTile);
        if constexpr (SCAN) loads_done();
        else loads_done<Load::N1>();  // the keys; the values may be on their way
        if (SCAN && !whole && __any(odd_values<kNarrowTile>(own, lane, 64))) {
          left = true;
          rows.ask(v + 8, n + 2);
          lds_reads_done();
          Load(a, it, rows, rows.row(v + 4, n + 1, lane), own, 0, lane).all();
          continue;
        }
        f32x16 s;
        products<kNarrowTile, 0, 1>(q, own, 0, w, NoLoader(), &s);
        // the keys have been read: the next ones' loads may overwrite them
        const bool more = v + 4 < it.n_tiles;
        const Load load(a, it, rows, rows.row(v + 4, n + 1, lane), own, 0, lane);
        lds_reads_done();
        if (more) {
          rows.ask(v + 8, n + 2);
          load.template all<0, Load::N0>();
        }
        x8 p[2];
        weigh<1>(a, it, &s, key0, whole, see, st, half, p);
        if (!more) loads_done();
        else if (rows.pages) loads_done<Load::N0 + 1>();
        else loads_done<Load::N0>();
        add_values<2, NT, 0>(p, own + kNarrowTile * R0, w, 0, &st, NoLoader());
        lds_reads_done();
        if (more) load.template all<Load::N0, Load::N>();
      }
      loads_done();
    }
    const float l = st.l + other_half(st.l, half);

    // The waves lay their sums side by side, and a wave takes a row at a time
    // of all four.
    constexpr int C = DV / 4, M = C < 32 ? C - 1 : 31, PER = DV / 64;
    typedef __attribute__((address_space(3))) u32x4 lds16;
    typedef float Values __attribute__((ext_vector_type(PER)));
    typedef __attribute__((address_space(3))) Values lds_values;
    lds_float *ml = (lds_float *)(lds + TILES_LDS);  // of wave w, row r: w * 32 + r
    __syncthreads();
    if (row < it.n_rows) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          f32x4 x;
#pragma unroll
          for (int j = 0; j < 4; ++j) x[j] = st.o[t][4 * y + j];
          *(lds16 *)(lds + ((wave * 32 + row) * C + ((8 * t + 2 * y + half) ^ (row & M))) * 16) =
              __builtin_bit_cast(u32x4, x);
        }
      if (half == 0) {
        ml[2 * (wave * 32 + row)] = st.m;
        ml[2 * (wave * 32 + row) + 1] = l;
      }
    }
    left = __syncthreads_or(left);  // (SCAN)
    bool odd = false;
    for (int r = wave; r < it.n_rows; r += 4) {
      float m[4], sum = 0.0f, top = -INFINITY;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        m[x] = ml[2 * (x * 32 + r)];
        top = fmaxf(top, m[x]);
      }
      Values o = {};
      const int chunk = lane * PER / 4, rest = lane * PER % 4;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float f = __builtin_amdgcn_exp2f(m[x] - finite_m(top));
        sum += ml[2 * (x * 32 + r) + 1] * f;
        o += *(const lds_values *)(lds + ((x * 32 + r) * C + (chunk ^ (r & M))) * 16 + rest * 4) * f;
      }
      float zero = sum * 0.0f;
#pragma unroll
      for (int e = 0; e < PER; ++e) zero = __builtin_fmaf(o[e], 0.0f, zero);
      odd |= !(zero == 0.0f);
      if (SCAN && left) {  // where `careful` looks for them: row r of all is in use no more
        lds_reads_done();
#pragma unroll
        for (int e = 0; e < PER; ++e) ((lds_float *)lds)[r * DV + lane * PER + e] = o[e];
        if (lane == 0) {
          ml[2 * r] = top;
          ml[2 * r + 1] = sum;
        }
        continue;
      }
      if (it.partial >= 0) {
        const int64_t at = static_cast<int64_t>(it.partial) + r;
        *reinterpret_cast<Values *>(a.sums + at * DV + lane * PER) = o;
        if (lane == 0) *reinterpret_cast<f32x2 *>(a.ml + 2 * at) = f32x2{top, sum};
        continue;
      }
      int64_t lse_at;
      T *to = reinterpret_cast<T *>(a.out + out_place(a, it, it.row0 + r, &lse_at)) + lane * PER;
      typedef T Out __attribute__((ext_vector_type(PER)));
      Out x;
#pragma unroll
      for (int e = 0; e < PER; ++e) x[e] = static_cast<T>(o[e] * inverse(sum));
      *reinterpret_cast<Out *>(to) = x;
      if (lane == 0 && a.lse) a.lse[lse_at] = log_sum(top, sum);
    }
    if constexpr (SCAN) {
      if (left) careful(a, it, lds);
      return true;
    } else {
      return !__syncthreads_or(odd);  // (what was written is written over)
    }
  }

  // An item's work.  False: its sums hold an infinity or NaN, and the item is to
  // be done again with SCAN.
  template <bool SCAN>
  static __device__ __forceinline__ bool item(const AttendArgs &a, const AttendItem &it,
                                              lds_u8 *lds) {
    if constexpr (IN_KEY) return latent<SCAN>(a, it, lds);
    else if constexpr (NARROW) return narrow<SCAN>(a, it, lds);
    else return it.wide ? wide<SCAN>(a, it, lds) : narrow<SCAN>(a, it, lds);
  }
  // Apart, so that the registers of the common case are allotted without it.
  static __device__ __attribute__((noinline)) void again(AttendArgs a, AttendItem it, lds_u8 *lds) {
    item<true>(uniform(a), uniform(it), uniform(lds));
  }
};

template <typename T, int DK, int DV, bool IN_KEY, bool NARROW>
__global__ __launch_bounds__(256, blocks_per_cu(DK == 576 ? 2 : DK / 128)) void k_attend(AttendArgs a) {
  typedef Attend<T, DK, DV, IN_KEY, NARROW> A;
  __shared__ __attribute__((aligned(1024))) uint8_t memory[A::LDS];
  lds_u8 *lds = (lds_u8 *)memory;
  // The arguments come in lines of 64 bytes, each a trip to memory: one of every
  // line is asked for here, so that no trip waits for another (two short prompts
  // of latent rows: 21.1 us so, 22.0 without).
  asm volatile("" ::"s"(a.list), "s"(a.sums), "s"(a.status), "s"(a.positions_at));
  const AttendItem it = reinterpret_cast<const AttendItem *>(a.list)[blockIdx.x];
  if (!item_fits(a, it, IN_KEY ? 2 : DK / 128, NARROW)) {
    if (threadIdx.x == 0 && a.status) atomicOr(a.status, GPB_STATUS_BAD_PLAN_INPUT);
    return;
  }
  if (!A::template item<false>(a, it, lds)) A::again(a, it, lds);
}

// The rows of one token and KV head: parts weighted by 2^(m - max m), in the
// order of the list.  A wave a row; a lane first takes a part's m and l, then
// DV / 64 values of every part, four parts' under way at once.  Bound by latency
// (the reference, m and l, sums: 4 us for 64 rows of 8 parts) and, with many
// rows, by the sums: 8.8 us for 22 MB.
template <typename T, int DV>
__global__ __launch_bounds__(256) void k_attend_join(AttendArgs a) {
  typedef Attend<T, 64, 64, false, false> A;  // for what depends on T alone
  const AttendJoin j = reinterpret_cast<const AttendJoin *>(a.list + a.joins_at)[blockIdx.x];
  const int lane = threadIdx.x & 63, r = blockIdx.y * 4 + wave_id();
  constexpr int PER = DV / 64;
  typedef float Values __attribute__((ext_vector_type(PER)));
  bool ok = j.row0 >= 0 && j.n_rows >= 1 && j.n_rows <= kNarrowRows &&
            static_cast<int64_t>(j.row0) + j.n_rows <= static_cast<int64_t>(a.n_tokens) * a.G &&
            j.kv_head >= 0 && j.kv_head < a.hkv && j.ref0 >= 0 && j.n_refs >= 1 &&
            j.ref0 <= a.n_refs - j.n_refs;
  const int32_t *refs = a.list + a.refs_at + (ok ? j.ref0 : 0);
  const int n = ok ? j.n_refs : 0;
  float top = -INFINITY;
  if (ok && r >= j.n_rows) return;
  for (int i = lane; i < n; i += 64) {
    if (refs[i] < 0 || refs[i] > a.n_partial_rows - j.n_rows) ok = false;
    else top = fmaxf(top, a.ml[2 * (static_cast<int64_t>(refs[i]) + r)]);
  }
  if (__any(!ok)) {
    if (lane == 0 && a.status) atomicOr(a.status, GPB_STATUS_BAD_PLAN_INPUT);
    return;
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d, 64));
  const float ref = A::finite_m(top);
  float l = 0.0f;
  Values o = {};
  for (int i0 = 0; i0 < n; i0 += 64) {
    int at = refs[min(i0 + lane, n - 1)] + r;
    float f = 0.0f;
    if (i0 + lane < n) {
      const f32x2 ml = *reinterpret_cast<const f32x2 *>(a.ml + 2 * static_cast<int64_t>(at));
      f = __builtin_amdgcn_exp2f(ml[0] - ref);
      l += ml[1] * f;
    }
    const int some = min(64, n - i0);
    for (int i = 0; i < some; i += 4) {  // four parts' values under way at once
      Values x[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        x[u] = *reinterpret_cast<const Values *>(
            a.sums + static_cast<int64_t>(__builtin_amdgcn_readlane(at, min(i + u, some - 1))) * DV +
            lane * PER);
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (i + u < some)
          o += x[u] * __builtin_bit_cast(
                          float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, f), i + u));
    }
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) l += __shfl_xor(l, d, 64);
  const int g = j.row0 + r;
  const int t = g / a.G, h = g - t * a.G + j.kv_head * a.G;
  const float inv = A::inverse(l);
  typedef T Out __attribute__((ext_vector_type(PER > 4 ? 4 : PER)));
  T *dst = reinterpret_cast<T *>(a.out + t * a.o_ts + h * a.o_hs) + lane * PER;
#pragma unroll
  for (int e = 0; e < PER; e += PER > 4 ? 4 : PER) {
    Out x;
#pragma unroll
    for (int y = 0; y < (PER > 4 ? 4 : PER); ++y) x[y] = static_cast<T>(o[e + y] * inv);
    *reinterpret_cast<Out *>(dst + e) = x;
  }
  if (lane == 0 && a.lse) a.lse[static_cast<int64_t>(t) * a.n_heads + h] = A::log_sum(top, l);
}

template <typename T, int DK, int DV, bool IN_KEY>
int launch_attend(const AttendArgs &a, bool narrow, hipStream_t st) {
  const dim3 items(a.n_items), block(256);
  int rc;
  if constexpr (IN_KEY) rc = launch(k_attend<T, DK, DV, true, false>, items, block, st, a);
  else rc = narrow ? launch(k_attend<T, DK, DV, false, true>, items, block, st, a)
                   : launch(k_attend<T, DK, DV, false, false>, items, block, st, a);
  if (rc == GPB_OK && a.n_joins > 0)
    rc = launch(k_attend_join<T, DV>,
                dim3(a.n_joins, static_cast<uint32_t>(std::min(a.G, kNarrowRows) + 3) / 4), block,
                st, a);
  return rc;
}

template <typename T>
int launch_format(int which, const AttendArgs &a, bool narrow, hipStream_t st) {
  if (which == 0) return launch_attend<T, 64, 64, false>(a, narrow, st);
  if (which == 1) return launch_attend<T, 128, 128, false>(a, narrow, st);
  return launch_attend<T, 576, 512, true>(a, narrow, st);
}

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
  return p->format.dtype == GPB_BF16
             ? launch_format<__bf16>(which, a, narrow, as_stream(stream))
             : launch_format<_Float16>(which, a, narrow, as_stream(stream));
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
