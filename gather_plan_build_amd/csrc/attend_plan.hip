// attend_plan.hip -- the work list of an attention (host code only).
//
// A batch is cut into segments: a request's queries over its own keys, or a
// group's queries over the keys that its requests share.  A segment's query
// rows (tokens times the heads of one KV head) are cut into blocks, one per
// workgroup, and a block's keys, which are whole tiles up to the last position
// that its queries reach, into parts where they would keep one workgroup busy
// longer than the batch keeps the GPU.  Blocks whose rows have one part write
// their results; the others write sums, and a join per token and KV head adds
// its parts in the order of the list, so results do not depend on timing.
#include <algorithm>
#include <new>
#include <utility>
#include <vector>

#include "attend.h"

namespace gpb {
namespace {

constexpr int kCus = 256, kXcds = 8;

struct Block {
  int64_t row0;
  int32_t n_rows;
  int32_t n_tiles, tile0, n_first, tile1;
  int32_t pos_min, pos_max;
  int32_t parts;
  int64_t partial;  // workspace row of (KV head 0, part 0), -1: direct
};

struct Segment {
  int32_t req;
  int64_t tok0, n_tok;
  int32_t key_lo, key_hi;
  bool grouped, wide;
  size_t block0, n_blocks;
};

struct Planner {
  const gpb_attend_shape &s;
  int32_t G;  // query heads per KV head
  int which;  // attention kernel
  std::vector<int64_t> q_start;
  std::vector<int32_t> pos;
  std::vector<Segment> segments;
  std::vector<Block> blocks;
  std::vector<int32_t> group_of;  // segment of a request's shared keys, or -1
  std::vector<int32_t> own;       // segment of a request's own keys, or -1

  int rows_of(bool wide) const { return gpb::rows_of(which, wide); }
  int tile_of(bool wide) const { return wide ? kWideTile : kNarrowTile; }

  // The tiles of a block: those of the first tokens (A) and those from the
  // window of its first query on (B), or one range where the two meet.
  void tiles(const Segment &g, Block *b) const {
    const int64_t tn = tile_of(g.wide);
    const int64_t lo = g.key_lo;
    const int64_t hi = std::min<int64_t>(g.key_hi, static_cast<int64_t>(b->pos_max) + 1);
    b->tile0 = static_cast<int32_t>(lo / tn);
    b->n_tiles = b->n_first = b->tile1 = 0;
    if (hi <= lo) return;
    const int64_t end = ceil_div64(hi, tn);
    const int64_t sunk = s.window > 0 ? std::min<int64_t>(hi, s.sinks) : lo;
    const int64_t near = s.window > 0
        ? std::max<int64_t>(lo, static_cast<int64_t>(b->pos_min) - s.window + 1) : lo;
    const int64_t a0 = lo / tn, a1 = sunk > lo ? ceil_div64(sunk, tn) : a0;
    const int64_t b0 = near < hi ? near / tn : end;
    if (a1 > a0 && a1 < b0) {
      b->n_first = static_cast<int32_t>(a1 - a0);
      // (shared keys may all lie behind the window of the group's queries)
      b->tile1 = b0 < end ? static_cast<int32_t>(b0) : 0;
      b->n_tiles = static_cast<int32_t>(b->n_first + (end - b0));
    } else {
      const int64_t from = a1 > a0 ? a0 : b0;
      b->tile0 = static_cast<int32_t>(from);
      b->n_tiles = b->n_first = static_cast<int32_t>(end - from);
    }
  }

  void add_segment(int32_t req, int64_t tok0, int64_t n_tok, int32_t lo, int32_t hi,
                   bool grouped) {
    Segment g{req, tok0, n_tok, lo, hi, grouped,
              which == 2 || n_tok * G > kNarrowRows, blocks.size(), 0};
    const int64_t M = rows_of(g.wide);
    auto add = [&](int64_t row0, int64_t n) {
      Block b{};
      b.row0 = row0;
      b.n_rows = static_cast<int32_t>(n);
      b.pos_min = INT32_MAX;
      b.pos_max = INT32_MIN;
      for (int64_t t = row0 / G; t <= (row0 + n - 1) / G; ++t) {
        b.pos_min = std::min(b.pos_min, pos[t]);
        b.pos_max = std::max(b.pos_max, pos[t]);
      }
      tiles(g, &b);
      blocks.push_back(b);
    };
    if (G <= M) {
      const int64_t per = M / G;
      for (int64_t t = 0; t < n_tok; t += per)
        add((tok0 + t) * G, std::min(per, n_tok - t) * G);
    } else {
      for (int64_t t = 0; t < n_tok; ++t)
        for (int64_t h = 0; h < G; h += M) add((tok0 + t) * G + h, std::min(M, G - h));
    }
    g.n_blocks = blocks.size() - g.block0;
    segments.push_back(g);
  }

  // The block of segment g that holds rows of token t from head h on, and the
  // place of that row in it.
  const Block &find(const Segment &g, int64_t t, int64_t h, int64_t *at) const {
    const int64_t M = rows_of(g.wide), i = t - g.tok0;
    size_t k;
    if (G <= M) {
      k = i / (M / G);
    } else {
      k = i * ceil_div64(G, M) + h / M;
    }
    const Block &b = blocks[g.block0 + k];
    *at = t * G + h - b.row0;
    return b;
  }
};

int plan_build(const gpb_row_format *f, const gpb_attend_shape *s, gpb_attend_plan *plan,
               int32_t *h_list, int64_t list_ints) {
  int rc = check_format(f);
  if (rc != GPB_OK) return rc;
  if (!s || !plan || list_ints < 0) return GPB_EINVAL;
  const int which = attend_kernel(*f);
  if (which < 0 || s->bs < 0 || s->n_heads < 1 || s->n_heads > 65536 ||
      s->n_heads % f->n_kv_heads || s->window < 0 || s->sinks < 0 || s->page_rows < 1 ||
      s->n_groups < 0 || (s->bs > 0 && (!s->h_q_lens || !s->h_kv_lens)) ||
      (s->n_groups > 0 && !s->h_groups))
    return GPB_EINVAL;
  Planner p{*s, s->n_heads / f->n_kv_heads, which};
  const int64_t hkv = f->n_kv_heads, G = p.G;
  int64_t tokens = 0, longest = 0;
  p.q_start.resize(s->bs);
  for (int32_t r = 0; r < s->bs; ++r) {
    const int64_t q = s->h_q_lens[r], n = s->h_kv_lens[r];
    if (q < 0 || n < 0) return GPB_EINVAL;
    p.q_start[r] = tokens;
    tokens += q;
    if (tokens > INT32_MAX) return GPB_ERANGE;
    longest = std::max(longest, n);
  }
  // rows of a KV head, positions and keys are int32 in the list
  if (tokens * G > INT32_MAX / 2 || tokens * s->n_heads > INT32_MAX || longest > INT32_MAX / 2)
    return GPB_ERANGE;
  p.pos.resize(tokens);
  for (int32_t r = 0; r < s->bs; ++r)
    for (int32_t j = 0; j < s->h_q_lens[r]; ++j)
      p.pos[p.q_start[r] + j] = s->h_kv_lens[r] - s->h_q_lens[r] + j;

  p.group_of.assign(s->bs, -1);
  p.own.assign(s->bs, -1);
  std::vector<int32_t> shared(s->bs, 0);
  int64_t done = 0;
  for (int32_t g = 0; g < s->n_groups; ++g) {
    const int64_t first = s->h_groups[3 * g], n = s->h_groups[3 * g + 1];
    const int32_t keys = s->h_groups[3 * g + 2];
    if (first < done || n < 1 || first + n > s->bs || keys < 1 || keys % s->page_rows)
      return GPB_EINVAL;
    done = first + n;
    int64_t group_tokens = 0;
    for (int64_t r = first; r < done; ++r) {
      if (keys > static_cast<int64_t>(s->h_kv_lens[r]) - s->h_q_lens[r]) return GPB_EINVAL;
      group_tokens += s->h_q_lens[r];
      if (n > 1) shared[r] = keys;
    }
    if (n == 1 || group_tokens == 0) continue;
    for (int64_t r = first; r < done; ++r)
      p.group_of[r] = static_cast<int32_t>(p.segments.size());
    p.add_segment(static_cast<int32_t>(first), p.q_start[first], group_tokens, 0, keys, true);
  }
  for (int32_t r = 0; r < s->bs; ++r) {
    if (s->h_q_lens[r] == 0) continue;
    const bool grouped = p.group_of[r] >= 0;
    p.own[r] = static_cast<int32_t>(p.segments.size());
    p.add_segment(r, p.q_start[r], s->h_q_lens[r], grouped ? shared[r] : 0, s->h_kv_lens[r],
                  grouped);
  }

  // Cut long ranges of keys into parts of at most `most` keys, none shorter
  // than min_keys (one query of 737 keys, 32 heads over 8: 13.4 us with parts of
  // 256 keys, 13.7 of 128, 15.7 of 64).  A workgroup's start and end take as
  // long as `start` keys: 2,723 queries over 3,481 to 8,153 keys, 32 heads over
  // 8, 128 wide, 326 us so, 347 with none and 326 with twice as many; 48 queries
  // behind 16,384 shared keys 58, 56 and 65.  A key counts the same in a wide, a
  // narrow and a half-empty item, which it is not: their lists are a compromise.
  int64_t total = 0, uncut = 0, longest_block = 1;
  for (const Segment &g : p.segments)
    for (size_t k = 0; k < g.n_blocks; ++k) {
      const int64_t keys = static_cast<int64_t>(p.tile_of(g.wide)) * p.blocks[g.block0 + k].n_tiles;
      total += hkv * keys;
      uncut += hkv;
      longest_block = std::max(longest_block, keys);
    }
  const int64_t slots = kCus * blocks_per_cu(which);
  const int64_t min_keys = 256, start = which == 2 ? 150 : 300;
  auto cut = [&](const Segment &g, const Block &b, int64_t most) {
    const int64_t keys = static_cast<int64_t>(b.n_tiles) * p.tile_of(g.wide);
    return std::max<int64_t>(1, std::min<int64_t>(b.n_tiles, ceil_div64(keys, most)));
  };
  // How long the batch takes, in keys, if its workgroups start the longest
  // first: the longest one where all run at once; else all of them spread
  // evenly, and the longest of those that had to wait, which starts when the
  // rest end.  A join costs a launch (160 keys' time of 33 ns: two requests of
  // 292 and 357 latent rows, 16 heads, take 21.0 us whole and 23.2 us in
  // parts; with half of it 4,200 queries of 128-wide heads take 281 us instead of
  // 263, twice as much changes nothing measured), and sums written and read again take the whole GPU about a key's
  // time per 19,000 values.
  std::vector<std::pair<int64_t, int64_t>> lengths;  // keys, how many
  auto span = [&](int64_t most) {
    lengths.clear();
    int64_t n = 0, sum = 0, longest = 0, rows = 0;
    for (const Segment &g : p.segments)
      for (size_t k = 0; k < g.n_blocks; ++k) {
        const Block &b = p.blocks[g.block0 + k];
        const int64_t parts = cut(g, b, most);
        const int64_t keys = static_cast<int64_t>(b.n_tiles) * p.tile_of(g.wide) / parts + start;
        lengths.emplace_back(keys, hkv * parts);
        n += hkv * parts;
        sum += hkv * parts * keys;
        longest = std::max(longest, keys);
        if (g.grouped || parts > 1) rows += hkv * parts * b.n_rows;
      }
    const int64_t again = rows > 0 ? 160 + rows * f->v_dim / 19000 : 0;
    if (n <= slots) return longest + again;
    std::sort(lengths.rbegin(), lengths.rend());
    int64_t before = 0, waits = 0;
    for (const auto &l : lengths) {
      waits = l.first;
      before += l.second;
      if (before > slots) break;
    }
    return std::max(longest, sum / slots + waits) + again;
  };
  // Parts of an even share of the work, or of the length among some multiples of
  // it, or uncut, that `span` finds best: 32 queries over 613 to 8,084 latent
  // rows 42 us so, 51 with three lengths to choose from and 59 with the even
  // share; 120 behind shared latent rows 148, 207 and 188; 2,500 queries of
  // 64-wide heads 205, 205 and 222; nothing measured is more than 4% slower.
  // With more than four blocks to a place the uncut ones fill the GPU evenly, and
  // the lists are the same either way, but the search takes its time on the host:
  // 44,600 queries over latent rows 0.7 ms without it, 2.5 with it.
  int64_t most = std::max(min_keys, ceil_div64(total, slots));
  if (uncut <= 4 * slots) {
    int64_t best = INT64_MAX;
    const int64_t even = most;
    for (int64_t part : {longest_block, even * 3, even * 2, even * 3 / 2, even * 5 / 4,
                         even * 9 / 8, even, even * 2 / 3, even / 2}) {
      part = std::max(min_keys, part);
      const int64_t t = span(part);
      if (t < best) best = t, most = part;
    }
  }
  int64_t n_items = 0, n_partial = 0, n_joins = 0, n_refs = 0;
  for (const Segment &g : p.segments)
    for (size_t k = 0; k < g.n_blocks; ++k) {
      Block &b = p.blocks[g.block0 + k];
      b.parts = static_cast<int32_t>(cut(g, b, most));
      b.partial = -1;
      if (g.grouped || b.parts > 1) {
        b.partial = n_partial;
        n_partial += hkv * b.parts * b.n_rows;
      }
      n_items += hkv * b.parts;
    }
  // (a launch has fewer than 2^32 threads)
  if (n_items > UINT32_MAX / 256 || n_partial > INT32_MAX) return GPB_ERANGE;

  // joins: every token's rows of a KV head in runs of at most 32 (which no
  // block cuts), where the token has more than one part
  std::vector<AttendJoin> joins;
  std::vector<int32_t> refs;
  for (int32_t r = 0; r < s->bs; ++r) {
    if (p.own[r] < 0) continue;
    const Segment *parts_of[2] = {p.group_of[r] >= 0 ? &p.segments[p.group_of[r]] : nullptr,
                                  &p.segments[p.own[r]]};
    for (int64_t t = p.q_start[r]; t < p.q_start[r] + s->h_q_lens[r]; ++t)
      for (int64_t h = 0; h < G; h += kNarrowRows) {
        int64_t at;
        if (!parts_of[0] && p.find(*parts_of[1], t, h, &at).partial < 0) continue;
        for (int64_t v = 0; v < hkv; ++v) {
          AttendJoin j{};
          j.row0 = static_cast<int32_t>(t * G + h);
          j.n_rows = static_cast<int32_t>(std::min<int64_t>(kNarrowRows, G - h));
          j.kv_head = static_cast<int32_t>(v);
          j.ref0 = static_cast<int32_t>(refs.size());
          for (const Segment *g : parts_of) {
            if (!g) continue;
            const Block &b = p.find(*g, t, h, &at);
            for (int64_t x = 0; x < b.parts; ++x)
              refs.push_back(
                  static_cast<int32_t>(b.partial + (v * b.parts + x) * b.n_rows + at));
          }
          j.n_refs = static_cast<int32_t>(refs.size()) - j.ref0;
          joins.push_back(j);
          if (refs.size() > INT32_MAX / 4u || joins.size() > UINT32_MAX / 256) return GPB_ERANGE;
        }
      }
  }
  n_joins = static_cast<int64_t>(joins.size());
  n_refs = static_cast<int64_t>(refs.size());
  const int64_t ints = n_items * kItemInts + n_joins * kJoinInts + n_refs + tokens;
  if (ints > INT32_MAX) return GPB_ERANGE;

  *plan = gpb_attend_plan{};
  plan->format = *f;
  plan->bs = s->bs; plan->n_heads = s->n_heads; plan->window = s->window;
  plan->sinks = s->sinks; plan->page_rows = s->page_rows; plan->n_groups = s->n_groups;
  plan->n_tokens = static_cast<int32_t>(tokens);
  plan->max_keys = static_cast<int32_t>(longest);
  plan->n_items = static_cast<int32_t>(n_items);
  for (const Segment &g : p.segments)
    for (size_t k = 0; g.wide && k < g.n_blocks; ++k)
      plan->n_wide += static_cast<int32_t>(hkv * p.blocks[g.block0 + k].parts);
  plan->n_joins = static_cast<int32_t>(n_joins);
  plan->n_refs = static_cast<int32_t>(n_refs);
  plan->n_partial_rows = static_cast<int32_t>(n_partial);
  plan->joins_at = static_cast<int32_t>(n_items * kItemInts);
  plan->refs_at = static_cast<int32_t>(plan->joins_at + n_joins * kJoinInts);
  plan->positions_at = static_cast<int32_t>(plan->refs_at + n_refs);
  plan->list_ints = static_cast<int32_t>(ints);
  plan->workspace_bytes = n_partial * (f->v_dim + 2) * 4;
  if (!h_list) return GPB_OK;
  if (list_ints < ints) return GPB_ERANGE;

  // Items, the longest first (the last workgroups to start are then short), the
  // KV heads of a part next to each other.
  struct Part { int64_t keys; const Segment *g; const Block *b; int32_t x, v; };
  std::vector<Part> parts;
  for (const Segment &g : p.segments)
    for (size_t k = 0; k < g.n_blocks; ++k) {
      const Block &b = p.blocks[g.block0 + k];
      for (int32_t x = 0; x < b.parts; ++x)
        for (int32_t v = 0; v < hkv; ++v)
          parts.push_back({static_cast<int64_t>(b.n_tiles / b.parts) * p.tile_of(g.wide), &g, &b,
                           x, v});
    }
  std::stable_sort(parts.begin(), parts.end(),
                   [](const Part &x, const Part &y) { return x.keys > y.keys; });
  // Item i runs on XCD i % 8, each with an L2 of its own.  The blocks of a group
  // read the same keys at one time, so those that read the same heads and keys
  // are dealt to as few XCDs as may be: 20 blocks of 64 rows over 32,768 shared
  // latent rows in 9 parts, 160 us so and 184 us with the blocks of a part on
  // any XCD.  (Other items: the heads, next to each other, find their own.)
  for (size_t first = 0, end; first < parts.size(); first = end) {
    for (end = first + 1; end < parts.size() && parts[end].keys == parts[first].keys &&
                          parts[end].g == parts[first].g;)
      ++end;
    if (!parts[first].g->grouped) continue;
    std::vector<Part> run(parts.begin() + first, parts.begin() + end);
    std::stable_sort(run.begin(), run.end(), [](const Part &x, const Part &y) {
      return x.v != y.v ? x.v < y.v : x.x < y.x;
    });
    size_t from = 0;
    for (size_t xcd = 0; xcd < kXcds; ++xcd)
      for (size_t i = first + (xcd + kXcds - first % kXcds) % kXcds; i < end; i += kXcds)
        parts[i] = run[from++];
  }
  AttendItem *out = reinterpret_cast<AttendItem *>(h_list);
  for (const Part &q : parts) {
    const Block &b = *q.b;
    const int64_t v0 = static_cast<int64_t>(b.n_tiles) * q.x / b.parts;
    const int64_t v1 = static_cast<int64_t>(b.n_tiles) * (q.x + 1) / b.parts;
    AttendItem it{};
    it.req = q.g->req; it.row0 = static_cast<int32_t>(b.row0); it.n_rows = b.n_rows;
    it.kv_head = q.v;
    it.key_lo = q.g->key_lo; it.key_hi = q.g->key_hi;
    it.n_tiles = static_cast<int32_t>(v1 - v0);
    if (v0 < b.n_first) {
      it.tile0 = static_cast<int32_t>(b.tile0 + v0);
      it.n_first = static_cast<int32_t>(std::min<int64_t>(v1, b.n_first) - v0);
      it.tile1 = b.tile1;
    } else {
      it.tile0 = static_cast<int32_t>(b.tile1 + v0 - b.n_first);
      it.n_first = it.n_tiles;
    }
    it.wide = q.g->wide;
    it.pos_min = b.pos_min; it.pos_max = b.pos_max;
    it.partial = b.partial < 0
                     ? -1
                     : static_cast<int32_t>(b.partial + (static_cast<int64_t>(q.v) * b.parts + q.x) *
                                                            b.n_rows);
    *out++ = it;
  }
  std::copy(joins.begin(), joins.end(),
            reinterpret_cast<AttendJoin *>(h_list + plan->joins_at));
  std::copy(refs.begin(), refs.end(), h_list + plan->refs_at);
  std::copy(p.pos.begin(), p.pos.end(), h_list + plan->positions_at);
  return GPB_OK;
}

}  // namespace
}  // namespace gpb

extern "C" int gpb_attend_plan_build(const gpb_row_format *format, const gpb_attend_shape *shape,
                                     gpb_attend_plan *plan, int32_t *h_list, int64_t list_ints) {
  try {
    return gpb::plan_build(format, shape, plan, h_list, list_ints);
  } catch (const std::bad_alloc &) {
    return GPB_ENOMEM;
  } catch (...) {
    return GPB_EINVAL;
  }
}
