// Host side of the serving step (include/kamera_step.h): argument validation, the attention's
// work list, packing into the workspace, page-copy ordering, launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>
#include <vector>

#include "kamera_step_desc.h"

using namespace kamera;

namespace {

constexpr size_t kAlign = 256;
size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
size_t elem_bytes(const kamera_layout* L) { return L->dtype == KAMERA_BF16 ? 2 : 4; }

int row_width(const kamera_layout* L) {
  return L->family == KAMERA_GQA ? L->num_kv_heads * L->head_dim : L->latent_dim + L->rope_dim;
}

// Shapes of a step that follow from the layout.
struct Shape {
  int heads, group, dk, dv, d_rot;
};
Shape shape_of(const kamera_layout* L, int num_q_heads) {
  if (L->family == KAMERA_GQA)
    return Shape{L->num_kv_heads, num_q_heads / L->num_kv_heads, L->head_dim, L->head_dim, L->head_dim};
  return Shape{1, num_q_heads, L->latent_dim + L->rope_dim, L->latent_dim, L->rope_dim};
}

// ------------------------------------------------------------------ validation
// Counts of a valid step: query tokens, page-table entries used.
struct Counts {
  int64_t tokens = 0, entries = 0;
};

// slots and key numbers are 32-bit in the kernels, with room for a tile beyond the last
constexpr int64_t kMaxSlot = (int64_t(1) << 31) - 4096;

int64_t table_entries(int32_t slot0, int64_t tokens, int P) { return tokens > 0 ? ceil_div(slot0 + tokens, P) : 0; }

kamera_status check_step(const kamera_layout* L, const kamera_step* s, Counts& n) {
  kamera_status st = host_check_layout(L);
  if (st != KAMERA_OK) return st;
  if (!s) return host_fail(KAMERA_E_NULL, "step is NULL");
  if (!(s->flags & (KAMERA_STEP_APPEND | KAMERA_STEP_ATTEND)) || (s->flags & ~(uint32_t)(KAMERA_STEP_APPEND | KAMERA_STEP_ATTEND | KAMERA_STEP_FIT)))
    return host_fail(KAMERA_E_UNSUPPORTED, "step.flags 0x%x", s->flags);
  if (s->num_requests < 0 || s->num_prefixes < 0) return host_fail(KAMERA_E_SHAPE, "negative count of requests or prefixes");
  if (s->reserved[0] || s->reserved[1]) return host_fail(KAMERA_E_SHAPE, "step.reserved must be 0");
  if ((s->num_requests && !s->requests) || (s->num_prefixes && !s->prefixes))
    return host_fail(KAMERA_E_NULL, "requests or prefixes is NULL");
  const bool attend = s->flags & KAMERA_STEP_ATTEND, append = s->flags & KAMERA_STEP_APPEND;
  if (s->num_q_heads < (attend ? 1 : 0) || s->num_q_heads > (1 << 16))
    return host_fail(KAMERA_E_SHAPE, "num_q_heads %d", s->num_q_heads);
  if (L->family == KAMERA_GQA && s->num_q_heads % L->num_kv_heads)
    return host_fail(KAMERA_E_SHAPE, "num_q_heads %d is not a multiple of num_kv_heads %d", s->num_q_heads, L->num_kv_heads);
  const Shape h = shape_of(L, s->num_q_heads);
  if (attend && h.dv < 1) return host_fail(KAMERA_E_SHAPE, "attention over rows without a latent");
  if (attend && h.dk > KAMERA_ATTEND_MAX_DIM)
    return host_fail(KAMERA_E_UNSUPPORTED, "key heads of %d columns (at most %d)", h.dk, (int)KAMERA_ATTEND_MAX_DIM);
  if (append && s->positions && !aligned(s->positions, sizeof(int32_t)))
    return host_fail(KAMERA_E_ALIGN, "positions must be 4-byte aligned");
  const int P = L->page_size;
  for (int i = 0; i < s->num_prefixes; ++i) {
    const kamera_prefix& p = s->prefixes[i];
    if (p.num_tokens < 0) return host_fail(KAMERA_E_SHAPE, "prefix %d: num_tokens < 0", i);
    if (p.num_tokens == 0) continue;
    if (!p.block_table) return host_fail(KAMERA_E_NULL, "prefix %d: block_table is NULL", i);
    if (p.slot0 < 0 || p.slot0 >= P) return host_fail(KAMERA_E_PAGE, "prefix %d: slot0 must be in [0, page_size)", i);
    if ((int64_t)p.slot0 + p.num_tokens >= kMaxSlot) return host_fail(KAMERA_E_SHAPE, "prefix %d: too many tokens", i);
    n.entries += table_entries(p.slot0, p.num_tokens, P);
  }
  for (int i = 0; i < s->num_requests; ++i) {
    const kamera_request& r = s->requests[i];
    if (r.num_tokens < 0 || r.num_queries < 0) return host_fail(KAMERA_E_SHAPE, "request %d: negative count", i);
    if (r.reserved) return host_fail(KAMERA_E_SHAPE, "request %d: reserved must be 0", i);
    if (r.flags & ~(uint32_t)KAMERA_REQUEST_ALL) return host_fail(KAMERA_E_UNSUPPORTED, "request %d: flags 0x%x", i, r.flags);
    if (r.prefix < -1 || r.prefix >= s->num_prefixes)
      return host_fail(KAMERA_E_SHAPE, "request %d: prefix %d of %d", i, r.prefix, s->num_prefixes);
    if (append && r.num_queries > r.num_tokens)
      return host_fail(KAMERA_E_SHAPE, "request %d: appends %d tokens but has %d", i, r.num_queries, r.num_tokens);
    if (append && !s->positions && r.num_queries) {
      const int64_t lim = int64_t(1) << 31;
      if (r.position0 <= -lim || r.position0 >= lim || r.position0 + r.num_tokens > lim)
        return host_fail(KAMERA_E_DELTA, "request %d: positions must stay within 2^31", i);
    }
    const int64_t kv = (int64_t)r.num_tokens + (r.prefix >= 0 ? s->prefixes[r.prefix].num_tokens : 0);
    if (kv >= kMaxSlot || (int64_t)r.slot0 + r.num_tokens >= kMaxSlot)
      return host_fail(KAMERA_E_SHAPE, "request %d: too many tokens", i);
    n.tokens += r.num_queries;
    if (r.num_tokens == 0) continue;
    if (!r.block_table) return host_fail(KAMERA_E_NULL, "request %d: block_table is NULL", i);
    if (r.slot0 < 0 || r.slot0 >= P) return host_fail(KAMERA_E_PAGE, "request %d: slot0 must be in [0, page_size)", i);
    n.entries += table_entries(r.slot0, r.num_tokens, P);
  }
  if (n.tokens * std::max(s->num_q_heads, 1) >= (int64_t(1) << 31) - 4096)
    return host_fail(KAMERA_E_SHAPE, "too many query rows");
  if (n.entries >= (int64_t(1) << 31)) return host_fail(KAMERA_E_SHAPE, "too many page-table entries");
  return KAMERA_OK;
}

kamera_status check_pool(const kamera_layout* L, const kamera_pool* pool) {
  if (!pool) return host_fail(KAMERA_E_NULL, "pool is NULL");
  const size_t es = elem_bytes(L);
  if (pool->num_pages < 1) return host_fail(KAMERA_E_SHAPE, "pool.num_pages must be >= 1");
  if (pool->reserved != 0) return host_fail(KAMERA_E_SHAPE, "pool.reserved must be 0");
  if (!pool->k_pool || (L->family == KAMERA_GQA && !pool->v_pool)) return host_fail(KAMERA_E_NULL, "a pool pointer is NULL");
  if (!aligned(pool->k_pool, es) || (pool->v_pool && !aligned(pool->v_pool, es)))
    return host_fail(KAMERA_E_ALIGN, "pool pointers must be aligned to %zu bytes", es);
  const int64_t min_ls = (int64_t)pool->num_pages * L->page_size * row_width(L);
  if (pool->layer_stride < 0 || (pool->layer_stride != 0 && pool->layer_stride < min_ls))
    return host_fail(KAMERA_E_SHAPE, "pool.layer_stride %lld smaller than one layer (%lld)",
                     (long long)pool->layer_stride, (long long)min_ls);
  return KAMERA_OK;
}

kamera_status check_workspace(const void* ws, size_t have, size_t need) {
  if (!ws) return host_fail(KAMERA_E_WORKSPACE, "workspace is NULL");
  if (!aligned(ws, kAlign)) return host_fail(KAMERA_E_ALIGN, "workspace must be %zu-byte aligned", kAlign);
  if (have < need) return host_fail(KAMERA_E_WORKSPACE, "workspace has %zu bytes, %zu needed", have, need);
  return KAMERA_OK;
}

// ------------------------------------------------------------------ attention work list
// A request whose rows alone fill a tile gains little from sharing its prefix's reads: it reads the
// prefix and its own tokens as one sequence, and its result needs no joining. (32 requests over an
// 8192-token prefix, 2 layers, us shared and alone. 28 + 4 heads: 28 rows a KV head 79 and 94, 84 rows
// 147 and 178, 119 rows 205 and 188. MLA, 16 heads: 32 rows 131 and 188, 64 rows 170 and 199, 128 rows
// 249 and 220.)
constexpr int64_t kShareRows = 96;

// What the choice of an item's length goes by, measured: the time of a workgroup around its keys (its
// item, page ids, rows and queries are read one after the other, its results joined and written), of
// one key of a tile while the chip is full, and of a partial row's column written and read again.
constexpr double kStartNs = 6000, kPartNs = 0.001;
double key_ns(int kernel, int tile) {
  if (kernel == ATTEND_LATENT) return tile == TILE_WIDE ? 60 : 20;
  if (kernel == ATTEND_HEADS) return tile == TILE_WIDE ? 30 : tile == TILE_PAIRS ? 38 : 25;
  return 40;
}

struct Work {
  std::vector<AttendRun> runs;
  std::vector<AttendItem> items;
  std::vector<int32_t> tok;
  std::vector<MergeToken> merge;
  int64_t part_rows = 0;
  int32_t wide = 0, pairs = 0, max_parts = 0;
  bool split = false, shared = false;  // keys of a run cut into ranges, a prefix read by a run of its own
};

// A plan for less workspace than the fastest one takes: ranges of 2^coarser times the length, and
// prefixes read by each request for itself. Without ranges and sharing no partial row is left.
struct Fit {
  int coarser = 0;
  bool share = true;
};

// Where each prefix's and request's table starts among the packed entries.
struct Tables {
  std::vector<int32_t> prefix, request;
};

// Layouts of the matrix-core kernels; they also need the pool in 16-byte pieces, and row numbers of
// 32 bits.
int matrix_kernel(const kamera_layout* L) {
  if (L->dtype != KAMERA_BF16) return ATTEND_PLAIN;
  if (L->family == KAMERA_GQA) return L->head_dim == 64 || L->head_dim == 128 ? ATTEND_HEADS : ATTEND_PLAIN;
  return L->latent_dim == 512 && L->rope_dim == 64 ? ATTEND_LATENT : ATTEND_PLAIN;
}
int pick_kernel(const kamera_layout* L, const kamera_pool* pool) {
  const int kernel = matrix_kernel(L);
  if (!aligned(pool->k_pool, 16) || (L->family == KAMERA_GQA && !aligned(pool->v_pool, 16)) || pool->layer_stride % 8) return ATTEND_PLAIN;
  if ((int64_t)pool->num_pages * L->page_size >= (int64_t(1) << 31)) return ATTEND_PLAIN;
  return kernel;
}

void plan_attention(const kamera_layout* L, const kamera_step* s, const Tables& tb, int kernel, Fit fit, Work& w) {
  const Shape h = shape_of(L, s->num_q_heads);
  const int G = h.group;
  w.runs.clear();
  w.items.clear();
  w.tok.clear();
  w.merge.clear();
  w.part_rows = 0;
  w.max_parts = 0;
  w.split = w.shared = false;
  // members of each prefix whose rows are few enough to share its reads
  std::vector<int32_t> members((size_t)s->num_prefixes, 0);
  auto few = [&](const kamera_request& r) {
    return fit.share && r.num_queries > 0 && r.prefix >= 0 && s->prefixes[r.prefix].num_tokens > 0 && (int64_t)r.num_queries * G < kShareRows;
  };
  for (int i = 0; i < s->num_requests; ++i)
    if (few(s->requests[i])) ++members[(size_t)s->requests[i].prefix];
  auto shares = [&](const kamera_request& r) { return few(r) && members[(size_t)r.prefix] > 1; };
  // runs: shared prefixes first
  std::vector<int32_t> prefix_run((size_t)s->num_prefixes, -1);
  for (int p = 0; p < s->num_prefixes; ++p) {
    if (members[(size_t)p] < 2) continue;
    w.shared = true;
    AttendRun r;
    std::memset(&r, 0, sizeof(r));
    r.pg_a = tb.prefix[(size_t)p];
    r.slot_a = s->prefixes[p].slot0;
    r.len_a = r.kv = s->prefixes[p].num_tokens;
    r.lim0 = r.kv - 1;
    r.listed = 1;
    r.tok0 = (int32_t)w.tok.size();
    int64_t t = 0;
    for (int i = 0; i < s->num_requests; t += s->requests[i++].num_queries)
      if (s->requests[i].prefix == p && shares(s->requests[i]))
        for (int j = 0; j < s->requests[i].num_queries; ++j) w.tok.push_back((int32_t)(t + j));
    r.ntok = (int32_t)w.tok.size() - r.tok0;
    const int32_t t0 = w.tok[(size_t)r.tok0];
    if (w.tok.back() - t0 == r.ntok - 1) {  // ascending and without gaps: no list needed
      w.tok.resize((size_t)r.tok0);
      r.listed = 0;
      r.tok0 = t0;
    }
    prefix_run[(size_t)p] = (int32_t)w.runs.size();
    w.runs.push_back(r);
  }
  std::vector<int32_t> own_run((size_t)s->num_requests, -1);
  int64_t tok = 0;
  for (int i = 0; i < s->num_requests; tok += s->requests[i++].num_queries) {
    const kamera_request& q = s->requests[i];
    if (q.num_queries == 0) continue;
    AttendRun r;
    std::memset(&r, 0, sizeof(r));
    if (q.prefix >= 0 && !shares(q)) {
      r.pg_a = tb.prefix[(size_t)q.prefix];
      r.slot_a = s->prefixes[q.prefix].slot0;
      r.len_a = s->prefixes[q.prefix].num_tokens;
    }
    r.pg_b = tb.request[(size_t)i];
    r.slot_b = q.slot0;
    r.kv = r.len_a + q.num_tokens;
    if (r.kv == 0 && shares(q)) continue;  // (no key at all: a run without keys writes the zeros)
    if (q.flags & KAMERA_REQUEST_ALL) {
      r.lim0 = r.kv - 1;
    } else {
      r.lim0 = r.len_a + q.num_tokens - q.num_queries;
      r.lstep = 1;
    }
    r.tok0 = (int32_t)tok;
    r.ntok = q.num_queries;
    r.direct = !shares(q);
    own_run[(size_t)i] = (int32_t)w.runs.size();
    w.runs.push_back(r);
  }
  const bool plain = kernel == ATTEND_PLAIN;
  const int64_t gran = plain ? 32 : 128, slots = plain ? 2048 : kernel == ATTEND_LATENT ? 256 : 512;
  // Tiles: the smallest that a run's rows fit, wide ones where they fit none.
  for (AttendRun& r : w.runs) {
    const int64_t rows = (int64_t)r.ntok * G;
    if (plain || rows <= tile_rows(kernel, TILE_NARROW)) r.tile = TILE_NARROW;
    else r.tile = kernel == ATTEND_HEADS && rows <= tile_rows(kernel, TILE_PAIRS) ? TILE_PAIRS : TILE_WIDE;
  }
  // Keys per item (a multiple of gran), for each class of tiles: the least estimate of the launch's
  // time. All classes share `slots` places; a class whose items are alike takes whole rounds of them
  // (8 heads of a 131072-key prefix in 69 ranges, 552 workgroups on 512 places: 137 us; in 64: 109 us).
  struct Class {
    int64_t longest = 0;
    double tiles = 0, keys = 0;
  } cls[3];
  for (const AttendRun& r : w.runs) {
    if (r.kv == 0) continue;
    const int64_t rows = (int64_t)r.ntok * G;
    Class& c = cls[r.tile];
    const double tiles = (double)ceil_div(rows, tile_rows(kernel, r.tile));
    c.longest = std::max<int64_t>(c.longest, r.kv);
    c.tiles += tiles;
    c.keys += tiles * r.kv;
  }
  double whole = 0;  // the launch's time if the places were always full and nothing split
  for (int k = 0; k < 3; ++k) whole += h.heads * (key_ns(kernel, k) * cls[k].keys + kStartNs * cls[k].tiles) / slots;
  int64_t chunk_of[3] = {gran, gran, gran};
  for (int k = 0; k < 3; ++k) {
    const Class& c = cls[k];
    const double per_key = key_ns(kernel, k);
    const bool alike = c.keys > 0.9 * c.tiles * c.longest;
    double best = 0;
    auto consider = [&](int64_t chunk) {
      double items = 0, parts = 0;
      for (const AttendRun& r : w.runs) {
        const int64_t rows = (int64_t)r.ntok * G, n = ceil_div(r.kv, chunk);
        if (r.tile != k) continue;
        items += (double)ceil_div(rows, tile_rows(kernel, k)) * n;
        if (n > 1 || !r.direct) parts += (double)rows * n;
      }
      items *= h.heads;
      const double one = kStartNs + per_key * std::min(chunk, c.longest), more = kStartNs * (items - c.tiles * h.heads) / slots;
      const double rounds = alike ? std::ceil(items / slots) * one : one * 5 / 4;
      const double ns = std::max(rounds, whole + more + (alike ? 0 : one / 4)) + kPartNs * h.dv * h.heads * parts;
      if (best == 0 || ns < best) {
        best = ns;
        chunk_of[k] = chunk;
      }
    };
    const int64_t lowest = (int64_t)round_up((size_t)std::max(gran, ceil_div(c.longest, kMaxSplits)), (size_t)gran);
    for (int64_t chunk = lowest;; chunk = (int64_t)round_up((size_t)(chunk + chunk / 3), (size_t)gran)) {
      consider(chunk);
      if (chunk >= c.longest) break;
    }
    for (int64_t round = 1; alike && round <= 4; ++round) {  // ranges that fill whole rounds
      const int64_t n = (int64_t)(round * slots / (c.tiles * h.heads));
      if (n > 0) consider(std::max(lowest, (int64_t)round_up((size_t)ceil_div(c.longest, n), (size_t)gran)));
    }
    for (int i = 0; i < fit.coarser && chunk_of[k] < c.longest; ++i) chunk_of[k] *= 2;
  }
  int32_t start[4] = {0, 0, 0, 0};  // each class's first item
  for (int c = 0; c < 3; ++c) {
    for (size_t k = 0; k < w.runs.size(); ++k) {
      AttendRun& r = w.runs[k];
      const int64_t rows = (int64_t)r.ntok * G;
      const int tile = tile_rows(kernel, c);
      if (r.tile != c) continue;
      const int64_t splits = std::max<int64_t>(ceil_div(r.kv, chunk_of[c]), 1);
      const int64_t chunk = (int64_t)round_up((size_t)std::max<int64_t>(ceil_div(r.kv, splits), 1), (size_t)gran);
      const int64_t n = std::max<int64_t>(ceil_div(r.kv, chunk), 1);
      r.splits = (int32_t)n;
      if (n > 1) {
        r.direct = 0;
        w.split = true;
      }
      if (!r.direct) {
        r.part0 = w.part_rows;
        w.part_rows += n * h.heads * rows;
      }
      for (int64_t row0 = 0; row0 < rows; row0 += tile) {
        const int64_t last = (std::min(row0 + tile, rows) - 1) / G;  // the tile's last token
        const int64_t end = std::min<int64_t>(r.kv, std::max<int64_t>(r.len_a - 1, r.lim0 + last * r.lstep) + 1);
        for (int64_t sp = 0; sp < n; ++sp) {
          AttendItem it;
          std::memset(&it, 0, sizeof(it));
          it.run = r;
          it.row0 = (int32_t)row0;
          it.kv0 = (int32_t)(sp * chunk);
          it.kv1 = (int32_t)std::max<int64_t>(it.kv0, std::min(end, (sp + 1) * chunk));
          it.split = (int32_t)sp;
          w.items.push_back(it);
        }
      }
    }
    // the longest first: the short ones fill the gaps at the end
    auto longer = [](const AttendItem& x, const AttendItem& y) { return x.kv1 - x.kv0 > y.kv1 - y.kv0; };
    if (!plain) std::stable_sort(w.items.begin() + start[c], w.items.end(), longer);
    start[c + 1] = (int32_t)w.items.size();
  }
  w.wide = start[1];
  w.pairs = start[2] - start[1];
  // tokens joined from parts
  std::vector<int32_t> listed((size_t)s->num_prefixes, 0);  // tokens of each prefix run so far
  auto part = [&](MergeToken& m, int slot, int run, int64_t j) {
    const AttendRun& r = w.runs[(size_t)run];
    m.part[slot] = r.part0;
    m.rows[slot] = (int32_t)((int64_t)r.ntok * G);
    m.row0[slot] = (int32_t)(j * G);
    m.splits[slot] = r.splits;
  };
  tok = 0;
  for (int i = 0; i < s->num_requests; tok += s->requests[i++].num_queries) {
    const kamera_request& q = s->requests[i];
    const int run = own_run[(size_t)i];
    if (run >= 0 && w.runs[(size_t)run].direct) continue;
    const bool sh = q.num_queries > 0 && shares(q);
    for (int j = 0; j < q.num_queries; ++j) {
      MergeToken m;
      std::memset(&m, 0, sizeof(m));
      m.token = (int32_t)(tok + j);
      if (sh) part(m, 0, prefix_run[(size_t)q.prefix], listed[(size_t)q.prefix]++);
      if (run >= 0) part(m, 1, run, j);
      w.max_parts = std::max(w.max_parts, m.splits[0] + m.splits[1]);
      w.merge.push_back(m);
    }
  }
}

// ------------------------------------------------------------------ workspace
struct Offsets {
  size_t pages, items, tok, merge, slots, pos, theta, upload, phase, ml, o, total;
};
Offsets carve(const kamera_layout* L, const kamera_step* s, const Counts& n, size_t items, size_t tok, size_t merge, int64_t part_rows) {
  Offsets f;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += round_up(bytes, kAlign);
    return here;
  };
  const bool append = s->flags & KAMERA_STEP_APPEND;
  const Shape h = shape_of(L, s->num_q_heads);
  f.pages = take((size_t)n.entries * 4);
  f.items = take(items * sizeof(AttendItem));
  f.tok = take(tok * 4);
  f.merge = take(merge * sizeof(MergeToken));
  f.slots = take(append ? (size_t)n.tokens * 8 : 0);
  f.pos = take(append && !s->positions ? (size_t)n.tokens * 4 : 0);
  f.theta = take(append ? (size_t)h.d_rot / 2 * 8 : 0);
  f.upload = at;
  f.phase = take(append ? (size_t)n.tokens * h.d_rot * 4 : 0);
  f.ml = take((size_t)part_rows * 8);
  f.o = take((size_t)part_rows * h.dv * 4);
  f.total = std::max<size_t>(at, kAlign);
  return f;
}
Offsets carve(const kamera_layout* L, const kamera_step* s, const Counts& n, const Work& w) {
  return carve(L, s, n, w.items.size(), w.tok.size(), w.merge.size(), w.part_rows);
}

// Bytes that a plan without ranges and sharing takes on any pool: it has no partial rows, and an item a
// tile, most of them in the kernel with the smallest tiles. Unlike the fastest plan's, they never grow
// when a request loses tokens or queries.
size_t least_bytes(const kamera_layout* L, const kamera_step* s, const Counts& n) {
  const int64_t group = shape_of(L, s->num_q_heads).group;
  size_t items = 0;
  if (s->flags & KAMERA_STEP_ATTEND)
    for (int i = 0; i < s->num_requests; ++i) items += (size_t)ceil_div(s->requests[i].num_queries * group, tile_rows(ATTEND_PLAIN, TILE_NARROW));
  return carve(L, s, n, items, 0, 0, 0).total;
}

void place_tables(const kamera_layout* L, const kamera_step* s, Tables& tb) {
  const int P = L->page_size;
  int64_t at = 0;
  tb.prefix.assign((size_t)s->num_prefixes, 0);
  tb.request.assign((size_t)s->num_requests, 0);
  for (int i = 0; i < s->num_prefixes; ++i) {
    tb.prefix[(size_t)i] = (int32_t)at;
    at += table_entries(s->prefixes[i].slot0, s->prefixes[i].num_tokens, P);
  }
  for (int i = 0; i < s->num_requests; ++i) {
    tb.request[(size_t)i] = (int32_t)at;
    at += table_entries(s->requests[i].slot0, s->requests[i].num_tokens, P);
  }
}

// Page ids inside the pool; appended slots distinct and outside every prefix.
kamera_status check_tables(const kamera_layout* L, const kamera_step* s, const kamera_pool* pool) {
  const int P = L->page_size;
  auto in_pool = [&](const char* what, int i, const int32_t* t, int64_t n) {
    for (int64_t k = 0; k < n; ++k)
      if (t[k] < 0 || t[k] >= pool->num_pages)
        return host_fail(KAMERA_E_PAGE, "%s %d: block_table[%lld] = %d outside [0, %d)", what, i, (long long)k, t[k],
                         pool->num_pages);
    return KAMERA_OK;
  };
  kamera_status st = KAMERA_OK;
  for (int i = 0; i < s->num_prefixes && st == KAMERA_OK; ++i)
    st = in_pool("prefix", i, s->prefixes[i].block_table, table_entries(s->prefixes[i].slot0, s->prefixes[i].num_tokens, P));
  for (int i = 0; i < s->num_requests && st == KAMERA_OK; ++i)
    st = in_pool("request", i, s->requests[i].block_table, table_entries(s->requests[i].slot0, s->requests[i].num_tokens, P));
  if (st != KAMERA_OK || !(s->flags & KAMERA_STEP_APPEND)) return st;
  struct Range {
    int32_t page, lo, hi, request;
  };
  thread_local std::vector<Range> ranges;
  ranges.clear();
  for (int i = 0; i < s->num_requests; ++i) {
    const kamera_request& r = s->requests[i];
    const int64_t lo = (int64_t)r.slot0 + r.num_tokens - r.num_queries, hi = (int64_t)r.slot0 + r.num_tokens;
    if (r.num_queries)
      for (int64_t k = lo / P; k * P < hi; ++k)
        ranges.push_back(Range{r.block_table[k], (int32_t)std::max<int64_t>(lo - k * P, 0),
                               (int32_t)std::min<int64_t>(hi - k * P, P), i});
  }
  std::sort(ranges.begin(), ranges.end(),
            [](const Range& a, const Range& b) { return a.page != b.page ? a.page < b.page : a.lo < b.lo; });
  for (size_t k = 1; k < ranges.size(); ++k)  // sorted by start: a clash anywhere shows between neighbours
    if (ranges[k].page == ranges[k - 1].page && ranges[k].lo < ranges[k - 1].hi)
      return host_fail(KAMERA_E_OVERLAP, "requests %d and %d both append to slot %d of page %d", ranges[k - 1].request,
                       ranges[k].request, ranges[k].lo, ranges[k].page);
  if (ranges.empty() || s->num_prefixes == 0) return KAMERA_OK;
  // prefixes may be long: mark the appended pages, look each prefix entry up
  thread_local std::vector<uint8_t> marked;
  if (marked.size() < (size_t)pool->num_pages) marked.resize((size_t)pool->num_pages, 0);
  for (const Range& r : ranges) marked[(size_t)r.page] = 1;
  for (int i = 0; i < s->num_prefixes && st == KAMERA_OK; ++i) {
    const kamera_prefix& p = s->prefixes[i];
    const int64_t n = table_entries(p.slot0, p.num_tokens, P);
    for (int64_t k = 0; k < n && st == KAMERA_OK; ++k) {
      if (!marked[(size_t)p.block_table[k]]) continue;
      const int64_t lo = std::max<int64_t>(p.slot0 - k * P, 0), hi = std::min<int64_t>((int64_t)p.slot0 + p.num_tokens - k * P, P);
      for (const Range& r : ranges)
        if (r.page == p.block_table[k] && r.lo < hi && lo < r.hi) {
          st = host_fail(KAMERA_E_OVERLAP, "request %d appends to page %d inside prefix %d", r.request, r.page, i);
          break;
        }
    }
  }
  for (const Range& r : ranges) marked[(size_t)r.page] = 0;
  return st;
}

kamera_status upload_step(const kamera_layout* L, const kamera_step* s, const kamera_pool* pool, void* ws,
                          size_t ws_bytes, hipStream_t stream, kamera_step_plan* plan) {
  Counts n;
  kamera_status st = check_step(L, s, n);
  if (st == KAMERA_OK) st = check_pool(L, pool);
  if (st == KAMERA_OK) st = check_tables(L, s, pool);
  if (st != KAMERA_OK) return st;
  const bool append = s->flags & KAMERA_STEP_APPEND, attend = s->flags & KAMERA_STEP_ATTEND;
  const int P = L->page_size;
  const Shape h = shape_of(L, s->num_q_heads);
  thread_local Tables tb;
  thread_local Work w;
  place_tables(L, s, tb);
  const int kernel = pick_kernel(L, pool);
  Fit fit;
  if (attend) plan_attention(L, s, tb, kernel, fit, w);
  else w = Work();
  Offsets f = carve(L, s, n, w);
  while ((s->flags & KAMERA_STEP_FIT) && f.total > ws_bytes && (w.split || w.shared)) {  // (each turn halves the partial rows, or ends the sharing)
    if (w.split) ++fit.coarser;
    else fit = Fit{0, false};
    plan_attention(L, s, tb, kernel, fit, w);
    f = carve(L, s, n, w);
  }
  st = check_workspace(ws, ws_bytes, f.total);
  if (st != KAMERA_OK) return st;
  // (the matrix-core kernels' workgroups lie along one dimension of the grid, which takes fewer than 2^32 threads)
  const int most = kernel == ATTEND_PLAIN ? 31 : kernel == ATTEND_HEADS ? 24 : 23;
  if ((int64_t)w.items.size() * h.heads >= (int64_t(1) << most)) return host_fail(KAMERA_E_SHAPE, "too many work items");

  thread_local std::vector<unsigned char> blob;
  blob.assign(f.upload, 0);
  int32_t* pages = reinterpret_cast<int32_t*>(blob.data() + f.pages);
  auto put = [&](int32_t at, const int32_t* t, int64_t entries) {
    if (entries) std::memcpy(pages + at, t, (size_t)entries * 4);
  };
  for (int i = 0; i < s->num_prefixes; ++i)
    put(tb.prefix[(size_t)i], s->prefixes[i].block_table, table_entries(s->prefixes[i].slot0, s->prefixes[i].num_tokens, P));
  for (int i = 0; i < s->num_requests; ++i)
    put(tb.request[(size_t)i], s->requests[i].block_table, table_entries(s->requests[i].slot0, s->requests[i].num_tokens, P));
  if (!w.items.empty()) std::memcpy(blob.data() + f.items, w.items.data(), w.items.size() * sizeof(AttendItem));
  if (!w.tok.empty()) std::memcpy(blob.data() + f.tok, w.tok.data(), w.tok.size() * 4);
  if (!w.merge.empty()) std::memcpy(blob.data() + f.merge, w.merge.data(), w.merge.size() * sizeof(MergeToken));
  if (append) {
    int64_t* slots = reinterpret_cast<int64_t*>(blob.data() + f.slots);
    int32_t* pos = reinterpret_cast<int32_t*>(blob.data() + f.pos);
    int64_t t = 0;
    for (int i = 0; i < s->num_requests; ++i) {
      const kamera_request& r = s->requests[i];
      for (int j = 0; j < r.num_queries; ++j, ++t) {
        const int64_t own = (int64_t)r.num_tokens - r.num_queries + j, at = r.slot0 + own;
        slots[t] = (int64_t)r.block_table[at / P] * P + at % P;
        if (!s->positions) pos[t] = (int32_t)(r.position0 + own);
      }
    }
    double* theta = reinterpret_cast<double*>(blob.data() + f.theta);
    for (int i = 0; i < h.d_rot / 2; ++i) theta[i] = std::pow(L->rope_base, -2.0 * i / h.d_rot);
  }

  StepArgs a;
  std::memset(&a, 0, sizeof(a));
  char* base = static_cast<char*>(ws);
  a.k_pool = static_cast<uint16_t*>(pool->k_pool);
  a.v_pool = static_cast<uint16_t*>(L->family == KAMERA_GQA ? pool->v_pool : pool->k_pool);
  a.row = row_width(L);
  a.layer_stride = pool->layer_stride ? pool->layer_stride : (int64_t)pool->num_pages * P * a.row;
  a.pages = reinterpret_cast<const int32_t*>(base + f.pages);
  a.items = reinterpret_cast<const AttendItem*>(base + f.items);
  a.tok = reinterpret_cast<const int32_t*>(base + f.tok);
  a.merge = reinterpret_cast<const MergeToken*>(base + f.merge);
  a.part_o = reinterpret_cast<float*>(base + f.o);
  a.part_ml = reinterpret_cast<float2*>(base + f.ml);
  a.slots = reinterpret_cast<const int64_t*>(base + f.slots);
  a.phase = reinterpret_cast<float*>(base + f.phase);
  a.pos = s->positions ? nullptr : reinterpret_cast<const int32_t*>(base + f.pos);
  a.positions = s->positions;
  a.theta = reinterpret_cast<const double*>(base + f.theta);
  a.family = L->family;
  a.dtype = L->dtype;
  a.pairing = L->pairing;
  a.heads = h.heads;
  a.group = h.group;
  a.dk = h.dk;
  a.dv = h.dv;
  a.num_q_heads = s->num_q_heads;
  a.d_rot = h.d_rot;
  a.latent = L->family == KAMERA_MLA ? L->latent_dim : 0;
  a.page_size = P;
  a.page_shift = (P & (P - 1)) == 0 ? __builtin_ctz((unsigned)P) : -1;
  // with b = ceil(log2 P): floor(2^(31 + b) / P) + 1 exceeds 2^(31 + b) / P by at most 2^b / (P 2^b),
  // which the 31 bits of a slot cannot raise to a whole
  a.page_bits = 31;
  while ((int64_t(1) << (a.page_bits - 31)) < P) ++a.page_bits;
  a.page_magic = (uint32_t)((uint64_t(1) << a.page_bits) / (uint64_t)P + 1);
  a.num_items = (int32_t)w.items.size();
  a.num_merge = (int32_t)w.merge.size();
  a.num_tokens = (int32_t)n.tokens;
  for (int k = 0; k < 3; ++k) a.mrope[k] = L->mrope_section[k];
  a.kernel = kernel;
  a.num_wide = w.wide;
  a.num_pairs = w.pairs;
  a.max_parts = w.max_parts;

  if (n.tokens > 0) {
    st = host_stage(blob.data(), f.upload, ws, stream);
    if (st != KAMERA_OK) return st;
    if (append) {
      const hipError_t e = launch_step_phase(a, stream);
      if (e != hipSuccess) return host_fail(KAMERA_E_HIP, "phase table launch failed: %s", hipGetErrorString(e));
    }
  }
  std::memset(plan, 0, sizeof(*plan));
  plan->workspace = ws;
  plan->num_tokens = (int32_t)n.tokens;
  plan->num_layers = L->num_layers;
  plan->flags = s->flags;
  std::memcpy(plan->detail, &a, sizeof(a));
  return KAMERA_OK;
}

kamera_status check_launch(const kamera_step_plan* plan, int32_t layer, uint32_t flag, StepArgs& a) {
  if (!plan) return host_fail(KAMERA_E_NULL, "plan is NULL");
  if (!plan->workspace) return host_fail(KAMERA_E_WORKSPACE, "plan has no workspace");
  if (!(plan->flags & flag)) return host_fail(KAMERA_E_UNSUPPORTED, "the step was not uploaded for this call (flags 0x%x)", plan->flags);
  if (layer < 0 || layer >= plan->num_layers)
    return host_fail(KAMERA_E_SHAPE, "layer %d outside [0, %d)", layer, plan->num_layers);
  std::memcpy(&a, plan->detail, sizeof(a));
  return KAMERA_OK;
}

kamera_status check_rows(const char* what, const void* p, int64_t& stride, int64_t width, size_t es) {
  if (!p) return host_fail(KAMERA_E_NULL, "%s is NULL", what);
  if (!aligned(p, es)) return host_fail(KAMERA_E_ALIGN, "%s must be aligned to %zu bytes", what, es);
  if (stride == 0) stride = width;
  if (stride < width) return host_fail(KAMERA_E_SHAPE, "%s: stride %lld below the row's %lld", what, (long long)stride, (long long)width);
  return KAMERA_OK;
}

// ------------------------------------------------------------------ page copies
struct CopyPlan {
  std::vector<int32_t> chain;
  std::vector<PageCopy> copies;
  int32_t rings = 0;        // the last chains: see CopyArgs
  bool independent = true;  // every chain is one copy
};

// Orders the copies so that each page is read for the last time before it is written. A copy
// whose pages no other copy writes or reads stands alone; the others form groups joined by
// the pages they share, each carried out in order, a cycle through a saved page. A long group in which
// each page is read once (one path or one cycle) is left in the order of its pages as a ring.
void order_copies(const int32_t* src, const int32_t* dst, int32_t n, int32_t num_pages, CopyPlan& out) {
  thread_local std::vector<int32_t> by_dst, readers, bound, up, size, start;
  thread_local std::vector<uint8_t> done, single;
  struct Entry {
    int32_t group;
    PageCopy copy;
  };
  thread_local std::vector<Entry> order;
  out.chain.clear();
  out.copies.clear();
  out.rings = 0;
  out.independent = true;
  by_dst.assign((size_t)num_pages, -1);
  readers.assign((size_t)num_pages, 0);
  for (int32_t i = 0; i < n; ++i) {
    if (src[i] == dst[i]) continue;
    by_dst[(size_t)dst[i]] = i;
    ++readers[(size_t)src[i]];
  }
  bound.clear();  // copies that share a page with another's destination
  for (int32_t i = 0; i < n; ++i) {
    if (src[i] == dst[i]) continue;
    if (readers[(size_t)dst[i]] == 0 && by_dst[(size_t)src[i]] < 0) {
      out.chain.push_back((int32_t)out.copies.size());
      out.copies.push_back(PageCopy{src[i], dst[i]});
    } else {
      bound.push_back(i);
    }
  }
  if (!bound.empty()) {
    out.independent = false;
    // groups: copies connected through a page that one writes and another reads
    up.resize((size_t)n);
    for (int32_t i = 0; i < n; ++i) up[(size_t)i] = i;
    auto root = [&](int32_t i) {
      while (up[(size_t)i] != i) i = up[(size_t)i] = up[(size_t)up[(size_t)i]];
      return i;
    };
    for (int32_t i : bound)
      if (by_dst[(size_t)src[i]] >= 0) up[(size_t)root(i)] = root(by_dst[(size_t)src[i]]);
    done.assign((size_t)n, 0);
    single.assign((size_t)n, 1);  // each page of the group is read once (and, below, there are enough of them)
    size.assign((size_t)n, 0);    // its copies
    for (int32_t i : bound) {
      const int32_t g = root(i);
      ++size[(size_t)g];
      if (readers[(size_t)src[i]] > 1) single[(size_t)g] = 0;
    }
    for (int32_t g = 0; g < n; ++g) single[(size_t)g] = single[(size_t)g] && size[(size_t)g] >= kLongChain;
    auto ring = [&](int32_t g) { return single[(size_t)g] != 0; };
    order.clear();
    for (int32_t i : bound)  // from pages nobody reads: write, then the page read becomes free to be written
      for (int32_t j = i; j >= 0 && !done[(size_t)j] && readers[(size_t)dst[j]] == 0;) {
        done[(size_t)j] = 1;
        order.push_back(Entry{root(j), PageCopy{src[j], dst[j]}});
        j = --readers[(size_t)src[j]] == 0 ? by_dst[(size_t)src[j]] : -1;
      }
    for (int32_t i : bound) {  // what is left are cycles
      if (done[(size_t)i]) continue;
      const int32_t g = root(i);
      if (!ring(g)) {
        order.push_back(Entry{g, PageCopy{dst[i], -1}});  // keep the page written first
        ++size[(size_t)g];
      }
      for (int32_t j = i; !done[(size_t)j]; j = by_dst[(size_t)src[j]]) {
        done[(size_t)j] = 1;
        order.push_back(Entry{g, PageCopy{src[j] == dst[i] && !ring(g) ? -1 : src[j], dst[j]}});
      }
    }
    // group after group, the rings last
    start.assign((size_t)n, 0);
    int32_t at = (int32_t)out.copies.size();
    for (int rings = 0; rings < 2; ++rings)
      for (int32_t g = 0; g < n; ++g) {
        if (size[(size_t)g] == 0 || ring(g) != (rings == 1)) continue;
        out.chain.push_back(at);
        start[(size_t)g] = at;
        at += size[(size_t)g];
        out.rings += rings;
      }
    out.copies.resize((size_t)at);
    for (const Entry& e : order) out.copies[(size_t)start[(size_t)e.group]++] = e.copy;
  }
  out.chain.push_back((int32_t)out.copies.size());
}

// chain starts, then the copies: a cycle adds one entry to its copies
size_t copies_bytes(int64_t n) {
  return round_up((size_t)(n + 1) * 4, kAlign) + round_up((size_t)(n + n / 2) * sizeof(PageCopy), kAlign);
}

kamera_status enqueue_copies(const kamera_layout* L, const kamera_pool* pool, const int32_t* src, const int32_t* dst,
                             int32_t n, void* ws, hipStream_t stream) {
  thread_local CopyPlan p;
  order_copies(src, dst, n, pool->num_pages, p);
  if (p.copies.empty()) return KAMERA_OK;
  CopyArgs a;
  std::memset(&a, 0, sizeof(a));
  const size_t es = elem_bytes(L);
  a.pool[0] = static_cast<char*>(pool->k_pool);
  a.pool[1] = static_cast<char*>(pool->v_pool);
  a.tensors = L->family == KAMERA_GQA ? 2 : 1;
  a.layers = L->num_layers;
  a.page_bytes = (int64_t)L->page_size * row_width(L) * (int64_t)es;
  a.layer_bytes = pool->layer_stride ? pool->layer_stride * (int64_t)es : (int64_t)pool->num_pages * a.page_bytes;
  a.chains = (int32_t)p.chain.size() - 1 - p.rings;
  a.rings = p.rings;
  auto fits = [&](int unit) {
    return a.page_bytes % unit == 0 && a.layer_bytes % unit == 0 && aligned(a.pool[0], (size_t)unit) &&
           (a.tensors == 1 || aligned(a.pool[1], (size_t)unit));
  };
  a.unit = fits(16) ? 16 : (fits(4) ? 4 : 2);
  hipError_t e;
  if (p.independent && a.chains <= kInlineCopies) {
    InlineCopies in;
    std::memcpy(in.c, p.copies.data(), p.copies.size() * sizeof(PageCopy));
    e = launch_copy_pages(a, &in, stream);
  } else {
    const size_t at = round_up(p.chain.size() * 4, kAlign);
    const size_t bytes = at + round_up(p.copies.size() * sizeof(PageCopy), kAlign);
    thread_local std::vector<unsigned char> blob;
    blob.assign(bytes, 0);
    std::memcpy(blob.data(), p.chain.data(), p.chain.size() * 4);
    std::memcpy(blob.data() + at, p.copies.data(), p.copies.size() * sizeof(PageCopy));
    const kamera_status st = host_stage(blob.data(), bytes, ws, stream);
    if (st != KAMERA_OK) return st;
    a.chain = p.independent ? nullptr : static_cast<const int32_t*>(ws);
    a.copies = reinterpret_cast<const PageCopy*>(static_cast<char*>(ws) + at);
    e = launch_copy_pages(a, nullptr, stream);
  }
  if (e != hipSuccess) return host_fail(KAMERA_E_HIP, "page copy launch failed: %s", hipGetErrorString(e));
  return KAMERA_OK;
}

// No C++ exception (host memory running out) leaves a C entry.
template <typename F>
kamera_status guarded(F f) {
  host_clear_error();
  try {
    return f();
  } catch (const std::bad_alloc&) {
    return host_fail(KAMERA_E_SHAPE, "out of host memory");
  } catch (...) {
    return host_fail(KAMERA_E_SHAPE, "unexpected host error");
  }
}

}  // namespace

extern "C" {

size_t kamera_step_workspace_bytes(const kamera_layout* layout, const kamera_step* step) {
  size_t bytes = 0;
  (void)guarded([&] {
    Counts n;
    kamera_status st = check_step(layout, step, n);
    if (st != KAMERA_OK) return st;
    Tables tb;
    Work w;
    place_tables(layout, step, tb);
    const bool attend = step->flags & KAMERA_STEP_ATTEND;
    // the pool's alignment decides between the kernels: enough for either
    if (attend) plan_attention(layout, step, tb, ATTEND_PLAIN, Fit{}, w);
    size_t need = carve(layout, step, n, w).total;
    if (step->flags & KAMERA_STEP_FIT) need = std::max(need, least_bytes(layout, step, n));
    if (attend && matrix_kernel(layout) != ATTEND_PLAIN) {
      plan_attention(layout, step, tb, matrix_kernel(layout), Fit{}, w);
      need = std::max(need, carve(layout, step, n, w).total);
    }
    bytes = need;
    return KAMERA_OK;
  });
  return bytes;
}

kamera_status kamera_step_upload(const kamera_layout* layout, const kamera_step* step, const kamera_pool* pool,
                                 void* workspace, size_t workspace_bytes, void* stream, kamera_step_plan* plan) {
  return guarded([&] {
    if (!plan) return host_fail(KAMERA_E_NULL, "plan is NULL");
    return upload_step(layout, step, pool, workspace, workspace_bytes, (hipStream_t)stream, plan);
  });
}

kamera_status kamera_step_append(const kamera_step_plan* plan, int32_t layer, const kamera_append_rows* rows,
                                 void* stream) {
  return guarded([&] {
    StepArgs a;
    kamera_status st = check_launch(plan, layer, KAMERA_STEP_APPEND, a);
    if (st != KAMERA_OK) return st;
    if (!rows) return host_fail(KAMERA_E_NULL, "rows is NULL");
    kamera_append_rows r = *rows;
    const size_t es = a.dtype == KAMERA_BF16 ? 2 : 4;
    const int64_t qw = (int64_t)a.num_q_heads * a.dk;
    if (r.reserved) return host_fail(KAMERA_E_SHAPE, "rows.reserved must be 0");
    if (!(r.eps >= 0.0f) || !std::isfinite(r.eps)) return host_fail(KAMERA_E_SHAPE, "eps must be >= 0 and finite");
    if (plan->num_tokens == 0) return KAMERA_OK;
    if ((r.q != nullptr) != (r.q_out != nullptr)) return host_fail(KAMERA_E_NULL, "q and q_out go together");
    if (r.q && a.num_q_heads == 0) return host_fail(KAMERA_E_SHAPE, "the step has no query heads");
    if (r.q) {
      if ((st = check_rows("q", r.q, r.q_stride, qw, es)) != KAMERA_OK) return st;
      if ((st = check_rows("q_out", r.q_out, r.q_out_stride, qw, es)) != KAMERA_OK) return st;
      if (r.q == r.q_out && r.q_stride != r.q_out_stride)
        return host_fail(KAMERA_E_SHAPE, "in place, q and q_out have one stride");
    }
    if ((st = check_rows("k", r.k, r.k_stride, a.row, es)) != KAMERA_OK) return st;
    if (a.family == KAMERA_GQA && (st = check_rows("v", r.v, r.v_stride, a.row, es)) != KAMERA_OK) return st;
    if (a.family == KAMERA_MLA && r.q_weight) return host_fail(KAMERA_E_UNSUPPORTED, "MLA queries carry no norm here");
    if (a.family == KAMERA_MLA && r.k_weight && a.latent == 0) return host_fail(KAMERA_E_SHAPE, "k_weight without a latent");
    if ((r.q_weight && !aligned(r.q_weight, es)) || (r.k_weight && !aligned(r.k_weight, es)))
      return host_fail(KAMERA_E_ALIGN, "weights must be aligned to %zu bytes", es);
    const hipError_t e = launch_step_append(a, layer, r, (hipStream_t)stream);
    if (e != hipSuccess) return host_fail(KAMERA_E_HIP, "append launch failed: %s", hipGetErrorString(e));
    return KAMERA_OK;
  });
}

kamera_status kamera_step_attend(const kamera_step_plan* plan, int32_t layer, const void* q, int64_t q_stride,
                                 void* out, int64_t out_stride, float* lse, float scale, void* stream) {
  return guarded([&] {
    StepArgs a;
    kamera_status st = check_launch(plan, layer, KAMERA_STEP_ATTEND, a);
    if (st != KAMERA_OK) return st;
    const size_t es = a.dtype == KAMERA_BF16 ? 2 : 4;
    if (!std::isfinite(scale)) return host_fail(KAMERA_E_SHAPE, "scale must be finite");
    if (plan->num_tokens == 0) return KAMERA_OK;
    if ((st = check_rows("q", q, q_stride, (int64_t)a.num_q_heads * a.dk, es)) != KAMERA_OK) return st;
    if ((st = check_rows("out", out, out_stride, (int64_t)a.num_q_heads * a.dv, es)) != KAMERA_OK) return st;
    if (lse && !aligned(lse, 4)) return host_fail(KAMERA_E_ALIGN, "lse must be 4-byte aligned");
    const hipError_t e = launch_step_attend(a, layer, q, q_stride, out, out_stride, lse, scale, (hipStream_t)stream);
    if (e != hipSuccess) return host_fail(KAMERA_E_HIP, "attention launch failed: %s", hipGetErrorString(e));
    return KAMERA_OK;
  });
}

size_t kamera_copy_pages_workspace_bytes(int32_t num_copies) { return num_copies < 0 ? 0 : copies_bytes(num_copies); }

kamera_status kamera_copy_pages(const kamera_layout* layout, const kamera_pool* pool, const int32_t* src,
                                const int32_t* dst, int32_t num_copies, void* workspace, size_t workspace_bytes,
                                void* stream) {
  return guarded([&] {
    kamera_status st = host_check_layout(layout);
    if (st == KAMERA_OK) st = check_pool(layout, pool);
    if (st != KAMERA_OK) return st;
    if (num_copies < 0) return host_fail(KAMERA_E_SHAPE, "num_copies < 0");
    if (num_copies && (!src || !dst)) return host_fail(KAMERA_E_NULL, "src or dst is NULL");
    std::vector<uint8_t> written((size_t)pool->num_pages, 0);
    for (int32_t i = 0; i < num_copies; ++i) {
      if (src[i] < 0 || src[i] >= pool->num_pages || dst[i] < 0 || dst[i] >= pool->num_pages)
        return host_fail(KAMERA_E_PAGE, "copy %d: page %d to %d outside [0, %d)", i, src[i], dst[i], pool->num_pages);
      if (written[(size_t)dst[i]]) return host_fail(KAMERA_E_OVERLAP, "copy %d: page %d is written twice", i, dst[i]);
      written[(size_t)dst[i]] = 1;
    }
    st = check_workspace(workspace, workspace_bytes, copies_bytes(num_copies));
    if (st != KAMERA_OK) return st;
    return enqueue_copies(layout, pool, src, dst, num_copies, workspace, (hipStream_t)stream);
  });
}

kamera_status kamera_compact_pages(const kamera_layout* layout, const kamera_pool* pool, int32_t* const* tables,
                                   const int32_t* lengths, int32_t num_tables, int32_t* num_live, void* workspace,
                                   size_t workspace_bytes, void* stream) {
  return guarded([&] {
    kamera_status st = host_check_layout(layout);
    if (st == KAMERA_OK) st = check_pool(layout, pool);
    if (st != KAMERA_OK) return st;
    if (num_tables < 0) return host_fail(KAMERA_E_SHAPE, "num_tables < 0");
    if (!num_live || (num_tables && (!tables || !lengths))) return host_fail(KAMERA_E_NULL, "tables, lengths or num_live is NULL");
    std::vector<int32_t> to((size_t)pool->num_pages, -1);  // where a live page goes
    int32_t live = 0;
    for (int32_t i = 0; i < num_tables; ++i) {
      if (lengths[i] < 0) return host_fail(KAMERA_E_SHAPE, "table %d: negative length", i);
      if (lengths[i] && !tables[i]) return host_fail(KAMERA_E_NULL, "table %d is NULL", i);
      for (int32_t k = 0; k < lengths[i]; ++k) {
        const int32_t p = tables[i][k];
        if (p < 0 || p >= pool->num_pages)
          return host_fail(KAMERA_E_PAGE, "table %d: entry %d = %d outside [0, %d)", i, k, p, pool->num_pages);
        if (to[(size_t)p] < 0) {
          to[(size_t)p] = p;
          ++live;
        }
      }
    }
    std::vector<int32_t> src, dst;
    for (int32_t p = live, hole = 0; p < pool->num_pages; ++p) {
      if (to[(size_t)p] < 0) continue;
      while (to[(size_t)hole] >= 0) ++hole;  // as many holes below `live` as live pages from it on
      src.push_back(p);
      dst.push_back(hole);
      to[(size_t)p] = hole;
      to[(size_t)hole] = hole;  // entries reached through two of the tables are rewritten twice: the second time is no change
      ++hole;
    }
    const int32_t n = (int32_t)src.size();
    st = check_workspace(workspace, workspace_bytes, copies_bytes(n));
    if (st == KAMERA_OK) st = enqueue_copies(layout, pool, src.data(), dst.data(), n, workspace, (hipStream_t)stream);
    if (st != KAMERA_OK) return st;
    for (int32_t i = 0; i < num_tables; ++i)
      for (int32_t k = 0; k < lengths[i]; ++k) tables[i][k] = to[(size_t)tables[i][k]];
    *num_live = live;
    return KAMERA_OK;
  });
}

}  // extern "C"
