// The serving step's host part against host-side stand-ins for its kernels (no GPU): every
// query row meets every key it sees exactly once and no other, partial rows are written and
// joined once, appended slots and page copies are what the interface says. Random steps and
// copy lists; exits 0 when all hold.
#include <algorithm>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
#include <random>
#include <vector>

#include "kamera_step_desc.h"

using namespace kamera;

static char g_error[512];
#define CHECK(c)                                                                    \
  do {                                                                              \
    if (!(c)) {                                                                     \
      std::printf("%s:%d: %s failed (%s)\n", __FILE__, __LINE__, #c, g_error);      \
      std::exit(1);                                                                 \
    }                                                                               \
  } while (0)

// ------------------------------------------------------------------ stand-ins
namespace {
struct Seen {  // what the step under test should come to
  const kamera_step* step;
  const kamera_layout* lay;
  std::vector<std::map<int64_t, int>> keys;  // per query token: key number (prefix first) -> times met by head 0, group 0
};
Seen* g_seen;

int64_t pool_slot(const StepArgs& a, int pg, int slot) {
  CHECK(slot >= 0);
  return (int64_t)a.pages[pg + slot / a.page_size] * a.page_size + slot % a.page_size;
}
}  // namespace

namespace kamera {
kamera_status host_fail(kamera_status st, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_error, sizeof(g_error), fmt, ap);
  va_end(ap);
  return st;
}
void host_clear_error() { g_error[0] = 0; }
kamera_status host_check_layout(const kamera_layout* L) { return L ? KAMERA_OK : KAMERA_E_NULL; }
kamera_status host_stage(const void* src, size_t bytes, void* dst, hipStream_t) {
  CHECK(bytes % 16 == 0);
  std::memcpy(dst, src, bytes);
  return KAMERA_OK;
}
hipError_t launch_step_phase(const StepArgs&, hipStream_t) { return hipSuccess; }

hipError_t launch_step_append(const StepArgs& a, int, const kamera_append_rows&, hipStream_t) {
  int64_t t = 0;
  for (int i = 0; i < g_seen->step->num_requests; ++i) {
    const kamera_request& r = g_seen->step->requests[i];
    for (int j = 0; j < r.num_queries; ++j, ++t) {
      const int64_t own = r.num_tokens - r.num_queries + j, at = r.slot0 + own;
      CHECK(a.slots[t] == (int64_t)r.block_table[at / a.page_size] * a.page_size + at % a.page_size);
      CHECK(a.pos && a.pos[t] == r.position0 + own);
    }
  }
  return hipSuccess;
}

// Walks the items as the kernels do; marks which partial rows exist and which keys each token met.
hipError_t launch_step_attend(const StepArgs& a, int, const void*, int64_t, void*, int64_t, float*, float, hipStream_t) {
  const kamera_step* s = g_seen->step;
  std::map<int64_t, int> part;      // partial row -> times written (head 0)
  std::map<int64_t, int> direct;    // (token, g) -> times written
  std::map<int64_t, std::vector<int64_t>> part_keys;  // partial row -> pool slots met
  std::vector<std::vector<int64_t>> met((size_t)a.num_tokens);
  for (int i = 0; i < a.num_items; ++i) {
    const AttendItem& it = a.items[i];
    const AttendRun& run = it.run;
    const int64_t rows = (int64_t)run.ntok * a.group;
    const int tile = tile_rows(a.kernel, run.tile);
    const int cls = i < a.num_wide ? TILE_WIDE : i < a.num_wide + a.num_pairs ? TILE_PAIRS : TILE_NARROW;
    CHECK(run.tile == cls);
    CHECK(it.row0 >= 0 && it.row0 < rows && it.kv0 >= 0 && it.kv1 <= run.kv && it.split < run.splits);
    for (int64_t row = it.row0; row < std::min<int64_t>(it.row0 + tile, rows); ++row) {
      const int64_t j = row / a.group, g = row % a.group;
      const int token = run.listed ? a.tok[run.tok0 + j] : (int)(run.tok0 + j);
      CHECK(token >= 0 && token < a.num_tokens);
      const int64_t end = std::min<int64_t>(it.kv1, std::max<int64_t>(run.len_a - 1, run.lim0 + j * run.lstep) + 1);
      std::vector<int64_t> slots;
      for (int64_t t = it.kv0; t < end; ++t)
        slots.push_back(t < run.len_a ? pool_slot(a, run.pg_a, run.slot_a + (int)t)
                                      : pool_slot(a, run.pg_b, run.slot_b + (int)(t - run.len_a)));
      if (run.direct) {
        CHECK(run.splits == 1 && direct[(int64_t)token * a.group + g]++ == 0);
        if (g == 0) met[(size_t)token].insert(met[(size_t)token].end(), slots.begin(), slots.end());
      } else {
        const int64_t pr = run.part0 + ((int64_t)it.split * a.heads + 0) * rows + row;
        CHECK(part[pr]++ == 0);
        part_keys[pr] = slots;
      }
    }
  }
  for (int i = 0; i < a.num_merge; ++i) {
    const MergeToken& m = a.merge[i];
    CHECK(m.token >= 0 && m.token < a.num_tokens);
    for (int g = 0; g < a.group; ++g) {
      CHECK(direct[(int64_t)m.token * a.group + g]++ == 0);
      for (int k = 0; k < 2; ++k)
        for (int sp = 0; sp < m.splits[k]; ++sp) {
          const int64_t pr = m.part[k] + ((int64_t)sp * a.heads + 0) * m.rows[k] + m.row0[k] + g;
          CHECK(part[pr]++ == 1);  // written once, joined once
          if (g == 0) met[(size_t)m.token].insert(met[(size_t)m.token].end(), part_keys[pr].begin(), part_keys[pr].end());
        }
    }
  }
  for (const auto& p : part) CHECK(p.second == 2);
  CHECK((int64_t)direct.size() == (int64_t)a.num_tokens * a.group);
  int64_t token = 0;
  const int P = a.page_size;
  for (int i = 0; i < s->num_requests; ++i) {
    const kamera_request& r = s->requests[i];
    for (int j = 0; j < r.num_queries; ++j, ++token) {
      std::vector<int64_t> want;
      auto add = [&](const int32_t* table, int slot0, int64_t n) {
        for (int64_t t = 0; t < n; ++t) want.push_back((int64_t)table[(slot0 + t) / P] * P + (slot0 + t) % P);
      };
      if (r.prefix >= 0) add(s->prefixes[r.prefix].block_table, s->prefixes[r.prefix].slot0, s->prefixes[r.prefix].num_tokens);
      const int64_t own = (r.flags & KAMERA_REQUEST_ALL) ? r.num_tokens : (int64_t)r.num_tokens - r.num_queries + j + 1;
      add(r.block_table, r.slot0, std::max<int64_t>(own, 0));
      std::sort(want.begin(), want.end());
      std::sort(met[(size_t)token].begin(), met[(size_t)token].end());
      CHECK(want == met[(size_t)token]);
    }
  }
  return hipSuccess;
}

hipError_t launch_copy_pages(const CopyArgs& a, const InlineCopies* in, hipStream_t) {
  CHECK(a.page_bytes % a.unit == 0);
  for (int tensor = 0; tensor < a.tensors; ++tensor)
    for (int layer = 0; layer < a.layers; ++layer) {
      char* base = a.pool[tensor] + layer * a.layer_bytes;
      for (int chain = a.chains - 1; chain >= 0; --chain) {  // chains do not depend on each other's order
        std::vector<char> kept((size_t)a.page_bytes), x((size_t)a.page_bytes);
        const int c0 = a.chain ? a.chain[chain] : chain, c1 = a.chain ? a.chain[chain + 1] : chain + 1;
        CHECK(!(in && a.chain));
        for (int c = c0; c < c1; ++c) {
          const PageCopy p = in ? in->c[c] : a.copies[c];
          if (p.src < 0) x = kept;
          else std::memcpy(x.data(), base + p.src * a.page_bytes, (size_t)a.page_bytes);
          if (p.dst < 0) kept = x;
          else std::memcpy(base + p.dst * a.page_bytes, x.data(), (size_t)a.page_bytes);
        }
      }
      for (int ring = a.chains; ring < a.chains + a.rings; ++ring) {  // as a list, the first page written kept for the last
        const int c0 = a.chain[ring], c1 = a.chain[ring + 1];
        CHECK(c1 - c0 >= kLongChain);
        std::vector<char> last(base + a.copies[c1 - 1].src * a.page_bytes, base + (a.copies[c1 - 1].src + 1) * a.page_bytes);
        for (int c = c0; c < c1; ++c) {
          CHECK(a.copies[c].src >= 0 && a.copies[c].dst >= 0 && (c + 1 == c1 || a.copies[c].src == a.copies[c + 1].dst));
          std::memcpy(base + a.copies[c].dst * a.page_bytes, c + 1 == c1 ? last.data() : base + a.copies[c].src * a.page_bytes, (size_t)a.page_bytes);
        }
      }
    }
  return hipSuccess;
}
}  // namespace kamera

// ------------------------------------------------------------------ random trials
namespace {
typedef std::mt19937_64 Rng;
int64_t draw(Rng& r, int64_t lo, int64_t hi) { return std::uniform_int_distribution<int64_t>(lo, hi)(r); }

struct Buffer {  // 256-byte aligned, exactly `bytes` long for the address sanitizer
  void* p;
  explicit Buffer(size_t bytes) : p(aligned_alloc(256, (bytes + 255) / 256 * 256)) {}
  ~Buffer() { free(p); }
};

void one_step(Rng& r) {
  kamera_layout L;
  std::memset(&L, 0, sizeof(L));
  L.family = draw(r, 0, 3) == 0 ? KAMERA_MLA : KAMERA_GQA;
  L.dtype = draw(r, 0, 2) == 0 ? KAMERA_F32 : KAMERA_BF16;
  L.num_layers = 1;
  const int dims[] = {64, 128, 80, 10};
  L.num_kv_heads = (int)draw(r, 1, 8);
  L.head_dim = dims[draw(r, 0, 3)];
  L.latent_dim = draw(r, 0, 1) ? 512 : 20;
  L.rope_dim = L.latent_dim == 512 ? 64 : 6;
  const int pages[] = {1, 3, 16, 64};
  L.page_size = pages[draw(r, 0, 3)];
  L.rope_base = 1e4;
  const int groups[] = {1, 2, 4, 7, 16, 33};
  const int group = groups[draw(r, 0, 5)];
  kamera_step s;
  std::memset(&s, 0, sizeof(s));
  s.num_q_heads = (L.family == KAMERA_GQA ? L.num_kv_heads : 1) * group;
  s.num_prefixes = (int)draw(r, 0, 3);
  s.num_requests = (int)draw(r, 0, 12);
  std::vector<kamera_prefix> pre((size_t)s.num_prefixes);
  std::vector<kamera_request> req((size_t)s.num_requests);
  std::vector<std::vector<int32_t>> tables;
  int32_t next = 0;
  auto table = [&](int slot0, int64_t n) {
    std::vector<int32_t> t((size_t)(n ? (slot0 + n + L.page_size - 1) / L.page_size : 0));
    for (int32_t& x : t) x = next++;
    tables.push_back(t);
  };
  const int64_t longest = draw(r, 0, 3) == 0 ? 5000 : 200;
  for (kamera_prefix& p : pre) {
    p.slot0 = (int)draw(r, 0, L.page_size - 1);
    p.num_tokens = (int)(draw(r, 0, 4) ? draw(r, 1, longest) : 0);
    table(p.slot0, p.num_tokens);
  }
  const bool append = draw(r, 0, 1);
  for (kamera_request& q : req) {
    std::memset(&q, 0, sizeof(q));
    q.slot0 = (int)draw(r, 0, L.page_size - 1);
    q.num_tokens = (int)(draw(r, 0, 6) ? draw(r, 1, longest) : 0);
    q.num_queries = (int)(draw(r, 0, 3) ? draw(r, 0, 3) : draw(r, 0, 150));
    if (append) q.num_queries = std::min(q.num_queries, q.num_tokens);
    q.prefix = (int)draw(r, -1, s.num_prefixes - 1);
    q.flags = draw(r, 0, 4) == 0 ? KAMERA_REQUEST_ALL : 0;
    q.position0 = draw(r, -100, 100);
    table(q.slot0, q.num_tokens);
  }
  std::vector<int32_t> order((size_t)std::max(next, 1));
  for (size_t i = 0; i < order.size(); ++i) order[i] = (int32_t)i;
  std::shuffle(order.begin(), order.end(), r);
  for (auto& t : tables)
    for (int32_t& x : t) x = order[(size_t)x];
  for (size_t i = 0; i < pre.size(); ++i) pre[i].block_table = tables[i].data();
  for (size_t i = 0; i < req.size(); ++i) req[i].block_table = tables[pre.size() + i].data();
  s.requests = req.data();
  s.prefixes = pre.data();
  s.flags = KAMERA_STEP_ATTEND | (append ? KAMERA_STEP_APPEND : 0);
  kamera_pool pool;
  std::memset(&pool, 0, sizeof(pool));
  char* fake = reinterpret_cast<char*>(uintptr_t(1) << 40);  // never read
  pool.k_pool = fake + (draw(r, 0, 3) == 0 ? 4 : 0);
  pool.v_pool = fake;
  pool.num_pages = (int32_t)order.size();
  const size_t bytes = kamera_step_workspace_bytes(&L, &s);
  CHECK(bytes > 0);
  Buffer ws(bytes);
  kamera_step_plan plan;
  Seen seen{&s, &L, {}};
  g_seen = &seen;
  CHECK(kamera_step_upload(&L, &s, &pool, ws.p, bytes, nullptr, &plan) == KAMERA_OK);
  CHECK(kamera_step_attend(&plan, 0, fake, 0, fake, 0, nullptr, 1.0f, nullptr) == KAMERA_OK);
  if (append) {
    kamera_append_rows rows;
    std::memset(&rows, 0, sizeof(rows));
    rows.k = rows.v = fake;
    CHECK(kamera_step_append(&plan, 0, &rows, nullptr) == KAMERA_OK);
  }
}

void one_copy(Rng& r, int exactly = 0) {
  kamera_layout L;
  std::memset(&L, 0, sizeof(L));
  L.family = KAMERA_GQA;
  L.dtype = KAMERA_F32;
  L.num_layers = 2;
  L.num_kv_heads = 1;
  L.head_dim = 2;
  L.page_size = 2;
  const int n = exactly ? exactly : (int)draw(r, 1, draw(r, 0, 1) ? 12 : 1500), copies = exactly ? n : (int)draw(r, 0, n);
  std::vector<int32_t> src((size_t)n), dst((size_t)n);
  for (int i = 0; i < n; ++i) src[(size_t)i] = dst[(size_t)i] = i;
  std::shuffle(dst.begin(), dst.end(), r);
  std::shuffle(src.begin(), src.end(), r);
  if (draw(r, 0, 1))
    for (int32_t& x : src) x = (int32_t)draw(r, 0, n - 1);
  if (exactly || draw(r, 0, 2) == 0)  // long chains
    for (int i = 0; i < n; ++i) src[(size_t)i] = (dst[(size_t)i] + 1) % n;
  std::vector<float> k((size_t)(2 * n * 4)), v(k.size());
  for (float& x : k) x = (float)draw(r, 0, 1 << 20);
  for (float& x : v) x = (float)draw(r, 0, 1 << 20);
  std::vector<float> want_k = k, want_v = v;
  for (int l = 0; l < 2; ++l)
    for (int i = 0; i < copies; ++i)
      for (int e = 0; e < 4; ++e) {
        want_k[(size_t)((l * n + dst[(size_t)i]) * 4 + e)] = k[(size_t)((l * n + src[(size_t)i]) * 4 + e)];
        want_v[(size_t)((l * n + dst[(size_t)i]) * 4 + e)] = v[(size_t)((l * n + src[(size_t)i]) * 4 + e)];
      }
  kamera_pool pool;
  std::memset(&pool, 0, sizeof(pool));
  pool.k_pool = k.data();
  pool.v_pool = v.data();
  pool.num_pages = n;
  const size_t bytes = kamera_copy_pages_workspace_bytes(copies);
  Buffer ws(bytes);
  CHECK(kamera_copy_pages(&L, &pool, src.data(), dst.data(), copies, ws.p, bytes, nullptr) == KAMERA_OK);
  CHECK(k == want_k && v == want_v);
}
}  // namespace

int main() {
  Rng r(12345);
  for (int i = 0; i < 150; ++i) one_step(r);
  for (int i = 0; i < 300; ++i) one_copy(r);
  for (int n = kLongChain - 3; n < kLongChain + 3; ++n) one_copy(r, n);  // one cycle
  std::printf("ok\n");
  return 0;
}
