// More of the serving step's host part on the CPU, with the stand-ins of step_host_check.cpp: host tables
// reached twice, workspaces that serve smaller steps. Exits 0 when all hold.
#define main step_host_check_main
#include "step_host_check.cpp"
#undef main

namespace {

// A pool of n pages whose every element names its page (and layer), with its layout.
struct Pages {
  kamera_layout L;
  kamera_pool pool;
  std::vector<float> k, v;
  explicit Pages(int n) {
    std::memset(&L, 0, sizeof(L));
    L.family = KAMERA_GQA;
    L.dtype = KAMERA_F32;
    L.num_layers = 2;
    L.num_kv_heads = 1;
    L.head_dim = 2;
    L.page_size = 2;
    k.resize((size_t)(2 * n * 4));
    for (size_t i = 0; i < k.size(); ++i) k[i] = (float)(i / 4);
    v = k;
    std::memset(&pool, 0, sizeof(pool));
    pool.k_pool = k.data();
    pool.v_pool = v.data();
    pool.num_pages = n;
  }
  // what page p of a layer held at first
  int held(int layer, int p) const { return (int)k[(size_t)((layer * pool.num_pages + p) * 4)] - layer * pool.num_pages; }
};

// Compaction of tables that lie in one array: entries [at, at + n) each.
void shared_tables(const std::vector<int32_t>& pages, int num_pages, const std::vector<std::pair<int, int>>& parts) {
  Pages p(num_pages);
  std::vector<int32_t> t = pages;
  std::vector<int32_t*> tables;
  std::vector<int32_t> lengths;
  std::vector<bool> named(pages.size(), false);
  for (const auto& x : parts) {
    tables.push_back(t.data() + x.first);
    lengths.push_back(x.second);
    for (int i = x.first; i < x.first + x.second; ++i) named[(size_t)i] = true;
  }
  std::map<int32_t, int> live;
  for (size_t i = 0; i < pages.size(); ++i)
    if (named[i]) live[pages[i]] = 1;
  const size_t bytes = kamera_copy_pages_workspace_bytes(num_pages);
  Buffer ws(bytes);
  int32_t n = -1;
  CHECK(kamera_compact_pages(&p.L, &p.pool, tables.data(), lengths.data(), (int32_t)tables.size(), &n, ws.p, bytes, nullptr) == KAMERA_OK);
  CHECK(n == (int32_t)live.size());
  for (size_t i = 0; i < t.size(); ++i) {
    if (!named[i]) {
      CHECK(t[i] == pages[i]);
      continue;
    }
    CHECK(t[i] >= 0 && t[i] < n);
    for (int layer = 0; layer < 2; ++layer) CHECK(p.held(layer, t[i]) == pages[i]);
  }
}

void compaction(Rng& r) {
  shared_tables({7, 8, 0}, 10, {{0, 3}, {0, 3}});                  // one array twice
  shared_tables({7, 8, 0, 9, 3}, 10, {{0, 5}, {0, 2}, {1, 3}});    // parts of it beside the whole
  shared_tables({5, 2, 5, 9}, 10, {{2, 2}, {0, 3}, {0, 4}});
  for (int i = 0; i < 200; ++i) {
    const int num = (int)draw(r, 1, 60), size = (int)draw(r, 1, 40);
    std::vector<int32_t> pages((size_t)size);
    for (int32_t& x : pages) x = (int32_t)draw(r, 0, num - 1);
    std::vector<std::pair<int, int>> parts;
    for (int k = (int)draw(r, 1, 4); k; --k) {
      const int at = (int)draw(r, 0, size - 1);
      parts.push_back({at, (int)draw(r, 0, size - at)});
    }
    shared_tables(pages, num, parts);
  }
}

// A step over pages of its own; its lengths and queries can be changed between uploads.
struct Steps {
  kamera_layout L;
  kamera_step s;
  kamera_pool pool;
  std::vector<kamera_prefix> pre;
  std::vector<kamera_request> req;
  std::vector<std::vector<int32_t>> tables;
  Steps(int family, int dtype, int heads, int kv_heads, int dim, std::vector<int64_t> prefixes, std::vector<std::pair<int64_t, int64_t>> requests,
        bool off_grid = false) {
    std::memset(&L, 0, sizeof(L));
    L.family = family;
    L.dtype = dtype;
    L.num_layers = 1;
    L.num_kv_heads = kv_heads;
    L.head_dim = dim;
    L.latent_dim = 512;
    L.rope_dim = 64;
    L.page_size = 16;
    L.rope_base = 1e4;
    std::memset(&s, 0, sizeof(s));
    s.num_q_heads = heads;
    s.num_prefixes = (int)prefixes.size();
    s.num_requests = (int)requests.size();
    pre.resize(prefixes.size());
    req.resize(requests.size());
    int32_t next = 0;
    auto table = [&](int64_t n) {
      std::vector<int32_t> t((size_t)((n + 15) / 16));
      for (int32_t& x : t) x = next++;
      tables.push_back(t);
    };
    for (int64_t n : prefixes) table(n);
    for (const auto& r : requests) table(r.first);
    for (size_t i = 0; i < pre.size(); ++i) pre[i] = kamera_prefix{tables[i].data(), 0, (int32_t)prefixes[i]};
    for (size_t i = 0; i < req.size(); ++i) {
      std::memset(&req[i], 0, sizeof(req[i]));
      req[i].block_table = tables[pre.size() + i].data();
      req[i].num_tokens = (int32_t)requests[i].first;
      req[i].num_queries = (int32_t)requests[i].second;
      req[i].prefix = pre.empty() ? -1 : (int)(i % pre.size());
    }
    s.requests = req.data();
    s.prefixes = pre.data();
    s.flags = KAMERA_STEP_ATTEND | KAMERA_STEP_FIT;
    std::memset(&pool, 0, sizeof(pool));
    pool.k_pool = reinterpret_cast<char*>((uintptr_t(1) << 40) + (off_grid ? 4 : 0));
    pool.v_pool = reinterpret_cast<char*>(uintptr_t(1) << 40);
    pool.num_pages = std::max(next, 1);
  }
  size_t bytes() { return kamera_step_workspace_bytes(&L, &s); }
  // Uploads and attends in `bytes` at ws; every place that the kernels write lies inside. Returns the partial rows.
  int64_t run(void* ws, size_t bytes) {
    kamera_step_plan plan;
    Seen seen{&s, &L, {}};
    g_seen = &seen;
    CHECK(kamera_step_upload(&L, &s, &pool, ws, bytes, nullptr, &plan) == KAMERA_OK);
    char* fake = reinterpret_cast<char*>(uintptr_t(1) << 40);
    CHECK(kamera_step_attend(&plan, 0, fake, 0, fake, 0, nullptr, 1.0f, nullptr) == KAMERA_OK);
    StepArgs a;
    std::memcpy(&a, plan.detail, sizeof(a));
    int64_t parts = 0;
    for (int i = 0; i < a.num_items; ++i) {
      const AttendRun& run = a.items[i].run;
      if (!run.direct) parts = std::max(parts, run.part0 + (int64_t)run.splits * a.heads * run.ntok * a.group);
    }
    const char *base = static_cast<char*>(ws), *end = base + bytes;
    if (parts) CHECK((char*)a.part_ml >= base && (char*)(a.part_ml + parts) <= (char*)a.part_o && (char*)(a.part_o + parts * a.dv) <= end);
    return parts;
  }
};

// Requests that see no key leave the others' ranges as they are.
void empty_requests() {
  std::vector<std::pair<int64_t, int64_t>> requests(40, {300, 1});
  Steps some(KAMERA_GQA, KAMERA_BF16, 32, 8, 128, {}, requests);
  requests.resize(200, {0, 1});
  Steps more(KAMERA_GQA, KAMERA_BF16, 32, 8, 128, {}, requests);
  const size_t bytes = std::max(some.bytes(), more.bytes());
  Buffer ws(bytes);
  CHECK(some.run(ws.p, bytes) == more.run(ws.p, bytes));
}

// One buffer, sized for the longest step, serves every shorter one.
void one_workspace(Rng& r) {
  struct Kind {
    int family, dtype, heads, kv_heads, dim;
    bool off_grid;
  };
  const Kind kinds[] = {{KAMERA_GQA, KAMERA_BF16, 32, 8, 128, false}, {KAMERA_GQA, KAMERA_BF16, 32, 8, 128, true}, {KAMERA_GQA, KAMERA_F32, 8, 2, 64, false},
                        {KAMERA_MLA, KAMERA_BF16, 16, 1, 0, false}, {KAMERA_MLA, KAMERA_F32, 3, 1, 0, false}, {KAMERA_GQA, KAMERA_BF16, 7, 1, 80, false}};
  for (const Kind& k : kinds)
    for (int turn = 0; turn < 6; ++turn) {
      std::vector<int64_t> prefixes;
      std::vector<std::pair<int64_t, int64_t>> requests;
      for (int i = (int)draw(r, 0, 2); i; --i) prefixes.push_back(draw(r, 1, turn < 3 ? 1200 : 300));
      for (int i = (int)draw(r, 1, 6); i; --i) requests.push_back({draw(r, 0, 600), draw(r, 0, 2) ? 1 : draw(r, 0, 60)});
      Steps st(k.family, k.dtype, k.heads, k.kv_heads, k.dim, prefixes, requests, k.off_grid);
      const size_t bytes = st.bytes();
      CHECK(bytes > 0);
      Buffer ws(bytes);
      st.run(ws.p, bytes);
      for (int again = 0; again < 12; ++again) {  // shorter in every way, requests and prefixes left out
        for (size_t i = 0; i < prefixes.size(); ++i) st.pre[i].num_tokens = (int32_t)draw(r, 0, 3) ? (int32_t)draw(r, 0, prefixes[i]) : (int32_t)prefixes[i];
        for (size_t i = 0; i < requests.size(); ++i) {
          st.req[i].num_tokens = draw(r, 0, 3) ? (int32_t)draw(r, 0, requests[i].first) : 0;
          st.req[i].num_queries = draw(r, 0, 3) ? (int32_t)draw(r, 0, requests[i].second) : (int32_t)requests[i].second;
          st.req[i].prefix = st.pre.empty() || draw(r, 0, 4) == 0 ? -1 : (int)(i % st.pre.size());
        }
        st.s.num_requests = (int)draw(r, 1, (int64_t)requests.size());
        st.run(ws.p, bytes);
      }
    }
  // sizes that fall as the step grows: 64 requests over 8192 shared tokens, 8 of them with more or fewer queries
  Steps many(KAMERA_GQA, KAMERA_BF16, 32, 8, 128, {8192}, std::vector<std::pair<int64_t, int64_t>>(64, {4192, 1}));
  const size_t most = many.bytes();
  Buffer ws(most);
  const int lengths[] = {4192, 2000, 800, 176, 64, 17, 1, 0};
  bool fell = false;
  for (int n : lengths) {
    for (kamera_request& q : many.req) q.num_tokens = n;
    fell = fell || many.bytes() > most;
    many.run(ws.p, most);
  }
  CHECK(fell);
  Steps wide(KAMERA_GQA, KAMERA_BF16, 32, 8, 128, {8192}, std::vector<std::pair<int64_t, int64_t>>(8, {1000, 256}));
  const size_t few = wide.bytes();
  Buffer ws2(few);
  for (int n : {256, 100, 23, 3, 1}) {
    for (kamera_request& q : wide.req) q.num_queries = n;
    wide.run(ws2.p, few);
  }
  wide.s.flags = KAMERA_STEP_ATTEND;  // without the flag, the refusal
  kamera_step_plan none;
  CHECK(wide.bytes() > few && kamera_step_upload(&wide.L, &wide.s, &wide.pool, ws2.p, few, nullptr, &none) == KAMERA_E_WORKSPACE);
  // the fastest plan wherever it fits; less and less of it down to no partial row at all; then a refusal
  Steps st(KAMERA_GQA, KAMERA_BF16, 32, 8, 128, {9000}, std::vector<std::pair<int64_t, int64_t>>(12, {500, 2}));
  size_t bytes = st.bytes();
  int64_t parts = st.run(Buffer(bytes).p, bytes);
  CHECK(parts > 0);
  kamera_step_plan plan;
  for (int refusals = 0; refusals == 0; bytes = bytes * 3 / 4 / 256 * 256) {
    Buffer b(bytes);
    if (kamera_step_upload(&st.L, &st.s, &st.pool, b.p, bytes, nullptr, &plan) != KAMERA_OK) {
      CHECK(kamera_step_upload(&st.L, &st.s, &st.pool, b.p, bytes, nullptr, &plan) == KAMERA_E_WORKSPACE);
      CHECK(parts == 0);
      ++refusals;
      continue;
    }
    const int64_t now = st.run(b.p, bytes);
    CHECK(now <= parts);
    parts = now;
  }
}

}  // namespace

int main() {
  Rng r(4711);
  compaction(r);
  one_workspace(r);
  empty_requests();
  std::printf("ok\n");
  return 0;
}
