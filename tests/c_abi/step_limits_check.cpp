// More of the serving step's host part on the CPU, with the stand-ins of step_host_check.cpp: host tables
// reached twice. Exits 0 when all hold.
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

}  // namespace

int main() {
  Rng r(4711);
  compaction(r);
  std::printf("ok\n");
  return 0;
}
