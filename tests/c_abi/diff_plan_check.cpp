// How differential attention's work is shared out, on the CPU, with the stand-ins of step_host_check.cpp: in launches
// that fill the chip's places no workgroup takes much longer than an even share of the whole, whatever the requests'
// lengths. Exits 0 when all hold.
//
// The bound: a run is left whole if its keys take at most 1.1 even shares W. Otherwise its class's range is the one of
// least estimate E = max(5/4 r, W + more + r/4) + parts (r: the range's time; for like runs max(rounds * r, W + more) + parts).
// So 5/4 r <= E <= E(r') for every other range r'; for one of W/2 that is max(5/8 W, 9/8 W + more + parts), more and parts
// being what at most two ranges for every share of each place cost (under 0.2 W where W is 10 starts or more): r <= 0.8 * 1.33 W.
// Like runs: r <= E <= E(r'), and with r' = W/8 that is at most W + r' + more + parts, under 1.25 W as well.
// Workgroups are taken up in order by places that become free, so that the launch ends at most an even share after its
// longest one: 2.25 W.
#define main step_host_check_main
#include "step_host_check.cpp"
#undef main

#include <queue>

namespace {
struct Launch {
  double ends, even, longest;  // in keys of a wide tile
  int64_t places;              // workgroups
} g_launch;
constexpr int kPlaces = 512;      // two workgroups a CU
constexpr double kStart = 6000 / 49.0, kPairs = 45 / 49.0;  // a workgroup's own time, a key of smaller tiles
}  // namespace

namespace kamera {
hipError_t launch_step_attend_diff(const StepArgs& a, int, const void*, int64_t, void*, int64_t, float*, float, const kamera_differential&, hipStream_t) {
  std::priority_queue<double, std::vector<double>, std::greater<double>> places;
  for (int i = 0; i < kPlaces; ++i) places.push(0);
  g_launch = Launch{0, 0, 0, (int64_t)a.num_items * a.heads};
  for (int i = 0; i < a.num_items; ++i) {
    const AttendItem& it = a.items[i];
    const double keys = it.kv1 - it.kv0, time = kStart * 128 / a.dk + (it.run.tile == TILE_WIDE ? 1 : kPairs) * keys;
    g_launch.longest = std::max(g_launch.longest, time);
    g_launch.even += time * a.heads / kPlaces;
    for (int h = 0; h < a.heads; ++h) {
      const double ends = places.top() + time;
      places.pop();
      places.push(ends);
      g_launch.ends = std::max(g_launch.ends, ends);
    }
  }
  return hipSuccess;
}
hipError_t launch_step_weigh(const StepArgs&, int, const void*, int64_t, const float*, float*, float, float, hipStream_t) { return hipSuccess; }
hipError_t launch_evict(const EvictArgs&, hipStream_t) { return hipSuccess; }
}  // namespace kamera

namespace {

struct Request {
  int64_t tokens, queries;
};

Launch plan(int heads, int kv_heads, int dim, int64_t prefix, const std::vector<Request>& requests) {
  kamera_layout L;
  std::memset(&L, 0, sizeof(L));
  L.family = KAMERA_GQA;
  L.dtype = KAMERA_BF16;
  L.num_layers = 1;
  L.num_kv_heads = kv_heads;
  L.head_dim = dim;
  L.page_size = 64;
  L.rope_base = 1e4;
  int32_t next = 0;
  auto table = [&](int64_t n) {
    std::vector<int32_t> t((size_t)(n + 63) / 64);
    for (int32_t& x : t) x = next++;
    return t;
  };
  std::vector<std::vector<int32_t>> tables;
  std::vector<kamera_request> req(requests.size());
  const std::vector<int32_t> shared = table(prefix);
  const kamera_prefix pre{shared.data(), 0, (int32_t)prefix};
  for (size_t i = 0; i < req.size(); ++i) {
    std::memset(&req[i], 0, sizeof(req[i]));
    tables.push_back(table(requests[i].tokens));
    req[i].block_table = tables.back().data();
    req[i].num_tokens = (int32_t)requests[i].tokens;
    req[i].num_queries = (int32_t)requests[i].queries;
    req[i].prefix = prefix ? 0 : -1;
  }
  kamera_step s;
  std::memset(&s, 0, sizeof(s));
  s.requests = req.data();
  s.num_requests = (int)req.size();
  s.prefixes = &pre;
  s.num_prefixes = prefix ? 1 : 0;
  s.num_q_heads = heads;
  s.flags = KAMERA_STEP_ATTEND | KAMERA_STEP_DIFFERENTIAL;
  kamera_pool pool;
  std::memset(&pool, 0, sizeof(pool));
  pool.k_pool = pool.v_pool = reinterpret_cast<char*>(uintptr_t(1) << 40);
  pool.num_pages = std::max(next, 1);
  const size_t bytes = kamera_step_workspace_bytes(&L, &s);
  CHECK(bytes > 0);
  std::vector<char> room(bytes + 256);
  void* ws = reinterpret_cast<void*>(((uintptr_t)room.data() + 255) / 256 * 256);
  kamera_step_plan p;
  CHECK(kamera_step_upload(&L, &s, &pool, ws, bytes, nullptr, &p) == KAMERA_OK);
  kamera_differential d;
  std::memset(&d, 0, sizeof(d));
  char* fake = reinterpret_cast<char*>(uintptr_t(1) << 40);
  CHECK(kamera_step_attend_diff(&p, 0, fake, 0, fake, 0, nullptr, 1.0f, &d, nullptr) == KAMERA_OK);
  return g_launch;
}

}  // namespace

bool shared_out(const Launch& l) {
  if (l.places < kPlaces || l.even < 10 * kStart) return true;
  return l.longest <= 1.25 * l.even && l.ends <= 2.25 * l.even;
}

int main() {
  // one long request among short ones, the first or the last of them: as with fewer of them
  for (int64_t longest : {30000, 120000}) {
    for (int n : {6, 7, 8, 9, 12, 16, 30}) {
      std::vector<Request> r((size_t)n, Request{1000, 300});
      for (size_t i : {(size_t)0, (size_t)(n - 1)}) {
        r.assign((size_t)n, Request{1000, 300});
        r[i].tokens = longest;
        const Launch l = plan(28, 4, 128, 0, r);
        std::snprintf(g_error, sizeof(g_error), "%d requests, %lld tokens: ends %.0f even %.0f longest %.0f", n, (long long)longest, l.ends, l.even, l.longest);
        CHECK(shared_out(l));
      }
    }
  }
  // requests alike: whole tiles for whole rounds of the places, the rest in pieces
  for (int queries : {256, 300, 320, 400}) {
    std::vector<Request> r(8, Request{queries + 100, queries});
    const Launch l = plan(28, 4, 128, 8192, r);
    std::snprintf(g_error, sizeof(g_error), "%d queries: ends %.0f even %.0f longest %.0f", queries, l.ends, l.even, l.longest);
    CHECK(l.longest >= 8192 || 8 * queries * 14 * 2 / 128 < kPlaces);
    CHECK(shared_out(l));
  }
  Rng r(1);
  for (int i = 0; i < 60; ++i) {
    const int kinds[][3] = {{28, 4, 128}, {32, 8, 128}, {32, 32, 128}, {16, 2, 128}, {16, 4, 64}, {12, 12, 64}};
    const int* k = kinds[draw(r, 0, 5)];
    std::vector<Request> q;
    const double lo = std::exp(draw(r, 0, 1000) / 1000.0 * 4 + 4), hi = lo * std::exp(draw(r, 0, 1000) / 1000.0 * 4);
    const int64_t prefix = draw(r, 0, 1) ? draw(r, 1, 20000) : 0;
    for (int n = (int)draw(r, 1, 40); n; --n) {
      const int64_t t = (int64_t)(lo * std::pow(hi / lo, draw(r, 0, 1000) / 1000.0));
      q.push_back({t, std::min<int64_t>(t, draw(r, 1, 700))});
    }
    const Launch l = plan(k[0], k[1], k[2], prefix, q);
    std::snprintf(g_error, sizeof(g_error), "batch %d: ends %.0f even %.0f longest %.0f", i, l.ends, l.even, l.longest);
    CHECK(shared_out(l));
  }
  std::printf("ok\n");
  return 0;
}
