// The host parts of differential attention, weighing and eviction on the CPU, with the stand-ins of
// step_host_check.cpp and more: every key meets the rows that see it once, differential work lists are those of
// pairs of heads, evictions carry out what the interface says, plans that fit a workspace stay inside it. Exits 0
// when all hold.
#define main step_host_check_main
#include "step_host_check.cpp"
#undef main

#include <set>

namespace {
const char *g_ws, *g_ws_end;
int64_t g_weigh_parts;
void inside(const void* p, size_t bytes) { CHECK((const char*)p >= g_ws && (const char*)p + bytes <= g_ws_end); }
}  // namespace

namespace kamera {
hipError_t launch_step_attend_diff(const StepArgs& a, int layer, const void* q, int64_t q_stride, void* out, int64_t out_stride, float* lse,
                                   float scale, const kamera_differential&, hipStream_t stream) {
  const kamera_layout* L = g_seen->lay;
  CHECK(a.differential && a.heads * 2 == L->num_kv_heads && a.group * a.heads == a.num_q_heads && a.group % 2 == 0 && a.dv == 2 * a.dk);
  CHECK(a.kernel == ATTEND_PLAIN || a.kernel == ATTEND_DIFF);
  for (int i = 0; i < a.num_items; ++i) {
    const AttendRun& run = a.items[i].run;
    CHECK(run.part0 % 2 == 0 && !(run.direct && a.kernel == ATTEND_PLAIN));
    const int64_t parts = run.direct ? 0 : run.part0 + (int64_t)run.splits * a.heads * run.ntok * a.group;
    inside(a.part_ml, (size_t)parts * 8);
    inside(a.part_o, (size_t)(parts * a.dv * 4));
    CHECK((char*)(a.part_ml + parts) <= (char*)a.part_o);
  }
  return launch_step_attend(a, layer, q, q_stride, out, out_stride, lse, scale, stream);
}

// Which rows of head 0 meet which slots; the join takes every partial sum once and no other.
hipError_t launch_step_weigh(const StepArgs& a, int, const void*, int64_t, const float*, float*, float, float, hipStream_t) {
  const kamera_step* s = g_seen->step;
  const int G = a.num_q_heads / a.heads, P = a.page_size, keys = weigh_keys(a.weigh_kernel);
  std::map<int64_t, std::map<int64_t, int>> met;  // slot -> (token, g) -> times
  std::map<int64_t, std::map<int64_t, int>> part;  // partial sum -> the same
  std::map<int64_t, int> writers;
  auto slot = [&](int pg, int slot0, int t) { return pool_slot(a, pg, slot0 + t); };
  g_weigh_parts = 0;
  for (int i = 0; i < a.num_weigh; ++i) {
    const WeighItem& it = a.weigh[i];
    CHECK(it.kv0 >= 0 && it.kv0 < it.kv1 && it.kv1 <= it.kv && it.kv1 - it.kv0 <= (it.ntok * G <= kFewRows ? weigh_keys_of_few(a.weigh_kernel) : keys) && it.row0 >= 0 && it.row0 < it.row1 && it.row1 <= (int64_t)it.ntok * G);
    for (int t = it.kv0; t < it.kv1; ++t) {
      std::map<int64_t, int> rows;
      for (int row = it.row0; row < it.row1; ++row) {
        const int j = (int)(((uint64_t)(uint32_t)row * a.group_magic) >> a.group_bits);
        CHECK(j == row / G);
        const int token = it.listed ? a.tok[it.tok0 + j] : it.tok0 + j;
        CHECK(token >= 0 && token < a.num_tokens);
        if (t <= it.lim0 + j * it.lstep) ++rows[(int64_t)token * G + row - j * G];
      }
      const bool appends = s->flags & KAMERA_STEP_APPEND;
      if (!it.listed && it.lstep) CHECK(it.fresh == (appends ? it.lim0 : it.kv));
      if (it.part < 0) {
        CHECK(writers[slot(it.pg, it.slot, t)]++ == 0);
        met[slot(it.pg, it.slot, t)] = rows;
      } else {
        const int64_t at = it.part + ((int64_t)it.split * a.heads) * it.kv + t;
        CHECK(part.find(at) == part.end());
        part[at] = rows;
        g_weigh_parts = std::max(g_weigh_parts, at + (int64_t)(a.heads - 1) * it.kv + 1);
      }
    }
  }
  if (g_weigh_parts) inside(a.weigh_part, (size_t)g_weigh_parts * 4);
  for (int k = 0; k < a.num_weigh_join; ++k) {
    const WeighJoin& j = a.weigh_join[k];
    CHECK(j.kv <= a.weigh_longest && j.tile == keys);
    for (int t = 0; t < j.kv; ++t) {
      const int kv0 = t / j.tile * j.tile;
      const int64_t row0 = j.lstep && kv0 > j.lim0 ? (int64_t)(kv0 - j.lim0) * G : 0;
      CHECK(writers[slot(j.pg, j.slot, t)]++ == 0);
      auto& m = met[slot(j.pg, j.slot, t)];
      for (int sp = (int)(row0 / j.rows); sp < j.splits; ++sp) {
        const auto p = part.find(j.part + ((int64_t)sp * a.heads) * j.kv + t);
        CHECK(p != part.end());
        for (const auto& x : p->second) m[x.first] += x.second;
        part.erase(p);
      }
    }
  }
  CHECK(part.empty());
  std::map<int64_t, std::map<int64_t, int>> want;
  int64_t token = 0;
  for (int i = 0; i < s->num_requests; ++i) {
    const kamera_request& r = s->requests[i];
    for (int j = 0; j < r.num_queries; ++j, ++token) {
      auto add = [&](const int32_t* table, int slot0, int64_t n, int64_t seen) {
        for (int64_t t = 0; t < n; ++t) {
          auto& m = want[(int64_t)table[(slot0 + t) / P] * P + (slot0 + t) % P];
          for (int g = 0; g < G && t < seen; ++g) ++m[token * G + g];
        }
      };
      if (r.prefix >= 0) add(s->prefixes[r.prefix].block_table, s->prefixes[r.prefix].slot0, s->prefixes[r.prefix].num_tokens, s->prefixes[r.prefix].num_tokens);
      add(r.block_table, r.slot0, r.num_tokens, (r.flags & KAMERA_REQUEST_ALL) ? r.num_tokens : (int64_t)r.num_tokens - r.num_queries + j + 1);
    }
  }
  CHECK(want.size() == met.size());
  CHECK(want == met);
  return hipSuccess;
}

// An eviction as its kernels carry it out, on host memory; rows of fp32.
hipError_t launch_evict(const EvictArgs& a, hipStream_t) {
  const int groups = a.heads / a.together, P = a.page_size;
  inside(a.starts, (size_t)a.layers * groups * a.num_seqs * 4);
  if (a.phase) inside(a.phase, (size_t)a.shifts * a.d_rot * 4);
  for (int i = 0; i < a.num_seqs; ++i) {
    const EvictSeq& s = a.seqs[i];
    const int keep = std::min(s.keep, s.num_tokens);
    CHECK(s.kept0 + keep <= a.total);
    if (keep == s.num_tokens) {
      for (int l = 0; l < a.layers * groups; ++l)
        for (int j = 0; j < keep; ++j) a.kept[(int64_t)l * a.total + s.kept0 + j] = j;
      continue;
    }
    CHECK(s.num_tokens <= a.longest && keep <= a.most_kept && s.num_tokens - keep < a.shifts);
    auto slot = [&](int t) {
      const int at = s.slot0 + t, pg = (int)(((uint64_t)(uint32_t)at * a.page_magic) >> a.page_bits);
      CHECK(pg == at / P);
      return (int64_t)a.pages[s.pg + pg] * P + at % P;
    };
    for (int layer = 0; layer < a.layers; ++layer)
      for (int g = 0; g < groups; ++g) {
        float* scores = a.scores + layer * a.scores_stride;
        auto score = [&](int t, int h) -> float& { return scores[(slot(t) / P * a.heads + h) * P + slot(t) % P]; };
        std::vector<std::pair<float, int>> ranked;
        for (int t = s.first; t < s.num_tokens - s.last; ++t) {
          float x = score(t, g * a.together);
          for (int h = 1; h < a.together; ++h) x += score(t, g * a.together + h);
          ranked.push_back({-x, t});
        }
        std::sort(ranked.begin(), ranked.end());
        std::set<int> stay;
        for (int t = 0; t < s.first; ++t) stay.insert(t);
        for (int t = s.num_tokens - s.last; t < s.num_tokens; ++t) stay.insert(t);
        for (int k = 0; k < keep - s.first - s.last; ++k) stay.insert(ranked[(size_t)k].second);
        CHECK((int)stay.size() == keep);
        int j = 0;
        for (int t : stay) {
          CHECK(j <= t);
          a.kept[((int64_t)layer * groups + g) * a.total + s.kept0 + j] = t;
          for (int h = g * a.together; h < (g + 1) * a.together; ++h) score(j, h) = score(t, h);
          for (int x = 0; x < a.tensors; ++x) {
            char* base = a.pool[x] + layer * a.layer_bytes + (int64_t)g * a.together * a.head_bytes;
            std::memmove(base + slot(j) * a.row_bytes, base + slot(t) * a.row_bytes, (size_t)(a.together * a.head_bytes));
          }
          ++j;
        }
      }
  }
  return hipSuccess;
}
}  // namespace kamera

namespace {

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
};

void run_more(Steps& st, void* ws, size_t bytes) {
  kamera_step_plan plan;
  Seen seen{&st.s, &st.L, {}};
  g_seen = &seen;
  g_ws = static_cast<char*>(ws);
  g_ws_end = g_ws + bytes;
  CHECK(kamera_step_upload(&st.L, &st.s, &st.pool, ws, bytes, nullptr, &plan) == KAMERA_OK);
  char* fake = reinterpret_cast<char*>(uintptr_t(1) << 40);
  kamera_differential d;
  std::memset(&d, 0, sizeof(d));
  if (st.s.flags & KAMERA_STEP_ATTEND) {
    const kamera_status other = kamera_step_attend(&plan, 0, fake, 0, fake, 0, nullptr, 1.0f, nullptr);
    const kamera_status diff = kamera_step_attend_diff(&plan, 0, fake, 0, fake, 0, nullptr, 1.0f, &d, nullptr);
    if (st.s.flags & KAMERA_STEP_DIFFERENTIAL) CHECK(other == KAMERA_E_UNSUPPORTED && diff == KAMERA_OK);
    else CHECK(other == KAMERA_OK && diff == KAMERA_E_UNSUPPORTED);
  }
  const kamera_status w = kamera_step_weigh(&plan, 0, fake, 0, (float*)fake, (float*)fake, 1.0f, 1.0f, nullptr);
  CHECK(w == ((st.s.flags & KAMERA_STEP_WEIGH) ? KAMERA_OK : KAMERA_E_UNSUPPORTED));
}

void steps(Rng& r) {
  struct Kind {
    int family, dtype, heads, kv_heads, dim;
    bool off_grid, diff;
  };
  const Kind kinds[] = {{KAMERA_GQA, KAMERA_BF16, 32, 8, 128, false, true}, {KAMERA_GQA, KAMERA_BF16, 28, 4, 128, false, true}, {KAMERA_GQA, KAMERA_BF16, 32, 8, 128, true, true},
                        {KAMERA_GQA, KAMERA_F32, 8, 2, 64, false, true}, {KAMERA_GQA, KAMERA_BF16, 6, 2, 10, false, true}, {KAMERA_GQA, KAMERA_BF16, 32, 8, 128, false, false},
                        {KAMERA_GQA, KAMERA_BF16, 7, 1, 64, false, false}, {KAMERA_MLA, KAMERA_BF16, 16, 1, 0, false, false}, {KAMERA_MLA, KAMERA_F32, 3, 1, 0, false, false}};
  for (const Kind& k : kinds)
    for (int turn = 0; turn < 5; ++turn) {
      std::vector<int64_t> prefixes;
      std::vector<std::pair<int64_t, int64_t>> requests;
      for (int i = (int)draw(r, 0, 2); i; --i) prefixes.push_back(draw(r, 1, turn < 3 ? 1200 : 300));
      for (int i = (int)draw(r, 1, 6); i; --i) requests.push_back({draw(r, 0, 600), draw(r, 0, 2) ? draw(r, 0, 2) : draw(r, 0, turn == 0 ? 300 : 60)});
      Steps st(k.family, k.dtype, k.heads, k.kv_heads, k.dim, prefixes, requests, k.off_grid);
      const uint32_t which[] = {KAMERA_STEP_ATTEND, KAMERA_STEP_WEIGH, KAMERA_STEP_ATTEND | KAMERA_STEP_WEIGH};
      st.s.flags = which[draw(r, 0, 2)] | (draw(r, 0, 2) ? KAMERA_STEP_FIT : 0) | (k.diff ? KAMERA_STEP_DIFFERENTIAL : 0);
      for (auto& q : st.req) q.flags = draw(r, 0, 4) == 0 ? KAMERA_REQUEST_ALL : 0;
      const size_t bytes = st.bytes();
      CHECK(bytes > 0);
      Buffer ws(bytes);
      run_more(st, ws.p, bytes);
      if (!(st.s.flags & KAMERA_STEP_FIT)) continue;
      for (int again = 0; again < 4; ++again) {  // shorter in every way
        for (size_t i = 0; i < prefixes.size(); ++i) st.pre[i].num_tokens = (int32_t)draw(r, 0, prefixes[i]);
        for (size_t i = 0; i < requests.size(); ++i) {
          st.req[i].num_tokens = (int32_t)draw(r, 0, requests[i].first);
          st.req[i].num_queries = (int32_t)draw(r, 0, requests[i].second);
          st.req[i].prefix = st.pre.empty() || draw(r, 0, 4) == 0 ? -1 : (int)(i % st.pre.size());
        }
        st.s.num_requests = (int)draw(r, 1, (int64_t)requests.size());
        run_more(st, ws.p, bytes);
      }
    }
  // rows cut into ranges, and a workspace without room for them
  Steps many(KAMERA_GQA, KAMERA_BF16, 28, 4, 64, {600}, {{1000, 400}, {20, 20}, {300, 300}});
  many.s.flags = KAMERA_STEP_WEIGH | KAMERA_STEP_FIT;
  const size_t bytes = many.bytes();
  Buffer ws(bytes);
  run_more(many, ws.p, bytes);
  CHECK(g_weigh_parts > 0);
  kamera_step_plan plan;
  size_t least = 256;
  while (kamera_step_upload(&many.L, &many.s, &many.pool, ws.p, least, nullptr, &plan) != KAMERA_OK) least += 256;
  CHECK(least < bytes);
  run_more(many, ws.p, least);
  CHECK(g_weigh_parts == 0);
  // more wide tiles than a round of places: some runs whole, the last queries of others in pieces
  for (int extra : {0, 3, 40, 150}) {
    Steps rounds(KAMERA_GQA, KAMERA_BF16, 128, 8, 128, {300}, {{200, 200}, {330 + extra, 330 + extra}, {5, 1}});
    rounds.s.flags = KAMERA_STEP_ATTEND | KAMERA_STEP_DIFFERENTIAL | KAMERA_STEP_FIT;
    const size_t need = rounds.bytes();
    Buffer w(need);
    run_more(rounds, w.p, need);
    rounds.req[1].num_queries -= 20;
    run_more(rounds, w.p, need);
  }
  // slots weighed twice
  Steps twice(KAMERA_GQA, KAMERA_F32, 8, 2, 64, {40}, {{40, 1}, {40, 1}});
  twice.s.flags = KAMERA_STEP_WEIGH;
  const size_t some = twice.bytes();
  Buffer ws2(some);
  run_more(twice, ws2.p, some);
  auto refused = [&] { CHECK(kamera_step_upload(&twice.L, &twice.s, &twice.pool, ws2.p, some, nullptr, &plan) == KAMERA_E_OVERLAP); };
  const int32_t* own = twice.req[1].block_table;
  twice.req[1].block_table = twice.req[0].block_table;
  refused();
  twice.req[1].num_queries = 0;  // it weighs nothing
  run_more(twice, ws2.p, some);
  twice.req[1].num_queries = 1;
  twice.req[1].block_table = twice.pre[0].block_table;
  refused();
  twice.req[1].block_table = own;
  std::vector<int32_t> repeats(own, own + 3);
  repeats[2] = repeats[1];
  twice.req[1].block_table = repeats.data();  // a page twice: tokens 16.. and 32..39
  refused();
  twice.req[1].num_tokens = 32;
  run_more(twice, ws2.p, some);
  repeats[2] = twice.req[0].block_table[2];  // one page of both: slots 0..7, and 8..15
  twice.req[1].num_tokens = 24;
  twice.req[1].slot0 = 8;
  repeats[0] = twice.req[0].block_table[2];
  run_more(twice, ws2.p, some);
}

void one_eviction(Rng& r) {
  kamera_layout L;
  std::memset(&L, 0, sizeof(L));
  const bool mla = draw(r, 0, 3) == 0;
  L.family = mla ? KAMERA_MLA : KAMERA_GQA;
  L.dtype = KAMERA_F32;
  L.num_layers = (int)draw(r, 1, 3);
  L.num_kv_heads = mla ? 0 : 4;
  L.head_dim = mla ? 0 : 2;
  L.latent_dim = 3;
  L.rope_dim = 2;
  L.rope_base = 1e4;
  const int sizes[] = {1, 3, 16};
  L.page_size = sizes[draw(r, 0, 2)];
  const int heads = mla ? 1 : 4, F = mla ? 5 : 8, P = L.page_size;
  std::vector<kamera_evict_seq> seqs((size_t)draw(r, 0, 5));
  std::vector<std::vector<int32_t>> tables(seqs.size());
  int32_t next = 0;
  for (size_t i = 0; i < seqs.size(); ++i) {
    kamera_evict_seq& s = seqs[i];
    std::memset(&s, 0, sizeof(s));
    s.slot0 = (int)draw(r, 0, P - 1);
    s.num_tokens = (int)draw(r, 0, 60);
    s.keep = (int)draw(r, 0, 70);
    s.first = (int)draw(r, 0, s.keep);
    s.last = (int)draw(r, 0, s.keep - s.first);
    tables[i].resize((size_t)(s.num_tokens ? (s.slot0 + s.num_tokens + P - 1) / P : 0));
    for (int32_t& x : tables[i]) x = next++;
  }
  std::vector<int32_t> order((size_t)next + 2);
  for (size_t i = 0; i < order.size(); ++i) order[i] = (int32_t)i;
  std::shuffle(order.begin(), order.end(), r);
  for (size_t i = 0; i < seqs.size(); ++i) {
    for (int32_t& x : tables[i]) x = order[(size_t)x];
    seqs[i].block_table = tables[i].data();
  }
  const size_t rows = order.size() * (size_t)P;
  std::vector<float> k(rows * (size_t)(F * L.num_layers)), v(k.size()), scores(rows * (size_t)(heads * L.num_layers));
  for (float& x : k) x = (float)draw(r, 0, 1 << 20);
  for (float& x : v) x = (float)draw(r, 0, 1 << 20);
  for (float& x : scores) x = (float)draw(r, 0, 40);  // ties
  std::vector<float> k1 = k, v1 = v, s1 = scores;
  kamera_eviction e;
  std::memset(&e, 0, sizeof(e));
  e.seqs = seqs.data();
  e.scores = scores.data();
  e.num_seqs = (int)seqs.size();
  const int together[] = {1, 2, 4};
  e.heads_together = mla ? 1 : together[draw(r, 0, 2)];
  e.flags = draw(r, 0, 1) ? KAMERA_EVICT_REANCHOR : 0;
  int64_t total = 0;
  for (const auto& s : seqs) total += std::min(s.keep, s.num_tokens);
  std::vector<int32_t> kept((size_t)(L.num_layers * (heads / e.heads_together) * total) + 1, -7);
  if (draw(r, 0, 1)) e.kept = kept.data();
  kamera_pool pool;
  std::memset(&pool, 0, sizeof(pool));
  pool.k_pool = k.data();
  pool.v_pool = mla ? nullptr : v.data();
  pool.num_pages = (int)order.size();
  const size_t bytes = kamera_evict_workspace_bytes(&L, &e);
  CHECK(bytes > 0);
  Buffer ws(bytes);
  g_ws = static_cast<char*>(ws.p);
  g_ws_end = g_ws + bytes;
  CHECK(kamera_evict(&L, &pool, &e, ws.p, bytes, nullptr) == KAMERA_OK);
  CHECK(kept.back() == -7);
  if (bytes > 256) CHECK(kamera_evict(&L, &pool, &e, ws.p, bytes - 256, nullptr) == KAMERA_E_WORKSPACE);
  // from the definition
  int64_t k0 = 0;
  const std::vector<float> was_k = k1, was_v = v1, was_s = s1;
  for (const auto& s : seqs) {
    auto slot = [&](int t) { return (size_t)(s.block_table[(s.slot0 + t) / P] * P + (s.slot0 + t) % P); };
    const int keep = std::min(s.keep, s.num_tokens);
    for (int l = 0; l < L.num_layers; ++l)
      for (int g = 0; g < heads; g += e.heads_together) {
        auto at = [&](int t, int h) { return (size_t)l * rows * (size_t)heads + (slot(t) / (size_t)P * (size_t)heads + (size_t)h) * (size_t)P + slot(t) % (size_t)P; };
        int j = 0;
        for (int t = 0; t < s.num_tokens; ++t) {
          int better = 0;  // of those between
          const bool ends = t < s.first || t >= s.num_tokens - s.last;
          auto sum = [&](int x) {
            float y = 0;
            for (int h = g; h < g + e.heads_together; ++h) y += was_s[at(x, h)];
            return y;
          };
          for (int x = s.first; x < s.num_tokens - s.last && !ends; ++x) better += sum(x) > sum(t) || (sum(x) == sum(t) && x < t);
          if (keep < s.num_tokens && !ends && better >= keep - s.first - s.last) continue;
          if (e.kept) CHECK(kept[(size_t)((l * (heads / e.heads_together) + g / e.heads_together) * total + k0 + j)] == t);
          for (int h = g; h < g + e.heads_together; ++h) {
            s1[at(j, h)] = was_s[at(t, h)];
            for (int c = h * (F / heads); c < (h + 1) * (F / heads); ++c) {
              k1[((size_t)l * rows + slot(j)) * (size_t)F + (size_t)c] = was_k[((size_t)l * rows + slot(t)) * (size_t)F + (size_t)c];
              if (!mla) v1[((size_t)l * rows + slot(j)) * (size_t)F + (size_t)c] = was_v[((size_t)l * rows + slot(t)) * (size_t)F + (size_t)c];
            }
          }
          ++j;
        }
        CHECK(j == keep);
      }
    k0 += keep;
  }
  CHECK(k == k1 && v == v1 && scores == s1);
}

}  // namespace

int main() {
  Rng r(2718);
  steps(r);
  for (int i = 0; i < 400; ++i) one_eviction(r);
  std::printf("ok\n");
  return 0;
}
