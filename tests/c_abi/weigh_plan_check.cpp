// Plans of weighing in workspaces of every size that is taken, on the CPU, with the stand-ins of step_host_check.cpp: the
// full size cuts the rows into ranges, the least one leaves them whole, for heads and latent rows of either type. Exits
// 0 when all hold.
#define main step_host_check_main
#include "step_host_check.cpp"
#undef main

namespace {
int g_items, g_joins;
int64_t g_rows;  // of all items, times their keys
}  // namespace

namespace kamera {
hipError_t launch_step_attend_diff(const StepArgs&, int, const void*, int64_t, void*, int64_t, float*, float, const kamera_differential&, hipStream_t) {
  return hipSuccess;
}
hipError_t launch_step_weigh(const StepArgs& a, int, const void*, int64_t, const float*, float*, float, float, hipStream_t) {
  g_items = a.num_weigh;
  g_joins = a.num_weigh_join;
  g_rows = 0;
  for (int i = 0; i < a.num_weigh; ++i) {
    const WeighItem& it = a.weigh[i];
    CHECK(it.part < 0 || a.num_weigh_join > 0);
    g_rows += (int64_t)(it.row1 - it.row0) * (it.kv1 - it.kv0);
  }
  return hipSuccess;
}
hipError_t launch_evict(const EvictArgs&, hipStream_t) { return hipSuccess; }
}  // namespace kamera

int main() {
  struct Kind {
    int family, dtype, heads, dim;
  };
  for (const Kind& k : {Kind{KAMERA_GQA, KAMERA_BF16, 14, 64}, Kind{KAMERA_GQA, KAMERA_BF16, 14, 80}, Kind{KAMERA_GQA, KAMERA_F32, 14, 64},
                        Kind{KAMERA_MLA, KAMERA_BF16, 16, 0}, Kind{KAMERA_MLA, KAMERA_F32, 16, 0}}) {
    kamera_layout L;
    std::memset(&L, 0, sizeof(L));
    L.family = k.family;
    L.dtype = k.dtype;
    L.num_layers = L.num_kv_heads = 1;
    L.head_dim = k.dim;
    L.latent_dim = 512;
    L.rope_dim = 64;
    L.page_size = 16;
    L.rope_base = 1e4;
    std::vector<int32_t> pages(100);
    for (int i = 0; i < 100; ++i) pages[(size_t)i] = i;
    kamera_request r[3];
    std::memset(r, 0, sizeof(r));
    const kamera_prefix pre{pages.data(), 0, 300};
    const int own[] = {200, 700, 30}, queries[] = {180, 120, 90}, at[] = {20, 33, 77};
    for (int i = 0; i < 3; ++i) {
      r[i].block_table = pages.data() + at[i];
      r[i].num_tokens = own[i];
      r[i].num_queries = queries[i];
      r[i].prefix = i == 2 ? -1 : 0;
    }
    kamera_step s;
    std::memset(&s, 0, sizeof(s));
    s.requests = r;
    s.num_requests = 3;
    s.prefixes = &pre;
    s.num_prefixes = 1;
    s.num_q_heads = k.heads;
    s.flags = KAMERA_STEP_WEIGH | KAMERA_STEP_FIT;
    kamera_pool pool;
    std::memset(&pool, 0, sizeof(pool));
    pool.k_pool = pool.v_pool = reinterpret_cast<char*>(uintptr_t(1) << 40);
    pool.num_pages = 100;
    const size_t full = kamera_step_workspace_bytes(&L, &s);
    Buffer ws(full);
    char* fake = reinterpret_cast<char*>(uintptr_t(1) << 40);
    int64_t rows = 0;
    bool whole = false, refused = false;
    for (size_t bytes = full / 256 * 256; bytes > 0; bytes -= 256) {
      kamera_step_plan p;
      const kamera_status st = kamera_step_upload(&L, &s, &pool, ws.p, bytes, nullptr, &p);
      if (st != KAMERA_OK) {
        CHECK(st == KAMERA_E_WORKSPACE);
        refused = true;
        break;
      }
      CHECK(kamera_step_weigh(&p, 0, fake, 0, (float*)fake, (float*)fake, 1.0f, 1.0f, nullptr) == KAMERA_OK);
      if (bytes == full / 256 * 256) {
        CHECK(g_joins > 0);
        rows = g_rows;
      }
      if (g_joins == 0) whole = true;
      CHECK((g_joins == 0) == whole);  // (the less room, the fewer ranges)
      CHECK(g_rows == rows);           // the same work
    }
    CHECK(whole && refused);
  }
  std::printf("ok\n");
  return 0;
}
