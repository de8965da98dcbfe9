// Entry points of differential attention, weighing and eviction (include/kamera_step.h). Their plans are made
// with the other operators' (kamera_step_host.cpp); an eviction, like a list of page copies, has none.
#include <hip/hip_runtime.h>

#include "kamera_evict_moves.h"
#include "kamera_step_host.h"

using namespace kamera;

namespace {

struct EvictOffsets {
  size_t seqs, pages, theta, upload, starts, phase, kept, total;
};
struct EvictCounts {
  int64_t tokens = 0, entries = 0, kept = 0;
  int32_t longest = 0, most_kept = 0, shifts = 0;  // of the sequences that lose tokens
  // What the workspace has room for, so that one for longer sequences serves shorter ones: table entries wherever the
  // tokens begin in a page, and shifts (tokens that leave a sequence, and 0) however many stay
  int64_t room_entries = 0, room_shifts = 0;
};

int kv_heads(const kamera_layout* L) { return L->family == KAMERA_GQA ? L->num_kv_heads : 1; }
int rotary(const kamera_layout* L) { return L->family == KAMERA_GQA ? L->head_dim : L->rope_dim; }

kamera_status check_eviction(const kamera_layout* L, const kamera_eviction* e, EvictCounts& n) {
  kamera_status st = host_check_layout(L);
  if (st != KAMERA_OK) return st;
  if (!e) return host_fail(KAMERA_E_NULL, "eviction is NULL");
  if (e->num_seqs < 0) return host_fail(KAMERA_E_SHAPE, "num_seqs < 0");
  if (e->num_seqs && !e->seqs) return host_fail(KAMERA_E_NULL, "seqs is NULL");
  if (e->flags & ~(uint32_t)KAMERA_EVICT_REANCHOR) return host_fail(KAMERA_E_UNSUPPORTED, "eviction.flags 0x%x", e->flags);
  if (e->reserved) return host_fail(KAMERA_E_SHAPE, "eviction.reserved must be 0");
  if (e->heads_together < 1 || kv_heads(L) % e->heads_together)
    return host_fail(KAMERA_E_SHAPE, "heads_together %d does not divide %d KV heads", e->heads_together, kv_heads(L));
  const int P = L->page_size;
  for (int i = 0; i < e->num_seqs; ++i) {
    const kamera_evict_seq& s = e->seqs[i];
    if (s.num_tokens < 0 || s.keep < 0 || s.first < 0 || s.last < 0) return host_fail(KAMERA_E_SHAPE, "sequence %d: negative count", i);
    if (s.reserved) return host_fail(KAMERA_E_SHAPE, "sequence %d: reserved must be 0", i);
    if (s.num_tokens == 0) continue;
    if (!s.block_table) return host_fail(KAMERA_E_NULL, "sequence %d: block_table is NULL", i);
    if (s.slot0 < 0 || s.slot0 >= P) return host_fail(KAMERA_E_PAGE, "sequence %d: slot0 must be in [0, page_size)", i);
    if ((int64_t)s.slot0 + s.num_tokens >= kMaxSlot) return host_fail(KAMERA_E_SHAPE, "sequence %d: too many tokens", i);
    n.entries += table_entries(s.slot0, s.num_tokens, P);
    n.room_entries += table_entries(P - 1, s.num_tokens, P);
    n.room_shifts = std::max<int64_t>(n.room_shifts, (int64_t)s.num_tokens + 1);
    n.tokens += s.num_tokens;
    n.kept += std::min(s.keep, s.num_tokens);
    if (s.keep >= s.num_tokens) continue;
    if ((int64_t)s.first + s.last > s.keep)
      return host_fail(KAMERA_E_SHAPE, "sequence %d: first %d and last %d are more than keep %d", i, s.first, s.last, s.keep);
    n.longest = std::max(n.longest, s.num_tokens);
    n.most_kept = std::max(n.most_kept, s.keep);
    n.shifts = std::max(n.shifts, s.num_tokens - s.keep + 1);
  }
  if (n.kept >= kMaxSlot || n.entries >= kMaxSlot) return host_fail(KAMERA_E_SHAPE, "too many tokens");
  return KAMERA_OK;
}

EvictOffsets carve(const kamera_layout* L, const kamera_eviction* e, const EvictCounts& n) {
  EvictOffsets f;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += round_up(bytes, kAlign);
    return here;
  };
  const bool turn = e->flags & KAMERA_EVICT_REANCHOR;
  const int64_t lists = (int64_t)L->num_layers * (kv_heads(L) / e->heads_together);
  f.seqs = take((size_t)e->num_seqs * sizeof(EvictSeq));
  f.pages = take((size_t)n.room_entries * 4);
  f.theta = take(turn ? (size_t)rotary(L) / 2 * 8 : 0);
  f.upload = at;
  f.starts = take((size_t)(lists * e->num_seqs) * 4);
  f.phase = take(turn ? (size_t)n.room_shifts * rotary(L) * 4 : 0);
  f.kept = take(e->kept ? 0 : (size_t)(lists * n.kept) * 4);
  f.total = std::max<size_t>(at, kAlign);
  return f;
}

kamera_status evict(const kamera_layout* L, const kamera_pool* pool, const kamera_eviction* e, void* ws, size_t ws_bytes, hipStream_t stream) {
  EvictCounts n;
  kamera_status st = check_eviction(L, e, n);
  if (st == KAMERA_OK) st = check_pool(L, pool);
  if (st != KAMERA_OK) return st;
  const int P = L->page_size, heads = kv_heads(L);
  const int64_t layer_scores = (int64_t)pool->num_pages * P * heads;
  if (n.tokens && !e->scores) return host_fail(KAMERA_E_NULL, "scores is NULL");
  if (!aligned(e->scores, 4) || !aligned(e->kept, 4)) return host_fail(KAMERA_E_ALIGN, "scores and kept must be 4-byte aligned");
  if (e->scores_stride != 0 && e->scores_stride < layer_scores)
    return host_fail(KAMERA_E_SHAPE, "scores_stride %lld smaller than one layer (%lld)", (long long)e->scores_stride, (long long)layer_scores);
  for (int i = 0; i < e->num_seqs; ++i) {
    const kamera_evict_seq& s = e->seqs[i];
    const int64_t m = table_entries(s.slot0, s.num_tokens, P);
    for (int64_t k = 0; k < m; ++k)
      if (s.block_table[k] < 0 || s.block_table[k] >= pool->num_pages)
        return host_fail(KAMERA_E_PAGE, "sequence %d: block_table[%lld] = %d outside [0, %d)", i, (long long)k, s.block_table[k], pool->num_pages);
  }
  {
    SlotCheck check(pool->num_pages, P);
    for (int i = 0; i < e->num_seqs; ++i)
      if (!check.add(e->seqs[i].block_table, e->seqs[i].slot0, e->seqs[i].num_tokens))
        return host_fail(KAMERA_E_OVERLAP, "sequence %d: slots of page %d belong to another sequence too, or to it twice", i, check.clash);
  }
  const EvictOffsets f = carve(L, e, n);
  st = check_workspace(ws, ws_bytes, f.total);
  if (st != KAMERA_OK) return st;
  if (n.longest == 0 && !(e->kept && n.kept)) return KAMERA_OK;  // all tokens stay

  thread_local std::vector<unsigned char> blob;
  blob.assign(f.upload, 0);
  EvictSeq* seqs = reinterpret_cast<EvictSeq*>(blob.data() + f.seqs);
  int32_t* pages = reinterpret_cast<int32_t*>(blob.data() + f.pages);
  int64_t at = 0, kept = 0;
  for (int i = 0; i < e->num_seqs; ++i) {
    const kamera_evict_seq& s = e->seqs[i];
    const int64_t m = table_entries(s.slot0, s.num_tokens, P);
    if (m) std::memcpy(pages + at, s.block_table, (size_t)m * 4);
    seqs[i] = EvictSeq{(int32_t)at, s.slot0, s.num_tokens, s.keep, s.first, s.last, (int32_t)kept, 0};
    at += m;
    kept += std::min(s.keep, s.num_tokens);
  }
  const int d_rot = rotary(L);
  const bool turn = (e->flags & KAMERA_EVICT_REANCHOR) && n.shifts > 0;
  if (turn) {
    double* theta = reinterpret_cast<double*>(blob.data() + f.theta);
    for (int i = 0; i < d_rot / 2; ++i) theta[i] = std::pow(L->rope_base, -2.0 * i / d_rot);
  }
  EvictArgs a;
  std::memset(&a, 0, sizeof(a));
  char* base = static_cast<char*>(ws);
  const int es = (int)elem_bytes(L), F = row_width(L);
  a.pool[0] = static_cast<char*>(pool->k_pool);
  a.pool[1] = static_cast<char*>(pool->v_pool);
  a.layer_bytes = (pool->layer_stride ? pool->layer_stride : (int64_t)pool->num_pages * P * F) * es;
  a.scores = e->scores;
  a.scores_stride = e->scores_stride ? e->scores_stride : layer_scores;
  a.seqs = reinterpret_cast<const EvictSeq*>(base + f.seqs);
  a.pages = reinterpret_cast<const int32_t*>(base + f.pages);
  a.kept = e->kept ? e->kept : reinterpret_cast<int32_t*>(base + f.kept);
  a.starts = reinterpret_cast<int32_t*>(base + f.starts);
  a.phase = turn ? reinterpret_cast<float*>(base + f.phase) : nullptr;
  a.theta = reinterpret_cast<const double*>(base + f.theta);
  a.num_seqs = e->num_seqs;
  a.layers = L->num_layers;
  a.heads = heads;
  a.together = e->heads_together;
  a.total = (int32_t)n.kept;
  a.page_size = P;
  reciprocal(P, a.page_magic, a.page_bits);
  a.row_bytes = F * es;
  a.head_bytes = F / heads * es;
  a.tensors = L->family == KAMERA_GQA ? 2 : 1;
  a.dtype = L->dtype;
  a.d_rot = d_rot;
  a.band0 = L->family == KAMERA_GQA ? 0 : L->latent_dim;
  a.pairing = L->pairing;
  a.shifts = n.shifts;
  a.longest = n.longest;
  a.most_kept = n.most_kept;
  if (evict_largest(evict_launches(a)) >= int64_t(1) << 31) return host_fail(KAMERA_E_SHAPE, "too many layers, heads and sequences for one call");
  st = host_stage(blob.data(), f.upload, ws, stream);
  if (st != KAMERA_OK) return st;
  const hipError_t err = launch_evict(a, stream);
  if (err != hipSuccess) return host_fail(KAMERA_E_HIP, "eviction launch failed: %s", hipGetErrorString(err));
  return KAMERA_OK;
}

}  // namespace

extern "C" {

kamera_status kamera_step_attend_diff(const kamera_step_plan* plan, int32_t layer, const void* q, int64_t q_stride, void* out,
                                      int64_t out_stride, float* lse, float scale, const kamera_differential* diff, void* stream) {
  return guarded([&] {
    StepArgs a;
    kamera_status st = check_launch(plan, layer, KAMERA_STEP_ATTEND, a);
    if (st != KAMERA_OK) return st;
    if (!(plan->flags & KAMERA_STEP_DIFFERENTIAL)) return host_fail(KAMERA_E_UNSUPPORTED, "the step was not uploaded as a differential one");
    if (!diff) return host_fail(KAMERA_E_NULL, "diff is NULL");
    if (diff->flags & ~(uint32_t)KAMERA_DIFF_NORM) return host_fail(KAMERA_E_UNSUPPORTED, "diff.flags 0x%x", diff->flags);
    if (!std::isfinite(scale) || !std::isfinite(diff->lambda_init) || !std::isfinite(diff->out_scale))
      return host_fail(KAMERA_E_SHAPE, "scale, lambda_init and out_scale must be finite");
    if (!(diff->eps >= 0.0f) || !std::isfinite(diff->eps)) return host_fail(KAMERA_E_SHAPE, "eps must be >= 0 and finite");
    const size_t es = a.dtype == KAMERA_BF16 ? 2 : 4;
    // pairs of KV heads in the place of heads
    a.heads /= 2;
    a.group *= 2;
    a.dv *= 2;
    if (plan->num_tokens == 0) return KAMERA_OK;
    if ((st = check_rows("q", q, q_stride, (int64_t)a.num_q_heads * a.dk, es)) != KAMERA_OK) return st;
    if ((st = check_rows("out", out, out_stride, (int64_t)a.num_q_heads / 2 * a.dv, es)) != KAMERA_OK) return st;
    if (!aligned(lse, 4) || !aligned(diff->lambdas, 4)) return host_fail(KAMERA_E_ALIGN, "lse and lambdas must be 4-byte aligned");
    if (!aligned(diff->norm_weight, es)) return host_fail(KAMERA_E_ALIGN, "norm_weight must be aligned to %zu bytes", es);
    const hipError_t e = launch_step_attend_diff(a, layer, q, q_stride, out, out_stride, lse, scale, *diff, (hipStream_t)stream);
    if (e != hipSuccess) return host_fail(KAMERA_E_HIP, "attention launch failed: %s", hipGetErrorString(e));
    return KAMERA_OK;
  });
}

kamera_status kamera_step_weigh(const kamera_step_plan* plan, int32_t layer, const void* q, int64_t q_stride, const float* lse,
                                float* scores, float scale, float decay, void* stream) {
  return guarded([&] {
    StepArgs a;
    kamera_status st = check_launch(plan, layer, KAMERA_STEP_WEIGH, a);
    if (st != KAMERA_OK) return st;
    if (!std::isfinite(scale) || !std::isfinite(decay)) return host_fail(KAMERA_E_SHAPE, "scale and decay must be finite");
    if (plan->num_tokens == 0) return KAMERA_OK;
    if ((st = check_rows("q", q, q_stride, (int64_t)a.num_q_heads * a.dk, a.dtype == KAMERA_BF16 ? 2 : 4)) != KAMERA_OK) return st;
    if (!lse || !scores) return host_fail(KAMERA_E_NULL, "lse or scores is NULL");
    if (!aligned(lse, 4) || !aligned(scores, 4)) return host_fail(KAMERA_E_ALIGN, "lse and scores must be 4-byte aligned");
    const hipError_t e = launch_step_weigh(a, layer, q, q_stride, lse, scores, scale, decay, (hipStream_t)stream);
    if (e != hipSuccess) return host_fail(KAMERA_E_HIP, "weighing launch failed: %s", hipGetErrorString(e));
    return KAMERA_OK;
  });
}

size_t kamera_evict_workspace_bytes(const kamera_layout* layout, const kamera_eviction* eviction) {
  size_t bytes = 0;
  (void)guarded([&] {
    EvictCounts n;
    const kamera_status st = check_eviction(layout, eviction, n);
    if (st == KAMERA_OK) bytes = carve(layout, eviction, n).total;
    return st;
  });
  return bytes;
}

kamera_status kamera_evict(const kamera_layout* layout, const kamera_pool* pool, const kamera_eviction* eviction, void* workspace,
                           size_t workspace_bytes, void* stream) {
  return guarded([&] { return evict(layout, pool, eviction, workspace, workspace_bytes, (hipStream_t)stream); });
}

kamera_status kamera_scores_layout(const kamera_layout* layout, kamera_layout* scores) {
  return guarded([&] {
    const kamera_status st = host_check_layout(layout);
    if (st != KAMERA_OK) return st;
    if (!scores) return host_fail(KAMERA_E_NULL, "scores is NULL");
    // a token's share of its page is one fp32 a head, moved as two 2-byte columns
    kamera_layout s = *layout;
    s.family = KAMERA_MLA;
    s.dtype = KAMERA_BF16;
    s.num_kv_heads = s.head_dim = 0;
    s.latent_dim = 2 * kv_heads(layout) - 2;
    s.rope_dim = 2;
    for (int k = 0; k < 3; ++k) s.mrope_section[k] = 0;
    *scores = s;
    return KAMERA_OK;
  });
}

}  // extern "C"
