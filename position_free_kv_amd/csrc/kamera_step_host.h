// Host helpers of the serving step's entry points (kamera_step_host.cpp, kamera_evict_host.cpp).
#pragma once

#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>
#include <vector>

#include "kamera_step_desc.h"

namespace kamera {

namespace {

constexpr size_t kAlign = 256;
size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
size_t elem_bytes(const kamera_layout* L) { return L->dtype == KAMERA_BF16 ? 2 : 4; }

int row_width(const kamera_layout* L) {
  return L->family == KAMERA_GQA ? L->num_kv_heads * L->head_dim : L->latent_dim + L->rope_dim;
}

// slots and key numbers are 32-bit in the kernels, with room for a tile beyond the last
constexpr int64_t kMaxSlot = (int64_t(1) << 31) - 4096;

int64_t table_entries(int32_t slot0, int64_t tokens, int P) { return tokens > 0 ? ceil_div(slot0 + tokens, P) : 0; }

// x / d = x * magic >> bits for 0 <= x < 2^31: with b = ceil(log2 d), floor(2^(31 + b) / d) + 1 exceeds
// 2^(31 + b) / d by at most 2^b / (d 2^b), which the 31 bits of x cannot raise to a whole
void reciprocal(int d, uint32_t& magic, int32_t& bits) {
  bits = 31;
  while ((int64_t(1) << (bits - 31)) < d) ++bits;
  magic = (uint32_t)((uint64_t(1) << bits) / (uint64_t)d + 1);
}

// Finds slots that two sequences (or one twice) name, in time proportional to their page-table entries.
// Page ids are inside the pool.
struct SlotCheck {
  struct Use {
    int32_t lo, hi, next, page;  // slots of the page; another use of it
  };
  std::vector<int32_t>& head;  // per page: its latest use, -1 between checks
  std::vector<Use>& uses;
  const int P;
  int32_t clash = -1;
  SlotCheck(int32_t num_pages, int page_size) : head(heads()), uses(all()), P(page_size) {
    clear();  // (what an exception may have left)
    if (head.size() < (size_t)num_pages) head.resize((size_t)num_pages, -1);
  }
  ~SlotCheck() { clear(); }
  bool add(const int32_t* table, int32_t slot0, int64_t tokens) {
    const int64_t n = table_entries(slot0, tokens, P);
    for (int64_t k = 0; k < n; ++k) {
      const Use u{(int32_t)std::max<int64_t>(slot0 - k * P, 0), (int32_t)std::min<int64_t>(slot0 + tokens - k * P, P), head[(size_t)table[k]], table[k]};
      for (int32_t o = u.next; o >= 0; o = uses[(size_t)o].next)
        if (uses[(size_t)o].lo < u.hi && u.lo < uses[(size_t)o].hi) {
          clash = table[k];
          return false;
        }
      uses.push_back(u);
      head[(size_t)table[k]] = (int32_t)uses.size() - 1;
    }
    return true;
  }

 private:
  static std::vector<int32_t>& heads() {
    thread_local std::vector<int32_t> v;
    return v;
  }
  static std::vector<Use>& all() {
    thread_local std::vector<Use> v;
    return v;
  }
  void clear() {
    for (const Use& u : uses) head[(size_t)u.page] = -1;
    uses.clear();
  }
};

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

}  // namespace kamera
