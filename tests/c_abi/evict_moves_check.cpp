// How moved rows are shared out to workgroups (csrc/kamera_evict_moves.h), on the CPU: of all the workgroups that a launch
// has, the surplus ones of a grid that is rounded up among them, each piece of work belongs to one, and the others have
// none. Exits 0 when all hold.
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <vector>

#include "kamera_evict_moves.h"

using namespace kamera;

#define CHECK(c)                                                        \
  do {                                                                  \
    if (!(c)) {                                                         \
      std::printf("%s:%d: %s failed\n", __FILE__, __LINE__, #c);        \
      std::exit(1);                                                     \
    }                                                                   \
  } while (0)

namespace {

struct Shape {
  int family, dtype, heads, dim, latent, rope, together, layers, seqs;
};

EvictArgs args_of(const Shape& s) {
  EvictArgs a;
  std::memset(&a, 0, sizeof(a));
  const int es = s.dtype == KAMERA_BF16 ? 2 : 4;
  const bool gqa = s.family == KAMERA_GQA;
  a.heads = gqa ? s.heads : 1;
  a.head_bytes = (gqa ? s.dim : s.latent + s.rope) * es;
  a.row_bytes = a.heads * a.head_bytes;
  a.tensors = gqa ? 2 : 1;
  a.together = s.together;
  a.layers = s.layers;
  a.num_seqs = s.seqs;
  a.dtype = s.dtype;
  a.d_rot = gqa ? s.dim : s.rope;
  a.band0 = gqa ? 0 : s.latent;
  a.most_kept = 1;
  a.shifts = 2;
  a.phase = reinterpret_cast<float*>(uintptr_t(1) << 40);
  return a;
}

// Workgroups that meet each piece of work of a move, one byte a piece
struct Met {
  const EvictArgs& a;
  const EvictMove& m;
  std::vector<unsigned char> times;
  Met(const EvictArgs& args, const EvictMove& move) : a(args), m(move), times((size_t)move.blocks, 0) {}
  void operator()(int64_t b) {
    EvictTask t;
    if (!evict_task(a, m, b, t)) return;
    const int groups = a.heads / a.together;
    CHECK(m.units > 0 && m.tensors > 0);
    CHECK(t.slice >= 0 && t.slice < m.slices && t.slice * m.slice < m.units && t.seq >= 0 && t.seq < a.num_seqs && t.group >= 0 && t.group < groups);
    CHECK(t.tensor >= m.tensor0 && t.tensor < m.tensor0 + m.tensors && t.tensor < a.tensors && t.layer >= 0 && t.layer < a.layers);
    const int64_t at = ((((int64_t)t.layer * m.tensors + t.tensor - m.tensor0) * groups + t.group) * a.num_seqs + t.seq) * m.slices + t.slice;
    CHECK(times[(size_t)at]++ == 0);
  }
  void all() {
    for (unsigned char x : times) CHECK(x == 1);
  }
};

void turned(const Shape& s) {
  const EvictArgs a = args_of(s);
  const EvictMoves m = evict_launches(a).moves;
  Met met[3] = {Met(a, m.turned), Met(a, m.plain0), Met(a, m.plain1)};
  const int64_t blocks = m.turned.blocks + m.plain0.blocks + m.plain1.blocks;
  CHECK(grid_blocks(blocks) >= blocks);
  for (int64_t n = 0; n < grid_blocks(blocks); ++n) {
    int64_t b = n;
    const int part = evict_part(m, b);
    if (part < 3) met[part](b);
  }
  for (Met& x : met) x.all();
}

void plain(const Shape& s, int tensor0, int tensors, int units) {
  const EvictArgs a = args_of(s);
  const EvictMove m = evict_move_of(a, tensor0, tensors, 0, units);
  Met met(a, m);
  for (int64_t b = 0; b < grid_blocks(m.blocks); ++b) met(b);
  met.all();
}

}  // namespace

int main() {
  const int G = KAMERA_GQA, M = KAMERA_MLA, B = KAMERA_BF16, F = KAMERA_F32;
  // a few workgroups; then just below and above one whole row of the grid (2^22), and above two
  turned(Shape{G, B, 8, 128, 0, 0, 2, 3, 5});
  turned(Shape{M, B, 1, 0, 512, 64, 1, 3, 5});
  turned(Shape{M, B, 1, 0, 0, 16, 1, 3, 5});
  turned(Shape{G, B, 4, 128, 0, 0, 1, 61, 5730});      // keys, and values in two slices: 61 * 5730 * 4 * 3
  turned(Shape{M, B, 1, 0, 512, 64, 1, 61, 7639});     // no values: 61 * 7639 * 9, 493 below
  turned(Shape{M, B, 1, 0, 512, 64, 1, 61, 7640});
  turned(Shape{M, B, 1, 0, 0, 16, 1, 3000, 1399});     // no latent either
  turned(Shape{M, B, 1, 0, 512, 64, 1, 1 << 14, 60});  // 8.8 million
  plain(Shape{G, B, 3, 10, 0, 0, 1, 2, 7}, 0, 2, 10);
  plain(Shape{G, F, 4, 128, 0, 0, 1, 70, 4000}, 0, 2, 32);
  plain(Shape{M, F, 1, 0, 20, 6, 1, 1 << 12, 1100}, 0, 1, 3);
  plain(Shape{M, F, 1, 0, 20, 6, 1, 1 << 12, 1100}, 0, 1, 0);
  std::printf("ok\n");
  return 0;
}
