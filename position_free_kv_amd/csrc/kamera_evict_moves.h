// How the rows that an eviction moves are shared out to workgroups (kernels: kamera_evict.hip).
#pragma once

#include <hip/hip_runtime.h>

#include "kamera_grid.h"
#include "kamera_step_desc.h"

namespace kamera {

constexpr int kSlice = 8;  // units of a slice, at most

// A part of what a launch moves: `tensors` of the pool from tensor0 on, columns from byte `at` of a group on, `units`
// units of them in slices of `slice`; its workgroups.
struct EvictMove {
  int tensor0, tensors, at, units, slice, slices;
  int64_t blocks;
};

inline EvictMove evict_move_of(const EvictArgs& a, int tensor0, int tensors, int at, int units) {
  EvictMove m{tensor0, tensors, at, units, units < kSlice ? units : kSlice, 1, 0};
  if (units > 0) m.slices = (units + m.slice - 1) / m.slice;
  if (units > 0) m.blocks = (int64_t)a.layers * tensors * (a.heads / a.together) * a.num_seqs * m.slices;
  return m;
}

// What workgroup b of a move walks over: a list's rows, in a slice of their columns of one tensor. false: the move has no
// workgroup of that number (a grid's surplus, or a move of nothing, which may have no tensors to divide by).
struct EvictTask {
  int slice, seq, group, tensor, layer;
};
__host__ __device__ inline bool evict_task(const EvictArgs& a, const EvictMove& m, int64_t b, EvictTask& t) {
  if (b >= m.blocks) return false;
  const int groups = a.heads / a.together;
  t.slice = (int)(b % m.slices);
  b /= m.slices;
  t.seq = (int)(b % a.num_seqs);
  b /= a.num_seqs;
  t.group = (int)(b % groups);
  b /= groups;
  t.tensor = m.tensor0 + (int)(b % m.tensors);
  t.layer = (int)(b / m.tensors);
  return true;
}

// Turned columns and the others, in one launch: their workgroups one after the other, then the grid's surplus. Number b of
// the launch becomes its number in a move: 0, 1 or 2; 3: it has no work.
struct EvictMoves {
  EvictMove turned, plain0, plain1;
};
__host__ __device__ inline int evict_part(const EvictMoves& m, int64_t& b) {
  if (b < m.turned.blocks) return 0;
  if ((b -= m.turned.blocks) < m.plain0.blocks) return 1;
  return (b -= m.plain0.blocks) < m.plain1.blocks ? 2 : 3;
}

// The launches of an eviction: lists, cosines, then the rows. How columns are read and written:
enum EvictColumns { EVICT_BY_16, EVICT_BY_4, EVICT_BY_2, EVICT_PAIRS };  // as they are, in pieces of so many bytes; turned pair by pair
struct EvictLaunches {
  int64_t lists, phases;  // workgroups of the selection, of the cosines
  bool together;          // all rows in one launch, turned ones in 16-byte pieces (`moves`); otherwise:
  EvictMoves moves;
  int parts;              // a launch each
  EvictMove part[3];
  EvictColumns columns[3];
};
constexpr int kEvictPhases = 256;  // cosines of a workgroup

inline EvictLaunches evict_launches(const EvictArgs& a) {
  EvictLaunches l{};
  const int es = a.dtype == KAMERA_BF16 ? 2 : 4, band = a.band0 * es, all = a.together * a.head_bytes;
  l.lists = (int64_t)a.layers * (a.heads / a.together) * a.num_seqs;
  if (a.most_kept == 0) return l;  // nothing moves
  // columns [at, at + bytes) of every group of some tensors, in units of `unit` bytes?
  auto fits = [&](int tensor0, int tensors, int at, int bytes, int unit) {
    bool ok = at % unit == 0 && bytes % unit == 0 && a.row_bytes % unit == 0 && a.layer_bytes % unit == 0 && all % unit == 0;
    for (int t = tensor0; t < tensor0 + tensors; ++t) ok = ok && (uintptr_t)a.pool[t] % (uintptr_t)unit == 0;
    return ok;
  };
  auto plain = [&](int tensor0, int tensors, int at, int bytes) {  // those columns as they are
    const int unit = fits(tensor0, tensors, at, bytes, 16) ? 16 : fits(tensor0, tensors, at, bytes, 4) ? 4 : 2;
    l.columns[l.parts] = unit == 16 ? EVICT_BY_16 : unit == 4 ? EVICT_BY_4 : EVICT_BY_2;
    l.part[l.parts++] = evict_move_of(a, tensor0, tensors, at, bytes / unit);
  };
  if (!a.phase) {
    plain(0, a.tensors, 0, all);
    return l;
  }
  l.phases = ((int64_t)a.shifts * (a.d_rot / 2) + kEvictPhases - 1) / kEvictPhases;
  l.together = es == 2 && a.d_rot % 16 == 0 && a.head_bytes % 16 == 0 && band % 16 == 0 && fits(0, a.tensors, 0, all, 16);
  if (l.together) {
    l.moves = EvictMoves{evict_move_of(a, 0, 1, band, a.together * (a.d_rot / 16)), evict_move_of(a, 0, 1, 0, band / 16),
                         evict_move_of(a, 1, a.tensors - 1, 0, all / 16)};
    return l;
  }
  plain(0, 1, 0, band);
  l.columns[l.parts] = EVICT_PAIRS;
  l.part[l.parts++] = evict_move_of(a, 0, 1, band, a.together * (a.d_rot / 2));
  if (a.tensors == 2) plain(1, 1, 0, all);
  return l;
}

// Workgroups of its largest launch.
inline int64_t evict_largest(const EvictLaunches& l) {
  int64_t n = l.lists > l.phases ? l.lists : l.phases;
  const int64_t together = l.moves.turned.blocks + l.moves.plain0.blocks + l.moves.plain1.blocks;
  n = together > n ? together : n;
  for (int i = 0; i < l.parts; ++i) n = l.part[i].blocks > n ? l.part[i].blocks : n;
  return n;
}

}  // namespace kamera
