// Eviction (include/kamera_step.h) for gfx950: which tokens stay, and their rows moved together.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kamera_evict_moves.h"

namespace kamera {

#define KGLOBAL __attribute__((address_space(1)))

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kWave = 64;

// Page and place in it of token t of a sequence.
__device__ __forceinline__ int64_t page_of(const EvictArgs& a, const EvictSeq& s, int t, int& place) {
  const int slot = s.slot0 + t;
  const int pg = (int)(((uint64_t)(uint32_t)slot * a.page_magic) >> a.page_bits);
  place = slot - pg * a.page_size;
  return ((const KGLOBAL int32_t*)a.pages)[s.pg + pg];
}

// ============================================================================
// Which tokens stay: a workgroup for each list (layer, group of heads, sequence). Scores become 32-bit
// numbers of the same order; the `want`-th highest of the tokens between the first and the last ones is
// found digit by digit (11, 11 and 10 bits, a count of each digit in LDS), then one pass in the tokens' order
// writes the numbers of those above it and of the first few equal to it. No order of atomics matters:
// counts are whole numbers. Lists of up to kSelect * 16 tokens stay in registers: all scores are read before any
// is written, so they move in the last pass. Bound by the waits between the passes (with 4 copies of the counts against
// conflicts 71 instead of 67 us): 28 layers x 4 heads of
// 1500 tokens in 9.3 us, 12 x 8 x 16 lists of 1000 to 8000 in 56 (67 with turns behind the list's end).
// 4, 16 or no scores of a thread held, whole calls in us (28 layers, 4 heads): 1500 tokens 45, 52 and 49; 2100 tokens
// -, 64 and 63; 4000 -, 104 and 109; 8000 -, 190 and 211.
// ============================================================================
constexpr int kSelect = 512;   // threads
constexpr int kDigits = 2048;
constexpr int kEach = 4;       // tokens of a thread in one turn of the last pass
constexpr int kHeldFew = 4, kHeldMost = 16;  // scores of a thread

__device__ __forceinline__ uint32_t rank_of(float x) {
  if (x != x) return 0;
  const uint32_t u = __float_as_uint(x + 0.0f);  // (-0 becomes 0)
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

struct List {
  EvictSeq seq;
  const KGLOBAL float* scores;  // of the layer, from the group's first head on
  __device__ __forceinline__ int64_t score_at(const EvictArgs& a, int t) const {
    int place;
    const int64_t page = page_of(a, seq, t, place);
    return page * a.heads * a.page_size + place;
  }
  __device__ __forceinline__ float score(const EvictArgs& a, int t) const {
    const KGLOBAL float* p = scores + score_at(a, t);
    float x = p[0];
    for (int h = 1; h < a.together; ++h) x += p[(int64_t)h * a.page_size];
    return x;
  }
  __device__ __forceinline__ uint32_t rank(const EvictArgs& a, int t) const { return rank_of(score(a, t)); }
};

__device__ __forceinline__ int wave_prefix(uint64_t mask) { return __popcll(mask & ((uint64_t(1) << (threadIdx.x & 63)) - 1)); }

// HELD > 0: token (wave * turns + i) * 64 + lane of the list is score i of its thread; 0: every pass reads them anew.
template <int HELD>
__device__ __forceinline__ void select_list(const EvictArgs& a, const List& l, KGLOBAL int32_t* kept, KGLOBAL int32_t* start, int keep) {
  __shared__ uint32_t count[kDigits];
  __shared__ int sums[kSelect / kWave][2];
  __shared__ int found[2];
  __shared__ int gone;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n = l.seq.num_tokens, lo = l.seq.first, hi = n - l.seq.last;  // ranked: [lo, hi)
  const int turns = HELD ? (n + kSelect - 1) / kSelect : 0;
  float held[HELD ? HELD : 1];
  auto token = [&](int i) { return (wave * turns + i) * kWave + lane; };
  auto ranked_one = [&](int i) { return i < turns && token(i) < hi && token(i) >= lo; };
  if constexpr (HELD != 0) {
    int64_t at[HELD];
#pragma unroll
    for (int i = 0; i < HELD; ++i) at[i] = l.score_at(a, min(token(min(i, turns - 1)), n - 1));
#pragma unroll
    for (int i = 0; i < HELD; ++i) held[i] = l.scores[at[i]];
    for (int h = 1; h < a.together; ++h) {
      float x[HELD];
#pragma unroll
      for (int i = 0; i < HELD; ++i) x[i] = l.scores[at[i] + (int64_t)h * a.page_size];
#pragma unroll
      for (int i = 0; i < HELD; ++i) held[i] += x[i];
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // (read, also where no rank is needed, before others write)
  }
  int want = keep - l.seq.first - l.seq.last;
  uint32_t border = 0, known = 0;  // bits of the border's rank found so far
  for (int pass = 0; pass < 3 && want > 0; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
    for (int i = tid; i < kDigits; i += kSelect) count[i] = 0;
    __syncthreads();
    auto add = [&](uint32_t r) {
      if ((r & known) == border) atomicAdd(&count[(r >> shift) & ((1u << bits) - 1)], 1u);
    };
    if constexpr (HELD != 0) {
#pragma unroll
      for (int i = 0; i < HELD; ++i) {
        if (i >= turns) break;
        if (ranked_one(i)) add(rank_of(held[i]));
      }
    } else {
      for (int t = lo + tid; t < hi; t += kSelect) add(l.rank(a, t));
    }
    __syncthreads();
    // the digit at which the counts from the highest on reach `want`
    constexpr int PER = kDigits / kSelect;
    int mine = 0;
    for (int i = 0; i < PER; ++i) mine += (int)count[kDigits - 1 - (tid * PER + i)];
    int up = mine;  // inclusive sum over the wave
    for (int d = 1; d < kWave; d <<= 1) {
      const int y = __shfl_up(up, d, kWave);
      if (lane >= d) up += y;
    }
    if (lane == 63) sums[wave][0] = up;
    __syncthreads();
    for (int w = 0; w < wave; ++w) up += sums[w][0];
    int before = up - mine;
    if (before < want && up >= want)
      for (int i = 0; i < PER; ++i) {
        const int digit = kDigits - 1 - (tid * PER + i), c = (int)count[digit];
        if (before < want && before + c >= want) {
          found[0] = digit;
          found[1] = want - before;
        }
        before += c;
      }
    __syncthreads();
    border |= (uint32_t)found[0] << shift;
    want = found[1];  // of those with the digit
    known |= ((1u << bits) - 1) << shift;
    __syncthreads();
  }
  const bool ranked = known != 0;
  // tokens that stay, in their order
  if (tid == 0) gone = n;
  int above = 0, equal = 0;  // of the turns before
  const bool with = HELD != 0 && a.together == 1;  // scores move with their tokens here
  KGLOBAL float* scores = (KGLOBAL float*)(float*)l.scores;
  constexpr int EACH = HELD ? HELD : kEach;
  for (int t0 = 0; t0 < n; t0 += kSelect * EACH) {  // (HELD: once)
    const int each = HELD ? turns : kEach;
    // whether the thread's token i is above the border (or stays whatever its score), or equal to it
    auto judge = [&](int i, bool& hit, bool& tie) {
      const int t = t0 + (wave * each + i) * kWave + lane;
      const bool there = t < n && (!HELD || i < turns);
      hit = there && (t < lo || t >= hi);
      tie = false;
      if (ranked && there && t >= lo && t < hi) {
        const uint32_t r = HELD ? rank_of(held[HELD ? i : 0]) : l.rank(a, t);
        hit = r > border;
        tie = r == border;
      }
    };
    int a0 = 0, e0 = 0;
    uint32_t hits = 0, equals = 0;
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      if (HELD && i >= turns) break;
      bool hit, tie;
      judge(i, hit, tie);
      hits |= (uint32_t)hit << i;
      equals |= (uint32_t)tie << i;
      a0 += __popcll(__ballot(hit));
      e0 += __popcll(__ballot(tie));
    }
    __syncthreads();
    if (lane == 0) {
      sums[wave][0] = a0;
      sums[wave][1] = e0;
    }
    __syncthreads();
    int abase = above, ebase = equal;
    for (int w = 0; w < kSelect / kWave; ++w) {
      if (w < wave) {
        abase += sums[w][0];
        ebase += sums[w][1];
      }
      above += sums[w][0];
      equal += sums[w][1];
    }
    int leaves = n;
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      if (HELD && i >= turns) break;
      const int t = t0 + (wave * each + i) * kWave + lane;
      const bool hit = hits >> i & 1, tie = equals >> i & 1;
      const uint64_t h = __ballot(hit), e = __ballot(tie);
      const int before = ebase + wave_prefix(e), j = abase + wave_prefix(h) + min(before, want);
      if (hit || (tie && before < want)) {
        kept[j] = t;
        if (with && j != t) scores[l.score_at(a, j)] = held[HELD ? i : 0];
      } else if (t < n && (!HELD || i < turns)) {
        leaves = min(leaves, t);
      }
      abase += __popcll(h);
      ebase += __popcll(e);
    }
    for (int d = 32; d; d >>= 1) leaves = min(leaves, __shfl_xor(leaves, d, kWave));
    if (lane == 0 && leaves < n) atomicMin(&gone, leaves);
  }
  __syncthreads();  // (the list is written, and visible to the workgroup)
  const int s0 = min(gone, keep);
  if (tid == 0) *start = s0;
  if (with) return;
  // The scores move with their tokens: a turn's reads are over before its writes begin, and later turns read
  // from places that earlier ones do not write, as token kept[j] >= j.
  for (int h = 0; h < a.together; ++h)
    for (int j0 = s0; j0 < keep; j0 += kSelect * kEach) {
      float x[kEach];
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int j = j0 + i * kSelect + tid;
        if (j < keep) x[i] = scores[l.score_at(a, kept[j]) + (int64_t)h * a.page_size];
      }
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int j = j0 + i * kSelect + tid;
        if (j < keep) scores[l.score_at(a, j) + (int64_t)h * a.page_size] = x[i];
      }
    }
}

template <int HELD>
__global__ __launch_bounds__(kSelect) void evict_select(EvictArgs a) {
  const int groups = a.heads / a.together, tid = threadIdx.x;
  int64_t b = block_number();
  const int si = (int)(b % a.num_seqs);
  b /= a.num_seqs;
  const int group = (int)(b % groups), layer = (int)(b / groups);
  if (layer >= a.layers) return;
  List l;
  l.seq = a.seqs[si];
  l.scores = (const KGLOBAL float*)a.scores + layer * a.scores_stride + (int64_t)group * a.together * a.page_size;
  const int n = l.seq.num_tokens, keep = min(l.seq.keep, n);
  KGLOBAL int32_t* kept = (KGLOBAL int32_t*)a.kept + ((int64_t)layer * groups + group) * a.total + l.seq.kept0;
  KGLOBAL int32_t* start = (KGLOBAL int32_t*)a.starts + ((int64_t)layer * groups + group) * a.num_seqs + si;
  if (keep == n || keep == 0) {
    for (int j = tid; j < keep; j += kSelect) kept[j] = j;
    if (tid == 0) *start = keep;
    return;
  }
  select_list<HELD>(a, l, kept, start, keep);
}

// cos/sin of turning back by t positions, formed in fp64 and rounded once
__global__ __launch_bounds__(kEvictPhases) void evict_phase(EvictArgs a) {
  const int half = a.d_rot >> 1;
  const int64_t i = (int64_t)block_number() * kEvictPhases + threadIdx.x, t = i / half;
  if (t >= a.shifts) return;
  const int p = (int)(i - t * half);
  double s, c;
  sincos(-(double)t * ((const KGLOBAL double*)a.theta)[p], &s, &c);
  a.phase[t * a.d_rot + p] = (float)c;
  a.phase[t * a.d_rot + half + p] = (float)s;
}

// ============================================================================
// Moves the kept rows together: a workgroup for each list, tensor and slice of the group's columns walks the
// list in turns of `side` x kTurn rows. All reads of a turn are over before its writes begin; a later turn's rows lie
// behind every row written so far (kept[j] >= j, ascending), so no other order is needed.
//
// K rows that are anchored anew from token i at j are turned by -(i - j) theta, in fp32 with cosines from fp64, rounded once.
//
// Bound by HBM: each moved row is read and written once. 16 sequences of 1000 to 8000 tokens, half of them kept, 12 layers of
// 8 heads of 128: 709 us for 2.9 GB, 4.1 TB/s. Slices of 128 bytes (8 pieces of 16), 8 rows a thread and turn: a cache line
// a row and slice, and enough workgroups; with rows looked up a turn ahead and passed by the caches 1090 -> 785 us the
// whole call. Slices of 64, 256 and 512 bytes, turns of 2, 4 and 16 rows, and cached stores were all slower.
// ============================================================================
constexpr int kMove = 256;  // threads
constexpr int kTurn = 8;    // rows of a thread in one turn

// Columns as they are, in pieces of a U.
template <typename U>
struct Plain {
  typedef U Held;
  static __device__ __forceinline__ void read(const EvictArgs&, const KGLOBAL char* row, int unit, Held& x) { x = __builtin_nontemporal_load((const KGLOBAL U*)row + unit); }
  static __device__ __forceinline__ void write(const EvictArgs&, KGLOBAL char* row, int unit, const Held& x, int) { __builtin_nontemporal_store(x, (KGLOBAL U*)row + unit); }
};

template <typename T>
__device__ __forceinline__ float wide(T x);
template <>
__device__ __forceinline__ float wide<uint16_t>(uint16_t x) {
  return __uint_as_float((uint32_t)x << 16);
}
template <>
__device__ __forceinline__ float wide<float>(float x) {
  return x;
}
template <typename T>
__device__ __forceinline__ T rounded(float x);
template <>
__device__ __forceinline__ uint16_t rounded<uint16_t>(float x) {
  return __builtin_bit_cast(uint16_t, (__bf16)x);  // to nearest even
}
template <>
__device__ __forceinline__ float rounded<float>(float x) {
  return x;
}

// Pairs of rotated columns, one a unit; `units` of them make a head, whose columns lie side by side.
template <typename T>
struct Turned {
  struct Held {
    T a, b;
  };
  static __device__ __forceinline__ void places(const EvictArgs& a, int unit, int& p, int& i, int& j) {
    const int half = a.d_rot >> 1, head = unit / half;
    p = unit - head * half;
    const int c0 = head * (a.head_bytes / (int)sizeof(T));
    i = c0 + (a.pairing == KAMERA_NEOX ? p : 2 * p);
    j = a.pairing == KAMERA_NEOX ? i + half : i + 1;
  }
  static __device__ __forceinline__ void read(const EvictArgs& a, const KGLOBAL char* row, int unit, Held& x) {
    int p, i, j;
    places(a, unit, p, i, j);
    x.a = ((const KGLOBAL T*)row)[i];
    x.b = ((const KGLOBAL T*)row)[j];
  }
  static __device__ __forceinline__ void write(const EvictArgs& a, KGLOBAL char* row, int unit, const Held& x, int back) {
    int p, i, j;
    places(a, unit, p, i, j);
    const KGLOBAL float* cs = (const KGLOBAL float*)a.phase + (int64_t)back * a.d_rot;
    const float c = cs[p], s = cs[(a.d_rot >> 1) + p], xa = wide<T>(x.a), xb = wide<T>(x.b);
    ((KGLOBAL T*)row)[i] = rounded<T>(xa * c - xb * s);
    ((KGLOBAL T*)row)[j] = rounded<T>(xa * s + xb * c);
  }
};

// The same for bf16 bands of 16 * n columns in 16-byte pieces: 8 pairs a unit, in two pieces (NeoX: of either half;
// GPT-J: side by side). (27 layers of 576 columns, 8 sequences: 354 us, pair by pair in a launch of their own 432.)
struct TurnedPieces {
  struct Held {
    u32x4 a, b;
  };
  static __device__ __forceinline__ void places(const EvictArgs& a, int unit, int& p, int& i, int& j) {
    const int units = a.d_rot >> 4, head = unit / units;
    p = unit - head * units;
    const int c0 = head * (a.head_bytes / 16);
    i = c0 + (a.pairing == KAMERA_NEOX ? p : 2 * p);
    j = a.pairing == KAMERA_NEOX ? i + units : i + 1;
  }
  static __device__ __forceinline__ void read(const EvictArgs& a, const KGLOBAL char* row, int unit, Held& x) {
    int p, i, j;
    places(a, unit, p, i, j);
    x.a = __builtin_nontemporal_load((const KGLOBAL u32x4*)row + i);
    x.b = __builtin_nontemporal_load((const KGLOBAL u32x4*)row + j);
  }
  static __device__ __forceinline__ void write(const EvictArgs& a, KGLOBAL char* row, int unit, const Held& x, int back) {
    int p, i, j;
    places(a, unit, p, i, j);
    const KGLOBAL f32x4* cs = (const KGLOBAL f32x4*)((const KGLOBAL float*)a.phase + (int64_t)back * a.d_rot) + 2 * p;
    const KGLOBAL f32x4* sn = cs + (a.d_rot >> 3);
    float f[16];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[2 * e] = __uint_as_float(x.a[e] << 16);
      f[2 * e + 1] = __uint_as_float(x.a[e] & 0xffff0000u);
      f[8 + 2 * e] = __uint_as_float(x.b[e] << 16);
      f[8 + 2 * e + 1] = __uint_as_float(x.b[e] & 0xffff0000u);
    }
    const f32x4 c[2] = {cs[0], cs[1]}, s[2] = {sn[0], sn[1]};
    const bool neox = a.pairing == KAMERA_NEOX;
    float y[16];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const float co = c[q >> 2][q & 3], si = s[q >> 2][q & 3];
      const float u = neox ? f[q] : f[2 * q], v = neox ? f[8 + q] : f[2 * q + 1];
      const float yu = u * co - v * si, yv = u * si + v * co;
      if (neox) {
        y[q] = yu;
        y[8 + q] = yv;
      } else {
        y[2 * q] = yu;
        y[2 * q + 1] = yv;
      }
    }
    u32x4 w[2];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e >> 2][e & 3] = (uint32_t)rounded<uint16_t>(y[2 * e]) | ((uint32_t)rounded<uint16_t>(y[2 * e + 1]) << 16);
    __builtin_nontemporal_store(w[0], (KGLOBAL u32x4*)row + i);
    __builtin_nontemporal_store(w[1], (KGLOBAL u32x4*)row + j);
  }
};

template <typename C>
__device__ __forceinline__ void move_rows(const EvictArgs& a, const EvictMove& m, int64_t b) {
  EvictTask task;
  if (!evict_task(a, m, b, task)) return;
  const int groups = a.heads / a.together, tid = threadIdx.x;
  const int slice = task.slice, si = task.seq, group = task.group, tensor = task.tensor, layer = task.layer;
  const EvictSeq seq = a.seqs[si];
  const int keep = min(seq.keep, seq.num_tokens);
  if (keep == seq.num_tokens) return;
  const int64_t list = (int64_t)layer * groups + group;
  const int start = ((const KGLOBAL int32_t*)a.starts)[list * a.num_seqs + si];
  const KGLOBAL int32_t* kept = (const KGLOBAL int32_t*)a.kept + list * a.total + seq.kept0;
  KGLOBAL char* pool = (KGLOBAL char*)(a.pool[tensor] + layer * a.layer_bytes + (int64_t)group * a.together * a.head_bytes + m.at);
  const int width = min(m.slice, m.units - slice * m.slice);  // units of this slice
  const int side = kMove / m.slice;                            // rows side by side
  const int row = tid / m.slice, in = tid - row * m.slice, unit = slice * m.slice + in;
  const bool mine = row < side && in < width;
  // A turn's rows are looked up while the turn before is on its way.
  typename C::Held x[kTurn];
  int from[kTurn], ahead[kTurn];
  int64_t src[kTurn], dst[kTurn];
  auto ask = [&](int j0, int (&f)[kTurn]) {
#pragma unroll
    for (int i = 0; i < kTurn; ++i) f[i] = kept[min(j0 + i * side + row, keep - 1)];
  };
  auto find = [&](int j0) {
#pragma unroll
    for (int i = 0; i < kTurn; ++i) {
      int place;
      from[i] = ahead[i];
      const int64_t page = page_of(a, seq, from[i], place);
      src[i] = (page * a.page_size + place) * a.row_bytes;
    }
  };
  if (start >= keep) return;
  ask(start, ahead);
  find(start);
  for (int j0 = start; j0 < keep; j0 += side * kTurn) {
    const int next = j0 + side * kTurn;
#pragma unroll
    for (int i = 0; i < kTurn; ++i)
      if (mine && j0 + i * side + row < keep) C::read(a, pool + src[i], unit, x[i]);
    int back[kTurn];
#pragma unroll
    for (int i = 0; i < kTurn; ++i) {
      const int j = min(j0 + i * side + row, keep - 1);
      int place;
      const int64_t page = page_of(a, seq, j, place);
      dst[i] = (page * a.page_size + place) * a.row_bytes;
      back[i] = from[i] - j;
    }
    if (next < keep) {
      ask(next, ahead);
      find(next);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kTurn; ++i)
      if (mine && j0 + i * side + row < keep) C::write(a, pool + dst[i], unit, x[i], back[i]);
  }
}

template <typename C>
__global__ __launch_bounds__(kMove) void evict_move(EvictArgs a, EvictMove m) {
  move_rows<C>(a, m, block_number());
}

// Turned columns and the others, in one launch.
__global__ __launch_bounds__(kMove) void evict_move_turned(EvictArgs a, EvictMoves m) {
  int64_t b = block_number();
  const int part = evict_part(m, b);
  if (part == 0) move_rows<TurnedPieces>(a, m.turned, b);
  else if (part == 1) move_rows<Plain<u32x4>>(a, m.plain0, b);
  else if (part == 2) move_rows<Plain<u32x4>>(a, m.plain1, b);
}

template <typename C>
void move(const EvictArgs& a, const EvictMove& m, hipStream_t stream) {
  if (m.blocks > 0) hipLaunchKernelGGL((evict_move<C>), grid_of(m.blocks), dim3(kMove), 0, stream, a, m);
}

}  // namespace

hipError_t launch_evict(const EvictArgs& a, hipStream_t stream) {
  const EvictLaunches l = evict_launches(a);
  if (a.longest <= kSelect * kHeldFew) hipLaunchKernelGGL(evict_select<kHeldFew>, grid_of(l.lists), dim3(kSelect), 0, stream, a);
  else if (a.longest <= kSelect * kHeldMost) hipLaunchKernelGGL(evict_select<kHeldMost>, grid_of(l.lists), dim3(kSelect), 0, stream, a);
  else hipLaunchKernelGGL(evict_select<0>, grid_of(l.lists), dim3(kSelect), 0, stream, a);
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && l.phases > 0) {
    hipLaunchKernelGGL(evict_phase, grid_of(l.phases), dim3(kEvictPhases), 0, stream, a);
    e = hipGetLastError();
  }
  if (e == hipSuccess && l.together) {
    hipLaunchKernelGGL(evict_move_turned, grid_of(l.moves.turned.blocks + l.moves.plain0.blocks + l.moves.plain1.blocks), dim3(kMove), 0, stream, a, l.moves);
    e = hipGetLastError();
  }
  for (int i = 0; i < l.parts && e == hipSuccess; ++i) {
    if (l.columns[i] == EVICT_BY_16) move<Plain<u32x4>>(a, l.part[i], stream);
    else if (l.columns[i] == EVICT_BY_4) move<Plain<uint32_t>>(a, l.part[i], stream);
    else if (l.columns[i] == EVICT_BY_2) move<Plain<uint16_t>>(a, l.part[i], stream);
    else if (a.dtype == KAMERA_BF16) move<Turned<uint16_t>>(a, l.part[i], stream);
    else move<Turned<float>>(a, l.part[i], stream);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace kamera
