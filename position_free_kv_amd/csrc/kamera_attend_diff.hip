// Differential attention over the paged pool (include/kamera_step.h): bf16 heads of 64 or 128 columns on the
// matrix cores (method and register layouts: kamera_attend.h; work list: kamera_step_desc.h), and the join of
// partial rows that makes an output row of its two maps, for any layout.
//
// The "head" of an item is a pair of KV heads: two keys of D columns a token, one value of 2 D columns. Rows
// of a run alternate between the maps (row = token's number * group + query head of the pair), and a wave takes
// 32 (or 16) rows of one map, so that a stage's values are brought into LDS once for both maps.
//
// Per pair, x = A0 V - lambda A1 V with A_e = softmax(scale q_e K_e^T), one pass over the keys with each map's running
// maximum and sum; y = x / sqrt(mean x^2 + eps) * weights * out_scale. The maps are combined, and the norm taken, in
// fp32 from sums in fp32; the weights are rounded to bf16 for the second product alone (at most 2^-8 of each), the output once.
// A query head and key cost 2 D + 4 D flops, half as much again as plain attention, for the same bytes of the pool.
//
// 8 requests with 2481 query tokens over an 8192-token prefix, 28 + 4 heads of 128: 0.93 PFLOP/s in this kernel (463
// GFLOP in 500 us; 0.8 on a slower machine), 76% of a large library product's rate; bound by the products and the
// softmax between them, which two waves a SIMD take in turn. 64 requests of one token over 8192 shared and 49300 own ones,
// 32 + 8 heads: 62 us and 12 in the join; bound by the own tokens' pages and by what a workgroup does before its first
// key (about 6 us).
#include <type_traits>

#include "kamera_attend.h"
#include "kamera_grid.h"

namespace kamera {

namespace {

constexpr int kWaveSize = 64;

// A stage of TS keys lies in four arrays of rows of 2 D bytes, one after the other: keys of the first map, of the
// second, first halves of the values, second halves. So one place in the pool's rows serves four loads.
template <int D>
constexpr int kRowBytes = 2 * D;
constexpr int kLds = 65536;

// N keys of a stage of TS from `first` on, by one wave. The page ids are asked for one stage ahead (find) and used only
// when the stage is loaded: loads return in order, so using them at once would wait for the stage in flight as well.
template <int D, int TS, int N, int ROWS>
struct PairRows {
  static constexpr int RPL = 1024 / kRowBytes<D>, LPR = 64 / RPL, NI = N / RPL;  // rows of an instruction, lanes of a row
  static_assert(N % RPL == 0, "whole instructions");
  int page[NI], place[NI];
  __device__ __forceinline__ void find(const StepArgs& a, const AttendRun& run, int t0, int first, int last) {
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));  // (see load)
#pragma unroll
    for (int i = 0; i < NI; ++i) page[i] = ((const KGLOBAL int32_t*)a.pages)[key_entry(a, run, min(t0 + first + i * RPL + lane / LPR, last), place[i])];
  }
  // k and v: the layer's rows from the pair's first column on
  __device__ __forceinline__ void load(const StepArgs& a, const uint16_t* k, const uint16_t* v, KLDS char* stage, int first) const {
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));  // what follows from it is made anew each stage: kept, it would cost the products registers
    const uint32_t row_bytes = 2u * (uint32_t)a.row;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      int pg = page[i];
      asm volatile("" : "+v"(pg));  // (the product stays here)
      const uint32_t row = (uint32_t)(pg * a.page_size + place[i]);  // (below 2^31)
      const uint32_t piece = (uint32_t)((lane & (LPR - 1)) ^ swz<ROWS, kRowBytes<D>>(first + i * RPL + lane / LPR)) << 4;
      const uint64_t at = (uint64_t)row * row_bytes + piece;
      KLDS char* to = stage + (first + i * RPL) * kRowBytes<D>;
#pragma unroll
      for (int x = 0; x < 4; ++x)
        __builtin_amdgcn_global_load_lds((const KGLOBAL void*)((const KGLOBAL char*)((x < 2 ? k : v) + (x & 1) * D) + at), (KLDS void*)(to + x * TS * kRowBytes<D>), 16, 0, 0);
    }
  }
};

__device__ __forceinline__ float wave_sum(float x) {
  for (int d = 32; d; d >>= 1) x += __shfl_xor(x, d, kWaveSize);
  return x;
}
template <typename T>
__device__ __forceinline__ float widened(T x) {
  if constexpr (sizeof(T) == 2) return __uint_as_float((uint32_t)x << 16);
  else return x;
}

// exp(q1 . k1) - exp(q2 . k2) + lambda_init, by one wave: its lanes' shares of the products, and what they make
__device__ __forceinline__ float2 lambda_products(const StepArgs& a, const kamera_differential& diff) {
  float2 d = make_float2(0.0f, 0.0f);
  if (!diff.lambdas) return d;
  const KGLOBAL float* p = (const KGLOBAL float*)diff.lambdas;
  for (int c = (int)threadIdx.x & 63; c < a.dk; c += kWaveSize) {
    d.x += p[c] * p[a.dk + c];
    d.y += p[2 * a.dk + c] * p[3 * a.dk + c];
  }
  return d;
}
__device__ __forceinline__ float lambda_from(const kamera_differential& diff, float2 d) {
  return diff.lambdas ? expf(wave_sum(d.x)) - expf(wave_sum(d.y)) + diff.lambda_init : diff.lambda_init;
}
// What a row x of `dv` columns is multiplied with, besides the weights, given its sum of squares.
__device__ __forceinline__ float norm_scale(const kamera_differential& diff, float squares, int dv) {
  if (!(diff.flags & KAMERA_DIFF_NORM)) return diff.out_scale;
  const float ms = squares / (float)dv + diff.eps;
  return ms == 0.0f ? 0.0f : diff.out_scale / sqrtf(ms);  // (zeros stay zeros)
}

// Results of a run that no other shares: the second map's wave passes its rows on through LDS at `place` (like lanes
// hold like values), the first map's makes the output. r: the row of the wave's own map. Every wave of the
// workgroup comes along; idle ones hold nothing.
template <typename S>
__device__ __forceinline__ void put_pairs(const StepArgs& a, const AttendIo& io, const kamera_differential& diff, const Lane& r, S& st, float l, int map,
                                          float lambda, f32x4* place, bool idle) {
  constexpr int kQuads = S::kScores / 4, ROWS = S::kScores == 16 ? 32 : 16;
  const int lane = threadIdx.x & 63;
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  if (io.lse && !idle && r.owned && S::group() == 0) io.lse[(int64_t)r.token * a.num_q_heads + r.qh] = l == 0.0f ? -INFINITY : (st.m + log2f(l)) * kLn2;
  __syncthreads();
  if (map == 1 && !idle) {
#pragma unroll
    for (int b = 0; b < S::kBlocks; ++b)
#pragma unroll
      for (int i = 0; i < kQuads; ++i)
        place[(b * kQuads + i) * 64 + lane] = (f32x4){st.o[b][4 * i] * inv, st.o[b][4 * i + 1] * inv, st.o[b][4 * i + 2] * inv, st.o[b][4 * i + 3] * inv};
  }
  __syncthreads();
  if (map == 1 || idle) return;
  float squares = 0.0f;
#pragma unroll
  for (int b = 0; b < S::kBlocks; ++b)
#pragma unroll
    for (int i = 0; i < kQuads; ++i) {
      __builtin_amdgcn_sched_barrier(0);  // (a few values at a time: registers are short)
      const f32x4 y = place[(b * kQuads + i) * 64 + lane];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = st.o[b][4 * i + e] * inv - lambda * y[e];
        st.o[b][4 * i + e] = x;
        squares += x * x;
      }
    }
  const float scale = norm_scale(diff, row_sum<ROWS>(squares), a.dv);
  if (!r.owned) return;
  uint16_t* out = (uint16_t*)io.out + (int64_t)r.token * io.out_stride + (int64_t)(r.qh >> 1) * a.dv;
  const KGLOBAL uint16_t* weights = (diff.flags & KAMERA_DIFF_NORM) ? (const KGLOBAL uint16_t*)diff.norm_weight : nullptr;
#pragma unroll
  for (int b = 0; b < S::kBlocks; ++b)
#pragma unroll
    for (int i = 0; i < kQuads; ++i) {
      __builtin_amdgcn_sched_barrier(0);
      const int c = S::column(b, i);
      float y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = st.o[b][4 * i + e] * scale * (weights ? widened<uint16_t>(weights[c + e]) : 1.0f);
      if (io.out_vec) {
        *(KGLOBAL u32x2*)(KGLOBAL void*)(out + c) = (u32x2){pack2(y[0], y[1]), pack2(y[2], y[3])};
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) out[c + e] = (uint16_t)pack2(y[e], 0.0f);
      }
    }
}

// ============================================================================
// Tiles of 128 rows: two waves a map, 32 rows each, share stages of 32 (D = 128) or 64 keys, two in LDS. A wave's 32 rows
// of 2 D columns of O are 128 registers (D = 128), its queries 32 more: 64 rows would leave one wave a SIMD. (All 256 are taken
// and 52 spilled, none among a stage's products; D = 64 takes 204.) One map a wave
// lets both maps share the values' stage, and LDS feeds 24 products of a stage's 32 keys from 24 KB a wave. Stages of
// four like arrays, one address for four loads: 689 -> 638 us in the case above; whole tiles for whole rounds of the chip's
// places (the planner's choice): 638 -> 520; results put out without partial rows where a run has no other: 520 -> 508.
// A ring of four stages whose loads take their places from a table in LDS: 526 -> 555 (more registers than there are).
// ============================================================================
template <int D>
__device__ __forceinline__ void wide_tile(const StepArgs& a, const AttendIo& io, const kamera_differential& diff, const AttendItem& it, int head,
                                          KLDS char* lds) {
  constexpr int TS = 4096 / D, N = TS / kWaves, NT = TS / 32;
  typedef State<D, 2 * D, 32, TS * kRowBytes<D>> S;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, map = wave & 1;
  const uint16_t* kp = a.k_pool + io.layer0 + head * 2 * D;
  const uint16_t* vp = a.v_pool + io.layer0 + head * 2 * D;
  const int first = wave * N, last = it.kv1 - 1;
  const bool any = it.kv1 > it.kv0;
  KLDS char* const stage[2] = {lds, lds + kLds / 2};
  PairRows<D, TS, N, 32> rows;
  if (any) {
    rows.find(a, it.run, it.kv0, first, last);
    rows.load(a, kp, vp, stage[0], first);
    rows.find(a, it.run, it.kv0 + TS, first, last);
  }
  const Lane r = lane_row(a, it, head, it.row0 + (wave >> 1) * 64 + 2 * (lane & 31) + map);
  const int end_min = __builtin_amdgcn_readfirstlane(r.end), end_max = __builtin_amdgcn_readlane(r.end, 31);
  bf16x8 q[S::kKSteps];
  S::load_q(io, r, q);
  S st;
  st.clear();
  auto work = [&](const KLDS char* s, int t) {
    const KLDS char* k = s + map * TS * kRowBytes<D>;
    walk<TS, NT>(st, q, k, k, s + 2 * TS * kRowBytes<D>, t, r.end, end_min, end_max, io.scale2);
  };
  if (any) {
    for (int t = it.kv0;;) {
      stage_barrier();
      if (t + TS < it.kv1) {
        rows.load(a, kp, vp, stage[1], first);
        rows.find(a, it.run, t + 2 * TS, first, last);
      }
      work(stage[0], t);
      if ((t += TS) >= it.kv1) break;
      stage_barrier();
      if (t + TS < it.kv1) {
        rows.load(a, kp, vp, stage[0], first);
        rows.find(a, it.run, t + 2 * TS, first, last);
      }
      work(stage[1], t);
      if ((t += TS) >= it.kv1) break;
    }
  }
  const float l = row_sum<32>(st.l);
  int tid = threadIdx.x;  // the row again: kept through the loop it would take registers from the products
  asm volatile("" : "+v"(tid));
  const Lane w = lane_row(a, it, head, it.row0 + (tid >> 7) * 64 + 2 * (tid & 31) + ((tid >> 6) & 1));
  static_assert(2 * 64 * S::kBlocks * S::kScores * 4 <= kLds, "two waves' results fit in LDS");
  if (it.run.direct) put_pairs(a, io, diff, w, st, l, map, lambda_from(diff, lambda_products(a, diff)), (f32x4*)(KLDS f32x4*)(lds + (wave >> 1) * (kLds / 2)), false);
  else put_state(a, io, it, head, w, st, l);
}

// ============================================================================
// Tiles of up to 64 rows (32: ROWS 16): a wave for each map and half of a stage of 64 (D = 128) or 128 keys. One
// buffer: the other workgroup of the CU computes while this one loads, and twice the bytes are on their way that two
// buffers of half the size would have. The halves are joined at the end.
// ============================================================================
template <int D, int ROWS>
__device__ __forceinline__ void narrow_tile(const StepArgs& a, const AttendIo& io, const kamera_differential& diff, const AttendItem& it, int head,
                                            KLDS char* lds, float (&ml)[2][kWaves][64]) {
  constexpr int TS = 8192 / D, N = TS / kWaves, HALF = TS / 2;
  typedef State<D, 2 * D, ROWS, TS * kRowBytes<D>> S;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), map = wave & 1, part = wave >> 1;
  const uint16_t* kp = a.k_pool + io.layer0 + head * 2 * D;
  const uint16_t* vp = a.v_pool + io.layer0 + head * 2 * D;
  const int first = wave * N, last = it.kv1 - 1;
  PairRows<D, TS, N, ROWS> rows;
  const bool any = it.kv1 > it.kv0;
  if (any) rows.find(a, it.run, it.kv0, first, last);
  Lane r = lane_row(a, it, head, it.row0 + 2 * S::row() + map);
  asm volatile("" : "+v"(r.token));  // (here: behind the stage's loads it would wait for them, and the queries after it)
  if (any) rows.load(a, kp, vp, lds, first);
  const int end_min = __builtin_amdgcn_readfirstlane(r.end), end_max = __builtin_amdgcn_readlane(r.end, ROWS - 1);
  bf16x8 q[S::kKSteps];
  S::load_q(io, r, q);
  S st;
  st.clear();
  for (int t = it.kv0; t < it.kv1; t += TS) {
    if (t + TS < it.kv1) rows.find(a, it.run, t + TS, first, last);
    stage_barrier();
    const KLDS char* k = (const KLDS char*)lds + (map * TS + part * HALF) * kRowBytes<D>;
    const KLDS char* v = (const KLDS char*)lds + (2 * TS + part * HALF) * kRowBytes<D>;
    walk<HALF, 1>(st, q, k, k, v, t + part * HALF, r.end, end_min, end_max, io.scale2);
    if (t + TS >= it.kv1) break;
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): read before it is overwritten
    __syncthreads();
    rows.load(a, kp, vp, lds, first);
  }
  float l = row_sum<ROWS>(st.l);
  static_assert(2 * 64 * S::kBlocks * S::kScores * 4 <= kLds, "two waves' results fit in LDS");
  join_two(st, l, part == 1, map, (f32x4*)(KLDS f32x4*)(lds + map * (kLds / 2)), ml);
  int tid = threadIdx.x;  // (as in the wide tile)
  asm volatile("" : "+v"(tid));
  const Lane w = lane_row(a, it, head, it.row0 + 2 * (tid & (ROWS - 1)) + ((tid >> 6) & 1));
  if (it.run.direct) put_pairs(a, io, diff, w, st, l, map, lambda_from(diff, lambda_products(a, diff)), (f32x4*)(KLDS f32x4*)lds, part == 1);
  else if (part == 0) put_state(a, io, it, head, w, st, l);
}

// One launch for all tiles, the wide ones first.
template <int D>
__global__ __launch_bounds__(kThreads, 2) void attend_diff(StepArgs a, AttendIo io, kamera_differential diff) {
  __shared__ __align__(1024) char lds[kLds];
  __shared__ float ml[2][kWaves][64];
  const int item = blockIdx.x / a.heads, head = blockIdx.x - item * a.heads;
  const AttendItem it = a.items[item];
  if (item < a.num_wide) wide_tile<D>(a, io, diff, it, head, (KLDS char*)lds);
  else if (item < a.num_wide + a.num_pairs) narrow_tile<D, 32>(a, io, diff, it, head, (KLDS char*)lds, ml);
  else narrow_tile<D, 16>(a, io, diff, it, head, (KLDS char*)lds, ml);
}

// ============================================================================
// Join of partial rows: an output row's two maps lie in neighbouring partial rows, 2 dv numbers side by side, which
// the threads share in 16-byte pieces. WPR waves a row; parts are taken in a fixed order. The maps' normalised
// rows meet in LDS, and the norm follows. All parts' statistics are read at once, then their rows, 8 of a wave at a
// time and none under a condition (a load under one is waited for before the next: 4 layers of 2 requests over 2000
// tokens 81 us that way, 69 this way). Bound by three dependent reads when rows are few, by the partial rows' bytes
// (written and read: 2 dv fp32 a query pair and part) when they are many. 64 tokens of 16 pairs in 18 parts: 12 us.
// ============================================================================
constexpr int kJoinParts = 2 * kMaxSplits;

__device__ __forceinline__ float wave_max(float x) {
  for (int d = 32; d; d >>= 1) x = fmaxf(x, __shfl_xor(x, d, kWaveSize));
  return x;
}
template <typename T>
__device__ __forceinline__ T narrowed(float x) {
  if constexpr (sizeof(T) == 2) return (T)pack2(x, 0.0f);
  else return x;
}

// The maximum or sum of WPR waves' values (all of a workgroup's threads come along)
template <int WPR, bool MAX>
__device__ __forceinline__ float2 over_waves(float2 x, float2 (&red)[2][WPR]) {
  if constexpr (WPR == 1) return x;
  if ((threadIdx.x & 63) == 0) red[MAX][threadIdx.x / kWaveSize] = x;
  __syncthreads();
  x = red[MAX][0];
  for (int i = 1; i < WPR; ++i) {
    const float2 y = red[MAX][i];
    x = MAX ? make_float2(fmaxf(x.x, y.x), fmaxf(x.y, y.y)) : make_float2(x.x + y.x, x.y + y.y);
  }
  return x;
}

// PIECES: 16-byte pieces of the two rows that a lane takes
template <typename T, int WPR, int PIECES>
__global__ __launch_bounds__(kThreads) void diff_join(StepArgs a, AttendIo io, kamera_differential diff) {
  constexpr int ROWS = kWaves / WPR;
  __shared__ float2 weight[ROWS][WPR == 1 ? kWaveSize : kJoinParts];
  __shared__ float2 red[ROWS][2][WPR];
  __shared__ f32x4 held[kWaves][PIECES * kWaveSize];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, sub = wave / WPR, seat = wave % WPR;
  const int outs = a.num_q_heads / 2;
  const int64_t task = (int64_t)block_number() * ROWS + sub;
  const bool live = task < (int64_t)a.num_merge * outs;
  const int64_t i = live ? task / outs : 0;
  const int oh = (int)(task % outs), head = 2 * oh / a.group, g = 2 * oh % a.group;
  const int quads = a.dv / 4;  // of a map's row
  const MergeToken mt = a.merge[i];
  const float2 products = lambda_products(a, diff);
  const int n = mt.splits[0] + mt.splits[1];  // (one at least)
  auto row = [&](int k) {  // of the first map; the second's is the next
    const int s = k >= mt.splits[0];
    return mt.part[s] + ((int64_t)(s ? k - mt.splits[0] : k) * a.heads + head) * mt.rows[s] + mt.row0[s] + g;
  };
  // every part's maxima and sums become its weights, all parts at once
  constexpr int MAXP = WPR == 1 ? kWaveSize : kJoinParts, TPR = WPR * kWaveSize, PER = MAXP / TPR;
  const int tid = threadIdx.x % TPR;
  const KGLOBAL f32x4* stats = (const KGLOBAL f32x4*)a.part_ml;  // (rows of the first map are even)
  f32x4 s[PER];
  float2 top = make_float2(-INFINITY, -INFINITY), sum = make_float2(0.0f, 0.0f);
  // (places behind the last part read it again: a load under a condition is waited for before the next one)
#pragma unroll
  for (int e = 0; e < PER; ++e) s[e] = stats[row(min(e * TPR + tid, n - 1)) >> 1];
  const T* weights = (diff.flags & KAMERA_DIFF_NORM) ? (const T*)diff.norm_weight : nullptr;
  float gain[(PIECES + 1) / 2][4];
#pragma unroll
  for (int j = 0; j < (PIECES + 1) / 2; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) gain[j][e] = 1.0f;
  if (weights) {
#pragma unroll
    for (int j = 0; j < (PIECES + 1) / 2; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) gain[j][e] = widened<T>(((const KGLOBAL T*)weights)[4 * min(j * kWaveSize + lane, quads - 1) + e]);
  }
#pragma unroll
  for (int e = 0; e < PER; ++e) {
    if (e * TPR + tid >= n) s[e] = (f32x4){-INFINITY, 0.0f, -INFINITY, 0.0f};
    if (s[e][1] != 0.0f) top.x = fmaxf(top.x, s[e][0]);
    if (s[e][3] != 0.0f) top.y = fmaxf(top.y, s[e][2]);
  }
  top = over_waves<WPR, true>(make_float2(wave_max(top.x), wave_max(top.y)), red[sub]);
#pragma unroll
  for (int e = 0; e < PER; ++e) {
    const float2 w = make_float2(s[e][1] == 0.0f ? 0.0f : s[e][0] == top.x ? 1.0f : __builtin_amdgcn_exp2f(s[e][0] - top.x),
                                 s[e][3] == 0.0f ? 0.0f : s[e][2] == top.y ? 1.0f : __builtin_amdgcn_exp2f(s[e][2] - top.y));
    sum.x += s[e][1] * w.x;
    sum.y += s[e][3] * w.y;
    if (e * TPR + tid < n) weight[sub][e * TPR + tid] = w;
  }
  sum = over_waves<WPR, false>(make_float2(wave_sum(sum.x), wave_sum(sum.y)), red[sub]);
  const float lambda = lambda_from(diff, products);
  __syncthreads();
  const KGLOBAL f32x4* parts = (const KGLOBAL f32x4*)a.part_o;
  f32x4 o[PIECES];
#pragma unroll
  for (int j = 0; j < PIECES; ++j) o[j] = (f32x4)(0.0f);
  // COUNT parts from k on: their rows are asked for together, then weighed
  int k = seat;
  auto take = [&](auto count) {
    constexpr int COUNT = decltype(count)::value;
    f32x4 x[COUNT][PIECES];
#pragma unroll
    for (int i = 0; i < COUNT; ++i) {
      const KGLOBAL f32x4* p = parts + row(k + i * WPR) * quads;
#pragma unroll
      for (int j = 0; j < PIECES; ++j) x[i][j] = p[min(j * kWaveSize + lane, 2 * quads - 1)];
    }
#pragma unroll
    for (int i = 0; i < COUNT; ++i) {
      const float2 w = weight[sub][k + i * WPR];
#pragma unroll
      for (int j = 0; j < PIECES; ++j) {
        const float wf = j * kWaveSize + lane < quads ? w.x : w.y;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][e] += x[i][j][e] * wf;  // (an empty part's row is 0)
      }
    }
    k += COUNT * WPR;
  };
  constexpr int MOST = PIECES <= 2 ? 8 : 16 / PIECES;
  while (k + (MOST - 1) * WPR < n) take(std::integral_constant<int, MOST>());
  if (MOST > 4 && k + 3 * WPR < n) take(std::integral_constant<int, 4>());
  if (MOST > 2 && k + WPR < n) take(std::integral_constant<int, 2>());
  if (k < n) take(std::integral_constant<int, 1>());
#pragma unroll
  for (int j = 0; j < PIECES; ++j) held[wave][j * kWaveSize + lane] = o[j];
  __syncthreads();
  if (seat != 0 || !live) return;
  const float inv0 = sum.x == 0.0f ? 0.0f : 1.0f / sum.x, inv1 = sum.y == 0.0f ? 0.0f : 1.0f / sum.y;
  f32x4 x[(PIECES + 1) / 2];
  float square = 0.0f;
#pragma unroll
  for (int j = 0; j < (PIECES + 1) / 2; ++j) {
    const int c = j * kWaveSize + lane;
    x[j] = (f32x4)(0.0f);
    if (c >= quads) continue;
    f32x4 y = held[wave][c], z = held[wave][quads + c];
#pragma unroll
    for (int w = 1; w < WPR; ++w) {
      const f32x4 y2 = held[wave + w][c], z2 = held[wave + w][quads + c];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        y[e] += y2[e];
        z[e] += z2[e];
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[j][e] = y[e] * inv0 - lambda * (z[e] * inv1);
      square += x[j][e] * x[j][e];
    }
  }
  const float scale = norm_scale(diff, wave_sum(square), a.dv);
  T* out = (T*)io.out + (int64_t)mt.token * io.out_stride + (int64_t)oh * a.dv;
#pragma unroll
  for (int j = 0; j < (PIECES + 1) / 2; ++j) {
    const int c = j * kWaveSize + lane;
    if (c >= quads) continue;
    float y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = x[j][e] * scale * gain[j][e];
    if (sizeof(T) == 2 && io.out_vec) {
      *(KGLOBAL u32x2*)(KGLOBAL void*)(out + 4 * c) = (u32x2){pack2(y[0], y[1]), pack2(y[2], y[3])};
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) out[4 * c + e] = narrowed<T>(y[e]);
    }
  }
  if (io.lse && lane < 2) {
    const float l = lane ? sum.y : sum.x, m = lane ? top.y : top.x;
    io.lse[(int64_t)mt.token * a.num_q_heads + 2 * oh + lane] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
  }
}

template <typename T, int WPR>
hipError_t join(const StepArgs& a, const AttendIo& io, const kamera_differential& diff, hipStream_t stream) {
  const int64_t rows = (int64_t)a.num_merge * (a.num_q_heads / 2);
  constexpr int ROWS = kWaves / WPR;
  const dim3 g = grid_of((rows + ROWS - 1) / ROWS), b(kThreads);
  const int pieces = (a.dv / 2 + kWaveSize - 1) / kWaveSize;
  if (pieces <= 1) hipLaunchKernelGGL((diff_join<T, WPR, 1>), g, b, 0, stream, a, io, diff);
  else if (pieces <= 2) hipLaunchKernelGGL((diff_join<T, WPR, 2>), g, b, 0, stream, a, io, diff);
  else if (pieces <= 4) hipLaunchKernelGGL((diff_join<T, WPR, 4>), g, b, 0, stream, a, io, diff);
  else hipLaunchKernelGGL((diff_join<T, WPR, 8>), g, b, 0, stream, a, io, diff);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_step_attend_diff(const StepArgs& a, int layer, const void* q, int64_t q_stride, void* out, int64_t out_stride,
                                   float* lse, float scale, const kamera_differential& diff, hipStream_t stream) {
  AttendIo io{q, out, lse, q_stride, out_stride, layer * a.layer_stride, fabsf(scale) * 1.44269504088896340736f, scale < 0.0f, 0, 0};
  // -inf marks a masked score: a scale of zero would make it NaN, the smallest one keeps it
  if (a.kernel != ATTEND_PLAIN) io.scale2 = fmaxf(io.scale2, 1.17549435e-38f);
  io.q_vec = q_stride % 8 == 0 && (uintptr_t)q % 16 == 0;
  io.out_vec = out_stride % 4 == 0 && (uintptr_t)out % 8 == 0;
  hipError_t e = hipSuccess;
  if (a.kernel == ATTEND_PLAIN) {
    e = launch_attend_plain(a, io, stream);
  } else if (a.num_items > 0) {
    const dim3 g((unsigned)((int64_t)a.num_items * a.heads)), b(kThreads);
    if (a.dk == 128) hipLaunchKernelGGL((attend_diff<128>), g, b, 0, stream, a, io, diff);
    else hipLaunchKernelGGL((attend_diff<64>), g, b, 0, stream, a, io, diff);
    e = hipGetLastError();
  }
  if (e != hipSuccess || a.num_merge == 0) return e;
  const int64_t rows = (int64_t)a.num_merge * (a.num_q_heads / 2);
  // Few rows are shared by 4 waves each. (4 layers, 32 + 8 heads of 128, whole calls in us with 1 and 4 waves a row: 32
  // rows 71 and 66, with 18 parts 86 and 69; 512 rows 175 and 165; 1024 rows 209 and 216; 2048 rows 298 and 320. 16
  // waves: 32 rows 75, 512 rows 189.)
  const bool wide = a.max_parts > kWaveSize || rows < 1024;
  if (a.dtype == KAMERA_BF16) return wide ? join<uint16_t, kWaves>(a, io, diff, stream) : join<uint16_t, 1>(a, io, diff, stream);
  return wide ? join<float, kWaves>(a, io, diff, stream) : join<float, 1>(a, io, diff, stream);
}

}  // namespace kamera
