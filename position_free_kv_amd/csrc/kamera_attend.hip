// Attention over the paged pool on the matrix cores: bf16 GQA/MHA rows with 64- or 128-wide heads
// (method and register layouts: kamera_attend.h; work list: kamera_step_desc.h).
#include "kamera_attend.h"

namespace kamera {

namespace {

template <int D>
constexpr int kRowsPerLoad = 1024 / (2 * D);  // tokens one wave instruction brings in

// NI wave instructions bring rows `first`, `first` + kRowsPerLoad, ... of a stage into LDS. The
// page ids are asked for one stage ahead (find) and used only when the stage is loaded: loads
// return in order, so using them at once would wait for the stage in flight as well.
template <int D, int NI, int ROWS>
struct Rows {
  int page[NI], place[NI];
  __device__ __forceinline__ void find(const StepArgs& a, const AttendRun& run, int t0, int first, int last) {
    constexpr int RPL = kRowsPerLoad<D>, LPR = 64 / RPL;  // lanes per row
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int t = min(t0 + first + i * RPL + lane / LPR, last);
      page[i] = ((const KGLOBAL int32_t*)a.pages)[key_entry(a, run, t, place[i])];
    }
  }
  // k and v: the layer's rows from this head's first column on
  __device__ __forceinline__ void load(const StepArgs& a, const uint16_t* k, const uint16_t* v, KLDS char* kbuf, KLDS char* vbuf,
                                       int first) const {
    constexpr int RPL = kRowsPerLoad<D>, LPR = 64 / RPL;
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int piece = (lane & (LPR - 1)) ^ swz<ROWS, 2 * D>(first + i * RPL + lane / LPR);
      const int64_t at = ((int64_t)page[i] * a.page_size + place[i]) * a.row + piece * 8;
      __builtin_amdgcn_global_load_lds((const KGLOBAL void*)(k + at), (KLDS void*)(kbuf + (first + i * RPL) * 2 * D), 16, 0, 0);
      __builtin_amdgcn_global_load_lds((const KGLOBAL void*)(v + at), (KLDS void*)(vbuf + (first + i * RPL) * 2 * D), 16, 0, 0);
    }
  }
};

// LDS of a workgroup: four places of 64 rows (keys or values) each.
constexpr int kStageKeys = 64;
template <int D>
constexpr int kPlace = kStageKeys * 2 * D;

// ============================================================================
// Tiles of 128 rows: 4 waves share stages of 64 keys, 32 rows each. A run of at most 64 rows gives its
// rows to two waves, which take the first half of a stage's keys, and again to the other two, which
// take the second half (PAIRS); the pairs' results are joined at the end.
//
// Bound by the loads into LDS and the clock together: 2481 query tokens of 28 + 4 heads over 8192 shared
// and their own keys (308 GFLOP) take 361 us, 0.85 PFLOP/s (a large library product: 1.22), while the clock
// holds (steps one after the other; the first twenty from rest 376 to 447). Of 427 us on another occasion:
// 335 without loads, 155 loads alone, 400 without the exponentials. Two workgroups of 64 KB share a CU: a
// tile of 256 rows with 8 waves (half the loads) took as long, four stages of 32 keys 443 us, and raised
// wave priority around the products 438.
// ============================================================================
template <int D, bool PAIRS>
__device__ __forceinline__ void wide_tile(const StepArgs& a, const AttendIo& io, const AttendItem& it, int head, KLDS char* k0, KLDS char* v0,
                                          KLDS char* k1, KLDS char* v1, float (&ml)[2][kWaves][64]) {
  constexpr int TS = kStageKeys, NI = TS / kRowsPerLoad<D> / kWaves;
  typedef State<D, D, 32> S;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const uint16_t* kp = a.k_pool + io.layer0 + head * D;
  const uint16_t* vp = a.v_pool + io.layer0 + head * D;
  const int first = wave * NI * kRowsPerLoad<D>, last = it.kv1 - 1;
  const bool any = it.kv1 > it.kv0;
  Rows<D, NI, 32> rows;
  if (any) {
    rows.find(a, it.run, it.kv0, first, last);
    rows.load(a, kp, vp, k0, v0, first);
    rows.find(a, it.run, it.kv0 + TS, first, last);
  }
  const int block = PAIRS ? wave & 1 : wave, part = PAIRS ? wave >> 1 : 0;  // rows, and keys of a stage
  const Lane r = lane_row(a, it, head, it.row0 + block * 32 + (lane & 31));
  const int end_min = __builtin_amdgcn_readfirstlane(r.end), end_max = __builtin_amdgcn_readlane(r.end, 31);
  bf16x8 q[S::kKSteps];
  S::load_q(io, r, q);
  S st;
  st.clear();
  auto stage = [&](const KLDS char* k, const KLDS char* v, int t) {
    constexpr int N = PAIRS ? 1 : 2;
    const int at = part * 32 * 2 * D;
    walk<32 * N, N>(st, q, k + at, k, v + at, t + part * 32, r.end, end_min, end_max, io.scale2);
  };
  if (any) {
    for (int t = it.kv0;;) {
      stage_barrier();
      if (t + TS < it.kv1) {
        rows.load(a, kp, vp, k1, v1, first);
        rows.find(a, it.run, t + 2 * TS, first, last);
      }
      stage(k0, v0, t);
      if ((t += TS) >= it.kv1) break;
      stage_barrier();
      if (t + TS < it.kv1) {
        rows.load(a, kp, vp, k0, v0, first);
        rows.find(a, it.run, t + 2 * TS, first, last);
      }
      stage(k1, v1, t);
      if ((t += TS) >= it.kv1) break;
    }
  }
  float l = row_sum<32>(st.l);
  if constexpr (PAIRS) {
    join_two(st, l, wave >= 2, wave & 1, wave & 1 ? (f32x4*)v0 : (f32x4*)k0, ml);
    if (wave >= 2) return;
  }
  put_state(a, io, it, head, r, st, l);
}

// ============================================================================
// Tiles of up to 32 rows (few queries on a KV head: reading the keys is what takes time). Each of the
// 4 waves walks stages of 32 keys of its own, at its own pace, and the four results are joined in LDS.
// One buffer a wave: two workgroups share a CU, so that the other waves' reads are in flight while one
// computes. Up to 16 rows take the products of 16 rows. Bound by reading pages: 32 + 8 heads, 16 requests
// over 131072 shared keys and 28296 own ones, 652 MB a layer in 130 us (5.0 TB/s; loads without products
// 135 us, products without loads 62). All heads of an item on one XCD: 139 us.
// ============================================================================
template <int D, int ROWS>
__device__ __forceinline__ void narrow_tile(const StepArgs& a, const AttendIo& io, const AttendItem& it, int head, KLDS char* mine,
                                            KLDS char* place0, KLDS char* place1, float (&ml)[2][kWaves][64]) {
  typedef State<D, D, ROWS> S;
  constexpr int TS = 32, NI = TS / kRowsPerLoad<D>, STEP = kWaves * TS;
  KLDS char *kbuf = mine, *vbuf = mine + TS * 2 * D;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint16_t* kp = a.k_pool + io.layer0 + head * D;
  const uint16_t* vp = a.v_pool + io.layer0 + head * D;
  const int last = it.kv1 - 1;
  int t = it.kv0 + wave * TS;
  Rows<D, NI, ROWS> rows;
  if (t < it.kv1) {
    rows.find(a, it.run, t, 0, last);
    rows.load(a, kp, vp, kbuf, vbuf, 0);
  }
  const Lane r = lane_row(a, it, head, it.row0 + S::row());
  const int end_min = __builtin_amdgcn_readfirstlane(r.end), end_max = __builtin_amdgcn_readlane(r.end, ROWS - 1);
  bf16x8 q[S::kKSteps];
  S::load_q(io, r, q);
  S st;
  st.clear();
  while (t < it.kv1) {
    rows.find(a, it.run, t + STEP, 0, last);
    __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0): this wave's stage has arrived
    __builtin_amdgcn_wave_barrier();
    walk<TS, 1>(st, q, (const KLDS char*)kbuf, (const KLDS char*)kbuf, (const KLDS char*)vbuf, t, r.end, end_min, end_max, io.scale2);
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): read before it is overwritten
    __builtin_amdgcn_wave_barrier();
    if ((t += STEP) < it.kv1) rows.load(a, kp, vp, kbuf, vbuf, 0);
  }
  float l = row_sum<ROWS>(st.l);
  join_waves(st, l, (f32x4*)place0, (f32x4*)place1, ml);
  if (wave == 0) put_state(a, io, it, head, r, st, l);
}

// One launch for all tiles, the wide ones first: what they compute runs beside what the narrow ones read.
template <int D>
__global__ __launch_bounds__(kThreads, 2) void attend_heads(StepArgs a, AttendIo io) {
  __shared__ __align__(1024) char p0[kPlace<D>], p1[kPlace<D>], p2[kPlace<D>], p3[kPlace<D>];
  __shared__ float ml[2][kWaves][64];
  static_assert(kPlace<D> >= 64 * 4 * D / 2, "a wave's result fits in a place");
  const int item = blockIdx.x / a.heads, head = blockIdx.x - item * a.heads;
  const AttendItem it = a.items[item];
  if (item < a.num_wide) {
    wide_tile<D, false>(a, io, it, head, (KLDS char*)p0, (KLDS char*)p1, (KLDS char*)p2, (KLDS char*)p3, ml);
  } else if (item < a.num_wide + a.num_pairs) {
    wide_tile<D, true>(a, io, it, head, (KLDS char*)p0, (KLDS char*)p1, (KLDS char*)p2, (KLDS char*)p3, ml);
  } else {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    KLDS char* mine = wave < 2 ? (wave ? (KLDS char*)p1 : (KLDS char*)p0) : (wave == 2 ? (KLDS char*)p2 : (KLDS char*)p3);
    if (it.run.ntok * a.group <= 16) narrow_tile<D, 16>(a, io, it, head, mine, (KLDS char*)p0, (KLDS char*)p1, ml);
    else narrow_tile<D, 32>(a, io, it, head, mine, (KLDS char*)p0, (KLDS char*)p1, ml);
  }
}

template <int D>
hipError_t launch(const StepArgs& a, const AttendIo& io, hipStream_t stream) {
  const int64_t blocks = (int64_t)a.num_items * a.heads;
  if (blocks > 0) hipLaunchKernelGGL((attend_heads<D>), dim3((unsigned)blocks), dim3(kThreads), 0, stream, a, io);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attend_heads(const StepArgs& a, const AttendIo& io, hipStream_t stream) {
  return a.dk == 128 ? launch<128>(a, io, stream) : launch<64>(a, io, stream);
}

}  // namespace kamera
