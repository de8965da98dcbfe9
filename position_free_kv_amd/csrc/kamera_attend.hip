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

// ============================================================================
// Tiles of 128 rows: 4 waves share stages of 64 keys, 32 rows each. A run of at most 64 rows gives its
// rows to two waves, which take the first half of a stage's keys, and again to the other two, which
// take the second half (PAIRS); the pairs' results are joined at the end.
// ============================================================================
template <int D, bool PAIRS>
__global__ __launch_bounds__(kThreads, 2) void attend_wide(StepArgs a, AttendIo io, int item0) {
  constexpr int TS = 64, NI = TS / kRowsPerLoad<D> / kWaves, BYTES = TS * 2 * D;
  typedef State<D, D, 32> S;
  __shared__ __align__(1024) char k0[BYTES], v0[BYTES], k1[BYTES], v1[BYTES];
  const int item = blockIdx.x / a.heads, head = blockIdx.x - item * a.heads;
  const AttendItem it = a.items[item0 + item];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const uint16_t* kp = a.k_pool + io.layer0 + head * D;
  const uint16_t* vp = a.v_pool + io.layer0 + head * D;
  const int first = wave * NI * kRowsPerLoad<D>, last = it.kv1 - 1;
  const bool any = it.kv1 > it.kv0;
  Rows<D, NI, 32> rows;
  if (any) {
    rows.find(a, it.run, it.kv0, first, last);
    rows.load(a, kp, vp, (KLDS char*)k0, (KLDS char*)v0, first);
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
        rows.load(a, kp, vp, (KLDS char*)k1, (KLDS char*)v1, first);
        rows.find(a, it.run, t + 2 * TS, first, last);
      }
      stage((const KLDS char*)k0, (const KLDS char*)v0, t);
      if ((t += TS) >= it.kv1) break;
      stage_barrier();
      if (t + TS < it.kv1) {
        rows.load(a, kp, vp, (KLDS char*)k0, (KLDS char*)v0, first);
        rows.find(a, it.run, t + 2 * TS, first, last);
      }
      stage((const KLDS char*)k1, (const KLDS char*)v1, t);
      if ((t += TS) >= it.kv1) break;
    }
  }
  float l = row_sum<32>(st.l);
  if constexpr (PAIRS) {
    static_assert(BYTES >= 64 * 4 * D / 2, "a wave's result fits in a buffer");
    __shared__ float ml[2][kWaves][64];
    join_two(st, l, wave >= 2, wave & 1, wave & 1 ? (f32x4*)v0 : (f32x4*)k0, ml);
    if (wave >= 2) return;
  }
  put_state(a, io, it, head, r, st, l);
}

// ============================================================================
// Tiles of up to 32 rows (few queries on a KV head: reading the keys is what takes time). Each of the
// 4 waves walks stages of its own, of 32 (128-wide) or 64 keys, at its own pace, and the four results
// are joined in LDS. One buffer a wave (16 KB): two workgroups share a CU, so that the other seven
// waves' reads are in flight while one computes. Up to 16 rows take the products of 16 rows.
// ============================================================================
template <int D>
constexpr int kStageKeys = 4096 / D;
template <int D>
constexpr int kStageBytes = kStageKeys<D> * 2 * D;

template <int D, int ROWS>
__device__ __forceinline__ void narrow_rows_of(const StepArgs& a, const AttendIo& io, const AttendItem& it, int head,
                                               KLDS char* kbuf, KLDS char* vbuf, f32x4* place, float (&ml)[2][kWaves][64]) {
  typedef State<D, D, ROWS> S;
  constexpr int TS = kStageKeys<D>, NI = TS / kRowsPerLoad<D>, STEP = kWaves * TS;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Lane r = lane_row(a, it, head, it.row0 + S::row());
  const int end_min = __builtin_amdgcn_readfirstlane(r.end), end_max = __builtin_amdgcn_readlane(r.end, ROWS - 1);
  const uint16_t* kp = a.k_pool + io.layer0 + head * D;
  const uint16_t* vp = a.v_pool + io.layer0 + head * D;
  const int last = it.kv1 - 1;
  int t = it.kv0 + wave * TS;
  Rows<D, NI, ROWS> rows;
  if (t < it.kv1) {
    rows.find(a, it.run, t, 0, last);
    rows.load(a, kp, vp, kbuf, vbuf, 0);
  }
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
  join_waves(st, l, place, ml);
  if (wave == 0) put_state(a, io, it, head, r, st, l);
}

template <int D>
__global__ __launch_bounds__(kThreads, 2) void attend_narrow(StepArgs a, AttendIo io) {
  __shared__ __align__(1024) char buf[kWaves][2][kStageBytes<D>];
  __shared__ float ml[2][kWaves][64];
  static_assert(sizeof(buf) >= 2 * 64 * 4 * D / 2, "two waves' results fit where the stages were");
  const int item = blockIdx.x / a.heads, head = blockIdx.x - item * a.heads;
  const AttendItem it = a.items[item];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  KLDS char *k = (KLDS char*)buf[wave][0], *v = (KLDS char*)buf[wave][1];
  f32x4* place = (f32x4*)&buf[0][0][0];
  if (it.run.ntok * a.group <= 16) narrow_rows_of<D, 16>(a, io, it, head, k, v, place, ml);
  else narrow_rows_of<D, 32>(a, io, it, head, k, v, place, ml);
}

template <int D>
hipError_t launch(const StepArgs& a, const AttendIo& io, hipStream_t stream) {
  const dim3 b(kThreads);
  auto grid = [&](int items) { return dim3((unsigned)((int64_t)items * a.heads)); };
  const int wide0 = a.num_narrow + a.num_pairs, wide = a.num_items - wide0;
  if (wide > 0) hipLaunchKernelGGL((attend_wide<D, false>), grid(wide), b, 0, stream, a, io, wide0);
  if (a.num_pairs > 0) hipLaunchKernelGGL((attend_wide<D, true>), grid(a.num_pairs), b, 0, stream, a, io, a.num_narrow);
  if (a.num_narrow > 0) hipLaunchKernelGGL((attend_narrow<D>), grid(a.num_narrow), b, 0, stream, a, io);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attend_heads(const StepArgs& a, const AttendIo& io, hipStream_t stream) {
  return a.dk == 128 ? launch<128>(a, io, stream) : launch<64>(a, io, stream);
}

}  // namespace kamera
