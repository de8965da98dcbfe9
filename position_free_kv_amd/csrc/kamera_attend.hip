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
// Tiles of 128 rows: 4 waves of 32 rows share stages of 64 keys.
// ============================================================================
template <int D>
__global__ __launch_bounds__(kThreads, 2) void attend_wide(StepArgs a, AttendIo io) {
  constexpr int TS = 64, NI = TS / kRowsPerLoad<D> / kWaves;
  __shared__ __align__(1024) char k0[TS * 2 * D], v0[TS * 2 * D], k1[TS * 2 * D], v1[TS * 2 * D];
  const int item = blockIdx.x / a.heads, head = blockIdx.x - item * a.heads;
  const AttendItem it = a.items[a.num_narrow + item];
  const AttendRun run = a.runs[it.run];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const Lane r = lane_row(a, run, it, head, it.row0 + wave * 32 + (lane & 31));
  const int end_min = __builtin_amdgcn_readfirstlane(r.end), end_max = __builtin_amdgcn_readlane(r.end, 31);
  typedef State<D, D, 32> S;
  bf16x8 q[S::kKSteps];
  S::load_q(io, r, q);
  S st;
  st.clear();
  const uint16_t* kp = a.k_pool + io.layer0 + head * D;
  const uint16_t* vp = a.v_pool + io.layer0 + head * D;
  const int first = wave * NI * kRowsPerLoad<D>, last = it.kv1 - 1;
  if (it.kv1 > it.kv0) {
    Rows<D, NI, 32> rows;
    rows.find(a, run, it.kv0, first, last);
    rows.load(a, kp, vp, (KLDS char*)k0, (KLDS char*)v0, first);
    rows.find(a, run, it.kv0 + TS, first, last);
    for (int t = it.kv0;;) {
      __syncthreads();  // this stage has arrived, the other buffer has been read
      if (t + TS < it.kv1) {
        rows.load(a, kp, vp, (KLDS char*)k1, (KLDS char*)v1, first);
        rows.find(a, run, t + 2 * TS, first, last);
      }
      walk<TS, 2>(st, q, (const KLDS char*)k0, (const KLDS char*)k0, (const KLDS char*)v0, t, r.end, end_min, end_max, io.scale2);
      if ((t += TS) >= it.kv1) break;
      __syncthreads();
      if (t + TS < it.kv1) {
        rows.load(a, kp, vp, (KLDS char*)k0, (KLDS char*)v0, first);
        rows.find(a, run, t + 2 * TS, first, last);
      }
      walk<TS, 2>(st, q, (const KLDS char*)k1, (const KLDS char*)k1, (const KLDS char*)v1, t, r.end, end_min, end_max, io.scale2);
      if ((t += TS) >= it.kv1) break;
    }
  }
  put_state(a, io, run, it, head, r, st, row_sum<32>(st.l));
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
__device__ __forceinline__ void narrow_rows_of(const StepArgs& a, const AttendIo& io, const AttendRun& run, const AttendItem& it, int head,
                                               KLDS char* kbuf, KLDS char* vbuf, f32x4* place, float (&ml)[2][kWaves][64]) {
  typedef State<D, D, ROWS> S;
  constexpr int TS = kStageKeys<D>, NI = TS / kRowsPerLoad<D>, STEP = kWaves * TS;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Lane r = lane_row(a, run, it, head, it.row0 + S::row());
  const int end_min = __builtin_amdgcn_readfirstlane(r.end), end_max = __builtin_amdgcn_readlane(r.end, ROWS - 1);
  const uint16_t* kp = a.k_pool + io.layer0 + head * D;
  const uint16_t* vp = a.v_pool + io.layer0 + head * D;
  const int last = it.kv1 - 1;
  int t = it.kv0 + wave * TS;
  Rows<D, NI, ROWS> rows;
  if (t < it.kv1) {
    rows.find(a, run, t, 0, last);
    rows.load(a, kp, vp, kbuf, vbuf, 0);
  }
  bf16x8 q[S::kKSteps];
  S::load_q(io, r, q);
  S st;
  st.clear();
  while (t < it.kv1) {
    rows.find(a, run, t + STEP, 0, last);
    __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0): this wave's stage has arrived
    __builtin_amdgcn_wave_barrier();
    walk<TS, 1>(st, q, (const KLDS char*)kbuf, (const KLDS char*)kbuf, (const KLDS char*)vbuf, t, r.end, end_min, end_max, io.scale2);
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): read before it is overwritten
    __builtin_amdgcn_wave_barrier();
    if ((t += STEP) < it.kv1) rows.load(a, kp, vp, kbuf, vbuf, 0);
  }
  float l = row_sum<ROWS>(st.l);
  join_waves(st, l, place, ml);
  if (wave == 0) put_state(a, io, run, it, head, r, st, l);
}

template <int D>
__global__ __launch_bounds__(kThreads, 2) void attend_narrow(StepArgs a, AttendIo io) {
  __shared__ __align__(1024) char buf[kWaves][2][kStageBytes<D>];
  __shared__ float ml[2][kWaves][64];
  static_assert(sizeof(buf) >= 2 * 64 * 4 * D / 2, "two waves' results fit where the stages were");
  const int item = blockIdx.x / a.heads, head = blockIdx.x - item * a.heads;
  const AttendItem it = a.items[item];
  const AttendRun run = a.runs[it.run];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  KLDS char *k = (KLDS char*)buf[wave][0], *v = (KLDS char*)buf[wave][1];
  f32x4* place = (f32x4*)&buf[0][0][0];
  if (run.ntok * a.group <= 16) narrow_rows_of<D, 16>(a, io, run, it, head, k, v, place, ml);
  else narrow_rows_of<D, 32>(a, io, run, it, head, k, v, place, ml);
}

template <int D>
hipError_t launch(const StepArgs& a, const AttendIo& io, hipStream_t stream) {
  const int64_t wide = (int64_t)(a.num_items - a.num_narrow) * a.heads, narrow = (int64_t)a.num_narrow * a.heads;
  if (wide > 0) hipLaunchKernelGGL((attend_wide<D>), dim3((unsigned)wide), dim3(kThreads), 0, stream, a, io);
  if (narrow > 0) hipLaunchKernelGGL((attend_narrow<D>), dim3((unsigned)narrow), dim3(kThreads), 0, stream, a, io);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attend_heads(const StepArgs& a, const AttendIo& io, hipStream_t stream) {
  return a.dk == 128 ? launch<128>(a, io, stream) : launch<64>(a, io, stream);
}

}  // namespace kamera
