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
template <int D, int NI>
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
      const int piece = (lane & (LPR - 1)) ^ swz(first + i * RPL + lane / LPR);
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
    Rows<D, NI> rows;
    rows.find(a, run, it.kv0, first, last);
    rows.load(a, kp, vp, (KLDS char*)k0, (KLDS char*)v0, first);
    rows.find(a, run, it.kv0 + TS, first, last);
    for (int t = it.kv0;;) {
      __syncthreads();  // this stage has arrived, the other buffer has been read
      if (t + TS < it.kv1) {
        rows.load(a, kp, vp, (KLDS char*)k1, (KLDS char*)v1, first);
        rows.find(a, run, t + 2 * TS, first, last);
      }
      walk<TS>(st, q, (const KLDS char*)k0, (const KLDS char*)k0, (const KLDS char*)v0, t, r.end, end_min, end_max, io.scale2);
      if ((t += TS) >= it.kv1) break;
      __syncthreads();
      if (t + TS < it.kv1) {
        rows.load(a, kp, vp, (KLDS char*)k0, (KLDS char*)v0, first);
        rows.find(a, run, t + 2 * TS, first, last);
      }
      walk<TS>(st, q, (const KLDS char*)k1, (const KLDS char*)k1, (const KLDS char*)v1, t, r.end, end_min, end_max, io.scale2);
      if ((t += TS) >= it.kv1) break;
    }
  }
  const float l = row_sum<32>(st.l);
  if (!r.owned) return;
  const int64_t part = part_row(a, run, it, head, r.row);
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  const int h = lane >> 5;
#pragma unroll
  for (int b = 0; b < S::kBlocks; ++b)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x[4] = {st.o[b][4 * i], st.o[b][4 * i + 1], st.o[b][4 * i + 2], st.o[b][4 * i + 3]};
      put<4>(a, io, run, part, r.token, r.qh, b * 32 + 8 * i + 4 * h, x, inv);
    }
  if (h == 0) put_stats(a, io, run, part, r.token, r.qh, st.m, l);
}

// ============================================================================
// Tiles of up to 32 rows (few queries on a KV head: reading the keys is what takes time): each of
// the 4 waves walks stages of its own, of 32 (128-wide) or 64 keys, at its own pace, and the four
// results are joined in LDS.
// ============================================================================
template <int D>
__global__ __launch_bounds__(kThreads, 1) void attend_narrow(StepArgs a, AttendIo io) {
  constexpr int TS = 4096 / D, NI = TS / kRowsPerLoad<D>, STAGE = TS * 2 * D;
  constexpr int OS = D + 4;  // floats between rows of a wave's result
  __shared__ __align__(1024) char b0[kWaves][2][STAGE], b1[kWaves][2][STAGE];
  __shared__ float ml[kWaves][2][32];
  const int item = blockIdx.x / a.heads, head = blockIdx.x - item * a.heads;
  const AttendItem it = a.items[item];
  const AttendRun run = a.runs[it.run];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const Lane r = lane_row(a, run, it, head, it.row0 + (lane & 31));
  const int end_min = __builtin_amdgcn_readfirstlane(r.end), end_max = __builtin_amdgcn_readlane(r.end, 31);
  typedef State<D, D, 32> S;
  bf16x8 q[S::kKSteps];
  S::load_q(io, r, q);
  S st;
  st.clear();
  const uint16_t* kp = a.k_pool + io.layer0 + head * D;
  const uint16_t* vp = a.v_pool + io.layer0 + head * D;
  const int last = it.kv1 - 1;
  constexpr int STEP = kWaves * TS;
  int t = it.kv0 + wave * TS;
  if (t < it.kv1) {
    KLDS char *ka = (KLDS char*)b0[wave][0], *va = (KLDS char*)b0[wave][1];
    KLDS char *kb = (KLDS char*)b1[wave][0], *vb = (KLDS char*)b1[wave][1];
    Rows<D, NI> rows;
    rows.find(a, run, t, 0, last);
    rows.load(a, kp, vp, ka, va, 0);
    rows.find(a, run, t + STEP, 0, last);
    for (;;) {
      __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0): this wave's stage has arrived
      __builtin_amdgcn_wave_barrier();
      if (t + STEP < it.kv1) {
        rows.load(a, kp, vp, kb, vb, 0);
        rows.find(a, run, t + 2 * STEP, 0, last);
      }
      walk<TS>(st, q, (const KLDS char*)ka, (const KLDS char*)ka, (const KLDS char*)va, t, r.end, end_min, end_max, io.scale2);
      if ((t += STEP) >= it.kv1) break;
      __builtin_amdgcn_s_waitcnt(0x0f70);
      __builtin_amdgcn_wave_barrier();
      if (t + STEP < it.kv1) {
        rows.load(a, kp, vp, ka, va, 0);
        rows.find(a, run, t + 2 * STEP, 0, last);
      }
      walk<TS>(st, q, (const KLDS char*)kb, (const KLDS char*)kb, (const KLDS char*)vb, t, r.end, end_min, end_max, io.scale2);
      if ((t += STEP) >= it.kv1) break;
    }
  }
  // every wave's rows, then their join: thread = (row, D / 8 columns)
  const float l = row_sum<32>(st.l);
  __syncthreads();  // the stages have been read: their place holds the results
  static_assert(kWaves / 2 * 32 * OS * 4 <= (int)sizeof(b0), "results fit where the stages were");
  auto result = [&](int i, int row) { return (float*)(i < kWaves / 2 ? &b0[0][0][0] : &b1[0][0][0]) + ((i & 1) * 32 + row) * OS; };
  const int h = lane >> 5;
#pragma unroll
  for (int b = 0; b < S::kBlocks; ++b)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *(f32x4*)(result(wave, lane & 31) + b * 32 + 8 * i + 4 * h) =
          (f32x4){st.o[b][4 * i], st.o[b][4 * i + 1], st.o[b][4 * i + 2], st.o[b][4 * i + 3]};
  if (h == 0) {
    ml[wave][0][lane] = st.m;
    ml[wave][1][lane] = l;
  }
  __syncthreads();
  const int row = threadIdx.x >> 3, d0 = (threadIdx.x & 7) * (D / 8);
  const Lane w = lane_row(a, run, it, head, it.row0 + row);
  if (!w.owned) return;
  float top = -INFINITY, sum = 0.0f, f[kWaves], x[D / 8];
#pragma unroll
  for (int i = 0; i < kWaves; ++i) top = fmaxf(top, ml[i][0][row]);
#pragma unroll
  for (int i = 0; i < kWaves; ++i) {
    const float mi = ml[i][0][row];
    f[i] = mi == -INFINITY ? (top == -INFINITY ? 1.0f : 0.0f) : (mi == top ? 1.0f : __builtin_amdgcn_exp2f(mi - top));
    sum += ml[i][1][row] * f[i];
  }
#pragma unroll
  for (int c = 0; c < D / 8; ++c) x[c] = 0.0f;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) {
    if (f[i] == 0.0f) continue;
#pragma unroll
    for (int c = 0; c < D / 8; c += 4) {
      const f32x4 y = *(const f32x4*)(result(i, row) + d0 + c);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[c + e] += y[e] * f[i];
    }
  }
  const int64_t part = part_row(a, run, it, head, w.row);
  put<D / 8>(a, io, run, part, w.token, w.qh, d0, x, sum == 0.0f ? 0.0f : 1.0f / sum);
  if ((threadIdx.x & 7) == 0) put_stats(a, io, run, part, w.token, w.qh, top, sum);
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
