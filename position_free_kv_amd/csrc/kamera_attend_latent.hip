// Attention over MLA rows on the matrix cores: bf16 rows of a 512-wide latent and a 64-wide rope
// band, one row a token for all query heads; keys are the whole row, values its latent (method and
// register layouts: kamera_attend.h; work list: kamera_step_desc.h).
//
// The row is staged once and read from LDS twice, as K and as V^T. A wave keeps 16 query rows: 72
// registers of queries and 128 of output, so that two waves share a SIMD and one's softmax runs under
// the other's products. LDS bounds the wide kernel: per 32 keys each of its 8 waves issues 68 products
// (1088 cycles; two waves a SIMD) and reads 68 KB, 544 KB together at 128 bytes a cycle: 4250 cycles,
// 1.29 PFLOP/s. 32 rows a wave would halve that traffic, but its 400 registers did not compile without
// many spills; this form has 9 (24 bytes of scratch a lane), a few of them reloaded in every step.
//
// 32 requests of 16 heads over 4096 shared and 15888 own keys take 28 us a layer: launch and the first
// dependent reads 7, queries 4, the partial rows (36 MB) 6, the keys 11; then the join, 9. Items of 256 keys
// instead of 128 halve the partial rows but took 34 us, the join 8.8 instead of 9.7.
#include "kamera_attend.h"

namespace kamera {

namespace {

constexpr int kLatent = 512, kRope = 64, kKey = kLatent + kRope;
constexpr int kLatentRow = 2 * kLatent, kRopeRow = 2 * kRope;
constexpr int kKeys = 32;  // keys per stage
constexpr int kLatents = kKeys * kLatentRow, kBands = kKeys * kRopeRow;  // 32 KB and 4 KB
typedef State<kKey, kLatent, 16> LatentState;

// Pool rows of a stage's keys: lane i holds that of key first + i % n. The page id is asked for one
// stage ahead and used when the stage is loaded.
struct LatentRows {
  int page, place;
  __device__ __forceinline__ void find(const StepArgs& a, const AttendRun& run, int t0, int first, int n, int last) {
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));  // (see load)
    const int t = min(t0 + first + (lane & (n - 1)), last);
    page = ((const KGLOBAL int32_t*)a.pages)[key_entry(a, run, t, place)];
  }
  // N keys of the stage from `first` on (a multiple of N): one instruction a latent, one for 8 bands
  template <int N>
  __device__ __forceinline__ void load(const StepArgs& a, const uint16_t* k, KLDS char* latents, KLDS char* bands, int first) const {
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));  // what follows from it is made anew each stage: kept, it would cost the products registers
    const int row = page * a.page_size + place;  // rows of 1152 bytes: their number fits 32 bits
    constexpr int M = N < 8 ? N : 8;  // latents a turn (each with an address in scalar registers), bands an instruction
#pragma nounroll
    for (int i0 = 0; i0 < N; i0 += M)
#pragma unroll
      for (int i1 = 0; i1 < M; ++i1) {
        const int i = i0 + i1;
        const uint16_t* p = k + (int64_t)__builtin_amdgcn_readlane(row, i) * kKey;
        const int piece = lane ^ swz<16, kLatentRow>(first + i);
        __builtin_amdgcn_global_load_lds((const KGLOBAL void*)(p + piece * 8), (KLDS void*)(latents + (first + i) * kLatentRow), 16, 0, 0);
      }
#pragma unroll
    for (int i = 0; i < N; i += M) {
      const int piece = (lane & 7) ^ swz<16, kRopeRow>(first + i + lane / 8);
      const uint16_t* p = k + (int64_t)__shfl(row, i + lane / 8, 64) * kKey + kLatent;
      if (lane < 8 * M)
        __builtin_amdgcn_global_load_lds((const KGLOBAL void*)(p + piece * 8),
                                         (KLDS void*)(bands + (first + i) * kRopeRow), 16, 0, 0);
    }
  }
};

// Steps with a mask leave values that are not finite out of the product (State::finite). A row that sees one
// under a weight of 0 gets its NaN here, after the wave has written the 16 rows from row0 on: over the item's
// keys, a lane for 8 columns. Taken only where a score of -inf was met, so it costs the usual case a test.
__device__ __forceinline__ void zero_times_inf(const StepArgs& a, const AttendIo& io, const AttendItem& it, int row0) {
  const int lane = threadIdx.x & 63;
  const uint16_t* k = a.k_pool + io.layer0 + lane * 8;
  __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0): the rows are written
#pragma nounroll
  for (int t = it.kv0; t < it.kv1; ++t) {
    int place;
    const int page = ((const KGLOBAL int32_t*)a.pages)[key_entry(a, it.run, t, place)];
    const u32x4 w = *(const KGLOBAL u32x4*)(k + ((int64_t)page * a.page_size + place) * kKey);
    uint32_t marks = 0;  // columns
#pragma unroll
    for (int i = 0; i < 4; ++i)
      marks |= ((w[i] & 0x7f80u) == 0x7f80u ? 1u << (2 * i) : 0u) | ((w[i] & 0x7f800000u) == 0x7f800000u ? 2u << (2 * i) : 0u);
    if (!__any(marks != 0)) continue;
#pragma nounroll
    for (int i = 0; i < 16; ++i) {
      const Lane r = lane_row(a, it, 0, row0 + i);
      if (!r.owned || t >= r.end) continue;
#pragma nounroll
      for (int e = 0; e < 8; ++e) {
        if (!(marks >> e & 1)) continue;
        const int c = lane * 8 + e;
        if (it.run.direct) ((KGLOBAL uint16_t*)io.out)[(int64_t)r.token * io.out_stride + (int64_t)r.qh * kLatent + c] = 0x7fc0;
        else ((KGLOBAL float*)a.part_o)[part_row(a, it, 0, r.row) * kLatent + c] = NAN;
      }
    }
  }
}

// ============================================================================
// Tiles of 128 rows: 8 waves of 16 rows share stages of 32 keys.
// ============================================================================
constexpr int kWideWaves = 8;
__device__ __forceinline__ void wide_tile(const StepArgs& a, const AttendIo& io, const AttendItem& it, KLDS char* k0, KLDS char* k1,
                                          KLDS char* r0, KLDS char* r1, volatile KLDS int* low) {
  const AttendRun& run = it.run;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  constexpr int PER = kKeys / kWideWaves;  // rows a wave brings in
  const int first = wave * PER, last = it.kv1 - 1;
  LatentRows rows;  // (asked for ahead of the queries, as loads return in order)
  if (it.kv1 > it.kv0) rows.find(a, run, it.kv0, first, PER, last);
  const Lane r = lane_row(a, it, 0, it.row0 + wave * 16 + (lane & 15));
  const int end_min = __builtin_amdgcn_readfirstlane(r.end), end_max = __builtin_amdgcn_readlane(r.end, 15);
  bf16x8 q[LatentState::kKSteps];
  LatentState::load_q(io, r, q);
  LatentState st;
  st.clear();
  const uint16_t* kp = a.k_pool + io.layer0;
  if (it.kv1 > it.kv0) {
    rows.load<PER>(a, kp, k0, r0, first);
    rows.find(a, run, it.kv0 + kKeys, first, PER, last);
    for (int t = it.kv0;;) {
      stage_barrier();
      if (t + kKeys < it.kv1) {
        rows.load<PER>(a, kp, k1, r1, first);
        rows.find(a, run, t + 2 * kKeys, first, PER, last);
      }
      walk<kKeys, 1>(st, q, (const KLDS char*)k0, (const KLDS char*)r0, (const KLDS char*)k0, t, r.end, end_min, end_max, io.scale2);
      if ((t += kKeys) >= it.kv1) break;
      stage_barrier();
      if (t + kKeys < it.kv1) {
        rows.load<PER>(a, kp, k0, r0, first);
        rows.find(a, run, t + 2 * kKeys, first, PER, last);
      }
      walk<kKeys, 1>(st, q, (const KLDS char*)k1, (const KLDS char*)r1, (const KLDS char*)k1, t, r.end, end_min, end_max, io.scale2);
      if ((t += kKeys) >= it.kv1) break;
    }
  }
  const float l = row_sum<16>(st.l);
  low[wave] = st.low;
  int tid = threadIdx.x;  // the row again: kept through the loop it would take registers from the products
  asm volatile("" : "+v"(tid));
  put_state(a, io, it, 0, lane_row(a, it, 0, it.row0 + (tid >> 6) * 16 + (tid & 15)), st, l);
  if (low[wave]) zero_times_inf(a, io, it, it.row0 + wave * 16);
}

// ============================================================================
// Tiles of up to 16 rows: each wave walks stages of its own (one buffer each: LDS holds no more),
// the four out of step with each other, and the results are joined pairwise through LDS.
// ============================================================================
__device__ __forceinline__ void narrow_tile(const StepArgs& a, const AttendIo& io, const AttendItem& it, KLDS char* mine, KLDS char* band,
                                            KLDS char* place0, KLDS char* place1, float (&ml)[2][kWaves][64], volatile KLDS int* low) {
  const AttendRun& run = it.run;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int last = it.kv1 - 1;
  int t = it.kv0 + wave * kKeys;
  LatentRows rows;  // (as in the wide tile)
  if (t < it.kv1) rows.find(a, run, t, 0, kKeys, last);
  const Lane r = lane_row(a, it, 0, it.row0 + (lane & 15));
  const int end_min = __builtin_amdgcn_readfirstlane(r.end), end_max = __builtin_amdgcn_readlane(r.end, 15);
  bf16x8 q[LatentState::kKSteps];
  LatentState::load_q(io, r, q);
  LatentState st;
  st.clear();
  const uint16_t* kp = a.k_pool + io.layer0;
  if (t < it.kv1) {
    for (; t < it.kv1; t += kWaves * kKeys) {
      rows.load<kKeys>(a, kp, mine, band, 0);
      rows.find(a, run, t + kWaves * kKeys, 0, kKeys, last);
      __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0): this wave's stage has arrived
      __builtin_amdgcn_wave_barrier();
      walk<kKeys, 1>(st, q, (const KLDS char*)mine, (const KLDS char*)band, (const KLDS char*)mine, t, r.end, end_min, end_max, io.scale2);
      __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): read before it is overwritten
      __builtin_amdgcn_wave_barrier();
    }
  }
  float l = row_sum<16>(st.l);
  static_assert(kLatents >= 64 * LatentState::kBlocks * 16, "a wave's result fits where a stage was");
  low[wave] = st.low;
  join_waves(st, l, (f32x4*)place0, (f32x4*)place1, ml);
  int tid = threadIdx.x;  // (as in the wide tile)
  asm volatile("" : "+v"(tid));
  if (wave != 0) return;
  put_state(a, io, it, 0, lane_row(a, it, 0, it.row0 + (tid & 15)), st, l);
  if (low[0] | low[1] | low[2] | low[3]) zero_times_inf(a, io, it, it.row0);
}

// One launch for both kinds of tiles, the wide ones first. Narrow tiles have work for 4 of the 8 waves.
__global__ __launch_bounds__(64 * kWideWaves, 2) void attend_latent(StepArgs a, AttendIo io) {
  __shared__ __align__(1024) char k0[kLatents], k1[kLatents], k2[kLatents], k3[kLatents];
  __shared__ __align__(1024) char r0[kBands], r1[kBands], r2[kBands], r3[kBands];
  __shared__ float ml[2][kWaves][64];
  __shared__ int low[kWideWaves];
  const AttendItem it = a.items[blockIdx.x];
  if ((int)blockIdx.x < a.num_wide) {
    wide_tile(a, io, it, (KLDS char*)k0, (KLDS char*)k1, (KLDS char*)r0, (KLDS char*)r1, (KLDS int*)low);
  } else {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (wave >= kWaves) return;  // (barriers count the waves that are left)
    KLDS char* mine = wave < 2 ? (wave ? (KLDS char*)k1 : (KLDS char*)k0) : (wave == 2 ? (KLDS char*)k2 : (KLDS char*)k3);
    KLDS char* band = wave < 2 ? (wave ? (KLDS char*)r1 : (KLDS char*)r0) : (wave == 2 ? (KLDS char*)r2 : (KLDS char*)r3);
    narrow_tile(a, io, it, mine, band, (KLDS char*)k0, (KLDS char*)k1, ml, (KLDS int*)low);
  }
}

}  // namespace

hipError_t launch_attend_latent(const StepArgs& a, const AttendIo& io, hipStream_t stream) {
  if (a.num_items > 0) hipLaunchKernelGGL(attend_latent, dim3((unsigned)a.num_items), dim3(64 * kWideWaves), 0, stream, a, io);
  return hipGetLastError();
}

}  // namespace kamera
