// Weighing (include/kamera_step.h): what each cached token receives of the attention weights of a step's queries.
// Work list: kamera_step_desc.h.
//
// Here the keys stay and the query rows pass by, the other way round than in the attention: a lane's sums
// belong to its keys, so that nothing is exchanged until the end, and every key's sum is one workgroup's (or a few
// ranges of rows are joined in their order).
//
// score[t] <- decay * score[t] + sum over rows that see t of exp(scale q . k_t - lse): the attention's lse makes the
// softmax's sum unnecessary, so that each key needs one pass over the rows and no running maximum. Sums are in fp32.
//
// 64 requests of one token over 8192 shared and 49300 own tokens, 32 + 8 heads of 128, a layer: 27 us; bound by reading the
// own keys (118 MB, 4.4 TB/s; longer ones 4.8, in whole rounds of workgroups and in broken ones alike). 2481 query
// tokens over 8192 shared and own tokens, 28 + 4 heads: 166 us for 154 GFLOP, 0.93 PFLOP/s (0.8 on a slower machine); bound by
// the products and the exponentials, which take about the same time and overlap in part (without branches between a stage's
// tiles the whole call took 183 instead of 181). 32 requests of one token, MLA, 16 heads, a layer: 15 us and 4 in the join;
// bound by dependent reads: item, tokens, lse, query rows.
#include "kamera_attend.h"
#include "kamera_grid.h"

namespace kamera {

namespace {

struct WeighIo {
  const void* q;
  const float* lse;
  float* scores;
  int64_t q_stride, layer0;
  float scale2;   // scale * log2(e)
  float decay;
  int32_t q_vec;  // rows of q in 16-byte pieces
  int32_t rows_of_token;  // query heads of a key head
};

constexpr float kLog2 = 1.44269504088896340736f;

// Query row `row` of key head `head`: its token in the run and its query head. (Differential: the heads of a
// pair of key heads take turns.)
struct QueryRow {
  int j, token, qh;
};
__device__ __forceinline__ QueryRow query_row(const StepArgs& a, const WeighIo& io, const WeighItem& it, int head, int row) {
  QueryRow r;
  r.j = (int)(((uint64_t)(uint32_t)row * a.group_magic) >> a.group_bits);
  const int g = row - r.j * io.rows_of_token;
  r.token = it.tok0 + r.j;
  if (it.listed) r.token = ((const KGLOBAL int32_t*)a.tok)[r.token];
  r.qh = a.differential ? (head >> 1) * 2 * io.rows_of_token + 2 * g + (head & 1) : head * io.rows_of_token + g;
  return r;
}

__device__ __forceinline__ int64_t slot_of(const StepArgs& a, int pg, int slot0, int t, int& place) {
  const int slot = slot0 + t, e = (int)(((uint64_t)(uint32_t)slot * a.page_magic) >> a.page_bits);
  place = slot - e * a.page_size;
  return ((const KGLOBAL int32_t*)a.pages)[pg + e];
}

__device__ __forceinline__ KGLOBAL float* score_at(const StepArgs& a, const WeighIo& io, int64_t page, int place, int head) {
  return (KGLOBAL float*)io.scores + (page * a.heads + head) * a.page_size + place;
}
// fresh: the token is the step's own
__device__ __forceinline__ void add_score(const StepArgs& a, const WeighIo& io, int64_t page, int place, int head, float sum, bool fresh) {
  KGLOBAL float* p = score_at(a, io, page, place, head);
  *p = io.decay == 0.0f || fresh ? sum : io.decay * *p + sum;
}

// ============================================================================
// Any layout: 16 lanes a key, 16 keys a workgroup, every lane NJ of its columns; ROWS rows at a time, all of them asked for
// before the first is used, and no read under a condition. Bound by their reads' latency. (fp32, whole calls in us with a row
// at a time and conditions, and so: 23 query tokens of 5 requests over 300 shared ones, 8 + 2 heads of 64, 63 and 36; MLA, 32
// requests, 16 heads, 2 layers, 3398 and 984 (1030 a row at a time).)
// ============================================================================
template <typename T>
__device__ __forceinline__ float widened(T x) {
  if constexpr (sizeof(T) == 2) return __uint_as_float((uint32_t)x << 16);
  else return x;
}

template <typename T, int NJ, int ROWS>
__global__ __launch_bounds__(kThreads) void weigh_plain(StepArgs a, WeighIo io) {
  const uint32_t block = block_number();
  const int item = (int)(block / (uint32_t)a.heads), head = (int)(block - (uint32_t)item * (uint32_t)a.heads);
  if (item >= a.num_weigh) return;
  const WeighItem it = a.weigh[item];
  const int lane = threadIdx.x & 15, t = it.kv0 + (threadIdx.x >> 4);
  int place;
  const int64_t page = slot_of(a, it.pg, it.slot, min(t, it.kv1 - 1), place);
  const KGLOBAL T* kp = (const KGLOBAL T*)a.k_pool + io.layer0 + (page * a.page_size + place) * a.row + (int64_t)head * a.dk;
  float k[NJ];
#pragma unroll
  for (int i = 0; i < NJ; ++i) {
    const int d = i * 16 + lane;
    k[i] = widened<T>(kp[min(d, a.dk - 1)]);
  }
  float sum = 0.0f;
  for (int row = it.row0; row < it.row1; row += ROWS) {
    // (rows behind the last and columns behind a row's end are read again and not used)
    QueryRow r[ROWS];
    float lse[ROWS], s[ROWS];
    T x[ROWS][NJ];
#pragma unroll
    for (int y = 0; y < ROWS; ++y) r[y] = query_row(a, io, it, head, min(row + y, it.row1 - 1));
#pragma unroll
    for (int y = 0; y < ROWS; ++y) {
      const KGLOBAL T* qp = (const KGLOBAL T*)io.q + (int64_t)r[y].token * io.q_stride + (int64_t)r[y].qh * a.dk;
      lse[y] = ((const KGLOBAL float*)io.lse)[(int64_t)r[y].token * a.num_q_heads + r[y].qh];
#pragma unroll
      for (int i = 0; i < NJ; ++i) x[y][i] = qp[min(i * 16 + lane, a.dk - 1)];
    }
#pragma unroll
    for (int y = 0; y < ROWS; ++y) {
      s[y] = 0.0f;
#pragma unroll
      for (int i = 0; i < NJ; ++i) s[y] += i * 16 + lane < a.dk ? widened<T>(x[y][i]) * k[i] : 0.0f;
    }
    for (int d = 8; d; d >>= 1)
#pragma unroll
      for (int y = 0; y < ROWS; ++y) s[y] += __shfl_xor(s[y], d, 16);
#pragma unroll
    for (int y = 0; y < ROWS; ++y) {
      const float w = exp2f(s[y] * io.scale2 - lse[y] * kLog2);
      sum += row + y < it.row1 && t <= it.lim0 + r[y].j * it.lstep && lse[y] != -INFINITY ? w : 0.0f;
    }
  }
  if (lane != 0 || t >= it.kv1) return;
  if (it.part >= 0) a.weigh_part[it.part + ((int64_t)it.split * a.heads + head) * it.kv + t] = sum;
  else add_score(a, io, page, place, head, sum, t >= it.fresh);
}

// ============================================================================
// On the matrix cores: S = Q K^T in tiles of 16 rows x 16 keys (v_mfma_f32_16x16x32_bf16). A wave holds
// 16 KT keys in registers for good; stages of SR query rows go through LDS, laid out as the attention
// lays out keys, NB stages in a ring. Lane 16 g + n gets the scores of key n and rows 4 g .. 4 g + 3, takes the
// row's lse off and adds up the exponentials. Where the rows lie, their lse and what they see is put into a
// table first, for up to TABLE rows at a time, so that the ring's loads depend on nothing else. (28 + 4 heads as above: two
// stages of 64 rows 181 us, three 201 to 206: the LDS then holds one workgroup less a CU. MLA: four stages of 16 rows, with
// the table 88 us, without it 91.)
// ============================================================================
template <int DK, int SR, int NB, int TABLE>
struct Stages {
  __align__(1024) char stage[NB][SR * 2 * DK];
  __align__(16) int64_t at[TABLE];   // element of q where the row begins
  __align__(16) float base[TABLE];   // lse * log2(e)
  __align__(16) int limit[TABLE];    // last key that the row sees; -1: it adds nothing
  int whole[TABLE / 16];             // 16 rows that add to all keys
};

// A wave's rows of a stage (SR / 4 of them) into LDS, swizzled like keys: the first DV columns (DK if there are fewer),
// then the others' rows. Always the same number of loads.
template <int DK, int DV, int SR>
struct QueryRows {
  typedef State<DK, DV, 16> S;
  static constexpr int PER = SR / kWaves;
  static constexpr int LPR = S::kKeyRow / 16 < 64 ? S::kKeyRow / 16 : 64, RPI = 64 / LPR;  // lanes of a row, rows of an instruction
  static constexpr int kBands = S::kRestRow ? (PER + 7) / 8 : 0;
  static constexpr int kLoads = PER / RPI + kBands;
  static_assert(S::kKeyRow <= 1024 && PER % RPI == 0 && (S::kRestRow == 0 || S::kRestRow == 128), "whole instructions");
  // at: the table's entries of the stage
  static __device__ __forceinline__ void load(const WeighIo& io, const int64_t* at, KLDS char* stage) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, first = wave * PER;
    // (all places first: one wait for LDS instead of one a load)
    const KGLOBAL uint16_t* x[kLoads];
    KLDS char* to[kLoads];
    const bool band = PER % 8 == 0 || lane / 8 < PER;
#pragma unroll
    for (int i = 0; i < PER / RPI; ++i) {
      const int r = first + i * RPI + lane / LPR;
      x[i] = (const KGLOBAL uint16_t*)io.q + at[r] + ((lane & (LPR - 1)) ^ swz<16, S::kKeyRow>(r)) * 8;
      to[i] = stage + (first + i * RPI) * S::kKeyRow;
    }
#pragma unroll
    for (int i = 0; i < kBands; ++i) {
      const int r = first + (band ? i * 8 + lane / 8 : 0);
      x[PER / RPI + i] = (const KGLOBAL uint16_t*)io.q + at[r] + DV + ((lane & 7) ^ swz<16, 128>(r)) * 8;
      to[PER / RPI + i] = stage + SR * S::kKeyRow + (first + i * 8) * 128;
    }
    if (io.q_vec) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i)
        if (i < PER / RPI || band) __builtin_amdgcn_global_load_lds((const KGLOBAL void*)x[i], (KLDS void*)to[i], 16, 0, 0);
    } else {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        if (i >= PER / RPI && !band) continue;
        u32x4 w;
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = (uint32_t)x[i][2 * e] | ((uint32_t)x[i][2 * e + 1] << 16);
        *(KLDS u32x4*)(to[i] + lane * 16) = w;
      }
    }
  }
};

// vmcnt(n), lgkmcnt(0): all but the last n loads have arrived, LDS reads and writes are done
template <int N>
__device__ __forceinline__ void wait_but() {
  static_assert(N < 64, "six bits");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x70);
}

template <int DK, int DV, int KT, int SR, int NB, int TABLE>
__device__ __forceinline__ void many_rows(const StepArgs& a, const WeighIo& io, const WeighItem& it, int head, Stages<DK, SR, NB, TABLE>& lds) {
  typedef State<DK, DV, 16> S;
  typedef QueryRows<DK, DV, SR> Q;
  static_assert(TABLE % SR == 0 && TABLE % kThreads == 0, "whole stages, whole turns of the threads");
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, n = lane & 15;
  const int key0 = it.kv0 + wave * 16 * KT;  // the wave's first key
  const bool any = key0 < it.kv1;
  int page[KT], place[KT];
#pragma unroll
  for (int x = 0; x < KT; ++x) page[x] = (int)slot_of(a, it.pg, it.slot, min(key0 + 16 * x + n, it.kv1 - 1), place[x]);
  bf16x8 k[KT][S::kKSteps];
  float sum[KT], old[KT];
#pragma unroll
  for (int x = 0; x < KT; ++x) sum[x] = old[x] = 0.0f;
  bool keys = false;
  for (int chunk = it.row0; chunk < it.row1; chunk += TABLE) {
    const int rows = min(it.row1 - chunk, TABLE), stages = (rows + SR - 1) / SR;
    if (chunk > it.row0) __syncthreads();  // (the table has been read)
    // (rows behind the last repeat it and add nothing; all tokens are asked for, then all lse)
    constexpr int TURNS = TABLE / kThreads;
    QueryRow q[TURNS];
    float lse[TURNS];
#pragma unroll
    for (int i = 0; i < TURNS; ++i) q[i] = query_row(a, io, it, head, min(chunk + i * kThreads + (int)threadIdx.x, it.row1 - 1));
#pragma unroll
    for (int i = 0; i < TURNS; ++i) lse[i] = ((const KGLOBAL float*)io.lse)[(int64_t)q[i].token * a.num_q_heads + q[i].qh];
#pragma unroll
    for (int i = 0; i < TURNS; ++i) {
      const int e = i * kThreads + (int)threadIdx.x, row = chunk + e;
      const int limit = row < it.row1 && lse[i] != -INFINITY ? it.lim0 + q[i].j * it.lstep : -1;
      const uint64_t all = __ballot(limit >= it.kv1 - 1);
      lds.at[e] = (int64_t)q[i].token * io.q_stride + (int64_t)q[i].qh * DK;
      lds.base[e] = lse[i] * kLog2;
      lds.limit[e] = limit;
      if ((lane & 15) == 0) lds.whole[e / 16] = ((all >> lane) & 0xffff) == 0xffff;
    }
    if (!keys) {  // (asked for behind the table's loads)
      keys = true;
#pragma unroll
      for (int x = 0; x < KT; ++x) {
        const KGLOBAL uint16_t* p = (const KGLOBAL uint16_t*)a.k_pool + io.layer0 + ((int64_t)page[x] * a.page_size + place[x]) * a.row + (int64_t)head * DK;
#pragma unroll
        for (int ks = 0; ks < S::kKSteps; ++ks) k[x][ks] = __builtin_bit_cast(bf16x8, *(const KGLOBAL u32x4*)(p + S::k_column(ks)));
        if (io.decay != 0.0f && it.part < 0) old[x] = *score_at(a, io, page[x], place[x], head);
      }
    }
    __syncthreads();
    auto load = [&](int s) { Q::load(io, lds.at + s * SR, (KLDS char*)lds.stage[s % NB]); };
    for (int s = 0; s < NB - 1 && s < stages; ++s) load(s);
    // the keys are waited for here: a first use inside the loop would wait for all loads in each turn
#pragma unroll
    for (int x = 0; x < KT; ++x)
#pragma unroll
      for (int ks = 0; ks < S::kKSteps; ++ks) {
        u32x4 w = __builtin_bit_cast(u32x4, k[x][ks]);
        asm volatile("" : "+v"(w));
        k[x][ks] = __builtin_bit_cast(bf16x8, w);
      }
#pragma nounroll
    for (int s = 0; s < stages; ++s) {
      // stage s is here, those after it (NB - 2 of them, unless the last ones are on their way) need not be
      if (s + NB - 2 < stages) wait_but<Q::kLoads * (NB - 2)>();
      else wait_but<0>();
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      if (s + NB - 1 < stages) load(s + NB - 1);
      if (!any) continue;
      const KLDS char* at = (const KLDS char*)lds.stage[s % NB];
#pragma unroll
      for (int r = 0; r < SR; r += 16) {
        const int e = s * SR + r;
        if (e >= rows) break;
        constexpr int CHAINS = KT >= 4 ? 1 : 4 / KT;  // products of a tile that do not wait for each other
        typename S::Acc part[CHAINS][KT], c[KT];
#pragma unroll
        for (int x = 0; x < KT; ++x)
#pragma unroll
          for (int y = 0; y < CHAINS; ++y) part[y][x] = (typename S::Acc)(0.0f);
#pragma unroll
        for (int ks = 0; ks < S::kKSteps; ++ks) {
          const bf16x8 q = S::k_operand(at + r * S::kKeyRow, at + SR * S::kKeyRow + r * S::kRestRow, 0, ks);
#pragma unroll
          for (int x = 0; x < KT; ++x) part[ks % CHAINS][x] = S::mfma(q, k[x][ks], part[ks % CHAINS][x]);
        }
#pragma unroll
        for (int x = 0; x < KT; ++x) {
          c[x] = part[0][x];
#pragma unroll
          for (int y = 1; y < CHAINS; ++y) c[x] += part[y][x];
        }
        const f32x4 b = *(const KLDS f32x4*)&lds.base[e + 4 * S::group()];
        if (__builtin_amdgcn_readfirstlane(lds.whole[e / 16])) {  // every row adds to every key
#pragma unroll
          for (int x = 0; x < KT; ++x)
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[x] += __builtin_amdgcn_exp2f(__builtin_fmaf(c[x][i], io.scale2, -b[i]));
        } else {
          typedef int i32x4 __attribute__((ext_vector_type(4)));
          const i32x4 lim = *(const KLDS i32x4*)&lds.limit[e + 4 * S::group()];
#pragma unroll
          for (int x = 0; x < KT; ++x) {
            const int t = key0 + 16 * x + n;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float w = __builtin_amdgcn_exp2f(__builtin_fmaf(c[x][i], io.scale2, -b[i]));
              sum[x] += t <= lim[i] ? w : 0.0f;
            }
          }
        }
      }
    }
  }
#pragma unroll
  for (int x = 0; x < KT; ++x) {
    const float total = row_sum<16>(sum[x]);
    const int t = key0 + 16 * x + n;
    if (lane >= 16 || t >= it.kv1) continue;
    if (it.part >= 0) a.weigh_part[it.part + ((int64_t)it.split * a.heads + head) * it.kv + t] = total;
    else *score_at(a, io, page[x], place[x], head) = io.decay == 0.0f || t >= it.fresh ? total : io.decay * old[x] + total;
  }
}

// ============================================================================
// At most 16 rows: they stay in registers, and each wave walks over 16 KT keys at a time, which go straight to LDS in
// a ring of its own of NB stages. Bound by reading the keys. In the walk there is nothing but that, no other load and
// no store, so that each wait is for one stage: where the keys lie is put into a table first, the sums go to LDS and
// are added to the scores at the end, which are asked for at the start. (64 requests, 32 + 8 heads, 4 layers: keys into
// the lanes that multiply them, 16 bytes a lane and row, with a store and conditions in the walk 131 us, without them
// 125, by way of LDS 115. Two stages ahead and 3 workgroups a CU 115, three and 2 123.)
// ============================================================================
template <int DK, int KT, int KEYS, int NB>
struct Walk {
  static constexpr int kWide = 16 * KT, kMine = KEYS / kWaves, kStage = kWide * 2 * DK;  // keys of a wave's step, of a wave; bytes of a stage
  static_assert(kMine % kWide == 0 && (NB > 1 || kMine == kWide), "whole steps, a ring of two where there are more than one");
  __align__(1024) char stage[kWaves][NB][kStage];
  uint32_t row[kWaves][kMine];  // of the pool
  float sum[kWaves][kMine];
};

template <int DK, int DV, int KT, int KEYS, int NB>
__device__ __forceinline__ void few_rows(const StepArgs& a, const WeighIo& io, const WeighItem& it, int head, Walk<DK, KT, KEYS, NB>& lds) {
  typedef State<DK, DV, 16> S;
  typedef Walk<DK, KT, KEYS, NB> W;
  constexpr int WIDE = W::kWide, STEP = kWaves * WIDE, MINE = W::kMine, EACH = (MINE + 63) / 64;
  constexpr int LPR = S::kKeyRow / 16 < 64 ? S::kKeyRow / 16 : 64, RPI = 64 / LPR, ROWS = WIDE / RPI, BANDS = S::kRestRow ? WIDE / 8 : 0, LOADS = ROWS + BANDS;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, n = lane & 15;
  const int last = it.kv1 - 1, first = it.kv0 + wave * WIDE;  // the wave's first key
  if (first > last) return;
  const KGLOBAL uint16_t* keys = (const KGLOBAL uint16_t*)a.k_pool + io.layer0 + (int64_t)head * DK;
  KLDS char* ring = (KLDS char*)lds.stage[wave];
  KLDS uint32_t* rows = (KLDS uint32_t*)lds.row[wave];
  KLDS float* sums = (KLDS float*)lds.sum[wave];
  // the wave's key number e
  auto key_of = [&](int e) { return first + e / WIDE * STEP + e % WIDE; };
  int page[EACH], place[EACH];
#pragma unroll
  for (int i = 0; i < EACH; ++i) page[i] = (int)slot_of(a, it.pg, it.slot, min(key_of(i * 64 + lane), last), place[i]);
  // the rows
  const QueryRow r = query_row(a, io, it, head, min(it.row0 + n, it.row1 - 1));
  QueryRow y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = query_row(a, io, it, head, min(it.row0 + 4 * S::group() + i, it.row1 - 1));
  float base[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) base[i] = ((const KGLOBAL float*)io.lse)[(int64_t)y[i].token * a.num_q_heads + y[i].qh];
  const KGLOBAL uint16_t* qp = (const KGLOBAL uint16_t*)io.q + (int64_t)r.token * io.q_stride + (int64_t)r.qh * DK;
  bf16x8 q[S::kKSteps];
  if (io.q_vec) {
#pragma unroll
    for (int ks = 0; ks < S::kKSteps; ++ks) q[ks] = __builtin_bit_cast(bf16x8, *(const KGLOBAL u32x4*)(qp + S::k_column(ks)));
  } else {
#pragma unroll
    for (int ks = 0; ks < S::kKSteps; ++ks) {
      u32x4 w;
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = (uint32_t)qp[S::k_column(ks) + 2 * e] | ((uint32_t)qp[S::k_column(ks) + 2 * e + 1] << 16);
      q[ks] = __builtin_bit_cast(bf16x8, w);
    }
  }
  KGLOBAL float* score[EACH];
  float old[EACH];
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
    if (EACH * 64 == MINE || lane < MINE) rows[i * 64 + lane] = (uint32_t)(page[i] * a.page_size + place[i]);  // (below 2^31)
    score[i] = score_at(a, io, page[i], place[i], head);
    old[i] = *score[i];
  }
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // (a wave reads its own entries alone)
  auto load = [&](int s) {
    KLDS char* stage = ring + s % NB * W::kStage;
    uint32_t at[LOADS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) at[i] = rows[s * WIDE + i * RPI + lane / LPR];
#pragma unroll
    for (int i = 0; i < BANDS; ++i) at[ROWS + i] = rows[s * WIDE + i * 8 + lane / 8];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const int piece = (lane & (LPR - 1)) ^ swz<16, S::kKeyRow>(i * RPI + lane / LPR);
      __builtin_amdgcn_global_load_lds((const KGLOBAL void*)(keys + (int64_t)at[i] * a.row + piece * 8), (KLDS void*)(stage + i * RPI * S::kKeyRow), 16, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < BANDS; ++i) {
      const int piece = (lane & 7) ^ swz<16, 128>(i * 8 + lane / 8);
      __builtin_amdgcn_global_load_lds((const KGLOBAL void*)(keys + (int64_t)at[ROWS + i] * a.row + DV + piece * 8), (KLDS void*)(stage + WIDE * S::kKeyRow + i * 8 * 128), 16, 0, 0);
    }
  };
  const int steps = (last - first) / STEP + 1;
  load(0);
  for (int s = 1; s < NB - 1 && s < steps; ++s) load(s);
  // the rows are waited for here: a first use inside the loop would wait for all loads in each turn
  int limit[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    limit[i] = it.row0 + 4 * S::group() + i < it.row1 && base[i] != -INFINITY ? it.lim0 + y[i].j * it.lstep : -1;
    base[i] *= kLog2;
  }
#pragma unroll
  for (int ks = 0; ks < S::kKSteps; ++ks) {
    u32x4 w = __builtin_bit_cast(u32x4, q[ks]);
    asm volatile("" : "+v"(w));
    q[ks] = __builtin_bit_cast(bf16x8, w);
  }
#pragma nounroll
  for (int s = 0; s < steps; ++s) {
    // stage s is here, those after it (NB - 2 of them, unless the last ones are on their way) need not be
    if (NB > 2 && s + NB - 2 < steps) wait_but<LOADS * (NB > 2 ? NB - 2 : 0)>();
    else wait_but<0>();
    asm volatile("" ::: "memory");
    if (NB > 1 && s + NB - 1 < steps) load(s + NB - 1);
    const KLDS char* at = ring + s % NB * W::kStage;
#pragma unroll
    for (int x = 0; x < KT; ++x) {
      typename S::Acc c = (typename S::Acc)(0.0f), c1 = c;  // (two chains of products)
#pragma unroll
      for (int ks = 0; ks < S::kKSteps; ks += 2) {
        c = S::mfma(q[ks], S::k_operand(at + x * 16 * S::kKeyRow, at + WIDE * S::kKeyRow + x * 16 * S::kRestRow, 0, ks), c);
        c1 = S::mfma(q[ks + 1], S::k_operand(at + x * 16 * S::kKeyRow, at + WIDE * S::kKeyRow + x * 16 * S::kRestRow, 0, ks + 1), c1);
      }
      c += c1;
      const int key = first + s * STEP + x * 16 + n;
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(c[i], io.scale2, -base[i]));
        sum += key <= limit[i] ? e : 0.0f;
      }
      sums[s * WIDE + x * 16 + n] = row_sum<16>(sum);  // (four lanes the same)
    }
  }
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
    const int e = i * 64 + lane, t = key_of(e);
    if ((EACH * 64 != MINE && e >= MINE) || t > last) continue;
    const float sum = sums[e];
    if (it.part >= 0) a.weigh_part[it.part + ((int64_t)it.split * a.heads + head) * it.kv + t] = sum;
    else *score[i] = io.decay == 0.0f || t >= it.fresh ? sum : io.decay * old[i] + sum;
  }
}

template <int DK, int DV, int KT, int SR, int NB, int TABLE, int FEW_KT, int FEW_NB>
__global__ __launch_bounds__(kThreads, 2) void weigh_matrix(StepArgs a, WeighIo io) {
  typedef Stages<DK, SR, NB, TABLE> Many;
  typedef Walk<DK, FEW_KT, weigh_keys_of_few(DK == DV ? ATTEND_HEADS : ATTEND_LATENT), FEW_NB> Few;
  __shared__ __align__(1024) char lds[sizeof(Many) > sizeof(Few) ? sizeof(Many) : sizeof(Few)];
  const int item = blockIdx.x / a.heads, head = blockIdx.x - item * a.heads;
  const WeighItem it = a.weigh[item];
  if (it.row1 - it.row0 <= kFewRows) few_rows<DK, DV>(a, io, it, head, *(Few*)lds);
  else many_rows<DK, DV, KT, SR, NB, TABLE>(a, io, it, head, *(Many*)lds);
}

// Sums of ranges of rows, joined in their order: a thread a key and head. A range that ends before the first row
// that sees a tile's keys has none of them.
__global__ __launch_bounds__(kThreads) void weigh_join(StepArgs a, WeighIo io) {
  const int64_t blocks = (a.weigh_longest + kThreads - 1) / kThreads;
  int64_t b = block_number();
  const int t = (int)(b % blocks) * kThreads + (int)threadIdx.x;
  b /= blocks;
  const int head = (int)(b % a.heads), run = (int)(b / a.heads);
  if (run >= a.num_weigh_join) return;
  const WeighJoin j = a.weigh_join[run];
  if (t >= j.kv) return;
  const int kv0 = t / j.tile * j.tile;
  const int64_t row0 = j.lstep && kv0 > j.lim0 ? (int64_t)(kv0 - j.lim0) * io.rows_of_token : 0;
  const KGLOBAL float* p = (const KGLOBAL float*)a.weigh_part + j.part + (int64_t)head * j.kv + t;
  int place;
  const int64_t page = slot_of(a, j.pg, j.slot, t, place);
  KGLOBAL float* score = score_at(a, io, page, place, head);
  const float old = *score;
  const int64_t stride = (int64_t)a.heads * j.kv;
  float sum = 0.0f;
  constexpr int kAtOnce = 8;
  for (int s = (int)(row0 / j.rows); s < j.splits; s += kAtOnce) {  // (places behind the last range read it again)
    float x[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) x[i] = p[min(s + i, j.splits - 1) * stride];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) sum += s + i < j.splits ? x[i] : 0.0f;
  }
  *score = io.decay == 0.0f || t >= j.fresh ? sum : io.decay * old + sum;
}

template <typename T>
hipError_t plain(const StepArgs& a, const WeighIo& io, hipStream_t stream) {
  const dim3 g = grid_of((int64_t)a.num_weigh * a.heads), b(kThreads);
  if (a.dk <= 128) hipLaunchKernelGGL((weigh_plain<T, 8, 8>), g, b, 0, stream, a, io);
  else if (a.dk <= 640) hipLaunchKernelGGL((weigh_plain<T, 40, 2>), g, b, 0, stream, a, io);
  else hipLaunchKernelGGL((weigh_plain<T, 64, 1>), g, b, 0, stream, a, io);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_step_weigh(const StepArgs& a, int layer, const void* q, int64_t q_stride, const float* lse, float* scores, float scale,
                             float decay, hipStream_t stream) {
  WeighIo io{q, lse, scores, q_stride, layer * a.layer_stride, scale * kLog2, decay, 0, a.num_q_heads / a.heads};
  io.q_vec = q_stride % 8 == 0 && (uintptr_t)q % 16 == 0;
  if (a.num_weigh == 0) return hipSuccess;
  hipError_t e;
  if (a.weigh_kernel == ATTEND_PLAIN) {
    e = a.dtype == KAMERA_BF16 ? plain<uint16_t>(a, io, stream) : plain<float>(a, io, stream);
  } else {
    const dim3 g((unsigned)((int64_t)a.num_weigh * a.heads)), b(kThreads);
    if (a.weigh_kernel == ATTEND_LATENT) hipLaunchKernelGGL((weigh_matrix<576, 512, 1, 16, 4, 256, 1, 1>), g, b, 0, stream, a, io);
    else if (a.dk == 128) hipLaunchKernelGGL((weigh_matrix<128, 128, 4, 64, 2, 1024, 1, 3>), g, b, 0, stream, a, io);
    else hipLaunchKernelGGL((weigh_matrix<64, 64, 4, 64, 2, 1024, 2, 3>), g, b, 0, stream, a, io);
    e = hipGetLastError();
  }
  if (e != hipSuccess || a.num_weigh_join == 0) return e;
  const int64_t blocks = (int64_t)((a.weigh_longest + kThreads - 1) / kThreads) * a.heads * a.num_weigh_join;
  if (blocks > 0x7fffffffLL) return hipErrorInvalidValue;
  hipLaunchKernelGGL(weigh_join, grid_of(blocks), dim3(kThreads), 0, stream, a, io);
  return hipGetLastError();
}

}  // namespace kamera
