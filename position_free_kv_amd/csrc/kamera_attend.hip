// Attention over the paged pool on the matrix cores (bf16 GQA/MHA rows with 64- or 128-wide
// heads): the kernels behind kamera_step_attend's work list (kamera_step_desc.h).
//
// A workgroup takes one KV head, a tile of query rows and a range of keys, and walks the range
// once with a running maximum and sum. Both products are transposed, so that one lane owns one
// query row throughout (v_mfma_f32_32x32x16_bf16; lane = 32 h + n):
//   S^T = K Q^T   A = K (row m = token, 8 columns at 8 h), B = Q^T (column n = row): the result
//                 gives lane (h, n) the scores of row n and tokens 8 (i / 4) + 4 h + i % 4
//   O^T = V^T P^T B = P^T: those same scores, exponentiated, are already the B operand if the
//                 k slots are numbered in that token order; A = V^T is read from LDS in the same
//                 order by the transposing reads (ds_read_b64_tr_b16: 16 lanes read 4 tokens x
//                 16 columns and each receives one column's 4 tokens).
// So the probabilities never leave their registers, the row's maximum and sum cost one exchange
// between the two halves of the wave, and rescaling O is a per-lane factor. O is rescaled only
// when a row's maximum has grown by more than 8 (base-2): until then probabilities are at most
// 2^8, which neither bf16 nor the fp32 sums mind.
//
// K and V go from the pool's pages straight into LDS (global_load_lds, 16 bytes a lane, every
// lane its own row address: pages may be of any size and order), double-buffered. 16-byte
// pieces of a token's row are stored at position piece ^ swz(token): the row reads of K (32
// tokens, one piece each) and the transposing reads of V (4 tokens x 32 bytes) then touch all
// banks evenly. Rows past the range's end repeat its last row and are masked.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kamera_step_desc.h"

namespace kamera {

namespace {

#define KGLOBAL __attribute__((address_space(1)))
#define KLDS __attribute__((address_space(3)))

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;
constexpr int kWaves = 4;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kGrow = 8.0f;  // a row's maximum may lag this far behind (base-2)

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  bf16x2 r;
  r.x = (__bf16)a;
  r.y = (__bf16)b;
  return __builtin_bit_cast(uint32_t, r);
}

// the value of the other half of the wave (lane ^ 32)
__device__ __forceinline__ float other_half(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float((threadIdx.x & 32) ? r[0] : r[1]);
}

__device__ __forceinline__ int swz(int token) { return ((token & 3) << 1) | ((token >> 2) & 1); }

template <int D>
struct Tile {
  static constexpr int kRowBytes = 2 * D;
  static constexpr int kRowsPerLoad = 1024 / kRowBytes;  // tokens one wave instruction brings in
  static constexpr int kKSteps = D / 16, kBlocks = D / 32;
};

// One lane's view of its query row and of the range of keys.
struct Lane {
  int row;           // row of the run (clamped to its last)
  bool owned;        // false: a repeat of the last row, not written
  int token, qh;
  int end;           // keys [kv0, end) are seen
};

__device__ __forceinline__ Lane lane_row(const StepArgs& a, const AttendRun& run, const AttendItem& it, int head, int row) {
  Lane r;
  const int rows = run.ntok * a.group;
  r.owned = row < rows;
  r.row = min(row, rows - 1);
  const int j = r.row / a.group;
  r.qh = head * a.group + (r.row - j * a.group);
  r.token = run.listed ? a.tok[run.tok0 + j] : run.tok0 + j;
  r.end = min(it.kv1, max(run.len_a - 1, run.lim0 + j * run.lstep) + 1);
  return r;
}

// Page-table entry and place in its page of key t of the run. The page is a product with the page
// size's reciprocal (exact for slots below 2^31), so any page size costs the same.
__device__ __forceinline__ int key_entry(const StepArgs& a, const AttendRun& run, int t, int& place) {
  const bool first = t < run.len_a;
  const int slot = first ? run.slot_a + t : run.slot_b + (t - run.len_a);
  const int pg = (int)(((uint64_t)(uint32_t)slot * a.page_magic) >> a.page_bits);
  place = slot - pg * a.page_size;
  return (first ? run.pg_a : run.pg_b) + pg;
}

// NI wave instructions bring rows `first`, `first` + kRowsPerLoad, ... of a stage into LDS. The
// page ids are asked for one stage ahead (find) and used only when the stage is loaded: loads
// return in order, so using them at once would wait for the stage in flight as well.
template <int D, int NI>
struct Rows {
  int page[NI], place[NI];
  __device__ __forceinline__ void find(const StepArgs& a, const AttendRun& run, int t0, int first, int last) {
    constexpr int RPL = Tile<D>::kRowsPerLoad, LPR = 64 / RPL;  // lanes per row
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
    constexpr int RPL = Tile<D>::kRowsPerLoad, LPR = 64 / RPL;
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

// Running state of a wave's 32 rows.
template <int D>
struct State {
  f32x16 o[Tile<D>::kBlocks];
  float m, l;  // l: this lane's tokens only (the halves are added at the end)

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int b = 0; b < Tile<D>::kBlocks; ++b) o[b] = (f32x16)(0.0f);
    m = -INFINITY;
    l = 0.0f;
  }

  __device__ __forceinline__ bf16x8 v_operand(const KLDS char* v, const int (&v_at)[2], int sub, int u, int b) const {
    const KLDS char* p = v + v_at[b & 1] + (sub * 32 + u * 16) * 2 * D + (b >> 1) * 128;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((KLDS s16x4*)p);
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((KLDS s16x4*)(p + 8 * 2 * D));
    typedef short s16x8 __attribute__((ext_vector_type(8)));
    const s16x8 both = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_bit_cast(bf16x8, both);
  }

  // the largest exponent field among 8 bf16 values
  static __device__ __forceinline__ uint32_t exponents(u32x4 w) {
    uint32_t x = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) x = max(x, max((w[i] >> 16) & 0x7f80u, w[i] & 0x7f80u));
    return x;
  }

  // O += P V for a stage in which some value is not finite and some row does not see every
  // token (rare: kept small rather than fast). p: NT x 2 operands.
  template <int NT>
  __device__ __forceinline__ void spoiled(const bf16x8 (&p)[2 * NT], const KLDS char* v, const int (&v_at)[2], int t0, int end) {
    const int h = (threadIdx.x & 63) >> 5;
#pragma nounroll
    for (int c = 0; c < 2 * NT; ++c) {
      bf16x8 pw = p[0];
#pragma unroll
      for (int x = 1; x < 2 * NT; ++x)
        if (c == x) pw = p[x];
      const u32x4 pu = __builtin_bit_cast(u32x4, pw);
#pragma unroll
      for (int b = 0; b < Tile<D>::kBlocks; ++b) {
        __builtin_amdgcn_sched_barrier(0);
        u32x4 w = __builtin_bit_cast(u32x4, v_operand(v, v_at, 0, c, b));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if ((w[i] & 0x7f80u) == 0x7f80u) w[i] &= 0xffff0000u;
          if ((w[i] & 0x7f800000u) == 0x7f800000u) w[i] &= 0xffffu;
        }
        o[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, w), pw, o[b], 0, 0, 0);
      }
#pragma nounroll
      for (int e = 0; e < 16; ++e) {  // token slot: half e >> 3, element e & 7
        const uint32_t pair = (e & 6) == 0 ? pu[0] : (e & 6) == 2 ? pu[1] : (e & 6) == 4 ? pu[2] : pu[3];
        const float mine = __uint_as_float((e & 1) ? pair & 0xffff0000u : pair << 16), theirs = other_half(mine);
        const float weight = h == (e >> 3) ? mine : theirs;
        const int slot = c * 16 + 8 * ((e & 7) >> 2) + 4 * (e >> 3) + (e & 3);
        if (t0 + slot >= end) continue;
#pragma unroll
        for (int b = 0; b < Tile<D>::kBlocks; ++b)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            __builtin_amdgcn_sched_barrier(0);
            const u32x2 w = *(const KLDS u32x2*)(v + slot * 2 * D + (((b * 4 + i) ^ swz(slot)) << 4) + 8 * h);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const float f = __uint_as_float((x & 1) ? w[x >> 1] & 0xffff0000u : w[x >> 1] << 16);
              if ((__float_as_uint(f) & 0x7f800000u) == 0x7f800000u) o[b][4 * i + x] += weight * f;
            }
          }
      }
    }
  }

  // NT x 32 keys from t0 on, in LDS at k and v.
  template <int NT>
  __device__ __forceinline__ void step(const bf16x8 (&q)[Tile<D>::kKSteps], const KLDS char* k, const KLDS char* v, int t0, int end,
                                       int end_min, float scale2) {
    const int lane = threadIdx.x & 63, h = lane >> 5;
    // K: token lane & 31, piece (2 ks + h) ^ swz; V: see the file's head
    const int k0 = (lane & 31) * 2 * D + ((h ^ swz(lane & 31)) << 4);
    const int k_at[4] = {k0, k0 ^ 32, k0 ^ 64, k0 ^ 96};
    const int v_tok = 4 * h + ((lane & 15) >> 2);
    const int v0 = v_tok * 2 * D + (((((lane >> 4) & 1) * 2 + ((lane >> 1) & 1)) ^ swz(v_tok)) << 4) + (lane & 1) * 8;
    const int v_at[2] = {v0, v0 ^ 64};
    f32x16 s[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      s[n] = (f32x16)(0.0f);
#pragma unroll
      for (int ks = 0; ks < Tile<D>::kKSteps; ++ks) {
        const bf16x8 a = *(const KLDS bf16x8*)(k + n * 32 * 2 * D + k_at[ks & 3] + (ks >> 2) * 128);
        s[n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, q[ks], s[n], 0, 0, 0);
      }
    }
    const bool edge = t0 + NT * 32 > end_min;  // a key some row of the wave does not see
    if (edge) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (t0 + n * 32 + 8 * (i >> 2) + 4 * h + (i & 3) >= end) s[n][i] = -INFINITY;
    }
    float top = s[0][0];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 16; ++i) top = fmaxf(top, s[n][i]);
    top = fmaxf(top, other_half(top)) * scale2;
    if (__any(top > m + kGrow)) {
      const float to = fmaxf(m, top);
      const float alpha = m == to ? 1.0f : __builtin_amdgcn_exp2f(m - to);
      m = to;
      l *= alpha;
#pragma unroll
      for (int b = 0; b < Tile<D>::kBlocks; ++b) o[b] *= alpha;
    }
    const float base = m == -INFINITY ? 0.0f : m;
    bf16x8 p[NT * 2];
    float sum = 0.0f;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(s[n][8 * u + 2 * i], scale2, -base));
          const float y = __builtin_amdgcn_exp2f(__builtin_fmaf(s[n][8 * u + 2 * i + 1], scale2, -base));
          sum += x + y;
          w[i] = pack2(x, y);
        }
        p[2 * n + u] = __builtin_bit_cast(bf16x8, w);
      }
    l += sum;
    // A value that is not finite would reach the rows that do not see its token as 0 * inf. Where
    // some row does not see all of the stage's tokens, look for one; if there is one, such values
    // stay out of the product and are added to the rows that see them one token at a time.
    if (edge) {
      uint32_t worst = 0;
#pragma nounroll
      for (int c = 0; c < 2 * NT; ++c)
#pragma unroll
        for (int b = 0; b < Tile<D>::kBlocks; ++b) worst = max(worst, exponents(__builtin_bit_cast(u32x4, v_operand(v, v_at, 0, c, b))));
      if (__any(worst == 0x7f80u)) {
        spoiled<NT>(p, v, v_at, t0, end);
        return;
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int b = 0; b < Tile<D>::kBlocks; ++b)
          o[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v_operand(v, v_at, n, u, b), p[2 * n + u], o[b], 0, 0, 0);
  }
};

// A stage of TS keys, 32 at a time, as far as a row of the wave sees.
template <int TS, int D>
__device__ __forceinline__ void walk(State<D>& st, const bf16x8 (&q)[Tile<D>::kKSteps], const KLDS char* k, const KLDS char* v, int t, int end,
                                     int end_min, int end_max, float scale2) {
#pragma nounroll
  for (int s = 0; s < TS && t + s < end_max; s += 32)
    st.template step<1>(q, k + s * 2 * D, v + s * 2 * D, t + s, end, end_min, scale2);
}

template <int D>
__device__ __forceinline__ void load_q(const AttendIo& io, const StepArgs& a, const Lane& r, bf16x8 (&q)[Tile<D>::kKSteps]) {
  const int h = (threadIdx.x & 63) >> 5;
  const KGLOBAL uint16_t* p = (const KGLOBAL uint16_t*)io.q + (int64_t)r.token * io.q_stride + (int64_t)r.qh * D + 8 * h;
#pragma unroll
  for (int ks = 0; ks < Tile<D>::kKSteps; ++ks) {
    u32x4 w;
    if (io.q_vec) {
      w = *(const KGLOBAL u32x4*)(p + 16 * ks);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = (uint32_t)p[16 * ks + 2 * i] | ((uint32_t)p[16 * ks + 2 * i + 1] << 16);
    }
    if (io.negate) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] ^= 0x80008000u;
    }
    q[ks] = __builtin_bit_cast(bf16x8, w);
  }
}

// N consecutive columns of a row's result: normalised into the output, or as a partial row.
template <int N>
__device__ __forceinline__ void put(const StepArgs& a, const AttendIo& io, const AttendRun& run, int64_t part, int token, int qh, int d,
                                    const float* x, float inv) {
  if (run.direct) {
    uint16_t* out = (uint16_t*)io.out + (int64_t)token * io.out_stride + (int64_t)qh * a.dv + d;
    if (io.out_vec) {
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        u32x2 w;
        w.x = pack2(x[i] * inv, x[i + 1] * inv);
        w.y = pack2(x[i + 2] * inv, x[i + 3] * inv);
        *(KGLOBAL u32x2*)(out + i) = w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) out[i] = (uint16_t)pack2(x[i] * inv, 0.0f);
    }
  } else {
    KGLOBAL float* out = (KGLOBAL float*)a.part_o + part * a.dv + d;
#pragma unroll
    for (int i = 0; i < N; i += 4) *(KGLOBAL f32x4*)(out + i) = (f32x4){x[i], x[i + 1], x[i + 2], x[i + 3]};
  }
}

__device__ __forceinline__ void put_stats(const StepArgs& a, const AttendIo& io, const AttendRun& run, int64_t part, int token, int qh,
                                          float m, float l) {
  if (!run.direct) a.part_ml[part] = make_float2(m, l);
  else if (io.lse) io.lse[(int64_t)token * a.num_q_heads + qh] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
}

__device__ __forceinline__ int64_t part_row(const StepArgs& a, const AttendRun& run, const AttendItem& it, int head, int row) {
  return run.part0 + ((int64_t)it.split * a.heads + head) * ((int64_t)run.ntok * a.group) + row;
}

// ============================================================================
// Tiles of 128 rows: 4 waves of 32 rows share stages of 64 keys.
// ============================================================================
template <int D>
__global__ __launch_bounds__(kThreads, 2) void attend_wide(StepArgs a, AttendIo io) {
  constexpr int TS = 64, NI = TS / Tile<D>::kRowsPerLoad / kWaves;
  __shared__ __align__(1024) char k0[TS * 2 * D], v0[TS * 2 * D], k1[TS * 2 * D], v1[TS * 2 * D];
  const int item = blockIdx.x / a.heads, head = blockIdx.x - item * a.heads;
  const AttendItem it = a.items[a.num_narrow + item];
  const AttendRun run = a.runs[it.run];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const Lane r = lane_row(a, run, it, head, it.row0 + wave * 32 + (lane & 31));
  const int end_min = __builtin_amdgcn_readfirstlane(r.end), end_max = __builtin_amdgcn_readlane(r.end, 31);
  bf16x8 q[Tile<D>::kKSteps];
  load_q<D>(io, a, r, q);
  State<D> st;
  st.clear();
  const uint16_t* kp = a.k_pool + io.layer0 + head * D;
  const uint16_t* vp = a.v_pool + io.layer0 + head * D;
  const int first = wave * NI * Tile<D>::kRowsPerLoad, last = it.kv1 - 1;
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
      walk<TS>(st, q, (const KLDS char*)k0, (const KLDS char*)v0, t, r.end, end_min, end_max, io.scale2);
      if ((t += TS) >= it.kv1) break;
      __syncthreads();
      if (t + TS < it.kv1) {
        rows.load(a, kp, vp, (KLDS char*)k0, (KLDS char*)v0, first);
        rows.find(a, run, t + 2 * TS, first, last);
      }
      walk<TS>(st, q, (const KLDS char*)k1, (const KLDS char*)v1, t, r.end, end_min, end_max, io.scale2);
      if ((t += TS) >= it.kv1) break;
    }
  }
  const float l = st.l + other_half(st.l);
  if (!r.owned) return;
  const int64_t part = part_row(a, run, it, head, r.row);
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  const int h = lane >> 5;
#pragma unroll
  for (int b = 0; b < Tile<D>::kBlocks; ++b)
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
  constexpr int TS = 4096 / D, NI = TS / Tile<D>::kRowsPerLoad, STAGE = TS * 2 * D;
  constexpr int OS = D + 4;  // floats between rows of a wave's result
  __shared__ __align__(1024) char b0[kWaves][2][STAGE], b1[kWaves][2][STAGE];
  __shared__ float ml[kWaves][2][32];
  const int item = blockIdx.x / a.heads, head = blockIdx.x - item * a.heads;
  const AttendItem it = a.items[item];
  const AttendRun run = a.runs[it.run];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const Lane r = lane_row(a, run, it, head, it.row0 + (lane & 31));
  const int end_min = __builtin_amdgcn_readfirstlane(r.end), end_max = __builtin_amdgcn_readlane(r.end, 31);
  bf16x8 q[Tile<D>::kKSteps];
  load_q<D>(io, a, r, q);
  State<D> st;
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
      walk<TS>(st, q, (const KLDS char*)ka, (const KLDS char*)va, t, r.end, end_min, end_max, io.scale2);
      if ((t += STEP) >= it.kv1) break;
      __builtin_amdgcn_s_waitcnt(0x0f70);
      __builtin_amdgcn_wave_barrier();
      if (t + STEP < it.kv1) {
        rows.load(a, kp, vp, ka, va, 0);
        rows.find(a, run, t + 2 * STEP, 0, last);
      }
      walk<TS>(st, q, (const KLDS char*)kb, (const KLDS char*)vb, t, r.end, end_min, end_max, io.scale2);
      if ((t += STEP) >= it.kv1) break;
    }
  }
  // every wave's rows, then their join: thread = (row, D / 8 columns)
  const float l = st.l + other_half(st.l);
  __syncthreads();  // the stages have been read: their place holds the results
  static_assert(kWaves / 2 * 32 * OS * 4 <= (int)sizeof(b0), "results fit where the stages were");
  auto result = [&](int i, int row) { return (float*)(i < kWaves / 2 ? &b0[0][0][0] : &b1[0][0][0]) + ((i & 1) * 32 + row) * OS; };
  const int h = lane >> 5;
#pragma unroll
  for (int b = 0; b < Tile<D>::kBlocks; ++b)
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

hipError_t launch_attend_mfma(const StepArgs& a, const AttendIo& io, hipStream_t stream) {
  return a.dk == 128 ? launch<128>(a, io, stream) : launch<64>(a, io, stream);
}

}  // namespace kamera
