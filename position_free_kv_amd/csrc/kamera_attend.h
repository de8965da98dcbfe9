// Device code shared by the matrix-core attention kernels (kamera_attend.hip: GQA/MHA heads,
// kamera_attend_latent.hip: MLA rows).
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
#pragma once

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

// Exchanges inside a wave without LDS: the swaps leave a row's value and its partner's in two
// registers, in the same order on both sides. Rows of 32 lanes: one partner; of 16: three.
struct Pair {
  float a, b;
};
__device__ __forceinline__ Pair halves(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return Pair{__uint_as_float(r[0]), __uint_as_float(r[1])};
}
__device__ __forceinline__ Pair quarters(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return Pair{__uint_as_float(r[0]), __uint_as_float(r[1])};
}
template <int ROWS>
__device__ __forceinline__ float row_max(float x) {
  Pair p = halves(x);
  x = fmaxf(p.a, p.b);
  if constexpr (ROWS == 32) return x;
  p = quarters(x);
  return fmaxf(p.a, p.b);
}
template <int ROWS>
__device__ __forceinline__ float row_sum(float x) {
  Pair p = halves(x);
  x = p.a + p.b;
  if constexpr (ROWS == 32) return x;
  p = quarters(x);
  return p.a + p.b;
}

__device__ __forceinline__ int swz(int token) { return ((token & 3) << 1) | ((token >> 2) & 1); }

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

// Running state of a wave's ROWS (32 or 16) query rows: keys of DK columns, values of DV. In LDS the
// first DV columns of a key are a row of 2 DV bytes, the others (MLA's rope band) a row of another
// place. 32 rows: v_mfma_f32_32x32x16_bf16, lane = 32 g + n; 16 rows:
// v_mfma_f32_16x16x32_bf16, lane = 16 g + n (n: the row; g: the k slots of an operand, 8 each). A step
// takes 32 keys. Score i of lane (g, n) is that of key slot_key(i).
template <int DK, int DV, int ROWS>
struct State {
  static constexpr int kRow = 2 * DV;
  static constexpr int kRestRow = 2 * (DK - DV);       // 0: no other columns
  static constexpr int kGroups = 64 / ROWS;            // 2 or 4
  static constexpr int kDepth = 8 * kGroups;           // k slots of a product: 16 or 32
  static constexpr int kKSteps = DK / kDepth;          // products of a score tile
  static constexpr int kTiles = 32 / ROWS;             // score tiles of a step: 1 or 2
  static constexpr int kScores = ROWS == 32 ? 16 : 4;  // values of a lane in one result tile
  static constexpr int kBlocks = DV / ROWS;            // output tiles
  static constexpr int kPSteps = 32 / kDepth;          // products a block takes of a step: 2 or 1
  static constexpr int kTurns = 128 / (16 * kGroups);  // products between bases 128 bytes apart: 4 or 2
  static constexpr int kVTurns = 128 / (2 * ROWS);     // output tiles likewise: 2 or 4
  static constexpr int kAhead = DV > 128 ? 2 : 4;            // operands read ahead of their products
  typedef float Acc __attribute__((ext_vector_type(kScores)));
  Acc o[kBlocks];
  float m, l;  // l: this lane's keys only (a row's lanes are added at the end)

  static __device__ __forceinline__ int group() { return (threadIdx.x & 63) / ROWS; }
  static __device__ __forceinline__ int row() { return threadIdx.x & (ROWS - 1); }
  // key of value i of score tile n
  static __device__ __forceinline__ int slot_key(int n, int i) {
    return ROWS == 32 ? 8 * (i >> 2) + 4 * group() + (i & 3) : 16 * n + 4 * group() + i;
  }
  static __device__ __forceinline__ Acc mfma(bf16x8 a, bf16x8 b, Acc c) {
    if constexpr (ROWS == 32) return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    else return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) o[b] = (Acc)(0.0f);
    m = -INFINITY;
    l = 0.0f;
  }

  // the row's queries: operand ks holds columns kDepth ks + 8 g on
  static __device__ __forceinline__ void load_q(const AttendIo& io, const Lane& r, bf16x8 (&q)[kKSteps]) {
    const KGLOBAL uint16_t* p = (const KGLOBAL uint16_t*)io.q + (int64_t)r.token * io.q_stride + (int64_t)r.qh * DK + 8 * group();
    u32x4 w[kKSteps];
    if (io.q_vec) {
#pragma unroll
      for (int ks = 0; ks < kKSteps; ++ks) w[ks] = *(const KGLOBAL u32x4*)(p + kDepth * ks);
    } else {
#pragma unroll
      for (int ks = 0; ks < kKSteps; ++ks)
#pragma unroll
        for (int i = 0; i < 4; ++i) w[ks][i] = (uint32_t)p[kDepth * ks + 2 * i] | ((uint32_t)p[kDepth * ks + 2 * i + 1] << 16);
    }
    const uint32_t sign = io.negate ? 0x80008000u : 0u;
#pragma unroll
    for (int ks = 0; ks < kKSteps; ++ks) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[ks][i] ^= sign;
      q[ks] = __builtin_bit_cast(bf16x8, w[ks]);
    }
  }

  // Lane's byte offsets of V^T operands: output tile b, step u: base[b % kVTurns] + ...
  static __device__ __forceinline__ void v_base(int (&at)[kVTurns]) {
    const int lane = threadIdx.x & 63;
    const int token = 4 * group() + ((lane & 15) >> 2);
    const int piece = (ROWS == 32 ? ((lane >> 4) & 1) * 2 : 0) + ((lane >> 1) & 1);
    const int v0 = token * kRow + ((piece ^ swz(token)) << 4) + (lane & 1) * 8;
#pragma unroll
    for (int i = 0; i < kVTurns; ++i) at[i] = v0 ^ (i * 2 * ROWS);
  }
  static __device__ __forceinline__ bf16x8 v_operand(const KLDS char* v, const int (&v_at)[kVTurns], int u, int b) {
    const KLDS char* p = v + v_at[b % kVTurns] + u * 16 * kRow + (b / kVTurns) * 128;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((KLDS s16x4*)p);
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((KLDS s16x4*)(p + (ROWS == 32 ? 8 : 16) * kRow));
    typedef short s16x8 __attribute__((ext_vector_type(8)));
    const s16x8 both = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_bit_cast(bf16x8, both);
  }

  // O += P V for a step whose keys some row does not see: a value that is not finite must reach the
  // rows that see its key (weight > 0) and no other, where a product would make 0 * inf = NaN. Such
  // values are left out of the product; where there is one, products of the same weights with marks
  // (1 for inf, -inf; both for NaN) tell which results it reaches.
  __device__ __forceinline__ void careful(const bf16x8 (&p)[kPSteps], const KLDS char* v, const int (&v_at)[kVTurns]) {
#pragma nounroll
    for (int u = 0; u < kPSteps; ++u) {
      const bf16x8 pw = kPSteps == 2 && u ? p[kPSteps - 1] : p[0];
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) {
        __builtin_amdgcn_sched_barrier(0);
        u32x4 w = __builtin_bit_cast(u32x4, v_operand(v, v_at, u, b));
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) top = max(top, max((w[i] >> 16) & 0x7f80u, w[i] & 0x7f80u));
        if (__any(top == 0x7f80u)) {
          u32x4 up, down;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            up[i] = down[i] = 0;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint32_t x = (w[i] >> (16 * e)) & 0xffffu, one = 0x3f80u << (16 * e);
              if ((x & 0x7f80u) != 0x7f80u) continue;
              if (x != 0xff80u) up[i] |= one;    // inf, NaN
              if (x != 0x7f80u) down[i] |= one;  // -inf, NaN
              w[i] &= e ? 0xffffu : 0xffff0000u;
            }
          }
          const Acc x = mfma(__builtin_bit_cast(bf16x8, up), pw, (Acc)(0.0f)), y = mfma(__builtin_bit_cast(bf16x8, down), pw, (Acc)(0.0f));
#pragma unroll
          for (int i = 0; i < kScores; ++i) o[b][i] += (x[i] > 0.0f ? INFINITY : 0.0f) + (y[i] > 0.0f ? -INFINITY : 0.0f);
        }
        o[b] = mfma(__builtin_bit_cast(bf16x8, w), pw, o[b]);
      }
    }
  }

  // The same where values are columns of the keys (MLA): a row that sees such a key has no finite score
  // for it and is NaN by that, so leaving the value out is enough.
  static __device__ __forceinline__ bf16x8 finite(bf16x8 x) {
    u32x4 w = __builtin_bit_cast(u32x4, x);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if ((w[i] & 0x7f80u) == 0x7f80u) w[i] &= 0xffff0000u;
      if ((w[i] & 0x7f800000u) == 0x7f800000u) w[i] &= 0xffffu;
    }
    return __builtin_bit_cast(bf16x8, w);
  }

  // 32 keys from t0 on, in LDS at k (rest: the columns from DV on) and v.
  __device__ __forceinline__ void step(const bf16x8 (&q)[kKSteps], const KLDS char* k, const KLDS char* rest, const KLDS char* v, int t0, int end, int end_min,
                                       float scale2) {
    // K: key n (+ ROWS), piece (kGroups ks + g) ^ swz(key)
    const int k0 = row() * kRow + ((group() ^ swz(row())) << 4);
    int k_at[kTurns], v_at[kVTurns];
#pragma unroll
    for (int i = 0; i < kTurns; ++i) k_at[i] = k0 ^ (i * 16 * kGroups);
    v_base(v_at);
    Acc s[kTiles];
#pragma unroll
    for (int n = 0; n < kTiles; ++n) s[n] = (Acc)(0.0f);
    // operands a few products ahead: all at once they would not fit the registers
    constexpr int kProducts = kKSteps * kTiles;  // product c: step c / kTiles, tile c % kTiles
    static_assert(kProducts % kAhead == 0 && kPSteps * kBlocks % kAhead == 0, "whole groups");
    bf16x8 a[2][kAhead];
    const int r0 = row() * kRestRow + ((group() ^ swz(row())) << 4);
    auto key = [&](int c) {
      const int ks = c / kTiles, ks_rest = ks - DV / kDepth;
      if (ks_rest >= 0)
        return *(const KLDS bf16x8*)(rest + (c % kTiles) * ROWS * kRestRow + (r0 ^ (ks_rest % kTurns * 16 * kGroups)) + (ks_rest / kTurns) * 128);
      return *(const KLDS bf16x8*)(k + (c % kTiles) * ROWS * kRow + k_at[ks % kTurns] + (ks / kTurns) * 128);
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) a[0][i] = key(i);
#pragma unroll
    for (int c = 0; c < kProducts; c += kAhead) {
      if (c + kAhead < kProducts) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) a[(c / kAhead + 1) & 1][i] = key(c + kAhead + i);
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) s[(c + i) % kTiles] = mfma(a[(c / kAhead) & 1][i], q[(c + i) / kTiles], s[(c + i) % kTiles]);
      __builtin_amdgcn_sched_barrier(0);
    }
    const bool edge = t0 + 32 > end_min;  // a key some row of the wave does not see
    if (edge) {
#pragma unroll
      for (int n = 0; n < kTiles; ++n)
#pragma unroll
        for (int i = 0; i < kScores; ++i)
          if (t0 + slot_key(n, i) >= end) s[n][i] = -INFINITY;
    }
    float top = s[0][0];
#pragma unroll
    for (int n = 0; n < kTiles; ++n)
#pragma unroll
      for (int i = 0; i < kScores; ++i) top = fmaxf(top, s[n][i]);
    top = row_max<ROWS>(top) * scale2;
    if (__any(top > m + kGrow)) {
      const float to = fmaxf(m, top);
      const float alpha = m == to ? 1.0f : __builtin_amdgcn_exp2f(m - to);
      m = to;
      l *= alpha;
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) o[b] *= alpha;
    }
    const float base = m == -INFINITY ? 0.0f : m;
    bf16x8 p[kPSteps];
    float sum = 0.0f;
#pragma unroll
    for (int u = 0; u < kPSteps; ++u) {
      u32x4 w;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float x[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int j = 2 * i + e;  // element of the operand: 8 u + j of tile 0, or j % 4 of tile j / 4
          const float sc = ROWS == 32 ? s[0][(8 * u + j) % kScores] : s[(j >> 2) % kTiles][j & 3];
          x[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc, scale2, -base));
        }
        sum += x[0] + x[1];
        w[i] = pack2(x[0], x[1]);
      }
      p[u] = __builtin_bit_cast(bf16x8, w);
    }
    l += sum;
    if (kRestRow == 0 && edge) {
      careful(p, v, v_at);
      return;
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) a[0][i] = v_operand(v, v_at, i / kBlocks, i % kBlocks);
#pragma unroll
    for (int c = 0; c < kPSteps * kBlocks; c += kAhead) {
      if (c + kAhead < kPSteps * kBlocks) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) a[(c / kAhead + 1) & 1][i] = v_operand(v, v_at, (c + kAhead + i) / kBlocks, (c + kAhead + i) % kBlocks);
      }
      __builtin_amdgcn_sched_barrier(0);
      if (kRestRow != 0 && edge) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) a[(c / kAhead) & 1][i] = finite(a[(c / kAhead) & 1][i]);
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) o[(c + i) % kBlocks] = mfma(a[(c / kAhead) & 1][i], p[(c + i) / kBlocks], o[(c + i) % kBlocks]);
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  // column of values 4 i on of output tile b
  static __device__ __forceinline__ int column(int b, int i) { return b * ROWS + (ROWS == 32 ? 8 * i : 0) + 4 * group(); }
};

// A stage of TS keys, 32 at a time, as far as a row of the wave sees.
template <int TS, int DK, int DV, int ROWS>
__device__ __forceinline__ void walk(State<DK, DV, ROWS>& st, const bf16x8 (&q)[State<DK, DV, ROWS>::kKSteps], const KLDS char* k,
                                     const KLDS char* rest, const KLDS char* v, int t, int end, int end_min, int end_max, float scale2) {
#pragma nounroll
  for (int s = 0; s < TS && t + s < end_max; s += 32) st.step(q, k + s * 2 * DV, rest + s * 2 * (DK - DV), v + s * 2 * DV, t + s, end, end_min, scale2);
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

}  // namespace

}  // namespace kamera
