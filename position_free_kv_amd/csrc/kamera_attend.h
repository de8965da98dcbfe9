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
// lane its own row address: pages may be of any size and order). Rows past the range's end repeat
// its last row and are masked. Steps whose keys every row sees (nearly all) carry no mask.
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

// Where a token's 16-byte pieces lie in its LDS row: piece ^ swz(token). LDS serves 256 bytes at a
// time over 64 banks: 16 lanes of a row read (16 tokens, one piece each) and 32 lanes of a transposing
// read (32 query rows: 4 tokens x 64 bytes, 16 rows: 8 tokens x 32 bytes) must fall into 16 different
// pieces of 256 bytes. BYTES: the LDS row, 128 (two tokens to 256 bytes) or a multiple of 256.
template <int ROWS, int BYTES>
__device__ __forceinline__ constexpr int swz(int token) {
  return BYTES % 256 == 0 ? (ROWS == 32 ? ((token & 3) << 2) | ((token >> 2) & 3) : ((token & 7) << 1) | ((token >> 3) & 1))
                          : (ROWS == 32 ? ((token & 2) << 1) | ((token >> 2) & 3) : (token & 6) | ((token >> 3) & 1));
}

// One lane's view of its query row and of the range of keys.
struct Lane {
  int row;           // row of the run (clamped to its last)
  bool owned;        // false: a repeat of the last row, not written
  int token, qh;
  int end;           // keys [kv0, end) are seen
};

__device__ __forceinline__ Lane lane_row(const StepArgs& a, const AttendItem& it, int head, int row) {
  const AttendRun& run = it.run;
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
// first DV columns of a key (DK if there are fewer) are a row, the others (MLA's rope band) a row of another
// place. 32 rows: v_mfma_f32_32x32x16_bf16, lane = 32 g + n; 16 rows:
// v_mfma_f32_16x16x32_bf16, lane = 16 g + n (n: the row; g: the k slots of an operand, 8 each). A step
// takes 32 keys. Score i of lane (g, n) is that of key slot_key(i). SPLIT: values lie in two arrays that many bytes
// apart, half of a row in each.
template <int DK, int DV, int ROWS, int SPLIT = 0>
struct State {
  static constexpr int kRow = SPLIT ? DV : 2 * DV;
  static constexpr int kKeyRow = 2 * (DK < DV ? DK : DV);
  static constexpr int kRestRow = 2 * DK - kKeyRow;    // 0: no other columns
  static constexpr int kGroups = 64 / ROWS;            // 2 or 4
  static constexpr int kDepth = 8 * kGroups;           // k slots of a product: 16 or 32
  static constexpr int kKSteps = DK / kDepth;          // products of a score tile
  static constexpr int kTiles = 32 / ROWS;             // score tiles of a step: 1 or 2
  static constexpr int kScores = ROWS == 32 ? 16 : 4;  // values of a lane in one result tile
  static constexpr int kBlocks = DV / ROWS;            // output tiles
  static constexpr int kPSteps = 32 / kDepth;          // products a block takes of a step: 2 or 1
  static constexpr bool kTight = DV > 128;             // registers are short: operands are read in small groups
  typedef float Acc __attribute__((ext_vector_type(kScores)));
  Acc o[kBlocks];
  float m, l;  // l: this lane's keys only (a row's lanes are added at the end)
  bool low;    // MLA: a row of the wave has met a score of -inf in a step with a mask

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
    low = false;
  }

  // First column of operand ks. With 32 rows they follow each other; with 16 two operands share 64
  // columns, group g taking 16 g on: LDS serves a 16-byte row read in groups of 16 lanes that mix two
  // g (lanes 0-3, 12-15, 20-23, 24-27, ...), which 8 g on would send to the same banks.
  static __device__ __forceinline__ constexpr int k_column(int ks) {
    return ROWS == 32 ? kDepth * ks + 8 * group() : 64 * (ks >> 1) + 16 * group() + 8 * (ks & 1);
  }
  // the row's queries
  static __device__ __forceinline__ void load_q(const AttendIo& io, const Lane& r, bf16x8 (&q)[kKSteps]) {
    const KGLOBAL uint16_t* p = (const KGLOBAL uint16_t*)io.q + (int64_t)r.token * io.q_stride + (int64_t)r.qh * DK;
    u32x4 w[kKSteps];
    if (io.q_vec) {
#pragma unroll
      for (int ks = 0; ks < kKSteps; ++ks) w[ks] = *(const KGLOBAL u32x4*)(p + k_column(ks));
    } else {
#pragma unroll
      for (int ks = 0; ks < kKSteps; ++ks)
#pragma unroll
        for (int i = 0; i < 4; ++i) w[ks][i] = (uint32_t)p[k_column(ks) + 2 * i] | ((uint32_t)p[k_column(ks) + 2 * i + 1] << 16);
    }
    const uint32_t sign = io.negate ? 0x80008000u : 0u;
#pragma unroll
    for (int ks = 0; ks < kKSteps; ++ks) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[ks][i] ^= sign;
      q[ks] = __builtin_bit_cast(bf16x8, w[ks]);
    }
  }

  // V^T operand of output tile b and product u: the lane reads 4 columns of key 4 g + (lane & 15) / 4, and of
  // the key 8 (or 16) further on
  static __device__ __forceinline__ bf16x8 v_operand(const KLDS char* v, int u, int b) {
    const int lane = threadIdx.x & 63;
    const int token = 4 * group() + ((lane & 15) >> 2);
    constexpr int next = ROWS == 32 ? 8 : 16;
    const int piece = (ROWS == 32 ? ((lane >> 4) & 1) * 2 : 0) + ((lane >> 1) & 1);
    const int at = token * kRow + ((piece ^ swz<ROWS, kRow>(token)) << 4) + (lane & 1) * 8;
    constexpr int kSpan = kRow % 256 == 0 ? 256 : 128;  // what the pieces' places are permuted in
    const int c = b * 2 * ROWS;
    const int on = c / kRow * SPLIT + c % kRow / kSpan * kSpan + u * 16 * kRow;
    const KLDS char* p = v + ((at ^ (c % kSpan)) + on);
    const KLDS char* p2 = v + ((at ^ (c % kSpan) ^ (ROWS == 32 ? 32 : 0)) + on + next * kRow);
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((KLDS s16x4*)p);
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((KLDS s16x4*)p2);
    typedef short s16x8 __attribute__((ext_vector_type(8)));
    const s16x8 both = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_bit_cast(bf16x8, both);
  }
  // K operand ks: key n (+ ROWS tile)
  static __device__ __forceinline__ bf16x8 k_operand(const KLDS char* k, const KLDS char* rest, int tile, int ks) {
    constexpr int kLaneBytes = ROWS == 32 ? 16 : 32;           // between groups
    const int c = ROWS == 32 ? 32 * ks : 128 * (ks >> 1) + 16 * (ks & 1);  // bytes of operand ks in the row
    if (c < kKeyRow) {
      constexpr int kSpan = kKeyRow % 256 == 0 ? 256 : 128;
      const int at = row() * kKeyRow + ((group() * kLaneBytes) ^ (swz<ROWS, kKeyRow>(row()) << 4));
      return *(const KLDS bf16x8*)(k + ((at ^ (c % kSpan)) + (c / kSpan) * kSpan + tile * ROWS * kKeyRow));
    }
    const int at = row() * kRestRow + ((group() * kLaneBytes) ^ (swz<ROWS, 128>(row()) << 4)), c2 = c - kKeyRow;
    return *(const KLDS bf16x8*)(rest + ((at ^ (c2 % 128)) + (c2 / 128) * 128 + tile * ROWS * kRestRow));
  }

  // Operand u: ones for the keys before `end` whose weight is 0 (t: the first of the 32), zeros elsewhere.
  static __device__ __forceinline__ bf16x8 seen_without_weight(const bf16x8& p, int u, int t, int end) {
    const u32x4 w = __builtin_bit_cast(u32x4, p);
    u32x4 z;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      z[i] = 0;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int j = 2 * i + e;
        const int key = t + (ROWS == 32 ? slot_key(0, 8 * u + j) : slot_key(j >> 2, j & 3));
        if (key < end && ((w[i] >> (16 * e)) & 0x7f80u) == 0) z[i] |= 0x3f80u << (16 * e);
      }
    }
    return __builtin_bit_cast(bf16x8, z);
  }

  // Adds `what` to the results of block b that a mark reaches with a weight.
  __device__ __forceinline__ void reach(int b, u32x4 marks, bf16x8 weights, float what) {
    const Acc x = mfma(__builtin_bit_cast(bf16x8, marks), weights, (Acc)(0.0f));
#pragma unroll
    for (int i = 0; i < kScores; ++i) o[b][i] += x[i] > 0.0f ? what : 0.0f;
    __builtin_amdgcn_sched_barrier(0);
  }

  // O += P V for a step whose keys some row does not see (end: the keys that the lane's row sees): a value
  // that is not finite must reach the rows that see its key and no other, where a product would make 0 * inf
  // = NaN. Such values are left out of the product; where there is one, products of the weights with marks
  // (1 for inf, -inf; both for NaN) tell which results it reaches, and a product of marks with the seen keys
  // of weight 0 tells where 0 * inf is due, as in the steps without a mask.
  __device__ __forceinline__ void careful(const bf16x8 (&p)[kPSteps], const KLDS char* v, int t, int end) {
#pragma nounroll
    for (int u = 0; u < kPSteps; ++u) {
      const bf16x8 pw = kPSteps == 2 && u ? p[kPSteps - 1] : p[0];
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) {
        __builtin_amdgcn_sched_barrier(0);
        u32x4 w = __builtin_bit_cast(u32x4, v_operand(v, u, b));
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
          reach(b, up, pw, INFINITY);
          reach(b, down, pw, -INFINITY);
          reach(b, up | down, seen_without_weight(pw, u, t, end), NAN);
        }
        o[b] = mfma(__builtin_bit_cast(bf16x8, w), pw, o[b]);
      }
    }
  }

  // The same where values are columns of the keys (MLA): they are left out of the product. A row that sees a
  // value that is not finite has no finite score for its key. One of inf or NaN makes the whole row NaN by
  // itself; one of -inf gives a weight of 0, and the 0 * inf that is due is put into the result afterwards (low).
  static __device__ __forceinline__ bf16x8 finite(bf16x8 x) {
    u32x4 w = __builtin_bit_cast(u32x4, x);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if ((w[i] & 0x7f80u) == 0x7f80u) w[i] &= 0xffff0000u;
      if ((w[i] & 0x7f800000u) == 0x7f800000u) w[i] &= 0xffffu;
    }
    return __builtin_bit_cast(bf16x8, w);
  }

  // scores of 32 keys
  __device__ __forceinline__ void score(Acc (&s)[kTiles], const bf16x8 (&q)[kKSteps], const KLDS char* k, const KLDS char* rest) const {
#pragma unroll
    for (int n = 0; n < kTiles; ++n) s[n] = (Acc)(0.0f);
    constexpr int kProducts = kKSteps * kTiles;  // product c: step c / kTiles, tile c % kTiles
    constexpr int A = kTight ? 2 : kProducts;    // operands read ahead of their products
    static_assert(kProducts % A == 0, "whole groups");
    bf16x8 a[2][A];
#pragma unroll
    for (int i = 0; i < A; ++i) a[0][i] = k_operand(k, rest, i % kTiles, i / kTiles);
#pragma unroll
    for (int c = 0; c < kProducts; c += A) {
      if (c + A < kProducts) {
#pragma unroll
        for (int i = 0; i < A; ++i) a[(c / A + 1) & 1][i] = k_operand(k, rest, (c + A + i) % kTiles, (c + A + i) / kTiles);
      }
      if (kTight) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < A; ++i) s[(c + i) % kTiles] = mfma(a[(c / A) & 1][i], q[(c + i) / kTiles], s[(c + i) % kTiles]);
      if (kTight) __builtin_amdgcn_sched_barrier(0);
    }
  }

  // O += P V for 32 keys from t on
  template <bool EDGE>
  __device__ __forceinline__ void add(const bf16x8 (&p)[kPSteps], const KLDS char* v, int t, int end) {
    if constexpr (EDGE && kRestRow == 0) {
      careful(p, v, t, end);
      return;
    }
    constexpr int kProducts = kPSteps * kBlocks, A = kTight ? 2 : kProducts;
    bf16x8 a[2][A];
#pragma unroll
    for (int i = 0; i < A; ++i) a[0][i] = v_operand(v, i / kBlocks, i % kBlocks);
#pragma unroll
    for (int c = 0; c < kProducts; c += A) {
      if (c + A < kProducts) {
#pragma unroll
        for (int i = 0; i < A; ++i) a[(c / A + 1) & 1][i] = v_operand(v, (c + A + i) / kBlocks, (c + A + i) % kBlocks);
      }
      if (kTight) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < A; ++i) {
        const bf16x8 x = EDGE ? finite(a[(c / A) & 1][i]) : a[(c / A) & 1][i];
        o[(c + i) % kBlocks] = mfma(x, p[(c + i) / kBlocks], o[(c + i) % kBlocks]);
      }
      if (kTight) __builtin_amdgcn_sched_barrier(0);
    }
  }

  // weights of 32 keys from their scores: rounded to bf16 for the product (off by at most 2^-8 of each), as
  // the matrix cores take them; their sum is that of the unrounded ones, in fp32
  __device__ __forceinline__ void weigh(bf16x8 (&p)[kPSteps], const Acc (&s)[kTiles], float scale2, float base) {
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
  }

  // NT x 32 keys from t0 on, in LDS at k (rest: the columns from DV on) and v. EDGE: some row does not see
  // some of them.
  template <int NT, bool EDGE>
  __device__ __forceinline__ void step(const bf16x8 (&q)[kKSteps], const KLDS char* k, const KLDS char* rest, const KLDS char* v, int t0,
                                       int end, float scale2) {
    Acc s[NT][kTiles];
#pragma unroll
    for (int n = 0; n < NT; ++n) score(s[n], q, k + n * 32 * kKeyRow, rest + n * 32 * kRestRow);
    float top = -INFINITY, bottom = INFINITY;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int x = 0; x < kTiles; ++x)
#pragma unroll
        for (int i = 0; i < kScores; ++i) {
          if (EDGE && kRestRow != 0) bottom = fminf(bottom, s[n][x][i]);
          if (EDGE && t0 + n * 32 + slot_key(x, i) >= end) s[n][x][i] = -INFINITY;
          top = fmaxf(top, s[n][x][i]);
        }
    if (EDGE && kRestRow != 0) low |= __any(bottom == -INFINITY) != 0;
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
    bf16x8 p[NT][kPSteps];
#pragma unroll
    for (int n = 0; n < NT; ++n) weigh(p[n], s[n], scale2, base);
#pragma unroll
    for (int n = 0; n < NT; ++n) add<EDGE>(p[n], v + n * 32 * kRow, t0 + n * 32, end);
  }

  // column of values 4 i on of output tile b
  static __device__ __forceinline__ int column(int b, int i) { return b * ROWS + (ROWS == 32 ? 8 * i : 0) + 4 * group(); }
};

// Every wave's part of a stage has arrived in LDS, and every wave has read the stage before. (The
// barrier alone orders LDS instructions; loads into LDS are counted with the memory ones.)
__device__ __forceinline__ void stage_barrier() {
  __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
  __syncthreads();
}

// A stage of TS keys, as far as a row of the wave sees: NT x 32 at a time while every row sees them all.
template <int TS, int NT, int DK, int DV, int ROWS, int SPLIT>
__device__ __forceinline__ void walk(State<DK, DV, ROWS, SPLIT>& st, const bf16x8 (&q)[State<DK, DV, ROWS, SPLIT>::kKSteps], const KLDS char* k,
                                     const KLDS char* rest, const KLDS char* v, int t, int end, int end_min, int end_max, float scale2) {
  typedef State<DK, DV, ROWS, SPLIT> S;
  int s = 0;
#pragma nounroll
  for (; s < TS && t + s + 32 * NT <= end_min; s += 32 * NT)
    st.template step<NT, false>(q, k + s * S::kKeyRow, rest + s * S::kRestRow, v + s * S::kRow, t + s, end, scale2);
#pragma nounroll
  for (; s < TS && t + s < end_max; s += 32) st.template step<1, true>(q, k + s * S::kKeyRow, rest + s * S::kRestRow, v + s * S::kRow, t + s, end, scale2);
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

__device__ __forceinline__ int64_t part_row(const StepArgs& a, const AttendItem& it, int head, int row) {
  return it.run.part0 + ((int64_t)it.split * a.heads + head) * ((int64_t)it.run.ntok * a.group) + row;
}

// A wave's result: normalised into the output, or as partial rows.
template <typename S>
__device__ __forceinline__ void put_state(const StepArgs& a, const AttendIo& io, const AttendItem& it, int head,
                                          const Lane& r, const S& st, float l) {
  if (!r.owned) return;
  const int64_t part = part_row(a, it, head, r.row);
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
  for (int b = 0; b < S::kBlocks; ++b)
#pragma unroll
    for (int i = 0; i < S::kScores / 4; ++i) {
      const float x[4] = {st.o[b][4 * i], st.o[b][4 * i + 1], st.o[b][4 * i + 2], st.o[b][4 * i + 3]};
      put<4>(a, io, it.run, part, r.token, r.qh, S::column(b, i), x, inv);
    }
  if (S::group() == 0) put_stats(a, io, it.run, part, r.token, r.qh, st.m, l);
}

// Joins two waves' results for the same rows: `giver` waves put theirs into LDS at `place` (like lanes
// hold like values), the others take slot `pair`'s. place's former use has ended in every wave only
// after the first barrier here; every wave of the workgroup comes along. l: sums over whole rows.
template <typename S>
__device__ __forceinline__ void join_two(S& st, float& l, bool giver, int pair, f32x4* place, float (&ml)[2][kWaves][64], bool idle = false) {
  constexpr int kQuads = S::kScores / 4;
  const int lane = threadIdx.x & 63;
  __syncthreads();
  if (giver && !idle) {
#pragma unroll
    for (int b = 0; b < S::kBlocks; ++b)
#pragma unroll
      for (int i = 0; i < kQuads; ++i)
        place[(b * kQuads + i) * 64 + lane] = (f32x4){st.o[b][4 * i], st.o[b][4 * i + 1], st.o[b][4 * i + 2], st.o[b][4 * i + 3]};
    ml[0][pair][lane] = st.m;
    ml[1][pair][lane] = l;
  }
  __syncthreads();
  if (!giver && !idle) {
    const float m = ml[0][pair][lane], top = fmaxf(st.m, m);
    const float f0 = st.m == top ? 1.0f : __builtin_amdgcn_exp2f(st.m - top), f1 = m == top ? 1.0f : __builtin_amdgcn_exp2f(m - top);
    st.m = top;
    l = l * f0 + ml[1][pair][lane] * f1;
#pragma unroll
    for (int b = 0; b < S::kBlocks; ++b)
#pragma unroll
      for (int i = 0; i < kQuads; ++i) {
        const f32x4 y = place[(b * kQuads + i) * 64 + lane];
#pragma unroll
        for (int e = 0; e < 4; ++e) st.o[b][4 * i + e] = st.o[b][4 * i + e] * f0 + y[e] * f1;
      }
  }
}

// Four waves' results for the same rows into wave 0's: 2 and 3 into 0 and 1, then 1 into 0. even, odd:
// LDS of a wave's result each.
template <typename S>
__device__ __forceinline__ void join_waves(S& st, float& l, f32x4* even, f32x4* odd, float (&ml)[2][kWaves][64]) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  join_two(st, l, wave >= 2, wave & 1, wave & 1 ? odd : even, ml);
  join_two(st, l, wave == 1, 0, even, ml, wave >= 2);
}

}  // namespace

}  // namespace kamera
