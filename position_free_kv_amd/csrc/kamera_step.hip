// Kernels of the serving step (include/kamera_step.h) for gfx950: cos/sin table, append,
// plain attention, the join of partial attention results, page copies.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kamera_grid.h"
#include "kamera_step_desc.h"

namespace kamera {

#define KGLOBAL __attribute__((address_space(1)))

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

constexpr int kWave = 64;
constexpr int kThreads = 256;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kLog2e = 1.44269504088896340736f;

// Element types by their storage: uint16_t holds bf16 bits, float itself.
template <typename T>
__device__ __forceinline__ float to_float(T x);
template <>
__device__ __forceinline__ float to_float<uint16_t>(uint16_t x) {
  return __uint_as_float((uint32_t)x << 16);
}
template <>
__device__ __forceinline__ float to_float<float>(float x) {
  return x;
}
template <typename T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ uint16_t from_float<uint16_t>(float x) {
  return __builtin_bit_cast(uint16_t, (__bf16)x);  // round to nearest even
}
template <>
__device__ __forceinline__ float from_float<float>(float x) {
  return x;
}

// N consecutive elements as floats
template <typename T, int N>
__device__ __forceinline__ void load_floats(const KGLOBAL T* p, float* x) {
  if constexpr (N == 1) {
    x[0] = to_float<T>(p[0]);
  } else if constexpr (sizeof(T) == 2) {
    const u32x2 w = *(const KGLOBAL u32x2*)p;
    x[0] = __uint_as_float(w.x << 16);
    x[1] = __uint_as_float(w.x & 0xffff0000u);
    x[2] = __uint_as_float(w.y << 16);
    x[3] = __uint_as_float(w.y & 0xffff0000u);
  } else {
    const f32x4 w = *(const KGLOBAL f32x4*)p;
    for (int e = 0; e < 4; ++e) x[e] = w[e];
  }
}

// Pool row (page * page_size + offset) of slot `slot` of a page table.
__device__ __forceinline__ int64_t pool_row(const StepArgs& a, const KGLOBAL int32_t* pages, int slot) {
  if (a.page_shift >= 0)
    return ((int64_t)pages[slot >> a.page_shift] << a.page_shift) + (slot & (a.page_size - 1));
  const int pg = slot / a.page_size;
  return (int64_t)pages[pg] * a.page_size + (slot - pg * a.page_size);
}

// ============================================================================
// cos/sin of the appended tokens: phi = position * base^(-2i/d_rot) in fp64, rounded once to
// fp32 (as the rehydrate operator's tables). Once a step, read by every layer: 4 d_rot bytes
// a token, against 2 (Hq + 2 Hkv) d bytes of rows. 7419 tokens: 4.1 us, 64 tokens: 2.9 us (latency).
// ============================================================================
__global__ __launch_bounds__(kThreads) void step_phase(StepArgs a) {
  const int half = a.d_rot >> 1;
  const int64_t n = (int64_t)a.num_tokens * half;
  const int64_t i = (int64_t)block_number() * kThreads + threadIdx.x;
  if (i >= n) return;
  const int64_t t = i / half;
  const int p = (int)(i - t * half);
  int32_t at;
  if (a.pos) {
    at = a.pos[t];
  } else {
    const int sections = a.mrope[0] + a.mrope[1] + a.mrope[2];
    const int c = sections == 0 || p < a.mrope[0] ? 0 : (p < a.mrope[0] + a.mrope[1] ? 1 : 2);
    at = a.positions[3 * t + c];
  }
  const double phi = (double)at * a.theta[p];
  double sd, cd;
  sincos(phi, &sd, &cd);
  a.phase[t * a.d_rot + p] = (float)cd;
  a.phase[t * a.d_rot + half + p] = (float)sd;
}

// ============================================================================
// Append, any layout: one wave per (token, unit); units are the query heads, the key heads
// (MLA: the one row), and for GQA the V row. Lanes walk the unit's pairs; a pair is read and
// written by one lane, so in-place queries are safe. Elements are read one by one: 7419 tokens of 32 + 8 +
// 8 bf16 heads of 128 take 114 us here and 31 us in append_heads, which is why layouts that allow it go there.
// ============================================================================
__device__ __forceinline__ float wave_sum(float x) {
  for (int d = 32; d; d >>= 1) x += __shfl_xor(x, d, kWave);
  return x;
}

template <typename T>
__global__ __launch_bounds__(kThreads) void append_plain(StepArgs a, int64_t layer0, kamera_append_rows r) {
  const int lane = threadIdx.x & 63;
  const int nq = r.q ? a.num_q_heads : 0;
  const int units = nq + a.heads + (a.family == KAMERA_GQA ? 1 : 0);
  const int64_t task = (int64_t)block_number() * (kThreads / kWave) + (threadIdx.x >> 6);
  const int64_t t = task / units;
  if (t >= a.num_tokens) return;
  const int u = (int)(task - t * units);
  const int64_t slot = a.slots[t];
  const T* x;
  T* y;
  const T* w = nullptr;
  int norm_cols = 0, band0 = 0;
  if (u < nq) {
    x = (const T*)r.q + t * r.q_stride + (int64_t)u * a.dk;
    y = (T*)r.q_out + t * r.q_out_stride + (int64_t)u * a.dk;
    band0 = a.latent;
    w = (const T*)r.q_weight;
    norm_cols = w ? a.dk : 0;
  } else if (u < nq + a.heads) {
    const int h = u - nq;
    x = (const T*)r.k + t * r.k_stride + (int64_t)h * a.dk;
    y = (T*)a.k_pool + layer0 + slot * a.row + (int64_t)h * a.dk;
    band0 = a.latent;
    w = (const T*)r.k_weight;
    norm_cols = w ? (a.family == KAMERA_MLA ? a.latent : a.dk) : 0;
  } else {
    x = (const T*)r.v + t * r.v_stride;
    y = (T*)a.v_pool + layer0 + slot * a.row;
    for (int c = lane; c < a.row; c += kWave) y[c] = x[c];
    return;
  }
  float scale = 1.0f;
  if (norm_cols) {
    float ss = 0.0f;
    for (int c = lane; c < norm_cols; c += kWave) {
      const float f = to_float<T>(x[c]);
      ss += f * f;
    }
    scale = 1.0f / sqrtf(wave_sum(ss) / (float)norm_cols + r.eps);
  }
  for (int c = lane; c < band0; c += kWave)
    y[c] = norm_cols ? from_float<T>(to_float<T>(x[c]) * scale * to_float<T>(w[c])) : x[c];
  const int half = a.d_rot >> 1;
  const float* cs = a.phase + t * a.d_rot;
  const bool normed = norm_cols > band0;  // the norm covers the band (GQA)
  for (int p = lane; p < half; p += kWave) {
    const int ia = band0 + (a.pairing == KAMERA_NEOX ? p : 2 * p);
    const int ib = a.pairing == KAMERA_NEOX ? ia + half : ia + 1;
    float xa = to_float<T>(x[ia]), xb = to_float<T>(x[ib]);
    if (normed) {
      xa = xa * scale * to_float<T>(w[ia]);
      xb = xb * scale * to_float<T>(w[ib]);
    }
    const float c = cs[p], s = cs[half + p];
    y[ia] = from_float<T>(xa * c - xb * s);
    y[ib] = from_float<T>(xa * s + xb * c);
  }
}

// ============================================================================
// Append, bf16 heads of 16 * 2^k columns in whole 16-byte pieces (HBM-bound: rows are read and written
// once). A lane holds 16 columns of a head, the two partners of each of its 8 pairs among them
// (NeoX: 8 of each half; GPT-J: 16 in a row), so `lanes` = d / 16 lanes make a head and the sum of
// squares is a few exchanges. A wave takes heads of one token in turn and keeps the token's cosines and
// sines; a token's heads are spread over `parts` waves when there are few tokens. 7419 tokens of 32 + 8 + 8
// heads of 128: 182 MB in 31.5 us, 5.8 TB/s (a large copy reaches 4.8); 64 tokens: 4.3 us, mostly latency.
// ============================================================================
__device__ __forceinline__ void widen(u32x4 w, float* x) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ u32x4 narrow(const float* x) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  u32x4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    bf16x2 r;
    r.x = (__bf16)x[2 * i];  // round to nearest even
    r.y = (__bf16)x[2 * i + 1];
    w[i] = __builtin_bit_cast(uint32_t, r);
  }
  return w;
}
// 8 pairs: NeoX (x[j], x[8 + j]), GPT-J (x[2 j], x[2 j + 1])
template <bool NEOX>
__device__ __forceinline__ void turn(float (&x)[16], const float (&c)[8], const float (&s)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float& a = x[NEOX ? j : 2 * j];
    float& b = x[NEOX ? 8 + j : 2 * j + 1];
    const float y = a * c[j] - b * s[j];
    b = a * s[j] + b * c[j];
    a = y;
  }
}
// the lane's columns of a band of 16 * lanes: two pieces of 8
template <bool NEOX>
__device__ __forceinline__ int piece(int lane, int lanes, int half) {
  return NEOX ? 8 * lane + (half ? 8 * lanes : 0) : 16 * lane + 8 * half;
}
__device__ __forceinline__ void load_phase(const StepArgs& a, int64_t t, int lane, float (&c)[8], float (&s)[8]) {
  const KGLOBAL f32x4* p = (const KGLOBAL f32x4*)(a.phase + t * a.d_rot) + 2 * lane;
  const KGLOBAL f32x4* q = (const KGLOBAL f32x4*)(a.phase + t * a.d_rot + a.d_rot / 2) + 2 * lane;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    c[j] = p[j >> 2][j & 3];
    s[j] = q[j >> 2][j & 3];
  }
}

template <bool NEOX>
__global__ __launch_bounds__(kThreads) void append_heads(StepArgs a, int64_t layer0, kamera_append_rows r, int lanes, int parts) {
  const int64_t wave = (int64_t)block_number() * (kThreads / kWave) + (threadIdx.x >> 6);
  const int64_t t = wave / parts;
  if (t >= a.num_tokens) return;
  const int lane = threadIdx.x & (lanes - 1), seat = (threadIdx.x & 63) / lanes, seats = kWave / lanes;
  const int nq = r.q ? a.num_q_heads : 0, heads = nq + 2 * a.heads;
  const int first = piece<NEOX>(lane, lanes, 0), second = piece<NEOX>(lane, lanes, 1);
  const int64_t slot = a.slots[t];
  float c[8], s[8];
  load_phase(a, t, lane, c, s);
  float wq[16], wk[16];
  if (r.q_weight) {
    widen(*(const KGLOBAL u32x4*)((const KGLOBAL uint16_t*)r.q_weight + first), wq);
    widen(*(const KGLOBAL u32x4*)((const KGLOBAL uint16_t*)r.q_weight + second), wq + 8);
  }
  if (r.k_weight) {
    widen(*(const KGLOBAL u32x4*)((const KGLOBAL uint16_t*)r.k_weight + first), wk);
    widen(*(const KGLOBAL u32x4*)((const KGLOBAL uint16_t*)r.k_weight + second), wk + 8);
  }
  for (int u = (int)(wave - t * parts) * seats + seat; u < heads; u += parts * seats) {
    const bool is_q = u < nq, is_v = u >= nq + a.heads;
    const int h = is_q ? u : is_v ? u - nq - a.heads : u - nq;
    const KGLOBAL uint16_t* x = is_q   ? (const KGLOBAL uint16_t*)r.q + t * r.q_stride + (int64_t)h * a.dk
                                : is_v ? (const KGLOBAL uint16_t*)r.v + t * r.v_stride + (int64_t)h * a.dk
                                       : (const KGLOBAL uint16_t*)r.k + t * r.k_stride + (int64_t)h * a.dk;
    KGLOBAL uint16_t* y = is_q ? (KGLOBAL uint16_t*)r.q_out + t * r.q_out_stride + (int64_t)h * a.dk
                               : (KGLOBAL uint16_t*)(is_v ? a.v_pool : a.k_pool) + layer0 + slot * a.row + (int64_t)h * a.dk;
    u32x4 lo = *(const KGLOBAL u32x4*)(x + first), hi = *(const KGLOBAL u32x4*)(x + second);
    float f[16];
    widen(lo, f);
    widen(hi, f + 8);
    float ss = 0.0f;
#pragma unroll
    for (int j = 0; j < 16; ++j) ss += f[j] * f[j];
    for (int d = 1; d < lanes; d <<= 1) ss += __shfl_xor(ss, d, kWave);  // (a head's lanes are here together)
    if (!is_v) {
      if (is_q ? r.q_weight != nullptr : r.k_weight != nullptr) {
        const float g = 1.0f / sqrtf(ss / (float)a.dk + r.eps);
#pragma unroll
        for (int j = 0; j < 16; ++j) f[j] = f[j] * g * (is_q ? wq[j] : wk[j]);
      }
      turn<NEOX>(f, c, s);
      lo = narrow(f);
      hi = narrow(f + 8);
    }
    *(KGLOBAL u32x4*)(y + first) = lo;
    *(KGLOBAL u32x4*)(y + second) = hi;
  }
}

// ============================================================================
// Append, bf16 MLA rows in whole 16-byte pieces. Three kinds of waves for a token: the rotary bands of
// its query heads and of its KV row (16 columns a lane, as above), the norm of the KV row's latent (8
// columns a lane and turn), and, unless queries are turned in place, their latents' copy. HBM-bound: 855
// tokens of 16 query heads, 33 MB a layer, 8.2 us (4.1 TB/s; the launch's own latency is half of it).
// ============================================================================
constexpr int kLatentTurns = 4;  // latents of at most 4 * 512 columns
constexpr int kCopyTurns = 4;    // pieces a lane copies

template <bool NEOX>
__global__ __launch_bounds__(kThreads) void append_latent(StepArgs a, int64_t layer0, kamera_append_rows r, int lanes, int bands, int copies) {
  const int waves = bands + 1 + copies;
  const int64_t wave = (int64_t)block_number() * (kThreads / kWave) + (threadIdx.x >> 6);
  const int64_t t = wave / waves;
  if (t >= a.num_tokens) return;
  const int j = (int)(wave - t * waves), tid = threadIdx.x & 63;
  const int nq = r.q ? a.num_q_heads : 0;
  const KGLOBAL uint16_t* q = (const KGLOBAL uint16_t*)r.q + t * r.q_stride;
  KGLOBAL uint16_t* qo = (KGLOBAL uint16_t*)r.q_out + t * r.q_out_stride;
  const KGLOBAL uint16_t* k = (const KGLOBAL uint16_t*)r.k + t * r.k_stride;
  KGLOBAL uint16_t* ko = (KGLOBAL uint16_t*)a.k_pool + layer0 + a.slots[t] * a.row;
  if (j < bands) {
    const int lane = tid & (lanes - 1), h = j * (kWave / lanes) + tid / lanes;
    if (h > nq) return;
    const KGLOBAL uint16_t* x = (h < nq ? q + (int64_t)h * a.dk : k) + a.latent;
    KGLOBAL uint16_t* y = (h < nq ? qo + (int64_t)h * a.dk : ko) + a.latent;
    const int first = piece<NEOX>(lane, lanes, 0), second = piece<NEOX>(lane, lanes, 1);
    float c[8], s[8], f[16];
    load_phase(a, t, lane, c, s);
    widen(*(const KGLOBAL u32x4*)(x + first), f);
    widen(*(const KGLOBAL u32x4*)(x + second), f + 8);
    turn<NEOX>(f, c, s);
    *(KGLOBAL u32x4*)(y + first) = narrow(f);
    *(KGLOBAL u32x4*)(y + second) = narrow(f + 8);
  } else if (j == bands) {
    u32x4 w[kLatentTurns];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < kLatentTurns; ++i) {
      const int c = (i * kWave + tid) * 8;
      if (c >= a.latent) continue;
      w[i] = *(const KGLOBAL u32x4*)(k + c);
      float f[8];
      widen(w[i], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) ss += f[e] * f[e];
    }
    const float g = r.k_weight ? 1.0f / sqrtf(wave_sum(ss) / (float)a.latent + r.eps) : 1.0f;
#pragma unroll
    for (int i = 0; i < kLatentTurns; ++i) {
      const int c = (i * kWave + tid) * 8;
      if (c >= a.latent) continue;
      if (r.k_weight) {
        float f[8], v[8];
        widen(w[i], f);
        widen(*(const KGLOBAL u32x4*)((const KGLOBAL uint16_t*)r.k_weight + c), v);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = f[e] * g * v[e];
        w[i] = narrow(f);
      }
      *(KGLOBAL u32x4*)(ko + c) = w[i];
    }
  } else {
    const int per = a.latent / 8, total = nq * per;  // pieces of a head, of the token
    u32x4 w[kCopyTurns];
    int at[kCopyTurns];
#pragma unroll
    for (int i = 0; i < kCopyTurns; ++i) {
      const int p = ((j - bands - 1) * kCopyTurns + i) * kWave + tid, h = p / per;
      at[i] = p < total ? h * a.dk + (p - h * per) * 8 : -1;
      if (at[i] >= 0) w[i] = *(const KGLOBAL u32x4*)(q + at[i]);
    }
#pragma unroll
    for (int i = 0; i < kCopyTurns; ++i)
      if (at[i] >= 0) *(KGLOBAL u32x4*)(qo + at[i]) = w[i];
  }
}

// ============================================================================
// Attention, any layout (head widths and alignments the matrix-core kernel does not take): one
// wave per row of the tile. A wave reads 4 tokens at a time, 16 lanes to a token, each lane
// holding VEC * NJ of the key's columns; every 16-lane group runs its own online softmax
// (running maximum m and sum l in base-2 logarithms, o scaled by exp2(m_old - m)) and the four
// are joined at the end. Bound by latency: 5 requests of 8 f32 heads over 300 shared keys take 10.4 us, of
// which the chain item, page id, row is most. On large work it is far behind the matrix cores (decode of
// 64 requests over 8192 shared keys, 4 layers: 5873 us, 255 with them), which take every bf16 layout they can.
// ============================================================================
// exp2(m - to) where m may still be -inf: nothing seen yet counts as zero
__device__ __forceinline__ float shrink(float m, float to) { return m == to ? 1.0f : exp2f(m - to); }

template <typename T, int VEC, int NJ>
__global__ __launch_bounds__(kThreads) void attend_plain(StepArgs a, AttendIo io) {
  const int block = (int)block_number(), item = block / a.heads, head = block - item * a.heads;
  if (item >= a.num_items) return;
  const AttendItem it = a.items[item];
  const AttendRun& run = it.run;
  const int lane = threadIdx.x & 63, dl = lane & 15, tg = lane >> 4;
  const int row = it.row0 + (threadIdx.x >> 6);  // (a tile's rows are the workgroup's waves)
  if (row >= run.ntok * a.group) return;
  const int j = row / a.group, g = row - j * a.group;
  const int token = run.listed ? a.tok[run.tok0 + j] : run.tok0 + j;
  const int qh = head * a.group + g;
  const int end = min(it.kv1, max(run.len_a - 1, run.lim0 + j * run.lstep) + 1);
  // (differential attention: a head is a pair of KV heads, whose keys belong to one map each)
  const KGLOBAL T* kp = (const KGLOBAL T*)a.k_pool + io.layer0 + (int64_t)(a.differential ? 2 * head + (g & 1) : head) * a.dk;
  const KGLOBAL T* vp = (const KGLOBAL T*)a.v_pool + io.layer0 + (int64_t)head * a.dv;
  const KGLOBAL int32_t* pages = (const KGLOBAL int32_t*)a.pages;
  const KGLOBAL T* qp = (const KGLOBAL T*)io.q + (int64_t)token * io.q_stride + (int64_t)qh * a.dk;
  float q[NJ * VEC], o[NJ * VEC];
#pragma unroll
  for (int i = 0; i < NJ; ++i) {
    const int d = (i * 16 + dl) * VEC;
    for (int e = 0; e < VEC; ++e) q[i * VEC + e] = o[i * VEC + e] = 0.0f;
    if (d < a.dk) load_floats<T, VEC>(qp + d, q + i * VEC);
    for (int e = 0; e < VEC; ++e) q[i * VEC + e] *= io.negate ? -io.scale2 : io.scale2;
  }
  float m = -INFINITY, l = 0.0f;
  for (int t0 = it.kv0; t0 < end; t0 += 4) {
    const int t = t0 + tg;
    const bool seen = t < end;
    int64_t at = 0;
    float s = 0.0f;
    if (seen) {
      at = (t < run.len_a ? pool_row(a, pages + run.pg_a, run.slot_a + t)
                          : pool_row(a, pages + run.pg_b, run.slot_b + (t - run.len_a))) * a.row;
#pragma unroll
      for (int i = 0; i < NJ; ++i) {
        const int d = (i * 16 + dl) * VEC;
        if (d >= a.dk) continue;
        float k[VEC];
        load_floats<T, VEC>(kp + at + d, k);
        for (int e = 0; e < VEC; ++e) s += q[i * VEC + e] * k[e];
      }
    }
    for (int d = 8; d; d >>= 1) s += __shfl_xor(s, d, 16);
    if (!seen) continue;
    const float to = fmaxf(m, s);
    const bool nothing = to == -INFINITY && s == -INFINITY;  // only -inf so far: weight 0, not exp(-inf + inf)
    const float alpha = shrink(m, to), p = nothing ? 0.0f : exp2f(s - to);  // (a score of inf: NaN)
    l = l * alpha + p;
    m = to;
#pragma unroll
    for (int i = 0; i < NJ; ++i) {
      const int d = (i * 16 + dl) * VEC;
      if (d >= a.dv) continue;
      float v[VEC];
      load_floats<T, VEC>(vp + at + d, v);
      for (int e = 0; e < VEC; ++e) o[i * VEC + e] = o[i * VEC + e] * alpha + p * v[e];  // (0 * inf is NaN)
    }
  }
  float top = m;
  for (int d = 16; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d, kWave));
  const float w = shrink(m, top);
  float sum = l * w;
  for (int d = 16; d < 64; d <<= 1) sum += __shfl_xor(sum, d, kWave);
#pragma unroll
  for (int i = 0; i < NJ * VEC; ++i) {
    float x = o[i] * w;
    for (int d = 16; d < 64; d <<= 1) x += __shfl_xor(x, d, kWave);
    o[i] = x;
  }
  if (tg) return;
  if (run.direct) {
    T* out = (T*)io.out + (int64_t)token * io.out_stride + (int64_t)qh * a.dv;
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    for (int i = 0; i < NJ; ++i)
      for (int e = 0; e < VEC; ++e) {
        const int d = (i * 16 + dl) * VEC + e;
        if (d < a.dv) out[d] = from_float<T>(o[i * VEC + e] * inv);
      }
    if (io.lse && dl == 0)
      io.lse[(int64_t)token * a.num_q_heads + qh] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
  } else {
    const int64_t pr = run.part0 + ((int64_t)it.split * a.heads + head) * ((int64_t)run.ntok * a.group) + row;
    for (int i = 0; i < NJ; ++i)
      for (int e = 0; e < VEC; ++e) {
        const int d = (i * 16 + dl) * VEC + e;
        if (d < a.dv) a.part_o[pr * a.dv + d] = o[i * VEC + e];
      }
    if (dl == 0) a.part_ml[pr] = make_float2(top, sum);
  }
}

// ============================================================================
// Join of partial results: TPR threads (a wave, or a workgroup where a row has many parts) for each
// (token, query head). First every part's maximum and sum become its weight, all parts at once; then
// the weighted rows are added, 16 bytes a thread, several parts side by side where a row is shorter
// than the threads; rows of more than 256 columns are shared by workgroups, which fills the chip where
// rows are few (512 MLA rows of 36 parts: 9.4 us with one workgroup a row, 9.2 with two). Parts are
// taken in a fixed order, so the result does not depend on which workgroup finished first.
// ============================================================================
constexpr int kJoinParts = 2 * kMaxSplits;
constexpr int kJoinQuads = kWave;  // quads of columns a workgroup takes (grid.z): a wave's parts side by side

struct Parts {
  MergeToken mt;
  int heads, head, g;
  __device__ __forceinline__ int count() const { return mt.splits[0] + mt.splits[1]; }
  __device__ __forceinline__ int64_t row(int k) const {
    const int s = k >= mt.splits[0];
    return mt.part[s] + ((int64_t)(s ? k - mt.splits[0] : k) * heads + head) * mt.rows[s] + mt.row0[s] + g;
  }
};

// TPR threads' maximum or sum, every thread receiving it (a workgroup's through `red`)
template <int TPR, bool MAX>
__device__ __forceinline__ float over_threads(float x, float* red) {
  for (int d = 32; d; d >>= 1) {
    const float y = __shfl_xor(x, d, kWave);
    x = MAX ? fmaxf(x, y) : x + y;
  }
  if constexpr (TPR == kWave) return x;
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
  __syncthreads();
  x = red[0];
  for (int i = 1; i < TPR / kWave; ++i) x = MAX ? fmaxf(x, red[i]) : x + red[i];
  return x;
}

template <typename T, int TPR>
__global__ __launch_bounds__(kThreads) void attend_join(StepArgs a, AttendIo io) {
  constexpr int ROWS = kThreads / TPR;  // rows of a workgroup
  constexpr int MAXP = TPR == kWave ? kWave : kJoinParts;
  __shared__ float weight[ROWS][MAXP];
  __shared__ f32x4 held[ROWS][TPR];
  __shared__ float red[ROWS][4];
  const int sub = threadIdx.x / TPR, tid = threadIdx.x - sub * TPR;
  const int64_t task = (int64_t)block_number() * ROWS + sub;
  const int64_t i = min(task / a.num_q_heads, (int64_t)a.num_merge - 1);
  const int qh = (int)(task % a.num_q_heads);
  const bool live = task < (int64_t)a.num_merge * a.num_q_heads;
  const Parts p{a.merge[i], a.heads, qh / a.group, qh % a.group};
  const int n = p.count();
  float top = -INFINITY, sum = 0.0f, m[MAXP / TPR], l[MAXP / TPR];
#pragma unroll
  for (int j = 0; j < MAXP / TPR; ++j) {
    const int k = j * TPR + tid;
    const float2 ml = k < n ? a.part_ml[p.row(k)] : make_float2(-INFINITY, 0.0f);
    m[j] = ml.x;
    l[j] = ml.y;
    if (ml.y != 0.0f) top = fmaxf(top, ml.x);
  }
  top = over_threads<TPR, true>(top, red[sub]);
#pragma unroll
  for (int j = 0; j < MAXP / TPR; ++j) {
    const int k = j * TPR + tid;
    const float w = l[j] == 0.0f ? 0.0f : shrink(m[j], top);
    if (k < n) weight[sub][k] = w;
    sum += l[j] * w;
  }
  sum = over_threads<TPR, false>(sum, red[sub]);
  __syncthreads();
  const int quads = a.dv / 4, c0 = blockIdx.z * kJoinQuads, wide = min(quads - c0, kJoinQuads);
  T* out = (T*)io.out + (int64_t)a.merge[i].token * io.out_stride + (int64_t)qh * a.dv;
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  const KGLOBAL f32x4* rows = (const KGLOBAL f32x4*)a.part_o;
  const int side = TPR / wide, first = tid / wide, c = c0 + tid % wide;  // `side` parts at a time, `wide` threads each
  f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
  if (first < side) {
#pragma unroll 8
    for (int k = first; k < n; k += side) {
      const float w = weight[sub][k];
      const f32x4 x = rows[p.row(k) * quads + c];
      for (int e = 0; e < 4; ++e) o[e] += x[e] * w;  // (an empty part's row is 0)
    }
  }
  if (side > 1) {
    held[sub][tid] = o;
    if (TPR == kWave) {
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    } else {
      __syncthreads();
    }
    if (first == 0)
      for (int s = 1; s < side; ++s) {
        const f32x4 x = held[sub][s * wide + tid];
        for (int e = 0; e < 4; ++e) o[e] += x[e];
      }
  }
  if (live && first == 0)
    for (int e = 0; e < 4; ++e) out[4 * c + e] = from_float<T>(o[e] * inv);
  if (live && io.lse && tid == 0 && blockIdx.z == 0)
    io.lse[(int64_t)a.merge[i].token * a.num_q_heads + qh] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
}

// Up to 4 parts a row: a thread for 16 bytes of a row, all its reads at once (78000 rows of 2 parts, 100 MB:
// 23 us; with a wave a row 47 us. With up to 16 parts this way is slower than the waves').
constexpr int kFewParts = 4;
template <typename T>
__global__ __launch_bounds__(kThreads) void attend_join_few(StepArgs a, AttendIo io) {
  constexpr int P = kFewParts;
  const int quads = a.dv / 4;
  const int64_t at = (int64_t)block_number() * kThreads + threadIdx.x, task = at / quads;
  const int c = (int)(at - task * quads);
  const int64_t i = task / a.num_q_heads;
  if (i >= a.num_merge) return;
  const int qh = (int)(task - i * a.num_q_heads);
  const Parts p{a.merge[i], a.heads, qh / a.group, qh % a.group};
  const int n = p.count();
  float2 ml[P];
  f32x4 x[P];
#pragma unroll
  for (int k = 0; k < P; ++k) {
    ml[k] = make_float2(-INFINITY, 0.0f);
    if (k < n) {
      const int64_t row = p.row(k);
      ml[k] = a.part_ml[row];
      x[k] = ((const KGLOBAL f32x4*)a.part_o)[row * quads + c];
    }
  }
  float top = -INFINITY, sum = 0.0f;
#pragma unroll
  for (int k = 0; k < P; ++k)
    if (ml[k].y != 0.0f) top = fmaxf(top, ml[k].x);
  f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int k = 0; k < P; ++k) {
    if (k >= n) continue;
    const float w = ml[k].y == 0.0f ? 0.0f : shrink(ml[k].x, top);  // (an empty part's row is 0)
    sum += ml[k].y * w;
    for (int e = 0; e < 4; ++e) o[e] += x[k][e] * w;
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  T* out = (T*)io.out + (int64_t)p.mt.token * io.out_stride + (int64_t)qh * a.dv + 4 * c;
  for (int e = 0; e < 4; ++e) out[e] = from_float<T>(o[e] * inv);
  if (io.lse && c == 0) io.lse[(int64_t)p.mt.token * a.num_q_heads + qh] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
}

// Rows that are not whole 16-byte pieces: a wave a row, one part after the other.
template <typename T>
__global__ __launch_bounds__(kThreads) void attend_join_any(StepArgs a, AttendIo io) {
  const int64_t task = (int64_t)block_number() * (kThreads / kWave) + (threadIdx.x >> 6);
  const int64_t i = task / a.num_q_heads;
  if (i >= a.num_merge) return;
  const int qh = (int)(task - i * a.num_q_heads);
  const int lane = threadIdx.x & 63;
  const Parts p{a.merge[i], a.heads, qh / a.group, qh % a.group};
  const int n = p.count();
  float top = -INFINITY, sum = 0.0f;
  for (int k = lane; k < n; k += kWave) {
    const float2 ml = a.part_ml[p.row(k)];
    if (ml.y != 0.0f) top = fmaxf(top, ml.x);
  }
  for (int d = 32; d; d >>= 1) top = fmaxf(top, __shfl_xor(top, d, kWave));
  for (int c = lane; c - lane < a.dv; c += kWave) {
    float o = 0.0f;
    sum = 0.0f;
    for (int k = 0; k < n; ++k) {
      const int64_t pr = p.row(k);
      const float2 ml = a.part_ml[pr];
      const float w = ml.y == 0.0f ? 0.0f : shrink(ml.x, top);  // (an empty part's row is 0)
      sum += ml.y * w;
      if (c < a.dv) o += a.part_o[pr * a.dv + c] * w;
    }
    if (c < a.dv)
      ((T*)io.out)[(int64_t)p.mt.token * io.out_stride + (int64_t)qh * a.dv + c] = from_float<T>(sum == 0.0f ? 0.0f : o / sum);
  }
  if (io.lse && lane == 0)
    io.lse[(int64_t)p.mt.token * a.num_q_heads + qh] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
}

// ============================================================================
// Page copies: each thread owns a few columns of the page in one layer of one tensor and carries its
// chain's copies out in order, so a page is never overwritten before its columns were read, without
// any ordering between threads. A source may be read earlier than its turn, never later: the reads of
// kBatch copies go out together, so that a long chain (a cycle through a thousand pages) does not wait
// for one page after the other. HBM-bound: 768 pages in 12 layers of a 4096-page pool, 1.21 GB, 221 us
// (5.5 TB/s); 64 pages in 28 layers, 117 MB, 18.3 us (6.4 TB/s).
// ============================================================================
constexpr int kBatch = 16;

template <typename U, bool CHAINS>
__global__ __launch_bounds__(kThreads) void copy_pages(CopyArgs a, InlineCopies in) {
  const int64_t cols = a.page_bytes / (int64_t)sizeof(U);
  const int64_t blocks = (cols + kThreads - 1) / kThreads;
  int64_t b = block_number();
  const int64_t col = (b % blocks) * kThreads + threadIdx.x;
  b /= blocks;
  const int chain = (int)(b % a.chains);
  b /= a.chains;
  const int layer = (int)(b % a.layers), tensor = (int)(b / a.layers);
  if (col >= cols || tensor >= a.tensors) return;
  U* base = (U*)(a.pool[tensor] + layer * a.layer_bytes) + col;
  if constexpr (!CHAINS) {  // each copy alone
    const PageCopy p = a.copies ? a.copies[chain] : in.c[chain];
    base[p.dst * cols] = base[p.src * cols];
  } else {
    U kept = {};
    const int c1 = a.chain[chain + 1];
    for (int c = a.chain[chain]; c < c1; c += kBatch) {
      U x[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (c + i < c1 && a.copies[c + i].src >= 0) x[i] = base[a.copies[c + i].src * cols];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (c + i >= c1) continue;
        const PageCopy p = a.copies[c + i];
        if (p.dst < 0) kept = x[i];
        else base[p.dst * cols] = p.src < 0 ? kept : x[i];
      }
    }
  }
}

// Rings: kSegments threads share a column, each a part of the ring. What a part reads last is what the
// next part writes first, so every thread reads that page before any of them writes: the parts then do
// not depend on each other. (A 1024-page cycle in 8 layers of GQA rows: 310 us, one thread a column 948.)
constexpr int kSegments = 16, kColumns = kThreads / kSegments;

template <typename U>
__global__ __launch_bounds__(kThreads) void copy_rings(CopyArgs a) {
  const int64_t cols = a.page_bytes / (int64_t)sizeof(U);
  const int64_t blocks = (cols + kColumns - 1) / kColumns;
  int64_t b = block_number();
  const int64_t col = (b % blocks) * kColumns + threadIdx.x % kColumns;
  b /= blocks;
  const int ring = a.chains + (int)(b % a.rings);
  b /= a.rings;
  const int layer = (int)(b % a.layers), tensor = (int)(b / a.layers);
  if (tensor >= a.tensors) return;  // (a whole workgroup)
  const KGLOBAL int32_t* copies = (const KGLOBAL int32_t*)a.copies;  // source, destination, source, ...
  const int r0 = a.chain[ring], n = a.chain[ring + 1] - r0, each = (n + kSegments - 1) / kSegments;
  const int c0 = r0 + min((int)(threadIdx.x / kColumns) * each, n), c1 = min(c0 + each, r0 + n);
  KGLOBAL U* base = (KGLOBAL U*)(a.pool[tensor] + layer * a.layer_bytes) + col;
  const bool mine = col < cols && c0 < c1;
  U last = {}, x[kBatch] = {};
  auto read = [&](int c) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (c + i < c1 - 1) x[i] = base[copies[2 * (c + i)] * cols];
  };
  if (mine) {
    last = base[copies[2 * (c1 - 1)] * cols];
    read(c0);  // (the first batch's as well)
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  if (!mine) return;
  for (int c = c0;;) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (c + i < c1) base[copies[2 * (c + i) + 1] * cols] = c + i == c1 - 1 ? last : x[i];
    if ((c += kBatch) >= c1) break;
    read(c);
  }
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <typename T, int VEC>
hipError_t plain_attend(const StepArgs& a, const AttendIo& io, int64_t grid, hipStream_t stream) {
  const int nj = ((a.dk > a.dv ? a.dk : a.dv) + 16 * VEC - 1) / (16 * VEC);
  const dim3 g = grid_of(grid), b(kThreads);
  if (nj * VEC <= 8) hipLaunchKernelGGL((attend_plain<T, VEC, 8 / VEC>), g, b, 0, stream, a, io);
  else if (nj * VEC <= 16) hipLaunchKernelGGL((attend_plain<T, VEC, 16 / VEC>), g, b, 0, stream, a, io);
  else if (nj * VEC <= 40) hipLaunchKernelGGL((attend_plain<T, VEC, 40 / VEC>), g, b, 0, stream, a, io);
  else hipLaunchKernelGGL((attend_plain<T, VEC, 64 / VEC>), g, b, 0, stream, a, io);
  return hipGetLastError();
}

template <typename T>
hipError_t plain_typed(const StepArgs& a, const AttendIo& io, hipStream_t stream) {
  const int64_t grid = (int64_t)a.num_items * a.heads;
  // four columns at a time where every row and head starts on a four-column boundary
  const size_t al = 4 * sizeof(T);
  const bool vec = a.dk % 4 == 0 && a.dv % 4 == 0 && a.row % 4 == 0 && io.q_stride % 4 == 0 && io.layer0 % 4 == 0 &&
                   (uintptr_t)io.q % al == 0 && (uintptr_t)a.k_pool % al == 0 && (uintptr_t)a.v_pool % al == 0;
  return vec ? plain_attend<T, 4>(a, io, grid, stream) : plain_attend<T, 1>(a, io, grid, stream);
}

template <typename T>
hipError_t attend_typed(const StepArgs& a, const AttendIo& io, hipStream_t stream) {
  if (a.num_items > 0) {
    const hipError_t e = a.kernel == ATTEND_HEADS    ? launch_attend_heads(a, io, stream)
                         : a.kernel == ATTEND_LATENT ? launch_attend_latent(a, io, stream)
                                                     : plain_typed<T>(a, io, stream);
    if (e != hipSuccess) return e;
  }
  const int64_t rows = (int64_t)a.num_merge * a.num_q_heads;
  if (rows == 0) return hipSuccess;
  const dim3 b(kThreads);
  const int64_t by_wave = ceil_div(rows, kThreads / kWave);
  const unsigned blocks = (unsigned)ceil_div(a.dv / 4, kJoinQuads);
  if (a.dv % 4) hipLaunchKernelGGL((attend_join_any<T>), grid_of(by_wave), b, 0, stream, a, io);
  else if (a.max_parts <= kFewParts) hipLaunchKernelGGL((attend_join_few<T>), grid_of(ceil_div(rows * (a.dv / 4), kThreads)), b, 0, stream, a, io);
  else if (join_by_wave(rows, a.max_parts)) hipLaunchKernelGGL((attend_join<T, kWave>), grid_of(by_wave, blocks), b, 0, stream, a, io);
  else hipLaunchKernelGGL((attend_join<T, kThreads>), grid_of(rows, blocks), b, 0, stream, a, io);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_step_phase(const StepArgs& a, hipStream_t stream) {
  const int64_t blocks = ceil_div((int64_t)a.num_tokens * (a.d_rot / 2), kThreads);
  if (blocks > 0x7fffffffLL) return hipErrorInvalidValue;
  hipLaunchKernelGGL(step_phase, grid_of(blocks), dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_step_append(const StepArgs& a, int layer, const kamera_append_rows& rows, hipStream_t stream) {
  const int64_t layer0 = layer * a.layer_stride;
  const dim3 b(kThreads);
  const bool gqa = a.family == KAMERA_GQA;
  // whole 16-byte pieces everywhere?
  auto pieces = [](const void* p, int64_t stride) { return p == nullptr || ((uintptr_t)p % 16 == 0 && stride % 8 == 0); };
  const int lanes = a.d_rot / 16;
  const bool vec = a.dtype == KAMERA_BF16 && a.d_rot % 16 == 0 && (lanes & (lanes - 1)) == 0 && a.row % 8 == 0 && layer0 % 8 == 0 &&
                   pieces(rows.q, rows.q_stride) && pieces(rows.q_out, rows.q_out_stride) && pieces(rows.k, rows.k_stride) &&
                   (!gqa || pieces(rows.v, rows.v_stride)) && pieces(rows.q_weight, 0) && pieces(rows.k_weight, 0) && pieces(a.k_pool, 0) &&
                   (!gqa || pieces(a.v_pool, 0)) && (gqa || (a.latent % 8 == 0 && a.latent <= kLatentTurns * kWave * 8));
  const int nq = rows.q ? a.num_q_heads : 0;
  auto grid = [&](int64_t waves) { return ceil_div(waves, kThreads / kWave); };
  int64_t blocks;
  if (vec && gqa) {
    // a wave for each group of heads it holds at once while there are few tokens; beyond 4096 waves,
    // heads in turn save reading the token's cosines and sines again
    const int turns = (int)ceil_div(nq + 2 * a.heads, kWave / lanes);
    int parts = turns;
    while (parts > 1 && (int64_t)a.num_tokens * (parts / 2) >= 4096) parts /= 2;
    blocks = grid((int64_t)a.num_tokens * parts);
    if (blocks > 0x7fffffffLL) return hipErrorInvalidValue;
    const dim3 g = grid_of(blocks);
    if (a.pairing == KAMERA_NEOX) hipLaunchKernelGGL((append_heads<true>), g, b, 0, stream, a, layer0, rows, lanes, parts);
    else hipLaunchKernelGGL((append_heads<false>), g, b, 0, stream, a, layer0, rows, lanes, parts);
  } else if (vec) {
    const int bands = (int)ceil_div(nq + 1, kWave / lanes);
    const int copies = nq == 0 || rows.q == rows.q_out ? 0 : (int)ceil_div((int64_t)nq * (a.latent / 8), kCopyTurns * kWave);
    blocks = grid((int64_t)a.num_tokens * (bands + 1 + copies));
    if (blocks > 0x7fffffffLL) return hipErrorInvalidValue;
    const dim3 g = grid_of(blocks);
    if (a.pairing == KAMERA_NEOX) hipLaunchKernelGGL((append_latent<true>), g, b, 0, stream, a, layer0, rows, lanes, bands, copies);
    else hipLaunchKernelGGL((append_latent<false>), g, b, 0, stream, a, layer0, rows, lanes, bands, copies);
  } else {
    blocks = grid((int64_t)a.num_tokens * (nq + a.heads + (gqa ? 1 : 0)));
    if (blocks > 0x7fffffffLL) return hipErrorInvalidValue;
    const dim3 g = grid_of(blocks);
    if (a.dtype == KAMERA_BF16) hipLaunchKernelGGL((append_plain<uint16_t>), g, b, 0, stream, a, layer0, rows);
    else hipLaunchKernelGGL((append_plain<float>), g, b, 0, stream, a, layer0, rows);
  }
  return hipGetLastError();
}

hipError_t launch_step_attend(const StepArgs& a, int layer, const void* q, int64_t q_stride, void* out,
                              int64_t out_stride, float* lse, float scale, hipStream_t stream) {
  AttendIo io{q, out, lse, q_stride, out_stride, layer * a.layer_stride, fabsf(scale) * kLog2e, scale < 0.0f, 0, 0};
  // -inf marks a masked score: a scale of zero would make it NaN, the smallest one keeps it
  if (a.kernel != ATTEND_PLAIN) io.scale2 = fmaxf(io.scale2, 1.17549435e-38f);
  io.q_vec = q_stride % 8 == 0 && (uintptr_t)q % 16 == 0;
  io.out_vec = out_stride % 4 == 0 && (uintptr_t)out % 8 == 0;
  if (a.dtype == KAMERA_BF16) return attend_typed<uint16_t>(a, io, stream);
  return attend_typed<float>(a, io, stream);
}

hipError_t launch_attend_plain(const StepArgs& a, const AttendIo& io, hipStream_t stream) {
  if (a.num_items == 0) return hipSuccess;
  return a.dtype == KAMERA_BF16 ? plain_typed<uint16_t>(a, io, stream) : plain_typed<float>(a, io, stream);
}

hipError_t launch_copy_pages(const CopyArgs& a, const InlineCopies* inl, hipStream_t stream) {
  const int64_t lists = (int64_t)a.layers * a.tensors, cols = a.page_bytes / a.unit;
  const int64_t blocks = ceil_div(cols, kThreads) * a.chains * lists, ring_blocks = ceil_div(cols, kColumns) * a.rings * lists;
  if (blocks > 0x7fffffffLL || ring_blocks > 0x7fffffffLL) return hipErrorInvalidValue;
  static const InlineCopies kNone = {};
  const InlineCopies& in = inl ? *inl : kNone;
  const dim3 g = grid_of(blocks), b(kThreads), gr = grid_of(ring_blocks);
  if (blocks > 0 && a.chain) {
    if (a.unit == 16) hipLaunchKernelGGL((copy_pages<u32x4, true>), g, b, 0, stream, a, in);
    else if (a.unit == 4) hipLaunchKernelGGL((copy_pages<uint32_t, true>), g, b, 0, stream, a, in);
    else hipLaunchKernelGGL((copy_pages<uint16_t, true>), g, b, 0, stream, a, in);
  } else if (blocks > 0) {
    if (a.unit == 16) hipLaunchKernelGGL((copy_pages<u32x4, false>), g, b, 0, stream, a, in);
    else if (a.unit == 4) hipLaunchKernelGGL((copy_pages<uint32_t, false>), g, b, 0, stream, a, in);
    else hipLaunchKernelGGL((copy_pages<uint16_t, false>), g, b, 0, stream, a, in);
  }
  if (ring_blocks > 0) {
    if (a.unit == 16) hipLaunchKernelGGL((copy_rings<u32x4>), gr, b, 0, stream, a);
    else if (a.unit == 4) hipLaunchKernelGGL((copy_rings<uint32_t>), gr, b, 0, stream, a);
    else hipLaunchKernelGGL((copy_rings<uint16_t>), gr, b, 0, stream, a);
  }
  return hipGetLastError();
}

}  // namespace kamera
