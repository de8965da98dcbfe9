// Internal records of the serving step, shared by its host part (kamera_step_host.cpp) and
// its kernels. The public interface is include/kamera_step.h.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

#include "kamera_step.h"

namespace kamera {

// ---------------------------------------------------------------- host helpers (kamera_host.cpp)
kamera_status host_fail(kamera_status st, const char* fmt, ...);
void host_clear_error();
kamera_status host_check_layout(const kamera_layout* L);
// `bytes` (a multiple of 16) of `src` into device memory through the pinned staging ring, stream-ordered
kamera_status host_stage(const void* src, size_t bytes, void* dst, hipStream_t stream);

// ---------------------------------------------------------------- attention work list
// A run is a set of query tokens that read the same keys: the members of a shared prefix
// (keys: the prefix), or one request (keys: its own tokens, or its prefix and its own tokens
// one after the other). Its rows are (token j of the run, query head g of a KV head's group):
// row = j * G + g, for every KV head.
struct alignas(16) AttendRun {
  int32_t pg_a, slot_a, len_a;  // first segment: tables entry, slot of its token 0, tokens
  int32_t pg_b, slot_b;         // second segment, its tokens numbered from len_a on
  int32_t kv;                   // tokens of both
  int32_t tok0;                 // first query token (or its index in the token list)
  int32_t ntok;
  int32_t listed;               // query tokens are tok[tok0 + j] rather than tok0 + j
  int32_t lim0, lstep;          // token j sees keys t <= max(len_a - 1, lim0 + j * lstep)
  int32_t direct;               // the only part of its tokens' results: written to the output
  int64_t part0;                // first partial row: part0 + (split * H + head) * (ntok * G) + row
  int32_t splits;               // ranges its keys are cut into
  int32_t tile;                 // TileClass
};
static_assert(sizeof(AttendRun) == 64, "run record");

// A workgroup's work for each KV head: rows [row0, row0 + tile) of a run, keys [kv0, kv1).
struct alignas(16) AttendItem {
  AttendRun run;  // a copy: one read less before a workgroup knows its work
  int32_t row0, kv0, kv1;
  int32_t split;
};
static_assert(sizeof(AttendItem) == 80, "item record");

// Query token whose result is joined from partial rows of up to two runs.
struct alignas(16) MergeToken {
  int64_t part[2];
  int32_t rows[2];    // rows of the run per (split, head)
  int32_t row0[2];    // the token's first row in the run
  int32_t splits[2];
  int32_t token, pad;
};
static_assert(sizeof(MergeToken) == 48, "merge record");

// ---------------------------------------------------------------- weighing work list
// A workgroup's work for each KV head: the weights that rows [row0, row1) of a run give to keys [kv0, kv1)
// of one segment (a prefix, or a request's own tokens). Rows as in AttendRun; token j sees keys
// t <= lim0 + j * lstep.
struct alignas(16) WeighItem {
  int32_t pg, slot, kv0, kv1;
  int32_t tok0, ntok, listed, lim0;
  int32_t lstep, row0, row1, split;
  int64_t part;  // partial sums of the run: part + (split * heads + head) * kv + key; -1: straight to the scores
  int32_t kv, fresh;  // keys from `fresh` on are the step's own: their scores start at 0
};
static_assert(sizeof(WeighItem) == 64, "weigh record");
// A run whose rows are cut into `splits` ranges of `rows` rows: its keys' sums are joined from those.
struct alignas(16) WeighJoin {
  int64_t part;
  int32_t pg, slot, kv, splits;
  int32_t fresh, pad;
  int32_t rows, lim0, lstep, tile;  // tile: keys of an item (the ranges before the first row that sees any of them hold nothing)
};
static_assert(sizeof(WeighJoin) == 48, "weigh join record");

// Kernel arguments of a step (held in the plan).
struct StepArgs {
  uint16_t* k_pool;
  uint16_t* v_pool;     // MLA: the same rows
  int64_t layer_stride; // elements
  const int32_t* pages;
  const AttendItem* items;
  const int32_t* tok;
  const MergeToken* merge;
  float* part_o;        // [partial rows][dv]
  float2* part_ml;      // [partial rows]: running maximum (base-2 logarithms) and sum
  const int64_t* slots; // [N] pool slot of every appended token
  float* phase;         // [N][2][d_rot / 2]: cosines, then sines
  const int32_t* pos;   // [N] positions (NULL: `positions`, the caller's [N][3])
  const int32_t* positions;
  const double* theta;  // [d_rot / 2] rope_base^(-2 i / d_rot)
  int32_t family, dtype, pairing, row;  // row = F
  int32_t heads, group, dk, dv;         // KV heads, query heads per KV head, key and value widths
  int32_t num_q_heads, d_rot, latent, page_size;
  int32_t page_shift, num_items, num_merge, num_tokens;
  int32_t mrope[3];
  int32_t kernel;       // attention kernel of the items (AttendKernel)
  uint32_t page_magic;  // slot / page_size = slot * page_magic >> page_bits, slot < 2^31
  int32_t page_bits;
  int32_t max_parts;    // most parts of a joined row
  int32_t num_wide, num_pairs;  // the items' order: wide, pairs, narrow
  const WeighItem* weigh;
  const WeighJoin* weigh_join;
  float* weigh_part;
  int32_t num_weigh, num_weigh_join, weigh_kernel, weigh_longest;  // longest: most keys of a joined run
  uint32_t group_magic;         // row / rows_of_a_token = row * group_magic >> group_bits, for weighing
  int32_t group_bits;
  int32_t differential;
};
static_assert(sizeof(StepArgs) <= sizeof(kamera_step_plan::detail), "step arguments held in the plan");

// PLAIN: any layout. HEADS: bf16 GQA/MHA heads of 64 or 128 columns; LATENT: bf16 MLA rows of 512 + 64
// columns; DIFF: differential attention of bf16 heads of 64 or 128 columns; all on the matrix cores.
enum AttendKernel { ATTEND_PLAIN = 0, ATTEND_HEADS = 1, ATTEND_LATENT = 2, ATTEND_DIFF = 3 };
// Tiles of rows. HEADS, DIFF: narrow 32, pairs 64, wide 128 rows; LATENT: narrow 16, wide 128; PLAIN: narrow 4.
enum TileClass { TILE_WIDE = 0, TILE_PAIRS = 1, TILE_NARROW = 2 };
constexpr int tile_rows(int kernel, int tile) {
  return tile == TILE_WIDE ? 128 : tile == TILE_PAIRS ? 64 : kernel == ATTEND_PLAIN ? 4 : kernel == ATTEND_LATENT ? 16 : 32;
}

constexpr int kMaxSplits = 512;  // ranges a run's keys are cut into, at most
// A wave joins a row where rows abound (2048 rows of 10 parts: 7.0 us, 8.9 us by workgroups; 1024 rows of
// 11: 6.4 us and 5.8) or parts are few, a workgroup otherwise.
constexpr bool join_by_wave(int64_t rows, int parts) { return parts <= 8 || (parts <= 64 && rows >= 2048); }

// One attention launch: what kamera_step_attend was given.
struct AttendIo {
  const void* q;
  void* out;
  float* lse;
  int64_t q_stride, out_stride, layer0;
  float scale2;            // |scale| * log2(e)
  int32_t negate;          // the scale is negative: scores of -q
  int32_t q_vec, out_vec;  // rows of q (16 bytes) and out (8 bytes) aligned for vector access
};
hipError_t launch_attend_heads(const StepArgs& a, const AttendIo& io, hipStream_t stream);
hipError_t launch_attend_latent(const StepArgs& a, const AttendIo& io, hipStream_t stream);
// partial rows by the plain kernel (kamera_step.hip), which differential attention joins by itself
hipError_t launch_attend_plain(const StepArgs& a, const AttendIo& io, hipStream_t stream);
// Differential attention; a: the step's arguments with half the heads, pairs of KV heads, of twice the group and value width
hipError_t launch_step_attend_diff(const StepArgs& a, int layer, const void* q, int64_t q_stride, void* out, int64_t out_stride,
                                   float* lse, float scale, const kamera_differential& diff, hipStream_t stream);

// Keys of a weighing workgroup: PLAIN 16; on the matrix cores HEADS 256, LATENT 64. Items of at most kFewRows rows
// walk over more of them (matrix cores). (64 requests of one token, 32 + 8 heads, 4 layers: 256, 512 and 1024 keys 116.4, 115
// and 116.6 us, 1024 186 instead of 177 for many rows, whose workgroups then find less LDS; as tiles of many rows 147. MLA, 32
// requests, 16 heads, 4 layers: 64, 128 and 256 keys 88, 89 and 103.)
constexpr int kFewRows = 16;
constexpr int weigh_keys(int kernel) { return kernel == ATTEND_PLAIN ? 16 : kernel == ATTEND_LATENT ? 64 : 256; }
constexpr int weigh_keys_of_few(int kernel) { return kernel == ATTEND_PLAIN ? 16 : kernel == ATTEND_LATENT ? 64 : 512; }
hipError_t launch_step_weigh(const StepArgs& a, int layer, const void* q, int64_t q_stride, const float* lse, float* scores, float scale,
                             float decay, hipStream_t stream);

hipError_t launch_step_phase(const StepArgs& a, hipStream_t stream);
hipError_t launch_step_append(const StepArgs& a, int layer, const kamera_append_rows& rows, hipStream_t stream);
hipError_t launch_step_attend(const StepArgs& a, int layer, const void* q, int64_t q_stride, void* out,
                              int64_t out_stride, float* lse, float scale, hipStream_t stream);

// ---------------------------------------------------------------- page copies
// A chain is a list of copies one thread carries out in order for its columns of the page:
// entry (src, dst); src < 0: from the register saved by an entry with dst < 0.
struct PageCopy {
  int32_t src, dst;
};
struct CopyArgs {
  char* pool[2];
  int64_t layer_bytes;      // between layers
  int64_t page_bytes;
  const int32_t* chain;     // [chains + 1] first copy of each chain; NULL: each copy is a chain of its own
  const PageCopy* copies;   // NULL: they travel as the kernel's argument
  int32_t chains, layers, tensors, unit;  // unit: bytes per access (16, 4 or 2)
  // After the chains: rings, lists of kLongChain or more copies in which each copy reads the page that
  // the next one writes (the last one possibly what the first writes), and no page is read twice.
  int32_t rings;
};
constexpr int kLongChain = 64;
constexpr int kInlineCopies = 400;
struct InlineCopies {
  PageCopy c[kInlineCopies];
};
hipError_t launch_copy_pages(const CopyArgs& a, const InlineCopies* inl, hipStream_t stream);

// ---------------------------------------------------------------- eviction
struct alignas(16) EvictSeq {
  int32_t pg, slot0, num_tokens, keep;  // pg: tables entry
  int32_t first, last, kept0, pad;      // kept0: sum of min(keep, num_tokens) of the sequences before it
};
static_assert(sizeof(EvictSeq) == 32, "eviction record");

struct EvictArgs {
  char* pool[2];
  int64_t layer_bytes;   // between layers of the pool
  float* scores;
  int64_t scores_stride;
  const EvictSeq* seqs;
  const int32_t* pages;
  int32_t* kept;         // [layers][groups][total]
  int32_t* starts;       // [layers][groups][num_seqs]: kept tokens before the first one that moves
  float* phase;          // [shifts][d_rot]: cosines, then sines, of turning back by 0, 1, ... positions; NULL: keys are not turned
  const double* theta;
  int32_t num_seqs, layers, heads, together;
  int32_t total, page_size, page_bits;
  uint32_t page_magic;
  int32_t row_bytes, head_bytes, tensors, dtype;  // bytes of a pool row, and of a head's columns in it
  int32_t d_rot, band0, pairing, shifts;          // band0: first rotated column of a head
  int32_t longest, most_kept;                     // most tokens, and most kept tokens, of a sequence that loses some
};
// (kamera_evict_moves.h: the largest launch has fewer than 2^31 workgroups)
hipError_t launch_evict(const EvictArgs& a, hipStream_t stream);

}  // namespace kamera
