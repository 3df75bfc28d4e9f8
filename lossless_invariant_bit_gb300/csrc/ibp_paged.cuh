// Internal declarations of the paged K/V operators.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "ibp.h"

namespace ibp {

// A cache's geometry as the kernels take it.  Strides in bytes.
struct PagedGeom {
  uint8_t *k, *v;
  uint64_t page_stride, head_stride, token_stride;
  uint32_t n_pages, page_lg, H, D, bf16;
  uint32_t* status;
  uint8_t *k_scales, *v_scales;  // NULL, or of pages held in 8 bits: [n_pages, H]
};

struct PagedBatchView {
  const int32_t *table, *kv_lens, *q_starts;
  uint64_t table_stride;
  uint32_t n_seqs, max_pages, n_tokens, max_q;
  uint64_t table_heads;  // entries between heads' tables; 0: all heads have one
};

// Tensor maps of the key and value pages: {D, page tokens, heads, pages} with
// boxes of {64, tokens, 1, 1}, 128-byte swizzle.
struct PagedMaps {
  CUtensorMap k, v;
};

struct PagedAttnArgs {
  PagedGeom g;
  PagedBatchView b;
  const uint8_t* q;
  uint64_t q_stride;        // bytes between tokens
  uint8_t* out;             // [n_tokens, q_heads, D]
  float* lse;               // NULL or [n_tokens, q_heads]
  float scale_log2;         // scale * log2(e)
  uint32_t causal, window, G;
  const int32_t* selected;  // NULL or [n_tokens, H, n_sel]
  uint32_t n_sel;
  uint32_t max_rows;        // of a sequence: the step kernel's most, the chunk kernel takes more
  uint8_t* ws;
};

struct PagedAppendArgs {
  PagedGeom g;
  PagedBatchView b;
  const uint8_t *kx, *vx, *q;
  uint8_t* q_out;
  uint64_t kv_stride, q_stride, qo_stride;
  uint32_t Hq;  // 0: no queries
  const uint8_t *q_norm, *k_norm;
  float eps;
  const float* cos_sin;
  uint32_t n_pos, rot, pairs;
};

// Sequences that change their lengths.
struct PagedTablesArgs {
  int32_t *table, *kv_lens, *free_pages;
  int32_t* state;           // how many pages are free; a counter that is 0 between calls
  const int32_t* target;
  int32_t* q_starts;
  int64_t* slots;           // NULL or [n_tokens]
  uint32_t* status;
  uint64_t table_stride;
  uint32_t n_seqs, max_pages, n_tokens, n_pages, page_lg;
};

// workspace of an attention call: the one-token kernel's pieces, then the chunk kernel's
constexpr uint64_t kStepWsBytes = 32ull << 20;

cudaError_t launch_paged_append(const PagedAppendArgs& a, int sm_count, cudaStream_t st);
cudaError_t launch_paged_bounds(const PagedGeom& g, const PagedBatchView& b, uint8_t* bounds,
                                cudaStream_t st);
cudaError_t launch_paged_scores(const PagedGeom& g, const PagedBatchView& b, const uint8_t* q,
                                uint64_t q_stride, uint32_t G, const uint8_t* bounds,
                                float* scores, int sm_count, cudaStream_t st);
cudaError_t launch_paged_select(const PagedGeom& g, const PagedBatchView& b, const float* scores,
                                uint32_t n_sel, int32_t* selected, int sm_count,
                                cudaStream_t st);
// Sequences with at most a.max_rows rows (new tokens x query heads of a K/V
// head), or tokens with a page list each.  At one row for each of 640 heads of 1984 keys
// this kernel takes 104 us and the chunk kernel 158 (a tile of 128 rows computes 1);
// past 16 rows a second tile would read the keys again.
constexpr uint32_t kStepRows = 16;
// behind: it may start while the chunk kernel of the same call ends.
cudaError_t launch_paged_step(const PagedAttnArgs& a, const PagedMaps& m, int sm_count, bool behind,
                              cudaStream_t st);
// Tokens of a page in one box of the maps, at most.
constexpr uint32_t kBoxTokens = 128;
// Sequences with more than a.max_rows rows.
cudaError_t launch_paged_chunk(const PagedAttnArgs& a, const PagedMaps& m, int sm_count,
                               cudaStream_t st);
// Joins its pieces: after it, and after the step kernel where the call has one.
cudaError_t launch_paged_chunk_join(const PagedAttnArgs& a, int sm_count, cudaStream_t st);

cudaError_t launch_paged_resize(const PagedTablesArgs& a, int sm_count, cudaStream_t st);

// What a cache's calls launch, by what its pages hold.
struct PagedLaunches {
  decltype(&launch_paged_append) append;
  decltype(&launch_paged_bounds) bounds;
  decltype(&launch_paged_step) step;
  decltype(&launch_paged_chunk) chunk;
  decltype(&launch_paged_chunk_join) chunk_join;
  // NULL, or makes 16-bit pages of what a call's chunk kernel reads, and their table.
  cudaError_t (*stage)(const PagedAttnArgs& a, const PagedAttnArgs& staged, int sm_count,
                       cudaStream_t st);
};

#ifdef __CUDACC__

// A sequence of the batch, checked: a sequence whose q_starts are out of order
// has no rows; one whose length does not fit its table has no keys.
struct PagedSeq {
  uint32_t q0, n, L;  // first row, new tokens, tokens in the cache
  bool ok;
};

__device__ __forceinline__ PagedSeq paged_seq(const PagedBatchView& b, uint32_t page_lg,
                                              uint32_t s) {
  const int32_t q0 = __ldg(b.q_starts + s), q1 = __ldg(b.q_starts + s + 1);
  const int32_t L = __ldg(b.kv_lens + s);
  PagedSeq r;
  r.ok = true;
  r.q0 = (uint32_t)q0;
  r.n = (uint32_t)(q1 - q0);
  r.L = (uint32_t)L;
  if (q0 < 0 || q1 < q0 || (uint32_t)q1 > b.n_tokens || r.n > b.max_q) {
    r.q0 = r.n = 0;
    r.ok = false;
  }
  if (L < 0 || (uint64_t)L > ((uint64_t)b.max_pages << page_lg)) {
    r.L = 0;
    r.ok = false;
  }
  return r;
}

// The last i in [0, n) with key(i) <= x, for keys that do not decrease (0 if none; some
// number below n if they do): 32 at a time, by a whole warp with one x.
template <typename Key>
__device__ __forceinline__ uint32_t warp_search(uint32_t n, uint64_t x, Key key) {
  const uint32_t lane = threadIdx.x & 31u;
  uint32_t lo = 0, len = n;
  while (len > 1u) {
    const uint32_t step = (len + 31u) / 32u;
    const uint32_t at = lane * step;
    const uint32_t reach =
        __popc(__ballot_sync(0xFFFFFFFFu, at < len && key(lo + at) <= x));
    const uint32_t k = reach ? reach - 1u : 0u;
    lo += k * step;
    len = min(step, len - k * step);
  }
  return lo;
}

// The sequence of row t; n_seqs when none holds it.  For a whole warp.
__device__ __forceinline__ uint32_t paged_find(const PagedBatchView& b, uint32_t t) {
  if (b.n_seqs == b.n_tokens && t < b.n_seqs && __ldg(b.q_starts + t) == (int32_t)t &&
      __ldg(b.q_starts + t + 1) == (int32_t)t + 1)
    return t;  // one row per sequence
  const uint32_t s = warp_search(b.n_seqs, t, [&](uint32_t i) {
    const int32_t q = __ldg(b.q_starts + i);
    return (uint64_t)(q < 0 ? 0 : q);
  });
  return __ldg(b.q_starts + s) <= (int32_t)t && (int32_t)t < __ldg(b.q_starts + s + 1) ? s
                                                                                        : b.n_seqs;
}

// Tiles of `size` rows (or tokens of pages) of a sequence, numbered so that a tile's
// sequence is found without sums over the sequences: sequence s owns the numbers from
// q_starts[s] / size + c * s on, which leaves room for its at most n / size + c tiles.
// Returns the sequence of tile x, and the first number it owns.  For a whole warp.
__device__ __forceinline__ uint32_t paged_find_tile(const PagedBatchView& b, uint32_t size,
                                                    uint32_t c, uint32_t x, uint32_t& first) {
  auto key = [&](uint32_t i) {
    const int32_t q = __ldg(b.q_starts + i);
    return (uint64_t)((uint32_t)(q < 0 ? 0 : q) / size) + (uint64_t)c * i;
  };
  const uint32_t s = warp_search(b.n_seqs, x, key);
  first = (uint32_t)key(s);
  return s;
}

#endif

}  // namespace ibp

struct ibp_paged {
  int status_at;
  ibp::PagedGeom g;
  int device, sm_count;
  ibp::PagedMaps maps;
  const ibp::PagedLaunches* launches;
};

namespace ibp {

// The launches of one call hand something to each other through memory that calls may share:
// attention its pieces through the workspace, a resize the list of free pages.  Calls that
// share it (several threads on one stream) are enqueued one after the other: a lock for
// each workspace, and for the tables.
std::mutex& call_lock(const void* shared);

// A handle on pages of 16-bit values, or of codes of one byte under the scales given;
// the descriptor is checked.
ibp_status paged_create(ibp_paged** out, const ibp_paged_desc* desc, uint8_t* k_scales,
                        uint8_t* v_scales, const PagedLaunches* launches);

}  // namespace ibp
