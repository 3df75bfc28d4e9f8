// C-ABI of the paged K/V cache's additions: handles on pages held in 8 bits, and page
// tables.
#include <mutex>

#include "ibp_internal.cuh"
#include "ibp_paged8.cuh"

namespace {

const ibp::PagedLaunches k8Bit = {&ibp::launch_paged8_append, &ibp::launch_paged8_bounds,
                                  &ibp::launch_paged8_step, &ibp::launch_paged8_chunk,
                                  &ibp::launch_paged8_chunk_join, &ibp::launch_paged8_stage};

inline bool misaligned(const void* p, uintptr_t to) {
  return (reinterpret_cast<uintptr_t>(p) & (to - 1u)) != 0;
}

}  // namespace

extern "C" {

ibp_status ibp_paged_create_8bit(ibp_paged** out, const ibp_paged_desc* d, void* k_scales,
                                 void* v_scales) {
  if (!out) return IBP_EINVAL;
  *out = nullptr;
  if (!k_scales || !v_scales) return IBP_EINVAL;
  return ibp::paged_create(out, d, static_cast<uint8_t*>(k_scales),
                           static_cast<uint8_t*>(v_scales), &k8Bit);
}

ibp_status ibp_paged_resize(const ibp_paged* c, const ibp_paged_tables* t, const int32_t* target,
                            int32_t* q_starts, int64_t* slots, uint32_t n_tokens,
                            ibp_stream_t stream) {
  if (!c || !t) return IBP_EINVAL;
  if (t->n_seqs == 0) return IBP_OK;
  if (!t->page_table || !t->kv_lens || !t->free_pages || !t->state || !target ||
      t->max_pages == 0 || t->table_stride < t->max_pages || (n_tokens && !q_starts))
    return IBP_EINVAL;
  // the limits of a batch
  if (((uint64_t)t->max_pages << c->g.page_lg) > (1ull << 30) || n_tokens > 0x1FFFFFFFu ||
      t->n_seqs > 0xFFFFFFu)
    return IBP_EINVAL;
  if (misaligned(t->page_table, 4) || misaligned(t->kv_lens, 4) || misaligned(t->free_pages, 4) ||
      misaligned(t->state, 4) || misaligned(target, 4) || misaligned(q_starts, 4) ||
      misaligned(slots, 8))
    return IBP_EALIGN;
  int d = -1;
  if (cudaGetDevice(&d) != cudaSuccess) return IBP_ECUDA;
  if (d != c->device) return IBP_EINVAL;
  ibp::PagedTablesArgs a;
  a.table = t->page_table;
  a.kv_lens = t->kv_lens;
  a.free_pages = t->free_pages;
  a.state = t->state;
  a.target = target;
  a.q_starts = q_starts;
  a.slots = n_tokens ? slots : nullptr;
  a.status = c->g.status;
  a.table_stride = t->table_stride;
  a.n_seqs = t->n_seqs;
  a.max_pages = t->max_pages;
  a.n_tokens = n_tokens;
  a.n_pages = c->g.n_pages;
  a.page_lg = c->g.page_lg;
  std::lock_guard<std::mutex> lock(ibp::call_lock(t->state));
  return ibp::launch_paged_resize(a, c->sm_count, reinterpret_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? IBP_OK
             : IBP_ECUDA;
}

}  // extern "C"
