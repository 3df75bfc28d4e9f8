// C-ABI of the paged K/V cache: handles, argument checks, launches.
#include <cmath>
#include <mutex>
#include <new>

#include "ibp_internal.cuh"
#include "ibp_paged.cuh"
#include "ibp_tma.cuh"

// Status words of the handles of a device: one block per device, kept until the
// process exits, so that a handle costs no device allocation (and freeing one no
// synchronisation).
namespace {

constexpr int kDevices = 64, kWords = 4096;

struct StatusPool {
  uint32_t* words = nullptr;  // 32 bytes apart
  bool used[kWords] = {};
  bool fresh[kWords] = {};  // cleared with the block, never given out since
  int next = 0;
};

std::mutex g_pool_mu;
StatusPool g_pool[kDevices];

// A word that no handle uses, cleared; -1: none left, or no memory.
int take_status(int device, uint32_t** word) {
  if (device < 0 || device >= kDevices) return -1;
  std::lock_guard<std::mutex> lock(g_pool_mu);
  StatusPool& p = g_pool[device];
  if (!p.words) {
    if (cudaMalloc(reinterpret_cast<void**>(&p.words), 32u * kWords) != cudaSuccess ||
        cudaMemset(p.words, 0, 32u * kWords) != cudaSuccess ||
        cudaStreamSynchronize(nullptr) != cudaSuccess) {
      cudaGetLastError();
      cudaFree(p.words);
      p.words = nullptr;
      return -1;
    }
    for (bool& f : p.fresh) f = true;
  }
  for (int i = 0; i < kWords; ++i) {
    const int at = (p.next + i) % kWords;
    if (p.used[at]) continue;
    *word = p.words + 8 * at;
    // a word used before may hold that handle's last error
    if (!p.fresh[at] && (cudaMemset(*word, 0, 4) != cudaSuccess ||
                         cudaStreamSynchronize(nullptr) != cudaSuccess)) {
      cudaGetLastError();
      return -1;
    }
    p.used[at] = true;
    p.fresh[at] = false;
    p.next = at + 1;
    return at;
  }
  return -1;
}

void give_status(int device, int at) {
  std::lock_guard<std::mutex> lock(g_pool_mu);
  g_pool[device].used[at] = false;
}

}  // namespace

// The launches of one attention call hand pieces to each other through its workspace, so
// calls that share one (several threads on one stream) are enqueued one after the other:
// a lock for each workspace, found by its address.
namespace {

constexpr size_t kLocks = 256;
std::mutex g_call_mu[kLocks];

std::mutex& call_lock(const void* workspace) {
  uint64_t x = reinterpret_cast<uintptr_t>(workspace);
  x = (x >> 4) * 0x9E3779B97F4A7C15ull;  // (workspaces lie far apart: the upper bits tell)
  return g_call_mu[x >> 56];
}

}  // namespace

struct ibp_paged {
  int status_at;
  ibp::PagedGeom g;
  int device, sm_count;
  ibp::PagedMaps maps;
};

namespace {

inline bool misaligned(const void* p, uintptr_t to) {
  return (reinterpret_cast<uintptr_t>(p) & (to - 1u)) != 0;
}

inline ibp_status cu(cudaError_t e) { return e == cudaSuccess ? IBP_OK : IBP_ECUDA; }

// The pages as {head_dim, tokens of a page, heads, pages}, in boxes of 64
// channels x `tokens` tokens: rows of 128 bytes, swizzled; channels past head_dim read as zero.
bool page_map(CUtensorMap* map, const ibp_paged_desc& d, void* base, uint32_t tokens) {
  const ibp::EncodeTiledFn f = ibp::encode_tiled();
  if (!f) return false;
  const cuuint64_t dims[4] = {d.head_dim, d.page_tokens, d.kv_heads, d.n_pages};
  const cuuint64_t strides[3] = {d.token_stride, d.head_stride, d.page_stride};
  const cuuint32_t box[4] = {64, tokens < d.page_tokens ? tokens : d.page_tokens, 1, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return f(map,
           d.dtype ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, base,
           dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The handle's device is current, and the batch is one (its arrays' contents
// are checked on the device).  *empty: there is nothing to do.
ibp_status check(const ibp_paged* c, const ibp_paged_batch* b, bool* empty) {
  if (!c || !b) return IBP_EINVAL;
  *empty = b->n_tokens == 0 || b->n_seqs == 0;
  if (*empty) return IBP_OK;
  if (!b->page_table || !b->kv_lens || !b->q_starts || b->max_pages == 0 ||
      b->max_q_tokens == 0 || b->table_stride < b->max_pages)
    return IBP_EINVAL;
  // positions are 30-bit numbers (blocks of them may reach past the last), rows with their
  // heads 31-bit ones
  if (((uint64_t)b->max_pages << c->g.page_lg) > (1ull << 30) || b->n_tokens > 0x1FFFFFFFu ||
      b->n_seqs > 0xFFFFFFu)
    return IBP_EINVAL;
  if (misaligned(b->page_table, 4) || misaligned(b->kv_lens, 4) || misaligned(b->q_starts, 4))
    return IBP_EALIGN;
  int d = -1;
  if (cudaGetDevice(&d) != cudaSuccess) return IBP_ECUDA;
  return d == c->device ? IBP_OK : IBP_EINVAL;
}

ibp::PagedBatchView view(const ibp_paged_batch* b) {
  return ibp::PagedBatchView{b->page_table, b->kv_lens,   b->q_starts, b->table_stride,
                             b->n_seqs,     b->max_pages, b->n_tokens, b->max_q_tokens};
}

// Query heads: a multiple of the K/V heads, with a 31-bit number of rows.
bool heads_ok(const ibp_paged* c, const ibp_paged_batch* b, uint32_t q_heads) {
  return q_heads != 0 && q_heads % c->g.H == 0 && q_heads <= 65536u &&
         (uint64_t)b->n_tokens * q_heads <= 0x7FFFFFFFull;
}

// A token stride of `heads` heads: long enough, a multiple of 16.
ibp_status stride_ok(uint64_t stride, uint64_t heads, uint32_t D) {
  if (stride % 16u) return IBP_EALIGN;
  return stride >= heads * D * 2u ? IBP_OK : IBP_EINVAL;
}

}  // namespace

extern "C" {

ibp_status ibp_paged_create(ibp_paged** out, const ibp_paged_desc* d) {
  if (!out) return IBP_EINVAL;
  *out = nullptr;
  if (!d || !d->k || !d->v) return IBP_EINVAL;
  if (d->page_tokens < 8u || d->page_tokens > 256u || (d->page_tokens & (d->page_tokens - 1u)) ||
      d->head_dim == 0 || d->head_dim % 16u || d->head_dim > IBP_PAGED_MAX_HEAD_DIM ||
      d->kv_heads == 0 || d->kv_heads > 4096u || d->n_pages == 0 || d->n_pages > 0x7FFFFFFFu ||
      d->dtype > 1u)
    return IBP_EINVAL;
  if (misaligned(d->k, 16) || misaligned(d->v, 16) || d->page_stride % 16u ||
      d->head_stride % 16u || d->token_stride % 16u)
    return IBP_EALIGN;
  const uint64_t row = d->head_dim * 2ull, most = 1ull << 40;  // strides of a tensor map
  if (d->token_stride < row || d->head_stride < row || d->page_stride < row ||
      d->token_stride >= most || d->head_stride >= most || d->page_stride >= most)
    return IBP_EINVAL;
  ibp_paged* c = new (std::nothrow) ibp_paged;
  if (!c) return IBP_ENOMEM;
  uint32_t lg = 0;
  while ((1u << lg) < d->page_tokens) ++lg;
  c->g = ibp::PagedGeom{static_cast<uint8_t*>(d->k), static_cast<uint8_t*>(d->v),
                        d->page_stride, d->head_stride, d->token_stride, d->n_pages, lg,
                        d->kv_heads, d->head_dim, d->dtype, nullptr};
  if (cudaGetDevice(&c->device) != cudaSuccess ||
      cudaDeviceGetAttribute(&c->sm_count, cudaDevAttrMultiProcessorCount, c->device) !=
          cudaSuccess ||
      !page_map(&c->maps.k, *d, d->k, ibp::kBoxTokens) ||
      !page_map(&c->maps.v, *d, d->v, ibp::kBoxTokens)) {
    delete c;
    return IBP_ECUDA;
  }
  c->status_at = take_status(c->device, &c->g.status);
  if (c->status_at < 0) {
    delete c;
    return IBP_ENOMEM;
  }
  *out = c;
  return IBP_OK;
}

ibp_status ibp_paged_destroy(ibp_paged* c) {
  if (!c) return IBP_OK;
  give_status(c->device, c->status_at);
  delete c;
  return IBP_OK;
}

ibp_status ibp_paged_status(const ibp_paged* c, ibp_stream_t stream, ibp_status* out, int reset) {
  if (!c || !out) return IBP_EINVAL;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  uint32_t v = 0;
  if (cudaMemcpyAsync(&v, c->g.status, 4, cudaMemcpyDeviceToHost, st) != cudaSuccess ||
      cudaStreamSynchronize(st) != cudaSuccess)
    return IBP_ECUDA;
  *out = static_cast<ibp_status>(v);
  if (reset && v) return cu(cudaMemsetAsync(c->g.status, 0, 4, st));
  return IBP_OK;
}

ibp_status ibp_paged_append(const ibp_paged* c, const ibp_paged_batch* b, const void* k,
                            const void* v, uint64_t kv_stride, const void* q, uint64_t q_stride,
                            void* q_out, uint64_t qo_stride, uint32_t q_heads, const void* q_norm,
                            const void* k_norm, float eps, const float* cos_sin, uint32_t n_pos,
                            uint32_t rot_dim, uint32_t pairs, ibp_stream_t stream) {
  bool empty;
  ibp_status e = check(c, b, &empty);
  if (e != IBP_OK || empty) return e;
  if (!k || !v || (q && !q_out) || (!q && q_norm)) return IBP_EINVAL;
  if (cos_sin && (rot_dim == 0 || rot_dim % 16u || rot_dim > c->g.D || n_pos == 0))
    return IBP_EINVAL;
  if (!(eps >= 0.f) || !std::isfinite(eps)) return IBP_EINVAL;
  if (q && (q_heads == 0 || q_heads > 65536u)) return IBP_EINVAL;
  if (misaligned(k, 16) || misaligned(v, 16) || misaligned(q, 16) || misaligned(q_out, 16) ||
      misaligned(q_norm, 16) || misaligned(k_norm, 16) || misaligned(cos_sin, 16))
    return IBP_EALIGN;
  if ((e = stride_ok(kv_stride, c->g.H, c->g.D)) != IBP_OK) return e;
  if (q && ((e = stride_ok(q_stride, q_heads, c->g.D)) != IBP_OK ||
            (e = stride_ok(qo_stride, q_heads, c->g.D)) != IBP_OK))
    return e;
  ibp::PagedAppendArgs a;
  a.g = c->g;
  a.b = view(b);
  a.kx = static_cast<const uint8_t*>(k);
  a.vx = static_cast<const uint8_t*>(v);
  a.q = static_cast<const uint8_t*>(q);
  a.q_out = static_cast<uint8_t*>(q_out);
  a.kv_stride = kv_stride;
  a.q_stride = q_stride;
  a.qo_stride = qo_stride;
  a.Hq = q ? q_heads : 0u;
  a.q_norm = static_cast<const uint8_t*>(q_norm);
  a.k_norm = static_cast<const uint8_t*>(k_norm);
  a.eps = eps;
  a.cos_sin = cos_sin;
  a.n_pos = n_pos;
  a.rot = cos_sin ? rot_dim : 0u;
  a.pairs = pairs;
  return cu(ibp::launch_paged_append(a, c->sm_count, reinterpret_cast<cudaStream_t>(stream)));
}

ibp_status ibp_paged_attention(const ibp_paged* c, const ibp_paged_batch* b, const void* q,
                               uint64_t q_stride, uint32_t q_heads, void* out, float* lse,
                               float scale, uint32_t causal, uint32_t window,
                               const int32_t* selected, uint32_t n_selected, void* workspace,
                               uint64_t workspace_bytes, ibp_stream_t stream) {
  bool empty;
  ibp_status e = check(c, b, &empty);
  if (e != IBP_OK || empty) return e;
  if (!q || !out || !workspace || workspace_bytes < IBP_PAGED_WORKSPACE_BYTES) return IBP_EINVAL;
  if (!heads_ok(c, b, q_heads)) return IBP_EINVAL;
  if (!(scale > 0.f) || !std::isfinite(scale)) return IBP_EINVAL;
  if (window && (!causal || window > 0x7FFFFFFFu)) return IBP_EINVAL;
  if (selected && (!causal || window || n_selected == 0 || n_selected > IBP_PAGED_MAX_SELECTED))
    return IBP_EINVAL;
  if (misaligned(q, 16) || misaligned(out, 16) || misaligned(workspace, 16) ||
      misaligned(lse, 4) || misaligned(selected, 4))
    return IBP_EALIGN;
  if ((e = stride_ok(q_stride, q_heads, c->g.D)) != IBP_OK) return e;
  ibp::PagedAttnArgs a;
  a.g = c->g;
  a.b = view(b);
  a.q = static_cast<const uint8_t*>(q);
  a.q_stride = q_stride;
  a.out = static_cast<uint8_t*>(out);
  a.lse = lse;
  a.scale_log2 = scale * 1.44269504088896f;
  a.causal = causal;
  a.window = window;
  a.G = q_heads / c->g.H;
  a.selected = selected;
  a.n_sel = n_selected;
  a.ws = static_cast<uint8_t*>(workspace);
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  // Lists of pages, and sequences with one tile of 16 rows at most, go to the step
  // kernel, the others to the chunk kernel; a batch may need both, and the step kernel's
  // CTAs then fill the SMs that the chunk kernel's have left.
  const bool few = selected || (uint64_t)b->max_q_tokens * a.G <= ibp::kStepRows;
  const bool both = !few && b->n_seqs > 1u;
  a.max_rows = few || both ? ibp::kStepRows : 0u;
  std::lock_guard<std::mutex> lock(call_lock(workspace));
  cudaError_t ce = few ? cudaSuccess : ibp::launch_paged_chunk(a, c->maps, c->sm_count, st);
  if (ce == cudaSuccess && (few || both))
    ce = ibp::launch_paged_step(a, c->maps, c->sm_count, both, st);
  if (ce == cudaSuccess && !few) ce = ibp::launch_paged_chunk_join(a, c->sm_count, st);
  return cu(ce);
}

ibp_status ibp_paged_bounds(const ibp_paged* c, const ibp_paged_batch* b, void* bounds,
                            ibp_stream_t stream) {
  bool empty;
  ibp_status e = check(c, b, &empty);
  if (e != IBP_OK || empty) return e;
  if (!bounds) return IBP_EINVAL;
  if (misaligned(bounds, 16)) return IBP_EALIGN;
  return cu(ibp::launch_paged_bounds(c->g, view(b), static_cast<uint8_t*>(bounds),
                                     reinterpret_cast<cudaStream_t>(stream)));
}

ibp_status ibp_paged_scores(const ibp_paged* c, const ibp_paged_batch* b, const void* q,
                            uint64_t q_stride, uint32_t q_heads, const void* bounds,
                            float* scores, ibp_stream_t stream) {
  bool empty;
  ibp_status e = check(c, b, &empty);
  if (e != IBP_OK || empty) return e;
  if (!q || !bounds || !scores || !heads_ok(c, b, q_heads)) return IBP_EINVAL;
  if (misaligned(q, 16) || misaligned(bounds, 16) || misaligned(scores, 4)) return IBP_EALIGN;
  if ((e = stride_ok(q_stride, q_heads, c->g.D)) != IBP_OK) return e;
  return cu(ibp::launch_paged_scores(c->g, view(b), static_cast<const uint8_t*>(q), q_stride,
                                     q_heads / c->g.H, static_cast<const uint8_t*>(bounds),
                                     scores, c->sm_count, reinterpret_cast<cudaStream_t>(stream)));
}

ibp_status ibp_paged_select(const ibp_paged* c, const ibp_paged_batch* b, const float* scores,
                            uint32_t n_selected, int32_t* selected, ibp_stream_t stream) {
  bool empty;
  ibp_status e = check(c, b, &empty);
  if (e != IBP_OK || empty) return e;
  if (!scores || !selected || n_selected == 0 || n_selected > IBP_PAGED_MAX_SELECTED)
    return IBP_EINVAL;
  if (misaligned(scores, 4) || misaligned(selected, 4)) return IBP_EALIGN;
  return cu(ibp::launch_paged_select(c->g, view(b), scores, n_selected, selected, c->sm_count,
                                     reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
