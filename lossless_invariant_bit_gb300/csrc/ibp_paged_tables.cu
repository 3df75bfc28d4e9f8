// Page tables on the GPU: sequences change their lengths, pages come from the list of free
// ones or go back to it, and the new tokens get their rows and slots.
//
// have = ceil(length / page), want = ceil(target / page).  All sequences' pages that go are
// numbered r = 0 .. R - 1 by sequence and place, those that come j = 0 .. J - 1; with n free
// pages at the start
//   free[n + R - 1 - r] = page r             (the last one first, so that a growth that is
//   page j = free[n + R - 1 - j]              taken back leaves the list as it was)
// Prefix sums of R, J and the new tokens T over the sequences place everything.
//
// Two kernels, the second behind the first: pages that go are on the list before any is
// taken from it.  Each CTA sums over all sequences for itself (a few kB from L2, where a
// hand-over would cost another launch), then takes an equal part of the pages, or of the new
// tokens.  A call that cannot be served as a whole changes nothing: every CTA finds the
// same sums.  Lengths and the list's length change when the last CTA has ended, since
// all of them read the old ones.  Few sequences and tokens go to one CTA, which does one after
// the other and needs one launch.
#include "ibp_paged.cuh"
#include "ibp_sm103.cuh"

namespace ibp {
namespace {

constexpr uint32_t kThreads = 256;
constexpr uint32_t kLooks = 4;  // tokens of a thread whose pages are looked up together

struct Sums {
  uint64_t gone, come, rows;
};

// A sequence's part of the sums.
struct Part {
  uint32_t old, have, want, gone, come, rows;
  bool ok;
};

__device__ __forceinline__ Part part_of(const PagedTablesArgs& a, uint32_t s) {
  const int32_t old = a.kv_lens[s], to = __ldg(a.target + s);
  const uint64_t most = (uint64_t)a.max_pages << a.page_lg;
  Part p{};
  p.ok = old >= 0 && to >= 0 && (uint64_t)old <= most && (uint64_t)to <= most;
  if (!p.ok) return p;
  const uint32_t up = (1u << a.page_lg) - 1u;
  p.old = (uint32_t)old;
  p.have = ((uint32_t)old + up) >> a.page_lg;
  p.want = ((uint32_t)to + up) >> a.page_lg;
  p.gone = p.have > p.want ? p.have - p.want : 0u;
  p.come = p.want > p.have ? p.want - p.have : 0u;
  p.rows = to > old ? (uint32_t)(to - old) : 0u;
  return p;
}

__device__ __forceinline__ uint64_t warp_sum(uint64_t x) {
#pragma unroll
  for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, d);
  return x;
}

// The sums over all sequences, and whether the call can be served; `own`: of sequence
// threadIdx.x.
template <uint32_t kT>
__device__ __forceinline__ bool total(const PagedTablesArgs& a, Sums& t, uint32_t& n_free,
                                      Part& own) {
  __shared__ uint64_t s_sum[3][kT / 32];
  __shared__ uint32_t s_bad;
  if (threadIdx.x == 0) s_bad = 0;
  __syncthreads();
  Sums m{0, 0, 0};
  bool ok = true;
  for (uint32_t s = threadIdx.x; s < a.n_seqs; s += kT) {
    const Part p = part_of(a, s);
    if (s == threadIdx.x) own = p;
    ok = ok && p.ok;
    m.gone += p.gone, m.come += p.come, m.rows += p.rows;
  }
  m.gone = warp_sum(m.gone), m.come = warp_sum(m.come), m.rows = warp_sum(m.rows);
  const uint32_t warp = threadIdx.x >> 5;
  if ((threadIdx.x & 31u) == 0u)
    s_sum[0][warp] = m.gone, s_sum[1][warp] = m.come, s_sum[2][warp] = m.rows;
  if (!ok) s_bad = 1;
  const int32_t n = a.state[0];
  __syncthreads();
  t = Sums{0, 0, 0};
  for (uint32_t w = 0; w < kT / 32; ++w)
    t.gone += s_sum[0][w], t.come += s_sum[1][w], t.rows += s_sum[2][w];
  n_free = (uint32_t)n;
  return !s_bad && n >= 0 && n_free + t.gone <= a.n_pages && t.come <= n_free + t.gone &&
         t.rows <= a.n_tokens;
}

// Sums of x before this thread, and over all threads.
template <uint32_t kT>
__device__ __forceinline__ uint32_t scan(uint32_t x, uint32_t (&s_warp)[kT / 32], uint32_t& all) {
  const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
  uint32_t inc = x;
#pragma unroll
  for (uint32_t d = 1; d < 32u; d <<= 1) {
    const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, inc, d);
    if (lane >= d) inc += v;
  }
  __syncthreads();
  if (lane == 31u) s_warp[warp] = inc;
  __syncthreads();
  uint32_t before = 0;
  all = 0;
  for (uint32_t w = 0; w < kT / 32; ++w) {
    if (w < warp) before += s_warp[w];
    all += s_warp[w];
  }
  return before + inc - x;
}

// The last of kT sums, which do not decrease, that is at most x.
template <uint32_t kT>
__device__ __forceinline__ uint32_t last_at_most(const uint32_t (&sums)[kT], uint32_t x) {
  uint32_t at = 0;
#pragma unroll
  for (uint32_t d = kT / 2; d; d >>= 1)
    if (sums[at + d] <= x) at += d;
  return at;
}

// The last CTA to come here sets what the others have read.
template <uint32_t kT>
__device__ __forceinline__ void finish(const PagedTablesArgs& a, bool ok, const Sums& t,
                                       uint32_t n_free) {
  __shared__ uint32_t s_last;
  __syncthreads();  // (every thread's reads and writes are before its CTA's ticket)
  if (gridDim.x == 1u) {
    s_last = 1u;
  } else if (threadIdx.x == 0) {
    __threadfence();
    s_last = atomicAdd(reinterpret_cast<uint32_t*>(a.state) + 1, 1u) == gridDim.x - 1u;
    __threadfence();
  }
  __syncthreads();
  if (!s_last) return;
  if (ok)
    for (uint32_t s = threadIdx.x; s < a.n_seqs; s += kT) a.kv_lens[s] = __ldg(a.target + s);
  if (threadIdx.x == 0) {
    if (ok)
      a.state[0] = (int32_t)(n_free + (uint32_t)t.gone - (uint32_t)t.come);
    else
      set_status(a.status, IBP_ERANGE);
    a.state[1] = 0;
  }
}

// Pages that go, onto the list.
template <uint32_t kT>
__device__ __forceinline__ void give(const PagedTablesArgs& a, const Sums& t, uint32_t n_free,
                                     const Part& own) {
  __shared__ uint32_t s_warp[kT / 32], s_sum[kT], s_want[kT];
  const uint32_t R = (uint32_t)t.gone;
  const uint32_t r0 = (uint32_t)((uint64_t)R * blockIdx.x / gridDim.x);
  const uint32_t r1 = (uint32_t)((uint64_t)R * (blockIdx.x + 1u) / gridDim.x);
  uint32_t base = 0;
  for (uint32_t c = 0; c < a.n_seqs && base < r1; c += kT) {
    Part p = own;
    if (c) p = c + threadIdx.x < a.n_seqs ? part_of(a, c + threadIdx.x) : Part{};
    uint32_t all;
    const uint32_t before = scan<kT>(p.gone, s_warp, all);
    s_sum[threadIdx.x] = base + before;
    s_want[threadIdx.x] = p.want;
    __syncthreads();
    const uint32_t from = max(r0, base) + threadIdx.x;
    uint32_t i = last_at_most<kT>(s_sum, from);
#pragma unroll 4
    for (uint32_t r = from; r < min(r1, base + all); r += kT) {
      while (i + 1u < kT && s_sum[i + 1u] <= r) ++i;
      a.free_pages[n_free + R - 1u - r] =
          a.table[(uint64_t)(c + i) * a.table_stride + s_want[i] + (r - s_sum[i])];
    }
    base += all;
    __syncthreads();
  }
}

// Rows, pages and slots of the new tokens, from the list with the pages that went.
template <uint32_t kT>
__device__ __forceinline__ void take(const PagedTablesArgs& a, bool ok, const Sums& t,
                                     uint32_t n_free, const Part& own) {
  __shared__ uint32_t s_warp[kT / 32], s_row[kT], s_page[kT], s_old[kT];
  const uint32_t T = ok ? (uint32_t)t.rows : 0u;
  const uint32_t t0 = (uint32_t)((uint64_t)T * blockIdx.x / gridDim.x);
  const uint32_t t1 = (uint32_t)((uint64_t)T * (blockIdx.x + 1u) / gridDim.x);
  const uint32_t top = ok ? n_free + (uint32_t)t.gone - 1u : 0u;
  const uint32_t lg = a.page_lg, P = 1u << lg;
  uint32_t row = 0, page = 0;  // sums before the sequences from c on
  const bool starts = blockIdx.x == 0;
  for (uint32_t c = 0; c < a.n_seqs && (starts || row < t1); c += kT) {
    const uint32_t s = c + threadIdx.x;
    Part p = own;
    if (c) p = s < a.n_seqs ? part_of(a, s) : Part{};
    if (!ok) p = Part{};
    uint32_t rows, pages;
    const uint32_t before = scan<kT>(p.rows, s_warp, rows);
    const uint32_t first = scan<kT>(p.come, s_warp, pages);
    s_row[threadIdx.x] = row + before;
    s_page[threadIdx.x] = page + first - p.have;  // number of its page i that is new: this + i
    s_old[threadIdx.x] = p.old;
    if (starts && s < a.n_seqs) {
      a.q_starts[s] = (int32_t)(row + before);
      if (s + 1u == a.n_seqs) a.q_starts[s + 1u] = (int32_t)(row + before + p.rows);
    }
    __syncthreads();
    const uint32_t end = min(t1, row + rows);
    uint32_t x = max(t0, row) + threadIdx.x;
    uint32_t i = last_at_most<kT>(s_row, x);
    // the sequence in registers, until its last token
    uint32_t next = 0, shift = 0, have = 0, taken = 0;
    int32_t* entries = nullptr;
    auto enter = [&] {
      while (i + 1u < kT && s_row[i + 1u] <= x) ++i;
      next = i + 1u < kT ? s_row[i + 1u] : ~0u;
      shift = s_old[i] - s_row[i];
      have = (s_old[i] + P - 1u) >> lg;
      taken = top - s_page[i];
      entries = a.table + (uint64_t)(c + i) * a.table_stride;
    };
    for (; x < end; x += kLooks * kT) {
      // looked up together; a new page's first token writes its entry
      uint32_t in[kLooks];
      int32_t id[kLooks];
      int32_t* entry[kLooks];
      const uint32_t x0 = x;
#pragma unroll
      for (uint32_t u = 0; u < kLooks; ++u, x += kT) {
        entry[u] = nullptr;
        id[u] = 0;
        if (x >= end) break;
        if (x >= next) enter();
        const uint32_t pos = x + shift, at = pos >> lg;
        const bool fresh = at >= have;
        in[u] = pos & (P - 1u);
        id[u] = *(fresh ? a.free_pages + (taken - at) : entries + at);
        if (fresh && in[u] == 0u) entry[u] = entries + at;
      }
      x = x0;
#pragma unroll
      for (uint32_t u = 0; u < kLooks; ++u) {
        const uint32_t y = x0 + u * kT;
        if (y >= end) break;
        if (entry[u]) *entry[u] = id[u];
        if (a.slots) a.slots[y] = ((int64_t)id[u] << lg) + in[u];
      }
    }
    row += rows;
    page += pages;
    __syncthreads();
  }
}

// All there is to do when no sequence may grow; else the rest is k_paged_take's.
__global__ void __launch_bounds__(kThreads) k_paged_give(PagedTablesArgs a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  Sums t;
  Part own{};
  uint32_t n_free;
  const bool ok = total<kThreads>(a, t, n_free, own);
  if (ok && t.gone) give<kThreads>(a, t, n_free, own);
  if (!a.n_tokens) finish<kThreads>(a, ok, t, n_free);
}

__global__ void __launch_bounds__(kThreads) k_paged_take(PagedTablesArgs a) {
  Sums t;
  Part own{};
  uint32_t n_free;
  const bool ok = total<kThreads>(a, t, n_free, own);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  take<kThreads>(a, ok, t, n_free, own);
  finish<kThreads>(a, ok, t, n_free);
}

// One CTA: the list is written before it is read.
__global__ void __launch_bounds__(kThreads) k_paged_resize(PagedTablesArgs a) {
  Sums t;
  Part own{};
  uint32_t n_free;
  const bool ok = total<kThreads>(a, t, n_free, own);
  if (ok && t.gone) give<kThreads>(a, t, n_free, own);
  __syncthreads();
  if (a.n_tokens) take<kThreads>(a, ok, t, n_free, own);
  finish<kThreads>(a, ok, t, n_free);
}

}  // namespace

cudaError_t launch_paged_resize(const PagedTablesArgs& a, int sm_count, cudaStream_t st) {
  // One CTA and one launch, or two: 20 sequences of 124 pages, up to 5 tokens each, 6.5 us against
  // 7.5;
  // 250 sequences of 2048 pages, 1.33 million new tokens, need the two (14.3 us).
  const uint64_t entries = (uint64_t)a.n_seqs * a.max_pages;
  if (entries <= 16u * kThreads && a.n_tokens <= 4u * kThreads) {
    k_paged_resize<<<1, kThreads, 0, st>>>(a);
    return cudaGetLastError();
  }
  // Two loads to a thread, two CTAs to an SM at most: a look-up waits for the last, and each CTA
  // takes the sums again (250 sequences: 14.3 us; one 16.2, three 15.3, four 16.5, six 20.8).
  auto ctas = [&](uint64_t n) {
    const uint64_t c = (n + 2u * kThreads - 1) / (2u * kThreads), most = 2ull * sm_count;
    return (unsigned)(c < 1u ? 1u : c > most ? most : c);
  };
  k_paged_give<<<ctas(entries), kThreads, 0, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !a.n_tokens) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas(a.n_tokens), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_paged_take, a);
}

}  // namespace ibp
