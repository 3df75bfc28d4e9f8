// What the attention kernels of few rows share, over 16-bit pages and over 8-bit ones:
// the list of blocks of all sequences and heads, what the producer tells the computing
// warps of a run of it, rows of the result, and the join of tiles that were cut.
#pragma once

#include "ibp_paged.cuh"
#include "ibp_sm103.cuh"

#ifdef __CUDACC__

namespace ibp {
namespace {

constexpr uint32_t kBlock = 128, kWarpKeys = 32;
constexpr uint32_t kMaxCtas = 512;
// in the place of a box's first position: nothing to read, a page id out of range
constexpr uint32_t kNoPage = 0xFFFFFFFFu, kBadPage = 0xFFFFFFFEu;

// One piece of a cut (sequence, head): 16 rows of running maximum, sum, output.
template <int kDP>
struct Piece {
  float m[16], l[16];
  float o[16][kDP];
};

// What the joining kernel is told by a CTA that ended a cut tile.
struct Join {
  uint32_t first, count;  // CTAs that hold its pieces: first .. first + count - 1; 0: none
  uint32_t q0, head;      // first row of the sequence (or token), K/V head
  uint32_t row0, rows;    // the tile's rows
  uint64_t tile_u;        // (the first kernel's: where its blocks begin in the list)
};

// What the producer tells the others of a run of blocks of one tile; count 0: no
// more.  A ring of 8: the producer has at most kStages blocks (each of a tile of its own,
// at worst) before it and tells of one more, while the others still write a tile's rows.
struct Info {
  uint32_t count;         // blocks
  uint32_t q0, head;      // first row of the sequence (or the token), K/V head
  uint32_t row0, rows;    // the tile's rows among the sequence's n * G
  uint32_t n, L, lo;      // tokens, keys, first key that a row sees
  uint32_t key0;          // first key of the run (without a page list)
  uint32_t whole, place;  // the run is the whole tile; else which of the CTA's pieces
  uint32_t pad;
};
constexpr uint32_t kInfos = 8;

// A tile: 16 rows of one (sequence, head), or of one (token, head) with a page
// list, and its blocks of keys.  Row r is query r % G of token r / G.
struct Tile {
  uint32_t s, head, rb;   // sequence (or token), K/V head, block of 16 rows
  uint32_t nrb;           // blocks of 16 rows of the sequence (or token)
  uint32_t q0, n, L;      // first row, tokens, keys
  uint32_t b0, nb;        // first block of keys, number of blocks (at least 1)
  uint32_t lo;            // first key that a row may see
  const int32_t* table;
  const int32_t* sel;
};

// Blocks of keys of a sequence's tiles; 0 when it has no row here.
__device__ __forceinline__ uint32_t seq_blocks(const PagedAttnArgs& a, const PagedSeq& q,
                                               uint32_t& b0, uint32_t& lo, uint32_t& nrb) {
  lo = 0;
  b0 = 0;
  nrb = (q.n * a.G + 15u) / 16u;
  if (q.n == 0 || q.n * a.G > a.max_rows) return 0;
  const uint32_t first = q.L >= q.n ? q.L - q.n : 0u;
  if (a.window && first + 1u > a.window) lo = first + 1u - a.window;
  b0 = lo / kBlock;
  const uint32_t b1 = (q.L + kBlock - 1u) / kBlock;
  return b1 > b0 ? b1 - b0 : 1u;
}

__device__ __forceinline__ uint32_t list_blocks(const PagedAttnArgs& a) {
  return max(1u, ((a.n_sel << a.g.page_lg) + kBlock - 1u) / kBlock);
}

// Fills in what follows from t.s and t.head.
template <bool kSel>
__device__ __forceinline__ void tile_of(const PagedAttnArgs& a, Tile& t) {
  if (kSel) {
    const uint32_t tok = t.s;
    const uint32_t s = paged_find(a.b, tok);
    PagedSeq q{0, 0, 0, false};
    if (s < a.b.n_seqs) {
      q = paged_seq(a.b, a.g.page_lg, s);
      if (!q.ok) set_status(a.g.status, IBP_ERANGE);
    }
    const int64_t pos = (int64_t)q.L - q.n + (tok - q.q0);
    t.q0 = tok;
    t.n = s < a.b.n_seqs ? 1u : 0u;  // a row of no sequence is left alone
    t.L = !q.ok || pos < 0 ? 0u : (uint32_t)pos + 1u;  // keys up to its own
    t.lo = 0;
    t.b0 = 0;
    t.nrb = (a.G + 15u) / 16u;
    t.nb = list_blocks(a);
    t.table = a.b.table + (s < a.b.n_seqs ? s : 0u) * a.b.table_stride;
    t.sel = a.selected + ((uint64_t)tok * a.g.H + t.head) * a.n_sel;
  } else {
    const PagedSeq q = paged_seq(a.b, a.g.page_lg, t.s);
    t.q0 = q.q0;
    t.n = q.n;
    t.L = q.L;
    t.nb = seq_blocks(a, q, t.b0, t.lo, t.nrb);
    t.table = a.b.table + t.s * a.b.table_stride;
    t.sel = nullptr;
  }
}

// Walks the list of blocks: which tile, which block of it.
struct Cursor {
  Tile t;
  uint32_t blk;  // block within the tile
};

template <bool kSel>
__device__ __forceinline__ void next_tile(const PagedAttnArgs& a, Cursor& c) {
  c.blk = 0;
  if (++c.t.rb < c.t.nrb) return;
  c.t.rb = 0;
  if (++c.t.head < a.g.H) {
    if (kSel) tile_of<kSel>(a, c.t);
    return;
  }
  c.t.head = 0;
  const uint32_t end = kSel ? a.b.n_tokens : a.b.n_seqs;
  do {
    if (++c.t.s >= end) return;
    tile_of<kSel>(a, c.t);
  } while (c.t.nb == 0);
}

// The list of blocks: its length, and this CTA's run [u0, u1) of it.
struct Run {
  Cursor ld;
  uint64_t u0, u1, total;
  uint64_t tile_u;  // position in the list of the current tile's first block
  uint32_t ctas;    // CTAs with a run: never more than blocks
};

// Where CTA b's run begins: total * b / ctas (b <= ctas <= kMaxCtas), by a division of 32 bits
// where the list is that short, as the quotients below are: one of 64 takes 0.2 us.
__device__ __forceinline__ uint64_t run_start(uint64_t total, uint32_t b, uint32_t ctas) {
  if (total >> 32) return total * b / ctas;
  const uint32_t n = (uint32_t)total, q = n / ctas;
  return (uint64_t)q * b + (n - q * ctas) * b / ctas;
}
__device__ __forceinline__ uint64_t quotient(uint64_t x, uint32_t d) {
  return x >> 32 ? x / d : (uint32_t)x / d;
}

template <bool kSel, uint32_t kThreads>
__device__ __forceinline__ Run step_run(const PagedAttnArgs& a,
                                        uint64_t (&s_scan)[kThreads / 32],
                                        uint64_t (&s_found)[2]) {
  const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31u, tid = threadIdx.x;
  Run r;
  Cursor& ld = r.ld;
  uint64_t u0 = 0, u1 = 0;
  uint32_t ctas = gridDim.x;
  uint64_t tile_u = 0;
  uint64_t total = 0;
  if (kSel) {
    const uint32_t nb = list_blocks(a), nrb = (a.G + 15u) / 16u;
    total = (uint64_t)a.b.n_tokens * a.g.H * nrb * nb;
    if (total < ctas) ctas = (uint32_t)total;
    if (blockIdx.x < ctas) {
      u0 = run_start(total, blockIdx.x, ctas);
      u1 = run_start(total, blockIdx.x + 1u, ctas);
      const uint64_t ti = quotient(u0, nb), th = quotient(ti, nrb), ts = quotient(th, a.g.H);
      ld.t.rb = (uint32_t)(ti - th * nrb);
      ld.t.head = (uint32_t)(th - ts * a.g.H);
      ld.t.s = (uint32_t)ts;
      ld.blk = (uint32_t)(u0 - ti * nb);
      tile_u = ti * nb;
      tile_of<kSel>(a, ld.t);
    }
    __syncthreads();
  } else {
    uint32_t b0, lo, nrb;
    uint64_t mine = 0, own = 0;  // own: of sequence tid
    for (uint32_t s = tid; s < a.b.n_seqs; s += kThreads) {
      const PagedSeq q = paged_seq(a.b, a.g.page_lg, s);
      if (!q.ok) set_status(a.g.status, IBP_ERANGE);
      const uint32_t n = seq_blocks(a, q, b0, lo, nrb);
      mine += (uint64_t)n * nrb;
      if (s == tid) own = mine;
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) mine += __shfl_xor_sync(0xFFFFFFFFu, mine, d);
    if (lane == 0) s_scan[warp] = mine;
    __syncthreads();
    for (uint32_t w = 0; w < kThreads / 32; ++w) total += s_scan[w];
    total *= a.g.H;
    if (total < ctas) ctas = (uint32_t)total;
    if (blockIdx.x < ctas) {
      u0 = run_start(total, blockIdx.x, ctas);
      u1 = run_start(total, blockIdx.x + 1u, ctas);
    }
    // the sequence that holds block u0: sums over as many sequences as threads at a time
    uint64_t base = 0;
    for (uint32_t c = 0; c < a.b.n_seqs && u0 < u1; c += kThreads) {
      uint64_t nb = own;
      if (c && c + tid < a.b.n_seqs) {
        nb = seq_blocks(a, paged_seq(a.b, a.g.page_lg, c + tid), b0, lo, nrb);
        nb *= nrb;
      } else if (c) {
        nb = 0;
      }
      uint64_t inc = nb;
#pragma unroll
      for (uint32_t d = 1; d < 32u; d <<= 1) {
        const uint64_t v = __shfl_up_sync(0xFFFFFFFFu, inc, d);
        if (lane >= d) inc += v;
      }
      __syncthreads();
      if (lane == 31u) s_scan[warp] = inc;
      __syncthreads();
      uint64_t before = 0, all = 0;
      for (uint32_t w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += s_scan[w];
        all += s_scan[w];
      }
      const uint64_t lo_u = base + (before + inc - nb) * a.g.H;
      if (u0 >= lo_u && u0 < lo_u + nb * a.g.H) {
        s_found[0] = c + tid;
        s_found[1] = lo_u;
      }
      base += all * a.g.H;
      if (u0 < base) break;
    }
    __syncthreads();
    if (u0 < u1) {
      ld.t.s = (uint32_t)s_found[0];
      ld.t.head = 0;
      tile_of<kSel>(a, ld.t);
      const uint64_t in = u0 - s_found[1], ti = quotient(in, ld.t.nb);
      const uint64_t th = quotient(ti, ld.t.nrb);
      ld.t.rb = (uint32_t)(ti - th * ld.t.nrb);
      ld.t.head = (uint32_t)th;
      ld.blk = (uint32_t)(in - ti * ld.t.nb);
      tile_u = u0 - ld.blk;
    }
  }
  r.u0 = u0, r.u1 = u1, r.total = total, r.tile_u = tile_u, r.ctas = ctas;
  return r;
}

// The producer's run of blocks of its current tile, from u on: their number (0 when there
// are no more), told to the others, and the join that this CTA asks for when it has
// the last piece of a tile that was cut.
__device__ __forceinline__ uint32_t tell_tile(const PagedAttnArgs& a, const Run& r, uint64_t u,
                                              bool more, Info* x, uint64_t* bar, Join& join) {
  const uint32_t lane = threadIdx.x & 31u;
  const uint32_t count = !more ? 0u
                         : r.u1 - u < r.ld.t.nb - r.ld.blk ? (uint32_t)(r.u1 - u)
                                                     : r.ld.t.nb - r.ld.blk;
  const bool ends = r.ld.blk + count == r.ld.t.nb;
  const bool whole = r.ld.blk == 0 && ends;
  if (lane == 0) {
    x->count = count;
    x->q0 = r.ld.t.q0;
    x->head = r.ld.t.head;
    x->row0 = r.ld.t.rb * 16u;
    x->rows = r.ld.t.n ? min(16u, r.ld.t.n * a.G - r.ld.t.rb * 16u) : 0u;
    x->n = r.ld.t.n;
    x->L = r.ld.t.L;
    x->lo = r.ld.t.lo;
    x->key0 = (r.ld.t.b0 + r.ld.blk) * kBlock;
    x->whole = whole;
    x->place = r.tile_u >= r.u0 ? 1u : 0u;
    mbar_arrive(bar);
    if (more && ends && !whole) {  // this CTA has the tile's last piece (end_join: its first)
      join.count = 1;
      join.tile_u = r.tile_u;
      join.q0 = r.ld.t.q0;
      join.rows = x->rows;
      join.row0 = x->row0;
      join.head = r.ld.t.head;
    }
  }
  return count;
}

// The CTA that holds the first block of the tile to be joined: found when the loads are on
// their way, not before the first.
__device__ __forceinline__ void end_join(const Run& r, Join& join) {
  if (join.count == 0) return;
  const uint64_t u = join.tile_u;
  uint32_t f = (uint32_t)(u * r.ctas / r.total);
  while (f + 1u < r.ctas && run_start(r.total, f + 1u, r.ctas) <= u) ++f;
  while (f > 0 && run_start(r.total, f, r.ctas) > u) --f;
  join.first = f;
  join.count = blockIdx.x - f + 1u;
}

// A barrier of the kCount warps that compute, and whether any of their threads says so.
template <uint32_t kCount>
__device__ __forceinline__ bool any_of(bool mine) {
  uint32_t any;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n"
      " barrier.cta.red.or.pred q, 1, %2, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(any)
      : "r"((uint32_t)mine), "n"(32u * kCount)
      : "memory");
  return any != 0u;
}

// One row of the result, by a warp: lane i holds channels i, i + 32, ...  A row
// that saw no key (its sum is 0) and one that could not be read are zero.
// kLift: the weights, and with them the sum and the outputs, are 2^kLift times the formula's.
template <int kDP, bool kBf16, int kLift>
__device__ __forceinline__ void store_row(const PagedAttnArgs& a, uint64_t at, uint32_t lane,
                                          const float (&o)[kDP / 32], float m, float l, bool bad) {
  const bool some = !bad && l != 0.f;
  const float inv = some ? 1.f / l : 0.f;
  uint16_t* dst = reinterpret_cast<uint16_t*>(a.out) + at * a.g.D;
#pragma unroll
  for (int i = 0; i < kDP / 32; ++i)
    if (lane + 32u * i < a.g.D)
      dst[lane + 32u * i] = (uint16_t)pack2(some ? o[i] * inv : 0.f, 0.f, kBf16);
  if (a.lse && lane == 0)
    a.lse[at] = some ? (m - (float)kLift + log2f(l)) * 0.69314718056f : -INFINITY;
}

// The kCount warps' rows of a tile (or of this CTA's run of it), joined: the result, or a
// piece of it.  A warp's rows lie in `merge`: outputs, then maximum, sum and whether it
// could not be read.
template <int kDP, bool kBf16, int kLift, uint32_t kCount>
__device__ __forceinline__ void merge_rows(const PagedAttnArgs& a, const Info* t, uint32_t rows,
                                           const float* merge, Piece<kDP>* pieces) {
  const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31u;
  Piece<kDP>* piece = pieces + 2u * blockIdx.x + t->place;
  for (uint32_t r = warp; r < rows; r += kCount) {
    float mm[kCount], mx = -INFINITY, ll = 0.f, ov[kDP / 32];
    bool isbad = false;
#pragma unroll
    for (uint32_t w = 0; w < kCount; ++w) {
      mm[w] = merge[(w * 16u + r) * (kDP + 4u) + kDP];
      mx = fmaxf(mx, mm[w]);
      isbad = isbad || merge[(w * 16u + r) * (kDP + 4u) + kDP + 2u] != 0.f;
    }
    const float base = mx == -INFINITY ? 0.f : mx;
#pragma unroll
    for (int i = 0; i < kDP / 32; ++i) ov[i] = 0.f;
#pragma unroll
    for (uint32_t w = 0; w < kCount; ++w) {
      const float* src = merge + (w * 16u + r) * (kDP + 4u);
      const float f = ex2(mm[w] - base);
      ll += f * src[kDP + 1];
#pragma unroll
      for (int i = 0; i < kDP / 32; ++i) ov[i] = fmaf(f, src[lane + 32u * i], ov[i]);
    }
    if (isbad) ll = INFINITY;  // a row that could not be read: zero, here or when joined
    if (t->whole) {
      const uint32_t R = t->row0 + r;
      const uint64_t at = ((uint64_t)(t->q0 + R / a.G) * a.g.H + t->head) * a.G + R % a.G;
      store_row<kDP, kBf16, kLift>(a, at, lane, ov, mx, ll, isbad);
    } else {
#pragma unroll
      for (int i = 0; i < kDP / 32; ++i) piece->o[r][lane + 32u * i] = ov[i];
      if (lane == 0) piece->m[r] = mx, piece->l[r] = ll;
    }
  }
}

// Joins the pieces of the tile that CTA blockIdx.x of the first kernel ended, a
// warp per row.
template <int kDP, bool kBf16, int kLift>
__global__ void __launch_bounds__(128) k_paged_step_join(PagedAttnArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // from here the chunk kernel's join may run beside this one
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Join* joins =
      reinterpret_cast<const Join*>(a.ws + kStepWsBytes - kMaxCtas * sizeof(Join));
  const Piece<kDP>* pieces = reinterpret_cast<const Piece<kDP>*>(a.ws);
  const uint4 j0 = __ldcg(reinterpret_cast<const uint4*>(joins + blockIdx.x));
  const uint4 j1 = __ldcg(reinterpret_cast<const uint4*>(joins + blockIdx.x) + 1);
  const uint32_t first = j0.x, count = j0.y, q0 = j0.z, head = j0.w, row0 = j1.x, rows = j1.y;
  const uint32_t lane = threadIdx.x & 31u;
  const uint32_t r = blockIdx.y * 4u + (threadIdx.x >> 5);
  if (count == 0 || r >= rows) return;
  // the first piece lies in its CTA's second place (the tile began there)
  auto at_piece = [&](uint32_t i) { return pieces + 2u * (first + i) + (i == 0u ? 1u : 0u); };
  // the first pieces' numbers, all on their way at once (a tile seldom has more)
  constexpr uint32_t kFirst = 4;
  float pm[kFirst], pl[kFirst], po[kFirst][kDP / 32], mx = -INFINITY;
#pragma unroll
  for (uint32_t i = 0; i < kFirst; ++i) {
    pm[i] = -INFINITY;
    if (i < count) {
      const Piece<kDP>* p = at_piece(i);
      pm[i] = __ldcg(&p->m[r]);
      pl[i] = __ldcg(&p->l[r]);
#pragma unroll
      for (int x = 0; x < kDP / 32; ++x) po[i][x] = __ldcg(&p->o[r][lane + 32u * x]);
    }
  }
  for (uint32_t i = kFirst + lane; i < count; i += 32u)
    mx = fmaxf(mx, __ldcg(&at_piece(i)->m[r]));
  if (count > kFirst)
#pragma unroll
    for (int d = 16; d; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, d));
#pragma unroll
  for (uint32_t i = 0; i < kFirst; ++i) mx = fmaxf(mx, pm[i]);
  const float base = mx == -INFINITY ? 0.f : mx;
  float ll = 0.f, ov[kDP / 32];
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kDP / 32; ++i) ov[i] = 0.f;
#pragma unroll
  for (uint32_t i = 0; i < kFirst; ++i)
    if (i < count) {
      const float f = ex2(pm[i] - base);
      bad = bad || pl[i] == INFINITY;
      ll += f * pl[i];
#pragma unroll
      for (int x = 0; x < kDP / 32; ++x) ov[x] = fmaf(f, po[i][x], ov[x]);
    }
#pragma unroll 4
  for (uint32_t i = kFirst; i < count; ++i) {
    const Piece<kDP>* p = at_piece(i);
    const float li = __ldcg(&p->l[r]);
    const float f = ex2(__ldcg(&p->m[r]) - base);
    bad = bad || li == INFINITY;
    ll += f * li;
#pragma unroll
    for (int x = 0; x < kDP / 32; ++x) ov[x] = fmaf(f, __ldcg(&p->o[r][lane + 32u * x]), ov[x]);
  }
  const uint64_t at = ((uint64_t)(q0 + (row0 + r) / a.G) * a.g.H + head) * a.G + (row0 + r) % a.G;
  store_row<kDP, kBf16, kLift>(a, at, lane, ov, mx, ll, bad);
}

// The join behind a step kernel of the same grid, which it waits for by itself.
template <int kDP, bool kBf16, int kLift>
cudaError_t launch_step_join(const PagedAttnArgs& a, uint32_t ctas, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, 4, 1);
  cfg.blockDim = dim3(128, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_paged_step_join<kDP, kBf16, kLift>, a);
}

static_assert(2u * kMaxCtas * sizeof(Piece<128>) + kMaxCtas * sizeof(Join) <= kStepWsBytes,
              "pieces and joins fit their part of the workspace");

}  // namespace
}  // namespace ibp

#endif
