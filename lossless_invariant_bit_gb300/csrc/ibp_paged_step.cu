// Attention of few rows over a paged K/V cache: the step of sequences that are
// being answered (one new token each, or a few), and tokens that attend to a
// list of pages each.
//
//   out = sum_j p_j v_j / sum_j p_j,   p_j = exp(scale q.k_j - m),  m = max_j
//
// in one pass over the keys, the running maximum and sum kept in fp32 and the
// output rescaled when the maximum grows.  Bound by HBM: every key and value is
// read once for at most 16 rows (the queries that share a K/V head, times the
// new tokens), 4 D rows operations against 4 D bytes.
//
//   - The work of all sequences and heads is one list of blocks of 128 keys;
//     each CTA takes an equal run of it (one CTA per SM), whatever the
//     lengths.  A (sequence, head) whose run is cut is joined by a second kernel
//     from the pieces' maxima, sums and unscaled outputs, in the order of the
//     pieces, so that results do not depend on timing.
//   - Each of the 4 warps takes 32 keys of a block, with a ring of stages in
//     shared memory of its own that it fills by TMA (a box per page) and waits
//     for by mbarrier: no barrier of the CTA within a run.
//   - 16 rows are one left operand of mma.sync m16n8k16: at 16 rows the keys'
//     bytes, not the products, are the bound, and a 128-row tcgen05 tile would be
//     7/8 padding (the chunk kernel takes what has more rows).
#include "ibp_paged.cuh"
#include "ibp_sm103.cuh"
#include "ibp_tma.cuh"

namespace ibp {
namespace {

constexpr uint32_t kWarps = 4, kBlock = 128, kWarpKeys = 32;
// page references of a stage beside page numbers: nothing to read, an id out of range
constexpr uint32_t kNoPage = 0xFFFFFFFFu, kBadPage = 0xFFFFFFFEu;
constexpr uint32_t kMaxCtas = 512;

// One piece of a cut (sequence, head): 16 rows of running maximum, sum, output.
template <int kDP>
struct Piece {
  float m[16], l[16];
  float o[16][kDP];
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// What the joining kernel is told by a CTA that ended a cut tile.
struct Join {
  uint32_t first, count;  // CTAs that hold its pieces: first .. first + count - 1; 0: none
  uint32_t q0, head;      // first row of the sequence (or token), K/V head
  uint32_t row0, rows;    // the tile's rows
  uint32_t pad[2];
};

template <int kDP>
struct StepShape {
  static constexpr uint32_t kHalves = kDP / 64;
  static constexpr uint32_t kHalfBytes = kWarpKeys * 128u;
  static constexpr uint32_t kTile = kHalves * kHalfBytes;      // keys (or values) of a stage
  static constexpr uint32_t kStages = kDP == 64 ? 2u : 3u;
  static constexpr uint32_t kRing = kStages * 2u * kTile;      // per warp
  static constexpr uint32_t kMerge = kWarps * 16u * (kDP + 4u) * 4u;
  static constexpr uint32_t kSmem = 1024u + kWarps * kRing + kMerge + 256u;
};

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

// What this lane loads of a warp's 32 keys of a block: one box, a page or 32 tokens of one.
struct PageRef {
  int32_t id;      // the page to read; -1: none
  uint32_t token;  // first token within it
  uint32_t ref;    // number among the sequence's pages << 9 | token, or kNoPage, kBadPage
};

template <bool kSel>
__device__ __forceinline__ PageRef page_of(const PagedAttnArgs& a, const Cursor& c, uint32_t warp,
                                           uint32_t lane) {
  const uint32_t lg = a.g.page_lg;
  const uint32_t box = lg < 5u ? 1u << lg : 32u;
  const uint32_t key = (c.t.b0 + c.blk) * kBlock + warp * kWarpKeys + lane * box;
  PageRef r{-1, key & ((1u << lg) - 1u), kNoPage};
  if (lane * box >= kWarpKeys) return r;
  uint32_t col = key >> lg;
  if (kSel) {
    if (col >= a.n_sel) return r;
    const int32_t v = __ldg(c.t.sel + col);
    if (v < 0 || c.t.L == 0 || (uint32_t)v > (c.t.L - 1u) >> lg) return r;
    col = (uint32_t)v;
    if ((col << lg) + r.token >= c.t.L) return r;
  } else if (key >= c.t.L || key + box <= c.t.lo) {
    return r;
  }
  const int32_t id = __ldg(c.t.table + col);
  if (id < 0 || (uint32_t)id >= a.g.n_pages) {
    r.ref = kBadPage;
    return r;
  }
  r.id = id;
  r.ref = col << 9 | r.token;
  return r;
}

__device__ __forceinline__ void tma_load_page(void* dst, const CUtensorMap* map, uint64_t* bar,
                                              uint32_t x, uint32_t token, uint32_t head,
                                              int32_t page) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_addr(bar)), "r"(x), "r"(token), "r"(head),
      "r"(page)
      : "memory");
}

// One row of the result, by a warp: lane i holds channels i, i + 32, ...  A row
// that saw no key (its sum is 0) and one that could not be read are zero.
template <int kDP, bool kBf16>
__device__ __forceinline__ void store_row(const PagedAttnArgs& a, uint64_t at, uint32_t lane,
                                          const float (&o)[kDP / 32], float m, float l, bool bad) {
  const bool some = !bad && l != 0.f;
  const float inv = some ? 1.f / l : 0.f;
  uint16_t* dst = reinterpret_cast<uint16_t*>(a.out) + at * a.g.D;
#pragma unroll
  for (int i = 0; i < kDP / 32; ++i)
    if (lane + 32u * i < a.g.D)
      dst[lane + 32u * i] = (uint16_t)pack2(some ? o[i] * inv : 0.f, 0.f, kBf16);
  if (a.lse && lane == 0) a.lse[at] = some ? (m + log2f(l)) * 0.69314718056f : -INFINITY;
}

template <int kDP, bool kBf16, bool kSel>
__global__ void __launch_bounds__(128, kDP == 64 ? 2 : 1)
    k_paged_step(const __grid_constant__ CUtensorMap map_k,
                 const __grid_constant__ CUtensorMap map_v, PagedAttnArgs a) {
  using S = StepShape<kDP>;
  constexpr int kKs = kDP / 16;  // k-steps of a score, n-tile pairs of an output
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023u) & ~static_cast<uintptr_t>(1023u));
  __shared__ uint64_t s_scan[8];
  __shared__ uint64_t s_found[2];
  __shared__ uint32_t s_ref[kWarps][S::kStages][4];  // the pages of each stage
  const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31u, tid = threadIdx.x;
  uint8_t* ring = smem + warp * S::kRing;
  float* merge = reinterpret_cast<float*>(smem + kWarps * S::kRing);
  uint64_t* full =
      reinterpret_cast<uint64_t*>(smem + kWarps * S::kRing + S::kMerge) + warp * S::kStages;
  Piece<kDP>* pieces = reinterpret_cast<Piece<kDP>*>(a.ws);
  Join* joins = reinterpret_cast<Join*>(a.ws + kStepWsBytes - kMaxCtas * sizeof(Join));

  if (lane == 0) {
    for (uint32_t i = 0; i < S::kStages; ++i) mbar_init(full + i, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  // ---- the list of blocks: its length, and this CTA's run [u0, u1) of it
  Cursor ld;
  uint64_t u0 = 0, u1 = 0;
  uint32_t ctas = gridDim.x;  // CTAs with a run: never more than blocks
  uint64_t tile_u = 0;  // position in the list of the current tile's first block
  uint64_t total = 0;
  if (kSel) {
    const uint32_t nb = list_blocks(a), nrb = (a.G + 15u) / 16u;
    total = (uint64_t)a.b.n_tokens * a.g.H * nrb * nb;
    if (total < ctas) ctas = (uint32_t)total;
    if (blockIdx.x < ctas) {
      u0 = total * blockIdx.x / ctas;
      u1 = total * (blockIdx.x + 1u) / ctas;
      const uint64_t ti = u0 / nb;
      ld.t.rb = (uint32_t)(ti % nrb);
      ld.t.head = (uint32_t)(ti / nrb % a.g.H);
      ld.t.s = (uint32_t)(ti / nrb / a.g.H);
      ld.blk = (uint32_t)(u0 - ti * nb);
      tile_u = ti * nb;
      tile_of<kSel>(a, ld.t);
    }
    __syncthreads();
  } else {
    uint32_t b0, lo, nrb;
    uint64_t mine = 0;
    for (uint32_t s = tid; s < a.b.n_seqs; s += 128u) {
      const PagedSeq q = paged_seq(a.b, a.g.page_lg, s);
      if (!q.ok) set_status(a.g.status, IBP_ERANGE);
      mine += (uint64_t)seq_blocks(a, q, b0, lo, nrb) * nrb;
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) mine += __shfl_xor_sync(0xFFFFFFFFu, mine, d);
    if (lane == 0) s_scan[warp] = mine;
    __syncthreads();
    for (uint32_t w = 0; w < kWarps; ++w) total += s_scan[w];
    total *= a.g.H;
    if (total < ctas) ctas = (uint32_t)total;
    if (blockIdx.x < ctas) {
      u0 = total * blockIdx.x / ctas;
      u1 = total * (blockIdx.x + 1u) / ctas;
    }
    // the sequence that holds block u0: sums over 128 sequences at a time
    uint64_t base = 0;
    for (uint32_t c = 0; c < a.b.n_seqs && u0 < u1; c += 128u) {
      uint64_t nb = 0;
      if (c + tid < a.b.n_seqs) {
        nb = seq_blocks(a, paged_seq(a.b, a.g.page_lg, c + tid), b0, lo, nrb);
        nb *= nrb;
      }
      uint64_t inc = nb;
#pragma unroll
      for (uint32_t d = 1; d < 32u; d <<= 1) {
        const uint64_t v = __shfl_up_sync(0xFFFFFFFFu, inc, d);
        if (lane >= d) inc += v;
      }
      __syncthreads();
      if (lane == 31u) s_scan[4 + warp] = inc;
      __syncthreads();
      uint64_t before = 0, all = 0;
      for (uint32_t w = 0; w < kWarps; ++w) {
        if (w < warp) before += s_scan[4 + w];
        all += s_scan[4 + w];
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
      const uint64_t in = u0 - s_found[1], ti = in / ld.t.nb;
      ld.t.rb = (uint32_t)(ti % ld.t.nrb);
      ld.t.head = (uint32_t)(ti / ld.t.nrb);
      ld.blk = (uint32_t)(in - ti * ld.t.nb);
      tile_u = u0 - ld.blk;
    }
  }
  Join join{};
  if (u0 < u1) {
    Cursor c = ld;  // the block being worked on; `ld` runs ahead with the loads
    uint64_t u_ld = u0;
    // fill stage i with the block under `ld`
    auto issue = [&](uint32_t st) {
      const PageRef r = page_of<kSel>(a, ld, warp, lane);
      const uint32_t box = a.g.page_lg < 5u ? 1u << a.g.page_lg : 32u;
      const uint32_t bytes = r.id >= 0 ? 2u * S::kHalves * box * 128u : 0u;
      const uint32_t all = __reduce_add_sync(0xFFFFFFFFu, bytes);
      if (lane < 4u) s_ref[warp][st][lane] = r.ref;
      if (lane == 0) mbar_expect_tx(full + st, all);
      __syncwarp();
      if (r.id >= 0) {
        uint8_t* k = ring + st * 2u * S::kTile + lane * box * 128u;
#pragma unroll
        for (uint32_t hf = 0; hf < S::kHalves; ++hf) {
          tma_load_page(k + hf * S::kHalfBytes, &map_k, full + st, 64u * hf, r.token, ld.t.head,
                        r.id);
          tma_load_page(k + S::kTile + hf * S::kHalfBytes, &map_v, full + st, 64u * hf, r.token,
                        ld.t.head, r.id);
        }
      }
      ++u_ld;
      if (++ld.blk == ld.t.nb && u_ld < u1) next_tile<kSel>(a, ld);
    };
#pragma unroll
    for (uint32_t i = 0; i < S::kStages; ++i)
      if (u_ld < u1) issue(i);

    uint32_t st = 0, ph = 0, lost_st = 0, lost_ph = 0;
    uint32_t qf[kKs][4];
    float o[2 * kKs][4];
    float m[2], l[2];
    bool fresh = true, lost = false, bad = false;
    const uint32_t r0 = lane >> 2, quad = lane & 3u;
    for (uint64_t u = u0; u < u1; ++u) {
      const uint32_t rows = c.t.n ? min(16u, c.t.n * a.G - c.t.rb * 16u) : 0u;
      if (fresh) {  // a new tile: its queries, as the left operand
        fresh = false;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t r = r0 + 8u * e;
          const uint32_t tt = (c.t.rb * 16u + r) / a.G, gg = (c.t.rb * 16u + r) % a.G;
          const uint8_t* src = a.q + (uint64_t)(c.t.q0 + tt) * a.q_stride +
                               ((uint64_t)c.t.head * a.G + gg) * a.g.D * 2u;
#pragma unroll
          for (int k = 0; k < kKs; ++k)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const uint32_t d = 16u * k + 8u * x + 2u * quad;
              qf[k][e + 2 * x] = r < rows && d < a.g.D
                                     ? __ldg(reinterpret_cast<const uint32_t*>(src + d * 2u))
                                     : 0u;
            }
        }
#pragma unroll
        for (int i = 0; i < 2 * kKs; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;
      }
      // ---- this warp's 32 keys
      const uint32_t key0 = (c.t.b0 + c.blk) * kBlock + warp * kWarpKeys;
      if (!lost && !mbar_wait(full + st, ph)) lost = bad = true, lost_st = st, lost_ph = ph;
      const uint32_t kb = smem_addr(ring + st * 2u * S::kTile), vb = kb + S::kTile;
      // which of the 32 keys exist: a bit each
      uint32_t there;
      {
        const uint32_t lg = a.g.page_lg, box_lg = lg < 5u ? lg : 5u;
        const uint32_t ref = s_ref[warp][st][lane >> box_lg];
        if (ref == kBadPage) {
          set_status(a.g.status, IBP_ERANGE);
          bad = true;
        }
        const uint32_t key = kSel ? ((ref >> 9) << lg) + (ref & 511u) + (lane & ((1u << box_lg) - 1u))
                                  : key0 + lane;
        there = __ballot_sync(0xFFFFFFFFu, ref < kBadPage && key < c.t.L && key >= c.t.lo && !lost);
      }
      if (there) {
        if (there != 0xFFFFFFFFu) {
          // rows of values that do not exist: zero, so that 0 * (what they hold) is 0
          for (uint32_t i = lane; i < kWarpKeys * S::kHalves * 8u; i += 32u) {
            const uint32_t row = i / 8u % kWarpKeys;
            if (!(there >> row & 1u)) {
              const uint32_t off = (i / (8u * kWarpKeys)) * S::kHalfBytes + row * 128u + i % 8u * 16u;
              asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(vb + off), "r"(0u)
                           : "memory");
            }
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
        }
        float sc[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[i][0] = sc[i][1] = sc[i][2] = sc[i][3] = 0.f;
#pragma unroll
        for (int k = 0; k < kKs; ++k) {
          // keys 8i..8i+7 x channels 16k..16k+15, two tiles of keys per load
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t b[4];
            const uint32_t row = 16u * i + (lane & 7u) + ((lane >> 4) << 3);
            const uint32_t ch = 2u * (k & 3) + ((lane >> 3) & 1u);
            ldmatrix4(b, kb + (k >> 2) * S::kHalfBytes + row * 128u + ((ch ^ (row & 7u)) << 4));
            mma_16816<kBf16>(sc[2 * i], qf[k], b[0], b[1]);
            mma_16816<kBf16>(sc[2 * i + 1], qf[k], b[2], b[3]);
          }
        }
        // ---- masks: what does not exist, and what lies beyond a row's position
        const bool partial =
            there != 0xFFFFFFFFu ||
            (!kSel && c.t.n > 1u &&
             (key0 + kWarpKeys + c.t.n > c.t.L + 1u || a.window));
        if (partial) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t tt = (c.t.rb * 16u + r0 + 8u * e) / a.G;
            const int64_t pos = kSel ? 0x7FFFFFFF : (int64_t)c.t.L - c.t.n + tt;
            const int64_t from = a.window ? pos - a.window : -1;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const uint32_t j = 8u * i + 2u * quad + x;
                const int64_t key = (int64_t)key0 + j;
                const bool see = (there >> j & 1u) &&
                                 (kSel || ((!a.causal || key <= pos) && key > from));
                if (!see) sc[i][2 * e + x] = -INFINITY;
              }
          }
        }
        // ---- running maximum and sum; weights as the left operand of the values
        uint32_t pf[2][4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float mx = sc[0][2 * e];
#pragma unroll
          for (int i = 0; i < 4; ++i) mx = fmaxf(mx, fmaxf(sc[i][2 * e], sc[i][2 * e + 1]));
          mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
          mx = fmaxf(m[e], mx * a.scale_log2);
          const float base = mx == -INFINITY ? 0.f : mx;
          const float f = ex2(m[e] - base);
          m[e] = mx;
          float sum = 0.f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float p0 = ex2(fmaf(sc[i][2 * e], a.scale_log2, -base));
            const float p1 = ex2(fmaf(sc[i][2 * e + 1], a.scale_log2, -base));
            sum += p0 + p1;
            pf[i >> 1][e + 2 * (i & 1)] = pack2(p0, p1, kBf16);
          }
          l[e] = l[e] * f + sum;
#pragma unroll
          for (int i = 0; i < 2 * kKs; ++i) {
            o[i][2 * e] *= f;
            o[i][2 * e + 1] *= f;
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)  // 16 keys at a time
#pragma unroll
          for (int k = 0; k < kKs; ++k) {
            uint32_t b[4];
            const uint32_t row = 16u * i + (lane & 15u);
            const uint32_t ch = 2u * (k & 3) + (lane >> 4);
            ldmatrix4_t(b, vb + (k >> 2) * S::kHalfBytes + row * 128u + ((ch ^ (row & 7u)) << 4));
            mma_16816<kBf16>(o[2 * k], pf[i], b[0], b[1]);
            mma_16816<kBf16>(o[2 * k + 1], pf[i], b[2], b[3]);
          }
      }
      __syncwarp();  // every lane has read the stage
      if (u_ld < u1 && !lost) issue(st);
      if (++st == S::kStages) st = 0, ph ^= 1u;

      // ---- end of the tile, or of this CTA's run: join the four warps
      const bool tile_end = c.blk + 1u == c.t.nb;
      if (tile_end || u + 1 == u1) {
        float* mw = merge + warp * 16u * (kDP + 4u);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          l[e] += __shfl_xor_sync(0xFFFFFFFFu, l[e], 1);
          l[e] += __shfl_xor_sync(0xFFFFFFFFu, l[e], 2);
          float* row = mw + (r0 + 8u * e) * (kDP + 4u);
          if (quad == 0) row[kDP] = m[e], row[kDP + 1] = l[e];
#pragma unroll
          for (int i = 0; i < 2 * kKs; ++i)
            *reinterpret_cast<float2*>(row + 8 * i + 2u * quad) =
                make_float2(o[i][2 * e], o[i][2 * e + 1]);
        }
        const bool isbad = __syncthreads_or(bad) != 0;
        const bool whole = tile_end && tile_u >= u0;
        Piece<kDP>* piece = pieces + 2u * blockIdx.x + (tile_u >= u0 ? 1u : 0u);
        for (uint32_t r = warp; r < rows; r += kWarps) {
          float mm[kWarps], mx = -INFINITY, ll = 0.f, ov[kDP / 32];
#pragma unroll
          for (uint32_t w = 0; w < kWarps; ++w) {
            mm[w] = merge[(w * 16u + r) * (kDP + 4u) + kDP];
            mx = fmaxf(mx, mm[w]);
          }
          const float base = mx == -INFINITY ? 0.f : mx;
#pragma unroll
          for (int i = 0; i < kDP / 32; ++i) ov[i] = 0.f;
#pragma unroll
          for (uint32_t w = 0; w < kWarps; ++w) {
            const float* src = merge + (w * 16u + r) * (kDP + 4u);
            const float f = ex2(mm[w] - base);
            ll += f * src[kDP + 1];
#pragma unroll
            for (int i = 0; i < kDP / 32; ++i) ov[i] = fmaf(f, src[lane + 32u * i], ov[i]);
          }
          if (isbad) ll = INFINITY;  // a row that could not be read: zero, here or when joined
          if (whole) {
            const uint32_t R = c.t.rb * 16u + r;
            const uint64_t at =
                ((uint64_t)(c.t.q0 + R / a.G) * a.g.H + c.t.head) * a.G + R % a.G;
            store_row<kDP, kBf16>(a, at, lane, ov, mx, ll, isbad);
          } else {
#pragma unroll
            for (int i = 0; i < kDP / 32; ++i) piece->o[r][lane + 32u * i] = ov[i];
            if (lane == 0) piece->m[r] = mx, piece->l[r] = ll;
          }
        }
        if (tile_end && !whole) {  // this CTA has the last piece
          // the CTA that holds the tile's first block
          uint64_t f = tile_u * ctas / total;
          while (f + 1 < ctas && total * (f + 1) / ctas <= tile_u) ++f;
          while (f > 0 && total * f / ctas > tile_u) --f;
          join.first = (uint32_t)f;
          join.count = blockIdx.x - (uint32_t)f + 1u;
          join.q0 = c.t.q0;
          join.rows = rows;
          join.row0 = c.t.rb * 16u;
          join.head = c.t.head;
        }
        __syncthreads();
        bad = false;
        fresh = true;
        if (u + 1 < u1) {
          tile_u += c.t.nb;
          next_tile<kSel>(a, c);
        }
      } else {
        ++c.blk;
      }
    }
    if (lost) {  // the copies in flight land before the CTA leaves (or their waits give up too)
      if (lane == 0) set_status(a.g.status, IBP_ETIMEOUT);
      for (uint32_t i = 0; i < S::kStages; ++i) mbar_wait(full + i, lost_ph ^ (i < lost_st ? 1u : 0u));
    }
  }
  if (tid == 0) joins[blockIdx.x] = join;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Joins the pieces of the tile that CTA blockIdx.x of the first kernel ended, a
// warp per row.
template <int kDP, bool kBf16>
__global__ void __launch_bounds__(128) k_paged_step_join(PagedAttnArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
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
  float mx = -INFINITY;
  for (uint32_t i = lane; i < count; i += 32u) mx = fmaxf(mx, __ldcg(&at_piece(i)->m[r]));
#pragma unroll
  for (int d = 16; d; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, d));
  const float base = mx == -INFINITY ? 0.f : mx;
  float ll = 0.f, ov[kDP / 32];
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kDP / 32; ++i) ov[i] = 0.f;
#pragma unroll 4
  for (uint32_t i = 0; i < count; ++i) {
    const Piece<kDP>* p = at_piece(i);
    const float li = __ldcg(&p->l[r]);
    const float f = ex2(__ldcg(&p->m[r]) - base);
    bad = bad || li == INFINITY;
    ll += f * li;
#pragma unroll
    for (int x = 0; x < kDP / 32; ++x) ov[x] = fmaf(f, __ldcg(&p->o[r][lane + 32u * x]), ov[x]);
  }
  const uint64_t at = ((uint64_t)(q0 + (row0 + r) / a.G) * a.g.H + head) * a.G + (row0 + r) % a.G;
  store_row<kDP, kBf16>(a, at, lane, ov, mx, ll, bad);
}

template <int kDP, bool kBf16, bool kSel>
cudaError_t launch(const PagedAttnArgs& a, const PagedMaps& m, int sm_count, cudaStream_t st) {
  using S = StepShape<kDP>;
  auto kern = k_paged_step<kDP, kBf16, kSel>;
  cudaError_t e = smem_limit(reinterpret_cast<const void*>(kern), S::kSmem);
  if (e != cudaSuccess) return e;
  uint32_t ctas = (uint32_t)sm_count * (kDP == 64 ? 2u : 1u);
  if (ctas > kMaxCtas) ctas = kMaxCtas;
  kern<<<ctas, 128, S::kSmem, st>>>(m.k, m.v, a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, 4, 1);
  cfg.blockDim = dim3(128, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_paged_step_join<kDP, kBf16>, a);
}

static_assert(2u * kMaxCtas * sizeof(Piece<128>) + kMaxCtas * sizeof(Join) <= kStepWsBytes,
              "pieces and joins fit their part of the workspace");

}  // namespace

cudaError_t launch_paged_step(const PagedAttnArgs& a, const PagedMaps& m, int sm_count,
                              cudaStream_t st) {
  const bool b = a.g.bf16 != 0u;
  if (a.selected) {
    if (a.g.D <= 64u)
      return b ? launch<64, true, true>(a, m, sm_count, st)
               : launch<64, false, true>(a, m, sm_count, st);
    return b ? launch<128, true, true>(a, m, sm_count, st)
             : launch<128, false, true>(a, m, sm_count, st);
  }
  if (a.g.D <= 64u)
    return b ? launch<64, true, false>(a, m, sm_count, st)
             : launch<64, false, false>(a, m, sm_count, st);
  return b ? launch<128, true, false>(a, m, sm_count, st)
           : launch<128, false, false>(a, m, sm_count, st);
}

}  // namespace ibp
