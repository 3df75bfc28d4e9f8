// What the attention kernels of chunks share, over 16-bit pages and over 8-bit ones: tiles
// and the list of their blocks, the tensor cores' instructions, and the join of tiles
// that were cut.
#pragma once

#include "ibp_paged.cuh"
#include "ibp_sm103.cuh"

#ifdef __CUDACC__

namespace ibp {
namespace {

constexpr uint32_t kRows = 128, kTileRows = 256, kKeys = 128;
constexpr uint32_t kMaxCtas = 192;
// What a tile costs beside its blocks of keys, in blocks: its queries, its first scores and
// its output take about 8000 cycles, a block 2800.  (24 sequences of 1 to 333 tokens, 32
// heads of 64 on 4: 79.8 us; 85.7 with none, 81.0 with 6.)
constexpr uint32_t kTileUnits = 3;
constexpr uint64_t kWsBytes = IBP_PAGED_WORKSPACE_BYTES - kStepWsBytes;

template <int kDP>
struct Piece {
  float m[kTileRows], l[kTileRows];
  float o[kDP][kTileRows];
};

struct Join {
  uint32_t first, count;  // CTAs that hold the tile's pieces; count 0: none
  uint32_t q0, head;      // first row of the sequence, K/V head
  uint32_t row0, rows;    // the tile's rows
  uint32_t pad[2];
};

static_assert(2u * kMaxCtas * sizeof(Piece<128>) + kMaxCtas * sizeof(Join) <= kWsBytes,
              "pieces and joins fit their part of the workspace");

// A tile of one sequence and head and its blocks of keys.
struct Tile {
  uint32_t s, head, t;    // sequence, head, tile of 256 rows
  uint32_t q0, n, L;
  uint32_t row0, rows;    // the tile's rows among the sequence's n * G
  uint32_t b0, nb;        // first block of keys, blocks (at least 1)
  uint32_t lo, hi;        // keys that any row of the tile sees
  bool two;               // the slots take alternate blocks of the same rows
};

// The blocks of a sequence's tile whose rows are of the tokens tok0 to tok1.
__device__ __forceinline__ void tile_keys(const PagedAttnArgs& a, uint32_t n, uint32_t L,
                                          uint32_t tok0, uint32_t tok1, uint32_t& lo,
                                          uint32_t& hi, uint32_t& b0, uint32_t& nb) {
  const int64_t first = (int64_t)L - n + tok0;
  const int64_t last = (int64_t)L - n + tok1;
  const int64_t h = a.causal ? last + 1 : (int64_t)L;
  const int64_t l = a.window ? first + 1 - (int64_t)a.window : 0;
  hi = h < 0 ? 0u : (uint32_t)h;
  lo = l < 0 ? 0u : (uint32_t)l;
  b0 = lo / kKeys;
  const uint32_t b1 = (hi + kKeys - 1u) / kKeys;
  nb = b1 > b0 ? b1 - b0 : 1u;
}

// Units of one head's tiles of a sequence.
__device__ __forceinline__ uint64_t seq_units(const PagedAttnArgs& a, const PagedSeq& q) {
  const uint32_t R = q.n * a.G;
  if (q.n == 0 || R <= a.max_rows) return 0;
  // the tiles' first tokens without a division for each
  const uint32_t per = kTileRows / a.G, rest = kTileRows % a.G;
  uint64_t sum = 0;
  uint32_t tok = 0, odd = 0;  // row r is query `odd` of token `tok`
  for (uint32_t r = 0; r < R; r += kTileRows) {
    uint32_t next = tok + per, more = odd + rest;
    if (more >= a.G) more -= a.G, ++next;
    uint32_t lo, hi, b0, nb;
    tile_keys(a, q.n, q.L, tok, R - r <= kTileRows ? q.n - 1u : next - (more == 0u), lo, hi, b0,
              nb);
    sum += nb + kTileUnits;
    tok = next, odd = more;
  }
  return sum;
}

__device__ __forceinline__ void set_tile(const PagedAttnArgs& a, Tile& t) {
  t.row0 = t.t * kTileRows;
  t.rows = min(kTileRows, t.n * a.G - t.row0);
  tile_keys(a, t.n, t.L, t.row0 / a.G, (t.row0 + t.rows - 1u) / a.G, t.lo, t.hi, t.b0, t.nb);
  t.two = t.rows <= kRows;
}

__device__ __forceinline__ void set_seq(const PagedAttnArgs& a, Tile& t) {
  const PagedSeq q = paged_seq(a.b, a.g.page_lg, t.s);
  t.q0 = q.q0;
  t.n = q.n;
  t.L = q.L;
}

__device__ __forceinline__ void next_tile(const PagedAttnArgs& a, Tile& t) {
  if ((t.t + 1u) * kTileRows < t.n * a.G) {
    ++t.t;
  } else {
    t.t = 0;
    if (++t.head == a.g.H) {
      t.head = 0;
      do {
        if (++t.s >= a.b.n_seqs) return;
        set_seq(a, t);
      } while (t.n == 0 || t.n * a.G <= a.max_rows);
    }
  }
  set_tile(a, t);
}

// A run of blocks of one tile: [blk, blk + count) of its t.nb.
struct Walk {
  Tile t;
  uint32_t at;  // the tile's unit at u
  uint32_t blk, count;
  uint64_t u, u1;  // position in the list of units, end of this CTA's run
  bool fresh;
};

__device__ __forceinline__ bool walk(const PagedAttnArgs& a, Walk& w) {
  if (w.u >= w.u1) return false;
  if (!w.fresh) {
    next_tile(a, w.t);
    w.at = 0;
  }
  w.fresh = false;
  const uint64_t left = w.u1 - w.u;
  const uint32_t all = w.t.nb + kTileUnits - w.at;  // units of the tile that are left
  const uint32_t take = all > left ? (uint32_t)left : all, to = w.at + take;
  w.blk = w.at > kTileUnits ? w.at - kTileUnits : 0u;
  w.count = to > kTileUnits ? to - kTileUnits - w.blk : 0u;
  w.u += take;
  w.at = to;
  return w.count > 0;  // (a run that ends before a tile's first block has ended)
}

// The matrix instructions of a block, as one run of code: the whole warp comes here
// and elect.sync names the lane that issues.  (With a lane of one's own choosing the
// compiler cannot tell that one lane issues, and each instruction took 60 to 130 cycles to
// issue, as long as it works.)
#define IBP_MMA_SS(inc)                                                         \
  " add.s64 a, a, " inc ";\n add.s64 b, b, " inc ";\n"                          \
  " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n"
#define IBP_MMA_TS(col)                                                         \
  " add.s64 b, b, 128;\n add.u32 c, %1, " col ";\n"                             \
  " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [c], b, %4, p;\n"

// S = Q K^T over 64 channels: low descriptor words of both, their common high word;
// accumulates from the start when `acc` is set.
__device__ __forceinline__ void mma_qk(uint32_t tmem, uint32_t qlo, uint32_t klo,
                                       uint32_t hi, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, q, e;\n .reg .b64 a, b;\n elect.sync _|e, 0xFFFFFFFF;\n"
      " setp.ne.b32 q, %5, 0;\n setp.eq.b32 p, 0, 0;\n"
      " mov.b64 a, {%1, %3};\n mov.b64 b, {%2, %3};\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, q;\n" IBP_MMA_SS("2")
          IBP_MMA_SS("2") IBP_MMA_SS("2") "}\n" ::"r"(tmem),
      "r"(qlo), "r"(klo), "r"(hi), "r"(idesc), "r"(acc)
      : "memory");
}

// One step of it, for the head sizes between.
__device__ __forceinline__ void mma_qk_step(uint32_t tmem, uint32_t qlo,
                                            uint32_t klo, uint32_t hi, uint32_t idesc,
                                            uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, e;\n .reg .b64 a, b;\n elect.sync _|e, 0xFFFFFFFF;\n"
      " setp.ne.b32 p, %5, 0;\n mov.b64 a, {%1, %3};\n mov.b64 b, {%2, %3};\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n}\n" ::"r"(tmem),
      "r"(qlo), "r"(klo), "r"(hi), "r"(idesc), "r"(acc)
      : "memory");
}

// O (+)= P V over 64 keys, P in tensor memory; accumulates from the start when `acc` is set.
__device__ __forceinline__ void mma_pv(uint32_t tmem, uint32_t p, uint32_t vlo,
                                       uint32_t hi, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, q, e;\n .reg .b64 b;\n .reg .b32 c;\n elect.sync _|e, 0xFFFFFFFF;\n"
      " setp.ne.b32 q, %5, 0;\n setp.eq.b32 p, 0, 0;\n mov.b64 b, {%2, %3};\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, q;\n" IBP_MMA_TS("8")
          IBP_MMA_TS("16") IBP_MMA_TS("24") "}\n" ::"r"(tmem),
      "r"(p), "r"(vlo), "r"(hi), "r"(idesc), "r"(acc)
      : "memory");
}

__device__ __forceinline__ void commit(uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred e;\n elect.sync _|e, 0xFFFFFFFF;\n"
      " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(
          smem_addr(bar))
      : "memory");
}

#define IBP_R32(v, o)                                                                          \
  "=r"(v[o + 0]), "=r"(v[o + 1]), "=r"(v[o + 2]), "=r"(v[o + 3]), "=r"(v[o + 4]),              \
      "=r"(v[o + 5]), "=r"(v[o + 6]), "=r"(v[o + 7]), "=r"(v[o + 8]), "=r"(v[o + 9]),          \
      "=r"(v[o + 10]), "=r"(v[o + 11]), "=r"(v[o + 12]), "=r"(v[o + 13]), "=r"(v[o + 14]),     \
      "=r"(v[o + 15]), "=r"(v[o + 16]), "=r"(v[o + 17]), "=r"(v[o + 18]), "=r"(v[o + 19]),     \
      "=r"(v[o + 20]), "=r"(v[o + 21]), "=r"(v[o + 22]), "=r"(v[o + 23]), "=r"(v[o + 24]),     \
      "=r"(v[o + 25]), "=r"(v[o + 26]), "=r"(v[o + 27]), "=r"(v[o + 28]), "=r"(v[o + 29]),     \
      "=r"(v[o + 30]), "=r"(v[o + 31])
#define IBP_W32(v, o)                                                                          \
  "r"(v[o + 0]), "r"(v[o + 1]), "r"(v[o + 2]), "r"(v[o + 3]), "r"(v[o + 4]), "r"(v[o + 5]),    \
      "r"(v[o + 6]), "r"(v[o + 7]), "r"(v[o + 8]), "r"(v[o + 9]), "r"(v[o + 10]),              \
      "r"(v[o + 11]), "r"(v[o + 12]), "r"(v[o + 13]), "r"(v[o + 14]), "r"(v[o + 15]),          \
      "r"(v[o + 16]), "r"(v[o + 17]), "r"(v[o + 18]), "r"(v[o + 19]), "r"(v[o + 20]),          \
      "r"(v[o + 21]), "r"(v[o + 22]), "r"(v[o + 23]), "r"(v[o + 24]), "r"(v[o + 25]),          \
      "r"(v[o + 26]), "r"(v[o + 27]), "r"(v[o + 28]), "r"(v[o + 29]), "r"(v[o + 30]),          \
      "r"(v[o + 31])

// 32 columns of this warp's lanes; the caller waits.
template <int kO, int kN>
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&r)[kN]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
      "%28, %29, %30, %31}, [%32];"
      : IBP_R32(r, kO)
      : "r"(addr));
}

template <int kO, int kN>
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&r)[kN]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
      "%28, %29, %30, %31, %32};" ::"r"(addr),
      IBP_W32(r, kO)
      : "memory");
}

// Waits for the loads; their registers are read only after it.
template <int kN>
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[kN]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < kN; ++i) asm volatile("" : "+r"(r[i]));
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tc_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// A barrier of the slots' eight warps, and whether all of them say so.
__device__ __forceinline__ bool all_of_eight(bool mine) {
  uint32_t all;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n"
      " barrier.cta.red.and.pred q, 2, 256, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(all)
      : "r"((uint32_t)mine)
      : "memory");
  return all != 0u;
}

// What the other warps are told of a run of blocks; count 0: there is no more.
struct Info {
  uint32_t count, two;    // blocks; the slots take alternate ones
  uint32_t q0, head;
  uint32_t row0, rows;
  uint32_t n, L;
  uint32_t lo, hi, key0;  // keys that any row sees, first key of the run
  uint32_t whole;         // the run is the whole tile: write the result, not a piece
  uint32_t place;         // which of the CTA's two pieces
  uint32_t s;             // sequence
  uint32_t all_lo, all_hi;  // keys that every row sees
};
// The list of units and this CTA's run of it: the walk's start, the list's length, the CTAs
// that have a run.
template <uint32_t kThreads>
__device__ __forceinline__ Walk chunk_run(const PagedAttnArgs& a, uint64_t* s_scan,
                                          uint64_t* s_found, uint64_t& total, uint32_t& ctas) {
  const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31u;
  uint64_t mine = 0, mine0 = 0;
  total = 0;
  for (uint32_t s = tid; s < a.b.n_seqs; s += kThreads) {
    const PagedSeq q = paged_seq(a.b, a.g.page_lg, s);
    if (!q.ok) set_status(a.g.status, IBP_ERANGE);
    mine += seq_units(a, q);
    if (s == tid) mine0 = mine;
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) mine += __shfl_xor_sync(0xFFFFFFFFu, mine, d);
  if (lane == 0) s_scan[warp] = mine;
  tc_before();
  __syncthreads();
  tc_after();
  for (uint32_t w = 0; w < kThreads / 32; ++w) total += s_scan[w];
  total *= a.g.H;
  ctas = total < gridDim.x ? (uint32_t)total : gridDim.x;
  Walk w0{};
  uint64_t u0 = 0;
  if (blockIdx.x < ctas) {
    u0 = total * blockIdx.x / ctas;
    w0.u1 = total * (blockIdx.x + 1u) / ctas;
    uint64_t base = 0;
    for (uint32_t c = 0; c < a.b.n_seqs; c += kThreads) {
      uint64_t nb = mine0;
      if (c) nb = c + tid < a.b.n_seqs ? seq_units(a, paged_seq(a.b, a.g.page_lg, c + tid)) : 0;
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
        s_found[1] = nb;
        s_found[2] = u0 - lo_u;
      }
      base += all * a.g.H;
      if (u0 < base) break;
    }
    __syncthreads();
    const uint64_t per_head = s_found[1], in = s_found[2];
    w0.t.s = (uint32_t)s_found[0];
    set_seq(a, w0.t);
    w0.t.head = (uint32_t)(in / per_head);
    uint64_t rem = in % per_head;
    w0.t.t = 0;
    set_tile(a, w0.t);
    while (rem >= w0.t.nb + kTileUnits) {
      rem -= w0.t.nb + kTileUnits;
      ++w0.t.t;
      set_tile(a, w0.t);
    }
    w0.at = (uint32_t)rem;
    w0.u = u0;
    w0.fresh = true;
  }
  return w0;
}

// One thread tells the others of a run of blocks, and keeps the join that this CTA asks for
// when the run is the last piece of a tile that was cut.
__device__ __forceinline__ void tell_run(const PagedAttnArgs& a, const Walk& w, uint64_t total,
                                         uint32_t ctas, bool more, Info* x, uint64_t* bar,
                                         Join& join) {
  const uint64_t tile_u = w.u - w.at + kTileUnits;  // the tile's first block in the list
  const bool whole = w.blk == 0 && w.count == w.t.nb;
  x->count = more ? w.count : 0u;
  x->two = w.t.two;
  x->q0 = w.t.q0;
  x->head = w.t.head;
  x->row0 = w.t.row0;
  x->rows = w.t.rows;
  x->n = w.t.n;
  x->L = w.t.L;
  x->lo = w.t.lo;
  x->hi = w.t.hi;
  x->key0 = (w.t.b0 + w.blk) * kKeys;
  x->whole = whole;
  x->place = w.blk == 0u ? 1u : 0u;
  x->s = w.t.s;
  {
    const int32_t first = (int32_t)(w.t.L - w.t.n + w.t.row0 / a.G);
    const int32_t last = (int32_t)(w.t.L - w.t.n + (w.t.row0 + w.t.rows - 1u) / a.G);
    x->all_hi = a.causal ? (uint32_t)max(first + 1, 0) : w.t.L;
    x->all_lo = a.window && last >= (int32_t)a.window
                    ? (uint32_t)(last + 1 - (int32_t)a.window)
                    : 0u;
  }
  mbar_arrive(bar);
  if (more && w.blk + w.count == w.t.nb && !whole) {
    uint64_t f = tile_u * ctas / total;
    while (f + 1 < ctas && total * (f + 1) / ctas <= tile_u) ++f;
    while (f > 0 && total * f / ctas > tile_u) --f;
    join.first = (uint32_t)f;
    join.count = blockIdx.x - (uint32_t)f + 1u;
    join.q0 = w.t.q0;
    join.head = w.t.head;
    join.row0 = w.t.row0;
    join.rows = w.t.rows;
  }
}

// The barriers between a CTA's warps.
struct Bars {
  uint64_t *full, *empty;   // of the ring's places: keys or values are there; were read
  uint64_t *s_full;         // per slot: scores are there
  uint64_t *p_full;         // per slot: half the weights (values, the next keys) are there
  uint64_t *p2_full;        // per slot: the other half
  uint64_t *turn;           // per slot: the other has issued its products
  uint64_t *q_full;         // the tile's queries are there
  uint64_t *o_full;         // every product of the tile is done
  uint64_t *done;           // per slot: its last products are done
};

// A warp's part of a slot's matrix products, of 16-bit operands of one type.
template <typename S, int kDP, bool kBf16, uint32_t kRing, typename InfoOf>
__device__ __forceinline__ void issue_products(const PagedAttnArgs& a, uint32_t slot,
                                               uint32_t tmem, const uint8_t* s_q,
                                               const uint8_t* s_kv, const Bars& bars,
                                               uint32_t* s_fail, InfoOf info_of) {
  const uint32_t lane = threadIdx.x & 31u;
  const uint32_t base_desc = (1u << 4) | ((uint32_t)kBf16 << 7) | ((uint32_t)kBf16 << 10) |
                             ((kRows >> 4) << 24);
  const uint32_t qk_desc = base_desc | ((kKeys >> 3) << 17);
  const uint32_t pv_desc = base_desc | ((a.g.D >> 3) << 17) | (1u << 16);
  // Descriptors of 128-byte swizzled tiles.  Queries and keys: rows along the
  // reduction, 8 to an atom of 1024 bytes.  Values, as the transposed operand: rows of
  // 64 channels for each key, 8 keys to an atom, the next 64 channels half a tile on.
  const uint32_t desc_hi = (uint32_t)(sw128_desc(0) >> 32);
  const uint32_t q_lo = (uint32_t)sw128_desc(smem_addr(s_q));
  const uint32_t kv_lo = (uint32_t)sw128_desc(smem_addr(s_kv));
  const uint32_t v_lead = ((S::kHalf >> 4) << 16) - (1u << 16);
  const uint32_t k_steps = a.g.D / 16u;
  const uint32_t ts = tmem + slot * 128u, to = tmem + 256u + slot * 128u;
  uint32_t e0 = 0, tiles = 0, pn = 0, tn = 0;
  bool go = true;
  // S = Q K^T; the other slot's turn begins with the last of it, since a turn takes
  // as long to pass on as two products to run
  // once its products are done; twice: for both slots
  auto release = [&](uint32_t e, bool twice) {
    commit(bars.empty + e % kRing);
    if (twice) commit(bars.empty + e % kRing);
  };
  auto qk = [&](uint32_t qslot, uint32_t e, bool two, bool pass) {
    const uint32_t qa = q_lo + qslot * (S::kTile >> 4);
    const uint32_t ka = kv_lo + (e % kRing) * (S::kTile >> 4);
    if (k_steps == kDP / 16u) {
      if (kDP == 128) mma_qk(ts, qa, ka, desc_hi, qk_desc, 0u);
      if (pass && lane == 0) mbar_arrive(bars.turn + (slot ^ 1u));
      __syncwarp();
      constexpr uint32_t kOff = kDP == 128 ? S::kHalf >> 4 : 0u;
      mma_qk(ts, qa + kOff, ka + kOff, desc_hi, qk_desc, kDP == 128 ? 1u : 0u);
    } else {
      for (uint32_t k = 0; k < k_steps; ++k) {
        const uint32_t off = (k >> 2) * (S::kHalf >> 4) + 2u * (k & 3u);
        mma_qk_step(ts, qa + off, ka + off, desc_hi, qk_desc, k ? 1u : 0u);
      }
      if (pass && lane == 0) mbar_arrive(bars.turn + (slot ^ 1u));
      __syncwarp();
    }
    commit(bars.s_full + slot);
    release(e, two);
  };
  while (go) {
    const Info* x = info_of(tiles);
    if (!x) break;
    const uint32_t nb = x->count;
    const bool two = x->two != 0u;
    const uint32_t step = two ? 2u : 1u, qslot = two ? 0u : slot;
    go = wait_or_fail(bars.q_full, tiles & 1u, s_fail);
    tc_after();
    uint32_t i = two ? slot : 0u;
    if (go && i < nb) {
      const uint32_t ek = e0 + 2u * i;
      go = wait_or_fail(bars.full + ek % kRing, (ek / kRing) & 1u, s_fail);
      tc_after();
      if (go) qk(qslot, ek, two, false);
    }
    // The slots take turns, so that one's products run while the other's weights are
    // computed (left alone they fall into step, and both wait for both).
    for (uint32_t b = 0; b < nb && go; b += step, i += step) {
      const uint32_t ev = e0 + 2u * i + 1u, ek = e0 + 2u * (i + step);
      const uint32_t va = kv_lo + v_lead + (ev % kRing) * (S::kTile >> 4);
      // the weights, and with them these values and the next keys
      const uint32_t parity = pn & 1u;
      go = wait_or_fail(bars.turn + slot, tn++ & 1u, s_fail);
      if (i < nb) go = go && wait_or_fail(bars.p_full + slot, parity, s_fail);
      tc_after();
      if (!go) break;
      if (i < nb) {
        mma_pv(to, ts, va, desc_hi, pv_desc, b ? 1u : 0u);
        go = wait_or_fail(bars.p2_full + slot, parity, s_fail);
        tc_after();
        if (!go) break;
        mma_pv(to, ts + 32u, va + 512u, desc_hi, pv_desc, 1u);
        release(ev, two);
        ++pn;
      }
      if (i + step < nb) {
        qk(qslot, ek, two, true);
      } else {
        if (lane == 0) mbar_arrive(bars.turn + (slot ^ 1u));
        __syncwarp();
      }
    }
    commit(bars.o_full);
    e0 += 2u * nb;
    ++tiles;
  }
  // whosever wait gave up: products in flight end before the tensor memory goes
  commit(bars.done + slot);
  mbar_wait(bars.done + slot, 0);
}

// Joins the pieces of the tile that CTA blockIdx.x of the first kernel ended, in the
// pieces' order: 32 rows per CTA (lane = row), 16 channels per warp.
template <int kDP, bool kBf16>
__device__ __forceinline__ void join_tile(const PagedAttnArgs& a) {
  const Join* joins = reinterpret_cast<const Join*>(a.ws + IBP_PAGED_WORKSPACE_BYTES -
                                                    kMaxCtas * sizeof(Join));
  const Piece<kDP>* pieces = reinterpret_cast<const Piece<kDP>*>(a.ws + kStepWsBytes);
  const uint4 j0 = __ldcg(reinterpret_cast<const uint4*>(joins + blockIdx.x));
  const uint4 j1 = __ldcg(reinterpret_cast<const uint4*>(joins + blockIdx.x) + 1);
  const uint32_t first = j0.x, count = j0.y, rows = j1.y;
  const uint32_t r = blockIdx.y * 32u + (threadIdx.x & 31u), d0 = (threadIdx.x >> 5) * 16u;
  if (count == 0 || r >= rows || d0 >= a.g.D) return;
  auto at_piece = [&](uint32_t i) { return pieces + 2u * (first + i) + (i == 0u ? 1u : 0u); };
  float mx = -INFINITY;
  for (uint32_t i = 0; i < count; ++i)
    if (__ldcg(&at_piece(i)->l[r]) != 0.f) mx = fmaxf(mx, __ldcg(&at_piece(i)->m[r]));
  const float base = mx == -INFINITY ? 0.f : mx;
  float ll = 0.f, ov[16];
  bool bad = false;
#pragma unroll
  for (int x = 0; x < 16; ++x) ov[x] = 0.f;
  for (uint32_t i = 0; i < count; ++i) {
    const Piece<kDP>* p = at_piece(i);
    const float li = __ldcg(&p->l[r]);
    const float f = ex2(__ldcg(&p->m[r]) - base);
    float v[16];
#pragma unroll
    for (int x = 0; x < 16; ++x) v[x] = __ldcg(&p->o[d0 + x][r]);
    if (li == 0.f) continue;
    bad = bad || li == INFINITY;
    ll += f * li;
#pragma unroll
    for (int x = 0; x < 16; ++x) ov[x] = fmaf(f, v[x], ov[x]);
  }
  const uint32_t R = j1.x + r;
  const uint64_t at = ((uint64_t)(j0.z + R / a.G) * a.g.H + j0.w) * a.G + R % a.G;
  const bool some = !bad && ll != 0.f;
  const float inv = some ? 1.f / ll : 0.f;
  uint32_t y[8];
#pragma unroll
  for (int x = 0; x < 8; ++x) y[x] = some ? pack2(ov[2 * x] * inv, ov[2 * x + 1] * inv, kBf16) : 0u;
  uint4* dst = reinterpret_cast<uint4*>(a.out + (at * a.g.D + d0) * 2u);
  dst[0] = make_uint4(y[0], y[1], y[2], y[3]);
  dst[1] = make_uint4(y[4], y[5], y[6], y[7]);
  if (a.lse && d0 == 0) a.lse[at] = some ? (mx + log2f(ll)) * 0.69314718056f : -INFINITY;
}

// Behind the step kernel's join (max_rows is set) every piece is there when this starts,
// since that join lets it start after its own wait: it waits at its end, so that what
// follows may count on both.
template <int kDP, bool kBf16>
__global__ void __launch_bounds__(kDP * 2) k_paged_chunk_join(PagedAttnArgs a) {
  if (!a.max_rows) asm volatile("griddepcontrol.wait;" ::: "memory");
  join_tile<kDP, kBf16>(a);
  if (a.max_rows) asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <int kDP, bool kBf16>
cudaError_t launch_chunk_join(const PagedAttnArgs& a, int sm_count, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((uint32_t)sm_count < kMaxCtas ? (uint32_t)sm_count : kMaxCtas, 8, 1);
  cfg.blockDim = dim3(kDP * 2, 1, 1);  // a warp per 16 channels
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_paged_chunk_join<kDP, kBf16>, a);
}

}  // namespace
}  // namespace ibp

#endif
