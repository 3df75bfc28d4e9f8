// Attention of chunks of new tokens over a paged K/V cache on the tensor cores.
//
//   S = Q K^T,  P = exp2(c S - c m),  O += P V,  l += rows of P
//
// over blocks of 128 keys, with m a reference maximum of each row that is moved
// (and O, l rescaled) only when the running maximum has outgrown it by 2^8: the
// result does not depend on the reference, and P stays within the 16-bit
// types.  Bound by the tensor cores and the exponentials together: 4 D
// operations a (row, key) against one exponential.
//
// One CTA per SM works on tiles of 256 rows of one (sequence, K/V head): row r is
// query r % G of token r / G, so the queries that share K/V fill a tile however
// few tokens a chunk has.  Two slots of 128 rows alternate: while the tensor
// cores work for one, four warps take the other's exponentials.
//   warp 0        TMA: keys and values of a block, a box per page, into a ring of 5 tiles
//   warp 1        one thread issues tcgen05.mma: S = Q K^T (both from shared
//                 memory) into 128 columns of tensor memory per slot, O += P V with P
//                 from tensor memory, over S's columns, and V as the transposed operand
//   warps 4 - 7   slot 0, warps 8 - 11 slot 1 (thread = row): queries into shared memory,
//                 then per block S -> registers, mask, maximum, exponentials, P
// A tile of at most 128 rows gives both slots the same rows, slot 0 the even
// blocks of keys and slot 1 the odd ones, and joins them at its end.
//
// The blocks of all tiles are one list, cut into equal runs, one per CTA; a tile
// that is cut is joined from its pieces by a second kernel, in order.
#include "ibp_paged.cuh"
#include "ibp_sm103.cuh"
#include "ibp_tma.cuh"

namespace ibp {
namespace {

constexpr uint32_t kRows = 128, kTileRows = 256, kKeys = 128, kRing = 5, kThreads = 384;
constexpr uint32_t kMaxCtas = 192;
constexpr uint64_t kWsBytes = IBP_PAGED_WORKSPACE_BYTES - kStepWsBytes;

template <int kDP>
struct Piece {
  float m[kTileRows], l[kTileRows];
  float o[kTileRows][kDP];
};

struct Join {
  uint32_t first, count;  // CTAs that hold the tile's pieces; count 0: none
  uint32_t q0, head;      // first row of the sequence, K/V head
  uint32_t row0, rows;    // the tile's rows
  uint32_t pad[2];
};

static_assert(2u * kMaxCtas * sizeof(Piece<128>) + kMaxCtas * sizeof(Join) <= kWsBytes,
              "pieces and joins fit their part of the workspace");

template <int kDP>
struct Shape {
  static constexpr uint32_t kHalves = kDP / 64;
  static constexpr uint32_t kHalf = 128u * 128u;            // 128 rows of 64 channels
  static constexpr uint32_t kTile = kHalves * kHalf;
  static constexpr uint32_t kSmem = 1024u + (2u + kRing) * kTile + 512u;
};

// A tile of one sequence and head and its blocks of keys.
struct Tile {
  uint32_t s, head, t;    // sequence, head, tile of 256 rows
  uint32_t q0, n, L;
  uint32_t row0, rows;    // the tile's rows among the sequence's n * G
  uint32_t b0, nb;        // first block of keys, blocks (at least 1)
  uint32_t lo, hi;        // keys that any row of the tile sees
  bool two;               // the slots take alternate blocks of the same rows
};

// The blocks of tile t of a sequence.
__device__ __forceinline__ void tile_keys(const PagedAttnArgs& a, uint32_t n, uint32_t L,
                                          uint32_t row0, uint32_t rows, uint32_t& lo,
                                          uint32_t& hi, uint32_t& b0, uint32_t& nb) {
  const int64_t first = (int64_t)L - n + row0 / a.G;
  const int64_t last = (int64_t)L - n + (row0 + rows - 1u) / a.G;
  const int64_t h = a.causal ? last + 1 : (int64_t)L;
  const int64_t l = a.window ? first + 1 - (int64_t)a.window : 0;
  hi = h < 0 ? 0u : (uint32_t)h;
  lo = l < 0 ? 0u : (uint32_t)l;
  b0 = lo / kKeys;
  const uint32_t b1 = (hi + kKeys - 1u) / kKeys;
  nb = b1 > b0 ? b1 - b0 : 1u;
}

// Blocks of one head's tiles of a sequence.
__device__ __forceinline__ uint64_t seq_blocks(const PagedAttnArgs& a, const PagedSeq& q) {
  const uint32_t R = q.n * a.G;
  if (q.n == 0 || R <= a.max_rows) return 0;
  uint64_t sum = 0;
  for (uint32_t r = 0; r < R; r += kTileRows) {
    uint32_t lo, hi, b0, nb;
    tile_keys(a, q.n, q.L, r, min(kTileRows, R - r), lo, hi, b0, nb);
    sum += nb;
  }
  return sum;
}

__device__ __forceinline__ void set_tile(const PagedAttnArgs& a, Tile& t) {
  t.row0 = t.t * kTileRows;
  t.rows = min(kTileRows, t.n * a.G - t.row0);
  tile_keys(a, t.n, t.L, t.row0, t.rows, t.lo, t.hi, t.b0, t.nb);
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
  uint32_t blk, count;
  uint64_t u, u1;  // position in the list of blocks, end of this CTA's run
  bool fresh;
};

__device__ __forceinline__ bool walk(const PagedAttnArgs& a, Walk& w) {
  if (w.u >= w.u1) return false;
  if (!w.fresh) {
    next_tile(a, w.t);
    w.blk = 0;
  }
  w.fresh = false;
  const uint64_t left = w.u1 - w.u;
  w.count = w.t.nb - w.blk;
  if (w.count > left) w.count = (uint32_t)left;
  w.u += w.count;
  return true;
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

// Descriptor of V as the transposed right operand: rows of 64 channels
// (128 bytes, swizzled) for each key; 8 keys to an atom of 1024 bytes, the next 64
// channels a half tile further.
__device__ __forceinline__ uint64_t v_desc(uint32_t saddr, uint32_t half_bytes) {
  uint64_t d = (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(half_bytes >> 4) << 16;  // leading: 64 channels on
  d |= (uint64_t)(1024u >> 4) << 32;       // stride: 8 keys on
  d |= (uint64_t)1u << 46;
  d |= (uint64_t)2u << 61;
  return d;
}

// The matrix instructions, issued by the lane with `on` set: the whole warp walks
// the same path, so that descriptors are uniform values.
__device__ __forceinline__ void mma_ss(uint32_t on, uint32_t tmem, uint64_t adesc,
                                       uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, e;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 e, %5, 0;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(on)
      : "memory");
}

// A from tensor memory.
__device__ __forceinline__ void mma_ts(uint32_t on, uint32_t tmem, uint32_t a, uint64_t bdesc,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, e;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 e, %5, 0;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(tmem),
      "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(on)
      : "memory");
}

__device__ __forceinline__ void commit(uint32_t on, uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred e;\n setp.ne.b32 e, %1, 0;\n"
      " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(
          smem_addr(bar)),
      "r"(on)
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

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Whether both slots (256 threads) say so; every tile has one such vote, so that
// neither waits for the other once one has given up.
__device__ __forceinline__ bool both_slots(bool mine) {
  uint32_t all;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n"
      " barrier.cta.red.and.pred q, 2, 256, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(all)
      : "r"((uint32_t)mine)
      : "memory");
  return all != 0u;
}

// A wait of a whole warp that also gives up once another role has.
__device__ __forceinline__ bool wait_or_fail(uint64_t* bar, uint32_t parity, uint32_t* fail) {
  const bool there = !*reinterpret_cast<volatile uint32_t*>(fail) && mbar_wait(bar, parity);
  if (!there) atomicExch(fail, 1u);
  return __all_sync(0xFFFFFFFFu, there);
}

template <int kDP, bool kBf16>
__global__ void __launch_bounds__(kThreads, 1)
    k_paged_chunk(const __grid_constant__ CUtensorMap map_k,
                  const __grid_constant__ CUtensorMap map_v, PagedAttnArgs a) {
  using S = Shape<kDP>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023u) & ~static_cast<uintptr_t>(1023u));
  uint8_t* s_q = smem;                  // 2 slots of queries
  uint8_t* s_kv = smem + 2u * S::kTile; // the ring: K, V, K, V, ...
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + (2u + kRing) * S::kTile);
  uint64_t* empty = full + kRing;
  uint64_t* s_full = empty + kRing;  // per slot: scores are there
  uint64_t* p_full = s_full + 2;     // per slot: weights are there
  uint64_t* q_full = p_full + 2;     // the tile's queries are there
  uint64_t* o_full = q_full + 1;     // every product of the tile is done
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(o_full + 1);
  uint32_t* s_fail = s_tmem + 1;
  uint32_t* s_bad = s_fail + 1;      // 8 blocks: bit per page with an id out of range
  __shared__ uint64_t s_scan[kThreads / 32];
  __shared__ uint64_t s_found[3];

  const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31u;
  Piece<kDP>* pieces = reinterpret_cast<Piece<kDP>*>(a.ws + kStepWsBytes);
  Join* joins = reinterpret_cast<Join*>(a.ws + IBP_PAGED_WORKSPACE_BYTES -
                                        kMaxCtas * sizeof(Join));
  if (tid == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_k)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_v)) : "memory");
    for (uint32_t i = 0; i < kRing; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, 1);
    }
    for (uint32_t i = 0; i < 2; ++i) {
      mbar_init(s_full + i, 1);
      mbar_init(p_full + i, 128);
    }
    mbar_init(q_full, 256);
    mbar_init(o_full, 1);
    *s_fail = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(s_tmem)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // ---- the list of blocks and this CTA's run of it
  uint64_t mine = 0, total = 0;
  for (uint32_t s = tid; s < a.b.n_seqs; s += kThreads) {
    const PagedSeq q = paged_seq(a.b, a.g.page_lg, s);
    if (!q.ok) set_status(a.g.status, IBP_ERANGE);
    mine += seq_blocks(a, q);
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) mine += __shfl_xor_sync(0xFFFFFFFFu, mine, d);
  if (lane == 0) s_scan[warp] = mine;
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = *s_tmem;
  for (uint32_t w = 0; w < kThreads / 32; ++w) total += s_scan[w];
  total *= a.g.H;
  const uint32_t ctas = total < gridDim.x ? (uint32_t)total : gridDim.x;
  Walk w0{};
  uint64_t u0 = 0;
  if (blockIdx.x < ctas) {
    u0 = total * blockIdx.x / ctas;
    w0.u1 = total * (blockIdx.x + 1u) / ctas;
    uint64_t base = 0;
    for (uint32_t c = 0; c < a.b.n_seqs; c += kThreads) {
      uint64_t nb = 0;
      if (c + tid < a.b.n_seqs) nb = seq_blocks(a, paged_seq(a.b, a.g.page_lg, c + tid));
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
    while (rem >= w0.t.nb) {
      rem -= w0.t.nb;
      ++w0.t.t;
      set_tile(a, w0.t);
    }
    w0.blk = (uint32_t)rem;
    w0.u = u0;
    w0.fresh = true;
  }
  Join join{};

  if (warp == 0) {
    // ---------------- producer: lane i loads page i of the block
    const uint32_t lg = a.g.page_lg, box_lg = lg < 7u ? lg : 7u;
    const uint32_t npg = kKeys >> box_lg;
    uint32_t e = 0, blocks = 0;  // ring entries filled, blocks begun
    bool go = true;
    Walk w = w0;
    while (go && walk(a, w)) {
      const int32_t* table = a.b.table + w.t.s * a.b.table_stride;
      auto page_at = [&](uint32_t b) {
        const uint32_t key = (w.t.b0 + b) * kKeys + (lane << box_lg);
        if (lane >= npg || key >= w.t.hi || key + (1u << box_lg) <= w.t.lo) return -1;
        const int32_t id = __ldg(table + (key >> lg));
        return id < 0 || (uint32_t)id >= a.g.n_pages ? -2 : id;
      };
      int32_t next = page_at(w.blk);
      for (uint32_t b = w.blk; b < w.blk + w.count && go; ++b, ++blocks) {
        const int32_t id = next;
        if (b + 1u < w.blk + w.count) next = page_at(b + 1u);
        const uint32_t token = ((w.t.b0 + b) * kKeys + (lane << box_lg)) & ((1u << lg) - 1u);
        const uint32_t bad = __ballot_sync(0xFFFFFFFFu, id == -2);
        const uint32_t bytes =
            __popc(__ballot_sync(0xFFFFFFFFu, id >= 0)) * (S::kHalves * 128u << box_lg);
#pragma unroll
        for (uint32_t kv = 0; kv < 2; ++kv, ++e) {
          const uint32_t st = e % kRing, round = e / kRing;
          if (round > 0) go = wait_or_fail(empty + st, (round - 1u) & 1u, s_fail);
          if (!go) break;
          if (lane == 0) {
            if (kv == 0) s_bad[blocks & 7u] = bad;
            mbar_expect_tx(full + st, bytes);
          }
          __syncwarp();
          if (id >= 0) {
            uint8_t* dst = s_kv + st * S::kTile + ((lane << box_lg) * 128u);
#pragma unroll
            for (uint32_t hf = 0; hf < S::kHalves; ++hf)
              tma_load_page(dst + hf * S::kHalf, kv ? &map_v : &map_k, full + st, 64u * hf, token,
                            w.t.head, id);
          }
        }
      }
    }
    // after a failure: the copies in flight land (or their waits give up too)
    if (!go)
      for (uint32_t i = e > kRing ? e - kRing : 0u; i < e; ++i)
        mbar_wait(full + i % kRing, (i / kRing) & 1u);
  } else if (warp == 1) {
    // ---------------- matrix products
    const uint32_t on = lane == 0 ? 1u : 0u;
    {
      const uint32_t base_desc = (1u << 4) | ((uint32_t)kBf16 << 7) | ((uint32_t)kBf16 << 10) |
                                 ((kRows >> 4) << 24);
      const uint32_t qk_desc = base_desc | ((kKeys >> 3) << 17);
      const uint32_t pv_desc = base_desc | ((a.g.D >> 3) << 17) | (1u << 16);
      uint32_t e0 = 0, tiles = 0, pn[2] = {0, 0};
      bool go = true;
      Walk w = w0;
      auto k_entry = [&](uint32_t i) { return e0 + 2u * i; };
      auto wait_entry = [&](uint32_t e) {
        go = go && wait_or_fail(full + e % kRing, (e / kRing) & 1u, s_fail);
        tc_after();
      };
      auto qk = [&](uint32_t slot, uint32_t qslot, uint32_t e) {
        const uint32_t qa = smem_addr(s_q + qslot * S::kTile);
        const uint32_t ka = smem_addr(s_kv + (e % kRing) * S::kTile);
#pragma unroll
        for (uint32_t k = 0; k < kDP / 16u; ++k) {
          if (16u * k >= a.g.D) break;
          const uint32_t off = (k >> 2) * S::kHalf + 32u * (k & 3u);
          mma_ss(on, tmem + slot * 128u, sw128_desc(qa + off), sw128_desc(ka + off), qk_desc,
                  k != 0u ? 1u : 0u);
        }
        commit(on, s_full + slot);
      };
      auto pv = [&](uint32_t slot, uint32_t e, bool first) {
        go = go && wait_or_fail(p_full + slot, pn[slot]++ & 1u, s_fail);
        tc_after();
        if (!go) return;
        const uint32_t va = smem_addr(s_kv + (e % kRing) * S::kTile);
#pragma unroll
        for (uint32_t k = 0; k < kKeys / 16u; ++k)
          mma_ts(on, tmem + 256u + slot * 128u, tmem + slot * 128u + 8u * k,
                     v_desc(va + 2048u * k, S::kHalf), pv_desc, first && k == 0u ? 0u : 1u);
      };
      while (go && walk(a, w)) {
        go = wait_or_fail(q_full, tiles & 1u, s_fail);
        tc_after();
        if (!go) break;
        const uint32_t nb = w.count;
        if (!w.t.two) {
          wait_entry(k_entry(0));
          if (!go) break;
          qk(0, 0, k_entry(0));
          qk(1, 1, k_entry(0));
          commit(on, empty + k_entry(0) % kRing);
          for (uint32_t i = 0; i < nb && go; ++i) {
            const uint32_t ev = k_entry(i) + 1u, ek = k_entry(i + 1u);
            wait_entry(ev);
            pv(0, ev, i == 0u);
            if (i + 1u < nb && go) {
              wait_entry(ek);
              if (go) qk(0, 0, ek);
            }
            pv(1, ev, i == 0u);
            commit(on, empty + ev % kRing);
            if (i + 1u < nb && go) {
              qk(1, 1, ek);
              commit(on, empty + ek % kRing);
            }
          }
        } else {
          for (uint32_t i = 0; i < 2u && i < nb && go; ++i) {
            wait_entry(k_entry(i));
            if (go) qk(i, 0, k_entry(i));
            commit(on, empty + k_entry(i) % kRing);
          }
          for (uint32_t i = 0; i < nb && go; ++i) {
            const uint32_t slot = i & 1u, ev = k_entry(i) + 1u, ek = k_entry(i + 2u);
            wait_entry(ev);
            pv(slot, ev, i < 2u);
            commit(on, empty + ev % kRing);
            if (i + 2u < nb && go) {
              wait_entry(ek);
              if (go) qk(slot, 0, ek);
              commit(on, empty + ek % kRing);
            }
          }
        }
        commit(on, o_full);
        e0 += 2u * nb;
        ++tiles;
      }
      if (!go) {  // products in flight finish before the tensor memory goes
        commit(on, o_full);
        mbar_wait(o_full, tiles & 1u);
      }
    }
  } else if (warp >= 4) {
    // ---------------- a slot's rows: thread = row
    const uint32_t slot = (warp - 4u) >> 2, wq = warp & 3u, r = wq * 32u + lane;
    const uint32_t lane_base = (wq * 32u) << 16;
    const uint32_t ts = tmem + lane_base + slot * 128u, to = tmem + lane_base + 256u + slot * 128u;
    const float c = a.scale_log2;
    uint32_t sn = 0, tiles = 0, blocks = 0, e0 = 0;
    bool go = true;
    Walk w = w0;
    while (go && walk(a, w)) {
      const uint64_t tile_u = w.u - w.count - w.blk;  // the tile's first block in the list
      const bool two = w.t.two;
      const uint32_t nrows = two ? w.t.rows : min(kRows, w.t.rows > slot * kRows ? w.t.rows - slot * kRows : 0u);
      const uint32_t row0 = w.t.row0 + (two ? 0u : slot * kRows);
      if (!two || slot == 0) {  // the slot's queries, 16 lanes a row
        uint8_t* dst = s_q + slot * S::kTile;
        constexpr uint32_t kCh = kDP / 8u;  // 16-byte chunks of a row
#pragma unroll 4
        for (uint32_t i = r; i < kRows * kCh; i += 128u) {
          const uint32_t row = i / kCh, ch = i % kCh;
          uint4 x = make_uint4(0, 0, 0, 0);
          if (row < nrows && ch * 8u < a.g.D) {
            const uint32_t R = row0 + row;
            x = __ldg(reinterpret_cast<const uint4*>(
                a.q + (uint64_t)(w.t.q0 + R / a.G) * a.q_stride +
                ((uint64_t)w.t.head * a.G + R % a.G) * a.g.D * 2u + ch * 16u));
          }
          *reinterpret_cast<uint4*>(dst + (ch >> 3) * S::kHalf + row * 128u +
                                    (((ch & 7u) ^ (row & 7u)) << 4)) = x;
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      }
      mbar_arrive(q_full);
      // this row's keys: [from, to)
      const bool live = r < nrows;
      const int64_t pos = (int64_t)w.t.L - w.t.n + (row0 + (live ? r : 0u)) / a.G;
      const uint32_t to_key = !live ? 0u : a.causal ? (uint32_t)(pos + 1 > 0 ? pos + 1 : 0) : w.t.L;
      const uint32_t from_key =
          a.window && pos + 1 > (int64_t)a.window ? (uint32_t)(pos + 1 - a.window) : 0u;
      float m = -INFINITY, base = 0.f, l = 0.f;  // running maximum (scaled), reference, sum
      bool rowbad = false;
      bool any = false;  // a product has been accumulated
      for (uint32_t i = two ? slot : 0u; i < w.count && go; i += two ? 2u : 1u) {
        go = wait_or_fail(s_full + slot, sn++ & 1u, s_fail);
        if (!go) break;
        tc_after();
        uint32_t sv[128];
        tmem_ld32<0>(ts, sv);
        tmem_ld32<32>(ts + 32u, sv);
        tmem_ld32<64>(ts + 64u, sv);
        tmem_ld32<96>(ts + 96u, sv);
        const uint32_t key0 = (w.t.b0 + w.blk + i) * kKeys;
        const uint32_t badp = s_bad[(blocks + i) & 7u];
        const bool edge = key0 + kKeys > w.t.hi || key0 < w.t.lo || badp;
        if (edge && (two || slot == 0)) {
          // values that no row sees: zero, so that 0 * (what they hold) is 0
          const uint32_t ev = e0 + 2u * i + 1u;
          go = wait_or_fail(full + ev % kRing, (ev / kRing) & 1u, s_fail);
          const uint32_t key = key0 + r;  // this thread's key
          const uint32_t pg = r >> (a.g.page_lg < 7u ? a.g.page_lg : 7u);
          if (go && (key >= w.t.hi || key < w.t.lo || (badp >> pg & 1u))) {
            const uint32_t va = smem_addr(s_kv + (ev % kRing) * S::kTile) + r * 128u;
#pragma unroll
            for (uint32_t x = 0; x < S::kHalves * 8u; ++x)
              asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                               va + (x >> 3) * S::kHalf + (x & 7u) * 16u),
                           "r"(0u)
                           : "memory");
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        tmem_wait_ld(sv);
        float s[128];
#pragma unroll
        for (int j = 0; j < 128; ++j) s[j] = __uint_as_float(sv[j]);
        uint32_t pw[64];
        if (__any_sync(0xFFFFFFFFu, key0 + kKeys > to_key || key0 < from_key) || badp) {
          const int32_t hi = (int32_t)to_key - (int32_t)key0, lo = (int32_t)from_key - (int32_t)key0;
#pragma unroll
          for (int j = 0; j < 128; ++j)
            if (j >= hi || j < lo) s[j] = -INFINITY;
          if (badp) {
            const uint32_t bl = a.g.page_lg < 7u ? a.g.page_lg : 7u;
#pragma unroll
            for (int j = 0; j < 128; ++j)
              if (badp >> ((uint32_t)j >> bl) & 1u) {
                rowbad = rowbad || (j < hi && j >= lo);
                s[j] = -INFINITY;
              }
            if (r == 0) set_status(a.g.status, IBP_ERANGE);
          }
        }
        float mx0 = s[0], mx1 = s[1], mx2 = s[2], mx3 = s[3];
#pragma unroll
        for (int j = 4; j < 128; j += 4) {
          mx0 = fmaxf(mx0, s[j]);
          mx1 = fmaxf(mx1, s[j + 1]);
          mx2 = fmaxf(mx2, s[j + 2]);
          mx3 = fmaxf(mx3, s[j + 3]);
        }
        m = fmaxf(m, fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3)) * c);
        const bool none = l == 0.f;  // this row has seen no key: any reference will do
        if (!any) {
          base = m == -INFINITY ? 0.f : m;
        } else if (__any_sync(0xFFFFFFFFu, m > base + 8.f || (none && m != -INFINITY))) {
          // every product issued so far is done (the scores came after it)
          const float nb = none && m != -INFINITY ? m : fmaxf(m, base);
          const float f = none ? 1.f : ex2(base - nb);
          base = nb;
          l *= f;
#pragma unroll
          for (uint32_t x = 0; x < kDP / 32u; ++x) {
            if (32u * x >= a.g.D) break;
            uint32_t o[32];
            tmem_ld32<0>(to + 32u * x, o);
            tmem_wait_ld(o);
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
            tmem_st32<0>(to + 32u * x, o);
          }
        }
        any = true;
        float l0 = 0.f, l1 = 0.f, l2 = 0.f, l3 = 0.f;
#pragma unroll
        for (int j = 0; j < 128; j += 4) {
          const float p0 = ex2(fmaf(s[j], c, -base)), p1 = ex2(fmaf(s[j + 1], c, -base));
          const float p2 = ex2(fmaf(s[j + 2], c, -base)), p3 = ex2(fmaf(s[j + 3], c, -base));
          l0 += p0;
          l1 += p1;
          l2 += p2;
          l3 += p3;
          pw[j / 2] = pack2(p0, p1, kBf16);
          pw[j / 2 + 1] = pack2(p2, p3, kBf16);
        }
        l += (l0 + l1) + (l2 + l3);
        tmem_st32<0>(ts, pw);
        tmem_st32<32>(ts + 32u, pw);
        tmem_wait_st();
        tc_before();
        mbar_arrive(p_full + slot);
      }
      blocks += w.count;
      e0 += 2u * w.count;
      go = go && wait_or_fail(o_full, tiles++ & 1u, s_fail);
      go = both_slots(go && *reinterpret_cast<volatile uint32_t*>(s_fail) == 0u);
      if (!go) break;
      tc_after();
      const bool whole = w.blk == 0 && w.count == w.t.nb;
      const bool ends = w.blk + w.count == w.t.nb;
      Piece<kDP>* piece = pieces + 2u * blockIdx.x + (tile_u >= u0 ? 1u : 0u);
      float f0 = 1.f, f1 = 0.f;
      // alternate blocks: slot 1 hands its sums to slot 0 through the free half of the
      // queries' space, 64 channels at a time, [channel][row]
      float* x_o = reinterpret_cast<float*>(s_q + S::kTile);
      if (two) {
        // (maximum, sum and the unread-page flag first)
        if (slot == 1) {
          x_o[r] = any ? base : -INFINITY;
          x_o[128u + r] = l;
          x_o[256u + r] = rowbad ? 1.f : 0.f;
        }
        asm volatile("bar.sync 1, 256;" ::: "memory");
        if (slot == 0) {
          const float b1 = x_o[r], l1 = x_o[128u + r];
          rowbad = rowbad || x_o[256u + r] != 0.f;
          const float nb = l1 != 0.f && b1 > base ? b1 : base;
          f0 = ex2(base - nb);
          f1 = b1 == -INFINITY ? 0.f : ex2(b1 - nb);
          l = l * f0 + l1 * f1;
          base = nb;
        }
        asm volatile("bar.sync 1, 256;" ::: "memory");
      }
      const bool some = live && !rowbad && l != 0.f;
      const uint32_t R = row0 + r;
      const uint64_t at = live ? ((uint64_t)(w.t.q0 + R / a.G) * a.g.H + w.t.head) * a.G + R % a.G
                               : 0u;
      const float inv = some ? 1.f / l : 0.f;
      const uint32_t pr = slot * kRows + r;
      const bool writes = live && !(two && slot == 1);
#pragma unroll
      for (uint32_t x = 0; x < kDP / 32u; ++x) {
        if (32u * x >= a.g.D) break;
        uint32_t o[32];
        tmem_ld32<0>(to + 32u * x, o);
        tmem_wait_ld(o);
        float of[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) of[j] = __uint_as_float(o[j]);
        if (two) {
          if (slot == 1)
#pragma unroll
            for (int j = 0; j < 32; ++j) x_o[j * 128 + r] = any ? of[j] : 0.f;
          asm volatile("bar.sync 1, 256;" ::: "memory");
          if (slot == 0)
#pragma unroll
            for (int j = 0; j < 32; ++j)
              of[j] = f1 != 0.f ? of[j] * f0 + x_o[j * 128 + r] * f1 : of[j] * f0;
          asm volatile("bar.sync 1, 256;" ::: "memory");
        }
        if (writes && whole) {
          uint8_t* dst = a.out + (at * a.g.D + 32u * x) * 2u;
#pragma unroll
          for (int v = 0; v < 4; ++v)
            if (32u * x + 8u * v < a.g.D) {
              uint32_t y[4];
#pragma unroll
              for (int j = 0; j < 4; ++j)
                y[j] = pack2(some ? of[8 * v + 2 * j] * inv : 0.f,
                             some ? of[8 * v + 2 * j + 1] * inv : 0.f, kBf16);
              *reinterpret_cast<uint4*>(dst + 16 * v) = make_uint4(y[0], y[1], y[2], y[3]);
            }
        } else if (writes) {
          float4* dst = reinterpret_cast<float4*>(&piece->o[pr][32u * x]);
#pragma unroll
          for (int v = 0; v < 8; ++v)
            dst[v] = make_float4(of[4 * v], of[4 * v + 1], of[4 * v + 2], of[4 * v + 3]);
        }
      }
      if (writes && whole) {
        if (a.lse) a.lse[at] = some ? (base + log2f(l)) * 0.69314718056f : -INFINITY;
      } else if (writes) {
        piece->m[pr] = base;
        piece->l[pr] = rowbad ? INFINITY : l;
      }
      tc_before();
      if (ends && !whole) {
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
    if (tid == 128u) joins[blockIdx.x] = join;
  }
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u)
                 : "memory");
  if (tid == 0 && *s_fail) set_status(a.g.status, IBP_ETIMEOUT);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Joins the pieces of the tile that CTA blockIdx.x of the first kernel ended: a
// warp per row, in the pieces' order.
template <int kDP, bool kBf16>
__global__ void __launch_bounds__(256) k_paged_chunk_join(PagedAttnArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Join* joins = reinterpret_cast<const Join*>(a.ws + IBP_PAGED_WORKSPACE_BYTES -
                                                    kMaxCtas * sizeof(Join));
  const Piece<kDP>* pieces = reinterpret_cast<const Piece<kDP>*>(a.ws + kStepWsBytes);
  const uint4 j0 = __ldcg(reinterpret_cast<const uint4*>(joins + blockIdx.x));
  const uint4 j1 = __ldcg(reinterpret_cast<const uint4*>(joins + blockIdx.x) + 1);
  const uint32_t first = j0.x, count = j0.y, rows = j1.y, lane = threadIdx.x & 31u;
  if (count == 0) return;
  auto at_piece = [&](uint32_t i) { return pieces + 2u * (first + i) + (i == 0u ? 1u : 0u); };
  for (uint32_t r = blockIdx.y * 8u + (threadIdx.x >> 5); r < rows; r += gridDim.y * 8u) {
    float mx = -INFINITY;
    for (uint32_t i = lane; i < count; i += 32u)
      if (__ldcg(&at_piece(i)->l[r]) != 0.f) mx = fmaxf(mx, __ldcg(&at_piece(i)->m[r]));
#pragma unroll
    for (int d = 16; d; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, d));
    const float base = mx == -INFINITY ? 0.f : mx;
    float ll = 0.f, ov[kDP / 32];
    bool bad = false;
#pragma unroll
    for (int x = 0; x < kDP / 32; ++x) ov[x] = 0.f;
    for (uint32_t i = 0; i < count; ++i) {
      const Piece<kDP>* p = at_piece(i);
      const float li = __ldcg(&p->l[r]);
      if (li == 0.f) continue;
      const float f = ex2(__ldcg(&p->m[r]) - base);
      bad = bad || li == INFINITY;
      ll += f * li;
#pragma unroll
      for (int x = 0; x < kDP / 32; ++x) ov[x] = fmaf(f, __ldcg(&p->o[r][lane + 32u * x]), ov[x]);
    }
    const uint32_t R = j1.x + r;
    const uint64_t at = ((uint64_t)(j0.z + R / a.G) * a.g.H + j0.w) * a.G + R % a.G;
    const bool some = !bad && ll != 0.f;
    const float inv = some ? 1.f / ll : 0.f;
    uint16_t* dst = reinterpret_cast<uint16_t*>(a.out) + at * a.g.D;
#pragma unroll
    for (int x = 0; x < kDP / 32; ++x)
      if (lane + 32u * x < a.g.D)
        dst[lane + 32u * x] = (uint16_t)pack2(some ? ov[x] * inv : 0.f, 0.f, kBf16);
    if (a.lse && lane == 0) a.lse[at] = some ? (mx + log2f(ll)) * 0.69314718056f : -INFINITY;
  }
}

template <int kDP, bool kBf16>
cudaError_t launch(const PagedAttnArgs& a, const PagedMaps& m, int sm_count, cudaStream_t st) {
  using S = Shape<kDP>;
  auto kern = k_paged_chunk<kDP, kBf16>;
  cudaError_t e = smem_limit(reinterpret_cast<const void*>(kern), S::kSmem);
  if (e != cudaSuccess) return e;
  const uint32_t ctas = (uint32_t)sm_count < kMaxCtas ? (uint32_t)sm_count : kMaxCtas;
  kern<<<ctas, kThreads, S::kSmem, st>>>(m.k, m.v, a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, 8, 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_paged_chunk_join<kDP, kBf16>, a);
}

}  // namespace

cudaError_t launch_paged_chunk(const PagedAttnArgs& a, const PagedMaps& m, int sm_count,
                               cudaStream_t st) {
  const bool b = a.g.bf16 != 0u;
  if (a.g.D <= 64u)
    return b ? launch<64, true>(a, m, sm_count, st) : launch<64, false>(a, m, sm_count, st);
  return b ? launch<128, true>(a, m, sm_count, st) : launch<128, false>(a, m, sm_count, st);
}

}  // namespace ibp
