// Attention of chunks of new tokens over a paged K/V cache on the tensor cores.
//
//   S = Q K^T,  P = exp2(c S - c m),  O += P V,  l += rows of P
//
// over blocks of 128 keys, with m a reference maximum of each row that is moved
// (and O, l rescaled) only when the running maximum has outgrown it by 2^8 (fp16: 2^4): the
// result does not depend on the reference, and P stays within the 16-bit
// types.  P is rounded to them, as the tensor cores take it, l is the sum of the unrounded
// weights.  In fp16 the reference lies 2^11 below the maximum that it was taken from, so that
// weights down to 2^-25 of the largest are normal numbers (P is at most 2^15).  Bound by the tensor cores and the exponentials together: 4 D
// operations a (row, key) against one exponential.
//
// One CTA per SM works on tiles of 256 rows of one (sequence, K/V head): row r is
// query r % G of token r / G, so the queries that share K/V fill a tile however
// few tokens a chunk has.  Two slots of 128 rows alternate: while the tensor
// cores work for one, four warps take the other's exponentials.
//   warps 0 - 3   slot 0, warps 4 - 7 slot 1 (thread = row): queries into shared memory,
//                 then per block S -> registers, mask, exponentials, maximum, P in two
//                 halves, so that P V begins while the second half is computed
//   warp 8        walks the tiles and tells the others of each through shared
//                 memory; TMA: keys and values of a block, a box per page, into a ring of
//                 5 tiles
//   warps 9, 10   issue tcgen05.mma, one for each slot, so that the tensor cores have the
//                 other slot's products while one waits: S = Q K^T (both from shared
//                 memory) into 128 columns of tensor memory, O += P V with P from tensor
//                 memory, over S's columns, and V as the transposed operand
//   warp 11       waits for keys and values in the issuing warp's place, and says so
//                 with the weights' barrier: one wait less between two products
// A tile of at most 128 rows gives both slots the same rows, slot 0 the even
// blocks of keys and slot 1 the odd ones, and joins them at its end.
//
// The blocks of all tiles, with some units in front of each for the tile itself, are one
// list, cut into equal runs, one per CTA; a tile that is cut is joined from its pieces
// by a second kernel, in order.
//
// Measured: 2048 tokens behind 6144, 64 query heads of 128 on 8, causal: 331 us, 1.45
// PFLOP/s, bound by the scores' products (both operands from shared memory: 740 to
// 830 cycles a block against 520 for the values') and the turns between the slots.
// Without turns (both issuers at will) 438 us; a tile's memory released by the
// tensor cores' own commits 338, by the waiting warp 346 to 357; weights written before
// the turn is taken 345 to 365.
#include "ibp_paged_chunk.cuh"
#include "ibp_tma.cuh"

namespace ibp {
namespace {

constexpr uint32_t kRing = 5, kThreads = 384;

template <int kDP>
struct Shape {
  static constexpr uint32_t kHalves = kDP / 64;
  static constexpr uint32_t kHalf = 128u * 128u;            // 128 rows of 64 channels
  static constexpr uint32_t kTile = kHalves * kHalf;
  static constexpr uint32_t kSmem = 1024u + (2u + kRing) * kTile + 512u;
};

// The blocks of a tile in which some rows see keys that others do not, and some of those
// keys' values are infinite or NaN: bit per key.  A tile's rows span at most 256
// positions, so there are at most 3 such blocks at either end of what they see.
constexpr uint32_t kOdd = 8;
struct Odd {
  uint32_t count, key0[kOdd], keys[kOdd][4];
};
// The ring of what the other warps are told: the walking warp is at most 3 tiles ahead, since
// each takes two of the 5 places for keys and values and a tile's queries wait for the
// tile before.
constexpr uint32_t kInfos = 8;
// Keys whose weights are computed before the first half of them is handed over: what
// waits for the first half's store is then hidden (64 to 112 measured alike).
constexpr int kEarly = 80;

// The registers of the launch, shared out again: 8 warps of 208 and 4 of 88 are
// the 12 of 168 that the launch came with.
__device__ __forceinline__ void reg_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 208;"); }
__device__ __forceinline__ void reg_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 88;"); }
static_assert(8 * 208 + 4 * 88 <= 12 * 168, "no more registers than the launch has");

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
  uint64_t* p_full = s_full + 2;     // per slot: half the weights (values, the next keys) are there
  uint64_t* p2_full = p_full + 2;    // per slot: the other half
  uint64_t* turn = p2_full + 2;      // per slot: the other has issued its products
  uint64_t* q_full = turn + 2;       // the tile's queries are there
  uint64_t* o_full = q_full + 1;     // every product of the tile is done
  uint64_t* done = o_full + 1;       // per slot: its last products are done
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(done + 2);
  uint32_t* s_fail = s_tmem + 1;
  uint32_t* s_bad = s_fail + 1;      // 8 blocks: bit per page with an id out of range
  __shared__ Info s_info[kInfos];
  __shared__ uint64_t info_full[kInfos];
  __shared__ Odd s_odd[2];  // of this tile and the next
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
      mbar_init(empty + i, 2);
    }
    for (uint32_t i = 0; i < 2; ++i) {
      mbar_init(s_full + i, 1);
      mbar_init(p_full + i, 5);
      mbar_init(p2_full + i, 4);
      mbar_init(turn + i, 1);
      mbar_init(done + i, 1);
    }
    for (uint32_t i = 0; i < kInfos; ++i) mbar_init(info_full + i, 1);
    mbar_init(q_full, 8);
    mbar_init(o_full, 2);
    *s_fail = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (tid == 0) mbar_arrive(turn);  // slot 0 begins
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(s_tmem)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // what comes behind may take the SMs that have ended (it waits for this grid itself)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  uint64_t total;
  uint32_t ctas;
  const Walk w0 = chunk_run<kThreads>(a, s_scan, s_found, total, ctas);
  const uint32_t tmem = *s_tmem;
  // the tile of number t, once its run is known; false: no more, or given up
  auto info_of = [&](uint32_t t) -> const Info* {
    const Info* x = s_info + t % kInfos;
    if (!wait_or_fail(info_full + t % kInfos, (t / kInfos) & 1u, s_fail)) return nullptr;
    return x->count ? x : nullptr;
  };

  if (warp == 8) {
    reg_dec();
    // ---------------- the walk, and loads: lane i loads page i of the block
    const uint32_t lg = a.g.page_lg, box_lg = lg < 7u ? lg : 7u;
    const uint32_t npg = kKeys >> box_lg;
    uint32_t e = 0, blocks = 0, tiles = 0;  // ring entries filled, blocks and tiles begun
    bool go = true;
    Walk w = w0;
    Join join{};
    while (go) {
      const bool more = walk(a, w);
      if (lane == 0) tell_run(a, w, total, ctas, more, s_info + tiles % kInfos,
                              info_full + tiles % kInfos, join);
      ++tiles;
      __syncwarp();
      if (!more) break;
      const int32_t* table =
          a.b.table + w.t.s * a.b.table_stride + w.t.head * a.b.table_heads;
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
    if (lane == 0) joins[blockIdx.x] = join;
    // whosever wait gave up: the copies in flight land (or these waits give up too)
    for (uint32_t i = e > kRing ? e - kRing : 0u; i < e; ++i)
      mbar_wait(full + i % kRing, (i / kRing) & 1u);
  } else if (warp == 9 || warp == 10) {
    reg_dec();
    const Bars bars{full, empty, s_full, p_full, p2_full, turn, q_full, o_full, done};
    issue_products<S, kDP, kBf16, kRing>(a, warp - 9u, tmem, s_q, s_kv, bars, s_fail, info_of);
  } else if (warp == 11) {
    reg_dec();
    // ---------------- keys and values are there: one arrival with each block's weights
    uint32_t e0 = 0, tiles = 0, blocks = 0, pn[2] = {0, 0};
    bool go = true;
    const uint32_t box_lg = a.g.page_lg < 7u ? a.g.page_lg : 7u;
    auto entry = [&](uint32_t e) {
      go = go && wait_or_fail(full + e % kRing, (e / kRing) & 1u, s_fail);
    };
    while (go) {
      Odd* odd = s_odd + (tiles & 1u);
      const Info* t = info_of(tiles++);
      if (!t) break;
      const uint32_t nb = t->count, two = t->two, step = two ? 2u : 1u;
      const int32_t lo = (int32_t)t->lo, hi = (int32_t)t->hi;
      const int32_t every_lo = (int32_t)t->all_lo, every_hi = (int32_t)t->all_hi;
      uint32_t n_odd = 0;
      if (lane == 0) odd->count = 0;
      for (uint32_t i = 0; i < nb && go; ++i, ++blocks) {
        const uint32_t ev = e0 + 2u * i + 1u;
        entry(ev);  // these values
        if (!go) break;
        // Values that no row sees become zero, so that 0 * (what they hold) is 0.  Where only
        // some rows see a key, infinities and NaN of its values become zero too, and are
        // added to the rows that see them at the tile's end.
        const int32_t key0 = (int32_t)(t->key0 + i * kKeys);
        const uint32_t badp = s_bad[blocks & 7u];
        const bool mixed = key0 + (int32_t)kKeys > every_hi || key0 < every_lo;
        if (mixed || badp || key0 + (int32_t)kKeys > hi || key0 < lo) {
          uint32_t found[4];
#pragma unroll
          for (uint32_t g = 0; g < 4; ++g) {
            const uint32_t row = 32u * g + lane;  // this thread's key
            const int32_t key = key0 + (int32_t)row;
            const uint32_t va = smem_addr(s_kv + (ev % kRing) * S::kTile) + row * 128u;
            // an exponent of ones, plus one, reaches the sign's place
            constexpr uint32_t kExp = kBf16 ? 0x7F807F80u : 0x7C007C00u;
            constexpr uint32_t kOne = kBf16 ? 0x00800080u : 0x04000400u;
            auto chunk = [&](uint32_t x) {
              return va + (x >> 3) * S::kHalf + (((x & 7u) ^ (lane & 7u)) << 4);
            };
            uint32_t hit = 0;
            if (key >= hi || key < lo || (badp >> (row >> box_lg) & 1u)) {
#pragma unroll 4
              for (uint32_t x = 0; x < S::kHalves * 8u; ++x)
                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(chunk(x)), "r"(0u)
                             : "memory");
            } else if (mixed) {
#pragma unroll 4
              for (uint32_t x = 0; x < S::kHalves * 8u; ++x) {
                uint32_t y[4];
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(y[0]), "=r"(y[1]), "=r"(y[2]), "=r"(y[3])
                             : "r"(chunk(x))
                             : "memory");
#pragma unroll
                for (int k = 0; k < 4; ++k) hit |= (y[k] & kExp) + kOne;
              }
              hit &= 0x80008000u;
              if (hit)
#pragma unroll 1
                for (uint32_t x = 0; x < S::kHalves * 32u; ++x) {
                  const uint32_t at = chunk(x >> 2) + 4u * (x & 3u);
                  uint32_t y;
                  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(y) : "r"(at) : "memory");
                  const uint32_t ones = (y & kExp) + kOne;  // a half's top bit
                  if (ones & 0x8000u) y &= 0xFFFF0000u;
                  if (ones & 0x80000000u) y &= 0x0000FFFFu;
                  asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(y) : "memory");
                }
            }
            found[g] = __ballot_sync(0xFFFFFFFFu, hit != 0u);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if ((found[0] | found[1] | found[2] | found[3]) && n_odd < kOdd) {
            if (lane == 0) {
              odd->key0[n_odd] = (uint32_t)key0;
              for (int g = 0; g < 4; ++g) odd->keys[n_odd][g] = found[g];
              odd->count = n_odd + 1u;
            }
            ++n_odd;
          }
        }
        if (i + step < nb) entry(e0 + 2u * (i + step));  // the slot's next keys
        if (!go) break;
        const uint32_t s0 = two ? i & 1u : 0u, s1 = two ? s0 : 1u;
        if (lane == 0)
          for (uint32_t x = s0; x <= s1; ++x) mbar_arrive(p_full + x);
        // the next arrival belongs to the next phase
        for (uint32_t x = s0; x <= s1 && go; ++x)
          go = wait_or_fail(p_full + x, pn[x]++ & 1u, s_fail);
      }
      e0 += 2u * nb;
    }
  } else {
    reg_inc();
    // ---------------- a slot's rows: thread = row
    const uint32_t slot = warp >> 2, wq = warp & 3u, r = wq * 32u + lane;
    const uint32_t lane_base = (wq * 32u) << 16;
    const uint32_t ts = tmem + lane_base + slot * 128u, to = tmem + lane_base + 256u + slot * 128u;
    const float c = a.scale_log2;
    const uint32_t box_lg = a.g.page_lg < 7u ? a.g.page_lg : 7u;
    // This warp's 32 rows of the slot's queries in shared memory, 16 bytes at a
    // time; between two tiles they hold the rows of the output.
    constexpr uint32_t kCh = kDP / 8u, kPer = 32u / kCh, kLd = 32u / kPer;
    uint8_t* s_rows = s_q + slot * S::kTile + wq * 32u * 128u;
    const uint32_t my_ch = lane % kCh, my_sub = lane / kCh;
    auto chunk_at = [&](uint32_t row, uint32_t ch) {
      return s_rows + (ch >> 3) * S::kHalf + row * 128u + (((ch & 7u) ^ (row & 7u)) << 4);
    };
    // The tile's queries: lane i knows where row i lies, 16 (or 8) lanes fetch a row.
    auto load_q = [&](const Info* t) {
      const uint32_t n = t->two ? (slot ? 0u : t->rows)
                                : (t->rows > slot * kRows ? t->rows - slot * kRows : 0u);
      if (!t->two || slot == 0) {
        const uint32_t R = t->row0 + slot * kRows + (r < n ? r : 0u), tok = R / a.G;
        const uint64_t p = reinterpret_cast<uint64_t>(
            a.q + (uint64_t)(t->q0 + tok) * a.q_stride +
            (uint64_t)(t->head * a.G + (R - tok * a.G)) * a.g.D * 2u);
#pragma unroll
        for (uint32_t i = 0; i < kLd; ++i) {
          const uint32_t row = i * kPer + my_sub;
          const uint64_t src = __shfl_sync(0xFFFFFFFFu, p, row) + my_ch * 16u;
          const bool there = wq * 32u + row < n && my_ch * 8u < a.g.D;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                           smem_addr(chunk_at(row, my_ch))),
                       "l"(there ? src : p), "r"(there ? 16u : 0u)
                       : "memory");
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
    };
    // Infinities and NaN of the values of the block's odd keys that this row sees, into
    // 32 channels of its sums: rare, and read again from the pages.
    auto add_odd = [&](const Info* t, uint32_t key0, const uint32_t (&keys)[4], uint32_t x,
                       int32_t from, int32_t to, uint32_t (&o)[32]) {
#pragma unroll 1
      for (uint32_t j = 0; j < kKeys; ++j) {
        const int32_t key = (int32_t)(key0 + j);
        if (!(keys[j >> 5] >> (j & 31u) & 1u) || key < from || key >= to) continue;
        const int32_t page =
            __ldg(a.b.table + t->s * a.b.table_stride + t->head * a.b.table_heads +
                  ((uint32_t)key >> a.g.page_lg));
        const uint16_t* v = reinterpret_cast<const uint16_t*>(
            a.g.v + (uint64_t)(uint32_t)page * a.g.page_stride + t->head * a.g.head_stride +
            ((uint32_t)key & ((1u << a.g.page_lg) - 1u)) * a.g.token_stride);
#pragma unroll
        for (int d = 0; d < 32; ++d)
          if (32u * x + d < a.g.D) {
            const float f = to_float(__ldg(v + 32u * x + d), kBf16);
            if (!(fabsf(f) < INFINITY)) o[d] = __float_as_uint(__uint_as_float(o[d]) + f);
          }
      }
    };
    uint32_t sn = 0, tiles = 0, blocks = 0;
    while (true) {
      bool go = true;
      const Info* t = info_of(tiles);
      if (!t) {
        all_of_eight(false);
        break;
      }
      load_q(t);
      const bool both = t->two != 0u;
      const uint32_t count = t->count;
      // this row, and its keys: [from, to)
      const bool live = r + (both ? 0u : slot * kRows) < t->rows;
      int32_t to_key, from_key;
      uint64_t at;  // its place among [n_tokens, q_heads]
      {
        const uint32_t R = t->row0 + (both ? 0u : slot * kRows) + (live ? r : 0u);
        const uint32_t tok = R / a.G;
        at = ((uint64_t)(t->q0 + tok) * a.g.H + t->head) * a.G + (R - tok * a.G);
        const int32_t pos = (int32_t)(t->L - t->n + tok);
        to_key = !live ? 0 : a.causal ? max(pos + 1, 0) : (int32_t)t->L;
        from_key = a.window && pos + 1 > (int32_t)a.window ? pos + 1 - (int32_t)a.window : 0;
      }
      int32_t key0 = (int32_t)t->key0;
      // keys that every row of the warp sees need no mask
      const int32_t all_to = __reduce_min_sync(0xFFFFFFFFu, live ? to_key : 0x7FFFFFFF);
      const int32_t all_from = __reduce_max_sync(0xFFFFFFFFu, live ? from_key : 0);
      float m = -INFINITY, base = 0.f, l = 0.f;  // running maximum (scaled), reference, sum
      bool rowbad = false;
      bool any = false;  // a product has been accumulated
      if (both) key0 += (int32_t)(slot * kKeys);
      for (uint32_t i = both ? slot : 0u; i < count; i += both ? 2u : 1u) {
        go = wait_or_fail(s_full + slot, sn++ & 1u, s_fail);
        if (!go) break;
        tc_after();
        uint32_t sv[128];
        tmem_ld32<0>(ts, sv);
        tmem_ld32<32>(ts + 32u, sv);
        tmem_ld32<64>(ts + 64u, sv);
        tmem_ld32<96>(ts + 96u, sv);
        const uint32_t badp = s_bad[(blocks + i) & 7u];
        const bool masked = key0 + (int32_t)kKeys > all_to || key0 < all_from || badp;
        // 32 keys from k0 on: a bit for each that this row sees
        auto seen = [&](int32_t k0) {
          const int32_t hi = min(max(to_key - k0, 0), 32), lo = min(max(from_key - k0, 0), 32);
          uint32_t v = (hi >= 32 ? ~0u : (1u << hi) - 1u) & (lo >= 32 ? 0u : ~0u << lo);
          if (badp) {  // pages with an id out of range
#pragma unroll 1
            for (int j = 0; j < 32; ++j)
              if ((v >> j & 1u) && (badp >> ((uint32_t)(k0 - key0 + j) >> box_lg) & 1u)) {
                rowbad = true;
                v &= ~(1u << j);
              }
            if (r == 0) set_status(a.g.status, IBP_ERANGE);
          }
          return v;
        };
        tmem_wait_ld(sv);
        if (masked)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const uint32_t v = seen(key0 + 32 * g);
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (!(v >> j & 1u)) sv[32 * g + j] = 0xFF800000u;
          }
        // The weights need a reference, not the maximum: they are computed with the one
        // at hand while the maximum is found, and again in the rare block whose
        // maximum has outgrown it.
        const uint64_t c2 = pair2(c, c);
        uint64_t l0, l1, b2;
        auto weights = [&](const int j, uint32_t (&w2)[32]) {  // 4 keys
          float p0, p1, p2, p3;
          halves2(fma2(pair2(__uint_as_float(sv[j]), __uint_as_float(sv[j + 1])), c2, b2), p0, p1);
          halves2(fma2(pair2(__uint_as_float(sv[j + 2]), __uint_as_float(sv[j + 3])), c2, b2), p2,
                  p3);
          p0 = ex2(p0), p1 = ex2(p1), p2 = ex2(p2), p3 = ex2(p3);
          l0 = add2(l0, pair2(p0, p1));
          l1 = add2(l1, pair2(p2, p3));
          w2[(j & 63) / 2] = pack2(p0, p1, kBf16);
          w2[(j & 63) / 2 + 1] = pack2(p2, p3, kBf16);
        };
        uint32_t pa[32], pb[32];
        b2 = pair2(-base, -base);
        l0 = l1 = 0;
        float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < 64; j += 4) {
          weights(j, pa);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            x[k] = max3(x[k], __uint_as_float(sv[2 * j + 2 * k]),
                        __uint_as_float(sv[2 * j + 2 * k + 1]));
        }
        m = fmaxf(m, fmaxf(max3(x[0], x[1], x[2]), x[3]) * c);
        const bool none = l == 0.f;  // this row has seen no key: any reference will do
        constexpr float kLift = kBf16 ? 0.f : 11.f, kMost = kBf16 ? 8.f : 15.f;
        if (__any_sync(0xFFFFFFFFu, m > base + kMost || (none && m != -INFINITY))) {
          const float nb = none && m != -INFINITY ? m - kLift : fmaxf(m - kLift, base);
          const float f = none ? 1.f : ex2(base - nb);
          base = nb;
          l *= f;
          // every product issued so far is done (the scores came after it)
          if (any)
#pragma unroll 1
            for (uint32_t d = 0; 32u * d < a.g.D; ++d) {
              uint32_t o[32];
              tmem_ld32<0>(to + 32u * d, o);
              tmem_wait_ld(o);
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
              tmem_st32<0>(to + 32u * d, o);
            }
          b2 = pair2(-base, -base);
          l0 = l1 = 0;
#pragma unroll
          for (int j = 0; j < 64; j += 4) weights(j, pa);
        }
        any = true;
        tmem_st32<0>(ts, pa);
        auto arrive = [&](uint64_t* bar) {
          tmem_wait_st();
          tc_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar);
        };
#pragma unroll
        for (int j = 64; j < kEarly; j += 4) weights(j, pb);
        arrive(p_full + slot);
#pragma unroll
        for (int j = kEarly; j < 128; j += 4) weights(j, pb);
        tmem_st32<0>(ts + 32u, pb);
        {
          float u, v;
          halves2(add2(l0, l1), u, v);
          l += u + v;
        }
        arrive(p2_full + slot);
        key0 += (int32_t)(both ? 2u * kKeys : kKeys);
      }
      blocks += count;
      go = go && wait_or_fail(o_full, tiles & 1u, s_fail);
      ++tiles;
      // The slots count on each other below: all eight warps go on, or all leave.  (Each
      // comes here, also one that gave up a wait which another saw end.)
      if (!all_of_eight(go)) break;
      tc_after();
      const bool whole = t->whole != 0u;
      const Odd& odd = s_odd[(tiles - 1u) & 1u];
      float f0 = 1.f, f1 = 0.f;
      // alternate blocks: slot 1 hands its sums to slot 0 through the space of its queries
      float* x_o = reinterpret_cast<float*>(s_q + S::kTile);
      if (both) {
        if (slot == 1) {
          x_o[r] = any ? base : -INFINITY;
          x_o[128u + r] = l;
          x_o[256u + r] = rowbad ? 1.f : 0.f;
        }
        asm volatile("barrier.cta.sync 1, 256;" ::: "memory");
        if (slot == 0) {
          const float b1 = x_o[r], l1 = x_o[128u + r];
          rowbad = rowbad || x_o[256u + r] != 0.f;
          const float nb = l1 == 0.f ? base : l == 0.f ? b1 : fmaxf(b1, base);
          f0 = l == 0.f ? 0.f : ex2(base - nb);
          f1 = l1 == 0.f ? 0.f : ex2(b1 - nb);
          l = l * f0 + l1 * f1;
          base = nb;
        }
        asm volatile("barrier.cta.sync 1, 256;" ::: "memory");
      }
      const bool some = live && !rowbad && l != 0.f;
      const float inv = some ? 1.f / l : 0.f;
      const bool mine = !(both && slot == 1);  // slot 0 writes for both
      Piece<kDP>* piece = pieces + 2u * blockIdx.x + t->place;
#pragma unroll 1
      for (uint32_t x = 0; 32u * x < a.g.D; ++x) {
        uint32_t o[32];
        tmem_ld32<0>(to + 32u * x, o);
        tmem_wait_ld(o);
        if (both) {
          if (slot == 1)
#pragma unroll
            for (int j = 0; j < 32; ++j) x_o[j * 128 + r] = any ? __uint_as_float(o[j]) : 0.f;
          asm volatile("barrier.cta.sync 1, 256;" ::: "memory");
          if (slot == 0)
#pragma unroll
            for (int j = 0; j < 32; ++j)
              o[j] = __float_as_uint((f0 != 0.f ? __uint_as_float(o[j]) * f0 : 0.f) +
                                     (f1 != 0.f ? x_o[j * 128 + r] * f1 : 0.f));
          asm volatile("barrier.cta.sync 1, 256;" ::: "memory");
        }
        if (mine)
          for (uint32_t k = 0; k < odd.count; ++k)
            add_odd(t, odd.key0[k], odd.keys[k], x, from_key, to_key, o);
        if (mine && whole) {
#pragma unroll
          for (uint32_t v = 0; v < 4; ++v) {
            uint32_t y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
              y[j] = some ? pack2(__uint_as_float(o[8 * v + 2 * j]) * inv,
                                  __uint_as_float(o[8 * v + 2 * j + 1]) * inv, kBf16)
                          : 0u;
            *reinterpret_cast<uint4*>(chunk_at(lane, 4u * x + v)) =
                make_uint4(y[0], y[1], y[2], y[3]);
          }
        } else if (mine && live) {
          float* dst = &piece->o[32u * x][slot * kRows + r];
#pragma unroll
          for (int j = 0; j < 32; ++j) dst[j * kTileRows] = __uint_as_float(o[j]);
        }
      }
      if (mine && whole) {  // rows of the output, 16 lanes (or 8) each
        __syncwarp();
#pragma unroll 4
        for (uint32_t i = 0; i < kLd; ++i) {
          const uint32_t row = i * kPer + my_sub;
          const uint64_t to_row = __shfl_sync(0xFFFFFFFFu, live ? at : ~0ull, row);
          if (to_row != ~0ull && my_ch * 8u < a.g.D)
            *reinterpret_cast<uint4*>(a.out + (to_row * a.g.D + my_ch * 8u) * 2u) =
                *reinterpret_cast<const uint4*>(chunk_at(row, my_ch));
        }
        if (a.lse && live) a.lse[at] = some ? (base + log2f(l)) * 0.69314718056f : -INFINITY;
        __syncwarp();
      } else if (mine && live) {
        piece->m[slot * kRows + r] = base;
        piece->l[slot * kRows + r] = rowbad ? INFINITY : l;
      }
      tc_before();
    }
  }
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == 9)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u)
                 : "memory");
  if (tid == 0 && *s_fail) set_status(a.g.status, IBP_ETIMEOUT);
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
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_paged_chunk(const PagedAttnArgs& a, const PagedMaps& m, int sm_count,
                               cudaStream_t st) {
  const bool b = a.g.bf16 != 0u;
  if (a.g.D <= 64u)
    return b ? launch<64, true>(a, m, sm_count, st) : launch<64, false>(a, m, sm_count, st);
  return b ? launch<128, true>(a, m, sm_count, st) : launch<128, false>(a, m, sm_count, st);
}

cudaError_t launch_paged_chunk_join(const PagedAttnArgs& a, int sm_count, cudaStream_t st) {
  const bool b = a.g.bf16 != 0u;
  if (a.g.D <= 64u)
    return b ? launch_chunk_join<64, true>(a, sm_count, st) : launch_chunk_join<64, false>(a, sm_count, st);
  return b ? launch_chunk_join<128, true>(a, sm_count, st) : launch_chunk_join<128, false>(a, sm_count, st);
}

}  // namespace ibp
