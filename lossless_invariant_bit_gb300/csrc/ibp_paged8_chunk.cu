// Attention of chunks of new tokens over a paged K/V cache of 8-bit codes, on the tensor
// cores.
//
//   S = Q K^T,  W = exp2(c S + b - m),  O += W V,  l += 2^-b W
//   k = 2^a code, v = 2^b code,  c = scale log2(e) 2^a: a, b the exponents of a key's page
//
// The tiles, the list of their blocks, the two slots of 128 rows that alternate, the issuing
// warps, the pieces and their join are those of the 16-bit pages' kernel
// (ibp_paged_chunk.cu).  What differs:
//
//   warps 12 - 15  fetch the codes of a block, 16 of a key at a time, straight into registers
//                  (keys and values in turn, one ring place ahead), convert them to fp16
//                  (exact) and store them as the tensor cores' swizzled operands.  What no
//                  row may see is not fetched, but zero
//   warp 8         walks the tiles, no more
//   scales         a page's codes are multiplied by its share of the block's scales (powers of
//                  two, exact) on the way; the block's keys' scale multiplies the rows' factor
//                  c, its values' goes into the exponent, and the sum takes 2^-b of it.  m
//                  refers to the largest c S + b, so W stays within fp16 however the
//                  blocks' scales differ
//   queries        fp16, or bf16 brought into its range by a power of two for each row (what that
//                  costs a score: ibp_paged8_step.cu)
//
// The products run in fp16, at the rate of bf16's: 8-bit products would need the queries and
// the weights in two or three parts each to keep their bits, and take as long.
//
// Measured: 2048 tokens of 8192, 64 query heads of 128 on 8, causal: 554 us, 0.87 PFLOP/s,
// bound by the conversions (every tile converts its keys again: about 3200 cycles a block of
// 128 keys against 2830 of products), which is why long chunks of bf16 go to the 16-bit
// pages' kernel, behind one conversion of their pages (k_paged8_stage).  24 sequences of up to
// 333 new tokens, heads of 64, with a window: 65 us of the batch's 82; no unit is full: of 116
// thousand cycles the rows' warps compute weights for 50 (2500 a block, exponentials 1050 of
// them) and wait 25 to 33 for scores, of keys whose conversion takes 2870 a block; queries, results
// and the run's start take 30.  Codes by TMA into tiles of their own, read from
// there: 513 us, but 92 for 78 where a batch is mixed: the products' operands come through
// the same memory.  Each page's scales in the rows' registers: 672.
#include "ibp_paged8.cuh"
#include "ibp_paged_chunk.cuh"
#include "ibp_tma.cuh"

namespace ibp {
namespace {

constexpr uint32_t kRing = 5, kThreads = 512;
// Blocks whose scales are kept: a block's are written when its keys' place in the ring is
// free, and then the weights of the third block before it are all computed.
constexpr uint32_t kAhead = 4;
constexpr uint32_t kInfos = 4;
// Weights are computed with a reference 2^11 below the largest, and rescaled when they pass
// 2^15: down to 2^-25 of the largest they are normal fp16 numbers.
constexpr float kLift = 11.f, kMost = 15.f;
// A block's codes times its pages' shares of its scales lie 2^7 below fp16's largest: exact for
// pages whose scales are down to 2^-22 of the block's.  A row's reference takes the block's
// scale of the values for that of its heaviest key, whose page may have a smaller one: the
// weights of keys in other blocks then lie lower by as much.  Lifted, fp16 holds them down to
// 2^-36 of the reference, so with values' scales down to 2^-11 of the block's nothing is
// lost above 2^-25 of the row's largest weight times scale.  A block whose pages differ by
// more is wide: its codes stay as they are, and its rows take each page's scales.
constexpr int32_t kUp = 7;
constexpr uint32_t kSpreadK = 22u, kSpreadV = 11u, kWide = 1u << 31;
// Keys whose weights are computed before the first half of them is handed over.
constexpr int kEarly = 80;

template <int kDP>
struct Shape8 {
  static constexpr uint32_t kHalves = kDP / 64;
  static constexpr uint32_t kHalf = 128u * 128u;  // 128 rows of 64 channels
  static constexpr uint32_t kTile = kHalves * kHalf;
  static constexpr uint32_t kSmall = 2048u;       // barriers and what the warps tell each other
  static constexpr uint32_t kSmem = 1024u + kSmall + (2u + kRing) * kTile;
};

// What lies before the tiles in shared memory.
struct Small {
  float4 scale[kAhead];      // of a block: keys' scale, values' exponent, 2^-exponent
  float2 page[kAhead][16];   // of a wide block's pages: keys' scale, values' exponent
  uint64_t scan[kThreads / 32 + 3];
  uint64_t full[kRing], empty[kRing], s_full[2], p_full[2], p2_full[2], turn[2], q_full, o_full;
  uint64_t done[2], info_full[kInfos], info_empty[kInfos];
  Info info[kInfos];
  int2 odd[kInfos];          // keys of a tile's run among which some values are NaN
  uint32_t bad[kAhead];      // bit per page that cannot be read, kWide
  uint32_t tmem, fail;
  uint8_t down[2 * kRows];   // exponents of the rows' powers of two
};
static_assert(sizeof(Small) <= Shape8<128>::kSmall, "it fits");

// The registers of the launch, shared out again: 8 warps of 176, 4 of 48 and 4 of 112 are the
// 16 of 128 that the launch came with.
__device__ __forceinline__ void reg_rows() { asm volatile("setmaxnreg.inc.sync.aligned.u32 176;"); }
__device__ __forceinline__ void reg_issue() { asm volatile("setmaxnreg.dec.sync.aligned.u32 48;"); }
__device__ __forceinline__ void reg_codes() { asm volatile("setmaxnreg.dec.sync.aligned.u32 112;"); }
static_assert(8 * 176 + 4 * 48 + 4 * 112 <= 16 * 128, "no more registers than the launch has");

// Loads, or zeros, without a branch: nothing waits for them before they are used.
__device__ __forceinline__ int32_t load_entry(const int32_t* p, bool there) {
  int32_t x;
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %2, 0;\n mov.b32 %0, 0;\n"
      " @p ld.global.nc.b32 %0, [%1];\n}\n"
      : "=&r"(x)
      : "l"(p), "r"((uint32_t)there));
  return x;
}
__device__ __forceinline__ uint32_t load_byte(const uint8_t* p, bool there) {
  uint32_t x;
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %2, 0;\n mov.b32 %0, 0;\n"
      " @p ld.global.nc.u8 %0, [%1];\n}\n"
      : "=&r"(x)
      : "l"(p), "r"((uint32_t)there));
  return x;
}
__device__ __forceinline__ uint4 load_codes(const uint8_t* p, bool there) {
  uint4 x;
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %5, 0;\n"
      " mov.b32 %0, 0;\n mov.b32 %1, 0;\n mov.b32 %2, 0;\n mov.b32 %3, 0;\n"
      " @p ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];\n}\n"
      : "=&r"(x.x), "=&r"(x.y), "=&r"(x.z), "=&r"(x.w)
      : "l"(p), "r"((uint32_t)there));
  return x;
}

// 2^e as fp16 (0 below its smallest), and two fp16 values times one.
__device__ __forceinline__ uint32_t fp16_power(int32_t e) {
  return e >= -14 ? (uint32_t)(min(e, kUp) + 15) << 10 : e >= -24 ? 1u << (e + 24) : 0u;
}
__device__ __forceinline__ uint32_t times2(uint32_t x, uint32_t f) {
  uint32_t y;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(f));
  return y;
}

// A warp's rows of the output times f.
__device__ __forceinline__ void rescale(uint32_t to, uint32_t D, float f) {
#pragma unroll 1
  for (uint32_t d = 0; 32u * d < D; ++d) {
    uint32_t o[32];
    tmem_ld32<0>(to + 32u * d, o);
    tmem_wait_ld(o);
#pragma unroll
    for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
    tmem_st32<0>(to + 32u * d, o);
  }
}

struct Sums {
  float m, base, l;
};

// The scores of a wide block, in place: each with its own page's scales, as exponents that need
// no factor; the reference moved to them, the sum added.  [from, to): the row's keys, of the
// block.  Rare, and a function: in the loop over the blocks its registers cost all of
// them 30 % of the kernel's time.
__device__ __noinline__ Sums wide_block(uint32_t ts, uint32_t to, uint32_t D, const float2* pages,
                                        uint32_t box_lg, uint32_t badp, float cr, int32_t from,
                                        int32_t end, bool any, Sums s) {
  float most = -INFINITY;
#pragma unroll 1
  for (int32_t q = 0; q < 128; q += 32) {
    uint32_t x[32];
    tmem_ld32<0>(ts + q, x);
    tmem_wait_ld(x);
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      const int32_t key = q + j;
      const uint32_t page = (uint32_t)key >> box_lg;
      const float2 p = pages[page];
      const bool see = key >= from && key < end && !(badp >> page & 1u);
      const float v = see ? fmaf(__uint_as_float(x[j]), row_factor(cr, p.x), p.y) : -INFINITY;
      most = fmaxf(most, v);
      x[j] = __float_as_uint(v);
    }
    tmem_st32<0>(ts + q, x);
  }
  tmem_wait_st();
  s.m = fmaxf(s.m, most);
  const bool none = s.l == 0.f;
  if (__any_sync(0xFFFFFFFFu, s.m > s.base + kMost || (none && s.m != -INFINITY))) {
    const float nb = none && s.m != -INFINITY ? s.m - kLift : fmaxf(s.m - kLift, s.base);
    const float f = none ? 1.f : ex2(s.base - nb);
    s.base = nb;
    s.l *= f;
    if (any) rescale(to, D, f);
  }
  // the block's sum by itself: many equal weights added to a long sum are all rounded one way
  float l[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
  for (int32_t q = 0; q < 128; q += 32) {
    uint32_t x[32];
    tmem_ld32<0>(ts + q, x);
    tmem_wait_ld(x);
#pragma unroll
    for (int j = 0; j < 32; ++j)
      l[j & 3] = fmaf(ex2(__uint_as_float(x[j]) - s.base),
                      ex2(-pages[(uint32_t)(q + j) >> box_lg].y), l[j & 3]);
  }
  s.l += (l[0] + l[1]) + (l[2] + l[3]);
  return s;
}

template <int kDP, bool kBf16>
__global__ void __launch_bounds__(kThreads, 1) k_paged8_chunk(PagedAttnArgs a) {
  using S = Shape8<kDP>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023u) & ~static_cast<uintptr_t>(1023u));
  Small& sm = *reinterpret_cast<Small*>(smem);
  uint8_t* s_q = smem + S::kSmall;       // 2 slots of queries
  uint8_t* s_kv = s_q + 2u * S::kTile;   // the ring: K, V, K, V, ...
  uint64_t *full = sm.full, *empty = sm.empty, *s_full = sm.s_full, *p_full = sm.p_full;
  uint64_t *p2_full = sm.p2_full, *q_full = &sm.q_full, *o_full = &sm.o_full;
  uint64_t *info_full = sm.info_full, *info_empty = sm.info_empty;
  uint32_t *s_fail = &sm.fail, *s_bad = sm.bad;
  uint8_t* s_down = sm.down;
  int2* s_odd = sm.odd;

  const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31u;
  Piece<kDP>* pieces = reinterpret_cast<Piece<kDP>*>(a.ws + kStepWsBytes);
  Join* joins = reinterpret_cast<Join*>(a.ws + IBP_PAGED_WORKSPACE_BYTES -
                                        kMaxCtas * sizeof(Join));
  if (tid == 0) {
    for (uint32_t i = 0; i < kRing; ++i) {
      mbar_init(full + i, 4);
      mbar_init(empty + i, 2);
    }
    for (uint32_t i = 0; i < 2; ++i) {
      mbar_init(s_full + i, 1);
      mbar_init(p_full + i, 5);
      mbar_init(p2_full + i, 4);
      mbar_init(sm.turn + i, 1);
      mbar_init(sm.done + i, 1);
    }
    for (uint32_t i = 0; i < kInfos; ++i) {
      mbar_init(info_full + i, 1);
      mbar_init(info_empty + i, 8);
    }
    mbar_init(q_full, 8);
    mbar_init(o_full, 2);
    sm.fail = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (tid == 0) mbar_arrive(sm.turn);  // slot 0 begins
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(&sm.tmem)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // what comes behind may take the SMs that have ended (it waits for this grid itself)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  uint64_t total;
  uint32_t ctas;
  const Walk w0 = chunk_run<kThreads>(a, sm.scan, sm.scan + kThreads / 32, total, ctas);
  const uint32_t tmem = sm.tmem;
  // the tile of number t, once its run is known; false: no more, or given up
  auto info_of = [&](uint32_t t) -> const Info* {
    const Info* x = sm.info + t % kInfos;
    if (!wait_or_fail(info_full + t % kInfos, (t / kInfos) & 1u, s_fail)) return nullptr;
    return x->count ? x : nullptr;
  };

  if (warp == 8) {
    reg_issue();
    // ---------------- the walk
    bool go = true;
    Walk w = w0;
    Join join{};
    for (uint32_t tiles = 0; go; ++tiles) {
      const bool more = walk(a, w);
      if (tiles >= kInfos)
        go = wait_or_fail(info_empty + tiles % kInfos, (tiles / kInfos - 1u) & 1u, s_fail);
      if (!go) break;
      if (lane == 0) {
        s_odd[tiles % kInfos] = make_int2(0x7FFFFFFF, 0);
        tell_run(a, w, total, ctas, more, sm.info + tiles % kInfos, info_full + tiles % kInfos,
                 join);
      }
      __syncwarp();
      if (!more) break;
    }
    if (lane == 0) joins[blockIdx.x] = join;
  } else if (warp == 9 || warp == 10) {
    reg_issue();
    const Bars bars{full, empty, s_full, p_full, p2_full, sm.turn, q_full, o_full, sm.done};
    issue_products<S, kDP, false, kRing>(a, warp - 9u, tmem, s_q, s_kv, bars, s_fail, info_of);
  } else if (warp == 11) {
    reg_issue();
    // ---------------- keys and values are there: one arrival with each block's weights
    uint32_t e0 = 0, pn[2] = {0, 0};
    bool go = true;
    auto entry = [&](uint32_t e) {
      go = go && wait_or_fail(full + e % kRing, (e / kRing) & 1u, s_fail);
    };
    for (uint32_t tiles = 0; go; ++tiles) {
      const Info* t = info_of(tiles);
      if (!t) break;
      const uint32_t nb = t->count, two = t->two, step = two ? 2u : 1u;
      for (uint32_t i = 0; i < nb && go; ++i) {
        entry(e0 + 2u * i + 1u);                             // these values
        if (i + step < nb) entry(e0 + 2u * (i + step));      // the slot's next keys
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
  } else if (warp >= 12) {
    reg_codes();
    // ---------------- 32 keys of a block: codes to fp16.  A lane's key is one of 8, its
    // channels 16 of 64 (so that 8 lanes' stores meet no bank twice).
    constexpr uint32_t kH = kDP / 64, kLoads = 4 * kH;
    const uint32_t cw = warp - 12u, r8 = lane & 7u, ch = lane >> 3;
    const uint32_t lg = a.g.page_lg, box_lg = lg < 7u ? lg : 7u;
    const uint32_t dst = smem_addr(s_kv) + (cw * 32u + r8) * 128u;
    const uint32_t off0 = ((2u * ch) ^ r8) << 4;  // (the other half: its neighbour)
    const bool lower = ch * 16u < a.g.D, upper = 64u + ch * 16u < a.g.D;
    uint32_t e = 0, blocks = 0, seen;
    uint64_t off[4];
    bool go = true;
    for (uint32_t tiles = 0; go; ++tiles) {
      const Info* t = info_of(tiles);
      if (!t) break;
      const uint32_t head = t->head;
      const int32_t lo = (int32_t)t->lo, hi = (int32_t)t->hi;
      const uint8_t* kp = a.g.k + head * a.g.head_stride + ch * 16u;
      const uint8_t* vp = a.g.v + head * a.g.head_stride + ch * 16u;
      // Lane i looks up page i of a block: its entry two blocks ahead, its scales one.
      const int32_t* table = a.b.table + t->s * a.b.table_stride;
      auto needed = [&](int32_t k0) {
        const int32_t key = k0 + (int32_t)(lane << box_lg);
        return lane < kKeys >> box_lg && key < hi && key + (1 << box_lg) > lo;
      };
      auto entry_at = [&](int32_t k0) {
        const int32_t key = k0 + (int32_t)(lane << box_lg);
        return load_entry(table + ((uint32_t)key >> lg), needed(k0));
      };
      // -1: not needed, -2: out of range
      auto id_of = [&](int32_t entry, int32_t k0) {
        return !needed(k0) ? -1 : (uint32_t)entry >= a.g.n_pages ? -2 : entry;
      };
      auto scale_at = [&](const uint8_t* scales, int32_t id) {
        return load_byte(scales + (uint64_t)(uint32_t)id * a.g.H + head, id >= 0);
      };
      // Where this lane's keys of the block from k0 on lie (keys 8 g of the warp's 32), and
      // which of them some row sees.
      auto locate = [&](int32_t ids, int32_t k0) {
        seen = 0;
#pragma unroll
        for (uint32_t g = 0; g < 4; ++g) {
          const uint32_t first = cw * 32u + 8u * g;
          const int32_t id = __shfl_sync(0xFFFFFFFFu, ids, first >> box_lg);
          const int32_t key = k0 + (int32_t)(first + r8);
          off[g] = (uint64_t)(uint32_t)id * a.g.page_stride +
                   ((uint32_t)key & ((1u << lg) - 1u)) * a.g.token_stride;
          if (id >= 0 && key >= lo && key < hi) seen |= 1u << g;
        }
      };
      auto fetch = [&](const uint8_t* from, uint32_t k) {
        return load_codes(from + off[k / kH] + 64u * (k % kH),
                          (seen >> (k / kH) & 1u) && (k % kH ? upper : lower));
      };
      auto store = [&](const uint4& x, uint32_t at, uint32_t k, uint32_t f) {
        at += (k % kH) * S::kHalf + (k / kH) * 1024u;
        uint32_t y[4];
        codes_to_fp16(x.x, y[0], y[1]);
        codes_to_fp16(x.y, y[2], y[3]);
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = times2(y[i], f);
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + off0), "r"(y[0]),
                     "r"(y[1]), "r"(y[2]), "r"(y[3]));
        codes_to_fp16(x.z, y[0], y[1]);
        codes_to_fp16(x.w, y[2], y[3]);
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = times2(y[i], f);
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + (off0 ^ 16u)), "r"(y[0]),
                     "r"(y[1]), "r"(y[2]), "r"(y[3]));
      };
      auto place = [&]() {  // the next one of the ring is free
        if (e >= kRing) go = go && wait_or_fail(empty + e % kRing, (e / kRing - 1u) & 1u, s_fail);
        return go;
      };
      auto hand = [&]() {
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(full + e % kRing);
        ++e;
      };
      int32_t key0 = (int32_t)t->key0;
      const int32_t all = key0 + (int32_t)(t->count * kKeys);  // keys of the run end here
      int32_t ids = id_of(entry_at(key0), key0);
      int32_t entry = key0 + (int32_t)kKeys < all ? entry_at(key0 + (int32_t)kKeys) : 0;
      uint32_t ks = scale_at(a.g.k_scales, ids), vs = scale_at(a.g.v_scales, ids);
      // The block's scales are the largest of its pages'; a page's codes are multiplied by what
      // its own are of them: keys' factor, values' factor, as fp16.
      uint32_t k_top, v_top, bad;
      bool fine, wide;
      auto powers_of = [&]() {
        fine = ids >= 0 && scale_ok(ks) && scale_ok(vs);
        bad = __ballot_sync(0xFFFFFFFFu, ids != -1 && !fine);
        k_top = __reduce_max_sync(0xFFFFFFFFu, fine ? ks : kScaleLow);
        v_top = __reduce_max_sync(0xFFFFFFFFu, fine ? vs : kScaleLow);
        wide = __any_sync(0xFFFFFFFFu, fine && (k_top - ks > kSpreadK || v_top - vs > kSpreadV));
        return wide ? 0x3C003C00u
                    : fp16_power((int32_t)(ks - k_top) + kUp) |
                          fp16_power((int32_t)(vs - v_top) + kUp) << 16;
      };
      uint4 x[kLoads], y[kLoads];
      locate(ids, key0);
#pragma unroll
      for (uint32_t k = 0; k < kLoads; ++k) x[k] = fetch(kp, k);
      for (; key0 < all; ++blocks, key0 += (int32_t)kKeys) {
        const int32_t key1 = key0 + (int32_t)kKeys, key2 = key1 + (int32_t)kKeys;
        const int32_t next = key1 < all ? id_of(entry, key1) : -1;
        if (key2 < all) entry = entry_at(key2);
        const uint32_t ks1 = scale_at(a.g.k_scales, next), vs1 = scale_at(a.g.v_scales, next);
        const uint32_t powers = powers_of();
        uint32_t power[4];
#pragma unroll
        for (uint32_t g = 0; g < 4; ++g)
          power[g] = __shfl_sync(0xFFFFFFFFu, powers, (cw * 32u + 8u * g) >> box_lg);
#pragma unroll
        for (uint32_t k = 0; k < kLoads; ++k) y[k] = fetch(vp, k);
        if (!place()) break;
        if (cw == 0 && lane == 0) {
          sm.scale[blocks % kAhead] =
              make_float4(scale_of(k_top - kUp), (float)((int32_t)v_top - 127 - kUp),
                          scale_of(254u + kUp - v_top), 0.f);
          s_bad[blocks % kAhead] = bad | (wide ? kWide : 0u);
        }
        if (wide && cw == 0 && lane < 16u)
          sm.page[blocks % kAhead][lane] =
              fine ? make_float2(scale_of(ks), (float)((int32_t)vs - 127)) : make_float2(1.f, 0.f);
        const uint32_t at_k = dst + (e % kRing) * S::kTile;
#pragma unroll
        for (uint32_t k = 0; k < kLoads; ++k)
          store(x[k], at_k, k, __byte_perm(power[k / kH], 0u, 0x1010));
        hand();
        ids = next, ks = ks1, vs = vs1;
        locate(ids, key1);
#pragma unroll
        for (uint32_t k = 0; k < kLoads; ++k) x[k] = fetch(kp, k);
        if (!place()) break;
        const uint32_t at_v = dst + (e % kRing) * S::kTile;
        // Where only some rows see a key, NaN of its values become zero, and go to the rows that
        // see them at the tile's end.
        const bool mixed = key1 > (int32_t)t->all_hi || key0 < (int32_t)t->all_lo;
        if (mixed || bad) {
#pragma unroll
          for (uint32_t k = 0; k < kLoads; ++k) {
            const uint32_t first = cw * 32u + 8u * (k / kH);
            if (bad >> (first >> box_lg) & 1u) y[k] = make_uint4(0u, 0u, 0u, 0u);
            if (mixed && (nan_codes(y[k].x) | nan_codes(y[k].y) | nan_codes(y[k].z) |
                          nan_codes(y[k].w))) {
              y[k].x &= ~((nan_codes(y[k].x) >> 7) * 0xFFu);
              y[k].y &= ~((nan_codes(y[k].y) >> 7) * 0xFFu);
              y[k].z &= ~((nan_codes(y[k].z) >> 7) * 0xFFu);
              y[k].w &= ~((nan_codes(y[k].w) >> 7) * 0xFFu);
              atomicMin(&s_odd[tiles % kInfos].x, key0 + (int32_t)(first + r8));
              atomicMax(&s_odd[tiles % kInfos].y, key0 + (int32_t)(first + r8) + 1);
            }
          }
        }
#pragma unroll
        for (uint32_t k = 0; k < kLoads; ++k)
          store(y[k], at_v, k, __byte_perm(power[k / kH], 0u, 0x3232));
        hand();
      }
    }
  } else {
    reg_rows();
    // ---------------- a slot's rows: thread = row
    const uint32_t slot = warp >> 2, wq = warp & 3u, r = wq * 32u + lane;
    const uint32_t lane_base = (wq * 32u) << 16;
    const uint32_t ts = tmem + lane_base + slot * 128u, to = tmem + lane_base + 256u + slot * 128u;
    const uint32_t box_lg = a.g.page_lg < 7u ? a.g.page_lg : 7u;
    // This warp's 32 rows of the slot's queries in shared memory, 16 bytes at a
    // time; between two tiles they hold the rows of the output.
    constexpr uint32_t kCh = kDP / 8u, kPer = 32u / kCh, kLd = 32u / kPer;
    uint8_t* s_rows = s_q + slot * S::kTile + wq * 32u * 128u;
    const uint32_t my_ch = lane % kCh, my_sub = lane / kCh;
    auto chunk_at = [&](uint32_t row, uint32_t ch) {
      return s_rows + (ch >> 3) * S::kHalf + row * 128u + (((ch & 7u) ^ (row & 7u)) << 4);
    };
    // The tile's queries: lane i knows where row i lies, 16 (or 8) lanes fetch a row.  bf16 ones
    // become fp16 under a power of two for each row, whose exponent is kept.
    auto load_q = [&](const Info* t) {
      const uint32_t n = t->two ? (slot ? 0u : t->rows)
                                : (t->rows > slot * kRows ? t->rows - slot * kRows : 0u);
      if (!t->two || slot == 0) {
        const uint32_t R = t->row0 + slot * kRows + (r < n ? r : 0u), tok = R / a.G;
        const uint64_t p = reinterpret_cast<uint64_t>(
            a.q + (uint64_t)(t->q0 + tok) * a.q_stride +
            (uint64_t)(t->head * a.G + (R - tok * a.G)) * a.g.D * 2u);
        if (kBf16) {
#pragma unroll 4
          for (uint32_t i = 0; i < kLd; ++i) {
            const uint32_t row = i * kPer + my_sub;
            const uint64_t src = __shfl_sync(0xFFFFFFFFu, p, row) + my_ch * 16u;
            uint4 x = make_uint4(0u, 0u, 0u, 0u);
            if (wq * 32u + row < n && my_ch * 8u < a.g.D)
              x = __ldg(reinterpret_cast<const uint4*>(src));
            uint32_t top = max(max(bf16_top(x.x), bf16_top(x.y)), max(bf16_top(x.z), bf16_top(x.w)));
#pragma unroll
            for (uint32_t d = 1; d < kCh; d <<= 1)
              top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
            const Lift lift = row_lift(top);
            *reinterpret_cast<uint4*>(chunk_at(row, my_ch)) =
                make_uint4(bf16_to_fp16(x.x, lift.up), bf16_to_fp16(x.y, lift.up),
                           bf16_to_fp16(x.z, lift.up), bf16_to_fp16(x.w, lift.up));
            if (my_ch == 0) s_down[slot * kRows + wq * 32u + row] = lift.byte;
          }
        } else {
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
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
    };
    // NaN among the values of the keys [from, to) that this row sees, into 32 channels of its
    // sums: rare, and read again from the pages.
    auto add_odd = [&](const Info* t, int32_t from, int32_t to, uint32_t x, uint32_t (&o)[32]) {
#pragma unroll 1
      for (int32_t key = from; key < to; ++key) {
        const int32_t page =
            __ldg(a.b.table + t->s * a.b.table_stride + ((uint32_t)key >> a.g.page_lg));
        if ((uint32_t)page >= a.g.n_pages) continue;
        const uint32_t* v = reinterpret_cast<const uint32_t*>(
            a.g.v + (uint64_t)(uint32_t)page * a.g.page_stride + t->head * a.g.head_stride +
            ((uint32_t)key & ((1u << a.g.page_lg) - 1u)) * a.g.token_stride + 32u * x);
#pragma unroll
        for (int d = 0; d < 8; ++d)
          if (32u * x + 4u * d < a.g.D) {
            const uint32_t nan = nan_codes(__ldg(v + d));
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (nan >> (8 * k + 7) & 1u) o[4 * d + k] = 0x7FFFFFFFu;
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
      // running maximum of scores + exponents of the values' scales, reference, sum
      float m = -INFINITY, base = 0.f, l = 0.f;
      float cr = a.scale_log2;  // the row's factor of the scores
      bool rowbad = false;
      bool any = false;  // a product has been accumulated
      if (both) key0 += (int32_t)(slot * kKeys);
      for (uint32_t i = both ? slot : 0u; i < count; i += both ? 2u : 1u) {
        go = wait_or_fail(s_full + slot, sn++ & 1u, s_fail);
        if (!go) break;
        tc_after();
        if (kBf16 && i < 2u)  // (behind the scores that were computed of them)
          cr = a.scale_log2 * scale_of(s_down[(both ? 0u : slot * kRows) + r]);
        float4 scale = sm.scale[(blocks + i) % kAhead];
        const uint32_t badp = s_bad[(blocks + i) % kAhead] & ~kWide;
        const bool wide = (s_bad[(blocks + i) % kAhead] & kWide) != 0u;
        if (wide) {
          const Sums x = wide_block(ts, to, a.g.D, sm.page[(blocks + i) % kAhead], box_lg, badp, cr,
                                    from_key - key0, to_key - key0, any, Sums{m, base, l});
          m = x.m, base = x.base, l = x.l;
          scale.y = scale.z = 0.f;
        }
        uint32_t sv[128];
        tmem_ld32<0>(ts, sv);
        tmem_ld32<32>(ts + 32u, sv);
        tmem_ld32<64>(ts + 64u, sv);
        tmem_ld32<96>(ts + 96u, sv);
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
        auto mask = [&](const int g) {
          const uint32_t v = seen(key0 + 32 * g);
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (!(v >> j & 1u)) sv[32 * g + j] = 0xFF800000u;
        };
        if (masked)
#pragma unroll
          for (int g = 0; g < 4; ++g) mask(g);
        // The weights need a reference, not the maximum: they are computed with the one
        // at hand while the maximum is found, and again in the rare block whose
        // maximum has outgrown it.
        const float c = wide ? 1.f : row_factor(cr, scale.x);
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
          w2[(j & 63) / 2] = pack2(p0, p1, 0u);
          w2[(j & 63) / 2 + 1] = pack2(p2, p3, 0u);
        };
        uint32_t pa[32], pb[32];
        b2 = pair2(scale.y - base, scale.y - base);
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
        m = fmaxf(m, fmaf(fmaxf(max3(x[0], x[1], x[2]), x[3]), c, scale.y));
        const bool none = l == 0.f;  // this row has seen no key: any reference will do
        if (__any_sync(0xFFFFFFFFu, m > base + kMost || (none && m != -INFINITY))) {
          const float nb = none && m != -INFINITY ? m - kLift : fmaxf(m - kLift, base);
          const float f = none ? 1.f : ex2(base - nb);
          base = nb;
          l *= f;
          // every product issued so far is done (the scores came after it)
          if (any) rescale(to, a.g.D, f);
          b2 = pair2(scale.y - base, scale.y - base);
          l0 = l1 = 0;
          // (the scores are read once more: kept, they would cost 64 registers in every block)
          tmem_ld32<0>(ts, sv);
          tmem_ld32<32>(ts + 32u, sv);
          tmem_wait_ld(sv);
          if (masked) mask(0), mask(1);
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
          l = fmaf(u + v, scale.z, l);
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
      const int32_t odd_from = s_odd[(tiles - 1u) % kInfos].x;
      const int32_t odd_to = s_odd[(tiles - 1u) % kInfos].y;
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
        if (mine) add_odd(t, max(odd_from, from_key), min(odd_to, to_key), x, o);
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
      __syncwarp();
      if (lane == 0) mbar_arrive(info_empty + (tiles - 1u) % kInfos);
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
cudaError_t launch(const PagedAttnArgs& a, int sm_count, cudaStream_t st) {
  using S = Shape8<kDP>;
  auto kern = k_paged8_chunk<kDP, kBf16>;
  const cudaError_t e = smem_limit(reinterpret_cast<const void*>(kern), S::kSmem);
  if (e != cudaSuccess) return e;
  const uint32_t ctas = (uint32_t)sm_count < kMaxCtas ? (uint32_t)sm_count : kMaxCtas;
  kern<<<ctas, kThreads, S::kSmem, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged8_chunk(const PagedAttnArgs& a, const PagedMaps&, int sm_count,
                                cudaStream_t st) {
  const bool b = a.g.bf16 != 0u;
  if (a.g.D <= 64u) return b ? launch<64, true>(a, sm_count, st) : launch<64, false>(a, sm_count, st);
  return b ? launch<128, true>(a, sm_count, st) : launch<128, false>(a, sm_count, st);
}

cudaError_t launch_paged8_chunk_join(const PagedAttnArgs& a, int sm_count, cudaStream_t st) {
  const bool b = a.g.bf16 != 0u;
  if (a.g.D <= 64u)
    return b ? launch_chunk_join<64, true>(a, sm_count, st)
             : launch_chunk_join<64, false>(a, sm_count, st);
  return b ? launch_chunk_join<128, true>(a, sm_count, st)
           : launch_chunk_join<128, false>(a, sm_count, st);
}

}  // namespace ibp
