// Attention of few rows over a paged K/V cache of 8-bit codes: the step of sequences that
// are being answered, and tokens that attend to a list of pages each.
//
//   out = sum_j p_j v_j / sum_j p_j,   p_j = exp(scale q.k_j - m)
//   k_j = 2^a code, v_j = 2^b code,    a, b the exponents of j's page and head
//
// The list of blocks of 128 keys, its equal runs for each CTA and the join of cut tiles are
// those of the 16-bit pages' kernel (ibp_paged_step.cuh).  What differs:
//
//   - Everything is transposed: keys (for the scores) and channels (for the sums) are the
//     rows of the matrix instructions, a tile's queries their 8 columns, two of them for
//     9 to 16.  Queries by rows waste half of each product on the 8 and fewer that a K/V
//     head has here: 75.5 us for 20 sequences of 1984 tokens, 32 heads of 128, where this takes
//     63.
//   - Codes become fp16 on their way from shared memory to the matrix units, one conversion
//     for two (every e4m3 number is an fp16 number); the products run in fp16 with fp32
//     sums whatever the type of the queries.  bf16 queries are brought into fp16's range
//     by a power of two for each row: 8 bits of each survive down to 2^-28 of the row's
//     largest, below that they are off by up to 2^-39 of it.  A score is then off by up to
//     scale 2^-39 max|q| sum|k|: below fp32's rounding of its sum, but where the keys are
//     zero or tiny in the channels in which the row is large.
//   - A page's scales never touch an element.  That of its keys multiplies the row's factor of
//     the scores; that of its values goes into the exponent, w_j = exp2(s_j + b - m), where m is
//     a reference at most 2^15 below the largest s_j + b: weights and values are then
//     products that need no scale however the pages' scales differ, and the sum takes
//     p_j = 2^-b w_j (8 keys in a row share a page).  With exponents in [-50, 50] neither can
//     leave fp32 before it has left the result.
//   - Transposed loads fetch two channels of a key as one 16-bit element, so the two
//     halves of a byte permutation are the operands of the even and the odd channels.
//
// Bound by HBM where there is enough to read: 325.5 MB of 325.1 MB in 63 us (20 x 1984 tokens),
// of which about 10 are the start, the last blocks and the join; 5.9 TB/s between them.  Page
// lists: 16 tokens x 128 pages of 16 in 23 us, 120 tokens x 24 pages of 32 (each token's pages
// are its own copies, 93 MB from L2) in 26.  One sequence of 517 tokens: 9.5 us, look-ups.
#include "ibp_paged_step.cuh"
#include "ibp_paged8.cuh"
#include "ibp_tma.cuh"

namespace ibp {
namespace {

// Weights are computed with a reference 2^11 below the largest, which moves (and what is
// summed with it) when they pass 2^15: what is 2^-25 of the largest is a normal fp16 number.
constexpr float kLift = 11.f, kMost = 15.f;

// kNT: tiles of 8 rows, 1 or 2.  Two groups of four computing warps take the blocks in turn; one
// warp loads keys, one values.  (Four groups hold four blocks of the ring and leave none to
// be on their way: 80 us for 66.)
template <int kDP, int kNT>
struct StepShape8 {
  static constexpr uint32_t kGroups = 2u, kWarps = 4u * kGroups;
  static constexpr uint32_t kThreads = 32u * (kWarps + 2u);
  static constexpr uint32_t kTile = kBlock * kDP;  // keys (or values) of a block, rows of kDP bytes
  // (kInfos - 2 at most: see Info)
  static constexpr uint32_t kStages = kDP == 128 && kNT == 2 ? 4u : 6u;
  // A place of the ring is always the same group's: a wait for a barrier's phase tells it from the
  // one before, not from the one before that.
  static_assert(kStages % kGroups == 0 && kStages <= kInfos - 2u, "");
  static constexpr uint32_t kRing = kStages * 2u * kTile;
  static constexpr uint32_t kRow = kDP + 4u;       // a row's floats in the warps' sums
  static constexpr uint32_t kSums = 8u * kNT * kRow;
  static constexpr uint32_t kMerge = 4u * kSums * 4u;  // a group's: the other's are added first
  static constexpr uint32_t kSmem = 1024u + kRing + kMerge + 256u;
};

// An 8 x 8 matrix of 16-bit values, two to a lane, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Four warps' rows of a tile (or of this CTA's run of it), joined: the result, or a piece of it.
// A thread takes channels d, d + kThreads, ... of all rows together, so that few rows are
// written by all warps too.
template <typename S, int kDP, bool kBf16>
__device__ __forceinline__ void merge_rows8(const PagedAttnArgs& a, const Info* t, uint32_t rows,
                                            const float* merge, Piece<kDP>* pieces) {
  Piece<kDP>* piece = pieces + 2u * blockIdx.x + t->place;
  for (uint32_t i = threadIdx.x; i < rows * kDP; i += 32u * S::kWarps) {
    const uint32_t r = i / kDP, d = i % kDP;
    const float* src = merge + r * S::kRow;
    float m[4], top = -INFINITY, l = 0.f, o = 0.f;
    bool bad = false;
#pragma unroll
    for (uint32_t w = 0; w < 4u; ++w) {
      const float* s = src + w * S::kSums + kDP;
      m[w] = s[0];
      top = fmaxf(top, m[w]);
      bad = bad || s[2] != 0.f;
    }
    const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
    for (uint32_t w = 0; w < 4u; ++w) {
      const float* s = src + w * S::kSums;
      const float f = ex2(m[w] - base);
      l = fmaf(f, s[kDP + 1], l);
      o = fmaf(f, s[d], o);
    }
    if (bad) l = INFINITY;  // a row that could not be read: zero, here or when joined
    if (t->whole) {
      const bool some = !bad && l != 0.f;
      const uint32_t R = t->row0 + r;
      const uint64_t at = ((uint64_t)(t->q0 + R / a.G) * a.g.H + t->head) * a.G + R % a.G;
      if (d < a.g.D)
        reinterpret_cast<uint16_t*>(a.out)[at * a.g.D + d] =
            (uint16_t)pack2(some ? o * (1.f / l) : 0.f, 0.f, kBf16);
      if (a.lse && d == 0) a.lse[at] = some ? (top + log2f(l)) * 0.69314718056f : -INFINITY;
    } else {
      piece->o[r][d] = o;
      if (d == 0) piece->m[r] = top, piece->l[r] = l;
    }
  }
}

template <int kDP, bool kBf16, bool kSel, int kNT>
__global__ void __launch_bounds__(StepShape8<kDP, kNT>::kThreads, 1)
    k_paged8_step(const __grid_constant__ CUtensorMap map_k,
                  const __grid_constant__ CUtensorMap map_v, PagedAttnArgs a) {
  using S = StepShape8<kDP, kNT>;
  constexpr int kKs = kDP / 16;  // k-steps of a score, 16-channel chunks of an output
  constexpr uint32_t kWarps = S::kWarps, kThreads = S::kThreads, kGroups = S::kGroups;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023u) & ~static_cast<uintptr_t>(1023u));
  __shared__ uint64_t s_scan[kThreads / 32];
  __shared__ uint64_t s_found[2];
  __shared__ uint32_t s_pos[S::kStages][16];  // first position of each box of a block
  __shared__ float2 s_scale[S::kStages][16];  // its page's keys' scale, values' exponent
  __shared__ Info s_info[kInfos];
  __shared__ uint32_t s_fail;
  const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31u, tid = threadIdx.x;
  float* merge = reinterpret_cast<float*>(smem + S::kRing);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::kRing + S::kMerge);
  uint64_t* empty = full + S::kStages;
  uint64_t* info_full = empty + S::kStages;
  Piece<kDP>* pieces = reinterpret_cast<Piece<kDP>*>(a.ws);
  Join* joins = reinterpret_cast<Join*>(a.ws + kStepWsBytes - kMaxCtas * sizeof(Join));

  if (tid == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_k)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_v)) : "memory");
    for (uint32_t i = 0; i < S::kStages; ++i) {
      mbar_init(full + i, 2);
      mbar_init(empty + i, kWarps / kGroups);
    }
    for (uint32_t i = 0; i < kInfos; ++i) mbar_init(info_full + i, 1);
    s_fail = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  Run run = step_run<kSel, kThreads>(a, s_scan, s_found);
  Cursor& ld = run.ld;
  const uint64_t u0 = run.u0, u1 = run.u1;
  if (warp >= kWarps) {
    // ---------------- producers: of the keys (which tells the others of the tiles, and of
    // the boxes of each block), of the values
    const bool keys = warp == kWarps;
    const CUtensorMap* map = keys ? &map_k : &map_v;
    const uint32_t lg = a.g.page_lg, box_lg = lg < 7u ? lg : 7u;
    const uint32_t per_lg = 7u - box_lg;        // boxes of a block
    const uint32_t grp = 32u >> per_lg;         // blocks whose boxes are looked up together
    Join join{};
    uint32_t blocks = 0, tiles = 0;
    bool go = true;
    uint64_t u = u0;
    for (bool first = true;; first = false) {
      const bool more = u < u1 && go;
      if (more && !first) {
        next_tile<kSel>(a, ld);
        run.tile_u = u;
      }
      uint32_t count = 0;
      if (keys)
        count = tell_tile(a, run, u, more, s_info + tiles % kInfos, info_full + tiles % kInfos,
                          join);
      else if (more)
        count = u1 - u < ld.t.nb - ld.blk ? (uint32_t)(u1 - u) : ld.t.nb - ld.blk;
      ++tiles;
      __syncwarp();
      if (!more) break;
      // box `lane` of the group of blocks from b on: its first position, its page, the
      // page's scales
      auto pos_at = [&](uint32_t b) {
        const uint32_t key = (ld.t.b0 + b) * kBlock + (lane << box_lg);
        if (b + (lane >> per_lg) >= ld.blk + count) return kNoPage;
        if (!kSel)
          return key >= ld.t.L || key + (1u << box_lg) <= ld.t.lo ? kNoPage : key;
        const uint32_t at = key >> lg;
        if (at >= a.n_sel) return kNoPage;
        const int32_t v = __ldg(ld.t.sel + at);
        if (v < 0 || ld.t.L == 0 || (uint32_t)v > (ld.t.L - 1u) >> lg) return kNoPage;
        const uint32_t p = ((uint32_t)v << lg) + (key & ((1u << lg) - 1u));
        return p >= ld.t.L ? kNoPage : p;
      };
      auto page_at = [&](uint32_t pos) {
        return pos == kNoPage ? -1 : __ldg(ld.t.table + (pos >> lg));
      };
      auto scales_at = [&](int32_t page) {
        return keys && (uint32_t)page < a.g.n_pages
                   ? page_scales(a.g, (uint32_t)page, ld.t.head)
                   : 0u;
      };
      uint32_t pos = pos_at(ld.blk);
      int32_t page = page_at(pos);
      uint32_t pos2 = pos_at(ld.blk + grp);
      uint32_t scales = scales_at(page);
      int32_t page2 = page_at(pos2);
      for (uint32_t b = ld.blk; b < ld.blk + count && go; ++b, ++blocks) {
        const uint32_t in = (b - ld.blk) & (grp - 1u);  // which block of the group
        if (in == 0 && b != ld.blk) {
          pos = pos2;
          page = page2;
          pos2 = pos_at(b + grp);
          scales = scales_at(page);
          page2 = page_at(pos2);
        }
        const uint32_t st = blocks % S::kStages, round = blocks / S::kStages;
        if (round > 0) go = wait_or_fail(empty + st, (round - 1u) & 1u, &s_fail);
        if (!go) break;
        const bool mine = (lane >> per_lg) == in;
        const bool there = mine && pos != kNoPage;
        const bool held = there && (uint32_t)page < a.g.n_pages;
        const uint32_t slot = lane & ((1u << per_lg) - 1u);
        const uint32_t boxes = __popc(__ballot_sync(0xFFFFFFFFu, held));
        if (held)
          tma_load_page(smem + (2u * st + (keys ? 0u : 1u)) * S::kTile + (slot << box_lg) * kDP, map,
                        full + st, 0u, pos & ((1u << lg) - 1u), ld.t.head, page);
        // (the scales are looked at once the copies are on their way)
        if (mine && keys) {
          const bool fine = held && scales_ok(scales);
          s_pos[st][slot] = there && !fine ? kBadPage : pos;
          s_scale[st][slot] =
              fine ? make_float2(scale_of(scales & 0xFFu), (float)((int32_t)(scales >> 8) - 127))
                   : make_float2(1.f, 0.f);
        }
        __syncwarp();
        if (lane == 0) mbar_expect_tx(full + st, boxes * ((uint32_t)kDP << box_lg));
        __syncwarp();
      }
      u += count;
    }
    end_join(run, join);
    if (keys && lane == 0) joins[blockIdx.x] = join;
    // whosever wait gave up: the copies in flight land before the CTA leaves (or these
    // waits give up too)
    for (uint32_t i = blocks > S::kStages ? blocks - S::kStages : 0u; i < blocks; ++i)
      mbar_wait(full + i % S::kStages, (i / S::kStages) & 1u);
  } else {
    // ---------------- 32 keys of every kGroups-th block
    const uint32_t group = warp / 4u, wk = warp % 4u;
    const uint32_t g = lane >> 2, quad = lane & 3u;
    const uint32_t box_lg = a.g.page_lg < 7u ? a.g.page_lg : 7u;
    uint32_t blocks = 0;
    bool go = true;
    for (uint32_t tiles = 0;; ++tiles) {
      const Info* t = s_info + tiles % kInfos;
      // a wait that gives up ends the tile like any other: the warps meet at its end,
      // and leave together
      go = wait_or_fail(info_full + tiles % kInfos, (tiles / kInfos) & 1u, &s_fail);
      const uint32_t count = go ? t->count : 0u;
      const uint32_t rows = count ? t->rows : 0u, row0 = t->row0, n = t->n, L = t->L, lo = t->lo;
      // The tile's queries are the right operand, row 8 x + g of them a lane's, its 4 channels of
      // each 16 those that it gets of a key.  Of the scores, and of the sums, it has rows
      // 8 x + 2 quad + e: index 2 x + e.
      uint32_t qf[kNT][kKs][2];
      float o[kKs][kNT][4];
      float m[2 * kNT], l[2 * kNT], cr[2 * kNT];
      bool bad[2 * kNT];  // rows that see a page that cannot be read
#pragma unroll
      for (int x = 0; x < kNT; ++x) {
        const uint32_t r = 8u * x + g;
        const uint32_t tt = (row0 + r) / a.G, gg = (row0 + r) - tt * a.G;
        const uint8_t* src = a.q + (uint64_t)(t->q0 + tt) * a.q_stride +
                             ((uint64_t)t->head * a.G + gg) * a.g.D * 2u;
#pragma unroll
        for (int k = 0; k < kKs; ++k) {
          const uint32_t d = 16u * k + 4u * quad;
          const uint2 v = r < rows && d < a.g.D ? __ldg(reinterpret_cast<const uint2*>(src + d * 2u))
                                                : make_uint2(0u, 0u);
          qf[x][k][0] = v.x, qf[x][k][1] = v.y;
        }
        float factor = a.scale_log2;
        if (kBf16) {
          uint32_t top = 0;
#pragma unroll
          for (int k = 0; k < kKs; ++k)
            top = max(top, max(bf16_top(qf[x][k][0]), bf16_top(qf[x][k][1])));
          top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
          top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
          const Lift lift = row_lift(top);
          factor *= lift.down;
#pragma unroll
          for (int k = 0; k < kKs; ++k) {
            qf[x][k][0] = bf16_to_fp16(qf[x][k][0], lift.up);
            qf[x][k][1] = bf16_to_fp16(qf[x][k][1], lift.up);
          }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          cr[2 * x + e] = __shfl_sync(0xFFFFFFFFu, factor, 8u * quad + 4u * e);
          m[2 * x + e] = -INFINITY;
          l[2 * x + e] = 0.f;
          bad[2 * x + e] = false;
        }
#pragma unroll
        for (int k = 0; k < kKs; ++k) o[k][x][0] = o[k][x][1] = o[k][x][2] = o[k][x][3] = 0.f;
      }
      for (uint32_t b = 0; b < count && go; ++b, ++blocks) {
        if (blocks % kGroups != group) continue;
        const uint32_t key0 = t->key0 + b * kBlock + wk * kWarpKeys;
        const uint32_t st = blocks % S::kStages;
        go = wait_or_fail(full + st, (blocks / S::kStages) & 1u, &s_fail);
        if (!go) break;
        const uint32_t kb = smem_addr(smem + st * 2u * S::kTile) + wk * kWarpKeys * kDP;
        const uint32_t vb = kb + S::kTile;
        // the position of row index i's token
        auto pos_of = [&](int i) {
          return (int32_t)(L - n + (row0 + 8u * (i >> 1) + 2u * quad + (i & 1)) / a.G);
        };
        // which of the 32 keys exist: a bit each
        uint32_t there;
        {
          const uint32_t at = wk * kWarpKeys + lane;
          const uint32_t first = s_pos[st][at >> box_lg];
          const uint32_t key = first + (at & ((1u << box_lg) - 1u));
          there = __ballot_sync(0xFFFFFFFFu, first < kBadPage && key < L && key >= lo);
          const uint32_t own = key0 + lane;  // (without a page list)
          const uint32_t lost =
              there == 0xFFFFFFFFu
                  ? 0u
                  : __ballot_sync(0xFFFFFFFFu,
                                  first == kBadPage && (kSel || (own < L && own >= lo)));
          if (lost) {
            if (lane == 0) set_status(a.g.status, IBP_ERANGE);
#pragma unroll
            for (int i = 0; i < 2 * kNT; ++i) {  // those of its keys that the row sees
              const int32_t pos = pos_of(i);
              const int32_t end = kSel || !a.causal ? 32 : pos + 1 - (int32_t)key0;
              const int32_t from = a.window && pos >= (int32_t)a.window
                                       ? pos + 1 - (int32_t)a.window - (int32_t)key0
                                       : 0;
              const uint32_t below = end <= 0 ? 0u : end >= 32 ? ~0u : (1u << end) - 1u;
              const uint32_t above = from <= 0 ? ~0u : from >= 32 ? 0u : ~0u << from;
              bad[i] = bad[i] || (lost & below & above) != 0u;
            }
          }
        }
        if (there) {
          if (there != 0xFFFFFFFFu) {
            // rows of values that do not exist: zero, so that 0 * (what they hold) is 0
            for (uint32_t i = lane; i < kWarpKeys * kKs; i += 32u) {
              const uint32_t row = i / kKs;
              if (!(there >> row & 1u))
                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                                 vb + row * kDP + i % kKs * 16u),
                             "r"(0u)
                             : "memory");
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
          }
          // Scores, keys by rows: of keys 16 y + 8 h + g, h = 0 and 1, at [y][x][2 h + e].
          float sc[2][kNT][4];
#pragma unroll
          for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int x = 0; x < kNT; ++x) sc[y][x][0] = sc[y][x][1] = sc[y][x][2] = sc[y][x][3] = 0.f;
#pragma unroll
          for (int c = 0; c < kKs / 4; ++c) {  // 64 channels
            uint32_t w[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i)  // 8 keys
              ldmatrix4(w[i], kb + code_chunk<kDP>(8u * i + (lane & 7u), 4u * c + (lane >> 3)));
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                uint32_t f[4];
                codes_to_fp16(w[2 * y][k], f[0], f[2]);
                codes_to_fp16(w[2 * y + 1][k], f[1], f[3]);
#pragma unroll
                for (int x = 0; x < kNT; ++x)
                  mma_16816<false>(sc[y][x], f, qf[x][4 * c + k][0], qf[x][4 * c + k][1]);
              }
          }
          // ---- masks: what does not exist, and what lies beyond a row's position
          const bool partial =
              there != 0xFFFFFFFFu ||
              (!kSel && n > 1u && (key0 + kWarpKeys + n > L + 1u || a.window));
          if (partial) {
#pragma unroll
            for (int i = 0; i < 2 * kNT; ++i) {
              const int64_t pos = kSel ? 0x7FFFFFFF : pos_of(i);
              const int64_t from = a.window ? pos - a.window : -1;
#pragma unroll
              for (int y = 0; y < 2; ++y)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const uint32_t j = 16u * y + 8u * h + g;
                  const int64_t key = (int64_t)key0 + j;
                  const bool see = (there >> j & 1u) &&
                                   (kSel || ((!a.causal || key <= pos) && key > from));
                  if (!see) sc[y][i >> 1][2 * h + (i & 1)] = -INFINITY;
                }
            }
          }
          // ---- the reference, where it has to move; weights and their sum
          float ks[4], lv[4], iv[4];  // of the page of keys 8i .. 8i + 7
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 s = s_scale[st][(wk * kWarpKeys + 8u * i) >> box_lg];
            ks[i] = s.x;
            lv[i] = s.y;
            iv[i] = __uint_as_float((uint32_t)(127 - (int32_t)s.y) << 23);
          }
          float most[2 * kNT];
          bool more = false;
#pragma unroll
          for (int i = 0; i < 2 * kNT; ++i) {
            most[i] = -INFINITY;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              float& s = sc[k >> 1][i >> 1][2 * (k & 1) + (i & 1)];
              s = fmaf(s, row_factor(cr[i], ks[k]), lv[k]);
              most[i] = fmaxf(most[i], s);
            }
            more = more || most[i] > m[i] + kMost;  // (-inf for a row that has seen no key)
          }
          if (__any_sync(0xFFFFFFFFu, more)) {
#pragma unroll
            for (int i = 0; i < 2 * kNT; ++i) {
#pragma unroll
              for (int d = 4; d < 32; d <<= 1)
                most[i] = fmaxf(most[i], __shfl_xor_sync(0xFFFFFFFFu, most[i], d));
              const float to = fmaxf(m[i], most[i] - kLift);
              const float f = to == -INFINITY ? 1.f : ex2(m[i] - to);
              m[i] = to;
              l[i] *= f;
#pragma unroll
              for (int k = 0; k < kKs; ++k) {
                o[k][i >> 1][i & 1] *= f;
                o[k][i >> 1][2 + (i & 1)] *= f;
              }
            }
          }
          uint32_t pf[2][kNT][2];
#pragma unroll
          for (int x = 0; x < kNT; ++x) {
            const float b0 = m[2 * x] == -INFINITY ? 0.f : m[2 * x];
            const float b1 = m[2 * x + 1] == -INFINITY ? 0.f : m[2 * x + 1];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float p0 = ex2(sc[k >> 1][x][2 * (k & 1)] - b0);
              const float p1 = ex2(sc[k >> 1][x][2 * (k & 1) + 1] - b1);
              l[2 * x] = fmaf(p0, iv[k], l[2 * x]);
              l[2 * x + 1] = fmaf(p1, iv[k], l[2 * x + 1]);
              pf[k >> 1][x][k & 1] = transpose8(pack2(p0, p1, 0u));
            }
          }
          if (!kSel && partial && n > 1u) {
            // Where only some rows see a key, NaN of its values go to those rows alone, and
            // become zero for the product.
            uint32_t hit = 0;
#pragma unroll
            for (uint32_t x = 0; x < kKs; ++x) {
              uint32_t y[4];
              asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                           : "=r"(y[0]), "=r"(y[1]), "=r"(y[2]), "=r"(y[3])
                           : "r"(vb + code_chunk<kDP>(lane, x))
                           : "memory");
#pragma unroll
              for (int k = 0; k < 4; ++k) hit |= nan_codes(y[k]);
            }
            uint32_t odd = __ballot_sync(0xFFFFFFFFu, hit != 0u);
            for (; odd; odd &= odd - 1u) {
              const uint32_t j = __ffs(odd) - 1u;
              const int64_t key = (int64_t)key0 + j;
#pragma unroll
              for (int k = 0; k < kKs; ++k) {
                const uint32_t at = vb + code_chunk<kDP>(j, k) + 2u * g;
                uint16_t y;
                asm volatile("ld.shared.u16 %0, [%1];" : "=h"(y) : "r"(at) : "memory");
                const uint32_t nan = nan_codes(y) & 0x8080u;
#pragma unroll
                for (int i = 0; i < 2 * kNT; ++i) {
                  const int64_t pos = pos_of(i);
                  if ((a.causal && key > pos) || (a.window && key <= pos - (int64_t)a.window))
                    continue;
                  if (nan & 0x80u) o[k][i >> 1][i & 1] = NAN;
                  if (nan & 0x8000u) o[k][i >> 1][2 + (i & 1)] = NAN;
                }
                __syncwarp();
                if (quad == 0 && nan)
                  asm volatile("st.shared.u16 [%0], %1;" ::"r"(at),
                               "h"((uint16_t)(y & ~((nan >> 7) * 0xFFu)))
                               : "memory");
              }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
          }
          // ---- values by rows: of channels 16 k + 2 g + h at [k][x][2 h + e]
#pragma unroll
          for (int y = 0; y < 2; ++y)  // 16 keys at a time
#pragma unroll
            for (int k = 0; k < kKs; k += 2) {
              uint32_t w[4];
              const uint32_t row = 16u * y + (lane & 15u);
              ldmatrix4_t(w, vb + code_chunk<kDP>(row, k + (lane >> 4)));
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                // two keys' even channel, their odd one
                uint32_t f[4];
                codes_to_fp16(__byte_perm(w[2 * j], 0u, 0x3120), f[0], f[1]);
                codes_to_fp16(__byte_perm(w[2 * j + 1], 0u, 0x3120), f[2], f[3]);
#pragma unroll
                for (int x = 0; x < kNT; ++x)
                  mma_16816<false>(o[k + j][x], f, pf[y][x][0], pf[y][x][1]);
              }
            }
        }
        __syncwarp();  // every lane has read the block
        if (lane == 0) mbar_arrive(empty + st);
      }
      // ---- end of the tile, or of this CTA's run: join the groups, then the warps
      float* mw = merge + wk * S::kSums;
#pragma unroll
      for (int i = 0; i < 2 * kNT; ++i) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], d);
        if (!go) bad[i] = true;
      }
      if (group == 1) {  // as it lies in the registers
        if (g == 0)
#pragma unroll
          for (int i = 0; i < 2 * kNT; ++i) {
            float* s = mw + 8 * kNT * kDP + (4 * i + quad) * 3;
            s[0] = m[i], s[1] = l[i], s[2] = bad[i] ? 1.f : 0.f;
          }
#pragma unroll
        for (int k = 0; k < kKs; ++k)
#pragma unroll
          for (int x = 0; x < kNT; ++x)
            *reinterpret_cast<float4*>(mw + ((k * kNT + x) * 32u + lane) * 4u) =
                make_float4(o[k][x][0], o[k][x][1], o[k][x][2], o[k][x][3]);
      }
      asm volatile("barrier.cta.sync 1, %0;" ::"n"(32u * kWarps) : "memory");
      if (group == 0) {
        float f0[2 * kNT], f1[2 * kNT];
#pragma unroll
        for (int i = 0; i < 2 * kNT; ++i) {
          const float* s = mw + 8 * kNT * kDP + (4 * i + quad) * 3;
          const float top = fmaxf(m[i], s[0]), base = top == -INFINITY ? 0.f : top;
          f0[i] = ex2(m[i] - base);
          f1[i] = ex2(s[0] - base);
          m[i] = top;
          l[i] = l[i] * f0[i] + s[1] * f1[i];
          bad[i] = bad[i] || s[2] != 0.f;
        }
#pragma unroll
        for (int k = 0; k < kKs; ++k)
#pragma unroll
          for (int x = 0; x < kNT; ++x) {
            const float4 y = *reinterpret_cast<const float4*>(mw + ((k * kNT + x) * 32u + lane) * 4u);
            o[k][x][0] = o[k][x][0] * f0[2 * x] + y.x * f1[2 * x];
            o[k][x][1] = o[k][x][1] * f0[2 * x + 1] + y.y * f1[2 * x + 1];
            o[k][x][2] = o[k][x][2] * f0[2 * x] + y.z * f1[2 * x];
            o[k][x][3] = o[k][x][3] * f0[2 * x + 1] + y.w * f1[2 * x + 1];
          }
        __syncwarp();  // read by every lane before any writes its rows
#pragma unroll
        for (int i = 0; i < 2 * kNT; ++i) {
          const uint32_t r = 8u * (i >> 1) + 2u * quad + (i & 1);
          if (r >= rows) continue;
          float* row = mw + r * S::kRow;
          if (g == 0) row[kDP] = m[i], row[kDP + 1] = l[i], row[kDP + 2] = bad[i] ? 1.f : 0.f;
#pragma unroll
          for (int k = 0; k < kKs; ++k)
            *reinterpret_cast<float2*>(row + 16 * k + 2u * g) =
                make_float2(o[k][i >> 1][i & 1], o[k][i >> 1][2 + (i & 1)]);
        }
      }
      asm volatile("barrier.cta.sync 1, %0;" ::"n"(32u * kWarps) : "memory");
      merge_rows8<S, kDP, kBf16>(a, t, rows, merge, pieces);
      // the sums have been read: the next tile may write its own
      if (any_of<kWarps>(!go || count == 0)) break;
    }
  }
  __syncthreads();
  if (tid == 0 && s_fail) set_status(a.g.status, IBP_ETIMEOUT);
  // launched behind the chunk kernel of the same call, it ends after it: what follows
  // this kernel may count on both
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <int kDP, bool kBf16, bool kSel, int kNT>
cudaError_t launch(const PagedAttnArgs& a, const PagedMaps& m, int sm_count, bool behind,
                   cudaStream_t st) {
  using S = StepShape8<kDP, kNT>;
  auto kern = k_paged8_step<kDP, kBf16, kSel, kNT>;
  cudaError_t e = smem_limit(reinterpret_cast<const void*>(kern), S::kSmem);
  if (e != cudaSuccess) return e;
  const uint32_t ctas = (uint32_t)sm_count < kMaxCtas ? (uint32_t)sm_count : kMaxCtas;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, 1, 1);
  cfg.blockDim = dim3(S::kThreads, 1, 1);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = behind ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, kern, m.k, m.v, a);
  if (e != cudaSuccess) return e;
  return launch_step_join<kDP, kBf16, 0>(a, ctas, st);
}

template <int kDP, bool kBf16>
cudaError_t launch_rows(const PagedAttnArgs& a, const PagedMaps& m, int sm_count, bool behind,
                        cudaStream_t st) {
  // Rows of a tile, at most: the queries of a token's head, of a sequence's tokens.  One tile
  // of 8 halves the products and leaves room for six blocks on their way.  One tile and two,
  // us: 20 x 1984 tokens, one query to a head, 62.9 and 76.4; 1 x 517 10.9 and 13.3; lists of 16
  // tokens 24.1 and 27.0, of 120 tokens 26.9 and 33.1.
  const bool few = a.G * (a.selected ? 1ull : a.b.max_q) <= 8u;
  if (a.selected)
    return few ? launch<kDP, kBf16, true, 1>(a, m, sm_count, behind, st)
               : launch<kDP, kBf16, true, 2>(a, m, sm_count, behind, st);
  return few ? launch<kDP, kBf16, false, 1>(a, m, sm_count, behind, st)
             : launch<kDP, kBf16, false, 2>(a, m, sm_count, behind, st);
}

}  // namespace

cudaError_t launch_paged8_step(const PagedAttnArgs& a, const PagedMaps& m, int sm_count,
                               bool behind, cudaStream_t st) {
  const bool b = a.g.bf16 != 0u;
  if (a.g.D <= 64u)
    return b ? launch_rows<64, true>(a, m, sm_count, behind, st)
             : launch_rows<64, false>(a, m, sm_count, behind, st);
  return b ? launch_rows<128, true>(a, m, sm_count, behind, st)
           : launch_rows<128, false>(a, m, sm_count, behind, st);
}

}  // namespace ibp
