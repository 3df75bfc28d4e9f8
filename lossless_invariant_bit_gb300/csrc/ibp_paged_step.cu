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
//     each CTA takes an equal run of it (one CTA per SM, two for small heads),
//     whatever the lengths.  A (sequence, head) whose run is cut is joined by a second
//     kernel from the pieces' maxima, sums and unscaled outputs, in the order of the
//     pieces, so that results do not depend on timing.
//   - A producer warp walks the list, looks pages up (32 boxes at a time, the next
//     ones while these load) and fills a ring of blocks in shared memory by TMA, a box
//     per page; it tells the others of each tile through shared memory.  Each of
//     the 4 other warps takes 32 keys of a block and waits for its mbarrier alone: no
//     barrier of the CTA within a tile.
//   - 16 rows are one left operand of mma.sync m16n8k16: at 16 rows the keys'
//     bytes, not the products, are the bound, and a 128-row tcgen05 tile would be
//     7/8 padding (the chunk kernel takes what has more rows).
//
// Measured: 20 sequences x 32 heads of 128 x 1984 keys in 104 us, 650 MB at 6.25 TB/s;
// one sequence of 517 keys 11 us, its look-ups, the first block and the join one
// after the other; lists of 128 pages of 16 for 16 tokens x 8 heads 32 us (134 MB at
// 4.2 TB/s: runs of 14 blocks are short beside the ring's start and the join).
#include "ibp_paged_step.cuh"
#include "ibp_tma.cuh"

namespace ibp {
namespace {

constexpr uint32_t kWarps = 4, kThreads = 32 * (kWarps + 1);

// Weights are rounded to 16 bits for the product with the values.  In fp16 they are 2^14
// times the formula's, the sum with them (the result does not change): the largest is
// 2^14, and what is 2^-28 of it still a normal number.  Unlifted, many keys of weights below
// 2^-14 beside one large one lose their bits, and below 2^-25 all of it.
template <bool kBf16>
constexpr int step_lift() {
  return kBf16 ? 0 : 14;
}

template <int kDP>
struct StepShape {
  static constexpr uint32_t kHalves = kDP / 64;
  static constexpr uint32_t kHalf = kBlock * 128u;             // 64 channels of a block
  static constexpr uint32_t kTile = kHalves * kHalf;           // keys (or values) of a block
  static constexpr uint32_t kStages = kDP == 64 ? 2u : 3u;
  static constexpr uint32_t kRing = kStages * 2u * kTile;
  static constexpr uint32_t kMerge = kWarps * 16u * (kDP + 4u) * 4u;
  static constexpr uint32_t kSmem = 1024u + kRing + kMerge + 256u;
};

template <int kDP, bool kBf16, bool kSel>
__global__ void __launch_bounds__(kThreads, kDP == 64 ? 2 : 1)
    k_paged_step(const __grid_constant__ CUtensorMap map_k,
                 const __grid_constant__ CUtensorMap map_v, PagedAttnArgs a) {
  using S = StepShape<kDP>;
  constexpr int kKs = kDP / 16;  // k-steps of a score, n-tile pairs of an output
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023u) & ~static_cast<uintptr_t>(1023u));
  __shared__ uint64_t s_scan[kWarps + 1];
  __shared__ uint64_t s_found[2];
  __shared__ uint32_t s_pos[S::kStages][16];  // first position of each box of a block
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
      mbar_init(full + i, 1);
      mbar_init(empty + i, kWarps);
    }
    for (uint32_t i = 0; i < kInfos; ++i) mbar_init(info_full + i, 1);
    s_fail = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  Run run = step_run<kSel, kThreads>(a, s_scan, s_found);
  Cursor& ld = run.ld;
  const uint64_t u0 = run.u0, u1 = run.u1;
  if (warp == kWarps) {
    // ---------------- producer
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
      const uint32_t count = tell_tile(a, run, u, more, s_info + tiles % kInfos,
                                       info_full + tiles % kInfos, join);
      ++tiles;
      __syncwarp();
      if (!more) break;
      // box `lane` of the group of blocks from b on: its first position, then its page
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
      uint32_t pos = pos_at(ld.blk);
      int32_t page = page_at(pos);
      uint32_t pos2 = pos_at(ld.blk + grp);
      for (uint32_t b = ld.blk; b < ld.blk + count && go; ++b, ++blocks) {
        const uint32_t in = (b - ld.blk) & (grp - 1u);  // which block of the group
        if (in == 0 && b != ld.blk) {
          pos = pos2;
          page = page_at(pos);
          pos2 = pos_at(b + grp);
        }
        const uint32_t st = blocks % S::kStages, round = blocks / S::kStages;
        if (round > 0) go = wait_or_fail(empty + st, (round - 1u) & 1u, &s_fail);
        if (!go) break;
        const bool mine = (lane >> per_lg) == in;
        const bool there = mine && pos != kNoPage;
        const bool bad = there && (page < 0 || (uint32_t)page >= a.g.n_pages);
        const uint32_t boxes = __popc(__ballot_sync(0xFFFFFFFFu, there && !bad));
        if (mine) s_pos[st][lane & ((1u << per_lg) - 1u)] = bad ? kBadPage : pos;
        __syncwarp();
        if (lane == 0) mbar_expect_tx(full + st, boxes * (2u * S::kHalves * 128u << box_lg));
        __syncwarp();
        if (there && !bad) {
          const uint32_t slot = lane & ((1u << per_lg) - 1u);
          uint8_t* k = smem + st * 2u * S::kTile + (slot << box_lg) * 128u;
#pragma unroll
          for (uint32_t hf = 0; hf < S::kHalves; ++hf) {
            tma_load_page(k + hf * S::kHalf, &map_k, full + st, 64u * hf,
                          pos & ((1u << lg) - 1u), ld.t.head, page);
            tma_load_page(k + S::kTile + hf * S::kHalf, &map_v, full + st, 64u * hf,
                          pos & ((1u << lg) - 1u), ld.t.head, page);
          }
        }
      }
      u += count;
    }
    end_join(run, join);
    if (lane == 0) joins[blockIdx.x] = join;
    // whosever wait gave up: the copies in flight land before the CTA leaves (or these
    // waits give up too)
    for (uint32_t i = blocks > S::kStages ? blocks - S::kStages : 0u; i < blocks; ++i)
      mbar_wait(full + i % S::kStages, (i / S::kStages) & 1u);
  } else {
    // ---------------- 32 keys of each block
    const uint32_t r0 = lane >> 2, quad = lane & 3u;
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
      uint32_t qf[kKs][4];
      float o[2 * kKs][4];
      float m[2], l[2];
      bool bad[2] = {false, false};  // rows that see a page that cannot be read
#pragma unroll
      for (int e = 0; e < 2; ++e) {  // the tile's queries, as the left operand
        const uint32_t r = r0 + 8u * e;
        const uint32_t tt = (row0 + r) / a.G, gg = (row0 + r) - tt * a.G;
        const uint8_t* src = a.q + (uint64_t)(t->q0 + tt) * a.q_stride +
                             ((uint64_t)t->head * a.G + gg) * a.g.D * 2u;
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
      for (uint32_t b = 0; b < count && go; ++b, ++blocks) {
        const uint32_t key0 = t->key0 + b * kBlock + warp * kWarpKeys;
        const uint32_t st = blocks % S::kStages;
        go = wait_or_fail(full + st, (blocks / S::kStages) & 1u, &s_fail);
        if (!go) break;
        const uint32_t kb = smem_addr(smem + st * 2u * S::kTile) + warp * kWarpKeys * 128u;
        const uint32_t vb = kb + S::kTile;
        // which of the 32 keys exist: a bit each
        uint32_t there;
        {
          const uint32_t at = warp * kWarpKeys + lane;
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
            for (int e = 0; e < 2; ++e) {  // those of its keys that the row sees
              const int32_t pos = (int32_t)(L - n + (row0 + r0 + 8u * e) / a.G);
              const int32_t end = kSel || !a.causal ? 32 : pos + 1 - (int32_t)key0;
              const int32_t from = a.window && pos >= (int32_t)a.window
                                       ? pos + 1 - (int32_t)a.window - (int32_t)key0
                                       : 0;
              const uint32_t below = end <= 0 ? 0u : end >= 32 ? ~0u : (1u << end) - 1u;
              const uint32_t above = from <= 0 ? ~0u : from >= 32 ? 0u : ~0u << from;
              bad[e] = bad[e] || (lost & below & above) != 0u;
            }
          }
        }
        if (there) {
          if (there != 0xFFFFFFFFu) {
            // rows of values that do not exist: zero, so that 0 * (what they hold) is 0
            for (uint32_t i = lane; i < kWarpKeys * S::kHalves * 8u; i += 32u) {
              const uint32_t row = i / 8u % kWarpKeys;
              if (!(there >> row & 1u)) {
                const uint32_t off = (i / (8u * kWarpKeys)) * S::kHalf + row * 128u + i % 8u * 16u;
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
              ldmatrix4(b, kb + (k >> 2) * S::kHalf + row * 128u + ((ch ^ (row & 7u)) << 4));
              mma_16816<kBf16>(sc[2 * i], qf[k], b[0], b[1]);
              mma_16816<kBf16>(sc[2 * i + 1], qf[k], b[2], b[3]);
            }
          }
          // ---- masks: what does not exist, and what lies beyond a row's position
          const bool partial =
              there != 0xFFFFFFFFu ||
              (!kSel && n > 1u && (key0 + kWarpKeys + n > L + 1u || a.window));
          if (partial) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint32_t tt = (row0 + r0 + 8u * e) / a.G;
              const int64_t pos = kSel ? 0x7FFFFFFF : (int64_t)L - n + tt;
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
            const float down = (float)step_lift<kBf16>() - base;
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float p0 = ex2(fmaf(sc[i][2 * e], a.scale_log2, down));
              const float p1 = ex2(fmaf(sc[i][2 * e + 1], a.scale_log2, down));
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
          if (!kSel && partial && n > 1u) {
            // Where only some rows see a key, infinities and NaN of its values go to those
            // rows alone, and become zero for the product.
            constexpr uint32_t kExp = kBf16 ? 0x7F80u : 0x7C00u;  // all ones: not finite
            bool found = false;
            for (uint32_t x = 0; x < S::kHalves * 8u; ++x) {
              uint32_t y[4];
              asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                           : "=r"(y[0]), "=r"(y[1]), "=r"(y[2]), "=r"(y[3])
                           : "r"(vb + (x >> 3) * S::kHalf + lane * 128u +
                                 (((x & 7u) ^ (lane & 7u)) << 4))
                           : "memory");
#pragma unroll
              for (int k = 0; k < 4; ++k)
                found = found || (y[k] & kExp) == kExp || (y[k] >> 16 & kExp) == kExp;
            }
            uint32_t odd = __ballot_sync(0xFFFFFFFFu, found);
            for (; odd; odd &= odd - 1u) {
              const uint32_t j = __ffs(odd) - 1u;
              bool see[2];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int64_t pos = (int64_t)L - n + (row0 + r0 + 8u * e) / a.G;
                const int64_t key = (int64_t)key0 + j;
                see[e] = (!a.causal || key <= pos) && (!a.window || key > pos - (int64_t)a.window);
              }
#pragma unroll
              for (int i = 0; i < 2 * kKs; ++i) {
                const uint32_t at = vb + (i >> 3) * S::kHalf + j * 128u +
                                    (((i & 7) ^ (j & 7u)) << 4) + quad * 4u;
                uint32_t y;
                asm volatile("ld.shared.b32 %0, [%1];" : "=r"(y) : "r"(at) : "memory");
                const bool bad0 = (y & kExp) == kExp, bad1 = (y >> 16 & kExp) == kExp;
                const float2 f = unpack2(y, kBf16);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  if (see[e] && bad0) o[i][2 * e] += f.x;
                  if (see[e] && bad1) o[i][2 * e + 1] += f.y;
                }
                __syncwarp();
                if (r0 == 0 && (bad0 || bad1))
                  asm volatile("st.shared.b32 [%0], %1;" ::"r"(at),
                               "r"((bad0 ? 0u : y & 0xFFFFu) | (bad1 ? 0u : y & 0xFFFF0000u))
                               : "memory");
              }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
          }
#pragma unroll
          for (int i = 0; i < 2; ++i)  // 16 keys at a time
#pragma unroll
            for (int k = 0; k < kKs; ++k) {
              uint32_t b[4];
              const uint32_t row = 16u * i + (lane & 15u);
              const uint32_t ch = 2u * (k & 3) + (lane >> 4);
              ldmatrix4_t(b, vb + (k >> 2) * S::kHalf + row * 128u + ((ch ^ (row & 7u)) << 4));
              mma_16816<kBf16>(o[2 * k], pf[i], b[0], b[1]);
              mma_16816<kBf16>(o[2 * k + 1], pf[i], b[2], b[3]);
            }
        }
        __syncwarp();  // every lane has read the block
        if (lane == 0) mbar_arrive(empty + st);
      }
      if (!go) bad[0] = bad[1] = true;
      // ---- end of the tile, or of this CTA's run: join the four warps
      float* mw = merge + warp * 16u * (kDP + 4u);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[e] += __shfl_xor_sync(0xFFFFFFFFu, l[e], 1);
        l[e] += __shfl_xor_sync(0xFFFFFFFFu, l[e], 2);
        float* row = mw + (r0 + 8u * e) * (kDP + 4u);
        if (quad == 0) row[kDP] = m[e], row[kDP + 1] = l[e], row[kDP + 2] = bad[e] ? 1.f : 0.f;
#pragma unroll
        for (int i = 0; i < 2 * kKs; ++i)
          *reinterpret_cast<float2*>(row + 8 * i + 2u * quad) =
              make_float2(o[i][2 * e], o[i][2 * e + 1]);
      }
      asm volatile("barrier.cta.sync 1, 128;" ::: "memory");
      merge_rows<kDP, kBf16, step_lift<kBf16>(), kWarps>(a, t, rows, merge, pieces);
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

template <int kDP, bool kBf16, bool kSel>
cudaError_t launch(const PagedAttnArgs& a, const PagedMaps& m, int sm_count, bool behind,
                   cudaStream_t st) {
  using S = StepShape<kDP>;
  auto kern = k_paged_step<kDP, kBf16, kSel>;
  cudaError_t e = smem_limit(reinterpret_cast<const void*>(kern), S::kSmem);
  if (e != cudaSuccess) return e;
  uint32_t ctas = (uint32_t)sm_count * (kDP == 64 ? 2u : 1u);
  if (ctas > kMaxCtas) ctas = kMaxCtas;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = behind ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, kern, m.k, m.v, a);
  if (e != cudaSuccess) return e;
  return launch_step_join<kDP, kBf16, step_lift<kBf16>()>(a, ctas, st);
}

}  // namespace

cudaError_t launch_paged_step(const PagedAttnArgs& a, const PagedMaps& m, int sm_count, bool behind,
                              cudaStream_t st) {
  const bool b = a.g.bf16 != 0u;
  if (a.selected) {
    if (a.g.D <= 64u)
      return b ? launch<64, true, true>(a, m, sm_count, behind, st)
               : launch<64, false, true>(a, m, sm_count, behind, st);
    return b ? launch<128, true, true>(a, m, sm_count, behind, st)
             : launch<128, false, true>(a, m, sm_count, behind, st);
  }
  if (a.g.D <= 64u)
    return b ? launch<64, true, false>(a, m, sm_count, behind, st)
             : launch<64, false, false>(a, m, sm_count, behind, st);
  return b ? launch<128, true, false>(a, m, sm_count, behind, st)
           : launch<128, false, false>(a, m, sm_count, behind, st);
}

}  // namespace ibp
