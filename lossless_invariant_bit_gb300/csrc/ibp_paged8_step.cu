// Attention of few rows over a paged K/V cache of 8-bit codes: the step of sequences that
// are being answered, and tokens that attend to a list of pages each.
//
//   out = sum_j p_j v_j / sum_j p_j,   p_j = exp(scale q.k_j - m)
//   k_j = 2^a code, v_j = 2^b code,    a, b the exponents of j's page and head
//
// The list of blocks, the ring, the warps' parts and the join are those of the 16-bit
// pages' kernel (ibp_paged_step.cu); a block holds half the bytes.  What differs:
//
//   - Codes become fp16 on their way from shared memory to the matrix units, one conversion
//     for two (every e4m3 number is an fp16 number); the products run in fp16 with fp32
//     sums whatever the type of the queries.  bf16 queries are brought into fp16's range
//     by a power of two for each row: 8 bits of each survive down to 2^-28 of the row's
//     largest, below that they lose bits that no score can show (2^-39 of it is dropped).
//   - A page's scales never touch an element.  That of its keys multiplies the row's factor of
//     the scores; that of its values goes into the exponent, w_j = exp2(s_j + b - m), where m is
//     the running maximum of s_j + b: weights and values are then products that need no
//     scale, w_j <= 2^kLift however the pages' scales differ, and the sum takes
//     p_j = 2^-b w_j, once for 8 keys (8 keys in a row share a page).  With exponents in
//     [-50, 50] neither can leave fp32 before it has left the result.
//   - Transposed loads fetch two channels of a key as one 16-bit element, so the two
//     halves of a byte permutation are the operands of the even and the odd channels.
#include "ibp_paged_step.cuh"
#include "ibp_paged8.cuh"
#include "ibp_tma.cuh"

namespace ibp {
namespace {

// Weights are 2^14 times the formula's, the sum with them: the largest is 2^14, what is
// 2^-28 of it still a normal fp16 number.
constexpr int kLift = 14;

template <int kDP>
struct StepShape8 {
  static constexpr uint32_t kTile = kBlock * kDP;  // keys (or values) of a block, rows of kDP bytes
  static constexpr uint32_t kStages = 5u;
  static constexpr uint32_t kRing = kStages * 2u * kTile;
  static constexpr uint32_t kMerge = kWarps * 16u * (kDP + 4u) * 4u;
  static constexpr uint32_t kSmem = 1024u + kRing + kMerge + 256u;
};

template <int kDP, bool kBf16, bool kSel>
__global__ void __launch_bounds__(kThreads, kDP == 64 ? 2 : 1)
    k_paged8_step(const __grid_constant__ CUtensorMap map_k,
                  const __grid_constant__ CUtensorMap map_v, PagedAttnArgs a) {
  using S = StepShape8<kDP>;
  constexpr int kKs = kDP / 16;  // k-steps of a score, 16-channel chunks of an output
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023u) & ~static_cast<uintptr_t>(1023u));
  __shared__ uint64_t s_scan[kWarps + 1];
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
      mbar_init(full + i, 1);
      mbar_init(empty + i, kWarps);
    }
    for (uint32_t i = 0; i < kInfos; ++i) mbar_init(info_full + i, 1);
    s_fail = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  Run run = step_run<kSel>(a, s_scan, s_found);
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
        return (uint32_t)page < a.g.n_pages ? page_scales(a.g, (uint32_t)page, ld.t.head) : 0u;
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
        if (held) {
          uint8_t* k = smem + st * 2u * S::kTile + (slot << box_lg) * kDP;
          const uint32_t token = pos & ((1u << lg) - 1u);
          tma_load_page(k, &map_k, full + st, 0u, token, ld.t.head, page);
          tma_load_page(k + S::kTile, &map_v, full + st, 0u, token, ld.t.head, page);
        }
        // (the scales are looked at once the copies are on their way)
        if (mine) {
          const bool fine = held && scales_ok(scales);
          s_pos[st][slot] = there && !fine ? kBadPage : pos;
          s_scale[st][slot] =
              fine ? make_float2(scale_of(scales & 0xFFu), (float)((int32_t)(scales >> 8) - 127))
                   : make_float2(1.f, 0.f);
        }
        __syncwarp();
        if (lane == 0) mbar_expect_tx(full + st, boxes * (2u * kDP << box_lg));
        __syncwarp();
      }
      u += count;
    }
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
      float m[2], l[2], cr[2];
      bool bad[2] = {false, false};  // rows that see a page that cannot be read
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        // The tile's queries, as the left operand: a lane's 4 channels of each 16 are those
        // that it gets of a key.
        const uint32_t r = r0 + 8u * e;
        const uint32_t tt = (row0 + r) / a.G, gg = (row0 + r) - tt * a.G;
        const uint8_t* src = a.q + (uint64_t)(t->q0 + tt) * a.q_stride +
                             ((uint64_t)t->head * a.G + gg) * a.g.D * 2u;
        uint2 x[kKs];
#pragma unroll
        for (int k = 0; k < kKs; ++k) {
          const uint32_t d = 16u * k + 4u * quad;
          x[k] = r < rows && d < a.g.D ? __ldg(reinterpret_cast<const uint2*>(src + d * 2u))
                                       : make_uint2(0u, 0u);
        }
        cr[e] = a.scale_log2;
        if (kBf16) {
          uint32_t top = 0;
#pragma unroll
          for (int k = 0; k < kKs; ++k) top = max(top, max(bf16_top(x[k].x), bf16_top(x[k].y)));
          top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
          top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
          const Lift lift = row_lift(top);
          cr[e] *= lift.down;
#pragma unroll
          for (int k = 0; k < kKs; ++k) {
            x[k].x = bf16_to_fp16(x[k].x, lift.up);
            x[k].y = bf16_to_fp16(x[k].y, lift.up);
          }
        }
#pragma unroll
        for (int k = 0; k < kKs; ++k) qf[k][e] = x[k].x, qf[k][e + 2] = x[k].y;
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
        const uint32_t kb = smem_addr(smem + st * 2u * S::kTile) + warp * kWarpKeys * kDP;
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
          float sc[4][4];
#pragma unroll
          for (int i = 0; i < 4; ++i) sc[i][0] = sc[i][1] = sc[i][2] = sc[i][3] = 0.f;
          // keys 8i .. 8i + 7, 64 channels for each load
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int h = 0; h < kKs / 4; ++h) {
              uint32_t x[4];
              const uint32_t row = 8u * i + (lane & 7u);
              ldmatrix4(x, kb + code_chunk<kDP>(row, 4u * h + (lane >> 3)));
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                uint32_t b0, b1;
                codes_to_fp16(x[k], b0, b1);
                mma_16816<false>(sc[i], qf[4 * h + k], b0, b1);
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
          float ks[4], lv[4], iv[4];  // of the page of keys 8i .. 8i + 7
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 s = s_scale[st][(warp * kWarpKeys + 8u * i) >> box_lg];
            ks[i] = s.x;
            lv[i] = s.y;
            iv[i] = __uint_as_float((uint32_t)(127 - (int32_t)s.y) << 23);
          }
          uint32_t pf[2][4];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float c[4], mx = -INFINITY;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              c[i] = row_factor(cr[e], ks[i]);
              mx = fmaxf(mx, fmaf(fmaxf(sc[i][2 * e], sc[i][2 * e + 1]), c[i], lv[i]));
            }
            mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
            mx = fmaxf(m[e], mx);
            const float base = mx == -INFINITY ? 0.f : mx;
            const float f = ex2(m[e] - base);
            m[e] = mx;
            const float down = (float)kLift - base;
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float p0 = ex2(fmaf(sc[i][2 * e], c[i], lv[i] + down));
              const float p1 = ex2(fmaf(sc[i][2 * e + 1], c[i], lv[i] + down));
              sum = fmaf(p0 + p1, iv[i], sum);
              pf[i >> 1][e + 2 * (i & 1)] = pack2(p0, p1, 0u);
            }
            l[e] = l[e] * f + sum;
#pragma unroll
            for (int i = 0; i < 2 * kKs; ++i) {
              o[i][2 * e] *= f;
              o[i][2 * e + 1] *= f;
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
              bool see[2];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int64_t pos = (int64_t)L - n + (row0 + r0 + 8u * e) / a.G;
                const int64_t key = (int64_t)key0 + j;
                see[e] = (!a.causal || key <= pos) && (!a.window || key > pos - (int64_t)a.window);
              }
#pragma unroll
              for (int i = 0; i < kKs; ++i) {
                const uint32_t at = vb + code_chunk<kDP>(j, i) + quad * 4u;
                uint32_t y;
                asm volatile("ld.shared.b32 %0, [%1];" : "=r"(y) : "r"(at) : "memory");
                const uint32_t nan = nan_codes(y);
#pragma unroll
                for (int c = 0; c < 4; ++c)  // channel 16 i + 4 quad + c
                  if (nan >> (8 * c + 7) & 1u) {
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                      if (see[e]) o[2 * i + (c & 1)][2 * e + (c >> 1)] = NAN;
                  }
                __syncwarp();
                if (r0 == 0 && nan)
                  asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(y & ~((nan >> 7) * 0xFFu))
                               : "memory");
              }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
          }
#pragma unroll
          for (int i = 0; i < 2; ++i)  // 16 keys at a time
#pragma unroll
            for (int k = 0; k < kKs; k += 2) {
              uint32_t x[4];
              const uint32_t row = 16u * i + (lane & 15u);
              ldmatrix4_t(x, vb + code_chunk<kDP>(row, k + (lane >> 4)));
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                // two keys' even channel, their odd one
                uint32_t e0, e1, d0, d1;
                codes_to_fp16(__byte_perm(x[2 * j], 0u, 0x3120), e0, d0);
                codes_to_fp16(__byte_perm(x[2 * j + 1], 0u, 0x3120), e1, d1);
                mma_16816<false>(o[2 * (k + j)], pf[i], e0, e1);
                mma_16816<false>(o[2 * (k + j) + 1], pf[i], d0, d1);
              }
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
        for (int i = 0; i < kKs; ++i)
          *reinterpret_cast<float4*>(row + 16 * i + 4u * quad) =
              make_float4(o[2 * i][2 * e], o[2 * i + 1][2 * e], o[2 * i][2 * e + 1],
                          o[2 * i + 1][2 * e + 1]);
      }
      asm volatile("barrier.cta.sync 1, 128;" ::: "memory");
      merge_rows<kDP, kBf16, kLift>(a, t, rows, merge, pieces);
      // the sums have been read: the next tile may write its own
      if (any_of_four(!go || count == 0)) break;
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
  using S = StepShape8<kDP>;
  auto kern = k_paged8_step<kDP, kBf16, kSel>;
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
  return launch_step_join<kDP, kBf16, kLift>(a, ctas, st);
}

}  // namespace

cudaError_t launch_paged8_step(const PagedAttnArgs& a, const PagedMaps& m, int sm_count,
                               bool behind, cudaStream_t st) {
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
