// The paged K/V cache's operators around its attention: appending new keys and
// values (normalised and rotated on the way), bounds of the pages' keys, scores
// of the pages, and the choice of the pages with the largest scores.
#include "ibp_paged.cuh"
#include "ibp_sm103.cuh"
#include "ibp_tma.cuh"

namespace ibp {
namespace {

// ---------------------------------------------------------------- append
// kLanes lanes hold a head, 8 channels each: 4 and their 4 rotation partners
// (channels 4 j and rot/2 + 4 j on, or 8 together when pairs are adjacent or past rot),
// so that a rotation needs no other lane and the sum of squares one shuffle
// tree.  A lane keeps its channels over all heads of a token, so the token's place,
// its cosines and sines and the norms' weights are fetched once; kAhead heads are in
// flight at a time.  Rounds of kSubs heads hold queries, keys or values alone.  HBM sets
// the floor (each byte is read and written once) and the schedulers' issue the time, so
// sums and products run on pairs of floats.  10 CTAs of 128 threads share an SM and three
// heads are in flight per lane: 51 us for 5,900 tokens of 64 + 8 + 8 heads of 128
// with both norms (243 MB, 4.8 TB/s); unbounded registers and four heads 62 us, 8 CTAs and
// four 53, 12 CTAs and two 51, 16 CTAs (32 registers, spilled) 52 to 55.
template <int kLanes, int kAhead, bool kBf16, bool kPairs>
__global__ void __launch_bounds__(128, 10) k_paged_append(PagedAppendArgs a, uint32_t per) {
  constexpr uint32_t kSubs = 128u / kLanes;  // heads side by side
  const uint32_t lane = threadIdx.x & (kLanes - 1u), sub = threadIdx.x / kLanes;
  const uint32_t t = blockIdx.x;
  const uint32_t nq = (a.Hq + kSubs - 1u) / kSubs, nk = (a.g.H + kSubs - 1u) / kSubs;
  const uint32_t r0 = blockIdx.y * per, r1 = min(nq + 2u * nk, r0 + per);
  // this lane's channels: 4 at c0, 4 at c1
  const bool mine = lane * 8u < a.g.D;
  const uint32_t half = a.rot / 2u;
  const bool split = !kPairs && lane * 8u < a.rot;
  const uint32_t c0 = split ? lane * 4u : lane * 8u, c1 = split ? half + lane * 4u : c0 + 4u;
  const bool turned = lane * 8u < a.rot;
  const uint64_t row = a.g.D * 2ull;
  // The rounds of one kind that fall to this CTA: a pointer walks over this thread's heads.
  struct Part {
    const uint8_t* src;  // this thread's head of the first round
    uint32_t h, n;       // that head, rounds
  };
  auto part = [&](const uint8_t* base, uint32_t first, uint32_t rounds) {
    const uint32_t lo = max(r0, first), hi = min(r1, first + rounds);
    const uint32_t h = (lo - first) * kSubs + sub;
    return Part{base + h * row, h, hi > lo ? hi - lo : 0u};
  };
  const Part pq = part(a.q + t * a.q_stride, 0, nq);
  const Part pk = part(a.kx + t * a.kv_stride, nq, nk);
  const Part pv = part(a.vx + t * a.kv_stride, nq + nk, nk);
  auto load = [&](const Part& p, uint32_t r, uint32_t heads) {
    uint4 x = make_uint4(0, 0, 0, 0);
    if (r < p.n && mine && p.h + r * kSubs < heads) {
      const uint8_t* src = p.src + (uint64_t)(r * kSubs) * row;
      const uint2 u = __ldcs(reinterpret_cast<const uint2*>(src + c0 * 2u));
      const uint2 v = __ldcs(reinterpret_cast<const uint2*>(src + c1 * 2u));
      x = make_uint4(u.x, u.y, v.x, v.y);
    }
    return x;
  };
  uint4 x[kAhead];
  const Part& p0 = pq.n ? pq : pk.n ? pk : pv;
#pragma unroll
  for (int i = 0; i < kAhead; ++i) x[i] = load(p0, i, pq.n ? a.Hq : a.g.H);
  // the norms' weights
  uint2 wq[2] = {}, wk[2] = {};
  if (a.q_norm && mine) {
    wq[0] = __ldg(reinterpret_cast<const uint2*>(a.q_norm + c0 * 2u));
    wq[1] = __ldg(reinterpret_cast<const uint2*>(a.q_norm + c1 * 2u));
  }
  if (a.k_norm && mine) {
    wk[0] = __ldg(reinterpret_cast<const uint2*>(a.k_norm + c0 * 2u));
    wk[1] = __ldg(reinterpret_cast<const uint2*>(a.k_norm + c1 * 2u));
  }
  // the token's place
  const uint32_t s = paged_find(a.b, t);
  if (s == a.b.n_seqs) return;  // a row of no sequence
  const PagedSeq q = paged_seq(a.b, a.g.page_lg, s);
  const uint32_t pos = q.L - q.n + (t - q.q0);  // (as a signed number: negative before the first)
  bool ok = q.ok && (int32_t)pos >= 0 && (!a.cos_sin || pos < a.n_pos);
  uint8_t *kd = nullptr, *vd = nullptr;
  if (ok) {
    const int32_t page = __ldg(a.b.table + s * a.b.table_stride + (pos >> a.g.page_lg));
    if (page >= 0 && (uint32_t)page < a.g.n_pages) {
      const uint64_t at = (uint64_t)(uint32_t)page * a.g.page_stride +
                          (pos & ((1u << a.g.page_lg) - 1u)) * a.g.token_stride;
      kd = a.g.k + at;
      vd = a.g.v + at;
    }
  }
  if (!kd) {
    ok = false;
    if (threadIdx.x == 0) set_status(a.g.status, IBP_ERANGE);
  }
  float4 cc = make_float4(0.f, 0.f, 0.f, 0.f), ss = cc;
  if (a.cos_sin && ok && turned) {
    const float* cs = a.cos_sin + (uint64_t)pos * a.rot + lane * 4u;
    cc = __ldg(reinterpret_cast<const float4*>(cs));
    ss = __ldg(reinterpret_cast<const float4*>(cs + half));
  }
  const float inv_d = 1.f / (float)a.g.D;
  // one kind's rounds: `first` says that their first heads are on their way already
  auto go = [&](const Part& p, uint32_t heads, const bool turns, const bool normed,
                const uint2 (&w)[2], uint8_t* dst, uint64_t head_stride, const bool zero,
                const bool first) {
    if (p.n == 0) return;
    if (!first)
#pragma unroll
      for (int i = 0; i < kAhead; ++i) x[i] = load(p, i, heads);
    dst += p.h * head_stride;
    for (uint32_t r = 0; r < p.n; r += kAhead) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (r + i >= p.n) break;
        uint4 y = x[i];
        x[i] = load(p, r + i + kAhead, heads);
        if (normed || turns) {  // the same for the whole CTA
          const uint32_t yw[4] = {y.x, y.y, y.z, y.w};
          uint64_t f[4];  // two channels each
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 v = unpack2(yw[k], kBf16);
            f[k] = pair2(v.x, v.y);
          }
          if (normed) {
            uint64_t s2 = mul2(f[0], f[0]);
#pragma unroll
            for (int k = 1; k < 4; ++k) s2 = fma2(f[k], f[k], s2);
            float sum, odd;
            halves2(s2, sum, odd);
            sum += odd;
#pragma unroll
            for (int d = kLanes / 2; d; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
            const float n = rsqrtf(fmaf(sum, inv_d, a.eps));
            const uint64_t n2 = pair2(n, n);
            const uint32_t gw[4] = {w[0].x, w[0].y, w[1].x, w[1].y};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 gf = unpack2(gw[k], kBf16);
              f[k] = mul2(f[k], mul2(n2, pair2(gf.x, gf.y)));
            }
          }
          if (turns && turned) {
            if (kPairs) {  // a pair of channels is a pair of the rotation
              const float c4[4] = {cc.x, cc.y, cc.z, cc.w}, s4[4] = {ss.x, ss.y, ss.z, ss.w};
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                float u, v;
                halves2(f[k], u, v);
                f[k] = fma2(f[k], pair2(c4[k], c4[k]), mul2(pair2(-v, u), pair2(s4[k], s4[k])));
              }
            } else {
              const uint64_t c2[2] = {pair2(cc.x, cc.y), pair2(cc.z, cc.w)};
              const uint64_t s2[2] = {pair2(ss.x, ss.y), pair2(ss.z, ss.w)};
              const uint64_t m2[2] = {pair2(-ss.x, -ss.y), pair2(-ss.z, -ss.w)};
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const uint64_t u = f[k], v = f[k + 2];
                f[k] = fma2(u, c2[k], mul2(v, m2[k]));
                f[k + 2] = fma2(v, c2[k], mul2(u, s2[k]));
              }
            }
          }
          uint32_t z[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float u, v;
            halves2(f[k], u, v);
            z[k] = pack2(u, v, kBf16);
          }
          y = make_uint4(z[0], z[1], z[2], z[3]);
        }
        if (mine && p.h + (r + i) * kSubs < heads) {
          uint8_t* d = dst + (uint64_t)((r + i) * kSubs) * head_stride;
          if (zero) y = make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint2*>(d + c0 * 2u) = make_uint2(y.x, y.y);
          *reinterpret_cast<uint2*>(d + c1 * 2u) = make_uint2(y.z, y.w);
        }
      }
    }
  };
  const bool turns = a.cos_sin != nullptr;
  go(pq, a.Hq, turns, a.q_norm != nullptr, wq, a.q_out + t * a.qo_stride, row, !ok, true);
  if (!ok) return;
  go(pk, a.g.H, turns, a.k_norm != nullptr, wk, kd, a.g.head_stride, false, pq.n == 0);
  go(pv, a.g.H, false, false, wk, vd, a.g.head_stride, false, pq.n == 0 && pk.n == 0);
}

template <bool kBf16>
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  if (kBf16) {
    const __nv_bfloat162 r = __hmin2_nan(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                         *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  const __half2 r =
      __hmin2_nan(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

template <bool kBf16>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  if (kBf16) {
    const __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                         *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  const __half2 r =
      __hmax2_nan(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// ---------------------------------------------------------------- bounds
// One warp per (page that got new tokens, head): 32 / kLanes tokens at a time,
// 8 channels per lane, their smallest and largest kept packed in pairs.  Minima
// and maxima of 16-bit values are exact in 16 bits.
template <int kLanes, bool kBf16>
__global__ void __launch_bounds__(128)
    k_paged_bounds(PagedGeom g, PagedBatchView b, uint8_t* bounds) {
  // the scores' CTAs may come up beside this kernel (they wait for its end)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t lane = threadIdx.x & 31u, sub = lane & (kLanes - 1u), row = lane / kLanes;
  const uint64_t id = (uint64_t)blockIdx.x * 4u + (threadIdx.x >> 5);
  const uint32_t tile = (uint32_t)(id / g.H), h = (uint32_t)(id % g.H);
  const uint32_t P = 1u << g.page_lg;
  uint32_t first;
  const uint32_t s = paged_find_tile(b, P, 2u, tile, first);
  const PagedSeq q = paged_seq(b, g.page_lg, s);
  if (!q.ok) {
    if (lane == 0) set_status(g.status, IBP_ERANGE);
    return;
  }
  if (q.n == 0 || q.L == 0 || tile < first) return;
  const uint32_t from = q.L > q.n ? q.L - q.n : 0u;  // the first new token that has a position
  const uint32_t p = (from >> g.page_lg) + (tile - first);
  if (p > (q.L - 1u) >> g.page_lg) return;
  const int32_t page = __ldg(b.table + s * b.table_stride + p);
  if (page < 0 || (uint32_t)page >= g.n_pages) {
    if (lane == 0) set_status(g.status, IBP_ERANGE);
    return;
  }
  const uint32_t held = min(P, q.L - p * P);
  const uint8_t* src = g.k + (uint64_t)(uint32_t)page * g.page_stride + h * g.head_stride +
                       sub * 16u;
  const bool mine = sub * 8u < g.D;
  const uint32_t inf = kBf16 ? 0x7F807F80u : 0x7C007C00u;
  uint32_t lo[4], hi[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) lo[i] = inf, hi[i] = inf | 0x80008000u;
  if (mine) {
#pragma unroll 4
    for (uint32_t t = row; t < held; t += 32u / kLanes) {
      const uint4 x = __ldg(reinterpret_cast<const uint4*>(src + t * g.token_stride));
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        lo[i] = min2<kBf16>(lo[i], w[i]);
        hi[i] = max2<kBf16>(hi[i], w[i]);
      }
    }
  }
#pragma unroll
  for (int d = kLanes; d < 32; d <<= 1)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo[i] = min2<kBf16>(lo[i], __shfl_xor_sync(0xFFFFFFFFu, lo[i], d));
      hi[i] = max2<kBf16>(hi[i], __shfl_xor_sync(0xFFFFFFFFu, hi[i], d));
    }
  if (mine && row == 0) {
    uint8_t* dst = bounds + ((uint64_t)(uint32_t)page * g.H + h) * g.D * 4u + sub * 16u;
    *reinterpret_cast<uint4*>(dst) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    *reinterpret_cast<uint4*>(dst + g.D * 2u) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
  }
}

// ---------------------------------------------------------------- scores
// sum_d max(q lo, q hi) = sum_d max(q, 0) hi + min(q, 0) lo: a product of
// [max(q, 0), min(q, 0)] with [hi, lo], whose 16-bit products are exact in fp32.
// A warp holds 16 rows (as many tokens of one sequence as their G queries
// allow; 16 of the G queries at a time when G > 16) as the left operand, and 32 pages'
// bounds in shared memory, all in flight together: bound by HBM where tokens are few.
// (16-byte asynchronous copies: a bulk copy for each page's 512 bytes took 35 us for
// 134 MB, as many as the copy engine starts.)
// The sum runs over the channels in any order, so a lane takes 8 channels
// together (one 16-byte load) where the instruction's layout wants pairs; rows are 16
// bytes longer than their bounds, so that eight pages' loads meet no bank twice.
constexpr uint32_t kScoreGroup = 32;  // pages of a warp at a time

template <int kDP>
constexpr uint32_t score_smem() {
  return 4u * kScoreGroup * (kDP * 4u + 16u);
}

// The sum of one query and one page as it is written: for scores whose products are NaN, as
// 0 * inf is (the bound that the other one outdoes is infinite).  Rare, and done once more
// at the end (in the loop over the pages it cost every call 1.4 %).
template <bool kBf16>
__device__ float score_as_written(const uint8_t* q, const uint8_t* bounds, uint32_t D) {
  float sum = 0.f;
#pragma unroll 1
  for (uint32_t d = 0; d < D; d += 2u) {
    const float2 x = unpack2(__ldg(reinterpret_cast<const uint32_t*>(q + d * 2u)), kBf16);
    const float2 lo = unpack2(__ldg(reinterpret_cast<const uint32_t*>(bounds + d * 2u)), kBf16);
    const float2 hi =
        unpack2(__ldg(reinterpret_cast<const uint32_t*>(bounds + (D + d) * 2u)), kBf16);
    auto larger = [](float u, float v) { return u > v || u != u ? u : v; };
    sum += larger(x.x * lo.x, x.x * hi.x);
    sum += larger(x.y * lo.y, x.y * hi.y);
  }
  return sum;
}

template <bool kBf16, int kDP>
__global__ void __launch_bounds__(128, 3)
    k_paged_scores(PagedGeom g, PagedBatchView b, const uint8_t* q, uint64_t q_stride, uint32_t G,
                   const uint8_t* bounds, float* scores, uint32_t per_warp) {
  constexpr int kC = kDP / 32;  // 16-byte chunks per lane
  extern __shared__ __align__(128) uint8_t s_bounds[];
  __shared__ float s_c[4][16][kScoreGroup + 1];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31u;
  const uint32_t quad = lane & 3u, r0 = lane >> 2;
  const uint32_t tpt = G >= 16u ? 1u : 16u / G;  // tokens of a tile
  const uint32_t h = blockIdx.y;
  const uint32_t stride = g.D * 4u + 16u;
  uint8_t* mine = s_bounds + warp * kScoreGroup * stride;
  uint32_t first;
  const uint32_t s = paged_find_tile(b, tpt, 1u, blockIdx.x, first);
  const PagedSeq sq = paged_seq(b, g.page_lg, s);
  if (!sq.ok && threadIdx.x == 0) set_status(g.status, IBP_ERANGE);
  const uint32_t t0 = (blockIdx.x - first) * tpt;
  if (blockIdx.x < first || t0 >= sq.n) return;
  const uint32_t nt = min(tpt, sq.n - t0);
  const uint32_t groups = (b.max_pages + kScoreGroup - 1u) / kScoreGroup;
  const uint32_t g0 = (blockIdx.z * 4u + warp) * per_warp;
  const uint32_t g1 = min(groups, g0 + per_warp);
  const int64_t pos_last = (int64_t)sq.L - sq.n + t0 + nt - 1;
  const uint32_t seen_last = pos_last < 0 ? 0u : (uint32_t)(pos_last >> g.page_lg) + 1u;
  const float hidden = __int_as_float((int)0xFF800000u);
  uint32_t qv[kC * 4 * 2];  // [chunk][4 words][row, row + 8]
  auto page_at = [&](uint32_t c) {
    return c + lane < seen_last ? __ldg(b.table + s * b.table_stride + c + lane) : -1;
  };
  // Half of a group's bounds, on their way: a page's 16-byte pieces to as many lanes
  // (the next power of two), 32 / kPiece pages at a time.
  constexpr uint32_t kPiece = kDP / 4u;
  const uint32_t piece = lane % kPiece, page0 = lane / kPiece;
  const uint8_t* from = bounds + ((uint64_t)h * g.D / 4u + piece) * 16u;
  const uint32_t to = smem_addr(mine) + page0 * stride + piece * 16u;
  const uint32_t page_bytes = g.H * g.D * 4u;
  auto copy_half = [&](uint32_t half, int32_t id) {
#pragma unroll 4
    for (uint32_t k = 0; k < kScoreGroup / 2u; k += 32u / kPiece) {
      const uint32_t at = half * (kScoreGroup / 2u) + k;
      const int32_t pid = __shfl_sync(0xFFFFFFFFu, id, at + page0);
      if ((uint32_t)pid < g.n_pages && piece < g.D / 4u)  // (negative: none)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + at * stride),
                     "l"(from + (uint64_t)(uint32_t)pid * page_bytes)
                     : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  const uint32_t blocks = tpt == 1u ? (G + 15u) / 16u : 1u;  // of 16 rows
  int32_t next = page_at(g0 * kScoreGroup), next2 = page_at((g0 + 1u) * kScoreGroup);
  copy_half(0, next);
  copy_half(1, next);
  bool odd = false;  // one of this lane's scores is NaN
  for (uint32_t gr = g0; gr < g1; ++gr) {
    const uint32_t c0 = gr * kScoreGroup;
    if (c0 >= seen_last) {
      for (uint32_t tt = 0; tt < nt; ++tt)
        if (c0 + lane < b.max_pages)
          scores[((uint64_t)(sq.q0 + t0 + tt) * g.H + h) * b.max_pages + c0 + lane] = hidden;
      continue;
    }
    int32_t id = next;  // this lane's page
    next = next2;
    next2 = page_at(c0 + 2u * kScoreGroup);
    if (c0 + lane < seen_last && (id < 0 || (uint32_t)id >= g.n_pages)) {
      set_status(g.status, IBP_ERANGE);
      id = -1;
    }
    float best = 0.f;  // over the queries of the earlier row blocks (G > 16)
    for (uint32_t rb = 0; rb < blocks; ++rb) {
      if (gr == g0 || blocks > 1u) {  // the rows' queries
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t r = rb * 16u + r0 + 8u * e;
          const uint32_t tt = r / G, gg = r % G;
          const bool live = tt < nt;
          const uint8_t* src = q + (uint64_t)(sq.q0 + t0 + tt) * q_stride +
                               ((uint64_t)h * G + gg) * g.D * 2u;
#pragma unroll
          for (int c = 0; c < kC; ++c) {
            const uint32_t ch = 32u * c + 8u * quad;
            uint4 x = make_uint4(0, 0, 0, 0);
            if (live && ch < g.D) x = __ldg(reinterpret_cast<const uint4*>(src + ch * 2u));
            qv[(c * 4 + 0) * 2 + e] = x.x;
            qv[(c * 4 + 1) * 2 + e] = x.y;
            qv[(c * 4 + 2) * 2 + e] = x.z;
            qv[(c * 4 + 3) * 2 + e] = x.w;
          }
        }
      }
#pragma unroll 1
      for (uint32_t half = 0; half < 2u; ++half) {
        if (rb == 0) {  // all but the half that was asked for last
          if (blocks == 1u)
            asm volatile("cp.async.wait_group 1;" ::: "memory");
          else
            asm volatile("cp.async.wait_all;" ::: "memory");
          __syncwarp();
        }
        // 16 pages, 8 to an instruction; the signs' products apart: four chains of sums
        const uint8_t* src = mine + (half * 16u + r0) * stride + quad * 16u;
        float acc[2][2][4] = {};
#pragma unroll
        for (int c = 0; c < kC; ++c) {
          uint32_t p[8], n[8];  // the queries split by sign
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            p[k] = max2<kBf16>(qv[c * 8 + k], 0u);
            n[k] = min2<kBf16>(qv[c * 8 + k], 0u);
          }
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint8_t* at = src + x * 8u * stride + c * 64u;
            uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
            if (32u * c + 8u * quad < g.D) {
              lo = *reinterpret_cast<const uint4*>(at);
              hi = *reinterpret_cast<const uint4*>(at + g.D * 2u);
            }
            mma_16816<kBf16>(acc[x][0], p, hi.x, hi.y);
            mma_16816<kBf16>(acc[x][1], n, lo.x, lo.y);
            mma_16816<kBf16>(acc[x][0], p + 4, hi.z, hi.w);
            mma_16816<kBf16>(acc[x][1], n + 4, lo.z, lo.w);
          }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float* d0 = &s_c[warp][r0][half * 16u + x * 8u + 2u * quad];
          float* d1 = &s_c[warp][r0 + 8u][half * 16u + x * 8u + 2u * quad];
          d0[0] = acc[x][0][0] + acc[x][1][0], d0[1] = acc[x][0][1] + acc[x][1][1];
          d1[0] = acc[x][0][2] + acc[x][1][2], d1[1] = acc[x][0][3] + acc[x][1][3];
        }
        // a half that has been read makes room for the next group's
        if (rb + 1u == blocks) {
          __syncwarp();
          copy_half(half, gr + 1u < g1 ? next : -1);
        }
      }
      __syncwarp();
      // the largest over each token's queries, kept by the lane of the page (memory of a
      // page that was not copied is never looked at)
      const uint32_t rows = tpt == 1u ? min(16u, G - rb * 16u) : G;
      for (uint32_t tt = 0; tt < nt; ++tt) {
        float m = s_c[warp][tt * G][lane];
        for (uint32_t i = 1; i < rows; ++i) {
          const float v = s_c[warp][tt * G + i][lane];
          m = (v > m || v != v) ? v : m;
        }
        if (rb) m = (best > m || best != best) ? best : m;
        best = m;
        const int64_t pos = (int64_t)sq.L - sq.n + t0 + tt;
        const bool seen = pos >= 0 && c0 + lane <= (uint32_t)(pos >> g.page_lg) && id >= 0;
        odd = odd || (seen && m != m);
        if (c0 + lane < b.max_pages && rb + 1u == blocks)
          scores[((uint64_t)(sq.q0 + t0 + tt) * g.H + h) * b.max_pages + c0 + lane] =
              seen ? m : hidden;
      }
      __syncwarp();
    }
  }
  if (!odd) return;
  for (uint32_t c = g0 * kScoreGroup + lane; c < min(b.max_pages, g1 * kScoreGroup);
       c += kScoreGroup)
#pragma unroll 1
    for (uint32_t tt = 0; tt < nt; ++tt) {
      float* at = scores + ((uint64_t)(sq.q0 + t0 + tt) * g.H + h) * b.max_pages + c;
      if (*at == *at) continue;  // (a page that is hidden, or that has no id, is not NaN)
      const uint32_t page = (uint32_t)__ldg(b.table + s * b.table_stride + c);
      const uint8_t* q0 = q + (uint64_t)(sq.q0 + t0 + tt) * q_stride + (uint64_t)h * G * g.D * 2u;
      float m = -INFINITY;
#pragma unroll 1
      for (uint32_t i = 0; i < G; ++i) {
        const float v = score_as_written<kBf16>(
            q0 + i * g.D * 2u, bounds + ((uint64_t)page * g.H + h) * g.D * 4u, g.D);
        m = (v > m || v != v) ? v : m;
      }
      *at = m;
    }
}

// ---------------------------------------------------------------- select
// Scores as whole numbers of the same order: the sign bit folded in, -0 as 0, NaN as inf.
__device__ __forceinline__ uint32_t order_key(float f) {
  if (f != f) f = INFINITY;
  const uint32_t u = __float_as_uint(f + 0.f);  // -0 + 0 is 0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// The row's place: its own page; the number of pages to choose from (0: none).
__device__ __forceinline__ uint32_t select_row(const PagedGeom& g, const PagedBatchView& b,
                                               uint32_t t, uint32_t s, uint32_t& own) {
  const PagedSeq q = paged_seq(b, g.page_lg, s);
  const int64_t pos = (int64_t)q.L - q.n + (t - q.q0);
  if (!q.ok) set_status(g.status, IBP_ERANGE);
  own = pos < 0 ? 0u : (uint32_t)(pos >> g.page_lg);
  return !q.ok || pos < 0 ? 0u : own + 1u;
}

// kWarps warps to a row, its scores in their registers (kPer each; a warp has a run of
// numbers), the own page's as +inf.  A threshold that n_sel of them reach is bracketed
// by counts, placed between the bracket's ends as if the count fell off
// exponentially there (tails do), every third time in the middle: 6 to 8 counts for
// 1000 normal scores.  Where no such threshold lies between two scores (equal ones,
// infinities) the n_sel-th largest is found bit by bit, and of those equal to it the
// first are taken.  Bound by issue: 59 kPer instructions a row of 1001, of them 2 kPer for
// each count and 9 kPer to write the numbers (7960 such rows in 23 us).  4 rows to a CTA
// when kWarps is 1.
template <int kWarps, int kPer>
__global__ void __launch_bounds__(kWarps == 1 ? 128 : kWarps * 32,
                                  kPer <= 16 ? 4 : kPer <= 32 && kWarps == 1 ? 6 : 1)
    k_paged_pick(PagedGeom g, PagedBatchView b, const float* scores, uint32_t n_sel,
                 int32_t* selected) {
  constexpr int kRowsPer = kWarps == 1 ? 4 : 1;
  __shared__ uint32_t s_sum[2][kWarps][2];
  const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31u;
  const uint64_t row = (uint64_t)blockIdx.x * kRowsPer + (kWarps == 1 ? warp : 0u);
  if (row >= (uint64_t)b.n_tokens * g.H) return;
  const uint32_t part = kWarps == 1 ? 0u : warp;
  const uint32_t t = (uint32_t)(row / g.H);
  int32_t* out = selected + row * n_sel;
  const uint32_t i0 = part * (32u * kPer) + lane;  // number of this lane's first score
  const float* src = scores + row * b.max_pages + i0;
  float v[kPer];  // fetched before the row's length is known
#pragma unroll
  for (int j = 0; j < kPer; ++j) v[j] = i0 + 32u * j < b.max_pages ? __ldcs(src + 32u * j) : 0.f;
  const uint32_t s = paged_find(b, t);
  if (s == b.n_seqs) return;
  uint32_t own;
  const uint32_t n = select_row(g, b, t, s, own);
  if (n <= n_sel) {
    for (uint32_t i = part * 32u + lane; i < n_sel; i += kWarps * 32u)
      out[i] = i < n ? (int32_t)i : -1;
    return;
  }
  uint32_t phase = 0;
  // the sum over the row; below: those of the warps before this one, of two values
  auto sum = [&](uint32_t x, uint32_t y, uint32_t* below) {
    x = __reduce_add_sync(0xFFFFFFFFu, x);
    if (below) {
      y = __reduce_add_sync(0xFFFFFFFFu, y);
      below[0] = below[1] = 0;
    }
    if (kWarps > 1) {
      if (lane == 0) s_sum[phase][part][0] = x, s_sum[phase][part][1] = y;
      __syncthreads();
      x = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        x += s_sum[phase][w][0];
        if (below && w < (int)part) below[0] += s_sum[phase][w][0], below[1] += s_sum[phase][w][1];
      }
      phase ^= 1u;
    }
    return x;
  };
  float lo = INFINITY, hi = -INFINITY;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const uint32_t i = i0 + 32u * j;
    if (i == own || v[j] != v[j]) v[j] = INFINITY;
    lo = i < n ? fminf(lo, v[j]) : lo;
    hi = i < n && i != own ? fmaxf(hi, v[j]) : hi;
    if (i >= n) v[j] = -INFINITY;
  }
  uint32_t klo = __reduce_min_sync(0xFFFFFFFFu, order_key(lo));
  uint32_t khi = __reduce_max_sync(0xFFFFFFFFu, order_key(hi));
  if (kWarps > 1) {
    if (lane == 0) s_sum[1][part][0] = klo, s_sum[1][part][1] = khi;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
      klo = min(klo, s_sum[1][w][0]), khi = max(khi, s_sum[1][w][1]);
  }
  // a is reached by `clo` scores, at least n_sel; z, at least the largest but the own, by the
  // own and no other, or by `chi`, too few
  auto score = [](uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k); };
  float a = score(klo), z = score(khi);
  uint32_t clo = n, chi = 1;
  if (n_sel == 1u) a = INFINITY, clo = z < INFINITY ? 1u : 2u;  // the own page, if no other is inf
  for (int k = 0; clo != n_sel && a > -INFINITY && z < INFINITY; ++k) {
    const float part_of = k % 3 == 2 ? 0.5f
                                     : __fdividef(__log2f((float)clo) - __log2f((float)n_sel),
                                                  __log2f((float)clo) - __log2f((float)chi));
    float c = fmaf(z - a, part_of, a);
    if (!(c > a && c < z)) c = a + 0.5f * (z - a);
    if (!(c > a && c < z) || k == 32) break;  // neighbours, or no end: bit by bit
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) m += v[j] >= c;
    m = sum(m, 0, nullptr);
    if (m >= n_sel)
      a = c, clo = m;
    else
      z = c, chi = m;
  }
  const uint32_t lt = (1u << lane) - 1u;
  uint32_t below[2];
  if (clo == n_sel && a > -INFINITY) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) m += v[j] >= a;
    if (kWarps > 1) sum(m, 0, below);
    int32_t* to = out + (kWarps > 1 ? below[0] : 0u);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const uint32_t w = __ballot_sync(0xFFFFFFFFu, v[j] >= a);
      if (v[j] >= a) to[__popc(w & lt)] = (int32_t)(i0 + 32u * j);
      to += __popc(w);
    }
    return;
  }
  // keys: 0 past the row's end, the own page's above all
  auto key = [&](int j) {
    const uint32_t i = i0 + 32u * j;
    return i == own ? 0xFFFFFFFFu : i < n ? order_key(v[j]) : 0u;
  };
  uint32_t thr = 0;
  for (int bit = 31; bit >= 0; --bit) {
    const uint32_t cand = thr | 1u << bit;
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) m += key(j) >= cand;
    if (sum(m, 0, nullptr) >= n_sel) thr = cand;
  }
  uint32_t above = 0, equal = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) above += key(j) > thr, equal += key(j) == thr;
  const uint32_t want = n_sel - sum(above, equal, below);  // of the equal ones
  uint32_t na = below[0], ne = below[1];
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const bool up = key(j) > thr, eq = key(j) == thr;
    const uint32_t bu = __ballot_sync(0xFFFFFFFFu, up), be = __ballot_sync(0xFFFFFFFFu, eq);
    const uint32_t e = ne + __popc(be & lt);
    if (up || (eq && e < want)) out[na + __popc(bu & lt) + min(e, want)] = (int32_t)(i0 + 32u * j);
    na += __popc(bu);
    ne += __popc(be);
  }
}

// Rows of more pages than that hold: one CTA to a row, the n_sel-th largest key
// found digit by digit, 8 bits from the top, with a histogram of the keys that share
// the digits found so far; then one ordered pass.
constexpr uint32_t kSelThreads = 256;

__global__ void __launch_bounds__(256)
    k_paged_select(PagedGeom g, PagedBatchView b, const float* scores, uint32_t n_sel,
                   int32_t* selected) {
  __shared__ uint32_t s_hist[256];
  __shared__ uint32_t s_warp[2][8];
  __shared__ uint32_t s_pick[2];
  const uint32_t t = blockIdx.x, h = blockIdx.y, tid = threadIdx.x;
  const uint32_t warp = tid >> 5, lane = tid & 31u;
  int32_t* out = selected + ((uint64_t)t * g.H + h) * n_sel;
  const uint32_t s = paged_find(b, t);
  if (s == b.n_seqs) return;
  uint32_t own;
  const uint32_t n = select_row(g, b, t, s, own);
  if (n <= n_sel) {
    for (uint32_t i = tid; i < n_sel; i += kSelThreads) out[i] = i < n ? (int32_t)i : -1;
    return;
  }
  const float* row = scores + ((uint64_t)t * g.H + h) * b.max_pages;
  auto key = [&](uint32_t i) { return i == own ? 0xFFFFFFFFu : order_key(__ldg(row + i)); };
  uint32_t prefix = 0, mask = 0, want = n_sel;  // want-th largest among those with the prefix
  for (int sh = 24; sh >= 0; sh -= 8) {
    s_hist[tid] = 0;
    __syncthreads();
    for (uint32_t i = tid; i < n; i += kSelThreads) {
      const uint32_t k = key(i);
      if ((k & mask) == prefix) atomicAdd(&s_hist[(k >> sh) & 255u], 1u);
    }
    __syncthreads();
    // how many lie in this digit's larger values: a suffix sum over the 256
    const uint32_t c = s_hist[255u - tid];
    uint32_t inc = c;
#pragma unroll
    for (uint32_t d = 1; d < 32u; d <<= 1) {
      const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, inc, d);
      if (lane >= d) inc += v;
    }
    if (lane == 31u) s_warp[0][warp] = inc;
    __syncthreads();
    for (uint32_t w = 0; w < warp; ++w) inc += s_warp[0][w];
    if (inc >= want && inc - c < want) {
      s_pick[0] = 255u - tid;
      s_pick[1] = want - (inc - c);
    }
    __syncthreads();
    prefix |= s_pick[0] << sh;
    mask |= 255u << sh;
    want = s_pick[1];
  }
  // `prefix` is the n_sel-th largest; `want` of those equal to it are taken
  const uint32_t per = (n + 255u) / 256u * 32u;  // a warp's run of numbers, a multiple of 32
  const uint32_t i0 = warp * per, i1 = min(n, i0 + per);
  uint32_t above = 0, equal = 0;
  for (uint32_t i = i0 + lane; i < i1; i += 32u) {
    const uint32_t k = key(i);
    above += k > prefix;
    equal += k == prefix;
  }
  above = __reduce_add_sync(0xFFFFFFFFu, above);
  equal = __reduce_add_sync(0xFFFFFFFFu, equal);
  __syncthreads();
  if (lane == 0) s_warp[0][warp] = above, s_warp[1][warp] = equal;
  __syncthreads();
  uint32_t na = 0, ne = 0;  // before this warp
  for (uint32_t w = 0; w < warp; ++w) na += s_warp[0][w], ne += s_warp[1][w];
  for (uint32_t i = i0; i < i1; i += 32u) {
    const uint32_t k = i + lane < i1 ? key(i + lane) : 0u;
    const bool hi = i + lane < i1 && k > prefix, eq = i + lane < i1 && k == prefix;
    const uint32_t bh = __ballot_sync(0xFFFFFFFFu, hi), be = __ballot_sync(0xFFFFFFFFu, eq);
    const uint32_t below = (1u << lane) - 1u;
    const uint32_t e = ne + __popc(be & below);
    if (hi || (eq && e < want)) out[na + __popc(bh & below) + min(e, want)] = (int32_t)(i + lane);
    na += __popc(bh);
    ne += __popc(be);
  }
}

uint32_t pow2_lanes(uint32_t D) { return D <= 32u ? 4u : D <= 64u ? 8u : 16u; }

}  // namespace

#define IBP_PAGED_LANES(CALL)                                                     \
  do {                                                                            \
    const uint32_t ln = pow2_lanes(D_);                                           \
    if (bf_) {                                                                    \
      if (ln == 4u) CALL(4, true);                                                \
      else if (ln == 8u) CALL(8, true);                                           \
      else CALL(16, true);                                                        \
    } else {                                                                      \
      if (ln == 4u) CALL(4, false);                                               \
      else if (ln == 8u) CALL(8, false);                                          \
      else CALL(16, false);                                                       \
    }                                                                             \
  } while (0)

cudaError_t launch_paged_append(const PagedAppendArgs& a, int sm_count, cudaStream_t st) {
  const uint32_t D_ = a.g.D;
  const bool bf_ = a.g.bf16 != 0u;
  // Rounds of a CTA: as many as leave 16 CTAs to each SM (a token's place is then looked up
  // for more heads), 16 at most.  At 5,900 tokens of 10 rounds: all of a token's in one CTA
  // 51 us, 5 rounds 53, 3 rounds 64, 2 rounds 72.
  const uint64_t subs = 128u / pow2_lanes(D_);
  const uint64_t rounds = (a.Hq + subs - 1) / subs + 2u * ((a.g.H + subs - 1) / subs);
  uint64_t per = rounds * a.b.n_tokens / (16ull * sm_count);
  per = per < 1u ? 1u : per > 16u ? 16u : per;
  const uint64_t y = (rounds + per - 1) / per;
  per = (rounds + y - 1) / y;
  if (y > 65535u) return cudaErrorInvalidValue;
  const dim3 grid(a.b.n_tokens, (unsigned)y);
#define IBP_CALL(L, B)                                                                    \
  do {                                                                                    \
    if (per >= 2u) {                                                                      \
      if (a.pairs) k_paged_append<L, 3, B, true><<<grid, 128, 0, st>>>(a, (uint32_t)per); \
      else k_paged_append<L, 3, B, false><<<grid, 128, 0, st>>>(a, (uint32_t)per);        \
    } else {                                                                              \
      if (a.pairs) k_paged_append<L, 1, B, true><<<grid, 128, 0, st>>>(a, (uint32_t)per); \
      else k_paged_append<L, 1, B, false><<<grid, 128, 0, st>>>(a, (uint32_t)per);        \
    }                                                                                     \
  } while (0)
  IBP_PAGED_LANES(IBP_CALL);
#undef IBP_CALL
  return cudaGetLastError();
}

cudaError_t launch_paged_bounds(const PagedGeom& g, const PagedBatchView& b, uint8_t* bounds,
                                cudaStream_t st) {
  const uint32_t D_ = g.D;
  const bool bf_ = g.bf16 != 0u;
  const uint64_t tiles = ((uint64_t)b.n_tokens >> g.page_lg) + 2ull * b.n_seqs;
  const uint64_t blocks = (tiles * g.H + 3u) / 4u;
  if (blocks > 0x7FFFFFFFull) return cudaErrorInvalidValue;
#define IBP_CALL(L, B) k_paged_bounds<L, B><<<(unsigned)blocks, 128, 0, st>>>(g, b, bounds)
  IBP_PAGED_LANES(IBP_CALL);
#undef IBP_CALL
  return cudaGetLastError();
}

cudaError_t launch_paged_scores(const PagedGeom& g, const PagedBatchView& b, const uint8_t* q,
                                uint64_t q_stride, uint32_t G, const uint8_t* bounds,
                                float* scores, int sm_count, cudaStream_t st) {
  const uint32_t tpt = G >= 16u ? 1u : 16u / G;
  const uint64_t tiles = (uint64_t)b.n_tokens / tpt + b.n_seqs;
  const uint64_t groups = (b.max_pages + kScoreGroup - 1u) / kScoreGroup;
  if (tiles > 0x7FFFFFFFull) return cudaErrorInvalidValue;
  // A row's groups of pages go to as many CTAs as the GPU holds at a time (at most three to
  // an SM, the same number to each tile), so that what a CTA looks up first is paid once:
  // 16 tokens x 8 heads x 2048 pages in 33.6 us (384 CTAs); six to an SM 35.9, two 38.9, one
  // 49.7.  (Tiles that hold rows: the numbers leave gaps.)
  const uint64_t full = b.n_tokens < (uint64_t)tpt * b.n_seqs
                            ? (b.n_tokens < b.n_seqs ? b.n_tokens : b.n_seqs)
                            : (b.n_tokens + tpt - 1u) / tpt;
  uint64_t z = 3ull * sm_count / (full * g.H);
  if (z < 1u) z = 1u;
  const uint64_t per = (groups + 4u * z - 1) / (4u * z);
  z = (groups + 4u * per - 1) / (4u * per);
  if (z > 65535u) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)tiles, g.H, (unsigned)z);
  cfg.blockDim = dim3(128, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
#define IBP_SCORES(B, DP)                                                                    \
  do {                                                                                       \
    const cudaError_t e =                                                                    \
        smem_limit(reinterpret_cast<const void*>(k_paged_scores<B, DP>), score_smem<DP>());  \
    if (e != cudaSuccess) return e;                                                          \
    cfg.dynamicSmemBytes = 4u * kScoreGroup * (g.D * 4u + 16u);                              \
    return cudaLaunchKernelEx(&cfg, k_paged_scores<B, DP>, g, b, q, q_stride, G, bounds,     \
                              scores, (uint32_t)per);                                        \
  } while (0)
  if (g.D <= 64u) {
    if (g.bf16) IBP_SCORES(true, 64);
    else IBP_SCORES(false, 64);
  } else {
    if (g.bf16) IBP_SCORES(true, 128);
    else IBP_SCORES(false, 128);
  }
#undef IBP_SCORES
  return cudaGetLastError();
}

cudaError_t launch_paged_select(const PagedGeom& g, const PagedBatchView& b, const float* scores,
                                uint32_t n_sel, int32_t* selected, int sm_count,
                                cudaStream_t st) {
  // One warp to a row when there are rows for every SM's issue slots (16 warps) and its
  // registers hold them: 7960 rows of 1001 in 23 us, 67 with 8 warps to each.  Else 8
  // warps: 128 rows of 2048 in 6.1 us, 9.1 with one.
  const uint64_t rows = (uint64_t)b.n_tokens * g.H;
  const uint32_t most = b.max_pages;
#define IBP_PICK(W, P, BLOCKS)                                                             \
  k_paged_pick<W, P><<<(unsigned)(BLOCKS), W == 1 ? 128 : W * 32, 0, st>>>(g, b, scores, n_sel, \
                                                                          selected)
  if (rows > 0x7FFFFFFFull) return cudaErrorInvalidValue;
  if (rows >= 16ull * sm_count && most <= 2048u) {
    const uint64_t blocks = (rows + 3u) / 4u;
    if (most <= 256u) IBP_PICK(1, 8, blocks);
    else if (most <= 512u) IBP_PICK(1, 16, blocks);
    else if (most <= 1024u) IBP_PICK(1, 32, blocks);
    else IBP_PICK(1, 64, blocks);
  } else if (most <= 16384u) {
    if (most <= 512u) IBP_PICK(8, 2, rows);
    else if (most <= 2048u) IBP_PICK(8, 8, rows);
    else if (most <= 8192u) IBP_PICK(8, 32, rows);
    else IBP_PICK(8, 64, rows);
  } else {
    k_paged_select<<<dim3(b.n_tokens, g.H), kSelThreads, 0, st>>>(g, b, scores, n_sel, selected);
  }
#undef IBP_PICK
  return cudaGetLastError();
}

}  // namespace ibp
