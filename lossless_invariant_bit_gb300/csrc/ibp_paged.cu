// The paged K/V cache's operators around its attention: appending new keys and
// values (normalised and rotated on the way), bounds of the pages' keys, scores
// of the pages, and the choice of the pages with the largest scores.
#include "ibp_paged.cuh"
#include "ibp_sm103.cuh"

namespace ibp {
namespace {

// ---------------------------------------------------------------- append
// kLanes lanes hold a head, 8 channels (16 bytes) each: the sum of squares is
// a shuffle tree over them, and a channel's rotation partner lies rot/2 channels
// away, a whole number of lanes (rot is a multiple of 16), or in the same lane
// (adjacent pairs).  Every byte is read and written once, 16 at a time.
template <int kLanes, bool kBf16>
__global__ void __launch_bounds__(256) k_paged_append(PagedAppendArgs a) {
  const uint32_t lane = threadIdx.x & (kLanes - 1u);
  const uint32_t heads = a.Hq + 2u * a.g.H;  // queries, keys, values of a token
  const uint64_t item = ((uint64_t)blockIdx.x * 256u + threadIdx.x) / kLanes;
  const bool live = item < (uint64_t)a.b.n_tokens * heads;
  const uint32_t t = live ? (uint32_t)(item / heads) : 0u;
  const uint32_t hh = live ? (uint32_t)(item % heads) : 0u;
  const uint32_t kind = hh < a.Hq ? 0u : hh < a.Hq + a.g.H ? 1u : 2u;
  const uint32_t h = kind == 0u ? hh : kind == 1u ? hh - a.Hq : hh - a.Hq - a.g.H;
  const bool mine = live && lane * 8u < a.g.D;
  uint4 x = make_uint4(0, 0, 0, 0);
  if (mine) {
    const uint8_t* src = kind == 0u   ? a.q + t * a.q_stride
                         : kind == 1u ? a.kx + t * a.kv_stride
                                      : a.vx + t * a.kv_stride;
    x = __ldcs(reinterpret_cast<const uint4*>(src + (uint64_t)h * a.g.D * 2u + lane * 16u));
  }
  // the token's place
  uint32_t s = a.b.n_seqs, pos = 0;
  bool ok = false;
  if (live) {
    s = paged_find(a.b, t);
    if (s < a.b.n_seqs) {
      const PagedSeq q = paged_seq(a.b, a.g.page_lg, s);
      pos = q.L - q.n + (t - q.q0);
      ok = q.ok && q.L >= q.n && (!a.cos_sin || pos < a.n_pos);
      if (!ok && lane == 0) set_status(a.g.status, IBP_ERANGE);
    }
  }
  uint8_t* dst = nullptr;
  if (kind == 0u) {
    dst = a.q_out + t * a.qo_stride + (uint64_t)h * a.g.D * 2u;
    if (s == a.b.n_seqs) dst = nullptr;  // a row of no sequence
  } else if (ok) {
    const int32_t page = __ldg(a.b.table + s * a.b.table_stride + (pos >> a.g.page_lg));
    if (page < 0 || (uint32_t)page >= a.g.n_pages) {
      if (lane == 0) set_status(a.g.status, IBP_ERANGE);
    } else {
      dst = (kind == 1u ? a.g.k : a.g.v) + (uint64_t)(uint32_t)page * a.g.page_stride +
            (pos & ((1u << a.g.page_lg) - 1u)) * a.g.token_stride + h * a.g.head_stride;
    }
  }
  // values pass the same shuffles as their neighbours in the warp, unchanged
  const uint8_t* w = kind == 0u ? a.q_norm : kind == 1u ? a.k_norm : nullptr;
  const bool turned = a.cos_sin && kind != 2u;
  float f[8];
  {
    const float2 f0 = unpack2(x.x, kBf16), f1 = unpack2(x.y, kBf16), f2 = unpack2(x.z, kBf16),
                 f3 = unpack2(x.w, kBf16);
    f[0] = f0.x, f[1] = f0.y, f[2] = f1.x, f[3] = f1.y;
    f[4] = f2.x, f[5] = f2.y, f[6] = f3.x, f[7] = f3.y;
  }
  if (a.q_norm || a.k_norm) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(f[i], f[i], ss);
#pragma unroll
    for (int d = kLanes / 2; d; d >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, d);
    if (w && mine) {
      const float r = rsqrtf(ss / (float)a.g.D + a.eps);
      const uint4 g = __ldg(reinterpret_cast<const uint4*>(w) + lane);
      const uint32_t gw[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 gf = unpack2(gw[i], kBf16);
        f[2 * i] *= r * gf.x;
        f[2 * i + 1] *= r * gf.y;
      }
    }
  }
  if (a.cos_sin) {
    const float* cs = a.cos_sin + (uint64_t)(ok ? pos : 0u) * a.rot;
    const uint32_t half = a.rot / 2u, c0 = lane * 8u;
    if (a.pairs) {
      if (turned && c0 < a.rot) {
        const float4 c = __ldg(reinterpret_cast<const float4*>(cs + c0 / 2u));
        const float4 n = __ldg(reinterpret_cast<const float4*>(cs + half + c0 / 2u));
        const float cc[4] = {c.x, c.y, c.z, c.w}, nn[4] = {n.x, n.y, n.z, n.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float u = f[2 * i], v = f[2 * i + 1];
          f[2 * i] = u * cc[i] - v * nn[i];
          f[2 * i + 1] = v * cc[i] + u * nn[i];
        }
      }
    } else {
      const bool low = c0 < half;
      const uint32_t hl = half / 8u;
      const uint32_t base = (threadIdx.x & 31u) & ~(kLanes - 1u);
      const uint32_t from = base + ((low ? lane + hl : lane - hl) & (kLanes - 1u));
      float p[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i] = __shfl_sync(0xFFFFFFFFu, f[i], from);
      if (turned && c0 < a.rot) {
        const float4* c4 = reinterpret_cast<const float4*>(cs + (low ? c0 : c0 - half));
        const float4* n4 = reinterpret_cast<const float4*>(cs + half + (low ? c0 : c0 - half));
        const float4 ca = __ldg(c4), cb = __ldg(c4 + 1), na = __ldg(n4), nb = __ldg(n4 + 1);
        const float cc[8] = {ca.x, ca.y, ca.z, ca.w, cb.x, cb.y, cb.z, cb.w};
        const float nn[8] = {na.x, na.y, na.z, na.w, nb.x, nb.y, nb.z, nb.w};
#pragma unroll
        for (int i = 0; i < 8; ++i)
          f[i] = low ? f[i] * cc[i] - p[i] * nn[i] : f[i] * cc[i] + p[i] * nn[i];
      }
    }
  }
  if (w || turned) {
    x.x = pack2(f[0], f[1], kBf16);
    x.y = pack2(f[2], f[3], kBf16);
    x.z = pack2(f[4], f[5], kBf16);
    x.w = pack2(f[6], f[7], kBf16);
  }
  if (kind == 0u && !ok) x = make_uint4(0, 0, 0, 0);
  if (mine && dst) *reinterpret_cast<uint4*>(dst + lane * 16u) = x;
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
  const uint32_t lane = threadIdx.x & 31u, sub = lane & (kLanes - 1u), row = lane / kLanes;
  const uint64_t id = (uint64_t)blockIdx.x * 4u + (threadIdx.x >> 5);
  const uint32_t tile = (uint32_t)(id / g.H), h = (uint32_t)(id % g.H);
  const uint32_t P = 1u << g.page_lg;
  uint32_t first;
  const uint32_t s = paged_find_tile(b, P, 2u, tile, first);
  const PagedSeq q = paged_seq(b, g.page_lg, s);
  if (!q.ok || q.L < q.n) {
    if (lane == 0) set_status(g.status, IBP_ERANGE);
    return;
  }
  if (q.n == 0 || tile < first) return;
  const uint32_t p = ((q.L - q.n) >> g.page_lg) + (tile - first);
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
// allow; 16 of the G queries at a time when G > 16) as the left operand and
// goes over pages, 8 to a matrix instruction.  The sum runs over the
// channels in any order, so a lane takes 8 channels together (one 16-byte
// load) where the instruction's layout wants pairs: four lanes cover 64 bytes
// of a page's bounds, straight from global memory into the operand's registers.
constexpr uint32_t kScoreGroup = 32;  // pages between two stores of scores

template <bool kBf16, int kDP>
__global__ void __launch_bounds__(128)
    k_paged_scores(PagedGeom g, PagedBatchView b, const uint8_t* q, uint64_t q_stride, uint32_t G,
                   const uint8_t* bounds, float* scores, uint32_t per_warp) {
  constexpr int kC = kDP / 32;  // 16-byte chunks per lane
  __shared__ float s_c[4][16][kScoreGroup + 1];
  const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31u;
  const uint32_t quad = lane & 3u, r0 = lane >> 2;
  const uint32_t tpt = G >= 16u ? 1u : 16u / G;  // tokens of a tile
  const uint32_t h = blockIdx.y;
  uint32_t first;
  const uint32_t s = paged_find_tile(b, tpt, 1u, blockIdx.x, first);
  const PagedSeq sq = paged_seq(b, g.page_lg, s);
  if (!sq.ok) {
    if (threadIdx.x == 0) set_status(g.status, IBP_ERANGE);
  }
  const uint32_t t0 = (blockIdx.x - first) * tpt;
  if (blockIdx.x < first || t0 >= sq.n) return;
  const uint32_t nt = min(tpt, sq.n - t0);
  const uint32_t groups = (b.max_pages + kScoreGroup - 1u) / kScoreGroup;
  const uint32_t g0 = (blockIdx.z * 4u + warp) * per_warp;
  const uint32_t g1 = min(groups, g0 + per_warp);
  const int64_t pos_last = (int64_t)sq.L - sq.n + t0 + nt - 1;
  const uint32_t seen_last = pos_last < 0 ? 0u : (uint32_t)(pos_last >> g.page_lg) + 1u;
  uint32_t qp[kC * 4 * 2], qn[kC * 4 * 2];  // [chunk][4 words][row, row + 8]
  for (uint32_t gr = g0; gr < g1; ++gr) {
    const uint32_t c0 = gr * kScoreGroup;
    float best = 0.f;  // over the queries of the earlier row blocks (G > 16)
    if (c0 < seen_last) {
      int32_t id = -1;
      if (c0 + lane < seen_last) {
        id = __ldg(b.table + s * b.table_stride + c0 + lane);
        if (id < 0 || (uint32_t)id >= g.n_pages) {
          set_status(g.status, IBP_ERANGE);
          id = -1;
        }
      }
      for (uint32_t rb = 0; rb * 16u < (tpt == 1u ? G : 16u); ++rb) {
        if (gr == g0 || G > 16u) {  // the rows' queries, split by sign
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
              const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                qp[(c * 4 + i) * 2 + e] = max2<kBf16>(w[i], 0u);
                qn[(c * 4 + i) * 2 + e] = min2<kBf16>(w[i], 0u);
              }
            }
          }
        }
#pragma unroll
        for (uint32_t nt8 = 0; nt8 < kScoreGroup / 8u; ++nt8) {
          const int32_t pid = __shfl_sync(0xFFFFFFFFu, id, nt8 * 8u + r0);
          float acc[4] = {0.f, 0.f, 0.f, 0.f};
          uint4 lo[kC], hi[kC];
          const uint8_t* src =
              bounds + ((uint64_t)(uint32_t)(pid < 0 ? 0 : pid) * g.H + h) * g.D * 4u;
#pragma unroll
          for (int c = 0; c < kC; ++c) {
            const uint32_t ch = 32u * c + 8u * quad;
            lo[c] = hi[c] = make_uint4(0, 0, 0, 0);
            if (pid >= 0 && ch < g.D) {
              lo[c] = __ldg(reinterpret_cast<const uint4*>(src + ch * 2u));
              hi[c] = __ldg(reinterpret_cast<const uint4*>(src + (g.D + ch) * 2u));
            }
          }
#pragma unroll
          for (int c = 0; c < kC; ++c) {
            const uint32_t* p = qp + c * 8;
            const uint32_t* n = qn + c * 8;
            mma_16816<kBf16>(acc, p, hi[c].x, hi[c].y);
            mma_16816<kBf16>(acc, p + 4, hi[c].z, hi[c].w);
            mma_16816<kBf16>(acc, n, lo[c].x, lo[c].y);
            mma_16816<kBf16>(acc, n + 4, lo[c].z, lo[c].w);
          }
          float* d0 = &s_c[warp][r0][nt8 * 8u + 2u * quad];
          float* d1 = &s_c[warp][r0 + 8u][nt8 * 8u + 2u * quad];
          d0[0] = acc[0], d0[1] = acc[1], d1[0] = acc[2], d1[1] = acc[3];
        }
        __syncwarp();
        // the largest over each token's queries, kept by the lane of the page
        const uint32_t rows = tpt == 1u ? min(16u, G - rb * 16u) : G;
        for (uint32_t tt = 0; tt < nt; ++tt) {
          float m = s_c[warp][tt * G][lane];
          for (uint32_t i = 1; i < rows; ++i) {
            const float v = s_c[warp][tt * G + i][lane];
            m = (v > m || v != v) ? v : m;
          }
          if (tpt == 1u && rb) m = (best > m || best != best) ? best : m;
          best = m;
          const int64_t pos = (int64_t)sq.L - sq.n + t0 + tt;
          const bool seen = pos >= 0 && c0 + lane <= (uint32_t)(pos >> g.page_lg) && id >= 0;
          if (c0 + lane < b.max_pages && (rb + 1u) * 16u >= (tpt == 1u ? G : 16u))
            scores[((uint64_t)(sq.q0 + t0 + tt) * g.H + h) * b.max_pages + c0 + lane] =
                seen ? m : __int_as_float((int)0xFF800000u);
        }
        __syncwarp();
      }
    } else {
      for (uint32_t tt = 0; tt < nt; ++tt)
        if (c0 + lane < b.max_pages)
          scores[((uint64_t)(sq.q0 + t0 + tt) * g.H + h) * b.max_pages + c0 + lane] =
              __int_as_float((int)0xFF800000u);
    }
  }
}

// ---------------------------------------------------------------- select
// One CTA per (token, K/V head).  Scores become whole numbers of the same order
// (the sign bit folded in, NaN above all, the token's own page above that); the
// n_sel-th largest is found digit by digit, 8 bits from the top, with a
// histogram of the candidates that share the digits found so far; then one
// ordered pass writes the numbers above it and the first of those equal to it.
constexpr uint32_t kSelThreads = 256, kSelKeys = 8192;

__device__ __forceinline__ uint32_t order_key(float f) {
  if (f != f) return 0xFFFFFFFEu;
  const uint32_t u = __float_as_uint(f + 0.f);  // -0 counts as 0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(256)
    k_paged_select(PagedGeom g, PagedBatchView b, const float* scores, uint32_t n_sel,
                   int32_t* selected) {
  __shared__ uint32_t s_key[kSelKeys];
  __shared__ uint32_t s_hist[256];
  __shared__ uint32_t s_warp[2][8];
  __shared__ uint32_t s_pick[2];
  const uint32_t t = blockIdx.x, h = blockIdx.y, tid = threadIdx.x;
  const uint32_t warp = tid >> 5, lane = tid & 31u;
  int32_t* out = selected + ((uint64_t)t * g.H + h) * n_sel;
  const uint32_t s = paged_find(b, t);
  if (s == b.n_seqs) return;
  const PagedSeq q = paged_seq(b, g.page_lg, s);
  const int64_t pos = (int64_t)q.L - q.n + (t - q.q0);
  if (!q.ok && tid == 0) set_status(g.status, IBP_ERANGE);
  const uint32_t own = pos < 0 ? 0u : (uint32_t)(pos >> g.page_lg);
  const uint32_t n = !q.ok || pos < 0 ? 0u : own + 1u;  // pages to choose from
  if (n <= n_sel) {
    for (uint32_t i = tid; i < n_sel; i += kSelThreads) out[i] = i < n ? (int32_t)i : -1;
    return;
  }
  const float* row = scores + ((uint64_t)t * g.H + h) * b.max_pages;
  const bool held = n <= kSelKeys;
  for (uint32_t i = tid; held && i < n; i += kSelThreads)
    s_key[i] = i == own ? 0xFFFFFFFFu : order_key(__ldg(row + i));
  auto key = [&](uint32_t i) {
    return held ? s_key[i] : i == own ? 0xFFFFFFFFu : order_key(__ldg(row + i));
  };
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

#define IBP_PAGED_LANES(KERN, GRID, BLOCK, ...)                                              \
  do {                                                                                       \
    const uint32_t ln = pow2_lanes(D_);                                                      \
    if (bf_) {                                                                               \
      if (ln == 4u) KERN<4, true><<<GRID, BLOCK, 0, st>>>(__VA_ARGS__);                      \
      else if (ln == 8u) KERN<8, true><<<GRID, BLOCK, 0, st>>>(__VA_ARGS__);                 \
      else KERN<16, true><<<GRID, BLOCK, 0, st>>>(__VA_ARGS__);                              \
    } else {                                                                                 \
      if (ln == 4u) KERN<4, false><<<GRID, BLOCK, 0, st>>>(__VA_ARGS__);                     \
      else if (ln == 8u) KERN<8, false><<<GRID, BLOCK, 0, st>>>(__VA_ARGS__);                \
      else KERN<16, false><<<GRID, BLOCK, 0, st>>>(__VA_ARGS__);                             \
    }                                                                                        \
  } while (0)

cudaError_t launch_paged_append(const PagedAppendArgs& a, cudaStream_t st) {
  const uint32_t D_ = a.g.D;
  const bool bf_ = a.g.bf16 != 0u;
  const uint64_t items = (uint64_t)a.b.n_tokens * (a.Hq + 2ull * a.g.H);
  const uint64_t per = 256u / pow2_lanes(D_);
  const uint64_t blocks = (items + per - 1) / per;
  if (blocks > 0x7FFFFFFFull) return cudaErrorInvalidValue;
  IBP_PAGED_LANES(k_paged_append, (unsigned)blocks, 256, a);
  return cudaGetLastError();
}

cudaError_t launch_paged_bounds(const PagedGeom& g, const PagedBatchView& b, uint8_t* bounds,
                                cudaStream_t st) {
  const uint32_t D_ = g.D;
  const bool bf_ = g.bf16 != 0u;
  const uint64_t tiles = ((uint64_t)b.n_tokens >> g.page_lg) + 2ull * b.n_seqs;
  const uint64_t blocks = (tiles * g.H + 3u) / 4u;
  if (blocks > 0x7FFFFFFFull) return cudaErrorInvalidValue;
  IBP_PAGED_LANES(k_paged_bounds, (unsigned)blocks, 128, g, b, bounds);
  return cudaGetLastError();
}

cudaError_t launch_paged_scores(const PagedGeom& g, const PagedBatchView& b, const uint8_t* q,
                                uint64_t q_stride, uint32_t G, const uint8_t* bounds,
                                float* scores, int sm_count, cudaStream_t st) {
  const uint32_t tpt = G >= 16u ? 1u : 16u / G;
  const uint64_t tiles = (uint64_t)b.n_tokens / tpt + b.n_seqs;
  const uint64_t groups = (b.max_pages + kScoreGroup - 1u) / kScoreGroup;
  if (tiles > 0x7FFFFFFFull) return cudaErrorInvalidValue;
  // enough warps to fill the GPU, as many groups of pages as that leaves to each
  const uint64_t rows = tiles * g.H;
  uint64_t per = (groups * rows + 24ull * sm_count - 1) / (24ull * sm_count);
  if (per > 16u) per = 16u;
  if (per < 1u) per = 1u;
  const uint64_t z = (groups + 4u * per - 1) / (4u * per);
  if (z > 65535u) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)tiles, g.H, (unsigned)z);
  if (g.D <= 64u) {
    if (g.bf16)
      k_paged_scores<true, 64><<<grid, 128, 0, st>>>(g, b, q, q_stride, G, bounds, scores,
                                                     (uint32_t)per);
    else
      k_paged_scores<false, 64><<<grid, 128, 0, st>>>(g, b, q, q_stride, G, bounds, scores,
                                                      (uint32_t)per);
  } else {
    if (g.bf16)
      k_paged_scores<true, 128><<<grid, 128, 0, st>>>(g, b, q, q_stride, G, bounds, scores,
                                                      (uint32_t)per);
    else
      k_paged_scores<false, 128><<<grid, 128, 0, st>>>(g, b, q, q_stride, G, bounds, scores,
                                                       (uint32_t)per);
  }
  return cudaGetLastError();
}

cudaError_t launch_paged_select(const PagedGeom& g, const PagedBatchView& b, const float* scores,
                                uint32_t n_sel, int32_t* selected, cudaStream_t st) {
  k_paged_select<<<dim3(b.n_tokens, g.H), kSelThreads, 0, st>>>(g, b, scores, n_sel, selected);
  return cudaGetLastError();
}

}  // namespace ibp
