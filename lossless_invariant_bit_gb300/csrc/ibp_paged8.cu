// The operators around the attention of a paged K/V cache held in 8 bits: appending keys
// and values as codes under their pages' scales, and bounds of the pages' keys.
#include "ibp_paged8.cuh"
#include "ibp_sm103.cuh"

namespace ibp {
namespace {

// The byte of the smallest scale 2^e with m <= 448 * 2^e: 448 = 1.75 * 2^8.
__device__ __forceinline__ uint32_t scale_for(float m) {
  const uint32_t bits = __float_as_uint(m);  // (m is not negative, and finite)
  const int32_t e = (int32_t)(bits >> 23) - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return (uint32_t)min(max(e, (int32_t)kScaleLow), (int32_t)kScaleHigh);
}

// Two values over a scale as two codes: to the nearest, ties to even, what the largest scale
// does not hold the largest code; NaN stays NaN.
__device__ __forceinline__ uint32_t codes2(uint64_t x, uint64_t inv) {
  uint16_t r;
  float lo, hi;
  halves2(mul2(x, inv), lo, hi);
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Infinities become NaN (x * 0 is).
__device__ __forceinline__ uint64_t without_inf(uint64_t x) { return fma2(x, 0ull, x); }

// Four codes under a larger scale.
__device__ __forceinline__ uint32_t rescale4(uint32_t x, float f) {
  uint32_t p[2];
  codes_to_fp16(x, p[0], p[1]);
  const float2 u = unpack2(p[0], 0u), v = unpack2(p[1], 0u);
  const uint64_t f2 = pair2(f, f);
  return codes2(pair2(u.x, u.y), f2) | codes2(pair2(v.x, v.y), f2) << 16;
}

// ---------------------------------------------------------------- append
// Codes of a page and head share a scale, so a unit of 2^unit_lg threads takes all new
// tokens of one (page, head) of the keys or of the values: it computes them, finds the
// largest magnitude, then rounds.  Values stay in registers between the two (kTokens tokens
// of 8 channels a thread); pages with more tokens than that go through twice, from the
// caches the second time.  A lane's channels are the 16-bit append's: 4 and their
// rotation partners.
//
// Bound by issue: 9.2 million warp instructions for the 5864 tokens x 16 heads of a prefill, of
// both kinds (norm, rotation, maximum, rounding); alone 21 us, beside the queries' kernel (42,
// issue too) 54.9 for both, 4.2 TB/s.  Keys, values and queries in one kernel 60 to 67; this
// kernel's CTAs ahead of the queries' 56 to 57.5.  A step of 20 tokens: 6.6 us, look-ups.
template <int kLanes, bool kBf16, bool kPairs>
__device__ __forceinline__ void append_units(const PagedAppendArgs& a, uint32_t unit_lg,
                                             uint32_t per) {
  constexpr int kTokens = 4;
  __shared__ float s_top[4];
  const uint32_t unit = 1u << unit_lg, tid = threadIdx.x;
  const uint32_t ut = tid & (unit - 1u);  // thread of the unit
  const uint32_t lane = ut & (kLanes - 1u), row = ut / kLanes, rows = unit / kLanes;
  const uint32_t P = 1u << a.g.page_lg;
  uint32_t first;
  const uint32_t s = paged_find_tile(a.b, P, 2u, blockIdx.x, first);
  const PagedSeq q = paged_seq(a.b, a.g.page_lg, s);
  if (!q.ok) {
    if (tid == 0) set_status(a.g.status, IBP_ERANGE);
    return;
  }
  if (q.n == 0 || blockIdx.x < first) return;
  if (q.n > q.L && tid == 0) set_status(a.g.status, IBP_ERANGE);  // tokens without a position
  if (q.L == 0) return;
  const uint32_t from = q.L > q.n ? q.L - q.n : 0u;  // the first new token that has a position
  const uint32_t page_at = (from >> a.g.page_lg) + (blockIdx.x - first);
  if (page_at > (q.L - 1u) >> a.g.page_lg) return;
  const int32_t page = __ldg(a.b.table + s * a.b.table_stride + page_at);
  if (page < 0 || (uint32_t)page >= a.g.n_pages) {
    if (tid == 0) set_status(a.g.status, IBP_ERANGE);
    return;
  }
  // the page's new tokens: slots [t0, t1); before them, what it holds
  const uint32_t p0 = page_at << a.g.page_lg;
  const uint32_t t0 = max(from, p0) - p0;
  uint32_t t1 = min(q.L - p0, P);
  if (a.cos_sin && p0 + t1 > a.n_pos) {
    if (tid == 0) set_status(a.g.status, IBP_ERANGE);
    t1 = a.n_pos > p0 ? a.n_pos - p0 : 0u;
  }
  if (t1 <= t0) return;
  const uint64_t next_row = rows * a.kv_stride, next_slot = rows * a.g.token_stride;
  // the CTA's units, a round of 128 / unit of them at a time: keys' heads, then values'
  for (uint32_t round = 0; round < per; ++round) {
    const uint32_t u = (blockIdx.y * per + round) * (128u >> unit_lg) + (tid >> unit_lg);
    const bool live = u < 2u * a.g.H, keys = u < a.g.H;
    const uint32_t h = !live ? 0u : keys ? u : u - a.g.H;
    uint8_t* scale = (keys ? a.g.k_scales : a.g.v_scales) + (uint64_t)(uint32_t)page * a.g.H + h;
    uint32_t was = t0 && live ? *scale : 0u;
    const bool mine = live && lane * 8u < a.g.D;
    const uint32_t half = a.rot / 2u;
    const bool turned = keys && lane * 8u < a.rot, split = !kPairs && lane * 8u < a.rot;
    const uint32_t c0 = split ? lane * 4u : lane * 8u, c1 = split ? half + lane * 4u : c0 + 4u;
    // row of slot t in the call's arrays: q0 + (p0 + t) - (L - n)
    const uint8_t* src = (keys ? a.kx : a.vx) + (uint64_t)h * a.g.D * 2u + c0 * 2u;
    const uint32_t apart = c1 - c0;
    const int64_t row0 = (int64_t)q.q0 + p0 - ((int64_t)q.L - q.n);
    uint8_t* dst = (keys ? a.g.k : a.g.v) + (uint64_t)(uint32_t)page * a.g.page_stride +
                   h * a.g.head_stride + c0;
    uint64_t w[4] = {};  // the norm's weights
    if (a.k_norm && mine) {
      const uint2 x = __ldg(reinterpret_cast<const uint2*>(a.k_norm + c0 * 2u));
      const uint2 y = __ldg(reinterpret_cast<const uint2*>(a.k_norm + c1 * 2u));
      const uint32_t z[4] = {x.x, x.y, y.x, y.y};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f = unpack2(z[k], kBf16);
        w[k] = pair2(f.x, f.y);
      }
    }
    const float inv_d = 1.f / (float)a.g.D;
    uint64_t f[kTokens][4];
    // the values of the unit's tokens from slot `at` on
    auto compute = [&](uint32_t at) {
      uint2 x[kTokens][2];
      const uint8_t* p = src + (uint64_t)(row0 + at + row) * a.kv_stride;
#pragma unroll
      for (int i = 0; i < kTokens; ++i, p += next_row) {
        const uint32_t t = at + i * rows + row;
        x[i][0] = x[i][1] = make_uint2(0u, 0u);
        if (mine && t >= t0 && t < t1) {
          x[i][0] = __ldg(reinterpret_cast<const uint2*>(p));
          x[i][1] = __ldg(reinterpret_cast<const uint2*>(p + 2u * apart));
        }
      }
      const float* cs = a.cos_sin + (uint64_t)(p0 + at + row) * a.rot + lane * 4u;
#pragma unroll
      for (int i = 0; i < kTokens; ++i, cs += rows * a.rot) {
        const uint32_t t = at + i * rows + row;
        const uint32_t z[4] = {x[i][0].x, x[i][0].y, x[i][1].x, x[i][1].y};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 v = unpack2(z[k], kBf16);
          f[i][k] = pair2(v.x, v.y);
        }
        if (a.k_norm && (keys || unit < 32u)) {  // (all lanes of a warp, or none)
          uint64_t s2 = mul2(f[i][0], f[i][0]);
#pragma unroll
          for (int k = 1; k < 4; ++k) s2 = fma2(f[i][k], f[i][k], s2);
          float sum, odd;
          halves2(s2, sum, odd);
          sum += odd;
#pragma unroll
          for (int d = kLanes / 2; d; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
          const float n = rsqrtf(fmaf(sum, inv_d, a.eps));
          if (keys)
#pragma unroll
            for (int k = 0; k < 4; ++k) f[i][k] = mul2(f[i][k], mul2(pair2(n, n), w[k]));
        }
        if (a.cos_sin && turned && t >= t0 && t < t1) {
          const float4 cc = __ldg(reinterpret_cast<const float4*>(cs));
          const float4 ss = __ldg(reinterpret_cast<const float4*>(cs + half));
          if (kPairs) {
            const float c4[4] = {cc.x, cc.y, cc.z, cc.w}, s4[4] = {ss.x, ss.y, ss.z, ss.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              float x0, x1;
              halves2(f[i][k], x0, x1);
              f[i][k] = fma2(f[i][k], pair2(c4[k], c4[k]), mul2(pair2(-x1, x0), pair2(s4[k], s4[k])));
            }
          } else {
            const uint64_t c2[2] = {pair2(cc.x, cc.y), pair2(cc.z, cc.w)};
            const uint64_t s2[2] = {pair2(ss.x, ss.y), pair2(ss.z, ss.w)};
            const uint64_t m2[2] = {pair2(-ss.x, -ss.y), pair2(-ss.z, -ss.w)};
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint64_t x0 = f[i][k], x1 = f[i][k + 2];
              f[i][k] = fma2(x0, c2[k], mul2(x1, m2[k]));
              f[i][k + 2] = fma2(x1, c2[k], mul2(x0, s2[k]));
            }
          }
        }
      }
    };
    const uint32_t step = rows * kTokens;
    const uint32_t begin = t0 & ~(step - 1u);
    uint32_t at;
    float top;
    // The largest magnitude (NaN have no part in it); where it is infinite, once more without
    // infinities, which become NaN codes.
    bool odd = false;
    while (true) {
      top = 0.f;
      for (at = begin;; at += step) {
        compute(at);
#pragma unroll
        for (int i = 0; i < kTokens; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (odd) f[i][k] = without_inf(f[i][k]);
            float x, y;
            halves2(f[i][k], x, y);
            top = fmaxf(top, fmaxf(fabsf(x), fabsf(y)));
          }
        if (at + step >= t1) break;
      }
      for (uint32_t d = 1; d < (unit < 32u ? unit : 32u); d <<= 1)
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
      if (unit > 32u) {
        __syncthreads();  // (what the last round wrote there has been read)
        if ((tid & 31u) == 0u) s_top[tid >> 5] = top;
        __syncthreads();
        const uint32_t w0 = tid >> unit_lg << (unit_lg - 5u);
        for (uint32_t i = 0; i < unit / 32u; ++i) top = fmaxf(top, s_top[w0 + i]);
      }
      if (odd || !__syncthreads_or(top == INFINITY)) break;
      odd = true;
    }
    uint32_t byte = scale_for(top);
    if (t0 && live) {
      if (scale_ok(was)) {
        byte = max(byte, was);
      } else {
        if (ut == 0) set_status(a.g.status, IBP_ERANGE);
        was = byte;  // what the page holds has no value: it is left
      }
      if (byte > was) {  // the codes that it holds, under the new scale
        const float down = scale_of(127u + was - byte);
        for (uint32_t t = row; t < t0; t += rows)
          if (mine) {
            uint32_t* p0 = reinterpret_cast<uint32_t*>(dst + t * a.g.token_stride);
            uint32_t* p1 = reinterpret_cast<uint32_t*>(dst + t * a.g.token_stride + apart);
            *p0 = rescale4(*p0, down);
            *p1 = rescale4(*p1, down);
          }
      }
    }
    if (ut == 0 && live) *scale = (uint8_t)byte;
    const float down = scale_of(254u - byte);
    const uint64_t inv = pair2(down, down);
    // backwards, beginning with what is still in registers
    for (;; at -= step) {
      uint8_t* d = dst + (at + row) * a.g.token_stride;
#pragma unroll
      for (int i = 0; i < kTokens; ++i, d += next_slot) {
        const uint32_t t = at + i * rows + row;
        if (!mine || t < t0 || t >= t1) continue;
        uint32_t z[2];
#pragma unroll
        for (int k = 0; k < 2; ++k)
          z[k] = codes2(f[i][2 * k], inv) | codes2(f[i][2 * k + 1], inv) << 16;
        *reinterpret_cast<uint32_t*>(d) = z[0];
        *reinterpret_cast<uint32_t*>(d + apart) = z[1];
      }
      if (at == begin) break;
      compute(at - step);
      if (odd)
#pragma unroll
        for (int i = 0; i < kTokens; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) f[i][k] = without_inf(f[i][k]);
    }
  }
}

// Behind the kernel of the queries, beside which it may run; it ends after it, so that what
// follows may count on both.
template <int kLanes, bool kBf16, bool kPairs>
__global__ void __launch_bounds__(128) k_paged8_append(PagedAppendArgs a, uint32_t unit_lg,
                                                       uint32_t per) {
  append_units<kLanes, kBf16, kPairs>(a, unit_lg, per);
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ---------------------------------------------------------------- bounds
// One warp per (page that got new tokens, head), 16 channels per lane: minima and maxima of
// the codes as fp16 (exact), then the scale, then one rounding to the 16-bit type (none for
// what an append has written, but beyond that type's range).  8 loads of 16 bytes in flight to
// a lane: 34 thousand tokens 11.3 us, 3.5 TB/s (4 in flight: 13.3), half of it start and look-ups
// of two waves of CTAs; 16 tokens 2.9.
template <int kLanes, bool kBf16>
__global__ void __launch_bounds__(128)
    k_paged8_bounds(PagedGeom g, PagedBatchView b, uint8_t* bounds) {
  // the scores' CTAs may come up beside this kernel (they wait for its end)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr uint32_t kAhead = 8;
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
  const uint32_t from = q.L > q.n ? q.L - q.n : 0u;
  const uint32_t p = (from >> g.page_lg) + (tile - first);
  if (p > (q.L - 1u) >> g.page_lg) return;
  const int32_t page = __ldg(b.table + s * b.table_stride + p);
  if (page < 0 || (uint32_t)page >= g.n_pages) {
    if (lane == 0) set_status(g.status, IBP_ERANGE);
    return;
  }
  const uint32_t byte = __ldg(g.k_scales + (uint64_t)(uint32_t)page * g.H + h);
  const uint32_t held = min(P, q.L - p * P);
  const uint8_t* src = g.k + (uint64_t)(uint32_t)page * g.page_stride + h * g.head_stride +
                       sub * 16u;
  const bool mine = sub * 16u < g.D;
  __half2 lo[8], hi[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lo[i] = __half2half2(__ushort_as_half(0x7C00u));
    hi[i] = __half2half2(__ushort_as_half(0xFC00u));
  }
  if (mine)
    for (uint32_t t0 = row; t0 < held; t0 += kAhead * (32u / kLanes)) {
      uint4 x[kAhead];  // on their way together; behind the last, the first once more
#pragma unroll
      for (uint32_t i = 0; i < kAhead; ++i) {
        const uint32_t t = t0 + i * (32u / kLanes);
        x[i] = __ldg(reinterpret_cast<const uint4*>(src + (t < held ? t : t0) * g.token_stride));
      }
#pragma unroll
      for (uint32_t k = 0; k < kAhead; ++k) {
        const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t y[2];
          codes_to_fp16(w[i], y[0], y[1]);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const __half2 v = *reinterpret_cast<const __half2*>(&y[k]);
            lo[2 * i + k] = __hmin2_nan(lo[2 * i + k], v);
            hi[2 * i + k] = __hmax2_nan(hi[2 * i + k], v);
          }
        }
      }
    }
  if (!scale_ok(byte)) {
    if (lane == 0) set_status(g.status, IBP_ERANGE);
    return;
  }
#pragma unroll
  for (int d = kLanes; d < 32; d <<= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      lo[i] = __hmin2_nan(lo[i], __shfl_xor_sync(0xFFFFFFFFu, lo[i], d));
      hi[i] = __hmax2_nan(hi[i], __shfl_xor_sync(0xFFFFFFFFu, hi[i], d));
    }
  if (mine && row == 0) {
    const float f = scale_of(byte);
    uint8_t* dst = bounds + ((uint64_t)(uint32_t)page * g.H + h) * g.D * 4u + sub * 32u;
    uint32_t y[8], z[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 u = __half22float2(lo[i]), v = __half22float2(hi[i]);
      y[i] = pack2(u.x * f, u.y * f, kBf16);
      z[i] = pack2(v.x * f, v.y * f, kBf16);
    }
    reinterpret_cast<uint4*>(dst)[0] = make_uint4(y[0], y[1], y[2], y[3]);
    reinterpret_cast<uint4*>(dst)[1] = make_uint4(y[4], y[5], y[6], y[7]);
    reinterpret_cast<uint4*>(dst + g.D * 2u)[0] = make_uint4(z[0], z[1], z[2], z[3]);
    reinterpret_cast<uint4*>(dst + g.D * 2u)[1] = make_uint4(z[4], z[5], z[6], z[7]);
  }
}

// ---------------------------------------------------------------- 16-bit pages
// Codes times scales as bf16 (exact), one head after the other, for the pages that the chunk
// kernel reads, in parts of 1024 units of 16 channels.  A sequence's keys (or values) are
// shared out over gridDim.z CTAs: what its table has room for beyond them costs nothing.
// The kernel on codes converts a tile's keys once for every 256 rows, 4400 cycles a block of
// 128 keys; of converted pages a block takes 2800, and the conversion, bound by the bytes, of
// 8192 tokens x 8 heads of 128 (16.8 MB to 33.5 MB) 13.6 us from a cold cache (16.2 with one
// load in flight).  A head's table has no page where one cannot be read.
constexpr uint32_t kStageUnits = 4;  // units of a thread, their loads in flight
constexpr uint32_t kStagePart = 256u * kStageUnits;

__global__ void __launch_bounds__(256) k_paged8_stage(PagedAttnArgs a, PagedAttnArgs to) {
  const uint32_t s = blockIdx.x;
  const PagedSeq q = paged_seq(a.b, a.g.page_lg, s);
  if (q.n == 0 || q.n * a.G <= a.max_rows) return;
  const uint32_t lg = a.g.page_lg, H = a.g.H;
  const uint32_t chunks = a.g.D / 16u, rows = chunks << lg, units = rows * H;
  const uint32_t parts = (units + kStagePart - 1u) / kStagePart;
  const int64_t first = (int64_t)q.L - q.n;
  const int64_t lo = a.window ? first + 1 - (int64_t)a.window : 0;
  const uint32_t i0 = lo > 0 ? (uint32_t)lo >> lg : 0u, i1 = (q.L + (1u << lg) - 1u) >> lg;
  const bool values = blockIdx.y != 0u;
  const uint8_t* codes = values ? a.g.v : a.g.k;
  const uint8_t* bytes = values ? a.g.v_scales : a.g.k_scales;
  for (uint32_t i = i0 + blockIdx.z / parts, part = blockIdx.z % parts; i < i1;) {
    const uint32_t at = s * a.b.max_pages + i;  // the page of what is made
    const int32_t page = __ldg(a.b.table + s * a.b.table_stride + i);
    const bool there = page >= 0 && (uint32_t)page < a.g.n_pages;
    if (!values && part == 0u)
      for (uint32_t h = threadIdx.x; h < H; h += blockDim.x)
        const_cast<int32_t*>(to.b.table)[s * to.b.table_stride + h * to.b.table_heads + i] =
            there && scales_ok(page_scales(a.g, (uint32_t)page, h)) ? (int32_t)at : -1;
    if (there) {
      const uint8_t* src = codes + (uint64_t)(uint32_t)page * a.g.page_stride;
      const uint8_t* scales = bytes + (uint64_t)(uint32_t)page * H;
      uint8_t* dst = (values ? to.g.v : to.g.k) + (uint64_t)at * to.g.page_stride;
      const uint32_t x0 = part * kStagePart + threadIdx.x;
      uint4 v[kStageUnits];
      float f[kStageUnits];
#pragma unroll
      for (uint32_t u = 0; u < kStageUnits; ++u) {
        const uint32_t x = x0 + 256u * u;
        if (x >= units) break;
        const uint32_t h = x / rows, r = x - h * rows, t = r / chunks, c = r - t * chunks;
        v[u] = __ldg(reinterpret_cast<const uint4*>(src + t * a.g.token_stride +
                                                    h * a.g.head_stride + c * 16u));
        f[u] = scale_of(__ldg(scales + h));
      }
#pragma unroll
      for (uint32_t u = 0; u < kStageUnits; ++u) {
        const uint32_t x = x0 + 256u * u;
        if (x >= units) break;
        const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
        uint32_t y[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t p[2];
          codes_to_fp16(w[k], p[0], p[1]);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float2 z = unpack2(p[j], 0u);
            y[2 * k + j] = pack2(z.x * f[u], z.y * f[u], 1u);
          }
        }
        uint4* d = reinterpret_cast<uint4*>(dst + (uint64_t)x * 32u);
        d[0] = make_uint4(y[0], y[1], y[2], y[3]);
        d[1] = make_uint4(y[4], y[5], y[6], y[7]);
      }
    }
    part += gridDim.z % parts;
    i += gridDim.z / parts;
    if (part >= parts) part -= parts, ++i;
  }
}

}  // namespace

cudaError_t launch_paged8_append(const PagedAppendArgs& a, int sm_count, cudaStream_t st) {
  if (a.Hq) {  // the queries, as beside 16-bit pages
    PagedAppendArgs q = a;
    q.g.H = 0;
    const cudaError_t e = launch_paged_append(q, sm_count, st);
    if (e != cudaSuccess) return e;
  }
  const uint32_t lanes = a.g.D <= 64u ? 8u : 16u;
  uint32_t unit_lg = 7;
  while (unit_lg > 4u && (1u << unit_lg) > (lanes << a.g.page_lg) / 4u) --unit_lg;
  const uint64_t tiles = ((uint64_t)a.b.n_tokens >> a.g.page_lg) + 2ull * a.b.n_seqs;
  const uint64_t rounds = (2ull * a.g.H + (128u >> unit_lg) - 1u) / (128u >> unit_lg);
  // Rounds of a CTA: as many as leave 6 CTAs to each SM (what a CTA looks up before its first
  // is 3 us of waiting): a prefill's append 54.9 us, with a round to a CTA 56.4.
  const uint64_t full = ((uint64_t)a.b.n_tokens >> a.g.page_lg) + 1u;
  uint64_t per = rounds * full / (6ull * sm_count);
  per = per < 1u ? 1u : per > rounds ? rounds : per;
  const uint64_t y = (rounds + per - 1u) / per;
  if (tiles > 0x7FFFFFFFull || y > 65535u) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)tiles, (unsigned)y, 1);
  cfg.blockDim = dim3(128, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.Hq ? 1 : 0;
#define IBP_CALL(L, B)                                                                        \
  return a.pairs                                                                              \
             ? cudaLaunchKernelEx(&cfg, k_paged8_append<L, B, true>, a, unit_lg, (uint32_t)per) \
             : cudaLaunchKernelEx(&cfg, k_paged8_append<L, B, false>, a, unit_lg, (uint32_t)per)
  if (lanes == 8u) {
    if (a.g.bf16) IBP_CALL(8, true);
    IBP_CALL(8, false);
  }
  if (a.g.bf16) IBP_CALL(16, true);
  IBP_CALL(16, false);
#undef IBP_CALL
}

cudaError_t launch_paged8_bounds(const PagedGeom& g, const PagedBatchView& b, uint8_t* bounds,
                                 cudaStream_t st) {
  const uint64_t tiles = ((uint64_t)b.n_tokens >> g.page_lg) + 2ull * b.n_seqs;
  const uint64_t blocks = (tiles * g.H + 3u) / 4u;
  if (blocks > 0x7FFFFFFFull) return cudaErrorInvalidValue;
#define IBP_CALL(L, B) k_paged8_bounds<L, B><<<(unsigned)blocks, 128, 0, st>>>(g, b, bounds)
  if (g.D <= 64u) {
    if (g.bf16) IBP_CALL(4, true);
    else IBP_CALL(4, false);
  } else {
    if (g.bf16) IBP_CALL(8, true);
    else IBP_CALL(8, false);
  }
#undef IBP_CALL
  return cudaGetLastError();
}

cudaError_t launch_paged8_stage(const PagedAttnArgs& a, const PagedAttnArgs& staged,
                                int sm_count, cudaStream_t st) {
  const uint32_t units = (a.g.H * (a.g.D / 16u)) << a.g.page_lg;
  const uint64_t most = (uint64_t)a.b.max_pages * ((units + kStagePart - 1u) / kStagePart);
  uint64_t z = 4ull * sm_count / a.b.n_seqs;  // (keys and values: 8 CTAs to an SM)
  z = z < 1u ? 1u : z > most ? most : z;
  k_paged8_stage<<<dim3(a.b.n_seqs, 2, (unsigned)z), 256, 0, st>>>(a, staged);
  return cudaGetLastError();
}

}  // namespace ibp
