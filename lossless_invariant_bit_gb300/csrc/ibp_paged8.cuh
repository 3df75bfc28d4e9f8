// Internal declarations of the paged K/V cache held in 8 bits: a page's keys (and values)
// of one head are e4m3 codes under one scale, a power of two held as its E8M0 byte.
#pragma once

#include "ibp_paged.cuh"
#ifdef __CUDACC__
#include "ibp_sm103.cuh"
#endif

namespace ibp {

cudaError_t launch_paged8_append(const PagedAppendArgs& a, int sm_count, cudaStream_t st);
cudaError_t launch_paged8_bounds(const PagedGeom& g, const PagedBatchView& b, uint8_t* bounds,
                                 cudaStream_t st);
cudaError_t launch_paged8_step(const PagedAttnArgs& a, const PagedMaps& m, int sm_count,
                               bool behind, cudaStream_t st);
cudaError_t launch_paged8_chunk(const PagedAttnArgs& a, const PagedMaps& m, int sm_count,
                                cudaStream_t st);
cudaError_t launch_paged8_chunk_join(const PagedAttnArgs& a, int sm_count, cudaStream_t st);

cudaError_t launch_paged8_stage(const PagedAttnArgs& a, const PagedAttnArgs& staged,
                                int sm_count, cudaStream_t st);

// Bytes of scales: 2^-50 to 2^50.  The range is bounded so that no power of a page's scale,
// nor the product of two pages', leaves fp32 where a result still depends on it.
constexpr uint32_t kScaleLow = 77u, kScaleHigh = 177u;

#ifdef __CUDACC__

__device__ __forceinline__ bool scale_ok(uint32_t byte) {
  return byte >= kScaleLow && byte <= kScaleHigh;
}

// The bytes of a page's scales for one head: keys' | values' << 8.
__device__ __forceinline__ uint32_t page_scales(const PagedGeom& g, uint32_t page, uint32_t head) {
  const uint64_t at = (uint64_t)page * g.H + head;
  return (uint32_t)__ldg(g.k_scales + at) | (uint32_t)__ldg(g.v_scales + at) << 8;
}
__device__ __forceinline__ bool scales_ok(uint32_t both) {
  return scale_ok(both & 0xFFu) && scale_ok(both >> 8);
}
__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(byte << 23); }

// Four codes as two pairs of fp16, exactly (NaN stays NaN).
__device__ __forceinline__ void codes_to_fp16(uint32_t x, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n"
      " cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(x));
}

// The top bit of each byte that is a NaN code (0x7F or 0xFF).
__device__ __forceinline__ uint32_t nan_codes(uint32_t x) {
  return ((x & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}

// Byte offset of 16 channels of a token in a tile written by TMA: rows of kDP bytes with the
// swizzle of that span (16-byte chunks, by the 128-byte line that the row lies in).
template <int kDP>
__device__ __forceinline__ uint32_t code_chunk(uint32_t row, uint32_t chunk) {
  if (kDP == 128) return row * 128u + ((chunk ^ (row & 7u)) << 4);
  return row * 64u + ((chunk ^ (row >> 1 & 3u)) << 4);
}

// bf16 queries for products in fp16: each row times a power of two that brings its largest
// magnitude into [2^14, 2^15).  Half a step of fp16's smallest numbers, 2^-25, is 2^-39 of it.
struct Lift {
  float up, down;
  uint8_t byte;  // down's exponent, as a scale's
};
// The larger magnitude of two bf16 values as bits, infinities and NaN apart.
__device__ __forceinline__ uint32_t bf16_top(uint32_t x) {
  const uint32_t a = x & 0x7FFFu, b = x >> 16 & 0x7FFFu;
  return max(a < 0x7F80u ? a : 0u, b < 0x7F80u ? b : 0u);
}
__device__ __forceinline__ Lift row_lift(uint32_t top) {
  const int32_t up = min(126, 14 + 127 - (int32_t)(top >> 7));  // (top: 254 at most, so >= -113)
  return Lift{__uint_as_float((uint32_t)(127 + up) << 23),
              __uint_as_float((uint32_t)(127 - up) << 23), (uint8_t)(127 - up)};
}
__device__ __forceinline__ uint32_t bf16_to_fp16(uint32_t x, float up) {
  return pack2(__uint_as_float(x << 16) * up, __uint_as_float(x & 0xFFFF0000u) * up, 0u);
}

// A row's factor for the scores of a page.  Never 0 or infinite: -inf (a score that is masked)
// or 0 times it stays what it is.
__device__ __forceinline__ float row_factor(float row, float page) {
  return fminf(fmaxf(row * page, 1e-37f), 1e37f);
}

#endif

}  // namespace ibp
