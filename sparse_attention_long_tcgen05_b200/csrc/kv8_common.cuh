// kv8_common.cuh -- e4m3 conversions and key look-up shared by the kernels of
// the 8-bit latent cache (codes of 576-wide rows, one exponent per 64 tokens).
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "dsa_common.cuh"
#include "dsa_kernels.h"

namespace dsa {

constexpr int kRow8 = 576;       // bytes of one cached row
constexpr int kExpMin = -64;     // exponents of a block's scale 2^e
constexpr int kExpMax = 63;

// 2^e for e in [-126, 127]. Sums of two block exponents stay inside.
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }

// Two floats to e4m3 (round to nearest even, saturating, NaN kept), low byte first.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

// Two e4m3 codes to floats (exact).
__device__ __forceinline__ float2 from_e4m3x2(uint32_t codes) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes), __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Four codes of a word times 2^-d, rounded to codes again.
__device__ __forceinline__ uint32_t rescale_e4m3x4(uint32_t w, float f) {
  const float2 a = from_e4m3x2(w & 0xffffu), b = from_e4m3x2(w >> 16);
  return to_e4m3x2(a.x * f, a.y * f) | (to_e4m3x2(b.x * f, b.y * f) << 16);
}

// The cached row of key position p (0 <= p <= pos) of sequence seq, or -1 when
// its page id is out of range.
__device__ __forceinline__ int64_t kv8_row(const KeySide& ks, int seq, int p) {
  if (!ks.paged) return p;
  const int pg = __ldg(ks.block_table + static_cast<int64_t>(seq) * ks.ld_block_table + (p >> 6));
  if (pg < 0 || pg >= ks.num_pages) return -1;
  return static_cast<int64_t>(pg) * 64 + (p & 63);
}

// Sequence and position of query qi; pos -1 when it is out of range.
__device__ __forceinline__ bool kv8_query(const KeySide& ks, int qi, int& seq, int& pos) {
  if (ks.paged) return paged_query(ks, qi, seq, pos);
  seq = 0;
  pos = ks.n_keys - ks.n_q + qi;
  return true;
}

}  // namespace dsa
