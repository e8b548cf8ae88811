// kv8_mqa.cu -- MQA attention over the 8-bit latent cache, over a selection or
// over every preceding key.
//
//   O[t,h] = sum_s softmax_s(scale * q[t,h] . kv[s]) * kv[s, 0:512],
//   kv[s] = decode(codes[s]) * 2^e(block of s)
//
// One CTA per (query, head): each warp takes every eighth key, holds the head's
// query in registers (18 columns a lane), adds the lanes' products and keeps an
// online softmax of its own over 16 value columns a lane; the warps' partial
// results are joined in shared memory.
#include "kv8_common.cuh"

namespace dsa {
namespace {

constexpr int kWarps = 8;

__global__ void __launch_bounds__(kWarps * 32)
kv8_mqa_kernel(const __grid_constant__ Kv8AttnArgs a) {
  __shared__ float s_m[kWarps], s_l[kWarps];
  __shared__ float s_o[kWarps][512];
  const int qi = blockIdx.x, h = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int seq, pos;
  if (!kv8_query(a.keys, qi, seq, pos) && threadIdx.x == 0 && h == 0)
    report(a.status, DSA_ERR_DEVICE_BOUNDS);
  const __nv_bfloat16* q = a.q + qi * a.ld_q + static_cast<int64_t>(h) * kRow8;
  // lane owns columns 4 (lane + 32 i) .. +3 for i < 4 and rope columns 512 + 2 lane, +1
  float qv[18];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) qv[4 * i + j] = __bfloat162float(q[4 * (lane + 32 * i) + j]);
  qv[16] = __bfloat162float(q[512 + 2 * lane]);
  qv[17] = __bfloat162float(q[513 + 2 * lane]);
  float m = -INFINITY, l = 0.f, o[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) o[i] = 0.f;
  const int n = a.idx != nullptr ? a.k : pos + 1;
  for (int j = warp; j < n; j += kWarps) {
    const int p = a.idx != nullptr ? __ldg(a.idx + qi * a.ld_idx + j) : j;
    if (p < 0) continue;
    const int64_t row = p <= pos ? kv8_row(a.keys, seq, p) : -1;
    if (row < 0) {
      if (lane == 0) report(a.status, DSA_ERR_DEVICE_BOUNDS);
      continue;
    }
    const uint8_t* kr = a.kv + row * a.ld_kv;
    const float f = pow2i(a.exps[row >> 6]);
    float v[18];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(kr) + lane + 32 * i);
      const float2 x = from_e4m3x2(w & 0xffffu), y = from_e4m3x2(w >> 16);
      v[4 * i] = x.x * f;
      v[4 * i + 1] = x.y * f;
      v[4 * i + 2] = y.x * f;
      v[4 * i + 3] = y.y * f;
    }
    const float2 x = from_e4m3x2(__ldg(reinterpret_cast<const uint16_t*>(kr + 512) + lane));
    v[16] = x.x * f;
    v[17] = x.y * f;
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < 18; ++i) dot = fmaf(qv[i], v[i], dot);
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, s);
    const float z = dot * a.scale_log2;
    const float m_new = fmaxf(m, z);
    const float alpha = exp2f(m - m_new), w = exp2f(z - m_new);
    l = l * alpha + w;
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = fmaf(o[i], alpha, w * v[i]);
    m = m_new;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) s_o[warp][4 * (lane + 32 * i) + j] = o[4 * i + j];
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
  __syncthreads();
  float mx = -INFINITY, sum = 0.f;
  for (int w = 0; w < kWarps; ++w)
    if (s_l[w] != 0.f) mx = fmaxf(mx, s_m[w]);
  float part[kWarps];
  for (int w = 0; w < kWarps; ++w) {
    part[w] = s_l[w] != 0.f ? exp2f(s_m[w] - mx) : 0.f;
    sum += part[w] * s_l[w];
  }
  const int64_t at = static_cast<int64_t>(qi) * a.heads + h;
  for (int d = threadIdx.x; d < 512; d += kWarps * 32) {
    float r = 0.f;
    for (int w = 0; w < kWarps; ++w) r = fmaf(part[w], s_o[w][d], r);
    a.out[at * 512 + d] = __float2bfloat16(sum != 0.f ? r / sum : 0.f);
  }
  if (threadIdx.x == 0 && a.lse != nullptr)
    a.lse[at] = sum != 0.f ? (mx + log2f(sum)) * 0.69314718055994531f : -INFINITY;
}

}  // namespace

size_t kv8_mqa_workspace(int32_t, int32_t, int64_t) { return 0; }

cudaError_t launch_kv8_mqa(const Kv8AttnArgs& a, int, int* launches, cudaStream_t stream) {
  kv8_mqa_kernel<<<dim3(a.keys.n_q, a.heads), kWarps * 32, 0, stream>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace dsa
