// kv8_weights.cu -- the running attention weight of each cached token.
//
//   w[i,s] = (1/H) sum_h exp(scale * q[i,h] . kv[s] - lse[i,h])
//   acc[b,s] = decay * acc[b,s] + sum over b's queries i, ascending, of w[i,s]
//
// The first kernel writes w per query (a warp per key, the heads in turn); the
// second adds the queries of a sequence in their order, so that the sums do not
// depend on which finishes first. Within one query an entry that repeats a key
// adds the same bits as the first, so the order of those two does not matter
// either, and they may be added with atomics.
#include "kv8_common.cuh"

namespace dsa {
namespace {

constexpr int kWarps = 8;
constexpr int kAccThreads = 256;

__global__ void __launch_bounds__(kWarps * 32)
kv8_weights_kernel(const __grid_constant__ Kv8WeightArgs w) {
  const Kv8AttnArgs& a = w.attn;
  const int qi = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int seq, pos;
  if (!kv8_query(a.keys, qi, seq, pos) && threadIdx.x == 0 && blockIdx.y == 0)
    report(a.status, DSA_ERR_DEVICE_BOUNDS);
  for (int j = blockIdx.y * kWarps + warp; j < w.n_cols; j += gridDim.y * kWarps) {
    const int p = a.idx != nullptr ? __ldg(a.idx + qi * a.ld_idx + j) : j;
    float sum = 0.f;
    const int64_t row = p >= 0 && p <= pos ? kv8_row(a.keys, seq, p) : -1;
    if (row >= 0) {
      const uint8_t* kr = a.kv + row * a.ld_kv;
      const float f = pow2i(a.exps[row >> 6]);
      float v[18];
#pragma unroll
      for (int i = 0; i < 9; ++i) {
        const float2 x = from_e4m3x2(__ldg(reinterpret_cast<const uint16_t*>(kr) + lane + 32 * i));
        v[2 * i] = x.x * f;
        v[2 * i + 1] = x.y * f;
      }
      for (int h = 0; h < a.heads; ++h) {
        const __nv_bfloat162* q = reinterpret_cast<const __nv_bfloat162*>(
            a.q + qi * a.ld_q + static_cast<int64_t>(h) * kRow8);
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < 9; ++i) {
          const float2 y = __bfloat1622float2(q[lane + 32 * i]);
          dot = fmaf(y.x, v[2 * i], fmaf(y.y, v[2 * i + 1], dot));
        }
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, s);
        const float lse = w.lse[static_cast<int64_t>(qi) * a.heads + h];
        if (lse != -INFINITY)
          sum += exp2f(fmaf(dot, a.scale_log2, -lse * 1.4426950408889634f));
      }
      sum /= static_cast<float>(a.heads);
    } else if (lane == 0 && p >= 0 && (a.idx != nullptr || p <= pos)) {
      report(a.status, DSA_ERR_DEVICE_BOUNDS);
    }
    if (lane == 0) w.w[static_cast<int64_t>(qi) * w.n_cols + j] = sum;
  }
}

// Queries of sequence b in ascending order: f(i, pos of i).
template <typename F>
__device__ __forceinline__ void for_queries(const KeySide& ks, int b, F f) {
  if (ks.paged && ks.q_seq != nullptr) {
    for (int i = 0; i < ks.n_q; ++i) {
      int seq, pos;
      if (__ldg(ks.q_seq + i) == b && paged_query(ks, i, seq, pos)) f(i, pos);
    }
  } else if (ks.paged) {
    int seq, pos;
    if (b < ks.n_q && paged_query(ks, b, seq, pos)) f(b, pos);
  } else {
    for (int i = 0; i < ks.n_q; ++i) f(i, ks.n_keys - ks.n_q + i);
  }
}

__device__ __forceinline__ int seq_len(const KeySide& ks, int b) {
  if (!ks.paged) return ks.n_keys;
  const int n = __ldg(ks.ctx_lens + b);
  return n < 0 || n > ks.max_pages * 64 ? 0 : n;
}

// Every key of the sequence: acc = decay * acc + the queries' weights.
__global__ void __launch_bounds__(kAccThreads)
kv8_acc_dense_kernel(const __grid_constant__ Kv8WeightArgs w, bool add) {
  const KeySide& ks = w.attn.keys;
  const int b = blockIdx.y;
  const int s = blockIdx.x * kAccThreads + threadIdx.x;
  if (s >= seq_len(ks, b)) return;
  float* acc = w.acc + b * w.ld_acc + s;
  float v = *acc * w.decay;
  if (add)
    for_queries(ks, b, [&](int i, int pos) {
      if (s <= pos) v += w.w[static_cast<int64_t>(i) * w.n_cols + s];
    });
  *acc = v;
}

// The selected keys: query after query.
__global__ void __launch_bounds__(1024)
kv8_acc_sparse_kernel(const __grid_constant__ Kv8WeightArgs w) {
  const KeySide& ks = w.attn.keys;
  const int b = blockIdx.x;
  float* acc = w.acc + b * w.ld_acc;
  for_queries(ks, b, [&](int i, int pos) {
    for (int j = threadIdx.x; j < w.n_cols; j += blockDim.x) {
      const int p = __ldg(w.attn.idx + i * w.attn.ld_idx + j);
      if (p >= 0 && p <= pos) atomicAdd(acc + p, w.w[static_cast<int64_t>(i) * w.n_cols + j]);
    }
    __syncthreads();
  });
}

}  // namespace

cudaError_t launch_kv8_accumulate(const Kv8WeightArgs& w, int num_sms, int* launches,
                                  cudaStream_t stream) {
  const KeySide& ks = w.attn.keys;
  const int n_seq = ks.paged ? ks.n_seq : 1;
  const int per = max(1, min((w.n_cols + kWarps - 1) / kWarps, 16 * num_sms / ks.n_q + 1));
  kv8_weights_kernel<<<dim3(ks.n_q, per), kWarps * 32, 0, stream>>>(w);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  ++*launches;
  const bool dense = w.attn.idx == nullptr;
  if (dense || w.decay != 1.f) {
    const int width = ks.paged ? ks.max_pages * 64 : ks.n_keys;
    kv8_acc_dense_kernel<<<dim3((width + kAccThreads - 1) / kAccThreads, n_seq), kAccThreads, 0, stream>>>(
        w, dense);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    ++*launches;
  }
  if (!dense) {
    kv8_acc_sparse_kernel<<<n_seq, 1024, 0, stream>>>(w);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    ++*launches;
  }
  return cudaSuccess;
}

}  // namespace dsa
