// kv8_evict.cu -- keeps the tokens of largest accumulated attention weight and
// moves them, in their order, into new pages of the 8-bit latent cache.
//
// Selection (kv8_keep_kernel): of a sequence of n > budget tokens the first
// `sink`, the last `recent` and between them the budget - sink - recent of
// largest weight stay. Weights become 32-bit keys whose integer order is the
// weights' order; three histogram passes over 11, 11 and 10 bits find the
// smallest kept key and how many of the keys equal to it stay (the ones of
// lowest position), and a last pass writes the kept positions in order.
// Move (kv8_move_kernel): a CTA per new page copies its 64 rows; the page's
// exponent is the largest of its rows' old ones, so codes move unchanged or
// are scaled down by a power of two. Bound: HBM, every kept row read and
// written once.
#include "kv8_common.cuh"

namespace dsa {
namespace {

constexpr int kKeepThreads = 1024;
constexpr int kMoveThreads = 256;

// Larger weight, larger key; -0 = +0; NaN below every number.
__device__ __forceinline__ uint32_t weight_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kKeepThreads)
kv8_keep_kernel(const __grid_constant__ Kv8EvictArgs a) {
  __shared__ uint32_t hist[2048];
  __shared__ uint32_t warp_n[2][kKeepThreads / 32];
  __shared__ uint32_t s_prefix, s_left;
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int n = a.c.ctx_lens[b];
  if (n < 0 || n > a.c.max_pages * 64) {
    if (tid == 0) report(a.status, DSA_ERR_DEVICE_BOUNDS);
    n = 0;
  }
  __syncthreads();                                 // new_lens may be ctx_lens
  if (tid == 0) a.new_lens[b] = min(n, a.budget);
  int32_t* kept = a.kept + b * a.ld_kept;
  float* acc_out = a.acc_out + b * a.ld_acc_out;
  const float* acc = a.acc + b * a.ld_acc;
  const int mid = a.budget - a.sink - a.recent;    // kept between sink and recent
  if (n <= a.budget) {
    for (int i = tid; i < a.budget; i += kKeepThreads) {
      kept[i] = i < n ? i : -1;
      if (i < n) acc_out[i] = acc[i];
    }
    return;
  }
  const int lo = a.sink, hi = n - a.recent;
  for (int i = tid; i < a.sink + a.recent; i += kKeepThreads) {
    const int at = i < a.sink ? i : i + mid;
    const int src = i < a.sink ? i : n - a.recent + (i - a.sink);
    kept[at] = src;
    acc_out[at] = acc[src];
  }
  if (mid == 0) return;
  // the mid-th largest key, 11 + 11 + 10 bits from the top
  uint32_t prefix = 0, left = mid;
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const int bits = pass == 2 ? 10 : 11;
    for (int i = tid; i < 2048; i += kKeepThreads) hist[i] = 0;
    __syncthreads();
    for (int i = lo + tid; i < hi; i += kKeepThreads) {
      const uint32_t key = weight_key(acc[i]);
      if (pass == 0 || (key >> (shift + bits)) == prefix)
        atomicAdd(&hist[(key >> shift) & ((1u << bits) - 1u)], 1u);
    }
    __syncthreads();
    if (tid == 0) {                                // simple: walk down from the top bin
      uint32_t sum = 0;
      int d = (1 << bits) - 1;
      while (sum + hist[d] < left) sum += hist[d--];
      s_prefix = (prefix << bits) | static_cast<uint32_t>(d);
      s_left = left - sum;
    }
    __syncthreads();
    prefix = s_prefix;
    left = s_left;
    __syncthreads();
  }
  // keys above the prefix stay, and the first `left` keys equal to it
  uint32_t base = 0, base_eq = 0;
  for (int i0 = lo; i0 < hi; i0 += kKeepThreads) {
    const int i = i0 + tid;
    const float x = i < hi ? acc[i] : 0.f;
    const uint32_t key = weight_key(x);
    const bool gt = i < hi && key > prefix, eq = i < hi && key == prefix;
    const uint32_t bg = __ballot_sync(0xffffffffu, gt), be = __ballot_sync(0xffffffffu, eq);
    if (lane == 0) {
      warp_n[0][warp] = __popc(bg);
      warp_n[1][warp] = __popc(be);
    }
    __syncthreads();
    uint32_t g = 0, e = 0, gt_all = 0, eq_all = 0;
    for (int w = 0; w < kKeepThreads / 32; ++w) {
      if (w == warp) {
        g = gt_all;
        e = eq_all;
      }
      gt_all += warp_n[0][w];
      eq_all += warp_n[1][w];
    }
    const uint32_t below = (1u << lane) - 1u;
    g += base + __popc(bg & below);
    e += base_eq + __popc(be & below);
    if (gt || (eq && e < left)) {
      const uint32_t at = a.sink + g + min(e, left);
      kept[at] = i;
      acc_out[at] = x;
    }
    base += gt_all;
    base_eq += eq_all;
    __syncthreads();
  }
}

__global__ void __launch_bounds__(kMoveThreads)
kv8_move_kernel(const __grid_constant__ Kv8EvictArgs a) {
  __shared__ int64_t s_row[64];
  __shared__ int s_exp[64];
  const int b = blockIdx.y, page = blockIdx.x, tid = threadIdx.x;
  const int m = min(64, a.new_lens[b] - page * 64);
  if (m <= 0) return;
  const int64_t to = a.dst_table[b * a.ld_dst + page];
  if (to < 0 || to >= a.c.num_pages) {
    if (tid == 0) report(a.status, DSA_ERR_DEVICE_BOUNDS);
    return;
  }
  if (tid < 64) {
    int64_t row = -1;
    int e = kExpMin;
    if (tid < m) {
      const int src = a.kept[b * a.ld_kept + page * 64 + tid];
      const int64_t pg = a.c.table[b * a.c.ld_table + (src >> 6)];
      if (pg >= 0 && pg < a.c.num_pages) {
        row = pg * 64 + (src & 63);
        e = a.c.exps[pg];
      } else {
        report(a.status, DSA_ERR_DEVICE_BOUNDS);
      }
    }
    s_row[tid] = row;
    s_exp[tid] = e;
  }
  __syncthreads();
  int e = kExpMin;
  for (int i = 0; i < m; ++i) e = max(e, s_exp[i]);
  for (int i = tid; i < m * (kRow8 / 16); i += kMoveThreads) {
    const int r = i / (kRow8 / 16), c = i % (kRow8 / 16);
    if (s_row[r] < 0) continue;
    uint4 x = *(reinterpret_cast<const uint4*>(a.c.codes + s_row[r] * a.c.ld) + c);
    const int d = s_exp[r] - e;
    if (d != 0) {
      const float f = pow2i(max(d, -126));
      x = make_uint4(rescale_e4m3x4(x.x, f), rescale_e4m3x4(x.y, f), rescale_e4m3x4(x.z, f),
                     rescale_e4m3x4(x.w, f));
    }
    *(reinterpret_cast<uint4*>(a.c.codes + (to * 64 + r) * a.c.ld) + c) = x;
  }
  if (a.idx_codes != nullptr) {
    for (int i = tid; i < m * 8; i += kMoveThreads) {
      const int r = i >> 3, c = i & 7;
      if (s_row[r] >= 0)
        *(reinterpret_cast<uint4*>(a.idx_codes + (to * 64 + r) * a.ld_idx) + c) =
            *(reinterpret_cast<const uint4*>(a.idx_codes + s_row[r] * a.ld_idx) + c);
    }
    if (tid < m && s_row[tid] >= 0) a.idx_scales[to * 64 + tid] = a.idx_scales[s_row[tid]];
  }
  if (tid == 0) a.c.exps[to] = static_cast<int8_t>(e);
}

}  // namespace

cudaError_t launch_kv8_evict(const Kv8EvictArgs& a, int* launches, cudaStream_t stream) {
  kv8_keep_kernel<<<a.c.n_seq, kKeepThreads, 0, stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  ++*launches;
  kv8_move_kernel<<<dim3((a.budget + 63) / 64, a.c.n_seq), kMoveThreads, 0, stream>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  ++*launches;
  return cudaSuccess;
}

}  // namespace dsa
