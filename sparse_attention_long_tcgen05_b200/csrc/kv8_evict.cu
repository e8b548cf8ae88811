// kv8_evict.cu -- keeps the tokens of largest accumulated attention weight and
// moves them, in their order, into new pages of the 8-bit latent cache.
//
// Selection (kv8_keep_kernel): of a sequence of n > budget tokens the first
// `sink`, the last `recent` and between them the budget - sink - recent of
// largest weight stay. Weights become 32-bit keys whose integer order is the
// weights' order; three histogram passes over 11, 11 and 10 bits find the
// smallest kept key and how many of the keys equal to it stay (the ones of
// lowest position), and a last pass writes the kept positions in order. A
// cluster of eight CTAs shares a sequence, an eighth of its positions each, and
// adds its histograms and counts through distributed shared memory; where the
// tables are shorter, or the sequences many, one CTA does it alone, which saves
// the cluster's barriers. Weights of exactly zero, which most tokens of a long
// sequence may have, are counted by ballots: as atomics they would all go to one
// address.
// Move (kv8_move_kernel): a CTA per new page copies its 64 rows; the page's
// exponent is the largest of its rows' old ones, so codes move unchanged or
// are scaled down by a power of two. Bound: HBM, every kept row read and
// written once.
#include "kv8_split.cuh"

namespace dsa {
namespace {

constexpr int kKeepThreads = 512;
constexpr int kMoveThreads = 512;

// Larger weight, larger key; -0 = +0; NaN below every number.
__device__ __forceinline__ uint32_t weight_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ uint4 ld_cluster_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// Sum of v over the lanes before this one, and over the whole warp in `all`.
__device__ __forceinline__ uint32_t warp_before(uint32_t v, int lane, uint32_t& all) {
  uint32_t inc = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const uint32_t up = __shfl_up_sync(0xffffffffu, inc, off);
    if (lane >= off) inc += up;
  }
  all = __shfl_sync(0xffffffffu, inc, 31);
  return inc - v;
}

// A barrier of the CTAs that share a sequence.
template <int CTAS>
__device__ __forceinline__ void meet() {
  if constexpr (CTAS > 1)
    cluster_sync();
  else
    __syncthreads();
}

template <int CTAS>
__global__ void __launch_bounds__(kKeepThreads, 2)
kv8_keep_kernel(const __grid_constant__ Kv8EvictArgs a) {
  __shared__ __align__(16) uint32_t hist[2048];
  __shared__ uint32_t warp_sum[kKeepThreads / 32];
  __shared__ uint32_t s_prefix, s_left, s_zero, s_count[2];
  const int b = blockIdx.x / CTAS, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = CTAS > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  griddep_launch_dependents();
  int n = a.c.ctx_lens[b];
  if (n < 0 || n > a.c.max_pages * 64) {
    if (tid == 0 && rank == 0) report(a.status, DSA_ERR_DEVICE_BOUNDS);
    n = 0;
  }
  meet<CTAS>();                                  // new_lens may be ctx_lens
  if (tid == 0 && rank == 0) a.new_lens[b] = min(n, a.budget);
  int32_t* const kept = a.kept + b * a.ld_kept;
  float* const acc_out = a.acc_out + b * a.ld_acc_out;
  const float* const acc = a.acc + b * a.ld_acc;
  const int mid = a.budget - a.sink - a.recent;    // kept between sink and recent
  const int first = rank * kKeepThreads + tid, step = CTAS * kKeepThreads;
  if (n <= a.budget) {
    for (int i = first; i < a.budget; i += step) {
      kept[i] = i < n ? i : -1;
      if (i < n) acc_out[i] = acc[i];
    }
    return;
  }
  for (int i = first; i < a.sink + a.recent; i += step) {
    const int at = i < a.sink ? i : i + mid;
    const int src = i < a.sink ? i : n - a.recent + (i - a.sink);
    kept[at] = src;
    acc_out[at] = acc[src];
  }
  if (mid == 0) return;
  // this CTA's positions [lo, hi)
  const int per = (n - a.recent - a.sink + CTAS - 1) / CTAS;
  const int lo = min(a.sink + rank * per, n - a.recent), hi = min(lo + per, n - a.recent);
  const uint32_t hist_addr = smem_u32(hist), count_addr = smem_u32(s_count);

  // f(i, weight) of each of them, eight loads at a time
  auto each = [&](auto f) {
    for (int i0 = lo + tid; i0 < hi; i0 += 8 * kKeepThreads) {
      float x[8];
#pragma unroll
      for (int t = 0; t < 8; ++t)
        if (i0 + t * kKeepThreads < hi) x[t] = __ldg(acc + i0 + t * kKeepThreads);
#pragma unroll
      for (int t = 0; t < 8; ++t)
        if (i0 + t * kKeepThreads < hi) f(i0 + t * kKeepThreads, x[t]);
    }
  };

  // the mid-th largest key, 11 + 11 + 10 bits from the top
  uint32_t prefix = 0, left = mid;
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const int bits = pass == 2 ? 10 : 11;
    for (int i = tid; i < 2048; i += kKeepThreads) hist[i] = 0;
    if (tid == 0) s_zero = 0;
    __syncthreads();
    uint32_t zeros = 0;
    each([&](int, float x) {
      zeros += x == 0.f;
      const uint32_t key = weight_key(x);
      if (x != 0.f && (pass == 0 || (key >> (shift + bits)) == prefix))
        atomicAdd(&hist[(key >> shift) & ((1u << bits) - 1u)], 1u);
    });
    zeros = __reduce_add_sync(0xffffffffu, zeros);
    if (lane == 0) atomicAdd(&s_zero, zeros);
    __syncthreads();
    if (tid == 0) {
      const uint32_t key = weight_key(0.f);
      if (pass == 0 || (key >> (shift + bits)) == prefix) hist[(key >> shift) & ((1u << bits) - 1u)] += s_zero;
    }
    meet<CTAS>();
    // four bins a thread, summed over the cluster, the highest bins in thread 0
    const int bin0 = 2044 - 4 * tid;
    uint4 h = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int r = 0; r < CTAS; ++r) {
      const uint4 v = CTAS > 1 ? ld_cluster_v4(mapa_shared(hist_addr + 4 * bin0, r))
                               : *reinterpret_cast<const uint4*>(hist + bin0);
      h.x += v.x;
      h.y += v.y;
      h.z += v.z;
      h.w += v.w;
    }
    const uint32_t mine = h.x + h.y + h.z + h.w;
    uint32_t all;
    uint32_t before = warp_before(mine, lane, all);
    if (lane == 0) warp_sum[warp] = all;
    __syncthreads();
    for (int w = 0; w < warp; ++w) before += warp_sum[w];
    if (before < left && left <= before + mine) {  // exactly one thread
      const uint32_t c[4] = {h.w, h.z, h.y, h.x};
      int d = 0;
      while (before + c[d] < left) before += c[d++];
      s_prefix = (prefix << bits) | static_cast<uint32_t>(bin0 + 3 - d);
      s_left = left - before;
    }
    meet<CTAS>();                                // (also: the histograms have been read)
    prefix = s_prefix;
    left = s_left;
  }

  // keys above the prefix stay, and the first `left` keys equal to it: how many of
  // both lie before this CTA's positions
  uint32_t n_gt = 0, n_eq = 0;
  each([&](int, float x) {
    const uint32_t key = weight_key(x);
    n_gt += key > prefix;
    n_eq += key == prefix;
  });
  if (tid < 2) s_count[tid] = 0;
  __syncthreads();
  n_gt = __reduce_add_sync(0xffffffffu, n_gt);
  n_eq = __reduce_add_sync(0xffffffffu, n_eq);
  if (lane == 0) {
    atomicAdd(&s_count[0], n_gt);
    atomicAdd(&s_count[1], n_eq);
  }
  meet<CTAS>();
  uint32_t base = 0, base_eq = 0;
  for (int r = 0; r < rank; ++r) {
    const uint32_t at = mapa_shared(count_addr, r);
    base += ld_shared_cluster_u32(at);
    base_eq += ld_shared_cluster_u32(at + 4);
  }
  for (int i0 = lo; i0 < hi; i0 += 4 * kKeepThreads) {
    float x[4];
    uint32_t packed = 0, flags = 0;                // counts: above in the low half, equal in the high
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int i = i0 + 4 * tid + t;
      x[t] = i < hi ? acc[i] : 0.f;
      const uint32_t key = weight_key(x[t]);
      if (i < hi && key > prefix) {
        packed += 1u;
        flags |= 1u << t;
      } else if (i < hi && key == prefix) {
        packed += 1u << 16;
        flags |= 16u << t;
      }
    }
    uint32_t all;
    uint32_t before = warp_before(packed, lane, all);
    __syncthreads();                               // warp_sum has been read
    if (lane == 0) warp_sum[warp] = all;
    __syncthreads();
    uint32_t total = 0;
#pragma unroll
    for (int w = 0; w < kKeepThreads / 32; ++w) {
      if (w < warp) before += warp_sum[w];
      total += warp_sum[w];
    }
    uint32_t g = base + (before & 0xffffu), e = base_eq + (before >> 16);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const bool gt = (flags >> t) & 1u, eq = (flags >> (4 + t)) & 1u;
      if (gt || (eq && e < left)) {
        const uint32_t at = a.sink + g + min(e, left);
        kept[at] = i0 + 4 * tid + t;
        acc_out[at] = x[t];
      }
      g += gt;
      e += eq;
    }
    base += total & 0xffffu;
    base_eq += total >> 16;
  }
  meet<CTAS>();                                  // no CTA leaves while its counts may be read
}

__global__ void __launch_bounds__(kMoveThreads, 4)
kv8_move_kernel(const __grid_constant__ Kv8EvictArgs a) {
  __shared__ int64_t s_row[64];
  __shared__ int s_exp[64];
  const int pages = (a.budget + 63) / 64;
  const int b = blockIdx.x / pages, page = blockIdx.x % pages, tid = threadIdx.x;
  griddep_wait();                                  // kept, new_lens
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
      const int e_src = pg >= 0 && pg < a.c.num_pages ? a.c.exps[pg] : kExpMax + 1;
      if (is_exponent(e_src)) {
        row = pg * 64 + (src & 63);
        e = e_src;
      } else {
        report(a.status, DSA_ERR_DEVICE_BOUNDS);
      }
    }
    s_row[tid] = row;
    s_exp[tid] = e;
  }
  __syncthreads();
  int e = max(s_exp[tid & 31], s_exp[32 + (tid & 31)]);   // (rows past m: the minimum)
  e = __reduce_max_sync(0xffffffffu, e);
  constexpr int kPieces = kRow8 / 16, kLoads = (64 * kPieces + kMoveThreads - 1) / kMoveThreads;
  uint4 x[kLoads];                                 // all loads before the first store
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int u = tid + i * kMoveThreads, r = u / kPieces;
    if (r < m && s_row[r] >= 0)
      x[i] = *(reinterpret_cast<const uint4*>(a.c.codes + s_row[r] * a.c.ld) + u % kPieces);
  }
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int u = tid + i * kMoveThreads, r = u / kPieces;
    if (r >= m || s_row[r] < 0) continue;
    const int d = s_exp[r] - e;
    if (d != 0) {
      const float f = pow2i(max(d, -126));
      x[i] = make_uint4(rescale_e4m3x4(x[i].x, f), rescale_e4m3x4(x[i].y, f), rescale_e4m3x4(x[i].z, f),
                        rescale_e4m3x4(x[i].w, f));
    }
    *(reinterpret_cast<uint4*>(a.c.codes + (to * 64 + r) * a.c.ld) + u % kPieces) = x[i];
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

// One CTA a sequence takes about 1.1 us more for every 1024 tokens; a cluster's barriers cost
// 6 us, and 37 clusters fill the device, so the more sequences the later they pay.
// Measured, one CTA / clusters, us a call with the move, tables of the given tokens:
//   1 sequence:    12288  21.5 / 22.5    16384  27.1 / 22.7    32768   38.9 / 24.6
//   16 sequences:  16384  28.7 / 32.8    24576  38.5 / 34.8    65536   89 / 43
//   32 sequences:  16384  35.4 / 42.6    24576  45.1 / 45.0    32768   53.5 / 45.8
//   64 sequences:  16384  44.0 / 78.6    32768  62.1 / 84.3    65536  106.5 / 98.5
//   150 sequences:  8192  86.4 / 201     16384  158 / 263
constexpr int32_t kOnePages = 192, kOnePagesASeq = 8;

cudaError_t launch_kv8_evict(const Kv8EvictArgs& a, int* launches, cudaStream_t stream) {
  cudaError_t e;
  if (a.c.max_pages <= kOnePages + int64_t(kOnePagesASeq) * a.c.n_seq) {
    kv8_keep_kernel<1><<<a.c.n_seq, kKeepThreads, 0, stream>>>(a);
    e = cudaGetLastError();
  } else {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(8 * a.c.n_seq);
    cfg.blockDim = dim3(kKeepThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 8;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kv8_keep_kernel<8>, a);
  }
  if (e != cudaSuccess) return e;
  ++*launches;
  e = launch_dependent(kv8_move_kernel, dim3(a.c.n_seq * ((a.budget + 63) / 64)), kMoveThreads, 0, stream, a);
  if (e != cudaSuccess) return e;
  ++*launches;
  return cudaSuccess;
}

}  // namespace dsa
