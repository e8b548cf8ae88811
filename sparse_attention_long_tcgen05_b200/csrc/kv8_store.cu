// kv8_store.cu -- quantises new latent rows into the 8-bit cache.
//
// A block of 64 tokens shares one scale 2^e: e = the smallest exponent with
// amax <= 448 * 2^e over the block's new values, but not below the exponent
// under which its earlier rows were stored; code = e4m3(x * 2^-e). When e
// grows, the earlier codes c become e4m3(c * 2^(e_old - e)), exact unless the
// result is an e4m3 subnormal.
//
// One CTA owns a block from its first new row on, so no two CTAs write one
// block and nothing is exchanged. CTA c looks at rows [c R, (c+1) R) for the
// rows that begin a sequence's run or a block, and quantises those blocks
// whole: once over the rows for the maximum, once more (from L2) to convert
// them. The bound is HBM, 3 bytes moved per bf16 element and 5 per fp32 element.
// (Keeping the rows in registers between the two reads them once, but leaves an
// SM one or two CTAs that load, then wait, then store: 38 us for the 62,000-row
// prefill of bf16 rows, 37 us for 33,000 fp32 rows.)
#include "kv8_common.cuh"

namespace dsa {
namespace {

constexpr int kStoreThreads = 512;

template <typename T>
__global__ void __launch_bounds__(kStoreThreads, 4)
kv8_store_kernel(const __grid_constant__ Kv8StoreArgs a) {
  constexpr int kPer = 16 / sizeof(T);              // elements of a 16-byte piece
  constexpr int kPieces = kRow8 / kPer;             // pieces of a row
  constexpr int kBatch = 3, kLoads = 64 * kPieces / kStoreThreads;   // 9 or 18 pieces a thread
  static_assert(kLoads % kBatch == 0, "");
  __shared__ uint32_t red[kStoreThreads / 32];
  const int tid = threadIdx.x;
  const Kv8Pages& c = a.c;

  int64_t r = static_cast<int64_t>(blockIdx.x) * a.rows_per_cta;
  const int64_t r_end = min(r + a.rows_per_cta, static_cast<int64_t>(a.n_rows));
  while (r < r_end) {
    // the run that row r belongs to: rows [run0, run1) of sequence b
    int b = 0;
    int64_t run0 = 0, run1 = a.n_rows;
    int64_t len = c.n_keys;
    if (c.table != nullptr) {
      if (a.cu == nullptr) {
        b = static_cast<int>(r);
        run0 = r;
        run1 = r + 1;
      } else {
        // the last b with cu[b] <= r: a warp looks at 32 places at a time
        int lo = 0, n = c.n_seq;
        while (n > 1) {
          const int step = (n + 31) / 32, at = (tid & 31) * step;
          const uint32_t le = __ballot_sync(0xffffffffu, at < n && __ldg(a.cu + lo + at) <= r);
          const int k = le != 0u ? 31 - __clz(le) : 0;
          lo += k * step;
          n = min(step, n - k * step);
        }
        b = lo;
        run0 = __ldg(a.cu + b);
        run1 = __ldg(a.cu + b + 1);
      }
      len = __ldg(c.ctx_lens + b);
    }
    const int64_t n_new = run1 - run0;
    if (run0 < 0 || run0 > r || run1 <= r || run1 > a.n_rows || n_new > len ||
        len > static_cast<int64_t>(c.max_pages) * 64) {
      if (tid == 0) report(a.status, DSA_ERR_DEVICE_BOUNDS);
      r = (run0 <= r && run1 > r) ? run1 : r + 1;
      continue;
    }
    const int64_t p = len - n_new + (r - run0);
    const int slot = static_cast<int>(p & 63);
    if (r != run0 && slot != 0) {                   // inside a block that begins earlier
      r = min(run1, r + 64 - slot);
      continue;
    }
    const int m = static_cast<int>(min(static_cast<int64_t>(64 - slot), run1 - r));
    int64_t page = p >> 6;
    if (c.table != nullptr) page = __ldg(c.table + static_cast<int64_t>(b) * c.ld_table + (p >> 6));
    const T* src = static_cast<const T*>(a.rows) + r * a.ld_rows;
    auto piece = [&](int u) {                       // of the block's m rows
      return __ldg(reinterpret_cast<const uint4*>(src + (u / kPieces) * a.ld_rows) + u % kPieces);
    };
    uint32_t amax = 0;                              // |x| as bits: ordered like the values
#pragma unroll 1
    for (int i0 = 0; i0 < kLoads && i0 * kStoreThreads < m * kPieces; i0 += kBatch) {
      uint4 v[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int u = tid + (i0 + i) * kStoreThreads;
        v[i] = u < m * kPieces ? piece(u) : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t x0 = (sizeof(T) == 2 ? w[j] << 16 : w[j]) & 0x7fffffffu;
          const uint32_t x1 = sizeof(T) == 2 ? w[j] & 0x7fff0000u : 0u;
          if (x0 < 0x7f800000u) amax = max(amax, x0);   // finite values only
          if (x1 < 0x7f800000u) amax = max(amax, x1);
        }
      }
    }
    if (page < 0 || page >= c.num_pages) {
      if (tid == 0) report(a.status, DSA_ERR_DEVICE_BOUNDS);
      r += m;
      continue;
    }
    const int e_old = c.exps[page];
    if (slot > 0 && !is_exponent(e_old)) {          // what the earlier rows stand for is not known
      if (tid == 0) report(a.status, DSA_ERR_DEVICE_BOUNDS);
      r += m;
      continue;
    }
    amax = __reduce_max_sync(0xffffffffu, amax);
    if ((tid & 31) == 0) red[tid >> 5] = amax;
    __syncthreads();
    amax = 0;
#pragma unroll
    for (int i = 0; i < kStoreThreads / 32; ++i) amax = max(amax, red[i]);
    // 448 = 1.75 * 2^8: amax = f * 2^x with f in [1, 2) needs x - 8, one more when f > 1.75
    int e = static_cast<int>(amax >> 23) - 127 - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);
    e = min(max(e, kExpMin), kExpMax);              // (0 and fp32 subnormals fall to the minimum)
    if (slot > 0) e = max(e, e_old);

    uint8_t* block = c.codes + page * 64 * c.ld;
    if (slot > 0 && e != e_old) {
      const float f = pow2i(max(e_old - e, -126));
      for (int i = tid; i < slot * (kRow8 / 16); i += kStoreThreads) {
        uint4* q = reinterpret_cast<uint4*>(block + (i / (kRow8 / 16)) * c.ld) + i % (kRow8 / 16);
        const uint4 x = *q;
        *q = make_uint4(rescale_e4m3x4(x.x, f), rescale_e4m3x4(x.y, f), rescale_e4m3x4(x.z, f),
                        rescale_e4m3x4(x.w, f));
      }
    }
    const float f = pow2i(-e);
    uint8_t* dst = block + slot * c.ld;
#pragma unroll 1
    for (int i0 = 0; i0 < kLoads && i0 * kStoreThreads < m * kPieces; i0 += kBatch) {
      uint4 v[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int u = tid + (i0 + i) * kStoreThreads;
        if (u < m * kPieces) v[i] = piece(u);
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int u = tid + (i0 + i) * kStoreThreads;
        if (u >= m * kPieces) break;
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        uint8_t* q = dst + (u / kPieces) * c.ld + (u % kPieces) * kPer;
        if constexpr (sizeof(T) == 2) {
          uint32_t y[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            y[j] = to_e4m3x2(__uint_as_float(w[j] << 16) * f, __uint_as_float(w[j] & 0xffff0000u) * f);
          *reinterpret_cast<uint2*>(q) = make_uint2(y[0] | (y[1] << 16), y[2] | (y[3] << 16));
        } else {
          *reinterpret_cast<uint32_t*>(q) =
              to_e4m3x2(__uint_as_float(w[0]) * f, __uint_as_float(w[1]) * f) |
              (to_e4m3x2(__uint_as_float(w[2]) * f, __uint_as_float(w[3]) * f) << 16);
        }
      }
    }
    if (tid == 0) c.exps[page] = static_cast<int8_t>(e);
    r += m;
    __syncthreads();                                // red is written again
  }
}

}  // namespace

cudaError_t launch_kv8_store(const Kv8StoreArgs& a_in, bool f32, int num_sms, cudaStream_t stream) {
  Kv8StoreArgs a = a_in;
  // One row a CTA while that fills the device (decode: every row begins a block
  // of its own), up to a block's 64 rows a CTA for long runs.
  a.rows_per_cta = min(64, max(1, a.n_rows / (4 * num_sms)));
  const int grid = (a.n_rows + a.rows_per_cta - 1) / a.rows_per_cta;
  if (f32)
    kv8_store_kernel<float><<<grid, kStoreThreads, 0, stream>>>(a);
  else
    kv8_store_kernel<__nv_bfloat16><<<grid, kStoreThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace dsa
