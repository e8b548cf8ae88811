// kv8_common.cuh -- what the kernels of the 8-bit latent cache (codes of 576-wide
// rows, one exponent per 64 tokens) share: e4m3 conversions, small tensor-core
// helpers, the split of the work, and the queries as two 8-bit terms.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "dsa_common.cuh"
#include "dsa_kernels.h"

namespace dsa {

constexpr int kRow8 = 576;       // bytes of one cached row
constexpr int kExpMin = -64;     // exponents of a block's scale 2^e
constexpr int kExpMax = 63;

__device__ __forceinline__ bool is_exponent(int e) { return e >= kExpMin && e <= kExpMax; }

// 2^e for e in [-126, 127]. Sums of two block exponents stay inside.
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }

// 2^e for e in [-149, 127]: below -126 a subnormal, whose product with a value
// large enough is exact all the same (no flushing to zero in this build).
__device__ __forceinline__ float pow2i_wide(int e) {
  return e >= -126 ? pow2i(e) : __int_as_float(1 << (149 + e));
}

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

// Sequence and position of query qi; pos -1 when it is out of range.
__device__ __forceinline__ bool kv8_query(const KeySide& ks, int qi, int& seq, int& pos) {
  if (ks.paged) return paged_query(ks, qi, seq, pos);
  seq = 0;
  pos = ks.n_keys - ks.n_q + qi;
  return true;
}

// ------------------------------------------------------------------ tensor-core pieces

// One lane of the (converged) warp: the MMA issuer's branch. Unlike a test of
// the lane number it leaves the code warp-uniform, so descriptors stay in
// uniform registers (measured: 48 instead of 55 cycles per small MMA).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// Descriptor of a K-major tile with 64-byte rows, 64-byte swizzle (512-byte
// aligned base; 8-row groups 512 bytes apart).
__device__ __forceinline__ uint64_t sw64_desc(uint32_t smem_addr) {
  return (static_cast<uint64_t>((smem_addr >> 4) & 0x3FFFu)) | (1ull << 16) |
         (static_cast<uint64_t>(512 >> 4) << 32) | (1ull << 46) | (4ull << 61);
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(taddr));
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}

// N consecutive TMEM columns of this thread's lane.
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[N]) {
  static_assert(N == 8 || N == 16 || N == 32, "");
  if constexpr (N == 8) tmem_ld8(taddr, r);
  if constexpr (N == 16) tmem_ld16(taddr, r);
  if constexpr (N == 32) tmem_ld32(taddr, r);
}

// 16 bytes global -> shared, or 16 zero bytes (the source is then not read).
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst_smem, const void* src, bool copy) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst_smem), "l"(src),
               "r"(copy ? 16 : 0)
               : "memory");
}

__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

// Whether any thread of the named barrier's has v; waits for all of them.
__device__ __forceinline__ bool named_bar_any(uint32_t id, uint32_t threads, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\t"
      "barrier.red.or.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(threads), "r"(v ? 1u : 0u)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two fp32 lanes in one instruction.
__device__ __forceinline__ uint64_t f2_pack(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 f2_unpack(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Four nonnegative fp16 values as sums of two e5m2 terms, a byte each. An
// e5m2 code is the upper byte of the fp16 of its value, so the first term is
// the value rounded to its upper byte, and what is left over, exact in fp16, is
// rounded the same way (halves away from zero). A NaN is lost here.
__device__ __forceinline__ void split_e5m2x4(__half2 a, __half2 b, uint32_t& hi, uint32_t& lo) {
  const uint32_t ua = (*reinterpret_cast<const uint32_t*>(&a) + 0x00800080u) & 0xff00ff00u;
  const uint32_t ub = (*reinterpret_cast<const uint32_t*>(&b) + 0x00800080u) & 0xff00ff00u;
  const __half2 ra = __hsub2(a, *reinterpret_cast<const __half2*>(&ua));
  const __half2 rb = __hsub2(b, *reinterpret_cast<const __half2*>(&ub));
  hi = __byte_perm(ua, ub, 0x7531);
  lo = __byte_perm(*reinterpret_cast<const uint32_t*>(&ra) + 0x00800080u,
                   *reinterpret_cast<const uint32_t*>(&rb) + 0x00800080u, 0x7531);
}

// Sums v[i] over the 32 lanes; lane l gets the sum of element l % N. The order
// of the additions is fixed.
template <int N>
__device__ __forceinline__ float reduce_columns(float (&v)[N], int lane) {
#pragma unroll
  for (int off = 16; off >= N; off >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], off);
#pragma unroll
  for (int off = N / 2; off >= 1; off >>= 1) {
    const bool up = (lane & off) != 0;
#pragma unroll
    for (int i = 0; i < off; ++i) {
      const float give = up ? v[i] : v[i + off];
      const float keep = up ? v[i + off] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, off);
    }
  }
  return v[0];
}

// ------------------------------------------------------------------ work split

constexpr int kTile = 128;       // keys of a tile = MMA M (keys on TMEM lanes)

// Tiles of query qi: fixed for a selection, else those of keys 0..pos (one,
// wholly masked, where there is none).
__device__ __forceinline__ int kv8_tiles(const KeySide& ks, bool sparse, int k, int qi) {
  if (sparse) return (k + kTile - 1) / kTile;
  int seq, pos;
  kv8_query(ks, qi, seq, pos);
  return pos / kTile + 1;
}

// The tiles of all queries in a row, cut into `workers` equal ranges, whatever
// their queries' lengths.
struct Kv8Range {
  int64_t t0, t1;     // this worker's tiles
  int qi;             // query of tile t0
  int j0;             // tile t0 within it
};

// Executed by the whole block (THREADS threads); scratch: THREADS / 32 + 2 words.
// whole (selections only): ranges of whole queries instead.
template <int THREADS>
__device__ __forceinline__ Kv8Range kv8_range(const KeySide& ks, bool sparse, int k, int worker,
                                              int workers, bool whole, int64_t* scratch) {
  Kv8Range r{};
  if (sparse) {
    const int64_t per = (k + kTile - 1) / kTile, total = per * ks.n_q;
    if (whole) {
      r.qi = static_cast<int>(static_cast<int64_t>(ks.n_q) * worker / workers);
      r.t0 = per * r.qi;
      r.t1 = per * (static_cast<int64_t>(ks.n_q) * (worker + 1) / workers);
      return r;
    }
    r.t0 = total * worker / workers;
    r.t1 = total * (worker + 1) / workers;
    r.qi = static_cast<int>(r.t0 / per);
    r.j0 = static_cast<int>(r.t0 % per);
    return r;
  }
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kW = THREADS / 32;
  // first the total, then the query that holds tile t0: one pass over the
  // queries each (the first pass's values are used again when it was the only one)
  int64_t total = 0, base = 0;
  for (int pass = 0; pass < 2; ++pass) {
    base = 0;
    for (int q0 = 0; q0 < ks.n_q; q0 += THREADS) {
      const int64_t mine = q0 + tid < ks.n_q ? kv8_tiles(ks, false, 0, q0 + tid) : 0;
      int64_t inc = mine;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int64_t up = __shfl_up_sync(0xffffffffu, inc, off);
        if (lane >= off) inc += up;
      }
      if (lane == 31) scratch[warp] = inc;
      __syncthreads();
      int64_t before = base, all = 0;
#pragma unroll
      for (int w = 0; w < kW; ++w) {
        if (w < warp) before += scratch[w];
        all += scratch[w];
      }
      const bool only = ks.n_q <= THREADS;
      if (only) {
        total = all;
        r.t0 = total * worker / workers;
        r.t1 = total * (worker + 1) / workers;
      }
      if ((only || pass == 1) && mine > 0 && before + inc - mine <= r.t0 && r.t0 < before + inc) {
        scratch[kW] = q0 + tid;
        scratch[kW + 1] = r.t0 - (before + inc - mine);
      }
      base += all;
      __syncthreads();
      if (only) pass = 1;
    }
    total = base;
    r.t0 = total * worker / workers;
    r.t1 = total * (worker + 1) / workers;
  }
  if (r.t1 > r.t0) {
    r.qi = static_cast<int>(scratch[kW]);
    r.j0 = static_cast<int>(scratch[kW + 1]);
  }
  __syncthreads();
  return r;
}

// One query's part of a worker's range.
struct Kv8Piece {
  int qi, j0, n, tiles;     // tiles [j0, j0 + n) of the query's `tiles`
};

struct Kv8Pieces {
  const Kv8AttnArgs& a;
  int64_t left;
  int qi, j0;
  __device__ Kv8Pieces(const Kv8AttnArgs& args, const Kv8Range& r)
      : a(args), left(r.t1 - r.t0), qi(r.qi), j0(r.j0) {}
  __device__ __forceinline__ bool next(Kv8Piece& p) {
    if (left <= 0) return false;
    p.qi = qi;
    p.j0 = j0;
    p.tiles = kv8_tiles(a.keys, a.idx != nullptr, a.k, qi);
    p.n = static_cast<int>(min(left, static_cast<int64_t>(p.tiles - j0)));
    left -= p.n;
    ++qi;
    j0 = 0;
    return true;
  }
};

// ------------------------------------------------------------------ queries as two e4m3 terms

// Writes the queries of ROWS heads (of which `live` exist) as the image of a B operand: row
// h of the tiles is e4m3(q 2^-s), row ROWS + h is e4m3 of 16 times what that left
// over, with s per head so that the largest element lies in [128, 256). The two
// terms hold a bf16 element exactly down to 2^-14 of the head's largest one and
// miss smaller ones by at most 2^-22 of it: the products with the cache's codes
// are as exact as the codes themselves. Four 128-byte-swizzled chunks of 128
// columns, 2 ROWS rows each, then the rope columns in 64-byte rows.
// Returns through set(h, s) the exponent of each head. An infinity or NaN makes
// the whole head NaN. Warp `warp` of WARPS takes ROWS / WARPS heads in a row.
// Each warp fetches its heads (up to four at a time) with 16-byte loads: two for
// the latent columns of a head, and one for the rope columns of four heads.
struct Q8Pieces {
  uint32_t hi[2], lo[2];                            // 8 codes of each term
};

// 8 bf16 times f = 2^(-s - 8). The fp16 of 2^-8 times a value has that value's
// e4m3 code in bits 7 to 14, below the sign.
__device__ __forceinline__ Q8Pieces split_q8(uint4 v, float f, bool bad) {
  const __half2 k4096 = __float2half2_rn(4096.f);   // 2^8 back, 16 of the second term
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  Q8Pieces r;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t h[2], l[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const __half2 x = __floats2half2_rn(__uint_as_float(w[2 * i + j] << 16) * f,
                                          __uint_as_float(w[2 * i + j] & 0xffff0000u) * f);
      const uint32_t u = (*reinterpret_cast<const uint32_t*>(&x) + 0x00400040u) & 0xff80ff80u;
      const __half2 rest = __hsub2(x, *reinterpret_cast<const __half2*>(&u));
      h[j] = ((u << 1) & 0x7f007f00u) | (u & 0x80008000u);
      l[j] = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(__hmul2(rest, k4096)), __NV_SATFINITE,
                                        __NV_E4M3);
    }
    r.hi[i] = bad ? 0x7f7f7f7fu : __byte_perm(h[0], h[1], 0x7531);
    r.lo[i] = bad ? 0x7f7f7f7fu : l[0] | (l[1] << 16);
  }
  return r;
}

__device__ __forceinline__ uint32_t bf16_amax(uint4 v) {   // as bits
  const uint32_t a = __vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu);
  const uint32_t b = __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu);
  const uint32_t c = __vmaxu2(a, b);
  return max(c & 0xffffu, c >> 16);
}

template <int ROWS, int WARPS, typename F>
__device__ __forceinline__ void stage_q8(uint8_t* tile, const __nv_bfloat16* q, int live, int warp,
                                         int lane, F set) {
  constexpr int kChunk = 2 * ROWS * 128;
  constexpr int kPerWarp = ROWS / WARPS, kBatch = kPerWarp < 4 ? kPerWarp : 4;
  static_assert(ROWS % WARPS == 0 && kPerWarp % kBatch == 0, "");
#pragma unroll 1
  for (int r0 = 0; r0 < kPerWarp; r0 += kBatch) {
    const int h0 = warp * kPerWarp + r0;            // heads h0 .. h0 + kBatch - 1
    const uint4* src = reinterpret_cast<const uint4*>(q + static_cast<int64_t>(h0) * kRow8);
    const uint4 none = make_uint4(0u, 0u, 0u, 0u);
    uint4 v[kBatch][2];
#pragma unroll
    for (int r = 0; r < kBatch; ++r) {
      v[r][0] = h0 + r < live ? __ldg(src + 72 * r + lane) : none;
      v[r][1] = h0 + r < live ? __ldg(src + 72 * r + 32 + lane) : none;
    }
    const int rr = lane >> 3;                       // the head whose rope columns this lane takes
    const uint4 vr = rr < kBatch && h0 + rr < live ? __ldg(src + 72 * rr + 64 + (lane & 7)) : none;
    uint32_t mr = bf16_amax(vr);
#pragma unroll
    for (int off = 4; off >= 1; off >>= 1) mr = max(mr, __shfl_xor_sync(0xffffffffu, mr, off));
    float f_mine = 0.f;                             // of head rr
    bool bad_mine = false;
#pragma unroll
    for (int r = 0; r < kBatch; ++r) {
      const int h = h0 + r;
      const uint32_t m = max(__reduce_max_sync(0xffffffffu, max(bf16_amax(v[r][0]), bf16_amax(v[r][1]))),
                             __shfl_sync(0xffffffffu, mr, 8 * r));
      const bool bad = m >= 0x7f80u;
      const int s = min(max(static_cast<int>(m >> 7) - 127 - 7, -112), 120);
      const float f = pow2i_wide(-s - 8);            // (s up to 120: 2^-128)
      if (rr == r) {
        f_mine = f;
        bad_mine = bad;
      }
      if (lane == 0) set(h, s);
      // lane's 8 columns 8 lane (+ 256): chunk lane / 16 (+ 2), 8-byte half of a 16-byte unit
      uint8_t* const at = tile + (lane >> 4) * kChunk + h * 128 + ((((lane & 15) >> 1) ^ (h & 7)) << 4) + 8 * (lane & 1);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const Q8Pieces c = split_q8(v[r][i], f, bad);
        *reinterpret_cast<uint2*>(at + 2 * i * kChunk) = make_uint2(c.hi[0], c.hi[1]);
        *reinterpret_cast<uint2*>(at + 2 * i * kChunk + ROWS * 128) = make_uint2(c.lo[0], c.lo[1]);
      }
    }
    if (rr < kBatch) {
      const int h = h0 + rr;
      const Q8Pieces c = split_q8(vr, f_mine, bad_mine);
      uint8_t* const at = tile + 4 * kChunk + h * 64 + ((((lane & 7) >> 1) ^ ((h >> 1) & 3)) << 4) + 8 * (lane & 1);
      *reinterpret_cast<uint2*>(at) = make_uint2(c.hi[0], c.hi[1]);
      *reinterpret_cast<uint2*>(at + ROWS * 64) = make_uint2(c.lo[0], c.lo[1]);
    }
  }
}

// Bytes of one such image, and of a head group's scales behind it.
template <int ROWS>
constexpr int kQ8Bytes = 2 * ROWS * kRow8;

// Copies `bytes` (a multiple of 16, both addresses 16-byte aligned) from global
// into this CTA's shared memory, counted on `bar` (complete_tx).
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// One query's head group per block: its operand image and, per head, the factor
// that turns hi + lo / 16 into base-2 logits. This is a kernel of its own, before the
// attention: there the conversion (~250 instructions a head and warp) stood
// between one query and the next, 6700 cycles of every 64-head query.
template <int ROWS, int WARPS>
__global__ void __launch_bounds__(32 * WARPS)
kv8_q8_kernel(const __nv_bfloat16* q, int64_t ld_q, int heads, int groups, int group_heads,
              float scale_log2, uint8_t* images, float* factors) {
  griddep_launch_dependents();
  const int64_t item = blockIdx.x;                  // query * groups + group
  const int head0 = static_cast<int>(item % groups) * group_heads;
  stage_q8<ROWS, WARPS>(images + item * kQ8Bytes<ROWS>,
                        q + (item / groups) * ld_q + static_cast<int64_t>(head0) * kRow8,
                        min(group_heads, heads - head0), threadIdx.x >> 5, threadIdx.x & 31,
                        [&](int h, int s) { factors[item * ROWS + h] = scale_log2 * pow2i(s); });
}

}  // namespace dsa
