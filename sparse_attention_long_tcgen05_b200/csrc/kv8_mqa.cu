// kv8_mqa.cu -- MQA attention over the 8-bit latent cache, over a selection or
// over every preceding key, on the 5th-generation tensor cores.
//
//   O[t,h] = sum_s softmax_s(scale * q[t,h] . kv[s]) * kv[s, 0:512],
//   kv[s] = decode(codes[s]) * 2^e(block of s)
//
// Everything runs on kind::f8f6f4: the cache's codes go from HBM into the
// operand tiles as they are, and the other operand is made to fit them.
//   - A query head becomes two e4m3 terms that together hold its bf16 values
//     (stage_q8), side by side as N = 2 x heads columns: one pass over the keys
//     gives both partial logits, which are added in fp32.
//   - A probability becomes two e5m2 terms, p ~ hi + lo, each added into the same
//     accumulator: together they carry p to 2^-7 at worst and 0.24 % in the rms (bf16:
//     2^-8, 0.16 %) down to 2^-20 of the running maximum, and smaller ones to 2^-26
//     of it, so that a key which takes nearly all the probability does not flush the
//     others. Measured against 64 bits, rms over the output: 0.17 to 0.23 %, of which
//     the output's own rounding to bf16 is 0.17 %. (Two e4m3 terms are more exact near
//     the maximum but end 2^-18 below it. A second term in e4m3 alone halves the
//     error, to bf16's 2^-8, but only above 2^-10 of the maximum, below which three
//     bits are left; P' has to stay below 2^12 for it, so the maximum moves more often:
//     1021-query chunk 701 -> 723 us with a shift of 2^7, 757 with 2^9.)
//   - The block scales are per key, and the keys lie on TMEM lanes (S^T = K Q^T,
//     M = 128 keys): each thread owns one key and multiplies by its scale. With
//     z the logits in log2 units, P' = 2^(z + e - M) is what multiplies the codes;
//     the running maximum M is taken over z + e, and the softmax sum is that of
//     P' 2^-e, so no other rescaling is needed. A row whose latent codes are all
//     zero adds to the sum alone, and in a block that an outlier has scaled up its
//     z + e would hide the others: it counts with an e of -96. Every other
//     row gives the output at least 2^-18 of 448 2^(z + e), so M is never further
//     than that above what the rows give.
// The value product runs transposed as well, O^T = V^T P (M = 128 value columns,
// N = heads): V^T is the key tile itself read MN-major, so each cached byte is
// staged once and used by both products, and O of 64 heads takes 256 of the 512
// TMEM columns of one SM. One CTA works on up to 64 heads; more heads are
// spread over two CTAs that walk the same keys side by side (the second reads
// them from L2). The tensor cores keep 25 bits of a sum and cut the rest: 1024 tiles
// of one sign lose less than 3e-4 of it, below the bf16 rounding of the output.
//
// A small-N MMA is bound by its operand reads from shared memory (4 KB of keys +
// N x 32 bytes, 128 bytes a cycle; measured 64, 48, 40 and 39 cycles for N = 128, 64,
// 32, 16), so a tile of 128 keys takes 18 x 64 + 32 x 48 = 2690 cycles at 64 heads
// and 18 x 40 + 32 x 39 = 1970 at 16. Against that stand 73.7 KB a tile from HBM: 3200
// cycles at the device's 6.56 TB/s. So few heads are bound by HBM and 128 heads by
// the tensor pipe (at 0.8 of what the bf16 rate would allow). As measured a tile of
// 64 heads takes ~4000 cycles: with 8 slots the copies of tile g + 2 wait for the
// values of tile g, and 1900 cycles of copy latency, the logits, 2250 cycles of
// softmax and the first value chunk of g + 2 follow one another, so two tiles take
// ~8200. ncu: tensor pipe 51 %, issue slots 47 %, L1 62 %.
//
// Work split: the tiles of all queries in a row are cut into equal ranges, one
// per CTA (per pair of CTAs above 64 heads), so ragged lengths, single queries
// and large batches all fill the device. A query cut by a range end leaves
// fp32 partial results that a second kernel joins.
//
// Roles: 16 warps (64 heads; else 8) for softmax and epilogue: warp w takes keys
// 32 (w & 3) .. of the tile, each four warps 16 heads (8 of 16); then one warp that
// issues the logits' MMAs, one that issues the values', and four that copy. (One
// issuing warp that polled for whichever could go on was bound by its own
// polling: 400 cycles a unit of 4 or 8 MMAs.)
#include <algorithm>

#include "kv8_gather.cuh"
#include "kv8_split.cuh"

namespace dsa {
namespace {

constexpr int kMaxWorkers = 148;
// P' is scaled by 2^kShift and kept within [0, kTop], e5m2's largest binade: the
// maximum M is only moved when a tile exceeds it by more than 2^6.
constexpr float kShift = 9.f;
constexpr float kTop = 32768.f;
// What a row without latent values has instead of its block's exponent when the
// maximum is taken: 2^17 such rows with the largest logit then sum to 2^122.
constexpr int kNoValuesExp = -96;
constexpr float kLn2 = 0.69314718055994531f;
// The largest |M| whose neighbours in fp32 (4 apart) still place the largest P'
// within kTop. A head whose maximum lies past it is NaN, not a guess: holding
// the maximum in two parts would give its one key instead, but cost every call 2 %.
constexpr float kMostM = 67108864.f;

// NP: heads of a CTA, padded. The ring takes what shared memory is left by the
// queries (2 NP x 576 bytes) and P: the tile whose logits are computed and the
// tile whose values are still wanted make 8 slots the least that keeps the
// tensor pipe from waiting for a copy in every tile (64 heads, 1021-query chunk:
// 944 us with 7 slots, 774 with 8 and an issuing warp for each product).
template <int NP> struct Cfg {
  static constexpr int kHeads = NP == 16 ? 8 : 16;   // heads of a softmax warp
  static constexpr int kSoftWarps = 4 * (NP / kHeads);
  static constexpr int kThreads = 32 * (kSoftWarps + 2 + kGatherWarps);
  static constexpr int kRing = NP == 64 ? 8 : NP == 32 ? 10 : 11;
  static constexpr int kMeta = NP == 64 ? 2 : 4;
  static constexpr uint32_t kTmem = NP == 64 ? 512 : NP == 32 ? 256 : 128;
  static constexpr uint32_t kColS = 4 * NP;          // two buffers of 2 NP columns
};

template <int NP>
struct Smem {
  Kv8Slots<Cfg<NP>::kRing> slots;
  alignas(1024) uint8_t q[2 * NP * 576];
  alignas(1024) uint8_t p[kTile * 128];              // row = key: first terms at byte 0, second at 64
  Kv8Ring<Cfg<NP>::kRing, Cfg<NP>::kMeta> ring;
  alignas(16) float head_scale[NP];                  // logit2 = (hi + lo / 16) 2^e head_scale
  alignas(16) float neg_ref[NP];                     // kShift - running maximum
  uint64_t q_full, p_full, pv_done, drained;
  uint64_t s_full[2], s_empty[2];
  uint32_t tmem_base;
  union {
    float tile_max[2][4][NP];                        // also the sums at a query's end
    int64_t scratch[Cfg<NP>::kThreads / 32 + 2];     // before the roles begin
  };
};

// Workspace: which query each worker's first and last range end cuts, then the
// partial results of slots 2 w (first) and 2 w + 1 (last).
struct Partials {
  int32_t* head_item;       // [workers] query cut by the worker's beginning, or -1
  int32_t* head_goes_on;    // [workers] 1: that query is cut by its end as well
  int32_t* tail_item;       // [workers] query that begins here and is cut by the end, or -1
  float2* ml;               // [2 workers][groups][NP] running maximum, sum
  float* o;                 // [2 workers][groups][NP][512]
  uint8_t* images;          // [n_q][groups] query operands (kv8_q8_kernel)
  float* factors;           // [n_q][groups][NP]
};

// Carves the workspace; returns its size. np: heads of a CTA, padded.
inline size_t carve(void* ws, int workers, int64_t n_q, int groups, int np, Partials* p) {
  const size_t rows = static_cast<size_t>(2) * workers * groups * np;
  const size_t o_bytes = rows * 512 * sizeof(float);
  const size_t ml_bytes = align256(rows * sizeof(float2));
  const size_t image_bytes = static_cast<size_t>(n_q) * groups * 2 * np * kRow8;
  const size_t factor_bytes = align256(static_cast<size_t>(n_q) * groups * np * sizeof(float));
  if (p != nullptr) {
    uint8_t* at = static_cast<uint8_t*>(ws);
    p->head_item = reinterpret_cast<int32_t*>(at);
    p->head_goes_on = p->head_item + kMaxWorkers;
    p->tail_item = p->head_goes_on + kMaxWorkers;
    p->o = reinterpret_cast<float*>(at += 2048);
    p->ml = reinterpret_cast<float2*>(at += o_bytes);
    p->images = at += ml_bytes;
    p->factors = reinterpret_cast<float*>(at + image_bytes);
  }
  return 2048 + o_bytes + ml_bytes + image_bytes + factor_bytes;
}
static_assert(3 * kMaxWorkers * sizeof(int32_t) <= 2048, "");

// Whether the row of a tile's key (its first chunk is the ring's `unit`) has any
// latent code other than zero: the first 16 nearly always tell. The tile's logits
// have been computed, so its chunks have landed; they stay until its value
// products are done. Looked at where the maximum is found anew only (1021-query
// chunk 681 -> 688 us, 64-sequence decode 58.1 -> 58.9; the copying warps reading
// them ahead from global memory instead: 690 and 61.6, 16 dense heads 103 -> 113).
template <int R, typename Ring>
__device__ __forceinline__ bool row_has_values(const Kv8Slots<R>& slots, Ring& ring, uint32_t unit, int key, int* status,
                                               uint64_t wait_ns, bool& ok) {
#pragma unroll 1
  for (uint32_t c = 0; c < 4; ++c, ++unit) {
    ok = mbar_wait(&ring.full[unit % R], (unit / R) & 1, status, wait_ns);
    if (!ok) return true;
    const uint4* const row = reinterpret_cast<const uint4*>(slots.chunk[unit % R] + key * 128);
#pragma unroll 1
    for (uint32_t x = 0; x < 8; ++x) {
      const uint4 v = row[x ^ (key & 7)];
      if (((v.x | v.y | v.z | v.w) & 0x7f7f7f7fu) != 0) return true;
    }
  }
  return false;
}

// kLimitArg: the pipeline waits take their bound from a.wait_ns.
template <int NP, bool kLimitArg>
__global__ void __launch_bounds__(Cfg<NP>::kThreads, 1)
kv8_mqa_kernel(const __grid_constant__ Kv8AttnArgs a, const __grid_constant__ Partials part, int groups,
               int group_heads, int workers, bool whole) {
  using C = Cfg<NP>;
  using Ring = Kv8Ring<C::kRing, C::kMeta>;
  constexpr int R = C::kRing, HN = C::kHeads, kQkWarp = C::kSoftWarps, kPvWarp = kQkWarp + 1;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Smem<NP>& S = *reinterpret_cast<Smem<NP>*>(smem_raw);
  const int warp = warp_id(), lane = threadIdx.x & 31;
  const int worker = blockIdx.x / groups, group = blockIdx.x % groups;
  const uint64_t wait_ns = kLimitArg ? a.wait_ns : kWaitLimitNs;
  const int head0 = group * group_heads;
  const int live = min(group_heads, a.heads - head0);
  if (smem_u32(smem_raw) & 1023u) {                  // (never: nothing static lies before it)
    report(a.status, DSA_ERR_CUDA);
    return;
  }

  const Kv8Range range = kv8_range<C::kThreads>(a.keys, a.idx != nullptr, a.k, worker, workers, whole, S.scratch);
  if (threadIdx.x == 0 && group == 0 && !whole) part.head_item[worker] = part.tail_item[worker] = -1;
  if (range.t0 == range.t1) return;
  if (threadIdx.x == 0) {
    S.ring.init();
    mbar_init(&S.q_full, 1);
    mbar_init(&S.p_full, C::kSoftWarps);
    mbar_init(&S.pv_done, 1);
    mbar_init(&S.drained, 2);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&S.s_full[b], 1);
      mbar_init(&S.s_empty[b], C::kSoftWarps);
    }
    fence_barrier_init();
  }
  if (warp == kQkWarp) tmem_alloc(&S.tmem_base, C::kTmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S.tmem_base;
  Kv8Pieces pieces(a, range);
  Kv8Piece pc;

  if (warp > kPvWarp) {
    // ------------------------------------------------------------ copies
    Kv8Gather<Ring> g{S.ring, S.slots, a, lane, warp - kPvWarp - 1, wait_ns};
    g.run(pieces);
    g.drain();
  } else if (warp == kQkWarp) {
    // ------------------------------------------------------------ S^T = K Q^T
    griddep_wait();                                  // the queries' operands
    kv8_logits<NP, R>(a, pieces, S.slots, S.ring, S.q, part.images, groups, group, &S.q_full, S.s_full, S.s_empty,
                      tmem + C::kColS, lane, wait_ns, [](uint32_t) {});
    // nothing is in flight when the block ends, whichever way it got here
    if (elect_one()) mma_commit(&S.drained);
    __syncwarp();
    mbar_wait_warp(&S.drained, 0, a.status);
  } else if (warp == kPvWarp) {
    // ------------------------------------------------------------ O^T += V^T P
    constexpr uint32_t idesc = make_idesc(NP, 0, 1, 1, 1);   // e4m3 codes, e5m2 probabilities
    const uint64_t p_desc = sw128_desc(smem_u32(S.p), 16384, 1024);
    const uint64_t v_desc = sw128_desc(smem_u32(S.slots.chunk[0]), 16384, 1024);
    uint32_t g = 0, slot = 0;
    bool ok = true;
    while (ok && pieces.next(pc)) {
      for (int j = 0; j < pc.n && ok; ++j, ++g) {
        ok = mbar_wait_warp(&S.p_full, g & 1, a.status, wait_ns);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint64_t vd = v_desc + slot * (kChunkB / 16);
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              mma_f8(tmem + c * NP, vd + 256 * k, p_desc + 256 * k, idesc, k > 0 || j > 0);
              mma_f8(tmem + c * NP, vd + 256 * k, p_desc + 256 * k + 4, idesc, 1);
            }
            mma_commit(&S.ring.empty[slot]);
            if (c == 3) mma_commit(&S.pv_done);
          }
          __syncwarp();
          if (++slot == R) slot = 0;
        }
      }
    }
    if (elect_one()) mma_commit(&S.drained);
    __syncwarp();
    mbar_wait_warp(&S.drained, 0, a.status);
  } else {
    // ------------------------------------------------------------ softmax and epilogue
    griddep_wait();                                  // the queries' factors
    const int sub = warp & 3;
    const int key = 32 * sub + lane;                 // this thread's key of each tile
    const int hb = (warp >> 2) * HN;                 // first of this warp's heads
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(32 * sub) << 16);
    const uint32_t s_col = C::kColS + hb;
    uint8_t* const p_row = S.p + key * 128;
    const uint32_t sw = key & 7;
    const uint32_t bar = 1 + (warp >> 2);            // the four warps of these heads
    constexpr uint32_t kBarAll = 1 + NP / HN;        // all softmax warps
    uint32_t g = 0;
    bool ok = true;
    bool more = pieces.next(pc);

    // factor of head hb + lane % HN of a query
    auto factor = [&](int qi) {
      return __ldcg(part.factors + (static_cast<int64_t>(qi) * groups + group) * NP + hb + lane % HN);
    };
    float next_factor = factor(pc.qi);

    // After a wait that ran out (reported) these warps go on without waiting: the
    // named barriers that they share are not bounded, so all of them must take
    // the same steps to the end.
    while (more) {
      // (all four warps of these heads write the same values, after the barriers
      // that end the last query)
      const float* const hs = S.head_scale + hb;
      if (lane < HN) S.head_scale[hb + lane] = next_factor;
      __syncwarp();
      if (pieces.left > 0) next_factor = factor(pc.qi + 1);
      float m_used = -INFINITY;                      // lane h % HN: running maximum of head hb + h
      uint64_t l[HN / 2];                            // this key's share of the sums, two heads a word
#pragma unroll
      for (int i = 0; i < HN / 2; ++i) l[i] = 0;
      for (int j = 0; j < pc.n; ++j, ++g) {
        const uint32_t b = g & 1;
        ok = ok && mbar_wait_warp(&S.ring.meta_full[g % C::kMeta], (g / C::kMeta) & 1, a.status, wait_ns) &&
             mbar_wait_warp(&S.s_full[b], (g >> 1) & 1, a.status, wait_ns);
        tc_fence_after();
        const int e_key = S.ring.key_exp[g % C::kMeta][key];
        const bool valid = e_key != kNoKey;
        const float ks = valid ? pow2i(e_key) : 0.f;
        uint64_t ks2 = f2_pack(ks, ks);
        uint64_t s[HN / 2];                          // (hi + lo / 16) 2^e, two heads a word
        {
          uint32_t v[HN], w[HN];
          tmem_ld<HN>(t_lane + s_col + b * (2 * NP), v);
          tmem_ld<HN>(t_lane + s_col + b * (2 * NP) + NP, w);
          tmem_wait_ld();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&S.s_empty[b]);
          const uint64_t k16 = f2_pack(0.0625f, 0.0625f);
#pragma unroll
          for (int i = 0; i < HN; i += 2)
            s[i / 2] = f2_mul(f2_fma(f2_pack(__uint_as_float(w[i]), __uint_as_float(w[i + 1])), k16,
                                     f2_pack(__uint_as_float(v[i]), __uint_as_float(v[i + 1]))), ks2);
        }
        // 2^(z - M) for the sum and P' = 2^(z + e - M) in fp16, with the maximum as
        // it stands; where P' is over kTop by it (in a query's first
        // tile, and at a head's first key, always) it is found anew
        const bool all_valid = __all_sync(0xffffffffu, valid);
        uint64_t w[HN / 2];
        __half2 p[HN / 2];
        auto weigh = [&]() {
          const ulonglong2* f4 = reinterpret_cast<const ulonglong2*>(hs);
          const ulonglong2* r4 = reinterpret_cast<const ulonglong2*>(S.neg_ref + hb);
#pragma unroll
          for (int i = 0; i < HN / 2; i += 2) {
            const ulonglong2 f = f4[i / 2], r = r4[i / 2];
            w[i] = f2_fma(s[i], f.x, r.x);
            w[i + 1] = f2_fma(s[i + 1], f.y, r.y);
          }
          if (!all_valid) {
#pragma unroll
            for (int i = 0; i < HN / 2; ++i)
              if (!valid) w[i] = f2_pack(-INFINITY, -INFINITY);
          }
#pragma unroll
          for (int i = 0; i < HN / 2; ++i) {
            const float2 x = f2_unpack(w[i]);
            w[i] = f2_pack(ex2(x.x), ex2(x.y));
            const float2 y = f2_unpack(f2_mul(w[i], ks2));
            p[i] = __floats2half2_rn(y.x, y.y);
          }
        };
        float alpha = 1.f;
        bool rescale = false;
        bool fresh = j == 0;
        if (!fresh) {
          weigh();
          __half2 top = p[0];
#pragma unroll
          for (int i = 1; i < HN / 2; ++i) top = __hmax2(top, p[i]);
          const float2 t2 = __half22float2(top);
          fresh = named_bar_any(bar, 128, fmaxf(t2.x, t2.y) > kTop);
        }
        if (fresh) {
          float mine = -INFINITY;
          bool landed = true;
          const bool none = ok && valid && !row_has_values<R>(S.slots, S.ring, 4 * g, key, a.status, wait_ns, landed);
          ok = __all_sync(0xffffffffu, landed) && ok;
          if (none) ks2 = 0;                         // any finite P' does for a row without values
          const float e_add = valid ? static_cast<float>(none ? kNoValuesExp : e_key) : -INFINITY;
#pragma unroll
          for (int i = 0; i < HN; ++i) {
            const float2 x = f2_unpack(s[i / 2]);
            const float m = warp_max(fmaf(i % 2 ? x.y : x.x, hs[i], e_add));
            if (lane % HN == i) mine = m;
          }
          if (lane < HN) S.tile_max[b][sub][hb + lane] = mine;
          named_bar_sync(bar, 128);
          float mx = -INFINITY;
#pragma unroll
          for (int t = 0; t < 4; ++t) mx = fmaxf(mx, S.tile_max[b][t][hb + lane % HN]);
          if (mx > -INFINITY) mx = fmaxf(mx, -kMostM);   // (a later tile may still be inside)
          if (mx > m_used) {
            alpha = ex2(m_used - mx);
            m_used = mx > kMostM ? NAN : mx;
          }
          rescale = j > 0;
          // (the four warps of these heads write the same values; without a key yet,
          // one that the first key exceeds)
          if (lane < HN) S.neg_ref[hb + lane] = m_used == -INFINITY ? 1e30f : kShift - m_used;
          __syncwarp();
          weigh();
          if (rescale) {
#pragma unroll
            for (int i = 0; i < HN; i += 2)
              l[i / 2] = f2_mul(l[i / 2], f2_pack(__shfl_sync(0xffffffffu, alpha, i),
                                                  __shfl_sync(0xffffffffu, alpha, i + 1)));
          }
        }
        uint32_t hi[HN / 4], lo[HN / 4];
#pragma unroll
        for (int i = 0; i < HN / 2; i += 2) {
          l[i] = f2_add(l[i], w[i]);
          l[i + 1] = f2_add(l[i + 1], w[i + 1]);
          split_e5m2x4(p[i], p[i + 1], hi[i / 2], lo[i / 2]);
        }
        // the value products of the tile before are done: P and O may be written
        if (g > 0) ok = ok && mbar_wait_warp(&S.pv_done, (g - 1) & 1, a.status, wait_ns);
        if (rescale) {
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int i = 0; i < HN; i += 8) {
              uint32_t o[8];
              tmem_ld8(t_lane + c * NP + hb + i, o);
              tmem_wait_ld();
#pragma unroll
              for (int t = 0; t < 8; ++t)
                o[t] = __float_as_uint(__uint_as_float(o[t]) * __shfl_sync(0xffffffffu, alpha, i + t));
              tmem_st8(t_lane + c * NP + hb + i, o);
            }
          tmem_wait_st();
        }
        if constexpr (HN == 8) {
          *reinterpret_cast<uint2*>(p_row + (sw << 4) + hb) = make_uint2(hi[0], hi[1]);
          *reinterpret_cast<uint2*>(p_row + ((4 ^ sw) << 4) + hb) = make_uint2(lo[0], lo[1]);
        } else {
          const uint32_t c = hb / 16;
          *reinterpret_cast<uint4*>(p_row + ((c ^ sw) << 4)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(p_row + (((c + 4) ^ sw) << 4)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.p_full);
      }
      const Kv8Piece done = pc;
      more = pieces.next(pc);

      // sums over the keys: lanes, then the four warps in order
      float ls[HN];
#pragma unroll
      for (int i = 0; i < HN / 2; ++i) {
        const float2 x = f2_unpack(l[i]);
        ls[2 * i] = x.x;
        ls[2 * i + 1] = x.y;
      }
      const float lw = reduce_columns<HN>(ls, lane);
      if (lane < HN) S.tile_max[g & 1][sub][hb + lane] = lw;
      named_bar_sync(bar, 128);
      const bool cut = done.n < done.tiles;
      const int64_t slot = 2 * worker + (done.j0 == 0 ? 1 : 0);
      const float* const sums = &S.tile_max[g & 1][0][hb + lane % HN];
      const float lt = ((sums[0] + sums[NP]) + sums[2 * NP]) + sums[3 * NP];
      const bool past = m_used == -kMostM;           // no key inside: a piece that counts for nothing, or NaN
      const float ref = m_used == -INFINITY ? 0.f : m_used - kShift;
      const float inv = past ? NAN : lt == 0.f ? 0.f : 1.f / lt;
      if (sub == 0 && lane < HN && hb + lane < live) {
        const int64_t h = head0 + hb + lane;
        if (cut)
          part.ml[(slot * groups + group) * NP + hb + lane] = make_float2(ref, past ? 0.f : lt);
        else if (a.lse != nullptr)
          a.lse[static_cast<int64_t>(done.qi) * a.heads + h] =
              past ? NAN : lt == 0.f ? -INFINITY : (ref + log2f(lt)) * kLn2;
      }
      ok = ok && mbar_wait_warp(&S.pv_done, (g - 1) & 1, a.status, wait_ns);
      tc_fence_after();
      // O^T: lane = value column, TMEM column = head
      if (cut) {
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          const int dim = c * 128 + 32 * sub + lane;
          uint32_t o[HN];
          tmem_ld<HN>(t_lane + c * NP + hb, o);
          tmem_wait_ld();
          float* dst = part.o + ((slot * groups + group) * NP + hb) * 512 + dim;
#pragma unroll
          for (int i = 0; i < HN; ++i)
            if (hb + i < live) dst[i * 512] = __uint_as_float(o[i]);
        }
      } else {
        // each warp turns its 32 columns x HN heads in a corner of the P tile (whose
        // last reader is done): words of two heads go in, and a lane takes 8 columns
        // of two heads out, 16 bytes a store
        uint32_t* const buf = reinterpret_cast<uint32_t*>(S.p) + warp * (16 * HN);
        __nv_bfloat16* const out =
            a.out + (static_cast<int64_t>(done.qi) * a.heads + head0 + hb) * 512 + 32 * sub;
        const int t2 = 2 * (lane >> 2), d8 = 8 * (lane & 3);
        float f[HN];
#pragma unroll
        for (int t = 0; t < HN; ++t) f[t] = __shfl_sync(0xffffffffu, inv, t);
        uint32_t o[HN];
        tmem_ld<HN>(t_lane + hb, o);
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          tmem_wait_ld();
#pragma unroll
          for (int t = 0; t < HN; t += 2) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(o[t]) * f[t],
                                                           __uint_as_float(o[t + 1]) * f[t + 1]);
            buf[t * 16 + lane] = *reinterpret_cast<const uint32_t*>(&v);
          }
          if (c < 3) tmem_ld<HN>(t_lane + (c + 1) * NP + hb, o);
          __syncwarp();
          if (t2 < HN) {
            const uint4 x = *reinterpret_cast<const uint4*>(buf + t2 * 16 + d8);
            const uint4 y = *reinterpret_cast<const uint4*>(buf + t2 * 16 + d8 + 4);
            __nv_bfloat16* const dst = out + t2 * 512 + c * 128 + d8;
            if (hb + t2 < live)
              *reinterpret_cast<uint4*>(dst) =
                  make_uint4(__byte_perm(x.x, x.y, 0x5410), __byte_perm(x.z, x.w, 0x5410),
                             __byte_perm(y.x, y.y, 0x5410), __byte_perm(y.z, y.w, 0x5410));
            if (hb + t2 + 1 < live)
              *reinterpret_cast<uint4*>(dst + 512) =
                  make_uint4(__byte_perm(x.x, x.y, 0x7632), __byte_perm(x.z, x.w, 0x7632),
                             __byte_perm(y.x, y.y, 0x7632), __byte_perm(y.z, y.w, 0x7632));
          }
          __syncwarp();
        }
        named_bar_sync(kBarAll, 32 * C::kSoftWarps); // the next P goes there
      }
      tc_fence_before();
      named_bar_sync(bar, 128);                      // the sums have been read
      if (threadIdx.x == 0 && group == 0) {
        if (cut && done.j0 > 0) {
          part.head_item[worker] = done.qi;
          part.head_goes_on[worker] = done.j0 + done.n < done.tiles;
        } else if (cut) {
          part.tail_item[worker] = done.qi;
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kQkWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmem);
  }
}

// Joins the pieces of each query that a range end cut. Block (w, x): the query
// that begins in worker w's range and goes on, four heads; its pieces are the last
// of worker w, then the first of the next workers that have any tiles, up to the
// one that does not go on. A thread takes four columns of a head, 128 a head.
constexpr int kJoinThreads = 512;

__global__ void __launch_bounds__(kJoinThreads, 4)
kv8_join_kernel(const __grid_constant__ Kv8AttnArgs a, const __grid_constant__ Partials part, int workers,
                int groups, int group_heads, int np) {
  __shared__ int32_t s_last;
  __shared__ int s_base[kJoinThreads / 32];
  __shared__ int16_t s_slot[kMaxWorkers];
  __shared__ float s_f[4][kMaxWorkers];              // factor of a piece, per head
  griddep_wait();
  const int w = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int qi = __ldcg(part.tail_item + w);
  const int i = w + 1 + tid;                         // (workers <= 148 < the threads)
  const bool mine = i < workers && __ldcg(part.head_item + i) == qi;
  const bool ends = mine && __ldcg(part.head_goes_on + i) == 0;
  if (qi < 0) return;
  if (ends) s_last = i;                              // one thread
  __syncthreads();
  const bool in = mine && i <= s_last;
  const uint32_t votes = __ballot_sync(0xffffffffu, in);
  if (lane == 0) s_base[warp] = __popc(votes);
  __syncthreads();
  int at = 1, n = 1;
#pragma unroll
  for (int x = 0; x < (kMaxWorkers + 31) / 32; ++x) {
    if (x < warp) at += s_base[x];
    n += s_base[x];
  }
  if (in) s_slot[at + __popc(votes & ((1u << lane) - 1u))] = static_cast<int16_t>(2 * i);
  if (tid == 0) s_slot[0] = static_cast<int16_t>(2 * w + 1);
  __syncthreads();
  const int hq = warp >> 2;                          // this thread's head of the four
  const int row = blockIdx.y * 4 + hq, group = row / np, h = row % np;   // (np is a multiple of 4)
  const bool live = h < min(group_heads, a.heads - group * group_heads);
  const int64_t head = static_cast<int64_t>(qi) * a.heads + group * group_heads + h;
  if ((warp & 3) == 0 && live) {                     // the factors, a warp a head
    float m = -INFINITY, l = 0.f;
    bool past = false;                               // a piece all of whose keys lie below -kMostM
    for (int x = lane; x < n; x += 32) {
      const float2 ml = __ldcg(part.ml + (static_cast<int64_t>(s_slot[x]) * groups + group) * np + h);
      if (ml.y != 0.f)
        m = fmaxf(m, ml.x);
      else
        past |= ml.x != 0.f;
    }
    past = __any_sync(0xffffffffu, past);
    m = warp_max(m);
    for (int x = lane; x < n; x += 32) {
      const float2 ml = __ldcg(part.ml + (static_cast<int64_t>(s_slot[x]) * groups + group) * np + h);
      const float f = ml.y != 0.f ? exp2f(ml.x - m) : 0.f;   // 0: no key of this piece counts
      s_f[hq][x] = f;
      l = fmaf(ml.y, f, l);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
    const float none = past ? NAN : 0.f;
    if (lane == 0 && a.lse != nullptr) a.lse[head] = l == 0.f ? none - INFINITY : (m + log2f(l)) * kLn2;
    const float inv = l == 0.f ? none : 1.f / l;
    __syncwarp();
    for (int x = lane; x < n; x += 32) s_f[hq][x] *= inv;
  }
  __syncthreads();
  if (!live) return;
  const int d4 = tid & 127;
  const int64_t stride = static_cast<int64_t>(groups) * np * 128;
  const float4* src = reinterpret_cast<const float4*>(part.o) + (static_cast<int64_t>(group) * np + h) * 128 + d4;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int x0 = 0; x0 < n; x0 += 4) {
    float4 v[4];
#pragma unroll
    for (int x = 0; x < 4; ++x)
      if (x0 + x < n) v[x] = __ldcg(src + s_slot[x0 + x] * stride);
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      if (x0 + x >= n) break;
      const float f = s_f[hq][x0 + x];
      o.x = fmaf(v[x].x, f, o.x);
      o.y = fmaf(v[x].y, f, o.y);
      o.z = fmaf(v[x].z, f, o.z);
      o.w = fmaf(v[x].w, f, o.w);
    }
  }
  const __nv_bfloat162 x = __floats2bfloat162_rn(o.x, o.y), y = __floats2bfloat162_rn(o.z, o.w);
  reinterpret_cast<uint2*>(a.out + head * 512)[d4] =
      make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
}

struct Split {
  int groups, group_heads, np, workers;
  bool whole;
};

// Head groups of at most 64, and as many workers as a B200 holds, but no more than
// there can be tiles. (A device with fewer SMs runs them in turn.)
// A cut costs its worker an fp32 result and the call a joining kernel, as much as
// about kCutTiles tiles. For selections, whose queries all have the same number of
// tiles, the ranges are whole queries where that is no slower: 64 decode queries of
// 16 tiles took 76 us cut for 74 workers and 64 us whole on 64.
constexpr int64_t kCutTiles = 6;

Split split(int32_t n_q, int32_t heads, int64_t max_keys, bool sparse) {
  Split s;
  s.groups = (heads + 63) / 64;
  s.group_heads = (heads + s.groups - 1) / s.groups;
  s.np = s.group_heads <= 16 ? 16 : s.group_heads <= 32 ? 32 : 64;
  const int64_t per = (max_keys + kTile - 1) / kTile, tiles = n_q * per;
  const int64_t most = kMaxWorkers / s.groups;
  s.workers = static_cast<int>(tiles < most ? tiles : most);
  s.whole = sparse && (n_q + most - 1) / most * per <= (tiles + most - 1) / most + kCutTiles;
  if (s.whole && n_q < s.workers) s.workers = n_q;
  return s;
}

template <int NP>
cudaError_t launch(const Kv8AttnArgs& a, const Split& s, const Partials& part, cudaStream_t stream) {
  const size_t smem = sizeof(Smem<NP>);
  static_assert(sizeof(Smem<NP>) <= 232448, "shared memory of one CTA");
  auto kernel = a.wait_ns != kWaitLimitNs ? kv8_mqa_kernel<NP, true> : kv8_mqa_kernel<NP, false>;
  cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  constexpr int kWarps = NP <= 32 ? NP : NP / 4;     // one head a warp where there are few, else four
  kv8_q8_kernel<NP, kWarps><<<a.keys.n_q * s.groups, 32 * kWarps, 0, stream>>>(
      a.q, a.ld_q, a.heads, s.groups, s.group_heads, a.scale_log2, part.images, part.factors);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return launch_dependent(kernel, dim3(s.workers * s.groups), Cfg<NP>::kThreads, smem, stream, a,
                          part, s.groups, s.group_heads, s.workers, s.whole);
}

// Queries of one pass: the operands of a long prefill would otherwise need as much
// workspace as its queries themselves. 16 queries a worker leave the last round
// of whole queries at most 1/16 idle.
int32_t pass_queries(int32_t n_q, int32_t heads) {
  const int32_t most = 16 * (kMaxWorkers / ((heads + 63) / 64));
  return n_q < most ? n_q : most;
}

}  // namespace

size_t kv8_mqa_workspace(int32_t n_q, int32_t heads, int64_t max_keys, bool sparse) {
  const int32_t most = pass_queries(n_q, heads);
  size_t bytes = 0;
  for (const int32_t n : {most, n_q % most}) {       // full passes and the last one
    if (n == 0) continue;
    const Split s = split(n, heads, max_keys, sparse);
    bytes = std::max(bytes, carve(nullptr, s.whole ? 0 : s.workers, n, s.groups, s.np, nullptr));
  }
  return bytes;
}

cudaError_t launch_kv8_mqa(const Kv8AttnArgs& all, int* launches, cudaStream_t stream) {
  const int64_t max_keys = all.idx != nullptr ? all.k
                           : all.keys.paged   ? static_cast<int64_t>(all.keys.max_pages) * 64
                                              : all.keys.n_keys;
  const int32_t most = pass_queries(all.keys.n_q, all.heads);
  for (int32_t q0 = 0; q0 < all.keys.n_q; q0 += most) {
    const Kv8AttnArgs a = kv8_block(all, q0, std::min(most, all.keys.n_q - q0));
    const Split s = split(a.keys.n_q, a.heads, max_keys, a.idx != nullptr);
    Partials part;
    carve(a.ws, s.whole ? 0 : s.workers, a.keys.n_q, s.groups, s.np, &part);
    cudaError_t e = s.np == 16   ? launch<16>(a, s, part, stream)
                    : s.np == 32 ? launch<32>(a, s, part, stream)
                                 : launch<64>(a, s, part, stream);
    if (e != cudaSuccess) return e;
    *launches += 2;
    if (s.whole) continue;
    e = launch_dependent(kv8_join_kernel, dim3(s.workers, s.groups * s.np / 4), kJoinThreads, 0, stream, a, part,
                         s.workers, s.groups, s.group_heads, s.np);
    if (e != cudaSuccess) return e;
    ++*launches;
  }
  return cudaSuccess;
}

}  // namespace dsa
