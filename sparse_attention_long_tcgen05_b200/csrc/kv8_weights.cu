// kv8_weights.cu -- the running attention weight of each cached token.
//
//   w[i,s] = (1/H) sum_h exp(scale * q[i,h] . kv[s] - lse[i,h])
//   acc[b,s] = decay * acc[b,s] + sum over b's queries i, ascending, of w[i,s]
//
// The first kernel computes w per query the way the attention computes its
// logits (kv8_mqa.cu): S^T = K Q^T on kind::f8f6f4 with every head's query as two
// e4m3 terms, N = 2 x heads columns (up to 256: one CTA takes all heads). With the
// keys on TMEM lanes the sum over the heads is a thread's own sum over its
// columns. No value product follows, so a chunk's ring slot is free as soon as
// its MMAs are done, and four slots suffice beside the queries of 128 heads
// (147 KB). A tile of 128 keys costs 18 x 128 tensor cycles at 128 heads, against
// 3200 cycles for its 73.7 KB at the device's HBM rate.
//
// The second kernel adds the queries of a sequence in their order, so that the
// sums do not depend on which finishes first. Within one query an entry that
// repeats a key adds the same bits as the first, so the order of those two does
// not matter either, and they may be added with atomics.
#include <algorithm>

#include "kv8_gather.cuh"
#include "kv8_split.cuh"

namespace dsa {
namespace {

constexpr int kAccThreads = 256;

template <int NP> struct Cfg {
  static constexpr int kHeads = NP == 128 ? 32 : 16;  // heads of a summing warp
  static constexpr int kSumWarps = 4 * (NP / kHeads);
  static constexpr int kThreads = 32 * (kSumWarps + 1 + kGatherWarps);
  static constexpr int kRing = NP == 128 ? 4 : NP == 64 ? 8 : 11;
  static constexpr uint32_t kTmem = 4 * NP < 32 ? 32 : 4 * NP;   // two buffers of 2 NP columns
};

template <int NP>
struct Smem {
  Kv8Slots<Cfg<NP>::kRing> slots;
  alignas(1024) uint8_t q[2 * NP * kRow8];
  Kv8Ring<Cfg<NP>::kRing, 8> ring;
  alignas(16) float head_scale[NP];                  // logit2 = (hi + lo / 16) 2^e head_scale
  alignas(16) float neg_lse[NP];                     // - lse log2(e)
  float sum[2][NP / Cfg<NP>::kHeads][kTile];         // of each group of heads
  int64_t scratch[Cfg<NP>::kThreads / 32 + 2];
  uint64_t q_full, drained, s_full[2], s_empty[2];
  uint32_t tmem_base;
};

// kLimitArg: the pipeline waits take their bound from a.wait_ns.
template <int NP, bool kLimitArg>
__global__ void __launch_bounds__(Cfg<NP>::kThreads, 1)
kv8_weights_kernel(const __grid_constant__ Kv8WeightArgs wa, const uint8_t* images, const float* factors) {
  using C = Cfg<NP>;
  using Ring = Kv8Ring<C::kRing, 8>;
  constexpr int R = C::kRing, HN = C::kHeads, kQkWarp = C::kSumWarps;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Smem<NP>& S = *reinterpret_cast<Smem<NP>*>(smem_raw);
  const Kv8AttnArgs& a = wa.attn;
  const uint64_t wait_ns = kLimitArg ? a.wait_ns : kWaitLimitNs;
  const int warp = warp_id(), lane = threadIdx.x & 31;
  if (smem_u32(smem_raw) & 1023u) {                  // (never: nothing static lies before it)
    report(a.status, DSA_ERR_CUDA);
    return;
  }
  const Kv8Range range = kv8_range<C::kThreads>(a.keys, a.idx != nullptr, a.k, blockIdx.x, gridDim.x, false, S.scratch);
  if (range.t0 == range.t1) return;
  if (threadIdx.x == 0) {
    S.ring.init();
    mbar_init(&S.q_full, 1);
    mbar_init(&S.drained, 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&S.s_full[b], 1);
      mbar_init(&S.s_empty[b], C::kSumWarps);
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

  if (warp > kQkWarp) {
    Kv8Gather<Ring> g{S.ring, S.slots, a, lane, warp - kQkWarp - 1, wait_ns};
    g.run(pieces);
    g.drain();
  } else if (warp == kQkWarp) {
    griddep_wait();                                  // the queries' operands
    kv8_logits<NP, R>(a, pieces, S.slots, S.ring, S.q, images, 1, 0, &S.q_full, S.s_full, S.s_empty, tmem, lane, wait_ns,
                      [&](uint32_t slot) { mma_commit(&S.ring.empty[slot]); });
    if (elect_one()) mma_commit(&S.drained);
    __syncwarp();
    mbar_wait_warp(&S.drained, 0, a.status);
  } else {
    griddep_wait();                                  // the queries' factors
    const int sub = warp & 3, grp = warp >> 2;
    const int key = 32 * sub + lane, hb = grp * HN;
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(32 * sub) << 16);
    const float inv_heads = 1.f / static_cast<float>(a.heads);
    uint32_t g = 0;
    bool ok = true;
    // After a wait that ran out (reported) these warps go on without waiting: the
    // named barrier that they share is not bounded.
    while (pieces.next(pc)) {
      named_bar_sync(1, 32 * C::kSumWarps);          // the last query's factors have been used
      for (int h = threadIdx.x; h < NP; h += 32 * C::kSumWarps) {
        S.head_scale[h] = __ldcg(factors + static_cast<int64_t>(pc.qi) * NP + h);
        const float lse = h < a.heads ? __ldg(wa.lse + static_cast<int64_t>(pc.qi) * a.heads + h) : -INFINITY;
        S.neg_lse[h] = lse == -INFINITY ? -INFINITY : -lse * 1.4426950408889634f;
      }
      named_bar_sync(1, 32 * C::kSumWarps);
      for (int j = 0; j < pc.n; ++j, ++g) {
        const uint32_t b = g & 1;
        ok = ok && mbar_wait_warp(&S.ring.meta_full[g % 8], (g / 8) & 1, a.status, wait_ns) &&
             mbar_wait_warp(&S.s_full[b], (g >> 1) & 1, a.status, wait_ns);
        tc_fence_after();
        const int e_key = S.ring.key_exp[g % 8][key];
        const bool valid = e_key != kNoKey;
        const float ks = valid ? pow2i(e_key) : 0.f;
        const uint64_t ks2 = f2_pack(ks, ks), k16 = f2_pack(0.0625f, 0.0625f);
        uint64_t sum = 0;
#pragma unroll
        for (int i0 = 0; i0 < HN; i0 += 16) {
          uint32_t v[16], w[16];
          tmem_ld<16>(t_lane + b * (2 * NP) + hb + i0, v);
          tmem_ld<16>(t_lane + b * (2 * NP) + NP + hb + i0, w);
          tmem_wait_ld();
          if (i0 + 16 == HN) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.s_empty[b]);
          }
          const ulonglong2* f4 = reinterpret_cast<const ulonglong2*>(S.head_scale + hb + i0);
          const ulonglong2* r4 = reinterpret_cast<const ulonglong2*>(S.neg_lse + hb + i0);
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            const ulonglong2 f = f4[i / 4], r = r4[i / 4];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              const int c = i + 2 * t;
              const uint64_t s = f2_mul(f2_fma(f2_pack(__uint_as_float(w[c]), __uint_as_float(w[c + 1])), k16,
                                               f2_pack(__uint_as_float(v[c]), __uint_as_float(v[c + 1]))), ks2);
              const float2 x = f2_unpack(f2_fma(s, t ? f.y : f.x, t ? r.y : r.x));
              sum = f2_add(sum, f2_pack(ex2(x.x), ex2(x.y)));
            }
          }
        }
        const float2 s2 = f2_unpack(sum);
        S.sum[b][grp][key] = s2.x + s2.y;
        named_bar_sync(1, 32 * C::kSumWarps);
        if (grp == 0) {
          float total = 0.f;
#pragma unroll
          for (int i = 0; i < NP / HN; ++i) total += S.sum[b][i][key];
          const int at = (pc.j0 + j) * kTile + key;
          if (at < wa.n_cols) wa.w[static_cast<int64_t>(pc.qi) * wa.n_cols + at] = valid ? total * inv_heads : 0.f;
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

// The queries of sequence b among c0 .. c0 + THREADS - 1, in ascending order, into
// list[] = (query, position); returns how many. Executed by the whole block, which
// meets before and after.
template <int THREADS>
__device__ __forceinline__ int list_queries(const KeySide& ks, int b, int c0, int2* list, int* counts) {
  const int i = c0 + threadIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  bool in = false;
  int seq, pos = -1;
  if (i < ks.n_q) {
    if (!ks.paged) {
      in = true;
      pos = ks.n_keys - ks.n_q + i;
    } else {
      in = (ks.q_seq != nullptr ? __ldg(ks.q_seq + i) : i) == b && paged_query(ks, i, seq, pos);
    }
  }
  const uint32_t votes = __ballot_sync(0xffffffffu, in);
  __syncthreads();
  if (lane == 0) counts[warp] = __popc(votes);
  __syncthreads();
  int at = 0, n = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) at += counts[w];
    n += counts[w];
  }
  if (in) list[at + __popc(votes & ((1u << lane) - 1u))] = make_int2(i, pos);
  __syncthreads();
  return n;
}

// Cached tokens of sequence b (all of them: a pass may see only the keys of its queries).
__device__ __forceinline__ int seq_len(const Kv8WeightArgs& w, int b) {
  const KeySide& ks = w.attn.keys;
  if (!ks.paged) return w.n_keys;
  const int n = __ldg(ks.ctx_lens + b);
  return n < 0 || n > ks.max_pages * 64 ? 0 : n;
}

// Every key of the sequence: acc = decay * acc + the queries' weights.
__global__ void __launch_bounds__(kAccThreads)
kv8_acc_dense_kernel(const __grid_constant__ Kv8WeightArgs w, int blocks, bool add) {
  __shared__ int2 list[kAccThreads];
  __shared__ int counts[kAccThreads / 32];
  griddep_wait();
  const KeySide& ks = w.attn.keys;
  const int b = blockIdx.x / blocks;
  const int s = (blockIdx.x % blocks) * kAccThreads + threadIdx.x;
  const bool live = s < seq_len(w, b);
  float* acc = w.acc + b * w.ld_acc + s;
  float v = live ? *acc * w.decay : 0.f;
  if (add) {
    const bool one = ks.paged && ks.q_seq == nullptr;          // query b alone
    for (int c0 = one ? b / kAccThreads * kAccThreads : 0; c0 < ks.n_q; c0 += kAccThreads) {
      const int n = list_queries<kAccThreads>(ks, b, c0, list, counts);
#pragma unroll 4
      for (int x = 0; x < n; ++x) {
        const int2 q = list[x];
        if (live && s <= q.y) v += __ldcg(w.w + static_cast<int64_t>(q.x) * w.n_cols + s);
      }
      if (one) break;
    }
  }
  if (live) *acc = v;
}

// The selected keys: query after query, the next one's entries on their way.
__global__ void __launch_bounds__(1024)
kv8_acc_sparse_kernel(const __grid_constant__ Kv8WeightArgs w) {
  __shared__ int2 list[1024];
  __shared__ int counts[32];
  griddep_wait();
  const KeySide& ks = w.attn.keys;
  const int b = blockIdx.x, tid = threadIdx.x;
  float* acc = w.acc + b * w.ld_acc;
  struct Part {
    int p[2];              // (a selection has at most 2048 entries)
    float v[2];
  };
  auto load = [&](int2 q) {
    Part r;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int j = tid + 1024 * t;
      r.p[t] = j < w.n_cols ? __ldg(w.attn.idx + q.x * w.attn.ld_idx + j) : -1;
      r.v[t] = j < w.n_cols ? __ldcg(w.w + static_cast<int64_t>(q.x) * w.n_cols + j) : 0.f;
    }
    return r;
  };
  const bool one = ks.paged && ks.q_seq == nullptr;            // query b alone
  for (int c0 = one ? b / 1024 * 1024 : 0; c0 < ks.n_q; c0 += 1024) {
    const int n = list_queries<1024>(ks, b, c0, list, counts);
    Part next = n > 0 ? load(list[0]) : Part{};
    for (int x = 0; x < n; ++x) {
      const Part now = next;
      const int pos = list[x].y;
      if (x + 1 < n) next = load(list[x + 1]);
#pragma unroll
      for (int t = 0; t < 2; ++t)
        if (now.p[t] >= 0 && now.p[t] <= pos) atomicAdd(acc + now.p[t], now.v[t]);
      __syncthreads();
    }
    if (one) break;
  }
}

int padded_heads(int heads) { return heads <= 16 ? 16 : heads <= 32 ? 32 : heads <= 64 ? 64 : 128; }

template <int NP>
cudaError_t launch(const Kv8WeightArgs& w, int workers, uint8_t* images, float* factors, cudaStream_t stream) {
  static_assert(sizeof(Smem<NP>) <= 232448, "shared memory of one CTA");
  auto kernel = w.attn.wait_ns != kWaitLimitNs ? kv8_weights_kernel<NP, true> : kv8_weights_kernel<NP, false>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(sizeof(Smem<NP>)));
  if (e != cudaSuccess) return e;
  constexpr int kWarps = NP <= 32 ? NP : NP / 4;     // one head a warp where there are few, else four
  kv8_q8_kernel<NP, kWarps><<<w.attn.keys.n_q, 32 * kWarps, 0, stream>>>(
      w.attn.q, w.attn.ld_q, w.attn.heads, 1, w.attn.heads, w.attn.scale_log2, images, factors);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return launch_dependent(kernel, dim3(workers), Cfg<NP>::kThreads, sizeof(Smem<NP>), stream, w,
                          static_cast<const uint8_t*>(images), static_cast<const float*>(factors));
}

// Queries of one pass: their weights stay within 64 MB and their operands within
// what 2048 queries take.
int32_t pass_queries(int32_t n_q, int64_t n_cols) {
  const int64_t most = std::max<int64_t>(1, std::min<int64_t>(2048, (int64_t(16) << 20) / n_cols));
  return n_q < most ? n_q : static_cast<int32_t>(most);
}

size_t weights_bytes(int32_t n, int64_t n_cols) { return align256(static_cast<size_t>(n) * n_cols * sizeof(float)); }

// One pass over w's queries and n_seq sequences.
cudaError_t pass(const Kv8WeightArgs& w, int n_seq, int num_sms, int* launches, cudaStream_t stream) {
  const KeySide& ks = w.attn.keys;
  const int np = padded_heads(w.attn.heads);
  uint8_t* const images = reinterpret_cast<uint8_t*>(w.w) + weights_bytes(ks.n_q, w.n_cols);
  float* const factors = reinterpret_cast<float*>(images + static_cast<size_t>(ks.n_q) * (2 * np * kRow8));
  const int64_t tiles = static_cast<int64_t>(ks.n_q) * ((w.n_cols + kTile - 1) / kTile);
  const int workers = static_cast<int>(tiles < num_sms ? tiles : num_sms);
  cudaError_t e = np == 16   ? launch<16>(w, workers, images, factors, stream)
                  : np == 32 ? launch<32>(w, workers, images, factors, stream)
                  : np == 64 ? launch<64>(w, workers, images, factors, stream)
                             : launch<128>(w, workers, images, factors, stream);
  if (e != cudaSuccess) return e;
  *launches += 2;
  const bool dense = w.attn.idx == nullptr;
  if (dense || w.decay != 1.f) {
    const int64_t width = ks.paged ? static_cast<int64_t>(ks.max_pages) * 64 : w.n_keys;
    const int64_t blocks = (width + kAccThreads - 1) / kAccThreads;
    if (blocks * n_seq > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    e = launch_dependent(kv8_acc_dense_kernel, dim3(static_cast<unsigned>(blocks * n_seq)), kAccThreads, 0, stream,
                         w, static_cast<int>(blocks), dense);
    if (e != cudaSuccess) return e;
    ++*launches;
  }
  if (!dense) {
    if ((e = launch_dependent(kv8_acc_sparse_kernel, dim3(n_seq), 1024, 0, stream, w)) != cudaSuccess) return e;
    ++*launches;
  }
  return cudaSuccess;
}

}  // namespace

size_t kv8_accumulate_workspace(int32_t n_q, int32_t heads, int64_t n_cols) {
  const int32_t n = pass_queries(n_q, n_cols);
  const int np = padded_heads(heads);
  return weights_bytes(n, n_cols) + static_cast<size_t>(n) * (2 * np * kRow8) +
         align256(static_cast<size_t>(n) * np * sizeof(float));
}

cudaError_t launch_kv8_accumulate(const Kv8WeightArgs& all, int num_sms, int* launches,
                                  cudaStream_t stream) {
  const KeySide& ks = all.attn.keys;
  const int32_t most = pass_queries(ks.n_q, all.n_cols);
  for (int32_t q0 = 0; q0 < ks.n_q; q0 += most) {
    const int32_t n = std::min(most, ks.n_q - q0);
    const bool last = q0 + n == ks.n_q;
    Kv8WeightArgs w = all;
    w.attn = kv8_block(all.attn, q0, n);
    w.lse += static_cast<int64_t>(q0) * all.attn.heads;
    int n_seq = ks.paged ? ks.n_seq : 1;
    if (ks.paged && ks.q_seq == nullptr) {           // this pass's sequences, and in the last the rest
      w.acc += q0 * all.ld_acc;
      n_seq = last ? ks.n_seq - q0 : n;
    } else if (q0 > 0) {
      w.decay = 1.f;                                 // every sequence has decayed in the first pass
    }
    const cudaError_t e = pass(w, n_seq, num_sms, launches, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace dsa
