// kv8_split.cuh -- what the two tensor-core kernels over the 8-bit latent cache
// share besides the copies: a worker's logits' MMAs,
// and dependent launches.
#pragma once

#include "kv8_gather.cuh"

namespace dsa {

// The warp that issues S^T = K Q^T of a worker's tiles into the TMEM columns d0 + 2 NP
// (tile & 1): M = 128 keys, N = 2 NP; the 64 rope columns and four chunks of 128
// columns of each tile. taken(slot) is called by the issuing lane after a
// chunk's MMAs. images: the queries' operands (kv8_q8_kernel).
template <int NP, int R, typename Ring, typename F>
__device__ __forceinline__ void kv8_logits(const Kv8AttnArgs& a, Kv8Pieces& pieces, Kv8Slots<R>& slots, Ring& ring,
                                           uint8_t* q_tile, const uint8_t* images, int groups, int group,
                                           uint64_t* q_full, uint64_t* s_full, uint64_t* s_empty, uint32_t d0,
                                           int lane, uint64_t wait_ns, F taken) {
  constexpr uint32_t idesc = make_idesc(2 * NP, 0, 0, 0, 0);
  const uint64_t q_desc = sw128_desc(smem_u32(q_tile), 16, 1024);
  const uint64_t qr_desc = sw64_desc(smem_u32(q_tile) + 4 * (2 * NP * 128));
  const uint64_t k_desc = sw128_desc(smem_u32(slots.chunk[0]), 16384, 1024);
  const uint64_t r_desc = sw64_desc(smem_u32(slots.rope));
  uint32_t g = 0, slot = 0, phase = 0, n_piece = 0;
  Kv8Piece pc;
  bool ok = true;
  while (ok && pieces.next(pc)) {
    // the operand of the query, once the last one's logits are all computed
    if (g > 0) ok = mbar_wait_warp(&s_full[(g - 1) & 1], ((g - 1) >> 1) & 1, a.status, wait_ns);
    if (!ok) break;
    if (elect_one()) {
      const uint8_t* image = images + (static_cast<int64_t>(pc.qi) * groups + group) * kQ8Bytes<NP>;
      mbar_arrive_expect_tx(q_full, kQ8Bytes<NP>);
#pragma unroll 1
      for (int c = 0; c < 8; ++c)
        bulk_load(q_tile + c * (kQ8Bytes<NP> / 8), image + c * (kQ8Bytes<NP> / 8), kQ8Bytes<NP> / 8, q_full);
    }
    __syncwarp();
    ok = mbar_wait_warp(q_full, n_piece & 1, a.status, wait_ns);
    // (given up or not, no copy may land once the block has ended)
    if (!ok) mbar_wait_warp(q_full, n_piece & 1, a.status);
    ++n_piece;
    for (int j = 0; j < pc.n && ok; ++j, ++g) {
      const uint32_t d = d0 + (g & 1) * (2 * NP);
      ok = mbar_wait_warp(&s_empty[g & 1], ((g >> 1) & 1) ^ 1, a.status, wait_ns);
      ok = ok && mbar_wait_warp(&ring.rope_full, g & 1, a.status, wait_ns);
      fence_proxy_async_smem();                      // the copies, before the MMAs read them
      tc_fence_after();
      if (ok && elect_one()) {
#pragma unroll
        for (int k = 0; k < 2; ++k) mma_f8(d, r_desc + 2 * k, qr_desc + 2 * k, idesc, k != 0);
        mma_commit(&ring.rope_empty);
      }
      __syncwarp();
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        ok = ok && mbar_wait_warp(&ring.full[slot], phase, a.status, wait_ns);
        fence_proxy_async_smem();
        tc_fence_after();
        const uint64_t kd = k_desc + slot * (kChunkB / 16), qd = q_desc + c * (2 * NP * 128 / 16);
        if (ok && elect_one()) {
#pragma unroll
          for (int k = 0; k < 4; ++k) mma_f8(d, kd + 2 * k, qd + 2 * k, idesc, 1);
          taken(slot);
          if (c == 3) mma_commit(&s_full[g & 1]);
        }
        __syncwarp();
        if (++slot == R) {
          slot = 0;
          phase ^= 1;
        }
      }
    }
  }
}

// Queries q0 .. q0 + n - 1 of a call as a call of their own (out and lse included).
inline Kv8AttnArgs kv8_block(const Kv8AttnArgs& all, int32_t q0, int32_t n) {
  Kv8AttnArgs a = all;
  KeySide& ks = a.keys;
  a.q += q0 * all.ld_q;
  if (a.idx != nullptr) a.idx += q0 * all.ld_idx;
  if (a.out != nullptr) a.out += static_cast<int64_t>(q0) * all.heads * 512;
  if (a.lse != nullptr) a.lse += static_cast<int64_t>(q0) * all.heads;
  ks.n_q = n;
  if (!ks.paged) {
    ks.n_keys = all.keys.n_keys - all.keys.n_q + q0 + n;
  } else {
    if (ks.q_pos != nullptr) ks.q_pos += q0;
    if (ks.q_seq != nullptr) {
      ks.q_seq += q0;
    } else {               // query i is sequence i
      ks.block_table += q0 * ks.ld_block_table;
      ks.ctx_lens += q0;
      ks.n_seq -= q0;
    }
  }
  return a;
}

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// A kernel that may start while the one before it on the stream still runs
// (griddep_wait marks where it needs it).
template <typename... P, typename... A>
inline cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                             A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace dsa
