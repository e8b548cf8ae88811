// kv8_gather.cuh -- the copying warps of the kernels that read the 8-bit latent
// cache: rows of a tile's 128 keys into swizzled shared-memory tiles.
#pragma once

#include "kv8_common.cuh"

namespace dsa {

constexpr int kGatherWarps = 4;      // warp g copies keys 32 g .. 32 g + 31 of a tile
constexpr int kChunkB = kTile * 128; // 128 columns of a tile's keys: 16 KB
constexpr int kRopeB = kTile * 64;   // the 64 rope columns: 8 KB
constexpr int8_t kNoKey = -128;      // key_exp of a key that does not count

// Arrives on `bar` (one of its expected arrivals) when all copies that this
// thread has issued have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// The ring of a kernel: R chunk slots, one slot for the rope columns, and the
// exponent of each key of a tile. A kernel whose chunk slots are freed by the
// value products, after the tile's softmax, needs META = 2 exponent slots for R <=
// 8 (slot 4 n of the chunk order waits for chunk 4 n - 8 of tile n - 2) and 4 for
// R <= 12.
template <int R>
struct Kv8Slots {
  alignas(1024) uint8_t chunk[R][kChunkB];
  alignas(1024) uint8_t rope[kRopeB];
};

template <int R, int META>
struct Kv8Ring {
  static constexpr int kSlots = R, kMeta = META;
  int8_t key_exp[META][kTile];
  uint64_t full[R], empty[R];
  uint64_t rope_full, rope_empty;
  uint64_t meta_full[META];

  __device__ void init() {
    for (int i = 0; i < R; ++i) {
      mbar_init(&full[i], 32 * kGatherWarps);
      mbar_init(&empty[i], 1);
    }
    mbar_init(&rope_full, 32 * kGatherWarps);
    mbar_init(&rope_empty, 1);
    for (int i = 0; i < META; ++i) mbar_init(&meta_full[i], kGatherWarps);
  }
};

// One copying warp. Units of a tile in the order in which the MMAs want them:
// chunks 0, 1, 2, 3, then the rope columns. Every lane's arrival on a unit's barrier is
// made by the copy engine when that lane's copies have landed
// (cp.async.mbarrier.arrive.noinc), so a warp only ever waits for free slots and
// runs as far ahead as the ring allows; the MMA issuer, having waited, makes the
// copied bytes visible to the tensor core with a proxy fence of its own.
template <typename Ring>
struct Kv8Gather {
  static constexpr int R = Ring::kSlots, kMeta = Ring::kMeta;
  Ring& ring;
  Kv8Slots<R>& slots;
  const Kv8AttnArgs& a;
  int lane, g;             // g: copying warp 0..3
  uint32_t n_chunk = 0, n_rope = 0, n_tile = 0;

  // Key position of this lane's row in tile j of query qi: p in [0, pos], or -1;
  // bad: an entry past the query's position.
  __device__ __forceinline__ int key_of(int qi, int pos, int j, bool& bad) const {
    const int r = j * kTile + 32 * g + lane;
    if (a.idx == nullptr) return r <= pos ? r : -1;
    const int e = r < a.k ? __ldg(a.idx + static_cast<int64_t>(qi) * a.ld_idx + r) : -1;
    bad = e > pos;
    return e > pos ? -1 : e;
  }

  // Tiles [j0, j0 + n) of query qi. False when a wait ran out.
  __device__ bool run(int qi, int j0, int n) {
    int seq, pos;
    const bool q_ok = kv8_query(a.keys, qi, seq, pos);
    if (!q_ok && lane == 0) report(a.status, DSA_ERR_DEVICE_BOUNDS);
    bool bad = false, any_bad = false;
    int p = key_of(qi, pos, j0, bad);
    any_bad |= bad;
    int64_t row = p >= 0 ? kv8_row(a.keys, seq, p) : -1;
    for (int j = j0; j < j0 + n; ++j) {
      // the next tile's entries are fetched now, its page ids below
      bool bad_next = false;
      const int p_next = j + 1 < j0 + n ? key_of(qi, pos, j + 1, bad_next) : -1;
      if (p >= 0 && row < 0) any_bad = true;      // a page id out of range
      const bool ok = row >= 0;
      const uint8_t* src = a.kv + (ok ? row * a.ld_kv : 0);
      const int8_t e = ok ? __ldg(a.exps + (row >> 6)) : kNoKey;
      const uint64_t src_bits = reinterpret_cast<uint64_t>(src);
      const uint32_t ok_mask = __ballot_sync(0xffffffffu, ok);
      // chunk copies: instruction i covers rows 4 i .. 4 i + 3 of this warp's 32
      uint64_t at[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        at[i] = __shfl_sync(0xffffffffu, src_bits, 4 * i + (lane >> 3)) + 16 * (lane & 7);
      int64_t row_next = -1;
#pragma unroll
      for (int u = 0; u < 5; ++u) {
        if (u == 4) {
          if (!mbar_wait_warp(&ring.rope_empty, (n_rope & 1) ^ 1, a.status)) return false;
          const uint32_t dst = smem_u32(slots.rope);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int rr = 8 * i + (lane >> 2);
            const uint64_t s = __shfl_sync(0xffffffffu, src_bits, rr) + 512 + 16 * (lane & 3);
            const int r = 32 * g + rr;
            cp_async16_or_zero(dst + r * 64 + ((((lane & 3) ^ (r >> 1)) & 3) << 4),
                               reinterpret_cast<const void*>(s), (ok_mask >> rr) & 1u);
          }
          cp_async_arrive(&ring.rope_full);
          ++n_rope;
        } else {
          const uint32_t slot = n_chunk % R;
          if (!mbar_wait_warp(&ring.empty[slot], ((n_chunk / R) & 1) ^ 1, a.status)) return false;
          if (u == 0) {
            const uint32_t ms = n_tile % kMeta;
            ring.key_exp[ms][32 * g + lane] = e;
            __syncwarp();
            if (lane == 0) mbar_arrive(&ring.meta_full[ms]);
            ++n_tile;
          }
          const uint32_t dst = smem_u32(slots.chunk[slot]);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int rr = 4 * i + (lane >> 3);
            const int r = 32 * g + rr;
            cp_async16_or_zero(dst + r * 128 + (((lane & 7) ^ (r & 7)) << 4),
                               reinterpret_cast<const void*>(at[i] + 128 * u), (ok_mask >> rr) & 1u);
          }
          cp_async_arrive(&ring.full[slot]);
          ++n_chunk;
        }
        if (u == 1 && p_next >= 0) row_next = kv8_row(a.keys, seq, p_next);
      }
      p = p_next;
      row = row_next;
      any_bad |= bad_next;
    }
    if (any_bad) report(a.status, DSA_ERR_DEVICE_BOUNDS);
    return true;
  }

  // No copy is in flight when the block ends.
  __device__ __forceinline__ void drain() {
    cp_async_commit();
    cp_async_wait_group<0>();
  }
};

}  // namespace dsa
