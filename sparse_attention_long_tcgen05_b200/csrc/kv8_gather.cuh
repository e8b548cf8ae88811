// kv8_gather.cuh -- the copying warps of the kernels that read the 8-bit latent
// cache: rows of a tile's 128 keys into swizzled shared-memory tiles.
#pragma once

#include "kv8_common.cuh"

namespace dsa {

constexpr int kGatherWarps = 4;      // warp g copies keys 32 g .. 32 g + 31 of a tile
constexpr int kChunkB = kTile * 128; // 128 columns of a tile's keys: 16 KB
constexpr int kRopeB = kTile * 64;   // the 64 rope columns: 8 KB
constexpr int8_t kNoKey = kExpMax + 1;   // key_exp of a key that does not count

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
// the rope columns (their slot is free first), then chunks 0 to 3. Every lane's arrival on a unit's barrier is
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
  uint64_t wait_ns;
  uint32_t n_chunk = 0, n_rope = 0, n_tile = 0;

  // What is known of this lane's key in one of the coming tiles: the selection's
  // entry as it stands (or the position), and the query it belongs to.
  struct Entry {
    int raw = -1, seq = 0, pos = -1;
    bool live = false;     // there is such a tile
  };

  // All tiles of the worker's range. An entry, its page id and its block's exponent
  // depend on one another, a memory latency each: the entry is loaded three tiles
  // ahead of its copies, the page id two, the exponent one, each used no sooner
  // than a tile later. (Looked up within one tile they stopped the copies for
  // 1500 cycles in each.) False when a wait ran out.
  __device__ bool run(Kv8Pieces& pieces) {
    bool any_bad = false;
    Kv8Piece pc{};
    int left = 0, j = 0, seq = 0, pos = -1;
    auto fetch = [&](Entry& s) {
      s.live = true;
      if (left == 0) {
        s.live = pieces.next(pc);
        if (!s.live) return;
        if (!kv8_query(a.keys, pc.qi, seq, pos)) any_bad = true;
        left = pc.n;
        j = pc.j0;
      }
      const int r = j * kTile + 32 * g + lane;
      if (a.idx == nullptr)
        s.raw = r <= pos ? r : -1;
      else
        s.raw = r < a.k ? __ldg(a.idx + static_cast<int64_t>(pc.qi) * a.ld_idx + r) : -1;
      s.seq = seq;
      s.pos = pos;
      ++j;
      --left;
    };
    // the key position, and the page id to come; -1: none
    auto look_up = [&](const Entry& s, int& p) -> int {
      p = s.live && s.raw >= 0 ? s.raw : -1;
      if (p >= 0 && p > s.pos) {   // past the query's position
        any_bad = true;
        p = -1;
      }
      if (!a.keys.paged || p < 0) return 0;
      return __ldg(a.keys.block_table + static_cast<int64_t>(s.seq) * a.keys.ld_block_table + (p >> 6));
    };
    auto row_of = [&](int p, int page) -> int64_t {
      if (p < 0) return -1;
      if (!a.keys.paged) return p;
      if (page < 0 || page >= a.keys.num_pages) {
        any_bad = true;
        return -1;
      }
      return static_cast<int64_t>(page) * 64 + (p & 63);
    };
    auto exp_of = [&](int64_t row) -> int {
      if (row < 0) return kNoKey;
      const int e = __ldg(a.exps + (row >> 6));
      if (is_exponent(e)) return e;
      any_bad = true;
      return kNoKey;
    };

    Entry s0, s1, s2, s3;
    fetch(s0);
    fetch(s1);
    fetch(s2);
    int p0, p1, p2 = -1;
    int page0 = look_up(s0, p0), page1 = look_up(s1, p1), page2 = 0;
    int64_t row = row_of(p0, page0), row1 = -1;
    int e = exp_of(row), e1 = kNoKey;
    bool live = s0.live, live1 = s1.live;
    while (live) {
      const bool ok = row >= 0;
      const uint64_t src_bits = reinterpret_cast<uint64_t>(a.kv + (ok ? row * a.ld_kv : 0));
      const uint32_t ok_mask = __ballot_sync(0xffffffffu, ok);
      // chunk copies: instruction i covers rows 4 i .. 4 i + 3 of this warp's 32
      uint64_t at[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        at[i] = __shfl_sync(0xffffffffu, src_bits, 4 * i + (lane >> 3)) + 16 * (lane & 7);
      if (!mbar_wait_warp(&ring.rope_empty, (n_rope & 1) ^ 1, a.status, wait_ns)) return false;
      const uint32_t dst_rope = smem_u32(slots.rope);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int rr = 8 * i + (lane >> 2);
        const uint64_t s = __shfl_sync(0xffffffffu, src_bits, rr) + 512 + 16 * (lane & 3);
        const int r = 32 * g + rr;
        cp_async16_or_zero(dst_rope + r * 64 + ((((lane & 3) ^ (r >> 1)) & 3) << 4),
                           reinterpret_cast<const void*>(s), (ok_mask >> rr) & 1u);
      }
      cp_async_arrive(&ring.rope_full);
      ++n_rope;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const uint32_t slot = n_chunk % R;
        if (!mbar_wait_warp(&ring.empty[slot], ((n_chunk / R) & 1) ^ 1, a.status, wait_ns)) return false;
        if (u == 0) {
          const uint32_t ms = n_tile % kMeta;
          ring.key_exp[ms][32 * g + lane] = static_cast<int8_t>(e);
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
        if (u == 0) fetch(s3);
        if (u == 1) page2 = look_up(s2, p2);
        if (u == 2) row1 = row_of(p1, page1);
        if (u == 3) e1 = exp_of(row1);
      }
      row = row1;
      e = e1;
      live = live1;
      p1 = p2;
      page1 = page2;
      live1 = s2.live;
      s2 = s3;
    }
    if (__any_sync(0xffffffffu, any_bad) && lane == 0) report(a.status, DSA_ERR_DEVICE_BOUNDS);
    return true;
  }

  // No copy is in flight when the block ends.
  __device__ __forceinline__ void drain() {
    cp_async_commit();
    cp_async_wait_group<0>();
  }
};

}  // namespace dsa
