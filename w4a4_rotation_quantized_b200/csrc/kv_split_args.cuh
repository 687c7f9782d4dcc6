// kv_split_args.cuh -- what the attention kernels that share a batch out (kv_split.cuh) and the kernel that joins
// their parts agree on.
#pragma once

#include "kv_split.cuh"

namespace qr {

struct SplitArgs {
  KvView v;
  SplitPlan plan;
  const __half* q;
  int64_t ldq;
  int32_t q_heads;
  float scale_log2;                            // scale * log2 e
  __half* out;
  int64_t ldo;
  float* lse;
  int64_t* prefix;                             // [batch + 1]; null: no item is cut
  float2* part_ml;                             // [2 blocks][heads of a block][rows]
  float* part_o;                               // ... [D]
  int32_t heads_log2;                          // heads of a block = 2^heads_log2
};

// A part's place: slot 0 holds the part that begins a block's range, slot 1 one that ends it.
__device__ __forceinline__ int64_t part_at(const SplitArgs& a, int32_t block, int slot, int head, int row) {
  return (((static_cast<int64_t>(block) * 2 + slot) << a.heads_log2) + head) * a.plan.rows + row;
}

// Writes N fp16 values of a finished row.
template <int N>
__device__ __forceinline__ void store_half(__half* to, const float (&x)[N]) {
  __half2 h[N / 2];
#pragma unroll
  for (int i = 0; i < N / 2; ++i) h[i] = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
  if constexpr (N >= 8) {
#pragma unroll
    for (int i = 0; i < N / 8; ++i) reinterpret_cast<uint4*>(to)[i] = reinterpret_cast<const uint4*>(h)[i];
  } else {
    *reinterpret_cast<uint2*>(to) = *reinterpret_cast<const uint2*>(h);
  }
}

__device__ __forceinline__ float row_lse(float m, float l) {
  return l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}
__device__ __forceinline__ float inverse_or_zero(float l) { return l == 0.0f ? 0.0f : 1.0f / l; }

// The item that unit `at` belongs to, and how many of its units a block with `left` units ahead takes.  *b:
// a sequence at or before the item's, which it becomes (the item's already unless SEARCH).  Called by whole warps.
struct Item {
  SeqRows rows;
  int32_t tile, block, unit, units;            // tile of rows, block of heads, first unit, units of the whole item
  int32_t take, seen;                          // units to take; tokens that the tile's last row sees
  bool whole;                                  // the item is taken whole
};
template <bool SEARCH = true>
__device__ __forceinline__ Item find_item(const KvView& v, const SplitPlan& p, const int64_t* prefix, int64_t at,
                                          int32_t left, int32_t* b) {
  int32_t lo = *b, hi = SEARCH ? v.batch - 1 : lo;   // the last b with prefix[b] <= at
  while (lo < hi) {
    const int32_t mid = (lo + hi + 1) >> 1;
    if (prefix[mid] <= at) lo = mid; else hi = mid - 1;
  }
  *b = lo;
  Item it;
  it.rows = seq_rows(v, lo);
  // the tile: 32 of them at a time, one a lane
  int64_t off = at - prefix[lo];
  int32_t tile = 0, tu = tile_units(p, it.rows, 0);
  if (off >= static_cast<int64_t>(tu) * p.head_blocks) {
    const int lane = static_cast<int>(threadIdx.x & 31);
    const int32_t tiles = seq_tiles(p, it.rows);
    for (int32_t t0 = 0;; t0 += 32) {
      const int64_t mine = t0 + lane < tiles ? static_cast<int64_t>(tile_units(p, it.rows, t0 + lane)) * p.head_blocks : 0;
      int64_t upto = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      const uint32_t there = __ballot_sync(0xffffffffu, off < upto);
      if (there != 0 || t0 + 32 >= tiles) {
        const int at_lane = there != 0 ? __ffs(there) - 1 : 0;
        tile = t0 + at_lane;
        off -= __shfl_sync(0xffffffffu, upto - mine, at_lane);
        break;
      }
      off -= __shfl_sync(0xffffffffu, upto, 31);
    }
    tu = tile_units(p, it.rows, tile);
  }
  it.tile = tile;
  it.block = p.head_blocks == 1 ? 0 : static_cast<int32_t>(static_cast<uint32_t>(off) / static_cast<uint32_t>(tu));
  it.unit = static_cast<int32_t>(off - static_cast<int64_t>(it.block) * tu);
  it.units = tu;
  it.take = min(tu - it.unit, left);
  it.whole = it.take == tu;
  it.seen = tile_seen(p, it.rows, it.tile);
  return it;
}

// Attention for many rows a key head (kv_prefill.cu): whether it takes the batch, its rows a tile, its launch.
bool kv_prefill_takes(const KvView& v);
int kv_prefill_rows(int head_dim);
cudaError_t launch_kv_prefill(const SplitArgs& a, cudaStream_t stream);

}  // namespace qr
