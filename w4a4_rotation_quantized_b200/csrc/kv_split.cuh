// kv_split.cuh -- how the attention kernels share a batch out: the work of all
// sequences as one line of units, cut into equal ranges, one a block.
//
// Lengths are on the device, so the cut is made there: every block adds up the
// units of the sequences (they are few against the keys) and finds its range.  An item
// (sequence, tile of query rows, block of heads) whose units fall into one range is
// finished by its block; one that ranges cut leaves its parts in the workspace, at
// most two a block, and the join kernel, which makes the same cut, adds them up in order.
#pragma once

#include "kv_device.cuh"

namespace qr {

struct SplitPlan {
  int32_t gq;                 // query heads of a key head
  int32_t rows;               // query rows (token, head of the group) of a tile
  int32_t unit;               // tokens of a unit
  int32_t head_blocks;        // blocks of key heads
  int32_t blocks;             // ranges
  int32_t causal;
};

// The rows of a sequence: the call's row of its first new token, how many of its
// new tokens are in the call's arrays, and how many tokens of it come before its first new one.
struct SeqRows {
  int32_t first, here, before, len;
};

__device__ __forceinline__ SeqRows seq_rows(const KvView& v, int32_t b) {
  SeqRows r;
  const int32_t c0 = v.cu[b], c1 = v.cu[b + 1];
  r.len = kv_len(v, b);
  r.first = c0;
  r.here = c0 < 0 || c1 <= c0 || c0 >= v.tokens ? 0 : min(c1, v.tokens) - c0;
  r.before = r.here > 0 ? r.len - (c1 - c0) : 0;
  return r;
}

// Tokens that new token i sees.
__device__ __forceinline__ int32_t seen(const SeqRows& r, int32_t i, int causal) {
  return causal ? min(max(r.before + i + 1, 0), r.len) : r.len;
}

// (the caller holds here * gq below 2^31)
__device__ __forceinline__ int32_t seq_tiles(const SplitPlan& p, const SeqRows& r) {
  return static_cast<int32_t>((static_cast<uint32_t>(r.here) * p.gq + p.rows - 1) / static_cast<uint32_t>(p.rows));
}

// Tokens that a tile's last row sees, and its units (at least one: rows that see nothing are written too).
__device__ __forceinline__ int32_t tile_seen(const SplitPlan& p, const SeqRows& r, int32_t tile) {
  if (!p.causal) return r.len;
  const uint32_t rows = static_cast<uint32_t>(r.here) * p.gq;
  const uint32_t last = min((static_cast<uint32_t>(tile) + 1) * p.rows, rows) - 1;
  return seen(r, static_cast<int32_t>(last / static_cast<uint32_t>(p.gq)), 1);
}
__device__ __forceinline__ int32_t tile_units(const SplitPlan& p, const SeqRows& r, int32_t tile) {
  return max(static_cast<int32_t>((static_cast<uint32_t>(tile_seen(p, r, tile)) + p.unit - 1) /
                                  static_cast<uint32_t>(p.unit)), 1);
}

// prefix[b] = units of the sequences before b, prefix[batch] = all.  Called by a whole block.  MANY: sequences have
// many tiles, a warp adds up one's; else a thread does.
template <int THREADS, bool MANY>
__device__ __forceinline__ void split_prefix(const KvView& v, const SplitPlan& p, int64_t* prefix) {
  __shared__ int64_t warp_sum[THREADS / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (MANY) {
    for (int32_t b = warp; b < v.batch; b += THREADS / 32) {
      const SeqRows r = seq_rows(v, b);
      const int32_t tiles = seq_tiles(p, r);
      int64_t x = 0;
      for (int32_t t = lane; t < tiles; t += 32) x += tile_units(p, r, t);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
      if (lane == 0) prefix[b + 1] = x * p.head_blocks;
    }
    __syncthreads();
  }
  int64_t base = 0;
  if (threadIdx.x == 0) prefix[0] = 0;
  for (int32_t b0 = 0; b0 < v.batch; b0 += THREADS) {
    const int32_t b = b0 + threadIdx.x;
    int64_t x = 0;
    if (b < v.batch) {
      if (MANY) {
        x = prefix[b + 1];
      } else {
        const SeqRows r = seq_rows(v, b);
        const int32_t tiles = seq_tiles(p, r);
        for (int32_t t = 0; t < tiles; ++t) x += tile_units(p, r, t);
        x *= p.head_blocks;
      }
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    int64_t below = base, all = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
      if (w < warp) below += warp_sum[w];
      all += warp_sum[w];
    }
    if (b < v.batch) prefix[b + 1] = below + x;
    base += all;
    __syncthreads();
  }
}

// The ranges: `blocks` of them at most, of one unit at least; the first
// `longer` have one unit more.
struct Ranges {
  int32_t blocks, each, longer;

  __device__ static __forceinline__ Ranges of(const SplitPlan& p, int64_t units) {
    Ranges r;
    if (units < 0x7FFFFFFF) {                             // (32-bit divisions are several times shorter)
      const uint32_t u = static_cast<uint32_t>(units);
      r.blocks = min(max(static_cast<int32_t>(u), 1), p.blocks);
      r.each = static_cast<int32_t>(u / static_cast<uint32_t>(r.blocks));
      r.longer = static_cast<int32_t>(u - static_cast<uint32_t>(r.blocks) * r.each);
    } else {
      r.blocks = p.blocks;
      r.each = static_cast<int32_t>(units / r.blocks);
      r.longer = static_cast<int32_t>(units % r.blocks);
    }
    return r;
  }
  __device__ __forceinline__ int64_t start(int32_t block) const {
    return static_cast<int64_t>(each) * block + min(block, longer);
  }
  __device__ __forceinline__ int32_t count(int32_t block) const {
    return block >= blocks ? 0 : each + (block < longer ? 1 : 0);
  }
  // the range that holds unit u
  __device__ __forceinline__ int32_t holder(int64_t u) const {
    const int64_t cut = static_cast<int64_t>(each + 1) * longer;
    const int64_t x = u < cut ? u : u - cut;
    const int32_t div = u < cut ? each + 1 : each;
    const int32_t q = x < 0x7FFFFFFF ? static_cast<int32_t>(static_cast<uint32_t>(x) / static_cast<uint32_t>(div))
                                     : static_cast<int32_t>(x / div);
    return u < cut ? q : longer + q;
  }
};

}  // namespace qr
