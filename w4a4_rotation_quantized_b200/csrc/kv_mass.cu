// kv_mass.cu -- the attention weight that each token of the paged 4-bit KV cache receives from the rows of a
// call, added to a running sum:
//   mass[b, j, t] += sum over the rows i that see t and the query heads of group j of 2^(x - lse log2 e),
//   x = s_k q . (c - z) scale log2 e.
// S^T = K Q^T on the warp matrix instructions, tokens in the 16 rows, 8 query rows in the columns, as in
// kv_attention.cu; here keys go in as the whole numbers c - z (exact in fp16 for zeros within +-900, the
// remainder meets the sum of the query's elements), because the result is held in fp32 and keeps what they keep.
// A token belongs to one warp, which goes through the rows in order: no atomics, equal calls give equal bits.
//
// Few rows a key head (single tokens): bound by the bytes of the keys, d/2 + 8 d/g a token and head.  A warp takes
// one group and 32 tokens at a time, the next ones under way in a ring in shared memory; warps of a block take
// neighbouring groups of the same tokens.  A warp has as many pieces as make some four blocks an SM (four pieces: 35.6 us
// for 32 sequences of up to 4096 tokens, 64/8 heads; 34.6 so, the start of a block being some microseconds).
// Many rows: a warp keeps 32 tokens' keys as operands in registers (16 where a head is 256 wide) and the block's
// eight warps go through the query rows together, 64 at a time through shared memory.  Under a causal mask the first
// tokens meet the most rows, so four blocks, a cluster, share the rows of 256 tokens and the first adds their sums up
// in order (a prompt of 2048 tokens, 32 heads: 247 us with one block of 8 warps an SM and all rows, 113 so).
#include <algorithm>
#include <cmath>

#include "kv_mma.cuh"
#include "kv_split.cuh"
#include "qr_internal.h"

namespace qr {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kLeastSteps = 4;                 // of 32 tokens, of a warp, at least (few rows)
constexpr int kRowsStaged = 64;                // query rows in shared memory (many rows)
constexpr int kShare = 4;                      // blocks that share the rows (many rows)

struct MassArgs {
  KvView v;
  const __half* q;
  int64_t ldq;
  int32_t q_heads, gq, per;                    // query heads of a key head; key heads of a group
  float scale_log2;
  int32_t causal;
  const float* lse;
  float* mass;
  int64_t ld_mass;
  int32_t groups_log2, steps;                  // groups of a block, pieces of a warp (few rows)
};

// Keys as the A operand: for word w the products with the low and the high nibbles, rows g and g + 8.
template <int D>
struct KeyFrag {
  uint32_t lo[D / 32][4], hi[D / 32][4];

  // tokens t0 + g and t0 + g + 8 of a stage; z1024: their fp16 pairs -(1032 + z)
  __device__ __forceinline__ void load(const uint8_t* keys, int t0, int g, int c, uint32_t za, uint32_t zb) {
    uint32_t xa[D / 32], xb[D / 32];
    load_key_words<D>(keys, t0 + g, c, xa);
    load_key_words<D>(keys, t0 + g + 8, c, xb);
    const uint32_t ya = add_half2(za, 0x63806380u), yb = add_half2(zb, 0x63806380u);      // -(72 + z)
#pragma unroll
    for (int w = 0; w < D / 32; ++w) {
      const uint32_t pa = xa[w] >> 8, pb = xb[w] >> 8;
      lo[w][0] = add_half2(nib_1024(xa[w]), za);
      lo[w][1] = add_half2(nib_1024(xb[w]), zb);
      lo[w][2] = add_half2(nib_1024(pa), za);
      lo[w][3] = add_half2(nib_1024(pb), zb);
      hi[w][0] = add_half2(nib_64(xa[w]), ya);
      hi[w][1] = add_half2(nib_64(xb[w]), yb);
      hi[w][2] = add_half2(nib_64(pa), ya);
      hi[w][3] = add_half2(nib_64(pb), yb);
    }
  }
  // sums with 8 query rows: columns 2c, 2c + 1 of rows g (s[0], s[1]) and g + 8
  __device__ __forceinline__ void scores(const uint4 (&b)[D / 32], float (&s)[4]) const {
    float t[4];
    mma_16x8x16_first(s, lo[0][0], lo[0][1], lo[0][2], lo[0][3], b[0].x, b[0].y);
    mma_16x8x16_first(t, hi[0][0], hi[0][1], hi[0][2], hi[0][3], b[0].z, b[0].w);
#pragma unroll
    for (int w = 1; w < D / 32; ++w) {
      mma_16x8x16(s, lo[w][0], lo[w][1], lo[w][2], lo[w][3], b[w].x, b[w].y);
      mma_16x8x16(t, hi[w][0], hi[w][1], hi[w][2], hi[w][3], b[w].z, b[w].w);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e] += t[e];
  }
};

// What a query row asks for: its lse log2 e (+inf: nothing), the tokens it sees, the sum of its elements.
struct RowNumbers {
  float lse2, qsum;
  int32_t limit;
};

__device__ __forceinline__ float lse_log2(float lse) { return lse == -INFINITY ? INFINITY : lse * 1.4426950408889634f; }

// A token's numbers from its group's scale and zero: scale, remainder of the zero, fp16 pair.
struct KeyNumbers {
  float sk, rest;
  uint32_t z1024;
};
__device__ __forceinline__ KeyNumbers key_numbers(float s, int32_t z, float scale_log2) {
  const int32_t zc = min(max(z, -900), 900);
  const __half2 h = __half2half2(__int2half_rn(-1032 - zc));
  return KeyNumbers{s * scale_log2, static_cast<float>(static_cast<int64_t>(z) - zc),
                    *reinterpret_cast<const uint32_t*>(&h)};
}

// Adds the weights of one tile: scores s of tokens ta (rows g) and ta + 8 with query columns 2c, 2c + 1.
template <bool PLAIN>
__device__ __forceinline__ void add_weights(const float (&s)[4], const float (&sk)[2], const float (&rest)[2],
                                            const bool (&is)[2], int32_t ta, const float (&lse2)[2],
                                            const float (&qsum)[2], const int32_t (&limit)[2], float (&sum)[2]) {
#pragma unroll
  for (int e = 0; e < 2; ++e)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (PLAIN) {
        sum[e] += exp2_fast(fmaf(s[2 * e + k], sk[e], -lse2[k]));
      } else {
        const float x = rest[e] != 0.0f ? fmaf(-rest[e], qsum[k], s[2 * e + k]) : s[2 * e + k];
        const float p = exp2_fast(fmaf(x, sk[e], -lse2[k]));
        // a row that sees nothing has lse2 = +inf, whatever the score is
        sum[e] += is[e] && ta + 8 * e < limit[k] && lse2[k] != INFINITY ? p : 0.0f;
      }
    }
}

template <int D>
constexpr int few_bytes() {                    // of a warp: two stages, the queries of 8 rows
  return 2 * KvStage<D>::kBytes + QueryFrag<D>::kBytes;
}

// Few rows.  grid: (blocks of tokens, blocks of groups, sequences)
template <int D>
__global__ void __launch_bounds__(kThreads) kv_mass_few_kernel(const MassArgs a) {
  using S = KvStage<D>;
  extern __shared__ __align__(128) uint8_t smem[];
  const KvView& v = a.v;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  const int gw = warp & ((1 << a.groups_log2) - 1), sw = warp >> a.groups_log2, ws = kWarps >> a.groups_log2;
  uint8_t* ring = smem + warp * few_bytes<D>();
  uint4* qf = reinterpret_cast<uint4*>(ring + 2 * S::kBytes);
  grid_dep_wait();
  grid_dep_launch();
  const int32_t b = blockIdx.z, j = (blockIdx.y << a.groups_log2) + gw;
  const SeqRows rows = seq_rows(v, b);
  const int32_t first = (blockIdx.x * ws + sw) * (32 * a.steps);
  const int32_t all_rows = rows.here * a.gq;
  const int32_t n_seen = all_rows > 0 ? seen(rows, rows.here - 1, a.causal) : 0;
  if (first >= n_seen) return;                           // (warps do not wait for each other)
  const int pieces = min((n_seen - first + 31) / 32, a.steps) * a.per;      // (tokens, head of the group)

  auto slot_of = [&](int i) -> int32_t {
    const int32_t t = first + i / a.per * 32 + lane;
    return i < pieces && t < n_seen ? static_cast<int32_t>(kv_slot(v, v.table, b, t)) : -1;
  };
  // starts the copy of piece i; returns which of its tokens are there
  auto fill = [&](int i, int32_t slot) -> uint32_t {
    const uint32_t there = __ballot_sync(0xffffffffu, slot >= 0);
    if (i < pieces) {
      const uint8_t* key = v.codes[0] + (j * a.per + i % a.per) * S::kRow + lane % S::kChunks * 16;
      S::template issue<true, false>(v, key, nullptr, j, max(slot, 0), smem_u32(ring + (i & 1) * S::kBytes), lane);
    }
    cp_async_commit();
    return there;
  };
  int32_t next = slot_of(1);
  uint32_t ahead = fill(0, slot_of(0));
  const int row_tiles = (all_rows + 7) / 8;
  float sum[2][2];
  int32_t put_tile = -1, put_head = -1;                  // what qf holds
  RowNumbers num{};                                      // of row lane & 7 of that tile
  for (int i = 0; i < pieces; ++i) {
    const uint32_t there = ahead;
    ahead = fill(i + 1, next);
    next = slot_of(i + 2);
    cp_async_wait<1>();
    __syncwarp();
    const uint8_t* st = ring + (i & 1) * S::kBytes;
    const int head = j * a.per + i % a.per;
    const int32_t t0 = first + i / a.per * 32;
    if (i % a.per == 0) sum[0][0] = sum[0][1] = sum[1][0] = sum[1][1] = 0.0f;
    const float* meta = reinterpret_cast<const float*>(st + S::kMeta);
    const KeyNumbers kn = key_numbers(meta[lane], __float_as_int(meta[32 + lane]), a.scale_log2);
    const bool odd = __any_sync(0xffffffffu, kn.rest != 0.0f) || there != 0xffffffffu;
    KeyFrag<D> f[2];
    float sk[2][2], rest[2][2];
    bool is[2][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t z[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int t = 16 * h + 8 * e + g;
        sk[h][e] = __shfl_sync(0xffffffffu, kn.sk, t);
        rest[h][e] = __shfl_sync(0xffffffffu, kn.rest, t);
        z[e] = __shfl_sync(0xffffffffu, kn.z1024, t);
        is[h][e] = (there >> t) & 1u;
      }
      f[h].load(st, 16 * h, g, c, z[0], z[1]);
    }
    for (int32_t tile = 0; tile < row_tiles; ++tile) {
      if (put_tile != tile || put_head != head) {
        put_tile = tile;
        put_head = head;
        __syncwarp();
        const int32_t r = tile * 8 + g;
        const __half* from = r < all_rows ? a.q + (rows.first + r / a.gq) * a.ldq +
                                                static_cast<int64_t>(head * a.gq + r % a.gq) * D : nullptr;
        float s = QueryFrag<D>::put(qf, from, lane);
        s += __shfl_xor_sync(0xffffffffu, s, 1);
        s += __shfl_xor_sync(0xffffffffu, s, 2);
        const int32_t rr = tile * 8 + (lane & 7);
        num = RowNumbers{INFINITY, __shfl_sync(0xffffffffu, s, (lane & 7) * 4), 0};
        if (rr < all_rows) {
          num.lse2 = lse_log2(a.lse[static_cast<int64_t>(rows.first + rr / a.gq) * a.q_heads + head * a.gq + rr % a.gq]);
          num.limit = seen(rows, rr / a.gq, a.causal);
        }
        __syncwarp();
      }
      float lse2[2], qsum[2];
      int32_t limit[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        lse2[k] = __shfl_sync(0xffffffffu, num.lse2, 2 * c + k);
        qsum[k] = __shfl_sync(0xffffffffu, num.qsum, 2 * c + k);
        limit[k] = __shfl_sync(0xffffffffu, num.limit, 2 * c + k);
      }
      // (rows of nobody see nothing: not plain)
      const bool plain = !odd && !__any_sync(0xffffffffu, min(limit[0], limit[1]) < t0 + 32 || lse2[0] == INFINITY || lse2[1] == INFINITY);
      uint4 bq[D / 32];
#pragma unroll
      for (int w = 0; w < D / 32; ++w) bq[w] = qf[w * 32 + lane];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float s[4];
        f[h].scores(bq, s);
        if (plain) add_weights<true>(s, sk[h], rest[h], is[h], t0 + 16 * h + g, lse2, qsum, limit, sum[h]);
        else add_weights<false>(s, sk[h], rest[h], is[h], t0 + 16 * h + g, lse2, qsum, limit, sum[h]);
      }
    }
    if ((i + 1) % a.per == 0) {
      // a token's columns lie in the four lanes of its row; then lane t takes token t
      float own = 0.0f;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = sum[h][e];
          x += __shfl_xor_sync(0xffffffffu, x, 1);
          x += __shfl_xor_sync(0xffffffffu, x, 2);
          x = __shfl_sync(0xffffffffu, x, (lane & 7) * 4);
          if ((lane >> 3) == 2 * h + e) own = x;
        }
      if ((there >> lane) & 1u) a.mass[(static_cast<int64_t>(b) * v.groups + j) * a.ld_mass + t0 + lane] += own;
    }
    __syncwarp();
  }
  cp_async_wait<0>();
}

template <int D>
struct Many {
  static constexpr int kTiles = D == 256 ? 1 : 2;              // of 16 tokens, of a warp
  static constexpr int kTokens = 16 * kTiles;
  static constexpr int kFrag = kRowsStaged / 8 * (D / 32) * 32;        // 16-byte entries of the staged queries
  static constexpr int kBytes = 2 * kFrag * 16 + 2 * kRowsStaged * 16 + kWarps * kTokens * 4;
};

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float x;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(addr) : "memory");
  return x;
}

// Many rows.  grid: (kShare times blocks of 8 kTokens tokens, groups, sequences), clusters of kShare
template <int D>
__global__ void __launch_bounds__(kThreads, D == 256 ? 1 : 2) kv_mass_many_kernel(const MassArgs a) {
  using M = Many<D>;
  extern __shared__ __align__(128) uint8_t smem[];
  const KvView& v = a.v;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  uint4* qf = reinterpret_cast<uint4*>(smem);                          // [2][rows / 8][word][lane]
  float4* qn = reinterpret_cast<float4*>(smem + 2 * M::kFrag * 16);    // [2][rows]: lse2, sum, limit
  grid_dep_wait();
  grid_dep_launch();
  const int32_t b = blockIdx.z, j = blockIdx.y;
  const SeqRows rows = seq_rows(v, b);
  const int32_t all_rows = rows.here * a.gq;
  const int32_t n_seen = all_rows > 0 ? seen(rows, rows.here - 1, a.causal) : 0;
  const int32_t block0 = blockIdx.x / kShare * (kWarps * M::kTokens);
  const int share = blockIdx.x % kShare;
  if (block0 >= n_seen) return;                          // (the whole cluster)
  const int32_t t0 = block0 + warp * M::kTokens;
  // this block's share of the rows, from the first new token that sees the block's first token on
  const int32_t first_row = a.causal ? max(block0 - rows.before, 0) * a.gq : 0;
  const int row0 = (first_row / kRowsStaged + share) * kRowsStaged;
  constexpr int kStride = kShare * kRowsStaged;

  int32_t slot[M::kTiles][2];                            // of tokens g and g + 8 of each tile
#pragma unroll
  for (int h = 0; h < M::kTiles; ++h)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int32_t t = t0 + 16 * h + 8 * e + g;
      slot[h][e] = t < n_seen ? static_cast<int32_t>(kv_slot(v, v.table, b, t)) : -1;
    }
  float sum[M::kTiles][2] = {};
  for (int hi = 0; hi < a.per; ++hi) {
    const int head = j * a.per + hi;
    KeyFrag<D> f[M::kTiles];
    float sk[M::kTiles][2], rest[M::kTiles][2];
    bool is[M::kTiles][2], odd = false;
#pragma unroll
    for (int h = 0; h < M::kTiles; ++h) {
      uint32_t z[2];
      uint32_t x[2][D / 32];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        is[h][e] = slot[h][e] >= 0;
        const int64_t s = max(slot[h][e], 0);
        const int64_t at = s * v.groups + j;
        const KeyNumbers kn = key_numbers(v.scales[0][at], v.zeros[0][at], a.scale_log2);
        sk[h][e] = kn.sk;
        rest[h][e] = kn.rest;
        z[e] = kn.z1024;
        odd |= !is[h][e] || kn.rest != 0.0f;
        // the words of column c: 16 bytes (or 8, 4) of the row, and for D = 256 16 more from its second half
        const uint8_t* from = v.codes[0] + s * (v.width / 2) + head * (D / 2);
#pragma unroll
        for (int w = 0; w < D / 32; ++w)
          x[e][w] = *reinterpret_cast<const uint32_t*>(from + QueryFrag<D>::first(c, w) / 2);
      }
      const uint32_t ya = add_half2(z[0], 0x63806380u), yb = add_half2(z[1], 0x63806380u);
#pragma unroll
      for (int w = 0; w < D / 32; ++w) {
        const uint32_t xa = x[0][w], xb = x[1][w], pa = xa >> 8, pb = xb >> 8;
        f[h].lo[w][0] = add_half2(nib_1024(xa), z[0]);
        f[h].lo[w][1] = add_half2(nib_1024(xb), z[1]);
        f[h].lo[w][2] = add_half2(nib_1024(pa), z[0]);
        f[h].lo[w][3] = add_half2(nib_1024(pb), z[1]);
        f[h].hi[w][0] = add_half2(nib_64(xa), ya);
        f[h].hi[w][1] = add_half2(nib_64(xb), yb);
        f[h].hi[w][2] = add_half2(nib_64(pa), ya);
        f[h].hi[w][3] = add_half2(nib_64(pb), yb);
      }
    }
    odd = __any_sync(0xffffffffu, odd);

    // rows of a stage: thread (tile of 8 rows, lane of the fragment) puts its share
    auto stage = [&](int32_t r0, int buf) {
      for (int e = warp; e < kRowsStaged / 8; e += kWarps) {
        const int32_t r = r0 + 8 * e + g;
        const __half* from = r < all_rows ? a.q + (rows.first + r / a.gq) * a.ldq +
                                                static_cast<int64_t>(head * a.gq + r % a.gq) * D : nullptr;
        float s = QueryFrag<D>::put(qf + buf * M::kFrag + e * (D / 32) * 32, from, lane);
        s += __shfl_xor_sync(0xffffffffu, s, 1);
        s += __shfl_xor_sync(0xffffffffu, s, 2);
        if (c == 0) {
          float lse2 = INFINITY;
          int32_t limit = 0;
          if (r < all_rows) {
            lse2 = lse_log2(a.lse[static_cast<int64_t>(rows.first + r / a.gq) * a.q_heads + head * a.gq + r % a.gq]);
            limit = seen(rows, r / a.gq, a.causal);
          }
          qn[buf * kRowsStaged + 8 * e + g] = make_float4(lse2, s, __int_as_float(limit), 0.0f);
        }
      }
    };
    __syncthreads();
    stage(row0, 0);
    int buf = 0;
    for (int32_t r0 = row0; r0 < all_rows; r0 += kStride, buf ^= 1) {
      __syncthreads();
      if (r0 + kStride < all_rows) stage(r0 + kStride, buf ^ 1);
#pragma unroll 1
      for (int e = 0; e < kRowsStaged / 8; ++e) {
        if (r0 + 8 * e >= all_rows) break;
        const float4 n0 = qn[buf * kRowsStaged + 8 * e + 2 * c], n1 = qn[buf * kRowsStaged + 8 * e + 2 * c + 1];
        const float lse2[2] = {n0.x, n1.x}, qsum[2] = {n0.y, n1.y};
        const int32_t limit[2] = {__float_as_int(n0.z), __float_as_int(n1.z)};
        const int32_t most = max(limit[0], limit[1]), least = min(limit[0], limit[1]);
        if (!__any_sync(0xffffffffu, most > t0)) continue;               // no row sees this warp's tokens
        const bool plain = !odd && !__any_sync(0xffffffffu, least < t0 + M::kTokens || lse2[0] == INFINITY || lse2[1] == INFINITY);
        uint4 bq[D / 32];
#pragma unroll
        for (int w = 0; w < D / 32; ++w) bq[w] = qf[buf * M::kFrag + (e * (D / 32) + w) * 32 + lane];
#pragma unroll
        for (int h = 0; h < M::kTiles; ++h) {
          float s[4];
          f[h].scores(bq, s);
          if (plain) add_weights<true>(s, sk[h], rest[h], is[h], t0 + 16 * h + g, lse2, qsum, limit, sum[h]);
          else add_weights<false>(s, sk[h], rest[h], is[h], t0 + 16 * h + g, lse2, qsum, limit, sum[h]);
        }
      }
    }
  }
  // the cluster's sums, added up by its first block
  float* own = reinterpret_cast<float*>(smem + 2 * M::kFrag * 16 + 2 * kRowsStaged * 16) + warp * M::kTokens;
#pragma unroll
  for (int h = 0; h < M::kTiles; ++h)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float x = sum[h][e];
      x += __shfl_xor_sync(0xffffffffu, x, 1);
      x += __shfl_xor_sync(0xffffffffu, x, 2);
      if (c == 0) own[16 * h + 8 * e + g] = x;
    }
  cluster_sync();
  if (share == 0 && lane < M::kTokens) {
    const int32_t t = t0 + lane;
    float x = own[lane];
    for (int k = 1; k < kShare; ++k) x += ld_cluster_f32(mapa_shared(smem_u32(own + lane), k));
    if (t < n_seen && kv_slot(v, v.table, b, t) >= 0)
      a.mass[(static_cast<int64_t>(b) * v.groups + j) * a.ld_mass + t] += x;
  }
  cluster_sync();
}

// Rows of a sequence and key head (on average) up to which keys are streamed.  Streamed against held, us: 32
// sequences of up to 4096 tokens, 64/8 heads: 26 rows 85 and 263, 49 rows 141 and 305; 32/32 heads, 31 rows: 458 and
// 1294; one sequence of 8192, 64/8 heads: 24 rows 20 and 26, 48 rows 35 and 30, 64 rows 44 and 33.
// A batch that mixes both kinds goes one way as a whole: 512 rows on 4096 tokens beside 255 single tokens, 64/8 heads, 33 ms
// where apart they take 166 and 137 us (24 rows on average: the prompt's 4096 rows of a key head are streamed, 8 at a time).
constexpr int kFewRows = 64;

template <int D>
cudaError_t run_mass(MassArgs& a, cudaStream_t stream) {
  const KvView& v = a.v;
  const int64_t rows = (static_cast<int64_t>(v.tokens) * a.gq + v.batch - 1) / v.batch;
  if (rows > kFewRows) {
    const int block = kWarps * Many<D>::kTokens;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(kv_mass_many_kernel<D>, Many<D>::kBytes, done);
    if (e != cudaSuccess) return e;
    return launch_pdl(kv_mass_many_kernel<D>, dim3(kShare * ((v.capacity + block - 1) / block), v.groups, v.batch),
                      dim3(kThreads), Many<D>::kBytes, stream, kShare, a);
  }
  while (a.groups_log2 < 3 && v.groups % (2 << a.groups_log2) == 0) ++a.groups_log2;
  const int step = 32 * (kWarps >> a.groups_log2);
  const int64_t steps = (static_cast<int64_t>(v.capacity) + step - 1) / step * (v.groups >> a.groups_log2) * v.batch;
  a.steps = static_cast<int32_t>(std::min<int64_t>(std::max<int64_t>(steps / (4 * sm_count()), kLeastSteps), 1024));
  const int block = step * a.steps;
  const int smem = kWarps * few_bytes<D>();
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(kv_mass_few_kernel<D>, smem, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(kv_mass_few_kernel<D>, dim3((v.capacity + block - 1) / block, v.groups >> a.groups_log2, v.batch),
                    dim3(kThreads), smem, stream, 1, a);
}

}  // namespace

qr_status launch_kv_mass(const KvView& v, const KvMassJob& j, cudaStream_t stream) {
  MassArgs a{};
  a.v = v;
  a.q = reinterpret_cast<const __half*>(j.q);
  a.ldq = j.ldq;
  a.q_heads = j.q_heads;
  a.gq = j.q_heads / v.heads;
  a.per = v.group / v.head_dim;
  a.scale_log2 = static_cast<float>(static_cast<double>(j.scale) * 1.4426950408889634);
  a.causal = j.causal;
  a.lse = j.lse;
  a.mass = j.mass;
  a.ld_mass = j.ld_mass;
  cudaError_t e;
  switch (v.head_dim) {
    case 32: e = run_mass<32>(a, stream); break;
    case 64: e = run_mass<64>(a, stream); break;
    case 128: e = run_mass<128>(a, stream); break;
    default: e = run_mass<256>(a, stream); break;
  }
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? QR_OK : QR_ERR_CUDA;
}

}  // namespace qr
