// kv_attention.cu -- attention over the paged 4-bit KV cache for few query rows
// a key head (single tokens, drafts): every code is read once from memory, so the bytes of the
// cache bound it, H_k (d + 16 d / g) a token.
//
// S^T = K Q^T and O^T += V^T W^T on the warp matrix instructions, tokens and output elements in the 16
// rows, 8 (or 16) query rows in the columns: with the queries as rows most of the products would be padding.
// Codes become fp16 operands in registers (kv_mma.cuh); the scales meet the scores and the weights:
//   x_t = s_k (sum q u - z' sum q) scale log2 e,   z' = z + 8, u = c + 8
//   o   = sum w_t (c - z),   w_t = s_v 2^(x_t - m),   l = sum 2^(x_t - m).
// The running maximum m is that of x_t + log2 s_v (with log2 s_v held to [-40, 40]): then the weights that are
// rounded for the matrix instructions are near 2^7 where they matter, whatever the values' scales are, and one factor
// rescales l and o alike.  2^7, so that a hundred thousand tokens that are light next to one heavy one, each too small
// for fp16 next to 1 (2^-25), still add up: at 1 they vanished, 3e-3 of the output where they were 2^-25.4 each.
// A weight goes in as two fp16, its rounding and the
// rest: the matrix instructions have room for that (1.5 a token and head).  The maximum is let lag: as long as no
// weight passes 2^15 nothing is rescaled, and the warp need not even find its maximum.  Zeros of values beyond +-900,
// which c - z would not survive in fp16, leave a remainder that is summed apart.
//
// A warp takes one key head and 32 tokens at a time, its own ring of such pieces in shared
// memory, filled by asynchronous copies ahead of their use; warps of a block take neighbouring heads
// of the same tokens (scales of 8 heads share a sector) and do not wait for each other.  With
// fewer heads than warps, warps share a head's tokens and join at the end of an item.
// Work is shared out by kv_split.cuh.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "kv_mma.cuh"
#include "kv_split_args.cuh"
#include "qr_internal.h"

namespace qr {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kStages = 2;                     // pieces of a warp's ring
constexpr int kStep = 32;                      // tokens of a piece
constexpr float kTop = 7.0f, kMost = 15.0f;    // log2 of the largest weight where m is set, and before it is raised

template <int D, int NC>
constexpr int ring_bytes() { return kWarps * (kStages * KvStage<D>::kBytes + KvStage<D>::kPrepared + NC * QueryFrag<D>::kBytes); }
template <int D, int NC>
constexpr int join_bytes() { return kWarps * 8 * NC * (D + 2) * 4; }
template <int D, int NC>
constexpr int tile_bytes() { return ring_bytes<D, NC>() > join_bytes<D, NC>() ? ring_bytes<D, NC>() : join_bytes<D, NC>(); }

template <int D, int NC>
__global__ void __launch_bounds__(kThreads, D == 256 || NC == 2 ? 1 : 2) kv_split_kernel(const SplitArgs a) {
  using S = KvStage<D>;
  using T = ValueTile<D>;
  constexpr int R = 8 * NC;
  extern __shared__ __align__(128) uint8_t smem[];
  const KvView& v = a.v;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  const int hb = 1 << a.heads_log2, hw = warp & (hb - 1), sw = warp >> a.heads_log2;
  const int ws = kWarps >> a.heads_log2;               // warps of a head
  uint8_t* ring = smem + warp * (kStages * S::kBytes + S::kPrepared + NC * QueryFrag<D>::kBytes);
  uint4* q = reinterpret_cast<uint4*>(ring + kStages * S::kBytes);                 // [NC][word][32]
  float* prep_rest = reinterpret_cast<float*>(q + NC * QueryFrag<D>::kBytes / 16); // [32]
  __half* prep_z = reinterpret_cast<__half*>(prep_rest + 32);                      // [32]
  uint32_t* piece_there = reinterpret_cast<uint32_t*>(prep_z + 32);                // [4]
  int32_t* row_limit = reinterpret_cast<int32_t*>(piece_there + 4);                // [16]
  const uint32_t ring_u32 = smem_u32(ring);
  int64_t* prefix = reinterpret_cast<int64_t*>(smem + tile_bytes<D, NC>());

  grid_dep_wait();
  grid_dep_launch();
  split_prefix<kThreads, false>(v, a.plan, prefix);
  const int64_t units = prefix[v.batch];
  if (blockIdx.x == 0 && a.prefix != nullptr)
    for (int32_t b = threadIdx.x; b <= v.batch; b += kThreads) a.prefix[b] = prefix[b];
  const Ranges ranges = Ranges::of(a.plan, units);
  const int64_t start = ranges.start(blockIdx.x);
  const int32_t count = ranges.count(blockIdx.x);
  int32_t b = 0;
  for (int32_t done = 0; done < count;) {
    const int64_t at = start + done;
    const Item it = find_item(v, a.plan, prefix, at, count - done, &b);
    const SeqRows& rows = it.rows;
    const int32_t tile = it.tile, block = it.block, u0 = it.unit, take = it.take, n_seen = it.seen;
    const bool whole = it.whole;
    const int head = (block << a.heads_log2) + hw;

    // queries of this tile: row r is new token r / gq, head r % gq of the group
    const int32_t row0 = tile * R, all_rows = rows.here * a.plan.gq;
    float qsum[NC][2];
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      const int32_t r = row0 + 8 * n + g;
      const __half* from = nullptr;
      if (r < all_rows)
        from = a.q + (rows.first + r / a.plan.gq) * a.ldq +
               static_cast<int64_t>(head * a.plan.gq + r % a.plan.gq) * D;
      float s = QueryFrag<D>::put(q + n * (D / 32) * 32, from, lane);
      s += __shfl_xor_sync(0xffffffffu, s, 1);
      s += __shfl_xor_sync(0xffffffffu, s, 2);
      qsum[n][0] = __shfl_sync(0xffffffffu, s, 8 * c);
      qsum[n][1] = __shfl_sync(0xffffffffu, s, 8 * c + 4);
    }
    if (lane < R) row_limit[lane] = row0 + lane < all_rows ? seen(rows, (row0 + lane) / a.plan.gq, a.plan.causal) : 0;
    const int32_t all_limit = seen(rows, row0 / a.plan.gq, a.plan.causal);      // seen by every row

    uint64_t o[T::kTiles][NC][2], l2[NC];                // pairs of columns 2c, 2c + 1
    float nm[NC][2];                                     // -m
#pragma unroll
    for (int i = 0; i < T::kTiles; ++i)
#pragma unroll
      for (int n = 0; n < NC; ++n) o[i][n][0] = o[i][n][1] = 0;
    float zs[NC][2];
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      l2[n] = 0;
      nm[n][0] = nm[n][1] = zs[n][0] = zs[n][1] = 0.0f;
    }
    uint32_t started = 0;                                // bit 2 n + k: the column has seen a key

    // this warp's pieces: 32 tokens from first + 32 ws i
    const int32_t first = u0 * a.plan.unit + sw * kStep;
    const int32_t pieces = min(take * (a.plan.unit / (ws * kStep)),
                               (max(n_seen - u0 * a.plan.unit, 0) + ws * kStep - 1) / (ws * kStep));
    const uint8_t* key = v.codes[0] + head * S::kRow + lane % S::kChunks * 16;
    const uint8_t* value = v.codes[1] + head * S::kRow + lane % S::kChunks * 16;
    const uint32_t group = head * D / v.group;
    const int32_t page0 = b * v.max_pages;               // (batch * max_pages may not pass 2^31)
    const int32_t* pages = v.table != nullptr ? v.table + page0 : nullptr;
    auto slot_of = [&](int32_t i) -> int32_t {
      const int32_t t = first + i * ws * kStep + lane, tc = max(min(t, n_seen - 1), 0);
      const int32_t p = kv_page(v, tc);
      const int32_t page = pages != nullptr ? pages[p] : page0 + p;
      return t < n_seen && static_cast<uint32_t>(page) < static_cast<uint32_t>(v.pages)
                 ? page * v.page_size + (tc - p * v.page_size) : -1;
    };
    // starts piece i into a stage, whose last word says which of its tokens are there
    auto fill = [&](int32_t i, int32_t slot, int stage) {
      const uint32_t there = __ballot_sync(0xffffffffu, slot >= 0);
      if (lane == 0) piece_there[stage] = there;
      if (i < pieces) S::template issue<true, true>(v, key, value, group, max(slot, 0), ring_u32 + stage * S::kBytes, lane);
      cp_async_commit();
    };
    int32_t slot = slot_of(0);
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
      const int32_t next = slot_of(i + 1);
      fill(i, slot, i);
      slot = next;
    }

    // one piece; PLAIN: every row sees every token, and no zero leaves a remainder
    auto piece = [&](auto plain, uint8_t* st, uint32_t there, int32_t t0, bool force) {
      constexpr bool PLAIN = decltype(plain)::value;
      const float4* prep = reinterpret_cast<const float4*>(st + S::kMeta);
      float x[2][NC][4], top[NC][2];
#pragma unroll
      for (int n = 0; n < NC; ++n) top[n][0] = top[n][1] = -INFINITY;
      float hi[2][NC][4];
      key_scores<D, NC>(st, lane, q, x, hi);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {                     // tokens g and g + 8
          const int t = 16 * h + 8 * e + g;
          const float4 k = prep[t];
#pragma unroll
          for (int n = 0; n < NC; ++n) {
            float* y = &x[h][n][2 * e];                   // x_t - m
#pragma unroll
            for (int i = 0; i < 2; ++i)
              y[i] = fmaf(fmaf(k.y, qsum[n][i], fmaf(hi[h][n][2 * e + i], 0.0625f, y[i])), k.x, nm[n][i]);
            if constexpr (!PLAIN) {
              const bool is = (there >> t) & 1u;
              if (!is || t0 + t >= row_limit[8 * n + 2 * c]) y[0] = -INFINITY;
              if (!is || t0 + t >= row_limit[8 * n + 2 * c + 1]) y[1] = -INFINITY;
            }
            top[n][0] = fmaxf(top[n][0], y[0] + k.z);
            top[n][1] = fmaxf(top[n][1], y[1] + k.z);
          }
        }
      }
      float over = top[0][0];
#pragma unroll
      for (int n = 0; n < NC; ++n) over = fmaxf(fmaxf(over, top[n][0]), top[n][1]);
      if (__any_sync(0xffffffffu, over > kMost) || force) {
#pragma unroll
        for (int n = 0; n < NC; ++n) {
          float up[2], f[2];                              // what m grows by
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float y = top[n][k];
#pragma unroll
            for (int s = 4; s < 32; s <<= 1) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, s));
            const uint32_t bit = 1u << (2 * n + k);
            up[k] = y == -INFINITY ? 0.0f : started & bit ? fmaxf(y - kTop, 0.0f) : y - kTop;
            f[k] = started & bit ? exp2_fast(-up[k]) : 1.0f;
            if (y != -INFINITY) started |= bit;
            zs[n][k] *= f[k];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              x[h][n][k] -= up[k];
              x[h][n][2 + k] -= up[k];
            }
          }
          nm[n][0] -= up[0];
          nm[n][1] -= up[1];
          const uint64_t f2 = f2_pack(f[0], f[1]);
          l2[n] = f2_mul(l2[n], f2);
#pragma unroll
          for (int j = 0; j < T::kTiles; ++j) {
            o[j][n][0] = f2_mul(o[j][n][0], f2);
            o[j][n][1] = f2_mul(o[j][n][1], f2);
          }
        }
      }
      uint32_t wh[2][NC][2], wl[2][NC][2], z1024[2][2];
      uint64_t lp[NC];                                     // the piece's share of l: few additions to a large sum
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int t = 16 * h + 8 * e + g;
          const float sv = prep[t].w;
          z1024[h][e] = *reinterpret_cast<const uint32_t*>(prep_z + 16 * h + 8 * e + 2 * c);
#pragma unroll
          for (int n = 0; n < NC; ++n) {
            const float y0 = x[h][n][2 * e], y1 = x[h][n][2 * e + 1];
            float w0, w1;
            const float p0 = exp2_fast(y0), p1 = exp2_fast(y1);
            lp[n] = h + e == 0 ? f2_pack(p0, p1) : f2_add(lp[n], f2_pack(p0, p1));
            w0 = p0 * sv;
            w1 = p1 * sv;
            if constexpr (!PLAIN) {
              if (y0 == -INFINITY) w0 = 0.0f;              // a scale that is not seen may be anything
              if (y1 == -INFINITY) w1 = 0.0f;
              const float r = prep_rest[t];
              if (r != 0.0f) {
                zs[n][0] = fmaf(w0, r, zs[n][0]);
                zs[n][1] = fmaf(w1, r, zs[n][1]);
              }
            }
            const __half2 hi = __floats2half2_rn(w0, w1);
            const float2 back = __half22float2(hi);
            float r0, r1;
            f2_unpack(f2_sub(f2_pack(w0, w1), f2_pack(back.x, back.y)), r0, r1);
            const __half2 lo = __floats2half2_rn(r0, r1);
            wh[h][n][e] = transpose_8x8(*reinterpret_cast<const uint32_t*>(&hi));
            wl[h][n][e] = transpose_8x8(*reinterpret_cast<const uint32_t*>(&lo));
          }
        }
      }
#pragma unroll
      for (int n = 0; n < NC; ++n) l2[n] = f2_add(l2[n], lp[n]);
      value_products<D, NC>(st + S::kCodes, g, c, z1024, wh, wl, o);
    };

    int stage = 0;
    bool force = true;                                   // some column may have seen no key yet
    for (int32_t i = 0; i < pieces; ++i) {
      const int32_t next = slot_of(i + kStages);
      fill(i + kStages - 1, slot, stage == 0 ? kStages - 1 : stage - 1);
      slot = next;
      cp_async_wait<kStages - 1>();
      __syncwarp();
      uint8_t* st = ring + stage * S::kBytes;
      const int32_t t0 = first + i * ws * kStep;
      // each lane makes one token's numbers ready for all, in place of the four it came with
      float4* prep = reinterpret_cast<float4*>(st + S::kMeta);
      const float* meta = reinterpret_cast<const float*>(prep);
      const uint32_t there = piece_there[stage];
      const int32_t zv = __float_as_int(meta[96 + lane]), zc = min(max(zv, -900), 900);
      const float sk = meta[lane] * (a.scale_log2 * 16777216.0f);
      const float zk = (static_cast<float>(__float_as_int(meta[32 + lane])) + 8.0f) * -0x1p-24f;
      const float sv = meta[64 + lane], lv = fminf(fmaxf(__log2f(sv), -40.0f), 40.0f);
      const bool plain = there == 0xffffffffu && t0 + kStep <= all_limit && !__any_sync(0xffffffffu, zv != zc);
      __syncwarp();
      prep[lane] = make_float4(sk, zk, lv, sv);
      prep_z[lane] = __int2half_rn(-1032 - zc);
      prep_rest[lane] = static_cast<float>(static_cast<int64_t>(zv) - zc);
      __syncwarp();
      if (plain) piece(std::true_type{}, st, there, t0, force);
      else piece(std::false_type{}, st, there, t0, force);
      if (force) force = __any_sync(0xffffffffu, started != (1u << (2 * NC)) - 1);
      stage = stage + 1 == kStages ? 0 : stage + 1;
      __syncwarp();
    }
    cp_async_wait<0>();

    float m[NC][2], l[NC][2];
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      f2_unpack(l2[n], l[n][0], l[n][1]);
      m[n][0] = -nm[n][0];
      m[n][1] = -nm[n][1];
    }
    // sums of column k of product j, row g or g + 8, without the remainder
    auto sum_of = [&](int j, int n, int k, bool upper) {
      float y[2];
      f2_unpack(o[j][n][upper], y[0], y[1]);
      return y[k] - zs[n][k];
    };
#pragma unroll
    for (int n = 0; n < NC; ++n)
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int s = 4; s < 32; s <<= 1) {
          l[n][k] += __shfl_xor_sync(0xffffffffu, l[n][k], s);
          zs[n][k] += __shfl_xor_sync(0xffffffffu, zs[n][k], s);
        }
    const int part = done == 0 ? 0 : 1;
    if (ws == 1) {
#pragma unroll
      for (int n = 0; n < NC; ++n)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int32_t r = 8 * n + 2 * c + k, rr = row0 + r;
          if (rr >= all_rows) continue;
          const float inv = whole ? inverse_or_zero(l[n][k]) : 1.0f;
          float y[T::kPer];
#pragma unroll
          for (int j = 0; j < T::kTiles; ++j) {
            y[T::element(j, false)] = sum_of(j, n, k, false) * inv;
            y[T::element(j, true)] = sum_of(j, n, k, true) * inv;
          }
          if (whole) {
            const int64_t token = rows.first + rr / a.plan.gq;
            const int h = head * a.plan.gq + rr % a.plan.gq;
            store_half(a.out + token * a.ldo + h * D + g * T::kPer, y);
            if (a.lse != nullptr && g == 0) a.lse[token * a.q_heads + h] = row_lse(m[n][k], l[n][k]);
          } else {
            const int64_t p = part_at(a, blockIdx.x, part, hw, r);
            float4* to = reinterpret_cast<float4*>(a.part_o + p * D + g * T::kPer);
#pragma unroll
            for (int j = 0; j < T::kPer / 4; ++j) to[j] = make_float4(y[4 * j], y[4 * j + 1], y[4 * j + 2], y[4 * j + 3]);
            if (g == 0) a.part_ml[p] = make_float2(m[n][k], l[n][k]);
          }
        }
    } else {
      // the warps of a head meet: rows of D sums, m and l in shared memory
      __syncthreads();
      float* mine = reinterpret_cast<float*>(smem) + warp * R * (D + 2);
#pragma unroll
      for (int n = 0; n < NC; ++n)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float* to = mine + (8 * n + 2 * c + k) * (D + 2);
#pragma unroll
          for (int j = 0; j < T::kTiles; ++j) {
            to[g * T::kPer + T::element(j, false)] = sum_of(j, n, k, false);
            to[g * T::kPer + T::element(j, true)] = sum_of(j, n, k, true);
          }
          if (g == 0) *reinterpret_cast<float2*>(to + D) = make_float2(m[n][k], l[n][k]);
        }
      __syncthreads();
      // a row's factors, one row a thread, in place of m.  A warp that saw no key (l = 0) has no maximum either; a row of
      // NaN has its l
      float* all = reinterpret_cast<float*>(smem);
      const int next = (R << a.heads_log2) * (D + 2);    // from a head's rows to those of its next warp
      for (int e = threadIdx.x; e < R << a.heads_log2; e += kThreads) {
        const int r = e % R, h0 = e / R;
        const int32_t rr = row0 + r;
        if (rr >= all_rows) continue;
        float* at = all + e * (D + 2) + D;
        float mm = -INFINITY, ll = 0.0f;
        for (int s = 0; s < ws; ++s) {
          const float2 ml = *reinterpret_cast<const float2*>(at + s * next);
          if (ml.y != 0.0f) mm = fmaxf(mm, ml.x);
        }
        for (int s = 0; s < ws; ++s) {
          const float2 ml = *reinterpret_cast<const float2*>(at + s * next);
          const float f = ml.y == 0.0f ? 0.0f : ml.x == mm ? 1.0f : exp2_fast(ml.x - mm);
          ll = fmaf(ml.y, f, ll);
          at[s * next] = f;
        }
        at[1] = whole ? inverse_or_zero(ll) : 1.0f;
        if (!whole) {
          a.part_ml[part_at(a, blockIdx.x, part, h0, r)] = make_float2(mm, ll);
        } else if (a.lse != nullptr) {
          const int h = ((block << a.heads_log2) + h0) * a.plan.gq + rr % a.plan.gq;
          a.lse[static_cast<int64_t>(rows.first + rr / a.plan.gq) * a.q_heads + h] = row_lse(mm, ll);
        }
      }
      __syncthreads();
      for (int e = threadIdx.x; e < (R << a.heads_log2) * (D / 2); e += kThreads) {
        const int d2 = e % (D / 2) * 2, hr = e / (D / 2), r = hr % R, h0 = hr / R;
        const int32_t rr = row0 + r;
        if (rr >= all_rows) continue;
        const float* from = all + hr * (D + 2);
        const float inv = from[D + 1];
        float y0 = 0.0f, y1 = 0.0f;
        for (int s = 0; s < ws; ++s) {
          const float f = from[s * next + D];
          const float2 y = *reinterpret_cast<const float2*>(from + s * next + d2);
          y0 = fmaf(y.x, f, y0);
          y1 = fmaf(y.y, f, y1);
        }
        if (whole) {
          const int64_t token = rows.first + rr / a.plan.gq;
          const int h = ((block << a.heads_log2) + h0) * a.plan.gq + rr % a.plan.gq;
          *reinterpret_cast<__half2*>(a.out + token * a.ldo + h * D + d2) = __floats2half2_rn(y0 * inv, y1 * inv);
        } else {
          *reinterpret_cast<float2*>(a.part_o + part_at(a, blockIdx.x, part, h0, r) * D + d2) = make_float2(y0, y1);
        }
      }
      __syncthreads();
    }
    done += take;
  }
}

// Adds up the parts of items that were cut.  JW = 1: one warp a row, its lanes the elements of the head; a block
// looks after the item that range blockIdx.y is the first to hold and not the last, if there is one, and
// takes 8 `loops` of its rows (token, query head).  JW = 8, for few rows with many parts: one block a row and 32
// elements, its warps take every eighth part.
// The sum over the parts of ranges first, first + JW, .. last (from jw on) of a row: r of head hb of a block.
template <int D, int JW, int E>
__device__ __forceinline__ void join_parts(const SplitArgs& a, const Ranges& ranges, int64_t u0, int32_t first,
                                           int32_t last, int jw, int hb, int r, int e0, float& m, float& l,
                                           float (&o)[E]) {
  constexpr int F = JW == 1 ? 8 : 16;                    // parts in flight
  const int lane = threadIdx.x & 31;
  m = -INFINITY;
  l = 0.0f;
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.0f;
  // 32 parts at a time: their m and l, one a lane, then their sums, several in flight
  for (int32_t c0 = first; c0 <= last; c0 += 32 * JW) {
    const int32_t blk = c0 + lane * JW + jw;
    int64_t p = 0;
    float2 x = make_float2(-INFINITY, 0.0f);
    if (blk <= last) {
      p = part_at(a, blk, ranges.start(blk) >= u0 ? 0 : 1, hb, r);
      x = a.part_ml[p];
    }
    float top = x.y != 0.0f ? x.x : -INFINITY;           // a part without a key has no m (a row of NaN has l)
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
    const float m1 = fmaxf(m, top);
    const float keep = m == m1 ? 1.0f : exp2_fast(m - m1);
    const float mine = x.y == 0.0f ? 0.0f : x.x == m1 ? 1.0f : exp2_fast(x.x - m1);
    float ls = x.y * mine;
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, s);
    l = fmaf(l, keep, ls);
    m = m1;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= keep;
    uint32_t left = __ballot_sync(0xffffffffu, x.y != 0.0f);
    while (left != 0) {
      float f8[F], y[F][E];
#pragma unroll
      for (int k = 0; k < F; ++k) {
        const int from = left != 0 ? __ffs(left) - 1 : -1;
        left &= left - 1;
        const int64_t pk = __shfl_sync(0xffffffffu, p, max(from, 0));
        f8[k] = __shfl_sync(0xffffffffu, mine, max(from, 0));
        const float* src = a.part_o + pk * D;
#pragma unroll
        for (int e = 0; e < E; ++e) y[k][e] = from >= 0 ? src[e0 + 32 * e] : 0.0f;
        if (from < 0) f8[k] = 0.0f;
      }
#pragma unroll
      for (int k = 0; k < F; ++k)
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(y[k][e], f8[k], o[e]);
    }
  }
}

template <int D, int JW>
__global__ void __launch_bounds__(256) kv_join_kernel(const SplitArgs a, int loops) {
  constexpr int E = JW == 1 ? D / 32 : 1;
  __shared__ float acc[JW][32];
  __shared__ float2 ml[JW];
  const KvView& v = a.v;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, jw = JW == 1 ? 0 : warp;
  const int e0 = JW == 1 ? lane : blockIdx.x % (D / 32) * 32 + lane;       // this lane's elements: e0 + 32 e
  grid_dep_wait();
  grid_dep_launch();
  const int64_t units = a.prefix[v.batch];
  const Ranges ranges = Ranges::of(a.plan, units);
  auto finish = [&](int32_t i, int32_t h, float m, float l, const float (&o)[E]) {
    const float inv = inverse_or_zero(l);
#pragma unroll
    for (int e = 0; e < E; ++e) a.out[i * a.ldo + h * D + e0 + 32 * e] = __float2half_rn(o[e] * inv);
    if (a.lse != nullptr && e0 == 0) a.lse[static_cast<int64_t>(i) * a.q_heads + h] = row_lse(m, l);
  };
  float m, l, o[E];
  if (JW == 1) {
    const int32_t c = blockIdx.y;
    if (c + 1 >= ranges.blocks) return;
    const int64_t u = ranges.start(c + 1) - 1;           // the last unit of the range
    int32_t n = 0;
    for (int32_t j = lane; j < v.batch; j += 32) n += a.prefix[j + 1] <= u ? 1 : 0;
    int32_t b = __reduce_add_sync(0xffffffffu, n);
    const Item it = find_item<false>(v, a.plan, a.prefix, u, 1, &b);
    const int32_t tu = tile_units(a.plan, it.rows, it.tile);
    const int64_t u0 = u - it.unit;
    const int32_t first = ranges.holder(u0), last = min(ranges.holder(u0 + tu - 1), ranges.blocks - 1);
    if (first != c || last == c) return;
    const int32_t all_rows = it.rows.here * a.plan.gq;
#pragma unroll 1
    for (int s = 0; s < loops; ++s) {
      const int32_t k = (blockIdx.x * loops + s) * 8 + warp;     // row of the item: head of the block, row of the tile
      const int32_t hb = k / a.plan.rows, r = k - hb * a.plan.rows, row = it.tile * a.plan.rows + r;
      if (hb >= (1 << a.heads_log2) || row >= all_rows) continue;
      join_parts<D, 1, E>(a, ranges, u0, first, last, 0, hb, r, e0, m, l, o);
      finish(it.rows.first + row / a.plan.gq, ((it.block << a.heads_log2) + hb) * a.plan.gq + row % a.plan.gq, m, l, o);
    }
    return;
  }
  const int64_t job = blockIdx.x / (D / 32);
  const int32_t i = static_cast<int32_t>(job / a.q_heads), h = static_cast<int32_t>(job % a.q_heads);
  const int32_t b = kv_seq_of_row(v, i);
  if (b >= v.batch) return;                              // (the whole block)
  const SeqRows rows = seq_rows(v, b);
  const int32_t ti = i - rows.first;
  if (ti < 0 || ti >= rows.here) return;
  const int hk = h / a.plan.gq;
  const int32_t row = ti * a.plan.gq + h % a.plan.gq, tile = row / a.plan.rows;
  int64_t u0 = a.prefix[b];
  for (int32_t t = 0; t < tile; ++t) u0 += static_cast<int64_t>(tile_units(a.plan, rows, t)) * a.plan.head_blocks;
  const int32_t tu = tile_units(a.plan, rows, tile);
  u0 += static_cast<int64_t>(hk >> a.heads_log2) * tu;
  const int32_t first = ranges.holder(u0), last = min(ranges.holder(u0 + tu - 1), ranges.blocks - 1);
  if (first >= last) return;
  join_parts<D, JW, E>(a, ranges, u0, first, last, jw, hk & ((1 << a.heads_log2) - 1), row % a.plan.rows, e0, m, l, o);
  acc[jw][lane] = o[0];
  if (lane == 0) ml[jw] = make_float2(m, l);
  __syncthreads();
  if (jw != 0) return;
  for (int w = 0; w < JW; ++w) m = fmaxf(m, ml[w].x);
  l = o[0] = 0.0f;
  for (int w = 0; w < JW; ++w) {
    const float2 x = ml[w];
    const float f = x.y == 0.0f ? 0.0f : x.x == m ? 1.0f : exp2_fast(x.x - m);
    l = fmaf(x.y, f, l);
    o[0] = fmaf(acc[w][lane], f, o[0]);
  }
  finish(i, h, m, l, o);
}

struct SplitSizes {
  int nc, heads_log2, blocks, unit, rows;
  bool prefill;                                // kv_prefill.cu
  bool whole;                                  // no item is cut: nothing to join
  int64_t prefix_bytes, ml_bytes, bytes;
};

// Short contexts on few heads: fewer heads a block, more warps a head (they join in shared memory), and items
// that are not cut, which spares the second kernel; taken where all items fit one wave of blocks with at
// most kWholePieces pieces a warp.  Elsewhere eight heads a block: warps that read the same tokens' scales
// share their sectors (one head a block: 64 us instead of 58 for one sequence of 131072 tokens, 64/8 heads).
constexpr int kWholePieces = 8;
// Rows of a sequence and key head (on average) up to which the codes go through registers, 16 rows a tile (8 for heads
// of 256); beyond, through shared memory to tcgen05, whose time hardly depends on the rows up to 128.
// Registers against tcgen05, us: 64 sequences of up to 4096 tokens, 64/8 heads: 26 rows 156 and 256, 37 rows 221 and
// 267, 47 rows 248 and 255; 16 of 2048, 32/32 heads: 23 rows 104 and 175.  With 32 to 64 items of 4096 tokens the tiles'
// starts and joins weigh more: 16 sequences, 28/4 heads: 16 rows 62 and 51, 29 rows 52 and 52; and 4, 64/8 heads, 48 and 39.
// A batch that mixes both kinds goes one way as a whole: 2048 rows on 4096 tokens beside 63 single tokens, 64/8 heads, 755 us
// where apart they take 412 and 88; 512 rows beside 255, 609 us (168 and 150).
constexpr int kFewRows = 32;

SplitSizes split_sizes(const KvView& v, int32_t q_heads) {
  SplitSizes s{};
  const int gq = q_heads / v.heads;
  const int64_t rows = (static_cast<int64_t>(v.tokens) * gq + v.batch - 1) / v.batch;   // of a sequence, on average
  s.prefill = rows > kFewRows && kv_prefill_takes(v);
  s.nc = rows > 8 && v.head_dim <= 128 ? 2 : 1;
  s.rows = s.prefill ? kv_prefill_rows(v.head_dim) : 8 * s.nc;
  s.blocks = sm_count() * (s.prefill || v.head_dim == 256 || s.nc == 2 ? 1 : 2);
  s.prefix_bytes = (8 * (static_cast<int64_t>(v.batch) + 1) + 255) / 256 * 256;
  auto parts = [&] {
    const int64_t n = (2ll * s.blocks << s.heads_log2) * s.rows;
    s.ml_bytes = n * 8;
    s.bytes = s.prefix_bytes + s.ml_bytes + n * v.head_dim * 4;
  };
  if (s.prefill) {
    s.unit = 128;
    parts();
    return s;
  }
  int most = 0;
  while (most < 3 && v.heads % (2 << most) == 0) ++most;
  const int64_t tiles = std::max<int64_t>(v.batch, (static_cast<int64_t>(v.tokens) * gq + 8 * s.nc - 1) / (8 * s.nc));
  while (s.heads_log2 < most && tiles * (v.heads >> s.heads_log2) > s.blocks) ++s.heads_log2;
  int step = kStep * (kWarps >> s.heads_log2);
  s.whole = tiles * (v.heads >> s.heads_log2) <= s.blocks && v.capacity <= kWholePieces * step;
  if (!s.whole) {
    s.heads_log2 = most;
    step = kStep * (kWarps >> most);
  }
  s.unit = s.whole ? kWholePieces * step : step;
  if (!s.whole) parts();
  return s;
}

// The kernel that joins what the ranges cut.
template <int D>
cudaError_t run_join(const SplitArgs& a, bool prefill, cudaStream_t stream) {
  // few rows with many parts: eight warps a row
  const int64_t rows = static_cast<int64_t>(a.v.tokens) * a.q_heads;
  const int64_t items = std::max<int64_t>(1, static_cast<int64_t>(a.v.batch) * a.plan.head_blocks);
  if (!prefill && rows <= 8 * sm_count() && a.plan.blocks > 8 * items)
    return launch_pdl(kv_join_kernel<D, 8>, dim3(static_cast<unsigned>(rows * (D / 32))), dim3(256), 0, stream, 1, a, 1);
  const int64_t most = std::min<int64_t>(a.plan.rows, static_cast<int64_t>(a.v.tokens) * a.plan.gq);
  const int64_t all = a.heads_log2 == 0 ? most : static_cast<int64_t>(a.plan.rows) << a.heads_log2;
  // (most blocks find that their range cuts nothing: of the many rows of a prompt's item a warp takes four, of few one)
  const int loops = prefill ? 4 : 1;
  const unsigned blocks = static_cast<unsigned>((all + 8 * loops - 1) / (8 * loops));
  return launch_pdl(kv_join_kernel<D, 1>, dim3(blocks, a.plan.blocks), dim3(256), 0, stream, 1, a, loops);
}

template <int D, int NC>
cudaError_t run_split(const SplitArgs& a, cudaStream_t stream) {
  const size_t smem = tile_bytes<D, NC>() + (a.v.batch + 1) * sizeof(int64_t);
  static std::atomic<uint64_t> done{0};
  constexpr int kMost = tile_bytes<D, NC>() + (4096 + 1) * 8;
  cudaError_t e = allow_smem(kv_split_kernel<D, NC>, kMost, done);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kv_split_kernel<D, NC>, dim3(a.plan.blocks), dim3(kThreads), smem, stream, 1, a);
  return e != cudaSuccess || a.prefix == nullptr ? e : run_join<D>(a, false, stream);
}

template <int D>
cudaError_t run_attention(const SplitArgs& a, const SplitSizes& s, cudaStream_t stream) {
  if (s.prefill) {
    const cudaError_t e = launch_kv_prefill(a, stream);
    return e != cudaSuccess ? e : run_join<D>(a, true, stream);
  }
  if constexpr (D <= 128)
    if (s.nc == 2) return run_split<D, 2>(a, stream);
  return run_split<D, 1>(a, stream);
}

}  // namespace

int64_t kv_attention_workspace(const KvView& v, int32_t q_heads) { return split_sizes(v, q_heads).bytes; }

qr_status launch_kv_attention(const KvView& v, const KvAttentionJob& j, cudaStream_t stream) {
  const SplitSizes s = split_sizes(v, j.q_heads);
  SplitArgs a{};
  a.v = v;
  a.plan.gq = j.q_heads / v.heads;
  a.plan.rows = s.rows;
  a.plan.unit = s.unit;
  a.plan.head_blocks = v.heads >> s.heads_log2;
  a.plan.blocks = s.blocks;
  a.plan.causal = j.causal;
  a.q = reinterpret_cast<const __half*>(j.q);
  a.ldq = j.ldq;
  a.q_heads = j.q_heads;
  a.scale_log2 = static_cast<float>(static_cast<double>(j.scale) * 1.4426950408889634);
  a.out = reinterpret_cast<__half*>(j.out);
  a.ldo = j.ldo;
  a.lse = j.lse;
  a.prefix = s.whole ? nullptr : static_cast<int64_t*>(j.workspace);
  a.part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(j.workspace) + s.prefix_bytes);
  a.part_o = reinterpret_cast<float*>(static_cast<uint8_t*>(j.workspace) + s.prefix_bytes + s.ml_bytes);
  a.heads_log2 = s.heads_log2;
  cudaError_t e;
  switch (v.head_dim) {
    case 32: e = run_attention<32>(a, s, stream); break;
    case 64: e = run_attention<64>(a, s, stream); break;
    case 128: e = run_attention<128>(a, s, stream); break;
    default: e = run_attention<256>(a, s, stream); break;
  }
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? QR_OK : QR_ERR_CUDA;
}

}  // namespace qr
