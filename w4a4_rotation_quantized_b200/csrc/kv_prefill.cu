// kv_prefill.cu -- attention over the paged 4-bit KV cache for many query rows a key head
// (prompts, chunks of prompts, drafts, cross attention): tensor-bound, 4 d operations a pair of
// query row and key.
//
// A block takes one key head and two tiles of 128 query rows (token, head of the group; one tile where a head
// is 256 wide) over a range of keys, 128 at a time:
//   S = Q K^T     tcgen05, both operands in shared memory, 128 x 64 fp32 in tensor memory, twice
//   W = 2^(y - m) softmax warps, one row a thread, written back over S as fp16
//   O += W V      tcgen05, W from tensor memory, V rows as they stand (MN-major), O in tensor memory
// Codes become fp16 operands in shared memory as the whole numbers c - z, exact (kv_mma.cuh); the scales stay out
// of them: with y_t = s_k (q . (c - z)) scale log2 e + log2 s_v the weight 2^(y - m) carries the value's scale, and
// l = sum 2^(y - m) / s_v.  m follows the maximum of y with a lag of up to 15, so that weights stay below 2^15 in fp16
// and those that matter are not small ones, whatever the scales are; log2 s_v is held to [-40, 40], a value scale
// below 2^-40 counts as 0.  Zeros beyond +-900 leave remainders, added to the scores and taken from the
// outputs apart, in a second version of the softmax loops that such blocks of keys take.
//
// 13 warps (so that a thread may have 128 registers): two softmax warpgroups (one a tile), four warps that load and
// unpack the next keys, one token a thread, one that issues the matrix instructions: while one tile is in its
// softmax the tensor cores have the other.  Two tiles share an unpacked key tile.  Scores come 64 keys at a time into
// two places a tile, so that the next ones are there when the softmax has done with the last.
// The softmax goes over the scores once, 32 columns at a time, with the maximum of the keys before: only when a
// weight of the columns at hand would pass 2^15 is m raised, by a whole number, and what has been made with the
// old one (l, O, the weights of these 64 keys) multiplied by that power of two.  The roles go through the block's
// items each on its own, so that the next item's queries and first scores are there when the softmax has written
// the last one's outputs.  Work is shared out and joined as in kv_split.cuh.
//
// 2048 new tokens on 8192, 64/8 heads of 128: 805 us, 597 TFLOP/s.  The softmax warps' instructions bound it, by their
// latency: two of them a scheduler, some 5 instructions a score.  Measured and left, against 842 us of the
// kernel as it was then: the next 32 columns loaded ahead (890 us: registers), both tiles' rows in one thread (1248 us: half
// the reads of the columns' numbers, but one softmax warp a scheduler), the maximum found first (1228 us).  128 keys at a
// time in one place took 835 us, but with waits that could mistake one completion for the next; it was not made sound.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "kv_mma.cuh"
#include "kv_split_args.cuh"
#include "qr_internal.h"

namespace qr {

namespace {

constexpr int kKeys = 128;                     // keys of a block step
constexpr int kSoftmaxThreads = 128;           // of a tile
constexpr int kUnpackThreads = 128;
constexpr int kThreadsP = 2 * kSoftmaxThreads + kUnpackThreads + 32;
constexpr int kMaxBatch = 2048;
// Steps whose products are summed in tensor memory, 8192 keys.  These sums cut what they are too small for instead of
// rounding it, some 2^-23.5 of themselves for every 16 keys (measured: 7e-4 of the result after 131072 keys, 1.5e-4
// after 32768, 4e-5 after 8192, a twelfth of the output's own rounding); chains are added up in fp32.
constexpr int32_t kChain = 64;

template <int D>
struct Shape {
  static constexpr int kTiles = D == 256 ? 1 : 2;
  static constexpr int kStages = D == 256 ? 1 : 2;
  static constexpr int kSubs = D < 64 ? 1 : D / 64;           // 128-byte columns of a row
  static constexpr int kTile = kSubs * 16384;                 // 128 rows
  static constexpr int kQ = kTiles * kTile;
  static constexpr int kStage = 2 * kTile;                    // keys, values
  static constexpr int kCols = 5 * kKeys * 4 + 32;            // numbers of the keys of a stage
  static constexpr int kBytes = kQ + kStages * kStage + kStages * kCols + 256;
  static constexpr int kWords = D / 8;                        // code words of a token's key, or its value
};

// Column numbers of a stage.
struct Cols {
  float *sk, *lv, *rsv, *rk, *rv;
  int32_t* rest;                               // [4]: any remainder among a warp's 32 keys
  __device__ __forceinline__ explicit Cols(uint8_t* p) {
    sk = reinterpret_cast<float*>(p);
    lv = sk + kKeys;
    rsv = lv + kKeys;
    rk = rsv + kKeys;
    rv = rk + kKeys;
    rest = reinterpret_cast<int32_t*>(rv + kKeys);
  }
};

// A wait names the completion it wants by its parity, so it must come when the one before is known to be over:
// kSFull, kPFull and kODone have a barrier for each place of a tile (2 t + place), since the products of one
// place may still run when the other's are waited for.
enum Bar { kQFull = 0, kKFull = 1, kVFull = 3, kFree = 5, kSFull = 7, kPFull = 11, kODone = 15, kORead = 19, kQFree = 21, kBars = 22 };

// Byte of the 16-byte chunk `chunk` (of 8 elements) of row r in a swizzled tile of 128 rows.
__device__ __forceinline__ int tile_at(int r, int chunk) {
  return (chunk >> 3) * 16384 + r * 128 + (((chunk & 7) ^ (r & 7)) << 4);
}

template <int D>
__global__ void __launch_bounds__(kThreadsP, 1) kv_prefill_kernel(const SplitArgs a, int32_t* status) {
  using P = Shape<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + (1024 - (smem_u32(smem_raw) & 1023)) % 1024;
  uint8_t* q_tile = smem;
  uint8_t* kv_tile = smem + P::kQ;
  uint8_t* cols_at = kv_tile + P::kStages * P::kStage;
  uint64_t* bars = reinterpret_cast<uint64_t*>(cols_at + P::kStages * P::kCols);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kBars);
  volatile int32_t* abort_flag = reinterpret_cast<volatile int32_t*>(tmem_slot + 1);
  int64_t* prefix = reinterpret_cast<int64_t*>(cols_at + P::kStages * P::kCols + 256);
  const KvView& v = a.v;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  if (tid == 0) {
    mbar_init(&bars[kQFull], kUnpackThreads);
    mbar_init(&bars[kQFree], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars[kKFull + i], kUnpackThreads);
      mbar_init(&bars[kVFull + i], kUnpackThreads);
      mbar_init(&bars[kFree + i], 1);
      for (int k = 0; k < 2; ++k) {
        mbar_init(&bars[kSFull + 2 * k + i], 1);
        mbar_init(&bars[kODone + 2 * k + i], 1);
        mbar_init(&bars[kPFull + 2 * k + i], kSoftmaxThreads);
      }
      mbar_init(&bars[kORead + i], kSoftmaxThreads);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 12) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  grid_dep_wait();
  grid_dep_launch();
  split_prefix<kThreadsP, true>(v, a.plan, prefix);
  const int64_t units = prefix[v.batch];
  if (blockIdx.x == 0)
    for (int32_t b = tid; b <= v.batch; b += kThreadsP) a.prefix[b] = prefix[b];
  const Ranges ranges = Ranges::of(a.plan, units);
  const int64_t start = ranges.start(blockIdx.x);
  const int32_t count = ranges.count(blockIdx.x);

  auto wait = [&](int bar, uint32_t n, int32_t code) -> bool {      // the n-th completion (from 0)
    return mbar_wait_bounded(&bars[bar], n & 1, abort_flag, status, code);
  };
  auto wait_warp = [&](int bar, uint32_t n, int32_t code) -> bool {  // ... by a whole warp, with one answer
    return __all_sync(0xffffffffu, wait(bar, n, code));
  };

  // what a role counts as it goes through the items: key tiles and items, of the block and of each query tile
  struct Counts {
    uint32_t steps, items, tile_steps[2], tile_items[2];
    __device__ __forceinline__ void next(int32_t take, int tiles) {
      steps += take;
      ++items;
      for (int t = 0; t < tiles; ++t) {
        tile_steps[t] += take;
        ++tile_items[t];
      }
    }
  } n{};
  auto tiles_of = [&](const Item& it) {
    return P::kTiles == 2 && it.tile * a.plan.rows + 128 < it.rows.here * a.plan.gq ? 2 : 1;
  };
  bool ok = true;
  int32_t b = 0;

  if (warp < 8) {
    // --------------------------------------------------------------- softmax
    const int t = warp >> 2;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;            // 32 (warp & 3) in the lane field
    const uint32_t o_at = tmem + lanes + 256 + t * D;
    const int r = 128 * t + (warp & 3) * 32 + lane;
    // the item's keys that this block takes, in chains: its first unit, its place among the parts, which also keeps the
    // sums between chains, and m and l so far
    int32_t run_unit = 0;
    int run_slot = 0;
    float run_m = 0.0f, run_l = 0.0f;
    for (int32_t done = 0, run_end = 0; done < count && ok;) {
      const Item it = find_item(v, a.plan, prefix, start + done, min(count - done, kChain), &b);
      const int tiles = tiles_of(it);
      if (done == run_end) {                               // another item
        run_unit = it.unit;
        run_slot = done == 0 ? 0 : 1;
        run_end = done + min(it.units - it.unit, count - done);
      }
      if (t < tiles) {
        const int32_t row0 = it.tile * a.plan.rows, rr = row0 + r;
        const bool has = rr < it.rows.here * a.plan.gq;
        const int32_t tok = has ? rr / a.plan.gq : 0, qh = it.block * a.plan.gq + (has ? rr % a.plan.gq : 0);
        const int32_t limit = has ? seen(it.rows, tok, a.plan.causal) : 0;
        const int32_t all_limit = seen(it.rows, (row0 + 128 * t) / a.plan.gq, a.plan.causal);
        float m = 0.0f, zs = 0.0f, qsum = 0.0f;
        uint64_t l2 = 0;
        bool started = !has, summed = false;               // (rows of nobody hold nothing up)
        for (int32_t j = 0; j < 2 * it.take; ++j) {
          const uint32_t step = n.steps + (j >> 1), nt = 2 * n.tile_steps[t] + j;     // j, nt: 64 keys at a time
          const int st = step % P::kStages, place = j & 1;
          const uint32_t s_at = tmem + lanes + 128 * t + 64 * place;
          ok = wait_warp(kSFull + 2 * t + place, nt >> 1, kDevTimeoutEpilogue) &&
               wait_warp(kKFull + st, step / P::kStages, kDevTimeoutEpilogue);      // (has been: to see its numbers)
          if (!ok) break;
          tc_fence_after();
          const Cols cols(cols_at + st * P::kCols);
          const int32_t t0 = it.unit * kKeys + j * 64;
          const int col0 = 64 * place;
          const int4 rest4 = *reinterpret_cast<const int4*>(cols.rest);
          const bool rest = (rest4.x | rest4.y | rest4.z | rest4.w) != 0;
          const bool plain = t0 + 64 <= all_limit && !rest;
          if (rest && !summed) {                           // sum of the row's queries, for remainders of key zeros
            summed = true;
            if (has) {
              const __half* q_row = a.q + (it.rows.first + tok) * a.ldq + static_cast<int64_t>(qh) * D;
              for (int e = 0; e < D; e += 8) {
                const uint4 x = *reinterpret_cast<const uint4*>(q_row + e);
                const __half2* h = reinterpret_cast<const __half2*>(&x);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const float2 f = __half22float2(h[i]);
                  qsum += f.x + f.y;
                }
              }
            }
          }
          const int32_t lim = limit - t0;
          // raises m where a weight would pass 2^15 (and sets it where no key has been seen)
          auto raise = [&](float top, int ch) -> bool {
            const bool high = started && top > m + 15.0f;
            const float up = high ? ceilf(top - m) : 0.0f, f = high ? exp2_fast(-up) : 1.0f;
            if (high) m += up;
            else if (!started && top != -INFINITY) {
              m = top;
              started = true;
            }
            if (!__any_sync(0xffffffffu, high)) return true;
            const uint64_t f2 = f2_pack(f, f);
            l2 = f2_mul(l2, f2);
            zs *= f;
            tmem_st_wait();
#pragma unroll 1
            for (int c = 0; c < ch; ++c) {                 // the weights of this key tile so far: f in fp32, for a weight
              // of 2^15 still counts where f is below all of fp16
              uint32_t w[16];
              tmem_ld_32x32b_x16(s_at + 16 * c, w);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const float2 y = __half22float2(*reinterpret_cast<const __half2*>(w + i));
                const __half2 x = __floats2half2_rn(y.x * f, y.y * f);
                w[i] = *reinterpret_cast<const uint32_t*>(&x);
              }
              tmem_st_32x32b_x16(s_at + 16 * c, w);
            }
            if (j > 0) {
              if (!wait_warp(kODone + 2 * t + 1 - place, (nt - 1) >> 1, kDevTimeoutEpilogue)) return false;   // O is complete up to here
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                tmem_ld_32x32b_x32(o_at + 32 * c, o);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                tmem_st_32x32b_x32(o_at + 32 * c, o);
              }
            }
            tmem_st_wait();
            return true;
          };
          // 32 columns.  MODE 0: every row sees every key; 1: not so; 2: and zeros leave remainders
          auto chunk = [&](auto mode, uint32_t (&s)[32], int ch) -> bool {
            constexpr int MODE = decltype(mode)::value;
            float top = -INFINITY;
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              const int col = col0 + 32 * ch + i;
              const float4 sk = *reinterpret_cast<const float4*>(cols.sk + col);
              const float4 lv = *reinterpret_cast<const float4*>(cols.lv + col);
              uint64_t x0 = f2_pack(__uint_as_float(s[i]), __uint_as_float(s[i + 1]));
              uint64_t x1 = f2_pack(__uint_as_float(s[i + 2]), __uint_as_float(s[i + 3]));
              if constexpr (MODE == 2) {
                const float4 rk = *reinterpret_cast<const float4*>(cols.rk + col);
                x0 = f2_fma(f2_pack(-rk.x, -rk.y), f2_pack(qsum, qsum), x0);
                x1 = f2_fma(f2_pack(-rk.z, -rk.w), f2_pack(qsum, qsum), x1);
              }
              float y[4];
              f2_unpack(f2_fma(x0, f2_pack(sk.x, sk.y), f2_pack(lv.x, lv.y)), y[0], y[1]);
              f2_unpack(f2_fma(x1, f2_pack(sk.z, sk.w), f2_pack(lv.z, lv.w)), y[2], y[3]);
              if constexpr (MODE > 0) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  if (32 * ch + i + k >= lim) y[k] = -INFINITY;
              }
              top = fmaxf(fmaxf(top, fmaxf(y[0], y[1])), fmaxf(y[2], y[3]));
#pragma unroll
              for (int k = 0; k < 4; ++k) s[i + k] = __float_as_uint(y[k]);
            }
            if (__any_sync(0xffffffffu, has && (!started || top > m + 15.0f)) && !raise(has ? top : -INFINITY, ch))
              return false;
            const uint64_t nm = f2_pack(-m, -m);
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              const int col = col0 + 32 * ch + i;
              const float4 rs = *reinterpret_cast<const float4*>(cols.rsv + col);
              float y[4];
              f2_unpack(f2_add(f2_pack(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), nm), y[0], y[1]);
              f2_unpack(f2_add(f2_pack(__uint_as_float(s[i + 2]), __uint_as_float(s[i + 3])), nm), y[2], y[3]);
#pragma unroll
              for (int k = 0; k < 4; ++k) y[k] = exp2_fast(y[k]);
              l2 = f2_fma(f2_pack(y[0], y[1]), f2_pack(rs.x, rs.y), l2);
              l2 = f2_fma(f2_pack(y[2], y[3]), f2_pack(rs.z, rs.w), l2);
              if constexpr (MODE == 2) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const float rv = cols.rv[col + k];
                  if (rv != 0.0f && y[k] != 0.0f) zs = fmaf(y[k], rv, zs);       // (NaN for a scale that is none)
                }
              }
              const __half2 h0 = __floats2half2_rn(y[0], y[1]), h1 = __floats2half2_rn(y[2], y[3]);
              w[i / 2] = *reinterpret_cast<const uint32_t*>(&h0);
              w[i / 2 + 1] = *reinterpret_cast<const uint32_t*>(&h1);
            }
            tmem_st_32x32b_x16(s_at + 16 * ch, w);         // over columns that have been read
            return true;
          };
          auto step_of = [&](auto mode) -> bool {
            uint32_t s[32];
            tmem_ld_32x32b_x32(s_at, s);
            tmem_ld_wait();
            if (!chunk(mode, s, 0)) return false;
            tmem_ld_32x32b_x32(s_at + 32, s);
            tmem_ld_wait();
            return chunk(mode, s, 1);
          };
          ok = plain ? step_of(std::integral_constant<int, 0>{})
                     : rest ? step_of(std::integral_constant<int, 2>{}) : step_of(std::integral_constant<int, 1>{});
          if (!ok) break;
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(&bars[kPFull + 2 * t + place]);
        }
        if (ok) ok = wait_warp(kODone + 2 * t + 1, n.tile_steps[t] + it.take - 1, kDevTimeoutEpilogue);
        if (!ok) break;
        tc_fence_after();
        float l, l1;
        f2_unpack(l2, l, l1);
        l += l1;
        // an item of several chains: what the ones before it left is added.  A chain that saw no key (l = 0) has no m
        const bool add = it.unit > run_unit;
        const bool last = done + it.take == run_end;
        const bool whole = run_unit == 0 && it.unit + it.take == it.units;
        float f0 = 0.0f, f1 = 1.0f;
        if (add) {
          const float top = fmaxf(run_l != 0.0f ? run_m : -INFINITY, l != 0.0f ? m : -INFINITY);
          f0 = run_l == 0.0f ? 0.0f : run_m == top ? 1.0f : exp2_fast(run_m - top);
          f1 = l == 0.0f ? 0.0f : m == top ? 1.0f : exp2_fast(m - top);
          m = top;
          l = fmaf(run_l, f0, l * f1);
        }
        run_m = m;
        run_l = l;
        const int64_t token = it.rows.first + tok, part = part_at(a, blockIdx.x, run_slot, 0, r);
        if (last && whole) {
          const float inv = inverse_or_zero(l);
          f0 *= inv;
          f1 *= inv;
        }
        __half* out = a.out + token * a.ldo + qh * D;
#pragma unroll 1
        for (int ch = 0; ch < D / 32; ++ch) {
          uint32_t o[32];
          tmem_ld_32x32b_x32(o_at + 32 * ch, o);
          tmem_ld_wait();
          if (ch == D / 32 - 1) {                          // O may be written again
            tc_fence_before();
            mbar_arrive(&bars[kORead + t]);
          }
          if (!has) continue;
          // columns of a chunk of 8 hold elements 0 4 1 5 2 6 3 7
          float y[32];
#pragma unroll
          for (int i = 0; i < 32; ++i)
            y[i] = (__uint_as_float(o[(i & 24) + ((i & 3) << 1) + ((i >> 2) & 1)]) - zs) * f1;
          float4* sums = reinterpret_cast<float4*>(a.part_o + part * D + 32 * ch);
          if (add) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 x = sums[i];
              y[4 * i] = fmaf(x.x, f0, y[4 * i]);
              y[4 * i + 1] = fmaf(x.y, f0, y[4 * i + 1]);
              y[4 * i + 2] = fmaf(x.z, f0, y[4 * i + 2]);
              y[4 * i + 3] = fmaf(x.w, f0, y[4 * i + 3]);
            }
          }
          if (last && whole) {
            store_half<32>(out + 32 * ch, y);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) sums[i] = make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
          }
        }
        if (has && last) {
          if (!whole) a.part_ml[part] = make_float2(m, l);
          else if (a.lse != nullptr) a.lse[token * a.q_heads + qh] = row_lse(m, l);
        }
      }
      n.next(it.take, tiles);
      done += it.take;
    }
  } else if (warp < 12) {
    // --------------------------------------------------- queries, keys, values
    const int tok = tid - 2 * kSoftmaxThreads;
    constexpr int W = P::kWords;
    const int64_t row_bytes = v.width >> 1;
    for (int32_t done = 0; done < count && ok;) {
      const Item it = find_item(v, a.plan, prefix, start + done, min(count - done, kChain), &b);
      const int tiles = tiles_of(it);
      const int head = it.block;
      // one token a thread: its key's codes are loaded a step ahead, its value's while the key is unpacked
      const int at = head * (D / 2);
      const uint32_t group = head * D / v.group;
      auto slot_of = [&](int32_t j) -> int64_t {
        const int32_t t = (it.unit + j) * kKeys + tok;
        return j < it.take && t < it.seen ? kv_slot(v, v.table, b, t) : -1;
      };
      auto load = [&](int side, int64_t slot, uint32_t (&x)[W]) {
        if (v.pages == 0) return;                          // nothing is held, and nothing may be read
        const uint4* from = reinterpret_cast<const uint4*>((side ? v.codes[1] : v.codes[0]) +
                                                           max(slot, static_cast<int64_t>(0)) * row_bytes + at);
#pragma unroll
        for (int i = 0; i < W / 4; ++i) {
          const uint4 y = from[i];
          x[4 * i] = y.x;
          x[4 * i + 1] = y.y;
          x[4 * i + 2] = y.z;
          x[4 * i + 3] = y.w;
        }
      };
      struct Numbers {
        float sk, sv;
        int32_t zk, zv;
      };
      auto numbers = [&](int64_t slot) {
        Numbers x{};
        if (v.pages > 0) {
          const uint32_t g = static_cast<uint32_t>(max(slot, static_cast<int64_t>(0))) * v.groups + group;
          x.sk = v.scales[0][g];
          x.zk = v.zeros[0][g];
          x.sv = v.scales[1][g];
          x.zv = v.zeros[1][g];
        }
        return x;
      };
      auto unpack = [&](const uint32_t (&w)[W], int32_t z, bool blank, uint8_t* tile) {
        const __half2 c1 = __half2half2(__int2half_rn(-1032 - z)), c0 = __half2half2(__int2half_rn(-72 - z));
        const uint32_t z1024 = *reinterpret_cast<const uint32_t*>(&c1), z64 = *reinterpret_cast<const uint32_t*>(&c0);
#pragma unroll
        for (int i = 0; i < W; ++i) {
          const uint32_t x = w[i], y = x >> 8;
          uint4 e = make_uint4(add_half2(nib_1024(x), z1024), add_half2(nib_64(x), z64),
                               add_half2(nib_1024(y), z1024), add_half2(nib_64(y), z64));
          if (blank) e = make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4*>(tile + tile_at(tok, i)) = e;
        }
      };
      uint32_t kw[W] = {}, vw[W] = {};
      int64_t slot = slot_of(0), next = slot_of(1);
      load(0, slot, kw);
      Numbers num = numbers(slot);
      // queries: row tok of each tile; elements of a chunk in the order 0 4 1 5 2 6 3 7.  Those of the item before
      // have met their last keys.
      if (n.items > 0) ok = wait_warp(kQFree, n.items - 1, kDevTimeoutProducer);
      if (!ok) break;
      for (int t = 0; t < tiles; ++t) {
        const int32_t rr = it.tile * a.plan.rows + 128 * t + tok;
        const __half* from = rr < it.rows.here * a.plan.gq
                                 ? a.q + (it.rows.first + rr / a.plan.gq) * a.ldq +
                                       static_cast<int64_t>(head * a.plan.gq + rr % a.plan.gq) * D
                                 : nullptr;
#pragma unroll 8
        for (int chunk = 0; chunk < D / 8; ++chunk) {
          uint4 x = make_uint4(0, 0, 0, 0);
          if (from != nullptr) x = *reinterpret_cast<const uint4*>(from + chunk * 8);
          *reinterpret_cast<uint4*>(q_tile + t * P::kTile + tile_at(tok, chunk)) =
              make_uint4(byte_perm(x.x, x.z, 0x5410), byte_perm(x.x, x.z, 0x7632), byte_perm(x.y, x.w, 0x5410),
                         byte_perm(x.y, x.w, 0x7632));
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(&bars[kQFull]);
      for (int32_t j = 0; j < it.take; ++j) {
        const uint32_t step = n.steps + j;
        const int st = step % P::kStages;
        load(1, slot, vw);
        const int64_t after = slot_of(j + 2);
        if (step >= P::kStages) ok = wait_warp(kFree + st, step / P::kStages - 1, kDevTimeoutProducer);
        if (!ok) break;
        uint8_t* kt = kv_tile + st * P::kStage;
        uint8_t* vt = kt + P::kTile;
        const bool is = slot >= 0;
        const int32_t zk = min(max(num.zk, -900), 900), zv = min(max(num.zv, -900), 900);
        const bool none = !(num.sv <= 0x1p40f), zero = num.sv < 0x1p-40f;
        {
          const Cols cols(cols_at + st * P::kCols);
          const float lv = fminf(fmaxf(__log2f(num.sv), -40.0f), 40.0f);
          const float rv = none ? NAN : zero ? 0.0f : static_cast<float>(static_cast<int64_t>(num.zv) - zv);
          const float rk = static_cast<float>(static_cast<int64_t>(num.zk) - zk);
          cols.sk[tok] = is ? num.sk * a.scale_log2 : 0.0f;
          cols.lv[tok] = is ? lv : -INFINITY;
          cols.rsv[tok] = is ? exp2_fast(-lv) : 0.0f;
          cols.rk[tok] = is ? rk : 0.0f;
          cols.rv[tok] = is ? rv : 0.0f;
          const bool any = __any_sync(0xffffffffu, is && (rk != 0.0f || rv != 0.0f));
          if (lane == 0) cols.rest[tok >> 5] = any;
        }
        unpack(kw, zk, false, kt);
        fence_proxy_async_smem();
        mbar_arrive(&bars[kKFull + st]);
        if (j + 1 < it.take) {
          load(0, next, kw);
          num = numbers(next);
        }
        unpack(vw, zv, zero || !is, vt);
        fence_proxy_async_smem();
        mbar_arrive(&bars[kVFull + st]);
        slot = next;
        next = after;
      }
      n.next(it.take, tiles);
      done += it.take;
    }
  } else {
    // -------------------------------------------------------------- MMA issue
    constexpr uint32_t kIdescS = idesc_f16(64);
    constexpr uint32_t kIdescO = idesc_f16(D) | (1u << 16);            // B with N contiguous
    const uint32_t q0 = smem_u32(q_tile), kv0 = smem_u32(kv_tile);
    for (int32_t done = 0; done < count && ok;) {
      const Item it = find_item(v, a.plan, prefix, start + done, min(count - done, kChain), &b);
      const int tiles = tiles_of(it);
      if (lane == 0) {
        // scores of tile t with 64 keys: half `place` of stage st
        auto scores = [&](int t, int st, int place) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t off = (k >> 2) * 16384 + (k & 3) * 32;
            mma_f16(tmem + 128 * t + 64 * place, smem_desc_kmajor(q0 + t * P::kTile + off, 128),
                    smem_desc_kmajor(kv0 + st * P::kStage + off + place * 8192, 128), kIdescS, k > 0);
          }
          mma_commit(&bars[kSFull + 2 * t + place]);
        };
        auto wait_keys = [&](uint32_t step) {
          const bool there = wait(kKFull + step % P::kStages, step / P::kStages, kDevTimeoutMma);
          if (there) tc_fence_after();
          return there;
        };
        ok = wait(kQFull, n.items, kDevTimeoutMma) && wait_keys(n.steps);
        for (int place = 0; place < 2 && ok; ++place)
          for (int t = 0; t < tiles; ++t) scores(t, n.steps % P::kStages, place);
        if (ok && it.take == 1) mma_commit(&bars[kQFree]);
        for (int32_t j = 0; j < 2 * it.take && ok; ++j) {
          const uint32_t step = n.steps + (j >> 1);
          const int st = step % P::kStages, place = j & 1;
          if (place == 0) ok = wait(kVFull + st, step / P::kStages, kDevTimeoutMma);
          for (int t = 0; t < tiles && ok; ++t) {
            ok = wait(kPFull + 2 * t + place, n.tile_steps[t] + (j >> 1), kDevTimeoutMma);
            // the outputs of the item before have been read
            if (ok && j == 0 && n.tile_items[t] > 0) ok = wait(kORead + t, n.tile_items[t] - 1, kDevTimeoutMma);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int s = 0; s < 4; ++s)
              mma_f16_ts(tmem + 256 + t * D, tmem + 128 * t + 64 * place + 8 * s,
                         smem_desc_mn_sw128(kv0 + st * P::kStage + P::kTile + 2048 * (4 * place + s), 16384), kIdescO,
                         j > 0 || s > 0);
            mma_commit(&bars[kODone + 2 * t + place]);
            if (t == tiles - 1 && place == 1) mma_commit(&bars[kFree + st]);
            // the same half of the next keys, into the place that these products have left (with one stage, both
            // halves when the stage is free)
            const bool more = j + 2 < 2 * it.take + (P::kStages == 1 ? 1 : 0);
            if (more && (P::kStages > 1 || place == 1)) {
              if (t == 0 && (P::kStages == 1 || place == 0) && !(ok = wait_keys(step + 1))) break;
              if (P::kStages == 1) scores(t, 0, 0);
              scores(t, (step + 1) % P::kStages, place);
              if (t == tiles - 1 && place == 1 && (j >> 1) + 2 == it.take) mma_commit(&bars[kQFree]);
            }
          }
        }
      }
      ok = __all_sync(0xffffffffu, ok);
      n.next(it.take, tiles);
      done += it.take;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 12) tmem_dealloc(tmem, 512);
}

template <int D>
cudaError_t run_prefill(const SplitArgs& a, cudaStream_t stream) {
  const int smem = Shape<D>::kBytes + 1024 + (a.v.batch + 1) * static_cast<int>(sizeof(int64_t));
  static std::atomic<uint64_t> done{0};
  constexpr int kMost = Shape<D>::kBytes + 1024 + (kMaxBatch + 1) * 8;
  const cudaError_t e = allow_smem(kv_prefill_kernel<D>, kMost, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(kv_prefill_kernel<D>, dim3(a.plan.blocks), dim3(kThreadsP), smem, stream, 1, a,
                    device_status_word());
}

}  // namespace

bool kv_prefill_takes(const KvView& v) { return v.batch <= kMaxBatch; }
int kv_prefill_rows(int head_dim) { return head_dim == 256 ? 128 : 256; }

cudaError_t launch_kv_prefill(const SplitArgs& a, cudaStream_t stream) {
  switch (a.v.head_dim) {
    case 32: return run_prefill<32>(a, stream);
    case 64: return run_prefill<64>(a, stream);
    case 128: return run_prefill<128>(a, stream);
    default: return run_prefill<256>(a, stream);
  }
}

}  // namespace qr
