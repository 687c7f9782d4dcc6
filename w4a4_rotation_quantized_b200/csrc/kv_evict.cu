// kv_evict.cu -- eviction from the paged 4-bit KV cache by accumulated attention
// weight: the choice of the tokens that stay, and their move.
//
// Choice (one block per sequence and group): of the n - recent older tokens the k = keep - recent with the largest
// mass.  A radix select over the order-preserving 32-bit keys finds the k-th largest key in four passes of 8 bits
// (counts in 256 x 8 bins, a column for every eighth lane, so that lanes that meet the same digit seldom meet
// the same address); a last pass writes, in order, the places whose key is above it, and of those equal to it
// the first, and moves the mass along.  Keys that fit stay in shared memory between the passes.  Everything is
// counted, nothing depends on the order in which threads run.
//
// Move: place j receives what was at kept[j] >= j.  Into other pages a block takes some places with all groups,
// whose rows lie side by side there: whole lines are written, and where groups keep the same token whole sectors
// of scales and zeros are read.  In place one block takes a (sequence, group, array) and goes up in pieces, each
// read whole before any of it is written: a piece's destinations lie at or below its own sources and below all
// later ones.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "kv_device.cuh"
#include "qr_internal.h"

namespace qr {

namespace {

constexpr int kFewTokens = 8192;                   // up to here 256 threads choose (several blocks an SM), else 1024
constexpr int kSelectUnroll = 4;
constexpr int kMoveThreads = 256;
constexpr int kMoveUnroll = 8;

// Orders like the float it comes from; NaN like -inf, -0 like +0.
__device__ __forceinline__ uint32_t mass_key(float x) {
  if (!(x > -INFINITY)) x = -INFINITY;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

constexpr int kColumns = 8;
constexpr int kKeysHeld = 40960;                   // in shared memory

template <int kSelectThreads>
__global__ void __launch_bounds__(kSelectThreads) kv_select_kernel(KvView v, const float* mass,
                                                                   float* mass_out, int64_t ld_mass,
                                                                   int32_t keep, int32_t recent,
                                                                   int32_t* kept, int32_t* lens_out,
                                                                   int32_t held) {
  grid_dep_wait();
  grid_dep_launch();
  constexpr int kSelectWarps = kSelectThreads / 32;
  extern __shared__ uint32_t keys[];               // [held]
  __shared__ uint32_t hist[256][kColumns];
  __shared__ uint32_t total[256];
  __shared__ uint32_t chosen[2];                  // the digit, and how many of its keys are still wanted
  __shared__ uint32_t warp_gt[kSelectWarps], warp_eq[kSelectWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t b = blockIdx.x, j = blockIdx.y;
  const int32_t n = kv_len(v, b), count = min(n, keep);
  const int64_t row = static_cast<int64_t>(b) * v.groups + j;
  const float* m = mass + row * ld_mass;
  float* m_out = mass_out + row * ld_mass;
  int32_t* to = kept + row * keep;
  if (j == 0 && tid == 0) lens_out[b] = count;
  const int32_t old = n > keep ? n - recent : 0;  // > keep - recent >= 0 where there is a choice
  const uint32_t want = n > keep ? static_cast<uint32_t>(keep - recent) : 0;
  uint32_t prefix = 0, left = want;               // keys with a larger prefix are all in
  if (want > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int e = tid; e < 256 * kColumns; e += kSelectThreads) (&hist[0][0])[e] = 0;
      __syncthreads();
      auto bin = [&](uint32_t k) {
        if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8)))
          atomicAdd(&hist[(k >> shift) & 255][lane % kColumns], 1u);
      };
      if (shift == 24) {
#pragma unroll 4
        for (int32_t t = tid; t < old; t += kSelectThreads) {
          const uint32_t k = mass_key(m[t]);
          if (t < held) keys[t] = k;
          bin(k);
        }
      } else {
#pragma unroll 4
        for (int32_t t = tid; t < min(old, held); t += kSelectThreads) bin(keys[t]);
#pragma unroll 4
        for (int32_t t = held + tid; t < old; t += kSelectThreads) bin(mass_key(m[t]));
      }
      __syncthreads();
      if (tid < 256) {
        uint32_t c = 0;
#pragma unroll
        for (int e = 0; e < kColumns; ++e) c += hist[tid][(e + tid) % kColumns];
        total[tid] = c;
      }
      __syncthreads();
      if (warp == 0) {                            // 8 digits a lane, from the top
        uint32_t own = 0;
        for (int e = 0; e < 8; ++e) own += total[255 - (lane * 8 + e)];
        uint32_t before = own;
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t x = __shfl_up_sync(0xffffffffu, before, o);
          if (lane >= o) before += x;
        }
        before -= own;
        if (before < left && before + own >= left) {
          for (int e = 0; e < 8; ++e) {
            const uint32_t c = total[255 - (lane * 8 + e)];
            if (before + c >= left) {
              chosen[0] = 255 - (lane * 8 + e);
              chosen[1] = left - before;
              break;
            }
            before += c;
          }
        }
      }
      __syncthreads();
      prefix |= chosen[0] << shift;
      left = chosen[1];
      __syncthreads();
    }
  }
  // `left` keys equal to prefix are wanted, the first ones; all above it are in.  A round's masses are read before its
  // places, none above its own, are written.
  int32_t at = 0;
  uint32_t eq_seen = 0;
  for (int32_t base = 0; base < old && want > 0; base += kSelectThreads * kSelectUnroll) {
    uint32_t gt[kSelectUnroll], eq[kSelectUnroll], ngt = 0, neq = 0;
    float x[kSelectUnroll];
#pragma unroll
    for (int u = 0; u < kSelectUnroll; ++u) {
      const int32_t t = base + (warp * kSelectUnroll + u) * 32 + lane;
      x[u] = t < old ? m[t] : 0.0f;
    }
#pragma unroll
    for (int u = 0; u < kSelectUnroll; ++u) {
      const int32_t t = base + (warp * kSelectUnroll + u) * 32 + lane;
      const uint32_t k = mass_key(x[u]);
      gt[u] = __ballot_sync(0xffffffffu, t < old && k > prefix);
      eq[u] = __ballot_sync(0xffffffffu, t < old && k == prefix);
      ngt += __popc(gt[u]);
      neq += __popc(eq[u]);
    }
    if (lane == 0) {
      warp_gt[warp] = ngt;
      warp_eq[warp] = neq;
    }
    __syncthreads();
    uint32_t g0 = lane < kSelectWarps ? warp_gt[lane] : 0u, e0 = lane < kSelectWarps ? warp_eq[lane] : 0u;   // one warp a lane
    const uint32_t all_gt = __reduce_add_sync(0xffffffffu, g0), all_eq = __reduce_add_sync(0xffffffffu, e0);
    g0 = __reduce_add_sync(0xffffffffu, lane < warp ? g0 : 0u);
    e0 = __reduce_add_sync(0xffffffffu, lane < warp ? e0 : 0u) + eq_seen;
#pragma unroll
    for (int u = 0; u < kSelectUnroll; ++u) {
      const int32_t t = base + (warp * kSelectUnroll + u) * 32 + lane;
      const uint32_t below = (1u << lane) - 1;
      const uint32_t rank_eq = e0 + __popc(eq[u] & below);
      // place: the larger keys before it, and the equal ones among the first `left`
      const uint32_t place = at + g0 + __popc(gt[u] & below) + min(rank_eq, left) - min(eq_seen, left);
      const bool in = ((gt[u] >> lane) & 1u) || (((eq[u] >> lane) & 1u) && rank_eq < left);
      if (in) {
        to[place] = t;
        m_out[place] = x[u];
      }
      g0 += __popc(gt[u]);
      e0 += __popc(eq[u]);
    }
    at += all_gt + min(eq_seen + all_eq, left) - min(eq_seen, left);
    eq_seen += all_eq;
    __syncthreads();
  }
  // the newest behind them (all, where there is no choice), nothing from there on
  const int32_t first = static_cast<int32_t>(want), from = n > keep ? old : 0;
  for (int32_t t0 = 0; t0 < count - first; t0 += kSelectThreads) {
    const int32_t t = t0 + tid;
    const float x = t < count - first ? m[from + t] : 0.0f;
    __syncthreads();
    if (t < count - first) {
      to[first + t] = from + t;
      m_out[first + t] = x;
    }
    __syncthreads();
  }
  for (int32_t t = count + tid; t < keep; t += kSelectThreads) to[t] = -1;
  for (int64_t t = count + tid; t < ld_mass; t += kSelectThreads) m_out[t] = 0.0f;
}

struct MoveArgs {
  KvView v;
  const int32_t* table_out;
  const int32_t* kept;
  int32_t keep;
  int32_t units;              // 16-byte units of a group's codes: group / 32
};

constexpr int kMovePlaces = 16;               // places of a block, into other pages

// Into other pages.  grid: (places, sequences)
__global__ void __launch_bounds__(kMoveThreads) kv_move_out_kernel(MoveArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  const KvView& v = a.v;
  const int32_t b = blockIdx.y, j0 = blockIdx.x * kMovePlaces;
  const int32_t count = min(kv_len(v, b), a.keep), here = min(count - j0, kMovePlaces);
  if (here <= 0) return;
  extern __shared__ int32_t src[];             // [place][group]: the slot that a place's group comes from, or -1
  __shared__ int32_t dst[kMovePlaces];
  for (int e = threadIdx.x; e < here * v.groups; e += kMoveThreads) {
    const int g = e / here, p = e - g * here;  // neighbouring places of a group lie side by side in kept
    const int32_t from = a.kept[(static_cast<int64_t>(b) * v.groups + g) * a.keep + j0 + p];
    src[p * v.groups + g] = from < 0 ? -1 : static_cast<int32_t>(kv_slot(v, v.table, b, from));
  }
  if (threadIdx.x < here) dst[threadIdx.x] = static_cast<int32_t>(kv_slot(v, a.table_out, b, j0 + threadIdx.x));
  __syncthreads();
  const uint32_t row = static_cast<uint32_t>(v.groups) * a.units;      // 16-byte units of a row of codes
  const uint32_t all = here * row;
  const uint4* from[2] = {reinterpret_cast<const uint4*>(v.codes[0]), reinterpret_cast<const uint4*>(v.codes[1])};
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    const uint4* codes = from[side];
    uint4* to = const_cast<uint4*>(codes);
    for (uint32_t e0 = threadIdx.x; e0 < all; e0 += kMoveThreads * kMoveUnroll) {
      uint4 x[kMoveUnroll];
      int64_t at[kMoveUnroll];
#pragma unroll
      for (int u = 0; u < kMoveUnroll; ++u) {
        const uint32_t e = e0 + u * kMoveThreads;
        at[u] = -1;
        if (e < all) {
          const uint32_t p = e / row, in = e - p * row;
          const int32_t s = src[p * v.groups + in / a.units], d = dst[p];
          if (s >= 0 && d >= 0) {
            x[u] = codes[static_cast<int64_t>(s) * row + in];
            at[u] = static_cast<int64_t>(d) * row + in;
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kMoveUnroll; ++u)
        if (at[u] >= 0) to[at[u]] = x[u];
    }
  }
  for (int e = threadIdx.x; e < here * v.groups; e += kMoveThreads) {
    const int p = e / v.groups, g = e - p * v.groups;
    const int32_t s = src[e], d = dst[p];
    if (s < 0 || d < 0) continue;
    const int64_t f = static_cast<int64_t>(s) * v.groups + g, t = static_cast<int64_t>(d) * v.groups + g;
    const float s0 = v.scales[0][f], s1 = v.scales[1][f];
    const int32_t z0 = v.zeros[0][f], z1 = v.zeros[1][f];
    v.scales[0][t] = s0;
    v.scales[1][t] = s1;
    v.zeros[0][t] = z0;
    v.zeros[1][t] = z1;
  }
}

// In place: a piece of kMoveThreads * kMoveUnroll elements of one array of a (sequence, group): codes go in 16-byte
// units, several to a row; scales and zeros in 4-byte ones.
template <bool CODES>
__device__ __forceinline__ void move_piece(const MoveArgs& a, int array, int32_t b, int32_t j, int32_t count,
                                           int64_t first) {
  using T = typename std::conditional<CODES, uint4, uint32_t>::type;
  const KvView& v = a.v;
  const int per = CODES ? a.units : 1;
  const int64_t all = static_cast<int64_t>(count) * per;
  uint8_t* p = array == 0   ? v.codes[0]
               : array == 1 ? v.codes[1]
               : array == 2 ? reinterpret_cast<uint8_t*>(v.scales[0])
               : array == 3 ? reinterpret_cast<uint8_t*>(v.scales[1])
               : array == 4 ? reinterpret_cast<uint8_t*>(v.zeros[0])
                            : reinterpret_cast<uint8_t*>(v.zeros[1]);
  T x[kMoveUnroll];
  T* dst[kMoveUnroll];
#pragma unroll
  for (int u = 0; u < kMoveUnroll; ++u) {
    const int64_t e = first + u * kMoveThreads + threadIdx.x;
    dst[u] = nullptr;
    if (e < all) {
      const int32_t to = static_cast<int32_t>(e / per), part = static_cast<int32_t>(e % per);
      const int32_t from = a.kept[(static_cast<int64_t>(b) * v.groups + j) * a.keep + to];
      if (from >= 0 && from != to) {
        const int64_t s0 = kv_slot(v, v.table, b, from), s1 = kv_slot(v, v.table, b, to);
        if (s0 >= 0 && s1 >= 0) {
          x[u] = reinterpret_cast<const T*>(p)[(s0 * v.groups + j) * per + part];
          dst[u] = reinterpret_cast<T*>(p) + (s1 * v.groups + j) * per + part;
        }
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < kMoveUnroll; ++u)
    if (dst[u] != nullptr) *dst[u] = x[u];
  __syncthreads();
}

// grid: (sequence, group, array).  Arrays 0, 1: codes; 2, 3: scales; 4, 5: zeros.
__global__ void __launch_bounds__(kMoveThreads) kv_move_kernel(MoveArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  const int32_t b = blockIdx.x, j = blockIdx.y;
  const int array = blockIdx.z;
  const int32_t n = kv_len(a.v, b);
  if (n <= a.keep) return;
  const int64_t all = static_cast<int64_t>(a.keep) * (array < 2 ? a.units : 1);
  for (int64_t first = 0; first < all; first += kMoveThreads * kMoveUnroll) {
    if (array < 2) move_piece<true>(a, array, b, j, a.keep, first);
    else move_piece<false>(a, array, b, j, a.keep, first);
  }
}

}  // namespace

qr_status launch_kv_evict(const KvView& v, const KvEvictJob& j, cudaStream_t stream) {
  const int32_t held = std::min(v.capacity, kKeysHeld);
  cudaError_t e;
  if (v.capacity <= kFewTokens) {
    e = launch_pdl(kv_select_kernel<256>, dim3(v.batch, v.groups), dim3(256), static_cast<size_t>(held) * 4, stream, 1, v,
                   j.mass, j.mass_out, j.ld_mass, j.keep, j.recent, j.kept, j.lens_out, held);
  } else {
    static std::atomic<uint64_t> done{0};
    e = allow_smem(kv_select_kernel<1024>, kKeysHeld * 4, done);
    if (e == cudaSuccess)
      e = launch_pdl(kv_select_kernel<1024>, dim3(v.batch, v.groups), dim3(1024), static_cast<size_t>(held) * 4, stream,
                     1, v, j.mass, j.mass_out, j.ld_mass, j.keep, j.recent, j.kept, j.lens_out, held);
  }
  if (e != cudaSuccess) return QR_ERR_CUDA;
  MoveArgs a{};
  a.v = v;
  a.table_out = j.table_out;
  a.kept = j.kept;
  a.keep = j.keep;
  a.units = v.group / 32;
  const int32_t most = std::min(j.keep, v.capacity);
  if (j.table_out == nullptr)
    e = launch_pdl(kv_move_kernel, dim3(v.batch, v.groups, 6), dim3(kMoveThreads), 0, stream, 1, a);
  else if (most > 0)
    e = launch_pdl(kv_move_out_kernel, dim3((most + kMovePlaces - 1) / kMovePlaces, v.batch), dim3(kMoveThreads),
                   static_cast<size_t>(kMovePlaces) * v.groups * 4, stream, 1, a);
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? QR_OK : QR_ERR_CUDA;
}

}  // namespace qr
