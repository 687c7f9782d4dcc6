// kv_evict.cu -- eviction from the paged 4-bit KV cache by accumulated attention
// weight: the choice of the tokens that stay, and their move.
//
// Choice (one block per sequence and group): of the n - recent older tokens the k =
// keep - recent with the largest mass.  A radix select over the order-preserving
// 32-bit keys finds the k-th largest key in four passes of 8 bits (counts in
// 256 x 32 bins, one column a lane, so that lanes that meet the same digit do not
// meet the same address); a last pass writes, in order, the places whose key is above it,
// and of those equal to it the first.  Everything is counted, nothing depends on the order in
// which threads run.
//
// Move: place j receives what was at kept[j] >= j.  Into other pages every piece moves
// on its own.  In place one block takes a (sequence, group, array) and goes up in
// pieces, each read whole before any of it is written: a piece's destinations lie at or below its
// own sources and below all later ones.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "kv_device.cuh"
#include "qr_internal.h"

namespace qr {

namespace {

constexpr int kSelectThreads = 1024;
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kSelectUnroll = 4;
constexpr int kMoveThreads = 256;
constexpr int kMoveUnroll = 8;

// Orders like the float it comes from; NaN like -inf, -0 like +0.
__device__ __forceinline__ uint32_t mass_key(float x) {
  if (!(x > -INFINITY)) x = -INFINITY;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kSelectThreads) kv_select_kernel(KvView v, const float* mass,
                                                                   int64_t ld_mass, int32_t keep,
                                                                   int32_t recent, int32_t* kept,
                                                                   int32_t* lens_out) {
  grid_dep_wait();
  grid_dep_launch();
  __shared__ uint32_t hist[256][32];
  __shared__ uint32_t total[256];
  __shared__ uint32_t chosen[2];                  // the digit, and how many of its keys are still wanted
  __shared__ uint32_t warp_gt[kSelectWarps], warp_eq[kSelectWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t b = blockIdx.x, j = blockIdx.y;
  const int32_t n = kv_len(v, b);
  const int64_t row = static_cast<int64_t>(b) * v.groups + j;
  const float* m = mass + row * ld_mass;
  int32_t* to = kept + row * keep;
  if (j == 0 && tid == 0) lens_out[b] = min(n, keep);
  if (n <= keep) {
    for (int32_t t = tid; t < keep; t += kSelectThreads) to[t] = t < n ? t : -1;
    return;
  }
  const int32_t old = n - recent;                 // > keep - recent >= 0
  const uint32_t want = static_cast<uint32_t>(keep - recent);
  uint32_t prefix = 0, left = want;               // keys with a larger prefix are all in
  if (want > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int e = tid; e < 256 * 32; e += kSelectThreads) (&hist[0][0])[e] = 0;
      __syncthreads();
      for (int32_t t = tid; t < old; t += kSelectThreads) {
        const uint32_t k = mass_key(m[t]);
        if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8)))
          atomicAdd(&hist[(k >> shift) & 255][lane], 1u);
      }
      __syncthreads();
      for (int dgt = warp; dgt < 256; dgt += kSelectWarps) {
        const uint32_t c = __reduce_add_sync(0xffffffffu, hist[dgt][lane]);
        if (lane == 0) total[dgt] = c;
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
  // `left` keys equal to prefix are wanted, the first ones; all above it are in
  int32_t at = 0;
  uint32_t eq_seen = 0;
  for (int32_t base = 0; base < old && want > 0; base += kSelectThreads * kSelectUnroll) {
    uint32_t gt[kSelectUnroll], eq[kSelectUnroll], ngt = 0, neq = 0;
#pragma unroll
    for (int u = 0; u < kSelectUnroll; ++u) {
      const int32_t t = base + (warp * kSelectUnroll + u) * 32 + lane;
      const uint32_t k = t < old ? mass_key(m[t]) : 0u;
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
    uint32_t g0 = warp_gt[lane], e0 = warp_eq[lane];          // one warp a lane
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
      if (in) to[place] = t;
      g0 += __popc(gt[u]);
      e0 += __popc(eq[u]);
    }
    at += all_gt + min(eq_seen + all_eq, left) - min(eq_seen, left);
    eq_seen += all_eq;
    __syncthreads();
  }
  for (int32_t t = tid; t < recent; t += kSelectThreads) to[keep - recent + t] = old + t;
}

struct MoveArgs {
  KvView v;
  const int32_t* table_out;
  const float* mass;
  float* mass_out;
  int64_t ld_mass;
  const int32_t* kept;
  int32_t keep;
  int32_t units;              // 16-byte units of a group's codes: group / 32
};

// A piece of kMoveThreads * kMoveUnroll elements of one array of a (sequence, group):
// codes go in 16-byte units, several to a row; scales, zeros and mass in 4-byte ones.
template <bool CODES>
__device__ __forceinline__ void move_piece(const MoveArgs& a, int array, int32_t b, int32_t j,
                                           int32_t count, int64_t first, bool in_place) {
  using T = typename std::conditional<CODES, uint4, uint32_t>::type;
  const KvView& v = a.v;
  const int64_t row = static_cast<int64_t>(b) * v.groups + j;
  const int per = CODES ? a.units : 1;
  const int64_t all = static_cast<int64_t>(count) * per;
  T x[kMoveUnroll];
  T* dst[kMoveUnroll];
#pragma unroll
  for (int u = 0; u < kMoveUnroll; ++u) {
    const int64_t e = first + u * kMoveThreads + threadIdx.x;
    dst[u] = nullptr;
    if (e < all) {
      const int32_t to = static_cast<int32_t>(e / per), part = static_cast<int32_t>(e % per);
      const int32_t from = a.kept[row * a.keep + to];
      if (from >= 0 && !(in_place && from == to)) {
        if (array == 6) {
          x[u] = *reinterpret_cast<const T*>(a.mass + row * a.ld_mass + from);
          dst[u] = reinterpret_cast<T*>(a.mass_out + row * a.ld_mass + to);
        } else {
          const int64_t s0 = kv_slot(v, v.table, b, from);
          const int64_t s1 = kv_slot(v, in_place ? v.table : a.table_out, b, to);
          if (s0 >= 0 && s1 >= 0) {
            uint8_t* p = CODES ? v.codes[array]
                               : array < 4 ? reinterpret_cast<uint8_t*>(v.scales[array - 2])
                                           : reinterpret_cast<uint8_t*>(v.zeros[array - 4]);
            x[u] = reinterpret_cast<const T*>(p)[(s0 * v.groups + j) * per + part];
            dst[u] = reinterpret_cast<T*>(p) + (s1 * v.groups + j) * per + part;
          }
        }
      }
    }
  }
  if (in_place) __syncthreads();
#pragma unroll
  for (int u = 0; u < kMoveUnroll; ++u)
    if (dst[u] != nullptr) *dst[u] = x[u];
  if (in_place) __syncthreads();
}

// grid: (sequence, group, array x pieces).  Arrays 0, 1: codes; 2, 3: scales; 4, 5: zeros; 6: mass.
__global__ void __launch_bounds__(kMoveThreads) kv_move_kernel(MoveArgs a, int pieces) {
  grid_dep_wait();
  grid_dep_launch();
  const KvView& v = a.v;
  const int32_t b = blockIdx.x, j = blockIdx.y;
  const int array = blockIdx.z / pieces, piece = blockIdx.z % pieces;
  const int32_t n = kv_len(v, b), count = min(n, a.keep);
  const bool in_place = array == 6 ? a.mass_out == a.mass : a.table_out == nullptr;
  const int64_t all = static_cast<int64_t>(count) * (array < 2 ? a.units : 1);
  constexpr int64_t kPiece = kMoveThreads * kMoveUnroll;
  // in place the first block takes all pieces, one after the other
  if (in_place && piece != 0) return;
  const int64_t step = in_place ? kPiece : kPiece * pieces;
  for (int64_t first = piece * kPiece; first < all; first += step) {
    if (array < 2) move_piece<true>(a, array, b, j, count, first, in_place);
    else move_piece<false>(a, array, b, j, count, first, in_place);
  }
  if (array == 6) {
    float* row = a.mass_out + (static_cast<int64_t>(b) * v.groups + j) * a.ld_mass;
    for (int64_t t = count + static_cast<int64_t>(piece) * kMoveThreads + threadIdx.x; t < a.ld_mass;
         t += in_place ? kMoveThreads : kMoveThreads * pieces)
      row[t] = 0.0f;
  }
}

}  // namespace

qr_status launch_kv_evict(const KvView& v, const KvEvictJob& j, cudaStream_t stream) {
  cudaError_t e = launch_pdl(kv_select_kernel, dim3(v.batch, v.groups), dim3(kSelectThreads), 0,
                             stream, 1, v, j.mass, j.ld_mass, j.keep, j.recent, j.kept, j.lens_out);
  if (e != cudaSuccess) return QR_ERR_CUDA;
  MoveArgs a{};
  a.v = v;
  a.table_out = j.table_out;
  a.mass = j.mass;
  a.mass_out = j.mass_out;
  a.ld_mass = j.ld_mass;
  a.kept = j.kept;
  a.keep = j.keep;
  a.units = v.group / 32;
  const int64_t most = static_cast<int64_t>(std::min(j.keep, v.capacity)) * a.units;
  const int64_t piece = kMoveThreads * kMoveUnroll;
  const int pieces = static_cast<int>(std::min<int64_t>((most + piece - 1) / piece, 64));
  e = launch_pdl(kv_move_kernel, dim3(v.batch, v.groups, 7 * pieces), dim3(kMoveThreads), 0, stream,
                 1, a, pieces);
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? QR_OK : QR_ERR_CUDA;
}

}  // namespace qr
