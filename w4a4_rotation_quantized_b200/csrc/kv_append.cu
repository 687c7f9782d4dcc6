// kv_append.cu -- the write into the paged 4-bit KV cache and the read back.
//
// Append, per token row: rope on the heads of q and k (each pair of elements turned by
// position * frequency, the position taken from the pair's axis), R3 = H_d / sqrt(d) on
// every head of both, q rounded to fp16, k and v quantized group-wise to
// asymmetric 4-bit codes at the token's slot.  The quantizer and the order of the
// butterfly's additions are those of kv_group_quant_kernel, so that without a rope
// both give the same bits.
//
// Memory-bound: 2 (H_q + 2 H_k) d bytes read and 2 H_q d + H_k (d + 16 d / g) written
// a token.  One warp takes one group of 32 E consecutive values of a row (whole
// heads) at a time, lane L elements [E L, E L + E): vector loads and stores, the
// butterflies in registers and by shuffles.  A rope turns (i, i + pairs): the
// lane reads its elements' partners from memory a second time (they are in
// L1, since another lane of the warp just asked for them), which is cheaper to
// address than a shuffle whose distance depends on the number of pairs.  The angles
// depend on the token alone, not on the head: a block forms the sines and cosines of
// its tokens once, in double precision (positions pass 2^17 radians, where a
// float32 product is off by more than the last bits of the codes), and its warps
// share them through shared memory.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "kv_device.cuh"
#include "qr_internal.h"
#include "row_quant.cuh"

namespace qr {

namespace {

constexpr int kAppendWarps = 8;
constexpr int kMaxPairs = 128;             // head_dim / 2
constexpr int kTokensPerBlock = 4;

struct AppendArgs {
  KvView v;
  const __half* src[3];                    // q, k, v (null: absent)
  int64_t ld[3];
  __half* q_rot;
  int32_t q_width;
  int32_t jobs[3];                         // groups of a row: q, k, v
  const float* inv_freq;                   // null: no rope
  const int32_t* axis;
  const int32_t* positions;
  int64_t ld_pos;
  int32_t pairs, axes, interleaved;
  int32_t head_bits;
  float inv_sqrt;
};

// Where the elements of a rope meet: the partner of element h of a head, and its pair;
// pair < 0 when h is not turned.
__device__ __forceinline__ int rope_pair(const AppendArgs& a, int h, int* partner, bool* second) {
  if (h >= 2 * a.pairs) return -1;
  if (a.interleaved) {
    *partner = h ^ 1;
    *second = h & 1;
    return h >> 1;
  }
  *second = h >= a.pairs;
  *partner = *second ? h - a.pairs : h + a.pairs;
  return *second ? h - a.pairs : h;
}

template <int E>
__global__ void __launch_bounds__(32 * kAppendWarps) kv_append_kernel(AppendArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  constexpr int G = 32 * E;
  constexpr int LE = E == 4 ? 2 : 3;
  using V = typename std::conditional<E == 4, uint2, uint4>::type;
  using C = typename std::conditional<E == 4, uint16_t, uint32_t>::type;
  __shared__ float2 turn[kTokensPerBlock][kMaxPairs];       // (cos, sin)
  __shared__ int32_t token_seq[kTokensPerBlock];
  __shared__ int64_t token_slot[kTokensPerBlock];           // -1: no place for k and v
  const KvView& v = a.v;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t i0 = blockIdx.x * kTokensPerBlock;

  if (warp < kTokensPerBlock) {
    const int32_t i = i0 + warp;
    int32_t b = v.batch;
    int64_t slot = -1;
    if (i < v.tokens) {
      b = kv_seq_of_row(v, i);
      if (b < v.batch) {
        const int32_t c0 = v.cu[b], c1 = v.cu[b + 1];
        if (i < c0 || c0 < 0) b = v.batch;                  // offsets that do not ascend
        else {
          const int32_t t = kv_len(v, b) - (c1 - i);
          if (t >= 0) slot = kv_slot(v, v.table, b, t);
        }
      }
    }
    if (lane == 0) {
      token_seq[warp] = b;
      token_slot[warp] = slot;
    }
  }
  if (a.inv_freq != nullptr) {
    for (int p = threadIdx.x; p < kTokensPerBlock * a.pairs; p += blockDim.x) {
      const int u = p / a.pairs, j = p - u * a.pairs;
      if (i0 + u >= v.tokens) break;
      const int32_t ax = a.axis != nullptr ? a.axis[j] : 0;
      double s = 0.0, c = 1.0;
      if (ax >= 0 && ax < a.axes)
        sincos(static_cast<double>(a.positions[ax * a.ld_pos + i0 + u]) *
                   static_cast<double>(a.inv_freq[j]), &s, &c);
      turn[u][j] = make_float2(static_cast<float>(c), static_cast<float>(s));
    }
  }
  __syncthreads();

  const int per_token = a.jobs[0] + a.jobs[1] + a.jobs[2];
  const int stride = gridDim.y * kAppendWarps;
  const int jobs = kTokensPerBlock * per_token;
  for (int job = blockIdx.y * kAppendWarps + warp; job < jobs; job += stride) {
    const int u = job / per_token;
    int g = job - u * per_token;
    const int32_t i = i0 + u;
    if (i >= v.tokens || token_seq[u] >= v.batch) continue;      // uniform over the warp
    const int side = g < a.jobs[0] ? 0 : g < a.jobs[0] + a.jobs[1] ? 1 : 2;
    g -= side == 0 ? 0 : side == 1 ? a.jobs[0] : a.jobs[0] + a.jobs[1];
    const int64_t slot = token_slot[u];
    if (side != 0 && slot < 0) continue;
    const __half* row = a.src[side] + i * a.ld[side];
    const int e0 = g * G + lane * E;
    const V raw = *reinterpret_cast<const V*>(row + e0);
    const __half* h = reinterpret_cast<const __half*>(&raw);
    float x[E];
#pragma unroll
    for (int j = 0; j < E; ++j) x[j] = __half2float(h[j]);
    if (side != 2) {
      if (a.inv_freq != nullptr) {
        const int d = v.head_dim, h0 = e0 & (d - 1);
        float o[E];                                         // the partners
        if (a.interleaved) {
#pragma unroll
          for (int j = 0; j < E; ++j) o[j] = x[j ^ 1];
        } else if (a.pairs % E == 0) {                      // a lane's elements share one side
          V rawp = raw;
          if (h0 < 2 * a.pairs)
            rawp = *reinterpret_cast<const V*>(row + (h0 < a.pairs ? e0 + a.pairs : e0 - a.pairs));
          const __half* hp = reinterpret_cast<const __half*>(&rawp);
#pragma unroll
          for (int j = 0; j < E; ++j) o[j] = __half2float(hp[j]);
        } else {
#pragma unroll
          for (int j = 0; j < E; ++j) {
            const int hh = h0 + j;
            o[j] = hh < 2 * a.pairs
                       ? __half2float(row[hh < a.pairs ? e0 + j + a.pairs : e0 + j - a.pairs])
                       : 0.0f;
          }
        }
#pragma unroll
        for (int j = 0; j < E; ++j) {
          int partner;
          bool second;
          const int p = rope_pair(a, h0 + j, &partner, &second);
          if (p >= 0) {
            const float2 cs = turn[u][p];
            const float xc = __fmul_rn(x[j], cs.x), os = __fmul_rn(o[j], cs.y);
            x[j] = second ? __fadd_rn(xc, os) : __fsub_rn(xc, os);
          }
        }
      }
#pragma unroll
      for (int b = 0; b < LE; ++b)
#pragma unroll
        for (int j = 0; j < E; ++j)
          if (!(j & (1 << b))) {
            const float p = x[j], q = x[j | (1 << b)];
            x[j] = p + q;
            x[j | (1 << b)] = p - q;
          }
#pragma unroll
      for (int lb = 0; lb < 5; ++lb)
        if (LE + lb < a.head_bits) {
          const bool upper = (lane >> lb) & 1;
#pragma unroll
          for (int j = 0; j < E; ++j) {
            const float o = __shfl_xor_sync(0xffffffffu, x[j], 1 << lb);
            x[j] = upper ? o - x[j] : x[j] + o;
          }
        }
    }
    if (side == 0) {
      V out;
      __half* oh = reinterpret_cast<__half*>(&out);
#pragma unroll
      for (int j = 0; j < E; ++j) oh[j] = __float2half_rn(x[j] * a.inv_sqrt);
      *reinterpret_cast<V*>(a.q_rot + static_cast<int64_t>(i) * a.q_width + e0) = out;
      continue;
    }
    float mx = x[0], mn = x[0];
#pragma unroll
    for (int j = 1; j < E; ++j) {
      mx = fmaxf(mx, x[j]);
      mn = fminf(mn, x[j]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    }
    const int64_t at = slot * v.groups + g;
    const RowQ q = asym_row_q(mn, mx, 1.0f, side == 1 ? a.inv_sqrt : 1.0f,
                              lane == 0 ? v.scales[side - 1] + at : nullptr,
                              v.zeros[side - 1] + at);
    C packed = 0;
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const float t = fminf(fmaxf(fmaf(x[j], q.r, q.c), q.lo), q.hi);
      packed |= static_cast<C>((__float_as_uint(t) & 0xFu) << (4 * j));
    }
    *reinterpret_cast<C*>(v.codes[side - 1] + at * (G / 2) + lane * (E / 2)) = packed;
  }
}

// One warp per group of a token's row: E codes a lane, one fp16 vector store.
template <int E>
__global__ void __launch_bounds__(256) kv_dequantize_kernel(KvView v, __half* k_out,
                                                            __half* v_out) {
  grid_dep_wait();
  grid_dep_launch();
  constexpr int G = 32 * E;
  using V = typename std::conditional<E == 4, uint2, uint4>::type;
  using C = typename std::conditional<E == 4, uint16_t, uint32_t>::type;
  const int lane = threadIdx.x & 31;
  const int32_t i = blockIdx.x;
  const int32_t b = kv_seq_of_row(v, i);
  if (b >= v.batch) return;
  const int32_t c0 = v.cu[b], c1 = v.cu[b + 1];
  if (i < c0 || c0 < 0) return;
  const int32_t t = kv_len(v, b) - (c1 - i);
  const int64_t slot = t >= 0 ? kv_slot(v, v.table, b, t) : -1;
  const int first = k_out != nullptr ? 0 : v.groups, last = v_out != nullptr ? 2 * v.groups : v.groups;
  for (int job = first + (threadIdx.x >> 5); job < last; job += 8) {
    const int side = job >= v.groups;
    const int g = job - side * v.groups;
    V out;
    __half* oh = reinterpret_cast<__half*>(&out);
#pragma unroll
    for (int j = 0; j < E; ++j) oh[j] = __float2half_rn(0.0f);
    if (slot >= 0) {
      const int64_t at = slot * v.groups + g;
      const float s = v.scales[side][at];
      const int32_t z = v.zeros[side][at];
      const C c = *reinterpret_cast<const C*>(v.codes[side] + at * (G / 2) + lane * (E / 2));
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const int32_t code = static_cast<int32_t>(((c >> (4 * j)) & 0xF) ^ 8) - 8;
        oh[j] = __float2half_rn(s * static_cast<float>(static_cast<int64_t>(code) - z));
      }
    }
    __half* dst = side == 0 ? k_out : v_out;
    *reinterpret_cast<V*>(dst + static_cast<int64_t>(i) * v.width + g * G + lane * E) = out;
  }
}

}  // namespace

qr_status launch_kv_append(const KvView& v, const KvAppendJob& j, cudaStream_t stream) {
  AppendArgs a{};
  a.v = v;
  a.src[0] = reinterpret_cast<const __half*>(j.q);
  a.src[1] = reinterpret_cast<const __half*>(j.k);
  a.src[2] = reinterpret_cast<const __half*>(j.v);
  a.ld[0] = j.ldq;
  a.ld[1] = j.ldk;
  a.ld[2] = j.ldv;
  a.q_rot = reinterpret_cast<__half*>(j.q_rot);
  a.q_width = j.q_heads * v.head_dim;
  a.jobs[0] = j.q != nullptr ? a.q_width / v.group : 0;
  a.jobs[1] = j.k != nullptr ? v.groups : 0;
  a.jobs[2] = j.v != nullptr ? v.groups : 0;
  if (j.rope != nullptr) {
    a.inv_freq = j.rope->inv_freq;
    a.axis = j.rope->axis;
    a.positions = j.rope->positions;
    a.ld_pos = j.rope->ld_pos;
    a.pairs = j.rope->pairs;
    a.axes = j.rope->axes;
    a.interleaved = j.rope->interleaved;
  }
  while ((1 << a.head_bits) < v.head_dim) ++a.head_bits;
  a.inv_sqrt = static_cast<float>(1.0 / std::sqrt(static_cast<double>(v.head_dim)));
  const int jobs = a.jobs[0] + a.jobs[1] + a.jobs[2];
  if (jobs == 0) return QR_OK;
  const unsigned blocks = (v.tokens + kTokensPerBlock - 1) / kTokensPerBlock;
  // few tokens: several blocks share the groups of theirs, up to one group a warp
  const int most = (kTokensPerBlock * jobs + kAppendWarps - 1) / kAppendWarps;
  const unsigned split = std::max(1, std::min<int>(most, 4 * sm_count() / static_cast<int>(std::min(blocks, 1u << 20))));
  const dim3 grid(blocks, split), block(32 * kAppendWarps);
  cudaError_t e = v.group == 128 ? launch_pdl(kv_append_kernel<4>, grid, block, 0, stream, 1, a)
                                 : launch_pdl(kv_append_kernel<8>, grid, block, 0, stream, 1, a);
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? QR_OK : QR_ERR_CUDA;
}

qr_status launch_kv_dequantize(const KvView& v, uint16_t* k_out, uint16_t* v_out,
                               cudaStream_t stream) {
  const dim3 grid(v.tokens), block(256);
  auto* k = reinterpret_cast<__half*>(k_out);
  auto* w = reinterpret_cast<__half*>(v_out);
  cudaError_t e = v.group == 128
                      ? launch_pdl(kv_dequantize_kernel<4>, grid, block, 0, stream, 1, v, k, w)
                      : launch_pdl(kv_dequantize_kernel<8>, grid, block, 0, stream, 1, v, k, w);
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? QR_OK : QR_ERR_CUDA;
}

}  // namespace qr
