// kv_append.cu -- the write into the paged 4-bit KV cache and the read back.
//
// Append, per token row: rope on the heads of q and k (each pair of elements turned by
// position * frequency, the position taken from the pair's axis), R3 = H_d / sqrt(d) on
// every head of both, q rounded to fp16, k and v quantized group-wise to
// asymmetric 4-bit codes at the token's slot.  The quantizer and the order of the
// butterfly's additions are those of kv_group_quant_kernel, so that without a rope
// both give the same bits.
//
// 2 (H_q + 2 H_k) d bytes read and 2 H_q d + H_k (d + 16 d / g) written a token, against some 14 operations an
// element: a lane holds 16 consecutive elements, so that four of the butterfly's stages run in registers (on
// pairs of fp32) and only those above them by shuffles (103 us for 7676 tokens of 32 + 2 x 32 heads of 128, 276
// with 4 elements a lane: the issue of 250 instructions for 128 elements bound it).  A rope turns (i, i + pairs): the lane reads
// its elements' partners from memory a second time (they are in L1, since another lane just asked for them), which
// is cheaper to address than shuffles whose distance depends on the number of pairs.  The angles depend on the
// token alone, not on the head: a block forms the sines and cosines of its tokens once, in double precision
// (positions pass 2^17 radians, where a float32 product is off by more than the last bits of the codes), and its
// warps share them through shared memory.
#include <algorithm>
#include <cmath>

#include "kv_device.cuh"
#include "qr_internal.h"
#include "row_quant.cuh"

namespace qr {

namespace {

constexpr int kAppendWarps = 8;
constexpr int kMaxPairs = 128;             // head_dim / 2
constexpr int kTokensPerBlock = 4;         // at most; one where tokens are few

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
  float inv_sqrt;
  int32_t per_block;                       // tokens of a block
};

constexpr int kLane = 16;                 // elements of a lane

// 16 consecutive fp16 values as fp32.
__device__ __forceinline__ void load_16(const __half* p, float (&x)[kLane]) {
  uint4 raw[2];
  raw[0] = reinterpret_cast<const uint4*>(p)[0];
  raw[1] = reinterpret_cast<const uint4*>(p)[1];
  const __half2* h = reinterpret_cast<const __half2*>(raw);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 f = __half22float2(h[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

// Place of pair p in a table of cosines or sines: 16 pairs (a lane's) 80 bytes apart, so that eight lanes' 16-byte
// reads meet all banks.
__device__ __forceinline__ int pair_at(int p) { return p + (p >> 4) * 4; }

// D: head_dim; G: group.
template <int D, int G>
__global__ void __launch_bounds__(32 * kAppendWarps, 4) kv_append_kernel(const AppendArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  // of the block's tokens: cosines, sines and sines with the other sign
  __shared__ __align__(16) float turn[kTokensPerBlock][3][kMaxPairs / 16 * 20];
  __shared__ int32_t token_seq[kTokensPerBlock];
  __shared__ int64_t token_slot[kTokensPerBlock];           // -1: no place for k and v
  const KvView& v = a.v;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t i0 = blockIdx.x * a.per_block;

  if (warp < a.per_block) {
    const int32_t i = i0 + warp;
    int32_t b = v.batch;
    int64_t slot = -1;
    if (i < v.tokens) {
      b = kv_seq_of_row(v, i);
      if (b < v.batch) {
        const int32_t c0 = v.cu[b], c1 = v.cu[b + 1];
        if (i < c0 || i >= c1 || c0 < 0) b = v.batch;       // offsets that do not ascend
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
    for (int p = threadIdx.x; p < a.per_block * a.pairs; p += blockDim.x) {
      const int u = p / a.pairs, j = p - u * a.pairs;
      if (i0 + u >= v.tokens) break;
      const int32_t ax = a.axis != nullptr ? a.axis[j] : 0;
      double s = 0.0, c = 1.0;
      if (ax >= 0 && ax < a.axes)
        sincos(static_cast<double>(a.positions[ax * a.ld_pos + i0 + u]) *
                   static_cast<double>(a.inv_freq[j]), &s, &c);
      turn[u][0][pair_at(j)] = static_cast<float>(c);
      turn[u][1][pair_at(j)] = static_cast<float>(s);
      turn[u][2][pair_at(j)] = -static_cast<float>(s);
    }
  }
  __syncthreads();

  constexpr int lanes = G / kLane, per = 32 / lanes;        // lanes of a group, groups of a warp
  const int lg = lane / lanes, in_group = lane % lanes * kLane;
  const int jq = (a.jobs[0] + per - 1) / per, jk = jq + (a.jobs[1] + per - 1) / per;
  const int per_token = jk + (a.jobs[2] + per - 1) / per;
#pragma unroll 1
  for (int u = 0; u < a.per_block; ++u)
#pragma unroll 1
    for (int job = blockIdx.y * kAppendWarps + warp; job < per_token; job += gridDim.y * kAppendWarps) {
    const int32_t i = i0 + u;
    if (i >= v.tokens || token_seq[u] >= v.batch) break;         // uniform over the warp
    const int side = job < jq ? 0 : job < jk ? 1 : 2;
    const int64_t slot = token_slot[u];
    if (side != 0 && slot < 0) break;
    const int g = (job - (side == 0 ? 0 : side == 1 ? jq : jk)) * per + lg;      // this lane's group
    const bool mine = g < (side == 0 ? a.jobs[0] : side == 1 ? a.jobs[1] : a.jobs[2]);
    const __half* row = (side == 0 ? a.src[0] + i * a.ld[0] : side == 1 ? a.src[1] + i * a.ld[1]
                                                                         : a.src[2] + i * a.ld[2]) +
                        (mine ? g * G : 0);
    float x[kLane];
    load_16(row + in_group, x);
    if (side != 2) {
      const int h0 = in_group & (D - 1);
      if (a.inv_freq != nullptr && h0 < 2 * a.pairs) {
        if (a.interleaved) {
#pragma unroll
          for (int j = 0; j < kLane; j += 2) {
            const int p = (h0 + j) >> 1;
            if (p < a.pairs) {
              const float c = turn[u][0][pair_at(p)], s = turn[u][1][pair_at(p)], xa = x[j], xb = x[j + 1];
              x[j] = __fsub_rn(__fmul_rn(xa, c), __fmul_rn(xb, s));
              x[j + 1] = __fadd_rn(__fmul_rn(xb, c), __fmul_rn(xa, s));
            }
          }
        } else if (a.pairs % kLane == 0) {                  // a lane's elements share one side
          const bool second = h0 >= a.pairs;
          float o[kLane];                                   // the partners
          load_16(row + in_group + (second ? -a.pairs : a.pairs), o);
          const float4* c = reinterpret_cast<const float4*>(turn[u][0] + pair_at(second ? h0 - a.pairs : h0));
          const float4* s = reinterpret_cast<const float4*>(turn[u][second ? 1 : 2] + pair_at(second ? h0 - a.pairs : h0));
#pragma unroll
          for (int j = 0; j < kLane; j += 4) {
            const float4 cj = c[j / 4], sj = s[j / 4];
            // products one by one: those of pairs (f2_mul) were fused into the sum, which is then rounded once only
            f2_unpack(f2_add(f2_pack(__fmul_rn(x[j], cj.x), __fmul_rn(x[j + 1], cj.y)),
                             f2_pack(__fmul_rn(o[j], sj.x), __fmul_rn(o[j + 1], sj.y))), x[j], x[j + 1]);
            f2_unpack(f2_add(f2_pack(__fmul_rn(x[j + 2], cj.z), __fmul_rn(x[j + 3], cj.w)),
                             f2_pack(__fmul_rn(o[j + 2], sj.z), __fmul_rn(o[j + 3], sj.w))), x[j + 2], x[j + 3]);
          }
        } else {
#pragma unroll
          for (int j = 0; j < kLane; ++j) {
            const int h = h0 + j;
            if (h < 2 * a.pairs) {
              const bool second = h >= a.pairs;
              const int p = second ? h - a.pairs : h;
              const float o = __half2float(row[in_group + j + (second ? -a.pairs : a.pairs)]);
              x[j] = __fadd_rn(__fmul_rn(x[j], turn[u][0][pair_at(p)]), __fmul_rn(o, turn[u][second ? 1 : 2][pair_at(p)]));
            }
          }
        }
      }
      wht_stages<0, 4>(x);                                  // the element bits held by the lane
#pragma unroll
      for (int lb = 0; lb < 4; ++lb)
        if ((16 << lb) < D) {                               // bits of the lane: x + o, or o - x
          const float sign = (lane >> lb) & 1 ? -1.0f : 1.0f;
          const uint64_t sign2 = f2_pack(sign, sign);
#pragma unroll
          for (int j = 0; j < kLane; j += 2) {
            const float o0 = __shfl_xor_sync(0xffffffffu, x[j], 1 << lb), o1 = __shfl_xor_sync(0xffffffffu, x[j + 1], 1 << lb);
            f2_unpack(f2_fma(f2_pack(x[j], x[j + 1]), sign2, f2_pack(o0, o1)), x[j], x[j + 1]);
          }
        }
    }
    if (side == 0) {
      if (!mine) continue;
      const uint64_t unit = f2_pack(a.inv_sqrt, a.inv_sqrt);
      __half2 out[8];
#pragma unroll
      for (int j = 0; j < kLane; j += 2) {
        float y0, y1;
        f2_unpack(f2_mul(f2_pack(x[j], x[j + 1]), unit), y0, y1);
        out[j / 2] = __floats2half2_rn(y0, y1);
      }
      uint4* to = reinterpret_cast<uint4*>(a.q_rot + static_cast<int64_t>(i) * a.q_width + g * G + in_group);
      to[0] = reinterpret_cast<const uint4*>(out)[0];
      to[1] = reinterpret_cast<const uint4*>(out)[1];
      continue;
    }
    float mx = x[0], mn = x[0];
#pragma unroll
    for (int j = 1; j < kLane; ++j) {
      mx = fmaxf(mx, x[j]);
      mn = fminf(mn, x[j]);
    }
#pragma unroll
    for (int o = lanes >> 1; o > 0; o >>= 1) {
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    }
    if (!mine) continue;
    const int64_t at = slot * v.groups + g;
    float* scale = (side == 1 ? v.scales[0] : v.scales[1]) + at;
    int32_t* zero = (side == 1 ? v.zeros[0] : v.zeros[1]) + at;
    const RowQ q = asym_row_q(mn, mx, 1.0f, side == 1 ? a.inv_sqrt : 1.0f, in_group == 0 ? scale : nullptr, zero);
    float lo8[8], hi8[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      lo8[j] = x[j];
      hi8[j] = x[8 + j];
    }
    *reinterpret_cast<uint2*>((side == 1 ? v.codes[0] : v.codes[1]) + at * (G / 2) + in_group / 2) =
        make_uint2(quant_word<true>(lo8, q.r, q.c, q.lo, q.hi), quant_word<true>(hi8, q.r, q.c, q.lo, q.hi));
  }
}

// A warp takes 512 values of a token's row at a time, 16 a lane: 8 bytes of codes in, two 16-byte stores out.
__global__ void __launch_bounds__(256) kv_dequantize_kernel(KvView v, __half* k_out, __half* v_out) {
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31;
  const int32_t i = blockIdx.x;
  const int32_t b = kv_seq_of_row(v, i);
  if (b >= v.batch) return;
  const int32_t c0 = v.cu[b], c1 = v.cu[b + 1];
  if (i < c0 || i >= c1 || c0 < 0) return;
  const int32_t t = kv_len(v, b) - (c1 - i);
  const int64_t slot = t >= 0 ? kv_slot(v, v.table, b, t) : -1;
  const int jobs = (v.width + 511) / 512;
  const int first = k_out != nullptr ? 0 : jobs, last = v_out != nullptr ? 2 * jobs : jobs;
  for (int job = first + (threadIdx.x >> 5); job < last; job += 8) {
    const bool values = job >= jobs;
    const int e0 = (values ? job - jobs : job) * 512 + lane * kLane;
    if (e0 >= v.width) continue;
    __half2 out[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) out[j] = __floats2half2_rn(0.0f, 0.0f);
    if (slot >= 0) {
      const int64_t at = slot * v.groups + e0 / v.group;
      const float s = (values ? v.scales[1] : v.scales[0])[at];
      const int32_t z = (values ? v.zeros[1] : v.zeros[0])[at];
      const uint2 w = *reinterpret_cast<const uint2*>((values ? v.codes[1] : v.codes[0]) + slot * (v.width / 2) + e0 / 2);
      if (z > -4000000 && z < 4000000) {
        // u = c + 8 in the low bits of 2^23: 2^23 + u - (2^23 + 8 + z) is c - z, exact
        const float off = 8388616.0f + static_cast<float>(z);
#pragma unroll
        for (int j = 0; j < kLane; j += 2) {
          const uint32_t x = ((j < 8 ? w.x : w.y) >> (4 * (j & 7))) ^ 0x88u;
          const float y0 = __uint_as_float((x & 15u) | 0x4B000000u) - off;
          const float y1 = __uint_as_float(((x >> 4) & 15u) | 0x4B000000u) - off;
          out[j / 2] = __floats2half2_rn(s * y0, s * y1);
        }
      } else {
#pragma unroll
        for (int j = 0; j < kLane; j += 2) {
          const uint32_t x = ((j < 8 ? w.x : w.y) >> (4 * (j & 7))) ^ 0x88u;
          const int64_t c1 = static_cast<int64_t>(x & 15u) - 8, c2 = static_cast<int64_t>((x >> 4) & 15u) - 8;
          out[j / 2] = __floats2half2_rn(s * static_cast<float>(c1 - z), s * static_cast<float>(c2 - z));
        }
      }
    }
    uint4* to = reinterpret_cast<uint4*>((values ? v_out : k_out) + static_cast<int64_t>(i) * v.width + e0);
    to[0] = reinterpret_cast<const uint4*>(out)[0];
    to[1] = reinterpret_cast<const uint4*>(out)[1];
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
  a.inv_sqrt = static_cast<float>(1.0 / std::sqrt(static_cast<double>(v.head_dim)));
  const int jobs = a.jobs[0] + a.jobs[1] + a.jobs[2];
  if (jobs == 0) return QR_OK;
  a.per_block = v.tokens <= 4 * sm_count() ? 1 : kTokensPerBlock;
  const unsigned blocks = (v.tokens + a.per_block - 1) / a.per_block;
  // few tokens: several blocks share the groups of theirs, up to one job a warp
  const int per = 32 * kLane / v.group;
  const int warps = (a.jobs[0] + per - 1) / per + (a.jobs[1] + per - 1) / per + (a.jobs[2] + per - 1) / per;
  const int most = (warps + kAppendWarps - 1) / kAppendWarps;
  const unsigned split = std::max(1, std::min<int>(most, 4 * sm_count() / static_cast<int>(std::min(blocks, 1u << 20))));
  const dim3 grid(blocks, split), block(32 * kAppendWarps);
  auto run = [&](auto kernel) { return launch_pdl(kernel, grid, block, 0, stream, 1, a); };
  cudaError_t e;
  if (v.group == 128)
    e = v.head_dim == 32 ? run(kv_append_kernel<32, 128>) : v.head_dim == 64 ? run(kv_append_kernel<64, 128>)
                                                          : run(kv_append_kernel<128, 128>);
  else
    e = v.head_dim == 32    ? run(kv_append_kernel<32, 256>)
        : v.head_dim == 64  ? run(kv_append_kernel<64, 256>)
        : v.head_dim == 128 ? run(kv_append_kernel<128, 256>)
                            : run(kv_append_kernel<256, 256>);
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? QR_OK : QR_ERR_CUDA;
}

qr_status launch_kv_dequantize(const KvView& v, uint16_t* k_out, uint16_t* v_out,
                               cudaStream_t stream) {
  const dim3 grid(v.tokens), block(256);
  auto* k = reinterpret_cast<__half*>(k_out);
  auto* w = reinterpret_cast<__half*>(v_out);
  cudaError_t e = launch_pdl(kv_dequantize_kernel, grid, block, 0, stream, 1, v, k, w);
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? QR_OK : QR_ERR_CUDA;
}

}  // namespace qr
