// kv_attention.cu -- attention over the paged 4-bit KV cache, and the attention
// weight that each cached token receives.
//
// One warp per (row, query head), its lanes over the head's elements: for each
// visible token the score is a warp sum, and the running maximum m, sum l and
// output o of the softmax are carried along,
//   m' = max(m, x),  l' = l e^(m - m') + e^(x - m'),  o' = o e^(m - m') + e^(x - m') v.
// The mass kernel turns this around: one warp per (sequence, group, token), which
// sums e^(x - lse) over the rows that see the token.
#include <cmath>

#include "kv_device.cuh"
#include "qr_internal.h"

namespace qr {

namespace {

// Values of a lane's E elements of head h in slot `slot`.
template <int E>
__device__ __forceinline__ void load_values(const KvView& v, int side, int64_t slot, int h, int lane,
                                            float (&x)[E]) {
  const int e = h * v.head_dim + lane * E;
  const int64_t g = slot * v.groups + e / v.group;
  const float s = v.scales[side][g];
  const int32_t z = v.zeros[side][g];
  const uint8_t* c = v.codes[side] + slot * (v.width / 2);
#pragma unroll
  for (int j = 0; j < E; ++j) {
    const int nib = (c[(e + j) >> 1] >> (4 * ((e + j) & 1))) & 0xF;
    x[j] = s * static_cast<float>(static_cast<int64_t>((nib ^ 8) - 8) - z);
  }
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Tokens that row i of a sequence sees.
__device__ __forceinline__ int32_t visible(int32_t len, int32_t rows, int32_t i, int causal) {
  return causal ? min(max(len - rows + i + 1, 0), len) : len;
}

template <int E>
__global__ void __launch_bounds__(256) kv_attention_kernel(KvView v, const __half* Q, int64_t ldq,
                                                           int32_t q_heads, float scale, int causal,
                                                           __half* out, int64_t ldo, float* lse) {
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31;
  const int64_t job = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int32_t i = static_cast<int32_t>(job / q_heads), h = static_cast<int32_t>(job % q_heads);
  if (i >= v.tokens) return;
  const int32_t b = kv_seq_of_row(v, i);
  if (b >= v.batch) return;
  const int32_t c0 = v.cu[b], c1 = v.cu[b + 1];
  if (i < c0 || c0 < 0) return;
  const int32_t n = visible(kv_len(v, b), c1 - c0, i - c0, causal);
  const int hk = h / (q_heads / v.heads);
  float q[E], o[E], x[E], m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int j = 0; j < E; ++j) {
    q[j] = __half2float(Q[i * ldq + h * 32 * E + lane * E + j]);
    o[j] = 0.0f;
  }
  for (int32_t t = 0; t < n; ++t) {
    const int64_t slot = kv_slot(v, v.table, b, t);
    if (slot < 0) continue;
    load_values<E>(v, 0, slot, hk, lane, x);
    float dot = 0.0f;
#pragma unroll
    for (int j = 0; j < E; ++j) dot = fmaf(q[j], x[j], dot);
    dot = warp_sum(dot) * scale;
    const float m1 = fmaxf(m, dot);
    const float keep = expf(m - m1), p = expf(dot - m1);
    load_values<E>(v, 1, slot, hk, lane, x);
#pragma unroll
    for (int j = 0; j < E; ++j) o[j] = fmaf(o[j], keep, p * x[j]);
    l = fmaf(l, keep, p);
    m = m1;
  }
  const float inv = l > 0.0f ? 1.0f / l : l == 0.0f ? 0.0f : l;      // NaN stays
#pragma unroll
  for (int j = 0; j < E; ++j)
    out[i * ldo + h * 32 * E + lane * E + j] = __float2half_rn(o[j] * inv);
  if (lse != nullptr && lane == 0)
    lse[static_cast<int64_t>(i) * q_heads + h] = l == 0.0f ? -INFINITY : m + logf(l);
}

template <int E>
__global__ void __launch_bounds__(256) kv_mass_kernel(KvView v, const __half* Q, int64_t ldq,
                                                      int32_t q_heads, float scale, int causal,
                                                      const float* lse, float* mass,
                                                      int64_t ld_mass) {
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31;
  const int32_t b = blockIdx.z, j = blockIdx.y;
  const int32_t t = blockIdx.x * 8 + (threadIdx.x >> 5);
  const int32_t len = kv_len(v, b);
  if (t >= len) return;
  const int64_t slot = kv_slot(v, v.table, b, t);
  if (slot < 0) return;
  const int32_t c0 = max(v.cu[b], 0), c1 = min(v.cu[b + 1], v.tokens);
  const int per = v.group / v.head_dim, gq = q_heads / v.heads;
  float sum = 0.0f;
  for (int hk = j * per; hk < (j + 1) * per; ++hk) {
    float x[E];
    load_values<E>(v, 0, slot, hk, lane, x);
    for (int32_t i = c0; i < c1; ++i) {
      if (t >= visible(len, v.cu[b + 1] - v.cu[b], i - v.cu[b], causal)) continue;
      for (int h = hk * gq; h < (hk + 1) * gq; ++h) {
        float dot = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e)
          dot = fmaf(__half2float(Q[i * ldq + h * 32 * E + lane * E + e]), x[e], dot);
        dot = warp_sum(dot) * scale;
        const float ls = lse[static_cast<int64_t>(i) * q_heads + h];
        sum += ls == -INFINITY ? 0.0f : expf(dot - ls);
      }
    }
  }
  if (lane == 0) mass[(static_cast<int64_t>(b) * v.groups + j) * ld_mass + t] += sum;
}

}  // namespace

int64_t kv_attention_workspace(const KvView& v, int32_t q_heads) {
  (void)v;
  (void)q_heads;
  return 0;
}

qr_status launch_kv_attention(const KvView& v, const KvAttentionJob& j, cudaStream_t stream) {
  const int64_t warps = static_cast<int64_t>(v.tokens) * j.q_heads;
  const dim3 grid(static_cast<unsigned>((warps + 7) / 8)), block(256);
  const auto* q = reinterpret_cast<const __half*>(j.q);
  auto* out = reinterpret_cast<__half*>(j.out);
  cudaError_t e;
  switch (v.head_dim) {
    case 32: e = launch_pdl(kv_attention_kernel<1>, grid, block, 0, stream, 1, v, q, j.ldq, j.q_heads, j.scale, j.causal, out, j.ldo, j.lse); break;
    case 64: e = launch_pdl(kv_attention_kernel<2>, grid, block, 0, stream, 1, v, q, j.ldq, j.q_heads, j.scale, j.causal, out, j.ldo, j.lse); break;
    case 128: e = launch_pdl(kv_attention_kernel<4>, grid, block, 0, stream, 1, v, q, j.ldq, j.q_heads, j.scale, j.causal, out, j.ldo, j.lse); break;
    default: e = launch_pdl(kv_attention_kernel<8>, grid, block, 0, stream, 1, v, q, j.ldq, j.q_heads, j.scale, j.causal, out, j.ldo, j.lse); break;
  }
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? QR_OK : QR_ERR_CUDA;
}

qr_status launch_kv_mass(const KvView& v, const KvMassJob& j, cudaStream_t stream) {
  const dim3 grid((v.capacity + 7) / 8, v.groups, v.batch), block(256);
  const auto* q = reinterpret_cast<const __half*>(j.q);
  cudaError_t e;
  switch (v.head_dim) {
    case 32: e = launch_pdl(kv_mass_kernel<1>, grid, block, 0, stream, 1, v, q, j.ldq, j.q_heads, j.scale, j.causal, j.lse, j.mass, j.ld_mass); break;
    case 64: e = launch_pdl(kv_mass_kernel<2>, grid, block, 0, stream, 1, v, q, j.ldq, j.q_heads, j.scale, j.causal, j.lse, j.mass, j.ld_mass); break;
    case 128: e = launch_pdl(kv_mass_kernel<4>, grid, block, 0, stream, 1, v, q, j.ldq, j.q_heads, j.scale, j.causal, j.lse, j.mass, j.ld_mass); break;
    default: e = launch_pdl(kv_mass_kernel<8>, grid, block, 0, stream, 1, v, q, j.ldq, j.q_heads, j.scale, j.causal, j.lse, j.mass, j.ld_mass); break;
  }
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? QR_OK : QR_ERR_CUDA;
}

}  // namespace qr
