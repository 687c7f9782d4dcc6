// kv_mass.cu -- the attention weight that each token of the paged 4-bit KV cache receives
// from the rows of a call, added to a running sum: one warp per (sequence, group, token).
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
