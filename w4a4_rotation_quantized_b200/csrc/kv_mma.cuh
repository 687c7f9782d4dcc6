// kv_mma.cuh -- 4-bit cache rows on the warp matrix instructions.
//
// Keys.  A nibble u in [0, 15] in bits 0-3 of a 16-bit half is the fp16 subnormal u 2^-24, in
// bits 4-7 u 2^-20: masked out of a word of codes, eight codes are four fp16 pairs after one shift
// and four logic operations (which flip bit 3, so that the two's-complement code c becomes
// u = c + 8), without a conversion.  Scale and zero meet the scores: s (c - z) = s (u - (z + 8)).
//
// Values.  The matrix instructions line products up by the exponents of their operands,
// where a subnormal counts as 2^-14: sums of products with u 2^-24 keep 2^-15 of a step, which is little
// for scores and too much for outputs that long sequences average down.  So a
// nibble is put behind the exponent of 1024 (or 64), where it makes 1024 + u (64 + u), and one fp16 addition
// of -(1032 + z) (or -(72 + z)) leaves c - z, a small whole number, exactly.
#pragma once

#include <cuda_fp16.h>

#include "kv_device.cuh"

namespace qr {

__device__ __forceinline__ uint32_t and_xor(uint32_t a, uint32_t mask, uint32_t flip) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(d) : "r"(a), "r"(mask), "r"(flip));
  return d;
}
__device__ __forceinline__ uint32_t nib_low(uint32_t x) { return and_xor(x, 0x000f000fu, 0x00080008u); }
__device__ __forceinline__ uint32_t nib_high(uint32_t x) { return and_xor(x, 0x00f000f0u, 0x00800080u); }

// 1024 + u and 64 + u of the low and the high nibble of each byte
__device__ __forceinline__ uint32_t nib_1024(uint32_t x) { return and_xor(x, 0x000f000fu, 0x64086408u); }
__device__ __forceinline__ uint32_t nib_64(uint32_t x) { return and_xor(x, 0x00f000f0u, 0x54805480u); }
__device__ __forceinline__ uint32_t add_half2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

__device__ __forceinline__ uint32_t byte_perm(uint32_t a, uint32_t b, uint32_t sel) {
  return __byte_perm(a, b, sel);
}

// d += A (16 x 16, rows) B (16 x 8, columns), fp16 in, fp32 accumulators.
__device__ __forceinline__ void mma_16x8x16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                            uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// d = A B
__device__ __forceinline__ void mma_16x8x16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                                  uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// 8 x 8 transpose of 16-bit elements across the warp: lane 4 r + c holds row r, columns 2c, 2c+1.
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// The 32 tokens of a step in a warp's shared memory: key codes, value codes (rows of D / 2 bytes),
// then the keys' scales and zeros and the values'.
template <int D>
struct KvStage {
  static constexpr int kRow = D / 2;
  static constexpr int kChunks = D / 32;              // 16-byte chunks of a row
  static constexpr int kCodes = 32 * kRow;
  static constexpr int kMeta = 2 * kCodes;
  static constexpr int kBytes = 2 * kCodes + 4 * 32 * 4;
  // what a warp keeps besides: a remainder and a half a token of the piece at hand, the tokens that are there
  // of every piece, the rows' limits
  static constexpr int kPrepared = 32 * 4 + 32 * 2 + 4 * 4 + 16 * 4;

  // Key row of token t: a lane of column c of the fragment reads chunk c (and c + 4 when D = 256;
  // less than a chunk when D < 128) of rows g and g + 8.  Only D = 256 needs a swizzle: its
  // rows are 128 bytes, and odd ones swap their halves.
  __device__ static __forceinline__ int key_at(int t, int chunk) {
    return t * kRow + ((D == 256 ? chunk ^ ((t & 1) << 2) : chunk) << 4);
  }
  // Value row of token t.  A lane reads the D / 16 bytes of row g of the tokens 2c, 2c + 1, 2c + 8,
  // 2c + 9; rows stand in the order 0 2 4 6 1 3 5 7, so that one such read meets four neighbours,
  // and chunks are swapped so that these fill all banks.
  __device__ static __forceinline__ int value_row(int t) {
    return (t & 24) | ((t & 1) << 2) | ((t >> 1) & 3);
  }
  __device__ static __forceinline__ int value_at(int row, int chunk) {
    const int x = D == 128 ? chunk ^ (row & 2) : D == 256 ? chunk ^ ((row & 3) << 1) : chunk;
    return row * kRow + (x << 4);
  }

  // Starts the copy of 32 tokens; lane t knows its token's slot (any slot for a token that is not there).
  // key, value: where chunk lane % kChunks of the head stands in a row; j: the head's group.  (A cache
  // has less than 2^32 groups.)
  template <bool KEYS, bool VALUES>
  __device__ static __forceinline__ void issue(const KvView& v, const uint8_t* key, const uint8_t* value,
                                               uint32_t j, uint32_t slot, uint32_t smem, int lane) {
    constexpr int kPer = 32 / kChunks;                  // tokens of one round of copies
    const uint32_t row_bytes = static_cast<uint32_t>(v.width) >> 1;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int t = i * kPer + lane / kChunks, chunk = lane % kChunks;
      const uint64_t off = static_cast<uint64_t>(__shfl_sync(0xffffffffu, slot, t)) * row_bytes;
      if (KEYS) cp_async_16(smem + key_at(t, chunk), key + off);
      if (VALUES) cp_async_16(smem + kCodes + value_at(value_row(t), chunk), value + off);
    }
    const uint32_t m = slot * static_cast<uint32_t>(v.groups) + j;
    if (KEYS) {
      cp_async_4(smem + kMeta + lane * 4, v.scales[0] + m);
      cp_async_4(smem + kMeta + 128 + lane * 4, v.zeros[0] + m);
    }
    if (VALUES) {
      cp_async_4(smem + kMeta + 256 + lane * 4, v.scales[1] + m);
      cp_async_4(smem + kMeta + 384 + lane * 4, v.zeros[1] + m);
    }
  }
};

// Queries as the B operand, in shared memory: lane 4 r + c owns, of query row r, the elements that column
// c's key words hold: word w covers 8 elements from first(w); pairs (e0, e4), (e2, e6) meet the low
// nibbles, (e1, e5), (e3, e7) the high ones.
template <int D>
struct QueryFrag {
  static constexpr int kWords = D / 32;
  static constexpr int kBytes = kWords * 32 * 16;       // of 8 rows: [word][lane] of 16 bytes

  __device__ static __forceinline__ int first(int c, int w) {
    return D == 256 ? (w >> 2) * 128 + c * 32 + (w & 3) * 8 : c * (D / 4) + w * 8;
  }
  // row: the query's elements, or null (zeros).  Returns the sum of the lane's elements.
  __device__ static __forceinline__ float put(uint4* frag, const __half* row, int lane) {
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
      uint4 x = make_uint4(0, 0, 0, 0);
      if (row != nullptr) x = *reinterpret_cast<const uint4*>(row + first(lane & 3, w));
      const uint32_t* p = reinterpret_cast<const uint32_t*>(&x);        // (e0 e1) (e2 e3) (e4 e5) (e6 e7)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(p + i));
        sum += f.x + f.y;
      }
      frag[w * 32 + lane] = make_uint4(byte_perm(x.x, x.z, 0x5410), byte_perm(x.y, x.w, 0x5410),
                                       byte_perm(x.x, x.z, 0x7632), byte_perm(x.y, x.w, 0x7632));
    }
    return sum;
  }
};

// The key words of one token row that a lane of column c holds.
template <int D>
__device__ __forceinline__ void load_key_words(const uint8_t* keys, int t, int c, uint32_t (&w)[D / 32]) {
  using S = KvStage<D>;
  if constexpr (D >= 128) {
#pragma unroll
    for (int i = 0; i < D / 128; ++i) {
      const uint4 x = *reinterpret_cast<const uint4*>(keys + S::key_at(t, c + 4 * i));
      w[4 * i] = x.x;
      w[4 * i + 1] = x.y;
      w[4 * i + 2] = x.z;
      w[4 * i + 3] = x.w;
    }
  } else if constexpr (D == 64) {
    const uint2 x = *reinterpret_cast<const uint2*>(keys + t * S::kRow + c * 8);
    w[0] = x.x;
    w[1] = x.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(keys + t * S::kRow + c * 4);
  }
}

// Sums over the low and the high nibbles, 2^-24 and 2^-20 sum q u, for 32 tokens (rows 16 h + g and 16 h +
// g + 8) and 8 NC queries.
template <int D, int NC>
__device__ __forceinline__ void key_scores(const uint8_t* keys, int lane, const uint4* q, float (&lo)[2][NC][4],
                                           float (&hi)[2][NC][4]) {
  const int g = lane >> 2, c = lane & 3;
  uint32_t x[2][2][D / 32];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    load_key_words<D>(keys, 16 * h + g, c, x[h][0]);
    load_key_words<D>(keys, 16 * h + g + 8, c, x[h][1]);
  }
#pragma unroll
  for (int w = 0; w < D / 32; ++w) {
    uint4 b[NC];
#pragma unroll
    for (int n = 0; n < NC; ++n) b[n] = q[(n * (D / 32) + w) * 32 + lane];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t xa = x[h][0][w], xb = x[h][1][w], ya = xa >> 8, yb = xb >> 8;
      const uint32_t l0 = nib_low(xa), l1 = nib_low(xb), l2 = nib_low(ya), l3 = nib_low(yb);
      const uint32_t h0 = nib_high(xa), h1 = nib_high(xb), h2 = nib_high(ya), h3 = nib_high(yb);
#pragma unroll
      for (int n = 0; n < NC; ++n) {
        if (w == 0) {
          mma_16x8x16_first(lo[h][n], l0, l1, l2, l3, b[n].x, b[n].y);
          mma_16x8x16_first(hi[h][n], h0, h1, h2, h3, b[n].z, b[n].w);
        } else {
          mma_16x8x16(lo[h][n], l0, l1, l2, l3, b[n].x, b[n].y);
          mma_16x8x16(hi[h][n], h0, h1, h2, h3, b[n].z, b[n].w);
        }
      }
    }
  }
}

// Output elements of the value product.  A lane of row g holds the elements g D/8 .. of a token, 4 bits
// each; product i of a pair of halves puts element i in its row g and element i + kHalf in row g + 8.
template <int D>
struct ValueTile {
  static constexpr int kPer = D / 8;                    // elements of a lane
  static constexpr int kHalf = kPer / 2 < 8 ? kPer / 2 : 8;
  static constexpr int kTiles = kPer / 2;               // products: 16 rows each
  // element (from g * kPer) of product i: row g, or row g + 8
  __device__ static __forceinline__ int element(int i, bool upper) {
    return (i / kHalf) * 2 * kHalf + (upper ? kHalf : 0) + i % kHalf;
  }
};

// o += V^T W^T for 32 tokens: W as fp16 pairs (high parts and the rest) of the tiles of 16; z1024: for each
// tile and the tokens (2c, 2c + 1), (2c + 8, 2c + 9) the fp16 pair -(1032 + z).  Columns 2c and 2c +
// 1 of o are a pair.  The matrix instructions cut what their sums are too small for instead of rounding
// it, so the sums of a piece start from zero and are added to o in fp32.
template <int D, int NC>
__device__ __forceinline__ void value_products(const uint8_t* vals, int g, int c, const uint32_t (&z1024)[2][2],
                                               const uint32_t (&wh)[2][NC][2], const uint32_t (&wl)[2][NC][2],
                                               uint64_t (&o)[ValueTile<D>::kTiles][NC][2]) {
  using S = KvStage<D>;
  uint32_t z64[2][2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int k = 0; k < 2; ++k) z64[h][k] = add_half2(z1024[h][k], 0x63806380u);      // + 960
  // a[h]: the operand of tile h of 16 tokens: rows g, g + 8 of tokens 2c, 2c + 1, then of 2c + 8, 2c + 9
  auto step = [&](int i, const uint32_t (&a)[2][4], bool high) {
    uint32_t u[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        u[h][k] = high ? add_half2(nib_64(a[h][k]), z64[h][k >> 1]) : add_half2(nib_1024(a[h][k]), z1024[h][k >> 1]);
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      float d[4];
      mma_16x8x16_first(d, u[0][0], u[0][1], u[0][2], u[0][3], wl[0][n][0], wl[0][n][1]);
      mma_16x8x16(d, u[1][0], u[1][1], u[1][2], u[1][3], wl[1][n][0], wl[1][n][1]);
      mma_16x8x16(d, u[0][0], u[0][1], u[0][2], u[0][3], wh[0][n][0], wh[0][n][1]);
      mma_16x8x16(d, u[1][0], u[1][1], u[1][2], u[1][3], wh[1][n][0], wh[1][n][1]);
      o[i][n][0] = f2_add(o[i][n][0], f2_pack(d[0], d[1]));
      o[i][n][1] = f2_add(o[i][n][1], f2_pack(d[2], d[3]));
    }
  };
  auto four = [&](int i, uint32_t (&a)[2][4]) {           // elements 0-3 of the halves in a
    step(i, a, false);
    step(i + 1, a, true);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int k = 0; k < 4; ++k) a[h][k] >>= 8;
    step(i + 2, a, false);
    step(i + 3, a, true);
  };
  // rows of the tokens 2c, 2c + 1, 2c + 8, 2c + 9 of a tile: 16 h + c + 4 k
  if constexpr (D >= 128) {
    constexpr int kPairs = D / 128;                     // pairs of words
    uint32_t x[2][4][2 * kPairs];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int row = 16 * h + c + 4 * k;
        if constexpr (D == 128) {
          const uint2 y = *reinterpret_cast<const uint2*>(vals + S::value_at(row, g >> 1) + (g & 1) * 8);
          x[h][k][0] = y.x;
          x[h][k][1] = y.y;
        } else {
          const uint4 y = *reinterpret_cast<const uint4*>(vals + S::value_at(row, g));
          x[h][k][0] = y.x;
          x[h][k][1] = y.y;
          x[h][k][2] = y.z;
          x[h][k][3] = y.w;
        }
      }
#pragma unroll
    for (int p = 0; p < kPairs; ++p)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const uint32_t sel = half ? 0x7632 : 0x5410;
        uint32_t a[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          a[h][0] = byte_perm(x[h][0][2 * p], x[h][1][2 * p], sel);
          a[h][1] = byte_perm(x[h][0][2 * p + 1], x[h][1][2 * p + 1], sel);
          a[h][2] = byte_perm(x[h][2][2 * p], x[h][3][2 * p], sel);
          a[h][3] = byte_perm(x[h][2][2 * p + 1], x[h][3][2 * p + 1], sel);
        }
        four(8 * p + 4 * half, a);
      }
  } else if constexpr (D == 64) {
    uint32_t a[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t x[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        x[k] = *reinterpret_cast<const uint32_t*>(vals + (16 * h + c + 4 * k) * S::kRow + g * 4);
      a[h][0] = byte_perm(x[0], x[1], 0x5410);
      a[h][1] = byte_perm(x[0], x[1], 0x7632);
      a[h][2] = byte_perm(x[2], x[3], 0x5410);
      a[h][3] = byte_perm(x[2], x[3], 0x7632);
    }
    four(0, a);
  } else {
    uint32_t a[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t x[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        x[k] = *reinterpret_cast<const uint16_t*>(vals + (16 * h + c + 4 * k) * S::kRow + g * 2);
      a[h][0] = x[0] | (x[1] << 16);
      a[h][1] = a[h][0] >> 8;
      a[h][2] = x[2] | (x[3] << 16);
      a[h][3] = a[h][2] >> 8;
    }
    step(0, a, false);
    step(1, a, true);
  }
}

}  // namespace qr
