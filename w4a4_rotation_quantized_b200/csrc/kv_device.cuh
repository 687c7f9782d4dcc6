// kv_device.cuh -- what the kernels on the paged 4-bit KV cache share: the
// cache and the batch as kernel parameters, the way from a row of the call to its
// sequence and from a token of a sequence to its slot.  Lengths, row offsets and
// the page table are read with plain loads: the kernel before this one on the
// stream, behind which this one may have started early, may have written them.
#pragma once

#include <cuda_fp16.h>

#include "qr_device.cuh"

namespace qr {

// Kernel-side view of qr_kv_cache and qr_kv_seqs.
struct KvView {
  uint8_t* codes[2];          // keys, values
  float* scales[2];
  int32_t* zeros[2];
  const int32_t* table;       // or null
  const int32_t* lens;
  const int32_t* cu;
  int32_t pages;              // whole pages in the cache
  int32_t page_size;
  uint32_t page_magic;        // t / page_size by multiplication, see kv_page
  uint32_t page_shift;
  int32_t max_pages;
  int32_t capacity;           // max_pages * page_size
  int32_t batch;
  int32_t heads, head_dim, group;
  int32_t width;              // heads * head_dim
  int32_t groups;             // width / group
  int32_t tokens;             // rows of the call's arrays
};

// t / page_size for 0 <= t < 2^30: with L = ceil(log2 page_size) and magic =
// floor(2^32 (2^L - page_size) / page_size) + 1, (umulhi(t, magic) + t) >> L
// (the round-up method; the sum stays below 2^31).
__device__ __forceinline__ int32_t kv_page(const KvView& v, int32_t t) {
  return static_cast<int32_t>((__umulhi(static_cast<uint32_t>(t), v.page_magic) +
                               static_cast<uint32_t>(t)) >> v.page_shift);
}

// Slot of token t (0 <= t < capacity) of sequence b under `table`, or -1 when the page number
// lies outside the cache.
__device__ __forceinline__ int64_t kv_slot(const KvView& v, const int32_t* table, int32_t b,
                                           int32_t t) {
  const int32_t p = kv_page(v, t);
  const int64_t at = static_cast<int64_t>(b) * v.max_pages + p;
  const int64_t page = table != nullptr ? static_cast<int64_t>(table[at]) : at;
  if (page < 0 || page >= v.pages) return -1;
  return page * v.page_size + (t - p * v.page_size);
}

__device__ __forceinline__ int32_t kv_len(const KvView& v, int32_t b) {
  return min(max(v.lens[b], 0), v.capacity);
}

// Sequence of row i: the number of sequences that end at or before it.  All
// lanes of a warp call it together; a result of `batch` means none.
__device__ __forceinline__ int32_t kv_seq_of_row(const KvView& v, int32_t i) {
  int32_t n = 0;
  for (int32_t j = static_cast<int32_t>(threadIdx.x & 31); j < v.batch; j += 32)
    n += v.cu[j + 1] <= i ? 1 : 0;
  return __reduce_add_sync(0xffffffffu, n);
}

}  // namespace qr
