// qr_kv_api.cu -- the extern "C" entry points on the paged 4-bit KV cache:
// argument validation on the host, then one or two launches on the caller's
// stream.  Nothing here allocates memory or reads device memory.
#include <cuda_runtime.h>

#include <cmath>

#include "kv_device.cuh"
#include "qr_internal.h"

namespace qr {

namespace {

template <int N>
bool aligned(const void* p) { return reinterpret_cast<uintptr_t>(p) % N == 0; }

// Checks a cache and a batch and makes the kernels' view of them.
qr_status make_view(const qr_kv_cache* c, const qr_kv_seqs* s, int64_t tokens, bool need_cu,
                    KvView* v) {
  if (c == nullptr || s == nullptr || tokens < 0) return QR_ERR_INVALID_ARG;
  if (c->heads <= 0 || c->group <= 0 || c->page_size <= 0 || c->slots < 0) return QR_ERR_INVALID_ARG;
  if (s->batch < 0 || s->max_pages < 0) return QR_ERR_INVALID_ARG;
  const int32_t d = c->head_dim;
  if (d != 32 && d != 64 && d != 128 && d != 256) return QR_ERR_UNSUPPORTED;
  const int64_t width = static_cast<int64_t>(c->heads) * d;
  if ((c->group != 128 && c->group != 256) || c->group % d != 0 || width % c->group != 0)
    return QR_ERR_UNSUPPORTED;
  if (width > 65536 || s->batch > 4096 || tokens > (1 << 30)) return QR_ERR_UNSUPPORTED;
  const int64_t capacity = static_cast<int64_t>(s->max_pages) * c->page_size;
  if (capacity >= (1 << 30) || c->slots / c->page_size > 0x7FFFFFFF) return QR_ERR_UNSUPPORTED;
  // slots and pages of the batch are counted in 32 bits, groups of the cache in unsigned ones
  if (c->slots > 0x7FFFFFFF || static_cast<int64_t>(s->batch) * s->max_pages > 0x7FFFFFFF ||
      c->slots * (width / c->group) > 0xFFFFFFFFll)
    return QR_ERR_UNSUPPORTED;
  if (c->slots > 0) {
    if (!c->k_codes || !c->k_scales || !c->k_zeros || !c->v_codes || !c->v_scales || !c->v_zeros)
      return QR_ERR_INVALID_ARG;
    if (!aligned<16>(c->k_codes) || !aligned<16>(c->v_codes) || !aligned<4>(c->k_scales) ||
        !aligned<4>(c->k_zeros) || !aligned<4>(c->v_scales) || !aligned<4>(c->v_zeros))
      return QR_ERR_ALIGNMENT;
  }
  if (s->batch > 0 && (s->kv_lens == nullptr || (need_cu && s->cu_q == nullptr)))
    return QR_ERR_INVALID_ARG;
  if (!aligned<4>(s->kv_lens) || !aligned<4>(s->cu_q) || !aligned<4>(s->block_table))
    return QR_ERR_ALIGNMENT;
  *v = KvView{};
  v->codes[0] = c->k_codes;
  v->codes[1] = c->v_codes;
  v->scales[0] = c->k_scales;
  v->scales[1] = c->v_scales;
  v->zeros[0] = c->k_zeros;
  v->zeros[1] = c->v_zeros;
  v->table = s->max_pages > 0 ? s->block_table : nullptr;   // (a table of no pages has no element to read)
  v->lens = s->kv_lens;
  v->cu = s->cu_q;
  v->pages = static_cast<int32_t>(c->slots / c->page_size);
  v->page_size = c->page_size;
  uint32_t l = 0;
  while ((int64_t(1) << l) < c->page_size) ++l;
  v->page_shift = l;
  v->page_magic = static_cast<uint32_t>(
      ((uint64_t(1) << 32) * ((uint64_t(1) << l) - c->page_size)) / c->page_size + 1);
  v->max_pages = s->max_pages;
  v->capacity = v->pages > 0 ? static_cast<int32_t>(capacity) : 0;   // no pages: nothing is held
  v->batch = s->batch;
  v->heads = c->heads;
  v->head_dim = d;
  v->group = c->group;
  v->width = static_cast<int32_t>(width);
  v->groups = static_cast<int32_t>(width / c->group);
  v->tokens = static_cast<int32_t>(tokens);
  return QR_OK;
}

// What the two attention calls ask of their queries.
qr_status check_queries(const KvView& v, const uint16_t* Q, int64_t ldq, int32_t q_heads, float scale) {
  if (q_heads <= 0 || q_heads % v.heads != 0 || !std::isfinite(scale)) return QR_ERR_INVALID_ARG;
  if (static_cast<int64_t>(q_heads) * v.head_dim > 65536) return QR_ERR_UNSUPPORTED;
  // query rows of a key head are counted in 32 bits
  if (static_cast<int64_t>(v.tokens) * (q_heads / v.heads) > 0x7FFF0000) return QR_ERR_UNSUPPORTED;
  if (v.tokens > 0) {
    if (Q == nullptr || ldq < static_cast<int64_t>(q_heads) * v.head_dim) return QR_ERR_INVALID_ARG;
    if (!aligned<16>(Q) || ldq % 8 != 0) return QR_ERR_ALIGNMENT;
  }
  return QR_OK;
}

}  // namespace

}  // namespace qr

using namespace qr;

extern "C" {

qr_status qr_kv_append(const qr_kv_cache* cache, const qr_kv_seqs* seqs, const qr_kv_rope* rope,
                       const uint16_t* Q, int64_t ldq, const uint16_t* K, int64_t ldk,
                       const uint16_t* V, int64_t ldv, int64_t tokens, int32_t q_heads,
                       uint16_t* q_rot, qr_stream stream) {
  KvView v;
  qr_status st = make_view(cache, seqs, tokens, true, &v);
  if (st != QR_OK) return st;
  if ((Q == nullptr) != (q_rot == nullptr)) return QR_ERR_INVALID_ARG;
  if (Q != nullptr) {
    if (q_heads <= 0) return QR_ERR_INVALID_ARG;
    const int64_t qw = static_cast<int64_t>(q_heads) * v.head_dim;
    if (qw % v.group != 0 || qw > 65536) return QR_ERR_UNSUPPORTED;
    if (tokens > 0 && ldq < qw) return QR_ERR_INVALID_ARG;
    if (!aligned<16>(Q) || !aligned<16>(q_rot) || ldq % 8 != 0) return QR_ERR_ALIGNMENT;
    if (Q == q_rot) return QR_ERR_INVALID_ARG;
  }
  if (tokens > 0 && ((K != nullptr && ldk < v.width) || (V != nullptr && ldv < v.width)))
    return QR_ERR_INVALID_ARG;
  if ((K != nullptr && (!aligned<16>(K) || ldk % 8 != 0)) ||
      (V != nullptr && (!aligned<16>(V) || ldv % 8 != 0)))
    return QR_ERR_ALIGNMENT;
  if (rope != nullptr) {
    if (rope->pairs < 1 || rope->pairs > v.head_dim / 2 || rope->axes < 1) return QR_ERR_INVALID_ARG;
    if (rope->inv_freq == nullptr) return QR_ERR_INVALID_ARG;
    if (tokens > 0 && (rope->positions == nullptr || rope->ld_pos < tokens)) return QR_ERR_INVALID_ARG;
    if (!aligned<4>(rope->inv_freq) || !aligned<4>(rope->axis) || !aligned<4>(rope->positions))
      return QR_ERR_ALIGNMENT;
  }
  if (tokens == 0 || v.batch == 0) return QR_OK;
  KvAppendJob j{rope, Q, K, V, ldq, ldk, ldv, q_heads, q_rot};
  return launch_kv_append(v, j, reinterpret_cast<cudaStream_t>(stream));
}

qr_status qr_kv_dequantize(const qr_kv_cache* cache, const qr_kv_seqs* seqs, int64_t tokens,
                           uint16_t* k_out, uint16_t* v_out, qr_stream stream) {
  KvView v;
  qr_status st = make_view(cache, seqs, tokens, true, &v);
  if (st != QR_OK) return st;
  if (!aligned<16>(k_out) || !aligned<16>(v_out)) return QR_ERR_ALIGNMENT;
  if (tokens == 0 || v.batch == 0 || (k_out == nullptr && v_out == nullptr)) return QR_OK;
  return launch_kv_dequantize(v, k_out, v_out, reinterpret_cast<cudaStream_t>(stream));
}

int64_t qr_kv_attention_workspace(const qr_kv_cache* cache, const qr_kv_seqs* seqs, int64_t tokens,
                                  int32_t q_heads) {
  KvView v;
  if (make_view(cache, seqs, tokens, true, &v) != QR_OK) return -1;
  if (q_heads <= 0 || q_heads % v.heads != 0 ||
      static_cast<int64_t>(q_heads) * v.head_dim > 65536)
    return -1;
  return v.tokens == 0 || v.batch == 0 ? 0 : kv_attention_workspace(v, q_heads);
}

qr_status qr_kv_attention(const qr_kv_cache* cache, const qr_kv_seqs* seqs, const uint16_t* Q,
                          int64_t ldq, int64_t tokens, int32_t q_heads, float scale, int32_t causal,
                          uint16_t* out, int64_t ldo, float* lse, void* workspace,
                          int64_t workspace_bytes, qr_stream stream) {
  KvView v;
  qr_status st = make_view(cache, seqs, tokens, true, &v);
  if (st == QR_OK) st = check_queries(v, Q, ldq, q_heads, scale);
  if (st != QR_OK) return st;
  if (tokens == 0 || v.batch == 0) return QR_OK;
  if (out == nullptr || ldo < static_cast<int64_t>(q_heads) * v.head_dim) return QR_ERR_INVALID_ARG;
  if (!aligned<16>(out) || ldo % 8 != 0 || !aligned<4>(lse) || !aligned<16>(workspace))
    return QR_ERR_ALIGNMENT;
  const int64_t need = kv_attention_workspace(v, q_heads);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return QR_ERR_INVALID_ARG;
  KvAttentionJob j{Q, ldq, q_heads, scale, causal != 0, out, ldo, lse, workspace};
  return launch_kv_attention(v, j, reinterpret_cast<cudaStream_t>(stream));
}

qr_status qr_kv_attention_mass(const qr_kv_cache* cache, const qr_kv_seqs* seqs, const uint16_t* Q,
                               int64_t ldq, int64_t tokens, int32_t q_heads, float scale,
                               int32_t causal, const float* lse, float* mass, int64_t ld_mass,
                               qr_stream stream) {
  KvView v;
  qr_status st = make_view(cache, seqs, tokens, true, &v);
  if (st == QR_OK) st = check_queries(v, Q, ldq, q_heads, scale);
  if (st != QR_OK) return st;
  if (tokens == 0 || v.batch == 0 || v.capacity == 0) return QR_OK;
  if (lse == nullptr || mass == nullptr || ld_mass < v.capacity) return QR_ERR_INVALID_ARG;
  if (!aligned<4>(lse) || !aligned<4>(mass)) return QR_ERR_ALIGNMENT;
  KvMassJob j{Q, ldq, q_heads, scale, causal != 0, lse, mass, ld_mass};
  return launch_kv_mass(v, j, reinterpret_cast<cudaStream_t>(stream));
}

qr_status qr_kv_evict(const qr_kv_cache* cache, const qr_kv_seqs* seqs, const float* mass,
                      int64_t ld_mass, int32_t keep, int32_t recent, const int32_t* table_out,
                      float* mass_out, int32_t* kept, int32_t* lens_out, qr_stream stream) {
  KvView v;
  const qr_status st = make_view(cache, seqs, 0, false, &v);
  if (st != QR_OK) return st;
  if (keep < 1 || recent < 0 || recent > keep) return QR_ERR_INVALID_ARG;
  if (keep >= (1 << 30)) return QR_ERR_UNSUPPORTED;
  if (v.batch == 0) return QR_OK;
  if (mass == nullptr || mass_out == nullptr || kept == nullptr || lens_out == nullptr ||
      ld_mass < v.capacity)
    return QR_ERR_INVALID_ARG;
  if (lens_out == v.lens) return QR_ERR_INVALID_ARG;
  // other pages only under a table of their own: without one both would be the same
  if (table_out != nullptr && table_out == seqs->block_table) return QR_ERR_INVALID_ARG;
  if (!aligned<4>(mass) || !aligned<4>(mass_out) || !aligned<4>(kept) || !aligned<4>(lens_out) ||
      !aligned<4>(table_out))
    return QR_ERR_ALIGNMENT;
  KvEvictJob j{mass, ld_mass, keep, recent, table_out, mass_out, kept, lens_out};
  return launch_kv_evict(v, j, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
