// extern "C" entry points of libqkv.so: host-side validation, then one launch each on the
// caller's stream. Nothing here allocates, frees or synchronises. The declarations, with
// argument meaning, layout, ownership and error behaviour, are in qkv.h.
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <cstring>

#include "qkv_internal.cuh"

namespace {

using qkv::kMaxGroup;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool finite_positive(float s) { return std::isfinite(s) && s > 0.f; }
qkv_status cuda_status(cudaError_t e) { return e == cudaSuccess ? QKV_OK : QKV_ERR_CUDA; }

// Shared checks of the two write calls' token inputs.
qkv_status check_write_inputs(const void* k, const void* v, int64_t num_tokens, int num_kv_heads,
                              int head_dim, int64_t token_stride, const int64_t* slot_mapping,
                              const void* k_cache, const void* v_cache, int64_t num_slots,
                              const qkv::WritePaging* pg = nullptr) {
  if (num_tokens < 0 || num_slots < 0 || num_kv_heads < 1) return QKV_ERR_ARG;
  if (!qkv::head_dim_ok(head_dim)) return QKV_ERR_UNSUPPORTED;
  if (num_tokens == 0) return QKV_OK;
  // one warp per head row: 2 T H warps of 32 threads must fit a grid of 2^31 - 1 blocks of 256
  if (num_tokens > (int64_t(1) << 32) / num_kv_heads) return QKV_ERR_ARG;
  if (!k || !v || !k_cache || !v_cache) return QKV_ERR_ARG;
  if (pg == nullptr ? !slot_mapping : (!pg->token_seq || !pg->token_pos || !pg->block_table)) return QKV_ERR_ARG;
  if (token_stride < static_cast<int64_t>(num_kv_heads) * head_dim) return QKV_ERR_ARG;
  if (token_stride % 8 != 0 || !aligned(k, 16) || !aligned(v, 16)) return QKV_ERR_ALIGN;
  if (pg == nullptr) {
    if (!aligned(slot_mapping, 8)) return QKV_ERR_ALIGN;
  } else {
    if (pg->block_size < 1 || pg->max_blocks < 1 || pg->num_seqs < 1) return QKV_ERR_ARG;
    if (static_cast<int64_t>(pg->max_blocks) * pg->block_size > INT32_MAX) return QKV_ERR_ARG;
    if (!aligned(pg->token_seq, 4) || !aligned(pg->token_pos, 4) || !aligned(pg->block_table, 4))
      return QKV_ERR_ALIGN;
  }
  return QKV_OK;
}

}  // namespace

extern "C" {

const char* qkv_status_str(qkv_status s) {
  switch (s) {
    case QKV_OK: return "ok";
    case QKV_ERR_ARG: return "invalid argument";
    case QKV_ERR_SCALE: return "per-layer scale is not finite and positive";
    case QKV_ERR_UNSUPPORTED: return "unsupported head_dim or GQA group";
    case QKV_ERR_ALIGN: return "pointer or stride misaligned";
    case QKV_ERR_CUDA: return "CUDA launch failed";
  }
  return "unknown status";
}

}  // extern "C"

namespace {

qkv_status write_int8_impl(const void* k, const void* v, bool f16, int64_t num_tokens, int num_kv_heads,
                           int head_dim, int64_t token_stride, const int64_t* slot_mapping, qkv_format layout,
                           void* k_cache, void* v_cache, float* k_scale, float* v_scale, int64_t num_slots,
                           uint32_t* dev_status, void* stream, const qkv::WritePaging* pg = nullptr) {
  qkv_status st = check_write_inputs(k, v, num_tokens, num_kv_heads, head_dim, token_stride, slot_mapping,
                                     k_cache, v_cache, num_slots, pg);
  if (st != QKV_OK) return st;
  if (layout != QKV_INT8_SIDE && layout != QKV_INT8_INLINE) return QKV_ERR_ARG;
  const bool inl = layout == QKV_INT8_INLINE;
  if (inl && (k_scale || v_scale)) return QKV_ERR_ARG;
  if (num_tokens == 0) return QKV_OK;
  if (!inl && (!k_scale || !v_scale)) return QKV_ERR_ARG;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16)) return QKV_ERR_ALIGN;
  if (!inl && (!aligned(k_scale, 4) || !aligned(v_scale, 4))) return QKV_ERR_ALIGN;
  if (dev_status && !aligned(dev_status, 4)) return QKV_ERR_ALIGN;
  return cuda_status(qkv::launch_write_int8(k, v, f16, head_dim, num_tokens, num_kv_heads, token_stride, slot_mapping, pg,
                                            inl, k_cache, v_cache, k_scale, v_scale, num_slots, dev_status,
                                            static_cast<cudaStream_t>(stream)));
}

qkv_status write_e4m3_impl(const void* k, const void* v, bool f16, int64_t num_tokens, int num_kv_heads,
                           int head_dim, int64_t token_stride, const int64_t* slot_mapping, void* k_cache,
                           void* v_cache, float k_scale, float v_scale, int64_t num_slots, uint32_t* dev_status,
                           void* stream, const qkv::WritePaging* pg = nullptr) {
  qkv_status st = check_write_inputs(k, v, num_tokens, num_kv_heads, head_dim, token_stride, slot_mapping,
                                     k_cache, v_cache, num_slots, pg);
  if (st != QKV_OK) return st;
  if (!finite_positive(k_scale) || !finite_positive(v_scale)) return QKV_ERR_SCALE;
  if (num_tokens == 0) return QKV_OK;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16)) return QKV_ERR_ALIGN;
  if (dev_status && !aligned(dev_status, 4)) return QKV_ERR_ALIGN;
  return cuda_status(qkv::launch_write_e4m3(k, v, f16, head_dim, num_tokens, num_kv_heads, token_stride, slot_mapping, pg,
                                            k_cache, v_cache, k_scale, v_scale, num_slots, dev_status,
                                            static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

qkv_status qkv_write_int8(const void* k, const void* v, int64_t num_tokens, int num_kv_heads, int head_dim,
                          int64_t token_stride, const int64_t* slot_mapping, qkv_format layout, void* k_cache,
                          void* v_cache, float* k_scale, float* v_scale, int64_t num_slots, uint32_t* dev_status,
                          void* stream) {
  return write_int8_impl(k, v, false, num_tokens, num_kv_heads, head_dim, token_stride, slot_mapping, layout,
                         k_cache, v_cache, k_scale, v_scale, num_slots, dev_status, stream);
}

qkv_status qkv_write_int8_f16(const void* k, const void* v, int64_t num_tokens, int num_kv_heads, int head_dim,
                              int64_t token_stride, const int64_t* slot_mapping, qkv_format layout, void* k_cache,
                              void* v_cache, float* k_scale, float* v_scale, int64_t num_slots,
                              uint32_t* dev_status, void* stream) {
  return write_int8_impl(k, v, true, num_tokens, num_kv_heads, head_dim, token_stride, slot_mapping, layout,
                         k_cache, v_cache, k_scale, v_scale, num_slots, dev_status, stream);
}

qkv_status qkv_write_e4m3(const void* k, const void* v, int64_t num_tokens, int num_kv_heads, int head_dim,
                          int64_t token_stride, const int64_t* slot_mapping, void* k_cache, void* v_cache,
                          float k_scale, float v_scale, int64_t num_slots, uint32_t* dev_status, void* stream) {
  return write_e4m3_impl(k, v, false, num_tokens, num_kv_heads, head_dim, token_stride, slot_mapping, k_cache,
                         v_cache, k_scale, v_scale, num_slots, dev_status, stream);
}

qkv_status qkv_write_e4m3_f16(const void* k, const void* v, int64_t num_tokens, int num_kv_heads, int head_dim,
                              int64_t token_stride, const int64_t* slot_mapping, void* k_cache, void* v_cache,
                              float k_scale, float v_scale, int64_t num_slots, uint32_t* dev_status,
                              void* stream) {
  return write_e4m3_impl(k, v, true, num_tokens, num_kv_heads, head_dim, token_stride, slot_mapping, k_cache,
                         v_cache, k_scale, v_scale, num_slots, dev_status, stream);
}

qkv_status qkv_write_ex(const qkv_write_desc* d, void* stream) {
  if (d == nullptr || d->size != sizeof(qkv_write_desc)) return QKV_ERR_ARG;
  const bool paged = d->slot_mapping == nullptr;
  if (!paged && (d->token_seq || d->token_pos || d->block_table)) return QKV_ERR_ARG;  // one addressing only
  const qkv::WritePaging pg{d->token_seq, d->token_pos, d->block_table, d->num_seqs, d->max_blocks, d->block_size};
  const qkv::WritePaging* pp = paged ? &pg : nullptr;
  if (d->act_fp16 != 0 && d->act_fp16 != 1) return QKV_ERR_ARG;
  const bool f16 = d->act_fp16 == 1;
  if (d->fmt == QKV_INT8_SIDE || d->fmt == QKV_INT8_INLINE)
    return write_int8_impl(d->k, d->v, f16, d->num_tokens, d->num_kv_heads, d->head_dim, d->token_stride,
                           d->slot_mapping, d->fmt, d->k_cache, d->v_cache, d->k_scale, d->v_scale, d->num_slots,
                           d->dev_status, stream, pp);
  if (d->fmt == QKV_E4M3) {
    if (d->k_scale || d->v_scale) return QKV_ERR_ARG;  // per-token scale tensors belong to the int8 side layout
    return write_e4m3_impl(d->k, d->v, f16, d->num_tokens, d->num_kv_heads, d->head_dim, d->token_stride,
                           d->slot_mapping, d->k_cache, d->v_cache, d->k_scale_layer, d->v_scale_layer,
                           d->num_slots, d->dev_status, stream, pp);
  }
  return QKV_ERR_ARG;
}

qkv_status qkv_e4m3_calibrate(const void* x, int64_t n, uint32_t* amax_bits, float* scale_out, void* stream) {
  if (n < 0 || !amax_bits || !scale_out || (n > 0 && !x)) return QKV_ERR_ARG;
  if (n > 0 && !aligned(x, 16)) return QKV_ERR_ALIGN;
  if (!aligned(amax_bits, 4) || !aligned(scale_out, 4)) return QKV_ERR_ALIGN;
  return cuda_status(qkv::launch_e4m3_calibrate(x, n, amax_bits, scale_out, static_cast<cudaStream_t>(stream)));
}

qkv_status qkv_calib_histogram(const void* x, int64_t n, uint64_t* hist, void* stream) {
  if (n < 0 || n > (int64_t(1) << 40) || !hist || (n > 0 && !x)) return QKV_ERR_ARG;
  if ((n > 0 && !aligned(x, 16)) || !aligned(hist, 8)) return QKV_ERR_ALIGN;
  if (n == 0) return QKV_OK;
  return cuda_status(qkv::launch_calib_histogram(x, n, hist, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

namespace {
qkv_status calib_stats_impl(const uint64_t* hist, bool f16, float scale, qkv_calib_summary* stats, void* stream) {
  if (!hist || !stats) return QKV_ERR_ARG;
  if (!(scale == 0.f || finite_positive(scale))) return QKV_ERR_SCALE;
  if (!aligned(hist, 8) || !aligned(stats, 8)) return QKV_ERR_ALIGN;
  return cuda_status(qkv::launch_calib_stats(hist, f16, scale, stats, static_cast<cudaStream_t>(stream)));
}
}  // namespace

extern "C" {

qkv_status qkv_calib_stats(const uint64_t* hist, float scale, qkv_calib_summary* stats, void* stream) {
  return calib_stats_impl(hist, false, scale, stats, stream);
}

qkv_status qkv_calib_stats_f16(const uint64_t* hist, float scale, qkv_calib_summary* stats, void* stream) {
  return calib_stats_impl(hist, true, scale, stats, stream);
}

}  // extern "C"

namespace {

// Paged-pool arguments of qsa_gather_attn_paged (absent for qsa_gather_attn).
struct Paging {
  const int32_t* block_table;
  const int32_t* row_seq;
  int64_t num_seqs;
  int max_blocks;
  int block_size;
};

qkv_status gather_impl(const void* q, int64_t rows, int num_q_heads, int num_kv_heads, int head_dim,
                       qkv_format fmt, const void* k_cache, const void* v_cache, const float* k_scale_tok,
                       const float* v_scale_tok, float k_scale_layer, float v_scale_layer, int64_t num_slots,
                       const int32_t* topk_idx, int topk, float softmax_scale, int num_splits, float* out,
                       float* lse, float* o_part, float* lse_part, uint32_t* dev_status, void* stream,
                       const Paging* pg, uint32_t* counters = nullptr, bool q_f16 = false,
                       const int32_t* topk_len = nullptr, int engine = QSA_ENGINE_DEFAULT,
                       uint32_t* sched = nullptr, bool shard = false, int64_t slot_lo = 0) {
  if (rows < 0 || topk < 0 || num_splits < 1 || num_slots < 0) return QKV_ERR_ARG;
  // a 16-bit pool is multiplied in its own type, so it needs a query of that type
  if ((fmt == QKV_F16 && !q_f16) || (fmt == QKV_BF16 && q_f16)) return QKV_ERR_ARG;
  if (q_f16 && pg != nullptr) return QKV_ERR_ARG;
  if (pg != nullptr) {
    if (pg->num_seqs < 1 || pg->max_blocks < 1 || pg->block_size < 1) return QKV_ERR_ARG;
    if (static_cast<int64_t>(pg->max_blocks) * pg->block_size > INT32_MAX) return QKV_ERR_ARG;
    if (pg->num_seqs * pg->max_blocks > INT32_MAX) return QKV_ERR_ARG;
  }
  if (num_q_heads < 1 || num_kv_heads < 1 || num_q_heads % num_kv_heads != 0) return QKV_ERR_ARG;
  if (!qkv::head_dim_ok(head_dim) || num_q_heads / num_kv_heads > kMaxGroup) return QKV_ERR_UNSUPPORTED;
  if (fmt != QKV_BF16 && fmt != QKV_INT8_SIDE && fmt != QKV_INT8_INLINE && fmt != QKV_E4M3 && fmt != QKV_F16)
    return QKV_ERR_ARG;
  if (!std::isfinite(softmax_scale)) return QKV_ERR_ARG;
  if (fmt == QKV_E4M3 && (!finite_positive(k_scale_layer) || !finite_positive(v_scale_layer)))
    return QKV_ERR_SCALE;
  const bool side = fmt == QKV_INT8_SIDE;
  if (side != (k_scale_tok != nullptr) || side != (v_scale_tok != nullptr)) return QKV_ERR_ARG;
  if (num_splits == 1) {
    if (!out || o_part || lse_part || counters) return QKV_ERR_ARG;
  } else if (counters != nullptr) {  // fused merge: partials and the merged output
    if (!out || !o_part || !lse_part) return QKV_ERR_ARG;
    if (!aligned(counters, 4)) return QKV_ERR_ALIGN;
  } else {
    if (out || lse || !o_part || !lse_part) return QKV_ERR_ARG;
  }
  if (static_cast<int64_t>(topk) + num_splits > INT32_MAX) return QKV_ERR_ARG;
  const int64_t head_chunks = (num_q_heads / num_kv_heads + 15) / 16;  // CTAs per (row, KV head, split)
  if (rows * num_kv_heads * head_chunks * static_cast<int64_t>(num_splits) > INT32_MAX) return QKV_ERR_ARG;
  // the kernels number records (slot * H + head) in 32 bits
  if (num_slots * num_kv_heads > INT32_MAX) return QKV_ERR_UNSUPPORTED;
  if (rows == 0) return QKV_OK;
  if (!q || !k_cache || !v_cache || (topk > 0 && !topk_idx)) return QKV_ERR_ARG;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16)) return QKV_ERR_ALIGN;
  if (topk_idx && !aligned(topk_idx, 4)) return QKV_ERR_ALIGN;
  if (topk_len && !aligned(topk_len, 4)) return QKV_ERR_ALIGN;
  if (side && (!aligned(k_scale_tok, 4) || !aligned(v_scale_tok, 4))) return QKV_ERR_ALIGN;
  if ((out && !aligned(out, 16)) || (o_part && !aligned(o_part, 16))) return QKV_ERR_ALIGN;
  if ((lse && !aligned(lse, 4)) || (lse_part && !aligned(lse_part, 4))) return QKV_ERR_ALIGN;
  if (dev_status && !aligned(dev_status, 4)) return QKV_ERR_ALIGN;
  if (engine == QSA_ENGINE_PERSISTENT) {
    if (sched == nullptr) return QKV_ERR_ARG;
    if (!aligned(sched, 4)) return QKV_ERR_ALIGN;
  }
  if (shard && (slot_lo < 0 || slot_lo > INT32_MAX || pg != nullptr)) return QKV_ERR_ARG;
  if (pg != nullptr) {
    if (!pg->block_table || !pg->row_seq) return QKV_ERR_ARG;
    if (!aligned(pg->block_table, 4) || !aligned(pg->row_seq, 4)) return QKV_ERR_ALIGN;
  }

  qkv::GatherArgs a;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k_cache = static_cast<const uint8_t*>(k_cache);
  a.v_cache = static_cast<const uint8_t*>(v_cache);
  a.k_scale_tok = k_scale_tok;
  a.v_scale_tok = v_scale_tok;
  a.k_scale_layer = k_scale_layer;
  a.v_scale_layer = v_scale_layer;
  a.num_slots = num_slots;
  a.topk_idx = topk_idx;
  a.topk_len = topk_len;
  a.rows = rows;
  a.num_q_heads = num_q_heads;
  a.num_kv_heads = num_kv_heads;
  a.head_dim = head_dim;
  a.topk = topk;
  a.num_splits = num_splits;
  a.softmax_scale = softmax_scale;
  a.out = out;
  a.lse = lse;
  a.o_part = o_part;
  a.lse_part = lse_part;
  a.dev_status = dev_status;
  a.counters = num_splits > 1 ? counters : nullptr;
  a.sched = engine == QSA_ENGINE_PERSISTENT ? sched : nullptr;
  a.shard = shard;
  a.slot_lo = shard ? slot_lo : 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (pg != nullptr) {
    a.block_table = pg->block_table;
    a.row_seq = pg->row_seq;
    a.num_seqs = pg->num_seqs;
    a.max_blocks = pg->max_blocks;
    a.block_size = pg->block_size;
    if (engine == QSA_ENGINE_TCGEN05) return QKV_ERR_UNSUPPORTED;
    switch (fmt) {
      case QKV_BF16: return cuda_status(qkv::launch_gather_paged_bf16(a, s));
      case QKV_INT8_SIDE: return cuda_status(qkv::launch_gather_paged_int8_side(a, s));
      case QKV_INT8_INLINE: return cuda_status(qkv::launch_gather_paged_int8_inline(a, s));
      case QKV_E4M3: return cuda_status(qkv::launch_gather_paged_e4m3(a, s));
    }
    return QKV_ERR_ARG;
  }
  if (q_f16) {
    if (engine == QSA_ENGINE_TCGEN05) return QKV_ERR_UNSUPPORTED;
    switch (fmt) {
      case QKV_INT8_SIDE: return cuda_status(qkv::launch_gather_f16q_int8_side(a, s));
      case QKV_INT8_INLINE: return cuda_status(qkv::launch_gather_f16q_int8_inline(a, s));
      case QKV_E4M3: return cuda_status(qkv::launch_gather_f16q_e4m3(a, s));
      case QKV_F16: return cuda_status(qkv::launch_gather_f16q_f16(a, s));
      default: return QKV_ERR_ARG;
    }
  }
  if (engine == QSA_ENGINE_TCGEN05) {
    if (fmt != QKV_INT8_SIDE || head_dim != 256 || num_q_heads / num_kv_heads > 16 || a.counters != nullptr ||
        shard)
      return QKV_ERR_UNSUPPORTED;
    return cuda_status(qkv::launch_umma_int8_side(a, s));
  }
  switch (fmt) {
    case QKV_BF16: return cuda_status(qkv::launch_gather_bf16(a, s));
    case QKV_INT8_SIDE: return cuda_status(qkv::launch_gather_int8_side(a, s));
    case QKV_INT8_INLINE: return cuda_status(qkv::launch_gather_int8_inline(a, s));
    case QKV_E4M3: return cuda_status(qkv::launch_gather_e4m3(a, s));
  }
  return QKV_ERR_ARG;
}

}  // namespace

extern "C" {

qkv_status qsa_gather_attn(const void* q, int64_t rows, int num_q_heads, int num_kv_heads, int head_dim,
                           qkv_format fmt, const void* k_cache, const void* v_cache, const float* k_scale_tok,
                           const float* v_scale_tok, float k_scale_layer, float v_scale_layer, int64_t num_slots,
                           const int32_t* topk_idx, int topk, float softmax_scale, int num_splits, float* out,
                           float* lse, float* o_part, float* lse_part, uint32_t* dev_status, void* stream) {
  return gather_impl(q, rows, num_q_heads, num_kv_heads, head_dim, fmt, k_cache, v_cache, k_scale_tok, v_scale_tok,
                     k_scale_layer, v_scale_layer, num_slots, topk_idx, topk, softmax_scale, num_splits, out, lse,
                     o_part, lse_part, dev_status, stream, nullptr);
}

qkv_status qsa_gather_attn_varlen(const void* q, int64_t rows, int num_q_heads, int num_kv_heads, int head_dim,
                                  qkv_format fmt, const void* k_cache, const void* v_cache,
                                  const float* k_scale_tok, const float* v_scale_tok, float k_scale_layer,
                                  float v_scale_layer, int64_t num_slots, const int32_t* topk_idx, int topk,
                                  const int32_t* topk_len, float softmax_scale, int num_splits, float* out,
                                  float* lse, float* o_part, float* lse_part, uint32_t* dev_status, void* stream) {
  if (rows > 0 && topk_len == nullptr) return QKV_ERR_ARG;
  return gather_impl(q, rows, num_q_heads, num_kv_heads, head_dim, fmt, k_cache, v_cache, k_scale_tok, v_scale_tok,
                     k_scale_layer, v_scale_layer, num_slots, topk_idx, topk, softmax_scale, num_splits, out, lse,
                     o_part, lse_part, dev_status, stream, nullptr, nullptr, false, topk_len);
}

qkv_status qsa_gather_attn_f16(const void* q, int64_t rows, int num_q_heads, int num_kv_heads, int head_dim,
                               qkv_format fmt, const void* k_cache, const void* v_cache, const float* k_scale_tok,
                               const float* v_scale_tok, float k_scale_layer, float v_scale_layer,
                               int64_t num_slots, const int32_t* topk_idx, int topk, float softmax_scale,
                               int num_splits, float* out, float* lse, float* o_part, float* lse_part,
                               uint32_t* dev_status, void* stream) {
  return gather_impl(q, rows, num_q_heads, num_kv_heads, head_dim, fmt, k_cache, v_cache, k_scale_tok, v_scale_tok,
                     k_scale_layer, v_scale_layer, num_slots, topk_idx, topk, softmax_scale, num_splits, out, lse,
                     o_part, lse_part, dev_status, stream, nullptr, nullptr, true);
}

qkv_status qsa_gather_attn_paged(const void* q, int64_t rows, int num_q_heads, int num_kv_heads, int head_dim,
                                 qkv_format fmt, const void* k_cache, const void* v_cache,
                                 const float* k_scale_tok, const float* v_scale_tok, float k_scale_layer,
                                 float v_scale_layer, int64_t num_slots, const int32_t* block_table,
                                 int64_t num_seqs, int max_blocks, int block_size, const int32_t* row_seq,
                                 const int32_t* topk_pos, int topk, float softmax_scale, int num_splits,
                                 float* out, float* lse, float* o_part, float* lse_part, uint32_t* dev_status,
                                 void* stream) {
  const Paging pg{block_table, row_seq, num_seqs, max_blocks, block_size};
  return gather_impl(q, rows, num_q_heads, num_kv_heads, head_dim, fmt, k_cache, v_cache, k_scale_tok, v_scale_tok,
                     k_scale_layer, v_scale_layer, num_slots, topk_pos, topk, softmax_scale, num_splits, out, lse,
                     o_part, lse_part, dev_status, stream, &pg);
}

qkv_status qsa_gather_attn_splitk_fused(const void* q, int64_t rows, int num_q_heads, int num_kv_heads,
                                        int head_dim, qkv_format fmt, const void* k_cache, const void* v_cache,
                                        const float* k_scale_tok, const float* v_scale_tok, float k_scale_layer,
                                        float v_scale_layer, int64_t num_slots, const int32_t* topk_idx, int topk,
                                        float softmax_scale, int num_splits, float* out, float* lse,
                                        float* o_part, float* lse_part, uint32_t* counters, uint32_t* dev_status,
                                        void* stream) {
  if (num_splits == 1)  // unsplit: the kernel writes out / lse itself; no workspace is touched
    return gather_impl(q, rows, num_q_heads, num_kv_heads, head_dim, fmt, k_cache, v_cache, k_scale_tok,
                       v_scale_tok, k_scale_layer, v_scale_layer, num_slots, topk_idx, topk, softmax_scale, 1, out,
                       lse, nullptr, nullptr, dev_status, stream, nullptr);
  if (num_splits > 1 && counters == nullptr) return QKV_ERR_ARG;
  return gather_impl(q, rows, num_q_heads, num_kv_heads, head_dim, fmt, k_cache, v_cache, k_scale_tok, v_scale_tok,
                     k_scale_layer, v_scale_layer, num_slots, topk_idx, topk, softmax_scale, num_splits, out, lse,
                     o_part, lse_part, dev_status, stream, nullptr, counters);
}

qkv_status qsa_suggest_num_splits(qkv_format fmt, int64_t rows, int num_q_heads, int num_kv_heads, int topk,
                                  int* num_splits) {
  if (!num_splits || rows < 0 || topk < 0) return QKV_ERR_ARG;
  if (num_q_heads < 1 || num_kv_heads < 1 || num_q_heads % num_kv_heads != 0) return QKV_ERR_ARG;
  if (num_q_heads / num_kv_heads > kMaxGroup) return QKV_ERR_UNSUPPORTED;
  int per_sm = 0;
  cudaError_t e = cudaErrorInvalidValue;
  switch (fmt) {
    case QKV_BF16:
    case QKV_F16: e = qkv::gather_ctas_per_sm_bf16(&per_sm); break;  // the same 16-bit ring
    case QKV_INT8_SIDE: e = qkv::gather_ctas_per_sm_int8_side(&per_sm); break;
    case QKV_INT8_INLINE: e = qkv::gather_ctas_per_sm_int8_inline(&per_sm); break;
    case QKV_E4M3: e = qkv::gather_ctas_per_sm_e4m3(&per_sm); break;
    default: return QKV_ERR_ARG;
  }
  if (e != cudaSuccess) return QKV_ERR_CUDA;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return QKV_ERR_CUDA;
  const int64_t units = rows * num_kv_heads * ((num_q_heads / num_kv_heads + 15) / 16);  // CTAs per split
  // one wave at up to two CTAs per SM: on the long-context and split-K workloads fewer, longer
  // CTAs per SM beat a third resident CTA (its prologue, epilogue and merge contend)
  const int64_t slots = static_cast<int64_t>(sms) * (per_sm < 1 ? 1 : (per_sm > 2 ? 2 : per_sm));
  int64_t p = units > 0 ? slots / units : 1;
  const int64_t cap = (static_cast<int64_t>(topk) + 127) / 128;  // at least 128 keys (8 tiles) per split
  if (p > cap) p = cap;
  if (p < 1) p = 1;
  *num_splits = static_cast<int>(p);
  return QKV_OK;
}

qkv_status qsa_gather_attn_ex(const qsa_gather_desc* d, void* stream) {
  if (d == nullptr || d->size != sizeof(qsa_gather_desc)) return QKV_ERR_ARG;
  if (d->q_fp16 != 0 && d->q_fp16 != 1) return QKV_ERR_ARG;
  if (d->engine != QSA_ENGINE_DEFAULT && d->engine != QSA_ENGINE_TCGEN05 && d->engine != QSA_ENGINE_PERSISTENT)
    return QKV_ERR_ARG;
  if (d->shard != 0 && d->shard != 1) return QKV_ERR_ARG;
  const bool paged = d->block_table != nullptr;
  if (!paged && d->row_seq != nullptr) return QKV_ERR_ARG;
  const Paging pg{d->block_table, d->row_seq, d->num_seqs, d->max_blocks, d->block_size};
  uint32_t* counters = d->num_splits > 1 ? d->counters : nullptr;  // an unsplit call merges nothing
  return gather_impl(d->q, d->rows, d->num_q_heads, d->num_kv_heads, d->head_dim, d->fmt, d->k_cache, d->v_cache,
                     d->k_scale_tok, d->v_scale_tok, d->k_scale_layer, d->v_scale_layer, d->num_slots, d->topk_idx,
                     d->topk, d->softmax_scale, d->num_splits, d->out, d->lse, d->o_part, d->lse_part, d->dev_status,
                     stream, paged ? &pg : nullptr, counters, d->q_fp16 != 0, d->topk_len, d->engine, d->sched,
                     d->shard != 0, d->slot_lo);
}

qkv_status qsa_splitk_merge(const float* o_part, const float* lse_part, int64_t rows, int num_q_heads,
                            int head_dim, int num_splits, float v_scale_post, float* out, float* lse,
                            void* stream) {
  if (rows < 0 || num_q_heads < 1 || num_splits < 1) return QKV_ERR_ARG;
  if (!qkv::head_dim_ok(head_dim)) return QKV_ERR_UNSUPPORTED;
  if (!std::isfinite(v_scale_post)) return QKV_ERR_ARG;
  if (rows == 0) return QKV_OK;
  if (rows > (int64_t(1) << 32) / num_q_heads) return QKV_ERR_ARG;  // one warp per (row, head): one grid
  if (!o_part || !lse_part || !out) return QKV_ERR_ARG;
  if (!aligned(o_part, 16) || !aligned(out, 16) || !aligned(lse_part, 4) || (lse && !aligned(lse, 4)))
    return QKV_ERR_ALIGN;
  return cuda_status(qkv::launch_splitk_merge(o_part, lse_part, rows, num_q_heads, head_dim, num_splits, v_scale_post,
                                              out, lse, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

namespace {

// The descriptor's paged or slot-id addressing, and the inputs of an append. axes: token_pos belongs to the paged addressing.
qkv_status check_append(const qkv_append_desc* d, bool axes = false) {
  const bool paged = d->slot_mapping == nullptr;
  if (!paged && (d->token_seq || d->block_table || (axes && d->token_pos))) return QKV_ERR_ARG;  // one addressing only
  const bool f16 = d->act_fp16 == 1;
  switch (d->fmt) {
    case QKV_BF16: if (f16) return QKV_ERR_ARG; break;  // a 16-bit pool takes activations of its own type
    case QKV_F16: if (!f16) return QKV_ERR_ARG; break;
    case QKV_INT8_SIDE:
    case QKV_INT8_INLINE:
    case QKV_E4M3: break;
    default: return QKV_ERR_ARG;
  }
  if (d->num_q_heads < 0 || (d->q == nullptr) != (d->q_out == nullptr)) return QKV_ERR_ARG;
  if (d->q != nullptr && d->num_q_heads < 1) return QKV_ERR_ARG;
  const int hq = d->q != nullptr ? d->num_q_heads : 0;
  const qkv::WritePaging pg{d->token_seq, d->token_pos, d->block_table, d->num_seqs, d->max_blocks, d->block_size};
  qkv_status st = check_write_inputs(d->k, d->v, d->num_tokens, d->num_kv_heads, d->head_dim, d->kv_stride,
                                     d->slot_mapping, d->k_cache, d->v_cache, d->num_slots, paged ? &pg : nullptr);
  if (st != QKV_OK) return st;
  if (d->num_positions < 0 || d->rotary_dim < 16 || d->rotary_dim % 16 != 0 || d->rotary_dim > d->head_dim)
    return QKV_ERR_ARG;
  if (d->interleaved != 0 && d->interleaved != 1) return QKV_ERR_ARG;
  const bool side = d->fmt == QKV_INT8_SIDE;
  if (side ? (!d->k_scale || !d->v_scale) && d->num_tokens > 0 : d->k_scale || d->v_scale) return QKV_ERR_ARG;
  if (d->fmt == QKV_E4M3 && (!finite_positive(d->k_scale_layer) || !finite_positive(d->v_scale_layer)))
    return QKV_ERR_SCALE;
  if (d->num_tokens == 0) return QKV_OK;
  // A launch of one row per lane group has at most append.cuh's kSmallWarps warps; one of four rows T ceil(rows / 4) or
  // fewer, which is at most T rows / 2 (rows is 3 or more, or 2: one unit), so 2^32 warps, 2^30 blocks of four.
  const int64_t rows = static_cast<int64_t>(hq) + 2 * static_cast<int64_t>(d->num_kv_heads);
  if (rows > INT32_MAX || d->num_tokens > (int64_t(1) << 33) / rows) return QKV_ERR_ARG;
  if ((!axes && !d->token_pos) || !d->cos_sin) return QKV_ERR_ARG;
  if (hq > 0) {
    const int64_t row = static_cast<int64_t>(hq) * d->head_dim;
    if (d->q_stride < row || d->q_out_stride < row) return QKV_ERR_ARG;
    if (d->q_stride % 8 != 0 || d->q_out_stride % 8 != 0 || !aligned(d->q, 16) || !aligned(d->q_out, 16))
      return QKV_ERR_ALIGN;
  }
  if (!aligned(d->token_pos, 4) || !aligned(d->cos_sin, 16)) return QKV_ERR_ALIGN;
  if (!aligned(d->k_cache, 16) || !aligned(d->v_cache, 16)) return QKV_ERR_ALIGN;
  if (side && (!aligned(d->k_scale, 4) || !aligned(d->v_scale, 4))) return QKV_ERR_ALIGN;
  if (d->dev_status && !aligned(d->dev_status, 4)) return QKV_ERR_ALIGN;
  return QKV_OK;
}

// A checked descriptor's fields.
qkv::AppendArgs append_args(const qkv_append_desc* d) {
  qkv::AppendArgs a = {};
  a.q = static_cast<const uint16_t*>(d->q);
  a.q_out = static_cast<uint16_t*>(d->q_out);
  a.k = static_cast<const uint16_t*>(d->k);
  a.v = static_cast<const uint16_t*>(d->v);
  a.num_tokens = d->num_tokens;
  a.num_q_heads = d->q != nullptr ? d->num_q_heads : 0;
  a.num_kv_heads = d->num_kv_heads;
  a.head_dim = d->head_dim;
  a.q_stride = d->q_stride;
  a.q_out_stride = d->q_out_stride;
  a.kv_stride = d->kv_stride;
  a.cos_sin = d->cos_sin;
  a.num_positions = d->num_positions;
  a.rotary_dim = d->rotary_dim;
  a.interleaved = d->interleaved == 1;
  a.token_pos = d->token_pos;
  a.slot_mapping = d->slot_mapping;
  a.paging = qkv::WritePaging{d->token_seq, d->token_pos, d->block_table, d->num_seqs, d->max_blocks, d->block_size};
  a.k_cache = static_cast<uint8_t*>(d->k_cache);
  a.v_cache = static_cast<uint8_t*>(d->v_cache);
  a.k_scale = d->k_scale;
  a.v_scale = d->v_scale;
  a.k_scale_layer = d->k_scale_layer;
  a.v_scale_layer = d->v_scale_layer;
  a.num_slots = d->num_slots;
  a.dev_status = d->dev_status;
  return a;
}

// Positions of several axes, and each pair's axis packed from the host's array. The positions' pointer is checked
// where there are tokens.
qkv_status check_axes(const int32_t* axis_pos, int num_axes, const uint8_t* pair_axis, int rotary_dim, int64_t num_tokens,
                      qkv::RopeAxes* out) {
  if (num_axes < 1 || num_axes > qkv::kMaxAxes) return QKV_ERR_ARG;
  *out = qkv::RopeAxes{axis_pos, num_axes, {}};
  for (int i = 0; pair_axis != nullptr && i < rotary_dim / 2; ++i) {
    if (pair_axis[i] >= num_axes) return QKV_ERR_ARG;
    out->pair_axis[i >> 4] |= static_cast<uint32_t>(pair_axis[i]) << (2 * (i & 15));
  }
  if (num_tokens > 0 && !axis_pos) return QKV_ERR_ARG;
  return aligned(axis_pos, 4) ? QKV_OK : QKV_ERR_ALIGN;
}

}  // namespace

extern "C" {

qkv_status qkv_append_rope(const qkv_append_desc* d, void* stream) {
  if (d == nullptr || d->size != sizeof(qkv_append_desc)) return QKV_ERR_ARG;
  if (d->act_fp16 != 0 && d->act_fp16 != 1) return QKV_ERR_ARG;
  const qkv_status st = check_append(d);
  if (st != QKV_OK || d->num_tokens == 0) return st;
  return cuda_status(qkv::launch_append_rope(append_args(d), d->fmt, d->act_fp16 == 1, static_cast<cudaStream_t>(stream)));
}

qkv_status qkv_append_axes(const qkv_append_axes_desc* d, void* stream) {
  if (d == nullptr || d->append.size != sizeof(qkv_append_axes_desc)) return QKV_ERR_ARG;
  const qkv_append_desc* p = &d->append;
  if (p->act_fp16 != 0 && p->act_fp16 != 1) return QKV_ERR_ARG;
  qkv_status st = check_append(p, true);
  if (st != QKV_OK) return st;
  qkv::RopeAxes axes;
  st = check_axes(d->axis_pos, d->num_axes, d->pair_axis, p->rotary_dim, p->num_tokens, &axes);
  if (st != QKV_OK || p->num_tokens == 0) return st;
  qkv::AppendArgs a = append_args(p);
  a.axes = axes;
  return cuda_status(qkv::launch_append_axes(a, p->fmt, p->act_fp16 == 1, static_cast<cudaStream_t>(stream)));
}

qkv_status qkv_read(const qkv_read_desc* d, void* stream) {
  if (d == nullptr || d->size != sizeof(qkv_read_desc)) return QKV_ERR_ARG;
  if (d->num_tokens < 0 || d->num_slots < 0 || d->num_kv_heads < 1) return QKV_ERR_ARG;
  if (!qkv::head_dim_ok(d->head_dim)) return QKV_ERR_UNSUPPORTED;
  if (d->fmt != QKV_BF16 && d->fmt != QKV_INT8_SIDE && d->fmt != QKV_INT8_INLINE && d->fmt != QKV_E4M3 && d->fmt != QKV_F16)
    return QKV_ERR_ARG;
  if (d->out_type != QKV_OUT_BF16 && d->out_type != QKV_OUT_F16 && d->out_type != QKV_OUT_F32) return QKV_ERR_ARG;
  if (d->fmt == QKV_E4M3 && (!finite_positive(d->k_scale_layer) || !finite_positive(d->v_scale_layer))) return QKV_ERR_SCALE;
  const bool side = d->fmt == QKV_INT8_SIDE, paged = d->slot_mapping == nullptr;
  if (!side && (d->k_scale || d->v_scale)) return QKV_ERR_ARG;
  if (!paged && (d->token_seq || d->token_pos || d->block_table)) return QKV_ERR_ARG;  // one addressing only
  // 2 T H rows, four per warp or more in large launches, four warps per block
  if (d->num_tokens > (int64_t(1) << 32) / d->num_kv_heads) return QKV_ERR_ARG;
  qkv::RopeAxes axes = {};
  if (d->cos_sin != nullptr) {
    if (d->num_positions < 0 || d->rotary_dim < 16 || d->rotary_dim % 16 != 0 || d->rotary_dim > d->head_dim) return QKV_ERR_ARG;
    if (d->interleaved != 0 && d->interleaved != 1) return QKV_ERR_ARG;
    const qkv_status st = check_axes(d->axis_pos, d->num_axes, d->pair_axis, d->rotary_dim, d->num_tokens, &axes);
    if (st != QKV_OK) return st;
    if (!aligned(d->cos_sin, 16)) return QKV_ERR_ALIGN;
  } else if (d->axis_pos != nullptr) {
    return QKV_ERR_ARG;  // positions without a table
  }
  if (d->num_tokens == 0) return QKV_OK;
  if (!d->k_cache || !d->v_cache || (!d->k_out && !d->v_out)) return QKV_ERR_ARG;
  if (side && (!d->k_scale || !d->v_scale)) return QKV_ERR_ARG;
  if (paged) {
    if (!d->token_seq || !d->token_pos || !d->block_table) return QKV_ERR_ARG;
    if (d->block_size < 1 || d->max_blocks < 1 || d->num_seqs < 1) return QKV_ERR_ARG;
    if (static_cast<int64_t>(d->max_blocks) * d->block_size > INT32_MAX) return QKV_ERR_ARG;
    if (!aligned(d->token_seq, 4) || !aligned(d->token_pos, 4) || !aligned(d->block_table, 4)) return QKV_ERR_ALIGN;
  } else if (!aligned(d->slot_mapping, 8)) {
    return QKV_ERR_ALIGN;
  }
  if (d->out_stride < static_cast<int64_t>(d->num_kv_heads) * d->head_dim) return QKV_ERR_ARG;
  if (d->out_stride % 8 != 0 || !aligned(d->k_out, 16) || !aligned(d->v_out, 16)) return QKV_ERR_ALIGN;
  if (!aligned(d->k_cache, 16) || !aligned(d->v_cache, 16)) return QKV_ERR_ALIGN;
  if (side && (!aligned(d->k_scale, 4) || !aligned(d->v_scale, 4))) return QKV_ERR_ALIGN;
  if (!aligned(d->dev_status, 4)) return QKV_ERR_ALIGN;
  qkv::ReadArgs a = {};
  a.k_cache = static_cast<const uint8_t*>(d->k_cache);
  a.v_cache = static_cast<const uint8_t*>(d->v_cache);
  a.k_scale = d->k_scale;
  a.v_scale = d->v_scale;
  a.k_scale_layer = d->k_scale_layer;
  a.v_scale_layer = d->v_scale_layer;
  a.num_slots = d->num_slots;
  a.num_tokens = d->num_tokens;
  a.num_kv_heads = d->num_kv_heads;
  a.head_dim = d->head_dim;
  a.slot_mapping = d->slot_mapping;
  a.paging = qkv::WritePaging{d->token_seq, d->token_pos, d->block_table, d->num_seqs, d->max_blocks, d->block_size};
  a.k_out = d->k_out;
  a.v_out = d->v_out;
  a.out_stride = d->out_stride;
  a.out_type = d->out_type;
  a.cos_sin = d->cos_sin;
  a.num_positions = d->num_positions;
  a.rotary_dim = d->rotary_dim;
  a.interleaved = d->interleaved == 1;
  a.axes = axes;
  a.dev_status = d->dev_status;
  return cuda_status(qkv::launch_read(a, d->fmt, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

namespace {

int64_t ceil_div(int64_t x, int64_t y) { return (x + y - 1) / y; }

// SMs of the current device, 0: none.
int sm_count() {
  static std::atomic<int> count[64] = {};
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  n = count[dev].load(std::memory_order_relaxed);
  if (n == 0 && cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess)
    count[dev].store(n, std::memory_order_relaxed);
  return n;
}

// K bytes that tiles of 16 pairs would read above which the prefix runs on tcgen05: its tiles read them once per
// 128 pairs or more, but a call costs some 6 us before the first key and after the last. In us, mma.sync | tcgen05:
// one KV head of 256, int8: 16 pairs at 12 MB 28 | 31, at 20 MB 37 | 35, at 32 MB 58 | 44; 128 pairs 18 | 21, 28 | 29,
// 39 | 29. 8 heads of 128, e4m3: 32 pairs at 6 MB 15 | 16, at 12 MB 20 | 17, at 20 MB 26 | 19. 4 heads of 128, bf16:
// 32 pairs at 12 MB 14 | 17, at 20 MB 19 | 17; 2048 pairs 23 | 19, 25 | 20. 2 heads of 256, fp16: 32 pairs at 12 MB
// 22 | 22, at 20 MB 33 | 21.
constexpr int64_t kUmmaMinBytes = 16 << 20;

// How a shared-prefix call is cut into key ranges: up to 16 CTAs per SM, so that ragged rows balance (64 rows x 64
// heads of 0 to 8192 e4m3 keys: 118 us, 121 with 8, 130 with 4), but none with fewer than 512 keys, since a CTA's
// start and its join cost as much as about 300 (8 x 5 drafts behind 126976 int8 keys: 131 us, 135 with 256, 144
// with 1024; one row of 65536: 31 us, 40, 37). Ranges of 64, 128 or 256 keys where all CTAs then run at once (with
// a tenth to spare) and the merge has at most 32 ranges to join. In us, ranges of at least 512 | 256 | 128 | 64:
// one row x 16 heads of 256, int8, 500 keys 17 | 13 | 11 | 9, 2000 keys 19 | 14 | 11 | 11, 8192 keys 20 | 15 | 15
// | 17; one row x 64 heads (8 KV heads) of 128, bf16, 1000 keys 14 | 11 | 8 | 7, 8192 keys 15 | 13 | 18 | 22; four
// such rows, e4m3, 1000 keys 13 | 10 | 9 | 9, 4096 keys 15 | 14 | 18 | 26.
struct PrefixPlan {
  int prefix_parts, own_parts, prefix_chunk;
  int umma_cg, umma_pairs, umma_ptiles;
  uint32_t umma_blocks, umma_teams, umma_share, umma_extra;
  int64_t ptiles, otiles;  // mma.sync tiles of the prefix (none: it runs on tcgen05) and of the rows' own keys
  int parts() const { return prefix_parts + own_parts; }
  int64_t rows_heads;
  int head_dim;
  // partial outputs, then partial log-sum-exps; a single part writes the output itself
  size_t o_bytes() const { return parts() > 1 ? static_cast<size_t>(parts()) * rows_heads * head_dim * 4 : 0; }
  size_t bytes() const { return o_bytes() + (parts() > 1 ? static_cast<size_t>(parts()) * rows_heads * 4 : 0); }
};

qkv_status check_prefix_shape(qkv_format fmt, int64_t rows, int num_q_heads, int num_kv_heads, int head_dim,
                              int prefix_len, int max_row_len) {
  if (rows < 0 || prefix_len < 0 || max_row_len < prefix_len || max_row_len > (1 << 30)) return QKV_ERR_ARG;
  if (num_q_heads < 1 || num_kv_heads < 1 || num_q_heads % num_kv_heads != 0) return QKV_ERR_ARG;
  if (!qkv::head_dim_ok(head_dim) || num_q_heads / num_kv_heads > kMaxGroup) return QKV_ERR_UNSUPPORTED;
  if (fmt != QKV_BF16 && fmt != QKV_INT8_SIDE && fmt != QKV_INT8_INLINE && fmt != QKV_E4M3 && fmt != QKV_F16)
    return QKV_ERR_ARG;
  if (rows > INT32_MAX / num_q_heads) return QKV_ERR_ARG;  // (row, head) pairs are numbered in 32 bits
  return QKV_OK;
}

int64_t row_bytes_of(qkv_format fmt, int head_dim) { return fmt == QKV_BF16 || fmt == QKV_F16 ? 2 * head_dim : head_dim; }

// CTAs of mma.sync tiles that are resident at a time.
int64_t resident_slots(int64_t row_bytes, int sms) { return static_cast<int64_t>(sms) * (row_bytes == 128 ? 3 : row_bytes == 256 ? 2 : 1); }

// Ranges that the keys of mma.sync tiles are cut into, as PrefixPlan's comment says.
int key_parts(int64_t tiles, int keys, int64_t row_bytes, int sms) {
  if (keys <= 0 || tiles <= 0) return 0;
  const int64_t slots = resident_slots(row_bytes, sms);
  int least = 64;
  while (least < 512 && (ceil_div(keys, least) > 32 || 10 * tiles * ceil_div(keys, least) > 9 * slots)) least *= 2;
  const int64_t want = ceil_div(16 * static_cast<int64_t>(sms), tiles), most = ceil_div(keys, least);
  return static_cast<int>(want < most ? want : most);
}

qkv_status plan_prefix(qkv_format fmt, int64_t rows, int num_q_heads, int num_kv_heads, int head_dim, int prefix_len,
                       int max_row_len, PrefixPlan* p) {
  const int sms = sm_count();
  if (sms < 1) return QKV_ERR_CUDA;
  const int G = num_q_heads / num_kv_heads, own = max_row_len - prefix_len;
  p->rows_heads = rows * num_q_heads;
  p->head_dim = head_dim;
  p->ptiles = ceil_div(rows * G, 16) * num_kv_heads;
  p->otiles = rows * ceil_div(G, 16) * num_kv_heads;
  const int64_t row_bytes = row_bytes_of(fmt, head_dim);
  auto parts_of = [&](int64_t tiles, int keys) { return key_parts(tiles, keys, row_bytes, sms); };
  p->prefix_parts = parts_of(p->ptiles, prefix_len);
  p->prefix_chunk = 0;
  if (p->prefix_parts > 0) {
    p->prefix_chunk = static_cast<int>(ceil_div(ceil_div(prefix_len, p->prefix_parts), 64) * 64);
    p->prefix_parts = static_cast<int>(ceil_div(prefix_len, p->prefix_chunk));
  }
  p->umma_cg = 0, p->umma_pairs = 0, p->umma_ptiles = 0;
  p->umma_blocks = 0, p->umma_teams = 0, p->umma_share = 0, p->umma_extra = 0;
  if (prefix_len > 0 && p->ptiles > kUmmaMinBytes / (prefix_len * row_bytes)) {
    // Two SMs per team where their tiles (512 pairs of 128-wide heads, 256 of 256-wide ones) are at least half
    // full. In us, one SM | two: 8 heads of 128, e4m3, 65536 keys, 256 pairs 99 | 118, 512 pairs 180 | 145; 4
    // heads of 128, bf16, 256 pairs 64.6 | 65.5, 512 pairs 113 | 81; one head of 256, int8, 128 pairs 40 | 38, 192
    // pairs 44 | 40, 256 pairs 46 | 42.
    p->umma_cg = rows * G > (head_dim == 128 ? 256 : 128) ? 2 : 1;
    p->umma_pairs = p->umma_cg == 1 ? 128 : head_dim == 128 ? 512 : 256;
    const int keys = head_dim == 256 && p->umma_cg == 1 ? 64 : 128;
    const int64_t nb = ceil_div(prefix_len, keys), pt = ceil_div(rows * G, p->umma_pairs);
    const int64_t total = pt * num_kv_heads * nb, teams = total < sms / p->umma_cg ? total : sms / p->umma_cg;
    if (total > INT32_MAX) return QKV_ERR_UNSUPPORTED;  // units are numbered in 32 bits
    p->umma_ptiles = static_cast<int>(pt);
    p->umma_blocks = static_cast<uint32_t>(nb);
    p->umma_teams = static_cast<uint32_t>(teams);
    p->umma_share = static_cast<uint32_t>(total / teams);
    p->umma_extra = static_cast<uint32_t>(total % teams);
    // a tile's nb units touch at most this many ranges
    p->prefix_parts = static_cast<int>(ceil_div(nb, p->umma_share) + 1);
    p->ptiles = 0;
  }
  p->own_parts = parts_of(p->otiles, own);
  // tiles of 8 pairs: at most twice as many
  if (2 * p->ptiles * p->prefix_parts + p->otiles * p->own_parts > INT32_MAX) return QKV_ERR_ARG;
  return QKV_OK;
}

cudaError_t launch_prefix_umma(const qkv::PrefixArgs& a, qkv_format fmt, cudaStream_t s) {
  switch (fmt) {
    case QKV_BF16: return qkv::launch_prefix_umma_bf16(a, s);
    case QKV_F16: return qkv::launch_prefix_umma_f16(a, s);
    case QKV_INT8_SIDE: return qkv::launch_prefix_umma_int8_side(a, s);
    case QKV_INT8_INLINE: return qkv::launch_prefix_umma_int8_inline(a, s);
    case QKV_E4M3: return qkv::launch_prefix_umma_e4m3(a, s);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_prefix_mma(const qkv::PrefixArgs& a, qkv_format fmt, bool overlaps, cudaStream_t s) {
  switch (fmt) {
    case QKV_BF16: return qkv::launch_prefix_mma_bf16(a, overlaps, s);
    case QKV_F16: return qkv::launch_prefix_mma_f16(a, overlaps, s);
    case QKV_INT8_SIDE: return qkv::launch_prefix_mma_int8_side(a, overlaps, s);
    case QKV_INT8_INLINE: return qkv::launch_prefix_mma_int8_inline(a, overlaps, s);
    case QKV_E4M3: return qkv::launch_prefix_mma_e4m3(a, overlaps, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

extern "C" {

qkv_status qkv_prefix_attn_workspace(qkv_format fmt, int64_t rows, int num_q_heads, int num_kv_heads, int head_dim,
                                     int prefix_len, int max_row_len, size_t* bytes) {
  if (!bytes) return QKV_ERR_ARG;
  qkv_status st = check_prefix_shape(fmt, rows, num_q_heads, num_kv_heads, head_dim, prefix_len, max_row_len);
  if (st != QKV_OK) return st;
  PrefixPlan p;
  st = plan_prefix(fmt, rows, num_q_heads, num_kv_heads, head_dim, prefix_len, max_row_len, &p);
  if (st == QKV_OK) *bytes = p.bytes();
  return st;
}

qkv_status qkv_prefix_attn(const qkv_prefix_desc* d, void* stream) {
  if (d == nullptr || d->size != sizeof(qkv_prefix_desc)) return QKV_ERR_ARG;
  if (d->q_fp16 != 0 && d->q_fp16 != 1) return QKV_ERR_ARG;
  qkv_status st = check_prefix_shape(d->fmt, d->rows, d->num_q_heads, d->num_kv_heads, d->head_dim, d->prefix_len,
                                     d->max_row_len);
  if (st != QKV_OK) return st;
  if ((d->fmt == QKV_F16 && !d->q_fp16) || (d->fmt == QKV_BF16 && d->q_fp16)) return QKV_ERR_ARG;
  if (!std::isfinite(d->softmax_scale) || d->num_slots < 0) return QKV_ERR_ARG;
  if (d->fmt == QKV_E4M3 && (!finite_positive(d->k_scale_layer) || !finite_positive(d->v_scale_layer)))
    return QKV_ERR_SCALE;
  const bool side = d->fmt == QKV_INT8_SIDE;
  if (side != (d->k_scale_tok != nullptr) || side != (d->v_scale_tok != nullptr)) return QKV_ERR_ARG;
  if (d->num_seqs < 1 || d->max_blocks < 1 || d->block_size < 1) return QKV_ERR_ARG;
  if (static_cast<int64_t>(d->max_blocks) * d->block_size > INT32_MAX) return QKV_ERR_ARG;
  if (d->max_row_len > static_cast<int64_t>(d->max_blocks) * d->block_size) return QKV_ERR_ARG;
  if (d->num_slots > INT32_MAX / d->num_kv_heads) return QKV_ERR_UNSUPPORTED;  // records are numbered in 32 bits
  if (d->q_stride < static_cast<int64_t>(d->num_q_heads) * d->head_dim) return QKV_ERR_ARG;
  if (d->rows == 0) return QKV_OK;
  if (!d->q || !d->out || !d->k_cache || !d->v_cache || !d->block_table || !d->row_seq || !d->row_len) return QKV_ERR_ARG;
  if (d->prefix_len > 0 && !d->prefix_blocks) return QKV_ERR_ARG;
  if (d->q_stride % 8 != 0 || !aligned(d->q, 16) || !aligned(d->out, 16)) return QKV_ERR_ALIGN;
  if (!aligned(d->k_cache, 16) || !aligned(d->v_cache, 16)) return QKV_ERR_ALIGN;
  if (side && (!aligned(d->k_scale_tok, 4) || !aligned(d->v_scale_tok, 4))) return QKV_ERR_ALIGN;
  if (!aligned(d->prefix_blocks, 4) || !aligned(d->block_table, 4) || !aligned(d->row_seq, 4) ||
      !aligned(d->row_len, 4) || !aligned(d->lse, 4) || !aligned(d->dev_status, 4) || !aligned(d->workspace, 16))
    return QKV_ERR_ALIGN;

  PrefixPlan p;
  st = plan_prefix(d->fmt, d->rows, d->num_q_heads, d->num_kv_heads, d->head_dim, d->prefix_len, d->max_row_len, &p);
  if (st != QKV_OK) return st;
  if (p.bytes() > 0 && (!d->workspace || d->workspace_bytes < p.bytes())) return QKV_ERR_ARG;

  qkv::PrefixArgs a;
  a.q = static_cast<const uint16_t*>(d->q);
  a.q_stride = d->q_stride;
  a.q_f16 = d->q_fp16 == 1;
  a.rows = d->rows;
  a.num_q_heads = d->num_q_heads;
  a.num_kv_heads = d->num_kv_heads;
  a.head_dim = d->head_dim;
  a.k_cache = static_cast<const uint8_t*>(d->k_cache);
  a.v_cache = static_cast<const uint8_t*>(d->v_cache);
  a.k_scale_tok = d->k_scale_tok;
  a.v_scale_tok = d->v_scale_tok;
  a.k_scale_layer = d->k_scale_layer;
  a.v_scale_layer = d->v_scale_layer;
  a.num_slots = d->num_slots;
  a.prefix_blocks = d->prefix_blocks;
  a.prefix_len = d->prefix_len;
  a.block_table = d->block_table;
  a.num_seqs = d->num_seqs;
  a.max_blocks = d->max_blocks;
  a.block_size = d->block_size;
  a.row_seq = d->row_seq;
  a.row_len = d->row_len;
  a.max_row_len = d->max_row_len;
  a.softmax_scale = d->softmax_scale;
  a.out = static_cast<uint16_t*>(d->out);
  a.lse = d->lse;
  a.merge_scale = d->fmt == QKV_E4M3 ? d->v_scale_layer : 1.f;
  a.dev_status = d->dev_status;
  const bool direct = p.parts() == 1 && p.umma_cg == 0;
  a.o_part = direct ? nullptr : static_cast<float*>(d->workspace);
  a.lse_part = direct ? nullptr : reinterpret_cast<float*>(static_cast<uint8_t*>(d->workspace) + p.o_bytes());
  a.prefix_parts = p.prefix_parts;
  a.own_parts = p.own_parts;
  a.prefix_chunk = p.prefix_chunk;
  // Tiles of 8 pairs where a sequence's rows bring no more than that on average: half of a 16-pair tile of own keys
  // would be empty. What stands for the sequences is the block table's rows; row_seq is not read here. In us, 8 | 16:
  // e4m3, 32 sequences of 1400 keys, 4 heads of 128, groups of 8, one row each 16 | 18, four rows 45 | 34; int8 20 |
  // 22, 51 | 40; bf16 24 | 29, 64 | 43. Tiles of the prefix take pairs of any rows and are full either way, so that 16
  // reads it half as often: 8 only where mma.sync has no prefix or one of at most twice the rows' own keys. Single
  // rows behind 2000 shared keys, 8 | 16: 32 rows with 300 of their own, e4m3 24 | 18, int8 25 | 21, with 1400 29 |
  // 31, 33 | 36; behind 500, 8 rows with 300 8.9 | 10.0, 8.9 | 10.7.
  const int G = d->num_q_heads / d->num_kv_heads;
  const bool prefix_rules = p.ptiles > 0 && d->prefix_len > 2 * static_cast<int64_t>(d->max_row_len - d->prefix_len);
  a.mma_pairs = G <= 8 && d->rows * G <= 8 * static_cast<int64_t>(d->num_seqs) && !prefix_rules ? 8 : 16;
  if (a.mma_pairs == 8 && p.ptiles > 0) p.ptiles = ceil_div(d->rows * G, 8) * d->num_kv_heads;
  a.prefix_items = p.ptiles * p.prefix_parts;
  a.own_items = p.otiles * p.own_parts;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  a.umma_cg = p.umma_cg;
  a.umma_pairs = p.umma_pairs;
  a.umma_ptiles = p.umma_ptiles;
  a.umma_blocks = p.umma_blocks;
  a.umma_teams = p.umma_teams;
  a.umma_share = p.umma_share;
  a.umma_extra = p.umma_extra;
  if (p.umma_cg > 0) e = launch_prefix_umma(a, d->fmt, s);
  if (e == cudaSuccess && a.prefix_items + a.own_items > 0) e = launch_prefix_mma(a, d->fmt, p.umma_cg > 0, s);
  if (e == cudaSuccess && !direct) e = qkv::launch_prefix_merge(a, s);
  return cuda_status(e);
}

}  // extern "C"

namespace {

// How a masked call runs: on mma.sync tiles of the rows over `parts` ranges of their keys, or on tcgen05 tiles of
// tile_rows rows (umma_cg > 0) that teams of umma_cg SMs take from the work list.
struct MaskedPlan {
  int64_t tiles;  // mma.sync tiles
  int parts;      // ranges of their keys
  int umma_cg, umma_pairs, tile_rows, block_keys, tile_cost;
  uint32_t umma_teams;
  int64_t rows, rows_heads;
  int head_dim;
  // Partial outputs, then partial log-sum-exps, then the work list. Of mma.sync tiles a single part writes the output
  // itself; a team of SMs leaves at most two partial tiles.
  int64_t part_rows() const { return umma_cg > 0 ? 2 * static_cast<int64_t>(umma_teams) * umma_pairs : parts > 1 ? parts * rows_heads : 0; }
  size_t o_bytes() const { return static_cast<size_t>(part_rows()) * head_dim * 4; }
  size_t list_at() const { return o_bytes() + (static_cast<size_t>(part_rows()) * 4 + 31) / 32 * 32; }
  size_t bytes() const { return list_at() + (umma_cg > 0 ? qkv::masked_plan_bytes(rows, tile_rows, umma_teams) : 0); }
};

qkv_status check_masked_shape(qkv_format fmt, int64_t rows, int64_t num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                              int max_row_end, int window) {
  if (num_seqs < 1 || window < 0) return QKV_ERR_ARG;
  return check_prefix_shape(fmt, rows, num_q_heads, num_kv_heads, head_dim, 0, max_row_end);
}

// Where a masked call runs on tcgen05 tiles: a sequence brings at least this many pairs on average (over the table's
// sequences, or the rows if those are fewer: where the rows lie is known on the device alone), and tiles of 16
// pairs would read at least so many bytes of keys and values, most of them from L2 (a tcgen05 call costs some 8 us more at its
// ends). In us, mma.sync | tcgen05: 16 heads of 256, int8: 8 sequences x 5 rows behind 1000 keys (20 MB) 23 | 32, behind
// 4000 (78 MB) 46 | 38, behind 8000 71 | 43; 64 x 4 behind 500 (62 MB) 29 | 40, behind 1000 54 | 46; 4 x 16 behind 2000
// (62 MB) 32 | 39, behind 4000 54 | 39. 64 heads of 128 in groups of 8, e4m3: 8 x 5 behind 1000 (39 MB) 25 | 32, behind
// 2000 (78 MB) 42 | 40, behind 8000 109 | 74; 64 x 4 (32 pairs) behind 1000 97 | 100, behind 8000 420 | 384; 64 x 2
// behind 4000 (16 pairs, 500 MB) 152 | 217. Groups of 4: 64 x 4 behind 8000 (16 pairs, 2 GB) 360 | 391.
constexpr int64_t kMaskedUmmaPairs = 32;
constexpr int64_t kMaskedUmmaBytes = 64 << 20;
// What a tile costs besides its key blocks, in blocks: with 0 | 3 | 6 | 12 of them prompts of documents of about 700 bf16
// rows took 278 | 248 | 252 | 256 us, three prompts of 77 to 1501 rows under a prefix mask 134 | 125 | 116 | 119, 2048 rows
// behind 8000 int8 keys 323 | 324 | 320 | 325.
constexpr int kMaskedTileCost = 6;

qkv_status plan_masked(qkv_format fmt, int64_t rows, int64_t num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                       int max_row_end, int window, MaskedPlan* p) {
  const int sms = sm_count();
  if (sms < 1) return QKV_ERR_CUDA;
  const int G = num_q_heads / num_kv_heads;
  // The sequences that have rows, as far as the host knows: the table may hold more, but no more than there are rows.
  const int64_t seqs = rows < num_seqs ? (rows > 0 ? rows : 1) : num_seqs;
  p->rows_heads = rows * num_q_heads;
  p->head_dim = head_dim;
  p->tiles = rows * ceil_div(G, 16) * num_kv_heads;
  // a tile's rows that follow each other see a window's keys and a few more
  const int64_t seen = window > 0 && window < max_row_end ? window : max_row_end, keys = seen < max_row_end - 16 ? seen + 16 : max_row_end;
  p->parts = key_parts(p->tiles, static_cast<int>(seen > 0 ? seen : 1), row_bytes_of(fmt, head_dim), sms);
  // Less than two waves of CTAs, or any number of them for one sequence (several may be of any lengths, which more parts
  // even out), are cut down to one. 1 row x 4 heads of 128 behind 60000 e4m3 keys in 118 parts 31 us, in 102 24; 8 heads: 48,
  // in 51 35; 3 rows x 16 heads of 256, int8: 52, in 91 39.
  const int64_t wave = 9 * resident_slots(row_bytes_of(fmt, head_dim), sms) / 10, ctas = p->tiles * p->parts;
  if (ctas > wave && (ctas < 2 * wave || seqs == 1) && p->tiles < wave) p->parts = static_cast<int>(wave / p->tiles);
  p->rows = rows;
  p->umma_cg = 0, p->umma_pairs = 0, p->tile_rows = 0, p->block_keys = 0, p->tile_cost = 0, p->umma_teams = 0;
  const int64_t pairs = rows * G / seqs;  // of a sequence, on average
  const int64_t tiles16 = ceil_div(rows * G, 16) * num_kv_heads;
  const bool large = keys > 0 && tiles16 >= kMaskedUmmaBytes / (keys * 2 * row_bytes_of(fmt, head_dim));
  bool umma = pairs >= kMaskedUmmaPairs && large;
  // Test of each kind of tiles at any size: QKV_TEST_MASKED_TILES=tcgen05 or mma (read at each call; unset in any other use).
  if (const char* t = std::getenv("QKV_TEST_MASKED_TILES")) umma = std::strcmp(t, "tcgen05") == 0 || (umma && std::strcmp(t, "mma") != 0);
  if (umma && max_row_end <= (1 << 27) && num_kv_heads <= 0xffff) {
    // Tiles of 256 pairs on a pair of SMs where a sequence has more than one of 128. In us, 128 | 256: 16 sequences x 18
    // rows x 64 heads of 128 in groups of 8 behind 8000 bf16 keys (144 pairs) 217 | 172, 16 rows each (128) 140 | 176; 16 x
    // 150 rows x 8 heads of 256, each its own group, 157 | 120, 100 rows each 159 | 170.
    p->umma_cg = pairs > 128 ? 2 : 1;
    p->umma_pairs = 128 * p->umma_cg;
    p->tile_rows = p->umma_pairs / G;
    p->block_keys = head_dim == 256 && p->umma_cg == 1 ? 64 : 128;
    p->umma_teams = static_cast<uint32_t>(sms / p->umma_cg);
    p->tile_cost = kMaskedTileCost;
    // a team's share is counted in 32 bits, however the rows are cut into tiles, and a chunk's work is
    const int64_t blocks = max_row_end / p->block_keys + 2 + p->tile_cost;
    if (rows > (int64_t(1) << 31) / blocks / num_kv_heads * p->umma_teams) p->umma_cg = 0;
  }
  if (p->umma_cg == 0 && p->tiles * p->parts > INT32_MAX) return QKV_ERR_ARG;
  return QKV_OK;
}

cudaError_t launch_masked_umma(const qkv::PrefixArgs& a, qkv_format fmt, cudaStream_t s) {
  switch (fmt) {
    case QKV_BF16: return qkv::launch_masked_umma_bf16(a, s);
    case QKV_F16: return qkv::launch_masked_umma_f16(a, s);
    case QKV_INT8_SIDE: return qkv::launch_masked_umma_int8_side(a, s);
    case QKV_INT8_INLINE: return qkv::launch_masked_umma_int8_inline(a, s);
    case QKV_E4M3: return qkv::launch_masked_umma_e4m3(a, s);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_masked_mma(const qkv::PrefixArgs& a, qkv_format fmt, cudaStream_t s) {
  switch (fmt) {
    case QKV_BF16: return qkv::launch_masked_mma_bf16(a, s);
    case QKV_F16: return qkv::launch_masked_mma_f16(a, s);
    case QKV_INT8_SIDE: return qkv::launch_masked_mma_int8_side(a, s);
    case QKV_INT8_INLINE: return qkv::launch_masked_mma_int8_inline(a, s);
    case QKV_E4M3: return qkv::launch_masked_mma_e4m3(a, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

extern "C" {

qkv_status qkv_masked_attn_workspace(qkv_format fmt, int64_t rows, int64_t num_seqs, int num_q_heads, int num_kv_heads,
                                     int head_dim, int max_row_end, int window, size_t* bytes) {
  if (!bytes) return QKV_ERR_ARG;
  qkv_status st = check_masked_shape(fmt, rows, num_seqs, num_q_heads, num_kv_heads, head_dim, max_row_end, window);
  if (st != QKV_OK) return st;
  MaskedPlan p;
  st = plan_masked(fmt, rows, num_seqs, num_q_heads, num_kv_heads, head_dim, max_row_end, window, &p);
  if (st == QKV_OK) *bytes = p.bytes();
  return st;
}

qkv_status qkv_masked_attn(const qkv_masked_desc* d, void* stream) {
  if (d == nullptr || d->size != sizeof(qkv_masked_desc)) return QKV_ERR_ARG;
  if (d->q_fp16 != 0 && d->q_fp16 != 1) return QKV_ERR_ARG;
  qkv_status st = check_masked_shape(d->fmt, d->rows, d->num_seqs, d->num_q_heads, d->num_kv_heads, d->head_dim, d->max_row_end,
                                     d->window);
  if (st != QKV_OK) return st;
  if ((d->fmt == QKV_F16 && !d->q_fp16) || (d->fmt == QKV_BF16 && d->q_fp16)) return QKV_ERR_ARG;
  if (!std::isfinite(d->softmax_scale) || d->num_slots < 0) return QKV_ERR_ARG;
  if (!(d->softcap == 0.f || (d->softcap >= 0x1p-20f && d->softcap <= 0x1p20f))) return QKV_ERR_ARG;
  if (d->fmt == QKV_E4M3 && (!finite_positive(d->k_scale_layer) || !finite_positive(d->v_scale_layer)))
    return QKV_ERR_SCALE;
  const bool side = d->fmt == QKV_INT8_SIDE;
  if (side != (d->k_scale_tok != nullptr) || side != (d->v_scale_tok != nullptr)) return QKV_ERR_ARG;
  if (d->max_blocks < 1 || d->block_size < 1) return QKV_ERR_ARG;
  if (static_cast<int64_t>(d->max_blocks) * d->block_size > INT32_MAX) return QKV_ERR_ARG;
  if (d->max_row_end > static_cast<int64_t>(d->max_blocks) * d->block_size) return QKV_ERR_ARG;
  if (d->num_slots > INT32_MAX / d->num_kv_heads) return QKV_ERR_UNSUPPORTED;  // records are numbered in 32 bits
  if (d->q_stride < static_cast<int64_t>(d->num_q_heads) * d->head_dim) return QKV_ERR_ARG;
  if (d->rows == 0) return QKV_OK;
  if (!d->q || !d->out || !d->k_cache || !d->v_cache || !d->block_table || !d->row_seq || !d->row_end) return QKV_ERR_ARG;
  if (d->q_stride % 8 != 0 || !aligned(d->q, 16) || !aligned(d->out, 16)) return QKV_ERR_ALIGN;
  if (!aligned(d->k_cache, 16) || !aligned(d->v_cache, 16)) return QKV_ERR_ALIGN;
  if (side && (!aligned(d->k_scale_tok, 4) || !aligned(d->v_scale_tok, 4))) return QKV_ERR_ALIGN;
  if (!aligned(d->block_table, 4) || !aligned(d->row_seq, 4) || !aligned(d->row_start, 4) || !aligned(d->row_end, 4) ||
      !aligned(d->row_pos, 4) || !aligned(d->slopes, 4) || !aligned(d->lse, 4) || !aligned(d->dev_status, 4) ||
      !aligned(d->workspace, 16))
    return QKV_ERR_ALIGN;

  MaskedPlan p;
  st = plan_masked(d->fmt, d->rows, d->num_seqs, d->num_q_heads, d->num_kv_heads, d->head_dim, d->max_row_end, d->window, &p);
  if (st != QKV_OK) return st;
  if (p.bytes() > 0 && (!d->workspace || d->workspace_bytes < p.bytes())) return QKV_ERR_ARG;

  qkv::PrefixArgs a = {};
  a.q = static_cast<const uint16_t*>(d->q);
  a.q_stride = d->q_stride;
  a.q_f16 = d->q_fp16 == 1;
  a.rows = d->rows;
  a.num_q_heads = d->num_q_heads;
  a.num_kv_heads = d->num_kv_heads;
  a.head_dim = d->head_dim;
  a.k_cache = static_cast<const uint8_t*>(d->k_cache);
  a.v_cache = static_cast<const uint8_t*>(d->v_cache);
  a.k_scale_tok = d->k_scale_tok;
  a.v_scale_tok = d->v_scale_tok;
  a.k_scale_layer = d->k_scale_layer;
  a.v_scale_layer = d->v_scale_layer;
  a.num_slots = d->num_slots;
  a.block_table = d->block_table;
  a.num_seqs = d->num_seqs;
  a.max_blocks = d->max_blocks;
  a.block_size = d->block_size;
  a.row_seq = d->row_seq;
  a.row_len = d->row_end;
  a.max_row_len = d->max_row_end;
  a.row_start = d->row_start;
  a.row_pos = d->window > 0 || d->slopes ? d->row_pos : nullptr;  // nothing else asks for positions
  a.window = d->window;
  a.softcap = d->softcap;
  a.slopes = d->slopes;
  a.softmax_scale = d->softmax_scale;
  a.out = static_cast<uint16_t*>(d->out);
  a.lse = d->lse;
  a.merge_scale = d->fmt == QKV_E4M3 ? d->v_scale_layer : 1.f;
  a.dev_status = d->dev_status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(d->workspace);
  const bool direct = p.part_rows() == 0;
  a.o_part = direct ? nullptr : reinterpret_cast<float*>(ws);
  a.lse_part = direct ? nullptr : reinterpret_cast<float*>(ws + p.o_bytes());
  cudaError_t e;
  if (p.umma_cg > 0) {
    a.plan = ws + p.list_at();
    a.umma_cg = p.umma_cg;
    a.umma_pairs = p.umma_pairs;
    a.umma_teams = p.umma_teams;
    a.tile_rows = p.tile_rows;
    a.block_keys = p.block_keys;
    a.tile_cost = p.tile_cost;
    a.plan_tiles_at = static_cast<int64_t>(qkv::masked_plan_tiles_at(d->rows, p.tile_rows, p.umma_teams));
    a.plan_chunks = qkv::masked_plan_chunks(d->rows, p.tile_rows);
    e = qkv::launch_masked_plan(a, s);
    if (e == cudaSuccess) e = launch_masked_umma(a, d->fmt, s);
    if (e == cudaSuccess) e = qkv::launch_masked_join(a, s);
  } else {
    a.own_parts = p.parts;
    a.own_items = p.tiles * p.parts;
    // tiles of 8 pairs where a sequence's rows bring no more than that on average, as for qkv_prefix_attn's own keys
    const int G = d->num_q_heads / d->num_kv_heads;
    a.mma_pairs = G <= 8 && d->rows * G <= 8 * d->num_seqs ? 8 : 16;
    e = launch_masked_mma(a, d->fmt, s);
    if (e == cudaSuccess && !direct) e = qkv::launch_masked_merge(a, s);
  }
  return cuda_status(e);
}

}  // extern "C"
