// Host API of the attention operators: argument validation and the launches of
// mlap_kv_append_*, mlap_paged_attention_* and mlap_window_attention_* (include/mlaprolog.h).
#include <cmath>
#include <cstring>

#include "attention.h"
#include "host_util.h"
#include "mlaprolog.h"

using namespace mlap;

namespace {

constexpr size_t kHeaderBytes = 256;    // the error word, padded to the workspace alignment

mlap_status_t want_half(const mlap_tensor_t& t, const char* name) {
  if (t.dtype != MLAP_DTYPE_FP16 && t.dtype != MLAP_DTYPE_BF16)
    return fail(MLAP_ERR_DTYPE, std::string(name) + " must be fp16 or bf16");
  return MLAP_OK;
}

mlap_status_t check_cache_mode(const char* mode) {
  if (mode != nullptr && std::strcmp(mode, "PA_BSND") != 0)
    return fail(MLAP_ERR_UNSUPPORTED, std::string("cache_mode '") + mode + "' not supported (PA_BSND only)");
  return MLAP_OK;
}

// cu_seqlens (B+1) and max_new of T token rows
mlap_status_t check_ragged(const mlap_tensor_t& cu, int64_t T, int64_t max_new, Ragged* r) {
  CHECK_STATUS(need(cu, "cu_seqlens", false, sizeof(int64_t)));
  CHECK_STATUS(want_dtype(cu, "cu_seqlens", MLAP_DTYPE_INT64));
  if (cu.ndim != 1 || cu.shape[0] < 1) return fail(MLAP_ERR_SHAPE, "cu_seqlens must be (B+1)");
  if (T > kMaxTokens) return fail(MLAP_ERR_UNSUPPORTED, "too many tokens");
  if (cu.shape[0] - 1 > kMaxTokens) return fail(MLAP_ERR_UNSUPPORTED, "too many sequences");
  if (max_new < 0 || (max_new == 0 && T > 0 && cu.shape[0] > 1))
    return fail(MLAP_ERR_SHAPE, "max_new must be positive");
  r->cu = static_cast<const int64_t*>(cu.data);
  r->ctx = nullptr;
  r->B = static_cast<int32_t>(cu.shape[0] - 1);
  r->T = T;
  r->max_new = static_cast<int32_t>(max_new < T ? max_new : T);
  return MLAP_OK;
}

// context_lens (B), block_table (B, MaxBlocks), the caches and their scales, for Nk heads
mlap_status_t check_pages(const mlap_tensor_t& ctx, const mlap_tensor_t& table,
                          const mlap_tensor_t& kc, const mlap_tensor_t& vc,
                          const mlap_tensor_t& ks, const mlap_tensor_t& vs, int64_t Nk, Ragged* r,
                          Pages* pg) {
  CHECK_STATUS(need(ctx, "context_lens", true, sizeof(int64_t)));
  CHECK_STATUS(want_dtype(ctx, "context_lens", MLAP_DTYPE_INT64));
  CHECK_STATUS(want_shape(ctx, "context_lens", {r->B}));
  CHECK_STATUS(need(table, "block_table", true, sizeof(int64_t)));
  CHECK_STATUS(want_dtype(table, "block_table", MLAP_DTYPE_INT64));
  if (table.ndim != 2 || table.shape[0] != r->B)
    return fail(MLAP_ERR_SHAPE, "block_table must be (B, MaxBlocks)");
  CHECK_STATUS(need(kc, "k_cache", true));
  CHECK_STATUS(need(vc, "v_cache", true));
  CHECK_STATUS(want_dtype(kc, "k_cache", MLAP_DTYPE_INT8));
  CHECK_STATUS(want_dtype(vc, "v_cache", MLAP_DTYPE_INT8));
  if (kc.ndim != 4) return fail(MLAP_ERR_SHAPE, "caches must be (BlockNum, BlockSize, Nk, D)");
  const int64_t num = kc.shape[0], bs = kc.shape[1];
  if (kc.shape[3] != kHeadDim) return fail(MLAP_ERR_UNSUPPORTED, "head dim D must be 128");
  CHECK_STATUS(want_shape(kc, "k_cache", {num, bs, Nk, kHeadDim}));
  CHECK_STATUS(want_shape(vc, "v_cache", {num, bs, Nk, kHeadDim}));
  if (bs <= 0 || bs % 16) return fail(MLAP_ERR_UNSUPPORTED, "BlockSize must be a positive multiple of 16");
  CHECK_STATUS(need(ks, "k_scale", true, sizeof(float)));
  CHECK_STATUS(need(vs, "v_scale", true, sizeof(float)));
  CHECK_STATUS(want_dtype(ks, "k_scale", MLAP_DTYPE_FP32));
  CHECK_STATUS(want_dtype(vs, "v_scale", MLAP_DTYPE_FP32));
  CHECK_STATUS(want_shape(ks, "k_scale", {num, Nk}));
  CHECK_STATUS(want_shape(vs, "v_scale", {num, Nk}));
  if (num > 0x7fffffff) return fail(MLAP_ERR_UNSUPPORTED, "BlockNum must be below 2^31");
  if (bs > kMaxBlockSize || table.shape[1] > kMaxTokens / bs)
    return fail(MLAP_ERR_UNSUPPORTED, "BlockSize must be at most 65536 and MaxBlocks * BlockSize at most 2^30");
  r->ctx = static_cast<const int64_t*>(ctx.data);
  pg->table = static_cast<const int64_t*>(table.data);
  pg->k = static_cast<int8_t*>(kc.data);
  pg->v = static_cast<int8_t*>(vc.data);
  pg->k_scale = static_cast<float*>(ks.data);
  pg->v_scale = static_cast<float*>(vs.data);
  pg->block_num = num;
  pg->max_blocks = static_cast<int32_t>(table.shape[1]);
  pg->block_size = static_cast<int32_t>(bs);
  pg->Nk = static_cast<int32_t>(Nk);
  pg->runs = fast_div(static_cast<uint32_t>(bs / 16));
  return MLAP_OK;
}

mlap_status_t check_heads(int64_t Nq, int64_t Nk) {
  if (Nk <= 0 || Nq < 0 || Nk > 65535 || Nq > 65535)
    return fail(MLAP_ERR_SHAPE, "head counts out of range");
  if (Nq % Nk) return fail(MLAP_ERR_SHAPE, "Nq must be a multiple of Nk");
  return MLAP_OK;
}

// q, out, the mask and the scale, which the two attentions share; Nk is given
mlap_status_t check_attn(const mlap_tensor_t& q, const mlap_tensor_t& out, int64_t Nk,
                         int64_t window, int64_t sinks, double scale, AttnParams* p) {
  CHECK_STATUS(need(q, "q", true));
  CHECK_STATUS(want_half(q, "q"));
  if (q.ndim != 3) return fail(MLAP_ERR_SHAPE, "q must be (T, Nq, D)");
  if (q.shape[2] != kHeadDim) return fail(MLAP_ERR_UNSUPPORTED, "head dim D must be 128");
  if (q.shape[1] <= 0) return fail(MLAP_ERR_SHAPE, "Nq must be positive");
  CHECK_STATUS(check_heads(q.shape[1], Nk));
  if (q.shape[1] / Nk > 128) return fail(MLAP_ERR_UNSUPPORTED, "more than 128 query heads share a k/v head");
  CHECK_STATUS(need(out, "out", true));
  CHECK_STATUS(want_dtype(out, "out", q.dtype));
  CHECK_STATUS(want_shape(out, "out", {q.shape[0], q.shape[1], kHeadDim}));
  if (window < 0 || sinks < 0) return fail(MLAP_ERR_SHAPE, "window and sinks must not be negative");
  const float scale_log2 = static_cast<float>(scale * 1.4426950408889634074);     // log2(e)
  if (!std::isfinite(scale_log2)) return fail(MLAP_ERR_SHAPE, "softmax_scale must be finite, in 32 bits too");
  const int64_t most = 0x7fffffff;                       // beyond every position
  p->q = q.data;
  p->out = out.data;
  p->Nq = static_cast<int32_t>(q.shape[1]);
  p->Nk = static_cast<int32_t>(Nk);
  p->window = window >= most ? 0 : static_cast<int32_t>(window);
  p->sinks = static_cast<int32_t>(sinks < most ? sinks : most);
  p->scale_log2 = scale_log2;
  p->bf16 = q.dtype == MLAP_DTYPE_BF16;
  return MLAP_OK;
}

bool overlap(const mlap_tensor_t& a, const mlap_tensor_t& b) {
  if (a.data == nullptr || b.data == nullptr) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.data), b0 = reinterpret_cast<uintptr_t>(b.data);
  const size_t an = numel(a) * dtype_bytes(a.dtype), bn = numel(b) * dtype_bytes(b.dtype);
  return a0 < b0 + bn && b0 < a0 + an;
}

mlap_status_t check_workspace(void* ws, size_t have, size_t want) {
  if (ws == nullptr || have < want) return fail(MLAP_ERR_WORKSPACE, "workspace too small");
  if (reinterpret_cast<uintptr_t>(ws) & 255u)
    return fail(MLAP_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  return MLAP_OK;
}

size_t window_workspace(const AttnParams& p) {
  return align_up(kHeaderBytes + (window_splits(p) ? tile_parts_workspace() : 0), 256);
}

size_t paged_workspace(const AttnParams& p) {
  return align_up(kHeaderBytes + (paged_chunk_pays(p) ? tile_parts_workspace() : paged_decode_workspace()), 256);
}

cudaError_t sm_count(int* sms) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  return e != cudaSuccess ? e : cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
}

// Tensor map of (T, N, D) 16-bit rows: boxes of 64 elements x `heads` x `tokens`, 128-byte swizzle,
// zero fill outside the tensor.
mlap_status_t rows_map(CUtensorMap* m, const mlap_tensor_t& t, int heads, int tokens) {
  EncodeTiledFn enc = get_encode_fn();
  if (enc == nullptr) return fail(MLAP_ERR_CUDA, "cuTensorMapEncodeTiled unavailable");
  const cuuint64_t dims[3] = {kHeadDim, static_cast<cuuint64_t>(t.shape[1]),
                              static_cast<cuuint64_t>(t.shape[0])};
  const cuuint64_t strides[2] = {kHeadDim * 2, static_cast<cuuint64_t>(t.shape[1]) * kHeadDim * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(heads), static_cast<cuuint32_t>(tokens)};
  const cuuint32_t es[3] = {1, 1, 1};
  const CUresult r =
      enc(m, t.dtype == MLAP_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
          3, t.data, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return fail(MLAP_ERR_CUDA, "cuTensorMapEncodeTiled failed (" + std::to_string(int(r)) + ")");
  return MLAP_OK;
}

// Map of a cache (BlockNum, BlockSize, Nk, D) whose boxes are 16 tokens of a head of a page.
mlap_status_t pages_map(CUtensorMap* m, const mlap_tensor_t& t) {
  EncodeTiledFn enc = get_encode_fn();
  if (enc == nullptr) return fail(MLAP_ERR_CUDA, "cuTensorMapEncodeTiled unavailable");
  const cuuint64_t dims[4] = {kHeadDim, static_cast<cuuint64_t>(t.shape[2]),
                              static_cast<cuuint64_t>(t.shape[1]), static_cast<cuuint64_t>(t.shape[0])};
  const cuuint64_t strides[3] = {kHeadDim, dims[1] * kHeadDim, dims[2] * dims[1] * kHeadDim};
  const cuuint32_t box[4] = {kHeadDim, 1, 16, 1};
  const cuuint32_t es[4] = {1, 1, 1, 1};
  const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, t.data, dims, strides, box, es,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return fail(MLAP_ERR_CUDA, "cuTensorMapEncodeTiled failed (" + std::to_string(int(r)) + ")");
  return MLAP_OK;
}

// ----------------------------------------------------------------------------------------------
mlap_status_t validate_append(const mlap_kv_append_args_t* a, KvAppendParams* p) {
  if (a == nullptr) return fail(MLAP_ERR_NULL, "args is NULL");
  const mlap_tensor_t& x = a->qkv;
  CHECK_STATUS(check_heads(a->Nq, a->Nk));
  CHECK_STATUS(need(x, "qkv", true));
  CHECK_STATUS(want_half(x, "qkv"));
  const int64_t heads = int64_t(a->Nq) + 2 * int64_t(a->Nk);
  if (x.ndim != 2) return fail(MLAP_ERR_SHAPE, "qkv must be (T, (Nq+2*Nk)*D)");
  if (x.shape[1] % heads) return fail(MLAP_ERR_SHAPE, "qkv width is not a multiple of Nq+2*Nk");
  if (x.shape[1] / heads != kHeadDim) return fail(MLAP_ERR_UNSUPPORTED, "head dim D must be 128");
  const int64_t T = x.shape[0];
  if (present(a->gamma_q) != (present(a->gamma_k) && a->Nq > 0))
    return fail(MLAP_ERR_NULL, "gamma_q is given exactly when gamma_k is and Nq > 0");
  for (auto* g : {&a->gamma_q, &a->gamma_k}) {
    if (!present(*g)) continue;
    CHECK_STATUS(need(*g, "gamma", false));
    CHECK_STATUS(want_dtype(*g, "gamma", x.dtype));
    CHECK_STATUS(want_shape(*g, "gamma", {kHeadDim}));
  }
  for (auto* t : {&a->cos, &a->sin}) {
    CHECK_STATUS(need(*t, "cos/sin", true));
    CHECK_STATUS(want_dtype(*t, "cos/sin", x.dtype));
    CHECK_STATUS(want_shape(*t, "cos/sin", {T, kHeadDim}));
  }
  CHECK_STATUS(check_ragged(a->cu_seqlens, T, a->max_new, &p->rag));
  CHECK_STATUS(check_pages(a->context_lens, a->block_table, a->k_cache, a->v_cache, a->k_scale,
                           a->v_scale, a->Nk, &p->rag, &p->pg));
  if (a->Nq > 0) {
    CHECK_STATUS(need(a->q_out, "q_out", true));
    CHECK_STATUS(want_dtype(a->q_out, "q_out", x.dtype));
    CHECK_STATUS(want_shape(a->q_out, "q_out", {T, a->Nq, kHeadDim}));
    if (overlap(a->q_out, x)) return fail(MLAP_ERR_UNSUPPORTED, "q_out must not overlap qkv");
  } else if (present(a->q_out)) {
    return fail(MLAP_ERR_UNSUPPORTED, "q_out needs query heads (Nq > 0)");
  }
  CHECK_STATUS(check_cache_mode(a->cache_mode));
  if (!(a->epsilon >= 0.0)) return fail(MLAP_ERR_SHAPE, "epsilon must be non-negative");
  p->qkv = x.data;
  p->gamma_q = a->gamma_q.data;
  p->gamma_k = a->gamma_k.data;
  p->cos = a->cos.data;
  p->sin = a->sin.data;
  p->q_out = a->q_out.data;
  p->Nq = a->Nq;
  p->eps = static_cast<float>(a->epsilon);
  p->bf16 = x.dtype == MLAP_DTYPE_BF16;
  return MLAP_OK;
}

mlap_status_t validate_paged(const mlap_paged_attention_args_t* a, AttnParams* p) {
  if (a == nullptr) return fail(MLAP_ERR_NULL, "args is NULL");
  if (a->k_cache.ndim != 4) return fail(MLAP_ERR_SHAPE, "caches must be (BlockNum, BlockSize, Nk, D)");
  const int64_t Nk = a->k_cache.shape[2];
  CHECK_STATUS(check_attn(a->q, a->out, Nk, a->window, a->sinks, a->softmax_scale, p));
  CHECK_STATUS(check_ragged(a->cu_seqlens, a->q.shape[0], a->max_new, &p->rag));
  CHECK_STATUS(check_pages(a->context_lens, a->block_table, a->k_cache, a->v_cache, a->k_scale,
                           a->v_scale, Nk, &p->rag, &p->pg));
  if (overlap(a->out, a->q)) return fail(MLAP_ERR_UNSUPPORTED, "out must not overlap q");
  CHECK_STATUS(check_cache_mode(a->cache_mode));
  p->k = p->v = nullptr;
  return MLAP_OK;
}

mlap_status_t validate_window(const mlap_window_attention_args_t* a, AttnParams* p) {
  if (a == nullptr) return fail(MLAP_ERR_NULL, "args is NULL");
  if (a->k.ndim != 3) return fail(MLAP_ERR_SHAPE, "k must be (T, Nk, D)");
  const int64_t Nk = a->k.shape[1];
  CHECK_STATUS(check_attn(a->q, a->out, Nk, a->window, a->sinks, a->softmax_scale, p));
  const int64_t T = a->q.shape[0];
  CHECK_STATUS(need(a->k, "k", true));
  CHECK_STATUS(need(a->v, "v", true));
  CHECK_STATUS(want_dtype(a->k, "k", a->q.dtype));
  CHECK_STATUS(want_dtype(a->v, "v", a->q.dtype));
  CHECK_STATUS(want_shape(a->k, "k", {T, Nk, kHeadDim}));
  CHECK_STATUS(want_shape(a->v, "v", {T, Nk, kHeadDim}));
  CHECK_STATUS(check_ragged(a->cu_seqlens, T, a->max_new, &p->rag));
  if (overlap(a->out, a->q) || overlap(a->out, a->k) || overlap(a->out, a->v))
    return fail(MLAP_ERR_UNSUPPORTED, "out must not overlap q, k or v");
  p->k = a->k.data;
  p->v = a->v.data;
  p->pg = Pages{};
  return MLAP_OK;
}

}  // namespace

// ================================================================================================
extern "C" {

mlap_status_t mlap_kv_append_get_workspace_size(const mlap_kv_append_args_t* args, size_t* bytes) {
  if (bytes == nullptr) return fail(MLAP_ERR_NULL, "bytes is NULL");
  KvAppendParams p{};
  CHECK_STATUS(validate_append(args, &p));
  *bytes = kHeaderBytes;
  return MLAP_OK;
}

mlap_status_t mlap_kv_append_execute(const mlap_kv_append_args_t* args, void* ws, size_t ws_bytes,
                                     void* stream) {
  KvAppendParams p{};
  CHECK_STATUS(validate_append(args, &p));
  if (p.rag.T == 0 || p.rag.B == 0) return MLAP_OK;
  CHECK_STATUS(check_workspace(ws, ws_bytes, kHeaderBytes));
  p.err = static_cast<uint32_t*>(ws);
  const cudaError_t e = launch_kv_append(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "append launch");
  return MLAP_OK;
}

mlap_status_t mlap_paged_attention_get_workspace_size(const mlap_paged_attention_args_t* args,
                                                      size_t* bytes) {
  if (bytes == nullptr) return fail(MLAP_ERR_NULL, "bytes is NULL");
  AttnParams p{};
  CHECK_STATUS(validate_paged(args, &p));
  *bytes = paged_workspace(p);
  return MLAP_OK;
}

mlap_status_t mlap_paged_attention_execute(const mlap_paged_attention_args_t* args, void* ws,
                                           size_t ws_bytes, void* stream) {
  AttnParams p{};
  CHECK_STATUS(validate_paged(args, &p));
  if (p.rag.T == 0 || p.rag.B == 0) return MLAP_OK;
  CHECK_STATUS(check_workspace(ws, ws_bytes, paged_workspace(p)));
  p.err = static_cast<uint32_t*>(ws);
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e == cudaSuccess && paged_chunk_pays(p)) {
    const int group = p.Nq / p.Nk;
    CUtensorMap q;
    CHECK_STATUS(rows_map(&q, args->q, group, window_attn_tokens(group)));
    e = launch_paged_chunk(q, p, static_cast<uint32_t*>(ws), static_cast<uint8_t*>(ws) + kHeaderBytes,
                           static_cast<cudaStream_t>(stream), sms);
  } else if (e == cudaSuccess) {
    CUtensorMap k{}, v{};
    if (p.pg.block_num > 0) {
      CHECK_STATUS(pages_map(&k, args->k_cache));
      CHECK_STATUS(pages_map(&v, args->v_cache));
    }
    e = launch_paged_decode(k, v, p, static_cast<uint32_t*>(ws), static_cast<uint8_t*>(ws) + kHeaderBytes,
                            static_cast<cudaStream_t>(stream), sms);
  }
  if (e != cudaSuccess) return cuda_fail(e, "paged attention launch");
  return MLAP_OK;
}

mlap_status_t mlap_window_attention_get_workspace_size(const mlap_window_attention_args_t* args,
                                                       size_t* bytes) {
  if (bytes == nullptr) return fail(MLAP_ERR_NULL, "bytes is NULL");
  AttnParams p{};
  CHECK_STATUS(validate_window(args, &p));
  *bytes = window_workspace(p);
  return MLAP_OK;
}

mlap_status_t mlap_window_attention_execute(const mlap_window_attention_args_t* args, void* ws,
                                            size_t ws_bytes, void* stream) {
  AttnParams p{};
  CHECK_STATUS(validate_window(args, &p));
  if (p.rag.T == 0 || p.rag.B == 0) return MLAP_OK;
  CHECK_STATUS(check_workspace(ws, ws_bytes, window_workspace(p)));
  p.err = static_cast<uint32_t*>(ws);
  const int group = p.Nq / p.Nk;
  CUtensorMap q, k, v, k8, v8;
  CHECK_STATUS(rows_map(&q, args->q, group, window_attn_tokens(group)));
  CHECK_STATUS(rows_map(&k, args->k, 1, 128));
  CHECK_STATUS(rows_map(&v, args->v, 1, 128));
  k8 = k;
  v8 = v;
  if (p.window > 0 && p.sinks > 0) {       // (read only by tiles that hold sinks and a window)
    CHECK_STATUS(rows_map(&k8, args->k, 1, 8));
    CHECK_STATUS(rows_map(&v8, args->v, 1, 8));
  }
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e == cudaSuccess) e = launch_window_attn(q, k, v, k8, v8, p, static_cast<uint32_t*>(ws), static_cast<uint8_t*>(ws) + kHeaderBytes,
                           static_cast<cudaStream_t>(stream), sms);
  if (e != cudaSuccess) return cuda_fail(e, "window attention launch");
  return MLAP_OK;
}

}  // extern "C"
