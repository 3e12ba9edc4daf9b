// kvq_latent.cu -- the C ABI of the latent caches (see include/kvq.h): argument
// validation, the pool header, and the launches.
#include <string.h>

#include <new>

#include "kvq_latent.cuh"

using kvq::aligned;
using kvq::cuda_fail;
using kvq::fail;

namespace {

bool tensor_scaled(int mode) { return mode == KVQ_FP8_PER_TENSOR || mode == KVQ_NVFP4 || mode == KVQ_NVFP4_4OVER6; }

kvq_status check_config(const kvq_latent_config* c) {
  if (!c) return fail(KVQ_ERR_INVALID_ARG, "config is NULL");
  if (!tensor_scaled(c->mode) && c->mode != KVQ_INT8_PER_TOKEN_HEAD && c->mode != KVQ_FP8_PER_TOKEN_HEAD)
    return fail(KVQ_ERR_UNSUPPORTED, "mode %d has no latent cache", c->mode);
  if (c->io_dtype != KVQ_F16 && c->io_dtype != KVQ_F32)
    return fail(KVQ_ERR_UNSUPPORTED, "io_dtype %d is not f16 or f32", c->io_dtype);
  if (c->num_pages <= 0) return fail(KVQ_ERR_INVALID_ARG, "num_pages must be positive");
  if (c->num_pages > (1 << 27)) return fail(KVQ_ERR_UNSUPPORTED, "num_pages %d: slots would pass 31 bits", c->num_pages);
  if (c->page_size != 16) return fail(KVQ_ERR_UNSUPPORTED, "a latent cache needs page_size 16 (got %d)", c->page_size);
  if (c->latent_dim != 256 && c->latent_dim != 512)
    return fail(KVQ_ERR_UNSUPPORTED, "latent_dim %d unsupported (256 or 512)", c->latent_dim);
  if (c->rope_dim != kvq::kLatentRope) return fail(KVQ_ERR_UNSUPPORTED, "rope_dim %d unsupported (64)", c->rope_dim);
  return KVQ_OK;
}
size_t pool_bytes(const kvq_latent_config* c) {
  return kvq::kHeaderBytes + (size_t)c->num_pages * kvq::latent_page_bytes(c->mode, c->latent_dim);
}
kvq_status check_cache(const kvq_latent* c) { return c ? KVQ_OK : fail(KVQ_ERR_INVALID_ARG, "cache is NULL"); }
bool stride_ok(int64_t elements, int esize) { return elements >= 0 && elements % (16 / esize) == 0; }

}  // namespace

namespace kvq {
Span latent_pages(const kvq_latent* c) { return Span{c->base + kHeaderBytes, c->base + pool_bytes(&c->cfg)}; }
}  // namespace kvq

extern "C" {

kvq_status kvq_latent_bytes(const kvq_latent_config* cfg, size_t* bytes) {
  kvq_status s = check_config(cfg);
  if (s) return s;
  if (!bytes) return fail(KVQ_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = pool_bytes(cfg);
  return KVQ_OK;
}

kvq_status kvq_latent_alloc(const kvq_latent_config* cfg, void* dev_buf, size_t bytes, kvq_latent** out) {
  kvq_status s = check_config(cfg);
  if (s) return s;
  if (!out) return fail(KVQ_ERR_INVALID_ARG, "out is NULL");
  *out = nullptr;
  if (!dev_buf) return fail(KVQ_ERR_INVALID_ARG, "dev_buf is NULL");
  if (!aligned(dev_buf, 256)) return fail(KVQ_ERR_INVALID_ARG, "dev_buf must be 256-byte aligned");
  if (bytes < pool_bytes(cfg)) return fail(KVQ_ERR_CAPACITY, "pool needs %zu bytes, got %zu", pool_bytes(cfg), bytes);
  unsigned char hdr[kvq::kHeaderBytes];
  memset(hdr, 0, sizeof hdr);
  const uint32_t magic = 0x4C51564Bu, version = 1;  // "KVQL"
  const float one = 1.0f;
  memcpy(hdr + 0, &magic, 4);
  memcpy(hdr + 4, &version, 4);
  memcpy(hdr + 8, &cfg->mode, 4);
  memcpy(hdr + kvq::kHdrKScaleOffset, &one, 4);
  memcpy(hdr + kvq::kHdrVScaleOffset, &one, 4);
  memcpy(hdr + 24, &cfg->num_pages, 4);
  memcpy(hdr + 28, &cfg->page_size, 4);
  memcpy(hdr + 32, &cfg->latent_dim, 4);
  memcpy(hdr + 36, &cfg->rope_dim, 4);
  cudaError_t e = cudaMemcpy(dev_buf, hdr, sizeof hdr, cudaMemcpyHostToDevice);
  if (e != cudaSuccess) return cuda_fail(e, "writing the pool header");
  kvq_latent* c = new (std::nothrow) kvq_latent();
  if (!c) return fail(KVQ_ERR_INVALID_ARG, "out of host memory");
  c->cfg = *cfg;
  c->base = static_cast<uint8_t*>(dev_buf);
  c->page_bytes = kvq::latent_page_bytes(cfg->mode, cfg->latent_dim);
  *out = c;
  return KVQ_OK;
}

kvq_status kvq_latent_free(kvq_latent* cache) {
  delete cache;
  return KVQ_OK;
}

kvq_status kvq_latent_set_scale(kvq_latent* cache, float scale, void* stream) {
  kvq_status s = check_cache(cache);
  if (s) return s;
  if (!(scale > 0.0f) || scale > 3.0e38f) return fail(KVQ_ERR_INVALID_ARG, "the scale must be finite and > 0");
  const float sc[2] = {scale, scale};
  // pageable source: the copy is staged before this call returns, so `sc` may go out of scope
  cudaError_t e = cudaMemcpyAsync(cache->base + kvq::kHdrKScaleOffset, sc, sizeof sc, cudaMemcpyHostToDevice,
                                  static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "setting the tensor scale");
  return KVQ_OK;
}

kvq_status kvq_latent_set_scale_from_amax(kvq_latent* cache, const float* dev_amax, void* stream) {
  kvq_status s = check_cache(cache);
  if (s) return s;
  if (!dev_amax || !aligned(dev_amax, 4)) return fail(KVQ_ERR_INVALID_ARG, "dev_amax must be non-NULL and 4-byte aligned");
  if (!tensor_scaled(cache->cfg.mode)) return fail(KVQ_ERR_MODE_MISMATCH, "mode %d has no per-tensor scale", cache->cfg.mode);
  const float div = cache->cfg.mode == KVQ_FP8_PER_TENSOR ? 448.0f : 2688.0f;
  cudaError_t e = kvq::launch_scales_from_amax(cache->base, dev_amax, dev_amax, div, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "scale launch");
  return KVQ_OK;
}

kvq_status kvq_latent_read_errors(kvq_latent* cache, uint32_t* flags, int clear, void* stream) {
  kvq_status s = check_cache(cache);
  if (s) return s;
  if (!flags) return fail(KVQ_ERR_INVALID_ARG, "flags is NULL");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint32_t v = 0;
  cudaError_t e = cudaMemcpyAsync(&v, cache->base + kvq::kHdrErrOffset, 4, cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e == cudaSuccess && clear) e = cudaMemsetAsync(cache->base + kvq::kHdrErrOffset, 0, 4, st);
  if (e != cudaSuccess) return cuda_fail(e, "reading the error word");
  *flags = v;
  return KVQ_OK;
}

kvq_status kvq_latent_write(kvq_latent* cache, const kvq_latent_rows* r, int mode, void* stream) {
  kvq_status s = check_cache(cache);
  if (s) return s;
  if (mode != cache->cfg.mode)
    return fail(KVQ_ERR_MODE_MISMATCH, "write mode %d but the cache holds mode %d", mode, cache->cfg.mode);
  if (!r) return fail(KVQ_ERR_INVALID_ARG, "the argument struct is NULL");
  const int esize = cache->cfg.io_dtype == KVQ_F16 ? 2 : 4;
  if (r->num_tokens < 0) return fail(KVQ_ERR_INVALID_ARG, "num_tokens < 0");
  if (r->max_position <= 0) return fail(KVQ_ERR_INVALID_ARG, "max_position must be positive");
  if (!(r->eps >= 0.0f) || r->eps > 3.0e38f) return fail(KVQ_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (!r->q_rope != !r->q_rope_out) return fail(KVQ_ERR_INVALID_ARG, "q_rope and q_rope_out go together");
  if (r->q_rope && r->num_q_heads <= 0) return fail(KVQ_ERR_INVALID_ARG, "num_q_heads must be positive");
  if (!stride_ok(r->latent_stride, esize) || !stride_ok(r->k_rope_stride, esize) || !stride_ok(r->q_stride, esize) ||
      !stride_ok(r->q_head_stride, esize) || !stride_ok(r->q_out_stride, esize) || !stride_ok(r->q_out_head_stride, esize))
    return fail(KVQ_ERR_INVALID_ARG, "strides must be non-negative multiples of 16 bytes");
  if (r->num_tokens == 0) return KVQ_OK;
  if (!r->latent || !r->k_rope || !r->positions || !r->cos_sin)
    return fail(KVQ_ERR_INVALID_ARG, "NULL latent, k_rope, positions or cos_sin");
  if (!aligned(r->latent, 16) || !aligned(r->k_rope, 16) || !aligned(r->q_rope, 16) || !aligned(r->q_rope_out, 16) ||
      !aligned(r->latent_weight, 16) || !aligned(r->cos_sin, 16) || !aligned(r->latent_out, 16) || !aligned(r->k_rope_out, 16))
    return fail(KVQ_ERR_INVALID_ARG, "rows, weights, cos_sin and outputs must be 16-byte aligned");
  if (!aligned(r->positions, 4) || !aligned(r->slot_mapping, 4))
    return fail(KVQ_ERR_INVALID_ARG, "positions and slot_mapping must be 4-byte aligned");
  cudaError_t e = kvq::launch_latent_write(cache, *r, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "latent write launch");
  return KVQ_OK;
}

kvq_status kvq_latent_read(const kvq_latent* cache, const int32_t* slot_mapping, int num_tokens, void* latent_out,
                           void* rope_out, int out_dtype, void* stream) {
  kvq_status s = check_cache(cache);
  if (s) return s;
  if (num_tokens < 0) return fail(KVQ_ERR_INVALID_ARG, "num_tokens < 0");
  if (out_dtype != KVQ_F16 && out_dtype != KVQ_F32) return fail(KVQ_ERR_UNSUPPORTED, "out_dtype %d", out_dtype);
  if (num_tokens == 0 || (!latent_out && !rope_out)) return KVQ_OK;
  if (!slot_mapping || !aligned(slot_mapping, 4))
    return fail(KVQ_ERR_INVALID_ARG, "slot_mapping must be non-NULL and 4-byte aligned");
  if (!aligned(latent_out, 16) || !aligned(rope_out, 16)) return fail(KVQ_ERR_INVALID_ARG, "outputs must be 16-byte aligned");
  cudaError_t e = kvq::launch_latent_read(cache, slot_mapping, num_tokens, latent_out, rope_out, out_dtype,
                                          static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "latent read launch");
  return KVQ_OK;
}

namespace {
kvq_status check_sizes(const kvq_latent* cache, int total_q, int num_seqs, int num_q_heads, int max_q_len, int max_len) {
  kvq_status s = check_cache(cache);
  if (s) return s;
  if (total_q < 0 || num_seqs < 0 || max_q_len < 0 || max_len < 0) return fail(KVQ_ERR_INVALID_ARG, "negative size");
  if (num_q_heads <= 0) return fail(KVQ_ERR_INVALID_ARG, "num_q_heads must be positive");
  if (num_q_heads > 65535) return fail(KVQ_ERR_UNSUPPORTED, "num_q_heads %d > 65535", num_q_heads);
  if ((long long)total_q * num_q_heads > 0x7fffffffll || (long long)max_q_len * num_q_heads > 0x7fffffffll)
    return fail(KVQ_ERR_UNSUPPORTED, "2^31 query rows or more");
  if (max_len > 0x7fffffff - 4096) return fail(KVQ_ERR_UNSUPPORTED, "sequences of 2^31 - 4096 tokens or more");
  return KVQ_OK;
}
// The checks that follow when there is work to do.
kvq_status check_call(const int32_t* cu_q_lens, const void* q, const void* out, const float* lse, int max_q_len) {
  if (max_q_len == 0) return fail(KVQ_ERR_INVALID_ARG, "max_q_len is 0 but there are query rows");
  if (!q || !out) return fail(KVQ_ERR_INVALID_ARG, "NULL q or out");
  if (!aligned(q, 16) || !aligned(out, 16)) return fail(KVQ_ERR_INVALID_ARG, "q and out must be 16-byte aligned");
  if (!cu_q_lens || !aligned(cu_q_lens, 4)) return fail(KVQ_ERR_INVALID_ARG, "cu_q_lens must be non-NULL and 4-byte aligned");
  if (!aligned(lse, 4)) return fail(KVQ_ERR_INVALID_ARG, "lse must be 4-byte aligned");
  return KVQ_OK;
}
kvq_status check_types(int out_dtype, float softmax_scale) {
  if (out_dtype != KVQ_F16 && out_dtype != KVQ_F32) return fail(KVQ_ERR_UNSUPPORTED, "out_dtype %d", out_dtype);
  if (!(softmax_scale > 0.0f) || softmax_scale > 3.0e38f)
    return fail(KVQ_ERR_INVALID_ARG, "softmax_scale must be finite and > 0");
  return KVQ_OK;
}
}  // namespace

kvq_status kvq_latent_plan(const kvq_latent* cache, int total_q, int num_seqs, int num_q_heads, int max_q_len,
                           int max_seq_len, int* num_splits, size_t* workspace_bytes) {
  kvq_status s = check_sizes(cache, total_q, num_seqs, num_q_heads, max_q_len, max_seq_len);
  if (s) return s;
  const kvq::LatentPlan p =
      kvq::plan_latent(cache, total_q, num_seqs, num_q_heads, max_q_len, max_seq_len, cache->cfg.io_dtype);
  if (num_splits) *num_splits = p.num_splits;
  if (workspace_bytes) *workspace_bytes = p.workspace_bytes;
  return KVQ_OK;
}

kvq_status kvq_latent_attention(const kvq_latent* cache, const void* q, int total_q, const int32_t* cu_q_lens,
                                const int32_t* block_table, int max_pages, const int32_t* seq_lens, int num_seqs,
                                int num_q_heads, int max_q_len, int max_seq_len, int mode, float softmax_scale,
                                int causal, void* out, int out_dtype, float* lse, void* workspace,
                                size_t workspace_bytes, void* stream) {
  kvq_status s = check_sizes(cache, total_q, num_seqs, num_q_heads, max_q_len, max_seq_len);
  if (s) return s;
  if (mode != cache->cfg.mode)
    return fail(KVQ_ERR_MODE_MISMATCH, "attention mode %d but the cache holds mode %d", mode, cache->cfg.mode);
  if (max_pages < 0) return fail(KVQ_ERR_INVALID_ARG, "negative size");
  if ((long long)max_seq_len > (long long)max_pages * 16)
    return fail(KVQ_ERR_INVALID_ARG, "max_seq_len %d exceeds max_pages * page_size", max_seq_len);
  s = check_types(out_dtype, softmax_scale);
  if (s || total_q == 0 || num_seqs == 0) return s;
  s = check_call(cu_q_lens, q, out, lse, max_q_len);
  if (s) return s;
  if (!block_table || !seq_lens) return fail(KVQ_ERR_INVALID_ARG, "NULL table or lens");
  if (!aligned(block_table, 4) || !aligned(seq_lens, 4))
    return fail(KVQ_ERR_INVALID_ARG, "block_table and seq_lens must be 4-byte aligned");
  const kvq::LatentPlan p = kvq::plan_latent(cache, total_q, num_seqs, num_q_heads, max_q_len, max_seq_len, out_dtype);
  if (p.workspace_bytes > 0) {
    if (!workspace || workspace_bytes < p.workspace_bytes)
      return fail(KVQ_ERR_CAPACITY, "workspace needs %zu bytes, got %zu", p.workspace_bytes, workspace ? workspace_bytes : 0);
    if (!aligned(workspace, 16)) return fail(KVQ_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  }
  kvq::LatentArgs a = {};
  a.pool = cache->base;
  a.q = q;
  a.cu_q = cu_q_lens;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.out = out;
  a.lse = lse;
  a.total_q = total_q;
  a.B = num_seqs;
  a.Hq = a.G = num_q_heads;
  a.Hkv = 1;
  a.num_pages = cache->cfg.num_pages;
  a.max_pages = max_pages;
  a.max_q_len = max_q_len;
  a.max_seq_len = max_seq_len;
  a.out_f32 = out_dtype == KVQ_F32;
  a.scale = softmax_scale;
  a.causal = causal != 0;
  a.block_bytes = cache->page_bytes;
  a.ws_o = static_cast<float*>(workspace);
  uint8_t* w = static_cast<uint8_t*>(workspace);
  a.ws_span = kvq::Span{w, w ? w + p.workspace_bytes : nullptr};
  cudaError_t e = kvq::launch_latent_attention(cache, p, a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "latent attention launch");
  return KVQ_OK;
}

kvq_status kvq_latent_prompt_attention(const kvq_latent* cache, const kvq_latent_prompt* p, void* stream) {
  kvq_status s = check_cache(cache);
  if (s) return s;
  if (!p) return fail(KVQ_ERR_INVALID_ARG, "the argument struct is NULL");
  s = check_sizes(cache, p->total_q, p->num_seqs, p->num_q_heads, p->max_q_len, p->max_k_len);
  if (s) return s;
  if (p->total_k < 0) return fail(KVQ_ERR_INVALID_ARG, "negative size");
  s = check_types(p->out_dtype, p->softmax_scale);
  if (s) return s;
  const int esize = cache->cfg.io_dtype == KVQ_F16 ? 2 : 4;
  if (!stride_ok(p->k_stride, esize) || !stride_ok(p->k_head_stride, esize) || !stride_ok(p->v_stride, esize) ||
      !stride_ok(p->v_head_stride, esize) || !stride_ok(p->k_rope_stride, esize))
    return fail(KVQ_ERR_INVALID_ARG, "strides must be non-negative multiples of 16 bytes");
  if (p->total_q == 0 || p->num_seqs == 0) return KVQ_OK;
  s = check_call(p->cu_q_lens, p->q, p->out, p->lse, p->max_q_len);
  if (s) return s;
  if (!p->cu_k_lens || !aligned(p->cu_k_lens, 4))
    return fail(KVQ_ERR_INVALID_ARG, "cu_k_lens must be non-NULL and 4-byte aligned");
  if (p->total_k > 0 && (!p->k || !p->k_rope || !p->v)) return fail(KVQ_ERR_INVALID_ARG, "NULL k, k_rope or v");
  if (!aligned(p->k, 16) || !aligned(p->k_rope, 16) || !aligned(p->v, 16))
    return fail(KVQ_ERR_INVALID_ARG, "k, k_rope and v must be 16-byte aligned");
  kvq::LatentArgs a = {};
  a.pool = cache->base;
  a.q = p->q;
  a.cu_q = p->cu_q_lens;
  a.cu_k = p->cu_k_lens;
  a.k = p->k;
  a.k_rope = p->k_rope;
  a.v = p->v;
  a.k_stride = p->k_stride;
  a.k_head_stride = p->k_head_stride;
  a.v_stride = p->v_stride;
  a.v_head_stride = p->v_head_stride;
  a.k_rope_stride = p->k_rope_stride;
  a.out = p->out;
  a.lse = p->lse;
  a.total_q = p->total_q;
  a.total_k = p->total_k;
  a.B = p->num_seqs;
  a.Hq = a.Hkv = p->num_q_heads;
  a.G = 1;
  a.max_q_len = p->max_q_len;
  a.max_seq_len = p->max_k_len;
  a.out_f32 = p->out_dtype == KVQ_F32;
  a.scale = p->softmax_scale;
  a.causal = p->causal != 0;
  cudaError_t e = kvq::launch_latent_prompt(cache, a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "latent prompt attention launch");
  return KVQ_OK;
}

}  // extern "C"
