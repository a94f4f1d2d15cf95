// Device-resident KV pools, host side: configuration checks, workspace carving and the C-ABI entry points.
#include <math.h>

#include <algorithm>
#include <new>

#include "kvs_rope.cuh"

using namespace kvs;

struct kvs_pool {
  PoolDims d;
  unsigned char *k, *v;     // [n_layer][n_slots][H_kv][bs][d]
  size_t layer_bytes;
  int device;
  unsigned* err;
  float *lse2, *prev_lse2, *prev_out;
  void* scratch;
  CUtensorMap* maps;        // per layer: K, V, and K as the products read its codes (E4M3)
  unsigned long long launches;
};

namespace {

constexpr size_t kAlign = 256;
constexpr int kTicketWord = 16;     // a counter of CTAs beside the status word, 0 between calls
size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
// [a, a + na) and [b, b + nb) share a byte
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool pool_dims(const kvs_pool_config* c, PoolDims* d) {
  if (!c) return false;
  if (c->n_layer < 1 || c->n_layer > 1024 || c->n_slots < 1) return false;
  if (c->n_q_head < 1 || c->n_kv_head < 1 || c->n_kv_head > 1024 || c->n_q_head % c->n_kv_head) return false;
  if (c->n_q_head / c->n_kv_head > 128) return false;
  if (c->head_dim != 64 && c->head_dim != 128) return false;
  if (c->block_size != 16 && c->block_size != 32 && c->block_size != 64 && c->block_size != 128) return false;
  if (c->max_ctx < 1 || c->max_ctx > (1 << 30) || c->max_req < 1 || c->max_req > kPoolMaxReq) return false;
  if ((long long)c->max_req * c->n_kv_head > 65535) return false;   // (request, kv head) pairs are a grid dimension
  if (c->max_tokens < 1 || c->max_tokens > (1 << 24)) return false;
  if (c->max_prefix_tokens < 0 || c->max_prefix_tokens > c->max_tokens) return false;
  if (c->kv_dtype != KVS_KV_BF16 && c->kv_dtype != KVS_KV_FP8_E4M3) return false;
  if (!(c->softmax_scale >= 0.f) || isinf(c->softmax_scale)) return false;
  if (!(c->k_scale >= 0.f) || !(c->v_scale >= 0.f) || isinf(c->k_scale) || isinf(c->v_scale)) return false;
  // rows of a layer are tensor-load coordinates (32 bits), and rows of a (request, kv head) are divided by G through 2^32 / G
  if ((long long)c->n_slots * c->n_kv_head * c->block_size > 0x7fff0000ll) return false;
  if ((long long)c->max_tokens * (c->n_q_head / c->n_kv_head) > (1 << 25)) return false;
  // row blocks of a call are counted in 32 bits, for any offsets: each request may be given all tokens
  if ((long long)c->max_req * c->max_tokens > (1ll << 37) / c->n_q_head) return false;
  d->NL = c->n_layer;
  d->n_slots = c->n_slots;
  d->Hq = c->n_q_head;
  d->Hkv = c->n_kv_head;
  d->G = c->n_q_head / c->n_kv_head;
  d->d = c->head_dim;
  d->bs = c->block_size;
  d->rt = 128 / d->G * d->G;
  d->g_magic = (unsigned)(((1ull << 32) + d->G - 1) / d->G);
  d->log2bs = 0;
  while ((1 << d->log2bs) < d->bs) ++d->log2bs;
  d->max_ctx = c->max_ctx;
  d->nb_max = (c->max_ctx + c->block_size - 1) / c->block_size;
  d->max_req = c->max_req;
  d->max_tokens = c->max_tokens;
  d->max_prefix_tokens = c->max_prefix_tokens;
  d->fp8 = c->kv_dtype == KVS_KV_FP8_E4M3;
  d->ebytes = d->fp8 ? 1 : 2;
  d->scale = c->softmax_scale > 0.f ? c->softmax_scale : (float)(1.0 / sqrt((double)c->head_dim));
  d->k_scale = d->fp8 && c->k_scale > 0.f ? c->k_scale : 1.f;
  d->v_scale = d->fp8 && c->v_scale > 0.f ? c->v_scale : 1.f;
  d->timeout_us = c->wait_timeout_us ? c->wait_timeout_us : 2000000u;
  return true;
}

struct PoolPlan {
  size_t err, lse2, prev_lse2, prev_out, scratch, total;
};
PoolPlan pool_plan(const PoolDims& d) {
  PoolPlan p;
  p.err = align_up((kTicketWord + 1) * 4);
  p.lse2 = align_up((size_t)d.max_tokens * d.Hq * 4);
  p.prev_lse2 = align_up((size_t)d.max_prefix_tokens * d.Hq * 4);
  p.prev_out = align_up((size_t)d.max_prefix_tokens * d.Hq * d.d * 4);
  p.scratch = align_up(std::max(pool_attn_scratch_bytes(d), pool_weight_scratch_bytes()));
  p.total = p.err + p.lse2 + p.prev_lse2 + p.prev_out + p.scratch;
  return p;
}

inline cudaStream_t S(kvs_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }
inline kvs_status cuda_status(cudaError_t e) { return e == cudaSuccess ? KVS_OK : KVS_ERR_CUDA; }

// Arguments every call on a layer shares.
bool call_ok(const kvs_pool* p, int layer, int n_req) {
  if (!p || layer < 0 || layer >= p->d.NL || n_req < 0 || n_req > p->d.max_req) return false;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  return dev == p->device;
}

bool query_ok(const kvs_pool* p, const void* q, long long q_stride, const int* cu_q, const int* ctx_len,
              const int* table, const void* out, int n_tok) {
  if (!q || !cu_q || !ctx_len || !table || !out) return false;
  const size_t row = (size_t)p->d.Hq * p->d.d;
  if (!aligned16(q) || !aligned16(out) || q_stride % 8 || q_stride < (long long)row) return false;
  // a row split over several CTAs is written while others may still read its q
  return !overlap(q, ((size_t)(n_tok - 1) * q_stride + row) * 2, out, n_tok * row * 2);
}

}  // namespace

namespace kvs {
bool make_pool_q_map(CUtensorMap* m, const PoolDims& d, const __nv_bfloat16* q, long long q_stride, int n_tok) {
  const uint64_t dims[3] = {(uint64_t)d.d, (uint64_t)d.Hq, (uint64_t)n_tok};
  const uint64_t strides[2] = {(uint64_t)d.d * 2, (uint64_t)q_stride * 2};
  const uint32_t box[3] = {64, (uint32_t)d.G, (uint32_t)(d.rt / d.G)};
  return encode_tmap(m, const_cast<__nv_bfloat16*>(q), 3, dims, strides, box, 2, 128);
}
}  // namespace kvs

extern "C" {

size_t kvs_pool_workspace_bytes(const kvs_pool_config* cfg) {
  PoolDims d;
  if (!pool_dims(cfg, &d)) return 0;
  return pool_plan(d).total;
}

kvs_status kvs_pool_create(const kvs_pool_config* cfg, void* d_k, void* d_v, void* d_workspace,
                           size_t workspace_bytes, kvs_pool** out) try {
  if (!out) return KVS_ERR_INVALID_ARG;
  *out = nullptr;
  PoolDims d;
  if (!pool_dims(cfg, &d)) return KVS_ERR_INVALID_ARG;
  const PoolPlan p = pool_plan(d);
  if (!d_k || !d_v || !d_workspace || workspace_bytes < p.total) return KVS_ERR_INVALID_ARG;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return KVS_ERR_CUDA;
  }
  for (void* x : {d_k, d_v, d_workspace}) {
    cudaPointerAttributes a;
    if (reinterpret_cast<uintptr_t>(x) % kAlign) return KVS_ERR_INVALID_ARG;
    if (cudaPointerGetAttributes(&a, x) != cudaSuccess || a.type != cudaMemoryTypeDevice || a.device != dev) {
      cudaGetLastError();
      return KVS_ERR_INVALID_ARG;
    }
  }
  const size_t bytes = (size_t)d.NL * d.n_slots * d.Hkv * d.bs * d.d * d.ebytes;
  if (overlap(d_k, bytes, d_v, bytes) || overlap(d_k, bytes, d_workspace, p.total) || overlap(d_v, bytes, d_workspace, p.total))
    return KVS_ERR_INVALID_ARG;
  kvs_pool* c = new (std::nothrow) kvs_pool();
  if (!c) return KVS_ERR_INVALID_ARG;
  c->maps = new (std::nothrow) CUtensorMap[3 * (size_t)d.NL];
  if (!c->maps) {
    delete c;
    return KVS_ERR_INVALID_ARG;
  }
  c->d = d;
  c->k = static_cast<unsigned char*>(d_k);
  c->v = static_cast<unsigned char*>(d_v);
  c->layer_bytes = (size_t)d.n_slots * d.Hkv * d.bs * d.d * d.ebytes;
  c->device = dev;
  c->launches = 0;
  unsigned char* b = static_cast<unsigned char*>(d_workspace);
  c->err = reinterpret_cast<unsigned*>(b); b += p.err;
  c->lse2 = reinterpret_cast<float*>(b); b += p.lse2;
  c->prev_lse2 = reinterpret_cast<float*>(b); b += p.prev_lse2;
  c->prev_out = reinterpret_cast<float*>(b); b += p.prev_out;
  c->scratch = b;
  // each layer's rows [n_slots * H_kv * bs][d]; a load brings one block's rows: 64 dims of bf16 (128 bytes,
  // swizzled as the products read them), or all dims of E4M3 codes, as they are
  const uint64_t rows = (uint64_t)d.n_slots * d.Hkv * d.bs;
  const uint32_t inner = (uint32_t)(d.fp8 ? d.d : 64);
  // (E4M3's third map: the same boxes of K, swizzled)
  for (int l = 0; l < d.NL; ++l)
    for (int x = 0; x < (d.fp8 ? 3 : 2); ++x)
      if (!make_tmap_2d(&c->maps[3 * l + x], (x == 1 ? c->v : c->k) + l * c->layer_bytes, (uint64_t)d.d, rows, inner,
                        (uint32_t)d.bs, d.ebytes, !d.fp8 ? 128 : x == 2 ? d.d : 0)) {
        kvs_pool_destroy(c);
        return KVS_ERR_CUDA;
      }
  if (cudaMemset(c->err, 0, p.err) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess) {
    kvs_pool_destroy(c);
    return KVS_ERR_CUDA;
  }
  *out = c;
  return KVS_OK;
} catch (...) {      // out of host memory
  return KVS_ERR_CUDA;
}

kvs_status kvs_pool_destroy(kvs_pool* c) {
  if (!c) return KVS_ERR_INVALID_ARG;
  delete[] c->maps;
  delete c;
  return KVS_OK;
}

kvs_status kvs_pool_poll_error(kvs_pool* c, kvs_status* device_status) {
  if (!c || !device_status || !call_ok(c, 0, 0)) return KVS_ERR_INVALID_ARG;
  unsigned v = 0;
  cudaError_t e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = cudaMemcpy(&v, c->err, sizeof(v), cudaMemcpyDeviceToHost);
  if (e == cudaSuccess) e = cudaMemset(c->err, 0, sizeof(v));
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  *device_status = static_cast<kvs_status>(v);
  return cuda_status(e);
}

unsigned long long kvs_pool_launch_count(kvs_pool* c) { return c ? c->launches : 0ull; }

kvs_status kvs_pool_append(kvs_pool* c, int layer, const void* d_k_new, const void* d_v_new, long long kv_stride,
                           const int* d_cu_q, const int* d_ctx_len, const int* d_block2slot, int n_req, int n_tok,
                           kvs_stream_t stream) try {
  if (!call_ok(c, layer, n_req) || n_tok < 0 || n_tok > c->d.max_tokens) return KVS_ERR_INVALID_ARG;
  const PoolDims& d = c->d;
  if (n_req == 0 || n_tok == 0) return KVS_OK;
  if (!d_k_new || !d_v_new || !d_cu_q || !d_ctx_len || !d_block2slot) return KVS_ERR_INVALID_ARG;
  if (kv_stride % 8 || kv_stride < (long long)d.Hkv * d.d) return KVS_ERR_INVALID_ARG;
  if (!aligned16(d_k_new) || !aligned16(d_v_new)) return KVS_ERR_INVALID_ARG;
  const PoolSeqs q = {d_cu_q, nullptr, d_ctx_len, d_block2slot, n_req, n_req, n_tok, 1, 0, 0};
  c->launches += 1;
  return cuda_status(launch_pool_append(d, c->k + layer * c->layer_bytes, c->v + layer * c->layer_bytes,
                                        static_cast<const __nv_bfloat16*>(d_k_new),
                                        static_cast<const __nv_bfloat16*>(d_v_new), kv_stride, q, c->err, S(stream)));
} catch (...) {      // out of host memory
  return KVS_ERR_CUDA;
}

kvs_status kvs_pool_attn(kvs_pool* c, int layer, const void* d_q, long long q_stride, const int* d_cu_q,
                         const int* d_ctx_len, const int* d_block2slot, int n_req, int n_tok, int window, int n_sink,
                         void* d_out, float* d_lse, float* d_weight, kvs_stream_t stream) try {
  if (!call_ok(c, layer, n_req) || window < 0 || n_sink < 0) return KVS_ERR_INVALID_ARG;
  const PoolDims& d = c->d;
  if (n_tok < 0 || n_tok > d.max_tokens) return KVS_ERR_INVALID_ARG;
  if (n_req == 0 || n_tok == 0) return KVS_OK;
  if (!query_ok(c, d_q, q_stride, d_cu_q, d_ctx_len, d_block2slot, d_out, n_tok)) return KVS_ERR_INVALID_ARG;
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(d_q);
  if (window >= d.max_ctx) window = 0;           // no key is that far away (and position + window stays in 32 bits)
  if (n_sink > d.max_ctx) n_sink = d.max_ctx;
  const unsigned char* k = c->k + layer * c->layer_bytes;
  const PoolSeqs seqs = {d_cu_q, nullptr, d_ctx_len, d_block2slot, n_req, n_req, n_tok, 1, window, n_sink};
  const PoolAttnOut o = {static_cast<__nv_bfloat16*>(d_out), d_lse, d_weight ? c->lse2 : nullptr, nullptr, nullptr, nullptr,
                         nullptr, 0};
  int n = 0;
  cudaError_t e = launch_pool_attn(d, k, c->v + layer * c->layer_bytes, &c->maps[3 * layer], q, q_stride, seqs, o,
                                   c->scratch, c->err, S(stream), &n);
  c->launches += n;
  if (e == cudaSuccess && d_weight) {
    e = launch_pool_weight(d, &c->maps[3 * layer], q, q_stride, seqs, c->lse2, d_weight, c->scratch, c->err, S(stream), &n);
    c->launches += n;
  }
  return cuda_status(e);
} catch (...) {      // out of host memory
  return KVS_ERR_CUDA;
}

kvs_status kvs_pool_prefix_attn(kvs_pool* c, int layer, const void* d_q, long long q_stride, const int* d_cu_q,
                                const int* d_ctx_len, const int* d_block2slot, int n_req, int n_tok,
                                const int* d_prefix_req, const int* d_prefix_len, const int* d_prefix2slot, int n_prefix,
                                void* d_out, float* d_lse, kvs_stream_t stream) try {
  if (!call_ok(c, layer, n_req) || n_prefix < 0 || n_prefix > c->d.max_req) return KVS_ERR_INVALID_ARG;
  const PoolDims& d = c->d;
  if (n_tok < 0 || n_tok > d.max_prefix_tokens) return KVS_ERR_INVALID_ARG;
  if (n_req == 0 || n_tok == 0) return KVS_OK;
  if (!query_ok(c, d_q, q_stride, d_cu_q, d_ctx_len, d_block2slot, d_out, n_tok)) return KVS_ERR_INVALID_ARG;
  if (n_prefix > 0 && (!d_prefix_req || !d_prefix_len || !d_prefix2slot)) return KVS_ERR_INVALID_ARG;
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(d_q);
  const unsigned char *k = c->k + layer * c->layer_bytes, *v = c->v + layer * c->layer_bytes;
  cudaError_t e = cudaSuccess;
  int n = 0;
  if (n_prefix > 0) {
    const PoolSeqs pre = {d_cu_q, d_prefix_req, d_prefix_len, d_prefix2slot, n_prefix, n_req, n_tok, 0, 0, 0};
    const PoolAttnOut o = {nullptr, nullptr, c->prev_lse2, c->prev_out, nullptr, nullptr, nullptr, 0};
    e = launch_pool_attn(d, k, v, &c->maps[3 * layer], q, q_stride, pre, o, c->scratch, c->err, S(stream), &n);
    c->launches += n;
  }
  if (e == cudaSuccess) {
    const PoolSeqs own = {d_cu_q, nullptr, d_ctx_len, d_block2slot, n_req, n_req, n_tok, 1, 0, 0};
    // without prefixes there are no earlier rows, and d_prefix_req may be NULL
    const PoolAttnOut o = {static_cast<__nv_bfloat16*>(d_out), d_lse, nullptr, nullptr, n_prefix > 0 ? c->prev_out : nullptr,
                           c->prev_lse2, d_prefix_req, n_prefix};
    e = launch_pool_attn(d, k, v, &c->maps[3 * layer], q, q_stride, own, o, c->scratch, c->err, S(stream), &n);
    c->launches += n;
  }
  return cuda_status(e);
} catch (...) {      // out of host memory
  return KVS_ERR_CUDA;
}

kvs_status kvs_pool_evict(kvs_pool* c, int layer, const float* d_weight, const int* d_ctx_len,
                          const int* d_block2slot, int n_req, int keep, int n_sink, int n_recent, const int* d_dst2slot,
                          int* d_kept, int* d_n_kept, float* d_weight_out, kvs_stream_t stream) try {
  if (!call_ok(c, layer, n_req)) return KVS_ERR_INVALID_ARG;
  const PoolDims& d = c->d;
  if (keep < 1 || keep > d.max_ctx || n_sink < 0 || n_recent < 0 || n_sink > keep || n_recent > keep - n_sink)
    return KVS_ERR_INVALID_ARG;
  if (n_req == 0) return KVS_OK;
  if (!d_weight || !d_ctx_len || !d_block2slot || !d_dst2slot || !d_kept || !d_n_kept || !d_weight_out) return KVS_ERR_INVALID_ARG;
  // what the call reads it may not write: other CTAs still read it
  const size_t weights = (size_t)n_req * d.Hkv * d.max_ctx * 4;
  if (overlap(d_weight, weights, d_weight_out, weights) || d_block2slot == d_dst2slot ||
      overlap(d_ctx_len, (size_t)n_req * 4, d_n_kept, (size_t)n_req * 4))
    return KVS_ERR_INVALID_ARG;
  c->launches += 2;
  return cuda_status(launch_pool_evict(d, c->k + layer * c->layer_bytes, c->v + layer * c->layer_bytes, d_weight, d_ctx_len,
                                       d_block2slot, n_req, keep, n_sink, n_recent, d_dst2slot, d_kept, d_n_kept,
                                       d_weight_out, c->err, S(stream)));
} catch (...) {      // out of host memory
  return KVS_ERR_CUDA;
}

kvs_status kvs_pool_reserve(kvs_pool* c, const int* d_ctx_len, int* d_n_held, int* d_block2slot, int* d_ring, int* d_ring_state,
                            int n_req, const int* d_cu_q, const int* d_pos_delta, int n_tok, long long* d_place, int* d_pos,
                            kvs_stream_t stream) try {
  if (!call_ok(c, 0, n_req) || n_tok < 0 || n_tok > c->d.max_tokens) return KVS_ERR_INVALID_ARG;
  if (n_req == 0) return n_tok == 0 ? KVS_OK : kvs_pool_places(c, d_cu_q, d_ctx_len, d_block2slot, 0, n_tok, d_pos_delta, d_place, d_pos, stream);
  if (!d_ctx_len || !d_n_held || !d_block2slot || !d_ring || !d_ring_state || d_ctx_len == d_n_held) return KVS_ERR_INVALID_ARG;
  if (n_tok == 0) d_cu_q = nullptr;
  if (n_tok > 0 && (!d_cu_q || !d_place)) return KVS_ERR_INVALID_ARG;
  const PoolTables t = {d_ctx_len, d_n_held, d_block2slot, d_ring, d_ring_state, d_cu_q, d_pos_delta, d_place, d_pos, n_req, n_tok};
  c->launches += 1;
  return cuda_status(launch_pool_tables(c->d, t, c->err + kTicketWord, c->err, S(stream)));
} catch (...) {      // out of host memory
  return KVS_ERR_CUDA;
}

kvs_status kvs_pool_places(kvs_pool* c, const int* d_cu_q, const int* d_ctx_len, const int* d_block2slot, int n_req, int n_tok,
                           const int* d_pos_delta, long long* d_place, int* d_pos, kvs_stream_t stream) try {
  if (!call_ok(c, 0, n_req) || n_tok < 0 || n_tok > c->d.max_tokens) return KVS_ERR_INVALID_ARG;
  if (n_tok == 0) return KVS_OK;
  if (!d_cu_q || !d_place || (n_req > 0 && (!d_ctx_len || !d_block2slot))) return KVS_ERR_INVALID_ARG;      // (no request: nobody's tokens)
  const PoolTables t = {d_ctx_len, nullptr, const_cast<int*>(d_block2slot), nullptr, nullptr, d_cu_q, d_pos_delta, d_place, d_pos, n_req, n_tok};
  c->launches += 1;
  return cuda_status(launch_pool_tables(c->d, t, c->err + kTicketWord, c->err, S(stream)));
} catch (...) {      // out of host memory
  return KVS_ERR_CUDA;
}

kvs_status kvs_pool_rotate_append(kvs_pool* c, const kvs_rope* rope, int layer, const void* d_q, long long q_stride,
                                  const void* d_k, const void* d_v, long long kv_stride, const float* d_q_norm,
                                  const float* d_k_norm, const int* d_pos, long long pos_stride, const long long* d_place,
                                  int n_tok, void* d_q_out, long long q_out_stride, kvs_stream_t stream) try {
  if (!call_ok(c, layer, 0) || !rope || n_tok < 0 || n_tok > c->d.max_tokens || pos_stride < 0) return KVS_ERR_INVALID_ARG;
  const PoolDims& d = c->d;
  if (rope->d.d != d.d) return KVS_ERR_INVALID_ARG;
  if (n_tok == 0) return KVS_OK;
  if (!d_q || !d_k || !d_v || !d_pos || !d_place || !d_q_out) return KVS_ERR_INVALID_ARG;
  const long long q_row = (long long)d.Hq * d.d, kv_row = (long long)d.Hkv * d.d;
  const long long most = (1ll << 40) / n_tok;      // (extents stay in 64 bits, and within any memory)
  if (q_stride % 8 || kv_stride % 8 || q_out_stride % 8 || q_stride < q_row || kv_stride < kv_row || q_out_stride < q_row || q_stride > most ||
      kv_stride > most || q_out_stride > most)
    return KVS_ERR_INVALID_ARG;
  for (const void* x : {d_q, d_k, d_v, static_cast<const void*>(d_q_out), static_cast<const void*>(d_q_norm), static_cast<const void*>(d_k_norm)})
    if (!aligned16(x)) return KVS_ERR_INVALID_ARG;
  // rows are written while others are still read: q in place, or apart from q, k and v (columns of the same rows may be)
  const bool in_place = d_q == d_q_out && q_stride == q_out_stride;
  auto meets = [&](const void* x, long long stride, long long row) {
    const size_t more = (size_t)(n_tok - 1) * 2;
    if (!overlap(x, more * stride + row * 2, d_q_out, more * q_out_stride + q_row * 2)) return false;
    if (stride != q_out_stride || n_tok == 1) return true;
    const uintptr_t a = reinterpret_cast<uintptr_t>(x), b = reinterpret_cast<uintptr_t>(d_q_out);
    const uintptr_t off = (a < b ? b - a : a - b) % (stride * 2), wa = (a < b ? row : q_row) * 2, wb = (a < b ? q_row : row) * 2;
    return !(off >= wa && off + wb <= (uintptr_t)stride * 2);
  };
  if ((!in_place && meets(d_q, q_stride, q_row)) || meets(d_k, kv_stride, kv_row) || meets(d_v, kv_stride, kv_row)) return KVS_ERR_INVALID_ARG;
  RopeRows a = {};
  const long long head = d.d;
  a.q = {static_cast<const __nv_bfloat16*>(d_q), static_cast<__nv_bfloat16*>(d_q_out), q_stride, head, q_out_stride, head, d_q_norm, d.Hq};
  a.k = {static_cast<const __nv_bfloat16*>(d_k), nullptr, kv_stride, head, 0, 0, d_k_norm, d.Hkv};
  a.v = {static_cast<const __nv_bfloat16*>(d_v), nullptr, kv_stride, head, 0, 0, nullptr, d.Hkv};
  a.pos = d_pos;
  a.pos_stride = pos_stride;
  a.place = d_place;
  a.kpool = c->k + layer * c->layer_bytes;
  a.vpool = c->v + layer * c->layer_bytes;
  a.n_slots = d.n_slots;
  a.bs = d.bs;
  a.log2bs = d.log2bs;
  a.fp8 = d.fp8;
  a.k_scale = d.k_scale;
  a.v_scale = d.v_scale;
  auto rcp = [](float s) { return s >= 0x1p-60f && s <= 0x1p60f ? 1.f / s : 0.f; };
  a.k_rcp = rcp(d.k_scale);
  a.v_rcp = rcp(d.v_scale);
  a.err = c->err;
  a.n_tok = n_tok;
  c->launches += 1;
  return cuda_status(launch_rope_rows(rope->d, a, S(stream)));
} catch (...) {      // out of host memory
  return KVS_ERR_CUDA;
}

kvs_status kvs_pool_reposition(kvs_pool* c, const kvs_rope* rope, int layer, const int* d_kept, const int* d_n_kept,
                               const int* d_block2slot, int n_req, int keep, kvs_stream_t stream) try {
  if (!call_ok(c, layer, n_req) || !rope || rope->d.d != c->d.d || rope->d.n_axis != 1) return KVS_ERR_INVALID_ARG;
  if (keep < 1 || keep > c->d.max_ctx) return KVS_ERR_INVALID_ARG;
  if (n_req == 0) return KVS_OK;
  if (!d_kept || !d_n_kept || !d_block2slot) return KVS_ERR_INVALID_ARG;
  c->launches += 1;
  return cuda_status(launch_pool_reposition(c->d, rope->d, c->k + layer * c->layer_bytes, d_kept, d_n_kept, d_block2slot, n_req, keep,
                                            c->err, S(stream)));
} catch (...) {      // out of host memory
  return KVS_ERR_CUDA;
}

}  // extern "C"
