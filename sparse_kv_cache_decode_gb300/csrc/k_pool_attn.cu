// Device-resident pools: attention over paged K/V, one warp per (query token, head).
#include <algorithm>

#include "kvs_pool.cuh"
#include "kvs_ptx.cuh"

namespace kvs {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kWarps = 4;

__device__ __forceinline__ float pool_elem(const unsigned char* p, size_t i, int fp8) {
  return fp8 ? e4m3_to_f32(p[i]) : __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[i]);
}

__global__ void __launch_bounds__(kWarps * 32)
    pool_attn_kernel(PoolDims d, const unsigned char* __restrict__ kpool, const unsigned char* __restrict__ vpool,
                     const __nv_bfloat16* __restrict__ q, long long q_stride, PoolSeqs seqs, PoolAttnOut o, unsigned* err) {
  kvs_pdl_entry();
  const int lane = threadIdx.x & 31;
  const long long i = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int tok = (int)(i / d.Hq), head = (int)(i - (long long)tok * d.Hq), h = head / d.G;
  if (tok >= seqs.n_tok) return;
  const int s = pool_seq_of(seqs, tok);
  if (s < 0) return;
  const SeqInfo r = pool_seq(d, seqs, s, err);
  if (tok < r.t0 || tok >= r.t1) return;
  const int pos = seqs.causal ? r.len - (r.t1 - tok) : r.len - 1;
  const int E = d.d / 32;
  float x[4], acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int e = 0; e < E; ++e)
    x[e] = __bfloat162float(q[tok * q_stride + head * d.d + e * 32 + lane]) * (d.scale * d.k_scale * kLog2e);
  const int low = seqs.causal && seqs.window ? max(0, pos - seqs.window + 1) : 0;
  const int n_first = seqs.causal && seqs.window ? min(low, seqs.n_sink) : 0;
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j < n_first + pos + 1 - low; ++j) {
    const int t = j < n_first ? j : low + j - n_first;
    const int slot = seqs.table[(size_t)s * d.nb_max + (t >> d.log2bs)];
    if (slot < 0 || slot >= d.n_slots) {
      set_error(err, KVS_ERR_BAD_INDEX);
      continue;
    }
    const size_t row = (((size_t)slot * d.Hkv + h) * d.bs + (t & (d.bs - 1))) * d.d;
    float a = 0.f;
    for (int e = 0; e < E; ++e) a += x[e] * pool_elem(kpool, row + e * 32 + lane, d.fp8);
    for (int w = 16; w; w >>= 1) a += __shfl_xor_sync(0xffffffffu, a, w);
    const float mn = fmaxf(m, a), f = exp2f(m - mn), p = exp2f(a - mn);
    l = l * f + p;
    m = mn;
    for (int e = 0; e < E; ++e) acc[e] = acc[e] * f + p * pool_elem(vpool, row + e * 32 + lane, d.fp8);
  }
  float lse2 = l > 0.f ? m + log2f(l) : -INFINITY;
  const size_t row = (size_t)tok * d.Hq + head;
  const float inv = l > 0.f ? d.v_scale / l : 0.f;
  float w0 = 0.f, w1 = inv;
  const bool has_prev = o.prev_out && s >= o.prev_req[0] && s < o.prev_req[o.n_prev];
  if (has_prev) {
    const float a = o.prev_lse2[row], M = fmaxf(a, lse2);
    if (M != -INFINITY) {
      const float ea = exp2f(a - M), eb = exp2f(lse2 - M);
      w0 = ea / (ea + eb);
      w1 = inv * (eb / (ea + eb));
      lse2 = M + log2f(ea + eb);
    }
  }
  for (int e = 0; e < E; ++e) {
    float y = acc[e] * w1;
    if (has_prev) y += w0 * o.prev_out[row * d.d + e * 32 + lane];
    if (o.out) o.out[row * d.d + e * 32 + lane] = __float2bfloat16(y);
    if (o.part_out) o.part_out[row * d.d + e * 32 + lane] = y;
  }
  if (lane == 0) {
    if (o.lse) o.lse[row] = lse2 * kLn2;
    if (o.lse2) o.lse2[row] = lse2;
  }
}

// One thread per key: its K row in registers, the request's query rows one after the other.
constexpr int kKeys = 128;

template <int D>
__global__ void __launch_bounds__(kKeys)
    pool_weight_kernel(PoolDims d, const unsigned char* __restrict__ kpool, const __nv_bfloat16* __restrict__ q,
                       long long q_stride, PoolSeqs seqs, const float* __restrict__ lse2, float* __restrict__ weight,
                       unsigned* err) {
  kvs_pdl_entry();
  const int u = blockIdx.y, s = u / d.Hkv, h = u - s * d.Hkv;
  const SeqInfo r = pool_seq(d, seqs, s, err);
  const int t = blockIdx.x * kKeys + threadIdx.x;
  if (t >= r.len) return;
  const int slot = seqs.table[(size_t)s * d.nb_max + (t >> d.log2bs)];
  float k[D];
  const bool ok = slot >= 0 && slot < d.n_slots;
  if (ok) {
    const size_t row = (((size_t)slot * d.Hkv + h) * d.bs + (t & (d.bs - 1))) * D;
#pragma unroll
    for (int e = 0; e < D; ++e) k[e] = pool_elem(kpool, row + e, d.fp8);
  }
  float sum = 0.f;
  const int p0 = r.len - (r.t1 - r.t0);
  for (int tok = r.t0 + max(0, t - p0); ok && tok < r.t1; ++tok) {
    const int pos = p0 + tok - r.t0;
    if (seqs.window && pos - t >= seqs.window && t >= seqs.n_sink) continue;
    float part = 0.f;
    for (int g = 0; g < d.G; ++g) {
      const __nv_bfloat16* x = q + tok * q_stride + (h * d.G + g) * D;
      float a = 0.f;
#pragma unroll
      for (int e = 0; e < D; ++e) a += k[e] * __bfloat162float(x[e]);
      part += exp2f(a * (d.scale * d.k_scale * kLog2e) - lse2[(size_t)tok * d.Hq + h * d.G + g]);
    }
    sum += part;
  }
  float* w = weight + (size_t)u * d.max_ctx + t;
  *w = t >= p0 ? sum : *w + sum;
}

}  // namespace

size_t pool_attn_scratch_bytes(const PoolDims&) { return 256; }

cudaError_t launch_pool_attn(const PoolDims& d, const unsigned char* k, const unsigned char* v, const CUtensorMap*,
                             const __nv_bfloat16* q, long long q_stride, const PoolSeqs& seqs, const PoolAttnOut& o,
                             void*, unsigned* err, cudaStream_t s, int* n_launched) {
  const long long rows = (long long)seqs.n_tok * d.Hq;
  *n_launched = 1;
  launch_pdl(pool_attn_kernel, dim3((unsigned)((rows + kWarps - 1) / kWarps)), dim3(kWarps * 32), 0, s, d, k, v, q, q_stride,
             seqs, o, err);
  return cudaGetLastError();
}

cudaError_t launch_pool_weight(const PoolDims& d, const unsigned char* k, const CUtensorMap*, const __nv_bfloat16* q,
                               long long q_stride, const PoolSeqs& seqs, const float* lse2, float* weight,
                               unsigned* err, cudaStream_t s) {
  const dim3 grid((d.max_ctx + kKeys - 1) / kKeys, seqs.n_seq * d.Hkv);
  if (d.d == 128)
    launch_pdl(pool_weight_kernel<128>, grid, dim3(kKeys), 0, s, d, k, q, q_stride, seqs, lse2, weight, err);
  else
    launch_pdl(pool_weight_kernel<64>, grid, dim3(kKeys), 0, s, d, k, q, q_stride, seqs, lse2, weight, err);
  return cudaGetLastError();
}

}  // namespace kvs
