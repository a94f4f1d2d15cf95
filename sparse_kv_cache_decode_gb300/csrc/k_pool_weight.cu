// Device-resident pools: softmax weight that each key receives.
#include "kvs_pool.cuh"
#include "kvs_ptx.cuh"

namespace kvs {

namespace {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float pool_elem(const unsigned char* p, size_t i, int fp8) {
  return fp8 ? e4m3_to_f32(p[i]) : __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[i]);
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
