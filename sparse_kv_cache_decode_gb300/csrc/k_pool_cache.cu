// Device-resident pools: new tokens into their blocks, and eviction by accumulated weight.
#include <algorithm>

#include "kvs_pool.cuh"
#include "kvs_ptx.cuh"

namespace kvs {

namespace {

// ------------------------------------------------------------------ append
// One thread per 8 elements of a token's K (blockIdx.y 0) or V (1) row of one kv head: 16 bytes in,
// 16 (bf16) or 8 (E4M3, rounded to nearest even, saturating) bytes out.
constexpr int kAppendThreads = 256;

__global__ void __launch_bounds__(kAppendThreads)
    pool_append_kernel(PoolDims d, unsigned char* kpool, unsigned char* vpool, const __nv_bfloat16* __restrict__ k_new,
                       const __nv_bfloat16* __restrict__ v_new, long long stride, PoolSeqs seqs, unsigned* err) {
  kvs_pdl_entry();
  const int vecs = d.Hkv * (d.d / 8);
  const long long i = (long long)blockIdx.x * kAppendThreads + threadIdx.x;
  const int tok = (int)(i / vecs);
  if (tok >= seqs.n_tok) return;
  const int rem = (int)(i - (long long)tok * vecs), h = rem / (d.d / 8), c = rem - h * (d.d / 8);
  const int s = pool_seq_of(seqs, tok);
  if (s < 0) return;
  const SeqInfo r = pool_seq(d, seqs, s, err);
  if (tok < r.t0 || tok >= r.t1) return;
  const int pos = r.len - (r.t1 - tok);
  if (pos < 0) {   // more query tokens than the context holds
    set_error(err, KVS_ERR_BAD_INDEX);
    return;
  }
  const int slot = seqs.table[(size_t)s * d.nb_max + (pos >> d.log2bs)];
  if (slot < 0 || slot >= d.n_slots) {
    set_error(err, KVS_ERR_BAD_INDEX);
    return;
  }
  const uint4 x = *reinterpret_cast<const uint4*>((blockIdx.y ? v_new : k_new) + tok * stride + h * d.d + c * 8);
  const size_t row = ((size_t)slot * d.Hkv + h) * d.bs + (pos & (d.bs - 1));
  unsigned char* dst = (blockIdx.y ? vpool : kpool) + (row * d.d + c * 8) * d.ebytes;
  if (!d.fp8) {
    *reinterpret_cast<uint4*>(dst) = x;
    return;
  }
  const float scale = blockIdx.y ? d.v_scale : d.k_scale;
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t o[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < 4; ++j)
    o[j >> 1] |= f32x2_to_e4m3x2(__fdiv_rn(bf16_lo(w[j]), scale), __fdiv_rn(bf16_hi(w[j]), scale)) << ((j & 1) * 16);
  *reinterpret_cast<uint2*>(dst) = make_uint2(o[0], o[1]);
}

// ------------------------------------------------------------------ evict: selection
// One CTA per (request, kv head).  The k-th largest weight of the tokens between the first n_sink and the
// last n_recent is found by radix selection on the ordered keys (score_key: NaN lowest, -0 == +0), 11 bits
// a pass: eleven bits split the exponent's range fine enough that few tokens share a histogram bin.
// Each bin has four counters, by lane, as the lanes of a warp often meet in a bin.
// Each warp owns a contiguous run of tokens, so the kept indices come out in order from one count per
// warp, a scan over the warps and ballots, without a barrier per step.
// Five passes read the keys: contexts of up to kSelCached tokens are copied to shared memory first, 8 loads in flight a
// thread (reading them from L2 in each pass took 39 us at 32K tokens, latency all of it); longer ones are read 8 at a
// time from L2.
constexpr int kSelThreads = 1024;
constexpr int kSelBins = 2048;
constexpr int kSelCached = 45056;
constexpr int kSelCopies = 4;

template <bool CACHED>
__global__ void __launch_bounds__(kSelThreads)
    pool_evict_select_kernel(PoolDims d, const float* __restrict__ weight, const int* __restrict__ ctx_len, int keep,
                             int n_sink, int n_recent, int* __restrict__ kept, int* __restrict__ n_kept,
                             unsigned* err) {
  kvs_pdl_entry();
  extern __shared__ uint32_t keys[];       // [len] (CACHED)
  __shared__ __align__(16) int hist[kSelBins * kSelCopies];
  __shared__ int warp_a[32], warp_b[32];
  __shared__ int pick[2];
  const int u = blockIdx.x, r = u / d.Hkv, h = u - r * d.Hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int NW = kSelThreads / 32, UN = 8;
  int len = ctx_len[r];
  if (len < 0 || len > d.max_ctx) {
    if (tid == 0) set_error(err, KVS_ERR_BAD_INDEX);
    len = 0;
  }
  const int n = min(keep, len);
  if (h == 0 && tid == 0) n_kept[r] = n;
  int* out = kept + (size_t)u * keep;
  const float* w = weight + (size_t)u * d.max_ctx;
  if (len <= keep) {
    for (int i = tid; i < n; i += kSelThreads) out[i] = i;
    return;
  }
  if (CACHED) {
    for (int t0 = tid; t0 < len; t0 += UN * kSelThreads) {
      float v[UN];
#pragma unroll
      for (int i = 0; i < UN; ++i) v[i] = t0 + i * kSelThreads < len ? w[t0 + i * kSelThreads] : 0.f;
#pragma unroll
      for (int i = 0; i < UN; ++i)
        if (t0 + i * kSelThreads < len) keys[t0 + i * kSelThreads] = score_key(v[i]);
    }
  }
  auto key_of = [&](int t) { return CACHED ? keys[t] : score_key(__ldcg(w + t)); };
  // tokens [lo, hi) compete for k places
  const int lo = n_sink, hi = len - n_recent, k = keep - n_sink - n_recent;
  uint32_t prefix = 0;        // key bits decided so far
  int left = k;               // places left for the keys that match the prefix
  if (k > 0) {
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11, bins = 1 << bits;
      for (int i = tid; i < kSelBins; i += kSelThreads) reinterpret_cast<int4*>(hist)[i] = make_int4(0, 0, 0, 0);
      __syncthreads();
      for (int t0 = lo + tid; t0 < hi; t0 += UN * kSelThreads) {
        uint32_t key[UN];
#pragma unroll
        for (int i = 0; i < UN; ++i) key[i] = t0 + i * kSelThreads < hi ? key_of(t0 + i * kSelThreads) : 0u;
#pragma unroll
        for (int i = 0; i < UN; ++i)
          if (t0 + i * kSelThreads < hi && (pass == 0 || (key[i] >> (shift + bits)) == prefix))
            atomicAdd(&hist[((key[i] >> shift) & (bins - 1)) * kSelCopies + (lane & 3)], 1);
      }
      __syncthreads();
      // the bin of the left-th key from the top: thread i owns the two bins bins-1-2i and bins-2-2i
      int c0 = 0, c1 = 0;
      if (2 * tid < bins) {
        const int4 a = reinterpret_cast<const int4*>(hist)[bins - 1 - 2 * tid], b4 = reinterpret_cast<const int4*>(hist)[bins - 2 - 2 * tid];
        c0 = a.x + a.y + a.z + a.w;
        c1 = b4.x + b4.y + b4.z + b4.w;
      }
      int x = c0 + c1;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (lane == 31) warp_a[warp] = x;
      __syncthreads();
      int before = x - c0 - c1;
      for (int i = 0; i < warp; ++i) before += warp_a[i];
      if (before < left && left <= before + c0 + c1) {
        const int first = before + c0 >= left;
        pick[0] = first ? bins - 1 - 2 * tid : bins - 2 - 2 * tid;
        pick[1] = first ? before : before + c0;
      }
      __syncthreads();
      prefix = (prefix << bits) | (uint32_t)pick[0];
      left -= pick[1];
      __syncthreads();
    }
  } else {
    prefix = 0xffffffffu;     // no key is above it, and no place is left for its equals
    left = 0;
    __syncthreads();          // the cached keys
  }
  // `left` places go to the earliest keys equal to the threshold, the rest to every key above it
  const int per = ((len + NW - 1) / NW + 31) / 32 * 32;
  const int b = min(len, warp * per), e = min(len, b + per);
  int n_gt = 0, n_eq = 0;
  for (int t0 = b; t0 < e; t0 += 32 * UN) {
    uint32_t key[UN];
#pragma unroll
    for (int i = 0; i < UN; ++i) {
      const int t = t0 + 32 * i + lane;
      key[i] = t < e && t >= lo && t < hi ? key_of(t) : 0u;
    }
#pragma unroll
    for (int i = 0; i < UN; ++i) {
      const int t = t0 + 32 * i + lane;
      const bool in = t < e, mid = in && t >= lo && t < hi;
      n_gt += __popc(__ballot_sync(0xffffffffu, in && (!mid || key[i] > prefix)));
      n_eq += __popc(__ballot_sync(0xffffffffu, mid && key[i] == prefix));
    }
  }
  if (lane == 0) {
    warp_a[warp] = n_gt;
    warp_b[warp] = n_eq;
  }
  __syncthreads();
  int at = 0, eq = 0;         // kept before this warp's run, equals before it
  for (int i = 0; i < warp; ++i) {
    at += warp_a[i] + min(warp_b[i], max(0, left - eq));
    eq += warp_b[i];
  }
  for (int t0 = b; t0 < e; t0 += 32 * UN) {
    uint32_t key[UN];
#pragma unroll
    for (int i = 0; i < UN; ++i) {
      const int t = t0 + 32 * i + lane;
      key[i] = t < e && t >= lo && t < hi ? key_of(t) : 0u;
    }
#pragma unroll
    for (int i = 0; i < UN; ++i) {
      const int t = t0 + 32 * i + lane;
      const bool in = t < e, mid = in && t >= lo && t < hi;
      const bool same = mid && key[i] == prefix;
      const unsigned eqs = __ballot_sync(0xffffffffu, same);
      const bool take = in && (!mid || key[i] > prefix || (same && eq + __popc(eqs & ((1u << lane) - 1)) < left));
      const unsigned m = __ballot_sync(0xffffffffu, take);
      if (take) out[at + __popc(m & ((1u << lane) - 1))] = t;
      at += __popc(m);
      eq += __popc(eqs);
    }
  }
}

// ------------------------------------------------------------------ evict: gather
// One warp copies 32 / VECS kept tokens of a (request, kv head) at a time, VECS 16-byte vectors of K and V
// rows together, kGatherDeep of them in flight: first all indices, then all slots, then all rows, so that a CTA pays
// three load latencies for its tokens and not three for each.
constexpr int kGatherThreads = 256;
constexpr int kGatherDeep = 8;

template <int VECS>   // 16-byte vectors of a token's K and V rows: 2 * d * ebytes / 16
__global__ void __launch_bounds__(kGatherThreads)
    pool_evict_gather_kernel(PoolDims d, unsigned char* __restrict__ kpool, unsigned char* __restrict__ vpool,
                             const float* __restrict__ weight, const int* __restrict__ ctx_len,
                             const int* __restrict__ table, int keep, const int* __restrict__ dst,
                             const int* __restrict__ kept, float* __restrict__ weight_out, unsigned* err) {
  kvs_pdl_entry();
  constexpr int PER = 32 / VECS;                                   // tokens per warp and step
  constexpr int SPAN = kGatherThreads / 32 * PER * kGatherDeep;    // tokens per CTA
  const int u = blockIdx.y, r = u / d.Hkv, h = u - r * d.Hkv;
  const int first = blockIdx.x * SPAN;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane / VECS, vec = lane % VECS;
  const bool is_v = vec >= VECS / 2;
  const int part = vec % (VECS / 2);
  unsigned char* pool = is_v ? vpool : kpool;
  constexpr int row_bytes = VECS / 2 * 16;
  int t[kGatherDeep];
  // (entries past the kept ones are in the buffer, and not used)
#pragma unroll
  for (int j = 0; j < kGatherDeep; ++j) {
    const int i = first + (j * (kGatherThreads / 32) + warp) * PER + sub;
    t[j] = i < keep ? kept[(size_t)u * keep + i] : 0;
  }
  int len = ctx_len[r];
  if (len < 0 || len > d.max_ctx) return;                          // reported by the selection
  const int n = min(keep, len);
  if (first >= n) return;
  int from_slot[kGatherDeep], to_slot[kGatherDeep];
  float wt[kGatherDeep];
#pragma unroll
  for (int j = 0; j < kGatherDeep; ++j) {
    const int i = first + (j * (kGatherThreads / 32) + warp) * PER + sub;
    from_slot[j] = to_slot[j] = -1;
    if (i < n) {
      from_slot[j] = table[(size_t)r * d.nb_max + (t[j] >> d.log2bs)];
      to_slot[j] = dst[(size_t)r * d.nb_max + (i >> d.log2bs)];
      if (vec == 0) wt[j] = weight[(size_t)u * d.max_ctx + t[j]];
    }
  }
  uint4 x[kGatherDeep];
  bool bad = false;
#pragma unroll
  for (int j = 0; j < kGatherDeep; ++j) {
    const int i = first + (j * (kGatherThreads / 32) + warp) * PER + sub;
    const bool ok = from_slot[j] >= 0 && from_slot[j] < d.n_slots && to_slot[j] >= 0 && to_slot[j] < d.n_slots;
    bad = bad || (i < n && !ok);
    if (ok)
      x[j] = __ldcs(reinterpret_cast<const uint4*>(
          pool + (((size_t)from_slot[j] * d.Hkv + h) * d.bs + (t[j] & (d.bs - 1))) * row_bytes + part * 16));
    else
      to_slot[j] = -1;
  }
#pragma unroll
  for (int j = 0; j < kGatherDeep; ++j) {
    const int i = first + (j * (kGatherThreads / 32) + warp) * PER + sub;
    if (to_slot[j] >= 0)
      *reinterpret_cast<uint4*>(pool + (((size_t)to_slot[j] * d.Hkv + h) * d.bs + (i & (d.bs - 1))) * row_bytes + part * 16) =
          x[j];
    if (i < n && vec == 0) weight_out[(size_t)u * d.max_ctx + i] = wt[j];
  }
  if (bad) set_error(err, KVS_ERR_BAD_INDEX);
}

}  // namespace

cudaError_t launch_pool_append(const PoolDims& d, unsigned char* k, unsigned char* v, const __nv_bfloat16* k_new,
                               const __nv_bfloat16* v_new, long long stride, const PoolSeqs& q, unsigned* err,
                               cudaStream_t s) {
  const long long vecs = (long long)q.n_tok * d.Hkv * (d.d / 8);
  launch_pdl(pool_append_kernel, dim3((unsigned)((vecs + kAppendThreads - 1) / kAppendThreads), 2), dim3(kAppendThreads),
             0, s, d, k, v, k_new, v_new, stride, q, err);
  return cudaGetLastError();
}

cudaError_t launch_pool_evict(const PoolDims& d, unsigned char* k, unsigned char* v, const float* weight,
                              const int* ctx_len, const int* table, int n_req, int keep, int n_sink, int n_recent,
                              const int* dst, int* kept, int* n_kept, float* weight_out, unsigned* err,
                              cudaStream_t s) {
  if (d.max_ctx <= kSelCached) {
    const int smem = d.max_ctx * 4;
    cudaError_t e1 = set_max_dynamic_smem(reinterpret_cast<const void*>(pool_evict_select_kernel<true>), kSelCached * 4);
    if (e1 != cudaSuccess) return e1;
    launch_pdl(pool_evict_select_kernel<true>, dim3(n_req * d.Hkv), dim3(kSelThreads), smem, s, d, weight, ctx_len, keep, n_sink,
               n_recent, kept, n_kept, err);
  } else {
    launch_pdl(pool_evict_select_kernel<false>, dim3(n_req * d.Hkv), dim3(kSelThreads), 0, s, d, weight, ctx_len, keep, n_sink,
               n_recent, kept, n_kept, err);
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int vecs = 2 * d.d * d.ebytes / 16;
  const int span = kGatherThreads / 32 * (32 / vecs) * kGatherDeep;
  const dim3 grid((keep + span - 1) / span, n_req * d.Hkv);
  if (vecs == 32)
    launch_pdl(pool_evict_gather_kernel<32>, grid, dim3(kGatherThreads), 0, s, d, k, v, weight, ctx_len, table, keep, dst,
               static_cast<const int*>(kept), weight_out, err);
  else if (vecs == 16)
    launch_pdl(pool_evict_gather_kernel<16>, grid, dim3(kGatherThreads), 0, s, d, k, v, weight, ctx_len, table, keep, dst,
               static_cast<const int*>(kept), weight_out, err);
  else
    launch_pdl(pool_evict_gather_kernel<8>, grid, dim3(kGatherThreads), 0, s, d, k, v, weight, ctx_len, table, keep, dst,
               static_cast<const int*>(kept), weight_out, err);
  return cudaGetLastError();
}

}  // namespace kvs
