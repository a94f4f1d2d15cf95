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
  if (pos < 0) return;   // a free place of the batch, or more query tokens than the context holds: no place, as no keys in attention
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
// A cluster of CTAs per (request, kv head), a contiguous run of its tokens each.  The k-th largest weight of the tokens
// between the first n_sink and the last n_recent is found by radix selection on the ordered keys (score_key: NaN lowest,
// -0 == +0), 11 bits a pass: eleven bits split the exponent's range fine enough that few tokens share a histogram bin.
// Each bin has four counters, by lane, as the lanes of a warp often meet in a bin; a CTA's sums of them are read by the
// whole cluster, every CTA of which finds the bin of the threshold by itself.
// Each warp owns a contiguous run of its CTA's tokens, so the kept indices come out in order from one count per
// warp, scans over the warps and the CTAs and ballots, without a barrier per step.
// Five passes read the keys: runs of up to kSelCached tokens are copied to shared memory first, 8 loads in flight a
// thread (reading them from L2 in each pass took 39 us at 32K tokens, latency all of it); longer ones are read 8 at a
// time from L2.  The selection of 2048 of 32K tokens (64 units) takes
// 19 us (28 with one CTA a unit), bound by the latencies of its passes.
constexpr int kSelThreads = 1024;
constexpr int kSelBins = 2048;
constexpr int kSelCached = 40960;
constexpr int kSelCopies = 4;
constexpr int kSelRun = 4096;       // tokens a CTA should have at least
constexpr int kSelCluster = 8;

// sum of the warp's earlier lanes' x, and of all
__device__ __forceinline__ int warp_scan(int x, int lane, int* total) {
  int y = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int z = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) y += z;
  }
  *total = __shfl_sync(0xffffffffu, y, 31);
  return y - x;
}

__device__ __forceinline__ int ld_cluster(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ int2 ld_cluster2(uint32_t addr) {
  int2 v;
  asm volatile("ld.shared::cluster.v2.s32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}

template <bool CACHED, int CS>      // CS: CTAs of a cluster
__global__ void __launch_bounds__(kSelThreads)
    pool_evict_select_kernel(PoolDims d, const float* __restrict__ weight, const int* __restrict__ ctx_len, int keep,
                             int n_sink, int n_recent, int* __restrict__ kept, int* __restrict__ n_kept,
                             unsigned* err) {
  kvs_pdl_entry();
  extern __shared__ __align__(16) uint32_t dyn[];
  int* sums = reinterpret_cast<int*>(dyn);      // [3][kSelBins] by pass, so that none is written while others read it
  uint32_t* keys = dyn + 3 * kSelBins;          // [the CTA's run] (CACHED)
  __shared__ int groups[3 * 32];                // sums of 64 bins, by pass
  __shared__ __align__(16) int hist[kSelBins * kSelCopies];
  __shared__ int warp_a[32], warp_b[32];
  __shared__ __align__(8) int both[2];
  __shared__ int pick[2];
  const int rank = CS > 1 ? (int)cluster_ctarank() : 0;
  const int u = blockIdx.x / CS, r = u / d.Hkv, h = u - r * d.Hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int NW = kSelThreads / 32, UN = 8;
  auto sync_all = [&]() {
    if (CS > 1) cluster_sync();
    else __syncthreads();
  };
  int len = ctx_len[r];
  if (len < 0 || len > d.max_ctx) {
    if (tid == 0) set_error(err, KVS_ERR_BAD_INDEX);
    len = 0;
  }
  const int n = min(keep, len);
  if (h == 0 && rank == 0 && tid == 0) n_kept[r] = n;
  int* out = kept + (size_t)u * keep;
  const float* w = weight + (size_t)u * d.max_ctx;
  if (len <= keep) {        // the whole cluster
    for (int i = rank * kSelThreads + tid; i < n; i += CS * kSelThreads) out[i] = i;
    return;
  }
  // the CTA's run [r0, r1)
  const int run = ((len + CS - 1) / CS + 31) / 32 * 32;
  const int r0 = min(len, rank * run), r1 = min(len, r0 + run);
  if (CACHED) {
    for (int t0 = r0 + tid; t0 < r1; t0 += UN * kSelThreads) {
      float v[UN];
#pragma unroll
      for (int i = 0; i < UN; ++i) v[i] = t0 + i * kSelThreads < r1 ? w[t0 + i * kSelThreads] : 0.f;
#pragma unroll
      for (int i = 0; i < UN; ++i)
        if (t0 + i * kSelThreads < r1) keys[t0 - r0 + i * kSelThreads] = score_key(v[i]);
    }
  }
  auto key_of = [&](int t) { return CACHED ? keys[t - r0] : score_key(__ldcg(w + t)); };
  // tokens [lo, hi) compete for k places; of them this CTA has [c0, c1)
  const int lo = n_sink, hi = len - n_recent, k = keep - n_sink - n_recent;
  const int c0 = max(lo, r0), c1 = min(hi, r1);
  uint32_t prefix = 0;        // key bits decided so far
  int left = k;               // places left for the keys that match the prefix
  if (k > 0) {
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11, bins = 1 << bits;
      for (int i = tid; i < kSelBins; i += kSelThreads) reinterpret_cast<int4*>(hist)[i] = make_int4(0, 0, 0, 0);
      __syncthreads();
      for (int t0 = c0 + tid; t0 < c1; t0 += UN * kSelThreads) {
        uint32_t key[UN];
#pragma unroll
        for (int i = 0; i < UN; ++i) key[i] = t0 + i * kSelThreads < c1 ? key_of(t0 + i * kSelThreads) : 0u;
#pragma unroll
        for (int i = 0; i < UN; ++i)
          if (t0 + i * kSelThreads < c1 && (pass == 0 || (key[i] >> (shift + bits)) == prefix))
            atomicAdd(&hist[((key[i] >> shift) & (bins - 1)) * kSelCopies + (lane & 3)], 1);
      }
      __syncthreads();
      // the bin of the left-th key from the top.  Thread i sums the two bins b0 = bins-2-2i and b0 + 1, warp w the 64 from
      // the 64w-th on; every warp learns all CTAs' sums of 64, and the one that holds the key finds the bin (all warps
      // reading all CTAs' bins took 3500 clocks a pass).
      int* in_warps = groups + pass * 32;
      const int b0 = bins - 2 - 2 * tid;
      int lo_n = 0, hi_n = 0;
      if (b0 >= 0) {
        const int4 a = reinterpret_cast<const int4*>(hist)[b0 + 1], b4 = reinterpret_cast<const int4*>(hist)[b0];
        lo_n = b4.x + b4.y + b4.z + b4.w;
        hi_n = a.x + a.y + a.z + a.w;
        if (CS > 1) *reinterpret_cast<int2*>(&sums[pass * kSelBins + b0]) = make_int2(lo_n, hi_n);
      }
      const int in_warp = __reduce_add_sync(0xffffffffu, lo_n + hi_n);
      if (lane == 0) in_warps[warp] = in_warp;
      __syncwarp();
      sync_all();
      int sum = in_warps[lane], all;
#pragma unroll
      for (int i = 1; i < CS; ++i) sum += ld_cluster(mapa_shared(smem_u32(&in_warps[lane]), (uint32_t)(rank + i) % CS));
      const int upto = warp_scan(sum, lane, &all);
      const int rest = left - __shfl_sync(0xffffffffu, upto, warp);      // the key's number from this warp's bins on
      if (rest > 0 && rest <= __shfl_sync(0xffffffffu, sum, warp)) {
#pragma unroll
        for (int i = 1; i < CS; ++i) {
          const int2 y = ld_cluster2(mapa_shared(smem_u32(&sums[pass * kSelBins + b0]), (uint32_t)(rank + i) % CS));
          lo_n += y.x;
          hi_n += y.y;
        }
        const int before = warp_scan(lo_n + hi_n, lane, &all);
        if (before < rest && rest <= before + lo_n + hi_n) {
          const bool first = before + hi_n >= rest;
          pick[0] = first ? b0 + 1 : b0;
          pick[1] = left - rest + (first ? before : before + hi_n);
        }
      }
      __syncthreads();
      prefix = (prefix << bits) | (uint32_t)pick[0];
      left -= pick[1];
    }
  } else {
    prefix = 0xffffffffu;     // no key is above it, and no place is left for its equals
    left = 0;
    __syncthreads();          // the cached keys
  }
  // `left` places go to the earliest keys equal to the threshold, the rest to every key above it
  const int per = ((r1 - r0 + NW - 1) / NW + 31) / 32 * 32;
  const int b = min(r1, r0 + warp * per), e = min(r1, b + per);
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
      n_gt += in && (!mid || key[i] > prefix);
      n_eq += mid && key[i] == prefix;
    }
  }
  n_gt = __reduce_add_sync(0xffffffffu, n_gt);
  n_eq = __reduce_add_sync(0xffffffffu, n_eq);
  if (lane == 0) {
    warp_a[warp] = n_gt;
    warp_b[warp] = n_eq;
  }
  __syncthreads();
  // keys above the threshold and equal to it before this warp's run
  int all_gt, all_eq;
  int at = warp_scan(warp_a[lane], lane, &all_gt), eq = warp_scan(warp_b[lane], lane, &all_eq);
  at = __shfl_sync(0xffffffffu, at, warp);
  eq = __shfl_sync(0xffffffffu, eq, warp);
  if (CS > 1) {
    if (tid == 0) {
      both[0] = all_gt;
      both[1] = all_eq;
    }
    __syncwarp();
    cluster_sync();
    for (int i = 0; i < rank; ++i) {
      const int2 v = ld_cluster2(mapa_shared(smem_u32(both), (uint32_t)i));
      at += v.x;
      eq += v.y;
    }
  }
  at += min(eq, left);        // the equals that were taken
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
  __syncwarp();
  if (CS > 1) cluster_sync();       // no CTA leaves while others read its shared memory
}

// ------------------------------------------------------------------ evict: gather
// One warp copies 32 / VECS kept tokens of a (request, kv head) at a time, VECS 16-byte vectors of K and V
// rows together, kGatherDeep of them in flight: first the indices, then the slots, then the rows.  Bound by the rows'
// bytes and by those three latencies, which small CTAs, many to an SM and each in another phase, hide best: the call took
// 36.8 us for 64 units of 2048 rows of 2 x 256 bytes with CTAs of 8 warps and 8 tokens in flight each, 34.2 with 2 tokens,
// 30.7 with 4 warps and 2 tokens, 42 with 2 warps or 1 token.  The rows are written as streams (8 us less in all).
constexpr int kGatherThreads = 128;
constexpr int kGatherDeep = 2;

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
      __stcs(reinterpret_cast<uint4*>(pool + (((size_t)to_slot[j] * d.Hkv + h) * d.bs + (i & (d.bs - 1))) * row_bytes + part * 16),
             x[j]);
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
  // CTAs per (request, kv head): as many as keep their runs long and have an SM each (two to an SM, the call took 48.6 us
  // at 64 runs of 32K tokens, against 45.1)
  const int units = n_req * d.Hkv;
  int cs = 1;
  while (cs < kSelCluster && d.max_ctx / (2 * cs) >= kSelRun && units * 2 * cs <= device_sm_count()) cs *= 2;
  const int run = ((d.max_ctx + cs - 1) / cs + 31) / 32 * 32, sums = 3 * kSelBins * 4;
  const bool cached = run <= kSelCached;
  const int smem = sums + (cached ? run * 4 : 0);
  auto select = [&](auto kernel) {
    cudaError_t e1 = set_max_dynamic_smem(reinterpret_cast<const void*>(kernel), sums + (cached ? kSelCached * 4 : 0));
    if (e1 != cudaSuccess) return e1;
    if (cs > 1)
      launch_pdl_cluster(kernel, dim3(units * cs), dim3(kSelThreads), smem, s, (unsigned)cs, d, weight, ctx_len, keep, n_sink,
                         n_recent, kept, n_kept, err);
    else
      launch_pdl(kernel, dim3(units), dim3(kSelThreads), smem, s, d, weight, ctx_len, keep, n_sink, n_recent, kept, n_kept, err);
    return cudaGetLastError();
  };
  cudaError_t e = cs == 1   ? cached ? select(pool_evict_select_kernel<true, 1>) : select(pool_evict_select_kernel<false, 1>)
                  : cs == 2 ? cached ? select(pool_evict_select_kernel<true, 2>) : select(pool_evict_select_kernel<false, 2>)
                  : cs == 4 ? cached ? select(pool_evict_select_kernel<true, 4>) : select(pool_evict_select_kernel<false, 4>)
                  : cached  ? select(pool_evict_select_kernel<true, 8>) : select(pool_evict_select_kernel<false, 8>);
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
