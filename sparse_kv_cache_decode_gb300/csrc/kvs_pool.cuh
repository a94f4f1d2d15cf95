// Declarations shared by the device-resident pool's translation units (not part of the C ABI).
#pragma once
#include "kvs_common.cuh"

namespace kvs {

constexpr int kPoolMaxReq = 2048;   // requests (or prefixes) per call

// Shape of one pool, as the kernels see it (passed by value).
struct PoolDims {
  int NL, n_slots;
  int Hq, Hkv, G, d, bs, log2bs;
  int rt;                 // rows of a row tile: the heads of 128 / G whole query tokens
  unsigned g_magic;       // ceil(2^32 / G), for division by G (G > 1)
  int max_ctx, nb_max, max_req, max_tokens, max_prefix_tokens;
  int fp8, ebytes;
  float scale;            // softmax scale
  float k_scale, v_scale; // of E4M3 codes (1 for bf16)
  unsigned timeout_us;
};

// The sequences of one attention call: sequence s has the query tokens [t0, t1) and `len` cached tokens
// reached through its row of `table`.  With seq_req the sequences are groups of requests (a shared
// prefix and the requests behind it), and their tokens are those of requests [seq_req[s], seq_req[s + 1]).
struct PoolSeqs {
  const int* cu_q;      // [n_req + 1]
  const int* seq_req;   // [n_seq + 1] or nullptr
  const int* len;       // [n_seq]
  const int* table;     // [n_seq][nb_max]
  int n_seq, n_req, n_tok;
  int causal;           // 0: every row sees every key of the sequence
  int window, n_sink;   // causal: p - t < window (0: no limit) or t < n_sink
};

struct SeqInfo {
  int t0, t1, len;
};

// Sequence s, checked: an invalid entry is reported and gives an empty sequence.
__device__ __forceinline__ SeqInfo pool_seq(const PoolDims& d, const PoolSeqs& q, int s, unsigned* err) {
  SeqInfo r;
  int a = s, b = s + 1;
  bool ok = true;
  if (q.seq_req) {
    a = q.seq_req[s];
    b = q.seq_req[s + 1];
    ok = a >= 0 && a <= b && b <= q.n_req;
  }
  r.t0 = r.t1 = r.len = 0;
  if (ok) {
    r.t0 = q.cu_q[a];
    r.t1 = q.cu_q[b];
    r.len = q.len[s];
    ok = r.t0 >= 0 && r.t0 <= r.t1 && r.t1 <= q.n_tok && r.len >= 0 && r.len <= d.max_ctx;
  }
  if (!ok) {
    set_error(err, KVS_ERR_BAD_INDEX);
    r.t0 = r.t1 = r.len = 0;
  }
  return r;
}

// The last sequence that starts at or before token `tok` (offsets ascending), or -1.
__device__ __forceinline__ int pool_seq_of(const PoolSeqs& q, int tok) {
  int lo = -1, hi = q.n_seq;   // start(lo) <= tok < start(hi)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    int a = q.seq_req ? q.seq_req[mid] : mid;
    a = min(max(a, 0), q.n_req);
    if (q.cu_q[a] <= tok) lo = mid; else hi = mid;
  }
  return lo;
}

cudaError_t launch_pool_append(const PoolDims& d, unsigned char* k, unsigned char* v, const __nv_bfloat16* k_new,
                               const __nv_bfloat16* v_new, long long stride, const PoolSeqs& q, unsigned* err,
                               cudaStream_t s);
// Attention of the sequences' rows.  Exactly one of out (bf16) and part_out (fp32, with part_lse) is
// written; with prev_out / prev_lse (fp32 rows and log2-sum-exps of an earlier call over other keys, for
// the tokens of requests [prev_req[0], prev_req[n_prev])) the result joins both.  lse: natural log, may be nullptr.
struct PoolAttnOut {
  __nv_bfloat16* out;
  float* lse;         // [n_tok][Hq] natural log, or nullptr
  float* lse2;        // [n_tok][Hq] base-2 log, or nullptr
  float* part_out;    // [n_tok][Hq][d]
  const float* prev_out;
  const float* prev_lse2;
  const int* prev_req;  // prefix_req; its first and last entries bound the requests that have one
  int n_prev;
};
// The query rows as [tokens][heads][dims]; a box holds 64 dims of the group's G heads of 128 / G tokens.
bool make_pool_q_map(CUtensorMap* m, const PoolDims& d, const __nv_bfloat16* q, long long q_stride, int n_tok);
size_t pool_attn_scratch_bytes(const PoolDims& d);
cudaError_t launch_pool_attn(const PoolDims& d, const unsigned char* k, const unsigned char* v, const CUtensorMap* tm,
                             const __nv_bfloat16* q, long long q_stride, const PoolSeqs& seqs, const PoolAttnOut& o,
                             void* scratch, unsigned* err, cudaStream_t s, int* n_launched);
// The kernel for few rows per (sequence, kv head): row blocks of nb rows (up to 32).
cudaError_t launch_pool_decode(const PoolDims& d, const CUtensorMap* tm, const __nv_bfloat16* q, long long q_stride,
                               const PoolSeqs& seqs, const PoolAttnOut& o, int nb, void* scratch, unsigned* err,
                               cudaStream_t s, int* n_launched);
size_t pool_weight_scratch_bytes();
cudaError_t launch_pool_weight(const PoolDims& d, const CUtensorMap* tm, const __nv_bfloat16* q, long long q_stride,
                               const PoolSeqs& seqs, const float* lse2, float* weight, void* scratch, unsigned* err,
                               cudaStream_t s, int* n_launched);
cudaError_t launch_pool_evict(const PoolDims& d, unsigned char* k, unsigned char* v, const float* weight,
                              const int* ctx_len, const int* table, int n_req, int keep, int n_sink, int n_recent,
                              const int* dst, int* kept, int* n_kept, float* weight_out, unsigned* err, cudaStream_t s);

}  // namespace kvs
