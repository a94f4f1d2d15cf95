// Declarations of the rotation of query and key rows shared by its translation units (not part of the C ABI).
#pragma once
#include "kvs_pool.cuh"

namespace kvs {

constexpr int kRopeMaxPairs = 128;
constexpr int kRopeMaxAxes = 8;

// What a kvs_rope holds, for rows of up to PAIRS pairs.
template <int PAIRS>
struct RopeParams {
  int d, rot, n_axis, adjacent;
  float rot_scale, eps;
  unsigned long long freq[PAIRS];   // turns per position, mod 1, in units of 2^-64
  unsigned char axis[PAIRS];
};
using RopeDims = RopeParams<kRopeMaxPairs>;

// Heads of all tokens, in and out, strides in elements.
struct RopeHeads {
  const __nv_bfloat16* src;
  __nv_bfloat16* dst;
  long long src_tok, src_head, dst_tok, dst_head;
  const float* norm;    // [d] or nullptr: no norm
  int n;                // heads
};

// One call over n_tok tokens.  With kpool K and V rows go to their places in the pool instead of k.dst.
struct RopeRows {
  RopeHeads q, k, v;
  const int* pos;               // [n_axis] rows of [n_tok], pos_stride apart
  long long pos_stride;
  const long long* place;       // [n_tok] (pool only)
  unsigned char *kpool, *vpool;
  int n_slots, bs, log2bs, fp8;
  float k_scale, v_scale;
  float k_rcp, v_rcp;           // 1 / scale, rounded; 0 where scale is beyond 2^+-60
  unsigned* err;
  int n_tok;
};

cudaError_t launch_rope_rows(const RopeDims& rd, const RopeRows& a, cudaStream_t s);
cudaError_t launch_pool_reposition(const PoolDims& d, const RopeDims& rd, unsigned char* k, const int* kept, const int* n_kept,
                                   const int* table, int n_req, int keep, unsigned* err, cudaStream_t s);

// Block tables from lengths (ring != nullptr: blocks are taken and given back), and where the call's tokens go.
struct PoolTables {
  const int* ctx_len;     // [n_req]
  int* n_held;            // [n_req] (ring only)
  int* table;             // [n_req][nb_max]
  int* ring;              // [n_slots] or nullptr
  int* state;             // [3]: first entry, free slots, blocks that were lacking
  const int* cu_q;        // [n_req + 1] or nullptr: no tokens
  const int* pos_delta;   // [n_req] or nullptr
  long long* place;       // [n_tok]
  int* pos;               // [n_tok] or nullptr
  int n_req, n_tok;
};
cudaError_t launch_pool_tables(const PoolDims& d, const PoolTables& t, unsigned* ticket, unsigned* err, cudaStream_t s);

}  // namespace kvs

// The opaque handle of the C ABI (host memory only).
struct kvs_rope {
  kvs::RopeDims d;
};
