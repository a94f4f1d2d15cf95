// Block tables of a batch from its lengths, and where the tokens of a call go.
//
// Each CTA reads the requests' lengths and counts the blocks that every request needs more or has too many of, and scans
// both counts (at most 2048 requests: a copy of the scan per CTA costs less than a second launch or a wait between CTAs).
// A block taken or given back, and a token, is then found among the requests by a binary search in shared memory, so that
// any spread of lengths is shared evenly by all threads.
//
// Nothing that a CTA reads is written by another: blocks come off the ring's front and go behind its end, tables of growing
// requests are written past what they hold, tables of shrinking ones are only read, and the blocks that are given back and
// taken in the same call are handed over by the thread that gives them.  The lengths held and the ring's state are written
// by the CTA that is the last to have read them.
#include <algorithm>

#include "kvs_rope.cuh"

namespace kvs {

namespace {

constexpr int kTabThreads = 512;
constexpr unsigned kTabMany = 1u << 30;      // sums stop here (no pool has as many slots)

__device__ __forceinline__ unsigned add_sat(unsigned a, unsigned b) { return min(a + b, kTabMany); }

// The last of x[0 .. n] (ascending, x[0] <= v) that is <= v.
__device__ __forceinline__ int last_at(const int* x, int n, int v) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (x[mid] <= v) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kTabThreads)
    pool_tables_kernel(PoolDims d, PoolTables t, unsigned* ticket, unsigned* err) {
  extern __shared__ int dyn[];
  const int n = t.n_req;
  int* cu = dyn;                 // [n + 1]
  int* ctx = cu + n + 1;         // [n]
  int* held = ctx + n;           // [n] blocks ahead of the call
  int* need = held + n;          // [n] and after it
  int* takes = need + n;         // [n + 1] blocks taken by the requests before
  int* gives = takes + n + 1;    // [n + 1]
  __shared__ unsigned warp_take[kTabThreads / 32], warp_give[kTabThreads / 32];
  __shared__ int is_last;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  kvs_pdl_entry();
  const bool alloc = t.ring != nullptr;
  int head = 0, n_free = 0;
  if (alloc) {
    head = t.state[0];
    n_free = t.state[1];
  }
  bool bad = false;
  // each thread counts a run of requests
  const int per = (n + kTabThreads - 1) / kTabThreads, r0 = min(n, tid * per), r1 = min(n, r0 + per);
  unsigned take = 0, give = 0;
  for (int r = r0; r < r1; ++r) {
    int len = t.ctx_len[r];
    const bool ok_len = len >= 0 && len <= d.max_ctx;
    const int blocks = ok_len ? (len + d.bs - 1) >> d.log2bs : 0;
    int had = alloc ? t.n_held[r] : blocks;
    const bool ok = ok_len && had >= 0 && had <= d.nb_max;
    bad |= !ok;
    if (!ok) had = 0;
    const int want = ok ? blocks : 0;
    ctx[r] = ok ? len : -1;
    held[r] = had;
    need[r] = want;
    take = add_sat(take, max(0, want - had));
    give = add_sat(give, max(0, had - want));
  }
  if (t.cu_q)
    for (int r = tid; r <= n; r += kTabThreads) cu[r] = t.cu_q[r];
  unsigned in_take = take, in_give = give;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned a = __shfl_up_sync(0xffffffffu, in_take, o), b = __shfl_up_sync(0xffffffffu, in_give, o);
    if (lane >= o) {
      in_take = add_sat(in_take, a);
      in_give = add_sat(in_give, b);
    }
  }
  if (lane == 31) {
    warp_take[warp] = in_take;
    warp_give[warp] = in_give;
  }
  __syncthreads();
  unsigned before_take = 0, before_give = 0, all_take = 0, all_give = 0;
#pragma unroll
  for (int w = 0; w < kTabThreads / 32; ++w) {
    if (w == warp) {
      before_take = all_take;
      before_give = all_give;
    }
    all_take = add_sat(all_take, warp_take[w]);
    all_give = add_sat(all_give, warp_give[w]);
  }
  // (sums that stopped are never used: such calls change nothing)
  before_take = add_sat(before_take, in_take - take);
  before_give = add_sat(before_give, in_give - give);
  for (int r = r0; r < r1; ++r) {
    takes[r] = (int)before_take;
    gives[r] = (int)before_give;
    bad |= t.cu_q && (cu[r] < 0 || cu[r] > cu[r + 1] || cu[r + 1] > t.n_tok);
    before_take = add_sat(before_take, max(0, need[r] - held[r]));
    before_give = add_sat(before_give, max(0, held[r] - need[r]));
  }
  if (tid == 0) {
    takes[n] = (int)all_take;
    gives[n] = (int)all_give;
  }
  // every read of n_held and state by this CTA is through
  __syncthreads();
  const bool ok_state = !alloc || (head >= 0 && head < d.n_slots && n_free >= 0 && n_free <= d.n_slots &&
                                   all_give <= (unsigned)(d.n_slots - n_free));
  const unsigned have = (unsigned)n_free + all_give;
  const bool lacking = ok_state && all_take > have;
  const bool change = alloc && ok_state && !lacking;
  bad |= !ok_state;
  if (bad) set_error(err, KVS_ERR_BAD_INDEX);
  if (alloc) {
    if (tid == 0) {
      is_last = 1;
      if (gridDim.x > 1) {
        __threadfence();
        is_last = atomicAdd(ticket, 1u) == gridDim.x - 1;
        __threadfence();
        if (is_last) *ticket = 0;
      }
    }
    __syncthreads();
    if (is_last) {
      if (tid == 0 && ok_state) {
        t.state[2] = lacking ? (int)(all_take - have) : 0;
        if (change) {
          const int at = head + (int)all_take;        // all_take <= have <= n_slots
          t.state[0] = at < d.n_slots ? at : at - d.n_slots;
          t.state[1] = (int)(have - all_take);
        }
        if (lacking) set_error(err, KVS_ERR_CAPACITY);
      }
      if (change)
        for (int r = tid; r < n; r += kTabThreads)
          if (ctx[r] >= 0) t.n_held[r] = need[r];
    }
  }
  const int stride = gridDim.x * kTabThreads, first = blockIdx.x * kTabThreads + tid;
  auto ring_at = [&](int i) {      // i-th entry from the front, i < 2 n_slots - head
    const int at = head + i;
    return t.ring + (at < d.n_slots ? at : at - d.n_slots);
  };
  if (change) {
    const int taken = (int)min(all_take, (unsigned)n_free);
    for (int i = first; i < taken; i += stride) {
      const int r = last_at(takes, n, i);
      t.table[(size_t)r * d.nb_max + held[r] + (i - takes[r])] = *ring_at(i);
    }
    for (int j = first; j < (int)all_give; j += stride) {
      const int r = last_at(gives, n, j);
      const int slot = t.table[(size_t)r * d.nb_max + need[r] + (j - gives[r])];
      *ring_at(n_free + j) = slot;
      const int i = n_free + j;
      if (i < (int)all_take) {
        const int to = last_at(takes, n, i);
        t.table[(size_t)to * d.nb_max + held[to] + (i - takes[to])] = slot;
      }
    }
  }
  if (!t.cu_q) return;
  for (int tok = first; tok < t.n_tok; tok += stride) {
    long long place = -1;
    int pos = 0;
    const int r = last_at(cu, n, tok);
    const int a = cu[r], b = cu[r + 1];
    // (offsets that cannot be, and requests of a bad length, are reported above: their tokens have no place)
    if (a >= 0 && b <= t.n_tok && tok >= a && tok < b && ctx[r] >= 0) {
      const int p = ctx[r] - (b - tok);
      pos = (int)((unsigned)p + (unsigned)(t.pos_delta ? t.pos_delta[r] : 0));
      if (p >= 0) {
        const int block = p >> d.log2bs;
        int slot = -1;
        bool known = true;
        if (block < held[r]) {
          slot = t.table[(size_t)r * d.nb_max + block];
        } else if (change) {
          const int i = takes[r] + (block - held[r]);
          if (i < n_free) {
            slot = *ring_at(i);
          } else {
            const int from = last_at(gives, n, i - n_free);
            slot = t.table[(size_t)from * d.nb_max + need[from] + (i - n_free - gives[from])];
          }
        } else {
          known = false;      // the block was lacking
        }
        if (slot >= 0 && slot < d.n_slots) place = ((long long)slot << d.log2bs) + (p & (d.bs - 1));
        else if (known) set_error(err, KVS_ERR_BAD_INDEX);
      }
    }
    t.place[tok] = place;
    if (t.pos) t.pos[tok] = pos;
  }
}

}  // namespace

cudaError_t launch_pool_tables(const PoolDims& d, const PoolTables& t, unsigned* ticket, unsigned* err, cudaStream_t s) {
  const long long blocks = t.ring ? (long long)t.n_req * d.nb_max : 0;
  const long long work = std::max<long long>(t.n_tok, blocks / 16);
  const int grid = (int)std::max(1ll, std::min<long long>((work + kTabThreads - 1) / kTabThreads, device_sm_count()));
  const int smem = (6 * t.n_req + 3) * 4;
  cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void*>(pool_tables_kernel), (6 * kPoolMaxReq + 3) * 4);
  if (e != cudaSuccess) return e;
  launch_pdl(pool_tables_kernel, dim3(grid), dim3(kTabThreads), (size_t)smem, s, d, t, ticket, err);
  return cudaGetLastError();
}

}  // namespace kvs
