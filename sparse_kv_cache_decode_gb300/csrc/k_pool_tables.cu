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
//
// Bound by latencies: the launch, one read of the lengths, the scan, a table entry, 3.0 us of which the launch is half (64 requests, a
// token each).  24 prompts of 494000 tokens in all: 6 us, four consecutive tokens a thread (6 MB of places and positions,
// 0.9 us at the rate of a copy); the blocks and the tokens in a launch each took 4 us more.
#include <algorithm>

#include "kvs_rope.cuh"

namespace kvs {

namespace {

constexpr int kTabThreads = 256;
constexpr int kTabDeep = 4;                  // moves of a thread on their way at once
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

template <int PER>      // consecutive tokens a thread places at a time
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
  int* delta = gives + n + 1;    // [n]
  __shared__ unsigned warp_take[kTabThreads / 32], warp_give[kTabThreads / 32];
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
  for (int r = r0; r < r1; r += 2) {      // (two requests' loads at once)
    int len[2], had[2], by[2];
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (r + k < r1) {
        len[k] = __ldg(t.ctx_len + r + k);
        had[k] = alloc ? t.n_held[r + k] : 0;
        by[k] = t.pos_delta ? __ldg(t.pos_delta + r + k) : 0;
      }
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (r + k < r1) {
        const bool ok_len = len[k] >= 0 && len[k] <= d.max_ctx;
        const int blocks = ok_len ? (len[k] + d.bs - 1) >> d.log2bs : 0;
        if (!alloc) had[k] = blocks;
        const bool ok = ok_len && had[k] >= 0 && had[k] <= d.nb_max;
        bad |= !ok;
        if (!ok) had[k] = 0;
        const int want = ok ? blocks : 0;
        ctx[r + k] = ok ? len[k] : -1;
        held[r + k] = had[k];
        need[r + k] = want;
        delta[r + k] = by[k];
        take = add_sat(take, max(0, want - had[k]));
        give = add_sat(give, max(0, had[k] - want));
      }
  }
  if (t.cu_q)
    for (int r = tid; r <= n; r += kTabThreads) cu[r] = __ldg(t.cu_q + r);
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
  const int busy = per ? (n + 32 * per - 1) / (32 * per) : 0;      // warps with requests
  for (int w = 0; w < busy; ++w) {
    if (w == warp) {
      before_take = all_take;
      before_give = all_give;
    }
    all_take = add_sat(all_take, warp_take[w]);
    all_give = add_sat(all_give, warp_give[w]);
  }
  // (sums that stopped are never used, nor those of warps without requests)
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
  if (alloc && warp == kTabThreads / 32 - 1) {      // (the warp that has the least of the rest to do)
    unsigned before = gridDim.x - 1;
    if (lane == 0 && gridDim.x > 1) asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(before) : "l"(ticket) : "memory");
    if (__shfl_sync(0xffffffffu, before, 0) == gridDim.x - 1) {
      if (lane == 0) {
        *ticket = 0;
        if (ok_state) t.state[2] = lacking ? (int)(all_take - have) : 0;
        if (change) {
          const int at = head + (int)all_take;        // all_take <= have <= n_slots
          t.state[0] = at < d.n_slots ? at : at - d.n_slots;
          t.state[1] = (int)(have - all_take);
        }
        if (lacking) set_error(err, KVS_ERR_CAPACITY);
      }
      if (change)
        for (int r = lane; r < n; r += 32)
          if (ctx[r] >= 0) t.n_held[r] = need[r];
    }
  }
  const int stride = gridDim.x * kTabThreads, first = blockIdx.x * kTabThreads + tid;
  auto ring_at = [&](int i) {      // i-th entry from the front, i < 2 n_slots - head
    const int at = head + i;
    return t.ring + (at < d.n_slots ? at : at - d.n_slots);
  };
  if (change) {
    bool lost = false;      // a slot outside the pool, in the ring or a row: it is moved as it is
    const int taken = (int)min(all_take, (unsigned)n_free);
    for (int i0 = first; i0 < taken; i0 += stride * kTabDeep) {
      int slot[kTabDeep];
#pragma unroll
      for (int k = 0; k < kTabDeep; ++k) slot[k] = i0 + k * stride < taken ? *ring_at(i0 + k * stride) : 0;
#pragma unroll
      for (int k = 0; k < kTabDeep; ++k) {
        const int i = i0 + k * stride;
        if (i >= taken) break;
        const int r = last_at(takes, n, i);
        lost |= (unsigned)slot[k] >= (unsigned)d.n_slots;
        t.table[(size_t)r * d.nb_max + held[r] + (i - takes[r])] = slot[k];
      }
    }
    for (int j0 = first; j0 < (int)all_give; j0 += stride * kTabDeep) {
      int slot[kTabDeep];
#pragma unroll
      for (int k = 0; k < kTabDeep; ++k) {
        const int j = j0 + k * stride;
        if (j < (int)all_give) {
          const int r = last_at(gives, n, j);
          slot[k] = t.table[(size_t)r * d.nb_max + need[r] + (j - gives[r])];
        }
      }
#pragma unroll
      for (int k = 0; k < kTabDeep; ++k) {
        const int j = j0 + k * stride, i = n_free + j;
        if (j >= (int)all_give) break;
        lost |= (unsigned)slot[k] >= (unsigned)d.n_slots;
        *ring_at(i) = slot[k];
        if (i < (int)all_take) {
          const int to = last_at(takes, n, i);
          t.table[(size_t)to * d.nb_max + held[to] + (i - takes[to])] = slot[k];
        }
      }
    }
    if (lost) set_error(err, KVS_ERR_BAD_INDEX);
  }
  if (!t.cu_q) return;
  // the slot of a request's block, or -1 where it has none
  auto slot_of = [&](int r, int block) {
    int slot = -1;
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
      return -1;      // the block was lacking
    }
    if (slot >= 0 && slot < d.n_slots) return slot;
    set_error(err, KVS_ERR_BAD_INDEX);
    return -1;
  };
  const bool wide = PER == 4 && ((reinterpret_cast<uintptr_t>(t.place) | reinterpret_cast<uintptr_t>(t.pos)) & 15) == 0;
  for (long long t0 = (long long)first * PER; t0 < t.n_tok; t0 += (long long)stride * PER) {
    long long place[PER];
    int pos[PER];
    int r = n ? last_at(cu, n, (int)t0) : 0, at_block = -1, slot = -1;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int tok = min((int)t0 + j, t.n_tok - 1);
      while (r + 1 < n && cu[r + 1] <= tok) {      // (offsets that descend end here as well: r grows)
        ++r;
        at_block = -1;
      }
      place[j] = -1;
      pos[j] = 0;
      if (n == 0) continue;      // nobody's
      const int a = cu[r], b = cu[r + 1];
      // (offsets that cannot be, and requests of a bad length, are reported above: their tokens have no place)
      if (a >= 0 && b <= t.n_tok && tok >= a && tok < b && ctx[r] >= 0) {
        const int p = ctx[r] - (b - tok);
        pos[j] = (int)((unsigned)p + (unsigned)delta[r]);
        if (p >= 0) {
          if (p >> d.log2bs != at_block) {
            at_block = p >> d.log2bs;
            slot = slot_of(r, at_block);
          }
          if (slot >= 0) place[j] = ((long long)slot << d.log2bs) + (p & (d.bs - 1));
        }
      }
    }
    if (wide && t0 + PER <= t.n_tok) {
      longlong2* to = reinterpret_cast<longlong2*>(t.place + t0);
      to[0] = make_longlong2(place[0], place[1 % PER]);
      to[1] = make_longlong2(place[2 % PER], place[3 % PER]);
      if (t.pos) *reinterpret_cast<int4*>(t.pos + t0) = make_int4(pos[0], pos[1 % PER], pos[2 % PER], pos[3 % PER]);
    } else {
#pragma unroll
      for (int j = 0; j < PER; ++j)
        if (t0 + j < t.n_tok) {
          t.place[t0 + j] = place[j];
          if (t.pos) t.pos[t0 + j] = pos[j];
        }
    }
  }
}

}  // namespace

cudaError_t launch_pool_tables(const PoolDims& d, const PoolTables& t, unsigned* ticket, unsigned* err, cudaStream_t s) {
  // A thread places one token (a batch's next tokens), or four where there are two for every thread of the GPU.  A call may move
  // as many blocks as the tables hold, and mostly moves few: up to 64 CTAs for large tables, with tokens or without (500 requests
  // that give 190 blocks back: 4.1 us with 1 to 64 CTAs, 4.4 with 244; 24 that give 7700: 13 us with 1, 4 with 12; 64 requests
  // of a token each, of which 8 end and give 16384 back, and the call that takes them again: 39 us with 1, 10.5 with 8, 7.1 with 64,
  // and 5.9 or 6.0 if none ends).
  const int sms = device_sm_count(), smem = (7 * t.n_req + 3) * 4;
  const bool many = t.n_tok > sms * kTabThreads * 2;
  auto ctas = [](long long threads, int most) { return (int)std::min<long long>((threads + kTabThreads - 1) / kTabThreads, most); };
  const int for_tokens = t.cu_q ? ctas(t.n_tok / (many ? 4 : 1), sms * 4) : 0;
  const int for_blocks = t.ring ? ctas((long long)t.n_req * d.nb_max / 4, 64) : 0;
  const int grid = std::max({1, for_tokens, for_blocks});
  auto go = [&](auto kernel) {
    cudaError_t e = cudaSuccess;      // (up to 47 KB need no asking)
    if (smem > 47 * 1024) e = set_max_dynamic_smem(reinterpret_cast<const void*>(kernel), (7 * kPoolMaxReq + 3) * 4);
    if (e != cudaSuccess) return e;
    launch_pdl(kernel, dim3(grid), dim3(kTabThreads), (size_t)smem, s, d, t, ticket, err);
    return cudaGetLastError();
  };
  return many ? go(pool_tables_kernel<4>) : go(pool_tables_kernel<1>);
}

}  // namespace kvs
