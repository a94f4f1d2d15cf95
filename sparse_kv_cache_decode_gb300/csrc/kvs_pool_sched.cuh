// The work of an attention call over a pool: its items, their tiles, each CTA's range and pieces, partial states and
// the output of a finished row.  Shared by the kernels for few and for many rows.
#pragma once
#include "kvs_pool_dev.cuh"

namespace kvs {
namespace pdev {

constexpr float kLn2 = 0.6931471805599453f;
constexpr float kMaxSum = 0x1p40f;              // largest sum of a tile's weights before m is set anew

struct Split {
  int n_cta;
  int min_per;      // tiles per CTA at least
};

// One item's partial state: which rows, and the last CTA that holds a piece of it (begun: in this CTA).
struct Meta {
  int t0, row0, nrows, head0, c1, seq, pad0, pad1;
};

// Scratch: meta [n_cta]; (m, l) [n_cta][2][256]; O [n_cta][2][256][d].
struct Scratch {
  Meta* meta;
  float2* ml;
  float* o;
};

__host__ __device__ inline Scratch scratch_of(void* p, int n_cta) {
  Scratch s;
  s.meta = static_cast<Meta*>(p);
  s.ml = reinterpret_cast<float2*>(s.meta + n_cta);
  s.o = reinterpret_cast<float*>(s.ml + (size_t)n_cta * 512);
  return s;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
// a / b, in 32 bits where they do
__device__ __forceinline__ long long div_ll(long long a, long long b) {
  return ((a | b) >> 31) == 0 ? (long long)((unsigned)a / (unsigned)b) : a / b;
}

// A CTA's piece of an item: rows [row0, row0 + nrows) of head h of sequence s against n of the item's nt tiles,
// from tile j0 on.  The item's rows see the keys [0, first) and [lo, hi).
struct __align__(16) Piece {
  int s, h, t0, row0, nrows;
  int p0;                 // position of the sequence's first query token
  int len;
  int first, lo, hi;
  int ns, lo_tile, nt;    // tiles of the first tokens, first tile of the span, tiles in all
  int j0, n;
  int pad;
};
static_assert(sizeof(Piece) == 64, "smem plan");

__device__ __forceinline__ void item_span(const PoolDims& d, const PoolSeqs& q, Piece& it) {
  if (!q.causal) {
    it.first = 0;
    it.lo = 0;
    it.hi = it.len;
  } else {
    const int pa = it.p0 + div_g(d, it.row0), pb = it.p0 + div_g(d, it.row0 + it.nrows - 1);
    it.hi = max(0, pb + 1);
    it.lo = q.window ? max(0, pa - q.window + 1) : 0;
    it.first = min(q.n_sink, it.lo);
  }
  it.lo_tile = it.lo / TOK;
  it.ns = min((it.first + TOK - 1) / TOK, it.lo_tile);
  it.nt = max(1, it.ns + (it.hi + TOK - 1) / TOK - it.lo_tile);
}

// Row block rb of a sequence: its rows and span.
__device__ __forceinline__ void item_rows(const PoolDims& d, const PoolSeqs& q, const SeqInfo& r, int RB, int rb, Piece& it) {
  it.t0 = r.t0;
  it.len = r.len;
  it.p0 = r.len - (r.t1 - r.t0);
  it.row0 = rb * RB;
  it.nrows = max(0, min(RB, (r.t1 - r.t0) * d.G - it.row0));
  item_span(d, q, it);
}

// Item number `pos` of the dealt-out order: position p = c * K + k is item k * n + c (the first n_items % n
// columns are one longer).
__device__ __forceinline__ int dealt(int p, int n_items, int n) {
  const int K = n_items / n, r = n_items - K * n;
  const int wide = r * (K + 1);
  if (p < wide) return (p % (K + 1)) * n + p / (K + 1);
  p -= wide;
  return (p % K) * n + r + p / K;
}

// Item i: the sequences' items follow one another, row block by row block, head by head.
__device__ __forceinline__ Piece item_at(const PoolDims& d, const PoolSeqs& q, const int* tab, int RB, int i, unsigned* err) {
  // the last sequence with tab[s] <= i (empty sequences hold no items, so it is the one that does)
  int lo = 0, hi = q.n_seq;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (tab[mid] <= i) lo = mid; else hi = mid;
  }
  Piece it;
  it.s = lo;
  const SeqInfo r = pool_seq(d, q, lo, err);
  const int local = i - tab[lo], rb = local / d.Hkv;
  it.h = local - rb * d.Hkv;
  item_rows(d, q, r, RB, rb, it);
  return it;
}

__device__ __forceinline__ int tile_base(const Piece& it, int j) { return (j < it.ns ? j : it.lo_tile + j - it.ns) * TOK; }
__device__ __forceinline__ bool key_seen(const Piece& it, int t) { return t < it.first || (t >= it.lo && t < it.hi); }
// every key of the tile at `base` is seen by some row
__device__ __forceinline__ bool tile_whole(const Piece& it, int base) {
  return (base >= it.lo && base + TOK <= it.hi) || base + TOK <= it.first;
}

// out / lse of one row from its joined state: D columns by the caller.
struct RowOut {
  float w_prev, w_new;    // weights of the earlier call's row and of this row's O
  float lse2;
};
__device__ __forceinline__ RowOut row_out(const PoolAttnOut& o, bool has_prev, size_t row, float m, float l, float v_scale) {
  RowOut r;
  r.w_prev = 0.f;
  r.w_new = l > 0.f ? v_scale / l : 0.f;
  r.lse2 = l > 0.f ? m + log2f(l) : -INFINITY;
  if (has_prev) {
    const float a = o.prev_lse2[row], M = fmaxf(a, r.lse2);
    if (M != -INFINITY) {
      const float ea = ex2(a - M), eb = ex2(r.lse2 - M), inv = 1.f / (ea + eb);
      r.w_prev = ea * inv;
      r.w_new *= eb * inv;
      r.lse2 = M + log2f(ea + eb);
    }
  }
  return r;
}
__device__ __forceinline__ void row_lse(const PoolAttnOut& o, size_t row, float lse2) {
  if (o.lse) o.lse[row] = lse2 * kLn2;
  if (o.lse2) o.lse2[row] = lse2;
}
// The CTA's range of the call's tiles: tab[s] = items before sequence s; plan[0..2] = its first item (position), that
// item's first tile, its tiles; plan[4] = items, plan[5] = tiles per CTA.  DEALT: the tiles in the order of dealt().
// Every thread of the CTA calls it; the caller synchronises behind it.  ws: 64 words of shared memory.
template <bool DEALT, int THREADS>
__device__ __forceinline__ void cta_range(const PoolDims& d, const PoolSeqs& seqs, int RB, int* tab, long long* ws, volatile int* plan,
                                          const Split& sp, int c, unsigned* err) {
  constexpr int NW = THREADS / 32;
  const int tid = threadIdx.x;
  const int per_s = (seqs.n_seq + THREADS - 1) / THREADS;
  const int s0 = min(seqs.n_seq, tid * per_s), s1 = min(seqs.n_seq, s0 + per_s);
  SeqInfo q1;                                // of the thread's last sequence
  // items and, in the order of sequences, tiles of a sequence
  auto seq_work = [&](int s, int* items) {
    q1 = pool_seq(d, seqs, s, err);
    const int n_rb = ((q1.t1 - q1.t0) * d.G + RB - 1) / RB;
    *items = n_rb * d.Hkv;
    long long v = 0;
    if (!DEALT)
      for (int rb = 0; rb < n_rb; ++rb) {
        Piece it;
        item_rows(d, seqs, q1, RB, rb, it);
        v += it.nt;
      }
    return v * d.Hkv;
  };
  int mine = 0, n1 = 0;
  long long tiles = 0, v1 = 0;
  for (int s = s0; s < s1; ++s) {
    v1 = seq_work(s, &n1);
    mine += n1;
    tiles += v1;
  }
  Scan r = block_scan(mine, tiles, ws, NW);
  const int n_items = r.n_all;
  {
    int at = r.n;
    for (int s = s0; s < s1; ++s) {
      tab[s] = at;
      if (s + 1 < s1) {      // the last one's count is not needed
        seq_work(s, &n1);
        at += n1;
      }
    }
    if (tid == 0) tab[seqs.n_seq] = n_items;
  }
  int i0 = 0, i1 = 0;
  if (DEALT) {
    __syncthreads();
    const int per_i = (n_items + THREADS - 1) / THREADS;
    i0 = min(n_items, tid * per_i);
    i1 = min(n_items, i0 + per_i);
    tiles = 0;
    for (int p = i0; p < i1; ++p) tiles += item_at(d, seqs, tab, RB, dealt(p, n_items, sp.n_cta), err).nt;
    r = block_scan(0, tiles, ws, NW);
  }
  const long long per = max((long long)sp.min_per, div_ll(r.v_all + sp.n_cta - 1, sp.n_cta));
  const long long f0 = per * c, f1 = min(r.v_all, f0 + per);
  if (f0 < f1 && f0 >= r.v && f0 < r.v + tiles) {
    long long f = r.v;
    int p = -1, j = 0;
    if (DEALT) {
      for (p = i0; p + 1 < i1; ++p) {
        const int nt = item_at(d, seqs, tab, RB, dealt(p, n_items, sp.n_cta), err).nt;
        if (f0 < f + nt) break;
        f += nt;
      }
      j = (int)(f0 - f);
    } else {
      for (int s = s0; s < s1 && p < 0; ++s) {
        const long long v = s1 - s0 == 1 ? v1 : seq_work(s, &n1);
        if (f0 >= f + v) {
          f += v;
          continue;
        }
        for (int rb = 0; p < 0; ++rb) {
          Piece it;
          item_rows(d, seqs, q1, RB, rb, it);
          const long long w = (long long)it.nt * d.Hkv;
          if (f0 < f + w) {
            const int h = (int)div_ll(f0 - f, it.nt);
            p = tab[s] + rb * d.Hkv + h;
            j = (int)(f0 - f - (long long)h * it.nt);
          }
          f += w;
        }
      }
    }
    plan[0] = p;
    plan[1] = j;
    plan[2] = (int)(f1 - f0);
  }
  if (tid == 0) {
    plan[4] = n_items;
    plan[5] = (int)per;
  }
}

// Plans the CTA's next kPieces pieces (one warp, a lane per piece): pieces[0 .. plan[3]); plan[2] = tiles left.
template <bool DEALT>
__device__ __forceinline__ void plan_pieces(const PoolDims& d, const PoolSeqs& seqs, int RB, const int* tab, volatile int* plan,
                                            Piece* pieces, int n_cta, unsigned* err) {
  const int lane = threadIdx.x & 31;
  int pos = plan[0], j0 = plan[1], left = plan[2], cnt = 0;
  const int n_items = plan[4];
  for (int x = 0; x < kPieces && left > 0; x += 32) {
    Piece it;
    it.nt = 0;
    if (pos + lane < n_items) it = item_at(d, seqs, tab, RB, DEALT ? dealt(pos + lane, n_items, n_cta) : pos + lane, err);
    it.j0 = lane == 0 ? j0 : 0;
    const long long w = it.nt - it.j0;
    long long incl = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    it.n = (int)max(0ll, min(w, left - (incl - w)));
    if (it.n > 0) pieces[x + lane] = it;
    const int got = __popc(__ballot_sync(0xffffffffu, it.n > 0));
    const long long all = __shfl_sync(0xffffffffu, incl, 31);
    left = (int)max(0ll, left - all);
    pos += got;
    cnt += got;
    j0 = 0;
  }
  __syncwarp();
  if (lane == 0) {
    plan[0] = pos;
    plan[1] = 0;
    plan[2] = pos < n_items ? left : 0;
    plan[3] = cnt;
  }
}

// The range and the first pieces of a CTA in one warp, for at most 32 sequences of at most RB rows each (a lane per sequence,
// then a lane per piece); false where there are more rows, and nothing is planned.  (The general way through the block
// took 3 us of a 9 us call.)
__device__ __forceinline__ bool plan_few(const PoolDims& d, const PoolSeqs& seqs, int RB, int* tab, volatile int* plan,
                                         Piece* pieces, const Split& sp, int c, unsigned* err) {
  const int lane = threadIdx.x & 31;
  SeqInfo q = {0, 0, 0};
  if (lane < seqs.n_seq) q = pool_seq(d, seqs, lane, err);
  const int R = (q.t1 - q.t0) * d.G;
  Piece it;
  item_rows(d, seqs, q, RB, 0, it);
  const int nt = R > 0 ? it.nt : 0;
  // tiles in 32 bits
  if (__any_sync(0xffffffffu, R > RB || (long long)nt * d.Hkv > (1 << 25))) return false;
  int incl = nt * d.Hkv;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  const unsigned some = __ballot_sync(0xffffffffu, nt > 0);
  const int before = __popc(some & ((1u << lane) - 1)) * d.Hkv;      // items before this lane's sequence
  if (lane < seqs.n_seq) tab[lane] = before;
  const int total = __shfl_sync(0xffffffffu, incl, 31), n_items = __popc(some) * d.Hkv;
  const int per = max(sp.min_per, (total + sp.n_cta - 1) / sp.n_cta);
  const int f0 = per * c, f1 = min(total, f0 + per);
  const unsigned at = __ballot_sync(0xffffffffu, f0 < f1 && f0 < incl);
  int cnt = 0, left = max(0, f1 - f0), pos = 0;
  if (at) {
    const int s0 = __ffs(at) - 1;
    const int off = f0 - __shfl_sync(0xffffffffu, incl - nt * d.Hkv, s0), nt0 = __shfl_sync(0xffffffffu, nt, s0);
    const int h0 = off / nt0, j0 = off - h0 * nt0;
    pos = __shfl_sync(0xffffffffu, before, s0) + h0;
    // piece `lane`: item pos + lane
    const int item = pos + lane, rank = item / d.Hkv;
    int s = 0;                             // the rank-th of the lanes in `some`
#pragma unroll
    for (int o = 16; o; o >>= 1)
      if (__popc(some & ((1u << (s + o)) - 1)) <= rank) s += o;
    if (item >= n_items) s = 0;
    const SeqInfo r = {__shfl_sync(0xffffffffu, q.t0, s), __shfl_sync(0xffffffffu, q.t1, s), __shfl_sync(0xffffffffu, q.len, s)};
    item_rows(d, seqs, r, RB, 0, it);
    it.s = s;
    it.h = item - rank * d.Hkv;
    it.j0 = lane == 0 ? j0 : 0;
    const int w = item < n_items ? it.nt - it.j0 : 0;
    int sum = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += y;
    }
    it.n = max(0, min(w, left - (sum - w)));
    if (it.n > 0) pieces[lane] = it;
    cnt = __popc(__ballot_sync(0xffffffffu, it.n > 0));
    left = max(0, left - __shfl_sync(0xffffffffu, sum, 31));
    pos += cnt;
  }
  __syncwarp();
  if (lane == 0) {
    tab[seqs.n_seq] = n_items;
    plan[0] = pos;
    plan[1] = 0;
    plan[2] = pos < n_items ? left : 0;
    plan[3] = cnt;
    plan[4] = n_items;
    plan[5] = per;
  }
  return true;
}

}  // namespace pdev

// The merge kernel behind an attention kernel: items of at most `rows` rows.
cudaError_t launch_pool_merge(const PoolDims& d, const PoolAttnOut& o, void* scratch, int n_cta, int rows, cudaStream_t s);

}  // namespace kvs
