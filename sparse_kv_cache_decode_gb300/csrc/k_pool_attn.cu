// Device-resident pools: attention of ragged query rows over paged K/V on the 5th-generation tensor cores.
//
// Rows.  The rows of a (sequence, kv head) are its query tokens times the group's G heads, row = token * G + g,
// so one K/V tile serves a whole group.  An item is a block of 128 * QT such rows; the keys its rows see are
// visited in tiles of 128 tokens: the tiles of the first n_sink tokens, then those of the window's span.
//   S = Q K^T (128 x 128, fp32 in tensor memory),  P = 2^(S scale log2 e - m) in bf16 over S's columns,
//   O (128 x d, fp32 in tensor memory) += P V,      out = v_scale O / l,  l = sum of P before its rounding.
// m is raised (and O rescaled) only when a tile's maximum passes it by more than 2^8, so P stays below 2^8.
// P is rounded to bf16 (relative error 2^-9 on average of both signs, as the output's own rounding); S, m, l
// and O are fp32.
//
// Two softmax groups of 4 warps, one thread per row.  Where an item has more than 128 rows each group takes
// 128 of them and both read every K/V tile; where it has at most 128 the groups take the tiles in turn over
// the same rows, and their states are joined at the end.  Either way one group's products run while the other
// computes its exponentials.
//
// Split.  The tiles of all items form one sequence that is cut into equal ranges, one per CTA (one CTA per SM);
// an item cut by a range's end leaves partial states (m, l, O) that the merge kernel joins.  The items are dealt
// out so that CTAs work on neighbouring items at the same time (their K/V windows overlap and meet in L2).
// Lengths, offsets and tables are read on the device: each CTA derives the sequence and its range from them.
//
// Roles: warp 0 brings K/V tiles with tensor loads, one per block and 64 dims, skipping blocks that no row of the
// item sees; warp 1 issues the products; warps 2-3 load Q; warps 4-11 are the softmax groups; with E4M3 pools
// warps 12-15 widen the codes to bf16 tiles (every E4M3 value is exact in bf16).
// Value rows that no row of the item sees are zeroed in shared memory before their product: they may hold
// anything, and 0 * NaN would reach every row.  All waits are bounded (KVS_ERR_TIMEOUT).
#include <algorithm>

#include <cuda_fp16.h>

#include "kvs_pool.cuh"
#include "kvs_ptx.cuh"
#include "kvs_tmem128.cuh"

namespace kvs {

namespace {
namespace pa {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kMaxGrowth = 8.f;
constexpr int TOK = 128;                      // tokens per tile
constexpr int MAX_SMEM = 227 * 1024;

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

template <int D, bool FP8, int QT>
struct Cfg {
  static constexpr int CHUNKS = D / 64;                       // 64-dim (128-byte) chunks of a bf16 row
  static constexpr int QTILE = TOK * D * 2;                   // one 128-row tile of Q
  static constexpr int TILE = TOK * D * 2;                    // one bf16 K or V tile
  static constexpr int CODES = TOK * D;                       // one tile of E4M3 codes
  static constexpr int THREADS = FP8 ? 512 : 384;
  static constexpr int FIXED = 2048 + 512 + 1024;             // group states, barriers, alignment
  static constexpr int ROOM = MAX_SMEM - FIXED - 4 * (kPoolMaxReq + 1) - QT * QTILE;
  static constexpr int STAGING = FP8 ? (D == 128 ? 3 : 4) : 0;         // code tiles in flight
  static constexpr int S_BF = (ROOM - STAGING * CODES) / TILE;
  static constexpr int STAGES = S_BF > 8 ? 8 : S_BF;
  static constexpr int RB = TOK * QT;
  static constexpr int OFF_RING = QT * QTILE;
  static constexpr int OFF_STG = OFF_RING + STAGES * TILE;
  static constexpr int OFF_ML = OFF_STG + STAGING * CODES;
  static constexpr int OFF_BAR = OFF_ML + 2048;
  static constexpr int OFF_TAB = OFF_BAR + 512;
  static_assert(STAGES >= 3, "shared memory plan");
  static_assert(OFF_TAB + 4 * (kPoolMaxReq + 1) + 1024 <= MAX_SMEM, "shared memory plan");
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// An item: rows [row0, row0 + nrows) of head h of sequence s, and the keys it sees: [0, first) and [lo, hi).
struct Item {
  int s, h, t0, row0, nrows, R;
  int p0;                 // position of the sequence's first query token
  int len;
  int first, lo, hi;      // keys some row of the item sees
  int ns, lo_tile, nt;    // tiles of the first tokens, first tile of the span, tiles in all
};

__device__ __forceinline__ void item_span(const PoolSeqs& q, int G, Item& it) {
  if (!q.causal) {
    it.first = 0;
    it.lo = 0;
    it.hi = it.len;
  } else {
    const int pa = it.p0 + it.row0 / G, pb = it.p0 + (it.row0 + it.nrows - 1) / G;
    it.hi = max(0, pb + 1);
    it.lo = q.window ? max(0, pa - q.window + 1) : 0;
    it.first = min(q.n_sink, it.lo);
  }
  it.lo_tile = it.lo / TOK;
  it.ns = min((it.first + TOK - 1) / TOK, it.lo_tile);
  it.nt = max(1, it.ns + (it.hi + TOK - 1) / TOK - it.lo_tile);
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

template <int RB>
__device__ __forceinline__ Item item_at(const PoolDims& d, const PoolSeqs& q, const int* tab, int i, unsigned* err) {
  // the last sequence with tab[s] <= i (empty sequences hold no items, so it is the one that does)
  int lo = 0, hi = q.n_seq;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (tab[mid] <= i) lo = mid; else hi = mid;
  }
  Item it;
  it.s = lo;
  const SeqInfo r = pool_seq(d, q, lo, err);
  const int local = i - tab[lo], rb = local / d.Hkv;
  it.h = local - rb * d.Hkv;
  it.t0 = r.t0;
  it.len = r.len;
  it.p0 = r.len - (r.t1 - r.t0);
  it.R = (r.t1 - r.t0) * d.G;
  it.row0 = rb * RB;
  it.nrows = max(0, min(RB, it.R - it.row0));
  item_span(q, d.G, it);
  return it;
}

__device__ __forceinline__ int tile_base(const Item& it, int j) { return (j < it.ns ? j : it.lo_tile + j - it.ns) * TOK; }
__device__ __forceinline__ bool key_seen(const Item& it, int t) { return t < it.first || (t >= it.lo && t < it.hi); }
// every key of the tile at `base` is seen by some row
__device__ __forceinline__ bool tile_whole(const Item& it, int base) {
  return (base >= it.lo && base + TOK <= it.hi) || base + TOK <= it.first;
}

// Exclusive scan over the CTA's threads (64-bit); ws: 33 words of shared memory.
__device__ __forceinline__ long long block_scan(long long v, long long* ws, int nw, long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) ws[warp] = x;
  __syncthreads();
  long long before = x - v, all = 0;
  for (int w = 0; w < nw; ++w) {
    if (w < warp) before += ws[w];
    all += ws[w];
  }
  *total = all;
  return before;
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
// 4 columns of a finished row at element e of the output arrays
__device__ __forceinline__ void row_store4(const PoolAttnOut& o, size_t e, float4 y) {
  if (o.part_out) *reinterpret_cast<float4*>(o.part_out + e) = y;
  else *reinterpret_cast<uint2*>(o.out + e) = make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
}

template <int D, bool FP8, int QT>
__global__ void __launch_bounds__(Cfg<D, FP8, QT>::THREADS, 1)
    pool_attn_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, PoolDims d,
                     const __nv_bfloat16* __restrict__ q, long long q_stride, PoolSeqs seqs, PoolAttnOut o,
                     void* scratch, Split sp, unsigned* err) {
  using C = Cfg<D, FP8, QT>;
  constexpr int RB = C::RB, S = C::STAGES, NW = C::THREADS / 32;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* ring = smem + C::OFF_RING;
  unsigned char* stg = smem + C::OFF_STG;
  float2* ml = reinterpret_cast<float2*>(smem + C::OFF_ML);           // [2][128]
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* kv_full = bars;             // [8]
  uint64_t* kv_empty = bars + 8;        // [8]
  uint64_t* raw_full = bars + 16;       // [4] code tiles (E4M3)
  uint64_t* raw_empty = bars + 20;      // [4]
  uint64_t* s_full = bars + 24;         // [2]
  uint64_t* p_full = bars + 26;         // [2]
  uint64_t* o_full = bars + 28;         // [2]
  uint64_t* q_full = bars + 30;
  uint64_t* q_free = bars + 31;
  uint64_t* drained = bars + 32;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 33);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* start = reinterpret_cast<int*>(tmem_slot + 2);                 // first position, its first tile, tiles, items
  int* tab = reinterpret_cast<int*>(smem + C::OFF_TAB);               // [n_seq + 1] items before each sequence
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c = blockIdx.x;

  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&kv_full[i], FP8 ? 4 : 1);
      mbar_init(&kv_empty[i], 1);
    }
    if (FP8)
      for (int i = 0; i < 4; ++i) {
        mbar_init(&raw_full[i], 1);
        mbar_init(&raw_empty[i], 4);
      }
    for (int g = 0; g < 2; ++g) {
      mbar_init(&s_full[g], 1);
      mbar_init(&p_full[g], 4);
      mbar_init(&o_full[g], 1);
    }
    mbar_init(q_full, 2);
    mbar_init(q_free, 1);
    mbar_init(drained, 1);
    *abort_flag = 0;
    start[2] = 0;
    mbar_fence_init();
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == 1) tmem_alloc(tmem_slot, 512);
  kvs_pdl_entry();

  // ------------------------------------------------------------------ the CTA's range of tiles
  const Scratch sc = scratch_of(scratch, sp.n_cta);
  {
    long long* ws = reinterpret_cast<long long*>(ml);
    const int per_s = (seqs.n_seq + C::THREADS - 1) / C::THREADS;
    int mine = 0;
    for (int s = tid * per_s; s < min(seqs.n_seq, (tid + 1) * per_s); ++s) {
      const SeqInfo r = pool_seq(d, seqs, s, err);
      mine += (int)(((long long)(r.t1 - r.t0) * d.G + RB - 1) / RB) * d.Hkv;
    }
    long long n_all;
    int at = (int)block_scan(mine, ws, NW, &n_all);
    for (int s = tid * per_s; s < min(seqs.n_seq, (tid + 1) * per_s); ++s) {
      const SeqInfo r = pool_seq(d, seqs, s, err);
      tab[s] = at;
      at += (int)(((long long)(r.t1 - r.t0) * d.G + RB - 1) / RB) * d.Hkv;
    }
    const int n_items = (int)n_all;
    if (tid == 0) tab[seqs.n_seq] = n_items;
    __syncthreads();
    const int per_i = (n_items + C::THREADS - 1) / C::THREADS;
    const int i0 = min(n_items, tid * per_i), i1 = min(n_items, i0 + per_i);
    long long tiles = 0, total;
    for (int p = i0; p < i1; ++p) tiles += item_at<RB>(d, seqs, tab, dealt(p, n_items, sp.n_cta), err).nt;
    long long f = block_scan(tiles, ws, NW, &total);
    const long long per = max((long long)sp.min_per, (total + sp.n_cta - 1) / sp.n_cta);
    const long long f0 = per * c, f1 = min(total, f0 + per);
    if (f0 < f1 && f0 >= f && f0 < f + tiles) {
      for (int p = i0; p < i1; ++p) {
        const int nt = item_at<RB>(d, seqs, tab, dealt(p, n_items, sp.n_cta), err).nt;
        if (f0 < f + nt) {
          start[0] = p;
          start[1] = (int)(f0 - f);
          start[2] = (int)(f1 - f0);
          break;
        }
        f += nt;
      }
    }
    if (tid == 0) {
      start[3] = n_items;
      start[4] = (int)per;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int n_items = start[3], per = start[4];
  const uint64_t timeout_ns = (uint64_t)d.timeout_us * 1000ull;
  auto wait = [&](uint64_t* bar, unsigned parity) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t = global_timer_ns();
    while (!mbar_try_wait(bar, parity)) {
      if (*abort_flag) return false;
      if (global_timer_ns() - t > timeout_ns) {
        set_error(err, KVS_ERR_TIMEOUT);
        *abort_flag = 1;
        return false;
      }
    }
    return true;
  };
  // the pieces of this CTA in order: (item, first tile, tiles)
  int pos = start[0], j0 = start[1], left = start[2];
  auto next_item = [&]() { return item_at<RB>(d, seqs, tab, dealt(pos, n_items, sp.n_cta), err); };
  auto advance = [&](int n) {
    left -= n;
    ++pos;
    j0 = 0;
  };

  if (warp == 0) {
    // ------------------------------------------------------------------ K/V tiles
    // a lane per (block, chunk) of a tile: K first, then V, each into the next slot of the ring
    constexpr int BOXES = FP8 ? 1 : C::CHUNKS;
    constexpr int SLOTS = FP8 ? C::STAGING : S;
    uint64_t* full = FP8 ? raw_full : kv_full;
    uint64_t* empty = FP8 ? raw_empty : kv_empty;
    const int pages = TOK >> d.log2bs;
    const int box_bytes = d.bs * (FP8 ? D : 128);
    int k = 0;
    bool ok = true;
    while (left > 0 && ok) {
      const Item it = next_item();
      const int n = min(left, it.nt - j0);
      const int* table = seqs.table + (size_t)it.s * d.nb_max;
      for (int j = j0; j < j0 + n && ok; ++j) {
        const int base = tile_base(it, j);
        // lane p: block p of the tile, its slot if some row sees one of its tokens
        int row = -1;
        if (lane < pages) {
          const int b0 = base + (lane << d.log2bs), b1 = b0 + d.bs;
          if ((b0 < it.first) || (b0 < it.hi && b1 > it.lo)) {
            const int slot = table[b0 >> d.log2bs];
            if (slot < 0 || slot >= d.n_slots) set_error(err, KVS_ERR_BAD_INDEX);
            else row = (slot * d.Hkv + it.h) * d.bs;
          }
        }
        const int n_load = __popc(__ballot_sync(0xffffffffu, row >= 0));
        for (int x = 0; x < 2; ++x, ++k) {
          const int s = k % SLOTS;
          ok = k < SLOTS || __all_sync(0xffffffffu, wait(&empty[s], ((k / SLOTS) & 1) ^ 1));
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(&full[s], (unsigned)(n_load * BOXES * box_bytes));
          __syncwarp();
          if (row >= 0) {
            unsigned char* dst = FP8 ? stg + s * C::CODES + lane * box_bytes : ring + s * C::TILE + lane * box_bytes;
            for (int b = 0; b < BOXES; ++b)
              tma_load_2d(dst + b * (TOK * 128), x ? &tmV : &tmK, b * 64, row, &full[s]);
          }
        }
      }
      advance(n);
    }
    __syncwarp();
    // no tensor load may still be writing this CTA's shared memory when it exits
    for (int i = max(0, k - SLOTS); i < k; ++i) mbar_wait(&full[i % SLOTS], (i / SLOTS) & 1, kDrainTimeoutNs);
  } else if (warp == 1) {
    // ------------------------------------------------------------------ products
    if (lane == 0) {
      const uint32_t id_qk = idesc_bf16_f32(128, TOK);
      const uint32_t id_pv = idesc_bf16_f32(128, D) | (1u << 16);     // V is read MN-major
      const uint64_t dq = smem_desc_sw128(smem_u32(smem));
      int N = 0, piece = 0;           // tiles before this piece; pieces
      int ops[2] = {0, 0};            // products S of each group so far
      bool ok = true;
      while (left > 0 && ok) {
        const Item it = next_item();
        const int n = min(left, it.nt - j0);
        const bool pair = it.nrows > 128;
        if (!wait(q_full, piece & 1)) break;
        const int n_ops = pair ? 2 * n : n;
        // operation x: tile x / 2 (pair) or x of the piece, group x % 2; its PV follows when the group's next
        // operation comes up
        auto pv = [&](int x) {
          const int g = x & 1, tile = N + (pair ? x >> 1 : x);
          const int first = x < 2, s = (2 * tile + 1) % S;
          if (!wait(&p_full[g], (ops[g] - 1) & 1) || !wait(&kv_full[s], ((2 * tile + 1) / S) & 1)) return false;
          tc_fence_after();
          const uint32_t v0 = smem_u32(ring + s * C::TILE);
#pragma unroll
          for (int kk = 0; kk < TOK / 16; ++kk)
            tc_mma_f16_ts(tmem + 256 + g * D, tmem + g * 128 + kk * 8, smem_desc_sw128_mn(v0 + kk * 2048, TOK * 128, 1024),
                          id_pv, !(first && kk == 0));
          if (!pair || g) tc_commit(&kv_empty[s]);
          if (x + 2 >= n_ops) tc_commit(&o_full[g]);
          return true;
        };
        for (int x = 0; x < n_ops && ok; ++x) {
          if (x >= 2) ok = pv(x - 2);
          if (!ok) break;
          const int g = x & 1, tile = N + (pair ? x >> 1 : x), s = (2 * tile) % S;
          if (!wait(&kv_full[s], ((2 * tile) / S) & 1)) { ok = false; break; }
          tc_fence_after();
          const uint64_t dk = smem_desc_sw128(smem_u32(ring + s * C::TILE));
          const uint64_t da = dq + (uint64_t)((pair ? g * C::QTILE : 0) >> 4);
#pragma unroll
          for (int k16 = 0; k16 < D / 16; ++k16) {
            const uint64_t off = (uint64_t)(((k16 >> 2) * (TOK * 128) + (k16 & 3) * 32) >> 4);
            tc_mma_f16(tmem + g * 128, da + off, dk + off, id_qk, k16 != 0);
          }
          tc_commit(&s_full[g]);
          ++ops[g];
          if (!pair || g) tc_commit(&kv_empty[s]);
          if (x == n_ops - 1) tc_commit(q_free);
        }
        for (int x = max(0, n_ops - 2); x < n_ops && ok; ++x) ok = pv(x);
        N += n;
        ++piece;
        advance(n);
      }
      // every product issued by this thread has finished before the tensor memory is released
      tc_commit(drained);
      mbar_wait(drained, 0, kDrainTimeoutNs);
    }
    __syncwarp();
  } else if (warp < 4) {
    // ------------------------------------------------------------------ Q, once the last piece's products have read it
    int piece = 0;
    while (left > 0) {
      const Item it = next_item();
      const int n = min(left, it.nt - j0);
      if (piece > 0 && !__all_sync(0xffffffffu, wait(q_free, (piece - 1) & 1))) break;
      constexpr int VEC = D / 8;       // 16-byte vectors of a row
      for (int i = tid - 64; i < it.nrows * VEC; i += 64) {
        const int r = i / VEC, v = i - r * VEC, row = it.row0 + r;
        const int tok = row / d.G, g = row - tok * d.G;
        const __nv_bfloat16* src = q + (it.t0 + tok) * q_stride + (it.h * d.G + g) * D + v * 8;
        unsigned char* dst = smem + (r >> 7) * C::QTILE + (v >> 3) * (TOK * 128) + (r & 127) * 128 + (((v & 7) ^ (r & 7)) << 4);
        cp_async16(dst, src, 16);
      }
      cp_async_commit();
      cp_async_wait_all();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
      ++piece;
      advance(n);
    }
    cp_async_wait_all();
  } else if (warp < 12) {
    // ------------------------------------------------------------------ softmax and output
    const int g = (warp - 4) >> 2, lr = (warp & 3) * 32 + lane;      // group; row of its 128
    const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t tS = trow + g * 128, tO = trow + 256 + g * D;
    const float sl2 = d.scale * d.k_scale * kLog2e;
    int N = 0, n_ops = 0, n_out[2] = {0, 0};
    while (left > 0) {
      const Item it = next_item();
      const int n = min(left, it.nt - j0);
      const bool pair = it.nrows > 128;
      const int r = pair ? g * 128 + lr : lr;                          // row of the item
      const bool live = r < it.nrows;
      const int row = it.row0 + r;
      // the keys this row sees, and those every row of this group sees
      int hi = live ? it.len : 0, lo = 0, first = 0, hi_all = it.len, lo_all = 0, first_all = 0;
      if (seqs.causal) {
        const int ra = it.row0 + (pair ? g * 128 : 0), rb = min(ra + 127, it.row0 + it.nrows - 1);
        const int p = it.p0 + row / d.G, pa = it.p0 + ra / d.G, pb = it.p0 + rb / d.G;
        hi = live ? max(0, p + 1) : 0;
        lo = seqs.window ? max(0, p - seqs.window + 1) : 0;
        first = min(seqs.n_sink, lo);
        hi_all = max(0, pa + 1);
        lo_all = seqs.window ? max(0, pb - seqs.window + 1) : 0;
        first_all = seqs.window ? min(seqs.n_sink, max(0, pa - seqs.window + 1)) : 0;
      }
      float m = -INFINITY, l = 0.f;
      const int step = pair ? 1 : 2;
      for (int j = pair ? 0 : g; j < n; j += step) {
        const int base = tile_base(it, j0 + j);
        wait(&s_full[g], n_ops & 1);
        tc_fence_after();
        float s[128];
        tmem_ld128(tS, s);
        const bool whole = (base + TOK <= hi_all && base >= lo_all) || base + TOK <= first_all;
        if (!whole) {
          const int h = hi - base, a = lo - base, f = first - base;
#pragma unroll
          for (int i = 0; i < 128; ++i)
            if (!(i < h && (i >= a || i < f))) s[i] = -INFINITY;
        }
        float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int i = 4; i < 128; i += 4) {
          mx[0] = fmaxf(mx[0], s[i]);
          mx[1] = fmaxf(mx[1], s[i + 1]);
          mx[2] = fmaxf(mx[2], s[i + 2]);
          mx[3] = fmaxf(mx[3], s[i + 3]);
        }
        const float tmax = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl2;
        const bool grow = tmax > m + kMaxGrowth || (m == -INFINITY && tmax != -INFINITY);
        const float m_new = grow ? tmax : m;
        // O holds earlier tiles' products (all finished: S of this tile was issued behind them)
        if (__any_sync(0xffffffffu, grow && l > 0.f)) {
          const float f = grow && l > 0.f ? ex2(m - m_new) : 1.f;
#pragma unroll 1
          for (int c0 = 0; c0 < D; c0 += 32) {
            float ov[32];
            tmem_ld32(tO + c0, ov);
#pragma unroll
            for (int i = 0; i < 32; ++i) ov[i] *= f;
            tmem_st32(tO + c0, ov);
          }
          l *= f;
        }
        m = m_new;
        const float neg = m == -INFINITY ? 0.f : -m;
        float ps[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c0 = 0; c0 < 128; c0 += 32) {
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const float a = ex2(fmaf(s[c0 + i], sl2, neg)), b = ex2(fmaf(s[c0 + i + 1], sl2, neg));
            ps[i & 2] += a;
            ps[(i & 2) + 1] += b;
            pk[i / 2] = pack_bf16x2(a, b);
          }
          tmem_st16(tS + c0 / 2, pk);
        }
        l += (ps[0] + ps[1]) + (ps[2] + ps[3]);
        tmem_wait_st();
        if (!FP8 && !tile_whole(it, base)) {
          // value rows that no row of the item sees (a row per thread)
          const int slot = 2 * (N + j) + 1;
          wait(&kv_full[slot % S], (slot / S) & 1);
          if (!key_seen(it, base + lr)) {
            unsigned char* vr = ring + (slot % S) * C::TILE + lr * 128;
            for (int b = 0; b < C::CHUNKS; ++b)
#pragma unroll
              for (int i = 0; i < 8; ++i) *reinterpret_cast<uint4*>(vr + b * (TOK * 128) + i * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[g]);
        ++n_ops;
      }
      // ---------------------------------------------------------------- the piece's end
      const bool begun = j0 == 0, done = j0 + n == it.nt;
      const int tok = it.t0 + row / d.G, head = it.h * d.G + row % d.G;
      const size_t orow = (size_t)tok * d.Hq + head;
      const bool whole = begun && done;
      const size_t prow = ((size_t)c * 2 + (begun ? 1 : 0)) * 256 + r;      // partial state's place
      const bool has_prev = o.prev_out && it.s >= o.prev_req[0] && it.s < o.prev_req[o.n_prev];
      float w0 = 1.f, w1 = 0.f;          // weights of the two groups' O
      int ca = 0, cb = D;                // columns this thread writes
      uint32_t tA = tO, tB = tO;
      if (pair) {
        wait(&o_full[g], n_out[g] & 1);
        ++n_out[0];
        ++n_out[1];
      } else {
        const int both = min(n, 2);       // groups with a tile
        wait(&o_full[0], n_out[0]++ & 1);
        if (both == 2) wait(&o_full[1], n_out[1]++ & 1);
        ml[g * 128 + lr] = make_float2(m, l);
        named_bar_sync(1, 256);
        const float2 a = ml[lr], b = ml[128 + lr];
        const float M = fmaxf(a.x, b.x);
        w0 = a.x == -INFINITY ? 0.f : ex2(a.x - M);
        w1 = b.x == -INFINITY ? 0.f : ex2(b.x - M);
        l = w0 * a.y + w1 * b.y;
        m = M;
        ca = g * (D / 2);
        cb = ca + D / 2;
        tA = trow + 256;
        tB = trow + 256 + D;
      }
      tc_fence_after();
      const bool one = pair || n < 2;    // a single O
      if (__any_sync(0xffffffffu, live)) {
        RowOut ro = {0.f, 1.f, 0.f};
        if (whole && live) ro = row_out(o, has_prev, orow, m, l, d.v_scale);
        const bool has = l > 0.f;
#pragma unroll 1
        for (int c0 = ca; c0 < cb; c0 += 32) {
          float x[32];
          tmem_ld32(tA + c0, x);
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = w0 > 0.f ? x[i] * w0 : 0.f;
          if (!one) {
            float y[32];
            tmem_ld32(tB + c0, y);
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] += w1 > 0.f ? y[i] * w1 : 0.f;
          }
          if (!live) continue;
          if (whole) {
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              float4 y = has ? make_float4(x[i] * ro.w_new, x[i + 1] * ro.w_new, x[i + 2] * ro.w_new, x[i + 3] * ro.w_new)
                             : make_float4(0.f, 0.f, 0.f, 0.f);
              if (has_prev && ro.w_prev > 0.f) {
                const float4 z = *reinterpret_cast<const float4*>(o.prev_out + orow * D + c0 + i);
                y = make_float4(y.x + ro.w_prev * z.x, y.y + ro.w_prev * z.y, y.z + ro.w_prev * z.z, y.w + ro.w_prev * z.w);
              }
              row_store4(o, orow * D + c0 + i, y);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              *reinterpret_cast<float4*>(sc.o + prow * D + c0 + i) =
                  has ? make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]) : make_float4(0.f, 0.f, 0.f, 0.f);
          }
        }
        if (live && (pair || g == 0)) {
          if (whole) row_lse(o, orow, ro.lse2);
          else sc.ml[prow] = make_float2(m, l);
        }
      }
      if (begun && !done && warp == 4 && lane == 0) {
        // the item goes on in the next CTAs: up to the one that holds its last tile
        const long long f_end = (long long)per * c + (start[2] - left) + it.nt;
        sc.meta[c] = {it.t0, it.row0, it.nrows, it.h * d.G, (int)((f_end - 1) / per), it.s, 0, 0};
      }
      tc_fence_before();
      if (!pair) named_bar_sync(1, 256);     // both groups have read the states and both O
      N += n;
      advance(n);
      if (left <= 0 && warp == 4 && lane == 0 && !(begun && !done)) sc.meta[c].nrows = 0;
    }
    if (start[2] == 0 && warp == 4 && lane == 0) sc.meta[c].nrows = 0;
  } else if constexpr (FP8) {
    // ------------------------------------------------------------------ E4M3 codes -> bf16 tiles
    int k = 0;
    bool ok = true;
    while (left > 0 && ok) {
      const Item it = next_item();
      const int n = min(left, it.nt - j0);
      for (int j = j0; j < j0 + n && ok; ++j) {
        const int base = tile_base(it, j);
        const bool part = !tile_whole(it, base);
        for (int x = 0; x < 2; ++x, ++k) {
          const int s = k % S, rs = k % C::STAGING;
          ok = __all_sync(0xffffffffu, wait(&raw_full[rs], (k / C::STAGING) & 1) &&
                                           (k < S || wait(&kv_empty[s], ((k / S) & 1) ^ 1)));
          if (!ok) break;
          const unsigned char* src = stg + rs * C::CODES;
          unsigned char* dst = ring + s * C::TILE;
          constexpr int VEC = D / 16;              // 16-code vectors of a row
#pragma unroll 4
          for (int i = tid - 384; i < TOK * VEC; i += 128) {
            const int row = i / VEC, v = i - row * VEC;
            uint4 w = *reinterpret_cast<const uint4*>(src + row * D + v * 16);
            if (x && part && !key_seen(it, base + row)) w = make_uint4(0, 0, 0, 0);
            const uint32_t in[4] = {w.x, w.y, w.z, w.w};
            uint32_t out[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              uint32_t h2;
              asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)(in[e >> 1] >> ((e & 1) * 16))));
              const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
              out[e] = pack_bf16x2(f.x, f.y);
            }
            unsigned char* p = dst + (v >> 2) * (TOK * 128) + row * 128;
            const int c16 = (v & 3) * 2;
            *reinterpret_cast<uint4*>(p + ((c16 ^ (row & 7)) << 4)) = make_uint4(out[0], out[1], out[2], out[3]);
            *reinterpret_cast<uint4*>(p + (((c16 + 1) ^ (row & 7)) << 4)) = make_uint4(out[4], out[5], out[6], out[7]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&raw_empty[rs]);
            mbar_arrive(&kv_full[s]);
          }
        }
      }
      advance(n);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the partial states of the items that a range's end cut: block (c, y) the rows [8 y, 8 y + 8) of the
// item that CTA c began, one warp per row.
constexpr int kMergeWarps = 8;

template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32)
    pool_merge_kernel(PoolDims d, PoolAttnOut o, void* scratch, int n_cta) {
  kvs_pdl_entry();
  const Scratch sc = scratch_of(scratch, n_cta);
  const int c = blockIdx.x, lane = threadIdx.x & 31;
  const int r = blockIdx.y * kMergeWarps + (threadIdx.x >> 5);
  const Meta mt = sc.meta[c];
  if (r >= mt.nrows) return;
  const int n = mt.c1 - c + 1;                           // pieces: (c, 1), (c + 1, 0) .. (c1, 0)
  auto place = [&](int i) { return ((size_t)(c + i) * 2 + (i == 0 ? 1 : 0)) * 256 + r; };
  float M = -INFINITY;
  for (int i = lane; i < n; i += 32) M = fmaxf(M, sc.ml[place(i)].x);
#pragma unroll
  for (int w = 16; w; w >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, w));
  float l = 0.f;
  constexpr int E = D / 32;
  float acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  for (int i0 = 0; i0 < n; i0 += 32) {
    float w = 0.f;
    if (i0 + lane < n) {
      const float2 v = sc.ml[place(i0 + lane)];
      w = v.x == -INFINITY ? 0.f : ex2(v.x - M);
      l += w * v.y;
    }
    const int cnt = min(32, n - i0);
#pragma unroll 4
    for (int i = 0; i < cnt; ++i) {
      const float wi = __shfl_sync(0xffffffffu, w, i);
      const float* p = sc.o + place(i0 + i) * D + lane * E;
      if (E == 4) {
        const float4 x = *reinterpret_cast<const float4*>(p);
        acc[0] += wi * x.x;
        acc[1] += wi * x.y;
        acc[E - 2] += wi * x.z;
        acc[E - 1] += wi * x.w;
      } else {
        const float2 x = *reinterpret_cast<const float2*>(p);
        acc[0] += wi * x.x;
        acc[1] += wi * x.y;
      }
    }
  }
#pragma unroll
  for (int w = 16; w; w >>= 1) l += __shfl_xor_sync(0xffffffffu, l, w);
  const int row = mt.row0 + r;
  const size_t orow = (size_t)(mt.t0 + row / d.G) * d.Hq + mt.head0 + row % d.G;
  const bool has_prev = o.prev_out && mt.seq >= o.prev_req[0] && mt.seq < o.prev_req[o.n_prev];
  const RowOut ro = row_out(o, has_prev, orow, M, l, d.v_scale);
#pragma unroll
  for (int e = 0; e < E; ++e) {
    acc[e] *= ro.w_new;
    if (has_prev && ro.w_prev > 0.f) acc[e] += ro.w_prev * o.prev_out[orow * D + lane * E + e];
  }
  const size_t at = orow * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; e += 2) {
    if (o.part_out) *reinterpret_cast<float2*>(o.part_out + at + e) = make_float2(acc[e], acc[e + 1]);
    else *reinterpret_cast<uint32_t*>(o.out + at + e) = pack_bf16x2(acc[e], acc[e + 1]);
  }
  if (lane == 0) row_lse(o, orow, ro.lse2);
}

template <int D, bool FP8, int QT>
cudaError_t launch(const PoolDims& d, const CUtensorMap* tm, const __nv_bfloat16* q, long long q_stride,
                   const PoolSeqs& seqs, const PoolAttnOut& o, void* scratch, unsigned* err, cudaStream_t s) {
  using C = Cfg<D, FP8, QT>;
  auto kern = pool_attn_kernel<D, FP8, QT>;
  const int smem = C::OFF_TAB + 4 * (seqs.n_seq + 1) + 1024;
  cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void*>(kern), MAX_SMEM);
  if (e != cudaSuccess) return e;
  Split sp;
  sp.n_cta = device_sm_count();
  sp.min_per = 2;
  launch_pdl(kern, dim3(sp.n_cta), dim3(C::THREADS), smem, s, tm[0], tm[1], d, q, q_stride, seqs, o, scratch, sp, err);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // an item has at most 128 * QT rows, and no more than the call has
  const int rows = (int)std::min<long long>(C::RB, (long long)seqs.n_tok * d.G);
  launch_pdl(pool_merge_kernel<D>, dim3(sp.n_cta, (rows + kMergeWarps - 1) / kMergeWarps), dim3(kMergeWarps * 32), 0, s, d, o,
             scratch, sp.n_cta);
  return cudaGetLastError();
}

}  // namespace pa
}  // namespace

size_t pool_attn_scratch_bytes(const PoolDims& d) {
  const size_t n = device_sm_count();
  return n * (sizeof(pa::Meta) + 512 * (sizeof(float2) + (size_t)d.d * 4));
}

cudaError_t launch_pool_attn(const PoolDims& d, const unsigned char*, const unsigned char*, const CUtensorMap* tm,
                             const __nv_bfloat16* q, long long q_stride, const PoolSeqs& seqs, const PoolAttnOut& o,
                             void* scratch, unsigned* err, cudaStream_t s, int* n_launched) {
  using namespace pa;
  *n_launched = 2;
  // rows per (sequence, head) on average: more than 128 rows pay for two row tiles per K/V tile
  const bool two = (long long)seqs.n_tok * d.G > 128ll * seqs.n_seq;
  if (d.d == 128) {
    if (d.fp8) return two ? launch<128, true, 2>(d, tm, q, q_stride, seqs, o, scratch, err, s)
                          : launch<128, true, 1>(d, tm, q, q_stride, seqs, o, scratch, err, s);
    return two ? launch<128, false, 2>(d, tm, q, q_stride, seqs, o, scratch, err, s)
               : launch<128, false, 1>(d, tm, q, q_stride, seqs, o, scratch, err, s);
  }
  if (d.fp8) return two ? launch<64, true, 2>(d, tm, q, q_stride, seqs, o, scratch, err, s)
                        : launch<64, true, 1>(d, tm, q, q_stride, seqs, o, scratch, err, s);
  return two ? launch<64, false, 2>(d, tm, q, q_stride, seqs, o, scratch, err, s)
             : launch<64, false, 1>(d, tm, q, q_stride, seqs, o, scratch, err, s);
}

}  // namespace kvs
