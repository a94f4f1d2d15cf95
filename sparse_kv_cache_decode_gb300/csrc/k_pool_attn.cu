// Device-resident pools: attention of ragged query rows over paged K/V on the 5th-generation tensor cores.
//
// Rows.  The rows of a (sequence, kv head) are its query tokens times the group's G heads, row = token * G + g,
// so one K/V tile serves a whole group.  A row tile holds the heads of 128 / G whole tokens, an item up to two of
// them; the keys its rows see are
// visited in tiles of 128 tokens: the tiles of the first n_sink tokens, then those of the window's span.
//   S = Q K^T (128 x 128, fp32 in tensor memory),  P = 2^(S scale log2 e - m) in bf16 over S's columns,
//   O (128 x d, fp32 in tensor memory) += P V,      out = v_scale O / l,  l = sum of P before its rounding.
// m is the maximum of the first tile that a row sees.  It is not looked for again: the scale cancels in O / l and fp32
// has room for weights above 1 (O < 2^40 * tiles * |v|), so it is enough to set m anew, and rescale O, when a tile's sum
// passes 2^40 (a logit some 23 above the first tile's largest).  P is rounded to bf16 (relative error 2^-9 on average of both signs, as the output's own rounding); S, m, l
// and O are fp32.
//
// Two softmax groups of 4 warps, one thread per row.  Where an item has two row tiles each group takes
// one of them and both read every K/V tile; where it has one the groups take the tiles in turn over
// the same rows, and their states are joined at the end.  Either way one group's products run while the other
// computes its exponentials.
//
// Split.  The tiles of all items form one sequence that is cut into equal ranges, one per CTA (one CTA per SM);
// an item cut by a range's end leaves partial states (m, l, O) that the merge kernel joins.  The items are dealt
// out so that CTAs work on neighbouring items at the same time (their K/V windows overlap and meet in L2).
// Lengths, offsets and tables are read on the device: each CTA derives the sequence and its range from them.
//
// Roles: warp 0 brings K/V tiles with tensor loads, one per block and 64 dims, skipping blocks that no row of the
// item sees; warp 1 issues the products; warp 2 brings Q; warps 4-11 are the softmax groups; with E4M3 pools
// warps 12-15 widen the codes to bf16 tiles (every E4M3 value is exact in bf16).
// Value rows that no row of the item sees are zeroed in shared memory before their product: they may hold
// anything, and 0 * NaN would reach every row.  All waits are bounded (KVS_ERR_TIMEOUT).
#include <algorithm>

#include "kvs_pool_sched.cuh"
#include "kvs_tmem128.cuh"

namespace kvs {

namespace {
namespace pa {

using namespace pdev;

template <int D, bool FP8>
struct Cfg {
  static constexpr int CHUNKS = D / 64;                       // 64-dim (128-byte) chunks of a bf16 row
  // Q: two row tiles, of one item or (up to one row tile each) of two items in turn
  static constexpr int QCHUNK = 256 * 128;
  static constexpr int QBYTES = CHUNKS * QCHUNK;
  static constexpr int TILE = TOK * D * 2;                    // one bf16 K or V tile
  static constexpr int CODES = TOK * D;                       // one tile of E4M3 codes
  static constexpr int THREADS = FP8 ? 512 : 384;
  static constexpr int FIXED = 2048 + 512 + 1024;             // group states, barriers, alignment
  static constexpr int ROOM = MAX_SMEM - FIXED - 4 * (kPoolMaxReq + 1) - kPieces * 64 - QBYTES;
  static constexpr int STAGING = FP8 ? (D == 128 ? 3 : 4) : 0;         // code tiles in flight
  static constexpr int S_BF = (ROOM - STAGING * CODES) / TILE;
  static constexpr int STAGES = S_BF > 8 ? 8 : S_BF;
  // registers of the helper and the softmax warps (the groups of 128 threads share the launch's registers)
  static constexpr int REGS_LOW = 72, REGS_HIGH = FP8 ? 184 : 216;
  static_assert(FP8 ? 2 * REGS_LOW + 2 * REGS_HIGH <= 4 * 128 : REGS_LOW + 2 * REGS_HIGH <= 3 * 168, "register plan");
  static constexpr int OFF_RING = QBYTES;
  static constexpr int OFF_STG = OFF_RING + STAGES * TILE;
  static constexpr int OFF_ML = OFF_STG + STAGING * CODES;
  static constexpr int OFF_BAR = OFF_ML + 2048;
  static constexpr int OFF_PIECES = OFF_BAR + 512;
  // room for 32 rows of 64 bytes a softmax warp, through which outputs are written row by row (d = 128 with E4M3 pools has none)
  static constexpr bool STAGE_OUT = ROOM - STAGING * CODES - STAGES * TILE >= 16384;
  static constexpr int OFF_OUT = OFF_PIECES + kPieces * 64;
  static constexpr int OFF_TAB = OFF_OUT + (STAGE_OUT ? 16384 : 0);
  static_assert(STAGES >= 3, "shared memory plan");
  static_assert(OFF_TAB + 4 * (kPoolMaxReq + 1) + 1024 <= MAX_SMEM, "shared memory plan");
};

template <int N>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N)); }

template <int D, bool FP8>
__global__ void __launch_bounds__(Cfg<D, FP8>::THREADS, 1)
    pool_attn_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const __grid_constant__ CUtensorMap tmQ, PoolDims d, PoolSeqs seqs, PoolAttnOut o, void* scratch,
                     Split sp, unsigned* err) {
  using C = Cfg<D, FP8>;
  constexpr int S = C::STAGES;
  const int RT = d.rt, RB = 2 * RT;     // rows of a row tile, of an item
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
  uint64_t* o_full = bars + 30;         // [2]
  uint64_t* q_full = bars + 32;         // [2] by piece parity
  uint64_t* q_free = bars + 34;         // [2] by piece parity
  uint64_t* drained = bars + 36;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 37);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  // position and first tile of the CTA's next piece, its tiles still to plan, pieces planned, items, tiles per CTA
  volatile int* plan = reinterpret_cast<volatile int*>(tmem_slot + 2);
  Piece* pieces = reinterpret_cast<Piece*>(smem + C::OFF_PIECES);
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
    mbar_init(&q_full[0], 1);
    mbar_init(&q_full[1], 1);
    mbar_init(&q_free[0], 1);
    mbar_init(&q_free[1], 1);
    mbar_init(drained, 1);
    *abort_flag = 0;
    plan[0] = plan[1] = plan[2] = 0;
    mbar_fence_init();
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
    tma_prefetch_desc(&tmQ);
  }
  if (warp == 1) tmem_alloc(tmem_slot, 512);
  kvs_pdl_entry();

  cta_range<true, C::THREADS>(d, seqs, RB, tab, reinterpret_cast<long long*>(ml), plan, sp, c, err);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = (uint32_t)uniform((int)*tmem_slot);
  const uint64_t timeout_ns = (uint64_t)d.timeout_us * 1000ull;
  const Scratch sc = scratch_of(scratch, sp.n_cta);
  auto wait = [&](uint64_t* bar, unsigned parity) { return bounded_wait(bar, parity, timeout_ns, abort_flag); };
  if (warp == 0) plan_pieces<true>(d, seqs, RB, tab, plan, pieces, sp.n_cta, err);
  __syncthreads();
  // Between two lists of pieces (long calls only): every role is done with the old one.
  auto more = [&]() {
    const int l = plan[2];
    __syncthreads();
    if (l <= 0) return false;
    if (warp == 0) plan_pieces<true>(d, seqs, RB, tab, plan, pieces, sp.n_cta, err);
    __syncthreads();
    return true;
  };

  if (warp == 0) {
    // ------------------------------------------------------------------ K/V tiles
    // a lane per block of a tile: K first, then V, each into the next slot of the ring
    regs_dec<C::REGS_LOW>();
    constexpr int BOXES = FP8 ? 1 : C::CHUNKS;
    constexpr int SLOTS = FP8 ? C::STAGING : S;
    uint64_t* full = FP8 ? raw_full : kv_full;
    uint64_t* empty = FP8 ? raw_empty : kv_empty;
    const int pages = TOK >> d.log2bs;
    const int box_bytes = d.bs * (FP8 ? D : 128);
    int k = 0;
    bool ok = true;
    do {
      const int cnt = plan[3];
      for (int i = 0; i < cnt && ok; ++i) {
        const Piece it = pieces[i];
        const int* table = seqs.table + (size_t)it.s * d.nb_max;
        for (int j = it.j0; j < it.j0 + it.n && ok; ++j) {
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
#pragma unroll
              for (int b = 0; b < BOXES; ++b)
                tma_load_2d(dst + b * (TOK * 128), x ? &tmV : &tmK, b * 64, row, &full[s]);
            }
          }
        }
      }
    } while (more());
    __syncwarp();
    // no tensor load may still be writing this CTA's shared memory when it exits
    for (int i = max(0, k - SLOTS); i < k; ++i) mbar_wait(&full[i % SLOTS], (i / SLOTS) & 1, kDrainTimeoutNs);
  } else if (warp == 1) {
    // ------------------------------------------------------------------ products
    // Two row tiles: per K/V tile, group by group: PV of this tile once P is there, then S of the next tile, which
    // overwrites P.  One row tile: S of tile x for group x % 2, PV of the group's last tile before it, oldest first,
    // across pieces.  The tensor pipe idles whenever this thread is late, so the waits ahead of a product are few:
    // K and V once per tile, P in halves.
    regs_dec<C::REGS_LOW>();
    const uint32_t id_qk = idesc_bf16_f32(128, TOK);
    const uint32_t id_pv = idesc_bf16_f32(128, D) | (1u << 16);     // V is read MN-major
    const uint32_t aq = smem_u32(smem) >> 4, ar = smem_u32(ring) >> 4;
    constexpr uint32_t kV = (uint32_t)(TOK * 128 >> 4) << 16;       // from one 64-dim block of V to the next
    int N = 0, piece = 0, qb = 0;   // tiles and pieces before this one, the half that holds its Q
    int pend0 = -1, pend1 = -1;     // one row tile: the groups' operations whose PV is due: tile * 4 + last * 2 + first
    int older = 0;                  // the group whose operation came first
    unsigned par0 = 0, par1 = 0;    // parity of each group's next P
    bool ok = true;
    auto qk = [&](int g, int s, int qrow) {
      const uint32_t k0 = ar + s * (C::TILE >> 4), q0 = aq + qrow * (128 >> 4), t = tmem + g * 128;
      mma_ss<false>(t, q0, k0, id_qk);
#pragma unroll
      for (int k16 = 1; k16 < D / 16; ++k16)
        mma_ss<true>(t, q0 + (((k16 >> 2) * C::QCHUNK + (k16 & 3) * 32) >> 4), k0 + (((k16 >> 2) * (TOK * 128) + (k16 & 3) * 32) >> 4),
                     id_qk);
      tc_commit(&s_full[g]);
    };
    auto pv = [&](int g, int s, bool first, unsigned& par) {
      ok = wait(&p_full[g], par);
      if (!ok) return;
      par ^= 1;
      tc_fence_after();
      const uint32_t v0 = (ar + s * (C::TILE >> 4)) | kV, t = tmem + 256 + g * D, p0 = tmem + g * 128;
      mma_ts(t, p0, v0, id_pv, !first);
#pragma unroll
      for (int kk = 1; kk < TOK / 16; ++kk) mma_ts(t, p0 + kk * 8, v0 + kk * (2048 >> 4), id_pv);
    };
    auto pv_due = [&](int g) {
      const int info = g ? pend1 : pend0, slot = 2 * (info >> 2) + 1, s = slot % S;
      if (g) pend1 = -1; else pend0 = -1;
      older = g ^ 1;
      ok = wait(&kv_full[s], (slot / S) & 1);
      if (!ok) return;
      if (g) pv(1, s, info & 1, par1); else pv(0, s, info & 1, par0);
      if (!ok) return;
      tc_commit(&kv_empty[s]);
      if (info & 2) tc_commit(&o_full[g]);
    };
    auto flush = [&]() {
      for (int y = 0; y < 2 && ok; ++y) {
        const int g = (older ? pend1 : pend0) >= 0 ? older : older ^ 1;
        if ((g ? pend1 : pend0) >= 0) pv_due(g);
      }
    };
    do {
      const int cnt = plan[3];
      if (elect_one()) {
        for (int i = 0; i < cnt && ok; ++i, ++piece) {
          const int nrows = pieces[i].nrows, n = pieces[i].n;
          qb = nrows <= RT ? qb ^ 1 : 0;
          if (nrows > RT || !mbar_try_wait(&q_full[piece & 1], (piece >> 1) & 1)) {
            flush();                       // while Q is on its way: what is due
            if (!ok || !wait(&q_full[piece & 1], (piece >> 1) & 1)) { ok = false; break; }
          }
          if (nrows > RT) {
            int s = (2 * N) % S;
            unsigned par = ((2 * N) / S) & 1;          // slot and parity of the next tile to wait for
            auto next = [&]() {
              if (++s == S) {
                s = 0;
                par ^= 1;
              }
            };
            int sv = 0, sk = 0;
            // V of tile t and K of tile t + 1, waited for ahead of the products before them
            auto next_kv = [&](bool with_k) {
              sv = s;
              ok = wait(&kv_full[s], par);
              next();
              if (with_k) {
                sk = s;
                ok = ok && wait(&kv_full[s], par);
                next();
              }
            };
            ok = wait(&kv_full[s], par);
            if (!ok) break;
            tc_fence_after();
            qk(0, s, 0);
            const int s0 = s;
            next();
            next_kv(n > 1);
            if (!ok) break;
            qk(1, s0, 128);
            tc_commit(&kv_empty[s0]);
            for (int t = 0; t + 1 < n; ++t) {
              pv(0, sv, t == 0, par0);
              if (!ok) break;
              qk(0, sk, 0);
              pv(1, sv, t == 0, par1);
              if (!ok) break;
              tc_commit(&kv_empty[sv]);
              const int s1 = sk;
              next_kv(t + 2 < n);
              if (!ok) break;
              qk(1, s1, 128);
              tc_commit(&kv_empty[s1]);
            }
            if (!ok) break;
            tc_commit(&q_free[piece & 1]);
            pv(0, sv, n == 1, par0);
            if (!ok) break;
            tc_commit(&o_full[0]);
            pv(1, sv, n == 1, par1);
            if (!ok) break;
            tc_commit(&kv_empty[sv]);
            tc_commit(&o_full[1]);
          } else {
            for (int x = 0; x < n && ok; ++x) {
              const int g = x & 1, tile = N + x, s = (2 * tile) % S;
              while ((g ? pend1 : pend0) >= 0 && ok) pv_due((older ? pend1 : pend0) >= 0 ? older : g);
              if (!ok || !wait(&kv_full[s], ((2 * tile) / S) & 1)) { ok = false; break; }
              tc_fence_after();
              qk(g, s, qb * 128);
              tc_commit(&kv_empty[s]);
              if (x == n - 1) tc_commit(&q_free[piece & 1]);
              const int info = tile * 4 + (x + 2 >= n ? 2 : 0) + (x < 2 ? 1 : 0);
              if (g) pend1 = info; else pend0 = info;
              if ((g ? pend0 : pend1) < 0) older = g;
            }
          }
          N += n;
        }
        if (ok) flush();
      }
      __syncwarp();
    } while (more());
    // every product issued here has finished before the tensor memory is released
    if (elect_one()) tc_commit(drained);
    mbar_wait(drained, 0, kDrainTimeoutNs);
    __syncwarp();
  } else if (warp == 2) {
    // ------------------------------------------------------------------ Q: whole tokens, so one load per row tile and chunk
    // Two items of at most one row tile each use the two places: piece p's Q waits for the products of piece p - 2, and
    // where one of p - 1 and p has two row tiles, for those of p - 1 as well.  A parity tells phases apart only while the one
    // waited for is the barrier's last: q_free[p & 1] completes phase p / 2 with piece p's products, which need the Q that
    // waits here for phase p / 2 - 1, and every phase is waited for, so none is passed unseen.  (With one barrier for all
    // pieces, phase p - 1 may be complete as well, and is at a new list of pieces: the wait for p - 2 would not end.)
    regs_dec<C::REGS_LOW>();
    int piece = 0, qb = 0, last_small = 1;
    bool ok = true;
    do {
      const int cnt = plan[3];
      if (elect_one()) {
        for (int i = 0; i < cnt && ok; ++i, ++piece) {
          const Piece& it = pieces[i];
          const int small = it.nrows <= RT;
          qb = small ? qb ^ 1 : 0;
          if (piece >= 2) ok = wait(&q_free[piece & 1], ((piece >> 1) - 1) & 1);
          if (ok && piece >= 1 && !(small && last_small)) ok = wait(&q_free[(piece - 1) & 1], ((piece - 1) >> 1) & 1);
          last_small = small;
          if (!ok) break;
          mbar_arrive_expect_tx(&q_full[piece & 1], (unsigned)((small ? 1 : 2) * C::CHUNKS * RT * 128));
          for (int x = 0; x < (small ? 1 : 2); ++x)
#pragma unroll
            for (int b = 0; b < C::CHUNKS; ++b)
              tma_load_3d(smem + b * C::QCHUNK + (qb + x) * (128 * 128), &tmQ, b * 64, it.h * d.G,
                          it.t0 + div_g(d, it.row0) + x * (RT / d.G), &q_full[piece & 1]);
        }
        // no load may still be on its way when the CTA exits
        for (int i = max(0, piece - 2); i < piece; ++i) mbar_wait(&q_full[i & 1], (i >> 1) & 1, kDrainTimeoutNs);
      }
      __syncwarp();
    } while (more());
  } else if (warp == 3) {
    regs_dec<C::REGS_LOW>();
    while (more()) {
    }
  } else if (warp < 12) {
    // ------------------------------------------------------------------ softmax and output
    regs_inc<C::REGS_HIGH>();
    const int g = (warp - 4) >> 2, lr = (warp & 3) * 32 + lane;      // group; row of its 128
    const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t tS = trow + g * 128, tO = trow + 256 + g * D;
    const float sl2 = d.scale * d.k_scale * kLog2e;
    int N = 0, n_ops = 0, n_out0 = 0, n_out1 = 0;
    if (warp == 4 && lane == 0) sc.meta[c].nrows = 0;
    do {
      const int cnt = plan[3];
      for (int i = 0; i < cnt; ++i) {
        const Piece& it = pieces[i];
        const int n = it.n, nrows = it.nrows, j0 = it.j0;
        const bool pair = nrows > RT;
        const int r = pair ? g * RT + lr : lr;                           // row of the item
        const bool live = lr < RT && r < nrows;
        const int row = it.row0 + r;
        // the keys this row sees, and those every row of this group sees
        int hi = live ? it.len : 0, lo = 0, first = 0, hi_all = it.len, lo_all = 0;
        if (seqs.causal) {
          const int ra = it.row0 + (pair ? g * RT : 0), rb = min(ra + RT - 1, it.row0 + nrows - 1);
          const int p = it.p0 + div_g(d, row), pa = it.p0 + div_g(d, ra), pb = it.p0 + div_g(d, rb);
          hi = live ? max(0, p + 1) : 0;
          hi_all = max(0, pa + 1);
          if (seqs.window) {
            lo = max(0, p - seqs.window + 1);
            first = min(seqs.n_sink, lo);
            lo_all = max(0, pb - seqs.window + 1);
          }
        }
        // tiles of the span that every row of the group sees as a whole: nothing to mask, no value row to zero
        const int ja = it.ns + (lo_all + TOK - 1) / TOK - it.lo_tile - j0;
        const unsigned n_whole = (unsigned)max(0, it.ns + hi_all / TOK - it.lo_tile - j0 - ja);
        float m = -INFINITY, l = 0.f;
        for (int j = pair ? 0 : g; j < n; j += pair ? 1 : 2) {
          wait(&s_full[g], n_ops & 1);
          tc_fence_after();
          float s[128];
          tmem_ld128(tS, s);
          if ((unsigned)(j - ja) >= n_whole) {
            const int base = tile_base(it, j0 + j);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const int off = base + 32 * w;
              const uint32_t vis = bits_below(hi - off) & (~bits_below(lo - off) | bits_below(first - off));
              if (__all_sync(0xffffffffu, vis == 0xffffffffu)) continue;
#pragma unroll
              for (int i2 = 0; i2 < 32; ++i2)
                if (!(vis & (1u << i2))) s[32 * w + i2] = -INFINITY;
            }
            if (!FP8 && !tile_whole(it, base)) {
              // value rows that no row of the item sees
              const int slot = 2 * (N + j) + 1;
              wait(&kv_full[slot % S], (slot / S) & 1);
              zero_rows(ring + (slot % S) * C::TILE, C::CHUNKS, lr & ~31, __ballot_sync(0xffffffffu, !key_seen(it, base + lr)));
              fence_proxy_async_smem();
            }
          }
          const uint64_t sl22 = pack2(sl2, sl2);
          // this row's m has to be set from the tile's maximum (lanes without a row hold whatever Q's place held: never)
          bool fix = live && m == -INFINITY;
#pragma unroll 1
          for (int pass = 0;; ++pass) {          // twice at most
            if (__any_sync(0xffffffffu, fix)) {
              float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
              for (int i2 = 4; i2 < 124; i2 += 8) {
#pragma unroll
                for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], s[i2 + 2 * e], s[i2 + 2 * e + 1]);
              }
#pragma unroll
              for (int e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], s[124 + e]);
              const float m_new = fix ? fmaxf(m, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl2) : m;
              // O holds earlier tiles' products (all finished: S of this tile was issued behind them)
              if (__any_sync(0xffffffffu, l > 0.f && m_new > m)) {
                const float f = l > 0.f ? ex2(m - m_new) : 1.f;
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += 16) {
                  float ov[16];
                  uint32_t ow[16];
                  tmem_ld16(tO + c0, ov);
#pragma unroll
                  for (int i2 = 0; i2 < 16; ++i2) ow[i2] = __float_as_uint(ov[i2] * f);
                  tmem_st16(tO + c0, ow);
                }
                l *= f;
              }
              m = m_new;
            }
            const float neg = m == -INFINITY ? 0.f : -m;
            const uint64_t neg2 = pack2(neg, neg);
            uint64_t ps0 = 0, ps1 = 0;
#pragma unroll
            for (int c0 = 0; c0 < 128; c0 += 32) {
              uint32_t pk[16];
#pragma unroll
              for (int i2 = 0; i2 < 32; i2 += 2) {
                float a, b;
                unpack2(fma2(pack2(s[c0 + i2], s[c0 + i2 + 1]), sl22, neg2), a, b);
                a = ex2(a);
                b = ex2(b);
                if (i2 & 2) ps1 = add2(ps1, pack2(a, b));
                else ps0 = add2(ps0, pack2(a, b));
                pk[i2 / 2] = pack_bf16x2(a, b);
              }
              tmem_st16(tS + c0 / 2, pk);
            }
            float a, b;
            unpack2(add2(ps0, ps1), a, b);
            // a row whose weights grew past the limit: set m anew and do the tile again (m is its maximum then)
            fix = live && a + b > kMaxSum;
            if (pass > 0 || !__any_sync(0xffffffffu, fix)) {
              l += a + b;
              break;
            }
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[g]);
          ++n_ops;
        }
        // -------------------------------------------------------------- the piece's end
        const bool begun = j0 == 0, done = j0 + n == it.nt, whole = begun && done;
        const int tok = it.t0 + div_g(d, row), head = it.h * d.G + row - div_g(d, row) * d.G;
        const size_t orow = (size_t)tok * d.Hq + head;
        const size_t prow = ((size_t)c * 2 + (begun ? 1 : 0)) * 256 + r;      // partial state's place
        const bool has_prev = o.prev_out && it.s >= o.prev_req[0] && it.s < o.prev_req[o.n_prev];
        float w0 = 1.f, w1 = 0.f;          // weights of the two groups' O
        int ca = 0, cb = D;                // columns this thread writes
        uint32_t tA = tO, tB = tO;
        const bool one = pair || n < 2;    // a single O
        if (pair) {
          wait(&o_full[g], (g ? n_out1 : n_out0) & 1);
          ++n_out0;
          ++n_out1;
        } else {
          wait(&o_full[0], n_out0++ & 1);
          if (!one) wait(&o_full[1], n_out1++ & 1);
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
        if (__any_sync(0xffffffffu, live)) {
          RowOut ro = {0.f, 1.f, 0.f};
          if (whole && live) ro = row_out(o, has_prev, orow, m, l, d.v_scale);
          const bool has = l > 0.f;
          const size_t to = whole ? orow : prow;             // this row's place among those written
          const unsigned lives = __ballot_sync(0xffffffffu, live);
#pragma unroll 1
          for (int c0 = ca; c0 < cb; c0 += 32) {
            float x[32];
            tmem_ld32(tA + c0, x);
#pragma unroll
            for (int i2 = 0; i2 < 32; ++i2) x[i2] = w0 > 0.f ? x[i2] * w0 : 0.f;
            if (!one) {
              float y[32];
              tmem_ld32(tB + c0, y);
#pragma unroll
              for (int i2 = 0; i2 < 32; ++i2) x[i2] += w1 > 0.f ? y[i2] * w1 : 0.f;
            }
            if (whole) {
              const bool prev = live && has_prev && ro.w_prev > 0.f;
              float4 z[8];
#pragma unroll
              for (int i2 = 0; i2 < 8; ++i2)       // the earlier call's row, all of it on its way at once
                z[i2] = prev ? __ldg(reinterpret_cast<const float4*>(o.prev_out + orow * D + c0) + i2) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
              for (int i2 = 0; i2 < 8; ++i2) {
                x[4 * i2] = (has ? x[4 * i2] * ro.w_new : 0.f) + ro.w_prev * z[i2].x;
                x[4 * i2 + 1] = (has ? x[4 * i2 + 1] * ro.w_new : 0.f) + ro.w_prev * z[i2].y;
                x[4 * i2 + 2] = (has ? x[4 * i2 + 2] * ro.w_new : 0.f) + ro.w_prev * z[i2].z;
                x[4 * i2 + 3] = (has ? x[4 * i2 + 3] * ro.w_new : 0.f) + ro.w_prev * z[i2].w;
              }
            } else if (!has) {
#pragma unroll
              for (int i2 = 0; i2 < 32; ++i2) x[i2] = 0.f;
            }
            float* f32 = whole ? o.part_out : sc.o;
            if constexpr (C::STAGE_OUT) {
              // 64 bytes of each of the warp's 32 rows at a time: written by rows' threads, read back by four threads a row
              unsigned char* st = smem + C::OFF_OUT + (warp - 4) * 2048;
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                if (!f32 && half) break;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  uint4 v;
                  if (f32) {
                    const int i2 = half * 16 + e * 4;
                    v = make_uint4(__float_as_uint(x[i2]), __float_as_uint(x[i2 + 1]), __float_as_uint(x[i2 + 2]),
                                   __float_as_uint(x[i2 + 3]));
                  } else {
                    v = make_uint4(pack_bf16x2(x[8 * e], x[8 * e + 1]), pack_bf16x2(x[8 * e + 2], x[8 * e + 3]),
                                   pack_bf16x2(x[8 * e + 4], x[8 * e + 5]), pack_bf16x2(x[8 * e + 6], x[8 * e + 7]));
                  }
                  *reinterpret_cast<uint4*>(st + lane * 64 + ((e ^ ((lane >> 1) & 3)) << 4)) = v;
                }
                __syncwarp();
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const int rr = e * 8 + (lane >> 2), part = lane & 3;
                  const uint4 v = *reinterpret_cast<const uint4*>(st + rr * 64 + ((part ^ ((rr >> 1) & 3)) << 4));
                  const size_t at = (size_t)__shfl_sync(0xffffffffu, (unsigned long long)to, rr) * D + c0;
                  if ((lives >> rr) & 1u) {
                    if (f32) *reinterpret_cast<uint4*>(f32 + at + half * 16 + part * 4) = v;
                    else *reinterpret_cast<uint4*>(o.out + at + part * 8) = v;
                  }
                }
                __syncwarp();
              }
            } else if (live) {
#pragma unroll
              for (int i2 = 0; i2 < 32; i2 += 8) {
                if (f32) {
                  *reinterpret_cast<float4*>(f32 + to * D + c0 + i2) = make_float4(x[i2], x[i2 + 1], x[i2 + 2], x[i2 + 3]);
                  *reinterpret_cast<float4*>(f32 + to * D + c0 + i2 + 4) = make_float4(x[i2 + 4], x[i2 + 5], x[i2 + 6], x[i2 + 7]);
                } else {
                  *reinterpret_cast<uint4*>(o.out + to * D + c0 + i2) =
                      make_uint4(pack_bf16x2(x[i2], x[i2 + 1]), pack_bf16x2(x[i2 + 2], x[i2 + 3]),
                                 pack_bf16x2(x[i2 + 4], x[i2 + 5]), pack_bf16x2(x[i2 + 6], x[i2 + 7]));
                }
              }
            }
          }
          if (live && (pair || g == 0)) {
            if (whole) row_lse(o, orow, ro.lse2);
            else sc.ml[prow] = make_float2(m, l);
          }
        }
        if (begun && !done && warp == 4 && lane == 0) {
          // the item goes on in the next CTAs: up to the one that holds its last tile
          const int per = plan[5];
          const long long f_end = (long long)per * c + N + it.nt;
          sc.meta[c] = {it.t0, it.row0, nrows, it.h * d.G, (int)((f_end - 1) / per), it.s, 0, 0};
        }
        tc_fence_before();
        if (!pair) named_bar_sync(1, 256);     // both groups have read the states and both O
        N += n;
      }
    } while (more());
  } else if constexpr (FP8) {
    // ------------------------------------------------------------------ E4M3 codes -> bf16 tiles
    regs_dec<C::REGS_LOW>();
    int k = 0;
    bool ok = true;
    do {
      const int cnt = plan[3];
      for (int i = 0; i < cnt && ok; ++i) {
        const Piece& it = pieces[i];
        const int j1 = it.j0 + it.n;
        for (int j = it.j0; j < j1 && ok; ++j) {
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
            for (int y = tid - 384; y < TOK * VEC; y += 128) {
              int row, v;
              widen_place<VEC>(y, row, v);
              uint4 w = *reinterpret_cast<const uint4*>(src + row * D + v * 16);
              if (x && part && !key_seen(it, base + row)) w = make_uint4(0, 0, 0, 0);
              widen16(w, dst + row * 128, TOK * 128, row, v);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(&raw_empty[rs]);
              mbar_arrive(&kv_full[s]);
            }
          }
        }
      }
    } while (more());
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
    if (lane == 0 && *abort_flag) set_error(err, KVS_ERR_TIMEOUT);
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
  constexpr int E = D / 32;
  const int row = mt.row0 + r;
  const size_t orow = (size_t)(mt.t0 + div_g(d, row)) * d.Hq + mt.head0 + row - div_g(d, row) * d.G, at = orow * D + lane * E;
  const float2 ml0 = lane < n ? sc.ml[place(lane)] : make_float2(-INFINITY, 0.f);
  // the earlier call's row, on its way while the parts are joined
  const bool has_prev = o.prev_out && mt.seq >= o.prev_req[0] && mt.seq < o.prev_req[o.n_prev];
  float prev[E];
#pragma unroll
  for (int e = 0; e < E; ++e) prev[e] = has_prev ? o.prev_out[at + e] : 0.f;
  float M = ml0.x;
  for (int i = lane + 32; i < n; i += 32) M = fmaxf(M, sc.ml[place(i)].x);
#pragma unroll
  for (int w = 16; w; w >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, w));
  float l = 0.f;
  float acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  for (int i0 = 0; i0 < n; i0 += 32) {
    float w = 0.f;
    if (i0 + lane < n) {
      const float2 v = i0 == 0 ? ml0 : sc.ml[place(i0 + lane)];
      w = v.x == -INFINITY ? 0.f : ex2(v.x - M);
      l += w * v.y;
    }
    const int cnt = min(32, n - i0);
#pragma unroll 8
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
  const RowOut ro = row_out(o, has_prev, orow, M, l, d.v_scale);
#pragma unroll
  for (int e = 0; e < E; ++e) {
    acc[e] *= ro.w_new;
    if (has_prev && ro.w_prev > 0.f) acc[e] += ro.w_prev * prev[e];
  }
#pragma unroll
  for (int e = 0; e < E; e += 2) {
    if (o.part_out) *reinterpret_cast<float2*>(o.part_out + at + e) = make_float2(acc[e], acc[e + 1]);
    else *reinterpret_cast<uint32_t*>(o.out + at + e) = pack_bf16x2(acc[e], acc[e + 1]);
  }
  if (lane == 0) row_lse(o, orow, ro.lse2);
}

template <int D, bool FP8>
cudaError_t launch(const PoolDims& d, const CUtensorMap* tm, const __nv_bfloat16* q, long long q_stride,
                   const PoolSeqs& seqs, const PoolAttnOut& o, void* scratch, unsigned* err, cudaStream_t s) {
  using C = Cfg<D, FP8>;
  auto kern = pool_attn_kernel<D, FP8>;
  cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void*>(kern), MAX_SMEM);
  if (e != cudaSuccess) return e;
  CUtensorMap tmQ;
  if (!make_pool_q_map(&tmQ, d, q, q_stride, seqs.n_tok)) return cudaErrorInvalidValue;
  const Split sp = {device_sm_count(), 2};
  launch_pdl(kern, dim3(sp.n_cta), dim3(C::THREADS), C::OFF_TAB + 4 * (seqs.n_seq + 1) + 1024, s, tm[0], tm[1], tmQ, d, seqs, o,
             scratch, sp, err);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // an item has at most two row tiles, and no more rows than the call
  return launch_pool_merge(d, o, scratch, sp.n_cta, (int)std::min<long long>(2 * d.rt, (long long)seqs.n_tok * d.G), s);
}

}  // namespace pa
}  // namespace

cudaError_t launch_pool_merge(const PoolDims& d, const PoolAttnOut& o, void* scratch, int n_cta, int rows, cudaStream_t s) {
  using namespace pa;
  const dim3 grid(n_cta, (rows + kMergeWarps - 1) / kMergeWarps);
  if (d.d == 128) launch_pdl(pool_merge_kernel<128>, grid, dim3(kMergeWarps * 32), 0, s, d, o, scratch, n_cta);
  else launch_pdl(pool_merge_kernel<64>, grid, dim3(kMergeWarps * 32), 0, s, d, o, scratch, n_cta);
  return cudaGetLastError();
}

size_t pool_attn_scratch_bytes(const PoolDims& d) {
  const size_t n = device_sm_count();
  return n * (sizeof(pdev::Meta) + 512 * (sizeof(float2) + (size_t)d.d * 4));
}

cudaError_t launch_pool_attn(const PoolDims& d, const unsigned char*, const unsigned char*, const CUtensorMap* tm,
                             const __nv_bfloat16* q, long long q_stride, const PoolSeqs& seqs, const PoolAttnOut& o,
                             void* scratch, unsigned* err, cudaStream_t s, int* n_launched) {
  using namespace pa;
  *n_launched = 2;
  // Few rows per (sequence, head), on average: they take the products' column side.  24 sequences of 8192 (1024) tokens, d 128,
  // few against many: bf16 4 rows 142 against 154 us (36 against 45), 32 rows 148 : 158 (44 : 48), 64 rows, in two
  // blocks or in one of 64 columns, 160 : 161 (56 : 50) at best; E4M3 4 rows 93 : 218 (29 : 50), 32 rows 132 : 221 (56 : 54),
  // 48 rows 232 : 222 (83 : 54).  These are equal sequences.  An average hides a mixed batch: 31 single tokens and a chunk of
  // 512 behind 8192 tokens each, 32 heads over 8, take 250 us in one call and 253 in a call each in bf16, but 387 : 235 with E4M3, and
  // 127 single tokens with a chunk of 900 behind 8192 take 750 : 728 and 1235 : 546.
  const long long rows = ((long long)seqs.n_tok * d.G + seqs.n_seq - 1) / seqs.n_seq;
  if (rows <= 32) return launch_pool_decode(d, tm, q, q_stride, seqs, o, (int)rows, scratch, err, s, n_launched);
  if (d.d == 128)
    return d.fp8 ? launch<128, true>(d, tm, q, q_stride, seqs, o, scratch, err, s)
                 : launch<128, false>(d, tm, q, q_stride, seqs, o, scratch, err, s);
  return d.fp8 ? launch<64, true>(d, tm, q, q_stride, seqs, o, scratch, err, s)
               : launch<64, false>(d, tm, q, q_stride, seqs, o, scratch, err, s);
}

}  // namespace kvs
