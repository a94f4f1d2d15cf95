// Device-resident pools: the softmax weight that each key receives, on the 5th-generation tensor cores.
//
//   w[t] = sum over the rows that see key t of 2^(S[t][row] scale log2 e - lse2[row]),   S = K Q^T
// The keys take the product's M side (tensor-memory lanes), the rows its columns, so one thread owns a key and sums its
// weights in registers: no exchange between threads, no atomics, the same order every time.  The log-sum-exps come
// from the attention call before.
//
// An item is 256 keys of a (request, kv head), a tile of 128 per group of 4 warps; it meets the row tiles that see
// one of its keys (T = 128 / G query tokens, T * G rows).  The row tiles of all items form one sequence that is cut
// into equal ranges, one per CTA (one per SM), as in the attention kernel; the sums of an item that a cut splits are
// joined in CTA order by the merge kernel.  Both the keys and the rows stream through rings, so a call of single
// tokens (one row tile per item) is bound by the keys' bytes and a prompt by the products and exponentials.
// A tile's sum joins the running sum with its rounding error kept (two-sum): a key of a long prompt receives 10^5
// terms.
//
// Roles: warp 0 brings K tiles, warp 1 issues the products, warp 2 brings Q tiles (tensor loads), warp 3 their
// log-sum-exps; warps 4-11 sum; with E4M3 pools warps 12-15 widen the codes.  Waits are bounded (KVS_ERR_TIMEOUT).
#include <algorithm>

#include "kvs_pool_dev.cuh"

namespace kvs {

namespace {
namespace pw {

using namespace pdev;

constexpr int KEYS = 2 * TOK;      // keys per item
constexpr int LSE_STAGES = 4;

struct Meta {
  int s, h, k0, c1, on, pad[3];
};

// Scratch: meta [n_cta]; sums [n_cta][2][256].
struct Scratch {
  Meta* meta;
  float* sum;
};
__host__ __device__ inline Scratch scratch_of(void* p, int n_cta) {
  Scratch s;
  s.meta = static_cast<Meta*>(p);
  s.sum = reinterpret_cast<float*>(s.meta + n_cta);
  return s;
}

template <int D, bool FP8>
struct Cfg {
  static constexpr int CHUNKS = D / 64;
  static constexpr int TILE = TOK * D * 2;                             // 128 bf16 rows of K or Q
  static constexpr int CODES = TOK * D;
  static constexpr int THREADS = FP8 ? 512 : 384;
  static constexpr int QS = 2;                                         // Q tiles in flight
  static constexpr int STAGING = FP8 ? 3 : 0;
  static constexpr int KS = FP8 ? 3 : 4;                               // bf16 K tiles
  static constexpr int OFF_K = QS * TILE;
  static constexpr int OFF_STG = OFF_K + KS * TILE;
  static constexpr int OFF_LSE = OFF_STG + STAGING * CODES;
  static constexpr int OFF_BAR = OFF_LSE + LSE_STAGES * TOK * 4;
  static constexpr int OFF_PIECES = OFF_BAR + 512;
  static constexpr int OFF_WS = OFF_PIECES + kPieces * 64;             // the scans' words
  static constexpr int OFF_TAB = OFF_WS + 512;
  static_assert(OFF_TAB + 4 * (kPoolMaxReq + 1) + 1024 <= MAX_SMEM, "shared memory plan");
};

// A CTA's piece of an item: keys [k0, k0 + 256) of head h of request s against n of the item's row tiles from
// rt0 + j0 on.
struct __align__(16) Piece {
  int s, h, t0, R, p0, len;
  int k0, rt0, nt, j0, n;
  int pad[5];
};
static_assert(sizeof(Piece) == 64, "smem plan");

// Row tiles that see one of the keys [k0, k0 + 256) of a request.
__device__ __forceinline__ void item_tiles(const PoolSeqs& q, int T, const SeqInfo& r, int kp, Piece& it) {
  it.t0 = r.t0;
  it.len = r.len;
  it.p0 = r.len - (r.t1 - r.t0);
  it.R = r.t1 - r.t0;
  it.k0 = kp * KEYS;
  const int k1 = min(it.len, it.k0 + KEYS);
  const int i_min = max(0, it.k0 - it.p0);
  int i_end = it.R;
  if (q.window && it.k0 >= q.n_sink) i_end = (int)min((long long)i_end, (long long)k1 - 1 + q.window - it.p0);
  it.rt0 = i_min / T;
  it.nt = i_end > i_min ? (i_end - 1) / T - it.rt0 + 1 : 0;
}

__device__ __forceinline__ Piece item_at(const PoolDims& d, const PoolSeqs& q, const int* tab, int T, int i, unsigned* err) {
  int lo = 0, hi = q.n_seq;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (tab[mid] <= i) lo = mid; else hi = mid;
  }
  Piece it;
  it.s = lo;
  const SeqInfo r = pool_seq(d, q, lo, err);
  const int local = i - tab[lo], kp = local / d.Hkv;
  it.h = local - kp * d.Hkv;
  item_tiles(q, T, r, kp, it);
  return it;
}

template <int D, bool FP8>
__global__ void __launch_bounds__(Cfg<D, FP8>::THREADS, 1)
    pool_weight_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmQ, PoolDims d,
                       PoolSeqs seqs, const float* __restrict__ lse2, float* __restrict__ weight, void* scratch, int n_cta,
                       unsigned* err) {
  using C = Cfg<D, FP8>;
  constexpr int NW = C::THREADS / 32, KS = C::KS, QS = C::QS;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* kring = smem + C::OFF_K;
  unsigned char* stg = smem + C::OFF_STG;
  float* lse_s = reinterpret_cast<float*>(smem + C::OFF_LSE);          // [LSE_STAGES][128]
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* k_full = bars;               // [4]
  uint64_t* k_empty = bars + 4;          // [4]
  uint64_t* raw_full = bars + 8;         // [4]
  uint64_t* raw_empty = bars + 12;       // [4]
  uint64_t* q_full = bars + 16;          // [2]
  uint64_t* q_empty = bars + 18;         // [2]
  uint64_t* l_full = bars + 20;          // [4]
  uint64_t* l_empty = bars + 24;         // [4]
  uint64_t* s_full = bars + 28;          // [group][buffer]
  uint64_t* s_empty = bars + 32;         // [group][buffer]
  uint64_t* drained = bars + 36;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 37);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* plan = reinterpret_cast<volatile int*>(tmem_slot + 2);
  const Piece* pieces = reinterpret_cast<const Piece*>(smem + C::OFF_PIECES);
  int* tab = reinterpret_cast<int*>(smem + C::OFF_TAB);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c = blockIdx.x;
  const int T = TOK / d.G, rows = T * d.G;      // query tokens and rows of a full row tile

  if (tid == 0) {
    for (int i = 0; i < 4; ++i) {
      mbar_init(&k_full[i], FP8 ? 4 : 1);
      mbar_init(&k_empty[i], 1);
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_empty[i], 4);
      mbar_init(&l_full[i], 1);
      mbar_init(&l_empty[i], 8);
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
    }
    mbar_init(drained, 1);
    *abort_flag = 0;
    plan[0] = plan[1] = plan[2] = 0;
    mbar_fence_init();
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmQ);
  }
  if (warp == 1) tmem_alloc(tmem_slot, 512);
  kvs_pdl_entry();

  // ------------------------------------------------------------------ the CTA's range of row tiles
  {
    long long* ws = reinterpret_cast<long long*>(smem + C::OFF_WS);
    const int per_s = (seqs.n_seq + C::THREADS - 1) / C::THREADS;
    const int s0 = min(seqs.n_seq, tid * per_s), s1 = min(seqs.n_seq, s0 + per_s);
    auto seq_work = [&](int s, int* items) {
      const SeqInfo r = pool_seq(d, seqs, s, err);
      const int n_kp = r.t1 > r.t0 ? (r.len + KEYS - 1) / KEYS : 0;
      *items = n_kp * d.Hkv;
      long long v = 0;
      if (r.t1 - r.t0 <= T && !seqs.window) {
        v = n_kp;                               // one row tile sees every key
      } else {
        for (int kp = 0; kp < n_kp; ++kp) {
          Piece it;
          item_tiles(seqs, T, r, kp, it);
          v += it.nt;
        }
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
    const Scan r = block_scan(mine, tiles, ws, NW);
    int at = r.n;
    for (int s = s0; s < s1; ++s) {
      tab[s] = at;
      if (s + 1 < s1) {
        seq_work(s, &n1);
        at += n1;
      }
    }
    if (tid == 0) tab[seqs.n_seq] = r.n_all;
    const long long per = (r.v_all + n_cta - 1) / n_cta;
    const long long f0 = per * c, f1 = min(r.v_all, f0 + per);
    if (f0 < f1 && f0 >= r.v && f0 < r.v + tiles) {
      long long f = r.v;
      int p = -1, j = 0;
      for (int s = s0; s < s1 && p < 0; ++s) {
        const long long v = s1 - s0 == 1 ? v1 : seq_work(s, &n1);
        if (f0 >= f + v) {
          f += v;
          continue;
        }
        const SeqInfo q1 = pool_seq(d, seqs, s, err);
        int kp = 0;
        if (q1.t1 - q1.t0 <= T && !seqs.window) {
          kp = (int)((f0 - f) / d.Hkv);
          f += (long long)kp * d.Hkv;
        }
        for (; p < 0; ++kp) {
          Piece it;
          item_tiles(seqs, T, q1, kp, it);
          const long long w = (long long)it.nt * d.Hkv;
          if (f0 < f + w) {
            const int h = (int)((f0 - f) / it.nt);
            p = tab[s] + kp * d.Hkv + h;
            j = (int)(f0 - f - (long long)h * it.nt);
          }
          f += w;
        }
      }
      plan[0] = p;
      plan[1] = j;
      plan[2] = (int)(f1 - f0);
    }
    if (tid == 0) {
      plan[4] = r.n_all;
      plan[5] = (int)per;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = (uint32_t)uniform((int)*tmem_slot);
  const uint64_t timeout_ns = (uint64_t)d.timeout_us * 1000ull;
  auto wait = [&](uint64_t* bar, unsigned parity) { return bounded_wait(bar, parity, timeout_ns, abort_flag); };
  // Plans the next kPieces pieces (warp 0, a lane per item); items that no row sees are passed over.
  auto plan_pieces = [&]() {
    int pos = plan[0], j0 = plan[1], left = plan[2], cnt = 0;
    const int n_items = plan[4];
    while (cnt <= kPieces - 32 && left > 0 && pos < n_items) {
      Piece it;
      it.nt = 0;
      if (pos + lane < n_items) it = item_at(d, seqs, tab, T, pos + lane, err);
      it.j0 = lane == 0 ? j0 : 0;
      const long long w = it.nt - it.j0;
      long long incl = w;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      it.n = (int)max(0ll, min(w, left - (incl - w)));
      const unsigned m = __ballot_sync(0xffffffffu, it.n > 0);
      if (it.n > 0) const_cast<Piece*>(pieces)[cnt + __popc(m & ((1u << lane) - 1))] = it;
      const long long all = __shfl_sync(0xffffffffu, incl, 31);
      left = (int)max(0ll, left - all);
      pos += 32;
      cnt += __popc(m);
      j0 = 0;
    }
    __syncwarp();
    if (lane == 0) {
      plan[0] = pos;
      plan[1] = 0;
      plan[2] = pos < n_items ? left : 0;
      plan[3] = cnt;
    }
  };
  if (warp == 0) plan_pieces();
  __syncthreads();
  auto more = [&]() {
    const int l = plan[2];
    __syncthreads();
    if (l <= 0) return false;
    if (warp == 0) plan_pieces();
    __syncthreads();
    return true;
  };
  const Scratch sc = scratch_of(scratch, n_cta);

  if (warp == 0) {
    // ------------------------------------------------------------------ K tiles, a lane per block
    constexpr int BOXES = FP8 ? 1 : C::CHUNKS;
    constexpr int SLOTS = FP8 ? C::STAGING : KS;
    uint64_t* full = FP8 ? raw_full : k_full;
    uint64_t* empty = FP8 ? raw_empty : k_empty;
    const int pages = TOK >> d.log2bs;
    const int box_bytes = d.bs * (FP8 ? D : 128);
    int k = 0;
    bool ok = true;
    do {
      const int cnt = plan[3];
      for (int i = 0; i < cnt && ok; ++i) {
        const Piece it = pieces[i];
        const int* table = seqs.table + (size_t)it.s * d.nb_max;
        for (int g = 0; g < 2 && it.k0 + g * TOK < it.len; ++g, ++k) {
          int row = -1;
          const int b0 = it.k0 + g * TOK + (lane << d.log2bs);
          if (lane < pages && b0 < it.len) {
            const int slot = table[b0 >> d.log2bs];
            // a block outside every window may have no slot; its keys are not summed
            if (slot >= 0 && slot < d.n_slots) row = (slot * d.Hkv + it.h) * d.bs;
          }
          const int n_load = __popc(__ballot_sync(0xffffffffu, row >= 0));
          const int s = k % SLOTS;
          ok = k < SLOTS || __all_sync(0xffffffffu, wait(&empty[s], ((k / SLOTS) & 1) ^ 1));
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(&full[s], (unsigned)(n_load * BOXES * box_bytes));
          __syncwarp();
          if (row >= 0) {
            unsigned char* dst = FP8 ? stg + s * C::CODES + lane * box_bytes : kring + s * C::TILE + lane * box_bytes;
#pragma unroll
            for (int b = 0; b < BOXES; ++b) tma_load_2d(dst + b * (TOK * 128), &tmK, b * 64, row, &full[s]);
          }
        }
      }
    } while (more());
    __syncwarp();
    for (int i = max(0, k - SLOTS); i < k; ++i) mbar_wait(&full[i % SLOTS], (i / SLOTS) & 1, kDrainTimeoutNs);
  } else if (warp == 1) {
    // ------------------------------------------------------------------ products
    const uint64_t dq0 = smem_desc_sw128(smem_u32(smem)), dk0 = smem_desc_sw128(smem_u32(kring));
    int k = 0, J = 0, ops0 = 0, ops1 = 0;
    bool ok = true;
    do {
      const int cnt = uniform(plan[3]);
      for (int i = 0; i < cnt && ok; ++i) {
        const int n = uniform(pieces[i].n), groups = uniform(pieces[i].k0 + TOK < pieces[i].len ? 2 : 1);
        const int tile0 = uniform(pieces[i].rt0 + pieces[i].j0), R = uniform(pieces[i].R);
        for (int g = 0; g < groups && ok; ++g) ok = __all_sync(0xffffffffu, wait(&k_full[(k + g) % KS], ((k + g) / KS) & 1));
        for (int j = 0; j < n && ok; ++j, ++J) {
          const int s = J % QS;
          ok = __all_sync(0xffffffffu, wait(&q_full[s], (J / QS) & 1));
          const int nr = min(T, R - (tile0 + j) * T) * d.G;
          const uint32_t idesc = idesc_bf16_f32(128, (nr + 15) & ~15);
          for (int g = 0; g < groups && ok; ++g) {
            const int op = g ? ops1++ : ops0++, b = g * 2 + (op & 1);
            if (op >= 2) ok = __all_sync(0xffffffffu, wait(&s_empty[b], ((op >> 1) - 1) & 1));
            if (!ok) break;
            tc_fence_after();
            const uint64_t da = dk0 + (uint64_t)((((k + g) % KS) * C::TILE) >> 4), db = dq0 + (uint64_t)((s * C::TILE) >> 4);
            if (elect_one()) {
#pragma unroll
              for (int k16 = 0; k16 < D / 16; ++k16) {
                const uint64_t off = (uint64_t)(((k16 >> 2) * (TOK * 128) + (k16 & 3) * 32) >> 4);
                tc_mma_f16(tmem + b * 128, da + off, db + off, idesc, k16 != 0);
              }
              tc_commit(&s_full[b]);
              if (g == groups - 1) tc_commit(&q_empty[s]);
              if (j == n - 1) tc_commit(&k_empty[(k + g) % KS]);
            }
          }
        }
        k += groups;
      }
      __syncwarp();
    } while (more());
    if (elect_one()) tc_commit(drained);
    mbar_wait(drained, 0, kDrainTimeoutNs);
    __syncwarp();
  } else if (warp == 2) {
    // ------------------------------------------------------------------ Q tiles: T tokens x G heads x 64 dims a load
    int J = 0;
    bool ok = true;
    do {
      const int cnt = plan[3];
      if (lane == 0) {
        for (int i = 0; i < cnt && ok; ++i) {
          const Piece& it = pieces[i];
          for (int j = 0; j < it.n; ++j, ++J) {
            const int s = J % QS;
            if (J >= QS && !wait(&q_empty[s], ((J / QS) & 1) ^ 1)) { ok = false; break; }
            mbar_arrive_expect_tx(&q_full[s], (unsigned)(C::CHUNKS * rows * 128));
#pragma unroll
            for (int b = 0; b < C::CHUNKS; ++b)
              tma_load_3d(smem + s * C::TILE + b * (TOK * 128), &tmQ, b * 64, it.h * d.G, it.t0 + (it.rt0 + it.j0 + j) * T,
                          &q_full[s]);
          }
        }
      }
      __syncwarp();
    } while (more());
    if (lane == 0)
      for (int i = max(0, J - QS); i < J; ++i) mbar_wait(&q_full[i % QS], (i / QS) & 1, kDrainTimeoutNs);
    __syncwarp();
  } else if (warp == 3) {
    // ------------------------------------------------------------------ the rows' log-sum-exps
    int J = 0;
    bool ok = true;
    do {
      const int cnt = plan[3];
      for (int i = 0; i < cnt && ok; ++i) {
        const Piece& it = pieces[i];
        const int n = it.n;
        for (int j = 0; j < n; ++j, ++J) {
          const int s = J % LSE_STAGES;
          const int tok0 = (it.rt0 + it.j0 + j) * T, nr = min(T, it.R - tok0) * d.G;
          float v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int row = e * 32 + lane;
            v[e] = -INFINITY;                      // (negated) a row that is not there weighs nothing
            if (row < nr) {
              const int tok = div_g(d, row);
              v[e] = -lse2[(size_t)(it.t0 + tok0 + tok) * d.Hq + it.h * d.G + row - tok * d.G];
              if (v[e] == INFINITY) v[e] = -INFINITY;   // nor does one that sees no key
            }
          }
          ok = J < LSE_STAGES || __all_sync(0xffffffffu, wait(&l_empty[s], ((J / LSE_STAGES) & 1) ^ 1));
          if (!ok) break;
#pragma unroll
          for (int e = 0; e < 4; ++e) lse_s[s * TOK + e * 32 + lane] = v[e];
          __syncwarp();
          if (lane == 0) mbar_arrive(&l_full[s]);
        }
      }
    } while (more());
  } else if (warp < 12) {
    // ------------------------------------------------------------------ sums: a key per thread
    const int g = (warp - 4) >> 2, lr = (warp & 3) * 32 + lane;
    const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16) + g * 256;
    const float sl2 = d.scale * d.k_scale * kLog2e;
    const uint64_t sl22 = pack2(sl2, sl2);
    int J = 0, ops = 0, N = 0;
    if (warp == 4 && lane == 0) sc.meta[c].on = 0;
    do {
      const int cnt = plan[3];
      for (int i = 0; i < cnt; ++i) {
        const Piece it = pieces[i];
        const int n = it.n, k0 = it.k0 + g * TOK, t = k0 + lr, len = it.len, p0 = it.p0;
        const bool act = k0 < len;               // the group's tile holds keys
        const int k1 = min(len, k0 + TOK) - 1;   // its last key
        const bool far = seqs.window && k1 >= seqs.n_sink;       // the window hides its keys from rows far behind them
        float sum = 0.f, low = 0.f;
        int tok0 = (it.rt0 + it.j0) * T;
        for (int j = 0; j < n; ++j, ++J, tok0 += T) {
          const int ls = J % LSE_STAGES;
          wait(&l_full[ls], (J / LSE_STAGES) & 1);
          if (act) {
            const int b = ops & 1;
            const int n_tok = min(T, it.R - tok0), nr = n_tok * d.G;
            const int pa = p0 + tok0, pb = pa + n_tok - 1;           // positions of the tile's first and last token
            const bool whole = k1 <= pa && n_tok == T && !(far && pb - k0 >= seqs.window);
            // the columns this key is seen by: rows from its own position on, to the window's end
            int ca = 0, cb = nr;
            if (!whole) {
              if (t > pa) ca = min(t - pa, T) * d.G;
              if (seqs.window && t >= seqs.n_sink) cb = min(cb, min(max(t - pa + seqs.window, 0), T) * d.G);
              if (t >= len) cb = 0;
            }
            wait(&s_full[g * 2 + b], (ops >> 1) & 1);
            tc_fence_after();
            uint64_t a0 = 0, a1 = 0;
            const uint32_t ts = trow + b * 128;
            const float4* lv = reinterpret_cast<const float4*>(lse_s + ls * TOK);
            auto chunk = [&](int c0, bool part) {        // 32 columns
              float x[32];
              tmem_ld32(ts + c0, x);
              if (part) {
                const uint32_t vis = bits_below(cb - c0) & ~bits_below(ca - c0);
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  if (!(vis & (1u << e))) x[e] = -INFINITY;
              }
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float4 z = lv[c0 / 4 + e];
                float p, q2;
                unpack2(fma2(pack2(x[4 * e], x[4 * e + 1]), sl22, pack2(z.x, z.y)), p, q2);
                a0 = add2(a0, pack2(ex2(p), ex2(q2)));
                unpack2(fma2(pack2(x[4 * e + 2], x[4 * e + 3]), sl22, pack2(z.z, z.w)), p, q2);
                a1 = add2(a1, pack2(ex2(p), ex2(q2)));
              }
            };
            if (whole && rows == TOK) {
#pragma unroll
              for (int c0 = 0; c0 < TOK; c0 += 32) chunk(c0, false);
            } else {
#pragma unroll 1
              for (int c0 = 0; c0 < nr; c0 += 32) chunk(c0, true);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s_empty[g * 2 + b]);
            ++ops;
            float x, y;
            unpack2(add2(a0, a1), x, y);
            // sum + low += x + y, the rounding error kept in low
            const float v = x + y, nsum = __fadd_rn(sum, v), bv = __fsub_rn(nsum, sum);
            low = __fadd_rn(low, __fadd_rn(__fsub_rn(sum, __fsub_rn(nsum, bv)), __fsub_rn(v, bv)));
            sum = nsum;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&l_empty[ls]);
        }
        sum += low;
        const bool begun = it.j0 == 0, done = it.j0 + n == it.nt;
        if (begun && done) {
          if (act && t < len) {
            float* w = weight + ((size_t)it.s * d.Hkv + it.h) * d.max_ctx + t;
            *w = t >= p0 ? sum : *w + sum;
          }
        } else {
          sc.sum[((size_t)c * 2 + (begun ? 1 : 0)) * KEYS + g * TOK + lr] = sum;
          if (begun && warp == 4 && lane == 0) {
            const int per = plan[5];
            const long long f_end = (long long)per * c + N + it.nt;
            sc.meta[c] = {it.s, it.h, it.k0, (int)((f_end - 1) / per), 1, {0, 0, 0}};
          }
        }
        N += n;
      }
    } while (more());
  } else if constexpr (FP8) {
    // ------------------------------------------------------------------ E4M3 codes -> bf16 tiles
    int k = 0;
    bool ok = true;
    do {
      const int cnt = plan[3];
      for (int i = 0; i < cnt && ok; ++i) {
        const Piece& it = pieces[i];
        for (int g = 0; g < 2 && it.k0 + g * TOK < it.len; ++g, ++k) {
          const int s = k % KS, rs = k % C::STAGING;
          ok = __all_sync(0xffffffffu, wait(&raw_full[rs], (k / C::STAGING) & 1) &&
                                           (k < KS || wait(&k_empty[s], ((k / KS) & 1) ^ 1)));
          if (!ok) break;
          constexpr int VEC = D / 16;
#pragma unroll 4
          for (int y = tid - 384; y < TOK * VEC; y += 128) {
            int row, v;
            widen_place<VEC>(y, row, v);
            widen16(*reinterpret_cast<const uint4*>(stg + rs * C::CODES + row * D + v * 16), kring + s * C::TILE + row * 128,
                    TOK * 128, row, v);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&raw_empty[rs]);
            mbar_arrive(&k_full[s]);
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

// Sums of the items that a range's end cut: block c the item that CTA c began, a thread per key.
__global__ void __launch_bounds__(KEYS)
    pool_weight_merge_kernel(PoolDims d, PoolSeqs seqs, float* __restrict__ weight, void* scratch, int n_cta, unsigned* err) {
  kvs_pdl_entry();
  const Scratch sc = scratch_of(scratch, n_cta);
  const int c = blockIdx.x;
  const Meta m = sc.meta[c];
  if (!m.on) return;
  const SeqInfo r = pool_seq(d, seqs, m.s, err);
  const int t = m.k0 + threadIdx.x;
  if (t >= r.len) return;
  float sum = sc.sum[((size_t)c * 2 + 1) * KEYS + threadIdx.x];
  for (int i = c + 1; i <= m.c1; ++i) sum += sc.sum[((size_t)i * 2) * KEYS + threadIdx.x];
  float* w = weight + ((size_t)m.s * d.Hkv + m.h) * d.max_ctx + t;
  *w = t >= r.len - (r.t1 - r.t0) ? sum : *w + sum;
}

template <int D, bool FP8>
cudaError_t launch(const PoolDims& d, const CUtensorMap* tm, const CUtensorMap& tmQ, const PoolSeqs& seqs, const float* lse2,
                   float* weight, void* scratch, unsigned* err, cudaStream_t s) {
  using C = Cfg<D, FP8>;
  auto kern = pool_weight_kernel<D, FP8>;
  cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void*>(kern), MAX_SMEM);
  if (e != cudaSuccess) return e;
  const int n = device_sm_count();
  launch_pdl(kern, dim3(n), dim3(C::THREADS), C::OFF_TAB + 4 * (seqs.n_seq + 1) + 1024, s, tm[0], tmQ, d, seqs, lse2, weight,
             scratch, n, err);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  launch_pdl(pool_weight_merge_kernel, dim3(n), dim3(KEYS), 0, s, d, seqs, weight, scratch, n, err);
  return cudaGetLastError();
}

}  // namespace pw
}  // namespace

size_t pool_weight_scratch_bytes() { return (size_t)device_sm_count() * (sizeof(pw::Meta) + 2 * pw::KEYS * sizeof(float)); }

cudaError_t launch_pool_weight(const PoolDims& d, const CUtensorMap* tm, const __nv_bfloat16* q, long long q_stride,
                               const PoolSeqs& seqs, const float* lse2, float* weight, void* scratch, unsigned* err,
                               cudaStream_t s, int* n_launched) {
  CUtensorMap tmQ;
  *n_launched = 0;
  if (!make_pool_q_map(&tmQ, d, q, q_stride, seqs.n_tok)) return cudaErrorInvalidValue;
  *n_launched = 2;
  if (d.d == 128)
    return d.fp8 ? pw::launch<128, true>(d, tm, tmQ, seqs, lse2, weight, scratch, err, s)
                 : pw::launch<128, false>(d, tm, tmQ, seqs, lse2, weight, scratch, err, s);
  return d.fp8 ? pw::launch<64, true>(d, tm, tmQ, seqs, lse2, weight, scratch, err, s)
               : pw::launch<64, false>(d, tm, tmQ, seqs, lse2, weight, scratch, err, s);
}

}  // namespace kvs
