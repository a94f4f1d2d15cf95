// Device-resident pools: attention for few rows per (sequence, kv head) on the 5th-generation tensor cores.
//
// A decode step has G rows (a group's heads) per K/V row, drafts a few times that: far fewer than a product's 128-row
// side.  Here the tokens take that side, and the rows the columns (NB = 8, 16 or 32 of them):
//   S^T = K Q^T (128 tokens x NB),   P^T = 2^(S^T scale log2 e - m) in bf16,   O^T += V^T P^T (d x NB)
// so that a tile of 128 tokens costs two products of 16 x (d / 16 + 8) small columns, and the 128 threads of the softmax
// share its exponentials, a token each: the kernel is bound by the K/V bytes.  V is read as the product's A operand with
// the dims contiguous (MN-major) from the same tile that the tensor loads bring; P^T goes through shared memory.
// S^T and O^T are in tensor memory.  m (per row) is the maximum of the first tile that the row sees and is set anew
// only when a weight passes 2^40; the sums l are kept per thread and reduced at a piece's end.
//
// The tiles of all items form one sequence that is cut into equal ranges, one per CTA (one per SM), as in the kernel
// for many rows; the same merge kernel joins the items that a cut splits.  (Joining them in the last of an item's CTAs to
// finish saves a launch, but its fences and serial loads cost more: 16.7 us against 13.3 for one request's token, both before
// one warp planned a CTA's work, which took the form kept to 12.0.)
//
// E4M3 pools.  S^T is a product of the K codes as they are with Q in E4M3: a row of Q is scaled by a power of two, so that its
// largest element lies in [2^7, 2^8), and split into two codes, q = hi + lo, whose products add up.  The 8 bits of a bf16
// significand are 4 + 4, so the split is exact for elements down to 2^-9 of the row's largest; below that it is off by
// at most 2^-10, half a step of E4M3's subnormals, which is at most 2^-17 of the largest.  V is widened to bf16
// tiles, whose product takes P^T in bf16 (P has no room in E4M3: its rounding would be an output's error).  Widening K as
// well was the kernel's bound: 2650 clocks a tile, 87 us for 32 requests' windows of 4096 tokens, against 67.
//
// Roles: warp 0 brings K/V tiles, warp 1 issues the products (S^T of a tile before O^T of the tile before it, across
// pieces), warp 2 loads Q, warps 4-7 are the softmax; with E4M3 pools warps 8-11 and 12-15 widen V's codes, every other
// tile each.
// Value rows that no row of the item sees are zeroed before their product.  All waits are bounded.
#include <algorithm>

#include "kvs_pool_sched.cuh"

namespace kvs {

namespace {
namespace pd {

using namespace pdev;

constexpr float kMaxArg = 40.f;     // log2 of the largest weight before m is set anew

template <int D, bool FP8, int NB>
struct Cfg {
  static constexpr int CHUNKS = D / 64;
  static constexpr int ML = 3 * 1024;
  static constexpr int NQ = NB < 16 ? 16 : NB;                // columns of the products
  static constexpr int QCHUNK = NQ * 128;                     // 64 dims of the rows (bf16)
  static constexpr int QBUF = CHUNKS * QCHUNK;                // one item's Q: bf16, or its high codes and behind them its low ones
  // P^T: 128 tokens of 128 bytes, 64 columns of room: two tiles of up to 32 columns side by side
  static constexpr int PBYTES = TOK * 128;
  static constexpr int PSTEP = 64;                            // bytes from one tile's P^T to the other's
  static constexpr int TILE = TOK * D * 2;
  static constexpr int CODES = TOK * D;
  static constexpr int THREADS = FP8 ? 512 : 256;
  static constexpr int ROOM = MAX_SMEM - ML - 512 - 2048 - 4 * (kPoolMaxReq + 1) - kPieces * 64 - 2 * QBUF - PBYTES;
  // bf16 tiles, K's and V's in turn; with E4M3 pools three of V's, three of K's codes, and two of V's codes, each for the warps
  // that widen it
  static constexpr int STAGES = FP8 ? 3 : ROOM / TILE > 8 ? 8 : ROOM / TILE;
  static constexpr int OFF_P = 2 * QBUF;
  static constexpr int OFF_RING = OFF_P + PBYTES;
  static constexpr int OFF_K = OFF_RING + STAGES * TILE;      // codes of K (E4M3)
  static constexpr int OFF_RAW = OFF_K + (FP8 ? 3 * CODES : 0);      // codes of V (E4M3)
  static constexpr int OFF_ML = OFF_RAW + (FP8 ? 2 * CODES : 0);     // m, l, factors, scales of Q, maxima by warp, places
  static constexpr int OFF_BAR = OFF_ML + ML;
  static constexpr int OFF_PIECES = OFF_BAR + 512;
  static constexpr int OFF_TAB = OFF_PIECES + kPieces * 64;
  static int bytes(int n_seq) { return OFF_TAB + 4 * (n_seq + 1) + 1024; }
  static_assert(STAGES >= 3 && OFF_TAB + 4 * (kPoolMaxReq + 1) + 1024 <= MAX_SMEM, "shared memory plan");
};

// Products of E4M3 codes, both operands K-major with rows of D bytes: swizzled by as many bytes, 8-row groups 8 D bytes apart.
template <int D, bool ACC>
__device__ __forceinline__ void mma_codes(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc) {
  constexpr uint32_t kHi = (8u * D >> 4) | (1u << 14) | ((D == 128 ? 2u : 4u) << 29);
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 x, y;\n setp.ne.u32 p, %5, 0;\n mov.b64 x, {%1, %3};\n mov.b64 y, {%2, %3};\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %4, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(kHi), "r"(idesc), "n"(ACC ? 1 : 0)
      : "memory");
}
// byte offset of 16-byte chunk c of row r in such an operand
template <int D>
__device__ __forceinline__ int code_chunk(int r, int c) { return r * D + ((c ^ (D == 128 ? r & 7 : (r >> 1) & 3)) << 4); }
// two fp32 that two E4M3 codes stand for (exact)
__device__ __forceinline__ float2 e4m3x2_to_f32(uint32_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)codes));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}
template <int D, bool FP8, int NB>
__global__ void __launch_bounds__(Cfg<D, FP8, NB>::THREADS, 1)
    pool_decode_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, PoolDims d,
                       const __nv_bfloat16* __restrict__ q, long long q_stride, PoolSeqs seqs, PoolAttnOut o, void* scratch,
                       Split sp, unsigned* err) {
  using C = Cfg<D, FP8, NB>;
  constexpr int S = C::STAGES, NQ = C::NQ;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* ring = smem + C::OFF_RING;
  unsigned char* raw = smem + C::OFF_RAW;
  float* m_s = reinterpret_cast<float*>(smem + C::OFF_ML);            // [64] m of the rows, -inf: none yet
  float* l_s = m_s + 64;                                              // [64] sums at a piece's end
  float* f_s = m_s + 128;                                             // [64] factors of a new m
  float* nm_s = m_s + 192;                                            // [64] -m as the exponents take it: 0 without m, -inf without a row
  // [4][32] softmax scale and scale of a row's codes of Q (E4M3), by piece: the softmax is done with piece p when Q of piece p + 4 is
  // loaded, as S^T of piece p + 2 has been issued over the tile before last
  float* q_s = m_s + 640;
  float* x_s = m_s + 256;                                             // [4][64] maxima or sums by warp
  long long* at_s = reinterpret_cast<long long*>(m_s + 512);          // [64] places of the output rows
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* kv_full = bars;             // [8] (E4M3: V's widened tiles)
  uint64_t* kv_empty = bars + 8;        // [8]
  uint64_t* k_full = bars + 16;         // [4] K's codes
  uint64_t* k_empty = bars + 20;        // [4]
  uint64_t* raw_full = bars + 24;       // [2] V's codes
  uint64_t* raw_empty = bars + 26;      // [2]
  uint64_t* s_full = bars + 32;         // [2]
  uint64_t* s_free = bars + 34;         // [2]
  uint64_t* p_full = bars + 36;         // [2]
  uint64_t* p_free = bars + 38;         // [2]
  uint64_t* q_full = bars + 40;         // [2] by piece
  uint64_t* q_free = bars + 42;         // [2]
  uint64_t* o_full = bars + 44;         // [2]
  uint64_t* o_free = bars + 46;         // [2]
  uint64_t* vote = bars + 48;           // [2] every softmax warp has looked at its weights' size
  uint64_t* drained = bars + 50;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 51);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* plan = reinterpret_cast<volatile int*>(tmem_slot + 2);
  volatile int* outgrown = reinterpret_cast<volatile int*>(tmem_slot + 8);     // [2] a weight has outgrown m
  Piece* pieces = reinterpret_cast<Piece*>(smem + C::OFF_PIECES);
  int* tab = reinterpret_cast<int*>(smem + C::OFF_TAB);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c = blockIdx.x;

  if (tid == 0) {
    for (int i = 0; i < 8; ++i) {
      mbar_init(&kv_full[i], FP8 ? 4 : 1);
      mbar_init(&kv_empty[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_free[i], 4);
      mbar_init(&p_full[i], 4);
      mbar_init(&p_free[i], 1);
      mbar_init(&q_full[i], 1);
      mbar_init(&q_free[i], 1);
      mbar_init(&o_full[i], 1);
      mbar_init(&o_free[i], 4);
      mbar_init(&vote[i], 4);
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_empty[i], 4);
      outgrown[i] = 0;
    }
    mbar_init(drained, 1);
    *abort_flag = 0;
    plan[0] = plan[1] = plan[2] = 0;
    mbar_fence_init();
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == 1) tmem_alloc(tmem_slot, 256);
  kvs_pdl_entry();
  volatile int* few = reinterpret_cast<volatile int*>(tmem_slot + 10);      // warp 0 has planned alone
  if (seqs.n_seq <= 32) {
    if (warp == 0) {
      const bool done = plan_few(d, seqs, NB, tab, plan, pieces, sp, c, err);
      if (lane == 0) *few = done;
    }
    tc_fence_before();
    __syncthreads();
  }
  const bool planned = seqs.n_seq <= 32 && *few;
  if (!planned) {
    cta_range<false, C::THREADS>(d, seqs, NB, tab, reinterpret_cast<long long*>(x_s), plan, sp, c, err);
    tc_fence_before();
    __syncthreads();
  }
  tc_fence_after();
  const uint32_t tmem = (uint32_t)uniform((int)*tmem_slot);
  const uint64_t timeout_ns = (uint64_t)d.timeout_us * 1000ull;
  const Scratch sc = scratch_of(scratch, sp.n_cta);
  auto wait = [&](uint64_t* bar, unsigned parity) { return bounded_wait(bar, parity, timeout_ns, abort_flag); };
  if (!planned) {
    if (warp == 0) plan_pieces<false>(d, seqs, NB, tab, plan, pieces, sp.n_cta, err);
    __syncthreads();
  }
  // Between two lists of pieces (long calls only): every role is done with the old one.
  auto more = [&]() {
    const int l = plan[2];
    __syncthreads();
    if (l <= 0) return false;
    if (warp == 0) plan_pieces<false>(d, seqs, NB, tab, plan, pieces, sp.n_cta, err);
    __syncthreads();
    return true;
  };
  // tensor memory: S^T [2 buffers], O^T [2, by piece]
  auto tS = [&](int b) { return tmem + b * 64; };
  auto tO = [&](int b) { return tmem + 128 + b * 64; };

  if (warp == 0) {
    // ------------------------------------------------------------------ K/V tiles: a lane per block of a tile
    constexpr int BOXES = FP8 ? 1 : C::CHUNKS;
    const int pages = TOK >> d.log2bs;
    const int box_bytes = d.bs * (FP8 ? D : 128);
    int k = 0, s = 0, T = 0;          // tiles of the ring (bf16: K's and V's in turn; E4M3: K's), V's code tiles
    unsigned par = 1;                 // of the slot's last release (the first round is free)
    bool ok = true;
    do {
      const int cnt = plan[3];
      for (int i = 0; i < cnt && ok; ++i) {
        const Piece it = pieces[i];
        const int* table = seqs.table + (size_t)it.s * d.nb_max;
        // the slot of this lane's block of tile j, fetched a tile ahead; -1: no row sees the block
        auto look = [&](int j) {
          if (lane >= pages || j >= it.j0 + it.n) return -1;
          const int b0 = tile_base(it, j) + (lane << d.log2bs), b1 = b0 + d.bs;
          return b0 < it.first || (b0 < it.hi && b1 > it.lo) ? table[b0 >> d.log2bs] : -2;
        };
        int slot = look(it.j0);
        for (int j = it.j0; j < it.j0 + it.n && ok; ++j) {
          const int now = slot;
          slot = look(j + 1);
          int row = -1;
          if (lane < pages && now != -2) {
            if (now < 0 || now >= d.n_slots) set_error(err, KVS_ERR_BAD_INDEX);
            else row = (now * d.Hkv + it.h) * d.bs;
          }
          const int n_load = __popc(__ballot_sync(0xffffffffu, row >= 0));
          for (int x = 0; x < 2; ++x) {
            const bool raw_v = FP8 && x;
            if (raw_v) ok = T < 2 || __all_sync(0xffffffffu, wait(&raw_empty[T & 1], ((T >> 1) - 1) & 1));
            else ok = k < S || __all_sync(0xffffffffu, wait(FP8 ? &k_empty[s] : &kv_empty[s], par));
            if (!ok) break;
            uint64_t* full = raw_v ? &raw_full[T & 1] : FP8 ? &k_full[s] : &kv_full[s];
            if (lane == 0) mbar_arrive_expect_tx(full, (unsigned)(n_load * BOXES * box_bytes));
            __syncwarp();
            if (row >= 0) {
              unsigned char* dst = (raw_v ? raw + (T & 1) * C::CODES : FP8 ? smem + C::OFF_K + s * C::CODES : ring + s * C::TILE) + lane * box_bytes;
#pragma unroll
              for (int b = 0; b < BOXES; ++b) tma_load_2d(dst + b * (TOK * 128), x ? &tmV : &tmK, b * 64, row, full);
            }
            if (raw_v) {
              ++T;
            } else {
              ++k;
              if (++s == S) {
                s = 0;
                par ^= 1;
              }
            }
          }
        }
      }
    } while (more());
    __syncwarp();
    // no tensor load may still be writing this CTA's shared memory when it exits
    for (int i = max(0, k - S); i < k; ++i) mbar_wait(FP8 ? &k_full[i % S] : &kv_full[i % S], (i / S) & 1, kDrainTimeoutNs);
    if (FP8)
      for (int i = max(0, T - 2); i < T; ++i) mbar_wait(&raw_full[i & 1], (i >> 1) & 1, kDrainTimeoutNs);
  } else if (warp == 1) {
    // ------------------------------------------------------------------ products
    // S^T: bf16, or E4M3 codes (whose format fields are 0)
    const uint32_t id_s = idesc_bf16_f32(128, NQ) & ~(FP8 ? (1u << 7) | (1u << 10) : 0u);
    const uint32_t id_o = idesc_bf16_f32(128, NQ) | (1u << 15) | (1u << 16);      // V and P^T are read MN-major
    const uint32_t aq = smem_u32(smem) >> 4, ap = smem_u32(smem + C::OFF_P) >> 4, ar = smem_u32(ring) >> 4;
    const uint32_t ak = smem_u32(smem + C::OFF_K) >> 4;
    // V^T: 64-dim blocks of a tile 16 KiB apart; at d = 64 the second block gives lanes 64-127, which are not used: it is
    // read 1 KiB on, still inside this CTA's shared memory
    constexpr uint32_t kV = (uint32_t)((D == 128 ? TOK * 128 : 1024) >> 4) << 16;
    int T = 0, pc = 0;                // tile and piece of the next S^T
    int To = 0, po = 0;               // and of the next O^T
    bool ok = true;
    do {
      const int cnt = plan[3];
      if (elect_one()) {
        int is = 0, js = 0, io = 0, jo = 0;      // the same within this list of pieces
        int n_s = cnt > 0 ? pieces[0].n : 0, n_o = n_s;
        auto s_t = [&]() {
          const int n = FP8 ? T : 2 * T, s = n % S, b = T & 1;      // K's place in the ring
          if (js == 0) ok = wait(&q_full[pc & 1], (pc >> 1) & 1);
          ok = ok && wait(FP8 ? &k_full[s] : &kv_full[s], (n / S) & 1) && (T < 2 || wait(&s_free[b], ((T >> 1) - 1) & 1));
          if (!ok) return;
          tc_fence_after();
          const uint32_t q0 = aq + (pc & 1) * (C::QBUF >> 4), t = tS(b);
          if constexpr (FP8) {
            const uint32_t k0 = ak + s * (C::CODES >> 4);
            mma_codes<D, false>(t, k0, q0, id_s);
#pragma unroll
            for (int k32 = 1; k32 < D / 32; ++k32) mma_codes<D, true>(t, k0 + k32 * 2, q0 + k32 * 2, id_s);
#pragma unroll
            for (int k32 = 0; k32 < D / 32; ++k32) mma_codes<D, true>(t, k0 + k32 * 2, q0 + (NQ * D >> 4) + k32 * 2, id_s);
          } else {
            const uint32_t k0 = ar + s * (C::TILE >> 4);
            mma_ss<false>(t, k0, q0, id_s);
#pragma unroll
            for (int k16 = 1; k16 < D / 16; ++k16)
              mma_ss<true>(t, k0 + (((k16 >> 2) * (TOK * 128) + (k16 & 3) * 32) >> 4),
                           q0 + (((k16 >> 2) * C::QCHUNK + (k16 & 3) * 32) >> 4), id_s);
          }
          tc_commit(&s_full[b]);
          tc_commit(FP8 ? &k_empty[s] : &kv_empty[s]);
          ++T;
          if (++js == n_s) {
            tc_commit(&q_free[pc & 1]);
            js = 0;
            ++pc;
            if (++is < cnt) n_s = pieces[is].n;
          }
        };
        auto o_t = [&]() {
          const int n = FP8 ? To : 2 * To + 1, s = n % S, b = To & 1;      // V's
          ok = wait(&kv_full[s], (n / S) & 1) && wait(&p_full[b], (To >> 1) & 1) &&
               (jo > 0 || po < 2 || wait(&o_free[po & 1], ((po >> 1) - 1) & 1));
          if (!ok) return;
          tc_fence_after();
          const uint32_t v0 = (ar + s * (C::TILE >> 4)) | kV, p0 = ap + b * (C::PSTEP >> 4), t = tO(po & 1);
          if (jo == 0) mma_ss<false>(t, v0, p0, id_o);
          else mma_ss<true>(t, v0, p0, id_o);
#pragma unroll
          for (int kk = 1; kk < TOK / 16; ++kk) mma_ss<true>(t, v0 + kk * (2048 >> 4), p0 + kk * (2048 >> 4), id_o);
          tc_commit(&kv_empty[s]);
          tc_commit(&p_free[b]);
          ++To;
          if (++jo == n_o) {
            tc_commit(&o_full[po & 1]);
            jo = 0;
            ++po;
            if (++io < cnt) n_o = pieces[io].n;
          }
        };
        while (ok && is < cnt) {
          s_t();
          if (ok && T - To == 2) o_t();
        }
        while (ok && To < T) o_t();
      }
      __syncwarp();
    } while (more());
    // every product issued here has finished before the tensor memory is released
    if (elect_one()) tc_commit(drained);
    mbar_wait(drained, 0, kDrainTimeoutNs);
    __syncwarp();
  } else if (warp == 2) {
    // ------------------------------------------------------------------ Q, a piece ahead
    int piece = 0;
    bool ok = true;
    do {
      const int cnt = plan[3];
      for (int i = 0; i < cnt && ok; ++i, ++piece) {
        const Piece& it = pieces[i];
        const int nrows = it.nrows, row0 = it.row0, t0 = it.t0, h = it.h;
        ok = piece < 2 || __all_sync(0xffffffffu, wait(&q_free[piece & 1], ((piece >> 1) - 1) & 1));
        if (!ok) break;
        constexpr int VEC = D / 8;       // 16-byte vectors of a row
        unsigned char* buf = smem + (piece & 1) * C::QBUF;
        if constexpr (!FP8) {
          for (int x = lane; x < nrows * VEC; x += 32) {
            const int r = x / VEC, v = x - r * VEC, row = row0 + r, tok = div_g(d, row), g = row - tok * d.G;
            cp_async16(buf + (v >> 3) * C::QCHUNK + r * 128 + (((v & 7) ^ (r & 7)) << 4),
                       q + (t0 + tok) * q_stride + (h * d.G + g) * D + v * 8, 16);
          }
          cp_async_commit();
          cp_async_wait_all();
        } else {
          // a step takes 32 / VEC rows, a vector per lane; up to 8 steps' loads in flight
          const float sl2 = d.scale * d.k_scale * kLog2e;
          constexpr int PER = 32 / VEC, DEEP = NB / PER < 8 ? NB / PER : 8;
          const int sub = lane / VEC, v = lane % VEC;
#pragma unroll 1
          for (int r0 = 0; r0 < nrows; r0 += PER * DEEP) {
            uint4 w[DEEP];
#pragma unroll
            for (int e = 0; e < DEEP; ++e) {
              const int r = r0 + e * PER + sub, row = row0 + r, tok = div_g(d, row), g = row - tok * d.G;
              w[e] = r < nrows ? *reinterpret_cast<const uint4*>(q + (t0 + tok) * q_stride + (h * d.G + g) * D + v * 8)
                               : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int e = 0; e < DEEP; ++e) {
              const int r = r0 + e * PER + sub;
              const uint32_t u[4] = {w[e].x, w[e].y, w[e].z, w[e].w};
              // the exponent field of the row's largest element (as bit patterns: magnitudes of bf16 compare as integers)
              uint32_t top = 0;
#pragma unroll
              for (int i2 = 0; i2 < 4; ++i2) top = max(top, max(u[i2] & 0x7fffu, (u[i2] >> 16) & 0x7fffu));
#pragma unroll
              for (int o2 = VEC / 2; o2; o2 >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o2));
              const uint32_t field = min(max(top >> 7, 8u), 254u);
              const float mult = __uint_as_float((261u - field) << 23);       // 2^7 / 2^exponent
              uint32_t hi[2] = {0, 0}, lo[2] = {0, 0};
#pragma unroll
              for (int i2 = 0; i2 < 4; ++i2) {
                const float a = bf16_lo(u[i2]) * mult, b2 = bf16_hi(u[i2]) * mult;
                const uint32_t c2 = f32x2_to_e4m3x2(a, b2);
                const float2 back = e4m3x2_to_f32(c2);
                hi[i2 >> 1] |= c2 << ((i2 & 1) * 16);
                lo[i2 >> 1] |= (uint32_t)f32x2_to_e4m3x2(a - back.x, b2 - back.y) << ((i2 & 1) * 16);
              }
              if (r < nrows) {
                *reinterpret_cast<uint2*>(buf + code_chunk<D>(r, v >> 1) + (v & 1) * 8) = make_uint2(hi[0], hi[1]);
                *reinterpret_cast<uint2*>(buf + NQ * D + code_chunk<D>(r, v >> 1) + (v & 1) * 8) = make_uint2(lo[0], lo[1]);
                // (infinities and NaN in a row leave it NaN)
                if (v == 0) q_s[(piece & 3) * 32 + r] = top >= 0x7f80u ? __int_as_float(0x7fc00000) : __uint_as_float((field - 7u) << 23) * sl2;
              }
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[piece & 1]);
      }
    } while (more());
    cp_async_wait_all();
  } else if (warp == 3) {
    while (more()) {
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------------ softmax and output: a token (a dim) per thread
    const int lr = (warp - 4) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp - 4) * 32) << 16;
    const float sl2 = d.scale * d.k_scale * kLog2e;
    int T = 0, piece = 0;
    if (lr == 0) sc.meta[c].nrows = 0;
    do {
      const int cnt = plan[3];
      for (int i = 0; i < cnt; ++i, ++piece) {
        const Piece it = pieces[i];
        const int n = it.n, nrows = it.nrows;
        // tiles of the span that every row sees as a whole
        int hi_all = it.len, lo_all = 0;
        const int pa = it.p0 + div_g(d, it.row0), pa_row = it.row0 - div_g(d, it.row0) * d.G;   // first row's position, head
        if (seqs.causal) {
          hi_all = max(0, pa + 1);
          lo_all = seqs.window ? max(0, it.p0 + div_g(d, it.row0 + nrows - 1) - seqs.window + 1) : 0;
        }
        const int ja = it.ns + (lo_all + TOK - 1) / TOK - it.lo_tile - it.j0;
        const unsigned n_whole = (unsigned)max(0, it.ns + hi_all / TOK - it.lo_tile - it.j0 - ja);
        const float* qs = q_s + (piece & 3) * 32;
        float l[NB];
#pragma unroll
        for (int x = 0; x < NB; ++x) l[x] = 0.f;
        if (lr < 64) m_s[lr] = -INFINITY;
        bool fresh = true;                       // some row has no m yet
        for (int j = 0; j < n; ++j, ++T) {
          const int b = T & 1;
          wait(&s_full[b], (T >> 1) & 1);
          // P's room is free as well: the product of the tile before last was issued before this S^T, whose commit covers it
          tc_fence_after();
          const bool edge = (unsigned)(j - ja) >= n_whole;
          const int base = tile_base(it, it.j0 + j), t = base + lr;
          uint32_t vis = 0xffffffffu;
          if (edge) {
            // the columns that see this token: rows from its own position on, to the window's end
            int ca = 0, cb = t < it.len ? nrows : 0;
            if (seqs.causal) {
              if (t > pa) ca = min(t - pa, NB + 1) * d.G - pa_row;
              if (seqs.window && t >= seqs.n_sink) cb = min(cb, min(max(t - pa + seqs.window, 0), NB + 1) * d.G - pa_row);
            }
            vis = bits_below(cb) & ~bits_below(ca);
            if (!FP8 && !tile_whole(it, base)) {
              // value rows that no row of the item sees
              const int slot = 2 * T + 1;
              wait(&kv_full[slot % S], (slot / S) & 1);
              zero_rows(ring + (slot % S) * C::TILE, C::CHUNKS, lr & ~31, __ballot_sync(0xffffffffu, !key_seen(it, t)));
            }
          }
          unsigned char* pr = smem + C::OFF_P + lr * 128;
          const int pc0 = b * 4;        // its first 16-byte chunk
          float x[NB];
#pragma unroll 1
          for (bool first = true;; first = false) {
            if constexpr (NB == 8) tmem_ld8(tS(b) + lanes, x);
            else if constexpr (NB == 16) tmem_ld16(tS(b) + lanes, x);
            else tmem_ld32(tS(b) + lanes, x);
            if (edge) {
#pragma unroll
              for (int y = 0; y < NB; ++y)
                if (!(vis & (1u << y))) x[y] = -INFINITY;
            }
            const bool set = fresh || !first;
            if (set) {
              // m of rows that have none, or that a weight has outgrown: the tile's maximum.  All 128 threads.
#pragma unroll
              for (int y = 0; y < NB; ++y) {
                const float v = warp_max(x[y]);
                if (lane == 0) x_s[(warp - 4) * 64 + y] = v;
              }
              named_bar_sync(2, 128);
              if (lr < NB) {
                const float v = fmaxf(fmaxf(x_s[lr], x_s[64 + lr]), fmaxf(x_s[128 + lr], x_s[192 + lr])) * (FP8 ? qs[lr] : sl2), m = m_s[lr];
                const float m2 = m == -INFINITY || v > m + kMaxArg ? v : m;
                f_s[lr] = m == -INFINITY || m2 == m ? 1.f : ex2(m - m2);
                m_s[lr] = m2;
                nm_s[lr] = lr >= nrows ? -INFINITY : m2 == -INFINITY ? 0.f : -m2;
              }
              if (lr == 0) outgrown[b] = 0;
              named_bar_sync(2, 128);
              bool none = false, scaled = false;
#pragma unroll
              for (int y = 0; y < NB; ++y) {
                none = none || (y < nrows && m_s[y] == -INFINITY);
                scaled = scaled || (y < nrows && f_s[y] != 1.f);
              }
              fresh = none;
              if (scaled) {
                // O^T holds the earlier tiles' products: all must have finished
                if (T >= 1) wait(&p_free[b ^ 1], ((T - 1) >> 1) & 1);
                tc_fence_after();
#pragma unroll
                for (int y = 0; y < NB; ++y) l[y] *= f_s[y];
                if (j > 0) {
#pragma unroll 1
                  for (int y = 0; y < NQ; y += 16) {
                    float ov[16];
                    uint32_t ow[16];
                    tmem_ld16(tO(piece & 1) + lanes + y, ov);
#pragma unroll
                    for (int e = 0; e < 16; ++e) ow[e] = __float_as_uint(y + e < nrows ? ov[e] * f_s[y + e] : ov[e]);
                    tmem_st16(tO(piece & 1) + lanes + y, ow);
                  }
                  tmem_wait_st();
                }
              }
            }
            float top = -INFINITY;
#pragma unroll
            for (int y = 0; y < NB; y += 4) {
              const float4 z = *reinterpret_cast<const float4*>(nm_s + y);
              const float4 f = FP8 ? *reinterpret_cast<const float4*>(qs + y) : make_float4(sl2, sl2, sl2, sl2);
              unpack2(fma2(pack2(x[y], x[y + 1]), pack2(f.x, f.y), pack2(z.x, z.y)), x[y], x[y + 1]);
              unpack2(fma2(pack2(x[y + 2], x[y + 3]), pack2(f.z, f.w), pack2(z.z, z.w)), x[y + 2], x[y + 3]);
              // (columns without a row: -inf, or NaN, which a maximum skips)
              top = max3(max3(top, x[y], x[y + 1]), x[y + 2], x[y + 3]);
            }
            // a weight that outgrows m: the warps vote (once a tile, so that the phases follow T), and all do the tile
            // again with a new m
            if (first) {
              const bool big = !set && __any_sync(0xffffffffu, top > kMaxArg);
              if (lane == 0) {
                if (big) outgrown[b] = 1;
                mbar_arrive(&vote[b]);
              }
            }
#pragma unroll
            for (int y = 0; y < NB; y += 8) {
#pragma unroll
              for (int e = 0; e < 8; ++e) x[y + e] = ex2(x[y + e]);
              *reinterpret_cast<uint4*>(pr + (((pc0 + (y >> 3)) ^ (lr & 7)) << 4)) =
                  make_uint4(pack_bf16x2(x[y], x[y + 1]), pack_bf16x2(x[y + 2], x[y + 3]), pack_bf16x2(x[y + 4], x[y + 5]),
                             pack_bf16x2(x[y + 6], x[y + 7]));
            }
            fence_proxy_async_smem();
            if (set) break;
            wait(&vote[b], (T >> 1) & 1);
            if (!outgrown[b]) break;
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&s_free[b]);
            mbar_arrive(&p_full[b]);
          }
#pragma unroll
          for (int y = 0; y < NB; y += 2) unpack2(add2(pack2(l[y], l[y + 1]), pack2(x[y], x[y + 1])), l[y], l[y + 1]);
        }
        // -------------------------------------------------------------- the piece's end: sums, then O^T, a dim per thread
#pragma unroll
        for (int y = 0; y < NB; ++y) {
#pragma unroll
          for (int w = 16; w; w >>= 1) l[y] += __shfl_xor_sync(0xffffffffu, l[y], w);
          if (lane == 0) x_s[(warp - 4) * 64 + y] = l[y];
        }
        named_bar_sync(2, 128);
        const bool begun = it.j0 == 0, done = it.j0 + n == it.nt, whole = begun && done;
        const bool has_prev = o.prev_out && it.s >= o.prev_req[0] && it.s < o.prev_req[o.n_prev];
        if (lr < nrows) {
          const float lsum = (x_s[lr] + x_s[64 + lr]) + (x_s[128 + lr] + x_s[192 + lr]);
          l_s[lr] = lsum;
          const int row = it.row0 + lr, tok = div_g(d, row);
          const size_t orow = (size_t)(it.t0 + tok) * d.Hq + it.h * d.G + row - tok * d.G;
          at_s[lr] = (long long)((whole ? orow : ((size_t)c * 2 + (begun ? 1 : 0)) * 256 + lr) * D);
          if (whole) {
            const RowOut ro = row_out(o, has_prev, orow, m_s[lr], lsum, d.v_scale);
            f_s[lr] = ro.w_new;
            x_s[lr] = ro.w_prev;
            row_lse(o, orow, ro.lse2);
          } else {
            sc.ml[((size_t)c * 2 + (begun ? 1 : 0)) * 256 + lr] = make_float2(m_s[lr], lsum);
          }
        }
        named_bar_sync(2, 128);
        wait(&o_full[piece & 1], (piece >> 1) & 1);
        tc_fence_after();
        if (D == 128 || warp < 6) {
#pragma unroll 1
          for (int y0 = 0; y0 < nrows; y0 += 8) {
            float v[8], z[8];
            tmem_ld8(tO(piece & 1) + lanes + y0, v);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              z[e] = whole && has_prev && y0 + e < nrows && x_s[y0 + e] > 0.f ? __ldg(o.prev_out + at_s[y0 + e] + lr) : 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int y = y0 + e;
              if (y >= nrows) break;
              if (!(l_s[y] > 0.f)) v[e] = 0.f;
              if (!whole) {
                sc.o[at_s[y] + lr] = v[e];
                continue;
              }
              const float r = v[e] * f_s[y] + (has_prev && x_s[y] > 0.f ? x_s[y] * z[e] : 0.f);
              if (o.part_out) o.part_out[at_s[y] + lr] = r;
              else o.out[at_s[y] + lr] = __float2bfloat16(r);
            }
          }
        }
        if (begun && !done && lr == 0) {
          // the item goes on in the next CTAs: up to the one that holds its last tile
          const int per = plan[5];
          const long long f_end = (long long)per * c + (T - n) + it.nt;
          sc.meta[c] = {it.t0, it.row0, nrows, it.h * d.G, (int)((f_end - 1) / per), it.s, 0, 0};
        }
        tc_fence_before();
        named_bar_sync(2, 128);          // sums and factors have been read
        if (lane == 0) mbar_arrive(&o_free[piece & 1]);
      }
    } while (more());
  } else if constexpr (FP8) {
    // ------------------------------------------------------------------ V's codes -> bf16 tiles: warps 8-11 and 12-15 in turn
    // Each four have a code tile of their own.  The ring's slots are shared; a wait for slot T % 3 never looks two phases
    // ahead, as these warps have waited for the product of tile T - 5 before.
    const int x = (warp - 8) >> 2, th = tid & 127;
    int T = 0;
    bool ok = true;
    do {
      const int cnt = plan[3];
      for (int i = 0; i < cnt && ok; ++i) {
        const Piece& it = pieces[i];
        const int j1 = it.j0 + it.n;
        for (int j = it.j0; j < j1 && ok; ++j, ++T) {
          if ((T & 1) != x) continue;
          ok = __all_sync(0xffffffffu, wait(&raw_full[x], (T >> 1) & 1));
          if (!ok) break;
          constexpr int VEC = D / 16, PER = TOK * VEC / 128;              // 16-code vectors of a row, of a thread
          const unsigned char* src = raw + x * C::CODES;
          uint4 w[PER];
#pragma unroll
          for (int e = 0; e < PER; ++e) {
            int row, v;
            widen_place<VEC>(th + e * 128, row, v);
            w[e] = *reinterpret_cast<const uint4*>(src + row * D + v * 16);
          }
          // the codes are in registers: the next ones may come (their load's latency is longer than the widening)
          __syncwarp();
          if (lane == 0) mbar_arrive(&raw_empty[x]);
          const int base = tile_base(it, j), s = T % S;
          if (!tile_whole(it, base)) {
#pragma unroll
            for (int e = 0; e < PER; ++e) {
              int row, v;
              widen_place<VEC>(th + e * 128, row, v);
              if (!key_seen(it, base + row)) w[e] = make_uint4(0, 0, 0, 0);
            }
          }
          ok = T < S || __all_sync(0xffffffffu, wait(&kv_empty[s], ((T / S) - 1) & 1));
          if (!ok) break;
          unsigned char* dst = ring + s * C::TILE;
#pragma unroll
          for (int e = 0; e < PER; ++e) {
            int row, v;
            widen_place<VEC>(th + e * 128, row, v);
            widen16(w[e], dst + row * 128, TOK * 128, row, v);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&kv_full[s]);
        }
      }
    } while (more());
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
    if (lane == 0 && *abort_flag) set_error(err, KVS_ERR_TIMEOUT);
  }
}

template <int D, bool FP8, int NB>
cudaError_t launch(const PoolDims& d, const CUtensorMap* tm, const __nv_bfloat16* q, long long q_stride,
                   const PoolSeqs& seqs, const PoolAttnOut& o, void* scratch, unsigned* err, cudaStream_t s, int* n_launched) {
  using C = Cfg<D, FP8, NB>;
  auto kern = pool_decode_kernel<D, FP8, NB>;
  cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void*>(kern), MAX_SMEM);
  if (e != cudaSuccess) return e;
  const Split sp = {device_sm_count(), 2};
  launch_pdl(kern, dim3(sp.n_cta), dim3(C::THREADS), C::bytes(seqs.n_seq), s, FP8 ? tm[2] : tm[0], tm[1], d, q, q_stride, seqs, o,
             scratch, sp, err);
  e = cudaGetLastError();
  *n_launched = 1;
  if (e != cudaSuccess) return e;
  *n_launched = 2;
  return launch_pool_merge(d, o, scratch, sp.n_cta, (int)std::min<long long>(NB, (long long)seqs.n_tok * d.G), s);
}

template <int D, bool FP8>
cudaError_t launch_nb(int nb, const PoolDims& d, const CUtensorMap* tm, const __nv_bfloat16* q, long long q_stride,
                      const PoolSeqs& seqs, const PoolAttnOut& o, void* scratch, unsigned* err, cudaStream_t s, int* n_launched) {
  if (nb <= 8) return launch<D, FP8, 8>(d, tm, q, q_stride, seqs, o, scratch, err, s, n_launched);
  if (nb <= 16) return launch<D, FP8, 16>(d, tm, q, q_stride, seqs, o, scratch, err, s, n_launched);
  return launch<D, FP8, 32>(d, tm, q, q_stride, seqs, o, scratch, err, s, n_launched);
}

}  // namespace pd
}  // namespace

cudaError_t launch_pool_decode(const PoolDims& d, const CUtensorMap* tm, const __nv_bfloat16* q, long long q_stride,
                               const PoolSeqs& seqs, const PoolAttnOut& o, int nb, void* scratch, unsigned* err,
                               cudaStream_t s, int* n_launched) {
  if (d.d == 128)
    return d.fp8 ? pd::launch_nb<128, true>(nb, d, tm, q, q_stride, seqs, o, scratch, err, s, n_launched)
                 : pd::launch_nb<128, false>(nb, d, tm, q, q_stride, seqs, o, scratch, err, s, n_launched);
  return d.fp8 ? pd::launch_nb<64, true>(nb, d, tm, q, q_stride, seqs, o, scratch, err, s, n_launched)
               : pd::launch_nb<64, false>(nb, d, tm, q, q_stride, seqs, o, scratch, err, s, n_launched);
}

}  // namespace kvs
