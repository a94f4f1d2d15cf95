// Norms and rotation of query and key rows, dense or into a pool, and the repositioning of cached keys.
//
// A head's d elements lie in d / 16 lanes, two chunks of 8 elements (16 bytes) each, chosen so that both elements of every
// rotated pair are in one lane: no exchange but the norm's sum.  Pair i of a row turns by pos * f_i.  The frequency is kept in
// turns, as an integer multiple of 2^-64: its product with any 32-bit position wraps around at whole turns by itself, exactly
// (fp32 products lose the angle beyond some thousand positions).  What is lost: the frequency's own rounding (2^-51 of it and
// 2^-64) times the position, and less than 2^-32 turns below the product's upper 32 bits.
#include <cuda_fp16.h>

#include <algorithm>

#include "kvs_ptx.cuh"
#include "kvs_rope.cuh"

namespace kvs {

namespace {

// cos and sin of m * f turns, two of them (two_pi: its sign is the angle's).  The product's upper word, a turn's fraction,
// becomes a float in [1, 2) by its upper 23 bits, rounded (a conversion would take the unit that the cosines need): off by
// 2^-24 turns, 2^-21.3.  The fast functions are off by 2^-21 for arguments in [-pi, pi].  Together 2^-20 at most, beside which the
// stored types' half steps are 2^-8 and 2^-4: the errors of results are the same as with exact cosines, and at most one E4M3
// code in 80,000, within 2^-21 of its row's largest value from a tie, is rounded to the other side.
constexpr float kTwoPi = 6.2831853f;
__device__ __forceinline__ float turn_bits(unsigned m, unsigned long long f) {      // 1.5 + the fraction's distance from whole turns
  const unsigned t = __umulhi(m, (unsigned)f) + (m * (unsigned)(f >> 32) + 0x80000100u);      // half a turn on, and half a step
  return __uint_as_float((t >> 9) | 0x3f800000u);
}
__device__ __forceinline__ void turn_cos_sin(unsigned m, float two_pi, unsigned long long f0, unsigned long long f1, float2& c, float2& s) {
  const float2 x = __fmul2_rn(__fadd2_rn(make_float2(turn_bits(m, f0), turn_bits(m, f1)), make_float2(-1.5f, -1.5f)), make_float2(two_pi, two_pi));
  c = make_float2(__cosf(x.x), __cosf(x.y));
  s = make_float2(__sinf(x.x), __sinf(x.y));
}
__device__ __forceinline__ unsigned magnitude(int pos) { return pos < 0 ? 0u - (unsigned)pos : (unsigned)pos; }

// The parameters by their address: lanes that read entries of their own take one load, where an indexed read of the constant
// bank is repeated for every lane (128 tokens of 12 steps 3.0 us that way, 2.45 by address; one token 1.83 and 1.65).
template <typename T>
__device__ __forceinline__ const T* by_address(const T& rd) {
  const T* p = &rd;
  asm volatile("" : "+l"(p));
  return p;
}

// Which elements are a pair: i and i + d / 2, i and i + rot / 2, or 2 i and 2 i + 1.
enum { kHalves, kPart, kAdjacent };

// What a lane holds of a row: chunks c0 and c1 (of 8 elements), and the pair of its j-th (a, b).
template <int D, int LAY>
struct LanePart {
  int c0, c1;
  __device__ __forceinline__ LanePart(int rot, int l) {
    const int n = rot / 16;
    c0 = l;
    c1 = l + D / 16;
    if (LAY == kPart && l < n) {
      c1 = l + n;
    } else if (LAY == kPart) {
      c0 = 2 * l;
      c1 = c0 + 1;
    }
  }
  // c1's distance, in chunks
  __device__ __forceinline__ int apart() const { return LAY == kPart ? c1 - c0 : D / 16; }
  __device__ __forceinline__ int pair(int j) const { return LAY == kAdjacent ? (j < 4 ? 4 * c0 + j : 4 * c1 + j - 4) : 8 * c0 + j; }
  // (the pair's number is past the rotated ones where the elements do not turn)
  __device__ __forceinline__ bool turns(int j, int rot) const { return LAY == kHalves || (LAY == kAdjacent ? pair(j) < rot / 2 : c0 < rot / 16); }
};

__device__ __forceinline__ uint32_t f32x2_to_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// A lane's pairs (a, b), two at a time: u = (a[2i], a[2i + 1]), v = (b[2i], b[2i + 1]).
struct Pairs {
  float2 u[4], v[4];
};
// ... of the elements x of its two chunks, and back
template <int LAY>
__device__ __forceinline__ Pairs to_pairs(const float (&x)[16]) {
  constexpr bool ADJ = LAY == kAdjacent;
  Pairs p;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    p.u[i] = ADJ ? make_float2(x[4 * i], x[4 * i + 2]) : make_float2(x[2 * i], x[2 * i + 1]);
    p.v[i] = ADJ ? make_float2(x[4 * i + 1], x[4 * i + 3]) : make_float2(x[8 + 2 * i], x[9 + 2 * i]);
  }
  return p;
}
template <int LAY>
__device__ __forceinline__ void from_pairs(const Pairs& p, float (&x)[16]) {
  constexpr bool ADJ = LAY == kAdjacent;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[ADJ ? 4 * i : 2 * i] = p.u[i].x;
    x[ADJ ? 4 * i + 2 : 2 * i + 1] = p.u[i].y;
    x[ADJ ? 4 * i + 1 : 8 + 2 * i] = p.v[i].x;
    x[ADJ ? 4 * i + 3 : 9 + 2 * i] = p.v[i].y;
  }
}

struct Raw {
  uint4 c0, c1;
};
__device__ __forceinline__ void unpack_bf16(const Raw& r, float (&x)[16]) {
  const uint32_t w[8] = {r.c0.x, r.c0.y, r.c0.z, r.c0.w, r.c1.x, r.c1.y, r.c1.z, r.c1.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[2 * i] = bf16_lo(w[i]);
    x[2 * i + 1] = bf16_hi(w[i]);
  }
}
__device__ __forceinline__ Raw pack_bf16(const float (&x)[16]) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = f32x2_to_bf16x2(x[2 * i], x[2 * i + 1]);
  return {make_uint4(w[0], w[1], w[2], w[3]), make_uint4(w[4], w[5], w[6], w[7])};
}
// Four E4M3 codes, rounded to nearest even, saturating
__device__ __forceinline__ uint32_t pack_e4m3x4(const float* x) {
  uint32_t r;
  asm("{.reg .b16 lo, hi;\n cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n mov.b32 %0, {lo, hi};}"
      : "=r"(r) : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]));
  return r;
}
__device__ __forceinline__ uint2 pack_e4m3(const float* x) { return make_uint2(pack_e4m3x4(x), pack_e4m3x4(x + 4)); }

enum { kDense, kPoolBf16, kPoolFp8 };

// What a warp does with rows of d elements, 32 / (d / 16) heads (a step) at a time.
template <int D, int LAY>
struct RowWarp {
  static constexpr int LPH = D / 16, HPW = 32 / LPH, NP = D / 64;
  const int lane, sub;
  const LanePart<D, LAY> at;
  const int rot;
  const float rot_scale, eps;
  // (a, b) -> (a cw + b sw, b dw + a ew): the rotation and the norm's weights
  float2 cw[4], sw[4], dw[4], ew[4];

  __device__ __forceinline__ RowWarp(const RopeParams<D / 2>& rd)
      : lane(threadIdx.x & 31), sub((threadIdx.x & 31) / LPH), at(rd.rot, (threadIdx.x & 31) % LPH), rot(rd.rot), rot_scale(rd.rot_scale), eps(rd.eps) {}

  // cos and sin of every pair of the row, by all lanes, to shared memory
  __device__ __forceinline__ void turns(const int (&pos)[NP], const unsigned long long (&freq)[NP], float2* turn) {
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      const float x = (turn_bits(magnitude(pos[j]), freq[j]) - 1.5f) * kTwoPi;
      const float scale = lane + 32 * j < rot / 2 ? rot_scale : 1.f;
      turn[lane + 32 * j] = make_float2(__cosf(x) * scale, __sinf(x) * (pos[j] < 0 ? -scale : scale));
    }
    __syncwarp();
  }
  struct Weights {
    float4 y[4];
  };
  __device__ __forceinline__ Weights weights(const float* norm) const {
    Weights w;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w.y[j] = norm ? __ldg(reinterpret_cast<const float4*>(norm) + (j < 2 ? 2 * at.c0 + j : 2 * at.c1 + j - 2)) : make_float4(1.f, 1.f, 1.f, 1.f);
    return w;
  }
  __device__ __forceinline__ void factors(const Weights& y, const float2* turn) {
    float x[16];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[4 * j] = y.y[j].x;
      x[4 * j + 1] = y.y[j].y;
      x[4 * j + 2] = y.y[j].z;
      x[4 * j + 3] = y.y[j].w;
    }
    const Pairs w = to_pairs<LAY>(x);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // the rotated pairs' numbers, or any unrotated pair's (there are as many pairs as elements that do not turn)
      const int n = LAY != kPart || at.turns(0, rot) ? at.pair(2 * i) : rot / 2;
      const float4 t = *reinterpret_cast<const float4*>(turn + n);      // cos, sin, cos, sin
      cw[i] = make_float2(t.x * w.u[i].x, t.z * w.u[i].y);
      sw[i] = make_float2(-t.y * w.v[i].x, -t.w * w.v[i].y);
      dw[i] = make_float2(t.x * w.v[i].x, t.z * w.v[i].y);
      ew[i] = make_float2(t.y * w.u[i].x, t.w * w.u[i].y);
    }
  }
  // the lane's part of a row, normed (if `norm`) and turned
  __device__ __forceinline__ void row(const Raw& r, bool norm, float (&x)[16]) const {
    unpack_bf16(r, x);
    Pairs p = to_pairs<LAY>(x);
    if (norm) {
      float2 sum = __ffma2_rn(p.v[0], p.v[0], __fmul2_rn(p.u[0], p.u[0]));
#pragma unroll
      for (int i = 1; i < 4; ++i) sum = __ffma2_rn(p.v[i], p.v[i], __ffma2_rn(p.u[i], p.u[i], sum));
      float s = sum.x + sum.y;
#pragma unroll
      for (int o = LPH / 2; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      const float inv = rsqrtf(s * (1.f / D) + eps);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        p.u[i] = __fmul2_rn(p.u[i], make_float2(inv, inv));
        p.v[i] = __fmul2_rn(p.v[i], make_float2(inv, inv));
      }
    }
    Pairs y;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y.u[i] = __ffma2_rn(p.v[i], sw[i], __fmul2_rn(p.u[i], cw[i]));
      y.v[i] = __ffma2_rn(p.u[i], ew[i], __fmul2_rn(p.v[i], dw[i]));
    }
    if (LAY != kHalves && rot != D) {       // an element that does not turn owes nothing to its partner, which may be infinite
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (!at.turns(2 * i, rot)) {
          y.u[i] = __fmul2_rn(p.u[i], cw[i]);
          y.v[i] = __fmul2_rn(p.v[i], dw[i]);
        }
    }
    from_pairs<LAY>(y, x);
  }
  __device__ __forceinline__ void store_bf16(void* to, const Raw& r) const {
    reinterpret_cast<uint4*>(to)[at.c0] = r.c0;
    reinterpret_cast<uint4*>(to)[at.c1] = r.c1;
  }
  // x / scale, rounded as the quantiser's division is.  With the reciprocal's rounding r at hand (0: scale is extreme) the quotient comes
  // from two corrections of x r by their exact remainders (Markstein, IBM J. Res. Dev. 34, 1990): the first is within a unit in the
  // last place, the second rounds correctly.  Quotients that saturate or become zero need none: the former may have no finite
  // remainder, the latter would lose their sign.  (16 divisions took 0.6 us of one token's 2.3.)
  __device__ __forceinline__ void store_e4m3(void* to, float (&x)[16], float scale, float r) const {
    if (r != 0.f) {
      const float2 rr = make_float2(r, r), ss = make_float2(-scale, -scale);
#pragma unroll
      for (int j = 0; j < 16; j += 2) {
        const float2 y = make_float2(x[j], x[j + 1]), q0 = __fmul2_rn(y, rr);
        const float2 q1 = __ffma2_rn(__ffma2_rn(q0, ss, y), rr, q0);
        const float2 q2 = __ffma2_rn(__ffma2_rn(q1, ss, y), rr, q1);
        x[j] = fabsf(q0.x) < 1024.f && fabsf(q0.x) > 0x1p-12f ? q2.x : q0.x;
        x[j + 1] = fabsf(q0.y) < 1024.f && fabsf(q0.y) > 0x1p-12f ? q2.y : q0.y;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j) x[j] = __fdiv_rn(x[j], scale);
    }
    reinterpret_cast<uint2*>(to)[at.c0] = pack_e4m3(x);
    reinterpret_cast<uint2*>(to)[at.c1] = pack_e4m3(x + 8);
  }
  __device__ __forceinline__ static const uint4* from(const RopeHeads& g, int tok, int h) {
    return reinterpret_cast<const uint4*>(g.src + tok * g.src_tok + h * g.src_head);
  }
  __device__ __forceinline__ static void* dense(const RopeHeads& g, int tok, int h) { return g.dst + tok * g.dst_tok + h * g.dst_head; }
};

// Where a token's K/V rows go: its row in head 0 of its slot.
struct PlaceRow {
  size_t row;
  bool there;
};
__device__ __forceinline__ PlaceRow place_row(const RopeRows& a, long long place) {
  PlaceRow p;
  p.there = place >= 0 && place < ((long long)a.n_slots << a.log2bs);
  if (place >= 0 && !p.there) set_error(a.err, KVS_ERR_BAD_INDEX);
  p.row = (size_t)(place >> a.log2bs) * a.k.n * a.bs + (place & (a.bs - 1));
  return p;
}

// Few tokens: a warp per step, everything it needs on its way at once.  One token of 32 + 2 x 8 heads into a bf16 pool: 1.65 us
// (3.3 with a loop over the token's steps), about the time of a launch.  From some 16 steps for each SM on, where the other
// kernel's warps have one each, its sharing of a token's angles wins: 128 tokens (1536 steps) 2.4 us here and 2.8 there, 256 3.7
// and 3.15; of 3 steps each, 512 tokens 2.0 and 2.3, 2048 4.1 and 3.6.
constexpr int kFewThreads = 128;
constexpr int kFewSteps = 16;      // steps for each SM, at most

template <int D, int LAY, int DST>
__global__ void __launch_bounds__(kFewThreads)
    rope_few_kernel(const __grid_constant__ RopeParams<D / 2> rd, const __grid_constant__ RopeRows a, int iq, int ik, int steps) {
  using W = RowWarp<D, LAY>;
  __shared__ __align__(16) float2 cos_sin[kFewThreads / 32][D / 2];
  W w(rd);
  float2* turn = cos_sin[threadIdx.x >> 5];
  unsigned long long freq[W::NP];
  int pos[W::NP];
  const auto* const rp = by_address(rd);
#pragma unroll
  for (int j = 0; j < W::NP; ++j) {
    freq[j] = rp->freq[w.lane + 32 * j];      // (past the rotated pairs: an angle of 0)
    pos[j] = rp->axis[w.lane + 32 * j];
  }
  const int item = blockIdx.x * (kFewThreads / 32) + (threadIdx.x >> 5), tok = item / steps, it = item - tok * steps;
  kvs_pdl_entry();
  if (tok >= a.n_tok) return;
  const bool is_q = it < iq, is_v = it >= iq + ik;
  long long place = -1;
  if (DST != kDense && !is_q) place = a.place[tok];
  const int h = (is_q ? it : is_v ? it - iq - ik : it - iq) * W::HPW + w.sub;
  const bool there = h < (is_q ? a.q.n : a.k.n);
  Raw raw = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
  if (there) {
    const uint4* src = is_q ? W::from(a.q, tok, h) : is_v ? W::from(a.v, tok, h) : W::from(a.k, tok, h);
    raw.c0 = __ldcs(src + w.at.c0);
    raw.c1 = __ldcs(src + w.at.c1);
  }
  if (DST != kDense && is_v) {
    const PlaceRow p = place_row(a, place);
    if (!there || !p.there) return;
    unsigned char* to = a.vpool + (p.row + (size_t)h * a.bs) * (DST == kPoolFp8 ? D : 2 * D);
    if (DST == kPoolFp8) {
      float x[16];
      unpack_bf16(raw, x);
      w.store_e4m3(to, x, a.v_scale, a.v_rcp);
    } else {
      w.store_bf16(to, raw);
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < W::NP; ++j) pos[j] = a.pos[pos[j] * a.pos_stride + tok];
  const float* norm = is_q ? a.q.norm : a.k.norm;
  const typename W::Weights weights = w.weights(norm);
  w.turns(pos, freq, turn);
  w.factors(weights, turn);
  float x[16];
  w.row(raw, norm != nullptr, x);
  if (DST == kDense || is_q) {
    if (there) w.store_bf16(is_q ? W::dense(a.q, tok, h) : W::dense(a.k, tok, h), pack_bf16(x));
    return;
  }
  const PlaceRow p = place_row(a, place);
  if (!there || !p.there) return;
  unsigned char* to = a.kpool + (p.row + (size_t)h * a.bs) * (DST == kPoolFp8 ? D : 2 * D);
  if (DST == kPoolFp8) w.store_e4m3(to, x, a.k_scale, a.k_rcp);
  else w.store_bf16(to, pack_bf16(x));
}

// Many tokens: the warps take whole tokens in turn, then equal runs of the steps left over.  The steps' rows come through a ring in
// shared memory, kStages - 1 steps ahead, in which every lane reads what it has copied itself.
//
// Bound by the rows' bytes, 3 KB on their way a warp; the norm's weights and the rotation are one set of factors, made once for
// a token's queries and once for its keys, so that a row costs 8 multiplications and 16 fused ones for 16 elements (in pairs).
// 16384 tokens of 32 + 2 x 8 heads of 128 into a bf16 pool: 66 us, 6.1 TB/s (59.3 at the rate of a copy).  Rows loaded into
// registers a step ahead took 83 us, three steps ahead 70; every warp at a run of its own (far from its neighbours') 70; 3 CTAs
// an SM with 80 registers 75.  11308 tokens of 28 + 4 heads, no norm: 31 us (27.3).
constexpr int kRopeThreads = 256;
constexpr int kStages = 4;
constexpr int kRopeCtas = 2;       // of an SM

__device__ __forceinline__ void cp_async16_at(uint32_t smem, const void* gmem, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;\n" ::"r"(smem), "l"(gmem), "l"(policy) : "memory");
}
__device__ __forceinline__ uint4 ld_shared16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

template <int D, int LAY, int DST>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas)
    rope_rows_kernel(const __grid_constant__ RopeParams<D / 2> rd, const __grid_constant__ RopeRows a, int iq, int ik, int steps) {
  using W = RowWarp<D, LAY>;
  constexpr int NW = kRopeThreads / 32;
  __shared__ __align__(16) float2 cos_sin[NW][D / 2];
  extern __shared__ __align__(16) uint4 ring_all[];     // [warps][kStages][2][32]
  W w(rd);
  float2* turn = cos_sin[threadIdx.x >> 5];
  const uint32_t ring_base = smem_u32(ring_all + (threadIdx.x >> 5) * (kStages * 64) + w.lane);
  unsigned long long freq[W::NP];
  int axis[W::NP];
  const auto* const rp = by_address(rd);
#pragma unroll
  for (int j = 0; j < W::NP; ++j) {
    freq[j] = rp->freq[w.lane + 32 * j];      // (past the rotated pairs: an angle of 0)
    axis[j] = rp->axis[w.lane + 32 * j];
  }
  const int ir = iq + ik;
  // The warp's tokens: every n_warps-th one, so that all warps are at neighbours, then an equal run of the steps of those left over.
  const int n_warps = gridDim.x * NW, me = blockIdx.x * NW + (threadIdx.x >> 5);
  int rounds = a.n_tok / n_warps;
  const long long rest = (long long)(a.n_tok - rounds * n_warps) * steps;
  const int s0 = (int)(rest * me / n_warps), s1 = (int)(rest * (me + 1) / n_warps);
  const int rest_tok = rounds * n_warps + s0 / steps, rest_it = s0 % steps;
  int left = rounds * steps + s1 - s0, tok = rounds ? me : rest_tok, it = rounds ? 0 : rest_it;
  auto go_on = [&](int& tok, int& it, int& rounds) {      // from a token's last step to the next token's first one
    it = rounds == 1 ? rest_it : 0;
    tok = rounds > 1 ? tok + n_warps : rounds == 1 ? rest_tok : tok + 1;
    rounds = max(0, rounds - 1);
  };
  kvs_pdl_entry();
  if (left == 0) return;
  // Fetching: the next step's rows into the ring (past the run's end: nothing, an empty group).  ahead_src: the lane's row of the next
  // step, ahead_h: its head, of ahead_n heads of queries, keys or values.
  int ahead = left, ahead_tok = tok, ahead_it = it, ahead_rounds = rounds, ahead_h = 0, ahead_n = 0;
  const uint4* ahead_src = nullptr;
  long long ahead_step = 0;
  auto aim = [&]() {      // at the heads of step ahead_it
    if (ahead_it < iq) {
      ahead_h = ahead_it * W::HPW + w.sub;
      ahead_n = a.q.n;
      ahead_src = W::from(a.q, ahead_tok, ahead_h);
      ahead_step = a.q.src_head * W::HPW / 8;
    } else if (ahead_it < ir) {
      ahead_h = (ahead_it - iq) * W::HPW + w.sub;
      ahead_n = a.k.n;
      ahead_src = W::from(a.k, ahead_tok, ahead_h);
      ahead_step = a.k.src_head * W::HPW / 8;
    } else {
      ahead_h = (ahead_it - ir) * W::HPW + w.sub;
      ahead_n = a.k.n;
      ahead_src = W::from(a.v, ahead_tok, ahead_h);
      ahead_step = a.v.src_head * W::HPW / 8;
    }
    ahead_src += w.at.c0;
  };
  aim();
  uint64_t once;      // rows are read once: what is written stays in L2 instead, for the attention
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(once));
  auto fetch = [&](uint32_t to) {
    if (ahead > 0) {
      if (ahead_h < ahead_n) {
        cp_async16_at(to, ahead_src, once);
        cp_async16_at(to + 512, ahead_src + w.at.apart(), once);
      }
      --ahead;
      ++ahead_it;
      ahead_h += W::HPW;
      ahead_src += ahead_step;
      if (ahead_it == iq || ahead_it >= ir) {      // other heads, or the next token's
        const bool through = ahead_it == steps;
        if (through) go_on(ahead_tok, ahead_it, ahead_rounds);
        if (ahead > 0 && (through || ahead_it == iq || ahead_it == ir)) aim();
      }
    }
    cp_async_commit();
  };
  int pos[W::NP];
  long long place = -1;
#pragma unroll
  for (int j = 0; j < W::NP; ++j) pos[j] = a.pos[axis[j] * a.pos_stride + tok];
  if (DST != kDense) place = a.place[tok];
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch(ring_base + i * 1024);
  uint32_t slot = 0;
  // the next step's rows, out of the ring, and another fetch into the slot before it
  auto arrive = [&]() {
    cp_async_wait<kStages - 2>();
    const Raw raw = {ld_shared16(ring_base + slot), ld_shared16(ring_base + slot + 512)};
    fetch(ring_base + ((slot + (kStages - 1) * 1024) & (kStages * 1024 - 1)));
    slot = (slot + 1024) & (kStages * 1024 - 1);
    return raw;
  };
  while (true) {
    const int last = min(steps, it + left);
    left -= last - it;
    // the next token's positions come while this one's rows are turned
    int next = tok, next_it = 0;
    if (left) go_on(next, next_it, rounds);
    int next_pos[W::NP];
    long long next_place = -1;
#pragma unroll
    for (int j = 0; j < W::NP; ++j) next_pos[j] = a.pos[axis[j] * a.pos_stride + next];
    if (DST != kDense) next_place = a.place[next];
    if (it < ir) {
      __syncwarp();       // (the last token's factors are read)
      w.turns(pos, freq, turn);
    }
    if (it < iq) {
      w.factors(w.weights(a.q.norm), turn);
      int h = it * W::HPW + w.sub;
      __nv_bfloat16* to = a.q.dst + tok * a.q.dst_tok + h * a.q.dst_head;
      for (const int end = min(last, iq); it < end; ++it, h += W::HPW, to += a.q.dst_head * W::HPW) {
        float x[16];
        w.row(arrive(), a.q.norm != nullptr, x);
        if (h < a.q.n) w.store_bf16(to, pack_bf16(x));
      }
    }
    if (it < last) {
      PlaceRow pl = {0, false};
      if (DST != kDense) pl = place_row(a, place);
      constexpr int ROW = DST == kPoolFp8 ? D : 2 * D;       // bytes of a row in the pool
      if (it < ir) {
        w.factors(w.weights(a.k.norm), turn);
        int h = (it - iq) * W::HPW + w.sub;
        __nv_bfloat16* to = a.k.dst + tok * a.k.dst_tok + h * a.k.dst_head;
        unsigned char* in_pool = a.kpool + (pl.row + (size_t)h * a.bs) * ROW;
        for (const int end = min(last, ir); it < end; ++it, h += W::HPW, to += a.k.dst_head * W::HPW, in_pool += W::HPW * a.bs * ROW) {
          float x[16];
          w.row(arrive(), a.k.norm != nullptr, x);
          if (DST == kDense) {
            if (h < a.k.n) w.store_bf16(to, pack_bf16(x));
          } else if (h < a.k.n && pl.there) {
            if (DST == kPoolFp8) w.store_e4m3(in_pool, x, a.k_scale, a.k_rcp);
            else w.store_bf16(in_pool, pack_bf16(x));
          }
        }
      }
      if (DST != kDense) {
        int h = (it - ir) * W::HPW + w.sub;
        unsigned char* in_pool = a.vpool + (pl.row + (size_t)h * a.bs) * ROW;
        for (; it < last; ++it, h += W::HPW, in_pool += W::HPW * a.bs * ROW) {
          const Raw raw = arrive();
          if (h < a.k.n && pl.there) {
            if (DST == kPoolFp8) {
              float x[16];
              unpack_bf16(raw, x);
              w.store_e4m3(in_pool, x, a.v_scale, a.v_rcp);
            } else {
              w.store_bf16(in_pool, raw);
            }
          }
        }
      }
    }
    if (!left) break;
    it = next_it;
    tok = next;
    place = next_place;
#pragma unroll
    for (int j = 0; j < W::NP; ++j) pos[j] = next_pos[j];
  }
}

// A warp turns 32 / (d / 16) kept keys of a (request, kv head) a step, in place, each by its own angles, and goes on to the next ones,
// `run` steps in all.  Rows come through a ring as above, their old positions and slots a step before them.
//
// Every key has angles of its own: 16 cosines and sines a lane and step, at 16 a clock of an SM 32 clocks, beside which some 180
// instructions a step take 45 of each scheduler's: more than an 8-bit row's bytes (a step's 1 KB: 44 clocks at the rate of a copy).
// 32 x 8 heads x 4096 keys of 128, E4M3: 62.0 us (40.2 for the bytes), the schedulers 69% busy, the same with 24 to 32 warps an
// SM and 3 or 4 stages; one step a warp took 132, four at once and no ring 74.  Angles by fused fp32 multiplications of a split
// frequency, fewer instructions than in integers, took 67: packed or not they use the unit that the rotation needs.  Lanes of 32
// elements took 70.7 (120 registers, 16 warps an SM).
// The same keys in bf16: 86 us, HBM (79.7).  8 x 8 x 2048 keys of which one in eight moves, bf16: 5.8 us (6.8 out of HBM).
constexpr int kRepThreads = 128;

constexpr int kRepStages = 4;
constexpr int kRepRun = 16;        // steps of a warp, at most

__device__ __forceinline__ void cp_async8_at(uint32_t smem, const void* gmem) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;\n" ::"r"(smem), "l"(gmem) : "memory");
}
__device__ __forceinline__ void cp_async16_at(uint32_t smem, const void* gmem) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(smem), "l"(gmem) : "memory");
}
__device__ __forceinline__ uint2 ld_shared8(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}

// Four E4M3 codes as fp32 (exact)
__device__ __forceinline__ void unpack_e4m3(uint32_t codes, float* x) {
  uint32_t h[2];
  asm("{.reg .b16 lo, hi;\n mov.b32 {lo, hi}, %2;\n cvt.rn.f16x2.e4m3x2 %0, lo;\n cvt.rn.f16x2.e4m3x2 %1, hi;}" : "=r"(h[0]), "=r"(h[1]) : "r"(codes));
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 y = __half22float2(*reinterpret_cast<__half2*>(&h[i]));
    x[2 * i] = y.x;
    x[2 * i + 1] = y.y;
  }
}

template <int D, int LAY, bool FP8>
__global__ void __launch_bounds__(kRepThreads, 6)
    pool_reposition_kernel(PoolDims d, const __grid_constant__ RopeParams<D / 2> rd, unsigned char* kpool, const int* __restrict__ kept,
                           const int* __restrict__ n_kept, const int* __restrict__ table, int keep, int run, unsigned* err) {
  constexpr int LPH = D / 16, HPW = 32 / LPH, ROW = FP8 ? D : 2 * D, CH = FP8 ? 8 : 16, S = kRepStages;      // CH: bytes of a chunk
  __shared__ __align__(16) unsigned char ring_all[kRepThreads / 32][S][2][32 * CH];
  __shared__ int2 what_all[kRepThreads / 32][S][32];      // positions to turn by, and the row's number in the layer
  const int lane = threadIdx.x & 31, sub = lane / LPH, l = lane % LPH;
  const LanePart<D, LAY> at(rd.rot, l);
  const uint32_t ring = smem_u32(&ring_all[threadIdx.x >> 5][0][0][lane * CH]);
  int2* what = &what_all[threadIdx.x >> 5][0][lane];
  unsigned long long freq[8];
  const auto* const rp = by_address(rd);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    freq[j] = at.turns(j, rd.rot) ? rp->freq[at.pair(j)] : 0ull;
    asm volatile("" : "+l"(freq[j]));      // (kept, not read from the parameters again each step)
  }
  const int u = blockIdx.y, r = u / d.Hkv, h = u - r * d.Hkv;
  const int first = (blockIdx.x * (kRepThreads / 32) + (threadIdx.x >> 5)) * run * HPW;
  kept += (size_t)u * keep;
  table += (size_t)r * d.nb_max;
  unsigned char* const pool = kpool + at.c0 * CH;
  kvs_pdl_entry();
  const int n = n_kept[r];
  if (n < 0 || n > keep) {
    if (threadIdx.x == 0) set_error(err, KVS_ERR_BAD_INDEX);
    return;
  }
  const int end = min(n, first + run * HPW);
  if (first >= end) return;
  const int steps = (end - first + HPW - 1) / HPW;
  // a step's old positions and slots come one step before its rows
  int by = 0, slot = 0, i = first + sub;
  auto find = [&]() {
    by = 0;
    if (i < end) {
      by = (int)((unsigned)i - (unsigned)kept[i]);
      slot = table[i >> d.log2bs];
    }
  };
  find();
  auto fetch = [&](int to) {
    int2 w = make_int2(by, -1);
    if (by != 0) {
      if ((unsigned)slot < (unsigned)d.n_slots) {
        w.y = (slot * d.Hkv + h) * d.bs + (i & (d.bs - 1));
        const unsigned char* p = pool + (size_t)(unsigned)w.y * ROW;
        if (FP8) {
          cp_async8_at(ring + to * (64 * CH), p);
          cp_async8_at(ring + to * (64 * CH) + 32 * CH, p + at.apart() * CH);
        } else {
          cp_async16_at(ring + to * (64 * CH), p);
          cp_async16_at(ring + to * (64 * CH) + 32 * CH, p + at.apart() * CH);
        }
      } else {
        set_error(err, KVS_ERR_BAD_INDEX);
      }
    }
    what[to * 32] = w;
    i += HPW;
    find();
    cp_async_commit();
  };
#pragma unroll
  for (int j = 0; j < S - 1; ++j) fetch(j);
  int at_slot = 0;
  for (int it = 0; it < steps; ++it) {
    cp_async_wait<S - 2>();
    const int2 w = what[at_slot * 32];
    float x[16];
    if (FP8) {
      const uint2 a = ld_shared8(ring + at_slot * (64 * CH)), b = ld_shared8(ring + at_slot * (64 * CH) + 32 * CH);
      unpack_e4m3(a.x, x);
      unpack_e4m3(a.y, x + 4);
      unpack_e4m3(b.x, x + 8);
      unpack_e4m3(b.y, x + 12);
    } else {
      unpack_bf16({ld_shared16(ring + at_slot * (64 * CH)), ld_shared16(ring + at_slot * (64 * CH) + 32 * CH)}, x);
    }
    fetch((at_slot + S - 1) % S);
    at_slot = (at_slot + 1) % S;
    const Pairs p = to_pairs<LAY>(x);
    Pairs y;
    const unsigned m = magnitude(w.x);
    const float two_pi = w.x < 0 ? -kTwoPi : kTwoPi;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float2 c, s;
      turn_cos_sin(m, two_pi, freq[2 * k], freq[2 * k + 1], c, s);
      y.u[k] = __ffma2_rn(__fmul2_rn(p.v[k], make_float2(-1.f, -1.f)), s, __fmul2_rn(p.u[k], c));
      y.v[k] = __ffma2_rn(p.u[k], s, __fmul2_rn(p.v[k], c));
      if (LAY != kHalves && !at.turns(2 * k, rd.rot)) {      // (owes nothing to its partner, which may be infinite)
        y.u[k] = p.u[k];
        y.v[k] = p.v[k];
      }
    }
    from_pairs<LAY>(y, x);
    if (w.y >= 0) {
      unsigned char* to = pool + (size_t)(unsigned)w.y * ROW;
      if (FP8) {
        *reinterpret_cast<uint2*>(to) = pack_e4m3(x);
        *reinterpret_cast<uint2*>(to + at.apart() * CH) = pack_e4m3(x + 8);
      } else {
        const Raw z = pack_bf16(x);
        *reinterpret_cast<uint4*>(to) = z.c0;
        *reinterpret_cast<uint4*>(to + at.apart() * CH) = z.c1;
      }
    }
  }
}

// The pairs that rows of d elements have (a kernel's parameters cost host time by their bytes: 0.15 us for 1.3 KB)
template <int D>
RopeParams<D / 2> params_of(const RopeDims& r) {
  RopeParams<D / 2> p = {r.d, r.rot, r.n_axis, r.adjacent, r.rot_scale, r.eps, {}, {}};
  std::copy_n(r.freq, D / 2, p.freq);
  std::copy_n(r.axis, D / 2, p.axis);
  return p;
}

template <int D, int LAY, int DST>
cudaError_t launch_rows(const RopeDims& rope, const RopeRows& a, cudaStream_t s) {
  const RopeParams<D / 2> rd = params_of<D>(rope);
  constexpr int HPW = 32 / (D / 16);
  const int sms = device_sm_count();
  const int iq = (a.q.n + HPW - 1) / HPW, ik = (a.k.n + HPW - 1) / HPW, steps = iq + ik * (DST == kDense ? 1 : 2);
  const long long warps = (long long)a.n_tok * steps;
  if (warps <= (long long)sms * kFewSteps) {
    const int grid = (int)((warps + kFewThreads / 32 - 1) / (kFewThreads / 32));
    launch_pdl(rope_few_kernel<D, LAY, DST>, dim3(grid), dim3(kFewThreads), 0, s, rd, a, iq, ik, steps);
    return cudaGetLastError();
  }
  constexpr int NW = kRopeThreads / 32;
  constexpr int smem = kRopeThreads * kStages * 32;
  static_assert(smem + NW * D / 2 * 8 <= 48 * 1024, "what a kernel may use without asking");
  const int grid = (int)std::min<long long>((warps + NW - 1) / NW, sms * kRopeCtas);
  launch_pdl(rope_rows_kernel<D, LAY, DST>, dim3(grid), dim3(kRopeThreads), (size_t)smem, s, rd, a, iq, ik, steps);
  return cudaGetLastError();
}

template <int D, int DST>
cudaError_t launch_rows(const RopeDims& rd, const RopeRows& a, cudaStream_t s) {
  if (rd.adjacent) return launch_rows<D, kAdjacent, DST>(rd, a, s);
  return rd.rot == D ? launch_rows<D, kHalves, DST>(rd, a, s) : launch_rows<D, kPart, DST>(rd, a, s);
}

template <int D, bool FP8>
cudaError_t launch_reposition(const PoolDims& d, const RopeDims& rope, unsigned char* k, const int* kept, const int* n_kept, const int* table,
                              int n_req, int keep, unsigned* err, cudaStream_t s) {
  const RopeParams<D / 2> rd = params_of<D>(rope);
  constexpr int HPW = 32 / (D / 16), NW = kRepThreads / 32;
  // steps of a warp: all of them, if one wave of warps does it, in runs that still even out over several waves if not
  const long long steps = (long long)n_req * d.Hkv * ((keep + HPW - 1) / HPW);
  const int run = (int)std::max(1ll, std::min<long long>(kRepRun, steps / (device_sm_count() * 32ll)));
  const dim3 grid((keep + NW * HPW * run - 1) / (NW * HPW * run), n_req * d.Hkv);
  auto go = [&](auto kernel) { launch_pdl(kernel, grid, dim3(kRepThreads), 0, s, d, rd, k, kept, n_kept, table, keep, run, err); };
  if (rd.adjacent) go(pool_reposition_kernel<D, kAdjacent, FP8>);
  else if (rd.rot == D) go(pool_reposition_kernel<D, kHalves, FP8>);
  else go(pool_reposition_kernel<D, kPart, FP8>);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope_rows(const RopeDims& rd, const RopeRows& a, cudaStream_t s) {
  if (!a.kpool)
    return rd.d == 64 ? launch_rows<64, kDense>(rd, a, s) : rd.d == 128 ? launch_rows<128, kDense>(rd, a, s) : launch_rows<256, kDense>(rd, a, s);
  if (a.fp8) return rd.d == 64 ? launch_rows<64, kPoolFp8>(rd, a, s) : launch_rows<128, kPoolFp8>(rd, a, s);
  return rd.d == 64 ? launch_rows<64, kPoolBf16>(rd, a, s) : launch_rows<128, kPoolBf16>(rd, a, s);
}

cudaError_t launch_pool_reposition(const PoolDims& d, const RopeDims& rd, unsigned char* k, const int* kept, const int* n_kept, const int* table,
                                   int n_req, int keep, unsigned* err, cudaStream_t s) {
  auto go = [&](auto kernel) { return kernel(d, rd, k, kept, n_kept, table, n_req, keep, err, s); };
  if (d.fp8) return d.d == 64 ? go(launch_reposition<64, true>) : go(launch_reposition<128, true>);
  return d.d == 64 ? go(launch_reposition<64, false>) : go(launch_reposition<128, false>);
}

}  // namespace kvs
