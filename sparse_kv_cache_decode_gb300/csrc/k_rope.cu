// Norms and rotation of query and key rows, dense or into a pool, and the repositioning of cached keys.
//
// A head's d elements lie in d / 16 lanes, two chunks of 8 elements (16 bytes) each, chosen so that both elements of every
// rotated pair are in one lane: no exchange but the norm's sum.  Pair i of a row turns by pos * f_i.  The angle is kept in
// turns, as an integer multiple of 2^-64: pos * f_i wraps around at whole turns by itself, exactly, for any 32-bit position
// (fp32 products lose the angle beyond some thousand positions); its upper 32 bits are off by less than 2^-32 turns.
#include <algorithm>

#include "kvs_ptx.cuh"
#include "kvs_rope.cuh"

namespace kvs {

namespace {

// cos and sin of pos * f turns
__device__ __forceinline__ void turn_cos_sin(int pos, unsigned long long f, float& c, float& s) {
  const int t = (int)((unsigned long long)((long long)pos * (long long)f) >> 32);
  sincospif((float)t * 0x1p-31f, &s, &c);
}

// What a lane holds of a row: chunks c0 and c1 (of 8 elements), and the pair of its j-th (a, b).
template <int D, bool ADJ>
struct LanePart {
  int c0, c1;
  __device__ __forceinline__ LanePart(int rot, int l) {
    const int n = rot / 16;
    if (ADJ || n == D / 16) {
      c0 = l;
      c1 = l + D / 16;
    } else if (l < n) {
      c0 = l;
      c1 = l + n;
    } else {
      c0 = 2 * l;
      c1 = c0 + 1;
    }
  }
  __device__ __forceinline__ int pair(int j) const { return ADJ ? (j < 4 ? 4 * c0 + j : 4 * c1 + j - 4) : 8 * c0 + j; }
  // (the pair's number is past the rotated ones where the elements do not turn)
  __device__ __forceinline__ bool turns(int j, int rot) const { return ADJ ? pair(j) < rot / 2 : c0 < rot / 16; }
};

__device__ __forceinline__ uint32_t f32x2_to_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// (a[j], b[j]) of two chunks, and back
template <bool ADJ, typename T>
__device__ __forceinline__ void to_pairs(const T (&x)[16], T (&a)[8], T (&b)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    a[j] = ADJ ? x[2 * j] : x[j];
    b[j] = ADJ ? x[2 * j + 1] : x[8 + j];
  }
}
template <bool ADJ, typename T>
__device__ __forceinline__ void from_pairs(const T (&a)[8], const T (&b)[8], T (&x)[16]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    x[ADJ ? 2 * j : j] = a[j];
    x[ADJ ? 2 * j + 1 : 8 + j] = b[j];
  }
}

__device__ __forceinline__ void unpack_bf16(const uint4& x0, const uint4& x1, float (&x)[16]) {
  const uint32_t w[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[2 * i] = bf16_lo(w[i]);
    x[2 * i + 1] = bf16_hi(w[i]);
  }
}
__device__ __forceinline__ void pack_bf16(const float (&x)[16], uint4& x0, uint4& x1) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = f32x2_to_bf16x2(x[2 * i], x[2 * i + 1]);
  x0 = make_uint4(w[0], w[1], w[2], w[3]);
  x1 = make_uint4(w[4], w[5], w[6], w[7]);
}
__device__ __forceinline__ uint2 pack_e4m3(const float* x) {
  return make_uint2(f32x2_to_e4m3x2(x[0], x[1]) | (f32x2_to_e4m3x2(x[2], x[3]) << 16),
                    f32x2_to_e4m3x2(x[4], x[5]) | (f32x2_to_e4m3x2(x[6], x[7]) << 16));
}

constexpr int kRopeThreads = 256;
enum { kDense, kPoolBf16, kPoolFp8 };

// One warp turns one token's heads (or a part of them: `parts` warps share a token), 32 / (d / 16) heads at a time.
template <int D, bool ADJ, int DST>
__global__ void __launch_bounds__(kRopeThreads)
    rope_rows_kernel(const __grid_constant__ RopeDims rd, const __grid_constant__ RopeRows a, int parts) {
  constexpr int LPH = D / 16, HPW = 32 / LPH;
  const int lane = threadIdx.x & 31, sub = lane / LPH, l = lane % LPH;
  const LanePart<D, ADJ> at(rd.rot, l);
  unsigned long long freq[8];
  int axis[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const bool live = at.turns(j, rd.rot);
    freq[j] = live ? rd.freq[at.pair(j)] : 0ull;      // (an angle of 0: cos 1, sin 0)
    axis[j] = live ? rd.axis[at.pair(j)] : 0;
  }
  const float scale0 = at.turns(0, rd.rot) ? rd.rot_scale : 1.f, scale1 = at.turns(7, rd.rot) ? rd.rot_scale : 1.f;
  kvs_pdl_entry();
  const int iq = (a.q.n + HPW - 1) / HPW, ik = (a.k.n + HPW - 1) / HPW, steps = iq + ik + (DST == kDense ? 0 : ik);
  const int per = (steps + parts - 1) / parts;
  const long long items = (long long)a.n_tok * parts, n_warps = (long long)gridDim.x * (kRopeThreads / 32);
  for (long long item = (long long)blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5); item < items; item += n_warps) {
    const int tok = (int)(item / parts), first = (int)(item - (long long)tok * parts) * per, last = min(steps, first + per);
    float cs[8], sn[8];
    if (first < iq + ik) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        turn_cos_sin(a.pos[axis[j] * a.pos_stride + tok], freq[j], cs[j], sn[j]);
        const float sc = j < 4 ? scale0 : scale1;
        cs[j] *= sc;
        sn[j] *= sc;
      }
    }
    size_t row = 0;        // the token's row in head 0 of its slot
    bool stored = true;
    if (DST != kDense && last > iq) {
      const long long p = a.place[tok];
      stored = p >= 0 && p < ((long long)a.n_slots << a.log2bs);
      if (p >= 0 && !stored) set_error(a.err, KVS_ERR_BAD_INDEX);
      row = (size_t)(p >> a.log2bs) * a.k.n * a.bs + (p & (a.bs - 1));
    }
    for (int it = first; it < last; ++it) {
      const bool is_q = it < iq, is_v = it >= iq + ik;
      const RopeHeads& g = is_q ? a.q : is_v ? a.v : a.k;
      const int h = (it - (is_q ? 0 : is_v ? iq + ik : iq)) * HPW + sub;
      const bool there = h < g.n;
      uint4 x0 = make_uint4(0, 0, 0, 0), x1 = x0;
      if (there) {
        const __nv_bfloat16* src = g.src + tok * g.src_tok + h * g.src_head;
        x0 = __ldcs(reinterpret_cast<const uint4*>(src) + at.c0);
        x1 = __ldcs(reinterpret_cast<const uint4*>(src) + at.c1);
      }
      float x[16];
      if (!is_v || DST == kPoolFp8) unpack_bf16(x0, x1, x);
      if (!is_v) {
        if (g.norm) {
          float sum = 0.f;
#pragma unroll
          for (int j = 0; j < 16; ++j) sum = fmaf(x[j], x[j], sum);
#pragma unroll
          for (int o = LPH / 2; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
          const float inv = rsqrtf(sum * (1.f / D) + rd.eps);
          const float4* w = reinterpret_cast<const float4*>(g.norm);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float4 y = __ldg(w + (j < 2 ? 2 * at.c0 + j : 2 * at.c1 + j - 2));
            x[4 * j] *= inv * y.x;
            x[4 * j + 1] *= inv * y.y;
            x[4 * j + 2] *= inv * y.z;
            x[4 * j + 3] *= inv * y.w;
          }
        }
        float u[8], v[8], p[8], r[8];
        to_pairs<ADJ>(x, u, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          p[j] = u[j] * cs[j] - v[j] * sn[j];
          r[j] = v[j] * cs[j] + u[j] * sn[j];
        }
        from_pairs<ADJ>(p, r, x);
        if (is_q || DST != kPoolFp8) pack_bf16(x, x0, x1);
      }
      if (DST == kDense || is_q) {
        if (there) {
          uint4* dst = reinterpret_cast<uint4*>(g.dst + tok * g.dst_tok + h * g.dst_head);
          dst[at.c0] = x0;
          dst[at.c1] = x1;
        }
      } else if (there && stored) {
        unsigned char* dst = (is_v ? a.vpool : a.kpool) + (row + (size_t)h * a.bs) * (DST == kPoolFp8 ? D : 2 * D);
        if (DST == kPoolBf16) {
          reinterpret_cast<uint4*>(dst)[at.c0] = x0;
          reinterpret_cast<uint4*>(dst)[at.c1] = x1;
        } else {
          const float scale = is_v ? a.v_scale : a.k_scale;
#pragma unroll
          for (int j = 0; j < 16; ++j) x[j] = __fdiv_rn(x[j], scale);
          reinterpret_cast<uint2*>(dst)[at.c0] = pack_e4m3(x);
          reinterpret_cast<uint2*>(dst)[at.c1] = pack_e4m3(x + 8);
        }
      }
    }
  }
}

// One warp turns 32 / (d / 16) kept keys of a (request, kv head) at a time, in place, each by its own angles.
constexpr int kRepThreads = 128;

template <int D, bool ADJ, bool FP8>
__global__ void __launch_bounds__(kRepThreads)
    pool_reposition_kernel(PoolDims d, const __grid_constant__ RopeDims rd, unsigned char* kpool, const int* __restrict__ kept,
                           const int* __restrict__ n_kept, const int* __restrict__ table, int keep, unsigned* err) {
  constexpr int LPH = D / 16, HPW = 32 / LPH;
  const int lane = threadIdx.x & 31, sub = lane / LPH, l = lane % LPH;
  const LanePart<D, ADJ> at(rd.rot, l);
  unsigned long long freq[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) freq[j] = at.turns(j, rd.rot) ? rd.freq[at.pair(j)] : 0ull;
  kvs_pdl_entry();
  const int u = blockIdx.y, r = u / d.Hkv, h = u - r * d.Hkv;
  const int n = n_kept[r];
  if (n < 0 || n > keep) {
    if (threadIdx.x == 0) set_error(err, KVS_ERR_BAD_INDEX);
    return;
  }
  const int i = (blockIdx.x * (kRepThreads / 32) + (threadIdx.x >> 5)) * HPW + sub;
  if (i >= n) return;
  const int by = (int)((unsigned)i - (unsigned)kept[(size_t)u * keep + i]);
  if (by == 0) return;
  const int slot = table[(size_t)r * d.nb_max + (i >> d.log2bs)];
  if (slot < 0 || slot >= d.n_slots) {
    set_error(err, KVS_ERR_BAD_INDEX);
    return;
  }
  unsigned char* row = kpool + (((size_t)slot * d.Hkv + h) * d.bs + (i & (d.bs - 1))) * (FP8 ? D : 2 * D);
  float x[16];
  if (FP8) {
    const uint2 a = reinterpret_cast<const uint2*>(row)[at.c0], b = reinterpret_cast<const uint2*>(row)[at.c1];
    const uint32_t w[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
    for (int j = 0; j < 16; ++j) x[j] = e4m3_to_f32((w[j >> 2] >> ((j & 3) * 8)) & 255u);
  } else {
    unpack_bf16(reinterpret_cast<const uint4*>(row)[at.c0], reinterpret_cast<const uint4*>(row)[at.c1], x);
  }
  float p[8], q[8];
  to_pairs<ADJ>(x, p, q);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float c, s;
    turn_cos_sin(by, freq[j], c, s);
    const float y = p[j] * c - q[j] * s;
    q[j] = q[j] * c + p[j] * s;
    p[j] = y;
  }
  from_pairs<ADJ>(p, q, x);
  if (FP8) {
    reinterpret_cast<uint2*>(row)[at.c0] = pack_e4m3(x);
    reinterpret_cast<uint2*>(row)[at.c1] = pack_e4m3(x + 8);
  } else {
    uint4 a, b;
    pack_bf16(x, a, b);
    reinterpret_cast<uint4*>(row)[at.c0] = a;
    reinterpret_cast<uint4*>(row)[at.c1] = b;
  }
}

template <int D, int DST>
cudaError_t launch_rows(const RopeDims& rd, const RopeRows& a, cudaStream_t s) {
  constexpr int HPW = 32 / (D / 16), NW = kRopeThreads / 32;
  const int steps = (a.q.n + HPW - 1) / HPW + (a.k.n + HPW - 1) / HPW * (DST == kDense ? 1 : 2);
  const int sms = device_sm_count();
  const long long want = (long long)sms * NW * 3;
  const int parts = (int)std::max(1ll, std::min<long long>(steps, want / a.n_tok));
  const long long ctas = ((long long)a.n_tok * parts + NW - 1) / NW;
  const int grid = (int)std::min<long long>(ctas, (long long)sms * 8);
  if (rd.adjacent)
    launch_pdl(rope_rows_kernel<D, true, DST>, dim3(grid), dim3(kRopeThreads), 0, s, rd, a, parts);
  else
    launch_pdl(rope_rows_kernel<D, false, DST>, dim3(grid), dim3(kRopeThreads), 0, s, rd, a, parts);
  return cudaGetLastError();
}

template <int D, bool FP8>
cudaError_t launch_reposition(const PoolDims& d, const RopeDims& rd, unsigned char* k, const int* kept, const int* n_kept, const int* table,
                              int n_req, int keep, unsigned* err, cudaStream_t s) {
  constexpr int SPAN = kRepThreads / 32 * (32 / (D / 16));
  const dim3 grid((keep + SPAN - 1) / SPAN, n_req * d.Hkv);
  if (rd.adjacent)
    launch_pdl(pool_reposition_kernel<D, true, FP8>, grid, dim3(kRepThreads), 0, s, d, rd, k, kept, n_kept, table, keep, err);
  else
    launch_pdl(pool_reposition_kernel<D, false, FP8>, grid, dim3(kRepThreads), 0, s, d, rd, k, kept, n_kept, table, keep, err);
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
