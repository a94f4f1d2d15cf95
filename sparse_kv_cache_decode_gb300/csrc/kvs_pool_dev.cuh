// Device helpers of the pool kernels that run on the tensor cores.
#pragma once
#include "kvs_pool.cuh"
#include "kvs_ptx.cuh"

namespace kvs {
namespace pdev {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int TOK = 128;                      // tokens per K/V tile
constexpr int MAX_SMEM = 227 * 1024;
constexpr int kPieces = 64;                   // pieces of work a CTA plans at a time

// n / G (n < 2^25)
__device__ __forceinline__ int div_g(const PoolDims& d, int n) { return d.G == 1 ? n : (int)__umulhi((unsigned)n, d.g_magic); }
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// One lane of the (whole) warp, always the same.  The products of a warp are issued under it from values that all
// lanes hold, so that descriptors stay in uniform registers (measured for 128 x 64 x 16 products: 28 cycles to
// issue one, against 51 under `lane == 0`).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred P;\n elect.sync _|P, 0xffffffff;\n selp.u32 %0, 1, 0, P;\n}\n" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// Products with descriptors given by their low words (start address / 16, and the leading offset / 16 of an MN-major
// operand in bits 16-29); the high word is the same for every operand here: 1024 bytes between 8-row groups, the
// version bit and the 128-byte swizzle.  The issuing warp shares its scheduler with two softmax warps and gets few of
// its slots, so every instruction around a product counts.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
template <bool ACC>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 x, y;\n setp.ne.u32 p, %5, 0;\n mov.b64 x, {%1, %3};\n mov.b64 y, {%2, %3};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(kDescHi), "r"(idesc), "n"(ACC ? 1 : 0)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 y;\n setp.ne.u32 p, 1, 0;\n mov.b64 y, {%2, %3};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(kDescHi), "r"(idesc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 y;\n setp.ne.u32 p, %5, 0;\n mov.b64 y, {%2, %3};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(kDescHi), "r"(idesc), "r"(acc)
      : "memory");
}

__device__ __forceinline__ void tma_load_3d(void* dst, const void* tm, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n" ::
          "r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

// Zeroes, in a tile of 128-byte rows with `chunks` 64-dim chunks, those of the calling warp's 32 rows (from row0 on) whose bit
// is set: 8 lanes a row, so that the stores of a step fill all banks.
__device__ __forceinline__ void zero_rows(unsigned char* tile, int chunks, int row0, uint32_t rows) {
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int i = 0; i < 32; i += 4) {
    const int r = i + (lane >> 3);
    if ((rows >> r) & 1u)
      for (int b = 0; b < chunks; ++b)
        *reinterpret_cast<uint4*>(tile + b * (TOK * 128) + (row0 + r) * 128 + (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
  }
}

// 8 columns of a thread's tensor-memory lane
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float (&v)[8]) {
  uint32_t r[8];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}

// pairs of fp32 in one 64-bit register
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t x, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// the lowest n bits (n < 0: none, n > 32: all)
__device__ __forceinline__ uint32_t bits_below(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }

// Exclusive scans of a count and a sum over the CTA's threads in one; ws: 64 words of shared memory.
struct Scan {
  int n, n_all;
  long long v, v_all;
};
__device__ __forceinline__ Scan block_scan(int n, long long v, long long* ws, int nw) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int xn = n;
  long long xv = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int yn = __shfl_up_sync(0xffffffffu, xn, o);
    const long long yv = __shfl_up_sync(0xffffffffu, xv, o);
    if (lane >= o) {
      xn += yn;
      xv += yv;
    }
  }
  __syncthreads();
  if (lane == 31) {
    ws[2 * warp] = xn;
    ws[2 * warp + 1] = xv;
  }
  __syncthreads();
  Scan r = {xn - n, 0, xv - v, 0};
  for (int w = 0; w < nw; ++w) {
    const int a = (int)ws[2 * w];
    const long long b = ws[2 * w + 1];
    if (w < warp) {
      r.n += a;
      r.v += b;
    }
    r.n_all += a;
    r.v_all += b;
  }
  return r;
}

// Bounded wait for the phase of the given parity.  Code that runs once per tile beside the softmax's long unrolled
// loops is limited by instruction fetch, so the rare path is short: the clock is read every 64th try, and the
// kernel's end reports a time-out (abort_flag) once for all.
__device__ __forceinline__ bool bounded_wait(uint64_t* bar, unsigned parity, uint64_t timeout_ns, volatile int* abort_flag) {
  if (__builtin_expect(mbar_try_wait(bar, parity), 1)) return true;
  uint64_t t = 0;
#pragma unroll 1
  for (unsigned n = 0; !mbar_try_wait(bar, parity); ++n) {
    if (n & 63u) continue;
    if (*abort_flag) return false;
    const uint64_t now = global_timer_ns();
    if (n == 0) t = now;
    if (now - t > timeout_ns) {
      *abort_flag = 1;
      return false;
    }
  }
  return true;
}

// Four E4M3 codes as bf16 pairs (codes 0, 1 and 2, 3), exactly: a code's exponent and mantissa bits at bf16's places
// stand for its value times 2^-120, subnormals included, and the product with 2^120 is exact.  All of it runs at the
// full integer and fma rates, which the conversion instructions do not.  (The NaN codes come out as +-480: pools
// hold finite values.)
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t a = __byte_perm(w, 0u, 0x1404), b = __byte_perm(w, 0u, 0x3424);   // a code in each half's upper byte
  const uint32_t x = ((a >> 4) & 0x07f007f0u) | (a & 0x80008000u), y = ((b >> 4) & 0x07f007f0u) | (b & 0x80008000u);
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(lo) : "r"(x), "r"(0x7b807b80u));           // 0x7b80: 2^120
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(hi) : "r"(y), "r"(0x7b807b80u));
}
// Row and vector (16 codes) that place y of a code tile is widened by.  At 8 vectors a row, 8 lanes take half of a row and
// the other half of the next: their 16-byte loads and stores then fill all banks (a row's two 64-dim chunks of bf16 are
// 16 KiB apart, on the same banks, and its own 8 vectors would meet there in pairs).
template <int VEC>
__device__ __forceinline__ void widen_place(int y, int& row, int& v) {
  if (VEC == 8) {
    const int sub = (y >> 2) & 1;
    row = (y >> 4) * 2 + sub;
    v = (y & 3) + 4 * (sub ^ ((y >> 3) & 1));
  } else {
    row = y / VEC;
    v = y - row * VEC;
  }
}
// 16 E4M3 codes (vector v of a row) as bf16 into the row of a K-major 128-byte-swizzled tile: `p` the row in its first
// 64-dim chunk, chunks `chunk` bytes apart.
__device__ __forceinline__ void widen16(const uint4& w, unsigned char* p, int chunk, int row, int v) {
  uint4 x, y;
  widen4(w.x, x.x, x.y);
  widen4(w.y, x.z, x.w);
  widen4(w.z, y.x, y.y);
  widen4(w.w, y.z, y.w);
  p += (v >> 2) * chunk;
  const int c16 = (v & 3) * 2;
  *reinterpret_cast<uint4*>(p + ((c16 ^ (row & 7)) << 4)) = x;
  *reinterpret_cast<uint4*>(p + (((c16 + 1) ^ (row & 7)) << 4)) = y;
}

}  // namespace pdev
}  // namespace kvs
