// AdamW over many tensors in one launch, with the two moments in fp32 or in 8 bits.
//
//   m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2,
//   p = p (1 - lr wd) - lr (m / (1 - b1^step)) / (sqrt(v / (1 - b2^step)) + eps).
//
// 8-bit state: blocks of 256 elements of a tensor (the last may be shorter), each
// with the largest magnitude of its moment as an fp32 scale a.
//   m: int8 c,  value a * fl32(c |c| / 127^2);   v: uint8 q, value a * fl32(q^4 / 255^4).
// The levels lie densest near zero in absolute terms and within 0.8% of each other at
// the top; a v above zero is never stored as zero (its quotient m / sqrt(v) would
// explode).  The code is that of the nearest root, rint(127 sqrt(|m| / a)) and
// rint(255 (v / a)^(1/4)), of the moments as fp32 numbers: every product and sum of
// their update is rounded once (no contraction), so the state is defined bit for bit.
// The root is taken with the approximate square root; only next to a border, closer than
// its error, is the choice made again, in fp64.
#include <math.h>

#include <algorithm>
#include <vector>

#include "common.cuh"

namespace lsq {

namespace {

constexpr int kBlk = 256;          // elements per scale: one warp, 8 per lane
constexpr int kChunk = 8 * kBlk;   // elements a CTA takes at a time, a block per warp
constexpr int kMtThreads = 256;

struct MtEntry {
  float* p;
  const void* g;
  void* m;
  void* v;
  float* ms;
  float* vs;
  int64_t n;
  float lr, wd;
  uint32_t chunk0;  // first chunk of this tensor in the launch
  uint32_t unused;
};

struct MtHead {
  float b1, b2, c1, c2, eps;
  float inv_bc1, inv_sqrt_bc2;
  int n;                  // tensors in this launch
  uint32_t chunks;        // chunks in this launch
  const int32_t* step;    // device step count, or null
  const int* gate;        // status word that keeps all as it is with a bad index, or null
  int* dev_err;
};

// The tensors travel in the kernel's parameters (at most 32,764 bytes), so a step
// needs no device table and a captured graph holds its own copy.
constexpr int kMtFew = 48;
constexpr int kMtMany = (32764 - (int)sizeof(MtHead)) / (int)sizeof(MtEntry);

template <int N>
struct MtArgs {
  MtHead h;
  MtEntry e[N];
};

// Approximate square root and reciprocal (relative errors 2^-23); subnormal inputs count
// as 0.
__device__ __forceinline__ float sqrt_ftz(float x) {
  float r;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_ftz(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// Pairs of fp32 numbers, an operation on both at once.  A paired product and a paired sum
// behind it are contracted to one rounding in spite of their modifiers, so where both
// roundings count (the moments) the sums are single ones.
__device__ __forceinline__ uint64_t two(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 both(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// The codes are rounded by adding 1.5 2^23, which leaves the nearest integer (ties to
// even) in the low bits without a conversion: those run on the pipe that the square
// roots need.  y is 127 sqrt(x / a), off by at most 127 (3/2 2^-23) and a rounding, less
// than 4e-5, or 255 (x / a)^(1/4), off by at most 255 (2.2 2^-23) and a rounding, less
// than 9e-5.  Where y lies within kNear of a border, the code is taken from the exact
// comparison: x 254^2 against a (2 b + 1)^2 (both exact in fp64, 40 bits), x 510^4 against
// a (2 b + 1)^4 (up to 60 bits: where the rounded products are equal, by what their rounding
// left, which one fused operation gives exactly); a tie goes to the even code.
constexpr float kRound = 12582912.f;
constexpr float kNear = 2e-4f;
__device__ __forceinline__ int exact_m(float x, float a, float y) {
  const int b = (int)floorf(y);
  if (fabsf(y - (float)b - 0.5f) > kNear) return (int)rintf(y);
  const double l = (double)x * 64516.0, r = (double)a * (double)((2 * b + 1) * (2 * b + 1));
  return l > r ? b + 1 : l < r ? b : b + (b & 1);
}
__device__ __forceinline__ int exact_v(float x, float a, float y) {
  const int b = (int)floorf(y);
  int k = (int)rintf(y);
  if (fabsf(y - (float)b - 0.5f) <= kNear) {
    const double o = (double)((2 * b + 1) * (2 * b + 1)), xd = (double)x, ad = (double)a;
    constexpr double kTop = 67652010000.0;  // 510^4
    const double l = xd * kTop, r = ad * (o * o);
    const double le = fma(xd, kTop, -l), re = fma(ad, o * o, -r);
    k = l > r || (l == r && le > re) ? b + 1 : l < r || le < re ? b : b + (b & 1);
  }
  return x > 0.f ? max(k, 1) : k;
}
__device__ __forceinline__ float inv_root(float a) { return __fdiv_rn(1.f, __fsqrt_rn(a)); }
// The roots of v are taken of 2^24 v, 2^12 too large: so that a subnormal v keeps its root
// (with an eps below 2^-63 that is the quotient's whole denominator).  From 2^100 on, where
// 2^24 v could overflow, by the exact square root.
constexpr float kRootUp = 16777216.f, kRootDown = 1.f / 4096.f;
constexpr uint32_t kHugeV = (127u + 100u) << 23;

// The values the codes stand for: fl32(c |c| / 127^2) at c + 128, and fl32(q^4 / 255^4).
__device__ __forceinline__ float level_m(int c) {
  return __fdiv_rn((float)(c * abs(c)), 16129.f);
}
__device__ __forceinline__ float level_v(int q) {
  const double d = (double)(q * q);
  return (float)(d * d / 4228250625.0);
}

// A block's scale: its largest magnitude, or 0 (every code 0) below the normal range.
__device__ __forceinline__ float scale_of(float top) { return top < 1.17549435e-38f ? 0.f : top; }

// Four elements of a tensor's array at offset o, of which `in` exist (all in a whole block).
template <bool WHOLE, class T4, class T>
__device__ __forceinline__ T4 load4(const void* base, int64_t o, int in) {
  T4 r;
  if (WHOLE || in >= 4) {
    r = *reinterpret_cast<const T4*>(static_cast<const T*>(base) + o);
  } else {
    T* e = reinterpret_cast<T*>(&r);
#pragma unroll
    for (int i = 0; i < 4; ++i) e[i] = i < in ? static_cast<const T*>(base)[o + i] : T(0);
  }
  return r;
}
template <bool WHOLE, class T4, class T>
__device__ __forceinline__ void store4(void* base, int64_t o, int in, T4 v) {
  if (WHOLE || in >= 4) {
    *reinterpret_cast<T4*>(static_cast<T*>(base) + o) = v;
  } else {
    const T* e = reinterpret_cast<const T*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < in) static_cast<T*>(base)[o + i] = e[i];
  }
}
struct alignas(8) U16x4 {
  uint16_t v[4];
};

// One block of a tensor (a warp): elements [base, base + left).
struct MtRates {
  float inv_bc1, isb2;
};
template <int BITS, int GBITS, bool WHOLE>
__device__ __forceinline__ void adamw_block(const MtHead& h, const MtEntry& e, const MtRates& r,
                                            const float* lm, const float* lv, int64_t base, int left,
                                            int lane) {
  const uint64_t b1 = two(h.b1, h.b1), b2 = two(h.b2, h.b2);
  const uint64_t c1 = two(h.c1, h.c1), c2 = two(h.c2, h.c2);
  const float decay = e.lr * e.wd, rate = e.lr * r.inv_bc1;
  float4 p4[2];
  uint64_t g[4], m[4], v[4];  // element pairs
  uint32_t mc[2], vc[2];
  float am = 0.f, av = 0.f;
  if (BITS == 8) {
    am = e.ms[base / kBlk];
    av = e.vs[base / kBlk];
  }
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int o = u * 128 + lane * 4, in = left - o;
    p4[u] = load4<WHOLE, float4, float>(e.p, base + o, in);
    if (GBITS == 32) {
      const float4 y = load4<WHOLE, float4, float>(e.g, base + o, in);
      g[2 * u] = two(y.x, y.y);
      g[2 * u + 1] = two(y.z, y.w);
    } else {
      const U16x4 y = load4<WHOLE, U16x4, uint16_t>(e.g, base + o, in);
      g[2 * u] = two(bf16_bits_to_float(y.v[0]), bf16_bits_to_float(y.v[1]));
      g[2 * u + 1] = two(bf16_bits_to_float(y.v[2]), bf16_bits_to_float(y.v[3]));
    }
    if (BITS == 8) {
      mc[u] = load4<WHOLE, uint32_t, uint8_t>(e.m, base + o, in);
      vc[u] = load4<WHOLE, uint32_t, uint8_t>(e.v, base + o, in);
    } else {
      const float4 y = load4<WHOLE, float4, float>(e.m, base + o, in);
      const float4 z = load4<WHOLE, float4, float>(e.v, base + o, in);
      m[2 * u] = two(y.x, y.y);
      m[2 * u + 1] = two(y.z, y.w);
      v[2 * u] = two(z.x, z.y);
      v[2 * u + 1] = two(z.z, z.w);
    }
  }
  if (BITS == 8) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t wm = mc[j >> 1] >> (16 * (j & 1)), wv = vc[j >> 1] >> (16 * (j & 1));
      m[j] = mul2(two(am, am), two(lm[wm & 255u], lm[(wm >> 8) & 255u]));
      v[j] = mul2(two(av, av), two(lv[wv & 255u], lv[(wv >> 8) & 255u]));
    }
  }
  // the moments; the bits of their largest magnitudes (NaN and infinity above all) give
  // the block's scales and tell whether any is not finite
  uint32_t tm = 0, tv = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 x0 = both(mul2(b1, m[j])), x1 = both(mul2(c1, g[j]));
    const float2 y0 = both(mul2(b2, v[j])), y1 = both(mul2(mul2(c2, g[j]), g[j]));
    const float2 x = make_float2(__fadd_rn(x0.x, x1.x), __fadd_rn(x0.y, x1.y));
    const float2 y = make_float2(__fadd_rn(y0.x, y1.x), __fadd_rn(y0.y, y1.y));
    m[j] = two(x.x, x.y);
    v[j] = two(y.x, y.y);
    tm = max(tm, max(__float_as_uint(x.x) & 0x7FFFFFFFu, __float_as_uint(x.y) & 0x7FFFFFFFu));
    tv = max(tv, max(__float_as_uint(y.x), __float_as_uint(y.y)));
  }
  uint32_t skip = 0;  // elements whose moments leave the finite range keep everything
  if (max(tm, tv) >= 0x7F800000u) {
    atomicOr(h.dev_err, DEV_ERR_NONFINITE);
    tm = tv = 0;
    for (int i = 0; i < 8; ++i) {
      const int off = (i >> 2) * 128 + lane * 4 + (i & 3);
      const int64_t at = base + off;
      float2 x = both(m[0]), y = both(v[0]);
#pragma unroll
      for (int j = 1; j < 4; ++j)
        if (j == i / 2) {
          x = both(m[j]);
          y = both(v[j]);
        }
      float mi = i & 1 ? x.y : x.x, vi = i & 1 ? y.y : y.x;
      if (!WHOLE && off >= left) {
        mi = vi = 0.f;  // no such element (its code 0 times a scale that is not finite)
      } else if (!(fabsf(mi) < INFINITY && vi < INFINITY)) {
        skip |= 1u << i;
        mi = BITS == 8 ? am * lm[static_cast<uint8_t*>(e.m)[at]] : static_cast<float*>(e.m)[at];
        vi = BITS == 8 ? av * lv[static_cast<uint8_t*>(e.v)[at]] : static_cast<float*>(e.v)[at];
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j == i / 2) {
          m[j] = i & 1 ? two(x.x, mi) : two(mi, x.y);
          v[j] = i & 1 ? two(y.x, vi) : two(vi, y.y);
        }
      // (a state that already was not finite counts as zero in the scale)
      const uint32_t bm = __float_as_uint(mi) & 0x7FFFFFFFu, bv = __float_as_uint(vi) & 0x7FFFFFFFu;
      tm = max(tm, bm < 0x7F800000u ? bm : 0u);
      tv = max(tv, bv < 0x7F800000u ? bv : 0u);
    }
  }
  float root[8];
  {
    const float isd = r.isb2 * kRootDown;
    const uint64_t is2 = two(isd, isd), ep2 = two(h.eps, h.eps), up2 = two(kRootUp, kRootUp);
    // the change of p first, then one sum: p itself is rounded once
    const uint64_t de2 = two(-decay, -decay), nr2 = two(-rate, -rate);
    float* pf = reinterpret_cast<float*>(p4);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 y = both(mul2(v[j], up2));
      root[2 * j] = sqrt_ftz(y.x);
      root[2 * j + 1] = sqrt_ftz(y.y);
      if (tv >= kHugeV) {
        const float2 z = both(v[j]);
        root[2 * j] = __fsqrt_rn(z.x) * 4096.f;
        root[2 * j + 1] = __fsqrt_rn(z.y) * 4096.f;
      }
      const float2 d = both(fma2(two(root[2 * j], root[2 * j + 1]), is2, ep2));
      const uint64_t u = mul2(m[j], two(rcp_ftz(d.x), rcp_ftz(d.y)));
      const uint64_t p0 = two(pf[2 * j], pf[2 * j + 1]);
      const float2 q = both(add2(p0, fma2(u, nr2, mul2(p0, de2))));
      pf[2 * j] = q.x;
      pf[2 * j + 1] = q.y;
    }
  }
  if (skip)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (skip >> i & 1u)
        reinterpret_cast<float*>(p4)[i] = e.p[base + (i >> 2) * 128 + lane * 4 + (i & 3)];
  if (BITS == 8) {
    am = scale_of(__uint_as_float(__reduce_max_sync(0xFFFFFFFFu, tm)));
    av = scale_of(__uint_as_float(__reduce_max_sync(0xFFFFFFFFu, tv)));
    const float im = am > 0.f ? __fdiv_rn(1.f, am) : 0.f, iv = av > 0.f ? inv_root(av) * kRootDown : 0.f;
    const uint64_t r2 = two(kRound, kRound), nr2 = two(-kRound, -kRound);
    const uint64_t im2 = two(im, im), iv2 = two(iv, iv), s127 = two(127.f, 127.f),
                   s255 = two(255.f, 255.f), neg = two(-1.f, -1.f);
    float worst = 0.f;  // the largest distance from an integer
    mc[0] = mc[1] = vc[0] = vc[1] = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 x = both(m[j]), z = both(v[j]);
      float2 q = both(mul2(two(fabsf(x.x), fabsf(x.y)), im2));
      uint64_t y = mul2(two(sqrt_ftz(q.x), sqrt_ftz(q.y)), s127);
      float2 s = both(y);
      y = two(copysignf(s.x, x.x), copysignf(s.y, x.y));
      uint64_t t = add2(y, r2);
      float2 d = both(fma2(add2(t, nr2), neg, y));
      worst = fmaxf(worst, fmaxf(fabsf(d.x), fabsf(d.y)));
      float2 k = both(t);
      mc[j >> 1] |= (__byte_perm(__float_as_uint(k.x), __float_as_uint(k.y), 0x0040) & 0xFFFFu)
                    << (16 * (j & 1));
      q = both(mul2(two(root[2 * j], root[2 * j + 1]), iv2));
      y = mul2(two(sqrt_ftz(q.x), sqrt_ftz(q.y)), s255);
      t = add2(y, r2);
      d = both(fma2(add2(t, nr2), neg, y));
      worst = fmaxf(worst, fmaxf(fabsf(d.x), fabsf(d.y)));
      k = both(t);
      // (a v above zero is stored as 1 at least; without a scale as 0)
      const uint32_t k0 = max(__float_as_uint(k.x) & 0xFFFFu, min(__float_as_uint(z.x), 1u));
      const uint32_t k1 = max(__float_as_uint(k.y) & 0xFFFFu, min(__float_as_uint(z.y), 1u));
      vc[j >> 1] |= (__byte_perm(k0, k1, 0x0040) & 0xFFFFu) << (16 * (j & 1));
    }
    if (worst > 0.5f - kNear || fminf(am, av) == 0.f) {  // a border near by, or no scale
      mc[0] = mc[1] = vc[0] = vc[1] = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 x = both(m[i / 2]), z = both(v[i / 2]);
        const float mi = i & 1 ? x.y : x.x, vi = i & 1 ? z.y : z.x;
        int k = am > 0.f ? exact_m(fabsf(mi), am, 127.f * sqrt_ftz(fabsf(mi) * im)) : 0;
        k = mi < 0.f ? -k : k;
        mc[i / 4] |= (uint32_t)(k & 255) << (8 * (i & 3));
        k = av > 0.f ? exact_v(vi, av, 255.f * sqrt_ftz(root[i] * iv)) : 0;
        vc[i / 4] |= (uint32_t)(k & 255) << (8 * (i & 3));
      }
    }
    if (lane == 0) {
      e.ms[base / kBlk] = am;
      e.vs[base / kBlk] = av;
    }
  }
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int o = u * 128 + lane * 4, in = left - o;
    store4<WHOLE, float4, float>(e.p, base + o, in, p4[u]);
    if (BITS == 8) {
      store4<WHOLE, uint32_t, uint8_t>(e.m, base + o, in, mc[u]);
      store4<WHOLE, uint32_t, uint8_t>(e.v, base + o, in, vc[u]);
    } else {
      const float2 x0 = both(m[2 * u]), x1 = both(m[2 * u + 1]);
      const float2 y0 = both(v[2 * u]), y1 = both(v[2 * u + 1]);
      store4<WHOLE, float4, float>(e.m, base + o, in, make_float4(x0.x, x0.y, x1.x, x1.y));
      store4<WHOLE, float4, float>(e.v, base + o, in, make_float4(y0.x, y0.y, y1.x, y1.y));
    }
  }
}

// One warp takes a block of 256 elements, lane l elements 4 l .. 4 l + 3 and 128 + 4 l
// .. 128 + 4 l + 3, so that every load and store of a warp is contiguous.  Memory
// bound by 28 bytes per element with an fp32 state (41.9 M parameters in 448 tensors: 190
// us, 6.2 TB/s), 16 and two scales per block with 8 bits; there the arithmetic comes before
// it, hence the pairs, the flushing roots and the one branch for all borders of a thread:
// 150 us, 4.5 TB/s, 84 instructions an element at 65% of the issue slots (a hundred took 205
// us).  The loads are not what is waited for: with the next block brought in ahead, through
// shared memory, it took 153 us, and longer with one contiguous share of the blocks per CTA.
template <int BITS, int GBITS, int N>
__global__ void __launch_bounds__(kMtThreads, 4)
    adamw_multi_kernel(const __grid_constant__ MtArgs<N> a) {
  __shared__ float lm[BITS == 8 ? 256 : 1], lv[BITS == 8 ? 256 : 1];
  __shared__ float bc[2];
  __shared__ int off;
  pdl_trigger();
  if (BITS == 8) {
    lm[threadIdx.x] = level_m((int)(int8_t)threadIdx.x);  // by the code's byte
    lv[threadIdx.x] = level_v((int)threadIdx.x);
  }
  pdl_wait();
  if (threadIdx.x == 0) {
    float i1 = a.h.inv_bc1, i2 = a.h.inv_sqrt_bc2;
    if (a.h.step) {
      const double t = (double)max(1, *a.h.step);
      i1 = (float)(1.0 / (1.0 - pow((double)a.h.b1, t)));
      i2 = (float)(1.0 / sqrt(1.0 - pow((double)a.h.b2, t)));
    }
    bc[0] = i1;
    bc[1] = i2;
    off = a.h.gate ? *a.h.gate & DEV_ERR_INDEX : 0;
  }
  __syncthreads();
  if (off) return;
  const MtRates r{bc[0], bc[1]};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (uint32_t c = blockIdx.x; c < a.h.chunks; c += gridDim.x) {
    int lo = 0, hi = a.h.n - 1;  // the last tensor whose first chunk is at or before c
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (a.e[mid].chunk0 <= c)
        lo = mid;
      else
        hi = mid - 1;
    }
    const MtEntry& e = a.e[lo];
    const int64_t base = (int64_t)(c - e.chunk0) * kChunk + warp * kBlk;
    if (base >= e.n) continue;  // uniform in the warp
    const int left = (int)min((int64_t)kBlk, e.n - base);
    if (left == kBlk)
      adamw_block<BITS, GBITS, true>(a.h, e, r, lm, lv, base, left, lane);
    else
      adamw_block<BITS, GBITS, false>(a.h, e, r, lm, lv, base, left, lane);
  }
}

// Codes to values and back, for a state that is saved, loaded or inspected.
__global__ void __launch_bounds__(256)
    state_decode_kernel(const uint8_t* codes, const float* scale,
                        int64_t n, int is_signed, float* out) {
  __shared__ float lut[256];
  pdl_trigger();
  lut[threadIdx.x] = is_signed ? level_m((int)(int8_t)threadIdx.x) : level_v((int)threadIdx.x);
  pdl_wait();
  __syncthreads();
  // a warp takes 512 codes, lane l codes 4 l .. 4 l + 3 of each 128, so that loads and
  // stores of a warp are contiguous (memory bound: 5 bytes per value; 41.9 M values: 36 us,
  // 5.8 TB/s)
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * 8;
  for (int64_t b = ((int64_t)blockIdx.x * 8 + (threadIdx.x >> 5)) * 512; b < n; b += warps * 512) {
    if (b + 512 <= n) {
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        w[k] = reinterpret_cast<const uint32_t*>(codes + b + k * 128)[lane];
      const float a0 = scale[b / kBlk], a1 = scale[b / kBlk + 1];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float a = k < 2 ? a0 : a1;
        __stcs(reinterpret_cast<float4*>(out + b + k * 128) + lane,
               make_float4(a * lut[w[k] & 255u], a * lut[(w[k] >> 8) & 255u],
                           a * lut[(w[k] >> 16) & 255u], a * lut[w[k] >> 24]));
      }
    } else {
      for (int64_t i = b + lane; i < n; i += 32) out[i] = scale[i / kBlk] * lut[codes[i]];
    }
  }
}

__global__ void __launch_bounds__(256)
    state_encode_kernel(const float* x, int64_t n, int is_signed,
                        uint8_t* codes, float* scale, int* dev_err) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t blocks = (n + kBlk - 1) / kBlk;
  bool bad = false;
  for (int64_t b = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); b < blocks;
       b += (int64_t)gridDim.x * 8) {
    float f[8], top = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t at = b * kBlk + i * 32 + lane;
      f[i] = at < n ? x[at] : 0.f;
      // not a state: kept out of the block's scale, stored as 0
      if (!(fabsf(f[i]) <= 3.402823466e38f) || (!is_signed && f[i] < 0.f)) {
        f[i] = 0.f;
        bad = true;
      }
      top = fmaxf(top, fabsf(f[i]));
    }
    const float a = scale_of(__uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(top))));
    const float ia = a > 0.f ? is_signed ? __fdiv_rn(1.f, a) : inv_root(a) : 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t at = b * kBlk + i * 32 + lane;
      int c = 0;
      if (a > 0.f) {
        c = is_signed ? exact_m(fabsf(f[i]), a, 127.f * sqrt_ftz(fabsf(f[i]) * ia))
                      : exact_v(f[i], a, 255.f * sqrt_ftz(__fsqrt_rn(f[i]) * ia));
        if (is_signed && f[i] < 0.f) c = -c;
      }
      if (at < n) codes[at] = (uint8_t)c;
    }
    if (lane == 0) scale[b] = a;
  }
  if (bad) atomicOr(dev_err, DEV_ERR_NONFINITE);
}

template <int BITS, int GBITS, int N>
int mt_launch(const MtArgs<N>& a, cudaStream_t st) {
  // four CTAs of 256 threads are resident on an SM (64 registers a thread with 8 bits); twice
  // as many are launched, so that those of the second half take over as the first end, and
  // more chunks than that are taken in turn
  const uint32_t grid = std::min<uint32_t>(a.h.chunks, (uint32_t)gemm_num_sms() * 8);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kMtThreads);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  LSQ_CUDA(::lsq::launched(cudaLaunchKernelEx(&cfg, adamw_multi_kernel<BITS, GBITS, N>, a)));
  return LSQ_OK;
}

template <int N>
int mt_dispatch(const MtArgs<N>& a, int bits, int gbits, cudaStream_t st) {
  if (bits == 8) return gbits == 32 ? mt_launch<8, 32, N>(a, st) : mt_launch<8, 16, N>(a, st);
  return gbits == 32 ? mt_launch<32, 32, N>(a, st) : mt_launch<32, 16, N>(a, st);
}

// Launches the tensors [t0, t1) (t1 - t0 <= N, their chunks below 2^31).
template <int N>
int mt_run(const lsq_adamw_tensor* t, int t0, int t1, const MtHead& head, int bits, int gbits,
           cudaStream_t st) {
  MtArgs<N> a;
  a.h = head;
  a.h.n = 0;
  uint32_t c = 0;
  for (int i = t0; i < t1; ++i) {
    if (t[i].n == 0) continue;
    MtEntry& e = a.e[a.h.n++];
    e.p = t[i].p;
    e.g = t[i].g;
    e.m = t[i].m;
    e.v = t[i].v;
    e.ms = t[i].m_scale;
    e.vs = t[i].v_scale;
    e.n = t[i].n;
    e.lr = t[i].lr;
    e.wd = t[i].weight_decay;
    e.chunk0 = c;
    e.unused = 0;
    c += (uint32_t)((t[i].n + kChunk - 1) / kChunk);
  }
  a.h.chunks = c;
  if (c == 0) return LSQ_OK;
  return mt_dispatch<N>(a, bits, gbits, st);
}

bool finite(float x) { return std::isfinite(x); }

int check_tensors(const lsq_adamw_tensor* t, int n, int bits) {
  // overlapping parameters would be written twice: in address order each must end
  // before the next begins (a list that is in order already needs no sort)
  uintptr_t end = 0;
  bool ordered = true;
  for (int i = 0; i < n; ++i) {
    const lsq_adamw_tensor& x = t[i];
    if (x.n < 0 || x.n > (int64_t(1) << 40))
      return set_error(LSQ_ERR_SHAPE, "adamw_multi_step: tensor %d has %lld elements", i,
                       (long long)x.n);
    if (!finite(x.lr) || !finite(x.weight_decay) || x.lr < 0.f || x.weight_decay < 0.f)
      return set_error(LSQ_ERR_INVALID, "adamw_multi_step: tensor %d: lr and weight_decay must be "
                       "finite and not negative", i);
    if (x.n == 0) continue;
    if (!x.p || !x.g || !x.m || !x.v || (bits == 8 && (!x.m_scale || !x.v_scale)))
      return set_error(LSQ_ERR_INVALID, "adamw_multi_step: tensor %d has a null pointer", i);
    if (!aligned16(x.p) || !aligned16(x.g) || !aligned16(x.m) || !aligned16(x.v))
      return set_error(LSQ_ERR_ALIGN,
                       "adamw_multi_step: tensor %d: p, g, m and v must be 16-byte aligned", i);
    if (bits == 8 && (((uintptr_t)x.m_scale | (uintptr_t)x.v_scale) & 3u))
      return set_error(LSQ_ERR_ALIGN, "adamw_multi_step: tensor %d: scales must be 4-byte aligned",
                       i);
    const uintptr_t b = (uintptr_t)x.p;
    if (b < end) ordered = false;
    end = b + (uintptr_t)x.n * 4;
  }
  if (ordered) return LSQ_OK;
  std::vector<std::pair<uintptr_t, uintptr_t>> r;
  for (int i = 0; i < n; ++i)
    if (t[i].n) r.emplace_back((uintptr_t)t[i].p, (uintptr_t)t[i].p + (uintptr_t)t[i].n * 4);
  std::sort(r.begin(), r.end());
  for (size_t i = 1; i < r.size(); ++i)
    if (r[i].first < r[i - 1].second)
      return set_error(LSQ_ERR_INVALID, "adamw_multi_step: two tensors overlap");
  return LSQ_OK;
}

}  // namespace

int launch_adamw_multi(const lsq_adamw_tensor* t, int n, const lsq_adamw_hyper* o,
                       cudaStream_t st, const int* gate) {
  MtHead h = {};
  h.b1 = o->beta1;
  h.b2 = o->beta2;
  h.c1 = (float)(1.0 - (double)o->beta1);
  h.c2 = (float)(1.0 - (double)o->beta2);
  h.eps = o->eps;
  h.step = o->step_dev;
  h.gate = gate;
  if (!o->step_dev) {
    h.inv_bc1 = (float)(1.0 / (1.0 - pow((double)o->beta1, (double)o->step)));
    h.inv_sqrt_bc2 = (float)(1.0 / sqrt(1.0 - pow((double)o->beta2, (double)o->step)));
  }
  h.dev_err = device_status_ptr();
  if (!h.dev_err) return set_error(LSQ_ERR_CUDA, "device status word unavailable");
  double elems = 0;
  for (int i = 0; i < n; ++i) elems += (double)t[i].n;
  const int prof = prof_begin(st);
  for (int t0 = 0; t0 < n;) {
    int t1 = t0;
    int64_t chunks = 0;  // a launch takes at most kMtMany tensors and 2^31 chunks
    while (t1 < n && t1 - t0 < kMtMany) {
      const int64_t c = (t[t1].n + kChunk - 1) / kChunk;
      if (t1 > t0 && chunks + c > INT32_MAX) break;
      chunks += c;
      ++t1;
    }
    // the parameters of few tensors fit 4 KB
    LSQ_TRY(t1 - t0 <= kMtFew ? mt_run<kMtFew>(t, t0, t1, h, o->state_bits, o->grad_bits, st)
                              : mt_run<kMtMany>(t, t0, t1, h, o->state_bits, o->grad_bits, st));
    t0 = t1;
  }
  if (prof >= 0)
    prof_end(prof, st, "adamw_multi", 0.0,
             elems * (8.0 + o->grad_bits / 8.0 + (o->state_bits == 8 ? 4.0 + 16.0 / kBlk : 16.0)));
  return LSQ_OK;
}

}  // namespace lsq

using namespace lsq;

extern "C" int64_t adamw_scale_floats(int64_t n) { return n <= 0 ? 0 : (n + kBlk - 1) / kBlk; }

int lsq::check_adamw_multi(const lsq_adamw_tensor* tensors, int n_tensors,
                           const lsq_adamw_hyper* opt) {
  if (!opt || (!tensors && n_tensors > 0))
    return set_error(LSQ_ERR_INVALID, "adamw_multi_step: null pointer");
  if (n_tensors < 0) return set_error(LSQ_ERR_SHAPE, "adamw_multi_step: negative tensor count");
  if (opt->state_bits != 8 && opt->state_bits != 32)
    return set_error(LSQ_ERR_INVALID, "adamw_multi_step: state_bits must be 8 or 32");
  if (opt->grad_bits != 16 && opt->grad_bits != 32)
    return set_error(LSQ_ERR_INVALID, "adamw_multi_step: grad_bits must be 16 (bf16) or 32");
  if (!opt->step_dev && opt->step < 1)
    return set_error(LSQ_ERR_SHAPE, "adamw_multi_step: step counts from 1");
  if (!(opt->beta1 >= 0.f && opt->beta1 < 1.f) || !(opt->beta2 >= 0.f && opt->beta2 < 1.f) ||
      !(opt->eps >= 1.17549435e-38f) || !std::isfinite(opt->eps))
    return set_error(LSQ_ERR_INVALID,
                     "adamw_multi_step: need 0 <= beta < 1 and a finite eps of at least 2^-126");
  return check_tensors(tensors, n_tensors, opt->state_bits);
}

extern "C" int adamw_multi_step(const lsq_adamw_tensor* tensors, int32_t n_tensors,
                                const lsq_adamw_hyper* opt, void* stream) {
  LSQ_TRY(check_adamw_multi(tensors, n_tensors, opt));
  return launch_adamw_multi(tensors, n_tensors, opt, static_cast<cudaStream_t>(stream));
}

static int check_state(const void* codes, const void* scale, const void* x, int64_t n,
                       int32_t is_signed, const char* who) {
  if (n <= 0) return set_error(LSQ_ERR_SHAPE, "%s: n must be positive", who);
  if (is_signed != 0 && is_signed != 1)
    return set_error(LSQ_ERR_INVALID, "%s: is_signed must be 0 or 1", who);
  if (!codes || !scale || !x) return set_error(LSQ_ERR_INVALID, "%s: null pointer", who);
  if (!aligned16(codes) || !aligned16(x) || ((uintptr_t)scale & 3u))
    return set_error(LSQ_ERR_ALIGN, "%s: codes and values must be 16-byte aligned", who);
  return LSQ_OK;
}

extern "C" int adamw_state_dequantize(const void* codes, const float* scale, int64_t n,
                                      int32_t is_signed, float* out, void* stream) {
  LSQ_TRY(check_state(codes, scale, out, n, is_signed, "adamw_state_dequantize"));
  const int64_t want = (n + 4095) / 4096;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::max<int64_t>(1, std::min<int64_t>(want, gemm_num_sms() * 8)));
  cfg.blockDim = dim3(256);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  LSQ_CUDA(::lsq::launched(cudaLaunchKernelEx(&cfg, state_decode_kernel,
                                              static_cast<const uint8_t*>(codes), scale, n,
                                              (int)is_signed, out)));
  return LSQ_OK;
}

extern "C" int adamw_state_quantize(const float* x, int64_t n, int32_t is_signed, void* codes,
                                    float* scale, void* stream) {
  LSQ_TRY(check_state(codes, scale, x, n, is_signed, "adamw_state_quantize"));
  int* err = device_status_ptr();
  if (!err) return set_error(LSQ_ERR_CUDA, "device status word unavailable");
  const int64_t want = ((n + kBlk - 1) / kBlk + 7) / 8;
  state_encode_kernel<<<(unsigned)std::min<int64_t>(want, gemm_num_sms() * 8), 256, 0,
                        static_cast<cudaStream_t>(stream)>>>(
      x, n, is_signed, static_cast<uint8_t*>(codes), scale, err);
  LSQ_CUDA(::lsq::launched(cudaGetLastError()));
  return LSQ_OK;
}
