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
// The root is taken with the approximate square root, whose error moves it by less
// than kNear; only next to a border is the choice made again, in fp64.
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

__device__ __forceinline__ float sqrt_approx(float x) {
  float r;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Nearest integer to y = 127 sqrt(x / a), x >= 0, from an approximation of y; within
// 1e-4 of a border k + 1/2 the choice is x 254^2 against a (2 k + 1)^2 (both exact
// in fp64), a tie to the even code.
__device__ __forceinline__ int code_m(float x, float a, float inv_a) {
  const float y = 127.f * sqrt_approx(x * inv_a);
  int k = __float2int_rn(y);
  const float kb = floorf(y);
  if (fabsf(y - kb - 0.5f) < 1e-4f) {
    const int b = (int)kb;
    const double l = (double)x * 64516.0, r = (double)a * (double)((2 * b + 1) * (2 * b + 1));
    k = l > r ? b + 1 : l < r ? b : b + (b & 1);
  }
  return min(k, 127);
}

// Nearest integer to y = 255 (x / a)^(1/4), as above with x 510^4 against a (2 k + 1)^4.
__device__ __forceinline__ int code_v(float x, float a, float inv_a) {
  const float y = 255.f * sqrt_approx(sqrt_approx(x * inv_a));
  int k = __float2int_rn(y);
  const float kb = floorf(y);
  if (fabsf(y - kb - 0.5f) < 2e-4f) {
    const int b = (int)kb;
    const double o = (double)((2 * b + 1) * (2 * b + 1));
    const double l = (double)x * 67652010000.0, r = (double)a * (o * o);
    k = l > r ? b + 1 : l < r ? b : b + (b & 1);
  }
  k = min(k, 255);
  return x > 0.f ? max(k, 1) : k;
}

// The values the codes stand for: fl32(c |c| / 127^2) at c + 128, and fl32(q^4 / 255^4).
__device__ __forceinline__ float level_m(int c) {
  return __fdiv_rn((float)(c * abs(c)), 16129.f);
}
__device__ __forceinline__ float level_v(int q) {
  const double d = (double)(q * q);
  return (float)(d * d / 4228250625.0);
}

__device__ __forceinline__ float warp_max_pos(float x) {  // x >= 0: the bits order as the values
  return __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(x)));
}
// A block's scale: its largest magnitude, or 0 (every code 0) below the normal range.
__device__ __forceinline__ float scale_of(float top) { return top < 1.17549435e-38f ? 0.f : top; }

// One warp takes a block of 256 elements, lane l elements 4 l .. 4 l + 3 and 128 + 4 l
// .. 128 + 4 l + 3, so that every load and store of a warp is contiguous.  Memory
// bound: 28 bytes per element with an fp32 state, 16 and two scales per block with 8 bits.
template <int BITS, int GBITS, int N>
__global__ void __launch_bounds__(kMtThreads)
    adamw_multi_kernel(const __grid_constant__ MtArgs<N> a) {
  __shared__ float lm[BITS == 8 ? 256 : 1], lv[BITS == 8 ? 256 : 1];
  __shared__ float bc[2];
  pdl_trigger();
  if (BITS == 8) {
    lm[threadIdx.x] = level_m((int)threadIdx.x - 128);
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
  }
  __syncthreads();
  const float inv_bc1 = bc[0], isb2 = bc[1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  bool bad = false;
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
    const int64_t left = e.n - base;
    if (left <= 0) continue;  // uniform in the warp
    const float lr = e.lr, decay = 1.f - lr * e.wd, rate = lr * inv_bc1;
    float* __restrict__ pp = e.p + base;
    float p[8], g[8], m[8], v[8];
    const bool whole = left >= kBlk;
    float am = 0.f, av = 0.f;
    if (BITS == 8) {
      am = e.ms[base / kBlk];
      av = e.vs[base / kBlk];
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int o = h * 128 + lane * 4;
      if (whole) {
        const float4 x = *reinterpret_cast<const float4*>(pp + o);
        p[4 * h] = x.x; p[4 * h + 1] = x.y; p[4 * h + 2] = x.z; p[4 * h + 3] = x.w;
        if (GBITS == 32) {
          const float4 y = *reinterpret_cast<const float4*>(static_cast<const float*>(e.g) + base + o);
          g[4 * h] = y.x; g[4 * h + 1] = y.y; g[4 * h + 2] = y.z; g[4 * h + 3] = y.w;
        } else {
          const uint2 y =
              *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(e.g) + base + o);
          const float2 y0 = unpack_bf16x2(y.x), y1 = unpack_bf16x2(y.y);
          g[4 * h] = y0.x; g[4 * h + 1] = y0.y; g[4 * h + 2] = y1.x; g[4 * h + 3] = y1.y;
        }
        if (BITS == 8) {
          const char4 cm = *reinterpret_cast<const char4*>(static_cast<int8_t*>(e.m) + base + o);
          const uchar4 cv = *reinterpret_cast<const uchar4*>(static_cast<uint8_t*>(e.v) + base + o);
          m[4 * h] = am * lm[cm.x + 128]; m[4 * h + 1] = am * lm[cm.y + 128];
          m[4 * h + 2] = am * lm[cm.z + 128]; m[4 * h + 3] = am * lm[cm.w + 128];
          v[4 * h] = av * lv[cv.x]; v[4 * h + 1] = av * lv[cv.y];
          v[4 * h + 2] = av * lv[cv.z]; v[4 * h + 3] = av * lv[cv.w];
        } else {
          const float4 y = *reinterpret_cast<const float4*>(static_cast<float*>(e.m) + base + o);
          const float4 z = *reinterpret_cast<const float4*>(static_cast<float*>(e.v) + base + o);
          m[4 * h] = y.x; m[4 * h + 1] = y.y; m[4 * h + 2] = y.z; m[4 * h + 3] = y.w;
          v[4 * h] = z.x; v[4 * h + 1] = z.y; v[4 * h + 2] = z.z; v[4 * h + 3] = z.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool in = o + i < left;
          p[4 * h + i] = in ? pp[o + i] : 0.f;
          g[4 * h + i] = !in ? 0.f
                         : GBITS == 32
                             ? static_cast<const float*>(e.g)[base + o + i]
                             : bf16_bits_to_float(static_cast<const uint16_t*>(e.g)[base + o + i]);
          if (BITS == 8) {
            m[4 * h + i] = in ? am * lm[static_cast<int8_t*>(e.m)[base + o + i] + 128] : 0.f;
            v[4 * h + i] = in ? av * lv[static_cast<uint8_t*>(e.v)[base + o + i]] : 0.f;
          } else {
            m[4 * h + i] = in ? static_cast<float*>(e.m)[base + o + i] : 0.f;
            v[4 * h + i] = in ? static_cast<float*>(e.v)[base + o + i] : 0.f;
          }
        }
      }
    }
    float tm = 0.f, tv = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float m1 = __fadd_rn(__fmul_rn(a.h.b1, m[i]), __fmul_rn(a.h.c1, g[i]));
      const float v1 = __fadd_rn(__fmul_rn(a.h.b2, v[i]), __fmul_rn(__fmul_rn(a.h.c2, g[i]), g[i]));
      // a gradient whose moments leave the finite range changes nothing of its element
      if (fabsf(m1) <= 3.402823466e38f && v1 <= 3.402823466e38f) {
        m[i] = m1;
        v[i] = v1;
        p[i] = p[i] * decay - rate * __fdividef(m1, sqrt_approx(v1) * isb2 + a.h.eps);
      } else {
        bad = true;
      }
      tm = fmaxf(tm, fabsf(m[i]));
      tv = fmaxf(tv, v[i]);
    }
    int cm[8], cv[8];
    if (BITS == 8) {
      am = scale_of(warp_max_pos(tm));
      av = scale_of(warp_max_pos(tv));
      const float im = am > 0.f ? __fdiv_rn(1.f, am) : 0.f, iv = av > 0.f ? __fdiv_rn(1.f, av) : 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int k = am > 0.f ? code_m(fabsf(m[i]), am, im) : 0;
        cm[i] = m[i] < 0.f ? -k : k;
        cv[i] = av > 0.f ? code_v(v[i], av, iv) : 0;
      }
      if (lane == 0) {
        e.ms[base / kBlk] = am;
        e.vs[base / kBlk] = av;
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int o = h * 128 + lane * 4;
      if (whole) {
        *reinterpret_cast<float4*>(pp + o) =
            make_float4(p[4 * h], p[4 * h + 1], p[4 * h + 2], p[4 * h + 3]);
        if (BITS == 8) {
          *reinterpret_cast<char4*>(static_cast<int8_t*>(e.m) + base + o) =
              make_char4((signed char)cm[4 * h], (signed char)cm[4 * h + 1],
                         (signed char)cm[4 * h + 2], (signed char)cm[4 * h + 3]);
          *reinterpret_cast<uchar4*>(static_cast<uint8_t*>(e.v) + base + o) =
              make_uchar4((unsigned char)cv[4 * h], (unsigned char)cv[4 * h + 1],
                          (unsigned char)cv[4 * h + 2], (unsigned char)cv[4 * h + 3]);
        } else {
          *reinterpret_cast<float4*>(static_cast<float*>(e.m) + base + o) =
              make_float4(m[4 * h], m[4 * h + 1], m[4 * h + 2], m[4 * h + 3]);
          *reinterpret_cast<float4*>(static_cast<float*>(e.v) + base + o) =
              make_float4(v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (o + i >= left) continue;
          pp[o + i] = p[4 * h + i];
          if (BITS == 8) {
            static_cast<int8_t*>(e.m)[base + o + i] = (int8_t)cm[4 * h + i];
            static_cast<uint8_t*>(e.v)[base + o + i] = (uint8_t)cv[4 * h + i];
          } else {
            static_cast<float*>(e.m)[base + o + i] = m[4 * h + i];
            static_cast<float*>(e.v)[base + o + i] = v[4 * h + i];
          }
        }
      }
    }
  }
  if (bad) atomicOr(a.h.dev_err, DEV_ERR_NONFINITE);
}

// Codes to values and back, for a state that is saved, loaded or inspected.
__global__ void __launch_bounds__(256)
    state_decode_kernel(const uint8_t* __restrict__ codes, const float* __restrict__ scale,
                        int64_t n, int is_signed, float* __restrict__ out) {
  __shared__ float lut[256];
  pdl_trigger();
  lut[threadIdx.x] = is_signed ? level_m((int)(int8_t)threadIdx.x) : level_v((int)threadIdx.x);
  pdl_wait();
  __syncthreads();
  const int64_t n16 = n / 16;
  const int64_t step = (int64_t)gridDim.x * 256;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n16; i += step) {
    const uint4 c = reinterpret_cast<const uint4*>(codes)[i];
    const float a = __ldg(scale + (i >> 4));
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int k = 0; k < 4; ++k)
      reinterpret_cast<float4*>(out)[i * 4 + k] =
          make_float4(a * lut[w[k] & 255u], a * lut[(w[k] >> 8) & 255u],
                      a * lut[(w[k] >> 16) & 255u], a * lut[w[k] >> 24]);
  }
  if (blockIdx.x == 0 && threadIdx.x < n - n16 * 16) {
    const int64_t i = n16 * 16 + threadIdx.x;
    out[i] = scale[i / kBlk] * lut[codes[i]];
  }
}

__global__ void __launch_bounds__(256)
    state_encode_kernel(const float* __restrict__ x, int64_t n, int is_signed,
                        uint8_t* __restrict__ codes, float* __restrict__ scale, int* dev_err) {
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
    const float a = scale_of(warp_max_pos(top));
    const float ia = a > 0.f ? __fdiv_rn(1.f, a) : 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t at = b * kBlk + i * 32 + lane;
      int c = 0;
      if (a > 0.f) {
        c = is_signed ? code_m(fabsf(f[i]), a, ia) : code_v(f[i], a, ia);
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
  // eight CTAs of 256 threads fill an SM; more chunks than that are taken in turn
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
                       cudaStream_t st) {
  MtHead h = {};
  h.b1 = o->beta1;
  h.b2 = o->beta2;
  h.c1 = (float)(1.0 - (double)o->beta1);
  h.c2 = (float)(1.0 - (double)o->beta2);
  h.eps = o->eps;
  h.step = o->step_dev;
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

extern "C" int adamw_multi_step(const lsq_adamw_tensor* tensors, int32_t n_tensors,
                                const lsq_adamw_hyper* opt, void* stream) {
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
      !(opt->eps > 0.f) || !std::isfinite(opt->eps))
    return set_error(LSQ_ERR_INVALID,
                     "adamw_multi_step: need 0 <= beta < 1 and a positive finite eps");
  LSQ_TRY(check_tensors(tensors, n_tensors, opt->state_bits));
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
  const int64_t want = (n / 16 + 255) / 256;
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
