// Attention inside packed documents, forward and backward: o = softmax(q k^T / sqrt(d)) v
// over the keys of a token's own document up to itself, or up to the end of the
// document's prompt, which is read in both directions.  Query head h reads kv head
// h / (H / Hkv).
//
// The work is split into tiles of at most 128 tokens of ONE document (the index lists
// them), so no product ever mixes two documents: a tile's rows all see one range of
// keys, masked only along the diagonal and behind the document's end, and what another
// document or the padding holds, infinities included, stays out.  Rows of a loaded tile
// behind that range are cleared in shared memory before a product reduces over them.
//
// All products run as tcgen05.mma from 128-byte-swizzled shared-memory tiles (TMA)
// into TMEM accumulators, fp16 operands and fp32 sums throughout.  The gradient of the
// output arrives in bf16, whose range fp16 lacks: its rows are scaled by powers of two
// first (dO' = 2^e dO with a largest magnitude in [1, 2); exact down to 2^-17 of it, and off
// by 2^-25 at most below), and the factors are taken out again in fp32.  The probabilities and
// score gradients that the backward rounds to fp16 are scaled towards the top of its range,
// the latter by what the norms of v allow, so that small ones keep their bits.  Every sum has
// a fixed order, so the results are deterministic.
#include <cuda.h>
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "packed.cuh"

namespace lsq {

namespace {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ uint8_t* align1024_p(uint8_t* p) {
  return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(p) + 1023) & ~uintptr_t(1023));
}

// 2^x (relative error 2^-22; results below 2^-126 are 0)
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Two fp32 operations at a time (each rounded as the single ones are).
__device__ __forceinline__ uint64_t pack_f32x2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpack_f32x2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// 32 bytes of a row (a whole sector) in one store: rows are written by a lane each, and
// two 16-byte halves of a sector cost two passes of the store path (an output tile of
// 128 x 128 took 3000 to 6500 cycles to write that way).
__device__ __forceinline__ void st_global32(void* p, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// ------------------------------------------------------------------ forward
// A persistent CTA per SM takes work items in turn.  An item is two streams of 128
// query rows of one document that read the same K and V tiles: two query heads of a kv
// head on the same rows where the group has an even number of heads, else two
// neighbouring row tiles of one head.  A stream goes through its keys in steps of 64:
//   S = Q_s K^T (TMEM) -> softmax warps of the stream: P = exp2(S c - m) as fp16 over
//   the same TMEM columns -> O_s += P V (A operand from TMEM).
// Two score buffers a stream let the products of step u + 2 and P V of step u run while
// the softmax of step u + 1 does, so that neither waits for the other's latency.
// The reference maximum m of a row moves only when a tile's maximum exceeds it by more
// than 2^8 (then O and the running sum are rescaled): the result is exact for any
// reference, and P stays below 2^8, well inside fp16.
//   warps 0-3, 4-7: softmax and epilogue of streams 0 and 1, a query row per thread
//   warp 8 : TMA producer (Q of each stream; a ring of K and V tiles)
//   warps 9, 10: the MMA issuers of streams 0 and 1 (warp 9 also allocates TMEM); one
//            warp for both left the tensor cores idle for the 300 to 800 cycles that its
//            waits took between the products of one stream and the other's
//   warp 11: clears the rows of a document's last V tile that lie behind its end
// Tensor bound by count: 4 d FLOP per pair and head; a step of both streams needs 1240
// cycles of products (measured alone: 48 cycles for a 128 x 64 x 16 product from shared
// memory, 64 for a 128 x 128 x 16 one with A from TMEM) and 1024 of exponentials, and takes
// 1770, in which the softmax threads are busy throughout.  One document of 16,384 tokens
// (32/8 heads, d 128): 2.25 ms in repeated calls, 980 TFLOP/s, the power limit holding the
// clock down (1.9 ms and 1150 for a few calls of a cool chip); 16,384 tokens in 34 documents
// (16/2): 108 us; 512 tokens: 10 us.
// Measured and set aside: polynomials for part of the exponentials (slower by 7%), steps of
// 128 keys with one buffer, the streams' exponentials made to alternate (1830 cycles), and
// the row maximum taken from the probabilities behind them (no change).
constexpr int kAQ = 128;   // queries per stream (UMMA M)
constexpr int kAK = 128;   // keys per K or V tile
constexpr int kStep = 64;  // keys per step (UMMA N of S, K of P V)
constexpr int kFThreads = 384;
constexpr int kWarpTma = 8, kWarpMma = 9, kWarpTail = 11;
constexpr float kRescaleLog2 = 8.f;

template <int D>
struct FwdSmem {
  static constexpr int DA = D / 64;                  // 64-element swizzle atoms along d
  static constexpr uint32_t kTile = 128 * D * 2;     // a tile of 128 rows of Q, K or V
  static constexpr int kRing = D == 128 ? 4 : 8;     // K and V tiles in flight
  static constexpr uint32_t kStage = 32 * 128;       // 32 rows of 64 columns of o, for each warp
  static constexpr uint32_t kBytes = 1024 + (2 + kRing) * kTile + 8 * kStage;
};

// Key steps of the rows [row, row + 128) of a tile's document (0: no such rows).
__device__ __forceinline__ int key_steps(const PackedTile& t, int row) {
  if (row >= t.end) return 0;
  return (min(t.end, max(row + kAQ, t.prompt)) - t.begin + kStep - 1) / kStep;
}
// Item of this CTA in round k: the items, heaviest first, are dealt forth and back, so
// that no CTA gets the heavier one every time; -1 behind the last.
__device__ __forceinline__ int deal(int k, int items) {
  const int w = k * (int)gridDim.x +
                ((k & 1) ? (int)(gridDim.x - 1 - blockIdx.x) : (int)blockIdx.x);
  return w < items ? w : -1;
}
// An item as stream s sees it: its first row, head and number of steps (0: none), and
// the steps of the longer stream.
struct FwdItem {
  int begin, end, prompt;
  int row, head, n, nu;
};
__device__ __forceinline__ FwdItem fwd_item(const PackedIndex& x, int w, int H, bool heads, int s) {
  FwdItem it;
  const int per = heads ? H / 2 : H;
  const PackedTile t = (heads ? x.tiles : x.tiles2)[w / per];
  it.begin = t.begin;
  it.end = t.end;
  it.prompt = t.prompt;
  it.head = heads ? 2 * (w % per) + s : w % per;
  it.row = heads ? t.row0 : t.row0 + s * kAQ;
  it.n = key_steps(t, it.row);
  it.nu = heads ? it.n : max(key_steps(t, t.row0), key_steps(t, t.row0 + kAQ));
  return it;
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
// The MMA warp runs its loop as a whole, so that the compiler sees uniform values and
// keeps descriptors in uniform registers; `lead` is nonzero in the one lane that issues.
// (With the loop inside a one-lane branch each product cost a dozen dependent
// instructions, and the issuing lane, not the tensor cores, set the pace.)
__device__ __forceinline__ uint32_t elect_lane() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r;
}
// D[tmem] (+)= A[smem] * B[smem]^T
__device__ __forceinline__ void mma_ss(uint32_t lead, uint32_t d_tmem, uint64_t adesc,
                                       uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem]^T: A holds two 16-bit elements per 32-bit column.
__device__ __forceinline__ void mma_ts(uint32_t lead, uint32_t d_tmem, uint32_t a_tmem,
                                       uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t lead, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          bar),
      "r"(lead)
      : "memory");
}

// Padding rows (behind the last document) hold no document: o = 0, lse = -inf.  The
// whole grid shares them.
template <int D>
__device__ __forceinline__ void fill_padding(int first, int64_t T, int H, uint16_t* out,
                                             float* lse_out) {
  const int64_t step = (int64_t)gridDim.x * blockDim.x;
  const int64_t i0 = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int64_t n = (T - first) * H * (D / 8);
  uint4* o = reinterpret_cast<uint4*>(out + (int64_t)first * H * D);
  for (int64_t i = i0; i < n; i += step) o[i] = make_uint4(0u, 0u, 0u, 0u);
  for (int64_t i = i0; i < (T - first) * H; i += step)
    lse_out[(i % H) * T + first + i / H] = -INFINITY;
}

// Clears rows [rows, all) of a swizzled tile of D columns (one warp).
template <int D>
__device__ __forceinline__ void zero_rows(uint8_t* tile, int rows, int all, int lane) {
  for (int a = 0; a < D / 64; ++a)
    for (uint32_t o = (uint32_t)rows * 128u + (uint32_t)lane * 16u; o < (uint32_t)all * 128u;
         o += 512u)
      *reinterpret_cast<uint4*>(tile + (uint32_t)a * all * 128u + o) = make_uint4(0u, 0u, 0u, 0u);
}

template <int D>
__global__ void __launch_bounds__(kFThreads, 1)
    packed_attn_fwd_kernel(const __grid_constant__ CUtensorMap tm_qkv,
                           const __grid_constant__ CUtensorMap tm_o,  // o, boxes of 32 rows
                           PackedIndex idx, int64_t T, int H, int Hkv, uint16_t* out,
                           float* lse_out, float sl2, int* dev_err) {
  using SM = FwdSmem<D>;
  constexpr int DA = SM::DA, NR = SM::kRing;
  extern __shared__ uint8_t attn_raw[];
  __shared__ __align__(8) uint64_t q_full[2], q_free[2], kv_full[NR], kv_free[NR];
  __shared__ __align__(8) uint64_t s_full[2][2], p_full[2][2], pv_done[2];
  __shared__ __align__(8) uint64_t o_full[2], o_free[2];
  __shared__ __align__(8) uint64_t tail_done[NR];
  __shared__ uint32_t tmem_sh;
  __shared__ int abort_sh;
  volatile int* abort_flag = &abort_sh;

  uint8_t* Qs = align1024_p(attn_raw);   // [2] Q tiles
  uint8_t* KV = Qs + 2 * SM::kTile;      // ring: K and V tiles in turn
  uint8_t* Os = KV + NR * SM::kTile;     // [8] staging of the softmax warps
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr uint32_t kColS = 0, kColO = 256;  // TMEM: S[stream][buffer] from 0, O at 256 and 384
  const int G = H / Hkv;
  const bool heads = G % 2 == 0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&q_full[i]), 1);
      mbar_init(smem_u32(&q_free[i]), 1);
      for (int b = 0; b < 2; ++b) {
        mbar_init(smem_u32(&s_full[i][b]), 1);
        mbar_init(smem_u32(&p_full[i][b]), 4);
      }
      mbar_init(smem_u32(&pv_done[i]), 1);
      mbar_init(smem_u32(&o_full[i]), 1);
      mbar_init(smem_u32(&o_free[i]), 4);
    }
    for (int i = 0; i < NR; ++i) {
      mbar_init(smem_u32(&kv_full[i]), 1);
      mbar_init(smem_u32(&kv_free[i]), 3);  // the two streams' products and the tail warp
      mbar_init(smem_u32(&tail_done[i]), 1);
    }
    abort_sh = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == kWarpMma) {
    tmem_alloc(smem_u32(&tmem_sh), 512);
    tmem_relinquish();
  }
  if (warp == kWarpTma && lane == 0) {
    tma_prefetch_desc(&tm_qkv);
    tma_prefetch_desc(&tm_o);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_sh;
  pdl_trigger();  // the next kernel may launch once all CTAs of this one run and have their TMEM
  pdl_wait();     // the index and q, k, v come from the kernels before
  const int items = heads ? idx.head[0] * (H / 2) : idx.head[1] * H;
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    return mbar_wait_short(smem_u32(bar), parity & 1u, abort_flag, dev_err);
  };

  // the same by a whole warp, which leaves it together: a lane that fell behind could
  // miss a phase
  auto wait_all = [&](uint64_t* bar, uint32_t parity) -> bool {
    return __all_sync(0xFFFFFFFFu, wait(bar, parity));
  };

  if (warp == kWarpTma) {
    // ---------------------------------------------------------------- TMA producer
    if (lane == 0) {
      uint32_t c = 0, nq[2] = {0, 0};  // ring tiles and Q tiles issued
      bool ok = true;
      auto load_kv = [&](int col, int row) -> bool {
        const uint32_t slot = c % NR;
        if (c >= NR && !wait(&kv_free[slot], c / NR - 1)) return false;
        const uint32_t fb = smem_u32(&kv_full[slot]);
        mbar_arrive_expect_tx(fb, SM::kTile);
        for (int a = 0; a < DA; ++a)
          tma_load_2d(smem_u32(KV + slot * SM::kTile + a * kAK * 128), &tm_qkv, fb, col + 64 * a, row);
        ++c;
        return true;
      };
      for (int k = 0, w; ok && (w = deal(k, items)) >= 0; ++k) {
        const FwdItem it = fwd_item(idx, w, H, heads, 0), it1 = fwd_item(idx, w, H, heads, 1);
        const int g = it.head / G;
        const int kc = (H + g) * D, vc = (H + Hkv + g) * D;
        const int n = (it.nu + 1) / 2;  // K and V tiles
        ok = load_kv(kc, it.begin) && load_kv(vc, it.begin);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (!ok || (s == 1 && it1.n == 0)) continue;
          if (nq[s] > 0) ok = wait(&q_free[s], nq[s] - 1);
          if (!ok) continue;
          ++nq[s];
          const uint32_t fb = smem_u32(&q_full[s]);
          mbar_arrive_expect_tx(fb, SM::kTile);
          for (int a = 0; a < DA; ++a)
            tma_load_2d(smem_u32(Qs + s * SM::kTile + a * kAQ * 128), &tm_qkv, fb,
                        (s ? it1.head : it.head) * D + 64 * a, s ? it1.row : it.row);
        }
        for (int j = 1; j < n && ok; ++j)
          ok = load_kv(kc, it.begin + j * kAK) && load_kv(vc, it.begin + j * kAK);
      }
    }
    __syncwarp();
  } else if (warp == kWarpMma || warp == kWarpMma + 1) {
    // ---------------------------------------------------------------- MMA issuers
    const int s = warp - kWarpMma;
    const uint32_t lead = elect_lane();
    const uint32_t idesc_s = umma_idesc_f16(kAQ, kStep);
    const uint32_t idesc_o = umma_idesc_f16(kAQ, D) | (1u << 16);  // B (V) MN-major
    const uint32_t ts = tmem + kColS + (uint32_t)s * 128, to = tmem + kColO + (uint32_t)s * 128;
    const uint64_t qd = umma_desc_k_sw128(smem_u32(Qs + s * SM::kTile));
    uint32_t c = 0, tails = 0;     // ring tiles; phase of each slot's tail_done
    uint32_t ni = 0;               // items of this stream
    uint32_t ns[2] = {0, 0};       // steps of each buffer
    bool ok = true;
    auto issue_s = [&](int b, uint32_t ck) {  // buffer b = the half of the K tile at ring count ck
      const uint64_t kd = umma_desc_k_sw128(smem_u32(KV + (ck % NR) * SM::kTile) +
                                            (uint32_t)b * kStep * 128u);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        constexpr uint32_t kAtom = 128 * 128 / 16;
        const uint32_t off = (uint32_t)(kk >> 2) * kAtom + (uint32_t)(kk & 3) * 2;
        mma_ss(lead, ts + (uint32_t)(b * kStep), qd + off, kd + off, idesc_s, kk > 0 ? 1u : 0u);
      }
      mma_commit(lead, smem_u32(&s_full[s][b]));
    };
    for (int k = 0, w; ok && (w = deal(k, items)) >= 0; ++k) {
      const FwdItem it = fwd_item(idx, w, H, heads, s);
      const int n = (it.nu + 1) / 2;
      const bool tail = it.begin + n * kAK > it.end;
      ok = wait_all(&kv_full[c % NR], c / NR);
      if (ok && it.n > 0) {
        ok = wait_all(&q_full[s], ni);
        if (!ok) break;
        tc_fence_after();
        issue_s(0, c);
        if (it.n > 1) issue_s(1, c);
        if (it.n <= 2) mma_commit(lead, smem_u32(&q_free[s]));
        // O of the stream's previous item has been read
        if (ni > 0) ok = wait_all(&o_free[s], ni - 1);
        ++ni;
      }
      if (ok) mma_commit(lead, smem_u32(&kv_free[c % NR]));
      for (int j = 0; j < n && ok; ++j) {
        const uint32_t cv = c + 2 * j + 1, ck = cv + 1;
        const uint64_t vd = umma_desc_mn_sw128(smem_u32(KV + (cv % NR) * SM::kTile),
                                               (uint32_t)(kAK * 128), 1024u);
        ok = wait_all(&kv_full[cv % NR], cv / NR);
        if (ok && tail && j == n - 1) ok = wait_all(&tail_done[cv % NR], tails >> (cv % NR));
        if (ok && j + 1 < n) ok = wait_all(&kv_full[ck % NR], ck / NR);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const int u = 2 * j + b;
          if (!ok || u >= it.n) continue;
          // P written (and O rescaled if its reference maximum moved)
          ok = wait_all(&p_full[s][b], ns[b]);
          if (!ok) continue;
          ++ns[b];
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < kStep / 16; ++kk)
            mma_ts(lead, to, ts + (uint32_t)(b * kStep + kk * 8),
                   vd + (uint32_t)((b * kStep + kk * 16) * 128 / 16), idesc_o,
                   (u > 0 || kk > 0) ? 1u : 0u);
          mma_commit(lead, smem_u32(&pv_done[s]));
          if (u + 2 < it.n) issue_s(b, ck);
          if (u + 3 == it.n) mma_commit(lead, smem_u32(&q_free[s]));  // the last scores
          if (u + 1 == it.n) mma_commit(lead, smem_u32(&o_full[s]));
        }
        if (!ok) break;
        mma_commit(lead, smem_u32(&kv_free[cv % NR]));
        if (j + 1 < n) mma_commit(lead, smem_u32(&kv_free[ck % NR]));
      }
      if (tail) tails ^= 1u << ((c + 2 * n - 1) % NR);
      c += 2 * n;
    }
  } else if (warp == kWarpTail) {
    // It follows every tile of the ring (so that it never falls a phase behind) and
    // gives each slot free again together with the products.
    uint32_t c = 0;
    bool ok = true;
    for (int k = 0, w; ok && (w = deal(k, items)) >= 0; ++k) {
      const FwdItem it = fwd_item(idx, w, H, heads, 0);
      const int n = (it.nu + 1) / 2;
      for (int i = 0; i < 2 * n && ok; ++i, ++c) {
        const uint32_t slot = c % NR;
        ok = wait_all(&kv_full[slot], c / NR);
        if (ok && i == 2 * n - 1 && it.begin + n * kAK > it.end) {
          // V rows behind the document belong to another one or to the padding:
          // cleared, since 0 * inf would reach this document's rows
          zero_rows<D>(KV + slot * SM::kTile, it.end - it.begin - (n - 1) * kAK, kAK, lane);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&tail_done[slot]));
        }
        if (lane == 0) mbar_arrive(smem_u32(&kv_free[slot]));
      }
    }
  } else {
    // ---------------------------------------------------------------- softmax (warps 0-7)
    const int s = warp >> 2;
    const int r = (warp & 3) * 32 + lane;  // query row of the stream = TMEM lane
    const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t to = trow + kColO + (uint32_t)s * 128;
    uint32_t ns[2] = {0, 0}, nv = 0, no = 0;  // steps of each buffer, P V products, items
    const uint64_t sl22 = pack_f32x2(sl2, sl2);
    bool ok = true;
    int w = deal(0, items);
    FwdItem it;
    if (w >= 0) it = fwd_item(idx, w, H, heads, s);
    for (int k = 1; ok && w >= 0; ++k) {
      // (the next item is looked up while this one's last product runs)
      const int w1 = deal(k, items);
      const int n = it.n;
      if (n == 0) {
        w = w1;
        if (w >= 0) it = fwd_item(idx, w, H, heads, s);
        continue;
      }
      const int q = it.row + r;
      const int kmax = min(max(q, it.prompt - 1), it.end - 1);  // the row's last key
      const int kall = min(max(it.row + (warp & 3) * 32, it.prompt - 1), it.end - 1);
      float m_ref = -INFINITY, l_run = 0.f;
#pragma unroll 2
      for (int u = 0; u < n; ++u) {
        const uint32_t ts = trow + kColS + (uint32_t)(s * 128 + (u & 1) * kStep);
        ok = wait_all(&s_full[s][u & 1], ns[u & 1]);
        if (!ok) break;
        ++ns[u & 1];
        tc_fence_after();
        uint32_t sv[kStep];
        tmem_ld32(ts, sv);
        tmem_ld32(ts + 32, sv + 32);
        tmem_ld_wait();
        const int k0 = it.begin + u * kStep;
        if (k0 + kStep - 1 > kall) {  // (uniform in the warp)
          const int last = kmax - k0;
#pragma unroll
          for (int e = 0; e < kStep; ++e)
            if (e > last) sv[e] = 0xFF800000u;  // -inf
        }
        float mt = -INFINITY, mt1 = -INFINITY;
#pragma unroll
        for (int e = 0; e < kStep; e += 4) {
          mt = fmaxf(fmaxf(mt, __uint_as_float(sv[e])), __uint_as_float(sv[e + 1]));
          mt1 = fmaxf(fmaxf(mt1, __uint_as_float(sv[e + 2])), __uint_as_float(sv[e + 3]));
        }
        mt = fmaxf(mt, mt1) * sl2;
        float corr = 1.f;
        bool moved = false;
        if (u == 0) {
          m_ref = mt;  // (finite for finite scores: every row sees its document's first key)
        } else if (mt > m_ref + kRescaleLog2) {
          corr = exp2f(m_ref - mt);
          m_ref = mt;
          l_run *= corr;
          moved = true;
        }
        if (__any_sync(0xFFFFFFFFu, moved)) {
          // the product before this step has written O (the one before that has, since
          // this step's scores were computed behind it)
          ok = wait_all(&pv_done[s], nv + u - 1);
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < D / 16; ++c) {
            uint32_t v[16];
            tmem_ld16(to + 16 * c, v);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * corr);
            tmem_st16(to + 16 * c, v);
          }
        }
        // P = exp2(s sl2 - m_ref) in fp16 (masked scores are -inf, so their p is 0) over
        // the scores' own columns, and the row sum
        const uint64_t nm2 = pack_f32x2(-m_ref, -m_ref);
        uint64_t rs = 0;  // (0, 0)
#pragma unroll
        for (int c = 0; c < kStep / 32; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float2 x = unpack_f32x2(fma_f32x2(
                pack_f32x2(__uint_as_float(sv[32 * c + e]), __uint_as_float(sv[32 * c + e + 1])),
                sl22, nm2));
            const float p0 = ex2(x.x), p1 = ex2(x.y);
            rs = add_f32x2(rs, pack_f32x2(p0, p1));
            pk[e >> 1] = pack_f16x2(p0, p1);
          }
          tmem_st16(ts + 16 * c, pk);
        }
        const float2 rsum = unpack_f32x2(rs);
        l_run += rsum.x + rsum.y;
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&p_full[s][u & 1]));
      }
      // -------------------------------------------------------------- epilogue
      // (a barrier of its own: pv_done may be two phases on, where a wait for the
      // phase before the last would not return)
      const bool live = q < it.end;
      const int wrow = it.row + (warp & 3) * 32, ocol = it.head * D;
      const bool whole = wrow + 32 <= it.end;  // (uniform in the warp)
      uint16_t* orow = out + (int64_t)q * H * D + (int64_t)it.head * D;
      float* lrow = lse_out + (int64_t)it.head * T + q;
      w = w1;
      if (w >= 0) it = fwd_item(idx, w, H, heads, s);
      ok = ok && wait_all(&o_full[s], no);
      if (!ok) break;
      ++no;
      nv += n;
      tc_fence_after();
      const float inv = 1.f / l_run;
      uint32_t ov[D];
#pragma unroll
      for (int c = 0; c < D / 32; ++c) tmem_ld32(to + 32 * c, ov + 32 * c);
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&o_free[s]));
      // A whole warp's rows go through its slice of shared memory to a bulk store, which
      // runs while the warp goes on: stored by the threads, each its own row 32 bytes at a
      // time, a tile took 3000 to 4500 cycles, a quarter of an item of 512 tokens (the
      // store path takes a request per row and sector).  Rows next to a document's end are
      // stored that way, since the bulk store would write those behind it.
      // Behind the CTA's last item the stream's Q tile is free too, and takes both halves.
      if (whole) {
        uint8_t* slice = w1 < 0 ? Qs + s * SM::kTile + (warp & 3) * DA * SM::kStage
                                : Os + warp * SM::kStage;
#pragma unroll
        for (int a = 0; a < DA; ++a) {
          if (w1 >= 0) {
            if (lane == 0) bulk_wait_read<0>();  // the slice's last store has read it
            __syncwarp();
          } else if (a > 0) {
            slice += SM::kStage;
          }
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const uint32_t* x = ov + 64 * a + 8 * c;
            uint32_t pk[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              pk[e] = pack_f16x2(__uint_as_float(x[2 * e]) * inv, __uint_as_float(x[2 * e + 1]) * inv);
            *reinterpret_cast<uint4*>(slice + lane * 128 + ((c ^ (lane & 7)) << 4)) =
                make_uint4(pk[0], pk[1], pk[2], pk[3]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&tm_o, smem_u32(slice), ocol + 64 * a, wrow);
            bulk_commit();
          }
        }
      } else if (live) {
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          uint32_t pk[8];
#pragma unroll
          for (int e = 0; e < 8; ++e)
            pk[e] = pack_f16x2(__uint_as_float(ov[16 * c + 2 * e]) * inv,
                               __uint_as_float(ov[16 * c + 2 * e + 1]) * inv);
          st_global32(orow + 16 * c, pk);
        }
      }
      if (live) *lrow = (m_ref + log2f(l_run)) * 0.69314718055994531f;
    }
    if (lane == 0) bulk_wait_all();
  }
  fill_padding<D>(idx.head[2], T, H, out, lse_out);

  // ------------------------------------------------------------------ teardown
  tc_fence_before();
  __syncthreads();
  if (abort_sh) settle_ns(2000000);  // let issued copies and MMAs land before freeing TMEM
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ backward
// Items of two kinds recompute the probabilities, p = exp2(s c - lse log2 e), and form
// ds = p (dp - delta) with delta = rowsum(dO o O): one kind owns keys (dK, dV), the other
// queries (dQ), so that no sum is shared between CTAs and none depends on their order.
// Both go through the other side in chunks of 64, keep P and dS in TMEM as fp16 A operands
// over the columns they come from, and split the issuing of products between two warps.
// One persistent kernel takes them all, a CTA its dK, dV items first, so that SMs that
// find none left go on with dQ while others still work on theirs.  (As two kernels, the
// second may read what the preparation wrote only when the first is done: backward of 512
// tokens in 5 documents (32/8 heads, d 128) took 36 us so against 30, of 16,384 in 34 (16/2)
// 268 against 257.)
//   warps 0-15: the gradient warps, four groups of four (a TMEM lane per thread): groups 0
//            and 2 take the two halves of the columns of one set (or stream), 1 and 3 of
//            the other.  (With two groups of whole rows a chunk took a thread 3700 cycles,
//            latency more than work: the products of two chunks need 2560.)
//   warp 16: TMA producer;  warps 17, 18: MMA issuers (warp 17 also allocates TMEM)
//   warp 19: clears rows behind a document's end, and (dK, dV) stages the queries' values
// The prepared values of a query and head: dO' = 2^e dO in fp16, its largest in [1, 2),
// e, delta' = 2^e delta and l = lse log2 e + e; of a key and kv head: |v|^2.
constexpr int kBC = 64;        // columns of a chunk (queries for dK/dV, keys for dQ)
constexpr int kBH = kBC / 2;   // columns of a thread
constexpr int kBThreads = 640;
constexpr int kBTma = 16, kBMma = 17, kBTail = 19;
constexpr int kWindow = 64;    // tokens of a window of the exponents' minima
// Items are handed out as CTAs come for them, heaviest first, the dQ items behind those of
// dK and dV: the TMA producer draws the next one from a counter (zeroed by the kernel that
// prepares dO') and passes it to the other 19 warps through a ring in shared memory.  What
// an item computes does not depend on who takes it.  (Dealt out beforehand, CTAs that come
// to dQ last, behind the longest dK, dV items, kept as large a share as the others.)
constexpr int kTake = 4;
constexpr int kTakers = 19;
// The exponent a for which |dP' - delta'| 2^a stays below 2^15, half of fp16's range, given
// the largest |v|^2 among the keys: |dP' - delta'| <= 2 |dO'| |v| < 4 sqrt(d) |v|.  Held where
// 2^(-e - a), which takes it out again beside 2^e, is a normal number.
constexpr int kUp = 15;
__device__ __forceinline__ int ds_exponent(float nv, int d, int e) {
  const int x = (int)(__float_as_uint(16.f * (float)d * nv) >> 23) - 126;  // 16 d |v|^2 < 2^x
  return max(min(kUp - ((x + 1) >> 1), 126 - e), -127 - e);
}
__device__ __forceinline__ float pow2i(int x) { return __int_as_float((127 + x) << 23); }
__device__ __forceinline__ float warp_min(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fminf(x, __shfl_xor_sync(0xFFFFFFFFu, x, o));
  return x;
}

// The largest |v|^2 of the keys [begin, end): whole windows by their maxima, the edges row by
// row (a window that reaches into another document must not count).  A lane's share; most
// documents take one round of loads.
__device__ __forceinline__ float largest_norm(const float* winnorm, const float* rownorm, int begin,
                                              int end, int lane) {
  const int w0 = (begin + kWindow - 1) / kWindow, w1 = end / kWindow;
  const int e0 = w0 < w1 ? w0 * kWindow : end, e1 = w0 < w1 ? w1 * kWindow : end;
  const int q = begin + lane, u = e1 + lane;
  const float a = w0 + lane < w1 ? winnorm[w0 + lane] : 0.f;
  const float b = q < e0 ? rownorm[q] : 0.f, c = q + 32 < e0 ? rownorm[q + 32] : 0.f;
  const float d = u < end ? rownorm[u] : 0.f, e = u + 32 < end ? rownorm[u + 32] : 0.f;
  float n = fmaxf(fmaxf(fmaxf(a, b), fmaxf(c, d)), e);
  for (int i = w0 + 32 + lane; i < w1; i += 32) n = fmaxf(n, winnorm[i]);
  for (int i = q + 64; i < e0; i += 32) n = fmaxf(n, rownorm[i]);
  return n;
}
__device__ __forceinline__ float warp_most(float x) {  // (of numbers that are not negative)
  return __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(x)));
}

// One CTA per window of 64 tokens and head; D / 8 lanes take a row, 16 bytes each, and a
// warp its eight tokens with all loads in flight (memory bound: 6 bytes per element).
// blockIdx.y >= H: the squared norms of the v rows of kv head blockIdx.y - H (0 for one that
// is not finite, which is latched: what it reaches is not finite whatever the scale).  e
// brings the row's largest magnitude to [1, 2), so its norm is below 2 sqrt(d).  A zero row
// takes e = 127 (it must not lower the least exponent of a tile); a row that is not finite
// takes e = 0, and its gradients come out not finite.  16,384 tokens of 16 heads, d 128: 38
// us, 5.3 TB/s (41 with the 64 registers a thread that the compiler takes by itself, and
// spills).
template <int D>
__global__ void __launch_bounds__(256, 3)
    packed_attn_prep_kernel(const uint16_t* qkv, const uint16_t* o,
                            const uint16_t* dout, const float* lse,
                            const int* head, int64_t T, int H, int Hkv,
                            uint16_t* dos, float2* stats,
                            float* rowexp, float* winexp, float* rownorm, float* winnorm,
                            uint32_t* taken, int* dev_err) {
  constexpr int LR = D / 8, RW = 32 / LR, IT = kWindow / 8 / RW;  // lanes a row, rows a warp, rounds
  __shared__ float low[8];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.y, col = (lane % LR) * 8;
  const int64_t live = head[2];
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *taken = 0;
  const int64_t t0 = (int64_t)blockIdx.x * kWindow + warp * (kWindow / 8) + lane / LR;
  if (h >= H) {
    bool bad = false;
    float most = 0.f;
    uint4 x[IT];
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int64_t t = t0 + i * RW;
      x[i] = t < live ? *reinterpret_cast<const uint4*>(qkv + t * (int64_t)(H + 2 * Hkv) * D +
                                                        (int64_t)(Hkv + h) * D + col)
                      : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int64_t t = t0 + i * RW;
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
      float n = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f = unpack_f16x2(w[k]);
        n += f.x * f.x + f.y * f.y;
      }
#pragma unroll
      for (int k = LR / 2; k > 0; k >>= 1) n += __shfl_xor_sync(0xFFFFFFFFu, n, k);
      if (!(n < INFINITY)) {
        bad = true;
        n = 0.f;
      }
      most = fmaxf(most, n);
      if (t < T && lane % LR == 0) rownorm[(int64_t)(h - H) * T + t] = n;
    }
    if (bad) atomicOr(dev_err, DEV_ERR_NONFINITE);
    most = warp_most(most);
    if (lane == 0) low[warp] = most;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int i = 1; i < 8; ++i) most = fmaxf(most, low[i]);
      winnorm[(int64_t)(h - H) * gridDim.x + blockIdx.x] = most;
    }
    return;
  }
  uint4 gr[IT], orow[IT];
  float ls[IT];
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int64_t t = t0 + i * RW;
    const int64_t at = (t * H + h) * D + col;
    const bool in = t < live;
    gr[i] = in ? *reinterpret_cast<const uint4*>(dout + at) : make_uint4(0u, 0u, 0u, 0u);
    orow[i] = in ? *reinterpret_cast<const uint4*>(o + at) : make_uint4(0u, 0u, 0u, 0u);
    ls[i] = in ? lse[(int64_t)h * T + t] : 0.f;
  }
  float emin = 127.f;
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int64_t t = t0 + i * RW;
    const uint32_t gw[4] = {gr[i].x, gr[i].y, gr[i].z, gr[i].w};
    const uint32_t ow[4] = {orow[i].x, orow[i].y, orow[i].z, orow[i].w};
    uint32_t n = 0;  // the largest magnitude's bits (those of NaN and infinity above all)
#pragma unroll
    for (int k = 0; k < 4; ++k)
      n = max(n, max((gw[k] & 0x7FFFu) << 16, gw[k] & 0x7FFF0000u));
#pragma unroll
    for (int k = LR / 2; k > 0; k >>= 1) n = max(n, __shfl_xor_sync(0xFFFFFFFFu, n, k));
    const int x = (int)(n >> 23);  // biased exponent
    const int e = n == 0 ? 127 : x == 255 ? 0 : 127 - max(1, x);
    const float up = ldexpf(1.f, e);
    float dl = 0.f;
    uint32_t p[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float2 g = unpack_bf16x2(gw[k]);
      const float2 y = unpack_f16x2(ow[k]);
      g.x *= up;
      g.y *= up;
      dl += g.x * y.x + g.y * y.y;
      p[k] = pack_f16x2(g.x, g.y);
    }
#pragma unroll
    for (int k = LR / 2; k > 0; k >>= 1) dl += __shfl_xor_sync(0xFFFFFFFFu, dl, k);
    if (t < T) {
      *reinterpret_cast<uint4*>(dos + (t * H + h) * D + col) = make_uint4(p[0], p[1], p[2], p[3]);
      if (lane % LR == 0) {
        const int64_t r = (int64_t)h * T + t;
        stats[r] = make_float2(fmaf(ls[i], kLog2e, (float)e), dl);
        rowexp[r] = (float)e;
      }
    }
    emin = fminf(emin, (float)e);
  }
  emin = warp_min(emin);
  if (lane == 0) low[warp] = emin;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < 8; ++i) emin = fminf(emin, low[i]);
    winexp[(int64_t)h * gridDim.x + blockIdx.x] = emin;
  }
}

// A thread's share of a gradient row, the columns [q, q + D/4) and [D/2 + q, ...): scaled,
// with cs (nullable; of the row's position, at column q) the rotation of the pairs
// (i, i + D/2) undone, to bf16 at out + q and out + D/2 + q.
template <int D>
__device__ __forceinline__ void store_grad_share(const uint32_t (&lo)[D / 4],
                                                 const uint32_t (&hi)[D / 4], float scale,
                                                 const float2* cs, uint16_t* out) {
#pragma unroll
  for (int c = 0; c < D / 4; c += 16) {
    uint32_t pa[8], pb[8];
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
      float a0 = __uint_as_float(lo[c + e]) * scale, a1 = __uint_as_float(lo[c + e + 1]) * scale;
      float b0 = __uint_as_float(hi[c + e]) * scale, b1 = __uint_as_float(hi[c + e + 1]) * scale;
      if (cs) {
        const float4 f = *reinterpret_cast<const float4*>(cs + c + e);
        const float x0 = a0, y0 = b0, x1 = a1, y1 = b1;
        a0 = x0 * f.x + y0 * f.y;
        b0 = y0 * f.x - x0 * f.y;
        a1 = x1 * f.z + y1 * f.w;
        b1 = y1 * f.z - x1 * f.w;
      }
      pa[e / 2] = pack_bf16x2(a0, a1);
      pb[e / 2] = pack_bf16x2(b0, b1);
    }
    st_global32(out + c, pa);
    st_global32(out + D / 2 + c, pb);
  }
}
// That share of an accumulator row in TMEM.
template <int D>
__device__ __forceinline__ void load_share(uint32_t t, uint32_t (&lo)[D / 4], uint32_t (&hi)[D / 4]) {
  if constexpr (D == 128) {
    tmem_ld32(t, lo);
    tmem_ld32(t + D / 2, hi);
  } else {
    tmem_ld16(t, lo);
    tmem_ld16(t + D / 2, hi);
  }
  tmem_ld_wait();
}

// ------------------------------------------------------------------ dK, dV
// An item: 128 keys of a document, a kv head and `nh` of its query heads.  For each of
// those heads the chunks of 64 queries that see some of the keys go by; chunk c is the
// gradient warps' set c % 2, so that one set's arithmetic runs while the products of the
// other's chunk do:
//   warp 17: S^T = K Q^T, dP'^T = V dO'^T          (buffers c % 2, 64 columns each)
//   sets   : P' = 2^u exp2(S^T c - l + emin) -> TMEM;  dS' = P' (dP' - delta') 2^(a - u) -> TMEM
//   warp 18: dV' += P' dO', dK' += dS' Q           (in order, so the sums are fixed)
// emin is the least exponent of the item's queries: 2^(emin - e) P <= 1, so all products
// carry the same factor 2^emin, taken out at the end with 2^u and 2^a.  Those bring P' and
// dS' to 2^15 at most (ds_exponent), so that a P or dS of 2^-29 of the largest possible is
// still a normal fp16 number and one of 2^-39 not yet 0.  With all heads of the
// group in one item (nh = G) the sums are the gradients, written in bf16; otherwise
// fp32 parts are left for packed_attn_sum_kernel.
// Tensor bound: 1280 cycles of products a chunk, which takes about 1760 (the chain from a
// chunk's scores to its dS' and on; two sets of warps hide one behind the other).  The whole
// backward of one document of 16,384 tokens (32/8 heads, d 128): 7.4 ms, 740 TFLOP/s.
template <int D>
struct DkvSmem {
  static constexpr uint32_t kTile = 128 * D * 2;  // K or V
  static constexpr uint32_t kQc = kBC * D * 2;    // a chunk of Q or dO'
  static constexpr int kRing = D == 128 ? 4 : 6;  // chunks in flight
  static constexpr uint32_t kBytes = 1024 + 2 * kTile + 2 * kRing * kQc + kRing * kBC * 8;
};

// Passes the items of one part of the kernel from the TMA producer, which draws them, to the
// other warps; the CTA's first one is known to all.
struct ItemRing {
  uint64_t full[kTake], free[kTake];
  int item[kTake];
};

// What both parts of the kernel read and write.
struct BwdArgs {
  PackedIndex idx;
  const float2* stats;
  const float *rowexp, *winexp, *rownorm, *winnorm;
  int64_t T;
  int H, Hkv, nh;
  float sl2, scale;
  const float2* cs;
  uint16_t* dqkv;
  float *dk, *dv;
  uint32_t* taken;
  int* dev_err;
};

// The CTA's dK, dV items: w0 is its first; -> the first number drawn that is none of them.
template <int D>
__device__ __forceinline__ uint32_t dkdv_part(const BwdArgs& a_, const CUtensorMap& tm_kv,  // qkv, boxes of 128 rows
                                              const CUtensorMap& tm_q,   // qkv, boxes of 64 rows
                                              const CUtensorMap& tm_do,  // dO', boxes of 64 rows
                                              uint8_t* dyn, uint32_t tmem, int items, bool many,
                                              uint32_t w0, int* abort_sh) {
  const PackedIndex& idx = a_.idx;
  const float2* stats = a_.stats;
  const float *rowexp = a_.rowexp, *winexp = a_.winexp;
  const float *rownorm = a_.rownorm, *winnorm = a_.winnorm;
  const int64_t T = a_.T;
  const int H = a_.H, Hkv = a_.Hkv, nh = a_.nh;
  const float sl2 = a_.sl2, scale = a_.scale;
  const float2* cs = a_.cs;
  uint16_t* dqkv = a_.dqkv;
  float *dk = a_.dk, *dv = a_.dv;
  int* dev_err = a_.dev_err;
  using SM = DkvSmem<D>;
  constexpr int DA = D / 64, NR = SM::kRing, kItems = 8;
  static_assert(NR % 2 == 0, "a ring slot always serves the same set of warps");
  static_assert(kItems > NR + 1, "an item's factors are kept until all have read them");
  static_assert(NR >= 3, "the chunk that an item is drawn behind has not left its slot");
  __shared__ __align__(8) uint64_t kv_full, kv_free, r_full[NR], r_free[NR], st_full[NR];
  __shared__ __align__(8) uint64_t s_full[2], dp_full[2], p_full[2], ds_full[2], s_free[2], dp_free[2];
  __shared__ __align__(8) uint64_t acc_full, acc_free;
  __shared__ __align__(8) ItemRing ring;
  __shared__ float factor_sh[kItems][3];  // 2^(a - u); of dV 2^(-emin - u); of dK
  __shared__ uint32_t next_sh;
  volatile int* abort_flag = abort_sh;

  uint8_t* Ks = dyn;
  uint8_t* Vs = Ks + SM::kTile;
  uint8_t* Qb = Vs + SM::kTile;             // [NR] chunks of Q
  uint8_t* dOb = Qb + NR * SM::kQc;         // [NR] chunks of dO'
  // [NR] 64 x (emin + u - l), 64 x -delta' 2^(a - u)
  float* st = reinterpret_cast<float*>(dOb + NR * SM::kQc);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr uint32_t kColS = 0, kColP = 2 * kBC, kColV = 4 * kBC, kColK = 4 * kBC + 128;

  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&kv_full), 1);
    mbar_init(smem_u32(&kv_free), 1);
    for (int i = 0; i < NR; ++i) {
      mbar_init(smem_u32(&r_full[i]), 1);
      mbar_init(smem_u32(&r_free[i]), 1);
      mbar_init(smem_u32(&st_full[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s_full[i]), 1);
      mbar_init(smem_u32(&dp_full[i]), 1);
      mbar_init(smem_u32(&p_full[i]), 8);
      mbar_init(smem_u32(&ds_full[i]), 8);
      mbar_init(smem_u32(&s_free[i]), 1);
      mbar_init(smem_u32(&dp_free[i]), 1);
    }
    mbar_init(smem_u32(&acc_full), 1);
    mbar_init(smem_u32(&acc_free), 16);
    for (int i = 0; i < kTake; ++i) {
      mbar_init(smem_u32(&ring.full[i]), 1);
      mbar_init(smem_u32(&ring.free[i]), kTakers);
    }
    next_sh = UINT32_MAX;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  __syncthreads();
  const int G = H / Hkv, parts = G / nh;
  const int per = Hkv * parts;              // items of a tile
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    return mbar_wait_short(smem_u32(bar), parity & 1u, abort_flag, dev_err);
  };
  auto wait_all = [&](uint64_t* bar, uint32_t parity) -> bool {
    return __all_sync(0xFFFFFFFFu, wait(bar, parity));
  };
  // item k of this CTA (-1: none is left), given and taken; the first is known
  auto give = [&](int k, uint32_t w) -> bool {
    if (many && k > 0) {
      const uint32_t n = (uint32_t)(k - 1), slot = n % kTake;
      if (n >= kTake && !wait(&ring.free[slot], n / kTake - 1)) return false;
      ring.item[slot] = w < (uint32_t)items ? (int)w : -1;
      mbar_arrive(smem_u32(&ring.full[slot]));
    }
    return w < (uint32_t)items;
  };
  auto take = [&](int k) -> int {
    if (k == 0) return w0 < (uint32_t)items ? (int)w0 : -1;
    if (!many) return -1;
    const uint32_t n = (uint32_t)(k - 1), slot = n % kTake;
    if (!wait_all(&ring.full[slot], n / kTake)) return -1;
    const int w = ring.item[slot];
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&ring.free[slot]));
    return w;
  };
  // an item's tile, first query head, first query and chunks of a head
  struct Item {
    PackedTile t;
    int g, h0, qs, nc;
  };
  auto item = [&](int w) {
    Item it;
    it.t = idx.ktiles[w / per];
    it.g = (w % per) / parts;
    it.h0 = it.g * G + (w % per) % parts * nh;
    // the queries that see some of these keys: from the first key on, or, where the
    // tile reaches into the prompt, the whole document
    it.qs = it.t.row0 < it.t.prompt ? it.t.begin : it.t.row0;
    it.nc = (it.t.end - it.qs + kBC - 1) / kBC;
    return it;
  };

  if (warp == kBTma) {
    if (lane == 0) {
      uint32_t c = 0, ni = 0;
      bool ok = true;
      uint32_t w = w0;
      for (int k = 0; ok && give(k, w); ++k) {
        const Item it = item((int)w);
        if (ni > 0) ok = wait(&kv_free, ni - 1);
        if (!ok) break;
        ++ni;
        mbar_arrive_expect_tx(smem_u32(&kv_full), 2 * SM::kTile);
        for (int a = 0; a < DA; ++a) {
          tma_load_2d(smem_u32(Ks + a * 128 * 128), &tm_kv, smem_u32(&kv_full),
                      (H + it.g) * D + 64 * a, it.t.row0);
          tma_load_2d(smem_u32(Vs + a * 128 * 128), &tm_kv, smem_u32(&kv_full),
                      (H + Hkv + it.g) * D + 64 * a, it.t.row0);
        }
        for (int hh = 0; hh < nh && ok; ++hh)
          for (int j = 0; j < it.nc; ++j, ++c) {
            const uint32_t slot = c % NR;
            if (c >= NR) ok = wait(&r_free[slot], c / NR - 1);
            if (!ok) break;
            const uint32_t fb = smem_u32(&r_full[slot]);
            mbar_arrive_expect_tx(fb, 2 * SM::kQc);
            for (int a = 0; a < DA; ++a) {
              tma_load_2d(smem_u32(Qb + slot * SM::kQc + a * kBC * 128), &tm_q, fb,
                          (it.h0 + hh) * D + 64 * a, it.qs + j * kBC);
              tma_load_2d(smem_u32(dOb + slot * SM::kQc + a * kBC * 128), &tm_do, fb,
                          (it.h0 + hh) * D + 64 * a, it.qs + j * kBC);
            }
          }
        // (drawn when three chunks are left: any sooner, and a CTA with a long item takes
        // another one from those that will be done before it)
        if (ok && c >= 3) ok = wait(&r_free[(c - 3) % NR], (c - 3) / NR);
        w = many ? gridDim.x + atomicAdd(a_.taken, 1u) : UINT32_MAX;
      }
      if (ok) next_sh = w;
    }
    __syncwarp();
  } else if (warp == kBMma) {
    // ---------------------------------------------------------------- S^T and dP'^T
    const uint32_t lead = elect_lane();
    const uint32_t id = umma_idesc_f16(128, kBC);
    const uint64_t kd = umma_desc_k_sw128(smem_u32(Ks)), vd = umma_desc_k_sw128(smem_u32(Vs));
    uint32_t c = 0, ni = 0;
    bool ok = true;
    for (int k = 0, w; ok && (w = take(k)) >= 0; ++k) {
      const Item it = item(w);
      ok = wait_all(&kv_full, ni);
      ++ni;
      const int n = nh * it.nc;
      for (int j = 0; j < n && ok; ++j, ++c) {
        const uint32_t slot = c % NR, b = c & 1;
        const uint64_t qd = umma_desc_k_sw128(smem_u32(Qb + slot * SM::kQc));
        const uint64_t dd = umma_desc_k_sw128(smem_u32(dOb + slot * SM::kQc));
        ok = wait_all(&r_full[slot], c / NR) && wait_all(&st_full[slot], c / NR);
        // dV of the chunk before the last has read the P in this buffer
        if (ok && c >= 2) ok = wait_all(&s_free[b], c / 2 - 1);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_ss(lead, tmem + kColS + b * kBC,
                 kd + (uint32_t)((kk >> 2) * (128 * 128 / 16) + (kk & 3) * 2),
                 qd + (uint32_t)((kk >> 2) * (kBC * 128 / 16) + (kk & 3) * 2), id, kk > 0 ? 1u : 0u);
        mma_commit(lead, smem_u32(&s_full[b]));
        if (c >= 2) ok = wait_all(&dp_free[b], c / 2 - 1);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_ss(lead, tmem + kColP + b * kBC,
                 vd + (uint32_t)((kk >> 2) * (128 * 128 / 16) + (kk & 3) * 2),
                 dd + (uint32_t)((kk >> 2) * (kBC * 128 / 16) + (kk & 3) * 2), id, kk > 0 ? 1u : 0u);
        mma_commit(lead, smem_u32(&dp_full[b]));
      }
      if (ok) mma_commit(lead, smem_u32(&kv_free));
    }
  } else if (warp == kBMma + 1) {
    // ---------------------------------------------------------------- dV' and dK'
    const uint32_t lead = elect_lane();
    const uint32_t id = umma_idesc_f16(128, D) | (1u << 16);  // B MN-major
    uint32_t c = 0, ni = 0;
    bool ok = true;
    for (int k = 0, w; ok && (w = take(k)) >= 0; ++k) {
      const Item it = item(w);
      if (ni > 0) ok = wait_all(&acc_free, ni - 1);
      ++ni;
      const int n = nh * it.nc;
      for (int j = 0; j < n && ok; ++j, ++c) {
        const uint32_t slot = c % NR, b = c & 1;
        const uint64_t qd = umma_desc_mn_sw128(smem_u32(Qb + slot * SM::kQc), kBC * 128, 1024u);
        const uint64_t dd = umma_desc_mn_sw128(smem_u32(dOb + slot * SM::kQc), kBC * 128, 1024u);
        ok = wait_all(&p_full[b], c / 2);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < kBC / 16; ++kk)
          mma_ts(lead, tmem + kColV, tmem + kColS + b * kBC + (kk >> 1) * kBH + (kk & 1) * 8, dd + (uint32_t)(kk * 128), id,
                 (j > 0 || kk > 0) ? 1u : 0u);
        mma_commit(lead, smem_u32(&s_free[b]));
        ok = wait_all(&ds_full[b], c / 2);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < kBC / 16; ++kk)
          mma_ts(lead, tmem + kColK, tmem + kColP + b * kBC + (kk >> 1) * kBH + (kk & 1) * 8, qd + (uint32_t)(kk * 128), id,
                 (j > 0 || kk > 0) ? 1u : 0u);
        mma_commit(lead, smem_u32(&dp_free[b]));
        mma_commit(lead, smem_u32(&r_free[slot]));
      }
      if (ok) mma_commit(lead, smem_u32(&acc_full));
    }
  } else if (warp == kBTail) {
    // ---------------------------------------------------------------- the queries' values
    uint32_t c = 0, ni = 0;
    bool ok = true;
    const int64_t nw = (T + kWindow - 1) / kWindow;
    for (int k = 0, w; ok && (w = take(k)) >= 0; ++k, ++ni) {
      const Item it = item(w);
      // the least exponent: whole windows by their minima, the edges token by token (a
      // window that reaches into another document must not count)
      const float nv = largest_norm(winnorm + it.g * nw, rownorm + it.g * T, it.t.begin, it.t.end,
                                    lane);
      float emin = 127.f;
      const int w0 = (it.qs + kWindow - 1) / kWindow, w1 = it.t.end / kWindow;
      const int e0 = w0 < w1 ? w0 * kWindow : it.t.end;  // [qs, e0) and [w1 .., end)
      const int e1 = w0 < w1 ? w1 * kWindow : it.t.end;
      // (loads of several heads in flight: one after the other they took 8 us an item)
#pragma unroll 4
      for (int hh = 0; hh < nh; ++hh) {
        const float* we = winexp + (int64_t)(it.h0 + hh) * nw;
        const float* re = rowexp + (int64_t)(it.h0 + hh) * T;
        const int q = it.qs + lane, u = e1 + lane;
        const float a = w0 + lane < w1 ? we[w0 + lane] : 127.f;
        const float b = q < e0 ? re[q] : 127.f, c = q + 32 < e0 ? re[q + 32] : 127.f;
        const float d = u < it.t.end ? re[u] : 127.f;
        const float e = u + 32 < it.t.end ? re[u + 32] : 127.f;
        emin = fminf(fminf(fminf(emin, a), fminf(b, c)), fminf(d, e));
        for (int i = w0 + 32 + lane; i < w1; i += 32) emin = fminf(emin, we[i]);
        for (int i = q + 64; i < e0; i += 32) emin = fminf(emin, re[i]);
      }
      emin = warp_min(emin);
      const int e_min = (int)emin, u = min(kUp, 126 - e_min);
      const int a = ds_exponent(warp_most(nv), D, e_min);
      const float mul = pow2i(a - u), lift = emin + (float)u;
      if (lane == 0) {
        factor_sh[ni % kItems][0] = mul;
        factor_sh[ni % kItems][1] = ex2(-lift);
        factor_sh[ni % kItems][2] = ex2(-(float)(e_min + a)) * scale;
      }
      for (int hh = 0; hh < nh && ok; ++hh) {
        const float2* sh = stats + (int64_t)(it.h0 + hh) * T;
        for (int j = 0; j < it.nc; ++j, ++c) {
          const uint32_t slot = c % NR;
          const int q0 = it.qs + j * kBC;
          float2 v[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int q = q0 + lane + 32 * i;
            v[i] = q < it.t.end ? sh[q] : make_float2(INFINITY, 0.f);
            v[i].x = lift - v[i].x;
          }
          ok = wait_all(&r_full[slot], c / NR);
          if (!ok) break;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            st[slot * 2 * kBC + lane + 32 * i] = v[i].x;
            st[slot * 2 * kBC + kBC + lane + 32 * i] = -v[i].y * mul;
          }
          if (q0 + kBC > it.t.end) {
            // queries behind the document: their P and dS are 0, and so must the rows be
            // that those multiply (0 * inf)
            zero_rows<D>(Qb + slot * SM::kQc, it.t.end - q0, kBC, lane);
            zero_rows<D>(dOb + slot * SM::kQc, it.t.end - q0, kBC, lane);
            fence_proxy_async_smem();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&st_full[slot]));
        }
      }
    }
  } else {
    // ---------------------------------------------------------------- gradient warps
    const uint32_t b = (warp >> 2) & 1;        // set: chunks c with c % 2 == b
    const int hf = warp >> 3;                  // columns 32 hf .. of a chunk
    const int r = (warp & 3) * 32 + lane;      // key of the tile = TMEM lane
    const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t ts = trow + kColS + b * kBC + hf * kBH, tp = trow + kColP + b * kBC + hf * kBH;
    const uint64_t sl22 = pack_f32x2(sl2, sl2);
    uint32_t c = 0, ni = 0;
    bool ok = true;
    for (int k = 0, w; ok && (w = take(k)) >= 0; ++k) {
      const Item it = item(w);
      const int kpos = it.t.row0 + r;
      // the queries [qlo, end) see this key; all of the warp's keys from qall on
      const int qlo = kpos < it.t.prompt ? it.t.begin : kpos;
      const int klast = it.t.row0 + (warp & 3) * 32 + 31;
      const int qall = klast < it.t.prompt ? it.t.begin : klast;
      const int n = nh * it.nc;
      int q0 = it.qs + hf * kBH;  // first query of this thread's columns
      for (int j = 0, jc = 0; j < n; ++j, ++c, q0 += kBC) {
        if (jc == it.nc) {  // the next head
          jc = 0;
          q0 = it.qs + hf * kBH;
        }
        ++jc;
        if ((c & 1) != b) continue;
        const uint32_t slot = c % NR, ph = c / 2;
        // pairs of (emin + u - l), and of -delta' 2^(a - u)
        const ulonglong2* l2 = reinterpret_cast<const ulonglong2*>(st + slot * 2 * kBC + hf * kBH);
        const ulonglong2* dl = l2 + kBC / 4;
        ok = wait_all(&s_full[b], ph);  // (and st: S^T is issued behind it)
        if (!ok) break;
        tc_fence_after();
        uint32_t sv[kBH];
        tmem_ld32(ts, sv);
        tmem_ld_wait();
        const bool whole = q0 >= qall && q0 + kBH <= it.t.end;  // (uniform in the warp)
        uint64_t p[kBH / 2];
#pragma unroll
        for (int e = 0; e < kBH / 2; e += 2) {
          const ulonglong2 v = l2[e / 2];
          const float2 x = unpack_f32x2(fma_f32x2(
              pack_f32x2(__uint_as_float(sv[2 * e]), __uint_as_float(sv[2 * e + 1])), sl22, v.x));
          const float2 y = unpack_f32x2(fma_f32x2(
              pack_f32x2(__uint_as_float(sv[2 * e + 2]), __uint_as_float(sv[2 * e + 3])), sl22, v.y));
          p[e] = pack_f32x2(ex2(x.x), ex2(x.y));
          p[e + 1] = pack_f32x2(ex2(y.x), ex2(y.y));
        }
        if (!whole) {
          const int lo = qlo - q0, hi = it.t.end - q0;
#pragma unroll
          for (int e = 0; e < kBH / 2; ++e) {
            const float2 x = unpack_f32x2(p[e]);
            p[e] = pack_f32x2(2 * e >= lo && 2 * e < hi ? x.x : 0.f,
                              2 * e + 1 >= lo && 2 * e + 1 < hi ? x.y : 0.f);
          }
        }
        uint32_t pk[kBH / 2];
#pragma unroll
        for (int e = 0; e < kBH / 2; ++e) {
          const float2 x = unpack_f32x2(p[e]);
          pk[e] = pack_f16x2(x.x, x.y);
        }
        tmem_st16(ts, pk);
        // (dP' is there by now: its load runs while the store of P' does)
        ok = wait_all(&dp_full[b], ph);
        if (!ok) break;
        tc_fence_after();
        tmem_ld32(tp, sv);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&p_full[b]));
        const float mul = factor_sh[ni % kItems][0];
        const uint64_t mul2 = pack_f32x2(mul, mul);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < kBH / 2; e += 2) {
          const ulonglong2 v = dl[e / 2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint64_t d = pack_f32x2(__uint_as_float(sv[2 * (e + i)]),
                                          __uint_as_float(sv[2 * (e + i) + 1]));
            float2 x = unpack_f32x2(mul_f32x2(p[e + i], fma_f32x2(d, mul2, i ? v.y : v.x)));
            if (!whole) {  // (dp behind the document may be anything)
              const float2 q = unpack_f32x2(p[e + i]);
              x.x = q.x != 0.f ? x.x : 0.f;
              x.y = q.y != 0.f ? x.y : 0.f;
            }
            pk[e + i] = pack_f16x2(x.x, x.y);
          }
        }
        tmem_st16(tp, pk);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ds_full[b]));
      }
      // -------------------------------------------------------------- epilogue: set 0
      // takes dV, set 1 dK
      ok = ok && wait_all(&acc_full, ni);
      if (!ok) break;
      tc_fence_after();
      uint32_t lo[D / 4], hi[D / 4];
      load_share<D>(trow + (b ? kColK : kColV) + hf * (D / 4), lo, hi);
      const float f = factor_sh[ni % kItems][b ? 2 : 1];
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&acc_free));
      ++ni;
      if (kpos < it.t.end) {
        if (parts == 1) {
          const int col = (b ? H + it.g : H + Hkv + it.g) * D + hf * (D / 4);
          store_grad_share<D>(lo, hi, f,
                              b && cs ? cs + (int64_t)idx.pos[kpos] * (D / 2) + hf * (D / 4) : nullptr,
                              dqkv + (int64_t)kpos * (H + 2 * Hkv) * D + col);
        } else {
          // (eight columns of consecutive tokens lie together, so that a warp's store is one
          // run of 1 KB: by rows a tile took 7000 to 9000 cycles to write)
          float* out = (b ? dk : dv) +
                       (((int64_t)(it.h0 / nh) * (D / 8) + hf * (D / 32)) * T + kpos) * 8;
#pragma unroll
          for (int e = 0; e < D / 4; e += 8) {
            uint32_t x[8], y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              x[i] = __float_as_uint(__uint_as_float(lo[e + i]) * f);
              y[i] = __float_as_uint(__uint_as_float(hi[e + i]) * f);
            }
            st_global32(out + (int64_t)(e / 8) * T * 8, x);
            st_global32(out + (int64_t)(D / 16 + e / 8) * T * 8, y);
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  return next_sh;
}

// dk and dv (bf16, into dqkv) from the fp32 parts of `parts` shares of each kv head's
// query heads, [share][D / 8][T][8], summed in order; with cs the rotation of k by its
// position undone.  The whole grid shares the tokens, a thread takes 4 pairs (i, i + D/2),
// two threads eight columns of a token, a warp 16 consecutive tokens.
template <int D>
__global__ void __launch_bounds__(256)
    packed_attn_sum_kernel(const float* dk, const float* dv, int parts, const int* head,
                           int64_t T, const int* pos, int Hkv, int64_t ld, int col0,
                           const float2* cs, uint16_t* dqkv) {
  constexpr int half = D / 2, chunks = half / 8;
  pdl_trigger();
  pdl_wait();
  const int64_t tokens = head[2];
  // (there are shares only where tokens / 128 Hkv is below the number of SMs: 32 bits do)
  const uint32_t n = (uint32_t)tokens * 4u * Hkv * chunks;
  for (uint32_t i = blockIdx.x * blockDim.x + threadIdx.x; i < n; i += gridDim.x * blockDim.x) {
    const uint32_t rest = (i >> 1) / (uint32_t)tokens;
    const int64_t t = (i >> 1) - rest * (uint32_t)tokens;
    const int ch = (int)(rest % chunks), hh = (int)(rest / chunks);
    const int col = ch * 8 + (int)(i & 1) * 4;
    const float* src = (hh < Hkv ? dk : dv) +
                       (((int64_t)(hh % Hkv) * parts * (D / 8) + ch) * T + t) * 8 + (i & 1) * 4;
    float a[4] = {0.f, 0.f, 0.f, 0.f}, b[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int k = 0; k < parts; ++k) {
      const float* x = src + (int64_t)k * (D / 8) * T * 8;
      const float4 u = *reinterpret_cast<const float4*>(x);
      const float4 v = *reinterpret_cast<const float4*>(x + (int64_t)chunks * T * 8);
      a[0] += u.x; a[1] += u.y; a[2] += u.z; a[3] += u.w;
      b[0] += v.x; b[1] += v.y; b[2] += v.z; b[3] += v.w;
    }
    if (cs && hh < Hkv) {
      const float2* c = cs + (int64_t)pos[t] * half + col;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f = c[k];
        const float x = a[k], y = b[k];
        a[k] = x * f.x + y * f.y;
        b[k] = y * f.x - x * f.y;
      }
    }
    uint16_t* out = dqkv + t * ld + col0 + hh * D + col;
    *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]));
    *reinterpret_cast<uint2*>(out + half) =
        make_uint2(pack_bf16x2(b[0], b[1]), pack_bf16x2(b[2], b[3]));
  }
}

// ------------------------------------------------------------------ dQ
// Items and streams as in the forward; a stream's chunk of 64 keys:
//   its MMA warp: S = Q K^T, dP' = dO' V^T;  its gradient warps: P' = 2^a exp2(S c - lse
//   log2 e), dS' = P' (dP' - delta') as fp16 over dP' in TMEM, a of each query (ds_exponent) by the
//   norms of v among the item's keys;  the MMA warp: dQ' += dS' K.
// S of the next chunk is computed while dS of this one is formed.
template <int D>
struct DqSmem {
  static constexpr uint32_t kTile = 128 * D * 2;  // Q or dO' of a stream
  static constexpr uint32_t kKc = kBC * D * 2;    // a chunk of K or V
  static constexpr int kRing = D == 128 ? 3 : 6;
  static constexpr uint32_t kBytes = 1024 + 4 * kTile + 2 * kRing * kKc;
};

// The CTA's dQ items: w0 is its first (or behind the last); `done` drawn numbers are none
// of them but lie before theirs.
template <int D>
__device__ __forceinline__ void dq_part(const BwdArgs& a_, const CUtensorMap& tm_q,   // qkv, boxes of 128 rows
                                        const CUtensorMap& tm_kv,  // qkv, boxes of 64 rows
                                        const CUtensorMap& tm_do,  // dO', boxes of 128 rows
                                        uint8_t* dyn, uint32_t tmem, int items, uint32_t done,
                                        bool many, uint32_t w0, int* abort_sh) {
  const PackedIndex& idx = a_.idx;
  const float2* stats = a_.stats;
  const float *rowexp = a_.rowexp, *rownorm = a_.rownorm, *winnorm = a_.winnorm;
  const int64_t T = a_.T, nw = (T + kWindow - 1) / kWindow;
  const int H = a_.H, Hkv = a_.Hkv;
  const float sl2 = a_.sl2, scale = a_.scale;
  const float2* cs = a_.cs;
  uint16_t* dqkv = a_.dqkv;
  int* dev_err = a_.dev_err;
  using SM = DqSmem<D>;
  constexpr int DA = D / 64, NR = SM::kRing;
  static_assert(NR >= 3, "the chunk that an item is drawn behind has not left its slot");
  __shared__ __align__(8) uint64_t q_full[2], q_free[2], r_full[NR], r_free[NR], k_clear[NR];
  __shared__ __align__(8) uint64_t s_full[2], s_free[2], dp_full[2], ds_full[2], dq_full[2], dq_free[2];
  __shared__ __align__(8) ItemRing ring;
  volatile int* abort_flag = abort_sh;

  uint8_t* Qs = dyn;                        // [2] Q of the streams
  uint8_t* dOs = Qs + 2 * SM::kTile;        // [2] dO'
  uint8_t* Kb = dOs + 2 * SM::kTile;        // [NR] chunks of K
  uint8_t* Vb = Kb + NR * SM::kKc;          // [NR] chunks of V
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr uint32_t kColS = 0, kColP = kBC, kColQ = 256;  // S and dP' of stream s at 128 s

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&q_full[i]), 1);
      mbar_init(smem_u32(&q_free[i]), 1);
      mbar_init(smem_u32(&s_full[i]), 1);
      mbar_init(smem_u32(&s_free[i]), 8);
      mbar_init(smem_u32(&dp_full[i]), 1);
      mbar_init(smem_u32(&ds_full[i]), 8);
      mbar_init(smem_u32(&dq_full[i]), 1);
      mbar_init(smem_u32(&dq_free[i]), 8);
    }
    for (int i = 0; i < NR; ++i) {
      mbar_init(smem_u32(&r_full[i]), 1);
      mbar_init(smem_u32(&r_free[i]), 3);  // the two streams' products and warp 19
      mbar_init(smem_u32(&k_clear[i]), 1);
    }
    for (int i = 0; i < kTake; ++i) {
      mbar_init(smem_u32(&ring.full[i]), 1);
      mbar_init(smem_u32(&ring.free[i]), kTakers);
    }
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  __syncthreads();
  const int G = H / Hkv;
  const bool heads = G % 2 == 0;
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    return mbar_wait_short(smem_u32(bar), parity & 1u, abort_flag, dev_err);
  };
  auto wait_all = [&](uint64_t* bar, uint32_t parity) -> bool {
    return __all_sync(0xFFFFFFFFu, wait(bar, parity));
  };
  // item k of this CTA (-1: none is left), given and taken; the first is known
  auto give = [&](int k, uint32_t w) -> bool {
    if (many && k > 0) {
      const uint32_t n = (uint32_t)(k - 1), slot = n % kTake;
      if (n >= kTake && !wait(&ring.free[slot], n / kTake - 1)) return false;
      ring.item[slot] = w < (uint32_t)items ? (int)w : -1;
      mbar_arrive(smem_u32(&ring.full[slot]));
    }
    return w < (uint32_t)items;
  };
  auto take = [&](int k) -> int {
    if (k == 0) return w0 < (uint32_t)items ? (int)w0 : -1;
    if (!many) return -1;
    const uint32_t n = (uint32_t)(k - 1), slot = n % kTake;
    if (!wait_all(&ring.full[slot], n / kTake)) return -1;
    const int w = ring.item[slot];
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&ring.free[slot]));
    return w;
  };

  if (warp == kBTma) {
    if (lane == 0) {
      uint32_t c = 0, nq[2] = {0, 0};
      bool ok = true;
      uint32_t w = w0;
      for (int k = 0; ok && give(k, w); ++k) {
        const FwdItem it = fwd_item(idx, (int)w, H, heads, 0),
                      it1 = fwd_item(idx, (int)w, H, heads, 1);
        const int g = it.head / G;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (!ok || (s == 1 && it1.n == 0)) continue;
          if (nq[s] > 0) ok = wait(&q_free[s], nq[s] - 1);
          if (!ok) continue;
          ++nq[s];
          const uint32_t fb = smem_u32(&q_full[s]);
          mbar_arrive_expect_tx(fb, 2 * SM::kTile);
          const int h = s ? it1.head : it.head, row = s ? it1.row : it.row;
          for (int a = 0; a < DA; ++a) {
            tma_load_2d(smem_u32(Qs + s * SM::kTile + a * 128 * 128), &tm_q, fb, h * D + 64 * a, row);
            tma_load_2d(smem_u32(dOs + s * SM::kTile + a * 128 * 128), &tm_do, fb, h * D + 64 * a,
                        row);
          }
        }
        for (int j = 0; j < it.nu && ok; ++j, ++c) {
          const uint32_t slot = c % NR;
          if (c >= NR) ok = wait(&r_free[slot], c / NR - 1);
          if (!ok) break;
          const uint32_t fb = smem_u32(&r_full[slot]);
          mbar_arrive_expect_tx(fb, 2 * SM::kKc);
          for (int a = 0; a < DA; ++a) {
            tma_load_2d(smem_u32(Kb + slot * SM::kKc + a * kBC * 128), &tm_kv, fb,
                        (H + g) * D + 64 * a, it.begin + j * kBC);
            tma_load_2d(smem_u32(Vb + slot * SM::kKc + a * kBC * 128), &tm_kv, fb,
                        (H + Hkv + g) * D + 64 * a, it.begin + j * kBC);
          }
        }
        if (ok && c >= 3) ok = wait(&r_free[(c - 3) % NR], (c - 3) / NR);  // as there
        w = many ? gridDim.x + atomicAdd(a_.taken, 1u) - done : UINT32_MAX;
      }
    }
    __syncwarp();
  } else if (warp == kBMma || warp == kBMma + 1) {
    // ---------------------------------------------------------------- MMA issuers
    const int s = warp - kBMma;
    const uint32_t lead = elect_lane();
    const uint32_t id_s = umma_idesc_f16(128, kBC);
    const uint32_t id_q = umma_idesc_f16(128, D) | (1u << 16);  // B (K) MN-major
    const uint32_t ts = tmem + kColS + (uint32_t)s * 128, tp = tmem + kColP + (uint32_t)s * 128;
    const uint32_t tq = tmem + kColQ + (uint32_t)s * 128;
    const uint64_t qd = umma_desc_k_sw128(smem_u32(Qs + s * SM::kTile));
    const uint64_t od = umma_desc_k_sw128(smem_u32(dOs + s * SM::kTile));
    uint32_t c = 0, ni = 0, nc = 0;  // ring chunks, items and chunks of this stream
    bool ok = true;
    auto scores = [&](uint32_t d, uint64_t a, uint8_t* tile, uint64_t* bar) {
      const uint64_t bd = umma_desc_k_sw128(smem_u32(tile));
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        mma_ss(lead, d, a + (uint32_t)((kk >> 2) * (128 * 128 / 16) + (kk & 3) * 2),
               bd + (uint32_t)((kk >> 2) * (kBC * 128 / 16) + (kk & 3) * 2), id_s, kk > 0 ? 1u : 0u);
      mma_commit(lead, smem_u32(bar));
    };
    for (int k = 0, w; ok && (w = take(k)) >= 0; ++k) {
      const FwdItem it = fwd_item(idx, w, H, heads, s);
      if (it.n > 0) {
        ok = wait_all(&q_full[s], ni) && wait_all(&r_full[c % NR], c / NR);
        // (the scores of the item before have been read: its dS came behind them)
        if (!ok) break;
        tc_fence_after();
        scores(ts, qd, Kb + (c % NR) * SM::kKc, &s_full[s]);
        scores(tp, od, Vb + (c % NR) * SM::kKc, &dp_full[s]);
        if (ni > 0) ok = wait_all(&dq_free[s], ni - 1);  // dQ' of the item before has been read
        ++ni;
      }
      for (int j = 0; j < it.nu && ok; ++j, ++c) {
        const uint32_t slot = c % NR, next = (c + 1) % NR;
        if (j < it.n) {
          const bool more = j + 1 < it.n;
          if (more) {
            ok = wait_all(&r_full[next], (c + 1) / NR) && wait_all(&s_free[s], nc);
            if (!ok) break;
            tc_fence_after();
            scores(ts, qd, Kb + next * SM::kKc, &s_full[s]);
          }
          if (j + 1 == it.nu && it.begin + it.nu * kBC > it.end)
            ok = wait_all(&k_clear[slot], c / NR);
          ok = ok && wait_all(&ds_full[s], nc);
          if (!ok) break;
          ++nc;
          tc_fence_after();
          const uint64_t kd = umma_desc_mn_sw128(smem_u32(Kb + slot * SM::kKc), kBC * 128, 1024u);
#pragma unroll
          for (int kk = 0; kk < kBC / 16; ++kk)
            mma_ts(lead, tq, tp + (kk >> 1) * kBH + (kk & 1) * 8, kd + (uint32_t)(kk * 128), id_q,
                   (j > 0 || kk > 0) ? 1u : 0u);
          if (more)
            scores(tp, od, Vb + next * SM::kKc, &dp_full[s]);
          else
            mma_commit(lead, smem_u32(&dq_full[s]));
          // Q and dO' are free behind the stream's last scores
          if (j + 2 == it.n || it.n == 1) mma_commit(lead, smem_u32(&q_free[s]));
        } else {
          ok = wait_all(&r_full[slot], c / NR);
          if (!ok) break;
        }
        mma_commit(lead, smem_u32(&r_free[slot]));
      }
    }
  } else if (warp == kBTail) {
    // Follows every chunk of the ring; keys behind the document: their dS is 0, and so
    // must the K rows be that those multiply (0 * inf).
    uint32_t c = 0;
    bool ok = true;
    for (int k = 0, w; ok && (w = take(k)) >= 0; ++k) {
      const FwdItem it = fwd_item(idx, w, H, heads, 0);
      for (int j = 0; j < it.nu && ok; ++j, ++c) {
        const uint32_t slot = c % NR;
        ok = wait_all(&r_full[slot], c / NR);
        if (!ok) break;
        const int rows = it.end - it.begin - j * kBC;
        if (rows < kBC) {
          zero_rows<D>(Kb + slot * SM::kKc, rows, kBC, lane);
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (lane == 0) {
          mbar_arrive(smem_u32(&k_clear[slot]));  // (every chunk: a phase per use of the slot)
          mbar_arrive(smem_u32(&r_free[slot]));
        }
      }
    }
  } else {
    // ---------------------------------------------------------------- gradient warps
    const int s = (warp >> 2) & 1;
    const int hf = warp >> 3;              // keys 32 hf .. of a chunk
    const int r = (warp & 3) * 32 + lane;  // query of the tile = TMEM lane
    const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16) + (uint32_t)s * 128;
    const uint32_t ts = trow + kColS + hf * kBH, tp = trow + kColP + hf * kBH;
    const uint64_t sl22 = pack_f32x2(sl2, sl2);
    uint32_t nc = 0, ni = 0;
    bool ok = true;
    for (int k = 0, w; ok && (w = take(k)) >= 0; ++k) {
      const FwdItem it = fwd_item(idx, w, H, heads, s);
      const int n = it.n;
      if (n == 0) continue;
      const int q = it.row + r;
      const int kmax = min(max(q, it.prompt - 1), it.end - 1);  // its last key
      const int kall = min(max(it.row + (warp & 3) * 32, it.prompt - 1), it.end - 1);
      const int64_t at = (int64_t)it.head * T + min(q, it.end - 1);
      const float2 sq = stats[at];
      const float e = rowexp[at];
      const int g = it.head / G;
      const float nv = largest_norm(winnorm + g * nw, rownorm + g * T, it.begin,
                                    min(it.end, it.begin + n * kBC), lane);
      const int a = ds_exponent(warp_most(nv), D, (int)e);
      const float nl = e - sq.x + (float)a;  // (P is not stored here: it takes the factor)
      const uint64_t nl2 = pack_f32x2(nl, nl), ndl = pack_f32x2(-sq.y, -sq.y);
      for (int j = 0; j < n; ++j, ++nc) {
        ok = wait_all(&s_full[s], nc);
        if (!ok) break;
        tc_fence_after();
        uint32_t sv[kBH];
        tmem_ld32(ts, sv);
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&s_free[s]));
        const int k0 = it.begin + j * kBC + hf * kBH;
        const int last = kmax - k0;
        const bool whole = k0 + kBH - 1 <= kall;  // (uniform in the warp)
        uint64_t p[kBH / 2];
#pragma unroll
        for (int i = 0; i < kBH / 2; ++i) {
          const float2 x = unpack_f32x2(fma_f32x2(
              pack_f32x2(__uint_as_float(sv[2 * i]), __uint_as_float(sv[2 * i + 1])), sl22, nl2));
          p[i] = pack_f32x2(ex2(x.x), ex2(x.y));
        }
        ok = wait_all(&dp_full[s], nc);
        if (!ok) break;
        tc_fence_after();
        tmem_ld32(tp, sv);
        tmem_ld_wait();
        uint32_t dsk[kBH / 2];
#pragma unroll
        for (int i = 0; i < kBH / 2; ++i) {
          const uint64_t d = pack_f32x2(__uint_as_float(sv[2 * i]), __uint_as_float(sv[2 * i + 1]));
          float2 x = unpack_f32x2(mul_f32x2(p[i], add_f32x2(d, ndl)));
          if (!whole) {  // (scores and dp behind the row's last key may be anything)
            x.x = 2 * i > last ? 0.f : x.x;
            x.y = 2 * i + 1 > last ? 0.f : x.y;
          }
          dsk[i] = pack_f16x2(x.x, x.y);
        }
        tmem_st16(tp, dsk);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ds_full[s]));
      }
      // -------------------------------------------------------------- epilogue
      ok = ok && wait_all(&dq_full[s], ni);
      if (!ok) break;
      ++ni;
      tc_fence_after();
      uint32_t lo[D / 4], hi[D / 4];
      load_share<D>(trow + kColQ + hf * (D / 4), lo, hi);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&dq_free[s]));
      if (q < it.end)
        store_grad_share<D>(lo, hi, scale * ex2(-e - (float)a),
                            cs ? cs + (int64_t)idx.pos[q] * (D / 2) + hf * (D / 4) : nullptr,
                            dqkv + (int64_t)q * (H + 2 * Hkv) * D + (int64_t)it.head * D +
                                hf * (D / 4));
    }
  }
  tc_fence_before();
  __syncthreads();
}

template <int D>
__global__ void __launch_bounds__(kBThreads, 1)
    packed_attn_bwd_kernel(const __grid_constant__ CUtensorMap tm_128,    // qkv, boxes of 128 rows
                           const __grid_constant__ CUtensorMap tm_64,     // qkv, boxes of 64 rows
                           const __grid_constant__ CUtensorMap tm_do128,  // dO', boxes of 128 rows
                           const __grid_constant__ CUtensorMap tm_do64,   // dO', boxes of 64 rows
                           const __grid_constant__ BwdArgs a) {
  extern __shared__ uint8_t bwd_raw[];
  __shared__ uint32_t tmem_sh;
  __shared__ int abort_sh;
  uint8_t* dyn = align1024_p(bwd_raw);
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) abort_sh = 0;
  if (warp == kBMma) {
    tmem_alloc(smem_u32(&tmem_sh), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_sh;
  pdl_trigger();
  pdl_wait();  // dO', its values, the index and the counter come from the kernels before
  const int G = a.H / a.Hkv;
  const int kitems = a.idx.head[0] * a.Hkv * (G / a.nh);
  const int qitems = G % 2 == 0 ? a.idx.head[0] * (a.H / 2) : a.idx.head[1] * a.H;
  // (both are below 2^31, their sum and what is drawn behind it below 2^32)
  const bool many = (uint32_t)kitems + (uint32_t)qitems > gridDim.x;  // (else one for each CTA)
  uint32_t w = blockIdx.x;
  if (w < (uint32_t)kitems)
    w = dkdv_part<D>(a, tm_128, tm_64, tm_do64, dyn, tmem, kitems, many, w, &abort_sh);
  // (every product and copy of the first part has been waited for, unless a wait gave up)
  if (w >= (uint32_t)kitems && w - (uint32_t)kitems < (uint32_t)qitems && !abort_sh)
    dq_part<D>(a, tm_128, tm_64, tm_do128, dyn, tmem, qitems, (uint32_t)kitems, many,
               w - (uint32_t)kitems, &abort_sh);
  {  // padding rows have no gradient
    const int64_t row = (int64_t)(a.H + 2 * a.Hkv) * (D / 8), first = a.idx.head[2];
    uint4* o = reinterpret_cast<uint4*>(a.dqkv) + first * row;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < (a.T - first) * row;
         i += (int64_t)gridDim.x * blockDim.x)
      o[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  tc_fence_before();
  __syncthreads();
  if (abort_sh) settle_ns(2000000);
  if (warp == kBMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Sets a kernel's dynamic shared memory limit once per device.
template <class K>
int allow_smem(K kernel, int bytes, bool (&done)[64]) {
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 64 && !done[dev]) {
    LSQ_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
    done[dev] = true;
  }
  return LSQ_OK;
}

template <class... P, class... A>
cudaError_t launch_dep(void (*k)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t st,
                       A... a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return ::lsq::launched(cudaLaunchKernelEx(&cfg, k, P(a)...));
}

template <int D>
int fwd_t(const uint16_t* qkv, const PackedIndex& x, int64_t T, int H, int Hkv, uint16_t* o,
          float* lse, cudaStream_t st) {
  using SM = FwdSmem<D>;
  static bool attr[64] = {false};
  LSQ_TRY(allow_smem(packed_attn_fwd_kernel<D>, (int)SM::kBytes, attr));
  const int64_t row = (int64_t)(H + 2 * Hkv) * D;
  CUtensorMap tm, to;
  LSQ_TRY(make_tmap_2d(&to, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, o, (uint64_t)H * D, (uint64_t)T,
                       (uint64_t)H * D, 64, 32, CU_TENSOR_MAP_SWIZZLE_128B));
  LSQ_TRY(make_tmap_2d(&tm, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, qkv, (uint64_t)row, (uint64_t)T,
                       (uint64_t)row, 64, kAQ, CU_TENSOR_MAP_SWIZZLE_128B));
  int* err = device_status_ptr();
  if (!err) return set_error(LSQ_ERR_CUDA, "device status word unavailable");
  const float sl2 = kLog2e / sqrtf((float)D);
  const int64_t items = (H / Hkv) % 2 == 0 ? (int64_t)x.cap * (H / 2) : (int64_t)x.cap2 * H;
  const unsigned grid = (unsigned)std::min<int64_t>(items, gemm_num_sms());
  LSQ_CUDA(launch_dep(packed_attn_fwd_kernel<D>, dim3(grid), kFThreads, SM::kBytes, st, tm, to, x, T, H,
                      Hkv, o, lse, sl2, err));
  return LSQ_OK;
}

struct BwdWs {
  uint16_t* dos;   // [T, H d] fp16 dO'
  float2* stats;   // [H, T] (lse log2 e + e, delta')
  float* rowexp;   // [H, T] e
  float* winexp;   // [H, windows] the least e of 64 tokens
  float* rownorm;  // [Hkv, T] |v|^2
  float* winnorm;  // [Hkv, windows] the largest |v|^2 of 64 tokens
  uint32_t* taken; // items handed out behind each CTA's first
  float *dk, *dv;  // [Hkv parts, d / 8, T, 8] fp32
};

// Into how many shares a kv head's query heads are split for dK and dV.  One share
// needs no partial sums (8 bytes written and read per token, share and dimension, and a
// launch) but leaves few items, and those of one long document are uneven; what a document's
// last tile lacks of 128 tokens is half a tile on average.  Wanted is more than an item for
// 16 tokens, since longer rows have longer items, up to nine items for ten SMs (dQ takes
// the SMs that are left).  Backward in us with one, two, four and eight shares:
// (32/8 heads, d 128) 512 tokens in 5 documents 30, 30, 33; in one 45, 35, 36; 1024 in 3:
// 43, 45, 53; 2048 in one 160, 152, 171; in 5: 77, 94, 112; (16/2) 512 in 5: 39, 30, 26, 30;
// 1024 in 20: 36, 32, 34, 39; 4096 in one 521, 302, 246, 284; in 10: 109, 84, 94, 114;
// (8/2, d 64) 1024 in 1000: 187, 205, 301.
int dkv_parts(int64_t T, int64_t n_docs, int H, int Hkv) {
  const int G = H / Hkv;
  const int64_t tiles = std::min(T, (T + kPackedTile - 1) / kPackedTile + n_docs / 2);
  for (int p = 1; p < G; ++p) {
    const int64_t items = tiles * Hkv * p;
    if (G % p == 0 && (items * 16 > T || items * 10 >= (int64_t)gemm_num_sms() * 9)) return p;
  }
  return G;
}

size_t carve_bwd(int64_t T, int H, int Hkv, int d, void* base, BwdWs* w) {
  Arena a;
  a.base = static_cast<uint8_t*>(base);
  a.cap = SIZE_MAX;
  BwdWs x;
  const int parts = dkv_parts(T, 0, H, Hkv);  // (the most that any number of documents takes)
  x.dos = a.take<uint16_t>((size_t)T * H * d);
  x.stats = a.take<float2>((size_t)T * H);
  x.rowexp = a.take<float>((size_t)T * H);
  x.winexp = a.take<float>((size_t)((T + kWindow - 1) / kWindow) * H);
  x.rownorm = a.take<float>((size_t)T * Hkv);
  x.winnorm = a.take<float>((size_t)((T + kWindow - 1) / kWindow) * Hkv);
  x.taken = a.take<uint32_t>(1);
  const size_t n = parts > 1 ? (size_t)T * Hkv * parts * d : 0;
  x.dk = a.take<float>(n);
  x.dv = a.take<float>(n);
  if (w) *w = x;
  return a.used;
}

template <int D>
int bwd_t(const uint16_t* qkv, const PackedIndex& x, const uint16_t* o, const float* lse,
          const uint16_t* dout, int64_t T, int H, int Hkv, const float2* cs, uint16_t* dqkv,
          int parts, const BwdWs& w, cudaStream_t st) {
  static bool attr[64] = {false};
  constexpr uint32_t smem = std::max(DkvSmem<D>::kBytes, DqSmem<D>::kBytes);
  LSQ_TRY(allow_smem(packed_attn_bwd_kernel<D>, (int)smem, attr));
  int* err = device_status_ptr();
  if (!err) return set_error(LSQ_ERR_CUDA, "device status word unavailable");
  const float scale = 1.f / sqrtf((float)D);
  const float sl2 = kLog2e * scale;
  const unsigned windows = (unsigned)((T + kWindow - 1) / kWindow);
  LSQ_CUDA(launch_dep(packed_attn_prep_kernel<D>, dim3(windows, (unsigned)(H + Hkv)), 256, 0, st,
                      qkv, o, dout, lse, x.head, T, H, Hkv, w.dos, w.stats, w.rowexp, w.winexp,
                      w.rownorm, w.winnorm, w.taken, err));
  const int64_t row = (int64_t)(H + 2 * Hkv) * D, hd = (int64_t)H * D;
  CUtensorMap qkv128, qkv64, do128, do64;
  LSQ_TRY(make_tmap_2d(&qkv128, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, qkv, (uint64_t)row, (uint64_t)T,
                       (uint64_t)row, 64, 128, CU_TENSOR_MAP_SWIZZLE_128B));
  LSQ_TRY(make_tmap_2d(&qkv64, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, qkv, (uint64_t)row, (uint64_t)T,
                       (uint64_t)row, 64, kBC, CU_TENSOR_MAP_SWIZZLE_128B));
  LSQ_TRY(make_tmap_2d(&do128, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, w.dos, (uint64_t)hd, (uint64_t)T,
                       (uint64_t)hd, 64, 128, CU_TENSOR_MAP_SWIZZLE_128B));
  LSQ_TRY(make_tmap_2d(&do64, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, w.dos, (uint64_t)hd, (uint64_t)T,
                       (uint64_t)hd, 64, kBC, CU_TENSOR_MAP_SWIZZLE_128B));
  const int sms = gemm_num_sms();
  // (at most: the documents' tiles are known on the device)
  const int64_t kitems = (int64_t)x.cap * Hkv * parts;
  const int64_t qitems = (H / Hkv) % 2 == 0 ? (int64_t)x.cap * (H / 2) : (int64_t)x.cap2 * H;
  const BwdArgs args{x, w.stats, w.rowexp, w.winexp, w.rownorm, w.winnorm, T, H, Hkv, H / Hkv / parts, sl2, scale, cs,
                     dqkv, w.dk, w.dv, w.taken, err};
  LSQ_CUDA(launch_dep(packed_attn_bwd_kernel<D>, dim3((unsigned)std::min<int64_t>(kitems + qitems, sms)),
                      kBThreads, smem, st, qkv128, qkv64, do128, do64, args));
  if (parts > 1) {
    // a thread for four pairs of columns of a token
    const int64_t n = T * 4 * Hkv * (D / 16);
    const unsigned grid = (unsigned)std::min<int64_t>((n + 255) / 256, (int64_t)sms * 8);
    LSQ_CUDA(launch_dep(packed_attn_sum_kernel<D>, dim3(grid), 256, 0, st, w.dk, w.dv, parts, x.head,
                        T, x.pos, Hkv, row, H * D, cs, dqkv));
  }
  return LSQ_OK;
}

constexpr int kMaxHeads = 32767;  // (H + Hkv is a grid dimension)
bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

int check_heads(int64_t T, int32_t H, int32_t Hkv, int32_t d, const char* who) {
  if (H <= 0 || Hkv <= 0 || H % Hkv != 0 || H > kMaxHeads)
    return set_error(LSQ_ERR_SHAPE, "%s: H must be a multiple of Hkv, at most %d", who, kMaxHeads);
  if (d != 64 && d != 128) return set_error(LSQ_ERR_SHAPE, "%s: d must be 64 or 128", who);
  // (items are counted in 32 bits; such a qkv would take 256 GiB)
  if (T * (H + 2 * (int64_t)Hkv) >= (int64_t(1) << 31))
    return set_error(LSQ_ERR_SHAPE, "%s: T (H + 2 Hkv) must be below 2^31", who);
  return LSQ_OK;
}

}  // namespace

int launch_packed_attention_fwd(const uint16_t* qkv, const int32_t* index, int n_docs, int64_t T,
                                int H, int Hkv, int d, uint16_t* o, float* lse, cudaStream_t st) {
  const PackedIndex x = packed_index_view(index, T, n_docs);
  const int prof = prof_begin(st);
  LSQ_TRY(d == 128 ? fwd_t<128>(qkv, x, T, H, Hkv, o, lse, st)
                   : fwd_t<64>(qkv, x, T, H, Hkv, o, lse, st));
  // (the pairs depend on the documents, which the host does not know)
  if (prof >= 0)
    prof_end(prof, st, "packed_attention_fwd", 0.0,
             2.0 * T * (double)(2 * H + 2 * Hkv) * d + 4.0 * T * H);
  return LSQ_OK;
}

size_t packed_attention_ws_bytes(int64_t T, int H, int Hkv, int d) {
  return carve_bwd(T, H, Hkv, d, nullptr, nullptr);
}

int launch_packed_attention_bwd(const uint16_t* qkv, const int32_t* index, int n_docs,
                                const uint16_t* o, const float* lse, const uint16_t* dout,
                                int64_t T, int H, int Hkv, int d, const float2* cs, uint16_t* dqkv,
                                void* ws, size_t ws_bytes, cudaStream_t st) {
  const PackedIndex x = packed_index_view(index, T, n_docs);
  BwdWs w;
  if (carve_bwd(T, H, Hkv, d, ws, &w) > ws_bytes)
    return set_error(LSQ_ERR_WORKSPACE, "packed attention: workspace too small");
  const int parts = dkv_parts(T, n_docs, H, Hkv);
  const int prof = prof_begin(st);
  LSQ_TRY(d == 128 ? bwd_t<128>(qkv, x, o, lse, dout, T, H, Hkv, cs, dqkv, parts, w, st)
                   : bwd_t<64>(qkv, x, o, lse, dout, T, H, Hkv, cs, dqkv, parts, w, st));
  if (prof >= 0)
    prof_end(prof, st, "packed_attention_bwd", 0.0,
             2.0 * T * (double)(4 * H + 4 * Hkv) * d + 4.0 * T * H);
  return LSQ_OK;
}

}  // namespace lsq

using namespace lsq;

extern "C" int packed_attention_fwd(const uint16_t* qkv, const int32_t* index, int32_t n_docs,
                                    int64_t T, int32_t H, int32_t Hkv, int32_t d, uint16_t* o,
                                    float* lse, void* stream) {
  LSQ_TRY(check_packed(T, n_docs, index, "packed_attention_fwd"));
  LSQ_TRY(check_heads(T, H, Hkv, d, "packed_attention_fwd"));
  if (!qkv || !o || !lse) return set_error(LSQ_ERR_INVALID, "packed_attention_fwd: null pointer");
  if (!aligned16(qkv) || !aligned32(o) || !aligned16(lse))
    return set_error(LSQ_ERR_ALIGN,
                     "packed_attention_fwd: pointers must be 16-byte aligned, o 32-byte");
  return launch_packed_attention_fwd(qkv, index, n_docs, T, H, Hkv, d, o, lse,
                                     static_cast<cudaStream_t>(stream));
}

extern "C" size_t packed_attention_workspace_bytes(int64_t T, int32_t H, int32_t Hkv, int32_t d) {
  if (T <= 0 || T > (int64_t(1) << 30) || check_heads(T, H, Hkv, d, "packed_attention") != LSQ_OK)
    return 0;
  return packed_attention_ws_bytes(T, H, Hkv, d);
}

extern "C" int packed_attention_bwd(const uint16_t* qkv, const int32_t* index, int32_t n_docs,
                                    const uint16_t* o, const float* lse, const uint16_t* dout,
                                    int64_t T, int32_t H, int32_t Hkv, int32_t d, uint16_t* dqkv,
                                    void* ws, size_t ws_bytes, void* stream) {
  LSQ_TRY(check_packed(T, n_docs, index, "packed_attention_bwd"));
  LSQ_TRY(check_heads(T, H, Hkv, d, "packed_attention_bwd"));
  if (!qkv || !o || !lse || !dout || !dqkv)
    return set_error(LSQ_ERR_INVALID, "packed_attention_bwd: null pointer");
  if (!aligned16(qkv) || !aligned16(o) || !aligned16(lse) || !aligned16(dout) || !aligned32(dqkv))
    return set_error(LSQ_ERR_ALIGN,
                     "packed_attention_bwd: pointers must be 16-byte aligned, dqkv 32-byte");
  const size_t need = packed_attention_ws_bytes(T, H, Hkv, d);
  if (!ws || ws_bytes < need)
    return set_error(LSQ_ERR_WORKSPACE, "packed_attention_bwd: workspace %zu < %zu", ws_bytes, need);
  if (!aligned32(ws))
    return set_error(LSQ_ERR_ALIGN, "packed_attention_bwd: the workspace must be 32-byte aligned");
  return launch_packed_attention_bwd(qkv, index, n_docs, o, lse, dout, T, H, Hkv, d, nullptr, dqkv,
                                     ws, ws_bytes, static_cast<cudaStream_t>(stream));
}
