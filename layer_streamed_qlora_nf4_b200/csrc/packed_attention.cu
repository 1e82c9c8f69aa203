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
// first (dO' = 2^e dO with a norm in [8, 16)), which loses nothing of bf16's 8 bits,
// and the factors are taken out again in fp32.  Every sum has a fixed order, so the
// results are deterministic.
#include <cuda.h>
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "packed.cuh"

namespace lsq {

namespace {

__device__ __forceinline__ uint8_t* align1024_p(uint8_t* p) {
  return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(p) + 1023) & ~uintptr_t(1023));
}

// 2^x (relative error 2^-22; results below 2^-126 are 0)
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
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
  static constexpr int kRing = D == 128 ? 5 : 8;     // K and V tiles in flight
  static constexpr uint32_t kBytes = 1024 + (2 + kRing) * kTile;
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
  const PackedTile t = heads ? x.tiles[w / per] : x.tiles2[w / per];
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
    packed_attn_fwd_kernel(const __grid_constant__ CUtensorMap tm_qkv, PackedIndex idx, int64_t T,
                           int H, int Hkv, uint16_t* __restrict__ out,
                           float* __restrict__ lse_out, float sl2, int* __restrict__ dev_err) {
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
  pdl_trigger();  // the next kernel may launch once all CTAs of this one run

  uint8_t* Qs = align1024_p(attn_raw);   // [2] Q tiles
  uint8_t* KV = Qs + 2 * SM::kTile;      // ring: K and V tiles in turn
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
  if (warp == kWarpTma && lane == 0) tma_prefetch_desc(&tm_qkv);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_sh;
  pdl_wait();  // the index and q, k, v come from the kernels before
  const int items = heads ? idx.head[0] * (H / 2) : idx.head[1] * H;
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    return mbar_wait_bounded(smem_u32(bar), parity & 1u, abort_flag, dev_err, DEV_ERR_WAIT_GEMM);
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
    bool ok = true;
    for (int k = 0, w; ok && (w = deal(k, items)) >= 0; ++k) {
      const FwdItem it = fwd_item(idx, w, H, heads, s);
      const int n = it.n;
      if (n == 0) continue;
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
        const float nm = -m_ref;
        float rs0 = 0.f, rs1 = 0.f;
#pragma unroll
        for (int c = 0; c < kStep / 32; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float p0 = ex2(fmaf(__uint_as_float(sv[32 * c + e]), sl2, nm));
            const float p1 = ex2(fmaf(__uint_as_float(sv[32 * c + e + 1]), sl2, nm));
            rs0 += p0;
            rs1 += p1;
            pk[e >> 1] = pack_f16x2(p0, p1);
          }
          tmem_st16(ts + 16 * c, pk);
        }
        l_run += rs0 + rs1;
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&p_full[s][u & 1]));
      }
      // -------------------------------------------------------------- epilogue
      // (a barrier of its own: pv_done may be two phases on, where a wait for the
      // phase before the last would not return)
      ok = ok && wait_all(&o_full[s], no);
      if (!ok) break;
      ++no;
      nv += n;
      tc_fence_after();
      const float inv = 1.f / l_run;
      const bool live = q < it.end;
      uint16_t* orow = out + (int64_t)q * H * D + (int64_t)it.head * D;
      uint32_t ov[D];
#pragma unroll
      for (int c = 0; c < D / 32; ++c) tmem_ld32(to + 32 * c, ov + 32 * c);
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&o_free[s]));
      if (live) {
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          uint32_t pk[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            pk[e] = pack_f16x2(__uint_as_float(ov[8 * c + 2 * e]) * inv,
                               __uint_as_float(ov[8 * c + 2 * e + 1]) * inv);
          *reinterpret_cast<uint4*>(orow + 8 * c) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
        }
        lse_out[(int64_t)it.head * T + q] = (m_ref + log2f(l_run)) * 0.69314718055994531f;
      }
    }
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
constexpr int kBThreads = 320;
constexpr int kBC = 64;  // columns of a chunk (queries for dK/dV, keys for dQ)

// Clears rows [rows, all) of two tiles that share a barrier (one warp) once their load has
// landed, and arrives on `done`; whole tiles only arrive.
template <int D>
__device__ __forceinline__ void zero_tail2(uint8_t* a, uint8_t* b, int rows, int all, uint32_t bar,
                                           uint32_t parity, int lane, uint32_t done,
                                           volatile int* abort_flag, int* dev_err) {
  if (rows < all) {
    bool ok = mbar_wait_bounded(bar, parity, abort_flag, dev_err, DEV_ERR_WAIT_GEMM);
    ok = __all_sync(0xFFFFFFFFu, ok);
    if (ok)
      for (int k = 0; k < D / 64; ++k)
        for (uint32_t o = (uint32_t)rows * 128u + (uint32_t)lane * 16u; o < (uint32_t)all * 128u;
             o += 512u) {
          *reinterpret_cast<uint4*>(a + (uint32_t)k * all * 128u + o) = make_uint4(0u, 0u, 0u, 0u);
          *reinterpret_cast<uint4*>(b + (uint32_t)k * all * 128u + o) = make_uint4(0u, 0u, 0u, 0u);
        }
    fence_proxy_async_smem();
  }
  __syncwarp();
  if (lane == 0) mbar_arrive(done);
}

// One warp per token and query head: dO' = fp16(2^e dO) with e such that the row's norm
// is in [8, 16), delta' = 2^e rowsum(dO o O), and e.  A zero row takes e = 127 (it must
// not lower the least exponent of a tile); a row that is not finite e = 0, and its
// gradients come out not finite.  Warps T H .. check the norms of the v rows.
template <int D>
__global__ void __launch_bounds__(256)
    packed_attn_prep_kernel(const uint16_t* __restrict__ qkv, const uint16_t* __restrict__ o,
                            const uint16_t* __restrict__ dout, const int* __restrict__ head,
                            int64_t T, int H, int Hkv, uint16_t* __restrict__ dos,
                            float* __restrict__ delta, float* __restrict__ rowexp, int* dev_err) {
  constexpr int E = D / 32;  // elements per lane
  pdl_trigger();
  pdl_wait();
  const int64_t w = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  const int64_t live = head[2];
  if (w >= T * H) {
    const int64_t t = (w - T * H) / Hkv;
    if (t >= live) return;
    const uint16_t* v = qkv + t * (int64_t)(H + 2 * Hkv) * D +
                        (int64_t)(H + Hkv + (w - T * H) % Hkv) * D + lane * E;
    float n = 0.f;
#pragma unroll
    for (int i = 0; i < E; i += 2) {
      const float2 x = unpack_f16x2(*reinterpret_cast<const uint32_t*>(v + i));
      n += x.x * x.x + x.y * x.y;
    }
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) n += __shfl_xor_sync(0xFFFFFFFFu, n, k);
    if (lane == 0 && !(n <= 2047.f * 2047.f)) atomicOr(dev_err, DEV_ERR_NONFINITE);
    return;
  }
  const int64_t t = w / H;
  const int h = (int)(w % H);
  const int64_t at = w * D + lane * E;
  float g[E];
  float n = 0.f, dl = 0.f;
#pragma unroll
  for (int i = 0; i < E; i += 2) {
    const float2 x = unpack_bf16x2(*reinterpret_cast<const uint32_t*>(dout + at + i));
    const float2 y = unpack_f16x2(*reinterpret_cast<const uint32_t*>(o + at + i));
    g[i] = t < live ? x.x : 0.f;
    g[i + 1] = t < live ? x.y : 0.f;
    dl += g[i] * y.x + g[i + 1] * y.y;
    n = fmaxf(n, fmaxf(fabsf(g[i]), fabsf(g[i + 1])));
    if (!(fabsf(g[i]) <= 3.4e38f && fabsf(g[i + 1]) <= 3.4e38f)) n = INFINITY;
  }
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) {
    dl += __shfl_xor_sync(0xFFFFFFFFu, dl, k);
    n = fmaxf(n, __shfl_xor_sync(0xFFFFFFFFu, n, k));
  }
  // the norm from values near 1, so that its squares neither overflow nor vanish
  int e = 0;
  if (n > 0.f && n <= 3.4e38f) {
    int x;
    frexpf(n, &x);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const float y = ldexpf(g[i], -x);
      s += y * y;
    }
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, k);
    int z;
    frexpf(sqrtf(s), &z);  // the norm is in [2^(x + z - 1), 2^(x + z))
    e = 4 - x - z;
  } else if (n == 0.f) {
    e = 127;
  }
  e = min(e, 127);
  uint32_t p[E / 2];
#pragma unroll
  for (int i = 0; i < E; i += 2) p[i / 2] = pack_f16x2(ldexpf(g[i], e), ldexpf(g[i + 1], e));
  if (E == 4)
    *reinterpret_cast<uint2*>(dos + at) = make_uint2(p[0], p[E / 2 - 1]);
  else
    *reinterpret_cast<uint32_t*>(dos + at) = p[0];
  if (lane == 0) {
    delta[(int64_t)h * T + t] = t < live ? ldexpf(dl, e) : 0.f;
    rowexp[(int64_t)h * T + t] = (float)e;
  }
}

template <int D>
struct PaDkvSmem {
  static constexpr uint32_t kKV = kAK * D * 2;   // K (fp16) or V (bf16): 128 keys
  static constexpr uint32_t kQc = kBC * D * 2;   // a chunk of Q or dO: 64 queries
  static constexpr uint32_t kPc = kAK * kBC * 2; // P^T or dS^T: 128 keys x 64 queries
  static constexpr uint32_t kBytes = 1024 + 2 * kKV + 4 * kQc + 2 * kPc;
};

// dK, dV of 128 keys for one query head: loops over the 64-query chunks at and
// after the key block (causal), accumulating dV += P^T dO and dK += dS^T Q in
// TMEM; writes dk = scale dK and dv per query head.
template <int D>
__global__ void __launch_bounds__(kBThreads, 1)
    packed_attn_dkdv_kernel(const __grid_constant__ CUtensorMap tm_kv,   // qkv, boxes of 128 rows
                            const __grid_constant__ CUtensorMap tm_q,    // qkv, boxes of 64 rows
                            const __grid_constant__ CUtensorMap tm_do,   // dO', boxes of 64 rows
                            PackedIndex idx, const float* __restrict__ lse,
                            const float* __restrict__ delta, const float* __restrict__ rowexp,
                            int64_t T, int H, int Hkv, float sl2, float scale,
                            float* __restrict__ dk, float* __restrict__ dv, int* __restrict__ dev_err) {
  using SM = PaDkvSmem<D>;
  constexpr int DA = D / 64;
  extern __shared__ uint8_t dkv_raw[];
  __shared__ __align__(8) uint64_t bar_kv, bar_tail, bar_q[2], bar_qfree[2], bar_sdp[2],
      bar_tfree[2], bar_ds, bar_pds;
  __shared__ uint32_t tmem_sh;
  __shared__ int abort_sh;
  volatile int* abort_flag = &abort_sh;
  pdl_trigger();

  uint8_t* Ks = align1024_p(dkv_raw);
  uint8_t* Vs = Ks + SM::kKV;
  uint8_t* Qb = Vs + SM::kKV;       // [2] Q chunks (fp16, then bf16)
  uint8_t* dOb = Qb + 2 * SM::kQc;  // [2] dO chunks (bf16)
  uint8_t* Pt = dOb + 2 * SM::kQc;  // P^T (bf16, K-major over queries)
  uint8_t* dSt = Pt + SM::kPc;      // dS^T
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.y;
  const int g = h / (H / Hkv);
  pdl_wait();
  if ((int)blockIdx.x >= idx.head[0]) return;
  const PackedTile tile = idx.tiles[blockIdx.x];
  const int k0 = tile.row0;
  // the queries that see some of these keys: from the first key on, or, where the
  // tile reaches into the prompt, the whole document
  const int qs = k0 < tile.prompt ? tile.begin : k0;
  const int nc = (tile.end - qs + kBC - 1) / kBC;
  constexpr uint32_t kColS = 0, kColP = 2 * kBC, kColV = 4 * kBC, kColK = 4 * kBC + 128;

  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&bar_kv), 1);
    mbar_init(smem_u32(&bar_tail), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&bar_q[i]), 1);
      mbar_init(smem_u32(&bar_qfree[i]), 1);
      mbar_init(smem_u32(&bar_sdp[i]), 1);
      mbar_init(smem_u32(&bar_tfree[i]), 8);
    }
    mbar_init(smem_u32(&bar_ds), 8);
    mbar_init(smem_u32(&bar_pds), 1);
    abort_sh = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == kWarpMma) {
    tmem_alloc(smem_u32(&tmem_sh), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_sh;

  if (warp == kWarpTma) {
    if (lane == 0) {
      mbar_arrive_expect_tx(smem_u32(&bar_kv), 2 * SM::kKV);
      for (int a = 0; a < DA; ++a) {
        tma_load_2d(smem_u32(Ks + a * kAK * 128), &tm_kv, smem_u32(&bar_kv), (H + g) * D + 64 * a,
                    k0);
        tma_load_2d(smem_u32(Vs + a * kAK * 128), &tm_kv, smem_u32(&bar_kv),
                    (H + Hkv + g) * D + 64 * a, k0);
      }
      for (int c = 0; c < nc; ++c) {
        const int qb = c & 1;
        if (c >= 2 && !mbar_wait_bounded(smem_u32(&bar_qfree[qb]), (uint32_t)(((c - 2) >> 1) & 1),
                                         abort_flag, dev_err, DEV_ERR_WAIT_GEMM))
          break;
        const int row = qs + c * kBC;
        const uint32_t fb = smem_u32(&bar_q[qb]);
        mbar_arrive_expect_tx(fb, 2 * SM::kQc);
        for (int a = 0; a < DA; ++a) {
          tma_load_2d(smem_u32(Qb + qb * SM::kQc + a * kBC * 128), &tm_q, fb, h * D + 64 * a, row);
          tma_load_2d(smem_u32(dOb + qb * SM::kQc + a * kBC * 128), &tm_do, fb, h * D + 64 * a, row);
        }
      }
    }
    __syncwarp();
    // rows of the last chunk behind the document are cleared: their P and dS are 0,
    // and 0 * inf would reach this document's gradients
    const int lb = (nc - 1) & 1;
    zero_tail2<D>(Qb + lb * SM::kQc, dOb + lb * SM::kQc, tile.end - qs - (nc - 1) * kBC, kBC,
                  smem_u32(&bar_q[lb]), (uint32_t)(((nc - 1) >> 1) & 1), lane, smem_u32(&bar_tail),
                  abort_flag, dev_err);
  } else if (warp == kWarpMma) {
    if (lane == 0) {
      const uint32_t id_s = umma_idesc_f16(kAK, kBC);            // S^T = K Q^T (fp16)
      const uint32_t id_dp = id_s;                                // dP'^T = V dO'^T
      const uint32_t id_acc = umma_idesc_f16(kAK, D) | (1u << 16);  // dV, dK: B MN-major
      bool ok = mbar_wait_bounded(smem_u32(&bar_kv), 0u, abort_flag, dev_err, DEV_ERR_WAIT_GEMM);
      auto issue_sdp = [&](int c) -> bool {
        const int qb = c & 1;
        if (!mbar_wait_bounded(smem_u32(&bar_q[qb]), (uint32_t)((c >> 1) & 1), abort_flag, dev_err,
                               DEV_ERR_WAIT_GEMM))
          return false;
        if (c >= 2 && !mbar_wait_bounded(smem_u32(&bar_tfree[qb]), (uint32_t)(((c - 2) >> 1) & 1),
                                         abort_flag, dev_err, DEV_ERR_WAIT_GEMM))
          return false;
        // (the last chunk's tail is cleared before any product reads it)
        if (c == nc - 1 && !mbar_wait_bounded(smem_u32(&bar_tail), 0u, abort_flag, dev_err,
                                              DEV_ERR_WAIT_GEMM))
          return false;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t ka = (uint32_t)((kk >> 2) * kAK * 128 + (kk & 3) * 32);
          const uint32_t kq = (uint32_t)((kk >> 2) * kBC * 128 + (kk & 3) * 32);
          tc_mma_bf16(tmem + kColS + (uint32_t)qb * kBC, umma_desc_k_sw128(smem_u32(Ks) + ka),
                      umma_desc_k_sw128(smem_u32(Qb + qb * SM::kQc) + kq), id_s, kk > 0 ? 1u : 0u);
          tc_mma_bf16(tmem + kColP + (uint32_t)qb * kBC, umma_desc_k_sw128(smem_u32(Vs) + ka),
                      umma_desc_k_sw128(smem_u32(dOb + qb * SM::kQc) + kq), id_dp, kk > 0 ? 1u : 0u);
        }
        tc_commit(smem_u32(&bar_sdp[qb]));
        return true;
      };
      ok = ok && issue_sdp(0);
      for (int c = 0; c < nc && ok; ++c) {
        const int qb = c & 1;
        if (c + 1 < nc) ok = issue_sdp(c + 1);
        if (!ok) break;
        ok = mbar_wait_bounded(smem_u32(&bar_ds), (uint32_t)(c & 1), abort_flag, dev_err,
                               DEV_ERR_WAIT_GEMM);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < kBC / 16; ++kk) {
          const uint32_t pa = (uint32_t)(kk * 32);
          const uint32_t bo = (uint32_t)kk * 16 * 128;
          const uint32_t acc = (c > 0 || kk > 0) ? 1u : 0u;
          tc_mma_bf16(tmem + kColV, umma_desc_k_sw128(smem_u32(Pt) + pa),
                      umma_desc_mn_sw128(smem_u32(dOb + qb * SM::kQc) + bo, kBC * 128, 1024u), id_acc,
                      acc);
          tc_mma_bf16(tmem + kColK, umma_desc_k_sw128(smem_u32(dSt) + pa),
                      umma_desc_mn_sw128(smem_u32(Qb + qb * SM::kQc) + bo, kBC * 128, 1024u), id_acc,
                      acc);
        }
        tc_commit(smem_u32(&bar_pds));       // P^T, dS^T read; dK, dV updated
        tc_commit(smem_u32(&bar_qfree[qb]));  // the Q and dO chunk read
      }
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- gradient warps
    const int r = (warp & 3) * 32 + lane;      // key row of the block = TMEM lane
    const int hf = warp >> 2;                  // queries 32 hf .. of each chunk
    const int kpos = k0 + r;
    // the queries that see this key
    const int qlo = kpos < tile.prompt ? tile.begin : kpos;
    const int qhi = kpos < tile.end ? tile.end : 0;
    const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const float* lse_h = lse + (int64_t)h * T;
    const float* delta_h = delta + (int64_t)h * T;
    const float* exp_h = rowexp + (int64_t)h * T;
    // the least of the queries' exponents: P is scaled by 2^(emin - e) <= 1, so that
    // the products with dO' = 2^e dO all carry the factor 2^emin
    float emin = INFINITY;
    for (int q = qs + lane; q < tile.end; q += 32) emin = fminf(emin, __ldg(exp_h + q));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) emin = fminf(emin, __shfl_xor_sync(0xFFFFFFFFu, emin, o));
    bool ok = true;
    // lse (log2 units, with the scale) and delta of the warp's 32 queries of a chunk:
    // lane i holds query i's, fetched one chunk ahead, and the lanes read them by shuffle
    auto fetch = [&](int c, float* l2v, float* dlv) {
      const int qq = min(qs + c * kBC + 32 * hf + lane, tile.end - 1);
      *l2v = __ldg(lse_h + qq) * 1.4426950408889634f + (__ldg(exp_h + qq) - emin);
      *dlv = __ldg(delta_h + qq);
    };
    float l2_own = 0.f, dl_own = 0.f;
    fetch(0, &l2_own, &dl_own);
    for (int c = 0; c < nc && ok; ++c) {
      const int qb = c & 1;
      const int q0 = qs + c * kBC + 32 * hf;  // this thread's first query
      float l2_next = 0.f, dl_next = 0.f;
      if (c + 1 < nc) fetch(c + 1, &l2_next, &dl_next);
      ok = mbar_wait_bounded(smem_u32(&bar_sdp[qb]), (uint32_t)((c >> 1) & 1), abort_flag, dev_err,
                             DEV_ERR_WAIT_GEMM);
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok) break;
      tc_fence_after();
      uint32_t sv[2][16], pv[2][16];
      tmem_ld16(trow + kColS + (uint32_t)(qb * kBC + 32 * hf), sv[0]);
      tmem_ld16(trow + kColS + (uint32_t)(qb * kBC + 32 * hf + 16), sv[1]);
      tmem_ld16(trow + kColP + (uint32_t)(qb * kBC + 32 * hf), pv[0]);
      tmem_ld16(trow + kColP + (uint32_t)(qb * kBC + 32 * hf + 16), pv[1]);
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bar_tfree[qb]));
      uint32_t ppk[16], dpk[16];
#pragma unroll
      for (int e = 0; e < 32; e += 2) {
        float p[2], d[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int qq = q0 + e + u;
          const bool live = qlo <= qq && qq < qhi;
          const float s = __uint_as_float(sv[(e + u) >> 4][(e + u) & 15]);
          const float dp = __uint_as_float(pv[(e + u) >> 4][(e + u) & 15]);
          const float l2 = __shfl_sync(0xFFFFFFFFu, l2_own, e + u);
          const float dl = __shfl_sync(0xFFFFFFFFu, dl_own, e + u);
          p[u] = live ? ex2(fmaf(s, sl2, -l2)) : 0.f;
          d[u] = live ? p[u] * (dp - dl) : 0.f;
        }
        ppk[e >> 1] = pack_f16x2(p[0], p[1]);
        dpk[e >> 1] = pack_f16x2(d[0], d[1]);
      }
      // the previous chunk's dV, dK products have read P^T and dS^T
      if (c > 0) {
        ok = mbar_wait_bounded(smem_u32(&bar_pds), (uint32_t)((c - 1) & 1), abort_flag, dev_err,
                               DEV_ERR_WAIT_GEMM);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
      }
#pragma unroll
      for (int cc = 0; cc < 4; ++cc) {
        const uint32_t off = sw128_offset((uint32_t)r, (uint32_t)(hf * 4 + cc));
        *reinterpret_cast<uint4*>(Pt + off) =
            make_uint4(ppk[4 * cc], ppk[4 * cc + 1], ppk[4 * cc + 2], ppk[4 * cc + 3]);
        *reinterpret_cast<uint4*>(dSt + off) =
            make_uint4(dpk[4 * cc], dpk[4 * cc + 1], dpk[4 * cc + 2], dpk[4 * cc + 3]);
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bar_ds));
      l2_own = l2_next;
      dl_own = dl_next;
    }
    // ---------------------------------------------------------------- epilogue
    if (ok) ok = mbar_wait_bounded(smem_u32(&bar_pds), (uint32_t)((nc - 1) & 1), abort_flag,
                                   dev_err, DEV_ERR_WAIT_GEMM);
    ok = __all_sync(0xFFFFFFFFu, ok);
    if (ok) {
      tc_fence_after();
      const bool live = kpos < tile.end;
      const float unscale = exp2f(-emin), ks = scale * unscale;
      const int64_t o = (int64_t)kpos * (int64_t)H * D + (int64_t)h * D + hf * (D / 2);
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t kv[16], vv[16];
        tmem_ld16(trow + kColK + (uint32_t)(hf * (D / 2) + 16 * c), kv);
        tmem_ld16(trow + kColV + (uint32_t)(hf * (D / 2) + 16 * c), vv);
        tmem_ld_wait();
        if (live) {
#pragma unroll
          for (int e = 0; e < 16; e += 4) {
            *reinterpret_cast<float4*>(dk + o + 16 * c + e) =
                make_float4(__uint_as_float(kv[e]) * ks, __uint_as_float(kv[e + 1]) * ks,
                            __uint_as_float(kv[e + 2]) * ks, __uint_as_float(kv[e + 3]) * ks);
            *reinterpret_cast<float4*>(dv + o + 16 * c + e) =
                make_float4(__uint_as_float(vv[e]) * unscale, __uint_as_float(vv[e + 1]) * unscale,
                            __uint_as_float(vv[e + 2]) * unscale, __uint_as_float(vv[e + 3]) * unscale);
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (abort_sh) settle_ns(2000000);
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D>
struct PaDqSmem {
  static constexpr uint32_t kQ = kAQ * D * 2;    // Q (fp16) or dO (bf16): 128 queries
  static constexpr uint32_t kKc = kBC * D * 2;   // a chunk of K or V: 64 keys
  static constexpr uint32_t kSc = kAQ * kBC * 2; // dS: 128 queries x 64 keys
  static constexpr uint32_t kBytes = 1024 + 2 * kQ + 4 * kKc + kSc;
};

// dQ of 128 queries for one query head: loops over the 64-key chunks up to the
// queries (causal), accumulating dQ += dS K in TMEM; writes dq = scale dQ.
template <int D>
__global__ void __launch_bounds__(kBThreads, 1)
    packed_attn_dq_kernel(const __grid_constant__ CUtensorMap tm_q,    // qkv, boxes of 128 rows
                          const __grid_constant__ CUtensorMap tm_kv,   // qkv, boxes of 64 rows
                          const __grid_constant__ CUtensorMap tm_do,   // dO', boxes of 128 rows
                          PackedIndex idx, const float* __restrict__ lse,
                          const float* __restrict__ delta, const float* __restrict__ rowexp,
                          int64_t T, int H, int Hkv, float sl2, float scale,
                          float* __restrict__ dq, int* __restrict__ dev_err) {
  using SM = PaDqSmem<D>;
  constexpr int DA = D / 64;
  extern __shared__ uint8_t dq_raw[];
  __shared__ __align__(8) uint64_t bar_qd, bar_kv[2], bar_tail, bar_kvfree[2], bar_sdp[2],
      bar_tfree[2], bar_ds, bar_dsfree;
  __shared__ uint32_t tmem_sh;
  __shared__ int abort_sh;
  volatile int* abort_flag = &abort_sh;
  pdl_trigger();

  uint8_t* Qs = align1024_p(dq_raw);
  uint8_t* dOs = Qs + SM::kQ;
  uint8_t* Kb = dOs + SM::kQ;       // [2] K chunks (fp16, then bf16)
  uint8_t* Vb = Kb + 2 * SM::kKc;   // [2] V chunks (bf16)
  uint8_t* dSs = Vb + 2 * SM::kKc;  // dS (fp16, K-major over keys)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.y;
  const int g = h / (H / Hkv);
  pdl_wait();
  if ((int)blockIdx.x >= idx.head[0]) return;
  const PackedTile tile = idx.tiles[blockIdx.x];
  const int q0 = tile.row0;
  const int kv_end = min(tile.end, max(q0 + kAQ, tile.prompt));  // keys this block sees
  const int nc = (kv_end - tile.begin + kBC - 1) / kBC;
  constexpr uint32_t kColS = 0, kColP = 2 * kBC, kColQ = 4 * kBC;

  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&bar_qd), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&bar_kv[i]), 1);
      mbar_init(smem_u32(&bar_kvfree[i]), 1);
      mbar_init(smem_u32(&bar_sdp[i]), 1);
      mbar_init(smem_u32(&bar_tfree[i]), 8);
    }
    mbar_init(smem_u32(&bar_ds), 8);
    mbar_init(smem_u32(&bar_dsfree), 1);
    mbar_init(smem_u32(&bar_tail), 1);
    abort_sh = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == kWarpMma) {
    tmem_alloc(smem_u32(&tmem_sh), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_sh;

  if (warp == kWarpTma) {
    if (lane == 0) {
      mbar_arrive_expect_tx(smem_u32(&bar_qd), 2 * SM::kQ);
      for (int a = 0; a < DA; ++a) {
        tma_load_2d(smem_u32(Qs + a * kAQ * 128), &tm_q, smem_u32(&bar_qd), h * D + 64 * a,
                    q0);
        tma_load_2d(smem_u32(dOs + a * kAQ * 128), &tm_do, smem_u32(&bar_qd), h * D + 64 * a,
                    q0);
      }
      for (int c = 0; c < nc; ++c) {
        const int kb = c & 1;
        if (c >= 2 && !mbar_wait_bounded(smem_u32(&bar_kvfree[kb]), (uint32_t)(((c - 2) >> 1) & 1),
                                         abort_flag, dev_err, DEV_ERR_WAIT_GEMM))
          break;
        const int row = tile.begin + c * kBC;
        const uint32_t fb = smem_u32(&bar_kv[kb]);
        mbar_arrive_expect_tx(fb, 2 * SM::kKc);
        for (int a = 0; a < DA; ++a) {
          tma_load_2d(smem_u32(Kb + kb * SM::kKc + a * kBC * 128), &tm_kv, fb, (H + g) * D + 64 * a,
                      row);
          tma_load_2d(smem_u32(Vb + kb * SM::kKc + a * kBC * 128), &tm_kv, fb,
                      (H + Hkv + g) * D + 64 * a, row);
        }
      }
    }
    __syncwarp();
    const int lb = (nc - 1) & 1;  // (as in the kernel above: keys behind the last one)
    zero_tail2<D>(Kb + lb * SM::kKc, Vb + lb * SM::kKc, kv_end - tile.begin - (nc - 1) * kBC, kBC,
                  smem_u32(&bar_kv[lb]), (uint32_t)(((nc - 1) >> 1) & 1), lane, smem_u32(&bar_tail),
                  abort_flag, dev_err);
  } else if (warp == kWarpMma) {
    if (lane == 0) {
      const uint32_t id_s = umma_idesc_f16(kAQ, kBC);            // S = Q K^T (fp16)
      const uint32_t id_dp = id_s;                                // dP' = dO' V^T
      const uint32_t id_acc = umma_idesc_f16(kAQ, D) | (1u << 16);  // dQ += dS K: B MN-major
      bool ok = mbar_wait_bounded(smem_u32(&bar_qd), 0u, abort_flag, dev_err, DEV_ERR_WAIT_GEMM);
      auto issue_sdp = [&](int c) -> bool {
        const int kb = c & 1;
        if (!mbar_wait_bounded(smem_u32(&bar_kv[kb]), (uint32_t)((c >> 1) & 1), abort_flag,
                               dev_err, DEV_ERR_WAIT_GEMM))
          return false;
        if (c == nc - 1 && !mbar_wait_bounded(smem_u32(&bar_tail), 0u, abort_flag, dev_err,
                                              DEV_ERR_WAIT_GEMM))
          return false;
        if (c >= 2 && !mbar_wait_bounded(smem_u32(&bar_tfree[kb]), (uint32_t)(((c - 2) >> 1) & 1),
                                         abort_flag, dev_err, DEV_ERR_WAIT_GEMM))
          return false;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t qa = (uint32_t)((kk >> 2) * kAQ * 128 + (kk & 3) * 32);
          const uint32_t ka = (uint32_t)((kk >> 2) * kBC * 128 + (kk & 3) * 32);
          tc_mma_bf16(tmem + kColS + (uint32_t)kb * kBC, umma_desc_k_sw128(smem_u32(Qs) + qa),
                      umma_desc_k_sw128(smem_u32(Kb + kb * SM::kKc) + ka), id_s, kk > 0 ? 1u : 0u);
          tc_mma_bf16(tmem + kColP + (uint32_t)kb * kBC, umma_desc_k_sw128(smem_u32(dOs) + qa),
                      umma_desc_k_sw128(smem_u32(Vb + kb * SM::kKc) + ka), id_dp, kk > 0 ? 1u : 0u);
        }
        tc_commit(smem_u32(&bar_sdp[kb]));
        return true;
      };
      ok = ok && issue_sdp(0);
      for (int c = 0; c < nc && ok; ++c) {
        const int kb = c & 1;
        if (c + 1 < nc) ok = issue_sdp(c + 1);
        if (!ok) break;
        ok = mbar_wait_bounded(smem_u32(&bar_ds), (uint32_t)(c & 1), abort_flag, dev_err,
                               DEV_ERR_WAIT_GEMM);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < kBC / 16; ++kk)
          tc_mma_bf16(tmem + kColQ, umma_desc_k_sw128(smem_u32(dSs) + (uint32_t)(kk * 32)),
                      umma_desc_mn_sw128(smem_u32(Kb + kb * SM::kKc) + (uint32_t)kk * 16 * 128,
                                         kBC * 128, 1024u),
                      id_acc, (c > 0 || kk > 0) ? 1u : 0u);
        tc_commit(smem_u32(&bar_dsfree));     // dS read; dQ updated
        tc_commit(smem_u32(&bar_kvfree[kb]));  // the K and V chunk read
      }
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- gradient warps
    const int r = (warp & 3) * 32 + lane;  // query row of the block = TMEM lane
    const int hf = warp >> 2;              // keys 32 hf .. of each chunk
    const int q = q0 + r;
    const int kmax = min(max(q, tile.prompt - 1), tile.end - 1);  // its last key
    const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const int64_t qq = (int64_t)h * T + min(q, tile.end - 1);
    const float l2 = __ldg(lse + qq) * 1.4426950408889634f;
    const float dl = __ldg(delta + qq);
    const float unscale = scale * exp2f(-__ldg(rowexp + qq));
    bool ok = true;
    for (int c = 0; c < nc && ok; ++c) {
      const int kb = c & 1;
      ok = mbar_wait_bounded(smem_u32(&bar_sdp[kb]), (uint32_t)((c >> 1) & 1), abort_flag, dev_err,
                             DEV_ERR_WAIT_GEMM);
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok) break;
      tc_fence_after();
      uint32_t sv[2][16], pv[2][16];
      tmem_ld16(trow + kColS + (uint32_t)(kb * kBC + 32 * hf), sv[0]);
      tmem_ld16(trow + kColS + (uint32_t)(kb * kBC + 32 * hf + 16), sv[1]);
      tmem_ld16(trow + kColP + (uint32_t)(kb * kBC + 32 * hf), pv[0]);
      tmem_ld16(trow + kColP + (uint32_t)(kb * kBC + 32 * hf + 16), pv[1]);
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bar_tfree[kb]));
      const int kfirst = tile.begin + c * kBC + 32 * hf;  // this thread's first key
      uint32_t dpk[16];
#pragma unroll
      for (int e = 0; e < 32; e += 2) {
        float d[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int key = kfirst + e + u;
          const bool live = key <= kmax;
          const float s = __uint_as_float(sv[(e + u) >> 4][(e + u) & 15]);
          const float dp = __uint_as_float(pv[(e + u) >> 4][(e + u) & 15]);
          const float p = live ? ex2(fmaf(s, sl2, -l2)) : 0.f;
          d[u] = live ? p * (dp - dl) : 0.f;
        }
        dpk[e >> 1] = pack_f16x2(d[0], d[1]);
      }
      // the previous chunk's dQ product has read dS
      if (c > 0) {
        ok = mbar_wait_bounded(smem_u32(&bar_dsfree), (uint32_t)((c - 1) & 1), abort_flag, dev_err,
                               DEV_ERR_WAIT_GEMM);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
      }
#pragma unroll
      for (int cc = 0; cc < 4; ++cc)
        *reinterpret_cast<uint4*>(dSs + sw128_offset((uint32_t)r, (uint32_t)(hf * 4 + cc))) =
            make_uint4(dpk[4 * cc], dpk[4 * cc + 1], dpk[4 * cc + 2], dpk[4 * cc + 3]);
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bar_ds));
    }
    if (ok) ok = mbar_wait_bounded(smem_u32(&bar_dsfree), (uint32_t)((nc - 1) & 1), abort_flag,
                                   dev_err, DEV_ERR_WAIT_GEMM);
    ok = __all_sync(0xFFFFFFFFu, ok);
    if (ok) {
      tc_fence_after();
      const bool live = q < tile.end;
      const int64_t o = (int64_t)q * (int64_t)H * D + (int64_t)h * D + hf * (D / 2);
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t v[16];
        tmem_ld16(trow + kColQ + (uint32_t)(hf * (D / 2) + 16 * c), v);
        tmem_ld_wait();
        if (live) {
#pragma unroll
          for (int e = 0; e < 16; e += 4)
            *reinterpret_cast<float4*>(dq + o + 16 * c + e) =
                make_float4(__uint_as_float(v[e]) * unscale, __uint_as_float(v[e + 1]) * unscale,
                            __uint_as_float(v[e + 2]) * unscale, __uint_as_float(v[e + 3]) * unscale);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (abort_sh) settle_ns(2000000);
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// dqkv (bf16) from dq and the query heads' dk and dv (fp32 [T, H d] each): k and v
// summed over their kv head's query heads in order, with cs the rotation of q and k
// by their position in the document undone, padding rows 0.  A thread takes 4 pairs
// (i, i + d/2).
__global__ void __launch_bounds__(256)
    packed_grad_kernel(const float* __restrict__ dq, const float* __restrict__ dk,
                       const float* __restrict__ dv, const int* __restrict__ head,
                       const int* __restrict__ pos, int64_t T, int H, int Hkv, int d,
                       const float2* __restrict__ cs, uint16_t* __restrict__ dqkv) {
  pdl_trigger();
  pdl_wait();
  const int half = d / 2, chunks = half / 4, rep = H / Hkv;
  const int64_t ld = (int64_t)(H + 2 * Hkv) * d, hd = (int64_t)H * d;
  const int64_t n = T * (H + 2 * Hkv) * chunks;
  const int64_t live = head[2];
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n;
       i += (int64_t)gridDim.x * blockDim.x) {
    const int ch = (int)(i % chunks);
    const int64_t th = i / chunks;
    const int hh = (int)(th % (H + 2 * Hkv));
    const int64_t t = th / (H + 2 * Hkv);
    uint16_t* out = dqkv + t * ld + (int64_t)hh * d + ch * 4;
    float a[4] = {0.f, 0.f, 0.f, 0.f}, b[4] = {0.f, 0.f, 0.f, 0.f};
    if (t < live) {
      const float* src = hh < H ? dq : hh < H + Hkv ? dk : dv;
      const int h0 = hh < H ? hh : ((hh - H) % Hkv) * rep;
      const int nh = hh < H ? 1 : rep;
      for (int k = 0; k < nh; ++k) {
        const float* s = src + t * hd + (int64_t)(h0 + k) * d + ch * 4;
        const float4 x = *reinterpret_cast<const float4*>(s);
        const float4 y = *reinterpret_cast<const float4*>(s + half);
        a[0] += x.x; a[1] += x.y; a[2] += x.z; a[3] += x.w;
        b[0] += y.x; b[1] += y.y; b[2] += y.z; b[3] += y.w;
      }
      if (cs && hh < H + Hkv) {
        const float2* c = cs + (int64_t)pos[t] * half + ch * 4;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 f = c[k];
          const float x = a[k], y = b[k];
          a[k] = x * f.x + y * f.y;
          b[k] = y * f.x - x * f.y;
        }
      }
    }
    *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]));
    *reinterpret_cast<uint2*>(out + half) =
        make_uint2(pack_bf16x2(b[0], b[1]), pack_bf16x2(b[2], b[3]));
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
  CUtensorMap tm;
  LSQ_TRY(make_tmap_2d(&tm, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, qkv, (uint64_t)row, (uint64_t)T,
                       (uint64_t)row, 64, kAQ, CU_TENSOR_MAP_SWIZZLE_128B));
  int* err = device_status_ptr();
  if (!err) return set_error(LSQ_ERR_CUDA, "device status word unavailable");
  const float sl2 = 1.4426950408889634f / sqrtf((float)D);
  const int64_t items = (H / Hkv) % 2 == 0 ? (int64_t)x.cap * (H / 2) : (int64_t)x.cap2 * H;
  const unsigned grid = (unsigned)std::min<int64_t>(items, gemm_num_sms());
  LSQ_CUDA(launch_dep(packed_attn_fwd_kernel<D>, dim3(grid), kFThreads, SM::kBytes, st, tm, x, T, H,
                      Hkv, o, lse, sl2, err));
  return LSQ_OK;
}

struct BwdWs {
  uint16_t* dos;   // [T, H d] fp16 dO'
  float* delta;    // [H, T] delta'
  float* rowexp;   // [H, T] e
  float *dq, *dk, *dv;  // [T, H d] fp32
};
size_t carve_bwd(int64_t T, int H, int d, void* base, BwdWs* w) {
  Arena a;
  a.base = static_cast<uint8_t*>(base);
  a.cap = SIZE_MAX;
  BwdWs x;
  const size_t n = (size_t)T * H * d;
  x.dos = a.take<uint16_t>(n);
  x.delta = a.take<float>((size_t)T * H);
  x.rowexp = a.take<float>((size_t)T * H);
  x.dq = a.take<float>(n);
  x.dk = a.take<float>(n);
  x.dv = a.take<float>(n);
  if (w) *w = x;
  return a.used;
}

template <int D>
int bwd_t(const uint16_t* qkv, const PackedIndex& x, const uint16_t* o, const float* lse,
          const uint16_t* dout, int64_t T, int H, int Hkv, const float2* cs, uint16_t* dqkv,
          const BwdWs& w, cudaStream_t st) {
  static bool attr_kv[64] = {false}, attr_q[64] = {false};
  LSQ_TRY(allow_smem(packed_attn_dkdv_kernel<D>, (int)PaDkvSmem<D>::kBytes, attr_kv));
  LSQ_TRY(allow_smem(packed_attn_dq_kernel<D>, (int)PaDqSmem<D>::kBytes, attr_q));
  int* err = device_status_ptr();
  if (!err) return set_error(LSQ_ERR_CUDA, "device status word unavailable");
  const float scale = 1.f / sqrtf((float)D);
  const float sl2 = 1.4426950408889634f * scale;
  const int64_t warps = T * (H + Hkv);
  LSQ_CUDA(launch_dep(packed_attn_prep_kernel<D>, dim3((unsigned)((warps + 7) / 8)), 256, 0, st, qkv,
                      o, dout, x.head, T, H, Hkv, w.dos, w.delta, w.rowexp, err));
  const int64_t row = (int64_t)(H + 2 * Hkv) * D, hd = (int64_t)H * D;
  CUtensorMap qkv128, qkv64, do128, do64;
  LSQ_TRY(make_tmap_2d(&qkv128, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, qkv, (uint64_t)row, (uint64_t)T,
                       (uint64_t)row, 64, kAK, CU_TENSOR_MAP_SWIZZLE_128B));
  LSQ_TRY(make_tmap_2d(&qkv64, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, qkv, (uint64_t)row, (uint64_t)T,
                       (uint64_t)row, 64, kBC, CU_TENSOR_MAP_SWIZZLE_128B));
  LSQ_TRY(make_tmap_2d(&do128, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, w.dos, (uint64_t)hd, (uint64_t)T,
                       (uint64_t)hd, 64, kAQ, CU_TENSOR_MAP_SWIZZLE_128B));
  LSQ_TRY(make_tmap_2d(&do64, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, w.dos, (uint64_t)hd, (uint64_t)T,
                       (uint64_t)hd, 64, kBC, CU_TENSOR_MAP_SWIZZLE_128B));
  const dim3 grid((unsigned)x.cap, (unsigned)H);
  LSQ_CUDA(launch_dep(packed_attn_dkdv_kernel<D>, grid, kBThreads, PaDkvSmem<D>::kBytes, st, qkv128,
                      qkv64, do64, x, lse, w.delta, w.rowexp, T, H, Hkv, sl2, scale, w.dk, w.dv,
                      err));
  LSQ_CUDA(launch_dep(packed_attn_dq_kernel<D>, grid, kBThreads, PaDqSmem<D>::kBytes, st, qkv128,
                      qkv64, do128, x, lse, w.delta, w.rowexp, T, H, Hkv, sl2, scale, w.dq, err));
  const int64_t items = T * (H + 2 * Hkv) * (D / 8);
  LSQ_CUDA(launch_dep(packed_grad_kernel,
                      dim3((unsigned)std::min<int64_t>((items + 255) / 256, gemm_num_sms() * 16)),
                      256, 0, st, w.dq, w.dk, w.dv, x.head, x.pos, T, H, Hkv, D, cs, dqkv));
  return LSQ_OK;
}

int check_heads(int64_t T, int32_t H, int32_t Hkv, int32_t d, const char* who) {
  if (H <= 0 || Hkv <= 0 || H % Hkv != 0 || H > 65535)
    return set_error(LSQ_ERR_SHAPE, "%s: H must be a multiple of Hkv, at most 65535", who);
  if (d != 64 && d != 128) return set_error(LSQ_ERR_SHAPE, "%s: d must be 64 or 128", who);
  if (T * (H + 2 * (int64_t)Hkv) > (int64_t(1) << 33))
    return set_error(LSQ_ERR_SHAPE, "%s: too many tokens and heads", who);
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
  return carve_bwd(T, H, d, nullptr, nullptr);
}

int launch_packed_attention_bwd(const uint16_t* qkv, const int32_t* index, int n_docs,
                                const uint16_t* o, const float* lse, const uint16_t* dout,
                                int64_t T, int H, int Hkv, int d, const float2* cs, uint16_t* dqkv,
                                void* ws, size_t ws_bytes, cudaStream_t st) {
  const PackedIndex x = packed_index_view(index, T, n_docs);
  BwdWs w;
  if (carve_bwd(T, H, d, ws, &w) > ws_bytes)
    return set_error(LSQ_ERR_WORKSPACE, "packed attention: workspace too small");
  const int prof = prof_begin(st);
  LSQ_TRY(d == 128 ? bwd_t<128>(qkv, x, o, lse, dout, T, H, Hkv, cs, dqkv, w, st)
                   : bwd_t<64>(qkv, x, o, lse, dout, T, H, Hkv, cs, dqkv, w, st));
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
  if (!aligned16(qkv) || !aligned16(o) || !aligned16(lse))
    return set_error(LSQ_ERR_ALIGN, "packed_attention_fwd: pointers must be 16-byte aligned");
  return launch_packed_attention_fwd(qkv, index, n_docs, T, H, Hkv, d, o, lse,
                                     static_cast<cudaStream_t>(stream));
}

extern "C" size_t packed_attention_workspace_bytes(int64_t T, int32_t H, int32_t Hkv, int32_t d) {
  if (T <= 0 || T > (int64_t(1) << 30) || H <= 0 || Hkv <= 0 || H % Hkv != 0 ||
      (d != 64 && d != 128))
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
  if (!aligned16(qkv) || !aligned16(o) || !aligned16(lse) || !aligned16(dout) || !aligned16(dqkv))
    return set_error(LSQ_ERR_ALIGN, "packed_attention_bwd: pointers must be 16-byte aligned");
  const size_t need = packed_attention_ws_bytes(T, H, Hkv, d);
  if (!ws || ws_bytes < need)
    return set_error(LSQ_ERR_WORKSPACE, "packed_attention_bwd: workspace %zu < %zu", ws_bytes, need);
  if (!aligned16(ws)) return set_error(LSQ_ERR_ALIGN, "packed_attention_bwd: unaligned workspace");
  return launch_packed_attention_bwd(qkv, index, n_docs, o, lse, dout, T, H, Hkv, d, nullptr, dqkv,
                                     ws, ws_bytes, static_cast<cudaStream_t>(stream));
}
