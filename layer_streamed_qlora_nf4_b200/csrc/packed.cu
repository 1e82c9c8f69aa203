// Operators of a packed fine-tuning step that are not attention: the index of the
// documents in a row of tokens, the targets of the tokens that are trained on, and
// the cross-entropy over the vocabulary with its gradient.
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "packed.cuh"

namespace lsq {

namespace {

constexpr int kIdxThreads = 1024;

// Inclusive sums over a warp, and over the CTA's 1024 threads (in thread order; sh holds
// 32 values).
__device__ __forceinline__ int64_t warp_scan(int64_t v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  v = warp_scan(v);
  __syncthreads();  // sh is free
  if (lane == 31) sh[warp] = v;
  __syncthreads();
  if (warp == 0) sh[lane] = warp_scan(sh[lane]);
  __syncthreads();
  return v + (warp > 0 ? sh[warp - 1] : 0);
}

// Index of the last entry of a[0, n) that is <= x (a ascending, a[0] <= x).
__device__ __forceinline__ int find_last(const int* a, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a[mid] <= x)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// How many tiles of a document of nt tiles, pt of which hold some of its prompt, have
// more work than w.  Query tiles of 128: tile i sees max(i + 1, pt) key tiles; of 256:
// taken as max(2 i + 2, pt); key tiles: tile i is seen by nt - i query tiles, by all nt
// where it holds some of the prompt.
enum ListKind { LIST_Q = 0, LIST_Q2 = 1, LIST_K = 2 };
__device__ __forceinline__ int work_of(int kind, int i, int nt, int pt) {
  return kind == LIST_Q ? max(i + 1, pt) : kind == LIST_Q2 ? max(2 * i + 2, pt) : i < pt ? nt : nt - i;
}
__device__ __forceinline__ int count_above(int kind, int nt, int pt, int w) {
  if (kind == LIST_K) return nt <= w ? 0 : pt + max(0, nt - w - pt);
  if (pt > w) return nt;
  return max(0, nt - (kind == LIST_Q ? w : w / 2));
}
// Tiles before tile i of the same document with the same work.
__device__ __forceinline__ int ties_before(int kind, int i, int pt) {
  const bool flat = kind == LIST_Q ? i + 1 <= pt : kind == LIST_Q2 ? 2 * i + 2 <= pt : i < pt;
  return flat ? i : 0;
}

// Every CTA scans all lengths, 1024 documents at a time (up to 32 of them in one warp,
// without the barriers of a scan over the block), and writes its own share of the tokens and
// tiles, each found by a binary search over the 1024 starts in shared memory: a
// single long document costs no more than many short ones.  Latency throughout: 2.4 us for
// 512 tokens in 5 documents, 4.1 for 16,384 in 40, 14 for 1024 in 1000.
__global__ void __launch_bounds__(kIdxThreads, 1)
    packed_index_kernel(const int32_t* lengths, const int32_t* prefix,
                        int n_docs, int T, PackedIndex x, int* dev_err) {
  __shared__ int64_t sh[32];
  __shared__ int64_t sums[2];
  __shared__ int tok0[kIdxThreads], t1[kIdxThreads], t2[kIdxThreads], doc_e[kIdxThreads],
      doc_p[kIdxThreads];
  const bool sorted = n_docs <= kIdxThreads, few = n_docs <= 32;
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x;
  const int gtid = blockIdx.x * kIdxThreads + tid, gsize = gridDim.x * kIdxThreads;
  int64_t base = 0;          // tokens, tiles of 128 and tiles of 256 before this chunk
  int base1 = 0, base2 = 0;
  bool bad = false;
  for (int d0 = 0; d0 < n_docs; d0 += kIdxThreads) {
    if (!few || tid < 32) {
      auto scan = [&](int64_t v, int64_t* total) {
        if (few) {
          v = warp_scan(v);
          *total = __shfl_sync(0xFFFFFFFFu, v, 31);
        } else {
          v = block_scan(v, sh);
          *total = sh[31];
        }
        return v;
      };
      const int d = d0 + tid;
      int len = d < n_docs ? lengths[d] : 0;
      int pre = d < n_docs && prefix ? prefix[d] : 0;
      if (len < 0 || pre < 0 || pre > len) bad = true;  // such a length counts as 0
      len = max(len, 0);
      int64_t all, all12;
      const int64_t end = base + scan(len, &all);
      if (end > T) bad = true;  // documents are cut where the row ends
      const int s = (int)min((int64_t)T, end - len), e = (int)min((int64_t)T, end);
      pre = min(max(pre, 0), e - s);
      const int n1 = (e - s + kPackedTile - 1) / kPackedTile;
      const int n2 = (e - s + 2 * kPackedTile - 1) / (2 * kPackedTile);
      const int64_t i12 = scan(((int64_t)n1 << 32) | (int64_t)n2, &all12);
      tok0[tid] = s;
      doc_e[tid] = e;
      doc_p[tid] = s + pre;
      t1[tid] = base1 + (int)(i12 >> 32) - n1;
      t2[tid] = base2 + (int)(i12 & 0xFFFFFFFF) - n2;
      if (tid == 0) {
        sums[0] = all;
        sums[1] = all12;
      }
    }
    __syncthreads();
    const int64_t total = base + sums[0], all12 = sums[1];
    const int nd = min(n_docs - d0, kIdxThreads);
    // documents of no tokens share their start with the next one: the last at or
    // before a token is the one that holds it
    const int c1 = (int)(all12 >> 32), c2 = (int)(all12 & 0xFFFFFFFF);
    const int hi = (int)min((int64_t)T, total);
    for (int t = (int)base + gtid; t < hi; t += gsize) {
      const int k = find_last(tok0, nd, t);
      x.pos[t] = t - tok0[k];
      x.key_end[t] = max(t + 1, doc_p[k]);
      x.doc_end[t] = doc_e[k];
    }
    // a tile's place: by its work, or (with more documents than one chunk) in order
    auto emit = [&](int kind, int i, const int* first, int before, int size, PackedTile* list,
                    int cap) {
      const int k = find_last(first, nd, before + i);
      const int at = before + i - first[k];  // tile of its document
      int place = before + i;
      if (sorted) {
        const int lane = tid & 31;
        auto tiles_of = [&](int len) { return (len + size - 1) / size; };
        const int pt = (doc_p[k] - tok0[k] + kPackedTile - 1) / kPackedTile;
        const int w = work_of(kind, at, tiles_of(doc_e[k] - tok0[k]), pt);
        place = 0;
        for (int d = lane; d < n_docs; d += 32) {
          const int nt = tiles_of(doc_e[d] - tok0[d]);
          const int dpt = (doc_p[d] - tok0[d] + kPackedTile - 1) / kPackedTile;
          const int above = count_above(kind, nt, dpt, w);
          place += d < k ? count_above(kind, nt, dpt, w - 1) : above;
        }
        place = __reduce_add_sync(0xFFFFFFFFu, place) + ties_before(kind, at, pt);
      }
      if ((tid & 31) == 0 && place < cap)
        list[place] = {tok0[k] + at * size, tok0[k], doc_e[k], doc_p[k]};
    };
    for (int i = gtid >> 5; i < 2 * c1 + c2; i += gsize >> 5) {  // (a warp takes a tile)
      if (i < c1)
        emit(LIST_Q, i, t1, base1, kPackedTile, x.tiles, x.cap);
      else if (i < 2 * c1)
        emit(LIST_K, i - c1, t1, base1, kPackedTile, x.ktiles, x.cap);
      else
        emit(LIST_Q2, i - 2 * c1, t2, base2, 2 * kPackedTile, x.tiles2, x.cap2);
    }
    base = hi;
    base1 += c1;
    base2 += c2;
    if (total > T) bad = true;
    __syncthreads();
  }
  // padding belongs to no document
  for (int t = (int)base + gtid; t < T; t += gsize) {
    x.pos[t] = 0;
    x.key_end[t] = (int)base;
    x.doc_end[t] = (int)base;
  }
  if (gtid == 0) {
    x.head[0] = min(base1, x.cap);
    x.head[1] = min(base2, x.cap2);
    x.head[2] = (int)base;
    for (int i = 3; i < 8; ++i) x.head[i] = 0;
  }
  if (bad) atomicOr(dev_err, DEV_ERR_INDEX);
}

// Target of token t: the next token, where that belongs to the same document, is not
// seen by t itself (a prompt read in both directions is not predicted), and is marked
// in loss_mask (if given); -1 elsewhere, and where the next token is below 0.  count: the integer sum over CTAs, the same
// in any order.  Memory bound (17 bytes a token), in practice the latency of a launch.
__global__ void __launch_bounds__(256)
    packed_targets_kernel(const int32_t* tokens, const int* key_end,
                          const int* doc_end, const uint8_t* loss_mask,
                          int T, int32_t* targets, int32_t* count) {
  pdl_trigger();
  pdl_wait();
  int n = 0;
  for (int t = blockIdx.x * 256 + threadIdx.x; t < T; t += gridDim.x * 256) {
    const bool on = t + 1 < doc_end[t] && key_end[t] == t + 1 && (!loss_mask || loss_mask[t + 1]);
    const int y = on ? max(tokens[t + 1], -1) : -1;  // (the loss takes none below 0 either)
    targets[t] = y;
    n += y >= 0;
  }
  n = __reduce_add_sync(0xFFFFFFFFu, n);
  if ((threadIdx.x & 31) == 0 && n) atomicAdd(count, n);
}

// ------------------------------------------------------------------ cross-entropy
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x) {  // 2^x, relative error 2^-22
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// (max, sum of exp relative to it) of two sets; (-inf, 0) is the empty set.  The maximum
// passes over NaN, the sum does not: of a set with a NaN it is NaN, whatever the maximum.
__device__ __forceinline__ void join(float& m, float& s, float mo, float so) {
  const float mn = fmaxf(m, mo);
  const float at = mn == -INFINITY ? 0.f : mn;  // (without a branch: with one 84 -> 88 us below)
  s = s * ex2((m - at) * kLog2e) + so * ex2((mo - at) * kLog2e);
  m = mn;
}

constexpr int kCeThreads = 256;
constexpr int kCeChunks = 2;  // bulk copies of a slice

// The pairs of a warp's lanes joined, the same in every lane.
__device__ __forceinline__ void warp_join(float& m, float& s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float mo = __shfl_xor_sync(0xFFFFFFFFu, m, o);
    const float so = __shfl_xor_sync(0xFFFFFFFFu, s, o);
    join(m, s, mo, so);
  }
}

// A cluster of C CTAs per row, each with a slice of the row in shared memory, so that
// the logits are read once: bulk copies bring the slice in, the online maximum and sum
// of exponentials follow them, the CTAs exchange their pairs through the cluster's shared
// memory, and the gradient is formed from the slice.  Memory bound: 4 bytes read and 2
// written per logit (512 rows of 128,256: 56 us at the measured copy rate).  Measured
// there: 98 us for one CTA per row that reads it twice (the rows in flight exceed the L2),
// 84 us for this form, 86 us for persistent clusters that refill a chunk with the next
// row's as soon as they are done with it, 100 us and more with shares re-read through L2;
// 2048 rows of 151,936 (40% with a target): 216 us.
// Elements are taken eight at a time from the first whose index in the whole array is a
// multiple of eight, so that any V moves in aligned 16-byte pieces; the few before and
// behind are rank 0's and the last rank's.
__global__ void __launch_bounds__(kCeThreads)
    packed_ce_kernel(const float* logits, const int32_t* targets,
                     int64_t V, const float* weight, const int32_t* count, float ranks,
                     uint16_t* dlogits, float* row_loss, int C,
                     int* dev_err) {
  extern __shared__ __align__(128) float slice[];
  __shared__ __align__(8) uint64_t bar[kCeChunks];
  __shared__ float red_m[kCeThreads / 32], red_s[kCeThreads / 32];
  __shared__ __align__(16) float pair[4];
  __shared__ int abort_sh;
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31;
  const int64_t row = blockIdx.x / C;
  const int rank = blockIdx.x % C;
  const int head = (int)min(V, (int64_t)((8 - (int)((row * V) & 7)) & 7));
  const int64_t n8 = (V - head) / 8;             // groups of eight
  const int64_t per = (n8 + C - 1) / C;
  const int64_t g0 = min(n8, per * rank);
  const int ng = (int)(min(n8, g0 + per) - g0);  // groups of this slice
  const int64_t first = head + g0 * 8;           // its first element
  const int64_t tail = head + n8 * 8;
  // the ragged ends: element `odd` of the row, one per thread
  const int64_t odd = rank == 0 && tid < head ? tid
                      : rank == C - 1 && tid >= 32 && tail + tid - 32 < V && tid < 40 ? tail + tid - 32
                                                                                     : -1;
  const float* x = logits + row * V;
  uint16_t* dx = dlogits ? dlogits + row * V : nullptr;
  if (tid == 0) {
    for (int i = 0; i < kCeChunks; ++i) mbar_init(smem_u32(&bar[i]), 1);
    abort_sh = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  __syncthreads();
  pdl_wait();
  const int64_t y = targets[row];
  if (y < 0 || y >= V) {  // (the same in the whole cluster)
    if (dx) {
      for (int i = tid; i < ng; i += kCeThreads)
        reinterpret_cast<uint4*>(dx + first)[i] = make_uint4(0u, 0u, 0u, 0u);
      if (odd >= 0) dx[odd] = 0;
    }
    if (tid == 0 && rank == 0) {
      row_loss[row] = 0.f;
      if (y >= V) atomicOr(dev_err, DEV_ERR_INDEX);
    }
    return;
  }
  const int cg = (ng + kCeChunks - 1) / kCeChunks;  // groups of a chunk
  if (tid == 0)
    for (int i = 0; i < kCeChunks; ++i) {
      const int a = min(ng, i * cg), n = min(ng, a + cg) - a;
      if (n == 0) continue;
      mbar_arrive_expect_tx(smem_u32(&bar[i]), (uint32_t)n * 32u);
      asm volatile(
          "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
              "r"(smem_u32(slice + a * 8)),
          "l"(x + first + (int64_t)a * 8), "r"((uint32_t)n * 32u), "r"(smem_u32(&bar[i]))
          : "memory");
    }
  float m = -INFINITY, s = 0.f;
  const float xo = odd >= 0 ? x[odd] : -INFINITY;
  if (xo > -INFINITY) {
    m = xo;
    s = 1.f;
  } else if (isnan(xo)) {
    s = xo;
  }
  const float4* s4 = reinterpret_cast<const float4*>(slice);
  for (int i = 0; i < kCeChunks; ++i) {
    const int a = min(ng, i * cg) * 2, e = min(ng, (i + 1) * cg) * 2;  // in float4
    if (a == e) break;
    // (one warp polls: all of them would keep the shared-memory pipe from the others)
    if (tid < 32) mbar_wait_short(smem_u32(&bar[i]), 0u, &abort_sh, dev_err);
    __syncthreads();
    for (int k = a + tid; k < e; k += 4 * kCeThreads) {
      float4 v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        v[j] = k + j * kCeThreads < e ? s4[k + j * kCeThreads]
                                      : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      float t = m;
#pragma unroll
      for (int j = 0; j < 4; ++j) t = fmaxf(t, fmaxf(fmaxf(v[j].x, v[j].y), fmaxf(v[j].z, v[j].w)));
      const float c = t == -INFINITY ? 0.f : -t * kLog2e;
      s *= m == -INFINITY ? 0.f : ex2(fmaf(m, kLog2e, c));
      m = t;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        s += (ex2(fmaf(v[j].x, kLog2e, c)) + ex2(fmaf(v[j].y, kLog2e, c))) +
             (ex2(fmaf(v[j].z, kLog2e, c)) + ex2(fmaf(v[j].w, kLog2e, c)));
    }
  }
  warp_join(m, s);
  if (lane == 0) {
    red_m[tid >> 5] = m;
    red_s[tid >> 5] = s;
  }
  __syncthreads();
  // one warp joins the warps' pairs (by all threads, one after the other, this took as
  // long as the row itself)
  if (tid < 32) {
    m = lane < kCeThreads / 32 ? red_m[lane] : -INFINITY;
    s = lane < kCeThreads / 32 ? red_s[lane] : 0.f;
    warp_join(m, s);
    if (lane == 0) {
      pair[0] = m;
      pair[1] = s;
    }
  }
  if (C > 1) {
    // (only warp 0's pair is to be seen by the others: it alone releases)
    if (tid < 32)
      asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    else
      asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    m = -INFINITY;
    s = 0.f;
    if (lane < C) {
      const float4 v = ld_shared_cluster_f4(mapa_shared(smem_u32(pair), (uint32_t)lane));
      m = v.x;
      s = v.y;
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) {
      const float mo = __shfl_xor_sync(0xFFFFFFFFu, m, o);
      const float so = __shfl_xor_sync(0xFFFFFFFFu, s, o);
      join(m, s, mo, so);
    }
    m = __shfl_sync(0xFFFFFFFFu, m, 0);
    s = __shfl_sync(0xFFFFFFFFu, s, 0);
    // done reading (the operands: not before the pairs have arrived)
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" : "+f"(m), "+f"(s)::"memory");
  } else {
    __syncthreads();
    m = pair[0];
    s = pair[1];
  }
  float c = weight ? weight[row] : 1.f;
  if (count) c = c * ranks / (float)max(1, *count);
  const float k = c / s, off = -m * kLog2e;
  auto grad = [&](float v, int64_t j) { return k * ex2(fmaf(v, kLog2e, off)) - (j == y ? c : 0.f); };
  if (dx) {
    const int yt = (int)min(max(y - first, (int64_t)-1), (int64_t)INT32_MAX);
    for (int i = tid; i < ng; i += kCeThreads) {
      const float4 a = s4[2 * i], b = s4[2 * i + 1];
      float g[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) g[e] = k * ex2(fmaf(g[e], kLog2e, off));
      if (yt >> 3 == i) {
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] -= (yt & 7) == e ? c : 0.f;
      }
      __stcs(reinterpret_cast<uint4*>(dx + first) + i,
             make_uint4(pack_bf16x2(g[0], g[1]), pack_bf16x2(g[2], g[3]), pack_bf16x2(g[4], g[5]),
                        pack_bf16x2(g[6], g[7])));
    }
    if (odd >= 0) dx[odd] = float_to_bf16_bits(grad(xo, odd));
  }
  if (tid == 0 && rank == 0) row_loss[row] = m + logf(s) - x[y];
  if (C > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The same for rows too long for a cluster's shared memory (above 450,000 logits): one CTA
// per row, which reads it twice.  256 rows of 500,001: 256 us, 3.0 TB/s of the bytes that
// the other form would move.
__global__ void __launch_bounds__(1024, 1)
    packed_ce_long_kernel(const float* logits, const int32_t* targets,
                          int64_t V, const float* weight,
                          const int32_t* count, float ranks, uint16_t* dlogits,
                          float* row_loss, int* dev_err) {
  __shared__ float red_m[32], red_s[32];
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x, y = targets[row];
  const float* x = logits + row * V;
  uint16_t* dx = dlogits ? dlogits + row * V : nullptr;
  const bool on = y >= 0 && y < V;
  float m = -INFINITY, s = 0.f;
  if (on)
    for (int64_t i = tid; i < V; i += 1024) {
      const float v = x[i];
      if (v > m) {
        s *= m == -INFINITY ? 0.f : ex2((m - v) * kLog2e);
        m = v;
      }
      s += m == -INFINITY && v == m ? 0.f : ex2((v - m) * kLog2e);
    }
  warp_join(m, s);
  if ((tid & 31) == 0) {
    red_m[tid >> 5] = m;
    red_s[tid >> 5] = s;
  }
  __syncthreads();
  m = red_m[tid & 31];
  s = red_s[tid & 31];
  warp_join(m, s);
  float c = on ? (weight ? weight[row] : 1.f) : 0.f;
  if (count) c = c * ranks / (float)max(1, *count);
  if (dx)
    for (int64_t i = tid; i < V; i += 1024)
      dx[i] = on ? float_to_bf16_bits(c / s * ex2((x[i] - m) * kLog2e) - (i == y ? c : 0.f))
                 : (uint16_t)0;
  if (tid == 0) {
    row_loss[row] = on ? m + logf(s) - x[y] : 0.f;
    if (y >= V) atomicOr(dev_err, DEV_ERR_INDEX);
  }
}

// loss (+)= sum over rows with a target of c_t row_loss[t], in a fixed order.
__global__ void __launch_bounds__(1024, 1)
    packed_loss_kernel(const float* row_loss, const int32_t* targets,
                       int64_t T, int64_t V, const float* weight,
                       const int32_t* count, float ranks, int accumulate, float* loss) {
  __shared__ float red[32];
  pdl_trigger();
  pdl_wait();
  float s = 0.f;
  for (int64_t t = threadIdx.x; t < T; t += 1024)
    if (targets[t] >= 0 && targets[t] < V) s += (weight ? weight[t] : 1.f) * row_loss[t];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x < 32) {
    s = red[threadIdx.x];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    if (threadIdx.x == 0) {
      if (count) s = s * ranks / (float)max(1, *count);
      *loss = (accumulate ? *loss : 0.f) + s;
    }
  }
}

constexpr int64_t kCeMaxSmem = 220 * 1024;

// CTAs of a row and bytes of shared memory of each: slices of at most 16,384 logits (64
// KB, three CTAs per SM, so that the copies of one overlap the arithmetic of another),
// as far as a portable cluster of eight goes; more CTAs for few rows.
int64_t ce_plan(int64_t T, int64_t V, int* C) {
  int c = 1;
  while (c < 8 && (V > 16384 * (int64_t)c || (V > 2048 * (int64_t)c && T * c < gemm_num_sms())))
    c *= 2;
  *C = c;
  return ((V / 8 + c - 1) / c) * 32 + 32;
}

template <class... P, class... A>
cudaError_t launch_dep(void (*k)(P...), unsigned grid, unsigned threads, cudaStream_t st, A... a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return ::lsq::launched(cudaLaunchKernelEx(&cfg, k, P(a)...));
}

}  // namespace

int launch_packed_index(const int32_t* lengths, const int32_t* prefix, int n_docs, int64_t T,
                        int32_t* index, cudaStream_t st) {
  int* err = device_status_ptr();
  if (!err) return set_error(LSQ_ERR_CUDA, "device status word unavailable");
  // a thread per token and a warp per tile, as far as 64 CTAs go: a row of many short
  // documents has as many tiles, and each looks at all documents
  const PackedIndex x = packed_index_view(index, T, n_docs);
  const int64_t work = std::max<int64_t>(T, 32 * (2 * (int64_t)x.cap + x.cap2));
  const unsigned grid = (unsigned)std::min<int64_t>(64, (work + kIdxThreads - 1) / kIdxThreads);
  LSQ_CUDA(launch_dep(packed_index_kernel, grid, kIdxThreads, st, lengths, prefix, n_docs, (int)T,
                      x, err));
  return LSQ_OK;
}

int launch_packed_targets(const int32_t* tokens, const int32_t* index, int n_docs, int64_t T,
                          const uint8_t* loss_mask, int32_t* targets, int32_t* count,
                          int accumulate, cudaStream_t st) {
  const PackedIndex x = packed_index_view(index, T, n_docs);
  if (!accumulate) LSQ_CUDA(cudaMemsetAsync(count, 0, sizeof(int32_t), st));
  const unsigned grid = (unsigned)std::min<int64_t>(512, (T + 255) / 256);
  LSQ_CUDA(launch_dep(packed_targets_kernel, grid, 256, st, tokens, x.key_end, x.doc_end, loss_mask,
                      (int)T, targets, count));
  return LSQ_OK;
}

int launch_packed_ce(const float* logits, int64_t T, int64_t V, const int32_t* targets,
                     const float* weight, const int32_t* count, uint16_t* dlogits,
                     float* row_loss, cudaStream_t st, int ranks) {
  int* err = device_status_ptr();
  if (!err) return set_error(LSQ_ERR_CUDA, "device status word unavailable");
  const int prof = prof_begin(st);
  int C = 1;  // CTAs of a row
  const int64_t smem = ce_plan(T, V, &C);
  if (smem > kCeMaxSmem || T * C > INT32_MAX) {
    LSQ_CUDA(launch_dep(packed_ce_long_kernel, (unsigned)T, 1024, st, logits, targets, V, weight,
                        count, (float)ranks, dlogits, row_loss, err));
  } else {
    static bool attr[64] = {false};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 64 && !attr[dev]) {
      LSQ_CUDA(cudaFuncSetAttribute(packed_ce_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)kCeMaxSmem));
      attr[dev] = true;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(T * C));
    cfg.blockDim = dim3(kCeThreads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)C;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    LSQ_CUDA(::lsq::launched(cudaLaunchKernelEx(&cfg, packed_ce_kernel, logits, targets, V, weight,
                                                count, (float)ranks, dlogits, row_loss, C, err)));
  }
  if (prof >= 0) prof_end(prof, st, "packed_ce", 0.0, (dlogits ? 6.0 : 4.0) * T * V);
  return LSQ_OK;
}

int launch_packed_loss(const float* row_loss, const int32_t* targets, int64_t T, int64_t V,
                       const float* weight, const int32_t* count, int accumulate, float* loss,
                       cudaStream_t st, int ranks) {
  LSQ_CUDA(launch_dep(packed_loss_kernel, 1, 1024, st, row_loss, targets, T, V, weight, count,
                      (float)ranks, accumulate, loss));
  return LSQ_OK;
}

int check_packed(int64_t T, int64_t n_docs, const void* index, const char* who) {
  if (T <= 0 || T > (int64_t(1) << 30))
    return set_error(LSQ_ERR_SHAPE, "%s: T must be in [1, 2^30]", who);
  if (n_docs <= 0 || n_docs > (int64_t(1) << 24))
    return set_error(LSQ_ERR_SHAPE, "%s: n_docs must be in [1, 2^24]", who);
  if (!index) return set_error(LSQ_ERR_INVALID, "%s: null index", who);
  if (!aligned16(index)) return set_error(LSQ_ERR_ALIGN, "%s: the index must be 16-byte aligned", who);
  return LSQ_OK;
}

}  // namespace lsq

using namespace lsq;

extern "C" int64_t packed_index_ints(int64_t T, int32_t n_docs) {
  if (T <= 0 || n_docs <= 0) return 0;
  return packed_index_words(T, n_docs);
}

extern "C" int packed_index(const int32_t* lengths, const int32_t* prefix, int32_t n_docs,
                            int64_t T, int32_t* index, void* stream) {
  LSQ_TRY(check_packed(T, n_docs, index, "packed_index"));
  if (!lengths) return set_error(LSQ_ERR_INVALID, "packed_index: null lengths");
  return launch_packed_index(lengths, prefix, n_docs, T, index, static_cast<cudaStream_t>(stream));
}

extern "C" int packed_targets(const int32_t* tokens, const int32_t* index, int32_t n_docs,
                              int64_t T, const uint8_t* loss_mask, int32_t* targets,
                              int32_t* count, int32_t accumulate, void* stream) {
  LSQ_TRY(check_packed(T, n_docs, index, "packed_targets"));
  if (!tokens || !targets || !count)
    return set_error(LSQ_ERR_INVALID, "packed_targets: null pointer");
  if (accumulate != 0 && accumulate != 1)
    return set_error(LSQ_ERR_INVALID, "packed_targets: accumulate must be 0 or 1");
  return launch_packed_targets(tokens, index, n_docs, T, loss_mask, targets, count, accumulate,
                               static_cast<cudaStream_t>(stream));
}

extern "C" int packed_cross_entropy(const float* logits, int64_t T, int64_t V,
                                    const int32_t* targets, const float* weight,
                                    const int32_t* count, uint16_t* dlogits, float* row_loss,
                                    float* loss, int32_t accumulate, void* stream) {
  if (T <= 0 || T > INT32_MAX || V <= 0 || V > INT32_MAX)
    return set_error(LSQ_ERR_SHAPE, "packed_cross_entropy: T and V must be in [1, 2^31)");
  if (!logits || !targets || !row_loss || !loss)
    return set_error(LSQ_ERR_INVALID, "packed_cross_entropy: null pointer");
  if (accumulate != 0 && accumulate != 1)
    return set_error(LSQ_ERR_INVALID, "packed_cross_entropy: accumulate must be 0 or 1");
  if (!aligned16(logits) || (dlogits && !aligned16(dlogits)))
    return set_error(LSQ_ERR_ALIGN,
                     "packed_cross_entropy: logits and dlogits must be 16-byte aligned");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  LSQ_TRY(launch_packed_ce(logits, T, V, targets, weight, count, dlogits, row_loss, st));
  return launch_packed_loss(row_loss, targets, T, V, weight, count, accumulate, loss, st);
}
