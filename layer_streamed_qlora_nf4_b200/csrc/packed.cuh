// Packed documents: the layout of the index that packed_index builds and the packed
// operators read.
//
// A row of T tokens holds n_docs documents behind one another; document k has
// lengths[k] tokens (0 is allowed), and tokens behind the last one are padding.  Token
// i of a document [s, e) with a prompt of p tokens sees the keys [s, max(i + 1, s + p)),
// so key j is seen by the queries [j < s + p ? s : j, e).
#pragma once

#include <stdint.h>

namespace lsq {

// One tile of consecutive tokens of one document: rows [row0, min(row0 + size, end)).
struct PackedTile {
  int row0;    // first token
  int begin;   // the document's first token
  int end;     // behind its last
  int prompt;  // behind its prompt (begin when it has none)
};

constexpr int kPackedTile = 128;

// int32 words: a header of 8 (tiles of 128, tiles of 256, tokens in documents), the
// tile lists, then per token its position in its document, the end of the keys it sees
// and the end of its document.  The lists are in order of falling work (with more than
// 1024 documents: in token order), so that persistent CTAs that take items in turn end
// together: query tiles by the keys they see, key tiles by the queries that see them.
struct PackedIndex {
  int* head;
  PackedTile* tiles;    // query tiles of 128 tokens
  PackedTile* ktiles;   // the same tiles in the key tiles' order
  PackedTile* tiles2;   // query tiles of 256 tokens
  int* pos;
  int* key_end;
  int* doc_end;
  int cap, cap2;        // room in the lists
};

inline int64_t packed_tile_cap(int64_t T, int64_t n_docs, int size) {
  const int64_t c = T / size + n_docs;
  return c < T ? c : T;
}
inline int64_t packed_index_words(int64_t T, int64_t n_docs) {
  return 8 + 4 * (2 * packed_tile_cap(T, n_docs, kPackedTile) +
                  packed_tile_cap(T, n_docs, 2 * kPackedTile)) + 3 * T;
}
inline PackedIndex packed_index_view(const int32_t* base, int64_t T, int64_t n_docs) {
  PackedIndex x;
  x.head = const_cast<int32_t*>(base);
  x.cap = (int)packed_tile_cap(T, n_docs, kPackedTile);
  x.cap2 = (int)packed_tile_cap(T, n_docs, 2 * kPackedTile);
  x.tiles = reinterpret_cast<PackedTile*>(x.head + 8);
  x.ktiles = x.tiles + x.cap;
  x.tiles2 = x.ktiles + x.cap;
  x.pos = reinterpret_cast<int*>(x.tiles2 + x.cap2);
  x.key_end = x.pos + T;
  x.doc_end = x.key_end + T;
  return x;
}

// A bounded wait like mbar_wait_bounded, which reads the clock only after 64 polls have
// failed: the read takes longer than most waits here.
#ifdef __CUDACC__
__device__ __forceinline__ bool mbar_wait_short(uint32_t bar, uint32_t parity,
                                                volatile int* abort_flag, int* dev_err) {
  uint64_t t0 = 0;
  for (uint32_t n = 1;; ++n) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((n & 63u) == 0) {
      if (*abort_flag) return false;
      const uint64_t t = globaltimer_ns();
      if (t0 == 0) {
        t0 = t;
      } else if (t - t0 > kWaitLimitNs) {
        *abort_flag = 1;
        atomicOr(dev_err, DEV_ERR_WAIT_GEMM);
        return false;
      }
    }
  }
}
#endif

}  // namespace lsq
