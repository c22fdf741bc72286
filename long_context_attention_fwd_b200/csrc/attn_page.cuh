// attn_page.cuh -- paged key/value caches: where a token lies, and the 4-bit page format.
//
// A cache is a pool of pages of 2^log_ps tokens; block_table[b][n] is the page that holds
// tokens n * 2^log_ps ... of sequence b.  cache_len[b] counts the cached tokens, the ones
// being appended among them, so new token i of n lies at position cache_len[b] - n + i.
//
// bf16 pages: [num_pages][page_size][Hkv][D], K and V apart (the dense cache's layout, with
// the tokens of one sequence in any order of pages).
//
// 4-bit pages: [num_pages][Hkv][page_size / 16][18 D bytes].  A unit of 16 tokens of one head
// is one run of bytes, so that a bulk copy brings it with its scales whatever the page size:
//     K codes [16][D / 2] | V codes [16][D / 2] | K scales [16][D / 64] | V scales [16][D / 64]
// A scale is 4 bytes per group of 64 elements: bf16 step s (low half) and bf16 minimum m (high
// half); an element is s * code + m, code in 0..15.  Codes lie in 4-byte words of eight
// (element j of a word at bits 4j..4j+3); word NG * i + g of a token holds elements
// 64 g + 8 i ... + 7 (NG = D / 64 groups), so the two groups' words that one MMA lane needs
// are neighbours.
#pragma once
#include <cstdint>

#include "sm100_ptx.cuh"

namespace attn_sm100 {
namespace page {

constexpr int kUnit = 16;                 // tokens of a unit of 4-bit pages
constexpr unsigned kStatusBadPage = 4u;   // status bit: a token or a length without a valid page

enum : unsigned { kSiteAppend = 0x500, kSiteGather, kSiteDecode, kSiteDecode4 };

// Byte offsets inside a unit of 4-bit pages.
template <int D>
struct Unit {
  static constexpr int NG = D / 64;           // groups of a token
  static constexpr int CODE = D / 2;          // code bytes of a token
  static constexpr int SCALE = 4 * NG;        // scale bytes of a token
  static constexpr int OFF_KC = 0;
  static constexpr int OFF_VC = kUnit * CODE;
  static constexpr int OFF_KS = 2 * kUnit * CODE;
  static constexpr int OFF_VS = OFF_KS + kUnit * SCALE;
  static constexpr int BYTES = OFF_VS + kUnit * SCALE;
  static_assert(BYTES == 18 * D, "unit size");
};

__device__ __forceinline__ void flag_bad_page(unsigned* status, unsigned site) {
  atomicOr(status, kStatusBadPage);
  atomicCAS(status + 1, 0u, site);
}

struct PageMap {
  const int32_t* table;      // [B][width]
  const int32_t* cache_len;  // [B]
  const int32_t* cu;         // [B + 1] offsets of the packed tokens, or nullptr: one token each
  int B, T, width, num_pages, log_ps;
};

enum Placed { kOutside, kNowhere, kBad, kFound };

// Position, page and slot of packed token t (0 <= t < T), found by a whole warp.  kOutside:
// behind the last sequence.  kNowhere: the position is negative (the sequence holds fewer
// tokens than it is said to get; an unused batch entry has cache_len 0).  kBad: past the
// table, or the table's page is not in the pool.  Whatever the arrays hold, a kFound result
// lies inside the pool.
__device__ __forceinline__ Placed place_token(const PageMap& m, int t, int& pos, int& pg, int& slot) {
  const int lane = threadIdx.x & 31;
  int b = t, end = t + 1;
  if (m.cu) {
    // The last i in 0..B with cu[i] <= t, by 32-way steps.
    int lo = 0, n = m.B + 1;
    do {
      const int step = (n + 31) >> 5;
      const int off = lane * step;
      const unsigned le = __ballot_sync(0xffffffffu, off < n && __ldg(m.cu + lo + off) <= t);
      if (le == 0) return kOutside;
      const int c = (31 - __clz(le)) * step;
      lo += c;
      n = min(step, n - c);
    } while (n > 1);
    if (lo >= m.B) return kOutside;
    b = lo;
    end = __ldg(m.cu + b + 1);
  }
  pos = int(unsigned(__ldg(m.cache_len + b)) - unsigned(end) + unsigned(t));
  if (pos < 0) return kNowhere;
  const int n = pos >> m.log_ps;
  if (n >= m.width) return kBad;
  pg = __ldg(m.table + (long long)b * m.width + n);
  if (pg < 0 || pg >= m.num_pages) return kBad;
  slot = pos & ((1 << m.log_ps) - 1);
  return kFound;
}

}  // namespace page
}  // namespace attn_sm100
