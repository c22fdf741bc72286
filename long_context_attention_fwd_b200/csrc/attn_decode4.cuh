// attn_decode4.cuh -- decode attention over a paged 4-bit key/value cache for sm_100a.
//
// One new query token per sequence attends to its cached tokens, whose K and V are held as
// x = s code + m per group of 64 elements (attn_page.cuh).  With q_h a head's query,
//     q_h . k_j = sum_g ( s_jg sum_{d in g} q_hd code_jd  +  m_jg sum_{d in g} q_hd )
//     o_hd      = sum_j (p_hj s_jg) code_jd  +  sum_j p_hj m_jg            (d in group g)
// so the codes enter the products as small integers and the scales meet scores and weights, of
// which there are 64 times fewer than codes.
//
// Bound by HBM when it is done right: 18 D bytes per 16 tokens and kv head for K and V together,
// 3.6 times less than bf16.  At 24 bytes per clock and SM, turning codes into operands is the
// larger part of the instructions, so each code is touched once, in registers, and never written
// back to shared memory: the products are mma.sync m16n8k16 with the codes as the A operand
// (16 tokens, or 16 elements of V, by 16) and the heads of a kv head as the 8-wide N side.  The
// wide tensor-core path would need 4 times the bytes through shared memory for operands of which
// a decode step uses 8 columns.
//   K: codes become fp16 by OR-ing them into the mantissa of 1024 (exact), one subtraction (or
//      fma for the upper nibble of a byte) leaves 0..15.  q is scaled by a power of two to fp16:
//      exact but for 2^-25 of the row's largest element.  Sums are fp32.
//   V: the words of two tokens are interleaved by byte permutes, so that the nibbles of a pair of
//      tokens land in one register; codes become bf16 by OR-ing into 128, exact too.  The weights
//      p s are rounded to bf16 (the steps are bf16 as well, and fp16 would not hold their range):
//      a relative 2^-9 of each weight, on top of the output's own bf16 rounding.
//
// Work: the tiles (32 tokens of one kv head) of all sequences form one line, cut into equal
// parts, one per block, whatever the lengths.  A block's warps take its tiles in turn; each has
// its own ring of bulk copies (a unit of 16 tokens is one run of bytes) and its own running
// maximum, sum and output.  At the end of a (sequence, kv head) the block's warps join theirs
// through shared memory; where the pair is shared with other blocks, each writes its part and the
// last one to finish joins them (done flags with the call's tag, as attn_decode_kernel does).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attn_page.cuh"

namespace attn_sm100 {
namespace decode4 {

constexpr int kTileUnits = 2;
constexpr int kTile = kTileUnits * page::kUnit;  // tokens of a tile
constexpr float kRescaleThreshold = 8.0f;        // weights stay below 2^8 of the running maximum

enum : unsigned { kSiteFull = 0x520, kSiteDrain };

// NT blocks of 8 heads per pass; a kv head with more than 8 query heads takes passes of 16.
template <int D, int NT>
struct Cfg {
  static constexpr int W = NT == 1 ? 16 : 8;  // warps
  static constexpr int NS = 2;                // ring stages of a warp
  static constexpr int THREADS = W * 32;
  static constexpr int HEADS = 8 * NT;
  static constexpr int TILE_BYTES = kTileUnits * page::Unit<D>::BYTES;
  static constexpr int OFF_RING = 0;
  static constexpr int OFF_O = OFF_RING + W * NS * TILE_BYTES;   // [W][HEADS][D] fp32
  static constexpr int OFF_ML = OFF_O + W * HEADS * D * 4;       // [W][HEADS][2] fp32
  static constexpr int OFF_BAR = OFF_ML + W * HEADS * 8;
  static constexpr int OFF_MISC = OFF_BAR + W * NS * 8;          // 64 bytes
  static constexpr int OFF_SCAN = OFF_MISC + 64;                 // [W] fp32/int scratch
  static constexpr int SMEM_BYTES = OFF_SCAN + W * 4;
  static_assert(TILE_BYTES % 16 == 0 && SMEM_BYTES <= 227 * 1024, "shared memory");
};

struct Params {
  const __nv_bfloat16* q;     // [B][Hq][D]
  const uint8_t* pages;
  const int32_t* table;       // [B][width]
  const int32_t* cache_len;   // [B], clamped to [0, width * page size]
  int B, Hq, Hkv, G, RB;      // G query heads per kv head, in RB passes of HEADS
  int width, num_pages, log_ps;
  float* o_part;              // [2 * grid][HEADS][D]: a block's first and last shared part
  float* ml_part;             // [2 * grid][HEADS][2]
  unsigned long long* flags;  // [2 * grid]
  unsigned long long tag;
  __nv_bfloat16* o;           // [B][Hq][D]
  float* lse;                 // [B][Hq]
  float scale_log2;
  unsigned* status;
  unsigned long long timeout_ns;
};

// Token of a unit that row i (0..7) of the first product holds (row i + 8: 8 more).  The order
// makes the four tokens that the second product reads at once fall into different banks.
__device__ __forceinline__ int token_of(int i) { return i ^ ((i >> 1) & 1); }

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Codes at bits 0-3 and 16-19 (or 4-7 and 20-23) of w as an fp16 pair.
__device__ __forceinline__ uint32_t f16_low(uint32_t w) {
  const uint32_t x = (w & 0x000f000fu) | 0x64006400u;  // 1024 + code
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&x), __floats2half2_rn(1024.f, 1024.f));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t f16_high(uint32_t w) {
  const uint32_t x = (w & 0x00f000f0u) | 0x64006400u;  // 1024 + 16 code
  const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&x), __floats2half2_rn(0.0625f, 0.0625f),
                            __floats2half2_rn(-64.f, -64.f));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// Codes at bits 0-3 and 16-19 of w as a bf16 pair.
__device__ __forceinline__ uint32_t bf16_low(uint32_t w) {
  const uint32_t x = (w & 0x000f000fu) | 0x43004300u;  // 128 + code
  const __nv_bfloat162 r =
      __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&x), __floats2bfloat162_rn(128.f, 128.f));
  return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ int tiles_of(const Params& p, int b) {
  const int cap = p.width << p.log_ps;
  const int L = min(max(__ldg(p.cache_len + b), 0), cap);
  return (L + kTile - 1) / kTile;
}

// Place on the line of tiles: tile j of the nt tiles of (sequence b, head block vh).
struct Cursor {
  int b, vh, j, nt;
  __device__ __forceinline__ void settle(const Params& p, int nv) {
    while (j >= nt) {
      j -= nt;
      if (++vh == nv) {
        vh = 0;
        do ++b;
        while (b < p.B && (nt = tiles_of(p, b)) == 0);
        if (b >= p.B) return;  // past the end of the line
      }
    }
  }
};

template <int D, int NT>
__global__ void __launch_bounds__(Cfg<D, NT>::THREADS, 1) attn_decode4_kernel(const Params p) {
  using C = Cfg<D, NT>;
  using U = page::Unit<D>;
  constexpr int NG = U::NG;
  constexpr int W = C::W;
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r = lane >> 2, c = lane & 3;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR) + warp * C::NS;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC);
  volatile int* s_merge = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  volatile int* s_start = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 8);   // b, offset
  int* s_scan = reinterpret_cast<int*>(smem + C::OFF_SCAN);
  float* s_o = reinterpret_cast<float*>(smem + C::OFF_O);
  float* s_ml = reinterpret_cast<float*>(smem + C::OFF_ML);
  const int nv = p.Hkv * p.RB;
  const WaitCtl wc{p.status, abort_flag, p.timeout_ns};

  if (tid == 0) *abort_flag = 0;
  if (lane == 0)
    for (int i = 0; i < C::NS; ++i) mbar_init(&full[i], 1);
  fence_mbar_init();

  // ---- this block's part [t0, t1) of the line, and where it starts
  int total = 0;
  for (int b = tid; b < p.B; b += C::THREADS) total += tiles_of(p, b);
  total = __reduce_add_sync(0xffffffffu, total);
  if (lane == 0) s_scan[warp] = total;
  __syncthreads();
  total = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) total += s_scan[w];
  total *= nv;
  const int chunk = max((total + int(gridDim.x) - 1) / int(gridDim.x), W);
  const int t0 = min(total, int(blockIdx.x) * chunk), t1 = min(total, t0 + chunk);
  __syncthreads();

  // Sequences without tokens: o = 0, lse = -inf.
  for (int b = blockIdx.x; b < p.B; b += gridDim.x)
    if (tiles_of(p, b) == 0)
      for (int i = tid; i < p.Hq * (D / 8); i += C::THREADS) {
        reinterpret_cast<uint4*>(p.o)[(long long)b * p.Hq * (D / 8) + i] = make_uint4(0u, 0u, 0u, 0u);
        if (i < p.Hq) p.lse[(long long)b * p.Hq + i] = -INFINITY;
      }
  if (t0 >= t1) return;

  if (warp == 0) {
    int before = 0;  // tiles (times nv) of the sequences before this group of 32
    for (int b0 = 0;; b0 += 32) {
      const int n = b0 + lane < p.B ? tiles_of(p, b0 + lane) * nv : 0;
      int incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      const unsigned past = __ballot_sync(0xffffffffu, before + incl > t0);
      if (past) {
        const int l = __ffs(past) - 1;
        if (lane == l) {
          s_start[0] = b0 + lane;
          s_start[1] = t0 - (before + incl - n);
        }
        break;
      }
      before += __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  __syncthreads();

  Cursor item;  // the (sequence, head block) the block is at; j counts from the item's own start
  item.b = s_start[0];
  item.nt = tiles_of(p, item.b);
  item.vh = s_start[1] / item.nt;
  item.j = s_start[1] % item.nt;

  // ---- this warp's copies: tiles t0 + warp, t0 + warp + W, ...
  uint8_t* ring = smem + C::OFF_RING + warp * C::NS * C::TILE_BYTES;
  const int upp_log = p.log_ps - 4;          // units of a page
  const int cap = p.width << p.log_ps;
  Cursor next = item;
  next.j += warp;
  next.settle(p, nv);
  int t_issue = t0 + warp;
  int pg_next = 0;
  auto fetch_page = [&] {                     // lane i: page of unit i of the next tile
    if (t_issue < t1 && lane < kTileUnits) {
      const int u = next.j * kTileUnits + lane;
      const int n = u >> upp_log;
      pg_next = n < p.width ? __ldg(p.table + (long long)next.b * p.width + n) : 0;
    }
  };
  auto issue = [&](int st) {
    if (t_issue >= t1) return;
    const int L = min(max(__ldg(p.cache_len + next.b), 0), cap);
    const int units = min(kTileUnits, (L + page::kUnit - 1) / page::kUnit - next.j * kTileUnits);
    if (lane == 0) mbar_arrive_expect_tx(&full[st], uint32_t(units) * U::BYTES);
    __syncwarp();
    // One copy per page: a tile lies in one page, or its units in a page each.
    const bool single = upp_log >= 1;
    if (lane < (single ? 1 : units)) {
      int pg = pg_next;
      if (pg < 0 || pg >= p.num_pages) {
        page::flag_bad_page(p.status, page::kSiteDecode4);
        pg = 0;
      }
      const int u = next.j * kTileUnits + lane;
      const uint8_t* src = p.pages + ((((long long)pg * p.Hkv + next.vh / p.RB) << upp_log) +
                                      (u & ((1 << upp_log) - 1))) * U::BYTES;
      bulk_load(ring + st * C::TILE_BYTES + lane * U::BYTES, src,
                uint32_t(single ? units : 1) * U::BYTES, &full[st]);
    }
    t_issue += W;
    next.j += W;
    if (t_issue < t1) next.settle(p, nv);
    fetch_page();
  };
  fetch_page();
  int issued = 0;
  for (; issued < C::NS && t_issue < t1; ++issued) issue(issued);

  // ---- tiles
  int done = 0;      // tiles this warp has taken
  int t = t0;        // start of the item on the line
  bool ok = true;
  const int key0 = token_of(r);
  while (t < t1) {
    const int e = min(t1, t + item.nt - item.j);         // end of the item's part
    const int L = min(max(__ldg(p.cache_len + item.b), 0), cap);
    const int g = item.vh / p.RB, rb = item.vh % p.RB;
    const int h0 = g * p.G + rb * C::HEADS;              // first query head of the pass
    const int nh = min(C::HEADS, p.G - rb * C::HEADS);
    const __nv_bfloat16* qrow = p.q + ((long long)item.b * p.Hq + h0) * D;

    uint32_t qf[NG][4][NT][2];
    float qsum[NG][NT][2], csc[NT][2];
    float m_run[NT][2], l_run[NT][2], om[NG][NT][2];
    float oacc[NG][4][NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e2 = 0; e2 < 2; ++e2) {
        m_run[nt][e2] = -INFINITY;
        l_run[nt][e2] = 0.f;
#pragma unroll
        for (int gg = 0; gg < NG; ++gg) om[gg][nt][e2] = 0.f;
      }
#pragma unroll
    for (int gg = 0; gg < NG; ++gg)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 4; ++k) oacc[gg][i][nt][k] = 0.f;

    if (t0 + warp + done * W < e) {
      // Queries of this warp's fragments: head nt * 8 + r, the elements of words 2c, 2c + 1.
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const bool have = nt * 8 + r < nh;
        float x[NG][2][8], big = 0.f, sum[NG];
#pragma unroll
        for (int gg = 0; gg < NG; ++gg) {
          sum[gg] = 0.f;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (have) v = __ldg(reinterpret_cast<const uint4*>(qrow + (nt * 8 + r) * D + gg * 64 + (2 * c + i) * 8));
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              x[gg][i][2 * k] = __uint_as_float(w[k] << 16);
              x[gg][i][2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              big = fmaxf(big, fabsf(x[gg][i][k]));
              sum[gg] += x[gg][i][k];
            }
          }
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
          big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
#pragma unroll
          for (int gg = 0; gg < NG; ++gg) sum[gg] += __shfl_xor_sync(0xffffffffu, sum[gg], o);
        }
        // 2^-ex brings the row's largest element into [1, 2); both powers are normal numbers.
        const int ex = min(max(int((__float_as_uint(big) >> 23) & 0xff) - 127, -126), 126);
        const float down = __uint_as_float(uint32_t(127 - ex) << 23);
        const float up = __uint_as_float(uint32_t(127 + ex) << 23);
#pragma unroll
        for (int gg = 0; gg < NG; ++gg)
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h)   // step 2i + h of the group: elements 2h, 2h + 4 | 2h + 1, 2h + 5
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const __half2 y = __floats2half2_rn(x[gg][i][2 * h + k] * down, x[gg][i][2 * h + k + 4] * down);
                qf[gg][2 * i + h][nt][k] = *reinterpret_cast<const uint32_t*>(&y);
              }
        // To the accumulator's layout: heads 2c and 2c + 1.
#pragma unroll
        for (int e2 = 0; e2 < 2; ++e2) {
          const int src = 4 * (2 * c + e2);
          csc[nt][e2] = __shfl_sync(0xffffffffu, up, src) * p.scale_log2;
          const float dn = __shfl_sync(0xffffffffu, down, src);
#pragma unroll
          for (int gg = 0; gg < NG; ++gg) qsum[gg][nt][e2] = __shfl_sync(0xffffffffu, sum[gg], src) * dn;
        }
      }
    }

    for (; t0 + warp + done * W < e; ++done) {
      const int st = done % C::NS;
      ok = ok && __all_sync(0xffffffffu, mbar_wait(&full[st], (done / C::NS) & 1, wc, kSiteFull));
      if (!ok) continue;
      const uint8_t* tile = ring + st * C::TILE_BYTES;
      const int key_base = (item.j + (t0 + warp + done * W - t)) * kTile;
      const bool ragged = key_base + kTile > L;

      // scores, times log2(e)
      float sc[kTileUnits][NT][4];
#pragma unroll
      for (int u = 0; u < kTileUnits; ++u) {
        const uint8_t* unit = tile + u * U::BYTES;
        uint32_t w[2][2 * NG];   // [token half][2 * word + group]
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const uint8_t* src = unit + U::OFF_KC + (key0 + 8 * hh) * U::CODE + c * 8 * NG;
          if constexpr (NG == 2) {
            const uint4 v = *reinterpret_cast<const uint4*>(src);
            w[hh][0] = v.x, w[hh][1] = v.y, w[hh][2] = v.z, w[hh][3] = v.w;
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(src);
            w[hh][0] = v.x, w[hh][1] = v.y;
          }
        }
        uint32_t sm[2][NG];
#pragma unroll
        for (int hh = 0; hh < 2; ++hh)
#pragma unroll
          for (int gg = 0; gg < NG; ++gg)
            sm[hh][gg] = *reinterpret_cast<const uint32_t*>(unit + U::OFF_KS + (key0 + 8 * hh) * U::SCALE + 4 * gg);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 4; ++k) sc[u][nt][k] = 0.f;
#pragma unroll
        for (int gg = 0; gg < NG; ++gg) {
          float acc[NT][4];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[nt][k] = 0.f;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t x0 = w[0][NG * i + gg], x1 = w[1][NG * i + gg];
            const uint32_t a0[4] = {f16_low(x0), f16_low(x1), f16_high(x0), f16_high(x1)};
            const uint32_t y0 = x0 >> 8, y1 = x1 >> 8;
            const uint32_t a1[4] = {f16_low(y0), f16_low(y1), f16_high(y0), f16_high(y1)};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma_f16(acc[nt], a0, qf[gg][2 * i][nt]);
              mma_f16(acc[nt], a1, qf[gg][2 * i + 1][nt]);
            }
          }
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const float s = __uint_as_float(sm[hh][gg] << 16), m = __uint_as_float(sm[hh][gg] & 0xffff0000u);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e2 = 0; e2 < 2; ++e2)
                sc[u][nt][2 * hh + e2] = fmaf(s, acc[nt][2 * hh + e2], fmaf(m, qsum[gg][nt][e2], sc[u][nt][2 * hh + e2]));
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 4; ++k) sc[u][nt][k] *= csc[nt][k & 1];
      }
      if (ragged) {
#pragma unroll
        for (int u = 0; u < kTileUnits; ++u)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (key_base + u * page::kUnit + key0 + 8 * (k >> 1) >= L) sc[u][nt][k] = -INFINITY;
      }

      // running maximum: moved only when a weight would pass 2^kRescaleThreshold
      bool need = false;
      float mx[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e2 = 0; e2 < 2; ++e2) {
          float x = fmaxf(sc[0][nt][e2], sc[0][nt][2 + e2]);
#pragma unroll
          for (int u = 1; u < kTileUnits; ++u) x = fmax3(x, sc[u][nt][e2], sc[u][nt][2 + e2]);
          mx[nt][e2] = x;
          need = need || x > m_run[nt][e2] + kRescaleThreshold;
        }
      if (__any_sync(0xffffffffu, need)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e2 = 0; e2 < 2; ++e2) {
            float x = mx[nt][e2];
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
            const float m_new = fmaxf(m_run[nt][e2], x);
            const float alpha = m_new == -INFINITY ? 1.f : ex2_approx(m_run[nt][e2] - m_new);
            m_run[nt][e2] = m_new;
            l_run[nt][e2] *= alpha;
#pragma unroll
            for (int gg = 0; gg < NG; ++gg) {
              om[gg][nt][e2] *= alpha;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                oacc[gg][i][nt][e2] *= alpha;
                oacc[gg][i][nt][2 + e2] *= alpha;
              }
            }
          }
      }

      // weights and the second product
      float mneg[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e2 = 0; e2 < 2; ++e2) mneg[nt][e2] = m_run[nt][e2] == -INFINITY ? 0.f : m_run[nt][e2];
#pragma unroll
      for (int u = 0; u < kTileUnits; ++u) {
        const uint8_t* unit = tile + u * U::BYTES;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            sc[u][nt][k] = ex2_approx(sc[u][nt][k] - mneg[nt][k & 1]);
            l_run[nt][k & 1] += sc[u][nt][k];
          }
        uint32_t wv[4][NG];   // tokens of pair slots 2c, 2c + 1, 2c + 8, 2c + 9
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint8_t* src = unit + U::OFF_VC + (token_of(2 * c + (k & 1)) + 8 * (k >> 1)) * U::CODE + r * 4 * NG;
          if constexpr (NG == 2) {
            const uint2 v = *reinterpret_cast<const uint2*>(src);
            wv[k][0] = v.x, wv[k][1] = v.y;
          } else {
            wv[k][0] = *reinterpret_cast<const uint32_t*>(src);
          }
        }
#pragma unroll
        for (int gg = 0; gg < NG; ++gg) {
          uint32_t pb[NT][2];
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            uint32_t sm = *reinterpret_cast<const uint32_t*>(unit + U::OFF_VS + (key0 + 8 * hh) * U::SCALE + 4 * gg);
            if (ragged && key_base + u * page::kUnit + key0 + 8 * hh >= L) sm = 0u;  // whatever lies there
            const float s = __uint_as_float(sm << 16), m = __uint_as_float(sm & 0xffff0000u);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const float p0 = sc[u][nt][2 * hh], p1 = sc[u][nt][2 * hh + 1];
              om[gg][nt][0] = fmaf(p0, m, om[gg][nt][0]);
              om[gg][nt][1] = fmaf(p1, m, om[gg][nt][1]);
              pb[nt][hh] = transpose8x8(pack_bf16x2(p0 * s, p1 * s));
            }
          }
          const uint32_t ab_lo = __byte_perm(wv[0][gg], wv[1][gg], 0x5410), ab_hi = __byte_perm(wv[0][gg], wv[1][gg], 0x7632);
          const uint32_t cd_lo = __byte_perm(wv[2][gg], wv[3][gg], 0x5410), cd_hi = __byte_perm(wv[2][gg], wv[3][gg], 0x7632);
#pragma unroll
          for (int i = 0; i < 4; ++i) {   // rows r: element i of the word; rows r + 8: element i + 4
            const uint32_t a[4] = {bf16_low(ab_lo >> (4 * i)), bf16_low(ab_hi >> (4 * i)),
                                   bf16_low(cd_lo >> (4 * i)), bf16_low(cd_hi >> (4 * i))};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_bf16(oacc[gg][i][nt], a, pb[nt]);
          }
        }
      }
      __syncwarp();  // every lane has read the stage
      issue(st);
    }

    // ---- join the warps' parts of this item
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e2 = 0; e2 < 2; ++e2) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          l_run[nt][e2] += __shfl_xor_sync(0xffffffffu, l_run[nt][e2], o);
#pragma unroll
          for (int gg = 0; gg < NG; ++gg) om[gg][nt][e2] += __shfl_xor_sync(0xffffffffu, om[gg][nt][e2], o);
        }
        const int h = nt * 8 + 2 * c + e2;
        if (h < nh) {
          if (r == 0) {
            s_ml[(warp * C::HEADS + h) * 2] = m_run[nt][e2];
            s_ml[(warp * C::HEADS + h) * 2 + 1] = l_run[nt][e2];
          }
#pragma unroll
          for (int gg = 0; gg < NG; ++gg) {
            const float add = om[gg][nt][e2];
            float4* dst = reinterpret_cast<float4*>(s_o + (warp * C::HEADS + h) * D + gg * 64 + r * 8);
            dst[0] = make_float4(oacc[gg][0][nt][e2] + add, oacc[gg][1][nt][e2] + add,
                                 oacc[gg][2][nt][e2] + add, oacc[gg][3][nt][e2] + add);
            dst[1] = make_float4(oacc[gg][0][nt][2 + e2] + add, oacc[gg][1][nt][2 + e2] + add,
                                 oacc[gg][2][nt][2 + e2] + add, oacc[gg][3][nt][2 + e2] + add);
          }
        }
      }
    __syncthreads();
    const int a_line = t - item.j, e_line = a_line + item.nt;   // the whole item on the line
    const bool shared_item = a_line < t0 || e_line > t1;
    const int slot = 2 * blockIdx.x + (a_line < t0 ? 0 : 1);
    for (int i = tid; i < nh * (D / 4); i += C::THREADS) {
      const int h = i / (D / 4), d4 = i % (D / 4);
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < W; ++w) M = fmaxf(M, s_ml[(w * C::HEADS + h) * 2]);
      const float Mz = M == -INFINITY ? 0.f : M;
      float l = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int w = 0; w < W; ++w) {
        const float x = ex2_approx(s_ml[(w * C::HEADS + h) * 2] - Mz);
        const float4 y = reinterpret_cast<const float4*>(s_o)[(w * C::HEADS + h) * (D / 4) + d4];
        l = fmaf(x, s_ml[(w * C::HEADS + h) * 2 + 1], l);
        o.x = fmaf(x, y.x, o.x), o.y = fmaf(x, y.y, o.y), o.z = fmaf(x, y.z, o.z), o.w = fmaf(x, y.w, o.w);
      }
      if (shared_item) {
        reinterpret_cast<float4*>(p.o_part)[((long long)slot * C::HEADS + h) * (D / 4) + d4] = o;
        if (d4 == 0) {
          p.ml_part[((long long)slot * C::HEADS + h) * 2] = M;
          p.ml_part[((long long)slot * C::HEADS + h) * 2 + 1] = l;
        }
      } else {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const long long row = (long long)item.b * p.Hq + h0 + h;
        reinterpret_cast<uint2*>(p.o)[row * (D / 4) + d4] =
            make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
        if (d4 == 0) p.lse[row] = l == 0.f ? -INFINITY : (M + log2f(l)) * 0.69314718055994530942f;
      }
    }
    if (shared_item) {
      const int c0 = a_line / chunk, c1 = (e_line - 1) / chunk;   // the blocks that share the item
      __threadfence();
      __syncthreads();
      if (warp == 0) {
        volatile unsigned long long* fl = p.flags;
        if (lane == 0) fl[slot] = p.tag;
        __syncwarp();
        __threadfence();
        // Block c0 started the item (unless it began exactly at its part: still its last slot).
        auto slot_of = [&](int k) { return 2 * k + (a_line < k * chunk ? 0 : 1); };
        bool all = true;
        for (int k = c0 + lane; k <= c1; k += 32) all = all && fl[slot_of(k)] == p.tag;
        all = __all_sync(0xffffffffu, all);
        if (all)
          for (int k = c0 + lane; k <= c1; k += 32) fl[slot_of(k)] = 0ull;
        if (lane == 0) *s_merge = all;
      }
      __syncthreads();
      if (*s_merge) {
        __threadfence();
        for (int i = tid; i < nh * (D / 4); i += C::THREADS) {
          const int h = i / (D / 4), d4 = i % (D / 4);
          float M = -INFINITY, l = 0.f;
          float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int k = c0; k <= c1; ++k) {
            const long long s = 2 * k + (a_line < k * chunk ? 0 : 1);
            M = fmaxf(M, __ldcg(p.ml_part + (s * C::HEADS + h) * 2));
          }
          const float Mz = M == -INFINITY ? 0.f : M;
#pragma unroll 4
          for (int k = c0; k <= c1; ++k) {
            const long long s = 2 * k + (a_line < k * chunk ? 0 : 1);
            const float x = ex2_approx(__ldcg(p.ml_part + (s * C::HEADS + h) * 2) - Mz);
            const float4 y = __ldcg(reinterpret_cast<const float4*>(p.o_part) + (s * C::HEADS + h) * (D / 4) + d4);
            l = fmaf(x, __ldcg(p.ml_part + (s * C::HEADS + h) * 2 + 1), l);
            o.x = fmaf(x, y.x, o.x), o.y = fmaf(x, y.y, o.y), o.z = fmaf(x, y.z, o.z), o.w = fmaf(x, y.w, o.w);
          }
          const float inv = l == 0.f ? 0.f : 1.f / l;
          const long long row = (long long)item.b * p.Hq + h0 + h;
          reinterpret_cast<uint2*>(p.o)[row * (D / 4) + d4] =
              make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
          if (d4 == 0) p.lse[row] = l == 0.f ? -INFINITY : (M + log2f(l)) * 0.69314718055994530942f;
        }
      }
    }
    __syncthreads();  // the join's buffers are free again

    item.j += e - t;
    t = e;
    if (t < t1) item.settle(p, nv);
  }

  // Copies still in flight (only when a wait gave up) land before shared memory is released.
  if (!ok && lane == 0) {
    const int n = (t_issue - t0 - warp) / W;   // tiles issued
    for (int k = max(0, n - C::NS); k < n; ++k)
      mbar_drain_checked(&full[k % C::NS], (k / C::NS) & 1, wc, kSiteDrain);
  }
}

}  // namespace decode4
}  // namespace attn_sm100
