// attn_decode4.cuh -- decode attention over a paged 4-bit key/value cache for sm_100a.
//
// One new query token per sequence attends to its cached tokens, whose K and V are held as
// x = s code + m per group of 64 elements (attn_page.cuh).  With q_h a head's query,
//     q_h . k_j = sum_g ( s_jg sum_{d in g} q_hd code_jd  +  m_jg sum_{d in g} q_hd )
//     o_hd      = sum_j (p_hj s_jg) code_jd  +  sum_j p_hj m_jg            (d in group g)
// so the codes enter the products as small integers and the scales meet scores and weights, of
// which there are 64 times fewer than codes.
//
// Its floor is HBM: 18 D bytes per 16 tokens and kv head for K and V together, 3.6 times less
// than bf16.  At the 24 bytes a clock that an SM gets, turning codes into operands is most of
// the instructions, so each code is touched once, in registers, and never written back to shared
// memory: the products are mma.sync m16n8k16 with the codes as the A operand (16 tokens, or 16
// elements of V, by 16) and the heads of a kv head as the 8-wide N side.  (A tcgen05 form was
// built: codes as e4m3 bytes in shared memory, tokens and then elements on the 128-row side, and
// the heads of q and of the weights in three e4m3 parts each on N.  It was right, and took 271 us
// where this takes 102: splitting the weights and handing every tile over between warps cost
// more than the products.)
//   A nibble needs no conversion: masked out of its word it is the fp16 subnormal code * 2^-24
//   (or code * 2^-20, the upper nibble of a byte), which the tensor cores multiply exactly; one
//   AND makes two operands.  The powers of two go into q (K) and into the final scale (V).
//   K: q is scaled by a power of two to fp16, exact but for 2^-38 of the row's largest element, 2^-34
//      for the elements that meet upper nibbles.
//   V: the words of two tokens are interleaved by byte permutes, so that the nibbles of a pair of
//      tokens land in one register.  The weights p s are rounded to fp16, a relative 2^-11 of
//      each weight where bf16 would cost 2^-8 (2^-25 below 2^-14).  fp16's range is kept by the
//      softmax's reference R_h, which is not the largest score but moves so that p s, p = 2^(x - R),
//      stays below 2^14 and its largest value over both groups so far is at least 1; sums of p and of
//      p m are fp32.  A group whose steps are so far below the other's that its weights are lost in
//      this shared range is done again in fp32 (plain_tiles): from ratios of about 2^9 on where one of
//      thousands of tokens has all the weight, of 2^13 or more where many share it.
//
// Work: the tiles (kTile tokens of one kv head) of all sequences form one line, with empty places
// for each start, cut into equal parts, one per block, whatever the lengths.  A block's warps take
// its tiles in turn; each has its own ring of asynchronous copies, its own reference, sum and output,
// and waits for nobody.
// (Copies are 16 bytes a lane: one bulk copy per unit, 2304 bytes, moved 4.3 TB/s at most, where
// these alone move 6.4.)
// At the end of a (sequence, kv head) the block's warps join theirs through shared memory; where
// the pair is shared with other blocks, each writes its part and the last one to finish joins
// them (done flags with the call's tag, as attn_decode_kernel does).
//
// Measured, D = 128, 28 / 4 heads: 48 sequences of 1-32K tokens in pages of 16, 391 MB, 97 us
// (4.0 TB/s, 62% of the copy rate); one of 32K, 14.4 us; one of 513, 9 us.  64 / 4 heads: 146 and
// (16 / 1) 21.0 us.  The first fills no pipe (issue and ALU are active half of the time, tensor a
// quarter): with two warps a scheduler, the copies, the conversions and the products largely add up
// (when it took 102 us: without the copies 81, without the products 72, without both 44; an m16n8k16
// holds its scheduler's issue for about 7 of its 8 cycles).  The others are latency: the length,
// the page, the codes and the join are loads behind one another.  Eight warps with 64-token tiles
// are the best of those tried: more warps need smaller tiles, whose scores, weights and copies
// overlap less (16 warps of 32 tokens 116 us, two blocks of 8 101 us but 20 us for one of 32K).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attn_page.cuh"

namespace attn_sm100 {
namespace decode4 {

constexpr int kTileUnits = 4;
constexpr int kTile = kTileUnits * page::kUnit;  // tokens of a tile
constexpr uint32_t kTopWeight = 0x7400u;         // 2^14 as fp16: a weight this large moves the reference
constexpr float kFirstWeight = 6.f;              // ... so that the largest becomes 2^6
// What else keeps p and p m inside fp32: a token counts in the reference with its steps, 2^-24 of
// its minima (steps can be 0 where minima are not) and 2^-88 at least, and the reference also
// moves when p reaches 2^100, or for every tile with a minimum of 2^10 or more.  (Next to a token
// without steps or minima, weights below 2^-100 of its own are lost.)
constexpr float kMinimumShare = 5.9604644775390625e-8f;
constexpr float kSmallStep = 3.2311742677852644e-27f;
constexpr float kTopP = 1.2676506002282294e30f;
constexpr float kTopMinimum = 1024.f;

constexpr int kEvenSteps = 6;                     // log2: steps this far below share the reference well
constexpr int kMaxParts = 160;                   // blocks that can share a (sequence, kv head)

// NT blocks of 8 heads per pass; a kv head with more than 8 query heads takes passes of 16, whose tiles
// are computed in halves at D = 128: the scores and weights of 64 tokens and 16 heads spilled (64 / 4
// heads, 48 sequences of 1-32K: 155 us, in halves 146; D = 64 does not spill: 114, in halves 120).
template <int D, int NT>
struct Cfg {
  static constexpr int W = 8;                 // warps
  static constexpr int NS = 2;                // ring stages of a warp
  static constexpr int TR = D == 128 ? kTileUnits / NT : kTileUnits;  // units computed at a time
  static constexpr int THREADS = W * 32;
  static constexpr int HEADS = 8 * NT;
  static constexpr int TILE_BYTES = kTileUnits * page::Unit<D>::BYTES;
  static constexpr int OFF_RING = 0;
  static constexpr int OFF_O = OFF_RING + W * NS * TILE_BYTES;   // [W][HEADS][D] fp32
  static constexpr int OFF_L = OFF_O + W * HEADS * D * 4;        // [W][HEADS] fp32
  static constexpr int OFF_WT = OFF_L + W * HEADS * 4;           // [kMaxParts][HEADS] fp32
  static constexpr int OFF_MISC = OFF_WT + kMaxParts * HEADS * 4;  // merge flag
  static constexpr int SMEM_BYTES = OFF_MISC + 16;
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
  float* l_part;              // [2 * grid][HEADS]
  unsigned long long* flags;  // [2 * grid]
  unsigned long long tag;
  __nv_bfloat16* o;           // [B][Hq][D]
  float* lse;                 // [B][Hq]
  float up_scale, scale_log2; // 2^11 scale log2(e) as a product; the second is above 0 (masked scores are -inf)
  unsigned* status;
};

// Token of a unit that row i (0..7) of the first product holds (row i + 8: 8 more).  The order
// spreads the four tokens that the second product reads at once over the banks.
__device__ __forceinline__ int token_of(int i) { return i ^ ((i >> 1) & 1); }

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        const uint32_t (&b)[2]) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b[0]), "r"(b[1]));
}
// 16 bytes, global to shared, past L1.
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t y;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(hi), "f"(lo));
  return y;
}
__device__ __forceinline__ uint32_t max_f16x2(uint32_t a, uint32_t b) {
  uint32_t y;
  asm("max.f16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  return y;
}
__device__ __forceinline__ float step_of(uint32_t sm) { return __uint_as_float(sm << 16); }
__device__ __forceinline__ float low_of(uint32_t sm) { return __uint_as_float(sm & 0xffff0000u); }

constexpr uint32_t kLowNibbles = 0x000f000fu, kHighNibbles = 0x00f000f0u;

__device__ __forceinline__ int length_of(const Params& p, int b) {
  return min(max(__ldg(p.cache_len + b), 0), p.width << p.log_ps);
}
__device__ __forceinline__ int tiles_of(int L) { return (L + kTile - 1) / kTile; }

// Place on the line of tiles: tile j of the nt tiles of (sequence b, head block vh).  settle: on to
// the item that j, past the end, lies in; returns the items passed.
struct Cursor {
  int b, vh, j, nt, L;
  __device__ __forceinline__ int settle(const Params& p, int nv) {
    int passed = 0;
    while (j >= nt) {
      j -= nt;
      ++passed;
      if (++vh == nv) {
        vh = 0;
        do {
          if (++b >= p.B) return passed;  // past the end of the line
          L = length_of(p, b);
          nt = tiles_of(L);
        } while (nt == 0);
      }
    }
    return passed;
  }
};

// A warp's tiles of an item (ntile of them, from `tile` on, `every` apart) in plain fp32, where steps
// of any size keep their part; some fifteen times slower than the products (48 sequences of 1-32K, 28
// / 4 heads, all done again: 1.6 ms; four heads at a time 1.0, but 1% of every other call).  few: the
// groups in doubt.  Where all their steps are 0, or no token has a step that is about 2^kEvenSteps
// below what its reference went by, there is no doubt and nothing is done (35 us in that case).
// q: the heads' rows; row: the sequence's pages; out, out_l: normalised outputs [nh][D] and log2
// sums [nh].
template <int D>
__device__ __forceinline__ void plain_tiles(const Params& p, const __nv_bfloat16* q, const int32_t* row, int g, int nh,
                                            int tile, int ntile, int every, int L, unsigned few, float* out, float* out_l) {
  using U = page::Unit<D>;
  static_assert(U::NG == 2, "a half warp for each group");
  const int lane = threadIdx.x & 31, upp_log = p.log_ps - 4;
  auto unit_at = [&](int u) {
    int pg = __ldg(row + (u >> upp_log));
    if (pg < 0 || pg >= p.num_pages) pg = 0;            // recorded by the copies
    return p.pages + ((((long long)pg * p.Hkv + g) << upp_log) + (u & ((1 << upp_log) - 1))) * U::BYTES;
  };
  unsigned seen = 0u;                                   // groups with a step above 0; a token like that
  for (int i = lane; i < ntile * kTile; i += 32) {
    const int t = (tile + i / kTile * every) * kTile + i % kTile;
    if (t >= L) break;
    const uint2 sm = *reinterpret_cast<const uint2*>(unit_at(t >> 4) + U::OFF_VS + (t & 15) * U::SCALE);
    // Exponents of the steps, and of what else the reference goes by (kMinimumShare, kSmallStep).
    const int s0 = (sm.x >> 7) & 0xff, s1 = (sm.y >> 7) & 0xff;
    const int other = max(max(int((sm.x >> 23) & 0xff), int((sm.y >> 23) & 0xff)) - 24, 127 - 88);
    seen |= (sm.x & 0xffffu ? 1u : 0u) | (sm.y & 0xffffu ? 2u : 0u);
    if ((sm.x | sm.y) != 0u && max(max(s0, s1), other) - min(s0, s1) > kEvenSteps) seen |= 4u;
  }
  seen = __reduce_or_sync(0xffffffffu, seen);
  if (!(seen & few) || !(seen & 4u)) return;

  const float scale_log2 = p.up_scale * 0x1p-11f * p.scale_log2;
  const int tok = lane & 15, half = lane >> 4;          // scores: a half of a token
  const int vw = lane >> 1, vj = 4 * (lane & 1);        // outputs: four elements of word vw
  const int vg = vw % U::NG, vd = 64 * vg + 8 * (vw / U::NG) + vj;
  constexpr int NH = 2;                                 // heads at a time, the last ones twice
  for (int h0 = 0; h0 < nh; h0 += NH) {
    float m[NH], l[NH], o[NH][4];
#pragma unroll
    for (int k = 0; k < NH; ++k) m[k] = -INFINITY, l[k] = o[k][0] = o[k][1] = o[k][2] = o[k][3] = 0.f;
#pragma unroll 1
    for (int i = 0; i < ntile * kTileUnits; ++i) {
      const int u = (tile + i / kTileUnits * every) * kTileUnits + i % kTileUnits;
      const int left = L - u * page::kUnit;
      if (left <= 0) break;
      const uint8_t* unit = unit_at(u);
      const uint32_t* kw = reinterpret_cast<const uint32_t*>(unit + U::OFF_KC + tok * U::CODE) + half;
      const uint32_t ks = reinterpret_cast<const uint32_t*>(unit + U::OFF_KS + tok * U::SCALE)[half];
      uint32_t vc[page::kUnit], vs[page::kUnit];
#pragma unroll
      for (int t = 0; t < page::kUnit; ++t) {           // behind the length: nothing
        vc[t] = t < left ? reinterpret_cast<const uint32_t*>(unit + U::OFF_VC + t * U::CODE)[vw] >> (4 * vj) : 0u;
        vs[t] = t < left ? reinterpret_cast<const uint32_t*>(unit + U::OFF_VS + t * U::SCALE)[vg] : 0u;
      }
      float x[NH] = {};
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        const uint32_t codes = kw[U::NG * w];
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = fmaf(step_of(ks), float(codes >> (4 * j) & 15u), low_of(ks));
#pragma unroll
        for (int k = 0; k < NH; ++k) {
          const uint4 v = __ldg(reinterpret_cast<const uint4*>(q + min(h0 + k, nh - 1) * D + 64 * half + 8 * w));
          const uint32_t e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) x[k] = fmaf(low_of(e[j]), y[2 * j + 1], fmaf(step_of(e[j]), y[2 * j], x[k]));
        }
      }
      float pr[NH];
#pragma unroll
      for (int k = 0; k < NH; ++k) {
        float y = (x[k] + __shfl_xor_sync(0xffffffffu, x[k], 16)) * scale_log2;
        if (tok >= left) y = -INFINITY;
        float top = fmaxf(m[k], y);
#pragma unroll
        for (int s = 1; s < 16; s <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
        const float ref = top == -INFINITY ? 0.f : top, alpha = ex2_approx(m[k] - ref);
        pr[k] = ex2_approx(y - ref);
        float sum = pr[k];
#pragma unroll
        for (int s = 1; s < 16; s <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
        m[k] = top;
        l[k] = fmaf(l[k], alpha, sum);
#pragma unroll
        for (int j = 0; j < 4; ++j) o[k][j] *= alpha;
      }
#pragma unroll
      for (int t = 0; t < page::kUnit; ++t) {
        float y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = fmaf(step_of(vs[t]), float(vc[t] >> (4 * j) & 15u), low_of(vs[t]));
#pragma unroll
        for (int k = 0; k < NH; ++k) {
          const float pt = __shfl_sync(0xffffffffu, pr[k], t);
#pragma unroll
          for (int j = 0; j < 4; ++j) o[k][j] = fmaf(pt, y[j], o[k][j]);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < NH; ++k) {
      const int h = min(h0 + k, nh - 1);
      const float inv = l[k] == 0.f ? 0.f : 1.f / l[k];
      *reinterpret_cast<float4*>(out + h * D + vd) = make_float4(o[k][0] * inv, o[k][1] * inv, o[k][2] * inv, o[k][3] * inv);
      if (lane == 0) out_l[h] = l[k] == 0.f ? -INFINITY : m[k] + log2f(l[k]);
    }
  }
}

template <int D, int NT>
__global__ void __launch_bounds__(Cfg<D, NT>::THREADS, 1) attn_decode4_kernel(const Params p) {
  using C = Cfg<D, NT>;
  using U = page::Unit<D>;
  constexpr int NG = U::NG;
  constexpr int W = C::W;
  constexpr int TU = kTileUnits, TR = C::TR;
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r = lane >> 2, c = lane & 3;
  volatile int* s_merge = reinterpret_cast<volatile int*>(smem + C::OFF_MISC);
  float* s_o = reinterpret_cast<float*>(smem + C::OFF_O);
  float* s_l = reinterpret_cast<float*>(smem + C::OFF_L);
  float* s_wt = reinterpret_cast<float*>(smem + C::OFF_WT);
  const int nv = p.Hkv * p.RB;

  // ---- this block's part [t0, t1) of the line, and where it starts (every warp by itself)
  int total = 0, longest = 0, live = 0;
  for (int b = lane; b < p.B; b += 32) {
    const int n = tiles_of(length_of(p, b));
    total += n;
    live += n > 0;
    longest = max(longest, n);
  }
  total = __reduce_add_sync(0xffffffffu, total) * nv;
  live = __reduce_add_sync(0xffffffffu, live) * nv;
  longest = __reduce_max_sync(0xffffffffu, longest);
  const int grid = int(gridDim.x);
  auto share = [&] {
    // Equal parts.  While they are short: whole rounds of the warps, and no cut through sequences
    // of at most two rounds (joining blocks costs more than a second round).
    int x = max((total + grid - 1) / grid, min(W, longest));
    if (longest > W && x < 4 * W) x = (x + W - 1) / W * W;
    return longest <= 2 * W ? max(x, longest) : x;
  };
  // With few sequences and heads, or short ones and a block for each, each begins at a block of its
  // own: a block that ends one and begins the next would be last (28 / 4 heads, 1-600 tokens: 32
  // sequences 9.0 us so; 33, which a lane each cannot hold, 15.7).  Otherwise every item has W places
  // without tiles behind it on the line, what its start and its join cost (64 sequences of 1-600
  // tokens: 55 us without them, 19 with them).
  int chunk = max(share(), 1);  // 0 without a token in the batch
  const bool apart = p.B <= 32 && (4 * p.B * nv <= grid || (longest <= 2 * W && live <= grid));
  if (apart) {
    const int n = lane < p.B ? tiles_of(length_of(p, lane)) : 0;
    while (int(__reduce_add_sync(0xffffffffu, (n + chunk - 1) / chunk)) * nv > grid) chunk += max(W, chunk / 16);
    total = __reduce_add_sync(0xffffffffu, (n + chunk - 1) / chunk) * nv * chunk;
  } else {
    total += live * W;
    chunk = share();
    if (longest <= 2 * W) chunk = max(chunk, longest + W);
  }
  const int t0 = min(total, int(blockIdx.x) * chunk);
  int t1 = min(total, t0 + chunk);

  // Sequences without tokens: o = 0, lse = -inf.  Lengths that the table has no pages for are recorded.
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    if (tid == 0 && __ldg(p.cache_len + b) > p.width << p.log_ps) page::flag_bad_page(p.status, page::kSiteDecode4);
    if (length_of(p, b) == 0)
      for (int i = tid; i < p.Hq * (D / 8); i += C::THREADS) {
        reinterpret_cast<uint4*>(p.o)[(long long)b * p.Hq * (D / 8) + i] = make_uint4(0u, 0u, 0u, 0u);
        if (i < p.Hq) p.lse[(long long)b * p.Hq + i] = -INFINITY;
      }
  }
  if (t0 >= t1) return;

  int start = t0;  // the block's first tile
  Cursor item;     // the (sequence, head block) the block is at; j counts from the item's own start
  for (int b0 = 0, before = 0;; b0 += 32) {
    const int L = b0 + lane < p.B ? length_of(p, b0 + lane) : 0;
    const int nt = tiles_of(L);                         // own: places on the line, per head
    const int own = apart ? (nt + chunk - 1) / chunk * chunk : nt > 0 ? nt + W : 0;
    const int n = own * nv;
    int incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const unsigned past = __ballot_sync(0xffffffffu, before + incl > t0);
    if (past) {
      const int l = __ffs(past) - 1;
      const int off = t0 - before - __shfl_sync(0xffffffffu, incl - n, l);
      item.b = b0 + l;
      item.L = __shfl_sync(0xffffffffu, L, l);
      item.nt = tiles_of(item.L);
      const int each = __shfl_sync(0xffffffffu, own, l);
      item.vh = off / each;
      item.j = off % each;
      if (apart) t1 = min(t1, t0 + item.nt - item.j);
      if (item.j >= item.nt) {                           // behind the item's tiles: on to the next
        start += each - item.j;
        item.j = item.nt;
        if (start < t1) item.settle(p, nv);
      }
      break;
    }
    before += __shfl_sync(0xffffffffu, incl, 31);
  }

  if (start >= t1) return;

  // ---- this warp's copies: tiles start + warp, start + warp + W, ...; the W places behind an item
  // keep the warps' turns as they are
  uint8_t* ring = smem + C::OFF_RING + warp * C::NS * C::TILE_BYTES;
  const uint32_t ring_lane = smem_u32(ring) + lane * 16;
  const int upp_log = p.log_ps - 4;                     // units of a page
  const long long page_bytes = ((long long)p.Hkv << upp_log) * U::BYTES;
  Cursor next = item;
  next.j += warp;
  int t_next = start + warp;
  int pg[TU] = {};                                      // pages of the next tile's units
  auto fetch_pages = [&] {
    const int32_t* row = p.table + (long long)next.b * p.width;
#pragma unroll
    for (int i = 0; i < TU; ++i) {
      const int u = next.j * TU + i;
      if (u * page::kUnit < next.L) pg[i] = __ldg(row + (u >> upp_log));
    }
  };
  auto issue = [&](int st) {
    if (t_next < t1) {
      const int g = p.RB == 1 ? next.vh : next.vh / p.RB;
      const uint8_t* src[TU];
#pragma unroll
      for (int i = 0; i < TU; ++i) {
        if (pg[i] < 0 || pg[i] >= p.num_pages) {
          page::flag_bad_page(p.status, page::kSiteDecode4);
          pg[i] = 0;
        }
        const int u = (next.j * TU + i) & ((1 << upp_log) - 1);
        src[i] = p.pages + pg[i] * page_bytes + ((g << upp_log) + u) * U::BYTES;
      }
      const int units = min(TU, ((next.L + page::kUnit - 1) >> 4) - next.j * TU);
      constexpr int CH = U::BYTES / 16;                 // 16-byte pieces of a unit
      const uint32_t dst = ring_lane + st * C::TILE_BYTES;
#pragma unroll
      for (int k = 0; k < (TU * CH + 31) / 32; ++k) {
        const int ch = k * 32 + lane;
        const uint8_t* from = src[0] + ch * 16;
#pragma unroll
        for (int i = 1; i < TU; ++i)
          if (ch >= i * CH) from = src[i] + (ch - i * CH) * 16;
        if (ch < units * CH) copy16(dst + k * 512, from);
      }
      t_next += W;
      next.j += W;
      if (t_next < t1) {
        t_next += W * next.settle(p, nv);
        if (t_next < t1) fetch_pages();
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if (t_next < t1) {
    t_next += W * next.settle(p, nv);
    if (t_next < t1) fetch_pages();
  }
#pragma unroll
  for (int i = 0; i < C::NS; ++i) issue(i);

  // ---- tiles
  int st = 0;                  // ring stage of this warp's next tile
  int t = start, tw = start + warp;  // start of the item's part on the line; this warp's next tile
  const int key0 = token_of(r);
  while (t < t1) {
    const int e = min(t1, t + item.nt - item.j);         // end of the item's part
    const int L = item.L;
    const int g = p.RB == 1 ? item.vh : item.vh / p.RB;
    const int rb = item.vh - g * p.RB;
    const int h0 = g * p.G + rb * C::HEADS;              // first query head of the pass
    const int nh = min(C::HEADS, p.G - rb * C::HEADS);

    uint32_t qf[NG][4][NT][2];
    float qsum[NG][NT][2], up_h[NT][2];
    float ref[NT][2], l_run[NT][2], om[NG][NT][2];
    float oacc[NG][4][NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e2 = 0; e2 < 2; ++e2) {
        ref[nt][e2] = -INFINITY;
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

    if (tw < e) {
      // Queries of this warp's fragments: head nt * 8 + r, the elements of words 2c, 2c + 1.
      const __nv_bfloat16* qrow = p.q + ((long long)item.b * p.Hq + h0) * D;
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
              sum[gg] = fmaf(x[gg][i][k], 0x1p-7f, sum[gg]);   // 64 of any size stay in fp32
            }
          }
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
          big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
#pragma unroll
          for (int gg = 0; gg < NG; ++gg) sum[gg] += __shfl_xor_sync(0xffffffffu, sum[gg], o);
        }
        // down = 2^(13 - ex) brings the row's largest element into [2^13, 2^14); up = 2^ex.
        const int ex = min(max(int((__float_as_uint(big) >> 23) & 0xff) - 127, -114), 127);
        const float down = __uint_as_float(uint32_t(140 - ex) << 23);
        const float up = __uint_as_float(uint32_t(127 + ex) << 23);
#pragma unroll
        for (int gg = 0; gg < NG; ++gg)
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h)   // step 2i + h: elements 2h, 2h + 4 | 2h + 1, 2h + 5 of word i
#pragma unroll
              for (int k = 0; k < 2; ++k)  // k = 1: upper nibbles, 16 times too large
                qf[gg][2 * i + h][nt][k] =
                    pack_f16x2(x[gg][i][2 * h + k] * down * (k ? 0.0625f : 1.f),
                               x[gg][i][2 * h + k + 4] * down * (k ? 0.0625f : 1.f));
        // To the accumulator's layout: heads 2c and 2c + 1.  An accumulator holds
        // 2^(13 - ex - 24) times the sum of q code; 2^ex and the rest (with the exponential's
        // argument) come back one after the other, since their product can leave fp32 where the
        // score does not.
#pragma unroll
        for (int e2 = 0; e2 < 2; ++e2) {
          const int src = 4 * (2 * c + e2);
          up_h[nt][e2] = __shfl_sync(0xffffffffu, up, src) * p.up_scale;
          const float dn = __shfl_sync(0xffffffffu, down, src);
#pragma unroll
          for (int gg = 0; gg < NG; ++gg)
            qsum[gg][nt][e2] = __shfl_sync(0xffffffffu, sum[gg], src) * dn * 0x1p-17f;
        }
      }
    }

    for (bool first = true; tw < e; tw += W, first = false, st = st + 1 == C::NS ? 0 : st + 1) {
      asm volatile("cp.async.wait_group %0;" ::"n"(C::NS - 1) : "memory");
      __syncwarp();
      uint8_t* whole = ring + st * C::TILE_BYTES;
      const int have = L - (item.j + (tw - t)) * kTile;   // tokens from the tile's first on
      if (have < kTile) {
        // Behind the length lies anything: codes are harmless, scales are not.
        for (int i = have + lane; i < kTile; i += 32) {
          uint8_t* unit = whole + (i >> 4) * U::BYTES;
#pragma unroll
          for (int gg = 0; gg < NG; ++gg) {
            reinterpret_cast<uint32_t*>(unit + U::OFF_KS)[(i & 15) * NG + gg] = 0u;
            reinterpret_cast<uint32_t*>(unit + U::OFF_VS)[(i & 15) * NG + gg] = 0u;
          }
        }
        __syncwarp();
      }

#pragma unroll 1
      for (int part = 0; part < TU / TR; ++part) {
        const uint8_t* tile = whole + part * TR * U::BYTES;
        const int left = have - part * TR * page::kUnit;
        if (TR < TU && left <= 0) break;
        // scores over the rest of their scale, x: x scale_log2 is in units of log2
        float x[TR][NT][4];
#pragma unroll
        for (int u = 0; u < TR; ++u) {
          const uint8_t* unit = tile + u * U::BYTES;
          uint32_t w[2][2 * NG];   // [token half][NG * word + group]
          uint32_t sm[2][NG];
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const uint8_t* src = unit + U::OFF_KC + (key0 + 8 * hh) * U::CODE + c * 8 * NG;
            const uint8_t* ssrc = unit + U::OFF_KS + (key0 + 8 * hh) * U::SCALE;
            if constexpr (NG == 2) {
              const uint4 v = *reinterpret_cast<const uint4*>(src);
              w[hh][0] = v.x, w[hh][1] = v.y, w[hh][2] = v.z, w[hh][3] = v.w;
              const uint2 y = *reinterpret_cast<const uint2*>(ssrc);
              sm[hh][0] = y.x, sm[hh][1] = y.y;
            } else {
              const uint2 v = *reinterpret_cast<const uint2*>(src);
              w[hh][0] = v.x, w[hh][1] = v.y;
              sm[hh][0] = *reinterpret_cast<const uint32_t*>(ssrc);
            }
          }
          float sc[NT][4];
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
              const uint32_t y0 = x0 >> 8, y1 = x1 >> 8;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                mma_f16(acc[nt], x0 & kLowNibbles, x1 & kLowNibbles, x0 & kHighNibbles, x1 & kHighNibbles, qf[gg][2 * i][nt]);
                mma_f16(acc[nt], y0 & kLowNibbles, y1 & kLowNibbles, y0 & kHighNibbles, y1 & kHighNibbles, qf[gg][2 * i + 1][nt]);
              }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const float s = step_of(sm[k >> 1][gg]), m = low_of(sm[k >> 1][gg]);
                const float y = m * qsum[gg][nt][k & 1];
                sc[nt][k] = gg == 0 ? fmaf(s, acc[nt][k], y) : sc[nt][k] + fmaf(s, acc[nt][k], y);
              }
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 4; ++k) x[u][nt][k] = sc[nt][k] * up_h[nt][k & 1];
        }
        if (left < TR * page::kUnit) {
#pragma unroll
          for (int u = 0; u < TR; ++u)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (u * page::kUnit + key0 + 8 * (k >> 1) >= left) x[u][nt][k] = -INFINITY;
        }

        // weights p s in fp16; the reference moves when one reaches 2^14 (and on the first tile)
        uint32_t vs[TR][2][NG];
#pragma unroll
        for (int u = 0; u < TR; ++u)
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const uint8_t* ssrc = tile + u * U::BYTES + U::OFF_VS + (key0 + 8 * hh) * U::SCALE;
            if constexpr (NG == 2) {
              const uint2 y = *reinterpret_cast<const uint2*>(ssrc);
              vs[u][hh][0] = y.x, vs[u][hh][1] = y.y;
            } else {
              vs[u][hh][0] = *reinterpret_cast<const uint32_t*>(ssrc);
            }
          }
        uint32_t pw[TR][NG][NT][2];
        float pr[TR][NT][4];
        float big = 0.f;   // the largest minimum, in magnitude
#pragma unroll
        for (int u = 0; u < TR; ++u)
#pragma unroll
          for (int gg = 0; gg < NG; ++gg) big = fmax3(big, fabsf(low_of(vs[u][0][gg])), fabsf(low_of(vs[u][1][gg])));
        auto weigh = [&]() -> bool {
          uint32_t top = 0u;
          float top_p = 0.f;
#pragma unroll
          for (int u = 0; u < TR; ++u)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int hh = 0; hh < 2; ++hh) {
                const float p0 = ex2_approx(fmaf(x[u][nt][2 * hh], p.scale_log2, -ref[nt][0]));
                const float p1 = ex2_approx(fmaf(x[u][nt][2 * hh + 1], p.scale_log2, -ref[nt][1]));
                pr[u][nt][2 * hh] = p0;
                pr[u][nt][2 * hh + 1] = p1;
                top_p = fmax3(top_p, p0, p1);
#pragma unroll
                for (int gg = 0; gg < NG; ++gg) {
                  const float s = step_of(vs[u][hh][gg]);
                  pw[u][gg][nt][hh] = pack_f16x2(p0 * s, p1 * s);
                  top = max_f16x2(top, pw[u][gg][nt][hh]);
                }
              }
          return (top & 0xffffu) >= kTopWeight || (top >> 16) >= kTopWeight || top_p >= kTopP || big >= kTopMinimum;
        };
        bool move = first && part == 0;
        if (!move) move = __any_sync(0xffffffffu, weigh());
        if (move) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e2 = 0; e2 < 2; ++e2) {
              float y = -INFINITY;
#pragma unroll
              for (int u = 0; u < TR; ++u)
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                  float s = kSmallStep;
#pragma unroll
                  for (int gg = 0; gg < NG; ++gg)
                    s = fmax3(s, step_of(vs[u][hh][gg]), fabsf(low_of(vs[u][hh][gg])) * kMinimumShare);
                  y = fmaxf(y, fmaf(x[u][nt][2 * hh + e2], p.scale_log2, __log2f(s)));
                }
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, o));
              const float was = ref[nt][e2];
              y = fmaxf(was, y - kFirstWeight);
              const float alpha = first && part == 0 ? 0.f : ex2_approx(was - y);
              ref[nt][e2] = y == -INFINITY ? 0.f : y;
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
          weigh();
        }

        // sums and the second product
#pragma unroll
        for (int u = 0; u < TR; ++u) {
          const uint8_t* unit = tile + u * U::BYTES;
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
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 4; ++k) l_run[nt][k & 1] += pr[u][nt][k];
#pragma unroll
          for (int gg = 0; gg < NG; ++gg) {
            uint32_t pb[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int hh = 0; hh < 2; ++hh) {
                const float m = low_of(vs[u][hh][gg]);
                om[gg][nt][0] = fmaf(pr[u][nt][2 * hh], m, om[gg][nt][0]);
                om[gg][nt][1] = fmaf(pr[u][nt][2 * hh + 1], m, om[gg][nt][1]);
                pb[nt][hh] = transpose8x8(pw[u][gg][nt][hh]);
              }
            uint32_t a = __byte_perm(wv[0][gg], wv[1][gg], 0x5410), b = __byte_perm(wv[0][gg], wv[1][gg], 0x7632);
            uint32_t cc = __byte_perm(wv[2][gg], wv[3][gg], 0x5410), d = __byte_perm(wv[2][gg], wv[3][gg], 0x7632);
#pragma unroll
            for (int i = 0; i < 4; i += 2) {   // rows r: element i of the word; rows r + 8: element i + 4
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                mma_f16(oacc[gg][i][nt], a & kLowNibbles, b & kLowNibbles, cc & kLowNibbles, d & kLowNibbles, pb[nt]);
                mma_f16(oacc[gg][i + 1][nt], a & kHighNibbles, b & kHighNibbles, cc & kHighNibbles, d & kHighNibbles, pb[nt]);
              }
              a >>= 8, b >>= 8, cc >>= 8, d >>= 8;
            }
          }
        }
      }
      __syncwarp();  // every lane has read the stage
      issue(st);
    }

    // ---- join the warps' parts of this item: normalised outputs, log2 sums
    if (tw - t >= W) {   // of the warps that had a tile
      // Groups in doubt.  The groups share a reference, and a group whose steps are far below the
      // other's has its weights among fp16's subnormals, each wrong by up to 2^-25.  A group is in
      // doubt where any head's sum of p s code over a lane's 8 elements of it is so small that this
      // could make up 2^-10 of it, codes being 15 at most.
      unsigned few = 0u;
      if constexpr (NG > 1) {
        const float least = float((tw - t) / W * kTile) * (15.f * 8.f * 0x1p-15f * 0x1p-24f);
#pragma unroll
        for (int gg = 0; gg < NG; ++gg) {
          float low = INFINITY;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e2 = 0; e2 < 2; ++e2) {
              auto two = [&](int i) { return oacc[gg][i][nt][e2] + oacc[gg][i][nt][2 + e2]; };
              low = fminf(low, two(0) + two(2) + 0.0625f * (two(1) + two(3)));
            }
          few |= __all_sync(0xffffffffu, low >= least) ? 0u : 1u << gg;
        }
      }
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
            const float l = l_run[nt][e2];
            const float inv = l == 0.f ? 0.f : 1.f / l;
            if (r == 0) s_l[warp * C::HEADS + h] = l == 0.f ? -INFINITY : ref[nt][e2] + log2f(l);
#pragma unroll
            for (int gg = 0; gg < NG; ++gg) {
              const float add = om[gg][nt][e2] * inv;
              const float lo = inv * 16777216.f, hi = inv * 1048576.f;   // undo the subnormals' 2^-24, 2^-20
              float4* dst = reinterpret_cast<float4*>(s_o + (warp * C::HEADS + h) * D + gg * 64 + r * 8);
              dst[0] = make_float4(fmaf(oacc[gg][0][nt][e2], lo, add), fmaf(oacc[gg][1][nt][e2], hi, add),
                                   fmaf(oacc[gg][2][nt][e2], lo, add), fmaf(oacc[gg][3][nt][e2], hi, add));
              dst[1] = make_float4(fmaf(oacc[gg][0][nt][2 + e2], lo, add), fmaf(oacc[gg][1][nt][2 + e2], hi, add),
                                   fmaf(oacc[gg][2][nt][2 + e2], lo, add), fmaf(oacc[gg][3][nt][2 + e2], hi, add));
            }
          }
        }
      if constexpr (NG > 1) {
        if (__builtin_expect(few != 0u, 0)) {   // behind the tile loop in the code: 2% of the call
          __syncwarp();
          plain_tiles<D>(p, p.q + ((long long)item.b * p.Hq + h0) * D, p.table + (long long)item.b * p.width, g, nh,
                         item.j + (tw - t) % W, (tw - t) / W, W, L, few, s_o + warp * C::HEADS * D, s_l + warp * C::HEADS);
        }
      }
    }
    __syncthreads();
    const int a_line = t - item.j, e_line = a_line + item.nt;   // the whole item on the line
    const bool shared_item = a_line < t0 || e_line > t1;
    const int slot = 2 * blockIdx.x + (a_line < t0 ? 0 : 1);
    const long long row0 = (long long)item.b * p.Hq + h0;
    const int nw = min(W, e - t);                               // warps that had a tile
    const int w0 = (t - start) % W;                                // the first of them
    for (int i = tid; i < nh * (D / 4); i += W * 32) {
      const int h = i / (D / 4), d4 = i % (D / 4);
      float M = -INFINITY;
#pragma unroll 4
      for (int k = 0; k < nw; ++k) M = fmaxf(M, s_l[((w0 + k) % W) * C::HEADS + h]);
      const float Mz = M == -INFINITY ? 0.f : M;
      float l = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int k = 0; k < nw; ++k) {
        const int w = (w0 + k) % W;
        const float y = ex2_approx(s_l[w * C::HEADS + h] - Mz);
        const float4 v = reinterpret_cast<const float4*>(s_o)[(w * C::HEADS + h) * (D / 4) + d4];
        l += y;
        o.x = fmaf(y, v.x, o.x), o.y = fmaf(y, v.y, o.y), o.z = fmaf(y, v.z, o.z), o.w = fmaf(y, v.w, o.w);
      }
      const float inv = l == 0.f ? 0.f : 1.f / l;
      o.x *= inv, o.y *= inv, o.z *= inv, o.w *= inv;
      const float lse2 = l == 0.f ? -INFINITY : M + log2f(l);
      if (shared_item) {
        reinterpret_cast<float4*>(p.o_part)[((long long)slot * C::HEADS + h) * (D / 4) + d4] = o;
        if (d4 == 0) p.l_part[(long long)slot * C::HEADS + h] = lse2;
      } else {
        reinterpret_cast<uint2*>(p.o)[(row0 + h) * (D / 4) + d4] = make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
        if (d4 == 0) p.lse[row0 + h] = lse2 * 0.69314718055994530942f;
      }
    }
    if (shared_item) {
      const int c0 = a_line / chunk, c1 = (e_line - 1) / chunk;   // the blocks that share the item
      // A block's slot: its first, unless the item begins in its part.
      auto slot_of = [&](int k) { return 2 * k + (a_line < k * chunk ? 0 : 1); };
      __threadfence();
      __syncthreads();
      if (warp == 0) {
        volatile unsigned long long* fl = p.flags;
        if (lane == 0) fl[slot] = p.tag;
        __syncwarp();
        __threadfence();
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
        const int parts = c1 - c0 + 1;
        for (int h = warp; h < nh; h += W) {   // the parts' weights, a warp per head
          constexpr int K = kMaxParts / 32;
          float y[K], M = -INFINITY, l = 0.f;
#pragma unroll
          for (int i = 0; i < K; ++i) {
            const int k = lane + 32 * i;
            y[i] = k < parts ? __ldcg(p.l_part + (long long)slot_of(c0 + k) * C::HEADS + h) : -INFINITY;
            M = fmaxf(M, y[i]);
          }
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
          const float Mz = M == -INFINITY ? 0.f : M;
#pragma unroll
          for (int i = 0; i < K; ++i) {
            y[i] = ex2_approx(y[i] - Mz);
            l += y[i];
          }
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
          const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
          for (int i = 0; i < K; ++i)
            if (lane + 32 * i < parts) s_wt[(lane + 32 * i) * C::HEADS + h] = y[i] * inv;
          if (lane == 0) p.lse[row0 + h] = l == 0.f ? -INFINITY : (M + log2f(l)) * 0.69314718055994530942f;
        }
        __syncthreads();
        for (int i = tid; i < nh * (D / 4); i += C::THREADS) {   // columns of four elements
          const int h = i / (D / 4);
          const float4* src = reinterpret_cast<const float4*>(p.o_part) + i;
          float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 16
          for (int k = 0; k < parts; ++k) {
            const float y = s_wt[k * C::HEADS + h];
            const float4 v = __ldcg(src + (long long)slot_of(c0 + k) * (C::HEADS * (D / 4)));
            o.x = fmaf(y, v.x, o.x), o.y = fmaf(y, v.y, o.y), o.z = fmaf(y, v.z, o.z), o.w = fmaf(y, v.w, o.w);
          }
          reinterpret_cast<uint2*>(p.o)[row0 * (D / 4) + i] = make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
        }
      }
    }
    __syncthreads();  // the join's buffers are free again

    item.j += e - t;
    t = e;
    if (t < t1) {
      item.settle(p, nv);
      t += W;
      tw += W;
    }
  }
}

}  // namespace decode4
}  // namespace attn_sm100
