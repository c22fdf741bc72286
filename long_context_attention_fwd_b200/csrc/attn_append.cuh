// attn_append.cuh -- writing a paged key/value cache, and reading a 4-bit one back.
//
// append_kernel takes the new tokens' q, k and v (strided rows of one projection's output, as a
// rule), turns the first 2 * half elements of q and k by their position's angles,
//     a' = a cos - b sin,   b' = b cos + a sin      (fp32, one rounding to bf16),
// with (a, b) = (x[j], x[j + half]) or, interleaved, (x[2j], x[2j + 1]), and writes k and v where
// the page table says: as bf16, or as 4-bit codes with a step and a minimum per 64 elements,
//     m = min x,  s = bf16((max x - m) / 15),  code = rint((x - m) / s) in 0..15,
// of the bf16 values x.  The quotient of the fp32 difference a = x - m is rounded as in exact
// arithmetic: a product with 1 / s gives a candidate, and the remainder a - code s, which fp32 holds
// exactly, corrects it.
// (IEEE divisions, 16 a thread, took the 4-bit append three times as long as the bf16 one.)
// A group with a NaN or an infinity, or whose range leaves fp32, gets s = m = NaN and reads back
// as NaN.
//
// Bound by HBM: every input element is read once and every output written once.  D / 16 threads
// hold a row in two 16-byte chunks, chosen so that rotation partners meet in one thread, and a
// thread's angles serve every head of the token.  A warp takes a token, or a share of its rows
// where there are fewer tokens than warps to fill the SMs; it has kAhead rows' loads in flight,
// and the first of them do not wait for the page table.  (A block per token: 152 us for 32K
// tokens of 28 + 2 x 4 heads where a warp per token takes 98, 94% of the copy
// rate.)  The 4-bit form waits for its loads (4.6 TB/s) and for issue (68%), neither of them full: a
// pass's codes follow its own loads (16 prompt chunks of up to 4K tokens and their read-back: 173 us,
// 75%).
#pragma once
#include <cuda_bf16.h>

#include "attn_page.cuh"

namespace attn_sm100 {
namespace append {

constexpr int kThreads = 256;
constexpr int kAhead = 2;  // rows a thread has in flight

struct Params {
  page::PageMap map;
  const __nv_bfloat16* q;   // nullptr: no queries
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  long long q_stride, k_stride, v_stride;  // elements from one token to the next
  const float* cos;         // [rope_len][half]; unused when half = 0
  const float* sin;
  int rope_len, half, interleaved;
  int nq, Hkv;              // query heads written (0 without q), kv heads
  int share_log;            // 2^share_log warps share a token
  __nv_bfloat16* q_out;     // [T][nq][D]
  __nv_bfloat16* k_pages;   // bf16 pages
  __nv_bfloat16* v_pages;
  uint8_t* pages;           // 4-bit pages
  unsigned* status;
};

struct Chunk {
  float x[8];
};

__device__ __forceinline__ Chunk unpack(const uint4 u) {
  Chunk c;
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c.x[2 * i] = __uint_as_float(w[i] << 16);
    c.x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
  return c;
}

__device__ __forceinline__ uint4 pack(const Chunk& c) {
  return make_uint4(pack_bf16x2(c.x[0], c.x[1]), pack_bf16x2(c.x[2], c.x[3]),
                    pack_bf16x2(c.x[4], c.x[5]), pack_bf16x2(c.x[6], c.x[7]));
}

// Products and sums are rounded one by one (no contraction), as a framework's elementwise
// operations round them.
__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
  const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  a = x;
}

__device__ __forceinline__ float min_nan(float a, float b) {
  float d;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// Eight codes of one word: round((x - m) / s), ties to even, in 0..15.
__device__ __forceinline__ uint32_t encode(const Chunk& c, float m, float s) {
  uint32_t w = 0;
  if (s < 1e-36f) {  // 1 / s may leave fp32; s = 0: equal elements, or a group that is not finite
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float t = s > 0.f ? rintf(__fdiv_rn(__fsub_rn(c.x[j], m), s)) : 0.f;
      w |= uint32_t(fminf(t, 15.f)) << (4 * j);
    }
    return w;
  }
  // The fma rounds a / s to a whole number in the low bits of its result.  1 / s is off by 2^-24,
  // so it errs only where a / s is within 2^-20 of a half; there the remainder decides.  No
  // clamp: a <= 15 s (1 + 2^-8).
  const float inv = __frcp_rn(s), half = 0.5f * s;
  constexpr float kWhole = 8388608.f;  // 2^23
  float t[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float a = __fsub_rn(c.x[j], m);        // >= 0: m is the group's minimum
    const float z = fmaf(a, inv, kWhole);
    t[j] = z - kWhole;
    const float rem = fmaf(-t[j], s, a);         // exact: t s has 12 bits, and a is near it
    if (fabsf(rem) >= half && (fabsf(rem) > half || (__float_as_uint(z) & 1u))) t[j] += rem > 0.f ? 1.f : -1.f;
  }
  const float lo = fmaf(4096.f, t[3], fmaf(256.f, t[2], fmaf(16.f, t[1], t[0]))) + kWhole;
  const float hi = fmaf(4096.f, t[7], fmaf(256.f, t[6], fmaf(16.f, t[5], t[4]))) + kWhole;
  return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x5410);
}

template <int D, bool KV4>
__global__ void __launch_bounds__(kThreads, 4) append_kernel(const Params p) {
  constexpr int TPR = D / 16;            // threads of a row
  constexpr int RPP = 32 / TPR;          // rows of a warp's pass
  const int lane = threadIdx.x & 31;
  const int tr = lane % TPR;
  const int rows = p.nq + 2 * p.Hkv;     // a token's rows: q heads, k heads, v heads
  const int hc = p.half / 8;
  const bool turned = tr < hc;
  const int ca = turned ? (p.interleaved ? 2 * tr : tr) : 2 * tr;
  const int cb = turned && !p.interleaved ? tr + hc : ca + 1;

  auto load = [&](int t, int row, uint4 (&u)[2]) {
    const __nv_bfloat16* src;
    if (row < p.nq) src = p.q + t * p.q_stride + row * D;
    else if (row < p.nq + p.Hkv) src = p.k + t * p.k_stride + (row - p.nq) * D;
    else src = p.v + t * p.v_stride + (row - p.nq - p.Hkv) * D;
    u[0] = reinterpret_cast<const uint4*>(src)[ca];  // plain loads: q_out may be q
    u[1] = reinterpret_cast<const uint4*>(src)[cb];
  };

  const long long items = (long long)p.map.T << p.share_log;
  const long long nwarp = (long long)gridDim.x * (kThreads / 32);
  const int stride = RPP << p.share_log;  // rows from one pass to the next
  for (long long item = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); item < items; item += nwarp) {
    const int t = int(item >> p.share_log);
    const int first = (int(item) & ((1 << p.share_log) - 1)) * RPP;   // the warp's first row
    const int r0 = first + lane / TPR;
    if (first >= rows) continue;
    uint4 u[kAhead][2];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (r0 + i * stride < rows) load(t, r0 + i * stride, u[i]);

    int pos, pg, slot;
    page::Placed st = page::place_token(p.map, t, pos, pg, slot);
    if (st == page::kFound && p.half > 0 && pos >= p.rope_len) st = page::kBad;
    if (st == page::kBad && lane == 0) page::flag_bad_page(p.status, page::kSiteAppend);
    if (st != page::kFound) continue;  // the same in every lane

    float c[8], s[8];
    if (turned) {
      // chunk tr's and its partner's angles; interleaved, a chunk of 8 elements has 4 angles
      const long long at = (long long)pos * p.half + 8 * tr;
      *reinterpret_cast<float4*>(c) = __ldg(reinterpret_cast<const float4*>(p.cos + at));
      *reinterpret_cast<float4*>(c + 4) = __ldg(reinterpret_cast<const float4*>(p.cos + at) + 1);
      *reinterpret_cast<float4*>(s) = __ldg(reinterpret_cast<const float4*>(p.sin + at));
      *reinterpret_cast<float4*>(s + 4) = __ldg(reinterpret_cast<const float4*>(p.sin + at) + 1);
    }

    for (int base = 0; first + base < rows; base += kAhead * stride) {
      if (base > 0) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
          if (r0 + base + i * stride < rows) load(t, r0 + base + i * stride, u[i]);
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int row = base + i * stride + r0;
        const bool live = row < rows;
        if (!__any_sync(0xffffffffu, live)) continue;
        if (live && turned && row < p.nq + p.Hkv) {
          Chunk a = unpack(u[i][0]), b = unpack(u[i][1]);
          if (p.interleaved) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              turn(a.x[2 * j], a.x[2 * j + 1], c[j], s[j]);
              turn(b.x[2 * j], b.x[2 * j + 1], c[4 + j], s[4 + j]);
            }
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) turn(a.x[j], b.x[j], c[j], s[j]);
          }
          u[i][0] = pack(a);
          u[i][1] = pack(b);
        }
        if (live && row < p.nq) {
          uint4* dst = reinterpret_cast<uint4*>(p.q_out + ((long long)t * p.nq + row) * D);
          dst[ca] = u[i][0];
          dst[cb] = u[i][1];
        }
        const int hv = row - p.nq;                // kv row: K heads, then V heads
        const bool is_v = hv >= p.Hkv;
        const int h = is_v ? hv - p.Hkv : hv;
        if constexpr (!KV4) {
          if (live && hv >= 0) {
            const long long tok = ((long long)pg << p.map.log_ps) + slot;
            uint4* dst = reinterpret_cast<uint4*>((is_v ? p.v_pages : p.k_pages) + (tok * p.Hkv + h) * D);
            dst[ca] = u[i][0];
            dst[cb] = u[i][1];
          }
        } else {
          using U = page::Unit<D>;
          if (!__any_sync(0xffffffffu, live && hv >= 0)) continue;
          // Minimum and maximum of each group over the row's threads.
          const Chunk a = unpack(u[i][0]), b = unpack(u[i][1]);
          const int ga = ca / 8, gb = cb / 8;
          float lo[U::NG], hi[U::NG];
          float la = a.x[0], ha = a.x[0], lb = b.x[0], hb = b.x[0];
#pragma unroll
          for (int j = 1; j < 8; ++j) {
            la = min_nan(la, a.x[j]), ha = max_nan(ha, a.x[j]);
            lb = min_nan(lb, b.x[j]), hb = max_nan(hb, b.x[j]);
          }
          if constexpr (U::NG == 1) {
            lo[0] = min_nan(la, lb), hi[0] = max_nan(ha, hb);
          } else {
            const bool one = ga == gb;               // both chunks in one group
            const float l = one ? min_nan(la, lb) : la, h2 = one ? max_nan(ha, hb) : ha;
            lo[0] = ga == 0 ? l : INFINITY, hi[0] = ga == 0 ? h2 : -INFINITY;
            lo[1] = ga == 1 ? l : one ? INFINITY : lb, hi[1] = ga == 1 ? h2 : one ? -INFINITY : hb;
          }
#pragma unroll
          for (int g = 0; g < U::NG; ++g)
#pragma unroll
            for (int o = 1; o < TPR; o <<= 1) {
              lo[g] = min_nan(lo[g], __shfl_xor_sync(0xffffffffu, lo[g], o));
              hi[g] = max_nan(hi[g], __shfl_xor_sync(0xffffffffu, hi[g], o));
            }
          uint32_t sm[U::NG];
          float step[U::NG];
#pragma unroll
          for (int g = 0; g < U::NG; ++g) {
            const __nv_bfloat16 sb = __float2bfloat16_rn(__fdiv_rn(__fsub_rn(hi[g], lo[g]), 15.f));
            step[g] = __bfloat162float(sb);
            if (step[g] < INFINITY) {
              sm[g] = uint32_t(__bfloat16_as_ushort(sb)) | __float_as_uint(lo[g] + 0.f);  // -0 becomes +0
            } else {
              step[g] = 0.f;
              sm[g] = 0x7FC07FC0u;
            }
          }
          if (live && hv >= 0) {
            const float ma = (U::NG == 2 && ga) ? lo[U::NG - 1] : lo[0];
            const float mb = (U::NG == 2 && gb) ? lo[U::NG - 1] : lo[0];
            const float sa = (U::NG == 2 && ga) ? step[U::NG - 1] : step[0];
            const float sb = (U::NG == 2 && gb) ? step[U::NG - 1] : step[0];
            const int upp_log = p.map.log_ps - 4;
            uint8_t* unit = p.pages + ((((long long)pg * p.Hkv + h) << upp_log) + (slot >> 4)) * U::BYTES;
            const int j = slot & 15;
            uint32_t* code = reinterpret_cast<uint32_t*>(unit + (is_v ? U::OFF_VC : U::OFF_KC) + j * U::CODE);
            const uint32_t wa = encode(a, ma, sa), wb = encode(b, mb, sb);
            if (U::NG == 2 && cb == ca + 8) {   // the same word of both groups: neighbours
              *reinterpret_cast<uint2*>(code + 2 * ca) = make_uint2(wa, wb);
            } else {
              code[U::NG * (ca & 7) + ga] = wa;
              code[U::NG * (cb & 7) + gb] = wb;
            }
            if (tr == 0) {
              uint32_t* sc = reinterpret_cast<uint32_t*>(unit + (is_v ? U::OFF_VS : U::OFF_KS) + j * U::SCALE);
#pragma unroll
              for (int g = 0; g < U::NG; ++g) sc[g] = sm[g];
            }
          }
        }
      }
    }
  }
}

// gather4_kernel: packed token t's K and V out of 4-bit pages, x = s * code + m in fp32 (the
// product is exact: 8 bits by 4), rounded once to bf16.  A warp takes a token, or a share of its
// rows where tokens are few; eight threads
// hold a row, each the word (or the two words of both groups) of eight elements, so that reads
// and writes are whole sectors.  Bound by HBM, by the bf16 rows it writes: four bytes of five
// (8 x 16-32K tokens, 4 heads: 487 MB in 92 us; a plain fill writes 3.9 TB/s).  With one row a lane
// in flight 32 registers let all 64 warps of an SM in; three rows and 40 took 101 us.
struct GatherParams {
  page::PageMap map;
  const uint8_t* pages;
  int Hkv, share_log;  // 2^share_log warps share a token
  __nv_bfloat16* k;  // [T][Hkv][D]
  __nv_bfloat16* v;
  unsigned* status;
};

// The eight elements of a word.  A code under the exponent of 2^(23 - 4 j) is 2^(23 - 4 j) + code,
// which needs neither a shift nor a conversion for the first five (the case above 92.3 -> 91.4 us,
// short ones as they were).
__device__ __forceinline__ uint4 decode_word(uint32_t w, uint32_t sm) {
  const float s = __uint_as_float(sm << 16), m = __uint_as_float(sm & 0xffff0000u);
  const uint32_t w2 = w >> 20;
  Chunk c;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int at = j < 5 ? j : j - 5;
    const uint32_t one = uint32_t(127 + 23 - 4 * at) << 23;
    const float code = __uint_as_float(((j < 5 ? w : w2) & (15u << (4 * at))) | one) - __uint_as_float(one);
    c.x[j] = fmaf(s, code, m);
  }
  return pack(c);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 8) gather4_kernel(const GatherParams p) {
  using U = page::Unit<D>;
  const long long nwarp = (long long)gridDim.x * (kThreads / 32);
  const long long items = (long long)p.map.T << p.share_log;
  const int lane = threadIdx.x & 31;
  const int i = lane & 7;                      // words i of each group
  const int rows = 2 * p.Hkv;
  for (long long item = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); item < items; item += nwarp) {
    const int t = int(item >> p.share_log);
    const int first = 4 * (int(item) & ((1 << p.share_log) - 1));
    int pos, pg, slot;
    const page::Placed st = page::place_token(p.map, t, pos, pg, slot);
    if (st == page::kOutside) continue;
    if (st == page::kBad && lane == 0) page::flag_bad_page(p.status, page::kSiteGather);
    for (int row = first + (lane >> 3); row < rows; row += 4 << p.share_log) {
      const bool is_v = row >= p.Hkv;
      const int h = is_v ? row - p.Hkv : row;
      uint4* dst = reinterpret_cast<uint4*>((is_v ? p.v : p.k) + ((long long)t * p.Hkv + h) * D) + i;
      uint2 w = make_uint2(0u, 0u), sc = make_uint2(0u, 0u);   // without a place: zeros
      if (st == page::kFound) {
        const uint8_t* unit =
            p.pages + ((((long long)pg * p.Hkv + h) << (p.map.log_ps - 4)) + (slot >> 4)) * U::BYTES;
        const int j = slot & 15;
        const uint8_t* code = unit + (is_v ? U::OFF_VC : U::OFF_KC) + j * U::CODE + 4 * U::NG * i;
        const uint8_t* scale = unit + (is_v ? U::OFF_VS : U::OFF_KS) + j * U::SCALE;
        if constexpr (U::NG == 2) {
          w = *reinterpret_cast<const uint2*>(code);
          sc = *reinterpret_cast<const uint2*>(scale);
        } else {
          w.x = *reinterpret_cast<const uint32_t*>(code);
          sc.x = *reinterpret_cast<const uint32_t*>(scale);
        }
      }
      dst[0] = decode_word(w.x, sc.x);
      if constexpr (U::NG == 2) dst[8] = decode_word(w.y, sc.y);
    }
  }
}

}  // namespace append
}  // namespace attn_sm100
