// The 4-bit KV page and the row quantiser shared by the kernels that write and read it.
//
// One (page, KV head) is one contiguous run of 2304 bytes, so that a decode warp brings it in
// with a single bulk copy: K codes [16 tokens][64 B], V codes [16][64 B], meta [16][4 words].
// A row's 128 dims are two groups of 64, each with its own scale s and minimum m; a code c in
// 0..15 stands for m + c s. Word 2 i + g of a row's 16 words holds dims 64 g + 8 i .. + 7 of
// group g in its nibbles, lowest first; the meta words of a token are (K g0, K g1, V g0, V g1),
// each the bf16 scale in the low half and the bf16 minimum in the high half.
#pragma once

#include "oda_common.cuh"

namespace oda {

constexpr int kKv4RowBytes = kHeadDim / 2;                   // one row's codes: 64 B
constexpr int kKv4VOff = kPage * kKv4RowBytes;               // V codes after the K codes
constexpr int kKv4MetaOff = 2 * kPage * kKv4RowBytes;        // meta after the codes
constexpr int kKv4MetaBytes = 16;                            // per token
constexpr int kKv4PageBytes = kKv4MetaOff + kPage * kKv4MetaBytes;
static_assert(kKv4PageBytes == ODA_KV4_PAGE_BYTES, "page size of the public header");

__device__ __forceinline__ float kv4_scale(uint32_t meta) { return bf16lo(meta); }
__device__ __forceinline__ float kv4_min(uint32_t meta) { return bf16hi(meta); }

// Word of a row that holds dims 8 li .. 8 li + 7 (li < 16).
__device__ __forceinline__ int kv4_word(int li) { return li < 8 ? 2 * li : 2 * (li - 8) + 1; }

__device__ __forceinline__ uint32_t bf2_max_nan(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Packed fp32 pairs (each lane rounded as the scalar instruction would).
__device__ __forceinline__ float2 f2_add(float2 a, float2 b) {
  float2 d;
  asm("{.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 f2_mul2(float2 a, float2 b) {
  float2 d;
  asm("{.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 f2_fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mov.b64 w, {%6, %7};\n\tfma.rn.f32x2 z, x, y, w;\n\tmov.b64 {%0, %1}, z;}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}

// The whole number nearest to a / s, halves to even, from a neighbour c of the quotient's.
__device__ __forceinline__ float kv4_half(float a, float s, float c) {
  const float e = fmaf(-c, s, a), twice = 2.f * fabsf(e);  // the remainder, exact
  const bool odd = (static_cast<int>(c) & 1) != 0;
  const float step = e > 0.f ? 1.f : -1.f;
  return twice > s || (twice == s && odd) ? c + step : c;
}

// Quantise a row pair, one warp: lane = 16 * isv + li holds dims 8 li .. 8 li + 7 of the K (lanes
// 0-15) or V row as bf16. Returns the lane's code word; `meta` is its group's word (the same in
// the group's 8 lanes). m is the group's least value (a bf16 input value, so stored exactly), s
// the bf16 next at or above (max - m) / 15, so that 15 s spans the group and every value is
// within s / 2 of what it reads back as. The codes are rint((x - m) / s), halves to even, division and
// all roundings as IEEE fp32 has them. They come from the product with the reciprocal, which is within
// 4e-6 of the quotient; where that is as close to a half, twice the remainder is compared with s. That
// decides as the division would: (k + 1/2) s has 13 bits, and a difference x - m that is not equal to it
// is off by more than half an ulp of the quotient. A group with an infinity or a NaN, or whose span
// overflows, reads back as NaN.
__device__ __forceinline__ uint32_t kv4_quantise(const uint4& v, int lane, uint32_t& meta) {
  // the group's (max, -min) as a bf16 pair, NaN if any value is one
  constexpr uint32_t kSigns = 0x80008000u;
  const uint32_t hi = bf2_max_nan(bf2_max_nan(v.x, v.y), bf2_max_nan(v.z, v.w));
  const uint32_t lo = bf2_max_nan(bf2_max_nan(v.x ^ kSigns, v.y ^ kSigns),
                                  bf2_max_nan(v.z ^ kSigns, v.w ^ kSigns));
  uint32_t ends = bf2_max_nan(__byte_perm(hi, lo, 0x5410), __byte_perm(hi, lo, 0x7632));
#pragma unroll
  for (int o = 1; o <= 4; o <<= 1) ends = bf2_max_nan(ends, __shfl_xor_sync(0xffffffffu, ends, o));
  const float m = -bf16hi(ends), span = bf16lo(ends) - m;
  const uint32_t sbits = (__float_as_uint(__fdiv_rn(span, 15.f)) + 0xffffu) & 0xffff0000u;
  meta = (sbits >> 16) | __float_as_uint(m);
  if (!(span <= 3.4028234e38f)) meta = 0x7fc07fc0u;
  const float s = __uint_as_float(sbits);
  if (!(s > 0.f) || meta == 0x7fc07fc0u) return 0u;  // a constant group: every code 0
  const float inv = __frcp_rn(s);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  constexpr float kRound = 12582912.f;  // 1.5 x 2^23: adding it leaves the nearest whole number
  float2 c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = f2_add(make_float2(bf16lo(w[i]), bf16hi(w[i])), make_float2(-m, -m));
    const float2 t = f2_mul2(a, make_float2(inv, inv));
    c[i] = f2_add(f2_add(t, make_float2(kRound, kRound)), make_float2(-kRound, -kRound));
    const float2 d = f2_add(t, make_float2(-c[i].x, -c[i].y));
    // (a subnormal scale has no finite reciprocal: neither product's distance is then a number)
    if (!(fmaxf(fabsf(d.x), fabsf(d.y)) < 0.49999f)) {
      if (inv <= 3.4028234e38f) {
        c[i].x = kv4_half(a.x, s, c[i].x);
        c[i].y = kv4_half(a.y, s, c[i].y);
      } else {
        c[i].x = rintf(__fdiv_rn(a.x, s));
        c[i].y = rintf(__fdiv_rn(a.y, s));
      }
    }
  }
  // codes to nibbles: sums of whole numbers below 2^16, then below the exponent of 2^23
  const float2 k16 = make_float2(256.f, 256.f);
  const float2 p = f2_fma2(c[1], k16, c[0]), q = f2_fma2(c[3], k16, c[2]);  // c0 + 256 c2, c1 + 256 c3
  const float x0 = fmaf(p.y, 16.f, p.x) + 8388608.f, x1 = fmaf(q.y, 16.f, q.x) + 8388608.f;
  return __byte_perm(__float_as_uint(x0), __float_as_uint(x1), 0x5410);
}

// Store a quantised row pair (lane layout of kv4_quantise) as token `row` of the page at
// `page`, which may be in global or in shared memory.
__device__ __forceinline__ void kv4_store_row(unsigned char* page, int row, uint32_t word,
                                              uint32_t meta, int lane) {
  const int li = lane & 15, isv = lane >> 4;
  *reinterpret_cast<uint32_t*>(page + isv * kKv4VOff + row * kKv4RowBytes + 4 * kv4_word(li)) = word;
  if ((lane & 7) == 0)
    *reinterpret_cast<uint32_t*>(page + kKv4MetaOff + row * kKv4MetaBytes + 4 * (lane >> 3)) = meta;
}

}  // namespace oda
