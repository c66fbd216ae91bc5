// The 4-bit KV page and the row quantiser shared by the kernels that write and read it.
//
// One (page, KV head) is one contiguous run of 2304 bytes, 144 16-byte pieces, so that a decode warp brings
// two of them in with nine copies a lane: K codes [16 tokens][64 B], V codes [16][64 B], meta [16][4 words].
// A row's 128 dims are two groups of 64, each with its own scale s and minimum m; a code c in
// 0..15 stands for m + c s. Word 2 i + g of a row's 16 words holds dims 64 g + 8 i .. + 7 of
// group g in its nibbles, lowest first; the meta words of a token are (K g0, K g1, V g0, V g1),
// each the bf16 scale in the low half and the bf16 minimum in the high half.
#pragma once

#include "oda_common.cuh"

namespace oda {

constexpr int kKv4Group = ODA_KV4_GROUP;                      // dims of a scale and minimum
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

__device__ __forceinline__ uint32_t bf2_min_nan(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
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

// Quantising. m is the group's least value (a bf16 input value, so stored exactly), s the bf16 next at or
// above (max - m) / 15, so that 15 s spans the group and every value is within s / 2 of what it reads back
// as. The codes are rint((x - m) / s), halves to even, division and all roundings as IEEE fp32 has them. A
// group with an infinity or a NaN, or whose span overflows, reads back as NaN.

// (max, -min) of eight values as a bf16 pair, NaN if any value is one.
__device__ __forceinline__ uint32_t kv4_ends(const uint4& v) {
  const uint32_t hi = bf2_max_nan(bf2_max_nan(v.x, v.y), bf2_max_nan(v.z, v.w));
  const uint32_t lo = bf2_min_nan(bf2_min_nan(v.x, v.y), bf2_min_nan(v.z, v.w)) ^ 0x80008000u;
  return bf2_max_nan(__byte_perm(hi, lo, 0x5410), __byte_perm(hi, lo, 0x7632));
}

struct Kv4Group {
  float m, s;  // s = 0: every code is 0 (a constant group, or one that reads back as NaN)
  float inv;   // of s; infinite: divide
  uint32_t meta;
};

// From the group's ends. The scale needs no division: 15 s has 12 bits, and a span one fp32 above 15 s has a
// quotient more than half an ulp above s, so s is the least bf16 with 15 s >= span; a product with slightly
// less than 1/15 finds it or the one below. (Spans so small that a remainder could round are divided.)
__device__ __forceinline__ Kv4Group kv4_group(uint32_t ends) {
  constexpr float kSmall = 7.9e-31f;  // 2^-100
  Kv4Group g;
  g.m = -bf16hi(ends);
  const float span = bf16lo(ends) - g.m;
  uint32_t sbits = (__float_as_uint(span * 0.06666665f) + 0xffffu) & 0xffff0000u;
  if (15.f * __uint_as_float(sbits) < span) sbits += 0x10000u;
  if (span < kSmall) sbits = (__float_as_uint(__fdiv_rn(span, 15.f)) + 0xffffu) & 0xffff0000u;
  g.meta = (sbits >> 16) | __float_as_uint(g.m);
  if (!(span <= 3.4028234e38f)) {
    g.meta = 0x7fc07fc0u;
    sbits = 0u;
  }
  g.s = __uint_as_float(sbits);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(g.inv) : "f"(g.s));  // within 2^-23
  if (sbits == 0u) g.inv = 0.f;
  else if (span < kSmall) g.inv = INFINITY;
  return g;
}

// Eight values' code word. The quotient is the product with the reciprocal and one correction by its remainder
// (exact, in one fma): within 2^-40 of a step of rounding the true one. That rounds to the code as the IEEE
// quotient does: (k + 1/2) s has 13 bits; a difference x - m equal to it gives k + 1/2 exactly, and any other
// is off by at least 1/256 more than half an ulp of the quotient.
__device__ __forceinline__ uint32_t kv4_codes(const uint4& v, const Kv4Group& g) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  constexpr float kRound = 12582912.f;  // 1.5 x 2^23: adding it leaves the nearest whole number in the low bits
  uint32_t word = 0u;
  if (g.inv <= 3.4028234e38f) {
#pragma unroll
    for (int i = 3; i >= 0; --i) {
      const float2 a = f2_add(make_float2(bf16lo(w[i]), bf16hi(w[i])), make_float2(-g.m, -g.m));
      const float2 inv = make_float2(g.inv, g.inv);
      const float2 t = f2_mul2(a, inv);
      const float2 e = f2_fma2(t, make_float2(-g.s, -g.s), a);
      const float2 c = f2_add(f2_fma2(e, inv, t), make_float2(kRound, kRound));
      word = (word << 4) + __float_as_uint(c.y);
      word = (word << 4) + __float_as_uint(c.x);
    }
    // (kRound's own bits, 0x4b400000 in each of the eight sums, add up to this)
    word -= 0x3f400000u;
  } else {
#pragma unroll 1
    for (int i = 7; i >= 0; --i) {
      const uint32_t x = i < 2 ? w[0] : i < 4 ? w[1] : i < 6 ? w[2] : w[3];
      const float a = ((i & 1) ? bf16hi(x) : bf16lo(x)) - g.m;
      word = (word << 4) + (uint32_t)rintf(__fdiv_rn(a, g.s));
    }
  }
  return g.s > 0.f ? word : 0u;
}

// Quantise a row pair, one warp: lane = 16 * isv + li holds dims 8 li .. 8 li + 7 of the K (lanes
// 0-15) or V row as bf16. Returns the lane's code word; `meta` is its group's word (the same in
// the group's 8 lanes).
__device__ __forceinline__ uint32_t kv4_quantise(const uint4& v, int lane, uint32_t& meta) {
  uint32_t ends = kv4_ends(v);
#pragma unroll
  for (int o = 1; o <= 4; o <<= 1) ends = bf2_max_nan(ends, __shfl_xor_sync(0xffffffffu, ends, o));
  const Kv4Group g = kv4_group(ends);
  meta = g.meta;
  return kv4_codes(v, g);
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
