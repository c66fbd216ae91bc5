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

// Quantise a row pair, one warp: lane = 16 * isv + li holds dims 8 li .. 8 li + 7 of the K (lanes
// 0-15) or V row as bf16. Returns the lane's code word; `meta` is its group's word (the same in
// the group's 8 lanes). m is the group's least value (a bf16 input value, so stored exactly), s
// the bf16 next at or above (max - m) / 15, so that 15 s spans the group and every value is
// within s / 2 of what it reads back as. The codes are rint((x - m) / s), division and all
// roundings as IEEE fp32 has them. A group with an infinity or a NaN, or whose span overflows,
// reads back as NaN.
__device__ __forceinline__ uint32_t kv4_quantise(const uint4& v, int lane, uint32_t& meta) {
  float x[8];
  unpack8(v, x);
  float lo = x[0], hi = x[0], z = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lo = fminf(lo, x[i]);
    hi = fmaxf(hi, x[i]);
    z = fmaf(x[i], 0.f, z);  // NaN as soon as one value is not finite
  }
#pragma unroll
  for (int o = 1; o <= 4; o <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  const float span = hi - lo;
  const unsigned bad = __ballot_sync(0xffffffffu, z != 0.f || isinf(span));
  if ((bad >> (lane & 24)) & 0xffu) {
    meta = 0x7fc07fc0u;
    return 0u;
  }
  const uint32_t sbits = (__float_as_uint(__fdiv_rn(span, 15.f)) + 0xffffu) & 0xffff0000u;
  const float s = __uint_as_float(sbits);
  meta = (sbits >> 16) | (__float_as_uint(lo) & 0xffff0000u);
  uint32_t w = 0;
  if (s > 0.f) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      w |= (uint32_t)min(__float2int_rn(__fdiv_rn(x[i] - lo, s)), 15) << (4 * i);
  }
  return w;
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
