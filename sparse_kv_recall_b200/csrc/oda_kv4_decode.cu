// Decode attention over the 4-bit paged cache, under every visibility rule, split over the whole
// GPU and merged inside the same launch (the work plan of the bf16 split kernel: equal contiguous
// shares of the flattened (sequence, KV head, page) list, one online softmax per warp for all the
// query heads of the KV head, the last CTA to arrive merges).
//
// Bound: a visible (position, KV head) row is 144 bytes instead of 512, so HBM leaves a warp a
// third of the time per row; what competes with it is instruction issue, and within it the integer
// pipe (half rate), which unpacks the codes. So both products run on the tensor cores straight from
// codes, and scales and minima are applied to sums instead of to elements:
//
//   K:  s_p = sum_groups [ S_g sum_d c q_d + M_g sum_d q_d ]   (S, M of token p)
//       mma.sync m16n8k16 fp16, A = 16 tokens x codes, B = columns (head, group) that hold the head's q
//       in the dims of their group and zero elsewhere. q is scaled by a power of two to the top of the
//       fp16 range: its eight significant bits fit, so every dim within 2^-28 of the head's largest is
//       exact. The codes enter times 2^-14, exact too: scales and minima up to 2^117 leave fp32's range
//       only where the score does.
//   V:  o_d = sum_p (w_p S_g) (c - z_p) + sum_p w_p (M_g + z_p S_g)
//       A = codes as dims x 16 tokens, B = w_p S_g as a sum of two fp16 (columns (head, part): 22
//       bits); the second sum has one term per token and group and runs on the CUDA cores. The codes
//       are centred, z_p = 8 and 7 in turn (7.5 on average): over a long history an offset would grow
//       with the token count and the signal only with its square root. w S enters times a running power
//       of two per head and group, r: lowered when a product passes 2^15 (to below 2^8), and raised with
//       the softmax maximum by what the earlier weights lose.
//
// A code becomes an fp16 by an and-or that puts its nibble into the mantissa of 1024 and one exact
// fp16 add or fma that takes the offset off.
//
// Measured (one B200, calls replayed from a graph, bf16 or fp32 out; 8 KV heads): one sequence of 131,073 tokens, 16
// query heads, 151 MB, 36.0 us (4.2 TB/s; some 10 of them before the first and after the last page); eight of
// 16,385, 39.3 us; sixteen of 8K to 64K, 32 query heads, 721 MB, 148.2 us (4.9 TB/s, 75 % of a copy's rate), and
// 163 to 170 us (4.3 TB/s, 67 %) where calls follow one another for long enough that the power cap lowers the clock. Two
// query heads per KV head: 58 % of the issue slots and 47 % of DRAM; four: 66 % and 59 %. Eight warps of two CTAs
// an SM and two pages a step are what 128 registers a thread and the stages leave; nine to twelve warps spill.
#include <cuda_fp16.h>
#include <math.h>

#include "oda_decode.cuh"
#include "oda_kv4.cuh"

namespace oda {

constexpr int kW4 = 8;               // warps per CTA
constexpr int kThreads4 = kW4 * 32;
constexpr int kPages4 = 2;           // pages a step takes
constexpr int kStages4 = 2;          // steps a warp holds in shared memory: one in use, one coming
constexpr int kStageBytes4 = kPages4 * kKv4PageBytes;
constexpr int kRefs4 = 64;           // page references a warp holds (two halves, refilled in turn)
constexpr int kCtasPerSm4 = 2;
constexpr int kMinShare4 = 32;       // pages per CTA at least (two steps a warp)
constexpr float kMergeRoom = 10.f;   // partials are weighed by 2^-10 and less: there are fewer than 2^10
constexpr int kPStride = 48;         // words per (page, head) of the weight exchange
constexpr int kPWords = 2 * 4 * kPStride;

struct Kv4Params {
  PlanArgs plan;
  unsigned char* cache;
  int batch, hkv, hq;
  const __nv_bfloat16* q;
  const __nv_bfloat16* k_new;  // nullable: quantise into slot t and attend it there
  const __nv_bfloat16* v_new;
  float scale_log2;
  void* out;
  int out_bf16;
  float* lse;
  float* scores;               // [batch][hq][cap] base-2 scores of visible positions
  int cap;
  float* ws_o;
  float* ws_lse;
  unsigned int* ws_ticket;
  int* status;
  unsigned long long* stats;
};

__device__ __forceinline__ void mma_16816_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t h2_fma(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t h2_add(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// (x & mask) | bits in one instruction
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t mask, uint32_t bits) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(d) : "r"(x), "r"(mask), "r"(bits));
  return d;
}
__device__ __forceinline__ uint32_t h2_pack(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ float2 h2_unpack(uint32_t v) {
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

// The four nibbles of each half of w as fp16 pairs c - Z (Z = 8 or 7), times 2^-14 with kDown: even ones sit in
// bits 0-3, odd ones in bits 4-7 of each half of w or of w >> 8.
template <int Z, bool kDown = false>
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t (&a)[4]) {
  constexpr uint32_t kBase = 0x64006400u;                             // 1024
  const uint32_t w8 = w >> 8;
  if constexpr (kDown) {
    static_assert(Z == 8, "the constants are for 8");
    constexpr uint32_t kEven = 0x04000400u, kOdd = 0x00400040u;       // 2^-14, 2^-18
    constexpr uint32_t kEvenZ = 0xac08ac08u, kOddZ = 0x9c809c80u;     // - 1032 x 2^-14, - 72 x 2^-14
    a[0] = h2_fma(and_or(w, 0x000f000fu, kBase), kEven, kEvenZ);
    a[1] = h2_fma(and_or(w, 0x00f000f0u, kBase), kOdd, kOddZ);
    a[2] = h2_fma(and_or(w8, 0x000f000fu, kBase), kEven, kEvenZ);
    a[3] = h2_fma(and_or(w8, 0x00f000f0u, kBase), kOdd, kOddZ);
  } else {
    constexpr uint32_t kEven = Z == 8 ? 0xe408e408u : 0xe407e407u;    // - (1024 + Z)
    constexpr uint32_t kOdd = Z == 8 ? 0xd480d480u : 0xd470d470u;     // - (64 + Z), after / 16
    a[0] = h2_add(and_or(w, 0x000f000fu, kBase), kEven);
    a[1] = h2_fma(and_or(w, 0x00f000f0u, kBase), 0x2c002c00u, kOdd);
    a[2] = h2_add(and_or(w8, 0x000f000fu, kBase), kEven);
    a[3] = h2_fma(and_or(w8, 0x00f000f0u, kBase), 0x2c002c00u, kOdd);
  }
}

// Lane roles. gid = lane / 4, tig = lane % 4. A step takes two pages. The accumulator columns are
// (head, group), so lane tig holds both groups of head tig of tokens gid and gid + 8 and forms their
// scores by itself. With four heads per KV head it does so for both pages; with fewer the columns are
// held twice and tig / 2 picks the page (with one head, the second is idle). For P.V the lane holds
// dims 64 g + 8 gid .. + 7 of both groups of the same head.
template <int G>
struct Roles {
  static constexpr int kHeads = G == 4 ? 4 : 2;
  static constexpr int kMine = G == 4 ? 2 : 1;  // pages whose scores a lane holds
  __device__ static int head(int tig) { return tig & (kHeads - 1); }
  __device__ static int page(int tig) { return G == 4 ? 0 : (tig >> 1); }
};

struct Kv4State {
  float m, l;          // base-2 reference of the weights and this lane's part of the softmax sum
  float corr[2];       // this lane's part of sum w (M_g + z S_g)
  float r[2];          // w S_g enters the tensor cores times this power of two
  float acc[8][4];     // tile 4 g + j: dims 64 g + 8 gid + j (0, 1) and + j + 4 (2, 3); columns
};                     // 2 tig, 2 tig + 1 are the two parts of the head

constexpr int kRTop = 253;             // exponent field of r at its largest, 2^126
// A power of two by its exponent field, and the field of a number >= 0.
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((unsigned)e << 23); }
__device__ __forceinline__ int pow2_exp(float x) { return (int)(__float_as_uint(x) >> 23); }

constexpr float kNoMax = -3.4028234e38f;  // m before any visible score: below every other
constexpr float kRoom = 7.f;  // scores stay this far below m: a weight times a scale or a value, and the sum of some
                              // hundred of them, is inside fp32 for the largest bf16 values too

// The group's q as B fragments (scaled to q') and, for the lane's own head, 2^-14 sum q' of each group and the
// factor that undoes q's power of two. K step s takes nibbles 2 (s & 1), 2 (s & 1) + 1 and those four further up of
// word e = s / 2 of the lane's 16-byte code chunk, which is all group e & 1.
template <int G>
__device__ __forceinline__ void load_q4(const __nv_bfloat16* q, int lane, uint4 (&v)[4]) {
  const int gid = lane >> 2, tig = lane & 3;
  const int head = (gid >> 1) & (Roles<G>::kHeads - 1);
#pragma unroll
  for (int e = 0; e < 4; ++e)
    v[e] = head < G ? *reinterpret_cast<const uint4*>(q + head * kHeadDim + 64 * (e & 1) +
                                                      8 * (2 * tig + (e >> 1)))
                    : make_uint4(0u, 0u, 0u, 0u);
}
template <int G>
__device__ __forceinline__ float prepare_q4(const uint4 (&v)[4], int lane, uint32_t (&b)[8][2], float (&qs)[2]) {
  using R = Roles<G>;
  const int gid = lane >> 2, tig = lane & 3;
  const int grp = gid & 1;
  float x[4][8];
  float top = 0.f, sum[2] = {0.f, 0.f};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    unpack8(v[e], x[e]);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      top = fmaxf(top, fabsf(x[e][k]));
      sum[e & 1] += x[e][k];
    }
  }
#pragma unroll
  for (int o = 1; o <= 2; o <<= 1) {
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    sum[0] += __shfl_xor_sync(0xffffffffu, sum[0], o);
    sum[1] += __shfl_xor_sync(0xffffffffu, sum[1], o);
  }
  const uint32_t f = min(268u - min(__float_as_uint(top) >> 23, 254u), 253u);  // |q| below 2^15
  const float up = __uint_as_float(f << 23);
#pragma unroll
  for (int s = 0; s < 8; ++s) {
    const int e = s >> 1, j = 2 * (s & 1);
    const bool mine = (e & 1) == grp;
    b[s][0] = mine ? h2_pack(x[e][j] * up, x[e][j + 4] * up) : 0u;
    b[s][1] = mine ? h2_pack(x[e][j + 1] * up, x[e][j + 5] * up) : 0u;
  }
  const int src = 8 * R::head(tig);  // a lane whose column is the lane's head
  qs[0] = __shfl_sync(0xffffffffu, sum[0] * up, src) * 0x1p-14f;
  qs[1] = __shfl_sync(0xffffffffu, sum[1] * up, src) * 0x1p-14f;
  return pow2(254 - (int)__shfl_sync(0xffffffffu, f, src));
}

// The pages of a warp's share. pos: first position + visible rows - 1 (a page's first position is a
// multiple of 16); negative: nothing to attend (past the share's end, or a bad page, reported). src: what to copy
// (for such a page the cache's first, which nothing of counts).
struct PageRefs {
  const unsigned char* src[kRefs4];
  int pos[kRefs4];
};

// Visible rows among the 16 positions from `pos`.
__device__ __forceinline__ int rows_in_page(const SeqPlan& s, int pos) {
  const int lo = max(s.row_lo, pos), hi = min(s.row_hi, pos + kPage - 1);
  const int glo = max(lo, s.gap_lo), ghi = min(hi, s.gap_hi - 1);
  return max(0, hi - lo + 1) - max(0, ghi - glo + 1);
}

// What a CTA works on: pages j0 .. j1 - 1 of the list of (sequence b, KV head g), units x .. x_end - 1 of the
// flattened list; CTAs first .. first + contrib - 1 hold parts of this (b, g). In shared memory, filled in by
// one thread: every warp's registers are spoken for.
constexpr int kPlans4 = 32;  // plans of the first sequences, kept for the pieces
struct Piece {
  SeqPlan plan;
  int b, g, j0, j1, x_end, first, contrib;
};

// One step over the two pages at `stage` (of a page with a negative entry no scale or minimum is used;
// its codes are finite numbers whatever they are). kq undoes q's power of two and the codes' and carries the
// softmax scale in base 2; qs is 2^-14 sum q' of each group.
template <int G, bool kScores>
__device__ __forceinline__ void kv4_step(const unsigned char* stage, int2 entry, const Piece& piece,
                                         const uint32_t (&qb)[8][2], float kq, const float (&qs)[2],
                                         Kv4State& st, uint32_t* pw, float* scores, int cap, int lane) {
  using R = Roles<G>;
  constexpr int NM = R::kMine, HG = R::kHeads;
  const int gid = lane >> 2, tig = lane & 3;
  const int myhead = R::head(tig), mypage = R::page(tig);

  // ---- sums c[page] of 2^-14 c q': token gid groups 0, 1; token gid + 8 groups 0, 1 ----
  float c[2][4];
  const unsigned char* kbase = stage + gid * kKv4RowBytes + 16 * tig;
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    const uint4 wa = *reinterpret_cast<const uint4*>(kbase + n * kKv4PageBytes);
    const uint4 wb = *reinterpret_cast<const uint4*>(kbase + n * kKv4PageBytes + 8 * kKv4RowBytes);
    const uint32_t a[4] = {wa.x, wa.y, wa.z, wa.w}, b[4] = {wb.x, wb.y, wb.z, wb.w};
    // (the codes enter as 2^-14 (c - 8); 8 qs brings the 8 back, so c is 2^-14 sum c q')
    c[n][0] = c[n][2] = 8.f * qs[0];
    c[n][1] = c[n][3] = 8.f * qs[1];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      uint32_t ca[4], cb[4];
      codes_f16<8, true>(a[e], ca);
      codes_f16<8, true>(b[e], cb);
      mma_16816_f16(c[n], ca[0], cb[0], ca[1], cb[1], qb[2 * e][0], qb[2 * e][1]);
      mma_16816_f16(c[n], ca[2], cb[2], ca[3], cb[3], qb[2 * e + 1][0], qb[2 * e + 1][1]);
    }
  }

  // ---- this lane's scores x[page][token gid, gid + 8] and the V meta of those tokens ----
  const unsigned char* mbase = stage + mypage * kKv4PageBytes + kKv4MetaOff + gid * kKv4MetaBytes;
  float x[NM][2];
  uint32_t vm[NM][2][2];  // [page][token][group]
#pragma unroll
  for (int n = 0; n < NM; ++n)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 m = *reinterpret_cast<const uint4*>(mbase + n * kKv4PageBytes + 8 * i * kKv4MetaBytes);
      vm[n][i][0] = m.z;
      vm[n][i][1] = m.w;
      x[n][i] = 0.f;
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const float cc = (NM == 1 && mypage) ? c[1][2 * i + g] : c[n][2 * i + g];
        const uint32_t km = g ? m.y : m.x;
        x[n][i] = fmaf(kv4_scale(km), cc, g ? fmaf(kv4_min(km), qs[g], x[n][i]) : kv4_min(km) * qs[g]);
      }
      x[n][i] *= kq;  // (rounded here once: what follows are differences of equal numbers)
    }

  const bool whole = (entry.x & entry.y & 15) == 15 && (entry.x | entry.y) >= 0;
  if (!whole) {  // (uniform) some row of these pages is hidden or absent: nothing of it may count
#pragma unroll
    for (int n = 0; n < NM; ++n) {
      const int mine = (NM == 2 ? n : mypage) ? entry.y : entry.x;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (mine < 0 || !row_visible(piece.plan, (mine & ~15) + gid + 8 * i)) {
          x[n][i] = -INFINITY;
          vm[n][i][0] = vm[n][i][1] = 0u;
        }
    }
  }
  if constexpr (kScores) {
    if (myhead < G) {
#pragma unroll
      for (int n = 0; n < NM; ++n) {
        const int mine = (NM == 2 ? n : mypage) ? entry.y : entry.x;
        float* dst = scores + (size_t)myhead * cap + (mine & ~15) + gid;
#pragma unroll
        for (int i = 0; i < 2; ++i)  // (what hides a row is looked up again: a score may be -inf)
          if (whole || (mine >= 0 && row_visible(piece.plan, (mine & ~15) + gid + 8 * i))) dst[8 * i] = x[n][i];
      }
    }
  }

  // ---- online softmax; m is raised only when a score comes within kRoom of it, to kRoom + kLazyMax above ----
  auto over_head = [&](float v) {  // maximum over the lanes that hold the head
    if (NM == 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
    return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
  };
  float top = fmaxf(x[0][0], x[0][1]);
  if (NM == 2) top = fmaxf(top, fmaxf(x[NM - 1][0], x[NM - 1][1]));
  if (__any_sync(0xffffffffu, top > st.m - kRoom)) {
    const float mx = over_head(top);
    const float m = mx > st.m - kRoom ? mx + (kRoom + kLazyMax) : st.m;
    const float d = m - st.m, al = ex2_fast(-d);
    st.m = m;
    st.l *= al;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      st.corr[g] *= al;
      // What the weights so far lose, r gets back, to 2^126: it belongs to the weights that count now, and a
      // row with a large scale that has become negligible does not leave the others below the fp16 range.
      const float back = fminf(floorf(d), (float)(kRTop - pow2_exp(st.r[g])));
      const float left = ex2_fast(back - d);  // al times that power of two
      st.r[g] = pow2(pow2_exp(st.r[g]) + (int)back);
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) st.acc[4 * g + j][i] *= left;
    }
  }

  // ---- weights times the V scales ----
  const float z = (gid & 4) ? 7.f : 8.f;  // what P.V subtracts from this lane's tokens' codes
  float y[NM][2][2];                      // [page][group][token]
#pragma unroll
  for (int n = 0; n < NM; ++n)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float w = ex2_fast(x[n][i] - st.m);
      st.l += w;
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const float s = kv4_scale(vm[n][i][g]);
        st.corr[g] = fmaf(w, fmaf(z, s, kv4_min(vm[n][i][g])), st.corr[g]);
        y[n][g][i] = w * s;
      }
    }
  float ymax[2];
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    ymax[g] = fmaxf(y[0][g][0], y[0][g][1]);
    if (NM == 2) ymax[g] = fmaxf(ymax[g], fmaxf(y[NM - 1][g][0], y[NM - 1][g][1]));
  }
  if (__any_sync(0xffffffffu, fmaxf(ymax[0] * st.r[0], ymax[1] * st.r[1]) > 32768.f)) {
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const float ym = over_head(ymax[g]);
      const int was = pow2_exp(st.r[g]);  // the largest weight to [2^7, 2^8)
      const int e = ym * st.r[g] > 32768.f ? 261 - min(pow2_exp(ym), 254) : was;
      const float less = pow2(max(0, 127 + e - was));
      st.r[g] = pow2(e);
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) st.acc[4 * g + j][i] *= less;
    }
  }
  // as two fp16 each
#pragma unroll
  for (int n = 0; n < NM; ++n) {
    uint32_t hi[2], lo[2];
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const float w0 = y[n][g][0] * st.r[g], w1 = y[n][g][1] * st.r[g];
      hi[g] = h2_pack(w0, w1);
      const float2 f = h2_unpack(hi[g]);
      lo[g] = h2_pack(w0 - f.x, w1 - f.y);
    }
    *reinterpret_cast<uint4*>(pw + ((mypage + n) * HG + myhead) * kPStride + 4 * gid) =
        make_uint4(hi[0], hi[1], lo[0], lo[1]);
  }
  __syncwarp();

  // ---- P.V ----
  const int bh = (gid >> 1) & (HG - 1), col = gid & 1;
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    const uint32_t* src = pw + (n * HG + bh) * kPStride + 2 * col;
    const uint2 b0 = *reinterpret_cast<const uint2*>(src + 4 * tig);
    const uint2 b1 = *reinterpret_cast<const uint2*>(src + 4 * (tig + 4));
    const unsigned char* vs = stage + n * kKv4PageBytes + kKv4VOff + tig * kKv4RowBytes + 8 * gid;
    const uint2 w0 = *reinterpret_cast<const uint2*>(vs);
    const uint2 w1 = *reinterpret_cast<const uint2*>(vs + 8 * kKv4RowBytes);
    const uint2 w2 = *reinterpret_cast<const uint2*>(vs + 4 * kKv4RowBytes);
    const uint2 w3 = *reinterpret_cast<const uint2*>(vs + 12 * kKv4RowBytes);
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const uint32_t u0 = g ? w0.y : w0.x, u1 = g ? w1.y : w1.x;
      const uint32_t u2 = g ? w2.y : w2.x, u3 = g ? w3.y : w3.x;
      uint32_t a0[4], a1[4], a2[4], a3[4];
      codes_f16<8>(__byte_perm(u0, u1, 0x5410), a0);  // tokens tig, tig + 8
      codes_f16<8>(__byte_perm(u0, u1, 0x7632), a1);
      codes_f16<7>(__byte_perm(u2, u3, 0x5410), a2);  // tokens tig + 4, tig + 12
      codes_f16<7>(__byte_perm(u2, u3, 0x7632), a3);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        mma_16816_f16(st.acc[4 * g + j], a0[j], a1[j], a2[j], a3[j], g ? b0.y : b0.x, g ? b1.y : b1.x);
    }
  }
  __syncwarp();  // the stage and the exchange area may be written again
}

__device__ __forceinline__ void kv4_write(const Kv4Params& p, int b, int h, int dim, float o, float l2) {
  const size_t row = (size_t)b * p.hq + h;
  if (p.out_bf16)
    static_cast<__nv_bfloat16*>(p.out)[row * kHeadDim + dim] = __float2bfloat16_rn(o);
  else
    static_cast<float*>(p.out)[row * kHeadDim + dim] = o;
  if (p.lse != nullptr && dim == 0)
    p.lse[row] = l2 == -INFINITY ? -INFINITY : l2 * 0.69314718055994531f;
}

struct Kv4Smem {
  static constexpr int kPOff = kW4 * kStages4 * kStageBytes4;
  static constexpr int kRefOff = kPOff + kW4 * kPWords * 4;
  static constexpr int kPreOff = kRefOff + kW4 * (int)sizeof(PageRefs);
  static constexpr int kBytes = kPreOff + (kMaxBatch + 1) * 4;
};

// Copy a step's two pages into its stage: 288 16-byte pieces, nine a lane, as one group of copies.
// (One bulk copy a page costs a warp more instructions than these nine, since the engine's operands are
// uniform registers: a 128K history took 5 % longer.)
__device__ __forceinline__ void kv4_copy(uint32_t dst, const unsigned char* a, const unsigned char* b,
                                         int lane, uint64_t policy) {
  constexpr int kPieces = kKv4PageBytes / 16;
  static_assert(2 * kPieces == 9 * 32, "nine pieces a lane");
  const unsigned char* pa = a + 16 * lane;
  const unsigned char* pb = b + 16 * lane - kKv4PageBytes;  // piece 144 is the second page's first
  dst += 16 * lane;
#pragma unroll
  for (int k = 0; k < 9; ++k) {
    const unsigned char* src = k < 4 ? pa : k > 4 ? pb : lane < kPieces - 128 ? pa : pb;
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst + 512 * k),
                 "l"(src + 512 * k), "l"(policy)
                 : "memory");
  }
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// One warp: references of its pages n0 .. n0 + 31 (page n is entry n % 2 of pair n / 2; a CTA's pairs are
// strided over its warps). Returns this lane's visible rows + 256 x pages.
__device__ __forceinline__ int kv4_refs(const Kv4Params& p, const Piece& piece, PageRefs& refs, int n0, int warp,
                                        int lane) {
  const int n = n0 + lane;
  const int j = piece.j0 + ((n >> 1) * kW4 + warp) * 2 + (n & 1);
  int pos = -1, seen = 0;
  const unsigned char* src = p.cache;
  if (j < piece.j1) {
    const PageRef r = page_ref(p.plan, piece.plan, piece.b, j);
    if (r.err != 0) {
      report(p.status, r.err);
    } else {
      const int rows = rows_in_page(piece.plan, r.lp * kPage);
      if (rows > 0) pos = r.lp * kPage + rows - 1;
      src = p.cache + ((size_t)r.pb * p.hkv + piece.g) * kKv4PageBytes;
      seen = rows + 256;
    }
  }
  refs.pos[n % kRefs4] = pos;
  refs.src[n % kRefs4] = src;
  return seen;
}

// Called, not inlined: what a step needs rarely keeps its registers and code to itself (128K history 36.0 us
// either way, ragged 8K..64K batch 148.4, 148.8 inlined).
__device__ __noinline__ int kv4_refs_call(const Kv4Params& p, const Piece& piece, PageRefs& refs, int n0, int warp,
                                          int lane) {
  return kv4_refs(p, piece, refs, n0, warp, lane);
}

// One warp, a step that holds the page of slot t: the step's K/V, quantised, take the slot in the cache and
// in this copy. (Inlined or called, the Local call of one 4K sequence, sink 4 and window 256, takes 7.9 to 8.4 us.)
__device__ __forceinline__ void kv4_commit(const Kv4Params& p, const Piece& piece, const PageRefs& refs, int s,
                                        unsigned char* stage, int lane) {
#pragma unroll 1
  for (int i = 0; i < 2; ++i) {
    const int pos = refs.pos[(2 * s + i) % kRefs4];
    if (pos < 0 || pos / kPage != piece.plan.t / kPage) continue;
    const uint4 v = *reinterpret_cast<const uint4*>((lane < 16 ? p.k_new : p.v_new) +
                                                    ((size_t)piece.b * p.hkv + piece.g) * kHeadDim +
                                                    8 * (lane & 15));
    uint32_t meta;
    const uint32_t word = kv4_quantise(v, lane, meta);
    const int row = piece.plan.t % kPage;
    kv4_store_row(stage + i * kKv4PageBytes, row, word, meta, lane);
    kv4_store_row(const_cast<unsigned char*>(refs.src[(2 * s + i) % kRefs4]), row, word, meta, lane);
  }
  __syncwarp();
}

template <int G, bool kScores>
__global__ void __launch_bounds__(kThreads4, kCtasPerSm4)
    kv4_decode_kernel(const __grid_constant__ Kv4Params p) {
  using R = Roles<G>;
  constexpr int HG = R::kHeads;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int s_align, s_last;
  __shared__ unsigned long long s_rows, s_pages;
  __shared__ Piece piece;
  __shared__ SeqPlan plans[kPlans4];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gid = lane >> 2, tig = lane & 3;
  unsigned char* stages = smem + warp * kStages4 * kStageBytes4;
  uint32_t* pw = reinterpret_cast<uint32_t*>(smem + Kv4Smem::kPOff) + warp * kPWords;
  PageRefs& refs = reinterpret_cast<PageRefs*>(smem + Kv4Smem::kRefOff)[warp];
  int* pre = reinterpret_cast<int*>(smem + Kv4Smem::kPreOff);
  const int B = p.batch, Hkv = p.hkv;
  const int cta = blockIdx.x;

  griddep_launch_dependents();
  griddep_wait();
  // ---- prefix of visible units per sequence, shares, this CTA's first piece ----
  if (tid == 0) {
    s_rows = 0;
    s_pages = 0;
    pre[0] = 0;
  }
#pragma unroll 1
  for (int b = tid; b < B; b += kThreads4) {
    const SeqPlan sp = make_plan(p.plan, b);
    pre[b + 1] = sp.npages * Hkv;
    if (b < kPlans4) plans[b] = sp;
    if (cta == 0 && sp.err != 0) report(p.status, sp.err);
  }
  __syncthreads();
  if (warp == 0) {
    int carry = 0;
    unsigned vmin = 0xffffffffu, vmax = 0u, active = 0u;
#pragma unroll 1
    for (int base = 0; base < B; base += 32) {
      const int i = base + lane;
      int v = i < B ? pre[i + 1] : 0;
      const unsigned nz = v > 0 ? (unsigned)v : 0u;
      vmin = min(vmin, __reduce_min_sync(0xffffffffu, nz ? nz : 0xffffffffu));
      vmax = max(vmax, __reduce_max_sync(0xffffffffu, nz));
      active += __popc(__ballot_sync(0xffffffffu, nz != 0u));
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int n = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += n;
      }
      v += carry;
      if (i < B) pre[i + 1] = v;
      carry = __shfl_sync(0xffffffffu, v, 31);
    }
    if (lane == 0) s_align = (active > 0 && vmin == vmax) ? (int)active * Hkv : 0;
  }
  __syncthreads();

  // Equal contiguous shares; with equal page counts the CTA count is a multiple of the non-empty
  // (sequence, KV head) pairs, so that every share falls inside one of them.
  const int T = pre[B];
  int Pe = T > 0 ? min((int)gridDim.x, (T - 1) / kMinShare4 + 1) : 0;
  if (s_align > 0) {
    const int up = (Pe + s_align - 1) / s_align * s_align;
    if (up <= (int)gridDim.x) Pe = up;
    else if (Pe >= s_align) Pe -= Pe % s_align;
  }
  // CTA c's share is [c T / Pe, (c + 1) T / Pe)
  const int each = Pe > 0 ? T / Pe : 0, more = Pe > 0 ? T % Pe : 0;
  const int share_end = cta < Pe ? (cta + 1) * each + (cta + 1) * more / Pe : 0;
  int x = cta < Pe ? cta * each + cta * more / Pe : 0;

  // (Whatever a piece or a CTA does once is written at one place in these loops: at several, inlined, it made
  // the kernel 108 KB of code, much of whose first execution waited for the instruction cache.)
#pragma unroll 1
  while (x < share_end) {
    if (tid == 0) {
      int lo = 0, hi = B - 1;  // the last sequence that starts at or before unit x
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (pre[mid] <= x) lo = mid; else hi = mid - 1;
      }
      const int npg = (pre[lo + 1] - pre[lo]) / Hkv;
      piece.plan = lo < kPlans4 ? plans[lo] : make_plan(p.plan, lo);
      piece.b = lo;
      piece.g = (x - pre[lo]) / npg;
      const int seg0 = pre[lo] + piece.g * npg;
      piece.j0 = x - seg0;
      piece.x_end = min(share_end, seg0 + npg);
      piece.j1 = piece.j0 + (piece.x_end - x);
    }
    __syncthreads();
    const int b = piece.b, g = piece.g, bg = b * Hkv + g;
    const int pairs = (piece.j1 - piece.j0 + 1) / 2;  // of pages, strided over the warps
    const int steps = pairs > warp ? (pairs - warp + kW4 - 1) / kW4 : 0;
    unsigned rows_vis = 0, pages_read = 0;  // this lane's pages

    uint4 qv[4];
    load_q4<G>(p.q + ((size_t)b * p.hq + g * G) * kHeadDim, lane, qv);  // (in flight beside the page table)
    auto fill = [&](int n0) {
      const int seen = kv4_refs(p, piece, refs, n0, warp, lane);
      rows_vis += seen & 255;
      pages_read += seen >> 8;
    };
    auto issue = [&](int s) {  // one group of copies a step, empty past the last
      if (s < steps) {
        const ulonglong2 src = *reinterpret_cast<const ulonglong2*>(&refs.src[2 * s % kRefs4]);
        // (the policy made anew each time: held in two registers it costs 1 to 3 % of a long call)
        kv4_copy(smem_addr(stages) + (s & 1) * kStageBytes4, reinterpret_cast<const unsigned char*>(src.x),
                 reinterpret_cast<const unsigned char*>(src.y), lane, l2_evict_first_policy());
      }
      copies_commit();
    };
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {  // step 0 on its way before the other half of the references is looked up
      if (h == 0 || steps > 16) fill(32 * h);
      __syncwarp();
      issue(h);
    }
    if (warp == kW4 - 1 && lane == 0) {  // (the warp with the fewest steps; needed at the merge)
      piece.first = cta_of(x - piece.j0, T, Pe);
      piece.contrib = cta_of(x - piece.j0 + (pre[b + 1] - pre[b]) / Hkv - 1, T, Pe) - piece.first + 1;
    }

    uint32_t qb[8][2];
    float qs[2];
    const float kq = prepare_q4<G>(qv, lane, qb, qs) * 0x1p14f * p.scale_log2;
    float* scores = nullptr;
    if constexpr (kScores) scores = p.scores + ((size_t)b * p.hq + g * G) * p.cap;

    Kv4State st;
    st.m = kNoMax;
    st.l = 0.f;
    st.corr[0] = st.corr[1] = 0.f;
    st.r[0] = st.r[1] = pow2(kRTop);
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) st.acc[t][i] = 0.f;

#pragma unroll 1
    for (int s = 0; s < steps; ++s) {
      if (s > 0 && s % 16 == 0 && s + 16 < steps) {  // the half that was used up last
        const int seen = kv4_refs_call(p, piece, refs, 2 * s + 32, warp, lane);
        rows_vis += seen & 255;
        pages_read += seen >> 8;
      }
      unsigned char* stage = stages + (s & 1) * kStageBytes4;
      copies_wait<1>();  // this lane's pieces of step s have landed ...
      __syncwarp();      // ... and the other lanes'
      const int2 entry = *reinterpret_cast<const int2*>(&refs.pos[2 * s % kRefs4]);
      if (p.k_new != nullptr) {  // (a page without visible rows is negative and never t's)
        const int t = piece.plan.t;
        if (min((unsigned)(entry.x ^ t), (unsigned)(entry.y ^ t)) < kPage) kv4_commit(p, piece, refs, s, stage, lane);
      }
      kv4_step<G, kScores>(stage, entry, piece, qb, kq, qs, st, pw, scores, p.cap, lane);
      issue(s + 2);
    }
    copies_wait<0>();

    // ---- merge the CTA's warps ----
#pragma unroll
    for (int o = 4; o <= 16; o <<= 1) {
      st.l += __shfl_xor_sync(0xffffffffu, st.l, o);
      st.corr[0] += __shfl_xor_sync(0xffffffffu, st.corr[0], o);
      st.corr[1] += __shfl_xor_sync(0xffffffffu, st.corr[1], o);
    }
    if (R::kMine == 1) {
      st.l += __shfl_xor_sync(0xffffffffu, st.l, 2);
      st.corr[0] += __shfl_xor_sync(0xffffffffu, st.corr[0], 2);
      st.corr[1] += __shfl_xor_sync(0xffffffffu, st.corr[1], 2);
    }
    if (p.stats != nullptr) {
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) {
        rows_vis += __shfl_xor_sync(0xffffffffu, rows_vis, o);
        pages_read += __shfl_xor_sync(0xffffffffu, pages_read, o);
      }
      if (lane == 0 && (rows_vis | pages_read)) {
        atomicAdd(&s_rows, (unsigned long long)rows_vis);
        atomicAdd(&s_pages, (unsigned long long)pages_read);
      }
    }
    __syncthreads();  // every warp is done with its stages: reuse them as merge scratch
    if (p.stats != nullptr && tid == 0) {
      if (s_rows) atomicAdd(&p.stats[ODA_STAT_ROWS], s_rows);
      if (s_pages) atomicAdd(&p.stats[ODA_STAT_PAGES], s_pages);
      s_rows = 0;
      s_pages = 0;
    }
    float* Mw = reinterpret_cast<float*>(smem);  // [kW4][HG]
    float* Lw = Mw + kW4 * HG;                   // [kW4][HG]
    float* Aw = Lw + kW4 * HG;                   // [kW4][HG][128]
    if (gid == 0 && tig < HG) {
      Mw[warp * HG + R::head(tig)] = st.m == kNoMax && st.l == 0.f ? -INFINITY : st.m;  // (a NaN stays)
      Lw[warp * HG + R::head(tig)] = st.l;
    }
    {
      if (tig < HG) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float inv = pow2(254 - pow2_exp(st.r[i]));
          float o[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            o[j] = fmaf(st.acc[4 * i + j][0] + st.acc[4 * i + j][1], inv, st.corr[i]);
            o[j + 4] = fmaf(st.acc[4 * i + j][2] + st.acc[4 * i + j][3], inv, st.corr[i]);
          }
          float4* dst = reinterpret_cast<float4*>(Aw + (warp * HG + tig) * kHeadDim + 64 * i + 8 * gid);
          dst[0] = make_float4(o[0], o[1], o[2], o[3]);
          dst[1] = make_float4(o[4], o[5], o[6], o[7]);
        }
      }
    }
    __syncthreads();
    const int n_contrib = piece.contrib;
    const size_t slot = (size_t)cta + bg;
#pragma unroll 1
    for (int e = tid; e < G * kHeadDim; e += kThreads4) {
      const int h = e / kHeadDim, dim = e % kHeadDim;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kW4; ++w) M = fmaxf(M, Mw[w * HG + h]);
      float o = 0.f, l2 = -INFINITY;
      if (M != -INFINITY) {
        float L = 0.f, a = 0.f;
#pragma unroll
        for (int w = 0; w < kW4; ++w) {
          const float ms = Mw[w * HG + h];
          const float f = ms == -INFINITY ? 0.f : ex2_fast(ms - M);
          L = fmaf(f, Lw[w * HG + h], L);
          a = fmaf(f, Aw[(w * HG + h) * kHeadDim + dim], a);
        }
        o = a / L;
        l2 = M + log2f(L);
      }
      if (n_contrib == 1) {
        kv4_write(p, b, g * G + h, dim, o, l2);
      } else {
        p.ws_o[(slot * G + h) * kHeadDim + dim] = o;
        if (dim == 0) p.ws_lse[slot * G + h] = l2;
      }
    }
    if (n_contrib > 1) {
      __syncthreads();  // the CTA's partial is written; thread 0 publishes it (release)
      if (tid == 0) s_last = ticket_arrive(&p.ws_ticket[piece.first]) == (unsigned)(n_contrib - 1);
      __syncthreads();  // ... and the last CTA's thread 0 acquired everyone's partials
      if (s_last) {
        // The partials come into shared memory by asynchronous copies, as many at a time as the stages
        // hold (all of a short call's at once), the first ones beside the log-sums.
        const size_t s0 = (size_t)piece.first + bg;
        float* sw = reinterpret_cast<float*>(smem);      // [n_contrib][G] log-sums, then weights
        float* so = sw + (n_contrib * G + 3) / 4 * 4;    // [chunk][G][128]
        const int chunk = (kW4 * kStages4 * kStageBytes4 / 4 - (n_contrib * G + 3)) / (G * kHeadDim);
        auto bring = [&](int first) {
          const int n = min(chunk, n_contrib - first) * G * kHeadDim / 4;
          const float* src = p.ws_o + (s0 + first) * G * kHeadDim;
#pragma unroll 4
          for (int i = tid; i < n; i += kThreads4) cp_async16(so + 4 * i, src + 4 * i);
        };
        bring(0);
#pragma unroll 1
        for (int i = tid; i < n_contrib * G; i += kThreads4) sw[i] = __ldcg(&p.ws_lse[s0 * G + i]);
        __shared__ float s_max[4], s_sum[4];
        __syncthreads();
        if (warp < G) {
          float m = -INFINITY, sum = 0.f;
          bool any = false;  // some log-sum is not -inf: a number, or a NaN, which a maximum passes over
#pragma unroll 1
          for (int s = lane; s < n_contrib; s += 32) {
            m = fmaxf(m, sw[s * G + warp]);
            any |= sw[s * G + warp] != -INFINITY;
          }
#pragma unroll
          for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
          if (__any_sync(0xffffffffu, any) && m == -INFINITY) m = 0.f;  // (NaNs alone: the weights are NaN)
          m += kMergeRoom;  // (the sum over the partials stays below the largest of them)
#pragma unroll 1
          for (int s = lane; s < n_contrib; s += 32) {
            const float ls = sw[s * G + warp];
            const float w = ls == -INFINITY ? 0.f : ex2_fast(ls - m);
            sw[s * G + warp] = w;
            sum += w;
          }
#pragma unroll
          for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
          if (lane == 0) {
            s_max[warp] = m;
            s_sum[warp] = sum;
          }
        }
        constexpr int kMine = (G * kHeadDim + kThreads4 - 1) / kThreads4;
        float a[kMine] = {};
#pragma unroll 1
        for (int first = 0; first < n_contrib; first += chunk) {
          if (first > 0) {
            __syncthreads();  // everyone is done with the chunk before
            bring(first);
          }
          cp_async_wait_all();
          __syncthreads();
          const int n = min(chunk, n_contrib - first);
#pragma unroll
          for (int k = 0; k < kMine; ++k) {
            const int e = tid + k * kThreads4;
            if (e < G * kHeadDim)
#pragma unroll 4
              for (int s = 0; s < n; ++s)
                a[k] = fmaf(sw[(first + s) * G + e / kHeadDim], so[s * G * kHeadDim + e], a[k]);
          }
        }
#pragma unroll
        for (int k = 0; k < kMine; ++k) {
          const int e = tid + k * kThreads4, h = e / kHeadDim;
          if (e >= G * kHeadDim) break;
          const bool none = s_max[h] == -INFINITY;
          kv4_write(p, b, g * G + h, e % kHeadDim, none ? 0.f : a[k] / s_sum[h],
                    none ? -INFINITY : s_max[h] + log2f(s_sum[h]));
        }
        if (tid == 0) p.ws_ticket[piece.first] = 0u;  // leave the tickets zeroed
      }
    }
    x = piece.x_end;
    __syncthreads();  // merge scratch is the next piece's stage memory, `piece` the next piece
  }

  // Sequences with nothing visible (bad length, empty keep list) but not gated off.
#pragma unroll 1
  for (int i = cta; i < B * Hkv; i += gridDim.x) {
    const int b = i / Hkv;
    if (pre[b + 1] == pre[b] && !(p.plan.gate != nullptr && p.plan.gate[b] == 0))
#pragma unroll 1
      for (int e = tid; e < G * kHeadDim; e += kThreads4)
        kv4_write(p, b, (i % Hkv) * G + e / kHeadDim, e % kHeadDim, 0.f, -INFINITY);
  }
}

// ---------------------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------------------
static size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// Tickets, then partials and their log-sums. A ticket belongs to the CTA a shared (sequence, KV head) begins in
// (only the last one that begins in a CTA reaches past it): as many as CTAs and in front, so that they lie in
// the same place for every batch and head count and one workspace serves calls of any.
struct Kv4Ws {
  size_t o_off, lse_off, total;
};

static Kv4Ws kv4_ws(int batch, int hkv, int G, int sms) {
  const size_t slots = (size_t)sms * kCtasPerSm4 + (size_t)batch * hkv;
  Kv4Ws w;
  w.o_off = up256((size_t)sms * kCtasPerSm4 * sizeof(unsigned));
  w.lse_off = w.o_off + up256(slots * G * kHeadDim * sizeof(float));
  w.total = w.lse_off + up256(slots * G * sizeof(float));
  return w;
}

int kv4_decode_ws_bytes(int batch, int hkv, int hq, size_t* bytes) {
  if (bytes == nullptr || batch < 0 || hkv < 1 || hq < 1) return ODA_ERR_INVALID_ARG;
  const int G = hq / hkv;
  if (hq % hkv != 0 || (G != 1 && G != 2 && G != 4)) return ODA_ERR_UNSUPPORTED_SHAPE;
  DeviceInfo di;
  const int rc = current_device_info(&di);
  if (rc != ODA_OK) return rc;
  *bytes = kv4_ws(batch, hkv, G, di.sms).total;
  return ODA_OK;
}

template <int G, bool kScores>
static int launch_kv4(const Kv4Params& p, const DeviceInfo& di, cudaStream_t st) {
  static bool done[64] = {false};
  if (di.device < 0 || di.device >= 64) return ODA_ERR_CUDA;
  if (!done[di.device]) {
    const cudaError_t e = cudaFuncSetAttribute(
        kv4_decode_kernel<G, kScores>, cudaFuncAttributeMaxDynamicSharedMemorySize, Kv4Smem::kBytes);
    if (e != cudaSuccess) return cuda_status(e);
    done[di.device] = true;
  }
  return cuda_status(launch_dependent(kv4_decode_kernel<G, kScores>, di.sms * kCtasPerSm4, kThreads4,
                                      Kv4Smem::kBytes, st, p));
}

int launch_kv4_decode(const oda_kv4* kv, const oda_visibility* vis, const void* q, int hq,
                      float scale, const void* k_new, const void* v_new, void* out, int out_dtype,
                      float* lse, float* scores, int cap, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_kv4(kv);
  if (rc != ODA_OK) return rc;
  const oda_kv k = kv4_as_kv(kv);
  if ((rc = check_visibility(&k, vis)) != ODA_OK) return rc;
  size_t need = 0;
  if ((rc = check_decode_args(&k, *vis, q, hq, scale, k_new, v_new, out, out_dtype, lse, ws)) != ODA_OK)
    return rc;
  if (kv->batch == 0) return ODA_OK;
  if ((rc = kv4_decode_ws_bytes(kv->batch, kv->num_kv_heads, hq, &need)) != ODA_OK) return rc;
  if (ws_bytes < need) return ODA_ERR_WORKSPACE_TOO_SMALL;
  DeviceInfo di;
  if ((rc = current_device_info(&di)) != ODA_OK) return rc;
  const int G = hq / kv->num_kv_heads;
  const Kv4Ws wl = kv4_ws(kv->batch, kv->num_kv_heads, G, di.sms);
  Kv4Params p;
  p.plan = plan_args(&k, *vis);
  p.cache = static_cast<unsigned char*>(kv->cache);
  p.batch = kv->batch;
  p.hkv = kv->num_kv_heads;
  p.hq = hq;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k_new = static_cast<const __nv_bfloat16*>(k_new);
  p.v_new = static_cast<const __nv_bfloat16*>(v_new);
  p.scale_log2 = scale * 1.4426950408889634f;
  p.out = out;
  p.out_bf16 = out_dtype == ODA_BF16;
  p.lse = lse;
  p.scores = scores;
  p.cap = cap;
  unsigned char* w = static_cast<unsigned char*>(ws);
  p.ws_o = reinterpret_cast<float*>(w + wl.o_off);
  p.ws_lse = reinterpret_cast<float*>(w + wl.lse_off);
  p.ws_ticket = reinterpret_cast<unsigned*>(w);
  p.status = kv->dev_status;
  p.stats = kv->stats;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (scores != nullptr) {
    switch (G) {
      case 1: return launch_kv4<1, true>(p, di, st);
      case 2: return launch_kv4<2, true>(p, di, st);
      default: return launch_kv4<4, true>(p, di, st);
    }
  }
  switch (G) {
    case 1: return launch_kv4<1, false>(p, di, st);
    case 2: return launch_kv4<2, false>(p, di, st);
    default: return launch_kv4<4, false>(p, di, st);
  }
}

}  // namespace oda

using namespace oda;

extern "C" int oda_kv4_decode_workspace_size(int32_t batch, int32_t num_kv_heads,
                                             int32_t num_q_heads, size_t* bytes) {
  return kv4_decode_ws_bytes(batch, num_kv_heads, num_q_heads, bytes);
}

extern "C" int oda_kv4_decode(const oda_kv4* kv, const oda_visibility* vis, const void* q,
                              int32_t num_q_heads, float scale, const void* k_new,
                              const void* v_new, void* out, int32_t out_dtype, float* lse, void* ws,
                              size_t ws_bytes, void* stream) {
  return launch_kv4_decode(kv, vis, q, num_q_heads, scale, k_new, v_new, out, out_dtype, lse, nullptr,
                           0, ws, ws_bytes, stream);
}
