// Eviction from the paged cache by accumulated attention weight: of a (sequence, KV head)'s slots
// the first `sink`, the last `recent` and the rest's heaviest are kept, `budget` in all, in ascending
// slot order (the Local rule takes "recent" from the slot order), and move to the destination pages,
// which may be the source's own.
//
// (A launch runs most of this code once, so loops of few trips are not unrolled: the instruction cache is cold.)
//
// One thread-block cluster takes one (sequence, KV head). The threshold weight is found by a radix select
// over order-preserving 32-bit keys, eight bits a pass from the highest bit in which any two keys differ,
// until few keys are left that are compared with one another; every later decision follows from it and from
// counts, so the result does not depend on any order of execution. Up to kAlone slots every CTA of the
// cluster selects by itself, from all the keys, and moves its share of the rows: a pass is then two CTA
// barriers, where histograms summed through distributed shared memory cost a cluster barrier and a remote
// read (2304 slots, budget 2048, one sequence of 8 KV heads: 23.1 us with shared histograms, 13.0 so).
// Longer sequences are shared out over the cluster.
//
// Bound: memory for the rows -- a kept row is read and written once (512 bytes in bf16, 144 in 4 bits), a
// weight is read a few times, mostly out of L2 or shared memory -- and before them, not overlapped, the
// selection's chain of barriers and scans. Four sequences of 20K to 32K cut down to 4096 (135 MB of bf16 rows):
// 44.5 us, of which the move takes 19, at the rate of a copy, and the selection 20; 16 sequences of 1.5K to
// 8K in 4 bits down to 2049: 34.9 us, 13 of them the move. (Fetching the recent rows, which move in any case,
// into L2 beside the selection: 48.5 us for the former.) In place, with a barrier before each round's stores:
// 50.3, 36.7, and 13.7 for the 2304 slots.
//
// In place, a move must not overwrite a row that has not been read. The i-th kept slot p_i is >= i,
// so when the rows of a round, a run [i0, i1) of the kept list, are all in registers before the
// first of them is stored, nothing a later round reads is lost: its sources are >= i1.
#include <math.h>

#include "oda_common.cuh"
#include "oda_internal.h"
#include "oda_kv4.cuh"

namespace oda {

constexpr int kEvictThreads = 512;
constexpr int kEvictWarps = kEvictThreads / 32;
constexpr int kPieces = 8;  // 16-byte pieces a thread moves per round
static_assert(kEvictThreads == 512, "threads 0-255 take a digit each, 256-511 clear the other histogram");

struct EvictParams {
  unsigned char* k_cache;  // 4-bit: the codes; v_cache unused
  unsigned char* v_cache;
  const int32_t* block_table;
  const int32_t* seq_lens;
  int hkv, max_blocks, num_blocks;
  const float* mass;
  float* mass_out;
  long long mass_tokens;
  int sink, recent, budget;
  const int32_t* gate;
  const int32_t* dst_table;
  int dst_blocks;
  int32_t* kept;
  int32_t* lens_out;
  unsigned* ticket;   // [batch], used with lens_alias
  int in_place;       // the destination is the source: order loads before stores
  int lens_alias;     // lens_out is seq_lens
  int* status;
};

// 16-byte pieces of a row pair, and where piece i of KV head g's row `at` (page * 16 + row in it) lies.
struct Bf16Rows {
  static constexpr int kCount = 32;
  __device__ static unsigned char* at(const EvictParams& p, unsigned at, int g, int i) {
    const size_t off = (((size_t)(at / kPage) * p.hkv + g) * kPage + at % kPage) * kRowBytes;
    return (i < 16 ? p.k_cache : p.v_cache) + off + 16 * (i & 15);
  }
};
struct Kv4Rows {
  static constexpr int kCount = 9;
  __device__ static unsigned char* at(const EvictParams& p, unsigned at, int g, int i) {
    const unsigned row = at % kPage;
    unsigned char* page = p.k_cache + ((size_t)(at / kPage) * p.hkv + g) * kKv4PageBytes;
    const unsigned off = i == 8 ? kKv4MetaOff + row * kKv4MetaBytes
                                : (i >> 2) * kKv4VOff + row * kKv4RowBytes + 16 * (i & 3);
    return page + off;
  }
};

__device__ __forceinline__ unsigned dsmem_ld_u32(const unsigned* local, unsigned rank) {
  return __float_as_uint(dsmem_ld(reinterpret_cast<const float*>(local), rank));
}

// Ascending order of floats as unsigned integers; -0 counts as 0, a NaN above everything.
__device__ __forceinline__ unsigned mass_key(float m) {
  if (isnan(m)) return 0xffffffffu;
  const unsigned u = __float_as_uint(m + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// The least of every lane's lo and the greatest of every lane's hi.
__device__ __forceinline__ void warp_range(unsigned& lo, unsigned& hi) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
}

__device__ __forceinline__ unsigned warp_scan(unsigned v, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

constexpr int kKeyCache = 8192;  // keys held in shared memory (a CTA's share of more is read again)
// Slots up to which each CTA of a cluster selects by itself. Sequences of n slots cut down to n / 2, 8 KV heads, us
// alone / shared:
//   n                             1100         2304         3600         4090         5000         6000         8000
//   bf16, 1 sequence, 16 CTAs   9.8 / 14.0  13.2 / 23.1  16.3 / 23.5  16.9 / 23.6  22.7 / 27.6  25.4 / 28.3  29.5 / 29.0
//   bf16, 4 sequences, 8       12.3 / 18.8  24.5 / 23.7  24.6 / 25.8  24.4 / 27.1  34.9 / 30.9  33.8 / 32.8  42.9 / 38.9
//   bf16, 16 sequences, 2      21.6 / 25.1  37.7 / 40.1  56.0 / 56.4  61.0 / 61.1  74.0 / 72.8  87.0 / 85.3   113 / 109
//   4 bits, 1 sequence, 16     10.5 / 14.8  14.5 / 23.6  17.5 / 23.9  18.1 / 23.8  20.1 / 24.2  22.0 / 24.3  25.6 / 24.6
//   4 bits, 4 sequences, 8     15.8 / 19.1  16.4 / 19.4  20.6 / 20.7  19.6 / 21.0  21.9 / 22.4  24.1 / 23.2  43.2 / 28.0
//   4 bits, 16 sequences, 2    14.5 / 17.5  21.2 / 23.3  27.6 / 28.2  31.4 / 31.8  36.6 / 36.0  43.5 / 42.3  55.6 / 53.6
// (Where 16 CTAs share one sequence's head, alone is faster up to about 7000.)
constexpr int kAlone = 4096;

constexpr int kFew = 128;     // keys that are compared with one another directly, by four threads each
constexpr int kAhead = 6;     // weights a thread has in flight (2304 slots: 13.3 us with 4 or 6, 13.9 with 8;
                              // 8K in 4 bits, 16 sequences: 38.1 with 4, 37.7 with 6, 37.1 with 8)
static_assert(kFew * 4 == kEvictThreads, "a thread per key and part of the comparisons");

struct EvictSmem {
  unsigned keys[kKeyCache];
  uint16_t list[kKeyCache];   // alone and cached: the kept slots
  unsigned hist[2][256];
  unsigned bad, in_place, digit, need, here, kmin, kmax, threshold;
  unsigned few[kFew], nfew;   // keys of the digit that holds the threshold, once they are few ...
  unsigned all[kFew], above;  // ... the cluster's, in rank order; this CTA's slots that stay above that digit
  unsigned wmin[kEvictWarps], wmax[kEvictWarps];
  unsigned gt[kEvictWarps], eq[kEvictWarps], total[2];
  unsigned src[2][kEvictThreads], dst[2][kEvictThreads];  // rows of two rounds, as page * 16 + row
};

template <class Rows, int C>
__global__ void __launch_bounds__(kEvictThreads, 2) evict_kernel(const EvictParams p) {
  extern __shared__ __align__(16) unsigned char smem[];
  EvictSmem& s = *reinterpret_cast<EvictSmem*>(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const unsigned rank = C == 1 ? 0u : cluster_ctarank();
  griddep_launch_dependents();
  griddep_wait();
  const int bg = blockIdx.x / C;
  const int b = bg / p.hkv, g = bg % p.hkv;
  const int len = p.seq_lens[b];
  const bool gated = p.gate != nullptr && p.gate[b] == 0;
  const bool bad_len = len < 1 || len > (long long)p.max_blocks * kPage;
  const int32_t* table = p.block_table + (size_t)b * p.max_blocks;
  const int32_t* dst_table = p.dst_table + (size_t)b * p.dst_blocks;
  const int keep = min(len, p.budget);
  const float* mass = p.mass + (size_t)bg * p.mass_tokens;
  float* mass_out = p.mass_out + (size_t)bg * p.mass_tokens;
  int32_t* kept = p.kept + (size_t)bg * p.budget;
  const bool usable = !gated && !bad_len;
  const bool select = usable && len > p.budget;
  const bool alone = C == 1 || len <= kAlone;  // (uniform over the cluster)
  const int parts = alone ? 1 : C, part = alone ? 0 : (int)rank;

  // the slots this CTA selects from; which are not kept in any case
  const int lo = (int)((long long)len * part / parts), hi = (int)((long long)len * (part + 1) / parts);
  const int free_lo = p.sink, free_hi = len - p.recent;
  const int my_lo = max(lo, free_lo), my_hi = min(hi, free_hi);
  const bool cached = hi - lo <= kKeyCache;
  auto key = [&](int i) { return cached ? s.keys[i - lo] : mass_key(mass[i]); };
  // One more of a digit. Where many keys are alike (slots that were never attended weigh nothing), the
  // warp's first key's digit is theirs: those are counted together.
  auto count = [&](unsigned* hist, bool on, unsigned digit) {
    const unsigned active = __ballot_sync(0xffffffffu, on);
    if (on) {
      const int first = __ffs(active) - 1;
      const unsigned same = __ballot_sync(active, digit == __shfl_sync(active, digit, first));
      if (!((same >> lane) & 1u)) atomicAdd(&hist[digit], 1u);
      else if (lane == first) atomicAdd(&hist[digit], (unsigned)__popc(same));
    }
  };

  // ---- page checks, keys and the range they span ----
  if (tid == 0) s.bad = s.nfew = s.above = 0u;
  for (int i = tid; i < 512; i += kEvictThreads) s.hist[i >> 8][i & 255] = 0u;
  __syncthreads();
  unsigned kmin = 0xffffffffu, kmax = 0u;
  if (usable) {
    // (the first pages' ids are on their way beside the weights)
    const int src_pages = (len + kPage - 1) / kPage, dst_pages = (keep + kPage - 1) / kPage;
    int i = part * kEvictThreads + tid;
    int src = i < src_pages ? table[i] : 0, dst = i < dst_pages ? dst_table[i] : -1;
    if (select) {
#pragma unroll 1
      for (int base = my_lo + tid; base < my_hi; base += kAhead * kEvictThreads) {
        float m[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
          if (base + u * kEvictThreads < my_hi) m[u] = mass[base + u * kEvictThreads];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          if (base + u * kEvictThreads >= my_hi) break;
          const unsigned k = mass_key(m[u]);
          if (cached) s.keys[base + u * kEvictThreads - lo] = k;
          kmin = min(kmin, k);
          kmax = max(kmax, k);
        }
      }
    }
    bool bad = false, same = false;  // (a destination table may be a copy of the source's)
#pragma unroll 1
    while (i < src_pages) {
      bad |= (unsigned)src >= (unsigned)p.num_blocks || (i < dst_pages && (unsigned)dst >= (unsigned)p.num_blocks);
      same |= dst == src;
      i += parts * kEvictThreads;
      if (i < src_pages) src = table[i];
      dst = i < dst_pages ? dst_table[i] : -1;
    }
    if (bad) atomicOr(&s.bad, 1u);
    if (same) atomicOr(&s.bad, 2u);
  }
  if (select) {
    warp_range(kmin, kmax);
    if (lane == 0) {
      s.wmin[warp] = kmin;
      s.wmax[warp] = kmax;
    }
  }
  __syncthreads();
  if (select) {
    kmin = s.wmin[lane % kEvictWarps];
    kmax = s.wmax[lane % kEvictWarps];
    warp_range(kmin, kmax);
  }
  unsigned flags = s.bad;
  if constexpr (C > 1) {
    if (!alone) {
      if (tid == 0) {
        s.kmin = kmin;
        s.kmax = kmax;
      }
      __syncthreads();
      cluster_sync();
      const unsigned r = lane % C;
      flags = dsmem_ld_u32(&s.bad, r);
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) flags |= __shfl_xor_sync(0xffffffffu, flags, o);
      kmin = dsmem_ld_u32(&s.kmin, r);
      kmax = dsmem_ld_u32(&s.kmax, r);
      warp_range(kmin, kmax);
    }
  }
  const bool bad_page = (flags & 1u) != 0u;
  const bool skip = !usable || bad_page;
  if (tid == 0) s.in_place = p.in_place || (flags & 2u) != 0u;  // (the same all over the cluster)
  if (tid == 0 && g == 0 && rank == 0) {
    if (!gated && (bad_len || bad_page)) report(p.status, bad_len ? ODA_DEV_BAD_LEN : ODA_DEV_BAD_BLOCK);
    if (!p.lens_alias) p.lens_out[b] = skip ? len : keep;
  }
  // In place, the last of the sequence's CTAs to have read the length writes the new one.
  auto leave = [&]() {
    if (p.lens_alias && tid == 0 && ticket_arrive(&p.ticket[b]) == (unsigned)(p.hkv * C - 1)) {
      p.ticket[b] = 0u;
      p.lens_out[b] = skip ? len : keep;
    }
  };
  if (skip) {
    leave();
    if (!alone) cluster_sync();  // nobody leaves while its shared memory may still be read
    return;
  }

  if (select) {
    unsigned need = p.budget - p.sink - p.recent;  // keys above the threshold stay, `need` of its equals
    unsigned threshold = 0xffffffffu;
    bool located = false;  // not alone: gt_before, eq_before count the CTAs before this one
    unsigned gt_before = 0u, eq_before = 0u;
    if (need > 0 && kmin == kmax) {
      threshold = kmin;
    } else if (need > 0) {
      int shift = 32 - __clz(kmin ^ kmax);  // above it all keys agree
      unsigned prefix = shift < 32 ? kmin >> shift : 0u;
#pragma unroll 1
      for (int pass = 0;; ++pass) {
        unsigned* hist = s.hist[pass & 1];
        const int bits = min(shift, 8), below = shift - bits;
        const unsigned mask = (1u << bits) - 1u;
#pragma unroll 1
        for (int base = my_lo; base < my_hi; base += kEvictThreads) {
          const int i = base + tid;
          const unsigned k = i < my_hi ? key(i) : 0u;
          const bool on = i < my_hi && (shift == 32 || (k >> shift) == prefix);
          if (pass == 0) count(hist, on, (k >> below) & mask);
          else if (on) atomicAdd(&hist[(k >> below) & mask], 1u);  // (few, and spread out)
        }
        __syncthreads();
        if (!alone) cluster_sync();
        // Thread t < 256: digit 255 - t, counted over the cluster, and the keys above it.
        unsigned n = 0u, upto = 0u;
        if (tid < 256) {
          const int digit = 255 - tid;
          if (alone) {
            n = hist[digit];
          } else if constexpr (C > 1) {
            unsigned v[C];
#pragma unroll
            for (int r = 0; r < C; ++r) v[r] = dsmem_ld_u32(&hist[digit], r);
#pragma unroll
            for (int r = 0; r < C; ++r) n += v[r];
          }
          upto = warp_scan(n, lane);
          if (lane == 31) s.gt[warp] = upto;
        } else {
          // the other histogram was last read before the barrier above
          s.hist[(pass + 1) & 1][tid - 256] = 0u;
        }
        __syncthreads();
        if (tid < 256) {
#pragma unroll 1
          for (int w = 0; w < warp; ++w) upto += s.gt[w];
          if (upto - n < need && upto >= need) {
            s.digit = 255 - tid;
            s.need = need - (upto - n);
            s.here = n;
          }
        }
        __syncthreads();
        prefix = (prefix << bits) | s.digit;
        shift = below;
        need = s.need;
        if (s.here == need || shift == 0) {  // every key of the digit stays, or they are all equal
          const bool all = s.here == need;
          threshold = (prefix << shift) - (all ? 1u : 0u);  // (not below 0: some free key does not stay)
          if (all) need = 0u;
          break;
        }
        if (s.here > kFew) continue;
        // Few enough to be compared with one another: the threshold is the one with fewer than `need` keys
        // above it and at least as many not below it.
        unsigned over = 0u;
#pragma unroll 1
        for (int i = my_lo + tid; i < my_hi; i += kEvictThreads) {
          const unsigned k = key(i) >> shift;
          if (k == prefix) s.few[atomicAdd(&s.nfew, 1u)] = key(i);
          over += k > prefix;
        }
        if (!alone) {
          over = warp_scan(over, lane);
          if (lane == 31 && over) atomicAdd(&s.above, over);
        }
        __syncthreads();
        int few = 0, few_before = 0;
        if (alone) {
          few = (int)s.nfew;
          if (tid < few) s.all[tid] = s.few[tid];
        } else if constexpr (C > 1) {
          // every slot of this CTA that is kept in any case, and the keys above the digit
          if (tid == 0) s.above += (unsigned)(hi - lo - max(0, my_hi - my_lo));
          cluster_sync();
          unsigned mine = 0u;
#pragma unroll
          for (int r = 0; r < C; ++r) {  // thread t: the cluster's t-th
            const int nr = (int)dsmem_ld_u32(&s.nfew, r);
            const unsigned ar = dsmem_ld_u32(&s.above, r);
            if (tid >= few && tid < few + nr) mine = dsmem_ld_u32(&s.few[tid - few], r);
            few += nr;
            few_before += r < (int)rank ? nr : 0;
            gt_before += r < (int)rank ? ar : 0u;
          }
          if (tid < few) s.all[tid] = mine;
        }
        __syncthreads();
        const unsigned mine = s.all[tid >> 2];  // (few <= kFew; what lies behind is not looked at)
        unsigned above = 0u, same = 0u;
#pragma unroll 4
        for (int j = tid & 3; j < few; j += 4) {
          const unsigned other = s.all[j];
          above += other > mine;
          same += other == mine;
        }
#pragma unroll
        for (int o = 1; o <= 2; o <<= 1) {
          above += __shfl_xor_sync(0xffffffffu, above, o);
          same += __shfl_xor_sync(0xffffffffu, same, o);
        }
        if ((tid >> 2) < few && above < need && above + same >= need) {  // (threads of equal keys write the same)
          s.threshold = mine;
          s.need = need - above;
        }
        __syncthreads();
        threshold = s.threshold;
        need = s.need;
        if (!alone) {
          const unsigned theirs = tid < few_before ? s.all[tid] : 0u;
          gt_before += (unsigned)__syncthreads_count(tid < few_before && theirs > threshold);
          eq_before = (unsigned)__syncthreads_count(tid < few_before && theirs == threshold);
          located = true;
        }
        break;
      }
    }

    // ---- count, then list: threads take consecutive runs of this CTA's slots (of odd length: the keys of a
    // warp's lanes then lie in different banks) ----
    const int per = ((hi - lo + kEvictThreads - 1) / kEvictThreads) | 1;
    const int tlo = min(hi, lo + tid * per), thi = min(hi, tlo + per);
    const bool choose = p.budget > p.sink + p.recent;
    auto classify = [&](int i, bool& above, bool& equal) {
      above = i < free_lo || i >= free_hi;
      equal = false;
      if (!above && choose) {
        const unsigned k = key(i);
        above = k > threshold;
        equal = k == threshold;
      }
    };
    unsigned gt = 0u, eq = 0u;
#pragma unroll 1
    for (int i = tlo; i < thi; ++i) {
      bool a, e;
      classify(i, a, e);
      gt += a;
      eq += e;
    }
    // scans over the warp, then the warps before
    const unsigned gt_upto = warp_scan(gt, lane), eq_upto = warp_scan(eq, lane);
    if (lane == 31) {
      s.gt[warp] = gt_upto;
      s.eq[warp] = eq_upto;
    }
    gt_before += gt_upto - gt;
    eq_before += eq_upto - eq;
    __syncthreads();
#pragma unroll 1
    for (int w = 0; w < warp; ++w) {
      gt_before += s.gt[w];
      eq_before += s.eq[w];
    }
    if (!alone && !located) {
      if (tid == kEvictThreads - 1) {
        s.total[0] = gt_before + gt;
        s.total[1] = eq_before + eq;
      }
      __syncthreads();
      cluster_sync();
#pragma unroll
      for (int r = 0; r < C - 1; ++r) {
        const unsigned gr = dsmem_ld_u32(&s.total[0], r), er = dsmem_ld_u32(&s.total[1], r);
        gt_before += r < (int)rank ? gr : 0u;
        eq_before += r < (int)rank ? er : 0u;
      }
    }
#pragma unroll 1
    for (int i = tlo; i < thi; ++i) {
      bool a, e;
      classify(i, a, e);
      if (a || (e && eq_before < need)) {
        const unsigned at = gt_before + min(eq_before, need);
        if (cached && alone) s.list[at] = (uint16_t)i;
        else kept[at] = i;
      }
      gt_before += a;
      eq_before += e;
    }
  } else {
#pragma unroll 1
    for (int i = rank * kEvictThreads + tid; i < p.budget; i += C * kEvictThreads)
      kept[i] = i < len ? i : -1;
  }
  if (alone) __syncthreads(); else cluster_sync();  // the whole list is written
  if (select && cached && alone)
#pragma unroll 1
    for (int i = rank * kEvictThreads + tid; i < keep; i += C * kEvictThreads) kept[i] = s.list[i];

  // ---- move, in rounds of the cluster; the rows of the next round are looked up beside this one's copies ----
  constexpr int kRound = kEvictThreads * kPieces / Rows::kCount < kEvictThreads
                             ? kEvictThreads * kPieces / Rows::kCount
                             : kEvictThreads;
  const bool listed = cached && alone;
  float m_next = 0.f;
  auto lookup = [&](int base) {  // thread t: row base + rank * kRound + t
    const int i = base + rank * kRound + tid;
    if (tid < kRound && i < keep) {
      const int from = !select ? i : listed ? (int)s.list[i] : kept[i];
      const int buf = (base / (C * kRound)) & 1;
      s.src[buf][tid] = (unsigned)table[from / kPage] * kPage + from % kPage;
      s.dst[buf][tid] = (unsigned)dst_table[i / kPage] * kPage + i % kPage;
      m_next = mass[from];
    }
  };
  lookup(0);
  __syncthreads();
#pragma unroll 1
  for (int base = 0; base < keep; base += C * kRound) {
    const int first = base + rank * kRound, buf = (base / (C * kRound)) & 1;
    const int rows = max(0, min(kRound, keep - first));
    const float m = m_next;
    uint4 v[kPieces];
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      const int e = tid + u * kEvictThreads;
      if (e < rows * Rows::kCount)
        v[u] = *reinterpret_cast<const uint4*>(Rows::at(p, s.src[buf][e / Rows::kCount], g, e % Rows::kCount));
    }
    lookup(base + C * kRound);
    if (s.in_place) {
      if (C > 1) cluster_sync(); else __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      const int e = tid + u * kEvictThreads;
      if (e < rows * Rows::kCount)
        *reinterpret_cast<uint4*>(Rows::at(p, s.dst[buf][e / Rows::kCount], g, e % Rows::kCount)) = v[u];
    }
    if (tid < rows) mass_out[first + tid] = m;
    __syncthreads();  // the next round's rows are looked up, this one's may be overwritten
  }
  // the slots given up weigh nothing until they are used again
#pragma unroll 1
  for (int i = keep + rank * kEvictThreads + tid; i < len; i += C * kEvictThreads) mass_out[i] = 0.f;
  leave();
  // Nothing is read from the other CTAs any more, but a cluster whose CTAs leave together makes room for the next
  // launch's at once (sequences of 20K to 32K, calls one behind the other: 44.3 us, 47 without).
  if (!alone) cluster_sync();
}

// CTAs per cluster: as many (at most 16) as keep all clusters within two waves of one CTA per SM,
// and no more than there are 256-slot runs in the longest sequence the table can hold.
static int evict_cluster(const DeviceInfo& di, long long rows, long long cap, int most) {
  int c = 1;
  while (c < most && rows * c * 2 <= 2ll * di.sms && cap > 256ll * c) c *= 2;
  return c;
}

template <class Rows>
static int prepare_evict(int device, int* most) {
  static int cached[64] = {0};
  if (device < 0 || device >= 64) return ODA_ERR_CUDA;
  if (cached[device] == 0) {
    constexpr auto kSmem = cudaFuncAttributeMaxDynamicSharedMemorySize;
    const int bytes = (int)sizeof(EvictSmem);
    cudaError_t e;
    if ((e = cudaFuncSetAttribute(evict_kernel<Rows, 16>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) !=
            cudaSuccess ||
        (e = cudaFuncSetAttribute(evict_kernel<Rows, 16>, kSmem, bytes)) != cudaSuccess ||
        (e = cudaFuncSetAttribute(evict_kernel<Rows, 8>, kSmem, bytes)) != cudaSuccess ||
        (e = cudaFuncSetAttribute(evict_kernel<Rows, 4>, kSmem, bytes)) != cudaSuccess ||
        (e = cudaFuncSetAttribute(evict_kernel<Rows, 2>, kSmem, bytes)) != cudaSuccess ||
        (e = cudaFuncSetAttribute(evict_kernel<Rows, 1>, kSmem, bytes)) != cudaSuccess)
      return cuda_status(e);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(16);
    cfg.blockDim = dim3(kEvictThreads);
    cfg.dynamicSmemBytes = sizeof(EvictSmem);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 16;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, evict_kernel<Rows, 16>, &cfg) != cudaSuccess) {
      cudaGetLastError();  // not fatal: eight CTAs are portable
      n = 0;
    }
    cached[device] = n > 0 ? 16 : 8;
  }
  *most = cached[device];
  return ODA_OK;
}

template <class Rows, int C>
static cudaError_t launch_evict_kernel(const EvictParams& p, long long rows, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * C));
  cfg.blockDim = dim3(kEvictThreads);
  cfg.dynamicSmemBytes = sizeof(EvictSmem);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = C;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = C > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, evict_kernel<Rows, C>, p);
}

static int evict_args(const oda_kv* kv, const float* mass, int64_t mass_tokens, int sink, int recent,
                      int budget, const int32_t* gate, const int32_t* dst_table, int dst_blocks,
                      const int32_t* kept, const float* mass_out, const int32_t* lens_out, const void* ws,
                      size_t ws_bytes) {
  const int rc = check_kv(kv);
  if (rc != ODA_OK) return rc;
  const long long cap = (long long)kv->max_blocks_per_seq * kPage;
  if (sink < 0 || recent < 0 || budget < 1 || (long long)sink + recent > budget || dst_blocks < 1)
    return ODA_ERR_INVALID_ARG;
  if (mass_tokens < cap) return ODA_ERR_INVALID_ARG;
  if ((long long)dst_blocks * kPage < budget && (long long)dst_blocks * kPage < cap)
    return ODA_ERR_INVALID_ARG;  // a destination shorter than what may be kept
  if (dst_table == kv->block_table && dst_blocks != kv->max_blocks_per_seq) return ODA_ERR_INVALID_ARG;
  // (slots and rounds of slots are counted in 32 bits)
  if (cap > (1ll << 31) - (1 << 16) || budget > (1ll << 31) - (1 << 16)) return ODA_ERR_UNSUPPORTED_SHAPE;
  if (kv->batch == 0) return ODA_OK;
  if (mass == nullptr || dst_table == nullptr || kept == nullptr || mass_out == nullptr ||
      lens_out == nullptr || ws == nullptr)
    return ODA_ERR_INVALID_ARG;
  if (!aligned_or_null(mass, 4) || !aligned_or_null(gate, 4) || !aligned_or_null(dst_table, 4) ||
      !aligned_or_null(kept, 4) || !aligned_or_null(mass_out, 4) || !aligned_or_null(lens_out, 4) ||
      !aligned_or_null(ws, 16))
    return ODA_ERR_INVALID_ARG;
  return ws_bytes < (size_t)kv->batch * sizeof(unsigned) ? ODA_ERR_WORKSPACE_TOO_SMALL : ODA_OK;
}

template <class Rows>
static int launch_evict(const oda_kv* kv, const float* mass, int64_t mass_tokens, int sink, int recent,
                        int budget, const int32_t* gate, const int32_t* dst_table, int dst_blocks,
                        int32_t* kept, float* mass_out, int32_t* lens_out, void* ws, size_t ws_bytes,
                        void* stream) {
  int rc = evict_args(kv, mass, mass_tokens, sink, recent, budget, gate, dst_table, dst_blocks, kept,
                      mass_out, lens_out, ws, ws_bytes);
  if (rc != ODA_OK || kv->batch == 0) return rc;
  DeviceInfo di;
  if ((rc = current_device_info(&di)) != ODA_OK) return rc;
  int most = 8;
  if ((rc = prepare_evict<Rows>(di.device, &most)) != ODA_OK) return rc;
  EvictParams p;
  p.k_cache = static_cast<unsigned char*>(kv->k_cache);
  p.v_cache = static_cast<unsigned char*>(kv->v_cache);
  p.block_table = kv->block_table;
  p.seq_lens = kv->seq_lens;
  p.hkv = kv->num_kv_heads;
  p.max_blocks = kv->max_blocks_per_seq;
  p.num_blocks = kv->num_blocks;
  p.mass = mass;
  p.mass_out = mass_out;
  p.mass_tokens = mass_tokens;
  p.sink = sink;
  p.recent = recent;
  p.budget = budget;
  p.gate = gate;
  p.dst_table = dst_table;
  p.dst_blocks = dst_blocks;
  p.kept = kept;
  p.lens_out = lens_out;
  p.ticket = static_cast<unsigned*>(ws);
  p.in_place = dst_table == kv->block_table || mass_out == mass;
  p.lens_alias = lens_out == kv->seq_lens;
  p.status = kv->dev_status;
  const long long rows = (long long)kv->batch * kv->num_kv_heads;
  const int C = evict_cluster(di, rows, (long long)kv->max_blocks_per_seq * kPage, most);
  if (rows * C >= (1ll << 31)) return ODA_ERR_UNSUPPORTED_SHAPE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  switch (C) {
    case 1: return cuda_status(launch_evict_kernel<Rows, 1>(p, rows, st));
    case 2: return cuda_status(launch_evict_kernel<Rows, 2>(p, rows, st));
    case 4: return cuda_status(launch_evict_kernel<Rows, 4>(p, rows, st));
    case 8: return cuda_status(launch_evict_kernel<Rows, 8>(p, rows, st));
    default: return cuda_status(launch_evict_kernel<Rows, 16>(p, rows, st));
  }
}

}  // namespace oda

using namespace oda;

extern "C" int oda_kv_evict_workspace_size(int32_t batch, size_t* bytes) {
  if (bytes == nullptr || batch < 0) return ODA_ERR_INVALID_ARG;
  *bytes = ((size_t)batch * sizeof(unsigned) + 255) / 256 * 256 + 256;
  return ODA_OK;
}

extern "C" int oda_kv_evict(const oda_kv* kv, const float* mass, int64_t mass_tokens, int32_t sink,
                            int32_t recent, int32_t budget, const int32_t* gate,
                            const int32_t* dst_block_table, int32_t dst_blocks_per_seq, int32_t* kept,
                            float* mass_out, int32_t* seq_lens_out, void* ws, size_t ws_bytes,
                            void* stream) {
  return launch_evict<Bf16Rows>(kv, mass, mass_tokens, sink, recent, budget, gate, dst_block_table,
                                dst_blocks_per_seq, kept, mass_out, seq_lens_out, ws, ws_bytes, stream);
}

extern "C" int oda_kv4_evict(const oda_kv4* kv, const float* mass, int64_t mass_tokens, int32_t sink,
                             int32_t recent, int32_t budget, const int32_t* gate,
                             const int32_t* dst_block_table, int32_t dst_blocks_per_seq, int32_t* kept,
                             float* mass_out, int32_t* seq_lens_out, void* ws, size_t ws_bytes,
                             void* stream) {
  const int rc = check_kv4(kv);
  if (rc != ODA_OK) return rc;
  const oda_kv k = kv4_as_kv(kv);
  return launch_evict<Kv4Rows>(&k, mass, mass_tokens, sink, recent, budget, gate, dst_block_table,
                               dst_blocks_per_seq, kept, mass_out, seq_lens_out, ws, ws_bytes, stream);
}
