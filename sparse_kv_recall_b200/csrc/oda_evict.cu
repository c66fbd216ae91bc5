// Eviction from the paged cache by accumulated attention weight: of a (sequence, KV head)'s slots
// the first `sink`, the last `recent` and the rest's heaviest are kept, `budget` in all, in ascending
// slot order (the Local rule takes "recent" from the slot order), and move to the destination pages,
// which may be the source's own.
//
// One thread-block cluster takes one (sequence, KV head); its CTAs share the slots. The threshold
// weight is found by a radix select over order-preserving 32-bit keys, eight bits a pass, the
// histograms summed through distributed shared memory; every later decision follows from it and
// from counts, so the result does not depend on any order of execution. Bound: memory -- a kept
// row is read and written once (512 bytes in bf16, 144 in 4 bits), a weight is read a few times,
// mostly out of L2.
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
  unsigned* ticket;   // [batch]
  int in_place;       // the destination may be the source: order loads before stores
  int* status;
};

// 16-byte pieces of a row pair, and where piece i of (page, KV head, row) lies.
struct Bf16Rows {
  static constexpr int kCount = 32;
  __device__ static unsigned char* at(const EvictParams& p, int pb, int g, int row, int i) {
    const size_t off = (((size_t)pb * p.hkv + g) * kPage + row) * kRowBytes;
    return (i < 16 ? p.k_cache : p.v_cache) + off + 16 * (i & 15);
  }
};
struct Kv4Rows {
  static constexpr int kCount = 9;
  __device__ static unsigned char* at(const EvictParams& p, int pb, int g, int row, int i) {
    unsigned char* page = p.k_cache + ((size_t)pb * p.hkv + g) * kKv4PageBytes;
    if (i == 8) return page + kKv4MetaOff + row * kKv4MetaBytes;
    return page + (i >> 2) * kKv4VOff + row * kKv4RowBytes + 16 * (i & 3);
  }
};

__device__ __forceinline__ unsigned dsmem_ld_u32(const unsigned* local, unsigned rank) {
  return __float_as_uint(dsmem_ld(reinterpret_cast<const float*>(local), rank));
}

// Ascending order of floats as unsigned integers; -0 counts as 0.
__device__ __forceinline__ unsigned mass_key(float m) {
  const unsigned u = __float_as_uint(m + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

constexpr int kKeyCache = 8192;  // keys of a CTA's slots kept in shared memory (more: read again)

template <class Rows, int C>
__global__ void __launch_bounds__(kEvictThreads) evict_kernel(const EvictParams p) {
  __shared__ unsigned s_keys[kKeyCache];
  __shared__ unsigned s_hist[2][256], s_half[512];
  __shared__ unsigned s_bad, s_digit, s_need, s_all;
  __shared__ unsigned s_gt[kEvictWarps], s_eq[kEvictWarps], s_total[2];
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

  // this CTA's slots; which of the sequence's are not kept in any case; how many of those stay
  const int lo = (int)((long long)len * rank / C), hi = (int)((long long)len * (rank + 1) / C);
  const int free_lo = p.sink, free_hi = len - p.recent;
  const int my_lo = max(lo, free_lo), my_hi = min(hi, free_hi);
  const bool cached = hi - lo <= kKeyCache;
  auto key = [&](int i) { return cached ? s_keys[i - lo] : mass_key(mass[i]); };
  // One more of a digit. The keys of a warp share few digits (weights of like size share their
  // exponents), so equal ones are counted by one of their lanes.
  auto count = [&](unsigned* hist, bool on, unsigned digit) {
    const unsigned active = __ballot_sync(0xffffffffu, on);
    if (on) {
      const unsigned same = __match_any_sync(active, digit);
      if ((int)(__ffs(same) - 1) == lane) atomicAdd(&hist[digit], (unsigned)__popc(same));
    }
  };

  // ---- before the first cluster barrier: page checks and the first digit's histogram ----
  if (tid == 0) s_bad = 0u;
  for (int i = tid; i < 512; i += kEvictThreads) s_hist[i >> 8][i & 255] = 0u;
  __syncthreads();
  if (usable) {
    const int src_pages = (len + kPage - 1) / kPage, dst_pages = (keep + kPage - 1) / kPage;
    bool bad = false;
    for (int i = rank * kEvictThreads + tid; i < src_pages; i += C * kEvictThreads)
      bad |= (unsigned)table[i] >= (unsigned)p.num_blocks;
    for (int i = rank * kEvictThreads + tid; i < dst_pages; i += C * kEvictThreads)
      bad |= (unsigned)dst_table[i] >= (unsigned)p.num_blocks;
    if (bad) s_bad = 1u;
  }
  if (select) {
    for (int base = my_lo; base < my_hi; base += kEvictThreads) {
      const int i = base + tid;
      unsigned k = 0u;
      if (i < my_hi) {
        k = mass_key(mass[i]);
        if (cached) s_keys[i - lo] = k;
      }
      count(s_hist[0], i < my_hi, k >> 24);
    }
  }
  __syncthreads();
  if (C > 1) cluster_sync();
  bool bad_page = false;
#pragma unroll
  for (int r = 0; r < C; ++r) bad_page |= (C == 1 ? s_bad : dsmem_ld_u32(&s_bad, r)) != 0u;
  const bool skip = !usable || bad_page;
  // Every CTA of the cluster has read the length: the last of the sequence's KV heads to get
  // here writes the new one (lens_out may be seq_lens).
  if (rank == 0 && tid == 0) {
    if (!gated && g == 0 && (bad_len || bad_page))
      report(p.status, bad_len ? ODA_DEV_BAD_LEN : ODA_DEV_BAD_BLOCK);
    if (ticket_arrive(&p.ticket[b]) == (unsigned)(p.hkv - 1)) {
      p.ticket[b] = 0u;
      p.lens_out[b] = skip ? len : keep;
    }
  }
  if (skip) {
    if (C > 1) cluster_sync();  // nobody leaves while its shared memory may still be read
    return;
  }

  if (select) {
    unsigned need = p.budget - p.sink - p.recent;  // keys above the threshold stay, `need` of its equals
    unsigned threshold = 0xffffffffu;
    if (need > 0) {
      unsigned prefix = 0u;
#pragma unroll 1
      for (int pass = 0; pass < 4; ++pass) {
        unsigned* hist = s_hist[pass & 1];
        const int shift = 24 - 8 * pass;
        if (pass > 0) {
          for (int base = my_lo; base < my_hi; base += kEvictThreads) {
            const int i = base + tid;
            const unsigned k = i < my_hi ? key(i) : 0u;
            count(hist, i < my_hi && (k >> (shift + 8)) == prefix, (k >> shift) & 255u);
          }
          __syncthreads();
          if (C > 1) cluster_sync();
        }
        {  // the cluster's histogram: thread (half, digit) sums half the CTAs' counts
          unsigned n = 0u;
          const int digit = tid & 255, half = tid >> 8;
          if constexpr (C == 1) {
            n = half == 0 ? hist[digit] : 0u;
          } else {
            unsigned v[C / 2];
#pragma unroll
            for (int r = 0; r < C / 2; ++r) v[r] = dsmem_ld_u32(&hist[digit], half * (C / 2) + r);
#pragma unroll
            for (int r = 0; r < C / 2; ++r) n += v[r];
          }
          s_half[tid] = n;
        }
        __syncthreads();
        if (warp == 0) {  // lane l: digits 8 l .. 8 l + 7; from the top
          unsigned n[8], sum = 0u;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            n[i] = s_half[8 * lane + i] + s_half[256 + 8 * lane + i];
            sum += n[i];
          }
          unsigned above = sum;  // keys in this lane's digits and the higher ones
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const unsigned v = __shfl_down_sync(0xffffffffu, above, o);
            if (lane + o < 32) above += v;
          }
          above -= sum;
          if (above < need && above + sum >= need) {
            unsigned a = above, here = 0u;
            int d = 0;
            bool found = false;
#pragma unroll
            for (int i = 7; i >= 0; --i) {
              if (!found) {
                if (a + n[i] >= need) {
                  found = true;
                  d = i;
                  here = n[i];
                } else {
                  a += n[i];
                }
              }
            }
            s_digit = 8 * lane + d;
            s_need = need - a;
            s_all = here == need - a;  // every key of the digit stays: no lower digit matters
          }
        } else if (pass < 3 && tid >= kEvictThreads - 256) {
          // the other histogram was last read before the cluster barrier above
          if (pass > 0) s_hist[(pass + 1) & 1][tid - (kEvictThreads - 256)] = 0u;
        }
        __syncthreads();
        prefix = (prefix << 8) | s_digit;
        need = s_need;
        if (s_all) {
          threshold = (prefix << shift) - 1u;  // (not below 0: some free key does not stay)
          need = 0u;
          break;
        }
        threshold = prefix;
      }
    }

    // ---- count, then list: warps take consecutive runs of this CTA's slots ----
    const int per = ((hi - lo + kEvictWarps - 1) / kEvictWarps + 31) / 32 * 32;
    const int wlo = min(hi, lo + warp * per), whi = min(hi, wlo + per);
    auto classify = [&](int i, bool& above, bool& equal) {
      above = equal = false;
      if (i >= whi) return;
      if (i < free_lo || i >= free_hi) {
        above = true;
      } else if (p.budget > p.sink + p.recent) {
        const unsigned k = key(i);
        above = k > threshold;
        equal = k == threshold;
      }
    };
    unsigned gt = 0u, eq = 0u;
    for (int base = wlo; base < whi; base += 32) {
      bool a, e;
      classify(base + lane, a, e);
      gt += __popc(__ballot_sync(0xffffffffu, a));
      eq += __popc(__ballot_sync(0xffffffffu, e));
    }
    if (lane == 0) {
      s_gt[warp] = gt;
      s_eq[warp] = eq;
    }
    __syncthreads();
    unsigned gt_before = 0u, eq_before = 0u;
    for (int w = 0; w < kEvictWarps; ++w) {
      if (w < warp) {
        gt_before += s_gt[w];
        eq_before += s_eq[w];
      }
    }
    if (tid == kEvictThreads - 1) {
      s_total[0] = gt_before + gt;
      s_total[1] = eq_before + eq;
    }
    __syncthreads();
    if (C > 1) cluster_sync();
#pragma unroll
    for (int r = 0; r < C - 1; ++r) {
      const unsigned gr = dsmem_ld_u32(&s_total[0], r), er = dsmem_ld_u32(&s_total[1], r);
      gt_before += r < (int)rank ? gr : 0u;
      eq_before += r < (int)rank ? er : 0u;
    }
    for (int base = wlo; base < whi; base += 32) {
      bool a, e;
      classify(base + lane, a, e);
      const unsigned am = __ballot_sync(0xffffffffu, a), em = __ballot_sync(0xffffffffu, e);
      const unsigned below = (1u << lane) - 1u;
      const unsigned my_eq = eq_before + __popc(em & below);
      if (a || (e && my_eq < need))
        kept[gt_before + __popc(am & below) + min(my_eq, need)] = base + lane;
      gt_before += __popc(am);
      eq_before += __popc(em);
    }
  } else {
    for (int i = rank * kEvictThreads + tid; i < p.budget; i += C * kEvictThreads)
      kept[i] = i < len ? i : -1;
  }
  if (C > 1) cluster_sync(); else __syncthreads();  // the whole list is written

  // ---- move ----
  constexpr int kRowsPerRound = kEvictThreads * kPieces / Rows::kCount;
  for (int base = 0; base < keep; base += C * kRowsPerRound) {
    const int first = base + rank * kRowsPerRound;
    const int rows = max(0, min(kRowsPerRound, keep - first));
    uint4 v[kPieces];
    float m = 0.f;
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      const int e = tid + u * kEvictThreads;
      if (e < rows * Rows::kCount) {
        const int s = kept[first + e / Rows::kCount];
        v[u] = *reinterpret_cast<const uint4*>(Rows::at(p, table[s / kPage], g, s % kPage, e % Rows::kCount));
      }
    }
    if (tid < rows) m = mass[kept[first + tid]];
    if (p.in_place) {
      if (C > 1) cluster_sync(); else __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      const int e = tid + u * kEvictThreads;
      if (e < rows * Rows::kCount) {
        const int i = first + e / Rows::kCount;
        *reinterpret_cast<uint4*>(Rows::at(p, dst_table[i / kPage], g, i % kPage, e % Rows::kCount)) = v[u];
      }
    }
    if (tid < rows) mass_out[first + tid] = m;
  }
  // the slots given up weigh nothing until they are used again
  for (int i = keep + rank * kEvictThreads + tid; i < len; i += C * kEvictThreads) mass_out[i] = 0.f;
  if (C > 1) cluster_sync();  // nobody leaves while its shared memory may still be read
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
    const cudaError_t e =
        cudaFuncSetAttribute(evict_kernel<Rows, 16>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return cuda_status(e);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(16);
    cfg.blockDim = dim3(kEvictThreads);
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
  if (cap >= (1ll << 31)) return ODA_ERR_UNSUPPORTED_SHAPE;
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
