// Append rows to the 4-bit cache and read rows back ([ODA] 접근 방법: the fully retained history,
// held in 144 bytes per position and KV head instead of 512).
//
// Bound: HBM bytes -- an appended row pair is 512 B read and 144 B written -- and close behind it
// instruction issue (some 90 instructions a row pair and warp). A warp takes U (row, KV head) units: its
// first U lanes look up where the units go, all at once, then for each unit the lanes hold 16 bytes of
// the K row (0-15) and of the V row (16-31), so a group of 64 dims is 8 lanes and its ends three
// shuffles. U = 8 where there are units enough to fill the GPU with such warps (the chain of dependent
// loads that finds a slot is then paid once for eight units, and four rows are in flight); else U = 1.
#include "oda_internal.h"
#include "oda_kv4.cuh"

namespace oda {

constexpr int kRowWarps = 8;
constexpr int kManyUnits = 8 * kRowWarps * 8 * 148;  // eight CTAs of U = 8 warps per SM

struct RowsParams {
  unsigned char* cache;
  const int32_t* block_table;
  const int32_t* seq_lens;
  int batch, hkv, max_blocks, num_blocks;
  const int32_t* cu_rows;  // nullable: [batch + 1]; null = row b is slot t of sequence b
  int num_rows;
  const int32_t* gate;
  int* status;
};

// Where row i of KV head g goes: the page and the row inside it (-1: the row belongs to no sequence, its
// sequence is gated off, or it has no valid slot, which is reported).
struct Slot {
  unsigned char* page;
  int row;
};
__device__ __forceinline__ Slot find_slot(const RowsParams& p, int i, int g) {
  Slot none;
  none.page = nullptr;
  none.row = -1;
  int b = i, before = i, count = 1;
  if (p.cu_rows != nullptr) {
    int lo = 0, hi = p.batch;  // the first sequence that ends after row i
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (p.cu_rows[mid + 1] <= i) lo = mid + 1; else hi = mid;
    }
    if (lo >= p.batch) return none;
    b = lo;
    before = p.cu_rows[b];
    count = p.cu_rows[b + 1] - before;
    if (i < before || i - before >= count) return none;
  }
  if (p.gate != nullptr && p.gate[b] == 0) return none;
  const int len = p.seq_lens[b];
  if (len < 1 || len > (long long)p.max_blocks * kPage || count > len) {
    report(p.status, ODA_DEV_BAD_LEN);
    return none;
  }
  const int t = len - count + (i - before);
  const int pb = p.block_table[(size_t)b * p.max_blocks + t / kPage];
  if (pb < 0 || pb >= p.num_blocks) {
    report(p.status, ODA_DEV_BAD_BLOCK);
    return none;
  }
  Slot s;
  s.page = p.cache + ((size_t)pb * p.hkv + g) * kKv4PageBytes;
  s.row = t % kPage;
  return s;
}

// The units of this warp: lane l < U holds unit l's row and head, and after resolve() its slot; the others
// ask for them.
template <int U>
struct Units {
  int i, g;
  Slot slot;
  __device__ __forceinline__ Units(const RowsParams& p, int lane) {
    const long long unit = ((long long)blockIdx.x * kRowWarps + (threadIdx.x >> 5)) * U + (lane < U ? lane : 0);
    i = (int)(unit / p.hkv);
    g = (int)(unit % p.hkv);
  }
  __device__ __forceinline__ void resolve(const RowsParams& p, int lane) {
    slot.page = nullptr;
    slot.row = -1;
    if (lane < U && i < p.num_rows) slot = find_slot(p, i, g);
  }
  __device__ __forceinline__ int row(int u) const { return __shfl_sync(0xffffffffu, i, u); }
  __device__ __forceinline__ int head(int u) const { return __shfl_sync(0xffffffffu, g, u); }
  __device__ __forceinline__ Slot at(int u) const {
    Slot s;
    s.page = reinterpret_cast<unsigned char*>(
        __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(slot.page), u));
    s.row = __shfl_sync(0xffffffffu, slot.row, u);
    return s;
  }
};

// The rows are requested before their slots are looked up: neither needs the other.
template <int U>
__global__ void __launch_bounds__(kRowWarps * 32)
    kv4_append_kernel(const RowsParams p, const __nv_bfloat16* k_new, const __nv_bfloat16* v_new,
                      long long k_stride, long long v_stride) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  Units<U> units(p, lane);
  const __nv_bfloat16* base = (lane < 16 ? k_new : v_new) + 8 * (lane & 15);
  const long long stride = lane < 16 ? k_stride : v_stride;
  uint4 v[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int i = units.row(u), g = units.head(u);
    v[u] = make_uint4(0u, 0u, 0u, 0u);
    if (i < p.num_rows) v[u] = *reinterpret_cast<const uint4*>(base + i * stride + g * kHeadDim);
  }
  units.resolve(p, lane);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const Slot s = units.at(u);
    if (s.row < 0) continue;  // (uniform)
    uint32_t meta;
    const uint32_t word = kv4_quantise(v[u], lane, meta);
    kv4_store_row(s.page, s.row, word, meta, lane);
  }
}

constexpr int kInFlight = 4;

template <int U, bool kBf16>
__global__ void __launch_bounds__(kRowWarps * 32)
    kv4_read_kernel(const RowsParams p, void* k_out, void* v_out) {
  constexpr int N = U < kInFlight ? U : kInFlight;
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int li = lane & 15, isv = lane >> 4;
  Units<U> units(p, lane);
  units.resolve(p, lane);
  const int code_off = isv * kKv4VOff + 4 * kv4_word(li), meta_off = kKv4MetaOff + 4 * (lane >> 3);
#pragma unroll
  for (int u0 = 0; u0 < U; u0 += N) {
    size_t at[N];
    uint32_t w[N], meta[N];
    bool ok[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const Slot s = units.at(u0 + n);
      ok[n] = s.row >= 0;
      at[n] = ((size_t)units.row(u0 + n) * p.hkv + units.head(u0 + n)) * kHeadDim + 8 * li;
      if (ok[n]) {
        w[n] = *reinterpret_cast<const uint32_t*>(s.page + code_off + s.row * kKv4RowBytes);
        meta[n] = *reinterpret_cast<const uint32_t*>(s.page + meta_off + s.row * kKv4MetaBytes);
      }
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
      if (!ok[n]) continue;
      const float2 s = make_float2(kv4_scale(meta[n]), kv4_scale(meta[n]));
      const float2 m = make_float2(kv4_min(meta[n]), kv4_min(meta[n]));
      float2 x[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {  // a nibble in the mantissa of 2^23 is 2^23 + c
        const uint32_t b = w[n] >> (8 * k);
        const float2 c = make_float2(__uint_as_float(0x4b000000u | (b & 15u)),
                                     __uint_as_float(0x4b000000u | ((b >> 4) & 15u)));
        x[k] = f2_fma2(f2_add(c, make_float2(-8388608.f, -8388608.f)), s, m);
      }
      if constexpr (kBf16) {
        uint32_t o[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(x[k].x, x[k].y);
          o[k] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(isv ? v_out : k_out) + at[n]) =
            make_uint4(o[0], o[1], o[2], o[3]);
      } else {
        float4* dst = reinterpret_cast<float4*>(static_cast<float*>(isv ? v_out : k_out) + at[n]);
        dst[0] = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
        dst[1] = make_float4(x[2].x, x[2].y, x[3].x, x[3].y);
      }
    }
  }
}

oda_kv kv4_as_kv(const oda_kv4* kv) {
  oda_kv k = {};
  k.k_cache = k.v_cache = kv->cache;
  k.block_table = kv->block_table;
  k.seq_lens = kv->seq_lens;
  k.batch = kv->batch;
  k.num_kv_heads = kv->num_kv_heads;
  k.head_dim = kv->head_dim;
  k.block_size = kv->block_size;
  k.max_blocks_per_seq = kv->max_blocks_per_seq;
  k.num_blocks = kv->num_blocks;
  k.dev_status = kv->dev_status;
  k.stats = kv->stats;
  return k;
}

int check_kv4(const oda_kv4* kv) {
  if (kv == nullptr) return ODA_ERR_INVALID_ARG;
  const oda_kv k = kv4_as_kv(kv);
  const int rc = check_kv(&k);
  if (rc != ODA_OK) return rc;
  return kv->max_blocks_per_seq >= (1 << 27) ? ODA_ERR_UNSUPPORTED_SHAPE : ODA_OK;  // 32-bit positions
}

// Host checks shared by append and read; *grid is 0 when there is nothing to do.
static int rows_params(const oda_kv4* kv, int32_t num_rows, const int32_t* cu_rows,
                       const int32_t* gate, RowsParams* p, unsigned* grid, bool* many) {
  *grid = 0;
  const int rc = check_kv4(kv);
  if (rc != ODA_OK) return rc;
  if (num_rows < 0 || (cu_rows == nullptr && num_rows != kv->batch)) return ODA_ERR_INVALID_ARG;
  if (!aligned_or_null(cu_rows, 4) || !aligned_or_null(gate, 4)) return ODA_ERR_INVALID_ARG;
  if (kv->batch == 0 || num_rows == 0) return ODA_OK;
  if (num_rows > 0x7fff0000) return ODA_ERR_UNSUPPORTED_SHAPE;  // (the last warps' rows pass num_rows)
  const long long units = (long long)num_rows * kv->num_kv_heads;
  *many = units >= kManyUnits;
  const long long per_cta = kRowWarps * (*many ? 8 : 1);
  const long long blocks = (units + per_cta - 1) / per_cta;
  if (blocks >= (1ll << 31)) return ODA_ERR_UNSUPPORTED_SHAPE;
  p->cache = static_cast<unsigned char*>(kv->cache);
  p->block_table = kv->block_table;
  p->seq_lens = kv->seq_lens;
  p->batch = kv->batch;
  p->hkv = kv->num_kv_heads;
  p->max_blocks = kv->max_blocks_per_seq;
  p->num_blocks = kv->num_blocks;
  p->cu_rows = cu_rows;
  p->num_rows = num_rows;
  p->gate = gate;
  p->status = kv->dev_status;
  *grid = (unsigned)blocks;
  return ODA_OK;
}

}  // namespace oda

using namespace oda;

extern "C" int oda_kv4_append(const oda_kv4* kv, const void* k_new, const void* v_new,
                              int64_t k_stride, int64_t v_stride, int32_t num_rows,
                              const int32_t* cu_rows, const int32_t* gate, void* stream) {
  RowsParams p;
  unsigned grid;
  bool many = false;
  const int rc = rows_params(kv, num_rows, cu_rows, gate, &p, &grid, &many);
  if (rc != ODA_OK) return rc;
  const int64_t row = (int64_t)kv->num_kv_heads * kHeadDim;
  if (k_stride < row || v_stride < row || k_stride % 8 != 0 || v_stride % 8 != 0)
    return ODA_ERR_INVALID_ARG;  // rows are read 16 bytes at a time
  if (grid == 0) return ODA_OK;
  if (k_new == nullptr || v_new == nullptr || !aligned_or_null(k_new, 16) ||
      !aligned_or_null(v_new, 16))
    return ODA_ERR_INVALID_ARG;
  return cuda_status(launch_dependent(
      many ? kv4_append_kernel<8> : kv4_append_kernel<1>, grid, kRowWarps * 32, 0,
      static_cast<cudaStream_t>(stream), p, static_cast<const __nv_bfloat16*>(k_new),
      static_cast<const __nv_bfloat16*>(v_new), (long long)k_stride, (long long)v_stride));
}

extern "C" int oda_kv4_read(const oda_kv4* kv, void* k_out, void* v_out, int32_t out_dtype,
                            int32_t num_rows, const int32_t* cu_rows, void* stream) {
  RowsParams p;
  unsigned grid;
  bool many = false;
  const int rc = rows_params(kv, num_rows, cu_rows, nullptr, &p, &grid, &many);
  if (rc != ODA_OK) return rc;
  if (out_dtype != ODA_F32 && out_dtype != ODA_BF16) return ODA_ERR_INVALID_ARG;
  if (grid == 0) return ODA_OK;
  if (k_out == nullptr || v_out == nullptr || !aligned_or_null(k_out, 16) ||
      !aligned_or_null(v_out, 16))
    return ODA_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const auto kernel = out_dtype == ODA_BF16 ? (many ? kv4_read_kernel<8, true> : kv4_read_kernel<1, true>)
                                            : (many ? kv4_read_kernel<8, false> : kv4_read_kernel<1, false>);
  return cuda_status(launch_dependent(kernel, grid, kRowWarps * 32, 0, st, p, k_out, v_out));
}
