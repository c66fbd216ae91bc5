// Append rows to the 4-bit cache and read rows back ([ODA] 접근 방법: the fully retained history,
// held in 144 bytes per position and KV head instead of 512).
//
// Bound: HBM bytes -- an appended row pair is 512 B read and 144 B written, one read back the reverse -- and
// for few rows the chain of dependent loads (ranges, length, page table, page) that finds a slot. A warp
// takes eight (row, KV head) units where there are enough of them to give every SM such warps: its first eight
// lanes look up where they go, all at once, and the rows of all eight are in flight together; else one unit.
// Measured, bf16 in and out, eight units a warp / one (us):
//   units       4,096        8,192        28,000       160,000
//   append      3.6 / 3.4    4.3 / 4.1    6.5 / 9.4    24.4 / 46.6 (105 MB: 66 % of a copy's rate)
//   read        3.2 / 3.0    3.3 / 3.6    4.9 / 7.7    19.8 / 39.7
#include "oda_internal.h"
#include "oda_kv4.cuh"

namespace oda {

constexpr int kRowWarps = 4;                       // (101,488 units appended: 17.6 us with 4, 18.2 with 8, 19.8 with 16)
constexpr int kMany = 8;                           // units a warp takes where there are many:
constexpr int kManyWarps = 8;                      // ... to give every SM this many such warps

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
//
// Eight units a warp: two at a time, 16 lanes each. Lane = 16 u + 8 isv + li holds dims 16 li .. 16 li + 15 of unit
// u's K or V row: a group of 64 dims is then four lanes, its ends two shuffles, and what is done once per lane is
// done for sixteen values.
template <int U>
__global__ void __launch_bounds__(kRowWarps * 32)
    kv4_append_many_kernel(const RowsParams p, const __nv_bfloat16* k_new, const __nv_bfloat16* v_new,
                           long long k_stride, long long v_stride) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, half = lane >> 4, isv = (lane >> 3) & 1, li = lane & 7;
  Units<U> units(p, lane);
  const __nv_bfloat16* base = (isv ? v_new : k_new) + 16 * li;
  const long long stride = isv ? v_stride : k_stride;
  uint4 v[U / 2][2];
#pragma unroll
  for (int u = 0; u < U / 2; ++u) {
    const int i = units.row(2 * u + half), g = units.head(2 * u + half);
    v[u][0] = v[u][1] = make_uint4(0u, 0u, 0u, 0u);
    if (i < p.num_rows) {
      const uint4* src = reinterpret_cast<const uint4*>(base + i * stride + g * kHeadDim);
      v[u][0] = src[0];
      v[u][1] = src[1];
    }
  }
  units.resolve(p, lane);
  // words 4 (li % 4) + g and two further of group g = li / 4
  const int word_off = isv * kKv4VOff + 16 * (li & 3) + 4 * (li >> 2);
  const int meta_off = kKv4MetaOff + 8 * isv + 4 * (li >> 2);
#pragma unroll
  for (int u = 0; u < U / 2; ++u) {
    const Slot s = units.at(2 * u + half);
    uint32_t ends = bf2_max_nan(kv4_ends(v[u][0]), kv4_ends(v[u][1]));
    ends = bf2_max_nan(ends, __shfl_xor_sync(0xffffffffu, ends, 1));
    ends = bf2_max_nan(ends, __shfl_xor_sync(0xffffffffu, ends, 2));
    const Kv4Group g = kv4_group(ends);
    const uint32_t w0 = kv4_codes(v[u][0], g), w1 = kv4_codes(v[u][1], g);
    if (s.row < 0) continue;
    uint32_t* dst = reinterpret_cast<uint32_t*>(s.page + word_off + s.row * kKv4RowBytes);
    dst[0] = w0;
    dst[2] = w1;
    if ((li & 3) == 0) *reinterpret_cast<uint32_t*>(s.page + meta_off + s.row * kKv4MetaBytes) = g.meta;
  }
}

__global__ void __launch_bounds__(kRowWarps * 32)
    kv4_append_kernel(const RowsParams p, const __nv_bfloat16* k_new, const __nv_bfloat16* v_new,
                      long long k_stride, long long v_stride) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  Units<1> units(p, lane);
  const int i = units.row(0), g = units.head(0);
  if (i >= p.num_rows) return;
  const uint4 v = *reinterpret_cast<const uint4*>((lane < 16 ? k_new + i * k_stride : v_new + i * v_stride) +
                                                  g * kHeadDim + 8 * (lane & 15));
  units.resolve(p, lane);
  const Slot s = units.at(0);
  if (s.row < 0) return;  // (uniform)
  uint32_t meta;
  const uint32_t word = kv4_quantise(v, lane, meta);
  kv4_store_row(s.page, s.row, word, meta, lane);
}

// Eight values of a code word, minimum + c * scale, as four pairs.
__device__ __forceinline__ void kv4_values(uint32_t w, uint32_t meta, float2 (&x)[4]) {
  const float2 s = make_float2(kv4_scale(meta), kv4_scale(meta));
  const float2 m = make_float2(kv4_min(meta), kv4_min(meta));
#pragma unroll
  for (int k = 0; k < 4; ++k) {  // a nibble in the mantissa of 2^23 is 2^23 + c
    const uint32_t b = w >> (8 * k);
    const float2 c = make_float2(__uint_as_float(0x4b000000u | (b & 15u)),
                                 __uint_as_float(0x4b000000u | ((b >> 4) & 15u)));
    x[k] = f2_fma2(f2_add(c, make_float2(-8388608.f, -8388608.f)), s, m);
  }
}

template <bool kBf16>
__device__ __forceinline__ void kv4_write_values(void* out, size_t at, uint32_t w, uint32_t meta) {
  float2 x[4];
  kv4_values(w, meta, x);
  if constexpr (kBf16) {
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[k].x, x[k].y);
      o[k] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(out) + at) = make_uint4(o[0], o[1], o[2], o[3]);
  } else {
    float4* dst = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
    dst[0] = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
    dst[1] = make_float4(x[2].x, x[2].y, x[3].x, x[3].y);
  }
}

// One unit a warp: lane 16 isv + li reads dims 8 li .. + 7.
template <bool kBf16>
__global__ void __launch_bounds__(kRowWarps * 32) kv4_read_kernel(const RowsParams p, void* k_out, void* v_out) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, li = lane & 15, isv = lane >> 4;
  Units<1> units(p, lane);
  units.resolve(p, lane);
  const Slot s = units.at(0);
  if (s.row < 0) return;
  const size_t at = ((size_t)units.row(0) * p.hkv + units.head(0)) * kHeadDim + 8 * li;
  const uint32_t w =
      *reinterpret_cast<const uint32_t*>(s.page + isv * kKv4VOff + s.row * kKv4RowBytes + 4 * kv4_word(li));
  const uint32_t meta =
      *reinterpret_cast<const uint32_t*>(s.page + kKv4MetaOff + s.row * kKv4MetaBytes + 4 * (lane >> 3));
  kv4_write_values<kBf16>(isv ? v_out : k_out, at, w, meta);
}

// Two at a time: lane 16 u + 8 isv + li reads dims 8 li .. + 7 of both groups, words 2 li and 2 li + 1.
template <int U, bool kBf16>
__global__ void __launch_bounds__(kRowWarps * 32)
    kv4_read_many_kernel(const RowsParams p, void* k_out, void* v_out) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, half = lane >> 4, isv = (lane >> 3) & 1, li = lane & 7;
  Units<U> units(p, lane);
  units.resolve(p, lane);
  const int code_off = isv * kKv4VOff + 8 * li, meta_off = kKv4MetaOff + 8 * isv;
  void* out = isv ? v_out : k_out;
  uint2 w[U / 2], meta[U / 2];
  bool ok[U / 2];
#pragma unroll
  for (int u = 0; u < U / 2; ++u) {
    const Slot s = units.at(2 * u + half);
    ok[u] = s.row >= 0;
    if (ok[u]) {
      w[u] = *reinterpret_cast<const uint2*>(s.page + code_off + s.row * kKv4RowBytes);
      meta[u] = *reinterpret_cast<const uint2*>(s.page + meta_off + s.row * kKv4MetaBytes);
    }
  }
#pragma unroll
  for (int u = 0; u < U / 2; ++u) {
    const size_t at = ((size_t)units.row(2 * u + half) * p.hkv + units.head(2 * u + half)) * kHeadDim + 8 * li;
    if (!ok[u]) continue;
    kv4_write_values<kBf16>(out, at, w[u].x, meta[u].x);
    kv4_write_values<kBf16>(out, at + kKv4Group, w[u].y, meta[u].y);
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

// Host checks shared by append and read; *work is false when there is nothing to do.
static int rows_params(const oda_kv4* kv, int32_t num_rows, const int32_t* cu_rows,
                       const int32_t* gate, RowsParams* p, bool* work) {
  *work = false;
  const int rc = check_kv4(kv);
  if (rc != ODA_OK) return rc;
  if (num_rows < 0 || (cu_rows == nullptr && num_rows != kv->batch)) return ODA_ERR_INVALID_ARG;
  if (!aligned_or_null(cu_rows, 4) || !aligned_or_null(gate, 4)) return ODA_ERR_INVALID_ARG;
  if (kv->batch == 0 || num_rows == 0) return ODA_OK;
  if (num_rows > 0x7fff0000) return ODA_ERR_UNSUPPORTED_SHAPE;  // (the last warps' rows pass num_rows)
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
  *work = true;
  return ODA_OK;
}

// CTAs, and whether a warp takes kMany units.
static int rows_grid(const RowsParams& p, unsigned* grid, bool* many) {
  DeviceInfo di;
  const int rc = current_device_info(&di);
  if (rc != ODA_OK) return rc;
  const long long units = (long long)p.num_rows * p.hkv;
  *many = units >= (long long)kMany * kManyWarps * di.sms;
  const long long per_cta = kRowWarps * (*many ? kMany : 1);
  const long long blocks = (units + per_cta - 1) / per_cta;
  if (blocks >= (1ll << 31)) return ODA_ERR_UNSUPPORTED_SHAPE;
  *grid = (unsigned)blocks;
  return ODA_OK;
}

}  // namespace oda

using namespace oda;

extern "C" int oda_kv4_append(const oda_kv4* kv, const void* k_new, const void* v_new,
                              int64_t k_stride, int64_t v_stride, int32_t num_rows,
                              const int32_t* cu_rows, const int32_t* gate, void* stream) {
  RowsParams p;
  bool work;
  int rc = rows_params(kv, num_rows, cu_rows, gate, &p, &work);
  if (rc != ODA_OK) return rc;
  const int64_t row = (int64_t)kv->num_kv_heads * kHeadDim;
  if (k_stride < row || v_stride < row || k_stride % 8 != 0 || v_stride % 8 != 0)
    return ODA_ERR_INVALID_ARG;  // rows are read 16 bytes at a time
  if (!work) return ODA_OK;
  if (k_new == nullptr || v_new == nullptr || !aligned_or_null(k_new, 16) ||
      !aligned_or_null(v_new, 16))
    return ODA_ERR_INVALID_ARG;
  unsigned grid;
  bool many;
  if ((rc = rows_grid(p, &grid, &many)) != ODA_OK) return rc;
  return cuda_status(launch_dependent(
      many ? kv4_append_many_kernel<kMany> : kv4_append_kernel, grid, kRowWarps * 32, 0,
      static_cast<cudaStream_t>(stream), p, static_cast<const __nv_bfloat16*>(k_new),
      static_cast<const __nv_bfloat16*>(v_new), (long long)k_stride, (long long)v_stride));
}

extern "C" int oda_kv4_read(const oda_kv4* kv, void* k_out, void* v_out, int32_t out_dtype,
                            int32_t num_rows, const int32_t* cu_rows, void* stream) {
  RowsParams p;
  bool work;
  int rc = rows_params(kv, num_rows, cu_rows, nullptr, &p, &work);
  if (rc != ODA_OK) return rc;
  if (out_dtype != ODA_F32 && out_dtype != ODA_BF16) return ODA_ERR_INVALID_ARG;
  if (!work) return ODA_OK;
  if (k_out == nullptr || v_out == nullptr || !aligned_or_null(k_out, 16) ||
      !aligned_or_null(v_out, 16))
    return ODA_ERR_INVALID_ARG;
  unsigned grid;
  bool many;
  if ((rc = rows_grid(p, &grid, &many)) != ODA_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const auto kernel = out_dtype == ODA_BF16
                          ? (many ? kv4_read_many_kernel<kMany, true> : kv4_read_kernel<true>)
                          : (many ? kv4_read_many_kernel<kMany, false> : kv4_read_kernel<false>);
  return cuda_status(launch_dependent(kernel, grid, kRowWarps * 32, 0, st, p, k_out, v_out));
}
