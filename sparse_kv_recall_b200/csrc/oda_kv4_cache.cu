// Append rows to the 4-bit cache and read rows back ([ODA] 접근 방법: the fully retained history,
// held in 144 bytes per position and KV head instead of 512).
//
// Bound: HBM bytes -- an appended row pair is 512 B read and 144 B written, and a handful of
// instructions per value. One warp takes one (row, KV head): its lanes hold 16 bytes of the K row
// (0-15) and of the V row (16-31), so a group of 64 dims is 8 lanes and its range three shuffles.
#include "oda_internal.h"
#include "oda_kv4.cuh"

namespace oda {

constexpr int kRowWarps = 8;

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

// Where row i goes: the page of (sequence, KV head 0) and the row inside it. False: the row
// belongs to no sequence, its sequence is gated off, or it has no valid slot (reported).
__device__ __forceinline__ bool find_slot(const RowsParams& p, int i, int lane, int* page, int* row) {
  int b = i, before = i, count = 1;
  if (p.cu_rows != nullptr) {
    b = 0;  // number of sequences that end at or before row i
    for (int k = lane; k < (p.batch + 31) / 32 * 32; k += 32)
      b += __popc(__ballot_sync(0xffffffffu, k < p.batch && p.cu_rows[k + 1] <= i));
    if (b >= p.batch) return false;
    before = p.cu_rows[b];
    count = p.cu_rows[b + 1] - before;
    if (i < before || i - before >= count) return false;
  }
  if (p.gate != nullptr && p.gate[b] == 0) return false;
  const int len = p.seq_lens[b];
  if (len < 1 || len > (long long)p.max_blocks * kPage || count > len) {
    if (lane == 0) report(p.status, ODA_DEV_BAD_LEN);
    return false;
  }
  const int t = len - count + (i - before);
  const int pb = p.block_table[(size_t)b * p.max_blocks + t / kPage];
  if (pb < 0 || pb >= p.num_blocks) {
    if (lane == 0) report(p.status, ODA_DEV_BAD_BLOCK);
    return false;
  }
  *page = pb;
  *row = t % kPage;
  return true;
}

__global__ void __launch_bounds__(kRowWarps * 32)
    kv4_append_kernel(const RowsParams p, const __nv_bfloat16* k_new, const __nv_bfloat16* v_new,
                      long long k_stride, long long v_stride) {
  const int lane = threadIdx.x & 31;
  const long long unit = (long long)blockIdx.x * kRowWarps + (threadIdx.x >> 5);
  const int i = (int)(unit / p.hkv), g = (int)(unit % p.hkv);
  if (i >= p.num_rows) return;
  const int li = lane & 15;
  const __nv_bfloat16* src = (lane < 16 ? k_new + i * k_stride : v_new + i * v_stride) +
                             (size_t)g * kHeadDim + 8 * li;
  const uint4 v = *reinterpret_cast<const uint4*>(src);
  int pb, row;
  if (!find_slot(p, i, lane, &pb, &row)) return;
  uint32_t meta;
  const uint32_t word = kv4_quantise(v, lane, meta);
  kv4_store_row(p.cache + ((size_t)pb * p.hkv + g) * kKv4PageBytes, row, word, meta, lane);
}

template <bool kBf16>
__global__ void __launch_bounds__(kRowWarps * 32)
    kv4_read_kernel(const RowsParams p, void* k_out, void* v_out) {
  const int lane = threadIdx.x & 31;
  const long long unit = (long long)blockIdx.x * kRowWarps + (threadIdx.x >> 5);
  const int i = (int)(unit / p.hkv), g = (int)(unit % p.hkv);
  if (i >= p.num_rows) return;
  int pb, row;
  if (!find_slot(p, i, lane, &pb, &row)) return;
  const int li = lane & 15, isv = lane >> 4;
  const unsigned char* page = p.cache + ((size_t)pb * p.hkv + g) * kKv4PageBytes;
  const uint32_t w = *reinterpret_cast<const uint32_t*>(page + isv * kKv4VOff + row * kKv4RowBytes +
                                                        4 * kv4_word(li));
  const uint32_t meta = *reinterpret_cast<const uint32_t*>(page + kKv4MetaOff + row * kKv4MetaBytes +
                                                           4 * (lane >> 3));
  const float s = kv4_scale(meta), m = kv4_min(meta);
  float x[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) x[k] = fmaf((float)((w >> (4 * k)) & 15u), s, m);
  const size_t at = ((size_t)i * p.hkv + g) * kHeadDim + 8 * li;
  if constexpr (kBf16) {
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * k], x[2 * k + 1]);
      o[k] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(isv ? v_out : k_out) + at) =
        make_uint4(o[0], o[1], o[2], o[3]);
  } else {
    float4* dst = reinterpret_cast<float4*>(static_cast<float*>(isv ? v_out : k_out) + at);
    dst[0] = make_float4(x[0], x[1], x[2], x[3]);
    dst[1] = make_float4(x[4], x[5], x[6], x[7]);
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
                       const int32_t* gate, RowsParams* p, unsigned* grid) {
  *grid = 0;
  const int rc = check_kv4(kv);
  if (rc != ODA_OK) return rc;
  if (num_rows < 0 || (cu_rows == nullptr && num_rows != kv->batch)) return ODA_ERR_INVALID_ARG;
  if (!aligned_or_null(cu_rows, 4) || !aligned_or_null(gate, 4)) return ODA_ERR_INVALID_ARG;
  if (kv->batch == 0 || num_rows == 0) return ODA_OK;
  const long long units = (long long)num_rows * kv->num_kv_heads;
  const long long blocks = (units + kRowWarps - 1) / kRowWarps;
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
  const int rc = rows_params(kv, num_rows, cu_rows, gate, &p, &grid);
  if (rc != ODA_OK) return rc;
  const int64_t row = (int64_t)kv->num_kv_heads * kHeadDim;
  if (k_stride < row || v_stride < row || k_stride % 8 != 0 || v_stride % 8 != 0)
    return ODA_ERR_INVALID_ARG;  // rows are read 16 bytes at a time
  if (grid == 0) return ODA_OK;
  if (k_new == nullptr || v_new == nullptr || !aligned_or_null(k_new, 16) ||
      !aligned_or_null(v_new, 16))
    return ODA_ERR_INVALID_ARG;
  kv4_append_kernel<<<grid, kRowWarps * 32, 0, static_cast<cudaStream_t>(stream)>>>(
      p, static_cast<const __nv_bfloat16*>(k_new), static_cast<const __nv_bfloat16*>(v_new), k_stride,
      v_stride);
  return cuda_status(cudaGetLastError());
}

extern "C" int oda_kv4_read(const oda_kv4* kv, void* k_out, void* v_out, int32_t out_dtype,
                            int32_t num_rows, const int32_t* cu_rows, void* stream) {
  RowsParams p;
  unsigned grid;
  const int rc = rows_params(kv, num_rows, cu_rows, nullptr, &p, &grid);
  if (rc != ODA_OK) return rc;
  if (out_dtype != ODA_F32 && out_dtype != ODA_BF16) return ODA_ERR_INVALID_ARG;
  if (grid == 0) return ODA_OK;
  if (k_out == nullptr || v_out == nullptr || !aligned_or_null(k_out, 16) ||
      !aligned_or_null(v_out, 16))
    return ODA_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (out_dtype == ODA_BF16)
    kv4_read_kernel<true><<<grid, kRowWarps * 32, 0, st>>>(p, k_out, v_out);
  else
    kv4_read_kernel<false><<<grid, kRowWarps * 32, 0, st>>>(p, k_out, v_out);
  return cuda_status(cudaGetLastError());
}
