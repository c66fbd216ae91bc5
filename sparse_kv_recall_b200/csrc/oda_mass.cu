// Decode attention that also accumulates the attention weight of every cached position: what
// eviction from the cache goes by (oda_evict.cu).
//
// A position's weight is 2^(s - lse) with the log-sum of the whole visible set, which is known only
// when the decode kernel's last merge is done. So the decode kernel leaves every visible position's
// score in the workspace (4 bytes a query head, where recomputing it would read the K row again:
// 256 bytes in bf16, 72 in 4 bits) and a second kernel, launched with a programmatic dependency,
// turns scores into weights and adds them up over the query heads of the KV head. Bound: latency (length,
// page and scores, then the weights' store) and memory, 4 G + 8 bytes per position and KV head, the scores
// mostly out of L2. Two sequences of 32,769 tokens, 8 KV heads, 32 query heads: 60.6 us in all, 53.6 of them the
// bf16 attention by itself (60.3 with mass_in as mass_out); eight of 9K to 16K in 4 bits, 16 query heads: 38.0,
// of them 31.7 (37.8).
#include <math.h>

#include "oda_decode.cuh"
#include "oda_internal.h"
#include "oda_plan.cuh"

namespace oda {

constexpr int kMassThreads = 256;

struct MassParams {
  PlanArgs plan;
  int hkv, hq, group;
  const float* scores;   // [batch][hq][cap], base 2
  int cap;
  const float* lse;      // [batch][hq], natural
  const float* mass_in;  // nullable (zero); may be mass_out
  float* mass_out;       // [batch][hkv][mass_tokens]
  long long mass_tokens;
  int blocks_per_row;
};

// Whether logical page lp is in the sequence's list.
__device__ __forceinline__ bool page_listed(const PlanArgs& a, const SeqPlan& s, int b, int lp) {
  if (a.mode != ODA_MODE_KEEP) {
#pragma unroll
    for (int i = 0; i < kMaxRuns; ++i)
      if (lp >= run_first(s, i) && lp < run_first(s, i) + run_len(s, i)) return true;
    return false;
  }
  const int32_t* kb = a.keep_blocks + (size_t)b * a.max_keep;
  int lo = 0, hi = s.npages;  // first entry >= lp
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (kb[mid] < lp) lo = mid + 1; else hi = mid;
  }
  return lo < s.npages && kb[lo] == lp;
}

// Four consecutive positions a thread. kAlias (mass_out is mass_in): only listed pages are touched (of a full
// history all are listed); otherwise every position of the sequence is written.
template <bool kAlias>
__global__ void __launch_bounds__(kMassThreads) mass_kernel(const MassParams p) {
  griddep_launch_dependents();
  griddep_wait();
  const int bg = blockIdx.x / p.blocks_per_row;
  const int b = bg / p.hkv, g = bg % p.hkv;
  int idx = ((blockIdx.x % p.blocks_per_row) * kMassThreads + threadIdx.x) * 4;
  // A full history's positions are known before its length is: what is needed of them is on its way beside it
  // (within the buffers whatever the length; unused where that says so). 32K tokens, 2 sequences of 8 KV heads and
  // 32 query heads: 59.8 us with the attention, 61.8 with one load behind the other.
  const bool whole = p.plan.mode == ODA_MODE_FULL;
  const bool ahead = whole && idx < p.cap;
  float4 s_ahead[4], m_ahead = make_float4(0.f, 0.f, 0.f, 0.f);
  int pb_ahead = 0;
  if (ahead) {
    pb_ahead = p.plan.block_table[(size_t)b * p.plan.max_blocks + idx / kPage];
#pragma unroll
    for (int h = 0; h < 4; ++h)
      if (h < p.group)
        s_ahead[h] = *reinterpret_cast<const float4*>(p.scores + ((size_t)b * p.hq + g * p.group + h) * p.cap + idx);
    if (p.mass_in != nullptr)
      m_ahead = *reinterpret_cast<const float4*>(p.mass_in + (size_t)bg * p.mass_tokens + idx);
  }
  const SeqPlan sp = make_plan(p.plan, b);
  if (sp.skip || sp.err != 0) return;
  bool listed = true;
  if (kAlias && !whole) {
    if (idx >= sp.npages * kPage) return;
    const PageRef r = page_ref(p.plan, sp, b, idx / kPage);
    if (r.err != 0) return;
    idx = r.lp * kPage + idx % kPage;
  } else {
    if (idx > sp.t) return;
    listed = whole || page_listed(p.plan, sp, b, idx / kPage);
    if (listed) {
      const int pb = ahead ? pb_ahead : p.plan.block_table[(size_t)b * p.plan.max_blocks + idx / kPage];
      listed = pb >= 0 && pb < p.plan.num_blocks;  // a bad page was not attended
    }
  }
  bool vis[4];
  bool any = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) any |= vis[i] = listed && row_visible(sp, idx + i);
  float w[4] = {0.f, 0.f, 0.f, 0.f};
  if (any) {
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      if (h >= p.group) break;
      const size_t row = (size_t)b * p.hq + g * p.group + h;
      const float4 s4 = ahead ? s_ahead[h] : *reinterpret_cast<const float4*>(p.scores + row * p.cap + idx);
      const float s[4] = {s4.x, s4.y, s4.z, s4.w};
      const float l = p.lse[row];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (vis[i])  // (the difference in natural units first: it is small where the weight is not)
          w[i] += ex2_fast(fmaf(s[i], 0.69314718055994531f, -l) * 1.4426950408889634f);
    }
  }
  const size_t at = (size_t)bg * p.mass_tokens + idx;
  float in[4] = {0.f, 0.f, 0.f, 0.f};
  if (p.mass_in != nullptr) {
    const float4 v = ahead ? m_ahead : *reinterpret_cast<const float4*>(p.mass_in + at);
    in[0] = v.x; in[1] = v.y; in[2] = v.z; in[3] = v.w;
  }
  if (idx + 3 <= sp.t) {
    *reinterpret_cast<float4*>(p.mass_out + at) =
        make_float4(in[0] + w[0], in[1] + w[1], in[2] + w[2], in[3] + w[3]);
  } else {
    for (int i = 0; i < 4 && idx + i <= sp.t; ++i) p.mass_out[at + i] = in[i] + w[i];
  }
}

static size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// Workspace: merge tickets (the 4-bit decode's lie in front of its own workspace), the decode call's, a log-sum per
// query head, the scores. The tickets are in the same place for every shape and nothing else has to be
// zero, so one workspace serves calls of any.
struct MassWs {
  size_t decode_off, decode, lse_off, scores_off, total;
};
static int mass_ws(int batch, int hkv, int hq, int max_blocks, bool kv4, MassWs* w) {
  if (batch < 0 || hkv < 1 || hq < 1 || max_blocks < 1) return ODA_ERR_INVALID_ARG;
  int rc;
  w->decode_off = 0;
  if (kv4) {
    rc = kv4_decode_ws_bytes(batch, hkv, hq, &w->decode);
  } else {
    size_t ticket = 0;
    rc = hq % hkv != 0 || (hq / hkv != 1 && hq / hkv != 2 && hq / hkv != 4)
             ? ODA_ERR_UNSUPPORTED_SHAPE
             : decode_ws_layout(batch, hkv, hq, &w->decode, &ticket);
    if (rc == ODA_OK) rc = decode_scores_tickets_bytes(&w->decode_off);
  }
  if (rc != ODA_OK) return rc;
  w->lse_off = w->decode_off + up256(w->decode);
  w->scores_off = w->lse_off + up256((size_t)batch * hq * sizeof(float));
  w->total = w->scores_off + (size_t)batch * hq * max_blocks * kPage * sizeof(float);
  return ODA_OK;
}

static int decode_mass(const oda_kv* kv, const oda_kv4* kv4, const oda_visibility* vis, const void* q,
                       int hq, float scale, const void* k_new, const void* v_new, void* out,
                       int out_dtype, float* lse, const float* mass_in, float* mass_out,
                       int64_t mass_tokens, void* ws, size_t ws_bytes, void* stream) {
  if (vis == nullptr) return ODA_ERR_INVALID_ARG;
  int rc = check_kv(kv);
  if (rc != ODA_OK) return rc;
  if ((rc = check_visibility(kv, vis)) != ODA_OK) return rc;
  if ((rc = check_decode_args(kv, *vis, q, hq, scale, k_new, v_new, out, out_dtype, lse, ws)) != ODA_OK)
    return rc;
  const long long cap = (long long)kv->max_blocks_per_seq * kPage;
  if (mass_tokens < cap || mass_tokens % 4 != 0) return ODA_ERR_INVALID_ARG;
  if (cap > (1ll << 31) - (1 << 16)) return ODA_ERR_UNSUPPORTED_SHAPE;  // (positions are counted in 32 bits)
  if (kv->batch == 0) return ODA_OK;
  if (mass_out == nullptr || !aligned_or_null(mass_out, 16) || !aligned_or_null(mass_in, 16))
    return ODA_ERR_INVALID_ARG;
  MassWs wl;
  rc = mass_ws(kv->batch, kv->num_kv_heads, hq, kv->max_blocks_per_seq, kv4 != nullptr, &wl);
  if (rc != ODA_OK) return rc;
  if (ws_bytes < wl.total) return ODA_ERR_WORKSPACE_TOO_SMALL;
  const long long blocks_per_row = (cap + 4 * kMassThreads - 1) / (4 * kMassThreads);
  if (blocks_per_row * kv->batch * kv->num_kv_heads >= (1ll << 31)) return ODA_ERR_UNSUPPORTED_SHAPE;
  unsigned char* w = static_cast<unsigned char*>(ws);
  float* l = lse != nullptr ? lse : reinterpret_cast<float*>(w + wl.lse_off);
  float* scores = reinterpret_cast<float*>(w + wl.scores_off);
  rc = kv4 != nullptr ? launch_kv4_decode(kv4, vis, q, hq, scale, k_new, v_new, out, out_dtype, l, scores,
                                          (int)cap, w + wl.decode_off, wl.decode, stream)
                      : launch_decode_scores(kv, *vis, q, hq, scale, k_new, v_new, out, out_dtype, l,
                                             scores, (int)cap, reinterpret_cast<unsigned*>(w),
                                             w + wl.decode_off, wl.decode, stream);
  if (rc != ODA_OK) return rc;

  MassParams p;
  p.plan = plan_args(kv, *vis);
  p.hkv = kv->num_kv_heads;
  p.hq = hq;
  p.group = hq / kv->num_kv_heads;
  p.scores = scores;
  p.cap = (int)cap;
  p.lse = l;
  p.mass_in = mass_in;
  p.mass_out = mass_out;
  p.mass_tokens = mass_tokens;
  p.blocks_per_row = (int)blocks_per_row;
  return cuda_status(launch_dependent(mass_out == mass_in ? mass_kernel<true> : mass_kernel<false>,
                                      (unsigned)(blocks_per_row * kv->batch * kv->num_kv_heads), kMassThreads, 0,
                                      static_cast<cudaStream_t>(stream), p));
}

}  // namespace oda

using namespace oda;

static int mass_ws_size(int batch, int hkv, int hq, int max_blocks, bool kv4, size_t* bytes) {
  if (bytes == nullptr) return ODA_ERR_INVALID_ARG;
  MassWs w;
  const int rc = mass_ws(batch, hkv, hq, max_blocks, kv4, &w);
  if (rc == ODA_OK) *bytes = w.total;
  return rc;
}

extern "C" int oda_decode_mass_workspace_size(int32_t batch, int32_t num_kv_heads, int32_t num_q_heads,
                                              int32_t max_blocks_per_seq, size_t* bytes) {
  return mass_ws_size(batch, num_kv_heads, num_q_heads, max_blocks_per_seq, false, bytes);
}

extern "C" int oda_kv4_decode_mass_workspace_size(int32_t batch, int32_t num_kv_heads,
                                                  int32_t num_q_heads, int32_t max_blocks_per_seq,
                                                  size_t* bytes) {
  return mass_ws_size(batch, num_kv_heads, num_q_heads, max_blocks_per_seq, true, bytes);
}

extern "C" int oda_decode_mass(const oda_kv* kv, const oda_visibility* vis, const void* q,
                               int32_t num_q_heads, float scale, const void* k_new, const void* v_new,
                               void* out, int32_t out_dtype, float* lse, const float* mass_in,
                               float* mass_out, int64_t mass_tokens, void* ws, size_t ws_bytes,
                               void* stream) {
  return decode_mass(kv, nullptr, vis, q, num_q_heads, scale, k_new, v_new, out, out_dtype, lse, mass_in,
                     mass_out, mass_tokens, ws, ws_bytes, stream);
}

extern "C" int oda_kv4_decode_mass(const oda_kv4* kv, const oda_visibility* vis, const void* q,
                                   int32_t num_q_heads, float scale, const void* k_new,
                                   const void* v_new, void* out, int32_t out_dtype, float* lse,
                                   const float* mass_in, float* mass_out, int64_t mass_tokens, void* ws,
                                   size_t ws_bytes, void* stream) {
  const int rc = check_kv4(kv);
  if (rc != ODA_OK) return rc;
  const oda_kv k = kv4_as_kv(kv);
  return decode_mass(&k, kv, vis, q, num_q_heads, scale, k_new, v_new, out, out_dtype, lse, mass_in,
                     mass_out, mass_tokens, ws, ws_bytes, stream);
}
