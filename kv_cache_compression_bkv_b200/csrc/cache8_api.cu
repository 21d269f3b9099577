// cache8_api.cu -- the entry points of the 8-bit cache (include/bkv.h):
// argument checks on the host, workspace carving, launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "bkv_internal.h"

namespace bkv {
namespace {

// cached rows, below 2^31 by more than any kernel steps past a length
constexpr long long kMaxRows = (1LL << 31) - 65536;
constexpr long long kMaxHeads = 65535;  // (sequence, KV head) pairs: a grid dimension

bool aligned(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

bool overlaps(const void *a, size_t na, const void *b, size_t nb) {
  if (!a || !b || na == 0 || nb == 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

struct Range {
  const void *p;
  size_t n;
};

// Whether any of the buffers a call writes shares memory with another of them
// or with one that it reads.
template <int kOut, int kIn>
bool any_overlap(const Range (&out)[kOut], const Range (&in)[kIn]) {
  for (int i = 0; i < kOut; ++i) {
    for (int j = i + 1; j < kOut; ++j)
      if (overlaps(out[i].p, out[i].n, out[j].p, out[j].n)) return true;
    for (int j = 0; j < kIn; ++j)
      if (overlaps(out[i].p, out[i].n, in[j].p, in[j].n)) return true;
  }
  return false;
}

bkv_status check_desc8(const bkv_cache8_desc *d) {
  if (!d) return BKV_ERR_INVALID_ARG;
  if (d->n_seqs < 1 || d->n_q_heads < 1 || d->n_kv_heads < 1 || d->head_dim < 1 || d->capacity < 1)
    return BKV_ERR_INVALID_ARG;
  if (d->n_q_heads % d->n_kv_heads != 0 || d->head_dim % 16 != 0) return BKV_ERR_INVALID_ARG;
  if (d->block != 16 && d->block != 32 && d->block != 64 && d->block != 128)
    return BKV_ERR_INVALID_ARG;
  if (d->capacity % d->block != 0) return BKV_ERR_INVALID_ARG;
  if (d->dtype != BKV_F32 && d->dtype != BKV_BF16) return BKV_ERR_INVALID_ARG;
  const long long heads = static_cast<long long>(d->n_seqs) * d->n_kv_heads;
  if (heads > kMaxHeads || d->capacity > kMaxRows / heads) return BKV_ERR_INVALID_ARG;
  return d->head_dim <= 128 ? BKV_OK : BKV_ERR_UNSUPPORTED;
}

size_t heads_of(const bkv_cache8_desc *d) { return static_cast<size_t>(d->n_seqs) * d->n_kv_heads; }
size_t code_bytes(const bkv_cache8_desc *d) {
  return heads_of(d) * static_cast<size_t>(d->capacity) * d->head_dim;
}
size_t scale_bytes(const bkv_cache8_desc *d) {
  return heads_of(d) * static_cast<size_t>(d->capacity / d->block) * sizeof(float);
}
size_t weight_bytes(const bkv_cache8_desc *d) {
  return heads_of(d) * static_cast<size_t>(d->capacity) * sizeof(float);
}
size_t elem_size(const bkv_cache8_desc *d) { return d->dtype == BKV_BF16 ? 2 : 4; }

bkv_status check_cache(const bkv_cache8_desc *d, const void *k8, const void *v8, const void *ks,
                       const void *vs, const void *lens) {
  const bkv_status st = check_desc8(d);
  if (st == BKV_ERR_INVALID_ARG) return st;
  if (!k8 || !v8 || !ks || !vs || !lens) return BKV_ERR_INVALID_ARG;
  if (!aligned(k8, 16) || !aligned(v8, 16) || !aligned(ks, 4) || !aligned(vs, 4) || !aligned(lens, 4))
    return BKV_ERR_INVALID_ARG;
  return st;
}

// Rows of queries per KV head, rows the call writes, and its key tiles (of 128
// keys and 8 rows at the least), within 32 bits.
bool rows_fit(const bkv_cache8_desc *d, int32_t T, int64_t max_len) {
  if (T < 1) return false;
  const long long rows = static_cast<long long>(d->n_q_heads / d->n_kv_heads) * T;
  const long long heads = static_cast<long long>(heads_of(d));
  return rows <= (1 << 24) && (rows + 32) <= kMaxRows / heads &&
         (rows + 7) / 8 * heads <= (kMaxRows >> 1) / ((max_len + 127) / 128 + 2);
}

size_t evict_workspace(const bkv_cache8_desc *d, long long K) {
  return align_up(static_cast<size_t>(d->n_seqs) * 4, kAlign) +
         align_up(heads_of(d) * static_cast<size_t>(K) * 4, kAlign);
}

}  // namespace
}  // namespace bkv

using namespace bkv;

extern "C" {

size_t bkv_cache8_workspace_size(const bkv_cache8_desc *desc, int64_t max_len, int32_t T, int64_t K,
                                 int32_t weights) {
  if (check_desc8(desc) != BKV_OK || max_len < 1 || max_len > desc->capacity || T < 0 || K < 0 ||
      K > kMaxRows || (T > 0 && !rows_fit(desc, T, max_len)))
    return 0;
  size_t n = 0;
  if (T > 0)
    n = plan_cache8_attend(desc->n_seqs, desc->n_q_heads, desc->n_kv_heads, desc->head_dim,
                           desc->dtype, max_len, T, weights != 0).bytes;
  if (K > 0) n = std::max(n, evict_workspace(desc, K));
  return n;
}

bkv_status bkv_cache8_append(const bkv_cache8_desc *desc, void *k8, void *v8, float *k_scale,
                             float *v_scale, const int32_t *lens, const void *k_new,
                             const void *v_new, int32_t T, const int32_t *n_new, void *stream) {
  const bkv_status st = check_cache(desc, k8, v8, k_scale, v_scale, lens);
  if (st == BKV_ERR_INVALID_ARG) return st;
  if (!k_new || !v_new || T < 1 || T > desc->capacity) return BKV_ERR_INVALID_ARG;
  if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(n_new, 4)) return BKV_ERR_INVALID_ARG;
  if (st != BKV_OK) return st;
  const size_t cb = code_bytes(desc), sb = scale_bytes(desc);
  const size_t nb = heads_of(desc) * static_cast<size_t>(T) * desc->head_dim * elem_size(desc);
  const size_t lb = static_cast<size_t>(desc->n_seqs) * 4;
  const Range out[] = {{k8, cb}, {v8, cb}, {k_scale, sb}, {v_scale, sb}};
  const Range in[] = {{k_new, nb}, {v_new, nb}, {lens, lb}, {n_new, lb}};
  if (any_overlap(out, in)) return BKV_ERR_INVALID_ARG;
  Cache8AppendArgs a{};
  a.k8 = static_cast<uint8_t *>(k8);
  a.v8 = static_cast<uint8_t *>(v8);
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.k_new = k_new;
  a.v_new = v_new;
  a.lens = lens;
  a.n_new = n_new;
  a.n_seqs = desc->n_seqs;
  a.n_kv_heads = desc->n_kv_heads;
  a.head_dim = desc->head_dim;
  a.block = desc->block;
  a.T = T;
  a.blocks_per_seq = (T + desc->block - 2) / desc->block + 1;
  a.cap = desc->capacity;
  return launch_cache8_append(a, desc->dtype, static_cast<cudaStream_t>(stream));
}

bkv_status bkv_cache8_attend(const bkv_cache8_desc *desc, const void *k8, const void *v8,
                             const float *k_scale, const float *v_scale, const int32_t *lens,
                             int64_t max_len, const void *q, int32_t T, const int32_t *n_new,
                             float scale, void *out, float *lse, const float *weights_in,
                             float *weights_out, float decay, void *workspace,
                             size_t workspace_bytes, void *stream) {
  const bkv_status st = check_cache(desc, k8, v8, k_scale, v_scale, lens);
  if (st == BKV_ERR_INVALID_ARG) return st;
  if (!q || !out || max_len < 1 || max_len > desc->capacity || !rows_fit(desc, T, max_len))
    return BKV_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(n_new, 4) || !aligned(lse, 4) ||
      !aligned(weights_in, 16) || !aligned(weights_out, 16))
    return BKV_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || scale < 0.f || !std::isfinite(decay) ||
      (weights_in && !weights_out))
    return BKV_ERR_INVALID_ARG;
  if (st != BKV_OK) return st;
  const size_t cb = code_bytes(desc), sb = scale_bytes(desc), wb = weight_bytes(desc);
  const size_t rows = static_cast<size_t>(desc->n_seqs) * desc->n_q_heads * T;
  const size_t qb = rows * desc->head_dim * elem_size(desc);
  const size_t lb = static_cast<size_t>(desc->n_seqs) * 4;
  const void *w_read = weights_in == weights_out ? nullptr : weights_in;
  const Cache8AttendPlan plan =
      plan_cache8_attend(desc->n_seqs, desc->n_q_heads, desc->n_kv_heads, desc->head_dim,
                         desc->dtype, max_len, T, weights_out != nullptr);
  const Range outs[] = {{out, qb}, {lse, rows * 4}, {weights_out, wb}, {workspace, plan.bytes}};
  const Range in[] = {{k8, cb}, {v8, cb}, {k_scale, sb}, {v_scale, sb},
                      {lens, lb}, {n_new, lb}, {q, qb}, {w_read, wb}};
  if (any_overlap(outs, in)) return BKV_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 16) || workspace_bytes < plan.bytes) return BKV_ERR_WORKSPACE;
  Cache8AttendArgs a{};
  a.k8 = static_cast<const uint8_t *>(k8);
  a.v8 = static_cast<const uint8_t *>(v8);
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.lens = lens;
  a.n_new = n_new;
  a.q = q;
  a.out = out;
  a.lse = lse;
  a.w_in = weights_in;
  a.w_out = weights_out;
  a.decay = decay;
  a.scale = scale != 0.f ? scale : 1.0f / std::sqrt(static_cast<float>(desc->head_dim));
  a.n_seqs = desc->n_seqs;
  a.n_q_heads = desc->n_q_heads;
  a.n_kv_heads = desc->n_kv_heads;
  a.head_dim = desc->head_dim;
  a.block = desc->block;
  a.T = T;
  a.group = desc->n_q_heads / desc->n_kv_heads;
  a.cap = desc->capacity;
  a.max_len = max_len;
  return launch_cache8_attend(a, plan, desc->dtype, workspace, static_cast<cudaStream_t>(stream));
}

bkv_status bkv_cache8_evict(const bkv_cache8_desc *desc, const void *k8, const void *v8,
                            const float *k_scale, const float *v_scale, const float *weights,
                            const int32_t *lens, int64_t max_len, int64_t K, int32_t sink,
                            int32_t recent, const bkv_cache8_desc *dst, void *k8_dst, void *v8_dst,
                            float *k_scale_dst, float *v_scale_dst, float *weights_dst,
                            int32_t *idx, int32_t *new_lens, void *workspace,
                            size_t workspace_bytes, void *stream) {
  bkv_status st = check_cache(desc, k8, v8, k_scale, v_scale, lens);
  if (st == BKV_ERR_INVALID_ARG) return st;
  bkv_status sd = check_cache(dst, k8_dst, v8_dst, k_scale_dst, v_scale_dst, lens);
  if (sd == BKV_ERR_INVALID_ARG) return sd;
  if (dst->n_seqs != desc->n_seqs || dst->n_kv_heads != desc->n_kv_heads ||
      dst->head_dim != desc->head_dim || dst->block != desc->block)
    return BKV_ERR_INVALID_ARG;
  if (!weights || !aligned(weights, 16) || !aligned(weights_dst, 16) || !aligned(idx, 4) ||
      !aligned(new_lens, 4))
    return BKV_ERR_INVALID_ARG;
  if (max_len < 1 || max_len > desc->capacity || K < 1 || K > kMaxRows || sink < 0 || recent < 0 ||
      static_cast<long long>(sink) + recent > K || dst->capacity < std::min<int64_t>(K, max_len))
    return BKV_ERR_INVALID_ARG;
  if (st != BKV_OK) return st;
  const bool in_place = k8_dst == k8 && v8_dst == v8 && k_scale_dst == k_scale &&
                        v_scale_dst == v_scale && dst->capacity == desc->capacity;
  const size_t cb = code_bytes(desc), sb = scale_bytes(desc), wb = weight_bytes(desc);
  const size_t dcb = code_bytes(dst), dsb = scale_bytes(dst), dwb = weight_bytes(dst);
  const size_t lb = static_cast<size_t>(desc->n_seqs) * 4;
  const size_t ib = heads_of(desc) * static_cast<size_t>(K) * 4;
  const size_t need = evict_workspace(desc, idx ? 0 : K);
  // in place the destination is the source; lens may be replaced by new_lens
  const bool same_w = in_place && weights_dst == weights;
  const Range outs[] = {{k8_dst, dcb}, {v8_dst, dcb}, {k_scale_dst, dsb}, {v_scale_dst, dsb},
                        {weights_dst, dwb}, {idx, ib}, {new_lens, lb}, {workspace, need}};
  const Range in[] = {{in_place ? nullptr : k8, cb}, {in_place ? nullptr : v8, cb},
                      {in_place ? nullptr : k_scale, sb}, {in_place ? nullptr : v_scale, sb},
                      {same_w ? nullptr : weights, wb},
                      {new_lens == lens ? nullptr : lens, lb}};
  if (any_overlap(outs, in)) return BKV_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 16) || workspace_bytes < need) return BKV_ERR_WORKSPACE;
  Cache8EvictArgs a{};
  a.k8 = static_cast<const uint8_t *>(k8);
  a.v8 = static_cast<const uint8_t *>(v8);
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.weights = weights;
  a.lens = lens;
  a.k8_dst = static_cast<uint8_t *>(k8_dst);
  a.v8_dst = static_cast<uint8_t *>(v8_dst);
  a.k_scale_dst = k_scale_dst;
  a.v_scale_dst = v_scale_dst;
  a.weights_dst = weights_dst;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  a.kept = reinterpret_cast<int32_t *>(ws);
  a.idx = idx ? idx : reinterpret_cast<int32_t *>(ws + align_up(lb, kAlign));
  a.new_lens = new_lens;
  a.n_seqs = desc->n_seqs;
  a.n_kv_heads = desc->n_kv_heads;
  a.head_dim = desc->head_dim;
  a.block = desc->block;
  a.sink = sink;
  a.recent = recent;
  a.cap = desc->capacity;
  a.dst_cap = dst->capacity;
  a.max_len = max_len;
  a.K = K;
  return launch_cache8_evict(a, in_place, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
