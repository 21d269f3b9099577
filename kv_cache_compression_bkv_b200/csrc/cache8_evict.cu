// cache8_evict.cu -- eviction from the 8-bit cache by accumulated attention
// weight: which rows stay (evict_select_kernel), and their compaction
// (evict_compact_kernel).
//
// Select: one CTA per (sequence, KV head).  A row of L > K positions keeps the
// first `sink`, the last `recent` and, of the rest, the K - sink - recent with
// the largest weights, ties to the lower position.  The weights are ranked as
// order-preserving 32-bit keys (order_key.cuh); three radix passes of 11, 11
// and 10 bits over a shared-memory histogram give the threshold key and how
// many of its ties stay.  The keys are staged in shared memory when the row
// fits, so HBM sees the row once.  Then every position becomes one bit of a
// mask (a ballot per 32 positions), ties are dropped by a prefix sum over the
// mask words, and the kept positions are written in ascending order at the
// words' prefix offsets.
//
// Compaction: a CTA takes 128 new rows of one (sequence, head, K or V), which
// are whole blocks of the new cache.  It gathers the rows' codes and old
// scales, reduces each new block's largest magnitude (exact: a code times a
// power of two), takes the scale that the append would take, moves the codes
// of the rows whose scale differs and writes them.  In place, a cluster of
// CTAs reads up to 8 x 128 rows, meets at the cluster barrier and only then
// writes them: new row i takes old row idx_i >= i, so every row, scale and
// weight a later round reads lies at or past that round's first row.
#include <cooperative_groups.h>

#include <algorithm>

#include "bkv_device_status.cuh"
#include "bkv_internal.h"
#include "cache8.cuh"
#include "order_key.cuh"

BKV_DEFINE_STATUS_ACCESSOR(take_status_cache8_evict)

namespace bkv {
namespace {

using namespace cache8;
namespace cg = cooperative_groups;

constexpr int kSelThreads = 1024;
constexpr int kBins = 2048;
constexpr int kStageMax = 45056;  // positions whose weights fit in shared memory
// mask words per thread: positions up to kSelThreads * 32 * kWordsMax
constexpr int kMaskWords(long long L) { return static_cast<int>((L + 31) / 32); }

// NaN ranks below every number
__device__ __forceinline__ uint32_t rank_key(float w) { return w != w ? 0u : order_key(w); }

// Exclusive prefix sum over the CTA of one value per thread; `total` for all.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t *s_warp, uint32_t *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // s_warp is free again
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  if (warp == 0) {
    uint32_t t = s_warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, t, o);
      if (lane >= o) t += y;
    }
    s_warp[lane] = t;
  }
  __syncthreads();
  *total = s_warp[31];
  return x - v + (warp ? s_warp[warp - 1] : 0u);
}

template <bool kStaged>
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const Cache8EvictArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ uint32_t s_hist[kBins];
  __shared__ uint32_t s_warp[32];
  __shared__ uint32_t s_bin, s_above;
  uint32_t *s_mask = reinterpret_cast<uint32_t *>(smem);              // above the threshold, or protected
  uint32_t *s_tie = s_mask + a.mask_words;                            // equal to it
  uint32_t *s_key = s_tie + a.mask_words;
  const int tid = threadIdx.x, lane = tid & 31;
  const int head = blockIdx.x, seq = head / a.n_kv_heads;
  const int L = a.lens[seq];
  if (L < 0 || L > a.max_len) {
    if (tid == 0) {
      record_device_status(BKV_DEV_ASSERT, 621);
      if (head % a.n_kv_heads == 0) a.kept[seq] = -1;
    }
    return;
  }
  const int K = static_cast<int>(a.K);
  if (tid == 0 && head % a.n_kv_heads == 0) a.kept[seq] = min(L, K);
  int32_t *idx = a.idx + static_cast<size_t>(head) * K;
  if (L <= K) {
    for (int i = tid; i < L; i += kSelThreads) idx[i] = i;
    return;
  }
  const float *w = a.weights + static_cast<size_t>(head) * a.cap;
  const int lo = a.sink, hi = L - a.recent;  // candidates: [lo, hi)
  uint32_t need = static_cast<uint32_t>(K - a.sink - a.recent);
  auto key_at = [&](int j) { return kStaged ? s_key[j] : rank_key(__ldg(w + j)); };

  uint32_t thr = 0, ties = 0;  // keep keys > thr, and the first `ties` equal to it
  if (need > 0) {
    uint32_t prefix = 0;
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const int bits = pass == 2 ? 10 : 11;
      for (int b = tid; b < kBins; b += kSelThreads) s_hist[b] = 0;
      __syncthreads();
      if (pass == 0 && kStaged) {
        for (int j = tid; j < L; j += kSelThreads) {
          const uint32_t k = rank_key(__ldg(w + j));
          s_key[j] = k;
          if (j >= lo && j < hi) atomicAdd(&s_hist[k >> 21], 1u);
        }
      } else {
        for (int j = lo + tid; j < hi; j += kSelThreads) {
          const uint32_t k = key_at(j);
          if (pass == 0 || (k >> (shift + bits)) == prefix)
            atomicAdd(&s_hist[(k >> shift) & ((1u << bits) - 1)], 1u);
        }
      }
      __syncthreads();
      // the bin that holds the need-th largest key: suffix counts, two bins a
      // thread, the largest bins first
      const int b1 = kBins - 1 - 2 * tid, b0 = b1 - 1;
      const uint32_t c1 = s_hist[b1], c0 = s_hist[b0];
      uint32_t total;
      const uint32_t above = block_scan(c0 + c1, s_warp, &total);
      if (above < need && need <= above + c1) {
        s_bin = static_cast<uint32_t>(b1);
        s_above = above;
      } else if (above + c1 < need && need <= above + c1 + c0) {
        s_bin = static_cast<uint32_t>(b0);
        s_above = above + c1;
      }
      __syncthreads();
      prefix = (prefix << bits) | s_bin;
      need -= s_above;
    }
    thr = prefix;
    ties = need;
  }
  // masks: a bit per position
  const int words = (L + 31) >> 5;
  for (int q = tid >> 5; q < words; q += kSelThreads / 32) {
    const int j = q * 32 + lane;
    const bool cand = j >= lo && j < hi;
    const uint32_t k = cand && ties > 0 ? key_at(j) : 0u;
    const uint32_t m = __ballot_sync(0xffffffffu,
                                     j < L && (!cand || (ties > 0 && k > thr)));
    const uint32_t t = __ballot_sync(0xffffffffu, cand && ties > 0 && k == thr);
    if (lane == 0) {
      s_mask[q] = m;
      s_tie[q] = t;
    }
  }
  __syncthreads();
  // each thread owns a run of words; ties kept in position order
  const int per = (words + kSelThreads - 1) / kSelThreads;
  const int q0 = min(tid * per, words), q1 = min(q0 + per, words);
  uint32_t cnt = 0, total;
  for (int q = q0; q < q1; ++q) cnt += __popc(s_tie[q]);
  uint32_t before = block_scan(cnt, s_warp, &total);
  cnt = 0;
  for (int q = q0; q < q1; ++q) {
    uint32_t t = s_tie[q];
    const uint32_t c = __popc(t);
    if (before + c > ties) {  // drop the highest positions
      const uint32_t stay = before < ties ? ties - before : 0u;
      for (uint32_t d = c; d > stay; --d) t &= ~(0x80000000u >> __clz(t));
    }
    before += c;
    const uint32_t m = s_mask[q] | t;
    s_mask[q] = m;
    cnt += __popc(m);
  }
  uint32_t at = block_scan(cnt, s_warp, &total);
  for (int q = q0; q < q1; ++q) {
    uint32_t m = s_mask[q];
    while (m) {
      idx[at++] = q * 32 + __ffs(m) - 1;
      m &= m - 1;
    }
  }
}

constexpr int kRows = 128;     // new rows per CTA and round
constexpr int kThreads = 256;
constexpr int kPieces = 4;     // 16-byte pieces per thread: 128 rows x 8 / 256

template <bool kInPlace>
__global__ void __launch_bounds__(kThreads) evict_compact_kernel(const Cache8EvictArgs a) {
  __shared__ int32_t s_idx[kRows];
  __shared__ int s_exp[kRows];           // the rows' old scale exponents
  __shared__ uint32_t s_max[kRows / 16]; // per new block: bits of the largest magnitude
  const int tid = threadIdx.x;
  unsigned u = blockIdx.x;
  const int part = u % a.ctas_per_head;  // in place: the rank in the cluster
  u /= a.ctas_per_head;
  const int kv = u & 1;
  const int head = u >> 1, seq = head / a.n_kv_heads;
  const int n = a.kept[seq];
  if (kv == 0 && part == 0 && tid == 0 && head % a.n_kv_heads == 0 && n >= 0 && a.new_lens)
    a.new_lens[seq] = n;
  const int pr = a.head_dim >> 4;
  const int block = a.block;
  const uint8_t *src = (kv ? a.v8 : a.k8) + static_cast<size_t>(head) * a.cap * a.head_dim;
  const float *src_scale = (kv ? a.v_scale : a.k_scale) + static_cast<size_t>(head) * (a.cap / block);
  uint8_t *dst = (kv ? a.v8_dst : a.k8_dst) + static_cast<size_t>(head) * a.dst_cap * a.head_dim;
  float *dst_scale = (kv ? a.v_scale_dst : a.k_scale_dst) + static_cast<size_t>(head) * (a.dst_cap / block);
  const float *w_src = a.weights + static_cast<size_t>(head) * a.cap;
  float *w_dst = a.weights_dst ? a.weights_dst + static_cast<size_t>(head) * a.dst_cap : nullptr;
  const int32_t *idx = a.idx + static_cast<size_t>(head) * a.K;

  // out of place: one round, this CTA's rows; in place: rounds of the cluster's
  // rows, the same number for all of its CTAs
  const int step = kInPlace ? kRows * a.ctas_per_head : INT32_MAX;
  for (int i0 = 0; kInPlace ? i0 < n : i0 == 0; i0 += step) {
    const int base = i0 + part * kRows;
    const int rows = max(0, min(kRows, n - base));
    if (!kInPlace && rows == 0) return;
    float wv = 0.f;
    if (tid < rows) {
      const int j = idx[base + tid];
      s_idx[tid] = j;
      s_exp[tid] = exp_of(kInPlace ? __ldcg(src_scale + j / block) : __ldg(src_scale + j / block));
      if (kv == 0 && w_dst) wv = kInPlace ? __ldcg(w_src + j) : __ldg(w_src + j);
    }
    if (tid >= kThreads - kRows / 16) s_max[tid - (kThreads - kRows / 16)] = 0;
    __syncthreads();
    uint4 c[kPieces];
    const int pieces = rows * pr;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int p = tid + i * kThreads;
      if (p < pieces) {
        const int r = p / pr;
        const uint4 *q = reinterpret_cast<const uint4 *>(
            src + static_cast<size_t>(s_idx[r]) * a.head_dim) + (p - r * pr);
        c[i] = kInPlace ? __ldcg(q) : __ldcs(q);
      }
    }
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int p = tid + i * kThreads;
      if (p < pieces) {
        const int r = p / pr;
        const float m = absmax16(c[i]) * pow2f(s_exp[r]);
        atomicMax(&s_max[r / block], __float_as_uint(m));
      }
    }
    // every read of this round has returned in every CTA before any write
    if (kInPlace) cg::this_cluster().sync(); else __syncthreads();
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int p = tid + i * kThreads;
      if (p < pieces) {
        const int r = p / pr;
        const int k = s_exp[r] - scale_exp(__uint_as_float(s_max[r / block]));
        if (k != 0) c[i] = rescale16(c[i], k);
        uint4 *q = reinterpret_cast<uint4 *>(dst + static_cast<size_t>(base) * a.head_dim) + p;
        if (kInPlace) __stcg(q, c[i]); else __stcs(q, c[i]);
      }
    }
    if (tid < rows) {
      if (tid % block == 0)
        dst_scale[(base + tid) / block] = pow2f(scale_exp(__uint_as_float(s_max[tid / block])));
      if (kv == 0 && w_dst) w_dst[base + tid] = wv;
    }
    if (kInPlace) __syncthreads();  // s_idx, s_exp and s_max are free again
  }
}

}  // namespace

bkv_status launch_cache8_evict(Cache8EvictArgs a, bool in_place, cudaStream_t stream) {
  if (injected_launch_failure()) return BKV_ERR_CUDA;
  static int done_staged[64], done_plain[64];
  a.mask_words = kMaskWords(a.max_len);
  const bool staged = a.max_len <= kStageMax;
  const int mask_bytes = 2 * 4 * a.mask_words;
  const int smem = mask_bytes + (staged ? 4 * static_cast<int>(a.max_len) : 0);
  const unsigned heads = static_cast<unsigned>(a.n_seqs) * a.n_kv_heads;
  if (staged) {
    if (!ensure_smem_limit(evict_select_kernel<true>, 200 << 10, done_staged)) return BKV_ERR_CUDA;
    evict_select_kernel<true><<<heads, kSelThreads, smem, stream>>>(a);
  } else {
    if (!ensure_smem_limit(evict_select_kernel<false>, 200 << 10, done_plain)) return BKV_ERR_CUDA;
    evict_select_kernel<false><<<heads, kSelThreads, smem, stream>>>(a);
  }
  if (cudaGetLastError() != cudaSuccess) return BKV_ERR_CUDA;
  const long long rows = std::min<long long>(a.K, a.max_len);
  long long per = (rows + kRows - 1) / kRows;
  if (in_place) {
    per = per >= 8 ? 8 : per >= 4 ? 4 : per >= 2 ? 2 : 1;  // the cluster's CTAs
    a.ctas_per_head = static_cast<int>(per);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(2 * heads * per));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = static_cast<unsigned>(per);
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, evict_compact_kernel<true>, a) != cudaSuccess) {
      cudaGetLastError();
      return BKV_ERR_CUDA;
    }
    return BKV_OK;
  }
  a.ctas_per_head = static_cast<int>(per);
  evict_compact_kernel<false><<<static_cast<unsigned>(2 * heads * per), kThreads, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? BKV_OK : BKV_ERR_CUDA;
}

}  // namespace bkv
