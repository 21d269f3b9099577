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
// Compaction: a CTA takes 128 new rows of one (sequence, head), K and V, which
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
constexpr int kMaskWords(long long L) { return static_cast<int>((L + 127) / 128 * 4); }

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
      // four positions a thread and step, kBatch steps' loads in flight; a row
      // is 16-byte aligned and allocated to a multiple of 16 positions
      constexpr int kBatch = 4;
      const int quads = (L + 3) >> 2;
      for (int q0 = tid; q0 < quads; q0 += kBatch * kSelThreads) {
        uint4 k[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const int q = q0 + u * kSelThreads;
          if (q >= quads) continue;
          if (kStaged && pass > 0) {
            k[u] = reinterpret_cast<const uint4 *>(s_key)[q];
          } else {
            const float4 f = __ldg(reinterpret_cast<const float4 *>(w) + q);
            k[u] = make_uint4(rank_key(f.x), rank_key(f.y), rank_key(f.z), rank_key(f.w));
            if (kStaged) reinterpret_cast<uint4 *>(s_key)[q] = k[u];
          }
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const int q = q0 + u * kSelThreads;
          if (q >= quads) continue;
          const uint32_t v[4] = {k[u].x, k[u].y, k[u].z, k[u].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int j = 4 * q + i;
            if (j >= lo && j < hi && (pass == 0 || (v[i] >> (shift + bits)) == prefix))
              atomicAdd(&s_hist[(v[i] >> shift) & ((1u << bits) - 1)], 1u);
          }
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
constexpr int kPieces = 4;     // 16-byte pieces of K, and of V, per thread: 128 rows x 8 / 256

// kPr: 16-byte pieces per row when it is a power of two (8, 4), 0: any number.
template <bool kInPlace, int kPr>
__global__ void __launch_bounds__(kThreads) evict_compact_kernel(const Cache8EvictArgs a) {
  __shared__ int32_t s_idx[kRows];
  __shared__ int s_exp[2][kRows];           // the rows' old scale exponents (K, V)
  __shared__ uint32_t s_max[2][kRows / 16]; // per new block: bits of the largest magnitude
  const int tid = threadIdx.x;
  const int head = blockIdx.x / a.ctas_per_head;
  const int part = blockIdx.x - head * a.ctas_per_head;  // in place: the rank in the cluster
  const int seq = head / a.n_kv_heads;
  const int n = a.kept[seq];
  if (part == 0 && tid == 0 && head - seq * a.n_kv_heads == 0 && n >= 0 && a.new_lens)
    a.new_lens[seq] = n;
  const int pr = kPr ? kPr : a.head_dim >> 4;
  const int lb = a.log2_block;
  const size_t D = a.head_dim;
  const size_t src0 = static_cast<size_t>(head) * a.cap * D;
  const size_t dst0 = static_cast<size_t>(head) * a.dst_cap * D;
  const size_t ssc0 = static_cast<size_t>(head) * (a.cap >> lb);
  const size_t dsc0 = static_cast<size_t>(head) * (a.dst_cap >> lb);
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
    // threads 0..127: the rows' positions and K scales, the others the V scales
    const int lr = tid & (kRows - 1);
    float wv = 0.f;
    if (lr < rows) {
      const int j = idx[base + lr];
      const float *sc = (tid < kRows ? a.k_scale : a.v_scale) + ssc0 + (j >> lb);
      s_exp[tid >= kRows][lr] = exp_of(kInPlace ? __ldcg(sc) : __ldg(sc));
      if (tid < kRows) {
        s_idx[lr] = j;
        if (w_dst) wv = kInPlace ? __ldcg(w_src + j) : __ldg(w_src + j);
      }
    }
    if (tid < 2 * (kRows / 16)) s_max[tid / (kRows / 16)][tid % (kRows / 16)] = 0;
    __syncthreads();
    uint4 c[2][kPieces];
    const int pieces = rows * pr;
    auto row_of = [&](int p) { return kPr == 8 ? p >> 3 : kPr == 4 ? p >> 2 : p / pr; };
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int p = tid + i * kThreads;
      if (p < pieces) {
        const int r = row_of(p);
        const size_t off = src0 + static_cast<size_t>(s_idx[r]) * D + (p - r * pr) * 16;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          const uint4 *q = reinterpret_cast<const uint4 *>((kv ? a.v8 : a.k8) + off);
          c[kv][i] = kInPlace ? __ldcg(q) : __ldcs(q);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int p = tid + i * kThreads;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        uint32_t m = 0;
        if (p < pieces) m = __float_as_uint(absmax16(c[kv][i]) * pow2f(s_exp[kv][row_of(p)]));
        if (kPr != 0) {  // a warp's rows (4 or 8, aligned) lie in one block
          m = __reduce_max_sync(0xffffffffu, m);
          if ((tid & 31) == 0 && p < pieces) atomicMax(&s_max[kv][row_of(p) >> lb], m);
        } else if (p < pieces) {
          atomicMax(&s_max[kv][row_of(p) >> lb], m);
        }
      }
    }
    // every read of this round has returned in every CTA before any write
    if (kInPlace) cg::this_cluster().sync(); else __syncthreads();
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int p = tid + i * kThreads;
      if (p < pieces) {
        const int r = row_of(p);
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          const int k = s_exp[kv][r] - scale_exp(__uint_as_float(s_max[kv][r >> lb]));
          if (k != 0) c[kv][i] = rescale16(c[kv][i], k);
          uint4 *q = reinterpret_cast<uint4 *>((kv ? a.v8_dst : a.k8_dst) + dst0 +
                                               static_cast<size_t>(base) * D) + p;
          if (kInPlace) __stcg(q, c[kv][i]); else __stcs(q, c[kv][i]);
        }
      }
    }
    if (lr < rows) {
      if ((lr & (a.block - 1)) == 0)
        (tid < kRows ? a.k_scale_dst : a.v_scale_dst)[dsc0 + ((base + lr) >> lb)] =
            pow2f(scale_exp(__uint_as_float(s_max[tid >= kRows][lr >> lb])));
      if (tid < kRows && w_dst) w_dst[base + lr] = wv;
    }
    if (kInPlace) __syncthreads();  // s_idx, s_exp and s_max are free again
  }
}

template <bool kInPlace>
auto compact_kernel_for(int head_dim) {
  return head_dim == 128  ? evict_compact_kernel<kInPlace, 8>
         : head_dim == 64 ? evict_compact_kernel<kInPlace, 4>
                          : evict_compact_kernel<kInPlace, 0>;
}

}  // namespace

bkv_status launch_cache8_evict(Cache8EvictArgs a, bool in_place, cudaStream_t stream) {
  if (injected_launch_failure()) return BKV_ERR_CUDA;
  static int done_staged[64], done_plain[64];
  a.mask_words = kMaskWords(a.max_len);
  a.log2_block = a.block == 16 ? 4 : a.block == 32 ? 5 : a.block == 64 ? 6 : 7;
  const bool staged = a.max_len <= kStageMax;
  const int mask_bytes = 2 * 4 * a.mask_words;
  const int smem = mask_bytes + (staged ? 4 * static_cast<int>((a.max_len + 3) / 4 * 4) : 0);
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
    cfg.gridDim = dim3(static_cast<unsigned>(heads * per));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = static_cast<unsigned>(per);
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, compact_kernel_for<true>(a.head_dim), a) != cudaSuccess) {
      cudaGetLastError();
      return BKV_ERR_CUDA;
    }
    return BKV_OK;
  }
  a.ctas_per_head = static_cast<int>(per);
  auto kernel = compact_kernel_for<false>(a.head_dim);
  kernel<<<static_cast<unsigned>(heads * per), kThreads, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? BKV_OK : BKV_ERR_CUDA;
}

}  // namespace bkv
