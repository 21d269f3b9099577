// cache8_evict.cu -- eviction from the 8-bit cache by accumulated attention
// weight: which rows stay (evict_select_kernel), and their compaction
// (evict_compact_kernel).
//
// Select: one CTA per (sequence, KV head).  A row of L > K positions keeps the
// first `sink`, the last `recent` and, of the rest, the K - sink - recent with
// the largest weights, ties to the lower position.  The row is read three
// times, from HBM once and then from L2, so that it takes no shared memory and
// several CTAs share an SM: a histogram of the weights' top 11 bits gives the
// bin of the threshold; the order-preserving keys (order_key.cuh) of that bin,
// a few percent, are listed in shared memory and two more radix steps over the
// list give the threshold and how many of its ties stay; last, each warp turns
// 1024 positions into 32 mask words by ballots, drops surplus ties by a prefix
// sum, and writes the kept positions in ascending order, a coalesced store per
// word.  Bound by instruction issue (a row is 4 bytes a position), so the inner
// loops take the weights as they are: bins by raw bits, put in order when they
// are summed, comparisons as floats, and no range checks but in the chunks
// where the candidates begin and end.  Measured: 288 rows of 8192 positions in 18
// us, 320 of 32768 in 48 (issue at 54% and more, 80% in the histogram; one row
// alone 12 us, a chain of some twenty barriers).
//
// Compaction: a CTA takes 128 new rows of one (sequence, head), K and V, which
// are whole blocks of the new cache.  It gathers the rows' codes and old
// scales, reduces each new block's largest magnitude (exact: a code times a
// power of two), takes the scale that the append would take, moves the codes
// of the rows whose scale differs and writes them.  In place, a cluster of
// CTAs reads up to 8 x 128 rows, meets at the cluster barrier and only then
// writes them: new row i takes old row idx_i >= i, so every row, scale and
// weight a later round reads lies at or past that round's first row.  Bound by
// HBM: 36 x 8 heads, 8192 rows of 128 to 4096, 97 us, 96% of the measured copy
// rate.  In place, where a cluster's reads wait for its writes, the whole eviction takes
// 150 us and 119 to another buffer (40 x 8 heads, 32768 rows to 6144: 266 and 217).
#include <cooperative_groups.h>

#include <algorithm>

#include "bkv_check.cuh"
#include "bkv_device_status.cuh"
#include "bkv_internal.h"
#include "cache8.cuh"
#include "order_key.cuh"

BKV_DEFINE_STATUS_ACCESSOR(take_status_cache8_evict)

namespace bkv {
namespace {

using namespace cache8;
namespace cg = cooperative_groups;

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kListMax = 8192;  // keys of the threshold's bin that are listed

// A weight as it is ranked: NaN as -infinity, -0 as +0.
__device__ __forceinline__ float ranked(float w) { return fmaxf(w + 0.f, -INFINITY); }
// Bins of raw bits, and the order of their values: negative floats (bins 1024
// and up) fall as their bits rise.
__device__ __forceinline__ uint32_t bin_of(float v) { return __float_as_uint(v) >> 21; }

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
  uint32_t t = lane < kSelWarps ? s_warp[lane] : 0u;  // every warp sums for itself
#pragma unroll
  for (int o = 1; o < kSelWarps; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, t, o);
    if (lane >= o) t += y;
  }
  *total = __shfl_sync(0xffffffffu, t, kSelWarps - 1);
  const uint32_t before = __shfl_sync(0xffffffffu, t, max(warp - 1, 0));
  return x - v + (warp ? before : 0u);
}

// The bin of the histogram that holds the need-th largest value; need becomes
// its rank within the bin.  kRaw: bins of raw bits, else of keys.  Leaves the
// histogram zeroed.
template <bool kRaw>
__device__ __forceinline__ uint32_t find_bin(uint32_t *s_hist, uint32_t *s_warp, uint32_t *s_bin,
                                             uint32_t *need) {
  // suffix counts: four bins a thread, the largest values first
  const int top = kBins - 4 - 4 * static_cast<int>(threadIdx.x);  // the four: top + 3 .. top
  const bool neg = kRaw && top < 1024;
  const int b = !kRaw ? top : neg ? 2044 - top : top - 1024;      // where they are
  const uint4 c = *reinterpret_cast<const uint4 *>(s_hist + b);
  *reinterpret_cast<uint4 *>(s_hist + b) = make_uint4(0, 0, 0, 0);
  uint32_t total;
  uint32_t above = block_scan(c.x + c.y + c.z + c.w, s_warp, &total);
  const uint32_t n[4] = {neg ? c.x : c.w, neg ? c.y : c.z, neg ? c.z : c.y, neg ? c.w : c.x};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (above < *need && *need <= above + n[i]) {
      s_bin[0] = static_cast<uint32_t>(neg ? b + i : b + 3 - i);
      s_bin[1] = above;
    }
    above += n[i];
  }
  __syncthreads();
  *need -= s_bin[1];
  return s_bin[0];
}

// Calls f(t, v) for the ranked weights of the row that are candidates, and
// done(first position, bits) after every kBatch * 4 of a lane, with the bits t
// for which f returned true: bit t is position first + 4 * kSelThreads * (t / 4)
// + t % 4.  Loads of a batch are in flight together; range checks only in the
// chunks of 128 positions where the candidates begin or end.
constexpr int kBatch = 4;
template <typename F, typename Done>
__device__ __forceinline__ void for_weights(const float *w, int L, int lo, int hi, F &&f, Done &&done) {
  const unsigned quads = (static_cast<unsigned>(L) + 3) >> 2;  // a row is allocated to whole quads
  const unsigned first = threadIdx.x & ~31u, lane = threadIdx.x & 31u;
  const unsigned l = static_cast<unsigned>(lo), h = static_cast<unsigned>(hi);
  for (unsigned q0 = first; q0 < quads; q0 += kBatch * kSelThreads) {
    float4 v[kBatch];
    uint32_t bits = 0;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const unsigned q = q0 + u * kSelThreads + lane;
      if (q < quads) v[u] = __ldg(reinterpret_cast<const float4 *>(w) + q);
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const unsigned j0 = 4 * (q0 + u * kSelThreads);  // this warp's 128 positions
      if (j0 >= h || j0 + 128 <= l) continue;
      const float y[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
      const bool inner = j0 >= l && j0 + 128 <= h;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const unsigned j = j0 + 4 * lane + i;
        if ((inner || (j >= l && j < h)) && f(ranked(y[i]))) bits |= 1u << (4 * u + i);
      }
    }
    done(4 * (q0 + lane), bits);
  }
}

__global__ void __launch_bounds__(kSelThreads, 3) evict_select_kernel(const Cache8EvictArgs a) {
  __shared__ __align__(16) uint32_t s_hist[kBins];
  __shared__ uint32_t s_list[kListMax];
  __shared__ uint32_t s_warp[kSelWarps];
  __shared__ uint32_t s_bin[2], s_count;
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
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
  float thr = INFINITY;  // keep weights > thr, and the first `ties` equal to it
  uint32_t ties = 0;
  if (need > 0) {
    for (int b = tid; b < kBins; b += kSelThreads) s_hist[b] = 0;
    if (tid == 0) s_count = 0;
    __syncthreads();
    for_weights(
        w, L, lo, hi,
        [&](float v) {
          atomicAdd(&s_hist[bin_of(v)], 1u);
          return false;
        },
        [](unsigned, uint32_t) {});
    __syncthreads();
    const uint32_t raw = find_bin<true>(s_hist, s_warp, s_bin, &need);
    // the bin's keys, listed, and their next 11 bits counted: found first, then
    // read again one by one, a few of a lane's 16
    for_weights(
        w, L, lo, hi, [&](float v) { return bin_of(v) == raw; },
        [&](unsigned j, uint32_t bits) {
          while (bits) {
            const int t = __ffs(bits) - 1;
            bits &= bits - 1;
            const unsigned at_w = j + 4 * kSelThreads * (t >> 2) + (t & 3);
            if (!BKV_CHECK(at_w < static_cast<unsigned>(L), 623)) continue;
            const uint32_t k = order_key(ranked(__ldg(w + at_w)));
            atomicAdd(&s_hist[(k >> 10) & 2047u], 1u);
            const uint32_t at = atomicAdd(&s_count, 1u);
            if (at < kListMax) s_list[at] = k;
          }
        });
    __syncthreads();
    const uint32_t top = raw < 1024 ? 1024 + raw : 2047 - raw;  // the bin's keys' top bits
    const uint32_t mid = (top << 11) | find_bin<false>(s_hist, s_warp, s_bin, &need);
    const uint32_t n = s_count;
    if (n <= kListMax) {
      for (uint32_t i = tid; i < n; i += kSelThreads)
        if ((s_list[i] >> 10) == mid) atomicAdd(&s_hist[s_list[i] & 1023u], 1u);
    } else {  // a crowded bin: the row again
      for_weights(
          w, L, lo, hi,
          [&](float v) {
            const uint32_t k = order_key(v);
            if ((k >> 10) == mid) atomicAdd(&s_hist[k & 1023u], 1u);
            return false;
          },
          [](unsigned, uint32_t) {});
    }
    __syncthreads();
    thr = key_value((mid << 10) | find_bin<false>(s_hist, s_warp, s_bin, &need));
    ties = need;
  }
  // Kept positions, 1024 a warp at a time: in step t of 8 a lane has positions
  // 128 t + 4 lane .. + 3, bits 4 t .. 4 t + 3 of its words.
  const unsigned lt = (1u << lane) - 1;
  uint32_t ties_before = 0, at0 = 0;
  for (unsigned base = 0; base < static_cast<unsigned>(L); base += 1024u * kSelWarps) {
    const unsigned jw = base + 1024u * warp, j0 = jw + 4 * lane;
    const unsigned l = static_cast<unsigned>(lo), h = static_cast<unsigned>(hi);
    uint32_t keep = 0, tie = 0;
    const bool inner = ties > 0 && jw >= l && jw + 1024 <= h;
    if (inner || jw < static_cast<unsigned>(L)) {
#pragma unroll 1
      for (int t0 = 0; t0 < 8; t0 += 4) {  // four loads in flight, within 40 registers
        float4 v[4];
#pragma unroll
        for (int t = 0; t < 4; ++t)  // a row is allocated to whole quads
          if (inner || j0 + 128 * (t0 + t) < static_cast<unsigned>(L))
            v[t] = __ldg(reinterpret_cast<const float4 *>(w + j0 + 128 * (t0 + t)));
        uint32_t k = 0, e = 0;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const float y[4] = {v[t].x, v[t].y, v[t].z, v[t].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float x = fmaxf(y[i], -INFINITY);
            if (x > thr) k |= 1u << (4 * t + i);
            if (x == thr) e |= 1u << (4 * t + i);
          }
        }
        keep |= k << (4 * t0);
        tie |= e << (4 * t0);
      }
      if (!inner) {  // the sink and the recent rows, and what lies past the end
        uint32_t cand = 0, there = 0;
#pragma unroll 1
        for (int t = 0; t < 32; ++t) {
          const unsigned j = j0 + 128 * (t >> 2) + (t & 3);
          if (j < static_cast<unsigned>(L)) there |= 1u << t;
          if (j >= l && j < h) cand |= 1u << t;
        }
        // without a candidate to keep (ties == 0) the threshold is infinity
        keep = (ties > 0 ? keep & cand : 0u) | (there & ~cand);
        tie &= ties > 0 ? cand : 0u;
      }
    }
    uint32_t total;
    // ties, in position order; most rows have no more than they keep
    const uint32_t mine = __reduce_add_sync(0xffffffffu, static_cast<unsigned>(__popc(tie)));
    uint32_t rank = ties_before + block_scan(lane == 0 ? mine : 0u, s_warp, &total);
    rank = __shfl_sync(0xffffffffu, rank, 0);  // ties before this warp's
    ties_before += total;
    if (rank + mine <= ties) {
      keep |= tie;
    } else if (rank < ties) {
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        const uint32_t n = (tie >> (4 * t)) & 15u;
        uint32_t before = 0, all = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const unsigned m = __ballot_sync(0xffffffffu, (n >> i) & 1u);
          before += __popc(m & lt);
          all += __popc(m);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if ((n >> i) & 1u) {
            if (rank + before < ties) keep |= 1u << (4 * t + i);
            ++before;
          }
        rank += all;
      }
    }
    const uint32_t kept = __reduce_add_sync(0xffffffffu, static_cast<unsigned>(__popc(keep)));
    uint32_t at = at0 + block_scan(lane == 0 ? kept : 0u, s_warp, &total);
    at = __shfl_sync(0xffffffffu, at, 0);
    at0 += total;
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      const uint32_t n = (keep >> (4 * t)) & 15u;
      uint32_t o = at;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const unsigned m = __ballot_sync(0xffffffffu, (n >> i) & 1u);
        o += __popc(m & lt);
        at += __popc(m);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if ((n >> i) & 1u) {
          const unsigned j = j0 + 128 * t + i;
          if (BKV_CHECK(o < static_cast<uint32_t>(K) && j < static_cast<unsigned>(L), 622))
            idx[o] = static_cast<int32_t>(j);
          ++o;
        }
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
  // launched while the select kernel ends: nothing of its is read before this.
  // The next kernel starts when this one ends: its CTAs beside the last of these
  // cost more than they win (36 layers of 8192 rows 120 us, and 117)
  pdl_wait();
  int n = a.kept[seq];
  if (!BKV_CHECK(n <= a.K && n <= a.dst_cap, 624)) n = -1;
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
      int j = idx[base + lr];
      // ascending positions, so that no row is overwritten before it is read
      if (!BKV_CHECK(j >= base + lr && j < a.cap, 625)) j = base + lr;
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
  a.log2_block = a.block == 16 ? 4 : a.block == 32 ? 5 : a.block == 64 ? 6 : 7;
  const unsigned heads = static_cast<unsigned>(a.n_seqs) * a.n_kv_heads;
  if (!launch_programmatic(evict_select_kernel, dim3(heads), kSelThreads, 0, 1, stream, a))
    return BKV_ERR_CUDA;
  const long long rows = std::min<long long>(a.K, a.max_len);
  long long per = (rows + kRows - 1) / kRows;
  if (in_place) per = per >= 8 ? 8 : per >= 4 ? 4 : per >= 2 ? 2 : 1;  // the cluster's CTAs
  a.ctas_per_head = static_cast<int>(per);
  const dim3 grid(static_cast<unsigned>(heads * per));
  auto kernel = in_place ? compact_kernel_for<true>(a.head_dim) : compact_kernel_for<false>(a.head_dim);
  const int cluster = in_place ? static_cast<int>(per) : 1;
  return launch_programmatic(kernel, grid, kThreads, 0, cluster, stream, a) ? BKV_OK : BKV_ERR_CUDA;
}

}  // namespace bkv
