// cache8_append.cu -- new K/V rows quantised into the 8-bit cache.
//
// One CTA per (block of rows touched, sequence, KV head, K or V), or per run of
// four blocks.  A block's new rows are read once into registers, their largest
// magnitude is reduced over the CTA, the block's scale follows from it (and from
// the scale of the rows the block already holds, which never shrinks), and the
// codes are written.  Only when the scale grows are the older rows of the block
// read, moved to the new scale and written back.  A block belongs to one CTA, so
// no two CTAs touch a scale.
//
// Whole prompts are bound by HBM: 4 of 8192 rows, 8 heads of 128 in bf16, 201 MB
// in 35.5 us, 87% of the measured copy rate (40 us with a select per element for
// those that are not finite, 43 with a CTA per block, 85 with a thread per
// element).  One decode step is a launch and three dependent loads (length, scale
// and row, codes): 2.3 us in a graph, 5 us as a call, which is its time on the host.
#include <cuda_bf16.h>

#include <algorithm>

#include "bkv_check.cuh"
#include "bkv_device_status.cuh"
#include "bkv_internal.h"
#include "cache8.cuh"

BKV_DEFINE_STATUS_ACCESSOR(take_status_cache8_append)

namespace bkv {
namespace {

using namespace cache8;

constexpr int kMaxThreads = 256;
constexpr int kLongRun = 4;  // blocks a CTA takes where there are many

// 16 elements as they are stored, and as floats
template <typename T>
struct Piece;
template <>
struct Piece<float> {
  float4 v[4];
  __device__ __forceinline__ void load(const float *p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __ldcs(reinterpret_cast<const float4 *>(p) + i);
  }
  __device__ __forceinline__ float at(int i) const {
    const float4 x = v[i >> 2];
    return (i & 3) == 0 ? x.x : (i & 3) == 1 ? x.y : (i & 3) == 2 ? x.z : x.w;
  }
  // the bits of the largest |x| among the finite elements; *odd: some are not finite
  __device__ __forceinline__ uint32_t amax(bool *odd) const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t b = __float_as_uint(at(i)) & 0x7fffffffu;
      if (b < 0x7f800000u) m = max(m, b); else *odd = true;
    }
    return m;
  }
};
template <>
struct Piece<__nv_bfloat16> {
  uint32_t v[8];
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 x = __ldcs(reinterpret_cast<const uint4 *>(p) + i);
      v[4 * i] = x.x, v[4 * i + 1] = x.y, v[4 * i + 2] = x.z, v[4 * i + 3] = x.w;
    }
  }
  __device__ __forceinline__ float at(int i) const {
    return __uint_as_float(i & 1 ? v[i >> 1] & 0xffff0000u : v[i >> 1] << 16);
  }
  __device__ __forceinline__ uint32_t amax(bool *odd) const {
    // two elements at a time; infinities and NaN are the largest, so only
    // where one turns up are the elements looked at one by one
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = __vmaxu2(m, v[i] & 0x7fff7fffu);
    m = max(m & 0xffffu, m >> 16);
    if (m >= 0x7f80u) {
      *odd = true;
      m = 0;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const uint32_t b = (i & 1 ? v[i >> 1] >> 16 : v[i >> 1]) & 0x7fffu;
        if (b < 0x7f80u) m = max(m, b);
      }
    }
    return m << 16;
  }
};

// kPieces: 16-element pieces per thread, as few as the sizes allow, so that
// more CTAs are resident and more loads in flight.  kRun: blocks a CTA takes
// one after another, the next one's rows loading while one is written; the
// lengths are then waited for once in kRun blocks.
template <typename T, int kPieces, int kRun>
__global__ void __launch_bounds__(kMaxThreads) append_kernel(const Cache8AppendArgs a) {
  __shared__ uint32_t s_max[2][kMaxThreads / 32];
  unsigned u = blockIdx.x;
  const int tb = u % a.runs_per_seq;
  u /= a.runs_per_seq;
  const int kv = u & 1;
  u >>= 1;
  const int seq = u / a.n_kv_heads;
  pdl_wait();
  pdl_launch_dependents();
  const int n = a.n_new ? a.n_new[seq] : a.T;
  const int len = a.lens[seq];
  if (n < 0 || n > a.T || len < n || len > a.cap) {
    if (threadIdx.x == 0) record_device_status(BKV_DEV_ASSERT, 601);
    return;
  }
  const int first = len - n;
  const size_t head = u;                   // sequence * n_kv_heads + KV head
  const int pr = a.head_dim >> 4;          // pieces per row
  uint8_t *head_codes = (kv ? a.v8 : a.k8) + head * a.cap * static_cast<size_t>(a.head_dim);
  float *head_scale = (kv ? a.v_scale : a.k_scale) + head * (a.cap / a.block);
  const T *head_src =
      static_cast<const T *>(kv ? a.v_new : a.k_new) + head * a.T * static_cast<size_t>(a.head_dim);
  int blk = first / a.block + tb * kRun;
  const int blk_end = min(blk + kRun, (len + a.block - 1) / a.block);
  if (n == 0) return;
  // a block's new rows [r0, r1), loaded while the block before is worked on
  Piece<T> v[kPieces];
  float was = 0.f;
  auto load = [&](int blk) {
    const int base = blk * a.block, r0 = max(base, first), r1 = min(base + a.block, len);
    if (r0 > base) was = head_scale[blk];
    const T *src = head_src + static_cast<size_t>(r0 - first) * a.head_dim;
    const int pieces = (r1 - r0) * pr;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int p = threadIdx.x + i * blockDim.x;
      if (p < pieces) v[i].load(src + static_cast<size_t>(p) * 16);
    }
  };
  if (blk < blk_end && BKV_CHECK(blk >= 0 && blk < a.cap / a.block, 602)) load(blk);
#pragma unroll 1
  for (int round = 0; blk < blk_end; ++blk, ++round) {
    if (!BKV_CHECK(blk >= 0 && blk < a.cap / a.block, 602)) return;  // the whole CTA
    const int base = blk * a.block, r0 = max(base, first), r1 = min(base + a.block, len);
    const int pieces = (r1 - r0) * pr;
    uint8_t *codes = head_codes + static_cast<size_t>(base) * a.head_dim;
    uint32_t amax = 0;
    bool odd = false;
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
      if (static_cast<int>(threadIdx.x + i * blockDim.x) < pieces) amax = max(amax, v[i].amax(&odd));
    amax = __reduce_max_sync(0xffffffffu, amax);
    uint32_t *s_m = s_max[round & 1];  // its last readers are a barrier behind
    if ((threadIdx.x & 31) == 0) s_m[threadIdx.x >> 5] = amax;
    __syncthreads();
    amax = 0;
    for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) amax = max(amax, s_m[w]);
    int e = scale_exp(__uint_as_float(amax));
    const bool held = r0 > base;
    const int e_was = held ? exp_of(was) : 0;
    if (held) e = max(e, e_was);
    const float inv = pow2f(-e);
    const Piece<T> *now = v;
    Piece<T> mine[kRun > 1 ? kPieces : 1];
    if constexpr (kRun > 1) {
#pragma unroll
      for (int i = 0; i < kPieces; ++i) mine[i] = v[i];
      now = mine;
      if (blk + 1 < blk_end) load(blk + 1);
    }
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int p = threadIdx.x + i * blockDim.x;
      if (p < pieces) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          w[k] = to_e4m3x2(now[i].at(4 * k) * inv, now[i].at(4 * k + 1) * inv) |
                 (to_e4m3x2(now[i].at(4 * k + 2) * inv, now[i].at(4 * k + 3) * inv) << 16);
        if (odd) {  // elements that are not finite become NaN codes
#pragma unroll
          for (int k = 0; k < 16; ++k)
            if ((__float_as_uint(now[i].at(k)) & 0x7fffffffu) >= 0x7f800000u)
              w[k >> 2] |= 0x7fu << (8 * (k & 3));
        }
        reinterpret_cast<uint4 *>(codes)[static_cast<size_t>(r0 - base) * pr + p] =
            make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    if (held && e > e_was) {
      for (int p = threadIdx.x; p < (r0 - base) * pr; p += blockDim.x) {
        uint4 *c = reinterpret_cast<uint4 *>(codes) + p;
        *c = rescale16(*c, e_was - e);
      }
    }
    // every thread has read the old scale before the barrier above
    if (threadIdx.x == 0) head_scale[blk] = pow2f(e);
  }
}

}  // namespace

bkv_status launch_cache8_append(Cache8AppendArgs a, int dtype, cudaStream_t stream) {
  if (injected_launch_failure()) return BKV_ERR_CUDA;
  // 128 threads at least, so that older rows that have to move to a larger
  // scale move quickly; up to 128 rows x 128 / 16 = 1024 pieces
  const int pieces = std::min(a.T, a.block) * a.head_dim / 16;
  const int threads = std::min(kMaxThreads, std::max(128, (pieces + 31) / 32 * 32));
  const int per = (pieces + threads - 1) / threads;
  // several blocks a CTA where that leaves work for every SM: 4 prompts of 8192
  // rows, 8 heads of 128, 43 us with one and 40 with four
  const long long blocks = 2LL * a.n_seqs * a.n_kv_heads * a.blocks_per_seq;
  const bool many = a.blocks_per_seq >= 8 && blocks >= 4 * 148 * 8;
  a.runs_per_seq = many ? (a.blocks_per_seq + kLongRun - 1) / kLongRun : a.blocks_per_seq;
  const long long ctas = 2LL * a.n_seqs * a.n_kv_heads * a.runs_per_seq;
  if (ctas > INT32_MAX) return BKV_ERR_INVALID_ARG;
  bool ok = false;
  auto launch = [&](auto kernel) {
    ok = launch_programmatic(kernel, dim3(static_cast<unsigned>(ctas)), threads, 0, 1, stream, a);
  };
  auto pick = [&](auto type) {
    using T = decltype(type);
    if (many)
      per == 1   ? launch(append_kernel<T, 1, kLongRun>)
      : per == 2 ? launch(append_kernel<T, 2, kLongRun>)
                 : launch(append_kernel<T, 4, kLongRun>);
    else
      per == 1   ? launch(append_kernel<T, 1, 1>)
      : per == 2 ? launch(append_kernel<T, 2, 1>)
                 : launch(append_kernel<T, 4, 1>);
  };
  if (dtype == BKV_BF16)
    pick(__nv_bfloat16{});
  else
    pick(float{});
  return ok ? BKV_OK : BKV_ERR_CUDA;
}

}  // namespace bkv
