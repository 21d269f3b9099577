// cache8_append.cu -- new K/V rows quantised into the 8-bit cache.
//
// One CTA per (block of rows touched, sequence, KV head, K or V).  The block's
// new rows are read once into registers, their largest magnitude is reduced
// over the CTA, the block's scale follows from it (and from the scale of the
// rows the block already holds, which never shrinks), and the codes are
// written.  Only when the scale grows are the older rows of the block read,
// moved to the new scale and written back.  A block belongs to one CTA, so no
// two CTAs touch a scale.  Bound by HBM for whole prompts; one decode step is
// a launch and three dependent loads (length, scale and row, codes).
#include <cuda_bf16.h>

#include <algorithm>

#include "bkv_device_status.cuh"
#include "bkv_internal.h"
#include "cache8.cuh"

BKV_DEFINE_STATUS_ACCESSOR(take_status_cache8_append)

namespace bkv {
namespace {

using namespace cache8;

constexpr int kMaxThreads = 256;

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

// A value that is not finite becomes a NaN code.
__device__ __forceinline__ float storable(float x, float inv, bool odd) {
  const float y = x * inv;
  if (odd && (__float_as_uint(x) & 0x7fffffffu) >= 0x7f800000u) return __uint_as_float(0x7fc00000u);
  return y;
}

// kPieces: 16-element pieces per thread, as few as the sizes allow, so that
// more CTAs are resident and more loads in flight.
template <typename T, int kPieces>
__global__ void __launch_bounds__(kMaxThreads) append_kernel(const Cache8AppendArgs a) {
  __shared__ uint32_t s_max[kMaxThreads / 32];
  unsigned u = blockIdx.x;
  const int tb = u % a.blocks_per_seq;
  u /= a.blocks_per_seq;
  const int kv = u & 1;
  u >>= 1;
  const int seq = u / a.n_kv_heads;
  const int n = a.n_new ? a.n_new[seq] : a.T;
  const int len = a.lens[seq];
  if (n < 0 || n > a.T || len < n || len > a.cap) {
    if (threadIdx.x == 0) record_device_status(BKV_DEV_ASSERT, 601);
    return;
  }
  const int first = len - n;
  const int blk = first / a.block + tb;
  const int base = blk * a.block;          // first row of the block
  const int r0 = max(base, first);         // its new rows: [r0, r1)
  const int r1 = min(base + a.block, len);
  if (r0 >= r1) return;
  const size_t head = u;                   // sequence * n_kv_heads + KV head
  const int pr = a.head_dim >> 4;          // pieces per row
  uint8_t *codes = (kv ? a.v8 : a.k8) + (head * a.cap + base) * static_cast<size_t>(a.head_dim);
  float *scale = (kv ? a.v_scale : a.k_scale) + head * (a.cap / a.block) + blk;
  const T *src = static_cast<const T *>(kv ? a.v_new : a.k_new) +
                 (head * a.T + (r0 - first)) * static_cast<size_t>(a.head_dim);
  const float was = r0 > base ? *scale : 0.f;
  const int pieces = (r1 - r0) * pr;
  Piece<T> v[kPieces];
  uint32_t amax = 0;
  bool odd = false;
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int p = threadIdx.x + i * blockDim.x;
    if (p < pieces) v[i].load(src + static_cast<size_t>(p) * 16);
  }
#pragma unroll
  for (int i = 0; i < kPieces; ++i)
    if (static_cast<int>(threadIdx.x + i * blockDim.x) < pieces) amax = max(amax, v[i].amax(&odd));
  amax = __reduce_max_sync(0xffffffffu, amax);
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = amax;
  __syncthreads();
  amax = 0;
  for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) amax = max(amax, s_max[w]);
  int e = scale_exp(__uint_as_float(amax));
  const bool held = r0 > base;
  const int e_was = held ? exp_of(was) : 0;
  if (held) e = max(e, e_was);
  const float inv = pow2f(-e);
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int p = threadIdx.x + i * blockDim.x;
    if (p < pieces) {
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        w[k] = to_e4m3x2(storable(v[i].at(4 * k), inv, odd), storable(v[i].at(4 * k + 1), inv, odd)) |
               (to_e4m3x2(storable(v[i].at(4 * k + 2), inv, odd),
                          storable(v[i].at(4 * k + 3), inv, odd)) << 16);
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
  if (threadIdx.x == 0) *scale = pow2f(e);
}

}  // namespace

bkv_status launch_cache8_append(const Cache8AppendArgs &a, int dtype, cudaStream_t stream) {
  if (injected_launch_failure()) return BKV_ERR_CUDA;
  const long long ctas = 2LL * a.n_seqs * a.n_kv_heads * a.blocks_per_seq;
  if (ctas > INT32_MAX) return BKV_ERR_INVALID_ARG;
  // 128 threads at least, so that older rows that have to move to a larger
  // scale move quickly; up to 128 rows x 128 / 16 = 1024 pieces
  const int pieces = std::min(a.T, a.block) * a.head_dim / 16;
  const int threads = std::min(kMaxThreads, std::max(128, (pieces + 31) / 32 * 32));
  const int per = (pieces + threads - 1) / threads;
  auto launch = [&](auto kernel) {
    kernel<<<static_cast<unsigned>(ctas), threads, 0, stream>>>(a);
  };
  if (dtype == BKV_BF16)
    per == 1   ? launch(append_kernel<__nv_bfloat16, 1>)
    : per == 2 ? launch(append_kernel<__nv_bfloat16, 2>)
               : launch(append_kernel<__nv_bfloat16, 4>);
  else
    per == 1   ? launch(append_kernel<float, 1>)
    : per == 2 ? launch(append_kernel<float, 2>)
               : launch(append_kernel<float, 4>);
  return cudaGetLastError() == cudaSuccess ? BKV_OK : BKV_ERR_CUDA;
}

}  // namespace bkv
