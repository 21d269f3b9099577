// cache8.cuh -- what the kernels of the 8-bit cache share: the e4m3 codes, the
// blocks' power-of-two scales, and the arguments each launcher takes.
//
// A cached value is code * scale: an e4m3 code per element and one scale for
// each block of `block` consecutive rows of a head.  The scale of a block whose
// largest magnitude is a is the smallest power of two s >= 2^-117 with
// a <= 448 s, so dividing by it is exact and a code is the value rounded to
// e4m3 (relative error at most 2^-4, absolute at most 2^-10 s below 2^-6 s);
// moving a code to another block's scale is exact too, but for codes that
// fall below e4m3's normal range.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace bkv {
namespace cache8 {

constexpr int kMinExp = -117;    // 448 * 2^-117 and 2^-9 * 2^-117 are normal floats

// The exponent of the scale of a block whose largest magnitude is `amax`
// (finite, >= 0): 448 = 1.75 * 2^8, so with amax = m 2^k the exponent is k - 8
// for m <= 1.75 and k - 7 above.
__device__ __forceinline__ int scale_exp(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(e, kMinExp);  // zeros and subnormals have exponent field 0
}

__device__ __forceinline__ float pow2f(int e) {  // -126 <= e <= 127
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

__device__ __forceinline__ int exp_of(float pow2) {
  return static_cast<int>(__float_as_uint(pow2) >> 23) - 127;
}

// two floats -> two e4m3 codes (lo in the low byte), round to nearest even
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// half pairs <-> code pairs; a code is exact in f16
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes16) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(codes16)));
  return r;
}
__device__ __forceinline__ uint32_t f16x2_to_e4m3x2(uint32_t h2) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h2));
  return r;
}

__device__ __forceinline__ __half2 as_half2(uint32_t x) {
  return *reinterpret_cast<__half2 *>(&x);
}
__device__ __forceinline__ uint32_t as_u32(__half2 x) { return *reinterpret_cast<uint32_t *>(&x); }

// Codes moved from one block's scale to another's, multiplied by 2^k (k = old
// exponent - new exponent).  In f16 the product is exact down to 2^-21, far
// below the 2^-10 under which e4m3 rounds to zero.  2^15 is f16's largest power:
// k > 15 (a small old code under a far smaller new scale) takes a second factor.
__device__ __forceinline__ uint32_t rescale4(uint32_t codes, __half2 f) {
  const uint32_t lo = as_u32(__hmul2(as_half2(e4m3x2_to_f16x2(codes)), f));
  const uint32_t hi = as_u32(__hmul2(as_half2(e4m3x2_to_f16x2(codes >> 16)), f));
  return f16x2_to_e4m3x2(lo) | (f16x2_to_e4m3x2(hi) << 16);
}
__device__ __forceinline__ uint4 rescale16(uint4 c, int k) {
  if (k > 15) {  // at most 17: from 2^-9 to 2^8
    const __half2 f = __float2half2_rn(pow2f(min(k, 24) - 9));
    c = make_uint4(rescale4(c.x, f), rescale4(c.y, f), rescale4(c.z, f), rescale4(c.w, f));
    k = 9;
  }
  // below 2^-24 every code becomes zero
  const __half2 f = __float2half2_rn(pow2f(max(k, -24)));
  return make_uint4(rescale4(c.x, f), rescale4(c.y, f), rescale4(c.z, f), rescale4(c.w, f));
}

// Bit 7 of each byte that is a NaN code.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t codes) {
  return ((codes & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}
__device__ __forceinline__ bool has_nan16(uint4 c) {
  return (nan_bytes(c.x) | nan_bytes(c.y) | nan_bytes(c.z) | nan_bytes(c.w)) != 0;
}
// NaN codes of a key that not every query row sees become zeros: a product with a
// probability of zero would carry them to every row.
__device__ __forceinline__ uint32_t without_nan4(uint32_t codes) {
  return codes & ~((nan_bytes(codes) >> 7) * 0xffu);
}
__device__ __forceinline__ uint4 without_nan16(uint4 c) {
  return make_uint4(without_nan4(c.x), without_nan4(c.y), without_nan4(c.z), without_nan4(c.w));
}
// The same, with put(i) called for each such element i of the 16.
template <typename Put>
__device__ __forceinline__ void hide_nan16(uint4 *codes, Put &&put) {
  if (!has_nan16(*codes)) return;
  uint8_t *byte = reinterpret_cast<uint8_t *>(codes);
#pragma unroll 1
  for (int i = 0; i < 16; ++i)
    if ((byte[i] & 0x7f) == 0x7f) {
      byte[i] = 0;
      put(i);
    }
}

__device__ __forceinline__ __half2 absmax4(uint32_t codes, __half2 m) {
  // __hmax2 returns the number where one operand is NaN, so NaN codes do not count
  m = __hmax2(m, __habs2(as_half2(e4m3x2_to_f16x2(codes))));
  return __hmax2(m, __habs2(as_half2(e4m3x2_to_f16x2(codes >> 16))));
}
__device__ __forceinline__ float absmax16(uint4 c) {
  __half2 m = __float2half2_rn(0.f);
  m = absmax4(c.w, absmax4(c.z, absmax4(c.y, absmax4(c.x, m))));
  return fmaxf(__low2float(m), __high2float(m));
}

// Programmatic dependent launch.  A kernel launched so may start while the one
// before it in the stream runs, once every CTA of that has passed
// pdl_launch_dependents or ended; pdl_wait holds it until that one has ended and
// its writes are there.  Every CTA waits before it ends, so that a kernel never
// ends before one that it follows; and a kernel that others may follow at once
// waits before it lets them start, so that what these read before their own wait
// (lengths) is complete.  One decode step's attention (28/4 heads, 8192 rows) 14.4 ->
// 13.5 us, eviction of one layer 16.4 -> 14.7, four prompts appended 36.9 -> 35.5.
__device__ __forceinline__ void pdl_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// cluster: CTAs per cluster, 1 for none
template <typename... Params, typename... Args>
bool launch_programmatic(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, int cluster,
                         cudaStream_t stream, const Args &...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess) return true;
  cudaGetLastError();
  return false;
}

}  // namespace cache8
}  // namespace bkv
