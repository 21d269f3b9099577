// cache8_weights_tc.cu -- attention weights over the 8-bit cache from the rows'
// lse, for more query rows than logits are kept of (bf16 queries, head_dim 64
// or 128): w_j = decay * w_in_j + sum_r exp(x_rj - lse_r).
//
// A CTA holds 128 keys of a (sequence, KV head) as the A operand, its codes
// turned into bf16 once (exact), and walks the query rows 128 at a time: TMA
// brings them as they are (bf16, one query head's tokens after another's; the
// sum does not ask for the order), 128 tokens of a head, or where T is below 128 as
// many heads' as follow each other (8 sequences to 8192 rows, 32/8 heads, 10 tokens:
// 92 us a head at a time, 46 so).  D[128 keys][128 rows] is formed on
// tcgen05 into one of two TMEM accumulators, and the four epilogue warps of that
// accumulator, a key a lane, add exp2(s f - z_r): f, the key's factor, is the
// lane's own, z_r comes from shared memory.  Two CTAs an SM, so that one's
// beginning and waits lie under the other's exps.
//
// Bound by exp: 16384 of them a tile, 1024 cycles at 16 a cycle, against 512 of
// MMA.  1024 tokens of 40/8 heads over 16384 rows: 235 to 239 us, exp's unit at work 78%
// of the time (271 us with four epilogue warps a CTA; the second product's own
// floor is 101 us of MMA and 140 of exp).  Keeping the logits instead would move
// 2 x 2.7 GB, 830 us at the measured copy rate.
#include <cuda_bf16.h>

#include <cfloat>

#include "bkv_check.cuh"
#include "bkv_device_status.cuh"
#include "cache8_attend.cuh"
#include "sm100.cuh"
#include "tma_host.h"

BKV_DEFINE_STATUS_ACCESSOR(take_status_cache8_weights_tc)

namespace bkv {
namespace {

using namespace cache8;
using namespace sm100;

enum : int { kWhereProd = 641, kWhereMma = 642, kWhereEpi = 643, kWhereDrain = 644 };

constexpr int kEpiWarps = 8;       // four per accumulator
constexpr int kThreads = (kEpiWarps + 2) * 32;  // and TMA, MMA
constexpr int kHalf = 128 * 128;   // bytes of 128 rows x 64 bf16

template <int D>
struct WCfg {
  static constexpr int kTileBytes = (D / 64) * kHalf;
  static constexpr int kStages = 2;
  static constexpr int kSmem = (1 + kStages) * kTileBytes + 1024;
};

struct WShared {
  uint64_t full[2], empty[2], tfull[2], tempty[2], drain;
  uint32_t tmem;
  alignas(16) float z[2][128];  // minus the lse of the rows of two tiles
  int token[2][128];            // and their tokens, INT32_MIN for none
  float sum[128];               // the odd tiles' part of the keys' sums
};

// two e4m3 codes -> two bf16, exact
__device__ __forceinline__ uint32_t e4m3x2_to_bf16x2(uint32_t codes16) {
  const float2 f = __half22float2(as_half2(e4m3x2_to_f16x2(codes16)));
  const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// kFlat: T < 128, tiles over the heads' tokens
template <int D, bool kFlat>
__global__ void __launch_bounds__(kThreads, 2)
    weights_tc_kernel(const AttendArgs p, const __grid_constant__ CUtensorMap q_map) {
  using Cfg = WCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ WShared sh;
  pdl_wait();
  const Cache8AttendArgs &a = p.a;
  const size_t head = blockIdx.y;
  const int seq = static_cast<int>(head) / a.n_kv_heads;
  const int kvh = static_cast<int>(head) - seq * a.n_kv_heads;
  const SeqInfo q = seq_info(a, seq);
  const int j0 = blockIdx.x * kTile;
  if (q.tiles == 0 || j0 >= q.len) return;
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t *s_k = smem, *s_q = s_k + Cfg::kTileBytes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // tiles of 128 tokens of a query head, from the first whose last token sees
  // one of these keys; of 128 rows over the heads' tokens for few tokens
  const int seen0 = q.len - q.n + 1;
  const int t_tiles = (q.n + 127) / 128;
  const int tb0 = max(0, (j0 - seen0 + 1) >> 7);
  const int per_head = max(t_tiles - tb0, 0);
  const int n_tiles = kFlat ? (a.group * a.T + 127) / 128 : per_head * a.group;

  if (warp == kEpiWarps + 1) {
    tmem_alloc(smem_u32(&sh.tmem), 256);
    tmem_relinquish();
    if (lane == 0) {
      for (int i = 0; i < 2; ++i) {
        mbar_init(smem_u32(&sh.full[i]), 1);
        mbar_init(smem_u32(&sh.empty[i]), 1);
        mbar_init(smem_u32(&sh.tfull[i]), 1);
        mbar_init(smem_u32(&sh.tempty[i]), 4);
      }
      mbar_init(smem_u32(&sh.drain), 1);
      fence_barrier_init();
    }
  }
  if (warp < kEpiWarps) {  // the keys' codes as bf16; keys past the end are zeros
    const uint4 *src = reinterpret_cast<const uint4 *>(a.k8 + (head * a.cap + j0) * D);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const int id = i * 256 + threadIdx.x;
      const int row = id / (D / 16), ch = id % (D / 16);
      uint4 c = make_uint4(0, 0, 0, 0);
      if (j0 + row < q.len) c = __ldg(src + id);
      const uint32_t w[4] = {c.x, c.y, c.z, c.w};
      uint32_t h[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        h[2 * k] = e4m3x2_to_bf16x2(w[k]);
        h[2 * k + 1] = e4m3x2_to_bf16x2(w[k] >> 16);
      }
      uint8_t *half = s_k + (ch >> 2) * kHalf;
      *reinterpret_cast<uint4 *>(half + sw128_offset(row, (ch & 3) * 2)) =
          make_uint4(h[0], h[1], h[2], h[3]);
      *reinterpret_cast<uint4 *>(half + sw128_offset(row, (ch & 3) * 2 + 1)) =
          make_uint4(h[4], h[5], h[6], h[7]);
    }
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;

  if (warp == kEpiWarps) {
    if (lane == 0) {
      prefetch_tensormap(&q_map);
      int it = 0;
      for (; it < n_tiles; ++it) {
        const int s = it & 1;
        if (!mbar_wait(smem_u32(&sh.empty[s]), ((it >> 1) & 1) ^ 1, kWhereProd)) break;
        const int g = kFlat ? 0 : it / per_head;
        const int r0 = kFlat ? it * 128 : g * a.T + (tb0 + it - g * per_head) * 128;
        const long long row = (static_cast<long long>(seq) * a.n_q_heads + kvh * a.group) * a.T + r0;
        mbar_arrive_expect_tx(smem_u32(&sh.full[s]), Cfg::kTileBytes);
#pragma unroll
        for (int h = 0; h < D / 64; ++h)
          tma_load_2d(smem_u32(s_q) + s * Cfg::kTileBytes + h * kHalf, &q_map, smem_u32(&sh.full[s]),
                      h * 64, static_cast<int>(row));
      }
      // loads that no MMA waited for must not outlive the CTA
      for (int t = max(it - 2, 0); t < it; ++t)
        mbar_wait(smem_u32(&sh.full[t & 1]), (t >> 1) & 1, kWhereDrain);
    }
  } else if (warp == kEpiWarps + 1) {
    constexpr uint32_t idesc = idesc_bf16_f32(128, 128);
    const uint64_t k_desc = smem_desc_k_sw128(smem_u32(s_k)), q_desc = smem_desc_k_sw128(smem_u32(s_q));
    for (int it = 0; it < n_tiles; ++it) {
      const int s = it & 1;
      if (!mbar_wait_warp(smem_u32(&sh.full[s]), (it >> 1) & 1, kWhereMma)) break;
      if (!mbar_wait_warp(smem_u32(&sh.tempty[s]), ((it >> 1) & 1) ^ 1, kWhereMma)) break;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = ((k >> 2) * kHalf + (k & 3) * 32) >> 4;
          umma_f16(tmem + 128u * s, k_desc + off, q_desc + s * (Cfg::kTileBytes >> 4) + off, idesc,
                   k != 0);
        }
        umma_commit(smem_u32(&sh.empty[s]));
        umma_commit(smem_u32(&sh.tfull[s]));
      }
      __syncwarp();
    }
    if (elect_one()) umma_commit(smem_u32(&sh.drain));
    __syncwarp();
    mbar_wait_warp(smem_u32(&sh.drain), 0, kWhereDrain);
  } else {
    const int s = warp >> 2, row = threadIdx.x & 127;  // accumulator, and tiles s, s + 2, ..
    const int key = j0 + row;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const float f = fminf(
        __ldg(a.k_scale + head * (a.cap >> p.log2_block) + (min(key, q.len - 1) >> p.log2_block)) *
            (a.scale * kLog2e),
        FLT_MAX);
    const float *lse2 = p.lse2 + head * a.group * a.T;
    float z_next = 0.f;
    int t_next = INT32_MIN;
    auto row_of = [&](int it) {  // this thread's row of tile it
      const int r = it * 128 + row, g = kFlat ? r / a.T : it / per_head;
      const int t = kFlat ? r - g * a.T : (tb0 + it - g * per_head) * 128 + row;
      const bool there = g < a.group && t < q.n;
      const float z = there && BKV_CHECK(t >= 0 && t < a.T, 645) ? __ldg(lse2 + t * a.group + g) : 0.f;
      z_next = z == -INFINITY ? z : -z;  // a row of logits of -infinity adds nothing
      t_next = there ? t : INT32_MIN;
    };
    bool ok = true;
    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    if (s < n_tiles) row_of(s);
    for (int it = s; it < n_tiles; it += 2) {
      // every warp of the four comes to both barriers in every round, whatever
      // its waits gave: the tile before's rows have been read, this one's are there
      asm volatile("bar.sync %0, 128;" ::"r"(1 + s) : "memory");
      sh.z[s][row] = z_next;
      sh.token[s][row] = t_next;
      if (it + 2 < n_tiles) row_of(it + 2);
      asm volatile("bar.sync %0, 128;" ::"r"(1 + s) : "memory");
      if (ok && !mbar_wait_warp(smem_u32(&sh.tfull[s]), (it >> 1) & 1, kWhereEpi)) ok = false;
      if (!ok) continue;
      tc_fence_after();
      // the tile's first token, and its columns that may be rows
      const int t0 = kFlat ? 0 : (tb0 + it % per_head) * 128;
      const int cols = kFlat ? min(a.group * a.T - it * 128, 128) : min(q.n - t0, 128);
      const bool masked =
          __any_sync(0xffffffffu, key >= seen0 + t0) || cols < 128 || (kFlat && q.n < a.T);
      const int chunks = kFlat ? (cols + 31) / 32 : 4;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (c >= chunks) break;
        float v[32];
        tmem_ld_32x32b_x32(tmem + 128u * s + lanes + 32u * c, v);
        tmem_ld_wait_regs(v);
        if (c == chunks - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sh.tempty[s]));
        }
        const float4 *zs = reinterpret_cast<const float4 *>(&sh.z[s][32 * c]);
        if (!masked) {
          const float2 f2 = make_float2(f, f);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float4 z = zs[i];
            const float2 y0 = __ffma2_rn(make_float2(v[4 * i], v[4 * i + 1]), f2, make_float2(z.x, z.y));
            const float2 y1 = __ffma2_rn(make_float2(v[4 * i + 2], v[4 * i + 3]), f2, make_float2(z.z, z.w));
            sum[0] = __fadd2_rn(sum[0], make_float2(ex2(y0.x), ex2(y0.y)));
            sum[1] = __fadd2_rn(sum[1], make_float2(ex2(y1.x), ex2(y1.y)));
          }
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const int col = 32 * c + i;
            const float e = ex2(fmaf(v[i], f, sh.z[s][col]));
            sum[i & 1].x += sh.token[s][col] > key - seen0 ? e : 0.f;
          }
        }
      }
    }
    const float2 both = __fadd2_rn(sum[0], sum[1]);
    float total = both.x + both.y;
    if (s == 1) sh.sum[row] = ok ? total : __uint_as_float(0x7fc00000u);
    asm volatile("bar.sync 3, 256;" ::: "memory");
    if (s == 0 && key < q.len) {
      total += sh.sum[row];
      // the new tokens' own rows start at zero
      if (a.w_in && key < q.len - q.n) total = fmaf(a.decay, a.w_in[head * a.cap + key], total);
      if (ok) a.w_out[head * a.cap + key] = total;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kEpiWarps + 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

template <int D, bool kFlat>
bool run(const AttendArgs &p, cudaStream_t stream) {
  static int done[64];
  using Cfg = WCfg<D>;
  static_assert(Cfg::kSmem + sizeof(WShared) <= 113 * 1024, "two CTAs an SM");
  if (!ensure_smem_limit(weights_tc_kernel<D, kFlat>, Cfg::kSmem, done)) return false;
  CUtensorMap map;
  const unsigned long long rows =
      static_cast<unsigned long long>(p.a.n_seqs) * p.a.n_q_heads * p.a.T;
  if (!make_bf16_rows_map(&map, p.a.q, rows, 128, D)) return false;
  const dim3 grid(static_cast<unsigned>((p.a.max_len + kTile - 1) / kTile),
                  static_cast<unsigned>(p.a.n_seqs) * p.a.n_kv_heads);
  return launch_programmatic(weights_tc_kernel<D, kFlat>, grid, kThreads, Cfg::kSmem, 1, stream, p, map);
}

}  // namespace

bool launch_weights_tc(const cache8::AttendArgs &p, cudaStream_t stream) {
  if (p.a.head_dim == 128)
    return p.a.T < 128 ? run<128, true>(p, stream) : run<128, false>(p, stream);
  return p.a.T < 128 ? run<64, true>(p, stream) : run<64, false>(p, stream);
}

}  // namespace bkv
