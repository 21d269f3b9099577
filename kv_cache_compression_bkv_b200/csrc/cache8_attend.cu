// cache8_attend.cu -- attention over the 8-bit cache, and the sum of each
// cached key's probabilities (its attention weight).
//
// For every (sequence, KV head) the query rows r = t * G + g (token t of the
// newest n, query head g of the group) attend to the keys j < len - n + t + 1:
//   x_rj = scale q_r . (code_j s_j),  p = softmax_j x,  o_r = sum_j p_rj v_j.
//
// Work split.  The unit is a tile of 128 keys of one (sequence, KV head, row
// block); the tiles of the whole call, in that order, are cut into equal runs,
// one per resident CTA, so a ragged batch leaves no CTA idle and a single long
// sequence uses every SM.  A run can begin and end inside a (sequence, head,
// row block), a "segment": a CTA that has a whole segment writes its output,
// one that has a part writes (max, sum, output) to its slot of the workspace and
// attend_finish_kernel joins the parts in their order.  The lengths are read on the
// device; the host needs only their upper bound.
//
// attend_mma_kernel (bf16, head_dim 64 or 128, up to 32 query rows a KV head):
// decode is bound by the codes' bytes, so each of the 4 warps streams its own 32
// keys of every tile through a private cp.async ring (no CTA barrier in the
// loop) and holds its own softmax statistics and output.  Codes become f16,
// exactly, two at a time (cvt.rn.f16x2.e4m3x2).  K is the A operand of
// mma.m16n8k16 and 8 query rows the B operand, so a group of up to 8 query heads
// costs no padding; more rows are more n-tiles (NT) under the same codes.  V is
// read transposed by ldmatrix.b8 and is the A operand of the second product.
// Both products' reduction indices are permuted so that the four consecutive
// bytes a lane holds are its fragment as they are: element order inside a
// contraction is free.  Queries become f16 under a power-of-two factor per
// row, exact but for elements 2^-32 and more below the row's largest (f16 holds
// bf16's 8 bits down to 2^-17, the largest is put at 2^14).
//   The f16 product, not the 8-bit one: the e4m3 mma.sync took longer here (one
// ragged batch 165 us against 147), and tcgen05 pads 8 rows to 128.
//   The probabilities are rounded to f16 (2^-11, summed in f32 before that),
// multiplied by the block's V scale under a power of two of the row's own, so that
// neither keys a row does not see nor such as get no probability cost it bits.
//   The softmax reference of a row is put 7 (in log2) under the largest logit, that
// of its outputs 7 under the largest logit plus V exponent, and they move only when
// one of these is passed by 15, so that the f16 operands stay under 2^15: one vote
// per tile instead of a max over lanes.
//   Measured: 32 sequences of 517 .. 16384 rows, 32/8 heads of 128, one token, in
// 109 to 114 us, 4.8 to 5.1 TB/s of codes, 75 to 79% of the measured copy rate.
// What is left is the GPU's memory channels, which serve its parts unevenly (CTAs of
// equal runs end 40 to 58 us into a shorter call; 2 to 6 times as many, shorter runs
// were slower, 131 us), and the join.
//
// attend_simt_kernel (f32, and other head sizes): the same split with f32
// products on the CUDA cores.
//
// More query rows: cache8_attend_tc.cu.
#include <cuda_bf16.h>

#include <algorithm>
#include <cfloat>
#include <type_traits>

#include "bkv_check.cuh"
#include "bkv_device_status.cuh"
#include "bkv_internal.h"
#include "cache8_attend.cuh"

BKV_DEFINE_STATUS_ACCESSOR(take_status_cache8_attend)

namespace bkv {
namespace {

using namespace cache8;

constexpr int kWarps = 4;                // the tensor-core kernel's
constexpr int kThreads = kWarps * 32;
constexpr int kKeys = 32;                // keys per warp and tile
constexpr int kSimtWarps = 8;            // the other kernels'
constexpr int kSimtThreads = kSimtWarps * 32;
constexpr int kSimtKeys = 16;

// The end of a CTA's part of a segment: kBufs buffers of its outputs (summed here;
// element (r, d) of a buffer at off(r, d)) and the row statistics m, l.  The outputs
// are averages already, as sums of values could pass f32's range: under l, or where
// share is given under a sum of the buffer's own, whose share of l is share[buffer
// kRows + r].  A whole segment goes out, a part to the CTA's slot.  first[d]: the
// lowest key whose NaN in V was left out (hide_nan16), for the rows that see it,
// where first[D] says that there are any; so does the result.  (With one token
// every row sees every key, and first is not looked at.)
template <int kRows, int kBufs, int kCta, typename T, typename Off>
__device__ __forceinline__ bool write_segment(const AttendArgs &p, const float *buf, int buf_stride,
                                              const float *share, const float *m, const float *l,
                                              const int *first,
                                              int seq, int unit, const SeqInfo &q, bool whole,
                                              int slot, Off &&off) {
  const Cache8AttendArgs &a = p.a;
  const int D = a.head_dim;
  const int kvh = unit / p.row_blocks, r0 = (unit - kvh * p.row_blocks) * kRows;
  const int rows = a.group * q.n;
  const bool nans = a.T > 1 && first[D] != 0;
  float *part = p.part + (static_cast<size_t>(blockIdx.x) * 2 + slot) * (kRows * (2 + D));
  for (int e = threadIdx.x; e < kRows * D; e += kCta) {
    const int r = e / D, d = e - r * D;
    const int o = off(r, d);
    float v = 0.f;
#pragma unroll
    for (int b = 0; b < kBufs; ++b) {
      const float x = buf[b * buf_stride + o];
      v = share ? fmaf(share[b * kRows + r], x, v) : v + x;
    }
    if (!whole) {
      part[2 * kRows + e] = v;
    } else if (r0 + r < rows) {
      store_out(static_cast<T *>(a.out) + q_row(a, seq, kvh, r0 + r) * D + d, v);
    }
  }
  if (nans) {  // the same elements again
#pragma unroll 1
    for (int e = threadIdx.x; e < kRows * D; e += kCta) {
      const int r = e / D, d = e - r * D;
      if (first[d] >= q.len - q.n + 1 + (r0 + r) / a.group) continue;
      const float v = __uint_as_float(0x7fc00000u);
      if (!whole) {
        part[2 * kRows + e] = v;
      } else if (r0 + r < rows) {
        store_out(static_cast<T *>(a.out) + q_row(a, seq, kvh, r0 + r) * D + d, v);
      }
    }
  }
  if (threadIdx.x < kRows) {
    const int r = threadIdx.x;
    if (!whole) {
      *reinterpret_cast<float2 *>(part + 2 * r) = make_float2(m[r], l[r]);
    } else if (r0 + r < rows) {
      store_lse(p, seq, kvh, r0 + r, m[r], l[r]);
    }
  }
  return nans;
}

// --------------------------------------------------- tensor-core kernel (bf16)

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Codes are read once a call: first to go from L2, where the kept logits and the
// parts wait for the join.
__device__ __forceinline__ uint64_t evict_first() {
  uint64_t policy;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
  return policy;
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool there,
                                           uint64_t policy) {
  const int n = there ? 16 : 0;  // 0: the 16 bytes are filled with zeros, nothing is read
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst),
               "l"(src), "r"(n), "l"(policy)
               : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int kPending>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

// A lane's part of query row r (n = lane / 4 of an n-tile): the elements of the
// 16-byte code chunks c and c + 4 (c = lane % 4).
template <int D>
struct RawQ {
  uint4 v[D / 64][2];
};
template <int D>
__device__ __forceinline__ void load_q_raw(const AttendArgs &p, int seq, int kvh, int r, int rows,
                                           RawQ<D> &q) {
  const int c = threadIdx.x & 3;
#pragma unroll
  for (int h = 0; h < D / 64; ++h)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      q.v[h][i] = make_uint4(0, 0, 0, 0);
      if (r < rows)
        q.v[h][i] = __ldg(reinterpret_cast<const uint4 *>(
                              static_cast<const __nv_bfloat16 *>(p.a.q) +
                              q_row(p.a, seq, kvh, r) * D + (c + 4 * h) * 16) + i);
    }
}

// The f16 B fragments of the rows for every k-step: word w of chunk c goes to
// k-step w, of chunk c + 4 to k-step 4 + w.  Returns the row's factor:
// f16 value * factor = q * scale * log2(e).
template <int D>
__device__ __forceinline__ float q_frags(const AttendArgs &p, const RawQ<D> &q, uint2 (&f)[D / 16]) {
  uint32_t amax = 0;
#pragma unroll
  for (int h = 0; h < D / 64; ++h)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t w[4] = {q.v[h][i].x, q.v[h][i].y, q.v[h][i].z, q.v[h][i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t lo = (w[k] & 0x7fffu) << 16, hi = w[k] & 0x7fff0000u;
        if (lo < 0x7f800000u) amax = max(amax, lo);
        if (hi < 0x7f800000u) amax = max(amax, hi);
      }
    }
  amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  // largest element to [2^14, 2^15)
  const int e = amax == 0 ? 0 : max(static_cast<int>(amax >> 23) - 127, -112);
  const float up = pow2f(14 - e);
#pragma unroll
  for (int h = 0; h < D / 64; ++h)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t w[4] = {q.v[h][i].x, q.v[h][i].y, q.v[h][i].z, q.v[h][i].w};
      uint32_t y[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        y[k] = as_u32(__floats2half2_rn(__uint_as_float(w[k] << 16) * up,
                                        __uint_as_float(w[k] & 0xffff0000u) * up));
      f[h * 4 + i * 2] = make_uint2(y[0], y[1]);
      f[h * 4 + i * 2 + 1] = make_uint2(y[2], y[3]);
    }
  return pow2f(e - 14) * (p.a.scale * kLog2e);
}

template <int D, int NT>
struct MmaCfg {
  static constexpr int kRows = 8 * NT;
  static constexpr int kStages = NT == 1 ? 3 : 2;
  static constexpr int kStageBytes = 2 * kKeys * D + 16;  // K, V and two scales each
  static constexpr int kRing = kWarps * kStages * kStageBytes;
  static constexpr int kBuf = kRows * D;                  // floats per merge buffer
  static constexpr int kQ = NT == 1 ? 0 : NT * (D / 16) * 32 * 8;
  static constexpr int kStat = (2 * kWarps * kRows + 3 * kRows + D + 1) * 4;
  static constexpr int kSmem = kRing + 2 * kBuf * 4 + kQ + kStat;
};

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, 2) attend_mma_kernel(const AttendArgs p) {
  using Cfg = MmaCfg<D, NT>;
  constexpr int KS = D / 16;  // k-steps of the first product
  constexpr int MT = D / 16;  // m-tiles of the second
  constexpr int CH = D / 16;  // 16-byte chunks per row
  extern __shared__ __align__(128) uint8_t smem[];
  float *s_buf = reinterpret_cast<float *>(smem + Cfg::kRing);
  uint2 *s_q = reinterpret_cast<uint2 *>(s_buf + 2 * Cfg::kBuf);
  float *s_m = reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(s_q) + Cfg::kQ);
  float *s_l = s_m + kWarps * Cfg::kRows;
  float *s_M = s_l + kWarps * Cfg::kRows, *s_L = s_M + Cfg::kRows, *s_rs = s_L + Cfg::kRows;
  int *s_first = reinterpret_cast<int *>(s_rs + Cfg::kRows);  // see write_segment

  const Cache8AttendArgs &a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  const int units = a.n_kv_heads * p.row_blocks;
  pdl_wait();
  pdl_launch_dependents();
  int mine;
  const Split w = split_of(a, units, p.ctas, &mine);
  const int t0 = blockIdx.x * w.run;
  if (t0 >= w.total) return;
  const int run = min(w.run, w.total - t0);

  const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(smem)) +
                        warp * Cfg::kStages * Cfg::kStageBytes;
  const uint8_t *ring_ptr = smem + warp * Cfg::kStages * Cfg::kStageBytes;

  const uint64_t policy = evict_first();
  // ---- loads: this lane's 16-byte pieces of a tile, with the swizzles that
  // make both reads below free of bank conflicts
  constexpr int PIECES = kKeys * CH / 32;
  const int lrow = lane / CH, lch = lane % CH;  // piece i: row lrow + i * (32 / CH)
  const uint32_t k_dst = lrow * D + (D == 128 ? lch ^ ((lrow & 1) << 2) : lch) * 16;
  const uint32_t v_dst0 = kKeys * D + lrow * D + (D == 128 ? lch ^ lrow : lch ^ ((lrow >> 1) & 3)) * 16;
  Cursor load, cur;
  cur.seek(a, w, units, mine, t0);
  if (!BKV_CHECK(cur.inside(a, units), 612)) return;  // the whole CTA
  load = cur;
  // the first segment's queries, ahead of the stream of codes
  RawQ<D> first_q;
  const int first_at = cur.at;
  if constexpr (NT == 1) {
    const int kvh = cur.unit / p.row_blocks;
    load_q_raw<D>(p, cur.seq, kvh, (cur.unit - kvh * p.row_blocks) * Cfg::kRows + g,
                  a.group * cur.q.n, first_q);
  }
  int load_unit = -1, load_seq = -1;
  const uint8_t *k_src = nullptr, *v_src = nullptr;
  const float *sc_src = nullptr;
  auto issue = [&](int stage) {
    if (load.unit != load_unit || load.seq != load_seq) {  // another segment
      load_unit = load.unit;
      load_seq = load.seq;
      const size_t head = static_cast<size_t>(load.seq) * a.n_kv_heads + load.unit / p.row_blocks;
      const size_t off = (head * a.cap + warp * kKeys) * D + lane * 16;
      k_src = a.k8 + off;
      v_src = a.v8 + off;
      // lanes 0..3: the K and V scales of the tile's first and second 16 keys
      sc_src = (lane & 1 ? a.v_scale : a.k_scale) + head * (a.cap >> p.log2_block);
    }
    const int j0 = load.tile * kTile + warp * kKeys;
    const int there = load.q.len - j0;  // rows of this warp's keys that exist
    if (there > 0) {
      const uint32_t dst = ring + stage * Cfg::kStageBytes;
      const size_t off = static_cast<size_t>(load.tile) * (kTile * D);
#pragma unroll
      for (int i = 0; i < PIECES; ++i) {
        const bool ok = lrow + i * (32 / CH) < there;
        const uint32_t vd = D == 128 ? v_dst0 ^ ((i & 1) << 6) : v_dst0;
        cp_async16(dst + k_dst + i * 512, k_src + off + i * 512, ok, policy);
        cp_async16(dst + vd + i * 512, v_src + off + i * 512, ok, policy);
      }
      if (lane < 4 && (lane >> 1) * 16 < there)
        cp_async4(dst + 2 * kKeys * D + lane * 4, sc_src + ((j0 + (lane >> 1) * 16) >> p.log2_block));
    }
    load.next(a, w, units);
  };
#pragma unroll 1
  for (int s = 0; s < Cfg::kStages - 1; ++s) {
    if (load.at < run) issue(s);
    cp_async_commit();
  }
  auto reset_first = [&]() {
    if (threadIdx.x < D) s_first[threadIdx.x] = INT32_MAX;
    if (threadIdx.x == 0) s_first[D] = 0;
    __syncthreads();
  };
  if (a.T > 1) reset_first();

  // ---- what a lane reads
  const int key0 = ((g >> 1) << 2) | (g & 1);  // and key0 + 2: rows g and g + 8 of an m-tile
  uint2 qf[NT == 1 ? KS : 1];
  float rs[NT][2];
  float o[MT][NT][4];
  // rows 8 nt + 2 c + i: a softmax reference m (log2) with the sum l of the
  // probabilities under it, and outputs in units of 2^-lh under it (lh: a whole number)
  float m[NT][2], l[NT][2], lh[NT][2];
  int kvh = 0, r0 = 0, seen0 = 0;
  bool fresh = true;
  int stage = 0, seg_tiles = 0;

  while (cur.at < run) {
    if (fresh) {  // a new segment: its queries, empty statistics
      fresh = false;
      seg_tiles = 0;
      kvh = cur.unit / p.row_blocks;
      r0 = (cur.unit - kvh * p.row_blocks) * Cfg::kRows;
      seen0 = cur.q.len - cur.q.n + 1;  // keys that token 0 sees
      const int rows = a.group * cur.q.n;
      if constexpr (NT == 1) {
        if (cur.at != first_at) load_q_raw<D>(p, cur.seq, kvh, r0 + g, rows, first_q);
        const float f = q_frags<D>(p, first_q, qf);
        rs[0][0] = __shfl_sync(0xffffffffu, f, (2 * c) * 4);
        rs[0][1] = __shfl_sync(0xffffffffu, f, (2 * c + 1) * 4);
      } else {
        if (warp < NT) {
          uint2 f[KS];
          RawQ<D> raw;
          load_q_raw<D>(p, cur.seq, kvh, r0 + warp * 8 + g, rows, raw);
          const float r = q_frags<D>(p, raw, f);
#pragma unroll
          for (int s = 0; s < KS; ++s) s_q[(warp * KS + s) * 32 + lane] = f[s];
          if (c == 0) s_rs[warp * 8 + g] = r;
        }
        __syncthreads();
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          rs[nt][0] = s_rs[nt * 8 + 2 * c];
          rs[nt][1] = s_rs[nt * 8 + 2 * c + 1];
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        m[nt][0] = m[nt][1] = -INFINITY;
        l[nt][0] = l[nt][1] = 0.f;
        lh[nt][0] = lh[nt][1] = 0.f;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[mt][nt][i] = 0.f;
      }
    }
    // the stage read in the last round is free
    if (load.at < run) issue(stage == 0 ? Cfg::kStages - 1 : stage - 1);
    cp_async_commit();
    cp_async_wait<Cfg::kStages - 1>();
    __syncwarp();
    const int j0 = cur.tile * kTile + warp * kKeys;
    const int there = cur.q.len - j0;
    if (there > 0) {
      const uint8_t *st = ring_ptr + stage * Cfg::kStageBytes;
      const float4 sc = *reinterpret_cast<const float4 *>(st + 2 * kKeys * D);
      const float ks[2] = {sc.x, sc.z};
      // the V scales' exponents; a block that is not there has the lowest
      const float lv[2] = {static_cast<float>(exp_of(sc.y)),
                           there > 16 ? static_cast<float>(exp_of(sc.w)) : -127.f};
      // ---- logits, 16 keys (an m-tile) at a time; the rows are in the order
      // that leaves lane c the probabilities of keys 4c .. 4c+3 when transposed
      const bool masked = j0 + kKeys > seen0 + r0 / a.group;
      float x[2][NT][4];
      bool grow = false;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) x[t][nt][i] = 0.f;
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
          const int ch = D == 128 ? (c + 4 * h) ^ ((key0 & 1) << 2) : c;
          const uint8_t *row = st + (t * 16 + key0) * D + ch * 16;
          const uint4 ka = *reinterpret_cast<const uint4 *>(row);
          const uint4 kb = *reinterpret_cast<const uint4 *>(row + 2 * D);
          const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint32_t a0 = e4m3x2_to_f16x2(wa[w]), a2 = e4m3x2_to_f16x2(wa[w] >> 16);
            const uint32_t a1 = e4m3x2_to_f16x2(wb[w]), a3 = e4m3x2_to_f16x2(wb[w] >> 16);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const uint2 b = NT == 1 ? qf[NT == 1 ? h * 4 + w : 0]
                                      : s_q[(nt * KS + h * 4 + w) * 32 + lane];
              mma16816(x[t][nt], a0, a1, a2, a3, b.x, b.y);
            }
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          // within f32's range, as logits of zero have to stay
          const float f0 = fminf(ks[t] * rs[nt][0], FLT_MAX), f1 = fminf(ks[t] * rs[nt][1], FLT_MAX);
          float(&y)[4] = x[t][nt];
          y[0] *= f0;
          y[1] *= f1;
          y[2] *= f0;
          y[3] *= f1;
          if (masked) {
            const int r = r0 + nt * 8 + 2 * c, j = j0 + t * 16 + key0;
            const int v0 = seen0 + r / a.group, v1 = seen0 + (r + 1) / a.group;
            if (j >= v0) y[0] = -INFINITY;
            if (j >= v1) y[1] = -INFINITY;
            if (j + 2 >= v0) y[2] = -INFINITY;
            if (j + 2 >= v1) y[3] = -INFINITY;
          }
#pragma unroll
          for (int i = 0; i < 2; ++i)
            grow |= fmaxf(y[i], y[i + 2]) > m[nt][i] + (15.f - fmaxf(lv[t] + lh[nt][i], 0.f));
          if (p.x_cols > 0) {
            const int col = r0 + nt * 8 + 2 * c;
            if (col < p.x_cols && t * 16 < there) {
              float *xs = p.x + ((static_cast<size_t>(cur.seq) * a.n_kv_heads + kvh) * p.x_len + j0 +
                                 t * 16 + key0) * p.x_cols + col;
              *reinterpret_cast<float2 *>(xs) = make_float2(y[0], y[1]);
              *reinterpret_cast<float2 *>(xs + 2 * p.x_cols) = make_float2(y[2], y[3]);
            }
          }
        }
      }
      // ---- a row's references: 7 (in log2) under the largest logit, and under the
      // largest logit plus V exponent, when they were set (the second to a whole
      // number), so that the probabilities and what the outputs add are at most 2^15
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float t0 = fmaxf(x[0][nt][i], x[0][nt][i + 2]);
            const float t1 = fmaxf(x[1][nt][i], x[1][nt][i + 2]);
            float t = fmaxf(t0, t1), u = fmaxf(t0 + lv[0], t1 + lv[1]);
#pragma unroll
            for (int s = 4; s < 32; s <<= 1) {
              t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, s));
              u = fmaxf(u, __shfl_xor_sync(0xffffffffu, u, s));
            }
            float f;
            if (move_reference(t - 7.f, u - 7.f, m[nt][i], l[nt][i], lh[nt][i], f)) {
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                o[mt][nt][i] *= f;
                o[mt][nt][i + 2] *= f;
              }
            }
          }
      }
      uint32_t b[NT][2][2];  // B fragments of the two k-steps: keys 4c .. 4c+3 of each m-tile
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float m0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0];
        const float m1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const float v0 = v_factor(lv[t], lh[nt][0]), v1 = v_factor(lv[t], lh[nt][1]);
          const float p0 = ex2(x[t][nt][0] - m0), p1 = ex2(x[t][nt][1] - m1);
          const float p2 = ex2(x[t][nt][2] - m0), p3 = ex2(x[t][nt][3] - m1);
          l[nt][0] += p0 + p2;
          l[nt][1] += p1 + p3;
          b[nt][t][0] = transpose8x8(as_u32(__floats2half2_rn(p0 * v0, p1 * v1)));
          b[nt][t][1] = transpose8x8(as_u32(__floats2half2_rn(p2 * v0, p3 * v1)));
        }
      }
      const int hidden = hidden_from(cur.q);
      if (j0 + kKeys > hidden) {  // keys that not every token sees: this lane's pieces
#pragma unroll 1
        for (int i = max(hidden - j0 - lrow + 32 / CH - 1, 0) / (32 / CH); i < PIECES; ++i) {
          const uint32_t at = (D == 128 ? v_dst0 ^ ((i & 1) << 6) : v_dst0) + i * 512;
          hide_nan16(reinterpret_cast<uint4 *>(smem + (st - smem) + at), [&](int e) {
            s_first[D] = 1;
            atomicMin(&s_first[lch * 16 + e], j0 + lrow + i * (32 / CH));
          });
        }
        __syncwarp();
      }
      // ---- outputs: V^T (A) by ldmatrix, 16 elements x 32 keys an m-tile
      const uint32_t vbase = ring + stage * Cfg::kStageBytes + kKeys * D + lane * D;
      const uint32_t vsw = D == 128 ? (lane & 7) << 4 : ((lane >> 1) & 3) << 4;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        uint32_t w[4];
        asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0,%1,%2,%3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "r"(vbase + ((mt << 4) ^ vsw))
                     : "memory");
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const uint32_t a0 = e4m3x2_to_f16x2(w[2 * t]), a2 = e4m3x2_to_f16x2(w[2 * t] >> 16);
          const uint32_t a1 = e4m3x2_to_f16x2(w[2 * t + 1]), a3 = e4m3x2_to_f16x2(w[2 * t + 1] >> 16);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16816(o[mt][nt], a0, a1, a2, a3, b[nt][t][0], b[nt][t][1]);
        }
      }
    }
    __syncwarp();  // every lane has read its stage
    stage = stage + 1 == Cfg::kStages ? 0 : stage + 1;
    ++seg_tiles;

    if (cur.tile + 1 == cur.q.tiles || cur.at + 1 == run) {  // the segment ends here
      const bool to_end = cur.tile + 1 == cur.q.tiles;
      const bool from_start = seg_tiles == cur.tile + 1;
      float lsum[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float t = l[nt][i];
          t += __shfl_xor_sync(0xffffffffu, t, 4);
          t += __shfl_xor_sync(0xffffffffu, t, 8);
          t += __shfl_xor_sync(0xffffffffu, t, 16);
          lsum[nt][i] = t;
          if (g == 0) {
            s_m[warp * Cfg::kRows + nt * 8 + 2 * c + i] = m[nt][i];
            s_l[warp * Cfg::kRows + nt * 8 + 2 * c + i] = t;
          }
        }
      __syncthreads();
      // this warp's factors: to the CTA's average, and from its units to the values'
      float f[NT][2], unit[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = nt * 8 + 2 * c + i;
          float M = -INFINITY;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w * Cfg::kRows + r]);
          float L = 0.f;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float mw = s_m[w * Cfg::kRows + r], lw = s_l[w * Cfg::kRows + r];
            L += mw == -INFINITY ? lw : ex2(mw - M) * lw;
          }
          f[nt][i] = (m[nt][i] != -INFINITY ? ex2(m[nt][i] - M)
                                            : lsum[nt][i] != lsum[nt][i] ? 1.f : 0.f) * inverse(L);
          unit[nt][i] = ex2(-lh[nt][i]);
          if (warp == 0 && g == 0) {
            s_M[r] = M;
            s_L[r] = L;
          }
        }
      auto at = [&](int mt, int nt, int i) { return ((mt * NT + nt) * 4 + i) * 32 + lane; };
      float *bf = s_buf + (warp & 1) * Cfg::kBuf;
      if (warp >= 2) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              bf[at(mt, nt, i)] = o[mt][nt][i] * f[nt][i & 1] * unit[nt][i & 1];
      }
      __syncthreads();
      if (warp < 2) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              bf[at(mt, nt, i)] += o[mt][nt][i] * f[nt][i & 1] * unit[nt][i & 1];
      }
      __syncthreads();
      const bool nans = write_segment<Cfg::kRows, 2, kThreads, __nv_bfloat16>(
          p, s_buf, Cfg::kBuf, nullptr, s_M, s_L, s_first, cur.seq, cur.unit, cur.q,
          from_start && to_end, from_start ? 1 : 0, [](int r, int d) {
            return (((d >> 4) * NT + (r >> 3)) * 4 + ((d >> 3) & 1) * 2 + (r & 1)) * 32 +
                   (d & 7) * 4 + ((r & 7) >> 1);
          });
      __syncthreads();
      if (nans) reset_first();
      fresh = true;
    }
    cur.next(a, w, units);
  }
}

// ------------------------------------------------------ CUDA-core kernel (f32)

__device__ __forceinline__ float load_q(const float *p) { return __ldg(p); }
__device__ __forceinline__ float load_q(const __nv_bfloat16 *p) { return __bfloat162float(*p); }

// the four values of a word of codes
__device__ __forceinline__ void values4(uint32_t w, float (&v)[4]) {
  const float2 lo = __half22float2(as_half2(e4m3x2_to_f16x2(w)));
  const float2 hi = __half22float2(as_half2(e4m3x2_to_f16x2(w >> 16)));
  v[0] = lo.x, v[1] = lo.y, v[2] = hi.x, v[3] = hi.y;
}

constexpr int kSimtRows = 8;  // query rows at a time, in weights_simt_kernel
constexpr int kMaxD = 128;

// The logits of R query rows (in shared memory, [R][D]) for one key (its codes
// in shared or global memory): two lanes a key, each every second 16-byte chunk;
// both get the sums.  Loops are kept short: at the sizes this path is for, a
// tile is over in the time that fetching long unrolled code takes.
template <int R>
__device__ __forceinline__ void simt_logits(const uint8_t *row, int D, int half, const float *s_q,
                                            float (&x)[R]) {
#pragma unroll
  for (int r = 0; r < R; ++r) x[r] = 0.f;
#pragma unroll 1
  for (int i = half * 16; i < D; i += 32) {
    const uint4 c = *reinterpret_cast<const uint4 *>(row + i);
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float v[4];
      values4(w[j], v);
      const float *q = s_q + i + 4 * j;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float4 y = *reinterpret_cast<const float4 *>(q + r * D);
        x[r] = fmaf(v[0], y.x, fmaf(v[1], y.y, fmaf(v[2], y.z, fmaf(v[3], y.w, x[r]))));
      }
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) x[r] += __shfl_xor_sync(0xffffffffu, x[r], 1);
}

// Dynamic shared memory: queries, the warps' merge buffers (each with its
// probabilities of a tile before), and per warp two stages of 16 keys' codes (rows
// padded by 16 bytes against bank conflicts).
constexpr int simt_stage_bytes(int D) { return 2 * kSimtKeys * (D + 16) + 16; }
constexpr int simt_smem(int D, int R) {
  return (1 + kSimtWarps) * R * D * 4 + kSimtWarps * 2 * simt_stage_bytes(D);
}
template <int R>
struct SimtShared {
  float m[kSimtWarps][R], l[kSimtWarps][R], share[kSimtWarps][R];
  float M[R], L[R];
  int first[kMaxD + 1];  // see write_segment
};

// R: query rows a row block has room for, 2, 4 or 8: the least that holds a KV head's,
// since empty ones cost as much as others.  f32, one token: 11 sequences of 1271
// rows, 16/8 heads of 128, 19 us with 2 and 35 with 8; 3 of 24153 rows, 2/1 heads of
// 96, 18 and 28.
template <typename T, int R>
__global__ void __launch_bounds__(kSimtThreads, 2) attend_simt_kernel(const AttendArgs p) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ SimtShared<R> sh;
  // what the plan's number of CTAs counts on: two an SM, of its 228 KB, 1 KB of each
  // CTA's is the system's
  static_assert(2 * (simt_smem(kMaxD, R) + sizeof(sh) + 1024) <= 228 * 1024, "two CTAs an SM");
  auto &s_m = sh.m, &s_l = sh.l, &s_share = sh.share;
  auto &s_M = sh.M, &s_L = sh.L;
  auto &s_first = sh.first;
  const Cache8AttendArgs &a = p.a;
  const int D = a.head_dim;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float *s_q = reinterpret_cast<float *>(smem);
  float *s_buf = s_q + R * D;
  // the probabilities of a tile, [key][R]: 16 R floats of the R D
  float *s_p = s_buf + warp * R * D;
  uint8_t *ring = reinterpret_cast<uint8_t *>(s_buf + kSimtWarps * R * D) +
                  warp * 2 * simt_stage_bytes(D);
  const int units = a.n_kv_heads * p.row_blocks;
  pdl_wait();
  pdl_launch_dependents();
  int mine;
  const Split w = split_of(a, units, p.ctas, &mine);
  const int t0 = blockIdx.x * w.run;
  if (t0 >= w.total) return;
  const int run = min(w.run, w.total - t0);
  Cursor cur, ahead;
  cur.seek(a, w, units, mine, t0);
  if (!BKV_CHECK(cur.inside(a, units), 613)) return;  // the whole CTA
  ahead = cur;
  const uint64_t policy = evict_first();
  // the next tile's codes and scales of this warp
  int issued = 0;
  auto issue = [&]() {
    const int j0 = ahead.tile * kTile + warp * kSimtKeys;
    if (ahead.at < run && j0 < ahead.q.len) {
      const uint32_t dst = static_cast<uint32_t>(__cvta_generic_to_shared(ring)) +
                           (issued & 1) * simt_stage_bytes(D);
      const size_t head = static_cast<size_t>(ahead.seq) * a.n_kv_heads + ahead.unit / p.row_blocks;
      const size_t off = (head * a.cap + j0) * D;
      const int ch = D >> 4;
#pragma unroll 1
      for (int q = lane; q < kSimtKeys * ch; q += 32) {
        const int key = q / ch;
        const uint32_t to = dst + key * (D + 16) + (q - key * ch) * 16;
        const bool there = j0 + key < ahead.q.len;
        cp_async16(to, a.k8 + off + q * 16, there, policy);
        cp_async16(to + kSimtKeys * (D + 16), a.v8 + off + q * 16, there, policy);
      }
      if (lane < 2)
        cp_async4(dst + 2 * kSimtKeys * (D + 16) + lane * 4,
                  (lane ? a.v_scale : a.k_scale) + head * (a.cap >> p.log2_block) + (j0 >> p.log2_block));
    }
    if (ahead.at < run) ahead.next(a, w, units);
    ++issued;
    cp_async_commit();
  };
  issue();
  auto reset_first = [&]() {
    if (threadIdx.x < D) s_first[threadIdx.x] = INT32_MAX;
    if (threadIdx.x == 0) s_first[D] = 0;
    __syncthreads();
  };
  if (a.T > 1) reset_first();
  float o[R][4], m[R], l[R], lh[R];  // references and units: see move_reference
  bool fresh = true;
  int seg_tiles = 0, stage = 0;
  while (cur.at < run) {
    const int kvh = cur.unit / p.row_blocks;
    const int r0 = (cur.unit - kvh * p.row_blocks) * R;
    const size_t head = static_cast<size_t>(cur.seq) * a.n_kv_heads + kvh;
    if (fresh) {
      fresh = false;
#pragma unroll 1
      for (int e = threadIdx.x; e < R * D; e += kSimtThreads) {
        const int r = e / D;
        s_q[e] = r0 + r < a.group * cur.q.n
                     ? load_q(static_cast<const T *>(a.q) + q_row(a, cur.seq, kvh, r0 + r) * D + e - r * D)
                     : 0.f;
      }
      __syncthreads();
#pragma unroll
      for (int r = 0; r < R; ++r) {
        m[r] = -INFINITY;
        l[r] = lh[r] = 0.f;
        o[r][0] = o[r][1] = o[r][2] = o[r][3] = 0.f;
      }
    }
    issue();
    cp_async_wait<1>();
    __syncwarp();
    const int j0 = cur.tile * kTile + warp * kSimtKeys;
    if (j0 < cur.q.len) {
      const uint8_t *st = ring + stage * simt_stage_bytes(D);
      const float *sc = reinterpret_cast<const float *>(st + 2 * kSimtKeys * (D + 16));
      const float f = fminf(sc[0] * (a.scale * kLog2e), FLT_MAX);
      const float lv = static_cast<float>(exp_of(sc[1]));
      const int j = j0 + (lane >> 1);
      float x[R];
      simt_logits<R>(st + (lane >> 1) * (D + 16), D, lane & 1, s_q, x);
      const int seen0 = cur.q.len - cur.q.n + 1;
      bool grow = false;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        x[r] = j < min(seen0 + (r0 + r) / a.group, cur.q.len) ? x[r] * f : -INFINITY;
        if (p.x_cols > r0 + r && (lane & 1) == 0 && j < cur.q.len)
          p.x[(head * p.x_len + j) * p.x_cols + r0 + r] = x[r];
        grow |= x[r] > m[r] + (15.f - fmaxf(lv + lh[r], 0.f));
      }
      // references move where they are passed by 2^15, all of the row block's
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          float t = x[r], g;
#pragma unroll
          for (int s = 2; s < 32; s <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, s));
          if (move_reference(t, t + lv, m[r], l[r], lh[r], g)) {
            o[r][0] *= g, o[r][1] *= g, o[r][2] *= g, o[r][3] *= g;
          }
        }
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float e = ex2(x[r] - (m[r] == -INFINITY ? 0.f : m[r]));
        if ((lane & 1) == 0) {
          s_p[(lane >> 1) * R + r] = e * v_factor(lv, lh[r]);
          l[r] += e;
        }
      }
      const int hidden = hidden_from(cur.q);
      if (j0 + kSimtKeys > hidden) {  // keys that not every token sees
        const int ch = D >> 4;
#pragma unroll 1
        for (int q = lane; q < kSimtKeys * ch; q += 32) {
          const int key = q / ch, e0 = (q - key * ch) * 16;
          if (j0 + key < hidden) continue;
          hide_nan16(reinterpret_cast<uint4 *>(ring + stage * simt_stage_bytes(D) +
                                               (kSimtKeys + key) * (D + 16) + e0),
                     [&](int e) {
                       s_first[D] = 1;
                       atomicMin(&s_first[e0 + e], j0 + key);
                     });
        }
      }
      __syncwarp();
      const uint8_t *vrow = st + kSimtKeys * (D + 16) + (lane * 4 < D ? lane * 4 : 0);
#pragma unroll 2
      for (int k = 0; k < kSimtKeys; ++k) {  // keys past the end: p = 0, codes 0
        float v[4];
        values4(*reinterpret_cast<const uint32_t *>(vrow + k * (D + 16)), v);
        alignas(16) float e[R];
        if constexpr (R == 2) {
          *reinterpret_cast<float2 *>(e) = *reinterpret_cast<const float2 *>(s_p + k * R);
        } else {
#pragma unroll
          for (int r = 0; r < R; r += 4)
            *reinterpret_cast<float4 *>(e + r) = *reinterpret_cast<const float4 *>(s_p + k * R + r);
        }
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[r][i] = fmaf(e[r], v[i], o[r][i]);
      }
    }
    __syncwarp();  // the stage and the probabilities have been read
    stage ^= 1;
    ++seg_tiles;
    if (cur.tile + 1 == cur.q.tiles || cur.at + 1 == run) {
#pragma unroll
      for (int r = 0; r < R; ++r) {  // the warp's averages
        float t = l[r];  // odd lanes: zero
#pragma unroll
        for (int s = 1; s < 32; s <<= 1) t += __shfl_xor_sync(0xffffffffu, t, s);
        if (lane == 0) {
          s_m[warp][r] = m[r];
          s_l[warp][r] = t;
        }
        const float f = inverse(t), unit = ex2(-lh[r]);
        if (lane * 4 < D)
          *reinterpret_cast<float4 *>(s_buf + (warp * R + r) * D + lane * 4) = make_float4(
              o[r][0] * f * unit, o[r][1] * f * unit, o[r][2] * f * unit, o[r][3] * f * unit);
      }
      __syncthreads();
      if (threadIdx.x < kSimtWarps * R) {
        const int k = threadIdx.x / R, r = threadIdx.x % R;
        float M = -INFINITY, L = 0.f;
        for (int k = 0; k < kSimtWarps; ++k) M = fmaxf(M, s_m[k][r]);
        // NaN logits leave no reference, and sums that have to stay
        auto part_of = [&](int k) {
          return s_m[k][r] == -INFINITY ? s_l[k][r] : ex2(s_m[k][r] - M) * s_l[k][r];
        };
        for (int k = 0; k < kSimtWarps; ++k) L += part_of(k);
        s_share[k][r] = part_of(k) * inverse(L);
        if (k == 0) {
          s_M[r] = M;
          s_L[r] = L;
        }
      }
      __syncthreads();
      const bool from_start = seg_tiles == cur.tile + 1;
      const bool to_end = cur.tile + 1 == cur.q.tiles;
      seg_tiles = 0;
      const bool nans = write_segment<R, kSimtWarps, kSimtThreads, T>(
          p, s_buf, R * D, s_share[0], s_M, s_L, s_first, cur.seq, cur.unit, cur.q,
          from_start && to_end, from_start ? 1 : 0, [D](int r, int d) { return r * D + d; });
      __syncthreads();
      if (nans) reset_first();
      fresh = true;
    }
    cur.next(a, w, units);
  }
}

// ------------------------------------------- the join of parts, and the weights

__device__ __forceinline__ void store_weight(const Cache8AttendArgs &a, size_t head, int j,
                                             const SeqInfo &q, float sum) {
  // the new tokens' own rows start at zero
  if (a.w_in && j < q.len - q.n) sum = fmaf(a.decay, a.w_in[head * a.cap + j], sum);
  a.w_out[head * a.cap + j] = sum;
}

// The reference and sum of a row over its parts, by a whole warp: a lane takes
// every 32nd part, then the lanes' pairs are joined.  stat(i): part i's pair.  A
// pair without a reference is of no keys, or of NaN logits, whose NaN sums stay.
__device__ __forceinline__ float2 join_pairs(float2 a, float2 b) {
  const float M = fmaxf(a.x, b.x);
  return make_float2(M, (a.x == -INFINITY ? a.y : ex2(a.x - M) * a.y) +
                            (b.x == -INFINITY ? b.y : ex2(b.x - M) * b.y));
}
template <typename Stat>
__device__ __forceinline__ float2 join_row(int parts, Stat &&stat) {
  float2 s = make_float2(-INFINITY, 0.f);
#pragma unroll 2
  for (int i = threadIdx.x & 31; i < parts; i += 32) s = join_pairs(s, stat(i));
#pragma unroll 1
  for (int o = 16; o > 0; o >>= 1)
    s = join_pairs(s, make_float2(__shfl_xor_sync(0xffffffffu, s.x, o),
                                  __shfl_xor_sync(0xffffffffu, s.y, o)));
  return s;
}

// The parts of a segment: the CTAs c0 .. c0 + n - 1 (n = 1: whole).
struct Parts {
  int c0, n;
};
__device__ __forceinline__ Parts parts_of(const Split &w, int first, int tiles) {
  Parts x;
  x.c0 = first / w.run;
  x.n = (first + tiles - 1) / w.run - x.c0 + 1;
  return x;
}

// The weights of keys j0 .. j1 - 1 from their kept logits, kQuad rows at a time.
// nan_rows: the rows whose lse is NaN, which goes to the keys that they see alone (a
// hidden key's logit is -infinity).
template <int kQuad, int kBatch>
__device__ __forceinline__ void weights_kept(const Cache8AttendArgs &a, const SeqInfo &q,
                                             const float *xh, int x_cols, const float *s_z,
                                             unsigned nan_rows, int rows, size_t head, int j0, int j1) {
  for (int j = j0 + threadIdx.x; j < j1; j += kBatch * kSimtThreads) {
    float sum[kBatch] = {}, old[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int ju = j + u * kSimtThreads;
      old[u] = a.w_in && ju < min(j1, q.len - q.n) ? a.w_in[head * a.cap + ju] : 0.f;
    }
#pragma unroll 2
    for (int r = 0; r < rows; r += kQuad) {  // x_cols is a multiple of kQuad
      float v[kBatch][kQuad];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const float *x = xh + static_cast<size_t>(min(j + u * kSimtThreads, j1 - 1)) * x_cols + r;
        if constexpr (kQuad == 4)
          *reinterpret_cast<float4 *>(v[u]) = *reinterpret_cast<const float4 *>(x);
        else
          *reinterpret_cast<float2 *>(v[u]) = *reinterpret_cast<const float2 *>(x);
      }
#pragma unroll
      for (int k = 0; k < kQuad; ++k) {
        const float z = s_z[r + k];  // infinity past the last row, and where it is NaN
#pragma unroll
        for (int u = 0; u < kBatch; ++u) sum[u] += ex2(v[u][k] - z);
      }
    }
    if (nan_rows != 0) {
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        for (unsigned left = nan_rows; left != 0; left &= left - 1)
          if (xh[static_cast<size_t>(min(j + u * kSimtThreads, j1 - 1)) * x_cols + __ffs(left) - 1] !=
              -INFINITY)
            sum[u] = __uint_as_float(0x7fc00000u);
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int ju = j + u * kSimtThreads;
      // the new tokens' own rows start at zero
      if (ju < j1)
        a.w_out[head * a.cap + ju] = a.w_in && ju < q.len - q.n ? fmaf(a.decay, old[u], sum[u]) : sum[u];
    }
  }
}

constexpr int kFewParts = 2;  // what runs as long as a segment, or longer, make

// First the CTAs that join: p.join_rows rows of a (sequence, KV head, row
// block) each, one row with every warp (few rows in many parts) or a row at a
// time per warp (many rows in few).  They write the rows of segments
// that several CTAs computed, and the empty rows of sequences without cached
// keys.  A row's parts are dealt to its warps in turn and the warps' sums added
// in order, so results do not depend on timing.
// Then, where the attention kernel kept its logits, the CTAs of the weights:
// one per p.w_keys keys of a (sequence, KV head), which need the rows' lse and so
// join the parts' statistics for themselves.
// Launched while the attention kernel runs: everything before the wait reads
// only the lengths, and every CTA waits, so that this kernel never ends first.
// Five CTAs an SM, 48 registers: one then fits beside two of the attention
// kernel's and has its beginning behind it when that ends.
template <int kRows, typename T>
__global__ void __launch_bounds__(kSimtThreads, 5) attend_finish_kernel(const AttendArgs p) {
  __shared__ float s_o[kSimtWarps][kMaxD];
  __shared__ float s_z[kMaxXRows];
  __shared__ bool s_nan[kMaxXRows];
  const Cache8AttendArgs &a = p.a;
  const int D = a.head_dim;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int units = a.n_kv_heads * p.row_blocks;
  const int per_unit = kRows / p.join_rows;
  const int joins = a.n_seqs * units * per_unit;
  const int stride = kRows * (2 + D);
  pdl_launch_dependents();
  int mine;
  // a part's statistics and output: slot 1 of the CTA the segment starts in,
  // slot 0 after it
  auto part = [&](const Parts &x, int i) {
    return p.part + (static_cast<size_t>(x.c0 + i) * 2 + (i == 0 ? 1 : 0)) * stride;
  };
  if (static_cast<int>(blockIdx.x) >= joins) {
    const int b = blockIdx.x - joins;
    const int head = b / p.w_chunks, j0 = (b - head * p.w_chunks) * p.w_keys;
    const int seq = head / a.n_kv_heads;
    const SeqInfo q = seq_info(a, seq);
    const bool none = q.tiles == 0 || j0 >= q.len;
    const Split w = split_of(a, units, p.ctas, &mine);
    const int before = counted_before(a, w, units, mine, seq);
    pdl_wait();
    if (none) return;
    const int rows = a.group * q.n;
    if (threadIdx.x < kMaxXRows && threadIdx.x >= rows) {
      s_z[threadIdx.x] = INFINITY;
      s_nan[threadIdx.x] = false;
    }
    for (int r = warp; r < rows; r += kSimtWarps) {
      const int unit = (head - seq * a.n_kv_heads) * p.row_blocks + r / kRows, row = r % kRows;
      Parts x = parts_of(w, before + unit * (q.tiles + w.pad) + w.pad, q.tiles);
      if (!BKV_CHECK(x.c0 >= 0 && x.n >= 1 && x.c0 + x.n <= p.ctas, 614)) x = {0, 1};
      float z;
      if (x.n == 1) {
        z = p.lse2[static_cast<size_t>(head) * a.group * a.T + r];
      } else {
        const float2 ml = join_row(x.n, [&](int i) {
          return *reinterpret_cast<const float2 *>(part(x, i) + 2 * row);
        });
        const float M = ml.x, L = ml.y;
        z = L > 0.f || L != L ? M + log2f(L) : -INFINITY;
      }
      if (lane == 0) {
        s_z[r] = z > -INFINITY ? z : INFINITY;  // rows that see nothing add nothing
        s_nan[r] = z != z;
      }
    }
    __syncthreads();
    static_assert(kMaxXRows == 32, "a row a lane");
    const unsigned nan_rows = __ballot_sync(0xffffffffu, s_nan[lane]);
    const int j1 = min(j0 + p.w_keys, q.len);
    const float *xh = p.x + static_cast<size_t>(head) * p.x_len * p.x_cols;
    // keys a thread has in flight: what the loads of one row pair take, or of a quad
    if ((p.x_cols & 3) == 0)
      weights_kept<4, 2>(a, q, xh, p.x_cols, s_z, nan_rows, rows, head, j0, j1);
    else
      weights_kept<2, 4>(a, q, xh, p.x_cols, s_z, nan_rows, rows, head, j0, j1);
    return;
  }
  const int u = blockIdx.x / per_unit;
  const int seq = u / units, unit = u - seq * units;
  const int kvh = unit / p.row_blocks;
  const int first = (blockIdx.x - u * per_unit) * p.join_rows;  // row of the row block
  const int r0 = (unit - kvh * p.row_blocks) * kRows + first;
  const SeqInfo q = seq_info(a, seq);
  const Split w = split_of(a, units, p.ctas, &mine);
  Parts x = {0, 0};
  if (q.tiles > 0)
    x = parts_of(w, counted_before(a, w, units, mine, seq) + unit * (q.tiles + w.pad) + w.pad, q.tiles);
  if (!BKV_CHECK(x.c0 >= 0 && x.n >= 0 && x.c0 + x.n <= p.ctas, 615)) x = {0, 0};
  pdl_wait();
  if (q.bad) {
    if (threadIdx.x == 0) record_device_status(BKV_DEV_ASSERT, 611);
    return;
  }
  if (x.n == 1) return;  // written by its CTA
  const int rows = min(p.join_rows, a.group * q.n - r0);
  if (p.join_rows > 1 && x.n >= 2 && x.n <= kFewParts) {
    // many rows in few parts: every lane has the parts' pairs of its row for
    // itself, two rows a warp at a time.  1024 tokens of 40/8 heads over 16384
    // rows: 20 us, and 33 with a lane per part and the lanes joined
    for (int i0 = 2 * warp; i0 < rows; i0 += 2 * kSimtWarps) {
      float2 ml[2][kFewParts];
      float4 v[2][kFewParts];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int row = first + min(i0 + k, rows - 1);
#pragma unroll
        for (int i = 0; i < kFewParts; ++i) {
          ml[k][i] = make_float2(-INFINITY, 0.f);
          v[k][i] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (i < x.n) {
            const float *s = part(x, i);
            ml[k][i] = *reinterpret_cast<const float2 *>(s + 2 * row);
            if (lane * 4 < D)
              v[k][i] = *reinterpret_cast<const float4 *>(s + 2 * kRows + row * D + lane * 4);
          }
        }
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float M = ml[k][0].x, l = 0.f, part_l[kFewParts];
#pragma unroll
        for (int i = 1; i < kFewParts; ++i) M = fmaxf(M, ml[k][i].x);
#pragma unroll
        for (int i = 0; i < kFewParts; ++i) {
          part_l[i] = (ml[k][i].x == -INFINITY ? 1.f : ex2(ml[k][i].x - M)) * ml[k][i].y;
          l += part_l[i];
        }
        const float inv = inverse(l);
        float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < kFewParts; ++i) {
          const float f = part_l[i] * inv;
          o[0] = fmaf(f, v[k][i].x, o[0]), o[1] = fmaf(f, v[k][i].y, o[1]);
          o[2] = fmaf(f, v[k][i].z, o[2]), o[3] = fmaf(f, v[k][i].w, o[3]);
        }
        if (i0 + k >= rows) break;
        if (lane * 4 < D)
          store_out4(static_cast<T *>(a.out) + q_row(a, seq, kvh, r0 + i0 + k) * D + lane * 4, o[0],
                     o[1], o[2], o[3]);
        if (lane == 0) store_lse(p, seq, kvh, r0 + i0 + k, M, l);
      }
    }
    return;
  }
  const int deal = p.join_rows == 1 ? kSimtWarps : 1;  // warps per row
  for (int i0 = warp / deal; i0 < rows; i0 += kSimtWarps / deal) {
    const int row = first + i0;
    const float2 ml = join_row(x.n, [&](int i) {
      return *reinterpret_cast<const float2 *>(part(x, i) + 2 * row);
    });
    const float M = ml.x, l = ml.y, inv = inverse(l);
    float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int i = warp % deal; i < x.n; i += deal) {
      const float *s = part(x, i);
      const float2 pair = *reinterpret_cast<const float2 *>(s + 2 * row);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (lane * 4 < D) v = *reinterpret_cast<const float4 *>(s + 2 * kRows + row * D + lane * 4);
      // no reference: no keys, or NaN
      const float f = (pair.x == -INFINITY ? 1.f : ex2(pair.x - M)) * pair.y * inv;
      o[0] = fmaf(f, v.x, o[0]), o[1] = fmaf(f, v.y, o[1]);
      o[2] = fmaf(f, v.z, o[2]), o[3] = fmaf(f, v.w, o[3]);
    }
    if (deal > 1) {
      if (lane * 4 < D)
        *reinterpret_cast<float4 *>(&s_o[warp][lane * 4]) = make_float4(o[0], o[1], o[2], o[3]);
      __syncthreads();  // one row: every warp comes here once
      if (warp != 0) return;
      for (int i = 1; i < kSimtWarps; ++i) {
        if (lane * 4 < D) {
          const float4 v = *reinterpret_cast<const float4 *>(&s_o[i][lane * 4]);
          o[0] += v.x, o[1] += v.y, o[2] += v.z, o[3] += v.w;
        }
      }
    }
    if (lane * 4 < D)
      store_out4(static_cast<T *>(a.out) + q_row(a, seq, kvh, r0 + i0) * D + lane * 4, o[0], o[1],
                 o[2], o[3]);
    if (lane == 0) store_lse(p, seq, kvh, r0 + i0, M, l);
  }
}

// From the keys again, for more query rows than logits are kept of.  A CTA has
// 128 keys, two lanes each, their codes in registers, and takes the rows that see
// any of them 8 at a time, the next ones' queries loading while these are used.
// 28 sequences with up to 62 tokens over up to 199 rows, 16/4 heads of 96 in f32: 86
// us, and 164 with codes read from L1 for every 8 rows and every row taken.
template <typename T>
__global__ void __launch_bounds__(kSimtThreads) weights_simt_kernel(const AttendArgs p) {
  __shared__ __align__(16) float s_q[2][kSimtRows * kMaxD];
  __shared__ float s_z[2][kSimtRows];
  pdl_wait();
  const Cache8AttendArgs &a = p.a;
  const int D = a.head_dim;
  const size_t head = blockIdx.y;
  const int seq = static_cast<int>(head) / a.n_kv_heads;
  const int kvh = static_cast<int>(head) - seq * a.n_kv_heads;
  const SeqInfo q = seq_info(a, seq);
  const int j0 = blockIdx.x * kTile;
  if (q.tiles == 0 || j0 >= q.len) return;
  const int j = j0 + (threadIdx.x >> 1), half = threadIdx.x & 1;
  const int jr = min(j, q.len - 1);
  const int rows = a.group * q.n;
  const float f =
      fminf(__ldg(a.k_scale + head * (a.cap / a.block) + jr / a.block) * (a.scale * kLog2e), FLT_MAX);
  constexpr int kChunks = kMaxD / 32;  // 16-byte chunks a lane
  uint4 c[kChunks];
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const int at = half * 16 + i * 32;
    c[i] = make_uint4(0, 0, 0, 0);
    if (at < D) c[i] = __ldg(reinterpret_cast<const uint4 *>(a.k8 + (head * a.cap + jr) * D + at));
  }
  constexpr int kLoads = kSimtRows * kMaxD / kSimtThreads;
  float next[kLoads], z_next = INFINITY;
  auto load = [&](int rb) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int e = threadIdx.x + i * kSimtThreads, r = rb + e / D;
      next[i] = e < kSimtRows * D && r < rows
                    ? load_q(static_cast<const T *>(a.q) + q_row(a, seq, kvh, r) * D + e % D) : 0.f;
    }
    const int r = rb + threadIdx.x;
    if (threadIdx.x < kSimtRows) {
      const float z = r < rows ? p.lse2[head * a.group * a.T + r] : -INFINITY;
      z_next = z == -INFINITY ? INFINITY : z;  // rows that see nothing add nothing
    }
  };
  const int seen0 = q.len - q.n + 1;
  // the first row that sees key j0 is that of token j0 - seen0 + 1
  const int first = max(j0 - seen0 + 1, 0) * a.group / kSimtRows * kSimtRows;
  float sum = 0.f;
  load(first);
  for (int rb = first, buf = 0; rb < rows; rb += kSimtRows, buf ^= 1) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int e = threadIdx.x + i * kSimtThreads;
      if (e < kSimtRows * D) s_q[buf][e] = next[i];
    }
    if (threadIdx.x < kSimtRows) s_z[buf][threadIdx.x] = z_next;
    __syncthreads();  // the other buffer's readers are a barrier behind
    if (rb + kSimtRows < rows) load(rb + kSimtRows);
    float x[kSimtRows] = {};
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int at = half * 16 + i * 32;
      if (at >= D) break;
      const uint32_t w[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float v[4];
        values4(w[k], v);
#pragma unroll
        for (int r = 0; r < kSimtRows; ++r) {
          const float4 y = *reinterpret_cast<const float4 *>(&s_q[buf][r * D + at + 4 * k]);
          x[r] = fmaf(v[0], y.x, fmaf(v[1], y.y, fmaf(v[2], y.z, fmaf(v[3], y.w, x[r]))));
        }
      }
    }
#pragma unroll
    for (int r = 0; r < kSimtRows; ++r) {
      x[r] += __shfl_xor_sync(0xffffffffu, x[r], 1);
      if (j < seen0 + (rb + r) / a.group) sum += exp2f(x[r] * f - s_z[buf][r]);
    }
  }
  if (j < q.len && half == 0) store_weight(a, head, j, q, sum);
}

// ------------------------------------------------------------------ launching

template <int D, int NT>
bool run_mma(const AttendArgs &p, cudaStream_t s) {
  static int done[64];
  using Cfg = MmaCfg<D, NT>;
  static_assert(Cfg::kSmem <= 113 * 1024, "shared memory");
  if (!ensure_smem_limit(attend_mma_kernel<D, NT>, Cfg::kSmem, done)) return false;
  return launch_programmatic(attend_mma_kernel<D, NT>, dim3(p.ctas), kThreads, Cfg::kSmem, 1, s, p);
}

template <int kRows, typename T>
bool run_finish(AttendArgs p, cudaStream_t s) {
  const long long segments = static_cast<long long>(p.a.n_seqs) * p.a.n_kv_heads * p.row_blocks;
  // a CTA's beginning costs as much as some rows: as few CTAs as fill the SMs
  const long long rows = segments * kRows;
  p.join_rows = rows <= 4 * kSms ? 1 : kRows % 64 != 0 || rows <= 32 * kSms ? std::min(kRows, 8) : 64;
  long long grid = segments * (kRows / p.join_rows);
  if (p.x_cols > 0) {
    // about four CTAs an SM: the lse of a CTA's rows cost it as much as some
    // hundreds of keys
    const long long heads = static_cast<long long>(p.a.n_seqs) * p.a.n_kv_heads;
    const long long keys = (heads * p.a.max_len / (4 * kSms) + kSimtThreads) / kSimtThreads;
    p.w_keys = kSimtThreads * static_cast<int>(std::min<long long>(keys, 64));
    p.w_chunks = static_cast<int>((p.a.max_len + p.w_keys - 1) / p.w_keys);
    grid += heads * p.w_chunks;
  }
  return launch_programmatic(attend_finish_kernel<kRows, T>, dim3(static_cast<unsigned>(grid)),
                             kSimtThreads, 0, 1, s, p);
}

template <typename T>
bool run_simt(const AttendArgs &p, int block_rows, cudaStream_t s) {
  auto run = [&](auto rows) {
    constexpr int R = decltype(rows)::value;
    static int done[64];
    if (!ensure_smem_limit(attend_simt_kernel<T, R>, simt_smem(kMaxD, R), done)) return false;
    return launch_programmatic(attend_simt_kernel<T, R>, dim3(p.ctas), kSimtThreads,
                               simt_smem(p.a.head_dim, R), 1, s, p) &&
           run_finish<R, T>(p, s);
  };
  return block_rows == 2   ? run(std::integral_constant<int, 2>())
         : block_rows == 4 ? run(std::integral_constant<int, 4>())
                           : run(std::integral_constant<int, 8>());
}

bool use_mma(int dtype, int head_dim) {
  return dtype == BKV_BF16 && (head_dim == 64 || head_dim == 128);
}

}  // namespace

namespace {
struct PreSections {
  size_t k, v, bytes;
};
PreSections pre_sections(int n_seqs, int n_kv_heads, int head_dim, long long max_len) {
  const size_t heads = static_cast<size_t>(n_seqs) * n_kv_heads, len = align_up(max_len, kTile);
  PreSections x;
  x.k = 0;
  x.v = align_up(heads * len * head_dim * 2, kAlign);
  x.bytes = 2 * x.v;
  return x;
}
}  // namespace

Cache8AttendPlan plan_cache8_attend(int n_seqs, int n_q_heads, int n_kv_heads, int head_dim,
                                    int dtype, long long max_len, int T, bool weights) {
  Cache8AttendPlan p{};
  const long long rows = static_cast<long long>(n_q_heads / n_kv_heads) * T;
  const bool mma = use_mma(dtype, head_dim);
  // 25 to 32 rows of 128 elements do not fit the registers: two row blocks of 16
  // read the codes twice and take 61 us (with weights 88) where one of 32 took 74
  // (115): 8 sequences of 8192 rows, 32/8 heads, 8 tokens
  p.nt = !mma || rows <= 8 ? 1 : rows <= 16 ? 2 : rows <= 24 ? 3 : head_dim == 128 ? 2 : 4;
  // Measured on both sides: 8 sequences to 8192 rows of 32/8 heads, 40 query rows
  // a KV head 69 us on tcgen05 and 107 us on mma.sync, 128 rows 89 and 184; 24
  // rows with weights (a key's logits are then kept) 109 and 48.
  p.row_tiles = mma && rows > 32 ? (rows <= 128 ? 1 : 2) : 0;
  p.block_rows = p.row_tiles ? 128 * p.row_tiles : 8 * p.nt;
  if (!mma) p.block_rows = rows <= 2 ? 2 : rows <= 4 ? 4 : 8;
  p.row_blocks = static_cast<int>((rows + p.block_rows - 1) / p.block_rows);
  // Every row block reads all of K and V.  One (up to 256 rows) turns the codes
  // into f16 as it goes, at the cost of converter warps and shared-memory
  // bandwidth; several share one conversion: 1024 tokens of 40/8 heads over
  // 16384 rows, 20 row blocks, took 490 us converting and 385
  // with the tiles expanded beforehand.
  p.expand = p.row_tiles == 2 && p.row_blocks > 1 &&
             static_cast<long long>(n_seqs) * n_kv_heads *
                     static_cast<long long>(align_up(max_len, kTile)) < INT32_MAX;
  const long long tiles = (max_len + kTile - 1) / kTile * n_seqs * n_kv_heads * p.row_blocks;
  const int resident = p.row_tiles ? kSms : 2 * kSms;
  p.ctas = static_cast<int>(std::min<long long>(tiles, resident));
  p.x_cols = weights && rows <= kMaxXRows ? static_cast<int>((rows + 1) / 2 * 2) : 0;
  const size_t part = static_cast<size_t>(p.ctas) * 2 * p.block_rows * (2 + head_dim) * 4;
  const size_t lse = static_cast<size_t>(n_seqs) * n_q_heads * T * 4;
  const size_t x = static_cast<size_t>(n_seqs) * n_kv_heads * align_up(max_len, kKeys) * p.x_cols * 4;
  p.part_off = 0;
  p.lse_off = align_up(part, kAlign);
  p.x_off = p.lse_off + align_up(lse, kAlign);
  p.pre_off = p.x_off + align_up(x, kAlign);
  p.bytes = p.pre_off;
  if (p.expand) p.bytes += kAlign + pre_sections(n_seqs, n_kv_heads, head_dim, max_len).bytes;
  return p;
}

bkv_status launch_cache8_attend(const Cache8AttendArgs &a, const Cache8AttendPlan &plan, int dtype,
                                void *ws, cudaStream_t stream) {
  if (injected_launch_failure()) return BKV_ERR_CUDA;
  AttendArgs p;
  p.a = a;
  p.row_blocks = plan.row_blocks;
  p.ctas = plan.ctas;
  p.log2_block = a.block == 16 ? 4 : a.block == 32 ? 5 : a.block == 64 ? 6 : 7;
  p.x_cols = plan.x_cols;
  p.x_len = static_cast<long long>(align_up(a.max_len, kKeys));
  uint8_t *w = static_cast<uint8_t *>(ws);
  p.part = reinterpret_cast<float *>(w + plan.part_off);
  p.lse2 = reinterpret_cast<float *>(w + plan.lse_off);
  p.x = reinterpret_cast<float *>(w + plan.x_off);
  p.pre_k = nullptr;
  p.pre_len = static_cast<long long>(align_up(a.max_len, kTile));
  if (plan.expand) {
    const PreSections x = pre_sections(a.n_seqs, a.n_kv_heads, a.head_dim, a.max_len);
    // 16 bytes are what the caller's pointer is aligned to, 32 what is stored at once
    uint8_t *e = reinterpret_cast<uint8_t *>(
        align_up(reinterpret_cast<uintptr_t>(w + plan.pre_off), kAlign));
    p.pre_k = reinterpret_cast<uint16_t *>(e + x.k);
    p.pre_v = reinterpret_cast<uint16_t *>(e + x.v);
  }
  const bool mma = use_mma(dtype, a.head_dim);
  bool ok;
  if (mma) {
    const bool wide = a.head_dim == 128;
    if (plan.row_tiles)
      ok = launch_attend_tc(p, plan.row_tiles, stream) &&
           (plan.row_tiles == 1 ? run_finish<128, __nv_bfloat16>(p, stream)
                                : run_finish<256, __nv_bfloat16>(p, stream)) &&
           (a.T == 1 || launch_mark_nan(p, stream));
    else if (plan.nt == 1)
      ok = (wide ? run_mma<128, 1>(p, stream) : run_mma<64, 1>(p, stream)) &&
           run_finish<8, __nv_bfloat16>(p, stream);
    else if (plan.nt == 2)
      ok = (wide ? run_mma<128, 2>(p, stream) : run_mma<64, 2>(p, stream)) &&
           run_finish<16, __nv_bfloat16>(p, stream);
    else if (plan.nt == 3)
      ok = (wide ? run_mma<128, 3>(p, stream) : run_mma<64, 3>(p, stream)) &&
           run_finish<24, __nv_bfloat16>(p, stream);
    else
      ok = run_mma<64, 4>(p, stream) && run_finish<32, __nv_bfloat16>(p, stream);
  } else if (dtype == BKV_BF16) {
    ok = run_simt<__nv_bfloat16>(p, plan.block_rows, stream);
  } else {
    ok = run_simt<float>(p, plan.block_rows, stream);
  }
  if (!ok) return BKV_ERR_CUDA;
  if (a.w_out && plan.x_cols == 0) {
    const unsigned heads = static_cast<unsigned>(a.n_seqs) * a.n_kv_heads;
    const unsigned tiles = static_cast<unsigned>((a.max_len + kTile - 1) / kTile);
    if (mma) return launch_weights_tc(p, stream) ? BKV_OK : BKV_ERR_CUDA;
    auto kernel = dtype == BKV_BF16 ? weights_simt_kernel<__nv_bfloat16> : weights_simt_kernel<float>;
    if (!launch_programmatic(kernel, dim3(tiles, heads), kSimtThreads, 0, 1, stream, p))
      return BKV_ERR_CUDA;
  }
  return BKV_OK;
}

}  // namespace bkv
