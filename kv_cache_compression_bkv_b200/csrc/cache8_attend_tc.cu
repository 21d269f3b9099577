// cache8_attend_tc.cu -- attention over the 8-bit cache for many query rows on
// the 5th-generation tensor cores (bf16 queries, head_dim 64 or 128).
//
// A CTA holds one or two tiles of 128 query rows of a (sequence, KV head) and
// walks its run of 128-key tiles (cache8_attend.cuh).  Both products are
// kind::f16 tcgen05.mma with f32 accumulators in TMEM:
//   S = Q K^T   Q and K f16 in shared memory, K-major, 128-byte swizzle
//   O += P V    P f16 in TMEM over the columns S was read from, V f16 in shared
//               memory as it is cached (keys x elements: MN-major)
// e4m3 codes are exact in f16, so converter warps turn each tile's codes into
// f16 once for all the CTA's rows.  The softmax warps multiply S by K's scales, 16
// columns at a time, and the probabilities by V's under a power of two of the
// row's own (move_reference), so no key costs another one's row any bits.  The
// f8f6f4 product would take the codes as they are, but then the probabilities have
// to be split into 8-bit parts to keep f16's 11 bits, which costs the softmax warps
// more than the conversion costs others.
//
// Warps: 4 per row tile do the softmax, one thread a row (TMEM lane); the
// converters load codes into registers ahead of need, half of them K, half V;
// one warp issues the MMAs.  With two row tiles the tensor cores work on one
// while the other's softmax runs; with one, S is double-buffered.
// A row's references are set 7 (in log2) under the largest logit (and logit plus V
// exponent) and move only when a 16-column sum of probabilities (times their V
// scale) passes 2^15, so the common path takes no maxima; moving them rescales O
// in TMEM, after the MMAs that are under way.
//
// Bound by the tensor cores and exp (a 256 x 128 tile: 2 x 2 x 512 cycles of
// MMA, 32768 exps at 16 a cycle, each 54% of the time in a long run, and waits for
// TMEM between them); one row tile with few rows by the converters.  Measured: 1024
// tokens of 40/8 heads of 128 over 16384 rows, 329 us (1.01 PFLOP/s of what is
// visible, 61% of the measured matrix rate); 8 sequences to 8192 rows of 32/8 heads,
// 40 query rows a KV head 69 us, 128 rows 89, 256 rows 113.
#include <cuda_bf16.h>

#include <cfloat>

#include "bkv_check.cuh"
#include "bkv_device_status.cuh"
#include "cache8_attend.cuh"
#include "sm100.cuh"
#include "tma_host.h"

BKV_DEFINE_STATUS_ACCESSOR(take_status_cache8_attend_tc)

namespace bkv {
namespace {

using namespace cache8;
using namespace sm100;

enum : int { kWhereConv = 631, kWhereMma = 632, kWhereSoft = 633, kWhereOut = 634, kWhereDrain = 635 };

// A CTA's part of a segment.
struct Part {
  int seq, unit, kvh, r0;   // r0: first query row of the row block
  int len, n, rows;         // rows: of the (sequence, KV head)
  int tile0, live;          // first tile, tiles that a row of the block sees
  bool from_start, to_end;
};

// Walks the parts of a CTA's run, in whole warps.
template <int kRows>
struct PartIter {
  Cursor c;
  int run;
  __device__ __forceinline__ bool next(const AttendArgs &p, const Split &w, int units, Part *x) {
    if (c.at >= run) return false;
    const Cache8AttendArgs &a = p.a;
    const int count = min(c.q.tiles - c.tile, run - c.at);
    x->seq = c.seq;
    x->unit = c.unit;
    x->kvh = c.unit / p.row_blocks;
    x->r0 = (c.unit - x->kvh * p.row_blocks) * kRows;
    x->len = c.q.len;
    x->n = c.q.n;
    x->rows = a.group * c.q.n;
    x->tile0 = c.tile;
    x->from_start = c.tile == 0;
    x->to_end = c.tile + count == c.q.tiles;
    const int last = min(x->r0 + kRows, x->rows) - 1;  // below r0: a block without rows
    const int sees = last < x->r0 ? 0 : max(c.q.len - c.q.n + 1 + last / a.group, 0);
    x->live = max(min(count, (sees + kTile - 1) / kTile - c.tile), 0);
    c.tile += count - 1;
    c.at += count - 1;
    c.next(a, w, units);
    return true;
  }
};

__device__ __forceinline__ void umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                        uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tmem_st_32x32b_x32(uint32_t taddr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
      "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Instruction descriptor of kind::f16 with f16 A/B, f32 D; b_mn: B is MN-major.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool b_mn) {
  return (1u << 4) | (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

// Shared-memory descriptor of an MN-major f16 operand with the 128-byte swizzle:
// rows of one K index hold 64 MN elements (128 B); 8 K indices are an atom of
// 1024 B, atoms along K follow each other, the next 64 MN elements lie
// `mn_stride` bytes on.
__device__ __forceinline__ uint64_t smem_desc_mn_sw128(uint32_t addr, uint32_t mn_stride) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((addr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(mn_stride >> 4) << 16;  // leading byte offset: along MN
  d |= static_cast<uint64_t>(1024u >> 4) << 32;      // stride byte offset: along K
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}

constexpr int kHalf = 128 * 128;  // bytes of 128 rows x 64 f16

template <int D, int RT, bool kPre>
struct TcCfg {
  static constexpr int kHalves = D / 64;
  static constexpr int kTileBytes = kHalves * kHalf;   // 128 rows (or keys) in f16
  static constexpr int kSoftWarps = 4 * RT;
  // warps that bring K and V: converters, or one that issues TMA loads
  // 12 warps, three to a scheduler, leave 168 registers a thread (13: 128)
  static constexpr int kConvWarps = kPre ? 1 : 11 - kSoftWarps;
  static constexpr int kThreads = (kSoftWarps + kConvWarps + 1) * 32;
  static constexpr int kSmem = (RT + 4) * kTileBytes + 1024;  // Q, two stages of K and V; alignment
};

struct TcShared {
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t q_full[2], s_full[2], p_full[2], pv_done[2], drain;
  uint32_t tmem;
};

// 16 codes as f16: elements 0..7 and 8..15.
__device__ __forceinline__ void convert16(uint4 c, uint4 *lo, uint4 *hi) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  uint32_t h[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[2 * i] = e4m3x2_to_f16x2(w[i]);
    h[2 * i + 1] = e4m3x2_to_f16x2(w[i] >> 16);
  }
  *lo = make_uint4(h[0], h[1], h[2], h[3]);
  *hi = make_uint4(h[4], h[5], h[6], h[7]);
}

template <int D, int RT, bool kPre>
__global__ void __launch_bounds__((TcCfg<D, RT, kPre>::kThreads), 1)
    attend_tc_kernel(const AttendArgs p, const __grid_constant__ CUtensorMap k_map,
                     const __grid_constant__ CUtensorMap v_map) {
  using Cfg = TcCfg<D, RT, kPre>;
  constexpr int kRows = 128 * RT;
  extern __shared__ uint8_t smem_raw[];
  __shared__ TcShared sh;
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t *s_q = smem, *s_k = s_q + RT * Cfg::kTileBytes, *s_v = s_k + 2 * Cfg::kTileBytes;

  pdl_wait();
  pdl_launch_dependents();
  const Cache8AttendArgs &a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int units = a.n_kv_heads * p.row_blocks;
  int mine;
  const Split w = split_of(a, units, p.ctas, &mine);
  const int t0 = blockIdx.x * w.run;
  if (t0 >= w.total) return;
  PartIter<kRows> parts;
  parts.run = min(w.run, w.total - t0);
  parts.c.seek(a, w, units, mine, t0);
  if (!BKV_CHECK(parts.c.inside(a, units), 636)) return;  // the whole CTA

  constexpr int kMmaWarp = Cfg::kSoftWarps + Cfg::kConvWarps;
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&sh.tmem), 512);
    tmem_relinquish();
    if (lane == 0) {
      for (int i = 0; i < 2; ++i) {
        mbar_init(smem_u32(&sh.k_full[i]), Cfg::kConvWarps);
        mbar_init(smem_u32(&sh.v_full[i]), Cfg::kConvWarps);
        mbar_init(smem_u32(&sh.k_empty[i]), 1);
        mbar_init(smem_u32(&sh.v_empty[i]), 1);
        mbar_init(smem_u32(&sh.q_full[i]), 4);
        mbar_init(smem_u32(&sh.s_full[i]), 1);
        mbar_init(smem_u32(&sh.p_full[i]), 4);
        mbar_init(smem_u32(&sh.pv_done[i]), 1);
      }
      mbar_init(smem_u32(&sh.drain), 1);
      fence_barrier_init();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  // columns: S (and P) of row tile or buffer i at 128 i, O of row tile i at 256 + 128 i
  auto s_col = [&](int i) { return tmem + 128u * i; };
  auto o_col = [&](int i) { return tmem + 256u + 128u * i; };

  if (warp == kMmaWarp) {
    // ------------------------------------------------------------- the MMAs
    constexpr uint32_t idesc_qk = idesc_f16_f32(128, 128, false);
    constexpr uint32_t idesc_pv = idesc_f16_f32(128, D, true);
    const uint64_t q_desc = smem_desc_k_sw128(smem_u32(s_q)), k_desc = smem_desc_k_sw128(smem_u32(s_k));
    const uint64_t v_desc = smem_desc_mn_sw128(smem_u32(s_v), kHalf);
    auto qk = [&](int x, int t, int buf) {  // S[buf] = Q_x K(t)^T
      if (elect_one()) {
        const uint64_t ad = q_desc + x * (Cfg::kTileBytes >> 4), bd = k_desc + (t & 1) * (Cfg::kTileBytes >> 4);
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
          const uint32_t off = ((s >> 2) * kHalf + (s & 3) * 32) >> 4;
          umma_f16(s_col(buf), ad + off, bd + off, idesc_qk, s != 0);
        }
        umma_commit(smem_u32(&sh.s_full[buf]));
      }
      __syncwarp();
    };
    auto pv = [&](int x, int t, int buf, bool first) {  // O_x += P[buf] V(t)
      if (elect_one()) {
        const uint64_t bd = v_desc + (t & 1) * (Cfg::kTileBytes >> 4);
#pragma unroll
        for (int s = 0; s < 8; ++s)
          umma_ts(o_col(x), s_col(buf) + 8u * s, bd + s * (2048 >> 4), idesc_pv, !(first && s == 0));
        umma_commit(smem_u32(&sh.pv_done[x]));
      }
      __syncwarp();
    };
    auto wait = [&](uint64_t *bar, int phase) {
      const bool ok = mbar_wait_warp(smem_u32(bar), phase & 1, kWhereMma);
      tc_fence_after();
      return ok;
    };
    auto commit = [&](uint64_t *bar) {
      if (elect_one()) umma_commit(smem_u32(bar));
      __syncwarp();
    };
    Part x;
    int t = 0, seg = 0;
    bool ok = true;
    while (ok && parts.next(p, w, units, &x)) {
      if (x.live == 0) continue;
      for (int i = 0; i < RT && ok; ++i) ok = wait(&sh.q_full[i], seg);
      ok = ok && wait(&sh.k_full[t & 1], t >> 1);
      if (!ok) break;
      for (int i = 0; i < RT; ++i) qk(i, t, RT == 2 ? i : t & 1);
      commit(&sh.k_empty[t & 1]);
      for (int j = 0; j < x.live && ok; ++j, ++t) {
        const bool more = j + 1 < x.live;
        if (RT == 1 && more) {
          if (!(ok = wait(&sh.k_full[(t + 1) & 1], (t + 1) >> 1))) break;
          qk(0, t + 1, (t + 1) & 1);
          commit(&sh.k_empty[(t + 1) & 1]);
        }
        if (!(ok = wait(&sh.v_full[t & 1], t >> 1))) break;
        for (int i = 0; i < RT; ++i) {
          if (!(ok = wait(&sh.p_full[i], t))) break;
          pv(i, t, RT == 2 ? i : t & 1, j == 0);
          if (RT == 2 && more) {
            if (i == 0 && !(ok = wait(&sh.k_full[(t + 1) & 1], (t + 1) >> 1))) break;
            qk(i, t + 1, i);
          }
        }
        if (!ok) break;
        commit(&sh.v_empty[t & 1]);
        if (RT == 2 && more) commit(&sh.k_empty[(t + 1) & 1]);
      }
      ++seg;
    }
    commit(&sh.drain);
    mbar_wait_warp(smem_u32(&sh.drain), 0, kWhereDrain);
  } else if (kPre && warp >= Cfg::kSoftWarps) {
    // ------------------------------------------------- TMA, from f16 tiles
    if (lane == 0) {
      prefetch_tensormap(&k_map);
      prefetch_tensormap(&v_map);
    }
    Part x;
    int t = 0;
    bool ok = true;
    while (ok && parts.next(p, w, units, &x)) {
      const long long row =
          (static_cast<long long>(x.seq) * a.n_kv_heads + x.kvh) * p.pre_len + x.tile0 * kTile;
      for (int j = 0; j < x.live && ok; ++j) {
        const int stage = t & 1, y = static_cast<int>(row) + j * kTile;
        for (int kv = 0; kv < 2 && ok; ++kv) {
          uint64_t *full = kv ? &sh.v_full[stage] : &sh.k_full[stage];
          if (!(ok = mbar_wait_warp(smem_u32(kv ? &sh.v_empty[stage] : &sh.k_empty[stage]),
                                    ((t >> 1) & 1) ^ 1, kWhereConv)))
            break;
          if (lane == 0) {
            mbar_arrive_expect_tx(smem_u32(full), Cfg::kTileBytes);
#pragma unroll
            for (int h = 0; h < Cfg::kHalves; ++h)
              tma_load_2d(smem_u32((kv ? s_v : s_k) + stage * Cfg::kTileBytes + h * kHalf),
                          kv ? &v_map : &k_map, smem_u32(full), h * 64, y);
          }
        }
        if (ok) ++t;
      }
    }
    // loads that no MMA waited for must not outlive the CTA
    for (int i = max(t - 2, 0); i < t; ++i) {
      mbar_wait_warp(smem_u32(&sh.k_full[i & 1]), (i >> 1) & 1, kWhereDrain);
      mbar_wait_warp(smem_u32(&sh.v_full[i & 1]), (i >> 1) & 1, kWhereDrain);
    }
  } else if (warp >= Cfg::kSoftWarps) {
    // ------------------------------------------------------- the converters
    // K and V of a tile in turn, each by all converter warps; NB of them are
    // held in registers ahead of need
    constexpr int CH = D / 16;                       // 16-code chunks per key
    constexpr int kThr = Cfg::kConvWarps * 32;
    constexpr int NP = (128 * CH + kThr - 1) / kThr; // pieces per thread
    constexpr int NB = RT == 2 ? 2 : 4;
    const int tid = (warp - Cfg::kSoftWarps) * 32 + lane;
    // piece i of a thread is row row0 + i * kStep, chunk pair ch of it; kStep mod 8
    // is 0 or 4, so the swizzle of odd pieces differs by bit 2 of the chunk or not
    constexpr int kStep = kThr / CH;
    static_assert(kThr % CH == 0 && kStep % 4 == 0, "rows of a thread's pieces");
    const int row0 = tid / CH, ch = tid % CH;
    // odd halves store their second 16 bytes first, which keeps the 8 lanes of a
    // row free of bank conflicts
    const int flip = (ch >> 2) & 1;
    const uint32_t to0 = (ch >> 2) * kHalf + sw128_offset(row0, (ch & 3) * 2 + flip);
    constexpr uint32_t swap4 = 4 << 4;
    PartIter<kRows> load_parts = parts;
    Part lx, x;
    lx.live = x.live = 0;
    int lj = -1, cj = -1;  // tiles within the parts being loaded and converted
    bool more = true;
    uint4 c[NB][NP];
    auto load = [&](int b) {
      if ((b & 1) == 0) {
        ++lj;
        while (more && lj >= lx.live) {
          more = load_parts.next(p, w, units, &lx);
          lj = 0;
          if (!more) lx.live = 0;
        }
      }
      if (!more) return;
      const int j0 = (lx.tile0 + lj) * kTile;
      const size_t head = static_cast<size_t>(lx.seq) * a.n_kv_heads + lx.kvh;
      const uint4 *src =
          reinterpret_cast<const uint4 *>((b & 1 ? a.v8 : a.k8) + (head * a.cap + j0) * D) + tid;
      const int left = min(lx.len - j0, kTile) * CH - tid;  // pieces from this thread's first on
      if (left >= (NP - 1) * kThr + 1) {
#pragma unroll
        for (int i = 0; i < NP; ++i) c[b][i] = __ldcs(src + i * kThr);
      } else {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          c[b][i] = make_uint4(0, 0, 0, 0);  // keys past the end are zeros
          if (i * kThr < left) c[b][i] = __ldcs(src + i * kThr);
        }
      }
    };
#pragma unroll
    for (int b = 0; b < NB; ++b) load(b);
    int t = -1;
    bool ok = true;
    while (ok) {
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const bool is_v = (b & 1) != 0;
        if (!is_v) {  // the next tile
          ++cj;
          ++t;
          while (ok && cj >= x.live) {
            ok = parts.next(p, w, units, &x);
            cj = 0;
          }
          if (!ok) break;
        }
        const int stage = t & 1;
        if (!(ok = mbar_wait_warp(smem_u32(is_v ? &sh.v_empty[stage] : &sh.k_empty[stage]),
                                  ((t >> 1) & 1) ^ 1, kWhereConv)))
          break;
        uint8_t *tile = (is_v ? s_v : s_k) + stage * Cfg::kTileBytes;
        const int hidden = x.len - x.n + 1 - (x.tile0 + cj) * kTile;  // row of the tile
        if (is_v && x.n > 1 && hidden < kTile) {
#pragma unroll
          for (int i = 0; i < NP; ++i)
            if (row0 + i * kStep >= hidden) c[b][i] = without_nan16(c[b][i]);
        }
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          if (128 * CH % kThr == 0 || i < NP - 1 || row0 + i * kStep < 128) {
            uint4 lo, hi;
            convert16(c[b][i], &lo, &hi);
            const uint32_t to = (to0 ^ (kStep % 8 != 0 && (i & 1) ? swap4 : 0u)) + i * kStep * 128;
            *reinterpret_cast<uint4 *>(tile + to) = flip ? hi : lo;
            *reinterpret_cast<uint4 *>(tile + (to ^ 16u)) = flip ? lo : hi;
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(is_v ? &sh.v_full[stage] : &sh.k_full[stage]));
        load(b);
      }
    }
  } else {
    // ---------------------------------------------------------- the softmax
    const int x_tile = warp >> 2;               // row tile
    const int trow = (warp & 3) * 32 + lane;    // row in it, TMEM lane
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const float scale = fminf(fmaxf(a.scale * kLog2e, FLT_MIN), FLT_MAX);
    const uint32_t scale_bits = (__float_as_uint(scale) & 0x7fffffu) | 0x800000u;
    Part x;
    int t = 0;
    bool ok = true;
    // Waits, once, until tile t - 1 of the part (its tile j - 1) is in O.  A phase
    // must not pass unwaited, or its parity would be taken for the next one's:
    // with two row tiles a tile's logits are made after the tile before is in
    // O; with one this is called for every tile before its P is handed on.
    int pv_seen = 0;  // tiles known to be in O
    auto wait_pv = [&](int j, int t) {
      if (j == 0 || pv_seen == t) return true;
      pv_seen = t;
      const bool done = mbar_wait_warp(smem_u32(&sh.pv_done[x_tile]), (t - 1) & 1, kWhereSoft);
      tc_fence_after();
      return done;
    };
    while (ok && parts.next(p, w, units, &x)) {
      const int r = x.r0 + x_tile * 128 + trow;
      const bool row = r < x.rows && BKV_CHECK(r >= 0 && r < a.group * a.T, 638);
      const int sees = x.len - x.n + 1 + r / a.group;  // keys this row sees
      const bool warp_rows = x.r0 + x_tile * 128 + (warp & 3) * 32 < x.rows;
      const bool whole = x.from_start && x.to_end;
      float ref = -INFINITY, l = 0.f, lh = 0.f;
      if (x.live > 0) {
        int q_exp;       // of the logits' factor, see k_factor
        int lh_exp = 0;  // lh
        // queries: f16 under a power of two per row, largest in [2^14, 2^15)
        // (read twice: once in registers costs spills in the loop below, 112 -> 119 us
        // for 8 sequences to 8192 rows of 32/8 heads, 64 tokens)
        {
          uint32_t amax = 0;
          const uint4 *src = reinterpret_cast<const uint4 *>(
              static_cast<const __nv_bfloat16 *>(a.q) + (row ? q_row(a, x.seq, x.kvh, r) * D : 0));
#pragma unroll 8
          for (int i = 0; i < D / 8; ++i) {
            const uint4 v = row ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
            const uint32_t y[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t lo = (y[k] & 0x7fffu) << 16, hi = y[k] & 0x7fff0000u;
              if (lo < 0x7f800000u) amax = max(amax, lo);
              if (hi < 0x7f800000u) amax = max(amax, hi);
            }
          }
          const int e = amax == 0 ? 0 : max(static_cast<int>(amax >> 23) - 127, -112);
          const float up = pow2f(14 - e);
          uint8_t *tile = s_q + x_tile * Cfg::kTileBytes;
#pragma unroll 8
          for (int i = 0; i < D / 8; ++i) {
            const uint4 v = row ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
            const uint32_t y[4] = {v.x, v.y, v.z, v.w};
            uint32_t h[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              h[k] = as_u32(__floats2half2_rn(__uint_as_float(y[k] << 16) * up,
                                              __uint_as_float(y[k] & 0xffff0000u) * up));
            *reinterpret_cast<uint4 *>(tile + (i >> 3) * kHalf + sw128_offset(trow, i & 7)) =
                make_uint4(h[0], h[1], h[2], h[3]);
          }
          q_exp = e - 14 + exp_of(scale) - 1;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sh.q_full[x_tile]));
        }
        const size_t block0 =
            (static_cast<size_t>(x.seq) * a.n_kv_heads + x.kvh) * (a.cap >> p.log2_block);
        for (int j = 0; j < x.live; ++j, ++t) {
          const int buf = RT == 2 ? x_tile : t & 1;
          // lanes 8 i + b: the exponent fields of K's and V's scale in columns 16 b ..
          uint32_t fields = 0;
          const int j0 = (x.tile0 + j) * kTile, jb = j0 + (lane & 7) * 16;
          if (jb < x.len)
            fields = __float_as_uint(__ldg(a.k_scale + block0 + (jb >> p.log2_block))) >> 23 |
                     __float_as_uint(__ldg(a.v_scale + block0 + (jb >> p.log2_block))) >> 23 << 16;
          if (!(ok = mbar_wait_warp(smem_u32(&sh.s_full[buf]), RT == 2 ? t & 1 : (t >> 1) & 1,
                                    kWhereSoft)))
            break;
          tc_fence_after();
          if (warp_rows) {
            const uint32_t s_addr = s_col(buf) + lanes;
            // the logits' factor under K's scale, row's power of two times `scale`,
            // within f32's normal range, as -infinity and zero have to stay; and what the
            // probabilities are multiplied by, 2^(lv + lh), bounded as in v_factor.  Put
            // together from exponents, which leaves the exp unit to the exps
            auto k_factor = [&](uint32_t fields) {
              const int e = __viaddmin_s32_relu(static_cast<int>(fields & 0xffffu), q_exp, 253);
              return __uint_as_float((static_cast<uint32_t>(e) << 23) + scale_bits);
            };
            auto v_exp = [&](uint32_t fields) { return static_cast<int>(fields >> 16); };
            const int nvis = sees - j0;
            const bool masked = __any_sync(0xffffffffu, nvis < kTile);
            if (masked) {  // hidden keys' logits become -infinity where they stand
#pragma unroll 1
              for (int c = 0; c < 4; ++c) {
                float v[32];
                uint32_t u[32];
                tmem_ld_32x32b_x32(s_addr + 32u * c, v);
                tmem_ld_wait_regs(v);
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  u[i] = __float_as_uint(c * 32 + i < nvis ? v[i] : -INFINITY);
                tmem_st_32x32b_x32(s_addr + 32u * c, u);
              }
              tmem_st_wait();
            }
            uint32_t ph[64];
            float sum = 0.f;
            bool fine = false;
            // probabilities under the row's reference, until it need not move; the
            // first tile begins with the move
            for (int round = j > 0 ? 0 : 1;; ++round) {
              if (round > 0) {
                float top = -INFINITY, top_v = -INFINITY;
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                  float v[32];
                  tmem_ld_32x32b_x32(s_addr + 32u * c, v);
                  tmem_ld_wait_regs(v);
#pragma unroll
                  for (int b = 0; b < 2; ++b) {
                    float m = -INFINITY;
#pragma unroll
                    for (int i = 0; i < 16; ++i) m = fmaxf(m, v[16 * b + i]);
                    const uint32_t here = __shfl_sync(0xffffffffu, fields, 2 * c + b);
                    m *= k_factor(here);
                    top = fmaxf(top, m);
                    top_v = fmaxf(top_v, m + static_cast<float>(v_exp(here) - 127));
                  }
                }
                float corr = 1.f, f;
                if (!fine && move_reference(top - 7.f, top_v - 7.f, ref, l, lh, f)) {
                  corr = f;
                  lh_exp = static_cast<int>(fminf(fmaxf(lh, -300.f), 300.f));
                }
                __syncwarp();
                if (j > 0) {
                  // O, once the MMAs of the tile before have added to it
                  if (!(ok = wait_pv(j, t))) break;
#pragma unroll 1
                  for (int c = 0; c < D / 32; ++c) {
                    float v[32];
                    uint32_t u[32];
                    tmem_ld_32x32b_x32(o_col(x_tile) + lanes + 32u * c, v);
                    tmem_ld_wait_regs(v);
#pragma unroll
                    for (int i = 0; i < 32; ++i) u[i] = __float_as_uint(v[i] * corr);
                    tmem_st_32x32b_x32(o_col(x_tile) + lanes + 32u * c, u);
                  }
                  tmem_st_wait();
                }
              }
              const float ru = ref == -INFINITY ? 0.f : ref;
              const float2 r2 = make_float2(-ru, -ru);
              fine = true;
              sum = 0.f;
              float v[2][32];  // the next columns are on their way while these are used
              tmem_ld_32x32b_x32(s_addr, v[0]);
              tmem_ld_wait_regs(v[0]);
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                if (c < 3) tmem_ld_32x32b_x32(s_addr + 32u * (c + 1), v[(c + 1) & 1]);
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                  const uint32_t here = __shfl_sync(0xffffffffu, fields, 2 * c + b);
                  const float f = k_factor(here);
                  const float g = __uint_as_float(
                      static_cast<uint32_t>(__viaddmin_s32_relu(v_exp(here), lh_exp, 253)) << 23);
                  const float2 f2 = make_float2(f, f), g2 = make_float2(g, g);
                  float2 part[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                  for (int i = 8 * b; i < 8 * b + 8; ++i) {
                    const float2 y =
                        __ffma2_rn(make_float2(v[c & 1][2 * i], v[c & 1][2 * i + 1]), f2, r2);
                    const float2 e = make_float2(ex2(y.x), ex2(y.y));
                    part[i & 1] = __fadd2_rn(part[i & 1], e);
                    const float2 h = __fmul2_rn(e, g2);
                    ph[c * 16 + i] = as_u32(__floats2half2_rn(h.x, h.y));
                  }
                  const float2 both = __fadd2_rn(part[0], part[1]);
                  const float s16 = both.x + both.y;
                  fine &= s16 <= 32768.f && s16 * g <= 32768.f;
                  sum += s16;
                }
                if (c < 3) tmem_ld_wait_regs(v[(c + 1) & 1]);
              }
              if (round > 0 || !__any_sync(0xffffffffu, !fine)) break;
            }
            if (!ok) break;
            // still above a bound under its own largest logits: not a number
            if (!fine) sum = __uint_as_float(0x7fc00000u);
            l += sum;
            __syncwarp();  // tcgen05 loads and stores are the whole warp's
            tmem_st_32x32b_x32(s_addr, ph);
            tmem_st_32x32b_x32(s_addr + 32u, ph + 32);
            tmem_st_wait();
          }
          if (RT == 1 && !(ok = wait_pv(j, t))) break;
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sh.p_full[x_tile]));
        }
        if (!ok) break;
        if (!(ok = mbar_wait_warp(smem_u32(&sh.pv_done[x_tile]), (t - 1) & 1, kWhereOut))) break;
        tc_fence_after();
      }
      if (!warp_rows) continue;
      // ---- the part's end: a whole segment goes out, a part to its slot
      float *part = p.part + (static_cast<size_t>(blockIdx.x) * 2 + (x.from_start ? 1 : 0)) *
                                 (kRows * (2 + D));
      const int pr = x_tile * 128 + trow;
      const float unit = ex2(-lh);  // of the outputs
      const float mul = inverse(l);
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        float v[32];
        __syncwarp();
        if (x.live > 0) {
          tmem_ld_32x32b_x32(o_col(x_tile) + lanes + 32u * c, v);
          tmem_ld_wait_regs(v);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = 0.f;
        }
        // rows without a visible key so far hold zeros, whatever the scale
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = l != 0.f ? v[i] * mul * unit : 0.f;
        if (row && whole) {
          __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + q_row(a, x.seq, x.kvh, r) * D + 32 * c;
#pragma unroll
          for (int i = 0; i < 32; i += 8) {
            uint4 y;
            __nv_bfloat162 h;
            h = __floats2bfloat162_rn(v[i], v[i + 1]), y.x = *reinterpret_cast<uint32_t *>(&h);
            h = __floats2bfloat162_rn(v[i + 2], v[i + 3]), y.y = *reinterpret_cast<uint32_t *>(&h);
            h = __floats2bfloat162_rn(v[i + 4], v[i + 5]), y.z = *reinterpret_cast<uint32_t *>(&h);
            h = __floats2bfloat162_rn(v[i + 6], v[i + 7]), y.w = *reinterpret_cast<uint32_t *>(&h);
            *reinterpret_cast<uint4 *>(out + i) = y;
          }
        } else if (row) {
          float4 *dst = reinterpret_cast<float4 *>(part + 2 * kRows + pr * D + 32 * c);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            dst[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        }
      }
      __syncwarp();
      tc_fence_before();
      if (row && whole) store_lse(p, x.seq, x.kvh, r, ref, l);
      if (row && !whole) *reinterpret_cast<float2 *>(part + 2 * pr) = make_float2(ref, l);
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// 32 aligned bytes at once: two stores of 16 would each leave gaps
__device__ __forceinline__ void store32(uint4 *to, uint4 lo, uint4 hi) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(lo.x),
               "r"(lo.y), "r"(lo.z), "r"(lo.w), "r"(hi.x), "r"(hi.y), "r"(hi.z), "r"(hi.w)
               : "memory");
}

// K and V of every sequence as f16 tiles of 128 keys (rows past the end zeros),
// for calls whose row blocks would each convert them again.  A copy: 1 byte read, 2
// written per element.
template <int D>
__global__ void __launch_bounds__(256) expand_kernel(const AttendArgs p) {
  constexpr int CH = D / 16, NP = 128 * CH / 256;
  pdl_wait();
  pdl_launch_dependents();
  const Cache8AttendArgs &a = p.a;
  const size_t head = blockIdx.y;
  const SeqInfo q = seq_info(a, static_cast<int>(head) / a.n_kv_heads);
  const int tile = blockIdx.x, j0 = tile * kTile;
  if (tile >= q.tiles) return;
  const size_t src = (head * a.cap + j0) * D;
  uint4 c[2][NP];
#pragma unroll
  for (int kv = 0; kv < 2; ++kv)
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int id = i * 256 + threadIdx.x;
      c[kv][i] = make_uint4(0, 0, 0, 0);
      if (j0 + id / CH < q.len)
        c[kv][i] = __ldcs(reinterpret_cast<const uint4 *>((kv ? a.v8 : a.k8) + src) + id);
    }
  const int hidden = hidden_from(q);
  if (j0 + kTile > hidden) {
#pragma unroll
    for (int i = 0; i < NP; ++i)
      if (j0 + (i * 256 + threadIdx.x) / CH >= hidden) c[1][i] = without_nan16(c[1][i]);
  }
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    uint4 *dst = reinterpret_cast<uint4 *>((kv ? p.pre_v : p.pre_k) + (head * p.pre_len + j0) * D);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      uint4 lo, hi;
      convert16(c[kv][i], &lo, &hi);
      store32(&dst[2 * (i * 256 + threadIdx.x)], lo, hi);
    }
  }
}

// The outputs that a NaN in V reaches where the kernel above left it out: those,
// in the NaN's element, of the tokens that see its row, among the call's own
// tokens' rows but the first.  The rows are looked through while the kernels
// before end.
template <int D>
__global__ void __launch_bounds__(256) mark_nan_kernel(const AttendArgs p) {
  constexpr int CH = D / 16, NP = 128 * CH / 256;
  const Cache8AttendArgs &a = p.a;
  const size_t head = blockIdx.y;
  const int seq = static_cast<int>(head) / a.n_kv_heads;
  const SeqInfo q = seq_info(a, seq);
  const int j0 = max(q.len - q.n + 1, 0) + static_cast<int>(blockIdx.x) * 128;
  const bool none = q.tiles == 0 || j0 >= q.len;
  const uint4 *src = reinterpret_cast<const uint4 *>(a.v8 + (head * a.cap + j0) * D);
  auto load = [&](int i) {
    const int id = i * 256 + threadIdx.x;
    return !none && j0 + id / CH < q.len ? __ldg(src + id) : make_uint4(0, 0, 0, 0);
  };
  bool any = false;
#pragma unroll
  for (int i = 0; i < NP; ++i) any |= has_nan16(load(i));
  pdl_wait();
  if (!any) return;
  for (int i = 0; i < NP; ++i) {
    uint4 c = load(i);
    const int id = i * 256 + threadIdx.x, j = j0 + id / CH;
    hide_nan16(&c, [&](int e) {
      const int t0 = j - (q.len - q.n);  // the first token that sees row j
      if (!BKV_CHECK(t0 >= 0 && j < q.len, 637)) return;
      for (int t = t0; t < q.n; ++t)
        for (int g = 0; g < a.group; ++g)
          static_cast<__nv_bfloat16 *>(a.out)[q_row(a, seq, static_cast<int>(head) - seq * a.n_kv_heads,
                                                    t * a.group + g) * D + id % CH * 16 + e] =
              __float2bfloat16(__uint_as_float(0x7fc00000u));
    });
  }
}

template <int D, int RT, bool kPre>
bool run_tc(const AttendArgs &p, cudaStream_t s) {
  static int done[64];
  using Cfg = TcCfg<D, RT, kPre>;
  static_assert(Cfg::kSmem + sizeof(TcShared) <= 227 * 1024, "shared memory");
  if (!ensure_smem_limit(attend_tc_kernel<D, RT, kPre>, Cfg::kSmem, done)) return false;
  CUtensorMap k_map{}, v_map{};
  if (kPre) {
    const unsigned heads = static_cast<unsigned>(p.a.n_seqs) * p.a.n_kv_heads;
    const unsigned long long rows = static_cast<unsigned long long>(heads) * p.pre_len;
    if (!make_bf16_rows_map(&k_map, p.pre_k, rows, 128, D) ||
        !make_bf16_rows_map(&v_map, p.pre_v, rows, 128, D))
      return false;
    if (!launch_programmatic(expand_kernel<D>, dim3(static_cast<unsigned>(p.pre_len / kTile), heads),
                             256, 0, 1, s, p))
      return false;
  }
  return launch_programmatic(attend_tc_kernel<D, RT, kPre>, dim3(p.ctas), Cfg::kThreads, Cfg::kSmem,
                             1, s, p, k_map, v_map);
}

template <int D>
bool run_mark_nan(const AttendArgs &p, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((p.a.T + 126) / 128),
                  static_cast<unsigned>(p.a.n_seqs) * p.a.n_kv_heads);
  return launch_programmatic(mark_nan_kernel<D>, grid, 256, 0, 1, s, p);
}

}  // namespace

bool launch_mark_nan(const cache8::AttendArgs &p, cudaStream_t s) {
  return p.a.head_dim == 128 ? run_mark_nan<128>(p, s) : run_mark_nan<64>(p, s);
}

bool launch_attend_tc(const cache8::AttendArgs &p, int row_tiles, cudaStream_t s) {
  if (p.pre_k)
    return p.a.head_dim == 128 ? run_tc<128, 2, true>(p, s) : run_tc<64, 2, true>(p, s);
  if (p.a.head_dim == 128)
    return row_tiles == 1 ? run_tc<128, 1, false>(p, s) : run_tc<128, 2, false>(p, s);
  return row_tiles == 1 ? run_tc<64, 1, false>(p, s) : run_tc<64, 2, false>(p, s);
}

}  // namespace bkv
