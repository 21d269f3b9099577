// cache8_attend.cuh -- what the attention kernels over the 8-bit cache share:
// their arguments, the cut of the work into runs of key tiles, and where rows
// and row statistics live.
#pragma once

#include <cuda_bf16.h>

#include "bkv_internal.h"
#include "cache8.cuh"

namespace bkv {
namespace cache8 {

constexpr int kTile = 128;               // keys per tile
constexpr int kSms = 148;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kMaxXRows = 32;  // query rows per KV head whose logits are kept for the weights

struct AttendArgs {
  Cache8AttendArgs a;
  int row_blocks, ctas, x_cols, log2_block, join_rows;
  int w_keys, w_chunks;  // keys per weights CTA, and its CTAs per (sequence, KV head)
  long long x_len;   // keys per (sequence, KV head) in x
  // [ctas][2]: the two ends' segments of a CTA's run, each (reference, sum)
  // [rows], then outputs [rows][head_dim], averages under the sum
  float *part;
  float *lse2;       // [n_seqs][n_kv_heads][group * T], log2 units
  float *x;          // [n_seqs][n_kv_heads][x_len][x_cols], log2 units
  // K's and V's codes as f16 tiles, [n_seqs][n_kv_heads][pre_len][head_dim]; NULL:
  // the codes are read
  uint16_t *pre_k, *pre_v;
  long long pre_len;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// True in one lane of the (converged) warp; as a predicate that the compiler
// knows to be one thread's, it leaves the MMAs' operands in uniform registers.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
}

// ----------------------------------------------------- a row's two references
//
// A row sums its probabilities p = 2^(x - m) in l, and its outputs from f16 operands
// p 2^(lv + lh) times codes, with lv the exponent of the key's V scale and lh a whole
// number of the row's own: its outputs are in units of 2^(m - lh).

// Moves them up to t (for p) and u (for the operands) where they lie below: true if
// so, and then f is what the outputs are multiplied by.  Stays where t is -infinity or
// NaN.
__device__ __forceinline__ bool move_reference(float t, float u, float &m, float &l, float &lh,
                                               float &f) {
  if (!(t > m || u > m - lh)) return false;
  const float to = fmaxf(m, t), up = to - m;       // from -infinity: infinity
  const float h = floorf(fminf(to - u, lh + up));  // to - h: u, or the old one, and 1 above at most
  const float g = ex2(-up);
  f = m == -INFINITY ? 0.f : ex2(h - lh - up);
  l *= g;
  m = to;
  lh = h;
  return true;
}

// 2^(lv + lh), bounded so that a probability of zero times it is zero.
__device__ __forceinline__ float v_factor(float lv, float lh) { return ex2(fminf(lv + lh, 126.f)); }

// 1 / l for a row's sum (to an ulp), 0 for one that sees nothing; NaN stays.
__device__ __forceinline__ float inverse(float l) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(l));
  return l > 0.f || l != l ? y : 0.f;
}

// ------------------------------------------------------------ the work split

struct SeqInfo {
  int len, n;   // cached rows, new tokens
  int tiles;    // key tiles per segment (0: nothing to do, or refused)
  bool bad;
};

__device__ __forceinline__ SeqInfo seq_info(const Cache8AttendArgs &a, int s) {
  SeqInfo q;
  q.len = a.lens[s];
  q.n = a.n_new ? a.n_new[s] : a.T;
  q.bad = q.len < 0 || q.len > a.max_len || q.n < 0 || q.n > a.T;
  q.tiles = q.bad || q.n == 0 ? 0 : (q.len + kTile - 1) / kTile;
  return q;
}

// The whole call's list of tiles and its cut into runs.  A segment counts as
// `pad` tiles more than it has, put before its first: what a CTA spends on
// beginning and ending one (queries, the merge of its warps), so that runs
// over many short sequences take no longer than the others.
struct Split {
  int total, run, pad;  // counted tiles, counted tiles per run
};

__device__ __forceinline__ int warp_sum(int x) {
  return static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(x)));
}
// Called by whole warps.  mine: the tiles of sequence `lane`, for the calls below.
__device__ __forceinline__ Split split_of(const Cache8AttendArgs &a, int units, int ctas, int *mine) {
  const int lane = threadIdx.x & 31;
  *mine = lane < a.n_seqs ? seq_info(a, lane).tiles : 0;
  int tiles = *mine, segments = *mine > 0 ? 1 : 0;
  for (int s = lane + 32; s < a.n_seqs; s += 32) {
    const int t = seq_info(a, s).tiles;
    tiles += t;
    segments += t > 0 ? 1 : 0;
  }
  tiles = warp_sum(tiles) * units;
  segments = warp_sum(segments) * units;
  Split w;
  w.pad = tiles >= 16 * ctas ? 2 : tiles >= 4 * ctas ? 1 : 0;
  w.total = tiles + w.pad * segments;
  w.run = max((w.total + ctas - 1) / ctas, 1);
  return w;
}
// Counted tiles before sequence `seq`.
__device__ __forceinline__ int counted_before(const Cache8AttendArgs &a, const Split &w, int units,
                                              int mine, int seq) {
  const int lane = threadIdx.x & 31;
  int sum = lane < seq && mine > 0 ? mine + w.pad : 0;
  for (int s = lane + 32; s < seq; s += 32) {
    const int t = seq_info(a, s).tiles;
    sum += t > 0 ? t + w.pad : 0;
  }
  return warp_sum(sum) * units;
}

// A position in the call's list of tiles.
struct Cursor {
  int seq, unit, tile;  // unit = KV head * row_blocks + row block
  int at;               // counted tiles from the run's start to this tile
  SeqInfo q;

  // Called by whole warps: the first tile at counted tile x (x < total) or after it.
  __device__ __forceinline__ void seek(const Cache8AttendArgs &a, const Split &w, int units,
                                       int mine, int x) {
    const int lane = threadIdx.x & 31;
    int before = 0;
    for (int s0 = 0;; s0 += 32) {
      int t = s0 == 0 ? mine : s0 + lane < a.n_seqs ? seq_info(a, s0 + lane).tiles : 0;
      t = t > 0 ? (t + w.pad) * units : 0;
      int sum = t;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += y;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, before + sum > x);
      if (hit != 0 || s0 + 32 >= a.n_seqs) {
        const int l = hit != 0 ? __ffs(hit) - 1 : 0;
        seq = s0 + l;
        x -= before + __shfl_sync(0xffffffffu, sum - t, l);
        break;
      }
      before += __shfl_sync(0xffffffffu, sum, 31);
    }
    q = seq_info(a, seq);
    unit = x / (q.tiles + w.pad);
    const int pos = x - unit * (q.tiles + w.pad) - w.pad;
    tile = max(pos, 0);
    at = max(-pos, 0);
  }
  // Whether it names a tile of the call (for the debug build).
  __device__ __forceinline__ bool inside(const Cache8AttendArgs &a, int units) const {
    return seq >= 0 && seq < a.n_seqs && unit >= 0 && unit < units && tile >= 0 && tile < q.tiles;
  }
  __device__ __forceinline__ void next(const Cache8AttendArgs &a, const Split &w, int units) {
    ++at;
    if (++tile < q.tiles) return;
    at += w.pad;
    tile = 0;
    if (++unit < units) return;
    unit = 0;
    do {
      if (++seq >= a.n_seqs) {
        at = INT32_MAX;  // past the end
        return;
      }
      q = seq_info(a, seq);
    } while (q.tiles == 0);
  }
};

// The first key that not every one of the call's tokens sees.
__device__ __forceinline__ int hidden_from(const SeqInfo &q) {
  return q.n > 1 ? q.len - q.n + 1 : INT32_MAX;
}

// Where row r of a (sequence, KV head) lives in q and out, in rows.
__device__ __forceinline__ size_t q_row(const Cache8AttendArgs &a, int seq, int kvh, int r) {
  const int t = r / a.group, g = r - t * a.group;
  return (static_cast<size_t>(seq) * a.n_q_heads + kvh * a.group + g) * a.T + t;
}

__device__ __forceinline__ void store_out(__nv_bfloat16 *p, float v) { *p = __float2bfloat16(v); }
__device__ __forceinline__ void store_out(float *p, float v) { *p = v; }
__device__ __forceinline__ void store_out4(__nv_bfloat16 *p, float a, float b, float c, float d) {
  __nv_bfloat162 x = __floats2bfloat162_rn(a, b), y = __floats2bfloat162_rn(c, d);
  *reinterpret_cast<uint2 *>(p) =
      make_uint2(*reinterpret_cast<uint32_t *>(&x), *reinterpret_cast<uint32_t *>(&y));
}
__device__ __forceinline__ void store_out4(float *p, float a, float b, float c, float d) {
  *reinterpret_cast<float4 *>(p) = make_float4(a, b, c, d);
}

// lse of a row from its max and sum (log2 units): log2 units for the weights
// pass, natural for the caller.
__device__ __forceinline__ void store_lse(const AttendArgs &p, int seq, int kvh, int r, float m,
                                          float l) {
  const Cache8AttendArgs &a = p.a;
  const float z = l > 0.f || l != l ? m + log2f(l) : -INFINITY;
  p.lse2[(static_cast<size_t>(seq) * a.n_kv_heads + kvh) * a.group * a.T + r] = z;
  if (a.lse) a.lse[q_row(a, seq, kvh, r)] = z * kLn2;
}

}  // namespace cache8

// cache8_attend_tc.cu: bf16, head_dim 64 or 128, p.row_tiles tiles of 128 query
// rows a CTA.
bool launch_attend_tc(const cache8::AttendArgs &p, int row_tiles, cudaStream_t stream);
// After the join: the outputs that a NaN in V reaches, for T > 1.
bool launch_mark_nan(const cache8::AttendArgs &p, cudaStream_t stream);
// cache8_weights_tc.cu: the weights from lse2 and the keys, after the above.
bool launch_weights_tc(const cache8::AttendArgs &p, cudaStream_t stream);

}  // namespace bkv
