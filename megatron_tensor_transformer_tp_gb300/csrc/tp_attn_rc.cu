// Softmax attention that stores no probabilities, its gradient, and both with
// a learned relative position bias, on the tcgen05 tensor cores.
//
// With x_ij = scale q_i . k_j (+ bias[bucket(j - i)]) over the keys that query
// i sees (its own sequence; j <= i if causal):
//   forward   lse_i = log sum_j exp(x_ij),  C_i = sum_j exp(x_ij - lse_i) v_j
//   backward  P_ij = exp(x_ij - lse_i),  D_i = dC_i . C_i,  dP_ij = dC_i . v_j,
//             dS_ij = P_ij (dP_ij - D_i),
//             dV_j = sum_i P_ij dC_i,  dK_j = scale sum_i dS_ij q_i,
//             dQ_i = scale sum_j dS_ij k_j,  dbias[u] = sum of dS_ij over bucket u.
// Scores and probabilities live in TMEM and registers only: 128 x 128 tiles,
// fp32 accumulators, exponentials as 2^(x log2 e).
//
// Three tensor-core kernels, one CTA an SM, in which one warp loads tiles by TMA,
// one or two issue products, 16 do the element-wise work (a TMEM lane is a row of
// the score tile) and one prepares tables:
//   rc_fwd_kernel   one or two 128-row query tiles of a head over its key tiles;
//                   the products of one run under the softmax of the other.
//   rc_dq_kernel    a 128-row query tile of a head over its key tiles.  It also
//                   computes D, and sums dS by relative distance for the bias.
//   rc_dkv_kernel   a 128-row key tile of a K/V head, over the query tiles of
//                   every query head that shares it.  It computes the
//                   transposed scores S^T = K Q^T and dP^T = V dC^T, so P^T
//                   and dS^T are A operands straight from TMEM.
// The backward computes the scores and dP in both of its kernels (seven products
// a tile instead of five): no output is summed by atomics, so results do not
// depend on the order in which CTAs run, and dQ needs no fp32 buffer in memory.
// CTAs are persistent and take items from a counter; where an item outlasts an
// SM's share of the work, clusters share items (cluster_parts).
//
// All three are bound by arithmetic: a tile of 128 x 128 scores of width 128 takes
// 512 cycles of tensor cores a product and reads 64 KB that other CTAs read too.
// Measured on a GB300 (cuBLAS reaches 1.87 PFLOP/s in bf16 there), in matrix work
// that the definition needs, four and ten flops a visible pair and column:
//   causal, one sequence of 16384, 8 heads of 128, 2 K/V heads
//     forward 343 us, 1.6 PFLOP/s; backward 1.18 ms, 1.17 PFLOP/s, which is 1.63
//     with the two products that are computed twice
//   causal, 2 x 2048, 32 heads of 128: 62 us, 1.11 PFLOP/s; 198 us, 0.87 PFLOP/s
//   bias of both directions, 4 x 1024, 16 heads of 64: 30 us; 96 us, 0.45 PFLOP/s:
//     at 64 columns a product takes 256 cycles and the element-wise work as long as
//     before, which with the waits between its steps is then the bound.
// Every wait on an mbarrier is bounded, as in the GEMM engine, and after one that
// runs out the CTA's warps leave.  Without a limit are the barriers of a warp pair, of
// the compute warps, of the CTA and of the cluster, which every warp reaches because
// nothing before them waits without a limit, and the waits for the kernel before,
// which ends for the same reason.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "tp_device.cuh"
#include "tp_internal.h"
#include "tp_tcgen05.cuh"

namespace tp {
namespace {

// Compute warps first, then the MMA warps, the TMA warp and a warp for tables
// (forward and dQ: the bias of a head; dK, dV: the rows' lse and D).  The forward
// has two compute warps on every 32 rows of a score tile (64 columns each) and two
// tiles, the backward kernels four (32 columns each).  16 warps against 8, with a
// product warp a query tile: forward of 16384, 8 heads of 128, 355 us and 447 us.
constexpr int kFwdWarps = 16, kBwdWarps = 16;
constexpr int kFwdThreads = 32 * (kFwdWarps + 4), kDkvThreads = 32 * (kBwdWarps + 4), kDqThreads = 32 * (kBwdWarps + 3);
constexpr int kPanel = 128 * 128;    // bytes of 128 rows x 64 bf16 columns (one swizzle width)
constexpr int kBarBytes = 512;
constexpr int kMaxSmem = 227 * 1024;  // of a CTA
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLn2Rest = static_cast<float>(0.6931471805599453094 - static_cast<double>(kLn2));
// Finite entries of the bias's table: half a step of an lse of this size is 2^-8,
// which is what the backward's probabilities are then off by, as much as their
// rounding to bf16.  Entries below count as -infinity, those above are reported.
constexpr float kMaxEntry = 131072.f;

// The smem distance table covers [-(md + kPad), md + kPad], so that a tile that
// holds any distance inside (-md, md) indexes it without clamping.
constexpr int kPad = 255;
// (an even number of entries over: whole 16 bytes)
__host__ __device__ constexpr int table_floats(int md) { return (2 * (md + kPad) + 1 + 3) & ~3; }

// ---------------------------------------------------------------------------
// PTX wrappers of this file
// ---------------------------------------------------------------------------
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1,
                                            int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

// D += A B with A (128 x 16 bf16, two per 32-bit column) in TMEM.
__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"(accumulate));
}

__device__ __forceinline__ float as_f(uint32_t u) { return __uint_as_float(u); }

// 32 columns of the warp's 32 lanes, without waiting for them.
__device__ __forceinline__ void tmem_ld32_issue(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
// Waits for the loads issued so far.  The registers pass through the statement,
// so no use of them can be moved in front of the wait.
__device__ __forceinline__ void tmem_ld32_wait(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                 "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]),
                 "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]),
                 "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]),
                 "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}
// 8 columns times f, in place.
__device__ __forceinline__ void tmem_scale8(uint32_t taddr, float f) {
  uint32_t r[8];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int q = 0; q < 8; ++q) r[q] = __float_as_uint(as_f(r[q]) * f);
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(taddr)
               : "memory");
}
// The same registers as they are.
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void named_bar(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// wait_bounded by a whole warp, with one answer for all of its lanes; the clock
// and the abort flag are looked at once in a while only.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, const WaitCtx& w) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  unsigned long long t0 = 0;
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 16; ++i)
      if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    const unsigned long long t = global_ns();
    if (t0 == 0) t0 = t;
    const bool late = t - t0 > w.limit_ns;
    if (late) {
      *w.abort_flag = 1;
      atomicOr(w.err, kErrTimeout);
    }
    if (__any_sync(0xffffffffu, late || *w.abort_flag)) return false;
  }
}

// Two fp32 values a register pair: one instruction for both.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Barrier `id` of `threads` threads; whether any of them said yes.
__device__ __forceinline__ bool named_bar_any(int id, int threads, bool yes) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 q, %3, 0;\n\t"
      "bar.red.or.pred p, %1, %2, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(any)
      : "r"(id), "r"(threads), "r"(static_cast<uint32_t>(yes))
      : "memory");
  return any != 0;
}

// ---------------------------------------------------------------------------
// Work items
// ---------------------------------------------------------------------------
// Unit `unit` of the launch: a run of `rows` tokens of a sequence.  Units are
// taken so that long contractions come early: by rank, the first (or, where
// `last_first`, the last) runs of all sequences, then their second ones and so
// on.  Sequences given by seq_starts are clamped into [0, T]; starts that
// decrease or leave [0, T] are reported in the error word by the first block.
// Called by a whole warp.
struct Unit {
  int start, len, tile;  // first token and length of the sequence, tile inside it
};
// Up to 32 sequences are held by a warp, a lane each; more go in their own
// order, looked for from where the CTA's last unit was found.  (Four a lane made
// the whole forward 4% slower.)
struct Units {
  int start, len, n;  // of the lane's sequence
  int rows, top;      // the longest sequence's runs; not held: the first sequence that is looked at next
  int64_t base;       // not held: units of the sequences before that one
  bool held;

  __device__ __forceinline__ static bool read(const RcParams& p, int i, int64_t& a, int64_t& e) {
    a = e = 0;
    if (i >= p.b) return true;
    a = __ldcg(p.seq_starts + i);
    e = __ldcg(p.seq_starts + i + 1);
    const bool fine = a >= 0 && e >= a && e <= p.T;
    a = min(max(a, static_cast<int64_t>(0)), p.T);
    e = min(max(e, a), p.T);
    return fine;
  }
  __device__ __forceinline__ Units(const RcParams& p, int rows_, int lane) : rows(rows_), top(0), base(0), held(false) {
    if (p.seq_starts == nullptr) return;
    held = p.b <= 32;
    int64_t a, e;
    bool fine = read(p, held ? lane : p.b, a, e);
    start = static_cast<int>(a);
    len = static_cast<int>(e - a);
    n = (len + rows - 1) / rows;
    top = held ? __reduce_max_sync(0xffffffffu, n) : 0;
    if (!held && blockIdx.x == 0)
      for (int i = lane; i < p.b; i += 32) fine &= read(p, i, a, e);
    if (!fine && blockIdx.x == 0) atomicOr(p.err, kErrInvalid);
  }
  // Units of rank below r.
  __device__ __forceinline__ int64_t below(int r) const { return __reduce_add_sync(0xffffffffu, min(n, r)); }
  // false: there is no such unit.  The units of one Units object never decrease.
  __device__ __forceinline__ bool find(const RcParams& p, int64_t unit, bool last_first, int lane, Unit& u) {
    if (p.seq_starts == nullptr) {
      const int per = (p.s + rows - 1) / rows;
      const int rank = static_cast<int>(unit / p.b), seq = static_cast<int>(unit % p.b);
      if (rank >= per) return false;
      u.tile = last_first ? per - 1 - rank : rank;
      u.start = seq * p.s;
      u.len = p.s;
      return true;
    }
    if (held) {
      if (unit >= below(top)) return false;
      int lo = 0, hi = top - 1;  // the rank: the largest r with below(r) <= unit
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (below(mid) <= unit) lo = mid;
        else hi = mid - 1;
      }
      // among the sequences that have this rank, in order
      const unsigned has = __ballot_sync(0xffffffffu, n > lo);
      const int src = __fns(has, 0, static_cast<int>(unit - below(lo)) + 1);
      u.start = __shfl_sync(0xffffffffu, start, src);
      u.len = __shfl_sync(0xffffffffu, len, src);
      const int runs = __shfl_sync(0xffffffffu, n, src);
      u.tile = last_first ? runs - 1 - lo : lo;
      return true;
    }
    for (; top < p.b; top += 32) {
      int64_t a, e;
      read(p, top + lane, a, e);
      const int runs = static_cast<int>((e - a + rows - 1) / rows);
      int64_t incl = runs;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, base + incl > unit);
      if (hit) {
        const int src = __ffs(hit) - 1;
        u.start = static_cast<int>(__shfl_sync(0xffffffffu, a, src));
        u.len = static_cast<int>(__shfl_sync(0xffffffffu, e - a, src));
        const int all = __shfl_sync(0xffffffffu, runs, src);
        const int t = static_cast<int>(unit - __shfl_sync(0xffffffffu, base + incl - runs, src));
        u.tile = last_first ? all - 1 - t : t;
        return true;
      }
      base += __shfl_sync(0xffffffffu, incl, 31);
    }
    return false;
  }
};

// ---------------------------------------------------------------------------
// Relative position bias
// ---------------------------------------------------------------------------
// Bucket of the distance delta = key - query.
__device__ __forceinline__ int bucket_of(const RcBias& b, int delta) {
  int add = 0, n = -delta;
  if (b.both) {
    if (delta > 0) add = b.side;
    n = delta > 0 ? delta : -delta;
  }
  n = max(n, 0);
  int lo = 0, hi = b.side - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (b.first[mid] <= n) lo = mid;
    else hi = mid - 1;
  }
  return add + lo;
}
// map[delta + md + kPad] = bucket of the clamped distance: of the arguments
// alone, so a kernel makes it before it waits for the one in front of it.
__device__ __forceinline__ void fill_map(const RcBias& b, uint8_t* map) {
  for (int i = threadIdx.x; i < table_floats(b.md); i += blockDim.x)
    map[i] = static_cast<uint8_t>(bucket_of(b, min(max(i - (b.md + kPad), -b.md), b.md)));
}
// tab[delta + md + kPad] = bias of the clamped distance; by one warp, through the
// head's column of the table in `vals`; the map's and the table's rows are padded
// to fours.  (Not times log2 e: the kernels take differences of entries and lse
// first, which are exact where both are large and their probabilities are not 0.)
__device__ __forceinline__ void fill_table_warp(const RcParams& p, int head, const uint8_t* map, float* vals,
                                                float* tab, int lane) {
  bool high = false;
  for (int u = lane; u < p.bias.nb; u += 32) {
    const float v = __ldcg(p.table + static_cast<int64_t>(u) * p.H + head);
    vals[u] = v < -kMaxEntry ? -INFINITY : v;
    high |= v > kMaxEntry;
  }
  if (high) atomicOr(p.err, kErrInvalid);
  __syncwarp();
  const int n = table_floats(p.bias.md);
#pragma unroll 2
  for (int i = 4 * lane; i < n; i += 128) {
    const uchar4 m = *reinterpret_cast<const uchar4*>(map + i);
    *reinterpret_cast<float4*>(tab + i) = make_float4(vals[m.x], vals[m.y], vals[m.z], vals[m.w]);
  }
}
// How a (query tile at r0, key tile at c0) pair of 128 x 128 sees the bias:
// 0 distances differ, +-1 every distance is clamped to the same end.
__device__ __forceinline__ int bias_side(int md, int r0, int c0) {
  if (c0 + 127 - r0 <= -md) return -1;
  if (c0 - r0 - 127 >= md) return 1;
  return 0;
}

// ---------------------------------------------------------------------------
// Pieces that the kernels share
// ---------------------------------------------------------------------------
struct HeadAt {
  int shard, local;
};
__device__ __forceinline__ HeadAt head_at(int head, int per_shard) {
  return HeadAt{head / per_shard, head % per_shard};
}

// 128 rows (from token) of one head as DP / 64 swizzled panels.
template <int DP>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* map, uint32_t bar, int token, HeadAt h) {
#pragma unroll
  for (int c = 0; c < DP / 64; ++c) tma_load_4d(dst + c * kPanel, map, bar, 64 * c, token, h.local, h.shard);
}
// Rows [row, 128) of a tile become zeros (a whole warp); the tensor cores see
// them after the caller's arrival on the tile's barrier.
template <int DP>
__device__ __forceinline__ void zero_rows(uint8_t* tile, int row, int lane) {
#pragma unroll
  for (int c = 0; c < DP / 64; ++c) {
    uint4* q = reinterpret_cast<uint4*>(tile + c * kPanel);
    for (int i = row * 8 + lane; i < 128 * 8; i += 32) q[i] = make_uint4(0, 0, 0, 0);
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
}
// Loads a tile whose rows from `valid` on belong to nobody: they hold another
// sequence's values, or anything, and would reach the sums as 0 x NaN.  The
// copy lands on the side barrier, the rows are cleared, then `bar` completes.
template <int DP>
__device__ __forceinline__ bool load_tail(uint8_t* smem_tile, const CUtensorMap* map, uint32_t bar,
                                          uint32_t tail_bar, uint32_t& tail_phase, int token, HeadAt h, int valid,
                                          int lane, const WaitCtx& w) {
  if (lane == 0) {
    mbar_arrive_expect_tx(tail_bar, DP / 64 * kPanel);
    load_tile<DP>(smem_addr(smem_tile), map, tail_bar, token, h);
  }
  __syncwarp();
  if (!wait_warp(tail_bar, tail_phase, w)) {
    // aborted: the copy still has to land before the CTA may end
    const unsigned long long t0 = global_ns();
    while (!mbar_try_wait(tail_bar, tail_phase) && global_ns() - t0 <= w.limit_ns) {
    }
    __syncwarp();
    return false;
  }
  tail_phase ^= 1u;
  zero_rows<DP>(smem_tile, valid, lane);
  if (lane == 0) mbar_arrive(bar);
  return true;
}

// The MMA warp runs its loop as a whole warp and one elected lane issues: the
// descriptors are then warp-uniform values.  Issued from a branch that only
// lane 0 takes, each 128 x 128 x 16 product cost 75 to 160 cycles of issue for
// its 64 cycles of work.
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok));
  return ok != 0;
}
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// S = A B^T over the head width: both K-major in shared memory, 128 x 128.
template <int KSTEPS>
__device__ __forceinline__ void mma_scores_k(uint32_t d_tmem, uint64_t ad, uint64_t bd, uint32_t idesc) {
#pragma unroll
  for (int kk = 0; kk < KSTEPS; ++kk) {
    const uint32_t off = ((kk >> 2) * kPanel + (kk & 3) * 32) >> 4;
    mma_bf16(d_tmem, ad + off, bd + off, idesc, kk > 0);
  }
}
template <int DP>
__device__ __forceinline__ void mma_scores(uint32_t d_tmem, uint32_t a, uint32_t b, int ksteps) {
  const uint64_t ad = sdesc(a, 16, 1024), bd = sdesc(b, 16, 1024);
  const uint32_t idesc = idesc_bf16(0, 0, 128);
  constexpr int K0 = DP == 128 ? 4 : 0;
  if (ksteps == K0 + 4) mma_scores_k<K0 + 4>(d_tmem, ad, bd, idesc);
  else if (ksteps == K0 + 3) mma_scores_k<K0 + 3>(d_tmem, ad, bd, idesc);
  else if (ksteps == K0 + 2) mma_scores_k<K0 + 2>(d_tmem, ad, bd, idesc);
  else mma_scores_k<K0 + 1>(d_tmem, ad, bd, idesc);
}
// The same with A (128 x 16 KSTEPS) in TMEM.
template <int KSTEPS>
__device__ __forceinline__ void mma_scores_ts_k(uint32_t d_tmem, uint32_t a_tmem, uint64_t bd, uint32_t idesc) {
#pragma unroll
  for (int kk = 0; kk < KSTEPS; ++kk)
    mma_bf16_ts(d_tmem, a_tmem + 8 * kk, bd + (((kk >> 2) * kPanel + (kk & 3) * 32) >> 4), idesc, kk > 0);
}
template <int DP>
__device__ __forceinline__ void mma_scores_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b, int ksteps) {
  const uint64_t bd = sdesc(b, 16, 1024);
  const uint32_t idesc = idesc_bf16(0, 0, 128);
  constexpr int K0 = DP == 128 ? 4 : 0;
  if (ksteps == K0 + 4) mma_scores_ts_k<K0 + 4>(d_tmem, a_tmem, bd, idesc);
  else if (ksteps == K0 + 3) mma_scores_ts_k<K0 + 3>(d_tmem, a_tmem, bd, idesc);
  else if (ksteps == K0 + 2) mma_scores_ts_k<K0 + 2>(d_tmem, a_tmem, bd, idesc);
  else mma_scores_ts_k<K0 + 1>(d_tmem, a_tmem, bd, idesc);
}

// D (+)= A B: A 128 x 128 bf16 in TMEM, B = 128 rows of a tile as stored
// (contraction over its rows).  Each compute warp writes its part of A where it
// read its scores: with PARTS parts, part x's columns start at 128 x / PARTS.
// FIRST, COUNT: the 16-row steps of each part that are taken.  STRIDE: TMEM
// columns from part to part, where not as above.
template <int PARTS, int FIRST = 0, int COUNT = 8 / PARTS, int STRIDE = 128 / PARTS>
__device__ __forceinline__ void mma_rows(uint32_t d_tmem, uint32_t a_tmem, uint32_t b, uint32_t idesc,
                                         bool accumulate) {
  const uint64_t bd = sdesc(b, kPanel, 1024);
#pragma unroll
  for (int h = 0; h < PARTS; ++h) {
#pragma unroll
    for (int kk = FIRST; kk < FIRST + COUNT; ++kk)
      mma_bf16_ts(d_tmem, a_tmem + STRIDE * h + 8 * kk, bd + (8 / PARTS * h + kk) * (2048 >> 4), idesc,
                  accumulate || h > 0 || kk > FIRST);
  }
}

// A row's columns that the first of two warps takes, in 32s.
__device__ __forceinline__ int first_columns(int d) { return min(d, 32 * ((d + 63) / 64)); }

// COLS fp32 values, scaled, as bf16 pairs.
template <int COLS>
__device__ __forceinline__ void pack_columns(const uint32_t* v, float mul, uint32_t* q) {
  const uint64_t mul2v = pack2(mul, mul);
#pragma unroll
  for (int i = 0; i < COLS / 2; ++i) {
    float a, b;
    unpack2(mul2(pack2(as_f(v[2 * i]), as_f(v[2 * i + 1])), mul2v), a, b);
    q[i] = pack_bf16x2(a, b);
  }
}
__device__ __forceinline__ void st_global32(__nv_bfloat16* out, const uint32_t* r) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(out), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// n of COLS bf16 values of each lane's row to memory, rows in order over the lanes
// and `ld` apart; `mine`: the row is stored.  By a whole warp.  `wide`: every row
// start is 32-byte aligned and n a multiple of 16.  Two lanes then swap halves, so
// that a store covers 64 bytes of a row: 64 KB by the 16 warps of all SMs at once
// take 2100 cycles, with 32 bytes a row 3100.
template <int COLS>
__device__ __forceinline__ void put_columns(const uint32_t* q, int n, bool mine, __nv_bfloat16* out, int64_t ld,
                                            bool wide) {
  if (wide) {
    const bool odd = threadIdx.x & 1;
    const bool other = __shfl_xor_sync(0xffffffffu, mine, 1);
    const bool first = odd ? other : mine, second = odd ? mine : other;
    __nv_bfloat16* row = (odd ? out - ld : out) + (odd ? 16 : 0);  // of the pair's first row
#pragma unroll
    for (int c = 0; c < COLS; c += 32) {
      const uint32_t* r = q + c / 2;
      uint32_t x[8], y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t v = __shfl_xor_sync(0xffffffffu, odd ? r[i] : r[8 + i], 1);
        x[i] = odd ? v : r[i];
        y[i] = odd ? r[8 + i] : v;
      }
      if (c + (odd ? 16 : 0) < n) {
        if (first) st_global32(row + c, x);
        if (second) st_global32(row + ld + c, y);
      }
    }
  } else if (mine) {
#pragma unroll
    for (int c = 0; c < COLS; c += 8)
      if (c < n) *reinterpret_cast<uint4*>(out + c) = make_uint4(q[c / 2], q[c / 2 + 1], q[c / 2 + 2], q[c / 2 + 3]);
  }
}
template <int COLS>
__device__ __forceinline__ void store_columns(const uint32_t* v, int n, float mul, bool mine, __nv_bfloat16* out,
                                              int64_t ld, bool wide) {
  uint32_t q[COLS / 2];
  pack_columns<COLS>(v, mul, q);
  put_columns<COLS>(q, n, mine, out, ld, wide);
}

// COLS bf16 columns from column `first` of the thread's row of a swizzled tile
// as COLS / 2 TMEM columns.
template <int COLS>
__device__ __forceinline__ void tile_to_tmem(uint32_t taddr, const uint8_t* tile, int row, int first) {
#pragma unroll
  for (int c = 0; c < COLS; c += 16) {
    uint4 v[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int col = first + c + 8 * q;  // 16 bytes; chunk x of a row lies at x ^ (row mod 8)
      v[q] = *reinterpret_cast<const uint4*>(tile + (col >> 6) * kPanel + row * 128 +
                                             ((((col & 63) >> 3) ^ (row & 7)) << 4));
    }
    const uint32_t r[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
    tmem_st8(taddr + c / 2, r);
  }
}

// What a row's log-sum-exp adds to its scores; a row that saw no key has no
// probabilities.
__device__ __forceinline__ float row_shift(float lse) { return lse == -INFINITY ? -INFINITY : -lse; }
// A row's log-sum-exp from its exponents' reference m (log2) and their sum l:
// (m + log2 l) ln 2, where m ln 2 keeps what its rounding would lose, so that the
// result is rounded once.
__device__ __forceinline__ float row_lse(float m, float l) {
  if (m == -INFINITY) return -INFINITY;
  const float t = __fmul_rn(m, kLn2);  // (not to be joined with the sum below)
  return t + fmaf(log2f(l), kLn2, fmaf(m, kLn2, -t) + m * kLn2Rest);
}

// The product of COLS columns from `first` of the thread's row of two tiles.
template <int COLS>
__device__ __forceinline__ float dot_tiles(const uint8_t* x, const uint8_t* y, int row, int first) {
  float acc = 0.f;
#pragma unroll
  for (int c = 0; c < COLS; c += 8) {
    const int col = first + c;
    const int at = (col >> 6) * kPanel + row * 128 + ((((col & 63) >> 3) ^ (row & 7)) << 4);
    const uint4 a = *reinterpret_cast<const uint4*>(x + at), b = *reinterpret_cast<const uint4*>(y + at);
    const uint32_t aa[4] = {a.x, a.y, a.z, a.w}, bb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float x0, x1, y0, y1;
      unpack_bf16x2(aa[q], x0, x1);
      unpack_bf16x2(bb[q], y0, y1);
      acc = fmaf(x0, y0, acc);
      acc = fmaf(x1, y1, acc);
    }
  }
  return acc;
}

// Copies in flight of the TMA warp: the barriers that one was issued on, and
// the phase that it completes.  After an abort they are waited for.
struct Flight {
  uint32_t used = 0, phase = 0;
  __device__ __forceinline__ void note(int i, uint32_t ph) {
    used |= 1u << i;
    phase = (phase & ~(1u << i)) | (ph << i);
  }
  __device__ __forceinline__ void drain(uint32_t bar0, unsigned long long limit_ns) const {
    for (int i = 0; i < 32; ++i) {
      if (!((used >> i) & 1u)) continue;
      const unsigned long long t0 = global_ns();
      while (!mbar_try_wait(bar0 + 8u * i, (phase >> i) & 1u))
        if (global_ns() - t0 > limit_ns) break;
    }
  }
};
__device__ __forceinline__ void drain_mma(uint32_t bar, unsigned long long limit_ns) {
  mma_commit(bar);
  const unsigned long long t0 = global_ns();
  while (!mbar_try_wait(bar, 0))
    if (global_ns() - t0 > limit_ns) break;
}

__device__ __forceinline__ void tmem_alloc512(uint32_t slot) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(512)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc512(uint32_t base) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(512) : "memory");
}

// Shared-memory head of every kernel here: barriers, the TMEM address, the
// abort flag and the CTA's items.
constexpr int kMaxBars = 48;
struct Head {
  uint64_t bar[kMaxBars];
  uint32_t tmem;
  int abort_flag;
  int items[16];
};
static_assert(sizeof(Head) <= kBarBytes, "barrier area");

__device__ __forceinline__ uint8_t* align1024(uint8_t* q) {
  return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(q) + 1023) & ~static_cast<uintptr_t>(1023));
}

// Items of a launch: unit u of head h is item u * heads + h.  A CTA begins with
// item blockIdx.x and then takes the next one from a counter of the launch, so
// long and short items balance whatever their order; the last CTA to leave
// clears the counters for the next launch with this slot.  Launches rotate over
// kRcSlots of them.  A captured launch may run beside any later one, so it gets
// a slot that no other launch ever has, or, when those are used up, none: its CTAs
// then take every gridDim.x-th item.  (12 packed sequences, backward with 16 / 4
// heads of 96: 275 us by counter, 421 us so; forward with 32 / 8 heads of 128: 191
// and 226 us; two sequences of 2048, backward: 198 and 206 us.)
constexpr int kRcSlots = 4096, kRcGraphSlots = 1 << 16;
__device__ int g_rc_items[2 * (kRcSlots + kRcGraphSlots)];
struct ItemWalk {
  Units units;
  int64_t item;
  int heads, index;  // index: head of the item
  bool first;
  __device__ __forceinline__ ItemWalk(const RcParams& p, int n, int rows, int lane)
      : units(p, rows, lane), item(blockIdx.x / p.parts), heads(n), index(0), first(true) {}
  // The next item that has rows, by a whole warp; false: there is none.
  // `zero`: an item without rows leaves that many zeros there.
  __device__ __forceinline__ bool next(const RcParams& p, bool last_first, int lane, Unit& u, float* zero = nullptr,
                                       int nzero = 0) {
    while (true) {
      if (!first) {
        if (p.items * p.parts <= gridDim.x) return false;  // an item each
        if (p.slot < 0) {
          item += gridDim.x;
        } else {
          int v = 0;
          if (lane == 0) v = atomicAdd(g_rc_items + 2 * p.slot, 1);
          item = static_cast<int64_t>(gridDim.x) + __shfl_sync(0xffffffffu, v, 0);
        }
      }
      if (item >= p.items) return false;
      first = false;
      index = static_cast<int>(item % heads);
      if (units.find(p, item / heads, last_first, lane, u)) return true;
      if (zero == nullptr) return false;  // nor do later items have rows
      for (int i = lane; i < nzero; i += 32) zero[item * nzero + i] = 0.f;
    }
  }
};

// Common entry: barriers 0 .. nbars-1 with the given counts, TMEM.  WAIT: for the
// kernels before.
template <int WARPS, bool WAIT = true, class Counts>
__device__ __forceinline__ void enter(Head* hd, int nbars, Counts&& count) {
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < nbars; ++i) mbar_init(smem_addr(hd->bar + i), count(i));
    hd->abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == WARPS) tmem_alloc512(smem_addr(&hd->tmem));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (WAIT) pdl_wait();
  pdl_trigger();
}
template <int WARPS>
__device__ __forceinline__ void leave(Head* hd) {
  tc_fence_before();
  __syncthreads();
  if ((threadIdx.x >> 5) == WARPS) {
    tc_fence_after();
    tmem_dealloc512(hd->tmem);
  }
}
template <int WARPS>
__device__ __forceinline__ void leave(Head* hd, const RcParams& p) {
  leave<WARPS>(hd);
  if (threadIdx.x == 0 && p.slot >= 0) {
    int* ctr = g_rc_items + 2 * p.slot;
    __threadfence();
    if (atomicAdd(ctr + 1, 1) == static_cast<int>(gridDim.x) - 1) {
      atomicExch(ctr, 0);
      atomicExch(ctr + 1, 0);
    }
  }
}

// Cluster of the CTAs that share an item.
__device__ __forceinline__ int cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return static_cast<int>(r);
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// 16 bytes at the same shared-memory address of CTA `rank`.
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr, int rank) {
  float4 v;
  asm volatile(
      "{\n\t.reg .b32 a;\n\t"
      "mapa.shared::cluster.u32 a, %4, %5;\n\t"
      "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];\n\t}"
      : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
      : "r"(addr), "r"(rank)
      : "memory");
  return v;
}

// ===========================================================================
// Forward
// ===========================================================================
// What the TMA warp tells the other warps of an item: two slots, so that it
// can be one item ahead.
struct FwdItem {
  int start, len, row0, head;  // row0: position of the first query row
  int n[2];                    // key tiles of the query tiles (0: there is none)
};

template <int DP>
struct FwdShape {
  static constexpr int kTile = DP / 64 * kPanel;
  static constexpr int kStages = DP == 128 ? 2 : 4;  // K tiles and V tiles held, each
  static constexpr int kPart = 2 * 2 * 256 * 4;  // row maxima and row sums of the two column halves
  static constexpr int kSmem = 2 * kTile + 2 * kStages * kTile + kBarBytes + kPart + 1024;
  // barriers
  static constexpr int qfull = 0, kfull = 2, vfull = kfull + kStages, tail = vfull + kStages, kempty = tail + 1,
                       vempty = kempty + kStages, sfull = vempty + kStages, pfull = sfull + 2, odone = pfull + 4,
                       ofree = odone + 2, qempty = ofree + 2, info = qempty + 2, tabfull = info + 2,
                       free_ = tabfull + 2, sread = free_ + 2, pvdone = sread + 2, drain = pvdone + 2,
                       count = drain + 2;
  static_assert(count <= kMaxBars && kempty <= 32, "barriers");
  template <bool BIAS>
  static uint32_t __device__ __forceinline__ arrivals(int i) {
    if (i >= pfull && i < odone) return 8u;
    if (i >= ofree && i < qempty) return 8u;
    if (i >= free_ && i < sread) return kFwdWarps + 2 + (BIAS ? 1 : 0);
    if (i >= sread && i < pvdone) return 8u;
    return i >= kempty && i < sfull ? 2u : 1u;
  }
};

// One pass over the keys with a running reference m and sum l a row,
//   O = sum_j 2^(x_j log2 e - m) v_j,  l = sum_j 2^(x_j log2 e - m),  C = O / l,
//   lse = (m + log2 l) ln 2,
// where m follows the row's maximum only when that has grown past m by 16, so O is
// rescaled rarely and no term exceeds 2^16.  Scores and probabilities stay in TMEM;
// probabilities are rounded to bf16 as operands of the second product, while l sums
// them in fp32.
//
// A tile of 128 x 128 x 128 is 1024 cycles of products and 16384 exponentials; a
// pair of query tiles takes 2500 cycles against 2056 of products, since each waits
// for the other's softmax at times.  16384, 8 heads of 128, causal: 342 us, 1.6
// PFLOP/s (86% of cuBLAS), 2 x 2048, 32 heads: 62 us (59%: a sequence has 8.5 key
// tiles a query tile, of which the diagonal's are half hidden, and an item's output
// and first scores take as long as one or two tiles more).  Two key and value tiles held, as much as fits
// beside two query tiles.
//
// Persistent: a CTA takes (query rows, head) items until there are none.  The
// TMA warp runs ahead into the next item's loads, and its first scores are
// computed while the last outputs are stored.
// SPLIT (where cluster_parts says so): the CTAs of a cluster share an
// item of one query tile, each with every p.parts-th key tile.  Their outputs,
// references and sums meet in shared memory, where each CTA joins its part of
// the rows, in the order of the ranks.
template <int DP, bool BIAS, bool SPLIT>
__global__ void __launch_bounds__(kFwdThreads, 1) rc_fwd_kernel(const __grid_constant__ RcParams p) {
  using L = FwdShape<DP>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint8_t* sQ = smem;
  uint8_t* sK = sQ + 2 * L::kTile;
  uint8_t* sV = sK + L::kStages * L::kTile;
  Head* hd = reinterpret_cast<Head*>(sV + L::kStages * L::kTile);
  volatile FwdItem* items = reinterpret_cast<volatile FwdItem*>(hd->items);
  float* part = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(hd) + kBarBytes);
  float* tabs = part + 1024;  // a table for each slot, the head's values, and the distances' buckets
  const int tabn = BIAS ? table_floats(p.bias.md) : 0;
  float* vals = tabs + 2 * tabn;
  uint8_t* map = reinterpret_cast<uint8_t*>(vals + kMaxRelBuckets);
  if (BIAS) fill_map(p.bias, map);
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  enter<kFwdWarps>(hd, L::count, L::template arrivals<BIAS>);
  const uint32_t bar0 = smem_addr(hd->bar);
  auto bar = [&](int i) { return bar0 + 8u * i; };
  const WaitCtx w{&hd->abort_flag, p.err, p.wait_limit_ns};
  const uint32_t tmem = uniform(hd->tmem);
  // TMEM: scores [0, 256), outputs from 256 and 384.  Heads to 64 wide leave 64
  // columns behind each output, where the probabilities go instead of over the
  // scores: the next scores then wait for the softmax to have read the last ones
  // only, not for the product of its probabilities.
  constexpr bool kApart = DP == 64;
  const int rank = SPLIT ? cluster_rank() : 0;
  auto key_tile = [&](int j) { return SPLIT ? rank + j * p.parts : j; };  // the CTA's j-th

  if (warp == kFwdWarps + 2) {
    Flight fl;
    uint32_t tail_phase = 0;
    uint32_t nq[2] = {0, 0}, c = 0;  // Q tiles loaded, K/V tiles loaded
    bool ok = true, skip = p.fault_skip != 0;
    if (lane == 0) {
      prefetch_tmap(&p.mapQ);
      prefetch_tmap(&p.mapK);
      prefetch_tmap(&p.mapV);
    }
    ItemWalk walk(p, p.H, 128 * p.sub, lane);
    for (uint32_t it = 0; ok; ++it) {
      const int slot = it & 1;
      Unit u{0, 0, 0};
      const bool found = walk.next(p, p.causal != 0, lane, u);
      if (!(ok = wait_warp(bar(L::free_ + slot), ((it >> 1) & 1) ^ 1, w))) break;
      const int row0 = u.tile * 128 * p.sub, head = walk.index, nk_all = (u.len + 127) >> 7;
      int n[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int r = row0 + 128 * t;
        n[t] = !found || t >= p.sub || r >= u.len ? 0 : p.causal ? min(nk_all, (r >> 7) + 1) : nk_all;
        if (SPLIT) n[t] = max(0, n[t] - rank + p.parts - 1) / p.parts;  // (may be none)
      }
      if (lane == 0) {
        items[slot].start = u.start;
        items[slot].len = u.len;
        items[slot].row0 = row0;
        items[slot].head = found ? head : -1;
        items[slot].n[0] = n[0];
        items[slot].n[1] = n[1];
        mbar_arrive(bar(L::info + slot));
      }
      if (!found) break;
      const HeadAt hq = head_at(head, p.hq), hk = head_at(head / p.group, p.hk);
      const int nmax = max(n[0], n[1]), start = u.start, len = u.len;
      auto load_q = [&](int t) {  // lane 0
        if (!wait_bounded(bar(L::qempty + t), (nq[t] & 1) ^ 1, w)) return false;
        mbar_arrive_expect_tx(bar(L::qfull + t), L::kTile);
        fl.note(L::qfull + t, nq[t] & 1);
        load_tile<DP>(smem_addr(sQ + t * L::kTile), &p.mapQ, bar(L::qfull + t), start + row0 + 128 * t, hq);
        return true;
      };
      if (lane == 0 && n[0] > 0) ok = load_q(0);
      ok = __shfl_sync(0xffffffffu, ok, 0);
      for (int j = 0; ok && j < nmax; ++j, ++c) {
        const int st = c % L::kStages, jk = key_tile(j);
        const uint32_t ph = (c / L::kStages) & 1;
        if (lane == 0) {
          ok = ok && wait_bounded(bar(L::kempty + st), ph ^ 1u, w);
          if (ok && !skip) {
            mbar_arrive_expect_tx(bar(L::kfull + st), L::kTile);
            fl.note(L::kfull + st, ph);
            load_tile<DP>(smem_addr(sK + st * L::kTile), &p.mapK, bar(L::kfull + st), start + 128 * jk, hk);
          }
          skip = false;
          if (ok && j == 0 && n[1] > 0) ok = load_q(1);
          ok = ok && wait_bounded(bar(L::vempty + st), ph ^ 1u, w);
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        if (128 * jk + 128 > len && start + len < p.T) {
          ok = load_tail<DP>(sV + st * L::kTile, &p.mapV, bar(L::vfull + st), bar(L::tail), tail_phase,
                             start + 128 * jk, hk, len - 128 * jk, lane, w);
          if (!ok) break;
        } else if (lane == 0) {
          mbar_arrive_expect_tx(bar(L::vfull + st), L::kTile);
          fl.note(L::vfull + st, ph);
          load_tile<DP>(smem_addr(sV + st * L::kTile), &p.mapV, bar(L::vfull + st), start + 128 * jk, hk);
        }
      }
      nq[0] += n[0] > 0;
      nq[1] += n[1] > 0;
    }
    if (lane == 0 && *w.abort_flag) fl.drain(bar0, p.wait_limit_ns);
    __syncwarp();
  } else if (BIAS && warp == kFwdWarps + 3) {
    // the bias of an item's head, into its slot's table
    for (uint32_t it = 0;; ++it) {
      const int slot = it & 1;
      if (!wait_warp(bar(L::info + slot), (it >> 1) & 1, w)) break;
      const int head = items[slot].head;
      if (head < 0) break;
      fill_table_warp(p, head, map, vals, tabs + slot * tabn, lane);
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(L::tabfull + slot));
        mbar_arrive(bar(L::free_ + slot));
      }
    }
  } else if (warp >= kFwdWarps && warp < kFwdWarps + 2) {
    // One MMA warp a query tile: while one waits, the other's products run.
    // Both go through every key tile, and a K or V stage is free when both have
    // passed it.
    const int t = warp - kFwdWarps;
    const int ksteps = (p.d + 15) >> 4;
    const uint32_t idesc_pv = idesc_bf16(0, 1, ksteps * 16);
    const uint32_t dO = tmem + 256 + 128 * t, tS = tmem + 128 * t, aP = kApart ? dO + 64 : tS;
    constexpr int kStride = kApart ? 32 : 64;  // from the first key half's probabilities to the second's
    uint32_t c = 0, np = 0, nq = 0;  // K/V tiles, probability tiles and items of this query tile so far
    bool ok = true, issued = false;
    for (uint32_t it = 0; ok; ++it) {
      const int slot = it & 1;
      if (!(ok = wait_warp(bar(L::info + slot), (it >> 1) & 1, w))) break;
      const bool end = uniform(items[slot].head) < 0;
      const int nt = uniform(items[slot].n[t]), nmax = max(nt, uniform(items[slot].n[t ^ 1]));
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(L::free_ + slot));
      if (end) break;
      auto kfull = [&](int j) {
        return wait_warp(bar(L::kfull + (c + j) % L::kStages), ((c + j) / L::kStages) & 1, w);
      };
      auto vfull = [&](int j) {
        return wait_warp(bar(L::vfull + (c + j) % L::kStages), ((c + j) / L::kStages) & 1, w);
      };
      auto scores = [&](int j) {
        const int st = (c + j) % L::kStages;
        if (elect_one()) {
          mma_scores<DP>(tS, smem_addr(sQ + t * L::kTile), smem_addr(sK + st * L::kTile), ksteps);
          mma_commit(bar(L::sfull + t));
          mma_commit(bar(L::kempty + st));
          if (j + 1 == nt) mma_commit(bar(L::qempty + t));
        }
        __syncwarp();
      };
      if (nt > 0) {
        if (!(ok = wait_warp(bar(L::qfull + t), nq & 1, w) && kfull(0))) break;
        tc_fence_after();
        issued = true;
        scores(0);
      }
      for (int j = 0; j < nt; ++j, ++np) {
        const int st = (c + j) % L::kStages;
        const uint32_t b = smem_addr(sV + st * L::kTile);
        // everything but the probabilities is waited for before they are, so the
        // products are issued as one run
        if (!(ok = vfull(j) && (j + 1 >= nt || kfull(j + 1)))) break;
        // the output of the item before has been read
        if (j == 0 && !(ok = wait_warp(bar(L::ofree + t), (nq & 1) ^ 1, w))) break;
        if (kApart) {
          if (!(ok = wait_warp(bar(L::sread + t), np & 1, w))) break;
          tc_fence_after();
          if (j + 1 < nt) scores(j + 1);
        }
        if (!(ok = wait_warp(bar(L::pfull + 2 * t), np & 1, w))) break;
        tc_fence_after();
        if (elect_one()) mma_rows<2, 0, 2, kStride>(dO, aP, b, idesc_pv, j > 0);
        __syncwarp();
        if (!(ok = wait_warp(bar(L::pfull + 2 * t + 1), np & 1, w))) break;
        tc_fence_after();
        if (elect_one()) {
          mma_rows<2, 2, 2, kStride>(dO, aP, b, idesc_pv, true);
          if (kApart) mma_commit(bar(L::pvdone + t));
          mma_commit(bar(L::vempty + st));
          if (j + 1 >= nt) mma_commit(bar(L::odone + t));
        }
        __syncwarp();
        if (!kApart && j + 1 < nt) scores(j + 1);
      }
      // key tiles that only the other query tile sees
      for (int j = nt; ok && j < nmax; ++j) {
        const int st = (c + j) % L::kStages;
        if ((ok = kfull(j)) && lane == 0) mbar_arrive(bar(L::kempty + st));
        if (ok && (ok = vfull(j)) && lane == 0) mbar_arrive(bar(L::vempty + st));
      }
      c += nmax;
      nq += nt > 0;
    }
    if (*w.abort_flag && issued && elect_one()) drain_mma(bar(L::drain + t), p.wait_limit_ns);
  } else if (warp < kFwdWarps) {
    const int t = warp >> 3, half = (warp >> 2) & 1, quarter = warp & 3;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t tS = lane_base + 128 * t, tO = lane_base + 256 + 128 * t;
    const uint32_t tP = kApart ? tO + 64 + 32 * half : tS + 64 * half;
    // the two warps of these rows meet at a barrier of their own
    const int pair_bar = 1 + 4 * t + quarter;
    float* mine_at = part + half * 256 + t * 128 + quarter * 32 + lane;
    const float* other_at = part + (half ^ 1) * 256 + t * 128 + quarter * 32 + lane;
    const int cut = first_columns(p.d);  // this warp's columns of the output
    const int ofirst = half ? cut : 0, olast = half ? p.d : cut;
    const float sl2 = p.scale_log2;
    uint32_t np = 0, nq = 0;  // score tiles and items of this query tile so far
    // After a failed wait an item runs on without waiting: the pair's barrier
    // needs both warps, nothing is stored at its end, and both leave together.
    bool ok = true;
    for (uint32_t it = 0;; ++it) {
      const int slot = it & 1;
      ok = ok && wait_warp(bar(L::info + slot), (it >> 1) & 1, w);
      if (named_bar_any(pair_bar, 64, !ok)) break;
      const int head = uniform(items[slot].head);
      if (head < 0) break;
      if (BIAS) ok = wait_warp(bar(L::tabfull + slot), (it >> 1) & 1, w);
      const int start = uniform(items[slot].start), len = uniform(items[slot].len);
      const int row0 = uniform(items[slot].row0), nt = uniform(items[slot].n[t]);
      const int row = row0 + 128 * t + quarter * 32 + lane;  // position in the sequence
      const float* tab = tabs + slot * tabn;
      float m = 0.f;             // the exponents' reference (log2)
      float l0 = 0.f, l1 = 0.f;  // sums of 2^(x - m) over this warp's columns
      for (int j = 0; j < nt; ++j, ++np) {
        ok = ok && wait_warp(bar(L::sfull + t), np & 1, w);
        tc_fence_after();
        uint32_t s[64];
        tmem_ld32_issue(tS + 64 * half, s);
        tmem_ld32_issue(tS + 64 * half + 32, s + 32);
        tmem_ld32_wait(s);
        tmem_ld32_wait(s + 32);
        if (kApart) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(L::sread + t));
        }
        const int jk = key_tile(j), c0 = 128 * jk + 64 * half, r0 = row0 + 128 * t;
        float mul = sl2, add = 0.f;  // the exponents: s mul + add log2 e
        if (BIAS) {
          const int side = bias_side(p.bias.md, r0, 128 * jk);
          if (side != 0) {
            add = tab[side < 0 ? 0 : 2 * (p.bias.md + kPad)];
          } else {
            const float* tb = tab + (c0 - row + p.bias.md + kPad);
#pragma unroll
            for (int c = 0; c < 64; ++c) s[c] = __float_as_uint(fmaf(as_f(s[c]), p.scale, tb[c]));
            mul = kLog2e;
          }
        }
        if ((p.causal && 128 * jk + 127 > r0) || 128 * jk + 128 > len) {
          const int seen = (p.causal ? min(len, row + 1) : len) - c0;  // columns this row sees
#pragma unroll
          for (int c = 0; c < 64; ++c) s[c] = c < seen ? s[c] : 0xff800000u;
        }
        float mx[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          mx[q] = fmaxf(as_f(s[q]), as_f(s[q + 4]));
#pragma unroll
          for (int c = 8 + q; c < 64; c += 8) mx[q] = fmaxf(fmaxf(mx[q], as_f(s[c])), as_f(s[c + 4]));
        }
        const float mh = fmaf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), mul, BIAS ? add * kLog2e : 0.f);
        // the product of the tile before has read its probabilities and added to the output
        if (kApart) {
          ok = ok && wait_warp(bar(L::pvdone + t), (np & 1) ^ 1, w);
          tc_fence_after();
        }
        // The exponents' reference is the first tile's maximum and follows the
        // running one only when a row's is 2^16 above it: up to there the
        // exponentials and their sums are as exact (fp32 and bf16 have the range),
        // and neither the maxima are exchanged nor the output rescaled.
        if (named_bar_any(pair_bar, 64, j == 0 || mh > m + 16.f)) {
          mine_at[0] = mh;
          named_bar(pair_bar, 64);
          const float mt = fmaxf(mh, other_at[0]);
          if (j == 0) {
            m = mt;
          } else {
            const float mn = mt > m + 16.f ? mt : m;
            const float f = m == mn ? 1.f : ex2_ftz(m - mn);  // (-infinity stays)
            l0 *= f;
            l1 *= f;
            m = mn;
            for (int c = ofirst; c < olast; c += 8) tmem_scale8(tO + c, f);
          }
        }
        // (a row that has seen no key yet: its bias is -infinity everywhere)
        const float ref = m == -INFINITY ? 0.f : m;
        const float off = BIAS ? fmaf(add, kLog2e, -ref) : -ref;
        const uint64_t scl2 = pack2(mul, mul), off2 = pack2(off, off);
        uint64_t sum[2] = {pack2(l0, l1), 0ull};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t pk[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            float a, b;
            unpack2(fma2(pack2(as_f(s[32 * h + 2 * c]), as_f(s[32 * h + 2 * c + 1])), scl2, off2), a, b);
            a = ex2_ftz(a);
            b = ex2_ftz(b);
            sum[c & 1] = add2(sum[c & 1], pack2(a, b));
            pk[c] = pack_bf16x2(a, b);
          }
          tmem_st16(tP + 16 * h, pk);
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(L::pfull + 2 * t + h));
        }
        unpack2(add2(sum[0], sum[1]), l0, l1);
      }
      if (lane == 0) mbar_arrive(bar(L::free_ + slot));
      if (nt > 0) {
        const float lh = l0 + l1;
        mine_at[512] = lh;
        named_bar(pair_bar, 64);
        const float lo = other_at[512];
        named_bar(pair_bar, 64);  // both have read before the next item writes
        const float l = half ? lo + lh : lh + lo;
        ok = ok && wait_warp(bar(L::odone + t), nq & 1, w);
        tc_fence_after();
        uint32_t o[64];
        const int from = SPLIT ? DP / 2 * half : ofirst;
        tmem_ld32_issue(tO + from, o);
        tmem_ld32_issue(tO + from + (DP == 128 ? 32 : 0), o + 32);
        tmem_ld32_wait(o);
        tmem_ld32_wait(o + 32);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::ofree + t));
        if (SPLIT) {
          // the Q, K and V stages are done with: fp32 rows there, 16 bytes at a time
          // and swizzled by the row
          const int r = quarter * 32 + lane;
          float4* row4 = reinterpret_cast<float4*>(sQ) + r * (DP / 4);
#pragma unroll
          for (int c = 0; c < DP / 2; c += 4)
            row4[((DP / 2 * half + c) / 4) ^ (r & (DP / 4 - 1))] =
                make_float4(as_f(o[c]), as_f(o[c + 1]), as_f(o[c + 2]), as_f(o[c + 3]));
          if (half == 0) {
            part[2 * r] = m;
            part[2 * r + 1] = l;
          }
          continue;
        }
        const int64_t token = static_cast<int64_t>(start) + row;
        const bool mine = ok && row < len;
        store_columns<DP / 2>(o, olast - ofirst, l > 0.f ? 1.f / l : 0.f, mine,
                              static_cast<__nv_bfloat16*>(p.C) + token * p.ld_c + static_cast<int64_t>(head) * p.d + ofirst,
                              p.ld_c, p.wide);
        if (mine && half == 0) p.lse[static_cast<int64_t>(head) * p.T + token] = row_lse(m, l);
        __syncwarp();
        ++nq;
      } else if (SPLIT && t == 0) {
        // no key tile for this CTA: nothing to add
        const int r = quarter * 32 + lane;
        float4* row4 = reinterpret_cast<float4*>(sQ) + r * (DP / 4);
#pragma unroll
        for (int c = 0; c < DP / 2; c += 4) row4[(DP / 2 * half + c) / 4] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (half == 0) {
          part[2 * r] = -INFINITY;
          part[2 * r + 1] = 0.f;
        }
      }
    }
  }
  if (SPLIT) {
    __syncwarp();
    cluster_sync();
    const int head = items[0].head;
    if (head >= 0) {
      const int start = items[0].start, len = items[0].len, row0 = items[0].row0, rows = 128 / p.parts;
      for (int x = threadIdx.x; x < rows * (DP / 4); x += kFwdThreads) {
        const int chunk = x % (DP / 4), r = rank * rows + x / (DP / 4), row = row0 + r;
        if (4 * chunk >= p.d || row >= len) continue;
        const uint32_t at =
            smem_addr(reinterpret_cast<float4*>(sQ) + r * (DP / 4) + (chunk ^ (r & (DP / 4 - 1))));
        const uint32_t ml = smem_addr(part + 4 * (r >> 1));  // (m, l) of rows r & ~1 and r | 1
        float top = -INFINITY;
        for (int c = 0; c < p.parts; ++c) {
          const float4 v = ld_cluster4(ml, c);
          top = fmaxf(top, r & 1 ? v.z : v.x);
        }
        float l = 0.f;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c = 0; c < p.parts; ++c) {
          const float4 v = ld_cluster4(ml, c), b = ld_cluster4(at, c);
          const float mc = r & 1 ? v.z : v.x;
          const float f = mc == top ? 1.f : ex2_ftz(mc - top);
          l = fmaf(r & 1 ? v.w : v.y, f, l);
          a.x = fmaf(b.x, f, a.x);
          a.y = fmaf(b.y, f, a.y);
          a.z = fmaf(b.z, f, a.z);
          a.w = fmaf(b.w, f, a.w);
        }
        const float mul = l > 0.f ? 1.f / l : 0.f;
        const int64_t token = static_cast<int64_t>(start) + row;
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.C) + token * p.ld_c + static_cast<int64_t>(head) * p.d +
                                  4 * chunk) =
            make_uint2(pack_bf16x2(a.x * mul, a.y * mul), pack_bf16x2(a.z * mul, a.w * mul));
        if (chunk == 0) p.lse[static_cast<int64_t>(head) * p.T + token] = row_lse(top, l);
      }
    }
    cluster_sync();
  }
  leave<kFwdWarps>(hd, p);
}

// ===========================================================================
// Backward
// ===========================================================================
// A Q tile is held from the scores to dK, longer than a dC tile: three stages
// of it for the wide heads, where they fit (the bias's table takes their place).
// With two the loads were late by half an iteration.
template <int DP, bool BIAS>
struct DkvShape {
  static constexpr int kTile = DP / 64 * kPanel;
  static constexpr int kQ = DP == 128 ? (BIAS ? 2 : 3) : 4, kO = DP == 128 ? 2 : 4;  // Q and dC tiles held
  static constexpr int kVec = 2 * 2 * 128 * 4;  // of two query tiles what is added to their exponents, and -D
  static constexpr int kSmem = (2 + kQ + kO) * kTile + kBarBytes + kVec;
  static constexpr int kvfull = 0, qfull = 1, ofull = qfull + kQ, tail = ofull + kO, qempty = tail + 1,
                       oempty = qempty + kQ, vecempty = oempty + kO, sfull = vecempty + 2,
                       dpfull = sfull + 2, pready = dpfull + 1, dsready = pready + 4, done = dsready + 2,
                       dfree = done + 1, kvempty = dfree + 1, info = kvempty + 1, free_ = info + 2,
                       drain = free_ + 2, count = drain + 2;
  static_assert(count <= kMaxBars && qempty <= 32, "barriers");
  static uint32_t __device__ __forceinline__ arrivals(int i) {
    if ((i >= pready && i < done) || i == vecempty || i == vecempty + 1 || i == dfree) return kBwdWarps;
    if (i >= free_ && i < drain) return kBwdWarps + 3;
    return i == done || i == kvempty || (i >= oempty && i < vecempty) || i == sfull || i == sfull + 1 ? 2u : 1u;
  }
};

// Stage and phase of a ring of tiles.
struct Ring {
  int stage, stages;
  uint32_t phase;
  __device__ __forceinline__ void next() {
    if (++stage == stages) {
      stage = 0;
      phase ^= 1u;
    }
  }
};

// What the TMA warp tells the other warps of an item (two slots).
struct DkvItem {
  int start, len, tile, head;  // head: the K/V head, -1: no more items
};

// The query tiles of a K/V head's key tile, head by head; every `step`-th.
struct QueryWalk {
  int g, i, i0, nq, step;
  __device__ __forceinline__ void skip(int n) {
    i += n;
    while (i >= nq) {
      i -= nq - i0;
      ++g;
    }
  }
  __device__ __forceinline__ void next() {
    if (step > 1) {
      skip(step);
    } else if (++i == nq) {
      i = i0;
      ++g;
    }
  }
};

// dV = sum over the query tiles of P^T dC, dK = scale sum of dS^T Q, in TMEM for the
// whole item.  One warp issues the two products through P, another the two through
// dS, so that each waits while the other's run.  At width 128 the products bound it:
// 2240 to 2450 cycles a tile against 2048 of products (with P and dS handed over in
// one piece 2780), and 5000 an item beside them: 3500 for 64 KB of dK and dV, which
// an SM stores at 32 bytes a cycle at best.  (To store them under the next item's
// first tile took as long: the 16 warps have no time to spare there.)  At width 64
// the warps' own work bounds it: 1800 cycles a tile against 1024, with 11
// instructions a score issued in 59% of the cycles, and 2900 an item.  P and dS in
// TMEM columns of their own there, so that the products run a tile further ahead,
// was 10% slower: two more waits a tile cost more than they hid.
//
// SPLIT: the CTAs of a cluster share an item, each with every p.parts-th query
// tile.  Their sums meet in shared memory, where each CTA adds up its part of
// the rows, in the order of the ranks.
//
// Begins before the kernel before it has ended (dQ's, or the sums of the bias's
// gradient, which follow it): that one waited for everything earlier, so Q, K, V,
// dC, lse, seq_starts and the table may be read at once (past L1, which may hold
// an earlier call's).  D is dQ's: it is waited for, unless the sums lie between.
// The last thing is to wait for the kernel before, for those behind.
template <int DP, bool BIAS, bool SPLIT>
__global__ void __launch_bounds__(kDkvThreads, 1) rc_dkv_kernel(const __grid_constant__ RcParams p) {
  using L = DkvShape<DP, BIAS>;
  extern __shared__ __align__(1024) uint8_t smem_wide[];
  uint8_t* smem = smem_wide;
  if (smem_addr(smem) & 1023u) {  // nothing of the launch is left for padding
    if (threadIdx.x == 0) atomicOr(p.err, kErrTimeout);
    pdl_wait();
    return;
  }
  uint8_t* sK = smem;
  uint8_t* sV = sK + L::kTile;
  uint8_t* sQ = sV + L::kTile;
  uint8_t* sO = sQ + L::kQ * L::kTile;
  Head* hd = reinterpret_cast<Head*>(sO + L::kO * L::kTile);
  float* vec = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(hd) + kBarBytes);  // [2][2][128]
  float* tabs = vec + 512;  // tables of two query heads, the head's values, and the distances' buckets
  const int tabn = BIAS ? table_floats(p.bias.md) : 0;
  float* vals = tabs + 2 * tabn;
  uint8_t* map = reinterpret_cast<uint8_t*>(vals + kMaxRelBuckets);
  if (BIAS) fill_map(p.bias, map);
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  volatile DkvItem* items = reinterpret_cast<volatile DkvItem*>(hd->items);
  enter<kBwdWarps, false>(hd, L::count, L::arrivals);
  const bool early = p.partial == nullptr;  // D may not be there yet
  const uint32_t bar0 = smem_addr(hd->bar);
  auto bar = [&](int i) { return bar0 + 8u * i; };
  const WaitCtx w{&hd->abort_flag, p.err, p.wait_limit_ns};
  const uint32_t tmem = uniform(hd->tmem);
  // Heads to 64 wide leave room for a second buffer of scores: they are computed
  // a tile ahead.
  constexpr bool kAhead = DP == 64;
  constexpr int kHalves = kAhead ? 1 : 2;  // P and dS are handed over in (where the products wait for them)
  constexpr uint32_t kOther = 384;  // columns from one score buffer to the other
  const uint32_t tS = tmem, tP = tmem + 128, tdV = tmem + 256, tdK = tmem + 256 + DP;
  struct Work {
    int start, len, kt, kvh, i0, nq, total;
    __device__ __forceinline__ QueryWalk walk(const RcParams& p, int rank) const {
      QueryWalk q{kvh * p.group, i0, i0, nq, SPLIT ? p.parts : 1};
      if (SPLIT && total > 0) q.skip(rank);
      return q;
    }
  };
  const int rank = SPLIT ? cluster_rank() : 0;
  auto work_of = [&](int start, int len, int tile, int head) {
    Work k;
    k.start = start;
    k.len = len;
    k.kt = tile;
    k.kvh = head;
    k.nq = (len + 127) >> 7;
    k.i0 = p.causal ? tile : 0;
    k.total = (k.nq - k.i0) * p.group;  // (query head, query tile) pairs
    if (SPLIT) k.total = (k.total - rank + p.parts - 1) / p.parts;  // (may be none)
    return k;
  };
  // the item in `slot`, once it is there
  auto read_item = [&](int slot) {
    return work_of(uniform(items[slot].start), uniform(items[slot].len), uniform(items[slot].tile),
                   uniform(items[slot].head));
  };

  if (warp == kBwdWarps + 2) {
    Flight fl;
    uint32_t tail_phase = 0, it = 0;  // it: (Q, dC) tiles loaded
    bool ok = true, skip = p.fault_skip != 0;
    if (lane == 0) {
      prefetch_tmap(&p.mapQ);
      prefetch_tmap(&p.mapO);
    }
    ItemWalk items_of(p, p.KV, 128, lane);
    for (uint32_t n = 0; ok; ++n) {
      const int slot = n & 1;
      Unit u{0, 0, 0};
      const bool found = items_of.next(p, false, lane, u);
      if (!(ok = wait_warp(bar(L::free_ + slot), ((n >> 1) & 1) ^ 1, w))) break;
      if (lane == 0) {
        items[slot].start = u.start;
        items[slot].len = u.len;
        items[slot].tile = u.tile;
        items[slot].head = found ? items_of.index : -1;
        mbar_arrive(bar(L::info + slot));
      }
      if (!found) break;
      const Work k = work_of(u.start, u.len, u.tile, items_of.index);
      const HeadAt hk = head_at(k.kvh, p.hk);
      QueryWalk q = k.walk(p, rank);
      const int start = k.start, len = k.len;
      for (int i = 0; ok && i < k.total; ++i, ++it, q.next()) {
        const int sq = it % L::kQ, so = it % L::kO;
        const uint32_t pq = (it / L::kQ) & 1, po = (it / L::kO) & 1;
        const HeadAt hq = head_at(q.g, p.hq);
        const bool torn = 128 * q.i + 128 > len && start + len < p.T;  // rows of nobody in the tile
        if (early && it == 1) pdl_wait();  // (the limits of the waits for all but the first tile run from here)
        if (lane == 0) ok = wait_bounded(bar(L::qempty + sq), pq ^ 1u, w);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        if (torn) {
          ok = load_tail<DP>(sQ + sq * L::kTile, &p.mapQ, bar(L::qfull + sq), bar(L::tail), tail_phase,
                             start + 128 * q.i, hq, len - 128 * q.i, lane, w);
          if (!ok) break;
        } else if (lane == 0) {
          mbar_arrive_expect_tx(bar(L::qfull + sq), L::kTile);
          fl.note(L::qfull + sq, pq);
          load_tile<DP>(smem_addr(sQ + sq * L::kTile), &p.mapQ, bar(L::qfull + sq), start + 128 * q.i, hq);
        }
        if (i == 0 && lane == 0) {
          // K and V of the item, once the last products of the one before have read theirs
          ok = wait_bounded(bar(L::kvempty), (n & 1) ^ 1, w);
          if (ok && !skip) {
            mbar_arrive_expect_tx(bar(L::kvfull), 2 * L::kTile);
            fl.note(L::kvfull, n & 1);
            load_tile<DP>(smem_addr(sK), &p.mapK, bar(L::kvfull), start + 128 * k.kt, hk);
            load_tile<DP>(smem_addr(sV), &p.mapV, bar(L::kvfull), start + 128 * k.kt, hk);
          }
          skip = false;
        }
        if (lane == 0) ok = ok && wait_bounded(bar(L::oempty + so), po ^ 1u, w);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        if (torn) {
          ok = load_tail<DP>(sO + so * L::kTile, &p.mapO, bar(L::ofull + so), bar(L::tail), tail_phase,
                             start + 128 * q.i, hq, len - 128 * q.i, lane, w);
        } else if (lane == 0) {
          mbar_arrive_expect_tx(bar(L::ofull + so), L::kTile);
          fl.note(L::ofull + so, po);
          load_tile<DP>(smem_addr(sO + so * L::kTile), &p.mapO, bar(L::ofull + so), start + 128 * q.i, hq);
        }
      }
    }
    if (lane == 0 && *w.abort_flag) fl.drain(bar0, p.wait_limit_ns);
    __syncwarp();
  } else if (warp == kBwdWarps + 3) {
    // What is added to the exponents of the query tiles, and -D, and a query head's
    // bias where it changes: -lse log2 e, in a tile of one distance with its bias,
    // (bias - lse) log2 e; in other tiles with a bias -lse, for they take that difference
    // for each key.  A row past the sequence gets probability 2^(x - inf) = 0.
    bool ok = true;
    uint32_t it = 0;
    if (early) pdl_wait();
    int tslot = 1;  // of the query head's table: the next one is taken where the head changes
    for (uint32_t n = 0; ok; ++n) {
      const int slot = n & 1;
      if (!(ok = wait_warp(bar(L::info + slot), (n >> 1) & 1, w))) break;
      const Work k = read_item(slot);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(L::free_ + slot));
      if (k.kvh < 0) break;
      QueryWalk q = k.walk(p, rank);
      int table_head = -1;
      for (int i = 0; i < k.total; ++i, ++it, q.next()) {
        const int buf = it & 1;
        float nl[4], nd[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int pos = 128 * q.i + 32 * x + lane;
          const int64_t at = static_cast<int64_t>(q.g) * p.T + k.start + pos;
          nl[x] = pos < k.len ? row_shift(__ldcg(p.lse + at)) : -INFINITY;
          nd[x] = pos < k.len ? -__ldcg(p.D + at) : 0.f;
        }
        if (!(ok = wait_warp(bar(L::vecempty + buf), ((it >> 1) & 1) ^ 1u, w))) break;
        if (BIAS && table_head != q.g) {
          // (the tile before the last one has been through: that head's table is free)
          table_head = q.g;
          tslot ^= 1;
          fill_table_warp(p, q.g, map, vals, tabs + tslot * tabn, lane);
          __syncwarp();
        }
        const int side = BIAS ? bias_side(p.bias.md, 128 * q.i, 128 * k.kt) : 0;
        if (!BIAS || side != 0) {
          const float add = BIAS ? tabs[tslot * tabn + (side < 0 ? 0 : 2 * (p.bias.md + kPad))] : 0.f;
#pragma unroll
          for (int x = 0; x < 4; ++x) nl[x] = (BIAS ? nl[x] + add : nl[x]) * kLog2e;
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          vec[256 * buf + 32 * x + lane] = nl[x];
          vec[256 * buf + 128 + 32 * x + lane] = nd[x];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::sfull + buf));  // with the scores
      }
    }
  } else if (warp == kBwdWarps || warp == kBwdWarps + 1) {
    // Warp 0: products through the scores, S^T = K Q^T, then dV += P^T dC.
    // Warp 1: through their gradient, dP^T = V dC^T, then dK += dS^T Q.
    const bool grad = warp == kBwdWarps + 1;
    const int ksteps = (p.d + 15) >> 4;
    const uint32_t idesc_out = idesc_bf16(0, 1, ksteps * 16);
    const uint32_t tX = grad ? tP : tS, tD = grad ? tdK : tdV;       // products, sums
    const uint32_t a = smem_addr(grad ? sV : sK);                    // A of the products
    Ring x{0, grad ? L::kO : L::kQ, 0u}, d{0, grad ? L::kQ : L::kO, 0u};  // of the next products, of the next sum
    const uint32_t xtiles = smem_addr(grad ? sO : sQ), dtiles = smem_addr(grad ? sQ : sO);
    const int xfull = grad ? L::ofull : L::qfull, dfull = grad ? L::qfull : L::ofull;
    const int out = grad ? L::dpfull : L::sfull;
    const bool ahead = kAhead && !grad;
    uint32_t it = 0;  // sums so far
    bool ok = true, issued = false;
    for (uint32_t n = 0; ok; ++n) {
      const int slot = n & 1;
      if (!(ok = wait_warp(bar(L::info + slot), (n >> 1) & 1, w))) break;
      const Work k = read_item(slot);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(L::free_ + slot));
      if (k.kvh < 0) break;
      if (SPLIT && k.total <= 0) continue;
      if (!(ok = wait_warp(bar(L::kvfull), n & 1, w))) break;
      for (int i = -1; i < k.total; ++i) {
        const bool more = i + 1 < k.total;
        const uint32_t tXi = tX + (ahead && (it & 1) ? kOther : 0);             // of this sum (after the first)
        const uint32_t tXn = tX + (ahead && ((it + (i >= 0)) & 1) ? kOther : 0);  // of the next products
        auto products = [&]() {  // by the elected lane
          mma_scores<DP>(tXn, a, xtiles + x.stage * L::kTile, ksteps);
          mma_commit(bar(grad ? out : out + ((it + (i >= 0)) & 1)));
          if (grad) mma_commit(bar(L::oempty + x.stage));
          if (i + 2 == k.total) mma_commit(bar(L::kvempty));
        };
        // the second tile is loaded when dQ has ended: its wait begins then
        if (early && i == 0 && it == 0) pdl_wait();
        if (more && !(ok = wait_warp(bar(xfull + x.stage), x.phase, w))) break;
        issued = true;
        if (ahead && more) {
          tc_fence_after();
          if (elect_one()) products();
          __syncwarp();
        }
        if (i >= 0) {
          if (!(ok = wait_warp(bar(dfull + d.stage), d.phase, w))) break;
          // the sums of the item before have been read
          if (i == 0 && !(ok = wait_warp(bar(L::dfree), (n & 1) ^ 1, w))) break;
          // P or dS comes in two halves of the contraction (16 of every 32 queries)
          // (P's barriers alternate: with scores a tile ahead, two tiles may be ready)
          const int ready = grad ? L::dsready : L::pready + 2 * (it & 1);
          const uint32_t rphase = grad ? it & 1 : (it >> 1) & 1;
          if (!(ok = wait_warp(bar(ready), rphase, w))) break;
          tc_fence_after();
          if (kHalves == 2) {
            if (elect_one()) mma_rows<4, 0, 1>(tD, tXi, dtiles + d.stage * L::kTile, idesc_out, i > 0);
            __syncwarp();
            if (!(ok = wait_warp(bar(ready + 1), rphase, w))) break;
          }
        }
        tc_fence_after();
        if (elect_one()) {
          if (i >= 0) {
            if (kHalves == 2) mma_rows<4, 1, 1>(tD, tXi, dtiles + d.stage * L::kTile, idesc_out, true);
            else mma_rows<4>(tD, tXi, dtiles + d.stage * L::kTile, idesc_out, i > 0);
            mma_commit(bar((grad ? L::qempty : L::oempty) + d.stage));
          }
          if (!ahead && more) products();
          if (!more) mma_commit(bar(L::done));
        }
        __syncwarp();
        if (i >= 0) {
          d.next();
          ++it;
        }
        if (more) x.next();
      }
    }
    if (*w.abort_flag && issued && elect_one()) drain_mma(bar(L::drain + grad), p.wait_limit_ns);
  } else if (warp < kBwdWarps) {
    const int part = warp >> 2;              // the 32 query columns of this warp
    const int key = (warp & 3) * 32 + lane;  // row of the transposed tile
    const uint32_t lb = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tPw = tP + lb + 32 * part;
    const uint64_t scl2 = pack2(p.scale_log2, p.scale_log2), log2e2 = pack2(kLog2e, kLog2e);
    // After a failed wait an item runs on without waiting and stores nothing.
    bool ok = true;
    if (early) pdl_wait();
    int tslot = 1;
    uint32_t it = 0;  // tiles so far
    for (uint32_t n = 0;; ++n) {
      const int slot = n & 1;
      ok = ok && wait_warp(bar(L::info + slot), (n >> 1) & 1, w);
      if (!ok) break;
      const Work k = read_item(slot);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(L::free_ + slot));
      if (k.kvh < 0) break;
      QueryWalk q = k.walk(p, rank);
      const int kt = k.kt;
      int table_head = -1;
      for (int i = 0; i < k.total; ++i, ++it, q.next()) {
        const int buf = it & 1;
        const uint32_t tSw = tS + lb + 32 * part + (kAhead && buf ? kOther : 0);
        if (BIAS && table_head != q.g) {
          table_head = q.g;
          tslot ^= 1;
        }
        const float4* nl4 = reinterpret_cast<const float4*>(vec + 256 * buf + 32 * part);
        const float4* nd4 = reinterpret_cast<const float4*>(vec + 256 * buf + 128 + 32 * part);
        ok = ok && wait_warp(bar(L::sfull + buf), (it >> 1) & 1, w);
        tc_fence_after();
        uint32_t s[32];
        tmem_ld32_issue(tSw, s);
        bool near = false;
        const float* tb = nullptr;
        if (BIAS) {
          near = bias_side(p.bias.md, 128 * q.i, 128 * kt) == 0;
          // distance of column c: key - query = (128 kt + key) - (128 i + 32 part + c)
          tb = tabs + tslot * tabn + (128 * (kt - q.i) + key - 32 * part + p.bias.md + kPad);
        }
        tmem_ld32_wait(s);
        const bool diagonal = p.causal && q.i == kt;
        const int first = key - 32 * part;  // the first query column that sees this key, on the diagonal
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t pk[8];
          if (BIAS && near) {
#pragma unroll
            for (int c = 16 * h; c < 16 * h + 16; c += 4) {
              const float4 n = nl4[c >> 2];
              float x[4];
              unpack2(fma2(pack2(as_f(s[c]), as_f(s[c + 1])), scl2,
                           mul2(add2(pack2(n.x, n.y), pack2(tb[-c], tb[-c - 1])), log2e2)),
                      x[0], x[1]);
              unpack2(fma2(pack2(as_f(s[c + 2]), as_f(s[c + 3])), scl2,
                           mul2(add2(pack2(n.z, n.w), pack2(tb[-c - 2], tb[-c - 3])), log2e2)),
                      x[2], x[3]);
#pragma unroll
              for (int e = 0; e < 4; ++e) s[c + e] = __float_as_uint(ex2_ftz(x[e]));
            }
          } else {
#pragma unroll
            for (int c = 16 * h; c < 16 * h + 16; c += 4) {
              const float4 n = nl4[c >> 2];
              float x[4];
              unpack2(fma2(pack2(as_f(s[c]), as_f(s[c + 1])), scl2, pack2(n.x, n.y)), x[0], x[1]);
              unpack2(fma2(pack2(as_f(s[c + 2]), as_f(s[c + 3])), scl2, pack2(n.z, n.w)), x[2], x[3]);
#pragma unroll
              for (int e = 0; e < 4; ++e) s[c + e] = __float_as_uint(ex2_ftz(x[e]));
            }
          }
          if (diagonal) {
#pragma unroll
            for (int c = 16 * h; c < 16 * h + 16; ++c) s[c] = c >= first ? s[c] : 0u;
          }
#pragma unroll
          for (int c = 0; c < 8; ++c) pk[c] = pack_bf16x2(as_f(s[16 * h + 2 * c]), as_f(s[16 * h + 2 * c + 1]));
          tmem_st8(tSw + 8 * h, pk);
          if (h + 1 == 2 || kHalves == 2) {
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(L::pready + 2 * buf + (kHalves == 2 ? h : 0)));
          }
        }
        ok = ok && wait_warp(bar(L::dpfull), it & 1, w);
        tc_fence_after();
        uint32_t g[32];
        tmem_ld32_issue(tPw, g);
        tmem_ld32_wait(g);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t pk[8];
#pragma unroll
          for (int c = 16 * h; c < 16 * h + 16; c += 4) {
            const float4 n = nd4[c >> 2];
            float a, b;
            unpack2(mul2(pack2(as_f(s[c]), as_f(s[c + 1])), add2(pack2(as_f(g[c]), as_f(g[c + 1])), pack2(n.x, n.y))),
                    a, b);
            pk[(c >> 1) & 7] = pack_bf16x2(a, b);
            unpack2(mul2(pack2(as_f(s[c + 2]), as_f(s[c + 3])),
                         add2(pack2(as_f(g[c + 2]), as_f(g[c + 3])), pack2(n.z, n.w))),
                    a, b);
            pk[((c >> 1) & 7) + 1] = pack_bf16x2(a, b);
          }
          tmem_st8(tPw + 8 * h, pk);
          if (h + 1 == 2 || kHalves == 2) {
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(L::dsready + (kHalves == 2 ? h : 0)));
          }
        }
        if (lane == 0) mbar_arrive(bar(L::vecempty + buf));
      }
      // dV by the first half of the warps, dK by the second; two warps share a row
      const int which = part >> 1, cut = SPLIT ? DP / 2 : first_columns(p.d);
      const int first = part & 1 ? cut : 0, cols = part & 1 ? p.d - cut : cut;
      const HeadAt hk = head_at(k.kvh, p.hk);
      const int pos = 128 * kt + key;
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.dQKV) + (static_cast<int64_t>(k.start) + pos) * p.ld_dqkv +
                           static_cast<int64_t>(hk.shard) * p.shard_w + static_cast<int64_t>(p.hq) * p.d +
                           static_cast<int64_t>(hk.local + (which ? 0 : p.hk)) * p.d + first;
      uint32_t r[DP / 2];
      if (SPLIT && k.total <= 0) {
#pragma unroll
        for (int c = 0; c < DP / 2; ++c) r[c] = 0u;
      } else {
        ok = ok && wait_warp(bar(L::done), n & 1, w);
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < DP / 64; ++c) tmem_ld32_issue((which ? tdK : tdV) + lb + first + 32 * c, r + 32 * c);
#pragma unroll
        for (int c = 0; c < DP / 64; ++c) tmem_ld32_wait(r + 32 * c);
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(L::dfree));
      if (SPLIT) {
        // the Q and dC stages are done with: fp32 rows there, 16 bytes at a time and
        // swizzled by the row
        float4* row4 = reinterpret_cast<float4*>(sQ) + (128 * which + key) * (DP / 4);
#pragma unroll
        for (int c = 0; c < DP / 2; c += 4)
          row4[((first + c) / 4) ^ (key & (DP / 4 - 1))] =
              make_float4(as_f(r[c]), as_f(r[c + 1]), as_f(r[c + 2]), as_f(r[c + 3]));
        continue;
      }
      store_columns<DP / 2>(r, cols, which ? p.scale : 1.f, ok && pos < k.len, out, p.ld_dqkv, p.wide);
      __syncwarp();
    }
  }
  if (SPLIT) {
    __syncwarp();
    cluster_sync();
    const int kvh = items[0].head;
    if (kvh >= 0) {
      const int start = items[0].start, len = items[0].len, kt = items[0].tile, rows = 128 / p.parts;
      const HeadAt hk = head_at(kvh, p.hk);
      for (int x = threadIdx.x; x < 2 * rows * (DP / 4); x += kDkvThreads) {
        const int chunk = x % (DP / 4), row = rank * rows + x / (DP / 4) % rows, which = x / (DP / 4) / rows;
        const int pos = 128 * kt + row;
        if (4 * chunk >= p.d || pos >= len) continue;
        const uint32_t at =
            smem_addr(reinterpret_cast<float4*>(sQ) + (128 * which + row) * (DP / 4) + (chunk ^ (row & (DP / 4 - 1))));
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c = 0; c < p.parts; ++c) {
          const float4 b = ld_cluster4(at, c);
          a.x += b.x;
          a.y += b.y;
          a.z += b.z;
          a.w += b.w;
        }
        const float mul = which ? p.scale : 1.f;
        const int64_t col = static_cast<int64_t>(hk.shard) * p.shard_w + static_cast<int64_t>(p.hq) * p.d +
                            static_cast<int64_t>(hk.local + (which ? 0 : p.hk)) * p.d + 4 * chunk;
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.dQKV) + (static_cast<int64_t>(start) + pos) * p.ld_dqkv + col;
        *reinterpret_cast<uint2*>(out) =
            make_uint2(pack_bf16x2(a.x * mul, a.y * mul), pack_bf16x2(a.z * mul, a.w * mul));
      }
    }
    cluster_sync();
  }
  pdl_wait();
  leave<kBwdWarps>(hd, p);
}

// TMEM: scores [0, 128), dP and then dS [128, 256), dQ [256, 384), Q [384, 448)
// and dC [448, 512); heads to 64 wide: a second dP [256, 384), dQ [384, 448),
// Q [448, 480), dC [480, 512), and dP is computed a tile ahead.  Q and dC stay
// there for the whole row of key tiles: the products read K and V from shared
// memory alone (both operands there would take all of its bandwidth), and three
// tiles of each fit.
template <int DP, bool WITH_BIAS>
struct DqShape {
  static constexpr int kTile = DP / 64 * kPanel;
  // K and V tiles held (a V tile is read once and soon; the bias's tables take one's place)
  static constexpr int kK = DP == 128 ? 3 : 4, kV = DP == 128 && WITH_BIAS ? 2 : kK;
  static constexpr int kDot = 4 * 128 * 4;  // partial sums of D
  static constexpr int kSmem = (kK + kV) * kTile + kBarBytes + kDot + 1024;
  static constexpr int qfull = 0, kfull = 1, vfull = kfull + kK, tail = vfull + kV, kempty = tail + 1,
                       vempty = kempty + kK, sfull = vempty + kV, sread = sfull + 1, dpfull = sread + 1,
                       dsready = dpfull + 1, done = dsready + 4, info = done + 1, tabfull = info + 2,
                       free_ = tabfull + 2, drain = free_ + 2, count = drain + 1;
  static_assert(count <= kMaxBars && kempty <= 32, "barriers");
  template <bool BIAS>
  static uint32_t __device__ __forceinline__ arrivals(int i) {
    if (i >= free_ && i < drain) return kBwdWarps + 1 + (BIAS ? 1 : 0);
    return (i >= dsready && i < done) || i == sread || i == qfull ? kBwdWarps : 1u;
  }
};
// What the TMA warp tells the other warps of an item (two slots).
struct DqItem {
  int start, len, r0, head, nk;  // r0: position of the first query row; head -1: no more items
  int col;                       // the head's first column of Q
  int64_t item;
};

// The bias gradient's shared memory: per compute warp the sums of its 32 x 32
// block by distance (63 of them), for two tiles; of two items the CTA's sums by
// distance and the warps' sums beyond the ends; and the buckets' ranges of distances.
constexpr int kDiag = 64;
__host__ __device__ constexpr int grad_floats(int md) {
  return 2 * kBwdWarps * kDiag + 2 * (2 * md + 1) + 4 * kBwdWarps + 2 * kMaxRelBuckets;
}

// dQ = scale sum over the key tiles of dS K, and D = dC . C of its rows.  At width
// 128: 1800 cycles a tile against 1536 of its three products, which wait for dS (Q
// and dC read from shared memory each time: 3440), and 6000 an item beside its
// tiles: Q and dC to TMEM, D, the last item's output, the first scores.  At width 64
// with the bias's gradient 2000 to 2300 cycles against 768, the 16 warps' work with
// 14 instructions a score, and 5000 an item, of which 1000 for its sums by bucket.
//
// The bias's gradient: a tile within the largest distance sums its dS along the
// diagonals by shuffles (1500 cycles, of which the shuffles are most; one running
// sum handed from lane to lane took 2700), other tiles add to a sum a row.  Both go
// to the item's sums by bucket in memory, and those to the table in fixed order.
//
// SPLIT: as for dK and dV, with every p.parts-th key tile (not with a bias, whose
// gradient's sums are an item's).
template <int DP, bool BIAS, bool SPLIT>
__global__ void __launch_bounds__(kDqThreads, 1) rc_dq_kernel(const __grid_constant__ RcParams p) {
  using L = DqShape<DP, BIAS>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint8_t* sK = smem;
  uint8_t* sV = sK + L::kK * L::kTile;
  Head* hd = reinterpret_cast<Head*>(sV + L::kV * L::kTile);
  volatile DqItem* items = reinterpret_cast<volatile DqItem*>(hd->items);
  const int md = BIAS ? p.bias.md : 0, tabn = BIAS ? table_floats(md) : 0;
  float* dots = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(hd) + kBarBytes);  // [4][128]
  float* tabs = dots + 512;                                         // a table for each slot
  float* vals = tabs + 2 * tabn;                                    // the head's values
  uint8_t* map = reinterpret_cast<uint8_t*>(vals + (BIAS ? kMaxRelBuckets : 0));  // the distances' buckets
  float* diag = reinterpret_cast<float*>(map + tabn);               // [2][kBwdWarps][kDiag]
  const int binn = 2 * md + 1;
  float* all_bins = diag + 2 * kBwdWarps * kDiag;                   // [2][2 md + 1]
  float* all_ends = all_bins + 2 * binn;                            // [2][2][kBwdWarps]
  int* from = reinterpret_cast<int*>(all_ends + 4 * kBwdWarps);     // the buckets' bins: from here
  int* to = from + kMaxRelBuckets;                                  // to before here (and which ends: bits 16, 17)
  const bool grad = BIAS && p.partial != nullptr;
  if (BIAS) fill_map(p.bias, map);
  if (grad) {
    for (int i = threadIdx.x; i < 2 * binn; i += kDqThreads) all_bins[i] = 0.f;
    // Bucket u holds the distances x with first[k] <= x < first[k + 1] on its side,
    // the last one also those of md and more; without buckets of their own, keys
    // behind the query count as distance 0.
    for (int u = threadIdx.x; u < p.bias.nb; u += kDqThreads) {
      const bool pos = p.bias.both && u >= p.bias.side;
      const int k = pos ? u - p.bias.side : u;
      const bool last = k + 1 == p.bias.side, all = !p.bias.both && k == 0;
      const int x0 = min(max(p.bias.first[k], pos ? 1 : 0), md), x1 = last ? md : min(p.bias.first[k + 1], md);
      from[u] = pos ? md + x0 : md - x1 + 1;
      to[u] = (all ? 2 * md : pos ? md + x1 : md - x0 + 1) | (last && !pos ? 1 << 16 : 0) |
              ((last && pos) || all ? 1 << 17 : 0);
    }
  }
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  enter<kBwdWarps>(hd, L::count, L::template arrivals<BIAS>);
  const uint32_t bar0 = smem_addr(hd->bar);
  auto bar = [&](int i) { return bar0 + 8u * i; };
  const WaitCtx w{&hd->abort_flag, p.err, p.wait_limit_ns};
  const uint32_t tmem = uniform(hd->tmem);
  constexpr bool kAhead = DP == 64;  // dP in two buffers
  constexpr int kHalves = kAhead ? 1 : 2;  // dS is handed over in (where the products wait for it)
  const uint32_t tP = tmem + 128, tdQ = tmem + (kAhead ? 384 : 256), tQ = tmem + (kAhead ? 448 : 384),
                 tO = tmem + (kAhead ? 480 : 448);

  const int rank = SPLIT ? cluster_rank() : 0;
  auto key_tile = [&](int j) { return SPLIT ? rank + j * p.parts : j; };  // the CTA's j-th

  if (warp == kBwdWarps + 1) {
    Flight fl;
    uint32_t tail_phase = 0;
    bool ok = true, skip = p.fault_skip != 0;
    if (lane == 0) {
      prefetch_tmap(&p.mapQ);
      prefetch_tmap(&p.mapO);
      prefetch_tmap(&p.mapK);
      prefetch_tmap(&p.mapV);
    }
    ItemWalk items_of(p, p.H, 128, lane);
    Ring kr{0, L::kK, 0u}, vr{0, L::kV, 0u};
    for (uint32_t n = 0; ok; ++n) {
      const int slot = n & 1;
      Unit u{0, 0, 0};
      const bool found = items_of.next(p, p.causal != 0, lane, u, grad ? p.partial : nullptr, p.bias.nb);
      if (!(ok = wait_warp(bar(L::free_ + slot), ((n >> 1) & 1) ^ 1, w))) break;
      const int nk_all = (u.len + 127) >> 7;
      int nk = p.causal ? min(nk_all, u.tile + 1) : nk_all;
      if (SPLIT) nk = max(0, nk - rank + p.parts - 1) / p.parts;  // (may be none)
      const HeadAt hq = head_at(items_of.index, p.hq), hk = head_at(items_of.index / p.group, p.hk);
      if (lane == 0) {
        items[slot].start = u.start;
        items[slot].len = u.len;
        items[slot].r0 = 128 * u.tile;
        items[slot].head = found ? items_of.index : -1;
        items[slot].col = hq.shard * p.shard_w + hq.local * p.d;
        items[slot].nk = nk;
        items[slot].item = items_of.item;
        mbar_arrive(bar(L::info + slot));
      }
      if (!found) break;
      if (SPLIT && nk == 0) continue;
      // Q and dC pass through a K and a V stage on their way to TMEM
      if (lane == 0) {
        ok = wait_bounded(bar(L::kempty + kr.stage), kr.phase ^ 1u, w);
        if (ok) {
          mbar_arrive_expect_tx(bar(L::kfull + kr.stage), L::kTile);
          fl.note(L::kfull + kr.stage, kr.phase);
          load_tile<DP>(smem_addr(sK + kr.stage * L::kTile), &p.mapQ, bar(L::kfull + kr.stage), u.start + 128 * u.tile,
                        hq);
          ok = wait_bounded(bar(L::vempty + vr.stage), vr.phase ^ 1u, w);
        }
        if (ok) {
          mbar_arrive_expect_tx(bar(L::vfull + vr.stage), L::kTile);
          fl.note(L::vfull + vr.stage, vr.phase);
          load_tile<DP>(smem_addr(sV + vr.stage * L::kTile), &p.mapO, bar(L::vfull + vr.stage), u.start + 128 * u.tile,
                        hq);
        }
      }
      kr.next();
      vr.next();
      // C follows Q
      if (lane == 0) {
        ok = ok && wait_bounded(bar(L::kempty + kr.stage), kr.phase ^ 1u, w);
        if (ok) {
          mbar_arrive_expect_tx(bar(L::kfull + kr.stage), L::kTile);
          fl.note(L::kfull + kr.stage, kr.phase);
          load_tile<DP>(smem_addr(sK + kr.stage * L::kTile), &p.mapC, bar(L::kfull + kr.stage), u.start + 128 * u.tile,
                        hq);
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      kr.next();
      for (int j = 0; ok && j < nk; ++j, kr.next(), vr.next()) {
        const int st = kr.stage, sv = vr.stage, jk = key_tile(j);
        const uint32_t ph = kr.phase;
        if (lane == 0) ok = wait_bounded(bar(L::kempty + st), ph ^ 1u, w);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        if (128 * jk + 128 > u.len && u.start + u.len < p.T) {
          ok = load_tail<DP>(sK + st * L::kTile, &p.mapK, bar(L::kfull + st), bar(L::tail), tail_phase,
                             u.start + 128 * jk, hk, u.len - 128 * jk, lane, w);
          if (!ok) break;
        } else if (lane == 0 && !skip) {
          mbar_arrive_expect_tx(bar(L::kfull + st), L::kTile);
          fl.note(L::kfull + st, ph);
          load_tile<DP>(smem_addr(sK + st * L::kTile), &p.mapK, bar(L::kfull + st), u.start + 128 * jk, hk);
        }
        skip = false;
        if (lane == 0) {
          ok = wait_bounded(bar(L::vempty + sv), vr.phase ^ 1u, w);
          if (ok) {
            mbar_arrive_expect_tx(bar(L::vfull + sv), L::kTile);
            fl.note(L::vfull + sv, vr.phase);
            load_tile<DP>(smem_addr(sV + sv * L::kTile), &p.mapV, bar(L::vfull + sv), u.start + 128 * jk, hk);
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
      }
    }
    if (lane == 0 && *w.abort_flag) fl.drain(bar0, p.wait_limit_ns);
    __syncwarp();
  } else if (BIAS && warp == kBwdWarps + 2) {
    // the bias of an item's head, into its slot's table
    for (uint32_t n = 0;; ++n) {
      const int slot = n & 1;
      if (!wait_warp(bar(L::info + slot), (n >> 1) & 1, w)) break;
      const int head = items[slot].head;
      if (head < 0) break;
      fill_table_warp(p, head, map, vals, tabs + slot * tabn, lane);
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(L::tabfull + slot));
        mbar_arrive(bar(L::free_ + slot));
      }
    }
  } else if (warp == kBwdWarps) {
    // After dS of a tile: dQ += dS K, dP = dC V^T of the next tile in dS's place,
    // and last the scores S = Q K^T of the one after, which nobody waits for yet:
    // they run while the compute warps make the next dS.
    const int ksteps = (p.d + 15) >> 4;
    const uint32_t idesc_out = idesc_bf16(0, 1, ksteps * 16);
    Ring kr{0, L::kK, 0u}, vr{0, L::kV, 0u}, dr{0, L::kK, 0u};  // of scores, of dP, of dQ
    uint32_t nd = 0, ns = 0;  // dS tiles and score tiles so far
    bool ok = true, issued = false;
    auto scores = [&]() {
      tc_fence_after();
      if (elect_one()) {
        mma_scores_ts<DP>(tmem, tQ, smem_addr(sK + kr.stage * L::kTile), ksteps);
        mma_commit(bar(L::sfull));
      }
      __syncwarp();
      kr.next();
      ++ns;
    };
    uint32_t np0 = 0;  // tiles of the items before
    auto dprobs = [&](int j) {  // by the elected lane
      mma_scores_ts<DP>(tP + (kAhead && ((np0 + j) & 1) ? 128 : 0), tO, smem_addr(sV + vr.stage * L::kTile), ksteps);
      // (a tile ahead, dP is issued before the scores of its tile, whose commit covers it)
      if (!kAhead) mma_commit(bar(L::dpfull));
      mma_commit(bar(L::vempty + vr.stage));
    };
    for (uint32_t n = 0; ok; ++n) {
      const int slot = n & 1;
      if (!(ok = wait_warp(bar(L::info + slot), (n >> 1) & 1, w))) break;
      const int nk = uniform(items[slot].nk);
      const bool end = uniform(items[slot].head) < 0;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(L::free_ + slot));
      if (end) break;
      if (SPLIT && nk == 0) continue;
      // Q and dC are in TMEM: Q's stage is free again
      if (!(ok = wait_warp(bar(L::qfull), n & 1, w))) break;
      if (lane == 0) mbar_arrive(bar(L::kempty + kr.stage));
      __syncwarp();
      kr.next();
      kr.next();  // C's; the compute warps release it and dC's
      vr.next();
      dr.next();
      dr.next();
      if (!(ok = wait_warp(bar(L::kfull + kr.stage), kr.phase, w))) break;
      issued = true;
      if (kAhead) {
        if (!(ok = wait_warp(bar(L::vfull + vr.stage), vr.phase, w))) break;
        tc_fence_after();
        if (elect_one()) dprobs(0);
        __syncwarp();
        vr.next();
      }
      scores();
      for (int j = -1; j < nk; ++j) {
        // the next dP: of tile j + 1 in place of tile j's dS, or (two buffers) of
        // tile j + 2
        const int jn = j + (kAhead ? 2 : 1);
        const bool more = jn < nk;
        const uint32_t tPj = tP + (kAhead && (nd & 1) ? 128 : 0);
        if (more && !(ok = wait_warp(bar(L::vfull + vr.stage), vr.phase, w))) break;
        if (j >= 0) {
          // dS comes in two halves of the contraction (16 of every 32 keys); its
          // barriers alternate: with dP a tile ahead, two tiles may be ready
          const int ready = L::dsready + 2 * (nd & 1);
          if (!(ok = wait_warp(bar(ready), (nd >> 1) & 1, w))) break;
          tc_fence_after();
          if (kHalves == 2) {
            if (elect_one()) mma_rows<4, 0, 1>(tdQ, tPj, smem_addr(sK + dr.stage * L::kTile), idesc_out, j > 0);
            __syncwarp();
            if (!(ok = wait_warp(bar(ready + 1), (nd >> 1) & 1, w))) break;
          }
        }
        tc_fence_after();
        if (elect_one()) {
          if (j >= 0) {
            if (kHalves == 2) mma_rows<4, 1, 1>(tdQ, tPj, smem_addr(sK + dr.stage * L::kTile), idesc_out, true);
            else mma_rows<4>(tdQ, tPj, smem_addr(sK + dr.stage * L::kTile), idesc_out, j > 0);
            mma_commit(bar(L::kempty + dr.stage));
          }
          if (more) dprobs(jn);
          if (j + 1 >= nk) mma_commit(bar(L::done));
        }
        __syncwarp();
        if (j >= 0) {
          dr.next();
          ++nd;
        }
        if (more) vr.next();
        if (j + 2 < nk) {
          if (!(ok = wait_warp(bar(L::kfull + kr.stage), kr.phase, w) && wait_warp(bar(L::sread), (ns - 1) & 1, w)))
            break;
          scores();
        }
      }
      np0 += nk;
    }
    if (*w.abort_flag && issued && elect_one()) drain_mma(bar(L::drain), p.wait_limit_ns);
  } else if (warp < kBwdWarps) {
    const int part = warp >> 2;  // the 32 key columns of this warp
    const int quarter = warp & 3;
    const uint32_t lb = static_cast<uint32_t>(quarter * 32) << 16;
    const uint64_t scl2 = pack2(p.scale_log2, p.scale_log2), log2e2 = pack2(kLog2e, kLog2e);
    uint32_t nt = 0;  // tiles so far
    uint32_t kc = 0, vc = 0;  // ring tiles so far
    // the columns of the output in 32s over the warps of a row; an item's are
    // stored when the next one's Q and dC are in place
    const int ofirst = 32 * part, ocols = min(p.d - ofirst, 32);
    uint32_t dq[16];
    __nv_bfloat16* prev = nullptr;  // where dq goes
    bool stored = false;            // if anywhere
    auto put = [&]() {
      if (prev != nullptr) put_columns<32>(dq, ocols, stored, prev, p.ld_dqkv, p.wide);
      __syncwarp();
    };
    // After a failed wait an item runs on without waiting: the named barriers
    // need every warp, nothing of the gradient is stored, and all leave together.
    bool ok = true;
    for (uint32_t n = 0;; ++n) {
      const int slot = n & 1;
      ok = ok && wait_warp(bar(L::info + slot), (n >> 1) & 1, w);
      if (named_bar_any(2, 32 * kBwdWarps, !ok)) break;
      const int head = uniform(items[slot].head);
      if (head < 0) {
        put();
        break;
      }
      const int start = uniform(items[slot].start), len = uniform(items[slot].len), r0 = uniform(items[slot].r0);
      const int nk = uniform(items[slot].nk);
      float4* row4 = reinterpret_cast<float4*>(sK) + (quarter * 32 + lane) * (DP / 4);  // SPLIT: the row's sums
      if (SPLIT && nk == 0) {
        // no key tile for this CTA: nothing to add
#pragma unroll
        for (int c = 0; c < DP / 16; ++c) row4[DP / 16 * part + c] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (lane == 0) mbar_arrive(bar(L::free_ + slot));
        continue;
      }
      const int row = r0 + quarter * 32 + lane;
      const bool mine = row < len;
      const float* tab = tabs + slot * tabn;
      float lse = 0.f, nd = 0.f;  // (lse is not looked at before the products have been asked for)
      if (mine) lse = __ldcg(p.lse + static_cast<int64_t>(head) * p.T + start + row);
      // this warp's quarter of the columns of Q and dC into TMEM; the item before
      // has been through its products
      {
        const int sk = kc % L::kK, sv = vc % L::kV;
        ok = ok && wait_warp(bar(L::kfull + sk), (kc / L::kK) & 1, w) &&
             wait_warp(bar(L::vfull + sv), (vc / L::kV) & 1, w);
        tile_to_tmem<DP / 4>(tQ + lb + DP / 8 * part, sK + sk * L::kTile, quarter * 32 + lane, DP / 4 * part);
        tile_to_tmem<DP / 4>(tO + lb + DP / 8 * part, sV + sv * L::kTile, quarter * 32 + lane, DP / 4 * part);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(L::qfull));
      // D of the rows: each warp its quarter of the columns, then the four sums
      {
        const int sc = (kc + 1) % L::kK, sv = vc % L::kV, r = quarter * 32 + lane;
        ok = ok && wait_warp(bar(L::kfull + sc), ((kc + 1) / L::kK) & 1, w);
        dots[128 * part + r] = dot_tiles<DP / 4>(sK + sc * L::kTile, sV + sv * L::kTile, r, DP / 4 * part);
        named_bar(1, 32 * kBwdWarps);
        if (threadIdx.x == 0) {
          mbar_arrive(bar(L::kempty + sc));
          mbar_arrive(bar(L::vempty + sv));
        }
        const float D = (dots[r] + dots[128 + r]) + (dots[256 + r] + dots[384 + r]);
        if (part == 0 && mine && rank == 0) p.D[static_cast<int64_t>(head) * p.T + start + row] = D;
        nd = -D;
      }
      const uint64_t nd2 = pack2(nd, nd);
      kc += nk + 2;
      vc += nk + 1;
      // the item before's output, while the first products of this one run
      put();
      const float nl = mine ? row_shift(lse) : 0.f;
      if (BIAS) ok = ok && wait_warp(bar(L::tabfull + slot), (n >> 1) & 1, w);
      float* bins = all_bins + slot * binn;
      float end_lo = 0.f, end_hi = 0.f;  // dS at distances <= -md and >= md, of the tile sums
      uint64_t far_lo = 0, far_hi = 0;   // and of this row in tiles all beyond an end
      for (int j = 0; j < nk; ++j, ++nt) {
        const int jk = key_tile(j), c0 = 128 * jk + 32 * part;  // key position of this warp's first column
        const uint32_t tPj = tP + lb + 32 * part + (kAhead && (nt & 1) ? 128 : 0);
        int side = 0;
        float off = nl;  // (differences with the bias come before the factor)
        const float* tb = nullptr;
        if (BIAS) {
          side = bias_side(md, r0, 128 * jk);
          if (side != 0) off += tab[side < 0 ? 0 : 2 * (md + kPad)];
          tb = tab + (c0 - row + md + kPad);
        }
        if (!BIAS || side != 0) off *= kLog2e;
        const uint64_t off2 = pack2(off, off);
        ok = ok && wait_warp(bar(L::sfull), nt & 1, w);
        tc_fence_after();
        uint32_t s[32];
        tmem_ld32_issue(tmem + lb + 32 * part, s);
        tmem_ld32_wait(s);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::sread));
        if (BIAS && side == 0) {
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            float x0, x1;
            unpack2(fma2(pack2(as_f(s[c]), as_f(s[c + 1])), scl2,
                         mul2(add2(off2, pack2(tb[c], tb[c + 1])), log2e2)),
                    x0, x1);
            s[c] = __float_as_uint(ex2_ftz(x0));
            s[c + 1] = __float_as_uint(ex2_ftz(x1));
          }
        } else {
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            float x0, x1;
            unpack2(fma2(pack2(as_f(s[c]), as_f(s[c + 1])), scl2, off2), x0, x1);
            s[c] = __float_as_uint(ex2_ftz(x0));
            s[c + 1] = __float_as_uint(ex2_ftz(x1));
          }
        }
        const bool masked = (p.causal && 128 * jk + 127 > r0) || 128 * jk + 128 > len;
        if (!kAhead) {
          ok = ok && wait_warp(bar(L::dpfull), nt & 1, w);
          tc_fence_after();
        }
        uint32_t g[32];
        tmem_ld32_issue(tPj, g);
        tmem_ld32_wait(g);
        const int seen = (p.causal ? min(len, row + 1) : len) - c0;
        uint64_t rowsum = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t pk[8];
#pragma unroll
          for (int c = 16 * h; c < 16 * h + 16; c += 2) {
            float a, b;
            unpack2(mul2(pack2(as_f(s[c]), as_f(s[c + 1])), add2(pack2(as_f(g[c]), as_f(g[c + 1])), nd2)), a, b);
            s[c] = __float_as_uint(a);
            s[c + 1] = __float_as_uint(b);
          }
          if (masked) {
#pragma unroll
            for (int c = 16 * h; c < 16 * h + 16; ++c) s[c] = c < seen ? s[c] : 0u;
          }
          if (BIAS && side != 0) {
#pragma unroll
            for (int c = 16 * h; c < 16 * h + 16; c += 2)
              rowsum = add2(rowsum, pack2(as_f(s[c]), as_f(s[c + 1])));
          }
#pragma unroll
          for (int c = 0; c < 8; ++c) pk[c] = pack_bf16x2(as_f(s[16 * h + 2 * c]), as_f(s[16 * h + 2 * c + 1]));
          tmem_st8(tPj + 8 * h, pk);
          if (h + 1 == 2 || kHalves == 2) {
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(L::dsready + 2 * (nt & 1) + (kHalves == 2 ? h : 0)));
          }
        }
        if (BIAS && grad) {
          if (side < 0) {
            far_lo = add2(far_lo, rowsum);
          } else if (side > 0) {
            far_hi = add2(far_hi, rowsum);
          } else {
            // Sums along the diagonals of the warp's 32 x 32 block: at column k lane
            // l takes the value of row (l + k) mod 32, which lies at distance -l,
            // or 32 - l past the last row.  (32 shuffles that do not wait for each
            // other; handing one running sum from lane to lane took 2700 cycles a
            // tile.)
            float* dt_sums = diag + (nt & 1) * kBwdWarps * kDiag;
            float* dw = dt_sums + warp * kDiag;
            if (!mine) {
#pragma unroll
              for (int c = 0; c < 32; ++c) s[c] = 0u;
            }
            float lo[2] = {0.f, 0.f}, hi[2] = {0.f, 0.f};
#pragma unroll
            for (int c = 0; c < 32; ++c) {
              const float v = as_f(__shfl_sync(0xffffffffu, s[c], (lane + c) & 31));
              if (lane + c < 32) lo[c & 1] += v;
              else hi[c & 1] += v;
            }
            dw[31 - lane] = lo[0] + lo[1];  // distance (31 - lane) - 31 + block offset
            if (lane > 0) dw[63 - lane] = hi[0] + hi[1];
            // (the next near tile writes the other buffer, and the one after that
            // comes behind the next one's barrier)
            named_bar(1, 32 * kBwdWarps);
            // thread x sums distance x - 127 of the tile over the warps' blocks, whose
            // offsets are 32 (part - quarter): two offsets hold the distance
            if (threadIdx.x < 255) {
              const int dt = static_cast<int>(threadIdx.x) - 127;
              const int k = (dt + 31) >> 5, at = dt - 32 * k + 31;
              float sum = 0.f;
#pragma unroll
              for (int qu = 0; qu < 4; ++qu) {
                if (qu + k >= 0 && qu + k < 4) sum += dt_sums[(4 * (qu + k) + qu) * kDiag + at];
                if (qu + k >= 1 && qu + k < 5 && at < 31) sum += dt_sums[(4 * (qu + k - 1) + qu) * kDiag + at + 32];
              }
              const int delta = 128 * jk - r0 + dt;
              if (delta <= -md) end_lo += sum;
              else if (delta >= md) end_hi += sum;
              else bins[delta + md] += sum;
            }
          }
        }
      }
      ok = ok && wait_warp(bar(L::done), n & 1, w);
      tc_fence_after();
      {
        uint32_t r[32];
        tmem_ld32_issue(tdQ + lb + 32 * min(part, DP / 32 - 1), r);
        tmem_ld32_wait(r);
        if (SPLIT && part < DP / 32) {
          // the K and V stages are done with: fp32 rows there, 16 bytes at a time and
          // swizzled by the row
#pragma unroll
          for (int c = 0; c < 32; c += 4)
            row4[(8 * part + c / 4) ^ (lane & (DP / 4 - 1))] =
                make_float4(as_f(r[c]), as_f(r[c + 1]), as_f(r[c + 2]), as_f(r[c + 3]));
        }
        if (!SPLIT) pack_columns<32>(r, p.scale, dq);
      }
      tc_fence_before();
      prev = static_cast<__nv_bfloat16*>(p.dQKV) + (static_cast<int64_t>(items[slot].start) + row) * p.ld_dqkv +
             items[slot].col + ofirst;
      if (SPLIT || ocols <= 0) prev = nullptr;  // (the whole warp)
      stored = ok && mine;
      if (BIAS && grad) {
        // the item's sums by bucket, in a fixed order: 16 lanes a bucket.  The next item
        // has bins and ends of its own; those of the one before are cleared here, which
        // every warp has read.
        constexpr int kN = 32 * kBwdWarps;
        float* ends = all_ends + 2 * kBwdWarps * slot;
        float a0, a1, b0, b1;
        unpack2(far_lo, a0, a1);
        unpack2(far_hi, b0, b1);
        float lo = end_lo + (mine ? a0 + a1 : 0.f), hi = end_hi + (mine ? b0 + b1 : 0.f);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          lo += __shfl_xor_sync(0xffffffffu, lo, o);
          hi += __shfl_xor_sync(0xffffffffu, hi, o);
        }
        if (lane == 0) {
          ends[warp] = lo;
          ends[kBwdWarps + warp] = hi;
        }
        named_bar(1, kN);
        const int l = lane & 15;
        static_assert(kBwdWarps == 16, "a lane an end's sum");
        for (int u0 = 2 * warp; u0 < p.bias.nb; u0 += 2 * kBwdWarps) {
          const int u = u0 + (lane >> 4);
          float a = 0.f;
          if (u < p.bias.nb) {
            const int end = to[u];
#pragma unroll 1
            for (int x = from[u] + l; x < (end & 0xffff); x += 16) a += bins[x];
            if (end & (1 << 16)) a += ends[l];
            if (end & (1 << 17)) a += ends[kBwdWarps + l];
          }
#pragma unroll
          for (int o = 8; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
          if (u < p.bias.nb && l == 0) p.partial[items[slot].item * p.bias.nb + u] = a;
        }
        for (int i = threadIdx.x; i < binn; i += kN) all_bins[(slot ^ 1) * binn + i] = 0.f;
      }
      if (lane == 0) mbar_arrive(bar(L::free_ + slot));
    }
  }
  if (SPLIT) {
    __syncwarp();
    cluster_sync();
    const int head = items[0].head;
    if (head >= 0) {
      const int start = items[0].start, len = items[0].len, r0 = items[0].r0, rows = 128 / p.parts;
      const HeadAt hq = head_at(head, p.hq);
      for (int x = threadIdx.x; x < rows * (DP / 4); x += kDqThreads) {
        const int chunk = x % (DP / 4), r = rank * rows + x / (DP / 4), row = r0 + r;
        if (4 * chunk >= p.d || row >= len) continue;
        const uint32_t at = smem_addr(reinterpret_cast<float4*>(sK) + r * (DP / 4) + (chunk ^ (r & 31 & (DP / 4 - 1))));
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c = 0; c < p.parts; ++c) {
          const float4 b = ld_cluster4(at, c);
          a.x += b.x;
          a.y += b.y;
          a.z += b.z;
          a.w += b.w;
        }
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.dQKV) + (static_cast<int64_t>(start) + row) * p.ld_dqkv +
                             static_cast<int64_t>(hq.shard) * p.shard_w + static_cast<int64_t>(hq.local) * p.d + 4 * chunk;
        *reinterpret_cast<uint2*>(out) =
            make_uint2(pack_bf16x2(a.x * p.scale, a.y * p.scale), pack_bf16x2(a.z * p.scale, a.w * p.scale));
      }
    }
    cluster_sync();
  }
  leave<kBwdWarps>(hd, p);
}

// dtable[u, h] (+)= the sum over the units' partial sums, in a fixed order: one
// block a head and bucket.
__global__ void __launch_bounds__(128) rc_bias_sum_kernel(const __grid_constant__ RcParams p, int64_t units) {
  pdl_wait();
  pdl_trigger();
  const int h = blockIdx.x, u = blockIdx.y;
  double a = 0.0;
  for (int64_t i = threadIdx.x; i < units; i += 128) a += p.partial[(i * p.H + h) * p.bias.nb + u];
  __shared__ double red[128];
  red[threadIdx.x] = a;
  __syncthreads();
  for (int o = 64; o > 0; o >>= 1) {
    if (threadIdx.x < o) red[threadIdx.x] += red[threadIdx.x + o];
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    float* out = p.dtable + static_cast<int64_t>(u) * p.H + h;
    *out = static_cast<float>(red[0] + (p.accumulate ? static_cast<double>(*out) : 0.0));
  }
}

// Whether every head's rows of `out` start on 32 bytes and are whole 32s long.
int wide_rows(const RcParams& p, const void* out, int64_t ld, int shard_w) {
  return (reinterpret_cast<uintptr_t>(out) & 31u) == 0 && ld % 16 == 0 && p.d % 16 == 0 && shard_w % 16 == 0;
}

// CTAs that share an item, by an estimate of the launch's time in tiles: the
// longest item or the mean work of an SM (items of equal length: rounds of them),
// and for each round what an item costs beside its tiles: 1.5, in pairs 5.5, in
// fours 7.5, in eights 9.5 (2 more in each of several rounds, as only single CTAs
// stay for the next item).  `once`: in one round only (the forward, whose single
// CTAs take pairs of query tiles).  n: tiles of a sequence of mean length (no matter
// if the sequences come by seq_starts or by s: equal rows are summed in the same
// order); mult: tiles an item for each of them.  So one long sequence among many
// short ones stays with single CTAs: 8192 tokens, 8 heads of 64, 1 K/V head, backward
// 213 us alone and 551 us beside 31 sequences of 64.  Pairs and fours of CTAs leave 8
// SMs over, eights 40.  Microseconds with 1, 2, 4 and 8, whole call, heads of 128:
//   forward   2048, 2 heads, causal             23   18   14*  31
//             4096, 2 heads                     41   28*  36   65
//   dQ        2048, 2 heads, causal             36   31   28*  44
//   dK, dV    512, 8 heads, 1 K/V head          54   38   28   24*
//             2048, 16 heads, 2 K/V, causal    190  112   74*  82
//             4096, 8 heads, 2 K/V             238  162* 173  226
//             16384, 8 heads, 2 K/V, causal   1135 1079*1115 1344
//             2048, 8 heads of 64, 8 K/V        38*  49   63  108   (* chosen)
int cluster_parts(const RcParams& p, int heads, int mult, bool once, int num_sms) {
  const int64_t seqs = p.b, n = (p.T + 128 * seqs - 1) / (128 * seqs), items = n * seqs * heads;
  int parts = 1;
  double best = 0;
  for (int c = 1; c <= 8; c *= 2) {
    const int64_t slots = c == 1 ? num_sms : (num_sms - (c < 8 ? 8 : 40)) / c;
    if (slots < 1) break;
    const int64_t rounds = (items + slots - 1) / slots, longest = n * mult;
    const double mean = 0.5 * (n + 1) * mult * items / (static_cast<double>(c) * slots);
    double t = p.causal ? static_cast<double>(longest) / c : static_cast<double>(rounds * ((longest + c - 1) / c));
    if (p.causal && mean > t) t = mean;
    t += rounds * (c == 1 ? 1.5 : (c == 2 ? 5.5 : c == 4 ? 7.5 : 9.5) + (rounds > 1 ? 2 : 0));
    if (c == 1 || (t < 0.95 * best && (!once || rounds == 1))) {
      best = t;
      parts = c;
    }
  }
  return parts;
}

// The counters of a launch of `blocks` CTAs (-1: none, it needs none or they are used up).
cudaError_t take_slot(RcParams& p, int64_t blocks, cudaStream_t st) {
  static std::atomic<unsigned> eager{0};
  static std::atomic<uint64_t> captured{0};
  p.slot = -1;
  if (p.items * p.parts <= blocks) return cudaSuccess;
  cudaStreamCaptureStatus status;
  const cudaError_t e = cudaStreamIsCapturing(st, &status);
  if (e != cudaSuccess) return e;
  if (status == cudaStreamCaptureStatusNone) {
    p.slot = static_cast<int>(eager.fetch_add(1) % kRcSlots);
  } else {
    const uint64_t n = captured.fetch_add(1);
    if (n < kRcGraphSlots) p.slot = kRcSlots + static_cast<int>(n);
  }
  return cudaSuccess;
}

// In clusters of p.parts CTAs, or single ones, at most one an SM.  The shared memory
// that a kernel may have is raised once a device, to all there is.
template <auto kernel>
cudaError_t launch_rc(int num_sms, int threads, int smem, RcParams& p, cudaStream_t st) {
  const int64_t blocks = p.parts > 1 ? p.items * p.parts : p.items < num_sms ? p.items : num_sms;
  constexpr int kDevices = 16;  // (on later ones it is set each time)
  static std::atomic<int> granted[kDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= kDevices || granted[dev].load(std::memory_order_acquire) == 0) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    if (e != cudaSuccess) return e;
    if (dev < kDevices) granted[dev].store(1, std::memory_order_release);
  }
  if ((e = take_slot(p, blocks, st)) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl_on() ? 1 : 0;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(p.parts);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.parts > 1 ? 2 : 1;
  const cudaError_t l = cudaLaunchKernelEx(&cfg, kernel, p);
  count_launches(1);
  return l != cudaSuccess ? l : cudaGetLastError();
}

// Runs of `rows` tokens: exactly, or for sequences that only the device knows
// an upper bound (each adds at most one run that is not full).
int64_t units_of(const RcParams& p, int rows) {
  if (p.seq_starts == nullptr) return static_cast<int64_t>(p.b) * ((p.s + rows - 1) / rows);
  return p.T / rows + p.b;
}

// Query tiles an item of the forward: two share their K and V tiles, and the
// softmax of one runs under the products of the other, so a pair takes about
// 1 / 0.7 of a single one's time; singles balance better where there are few.
// Estimated by the slowest SM.  One sequence of 2048, 16 heads of 128: 44 us
// with one and 35 us with two without the causal mask, 25 us and 32 us with it.
int query_tiles(const RcParams& p, int num_sms) {
  if (p.seq_starts != nullptr) return units_of(p, 256) * p.H >= num_sms ? 2 : 1;  // lengths are on the device
  const int64_t n = static_cast<int64_t>(p.b) * p.H, one = (p.s + 127) / 128, two = (p.s + 255) / 256;
  const auto per_sm = [&](int64_t x) { return (x + num_sms - 1) / num_sms; };
  int64_t t1, t2;
  if (p.causal) {
    t1 = max(one, per_sm(n * (one * (one + 1) / 2)));
    t2 = max(one, per_sm(n * (two * (two + 1) - (one & 1))));
  } else {
    t1 = per_sm(n * one) * one;
    t2 = per_sm(n * two) * one;
  }
  return 7 * t1 < 10 * t2 ? 1 : 2;
}

template <int DP, bool BIAS>
cudaError_t fwd_t(RcParams& p, int num_sms, cudaStream_t st) {
  const int smem = FwdShape<DP>::kSmem + (BIAS ? 9 * table_floats(p.bias.md) + 4 * kMaxRelBuckets : 0);
  p.wide = wide_rows(p, p.C, p.ld_c, 0);
  p.parts = cluster_parts(p, p.H, 1, true, num_sms);
  p.sub = p.parts > 1 ? 1 : query_tiles(p, num_sms);
  p.items = units_of(p, 128 * p.sub) * p.H;
  if (p.parts > 1) return launch_rc<rc_fwd_kernel<DP, BIAS, true>>(num_sms, kFwdThreads, smem, p, st);
  return launch_rc<rc_fwd_kernel<DP, BIAS, false>>(num_sms, kFwdThreads, smem, p, st);
}
template <int DP, bool BIAS>
cudaError_t bwd_t(RcParams& p, int num_sms, cudaStream_t st) {
  p.parts = 1;
  const int64_t units = units_of(p, 128);
  const int n = BIAS ? table_floats(p.bias.md) : 0;
  p.wide = wide_rows(p, p.dQKV, p.ld_dqkv, p.shard_w);
  // dQ first: it leaves D for dK and dV
  p.items = units * p.H;
  // (two tables of floats, a head's values, a byte a distance, the sums)
  const int dq_smem =
      (DqShape<DP, BIAS>::kSmem) + 9 * n + (BIAS ? 4 * (kMaxRelBuckets + grad_floats(p.bias.md)) : 0);
  if (!BIAS) p.parts = cluster_parts(p, p.H, 1, false, num_sms);
  cudaError_t e = p.parts > 1 ? launch_rc<rc_dq_kernel<DP, BIAS, !BIAS>>(num_sms, kDqThreads, dq_smem, p, st)
                              : launch_rc<rc_dq_kernel<DP, BIAS, false>>(num_sms, kDqThreads, dq_smem, p, st);
  p.fault_skip = p.fault_second;
  if (e != cudaSuccess) return e;
  if (BIAS && p.partial != nullptr) {
    e = launch_k(rc_bias_sum_kernel, dim3(p.H, p.bias.nb), dim3(128), 0, st, p, units);
    count_launches(1);
    if (e != cudaSuccess) return e;
  }
  p.items = units * p.KV;
  // (two tables of floats, a head's values, a byte a distance)
  const int dkv_smem = (DkvShape<DP, BIAS>::kSmem) + 9 * n + (BIAS ? 4 * kMaxRelBuckets : 0);
  p.parts = cluster_parts(p, p.KV, p.group, false, num_sms);
  e = p.parts > 1 ? launch_rc<rc_dkv_kernel<DP, BIAS, true>>(num_sms, kDkvThreads, dkv_smem, p, st)
                  : launch_rc<rc_dkv_kernel<DP, BIAS, false>>(num_sms, kDkvThreads, dkv_smem, p, st);
  p.parts = 1;
  return e;
}

}  // namespace

size_t rc_dot_bytes(int64_t T, int H) { return (static_cast<size_t>(T) * H * 4 + 255) / 256 * 256; }
size_t rc_partial_bytes(const RcParams& p) {
  return static_cast<size_t>(p.T / 128 + p.b) * p.H * p.bias.nb * 4;  // units_of of any sequences
}

cudaError_t launch_rc_fwd(RcParams& p, int num_sms, cudaStream_t st) {
  if (p.d <= 64) return p.bias.nb ? fwd_t<64, true>(p, num_sms, st) : fwd_t<64, false>(p, num_sms, st);
  return p.bias.nb ? fwd_t<128, true>(p, num_sms, st) : fwd_t<128, false>(p, num_sms, st);
}

cudaError_t launch_rc_bwd(RcParams& p, int num_sms, cudaStream_t st) {
  if (p.d <= 64) return p.bias.nb ? bwd_t<64, true>(p, num_sms, st) : bwd_t<64, false>(p, num_sms, st);
  return p.bias.nb ? bwd_t<128, true>(p, num_sms, st) : bwd_t<128, false>(p, num_sms, st);
}

}  // namespace tp
