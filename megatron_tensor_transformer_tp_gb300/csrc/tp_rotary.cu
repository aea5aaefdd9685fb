// Rotation of query and key heads by their tokens' positions, and the norm of
// every query and key head with that rotation in the same pass; forward and
// backward ("Megatron" walkthrough, section ParallelSelfAttention: between the
// QKV projection and the attention of each head; "Megatron tensor / model
// parallelism" notes, section Self-Attention层).
//
// Pair k of a head, at position t, turns by the angle t f_k (Su et al.,
// "RoFormer", 2021):  y1 = m (x1 cos - x2 sin),  y2 = m (x1 sin + x2 cos).
// The gradient is the transposed matrix: the same with -sin.  With the norm,
//   n = x r,  r = 1 / sqrt(mean x^2 + eps),  y = R (n g)
// (centred: x less its mean first), and backward, with e = (R^T dy) g,
//   dg = sum over rows and heads of (R^T dy) n,  dx = r (e - n mean(e n))
// (centred: less r mean(e) too).
//
// Angles without 64-bit floating point: f_k / 2 pi, the turns a position, comes
// as a 64-bit fraction of a turn; its product with the position modulo 2^64 is
// exact and drops the whole turns by itself; its upper 32 bits are the angle.  A
// position costs one integer product a pair, and the range reduction loses
// nothing at far ones: the fraction's own error, 2^-52 of itself and 2^-64 of a
// turn, times the position is all there is.
//
// One kernel form streams all of it: each value is read once and written once.
// A group of G lanes holds one head, 16 values a lane: 8 pairs of partners, so
// that no value crosses lanes but in the norm's sums, and a head may be
// written over itself.  A block takes a chunk of heads, one a group, and walks
// down its rows a tile at a time, so that a group's column, kind, gains and
// gain sums never change.  The tile's cosines and sines are computed once, into
// shared memory, while the tile before is worked on.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stddef.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <atomic>
#include <mutex>

#include "tp_device.cuh"
#include "tp_entry.h"
#include "tp_internal.h"

namespace tp {
namespace {

constexpr int kRoMaxD = 512;       // head width
constexpr int kRoPairs = kRoMaxD / 2;
constexpr int kRoMaxHeads = 4096;  // query and key heads
constexpr int kRoThreads = 256;    // of a block
constexpr int kRoFew = 160;        // of a smaller one
constexpr int kRoRows = 64;        // most rows of a tile
constexpr int kRoTable = 16384;    // bytes that its table should not exceed
constexpr int kRoShared = 228 << 10;  // shared memory of an SM; a block takes 1 KB besides its own
constexpr int kRoCluster = 8;      // blocks of a cluster
constexpr int kRoParts = 1024;     // most blocks of the backward with gains
constexpr int64_t kRoOneWave = 112 << 20;  // most bytes of a forward call that runs in one wave of blocks

enum RoMode : int { RO_ROTATE = 0, RO_NORM_FWD = 1, RO_NORM_BWD = 2 };

struct RoParams {
  const void* x;    // rotation: what is turned; norm: its input
  const void* dy;   // norm backward: gradient of the output
  void* out;
  int64_t ld_x, ld_dy, ld_out;
  const int64_t* starts;     // device, b + 1 values, or null
  const int64_t* positions;  // device, T values, or null
  const float* gq;
  const float* gk;           // gains, or null: one
  float* partial;            // (blocks, 2, d) sums of the gains' gradients, or null
  float *dgq, *dgk;          // the gains' gradients
  int accumulate;
  int cluster;               // blocks of the launch, a cluster that adds its sums by itself; 0: each block leaves its own
  int64_t T;
  int b, s;        // s: tokens of every sequence (no starts, no positions)
  int d, hq, hk;   // head width; query and key heads a shard
  int hs;          // heads a shard in memory: hq + 2 hk
  int items;       // query and key heads a row
  int copied;      // values a row that are copied, 0 in place
  int pairs;       // rotated pairs a head
  int G, log_g;    // lanes a head
  int slots;       // half layout: slots a head; interleaved: lanes a head that have values
  int rot_slots;   // those with rotated pairs
  int row_floats;  // floats of a row of the table
  int fill_rows;   // rows that a block's threads fill at the same time
  int chunks;      // parts that the heads are cut into, a block takes one
  int chunk_heads; // heads of a chunk
  int parts;       // rows a block works on at the same time
  int steps;       // of a tile, a multiple of the stages
  uint32_t apart;  // rows from one step to the next
  int centred;
  float eps, amp;
  float amp_sin;   // negative for the transposed rotation
  unsigned* err;
  uint64_t turn[kRoPairs];  // turns a position, 64-bit fractions
};

// ---------------------------------------------------------------------------
// Vectors of V elements as 32-bit words (V = 1: one word an element)
// ---------------------------------------------------------------------------
template <class E, int V>
struct Words {
  static constexpr int N = V == 1 ? 1 : V * static_cast<int>(sizeof(E)) / 4;
};

template <class E, int V>
__device__ __forceinline__ void load_vec(const E* p, uint32_t* w) {
  constexpr int N = Words<E, V>::N;
  if constexpr (N == 1) {
    if constexpr (V * sizeof(E) == 2) w[0] = *reinterpret_cast<const uint16_t*>(p);
    else w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (N == 2) {
    const uint2 q = *reinterpret_cast<const uint2*>(p);
    w[0] = q.x;
    w[1] = q.y;
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4 q = reinterpret_cast<const uint4*>(p)[i];
      w[4 * i] = q.x;
      w[4 * i + 1] = q.y;
      w[4 * i + 2] = q.z;
      w[4 * i + 3] = q.w;
    }
  }
}

template <class E, int V>
__device__ __forceinline__ void store_words(E* p, const uint32_t* w) {
  constexpr int N = Words<E, V>::N;
  if constexpr (N == 1) {
    if constexpr (V * sizeof(E) == 2) *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(w[0]);
    else *reinterpret_cast<uint32_t*>(p) = w[0];
  } else if constexpr (N == 2) {
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
      reinterpret_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  }
}

template <class E, int V>
__device__ __forceinline__ void unpack(const uint32_t* w, float* f) {
  if constexpr (sizeof(E) == 4) {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = __uint_as_float(w[i]);
  } else if constexpr (V == 1) {
    f[0] = __uint_as_float(w[0] << 16);
  } else {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}

// The result's one rounding to bf16.
template <class E, int V>
__device__ __forceinline__ void pack(const float* f, uint32_t* w) {
  if constexpr (sizeof(E) == 4) {
#pragma unroll
    for (int i = 0; i < V; ++i) w[i] = __float_as_uint(f[i]);
  } else if constexpr (V == 1) {
    w[0] = __bfloat16_as_ushort(__float2bfloat16_rn(f[0]));
  } else {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) w[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
  }
}

// Two fp32 operations an instruction (sm_100 and up): the kernels issue about
// one instruction a value otherwise, more than the memory leaves time for.
__device__ __forceinline__ void fma2(float* d, const float* a, const float* b, const float* c) {
  asm("{.reg .b64 a, b, c;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 a, a, b, c;\n\tmov.b64 {%0, %1}, a;}"
      : "=f"(d[0]), "=f"(d[1])
      : "f"(a[0]), "f"(a[1]), "f"(b[0]), "f"(b[1]), "f"(c[0]), "f"(c[1]));
}
__device__ __forceinline__ void mul2(float* d, const float* a, const float* b) {
  asm("{.reg .b64 a, b;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;}"
      : "=f"(d[0]), "=f"(d[1])
      : "f"(a[0]), "f"(a[1]), "f"(b[0]), "f"(b[1]));
}

// A gain.  The kernel before may be the optimizer's step of it, still writing when this one is launched: so this is an
// ordinary load that stays behind pdl_wait, not one of read-only data.  (Two sequences of 2048, 32 heads of 128, norm's
// forward: 32.1 us, as with read-only loads; past the L1 by __ldcg 37.9, every group of lanes reads the same lines.)
__device__ __forceinline__ float load_gain(const float* p) {
  float v;
  asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
  return v;
}

// ---------------------------------------------------------------------------
// Rows
// ---------------------------------------------------------------------------
// The starts of the sequences as a warp holds them: up to 31 sequences a start a
// lane, so that one load answers everything; more are looked for in memory.
struct Starts {
  const int64_t* from;  // null: every row is used
  int b, lane;
  int held;        // the lane's start, limited to [-1, 2^31 - 1]; behind the last one the largest
  int first, end;  // rows of sequences

  __device__ __forceinline__ static int limited(int64_t v) {
    return static_cast<int>(min(max(v, static_cast<int64_t>(-1)), static_cast<int64_t>(INT32_MAX)));
  }
  // Reads them, and reports starts that decrease or leave the buffer.
  __device__ __forceinline__ Starts(const RoParams& p) : from(p.starts), b(p.b), lane(threadIdx.x & 31), held(0) {
    first = 0;
    end = static_cast<int>(p.T);
    if (from == nullptr) return;
    bool fine = true;
    if (b < 32) {
      const int64_t v = lane <= b ? __ldcg(from + lane) : INT64_MAX;
      const int64_t after = __shfl_down_sync(0xffffffffu, v, 1);
      fine = lane > b || (v >= 0 && v <= p.T && (lane == b || after >= v));
      held = limited(v);
      first = max(__shfl_sync(0xffffffffu, held, 0), 0);
      end = min(__shfl_sync(0xffffffffu, held, b), end);
    } else {
      first = max(limited(__ldcg(from)), 0);
      end = min(limited(__ldcg(from + b)), end);
      for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < b;
           i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t a = __ldcg(from + i), e = __ldcg(from + i + 1);
        fine &= a >= 0 && e >= a && e <= p.T;
      }
    }
    if (!fine) atomicOr(p.err, kErrInvalid);
  }
  // Start of the sequence that row t belongs to: the last one that is not behind
  // it.  Called by a whole warp.  Any contents of memory end the search in
  // ceil(log32(b)) steps, inside the array.
  __device__ __forceinline__ int of(int t) const {
    if (b < 32) {
      const unsigned below = __ballot_sync(0xffffffffu, lane < b && held <= t);
      return __shfl_sync(0xffffffffu, held, below ? 31 - __clz(below) : 0);
    }
    int lo = 0, hi = b, at = 0;
    while (hi > lo) {
      const int step = (hi - lo + 31) / 32;
      const int i = lo + lane * step;
      const int v = i < hi ? limited(__ldcg(from + i)) : INT32_MAX;
      const unsigned below = __ballot_sync(0xffffffffu, v <= t);
      const int last = below ? 31 - __clz(below) : 0;
      at = __shfl_sync(0xffffffffu, v, last);
      lo = lo + last * step;
      hi = min(hi, lo + step);
      if (step == 1) break;
    }
    return at;
  }
};

// Positions of the rows of a tile: `steps` steps of p.parts rows, p.apart rows
// apart.  Rows behind the buffer's have none.
__device__ __forceinline__ void fill_positions(const RoParams& p, const Starts& starts, uint32_t row0, int steps,
                                               int64_t* pos) {
  const int n = steps * p.parts;
  const uint32_t T = static_cast<uint32_t>(p.T);
  auto row_of = [&](int r) {
    const int step = p.parts == 1 ? r : r / p.parts;
    return row0 + static_cast<uint32_t>(step) * p.apart + (r - step * p.parts);
  };
  if (p.positions == nullptr && starts.from != nullptr) {
    for (int r = threadIdx.x >> 5; r < n; r += blockDim.x >> 5) {
      const uint32_t t = row_of(r);
      if (t >= T) continue;
      const int at = starts.of(static_cast<int>(t));
      if (starts.lane == 0) pos[r] = static_cast<int>(t) - at;
    }
  } else if (static_cast<int>(threadIdx.x) < n) {
    const uint32_t t = row_of(threadIdx.x);
    if (t < T) pos[threadIdx.x] = p.positions ? __ldcg(p.positions + t) : static_cast<int64_t>(t % p.s);
  }
}

// A row of the table has, for every slot of kPairs pairs, their cosines, sines and
// negated sines, times the amplitude, in kSlot floats: with 28 for 8 pairs the
// 16-byte reads of eight lanes fall on different banks.
template <int V, bool INTER>
constexpr int kPairs = INTER ? 8 : V;
template <int V, bool INTER>
constexpr int kSlot = kPairs<V, INTER> == 8 ? 28 : 3 * V;

// Where pair k's cosine lies in its row.  Interleaved: V / 2 pairs a vector,
// vector v is number v / used of lane v % used.
template <int V, bool INTER>
__device__ __forceinline__ int place(const RoParams& p, int k) {
  if constexpr (INTER) {
    const int v = k / (V / 2), j = v / p.slots;
    return (v - j * p.slots) * kSlot<V, INTER> + j * (V / 2) + k % (V / 2);
  } else {
    return k / V * kSlot<V, INTER> + k % V;
  }
}

// Cosine and sine of the angle of a position, whose turns are a whole number of
// 2^-32nds.  The nearest quarter turn is taken off in whole numbers, which leaves
// x in [-pi/4, pi/4]; there Taylor's series to x^9 and x^8 leave out less than
// 2.6e-8, below half a step of 1.
__device__ __forceinline__ void cos_sin(int64_t position, uint64_t turn, float* c, float* s) {
  const uint32_t u = static_cast<uint32_t>((static_cast<uint64_t>(position) * turn) >> 32);
  const uint32_t quarter = (u + (1u << 29)) >> 30;
  const float x = static_cast<float>(static_cast<int32_t>(u << 2)) * 3.6572951981e-10f;  // pi / 2 2^-32
  const float y = x * x;
  float p = fmaf(y, 2.7557319224e-6f, -1.9841269841e-4f);  // 1 / 9!, -1 / 7!
  p = fmaf(y, p, 8.3333333333e-3f);
  p = fmaf(y, p, -1.6666666667e-1f);
  p = fmaf(x * y, p, x);
  float q = fmaf(y, 2.4801587302e-5f, -1.3888888889e-3f);  // 1 / 8!, -1 / 6!
  q = fmaf(y, q, 4.1666666667e-2f);
  q = fmaf(y, q, -0.5f);
  q = fmaf(y, q, 1.f);
  const bool odd = quarter & 1;
  *s = __uint_as_float(__float_as_uint(odd ? q : p) ^ (quarter & 2) << 30);
  *c = __uint_as_float(__float_as_uint(odd ? p : q) ^ ((quarter + 1) & 2) << 30);
}

// The table of a tile's n rows.  A thread keeps its pair and goes from row to row.
template <int V, bool INTER>
__device__ __forceinline__ void fill_table(const RoParams& p, int n, const int64_t* pos, const uint64_t* turn, int r0,
                                           int k0, float* tab) {
  for (int k = k0; k < p.pairs; k += blockDim.x) {
    const uint64_t t = turn[k];
    float* to = tab + place<V, INTER>(p, k);
    for (int r = r0; r < n; r += p.fill_rows) {
      float c, s;
      cos_sin(pos[r], t, &c, &s);
      float* row = to + r * p.row_floats;
      c *= p.amp;
      s *= p.amp_sin;
      row[0] = c;
      row[kPairs<V, INTER>] = s;
      row[2 * kPairs<V, INTER>] = -s;
    }
  }
}

template <int N>
__device__ __forceinline__ void read_table(const float* from, float* f) {
  if constexpr (N == 1) {
    f[0] = from[0];
  } else if constexpr (N == 2) {
    const float2 a = *reinterpret_cast<const float2*>(from);
    f[0] = a.x; f[1] = a.y;
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 a = *reinterpret_cast<const float4*>(from + i);
      f[i] = a.x; f[i + 1] = a.y; f[i + 2] = a.z; f[i + 3] = a.w;
    }
  }
}

// One thread's copy of 4, 8 or 16 bytes into shared memory, not waited for.
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t to, const void* from) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(from), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

// ---------------------------------------------------------------------------
// A lane's part of a head
// ---------------------------------------------------------------------------
// 16 / V vectors of V values, so that the lanes' vectors lie side by side in the
// row.  Half layout: 8 / V slots of two vectors, a and b; the rotated ones first,
// their vectors n_rot / 2 apart, pair e of a slot element e of both; then what is
// not rotated.  Interleaved: pairs are elements 2e and 2e + 1 of a vector.  The
// lane's values are held as f[0..7], the pairs' first elements, and f[8..15],
// their second ones.
template <class E, int V, bool INTER>
struct Lane {
  static constexpr int S = 8 / V;
  static constexpr int N = Words<E, V>::N;
  static constexpr int kWords = 2 * S * N;
  int a[S], b[S];     // columns of a slot's vectors
  bool ha[S], hb[S];  // and whether the head has them
  int turned[2 * S];  // rotated pairs of the slot (half layout), of the vector (interleaved)
  int first;          // the lane's number; slot i is number first + i G
  // The lane's units of 4, 8 or 16 bytes in a stage: those of one number lie side
  // by side, lane after lane (no two lanes of a warp on one bank).  Single
  // elements (V = 1) lie as in the row.
  static constexpr int U = V * sizeof(E) < 16 ? V * sizeof(E) : 16;
  uint32_t at0, apart;

  // home: the group's place in a stage
  __device__ __forceinline__ Lane(const RoParams& p, int lane, uint32_t home) : first(lane & (p.G - 1)) {
    at0 = V == 1 ? home : home + first * U;
    apart = p.G * U;
#pragma unroll
    for (int i = 0; i < S; ++i) {
      if (INTER) {
        a[i] = (first + 2 * i * p.slots) * V;
        b[i] = a[i] + p.slots * V;
        ha[i] = first < p.slots && a[i] < p.d;
        hb[i] = first < p.slots && b[i] < p.d;
        turned[2 * i] = ha[i] ? min(max(p.pairs - a[i] / 2, 0), V / 2) : 0;
        turned[2 * i + 1] = hb[i] ? min(max(p.pairs - b[i] / 2, 0), V / 2) : 0;
        continue;
      }
      const int slot = first + i * p.G, rest = p.slots - p.rot_slots;
      if (slot < p.rot_slots) {
        a[i] = slot * V;
        b[i] = a[i] + p.pairs;
      } else {
        a[i] = 2 * p.pairs + (slot - p.rot_slots) * V;
        b[i] = a[i] + rest * V;
      }
      ha[i] = slot < p.slots && a[i] < p.d;
      hb[i] = slot < p.slots && b[i] < p.d;
      turned[i] = slot < p.rot_slots ? V : 0;
    }
  }
  // Zeros in place of what the head does not have: nothing is copied there.
  __device__ __forceinline__ void clear(uint8_t* stage) const {
    if constexpr (V > 1) {
#pragma unroll
      for (int u = 0; u < 16 * static_cast<int>(sizeof(E)) / U; ++u) {
        const int v = u * U / (V * static_cast<int>(sizeof(E)));
        if (v % 2 ? hb[v / 2] : ha[v / 2]) continue;
#pragma unroll
        for (int k = 0; k < U; k += 4) *reinterpret_cast<uint32_t*>(stage + at0 + u * apart + k) = 0u;
      }
    }
  }
  // Copies the lane's part of a head into its place of a stage.  With single
  // elements every G-th 16 bytes of the head, which other lanes read.
  __device__ __forceinline__ void fetch(const RoParams& p, const uint8_t* head, uint32_t stage) const {
    if constexpr (V == 1) {
      for (int c = first * 16; c < p.d * static_cast<int>(sizeof(E)); c += p.G * 16)
        copy_async<16>(stage + at0 + c, head + c);
    } else {
      constexpr int B = V * sizeof(E);
#pragma unroll
      for (int i = 0; i < S; ++i) {
        const uint8_t *pa = head + a[i] * sizeof(E), *pb = head + b[i] * sizeof(E);
#pragma unroll
        for (int k = 0; k < B / U; ++k) {
          if (ha[i]) copy_async<U>(stage + at0 + (2 * i * (B / U) + k) * apart, pa + k * U);
          if (hb[i]) copy_async<U>(stage + at0 + ((2 * i + 1) * (B / U) + k) * apart, pb + k * U);
        }
      }
    }
  }
  // The lane's vectors from a stage.
  __device__ __forceinline__ void read(const uint8_t* stage, uint32_t* w) const {
    if constexpr (V == 1) {
#pragma unroll
      for (int i = 0; i < S; ++i) {
        w[2 * i] = w[2 * i + 1] = 0u;
        if (ha[i]) load_vec<E, V>(reinterpret_cast<const E*>(stage + at0) + a[i], w + 2 * i);
        if (hb[i]) load_vec<E, V>(reinterpret_cast<const E*>(stage + at0) + b[i], w + 2 * i + 1);
      }
    } else {
#pragma unroll
      for (int u = 0; u < 16 * static_cast<int>(sizeof(E)) / U; ++u) {
        const uint8_t* from = stage + at0 + u * apart;
        if constexpr (U == 16) {
          const uint4 q = *reinterpret_cast<const uint4*>(from);
          w[4 * u] = q.x; w[4 * u + 1] = q.y; w[4 * u + 2] = q.z; w[4 * u + 3] = q.w;
        } else if constexpr (U == 8) {
          const uint2 q = *reinterpret_cast<const uint2*>(from);
          w[2 * u] = q.x; w[2 * u + 1] = q.y;
        } else {
          w[u] = *reinterpret_cast<const uint32_t*>(from);
        }
      }
    }
  }
  // Writes the lane's vectors; single elements go through shared memory.
  __device__ __forceinline__ void store(const RoParams& p, uint8_t* stage, uint8_t* head, bool mine,
                                        const uint32_t* w) const {
    if constexpr (V == 1) {
      __syncwarp();  // the others have read theirs
      put(reinterpret_cast<E*>(stage + at0), w);
      __syncwarp();
      if (mine) {
        for (int c = first * 16; c < p.d * static_cast<int>(sizeof(E)); c += p.G * 16)
          *reinterpret_cast<uint4*>(head + c) = *reinterpret_cast<const uint4*>(stage + at0 + c);
      }
    } else if (mine) {
      put(reinterpret_cast<E*>(head), w);
    }
  }
  __device__ __forceinline__ void put(E* head, const uint32_t* w) const {
#pragma unroll
    for (int i = 0; i < S; ++i) {
      if (ha[i]) store_words<E, V>(head + a[i], w + 2 * N * i);
      if (hb[i]) store_words<E, V>(head + b[i], w + 2 * N * i + N);
    }
  }
  __device__ __forceinline__ void floats(const uint32_t* w, float* f) const {
    float v[16];
#pragma unroll
    for (int i = 0; i < 2 * S; ++i) unpack<E, V>(w + N * i, v + V * i);
#pragma unroll
    for (int i = 0; i < 16; ++i) f[at(i)] = v[i];
  }
  __device__ __forceinline__ void words(const float* f, uint32_t* w) const {
    float v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = f[at(i)];
#pragma unroll
    for (int i = 0; i < 2 * S; ++i) pack<E, V>(v + V * i, w + N * i);
  }
  // Place in f of element i of the lane's vectors in a row.
  __device__ __forceinline__ static constexpr int at(int i) {
    return INTER ? (i & 1) * 8 + i / 2 : (i / V & 1) * 8 + i / (2 * V) * V + i % V;
  }
  // fn(place in f, column) for every value that the head has.
  template <class F>
  __device__ __forceinline__ void each(F&& fn) const {
#pragma unroll
    for (int i = 0; i < S; ++i) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        if (ha[i]) fn(at(2 * V * i + e), a[i] + e);
        if (hb[i]) fn(at(2 * V * i + V + e), b[i] + e);
      }
    }
  }
  // Rotates the lane's pairs; what is not rotated is not touched.
  __device__ __forceinline__ void turn(const RoParams& p, const float* row, float* f) const {
    if constexpr (INTER) {
      if (turned[0] == 0) return;  // (the vectors' columns rise)
      const float* from = row + first * kSlot<V, INTER>;
      float c[8], s[8], z[8];
      read_table<8>(from, c);
      read_table<8>(from + 8, s);
      read_table<8>(from + 16, z);
#pragma unroll
      for (int j = 0; j < 2 * S; ++j) {
        constexpr int P = V / 2;
        if (turned[j] == P) {
          pairs<P>(f + j * P, f + 8 + j * P, c + j * P, s + j * P, z + j * P);
        } else {
          // the last vector of a part that does not fill it
#pragma unroll
          for (int e = 0; e < P; ++e)
            if (e < turned[j]) pairs<1>(f + j * P + e, f + 8 + j * P + e, c + j * P + e, s + j * P + e, z + j * P + e);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < S; ++i) {
        if (turned[i] == 0) continue;
        const float* from = row + (first + i * p.G) * kSlot<V, INTER>;
        float c[V], s[V], z[V];
        read_table<V>(from, c);
        read_table<V>(from + V, s);
        read_table<V>(from + 2 * V, z);
        pairs<V>(f + V * i, f + 8 + V * i, c, s, z);
      }
    }
  }
  // N pairs (x, y) <- (x c - y s, x s + y c), z = -s
  template <int N>
  __device__ __forceinline__ static void pairs(float* x, float* y, const float* c, const float* s, const float* z) {
    if constexpr (N == 1) {
      const float u = fmaf(x[0], c[0], y[0] * z[0]);
      y[0] = fmaf(x[0], s[0], y[0] * c[0]);
      x[0] = u;
    } else {
#pragma unroll
      for (int e = 0; e < N; e += 2) {
        float u[2], v[2];
        mul2(u, y + e, z + e);
        mul2(v, y + e, c + e);
        fma2(y + e, x + e, s + e, v);
        fma2(x + e, x + e, c + e, u);
      }
    }
  }
};

// Sums of N values each over the G lanes of a head (a power of two); every
// lane of the warp takes part.  One branch for the usual widths, not one a step.
template <int N, int FROM>
__device__ __forceinline__ void lane_sums(float* v) {
#pragma unroll
  for (int o = FROM; o > 0; o >>= 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  }
}
template <int N>
__device__ __forceinline__ void group_sums(float* v, int G) {
  if (G == 8) return lane_sums<N, 4>(v);
  if (G == 4) return lane_sums<N, 2>(v);
  if (G >= 16) {
    if (G == 32) lane_sums<N, 16>(v);
    else lane_sums<N, 8>(v);
  } else if (G == 2) {
    lane_sums<N, 1>(v);
  }
}

// sum over f[i] g[i]: two chains of 8
__device__ __forceinline__ float dot16(const float* f, const float* g) {
  float t[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 16; i += 2) fma2(t, f + i, g + i, t);
  return t[0] + t[1];
}

// ---------------------------------------------------------------------------
// The kernel
// ---------------------------------------------------------------------------
// A sum of the gains' gradients, column c of (2, d).
__device__ __forceinline__ void add_gain(float* dgq, float* dgk, int d, int c, float t, int accumulate) {
  float* to = c < d ? dgq : dgk;
  if (to == nullptr) return;
  to += c < d ? c : c - d;
  *to = accumulate ? *to + t : t;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The value at the same shared-memory address of the cluster's block `rank`.
__device__ __forceinline__ float read_cluster(const float* at, int rank) {
  float v;
  asm volatile("{.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.f32 %0, [a];}"
               : "=f"(v)
               : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(at))), "r"(rank)
               : "memory");
  return v;
}

// Head of a group of the chunk.
__device__ __forceinline__ int block_head(const RoParams& p, int chunk, int slot) {
  const int log_unit = 5 - p.log_g, in_unit = slot & ((1 << log_unit) - 1);
  return p.chunks == 1 ? slot : (((slot >> log_unit) * p.chunks + chunk) << log_unit) + in_unit;
}

// Rows on their way to a group, the one that is worked on among them.  (The backward, 65536 rows of 8 + 2 heads: 92 us;
// with 4, 123: one block less an SM.)
template <class E, int MODE>
constexpr int kDepth = sizeof(E) == 4 ? 2 : MODE == RO_NORM_BWD ? 3 : 4;
// A stage: the groups' heads and, behind those of x, the values that are copied (of dy in the backward).  Constants for
// blocks of up to NT threads: with a size known at the launch, addresses took registers that the kernels lack (two
// sequences of 2048, 32 heads of 128, norm's forward: 39 us, 33 so).
template <class E, int NT>
constexpr uint32_t kStageY = NT * 16 * sizeof(E);
template <class E, int NT>
constexpr uint32_t kStageX = kStageY<E, NT> + NT * 8 * sizeof(E);
// Most blocks on an SM, by their registers: 128 a thread, or 96 for the smaller blocks' forward.  (Stages and table may
// leave room for fewer.)  More blocks with fewer registers were slower (norm's forward, 3 blocks of 256 threads: two
// sequences of 2048, 32 heads of 128, interleaved, 38 us instead of 32; 5 blocks of 160: 12000 rows of 16 + 4 heads of 96
// 30 instead of 26).
template <int MODE, int NT>
constexpr int kBlocks = NT != kRoFew ? 2 : MODE == RO_NORM_BWD ? 3 : 4;

template <class E, int V, bool INTER, int MODE, int NT>
__global__ void __launch_bounds__(NT, kBlocks<MODE, NT>)
    rotary_kernel(const __grid_constant__ RoParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int64_t pos[2][kRoRows];
  using LaneT = Lane<E, V, INTER>;
  constexpr bool kBwd = MODE == RO_NORM_BWD;
  constexpr int D = kDepth<E, MODE>;
  constexpr uint32_t stage = kStageX<E, NT>, stage_y = kStageY<E, NT>;
  constexpr uint32_t ys = D * stage;  // the stages of dy lie behind those of x
  uint64_t* turn = reinterpret_cast<uint64_t*>(smem + ys + (kBwd ? D * stage_y : 0));
  float* tab = reinterpret_cast<float*>(turn + ((p.pairs + 1) & ~1));
  // the group's head: the chunks take turns by runs of a warp's heads
  const int group = threadIdx.x >> p.log_g;
  const LaneT L(p, threadIdx.x & 31, group * p.G * 16 * sizeof(E));
  const int block = blockIdx.x / p.chunks, chunk = blockIdx.x - block * p.chunks;
  const int part = group / p.chunk_heads, slot = group - part * p.chunk_heads;
  const int head = block_head(p, chunk, slot);
  const bool active = part < p.parts && head < p.items;
  const int in_shard = p.hq + p.hk, shard = head / in_shard, place_in = head - shard * in_shard;
  const bool key = place_in >= p.hq;
  // eight of the value heads' columns, numbered through the shards: half as many as the lane's own at most, so one
  // such run a lane is enough
  const int v_at = (head * p.G + L.first) * 8, v_width = p.hk * p.d, v_shard = v_at / v_width;
  const bool copies = active && v_at < p.copied;
  // the block's rows: p.parts at a time, p.apart apart
  const uint32_t base = block * p.parts, T = static_cast<uint32_t>(p.T);
  const int total = (T - base + p.apart - 1) / p.apart;  // steps
  // the thread's first row and pair of a table: whole rows of pairs side by side, or, of more pairs than threads, parts
  // of one
  const bool wide = p.pairs > static_cast<int>(blockDim.x);
  const int fill_r = wide ? 0 : threadIdx.x / max(p.pairs, 1);
  const int fill_k = wide ? threadIdx.x : threadIdx.x - fill_r * p.pairs;
  const int r0 = fill_r < p.fill_rows ? fill_r : INT32_MAX;

  for (int i = threadIdx.x; i < p.pairs; i += blockDim.x) turn[i] = p.turn[i];
#pragma unroll
  for (int i = 0; i < D; ++i) {
    L.clear(smem + i * stage);
    if (kBwd) L.clear(smem + ys + i * stage_y);
  }
  // column of the head's rows
  const int64_t col = static_cast<int64_t>(shard * p.hs + place_in) * p.d;
  uint32_t row = base + part;
  const uint8_t* fx = static_cast<const uint8_t*>(p.x) + (row * p.ld_x + col) * sizeof(E);
  const uint8_t* fy = static_cast<const uint8_t*>(p.dy) + (row * p.ld_dy + col) * sizeof(E);
  uint8_t* to = static_cast<uint8_t*>(p.out) + (row * p.ld_out + col) * sizeof(E);
  // from there to the value columns
  const int64_t to_v = (static_cast<int64_t>(v_shard * p.hs + in_shard) * p.d + v_at - v_shard * v_width - col) *
                       static_cast<int64_t>(sizeof(E));
  const uint32_t v_home = stage_y + threadIdx.x * 8 * sizeof(E);
  const int64_t step_x = p.apart * p.ld_x * sizeof(E), step_dy = p.apart * p.ld_dy * sizeof(E);
  const int64_t step_out = p.apart * p.ld_out * sizeof(E);
  pdl_wait();
  pdl_trigger();
  // fetches a row into stage `into`; unused rows too, so that nothing waits for the starts
  const uint32_t smem_at = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
  uint32_t f_row = row;
  int f_left = active ? total : 0;
  auto fetch = [&](int into) {
    if (f_left > 0 && f_row < T) {
      L.fetch(p, fx, smem_at + into * stage);
      if (kBwd) L.fetch(p, fy, smem_at + ys + into * stage_y);
      if (copies) {
#pragma unroll
        for (uint32_t k = 0; k < 8 * sizeof(E); k += 16)
          copy_async<16>(smem_at + into * stage + v_home + k, (kBwd ? fy : fx) + to_v + k);
      }
    }
    copies_commit();
    --f_left;
    f_row += p.apart;
    fx += step_x;
    if (kBwd) fy += step_dy;
  };
#pragma unroll
  for (int i = 0; i < D - 1; ++i) fetch(i);
  const Starts starts(p);
  const uint32_t first = starts.first;
  const uint32_t used = active && starts.end > starts.first ? starts.end - starts.first : 0;  // (starts may decrease)
  fill_positions(p, starts, base, min(p.steps, total), pos[0]);
  if (total > p.steps) fill_positions(p, starts, base + p.steps * p.apart, min(p.steps, total - p.steps), pos[1]);
  float g[MODE != RO_ROTATE ? 16 : 1], sum[kBwd ? 16 : 1];
  if (MODE != RO_ROTATE) {
    const float* gain = key ? p.gk : p.gq;
#pragma unroll
    for (int i = 0; i < 16; ++i) g[i] = 0.f;
    L.each([&](int i, int c) { g[i] = gain == nullptr ? 1.f : load_gain(gain + c); });
  }
  if (kBwd) {
#pragma unroll
    for (int i = 0; i < 16; ++i) sum[i] = 0.f;
  }
  __syncthreads();
  fill_table<V, INTER>(p, min(p.steps, total) * p.parts, pos[0], turn, r0, fill_k, tab);
  const float inv_d = 1.f / static_cast<float>(p.d);
  const int tab_floats = p.steps * p.parts * p.row_floats;

  // a row: stage `from` holds it, and the row D - 1 steps ahead goes into the stage before
  auto work = [&](int from, const float* angles) {
    const bool mine = row - first < used;
    if (V == 1) __syncwarp();  // the stage that is filled now is read
    fetch((from + D - 1) % D);
    copies_wait<D - 1>();
    if (V == 1) __syncwarp();
    uint8_t* sx = smem + from * stage;
    uint8_t* sy = smem + ys + from * stage_y;
    uint32_t w[LaneT::kWords];
    float f[16];
    if (!kBwd) {
      L.read(sx, w);
      L.floats(w, f);
      if (MODE == RO_NORM_FWD) {
        if (p.centred) {
          float m = 0.f;
#pragma unroll
          for (int i = 0; i < 16; ++i) m += f[i];
          group_sums<1>(&m, p.G);
          m *= -inv_d;
          L.each([&](int i, int) { f[i] += m; });
        }
        float q = dot16(f, f);
        group_sums<1>(&q, p.G);
        const float inv = rsqrtf(fmaf(q, inv_d, p.eps)), invs[2] = {inv, inv};
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          mul2(f + i, f + i, invs);
          mul2(f + i, f + i, g + i);
        }
      }
      if (mine) {
        L.turn(p, angles, f);
        L.words(f, w);
      }
      L.store(p, sx, to, mine, w);
    } else {
      float e[16];
      L.read(sy, w);
      L.floats(w, e);
      if (mine) L.turn(p, angles, e);
      L.read(sx, w);
      L.floats(w, f);
      float mean = 0.f;
      if (p.centred) {
        float m[2] = {0.f, 0.f};  // sums of x and of e g
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          m[0] += f[i];
          m[1] = fmaf(e[i], g[i], m[1]);
        }
        group_sums<2>(m, p.G);
        const float less = m[0] * -inv_d;
        L.each([&](int i, int) { f[i] += less; });
        mean = m[1] * inv_d;
      }
      float q[2], along[2] = {0.f, 0.f};  // sums of x^2 and of e g x
      q[0] = dot16(f, f);
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        float t[2];
        mul2(t, e + i, f + i);
        fma2(along, t, g + i, along);
      }
      q[1] = along[0] + along[1];
      group_sums<2>(q, p.G);
      const float inv = rsqrtf(fmaf(q[0], inv_d, p.eps));
      // dx = inv e g - x inv (inv (inv q1 / d)): in this order nothing is larger than the result's parts
      const float k = -inv * (inv * (inv * (q[1] * inv_d)));
      if (mine) {
        const float invs[2] = {inv, inv}, ks[2] = {k, k}, shift[2] = {-inv * mean, -inv * mean};
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          float t[2];
          mul2(e + i, e + i, invs);
          fma2(sum + i, e + i, f + i, sum + i);
          if (p.centred) fma2(t, f + i, ks, shift);
          else mul2(t, f + i, ks);
          fma2(e + i, e + i, g + i, t);
        }
        L.words(e, w);
      }
      L.store(p, sy, to, mine, w);
    }
    if (mine && copies) {
#pragma unroll
      for (uint32_t k = 0; k < 8 * sizeof(E); k += 16)
        *reinterpret_cast<uint4*>(to + to_v + k) = *reinterpret_cast<const uint4*>(sx + v_home + k);
    }
    row += p.apart;
    to += step_out;
  };
  int left = total;
  uint32_t ahead = base + 2 * p.steps * p.apart;  // first row of the tile after the next
  for (int even = 0; left > 0; left -= p.steps, ahead += p.steps * p.apart, even ^= 1) {
    __syncthreads();  // this tile's table and the next one's positions are there; the last tile's are read
    if (left > p.steps)
      fill_table<V, INTER>(p, min(p.steps, left - p.steps) * p.parts, pos[even ^ 1], turn, r0, fill_k,
                           tab + (even ^ 1) * tab_floats);
    if (left > 2 * p.steps) fill_positions(p, starts, ahead, min(p.steps, left - 2 * p.steps), pos[even]);
    const float* angles = tab + even * tab_floats + part * p.row_floats;
    const int n = min(p.steps, left);
    // (steps is a multiple of D: a tile begins at stage 0)
    for (int i = 0; i < n; i += D) {
#pragma unroll
      for (int j = 0; j < D; ++j) {
        if (i + j >= n) break;
        work(j, angles);
        angles += p.parts * p.row_floats;
      }
    }
  }
  copies_wait<0>();
  if constexpr (kBwd) {
    if (p.partial == nullptr) return;
    // the block's groups of each kind, in their order
    __syncthreads();
    const int d = p.d;
    float* red = reinterpret_cast<float*>(smem);
    for (int what = 0; what < 2; ++what) {
      // a warp's groups first: values of the other kind count as zero
      float t[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) t[i] = active && key == (what == 1) ? sum[i] : 0.f;
      for (int o = p.G; o < 32; o <<= 1) {
#pragma unroll
        for (int i = 0; i < 16; ++i) t[i] += __shfl_xor_sync(0xffffffffu, t[i], o);
      }
      if ((static_cast<int>(threadIdx.x) & 31) < p.G) {
        float* to = red + (static_cast<size_t>(threadIdx.x >> 5) * 2 + what) * d;
        L.each([&](int i, int c) { to[c] = t[i]; });
      }
    }
    __syncthreads();
    const int warps = blockDim.x >> 5;
    float* sums = p.cluster ? red + warps * 2 * d : p.partial + static_cast<size_t>(blockIdx.x) * 2 * d;
    for (int c = threadIdx.x; c < 2 * d; c += blockDim.x) {
      float t = 0.f;
      for (int w = 0; w < warps; ++w) t += red[static_cast<size_t>(w) * 2 * d + c];
      sums[c] = t;
    }
    if (p.cluster == 0) return;
    cluster_sync();
    for (int c = blockIdx.x * blockDim.x + threadIdx.x; c < 2 * d; c += p.cluster * blockDim.x) {
      float t = 0.f;
      for (int k = 0; k < p.cluster; ++k) t += read_cluster(sums + c, k);
      add_gain(p.dgq, p.dgk, d, c, t, p.accumulate);
    }
    cluster_sync();  // the others have read this block's
  }
}

// The blocks' sums: eight columns a block, 32 rows at a time in their order,
// then a tree.
constexpr int kGainColumns = 8;
__global__ void __launch_bounds__(32 * kGainColumns) qk_gain_sum_kernel(const float* __restrict__ partial, int parts,
                                                                       int d, float* dgq, float* dgk,
                                                                       int accumulate) {
  __shared__ float red[kGainColumns][33];
  const int c = threadIdx.x % kGainColumns, r = threadIdx.x / kGainColumns;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  pdl_wait();
  pdl_trigger();
  const float* from = partial + blockIdx.x * kGainColumns + c;
  float t = 0.f;
  for (int i = r; i < parts; i += 32 * 8) {
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = i + 32 * k < parts ? __ldcg(from + static_cast<size_t>(i + 32 * k) * 2 * d) : 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) t += v[k];
  }
  red[c][r] = t;
  __syncthreads();
  t = red[warp][lane];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  if (lane == 0) add_gain(dgq, dgk, d, blockIdx.x * kGainColumns + warp, t, accumulate);
}

// ---------------------------------------------------------------------------
// Launches
// ---------------------------------------------------------------------------
struct RoCall {
  RoMode mode;
  bool f32, inter;
  int vec, num_sms;
  cudaStream_t stream;
  RoParams p;  // last, its frequencies at its end: those are not cleared
};

// Warps of a block, chunks of heads and rows at the same time: as few idle groups as possible (of the threads that the
// block's stages are made for), and among equals few chunks, as each computes tables of its own.
int lay_out(RoParams* p, int max_parts) {
  const int unit = 32 / p->G, units = (p->items + unit - 1) / unit;
  int threads = 0;
  double best = 0.0;
  for (int warps = kRoThreads / 32; warps >= 4; --warps) {
    const bool few = warps * 32 <= kRoFew;
    const int groups = warps * unit, room = (few ? kRoFew : kRoThreads) / 32 * unit;
    for (int chunks = (units + warps - 1) / warps, tries = 0; tries < 3 && chunks <= kRoParts; ++chunks, ++tries) {
      const int heads = chunks == 1 ? p->items : (units + chunks - 1) / chunks * unit;
      const int parts = std::min(groups / heads, max_parts);
      const double busy = static_cast<double>(p->items) * parts / (static_cast<double>(room) * chunks);
      const double worth = busy / (1.0 + 0.01 * (chunks - 1)) * (few ? 0.98 : 1.0);
      if (worth > best + 1e-9) {
        best = worth;
        p->chunks = chunks;
        p->chunk_heads = heads;
        p->parts = parts;
        threads = warps * 32;
      }
    }
  }
  return threads;
}

// launch_k, the grid one cluster.
cudaError_t launch_cluster(void (*kernel)(RoParams), unsigned grid, int threads, size_t smem, cudaStream_t st,
                           const RoParams& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl_on() ? 1 : 0;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = grid;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <class E, int V, bool INTER, int MODE, int NT>
cudaError_t launch_block(RoCall& c, int threads, int max_rows) {
  constexpr int D = kDepth<E, MODE>;
  constexpr bool kBwd = MODE == RO_NORM_BWD;
  RoParams& p = c.p;
  p.steps = std::max(1, std::min(8, max_rows / p.parts) / D) * D;
  p.fill_rows = std::max(1, threads / std::max(1, p.pairs));
  size_t smem = (kStageX<E, NT> + (kBwd ? kStageY<E, NT> : 0)) * D + ((p.pairs + 1) & ~1) * 8 +
                static_cast<size_t>(2) * p.steps * p.parts * p.row_floats * 4;
  if (kBwd) smem = std::max(smem, static_cast<size_t>(threads / 32 + 1) * 8 * p.d);
  // Blocks that an SM holds at once: rows are dealt out evenly, so blocks beyond those would be a nearly empty second
  // wave.  (By the registers' limit alone / so: 16384 rows of 8 + 2 heads of 128, rotation 20.4 / 18.8 us, norm's forward
  // 24.0 / 20.4; 8192 in fp32, norm's backward 31.5 / 27.1.)
  const int fit = std::min(kBlocks<MODE, NT>, static_cast<int>(kRoShared / (smem + sizeof(int64_t[2][kRoRows]) + 1024)));
  const int64_t rows = (p.T + p.parts - 1) / p.parts;  // steps of all blocks of a chunk
  // Waves of blocks of the forward.  Several where the call is long: the next kernel's blocks find room while the last
  // ones end, and set-up hides behind the others' copies; one where set-up counts.  The size at which that changes
  // differs with the heads, so the limit is a compromise.  us by waves 1 / 2 / 3 / 5, calls on three sets of buffers:
  //   norm's forward, 16 + 4 heads of 96, 101 MB 20.0 21.2 21.8 25.2, 118 MB 22.6 23.6 24.2 27.6 (the rule takes 3),
  //     221 MB 38.8 40.6 40.4 41.3 (5); 32 + 32 heads of 128, 201 MB 33.9 32.1 31.9 32.5 (4: 32.0)
  //   rotation, 8 + 2 heads of 128, 61 MB 11.9 11.2 12.0 14.7 (1), 101 MB 18.7 17.7 17.2 19.2 (1), 123 MB 22.0 21.0 20.4 21.8
  //     (3), 403 MB 68.5 65.3 62.7 62.1 (18: 60.9); 32 + 8 heads of 128, 295 MB 49.9 47.2 45.0 44.3 (5)
  // The backward: one, as every block leaves sums of the gains' gradients (two: 48.7 -> 52.7).
  const int64_t wave = std::max(1, std::min(fit * c.num_sms, kRoParts) / p.chunks);
  const int64_t bytes = 2 * p.T * (static_cast<int64_t>(p.items) * p.d + p.copied) * static_cast<int64_t>(sizeof(E));
  int64_t blocks = wave;
  if (!kBwd && bytes > kRoOneWave) blocks *= (rows + 8 * wave - 1) / (8 * wave);
  blocks = std::min(blocks, rows);
  // Up to 32 steps of the backward run as one cluster, which adds the gains' gradients by itself: one launch on the host
  // instead of two, but fewer blocks on the GPU.  (96 rows of 8 + 8 heads of 64, 24 steps: 11.1 us a call instead of 13.4;
  // 6.8 us on the GPU instead of 5.6, which is what a replayed graph pays.)
  if (kBwd && p.partial && p.chunks <= kRoCluster && rows * p.chunks <= 4 * kRoCluster) {
    blocks = std::min<int64_t>(rows, kRoCluster / p.chunks);
    p.cluster = static_cast<int>(blocks * p.chunks);
  }
  p.apart = static_cast<uint32_t>(blocks * p.parts);
  const unsigned grid = static_cast<unsigned>(blocks * p.chunks);
  count_launches(1);
  if (p.cluster) return launch_cluster(rotary_kernel<E, V, INTER, MODE, NT>, grid, threads, smem, c.stream, p);
  const cudaError_t e = launch_k(rotary_kernel<E, V, INTER, MODE, NT>, grid, threads, smem, c.stream, p);
  if (e != cudaSuccess || !kBwd || p.partial == nullptr) return e;
  count_launches(1);
  return launch_k(qk_gain_sum_kernel, 2 * p.d / kGainColumns, 32 * kGainColumns, 0, c.stream,
                  static_cast<const float*>(p.partial), static_cast<int>(grid), p.d, p.dgq, p.dgk, p.accumulate);
}

// The call with its kernel, or (c null) the kernels' shared memory limits of the current device.
template <class E, int V, bool INTER, int MODE>
cudaError_t launch_mode(RoCall* c) {
  if (c == nullptr) {
    constexpr int kMost = 160 * 1024;
    const cudaError_t e = cudaFuncSetAttribute(rotary_kernel<E, V, INTER, MODE, kRoThreads>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
    return e != cudaSuccess ? e : cudaFuncSetAttribute(rotary_kernel<E, V, INTER, MODE, kRoFew>,
                                                       cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
  }
  RoParams& p = c->p;
  p.row_floats = p.rot_slots * kSlot<V, INTER>;
  const int max_rows = p.pairs ? std::max(1, std::min(kRoRows, kRoTable / (4 * p.row_floats))) : kRoRows;
  const int threads = lay_out(&p, std::max(1, max_rows / kDepth<E, MODE>));
  return threads <= kRoFew ? launch_block<E, V, INTER, MODE, kRoFew>(*c, threads, max_rows)
                           : launch_block<E, V, INTER, MODE, kRoThreads>(*c, threads, max_rows);
}

template <class E, int V, bool INTER>
cudaError_t launch_as(RoCall* c) {
  if (c == nullptr) {
    cudaError_t e = launch_mode<E, V, INTER, RO_ROTATE>(nullptr);
    if (e == cudaSuccess) e = launch_mode<E, V, INTER, RO_NORM_FWD>(nullptr);
    return e != cudaSuccess ? e : launch_mode<E, V, INTER, RO_NORM_BWD>(nullptr);
  }
  if (c->mode == RO_ROTATE) return launch_mode<E, V, INTER, RO_ROTATE>(c);
  if (c->mode == RO_NORM_FWD) return launch_mode<E, V, INTER, RO_NORM_FWD>(c);
  return launch_mode<E, V, INTER, RO_NORM_BWD>(c);
}

cudaError_t launch_call(void* call) {
  RoCall* c = static_cast<RoCall*>(call);
  if (c->f32) {
    if (c->inter) return launch_as<float, 4, true>(c);
    if (c->vec == 4) return launch_as<float, 4, false>(c);
    return c->vec == 2 ? launch_as<float, 2, false>(c) : launch_as<float, 1, false>(c);
  }
  if (c->inter) return launch_as<__nv_bfloat16, 8, true>(c);
  if (c->vec == 8) return launch_as<__nv_bfloat16, 8, false>(c);
  if (c->vec == 4) return launch_as<__nv_bfloat16, 4, false>(c);
  return c->vec == 2 ? launch_as<__nv_bfloat16, 2, false>(c) : launch_as<__nv_bfloat16, 1, false>(c);
}

// Once a device, at the first call with it current.
cudaError_t set_up() {
  static std::mutex mu;
  static std::atomic<bool> done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || dev < 0 || dev >= 64) return e != cudaSuccess ? e : cudaErrorInvalidDevice;
  if (done[dev].load(std::memory_order_acquire)) return cudaSuccess;
  std::lock_guard<std::mutex> lk(mu);
  if (done[dev].load(std::memory_order_relaxed)) return cudaSuccess;
  constexpr cudaError_t (*kAll[])(RoCall*) = {
      launch_as<float, 4, true>,          launch_as<float, 4, false>,         launch_as<float, 2, false>,
      launch_as<float, 1, false>,         launch_as<__nv_bfloat16, 8, true>,  launch_as<__nv_bfloat16, 8, false>,
      launch_as<__nv_bfloat16, 4, false>, launch_as<__nv_bfloat16, 2, false>, launch_as<__nv_bfloat16, 1, false>};
  for (auto kernels : kAll)
    if ((e = kernels(nullptr)) != cudaSuccess) return e;
  done[dev].store(true, std::memory_order_release);
  return cudaSuccess;
}

// ---------------------------------------------------------------------------
// Arguments
// ---------------------------------------------------------------------------
inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Turns a position as a 64-bit fraction.  The constant and the product are rounded, 2^-52 of the turns together; what
// is behind the fraction's 64 bits is cut off.
uint64_t turn_fraction(double freq) {
  double turns = freq * 0.15915494309189533577;  // 1 / 2 pi
  if (turns >= 1.0) turns -= floor(turns);       // exact
  return static_cast<uint64_t>(turns * 0x1p64);  // 0 <= turns < 1
}

// Numbers of rows and heads, and the head width but for its multiple.
bool head_sizes(const tp_attn_config* cfg) {
  return cfg->T >= 0 && cfg->T <= INT32_MAX - 511 && cfg->n_heads >= 1 && cfg->n_kv_heads >= 1 && cfg->N >= 1 &&
         cfg->N <= 8 && cfg->n_heads % cfg->N == 0 && cfg->n_kv_heads % cfg->N == 0 &&
         cfg->n_heads % cfg->n_kv_heads == 0 && cfg->d >= 1 && cfg->d <= kRoMaxD &&
         cfg->n_heads <= kRoMaxHeads - cfg->n_kv_heads;
}

// Sizes and the rotation into c, without pointers.
tp_status ro_sizes(const tp_attn_config* cfg, const tp_rotary_config* rot, bool norm, const int64_t* seq_starts,
                   const int64_t* positions, bool f32, RoCall* c) {
  if (cfg == nullptr || (rot == nullptr && !norm)) return TP_ERR_INVALID;
  if (!head_sizes(cfg)) return TP_ERR_INVALID;
  if (cfg->T > 0) {
    if (seq_starts != nullptr) {
      if (cfg->b < 1 || cfg->b > (1 << 22)) return TP_ERR_INVALID;
    } else if (positions == nullptr) {
      if (cfg->b < 1 || cfg->s < 1 || cfg->s > cfg->T || cfg->b > cfg->T || cfg->b * cfg->s != cfg->T)
        return TP_ERR_INVALID;
    }
  }
  RoParams& p = c->p;
  const int n_rot = rot ? rot->n_rot : 0;
  if (n_rot < (norm ? 0 : 2) || n_rot > cfg->d || n_rot % 2 != 0) return TP_ERR_INVALID;
  if (n_rot > 0) {
    if (rot->freq == nullptr || !(rot->amplitude >= 0.f) || !isfinite(rot->amplitude)) return TP_ERR_INVALID;
    for (int k = 0; k < n_rot / 2; ++k) {
      if (!(rot->freq[k] >= 0.0) || !(rot->freq[k] <= 1048576.0)) return TP_ERR_INVALID;
      p.turn[k] = turn_fraction(rot->freq[k]);
    }
  }
  if (cfg->d % 8 != 0) return TP_ERR_ALIGN;
  p.T = cfg->T;
  p.b = seq_starts ? static_cast<int>(cfg->b) : 0;
  p.s = seq_starts || positions ? 1 : static_cast<int>(cfg->s);
  p.d = cfg->d;
  p.hq = cfg->n_heads / cfg->N;
  p.hk = cfg->n_kv_heads / cfg->N;
  p.hs = p.hq + 2 * p.hk;
  p.pairs = n_rot / 2;
  p.amp = n_rot > 0 && rot->amplitude > 0.f ? rot->amplitude : 1.f;
  p.amp_sin = p.amp;
  c->inter = n_rot > 0 && rot->interleaved != 0;
  // Vectors of 16 bytes.  Partners in the half layout lie n_rot / 2 apart: the
  // widest that keep both ends of a pair aligned (8192 rows of 16 + 16 heads of 64
  // with n_rot = 20, rotation: 28 us by twos, 39 by single elements).
  const int widest = f32 ? 4 : 8;
  c->vec = c->inter || p.pairs % widest == 0 ? widest : p.pairs % 4 == 0 ? 4 : p.pairs % 2 == 0 ? 2 : 1;
  const int v = c->vec;
  int lanes;
  if (c->inter) {
    lanes = p.slots = (p.d + 15) / 16;
    p.rot_slots = std::min(p.slots, (2 * p.pairs + v - 1) / v);
  } else {
    p.rot_slots = p.pairs / v;
    p.slots = p.rot_slots + ((p.d - n_rot) / v + 1) / 2;
    lanes = (p.slots + 8 / v - 1) / (8 / v);
  }
  p.G = 1;
  while (p.G < lanes) p.G <<= 1, ++p.log_g;
  return TP_OK;
}

void clear(RoCall* c) { memset(static_cast<void*>(c), 0, offsetof(RoCall, p) + offsetof(RoParams, turn)); }

// What every call checks and fills in.
tp_status ro_args(tp_dtype dt, RoMode mode, const tp_attn_config* cfg, const tp_rotary_config* rot,
                  const tp_qk_norm_config* norm, const int64_t* seq_starts, const int64_t* positions, const void* x,
                  int64_t ld_x, const void* dy, int64_t ld_dy, void* out, int64_t ld_out, RoCall* c) {
  if (dt != TP_F32 && dt != TP_BF16) return TP_ERR_UNSUPPORTED;
  const bool with_norm = mode != RO_ROTATE;
  if (with_norm && norm == nullptr) return TP_ERR_INVALID;
  tp_status st = ro_sizes(cfg, rot, with_norm, seq_starts, positions, dt == TP_F32, c);
  if (st == TP_ERR_INVALID) return st;
  if (with_norm && ((norm->kind != TP_NORM_RMS && norm->kind != TP_NORM_LAYER) || !(norm->eps > 0.f) ||
                    !isfinite(norm->eps)))
    return TP_ERR_INVALID;
  if (st != TP_OK || cfg->T == 0) return st;
  if (!x || !out || (mode == RO_NORM_BWD && !dy)) return TP_ERR_INVALID;
  RoParams& p = c->p;
  const int64_t width = static_cast<int64_t>(p.hs) * cfg->N * p.d;
  auto pitch = [&](int64_t ld) { return ld >= width && ld <= (int64_t{1} << 36); };
  if (!pitch(ld_x) || !pitch(ld_out) || (dy && !pitch(ld_dy))) return TP_ERR_INVALID;
  const int64_t unit = dt == TP_F32 ? 4 : 8;
  if (!aligned(x, 16) || !aligned(out, 16) || !aligned(dy, 16) || ld_x % unit != 0 || ld_out % unit != 0 ||
      (dy && ld_dy % unit != 0) || !aligned(seq_starts, 8) || !aligned(positions, 8))
    return TP_ERR_ALIGN;
  // in place: the values' heads stay, and every element is written by the lane that read it
  const void* src = mode == RO_NORM_BWD ? dy : x;
  if (out == src && ld_out != (mode == RO_NORM_BWD ? ld_dy : ld_x)) return TP_ERR_INVALID;
  if (mode == RO_NORM_BWD && out == x) return TP_ERR_INVALID;
  p.x = x;
  p.dy = dy;
  p.out = out;
  p.ld_x = ld_x;
  p.ld_dy = ld_dy;
  p.ld_out = ld_out;
  p.starts = seq_starts;
  p.positions = positions;
  p.items = (p.hq + p.hk) * cfg->N;
  p.copied = out == src ? 0 : p.hk * cfg->N * p.d;
  p.centred = with_norm && norm->kind == TP_NORM_LAYER;
  p.eps = with_norm ? norm->eps : 0.f;
  c->mode = mode;
  c->f32 = dt == TP_F32;
  return TP_OK;
}

tp_status ro_run(const char* name, RoCall* c, void* stream) {
  const tp_status st = entry_device(&c->num_sms, &c->p.err);
  if (st != TP_OK) return st;
  if (set_up() != cudaSuccess) return TP_ERR_CUDA;
  c->stream = static_cast<cudaStream_t>(stream);
  return entry_timed(name, c->stream, launch_call, c) == cudaSuccess ? TP_OK : TP_ERR_CUDA;
}

size_t gain_bytes(int d) { return static_cast<size_t>(kRoParts) * 8 * d; }

}  // namespace
}  // namespace tp

using namespace tp;

extern "C" tp_status tp_rotary_frequencies(const tp_rotary_scaling* sc, double* freq, float* amplitude) {
  if (sc == nullptr || freq == nullptr || amplitude == nullptr) return TP_ERR_INVALID;
  const int n = sc->n_rot;
  if (n < 2 || n > kRoMaxD || n % 2 != 0 || !(sc->base > 1.0) || !isfinite(sc->base)) return TP_ERR_INVALID;
  if (sc->kind < TP_ROTARY_PLAIN || sc->kind > TP_ROTARY_BY_PAIR) return TP_ERR_INVALID;
  const bool scaled = sc->kind != TP_ROTARY_PLAIN;
  if (scaled && (!(sc->factor >= 1.0) || !isfinite(sc->factor))) return TP_ERR_INVALID;
  const bool parts = sc->kind == TP_ROTARY_BY_TURNS || sc->kind == TP_ROTARY_BY_PAIR;
  if (parts && (!(sc->trained >= 1.0) || !isfinite(sc->trained) || !(sc->low > 0.0) || !(sc->high > sc->low) ||
                !isfinite(sc->high)))
    return TP_ERR_INVALID;
  double base = sc->base;
  if (sc->kind == TP_ROTARY_BASE) {
    if (n < 4) return TP_ERR_INVALID;  // its exponent is n / (n - 2)
    base *= pow(sc->factor, n / (n - 2.0));
    if (!isfinite(base)) return TP_ERR_INVALID;
  }
  *amplitude = 1.f;
  const double two_pi = 6.28318530717958647693;
  double from = 0.0, to = 0.0;
  if (sc->kind == TP_ROTARY_BY_PAIR) {
    auto pair_of = [&](double turns) { return n * log(sc->trained / (turns * two_pi)) / (2.0 * log(base)); };
    from = std::max(floor(pair_of(sc->high)), 0.0);
    to = std::min(ceil(pair_of(sc->low)), n - 1.0);
    *amplitude = static_cast<float>(0.1 * log(sc->factor) + 1.0);
  }
  for (int k = 0; k < n / 2; ++k) {
    const double f = pow(base, -2.0 * k / n);
    double kept = 1.0;  // share that keeps its frequency, the rest is interpolated
    if (sc->kind == TP_ROTARY_LINEAR) kept = 0.0;
    if (sc->kind == TP_ROTARY_BY_TURNS) kept = (sc->trained * f / two_pi - sc->low) / (sc->high - sc->low);
    if (sc->kind == TP_ROTARY_BY_PAIR) kept = 1.0 - (k - from) / std::max(to - from, 1e-3);
    kept = std::min(std::max(kept, 0.0), 1.0);
    freq[k] = scaled && kept < 1.0 ? f * kept + f / sc->factor * (1.0 - kept) : f;
  }
  return TP_OK;
}

extern "C" tp_status tp_rotary_fwd(tp_dtype dt, const tp_attn_config* cfg, const tp_rotary_config* rot,
                                   const int64_t* seq_starts, const int64_t* positions, const void* QKV,
                                   int64_t ld_qkv, void* Out, int64_t ld_out, void* stream) {
  RoCall c;
  clear(&c);
  const tp_status st = ro_args(dt, RO_ROTATE, cfg, rot, nullptr, seq_starts, positions, QKV, ld_qkv, nullptr, 0, Out,
                               ld_out, &c);
  if (st != TP_OK || cfg->T == 0) return st;
  return ro_run("rotary_fwd", &c, stream);
}

extern "C" tp_status tp_rotary_bwd(tp_dtype dt, const tp_attn_config* cfg, const tp_rotary_config* rot,
                                   const int64_t* seq_starts, const int64_t* positions, const void* dOut,
                                   int64_t ld_dout, void* dQKV, int64_t ld_dqkv, void* stream) {
  RoCall c;
  clear(&c);
  const tp_status st = ro_args(dt, RO_ROTATE, cfg, rot, nullptr, seq_starts, positions, dOut, ld_dout, nullptr, 0,
                               dQKV, ld_dqkv, &c);
  if (st != TP_OK || cfg->T == 0) return st;
  c.p.amp_sin = -c.p.amp;
  return ro_run("rotary_bwd", &c, stream);
}

extern "C" tp_status tp_qk_norm_rotary_fwd(tp_dtype dt, const tp_attn_config* cfg, const tp_qk_norm_config* norm,
                                           const tp_rotary_config* rot, const float* gq, const float* gk,
                                           const int64_t* seq_starts, const int64_t* positions, const void* QKV,
                                           int64_t ld_qkv, void* Out, int64_t ld_out, void* stream) {
  RoCall c;
  clear(&c);
  const tp_status st = ro_args(dt, RO_NORM_FWD, cfg, rot, norm, seq_starts, positions, QKV, ld_qkv, nullptr, 0, Out,
                               ld_out, &c);
  if (st != TP_OK || cfg->T == 0) return st;
  if (!aligned(gq, 4) || !aligned(gk, 4)) return TP_ERR_ALIGN;
  c.p.gq = gq;
  c.p.gk = gk;
  return ro_run("qk_norm_rotary_fwd", &c, stream);
}

extern "C" tp_status tp_qk_norm_rotary_bwd(tp_dtype dt, const tp_attn_config* cfg, const tp_qk_norm_config* norm,
                                           const tp_rotary_config* rot, const float* gq, const float* gk,
                                           const int64_t* seq_starts, const int64_t* positions, const void* QKV,
                                           int64_t ld_qkv, const void* dOut, int64_t ld_dout, void* dQKV,
                                           int64_t ld_dqkv, float* dgq, float* dgk, int accumulate, void* workspace,
                                           size_t ws_bytes, void* stream) {
  RoCall c;
  clear(&c);
  const tp_status st = ro_args(dt, RO_NORM_BWD, cfg, rot, norm, seq_starts, positions, QKV, ld_qkv, dOut, ld_dout,
                               dQKV, ld_dqkv, &c);
  if (st != TP_OK) return st;
  if (!aligned(gq, 4) || !aligned(gk, 4) || !aligned(dgq, 4) || !aligned(dgk, 4)) return TP_ERR_ALIGN;
  // (null gradients and null gains are equal, and allowed)
  for (const float* g : {dgq, dgk})
    if (g != nullptr && (g == gq || g == gk)) return TP_ERR_INVALID;
  if (dgq != nullptr && dgq == dgk) return TP_ERR_INVALID;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cfg->T == 0) {
    // no rows: the gains' gradients are zero
    if (accumulate) return TP_OK;
    for (float* g : {dgq, dgk})
      if (g != nullptr && cudaMemsetAsync(g, 0, static_cast<size_t>(cfg->d) * 4, s) != cudaSuccess) return TP_ERR_CUDA;
    return TP_OK;
  }
  if (dgq != nullptr || dgk != nullptr) {
    if (workspace == nullptr || ws_bytes < gain_bytes(cfg->d)) return TP_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return TP_ERR_ALIGN;
    c.p.partial = static_cast<float*>(workspace);
  }
  c.p.gq = gq;
  c.p.gk = gk;
  c.p.amp_sin = -c.p.amp;
  c.p.dgq = dgq;
  c.p.dgk = dgk;
  c.p.accumulate = accumulate;
  return ro_run("qk_norm_rotary_bwd", &c, stream);
}

extern "C" size_t tp_qk_norm_rotary_workspace_size(const tp_attn_config* cfg) {
  if (cfg == nullptr || !head_sizes(cfg) || cfg->T == 0 || cfg->d % 8 != 0) return 0;
  return gain_bytes(cfg->d);
}
