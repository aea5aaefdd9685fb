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
// exact and drops the whole turns by itself, and its upper 32 bits are the
// angle for sincospif.  A position costs one integer product a pair, and far
// ones lose nothing to the range reduction.
//
// Every kernel streams: each value is read once and written once.  A block
// takes a few rows; their cosines and sines are computed once into shared
// memory and used by all heads.  A group of G lanes holds one head, 16 values
// a lane: two vectors whose elements are partners (half layout: a distance of
// n_rot / 2 apart), so that no value crosses lanes but in the norm's sums, and
// a head may be written over itself.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>

#include "tp_device.cuh"
#include "tp_entry.h"
#include "tp_internal.h"

namespace tp {
namespace {

constexpr int kRoThreads = 256;
constexpr int kRoWarps = kRoThreads / 32;
constexpr int kRoRows = 8;       // most rows a block takes at a time
constexpr int kRoMaxD = 512;     // head width
constexpr int kRoPairs = kRoMaxD / 2;
constexpr int kRoParts = 1024;   // most blocks of the backward with gains
constexpr int kRoElems = 16;     // values of a head a lane holds

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
  int64_t T;
  int b, s;        // s: tokens of every sequence (no starts, no positions)
  int d, hq, hk;   // head width; query and key heads a shard
  int hs;          // heads a shard in memory: hq + 2 hk
  int per;         // heads a shard that are visited: hs, or hq + hk where the values stay where they are
  int items;       // visited heads a row
  int pairs;       // rotated pairs a head
  int G;           // lanes a head
  int slots;       // pairs of vectors a head, the last one's second may be missing
  int rot_slots;   // those with rotated elements
  int width;       // cosines a row in shared memory
  int rows;        // rows a block takes at a time
  int back;        // the transposed rotation
  int centred;
  float eps, amp;
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
  if constexpr (V == 1) {
    if constexpr (sizeof(E) == 2) w[0] = *reinterpret_cast<const uint16_t*>(p);
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
  if constexpr (V == 1) {
    if constexpr (sizeof(E) == 2) *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(w[0]);
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
    for (int i = 0; i < V / 2; ++i) unpack_bf16x2(w[i], f[2 * i], f[2 * i + 1]);
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

// Sum over the G lanes of a head (G a power of two); every lane of the warp
// takes part.
__device__ __forceinline__ float group_sum(float v, int G) {
  for (int o = G >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// ---------------------------------------------------------------------------
// Rows
// ---------------------------------------------------------------------------
// Start of the sequence that row t belongs to: the last start that is not
// behind it.  32 starts a step; called by a whole warp.  Any contents of
// `starts` end it in ceil(log32(b)) steps, inside the array.
__device__ __forceinline__ int64_t start_of(const int64_t* starts, int b, int64_t t, int lane) {
  int lo = 0, hi = b;
  int64_t at = 0;
  while (hi > lo) {
    const int step = (hi - lo + 31) / 32;
    const int i = lo + lane * step;
    const int64_t v = i < hi ? __ldcg(starts + i) : INT64_MAX;
    const unsigned below = __ballot_sync(0xffffffffu, v <= t);
    const int last = below ? 31 - __clz(below) : 0;
    at = __shfl_sync(0xffffffffu, v, last);
    lo = lo + last * step;
    hi = min(hi, lo + step);
    if (step == 1) break;
  }
  return at;
}

// Rows of sequences lie in [first, end); reports starts that decrease or leave
// the buffer.
__device__ __forceinline__ void used_rows(const RoParams& p, int64_t& first, int64_t& end) {
  first = 0;
  end = p.T;
  if (p.starts == nullptr) return;
  first = max(__ldcg(p.starts), static_cast<int64_t>(0));
  end = min(__ldcg(p.starts + p.b), p.T);
  bool fine = true;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kRoThreads + threadIdx.x; i < p.b;
       i += static_cast<int64_t>(gridDim.x) * kRoThreads) {
    const int64_t a = __ldcg(p.starts + i), e = __ldcg(p.starts + i + 1);
    fine &= a >= 0 && e >= a && e <= p.T;
  }
  if (!fine) atomicOr(p.err, kErrInvalid);
}

// Positions of the tile's rows, 8 lanes a warp at most.
__device__ __forceinline__ void fill_positions(const RoParams& p, int64_t row0, int n, int64_t first, int64_t end,
                                               int64_t* pos) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int r = warp; r < n; r += kRoWarps) {
    const int64_t t = row0 + r;
    int64_t at;
    if (p.positions != nullptr) at = __ldcg(p.positions + t);
    else if (p.starts != nullptr) at = t - start_of(p.starts, p.b, t, lane);
    else at = t % p.s;
    if (lane == 0) pos[r] = at;
  }
}

// Where the cosine of pair k lies in its row.  Vectors of 8 are read as two
// quads, each quad's lanes side by side.
template <int V>
__device__ __forceinline__ int place(int k, int rot_slots) {
  if constexpr (V == 8) return (((k & 7) >> 2) * rot_slots + (k >> 3)) * 4 + (k & 3);
  else return k;
}

// Cosines and sines of the tile's rows, times the amplitude.
template <int V>
__device__ __forceinline__ void fill_table(const RoParams& p, int n, const int64_t* pos, float* tab) {
  const int w = p.width;
  for (int i = threadIdx.x; i < n * w; i += kRoThreads) {
    const int r = i / w, k = i - r * w;
    float c = 1.f, s = 0.f;
    if (k < p.pairs) {
      const uint64_t turns = static_cast<uint64_t>(pos[r]) * p.turn[k];
      const int32_t half_turns = static_cast<int32_t>((turns + (uint64_t{1} << 31)) >> 32);
      sincospif(static_cast<float>(half_turns) * 0x1p-31f, &s, &c);
      c *= p.amp;
      s *= p.back ? -p.amp : p.amp;
    }
    float* row = tab + static_cast<size_t>(r) * 2 * w + place<V>(k, p.rot_slots);
    row[0] = c;
    row[w] = s;
  }
}

template <int V>
__device__ __forceinline__ void read_table(const float* row, int slot, int rot_slots, float* f) {
  if constexpr (V == 8) {
    const float4 a = reinterpret_cast<const float4*>(row)[slot];
    const float4 b = reinterpret_cast<const float4*>(row)[rot_slots + slot];
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  } else if constexpr (V == 4) {
    const float4 a = reinterpret_cast<const float4*>(row)[slot];
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  } else {
    f[0] = row[slot];
  }
}

// ---------------------------------------------------------------------------
// A lane's part of a head
// ---------------------------------------------------------------------------
// Vectors of slot i: columns a and b of the head; a < 0: none, b < 0: only a.
// Half layout: rotated slots first, their vectors n_rot / 2 apart, then
// what is not rotated, vector after vector.  Interleaved (V = 8): vectors side by
// side.
template <int V, bool INTER>
__device__ __forceinline__ void columns(const RoParams& p, int slot, int& a, int& b) {
  if (slot >= p.slots) {
    a = b = -1;
    return;
  }
  if (INTER) {
    a = 16 * slot;
    b = a + 8;
  } else if (slot < p.rot_slots) {
    a = slot * V;
    b = a + p.pairs;
  } else {
    a = 2 * p.pairs + 2 * (slot - p.rot_slots) * V;
    b = a + V;
  }
  if (b >= p.d) b = -1;
}

template <class E, int V, bool INTER>
struct Lane {
  static constexpr int S = 8 / V;  // slots
  static constexpr int N = Words<E, V>::N;
  static constexpr int kWords = 2 * S * N;
  int a[S], b[S];
  int first;  // the first slot; slot i is first + i G

  __device__ __forceinline__ Lane(const RoParams& p, int lane) : first(lane & (p.G - 1)) {
#pragma unroll
    for (int i = 0; i < S; ++i) columns<V, INTER>(p, first + i * p.G, a[i], b[i]);
  }
  __device__ __forceinline__ void load(const E* head, uint32_t* w) const {
#pragma unroll
    for (int i = 0; i < S; ++i) {
#pragma unroll
      for (int k = 0; k < 2 * N; ++k) w[2 * N * i + k] = 0u;
      if (a[i] >= 0) load_vec<E, V>(head + a[i], w + 2 * N * i);
      if (b[i] >= 0) load_vec<E, V>(head + b[i], w + 2 * N * i + N);
    }
  }
  __device__ __forceinline__ void store(E* head, const uint32_t* w) const {
#pragma unroll
    for (int i = 0; i < S; ++i) {
      if (a[i] >= 0) store_words<E, V>(head + a[i], w + 2 * N * i);
      if (b[i] >= 0) store_words<E, V>(head + b[i], w + 2 * N * i + N);
    }
  }
  // f[2 V i ..]: slot i's vector a, then b
  __device__ __forceinline__ void floats(const uint32_t* w, float* f) const {
#pragma unroll
    for (int i = 0; i < 2 * S; ++i) unpack<E, V>(w + N * i, f + V * i);
  }
  __device__ __forceinline__ void words(const float* f, uint32_t* w) const {
#pragma unroll
    for (int i = 0; i < 2 * S; ++i) pack<E, V>(f + V * i, w + N * i);
  }
  // Rotates the lane's pairs; what is not rotated is not touched.
  __device__ __forceinline__ void turn(const RoParams& p, const float* row, float* f) const {
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const int slot = first + i * p.G;
      if (slot >= p.rot_slots) continue;
      float c[V], s[V];
      read_table<V>(row, slot, p.rot_slots, c);
      read_table<V>(row + p.width, slot, p.rot_slots, s);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const int u = INTER ? 2 * e : 2 * V * i + e, v = INTER ? u + 1 : u + V;
        if (INTER && slot * 8 + e >= p.pairs) continue;
        const float x = f[u], y = f[v];
        f[u] = x * c[e] - y * s[e];
        f[v] = fmaf(x, s[e], y * c[e]);
      }
    }
  }
  // f[j] <- fn(f[j], column) for the columns that the lane has
  template <class F>
  __device__ __forceinline__ void each(F&& fn) const {
#pragma unroll
    for (int i = 0; i < S; ++i) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        if (a[i] >= 0) fn(2 * V * i + e, a[i] + e);
        if (b[i] >= 0) fn(2 * V * i + V + e, b[i] + e);
      }
    }
  }
};

// A group's walk over the tile's (row, head) pairs.
struct Walk {
  int r, h, dr, dh, items;
  __device__ __forceinline__ Walk(int group, int groups, int items_) : items(items_) {
    r = group / items;
    h = group - r * items;
    dr = groups / items;
    dh = groups - dr * items;
  }
  __device__ __forceinline__ void step() {
    r += dr;
    h += dh;
    if (h >= items) {
      h -= items;
      ++r;
    }
  }
};

// Column of visited head h, and what it is: 0 query, 1 key, 2 value.
__device__ __forceinline__ int head_column(const RoParams& p, int h, int& kind) {
  const int shard = h / p.per, at = h - shard * p.per;
  kind = at < p.hq ? 0 : at < p.hq + p.hk ? 1 : 2;
  return (shard * p.hs + at) * p.d;
}

__device__ __forceinline__ void fill_gains(const RoParams& p, float* gains) {
  for (int i = threadIdx.x; i < 2 * p.d; i += kRoThreads) {
    const float* g = i < p.d ? p.gq : p.gk;
    gains[i] = g == nullptr ? 1.f : __ldg(g + (i < p.d ? i : i - p.d));
  }
}

// Mean (0 unless centred) and 1 / sqrt(mean square + eps) of the lane's head;
// x loses the mean.  Sums are fp32.
template <class L>
__device__ __forceinline__ float norm_of(const RoParams& p, const L& lane, float* x) {
  const float inv_d = 1.f / static_cast<float>(p.d);
  if (p.centred) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < kRoElems; ++i) m += x[i];
    m = group_sum(m, p.G) * inv_d;
    lane.each([&](int i, int) { x[i] -= m; });
  }
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < kRoElems; ++i) q = fmaf(x[i], x[i], q);
  return rsqrtf(group_sum(q, p.G) * inv_d + p.eps);
}

// ---------------------------------------------------------------------------
// Rotation, and the norm's forward
// ---------------------------------------------------------------------------
template <class E, int V, bool INTER, bool NORM>
__global__ void __launch_bounds__(kRoThreads) rotary_kernel(const __grid_constant__ RoParams p) {
  extern __shared__ __align__(16) float smem[];
  __shared__ int64_t pos[kRoRows];
  float* tab = smem;
  float* gains = smem + static_cast<size_t>(p.rows) * 2 * p.width;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * p.rows;
  const int n = static_cast<int>(min(static_cast<int64_t>(p.rows), p.T - row0));
  int64_t first, end;
  pdl_wait();
  pdl_trigger();
  used_rows(p, first, end);
  const Lane<E, V, INTER> L(p, threadIdx.x & 31);
  const E* x = static_cast<const E*>(p.x);
  E* out = static_cast<E*>(p.out);
  const int groups = kRoThreads / p.G;
  Walk at(threadIdx.x / p.G, groups, p.items);
  uint32_t next[Lane<E, V, INTER>::kWords];
  int kind = 2, col = 0;
  if (at.r < n) {
    col = head_column(p, at.h, kind);
    L.load(x + (row0 + at.r) * p.ld_x + col, next);
  }
  fill_positions(p, row0, n, first, end, pos);
  if (NORM) fill_gains(p, gains);
  __syncthreads();
  fill_table<V>(p, n, pos, tab);
  __syncthreads();
  const int steps = (n * p.items + groups - 1) / groups;
  for (int i = 0; i < steps; ++i) {
    uint32_t w[Lane<E, V, INTER>::kWords];
#pragma unroll
    for (int k = 0; k < Lane<E, V, INTER>::kWords; ++k) w[k] = next[k];
    const int r = at.r, what = kind;
    const bool mine = r < n;
    const int64_t row = row0 + r;
    E* to = out + row * p.ld_out + col;
    at.step();
    if (at.r < n) {
      col = head_column(p, at.h, kind);
      L.load(x + (row0 + at.r) * p.ld_x + col, next);
    }
    float f[kRoElems];
    L.floats(w, f);
    if (NORM) {
      float v[kRoElems];
#pragma unroll
      for (int k = 0; k < kRoElems; ++k) v[k] = mine ? f[k] : 0.f;
      const float inv = norm_of(p, L, v);
      if (what != 2) {
        const float* g = gains + (what == 1 ? p.d : 0);
        L.each([&](int k, int c) { f[k] = v[k] * inv * g[c]; });
      }
    }
    if (mine && row >= first && row < end) {
      if (what != 2) {
        L.turn(p, tab + static_cast<size_t>(r) * 2 * p.width, f);
        L.words(f, w);
      }
      L.store(to, w);
    }
  }
}

// ---------------------------------------------------------------------------
// The norm's backward
// ---------------------------------------------------------------------------
// Blocks take tiles in turn; every lane sums its columns' part of the gains'
// gradients over all heads it sees, then the block sums its warps' in order.
template <class E, int V, bool INTER>
__global__ void __launch_bounds__(kRoThreads) qk_norm_bwd_kernel(const __grid_constant__ RoParams p) {
  extern __shared__ __align__(16) float smem[];
  __shared__ int64_t pos[kRoRows];
  using LaneT = Lane<E, V, INTER>;
  float* gains = smem;
  float* tab = smem + 2 * p.d;
  pdl_wait();
  pdl_trigger();
  int64_t first, end;
  used_rows(p, first, end);
  fill_gains(p, gains);
  const LaneT L(p, threadIdx.x & 31);
  const E* x = static_cast<const E*>(p.x);
  const E* dy = static_cast<const E*>(p.dy);
  E* out = static_cast<E*>(p.out);
  const int groups = kRoThreads / p.G;
  const float inv_d = 1.f / static_cast<float>(p.d);
  float sum[2][kRoElems];
#pragma unroll
  for (int i = 0; i < kRoElems; ++i) sum[0][i] = sum[1][i] = 0.f;
  for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * p.rows; row0 < p.T;
       row0 += static_cast<int64_t>(gridDim.x) * p.rows) {
    const int n = static_cast<int>(min(static_cast<int64_t>(p.rows), p.T - row0));
    Walk at(threadIdx.x / p.G, groups, p.items);
    uint32_t nx[LaneT::kWords], ny[LaneT::kWords];
    int kind = 2, col = 0;
    auto fetch = [&] {
      if (at.r >= n) return;
      col = head_column(p, at.h, kind);
      if (kind != 2) L.load(x + (row0 + at.r) * p.ld_x + col, nx);
      L.load(dy + (row0 + at.r) * p.ld_dy + col, ny);
    };
    fetch();
    __syncthreads();  // the last tile's table and positions are read
    fill_positions(p, row0, n, first, end, pos);
    __syncthreads();
    fill_table<V>(p, n, pos, tab);
    __syncthreads();
    const int steps = (n * p.items + groups - 1) / groups;
    for (int i = 0; i < steps; ++i) {
      uint32_t wx[LaneT::kWords], wy[LaneT::kWords];
#pragma unroll
      for (int k = 0; k < LaneT::kWords; ++k) wx[k] = nx[k], wy[k] = ny[k];
      const int r = at.r, what = kind;
      const int64_t row = row0 + r;
      const bool mine = r < n && row >= first && row < end;
      const bool turned = mine && what != 2;
      E* to = out + row * p.ld_out + col;
      at.step();
      fetch();
      float v[kRoElems], e[kRoElems];
#pragma unroll
      for (int k = 0; k < LaneT::kWords; ++k) {
        if (!turned) wx[k] = 0u;
      }
      L.floats(wx, v);
      L.floats(wy, e);
      const float inv = norm_of(p, L, v);
      float along = 0.f, mean = 0.f;
      if (turned) {
        L.turn(p, tab + static_cast<size_t>(r) * 2 * p.width, e);
        const float* g = gains + (what == 1 ? p.d : 0);
        L.each([&](int k, int c) {
          v[k] *= inv;
          const float t = e[k] * v[k];
          sum[0][k] += what == 0 ? t : 0.f;
          sum[1][k] += what == 1 ? t : 0.f;
          e[k] *= g[c];
          along = fmaf(e[k], v[k], along);
          mean += e[k];
        });
      }
      along = group_sum(along, p.G) * inv_d;
      mean = p.centred ? group_sum(mean, p.G) * inv_d : 0.f;
      if (turned) {
#pragma unroll
        for (int k = 0; k < kRoElems; ++k) e[k] = inv * (fmaf(-v[k], along, e[k]) - mean);
        L.words(e, wy);
      }
      if (mine) L.store(to, wy);
    }
  }
  if (p.partial == nullptr) return;
  // groups of a warp, then warps
  for (int o = p.G; o < 32; o <<= 1) {
#pragma unroll
    for (int k = 0; k < kRoElems; ++k) {
      sum[0][k] += __shfl_xor_sync(0xffffffffu, sum[0][k], o);
      sum[1][k] += __shfl_xor_sync(0xffffffffu, sum[1][k], o);
    }
  }
  __syncthreads();
  if ((threadIdx.x & 31) < p.G) {
    float* mine = smem + static_cast<size_t>(threadIdx.x >> 5) * 2 * p.d;
    L.each([&](int k, int c) {
      mine[c] = sum[0][k];
      mine[p.d + c] = sum[1][k];
    });
  }
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * p.d; c += kRoThreads) {
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < kRoWarps; ++w) t += smem[static_cast<size_t>(w) * 2 * p.d + c];
    p.partial[static_cast<size_t>(blockIdx.x) * 2 * p.d + c] = t;
  }
}

// The blocks' sums in their order: 32 columns a block, 32 rows at a time.
__global__ void __launch_bounds__(1024) qk_gain_sum_kernel(const float* __restrict__ partial, int parts, int d,
                                                           float* dgq, float* dgk, int accumulate) {
  pdl_wait();
  pdl_trigger();
  __shared__ float red[32][33];
  const int c = blockIdx.x * 32 + threadIdx.x % 32, r = threadIdx.x / 32;
  float t = 0.f;
  if (c < 2 * d)
    for (int i = r; i < parts; i += 32) t += __ldcg(partial + static_cast<size_t>(i) * 2 * d + c);
  red[r][threadIdx.x % 32] = t;
  __syncthreads();
  if (r != 0 || c >= 2 * d) return;
  for (int i = 1; i < 32; ++i) t += red[i][threadIdx.x];
  float* to = c < d ? dgq : dgk;
  if (to == nullptr) return;
  to += c < d ? c : c - d;
  *to = accumulate ? *to + t : t;
}

// ---------------------------------------------------------------------------
// Launches
// ---------------------------------------------------------------------------
struct RoCall {
  RoParams p;
  RoMode mode;
  bool f32, inter;
  int vec, num_sms, accumulate;
  float *dgq, *dgk;
  cudaStream_t stream;
};

template <class E, int V, bool INTER>
cudaError_t launch_as(const RoCall& c) {
  RoParams p = c.p;
  const size_t row_bytes = static_cast<size_t>(2) * p.width * 4;
  if (c.mode != RO_NORM_BWD) {
    p.rows = static_cast<int>(std::min<int64_t>(kRoRows, std::max<int64_t>(1, p.T / (8 * c.num_sms))));
    const unsigned grid = static_cast<unsigned>((p.T + p.rows - 1) / p.rows);
    const size_t smem = p.rows * row_bytes + (c.mode == RO_NORM_FWD ? 8 * p.d : 0);
    count_launches(1);
    return c.mode == RO_NORM_FWD ? launch_k(rotary_kernel<E, V, INTER, true>, grid, kRoThreads, smem, c.stream, p)
                                 : launch_k(rotary_kernel<E, V, INTER, false>, grid, kRoThreads, smem, c.stream, p);
  }
  p.rows = static_cast<int>(std::min<int64_t>(4, std::max<int64_t>(1, p.T / (8 * c.num_sms))));
  const unsigned grid = static_cast<unsigned>(
      std::min<int64_t>((p.T + p.rows - 1) / p.rows, std::min(kRoParts, 4 * c.num_sms)));
  const size_t smem = std::max(8 * static_cast<size_t>(p.d) + p.rows * row_bytes,
                               p.partial ? static_cast<size_t>(kRoWarps) * 8 * p.d : 0);
  count_launches(1);
  cudaError_t e = launch_k(qk_norm_bwd_kernel<E, V, INTER>, grid, kRoThreads, smem, c.stream, p);
  if (e != cudaSuccess || p.partial == nullptr) return e;
  count_launches(1);
  return launch_k(qk_gain_sum_kernel, (2 * p.d + 31) / 32, 1024, 0, c.stream, static_cast<const float*>(p.partial),
                  static_cast<int>(grid), p.d, c.dgq, c.dgk, c.accumulate);
}

template <class E>
cudaError_t launch_typed(const RoCall& c) {
  if (c.inter) return launch_as<E, 8, true>(c);
  if (c.vec == 8) return launch_as<E, 8, false>(c);
  if (c.vec == 4) return launch_as<E, 4, false>(c);
  return launch_as<E, 1, false>(c);
}

cudaError_t launch_call(void* call) {
  const RoCall& c = *static_cast<const RoCall*>(call);
  return c.f32 ? launch_typed<float>(c) : launch_typed<__nv_bfloat16>(c);
}

// ---------------------------------------------------------------------------
// Arguments
// ---------------------------------------------------------------------------
inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Turns a position as a 64-bit fraction.
uint64_t turn_fraction(double freq) {
  const double turns = fmod(freq * 0.15915494309189533577, 1.0);  // 1 / 2 pi
  return static_cast<uint64_t>(turns * 0x1p64);                   // 0 <= turns < 1
}

// Sizes and the rotation into c, without pointers.
tp_status ro_sizes(const tp_attn_config* cfg, const tp_rotary_config* rot, bool norm, const int64_t* seq_starts,
                   const int64_t* positions, RoCall* c) {
  if (cfg == nullptr || (rot == nullptr && !norm)) return TP_ERR_INVALID;
  if (cfg->T < 0 || cfg->T > INT32_MAX - 511 || cfg->n_heads < 1 || cfg->n_kv_heads < 1 || cfg->N < 1 || cfg->N > 8 ||
      cfg->n_heads % cfg->N != 0 || cfg->n_kv_heads % cfg->N != 0 || cfg->n_heads % cfg->n_kv_heads != 0 ||
      cfg->d < 1 || cfg->d > kRoMaxD)
    return TP_ERR_INVALID;
  if ((static_cast<int64_t>(cfg->n_heads) + 2 * static_cast<int64_t>(cfg->n_kv_heads)) * cfg->d > INT32_MAX / kRoRows)
    return TP_ERR_INVALID;
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
  c->inter = n_rot > 0 && rot->interleaved != 0;
  // Partners in the half layout lie n_rot / 2 apart: the widest vectors that
  // keep both ends of a pair aligned.
  c->vec = c->inter || p.pairs % 8 == 0 ? 8 : p.pairs % 4 == 0 ? 4 : 1;
  const int v = c->vec;
  p.rot_slots = (p.pairs + v - 1) / v;
  p.slots = c->inter ? (p.d + 15) / 16 : p.rot_slots + ((p.d - n_rot) / v + 1) / 2;
  p.width = p.rot_slots * v;
  const int lanes = (p.slots + 8 / v - 1) / (8 / v);
  p.G = 1;
  while (p.G < lanes) p.G <<= 1;
  return TP_OK;
}

// What every call checks and fills in.
tp_status ro_args(tp_dtype dt, RoMode mode, const tp_attn_config* cfg, const tp_rotary_config* rot,
                  const tp_qk_norm_config* norm, const int64_t* seq_starts, const int64_t* positions, const void* x,
                  int64_t ld_x, const void* dy, int64_t ld_dy, void* out, int64_t ld_out, RoCall* c) {
  if (dt != TP_F32 && dt != TP_BF16) return TP_ERR_UNSUPPORTED;
  const bool with_norm = mode != RO_ROTATE;
  if (with_norm && norm == nullptr) return TP_ERR_INVALID;
  tp_status st = ro_sizes(cfg, rot, with_norm, seq_starts, positions, c);
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
  p.per = out == src ? p.hq + p.hk : p.hs;
  p.items = p.per * cfg->N;
  p.centred = with_norm && norm->kind == TP_NORM_LAYER;
  p.eps = with_norm ? norm->eps : 0.f;
  c->mode = mode;
  c->f32 = dt == TP_F32;
  return TP_OK;
}

tp_status ro_run(const char* name, RoCall* c, void* stream) {
  const tp_status st = entry_device(&c->num_sms, &c->p.err);
  if (st != TP_OK) return st;
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
  memset(&c, 0, sizeof(c));
  const tp_status st = ro_args(dt, RO_ROTATE, cfg, rot, nullptr, seq_starts, positions, QKV, ld_qkv, nullptr, 0, Out,
                               ld_out, &c);
  if (st != TP_OK || cfg->T == 0) return st;
  return ro_run("rotary_fwd", &c, stream);
}

extern "C" tp_status tp_rotary_bwd(tp_dtype dt, const tp_attn_config* cfg, const tp_rotary_config* rot,
                                   const int64_t* seq_starts, const int64_t* positions, const void* dOut,
                                   int64_t ld_dout, void* dQKV, int64_t ld_dqkv, void* stream) {
  RoCall c;
  memset(&c, 0, sizeof(c));
  const tp_status st = ro_args(dt, RO_ROTATE, cfg, rot, nullptr, seq_starts, positions, dOut, ld_dout, nullptr, 0,
                               dQKV, ld_dqkv, &c);
  if (st != TP_OK || cfg->T == 0) return st;
  c.p.back = 1;
  return ro_run("rotary_bwd", &c, stream);
}

extern "C" tp_status tp_qk_norm_rotary_fwd(tp_dtype dt, const tp_attn_config* cfg, const tp_qk_norm_config* norm,
                                           const tp_rotary_config* rot, const float* gq, const float* gk,
                                           const int64_t* seq_starts, const int64_t* positions, const void* QKV,
                                           int64_t ld_qkv, void* Out, int64_t ld_out, void* stream) {
  RoCall c;
  memset(&c, 0, sizeof(c));
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
  memset(&c, 0, sizeof(c));
  const tp_status st = ro_args(dt, RO_NORM_BWD, cfg, rot, norm, seq_starts, positions, QKV, ld_qkv, dOut, ld_dout,
                               dQKV, ld_dqkv, &c);
  if (st != TP_OK) return st;
  if (!aligned(gq, 4) || !aligned(gk, 4) || !aligned(dgq, 4) || !aligned(dgk, 4)) return TP_ERR_ALIGN;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cfg->T == 0) {
    // no rows: the gains' gradients are zero
    if (accumulate) return TP_OK;
    for (float* g : {dgq, dgk})
      if (g != nullptr && cudaMemsetAsync(g, 0, static_cast<size_t>(cfg->d) * 4, s) != cudaSuccess) return TP_ERR_CUDA;
    return TP_OK;
  }
  if (dgq != nullptr || dgk != nullptr) {
    // (null gradients and null gains are equal, and allowed)
    for (const float* g : {dgq, dgk})
      if (g != nullptr && (g == gq || g == gk)) return TP_ERR_INVALID;
    if (dgq == dgk) return TP_ERR_INVALID;
    if (workspace == nullptr || ws_bytes < gain_bytes(cfg->d)) return TP_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return TP_ERR_ALIGN;
    c.p.partial = static_cast<float*>(workspace);
  }
  c.p.gq = gq;
  c.p.gk = gk;
  c.p.back = 1;
  c.dgq = dgq;
  c.dgk = dgk;
  c.accumulate = accumulate;
  return ro_run("qk_norm_rotary_bwd", &c, stream);
}

extern "C" size_t tp_qk_norm_rotary_workspace_size(const tp_attn_config* cfg) {
  if (cfg == nullptr || cfg->T < 1 || cfg->d < 8 || cfg->d > kRoMaxD || cfg->d % 8 != 0) return 0;
  return gain_bytes(cfg->d);
}
