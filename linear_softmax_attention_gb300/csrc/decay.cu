// Causal linear attention with a decay per head on the CUDA cores: fp32, and bf16
// shapes that the tensor-core path does not take; the scan over segments and the
// one-token step.  decay.cuh has the form that every pass follows.
//
// Bound by the latencies of a pass's steps (loads, weights, rows, state, a barrier
// after each) with two CTAs on an SM: 65 % of shared memory's rate and 40 % of the
// multiplies' are in use.  Of the causal halves only the 16 x 16 blocks that rows see
// are formed.  (8 x 4 of a product in a thread, with the terms split among groups of
// warps, needs a quarter fewer reads, but another barrier: 355 us instead of 337.)
// Measured (one GB300): 8 x 8 x 4096 x 64 fp32 337 us; 1 x 16 x 8192 x 128 441 us; 3 x 5
// x 1777 x 40 42 us; backward 2 x 4 x 2048 x 64 68 us.  (mma.sync on two tf32 parts of
// every factor took 299, 469, 37 and 60 us, but its sums are cut off: errors of
// 1.1e-6 of the outputs against 3e-7.)
#include <algorithm>
#include <type_traits>

#include "decay.cuh"

namespace favor {
namespace {

constexpr int kC = 64;               // tokens of a chunk
constexpr int kThreads = 256;        // 16 x 16
constexpr int kPS = kC + 4;          // row of the weights tile

// ---- tiles in shared memory -----------------------------------------------------
template <int DP> struct Tile {
  static constexpr int S = DP + 4;   // row: 16-byte pieces of neighbouring rows fall on other banks
};

// Rows [0, n) of a head from p on, on their way to a tile: every thread's loads are
// issued together, then stored; zeros behind the rows and the d channels.
// In 16-byte pieces (PIECE 16), else one by one.
template <typename T, int DP, int PIECE> struct Fetch {
  static constexpr int E = PIECE / (int)sizeof(T), kPer = (DP + E - 1) / E, N = (kC * kPer + kThreads - 1) / kThreads;
  using Raw = typename std::conditional<PIECE == 16, uint4, T>::type;
  Raw raw[N];
  __device__ __forceinline__ void issue(const T* p, int64_t ls, int n, int d) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = threadIdx.x + i * kThreads, r = e / kPer, c = (e - r * kPer) * E;
      raw[i] = r < n && c < d ? *reinterpret_cast<const Raw*>(p + r * ls + c) : Raw{};
    }
  }
  // returns whether this thread met infinities or NaN
  __device__ __forceinline__ bool store(float* tile) const {
    constexpr int S = Tile<DP>::S;
    float odd = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = threadIdx.x + i * kThreads, r = e / kPer, c = (e - r * kPer) * E;
      if (kC * kPer % kThreads != 0 && r >= kC) break;
      float f[E];
      if constexpr (PIECE != 16) {
        f[0] = to_f32(raw[i]);
        tile[r * S + c] = f[0];
      } else {
        const unsigned w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
        if constexpr (sizeof(T) == 4) {
#pragma unroll
          for (int k = 0; k < 4; ++k) f[k] = __uint_as_float(w[k]);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            f[2 * k] = __uint_as_float(w[k] << 16);
            f[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
          }
        }
#pragma unroll
        for (int k = 0; k < E; k += 4)
          *reinterpret_cast<float4*>(tile + r * S + c + k) = make_float4(f[k], f[k + 1], f[k + 2], f[k + 3]);
      }
#pragma unroll
      for (int k = 0; k < E; ++k) odd = fmaf(f[k], 0.f, odd);
    }
    return odd != 0.f;               // infinities and NaN make it NaN
  }
};

// X tiles side by side, their loads in flight together (one by one where single
// elements would take too many registers); whether the last one has infinities or NaN
template <typename T, int DP, int X>
__device__ __forceinline__ bool load_tiles(float* tiles, const T* const (&p)[X], const int64_t (&ls)[X], int n, int d,
                                           int piece) {
  constexpr int kTile = kC * Tile<DP>::S;
  bool odd = false;
  if (piece == 16) {
    Fetch<T, DP, 16> f[X];
#pragma unroll
    for (int x = 0; x < X; ++x) f[x].issue(p[x], ls[x], n, d);
#pragma unroll
    for (int x = 0; x < X; ++x) odd = f[x].store(tiles + x * kTile);
  } else {
#pragma unroll
    for (int x = 0; x < X; ++x) {
      Fetch<T, DP, (int)sizeof(T)> f;
      f.issue(p[x], ls[x], n, d);
      odd = f.store(tiles + x * kTile);
    }
  }
  return odd;
}

// The columns of a thread: V side by side, 16 V apart
template <int DP> struct Cols {
  static constexpr int N = DP / 16, V = N < 4 ? N : 4;
  static __device__ __forceinline__ int at(int j) { return (threadIdx.x & 15) * V + (j / V) * 16 * V + j % V; }
  static __device__ __forceinline__ int row(int i) { return (threadIdx.x >> 4) * V + (i / V) * 16 * V + i % V; }
};
template <int V> __device__ __forceinline__ void load_v(float* f, const float* p) {
  if constexpr (V == 4) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    f[0] = v.x;
    f[1] = v.y;
    f[2] = v.z;
    f[3] = v.w;
  } else if constexpr (V == 2) {
    const float2 v = *reinterpret_cast<const float2*>(p);
    f[0] = v.x;
    f[1] = v.y;
  } else {
    f[0] = *p;
  }
}

template <int V> __device__ __forceinline__ void store_v(float* p, const float (&f)[V]) {
  if constexpr (V == 4) *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  else *p = f[0];
}

__device__ __forceinline__ float2 twice(float x) { return make_float2(x, x); }
// columns two by two (one by one where a thread has a single one)
template <int N> struct Acc {
  float2 v[N > 1 ? N / 2 : 1];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int j = 0; j < (N > 1 ? N / 2 : 1); ++j) v[j] = twice(0.f);
  }
  __device__ __forceinline__ void add(float x, const float (&y)[N]) {
    if constexpr (N == 1) {
      v[0].x = fmaf(x, y[0], v[0].x);
    } else {
#pragma unroll
      for (int j = 0; j < N / 2; ++j) v[j] = fma2(twice(x), make_float2(y[2 * j], y[2 * j + 1]), v[j]);
    }
  }
  __device__ __forceinline__ float operator[](int j) const { return j & 1 ? v[j / 2].y : v[j / 2].x; }
  __device__ __forceinline__ void scale(float x) {
#pragma unroll
    for (int j = 0; j < (N > 1 ? N / 2 : 1); ++j) v[j] = mul2(v[j], twice(x));
  }
};

// acc[row][col] += sum_k X[row][k] Y[k][col], rows 16 apart, over k < K (a
// multiple of 4; what lies between d and it is 0).  SEES: X are weights [64][64]: of
// 16 x 16 blocks only those that the rows see; GUARD: of them only the terms.
template <int DP, bool SEES, bool GUARD>
__device__ __forceinline__ void rows_times(Acc<DP / 16> (&acc)[4], const float* X, int xs, const float* Y, int ys,
                                           int K, bool rev) {
  using C = Cols<DP>;
  const int r0 = threadIdx.x >> 4;
#pragma unroll 2
  for (int k = 0; k < K; k += 4) {
    float x[4][4];
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (!SEES || (rev ? k / 16 >= r : k / 16 <= r)) load_v<4>(x[r], X + (r0 + 16 * r) * xs + k);
    float y[4][C::N];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < C::N; j += C::V) load_v<C::V>(y[i] + j, Y + (k + i) * ys + C::at(j));
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if (SEES && (rev ? k / 16 < r : k / 16 > r)) continue;     // the same for all threads
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool sees = !GUARD || (rev ? k + i >= r0 + 16 * r : k + i <= r0 + 16 * r);
        if (sees) acc[r].add(x[r][i], y[i]);
      }
    }
  }
}

// m[i][j] += sum_t w[t] B[t][row i] C[t][col j] over t < n
template <int DP>
__device__ __forceinline__ void gain_times(Acc<DP / 16> (&m)[DP / 16], const float* B, const float* Cc,
                                           const float* w, int n) {
  using C = Cols<DP>;
  constexpr int S = Tile<DP>::S;
#pragma unroll 2
  for (int t = 0; t < n; ++t) {
    float b[C::N], c[C::N];
    const float u = w[t];
#pragma unroll
    for (int j = 0; j < C::N; j += C::V) {
      load_v<C::V>(b + j, B + t * S + C::row(j));
      load_v<C::V>(c + j, Cc + t * S + C::at(j));
    }
#pragma unroll
    for (int i = 0; i < C::N; ++i) m[i].add(b[i] * u, c);
  }
}

struct PassSet {
  DecayPass pass[3];
};

// One segment of one head: chunk by chunk, the state M in shared memory.
// blockIdx.y: which of the passes beside one another.
template <typename T, int DP>
__global__ void __launch_bounds__(kThreads, DP <= 64 ? 2 : 1)
    decay_pass_kernel(const __grid_constant__ PassSet set, const __grid_constant__ DecayShape s, int piece) {
  using C = Cols<DP>;
  constexpr int S = Tile<DP>::S, MS = DP + 4;
  extern __shared__ __align__(16) float sm[];
  float *A = sm, *Bt = A + kC * S, *Ct = Bt + kC * S, *P = Ct + kC * S, *M = P + kC * kPS;
  __shared__ float fade[kC + 1], u[kC];      // l^0 .. l^64; the gains' weights
  const DecayPass& p = set.pass[blockIdx.y];
  const int bh = blockIdx.x / s.segs, seg = blockIdx.x - bh * s.segs, b = bh / s.H, h = bh - b * s.H;
  const float g2 = s.g[h] * kLog2e;
  const int len = decay_length(s, b);
  const int first = seg * s.seg_tokens;
  const int end = min(first + s.seg_tokens, s.L), stop = min(end, len);     // rows to write, tokens
  const int d = s.d, K = (d + 3) / 4 * 4;
  const bool rev = p.rev;
  const T* a0 = static_cast<const T*>(p.a) + b * p.as.b + h * p.as.h;
  const T* b0 = static_cast<const T*>(p.b) + b * p.bs.b + h * p.bs.h;
  const T* c0 = static_cast<const T*>(p.c) + b * p.cs.b + h * p.cs.h;
  T* o0 = static_cast<T*>(p.o) + b * p.os.b + h * p.os.h;
  const float* start = p.start == nullptr ? nullptr : p.start + ((int64_t)bh * s.segs + seg) * d * d;
  constexpr int kAhead = DP * DP / kThreads < 16 ? DP * DP / kThreads : 16;
#pragma unroll 1
  for (int e0 = threadIdx.x; e0 < DP * DP; e0 += kAhead * kThreads) {
    float v[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int e = e0 + i * kThreads, x = e / DP, y = e - x * DP;
      v[i] = start != nullptr && x < d && y < d ? start[x * d + y] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int e = e0 + i * kThreads, x = e / DP, y = e - x * DP;
      M[p.transposed ? y * MS + x : x * MS + y] = v[i];
    }
  }
  if (threadIdx.x <= kC) fade[threadIdx.x] = decay_power(g2, threadIdx.x);
  const int chunks = stop > first ? (stop - first + kC - 1) / kC : 0;
  const int r0 = threadIdx.x >> 4;
#pragma unroll 1
  for (int i = 0; i < chunks; ++i) {
    const int t0 = first + (rev ? chunks - 1 - i : i) * kC;
    const int n = min(kC, stop - t0);
    __syncthreads();                          // the tiles of the chunk before are read
    const T* const from[3] = {a0 + (int64_t)t0 * p.as.l, b0 + (int64_t)t0 * p.bs.l, c0 + (int64_t)t0 * p.cs.l};
    const int64_t ls[3] = {p.as.l, p.bs.l, p.cs.l};
    const bool odd = load_tiles<T, DP, 3>(A, from, ls, n, d, piece);
    if (threadIdx.x < kC) u[threadIdx.x] = threadIdx.x < n ? p.s_u * fade[rev ? threadIdx.x + 1 : n - 1 - threadIdx.x] : 0.f;
    // infinities and NaN of rows that a token may not see would meet its zero weights
    const bool guard = __syncthreads_or(odd);
    // weights, in the 16 x 16 blocks that rows see
    {
      float2 acc[4][4] = {};
#pragma unroll 2
      for (int k = 0; k < K; k += 4) {
        float x[4][4], y[4][4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          load_v<4>(x[r], A + (r0 + 16 * r) * S + k);
          load_v<4>(y[r], Bt + ((threadIdx.x & 15) + 16 * r) * S + k);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            if (r != c && rev != (c > r)) continue;
            acc[r][c] = fma2(make_float2(x[r][0], x[r][1]), make_float2(y[c][0], y[c][1]), acc[r][c]);
            acc[r][c] = fma2(make_float2(x[r][2], x[r][3]), make_float2(y[c][2], y[c][3]), acc[r][c]);
          }
      }
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int row = r0 + 16 * r, col = (threadIdx.x & 15) + 16 * c;
          const int apart = rev ? col - row : row - col;
          P[row * kPS + col] = apart >= 0 && col < n ? p.s_w * fade[apart] * (acc[r][c].x + acc[r][c].y) : 0.f;
        }
    }
    __syncthreads();
    Acc<C::N> acc[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) acc[r].clear();
    rows_times<DP, false, false>(acc, A, S, M, MS, K, false);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = r0 + 16 * r;
      acc[r].scale(row < n ? p.s_r * fade[rev ? n - 1 - row : row + 1] : 0.f);
    }
    if (guard) rows_times<DP, true, true>(acc, P, kPS, Ct, S, kC, rev);
    else rows_times<DP, true, false>(acc, P, kPS, Ct, S, kC, rev);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = r0 + 16 * r;
      T* o = o0 + (int64_t)(t0 + row) * p.os.l;
      if (row < n)
#pragma unroll
        for (int j = 0; j < C::N; ++j)
          if (C::at(j) < d) o[C::at(j)] = from_f32<T>(acc[r][j]);
    }
    if (i + 1 == chunks && p.last == nullptr) break;
    __syncthreads();                          // M is read
    Acc<C::N> m[C::N];
    const float all = fade[n];
#pragma unroll
    for (int x = 0; x < C::N; ++x) {
      float v[C::N];
#pragma unroll
      for (int y = 0; y < C::N; y += C::V) load_v<C::V>(v + y, M + C::row(x) * MS + C::at(y));
      m[x].clear();
      m[x].add(all, v);
    }
    gain_times<DP>(m, Bt, Ct, u, n);
#pragma unroll
    for (int x = 0; x < C::N; ++x)
#pragma unroll
      for (int y = 0; y < C::N; ++y) M[C::row(x) * MS + C::at(y)] = m[x][y];
  }
  // rows behind the sequence's end
  const int from = max(stop, first);
  for (int64_t e = threadIdx.x; e < (int64_t)(end - from) * d; e += kThreads) {
    const int r = (int)(e / d), c = (int)(e - (int64_t)r * d);
    o0[(int64_t)(from + r) * p.os.l + c] = from_f32<T>(0.f);
  }
  if (p.last != nullptr) {
    __syncthreads();
    float* last = p.last + (int64_t)bh * d * d;
    // a reversed pass ends with the gradient of the state before its first token
    for (int e = threadIdx.x; e < d * d; e += kThreads) {
      const int x = e / d, y = e - x * d;
      last[e] = p.transposed ? M[y * MS + x] : M[x * MS + y];
    }
  }
}

struct Gains {
  DecayGain kind[2];
};

// The gain of one segment, in registers; block (segment, head, kind).  Shared memory
// returns 128 bytes a cycle, whatever lanes share: a thread holds 8 x 8 of the product
// where there are so many, and groups of threads take the chunk's tokens in turn; their
// sums are added at the end, in order.  3 x 5 x 1777 x 40, under the profiler: 13 us,
// with 4 x 4 of all tokens 20.
template <int DP> struct GainTile {
  static constexpr int N = DP >= 64 ? 8 : DP / 8, V = N < 4 ? N : 4;
  static constexpr int kSide = DP / N, kGroup = kSide * kSide, kGroups = kThreads / kGroup;
  static __device__ __forceinline__ int at(int place, int j) { return place * V + (j / V) * kSide * V + j % V; }
};
template <typename T, int DP>
__global__ void __launch_bounds__(kThreads, DP <= 64 ? 2 : 1) decay_gain_kernel(Gains gains, DecayShape s, int piece) {
  using G = GainTile<DP>;
  constexpr int S = Tile<DP>::S, N = G::N;
  extern __shared__ __align__(16) float sm[];
  float *Bt = sm, *Ct = Bt + kC * S;
  __shared__ float u[kC];
  const DecayGain& p = gains.kind[blockIdx.z];
  const int bh = blockIdx.x / s.segs, seg = blockIdx.x - bh * s.segs, b = bh / s.H, h = bh - b * s.H, d = s.d;
  const float g2 = s.g[h] * kLog2e;
  const int first = seg * s.seg_tokens, stop = min(min(first + s.seg_tokens, s.L), decay_length(s, b));
  const T* b0 = static_cast<const T*>(p.b) + b * p.bs.b + h * p.bs.h;
  const T* c0 = static_cast<const T*>(p.c) + b * p.cs.b + h * p.cs.h;
  const int group = threadIdx.x / G::kGroup, ty = threadIdx.x % G::kGroup / G::kSide, tx = threadIdx.x % G::kSide;
  Acc<N> m[N];
#pragma unroll
  for (int x = 0; x < N; ++x) m[x].clear();
#pragma unroll 1
  for (int t0 = first; t0 < stop; t0 += kC) {
    const int n = min(kC, stop - t0);
    __syncthreads();
    const T* const from[2] = {b0 + (int64_t)t0 * p.bs.l, c0 + (int64_t)t0 * p.cs.l};
    const int64_t ls[2] = {p.bs.l, p.cs.l};
    load_tiles<T, DP, 2>(Bt, from, ls, n, d, piece);
    if (threadIdx.x < n) {
      const int t = t0 + threadIdx.x;
      u[threadIdx.x] = p.s_u * decay_power(g2, p.rev ? t - first + 1 : stop - 1 - t);
    }
    __syncthreads();
#pragma unroll 2
    for (int t = group; t < n; t += G::kGroups) {
      float bv[N], cv[N];
      const float w = u[t];
#pragma unroll
      for (int j = 0; j < N; j += G::V) {
        load_v<G::V>(bv + j, Bt + t * S + G::at(ty, j));
        load_v<G::V>(cv + j, Ct + t * S + G::at(tx, j));
      }
#pragma unroll
      for (int i = 0; i < N; ++i) m[i].add(bv[i] * w, cv);
    }
  }
  float* out = p.out + ((int64_t)bh * s.segs + seg) * d * d;
  // the groups' sums one after another, in the tiles' place
#pragma unroll 1
  for (int k = 1; k < G::kGroups; ++k) {
    __syncthreads();
    if (group == k)
#pragma unroll
      for (int x = 0; x < N; ++x)
#pragma unroll
        for (int y = 0; y < N; ++y) sm[(x * N + y) * G::kGroup + threadIdx.x % G::kGroup] = m[x][y];
    __syncthreads();
    if (group == 0)
#pragma unroll
      for (int x = 0; x < N; ++x) {
        float v[N];
#pragma unroll
        for (int y = 0; y < N; ++y) v[y] = sm[(x * N + y) * G::kGroup + threadIdx.x];
        m[x].add(1.f, v);
      }
  }
  if (group == 0)
#pragma unroll
    for (int x = 0; x < N; ++x)
#pragma unroll
      for (int y = 0; y < N; ++y)
        if (G::at(ty, x) < d && G::at(tx, y) < d) out[G::at(ty, x) * d + G::at(tx, y)] = m[x][y];
}

struct Scans {
  DecayScan kind[2];
};

// A thread takes V neighbouring elements of a head's state through its segments,
// AHEAD segments' gains in flight.
template <int V, int AHEAD>
__global__ void __launch_bounds__(kThreads) decay_scan_kernel(Scans scans, DecayShape s, int blocks) {
  // the passes may take their places and wait
  asm volatile("griddepcontrol.launch_dependents;");
  const DecayScan& p = scans.kind[blockIdx.z];
  const int dd = s.d * s.d;
  const int bh = blockIdx.x / blocks, b = bh / s.H, h = bh - b * s.H;
  const int e = ((blockIdx.x - bh * blocks) * kThreads + threadIdx.x) * V;
  if (e >= dd) return;
  const int64_t step = (int64_t)dd * p.pieces;
  float* st = p.states + (int64_t)bh * s.segs * step + e;
  const float g2 = s.g[h] * kLog2e;
  const int len = decay_length(s, b);
  const float whole = decay_power(g2, s.seg_tokens);
  tc::griddep_wait();
  float m[V];
#pragma unroll
  for (int v = 0; v < V; ++v) m[v] = 0.f;
  if (p.first != nullptr) load_v<V>(m, p.first + (int64_t)bh * dd + e);
  for (int i0 = 0; i0 < s.segs; i0 += AHEAD) {
    float gain[AHEAD][2][V];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      const int i = i0 + j, seg = p.rev ? s.segs - 1 - i : i;
      if (i < s.segs) {
        load_v<V>(gain[j][0], st + seg * step);
        if (p.pieces > 1) load_v<V>(gain[j][1], st + seg * step + dd);
      }
    }
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      const int i = i0 + j, seg = p.rev ? s.segs - 1 - i : i;
      if (i >= s.segs) break;
      if constexpr (V == 4) *reinterpret_cast<float4*>(st + seg * step) = make_float4(m[0], m[1], m[2], m[3]);
      else st[seg * step] = m[0];
      const int n = min(max(len - seg * s.seg_tokens, 0), s.seg_tokens);
      if (n == 0) continue;
      const float all = n == s.seg_tokens ? whole : decay_power(g2, n);
#pragma unroll
      for (int v = 0; v < V; ++v)
        m[v] = fmaf(all, m[v], p.pieces > 1 ? gain[j][0][v] + gain[j][1][v] : gain[j][0][v]);
    }
  }
  if (p.last != nullptr) {
    float* last = p.last + (int64_t)bh * dd + e;
#pragma unroll
    for (int v = 0; v < V; ++v) last[v] = m[v];
  }
}

// One token of one sequence and head.  Bound by memory: the state is read and
// written once.  A row of the state belongs to d / V neighbouring lanes; each
// thread keeps V columns' part of o, which are added through shared memory.  256 x
// 8 x 64: 14.0 us, 4.8 TB/s (element by element 17.8), 256 x 8 x 128: 43.5 us, 6.2 TB/s.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads) decay_step_kernel(DecayStep p) {
  __shared__ float qs[kDecayMaxD], ks[kDecayMaxD], part[kThreads * V];
  const int bh = blockIdx.x, b = bh / p.H, h = bh - b * p.H, d = p.d;
  const T* q = static_cast<const T*>(p.q) + b * p.qs[0] + h * p.qs[1];
  const T* k = static_cast<const T*>(p.k) + b * p.ks[0] + h * p.ks[1];
  const T* v = static_cast<const T*>(p.v) + b * p.vs[0] + h * p.vs[1];
  const float l = exp2f(p.g[h] * kLog2e);
  const float* s = p.state + (int64_t)bh * d * d;
  float* next = p.next + (int64_t)bh * d * d;
  const int per = d / V, rows = kThreads / per;       // lanes of a row, rows at once
  const int r0 = threadIdx.x / per, c = (threadIdx.x - r0 * per) * V;
  const bool in = r0 < rows;
  if (threadIdx.x < d) {
    qs[threadIdx.x] = to_f32(q[threadIdx.x]);
    ks[threadIdx.x] = to_f32(k[threadIdx.x]);
  }
  float vc[V], o[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    vc[i] = in ? to_f32(v[c + i]) : 0.f;
    o[i] = 0.f;
  }
  __syncthreads();
  if (in) {
    constexpr int kAhead = 8 / V > 4 ? 8 / V : 4;
    for (int x0 = r0; x0 < d; x0 += kAhead * rows) {
      float m[kAhead][V];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int x = x0 + j * rows;
        if (x < d) load_v<V>(m[j], s + x * d + c);
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int x = x0 + j * rows;
        if (x < d) {
#pragma unroll
          for (int i = 0; i < V; ++i) {
            m[j][i] = fmaf(l, m[j][i], ks[x] * vc[i]);
            o[i] = fmaf(qs[x], m[j][i], o[i]);
          }
          if constexpr (V == 4) *reinterpret_cast<float4*>(next + x * d + c) = make_float4(m[j][0], m[j][1], m[j][2], m[j][3]);
          else next[x * d + c] = m[j][0];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) part[r0 * d + c + i] = o[i];
  }
  __syncthreads();
  if (threadIdx.x < d) {
    float sum = 0.f;
    for (int r = 0; r < rows; ++r) sum += part[r * d + threadIdx.x];
    T* out = static_cast<T*>(p.o) + b * p.os[0] + h * p.os[1];
    out[threadIdx.x] = from_f32<T>(p.scale * sum);
  }
}

// A few tokens of one sequence and head, each state read and written once, as by the
// step; the tokens meet one another through weights (o's form over one chunk).  A
// thread keeps its elements of the state, NR rows of V columns, in registers: one read
// of q and k in shared memory goes to V of them.  Bound by memory for a token or two
// (1024 heads of 128: 34 us, floor 20), then by the tokens: about 0.5 us each with two
// CTAs on an SM.
template <typename T, int V, int NR>
__global__ void __launch_bounds__(kThreads, V * NR <= 16 ? 4 : 2)
    decay_few_kernel(const __grid_constant__ DecayPass p, const __grid_constant__ DecayShape s) {
  constexpr int kRow = kDecayMaxD + 4, kAtOnce = 4, W = NR < 4 ? NR : 4;
  static_assert(kDecayMaxD % NR == 0, "rows of the last thread");
  __shared__ __align__(16) float rows[3][kDecayFew][kRow];       // q, k, v; zeros to the threads' last row
  __shared__ float part[kAtOnce][kThreads * V], w[kDecayFew][kDecayFew], fade[kDecayFew + 1];
  const int bh = blockIdx.x, b = bh / s.H, h = bh - b * s.H, d = s.d, n = decay_length(s, b);
  const float g2 = s.g[h] * kLog2e;
  const int per = d / V, groups = (d + NR - 1) / NR;
  const int r0 = threadIdx.x / per, c = (threadIdx.x - r0 * per) * V, x0 = r0 * NR;
  const int here = r0 < groups ? min(NR, d - x0) : 0;            // rows of this thread
  const int64_t at = (int64_t)bh * d * d + (int64_t)x0 * d + c;
  float m[NR][V];
#pragma unroll
  for (int j = 0; j < NR; ++j) {
#pragma unroll
    for (int i = 0; i < V; ++i) m[j][i] = 0.f;
    if (p.start != nullptr && j < here) load_v<V>(m[j], p.start + at + j * d);
  }
  const T* const from[3] = {static_cast<const T*>(p.a) + b * p.as.b + h * p.as.h,
                            static_cast<const T*>(p.b) + b * p.bs.b + h * p.bs.h,
                            static_cast<const T*>(p.c) + b * p.cs.b + h * p.cs.h};
  const int64_t ls[3] = {p.as.l, p.bs.l, p.cs.l};
  const int dp = max((d + 3) / 4 * 4, groups * NR);
#pragma unroll
  for (int x = 0; x < 3; ++x)
#pragma unroll 4
    for (int e = threadIdx.x; e < n * dp; e += kThreads) {
      const int t = e / dp, y = e - t * dp;
      rows[x][t][y] = y < d ? to_f32(from[x][t * ls[x] + y]) : 0.f;
    }
  if (threadIdx.x <= kDecayFew) fade[threadIdx.x] = decay_power(g2, threadIdx.x);
  __syncthreads();
  {
    static_assert(kDecayFew * kDecayFew == kThreads, "a weight a thread");
    const int t = threadIdx.x / kDecayFew, j = threadIdx.x % kDecayFew;
    if (t < n && j <= t) {
      float sum[4] = {};
#pragma unroll 4
      for (int y = 0; y < d; y += 4) {
        float a[4], k[4];
        load_v<4>(a, &rows[0][t][y]);
        load_v<4>(k, &rows[1][j][y]);
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[i] = fmaf(a[i], k[i], sum[i]);
      }
      w[t][j] = fade[t - j] * ((sum[0] + sum[1]) + (sum[2] + sum[3]));
    }
  }
  T* out = static_cast<T*>(p.o) + b * p.os.b + h * p.os.h;
  for (int t0 = 0; t0 < n; t0 += kAtOnce) {
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      if (t0 + i >= n || here == 0) break;
      float o[V] = {};
#pragma unroll
      for (int j = 0; j < NR; j += W) {
        float q[W];
        load_v<W>(q, &rows[0][t0 + i][x0 + j]);
#pragma unroll
        for (int x = 0; x < W; ++x)
#pragma unroll
          for (int e = 0; e < V; ++e) o[e] = fmaf(q[x], m[j + x][e], o[e]);
      }
#pragma unroll
      for (int e = 0; e < V; ++e) part[i][r0 * d + c + e] = o[e];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < kAtOnce * d; e += kThreads) {
      const int i = e / d, y = e - i * d, t = t0 + i;
      if (t >= n) break;
      float old = 0.f, sum = 0.f;
#pragma unroll 8
      for (int g = 0; g < groups; ++g) old += part[i][g * d + y];
#pragma unroll 4
      for (int j = 0; j <= t; ++j) sum = fmaf(w[t][j], rows[2][j][y], sum);
      out[t * p.os.l + y] = from_f32<T>(p.s_w * fmaf(fade[t + 1], old, sum));
    }
    __syncthreads();
  }
  // rows behind the sequence's end
  for (int e = threadIdx.x; e < (s.L - n) * d; e += kThreads) {
    const int t = e / d;
    out[(n + t) * p.os.l + e - t * d] = from_f32<T>(0.f);
  }
  if (p.last == nullptr || here == 0) return;
  const float all = fade[n];
#pragma unroll
  for (int j = 0; j < NR; ++j)
#pragma unroll
    for (int e = 0; e < V; ++e) m[j][e] *= all;
#pragma unroll 1
  for (int t = 0; t < n; ++t) {
    float v[V];
    load_v<V>(v, &rows[2][t][c]);
    const float u = fade[n - 1 - t];
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] *= u;
#pragma unroll
    for (int j = 0; j < NR; j += W) {
      float k[W];
      load_v<W>(k, &rows[1][t][x0 + j]);
#pragma unroll
      for (int x = 0; x < W; ++x)
#pragma unroll
        for (int e = 0; e < V; ++e) m[j + x][e] = fmaf(k[x], v[e], m[j + x][e]);
    }
  }
#pragma unroll
  for (int j = 0; j < NR; ++j)
    if (j < here) store_v<V>(p.last + at + j * d, m[j]);
}

template <int DP> constexpr size_t pass_smem() { return (3 * (size_t)kC * (DP + 4) + kC * kPS + DP * (DP + 4)) * 4; }
template <int DP> constexpr size_t gain_smem() { return 2 * (size_t)kC * (DP + 4) * 4; }

template <typename T, int DP>
cudaError_t run_pass(const PassSet& set, int n, const DecayShape& s, int piece, cudaStream_t stream) {
  const auto kernel = decay_pass_kernel<T, DP>;
  const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), pass_smem<DP>());
  if (e != cudaSuccess) return e;
  kernel<<<dim3(s.segs * s.BH(), n), kThreads, pass_smem<DP>(), stream>>>(set, s, piece);
  return cudaGetLastError();
}
template <typename T, int DP>
cudaError_t run_gains(const Gains& gains, int n, const DecayShape& s, int piece, cudaStream_t stream) {
  const auto kernel = decay_gain_kernel<T, DP>;
  const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), gain_smem<DP>());
  if (e != cudaSuccess) return e;
  kernel<<<dim3(s.segs * s.BH(), 1, n), kThreads, gain_smem<DP>(), stream>>>(gains, s, piece);
  return cudaGetLastError();
}

}  // namespace

void decay_simt_plan(DecayShape* s, int passes) { decay_segments(s, kC, (s->d <= 64 ? 2 : 1) * sm_count(), passes, 1); }

#define FAVOR_DECAY(call, T)              \
  if (s.d <= 16) return call<T, 16>;      \
  if (s.d <= 32) return call<T, 32>;      \
  if (s.d <= 64) return call<T, 64>;      \
  return call<T, 128>

cudaError_t decay_simt_passes(const DecayPass* passes, int n, const DecayShape& s, bool bf16, int piece,
                              cudaStream_t stream) {
  PassSet set{};
  for (int i = 0; i < n; ++i) set.pass[i] = passes[i];
  auto pick = [&]() -> cudaError_t (*)(const PassSet&, int, const DecayShape&, int, cudaStream_t) {
    if (bf16) { FAVOR_DECAY(run_pass, __nv_bfloat16); }
    FAVOR_DECAY(run_pass, float);
  };
  return pick()(set, n, s, piece, stream);
}

cudaError_t decay_simt_gains(const DecayGain* gains, int n, const DecayShape& s, bool bf16, int piece,
                             cudaStream_t stream) {
  Gains g{};
  for (int i = 0; i < n; ++i) g.kind[i] = gains[i];
  auto pick = [&]() -> cudaError_t (*)(const Gains&, int, const DecayShape&, int, cudaStream_t) {
    if (bf16) { FAVOR_DECAY(run_gains, __nv_bfloat16); }
    FAVOR_DECAY(run_gains, float);
  };
  return pick()(g, n, s, piece, stream);
}
#undef FAVOR_DECAY

cudaError_t decay_scan_states(const DecayScan* scans, int n, const DecayShape& s, cudaStream_t stream) {
  Scans g{};
  for (int i = 0; i < n; ++i) g.kind[i] = scans[i];
  // 16-byte pieces where there are threads enough, else single elements with twice the segments in flight (64 heads of
  // 64 x 64 under the profiler: 6.1 us, with single elements 9.4)
  bool wide = (int64_t)s.BH() * n * s.d * s.d >= (int64_t)4 * kThreads * sm_count() && s.d % 2 == 0;
  for (int i = 0; i < n; ++i) wide = wide && reinterpret_cast<uintptr_t>(scans[i].first) % 16 == 0;
  const int per = kThreads * (wide ? 4 : 1), blocks = (s.d * s.d + per - 1) / per;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(blocks * s.BH()), 1, (unsigned)n);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return wide ? cudaLaunchKernelEx(&cfg, decay_scan_kernel<4, 8>, g, s, blocks)
              : cudaLaunchKernelEx(&cfg, decay_scan_kernel<1, 16>, g, s, blocks);
}

template <typename T>
cudaError_t run_few(const DecayPass& p, const DecayShape& s, bool vec, cudaStream_t stream) {
  const int most = kThreads / (vec ? s.d / 4 : s.d), nr = (s.d + most - 1) / most;       // rows of a thread
  const auto kernel = vec ? nr <= 1   ? decay_few_kernel<T, 4, 1>
                            : nr <= 4 ? decay_few_kernel<T, 4, 4>
                            : nr <= 8 ? decay_few_kernel<T, 4, 8>
                                      : decay_few_kernel<T, 4, 16>
                          : nr <= 4 ? decay_few_kernel<T, 1, 4> : nr <= 16 ? decay_few_kernel<T, 1, 16> : decay_few_kernel<T, 1, 64>;
  kernel<<<s.BH(), kThreads, 0, stream>>>(p, s);
  return cudaGetLastError();
}
cudaError_t decay_few(const DecayPass& p, const DecayShape& s, bool bf16, cudaStream_t stream) {
  const bool vec = s.d % 4 == 0 && (reinterpret_cast<uintptr_t>(p.start) | reinterpret_cast<uintptr_t>(p.last)) % 16 == 0;
  return bf16 ? run_few<__nv_bfloat16>(p, s, vec, stream) : run_few<float>(p, s, vec, stream);
}

cudaError_t launch_decay_step(const DecayStep& p, bool bf16, cudaStream_t stream) {
  const int n = p.B * p.H;
  if (bf16 && p.vec) decay_step_kernel<__nv_bfloat16, 4><<<n, kThreads, 0, stream>>>(p);
  else if (bf16) decay_step_kernel<__nv_bfloat16, 1><<<n, kThreads, 0, stream>>>(p);
  else if (p.vec) decay_step_kernel<float, 4><<<n, kThreads, 0, stream>>>(p);
  else decay_step_kernel<float, 1><<<n, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace favor
