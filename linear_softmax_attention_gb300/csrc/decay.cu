// Causal linear attention with a decay per head on the CUDA cores: fp32 and
// the shapes that the tensor-core path does not take; the scan over segments
// and the one-token step.  decay.cuh has the form that every pass follows.
#include <algorithm>

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

// Rows [t0, t0 + n) of one head into fp32 tile rows, zeros behind them and
// behind the d channels; returns whether this thread met infinities or NaN.
template <typename T, int DP>
__device__ __forceinline__ bool load_tile(float* tile, const T* p, int64_t ls, int n, int d, int piece) {
  constexpr int S = Tile<DP>::S;
  float odd = 0.f;
  if (piece == 16) {
    constexpr int E = 16 / sizeof(T);
    const int per = DP / E > 0 ? DP / E : 1;
    for (int e = threadIdx.x; e < kC * per; e += kThreads) {
      const int r = e / per, c = (e - r * per) * E;
      float f[E];
#pragma unroll
      for (int i = 0; i < E; ++i) f[i] = 0.f;
      if (r < n && c < d) {
        const uint4 raw = *reinterpret_cast<const uint4*>(p + r * ls + c);
        const unsigned w[4] = {raw.x, raw.y, raw.z, raw.w};
        if constexpr (sizeof(T) == 4) {
#pragma unroll
          for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(w[i]);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < E; i += 4)
        *reinterpret_cast<float4*>(tile + r * S + c + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
#pragma unroll
      for (int i = 0; i < E; ++i) odd = fmaf(f[i], 0.f, odd);
    }
  } else {
    for (int e = threadIdx.x; e < kC * DP; e += kThreads) {
      const int r = e / DP, c = e - r * DP;
      const float f = r < n && c < d ? to_f32(p[r * ls + c]) : 0.f;
      tile[r * S + c] = f;
      odd = fmaf(f, 0.f, odd);
    }
  }
  return odd != 0.f;                 // infinities and NaN make it NaN
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

// acc[row][col] += sum_k X[row][k] Y[k][col] over k < K (a multiple of 4), rows
// 16 apart; with GUARD only the terms of k that row may see
template <int DP, bool GUARD>
__device__ __forceinline__ void rows_times(float (&acc)[4][DP / 16], const float* X, int xs, const float* Y, int ys,
                                           int K, bool rev) {
  using C = Cols<DP>;
  const int r0 = threadIdx.x >> 4;
#pragma unroll 2
  for (int k = 0; k < K; k += 4) {
    float x[4][4];
#pragma unroll
    for (int r = 0; r < 4; ++r) load_v<4>(x[r], X + (r0 + 16 * r) * xs + k);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float y[C::N];
#pragma unroll
      for (int j = 0; j < C::N; j += C::V) load_v<C::V>(y + j, Y + (k + i) * ys + C::at(j));
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const bool sees = !GUARD || (rev ? k + i >= r0 + 16 * r : k + i <= r0 + 16 * r);
        if (sees)
#pragma unroll
          for (int j = 0; j < C::N; ++j) acc[r][j] = fmaf(x[r][i], y[j], acc[r][j]);
      }
    }
  }
}

// m[i][j] += sum_t w[t] B[t][row i] C[t][col j] over t < n
template <int DP>
__device__ __forceinline__ void gain_times(float (&m)[DP / 16][DP / 16], const float* B, const float* Cc,
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
    for (int i = 0; i < C::N; ++i) {
      const float x = b[i] * u;
#pragma unroll
      for (int j = 0; j < C::N; ++j) m[i][j] = fmaf(x, c[j], m[i][j]);
    }
  }
}

// One segment of one head: chunk by chunk, the state M in shared memory.
template <typename T, int DP>
__global__ void __launch_bounds__(kThreads) decay_pass_kernel(DecayPass p, DecayShape s, int piece) {
  using C = Cols<DP>;
  constexpr int S = Tile<DP>::S, MS = DP + 4;
  extern __shared__ __align__(16) float sm[];
  float *A = sm, *Bt = A + kC * S, *Ct = Bt + kC * S, *P = Ct + kC * S, *M = P + kC * kPS;
  __shared__ float fade[kC + 1], u[kC];      // l^0 .. l^64; the gains' weights
  const int bh = blockIdx.x / s.segs, seg = blockIdx.x - bh * s.segs, b = bh / s.H, h = bh - b * s.H;
  const float g2 = s.g[h] * kLog2E;
  const int len = decay_length(s, b);
  const int first = seg * s.seg_tokens;
  const int end = min(first + s.seg_tokens, s.L), stop = min(end, len);     // rows to write, tokens
  const int d = s.d;
  const T* a0 = static_cast<const T*>(p.a) + b * p.as.b + h * p.as.h;
  const T* b0 = static_cast<const T*>(p.b) + b * p.bs.b + h * p.bs.h;
  const T* c0 = static_cast<const T*>(p.c) + b * p.cs.b + h * p.cs.h;
  T* o0 = static_cast<T*>(p.o) + b * p.os.b + h * p.os.h;
  const float* start = p.start == nullptr ? nullptr : p.start + ((int64_t)bh * s.segs + seg) * d * d;
  for (int e = threadIdx.x; e < DP * DP; e += kThreads) {
    const int x = e / DP, y = e - x * DP;
    // consecutive threads read consecutive elements of either order
    float v = 0.f;
    if (start != nullptr && x < d && y < d) v = start[x * d + y];
    M[p.transposed ? y * MS + x : x * MS + y] = v;
  }
  if (threadIdx.x <= kC) fade[threadIdx.x] = decay_power(g2, threadIdx.x);
  const int chunks = stop > first ? (stop - first + kC - 1) / kC : 0;
  const int r0 = threadIdx.x >> 4;
  for (int i = 0; i < chunks; ++i) {
    const int t0 = first + (p.rev ? chunks - 1 - i : i) * kC;
    const int n = min(kC, stop - t0);
    __syncthreads();                          // the tiles of the chunk before are read
    load_tile<T, DP>(A, a0 + (int64_t)t0 * p.as.l, p.as.l, n, d, piece);
    load_tile<T, DP>(Bt, b0 + (int64_t)t0 * p.bs.l, p.bs.l, n, d, piece);
    const bool odd = load_tile<T, DP>(Ct, c0 + (int64_t)t0 * p.cs.l, p.cs.l, n, d, piece);
    if (threadIdx.x < kC) u[threadIdx.x] = threadIdx.x < n ? p.s_u * fade[p.rev ? threadIdx.x + 1 : n - 1 - threadIdx.x] : 0.f;
    // infinities and NaN of rows that a token may not see would meet its zero weights
    const bool guard = __syncthreads_or(odd);
    // weights
    {
      float acc[4][4] = {};
#pragma unroll 2
      for (int k = 0; k < DP; k += 4) {
        float x[4][4], y[4][4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          load_v<4>(x[r], A + (r0 + 16 * r) * S + k);
          load_v<4>(y[r], Bt + ((threadIdx.x & 15) + 16 * r) * S + k);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[r][c] = fmaf(x[r][e], y[c][e], acc[r][c]);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int row = r0 + 16 * r, col = (threadIdx.x & 15) + 16 * c;
          const int apart = p.rev ? col - row : row - col;
          P[row * kPS + col] = apart >= 0 && col < n ? p.s_w * fade[apart] * acc[r][c] : 0.f;
        }
    }
    __syncthreads();
    float acc[4][C::N];
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int j = 0; j < C::N; ++j) acc[r][j] = 0.f;
    rows_times<DP, false>(acc, A, S, M, MS, DP, false);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = r0 + 16 * r;
      const float w = row < n ? p.s_r * fade[p.rev ? n - 1 - row : row + 1] : 0.f;
#pragma unroll
      for (int j = 0; j < C::N; ++j) acc[r][j] *= w;
    }
    if (guard) rows_times<DP, true>(acc, P, kPS, Ct, S, kC, p.rev);
    else rows_times<DP, false>(acc, P, kPS, Ct, S, kC, p.rev);
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
    float m[C::N][C::N];
    const float all = fade[n];
#pragma unroll
    for (int x = 0; x < C::N; ++x)
#pragma unroll
      for (int y = 0; y < C::N; y += C::V) {
        load_v<C::V>(&m[x][y], M + C::row(x) * MS + C::at(y));
#pragma unroll
        for (int v = 0; v < C::V; ++v) m[x][y + v] *= all;
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

// The gain of one segment, in registers; block (segment, head, kind)
template <typename T, int DP>
__global__ void __launch_bounds__(kThreads) decay_gain_kernel(Gains gains, DecayShape s, int piece) {
  using C = Cols<DP>;
  constexpr int S = Tile<DP>::S;
  extern __shared__ __align__(16) float sm[];
  float *Bt = sm, *Ct = Bt + kC * S;
  __shared__ float u[kC];
  const DecayGain& p = gains.kind[blockIdx.z];
  const int bh = blockIdx.x / s.segs, seg = blockIdx.x - bh * s.segs, b = bh / s.H, h = bh - b * s.H, d = s.d;
  const float g2 = s.g[h] * kLog2E;
  const int first = seg * s.seg_tokens, stop = min(min(first + s.seg_tokens, s.L), decay_length(s, b));
  const T* b0 = static_cast<const T*>(p.b) + b * p.bs.b + h * p.bs.h;
  const T* c0 = static_cast<const T*>(p.c) + b * p.cs.b + h * p.cs.h;
  float m[C::N][C::N];
#pragma unroll
  for (int x = 0; x < C::N; ++x)
#pragma unroll
    for (int y = 0; y < C::N; ++y) m[x][y] = 0.f;
  for (int t0 = first; t0 < stop; t0 += kC) {
    const int n = min(kC, stop - t0);
    __syncthreads();
    load_tile<T, DP>(Bt, b0 + (int64_t)t0 * p.bs.l, p.bs.l, n, d, piece);
    load_tile<T, DP>(Ct, c0 + (int64_t)t0 * p.cs.l, p.cs.l, n, d, piece);
    if (threadIdx.x < n) {
      const int t = t0 + threadIdx.x;
      u[threadIdx.x] = p.s_u * decay_power(g2, p.rev ? t - first + 1 : stop - 1 - t);
    }
    __syncthreads();
    gain_times<DP>(m, Bt, Ct, u, n);
  }
  float* out = p.out + ((int64_t)bh * s.segs + seg) * d * d;
#pragma unroll
  for (int x = 0; x < C::N; ++x)
#pragma unroll
    for (int y = 0; y < C::N; ++y)
      if (C::row(x) < d && C::at(y) < d) out[C::row(x) * d + C::at(y)] = m[x][y];
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
  const float g2 = s.g[h] * kLog2E;
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
// thread keeps V columns' part of o, which are added through shared memory.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads) decay_step_kernel(DecayStep p) {
  __shared__ float qs[kDecayMaxD], ks[kDecayMaxD], part[kThreads * V];
  const int bh = blockIdx.x, b = bh / p.H, h = bh - b * p.H, d = p.d;
  const T* q = static_cast<const T*>(p.q) + b * p.qs[0] + h * p.qs[1];
  const T* k = static_cast<const T*>(p.k) + b * p.ks[0] + h * p.ks[1];
  const T* v = static_cast<const T*>(p.v) + b * p.vs[0] + h * p.vs[1];
  const float l = exp2f(p.g[h] * kLog2E);
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

template <int DP> constexpr size_t pass_smem() { return (3 * (size_t)kC * (DP + 4) + kC * kPS + DP * (DP + 4)) * 4; }
template <int DP> constexpr size_t gain_smem() { return 2 * (size_t)kC * (DP + 4) * 4; }

template <typename T, int DP>
cudaError_t run_pass(const DecayPass& p, const DecayShape& s, int piece, cudaStream_t stream) {
  const auto kernel = decay_pass_kernel<T, DP>;
  const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), pass_smem<DP>());
  if (e != cudaSuccess) return e;
  kernel<<<s.segs * s.BH(), kThreads, pass_smem<DP>(), stream>>>(p, s, piece);
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

void decay_simt_plan(DecayShape* s) { decay_segments(s, kC, (s->d <= 64 ? 2 : 1) * sm_count(), 1); }

#define FAVOR_DECAY(call, T)              \
  if (s.d <= 16) return call<T, 16>;      \
  if (s.d <= 32) return call<T, 32>;      \
  if (s.d <= 64) return call<T, 64>;      \
  return call<T, 128>

cudaError_t decay_simt_pass(const DecayPass& p, const DecayShape& s, bool bf16, int piece, cudaStream_t stream) {
  auto pick = [&]() -> cudaError_t (*)(const DecayPass&, const DecayShape&, int, cudaStream_t) {
    if (bf16) { FAVOR_DECAY(run_pass, __nv_bfloat16); }
    FAVOR_DECAY(run_pass, float);
  };
  return pick()(p, s, piece, stream);
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
  // 16-byte pieces where there are threads enough, else single elements with twice the segments in flight
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

cudaError_t launch_decay_step(const DecayStep& p, bool bf16, cudaStream_t stream) {
  const int n = p.B * p.H;
  if (bf16 && p.vec) decay_step_kernel<__nv_bfloat16, 4><<<n, kThreads, 0, stream>>>(p);
  else if (bf16) decay_step_kernel<__nv_bfloat16, 1><<<n, kThreads, 0, stream>>>(p);
  else if (p.vec) decay_step_kernel<float, 4><<<n, kThreads, 0, stream>>>(p);
  else decay_step_kernel<float, 1><<<n, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace favor
