// Root-mean-square norm of each head's queries and keys and their rotation by
// positions, in one pass, and its backward pass with the weights' gradients.
//
// Bound by memory: a row is read once, its sum of squares formed from
// registers, and written once; the backward pass recomputes the norm from x and
// takes both sums that it needs,
//   sum x^2  and  sum (z w) x  with  z = R^T dy,
// together.  A row belongs to 1 to 32 neighbouring lanes, about 16 channels each;
// a group of lanes walks the heads of its token, so that sines, cosines and
// weights stay in registers, with several heads' loads in flight.
#include <algorithm>
#include <type_traits>

#include "ops.cuh"
#include "rotary.cuh"

namespace favor {
namespace {

constexpr int kThreads = 256;
constexpr int kSumRows = 32;

// E elements side by side <-> fp32
template <typename T, int E> struct Vec {
  using Raw = typename std::conditional<sizeof(T) * E == 16, uint4,
              typename std::conditional<sizeof(T) * E == 8, uint2,
              typename std::conditional<sizeof(T) * E == 4, unsigned, unsigned short>::type>::type>::type;
  static __device__ __forceinline__ void unpack(const Raw& raw, float* f) {
    if constexpr (sizeof(Raw) == 2) {
      f[0] = __uint_as_float((unsigned)raw << 16);
    } else {
      constexpr int W = sizeof(Raw) / 4;
      unsigned w[W];
      words(raw, w);
#pragma unroll
      for (int i = 0; i < W; ++i) {
        if constexpr (sizeof(T) == 4) {
          f[i] = __uint_as_float(w[i]);
        } else {
          f[2 * i] = __uint_as_float(w[i] << 16);
          f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
      }
    }
  }
  static __device__ __forceinline__ Raw pack(const float* f) {
    if constexpr (sizeof(Raw) == 2) {
      return __bfloat16_as_ushort(__float2bfloat16_rn(f[0]));
    } else {
      constexpr int W = sizeof(Raw) / 4;
      unsigned w[W];
#pragma unroll
      for (int i = 0; i < W; ++i) {
        if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(f[i]);
        else w[i] = tc::pack_bf16(f[2 * i], f[2 * i + 1]);
      }
      if constexpr (W == 4) return make_uint4(w[0], w[1], w[2], w[3]);
      else if constexpr (W == 2) return make_uint2(w[0], w[1]);
      else return w[0];
    }
  }

 private:
  static __device__ __forceinline__ void words(const uint4& r, unsigned* w) {
    w[0] = r.x;
    w[1] = r.y;
    w[2] = r.z;
    w[3] = r.w;
  }
  static __device__ __forceinline__ void words(const uint2& r, unsigned* w) {
    w[0] = r.x;
    w[1] = r.y;
  }
  static __device__ __forceinline__ void words(unsigned r, unsigned* w) { w[0] = r; }
};

struct Side {                         // q or k
  const void *x, *dy;                 // dy: backward
  void* out;
  Strides xs, dys, os;
  const float* w;
  float* part;                        // backward: the CTAs' sums [CTA][d], or NULL
  int heads, share, parts;            // heads of a CTA, CTAs of a token's heads
};

struct Work {
  Side side[2];
  const int32_t* pos;
  const uint64_t* table;
  int end[FAVOR_ROTARY_MAX_AXES];     // pairs of the axes up to and with each
  FastDiv l;                          // tokens of a row
  int tokens, L, d, P, pos_B;
  int lanes, items;                   // lanes of a row; pieces (pairs of pieces) of it
  bool halves;
  float eps;
};

// A row in this thread: item j of lane `lane` is piece (pair of pieces) j lanes +
// lane.  PAIRED: the two halves of E pairs (or E channels behind the pairs),
// else E channels side by side, pairs among them adjacent.
template <typename T, int E, bool PAIRED, int NI> struct Row {
  static constexpr int W = PAIRED ? 2 * E : E, N = PAIRED ? E : E / 2;
  using V = Vec<T, E>;
  using Raw = typename V::Raw;
  static constexpr int R = PAIRED ? 2 : 1;
  int c0[NI], c1[NI];                 // first channels of the pieces; -1: none
  float cs[NI][N], sn[NI][N], w[NI][W];

  __device__ __forceinline__ void places(const Work& k, int lane) {
    const int turning = PAIRED ? k.P / E : 2 * k.P / E;
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      const int item = j * k.lanes + lane;
      const bool in = item < k.items, turns = item < turning;
      if constexpr (!PAIRED) {
        c0[j] = in ? item * E : -1;
        c1[j] = -1;
      } else if (E == 1 && !k.halves) {
        c0[j] = !in ? -1 : turns ? 2 * item : item + k.P;
        c1[j] = turns ? 2 * item + 1 : -1;
      } else {
        c0[j] = !in ? -1 : turns ? item * E : 2 * k.P + (item - turning) * E;
        c1[j] = turns ? item * E + k.P : -1;
      }
    }
  }
  __device__ __forceinline__ void weights(const float* p) {
#pragma unroll
    for (int j = 0; j < NI; ++j)
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const int c = i < E ? c0[j] : c1[j];
        w[j][i] = c < 0 ? 0.f : p == nullptr ? 1.f : p[c + i % E];
      }
  }
  // sines and cosines of token t of sequence b; channels without a position do not turn
  __device__ __forceinline__ void angles(const Work& k, int b, int t, int lane) {
    int axis = -1;
    int32_t at = 0;
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      const int item = j * k.lanes + lane;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int p = item * N + i;
        cs[j][i] = 1.f;
        sn[j][i] = 0.f;
        if (p < k.P) {
          const int a = (p >= k.end[0]) + (p >= k.end[1]) + (p >= k.end[2]);
          if (a != axis) {
            axis = a;
            at = k.pos[((int64_t)a * k.pos_B + (k.pos_B > 1 ? b : 0)) * k.L + t];
          }
          sine_cosine(at, k.table[p], &sn[j][i], &cs[j][i]);
        }
      }
    }
  }
  __device__ __forceinline__ void load(Raw (&raw)[NI][R], const T* row) const {
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      raw[j][0] = c0[j] >= 0 ? *reinterpret_cast<const Raw*>(row + c0[j]) : Raw{};
      if constexpr (PAIRED) raw[j][1] = c1[j] >= 0 ? *reinterpret_cast<const Raw*>(row + c1[j]) : Raw{};
    }
  }
  __device__ __forceinline__ void unpack(const Raw (&raw)[NI][R], float (&v)[NI][W]) const {
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      V::unpack(raw[j][0], v[j]);
      if constexpr (PAIRED) V::unpack(raw[j][1], v[j] + E);
    }
  }
  __device__ __forceinline__ void store(T* row, const float (&v)[NI][W]) const {
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      if (c0[j] >= 0) *reinterpret_cast<Raw*>(row + c0[j]) = V::pack(v[j]);
      if constexpr (PAIRED)
        if (c1[j] >= 0) *reinterpret_cast<Raw*>(row + c1[j]) = V::pack(v[j] + E);
    }
  }
  // the pairs turned by their angles, or back
  template <bool BACK> __device__ __forceinline__ void turn(float (&v)[NI][W]) const {
#pragma unroll
    for (int j = 0; j < NI; ++j)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float &u = v[j][PAIRED ? i : 2 * i], &z = v[j][PAIRED ? E + i : 2 * i + 1];
        const float c = cs[j][i], s = BACK ? -sn[j][i] : sn[j][i];
        const float a = u * c - z * s;
        z = u * s + z * c;
        u = a;
      }
  }
};

__device__ __forceinline__ float lanes_sum(float v, int lanes) {
  for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// 1 / sqrt(x); NaN for infinity: a sum of squares that has left fp32 gives no zeros
__device__ __forceinline__ float inverse_root(float x) { return fmaf(x, 0.f, rsqrtf(x)); }

// heads of a thread whose loads are in flight together
template <int NI, int R, int E, bool BWD>
constexpr int kHeads = (E > 2 ? 8 : 4) / (NI * R * (BWD ? 2 : 1)) > 0 ? (E > 2 ? 8 : 4) / (NI * R * (BWD ? 2 : 1)) : 1;

template <typename T, int E, bool PAIRED, int NI, bool BWD>
__global__ void __launch_bounds__(kThreads) qk_norm_kernel(const __grid_constant__ Work k) {
  using Rw = Row<T, E, PAIRED, NI>;
  using Raw = typename Rw::Raw;
  constexpr int W = Rw::W, HB = kHeads<NI, Rw::R, E, BWD>;
  const int qparts = k.side[0].parts;
  const bool keys = (int)blockIdx.y >= qparts;
  const Side& s = k.side[keys];
  const int part = blockIdx.y - (keys ? qparts : 0);
  const int h0 = part * s.share, h1 = h0 + min(s.share, s.heads - h0);
  const int lane = threadIdx.x & (k.lanes - 1), group = threadIdx.x / k.lanes, groups = kThreads / k.lanes;
  const float inv_d = 1.f / k.d;
  Rw row;
  row.places(k, lane);
  row.weights(s.w);
  float dw[NI][W];
#pragma unroll
  for (int j = 0; j < NI; ++j)
#pragma unroll
    for (int i = 0; i < W; ++i) dw[j][i] = 0.f;
  // a CTA's groups walk together: every lane of a warp takes part in the sums
  for (int64_t base = (int64_t)blockIdx.x * groups; base < k.tokens; base += (int64_t)gridDim.x * groups) {
    const int64_t token = base + group;
    const bool real = token < k.tokens;
    const uint32_t tk = real ? (uint32_t)token : 0u;
    const int b = (int)k.l.div(tk), t = (int)tk - b * k.L;
    row.angles(k, b, t, lane);
    const T* x0 = static_cast<const T*>(s.x) + b * s.xs.b + t * s.xs.l;
    const T* dy0 = BWD ? static_cast<const T*>(s.dy) + b * s.dys.b + t * s.dys.l : nullptr;
    T* o0 = static_cast<T*>(s.out) + b * s.os.b + t * s.os.l;
    for (int hb = h0; hb < h1; hb += HB) {
      Raw rx[HB][NI][Rw::R], ry[BWD ? HB : 1][NI][Rw::R];
#pragma unroll
      for (int i = 0; i < HB; ++i) {
        const int h = min(hb + i, h1 - 1);
        row.load(rx[i], x0 + h * s.xs.h);
        if constexpr (BWD) row.load(ry[i], dy0 + h * s.dys.h);
      }
#pragma unroll
      for (int i = 0; i < HB; ++i) {
        const bool here = real && hb + i < h1;
        float x[NI][W];
        row.unpack(rx[i], x);
        float sq = 0.f;
#pragma unroll
        for (int j = 0; j < NI; ++j)
#pragma unroll
          for (int e = 0; e < W; ++e) sq = fmaf(x[j][e], x[j][e], sq);
        if constexpr (!BWD) {
          const float r = inverse_root(fmaf(lanes_sum(sq, k.lanes), inv_d, k.eps));
#pragma unroll
          for (int j = 0; j < NI; ++j)
#pragma unroll
            for (int e = 0; e < W; ++e) x[j][e] *= r * row.w[j][e];
          row.template turn<false>(x);
          if (here) row.store(o0 + (hb + i) * s.os.h, x);
        } else {
          float z[NI][W];
          row.unpack(ry[i], z);
          row.template turn<true>(z);
          float zx = 0.f;
#pragma unroll
          for (int j = 0; j < NI; ++j)
#pragma unroll
            for (int e = 0; e < W; ++e) zx = fmaf(z[j][e] * row.w[j][e], x[j][e], zx);
          sq = lanes_sum(sq, k.lanes);
          zx = lanes_sum(zx, k.lanes);
          const float r = inverse_root(fmaf(sq, inv_d, k.eps));
          const float along = r * r * (zx * inv_d);
#pragma unroll
          for (int j = 0; j < NI; ++j)
#pragma unroll
            for (int e = 0; e < W; ++e) {
              if (here) dw[j][e] = fmaf(z[j][e], x[j][e] * r, dw[j][e]);
              x[j][e] = r * (z[j][e] * row.w[j][e] - x[j][e] * along);
            }
          if (here) row.store(o0 + (hb + i) * s.os.h, x);
        }
      }
    }
  }
  if constexpr (BWD) {
    if (s.part == nullptr) return;
    // the groups' sums side by side, then column by column
    extern __shared__ float sums[];
#pragma unroll
    for (int j = 0; j < NI; ++j)
#pragma unroll
      for (int e = 0; e < W; ++e) {
        const int c = e < E ? row.c0[j] : row.c1[j];
        if (c >= 0) sums[group * k.d + c + e % E] = dw[j][e];
      }
    __syncthreads();
    float* out = s.part + ((int64_t)part * gridDim.x + blockIdx.x) * k.d;
    for (int c = threadIdx.x; c < k.d; c += kThreads) {
      float v = sums[c];
      for (int g = 1; g < groups; ++g) v += sums[g * k.d + c];
      out[c] = v;
    }
  }
}

struct Sums {
  const float* part[2];
  float* out[2];
  int n[2];
};
// The CTAs' sums in their order: a block per 32 columns of a weight
__global__ void __launch_bounds__(32 * kSumRows) qk_norm_sum_kernel(Sums k, int d) {
  __shared__ float s[kSumRows][32];
  const int lane = threadIdx.x & 31, row = threadIdx.x >> 5, c = blockIdx.x * 32 + lane, side = blockIdx.y;
  tc::griddep_wait();
  if (k.out[side] == nullptr) return;
  float v = 0.f;
  if (c < d)
#pragma unroll 8
    for (int i = row; i < k.n[side]; i += kSumRows) v += k.part[side][(int64_t)i * d + c];
  s[row][lane] = v;
  __syncthreads();
  if (row == 0 && c < d) {
#pragma unroll
    for (int i = 1; i < kSumRows; ++i) v += s[i][lane];
    k.out[side][c] = v;
  }
}

struct Plan {
  int E, NI, lanes, items;
  bool paired;
  int ctas, share[2], parts[2];
};

Plan make_plan(const QkNormArgs& a, bool bf16, int piece, bool backward) {
  Plan p{};
  const int e = bf16 ? 2 : 4;
  auto whole = [&](int n) {
    return piece >= n * e && (a.halves ? a.pairs % n == 0 : 2 * a.pairs % n == 0) && a.d % n == 0;
  };
  p.E = whole(16 / e) ? 16 / e : whole(2) ? 2 : 1;
  p.paired = a.halves || p.E == 1;
  p.items = p.E == 1 ? a.d - a.pairs : p.paired ? a.pairs / p.E + (a.d - 2 * a.pairs) / p.E : a.d / p.E;
  const int width = p.paired ? 2 * p.E : p.E;
  p.NI = std::max(1, 16 / width);
  auto lanes = [&] {
    int n = 1;
    while (n * p.NI < p.items) n *= 2;
    return n;
  };
  if (lanes() > 32) p.NI *= 2;
  p.lanes = lanes();
  const int64_t tokens = (int64_t)a.B * a.L, groups = kThreads / p.lanes;
  const int64_t sms = sm_count(), wide = (tokens + groups - 1) / groups;
  // backward: CTAs that walk, so that their sums of the weights' gradients stay few
  p.ctas = (int)(backward ? std::min<int64_t>(wide, 4 * sms) : wide);
  // enough CTAs for every SM: fewer heads each where tokens are few
  const int64_t want = std::max<int64_t>(1, 8 * sms / std::max(1, p.ctas));
  const int heads[2] = {a.Hq, a.Hk};
  for (int i = 0; i < 2; ++i) {
    if (heads[i] == 0) continue;
    const int64_t parts = std::min<int64_t>(std::min(heads[i], 16384), want);
    p.share[i] = (int)((heads[i] + parts - 1) / parts);
    p.parts[i] = (heads[i] + p.share[i] - 1) / p.share[i];
  }
  return p;
}

template <typename T, int E, bool PAIRED, int NI>
cudaError_t run(const Work& w, const Plan& p, bool backward, cudaStream_t stream) {
  const dim3 grid(p.ctas, p.parts[0] + p.parts[1]);
  if (!backward) {
    qk_norm_kernel<T, E, PAIRED, NI, false><<<grid, kThreads, 0, stream>>>(w);
    return cudaGetLastError();
  }
  const size_t smem = (size_t)(kThreads / p.lanes) * w.d * sizeof(float);
  const auto kernel = qk_norm_kernel<T, E, PAIRED, NI, true>;
  const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), smem);
  if (e != cudaSuccess) return e;
  kernel<<<grid, kThreads, smem, stream>>>(w);
  return cudaGetLastError();
}

template <typename T, int E, int NI>
cudaError_t run_paired(const Work& w, const Plan& p, bool backward, cudaStream_t stream) {
  return p.NI > NI ? run<T, E, true, 2 * NI>(w, p, backward, stream) : run<T, E, true, NI>(w, p, backward, stream);
}

template <typename T>
cudaError_t run_type(const Work& w, const Plan& p, bool backward, cudaStream_t stream) {
  constexpr int F = 16 / sizeof(T);
  if (p.E == 1) return run_paired<T, 1, 8>(w, p, backward, stream);
  if (p.E == 2) return p.paired ? run_paired<T, 2, 4>(w, p, backward, stream) : run<T, 2, false, 8>(w, p, backward, stream);
  return p.paired ? run_paired<T, F, 8 / F>(w, p, backward, stream) : run<T, F, false, 16 / F>(w, p, backward, stream);
}

}  // namespace

size_t qk_norm_workspace_bytes(const QkNormArgs& a) {
  // what any kernel of the shape may write, whatever the tensors' alignment and the pairs
  size_t most = 0;
  for (int lanes = 1; lanes <= 32; lanes *= 2) {
    const int64_t groups = kThreads / lanes, wide = ((int64_t)a.B * a.L + groups - 1) / groups;
    const int64_t ctas = std::min<int64_t>(wide, 4 * sm_count()), want = std::max<int64_t>(1, 8 * sm_count() / ctas);
    size_t n = 0;
    for (const int heads : {a.Hq, a.Hk}) n += (size_t)ctas * std::min<int64_t>(heads, want);
    most = std::max(most, n);
  }
  return most * a.d * sizeof(float);
}

cudaError_t launch_qk_norm(const QkNormArgs& a, bool bf16, int piece, bool backward, float* ws, cudaStream_t stream) {
  const Plan p = make_plan(a, bf16, piece, backward);
  Work w{};
  const void *x[2] = {a.q, a.k}, *dy[2] = {a.dqo, a.dko};
  void* out[2] = {a.qo, a.ko};
  const Strides xs[2] = {a.qs, a.ks}, dys[2] = {a.dqos, a.dkos}, os[2] = {a.qos, a.kos};
  const float* weight[2] = {a.wq, a.wk};
  float* dw[2] = {a.dwq, a.dwk};
  const int heads[2] = {a.Hq, a.Hk};
  Sums sums{};
  bool any = false;
  float* at = ws;
  for (int i = 0; i < 2; ++i) {
    Side& s = w.side[i];
    s.x = x[i];
    s.dy = dy[i];
    s.out = out[i];
    s.xs = xs[i];
    s.dys = dys[i];
    s.os = os[i];
    s.w = weight[i];
    s.heads = heads[i];
    s.share = p.share[i];
    s.parts = p.parts[i];
    if (backward && dw[i] != nullptr && heads[i] > 0) {
      any = true;
      s.part = at;
      sums.part[i] = at;
      sums.out[i] = dw[i];
      sums.n[i] = p.ctas * p.parts[i];
      at += (int64_t)sums.n[i] * a.d;
    }
  }
  w.pos = a.pos;
  w.table = a.table;
  int end = 0;
  for (int i = 0; i < FAVOR_ROTARY_MAX_AXES; ++i) w.end[i] = end += i < a.n_axes ? a.sections[i] : 0;
  w.l = FastDiv((uint32_t)a.L);
  w.tokens = a.B * a.L;
  w.L = a.L;
  w.d = a.d;
  w.P = a.pairs;
  w.pos_B = a.pos_B;
  w.lanes = p.lanes;
  w.items = p.items;
  w.halves = a.halves;
  w.eps = a.eps;
  cudaError_t e = bf16 ? run_type<__nv_bfloat16>(w, p, backward, stream) : run_type<float>(w, p, backward, stream);
  if (e != cudaSuccess || !any) return e;
  qk_norm_sum_kernel<<<dim3((a.d + 31) / 32, 2), 32 * kSumRows, 0, stream>>>(sums, a.d);
  return cudaGetLastError();
}

}  // namespace favor
