// Root-mean-square norm of each head's queries and keys and their rotation by
// positions, in one pass, and its backward pass with the weights' gradients.
//
// Bound by memory: a row is read once, its sum of squares formed from
// registers, and written once; the backward pass recomputes the norm from x and
// takes both sums that it needs,
//   sum x^2  and  sum (z w) x  with  z = R^T dy,
// together.  A row belongs to 1 to 32 neighbouring lanes, about 16 channels each;
// a group of lanes walks the heads of its token, q's and k's, so that sines and
// cosines are formed once, and each thread copies its pieces of the next rows
// ahead into its own places in shared memory.
//
// Measured (one GB300; copy rate 6682 GB/s): 65536 tokens x (16 + 16) heads of 128
// bf16 out of a joint [B, L, 3, H, d] buffer 167 us, 6.4 TB/s; backward of (16 + 4)
// heads 168 us, 6.0 TB/s; 2 x 12288 x (8 + 8) heads of 64 fp32 35 and 62 us, bf16
// 21.4 and 39 us (floors 30, 45, 15 and 23): there the waves' ends and, backward,
// the second kernel show.  256 tokens of (8 + 8) heads of 64: 3.6 us.
#include <float.h>

#include <algorithm>
#include <type_traits>

#include "ops.cuh"
#include "rotary.cuh"

namespace favor {
namespace {

// Small CTAs spread evenly over the SMs (2 x 12288 x (8 + 8) heads of 64 bf16
// forward: 21.9 us, 25.1 with 128 threads, 27.5 with 256); the backward pass's leave
// sums behind that are added up after (39 us, 51 with 256).
template <bool BWD> constexpr int kThreads = BWD ? 128 : 64;
constexpr int kSumRows = 32;
constexpr int kMostParts = 64;       // CTAs that a token's heads are shared out to, at most

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
};

struct Work {
  Side side[2];
  const int32_t* pos;
  const uint64_t* table;
  int end[FAVOR_ROTARY_MAX_AXES];     // pairs of the axes up to and with each
  FastDiv l;                          // tokens of a row
  int tokens, L, d, P, pos_B;
  int Hq, heads, share;               // heads of q, of q and k, of a CTA
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
  float cs[NI][N], sn[NI][N];

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
  // rounded once, to the nearest
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
    if constexpr (PAIRED && E > 1) {
#pragma unroll
      for (int j = 0; j < NI; ++j)
#pragma unroll
        for (int i = 0; i < E; i += 2) {
          const float2 u = make_float2(v[j][i], v[j][i + 1]), z = make_float2(v[j][E + i], v[j][E + i + 1]);
          const float2 c = make_float2(cs[j][i], cs[j][i + 1]);
          const float2 s = BACK ? make_float2(-sn[j][i], -sn[j][i + 1]) : make_float2(sn[j][i], sn[j][i + 1]);
          const float2 a = fma2(u, c, mul2(make_float2(-z.x, -z.y), s)), b = fma2(u, s, mul2(z, c));
          v[j][i] = a.x;
          v[j][i + 1] = a.y;
          v[j][E + i] = b.x;
          v[j][E + i + 1] = b.y;
        }
    } else {
#pragma unroll
      for (int j = 0; j < NI; ++j)
#pragma unroll
        for (int i = 0; i < N; ++i) {
          constexpr int kZ = PAIRED ? E : 1;
          float &u = v[j][PAIRED ? i : 2 * i], &z = v[j][PAIRED ? i + kZ : 2 * i + kZ];
          const float c = cs[j][i], s = BACK ? -sn[j][i] : sn[j][i];
          const float a = u * c - z * s;
          z = u * s + z * c;
          u = a;
        }
    }
  }
};

// The next rows of X tensors on their way: each thread's own places in shared
// memory, S rows deep (elements of two bytes, which no asynchronous copy takes,
// are stored there at once).
template <typename T, int E, bool PAIRED, int NI, int X> struct Ring {
  using Rw = Row<T, E, PAIRED, NI>;
  using Raw = typename Rw::Raw;
  static constexpr int kRow = X * NI * Rw::R * (int)sizeof(Raw);
  static constexpr int S = kRow <= 16 ? 8 : kRow <= 32 ? 6 : kRow <= 64 ? 3 : 2;
  static constexpr int kT = kThreads<X == 2>;
  static constexpr size_t kBytes = (size_t)S * kRow * kT;
  Raw* mine;
  int in = 0, out = 0;
  __device__ __forceinline__ explicit Ring(void* ring) : mine(static_cast<Raw*>(ring) + threadIdx.x) {}
  __device__ __forceinline__ Raw* place(int stage, int x, int j, int r) const {
    return mine + (((stage * X + x) * NI + j) * Rw::R + r) * kT;
  }
  __device__ __forceinline__ void copy(Raw* to, const T* from, bool here) {
    if constexpr (sizeof(Raw) == 2) {
      *to = here ? *reinterpret_cast<const Raw*>(from) : Raw{};
    } else if constexpr (sizeof(Raw) == 16) {
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tc::smem_addr(to)), "l"(from),
                   "r"(here ? 16 : 0)
                   : "memory");
    } else {
      asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(tc::smem_addr(to)), "l"(from),
                   "n"(sizeof(Raw)), "r"(here ? (int)sizeof(Raw) : 0)
                   : "memory");
    }
  }
  // starts the copies of a row of tensor x; pieces that the row lacks become 0
  __device__ __forceinline__ void fetch(const Rw& row, int x, const T* from, bool real) {
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      const bool h0 = real && row.c0[j] >= 0;
      copy(place(in, x, j, 0), h0 ? from + row.c0[j] : from, h0);
      if constexpr (PAIRED) {
        const bool h1 = real && row.c1[j] >= 0;
        copy(place(in, x, j, 1), h1 ? from + row.c1[j] : from, h1);
      }
    }
  }
  __device__ __forceinline__ void fetched() {
    asm volatile("cp.async.commit_group;" ::: "memory");
    in = in + 1 == S ? 0 : in + 1;
  }
  __device__ __forceinline__ void wait() { asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory"); }
  __device__ __forceinline__ void take(int x, float (&v)[NI][Rw::W]) const {
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      Rw::V::unpack(*place(out, x, j, 0), v[j]);
      if constexpr (PAIRED) Rw::V::unpack(*place(out, x, j, 1), v[j] + E);
    }
  }
  __device__ __forceinline__ void taken() { out = out + 1 == S ? 0 : out + 1; }
};

// values two by two (W is even)
template <int NI, int W, typename F> __device__ __forceinline__ void each(F&& f) {
#pragma unroll
  for (int j = 0; j < NI; ++j)
#pragma unroll
    for (int e = 0; e < W; e += 2) f(j, e);
}
template <int W> __device__ __forceinline__ float2 get(const float (&x)[W], int e) { return make_float2(x[e], x[e + 1]); }
template <int W> __device__ __forceinline__ void put(float (&x)[W], int e, float2 v) {
  x[e] = v.x;
  x[e + 1] = v.y;
}
__device__ __forceinline__ float2 twice(float x) { return make_float2(x, x); }

__device__ __forceinline__ float lanes_sum(float v, int lanes) {
  for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// 1 / sqrt(x); NaN for infinity: a sum of squares that has left fp32 gives no zeros
__device__ __forceinline__ float inverse_root(float x) { return fmaf(x, 0.f, rsqrtf(x)); }

// A group's rows in their order: the heads [h0, h1) of its tokens, q's first.
template <typename T> struct Walk {
  const Work& k;
  int64_t base, stride, token;        // the CTA's first token, the step, this group's
  int group, h0, h1, h;
  bool real;
  const T *q, *kk, *dq, *dk;          // the token's rows of head 0
  __device__ __forceinline__ Walk(const Work& w, int g, int groups, int from, int to)
      : k(w), base((int64_t)blockIdx.x * groups), stride((int64_t)gridDim.x * groups), group(g), h0(from), h1(to), h(from) {
    place();
  }
  __device__ __forceinline__ bool more() const { return base < k.tokens; }
  __device__ __forceinline__ void place() {
    token = base + group;
    real = token < k.tokens;
    const uint32_t tk = real ? (uint32_t)token : 0u;
    const int b = (int)k.l.div(tk), t = (int)tk - b * k.L;
    auto at = [&](const void* p, const Strides& s) { return static_cast<const T*>(p) + b * s.b + t * s.l; };
    q = at(k.side[0].x, k.side[0].xs);
    kk = at(k.side[1].x, k.side[1].xs);
    dq = at(k.side[0].dy, k.side[0].dys);
    dk = at(k.side[1].dy, k.side[1].dys);
  }
  __device__ __forceinline__ const T* x() const {
    return h < k.Hq ? q + h * k.side[0].xs.h : kk + (h - k.Hq) * k.side[1].xs.h;
  }
  __device__ __forceinline__ const T* dy() const {
    return h < k.Hq ? dq + h * k.side[0].dys.h : dk + (h - k.Hq) * k.side[1].dys.h;
  }
  __device__ __forceinline__ void next() {
    if (++h < h1) return;
    h = h0;
    base += stride;
    place();
  }
};

template <typename T, int E, bool PAIRED, int NI, bool BWD>
__global__ void __launch_bounds__(kThreads<BWD>, NI * (PAIRED ? 2 * E : E) > 16 || E == 1 ? 1 : BWD ? 4 : 12)
    qk_norm_kernel(const __grid_constant__ Work k) {
  using Rw = Row<T, E, PAIRED, NI>;
  using Rn = Ring<T, E, PAIRED, NI, BWD ? 2 : 1>;
  constexpr int W = Rw::W, kT = kThreads<BWD>;
  extern __shared__ __align__(16) float smem[];
  float* weights = smem;                                         // [2][d], then the ring
  const int lane = threadIdx.x & (k.lanes - 1), group = threadIdx.x / k.lanes, groups = kT / k.lanes;
  const int h0 = blockIdx.y * k.share, h1 = h0 + min(k.share, k.heads - h0);
  const float inv_d = 1.f / k.d;
  Rw row;
  row.places(k, lane);
  Rn ring(smem + (2 * k.d + 3) / 4 * 4);
  Walk<T> ahead(k, group, groups, h0, h1);
  auto fetch = [&] {
    if (ahead.more()) {
      ring.fetch(row, 0, ahead.x(), ahead.real);
      if constexpr (BWD) ring.fetch(row, 1, ahead.dy(), ahead.real);
      ahead.next();
    }
    ring.fetched();
  };
#pragma unroll
  for (int i = 0; i < Rn::S - 1; ++i) fetch();
  for (int c = threadIdx.x; c < 2 * k.d; c += kT) {
    const float* w = k.side[c >= k.d].w;
    weights[c] = w == nullptr ? 1.f : w[c >= k.d ? c - k.d : c];
  }
  __syncthreads();
  float dw[BWD ? 2 : 1][NI][W];
  if constexpr (BWD) {
#pragma unroll
    for (int j = 0; j < NI; ++j)
#pragma unroll
      for (int e = 0; e < W; ++e) dw[0][j][e] = dw[1][j][e] = 0.f;
  }
  // a CTA's groups walk together: every lane of a warp takes part in the sums
  for (int64_t base = (int64_t)blockIdx.x * groups; base < k.tokens; base += (int64_t)gridDim.x * groups) {
    const int64_t token = base + group;
    const bool real = token < k.tokens;
    const uint32_t tk = real ? (uint32_t)token : 0u;
    const int b = (int)k.l.div(tk), t = (int)tk - b * k.L;
    row.angles(k, b, t, lane);
    auto heads = [&](const Side& s, const float* w0, int from, int to, float (&sums)[NI][W]) {
      T* o = static_cast<T*>(s.out) + b * s.os.b + t * s.os.l + from * s.os.h;
      for (int h = from; h < to; ++h, o += s.os.h) {
        fetch();
        ring.wait();
        float x[NI][W], w[NI][W];
        ring.take(0, x);
#pragma unroll
        for (int j = 0; j < NI; ++j)
#pragma unroll
          for (int e = 0; e < W; e += E) {
            const int c = e < E ? row.c0[j] : row.c1[j];
            const float* at = w0 + max(c, 0);
            if constexpr (E % 4 == 0) {
#pragma unroll
              for (int i = 0; i < E; i += 4) {
                const float4 v = *reinterpret_cast<const float4*>(at + i);
                w[j][e + i] = v.x;
                w[j][e + i + 1] = v.y;
                w[j][e + i + 2] = v.z;
                w[j][e + i + 3] = v.w;
              }
            } else {
#pragma unroll
              for (int i = 0; i < E; ++i) w[j][e + i] = at[i];
            }
          }
        float2 sq2 = make_float2(0.f, 0.f);
        each<NI, W>([&](int j, int e) {
          const float2 v = get(x[j], e);
          sq2 = fma2(v, v, sq2);
        });
        float sq = sq2.x + sq2.y;
        if constexpr (!BWD) {
          ring.taken();
          const float r = inverse_root(fmaf(lanes_sum(sq, k.lanes), inv_d, k.eps));
          each<NI, W>([&](int j, int e) { put(x[j], e, mul2(get(x[j], e), mul2(twice(r), get(w[j], e)))); });
          row.template turn<false>(x);
        } else {
          float z[NI][W];
          ring.take(1, z);
          ring.taken();
          row.template turn<true>(z);
          float2 zx2 = make_float2(0.f, 0.f);
          each<NI, W>([&](int j, int e) {
            const float2 zw = mul2(get(z[j], e), get(w[j], e));
            zx2 = fma2(zw, get(x[j], e), zx2);
            put(w[j], e, zw);
          });
          float zx = zx2.x + zx2.y;
          for (int m = k.lanes >> 1; m > 0; m >>= 1) {
            sq += __shfl_xor_sync(0xffffffffu, sq, m);
            zx += __shfl_xor_sync(0xffffffffu, zx, m);
          }
          const float r = inverse_root(fmaf(sq, inv_d, k.eps));
          // r^2 leaves fp32 where the mean square and eps are below 2^-128; its product with the mean need not
          const float m = zx * inv_d, rr = r * r;
          const float2 along = twice(-(rr <= FLT_MAX ? rr * m : r * (r * m))), r2 = twice(r);
          each<NI, W>([&](int j, int e) {
            const float2 v = get(x[j], e);
            if (real) put(sums[j], e, fma2(get(z[j], e), mul2(v, r2), get(sums[j], e)));
            put(x[j], e, mul2(r2, fma2(v, along, get(w[j], e))));
          });
        }
        if (real) row.store(o, x);
      }
    };
    heads(k.side[0], weights, h0, min(h1, k.Hq), dw[0]);
    heads(k.side[1], weights + k.d, max(h0 - k.Hq, 0), h1 - k.Hq, dw[BWD ? 1 : 0]);
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");           // nothing is on its way any more
  if constexpr (BWD) {
    // the kernel that adds the CTAs' sums may take its place and wait
    asm volatile("griddepcontrol.launch_dependents;");
    // the groups' sums side by side in the ring's place, then column by column
    float* sums = smem;
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      float* part = k.side[side].part;
      if (part == nullptr) continue;
      __syncthreads();
#pragma unroll
      for (int j = 0; j < NI; ++j)
#pragma unroll
        for (int e = 0; e < W; ++e) {
          const int c = e < E ? row.c0[j] : row.c1[j];
          if (c >= 0) sums[group * k.d + c + e % E] = dw[side][j][e];
        }
      __syncthreads();
      float* out = part + ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * k.d;
      for (int c = threadIdx.x; c < k.d; c += kT) {
        float v = sums[c];
#pragma unroll 8
        for (int g = 1; g < groups; ++g) v += sums[g * k.d + c];
        out[c] = v;
      }
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
  int ctas, share, parts;             // CTAs beside one another; heads of one, CTAs of a token's heads
};

// CTAs of a launch: at most about four waves of those that are resident walk the
// tokens, and a token's heads go to the number of CTAs with the least work for the
// fullest SM, in rows: a CTA's own and `extra` for its angles (and, backward, the sums it
// leaves) times the CTAs, of which 12 (4) run at once and fewer than 6 cost as 6, and
// one for the start and end.  A token's heads in 1, 2, 4 and 8 CTAs forward:
// 16384 x 32 heads of 128 bf16 54.1, 47.2, 49.3, 59.0 us (taken: 2), 2 x 12288 x 16 of 64
// fp32 37.8, 35.5, 34.3, 40.3 (2), bf16 22.0, 22.6, 25.3, 33.5 (1), 4 x 2048 x 32 of 96
// fp32 36.7, 38.6, 35.5, 37.2 (1), 256 x 16 of 64 bf16 9.7, 6.9, 5.5, 5.0 (16: 4.6).
// Backward: 75, 81, 97, 141 (1); 62, 61, 69, 95 (1); 40, 41, 55, 85 (1); 54, 58, 63, 74
// (2); 13, 9.7, 8.2, 7.6 (8).  The counts are those of pieces of 16 bytes; the other kernels
// have fewer CTAs to an SM, and the rule serves them so: pieces of two elements, 2 x 4096 x
// 16 heads of 90 bf16 forward 18.0, 18.7, 19.5, 25.4 us (1), backward 31.6, 32.1, 38.8, 50.6 (1),
// 3 x 1111 x 10 of 90 fp32 9.1, 7.9, 7.4, 9.4 (2) and 18.3, 14.8, 18.2, 17.5 (2); rows of 512,
// 8192 x 16 heads bf16 51.8, 56.8, 70, 102 (1) and 83, 105, 154, 250 (1); single elements, 2 x
// 4096 x 16 heads of 33 fp32 15.6, 17.5, 17.0, 18.9 (2) and 27.7, 31.2, 37.3, 45.3 (2), bf16 17.1,
// 18.3, 20.9, 25.1 (2) and 25.1, 28.4, 34.4, 44.8 (2): there it takes one CTA too many.
void share_out(Plan* p, int64_t tokens, int heads, bool bf16, bool backward) {
  const int64_t sms = sm_count(), groups = (backward ? kThreads<true> : kThreads<false>) / p->lanes;
  const int64_t units = std::min((tokens + groups - 1) / groups, (backward ? 16 : 48) * sms);
  const double extra = backward ? 4 : bf16 ? 2.8 : 1.25;
  double best = -1;
  for (int parts = 1; parts <= std::min(heads, kMostParts); ++parts) {
    const int share = (int)(((int64_t)heads + parts - 1) / parts);
    const int64_t ctas = (units * parts + sms - 1) / sms;        // of the fullest SM
    const double rounds = backward ? (double)units * parts / sms + 1.5
                                   : ctas / 12 * 12 + (ctas % 12 > 0 ? std::max<int64_t>(ctas % 12, 6) : 0) + 1;
    const double cost = rounds * (share + extra);
    if (best < 0 || cost < best) {
      best = cost;
      p->share = share;
    }
  }
  p->share = std::max(p->share, heads / 32768 + 1);
  p->parts = (int)(((int64_t)heads + p->share - 1) / p->share);
  p->ctas = (int)units;
}

// Pieces of 16 bytes, else of two elements, where the rows and each half of the
// pairs are made of whole ones, else pair by pair: 16384 x (16 + 16) heads of 128
// bf16 forward 65, 82 and 165 us for halves, 65, 75 and 173 for adjacent pairs;
// backward 80, 114 and 256, and 80, 111 and 265.
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
  share_out(&p, (int64_t)a.B * a.L, a.Hq + a.Hk, bf16, backward);
  return p;
}

template <typename T, int E, bool PAIRED, int NI>
cudaError_t run(const Work& w, const Plan& p, bool backward, cudaStream_t stream) {
  const auto kernel = backward ? qk_norm_kernel<T, E, PAIRED, NI, true> : qk_norm_kernel<T, E, PAIRED, NI, false>;
  const size_t ring = backward ? Ring<T, E, PAIRED, NI, 2>::kBytes : Ring<T, E, PAIRED, NI, 1>::kBytes;
  size_t smem = (2 * (size_t)w.d + 3) / 4 * 16 + ring;
  if (backward) smem = std::max(smem, (size_t)(kThreads<true> / p.lanes) * w.d * sizeof(float));
  const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), smem);
  if (e != cudaSuccess) return e;
  kernel<<<dim3(p.ctas, p.parts), backward ? kThreads<true> : kThreads<false>, smem, stream>>>(w);
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
    Plan p{};
    p.lanes = lanes;
    share_out(&p, (int64_t)a.B * a.L, a.Hq + a.Hk, true, true);
    most = std::max(most, (size_t)p.ctas * p.parts * (a.Hk > 0 ? 2 : 1));
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
    if (backward && dw[i] != nullptr && heads[i] > 0) {
      any = true;
      s.part = at;
      sums.part[i] = at;
      sums.out[i] = dw[i];
      sums.n[i] = p.ctas * p.parts;
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
  w.Hq = a.Hq;
  w.heads = a.Hq + a.Hk;
  w.share = p.share;
  w.lanes = p.lanes;
  w.items = p.items;
  w.halves = a.halves;
  w.eps = a.eps;
  cudaError_t e = bf16 ? run_type<__nv_bfloat16>(w, p, backward, stream) : run_type<float>(w, p, backward, stream);
  if (e != cudaSuccess || !any) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((a.d + 31) / 32, 2);
  cfg.blockDim = dim3(32 * kSumRows);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, qk_norm_sum_kernel, sums, a.d);
}

}  // namespace favor
