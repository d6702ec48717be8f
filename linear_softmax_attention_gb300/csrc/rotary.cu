// Rotation of queries and keys by positions on one to four axes.
//
// Bound by memory: every channel is read and written once.  A thread takes one
// piece of a token's channels, 16 bytes or two elements (two pieces where the
// pairs are halves apart), in every head of its share: the sines and cosines
// of the token are formed once and used for all of them, and the heads' loads
// are in flight together.  The heads are shared out over more threads only
// where the tokens are few.
//
// Measured (one GB300; copy rate 6779 GB/s): 2 x 12288 tokens x (8 + 8) heads
// of 64 fp32 34.0 us, 5.9 TB/s; 65536 tokens x (16 + 4) heads of 128 bf16 on
// three axes 105 us, 6.4 TB/s.  With one head a token's sines are not shared
// (65536 x (1 + 1) heads of 64 bf16: 12.6 us, 2.7 TB/s).
#include <algorithm>

#include "ops.cuh"

namespace favor {
namespace {

constexpr int kThreads = 256;
// heads of a thread whose loads are in flight together
template <int E> constexpr int kHeadsOf = E > 2 ? 4 : 8;

// Sine and cosine of a pair's angle.  The position times the pair's fraction of
// a turn per unit, in 64-bit fixed point, wraps to the exact fraction of a
// turn, of which the upper 32 bits are kept.  The nearest quarter turn is taken
// off exactly, in whole numbers; what is left, z in [-pi/4, pi/4], goes into
// the Taylor series of sin (to z^9) and cos (to z^10), whose remainders there
// are below 2e-9 and 2e-10, and the quarters turn the two.
__device__ __forceinline__ void sine_cosine(int32_t pos, uint64_t per_unit, float* sn, float* cs) {
  const uint64_t turn = static_cast<uint64_t>(static_cast<int64_t>(pos)) * per_unit;
  const uint32_t u = static_cast<uint32_t>(turn >> 32);
  const uint32_t quarter = (u + (1u << 29)) >> 30;
  const float z = static_cast<float>(static_cast<int32_t>(u - (quarter << 30))) * (6.283185307179586f * 0x1p-32f);
  const float z2 = z * z;
  float s = 1.f / 362880;
  s = fmaf(s, z2, -1.f / 5040);
  s = fmaf(s, z2, 1.f / 120);
  s = fmaf(s, z2, -1.f / 6);
  s = fmaf(s * z2, z, z);
  float c = -1.f / 3628800;
  c = fmaf(c, z2, 1.f / 40320);
  c = fmaf(c, z2, -1.f / 720);
  c = fmaf(c, z2, 1.f / 24);
  c = fmaf(c, z2, -0.5f);
  c = fmaf(c, z2, 1.f);
  const bool odd = quarter & 1;
  const float a = odd ? c : s, b = odd ? s : c;
  *sn = __uint_as_float(__float_as_uint(a) ^ ((quarter & 2) << 30));
  *cs = __uint_as_float(__float_as_uint(b) ^ (((quarter + 1) & 2) << 30));
}

struct Axes {
  int end[FAVOR_ROTARY_MAX_AXES];     // pairs of the axes up to and with each
};

struct Shared {                       // what q's and k's heads have in common
  Strides is, os;
  const void* in;
  void* out;
};

// E elements side by side
template <typename T, int E> struct Piece;
template <> struct Piece<float, 4> {
  using Raw = float4;
  static __device__ __forceinline__ void unpack(const Raw& r, float* f) {
    f[0] = r.x;
    f[1] = r.y;
    f[2] = r.z;
    f[3] = r.w;
  }
  static __device__ __forceinline__ Raw pack(const float* f) { return make_float4(f[0], f[1], f[2], f[3]); }
};
template <> struct Piece<__nv_bfloat16, 8> {
  using Raw = uint4;
  static __device__ __forceinline__ void unpack(const Raw& r, float* f) {
    const unsigned w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ Raw pack(const float* f) {
    unsigned w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const unsigned*>(&v);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

template <> struct Piece<float, 2> {
  using Raw = float2;
  static __device__ __forceinline__ void unpack(const Raw& r, float* f) {
    f[0] = r.x;
    f[1] = r.y;
  }
  static __device__ __forceinline__ Raw pack(const float* f) { return make_float2(f[0], f[1]); }
};
template <> struct Piece<__nv_bfloat16, 2> {
  using Raw = unsigned;
  static __device__ __forceinline__ void unpack(const Raw& r, float* f) {
    f[0] = __uint_as_float(r << 16);
    f[1] = __uint_as_float(r & 0xffff0000u);
  }
  static __device__ __forceinline__ Raw pack(const float* f) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(f[0], f[1]);
    return *reinterpret_cast<const unsigned*>(&v);
  }
};

struct Work {
  Shared q, k;
  const int32_t* pos;
  const uint64_t* table;
  Axes ax;
  FastDiv l, items;                   // tokens of a row; pieces (pairs of pieces) of a token
  int tokens, per_cta, pos_B, L, P, Hq, heads, share;
  float sign;
};

// a token's channels in the first head of q or k
template <typename T>
struct Token {
  const T* in;
  T* out;
  __device__ __forceinline__ Token(const Shared& s, int b, int t)
      : in(static_cast<const T*>(s.in) + b * s.is.b + t * s.is.l),
        out(static_cast<T*>(s.out) + b * s.os.b + t * s.os.l) {}
};

// A token's position on the axis of pair p; `axis` and `at`: of the pair before
// (-1: none), so that a thread loads once per axis
__device__ __forceinline__ void position(const Work& w, int b, int t, int p, int* axis, int32_t* at) {
  const int a = (p >= w.ax.end[0]) + (p >= w.ax.end[1]) + (p >= w.ax.end[2]);
  if (a == *axis) return;
  *axis = a;
  *at = w.pos[((int64_t)a * w.pos_B + (w.pos_B > 1 ? b : 0)) * w.L + t];
}

template <typename T, int E, bool HALVES>
__global__ void __launch_bounds__(kThreads) rotary_pieces_kernel(Work w) {
  using P = Piece<T, E>;
  using Raw = typename P::Raw;
  constexpr int N = HALVES ? E : E / 2;                // pairs of a thread
  constexpr int kHeads = kHeadsOf<E>;
  const int items = w.items.d;
  const int within = items <= kThreads ? w.items.div(threadIdx.x) : 0;
  const int64_t token = (int64_t)blockIdx.x * w.per_cta + within;
  if (within >= w.per_cta || token >= w.tokens) return;
  const int b = (int)w.l.div((uint32_t)token), t = (int)token - b * w.L;
  const int h0 = blockIdx.y * w.share, h1 = h0 + min(w.share, w.heads - h0);
  const Token<T> q(w.q, b, t), k(w.k, b, t);
  for (int item = threadIdx.x - within * items; item < items; item += kThreads) {
    const int turning = HALVES ? w.P / E : 2 * w.P / E;
    const bool turns = item < turning;
    // first channel of the piece, and of the second half's
    const int c0 = HALVES && !turns ? 2 * w.P + (item - turning) * E : item * E, c1 = c0 + w.P;
    float cs[N], sn[N];
    int axis = -1;
    int32_t at = 0;
    if (turns) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int p = HALVES ? c0 + i : c0 / 2 + i;
        position(w, b, t, p, &axis, &at);
        sine_cosine(at, w.table[p], &sn[i], &cs[i]);
        sn[i] *= w.sign;
      }
    }
    for (int hb = h0; hb < h1; hb += kHeads) {
      Raw r0[kHeads], r1[kHeads];
#pragma unroll
      for (int i = 0; i < kHeads; ++i) {
        const int hh = hb + i;
        if (hh < h1) {
          const T* in = hh < w.Hq ? q.in + hh * w.q.is.h : k.in + (hh - w.Hq) * w.k.is.h;
          r0[i] = *reinterpret_cast<const Raw*>(in + c0);
          if (HALVES && turns) r1[i] = *reinterpret_cast<const Raw*>(in + c1);
        }
      }
#pragma unroll
      for (int i = 0; i < kHeads; ++i) {
        const int hh = hb + i;
        if (hh < h1) {
          T* out = hh < w.Hq ? q.out + hh * w.q.os.h : k.out + (hh - w.Hq) * w.k.os.h;
          if (turns) {
            float u[E], v[E], a[E], c[E];
            P::unpack(r0[i], u);
            if constexpr (HALVES) {
              P::unpack(r1[i], v);
#pragma unroll
              for (int j = 0; j < E; ++j) {
                a[j] = u[j] * cs[j] - v[j] * sn[j];
                c[j] = u[j] * sn[j] + v[j] * cs[j];
              }
              *reinterpret_cast<Raw*>(out + c1) = P::pack(c);
            } else {
#pragma unroll
              for (int j = 0; j < N; ++j) {
                a[2 * j] = u[2 * j] * cs[j] - u[2 * j + 1] * sn[j];
                a[2 * j + 1] = u[2 * j] * sn[j] + u[2 * j + 1] * cs[j];
              }
            }
            *reinterpret_cast<Raw*>(out + c0) = P::pack(a);
          } else {
            *reinterpret_cast<Raw*>(out + c0) = r0[i];
          }
        }
      }
    }
  }
}

// Any strides and sizes: a thread per pair, or channel behind the pairs
template <typename T>
__global__ void __launch_bounds__(kThreads) rotary_pairs_kernel(Work w, bool halves) {
  constexpr int kHeads = kHeadsOf<1>;
  const int items = w.items.d;
  const int within = items <= kThreads ? w.items.div(threadIdx.x) : 0;
  const int64_t token = (int64_t)blockIdx.x * w.per_cta + within;
  if (within >= w.per_cta || token >= w.tokens) return;
  const int b = (int)w.l.div((uint32_t)token), t = (int)token - b * w.L;
  const int h0 = blockIdx.y * w.share, h1 = h0 + min(w.share, w.heads - h0);
  const Token<T> q(w.q, b, t), k(w.k, b, t);
  for (int p = threadIdx.x - within * items; p < items; p += kThreads) {
    const bool turns = p < w.P;
    const int iu = !turns ? p + w.P : halves ? p : 2 * p, iv = !turns ? iu : halves ? p + w.P : 2 * p + 1;
    float cs = 1.f, sn = 0.f;
    if (turns) {
      int axis = -1;
      int32_t at = 0;
      position(w, b, t, p, &axis, &at);
      sine_cosine(at, w.table[p], &sn, &cs);
      sn *= w.sign;
    }
    for (int hb = h0; hb < h1; hb += kHeads) {
      T u[kHeads], v[kHeads];
#pragma unroll
      for (int i = 0; i < kHeads; ++i) {
        const int hh = hb + i;
        if (hh < h1) {
          const T* in = hh < w.Hq ? q.in + hh * w.q.is.h : k.in + (hh - w.Hq) * w.k.is.h;
          u[i] = in[iu];
          v[i] = in[iv];
        }
      }
#pragma unroll
      for (int i = 0; i < kHeads; ++i) {
        const int hh = hb + i;
        if (hh < h1) {
          T* out = hh < w.Hq ? q.out + hh * w.q.os.h : k.out + (hh - w.Hq) * w.k.os.h;
          if (turns) {
            const float x = to_f32(u[i]), y = to_f32(v[i]);
            out[iu] = from_f32<T>(x * cs - y * sn);
            out[iv] = from_f32<T>(x * sn + y * cs);
          } else {
            out[iu] = u[i];
          }
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, bool bf16, int piece, cudaStream_t stream) {
  Work w{};
  w.q = Shared{a.qs, a.qos, a.q, a.qo};
  w.k = Shared{a.ks, a.kos, a.k, a.ko};
  w.pos = a.pos;
  w.table = a.table;
  int end = 0;
  for (int i = 0; i < FAVOR_ROTARY_MAX_AXES; ++i) w.ax.end[i] = end += i < a.n_axes ? a.sections[i] : 0;
  w.l = FastDiv((uint32_t)a.L);
  w.tokens = a.B * a.L;
  w.pos_B = a.pos_B;
  w.L = a.L;
  w.P = a.pairs;
  w.Hq = a.Hq;
  w.heads = a.Hq + a.Hk;
  w.sign = a.inverse ? -1.f : 1.f;
  // Pieces of 16 bytes, else of two elements, where the rows and each half of
  // the pairs (all of them, where they are side by side) are made of whole
  // ones, else pair by pair (16384 x 16 heads of 128 bf16: 31.2, 32.8 and 43.2 us
  // for halves, 31.0, 38.4 and 43.7 for adjacent pairs).
  const int e = bf16 ? 2 : 4;
  auto whole = [&](int n) { return piece >= n * e && (a.halves ? a.pairs % n == 0 : 2 * a.pairs % n == 0); };
  const int E = whole(16 / e) ? 16 / e : whole(2) ? 2 : 1;
  const int items = E == 1 ? a.d - a.pairs : a.halves ? a.pairs / E + (a.d - 2 * a.pairs) / E : a.d / E;
  w.items = FastDiv((uint32_t)items);
  w.per_cta = std::max(1, kThreads / items);
  // Enough threads for every SM's 2048: fewer heads each where tokens are few
  // (256 tokens x 16 heads of 64 bf16: 3.3 us, with all heads in one thread
  // 7.0; 512 tokens x 32 heads of 128: 5.9 against 11.4).
  const int64_t threads = (int64_t)w.tokens * items, want = (int64_t)sm_count() * 2048;
  const int64_t parts = std::min<int64_t>(std::min(w.heads, 65535), std::max<int64_t>(1, want / threads));
  w.share = (int)((w.heads + parts - 1) / parts);
  const dim3 grid((unsigned)(((int64_t)w.tokens + w.per_cta - 1) / w.per_cta),
                  (unsigned)(((int64_t)w.heads + w.share - 1) / w.share));
  using B16 = __nv_bfloat16;
  if (E == 1) {
    if (bf16) rotary_pairs_kernel<B16><<<grid, kThreads, 0, stream>>>(w, a.halves);
    else rotary_pairs_kernel<float><<<grid, kThreads, 0, stream>>>(w, a.halves);
  } else if (E == 2) {
    if (bf16 && a.halves) rotary_pieces_kernel<B16, 2, true><<<grid, kThreads, 0, stream>>>(w);
    else if (bf16) rotary_pieces_kernel<B16, 2, false><<<grid, kThreads, 0, stream>>>(w);
    else if (a.halves) rotary_pieces_kernel<float, 2, true><<<grid, kThreads, 0, stream>>>(w);
    else rotary_pieces_kernel<float, 2, false><<<grid, kThreads, 0, stream>>>(w);
  } else {
    if (bf16 && a.halves) rotary_pieces_kernel<B16, 8, true><<<grid, kThreads, 0, stream>>>(w);
    else if (bf16) rotary_pieces_kernel<B16, 8, false><<<grid, kThreads, 0, stream>>>(w);
    else if (a.halves) rotary_pieces_kernel<float, 4, true><<<grid, kThreads, 0, stream>>>(w);
    else rotary_pieces_kernel<float, 4, false><<<grid, kThreads, 0, stream>>>(w);
  }
  return cudaGetLastError();
}

}  // namespace favor
