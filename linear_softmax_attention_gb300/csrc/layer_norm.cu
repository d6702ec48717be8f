// Layer norm over the last axis, forward and backward with the reduction of
// the weight's gradient.
//
// Bound by memory: a row is read once, kept in the thread (at most 16 values of
// it), its mean and then its centred second moment summed from there, and
// written once; the backward pass recomputes both from x instead of reading
// them.  Rows of up to 512 values belong to a group of 4 to 32 lanes of a
// warp, longer ones to a CTA.  The CTAs walk the rows with a stride; each
// thread copies its pieces of the next rows ahead into its own places in
// shared memory (48 to 64 KB in flight per SM, which registers alone could not
// hold), while gamma and beta, and in the backward pass the columns' sums,
// stay in the thread, too.  They are in registers but where 16 values meet a
// limit of 64 of them (CTAs of more than 512 threads: rows above 8192), or come
// one by one (odd rows of 257 to 512 values and from 1025 on): the backward pass
// then spills 350 to 960 bytes a thread, the forward pass up to 200.
//
// Measured (one GB300; copy rate 6779 GB/s): 65536 x 16 rows of 128 bf16 94 us
// forward, 5.7 TB/s (98 us out of a [B, L, 3, H, d] buffer), 123 us backward,
// 6.6 TB/s; 32768 rows of 512 fp32 22.9 and 35.6 us, 5.9 and 5.7 TB/s, bf16
// 13.2 and 24.8 us, of which the two launches, the joins of the columns' sums
// and the second kernel are about 7.  Small calls are bound by their launches
// (8 rows of 512: 2.7 us; backward of 64 rows: 5.1).  480 MB by width, forward
// and backward (floors 142 and 212 us): fp32 2048 to 8192 152 to 154 and 214 to
// 221 us, 12288 151 and 406, 333 288 and 830, 771 237 and 465, 1025 312 and 1105,
// 4099 287 and 1376; bf16 2048 to 8192 149 to 163 and 233 to 272, 12288 161 and
// 535, 333 542 and 2096, 771 449 and 875, 1025 548 and 2605, 4099 542 and 3176.
#include <algorithm>

#include "ops.cuh"
#include "tc_ptx.cuh"

namespace favor {
namespace {

constexpr int kWarps = 8;             // of a CTA that shares its rows out by groups of lanes
constexpr int kMaxValues = 16;        // of a row in one thread
constexpr int kSumRows = 32, kSumThreads = 32 * kSumRows;

// VW values side by side: 16 bytes, two elements or one
template <typename T, int VW> struct Piece;
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
template <> struct Piece<float, 1> {
  using Raw = float;
  static __device__ __forceinline__ void unpack(const Raw& r, float* f) { f[0] = r; }
  static __device__ __forceinline__ Raw pack(const float* f) { return f[0]; }
};
template <> struct Piece<__nv_bfloat16, 1> {
  using Raw = __nv_bfloat16;
  static __device__ __forceinline__ void unpack(const Raw& r, float* f) { f[0] = __bfloat162float(r); }
  static __device__ __forceinline__ Raw pack(const float* f) { return __float2bfloat16_rn(f[0]); }
};

// How the rows are shared out: `lanes` threads per row (4 to 32, or a CTA's
// 64 to 1024), groups of them per CTA, CTAs.
struct Plan {
  int lanes, threads, groups, ctas;
};

// Sums of N values over the threads of a row; every one of them gets them.
// scratch: [32][N] for a CTA's rows; a call must not follow one on the same
// scratch with no call on another between them, whose barrier the reads need.
template <int N, int CTA>
__device__ __forceinline__ void row_sum(float (&v)[N], int lanes, float* scratch) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (CTA > 0) {
      v[i] = warp_sum(v[i]);
    } else {
      for (int o = lanes >> 1; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    }
  }
  if constexpr (CTA > 0) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) scratch[warp * N + i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = warp_sum(lane < warps ? scratch[lane * N + i] : 0.f);
  }
}

// A row's pieces in this thread: piece j holds the columns from
// (j lanes + lane) VW on.  Those of the next S rows of N tensors are on their
// way, in the thread's own places in shared memory (bf16 elements one by one,
// which no asynchronous copy takes, in registers: one row ahead).
template <typename T, int VW, int NV, int CTA>
struct Kind {};
template <typename T, int VW, int NV, int N>
struct Ahead {
  using Raw = typename Piece<T, VW>::Raw;
  static constexpr bool kAsync = sizeof(Raw) >= 4;
  static constexpr int S = !kAsync ? 1 : N == 2 ? (NV * VW * sizeof(T) <= 16 ? 3 : NV * VW * sizeof(T) <= 32 ? 2 : 1)
                                                : (NV * VW * sizeof(T) <= 16 ? 4 : NV * VW * sizeof(T) <= 32 ? 2 : 1);
  static constexpr size_t kBytes = kAsync ? (size_t)S * N * NV * sizeof(Raw) : 0;   // per thread
  Raw regs[kAsync ? 1 : N][kAsync ? 1 : NV];
  Raw* mine;
  int stage;
  __device__ __forceinline__ Ahead(void* ring) : mine(static_cast<Raw*>(ring) + threadIdx.x), stage(0) {}
  __device__ __forceinline__ Raw* place(int n, int j) const {
    return mine + ((stage * N + n) * NV + j) * (int)blockDim.x;
  }
  // starts tensor n's copies of a row (none of them where !in)
  __device__ __forceinline__ void fetch(int n, const T* any, const T* row, int lane, int lanes, int d, bool in) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * lanes + lane) * VW;
      const bool here = in && c < d;
      if constexpr (kAsync) {
        const uint32_t to = tc::smem_addr(place(n, j));
        const T* from = here ? row + c : any;         // a source for the copy of no bytes: zeros
        if constexpr (sizeof(Raw) == 16)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(here ? 16 : 0)
                       : "memory");
        else
          asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(to), "l"(from), "n"(sizeof(Raw)),
                       "r"(here ? (int)sizeof(Raw) : 0)
                       : "memory");
      } else {
        regs[n][j] = here ? *reinterpret_cast<const Raw*>(row + c) : Raw{};
      }
    }
  }
  __device__ __forceinline__ void commit() {
    if constexpr (kAsync) asm volatile("cp.async.commit_group;" ::: "memory");
  }
  __device__ __forceinline__ void wait() {
    if constexpr (kAsync) asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory");
  }
  // nothing is on its way any more
  __device__ __forceinline__ void drain() {
    if constexpr (kAsync) asm volatile("cp.async.wait_group 0;" ::: "memory");
  }
  __device__ __forceinline__ void take(int n, float (&x)[NV][VW]) const {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if constexpr (kAsync) Piece<T, VW>::unpack(*place(n, j), x[j]);
      else Piece<T, VW>::unpack(regs[n][j], x[j]);
    }
  }
  __device__ __forceinline__ void advance() { stage = stage + 1 == S ? 0 : stage + 1; }
};

// Values two by two through the packed fp32 instructions, one by one where a
// piece is one element
template <int VW> struct Each {
  template <typename F>
  static __device__ __forceinline__ void go(F&& f) {
    if constexpr (VW > 1) {
#pragma unroll
      for (int i = 0; i < VW; i += 2) f(i);
    } else {
      f(0);
    }
  }
  // (a pair of) x at i, and back; the second of a single value is 0
  static __device__ __forceinline__ float2 get(const float (&x)[VW], int i) {
    return VW > 1 ? make_float2(x[i], x[VW > 1 ? i + 1 : 0]) : make_float2(x[0], 0.f);
  }
  static __device__ __forceinline__ void put(float (&x)[VW], int i, float2 v) {
    x[i] = v.x;
    if (VW > 1) x[VW > 1 ? i + 1 : 0] = v.y;
  }
};
__device__ __forceinline__ float2 twice(float x) { return make_float2(x, x); }

// x becomes x - mean (0 behind the row); returns this thread's part of the sum
// of its squares
template <int VW, int NV, int CTA>
__device__ __forceinline__ float centre(float (&x)[NV][VW], int lane, int lanes, int d, float inv_d, float* scratch) {
  using E = Each<VW>;
  float2 s2 = twice(0.f);
#pragma unroll
  for (int j = 0; j < NV; ++j) E::go([&](int i) { s2 = add2(s2, E::get(x[j], i)); });
  float s[1] = {s2.x + s2.y};
  row_sum<1, CTA>(s, lanes, scratch);
  const float2 mean = twice(-s[0] * inv_d);
  const bool whole = NV * VW * lanes == d;            // no thread has places behind the row
  float2 v2 = twice(0.f);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const bool in = whole || (j * lanes + lane) * VW < d;
    E::go([&](int i) {
      float2 c = add2(E::get(x[j], i), mean);
      if (VW == 1) c.y = 0.f;
      if (!in) c = twice(0.f);
      E::put(x[j], i, c);
      v2 = fma2(c, c, v2);
    });
  }
  return v2.x + v2.y;
}

// VW fp32 values at p, by 16 bytes where they lie so
template <int VW>
__device__ __forceinline__ void load_values(float (&w)[VW], const float* p, bool by16) {
  if constexpr (VW >= 4) {
    if (by16) {
#pragma unroll
      for (int i = 0; i < VW; i += 4) {
        const float4 v = *reinterpret_cast<const float4*>(p + i);
        w[i] = v.x;
        w[i + 1] = v.y;
        w[i + 2] = v.z;
        w[i + 3] = v.w;
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < VW; ++i) w[i] = p[i];
}
template <int VW>
__device__ __forceinline__ void store_values(float* p, const float (&w)[VW]) {   // 16-byte aligned where VW >= 4
  if constexpr (VW >= 4) {
#pragma unroll
    for (int i = 0; i < VW; i += 4) *reinterpret_cast<float4*>(p + i) = make_float4(w[i], w[i + 1], w[i + 2], w[i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < VW; ++i) p[i] = w[i];
  }
}
template <int VW, int NV>
__device__ __forceinline__ void load_weights(float (&w)[NV][VW], const float* p, int lane, int lanes, int d,
                                             float none) {
  const bool by16 = reinterpret_cast<uintptr_t>(p) % 16 == 0;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * lanes + lane) * VW;
    if (p != nullptr && c < d) {
      load_values<VW>(w[j], p + c, by16);
    } else {
#pragma unroll
      for (int i = 0; i < VW; ++i) w[j][i] = none;
    }
  }
}

// 1 / sqrt(x); NaN for infinity: a variance that has left fp32 gives no zeros
__device__ __forceinline__ float inverse_root(float x) { return fmaf(x, 0.f, rsqrtf(x)); }

template <typename T, int VW, int NV, int CTA>
__global__ void __launch_bounds__(CTA > 0 ? CTA : 32 * kWarps, CTA > 256 ? 1 : NV * VW > 8 ? 3 : 4)
    norm_fwd_kernel(NormArgs p, Rows rows, uint32_t n, Plan plan) {
  using P = Piece<T, VW>;
  using A = Ahead<T, VW, NV, 1>;
  using E = Each<VW>;
  __shared__ float scratch[64];
  extern __shared__ __align__(16) float ring[];
  const int lanes = plan.lanes, lane = CTA > 0 ? threadIdx.x : threadIdx.x & (lanes - 1);
  const uint32_t group = CTA > 0 ? blockIdx.x : blockIdx.x * plan.groups + threadIdx.x / lanes;
  const uint32_t stride = (uint32_t)plan.ctas * plan.groups;
  const float inv_d = 1.f / p.d;
  const T* x0 = static_cast<const T*>(p.x);
  A ahead(ring);
  auto fetch = [&](uint32_t r) {
    ahead.fetch(0, x0, x0 + rows.offset(0, r), lane, lanes, p.d, r < n);
    ahead.commit();
  };
#pragma unroll
  for (int s = 0; s < A::S; ++s) {
    fetch(group + s * stride);
    ahead.advance();
  }
  float w[NV][VW], z[NV][VW];
  load_weights<VW, NV>(w, p.gamma, lane, lanes, p.d, 1.f);
  load_weights<VW, NV>(z, p.beta, lane, lanes, p.d, 0.f);
  const bool affine = p.gamma != nullptr || p.beta != nullptr;
  // every thread of a warp (of a CTA) walks as long as its first one
  const uint32_t first = CTA > 0 ? group : group - (threadIdx.x & 31) / lanes;
  for (uint32_t r = group, r0 = first; r0 < n; r += stride, r0 += stride) {
    float x[NV][VW];
    ahead.wait();
    ahead.take(0, x);
    fetch(r + A::S * stride);
    ahead.advance();
    float v[1] = {centre<VW, NV, CTA>(x, lane, lanes, p.d, inv_d, scratch)};
    row_sum<1, CTA>(v, lanes, scratch + 32);
    const float rstd = inverse_root(fmaf(v[0], inv_d, p.eps));
    T* y = static_cast<T*>(p.y) + rows.offset(1, r);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * lanes + lane) * VW;
      E::go([&](int i) {
        float2 v = mul2(E::get(x[j], i), twice(rstd));
        if (affine) v = fma2(v, E::get(w[j], i), E::get(z[j], i));
        E::put(x[j], i, v);
      });
      if (r < n && c < p.d) *reinterpret_cast<typename P::Raw*>(y + c) = P::pack(x[j]);
    }
  }
  ahead.drain();
}

// dx, and the sums of dy xh and dy over the CTA's rows, [CTA][2][d] in `part`
// (NULL: not wanted).
template <typename T, int VW, int NV, int CTA>
__global__ void __launch_bounds__(CTA > 0 ? CTA : 32 * kWarps, CTA > 256 ? 1 : NV * VW <= 4 ? 4 : 2)
    norm_bwd_kernel(NormArgs p, Rows rows, uint32_t n, Plan plan, float* part) {
  using P = Piece<T, VW>;
  using A = Ahead<T, VW, NV, 2>;
  using E = Each<VW>;
  __shared__ float scratch[32 + 3 * 32];
  extern __shared__ __align__(16) float ring[];
  const int lanes = plan.lanes, lane = CTA > 0 ? threadIdx.x : threadIdx.x & (lanes - 1);
  const uint32_t group = CTA > 0 ? blockIdx.x : blockIdx.x * plan.groups + threadIdx.x / lanes;
  const uint32_t stride = (uint32_t)plan.ctas * plan.groups;
  const float inv_d = 1.f / p.d;
  const T *x0 = static_cast<const T*>(p.x), *dy0 = static_cast<const T*>(p.dy);
  A ahead(ring);
  auto fetch = [&](uint32_t r) {
    ahead.fetch(0, x0, x0 + rows.offset(0, r), lane, lanes, p.d, r < n);
    ahead.fetch(1, dy0, dy0 + rows.offset(1, r), lane, lanes, p.d, r < n);
    ahead.commit();
  };
#pragma unroll
  for (int s = 0; s < A::S; ++s) {
    fetch(group + s * stride);
    ahead.advance();
  }
  float w[NV][VW], dw[NV][VW], dz[NV][VW];
  load_weights<VW, NV>(w, p.gamma, lane, lanes, p.d, 1.f);
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < VW; ++i) dw[j][i] = dz[j][i] = 0.f;
  const uint32_t first = CTA > 0 ? group : group - (threadIdx.x & 31) / lanes;
  for (uint32_t r = group, r0 = first; r0 < n; r += stride, r0 += stride) {
    float x[NV][VW], dy[NV][VW];
    ahead.wait();
    ahead.take(0, x);
    ahead.take(1, dy);
    fetch(r + A::S * stride);
    ahead.advance();
    // one more sum of three values: (x - mean)^2, n = dy gamma, n (x - mean)
    float s[3] = {centre<VW, NV, CTA>(x, lane, lanes, p.d, inv_d, scratch), 0.f, 0.f};
    float2 s1 = twice(0.f), s2 = twice(0.f);
#pragma unroll
    for (int j = 0; j < NV; ++j)
      E::go([&](int i) {                              // dy is 0 behind the row
        const float2 g = E::get(dy[j], i), m = mul2(g, E::get(w[j], i));
        E::put(dz[j], i, add2(E::get(dz[j], i), g));
        s1 = add2(s1, m);
        s2 = fma2(m, E::get(x[j], i), s2);
      });
    s[1] = s1.x + s1.y;
    s[2] = s2.x + s2.y;
    row_sum<3, CTA>(s, lanes, scratch + 32);
    const float rstd = inverse_root(fmaf(s[0], inv_d, p.eps));
    const float2 m1 = twice(-s[1] * inv_d), m2 = twice(-s[2] * rstd * inv_d);
    T* dx = static_cast<T*>(p.dx) + rows.offset(2, r);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * lanes + lane) * VW;
      E::go([&](int i) {
        const float2 xh = mul2(E::get(x[j], i), twice(rstd)), g = E::get(dy[j], i);
        E::put(dw[j], i, fma2(g, xh, E::get(dw[j], i)));
        E::put(x[j], i, mul2(fma2(xh, m2, fma2(g, E::get(w[j], i), m1)), twice(rstd)));
      });
      if (r < n && c < p.d) *reinterpret_cast<typename P::Raw*>(dx + c) = P::pack(x[j]);
    }
  }
  ahead.drain();
  if (part == nullptr) return;
  // the kernel that adds the CTAs' sums may take its place and wait
  asm volatile("griddepcontrol.launch_dependents;");
  float* out = part + (size_t)blockIdx.x * 2 * p.d;
  if constexpr (CTA == 0) {
    // the groups' sums side by side in the ring's place, [groups][2][d], then
    // added up column by column
    __syncthreads();
    float* sums = ring + (threadIdx.x / lanes) * 2 * p.d;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * lanes + lane) * VW;
      if (c < p.d) {
        store_values<VW>(sums + c, dw[j]);
        store_values<VW>(sums + p.d + c, dz[j]);
      }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * p.d; c += blockDim.x) {
      float v = ring[c];
#pragma unroll 8
      for (int g = 1; g < plan.groups; ++g) v += ring[g * 2 * p.d + c];
      out[c] = v;
    }
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * lanes + lane) * VW;
      if (c < p.d) {
        store_values<VW>(out + c, dw[j]);
        store_values<VW>(out + p.d + c, dz[j]);
      }
    }
  }
}

// The CTAs' sums in their order: a block per 32 columns of [2 d]
__global__ void __launch_bounds__(kSumThreads) norm_sum_kernel(const float* part, int ctas, int d, float* dgamma,
                                                               float* dbeta) {
  __shared__ float s[kSumRows][32];
  const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  tc::griddep_wait();
  float v = 0.f;
  if (c < 2 * d) {
#pragma unroll 8
    for (int i = row; i < ctas; i += kSumRows) v += part[(size_t)i * 2 * d + c];
  }
  s[row][lane] = v;
  __syncthreads();
  if (row == 0 && c < 2 * d) {
#pragma unroll
    for (int i = 1; i < kSumRows; ++i) v += s[i][lane];
    float* out = c < d ? dgamma : dbeta;
    if (out != nullptr) out[c < d ? c : c - d] = v;
  }
}

// Values of a piece: 16 bytes where every tensor's rows are made of them,
// else two elements, else one.  16384 x 16 rows of 128 bf16: 29.0, 39.8 and 52.7
// us forward, 43.5, 66.6 and 103.9 backward.
int piece_values(bool bf16, int piece) { return piece >= 16 ? (bf16 ? 8 : 4) : piece >= (bf16 ? 4 : 8) ? 2 : 1; }

// CTAs: as many as the registers let be resident, so that every one walks
// about the same number of rows
Plan make_plan(int64_t rows, int d, int vw, bool backward) {
  const int pieces = (d + vw - 1) / vw, per = kMaxValues / vw;     // pieces of a row, of a thread at most
  Plan p;
  if (pieces <= 32 * per) {
    // 16-byte pieces: as many values a thread as there may be; what a row costs
    // beside them (its address, sums over lanes, root) is then shared by the
    // most of them.  16 values against 8 (65536 x 16 rows of 128 bf16): 94
    // against 126 us.  Smaller pieces: 8 values, so that the lanes' accesses
    // stay near to one another (3 x 10 x 36507 rows of 106 fp32, backward: 311
    // us, with 16 values 688, with 4 476).
    p.lanes = 4;
    while (p.lanes < 32 && p.lanes * (vw >= 4 ? per : per / 2) < pieces) p.lanes *= 2;
    p.threads = 32 * kWarps;
    p.groups = p.threads / p.lanes;
  } else {
    // smaller pieces: 4 values a thread while 256 threads hold the row (3333
    // rows of 771 fp32, backward: 19.4 us, with 16 values 23.2)
    const int most = vw <= 2 && pieces <= 256 * (4 / vw) ? 4 / vw : per;
    p.threads = p.lanes = ((pieces + most - 1) / most + 31) / 32 * 32;
    p.groups = 1;
  }
  const int values = (pieces + p.lanes - 1) / p.lanes * vw;
  // threads of an SM
  const int resident = p.threads <= 256 && values <= (backward ? 4 : 8) ? 1024 : backward ? 512 : 768;
  const int64_t per_sm = std::max(1, resident / p.threads);
  int64_t ctas = std::min<int64_t>((rows + p.groups - 1) / p.groups, per_sm * sm_count());
  // every CTA's sums are added up after: rows enough for each to make that little
  if (backward) ctas = std::min(ctas, std::max<int64_t>(2 * sm_count(), rows / (8 * p.groups)));
  p.ctas = (int)ctas;
  return p;
}

// (T, VW, NV, CTA) of a plan; CTA: the most threads of a row's CTA, 0 for groups of
// lanes (fewer threads may use more registers)
template <typename F>
cudaError_t dispatch(const Plan& plan, int d, bool bf16, int vw, F&& f) {
  const int nv = ((d + vw - 1) / vw + plan.lanes - 1) / plan.lanes;
#define FAVOR_NORM(T, VW, NV)                           \
  return plan.lanes <= 32    ? f(Kind<T, VW, NV, 0>{})   \
         : plan.lanes <= 256 ? f(Kind<T, VW, NV, 256>{}) \
         : plan.lanes <= 512 ? f(Kind<T, VW, NV, 512>{}) \
                             : f(Kind<T, VW, NV, 1024>{})
  if (bf16 && vw == 8) {
    if (nv <= 1) { FAVOR_NORM(__nv_bfloat16, 8, 1); }
    FAVOR_NORM(__nv_bfloat16, 8, 2);
  }
  if (!bf16 && vw == 4) {
    if (nv <= 1) { FAVOR_NORM(float, 4, 1); }
    if (nv <= 2) { FAVOR_NORM(float, 4, 2); }
    FAVOR_NORM(float, 4, 4);
  }
  if (bf16 && vw == 2) {
    if (nv <= 2) { FAVOR_NORM(__nv_bfloat16, 2, 2); }
    if (nv <= 4) { FAVOR_NORM(__nv_bfloat16, 2, 4); }
    FAVOR_NORM(__nv_bfloat16, 2, 8);
  }
  if (vw == 2) {
    if (nv <= 2) { FAVOR_NORM(float, 2, 2); }
    if (nv <= 4) { FAVOR_NORM(float, 2, 4); }
    FAVOR_NORM(float, 2, 8);
  }
  if (bf16) {
    if (nv <= 4) { FAVOR_NORM(__nv_bfloat16, 1, 4); }
    if (nv <= 8) { FAVOR_NORM(__nv_bfloat16, 1, 8); }
    FAVOR_NORM(__nv_bfloat16, 1, 16);
  }
  if (nv <= 4) { FAVOR_NORM(float, 1, 4); }
  if (nv <= 8) { FAVOR_NORM(float, 1, 8); }
  FAVOR_NORM(float, 1, 16);
#undef FAVOR_NORM
}

template <typename T, int VW, int NV, int CTA>
cudaError_t fwd(Kind<T, VW, NV, CTA>, const NormArgs& a, const Rows& rows, uint32_t n, const Plan& plan,
                cudaStream_t stream) {
  const size_t smem = Ahead<T, VW, NV, 1>::kBytes * plan.threads;
  const auto kernel = norm_fwd_kernel<T, VW, NV, CTA>;
  const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), smem);
  if (e != cudaSuccess) return e;
  kernel<<<plan.ctas, plan.threads, smem, stream>>>(a, rows, n, plan);
  return cudaGetLastError();
}

template <typename T, int VW, int NV, int CTA>
cudaError_t bwd(Kind<T, VW, NV, CTA>, const NormArgs& a, const Rows& rows, uint32_t n, const Plan& plan, float* part,
                cudaStream_t stream) {
  const size_t sums = CTA == 0 ? (size_t)plan.groups * 2 * a.d * sizeof(float) : 0;
  const size_t smem = std::max(Ahead<T, VW, NV, 2>::kBytes * plan.threads, sums);
  const auto kernel = norm_bwd_kernel<T, VW, NV, CTA>;
  const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), smem);
  if (e != cudaSuccess) return e;
  kernel<<<plan.ctas, plan.threads, smem, stream>>>(a, rows, n, plan, part);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_fwd(const NormArgs& a, bool bf16, int piece, cudaStream_t stream) {
  const uint32_t n = (uint32_t)a.B * a.H * a.L;
  const Strides s[2] = {a.xs, a.ys};
  const Rows rows = make_rows(a.B, a.H, a.L, s, 2);
  const int vw = piece_values(bf16, piece);
  const Plan plan = make_plan(n, a.d, vw, false);
  return dispatch(plan, a.d, bf16, vw, [&](auto kind) { return fwd(kind, a, rows, n, plan, stream); });
}

// what any kernel of a shape may write, whatever the tensors' alignment
size_t norm_bwd_workspace_bytes(int64_t rows, int d, bool bf16) {
  int ctas = 0;
  for (const int vw : {bf16 ? 8 : 4, 2, 1}) ctas = std::max(ctas, make_plan(rows, d, vw, true).ctas);
  return (size_t)ctas * 2 * d * sizeof(float);
}

cudaError_t launch_norm_bwd(const NormArgs& a, bool bf16, int piece, float* ws, cudaStream_t stream) {
  const uint32_t n = (uint32_t)a.B * a.H * a.L;
  const Strides s[3] = {a.xs, a.dys, a.dxs};
  const Rows rows = make_rows(a.B, a.H, a.L, s, 3);
  const int vw = piece_values(bf16, piece);
  const Plan plan = make_plan(n, a.d, vw, true);
  const bool sums = a.dgamma != nullptr || a.dbeta != nullptr;
  cudaError_t e = dispatch(plan, a.d, bf16, vw, [&](auto kind) {
    return bwd(kind, a, rows, n, plan, sums ? ws : nullptr, stream);
  });
  if (e != cudaSuccess || !sums) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((2 * a.d + 31) / 32));
  cfg.blockDim = dim3(kSumThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, norm_sum_kernel, static_cast<const float*>(ws), plan.ctas, a.d, a.dgamma, a.dbeta);
}

}  // namespace favor
