// Layer norm over the last axis, forward and backward with the reduction of
// the weight's gradient.
//
// Bound by memory: a row is read once, kept in registers (at most 16 values a
// thread), its mean and then its centred second moment summed from there, and
// written once; the backward pass recomputes both from x instead of reading
// them.  Rows of up to 512 values belong to a group of 4 to 32 lanes of a
// warp, longer ones to a CTA.  The CTAs walk the rows with a stride, the next
// row's loads in flight while one is worked on; gamma and beta, and in the
// backward pass the columns' sums, stay in registers meanwhile.
#include <algorithm>

#include "ops.cuh"
#include "tc_ptx.cuh"

namespace favor {
namespace {

constexpr int kWarps = 8;             // of a CTA that shares its rows out by groups of lanes
constexpr int kMaxValues = 16;        // of a row in one thread
constexpr int kSumRows = 8, kSumThreads = 32 * kSumRows;

// VW values side by side: 16 bytes, or one element
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
// scratch: [2][32][N] for a CTA's rows, flipped by the caller's parity.
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

// One row's values in this thread: piece j holds the columns from
// (j lanes + lane) VW on
template <typename T, int VW, int NV, int CTA>
struct Row {
  using P = Piece<T, VW>;
  using Raw = typename P::Raw;
  Raw raw[NV];
  __device__ __forceinline__ void load(const T* row, int lane, int lanes, int d, bool in) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * lanes + lane) * VW;
      if (in && c < d) raw[j] = *reinterpret_cast<const Raw*>(row + c);
      else raw[j] = Raw{};
    }
  }
};

// mean and 1 / sqrt(var + eps); x becomes x - mean (0 behind the row)
template <int VW, int NV, int CTA>
__device__ __forceinline__ float centre(float (&x)[NV][VW], int lane, int lanes, int d, float inv_d, float eps,
                                        float* scratch) {
  float s[1] = {0.f};
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < VW; ++i) s[0] += x[j][i];
  row_sum<1, CTA>(s, lanes, scratch);
  const float mean = s[0] * inv_d;
  float v[1] = {0.f};
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const bool in = (j * lanes + lane) * VW < d;
#pragma unroll
    for (int i = 0; i < VW; ++i) {
      x[j][i] = in ? x[j][i] - mean : 0.f;
      v[0] = fmaf(x[j][i], x[j][i], v[0]);
    }
  }
  row_sum<1, CTA>(v, lanes, scratch + 32);
  return 1.f / sqrtf(fmaf(v[0], inv_d, eps));
}

template <int VW, int NV>
__device__ __forceinline__ void load_weights(float (&w)[NV][VW], const float* p, int lane, int lanes, int d,
                                             float none) {
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * lanes + lane) * VW;
#pragma unroll
    for (int i = 0; i < VW; ++i) w[j][i] = p != nullptr && c < d ? p[c + i] : none;
  }
}

template <typename T, int VW, int NV, int CTA>
__global__ void __launch_bounds__(CTA > 0 ? CTA : 32 * kWarps) norm_fwd_kernel(NormArgs p, Rows rows, uint32_t n,
                                                                            Plan plan) {
  using P = Piece<T, VW>;
  __shared__ float scratch[64];
  const int lanes = plan.lanes, lane = CTA > 0 ? threadIdx.x : threadIdx.x & (lanes - 1);
  const uint32_t group = CTA > 0 ? blockIdx.x : blockIdx.x * plan.groups + threadIdx.x / lanes;
  const uint32_t stride = (uint32_t)plan.ctas * plan.groups;
  const float inv_d = 1.f / p.d;
  float w[NV][VW], z[NV][VW];
  load_weights<VW, NV>(w, p.gamma, lane, lanes, p.d, 1.f);
  load_weights<VW, NV>(z, p.beta, lane, lanes, p.d, 0.f);
  uint32_t b, h, t;
  Row<T, VW, NV, CTA> next;
  rows.split(group, &b, &h, &t);
  next.load(static_cast<const T*>(p.x) + rows.offset(0, b, h, t), lane, lanes, p.d, group < n);
  // every thread of a warp (of a CTA) walks as long as its first one
  const uint32_t first = CTA > 0 ? group : group - (threadIdx.x & 31) / lanes;
  for (uint32_t r = group, r0 = first; r0 < n; r += stride, r0 += stride) {
    float x[NV][VW];
#pragma unroll
    for (int j = 0; j < NV; ++j) P::unpack(next.raw[j], x[j]);
    T* y = static_cast<T*>(p.y) + rows.offset(1, b, h, t);
    if (r0 + stride < n) {
      rows.split(r + stride, &b, &h, &t);
      next.load(static_cast<const T*>(p.x) + rows.offset(0, b, h, t), lane, lanes, p.d, r + stride < n);
    }
    const float rstd = centre<VW, NV, CTA>(x, lane, lanes, p.d, inv_d, p.eps, scratch);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * lanes + lane) * VW;
#pragma unroll
      for (int i = 0; i < VW; ++i) x[j][i] = fmaf(x[j][i] * rstd, w[j][i], z[j][i]);
      if (r < n && c < p.d) *reinterpret_cast<typename P::Raw*>(y + c) = P::pack(x[j]);
    }
  }
}

// dx, and the sums of dy xh and dy over the CTA's rows, [CTA][2][d] in `part`
// (NULL: not wanted).
template <typename T, int VW, int NV, int CTA>
__global__ void __launch_bounds__(CTA > 0 ? CTA : 32 * kWarps, CTA > 256 ? 1 : 2) norm_bwd_kernel(NormArgs p, Rows rows,
                                                                                     uint32_t n, Plan plan,
                                                                                     float* part) {
  using P = Piece<T, VW>;
  __shared__ float scratch[128];
  extern __shared__ float sums[];                     // [groups / 2][2][d], rows shared out by lanes
  const int lanes = plan.lanes, lane = CTA > 0 ? threadIdx.x : threadIdx.x & (lanes - 1);
  const uint32_t group = CTA > 0 ? blockIdx.x : blockIdx.x * plan.groups + threadIdx.x / lanes;
  const uint32_t stride = (uint32_t)plan.ctas * plan.groups;
  const float inv_d = 1.f / p.d;
  float w[NV][VW], dw[NV][VW], dz[NV][VW];
  load_weights<VW, NV>(w, p.gamma, lane, lanes, p.d, 1.f);
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < VW; ++i) dw[j][i] = dz[j][i] = 0.f;
  uint32_t b, h, t;
  Row<T, VW, NV, CTA> nx, ny;
  auto load = [&](uint32_t r) {
    rows.split(r, &b, &h, &t);
    nx.load(static_cast<const T*>(p.x) + rows.offset(0, b, h, t), lane, lanes, p.d, r < n);
    ny.load(static_cast<const T*>(p.dy) + rows.offset(1, b, h, t), lane, lanes, p.d, r < n);
  };
  load(group);
  const uint32_t first = CTA > 0 ? group : group - (threadIdx.x & 31) / lanes;
  for (uint32_t r = group, r0 = first; r0 < n; r += stride, r0 += stride) {
    float x[NV][VW], dy[NV][VW];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      P::unpack(nx.raw[j], x[j]);
      P::unpack(ny.raw[j], dy[j]);
    }
    T* dx = static_cast<T*>(p.dx) + rows.offset(2, b, h, t);
    if (r0 + stride < n) load(r + stride);
    const float rstd = centre<VW, NV, CTA>(x, lane, lanes, p.d, inv_d, p.eps, scratch);
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < VW; ++i) {
        x[j][i] *= rstd;                              // xh; dy is 0 behind the row
        dw[j][i] = fmaf(dy[j][i], x[j][i], dw[j][i]);
        dz[j][i] += dy[j][i];
        dy[j][i] *= w[j][i];
        s[0] += dy[j][i];
        s[1] = fmaf(dy[j][i], x[j][i], s[1]);
      }
    row_sum<2, CTA>(s, lanes, scratch + 64);
    const float m1 = s[0] * inv_d, m2 = s[1] * inv_d;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * lanes + lane) * VW;
#pragma unroll
      for (int i = 0; i < VW; ++i) x[j][i] = rstd * (dy[j][i] - m1 - x[j][i] * m2);
      if (r < n && c < p.d) *reinterpret_cast<typename P::Raw*>(dx + c) = P::pack(x[j]);
    }
  }
  if (part == nullptr) return;
  if constexpr (CTA == 0) {
    // the groups' sums, halved until the first group has them all
    const int me = threadIdx.x / lanes;
    for (int half = plan.groups >> 1; half > 0; half >>= 1) {
      __syncthreads();
      if (me >= half && me < 2 * half)
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int i = 0; i < VW; ++i) {
            const int c = (j * lanes + lane) * VW + i;
            if (c < p.d) {
              sums[(me - half) * 2 * p.d + c] = dw[j][i];
              sums[(me - half) * 2 * p.d + p.d + c] = dz[j][i];
            }
          }
      __syncthreads();
      if (me < half)
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int i = 0; i < VW; ++i) {
            const int c = (j * lanes + lane) * VW + i;
            if (c < p.d) {
              dw[j][i] += sums[me * 2 * p.d + c];
              dz[j][i] += sums[me * 2 * p.d + p.d + c];
            }
          }
    }
    if (me > 0) return;
  }
  float* out = part + (size_t)blockIdx.x * 2 * p.d;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < VW; ++i) {
      const int c = (j * lanes + lane) * VW + i;
      if (c < p.d) {
        out[c] = dw[j][i];
        out[p.d + c] = dz[j][i];
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

// CTAs: as many as are resident (the backward pass's hold half the SM's
// registers each), so that every one walks about the same number of rows
Plan make_plan(int64_t rows, int d, bool bf16, bool vec, bool backward) {
  const int vw = vec ? (bf16 ? 8 : 4) : 1;
  const int pieces = (d + vw - 1) / vw, per = kMaxValues / vw;     // pieces of a row, of a thread at most
  Plan p;
  int64_t per_sm;
  if (pieces <= 32 * per) {
    p.lanes = 4;
    while (p.lanes < 32 && p.lanes < pieces) p.lanes *= 2;
    p.threads = 32 * kWarps;
    p.groups = p.threads / p.lanes;
    per_sm = backward ? 2 : 6;
  } else {
    p.threads = p.lanes = ((pieces + per - 1) / per + 31) / 32 * 32;
    p.groups = 1;
    per_sm = std::max(1, (backward ? 640 : 1024) / p.threads);
  }
  p.ctas = (int)std::min<int64_t>((rows + p.groups - 1) / p.groups, per_sm * sm_count());
  return p;
}

// (T, VW, NV, CTA) of a plan; CTA: the most threads of a row's CTA, 0 for groups of
// lanes (up to 256 threads may use twice the registers)
template <typename F>
cudaError_t dispatch(const Plan& plan, int d, bool bf16, bool vec, F&& f) {
  const int vw = vec ? (bf16 ? 8 : 4) : 1;
  const int nv = ((d + vw - 1) / vw + plan.lanes - 1) / plan.lanes;
#define FAVOR_NORM(T, VW, NV)                          \
  return plan.lanes <= 32    ? f(Row<T, VW, NV, 0>{})   \
         : plan.lanes <= 256 ? f(Row<T, VW, NV, 256>{}) \
                             : f(Row<T, VW, NV, 1024>{})
  if (bf16 && vec) {
    if (nv <= 1) { FAVOR_NORM(__nv_bfloat16, 8, 1); }
    FAVOR_NORM(__nv_bfloat16, 8, 2);
  }
  if (bf16) {
    if (nv <= 4) { FAVOR_NORM(__nv_bfloat16, 1, 4); }
    FAVOR_NORM(__nv_bfloat16, 1, 16);
  }
  if (vec) {
    if (nv <= 1) { FAVOR_NORM(float, 4, 1); }
    if (nv <= 2) { FAVOR_NORM(float, 4, 2); }
    FAVOR_NORM(float, 4, 4);
  }
  if (nv <= 4) { FAVOR_NORM(float, 1, 4); }
  FAVOR_NORM(float, 1, 16);
#undef FAVOR_NORM
}

template <typename T, int VW, int NV, int CTA>
cudaError_t fwd(Row<T, VW, NV, CTA>, const NormArgs& a, const Rows& rows, uint32_t n, const Plan& plan,
                cudaStream_t stream) {
  norm_fwd_kernel<T, VW, NV, CTA><<<plan.ctas, plan.threads, 0, stream>>>(a, rows, n, plan);
  return cudaGetLastError();
}

template <typename T, int VW, int NV, int CTA>
cudaError_t bwd(Row<T, VW, NV, CTA>, const NormArgs& a, const Rows& rows, uint32_t n, const Plan& plan, float* part,
                cudaStream_t stream) {
  const size_t smem = part != nullptr && CTA == 0 ? (size_t)(plan.groups / 2) * 2 * a.d * sizeof(float) : 0;
  const auto kernel = norm_bwd_kernel<T, VW, NV, CTA>;
  if (smem > 0) {
    const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), smem);
    if (e != cudaSuccess) return e;
  }
  kernel<<<plan.ctas, plan.threads, smem, stream>>>(a, rows, n, plan, part);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_fwd(const NormArgs& a, bool bf16, bool vec, cudaStream_t stream) {
  const uint32_t n = (uint32_t)a.B * a.H * a.L;
  const Strides s[2] = {a.xs, a.ys};
  const Rows rows = make_rows(a.B, a.H, a.L, s, 2);
  const Plan plan = make_plan(n, a.d, bf16, vec, false);
  return dispatch(plan, a.d, bf16, vec, [&](auto kind) { return fwd(kind, a, rows, n, plan, stream); });
}

// what either kernel of a shape may write, whatever the pointers' alignment
size_t norm_bwd_workspace_bytes(int64_t rows, int d, bool bf16) {
  const int ctas = std::max(make_plan(rows, d, bf16, false, true).ctas, make_plan(rows, d, bf16, true, true).ctas);
  return (size_t)ctas * 2 * d * sizeof(float);
}

cudaError_t launch_norm_bwd(const NormArgs& a, bool bf16, bool vec, float* ws, cudaStream_t stream) {
  const uint32_t n = (uint32_t)a.B * a.H * a.L;
  const Strides s[3] = {a.xs, a.dys, a.dxs};
  const Rows rows = make_rows(a.B, a.H, a.L, s, 3);
  const Plan plan = make_plan(n, a.d, bf16, vec, true);
  const bool sums = a.dgamma != nullptr || a.dbeta != nullptr;
  cudaError_t e = dispatch(plan, a.d, bf16, vec, [&](auto kind) {
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
