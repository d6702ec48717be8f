// Layer norm over the last axis, forward and backward with the reduction of
// the weight's gradient.
#include "ops.cuh"

namespace favor {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

struct RowDiv {
  FastDiv l, h;
};
__device__ __forceinline__ int64_t row_offset(const Strides& s, uint32_t row, const RowDiv& dv) {
  const uint32_t bh = dv.l.div(row), t = row - bh * dv.l.d;
  const uint32_t b = dv.h.div(bh), h = bh - b * dv.h.d;
  return b * s.b + h * s.h + t * s.l;
}

// mean and 1 / sqrt(var + eps) of a row, one warp
template <typename T>
__device__ __forceinline__ void row_stats(const T* x, int d, float eps, float* mean, float* rstd) {
  const int lane = threadIdx.x & 31;
  float s = 0.f;
  for (int c = lane; c < d; c += 32) s += to_f32(x[c]);
  const float mu = warp_sum(s) / d;
  float v = 0.f;
  for (int c = lane; c < d; c += 32) {
    const float u = to_f32(x[c]) - mu;
    v = fmaf(u, u, v);
  }
  *mean = mu;
  *rstd = 1.f / sqrtf(warp_sum(v) / d + eps);
}

// one warp per row
template <typename T>
__global__ void norm_fwd_kernel(NormArgs p, RowDiv dv, uint32_t rows) {
  const uint32_t row = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (row >= rows) return;
  const T* x = static_cast<const T*>(p.x) + row_offset(p.xs, row, dv);
  T* y = static_cast<T*>(p.y) + row_offset(p.ys, row, dv);
  float mu, r;
  row_stats(x, p.d, p.eps, &mu, &r);
  for (int c = threadIdx.x & 31; c < p.d; c += 32) {
    const float w = p.gamma != nullptr ? p.gamma[c] : 1.f, z = p.beta != nullptr ? p.beta[c] : 0.f;
    y[c] = from_f32<T>(fmaf((to_f32(x[c]) - mu) * r, w, z));
  }
}

template <typename T>
__global__ void norm_stats_kernel(NormArgs p, RowDiv dv, uint32_t rows, float2* stats) {
  const uint32_t row = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (row >= rows) return;
  float mu, r;
  row_stats(static_cast<const T*>(p.x) + row_offset(p.xs, row, dv), p.d, p.eps, &mu, &r);
  if ((threadIdx.x & 31) == 0) stats[row] = make_float2(mu, r);
}

// the columns' sums: a block per 32 columns
template <typename T>
__global__ void norm_bwd_columns_kernel(NormArgs p, RowDiv dv, uint32_t rows, const float2* stats) {
  __shared__ float2 part[kWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float sg = 0.f, sb = 0.f;
  if (c < p.d) {
    for (uint32_t row = warp; row < rows; row += kWarps) {
      const float dy = to_f32((static_cast<const T*>(p.dy) + row_offset(p.dys, row, dv))[c]);
      const float x = to_f32((static_cast<const T*>(p.x) + row_offset(p.xs, row, dv))[c]);
      sg = fmaf(dy, (x - stats[row].x) * stats[row].y, sg);
      sb += dy;
    }
  }
  part[warp][lane] = make_float2(sg, sb);
  __syncthreads();
  if (warp == 0 && c < p.d) {
    for (int i = 1; i < kWarps; ++i) {
      sg += part[i][lane].x;
      sb += part[i][lane].y;
    }
    if (p.dgamma != nullptr) p.dgamma[c] = sg;
    if (p.dbeta != nullptr) p.dbeta[c] = sb;
  }
}

// one warp per row
template <typename T>
__global__ void norm_bwd_rows_kernel(NormArgs p, RowDiv dv, uint32_t rows) {
  const uint32_t row = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (row >= rows) return;
  const int lane = threadIdx.x & 31;
  const T* x = static_cast<const T*>(p.x) + row_offset(p.xs, row, dv);
  const T* dy = static_cast<const T*>(p.dy) + row_offset(p.dys, row, dv);
  T* dx = static_cast<T*>(p.dx) + row_offset(p.dxs, row, dv);
  float mu, r, a = 0.f, b = 0.f;
  row_stats(x, p.d, p.eps, &mu, &r);
  for (int c = lane; c < p.d; c += 32) {
    const float n = to_f32(dy[c]) * (p.gamma != nullptr ? p.gamma[c] : 1.f);
    a += n;
    b = fmaf(n, (to_f32(x[c]) - mu) * r, b);
  }
  a = warp_sum(a) / p.d;
  b = warp_sum(b) / p.d;
  for (int c = lane; c < p.d; c += 32) {
    const float n = to_f32(dy[c]) * (p.gamma != nullptr ? p.gamma[c] : 1.f);
    dx[c] = from_f32<T>(r * (n - a - (to_f32(x[c]) - mu) * r * b));
  }
}

RowDiv row_div(const NormArgs& a) { return RowDiv{FastDiv(a.L), FastDiv(a.H)}; }

}  // namespace

cudaError_t launch_norm_fwd(const NormArgs& a, bool bf16, bool vec, cudaStream_t stream) {
  (void)vec;
  const uint32_t rows = (uint32_t)a.B * a.H * a.L;
  const unsigned grid = (rows + kWarps - 1) / kWarps;
  if (bf16) norm_fwd_kernel<__nv_bfloat16><<<grid, kThreads, 0, stream>>>(a, row_div(a), rows);
  else norm_fwd_kernel<float><<<grid, kThreads, 0, stream>>>(a, row_div(a), rows);
  return cudaGetLastError();
}

size_t norm_bwd_workspace_bytes(int64_t rows, int d, bool bf16) {
  (void)d;
  (void)bf16;
  return (size_t)rows * sizeof(float2);
}

cudaError_t launch_norm_bwd(const NormArgs& a, bool bf16, bool vec, float* ws, cudaStream_t stream) {
  (void)vec;
  const uint32_t rows = (uint32_t)a.B * a.H * a.L;
  const unsigned grid = (rows + kWarps - 1) / kWarps, cols = (a.d + 31) / 32;
  float2* st = reinterpret_cast<float2*>(ws);
  const bool sums = a.dgamma != nullptr || a.dbeta != nullptr;
  auto go = [&](auto tag) {
    using T = decltype(tag);
    if (sums) {
      // the columns first: dx may take the place of x or dy
      norm_stats_kernel<T><<<grid, kThreads, 0, stream>>>(a, row_div(a), rows, st);
      norm_bwd_columns_kernel<T><<<cols, kThreads, 0, stream>>>(a, row_div(a), rows, st);
    }
    norm_bwd_rows_kernel<T><<<grid, kThreads, 0, stream>>>(a, row_div(a), rows);
  };
  if (bf16) go(__nv_bfloat16{});
  else go(float{});
  return cudaGetLastError();
}

}  // namespace favor
