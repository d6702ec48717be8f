// Gated linear recurrence h_t = exp(g_t) h_{t-1} + x_t per channel, forward,
// backward and one token.
#include "ops.cuh"

namespace favor {
namespace {

constexpr int kThreads = 128;

// exp(g) = 0 drops the state, whatever it is
__device__ __forceinline__ float apply(float a, float h, float x) { return a == 0.f ? x : fmaf(a, h, x); }

// one thread per channel walks the tokens
template <typename T>
__global__ void scan_fwd_kernel(ScanArgs p) {
  const int64_t n = (int64_t)p.B * p.H * p.d;
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= n) return;
  const int64_t bh = i / p.d, c = i - bh * p.d, b = bh / p.H, hd = bh - b * p.H;
  const T* x = static_cast<const T*>(p.x) + b * p.xs.b + hd * p.xs.h + c;
  const T* g = static_cast<const T*>(p.g) + b * p.gs.b + hd * p.gs.h + c;
  T* out = static_cast<T*>(p.h) + b * p.hs.b + hd * p.hs.h + c;
  float h = p.first != nullptr ? p.first[i] : 0.f;
  for (int t = 0; t < p.L; ++t) {
    h = apply(expf(to_f32(g[t * p.gs.l])), h, to_f32(x[t * p.xs.l]));
    out[t * p.hs.l] = from_f32<T>(h);
  }
  if (p.last != nullptr) p.last[i] = h;
}

template <typename T>
__global__ void scan_bwd_kernel(ScanArgs p) {
  const int64_t n = (int64_t)p.B * p.H * p.d;
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= n) return;
  const int64_t bh = i / p.d, c = i - bh * p.d, b = bh / p.H, hd = bh - b * p.H;
  const T* g = static_cast<const T*>(p.g) + b * p.gs.b + hd * p.gs.h + c;
  const T* h = static_cast<const T*>(p.h_in) + b * p.his.b + hd * p.his.h + c;
  const T* dh = static_cast<const T*>(p.dh) + b * p.dhs.b + hd * p.dhs.h + c;
  T* dx = static_cast<T*>(p.dx) + b * p.dxs.b + hd * p.dxs.h + c;
  T* dg = static_cast<T*>(p.dg) + b * p.dgs.b + hd * p.dgs.h + c;
  float carry = p.first != nullptr ? p.first[i] : 0.f;
  for (int t = p.L - 1; t >= 0; --t) {
    const float a = expf(to_f32(g[t * p.gs.l]));
    const float u = to_f32(dh[t * p.dhs.l]) + carry;
    const float prev = t > 0 ? to_f32(h[(t - 1) * p.his.l]) : (p.h0 != nullptr ? p.h0[i] : 0.f);
    carry = a == 0.f ? 0.f : a * u;
    dx[t * p.dxs.l] = from_f32<T>(u);
    dg[t * p.dgs.l] = from_f32<T>(a == 0.f ? 0.f : carry * prev);
  }
  if (p.last != nullptr) p.last[i] = carry;
}

template <typename T>
__global__ void scan_step_kernel(const T* x, const T* g, T* h, const float* state, float* new_state, int n) {
  const int i = blockIdx.x * kThreads + threadIdx.x;
  if (i >= n) return;
  const float v = apply(expf(to_f32(g[i])), state[i], to_f32(x[i]));
  new_state[i] = v;
  h[i] = from_f32<T>(v);
}

}  // namespace

cudaError_t launch_scan(const ScanArgs& a, bool backward, bool bf16, bool pairs, cudaStream_t stream) {
  (void)pairs;
  const int64_t n = (int64_t)a.B * a.H * a.d;
  const unsigned grid = (unsigned)((n + kThreads - 1) / kThreads);
  if (backward) {
    if (bf16) scan_bwd_kernel<__nv_bfloat16><<<grid, kThreads, 0, stream>>>(a);
    else scan_bwd_kernel<float><<<grid, kThreads, 0, stream>>>(a);
  } else {
    if (bf16) scan_fwd_kernel<__nv_bfloat16><<<grid, kThreads, 0, stream>>>(a);
    else scan_fwd_kernel<float><<<grid, kThreads, 0, stream>>>(a);
  }
  return cudaGetLastError();
}

cudaError_t launch_scan_step(const void* x, const void* g, void* h, const float* state, float* new_state, int64_t n,
                             bool bf16, cudaStream_t stream) {
  const unsigned grid = (unsigned)((n + kThreads - 1) / kThreads);
  if (bf16)
    scan_step_kernel<<<grid, kThreads, 0, stream>>>(static_cast<const __nv_bfloat16*>(x),
                                                    static_cast<const __nv_bfloat16*>(g),
                                                    static_cast<__nv_bfloat16*>(h), state, new_state, (int)n);
  else
    scan_step_kernel<<<grid, kThreads, 0, stream>>>(static_cast<const float*>(x), static_cast<const float*>(g),
                                                    static_cast<float*>(h), state, new_state, (int)n);
  return cudaGetLastError();
}

}  // namespace favor
