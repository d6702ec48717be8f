// Rotation of queries and keys by positions on one to four axes.
#include "ops.cuh"

namespace favor {
namespace {

constexpr int kThreads = 256;

// The angle of a pair, in half turns: the position times the pair's fraction
// of a turn per unit, in 64-bit fixed point, wraps to the exact fraction of a
// turn; its upper 32 bits as a signed number are the angle to 2^-32 turns.
__device__ __forceinline__ float half_turns(int32_t pos, uint64_t per_unit) {
  const uint64_t turn = static_cast<uint64_t>(static_cast<int64_t>(pos)) * per_unit;
  return static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f;
}

struct Axes {
  int end[FAVOR_ROTARY_MAX_AXES];   // pairs of the axes up to and with each
};

// one thread per pair (or channel behind the last pair) of a row
template <typename T>
__global__ void rotary_kernel(const T* in, T* out, Strides is, Strides os, const int32_t* pos, int pos_B,
                              const uint64_t* table, Axes ax, int H, int L, int d, int P, int halves, float sign,
                              int64_t total) {
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= total) return;
  const int items = d - P;          // P pairs and d - 2 P channels
  const int64_t row = i / items;
  const int p = (int)(i - row * items);
  const int64_t bh = row / L, t = row - bh * L, b = bh / H, h = bh - b * H;
  in += b * is.b + h * is.h + t * is.l;
  out += b * os.b + h * os.h + t * os.l;
  if (p >= P) {
    out[p + P] = in[p + P];
    return;
  }
  int a = 0;
  while (p >= ax.end[a]) ++a;
  const int32_t at = pos[((int64_t)a * pos_B + (pos_B > 1 ? b : 0)) * L + t];
  float s, c;
  sincospif(half_turns(at, table[p]), &s, &c);
  s *= sign;
  const int iu = halves ? p : 2 * p, iv = halves ? p + P : 2 * p + 1;
  const float u = to_f32(in[iu]), v = to_f32(in[iv]);
  out[iu] = from_f32<T>(u * c - v * s);
  out[iv] = from_f32<T>(u * s + v * c);
}

template <typename T>
void go(const RotaryArgs& a, const Axes& ax, const void* in, void* out, const Strides& is, const Strides& os, int H,
        cudaStream_t stream) {
  const int64_t total = (int64_t)a.B * H * a.L * (a.d - a.pairs);
  rotary_kernel<T><<<(unsigned)((total + kThreads - 1) / kThreads), kThreads, 0, stream>>>(
      static_cast<const T*>(in), static_cast<T*>(out), is, os, a.pos, a.pos_B, a.table, ax, H, a.L, a.d, a.pairs,
      a.halves ? 1 : 0, a.inverse ? -1.f : 1.f, total);
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, bool bf16, bool vec, cudaStream_t stream) {
  (void)vec;
  Axes ax;
  int end = 0;
  for (int i = 0; i < FAVOR_ROTARY_MAX_AXES; ++i) ax.end[i] = end += i < a.n_axes ? a.sections[i] : 0;
  if (bf16) {
    go<__nv_bfloat16>(a, ax, a.q, a.qo, a.qs, a.qos, a.Hq, stream);
    if (a.Hk > 0) go<__nv_bfloat16>(a, ax, a.k, a.ko, a.ks, a.kos, a.Hk, stream);
  } else {
    go<float>(a, ax, a.q, a.qo, a.qs, a.qos, a.Hq, stream);
    if (a.Hk > 0) go<float>(a, ax, a.k, a.ko, a.ks, a.kos, a.Hk, stream);
  }
  return cudaGetLastError();
}

}  // namespace favor
