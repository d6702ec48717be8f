// Shared pieces of the sequence operators (favor_ops.h): tensor views and
// their checks on the host, strided addressing and vector pieces on the device.
#pragma once

#include "common.cuh"
#include "favor_ops.h"
#include "tc_ptx.cuh"

namespace favor {

constexpr int kNormMaxD = 16384;

// ---- views ----------------------------------------------------------------
// Element strides of B, H and L (extents of 1 and, for flat arrays, all of
// them have stride 0).
struct Strides {
  int64_t b, h, l;
};

// A tensor as the argument checks see it: extents and element strides of B,
// H, L and the last axis (whose stride is 1).
struct View {
  const void* p;
  int esz;
  int64_t n[4];
  int64_t s[3];
  Strides strides() const { return Strides{s[0], s[1], s[2]}; }
  // every row starts on a multiple of `bytes` and consists of whole pieces of it
  bool pieces(int bytes) const {
    const int64_t e = bytes / esz;
    return reinterpret_cast<uintptr_t>(p) % bytes == 0 && n[3] % e == 0 && s[0] % e == 0 && s[1] % e == 0 &&
           s[2] % e == 0;
  }
};

// false: null, misaligned, a negative or an absurd stride
bool make_view(View* v, const void* p, const int64_t* strides, int B, int H, int L, int d, int esz);
// n elements side by side
View flat_view(const void* p, int64_t n, int esz);
// two elements of the view share an address (or its strides do not nest)
bool self_overlap(const View& v);
bool same_view(const View& a, const View& b);
bool overlap(const View& a, const View& b);

// ---- division of n < 2^31 by a constant of the launch -------------------------
// m = ceil(2^s / d) with s = 31 + ceil(log2 d): m d exceeds 2^s by less than d,
// so n m / 2^s exceeds n / d by less than n / 2^s < 1 / d, and its floor is
// that of n / d.  m <= 2^32: the product fits 64 bits.
struct FastDiv {
  uint64_t m;
  uint32_t shift, d;
  __host__ __device__ FastDiv() : m(0), shift(0), d(1) {}
  explicit FastDiv(uint32_t div) : d(div) {
    uint32_t l = 0;
    while ((1ull << l) < div) ++l;
    shift = 31 + l;
    m = ((1ull << shift) + div - 1) / div;
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const { return static_cast<uint32_t>((n * m) >> shift); }
};

// ---- rows -------------------------------------------------------------------
// Offsets of the rows (b, h, t), t fastest, of up to three tensors.  Axes that
// every tensor walks with one stride are merged, so that contiguous tensors
// need no division.
struct Rows {
  FastDiv l, h;          // extents of the inner two axes; 1: merged away or single
  Strides s[3];
  // row -> (b, h, t)
  __device__ __forceinline__ void split(uint32_t row, uint32_t* b, uint32_t* hh, uint32_t* t) const {
    uint32_t r = row;
    *t = 0;
    *hh = 0;
    if (l.d > 1) {
      r = l.div(row);
      *t = row - r * l.d;
    }
    *b = r;
    if (h.d > 1) {
      *b = h.div(r);
      *hh = r - *b * h.d;
    }
  }
  __device__ __forceinline__ int64_t offset(int i, uint32_t row) const {
    if (l.d == 1 && h.d == 1) return row * s[i].b;
    uint32_t b, hh, t;
    split(row, &b, &hh, &t);
    return b * s[i].b + hh * s[i].h + t * s[i].l;
  }
};
Rows make_rows(int B, int H, int L, const Strides* s, int n);

// ---- two fp32 operations in one instruction --------------------------------------
__device__ __forceinline__ unsigned long long f32x2_bits(float2 a) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.x), "f"(a.y));
  return r;
}
__device__ __forceinline__ float2 f32x2_of(unsigned long long r) {
  float2 a;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a.x), "=f"(a.y) : "l"(r));
  return a;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(f32x2_bits(a)), "l"(f32x2_bits(b)), "l"(f32x2_bits(c)));
  return f32x2_of(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(f32x2_bits(a)), "l"(f32x2_bits(b)));
  return f32x2_of(r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(f32x2_bits(a)), "l"(f32x2_bits(b)));
  return f32x2_of(r);
}

// ---- launchers ------------------------------------------------------------------
struct ScanArgs {
  const void *x, *g, *h_in, *dh;      // forward: x, g; backward: g, h_in, dh
  void *h, *dx, *dg;                  // forward: h; backward: dx, dg
  Strides xs, gs, his, dhs, hs, dxs, dgs;
  const float* first;                 // h0 (forward), dhT (backward): the carry at the start, or NULL
  const float* h0;                    // backward: h_{-1}, or NULL
  float* last;                        // hT (forward), dh0 (backward), or NULL
  int32_t* status;
  int B, H, L, d;
  long long wait_cycles = tc::kWaitLimitCycles;   // limit of a wait inside a cluster
  int quits = -1;                     // a CTA of each cluster whose waits run out at once (a test's), -1: none
};
// align: pieces of this many bytes (16, 4 or 2) make up every row of every tensor
cudaError_t launch_scan(const ScanArgs& a, bool backward, bool bf16, int align, cudaStream_t stream);
cudaError_t launch_scan_step(const void* x, const void* g, void* h, const float* state, float* new_state, int64_t n,
                             bool bf16, cudaStream_t stream);

struct NormArgs {
  const void *x, *dy;
  void *y, *dx;
  Strides xs, dys, ys, dxs;
  const float *gamma, *beta;
  float *dgamma, *dbeta;
  float eps;
  int B, H, L, d;
};
// piece: every tensor's rows are made of pieces of this many bytes (16, two elements or one)
cudaError_t launch_norm_fwd(const NormArgs& a, bool bf16, int piece, cudaStream_t stream);
cudaError_t launch_norm_bwd(const NormArgs& a, bool bf16, int piece, float* ws, cudaStream_t stream);
size_t norm_bwd_workspace_bytes(int64_t rows, int d, bool bf16);

struct RotaryArgs {
  const void *q, *k;
  void *qo, *ko;
  Strides qs, ks, qos, kos;
  int B, Hq, Hk, L, d;                // Hk = 0: no keys
  const int32_t* pos;
  int pos_B, n_axes, sections[FAVOR_ROTARY_MAX_AXES], pairs;
  const uint64_t* table;
  bool halves, inverse;
};
cudaError_t launch_rotary(const RotaryArgs& a, bool bf16, int piece, cudaStream_t stream);

constexpr int kQkNormMaxD = 512;
struct QkNormArgs {
  const void *q, *k, *dqo, *dko;      // dqo, dko: backward, the gradients of the outputs
  void *qo, *ko;                      // forward: the outputs; backward: dq, dk
  Strides qs, ks, dqos, dkos, qos, kos;
  const float *wq, *wk;
  float *dwq, *dwk;
  float eps;
  int B, Hq, Hk, L, d;                // Hk = 0: no keys
  const int32_t* pos;
  int pos_B, n_axes, sections[FAVOR_ROTARY_MAX_AXES], pairs;
  const uint64_t* table;
  bool halves;
};
cudaError_t launch_qk_norm(const QkNormArgs& a, bool bf16, int piece, bool backward, float* ws, cudaStream_t stream);
size_t qk_norm_workspace_bytes(const QkNormArgs& a);

}  // namespace favor
