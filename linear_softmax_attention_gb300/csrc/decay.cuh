// Causal linear attention with a decay per head: what its two paths share.
//
// Every pass of it, forward and backward, is one form.  Over the n tokens of a
// chunk, with three rows a_i, b_j, c_j and a state M [x][y] that the chunk
// meets,
//   out_i = s_w sum_j w(i, j) (a_i . b_j) c_j + s_r r(i) M^T a_i
//   M'    = l^n M + s_u sum_j u(j) b_j c_j^T
// where w(i, j) = l^(i-j), j <= i; r(i) = l^(i+1); u(j) = l^(n-1-j), or, walking
// the chunks back ("rev"), w(i, j) = l^(j-i), j >= i; r(i) = l^(n-1-i);
// u(j) = l^(j+1):
//   o:  a = q,  b = k,  c = v         M = S       s_w = s_r = scale, s_u = 1
//   dq: a = do, b = v,  c = k         M = S^T     s_w = s_r = scale, s_u = 1
//   dk: a = v,  b = do, c = q  (rev)  M = R^T     s_w = scale, s_r = 1, s_u = scale
//   dv: a = k,  b = q,  c = do (rev)  M = R       s_w = scale, s_r = 1, s_u = scale
// with S the state before the chunk and R the gradient of the state behind it.
// A sequence is cut into segments of whole chunks; where there is more than
// one, their gains (M' from M = 0) come first, a scan over the segments makes
// them the states that each one starts from, and then all of them run at once.
#pragma once

#include "ops.cuh"

namespace favor {

constexpr int kDecayMaxD = 128;

struct DecayPass {
  const void *a, *b, *c;
  void* o;
  Strides as, bs, cs, os;
  const float* start;        // fp32 [B H][segs][d][d]: what each segment starts from; NULL: zeros
  float* last;               // one segment: M behind it, [B H][d][d], or NULL (may be `start`)
  bool transposed;           // start and last hold M^T
  bool rev;
  float s_w, s_r, s_u;
};

// the gains of one kind of state: sum_j u(j) b_j c_j^T over each segment
struct DecayGain {
  const void *b, *c;
  Strides bs, cs;
  float* out;                // [B H][segs][d][d]
  float s_u;
  bool rev;
};

struct DecayShape {
  const float* g;
  const int32_t* lengths;
  int32_t* status;
  int B, H, L, d;
  int segs, seg_tokens;
  __host__ __device__ int BH() const { return B * H; }
};

// tokens of sequence b
__device__ __forceinline__ int decay_length(const DecayShape& s, int b) {
  return s.lengths == nullptr ? s.L : min(max(s.lengths[b], 0), s.L);
}
// l^n of l = 2^g2; l^0 = 1 whatever l is
__device__ __forceinline__ float decay_power(float g2, int n) { return n == 0 ? 1.f : exp2f(g2 * n); }

// Segments of whole chunks for a sequence, one where there are no more than `one`
// chunks: as many as make the waves of CTAs (`slots` of them are resident) the
// cheapest, counting about two chunks' time for a CTA's start and a little for each
// segment of the scan, which takes them one after another (128 at most).  Half, three
// quarters, twice and three times that number of CTAs: 8 x 8 x 4096 x 64 bf16 74, 61,
// 59 and 63 us against 54; 1 x 16 x 16384 x 128 158, 117, 117 and 130 against 108.
inline void decay_segments(DecayShape* s, int chunk, int slots, int passes, int one) {
  const int chunks = (s->L + chunk - 1) / chunk;
  const int most = chunks <= one ? 1 : std::min(chunks, 128);
  double best = -1;
  for (int want = 1; want <= most; ++want) {
    const int per = (chunks + want - 1) / want, segs = (chunks + per - 1) / per;
    const int64_t waves = ((int64_t)segs * s->BH() * passes + slots - 1) / slots;
    const double cost = waves * (per + 2.0) + 0.05 * segs;
    if (best < 0 || cost < best) {
      best = cost;
      s->segs = segs;
      s->seg_tokens = per * chunk;
    }
  }
}

// CUDA-core path: fp32 arithmetic, any d <= 128 and any strides
// segments for `passes` passes side by side
void decay_simt_plan(DecayShape* s, int passes);
cudaError_t decay_simt_gains(const DecayGain* gains, int n, const DecayShape& s, bool bf16, int piece,
                             cudaStream_t stream);
// up to three side by side
cudaError_t decay_simt_passes(const DecayPass* passes, int n, const DecayShape& s, bool bf16, int piece,
                              cudaStream_t stream);
// gains -> the states that the segments start from, in place; `first` [B H][d][d] (NULL: zeros) before the first
// segment (behind the last one where rev), `last` what follows the others (NULL: not wanted).  pieces: a segment's
// gain is the sum of that many, side by side; its state takes the place of the first
struct DecayScan {
  float* states;
  const float* first;
  float* last;
  bool rev;
  int pieces;                // 1 or 2
};
cudaError_t decay_scan_states(const DecayScan* scans, int n, const DecayShape& s, cudaStream_t stream);

// whole sequences of at most kDecayFew tokens, forward, any d <= 128 and any strides: o, and M
// behind them at p.last (NULL: not wanted; may be p.start).  1, 4 and 16 tokens of 1024 heads
// of 128 bf16: 34, 45 and 79 us (as a chunk on the tensor cores 158, 159 and 163, on the CUDA
// cores 165 to 177), of 64: 12, 15 and 30 (46), of two heads of 128: 6.2, 7.7 and 13.8 (13.8),
// of 64: 4.8, 4.9 and 8.9 (9.0); 17 tokens take the other paths
constexpr int kDecayFew = 16;
cudaError_t decay_few(const DecayPass& p, const DecayShape& s, bool bf16, cudaStream_t stream);

struct DecayStep {
  const void *q, *k, *v;
  void* o;
  int64_t qs[2], ks[2], vs[2], os[2];
  const float *g, *state;
  float* next;
  float scale;
  int B, H, d;
  bool vec;                  // 16-byte pieces of the states
};
cudaError_t launch_decay_step(const DecayStep& p, bool bf16, cudaStream_t stream);

}  // namespace favor
