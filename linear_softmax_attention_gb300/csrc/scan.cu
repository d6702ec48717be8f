// Gated linear recurrence h_t = exp(g_t) h_{t-1} + x_t per channel, forward,
// backward and one token.
//
// A run of tokens acts on the state before it as one affine map, h -> A h + s
// with A the product of its gates and s its own sum; two runs in sequence
// compose to (A1 A2, A2 s1 + s2).  The backward pass is the same recurrence
// against time: c_t = a_t c_{t+1} + a_t dh_t, dx_t = dh_t + c_{t+1},
// dg_t = c_t h_{t-1}.
//
// Bound by memory: every element is read and written once.  Channels are
// independent, but a whole GPU of them is rare, so a cluster of CTAs walks
// 32 lanes of channels together, R tokens per warp, W worker warps and K CTAs
// per step.  The workers copy their tokens ahead into a ring in shared memory
// and form their runs' maps; one more warp per CTA joins the maps in a fixed
// order, within the CTA through shared memory and across the cluster through
// distributed shared memory, while the workers form the next step's maps; then
// they walk their runs once more from the state before them and write.
// Nothing is read twice and nothing is passed through global memory, so the
// call needs no workspace and its bits do not depend on timing.
//
// Measured (one GB300; copy rate 6779 GB/s): 65536 tokens x 2048 channels fp32
// 240 to 244 us forward, 6.6 TB/s; 8 x 16 heads x 4096 x 128 bf16 78 us forward,
// 5.1 TB/s, and 106 us backward, 6.3 TB/s; 4 x 8 x 8192 x 64 bf16 25 us forward,
// 4.0 TB/s; 2 x 8 x 12288 x 64 bf16 35.5 us backward, 3.5 TB/s.  What holds the
// last two back is how little is resident: 256 CTAs of 6 warps (forward) and
// 192 of 10 (backward) leave 7 and 14 SMs empty and 34 and 84 with one CTA; on
// those with two, 56 and 68 % of the issue slots are used, by 3 to 5 warps a
// scheduler that otherwise wait for fixed latencies, the step's barriers and
// the fetching of instructions (54 and 86 of them per token and pair of
// channels).  Tried and slower at 4 x 8 x 8192
// x 64, at the time against 26 us: three CTAs an SM (39 us, the registers
// spill), single channels of bf16 (33), the sending and the gathering of maps
// in two warps (28), a cluster barrier a step in place of the counted stores
// (48: its release waits for the global stores' acknowledgement).
#include <mutex>

#include "ops.cuh"
#include "tc_ptx.cuh"

namespace favor {
namespace {

constexpr int kMaxCluster = 16;       // CTAs of a cluster
constexpr int kFold = 4;              // maps read together while they are joined
constexpr int kStages = 3;            // runs of a warp in its ring
constexpr int kStepThreads = 128;

// ---- V = 1 or 2 channels of a lane, fp32 ------------------------------------------
// Two channels go through the packed fp32 instructions.
template <int V> struct Vec { float f[V]; };
__device__ __forceinline__ Vec<1> fma_(Vec<1> a, Vec<1> b, Vec<1> c) { return {fmaf(a.f[0], b.f[0], c.f[0])}; }
__device__ __forceinline__ Vec<1> mul_(Vec<1> a, Vec<1> b) { return {a.f[0] * b.f[0]}; }
__device__ __forceinline__ Vec<1> add_(Vec<1> a, Vec<1> b) { return {a.f[0] + b.f[0]}; }
__device__ __forceinline__ float2 both(const Vec<2>& a) { return make_float2(a.f[0], a.f[1]); }
__device__ __forceinline__ Vec<2> fma_(Vec<2> a, Vec<2> b, Vec<2> c) {
  const float2 r = fma2(both(a), both(b), both(c));
  return {r.x, r.y};
}
__device__ __forceinline__ Vec<2> mul_(Vec<2> a, Vec<2> b) {
  const float2 r = mul2(both(a), both(b));
  return {r.x, r.y};
}
__device__ __forceinline__ Vec<2> add_(Vec<2> a, Vec<2> b) {
  const float2 r = add2(both(a), both(b));
  return {r.x, r.y};
}

// A h + s, where A = 0 drops h, whatever it is
template <int V>
__device__ __forceinline__ Vec<V> apply(const Vec<V>& A, const Vec<V>& s, const Vec<V>& h) {
  Vec<V> r = fma_(A, h, s);
#pragma unroll
  for (int v = 0; v < V; ++v) r.f[v] = A.f[v] == 0.f ? s.f[v] : r.f[v];
  return r;
}

// 0 for finite values, NaN otherwise: 0 times an infinity or NaN is NaN
template <int V>
__device__ __forceinline__ Vec<V> residue(const Vec<V>& a, const Vec<V>& r) {
  Vec<V> zero;
#pragma unroll
  for (int v = 0; v < V; ++v) zero.f[v] = 0.f;
  return fma_(a, zero, r);
}
__device__ __forceinline__ float sum(const Vec<1>& r) { return r.f[0]; }
__device__ __forceinline__ float sum(const Vec<2>& r) { return r.f[0] + r.f[1]; }
__device__ __forceinline__ float product(const Vec<1>& r) { return r.f[0]; }
__device__ __forceinline__ float product(const Vec<2>& r) { return r.f[0] * r.f[1]; }
template <int V>
__device__ __forceinline__ bool none(const Vec<V>& r) { return sum(r) == 0.f; }
template <int V>
__device__ __forceinline__ bool finite(const Vec<V>& a) {
  Vec<V> zero;
#pragma unroll
  for (int v = 0; v < V; ++v) zero.f[v] = 0.f;
  return none(residue(a, zero));
}

// V channels side by side as they lie in memory
template <typename T, int V> struct Piece;
template <> struct Piece<float, 1> {
  using Raw = float;
  static __device__ __forceinline__ Vec<1> unpack(Raw r) { return {r}; }
  static __device__ __forceinline__ Raw pack(const Vec<1>& a) { return a.f[0]; }
};
template <> struct Piece<__nv_bfloat16, 1> {
  using Raw = unsigned short;
  static __device__ __forceinline__ Vec<1> unpack(Raw r) { return {__uint_as_float((unsigned)r << 16)}; }
  static __device__ __forceinline__ Raw pack(const Vec<1>& a) {
    return __bfloat16_as_ushort(__float2bfloat16_rn(a.f[0]));
  }
};
template <> struct Piece<__nv_bfloat16, 2> {
  using Raw = unsigned;
  static __device__ __forceinline__ Vec<2> unpack(Raw r) {
    return {__uint_as_float(r << 16), __uint_as_float(r & 0xffff0000u)};
  }
  static __device__ __forceinline__ Raw pack(const Vec<2>& a) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a.f[0], a.f[1]);
    return *reinterpret_cast<const unsigned*>(&v);
  }
};

template <int V>
__device__ __forceinline__ Vec<V> exp_(Vec<V> g) {
#pragma unroll
  for (int v = 0; v < V; ++v) g.f[v] = expf(g.f[v]);
  return g;
}
template <int V>
__device__ __forceinline__ Vec<V> all(float x) {
  Vec<V> r;
#pragma unroll
  for (int v = 0; v < V; ++v) r.f[v] = x;
  return r;
}

// ---- the ring of tokens ---------------------------------------------------------------
// N arrays, R tokens of each per thread and stage, word order
// [stage][array][token][thread].  Every warp copies and reads only its own
// places, so that a warp's barrier orders copies and reads.
template <int BYTES>
__device__ __forceinline__ void copy_async(void* dst, const void* src, bool in) {
  const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
  const int n = in ? BYTES : 0;               // 0: the place is filled with zeros
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(d), "l"(src), "n"(BYTES), "r"(n) : "memory");
}
__device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_but() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// ---- joining the runs ----------------------------------------------------------------------
// The map (A, s) of one channel.  A = -0: a closed gate, what was before is
// dropped.  A = +0: open gates whose product is below fp32; nothing finite gets
// through, but infinities and NaN do.  Where one of several gates is closed the
// product of their A is a 0, and the "or" of their signs its sign.
struct alignas(8) Map {
  float A, s;
};
__device__ __forceinline__ bool finite(float x) { return fabsf(x) < INFINITY; }
__device__ __forceinline__ bool closed(float A) { return __float_as_uint(A) == 0x80000000u; }
__device__ __forceinline__ uint32_t sign(float A) { return __float_as_uint(A) & 0x80000000u; }
// after `m`, the map `x` (signs are set once all are multiplied)
__device__ __forceinline__ Map then(const Map& m, const Map& x) { return {m.A * x.A, fmaf(x.A, m.s, x.s)}; }
// the same where infinities or NaN are about
__device__ __forceinline__ float through(const Map& x, float h) {
  return closed(x.A) ? x.s : fmaf(x.A == 0.f && !finite(h) ? 1.f : x.A, h, x.s);
}
__device__ __forceinline__ Map then_checked(const Map& m, const Map& x) {
  return {closed(x.A) ? -0.f : m.A * x.A, through(x, m.s)};
}

// A map into another CTA of the cluster, counted there by the barrier `bar`.
// (A cluster barrier with release semantics instead would wait, every step,
// until the global stores of the step before have been acknowledged.)
__device__ __forceinline__ void send(uint32_t at, const Map& m, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(at),
               "f"(m.A), "f"(m.s), "r"(bar)
               : "memory");
}

// Bounded wait for the cluster's maps, which acquires what the other CTAs have
// written; `limit` cycles, 0: as if they were over.
__device__ __forceinline__ bool wait_maps(uint64_t* bar, uint32_t parity, long long limit, const tc::WaitCtx& ctx) {
  const uint32_t a = tc::smem_addr(bar);
  if (limit > 0) {
    if (tc::mbar_try_wait_cluster(a, parity)) return true;
    const long long t0 = tc::sm_cycles();
    do {
      if (tc::mbar_try_wait_cluster(a, parity)) return true;
      if (*ctx.abort_flag) return false;
    } while (tc::sm_cycles() - t0 <= limit);
  }
  *ctx.abort_flag = 1;
  report_status(ctx.status, FAVOR_ERR_TIMEOUT);
  return false;
}

template <int V, int MW>
struct Joint {
  Map warp[2][V][MW][32];      // the runs' maps, from the workers
  float in[2][V][MW][32];      // the state before each run, to the workers
  uint64_t bar[2][V];
  int abort_flag;
};

// Hardware barriers between the workers and the joiners: "maps" of a step are
// there (the joiners wait), "states" of a step are there (the workers wait);
// two of each, by the step's parity.  The instructions want the warp together,
// which lanes with and without infinities have left.
__device__ __forceinline__ void bar_sync(int id, int threads) {
  __syncwarp();
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void bar_arrive(int id, int threads) {
  __syncwarp();
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
constexpr int kBarMaps = 1, kBarStates = 3;

// A joiner's walk over the steps, for channel v of each lane.  A buffer of
// parity n & 1 is free again at step n + 2: the workers hand over a step's
// maps only after they have read the states of the step two before, and a CTA
// sends its map of step n + 2 only when it has every CTA's of step n + 1,
// which they send after their reads of step n.  cta: the CTAs' maps,
// [2][V][K][32].  Returns the state behind the last step.  After a wait that
// ran out the warp only keeps its workers going: the barrier's phase is not
// over, so it is not armed again, and a map of a later step could end the wait
// of another CTA for this one.
template <int V, int MW>
__device__ float join(Joint<V, MW>& sm, Map (*cta)[32], int v, int steps, int K, int W, int rank, int lane, float carry,
                      long long limit, const tc::WaitCtx& ctx) {
  bool alive = true;
  const uint32_t me = tc::smem_addr(&sm);
  const uint32_t peer = K > 1 && lane < K ? tc::map_to_rank(me, lane) : 0;
  const int threads = (W + V) * 32;
  for (int n = 0; n < steps; ++n) {
    const int buf = n & 1;
    Map(*const there)[32] = cta + (buf * V + v) * K;
    uint64_t* const bar = &sm.bar[buf][v];
    if (K > 1 && alive && lane == 0) tc::mbar_arrive_expect_tx(bar, K * 32 * (int)sizeof(Map));
    bar_sync(kBarMaps + buf, threads);
    Map m[MW];
#pragma unroll
    for (int w = 0; w < MW; ++w)
      if (w < W) m[w] = sm.warp[buf][v][w][lane];
    float h = carry;
    if (K > 1 && alive) {
      Map total = m[0];
      uint32_t shut = sign(m[0].A);
#pragma unroll
      for (int w = 1; w < MW; ++w)
        if (w < W) {
          total = then(total, m[w]);
          shut |= sign(m[w].A);
        }
      // 0 times an infinity or NaN is NaN and stays so: only then are closed gates looked for
      if (!(finite(total.s) && finite(total.A))) {
        total = m[0];
#pragma unroll
        for (int w = 1; w < MW; ++w)
          if (w < W) total = then_checked(total, m[w]);
      }
      total.A = __uint_as_float((__float_as_uint(total.A) & 0x7fffffffu) | shut);
      const uint32_t at = tc::smem_addr(&there[rank][lane]) - me, bar_at = tc::smem_addr(bar) - me;
#pragma unroll 1
      for (int r0 = 0; r0 < K; r0 += kFold) {
        uint32_t to[kFold];
#pragma unroll
        for (int r = 0; r < kFold; ++r) to[r] = __shfl_sync(0xffffffffu, peer, r0 + r);
#pragma unroll
        for (int r = 0; r < kFold; ++r)
          if (r0 + r < K) send(to[r] + at, total, to[r] + bar_at);
      }
      alive = __all_sync(0xffffffffu, wait_maps(bar, (n >> 1) & 1, limit, ctx));
      float r = carry;
#pragma unroll 1
      for (int c0 = 0; c0 < K; c0 += kFold) {
        Map c[kFold];
#pragma unroll
        for (int i = 0; i < kFold; ++i)
          if (c0 + i < K) c[i] = there[c0 + i][lane];
#pragma unroll
        for (int i = 0; i < kFold; ++i)
          if (c0 + i < K) {
            if (c0 + i == rank) h = r;
            r = fmaf(c[i].A, r, c[i].s);
          }
      }
      if (!finite(r)) {
        r = carry;
        for (int c = 0; c < K; ++c) {
          if (c == rank) h = r;
          r = through(there[c][lane], r);
        }
      }
      carry = r;
    }
    const float first = h;
#pragma unroll
    for (int w = 0; w < MW; ++w)
      if (w < W) {
        sm.in[buf][v][w][lane] = h;
        h = fmaf(m[w].A, h, m[w].s);
      }
    if (!finite(h)) {
      h = first;
#pragma unroll
      for (int w = 0; w < MW; ++w)
        if (w < W) {
          sm.in[buf][v][w][lane] = h;
          h = through(m[w], h);
        }
    }
    if (K == 1) carry = h;
    bar_arrive(kBarStates + buf, threads);
  }
  return carry;
}

// The lane's channels: slots of V channels over all of (B, H, d / V)
struct Lane {
  int b, h, c;
  bool valid;
};
__device__ __forceinline__ Lane find_lane(const ScanArgs& p, int V, uint32_t slots, uint32_t slot, int unit) {
  Lane ln;
  ln.valid = slot < slots;
  // idle lanes read the last slot (where `unit` slots go at once, the last
  // unit's first) and write nothing
  const uint32_t q = ln.valid ? slot : slots - unit;
  const uint32_t per_head = p.d / V, bh = q / per_head;
  ln.c = (int)(q - bh * per_head) * V;
  ln.b = (int)(bh / p.H);
  ln.h = (int)(bh - (uint32_t)ln.b * p.H);
  return ln;
}

// One walk over the tokens in the order of u (forward t = u, backward
// t = L - 1 - u).  S: stages of the ring; C: bytes of a copy into it, 16 (four
// lanes' channels at once), 4 (a lane's own) or 2 (which no asynchronous copy
// takes: loads that wait in registers until the next fetch).
template <typename T, int V, int MW, int R, int S, int C, bool BACK>
__global__ void __launch_bounds__((MW + V) * 32, 2) scan_kernel(ScanArgs p, uint32_t slots, int K, int W) {
  using P = Piece<T, V>;
  using Raw = typename P::Raw;
  constexpr int N = BACK ? 3 : 2;
  constexpr int M = C / (int)sizeof(Raw);             // lanes of a copy
  __shared__ Joint<V, MW> sm;
  extern __shared__ __align__(16) unsigned char ring_bytes[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = K > 1 ? (int)tc::cluster_ctarank() : 0;
  const uint32_t tile = blockIdx.x / K;
  const Lane ln = find_lane(p, V, slots, tile * 32 + lane, 1);
  const int64_t ch = ((int64_t)ln.b * p.H + ln.h) * p.d + ln.c;
  const int step = K * W * R, steps = (p.L + step - 1) / step;
  // read before the clusters' first barrier: `last` may be the same array, and
  // one CTA writes it for all
  float first = 0.f;
  if (warp >= W && p.first != nullptr) first = p.first[ch + warp - W];
  if (K > 1) {
    if (threadIdx.x == 0) {
#pragma unroll
      for (int i = 0; i < 2 * V; ++i) tc::mbar_init(&sm.bar[i / V][i % V], 1);
      tc::fence_barrier_init();
      sm.abort_flag = 0;
    }
    tc::cluster_sync();
  }
  if (warp >= W) {                                    // there are no such warps where W = 1
    const int v = warp - W;
    const float carry = join<V, MW>(sm, reinterpret_cast<Map(*)[32]>(ring_bytes), v, steps, K, W, rank, lane, first,
                                rank == p.quits ? 0 : p.wait_cycles, tc::WaitCtx{&sm.abort_flag, p.status});
    // A CTA whose wait ran out keeps its shared memory until the others of its
    // cluster have ended, whose maps may still be on their way to it (threads
    // that have exited count as arrived).
    if (K > 1 && __any_sync(0xffffffffu, *static_cast<volatile int*>(&sm.abort_flag))) tc::cluster_sync();
    // tokens behind the last one are identities: carry is the state after it
    if (p.last != nullptr && rank == 0 && ln.valid) p.last[ch + v] = carry;
    return;
  }

  // the lane whose channels this thread copies: its own, or where a copy
  // holds several lanes' the first of them
  const Lane cl = M > 1 ? find_lane(p, V, slots, tile * 32 + (lane % (32 / M)) * M, M) : ln;
  auto base = [&](const void* q, const Strides& st, const Lane& at) {
    return static_cast<const T*>(q) + at.b * st.b + at.h * st.h + at.c;
  };
  // arrays in: gates first, then x or dh, then (backward) h of the token before
  const T* src[N];
  int ld[N];
  src[0] = base(p.g, p.gs, cl);
  ld[0] = (int)p.gs.l;
  src[1] = BACK ? base(p.dh, p.dhs, cl) : base(p.x, p.xs, cl);
  ld[1] = (int)(BACK ? p.dhs.l : p.xs.l);
  if constexpr (BACK) {
    src[2] = base(p.h_in, p.his, cl);
    ld[2] = (int)p.his.l;
  }
  T* out = const_cast<T*>(BACK ? base(p.dx, p.dxs, ln) : base(p.h, p.hs, ln));
  T* out2 = BACK ? const_cast<T*>(base(p.dg, p.dgs, ln)) : nullptr;
  const int lo = (int)(BACK ? p.dxs.l : p.hs.l), lo2 = (int)p.dgs.l;

  Raw* ring = reinterpret_cast<Raw*>(ring_bytes + (K > 1 ? 2 * V * K * 32 * sizeof(Map) : 0)) + threadIdx.x;
  constexpr int kRow = MW * 32;                // a constant, so that a run's words have constant offsets
  auto place = [&](int stage, int n, int i) -> Raw* { return ring + stage * (N * R * kRow) + (n * R + i) * kRow; };
  Raw waiting[C == 2 ? N : 1][R];
  int waiting_stage = -1;
  // starts the copies of the run that begins at u
  auto fetch = [&](int stage, int u) {
    if constexpr (C == 2) {
      if (waiting_stage >= 0)
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
          for (int i = 0; i < R; ++i) *place(waiting_stage, n, i) = waiting[n][i];
      waiting_stage = stage;
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
      // h of the token before: none before the first
      const int t0 = (BACK ? p.L - 1 - u : u) - (n == 2 ? 1 : 0), have = p.L - u - (n == 2 ? 1 : 0);
      const int sign = BACK ? -1 : 1;
      if constexpr (C == 2) {
#pragma unroll
        for (int i = 0; i < R; ++i)
          waiting[n][i] =
              i < have ? *reinterpret_cast<const Raw*>(src[n] + (int64_t)(t0 + sign * i) * ld[n]) : Raw{};
      } else {
        const int i0 = lane / (32 / M);               // M tokens of the warp at once
        Raw* to = place(stage, n, i0) + ((lane % (32 / M)) * M - lane);
        if (have >= R) {
          const T* q = src[n] + (int64_t)(t0 + sign * i0) * ld[n];
#pragma unroll
          for (int i = 0; i < R; i += M) copy_async<C>(to + i * kRow, q + (int64_t)(sign * i) * ld[n], true);
        } else {
          for (int i = 0; i < R; i += M) {
            const bool in = i0 + i < have;
            copy_async<C>(to + i * kRow, in ? src[n] + (int64_t)(t0 + sign * (i0 + i)) * ld[n] : src[n], in);
          }
        }
      }
    }
  };
  auto get = [&](int stage, int n, int i) -> Vec<V> { return P::unpack(*place(stage, n, i)); };

  // a run's gates and its map; true if all of it is finite
  auto form = [&](int stage, int buf, Vec<V> (&a)[R], Vec<V>& A, Vec<V>& s) -> bool {
    A = all<V>(1.f);
    s = all<V>(0.f);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      a[i] = exp_(get(stage, 0, i));
      const Vec<V> x = get(stage, 1, i);
      s = BACK ? mul_(a[i], add_(x, s)) : fma_(a[i], s, x);
      A = mul_(A, a[i]);
    }
    // An infinity or NaN lives on in s and A to the end of the run (0 times it
    // is NaN): only then, or where a product is 0, is each gate looked at.
    const Vec<V> r = residue(s, residue(A, all<V>(0.f)));
    bool plain = true;
    if (!(product(A) > sum(r))) {
      plain = sum(r) == 0.f;
      if (!plain) {
        A = all<V>(1.f);
        s = all<V>(0.f);
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const Vec<V> x = get(stage, 1, i);
          if constexpr (BACK) s = apply(a[i], all<V>(0.f), add_(x, s));
          else s = apply(a[i], x, s);
          A = apply(a[i], all<V>(0.f), A);
        }
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float least = a[0].f[v];
#pragma unroll
        for (int i = 1; i < R; ++i) least = fminf(least, a[i].f[v]);
        if (least == 0.f) A.f[v] = -0.f;
      }
    }
    if (W > 1) {
#pragma unroll
      for (int v = 0; v < V; ++v) sm.warp[buf][v][warp][lane] = Map{A.f[v], s.f[v]};
      bar_arrive(kBarMaps + buf, (W + V) * 32);
    }
    return plain;
  };
  // the run's outputs from the state before it
  auto finish = [&](int stage, int u, const Vec<V> (&a)[R], const Vec<V>& in, bool plain) {
    const int have = p.L - u;
    const int t = BACK ? p.L - 1 - u : u;
    T* po = out + (int64_t)t * lo;
    T* po2 = BACK ? out2 + (int64_t)t * lo2 : nullptr;
    // whole runs of finite values (backward: without token 0)
    if (__all_sync(0xffffffffu, plain && finite(in) && ln.valid) && have >= R + (BACK ? 1 : 0)) {
      Vec<V> c = in, odd = all<V>(0.f);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const Vec<V> x = get(stage, 1, i);
        if constexpr (BACK) {
          const Vec<V> dx = add_(x, c);
          c = mul_(a[i], dx);
          const Vec<V> dg = mul_(c, get(stage, 2, i));
          odd = residue(dg, odd);
          *reinterpret_cast<Raw*>(po - (int64_t)i * lo) = P::pack(dx);
          *reinterpret_cast<Raw*>(po2 - (int64_t)i * lo2) = P::pack(dg);
        } else {
          c = fma_(a[i], c, x);
          *reinterpret_cast<Raw*>(po + (int64_t)i * lo) = P::pack(c);
        }
      }
      // forward: a state that grew out of fp32 inside the run is no more finite at its end
      if (none(BACK ? odd : residue(c, odd))) return;
    }
    // the others, those whose state overflows and those whose dg an h that is not finite has touched
    if (!ln.valid) return;
    Vec<V> c = in;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (i < have) {
        const Vec<V> x = get(stage, 1, i);
        if constexpr (BACK) {
          const Vec<V> dx = add_(x, c);
          Vec<V> h = get(stage, 2, i);
          if (t == i) {                               // before token 0: the initial state
#pragma unroll
            for (int v = 0; v < V; ++v) h.f[v] = p.h0 != nullptr ? p.h0[ch + v] : 0.f;
          }
          c = apply(a[i], all<V>(0.f), dx);
          Vec<V> dg;
#pragma unroll
          for (int v = 0; v < V; ++v)                 // a closed gate passes nothing on
            dg.f[v] = a[i].f[v] == 0.f ? 0.f : c.f[v] * h.f[v];
          *reinterpret_cast<Raw*>(po - (int64_t)i * lo) = P::pack(dx);
          *reinterpret_cast<Raw*>(po2 - (int64_t)i * lo2) = P::pack(dg);
        } else {
          c = apply(a[i], x, c);
          *reinterpret_cast<Raw*>(po + (int64_t)i * lo) = P::pack(c);
        }
      }
    }
  };

  int u = (rank * W + warp) * R;
#pragma unroll
  for (int st = 0; st < S; ++st) {
    fetch(st, u + st * step);
    commit();
  }
  auto landed = [&]() {
    wait_but<S - 2>();
    __syncwarp();
  };
  Vec<V> a[R], A, s;
  landed();
  bool plain = form(0, 0, a, A, s);
  if (W == 1) {                                       // one run, one step
    Vec<V> in = all<V>(0.f);
    if (p.first != nullptr)
#pragma unroll
      for (int v = 0; v < V; ++v) in.f[v] = p.first[ch + v];
    finish(0, u, a, in, plain);
    wait_but<0>();
    if (p.last != nullptr && ln.valid)
#pragma unroll
      for (int v = 0; v < V; ++v) p.last[ch + v] = through(Map{A.f[v], s.f[v]}, in.f[v]);
    return;
  }
  int stage = 0, n = 0;
  // one step: forms the next run's gates b while this one's maps are joined
  auto advance = [&](const Vec<V> (&a)[R], bool plain, Vec<V> (&b)[R]) -> bool {
    const int next = stage + 1 == S ? 0 : stage + 1;
    bool plain_next = true;
    if (n + 1 < steps) {
      landed();
      plain_next = form(next, (n + 1) & 1, b, A, s);
    }
    bar_sync(kBarStates + (n & 1), (W + V) * 32);
    Vec<V> in;
#pragma unroll
    for (int v = 0; v < V; ++v) in.f[v] = sm.in[n & 1][v][warp][lane];
    finish(stage, u, a, in, plain);
    __syncwarp();
    fetch(stage, u + S * step);
    commit();
    stage = next;
    u += step;
    ++n;
    return plain_next;
  };
  Vec<V> b[R];
  while (n < steps) {
    plain = advance(a, plain, b);
    if (n < steps) plain = advance(b, plain, a);
  }
  wait_but<0>();
}

template <typename T>
__global__ void scan_step_kernel(const T* x, const T* g, T* h, const float* state, float* new_state, int n) {
  const int i = blockIdx.x * kStepThreads + threadIdx.x;
  if (i >= n) return;
  const Vec<1> v = apply(Vec<1>{expf(to_f32(g[i]))}, Vec<1>{to_f32(x[i])}, Vec<1>{state[i]});
  new_state[i] = v.f[0];
  h[i] = from_f32<T>(v.f[0]);
}

// How many clusters of each size a device holds at once (of 1: CTAs).
struct Fits {
  bool known;
  int clusters[kMaxCluster + 1];
};
template <typename F>
cudaError_t ask_fits(Fits* fits, const void* kernel, int threads, F&& bytes) {
  int per_sm = 0;
  cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, bytes(1));
  if (e != cudaSuccess) return e;
  fits->clusters[1] = per_sm * sm_count();
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  for (int k = 2; k <= kMaxCluster; ++k) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {(unsigned)k, 1, 1};
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)k);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = bytes(k);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&fits->clusters[k], kernel, &cfg);
    if (e != cudaSuccess) return e;
  }
  fits->known = true;
  return cudaSuccess;
}

template <typename T, int V, int MW, int R, int C, bool BACK>
cudaError_t go(const ScanArgs& a, cudaStream_t stream) {
  constexpr int S = kStages;
  const auto kernel = scan_kernel<T, V, MW, R, S, C, BACK>;
  const void* id = reinterpret_cast<const void*>(kernel);
  const int64_t slots = (int64_t)a.B * a.H * (a.d / V), tiles = (slots + 31) / 32;
  const int64_t runs = ((int64_t)a.L + R - 1) / R;
  int W = 1, K = 1;
  while (W < MW && W < runs) W *= 2;
  constexpr size_t ring = (size_t)S * (BACK ? 3 : 2) * R * MW * 32 * sizeof(typename Piece<T, V>::Raw);
  auto bytes = [](int k) { return ring + (k > 1 ? 2 * V * k * 32 * sizeof(Map) : 0); };
  cudaError_t e = ensure_dynamic_smem(id, bytes(kMaxCluster));
  if (e != cudaSuccess) return e;
  if (runs > MW) {
    // CTAs of a cluster: a wave of clusters of K takes time as 1 / K.  The
    // smallest K whose waves take at most a tenth longer than the best's.  A
    // GB300 holds 304 CTAs at once, but only 152, 97, 74, 58, 46, 38, 36, 30, 28,
    // 23, 23, 19, 14, 14, 14 clusters of 2, 3, .. 16.  Every K measured, in us
    // (V = forward, A = backward; K = 4, 6, 8, 9, 12, 13, 16):
    //   V bf16  16 tiles x 12288   48.1  33.8  32.8  32.0 *25.3  26.2  37.0
    //   V bf16  32 tiles x 8192    35.7  31.7 *25.5  41.4  37.3  37.0  44.3
    //   V bf16  64 tiles x 8192   *43.3  59.9  48.3  65.3  56.5  70.7  74.4
    //   V fp32  64 tiles x 8192   *36.5  48.0  40.8  51.5  50.2  63.3  66.7
    //   A bf16  16 tiles x 12288   54.6  38.7  46.4  43.7 *34.1  35.9  46.6
    //   A bf16  32 tiles x 8192    38.8  43.0 *35.6  48.9  47.5  49.0  53.1
    //   A fp32  64 tiles x 8192   *51.1  67.6  55.6  69.0  62.6  77.0  80.8
    //   A fp32  19 tiles x 1777    12.1   9.9  11.1  11.1  *9.2   9.6  12.5
    // (* the rule's; the fastest of all sixteen in each).  At 256 tiles it is 1
    // (78.4, K = 2 84.0; backward 106.4 and 114.3).  The rule is off at 8 tiles x
    // 16384, where 12 takes 25.4 and 30.3 us and it has 16 take 26.9 and 37.5;
    // of the sizes it does not try, 5 would be faster at 48 tiles x 8192 (36.9,
    // with 4 42.0).
    static std::mutex mu;
    static Fits known[64];
    int dev = 0;
    e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    Fits fits;
    {
      std::lock_guard<std::mutex> lock(mu);
      if (!known[dev].known) {
        e = ask_fits(&known[dev], id, (W + V) * 32, bytes);
        if (e != cudaSuccess) return e;
      }
      fits = known[dev];
    }
    double best = 0;
    for (const bool pick : {false, true})
      for (const int k : {1, 2, 3, 4, 6, 8, 12, 16}) {
        if (fits.clusters[k] < 1 || (k > 1 && (int64_t)(k - 1) * W >= runs)) continue;
        const int64_t waves = (tiles + fits.clusters[k] - 1) / fits.clusters[k];
        const double rate = (double)k / (double)waves;
        if (!pick) {
          best = rate > best ? rate : best;
        } else if (rate >= 0.9 * best) {
          K = k;
          break;
        }
      }
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {(unsigned)K, 1, 1};
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(tiles * K));
  cfg.blockDim = dim3(W > 1 ? (W + V) * 32 : 32);
  cfg.dynamicSmemBytes = bytes(K);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = K > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, a, (uint32_t)slots, K, W);
}

template <bool BACK>
cudaError_t go(const ScanArgs& a, bool bf16, int align, cudaStream_t stream) {
  using B16 = __nv_bfloat16;
  // 16-byte copies where every row is made of whole ones (a quarter of the
  // copy instructions), else 4-byte ones; bf16 channels in pairs where rows are
  // made of whole pairs, else one by one.  4 x 8 heads x 8192 x 64 bf16
  // forward: 24.9, 32.5 and 48.5 us; fp32 36.3 and 59.0; 2 x 8 x 12288 x 64
  // bf16 backward: 34.1, 45.7 and 58.5.
  // Workers of a CTA and tokens of a run.  Longer runs share what a run costs
  // among more tokens, as far as two runs' gates stay in registers: forward
  // 4 x 16 against 8 x 8 bf16 24.9 against 26.9 us (4 x 8 x 8192 x 64), 4 x 24
  // against 8 x 8 fp32 238 against 264 us (65536 x 2048; 4 x 28 247).  The
  // backward pass, with three arrays in its ring, spills at 16 and keeps 8 x 8
  // (bf16, 2 x 8 x 12288 x 64: 34.0 us, 4 x 16 35.1, 4 x 12 34.9).
  if constexpr (BACK) {
    if (!bf16) return align >= 16 ? go<float, 1, 8, 8, 16, BACK>(a, stream) : go<float, 1, 8, 8, 4, BACK>(a, stream);
    if (align >= 4)
      return align >= 16 ? go<B16, 2, 8, 8, 16, BACK>(a, stream) : go<B16, 2, 8, 8, 4, BACK>(a, stream);
  } else {
    if (!bf16) return align >= 16 ? go<float, 1, 4, 24, 16, BACK>(a, stream) : go<float, 1, 4, 24, 4, BACK>(a, stream);
    if (align >= 4)
      return align >= 16 ? go<B16, 2, 4, 16, 16, BACK>(a, stream) : go<B16, 2, 4, 16, 4, BACK>(a, stream);
  }
  return go<B16, 1, 8, 8, 2, BACK>(a, stream);
}

}  // namespace

cudaError_t launch_scan(const ScanArgs& a, bool backward, bool bf16, int align, cudaStream_t stream) {
  return backward ? go<true>(a, bf16, align, stream) : go<false>(a, bf16, align, stream);
}

cudaError_t launch_scan_step(const void* x, const void* g, void* h, const float* state, float* new_state, int64_t n,
                             bool bf16, cudaStream_t stream) {
  const unsigned grid = (unsigned)((n + kStepThreads - 1) / kStepThreads);
  if (bf16)
    scan_step_kernel<<<grid, kStepThreads, 0, stream>>>(static_cast<const __nv_bfloat16*>(x),
                                                        static_cast<const __nv_bfloat16*>(g),
                                                        static_cast<__nv_bfloat16*>(h), state, new_state, (int)n);
  else
    scan_step_kernel<<<grid, kStepThreads, 0, stream>>>(static_cast<const float*>(x), static_cast<const float*>(g),
                                                        static_cast<float*>(h), state, new_state, (int)n);
  return cudaGetLastError();
}

}  // namespace favor
