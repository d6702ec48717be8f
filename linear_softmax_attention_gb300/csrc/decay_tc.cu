// Causal linear attention with a decay per head on the tensor cores: bf16, d <=
// 128 in whole 16-byte pieces (decay.cuh has the form that every pass follows).
//
// The gains of the segments come first, exact to fp32's sums: b's faded rows are
// kept as three bf16 parts (24 bits; two were 2.5e-6 off), c's rows as they are, and
// each chunk's products are added up in registers (the tensor cores cut their sums
// off: 32 chunks in one accumulator were 4e-6 off, single ones are 1e-7).
// From them come the states that segments start from and the states returned.
//
// A pass then walks each segment's chunks.  P = A B^T; P is faded and masked on
// its way from tensor memory to registers and back, as the bf16 operand of O = P C;
// rows leave as O + r(i) I with I = A M.  The state M stays in fp32 in tensor
// memory and meets A as two bf16 parts; what it takes in are the products of c's
// rows with b's, faded and rounded to bf16 (in b's own place).  So a term of o is
// rounded once beside o itself: its weight within a chunk, its key across chunks.
// The decays never appear as l^-j: every factor is a power l^n, n >= 0.
//
// One warp issues the products, one the copies; the others share the work on
// registers, 32 columns of a quarter of the lanes each:
//   weights (P -> P')       while the gain's and I's products run before it,
//   b's faded rows          while O = P' C runs,
//   rows out (O, I -> o)    while the gain runs,
//   the state's copy, faded while the next chunk's P runs.
//
// Two CTAs on an SM take 5000 to 5600 cycles for a chunk of d = 64 each, whose bytes
// are 5700 of the SM's share of memory's rate (b and c may still be in the L2 cache):
// what is left lies around them.  The gains read b's and c's rows a first time (1600
// cycles a chunk, 1420 by the bytes), there are three launches, each CTA's first chunk
// waits for everything, and CTAs do not come out even (256 on 304 places).  Measured (one GB300): 8
// x 8 x 4096 x 64 54 us (gains 20, scan 5, pass 29; floor 20), 1 x 16 x 65536 x 128 350
// us (161), backward of 2 x 8 x 12288 x 64 87 us (26) and of 8 x 8 x 4096 x 64 113 (35).
// The tensor pipe is 20 to 27 % busy, DRAM 37 to 49 %.  On the CUDA cores the same
// shapes took 363 us (8 x 8 x 4096 x 64), 916 (1 x 16 x 16384 x 128; here 108) and,
// of 64 tokens in each of 32 heads, 13.5 (here 8.7).
#include <string.h>

#include <algorithm>

#include "decay_tc.cuh"
#include "tc_util.cuh"

namespace favor {
namespace {

using namespace tc;

constexpr int kM = 128;              // tokens of a chunk
// Chunks of a sequence that is one segment and whose gains run beside the passes:
// 32 heads of 64 tokens 8.7 us (gains, scan and pass behind one another 13.0), of 333
// 13.5 (15.5), of 512 16.1 (16.8), of 1024 24.4 (20.6); 256 heads of 512 35 (40).
constexpr int kShort = 4;

template <int D> struct Cfg {
  static constexpr int kParts = D / 32;                    // warps of a quarter of the lanes, 32 columns each
  static constexpr int kEpi = 128 * kParts, kEpiWarps = 4 * kParts;
  static constexpr int kThreads = kEpi + 64;
  static constexpr int kCtas = D == 64 ? 2 : 1;            // of an SM
  static constexpr int kAtoms = D / 64;                    // 128-byte columns of a tile
  static constexpr int kTile = kAtoms * kAtom;
  // the pass: a ring of tiles (two chunks at d <= 64) and the state's copy, [2 D rows: hi, rest][D]
  static constexpr int kSlots = D == 64 ? 6 : 5;
  static constexpr int kImg = kSlots * kTile;
  static constexpr int kImgAtom = 2 * D * 128;
  static constexpr int kBars = kImg + kAtoms * kImgAtom;
  static constexpr int kPowers = kBars + 176;              // l^15 .. l^0 (walking back: l^0 .. l^15)
  static constexpr int kDiag = kPowers + 64;               // factors of a diagonal group, see below
  static constexpr int kFade = kDiag + 64 * 4;             // l^0 .. l^128
  static constexpr int kSmem = kFade + 129 * 4;
  // tensor memory: P (P' over its first half), O, I, M
  static constexpr uint32_t kCols = D == 64 ? 256 : 512;
  static constexpr uint32_t kP = 0, kO = D == 64 ? 64 : 128, kI = D == 64 ? 128 : 256, kState = D == 64 ? 192 : 384;
  // the gains (64 of b's columns a CTA): tiles of chunks to come, and b's rows in three parts, twice
  static constexpr int kDepthB = D == 64 ? 4 : 2, kDepthC = D == 64 ? 4 : 3;
  static constexpr int kTilesC = kDepthB * kAtom;
  static constexpr int kSplit = kTilesC + kDepthC * kTile;
  static constexpr int kGainBars = kSplit + 2 * 3 * kAtom;
  static constexpr int kGainSmem = kGainBars + 192;
};
// an SM's 228 KB, 1 KB of it reserved for each CTA
static_assert(2 * (Cfg<64>::kSmem + 1024) <= 233472 && Cfg<128>::kSmem <= 232448, "shared memory");
static_assert(Cfg<64>::kGainSmem <= 232448 && Cfg<128>::kGainSmem <= 232448, "shared memory");
// gains that wait for the passes beside them are never on an SM with one of those, which could want their tensor memory
static_assert(Cfg<64>::kSmem + Cfg<64>::kGainSmem > 233472 && Cfg<128>::kSmem + Cfg<128>::kGainSmem > 233472, "apart");

// waits for a phase although other waits have run out: copies and products in
// flight must end before their memory goes
__device__ __forceinline__ void drain(uint64_t* bar, uint32_t parity) {
  const long long t0 = sm_cycles();
  while (!mbar_try_wait(smem_addr(bar), parity) && sm_cycles() - t0 <= kWaitLimitCycles) {
  }
}

// bar.sync among `count` threads; whether any of them has v
__device__ __forceinline__ bool named_bar_or(int id, int count, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %3, 0;\n\t"
      "barrier.cta.red.or.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(count), "r"(v ? 1u : 0u)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ __forceinline__ float2 both(uint32_t w) { return make_float2(bf_lo(w), bf_hi(w)); }
__device__ __forceinline__ uint32_t pack2(float2 v) { return pack_bf16(v.x, v.y); }
template <int N> __device__ __forceinline__ float2 pair(const uint32_t (&x)[N], int e) {
  return make_float2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1]));
}

// 32 columns of row `row` of a tile times u, rounded to bf16, in their place; 0 where !in
__device__ __forceinline__ void fade_rows(uint8_t* tile, int row, int part, float u, bool in) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int col = part * 32 + c * 8;
    uint4* at = reinterpret_cast<uint4*>(tile + (col >> 6) * kAtom + row * 128 +
                                         ((((col & 63) >> 3) ^ (row & 7)) << 4));
    uint4 w = in ? *at : make_uint4(0, 0, 0, 0);
    w.x = pack2(mul2(both(w.x), make_float2(u, u)));
    w.y = pack2(mul2(both(w.y), make_float2(u, u)));
    w.z = pack2(mul2(both(w.z), make_float2(u, u)));
    w.w = pack2(mul2(both(w.w), make_float2(u, u)));
    *at = w;
  }
}

// 32 columns of a row of a 64-column tile times u as three bf16 parts, whose sum has all of fp32's bits
__device__ __forceinline__ void fade_rows3(const uint8_t* tile, uint8_t* parts, int row, int part, float u, bool in) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int off = row * 128 + (((part * 4 + c) ^ (row & 7)) << 4);
    const uint4 raw = in ? *reinterpret_cast<const uint4*>(tile + off) : make_uint4(0, 0, 0, 0);
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    uint32_t h[3][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 a = mul2(both(w[i]), make_float2(u, u));
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        h[k][i] = pack2(a);
        if (k < 2) a = fma2(both(h[k][i]), make_float2(-1.f, -1.f), a);
      }
    }
#pragma unroll
    for (int k = 0; k < 3; ++k)
      *reinterpret_cast<uint4*>(parts + k * kAtom + off) = make_uint4(h[k][0], h[k][1], h[k][2], h[k][3]);
  }
}

// rows [n, 128) of a tile: 0 (what lies behind a sequence's end may be anything)
template <int D>
__device__ __forceinline__ void clear_rows(uint8_t* tile, int n, int tid, int threads) {
  for (int e = tid; e < (kM - n) * 8 * Cfg<D>::kAtoms; e += threads) {
    const int a = e / ((kM - n) * 8), r = e - a * (kM - n) * 8;
    *reinterpret_cast<uint4*>(tile + a * kAtom + n * 128 + r * 16) = make_uint4(0, 0, 0, 0);
  }
}

// acc [128 lanes][N] (+)= a^T b over a chunk's 128 tokens; a's columns in atoms `lbo` apart (0: at
// d <= 64 the upper half of the lanes repeats the lower one)
template <int N>
__device__ __forceinline__ void issue_gain(uint32_t acc, uint32_t a, uint32_t lbo, uint32_t b, bool add) {
  constexpr uint32_t id = idesc_bf16(kM, N, true, true);
  const uint64_t a0 = sdesc(a, lbo, 1024), b0 = sdesc(b, kAtom, 1024);
#pragma unroll
  for (int k = 0; k < kM / 16; ++k) mma_bf16(acc, dadd(a0, kstep_mn(k)), dadd(b0, kstep_mn(k)), id, add || k > 0);
}

// ---------------------------------------------------------------------------
// a pass
// ---------------------------------------------------------------------------
struct PassParams {
  DecayShape s;
  // what each segment starts from, `step` elements apart, NULL: zeros
  const float* start;
  int64_t step;
  bool transposed;                    // it holds M^T
  bool rev;
  float s_w, s_r, s_u;
  const __nv_bfloat16* c;             // for rows with infinities or NaN
  __nv_bfloat16* o;                   // for rows behind a sequence's last chunk
  Strides cs, os;
};

template <int D>
__device__ __forceinline__ void pass_body(const CUtensorMap& map_a, const CUtensorMap& map_b, const CUtensorMap& map_c,
                                          const CUtensorMap& map_o, const PassParams& p, uint8_t* sm) {
  using C = Cfg<D>;
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + C::kBars);          // [kSlots]
  uint64_t *scores = full + 6, *out_bar = full + 7, *gain_bar = full + 8, *again_bar = full + 9;
  uint64_t *weights_done = full + 10, *faded_done = full + 11, *rows_done = full + 12, *copy_done = full + 13;
  uint64_t* end_bar = full + 14;
  // What the copies' warp waits for, by the chunk's parity: nothing but its own copies keeps the others from running
  // on, and a phase that is followed by another before it is looked at would never be seen (chunk i + 2 needs copies
  // that are made after the waits for chunk i, so that no barrier runs two phases ahead).
  uint64_t *rows_free = full + 15, *gain_free = full + 17;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(full + 19);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint32_t* odd_rows = reinterpret_cast<uint32_t*>(full + 20);          // [4] rows of c with infinities or NaN
  float* powers = reinterpret_cast<float*>(sm + C::kPowers);
  float* diag = reinterpret_cast<float*>(sm + C::kDiag);
  float* fade = reinterpret_cast<float*>(sm + C::kFade);

  const DecayShape& s = p.s;
  const bool rev = p.rev;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int bh = blockIdx.x / s.segs, seg = blockIdx.x - bh * s.segs, b = bh / s.H, h = bh - b * s.H;
  const float g2 = s.g[h] * kLog2e;
  const int len = decay_length(s, b), first = seg * s.seg_tokens, end = min(first + s.seg_tokens, s.L);
  const int stop = min(end, len);
  const int live = stop > first ? (stop - first + kM - 1) / kM : 0;     // chunks with tokens
  const WaitCtx wctx{abort_flag, s.status};
  // the i-th chunk in the pass's order
  auto token0 = [&](int i) { return first + (rev ? live - 1 - i : i) * kM; };
  auto tokens = [&](int i) { return min(kM, stop - token0(i)); };
  // its tiles: kind 0: b, 1: a, 2: c
  auto slot = [&](int i, int kind) { return sm + ((3 * i + kind) % C::kSlots) * C::kTile; };
  auto slot_full = [&](int i, int kind) { return full + (3 * i + kind) % C::kSlots; };
  auto slot_phase = [&](int i, int kind) { return ((3 * i + kind) / C::kSlots) & 1; };

  if (threadIdx.x == 0) {
    for (int i = 0; i < 10; ++i) mbar_init(full + i, 1);
    for (int i = 10; i < 14; ++i) mbar_init(full + i, C::kEpiWarps);
    mbar_init(end_bar, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(rows_free + i, C::kEpiWarps);
      mbar_init(gain_free + i, 1);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == C::kEpiWarps) {
    tmem_alloc(tmem_slot, C::kCols);
    tmem_relinquish();
  }
  // diag[31 - i + j]: the weight of column j for row i of a 32 x 32 group on the diagonal
  for (int e = threadIdx.x; e < 129 + 16 + 63; e += C::kThreads) {
    const int k = e < 129 ? e : e < 145 ? (rev ? e - 129 : 144 - e) : rev ? e - 145 - 31 : 31 - (e - 145);
    const float f = k < 0 ? 0.f : decay_power(g2, k);
    if (e < 129) fade[e] = f;
    else if (e < 145) powers[e - 129] = f;
    else diag[e - 145] = f * p.s_w;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == C::kEpiWarps) {
    // ---- products
    if (lane == 0) {
      bool ok = true;
      for (int i = 0; i < live; ++i) {
        ok = mbar_wait(slot_full(i, 0), slot_phase(i, 0), wctx) && mbar_wait(slot_full(i, 1), slot_phase(i, 1), wctx);
        if (!ok) break;
        const uint64_t a0 = sdesc(smem_addr(slot(i, 1)), 16, 1024);
        {
          constexpr uint32_t id = idesc_bf16(kM, kM, false, false);
          const uint64_t b0 = sdesc(smem_addr(slot(i, 0)), 16, 1024);
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            mma_bf16(tmem + C::kP, dadd(a0, kstep_k(k, kAtom)), dadd(b0, kstep_k(k, kAtom)), id, k > 0);
          mma_commit(scores);
        }
        constexpr uint32_t id = idesc_bf16(kM, D, false, true);
        ok = mbar_wait(copy_done, i & 1, wctx);
        if (!ok) break;
        tc_fence_after();
        {
          const uint64_t m0 = sdesc(smem_addr(sm + C::kImg), C::kImgAtom, 1024);
#pragma unroll
          for (int k = 0; k < 2 * D / 16; ++k)
            mma_bf16(tmem + C::kI, dadd(a0, kstep_k(k % (D / 16), kAtom)), dadd(m0, kstep_mn(k)), id, k > 0);
        }
        ok = mbar_wait(slot_full(i, 2), slot_phase(i, 2), wctx) && mbar_wait(weights_done, i & 1, wctx);
        if (!ok) break;
        tc_fence_after();
        const uint64_t c0 = sdesc(smem_addr(slot(i, 2)), kAtom, 1024);
#pragma unroll
        for (int k = 0; k < kM / 16; ++k)
          mma_bf16_ts(tmem + C::kO, tmem + C::kP + k * 8, dadd(c0, kstep_mn(k)), id, k > 0);
        mma_commit(out_bar);
        if (i + 1 < live) {
          ok = mbar_wait(faded_done, i & 1, wctx);
          if (!ok) break;
          tc_fence_after();
          issue_gain<D>(tmem + C::kState, smem_addr(slot(i, 0)), D == 64 ? 0 : kAtom, smem_addr(slot(i, 2)), true);
          mma_commit(gain_bar);
          mma_commit(gain_free + (i & 1));
        }
        ok = mbar_wait(rows_done, i & 1, wctx);                  // P and O are read
        if (!ok) break;
        tc_fence_after();
      }
      // after a wait that ran out (the others may then arrive without having waited): what is in flight ends before its
      // memory goes
      if (!ok || *abort_flag) {
        mma_commit(end_bar);
        drain(end_bar, 0);
      }
    }
    __syncwarp();
  } else if (warp == C::kEpiWarps + 1) {
    // ---- copies
    if (lane == 0) {
      uint32_t issued = 0, phases = 0;                           // of the slots
      auto load = [&](int i, int kind) {
        if (i >= live) return;
        const uint32_t bit = 1u << ((3 * i + kind) % C::kSlots);
        issued |= bit;
        phases = slot_phase(i, kind) ? phases | bit : phases & ~bit;
        const CUtensorMap* map = kind == 0 ? &map_b : kind == 1 ? &map_a : &map_c;
        uint64_t* bar = slot_full(i, kind);
        mbar_arrive_expect_tx(bar, C::kTile);
#pragma unroll
        for (int a = 0; a < C::kAtoms; ++a) tma_load_4d(slot(i, kind) + a * kAtom, map, a * 64, token0(i), h, b, bar);
      };
      load(0, 0);
      load(0, 1);
      load(0, 2);
      load(1, 0);
      load(1, 1);
      if (C::kSlots == 6) load(1, 2);
      bool ok = true;
      for (int i = 0; i < live; ++i) {
        ok = mbar_wait(rows_free + (i & 1), i >> 1 & 1, wctx);
        if (!ok) break;
#pragma unroll
        for (int a = 0; a < C::kAtoms; ++a) tma_store_4d(&map_o, a * 64, token0(i), h, b, slot(i, 1) + a * kAtom);
        bulk_commit();
        if (i + 1 == live) break;
        // b and c are read, and the rows leave from a's place
        ok = mbar_wait(gain_free + (i & 1), i >> 1 & 1, wctx);
        if (!ok) break;
        if constexpr (C::kSlots == 6) {
          load(i + 2, 0);
          load(i + 2, 2);
        } else {
          load(i + 1, 2);
          load(i + 2, 1);
        }
        bulk_wait_read0();
        load(i + 2, C::kSlots == 6 ? 1 : 0);
      }
      bulk_wait0();
      if (!ok || *abort_flag)
        for (int x = 0; x < C::kSlots; ++x)
          if (issued >> x & 1) drain(full + x, phases >> x & 1);
    }
    __syncwarp();
  } else {
    const int q = warp & 3, part = warp >> 2, t = 32 * q + lane;        // this thread's lane of tensor memory, columns
    const uint32_t lane_off = static_cast<uint32_t>(32 * q) << 16;
    const int x = t & (D - 1);                                           // its row of the state
    int again = 0;

    // The state's copy for I = A M, as hi part and rest (at d <= 64 the lanes' lower half writes one, the upper
    // half, which repeats it, the other); the state itself fades over the chunk.
    auto copy_state = [&](uint32_t (&m)[32], float all) {
      uint32_t w[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) w[e] = pack2(pair(m, e));
      const uint32_t img = smem_addr(sm + C::kImg);
      if (D == 128 || t < 64) store_row<16>(img, C::kImgAtom, x, part * 32, w);
      if (D == 128 || t >= 64) {
#pragma unroll
        for (int e = 0; e < 16; ++e)
          w[e] = pack2(fma2(both(w[e]), make_float2(-1.f, -1.f), pair(m, e)));
        store_row<16>(img, C::kImgAtom, D + x, part * 32, w);
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float2 v = mul2(pair(m, e), make_float2(all, all));
        m[2 * e] = __float_as_uint(v.x);
        m[2 * e + 1] = __float_as_uint(v.y);
      }
      tmem_st32(tmem + C::kState + lane_off + part * 32, m);
      tmem_st_wait();
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(copy_done);
    };

    // The state that the segment starts from, through the copy's place in shared memory ([D][D] fp32, 16-byte pieces of
    // row x moved by x mod 8).
    {
      const int d = s.d, d4 = d / 4;
      float4* state = reinterpret_cast<float4*>(sm + C::kImg);
      griddep_wait();                                                    // the states are written
      const float4* from = reinterpret_cast<const float4*>(p.start + ((int64_t)bh * s.segs + seg) * p.step);
      constexpr int kPlaces = 4;
#pragma unroll
      for (int e0 = threadIdx.x; e0 < D * D / 4; e0 += kPlaces * C::kEpi) {
        float4 m[kPlaces];
#pragma unroll
        for (int k = 0; k < kPlaces; ++k) {
          const int e = e0 + k * C::kEpi, row = e / (D / 4), c = e & (D / 4 - 1);
          m[k] = p.start != nullptr && row < d && c < d4 ? from[row * d4 + c] : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int k = 0; k < kPlaces; ++k) {
          const int e = e0 + k * C::kEpi, row = e / (D / 4), c = e & (D / 4 - 1);
          state[row * (D / 4) + (c ^ (row & 7))] = m[k];
        }
      }
      if (live > 0) {
        named_bar(5, C::kEpi);
        uint32_t w[32];
        if (!p.transposed) {
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float4 v = state[x * (D / 4) + ((part * 8 + e / 4) ^ (x & 7))];
            w[e] = __float_as_uint(v.x);
            w[e + 1] = __float_as_uint(v.y);
            w[e + 2] = __float_as_uint(v.z);
            w[e + 3] = __float_as_uint(v.w);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const int row = part * 32 + e;
            w[e] = reinterpret_cast<const uint32_t*>(state)[row * D + (((x >> 2) ^ (row & 7)) << 2) + (x & 3)];
          }
        }
        named_bar(5, C::kEpi);                                           // the copy takes the place
        copy_state(w, fade[tokens(0)]);
      }
    }

    for (int i = 0; i < live; ++i) {
      const int n = tokens(i);
      // ---- the weights: faded, masked, rounded to bf16
      if (n < kM && token0(i) + n < s.L) {
        mbar_wait(slot_full(i, 2), slot_phase(i, 2), wctx);
        clear_rows<D>(slot(i, 2), n, threadIdx.x, C::kEpi);
        fence_proxy_async_smem();
      }
      mbar_wait(scores, i & 1, wctx);
      __syncwarp();
      tc_fence_after();
      {
        constexpr int G = 4 / C::kParts;                         // groups of 32 columns of a thread
        float2 power[8];                                         // l^(15 - k), walking back l^k
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const float4 v = *reinterpret_cast<const float4*>(powers + 2 * e);
          power[e] = make_float2(v.x, v.y);
          power[e + 1] = make_float2(v.z, v.w);
        }
        uint32_t w[G][16];
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const int grp = part * G + g, j0 = grp * 32;
          if (rev ? grp < q : grp > q) {
#pragma unroll
            for (int e = 0; e < 16; ++e) w[g][e] = 0u;
            continue;
          }
          uint32_t sc[32];
          tmem_ld32(tmem + C::kP + lane_off + j0, sc);
          tmem_ld_wait();
          if (grp != q) {
            // 16 columns from jh on: l^(t - j) = l^(t - jh - 15) l^(15 - k), l^(j - t) = l^(jh - t) l^k
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const float base = p.s_w * fade[rev ? j0 + 16 * hf - t : t - j0 - 16 * hf - 15];
#pragma unroll
              for (int e = 0; e < 8; ++e)
                w[g][8 * hf + e] = pack2(mul2(pair(sc, 8 * hf + e), mul2(make_float2(base, base), power[e])));
            }
            if (rev && n < j0 + 32) {
              // columns behind the last token (a sequence's last chunk)
#pragma unroll
              for (int e = 0; e < 16; ++e)
                w[g][e] &= (j0 + 2 * e < n ? 0xffffu : 0u) | (j0 + 2 * e + 1 < n ? 0xffff0000u : 0u);
            }
          } else {
            const float* f = diag + 31 - lane;
            uint32_t in = rev ? 0xffffffffu << lane : 0xffffffffu >> (31 - lane);
            if (n < j0 + 32) in &= n > j0 ? (1u << (n - j0)) - 1 : 0u;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float v0 = __uint_as_float(sc[2 * e]) * f[2 * e], v1 = __uint_as_float(sc[2 * e + 1]) * f[2 * e + 1];
              w[g][e] = pack_bf16(in >> (2 * e) & 1 ? v0 : 0.f, in >> (2 * e + 1) & 1 ? v1 : 0.f);
            }
          }
        }
        // the weights take the scores' columns: every warp of these lanes has read its own
        tc_fence_before();
        named_bar(1 + q, 32 * C::kParts);
        tc_fence_after();
#pragma unroll
        for (int g = 0; g < G; ++g) tmem_st16(tmem + C::kP + lane_off + (part * G + g) * 16, w[g]);
        tmem_st_wait();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(weights_done);
      // ---- b's faded rows in b's place (P has read it)
      if (i + 1 < live) {
        const int row = threadIdx.x & 127;
        fade_rows(slot(i, 0), row, threadIdx.x >> 7, row < n ? p.s_u * fade[rev ? row + 1 : n - 1 - row] : 0.f, row < n);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(faded_done);
      }
      // ---- rows out, through a's place
      mbar_wait(out_bar, i & 1, wctx);
      __syncwarp();
      tc_fence_after();
      const float r = t < n ? p.s_r * fade[rev ? n - 1 - t : t + 1] : 0.f;
      for (bool patch = false;;) {
        uint32_t o[32], in[32];
        tmem_ld32(tmem + C::kO + lane_off + part * 32, o);
        tmem_ld32(tmem + C::kI + lane_off + part * 32, in);
        tmem_ld_wait();
        if (patch) {
          // what the infinities and NaN of c's rows, left out of the product, add to the rows that see them
          const __nv_bfloat16* c = p.c + b * p.cs.b + h * p.cs.h + (int64_t)token0(i) * p.cs.l;
          for (int j = 0; j < n; ++j) {
            if (!(odd_rows[j >> 5] >> (j & 31) & 1)) continue;
            const uint32_t pair = tmem_ld1(tmem + C::kP + lane_off + (j >> 1));
            tmem_ld_wait();
            const float w = j & 1 ? bf_hi(pair) : bf_lo(pair);
            const bool sees = rev ? j >= t : j <= t;
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const int y = part * 32 + e;
              const float v = y < s.d ? __bfloat162float(c[j * p.cs.l + y]) : 0.f;
              if (sees && v * 0.f != 0.f) o[e] = __float_as_uint(fmaf(w, v, __uint_as_float(o[e])));
            }
          }
        }
        float2 bad = make_float2(0.f, 0.f);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float2 v = pair(o, e);
          bad = fma2(v, make_float2(0.f, 0.f), bad);
          o[e] = t < n ? pack2(fma2(pair(in, e), make_float2(r, r), v)) : 0u;
        }
        store_row<16>(smem_addr(slot(i, 1)), kAtom, t, part * 32, o);
        // rare: a product with zero weights has met infinities or NaN of rows that must not be seen
        const bool odd = named_bar_or(5, C::kEpi, !patch && t < n && bad.x + bad.y != 0.f);
        if (!odd) break;
        uint8_t* ct = slot(i, 2);
        if (threadIdx.x < 4) odd_rows[threadIdx.x] = 0;
        // the gain has read c
        if (i + 1 < live) mbar_wait(gain_bar, i & 1, wctx);
        named_bar(5, C::kEpi);
#pragma unroll 1
        for (int e = threadIdx.x; e < C::kTile / 16; e += C::kEpi) {
          uint4 raw = *reinterpret_cast<const uint4*>(ct + e * 16);
          uint32_t v[4] = {raw.x, raw.y, raw.z, raw.w};
          bool found = false;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if ((v[k] & 0x7f80u) == 0x7f80u) {
              v[k] &= 0xffff0000u;
              found = true;
            }
            if ((v[k] & 0x7f800000u) == 0x7f800000u) {
              v[k] &= 0xffffu;
              found = true;
            }
          }
          if (found) {
            const int row = (e * 16 % kAtom) / 128;
            *reinterpret_cast<uint4*>(ct + e * 16) = make_uint4(v[0], v[1], v[2], v[3]);
            atomicOr(&odd_rows[row >> 5], 1u << (row & 31));
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        named_bar(5, C::kEpi);
        const bool made = threadIdx.x == 0 && !*abort_flag;
        if (made) {
          tc_fence_after();
          constexpr uint32_t id = idesc_bf16(kM, D, false, true);
          const uint64_t c0 = sdesc(smem_addr(ct), kAtom, 1024);
#pragma unroll 1
          for (int k = 0; k < kM / 16; ++k)
            mma_bf16_ts(tmem + C::kO, tmem + C::kP + k * 8, dadd(c0, kstep_mn(k)), id, k > 0);
          mma_commit(again_bar);
        }
        __syncwarp();
        if (!mbar_wait(again_bar, again & 1, wctx) && made) drain(again_bar, again & 1);
        ++again;
        __syncwarp();
        tc_fence_after();
        patch = true;
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(rows_done);
        mbar_arrive(rows_free + (i & 1));
      }
      // ---- the next chunk's copy of the state
      if (i + 1 < live) {
        mbar_wait(gain_bar, i & 1, wctx);
        __syncwarp();
        tc_fence_after();
        uint32_t m[32];
        tmem_ld32(tmem + C::kState + lane_off + part * 32, m);
        tmem_ld_wait();
        copy_state(m, fade[tokens(i + 1)]);
      }
    }
    // rows of chunks behind the sequence's end
    if (first + live * kM < end) {
      __nv_bfloat16* o = p.o + b * p.os.b + h * p.os.h;
      const int from = first + live * kM, d8 = s.d / 8;
      for (int64_t e = threadIdx.x; e < (int64_t)(end - from) * d8; e += C::kEpi) {
        const int row = (int)(e / d8), c = (int)(e - (int64_t)row * d8) * 8;
        *reinterpret_cast<uint4*>(o + (int64_t)(from + row) * p.os.l + c) = make_uint4(0, 0, 0, 0);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == C::kEpiWarps) tmem_dealloc(tmem, C::kCols);
}

// Up to three passes side by side (the gradients'), blockIdx.y the pass
struct Passes {
  CUtensorMap a[3], b[3], c[3], o[3];
  PassParams p[3];
};

template <int D>
__global__ void __launch_bounds__(Cfg<D>::kThreads, Cfg<D>::kCtas)
    decay_tc_pass_kernel(const __grid_constant__ Passes ps) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const int k = blockIdx.y;
  // what runs beside the passes may start (one segment: the gains; others wait for the passes' end)
  asm volatile("griddepcontrol.launch_dependents;");
  if (smem_addr(smem) % 1024 != 0) {                             // tiles are read by 1024-byte swizzle blocks
    if (threadIdx.x == 0) report_status(ps.p[k].s.status, FAVOR_ERR_CUDA);
    return;
  }
  pass_body<D>(ps.a[k], ps.b[k], ps.c[k], ps.o[k], ps.p[k], smem);
}

// ---------------------------------------------------------------------------
// The gains of the segments: sum_j u(j) b_j c_j^T, every factor reaching to the
// segment's end (its front, walking back).  The chunks of all kinds and heads are
// one list, of which every CTA takes an even share: a segment may be cut in two
// pieces, [0] from its front and [1], which are kept side by side (a share is
// never shorter than a segment).  A CTA takes 64 of b's columns: at d <= 128 two
// neighbours have one share and meet c's tiles in L2.
// Eight warps split b's rows in three parts while the tensor cores take the chunk
// before, c^T [hi | middle | low] in one product, and four warps add the sums of
// the one before that up in registers.
// ---------------------------------------------------------------------------
struct GainParams {
  DecayShape s;
  float* out[2];                      // [B H][segs][2][d][d]; `ends`: [B H][d][d]
  const float* first[2];
  bool ends;                          // one segment: what is left is the state behind it, from `first` (NULL: zeros)
  float s_u[2];
  bool rev[2];
  int chunks, per, unit;              // of a sequence, of a segment, of what a share is made of
  long long total;                    // entries of the list: [kind][head][chunk]
};
struct GainMaps {
  CUtensorMap b[2], c[2];
};
constexpr int kSplitWarps = 8, kTakeWarps = 4, kGainThreads = 32 * (kSplitWarps + kTakeWarps + 2);

// One CTA's share of the list as runs, each inside one segment.
struct Runs {
  const GainParams& p;
  long long x, x1;
  int kind, bh, b, h, seg, c0, c1, len;                    // the run's chunks [c0, c1) of its sequence
  __device__ __forceinline__ Runs(const GainParams& prm, long long from, long long to) : p(prm), x(from), x1(to) {
    const int row = (int)(from / p.chunks);                      // [kind][b][h]
    c1 = (int)(from - (long long)row * p.chunks);
    kind = row >= p.s.BH();
    bh = row - kind * p.s.BH();
    b = bh / p.s.H;
    h = bh - b * p.s.H;
    seg = c1 / p.per;
    len = x < x1 ? decay_length(p.s, b) : 0;
  }
  __device__ __forceinline__ bool next() {
    if (x >= x1) return false;
    if (c1 == p.chunks) {                                        // the next row's first segment
      c1 = seg = 0;
      ++bh;
      if (++h == p.s.H) {
        h = 0;
        if (++b == p.s.B) b = bh = 0, ++kind;
        len = decay_length(p.s, b);
      }
    } else if (c1 == (seg + 1) * p.per) {
      ++seg;
    }
    c0 = c1;
    c1 = (int)min((long long)min((seg + 1) * p.per, p.chunks), c0 + (x1 - x));
    x += c1 - c0;
    return true;
  }
  __device__ __forceinline__ int first() const { return seg * p.s.seg_tokens; }
  __device__ __forceinline__ int stop() const { return min(min(first() + p.s.seg_tokens, p.s.L), len); }
  // chunks of the run that have tokens
  __device__ __forceinline__ int live() const {
    return min(max((stop() - c0 * kM + kM - 1) / kM, 0), c1 - c0);
  }
};

template <int D>
__global__ void __launch_bounds__(kGainThreads, 1)
    decay_tc_gain_kernel(const __grid_constant__ GainMaps maps, const __grid_constant__ GainParams p) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t sm[];
  const DecayShape& s = p.s;
  // the passes may take their places and wait
  asm volatile("griddepcontrol.launch_dependents;");
  if (smem_addr(sm) % 1024 != 0) {
    if (threadIdx.x == 0) report_status(s.status, FAVOR_ERR_CUDA);
    return;
  }
  uint64_t *b_full = reinterpret_cast<uint64_t*>(sm + C::kGainBars), *c_full = b_full + 4;
  uint64_t *b_free = b_full + 8, *c_free = b_full + 12;                                              // of the places
  uint64_t *split = b_full + 16, *done = b_full + 18, *taken = b_full + 20, *end_bar = b_full + 22;  // [2] but the last
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(b_full + 23);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const WaitCtx wctx{abort_flag, s.status};
  const int half = D == 64 ? 0 : blockIdx.x & 1, share = D == 64 ? blockIdx.x : blockIdx.x >> 1;
  const int shares = D == 64 ? gridDim.x : gridDim.x >> 1;
  const long long units = p.total / p.unit;
  const long long x0 = units * share / shares * p.unit, x1 = units * (share + 1) / shares * p.unit;
  // lane = c's column; columns: b's 64 columns' three parts, twice
  constexpr uint32_t kCols = 512, kAcc = 192, kAccStep = 256;
  auto tile_b = [&](int j) { return sm + j % C::kDepthB * kAtom; };
  auto tile_c = [&](int j) { return sm + C::kTilesC + j % C::kDepthC * C::kTile; };
  auto parts = [&](int j) { return sm + C::kSplit + (j & 1) * 3 * kAtom; };

  if (threadIdx.x == 0) {
    for (int i = 0; i < 23; ++i) {
      const bool splits = (i >= 8 && i < 12) || i == 16 || i == 17;
      mbar_init(b_full + i, splits ? kSplitWarps : i == 20 || i == 21 ? kTakeWarps : 1);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  constexpr int kProducts = kSplitWarps + kTakeWarps;
  if (warp == kProducts) {
    tmem_alloc(tmem_slot, kCols);
    tmem_relinquish();
  } else if (threadIdx.x == 32 * (kProducts + 1)) {
    for (int k = 0; k < 2; ++k) {
      prefetch_tmap(&maps.b[k]);
      prefetch_tmap(&maps.c[k]);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == kProducts) {
    // ---- products
    if (lane == 0) {
      int n = 0;                                                 // chunks of the share
      for (Runs run(p, x0, x1); run.next();) n += run.live();
      bool ok = true, ready = false;
      constexpr uint32_t id = idesc_bf16(kM, kAcc, true, true);
      for (int j = 0; j < n; ++j) {
        uint64_t* const waits[3] = {c_full + j % C::kDepthC, split + (j & 1), taken + (j & 1)};
        ok = ready || (mbar_wait(waits[0], j / C::kDepthC & 1, wctx) && mbar_wait(waits[1], j >> 1 & 1, wctx) &&
                       (j < 2 || mbar_wait(waits[2], (j - 2) >> 1 & 1, wctx)));
        if (!ok) break;
        tc_fence_after();
        const uint64_t a0 = sdesc(smem_addr(tile_c(j)), D == 64 ? 0 : kAtom, 1024);
        const uint64_t b0 = sdesc(smem_addr(parts(j)), kAtom, 1024);
        const uint32_t acc = tmem + (j & 1) * kAccStep;
#pragma unroll
        for (int k = 0; k < kM / 16; ++k) {
          mma_bf16(acc, dadd(a0, kstep_mn(k)), dadd(b0, kstep_mn(k)), id, k > 0);
          // what the next chunk waits for is looked at while products are queued
          if (k == kM / 16 - 3 && j + 1 < n) {
            const int x = j + 1;
            ready = mbar_test_wait(smem_addr(c_full + x % C::kDepthC), x / C::kDepthC & 1) &&
                    mbar_test_wait(smem_addr(split + (x & 1)), x >> 1 & 1) &&
                    (x < 2 || mbar_test_wait(smem_addr(taken + (x & 1)), (x - 2) >> 1 & 1));
          }
        }
        mma_commit(done + (j & 1));
        mma_commit(c_free + j % C::kDepthC);
      }
      // what is in flight ends before its memory goes, even if the sums' warps have stopped waiting for it
      mma_commit(end_bar);
      drain(end_bar, 0);
    }
    __syncwarp();
  } else if (warp == kProducts + 1) {
    // ---- copies, kDepth chunks ahead
    if (lane == 0) {
      Runs run(p, x0, x1);
      bool ok = true;
      int j = 0, jc = 0;
      while (ok && run.next()) {
        const int live = run.live();
        for (int i = 0; i < live; ++i) {
          const int t0 = (run.c0 + i) * kM;
          // b's place is free once its rows are split, c's once the products have ended (barriers of the places: those
          // of the chunks' parity could run two phases ahead of this warp)
          const int nb = j / C::kDepthB, nc = jc / C::kDepthC;
          // (after a wait that ran out the rows' warps free it without having waited for what is on its way there)
          if (nb > 0 && !(ok = mbar_wait(b_free + j % C::kDepthB, (nb - 1) & 1, wctx) && !*abort_flag)) break;
          mbar_arrive_expect_tx(b_full + j % C::kDepthB, kAtom);
          tma_load_4d(tile_b(j), &maps.b[run.kind], half * 64, t0, run.h, run.b, b_full + j % C::kDepthB);
          ++j;
          if (nc > 0 && !(ok = mbar_wait(c_free + jc % C::kDepthC, (nc - 1) & 1, wctx))) break;
          mbar_arrive_expect_tx(c_full + jc % C::kDepthC, C::kTile);
#pragma unroll
          for (int a = 0; a < C::kAtoms; ++a)
            tma_load_4d(tile_c(jc) + a * kAtom, &maps.c[run.kind], a * 64, t0, run.h, run.b, c_full + jc % C::kDepthC);
          ++jc;
        }
      }
      // the last copies have landed, whoever still waits for them
      for (int k = 0; k < C::kDepthB && k < j; ++k) drain(b_full + k, (j - 1 - k) / C::kDepthB & 1);
      for (int k = 0; k < C::kDepthC && k < jc; ++k) drain(c_full + k, (jc - 1 - k) / C::kDepthC & 1);
    }
    __syncwarp();
  } else if (warp < kSplitWarps) {
    // ---- b's rows in three parts
    const int row = threadIdx.x & 127;
    Runs run(p, x0, x1);
    int j = 0, h = -1;                                           // chunks so far
    float g2 = 0.f;
    while (run.next()) {
      if (run.h != h) {
        h = run.h;
        g2 = s.g[h] * kLog2e;
      }
      const float s_u = p.s_u[run.kind];
      const bool rev = p.rev[run.kind];
      const int first = run.first(), stop = run.stop(), live = run.live();
      for (int i = 0; i < live; ++i, ++j) {
        const int t0 = (run.c0 + i) * kM, n = min(kM, stop - t0), at = t0 + row;
        const float u = row < n ? s_u * decay_power(g2, rev ? at - first + 1 : stop - 1 - at) : 0.f;
        mbar_wait(b_full + j % C::kDepthB, j / C::kDepthB & 1, wctx);
        if (j >= 2) mbar_wait(done + (j & 1), (j - 2) >> 1 & 1, wctx);         // the parts' place is read
        fade_rows3(tile_b(j), parts(j), row, threadIdx.x >> 7, u, row < n);
        if (n < kM && t0 + n < s.L) {
          mbar_wait(c_full + j % C::kDepthC, j / C::kDepthC & 1, wctx);
          clear_rows<D>(tile_c(j), n, threadIdx.x, 32 * kSplitWarps);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(split + (j & 1));
          mbar_arrive(b_free + j % C::kDepthB);
        }
      }
    }
  } else {
    // ---- the sums: lane = c's column y, N of b's columns from col on (at d <= 64 two lanes hold the same ones)
    const int q = warp & 3, t = 32 * q + lane, y = t & (D - 1), d = s.d;
    constexpr int N = D / 2;
    const int col = t / D * N;
    const uint32_t at = tmem + (static_cast<uint32_t>(32 * q) << 16) + col;
    float sum[N];
    Runs run(p, x0, x1);
    int j = 0;
    while (run.next()) {
      const int live = run.live();
#pragma unroll
      for (int e = 0; e < N; ++e) sum[e] = 0.f;
      for (int i = 0; i < live; ++i, ++j) {
        mbar_wait(done + (j & 1), j >> 1 & 1, wctx);
        __syncwarp();
        tc_fence_after();
#pragma unroll
        for (int n = 0; n < N; n += 8) {
          uint32_t v[3][8];
#pragma unroll
          for (int k = 0; k < 3; ++k) tmem_ld8(at + (j & 1) * kAccStep + k * 64 + n, v[k]);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 8; ++e)
            sum[n + e] += __uint_as_float(v[0][e]) + (__uint_as_float(v[1][e]) + __uint_as_float(v[2][e]));
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(taken + (j & 1));
      }
      const int64_t dd = (int64_t)d * d;
      if (p.ends) {
        // the pass beside may start from the state that this one takes the place of
        griddep_wait();
        const float all = decay_power(s.g[run.h] * kLog2e, min(run.stop(), run.len) - run.first());
        const int64_t to = run.bh * dd + (int64_t)(half * 64 + col) * d + y;
        const float* from = p.first[run.kind];
        const int left = y < d ? d - half * 64 - col : 0;
#pragma unroll
        for (int n = 0; n < N; n += 16) {                        // (`from` may be what is written: loads together first)
          float m[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) m[e] = from != nullptr && n + e < left ? from[to + (n + e) * d] : 0.f;
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (n + e < left) p.out[run.kind][to + (n + e) * d] = live > 0 ? fmaf(all, m[e], sum[n + e]) : m[e];
        }
      } else if (y < d) {
        const bool front = run.c0 == run.seg * p.per, whole = front && run.c1 == min((run.seg + 1) * p.per, p.chunks);
        float* out = p.out[run.kind] + (((int64_t)run.bh * s.segs + run.seg) * 2 + (front ? 0 : 1)) * dd +
                     (int64_t)(half * 64 + col) * d + y;
        const int left = d - half * 64 - col;
#pragma unroll
        for (int e = 0; e < N; ++e) {
          if (e < left) {
            out[e * d] = sum[e];
            if (whole) out[dd + e * d] = 0.f;
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kProducts) tmem_dealloc(tmem, kCols);
}

CUtensorMap map_of(const DecayMap& m) {
  CUtensorMap map;
  static_assert(sizeof(map) == sizeof(m.bytes), "map");
  memcpy(&map, m.bytes, sizeof(map));
  return map;
}

template <int D>
cudaError_t run_passes(const DecayTcPass* passes, int n, const DecayShape& s, cudaStream_t stream) {
  const auto kernel = decay_tc_pass_kernel<D>;
  const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), Cfg<D>::kSmem);
  if (e != cudaSuccess) return e;
  Passes ps{};
  for (int i = 0; i < n; ++i) {
    const DecayTcPass& a = passes[i];
    ps.a[i] = map_of(*a.a);
    ps.b[i] = map_of(*a.b);
    ps.c[i] = map_of(*a.c);
    ps.o[i] = map_of(*a.o);
    PassParams& p = ps.p[i];
    p.s = s;
    p.start = a.p.start;
    p.step = a.step;
    p.transposed = a.p.transposed;
    p.s_w = a.p.s_w;
    p.s_r = a.p.s_r;
    p.s_u = a.p.s_u;
    p.c = static_cast<const __nv_bfloat16*>(a.p.c);
    p.o = static_cast<__nv_bfloat16*>(a.p.o);
    p.cs = a.p.cs;
    p.os = a.p.os;
    p.rev = a.p.rev;
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(s.segs * s.BH()), (unsigned)n);
  cfg.blockDim = dim3(Cfg<D>::kThreads);
  cfg.dynamicSmemBytes = Cfg<D>::kSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = passes[0].after_scan ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, ps);
}

template <int D>
cudaError_t run_gains(const DecayTcGain* gains, int n, const DecayShape& s, cudaStream_t stream) {
  const auto kernel = decay_tc_gain_kernel<D>;
  const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), Cfg<D>::kGainSmem);
  if (e != cudaSuccess) return e;
  GainMaps maps{};
  GainParams p{};
  p.s = s;
  for (int i = 0; i < n; ++i) {
    maps.b[i] = map_of(*gains[i].b);
    maps.c[i] = map_of(*gains[i].c);
    p.out[i] = gains[i].p.out;
    p.s_u[i] = gains[i].p.s_u;
    p.rev[i] = gains[i].p.rev;
    p.first[i] = gains[i].first;
  }
  p.ends = gains[0].ends;
  p.chunks = (s.L + kM - 1) / kM;
  p.per = s.seg_tokens / kM;
  p.total = (long long)n * s.BH() * p.chunks;
  p.unit = p.ends ? p.chunks : 1;
  // shares that are no shorter than a segment
  constexpr int kHalves = D / 64;
  const int shares = (int)std::max<long long>(1, std::min<long long>(sm_count() / kHalves, p.total / p.per));
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(shares * kHalves));
  cfg.blockDim = dim3(kGainThreads);
  cfg.dynamicSmemBytes = Cfg<D>::kGainSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = p.ends ? 1 : 0;                                 // beside the passes
  return cudaLaunchKernelEx(&cfg, kernel, maps, p);
}

}  // namespace

bool decay_tc_takes(const View* const* views, int n, bool bf16, int d) {
  if (!bf16 || d > 128 || get_encode() == nullptr) return false;
  for (int i = 0; i < n; ++i) {
    const View& v = *views[i];
    if (!v.pieces(16)) return false;
    // strides of a map: above 0, below 2^40 bytes
    for (int k = 0; k < 3; ++k)
      if (v.n[k] > 1 && (v.s[k] <= 0 || v.s[k] >= int64_t(1) << 39)) return false;
  }
  return true;
}

void decay_tc_plan(DecayShape* s, int passes) {
  decay_segments(s, kM, (s->d <= 64 ? 2 : 1) * sm_count(), passes, kShort);
}

// [B, H, L, d] as a map {d, L, H, B}; box {64, 128, 1, 1}; 128-byte swizzle; what lies outside reads as 0
bool decay_tc_map(DecayMap* out, const View& v) {
  auto stride = [&](int k) { return static_cast<cuuint64_t>(v.n[k] > 1 ? v.s[k] : v.n[3]) * 2; };
  cuuint64_t dims[4] = {(cuuint64_t)v.n[3], (cuuint64_t)v.n[2], (cuuint64_t)v.n[1], (cuuint64_t)v.n[0]};
  cuuint64_t strides[3] = {stride(2), stride(1), stride(0)};
  cuuint32_t box[4] = {64, (cuuint32_t)kM, 1, 1};
  cuuint32_t ones[4] = {1, 1, 1, 1};
  CUtensorMap map;
  const CUresult r = get_encode()(&map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(v.p), dims, strides, box,
                                  ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return false;
  memcpy(out->bytes, &map, sizeof(map));
  return true;
}

bool decay_tc_ends_beside(const DecayShape& s) { return s.L <= kShort * kM; }

cudaError_t decay_tc_passes(const DecayTcPass* passes, int n, const DecayShape& s, cudaStream_t stream) {
  return s.d <= 64 ? run_passes<64>(passes, n, s, stream) : run_passes<128>(passes, n, s, stream);
}

cudaError_t decay_tc_gains(const DecayTcGain* gains, int n, const DecayShape& s, cudaStream_t stream) {
  return s.d <= 64 ? run_gains<64>(gains, n, s, stream) : run_gains<128>(gains, n, s, stream);
}

}  // namespace favor
