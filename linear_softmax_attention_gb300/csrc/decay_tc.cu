// Causal linear attention with a decay per head on the tensor cores: bf16, d <=
// 128 in whole 16-byte pieces (decay.cuh has the form that every pass follows).
//
// The gains of the segments come first, exact to fp32's sums: b's faded rows are
// kept as three bf16 parts (24 bits), c's rows as they are, and the products of
// every two chunks of 128 tokens are added up in registers (the tensor cores cut
// their sums off: 32 chunks in one accumulator were 4e-6 off, two are 1e-7).
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
// A warp of its own issues copies and products; the others share the work on
// registers, 32 columns of a quarter of the lanes each:
//   weights (P -> P')       while the gain's and I's products run before it,
//   b's faded rows          while O = P' C runs,
//   rows out (O, I -> o)    while the gain runs,
//   the state's copy, faded while the next chunk's P runs.
#include <string.h>

#include <algorithm>

#include "decay_tc.cuh"
#include "tc_util.cuh"

namespace favor {
namespace {

using namespace tc;

constexpr int kM = 128;              // tokens of a chunk

template <int D> struct Cfg {
  static constexpr int kParts = D / 32;                    // warps of a quarter of the lanes, 32 columns each
  static constexpr int kEpi = 128 * kParts, kEpiWarps = 4 * kParts;
  static constexpr int kThreads = kEpi + 32;
  static constexpr int kCtas = D == 64 ? 2 : 1;            // of an SM
  static constexpr int kAtoms = D / 64;                    // 128-byte columns of a tile
  static constexpr int kTile = kAtoms * kAtom;
  // the pass: a ring of tiles (two chunks at d <= 64) and the state's copy, [2 D rows: hi, rest][D]
  static constexpr int kSlots = D == 64 ? 6 : 5;
  static constexpr int kImg = kSlots * kTile;
  static constexpr int kImgAtom = 2 * D * 128;
  static constexpr int kBars = kImg + kAtoms * kImgAtom;
  static constexpr int kFade = kBars + 160;                // l^0 .. l^128
  static constexpr int kSmem = kFade + 132 * 4;
  // tensor memory: P (P' over its first half), O, I, M
  static constexpr uint32_t kCols = D == 64 ? 256 : 512;
  static constexpr uint32_t kP = 0, kO = D == 64 ? 64 : 128, kI = D == 64 ? 128 : 256, kState = D == 64 ? 192 : 384;
  // the gains: four tiles, and b's rows in three parts
  static constexpr int kGainSlots = 4;
  static constexpr int kParts3 = kGainSlots * kTile;
  static constexpr int kGainBars = kParts3 + 3 * kTile;
  static constexpr int kGainSmem = kGainBars + 128;
};
// an SM's 228 KB, 1 KB of it reserved for each CTA
static_assert(2 * (Cfg<64>::kSmem + 1024) <= 233472 && Cfg<128>::kSmem <= 232448, "shared memory");
static_assert(2 * (Cfg<64>::kGainSmem + 1024) <= 233472 && Cfg<128>::kGainSmem <= 232448, "shared memory");

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

// 32 columns of row `row` of a tile times u, rounded to bf16, in their place; 0 where !in
__device__ __forceinline__ void fade_rows(uint8_t* tile, int row, int part, float u, bool in) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int col = part * 32 + c * 8;
    uint4* at = reinterpret_cast<uint4*>(tile + (col >> 6) * kAtom + row * 128 +
                                         ((((col & 63) >> 3) ^ (row & 7)) << 4));
    uint4 w = in ? *at : make_uint4(0, 0, 0, 0);
    w.x = pack_bf16(bf_lo(w.x) * u, bf_hi(w.x) * u);
    w.y = pack_bf16(bf_lo(w.y) * u, bf_hi(w.y) * u);
    w.z = pack_bf16(bf_lo(w.z) * u, bf_hi(w.z) * u);
    w.w = pack_bf16(bf_lo(w.w) * u, bf_hi(w.w) * u);
    *at = w;
  }
}

// the same as three bf16 parts whose sum has all of fp32's bits
template <int TILE>
__device__ __forceinline__ void fade_rows3(const uint8_t* tile, uint8_t* parts, int row, int part, float u, bool in) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int col = part * 32 + c * 8;
    const int off = (col >> 6) * kAtom + row * 128 + ((((col & 63) >> 3) ^ (row & 7)) << 4);
    const uint4 raw = in ? *reinterpret_cast<const uint4*>(tile + off) : make_uint4(0, 0, 0, 0);
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    uint32_t h[3][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a = bf_lo(w[i]) * u, b = bf_hi(w[i]) * u;
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        h[k][i] = pack_bf16(a, b);
        if (k < 2) {
          a -= bf_lo(h[k][i]);
          b -= bf_hi(h[k][i]);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < 3; ++k)
      *reinterpret_cast<uint4*>(parts + k * TILE + off) = make_uint4(h[k][0], h[k][1], h[k][2], h[k][3]);
  }
}

// rows [n, 128) of a tile: 0 (what lies behind a sequence's end may be anything)
template <int D>
__device__ __forceinline__ void clear_rows(uint8_t* tile, int n, int tid) {
  for (int e = tid; e < (kM - n) * 8 * Cfg<D>::kAtoms; e += Cfg<D>::kEpi) {
    const int a = e / ((kM - n) * 8), r = e - a * (kM - n) * 8;
    *reinterpret_cast<uint4*>(tile + a * kAtom + n * 128 + r * 16) = make_uint4(0, 0, 0, 0);
  }
}

// acc (+)= b^T c over a chunk's 128 tokens, b's columns in atoms `lbo` apart (0: at d <= 64
// the upper half of the lanes repeats the lower one)
template <int D>
__device__ __forceinline__ void issue_gain(uint32_t acc, uint32_t b, uint32_t lbo, uint32_t c, bool add) {
  constexpr uint32_t id = idesc_bf16(kM, D, true, true);
  const uint64_t a0 = sdesc(b, lbo, 1024), b0 = sdesc(c, kAtom, 1024);
#pragma unroll
  for (int k = 0; k < kM / 16; ++k) mma_bf16(acc, dadd(a0, kstep_mn(k)), dadd(b0, kstep_mn(k)), id, add || k > 0);
}

// ---------------------------------------------------------------------------
// a pass
// ---------------------------------------------------------------------------
struct PassParams {
  DecayShape s;
  // What a segment starts from: `start` [B H][segs][d][d] where it is set; else
  // `edge` [B H][d][d] (NULL: zeros) taken through the gains of the segments
  // before it, [B H][segs][d][d]; `last`: what the last segment leaves.
  const float *start, *edge, *gains;
  float* last;
  bool transposed;                    // all of them hold M^T
  float s_w, s_r, s_u;
  const __nv_bfloat16* c;             // for rows with infinities or NaN
  __nv_bfloat16* o;                   // for rows behind a sequence's last chunk
  Strides cs, os;
};

// tokens of segment i of a sequence of len
__device__ __forceinline__ int seg_live(const DecayShape& s, int len, int i) {
  return min(max(len - i * s.seg_tokens, 0), s.seg_tokens);
}

template <int D, bool REV>
__device__ __forceinline__ void pass_body(const CUtensorMap& map_a, const CUtensorMap& map_b, const CUtensorMap& map_c,
                                          const CUtensorMap& map_o, const PassParams& p, uint8_t* sm) {
  using C = Cfg<D>;
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + C::kBars);          // [kSlots]
  uint64_t *scores = full + 6, *out_bar = full + 7, *gain_bar = full + 8, *again_bar = full + 9;
  uint64_t *weights_done = full + 10, *faded_done = full + 11, *rows_done = full + 12, *copy_done = full + 13;
  uint64_t* end_bar = full + 14;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(full + 15);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint32_t* odd_rows = tmem_slot + 2;                                   // [4] rows of c with infinities or NaN
  float* fade = reinterpret_cast<float*>(sm + C::kFade);

  const DecayShape& s = p.s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int bh = blockIdx.x / s.segs, seg = blockIdx.x - bh * s.segs, b = bh / s.H, h = bh - b * s.H;
  const float g2 = s.g[h] * kLog2E;
  const int len = decay_length(s, b), first = seg * s.seg_tokens, end = min(first + s.seg_tokens, s.L);
  const int stop = min(end, len);
  const int live = stop > first ? (stop - first + kM - 1) / kM : 0;     // chunks with tokens
  const WaitCtx wctx{abort_flag, s.status};
  // the i-th chunk in the pass's order
  auto token0 = [&](int i) { return first + (REV ? live - 1 - i : i) * kM; };
  auto tokens = [&](int i) { return min(kM, stop - token0(i)); };
  // its tiles: kind 0: b, 1: a, 2: c
  auto slot = [&](int i, int kind) { return sm + ((3 * i + kind) % C::kSlots) * C::kTile; };
  auto slot_full = [&](int i, int kind) { return full + (3 * i + kind) % C::kSlots; };
  auto slot_phase = [&](int i, int kind) { return ((3 * i + kind) / C::kSlots) & 1; };

  if (threadIdx.x == 0) {
    for (int i = 0; i < 10; ++i) mbar_init(full + i, 1);
    for (int i = 10; i < 14; ++i) mbar_init(full + i, C::kEpiWarps);
    mbar_init(end_bar, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == C::kEpiWarps) {
    tmem_alloc(tmem_slot, C::kCols);
    tmem_relinquish();
  }
  if (threadIdx.x <= kM) fade[threadIdx.x] = decay_power(g2, threadIdx.x);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == C::kEpiWarps) {
    // ---- copies and products
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
      for (int i = 0; i < live && ok; ++i) {
        const bool more = i + 1 < live;
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
        if (i > 0) {
          // the chunk before: b and c are read, and the rows leave from a's place
          ok = mbar_wait(gain_bar, (i - 1) & 1, wctx);
          if (!ok) break;
          if constexpr (C::kSlots == 6) {
            load(i + 1, 0);
            load(i + 1, 2);
          } else {
            load(i, 2);
            load(i + 1, 1);
          }
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
        if (i > 0) {
          bulk_wait_read0();
          load(i + 1, C::kSlots == 6 ? 1 : 0);
        }
        ok = mbar_wait(slot_full(i, 2), slot_phase(i, 2), wctx) && mbar_wait(weights_done, i & 1, wctx);
        if (!ok) break;
        tc_fence_after();
        const uint64_t c0 = sdesc(smem_addr(slot(i, 2)), kAtom, 1024);
#pragma unroll
        for (int k = 0; k < kM / 16; ++k)
          mma_bf16_ts(tmem + C::kO, tmem + C::kP + k * 8, dadd(c0, kstep_mn(k)), id, k > 0);
        mma_commit(out_bar);
        if (more) {
          ok = mbar_wait(faded_done, i & 1, wctx);
          if (!ok) break;
          tc_fence_after();
          issue_gain<D>(tmem + C::kState, smem_addr(slot(i, 0)), D == 64 ? 0 : kAtom, smem_addr(slot(i, 2)), true);
          mma_commit(gain_bar);
        }
        ok = mbar_wait(rows_done, i & 1, wctx);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int a = 0; a < C::kAtoms; ++a) tma_store_4d(&map_o, a * 64, token0(i), h, b, slot(i, 1) + a * kAtom);
        bulk_commit();
      }
      bulk_wait0();
      if (!ok) {
        // after a wait that ran out: what is in flight ends before its memory goes
        for (int x = 0; x < C::kSlots; ++x)
          if (issued >> x & 1) drain(full + x, phases >> x & 1);
        mma_commit(end_bar);
        drain(end_bar, 0);
      }
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
      for (int e = 0; e < 16; ++e) w[e] = pack_bf16(__uint_as_float(m[2 * e]), __uint_as_float(m[2 * e + 1]));
      const uint32_t img = smem_addr(sm + C::kImg);
      if (D == 128 || t < 64) store_row<16>(img, C::kImgAtom, x, part * 32, w);
      if (D == 128 || t >= 64) {
#pragma unroll
        for (int e = 0; e < 16; ++e)
          w[e] = pack_bf16(__uint_as_float(m[2 * e]) - bf_lo(w[e]), __uint_as_float(m[2 * e + 1]) - bf_hi(w[e]));
        store_row<16>(img, C::kImgAtom, D + x, part * 32, w);
      }
#pragma unroll
      for (int e = 0; e < 32; ++e) m[e] = __float_as_uint(__uint_as_float(m[e]) * all);
      tmem_st32(tmem + C::kState + lane_off + part * 32, m);
      tmem_st_wait();
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(copy_done);
    };

    // The state that the segment starts from, 16 bytes of it at a time with eight segments' gains in flight, through
    // the copy's place in shared memory ([D][D] fp32, 16-byte pieces of row x moved by x mod 8).
    {
      const int d = s.d, d4 = d / 4, pieces = d * d4;
      const int64_t dd = (int64_t)d * d;
      float4* state = reinterpret_cast<float4*>(sm + C::kImg);
      griddep_wait();                                                    // the gains (or states) are written
      const float4* from = reinterpret_cast<const float4*>(
          p.start != nullptr ? p.start + ((int64_t)bh * s.segs + seg) * dd : p.edge != nullptr ? p.edge + bh * dd : nullptr);
      const bool lasts = p.last != nullptr && seg == (REV ? 0 : s.segs - 1);
      const int before = p.start != nullptr ? 0 : REV ? s.segs - 1 - seg : seg;
      const float4* gains = reinterpret_cast<const float4*>(p.gains + (int64_t)bh * s.segs * dd);
      const float whole = decay_power(g2, s.seg_tokens);
      if (d < D) {                                                       // channels behind the d are 0
        for (int e = threadIdx.x; e < D * D / 4; e += C::kEpi) state[e] = make_float4(0.f, 0.f, 0.f, 0.f);
        named_bar(5, C::kEpi);
      }
      constexpr int kPlaces = 4, kAhead = 4;                             // loads in flight: their product
#pragma unroll 1
      for (int e0 = threadIdx.x; e0 < pieces; e0 += kPlaces * C::kEpi) {
        auto piece = [&](const float4* st, int k) {
          const int e = e0 + k * C::kEpi;
          return e < pieces ? st[e] : make_float4(0.f, 0.f, 0.f, 0.f);
        };
        auto then = [](float4 m, float all, float4 g) {
          return make_float4(fmaf(m.x, all, g.x), fmaf(m.y, all, g.y), fmaf(m.z, all, g.z), fmaf(m.w, all, g.w));
        };
        float4 m[kPlaces];
#pragma unroll
        for (int k = 0; k < kPlaces; ++k) m[k] = from != nullptr ? piece(from, k) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int j0 = 0; j0 < before; j0 += kAhead) {
          float4 gain[kAhead][kPlaces];
#pragma unroll
          for (int j = 0; j < kAhead; ++j)
            if (j0 + j < before)
#pragma unroll
              for (int k = 0; k < kPlaces; ++k)
                gain[j][k] = piece(gains + (REV ? s.segs - 1 - j0 - j : j0 + j) * (dd / 4), k);
#pragma unroll
          for (int j = 0; j < kAhead; ++j) {
            if (j0 + j >= before) break;
            const int n = seg_live(s, len, REV ? s.segs - 1 - j0 - j : j0 + j);
            if (n == 0) continue;
            const float all = n == s.seg_tokens ? whole : decay_power(g2, n);
#pragma unroll
            for (int k = 0; k < kPlaces; ++k) m[k] = then(m[k], all, gain[j][k]);
          }
        }
        const int n = seg_live(s, len, seg);
        const float all = decay_power(g2, n);
#pragma unroll
        for (int k = 0; k < kPlaces; ++k) {
          const int e = e0 + k * C::kEpi, row = e / d4, c = e - row * d4;
          if (e >= pieces) break;
          state[row * (D / 4) + (c ^ (row & 7))] = m[k];
          if (lasts)
            reinterpret_cast<float4*>(p.last + bh * dd)[e] = n > 0 ? then(m[k], all, gains[seg * (dd / 4) + e]) : m[k];
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
        clear_rows<D>(slot(i, 2), n, threadIdx.x);
        fence_proxy_async_smem();
      }
      mbar_wait(scores, i & 1, wctx);
      __syncwarp();
      tc_fence_after();
      {
        constexpr int G = 4 / C::kParts;                         // groups of 32 columns of a thread
        uint32_t w[G][16];
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const int grp = part * G + g, j0 = grp * 32;
          if (REV ? grp < q : grp > q) {
#pragma unroll
            for (int e = 0; e < 16; ++e) w[g][e] = 0u;
            continue;
          }
          uint32_t sc[32];
          tmem_ld32(tmem + C::kP + lane_off + j0, sc);
          tmem_ld_wait();
          if (grp != q && (!REV || n == kM)) {
            // whole groups of 16: l^(i - j) = l^(i - j0 - 15) l^(15 - k)
            float power[16];                                     // l^0 .. l^15
#pragma unroll
            for (int e = 0; e < 16; e += 4)
              *reinterpret_cast<float4*>(power + e) = *reinterpret_cast<const float4*>(fade + e);
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const int jh = j0 + 16 * hf;
              const float base = p.s_w * fade[REV ? jh - t : t - jh - 15];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float f0 = base * power[REV ? 2 * e : 15 - 2 * e];
                const float f1 = base * power[REV ? 2 * e + 1 : 14 - 2 * e];
                w[g][8 * hf + e] = pack_bf16(__uint_as_float(sc[16 * hf + 2 * e]) * f0,
                                             __uint_as_float(sc[16 * hf + 2 * e + 1]) * f1);
              }
            }
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float v[2];
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const int j = j0 + 2 * e + k, apart = REV ? j - t : t - j;
                const bool in = apart >= 0 && j < n;
                v[k] = in ? __uint_as_float(sc[2 * e + k]) * (p.s_w * fade[in ? apart : 0]) : 0.f;
              }
              w[g][e] = pack_bf16(v[0], v[1]);
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
        fade_rows(slot(i, 0), row, threadIdx.x >> 7, row < n ? p.s_u * fade[REV ? row + 1 : n - 1 - row] : 0.f, row < n);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(faded_done);
      }
      // ---- rows out, through a's place
      mbar_wait(out_bar, i & 1, wctx);
      __syncwarp();
      tc_fence_after();
      const float r = t < n ? p.s_r * fade[REV ? n - 1 - t : t + 1] : 0.f;
      auto rows_out = [&](bool patch) {
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
            const bool sees = REV ? j >= t : j <= t;
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const int y = part * 32 + e;
              const float v = y < s.d ? __bfloat162float(c[j * p.cs.l + y]) : 0.f;
              if (sees && v * 0.f != 0.f) o[e] = __float_as_uint(fmaf(w, v, __uint_as_float(o[e])));
            }
          }
        }
        float bad = 0.f;
#pragma unroll
        for (int e = 0; e < 32; ++e) bad = fmaf(__uint_as_float(o[e]), 0.f, bad);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float v0 = fmaf(__uint_as_float(in[2 * e]), r, __uint_as_float(o[2 * e]));
          const float v1 = fmaf(__uint_as_float(in[2 * e + 1]), r, __uint_as_float(o[2 * e + 1]));
          o[e] = t < n ? pack_bf16(v0, v1) : 0u;
        }
        store_row<16>(smem_addr(slot(i, 1)), kAtom, t, part * 32, o);
        return t < n && bad != 0.f;
      };
      // rare: a product with zero weights has met infinities or NaN of rows that must not be seen
      if (named_bar_or(5, C::kEpi, rows_out(false))) {
        uint8_t* ct = slot(i, 2);
        if (threadIdx.x < 4) odd_rows[threadIdx.x] = 0;
        // the gain has read c
        if (i + 1 < live) mbar_wait(gain_bar, i & 1, wctx);
        named_bar(5, C::kEpi);
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
        if (threadIdx.x == 0 && !*abort_flag) {
          tc_fence_after();
          constexpr uint32_t id = idesc_bf16(kM, D, false, true);
          const uint64_t c0 = sdesc(smem_addr(ct), kAtom, 1024);
#pragma unroll
          for (int k = 0; k < kM / 16; ++k)
            mma_bf16_ts(tmem + C::kO, tmem + C::kP + k * 8, dadd(c0, kstep_mn(k)), id, k > 0);
          mma_commit(again_bar);
        }
        __syncwarp();
        mbar_wait(again_bar, again & 1, wctx);
        ++again;
        __syncwarp();
        tc_fence_after();
        rows_out(true);
        named_bar(5, C::kEpi);                                   // odd_rows is read
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(rows_done);
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
    if (*abort_flag && threadIdx.x == 0 && again > 0) drain(again_bar, (again - 1) & 1);
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
  bool rev[3];
};

template <int D>
__global__ void __launch_bounds__(Cfg<D>::kThreads, Cfg<D>::kCtas)
    decay_tc_pass_kernel(const __grid_constant__ Passes ps) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const int k = blockIdx.y;
  if (smem_addr(smem) % 1024 != 0) {                             // tiles are read by 1024-byte swizzle blocks
    if (threadIdx.x == 0) report_status(ps.p[k].s.status, FAVOR_ERR_CUDA);
    return;
  }
  if (ps.rev[k]) pass_body<D, true>(ps.a[k], ps.b[k], ps.c[k], ps.o[k], ps.p[k], smem);
  else pass_body<D, false>(ps.a[k], ps.b[k], ps.c[k], ps.o[k], ps.p[k], smem);
}

// ---------------------------------------------------------------------------
// The gains of the segments: sum_j u(j) b_j c_j^T, every factor reaching to the
// segment's end (its front, walking back).
// ---------------------------------------------------------------------------
struct GainParams {
  DecayShape s;
  float* out[2];
  float s_u[2];
  bool rev[2];
};
struct GainMaps {
  CUtensorMap b[2], c[2];
};
// chunks in one accumulator (at d <= 128 it takes all three parts' products)
template <int D> constexpr int kGroup = D == 64 ? 2 : 1;

template <int D>
__global__ void __launch_bounds__(Cfg<D>::kEpi, Cfg<D>::kCtas)
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
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + C::kGainBars);
  uint64_t *full = bars, *done = bars + 4;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 5);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int kind = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q = warp & 3, part = warp >> 2, t = 32 * q + lane;
  const uint32_t lane_off = static_cast<uint32_t>(32 * q) << 16;
  const int bh = blockIdx.x / s.segs, seg = blockIdx.x - bh * s.segs, b = bh / s.H, h = bh - b * s.H;
  const float g2 = s.g[h] * kLog2E;
  const int first = seg * s.seg_tokens, stop = min(min(first + s.seg_tokens, s.L), decay_length(s, b));
  const int live = stop > first ? (stop - first + kM - 1) / kM : 0;
  const WaitCtx wctx{abort_flag, s.status};
  const CUtensorMap *map_b = &maps.b[kind], *map_c = &maps.c[kind];
  const bool rev = p.rev[kind];
  const float s_u = p.s_u[kind];
  auto slot = [&](int i, int k) { return sm + ((2 * i + k) % C::kGainSlots) * C::kTile; };
  auto slot_full = [&](int i, int k) { return full + (2 * i + k) % C::kGainSlots; };
  auto slot_phase = [&](int i, int k) { return ((2 * i + k) / C::kGainSlots) & 1; };
  constexpr uint32_t kCols = 128;                                // d <= 64: hi and middle parts' sums, the low parts'

  if (threadIdx.x == 0) {
    for (int i = 0; i < 5; ++i) mbar_init(bars + i, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0) {
    tmem_alloc(tmem_slot, kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const bool loader = threadIdx.x == 32, issuer = threadIdx.x == 0;
  int loads = 0, commits = 0;
  auto load = [&](int i, int k) {
    if (i >= live || *abort_flag) return;
    ++loads;
    uint64_t* bar = slot_full(i, k);
    mbar_arrive_expect_tx(bar, C::kTile);
#pragma unroll
    for (int a = 0; a < C::kAtoms; ++a)
      tma_load_4d(slot(i, k) + a * kAtom, k == 0 ? map_b : map_c, a * 64, first + i * kM, h, b, bar);
  };
  if (loader) {
    load(0, 0);
    load(0, 1);
    load(1, 0);
  }
  const int row = threadIdx.x & 127;
  float sum[32];
#pragma unroll
  for (int e = 0; e < 32; ++e) sum[e] = 0.f;
  auto take = [&] {
    uint32_t x[32];
    tmem_ld32(tmem + lane_off + part * 32, x);
    tmem_ld_wait();
#pragma unroll
    for (int e = 0; e < 32; ++e) sum[e] += __uint_as_float(x[e]);
    if constexpr (D == 64) {
      if (t < 64) {                                              // whole warps
        tmem_ld32(tmem + 64 + lane_off + part * 32, x);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 32; ++e) sum[e] += __uint_as_float(x[e]);
      }
    }
    tc_fence_before();
  };
  for (int i = 0; i < live; ++i) {
    const int t0 = first + i * kM, n = min(kM, stop - t0);
    const float u = row < n ? s_u * decay_power(g2, rev ? t0 + row - first + 1 : stop - 1 - t0 - row) : 0.f;
    mbar_wait(slot_full(i, 0), slot_phase(i, 0), wctx);
    if (i > 0) {
      mbar_wait(done, (i - 1) & 1, wctx);                        // the product before has read b's parts
      if (i % kGroup<D> == 0) {
        __syncwarp();
        tc_fence_after();
        take();
      }
    }
    fade_rows3<C::kTile>(slot(i, 0), sm + C::kParts3, row, threadIdx.x >> 7, u, row < n);
    if (n < kM && t0 + n < s.L) {
      mbar_wait(slot_full(i, 1), slot_phase(i, 1), wctx);
      clear_rows<D>(slot(i, 1), n, threadIdx.x);
    }
    fence_proxy_async_smem();
    __syncthreads();
    if (issuer) {
      const bool in = mbar_wait(slot_full(i, 1), slot_phase(i, 1), wctx);
      if (in && !*abort_flag) {
        tc_fence_after();
        const uint32_t parts = smem_addr(sm + C::kParts3), c = smem_addr(slot(i, 1));
        const bool add = i % kGroup<D> > 0;
        issue_gain<D>(tmem, parts, kAtom, c, add);
        if constexpr (D == 64) {
          issue_gain<D>(tmem + 64, parts + 2 * C::kTile, 0, c, add);
        } else {
          issue_gain<D>(tmem, parts + C::kTile, kAtom, c, true);
          issue_gain<D>(tmem, parts + 2 * C::kTile, kAtom, c, true);
        }
        mma_commit(done);
        ++commits;
      }
    }
    if (loader) {
      load(i + 1, 1);
      load(i + 2, 0);
    }
    __syncwarp();
  }
  if (live > 0) {
    mbar_wait(done, (live - 1) & 1, wctx);
    __syncwarp();
    tc_fence_after();
    take();
  }
  const int x = t & (D - 1);
  if constexpr (D == 64) {
    // the middle parts' sums join the others
    float* buf = reinterpret_cast<float*>(sm + C::kParts3);
    if (t >= 64)
#pragma unroll
      for (int e = 0; e < 32; ++e) buf[x * 65 + part * 32 + e] = sum[e];
    __syncthreads();
    if (t < 64)
#pragma unroll
      for (int e = 0; e < 32; ++e) sum[e] += buf[x * 65 + part * 32 + e];
  }
  if ((D == 128 || t < 64) && x < s.d) {
    float* out = p.out[kind] + (int64_t)blockIdx.x * s.d * s.d + x * s.d;
#pragma unroll
    for (int e = 0; e < 32; e += 4)                              // d is a multiple of 8
      if (part * 32 + e < s.d)
        *reinterpret_cast<float4*>(out + part * 32 + e) = make_float4(sum[e], sum[e + 1], sum[e + 2], sum[e + 3]);
  }
  if (loader)
    for (int k = max(0, loads - C::kGainSlots); k < loads; ++k) drain(full + k % C::kGainSlots, (k / C::kGainSlots) & 1);
  if (issuer && commits > 0) drain(done, (commits - 1) & 1);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, kCols);
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
    p.edge = a.edge;
    p.gains = a.gains;
    p.last = a.p.last;
    p.transposed = a.p.transposed;
    p.s_w = a.p.s_w;
    p.s_r = a.p.s_r;
    p.s_u = a.p.s_u;
    p.c = static_cast<const __nv_bfloat16*>(a.p.c);
    p.o = static_cast<__nv_bfloat16*>(a.p.o);
    p.cs = a.p.cs;
    p.os = a.p.os;
    ps.rev[i] = a.p.rev;
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
  cfg.numAttrs = passes[0].after_gains ? 1 : 0;
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
  }
  kernel<<<dim3(s.segs * s.BH(), n), Cfg<D>::kEpi, Cfg<D>::kGainSmem, stream>>>(maps, p);
  return cudaGetLastError();
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

void decay_tc_plan(DecayShape* s, int passes) { decay_segments(s, kM, (s->d <= 64 ? 2 : 1) * sm_count() / passes); }

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

cudaError_t decay_tc_passes(const DecayTcPass* passes, int n, const DecayShape& s, cudaStream_t stream) {
  return s.d <= 64 ? run_passes<64>(passes, n, s, stream) : run_passes<128>(passes, n, s, stream);
}

cudaError_t decay_tc_gains(const DecayTcGain* gains, int n, const DecayShape& s, cudaStream_t stream) {
  return s.d <= 64 ? run_gains<64>(gains, n, s, stream) : run_gains<128>(gains, n, s, stream);
}

}  // namespace favor
