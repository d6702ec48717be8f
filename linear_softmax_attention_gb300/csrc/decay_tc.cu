// Causal linear attention with a decay per head on the tensor cores: bf16, d <=
// 128 in whole 16-byte pieces (decay.cuh has the form that every pass follows).
//
// Chunks of 128 tokens.  P = A B^T and I = A M come first, M^T being a bf16 copy
// of the state; P is faded and masked on its way from tensor memory to
// registers and back, as the bf16 operand of O = P C, while the state takes in
// the chunk's gain.  Rows leave as O + r(i) I.
//  - The state stays in fp32 in tensor memory.  What it takes in is the product
//    of b's faded rows, kept as two bf16 parts (hi + lo: 16 bits of each), with c's
//    rows as they are, so that the states that are returned keep fp32's digits
//    but for 2^-16 of each term.  At d <= 64 the two parts' products stand in the
//    two halves of the lanes (one product of 128 rows), at d <= 128 they are added
//    to one accumulator.
//  - The decays never appear as l^-j: every factor is a power l^n, n >= 0.
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
  static constexpr int kThreads = 128 * kParts;
  static constexpr int kAtoms = D / 64;                    // 128-byte columns of a tile
  static constexpr int kTile = kAtoms * kAtom;
  static constexpr int kSlots = 4;
  static constexpr int kBp = kSlots * kTile;               // b's faded rows: hi tile, lo tile
  static constexpr int kImg = kBp + 2 * kTile;             // the state's copy, [x][y]
  static constexpr int kImgAtom = D * 128;
  static constexpr int kBars = kImg + kAtoms * kImgAtom;
  static constexpr int kFade = kBars + 128;                // l^0 .. l^128
  static constexpr int kSmem = kFade + 132 * 4 + 1024;
  // tensor memory: P (P' over its first half), O, I, M
  static constexpr uint32_t kCols = D == 64 ? 256 : 512;
  static constexpr uint32_t kP = 0, kO = D == 64 ? 64 : 128, kI = D == 64 ? 128 : 256, kState = D == 64 ? 192 : 384;
  static constexpr int kGainBars = kBp + 2 * kTile;
  static constexpr int kGainSmem = kGainBars + 128 + 1024;
};
static_assert(2 * (Cfg<64>::kSmem + 1024) <= 233472 && Cfg<128>::kSmem <= 232448, "shared memory");

// waits for a phase although other waits have run out: copies and products in
// flight must end before their memory goes
__device__ __forceinline__ void drain(uint64_t* bar, uint32_t parity) {
  const long long t0 = sm_cycles();
  while (!mbar_try_wait(smem_addr(bar), parity) && sm_cycles() - t0 <= kWaitLimitCycles) {
  }
}

// b's rows of a chunk, times u, as hi and lo parts; rows from n on are 0
template <int D>
__device__ __forceinline__ void fade_rows(const uint8_t* tile, uint8_t* hi, uint8_t* lo, int row, int part, float u,
                                          bool in) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int col = part * 32 + c * 8;
    const int off = (col >> 6) * kAtom + row * 128 + ((((col & 63) >> 3) ^ (row & 7)) << 4);
    const uint4 raw = *reinterpret_cast<const uint4*>(tile + off);
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    uint32_t h[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = in ? __uint_as_float(w[i] << 16) * u : 0.f;
      const float b = in ? __uint_as_float(w[i] & 0xffff0000u) * u : 0.f;
      h[i] = pack_bf16(a, b);
      l[i] = pack_bf16(a - __uint_as_float(h[i] << 16), b - __uint_as_float(h[i] & 0xffff0000u));
    }
    *reinterpret_cast<uint4*>(hi + off) = make_uint4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<uint4*>(lo + off) = make_uint4(l[0], l[1], l[2], l[3]);
  }
}

// rows [n, 128) of a tile: 0 (what lies behind a sequence's end may be anything)
template <int D>
__device__ __forceinline__ void clear_rows(uint8_t* tile, int n) {
  for (int e = threadIdx.x; e < (kM - n) * 8 * Cfg<D>::kAtoms; e += Cfg<D>::kThreads) {
    const int a = e / ((kM - n) * 8), r = e - a * (kM - n) * 8;
    *reinterpret_cast<uint4*>(tile + a * kAtom + n * 128 + r * 16) = make_uint4(0, 0, 0, 0);
  }
}

// M += [hi | lo]^T C over the chunk's 128 tokens
template <int D>
__device__ __forceinline__ void issue_gain(uint32_t state, uint32_t bp, uint32_t c, bool add) {
  constexpr uint32_t id = idesc_bf16(kM, D, true, true);
  const uint64_t b0 = sdesc(c, kAtom, 1024);
  const uint64_t a0 = sdesc(bp, kAtom, 1024);
#pragma unroll
  for (int k = 0; k < kM / 16; ++k) mma_bf16(state, dadd(a0, kstep_mn(k)), dadd(b0, kstep_mn(k)), id, add || k > 0);
  if constexpr (D == 128) {
    const uint64_t a1 = sdesc(bp + Cfg<D>::kTile, kAtom, 1024);
#pragma unroll
    for (int k = 0; k < kM / 16; ++k) mma_bf16(state, dadd(a1, kstep_mn(k)), dadd(b0, kstep_mn(k)), id, true);
  }
}

// The state in tensor memory to [d][d] in global memory (its transpose where
// asked), hi and lo parts added; `buf`: 64 x 65 floats at d <= 64.
template <int D>
__device__ __forceinline__ void store_state(uint32_t tmem_state, float* buf, float* out, int d, bool transposed, int t,
                                            int part, uint32_t lane_off) {
  uint32_t x[32];
  tmem_ld32(tmem_state + lane_off + part * 32, x);
  tmem_ld_wait();
  if constexpr (D == 64) {
    if (t >= 64)
#pragma unroll
      for (int i = 0; i < 32; ++i) buf[(t - 64) * 65 + part * 32 + i] = __uint_as_float(x[i]);
    __syncthreads();
    if (t < 64)
#pragma unroll
      for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) + buf[t * 65 + part * 32 + i]);
  }
  if (t < d)
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const int y = part * 32 + i;
      if (y < d) out[transposed ? y * d + t : t * d + y] = __uint_as_float(x[i]);
    }
}

struct PassParams {
  DecayShape s;
  const float* start;
  float* last;
  bool transposed;
  float s_w, s_r, s_u;
  const __nv_bfloat16* c;             // for rows with infinities or NaN
  __nv_bfloat16* o;                   // for rows behind a sequence's last chunk
  Strides cs, os;
};

template <int D, bool REV>
__global__ void __launch_bounds__(Cfg<D>::kThreads, D == 64 ? 2 : 1)
    decay_tc_pass_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                         const __grid_constant__ CUtensorMap map_c, const __grid_constant__ CUtensorMap map_o,
                         const __grid_constant__ PassParams p) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + C::kBars);
  uint64_t *full = bars, *scores_bar = bars + 4, *out_bar = bars + 5, *again_bar = bars + 6;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 7);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* odd = reinterpret_cast<int*>(tmem_slot + 2);            // [chunk parity] infinities or NaN among the outputs
  uint32_t* odd_rows = tmem_slot + 4;                          // [4] rows of c with infinities or NaN
  float* fade = reinterpret_cast<float*>(sm + C::kFade);

  const DecayShape& s = p.s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q = warp & 3, part = warp >> 2, t = 32 * q + lane;  // this thread's lane of tensor memory (row), columns
  const uint32_t lane_off = static_cast<uint32_t>(32 * q) << 16;
  const int bh = blockIdx.x / s.segs, seg = blockIdx.x - bh * s.segs, b = bh / s.H, h = bh - b * s.H;
  const float g2 = s.g[h] * kLog2E;
  const int len = decay_length(s, b), first = seg * s.seg_tokens, end = min(first + s.seg_tokens, s.L);
  const int stop = min(end, len);
  const int live = stop > first ? (stop - first + kM - 1) / kM : 0;     // chunks with tokens
  const int chunks = (end - first + kM - 1) / kM;                        // chunks with rows
  const WaitCtx wctx{abort_flag, s.status};
  // the i-th chunk in the pass's order, of the live ones
  auto token0 = [&](int i) { return first + (REV ? live - 1 - i : i) * kM; };
  auto tokens = [&](int i) { return min(kM, stop - token0(i)); };
  auto slot = [&](int i, int kind) { return sm + ((3 * i + kind) % C::kSlots) * C::kTile; };
  auto slot_full = [&](int i, int kind) { return full + (3 * i + kind) % C::kSlots; };
  auto slot_phase = [&](int i, int kind) { return ((3 * i + kind) / C::kSlots) & 1; };

  if (threadIdx.x == 0) {
    for (int i = 0; i < 7; ++i) mbar_init(bars + i, 1);
    *abort_flag = 0;
    odd[0] = odd[1] = 0;
    fence_barrier_init();
  }
  if (warp == 0) {
    tmem_alloc(tmem_slot, C::kCols);
    tmem_relinquish();
  }
  if (threadIdx.x <= kM) fade[threadIdx.x] = decay_power(g2, threadIdx.x);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // copies of the pass's tiles: kind 0: b, 1: a, 2: c
  const bool loader = threadIdx.x == 32, issuer = threadIdx.x == 0;
  int loads = 0;                                                // the loader's
  auto load = [&](int i, int kind) {
    if (i >= live || *abort_flag) return;
    ++loads;
    const CUtensorMap* map = kind == 0 ? &map_b : kind == 1 ? &map_a : &map_c;
    uint64_t* bar = slot_full(i, kind);
    mbar_arrive_expect_tx(bar, C::kTile);
#pragma unroll
    for (int a = 0; a < C::kAtoms; ++a) tma_load_4d(slot(i, kind) + a * kAtom, map, a * 64, token0(i), h, b, bar);
  };
  if (loader) {
    load(0, 0);
    load(0, 1);
    load(0, 2);
    load(1, 0);
  }
  // the state that the segment starts from (hi lanes; the lo lanes start from 0)
  {
    uint32_t x[32];
    const float* start = p.start == nullptr ? nullptr : p.start + ((int64_t)bh * s.segs + seg) * s.d * s.d;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const int y = part * 32 + i;
      float v = 0.f;
      if (start != nullptr && t < s.d && y < s.d) v = start[p.transposed ? y * s.d + t : t * s.d + y];
      x[i] = __float_as_uint(v);
    }
    tmem_st32(tmem + C::kState + lane_off + part * 32, x);
    tmem_st_wait();
  }
  int again = 0;
  for (int i = 0; i <= live; ++i) {
    // ---- rows of the chunk before; this chunk's copy of the state
    if (i > 0) {
      mbar_wait(out_bar, (i - 1) & 1, wctx);
      __syncwarp();
      tc_fence_after();
      const int n = tokens(i - 1);
      const float r = t < n ? p.s_r * fade[REV ? n - 1 - t : t + 1] : 0.f;
      auto rows_out = [&](bool patch) {
        uint32_t o[32], in[32];
        tmem_ld32(tmem + C::kO + lane_off + part * 32, o);
        tmem_ld32(tmem + C::kI + lane_off + part * 32, in);
        tmem_ld_wait();
        if (patch) {
          // what the infinities and NaN of c's rows, left out of the product, add to the rows that see them
          const __nv_bfloat16* c = p.c + b * p.cs.b + h * p.cs.h + (int64_t)token0(i - 1) * p.cs.l;
          for (int j = 0; j < n; ++j) {
            if (!(odd_rows[j >> 5] >> (j & 31) & 1)) continue;
            const uint32_t pair = tmem_ld1(tmem + C::kP + lane_off + (j >> 1));
            tmem_ld_wait();
            const float w = __uint_as_float(j & 1 ? pair & 0xffff0000u : pair << 16);
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
        if (!patch && t < n && bad != 0.f) odd[(i - 1) & 1] = 1;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float v0 = fmaf(__uint_as_float(in[2 * e]), r, __uint_as_float(o[2 * e]));
          const float v1 = fmaf(__uint_as_float(in[2 * e + 1]), r, __uint_as_float(o[2 * e + 1]));
          o[e] = t < n ? pack_bf16(v0, v1) : 0u;
        }
        store_row<16>(smem_addr(slot(i - 1, 1)), kAtom, t, part * 32, o);
      };
      rows_out(false);
      // rare: a product with zero weights has met infinities or NaN of rows that must not be seen
      tc_fence_before();
      fence_proxy_async_smem();
      __syncthreads();
      tc_fence_after();
      if (odd[(i - 1) & 1] != 0) {
        uint8_t* ct = slot(i - 1, 2);
        if (threadIdx.x < 4) odd_rows[threadIdx.x] = 0;
        __syncthreads();
        for (int e = threadIdx.x; e < C::kTile / 16; e += C::kThreads) {
          uint4 raw = *reinterpret_cast<const uint4*>(ct + e * 16);
          uint32_t* w = reinterpret_cast<uint32_t*>(&raw);
          bool found = false;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if ((w[k] & 0x7f80u) == 0x7f80u) {
              w[k] &= 0xffff0000u;
              found = true;
            }
            if ((w[k] & 0x7f800000u) == 0x7f800000u) {
              w[k] &= 0xffffu;
              found = true;
            }
          }
          if (found) {
            const int row = (e * 16 % kAtom) / 128;
            *reinterpret_cast<uint4*>(ct + e * 16) = raw;
            atomicOr(&odd_rows[row >> 5], 1u << (row & 31));
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        if (issuer && !*abort_flag) {
          constexpr uint32_t id = idesc_bf16(kM, D, false, true);
          const uint64_t b0 = sdesc(smem_addr(ct), kAtom, 1024);
#pragma unroll
          for (int k = 0; k < kM / 16; ++k)
            mma_bf16_ts(tmem + C::kO, tmem + C::kP + k * 8, dadd(b0, kstep_mn(k)), id, k > 0);
          mma_commit(again_bar);
        }
        __syncwarp();
        mbar_wait(again_bar, again & 1, wctx);
        ++again;
        __syncwarp();
        tc_fence_after();
        rows_out(true);
        fence_proxy_async_smem();
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        if (threadIdx.x == 0) odd[(i - 1) & 1] = 0;
      }
      if (loader && !*abort_flag) {
#pragma unroll
        for (int a = 0; a < C::kAtoms; ++a)
          tma_store_4d(&map_o, a * 64, token0(i - 1), h, b, slot(i - 1, 1) + a * kAtom);
        bulk_commit();
        load(i + 1, 0);                              // where c was
      }
      __syncwarp();
    }
    if (i == live) break;
    if (issuer) {
      bool in = mbar_wait(slot_full(i, 0), slot_phase(i, 0), wctx);
      in = mbar_wait(slot_full(i, 1), slot_phase(i, 1), wctx) && in;
      if (in && !*abort_flag) {
        constexpr uint32_t id = idesc_bf16(kM, kM, false, false);
        const uint64_t a0 = sdesc(smem_addr(slot(i, 1)), 16, 1024), b0 = sdesc(smem_addr(slot(i, 0)), 16, 1024);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          mma_bf16(tmem + C::kP, dadd(a0, kstep_k(k, kAtom)), dadd(b0, kstep_k(k, kAtom)), id, k > 0);
        mma_commit(scores_bar);
      }
    }
    __syncwarp();
    const int n = tokens(i);
    const bool more = i + 1 < live || p.last != nullptr;
    // ---- the state's bf16 copy; the state itself fades over the chunk
    {
      uint32_t x[32];
      tmem_ld32(tmem + C::kState + lane_off + part * 32, x);
      tmem_ld_wait();
      if (D == 128 || t < 64) {
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) w[e] = pack_bf16(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1]));
        store_row<16>(smem_addr(sm + C::kImg), C::kImgAtom, t, part * 32, w);
      }
      if (more) {
        const float all = fade[n];
#pragma unroll
        for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * all);
        tmem_st32(tmem + C::kState + lane_off + part * 32, x);
        tmem_st_wait();
      }
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (issuer && !*abort_flag) {
      constexpr uint32_t id = idesc_bf16(kM, D, false, true);
      const uint64_t a0 = sdesc(smem_addr(slot(i, 1)), 16, 1024);
      const uint64_t m0 = sdesc(smem_addr(sm + C::kImg), C::kImgAtom, 1024);
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
        mma_bf16(tmem + C::kI, dadd(a0, kstep_k(k, kAtom)), dadd(m0, kstep_mn(k)), id, k > 0);
    }
    if (loader && i > 0) {
      bulk_wait_read0();
      load(i, 2);                                    // where the rows were
    }
    __syncwarp();
    // ---- b's faded rows for the gain
    mbar_wait(slot_full(i, 0), slot_phase(i, 0), wctx);
    if (more) {
      const int row = threadIdx.x & 127;
      fade_rows<D>(slot(i, 0), sm + C::kBp, sm + C::kBp + C::kTile, row, threadIdx.x >> 7,
                   row < n ? p.s_u * fade[REV ? row + 1 : n - 1 - row] : 0.f, row < n);
    }
    if (n < kM && token0(i) + n < s.L) {
      mbar_wait(slot_full(i, 2), slot_phase(i, 2), wctx);
      clear_rows<D>(slot(i, 2), n);
    }
    fence_proxy_async_smem();
    // ---- the weights: faded, masked, rounded to bf16 (each is one term's factor)
    mbar_wait(scores_bar, i & 1, wctx);
    __syncwarp();
    tc_fence_after();
    {
      constexpr int G = 4 / C::kParts;                           // groups of 32 columns of a thread
      float power[16];                                           // l^0 .. l^15
#pragma unroll
      for (int e = 0; e < 16; e += 4) *reinterpret_cast<float4*>(power + e) = *reinterpret_cast<const float4*>(fade + e);
      uint32_t w[G][16];
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const int grp = part * G + g, j0 = grp * 32;
        if (REV ? grp < q : grp > q) {
#pragma unroll
          for (int e = 0; e < 16; ++e) w[g][e] = 0u;
          continue;
        }
        uint32_t x[32];
        tmem_ld32(tmem + C::kP + lane_off + j0, x);
        tmem_ld_wait();
        if (grp != q && (!REV || n == kM)) {
          // whole groups of 16: l^(i - j) = l^(i - j0 - 15) l^(15 - k)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const int jh = j0 + 16 * hf;
            const float base = p.s_w * fade[REV ? jh - t : t - jh - 15];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float f0 = base * power[REV ? 2 * e : 15 - 2 * e], f1 = base * power[REV ? 2 * e + 1 : 14 - 2 * e];
              w[g][8 * hf + e] = pack_bf16(__uint_as_float(x[16 * hf + 2 * e]) * f0,
                                           __uint_as_float(x[16 * hf + 2 * e + 1]) * f1);
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
              v[k] = in ? __uint_as_float(x[2 * e + k]) * (p.s_w * fade[in ? apart : 0]) : 0.f;
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
    __syncthreads();
    tc_fence_after();
    if (issuer) {
      const bool in = mbar_wait(slot_full(i, 2), slot_phase(i, 2), wctx);
      if (in && !*abort_flag) {
        constexpr uint32_t id = idesc_bf16(kM, D, false, true);
        const uint64_t c0 = sdesc(smem_addr(slot(i, 2)), kAtom, 1024);
#pragma unroll
        for (int k = 0; k < kM / 16; ++k)
          mma_bf16_ts(tmem + C::kO, tmem + C::kP + k * 8, dadd(c0, kstep_mn(k)), id, k > 0);
        if (more) issue_gain<D>(tmem + C::kState, smem_addr(sm + C::kBp), smem_addr(slot(i, 2)), true);
        mma_commit(out_bar);
      }
    }
    if (loader) load(i + 1, 1);                      // where b was
    __syncwarp();
  }
  // rows of chunks behind the sequence's end
  if (live < chunks) {
    __nv_bfloat16* o = p.o + b * p.os.b + h * p.os.h;
    const int from = max(first + live * kM, first), d8 = s.d / 8;
    for (int64_t e = threadIdx.x; e < (int64_t)(end - from) * d8; e += C::kThreads) {
      const int r = (int)(e / d8), c = (int)(e - (int64_t)r * d8) * 8;
      *reinterpret_cast<uint4*>(o + (int64_t)(from + r) * p.os.l + c) = make_uint4(0, 0, 0, 0);
    }
  }
  if (p.last != nullptr) {
    store_state<D>(tmem + C::kState, reinterpret_cast<float*>(sm + C::kBp), p.last + (int64_t)bh * s.d * s.d, s.d,
                   p.transposed, t, part, lane_off);
  }
  // after a wait that ran out: what is in flight ends before its memory goes
  if (loader) {
    bulk_wait0();
    for (int x = max(0, loads - C::kSlots); x < loads; ++x) drain(full + x % C::kSlots, (x / C::kSlots) & 1);
  }
  if (issuer && *abort_flag) {
    mma_commit(again_bar);
    drain(again_bar, again & 1);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, C::kCols);
}

// ---------------------------------------------------------------------------
// The gains of the segments: sum_j u(j) b_j c_j^T, every factor reaching to the
// segment's end (its front, walking back), so that the accumulator is only
// added to.
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

template <int D>
__global__ void __launch_bounds__(Cfg<D>::kThreads, D == 64 ? 2 : 1)
    decay_tc_gain_kernel(const __grid_constant__ GainMaps maps, const __grid_constant__ GainParams p) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + C::kGainBars);
  uint64_t *full = bars, *done = bars + 4;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 5);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const DecayShape& s = p.s;
  const int kind = blockIdx.z;
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
  auto slot = [&](int i, int k) { return sm + ((2 * i + k) % C::kSlots) * C::kTile; };
  auto slot_full = [&](int i, int k) { return full + (2 * i + k) % C::kSlots; };
  auto slot_phase = [&](int i, int k) { return ((2 * i + k) / C::kSlots) & 1; };
  constexpr uint32_t kCols = D == 64 ? 64 : 128;

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
  for (int i = 0; i < live; ++i) {
    const int t0 = first + i * kM, n = min(kM, stop - t0);
    const float u = row < n ? s_u * decay_power(g2, rev ? t0 + row - first + 1 : stop - 1 - t0 - row) : 0.f;
    mbar_wait(slot_full(i, 0), slot_phase(i, 0), wctx);
    if (i > 0) mbar_wait(done, (i - 1) & 1, wctx);          // the product before has read b's faded rows
    fade_rows<D>(slot(i, 0), sm + C::kBp, sm + C::kBp + C::kTile, row, threadIdx.x >> 7, u, row < n);
    if (n < kM && t0 + n < s.L) {
      mbar_wait(slot_full(i, 1), slot_phase(i, 1), wctx);
      clear_rows<D>(slot(i, 1), n);
    }
    fence_proxy_async_smem();
    __syncthreads();
    if (issuer) {
      const bool in = mbar_wait(slot_full(i, 1), slot_phase(i, 1), wctx);
      if (in && !*abort_flag) {
        tc_fence_after();
        issue_gain<D>(tmem, smem_addr(sm + C::kBp), smem_addr(slot(i, 1)), i > 0);
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
  float* out = p.out[kind] + (int64_t)blockIdx.x * s.d * s.d;
  if (live > 0) {
    mbar_wait(done, (live - 1) & 1, wctx);
    __syncwarp();
    tc_fence_after();
    store_state<D>(tmem, reinterpret_cast<float*>(sm + C::kBp), out, s.d, false, t, part, lane_off);
  } else {
    for (int e = threadIdx.x; e < s.d * s.d; e += C::kThreads) out[e] = 0.f;
  }
  if (loader)
    for (int x = max(0, loads - C::kSlots); x < loads; ++x) drain(full + x % C::kSlots, (x / C::kSlots) & 1);
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

template <int D, bool REV>
cudaError_t run_pass(const DecayTcPass& a, const DecayShape& s, cudaStream_t stream) {
  const auto kernel = decay_tc_pass_kernel<D, REV>;
  const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), Cfg<D>::kSmem);
  if (e != cudaSuccess) return e;
  PassParams p{};
  p.s = s;
  p.start = a.p.start;
  p.last = a.p.last;
  p.transposed = a.p.transposed;
  p.s_w = a.p.s_w;
  p.s_r = a.p.s_r;
  p.s_u = a.p.s_u;
  p.c = static_cast<const __nv_bfloat16*>(a.p.c);
  p.o = static_cast<__nv_bfloat16*>(a.p.o);
  p.cs = a.p.cs;
  p.os = a.p.os;
  kernel<<<s.segs * s.BH(), Cfg<D>::kThreads, Cfg<D>::kSmem, stream>>>(map_of(*a.a), map_of(*a.b), map_of(*a.c),
                                                                       map_of(*a.o), p);
  return cudaGetLastError();
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
  kernel<<<dim3(s.segs * s.BH(), 1, n), Cfg<D>::kThreads, Cfg<D>::kGainSmem, stream>>>(maps, p);
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

void decay_tc_plan(DecayShape* s) { decay_segments(s, kM, (s->d <= 64 ? 2 : 1) * sm_count()); }

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

cudaError_t decay_tc_pass(const DecayTcPass& p, const DecayShape& s, cudaStream_t stream) {
  if (s.d <= 64) return p.p.rev ? run_pass<64, true>(p, s, stream) : run_pass<64, false>(p, s, stream);
  return p.p.rev ? run_pass<128, true>(p, s, stream) : run_pass<128, false>(p, s, stream);
}

cudaError_t decay_tc_gains(const DecayTcGain* gains, int n, const DecayShape& s, cudaStream_t stream) {
  return s.d <= 64 ? run_gains<64>(gains, n, s, stream) : run_gains<128>(gains, n, s, stream);
}

}  // namespace favor
