// C ABI entry points of the sequence operators: argument checks and dispatch.
#include <algorithm>
#include <cmath>
#include <initializer_list>

#include "decay_tc.cuh"
#include "favor_selftest.h"
#include "ops.cuh"

namespace favor {

bool make_view(View* v, const void* p, const int64_t* strides, int B, int H, int L, int d, int esz) {
  if (p == nullptr || reinterpret_cast<uintptr_t>(p) % esz != 0) return false;
  v->p = p;
  v->esz = esz;
  const int64_t n[4] = {B, H, L, d};
  for (int i = 0; i < 4; ++i) v->n[i] = n[i];
  int64_t packed = d;
  for (int i = 2; i >= 0; --i) {
    const int64_t s = strides != nullptr ? strides[i] : packed;
    // the largest offset stays far inside 64 bits
    if (n[i] > 1 && (s < 0 || s > (int64_t(1) << 56) / n[i])) return false;
    v->s[i] = n[i] > 1 ? s : 0;
    if (strides == nullptr) {
      if (packed > (int64_t(1) << 56) / n[i]) return false;
      packed *= n[i];
    }
  }
  return true;
}

View flat_view(const void* p, int64_t n, int esz) { return View{p, esz, {1, 1, 1, n}, {0, 0, 0}}; }

namespace {

// axes of the first three with more than one element, largest stride first
int by_stride(const View& v, int order[3]) {
  int k = 0;
  for (int i = 0; i < 3; ++i)
    if (v.n[i] > 1) order[k++] = i;
  std::sort(order, order + k, [&](int a, int b) { return v.s[a] > v.s[b]; });
  return k;
}

int64_t reach(const View& v) {   // elements from the first to behind the last
  int64_t r = v.n[3];
  for (int i = 0; i < 3; ++i) r += (v.n[i] - 1) * v.s[i];
  return r;
}

// Does delta = sum_i s_i k_i + k_d have a solution with -(nb_i - 1) <= k_i <=
// na_i - 1?  Axes from order[i] on, strides falling.
bool hits(const View& a, const View& b, const int* order, int left, int64_t delta) {
  if (left == 0) return delta > -b.n[3] && delta < a.n[3];
  int64_t lo = -(b.n[3] - 1), hi = a.n[3] - 1;        // what the inner axes reach
  for (int i = 1; i < left; ++i) {
    lo -= (b.n[order[i]] - 1) * a.s[order[i]];
    hi += (a.n[order[i]] - 1) * a.s[order[i]];
  }
  const int ax = *order;
  const int64_t s = a.s[ax];
  if (s == 0) return hits(a, b, order + 1, left - 1, delta);
  auto floor_div = [](int64_t x, int64_t y) { return x / y - (x % y != 0 && (x < 0) != (y < 0)); };
  const int64_t k0 = std::max(-floor_div(hi - delta, s), -(b.n[ax] - 1));
  const int64_t k1 = std::min(floor_div(delta - lo, s), a.n[ax] - 1);
  if (k1 - k0 > 3) return true;                       // strides that do not nest: taken as an overlap
  for (int64_t k = k0; k <= k1; ++k)
    if (hits(a, b, order + 1, left - 1, delta - k * s)) return true;
  return false;
}

}  // namespace

bool self_overlap(const View& v) {
  int order[3];
  const int k = by_stride(v, order);
  int64_t inner = v.n[3];
  for (int i = k - 1; i >= 0; --i) {
    if (v.s[order[i]] < inner) return true;
    inner += (v.n[order[i]] - 1) * v.s[order[i]];
  }
  return false;
}

bool same_view(const View& a, const View& b) {
  if (a.p != b.p || a.esz != b.esz) return false;
  for (int i = 0; i < 4; ++i)
    if (a.n[i] != b.n[i]) return false;
  for (int i = 0; i < 3; ++i)
    if (a.s[i] != b.s[i]) return false;
  return true;
}

bool overlap(const View& a, const View& b) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  const uintptr_t a1 = a0 + (uintptr_t)reach(a) * a.esz, b1 = b0 + (uintptr_t)reach(b) * b.esz;
  if (a1 <= b0 || b1 <= a0) return false;
  if (a.esz != b.esz) return true;
  View x = a, y = b;
  int order[3], k = 0;
  for (int i = 0; i < 3; ++i) {
    if (a.n[i] == 1 && b.n[i] == 1) continue;
    if (a.n[i] > 1 && b.n[i] > 1 && a.s[i] != b.s[i]) return true;
    x.s[i] = y.s[i] = a.n[i] > 1 ? a.s[i] : b.s[i];
    order[k++] = i;
  }
  std::sort(order, order + k, [&](int i, int j) { return x.s[i] > x.s[j]; });
  const int64_t bytes = static_cast<int64_t>(b0) - static_cast<int64_t>(a0);
  if (bytes % a.esz != 0) return true;
  return hits(x, y, order, k, bytes / a.esz);
}

Rows make_rows(int B, int H, int L, const Strides* s, int n) {
  Rows r{};
  for (int i = 0; i < n; ++i) r.s[i] = s[i];
  // (b, h, t) -> rows of one axis: first t into h, then h into b
  bool t_in_h = true, h_in_b = true;
  for (int i = 0; i < n; ++i) t_in_h = t_in_h && (H == 1 || L == 1 || s[i].h == L * s[i].l);
  int h_ext = H, l_ext = L;
  if (t_in_h) {
    // one axis of H L rows, kept as h
    for (int i = 0; i < n; ++i)
      if (L > 1) r.s[i].h = s[i].l;
    const int64_t hl = (int64_t)H * L;
    l_ext = 1;
    for (int i = 0; i < n; ++i) h_in_b = h_in_b && (B == 1 || hl == 1 || s[i].b == hl * r.s[i].h);
    h_ext = (int)hl;
  } else {
    for (int i = 0; i < n; ++i) h_in_b = h_in_b && B == 1;
    if (B == 1) {
      // (h, t) only: h is what remains of the division by L
      for (int i = 0; i < n; ++i) r.s[i].b = s[i].h;
      r.l = FastDiv((uint32_t)L);
      r.h = FastDiv(1);
      return r;
    }
    h_in_b = false;
  }
  if (h_in_b) {
    for (int i = 0; i < n; ++i)
      if (h_ext > 1) r.s[i].b = r.s[i].h;
    h_ext = 1;
  }
  r.l = FastDiv((uint32_t)l_ext);
  r.h = FastDiv((uint32_t)h_ext);
  return r;
}

}  // namespace favor

namespace {

using favor::View;

favor_status sizes_ok(int B, int H, int L, int d, favor_dtype dt) {
  if (B < 1 || H < 1 || L < 1 || d < 1) return FAVOR_ERR_INVALID_ARG;
  if (dt != FAVOR_F32 && dt != FAVOR_BF16) return FAVOR_ERR_INVALID_ARG;
  return FAVOR_OK;
}

int elem(favor_dtype dt) { return dt == FAVOR_BF16 ? 2 : 4; }

// An fp32 array of n elements: NULL is fine (and left out of the overlap checks)
bool flat_ok(const float* p) { return p == nullptr || reinterpret_cast<uintptr_t>(p) % 4 == 0; }

// `out` against another tensor: fine where it is the same view and that is allowed
bool clash(const View& out, const View& other, bool in_place) {
  if (in_place && favor::same_view(out, other)) return false;
  return favor::overlap(out, other);
}
bool clash(const View& out, const float* p, int64_t n) {
  return p != nullptr && favor::overlap(out, favor::flat_view(p, n, 4));
}
bool clash(const float* out, int64_t n, const float* p, int64_t np, bool in_place) {
  if (out == nullptr || p == nullptr || (in_place && out == p && n == np)) return false;
  return favor::overlap(favor::flat_view(out, n, 4), favor::flat_view(p, np, 4));
}

// 32-bit token strides and positions of the scan kernels
bool scan_fits(std::initializer_list<const View*> views) {
  for (const View* v : views)
    if (v->n[2] > (1 << 30) || v->s[2] >= (int64_t(1) << 31)) return false;
  return true;
}

// the most bytes, 16 or less, of which all the views' rows are made
int common_piece(std::initializer_list<const View*> views) {
  int piece = 16;
  for (const View* v : views)
    while (piece > v->esz && !v->pieces(piece)) piece /= 2;
  return piece;
}

favor_status done(cudaError_t e) { return e == cudaSuccess ? FAVOR_OK : FAVOR_ERR_CUDA; }

bool positive(float x) { return std::isfinite(x) && x > 0.f; }

// Sizes, positions and pairs of a rotation; counts the pairs.
favor_status turns_ok(int B, int Hq, int Hk, bool keys, int L, int d, const int32_t* pos, int pos_B, int n_axes,
                      const int* sections, const uint64_t* table, favor_pairing pairing, favor_dtype dt, int* counts,
                      int* n_pairs) {
  favor_status st = sizes_ok(B, Hq, L, d, dt);
  if (st == FAVOR_OK && keys) st = sizes_ok(B, Hk, L, d, dt);
  if (st != FAVOR_OK) return st;
  if (pairing != FAVOR_PAIR_ADJACENT && pairing != FAVOR_PAIR_HALVES) return FAVOR_ERR_INVALID_ARG;
  if (n_axes < 1 || n_axes > FAVOR_ROTARY_MAX_AXES || sections == nullptr) return FAVOR_ERR_INVALID_ARG;
  if (pos_B != 1 && pos_B != B) return FAVOR_ERR_INVALID_ARG;
  if (pos == nullptr || reinterpret_cast<uintptr_t>(pos) % 4 != 0) return FAVOR_ERR_INVALID_ARG;
  if (table == nullptr || reinterpret_cast<uintptr_t>(table) % 8 != 0) return FAVOR_ERR_INVALID_ARG;
  int64_t pairs = 0;
  for (int i = 0; i < n_axes; ++i) {
    if (sections[i] < 0) return FAVOR_ERR_INVALID_ARG;
    counts[i] = sections[i];
    pairs += sections[i];
  }
  if (pairs < 1 || 2 * pairs > d) return FAVOR_ERR_INVALID_ARG;
  *n_pairs = static_cast<int>(pairs);
  const int64_t lim = int64_t(1) << 31;
  if (d > favor::kNormMaxD || (int64_t)B * Hq >= lim || (int64_t)B * Hq * L >= lim) return FAVOR_ERR_UNSUPPORTED;
  if (keys && ((int64_t)B * Hk >= lim || (int64_t)B * Hk * L >= lim)) return FAVOR_ERR_UNSUPPORTED;
  // the kernels' steps over the heads stay inside 32 bits
  if ((int64_t)Hq + (keys ? Hk : 0) > lim - 16) return FAVOR_ERR_UNSUPPORTED;
  return FAVOR_OK;
}

favor_status rotary(const void* q, const int64_t* qs, void* qo, const int64_t* qos, const void* k, const int64_t* ks,
                    void* ko, const int64_t* kos, int B, int Hq, int Hk, int L, int d, const int32_t* pos, int pos_B,
                    int n_axes, const int* sections, const uint64_t* table, favor_pairing pairing, bool inverse,
                    favor_dtype dt, void* stream) {
  const bool keys = k != nullptr || ko != nullptr;
  favor::RotaryArgs a{};
  const favor_status st =
      turns_ok(B, Hq, Hk, keys, L, d, pos, pos_B, n_axes, sections, table, pairing, dt, a.sections, &a.pairs);
  if (st != FAVOR_OK) return st;
  const int pairs = a.pairs;
  const int e = elem(dt);
  View vq, vqo, vk{}, vko{};
  if (!favor::make_view(&vq, q, qs, B, Hq, L, d, e) || !favor::make_view(&vqo, qo, qos, B, Hq, L, d, e))
    return FAVOR_ERR_INVALID_ARG;
  if (favor::self_overlap(vqo) || clash(vqo, vq, true)) return FAVOR_ERR_INVALID_ARG;
  const View vpos = favor::flat_view(pos, (int64_t)n_axes * pos_B * L, 4), vtab = favor::flat_view(table, pairs, 8);
  if (clash(vqo, vpos, false) || clash(vqo, vtab, false)) return FAVOR_ERR_INVALID_ARG;
  int piece = common_piece({&vq, &vqo});
  if (keys) {
    if (!favor::make_view(&vk, k, ks, B, Hk, L, d, e) || !favor::make_view(&vko, ko, kos, B, Hk, L, d, e))
      return FAVOR_ERR_INVALID_ARG;
    if (favor::self_overlap(vko) || clash(vko, vk, true) || clash(vko, vq, false) || clash(vqo, vk, false) ||
        clash(vqo, vko, false) || clash(vko, vpos, false) || clash(vko, vtab, false))
      return FAVOR_ERR_INVALID_ARG;
    piece = std::min(piece, common_piece({&vk, &vko}));
  }
  a.q = q;
  a.k = k;
  a.qo = qo;
  a.ko = ko;
  a.qs = vq.strides();
  a.qos = vqo.strides();
  if (keys) {
    a.ks = vk.strides();
    a.kos = vko.strides();
  }
  a.B = B;
  a.Hq = Hq;
  a.Hk = keys ? Hk : 0;
  a.L = L;
  a.d = d;
  a.pos = pos;
  a.pos_B = pos_B;
  a.n_axes = n_axes;
  a.table = table;
  a.halves = pairing == FAVOR_PAIR_HALVES;
  a.inverse = inverse;
  return done(favor::launch_rotary(a, dt == FAVOR_BF16, piece, static_cast<cudaStream_t>(stream)));
}

favor_status fwd_gated_scan(const void* x, const int64_t* x_strides, const void* g, const int64_t* g_strides,
                            void* h, const int64_t* h_strides, const float* h0, float* hT, int B, int H, int L, int d,
                            favor_dtype dt, long long wait_cycles, int quits, int32_t* dev_status, void* stream) {
  const favor_status st = sizes_ok(B, H, L, d, dt);
  if (st != FAVOR_OK) return st;
  if (!flat_ok(h0) || !flat_ok(hT)) return FAVOR_ERR_INVALID_ARG;
  if ((int64_t)B * H * d >= (int64_t(1) << 31) || (int64_t)B * H >= (int64_t(1) << 31)) return FAVOR_ERR_UNSUPPORTED;
  const int e = elem(dt);
  View vx, vg, vh;
  if (!favor::make_view(&vx, x, x_strides, B, H, L, d, e) || !favor::make_view(&vg, g, g_strides, B, H, L, d, e) ||
      !favor::make_view(&vh, h, h_strides, B, H, L, d, e))
    return FAVOR_ERR_INVALID_ARG;
  const int64_t n = (int64_t)B * H * d;
  if (!scan_fits({&vx, &vg, &vh})) return FAVOR_ERR_UNSUPPORTED;
  if (favor::self_overlap(vh) || clash(vh, vx, true) || clash(vh, vg, true) || clash(vh, h0, n) || clash(vh, hT, n) ||
      clash(vx, hT, n) || clash(vg, hT, n) || clash(hT, n, h0, n, true))
    return FAVOR_ERR_INVALID_ARG;
  favor::ScanArgs a{};
  a.x = x;
  a.g = g;
  a.h = h;
  a.xs = vx.strides();
  a.gs = vg.strides();
  a.hs = vh.strides();
  a.status = dev_status;
  a.first = h0;
  a.last = hT;
  a.B = B;
  a.H = H;
  a.L = L;
  a.d = d;
  a.wait_cycles = wait_cycles;
  a.quits = quits;
  return done(favor::launch_scan(a, false, dt == FAVOR_BF16, common_piece({&vx, &vg, &vh}),
                                 static_cast<cudaStream_t>(stream)));
}

// ---- norms of queries and keys with their rotation --------------------------------
bool qk_norm_sizes(int B, int Hq, int Hk, int L, int d) {
  const int64_t lim = int64_t(1) << 31;
  return d <= favor::kQkNormMaxD && (int64_t)B * Hq < lim && (int64_t)B * Hq * L < lim && (int64_t)B * Hk < lim &&
         (int64_t)B * Hk * L < lim && (int64_t)Hq + Hk <= lim - 16;
}

struct QkSide {
  const void *x, *dy;
  void* out;
  const int64_t *xs, *dys, *os;
  const float* w;
  float* dw;
  int heads;
  View vx, vdy, vout;
};

favor_status qk_norm(QkSide* side, bool keys, float eps, int B, int L, int d, const int32_t* pos, int pos_B,
                     int n_axes, const int* sections, const uint64_t* table, favor_pairing pairing, favor_dtype dt,
                     bool backward, void* workspace, size_t ws_bytes, void* stream) {
  favor::QkNormArgs a{};
  const favor_status st = turns_ok(B, side[0].heads, side[1].heads, keys, L, d, pos, pos_B, n_axes, sections, table,
                                   pairing, dt, a.sections, &a.pairs);
  if (st != FAVOR_OK) return st;
  if (!positive(eps)) return FAVOR_ERR_INVALID_ARG;
  if (d > favor::kQkNormMaxD) return FAVOR_ERR_UNSUPPORTED;
  const int e = elem(dt), n = keys ? 2 : 1;
  a.B = B;
  a.Hq = side[0].heads;
  a.Hk = keys ? side[1].heads : 0;
  a.L = L;
  a.d = d;
  const bool sums = backward && (side[0].dw != nullptr || (keys && side[1].dw != nullptr));
  const size_t need = sums ? favor::qk_norm_workspace_bytes(a) : 0;
  if (need > 0 &&
      (workspace == nullptr || reinterpret_cast<uintptr_t>(workspace) % 256 != 0 || ws_bytes < need))
    return FAVOR_ERR_INVALID_ARG;
  const View vpos = favor::flat_view(pos, (int64_t)n_axes * pos_B * L, 4), vtab = favor::flat_view(table, a.pairs, 8);
  const View vw = favor::flat_view(workspace, (int64_t)need, 1);
  int piece = 16;
  for (int i = 0; i < n; ++i) {
    QkSide& s = side[i];
    if (!flat_ok(s.w) || !flat_ok(s.dw) || !favor::make_view(&s.vx, s.x, s.xs, B, s.heads, L, d, e) ||
        !favor::make_view(&s.vout, s.out, s.os, B, s.heads, L, d, e) ||
        (backward && !favor::make_view(&s.vdy, s.dy, s.dys, B, s.heads, L, d, e)))
      return FAVOR_ERR_INVALID_ARG;
    piece = std::min(piece, common_piece({&s.vx, &s.vout}));
    if (backward) piece = std::min(piece, common_piece({&s.vdy}));
    if (!backward) s.dw = nullptr;
  }
  for (int i = 0; i < n; ++i) {
    const QkSide& s = side[i];
    if (favor::self_overlap(s.vout) || clash(s.vout, vpos, false) || clash(s.vout, vtab, false) ||
        (need > 0 && (clash(vw, vpos, false) || clash(vw, vtab, false))))
      return FAVOR_ERR_INVALID_ARG;
    if (s.dw != nullptr && (clash(vpos, s.dw, d) || clash(vtab, s.dw, d))) return FAVOR_ERR_INVALID_ARG;
    for (int j = 0; j < n; ++j) {
      const QkSide& o = side[j];
      if (clash(s.vout, o.vx, i == j) || (backward && clash(s.vout, o.vdy, i == j)) || clash(s.vout, o.w, d) ||
          clash(s.vout, o.dw, d) || (j != i && clash(s.vout, o.vout, false)))
        return FAVOR_ERR_INVALID_ARG;
      if (s.dw != nullptr && (clash(o.vx, s.dw, d) || clash(o.vdy, s.dw, d) || clash(s.dw, d, o.w, d, false) ||
                              (j != i && clash(s.dw, d, o.dw, d, false))))
        return FAVOR_ERR_INVALID_ARG;
    }
    if (need > 0 && (favor::overlap(vw, s.vx) || favor::overlap(vw, s.vdy) || favor::overlap(vw, s.vout) ||
                     clash(vw, s.w, d) || clash(vw, s.dw, d)))
      return FAVOR_ERR_INVALID_ARG;
  }
  const QkSide& q = side[0];
  a.q = q.x;
  a.dqo = q.dy;
  a.qo = q.out;
  a.qs = q.vx.strides();
  a.qos = q.vout.strides();
  if (backward) a.dqos = q.vdy.strides();
  a.wq = q.w;
  a.dwq = q.dw;
  if (keys) {
    const QkSide& k = side[1];
    a.k = k.x;
    a.dko = k.dy;
    a.ko = k.out;
    a.ks = k.vx.strides();
    a.kos = k.vout.strides();
    if (backward) a.dkos = k.vdy.strides();
    a.wk = k.w;
    a.dwk = k.dw;
  }
  a.eps = eps;
  a.pos = pos;
  a.pos_B = pos_B;
  a.n_axes = n_axes;
  a.table = table;
  a.halves = pairing == FAVOR_PAIR_HALVES;
  return done(favor::launch_qk_norm(a, dt == FAVOR_BF16, piece, backward, static_cast<float*>(workspace),
                                    static_cast<cudaStream_t>(stream)));
}

// ---- causal linear attention with a decay per head --------------------------------
favor_status decay_sizes(int B, int H, int L, int d, favor_dtype dt) {
  const favor_status st = sizes_ok(B, H, L, d, dt);
  if (st != FAVOR_OK) return st;
  if (d > favor::kDecayMaxD || (int64_t)B * H >= (1 << 20) || L > (1 << 30)) return FAVOR_ERR_UNSUPPORTED;
  return FAVOR_OK;
}

favor::DecayShape decay_shape(const float* g, const int32_t* lengths, int32_t* status, int B, int H, int L, int d) {
  favor::DecayShape s{};
  s.g = g;
  s.lengths = lengths;
  s.status = status;
  s.B = B;
  s.H = H;
  s.L = L;
  s.d = d;
  return s;
}

int64_t decay_states(const favor::DecayShape& s) { return (int64_t)s.BH() * s.segs * s.d * s.d; }

// the flat operands of a call: what may not meet an output
struct Flat {
  View v[8];
  int n = 0;
  bool add(const void* p, int64_t count, int esz = 4) {
    if (p == nullptr) return true;
    if (reinterpret_cast<uintptr_t>(p) % 4 != 0) return false;
    v[n++] = favor::flat_view(p, count, esz);
    return true;
  }
  bool meets(const View& out) const {
    for (int i = 0; i < n; ++i)
      if (favor::overlap(v[i], out)) return true;
    return false;
  }
};

size_t decay_workspace(int B, int H, int L, int d, favor_dtype dt, bool backward) {
  // what either path may need, whatever the tensors' alignment
  favor::DecayShape s = decay_shape(nullptr, nullptr, nullptr, B, H, L, d);
  favor::decay_simt_plan(&s, backward ? 3 : 1);
  int64_t states = s.segs > 1 ? decay_states(s) : 0;
  if (dt == FAVOR_BF16) {
    favor::decay_tc_plan(&s, backward ? 3 : 1);
    if (!favor::decay_tc_ends_beside(s)) states = std::max(states, 2 * decay_states(s));      // in two pieces
  }
  return (size_t)states * (backward ? 2 : 1) * sizeof(float);
}

bool by16(const float* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

favor_status workspace_ok(const void* ws, size_t have, size_t need) {
  if (need == 0) return FAVOR_OK;
  if (ws == nullptr || reinterpret_cast<uintptr_t>(ws) % 256 != 0 || have < need) return FAVOR_ERR_INVALID_ARG;
  return FAVOR_OK;
}

}  // namespace

extern "C" {

favor_status favor_fwd_gated_scan(const void* x, const int64_t* x_strides, const void* g, const int64_t* g_strides,
                                  void* h, const int64_t* h_strides, const float* h0, float* hT, int B, int H, int L,
                                  int d, favor_dtype dt, int32_t* dev_status, void* stream) {
  return fwd_gated_scan(x, x_strides, g, g_strides, h, h_strides, h0, hT, B, H, L, d, dt, favor::tc::kWaitLimitCycles,
                        -1, dev_status, stream);
}

favor_status favor_selftest_scan_timeout(const void* x, const void* g, void* h, float* hT, int B, int H, int L, int d,
                                         favor_dtype dt, int64_t wait_cycles, int quits, int32_t* status,
                                         void* stream) {
  if (status == nullptr || wait_cycles < 0 || wait_cycles > favor::tc::kWaitLimitCycles) return FAVOR_ERR_INVALID_ARG;
  return fwd_gated_scan(x, nullptr, g, nullptr, h, nullptr, nullptr, hT, B, H, L, d, dt, wait_cycles, quits, status,
                        stream);
}

favor_status favor_bwd_gated_scan(const void* g, const int64_t* g_strides, const void* h, const int64_t* h_strides,
                                  const void* dh, const int64_t* dh_strides, void* dx, const int64_t* dx_strides,
                                  void* dg, const int64_t* dg_strides, const float* h0, const float* dhT, float* dh0,
                                  int B, int H, int L, int d, favor_dtype dt, int32_t* dev_status, void* stream) {
  const favor_status st = sizes_ok(B, H, L, d, dt);
  if (st != FAVOR_OK) return st;
  if (!flat_ok(h0) || !flat_ok(dhT) || !flat_ok(dh0)) return FAVOR_ERR_INVALID_ARG;
  if ((int64_t)B * H * d >= (int64_t(1) << 31) || (int64_t)B * H >= (int64_t(1) << 31)) return FAVOR_ERR_UNSUPPORTED;
  const int e = elem(dt);
  View vg, vh, vdh, vdx, vdg;
  if (!favor::make_view(&vg, g, g_strides, B, H, L, d, e) || !favor::make_view(&vh, h, h_strides, B, H, L, d, e) ||
      !favor::make_view(&vdh, dh, dh_strides, B, H, L, d, e) ||
      !favor::make_view(&vdx, dx, dx_strides, B, H, L, d, e) || !favor::make_view(&vdg, dg, dg_strides, B, H, L, d, e))
    return FAVOR_ERR_INVALID_ARG;
  const int64_t n = (int64_t)B * H * d;
  if (!scan_fits({&vg, &vh, &vdh, &vdx, &vdg})) return FAVOR_ERR_UNSUPPORTED;
  if (favor::self_overlap(vdx) || favor::self_overlap(vdg) || clash(vdx, vdg, false) || clash(vdx, vg, false) ||
      clash(vdx, vh, false) || clash(vdx, vdh, true) || clash(vdg, vg, true) || clash(vdg, vh, false) ||
      clash(vdg, vdh, false))
    return FAVOR_ERR_INVALID_ARG;
  for (const View* out : {&vdx, &vdg})
    if (clash(*out, h0, n) || clash(*out, dhT, n) || clash(*out, dh0, n)) return FAVOR_ERR_INVALID_ARG;
  if (clash(vg, dh0, n) || clash(vh, dh0, n) || clash(vdh, dh0, n) || clash(dh0, n, h0, n, false) ||
      clash(dh0, n, dhT, n, true))
    return FAVOR_ERR_INVALID_ARG;
  favor::ScanArgs a{};
  a.g = g;
  a.h_in = h;
  a.dh = dh;
  a.dx = dx;
  a.dg = dg;
  a.gs = vg.strides();
  a.his = vh.strides();
  a.dhs = vdh.strides();
  a.dxs = vdx.strides();
  a.dgs = vdg.strides();
  a.status = dev_status;
  a.first = dhT;
  a.h0 = h0;
  a.last = dh0;
  a.B = B;
  a.H = H;
  a.L = L;
  a.d = d;
  return done(favor::launch_scan(a, true, dt == FAVOR_BF16, common_piece({&vg, &vh, &vdh, &vdx, &vdg}),
                                 static_cast<cudaStream_t>(stream)));
}

favor_status favor_gated_scan_step(const void* x, const void* g, void* h, const float* state, float* new_state, int B,
                                   int H, int d, favor_dtype dt, void* stream) {
  const favor_status st = sizes_ok(B, H, 1, d, dt);
  if (st != FAVOR_OK) return st;
  const int e = elem(dt);
  for (const void* p : {x, g, static_cast<const void*>(h)})
    if (p == nullptr || reinterpret_cast<uintptr_t>(p) % e != 0) return FAVOR_ERR_INVALID_ARG;
  if (state == nullptr || new_state == nullptr || !flat_ok(state) || !flat_ok(new_state)) return FAVOR_ERR_INVALID_ARG;
  const int64_t n = (int64_t)B * H * d;
  if (n >= (int64_t(1) << 31) || (int64_t)B * H >= (int64_t(1) << 31)) return FAVOR_ERR_UNSUPPORTED;
  const View vx = favor::flat_view(x, n, e), vg = favor::flat_view(g, n, e), vh = favor::flat_view(h, n, e);
  const View vn = favor::flat_view(new_state, n, 4);
  if (clash(vh, vx, true) || clash(vh, vg, true) || clash(vh, state, n) || clash(vh, new_state, n) ||
      favor::overlap(vn, vx) || favor::overlap(vn, vg) || clash(new_state, n, state, n, true))
    return FAVOR_ERR_INVALID_ARG;
  return done(favor::launch_scan_step(x, g, h, state, new_state, n, dt == FAVOR_BF16,
                                      static_cast<cudaStream_t>(stream)));
}

favor_status favor_fwd_layer_norm(const void* x, const int64_t* x_strides, void* y, const int64_t* y_strides,
                                  const float* gamma, const float* beta, float eps, int B, int H, int L, int d,
                                  favor_dtype dt, void* stream) {
  const favor_status st = sizes_ok(B, H, L, d, dt);
  if (st != FAVOR_OK) return st;
  if (!positive(eps) || !flat_ok(gamma) || !flat_ok(beta)) return FAVOR_ERR_INVALID_ARG;
  if (d > favor::kNormMaxD || (int64_t)B * H >= (int64_t(1) << 31) || (int64_t)B * H * L >= (int64_t(1) << 31))
    return FAVOR_ERR_UNSUPPORTED;
  const int e = elem(dt);
  View vx, vy;
  if (!favor::make_view(&vx, x, x_strides, B, H, L, d, e) || !favor::make_view(&vy, y, y_strides, B, H, L, d, e))
    return FAVOR_ERR_INVALID_ARG;
  if (favor::self_overlap(vy) || clash(vy, vx, true) || clash(vy, gamma, d) || clash(vy, beta, d))
    return FAVOR_ERR_INVALID_ARG;
  favor::NormArgs a{};
  a.x = x;
  a.y = y;
  a.xs = vx.strides();
  a.ys = vy.strides();
  a.gamma = gamma;
  a.beta = beta;
  a.eps = eps;
  a.B = B;
  a.H = H;
  a.L = L;
  a.d = d;
  return done(favor::launch_norm_fwd(a, dt == FAVOR_BF16, common_piece({&vx, &vy}),
                                     static_cast<cudaStream_t>(stream)));
}

size_t favor_bwd_layer_norm_workspace_bytes(int B, int H, int L, int d, favor_dtype dt) {
  if (sizes_ok(B, H, L, d, dt) != FAVOR_OK || d > favor::kNormMaxD) return 0;
  if ((int64_t)B * H >= (int64_t(1) << 31) || (int64_t)B * H * L >= (int64_t(1) << 31)) return 0;
  return favor::norm_bwd_workspace_bytes((int64_t)B * H * L, d, dt == FAVOR_BF16);
}

favor_status favor_bwd_layer_norm(const void* x, const int64_t* x_strides, const void* dy, const int64_t* dy_strides,
                                  void* dx, const int64_t* dx_strides, const float* gamma, float* dgamma,
                                  float* dbeta, float eps, int B, int H, int L, int d, favor_dtype dt,
                                  void* workspace, size_t ws_bytes, void* stream) {
  const favor_status st = sizes_ok(B, H, L, d, dt);
  if (st != FAVOR_OK) return st;
  if (!positive(eps) || !flat_ok(gamma) || !flat_ok(dgamma) || !flat_ok(dbeta)) return FAVOR_ERR_INVALID_ARG;
  if (d > favor::kNormMaxD || (int64_t)B * H >= (int64_t(1) << 31) || (int64_t)B * H * L >= (int64_t(1) << 31))
    return FAVOR_ERR_UNSUPPORTED;
  const int e = elem(dt);
  View vx, vdy, vdx;
  if (!favor::make_view(&vx, x, x_strides, B, H, L, d, e) || !favor::make_view(&vdy, dy, dy_strides, B, H, L, d, e) ||
      !favor::make_view(&vdx, dx, dx_strides, B, H, L, d, e))
    return FAVOR_ERR_INVALID_ARG;
  if (favor::self_overlap(vdx) || clash(vdx, vx, true) || clash(vdx, vdy, true) || clash(vdx, gamma, d))
    return FAVOR_ERR_INVALID_ARG;
  const bool sums = dgamma != nullptr || dbeta != nullptr;
  for (const float* out : {dgamma, dbeta})
    if (clash(vx, out, d) || clash(vdy, out, d) || clash(vdx, out, d) || clash(out, d, gamma, d, false))
      return FAVOR_ERR_INVALID_ARG;
  if (clash(dgamma, d, dbeta, d, false)) return FAVOR_ERR_INVALID_ARG;
  if (sums) {
    const size_t need = favor::norm_bwd_workspace_bytes((int64_t)B * H * L, d, dt == FAVOR_BF16);
    if (need > 0) {
      if (workspace == nullptr || reinterpret_cast<uintptr_t>(workspace) % 256 != 0 || ws_bytes < need)
        return FAVOR_ERR_INVALID_ARG;
      const View vw = favor::flat_view(workspace, (int64_t)need, 1);
      if (favor::overlap(vw, vx) || favor::overlap(vw, vdy) || favor::overlap(vw, vdx)) return FAVOR_ERR_INVALID_ARG;
      for (const float* p : {gamma, static_cast<const float*>(dgamma), static_cast<const float*>(dbeta)})
        if (clash(vw, p, d)) return FAVOR_ERR_INVALID_ARG;
    }
  }
  favor::NormArgs a{};
  a.x = x;
  a.dy = dy;
  a.dx = dx;
  a.xs = vx.strides();
  a.dys = vdy.strides();
  a.dxs = vdx.strides();
  a.gamma = gamma;
  a.dgamma = dgamma;
  a.dbeta = dbeta;
  a.eps = eps;
  a.B = B;
  a.H = H;
  a.L = L;
  a.d = d;
  return done(favor::launch_norm_bwd(a, dt == FAVOR_BF16, common_piece({&vx, &vdy, &vdx}),
                                     static_cast<float*>(workspace), static_cast<cudaStream_t>(stream)));
}

favor_status favor_fwd_rotary(const void* q, const int64_t* q_strides, void* q_out, const int64_t* q_out_strides,
                              const void* k, const int64_t* k_strides, void* k_out, const int64_t* k_out_strides,
                              int B, int Hq, int Hk, int L, int d, const int32_t* pos, int pos_B, int n_axes,
                              const int* sections, const uint64_t* table, favor_pairing pairing, favor_dtype dt,
                              void* stream) {
  return rotary(q, q_strides, q_out, q_out_strides, k, k_strides, k_out, k_out_strides, B, Hq, Hk, L, d, pos, pos_B,
                n_axes, sections, table, pairing, false, dt, stream);
}

favor_status favor_bwd_rotary(const void* dq_out, const int64_t* dq_out_strides, void* dq, const int64_t* dq_strides,
                              const void* dk_out, const int64_t* dk_out_strides, void* dk, const int64_t* dk_strides,
                              int B, int Hq, int Hk, int L, int d, const int32_t* pos, int pos_B, int n_axes,
                              const int* sections, const uint64_t* table, favor_pairing pairing, favor_dtype dt,
                              void* stream) {
  return rotary(dq_out, dq_out_strides, dq, dq_strides, dk_out, dk_out_strides, dk, dk_strides, B, Hq, Hk, L, d, pos,
                pos_B, n_axes, sections, table, pairing, true, dt, stream);
}

favor_status favor_fwd_qk_norm_rotary(const void* q, const int64_t* q_strides, void* q_out,
                                      const int64_t* q_out_strides, const void* k, const int64_t* k_strides,
                                      void* k_out, const int64_t* k_out_strides, const float* q_weight,
                                      const float* k_weight, float eps, int B, int Hq, int Hk, int L, int d,
                                      const int32_t* pos, int pos_B, int n_axes, const int* sections,
                                      const uint64_t* table, favor_pairing pairing, favor_dtype dt, void* stream) {
  QkSide side[2] = {{q, nullptr, q_out, q_strides, nullptr, q_out_strides, q_weight, nullptr, Hq, {}, {}, {}},
                    {k, nullptr, k_out, k_strides, nullptr, k_out_strides, k_weight, nullptr, Hk, {}, {}, {}}};
  return qk_norm(side, k != nullptr || k_out != nullptr, eps, B, L, d, pos, pos_B, n_axes, sections, table, pairing,
                 dt, false, nullptr, 0, stream);
}

favor_status favor_bwd_qk_norm_rotary(const void* q, const int64_t* q_strides, const void* dq_out,
                                      const int64_t* dq_out_strides, void* dq, const int64_t* dq_strides,
                                      const void* k, const int64_t* k_strides, const void* dk_out,
                                      const int64_t* dk_out_strides, void* dk, const int64_t* dk_strides,
                                      const float* q_weight, const float* k_weight, float* dq_weight,
                                      float* dk_weight, float eps, int B, int Hq, int Hk, int L, int d,
                                      const int32_t* pos, int pos_B, int n_axes, const int* sections,
                                      const uint64_t* table, favor_pairing pairing, favor_dtype dt, void* workspace,
                                      size_t ws_bytes, void* stream) {
  QkSide side[2] = {{q, dq_out, dq, q_strides, dq_out_strides, dq_strides, q_weight, dq_weight, Hq, {}, {}, {}},
                    {k, dk_out, dk, k_strides, dk_out_strides, dk_strides, k_weight, dk_weight, Hk, {}, {}, {}}};
  return qk_norm(side, k != nullptr || dk_out != nullptr || dk != nullptr, eps, B, L, d, pos, pos_B, n_axes, sections,
                 table, pairing, dt, true, workspace, ws_bytes, stream);
}

size_t favor_bwd_qk_norm_rotary_workspace_bytes(int B, int Hq, int Hk, int L, int d, favor_dtype dt) {
  if (sizes_ok(B, Hq, L, d, dt) != FAVOR_OK || Hk < 0 || !qk_norm_sizes(B, Hq, Hk, L, d)) return 0;
  favor::QkNormArgs a{};
  a.B = B;
  a.Hq = Hq;
  a.Hk = Hk;
  a.L = L;
  a.d = d;
  return favor::qk_norm_workspace_bytes(a);
}

size_t favor_decay_attention_workspace_bytes(int B, int H, int L, int d, favor_dtype dt, int backward) {
  if (decay_sizes(B, H, L, d, dt) != FAVOR_OK) return 0;
  return decay_workspace(B, H, L, d, dt, backward != 0);
}

favor_status favor_fwd_decay_attention(const void* q, const int64_t* q_strides, const void* k,
                                       const int64_t* k_strides, const void* v, const int64_t* v_strides, void* o,
                                       const int64_t* o_strides, const float* g, const int32_t* lengths,
                                       const float* S0, float* ST, float scale, int B, int H, int L, int d,
                                       favor_dtype dt, void* workspace, size_t ws_bytes, int32_t* dev_status,
                                       void* stream) {
  favor_status st = decay_sizes(B, H, L, d, dt);
  if (st != FAVOR_OK) return st;
  if (g == nullptr || !std::isfinite(scale)) return FAVOR_ERR_INVALID_ARG;
  const int e = elem(dt);
  View vq, vk, vv, vo;
  if (!favor::make_view(&vq, q, q_strides, B, H, L, d, e) || !favor::make_view(&vk, k, k_strides, B, H, L, d, e) ||
      !favor::make_view(&vv, v, v_strides, B, H, L, d, e) || !favor::make_view(&vo, o, o_strides, B, H, L, d, e))
    return FAVOR_ERR_INVALID_ARG;
  const int64_t states = (int64_t)B * H * d * d;
  const size_t need = decay_workspace(B, H, L, d, dt, false);
  st = workspace_ok(workspace, ws_bytes, need);
  if (st != FAVOR_OK) return st;
  Flat flat;
  if (!flat.add(g, H) || !flat.add(lengths, B) || !flat.add(S0, states) || !flat_ok(ST)) return FAVOR_ERR_INVALID_ARG;
  const View ws_view = favor::flat_view(workspace, (int64_t)need, 1);
  if (favor::self_overlap(vo) || flat.meets(vo) || clash(vo, ST, states) ||
      (need > 0 && (favor::overlap(vo, ws_view) || flat.meets(ws_view) || clash(ws_view, ST, states))))
    return FAVOR_ERR_INVALID_ARG;
  for (const View* in : {&vq, &vk, &vv})
    if (favor::overlap(vo, *in) || clash(*in, ST, states) || (need > 0 && favor::overlap(*in, ws_view)))
      return FAVOR_ERR_INVALID_ARG;
  if (ST != nullptr) {
    if (ST == S0) --flat.n;                              // S0 was added last
    if (flat.meets(favor::flat_view(ST, states, 4))) return FAVOR_ERR_INVALID_ARG;
  }
  const auto strm = static_cast<cudaStream_t>(stream);
  const bool bf16 = dt == FAVOR_BF16;
  const int piece = common_piece({&vq, &vk, &vv});
  favor::DecayShape s = decay_shape(g, lengths, dev_status, B, H, L, d);
  favor::DecayPass p{};
  p.a = q;
  p.b = k;
  p.c = v;
  p.o = o;
  p.as = vq.strides();
  p.bs = vk.strides();
  p.cs = vv.strides();
  p.os = vo.strides();
  p.s_w = p.s_r = scale;
  p.s_u = 1.f;
  if (L <= favor::kDecayFew) {
    p.start = S0;
    p.last = ST;
    return done(favor::decay_few(p, s, bf16, strm));
  }
  const View* all[4] = {&vq, &vk, &vv, &vo};
  favor::DecayMap maps[4];
  bool tc = favor::decay_tc_takes(all, 4, bf16, d) && by16(S0);
  for (int i = 0; i < 4 && tc; ++i) tc = favor::decay_tc_map(&maps[i], *all[i]);
  if (tc) favor::decay_tc_plan(&s, 1);
  else favor::decay_simt_plan(&s, 1);
  float* ws = static_cast<float*>(workspace);
  const favor::DecayGain gain{k, v, vk.strides(), vv.strides(), ws, 1.f, false};
  const favor::DecayScan scan{ws, S0, ST, false, tc ? 2 : 1};
  cudaError_t err = cudaSuccess;
  if (!tc) {
    if (s.segs > 1) {
      err = favor::decay_simt_gains(&gain, 1, s, bf16, piece, strm);
      if (err == cudaSuccess) err = favor::decay_scan_states(&scan, 1, s, strm);
    }
    p.start = s.segs > 1 ? ws : S0;
    p.last = s.segs > 1 ? nullptr : ST;
    if (err == cudaSuccess) err = favor::decay_simt_passes(&p, 1, s, bf16, piece, strm);
    return done(err);
  }
  const int64_t dd = (int64_t)d * d;
  favor::DecayTcPass pass{p, dd, false, &maps[0], &maps[1], &maps[2], &maps[3]};
  pass.p.start = S0;
  favor::DecayTcGain tc_gain{gain, nullptr, false, &maps[1], &maps[2]};
  const bool beside = favor::decay_tc_ends_beside(s);
  if (s.segs > 1 || (ST != nullptr && !beside)) {
    err = favor::decay_tc_gains(&tc_gain, 1, s, strm);
    if (err == cudaSuccess) err = favor::decay_scan_states(&scan, 1, s, strm);
    pass.p.start = ws;
    pass.step = 2 * dd;
    pass.after_scan = true;
  }
  if (err == cudaSuccess) err = favor::decay_tc_passes(&pass, 1, s, strm);
  if (err == cudaSuccess && beside && ST != nullptr) {
    tc_gain.p.out = ST;
    tc_gain.first = S0;
    tc_gain.ends = true;
    err = favor::decay_tc_gains(&tc_gain, 1, s, strm);
  }
  return done(err);
}

favor_status favor_bwd_decay_attention(const void* q, const int64_t* q_strides, const void* k,
                                       const int64_t* k_strides, const void* v, const int64_t* v_strides,
                                       const void* d_o, const int64_t* do_strides, void* dq,
                                       const int64_t* dq_strides, void* dk, const int64_t* dk_strides, void* dv,
                                       const int64_t* dv_strides, const float* g, const int32_t* lengths,
                                       const float* S0, const float* dST, float* dS0, float scale, int B, int H,
                                       int L, int d, favor_dtype dt, void* workspace, size_t ws_bytes,
                                       int32_t* dev_status, void* stream) {
  favor_status st = decay_sizes(B, H, L, d, dt);
  if (st != FAVOR_OK) return st;
  if (g == nullptr || !std::isfinite(scale)) return FAVOR_ERR_INVALID_ARG;
  const int e = elem(dt);
  View in[4], out[3];
  const void* inp[4] = {q, k, v, d_o};
  const int64_t* ins[4] = {q_strides, k_strides, v_strides, do_strides};
  void* outp[3] = {dq, dk, dv};
  const int64_t* outs[3] = {dq_strides, dk_strides, dv_strides};
  for (int i = 0; i < 4; ++i)
    if (!favor::make_view(&in[i], inp[i], ins[i], B, H, L, d, e)) return FAVOR_ERR_INVALID_ARG;
  for (int i = 0; i < 3; ++i)
    if (!favor::make_view(&out[i], outp[i], outs[i], B, H, L, d, e) || favor::self_overlap(out[i]))
      return FAVOR_ERR_INVALID_ARG;
  const int64_t states = (int64_t)B * H * d * d;
  const size_t need = decay_workspace(B, H, L, d, dt, true);
  st = workspace_ok(workspace, ws_bytes, need);
  if (st != FAVOR_OK) return st;
  // all that an output may not meet: the flat operands, the inputs and the other outputs
  Flat flat;
  if (!flat.add(g, H) || !flat.add(lengths, B) || !flat.add(S0, states) || !flat.add(dST, states) || !flat_ok(dS0))
    return FAVOR_ERR_INVALID_ARG;
  const View ws_view = favor::flat_view(workspace, (int64_t)need, 1);
  if (need > 0 && flat.meets(ws_view)) return FAVOR_ERR_INVALID_ARG;
  for (int i = 0; i < 3; ++i) {
    if (flat.meets(out[i]) || clash(out[i], dS0, states) || (need > 0 && favor::overlap(out[i], ws_view)))
      return FAVOR_ERR_INVALID_ARG;
    for (const View& v_in : in)
      if (favor::overlap(out[i], v_in)) return FAVOR_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (favor::overlap(out[i], out[j])) return FAVOR_ERR_INVALID_ARG;
  }
  for (const View& v_in : in)
    if (clash(v_in, dS0, states) || (need > 0 && favor::overlap(v_in, ws_view))) return FAVOR_ERR_INVALID_ARG;
  if (dS0 != nullptr) {
    const View vd = favor::flat_view(dS0, states, 4);
    if (dS0 == dST) --flat.n;                            // dST was added last
    if (flat.meets(vd) || (need > 0 && favor::overlap(ws_view, vd))) return FAVOR_ERR_INVALID_ARG;
  }
  const auto strm = static_cast<cudaStream_t>(stream);
  const bool bf16 = dt == FAVOR_BF16;
  const int piece = common_piece({&in[0], &in[1], &in[2], &in[3]});
  favor::DecayShape s = decay_shape(g, lengths, dev_status, B, H, L, d);
  const View* all[7] = {&in[0], &in[1], &in[2], &in[3], &out[0], &out[1], &out[2]};
  favor::DecayMap maps[7];
  bool tc = favor::decay_tc_takes(all, 7, bf16, d) && by16(S0) && by16(dST);
  for (int i = 0; i < 7 && tc; ++i) tc = favor::decay_tc_map(&maps[i], *all[i]);
  if (tc) favor::decay_tc_plan(&s, 3);
  else favor::decay_simt_plan(&s, 3);
  float *ws = static_cast<float*>(workspace), *ws_r = ws != nullptr ? ws + (tc ? 2 : 1) * decay_states(s) : nullptr;
  const favor::DecayGain gains[2] = {{k, v, in[1].strides(), in[2].strides(), ws, 1.f, false},
                                     {q, d_o, in[0].strides(), in[3].strides(), ws_r, scale, true}};
  const favor::DecayScan scans[2] = {{ws, S0, nullptr, false, tc ? 2 : 1}, {ws_r, dST, dS0, true, tc ? 2 : 1}};
  // dq, dk, dv: rows a, b, c among q, k, v, do
  const int abc[3][3] = {{3, 2, 1}, {2, 3, 0}, {1, 0, 3}};
  favor::DecayTcPass passes[3] = {};
  for (int i = 0; i < 3; ++i) {
    const View &a = in[abc[i][0]], &b = in[abc[i][1]], &c = in[abc[i][2]];
    favor::DecayPass& p = passes[i].p;
    p.a = a.p;
    p.b = b.p;
    p.c = c.p;
    p.o = outp[i];
    p.as = a.strides();
    p.bs = b.strides();
    p.cs = c.strides();
    p.os = out[i].strides();
    p.rev = i > 0;
    p.transposed = i < 2;
    p.s_w = scale;
    p.s_r = i == 0 ? scale : 1.f;
    p.s_u = i == 0 ? 1.f : scale;
    p.start = i == 0 ? S0 : dST;
    passes[i].step = (int64_t)d * d;
    passes[i].a = &maps[abc[i][0]];
    passes[i].b = &maps[abc[i][1]];
    passes[i].c = &maps[abc[i][2]];
    passes[i].o = &maps[4 + i];
  }
  cudaError_t err = cudaSuccess;
  if (!tc) {
    if (s.segs > 1) {
      err = favor::decay_simt_gains(gains, 2, s, bf16, piece, strm);
      if (err == cudaSuccess) err = favor::decay_scan_states(scans, 2, s, strm);
    }
    favor::DecayPass simt[3];
    for (int i = 0; i < 3; ++i) {
      simt[i] = passes[i].p;
      if (s.segs > 1) simt[i].start = i == 0 ? ws : ws_r;
      else if (i == 2) simt[i].last = dS0;
    }
    // one segment leaves dS0 itself, which may be the dST that dk reads: dv follows
    const bool apart = s.segs == 1 && dS0 != nullptr && dS0 == dST;
    if (err == cudaSuccess) err = favor::decay_simt_passes(simt, apart ? 2 : 3, s, bf16, piece, strm);
    if (err == cudaSuccess && apart) err = favor::decay_simt_passes(simt + 2, 1, s, bf16, piece, strm);
    return done(err);
  }
  favor::DecayTcGain tc_gains[2] = {{gains[0], nullptr, false, &maps[1], &maps[2]},
                                    {gains[1], nullptr, false, &maps[0], &maps[3]}};
  const bool beside = favor::decay_tc_ends_beside(s);
  if (s.segs > 1 || (dS0 != nullptr && !beside)) {
    const int from = s.segs > 1 ? 0 : 1;                 // one segment: only what dS0 is made of
    err = favor::decay_tc_gains(tc_gains + from, 2 - from, s, strm);
    if (err == cudaSuccess) err = favor::decay_scan_states(scans + from, 2 - from, s, strm);
    for (auto& p : passes) p.after_scan = true;
    for (int i = from; i < 3; ++i) {
      passes[i].p.start = i == 0 ? ws : ws_r;
      passes[i].step = 2 * (int64_t)d * d;
    }
  }
  if (err == cudaSuccess) err = favor::decay_tc_passes(passes, 3, s, strm);
  if (err == cudaSuccess && beside && dS0 != nullptr) {
    tc_gains[1].p.out = dS0;
    tc_gains[1].first = dST;
    tc_gains[1].ends = true;
    err = favor::decay_tc_gains(tc_gains + 1, 1, s, strm);
  }
  return done(err);
}

favor_status favor_decay_attention_step(const void* q, const int64_t* q_strides, const void* k,
                                        const int64_t* k_strides, const void* v, const int64_t* v_strides, void* o,
                                        const int64_t* o_strides, const float* g, const float* state,
                                        float* new_state, float scale, int B, int H, int d, favor_dtype dt,
                                        void* stream) {
  const favor_status st = decay_sizes(B, H, 1, d, dt);
  if (st != FAVOR_OK) return st;
  if (g == nullptr || state == nullptr || new_state == nullptr || !flat_ok(g) || !flat_ok(state) ||
      !flat_ok(new_state) || !std::isfinite(scale))
    return FAVOR_ERR_INVALID_ARG;
  const int e = elem(dt);
  const void* p[4] = {q, k, v, o};
  const int64_t* strides[4] = {q_strides, k_strides, v_strides, o_strides};
  View views[4];
  for (int i = 0; i < 4; ++i) {
    int64_t s3[3] = {(int64_t)H * d, d, 0};
    if (strides[i] != nullptr) {
      s3[0] = strides[i][0];
      s3[1] = strides[i][1];
    }
    if (!favor::make_view(&views[i], p[i], s3, B, H, 1, d, e)) return FAVOR_ERR_INVALID_ARG;
  }
  const int64_t n = (int64_t)B * H * d * d;
  const View vn = favor::flat_view(new_state, n, 4), vg = favor::flat_view(g, H, 4);
  if (favor::self_overlap(views[3]) || clash(views[3], state, n) || favor::overlap(views[3], vn) ||
      favor::overlap(views[3], vg) || favor::overlap(vn, vg) || clash(new_state, n, state, n, true))
    return FAVOR_ERR_INVALID_ARG;
  for (int i = 0; i < 3; ++i)
    if (favor::overlap(views[3], views[i]) || favor::overlap(vn, views[i])) return FAVOR_ERR_INVALID_ARG;
  favor::DecayStep a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.o = o;
  int64_t* to[4] = {a.qs, a.ks, a.vs, a.os};
  for (int i = 0; i < 4; ++i) {
    to[i][0] = views[i].s[0];
    to[i][1] = views[i].s[1];
  }
  a.g = g;
  a.state = state;
  a.next = new_state;
  a.scale = scale;
  a.B = B;
  a.H = H;
  a.d = d;
  a.vec = d % 4 == 0 && reinterpret_cast<uintptr_t>(state) % 16 == 0 && reinterpret_cast<uintptr_t>(new_state) % 16 == 0;
  return done(favor::launch_decay_step(a, dt == FAVOR_BF16, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
