// C ABI entry points of the sequence operators: argument checks and dispatch.
#include <algorithm>
#include <cmath>
#include <initializer_list>

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

favor_status rotary(const void* q, const int64_t* qs, void* qo, const int64_t* qos, const void* k, const int64_t* ks,
                    void* ko, const int64_t* kos, int B, int Hq, int Hk, int L, int d, const int32_t* pos, int pos_B,
                    int n_axes, const int* sections, const uint64_t* table, favor_pairing pairing, bool inverse,
                    favor_dtype dt, void* stream) {
  const bool keys = k != nullptr || ko != nullptr;
  favor_status st = sizes_ok(B, Hq, L, d, dt);
  if (st == FAVOR_OK && keys) st = sizes_ok(B, Hk, L, d, dt);
  if (st != FAVOR_OK) return st;
  if (pairing != FAVOR_PAIR_ADJACENT && pairing != FAVOR_PAIR_HALVES) return FAVOR_ERR_INVALID_ARG;
  if (n_axes < 1 || n_axes > FAVOR_ROTARY_MAX_AXES || sections == nullptr) return FAVOR_ERR_INVALID_ARG;
  if (pos_B != 1 && pos_B != B) return FAVOR_ERR_INVALID_ARG;
  if (pos == nullptr || reinterpret_cast<uintptr_t>(pos) % 4 != 0) return FAVOR_ERR_INVALID_ARG;
  if (table == nullptr || reinterpret_cast<uintptr_t>(table) % 8 != 0) return FAVOR_ERR_INVALID_ARG;
  favor::RotaryArgs a{};
  int64_t pairs = 0;
  for (int i = 0; i < n_axes; ++i) {
    if (sections[i] < 0) return FAVOR_ERR_INVALID_ARG;
    a.sections[i] = sections[i];
    pairs += sections[i];
  }
  if (pairs < 1 || 2 * pairs > d) return FAVOR_ERR_INVALID_ARG;
  const int64_t lim = int64_t(1) << 31;
  if (d > favor::kNormMaxD || (int64_t)B * Hq >= lim || (int64_t)B * Hq * L >= lim) return FAVOR_ERR_UNSUPPORTED;
  if (keys && ((int64_t)B * Hk >= lim || (int64_t)B * Hk * L >= lim)) return FAVOR_ERR_UNSUPPORTED;
  // the kernels' steps over the heads stay inside 32 bits
  if ((int64_t)Hq + (keys ? Hk : 0) > lim - 16) return FAVOR_ERR_UNSUPPORTED;
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
  a.pairs = static_cast<int>(pairs);
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

}  // extern "C"
