/*
 * favor_ops.h — C ABI of the sequence operators beside the FAVOR+ attention
 * (favor.h): what happens to queries and keys before the feature map (layer
 * norm, rotary positions, both in one pass with a root-mean-square norm), the
 * gated linear recurrence, the decayed sibling of the causal pass's prefix
 * sum, and causal linear attention with a decay per head.
 *
 * Conventions shared by every call (those of favor.h unless stated here):
 *  - Tensors are [B, H, L, d], d fastest with unit stride, of dtype `dt`
 *    (FAVOR_F32 or FAVOR_BF16); arithmetic, sums and statistics are fp32.
 *  - Each tensor is followed by its strides: an int64_t[3] on the host with
 *    the element strides of B, H and L, or NULL for a contiguous tensor, so
 *    that a view (queries inside a joint projection's [B, L, 3, H, d]
 *    output) needs no copy.  Strides are >= 0; the stride of an extent of 1
 *    is ignored.  An input may have a stride of 0 (a broadcast); an output
 *    must not map two elements to one address (FAVOR_ERR_INVALID_ARG).
 *    Offsets are 64-bit: tensors beyond 2^31 elements are fine.
 *  - Pointers are aligned to their element.  Tensors whose pointers and
 *    strides are multiples of 16 bytes and whose rows are whole 16-byte
 *    pieces run fastest, then those made of two elements, then all others.
 *  - An output may be the very input it replaces (same pointer and strides)
 *    where the call says so.  Any other overlap of an output with an input
 *    or another output is FAVOR_ERR_INVALID_ARG; two views with the same
 *    strides (the queries and keys of one buffer) are compared element by
 *    element, other pairs by their byte ranges.
 *  - B, H, L, d >= 1.  Calls allocate nothing and do not synchronise; all
 *    launches are asynchronous on `stream`, and results do not depend on
 *    timing (no floating-point atomics).  The order of sums (a row's, the
 *    rows', a scan's runs of tokens) is fixed by the shape, the type, the
 *    device and the tensors' alignment (16 bytes, two elements or one, as
 *    above): the same values at another alignment may differ in their last
 *    bits.  NaN and infinities pass through as the formulas have them unless
 *    stated.
 */
#ifndef FAVOR_OPS_H_
#define FAVOR_OPS_H_

#include "favor.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * favor_fwd_gated_scan — gated linear recurrence over the tokens, each of
 * the B H d channels by itself:
 *   h_t = exp(g_t) h_{t-1} + x_t,   h_{-1} = h0,   hT = h_{L-1}
 * g: logarithm of the gate (<= 0 for a decay; not checked: positive ones are
 * fine while the products of consecutive gates stay finite in fp32, since a
 * run of tokens is applied as one map).  Where exp(g_t)
 * is 0 in fp32 (minus infinity, the type's lowest value) the state is
 * dropped, h_t = x_t, whatever it was, infinities and NaN included: such a
 * gate starts a new sequence packed into the same row.  Infinities and NaN end
 * there alone.  The gates of a run of tokens are multiplied in fp32 before they
 * meet the state (the runs, of at most 96 tokens, follow the shape, the
 * tensors' alignment and the device): a product below fp32's normal numbers has
 * fewer bits or is 0, so that a finite state h is off by at most 2^-143 |h|.
 * A token with g = 0 and x = 0 carries the state over, which is how padding
 * behind a short sequence leaves hT at its last token.
 * h0: fp32 [B, H, d] contiguous, NULL for zeros.  hT: the same, NULL if not
 * wanted; hT may be h0.  h may be x or g.  h is rounded to dt once, the
 * state is carried in fp32.  dev_status: a bounded wait of a cluster's CTAs
 * on one another that ran out is reported there (FAVOR_ERR_TIMEOUT).
 * Supported: B H d < 2^31, L <= 2^30, token strides below 2^31.
 */
favor_status favor_fwd_gated_scan(const void* x, const int64_t* x_strides,
                                  const void* g, const int64_t* g_strides,
                                  void* h, const int64_t* h_strides,
                                  const float* h0, float* hT,
                                  int B, int H, int L, int d, favor_dtype dt,
                                  int32_t* dev_status, void* stream);

/*
 * favor_bwd_gated_scan — its gradients, for dh = dL/dh and dhT = dL/dhT
 * (fp32 [B, H, d], NULL for zeros):
 *   c_L = dhT,  dx_t = dh_t + c_{t+1},  c_t = exp(g_t) dx_t,
 *   dg_t = c_t h_{t-1},  dh0 = c_0
 * h is the forward call's output, h0 its initial state (NULL for zeros).
 * Where exp(g_t) is 0, c_t and dg_t are 0 whatever the other factors are.
 * dh0: fp32 [B, H, d], NULL if not wanted; dh0 may be dhT.  dx may be dh and
 * dg may be g; neither may be h.
 */
favor_status favor_bwd_gated_scan(const void* g, const int64_t* g_strides,
                                  const void* h, const int64_t* h_strides,
                                  const void* dh, const int64_t* dh_strides,
                                  void* dx, const int64_t* dx_strides,
                                  void* dg, const int64_t* dg_strides,
                                  const float* h0, const float* dhT, float* dh0,
                                  int B, int H, int L, int d, favor_dtype dt,
                                  int32_t* dev_status, void* stream);

/*
 * favor_gated_scan_step — one token: x, g and h contiguous [B, H, d] (this call
 * alone takes no strides),
 *   new_state = exp(g) state + x (fp32 [B, H, d]),  h = new_state rounded to dt
 * new_state may be state, and h may be x or g.  State and h equal row t of
 * the forward call over the whole sequence, given the state of the tokens
 * before it.
 */
favor_status favor_gated_scan_step(const void* x, const void* g, void* h,
                                   const float* state, float* new_state,
                                   int B, int H, int d, favor_dtype dt, void* stream);

/*
 * favor_fwd_layer_norm — over the last axis of each row:
 *   y = (x - mean) / sqrt(var + eps) * gamma + beta,  var = mean (x - mean)^2
 * gamma, beta: fp32 [d], each NULL for 1 and 0.  eps > 0 and finite.  y may
 * be x.  A row whose sum or sum of squares leaves fp32 (values beyond about
 * 2^57) is NaN, as one with infinities or NaN is; rows do not touch one another.
 * Supported: d <= 16384, B H L < 2^31.
 */
favor_status favor_fwd_layer_norm(const void* x, const int64_t* x_strides,
                                  void* y, const int64_t* y_strides,
                                  const float* gamma, const float* beta, float eps,
                                  int B, int H, int L, int d, favor_dtype dt, void* stream);

/*
 * favor_bwd_layer_norm — its gradients for dy = dL/dy; with
 * xh = (x - mean) / sqrt(var + eps) (recomputed from x) and n = dy gamma:
 *   dx = (n - mean n - xh mean(n xh)) / sqrt(var + eps)
 *   dgamma = sum over the rows of dy xh,  dbeta = sum over the rows of dy
 * dgamma, dbeta: fp32 [d], overwritten, each NULL if not wanted.  dx may be
 * dy or x.  The rows are summed in a fixed order (see above).  Workspace of
 * favor_bwd_layer_norm_workspace_bytes(...) bytes, 256-byte aligned (0 bytes,
 * and NULL allowed, where dgamma and dbeta are both NULL); calls that share one
 * must be ordered on one stream.
 */
favor_status favor_bwd_layer_norm(const void* x, const int64_t* x_strides,
                                  const void* dy, const int64_t* dy_strides,
                                  void* dx, const int64_t* dx_strides,
                                  const float* gamma, float* dgamma, float* dbeta, float eps,
                                  int B, int H, int L, int d, favor_dtype dt,
                                  void* workspace, size_t ws_bytes, void* stream);
/* The size follows the current device's number of SMs: asked for with the
 * device current that the call runs on.  0 for arguments outside the supported
 * shapes. */
size_t favor_bwd_layer_norm_workspace_bytes(int B, int H, int L, int d, favor_dtype dt);

/*
 * favor_fwd_rotary — rotates queries and keys by their tokens' positions on
 * one to four axes (a text's index; an image's row and column; a video's
 * time, row and column).  The first 2 P of the d channels form P pairs
 * (u, v); pair p belongs to one axis a, turns by table[p] per unit of
 * position and becomes
 *   (u cos t - v sin t, u sin t + v cos t),  t = 2 pi (pos_a table[p] / 2^64)
 * and the other channels are copied.  Rotating q and k before the feature
 * map makes the attention estimate softmax over relative positions.
 *  - q [B, Hq, L, d] -> q_out, k [B, Hk, L, d] -> k_out; k and k_out may both
 *    be NULL (Hk is then ignored).  q_out may be q, k_out may be k.
 *  - pos: device int32 [n_axes, pos_B, L] contiguous, any value; pos_B = B,
 *    or 1 for positions shared by the batch.
 *  - table: device uint64 [P], the fraction of a turn per unit of position in
 *    64-bit fixed point (a turn is 2^64): the product with a position wraps
 *    to the exact fraction of a turn, so far positions lose nothing.
 *  - sections: host int[n_axes], the pairs of each axis in order (>= 0);
 *    their sum is P >= 1, 2 P <= d.
 *  - pairing: FAVOR_PAIR_ADJACENT (channels 2p and 2p + 1) or
 *    FAVOR_PAIR_HALVES (channels p and p + P).
 * Supported: B Hq L and B Hk L < 2^31, Hq + Hk <= 2^31 - 16, d <= 16384.
 */
typedef enum favor_pairing { FAVOR_PAIR_ADJACENT = 0, FAVOR_PAIR_HALVES = 1 } favor_pairing;
#define FAVOR_ROTARY_MAX_AXES 4

favor_status favor_fwd_rotary(const void* q, const int64_t* q_strides, void* q_out, const int64_t* q_out_strides,
                              const void* k, const int64_t* k_strides, void* k_out, const int64_t* k_out_strides,
                              int B, int Hq, int Hk, int L, int d,
                              const int32_t* pos, int pos_B, int n_axes, const int* sections,
                              const uint64_t* table, favor_pairing pairing, favor_dtype dt, void* stream);

/* favor_bwd_rotary — the gradients of q and k for those of q_out and k_out:
 * the rotation by the opposite angles; arguments as above. */
favor_status favor_bwd_rotary(const void* dq_out, const int64_t* dq_out_strides, void* dq, const int64_t* dq_strides,
                              const void* dk_out, const int64_t* dk_out_strides, void* dk, const int64_t* dk_strides,
                              int B, int Hq, int Hk, int L, int d,
                              const int32_t* pos, int pos_B, int n_axes, const int* sections,
                              const uint64_t* table, favor_pairing pairing, favor_dtype dt, void* stream);

/*
 * favor_fwd_qk_norm_rotary — root-mean-square norm of each head's queries and
 * keys and their rotation by positions, in one pass over the rows:
 *   y = R(pos) (x w / sqrt(mean x^2 + eps))
 * with w = q_weight for q and k_weight for k (fp32 [d], NULL for 1) and the
 * rotation R of favor_fwd_rotary, whose arguments (pos, sections, table,
 * pairing) and limits these are.  eps > 0 and finite (an eps, squares and means
 * below fp32's normal numbers, 2^-126, have fewer bits).  The normed row is kept
 * in fp32 and rounded once, after the rotation.  q_out may be q, k_out may be k.
 * A row whose sum of squares leaves fp32 (values beyond about 2^60) is NaN, as
 * one with infinities or NaN is; rows do not touch one another.
 * Supported: d <= 512, besides the limits of favor_fwd_rotary.
 */
favor_status favor_fwd_qk_norm_rotary(const void* q, const int64_t* q_strides, void* q_out,
                                      const int64_t* q_out_strides, const void* k, const int64_t* k_strides,
                                      void* k_out, const int64_t* k_out_strides, const float* q_weight,
                                      const float* k_weight, float eps, int B, int Hq, int Hk, int L, int d,
                                      const int32_t* pos, int pos_B, int n_axes, const int* sections,
                                      const uint64_t* table, favor_pairing pairing, favor_dtype dt, void* stream);

/*
 * favor_bwd_qk_norm_rotary — its gradients for dy = dL/dy (dq_out, dk_out);
 * with z = R(pos)^T dy, r = 1 / sqrt(mean x^2 + eps) (recomputed from x) and
 * xh = x r:
 *   dx = r (z w - xh mean(z w xh)),  dw = sum over the rows of z xh
 * dq_weight, dk_weight: fp32 [d], overwritten, each NULL if not wanted; summed
 * over all rows of q (of k) in a fixed order.  dq may be dq_out or q, dk may be
 * dk_out or k.  k, dk_out and dk may all be NULL (no keys; k_weight and
 * dk_weight are then ignored).
 * Workspace of favor_bwd_qk_norm_rotary_workspace_bytes(...) bytes, 256-byte
 * aligned (0 bytes, and NULL allowed, where neither dq_weight nor dk_weight is
 * wanted); calls that share one must be ordered on one stream.
 */
favor_status favor_bwd_qk_norm_rotary(const void* q, const int64_t* q_strides, const void* dq_out,
                                      const int64_t* dq_out_strides, void* dq, const int64_t* dq_strides,
                                      const void* k, const int64_t* k_strides, const void* dk_out,
                                      const int64_t* dk_out_strides, void* dk, const int64_t* dk_strides,
                                      const float* q_weight, const float* k_weight, float* dq_weight,
                                      float* dk_weight, float eps, int B, int Hq, int Hk, int L, int d,
                                      const int32_t* pos, int pos_B, int n_axes, const int* sections,
                                      const uint64_t* table, favor_pairing pairing, favor_dtype dt, void* workspace,
                                      size_t ws_bytes, void* stream);
/* The size follows the current device's number of SMs: asked for with the
 * device current that the call runs on.  0 for arguments outside the supported
 * shapes; Hk = 0: no keys. */
size_t favor_bwd_qk_norm_rotary_workspace_bytes(int B, int Hq, int Hk, int L, int d, favor_dtype dt);

/*
 * favor_fwd_decay_attention — causal linear attention whose memory fades by
 * one factor per head and token, l = exp(g_h):
 *   S_t = l S_{t-1} + k_t v_t^T,  S_{-1} = S0,  o_t = scale S_t^T q_t
 *   (o_t = scale sum_{s<=t} l^(t-s) (q_t . k_s) v_s + scale l^(t+1) S0^T q_t)
 * with neither a feature map nor a normaliser: the heads' outputs are normed
 * by the layer (favor_fwd_layer_norm).
 *  - g: device fp32 [H], the logarithms of the decays, <= 0 (not checked).  0 is
 *    plain causal linear attention; with minus infinity a token sees itself
 *    alone.  (Positive g: tokens, zeros too, are weighted by powers of l that
 *    reach over a run of tokens, at most the sequence.  The values are the
 *    formula's while l^L, its products with what the tensors hold and the states
 *    stay finite in fp32.)  The decays are constants of the heads and have no
 *    gradient.
 *  - lengths: device int32 [B], the tokens of each sequence, or NULL for L
 *    each; values are clamped to [0, L].  Rows of q, k and v at and behind a
 *    sequence's end are not used, whatever they hold, and its rows of o there
 *    are 0.
 *  - S0, ST: fp32 [B, H, d, d] contiguous (first index the key's channel, second
 *    the value's), S0 NULL for zeros, ST NULL if not wanted: the state after
 *    each sequence's last token (S0 where it has none).  ST may be S0.
 *  - workspace: favor_decay_attention_workspace_bytes(...) bytes, 256-byte
 *    aligned (NULL allowed where that is 0); calls that share one must be
 *    ordered on one stream.
 *  - dev_status: a bounded wait that ran out is reported there
 *    (FAVOR_ERR_TIMEOUT).
 * Infinities and NaN in a token of k or v reach its own and later rows of its
 * head, in a token of q its own row; on the tensor cores (bf16, below) rows and
 * states behind it may be NaN where the formula has an infinity.  No output may
 * overlap an input (but ST may be S0).
 * States and sums are fp32, and with fp32 tensors everything else is, too.
 * With bf16 tensors ST is formed from factors with all of
 * fp32's bits, while a term of o is rounded to bf16 once beside o's own rounding:
 * its weight where query and key are in one chunk of 128 tokens, its key where
 * they are not (tensors whose rows are no whole 16-byte pieces, or with a
 * stride of 0, S0 or dST off 16 bytes and forward calls of L <= 16 are taken as fp32
 * ones, on the CUDA cores: several times slower where sequences are long).  For
 * outputs off by their own rounding alone the same values are passed as fp32
 * tensors.
 * Supported: d <= 128, B H < 2^20, L <= 2^30.
 */
favor_status favor_fwd_decay_attention(const void* q, const int64_t* q_strides, const void* k,
                                       const int64_t* k_strides, const void* v, const int64_t* v_strides, void* o,
                                       const int64_t* o_strides, const float* g, const int32_t* lengths,
                                       const float* S0, float* ST, float scale, int B, int H, int L, int d,
                                       favor_dtype dt, void* workspace, size_t ws_bytes, int32_t* dev_status,
                                       void* stream);

/*
 * favor_bwd_decay_attention — its gradients for do = dL/do and dST = dL/dST
 * (fp32 [B, H, d, d], NULL for zeros):
 *   R_t = l R_{t+1} + scale q_t do_t^T  (R behind the last token: dST, unfaded)
 *   dq_t = scale S_t do_t,  dk_t = R_t v_t,  dv_t = R_t^T k_t,  dS0 = l R_0
 * from the forward call's q, k, v, g, lengths, scale and S0 (S_t is formed
 * again).  dS0: fp32 [B, H, d, d], NULL if not wanted; dS0 may be dST.  Rows of
 * dq, dk and dv at and behind a sequence's end are 0.  No other output may
 * overlap an input or another output.  Workspace and dev_status as above, with
 * `backward` set in the size.
 */
favor_status favor_bwd_decay_attention(const void* q, const int64_t* q_strides, const void* k,
                                       const int64_t* k_strides, const void* v, const int64_t* v_strides,
                                       const void* d_o, const int64_t* do_strides, void* dq,
                                       const int64_t* dq_strides, void* dk, const int64_t* dk_strides, void* dv,
                                       const int64_t* dv_strides, const float* g, const int32_t* lengths,
                                       const float* S0, const float* dST, float* dS0, float scale, int B, int H,
                                       int L, int d, favor_dtype dt, void* workspace, size_t ws_bytes,
                                       int32_t* dev_status, void* stream);
/* The size follows the current device's number of SMs: asked for with the
 * device current that the call runs on.  0: none is needed, or the arguments
 * are outside the supported shapes. */
size_t favor_decay_attention_workspace_bytes(int B, int H, int L, int d, favor_dtype dt, int backward);

/*
 * favor_decay_attention_step — one token of each sequence:
 *   new_state = l state + k v^T,  o = scale new_state^T q
 * q, k, v, o: [B, H, d] with d fastest and, each, an int64_t[2] of the element
 * strides of B and H, or NULL for a contiguous tensor.  state, new_state: fp32
 * [B, H, d, d]; new_state may be state.  o may not overlap anything else.
 * Everything is fp32 but the rounding of o: row t of the forward call, given the
 * state of the tokens before it, but for that call's roundings.
 * Supported: d <= 128, B H < 2^20.
 */
favor_status favor_decay_attention_step(const void* q, const int64_t* q_strides, const void* k,
                                        const int64_t* k_strides, const void* v, const int64_t* v_strides, void* o,
                                        const int64_t* o_strides, const float* g, const float* state,
                                        float* new_state, float scale, int B, int H, int d, favor_dtype dt,
                                        void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FAVOR_OPS_H_ */
