// Internal interface of the gated delta rule's kernels (delta_*.hip) and its
// host side (delta_api.cpp).
//
// The recurrence, per sequence and value head (state S, V x K, one row per
// value channel; alpha_t = e^{g_t}):
//   u_t = beta_t (v_t - alpha_t S_{t-1} k_t),  S_t = alpha_t S_{t-1} + u_t k_t^T,
//   o_t = scale S_t q_t.
// Over a chunk of kDeltaC tokens, with G_t the running sum of g inside the
// chunk and S the state entering it, the corrections u solve a unit lower
// triangular system:
//   (I + L) u = beta v - beta e^G (k S^T),   L_ts = beta_t e^{G_t - G_s} k_t.k_s  (s < t)
//   o_t = scale e^{G_t} S q_t + sum_{s<=t} P_ts u_s,  P_ts = scale e^{G_t - G_s} q_t.k_s
//   S' = e^{G_C} S + sum_t e^{G_C - G_t} u_t k_t^T
// T = (I + L)^-1 and P do not depend on the state, so one kernel forms them for
// every chunk in parallel (delta_prep.hip) and a second walks the chunks in
// order with the state in registers (delta_pass.hip).
#pragma once
#include "ssm_internal.h"

namespace ssm {

constexpr int kDeltaC = 64;        // tokens per chunk
constexpr int kDeltaMaxK = 128;    // key channels the kernels hold
constexpr int kDeltaFrag = 1024;   // bytes of an operand fragment: 64 lanes x 8 bf16
constexpr int kDeltaTri = 6;       // fragments of a triangular 64 x 64 operand (of 8)
// floats of a (chunk, head)'s coefficients, in rows of 64: beta; beta e^G rk;
// scale e^G rq; e^{G_C - G} rk; [e^{G_C}]; rk; rq; e^G; G in 64 bits (2 rows);
// e^{G_C - G}
constexpr int kDeltaSc = 11 * kDeltaC;
enum DeltaScRow { kScBeta = 0, kScR, kScO, kScU, kScGamma, kScRk, kScRq, kScEg, kScG, kScEl = kScG + 2 };

// bf16 parts that stand for a 32-bit operand of a matrix product: the inputs (bf16
// inputs are exact in one), and everything formed from them, T, P, S, u and the
// gradients, which keep all 24 bits, as sums and states are held in 32.  Two parts of
// the operands that only reach o left it 3e-5 of its largest value off instead of 2e-7:
// small outputs of a bf16 o were then off by more than its own rounding.
template <typename IN>
struct DeltaParts;
struct bf16s;
template <>
struct DeltaParts<bf16s> {
  static constexpr int in = 1, state = 3;
};
template <>
struct DeltaParts<float> {
  static constexpr int in = 3, state = 3;
};

struct DeltaArgs {
  const void *q, *k, *v;     // rows of a token: (hk, K), (hk, K), (h, V); strides in elements
  long q_stride, k_stride, v_stride;
  const float *g, *beta;     // (tokens, h)
  const int32_t* cu;         // (nseq + 1) token offsets, or null: nseq sequences of seqlen tokens
  const float* state_in;     // (nseq, h, V, K) or null
  float* state_out;          // or null
  void* o;                   // (tokens, h, V)
  int nseq, seqlen, hk, h, K, V;
  long tokens;
  long slots;                // chunk slots over all sequences
  float scale, eps;
  int qk_norm, vec_qk, vec_state;
  // workspace (operand fragments and coefficients, written by the prep kernel)
  unsigned char *kf, *qf, *ktf, *tf, *pf;
  unsigned char *qtf, *ttf, *ptf;  // backward only
  float* sc;
  // backward
  // per (slot, head), K and V padded to delta_kp and delta_vp with zeros:
  float *s_chunk, *ds_chunk;       // (K, V) state entering / state gradient leaving the chunk
  float *u_chunk, *dr_chunk;       // (64, V)
  const void* dout;                // (tokens, h, V)
  const float* dstate_out;         // (nseq, h, V, K) or null
  void *dq, *dk, *dv;              // dense, or null
  float *dg, *dbeta, *dstate_in;   // or null
  float *dq_part, *dk_part;        // (tokens, h, delta_kp) where heads share q and k
};

struct DeltaLaunch {
  DeltaArgs a;
  int in_dtype, o_dtype, grad_dtype;
};

inline int delta_kp(int K) { return K <= 64 ? 64 : 128; }
__host__ __device__ inline int delta_vp(int V) { return (V + 31) / 32 * 32; }
// Value channels per workgroup of the walks, in slices of 16: 32 once that still leaves
// every CU a workgroup (the operands of T, P and the keys are then read half as often
// and a chunk's three exchanges serve twice the work), else 16.  With 256 workgroups or
// more at 32: packed call 480 us against 609, training walks 120 and 154 against 140
// and 179; with fewer: prompt 295 us at 16 against 443.
inline int delta_nv(long groups, int V) { return groups * ((V + 31) / 32) >= 256 && V > 16 ? 2 : 1; }
// Workgroups per (sequence, head), and of a walk (backward: the kept tiles are padded,
// the slices cover delta_vp channels)
inline long delta_slices(long groups, int V, bool backward) {
  const int width = 16 * delta_nv(groups, V);
  return ((backward ? delta_vp(V) : V) + width - 1) / width;
}
inline long delta_walk_blocks(long groups, int V, bool backward) {
  return (groups + 7) / 8 * 8 * delta_slices(groups, V, backward);
}
hipError_t launch_delta_prep(const DeltaLaunch& l, bool backward, hipStream_t s);
// The forward walk; save: also writes s_chunk and u_chunk, and no output.
hipError_t launch_delta_pass(const DeltaLaunch& l, bool save, hipStream_t s);
hipError_t launch_delta_reverse(const DeltaLaunch& l, hipStream_t s);
hipError_t launch_delta_grads(const DeltaLaunch& l, hipStream_t s);

struct DeltaStepArgs {
  const void *q, *k, *v;
  long q_stride, k_stride, v_stride;
  const float *g, *beta;
  float* state;
  void* o;
  int batch, hk, h, K, V, o_bf16;
  float scale, eps;
  int qk_norm;
  int vec;  // K % 8 == 0 and every row 16-byte aligned
};
hipError_t launch_delta_step(const DeltaStepArgs& a, int in_dtype, hipStream_t s);

// ---- block norm -----------------------------------------------------------
struct NormArgs {
  const void *x, *z, *res;
  const float *norm_w, *scale, *out_w;
  void *out, *res_out;
  long rows;      // rows the kernel normalises: rows of the call x groups
  int n;          // their length
  int groups;     // groups per row of the call (1 unless a pure grouped norm)
  int w_period;   // weights are indexed by (row % w_period) * n + i
  long x_stride, z_stride;  // between rows of the call, in elements
  int x_dtype, res_dtype, out_dtype;
  float eps;
  int gate_first;
  int vec;        // elements per access: 8, 4 or 1
  // backward
  const void *dout, *dres;
  int dout_dtype, dres_dtype, grad_dtype;
  void *dx, *dz, *dresidual;
  float *dnorm_w, *dscale, *dout_w;
  float* part;    // (parts, 3, n) partial column sums, part p of weight row p % w_period
  int parts;
};
hipError_t launch_norm_fwd(const NormArgs& a, hipStream_t s);
hipError_t launch_norm_bwd(const NormArgs& a, hipStream_t s);
int norm_bwd_parts(long rows, int n, int period);
constexpr int kNormMax = 16384;  // longest normalised row
// most weight rows of the backward: workgroups and partial rows are whole turns round
// them, which keeps both and the steps between a weight row's partials in 31 bits
constexpr int kNormMaxPeriod = 1 << 22;

}  // namespace ssm
