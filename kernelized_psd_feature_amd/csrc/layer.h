// Arguments and launchers of the rotary and layer norm kernels.
#pragma once

#include <hip/hip_runtime.h>

namespace kata {

struct RotaryArgs {
  const void *q, *k;                       // k may be null (Hk = 0)
  void *oq, *ok;
  const double* rates;                     // [rot / 2] radians a token
  const void* positions;                   // int32 or int64, or null: offset + t
  const int* axes;                         // [rot / 2] the axis of each pair, or null: one axis
  long long pos_a, pos_b, pos_t, offset;
  long long sq[3], sk[3], soq[3], sok[3];  // element strides of (b, t, h)
  int B, T, H, Hk, D, rot, pos64, inverse, n_axes;
  float magnitude;
  int TT;                                  // tokens of a workgroup
};
// aligned: every pointer and stride is a multiple of 16 bytes.
hipError_t launch_rotary(RotaryArgs& a, bool bf16, bool aligned, bool interleaved, hipStream_t st);

// The norm of every head of q and k, and their turn; backward: of the gradients dq, dk back to the inputs.
struct QkNormArgs {
  const void *q, *k, *dq, *dk, *wq, *wk;   // k may be null (Hk = 0), the weights too: ones
  void *oq, *ok;                           // outputs (backward: the inputs' gradients)
  void *dwq, *dwk;                         // null: not wanted
  float* part;                             // backward workspace [blocks][2][D]
  const double* rates;
  const void* positions;
  const int* axes;
  long long pos_a, pos_b, pos_t, offset;
  long long sq[3], sk[3], soq[3], sok[3], sdq[3], sdk[3];
  int B, T, H, Hk, D, rot, pos64, inverse, n_axes, w_bf16;
  float magnitude, eps, count;             // count: what a row's sum of squares is divided by
  int TT, R, blocks;                       // tokens of a workgroup, lanes of a row, workgroups (backward)
};
// aligned: every pointer and stride is a multiple of 16 bytes.
hipError_t launch_qk_norm(QkNormArgs& a, bool bf16, bool aligned, bool interleaved, bool backward, hipStream_t st);

struct NormArgs {
  const void *x, *dy, *w, *b;              // w, b may be null: ones, zeros
  void *y, *dx, *dw, *db;                  // any may be null in the backward pass
  float *mean, *rstd;                      // [rows]; null in a forward pass that keeps none
  float* part;                             // backward workspace [blocks][2][N]
  long long rows, sx, sdy, sy, sdx;        // row strides in elements
  int N, w_bf16, blocks;
  float eps;
};
hipError_t launch_norm_fwd(NormArgs& a, bool bf16, bool aligned, hipStream_t st);
hipError_t launch_norm_bwd(NormArgs& a, bool bf16, bool aligned, hipStream_t st);
}  // namespace kata
