// Arguments and launchers of the rotary and layer norm kernels.
#pragma once

#include <hip/hip_runtime.h>

namespace kata {

struct RotaryArgs {
  const void *q, *k;                       // k may be null (Hk = 0)
  void *oq, *ok;
  const double* rates;                     // [rot / 2] radians a token
  const void* positions;                   // int32 or int64, or null: offset + t
  long long pos_b, pos_t, offset;
  long long sq[3], sk[3], soq[3], sok[3];  // element strides of (b, t, h)
  int B, T, H, Hk, D, rot, pos64, inverse;
  float magnitude;
  int TT;                                  // tokens of a workgroup
};
// aligned: every pointer and stride is a multiple of 16 bytes.
hipError_t launch_rotary(RotaryArgs& a, bool bf16, bool aligned, bool interleaved, hipStream_t st);

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
