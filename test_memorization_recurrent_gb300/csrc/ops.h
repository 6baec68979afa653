// ops.h -- internal interface between the C-ABI host layer and the kernels of the
// layer operators.
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace atlas {

constexpr int kSMs = 152;  // of a GB300

struct NormArgs {
  const void* x;    // backward: h
  const void* r;    // backward: dh
  const void* w;
  const void* dy;
  void* y;          // backward: dx
  void* r_out;
  float* scale;
  float* dw;
  float* part;      // backward: [blocks, d] partial sums of dw
  long rows, sx, sr, sy;
  int d, dt, rt, wt, ot, group;
  float eps, inv_d;  // 1 / d, set at the launch
  int ng, gshift;    // groups of a row, log2 of a group that is a power of two; set at the launch
  int wide;         // every pointer and stride allows 8-element accesses
};
int norm_forward_launch(const NormArgs& a, cudaStream_t st);
size_t norm_backward_workspace(const NormArgs& a);
int norm_backward_launch(const NormArgs& a, cudaStream_t st);

// Sequences and states, as described in atlas_ops.h.
struct SeqArgs {
  const int* start;
  const int* slot;
  const uint8_t* carry;
  int* status;
  int B, L, n_slots;
};

struct ConvArgs {
  SeqArgs s;
  const void* x;
  const void* w;
  const void* bias;
  void* y;
  const void* st_in;
  void* st_out;
  const void* dy;
  float* dstate;
  void* dx;
  float* dw;
  float* dbias;
  void* ws;
  int C, W, act, dt, wt, hd;
  long xb, xt, yb, yt, yh;
  int wide;  // x, y and the states allow accesses of four elements (backward: 16 bytes)
};
int conv_forward_launch(const ConvArgs& a, cudaStream_t st);
size_t conv_backward_workspace(const ConvArgs& a);
int conv_backward_launch(const ConvArgs& a, cudaStream_t st);

struct ScanArgs {
  SeqArgs s;
  const void* x;
  const void* dt;
  const void* Bm;
  const void* Cm;
  const void* z;
  const float* A;
  const float* Dk;
  const float* bias;
  void* y;
  const float* h_in;
  float* h_out;
  void* ws;
  int D, N, G, type, softplus;
  long xb, xt, tb, tt, zb, zt, yb, yt, bb, bt, cb, ct;
  int wide;    // x, dt, z, y allow 16-byte accesses
  int wide_n;  // and so do B and C
  // backward
  const void* dy;
  float* dh;
  void* dx;
  void* ddt;
  void* dB;
  void* dC;
  void* dz;
  float* dA;
  float* dD;
  float* dbias;
};
size_t scan_workspace(const ScanArgs& a);
int scan_forward_launch(const ScanArgs& a, cudaStream_t st);
size_t scan_backward_workspace(const ScanArgs& a);
int scan_backward_launch(const ScanArgs& a, cudaStream_t st);

}  // namespace atlas
