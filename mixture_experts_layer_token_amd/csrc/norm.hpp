// Launches of the norm of rows and of the norm and clipping of gradients; arguments are validated by the entry points.
#pragma once

#include "common.hpp"

namespace moe {

struct NormArgs {
  int rows, H, rms;
  float eps;
  const void* x;
  long long ldx, ldy;  // elements between rows of x, and of y or dy; dx and add are contiguous
  const void* weight;  // or null: ones
  const void* bias;    // or null: zeros
  int par_bf16;        // type of weight and bias and of their gradients
  void* y;
  float* stats;  // [rows][2] = mean (RMS: 0), 1 / sqrt(variance + eps); forward: or null
  // gradient
  const void* dy;
  const void* add;  // or null
  void* dx;
  void* dweight;  // or null
  void* dbias;    // or null
  float* part;    // [parts][2][H]: sums of dy xh and of dy over a part of the rows; or null with neither
  float* sums;    // [rows][2], of rows too long for the registers
};

int launch_norm(const NormArgs& a, int dt, hipStream_t s);
int launch_norm_grad(const NormArgs& a, int dt, hipStream_t s);
int norm_parts(int rows, int H);            // parts of the rows whose sums are added up in the end
bool norm_long(int H);                      // rows too long for the registers
inline size_t norm_workspace(int rows, int H) {
  return ((size_t)norm_parts(rows, H) * 2 * H * 4 + (norm_long(H) ? (size_t)rows * 8 : 0) + 255) / 256 * 256;
}

int launch_grad_norm(const moe_tensor* t, int n, int clip, float max_norm, float* norm, double* part, hipStream_t s);
size_t grad_norm_workspace(int n);

}  // namespace moe
