// Launches of the row-wise operators beside the grouped products (8-bit quantization, SwiGLU gate, gradient
// of the combine); arguments are validated by the entry points.
#pragma once

#include "common.hpp"

namespace moe {

int launch_quant_rows(const void* x, int xdt, int rows, int K, int act, const int32_t* n_rows, int8_t* q,
                      float* scale, hipStream_t s);
// dh null: h = SiLU(g) u; else dgu, and h unless it is null
int launch_swiglu(const void* gu, const void* dh, int dt, int rows, int I, const int32_t* n_rows, void* dgu, void* h,
                  hipStream_t s);
int launch_combine_grad(const void* dout, int odt, const float* y, const float* w, const int32_t* inv, int T, int k,
                        int H, void* dy, int ydt, float* dw, const int32_t* ids, int E, float* dlogits,
                        hipStream_t s);

}  // namespace moe
