// Arguments and launchers of the int8 quantise / dequantise kernels.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qg {

// 64 bytes, as the MXFP4 kernels' arguments: what a launch costs the host grows with them.
struct I8QuantArgs {
  void* X;              // values: T x K (or T x 2K: gate, up), R x K for the way back
  const int32_t* rows;  // source row of each output row, or null
  char* Q;              // codes
  float* S;             // a scale per row
  int32_t ldx;          // elements
  int32_t ldq, lds;     // bytes, elements
  int32_t T, K;
  int32_t R;            // rows of Q and S
  int32_t cpr;          // units (8 consecutive elements) per row
};

constexpr int64_t kI8QuantMaxK = 65536;  // a row stays in the registers of 1024 lanes

// x_type: DType of X; swiglu: gate and up instead of values
hipError_t launch_i8_quantize(const I8QuantArgs& a, int x_type, bool swiglu, hipStream_t s);
hipError_t launch_i8_dequantize(const I8QuantArgs& a, int x_type, int cus, hipStream_t s);

}  // namespace qg
