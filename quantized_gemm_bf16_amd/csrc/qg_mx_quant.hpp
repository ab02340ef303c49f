// Arguments and launchers of the MXFP4 quantise / dequantise kernels.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qg {

// 64 bytes: what a launch costs the host grows with its arguments (an empty
// kernel 1.3 us, with 256 bytes of them 3.4).
struct MxQuantArgs {
  void* X;              // values: T x K (or T x 2K: gate, up), R x K for the way back
  const int32_t* rows;  // source row of each output row, or null
  char* Q;              // codes, two a byte
  char* S;              // E8M0 scales
  int32_t ldx;          // elements
  int32_t ldq, lds;     // bytes
  int32_t T, K;
  int32_t R;            // rows of Q and S
  int32_t cpr;          // units (8 consecutive elements) per row
};

// x_type: DType of X; swiglu: gate and up instead of values
hipError_t launch_mx_quantize(const MxQuantArgs& a, int x_type, bool swiglu, int cus, hipStream_t s);
hipError_t launch_mx_dequantize(const MxQuantArgs& a, int x_type, int cus, hipStream_t s);
// Workgroups of a launch that takes `per_lane` units per lane (one at least, so
// that at one they bound what the engine may launch).
int64_t mx_quant_blocks(int64_t units, int per_lane);

}  // namespace qg
