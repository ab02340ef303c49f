// Arguments and launchers of the MXFP4 quantise / dequantise kernels.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qg {

struct MxQuantArgs {
  const void* X;        // T x K (or T x 2K: gate, up)
  const int32_t* rows;  // source row of each output row, or null
  char* Q;              // codes, two a byte
  char* S;              // E8M0 scales
  void* Y;              // dequantise: the values
  int64_t ldx;          // elements (X, Y)
  int64_t ldq, lds;     // bytes
  int64_t units;        // rows * cpr
  int32_t T, K;
  int32_t cpr;          // units (8 consecutive elements) per row
  int32_t x_type;       // DType of X / Y
  int32_t swiglu;
};

hipError_t launch_mx_quantize(const MxQuantArgs& a, int cus, hipStream_t s);
hipError_t launch_mx_dequantize(const MxQuantArgs& a, int cus, hipStream_t s);
// Workgroups of a launch that takes `per_lane` units per lane (one at least, so
// that at one they bound what the engine may launch).
int64_t mx_quant_blocks(int64_t units, int per_lane);

}  // namespace qg
