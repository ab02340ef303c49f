// Arguments and launchers of the kernels around an expert block's products:
// choosing experts, sorting the choices by expert, putting the results together.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qg {

constexpr int kRouteMaxExperts = 1024, kRouteMaxK = 32, kRouteMaxGroups = 64;
constexpr int kGroupMaxExperts = 1023;  // what a grouped product takes
constexpr int64_t kGroupMaxEntries = int64_t(1) << 30;
constexpr int64_t kGroupAlone = 8192;  // entries that one workgroup sorts without a workspace

// (each 64 bytes at most, where they can be: what a launch costs the host grows with its arguments)
struct RouteArgs {
  const void* X;      // logits, T x E
  const float* bias;  // E, or null
  int32_t* ids;       // T x K
  float* W;           // T x K
  int32_t T;
  int32_t ldx, ldi, ldw;  // elements
  float scale;
  int16_t per;            // experts per group
  int8_t K;               // experts per token
  int8_t groups, kept;    // groups, groups kept
  int8_t shift;           // log2 of the lanes that take one group
  int8_t flags;           // RouteFlag
};
enum RouteFlag : int8_t { ROUTE_SIGMOID = 1, ROUTE_BEST2 = 2, ROUTE_RENORM = 4 };

struct GroupArgs {
  const int32_t* ids;  // T x K
  int32_t* offsets;    // E + 1
  int32_t* rows;       // T * K
  int32_t* back;       // T * K
  int32_t* counts;     // chunks x E (more than one chunk)
  int32_t n, K, ldi;   // T * K, K, pitch
  int32_t E;
  int32_t chunk, chunks;  // entries per workgroup, workgroups
};

struct CombineArgs {
  const void* R;        // results, N x H
  const int32_t* back;  // T x K
  const float* W;       // T x K
  void* Y;              // T x H
  int32_t ldr, ldw, ldy;  // elements
  int32_t T, K, N, H;
};
struct CombineAddArgs : CombineArgs {
  const void* C;  // T x H
  int32_t ldc;
  int32_t c_type;
  float beta;
};

hipError_t launch_route(const RouteArgs& a, int x_type, int cus, hipStream_t s);
// Entries of one workgroup's range and the number of ranges, for n entries.
// (workspace: the caller has one for the table of counts)
void group_chunks(int64_t n, bool workspace, int* chunk, int* chunks);
hipError_t launch_group(const GroupArgs& a, hipStream_t s);
// C is read where a.beta is not zero.
hipError_t launch_combine(const CombineAddArgs& a, int r_type, int y_type, hipStream_t s);

}  // namespace qg
