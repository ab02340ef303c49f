// Explicit instantiations of the MXFP4 skinny kernels listed in qg_kernel_list.inc.
#include "qg_mx_skinny.hpp"

namespace qg {
#define QG_TILE_BF16(BM, BN, WM, WN, ST, RB)
#define QG_TILE_BF16_BIG(BM, BN, WM, WN, ST, RB)
#define QG_TILE_F16(BM, BN, WM, WN, ST, RB)
#define QG_TILE_I8(BM, BN, WM, WN, ST, RB)
#define QG_SKINNY_BF16(BN, NW, MT, DP, BB, NS)
#define QG_SKINNY_F16(BN, NW, MT, DP, BB, NS)
#define QG_SKINNY_I8(BN, NW, MT, DP, BB, NS)
#define QG_W4(MT, BN, WN, WK, ST)
#define QG_F8(BM, BN, WM, WN, ST)
#define QG_MX(BM, BN, WM, WN, ST, RB, WK)
#define QG_MX_SKINNY(BN, NW, MT, DP, SH) \
  template hipError_t launch_mx_skinny<MxSkinnyCfg<BN, NW, MT, DP, SH>>(const Args&, int, hipStream_t);
#include "qg_kernel_list.inc"
}  // namespace qg
