// Products of MXFP4 rows x MXFP4 matrices.
#include "product_dev.h"

namespace mc {

int launch_product_fp4(const ProductArgs& a, hipStream_t s) { return launch_by_size<MC_MXFP4, MC_MXFP4>(a, s); }

}  // namespace mc
