// Products of bf16 rows x bf16 matrices.
#include "product_dev.h"

namespace mc {

int launch_product_bf16(const ProductArgs& a, hipStream_t s) { return launch_by_size<MC_BF16, MC_BF16>(a, s); }

}  // namespace mc
