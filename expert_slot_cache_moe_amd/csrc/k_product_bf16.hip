// The products over bf16 matrices (k_product.inc).
#include "k_product.inc"

namespace moe {
namespace product_detail {
hipError_t launch_bf16(const ProductParams &p, int form, hipStream_t s) {
    return launch_format<MOE_FMT_BF16>(p, form, s);
}
}  // namespace product_detail
}  // namespace moe
