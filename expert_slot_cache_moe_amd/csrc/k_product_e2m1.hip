// The products over E2M1 matrices (k_product.inc).
#include "k_product.inc"

namespace moe {
namespace product_detail {
hipError_t launch_e2m1(const ProductParams &p, int form, hipStream_t s) {
    return launch_format<MOE_FMT_E2M1>(p, form, s);
}
}  // namespace product_detail
}  // namespace moe
