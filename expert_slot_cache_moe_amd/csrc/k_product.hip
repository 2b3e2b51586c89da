// Which form of the products (k_product.inc) a call takes.
#include "k_product.inc"

namespace moe {
namespace product_detail {
hipError_t launch_bf16(const ProductParams &p, int form, hipStream_t s);
hipError_t launch_e2m1(const ProductParams &p, int form, hipStream_t s);
hipError_t launch_mxfp4(const ProductParams &p, int form, hipStream_t s);

namespace {
// The form by the mean number of places of a matrix.
int form_of(const ProductParams &p) {
    if (p.k < kTileMinK) return 1;
    const int64_t groups = p.offsets == nullptr ? 1 : std::min(p.G, p.R);
    const int64_t mean = p.R / groups;
    return mean >= 1024 ? 6 : mean >= 64 ? 5 : mean >= 6 ? 4 : 1;
}
}  // namespace
}  // namespace product_detail

using namespace product_detail;

bool product_launchable(const ProductParams &p) {
    const int64_t tiles = (p.n + kTile - 1) / kTile;
    return tiles * max_pieces(p, kTile) < (1ll << 32) / (8 * kWave);
}

hipError_t launch_product(const ProductParams &p, hipStream_t s) {
    const int form = form_of(p);
    switch (p.fmt) {
        case MOE_FMT_BF16: return launch_bf16(p, form, s);
        case MOE_FMT_E2M1: return launch_e2m1(p, form, s);
        default: return launch_mxfp4(p, form, s);
    }
}

}  // namespace moe
