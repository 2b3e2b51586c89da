// Which form of the products (k_product.inc) a call takes.
#include "k_product.inc"

namespace moe {
namespace product_detail {
hipError_t launch_bf16(const ProductParams &p, int form, hipStream_t s);
hipError_t launch_e2m1(const ProductParams &p, int form, hipStream_t s);
hipError_t launch_mxfp4(const ProductParams &p, int form, hipStream_t s);

namespace {

// Blocks that are to be found, were the places spread evenly over the groups.
int64_t even_blocks(const ProductParams &p, int form) {
    const int64_t groups = p.offsets == nullptr ? 1 : std::min(p.G, p.R), length = form_places(form);
    return groups * ((p.R + groups * length - 1) / (groups * length)) * form_grid(p, form).tiles;
}

// Up to so many blocks of the split form: it has one launch's latency, where
// a tile passes all of k stage by stage (dense bf16, us, split / 32 places:
// 256 blocks of k 2048 6.3 / 12.1, 512 10.3 / 12.1, 1024 18.5 / 12.2; 512 of k
// 4096 17.6 / 29.9, 1024 33.1 / 30.1; 512 of k 1024 6.8 / 8.2, 1024 11.5 /
// 8.3).  With rows of x that are no whole vectors of eight fewer (k 1061, 132
// blocks 9.3 / 12.4, 264 14.3 / 12.5), with 4-bit weights more (MXFP4, k 1056,
// 792 blocks 8.6 / 10.5; k 1024, 1024 blocks 9.5 / 8.3).
constexpr int64_t kSplitBlocks = 512, kSplitBlocksCut = 192, kSplitBlocksCodes = 800;
// The mean places of a matrix from which a tile of 64, 128, 256 places pays
// (bf16, 64 matrices of 2048 x 2048, us at 32 / 64 / 128 / 256 places: mean 4
// 122 117 122 137, 32 128 122 129 144, 64 191 127 142 151, 96 254 153 141
// 186, 192 439 254 177 192, 256 574 324 226 205; 160 of 512 x 1024: mean 8 27
// 28 32 59, 16 29 29 33 60, 64 63 42 40 68, 96 81 55 44 70, 256 163 110 84
// 82), and for 4 bits one of 64 (E2M1, 64 of 2048 x 2048, 32 / 64 places: mean
// 32 53 60, 48 68 64, 96 127 101).
constexpr int64_t kMean64 = 12, kMean128 = 72, kMean256 = 224, kMeanCodes64 = 40;
// A larger tile is taken only where there is a block for each of the 256 CUs
// (dense 4096 x 4096, us at 64 / 128 / 256 places: 512 rows 42 45 106, 1024 62
// 48 106, 2048 140 79 107, 4096 284 157 136), or for half of them where each
// piece more reads a matrix of its own again (32 / 64 places, 128 and 132
// blocks of 64: 8 matrices of 1024 x 2048 27.7 / 19.3, 33 of 138 x 2656 33.6 /
// 25.9, 66 blocks 22.5 / 24.4; a dense 1024 x 1024 of 128 blocks 8.7 / 11.3;
// MXFP4, 24 of 515 x 1056, 240 blocks 19.0 / 22.0).
constexpr int64_t kEnoughBlocks = 256, kEnoughBlocksGrouped = 120;

int form_of(const ProductParams &p) {
    const bool wide = p.fmt == MOE_FMT_BF16;
    if (p.k < (wide ? kTileMinK : kCodesMinK) || p.n / (p.act == MOE_ACT_SWIGLU ? 2 : 1) < kTileMinCols) return kSplit;
    const bool cut = p.k % 8 != 0 || p.x_stride % 8 != 0;
    if (even_blocks(p, kSplit) <= (!wide ? kSplitBlocksCodes : cut ? kSplitBlocksCut : kSplitBlocks)) return kSplit;
    const int64_t groups = p.offsets == nullptr ? 1 : std::min(p.G, p.R), mean = p.R / groups;
    int form;
    if (wide)
        form = mean >= kMean256 ? kTile256 : mean >= kMean128 ? kTile128 : mean >= kMean64 ? kTile64 : kTile32;
    else
        form = mean >= kMeanCodes64 ? kTile64 : kTile32;
    const int64_t enough = wide && p.offsets != nullptr ? kEnoughBlocksGrouped : kEnoughBlocks;
    while (form > kTile32 && even_blocks(p, form) < enough) --form;
    return form;
}

}  // namespace
}  // namespace product_detail

using namespace product_detail;

bool product_launchable(const ProductParams &p) {
    const Grid g = form_grid(p, form_of(p));
    return g.blocks * g.threads < (1ll << 32);
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
