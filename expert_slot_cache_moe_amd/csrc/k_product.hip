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
// 256 blocks of k 2048 6.2 / 12.0, 512 10.3 / 14.4, 1024 18.7 / 14.6; 512 of k
// 4096 17.8 / 25.3, 1024 33.2 / 26.2; 1024 of k 1024 11.6 / 10.3, 2048 21.1 /
// 12.2).  With rows of x that are no whole vectors of eight only one for each
// CU (k 203, 256 blocks 4.6 / 5.4, 320 7.0 / 5.4; k 1061, 192 and 256 8.4 /
// 9.8, 320 14.6 / 9.8; k 2051, 256 12.5 / 15.4, 320 22.7 / 15.3; grouped, 515
// columns of k 1061, 198 8.9 / 12.7, 264 13.8 / 12.7), with 4-bit weights
// more (E2M1 and MXFP4, k 1024, 768 blocks 7.4 / 9.2 and 7.3 / 8.4, 832 8.6 /
// 9.1 and 8.5 / 8.4; k 2048, 768 11.7 / 15.2 and 11.4 / 13.3, 832 14.1 / 15.0
// and 13.9 / 13.4; k 1024, 1280 10.6 / 9.3 and 10.3 / 8.4).
constexpr int64_t kSplitBlocks = 512, kSplitBlocksCut = 256, kSplitBlocksCodes = 800;
// The mean places of a matrix from which a tile of 64, 128, 256 places pays
// (bf16, 64 matrices of 2048 x 2048, us at 32 / 64 / 128 / 256 places: mean 8
// 96 96 95 132, 16 103 97 96 128, 48 156 107 115 134, 64 195 117 116 136, 96
// 261 153 126 187, 192 444 253 176 197, 256 578 326 224 201; 160 of 512 x
// 1024: mean 8 27 28 34 64, 16 29 30 34 64, 64 64 40 41 66, 96 80 55 44 67,
// 256 161 110 82 79; between 6 and 24 places 32 and 64 are within 4 % of each
// other where the groups are alike, and 64 is up to 15 % faster where some are
// longer: popular rows, 96 of 1024 x 2048, mean 8 83 72, 12 84 74, 16 84 84),
// and for 4 bits one of 64 (E2M1, 64 of 2048 x 2048, 32 / 64 places: mean 32
// 52 60, 48 67 63, 96 117 98).
constexpr int64_t kMean64 = 12, kMean128 = 72, kMean256 = 224, kMeanCodes64 = 40;
// A larger tile is taken only where there is a block for each of the 256 CUs
// (dense 4096 x 4096, us at 64 / 128 / 256 places: 512 rows 41 41 92, 1024 56
// 44 98, 2048 139 76 97, 4096 281 151 120), or for half of them where each
// piece more reads a matrix of its own again (32 / 64 places, 128 and 132
// blocks of 64: 8 matrices of 1024 x 2048 22.4 / 17.6, 33 of 138 x 2656 22.1 /
// 23.3; a dense 1024 x 1024 of 128 blocks 8.1 / 9.3; MXFP4, 24 of 515 x 1056,
// 240 blocks 13.3 / 13.4).
constexpr int64_t kEnoughBlocks = 256, kEnoughBlocksGrouped = 120;

int form_of(const ProductParams &p) {
    const bool wide = p.fmt == MOE_FMT_BF16;
    if (p.n / (p.act == MOE_ACT_SWIGLU ? 2 : 1) < kTileMinCols) return kSplit;
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
