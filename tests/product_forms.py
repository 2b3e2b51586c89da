"""Which form a product takes, by the rule and the constants of
csrc/k_product.hip, so that a test can say which kernel it means to reach."""
import os
import re

SPLIT, TILE32, TILE64, TILE128, TILE256 = range(5)
NAMES = ("split", "tile32", "tile64", "tile128", "tile256")

_CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "expert_slot_cache_moe_amd", "csrc")


def constants():
    out = {}
    for name in ("k_product.hip", "k_product.inc"):
        with open(os.path.join(_CSRC, name)) as f:
            for line in re.findall(r"constexpr (?:int64_t|int) ([^;]*);", f.read()):
                out.update((k, int(v)) for k, v in re.findall(r"(k\w+) = (\d+)(?=,|$)", line))
    return out


def form_of(fmt, n, k, R, groups=None, swiglu=False, x_stride=None):
    """groups None: a dense product."""
    c = constants()
    wide, dense = fmt == "bf16", groups is None
    if n // (2 if swiglu else 1) < c["kTileMinCols"]:
        return SPLIT
    g = 1 if dense else min(groups, R)

    def blocks(form):
        places = 16 << form
        rows = (32 if swiglu else 16) if form == SPLIT else 256 if form == TILE256 else 128
        return g * -(-R // (g * places)) * -(-n // rows)

    cut = k % 8 != 0 or (k if x_stride is None else x_stride) % 8 != 0
    if blocks(SPLIT) <= (c["kSplitBlocksCodes"] if not wide else c["kSplitBlocksCut"] if cut else c["kSplitBlocks"]):
        return SPLIT
    mean = R // g
    if wide:
        form = TILE32 + sum(mean >= c[m] for m in ("kMean64", "kMean128", "kMean256"))
    else:
        form = TILE64 if mean >= c["kMeanCodes64"] else TILE32
    enough = c["kEnoughBlocksGrouped" if wide and not dense else "kEnoughBlocks"]
    while form > TILE32 and blocks(form) < enough:
        form -= 1
    return form
