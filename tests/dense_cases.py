"""Sizes that together reach every kernel of the dense matrix operators: each
tile in each product (forward, dx, dw), whole and with its contraction split, the
float32 tiles with whole and with ragged groups of four, the 64-row bf16 tile's
short ring, and the weight-streaming kernel of every height.  test_dense_cpu.py
holds them to that, so a change of the choice shows there."""
import re

import bitwise_deterministic_moe_amd as moe

# (dtype, rows, d_in, d_out)
CASES = [
    ("bf16", 1, 1, 1), ("bf16", 3, 3425, 1), ("bf16", 17, 3, 1224), ("bf16", 21, 3399, 1), ("bf16", 35, 1, 1),
    ("bf16", 47, 5891, 1), ("bf16", 53, 1, 1), ("bf16", 55, 3893, 1), ("bf16", 86, 8495, 6035), ("bf16", 136, 5, 139),
    ("bf16", 135, 8539, 5057), ("bf16", 156, 8519, 3148), ("bf16", 199, 8216, 80), ("bf16", 277, 1168, 7936),
    ("bf16", 341, 840, 3248), ("bf16", 588, 7548, 629), ("bf16", 4383, 208, 1784), ("bf16", 5490, 6680, 184),
    ("bf16", 5649, 4656, 136), ("bf16", 6352, 8328, 136), ("bf16", 6519, 130, 6696), ("bf16", 6771, 147, 5940),
    ("bf16", 7320, 1698, 1), ("bf16", 8602, 5720, 136),
    ("f32", 1, 1, 1), ("f32", 1, 3405, 1), ("f32", 17, 2258, 1), ("f32", 32, 4, 4), ("f32", 37, 168, 1), ("f32", 58, 196, 4),
    ("f32", 212, 706, 4649), ("f32", 261, 8, 216), ("f32", 277, 1, 211), ("f32", 594, 1826, 639), ("f32", 725, 480, 4192),
    ("f32", 734, 656, 1520), ("f32", 2582, 1160, 216), ("f32", 6209, 580, 242), ("f32", 6658, 175, 454),
]


def kernels(dtype, rows, d, f):
    """The product kernels of one case's calls, without the numbers of chunks."""
    found = set()
    for kind, names in (("linear", moe.moe_linear_stage_names), ("glu", moe.moe_glu_stage_names)):
        for call in (0, 1):
            for n in names(rows, d, f, call, dtype, "relu"):
                if "_" in n and not n.endswith("copy"):
                    found.add((kind, dtype, re.sub(r"_split\d+", "_split", n)))
    return found


def every_kernel():
    want = set()
    for kind in ("linear", "glu"):
        for split in ("", "_split"):
            for product in (kind, "dx", "dw"):
                for tile in ("256x256", "128x256", "128x128", "64x64"):
                    want.add((kind, "bf16", f"{product}_{tile}{split}"))
                for tile in ("128x128_parts", "64x64_f32"):
                    for odd in ("", "_odd"):
                        want.add((kind, "f32", f"{product}_{tile}{odd}{split}"))
            for rows in (16, 32, 48, 64):
                want.add((kind, "bf16", f"{kind}_few{rows}{split}"))
            for rows in (16, 32):
                want.add((kind, "f32", f"{kind}_few{rows}{split}"))
        for product in (kind, "dx", "dw"):
            want.add((kind, "bf16", f"{product}_64x64_short"))
    return want
