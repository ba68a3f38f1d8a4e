"""Sizes that together reach every kernel of the products in 8-bit integers: the weight
stream with one wave and with four on a contraction, quantising x itself and not, each
tile, and the split contraction in every number of chunks, most with slices that the
chunks do not share evenly and a last one that is not full.  test_int8_cpu.py holds
them to that, so a change of the choice shows there."""
import bitwise_deterministic_moe_amd as moe

# (kernel, type, rows, d_in, d_out, activation)
LINEAR = [
    ("few4_quantize", "bf16", 4, 6759, 130, "silu"), ("few4_quantize", "f32", 3, 8000, 77, "none"),
    ("few4", "bf16", 13, 11727, 1069, "silu"), ("few4", "f32", 9, 3001, 333, "gelu"),
    ("few1_quantize", "bf16", 1, 1000, 33001, "none"), ("few1_quantize", "f32", 4, 1555, 32801, "silu"),
    ("few1", "bf16", 9, 1000, 33001, "silu"), ("few1", "f32", 16, 700, 32753, "none"),
    ("256x256", "bf16", 4096, 2048, 8192, "gelu"), ("256x256", "bf16", 4076, 1999, 8010, "silu"),
    ("256x256", "f32", 4000, 1999, 8190, "gelu"), ("256x256", "f32", 2623, 1312, 5677, "none"),
    ("128x128", "bf16", 1716, 632, 5767, "silu"), ("128x128", "f32", 1508, 557, 7110, "none"),
    ("128x64", "bf16", 220, 698, 29857, "silu"), ("128x64", "f32", 240, 1108, 28283, "none"),
    ("128x64_deep", "bf16", 106, 4080, 19765, "silu"), ("128x64_deep", "f32", 1114, 1553, 4176, "none"),
    ("64x64", "bf16", 3950, 576, 962, "silu"), ("64x64", "f32", 2089, 130, 5902, "none"),
    ("64x64_deep", "bf16", 591, 1626, 115, "silu"), ("64x64_deep", "f32", 27, 300, 176, "gelu"),
    ("64x64_deep_split2", "bf16", 110, 7513, 5499, "silu"), ("64x64_deep_split2", "f32", 1010, 10500, 761, "none"),
    ("64x64_deep_split4", "bf16", 95, 3866, 177, "none"), ("64x64_deep_split4", "f32", 407, 10808, 624, "silu"),
    ("64x64_deep_split8", "bf16", 617, 12453, 186, "gelu"), ("64x64_deep_split8", "f32", 82, 9498, 1505, "none"),
]
# (kernel, type, rows of each expert (cycled), experts, d_in, d_out, rows behind the last, activation)
EXPERTS = [
    ("few4_quantize", "bf16", [1, 0, 2], 31, 114, 40, 3, "silu"), ("few4_quantize", "f32", [1], 3, 2040, 300, 0, "relu2"),
    ("few4", "bf16", [0, 1], 60, 13616, 33, 1, "silu"), ("few4", "f32", [1, 4, 0], 5, 4144, 65, 2, "none"),
    ("few1_quantize", "bf16", [1], 22, 2048, 2048, 0, "relu2"), ("few1_quantize", "f32", [1, 0, 3], 300, 1000, 200, 1, "silu"),
    ("few1", "bf16", [1, 0, 3], 40, 2100, 999, 2, "silu"), ("few1", "f32", [2], 9, 3333, 2000, 0, "none"),
    ("256x256", "bf16", [2950, 1091], 2, 1075, 3812, 9, "silu"), ("256x256", "f32", [4413], 1, 1730, 2963, 2, "none"),
    ("128x128", "bf16", [1500, 1, 1579], 3, 2115, 2151, 3, "silu"), ("128x128", "f32", [900, 0, 930, 2], 8, 704, 2025, 3, "none"),
    ("128x64", "bf16", [5090], 1, 853, 1089, 7, "none"), ("128x64", "f32", [379], 1, 864, 15038, 1, "silu"),
    ("128x64_deep", "bf16", [3000, 2040], 2, 1581, 661, 8, "silu"), ("128x64_deep", "f32", [1100], 1, 1553, 4176, 14, "none"),
    ("64x64", "bf16", [5, 0, 17], 236, 27, 678, 2, "silu"), ("64x64", "f32", [500, 365], 2, 70, 7478, 0, "none"),
    ("64x64_deep", "bf16", [300, 70, 1, 0], 18, 1536, 70, 4, "silu"), ("64x64_deep", "f32", [20], 4, 2251, 81, 3, "none"),
]
TILES = ("256x256", "128x128", "128x64_deep", "128x64", "64x64", "64x64_deep")
FEW = ("few4_quantize", "few4", "few1_quantize", "few1")
SPLITS = ("64x64_deep_split2", "64x64_deep_split4", "64x64_deep_split8")


def product(names):
    """The product kernel of a call's names."""
    return next(n for n in names if n not in ("quantize", "join"))


def counts(cycle, experts):
    return [cycle[e % len(cycle)] for e in range(experts)]


def linear_kernel(dtype, rows, k, f, act):
    return product(moe.moe_int8_stage_names(rows, k, f, 0, dtype, act))


def experts_kernel(dtype, cycle, experts, k, f, behind, act):
    return product(moe.moe_int8_stage_names(sum(counts(cycle, experts)) + behind, k, f, experts, dtype, act))
