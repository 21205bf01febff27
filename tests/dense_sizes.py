"""Sizes that between them take every product kernel of the dense operators:
each tile, wave groups or not, each layout of the operands, each epilogue, rows
on 16 bytes or not, sums in one part or several.  test_dense_host checks that
they do (the rule that chooses may change), test_gpu_dense_tiles runs them."""
import torch

BF, HF, FP = torch.bfloat16, torch.float16, torch.float32

# type, result's type, M, K, N, activation, residual
LINEAR = [
    (BF, FP, 72, 8, 8, 'none', False), (BF, FP, 72, 8, 8, 'silu', False), (BF, BF, 77, 8, 8, 'none', False),
    (HF, HF, 72, 9, 8, 'none', True), (HF, HF, 75, 8, 9, 'none', True), (BF, BF, 85, 8, 8, 'silu', True),
    (BF, BF, 79, 8, 9, 'none', False), (HF, FP, 96, 8, 8, 'gelu', True), (BF, FP, 75, 8, 11, 'gelu', False),
    (BF, FP, 72, 8, 13, 'none', True), (HF, FP, 91, 8, 11, 'silu', True), (BF, FP, 107, 8, 11, 'none', False),
    (HF, HF, 104, 11, 9, 'gelu', True), (BF, FP, 71, 19, 8, 'none', True), (HF, HF, 96, 13, 9, 'silu', False),
    (FP, FP, 72, 79, 8, 'silu', False), (FP, FP, 101, 72, 8, 'none', True), (FP, FP, 71, 104, 8, 'gelu', True),
    (FP, FP, 111, 79, 8, 'none', False), (HF, HF, 69, 563, 8, 'none', True), (BF, BF, 80, 521, 8, 'gelu', True),
    (HF, HF, 75, 608, 8, 'silu', False), (BF, BF, 71, 693, 8, 'none', False), (FP, FP, 72, 3687, 9, 'silu', False),
    (FP, FP, 96, 3200, 9, 'none', True), (FP, FP, 87, 3680, 11, 'silu', True), (BF, BF, 33656, 8, 16, 'none', True),
    (HF, FP, 33617, 21, 8, 'none', True), (BF, FP, 32904, 16, 24, 'gelu', True),
    (HF, FP, 11577, 8, 152, 'none', False), (BF, FP, 32891, 8, 56, 'gelu', False),
    (HF, HF, 11256, 8, 168, 'none', False), (HF, HF, 33057, 8, 72, 'silu', False),
    (BF, BF, 22925, 8, 155, 'none', False), (BF, FP, 18583, 8, 195, 'silu', False),
    (HF, FP, 7360, 8, 535, 'none', False), (HF, HF, 487, 8, 8749, 'silu', False),
    (BF, BF, 32769, 8, 160, 'none', False), (BF, BF, 136, 552, 601, 'none', False),
    (BF, BF, 32803, 199, 8, 'gelu', True), (HF, HF, 17669, 400, 8, 'gelu', False),
    (FP, FP, 21216, 456, 13, 'silu', True), (HF, HF, 12245, 1288, 13, 'none', True),
    (BF, BF, 3080, 4757, 21, 'silu', True), (FP, FP, 23840, 201, 72, 'none', False),
    (BF, BF, 304, 808, 1489, 'silu', False), (BF, FP, 83, 3083, 1601, 'none', False),
    (FP, FP, 25119, 205, 80, 'gelu', False), (FP, FP, 22144, 221, 88, 'none', True),
    (FP, FP, 367, 224, 5488, 'gelu', True), (FP, FP, 9640, 768, 69, 'none', False),
    (FP, FP, 4120, 1807, 69, 'none', True), (FP, FP, 5651, 523, 189, 'gelu', True),
    (HF, FP, 1232, 72, 8447, 'none', True), (FP, FP, 87, 1824, 5539, 'silu', False),
    (HF, FP, 12072, 73, 1000, 'none', False), (FP, FP, 23013, 312, 129, 'gelu', False),
    (FP, FP, 17003, 431, 137, 'gelu', True), (FP, FP, 18184, 537, 152, 'silu', True),
    (FP, FP, 17440, 488, 193, 'none', False), (FP, FP, 1665, 143, 8264, 'none', True),
    (BF, BF, 16792, 1896, 72, 'none', False), (HF, HF, 17968, 1887, 72, 'none', True),
    (BF, BF, 18384, 1567, 88, 'silu', False), (HF, HF, 11157, 79, 3047, 'gelu', True),
    (FP, FP, 8800, 2272, 144, 'gelu', False), (BF, BF, 139, 5791, 3613, 'none', True),
    (HF, HF, 72, 5705, 7265, 'gelu', False), (HF, HF, 5584, 3211, 167, 'none', False),
    (HF, HF, 8112, 5723, 65, 'silu', True), (HF, HF, 1565, 224, 8721, 'none', True),
    (HF, HF, 297, 1920, 8168, 'gelu', True), (FP, FP, 2064, 2045, 1429, 'none', True),
    (HF, HF, 17912, 2616, 153, 'gelu', True), (BF, BF, 17416, 4001, 149, 'none', False),
    (HF, HF, 2072, 1047, 5960, 'none', True), (HF, HF, 2423, 3339, 1675, 'none', True),
    (BF, BF, 17168, 4584, 184, 'gelu', False), (HF, HF, 432, 5507, 8312, 'silu', True),
    (HF, HF, 9225, 5661, 403, 'gelu', False),
]

# type, M, D, F, O
GATED = [
    (BF, 71, 9, 8, 9), (HF, 2880, 8, 9, 8), (HF, 64, 555, 8, 555), (FP, 73, 152, 743, 152), (BF, 2089, 8, 976, 8),
    (HF, 709, 31, 3120, 31), (HF, 5912, 8, 2141, 8), (BF, 3168, 8, 4013, 8), (HF, 112, 3351, 688, 3351),
    (FP, 632, 840, 1639, 840), (HF, 17115, 1965, 40, 1965), (HF, 3631, 1547, 525, 1547),
]

# type, batch, m, n
ORTHOGONALIZE = [
    (BF, 1, 8, 8), (HF, 1, 9, 8), (HF, 1, 8, 9), (FP, 1, 8, 9), (FP, 1, 9, 8), (HF, 1, 11, 9), (BF, 1, 2264, 8),
    (FP, 1, 144, 141), (HF, 1, 136, 864), (HF, 9, 8, 4129), (BF, 1, 659, 653), (BF, 1, 816, 843), (FP, 9, 321, 344),
    (FP, 4, 1881, 257), (HF, 9, 505, 455), (BF, 1, 1033, 2041), (FP, 4, 467, 1168), (BF, 1, 1439, 1576),
    (BF, 1, 1603, 1488), (BF, 9, 587, 464), (HF, 9, 129, 3040), (FP, 1, 2384, 1689), (BF, 9, 675, 664),
    (FP, 1, 1688, 2413), (BF, 9, 645, 709), (HF, 1, 2523, 1648), (FP, 1, 2007, 2112), (BF, 1, 2096, 2048),
    (HF, 1, 2415, 1795), (HF, 1, 1773, 2447), (HF, 1, 1679, 2624), (FP, 9, 657, 773), (FP, 1, 2224, 2104),
    (BF, 9, 703, 777), (BF, 4, 1168, 1149), (FP, 9, 4568, 135), (FP, 9, 133, 5243), (HF, 9, 5320, 136),
    (FP, 9, 141, 5344), (FP, 9, 6025, 136), (FP, 4, 1317, 1456), (HF, 9, 135, 6683), (HF, 9, 4576, 209),
    (BF, 9, 4384, 221), (FP, 9, 1088, 928), (BF, 9, 699, 1664), (HF, 4, 2016, 1344), (BF, 2, 1009, 5495),
    (HF, 9, 457, 2992), (BF, 2, 3943, 1624), (FP, 4, 3479, 1304), (BF, 4, 2296, 2032), (FP, 4, 1287, 3913),
    (BF, 9, 1589, 1632), (BF, 9, 1800, 1755), (BF, 4, 1949, 3721),
]
