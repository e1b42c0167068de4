"""Sizes for each kernel behind the MX products, with the kernel and the parts of K that they are for.  A CPU test
holds the launcher to them at a B200's 148 SMs, so the GPU tests that use them keep reaching that kernel."""

SMS = 148

# M, N, K, n_out, act, residual, (kernel, parts)
LINEAR = [
    (128, 264, 7456, 1, "none", True, ("few", 4)),
    (385, 1032, 4128, 1, "silu", True, ("few", 2)),
    (300, 2056, 4128, 1, "gelu_tanh", False, ("few", 2)),
    (3000, 2056, 512, 1, "none", True, ("pairs", 1)),           # a segment that ends inside a box
    (5000, 2056, 1056, 1, "none", True, ("pairs", 1)),          # several tiles a pair; ragged M, N and K
    (5000, 2056, 1056, 1, "gelu_tanh", True, ("pairs", 1)),
    (4700, 4104, 96, 1, "none", True, ("pairs", 1)),            # one step of K, of three blocks
    (2600, 4104, 1184, 1, "none", False, ("pairs", 1)),
    (4200, 3 * 1032, 1312, 3, "silu", False, ("pairs", 1)),
    (5000, 4 * 520, 1056, 4, "none", False, ("pairs", 1)),
    (512, 4096, 3104, 1, "none", True, ("pairs_split", 2)),
    (700, 2056, 3104, 1, "none", True, ("pairs_split", 2)),     # ragged M, N and K
    (257, 4040, 4096, 1, "gelu_tanh", True, ("pairs_split", 2)),  # a CTA without a row
    (300, 3976, 4096, 1, "silu", False, ("pairs_split", 2)),    # columns that do not exist
    (300, 3 * 1032, 4128, 3, "none", False, ("pairs_split", 2)),
]

# M, F, K, (kernel, parts)
GATED = [
    (16, 256, 4096, ("few", 4)),
    (300, 256, 160, ("pairs", 1)),
    (900, 1152, 1056, ("pairs", 1)),
    (2500, 3200, 512, ("pairs", 1)),       # several tiles a pair
    (300, 2048, 4096, ("pairs_split", 2)),
    (700, 1152, 3104, ("pairs_split", 2)),
]
