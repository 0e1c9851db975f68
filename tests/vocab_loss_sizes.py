"""Sizes of the vocabulary loss, with the way each is cut that it stands for.  The choice of tiles is an
estimate that may be fitted again: a test of the plans on the host says when a size here no longer
reaches the kernels that it is here for."""

# T, d, V, dtype, and of the plan: tiles of the backward's logits, dh and dw, several pieces of the
# vocabulary, dh's sum split, dw's sum split.
PLANS = [
    # 256x256 tiles: one piece; dw unsplit and split; ragged pieces whose dh is accumulated
    (13640, 976, 1547, "bf16", 256, 256, 256, False, False, True),
    (70, 224, 119576, "bf16", 256, 256, 256, False, True, False),
    (3624, 400, 13635, "bf16", 256, 256, 256, False, True, True),
    (6496, 432, 15782, "bf16", 256, 256, 256, True, True, True),
    (841, 136, 88516, "bf16", 256, 256, 256, True, True, False),
    (6796, 2208, 10388, "bf16", 256, 256, 256, True, False, False),
    # and whole tiles and K steps only (T and the words multiples of 256, d of 256)
    (2048, 512, 40960, "bf16", 256, 256, 256, True, True, False),
    (8192, 512, 16384, "bf16", 256, 256, 256, True, True, True),
    (4096, 4096, 16384 + 256, "bf16", 256, 256, 256, True, False, False),
    # dh and dw in tiles of different sizes
    (3269, 1208, 21054, "bf16", 256, 128, 256, True, False, False),
    (8989, 392, 10470, "bf16", 256, 128, 256, True, False, True),
    (10395, 144, 6145, "bf16", 256, 256, 128, False, True, True),
    (16251, 160, 6051, "bf16", 256, 256, 128, True, True, True),
    (495, 176, 141576, "bf16", 256, 256, 64, True, True, False),
    (83, 3288, 13325, "bf16", 64, 128, 256, False, True, False),
    (82, 224, 62803, "bf16", 256, 64, 256, False, True, False),
    (65, 3568, 8053, "bf16", 64, 256, 256, False, True, False),
    # several pieces in the smaller tiles
    (1284, 8, 53240, "bf16", 256, 64, 64, True, True, False),
    (357, 72, 195420, "bf16", 256, 128, 128, True, True, False),
    (815, 72, 115738, "f32", 64, 128, 128, True, True, False),
    (1391, 24, 90023, "f32", 128, 64, 64, True, True, False),
    (1162, 8, 59540, "f32", 64, 64, 64, True, True, False),
    (4827, 80, 15695, "f32", 128, 128, 128, True, True, True),
]

# T, d, V, dtype and the forward's tiles.  The last two: at most 64 tokens against 128 MB of words, read
# past the caches.
FORWARD = [(40, 64, 1000, "bf16", 64), (40, 64, 1000, "f32", 64), (200, 72, 700, "bf16", 64), (1010, 1000, 3990, "bf16", 128),
           (1990, 512, 3990, "f32", 128), (700, 200, 16421, "bf16", 256), (7, 2048, 33001, "bf16", 64), (50, 2048, 16421, "f32", 64)]
