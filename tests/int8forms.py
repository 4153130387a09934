"""Sizes that the 8-bit product's tests share: for each kernel, some where its ring of buffers goes round."""

import numpy as np

# kernel -> columns a stage, buffers (k_int8_tile.hip); of the kernel without LDS, what four waves take at a time and
# the chunks that a wave has on their way
PIPELINES = {"256x256": (64, 4), "256x128": (128, 3), "128x64": (128, 3), "64x128": (128, 2), "64x64": (256, 3),
             "32x32": (256, 4), "32x16": (256, 4), "rows": (512, 3)}

# (tokens, rows, cols) -> kernel: odd sizes with a last stage of a few columns, and whole ones
LONG = {
    (4001, 4090, 1156): "256x256", (3841, 3903, 1092): "256x256", (4090, 4093, 1284): "256x256", (4096, 4096, 1280): "256x256",
    (1531, 4099, 4100): "256x128", (2003, 4091, 1412): "256x128", (2048, 4096, 2048): "256x128",
    (499, 4099, 2052): "128x64", (990, 4001, 1412): "128x64", (512, 4096, 4096): "128x64",
    (777, 5001, 2052): "64x128", (770, 5003, 908): "64x128",
    (253, 4095, 4100): "64x64", (999, 1001, 2820): "64x64", (256, 4096, 4096): "64x64",
    (61, 4099, 11012): "32x32", (127, 2051, 4356): "32x32", (64, 4096, 4096): "32x32",
    (21, 3001, 5004): "32x16", (9, 11007, 3844): "32x16", (32, 2048, 4096): "32x16",
    (7, 4097, 11012): "rows", (16, 8191, 2052): "rows", (1, 4096, 4096): "rows",
}


def random_size(seed):
    """Tokens, rows and columns over the whole range of a layer's calls, up to 2^34 products."""
    rng = np.random.default_rng(5000 + seed)
    while True:
        tokens, rows, words = (int(np.exp(rng.uniform(np.log(lo), np.log(hi))))
                               for lo, hi in ((2, 6000), (400, 12000), (100, 2800)))
        if 2 ** 26 <= tokens * rows * 4 * words <= 2 ** 34:
            return tokens, rows, 4 * words
